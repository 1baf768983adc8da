// attn_fp4.cu -- attention over every visible row of a 4-bit cache, and the attention each row received.
//
// For query (b, t), vis = clamp((start_pos + t + 1) // ratio - dropped, 0, n_rows) rows are visible:
//   s_hj = softmax_scale q_h . k_j,  L_h = ln(sum_j e^{s_hj} + e^{sink_h} + e^{prev_lse_h})
//   out_h = (sum_j e^{s_hj} k_j + e^{prev_lse_h} prev_out_h) / e^{L_h}
//   row_weight[b, j] += sum_{t, h} e^{s_hj - L_h}
// k_j = the row's E2M1 codes times its E4M3 scale per 16, serving as key and value for all heads.
//
// attn_fp4_kernel: persistent CTAs, one per SM; the queries' 64-row tiles form one long list that is cut
// into equal contiguous pieces, so a few long queries, many short ones and ragged batches all fill
// the GPU.  A query whose tiles fall to several CTAs leaves one fp32 partial per CTA; merge_kernel joins
// them.  Two tile buffers; 19 working warps:
//   * warps 8..15 decode the rows into the free buffer, from codes loaded a tile ahead, one half (256 dims)
//     at a time as the PV two tiles earlier releases it;
//   * warp 16 issues the QKs, S^T = tile . Q^T (M = 64 rows, N = heads), warp 17 the PVs, O^T += V^T . P^T (M = 128
//     dims per block, K = 64 rows; the same tile read as an MN-major operand);
//   * warp 18 asks for the rows of the next tiles, into L2;
//   * warps 0..7 load Q, run the online softmax (two sets of 32 heads; what P is relative to moves only when a
//     score passes the largest so far by 2^8) and write the outputs.
// With 512 dims, Q (64 KB), two tiles of 64 rows (128 KB) and two P^T (16 KB) fill shared memory.  One tile of
// 128 rows instead would take a quarter off the QK (48 cycles a step for M = 128, 32 for M = 64), but leaves
// decode, QK, softmax and PV of a tile to run one after another: 8,400 cycles per 128 rows.
// Bound by shared memory: of a tile at 128 B a cycle, QK 1024 cycles, PV 768, the decoded stores 512 and P^T, together
// 2430 of the 2800 that a tile takes.  (The QK's 1024 are the tensor core's too, which takes N / 2 cycles for
// M = 64, half its rate: fewer operand bytes alone would not shorten it.  Steps of M = 64 measured 25, 32 and 64 cycles for
// N = 32, 64 and 128, of M = 128 48 for N = 64.)  2048 queries over up to 2048 rows: 701 us, 18,000 of a query's 100,000 cycles
// for its Q and outputs; one query each over 32 x 16384 rows: 95 us (20 of them set-up, change of query and partial
// outputs), and the merge 12.  QK and PV issued by one warp in turn took 832 and 112 us, outputs scaled by shuffles 765.
//
// f16 operands: an E2M1 value (2 significant bits) times an E4M3 value (4) is exact in f16 (at most 6
// significant bits, magnitudes 2^-10 .. 2688), so the tile is exact.  Q is bf16: each head's values are
// scaled by a power of two that puts its largest into [2^12, 2^13) and is undone in fp32 with the
// softmax scale; an element down to 2^-26 of the head's largest keeps all its 8 bits, smaller ones are
// off by less than 2^-37 of the largest.  P is rounded to f16 for the PV product; its sum l is taken before the
// rounding, in fp32.  P is held at 2^7 .. 2^15 for the row of the largest score, not at 1: f16 keeps 11 bits down to 2^-14
// and steps of 2^-24 below, so a row's probability is off by 2^-11 of itself or, if that is more, by 2^-32 of the
// largest's (2^-25 with the largest at 1: rows 17.5 below the largest score were lost to the output, and 2^20 of
// them 19 below are 0.6 % of it).
//
// Row weights (only when asked for): p = e^{s - L} needs the final L, so they come after the merge.  A few queries a
// sequence (decoding, drafts) leave their scores in the workspace, 4 bytes each, and row_weight_scores_kernel sums
// them; row_weight_kernel computes S^T again from the codes.  Each row tile belongs to one CTA, which adds the queries
// in order: no atomics.  With many queries row_weight_kernel's CTAs split over them and a last kernel adds the parts.
#include <cuda_fp16.h>
#include <math.h>
#include <stddef.h>

#include "sti_attn_util.cuh"
#include "sti_internal.h"
#include "sti_ptx.cuh"

namespace sti {
namespace {

constexpr int kThreads = 640;                  // 8 softmax warps, 8 decoding warps, 2 MMA warps, 1 that
                                               // prefetches (and 1 that only completes its warpgroup)
// registers per thread after setmaxnreg: 256 x 128 + 256 x 80 + 128 x 64 = 61,440, the 640 x 96 of the launch
constexpr int kRegsSoft = 128, kRegsDecode = 80, kRegsMma = 64;
constexpr int kRows = 64;                      // rows per tile
constexpr uint32_t kQBlk = 64 * 128;           // a Q column block: 64 heads x 64 dims
constexpr uint32_t kTBlk = kRows * 128;        // a tile column block: 64 rows x 64 dims
constexpr uint32_t kPBuf = kRows * 128;        // a P^T buffer: 64 rows x 64 heads
constexpr uint32_t kTmO = 128;                 // TMEM: S^T of tile parity b at columns [64 b, 64 b + 64), O^T d-block
                                               // m at [128 + 64 m, 192 + 64 m)
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.69314718055994531f;
constexpr float kTopNew = 7.f, kTopMost = 15.f;   // log2 of the largest P: when a head's reference is set, and at
                                                  // most (f16 ends below 2^16)
constexpr int kAhead = 3;                      // tiles whose rows are asked for ahead
constexpr int kWTiles = 32;                    // row weights: tiles per chunk (accumulators in shared memory)
constexpr int kScoreQueries = 8;               // row weights from kept scores: at most this many query groups a sequence,
constexpr int kScoreTiles = 16384;             // and this many tiles of scores (256 MB)
constexpr int kManyTiles = 4096;               // row weights from scores: from here on a block takes four tiles
constexpr uint32_t kBarSoft = 3;               // named barriers: 1, 2 the head groups, 3 all softmax warps

// instruction descriptor, kind::f16 with f16 A/B (format 0) and fp32 accumulator
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N, bool a_mn_major, bool b_mn_major) {
    return (1u << 4) | ((a_mn_major ? 1u : 0u) << 15) | ((b_mn_major ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) |
           ((uint32_t)(M >> 4) << 24);
}

// umma_bf16's instruction with the descriptors as (low, high) words, so that stepping through an operand is
// one 32-bit add: the issuing thread is alone, and every instruction between two MMAs delays the second.
template <bool ACC>
__device__ __forceinline__ void umma(uint32_t d_tmem, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo, uint32_t b_hi,
                                     uint32_t idesc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "mov.b64 a, {%1, %2};\n\t"
        "mov.b64 b, {%3, %4};\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, p;\n\t}" ::"r"(d_tmem),
        "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "n"(ACC ? 1 : 0)
        : "memory");
}
__device__ __forceinline__ uint32_t lo32(uint64_t v) { return (uint32_t)v; }
__device__ __forceinline__ uint32_t hi32(uint64_t v) { return (uint32_t)(v >> 32); }

// Keep the value from being combined with constants ahead of time: the descriptors of a tile's 64 MMAs, all
// known before the loop, would otherwise be kept (and spilled) as 64 values instead of one and an add each.
__device__ __forceinline__ uint32_t opaque(uint32_t v) {
    asm volatile("" : "+r"(v));
    return v;
}
// S^T (+)= tile . Q^T over d-block m (two column blocks).  a, b: low descriptor words of the tile and Q.
__device__ __forceinline__ void qk_blocks(int m, uint32_t s_tmem, uint32_t a, uint32_t b, uint32_t hi, uint32_t idesc) {
    a = opaque(a);
    b = opaque(b);
#pragma unroll
    for (int k = 8 * m; k < 8 * m + 8; ++k) {
        const uint32_t ak = a + (k >> 2) * (kTBlk / 16) + 2 * (k & 3), bk = b + (k >> 2) * (kQBlk / 16) + 2 * (k & 3);
        if (k == 0) umma<false>(s_tmem, ak, hi, bk, hi, idesc);
        else umma<true>(s_tmem, ak, hi, bk, hi, idesc);
    }
}
// O^T (+)= V^T . P^T: one d-block, four K steps.
template <bool FIRST>
__device__ __forceinline__ void pv_block(uint32_t o_tmem, uint32_t a, uint32_t a_hi, uint32_t b, uint32_t b_hi,
                                         uint32_t idesc) {
    a = opaque(a);
    b = opaque(b);
#pragma unroll
    for (int k = 0; k < kRows / 16; ++k) {
        if (FIRST && k == 0) umma<false>(o_tmem, a, a_hi, b, b_hi, idesc);
        else umma<true>(o_tmem, a + 128 * k, a_hi, b + 128 * k, b_hi, idesc);
    }
}
// S^T of 16 rows (a warp's TMEM lanes 0..15: M = 64 accumulators lie there) x 32 heads: lane l receives, for
// g < 4, heads 8 g + 2 (l % 4) + {0, 1} of row l / 4 in r[4 g], r[4 g + 1] and of row l / 4 + 8 in r[4 g + 2], r[4 g + 3].
__device__ __forceinline__ void tmem_ld_rows16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

template <int N>
__device__ __forceinline__ void regs_up() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_down() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// Bounded wait, as attn_wait, for waits that come several times per tile: reading the global timer takes
// about 200 ns, so it is read only every 256th failed poll (a failed try_wait has already slept a while).
// A wait by parity passes at once when the phase before the awaited one is still open, so every waiter here comes after
// that phase: most wait for a barrier's phases in order; those that wait for freed[.] of some tile n alone
// have seen S^T of n, whose tile was decoded after freed[.] of n - 2.
__device__ __forceinline__ bool tile_wait(uint64_t* bar, uint32_t parity, uint32_t* status, volatile int* abort) {
    uint64_t t0 = 0;
    for (uint32_t i = 1;; ++i) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((i & 255u) == 0u) {
            if (*abort) return false;
            const uint64_t now = global_timer_ns();
            if (t0 == 0) t0 = now;
            else if (now - t0 > STI_WAIT_TIMEOUT_NS) {
                if (status) atomicOr(status, 2u /* STI_FLAG_TIMEOUT */);
                *abort = 1;
                return false;
            }
        }
    }
}

// tile_wait for a converged warp.  The vote makes the result visibly warp-uniform; without it the compiler
// treats what follows as divergent, and the MMAs of the issuing warp take three times as long to issue.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, uint32_t* status, volatile int* abort) {
    return __all_sync(kWarpFull, tile_wait(bar, parity, status, abort));
}

// One lane of the (converged) warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

// ------------------------------------------------------------------ the list of tiles

__device__ __forceinline__ int visible_rows(const AttnFp4Params& p, int b, int t) {
    // start_pos >= 0 and t < 2^30: the sum fits 32 unsigned bits (a 64-bit division takes some hundred cycles)
    const uint32_t groups = ((uint32_t)__ldg(p.start_pos + b) + (uint32_t)t + 1u) / (uint32_t)p.ratio;
    const int64_t v = (int64_t)groups - (p.dropped ? __ldg(p.dropped + b) : 0);
    return v < 0 ? 0 : v > p.n_rows ? p.n_rows : (int)v;
}

// Query groups: `pack` consecutive queries of a sequence whose heads together fill the 64 rows of Q (pack = 1: one
// query).  In memory they are one query of pack * h heads, each head with its own number of visible rows.
struct Group {
    int b, t0, heads;
    int64_t row0;       // of q, out, prev_out, lse, prev_lse: their first head
};
__device__ __forceinline__ Group group_of(const AttnFp4Params& p, int u) {
    Group g;
    g.b = u / p.groups;
    g.t0 = (u - g.b * p.groups) * p.pack;
    g.heads = min(p.pack, p.s - g.t0) * p.h;
    g.row0 = ((int64_t)g.b * p.s + g.t0) * p.h;
    return g;
}
// rows that the last query of group u (of sequence b) sees
__device__ __forceinline__ int group_rows(const AttnFp4Params& p, int b, int u) {
    return visible_rows(p, b, min((u + 1) * p.pack, p.s) - 1);
}
// rows that head hd of the group sees
__device__ __forceinline__ int head_rows(const AttnFp4Params& p, const Group& g, int hd) {
    return hd < g.heads ? visible_rows(p, g.b, g.t0 + hd / p.h) : 0;
}

struct Work {           // this CTA's piece of the list
    long long lo, hi;   // tiles [lo, hi) of the list
    int q, off;         // the first one: tile `off` of query group q
    long long total;
    int ctas;           // CTAs that have tiles
};

struct Seg {            // a run of one group's tiles
    int q, b, vis, nt, t0, t1;
};

// Walk the piece: group by group, those without a visible row skipped.
struct Walk {
    long long pos, hi;
    int q, off;
    __device__ __forceinline__ explicit Walk(const Work& w) : pos(w.lo), hi(w.hi), q(w.q), off(w.off) {}
    __device__ __forceinline__ bool next(const AttnFp4Params& p, Seg& s) {
        while (pos < hi) {
            s.q = q;
            s.b = q / p.groups;
            s.vis = group_rows(p, s.b, q - s.b * p.groups);
            s.nt = (s.vis + kRows - 1) / kRows;
            s.t0 = off;
            s.t1 = (long long)(s.nt - off) < hi - pos ? s.nt : off + (int)(hi - pos);
            off = 0;
            ++q;
            if (s.nt > 0) {
                pos += s.t1 - s.t0;
                return true;
            }
        }
        return false;
    }
};

// Cut the list of `n` items (item i has tiles(i) tiles) into `parts` equal pieces; this CTA takes piece
// `part`.  Every thread of the block calls it.
template <class F>
__device__ __forceinline__ void plan_work(int n, int part, int parts, long long* scratch, Work* w, F tiles) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (n + kThreads - 1) / kThreads;
    const long long i0 = (long long)tid * per;
    long long sum = 0;
    for (int k = 0; k < per && i0 + k < n; ++k) sum += tiles((int)(i0 + k));
    long long inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(kWarpFull, inc, o);
        if (lane >= o) inc += u;
    }
    if (lane == 31) scratch[warp] = inc;
    __syncthreads();
    long long before = 0, total = 0;
    for (int k = 0; k < kThreads / 32; ++k) {
        if (k < warp) before += scratch[k];
        total += scratch[k];
    }
    const long long first = before + inc - sum;
    const int ctas = total < parts ? (int)total : parts;
    long long lo = 0, hi = 0;
    if (part < ctas) {
        lo = (long long)part * total / ctas;
        hi = (long long)(part + 1) * total / ctas;
    }
    if (tid == 0) {
        w->lo = lo;
        w->hi = hi;
        w->total = total;
        w->ctas = ctas;
        w->q = w->off = 0;
    }
    __syncthreads();
    if (lo < hi && first <= lo && lo < first + sum) {
        long long at = first;
        int i = (int)i0;
        for (;; ++i) {
            const int c = tiles(i);
            if (at + c > lo) break;
            at += c;
        }
        w->q = i;
        w->off = (int)(lo - at);
    }
    __syncthreads();
}

// ------------------------------------------------------------------ operands

// Decoding: a warp takes 8 rows of a tile, a lane 32 codes (16 bytes, 2 scales) of one row in every d-block:
// lane = 4 (row % 8) + quarter of the d-block, so that a warp's load covers 64 contiguous bytes of 8 rows (one
// row per lane would touch 32 cache lines per load) and its stores spread over all banks.
template <int NM>
struct Codes {
    uint4 c[NM];
    uint16_t s[NM];
};

template <int NM>
__device__ __forceinline__ void load_codes(const AttnFp4Params& p, int b, int row0, int vis, int n_cb, Codes<NM>& r) {
    const int lane = threadIdx.x & 31, ch = lane & 3;
    const int row = row0 + ((threadIdx.x >> 5) & 7) * 8 + (lane >> 2);
    if (row >= vis) return;
    const uint8_t* cr = p.codes + (int64_t)b * p.codes_bstride + (int64_t)row * (p.d / 2) + ch * 16;
    const uint8_t* sr = p.scales + (int64_t)b * p.scales_bstride + (int64_t)row * (p.d / 16) + ch * 2;
#pragma unroll
    for (int m = 0; m < NM; ++m) {
        if (2 * m + (ch >> 1) < n_cb) {
            // codes are read once: not kept in L1, whose fill the loads would wait for
            asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                         : "=r"(r.c[m].x), "=r"(r.c[m].y), "=r"(r.c[m].z), "=r"(r.c[m].w)
                         : "l"(cr + 64 * m));
            r.s[m] = __ldg(reinterpret_cast<const uint16_t*>(sr + 8 * m));
        }
    }
}

// Bring the codes and scales of rows [row0, row1) into L2 (one thread; whole 16-byte pieces of them).
__device__ __forceinline__ void prefetch_rows(const AttnFp4Params& p, int b, int row0, int row1) {
    if (row0 >= row1) return;
    const uint32_t rows = (uint32_t)(row1 - row0);
    prefetch_l2_bulk(p.codes + (int64_t)b * p.codes_bstride + (int64_t)row0 * (p.d / 2), rows * (uint32_t)(p.d / 2));
    const uintptr_t s0 = reinterpret_cast<uintptr_t>(p.scales + (int64_t)b * p.scales_bstride + (int64_t)row0 * (p.d / 16));
    const uintptr_t lo = (s0 + 15) & ~(uintptr_t)15, hi = (s0 + rows * (uint32_t)(p.d / 16)) & ~(uintptr_t)15;
    if (lo < hi) prefetch_l2_bulk(reinterpret_cast<const void*>(lo), (uint32_t)(hi - lo));
}

// Eight codes (nibble i = element i) times the scale pair s2 = (s, s), as eight f16.
__device__ __forceinline__ uint4 decode8(uint32_t w, __half2 s2) {
    uint32_t o[4];
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3])
        : "r"(w));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 v = __hmul2(*reinterpret_cast<const __half2*>(&o[i]), s2);
        o[i] = *reinterpret_cast<const uint32_t*>(&v);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// 32 elements of a tile row from their codes and two scales; zeros when the row is not visible.  `dst`: the row's
// 128 bytes in the column block ch / 2 of the d-block, of which they are half ch % 2.  The upper two quarters
// store their 16-byte pieces in the order 2, 3, 0, 1: eight consecutive lanes (two rows, four quarters) then
// write eight different positions of the swizzled rows; in the same order they would meet on four.
__device__ __forceinline__ void decode_quarter(uint8_t* dst, int row, int ch, bool valid, const uint4& c, uint32_t s) {
    uint32_t h = 0u;   // the scales as f16
    if (valid)
        asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(h) : "r"(s));
    const bool turn = (ch & 2) != 0;
    const uint32_t w[4] = {turn ? c.z : c.x, turn ? c.w : c.y, turn ? c.x : c.z, turn ? c.y : c.w};
    const uint32_t sc[2] = {__byte_perm(h, h, turn ? 0x3232 : 0x1010), __byte_perm(h, h, turn ? 0x1010 : 0x3232)};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        *reinterpret_cast<uint4*>(dst + (((4 * (ch & 1) + (i ^ (ch & 2))) ^ (row & 7)) << 4)) =
            valid ? decode8(w[i], *reinterpret_cast<const __half2*>(&sc[i >> 1])) : make_uint4(0, 0, 0, 0);
}

// Decode this thread's part of the tile into the buffer at t_s, half by half: `released(h)` waits until half h
// may be overwritten (false: gave up), full[h] gets one arrival per warp.
// kTag: a NaN scale counts as 0, and tag[row] = serial marks its row.
template <int NM, bool kTag, class F>
__device__ __forceinline__ bool decode_tile(uint8_t* t_s, int row0, int vis, int n_cb, const Codes<NM>& r, uint64_t* full,
                                            uint32_t* tag, uint32_t serial, F released) {
    const int lane = threadIdx.x & 31, ch = lane & 3;
    const int row = ((threadIdx.x >> 5) & 7) * 8 + (lane >> 2);
#pragma unroll
    for (int h = 0; h < (NM + 1) / 2; ++h) {
        if (!released(h)) return false;
#pragma unroll
        for (int m = 2 * h; m < NM && m < 2 * h + 2; ++m) {
            const int cb = 2 * m + (ch >> 1);
            uint32_t sc = r.s[m];
            if (kTag && cb < n_cb && row0 + row < vis) {
                const bool n0 = (sc & 0x7Fu) == 0x7Fu, n1 = (sc & 0x7F00u) == 0x7F00u;
                if (n0) sc &= 0xFF00u;
                if (n1) sc &= 0x00FFu;
                if (n0 || n1) tag[row] = serial;
            }
            if (cb < n_cb) decode_quarter(t_s + (size_t)cb * kTBlk + row * 128, row, ch, row0 + row < vis, r.c[m], sc);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[h]);
    }
    return true;
}

// The group's heads as f16 into the swizzled column blocks at q_s, four softmax threads per head, each head
// scaled by 2^f; qc[head] = scale_log2 * 2^-f.
template <int NM>
__device__ __forceinline__ void load_q(const AttnFp4Params& p, const Group& grp, uint8_t* q_s, float* qc) {
    const int head = threadIdx.x >> 2, part = threadIdx.x & 3;
    const int n = p.d / 8;   // 16-byte chunks of a head: part, part + 4, ... (at most sixteen per thread)
    const bool in = head < grp.heads;
    const uint4* src = reinterpret_cast<const uint4*>(p.q + (grp.row0 + (in ? head : 0)) * p.d);
    uint4 v[4 * NM];
    uint32_t mx = 0;
#pragma unroll
    for (int k = 0; k < 4 * NM; ++k) {
        v[k] = make_uint4(0, 0, 0, 0);
        if (in && part + 4 * k < n) v[k] = __ldg(src + part + 4 * k);
    }
#pragma unroll
    for (int k = 0; k < 4 * NM; ++k)
        mx = __vmaxu2(mx, __vmaxu2(__vmaxu2(v[k].x & 0x7FFF7FFFu, v[k].y & 0x7FFF7FFFu),
                                   __vmaxu2(v[k].z & 0x7FFF7FFFu, v[k].w & 0x7FFF7FFFu)));
    mx = max(mx & 0xFFFFu, mx >> 16);
#pragma unroll
    for (int o = 1; o <= 2; o <<= 1) mx = max(mx, __shfl_xor_sync(kWarpFull, mx, o));
    int f = 139 - (int)(mx >> 7);   // largest into [2^12, 2^13); mx >> 7: its exponent field
    f = f > 127 ? 127 : f;          // (-116 .. 127)
    const float up = __uint_as_float((uint32_t)(f + 127) << 23);
    // 2^-f: subnormal at f = 127
    const float down = f == 127 ? __uint_as_float(0x00400000u) : __uint_as_float((uint32_t)(127 - f) << 23);
    if (part == 0) qc[head] = in ? p.scale_log2 * down : 0.f;
#pragma unroll
    for (int k = 0; k < 4 * NM; ++k) {
        if (!in || part + 4 * k >= n) continue;
        const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __half2 x = __floats2half2_rn(__uint_as_float(w[i] << 16) * up,
                                                __uint_as_float(w[i] & 0xFFFF0000u) * up);
            o[i] = *reinterpret_cast<const uint32_t*>(&x);
        }
        const int chunk = part + 4 * (k & 1);   // of column block k / 2
        *reinterpret_cast<uint4*>(q_s + (k >> 1) * kQBlk + head * 128 + ((chunk ^ (head & 7)) << 4)) =
            make_uint4(o[0], o[1], o[2], o[3]);
    }
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// ------------------------------------------------------------------ attention

struct __align__(16) Tail {
    float2 cm[2][4][32];      // [head group][warp of the group]: its copy of (softmax scale, -reference)
    float qc[64];             // per head: softmax scale (log2) over its f16 scaling
    float red[2][2][4][32];   // [tile parity][group][warp]: per-warp maxima
    float lsum[2][4][32];
    int hvis[2][64];          // [segment parity] per head: its visible rows (kPack)
    uint32_t nan_tag[2][kRows];   // [tile parity][row]: 1 + the last tile in which it held a NaN (kPack)
    Work work;
    long long scratch[kThreads / 32];
    uint64_t full[2][2];      // [buffer][half of the dims] decoded: one arrival per decoding warp
    uint64_t freed[2][2];     // the PV has read it
    uint64_t s_full[2], p_full[2];
    uint64_t q_full;
    uint32_t tmem_base;
    int abort;
    int qk_tile;              // tiles whose QK was issued, for the prefetching warp
};

size_t attn_smem(int d) {
    const int n_cb = (d + 127) / 128 * 2;
    return 1024 + (size_t)n_cb * (kQBlk + 2 * kTBlk) + 2 * kPBuf + sizeof(Tail);
}

// What no thread writes later: Q rows of heads >= h, the dims past d of the last d-block.
__device__ __forceinline__ void zero_padding(int h, int n_cb, int n_m, uint8_t* q_s, uint8_t* t_s) {
    for (int i = threadIdx.x; i < 2 * n_m * 64 * 8; i += kThreads)
        if (((i >> 3) & 63) >= h || (i >> 9) >= n_cb) reinterpret_cast<uint4*>(q_s)[i] = make_uint4(0, 0, 0, 0);
    if (n_cb & 1)
        for (int i = threadIdx.x; i < 2 * (int)kTBlk / 16; i += kThreads) {
            const int buf = i / (int)(kTBlk / 16), k = i % (int)(kTBlk / 16);
            reinterpret_cast<uint4*>(t_s + (size_t)(2 * n_m * buf + n_cb) * kTBlk)[k] = make_uint4(0, 0, 0, 0);
        }
}

// What a kernel does besides: kPlain nothing, kKeeps keeps the scores for the row weights, kPacks takes groups of
// several queries (and keeps the scores when there is room for them).
enum Mode { kPlain, kKeeps, kPacks };

template <int NM, Mode kMode>   // d-blocks of 128 dims
__global__ void __launch_bounds__(kThreads, 1) attn_fp4_kernel(const AttnFp4Params p) {
    constexpr bool kPack = kMode == kPacks;
    constexpr int kHalves = (NM + 1) / 2;
    constexpr uint32_t kTile = 2 * NM * kTBlk;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const int n_cb = p.d / 64;                 // column blocks of 64 dims
    uint8_t* q_s = smem;                       // [2 NM][64 heads][128 B]
    uint8_t* t_s = q_s + 2 * NM * kQBlk;       // two tiles [2 NM][64 rows][128 B]
    uint8_t* p_s = t_s + 2 * kTile;            // two P^T [64 rows][64 heads] f16
    Tail* tl = reinterpret_cast<Tail*>(p_s + 2 * kPBuf);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int nq = p.B * p.groups;
    const int hp = p.pack * p.h;               // heads of a full group
    const int sets = hp > 32 ? 2 : 1;          // sets of 32 heads
    volatile int* abort = &tl->abort;

    if (warp == 16) {
        tmem_alloc(&tl->tmem_base, NM <= 2 ? 256 : 512);
        tmem_relinquish();
    }
    if (tid == 0) {
        for (int k = 0; k < 2; ++k) {
            for (int h = 0; h < 2; ++h) {
                mbar_init(&tl->full[k][h], 8);
                mbar_init(&tl->freed[k][h], 1);
            }
            mbar_init(&tl->s_full[k], 1);
            mbar_init(&tl->p_full[k], 4 * sets);
        }
        mbar_init(&tl->q_full, 8);
        tl->abort = 0;
        tl->qk_tile = 0;
        fence_mbar_init();
    }
    if (kPack && tid < 2 * kRows) tl->nan_tag[0][tid] = 0u;
    zero_padding(hp, n_cb, NM, q_s, t_s);
    fence_proxy_async_smem();
    plan_work(nq, blockIdx.x, gridDim.x, tl->scratch, &tl->work,
              [&](int q) { return (group_rows(p, q / p.groups, q % p.groups) + kRows - 1) / kRows; });
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(kWarpFull, tl->tmem_base, 0);   // warp-uniform, as the compiler can see
    const Work wk = tl->work;
    griddep_launch_dependents();

    if (warp >= 16) {
        regs_down<kRegsMma>();
        // -------------------------------------------------------------- MMA issue
        // Warp 16 issues the QKs and warp 17 the PVs, each as its operands come: in one warp's order a PV waits for the
        // next tile's QK, that for its decode, and the decode for the buffer of the PV before.
        const int n_mma = (hp + 15) / 16 * 16;
        uint32_t n = 0;
        bool ok = true;   // the whole warp waits, one elected lane issues (so the operands stay warp-uniform)
        auto wait = [&](uint64_t* bar, uint32_t parity) {
            ok = warp_wait(bar, parity, p.status, abort);
            tc_fence_after();
            return ok;
        };
        Walk walk(wk);
        Seg sg;
        if (warp == 16) {
            // the tile and Q, both K-major
            const uint32_t idesc = idesc_f16_f32(kRows, n_mma, false, false);
            const uint64_t dk = sdesc(smem_u32(t_s), 16, 1024, kLayoutSW128), dq = sdesc(smem_u32(q_s), 16, 1024, kLayoutSW128);
            uint32_t qn = 0;
            int2 rec = make_int2(-1, 0);
            while (ok && walk.next(p, sg)) {
                if (sg.t0 == 0 && sg.t1 < sg.nt) {
                    const long long last = walk.pos - sg.t1 + sg.nt - 1;   // list position of the query's last tile
                    int c = (int)(last * wk.ctas / wk.total);
                    while ((long long)(c + 1) * wk.total / wk.ctas <= last) ++c;
                    while ((long long)c * wk.total / wk.ctas > last) --c;
                    rec = make_int2(sg.q, c);
                }
                if (!wait(&tl->q_full, qn & 1u)) break;
                ++qn;
                for (int t = sg.t0; t < sg.t1 && ok; ++t, ++n) {
                    if (lane == 0) tl->qk_tile = (int)n;
                    const uint32_t buf = n & 1u;   // its S^T has been read: the tile was decoded after the PV of n - 2
#pragma unroll
                    for (int h = 0; h < kHalves; ++h) {
                        if (!wait(&tl->full[buf][h], (n >> 1) & 1u)) break;
                        if (elect_one()) {
#pragma unroll
                            for (int m = 2 * h; m < NM && m < 2 * h + 2; ++m)
                                qk_blocks(m, tmem + 64u * buf, lo32(dk) + buf * (kTile / 16), lo32(dq), hi32(dk), idesc);
                            if (h == kHalves - 1) umma_commit(&tl->s_full[buf]);
                        }
                        __syncwarp();
                    }
                }
            }
            if (lane == 0) p.rec[blockIdx.x] = rec;
        } else if (warp == 17) {
            // the tile and P^T, both MN-major
            const uint32_t idesc = idesc_f16_f32(128, n_mma, true, true);
            const uint64_t dv = sdesc(smem_u32(t_s), kTBlk, 1024, kLayoutSW128), dp = sdesc(smem_u32(p_s), kPBuf, 1024, kLayoutSW128);
            while (ok && walk.next(p, sg)) {
                for (int t = sg.t0; t < sg.t1; ++t, ++n) {
                    const uint32_t buf = n & 1u;
                    if (!wait(&tl->p_full[buf], (n >> 1) & 1u)) break;
                    if (elect_one()) {
#pragma unroll
                        for (int m = 0; m < NM; ++m) {
                            const uint32_t o = tmem + kTmO + 64u * (uint32_t)m;
                            const uint32_t a = lo32(dv) + buf * (kTile / 16) + (uint32_t)m * (2 * kTBlk / 16);
                            const uint32_t b = lo32(dp) + buf * (kPBuf / 16);
                            if (t == sg.t0) pv_block<true>(o, a, hi32(dv), b, hi32(dp), idesc);
                            else pv_block<false>(o, a, hi32(dv), b, hi32(dp), idesc);
                            if ((m & 1) || m == NM - 1) umma_commit(&tl->freed[buf][m >> 1]);
                        }
                    }
                    __syncwarp();
                }
            }
        } else if (warp == 18 && lane == 0) {
            // The rows of the next kAhead tiles are on their way to L2 when a tile is decoded (64 long rows of one query
            // each: 112 -> 106 us), asked for by a sequence's first query only: the others find them there.
            volatile int* now = &tl->qk_tile;
            bool on = true;
            while (on && walk.next(p, sg)) {
                const bool asks = sg.q == sg.b * p.groups;
                for (int t = sg.t0; on && t < sg.t1; ++t, ++n) {
                    if (!asks) continue;
                    prefetch_rows(p, sg.b, t * kRows, min((t + 1) * kRows, sg.vis));
                    // wait (a while at most) until the tile kAhead before is at hand
                    for (int i = 0; *now + kAhead < (int)n && on; ++i) {
                        on = i < 100000 && !*abort;
                        __nanosleep(200);
                    }
                }
            }
        }
        __syncwarp();
    } else if (warp >= 8) {
        regs_down<kRegsDecode>();
        // -------------------------------------------------------------- decode
        uint32_t n = 0;
        bool dead = false;
        Walk walk(wk);
        Seg cur;
        Codes<NM> codes;
        bool more = walk.next(p, cur);
        int t = cur.t0;
        if (more) load_codes<NM>(p, cur.b, t * kRows, cur.vis, n_cb, codes);
        while (more && !dead) {
            const uint32_t buf = n & 1u;
            dead = !decode_tile<NM, kPack>(t_s + buf * kTile, t * kRows, cur.vis, n_cb, codes, tl->full[buf], tl->nan_tag[buf],
                                           n + 1u, [&](int h) {
                return n < 2 || warp_wait(&tl->freed[buf][h], ((n >> 1) - 1) & 1u, p.status, abort);
            });
            ++n;
            if (++t == cur.t1) {
                more = walk.next(p, cur);
                t = cur.t0;
            }
            if (more) load_codes<NM>(p, cur.b, t * kRows, cur.vis, n_cb, codes);
        }
    } else {
        regs_up<kRegsSoft>();
        // -------------------------------------------------------------- Q, softmax, outputs
        const int set = warp >> 2, qd = warp & 3;
        const int row = 16 * qd + (lane >> 2);   // this thread's tile rows: row, row + 8
        const int l4 = lane & 3;                 // its heads: 32 set + 8 g + 2 l4 + {0, 1}
        const bool active = set < sets;          // this warp's set has heads
        const uint32_t lane_base = (uint32_t)(32 * qd) << 16;
        const uint32_t bar_set = 1u + (uint32_t)set;
        uint32_t n = 0;
        bool dead = false;
        float m_run = -INFINITY;                 // what P is relative to, in log2: lane l: head 32 set + l
        float l_thr[8];                          // running sums of the thread's heads over its rows

        auto mwait = [&](uint64_t* bar, uint32_t parity) {
            if (!dead) dead = !warp_wait(bar, parity, p.status, abort);
        };

        // One tile's probabilities.  cm holds (c, -m) of the thread's heads: c the softmax scale (log2) over the head's
        // f16 scaling, m its reference, 2^-7 of the maximum that it was taken from; so y = S c - m is one FMA and 2^y the
        // probability.
        float2 cm[8];
        auto load_cm = [&]() {   // from the warp's copy, which has every head of the group
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const float4 v = *reinterpret_cast<const float4*>(&tl->cm[set][qd][8 * g + 2 * l4]);
                cm[2 * g] = make_float2(v.x, v.y);
                cm[2 * g + 1] = make_float2(v.z, v.w);
            }
        };
        // vis: rows that the group's last query sees; row0: this thread's first one; tile: of all the groups' (kept scores)
        int hv[8] = {};   // kPack: rows that each of the thread's heads sees
        auto softmax = [&](int vis, int row0, bool first, int64_t tile) {
            const uint32_t buf = n & 1u;
            mwait(&tl->s_full[buf], (n >> 1) & 1u);
            tc_fence_after();
            const bool v0 = vis > row0 && !dead, v1 = vis > row0 + 8 && !dead;
            auto sees = [&](int i, int second) {   // the thread's head i its first or second row
                if (kPack) return hv[i] > row0 + 8 * second && !dead;
                return second ? v1 : v0;
            };
            const uint32_t ts = tmem + lane_base + 64u * buf + 32u * (uint32_t)set;
            uint32_t r[16];
            tmem_ld_rows16(ts, r);
            tmem_ld_wait();
            if (kPack) {
                // a NaN row was decoded as 0, so that P = 0 keeps it from the heads that do not see it
                const bool n0 = tl->nan_tag[buf][row] == n + 1u, n1 = tl->nan_tag[buf][row + 8] == n + 1u;
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    if (n0) r[4 * g] = r[4 * g + 1] = 0x7FFFFFFFu;
                    if (n1) r[4 * g + 2] = r[4 * g + 3] = 0x7FFFFFFFu;
                }
            }
            if (kMode == kKeeps || (kPack && p.scores)) {
                float4* sc = reinterpret_cast<float4*>(p.scores) + (tile * 8 + warp) * 128 + lane;
#pragma unroll
                for (int g = 0; g < 4; ++g)
                    __stcs(sc + 32 * g, make_float4(__uint_as_float(r[4 * g]) * cm[2 * g].x,
                                                    __uint_as_float(r[4 * g + 1]) * cm[2 * g + 1].x,
                                                    __uint_as_float(r[4 * g + 2]) * cm[2 * g].x,
                                                    __uint_as_float(r[4 * g + 3]) * cm[2 * g + 1].x));
            }
            float y[16];
            float top0 = -INFINITY, top1 = -INFINITY;
            auto scale = [&]() {
#pragma unroll
                for (int g = 0; g < 4; ++g)
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        y[4 * g + c] = fmaf(__uint_as_float(r[4 * g + c]), cm[2 * g + (c & 1)].x, cm[2 * g + (c & 1)].y);
            };
            scale();
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                if (kPack) {
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        if (sees(2 * g + (c & 1), c >> 1)) top0 = fmaxf(top0, y[4 * g + c]);
                } else {
                    top0 = fmaxf(top0, fmaxf(y[4 * g], y[4 * g + 1]));
                    top1 = fmaxf(top1, fmaxf(y[4 * g + 2], y[4 * g + 3]));
                }
            }
            // the references stay unless a visible score passes the maximum that its head's was taken from by 2^8
            const bool need = !named_bar_and(bar_set, 128, !(first || ((kPack || v0) && top0 > kTopMost) || (v1 && top1 > kTopMost)));
            if (need) {
                float* red = &tl->red[buf][set][qd][0];
#pragma unroll
                for (int g = 0; g < 4; ++g)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        float v = fmaxf(sees(2 * g + c, 0) ? y[4 * g + c] : -INFINITY,
                                        sees(2 * g + c, 1) ? y[4 * g + 2 + c] : -INFINITY);
#pragma unroll
                        for (int o = 4; o <= 16; o <<= 1) v = fmaxf(v, __shfl_xor_sync(kWarpFull, v, o));
                        if (lane < 4) red[8 * g + 2 * lane + c] = v;
                    }
                named_bar_sync(bar_set, 128);
                const float* rr = &tl->red[buf][set][0][lane];
                float2* own = &tl->cm[set][qd][0];
                const float old = -own[lane].y;            // what y is relative to
                const float mt = fmaxf(fmaxf(rr[0], rr[32]), fmaxf(rr[64], rr[96])) + old;
                const float m_new = (m_run == -INFINITY || mt > m_run + kTopMost) ? fmaxf(m_run, mt - kTopNew) : m_run;
                const float alpha = (m_new == m_run) ? 1.f : exp2f(m_run - m_new);
                m_run = m_new;
                __syncwarp();
                // a head without any finite score keeps -inf; its exponents are taken from 0, so that NaN
                // scores show in its output
                own[lane].y = m_new == -INFINITY ? 0.f : -m_new;
                __syncwarp();
                load_cm();
                scale();
                if (!first && !dead && __any_sync(kWarpFull, alpha != 1.f)) {
                    mwait(&tl->freed[buf ^ 1u][kHalves - 1], ((n - 1) >> 1) & 1u);   // the previous tile's PV is done
                    tc_fence_after();
#pragma unroll 1
                    for (int k = 0; k < 2 * NM; ++k) {
                        const uint32_t ta = tmem + lane_base + kTmO + 32u * (uint32_t)(2 * (k >> 1) + set) + 16u * (k & 1);
                        uint32_t o[16];
                        tmem_ld16(ta, o);
                        tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            o[i] = __float_as_uint(__uint_as_float(o[i]) * __shfl_sync(kWarpFull, alpha, 16 * (k & 1) + i));
                        tmem_st16(ta, o);
                    }
                    tmem_st_wait();
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        l_thr[2 * g] *= __shfl_sync(kWarpFull, alpha, 8 * g + 2 * l4);
                        l_thr[2 * g + 1] *= __shfl_sync(kWarpFull, alpha, 8 * g + 2 * l4 + 1);
                    }
                }
            }
            uint8_t* prow = p_s + buf * kPBuf + row * 128 + 4 * l4;
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const float a0 = sees(2 * g, 0) ? fast_exp2(y[4 * g]) : 0.f, a1 = sees(2 * g + 1, 0) ? fast_exp2(y[4 * g + 1]) : 0.f;
                const float b0 = sees(2 * g, 1) ? fast_exp2(y[4 * g + 2]) : 0.f, b1 = sees(2 * g + 1, 1) ? fast_exp2(y[4 * g + 3]) : 0.f;
                l_thr[2 * g] += a0 + b0;
                l_thr[2 * g + 1] += a1 + b1;
                const int at = ((4 * set + g) ^ (row & 7)) << 4;
                *reinterpret_cast<uint32_t*>(prow + at) = pack_f16x2(a0, a1);
                *reinterpret_cast<uint32_t*>(prow + 8 * 128 + at) = pack_f16x2(b0, b1);
            }
            fence_proxy_async_smem();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&tl->p_full[buf]);
        };

        // a segment's O^T and sums: the group's output when the segment holds all its tiles, else a partial
        // (slot >= 0: where); par: the segment's parity; sink, prev_lse: of head 32 set + lane
        auto epilogue = [&](int q, int slot, int par, float sink, float prev_lse) {
            const Group grp = group_of(p, q);
            // 16 heads x 32 dims of this warp at a time: k / 2 the d-block, heads 32 set + 16 (k & 1) ...
            // Pieces of 8 dims, two per lane: piece c = lane + 32 j is head c / 4, dims 8 (c % 4) ...
            auto piece = [&](int k, int j, int64_t& at) {
                const int c = lane + 32 * j;
                const int hw = 32 * set + 16 * (k & 1) + (c >> 2), dw = 128 * (k >> 1) + 32 * qd + 8 * (c & 3);
                at = (grp.row0 + hw) * p.d + dw;
                return k < 2 * NM && hw < grp.heads && dw < p.d;
            };
            const bool joins = p.prev_out != nullptr && slot < 0;
            uint4 pre[2][2];   // [k & 1]: prev_out, loaded two steps ahead
            auto load_prev = [&](int k, uint4* v) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    int64_t at;
                    v[j] = make_uint4(0, 0, 0, 0);
                    if (piece(k, j, at)) v[j] = *reinterpret_cast<const uint4*>(p.prev_out + at);
                }
            };
            if (joins) {
                load_prev(0, pre[0]);
                load_prev(1, pre[1]);
            }
            mwait(&tl->freed[(n - 1) & 1u][kHalves - 1], ((n - 1) >> 1) & 1u);
            tc_fence_after();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float v = l_thr[i];
#pragma unroll
                for (int o = 4; o <= 16; o <<= 1) v += __shfl_xor_sync(kWarpFull, v, o);
                if (lane < 4) tl->lsum[set][qd][8 * (i >> 1) + 2 * lane + (i & 1)] = v;
            }
            named_bar_sync(bar_set, 128);
            const float* ls = &tl->lsum[set][0][lane];
            const float lt = (ls[0] + ls[32]) + (ls[64] + ls[96]);
            const int hh = 32 * set + lane;
            float inv = 0.f, wp = 0.f;
            if (slot >= 0) {
                if (qd == 0) p.part_ml[slot * 64 + hh] = make_float2(m_run, lt);
            } else if (kPack && hh < grp.heads && tl->hvis[par][hh] == 0) {
                // a query that sees no row, next to one that does: what it had
                wp = prev_lse == -INFINITY ? 0.f : 1.f;
                if (p.lse && qd == 0) p.lse[grp.row0 + hh] = prev_lse;
            } else if (hh < grp.heads) {
                // everything relative to the largest of the reference, the sink and prev_lse
                const float sk = sink * kLog2e, pl = prev_lse * kLog2e;
                float mx = fmaxf(m_run, fmaxf(sk, pl));
                if (mx == -INFINITY) mx = 0.f;
                const float f = lt == 0.f ? 0.f : m_run == -INFINITY ? exp2f(-mx) : exp2f(m_run - mx);   // (inf * 0)
                const float ep = exp2f(pl - mx);
                const float den = lt * f + exp2f(sk - mx) + ep;
                inv = f / den;
                wp = ep / den;
                if (p.lse && qd == 0) p.lse[grp.row0 + hh] = (mx + log2f(den)) * kLn2;
            }
            // The steps turn O^T over through shared memory, in fp32: lanes hold dims, the pieces are a head's.  The
            // heads' factors take the place of (c, -m), which the next segment sets anew.
            float* stg = reinterpret_cast<float*>(p_s) + warp * 16 * 32;   // this warp's [16 heads][32 dims]
            float2* fac = &tl->cm[set][qd][0];
            fac[lane] = make_float2(inv, wp);
#pragma unroll 1
            for (int m = 0; m < NM; ++m)
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const int k = 2 * m + half, h0 = 16 * half;
                    const int dd = 128 * m + 32 * qd + lane;
                    uint32_t r[16];
                    tmem_ld16(tmem + lane_base + kTmO + 64u * (uint32_t)m + 32u * (uint32_t)set + (uint32_t)h0, r);
                    tmem_ld_wait();
                    if (slot >= 0) {
                        float* po = p.part_o + ((int64_t)slot * hp + 32 * set + h0) * p.d + dd;
                        if (dd < p.d) {
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                if (32 * set + h0 + i < hp) po[i * p.d] = __uint_as_float(r[i]);
                        }
                        continue;
                    }
#pragma unroll
                    for (int i = 0; i < 16; ++i) stg[i * 32 + lane] = __uint_as_float(r[i]);
                    __syncwarp();
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int c = lane + 32 * j;
                        const float2 f = fac[h0 + (c >> 2)];
                        const float4* src = reinterpret_cast<const float4*>(stg + (c >> 2) * 32 + 8 * (c & 3));
                        const float4 lo = src[0], hi = src[1];
                        float v[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
                        const uint32_t pw[4] = {pre[half][j].x, pre[half][j].y, pre[half][j].z, pre[half][j].w};
                        uint32_t o[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            float x0 = v[2 * i] * f.x, x1 = v[2 * i + 1] * f.x;
                            if (joins) {   // weight 0: prev_out is not used
                                x0 = f.y != 0.f ? x0 + f.y * __uint_as_float(pw[i] << 16) : x0;
                                x1 = f.y != 0.f ? x1 + f.y * __uint_as_float(pw[i] & 0xFFFF0000u) : x1;
                            }
                            o[i] = dead ? 0u : pack_bf16x2(x0, x1);
                        }
                        int64_t at;
                        if (piece(k, j, at)) *reinterpret_cast<uint4*>(p.out + at) = make_uint4(o[0], o[1], o[2], o[3]);
                    }
                    if (joins) load_prev(k + 2, pre[half]);
                    __syncwarp();
                }
        };

        Walk walk(wk);
        Seg sg;
        int pend_q = -1, pend_slot = -1;       // the segment whose output is pending
        float pend_sink = -INFINITY, pend_lse = -INFINITY;   // and what it is joined with
        int par = 0;                           // segment parity
        while (walk.next(p, sg)) {
            // the Q buffer is free: this warp has seen the last S^T of the previous query (a warp whose head
            // group is empty writes no Q)
            const Group grp = group_of(p, sg.q);
            load_q<NM>(p, grp, q_s, tl->qc);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&tl->q_full);
            if (kPack && tid < 64) tl->hvis[par][tid] = head_rows(p, grp, tid);   // (every warp is done with par's last)
            if (tid == 0) {   // what the next segment and this one's end will read, into L2
                const uint32_t row = (uint32_t)p.d * 2;
                if (sg.q + 1 < nq) {
                    const Group nx = group_of(p, sg.q + 1);
                    prefetch_l2_bulk(p.q + nx.row0 * p.d, (uint32_t)nx.heads * row);
                }
                if (p.prev_out) prefetch_l2_bulk(p.prev_out + grp.row0 * p.d, (uint32_t)grp.heads * row);
            }
            if (pend_q >= 0 && active) epilogue(pend_q, pend_slot, par ^ 1, pend_sink, pend_lse);
            named_bar_sync(kBarSoft, 256);     // the staging area is every warp's P^T; qc is complete
            m_run = -INFINITY;
            tl->cm[set][qd][lane] = make_float2(tl->qc[32 * set + lane], 0.f);
            __syncwarp();
            load_cm();
            if (kPack) {
#pragma unroll
                for (int i = 0; i < 8; ++i) hv[i] = tl->hvis[par][32 * set + 8 * (i >> 1) + 2 * l4 + (i & 1)];
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) l_thr[i] = 0.f;
            for (int t = sg.t0; t < sg.t1; ++t, ++n)
                if (active)
                    softmax(sg.vis, t * kRows + row, t == sg.t0,
                            kMode == kPlain ? 0 : (int64_t)sg.q * ((p.n_rows + kRows - 1) / kRows) + t);
            par ^= 1;
            pend_q = sg.q;
            const int hh = 32 * set + lane;
            if (hh < grp.heads) {
                if (p.sink) pend_sink = __ldg(p.sink + (kPack ? hh % p.h : hh));
                pend_lse = p.prev_lse ? __ldg(p.prev_lse + grp.row0 + hh) : -INFINITY;
            }
            pend_slot = sg.t0 == 0 && sg.t1 == sg.nt ? -1 : 2 * (int)blockIdx.x + (sg.t0 == 0 ? 1 : 0);
        }
        if (pend_q >= 0 && active) epilogue(pend_q, pend_slot, par ^ 1, pend_sink, pend_lse);

        // groups without a visible row
        for (int q = blockIdx.x; q < nq; q += gridDim.x) {
            const Group grp = group_of(p, q);
            if (visible_rows(p, grp.b, min(grp.t0 + p.pack, p.s) - 1) > 0) continue;
            for (int i = tid; i < grp.heads; i += 256)
                if (p.lse) p.lse[grp.row0 + i] = p.prev_lse ? p.prev_lse[grp.row0 + i] : -INFINITY;
            const int chunks = p.d / 8;
#pragma unroll 4
            for (int i = tid; i < grp.heads * chunks; i += 256) {
                uint4 v = make_uint4(0, 0, 0, 0);
                if (p.prev_out) {
                    v = reinterpret_cast<const uint4*>(p.prev_out + grp.row0 * p.d)[i];
                    if (p.prev_lse[grp.row0 + i / chunks] == -INFINITY) v = make_uint4(0, 0, 0, 0);
                }
                reinterpret_cast<uint4*>(p.out + grp.row0 * p.d)[i] = v;
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (*abort) {   // a wait gave up: let the MMAs in flight finish before the CTA's memory goes
        const uint64_t t0 = global_timer_ns();
        while (global_timer_ns() - t0 < 50000ull) {
        }
    }
    if (warp == 16) {
        tc_fence_after();
        tmem_dealloc(tmem, NM <= 2 ? 256 : 512);
    }
}

// ------------------------------------------------------------------ joining split queries

// Block (x, head, z): the x-th split query group (there are at most gridDim.x), dims 4 W z .. 4 W (z + 1) - 1; thread
// (g, i), g < G, dims 4 (W z + i) + {0..3} of every G-th part, four parts in flight; their sums join in shared memory
// in a fixed order.  G follows from the parts of a query when all are alike: a single long query (152 parts) needs many loads
// in flight (20 us with G = 8, W = 128), thousands of short ones (two parts each) would spend their time starting wide
// blocks.  A long query among short ones gets the short ones' G: one of 65536 rows x 512 among 59 of 300 takes 58 us for
// the call, alone 29.
template <int G, int W>
__global__ void __launch_bounds__(G * W) merge_kernel(const AttnFp4Params p) {
    __shared__ float fac[256];
    __shared__ float stat[2];
    __shared__ float4 part[G][W];
    const int hh = blockIdx.y, tid = threadIdx.x, lane = tid & 31;
    const int g = tid / W, ti = tid % W, i4 = (int)blockIdx.z * W + ti;
    __shared__ int3 found;   // (query, first CTA, last CTA)
    griddep_wait();
    griddep_launch_dependents();
    // One warp reads all records at once and takes the blockIdx.x-th real one (read one after another, and looked
    // through by every warp, a single query's 152 took 50 and 13 us; dealt out by the CTA they come from, equal
    // queries' records all fall to a few blocks).
    if (tid < 32) {
        int2 r[5];
        int cnt = 0;
        if (lane == 0) found.x = -1;
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 5; ++k) r[k] = lane + 32 * k < p.grid ? __ldcg(p.rec + lane + 32 * k) : make_int2(-1, 0);
#pragma unroll
        for (int k = 0; k < 5; ++k) {
            const uint32_t real = __ballot_sync(kWarpFull, r[k].x >= 0);
            if (r[k].x >= 0 && cnt + __popc(real & ((1u << lane) - 1u)) == (int)blockIdx.x)
                found = make_int3(r[k].x, lane + 32 * k, r[k].y);
            cnt += __popc(real);
        }
    }
    __syncthreads();
    const int3 rec = found;
    if (rec.x < 0) return;
    const int c = rec.y;
    const int parts = rec.z - c + 1;   // slots 2c + 1, 2 (c + 1), 2 (c + 2), ...
    auto slot = [&](int i) { return i == 0 ? 2 * c + 1 : 2 * (c + i); };
    const Group grp = group_of(p, rec.x);
    if (hh >= grp.heads) return;
    const bool seen = p.pack == 1 || head_rows(p, grp, hh) > 0;
    const int64_t at = grp.row0 + hh;
    const int hp = p.pack * p.h;
    // the partial outputs start loading before their factors are known
    float4 v[4];
    const bool in = 4 * i4 < p.d;
    const float4* src = reinterpret_cast<const float4*>(p.part_o + (int64_t)hh * p.d) + (in ? i4 : 0);
    const int64_t step = (int64_t)hp * p.d / 4;
    auto load = [&](int i) { return __ldcg(src + slot(i < parts ? i : parts - 1) * step); };   // always a part
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = load(g + k * G);
    const float sk = p.sink && seen ? __ldg(p.sink + hh % p.h) * kLog2e : -INFINITY;
    const float pl_in = p.prev_lse ? p.prev_lse[at] : -INFINITY, pl = pl_in * kLog2e;
    if (tid < 32) {
        float2 ml[5];   // parts <= 160
#pragma unroll
        for (int k = 0; k < 5; ++k)
            ml[k] = lane + 32 * k < parts ? __ldcg(p.part_ml + slot(lane + 32 * k) * 64 + hh) : make_float2(-INFINITY, 0.f);
        float mx = fmaxf(sk, pl);
#pragma unroll
        for (int k = 0; k < 5; ++k) mx = fmaxf(mx, ml[k].x);
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kWarpFull, mx, o));
        if (mx == -INFINITY) mx = 0.f;
        float l = 0.f;
#pragma unroll
        for (int k = 0; k < 5; ++k) {
            if (lane + 32 * k < parts) {
                // a part of which the head sees nothing: not inf * 0
                const float f = ml[k].y == 0.f ? 0.f : exp2f((ml[k].x == -INFINITY ? 0.f : ml[k].x) - mx);
                fac[lane + 32 * k] = f;
                l += ml[k].y * f;
            }
        }
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) l += __shfl_xor_sync(kWarpFull, l, o);
        const float ep = exp2f(pl - mx);
        const float den = l + exp2f(sk - mx) + ep;
        if (lane == 0) {   // a query that sees no row, next to one that does, keeps what it had
            stat[0] = seen ? 1.f / den : 0.f;
            stat[1] = seen ? ep / den : pl == -INFINITY ? 0.f : 1.f;
            if (p.lse && blockIdx.z == 0) p.lse[at] = seen ? (mx + log2f(den)) * kLn2 : pl_in;
        }
    }
    __syncthreads();
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = g; i0 < parts; i0 += 4 * G) {
        float4 w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) w[k] = load(i0 + (4 + k) * G);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int i = i0 + k * G;
            if (i < parts) {
                const float f = fac[i];
                o.x += f * v[k].x;
                o.y += f * v[k].y;
                o.z += f * v[k].z;
                o.w += f * v[k].w;
            }
            v[k] = w[k];
        }
    }
    part[g][ti] = o;
    __syncthreads();
    if (g == 0 && in) {
#pragma unroll
        for (int k = 1; k < G; ++k) {
            const float4 q = part[k][ti];
            o.x += q.x;
            o.y += q.y;
            o.z += q.z;
            o.w += q.w;
        }
        const float inv = stat[0], wp = stat[1];
        o.x *= inv;
        o.y *= inv;
        o.z *= inv;
        o.w *= inv;
        if (wp != 0.f && p.prev_out) {
            const uint2 pv = *reinterpret_cast<const uint2*>(p.prev_out + at * p.d + 4 * i4);
            o.x += wp * __uint_as_float(pv.x << 16);
            o.y += wp * __uint_as_float(pv.x & 0xFFFF0000u);
            o.z += wp * __uint_as_float(pv.y << 16);
            o.w += wp * __uint_as_float(pv.y & 0xFFFF0000u);
        }
        *reinterpret_cast<uint2*>(p.out + at * p.d + 4 * i4) =
            make_uint2(pack_bf16x2(o.x, o.y), pack_bf16x2(o.z, o.w));
    }
}

// ------------------------------------------------------------------ row weights

struct __align__(16) WTail {
    int hvis[2][64];                 // [query parity] per head: its visible rows
    float2 cl[2][64];                // [query parity] per head: (softmax scale over the f16 scaling, -lse in log2)
    float qc[64];
    float acc[kWTiles][2][kRows];    // [tile of the chunk][head group][row]
    Work work;
    long long scratch[kThreads / 32];
    uint64_t full[2][2];
    uint64_t freed[2][2];            // the QK has read it
    uint64_t s_full[2];              // [tile parity] S^T done
    uint64_t s_free[2];              // S^T read
    uint64_t q_full;
    uint32_t tmem_base;
    int abort;
};

size_t row_weight_smem(int d) {
    const int n_cb = (d + 127) / 128 * 2;
    return 1024 + (size_t)n_cb * (kQBlk + 2 * kTBlk) + sizeof(WTail);
}

// One CTA's work: its piece of the sequences' tiles in chunks of at most kWTiles tiles of one sequence; per
// chunk its queries [ta, tb) of that sequence; per query the chunk's tiles that the query sees.
struct WWalk {
    long long pos, hi;
    int b, off, ta, tb;
    int t0, t1, vis_all;   // the chunk: tiles [t0, t1) of sequence `seq`
    int seq, q, end, k;    // the query, the end of its tiles, the tile
    __device__ __forceinline__ WWalk(const Work& w, int ta_, int tb_)
        : pos(w.lo), hi(w.hi), b(w.q), off(w.off), ta(ta_), tb(tb_), t0(0), t1(0), vis_all(0), seq(0), q(tb_), end(0), k(0) {}
    __device__ __forceinline__ bool chunk(const AttnFp4Params& p) {
        while (pos < hi) {
            seq = b;
            vis_all = visible_rows(p, b, p.s - 1);
            const int nt = (vis_all + kRows - 1) / kRows;
            t0 = off;
            t1 = (long long)(nt - off) < hi - pos ? nt : off + (int)(hi - pos);
            if (t1 - t0 > kWTiles) t1 = t0 + kWTiles;
            pos += t1 - t0;
            off = t1;
            if (off >= nt) {
                ++b;
                off = 0;
            }
            if (t1 > t0) return true;
        }
        return false;
    }
    // first tile of the next query (from q on) that sees one of the chunk's; false: none is left
    __device__ __forceinline__ bool query(const AttnFp4Params& p) {
        for (; q < tb; ++q) {
            const int nt = (group_rows(p, seq, q) + kRows - 1) / kRows;
            end = nt < t1 ? nt : t1;
            k = t0;
            if (k < end) return true;
        }
        return false;
    }
};

template <int NM>
__global__ void __launch_bounds__(kThreads, 1) row_weight_kernel(const AttnFp4Params p) {
    constexpr int kHalves = (NM + 1) / 2;
    constexpr uint32_t kTile = 2 * NM * kTBlk;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const int n_cb = p.d / 64;
    uint8_t* q_s = smem;
    uint8_t* t_s = q_s + 2 * NM * kQBlk;
    WTail* tl = reinterpret_cast<WTail*>(t_s + 2 * kTile);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int hp = p.pack * p.h, sets = hp > 32 ? 2 : 1;
    volatile int* abort = &tl->abort;
    // this CTA's queries of every sequence, and its piece of the tiles
    const int split = (int)blockIdx.x % p.w_split;
    const int ta = (int)((long long)split * p.groups / p.w_split);
    const int tb = (int)((long long)(split + 1) * p.groups / p.w_split);

    if (warp == 16) {
        tmem_alloc(&tl->tmem_base, 128);
        tmem_relinquish();
    }
    if (tid == 0) {
        for (int k = 0; k < 2; ++k) {
            for (int h = 0; h < 2; ++h) {
                mbar_init(&tl->full[k][h], 8);
                mbar_init(&tl->freed[k][h], 1);
            }
            mbar_init(&tl->s_full[k], 1);
            mbar_init(&tl->s_free[k], 4 * sets);
        }
        mbar_init(&tl->q_full, 8);
        tl->abort = 0;
        fence_mbar_init();
    }
    zero_padding(hp, n_cb, NM, q_s, t_s);
    fence_proxy_async_smem();
    plan_work(p.B, (int)blockIdx.x / p.w_split, (int)gridDim.x / p.w_split, tl->scratch, &tl->work,
              [&](int b) { return (visible_rows(p, b, p.s - 1) + kRows - 1) / kRows; });
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(kWarpFull, tl->tmem_base, 0);
    WWalk w(tl->work, ta, tb);
    griddep_wait();   // lse is complete from here on

    if (warp >= 16) {
        regs_down<kRegsMma>();
        const uint32_t idesc_qk = idesc_f16_f32(kRows, (hp + 15) / 16 * 16, false, false);
        const uint64_t dk = sdesc(smem_u32(t_s), 16, 1024, kLayoutSW128), dq = sdesc(smem_u32(q_s), 16, 1024, kLayoutSW128);
        uint32_t n = 0, qn = 0;
        int have = -1;
        bool ok = warp == 16;
        auto wait = [&](uint64_t* bar, uint32_t parity) {
            ok = warp_wait(bar, parity, p.status, abort);
            tc_fence_after();
            return ok;
        };
        while (ok && w.chunk(p)) {
            for (w.q = ta; ok && w.query(p); ++w.q) {
                if (have != w.seq * p.groups + w.q) {   // another query: its Q
                    if (!wait(&tl->q_full, qn & 1u)) break;
                    ++qn;
                    have = w.seq * p.groups + w.q;
                }
                for (int k = w.k; k < w.end && ok; ++k, ++n) {
                    const uint32_t buf = n & 1u;
                    if (n >= 2 && !wait(&tl->s_free[buf], ((n >> 1) - 1) & 1u)) break;
#pragma unroll
                    for (int h = 0; h < kHalves; ++h) {
                        if (!wait(&tl->full[buf][h], (n >> 1) & 1u)) break;
                        if (elect_one()) {
#pragma unroll
                            for (int m = 2 * h; m < NM && m < 2 * h + 2; ++m)
                                qk_blocks(m, tmem + 64u * buf, lo32(dk) + buf * (kTile / 16), lo32(dq), hi32(dk), idesc_qk);
                            umma_commit(&tl->freed[buf][h]);
                            if (h == kHalves - 1) umma_commit(&tl->s_full[buf]);
                        }
                        __syncwarp();
                    }
                }
            }
        }
        __syncwarp();
    } else if (warp >= 8) {
        regs_down<kRegsDecode>();
        uint32_t n = 0;
        bool dead = false;
        Codes<NM> codes;
        while (!dead && w.chunk(p)) {
            w.q = ta;
            bool more = w.query(p);
            if (more) load_codes<NM>(p, w.seq, w.k * kRows, w.vis_all, n_cb, codes);
            while (more && !dead) {
                const uint32_t buf = n & 1u;
                dead = !decode_tile<NM, false>(t_s + buf * kTile, w.k * kRows, w.vis_all, n_cb, codes, tl->full[buf], nullptr, 0u,
                                               [&](int h) {
                    return n < 2 || warp_wait(&tl->freed[buf][h], ((n >> 1) - 1) & 1u, p.status, abort);
                });
                ++n;
                if (++w.k == w.end) {
                    ++w.q;
                    more = w.query(p);
                }
                if (more) load_codes<NM>(p, w.seq, w.k * kRows, w.vis_all, n_cb, codes);
            }
        }
    } else {
        regs_up<kRegsSoft>();
        const int set = warp >> 2, qd = warp & 3;
        const int row = 16 * qd + (lane >> 2), l4 = lane & 3;
        const bool active = set < sets;
        const uint32_t lane_base = (uint32_t)(32 * qd) << 16;
        uint32_t n = 0, qn = 0;
        int have = -1;
        bool dead = false;
        while (w.chunk(p)) {
            for (int i = tid; i < (w.t1 - w.t0) * 2 * kRows; i += 256) (&tl->acc[0][0][0])[i] = 0.f;
            named_bar_sync(kBarSoft, 256);
            for (w.q = ta; w.query(p); ++w.q) {
                const int qi = w.seq * p.groups + w.q;
                if (have != qi) {
                    // the Q buffer is free: this warp has seen the previous query's last S^T
                    qn ^= 1u;
                    const Group grp = group_of(p, qi);
                    load_q<NM>(p, grp, q_s, tl->qc);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&tl->q_full);
                    if (lane < 8) {   // the warp's own eight heads
                        const int hd = 8 * warp + lane;
                        tl->cl[qn][hd] =
                            make_float2(tl->qc[hd], hd < grp.heads ? -__ldcg(p.lse + grp.row0 + hd) * kLog2e : 0.f);
                        tl->hvis[qn][hd] = head_rows(p, grp, hd);
                    }
                    named_bar_sync(kBarSoft, 256);
                    have = qi;
                }
                for (int k = w.k; k < w.end; ++k, ++n) {
                    if (!active) continue;
                    const uint32_t buf = n & 1u;
                    if (!dead) dead = !warp_wait(&tl->s_full[buf], (n >> 1) & 1u, p.status, abort);
                    tc_fence_after();
                    uint32_t r[16];
                    tmem_ld_rows16(tmem + lane_base + 64u * buf + 32u * (uint32_t)set, r);
                    tmem_ld_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&tl->s_free[buf]);
                    // probabilities of the thread's two rows, summed over its heads, then over the four lanes of a row
                    float a = 0.f, b = 0.f;
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        const int hd = 32 * set + 8 * g + 2 * l4;
                        const float4 v = *reinterpret_cast<const float4*>(&tl->cl[qn][hd]);
                        const float a0 = fast_exp2(fmaf(__uint_as_float(r[4 * g]), v.x, v.y));
                        const float a1 = fast_exp2(fmaf(__uint_as_float(r[4 * g + 1]), v.z, v.w));
                        const float b0 = fast_exp2(fmaf(__uint_as_float(r[4 * g + 2]), v.x, v.y));
                        const float b1 = fast_exp2(fmaf(__uint_as_float(r[4 * g + 3]), v.z, v.w));
                        const int2 hv = *reinterpret_cast<const int2*>(&tl->hvis[qn][hd]);
                        const int j = k * kRows + row;
                        a += (hv.x > j ? a0 : 0.f) + (hv.y > j ? a1 : 0.f);
                        b += (hv.x > j + 8 ? b0 : 0.f) + (hv.y > j + 8 ? b1 : 0.f);
                    }
#pragma unroll
                    for (int o = 1; o <= 2; o <<= 1) {
                        a += __shfl_xor_sync(kWarpFull, a, o);
                        b += __shfl_xor_sync(kWarpFull, b, o);
                    }
                    if (l4 < 2 && !dead) {   // lane 0 of the four: the first row, lane 1: the second
                        tl->acc[k - w.t0][set][row + 8 * l4] += l4 ? b : a;
                    }
                }
            }
            named_bar_sync(kBarSoft, 256);
            for (int i = tid; i < (w.t1 - w.t0) * kRows; i += 256) {
                const int j = w.t0 * kRows + i;
                if (j < w.vis_all) {
                    const float v = tl->acc[i / kRows][0][i % kRows] + tl->acc[i / kRows][1][i % kRows];
                    if (p.w_split > 1) p.w_part[((int64_t)split * p.B + w.seq) * p.n_rows + j] = v;
                    else p.row_weight[(int64_t)w.seq * p.row_weight_bstride + j] += v;
                }
            }
            named_bar_sync(kBarSoft, 256);
        }
    }

    tc_fence_before();
    __syncthreads();
    if (*abort) {
        const uint64_t t0 = global_timer_ns();
        while (global_timer_ns() - t0 < 50000ull) {
        }
    }
    if (warp == 16) {
        tc_fence_after();
        tmem_dealloc(tmem, 128);
    }
}

// Row weights from the kept scores (in units of log2, as the softmax threads held them): block (x, b) takes `per` tiles
// of sequence b and adds each one's query groups in order.  Per score 4 bytes are read and one 2^x taken.
__global__ void __launch_bounds__(256, 6) row_weight_scores_kernel(const AttnFp4Params p, int per) {
    __shared__ float part[2][kRows];
    __shared__ int hvis[kScoreQueries][64];    // [group] per head: its visible rows
    __shared__ float lse[kScoreQueries][64];   // in log2; read once per block: every block of a sequence wants the same
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int set = warp >> 2, row = 16 * (warp & 3) + (lane >> 2), l4 = lane & 3;
    const bool active = 32 * set < p.pack * p.h;
    const int tiles = (p.n_rows + kRows - 1) / kRows;
    griddep_wait();
    const int b = blockIdx.y;
    const int vis_all = visible_rows(p, b, p.s - 1);
    int t = blockIdx.x * per;
    const int end = min(t + per, (vis_all + kRows - 1) / kRows);
    if (t >= end) return;
    float4 v[4];
    auto load = [&](int tt, int kk) {
        const int64_t q = (int64_t)b * p.groups + kk;
        const float4* sc = reinterpret_cast<const float4*>(p.scores) + ((q * tiles + tt) * 8 + warp) * 128 + lane;
#pragma unroll
        for (int g = 0; g < 4; ++g) v[g] = __ldcs(sc + 32 * g);
    };
    // the groups see ever more rows: those from the first one on that sees the tile's first row
    auto first = [&](int tt, int kk) {
        while (group_rows(p, b, kk) <= tt * kRows) ++kk;
        return kk;
    };
    int k0 = first(t, 0), k = k0;
    if (active) load(t, k);
    for (int i = tid; i < p.groups * 64; i += 256) {
        const int hd = i & 63;
        const Group grp = group_of(p, b * p.groups + (i >> 6));
        lse[i >> 6][hd] = hd < grp.heads ? __ldcg(p.lse + grp.row0 + hd) * kLog2e : 0.f;
        hvis[i >> 6][hd] = head_rows(p, grp, hd);
    }
    __syncthreads();
    while (t < end) {
        float sum0 = 0.f, sum1 = 0.f;
        const int k_next = t + 1 < end ? first(t + 1, k0) : 0;
        if (active)
            for (k = k0; k < p.groups; ++k) {
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const int hd = 32 * set + 8 * g + 2 * l4, j = t * kRows + row;
                    const float2 l = *reinterpret_cast<const float2*>(&lse[k][hd]);
                    const int2 hv = *reinterpret_cast<const int2*>(&hvis[k][hd]);
                    sum0 += (hv.x > j ? fast_exp2(v[g].x - l.x) : 0.f) + (hv.y > j ? fast_exp2(v[g].y - l.y) : 0.f);
                    sum1 += (hv.x > j + 8 ? fast_exp2(v[g].z - l.x) : 0.f) + (hv.y > j + 8 ? fast_exp2(v[g].w - l.y) : 0.f);
                }
                if (k + 1 < p.groups) load(t, k + 1);
                else if (t + 1 < end) load(t + 1, k_next);
            }
#pragma unroll
        for (int o = 1; o <= 2; o <<= 1) {
            sum0 += __shfl_xor_sync(kWarpFull, sum0, o);
            sum1 += __shfl_xor_sync(kWarpFull, sum1, o);
        }
        if (l4 == 0) {
            part[set][row] = sum0;
            part[set][row + 8] = sum1;
        }
        __syncthreads();
        if (tid < kRows && t * kRows + tid < vis_all)
            p.row_weight[(int64_t)b * p.row_weight_bstride + t * kRows + tid] += part[0][tid] + part[1][tid];
        __syncthreads();
        ++t;
        k0 = k_next;
    }
}

// The query splits' partial row weights, added in order; block (x, b) takes rows of sequence b.
__global__ void __launch_bounds__(256) row_weight_add_kernel(const AttnFp4Params p) {
    const int b = blockIdx.y;
    griddep_wait();
    const int vis = visible_rows(p, b, p.s - 1);
    for (int j = blockIdx.x * 256 + threadIdx.x; j < vis; j += gridDim.x * 256) {
        float v = 0.f;
        for (int k = 0; k < p.w_split; ++k) v += __ldcg(p.w_part + ((int64_t)k * p.B + b) * p.n_rows + j);
        p.row_weight[(int64_t)b * p.row_weight_bstride + j] += v;
    }
}

template <class... T>
cudaError_t launch_after(void (*kernel)(T...), dim3 grid, int threads, size_t smem, cudaStream_t stream, T... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace

AttnFp4Plan attn_fp4_plan(int B, int s, int h, int n_rows, int num_sms) {
    AttnFp4Plan l;
    // Few heads: as many queries of a sequence as fill the 64 rows of Q share a tile, which costs the same for any number
    // of heads (2048 x 16 heads over 2048 rows 659 -> 235 us, 131,072 queries of one head over 20 rows 3853 -> 80).
    l.pack = h <= 32 ? 64 / h : 1;
    if (l.pack > s) l.pack = s;
    const int groups = l.groups = (s + l.pack - 1) / l.pack;
    const int64_t tiles = ((int64_t)n_rows + kRows - 1) / kRows;
    const int64_t all = tiles * B;                                   // row tiles at most
    const int64_t list = all * groups > 0 ? all * groups : 1;
    l.grid = (int)(list < num_sms ? list : num_sms);
    // Row weights: loading a query costs as much as two of its tiles, so a CTA takes about kWTiles tiles of each and
    // the CTAs that this leaves over take other queries (never fewer with more SMs: the workspace counts on it); with
    // few tiles every CTA takes them all.
    int64_t split = all >= 2 * kWTiles ? num_sms * kWTiles / all : num_sms;
    const int64_t most = groups < num_sms ? groups : num_sms;
    split = split > most ? most : split < 1 ? 1 : split;
    const int64_t share = (groups + split - 1) / split;
    split = (groups + share - 1) / share;                            // the same share with fewer CTAs
    l.w_split = (int)split;
    const int64_t per = num_sms / split;
    l.w_grid = (int)(split * (all < per ? (all > 0 ? all : 1) : per));
    // Keeping the scores (256 bytes a row, next to the 288 of its codes) costs less than computing them again: row
    // weights of 32 x 1, 16 x 2 and 4 x 8 queries over 16384 rows 42, 42 and 38 us, computed again 92, 90 and 83; of 8
    // queries over 1024 rows 7 and 9 us.  Many queries would ask for too large a workspace and, with few rows, for too
    // few blocks.
    l.score_bytes = groups > kScoreQueries || tiles * groups > kScoreTiles / B ? 0 : (size_t)(tiles * groups * B) * kRows * 64 * 4;
    return l;
}

namespace {
template <int NM>
cudaError_t launch_nm(const AttnFp4Params& p, cudaStream_t stream) {
    const int nq = p.B * p.groups;
    size_t smem = attn_smem(p.d);
    auto* kernel = p.pack > 1 ? attn_fp4_kernel<NM, kPacks> : p.scores ? attn_fp4_kernel<NM, kKeeps> : attn_fp4_kernel<NM, kPlain>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    kernel<<<p.grid, kThreads, smem, stream>>>(p);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    const int parts = p.grid / nq + 1;   // of a query, when they are alike
    const unsigned mx = (unsigned)(nq < p.grid ? nq : p.grid), mh = (unsigned)(p.pack * p.h);
    e = parts > 16  ? launch_after(merge_kernel<16, 32>, dim3(mx, mh, (unsigned)NM), 512, 0, stream, p)
        : parts > 4 ? launch_after(merge_kernel<2, 128>, dim3(mx, mh), 256, 0, stream, p)
                    : launch_after(merge_kernel<1, 128>, dim3(mx, mh), 128, 0, stream, p);
    if (e != cudaSuccess || !p.row_weight || p.n_rows == 0) return e;
    // (B fits a grid's y: scores are kept up to kScoreTiles sequences, and split queries mean at most num_sms kWTiles / 2)
    if (p.scores) {
        const int tiles = (p.n_rows + kRows - 1) / kRows, per = (int64_t)tiles * p.B >= kManyTiles ? 4 : 1;
        return launch_after(row_weight_scores_kernel,
                            dim3((unsigned)((tiles + per - 1) / per), (unsigned)p.B), 256, 0, stream, p, per);
    }
    smem = row_weight_smem(p.d);
    e = cudaFuncSetAttribute(row_weight_kernel<NM>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    e = launch_after(row_weight_kernel<NM>, dim3((unsigned)p.w_grid), kThreads, smem, stream, p);
    if (e != cudaSuccess || p.w_split == 1) return e;
    const int blocks = (p.n_rows + 255) / 256;
    return launch_after(row_weight_add_kernel, dim3((unsigned)(blocks < 64 ? blocks : 64), (unsigned)p.B), 256, 0, stream,
                        p);
}
}  // namespace

cudaError_t launch_attn_fp4(const AttnFp4Params& p, cudaStream_t stream) {
    if (p.B * p.s == 0) return cudaSuccess;
    switch ((p.d + 127) / 128) {
        case 1: return launch_nm<1>(p, stream);
        case 2: return launch_nm<2>(p, stream);
        case 3: return launch_nm<3>(p, stream);
        default: return launch_nm<4>(p, stream);
    }
}

}  // namespace sti
