// attn_fp4.cu -- attention over every visible row of a 4-bit cache, and the attention each row received.
//
// For query (b, t), vis = clamp((start_pos + t + 1) // ratio - dropped, 0, n_rows) rows are visible:
//   s_hj = softmax_scale q_h . k_j,  L_h = ln(sum_j e^{s_hj} + e^{sink_h} + e^{prev_lse_h})
//   out_h = (sum_j e^{s_hj} k_j + e^{prev_lse_h} prev_out_h) / e^{L_h}
//   row_weight[b, j] += sum_{t, h} e^{s_hj - L_h}
// k_j = the row's E2M1 codes times its E4M3 scale per 16, serving as key and value for all heads.
//
// attn_fp4_kernel: persistent CTAs, one per SM; the queries' 128-row tiles form one long list that is cut
// into equal contiguous pieces, so a few long queries, many short ones and ragged batches all fill
// the GPU.  A query whose tiles fall to several CTAs leaves one fp32 partial per CTA; merge_kernel joins
// them.  Roles (640 threads):
//   * warps 8..15 load the rows' codes into registers and decode them into the shared tile, each its own
//     d-block (128 dims), as soon as the previous tile's PV releases it;
//   * warp -4 issues the MMAs:  S^T = tile . Q^T (M = 128 rows, N = heads), O^T += V^T . P^T (M = 128
//     dims per block, K = 128 rows; the same tile read as an MN-major operand);
//   * warps 0..7 load Q, run the online softmax (thread = row, two groups of 32 heads; the running
//     maxima move only when a score passes them by 2^8) and write the outputs.
// The decode runs in its own warps so that it overlaps the MMAs and the softmax.
//
// f16 operands: an E2M1 value (2 significant bits) times an E4M3 value (4) is exact in f16 (at most 6
// significant bits, magnitudes 2^-10 .. 2688), so the tile is exact.  Q is bf16: each head's values are
// scaled by a power of two that puts its largest into [2^12, 2^13) and is undone in fp32 with the
// softmax scale; an element down to 2^-26 of the head's largest keeps all its 8 bits, smaller ones are
// off by less than 2^-37 of the largest.  P is rounded to f16 (2^-11) for the PV product; its sum l is
// taken before the rounding, in fp32.
//
// row_weight_kernel (only when asked for): p = e^{s - L} needs the final L, so it runs after the merge and
// recomputes S^T (the tile's codes are read again, mostly from L2: cheaper than storing 4 bytes per
// score).  Each row tile belongs to one CTA, which adds the queries in order: no atomics.  When there are
// fewer tiles than SMs, queries split over CTAs and a last kernel adds the parts in order.
#include <cuda_fp16.h>
#include <math.h>
#include <stddef.h>

#include "sti_attn_util.cuh"
#include "sti_internal.h"
#include "sti_ptx.cuh"

namespace sti {
namespace {

constexpr int kThreads = 640;                  // warps 17..19 only complete the MMA warp's warpgroup
// registers per thread after the roles' setmaxnreg: 256 x 128 + 256 x 80 + 128 x 64 = 61,440, the
// 640 x 96 of the launch
constexpr int kRegsSoft = 128, kRegsDecode = 80, kRegsMma = 64;
constexpr int kRows = 128;                     // rows per tile
constexpr uint32_t kQBlk = 64 * 128;           // a Q column block: 64 heads x 64 dims
constexpr uint32_t kTBlk = kRows * 128;        // a tile column block: 128 rows x 64 dims
constexpr uint32_t kTmS = 0;                   // TMEM columns of S^T
constexpr uint32_t kTmO = 64;                  // O^T d-block m at [64 + 64 m, 128 + 64 m)
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.69314718055994531f;
constexpr int kWTiles = 16;                    // row weights: tiles per chunk (accumulators in shared memory)

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
// S^T (+)= tile . Q^T over one d-block (two column blocks).  a, b: low descriptor words of the tile and Q.
__device__ __forceinline__ void qk_blocks(bool first, uint32_t s_tmem, uint32_t a, uint32_t b, uint32_t hi,
                                          uint32_t idesc) {
    a = opaque(a);
    b = opaque(b);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const uint32_t ak = a + (k >> 2) * (kTBlk / 16) + 2 * (k & 3), bk = b + (k >> 2) * (kQBlk / 16) + 2 * (k & 3);
        if (first && k == 0) umma<false>(s_tmem, ak, hi, bk, hi, idesc);
        else umma<true>(s_tmem, ak, hi, bk, hi, idesc);
    }
}
// O^T (+)= V^T . P^T: one d-block, eight K steps.
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
    const int64_t v = ((int64_t)__ldg(p.start_pos + b) + t + 1) / p.ratio - (p.dropped ? __ldg(p.dropped + b) : 0);
    return v < 0 ? 0 : v > p.n_rows ? p.n_rows : (int)v;
}

struct Work {           // this CTA's piece of the list
    long long lo, hi;   // tiles [lo, hi) of the list
    int q, off;         // the first one: tile `off` of query q
    long long total;
    int ctas;           // CTAs that have tiles
};

struct Seg {            // a run of one query's tiles
    int q, b, vis, nt, t0, t1;
};

// Walk the piece: query by query, those without a visible row skipped.
struct Walk {
    long long pos, hi;
    int q, off;
    __device__ __forceinline__ explicit Walk(const Work& w) : pos(w.lo), hi(w.hi), q(w.q), off(w.off) {}
    __device__ __forceinline__ bool next(const AttnFp4Params& p, Seg& s) {
        while (pos < hi) {
            s.q = q;
            s.b = q / p.s;
            s.vis = visible_rows(p, s.b, q - s.b * p.s);
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

// Decoding: the 8 decoding warps are dealt out to the NM d-blocks, so that each d-block is refilled by its
// own warps as soon as the PV releases it (one group walking from block to block pays the latency of its
// stores, the fence and the next wait on the way: 850 cycles per d-block).  A d-block of a tile is 256 units
// of one row x one column block (64 dims: 32 code bytes, 4 scale bytes); a thread takes U of them.
template <int NM>
struct Deal {
    static constexpr int kWarps = NM == 1 ? 8 : NM == 2 ? 4 : 2;   // per d-block (NM == 3: two warps idle)
    static constexpr int U = 8 / kWarps;
};
template <int U>
struct Codes {
    uint4 c[U][2];
    uint32_t s[U];
};

// Unit u of thread `lt` of d-block m's warps.
template <int NM>
__device__ __forceinline__ void unit_of(int u, int lt, int m, int& row, int& cb) {
    const int i = u * 32 * Deal<NM>::kWarps + lt;
    row = i & 127;
    cb = 2 * m + (i >> 7);
}

template <int NM>
__device__ __forceinline__ void load_units(const AttnFp4Params& p, int b, int row0, int vis, int m, int lt, int n_cb,
                                           Codes<Deal<NM>::U>& r) {
    const uint8_t* cb0 = p.codes + (int64_t)b * p.codes_bstride;
    const uint8_t* sb0 = p.scales + (int64_t)b * p.scales_bstride;
#pragma unroll
    for (int u = 0; u < Deal<NM>::U; ++u) {
        int row, cb;
        unit_of<NM>(u, lt, m, row, cb);
        row += row0;
        if (row < vis && cb < n_cb) {
            const uint8_t* cr = cb0 + (int64_t)row * (p.d / 2) + cb * 32;
            r.c[u][0] = __ldg(reinterpret_cast<const uint4*>(cr));
            r.c[u][1] = __ldg(reinterpret_cast<const uint4*>(cr + 16));
            r.s[u] = __ldg(reinterpret_cast<const uint32_t*>(sb0 + (int64_t)row * (p.d / 16) + cb * 4));
        }
    }
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

// 64 elements of row fr (one column block at dst) from their codes; zeros when the row is not visible.
__device__ __forceinline__ void decode_block(uint8_t* dst, int fr, bool valid, const uint4& c0, const uint4& c1,
                                             uint32_t s) {
    if (valid) {
        uint32_t h01, h23;   // the four scales as f16
        asm("{\n\t.reg .b16 lo, hi;\n\t"
            "mov.b32 {lo, hi}, %2;\n\t"
            "cvt.rn.f16x2.e4m3x2 %0, lo;\n\t"
            "cvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
            : "=r"(h01), "=r"(h23)
            : "r"(s));
        const uint32_t w[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
        const uint32_t sc[4] = {__byte_perm(h01, h01, 0x1010), __byte_perm(h01, h01, 0x3232),
                                __byte_perm(h23, h23, 0x1010), __byte_perm(h23, h23, 0x3232)};
#pragma unroll
        for (int c = 0; c < 8; ++c)
            *reinterpret_cast<uint4*>(dst + ((c ^ (fr & 7)) << 4)) =
                decode8(w[c], *reinterpret_cast<const __half2*>(&sc[c >> 1]));
    } else {
#pragma unroll
        for (int c = 0; c < 8; ++c) *reinterpret_cast<uint4*>(dst + (c << 4)) = make_uint4(0, 0, 0, 0);
    }
}

template <int NM>
__device__ __forceinline__ void decode_units(uint8_t* t_s, int row0, int vis, int m, int lt, int n_cb,
                                             const Codes<Deal<NM>::U>& r) {
#pragma unroll
    for (int u = 0; u < Deal<NM>::U; ++u) {
        int row, cb;
        unit_of<NM>(u, lt, m, row, cb);
        if (cb < n_cb) decode_block(t_s + (size_t)cb * kTBlk + row * 128, row, row0 + row < vis, r.c[u][0], r.c[u][1], r.s[u]);
    }
}

// Query qi's heads as f16 into the swizzled column blocks at q_s, four threads per head, each head
// scaled by 2^f; qc[head] = scale_log2 * 2^-f.  `t`: thread of the loading group (4 threads per head).
__device__ __forceinline__ void load_q(const AttnFp4Params& p, int qi, int t, uint8_t* q_s, float* qc) {
    const int head = t >> 2, part = t & 3;
    const int n = p.d / 8;
    const bool in = head < p.h;
    const uint4* src = reinterpret_cast<const uint4*>(p.q + ((int64_t)qi * p.h + (in ? head : 0)) * p.d);
    uint32_t mx = 0;
    if (in) {
#pragma unroll 8
        for (int k = part; k < n; k += 4) {
            const uint4 v = __ldg(src + k);
            mx = __vmaxu2(mx, __vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu),
                                       __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu)));
        }
    }
    mx = max(mx & 0xFFFFu, mx >> 16);
    mx = max(mx, __shfl_xor_sync(kWarpFull, mx, 1));
    mx = max(mx, __shfl_xor_sync(kWarpFull, mx, 2));
    int f = 139 - (int)(mx >> 7);   // largest into [2^12, 2^13); mx >> 7: its exponent field
    f = f > 127 ? 127 : f;          // (-116 .. 127)
    const float up = __uint_as_float((uint32_t)(f + 127) << 23);
    // 2^-f: subnormal at f = 127
    const float down = f == 127 ? __uint_as_float(0x00400000u) : __uint_as_float((uint32_t)(127 - f) << 23);
    if (in) {
        if (part == 0) qc[head] = p.scale_log2 * down;
#pragma unroll 8
        for (int k = part; k < n; k += 4) {
            const uint4 v = __ldg(src + k);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
            uint32_t o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const __half2 x = __floats2half2_rn(__uint_as_float(w[i] << 16) * up,
                                                    __uint_as_float(w[i] & 0xFFFF0000u) * up);
                o[i] = *reinterpret_cast<const uint32_t*>(&x);
            }
            *reinterpret_cast<uint4*>(q_s + (k >> 3) * kQBlk + head * 128 + (((k & 7) ^ (head & 7)) << 4)) =
                make_uint4(o[0], o[1], o[2], o[3]);
        }
    } else if (part == 0) {
        qc[head] = 0.f;
    }
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float bf16_f(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }

// ------------------------------------------------------------------ attention

struct __align__(16) Tail {
    float2 cm[2][4][32];      // each warp's copy of its head group's (softmax scale, -running maximum)
    float qc[2][64];          // [segment parity] per head: softmax scale (log2) over its f16 scaling
    float red[2][2][4][32];   // [tile parity][group][warp]: per-warp maxima
    float lsum[2][4][32];
    Work work;
    long long scratch[kThreads / 32];
    uint64_t full[4];         // d-block m of the tile decoded: one arrival per warp
    uint64_t pv[4];           // the tile's PV of d-block m done
    uint64_t s_full, p_full, q_full;
    uint32_t tmem_base;
    int abort;
};

size_t attn_smem(int d) {
    const int n_cb = (d + 127) / 128 * 2;
    return 1024 + (size_t)n_cb * (kQBlk + kTBlk) + kRows * 128 + sizeof(Tail);
}

template <int NM>   // d-blocks of 128 dims
__global__ void __launch_bounds__(kThreads, 1) attn_fp4_kernel(const AttnFp4Params p) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const int n_cb = p.d / 64;                 // column blocks of 64 dims
    constexpr int n_m = NM;
    uint8_t* q_s = smem;                       // [2 n_m][64 heads][128 B]
    uint8_t* t_s = q_s + 2 * n_m * kQBlk;      // [2 n_m][128 rows][128 B]
    uint8_t* p_s = t_s + 2 * n_m * kTBlk;      // P^T [128 rows][64 heads] f16
    Tail* tl = reinterpret_cast<Tail*>(p_s + kRows * 128);

    // warps -4 .. -1: the MMA warp's warpgroup, 0 .. 7: softmax, 8 .. 15: decode
    const int tid = (int)threadIdx.x - 128, warp = ((int)threadIdx.x >> 5) - 4, lane = threadIdx.x & 31;
    const int nq = p.B * p.s;
    const int groups = p.h > 32 ? 2 : 1;       // groups of 32 heads
    const uint32_t n_mma = 32u * (uint32_t)groups;
    volatile int* abort = &tl->abort;

    if (warp == -4) {
        tmem_alloc(&tl->tmem_base, n_m <= 2 ? 256 : 512);
        tmem_relinquish();
    }
    if (tid == 0) {
        for (int m = 0; m < 4; ++m) {
            mbar_init(&tl->full[m], Deal<NM>::kWarps);
            mbar_init(&tl->pv[m], 1);
        }
        mbar_init(&tl->s_full, 1);
        mbar_init(&tl->p_full, 4 * groups);
        mbar_init(&tl->q_full, 4 * groups);
        tl->abort = 0;
        fence_mbar_init();
    }
    // what no thread writes later: Q rows of heads >= h, the dims past d of the last d-block
    for (int i = threadIdx.x; i < 2 * n_m * 64 * 8; i += kThreads)
        if (((i >> 3) & 63) >= p.h || (i >> 9) >= n_cb) reinterpret_cast<uint4*>(q_s)[i] = make_uint4(0, 0, 0, 0);
    if (n_cb & 1)
        for (int i = threadIdx.x; i < (int)kTBlk / 16; i += kThreads)
            reinterpret_cast<uint4*>(t_s + (size_t)n_cb * kTBlk)[i] = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
    plan_work(nq, blockIdx.x, gridDim.x, tl->scratch, &tl->work,
              [&](int q) { return (visible_rows(p, q / p.s, q % p.s) + kRows - 1) / kRows; });
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(kWarpFull, tl->tmem_base, 0);   // warp-uniform, as the compiler can see
    const Work wk = tl->work;
    griddep_launch_dependents();

    if (warp >= 8) {
        regs_down<kRegsDecode>();
        // -------------------------------------------------------------- decode: thread = (row, column block parity)
        const int m = (warp - 8) / Deal<NM>::kWarps, lt = (warp - 8) % Deal<NM>::kWarps * 32 + lane;
        if (m < NM) {
            uint32_t n = 0;
            bool dead = false;
            Walk walk(wk);
            Seg sg;
            while (!dead && walk.next(p, sg)) {
                for (int t = sg.t0; t < sg.t1 && !dead; ++t, ++n) {
                    Codes<Deal<NM>::U> r;
                    load_units<NM>(p, sg.b, t * kRows, sg.vis, m, lt, n_cb, r);
                    if (n > 0) dead = !warp_wait(&tl->pv[m], (n - 1) & 1u, p.status, abort);
                    if (dead) break;
                    decode_units<NM>(t_s, t * kRows, sg.vis, m, lt, n_cb, r);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&tl->full[m]);
                }
            }
        }
    } else if (warp < 0) {
        regs_down<kRegsMma>();
        // -------------------------------------------------------------- MMA issue
        const uint32_t idesc_qk = idesc_f16_f32(kRows, (int)n_mma, false, false);
        const uint32_t idesc_pv = idesc_f16_f32(kRows, (int)n_mma, true, true);
        // descriptors of the tile and Q (K-major), the tile (MN-major) and P^T (MN-major)
        const uint64_t dk = sdesc(smem_u32(t_s), 16, 1024, kLayoutSW128), dq = sdesc(smem_u32(q_s), 16, 1024, kLayoutSW128);
        const uint64_t dv = sdesc(smem_u32(t_s), kTBlk, 1024, kLayoutSW128);
        const uint64_t dp = sdesc(smem_u32(p_s), kRows * 128u, 1024, kLayoutSW128);
        uint32_t n = 0, qn = 0;
        Walk walk(wk);
        Seg sg;
        // the whole warp waits, one elected lane issues (so the operands stay warp-uniform)
        bool ok = warp == -4;
        auto wait = [&](uint64_t* bar, uint32_t parity) {
            ok = warp_wait(bar, parity, p.status, abort);
            tc_fence_after();
            return ok;
        };
        while (ok && walk.next(p, sg)) {
            if (!wait(&tl->q_full, qn & 1u)) break;
            ++qn;
            for (int t = sg.t0; t < sg.t1 && ok; ++t, ++n) {
#pragma unroll
                for (int m = 0; m < NM; ++m) {
                    if (!wait(&tl->full[m], n & 1u)) break;
                    if (elect_one()) {
                        qk_blocks(m == 0, tmem + kTmS, lo32(dk) + (uint32_t)m * (2 * kTBlk / 16),
                                  lo32(dq) + (uint32_t)m * (2 * kQBlk / 16), hi32(dk), idesc_qk);
                        if (m == NM - 1) umma_commit(&tl->s_full);
                    }
                    __syncwarp();
                }
                if (!ok) break;
                if (!wait(&tl->p_full, n & 1u)) break;
                if (elect_one()) {
#pragma unroll
                    for (int m = 0; m < NM; ++m) {
                        const uint32_t o = tmem + kTmO + 64u * (uint32_t)m, a = lo32(dv) + (uint32_t)m * (2 * kTBlk / 16);
                        if (t == sg.t0) pv_block<true>(o, a, hi32(dv), lo32(dp), hi32(dp), idesc_pv);
                        else pv_block<false>(o, a, hi32(dv), lo32(dp), hi32(dp), idesc_pv);
                        umma_commit(&tl->pv[m]);
                    }
                }
                __syncwarp();
            }
        }
        __syncwarp();
    } else {
        regs_up<kRegsSoft>();
        if (warp < 4 * groups) {
        // -------------------------------------------------------------- Q, softmax, outputs
        const int set = warp >> 2, qd = warp & 3;
        const int row = 32 * qd + lane;
        const uint32_t lane_base = (uint32_t)(32 * qd) << 16;
        const uint32_t bar_set = 1u + (uint32_t)set;
        const uint32_t n_soft = 128u * (uint32_t)groups;
        uint32_t n = 0;
        int qbuf = 0;
        bool dead = false;
        float m_run = -INFINITY;   // lane l: head 32 set + l
        float l_thr[32];

        auto mwait = [&](uint64_t* bar, uint32_t parity) {
            if (!dead) dead = !warp_wait(bar, parity, p.status, abort);
        };

        // One tile's probabilities.  cm holds (c, -m) of each head: c the softmax scale (log2) over the head's f16
        // scaling, m its running maximum, so y = S c - m is one FMA and 2^y the probability.
        auto softmax = [&](bool valid, bool first) {
            mwait(&tl->s_full, n & 1u);
            tc_fence_after();
            valid = valid && !dead;
            const float2* cm = &tl->cm[set][qd][0];
            uint32_t r[32];
            tmem_ld32(tmem + lane_base + kTmS + 32u * (uint32_t)set, r);
            tmem_ld_wait();
            float y[32];
            float top = -INFINITY;
#pragma unroll
            for (int c = 0; c < 16; ++c) {
                const float4 v = *reinterpret_cast<const float4*>(cm + 2 * c);
                y[2 * c] = fmaf(__uint_as_float(r[2 * c]), v.x, v.y);
                y[2 * c + 1] = fmaf(__uint_as_float(r[2 * c + 1]), v.z, v.w);
                top = fmaxf(top, fmaxf(y[2 * c], y[2 * c + 1]));
            }
            // the maxima stay unless a visible score passes its head's by 2^8
            const bool need = !named_bar_and(bar_set, 128, !(first || (valid && top > 8.f)));
            if (need) {
                {
                    float v2[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i) v2[i] = valid ? y[i] : -INFINITY;
                    warp_reduce_scatter_n<32, true>(v2);
                    tl->red[n & 1u][set][qd][lane] = v2[0];
                }
                named_bar_sync(bar_set, 128);
                const float* rr = &tl->red[n & 1u][set][0][0];
                const float old = -cm[lane].y;    // what y is relative to
                const float mt = fmaxf(fmaxf(rr[lane], rr[32 + lane]), fmaxf(rr[64 + lane], rr[96 + lane])) + old;
                const float m_new = (m_run == -INFINITY || mt > m_run + 8.f) ? fmaxf(m_run, mt) : m_run;
                const float alpha = (m_new == m_run) ? 1.f : exp2f(m_run - m_new);
                m_run = m_new;
                // a head without any finite score keeps -inf; its exponents are taken from 0, so that NaN
                // scores show in its output
                const float neg = m_new == -INFINITY ? 0.f : -m_new;
                __syncwarp();
                tl->cm[set][qd][lane].y = neg;
                __syncwarp();
                tmem_ld32(tmem + lane_base + kTmS + 32u * (uint32_t)set, r);   // again: y of the new maxima
                tmem_ld_wait();
#pragma unroll
                for (int c = 0; c < 16; ++c) {
                    const float4 v = *reinterpret_cast<const float4*>(cm + 2 * c);
                    y[2 * c] = fmaf(__uint_as_float(r[2 * c]), v.x, v.y);
                    y[2 * c + 1] = fmaf(__uint_as_float(r[2 * c + 1]), v.z, v.w);
                }
                if (!first && !dead && __any_sync(kWarpFull, alpha != 1.f)) {
#pragma unroll 1
                    for (int m = 0; m < n_m; ++m) {
                        const uint32_t ta = tmem + lane_base + kTmO + 64u * (uint32_t)m + 32u * (uint32_t)set;
#pragma unroll 1
                        for (int hf = 0; hf < 2; ++hf) {
                            uint32_t o[16];
                            tmem_ld16(ta + 16u * (uint32_t)hf, o);
                            tmem_ld_wait();
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                o[i] = __float_as_uint(__uint_as_float(o[i]) * __shfl_sync(kWarpFull, alpha, 16 * hf + i));
                            tmem_st16(ta + 16u * (uint32_t)hf, o);
                        }
                    }
                    tmem_st_wait();
#pragma unroll
                    for (int i = 0; i < 32; ++i) l_thr[i] *= __shfl_sync(kWarpFull, alpha, i);
                }
            }
            uint8_t* prow = p_s + row * 128;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                uint32_t pk[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int i = 8 * c + 2 * j;
                    const float e0 = valid ? fast_exp2(y[i]) : 0.f, e1 = valid ? fast_exp2(y[i + 1]) : 0.f;
                    l_thr[i] += e0;
                    l_thr[i + 1] += e1;
                    pk[j] = pack_f16x2(e0, e1);
                }
                *reinterpret_cast<uint4*>(prow + (((4 * set + c) ^ (row & 7)) << 4)) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
            }
            fence_proxy_async_smem();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&tl->p_full);
        };

        // a segment's O^T and sums: the query's output when the segment holds all its tiles, else a partial
        auto epilogue = [&](const Seg& sg) {
            mwait(&tl->pv[n_m - 1], (n - 1) & 1u);
            tc_fence_after();
            {
                float v2[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) v2[i] = l_thr[i];
                warp_reduce_scatter_n<32, false>(v2);
                tl->lsum[set][qd][lane] = v2[0];
            }
            named_bar_sync(bar_set, 128);
            const float* ls = &tl->lsum[set][0][0];
            const float lt = (ls[lane] + ls[32 + lane]) + (ls[64 + lane] + ls[96 + lane]);
            const int hh = 32 * set + lane;
            if (sg.t0 > 0 || sg.t1 < sg.nt) {
                const int slot = 2 * (int)blockIdx.x + (sg.t0 == 0 ? 1 : 0);
                if (qd == 0) p.part_ml[slot * 64 + hh] = make_float2(m_run, lt);
                float* po = p.part_o + (int64_t)slot * p.h * p.d;
#pragma unroll 1
                for (int m = 0; m < n_m; ++m) {
                    const int dd = 128 * m + 32 * qd + lane;
                    uint32_t r[32];
                    tmem_ld32(tmem + lane_base + kTmO + 64u * (uint32_t)m + 32u * (uint32_t)set, r);
                    tmem_ld_wait();
                    if (dd < p.d) {
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (32 * set + i < p.h) po[(32 * set + i) * p.d + dd] = __uint_as_float(r[i]);
                    }
                }
            } else {
                float inv = 0.f, wp = 0.f;
                if (hh < p.h) {
                    // everything relative to the largest of the running maximum, the sink and prev_lse
                    const float sk = p.sink ? __ldg(p.sink + hh) * kLog2e : -INFINITY;
                    const float pl = p.prev_lse ? __ldg(p.prev_lse + (int64_t)sg.q * p.h + hh) * kLog2e : -INFINITY;
                    float mx = fmaxf(m_run, fmaxf(sk, pl));
                    if (mx == -INFINITY) mx = 0.f;
                    const float f = m_run == -INFINITY ? exp2f(-mx) : exp2f(m_run - mx);
                    const float ep = exp2f(pl - mx);
                    const float den = lt * f + exp2f(sk - mx) + ep;
                    inv = f / den;
                    wp = ep / den;
                    if (p.lse && qd == 0) p.lse[(int64_t)sg.q * p.h + hh] = (mx + log2f(den)) * kLn2;
                }
                float invh[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) invh[i] = __shfl_sync(kWarpFull, inv, i);
                uint16_t* orow = p.out + (int64_t)sg.q * p.h * p.d;
                uint16_t* stg = reinterpret_cast<uint16_t*>(p_s) + warp * 32 * 32;   // this warp's [32 heads][32 dims]
                const bool odd = (lane & 1) != 0;
#pragma unroll 1
                for (int m = 0; m < n_m; ++m) {
                    const int dd = 128 * m + 32 * qd + lane;
                    uint32_t r[32];
                    tmem_ld32(tmem + lane_base + kTmO + 64u * (uint32_t)m + 32u * (uint32_t)set, r);
                    tmem_ld_wait();
                    float vv[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i) vv[i] = dead ? 0.f : __uint_as_float(r[i]) * invh[i];
                    if (p.prev_out) {
                        const uint16_t* pr = p.prev_out + (int64_t)sg.q * p.h * p.d + dd;
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            const float w = __shfl_sync(kWarpFull, wp, i);
                            if (w != 0.f && 32 * set + i < p.h && dd < p.d)   // weight 0: prev_out is not used
                                vv[i] += w * bf16_f(pr[(32 * set + i) * p.d]);
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 32; i += 2) {
                        const float send = odd ? vv[i] : vv[i + 1];
                        const float recv = __shfl_xor_sync(kWarpFull, send, 1);
                        const uint32_t pk = odd ? pack_bf16x2(recv, vv[i + 1]) : pack_bf16x2(vv[i], recv);
                        *reinterpret_cast<uint32_t*>(stg + (i + (odd ? 1 : 0)) * 32 + (lane & ~1)) = pk;
                    }
                    __syncwarp();
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int c = lane + 32 * k;
                        const int hw = 32 * set + (c >> 2);
                        const int dw = 128 * m + 32 * qd + 8 * (c & 3);
                        if (hw < p.h && dw < p.d)
                            *reinterpret_cast<uint4*>(orow + (int64_t)hw * p.d + dw) =
                                *reinterpret_cast<const uint4*>(stg + c * 8);
                    }
                    __syncwarp();
                }
            }
            named_bar_sync(3, n_soft);   // the staging area is the P^T buffer of every warp
        };

        // queries without a visible row
        for (int q = blockIdx.x; q < nq; q += gridDim.x) {
            if (visible_rows(p, q / p.s, q % p.s) > 0) continue;
            for (int hh = warp; hh < p.h; hh += 4 * groups) {
                const int64_t at = (int64_t)q * p.h + hh;
                const float pl = p.prev_lse ? p.prev_lse[at] : -INFINITY;
                if (p.lse && lane == 0) p.lse[at] = pl;
                for (int k = lane; k < p.d / 8; k += 32) {
                    uint4 v = make_uint4(0, 0, 0, 0);
                    if (pl != -INFINITY) v = reinterpret_cast<const uint4*>(p.prev_out + at * p.d)[k];
                    reinterpret_cast<uint4*>(p.out + at * p.d)[k] = v;
                }
            }
        }

        Walk walk(wk);
        Seg sg, prev;
        bool pending = false;
        int2 rec = make_int2(-1, 0);
        while (walk.next(p, sg)) {
            // the Q buffer is free: this thread has seen the last S^T of the previous query
            // (another warp may still scale that S^T: qc has two buffers)
            qbuf ^= 1;
            load_q(p, sg.q, tid, q_s, tl->qc[qbuf]);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&tl->q_full);
            if (pending) epilogue(prev);
            named_bar_sync(3, n_soft);
            m_run = -INFINITY;
            tl->cm[set][qd][lane] = make_float2(tl->qc[qbuf][32 * set + lane], 0.f);
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 32; ++i) l_thr[i] = 0.f;
            for (int t = sg.t0; t < sg.t1; ++t, ++n) softmax(t * kRows + row < sg.vis, t == sg.t0);
            prev = sg;
            pending = true;
            if (sg.t0 == 0 && sg.t1 < sg.nt) {
                const long long last = walk.pos - sg.t1 + sg.nt - 1;   // list position of the query's last tile
                int c = (int)(last * wk.ctas / wk.total);
                while ((long long)(c + 1) * wk.total / wk.ctas <= last) ++c;
                while ((long long)c * wk.total / wk.ctas > last) --c;
                rec = make_int2(sg.q, c);
            }
        }
        if (pending) epilogue(prev);
        if (tid == 0) p.rec[blockIdx.x] = rec;
        }
    }

    tc_fence_before();
    __syncthreads();
    if (*abort) {   // a wait gave up: let the MMAs in flight finish before the CTA's memory goes
        const uint64_t t0 = global_timer_ns();
        while (global_timer_ns() - t0 < 50000ull) {
        }
    }
    if (warp == -4) {
        tc_fence_after();
        tmem_dealloc(tmem, n_m <= 2 ? 256 : 512);
    }
}

// ------------------------------------------------------------------ joining split queries

// Block (x, head): the split queries that start in CTAs x, x + gridDim.x, ... of the attention kernel.
// Thread i takes dims 4i .. 4i + 3.
__global__ void __launch_bounds__(128) merge_kernel(const AttnFp4Params p) {
    __shared__ float fac[1024];
    __shared__ float stat[2];
    const int hh = blockIdx.y, tid = threadIdx.x, lane = tid & 31;
    griddep_wait();
    griddep_launch_dependents();
    for (int c = blockIdx.x; c < p.grid; c += gridDim.x) {
        const int2 rec = p.rec[c];
        if (rec.x < 0) continue;
        const int parts = rec.y - c + 1;   // slots 2c + 1, 2 (c + 1), 2 (c + 2), ...
        auto slot = [&](int i) { return i == 0 ? 2 * c + 1 : 2 * (c + i); };
        const int64_t at = (int64_t)rec.x * p.h + hh;
        const float sk = p.sink ? __ldg(p.sink + hh) * kLog2e : -INFINITY;
        const float pl = p.prev_lse ? p.prev_lse[at] * kLog2e : -INFINITY;
        if (tid < 32) {
            float mx = fmaxf(sk, pl);
            for (int i = lane; i < parts; i += 32) mx = fmaxf(mx, p.part_ml[slot(i) * 64 + hh].x);
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kWarpFull, mx, o));
            if (mx == -INFINITY) mx = 0.f;
            float l = 0.f;
            for (int i = lane; i < parts; i += 32) {
                const float2 ml = p.part_ml[slot(i) * 64 + hh];
                const float f = exp2f((ml.x == -INFINITY ? 0.f : ml.x) - mx);
                fac[i] = f;
                l += ml.y * f;
            }
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) l += __shfl_xor_sync(kWarpFull, l, o);
            const float ep = exp2f(pl - mx);
            const float den = l + exp2f(sk - mx) + ep;
            if (lane == 0) {
                stat[0] = 1.f / den;
                stat[1] = ep / den;
                if (p.lse) p.lse[at] = (mx + log2f(den)) * kLn2;
            }
        }
        __syncthreads();
        if (4 * tid < p.d) {
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
            for (int i = 0; i < parts; ++i) {
                const float4 v = __ldcg(reinterpret_cast<const float4*>(
                    p.part_o + ((int64_t)slot(i) * p.h + hh) * p.d + 4 * tid));
                const float f = fac[i];
                o.x += f * v.x;
                o.y += f * v.y;
                o.z += f * v.z;
                o.w += f * v.w;
            }
            const float inv = stat[0], wp = stat[1];
            o.x *= inv;
            o.y *= inv;
            o.z *= inv;
            o.w *= inv;
            if (wp != 0.f && p.prev_out) {
                const uint2 v = *reinterpret_cast<const uint2*>(p.prev_out + at * p.d + 4 * tid);
                o.x += wp * __uint_as_float(v.x << 16);
                o.y += wp * __uint_as_float(v.x & 0xFFFF0000u);
                o.z += wp * __uint_as_float(v.y << 16);
                o.w += wp * __uint_as_float(v.y & 0xFFFF0000u);
            }
            *reinterpret_cast<uint2*>(p.out + at * p.d + 4 * tid) =
                make_uint2(pack_bf16x2(o.x, o.y), pack_bf16x2(o.z, o.w));
        }
        __syncthreads();
    }
}

// ------------------------------------------------------------------ row weights

struct __align__(16) WTail {
    float2 cl[2][64];                // [query parity] per head: (softmax scale over the f16 scaling, -lse in log2)
    float qc[64];
    float acc[kWTiles][2][kRows];    // [tile of the chunk][head group][row]
    Work work;
    long long scratch[kThreads / 32];
    uint64_t full[4];
    uint64_t freed[4];               // the tile's QK has read d-block m
    uint64_t s_full[2];              // [tile parity] S^T done
    uint64_t s_free[2];              // S^T read
    uint64_t q_full;
    uint32_t tmem_base;
    int abort;
};

size_t row_weight_smem(int d) {
    const int n_cb = (d + 127) / 128 * 2;
    return 1024 + (size_t)n_cb * (kQBlk + kTBlk) + sizeof(WTail);
}

// The CTA's tiles in chunks of one sequence (at most kWTiles tiles); within a chunk, for each of the CTA's
// queries, the chunk's tiles.  Items of the list are the sequences.
struct WWalk {
    long long pos, hi;
    int b, off;
    __device__ __forceinline__ explicit WWalk(const Work& w) : pos(w.lo), hi(w.hi), b(w.q), off(w.off) {}
    __device__ __forceinline__ bool next(const AttnFp4Params& p, Seg& s) {
        while (pos < hi) {
            s.b = b;
            s.vis = visible_rows(p, b, p.s - 1);
            s.nt = (s.vis + kRows - 1) / kRows;
            s.t0 = off;
            s.t1 = (long long)(s.nt - off) < hi - pos ? s.nt : off + (int)(hi - pos);
            if (s.t1 - s.t0 > kWTiles) s.t1 = s.t0 + kWTiles;
            pos += s.t1 - s.t0;
            off = s.t1;
            if (off >= s.nt) {
                ++b;
                off = 0;
            }
            if (s.t1 > s.t0) return true;
        }
        return false;
    }
};

template <int NM>
__global__ void __launch_bounds__(kThreads, 1) row_weight_kernel(const AttnFp4Params p) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const int n_cb = p.d / 64;
    constexpr int n_m = NM;
    uint8_t* q_s = smem;
    uint8_t* t_s = q_s + 2 * n_m * kQBlk;
    WTail* tl = reinterpret_cast<WTail*>(t_s + 2 * n_m * kTBlk);

    const int tid = (int)threadIdx.x - 128, warp = ((int)threadIdx.x >> 5) - 4, lane = threadIdx.x & 31;
    const int groups = p.h > 32 ? 2 : 1;
    const uint32_t n_mma = 32u * (uint32_t)groups;
    volatile int* abort = &tl->abort;
    // this CTA's queries of every sequence, and its piece of the tiles
    const int split = (int)blockIdx.x % p.w_split;
    const int ta = (int)((long long)split * p.s / p.w_split), tb = (int)((long long)(split + 1) * p.s / p.w_split);

    if (warp == -4) {
        tmem_alloc(&tl->tmem_base, 256);
        tmem_relinquish();
    }
    if (tid == 0) {
        for (int m = 0; m < 4; ++m) {
            mbar_init(&tl->full[m], Deal<NM>::kWarps);
            mbar_init(&tl->freed[m], 1);
        }
        for (int k = 0; k < 2; ++k) {
            mbar_init(&tl->s_full[k], 1);
            mbar_init(&tl->s_free[k], 4 * groups);
        }
        mbar_init(&tl->q_full, 4 * groups);
        tl->abort = 0;
        fence_mbar_init();
    }
    for (int i = threadIdx.x; i < 2 * n_m * 64 * 8; i += kThreads)
        if (((i >> 3) & 63) >= p.h || (i >> 9) >= n_cb) reinterpret_cast<uint4*>(q_s)[i] = make_uint4(0, 0, 0, 0);
    if (n_cb & 1)
        for (int i = threadIdx.x; i < (int)kTBlk / 16; i += kThreads)
            reinterpret_cast<uint4*>(t_s + (size_t)n_cb * kTBlk)[i] = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
    plan_work(p.B, (int)blockIdx.x / p.w_split, (int)gridDim.x / p.w_split, tl->scratch, &tl->work,
              [&](int b) { return (visible_rows(p, b, p.s - 1) + kRows - 1) / kRows; });
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(kWarpFull, tl->tmem_base, 0);   // warp-uniform, as the compiler can see
    const Work wk = tl->work;
    griddep_wait();   // lse is complete from here on

    // a query's tiles within the chunk: those with a row it sees
    auto last_tile = [&](const Seg& sg, int t) {
        const int nt = (visible_rows(p, sg.b, t) + kRows - 1) / kRows;
        return nt < sg.t1 ? nt : sg.t1;
    };

    if (warp >= 8) {
        regs_down<kRegsDecode>();
        const int m = (warp - 8) / Deal<NM>::kWarps, lt = (warp - 8) % Deal<NM>::kWarps * 32 + lane;
        if (m < NM) {
            uint32_t n = 0;
            bool dead = false;
            WWalk walk(wk);
            Seg sg;
            while (!dead && walk.next(p, sg)) {
                for (int t = ta; t < tb && !dead; ++t) {
                    const int end = last_tile(sg, t);
                    for (int k = sg.t0; k < end && !dead; ++k, ++n) {
                        Codes<Deal<NM>::U> r;
                        load_units<NM>(p, sg.b, k * kRows, sg.vis, m, lt, n_cb, r);
                        if (n > 0) dead = !warp_wait(&tl->freed[m], (n - 1) & 1u, p.status, abort);
                        if (dead) break;
                        decode_units<NM>(t_s, k * kRows, sg.vis, m, lt, n_cb, r);
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&tl->full[m]);
                    }
                }
            }
        }
    } else if (warp < 0) {
        regs_down<kRegsMma>();
        const uint32_t idesc_qk = idesc_f16_f32(kRows, (int)n_mma, false, false);
        const uint64_t dk = sdesc(smem_u32(t_s), 16, 1024, kLayoutSW128), dq = sdesc(smem_u32(q_s), 16, 1024, kLayoutSW128);
        uint32_t n = 0, qn = 0;
        int have = -1;
        bool ok = warp == -4;
        auto wait = [&](uint64_t* bar, uint32_t parity) {
            ok = warp_wait(bar, parity, p.status, abort);
            tc_fence_after();
            return ok;
        };
        WWalk walk(wk);
        Seg sg;
        while (ok && walk.next(p, sg)) {
            for (int t = ta; t < tb && ok; ++t) {
                const int end = last_tile(sg, t);
                if (sg.t0 >= end) continue;
                if (have != sg.b * p.s + t) {   // another query: its Q
                    if (!wait(&tl->q_full, qn & 1u)) break;
                    ++qn;
                    have = sg.b * p.s + t;
                }
                for (int k = sg.t0; k < end && ok; ++k, ++n) {
                    const uint32_t st = n & 1u;
                    if (n >= 2 && !wait(&tl->s_free[st], ((n >> 1) - 1) & 1u)) break;
#pragma unroll
                    for (int m = 0; m < NM; ++m) {
                        if (!wait(&tl->full[m], n & 1u)) break;
                        if (elect_one()) {
                            qk_blocks(m == 0, tmem + 64u * st, lo32(dk) + (uint32_t)m * (2 * kTBlk / 16),
                                      lo32(dq) + (uint32_t)m * (2 * kQBlk / 16), hi32(dk), idesc_qk);
                            umma_commit(&tl->freed[m]);
                            if (m == NM - 1) umma_commit(&tl->s_full[st]);
                        }
                        __syncwarp();
                    }
                }
            }
        }
        __syncwarp();
    } else {
        regs_up<kRegsSoft>();
        if (warp < 4 * groups) {
        const int set = warp >> 2, qd = warp & 3;
        const int row = 32 * qd + lane;
        const uint32_t lane_base = (uint32_t)(32 * qd) << 16;
        const uint32_t n_soft = 128u * (uint32_t)groups;
        uint32_t n = 0;
        int have = -1, qbuf = 0;
        bool dead = false;
        WWalk walk(wk);
        Seg sg;
        while (walk.next(p, sg)) {
            for (int k = 0; k < sg.t1 - sg.t0; ++k) tl->acc[k][set][row] = 0.f;
            for (int t = ta; t < tb; ++t) {
                const int end = last_tile(sg, t);
                if (sg.t0 >= end) continue;
                const int q = sg.b * p.s + t;
                if (have != q) {   // this thread has seen the previous query's last S^T: the Q buffer is free
                    qbuf ^= 1;
                    load_q(p, q, tid, q_s, tl->qc);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane < 8) {   // the warp's own eight heads
                        const int hd = 8 * warp + lane;
                        tl->cl[qbuf][hd] =
                            make_float2(tl->qc[hd], hd < p.h ? -__ldcg(p.lse + (int64_t)q * p.h + hd) * kLog2e : 0.f);
                    }
                    if (lane == 0) mbar_arrive(&tl->q_full);
                    named_bar_sync(3, n_soft);
                    have = q;
                }
                const int vis = visible_rows(p, sg.b, t);
                for (int k = sg.t0; k < end; ++k, ++n) {
                    const uint32_t st = n & 1u;
                    if (!dead) dead = !warp_wait(&tl->s_full[st], (n >> 1) & 1u, p.status, abort);
                    tc_fence_after();
                    uint32_t r[32];
                    tmem_ld32(tmem + lane_base + 64u * st + 32u * (uint32_t)set, r);
                    tmem_ld_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&tl->s_free[st]);
                    if (k * kRows + row < vis && !dead) {
                        float sum = 0.f;
                        const int hn = p.h - 32 * set < 32 ? p.h - 32 * set : 32;
#pragma unroll
                        for (int c = 0; c < 16; ++c) {
                            const float4 v = *reinterpret_cast<const float4*>(&tl->cl[qbuf][32 * set + 2 * c]);
                            const float e0 = fast_exp2(fmaf(__uint_as_float(r[2 * c]), v.x, v.y));
                            const float e1 = fast_exp2(fmaf(__uint_as_float(r[2 * c + 1]), v.z, v.w));
                            if (2 * c < hn) sum += e0;
                            if (2 * c + 1 < hn) sum += e1;
                        }
                        tl->acc[k - sg.t0][set][row] += sum;
                    }
                }
            }
            named_bar_sync(3, n_soft);
            // the chunk's rows: thread = (row, every second tile) when there are two groups
            for (int k = sg.t0 + set; k < sg.t1; k += groups) {
                const int j = k * kRows + row;
                if (j < sg.vis) {
                    float v = tl->acc[k - sg.t0][0][row];
                    if (groups == 2) v += tl->acc[k - sg.t0][1][row];
                    if (p.w_split > 1) p.w_part[((int64_t)split * p.B + sg.b) * p.n_rows + j] = v;
                    else p.row_weight[(int64_t)sg.b * p.row_weight_bstride + j] += v;
                }
            }
            named_bar_sync(3, n_soft);
        }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (*abort) {
        const uint64_t t0 = global_timer_ns();
        while (global_timer_ns() - t0 < 50000ull) {
        }
    }
    if (warp == -4) {
        tc_fence_after();
        tmem_dealloc(tmem, 256);
    }
}

// The query splits' partial row weights, added in order.
__global__ void __launch_bounds__(256) row_weight_add_kernel(const AttnFp4Params p) {
    const int b = blockIdx.y;
    griddep_wait();
    for (int bb = b; bb < p.B; bb += gridDim.y) {
        const int vis = visible_rows(p, bb, p.s - 1);
        for (int j = blockIdx.x * 256 + threadIdx.x; j < vis; j += gridDim.x * 256) {
            float v = 0.f;
            for (int k = 0; k < p.w_split; ++k) v += __ldcg(p.w_part + ((int64_t)k * p.B + bb) * p.n_rows + j);
            p.row_weight[(int64_t)bb * p.row_weight_bstride + j] += v;
        }
    }
}

template <class K>
cudaError_t launch_after(K* kernel, dim3 grid, int threads, size_t smem, const AttnFp4Params& p, cudaStream_t stream) {
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
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace

void attn_fp4_plan(int B, int s, int n_rows, int num_sms, int* grid, int* w_grid, int* w_split) {
    const int64_t tiles = ((int64_t)n_rows + kRows - 1) / kRows;
    const int64_t all = tiles * B;                                   // row tiles at most
    const int64_t list = all * s > 0 ? all * s : 1;
    *grid = (int)(list < num_sms ? list : num_sms);
    int64_t split = all > 0 ? num_sms / all : 1;                     // CTAs per row tile
    split = split < 1 ? 1 : split > s ? s : split;
    *w_split = (int)split;
    const int64_t per = num_sms / split;
    *w_grid = (int)(split * (all < per ? (all > 0 ? all : 1) : per));
}

namespace {
template <int NM>
cudaError_t launch_nm(const AttnFp4Params& p, cudaStream_t stream) {
    const int nq = p.B * p.s;
    size_t smem = attn_smem(p.d);
    cudaError_t e = cudaFuncSetAttribute(attn_fp4_kernel<NM>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    attn_fp4_kernel<NM><<<p.grid, kThreads, smem, stream>>>(p);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    e = launch_after(merge_kernel, dim3((unsigned)(nq < p.grid ? nq : p.grid), (unsigned)p.h), 128, 0, p, stream);
    if (e != cudaSuccess || !p.row_weight || p.n_rows == 0) return e;
    smem = row_weight_smem(p.d);
    e = cudaFuncSetAttribute(row_weight_kernel<NM>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    e = launch_after(row_weight_kernel<NM>, dim3((unsigned)p.w_grid), kThreads, smem, p, stream);
    if (e != cudaSuccess || p.w_split == 1) return e;
    const int blocks = (p.n_rows + 255) / 256;
    return launch_after(row_weight_add_kernel,
                        dim3((unsigned)(blocks < 64 ? blocks : 64), (unsigned)(p.B < 65535 ? p.B : 65535)), 256, 0, p,
                        stream);
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
