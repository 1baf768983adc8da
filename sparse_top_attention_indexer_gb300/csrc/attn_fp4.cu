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
//   * warps 8..15 load the rows' codes into registers and decode them into the shared tile, one pair of
//     column blocks (128 dims) at a time, as the previous tile's PV releases them;
//   * warp 16 issues the MMAs:  S^T = tile . Q^T (M = 128 rows, N = heads), O^T += V^T . P^T (M = 128
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
// registers per thread after the roles' setmaxnreg: 256 x 128 + 256 x 80 + 128 x 48 = 59,392, within the
// 640 x 96 = 61,440 of the launch
constexpr int kRegsSoft = 128, kRegsDecode = 80, kRegsMma = 48;
constexpr int kRows = 128;                     // rows per tile
constexpr uint32_t kQBlk = 64 * 128;           // a Q column block: 64 heads x 64 dims
constexpr uint32_t kTBlk = kRows * 128;        // a tile column block: 128 rows x 64 dims
constexpr uint32_t kTmS0 = 0, kTmS1 = 64;      // TMEM columns of the two S^T partials
constexpr uint32_t kTmO = 128;                 // O^T d-block m at [128 + 64 m, 192 + 64 m)
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.69314718055994531f;
constexpr int kWTiles = 16;                    // row weights: tiles per chunk (accumulators in shared memory)

// instruction descriptor, kind::f16 with f16 A/B (format 0) and fp32 accumulator
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N, bool a_mn_major, bool b_mn_major) {
    return (1u << 4) | ((a_mn_major ? 1u : 0u) << 15) | ((b_mn_major ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) |
           ((uint32_t)(M >> 4) << 24);
}

template <int N>
__device__ __forceinline__ void regs_up() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_down() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
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

// The codes and scales of one row's column blocks fh, fh + 2, ... (row fr of a tile), as loaded.
struct RowCodes {
    uint4 c[4][2];
    uint32_t s[4];
};

__device__ __forceinline__ void load_row(const AttnFp4Params& p, int b, int row, int fh, int n_cb, RowCodes& r) {
    const uint8_t* cr = p.codes + (int64_t)b * p.codes_bstride + (int64_t)row * (p.d / 2);
    const uint8_t* sr = p.scales + (int64_t)b * p.scales_bstride + (int64_t)row * (p.d / 16);
#pragma unroll
    for (int m = 0; m < 4; ++m) {
        const int j = 2 * m + fh;
        if (j >= n_cb) break;
        r.c[m][0] = __ldg(reinterpret_cast<const uint4*>(cr + j * 32));
        r.c[m][1] = __ldg(reinterpret_cast<const uint4*>(cr + j * 32 + 16));
        r.s[m] = __ldg(reinterpret_cast<const uint32_t*>(sr + j * 4));
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
    float mcp[2][4][32];      // each warp's copy of its head group's running maxima
    float qc[2][64];          // [segment parity] per head: softmax scale (log2) over its f16 scaling
    float red[2][2][4][32];   // [tile parity][group][warp]: per-warp maxima
    float lsum[2][4][32];
    Work work;
    long long scratch[kThreads / 32];
    uint64_t full[8];         // column block j of the tile decoded: one arrival per decoding warp of its parity
    uint64_t pv[4];           // the tile's PV of d-block m done
    uint64_t s_full, p_full, q_full;
    uint32_t tmem_base;
    int abort;
};

size_t attn_smem(int d) {
    const int n_cb = (d + 127) / 128 * 2;
    return 1024 + (size_t)n_cb * (kQBlk + kTBlk) + kRows * 128 + sizeof(Tail);
}

__global__ void __launch_bounds__(kThreads, 1) attn_fp4_kernel(const AttnFp4Params p) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const int n_cb = p.d / 64;                 // column blocks of 64 dims
    const int n_m = (n_cb + 1) / 2;            // d-blocks of 128
    uint8_t* q_s = smem;                       // [2 n_m][64 heads][128 B]
    uint8_t* t_s = q_s + 2 * n_m * kQBlk;      // [2 n_m][128 rows][128 B]
    uint8_t* p_s = t_s + 2 * n_m * kTBlk;      // P^T [128 rows][64 heads] f16
    Tail* tl = reinterpret_cast<Tail*>(p_s + kRows * 128);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int nq = p.B * p.s;
    const int groups = p.h > 32 ? 2 : 1;       // groups of 32 heads
    const uint32_t n_mma = 32u * (uint32_t)groups;
    volatile int* abort = &tl->abort;

    if (warp == 16) {
        tmem_alloc(&tl->tmem_base, n_m <= 2 ? 256 : 512);
        tmem_relinquish();
    }
    if (tid == 0) {
        for (int j = 0; j < 8; ++j) mbar_init(&tl->full[j], 4);
        for (int m = 0; m < 4; ++m) mbar_init(&tl->pv[m], 1);
        mbar_init(&tl->s_full, 1);
        mbar_init(&tl->p_full, 4 * groups);
        mbar_init(&tl->q_full, 4 * groups);
        tl->abort = 0;
        fence_mbar_init();
    }
    // what no thread writes later: Q rows of heads >= h, the dims past d of the last d-block
    for (int i = tid; i < 2 * n_m * 64 * 8; i += kThreads)
        if (((i >> 3) & 63) >= p.h) reinterpret_cast<uint4*>(q_s)[i] = make_uint4(0, 0, 0, 0);
    if (n_cb & 1)
        for (int i = tid; i < (int)kTBlk / 16; i += kThreads)
            reinterpret_cast<uint4*>(t_s + (size_t)n_cb * kTBlk)[i] = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
    plan_work(nq, blockIdx.x, gridDim.x, tl->scratch, &tl->work,
              [&](int q) { return (visible_rows(p, q / p.s, q % p.s) + kRows - 1) / kRows; });
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tl->tmem_base;
    const Work wk = tl->work;
    griddep_launch_dependents();

    if (warp >= 8 && warp < 16) {
        regs_down<kRegsDecode>();
        // -------------------------------------------------------------- decode: thread = (row, column block parity)
        const int fr = tid & 127, fh = (tid >> 7) & 1;
        uint32_t n = 0;
        bool dead = false;
        Walk walk(wk);
        Seg sg;
        while (!dead && walk.next(p, sg)) {
            for (int t = sg.t0; t < sg.t1 && !dead; ++t, ++n) {
                const int row = t * kRows + fr;
                const bool valid = row < sg.vis;
                RowCodes r;
                if (valid) load_row(p, sg.b, row, fh, n_cb, r);
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    const int j = 2 * m + fh;
                    if (2 * m >= n_cb) break;
                    if (n > 0) {
                        if (!dead) dead = !attn_wait(&tl->pv[m], (n - 1) & 1u, p.status, abort);
                        dead = __any_sync(kWarpFull, dead);
                    }
                    if (dead || j >= n_cb) continue;
                    decode_block(t_s + (size_t)j * kTBlk + fr * 128, fr, valid, r.c[m][0], r.c[m][1], r.s[m]);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&tl->full[j]);
                }
            }
        }
    } else if (warp >= 16) {
        regs_down<kRegsMma>();
        // -------------------------------------------------------------- MMA issue
        const uint32_t idesc_qk = idesc_f16_f32(kRows, (int)n_mma, false, false);
        const uint32_t idesc_pv = idesc_f16_f32(kRows, (int)n_mma, true, true);
        const uint32_t q0 = smem_u32(q_s), t0 = smem_u32(t_s), p0 = smem_u32(p_s);
        uint32_t n = 0, qn = 0;
        Walk walk(wk);
        Seg sg;
        bool ok = warp == 16 && lane == 0;
        while (ok && walk.next(p, sg)) {
            ok = attn_wait(&tl->q_full, qn & 1u, p.status, abort);
            ++qn;
            for (int t = sg.t0; t < sg.t1 && ok; ++t, ++n) {
                for (int j = 0; j < n_cb && ok; ++j) {
                    ok = attn_wait(&tl->full[j], n & 1u, p.status, abort);
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll
                    for (int kq = 0; kq < 4; ++kq) {
                        const int kk = 4 * j + kq;
                        umma_bf16(tmem + ((kk & 1) ? kTmS1 : kTmS0),
                                  sdesc(t0 + (uint32_t)j * kTBlk + (uint32_t)kq * 32u, 16, 1024, kLayoutSW128),
                                  sdesc(q0 + (uint32_t)j * kQBlk + (uint32_t)kq * 32u, 16, 1024, kLayoutSW128),
                                  idesc_qk, kk >= 2 ? 1u : 0u);
                    }
                }
                if (!ok) break;
                umma_commit(&tl->s_full);
                ok = attn_wait(&tl->p_full, n & 1u, p.status, abort);
                if (!ok) break;
                tc_fence_after();
                for (int m = 0; m < n_m; ++m) {
#pragma unroll
                    for (int kk = 0; kk < kRows / 16; ++kk)
                        umma_bf16(tmem + kTmO + 64u * (uint32_t)m,
                                  sdesc(t0 + (uint32_t)(2 * m) * kTBlk + (uint32_t)kk * 2048u, kTBlk, 1024,
                                        kLayoutSW128),
                                  sdesc(p0 + (uint32_t)kk * 2048u, kRows * 128u, 1024, kLayoutSW128), idesc_pv,
                                  (t > sg.t0 || kk > 0) ? 1u : 0u);
                    umma_commit(&tl->pv[m]);
                }
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
            if (!dead) dead = !attn_wait(bar, parity, p.status, abort);
            dead = __any_sync(kWarpFull, dead);
        };

        auto softmax = [&](bool valid, bool first) {
            mwait(&tl->s_full, n & 1u);
            tc_fence_after();
            valid = valid && !dead;
            float x[32];
            {
                uint32_t r0[32], r1[32];
                tmem_ld32(tmem + lane_base + kTmS0 + 32u * (uint32_t)set, r0);
                tmem_ld32(tmem + lane_base + kTmS1 + 32u * (uint32_t)set, r1);
                tmem_ld_wait();
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    const float4 q4 = *reinterpret_cast<const float4*>(&tl->qc[qbuf][32 * set + 4 * c]);
                    const float qv[4] = {q4.x, q4.y, q4.z, q4.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        x[4 * c + e] = valid ? (__uint_as_float(r0[4 * c + e]) + __uint_as_float(r1[4 * c + e])) * qv[e]
                                             : -INFINITY;
                }
            }
            const float* mc = &tl->mcp[set][qd][0];
            bool need = first;
            if (!first) {
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    const float4 m4 = *reinterpret_cast<const float4*>(mc + 4 * c);
                    need = need || x[4 * c] > m4.x + 8.f || x[4 * c + 1] > m4.y + 8.f || x[4 * c + 2] > m4.z + 8.f ||
                           x[4 * c + 3] > m4.w + 8.f;
                }
            }
            need = !named_bar_and(bar_set, 128, !need);
            if (need) {
                {
                    float v2[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i) v2[i] = x[i];
                    warp_reduce_scatter_n<32, true>(v2);
                    tl->red[n & 1u][set][qd][lane] = v2[0];
                }
                named_bar_sync(bar_set, 128);
                const float* rr = &tl->red[n & 1u][set][0][0];
                const float mt = fmaxf(fmaxf(rr[lane], rr[32 + lane]), fmaxf(rr[64 + lane], rr[96 + lane]));
                const float m_new = (m_run == -INFINITY || mt > m_run + 8.f) ? fmaxf(m_run, mt) : m_run;
                const float alpha = (m_new == m_run) ? 1.f : exp2f(m_run - m_new);
                m_run = m_new;
                // a head without any finite score keeps -inf; its exponents are taken from 0, so that NaN
                // scores show in its output
                tl->mcp[set][qd][lane] = m_new == -INFINITY ? 0.f : m_new;
                __syncwarp();
                if (!first && !dead && __any_sync(kWarpFull, alpha != 1.f)) {
#pragma unroll 1
                    for (int m = 0; m < n_m; ++m) {
                        const uint32_t ta = tmem + lane_base + kTmO + 64u * (uint32_t)m + 32u * (uint32_t)set;
                        uint32_t r[32];
                        tmem_ld32(ta, r);
                        tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            r[i] = __float_as_uint(__uint_as_float(r[i]) * __shfl_sync(kWarpFull, alpha, i));
                        tmem_st32(ta, r);
                    }
                    tmem_st_wait();
#pragma unroll
                    for (int i = 0; i < 32; ++i) l_thr[i] *= __shfl_sync(kWarpFull, alpha, i);
                }
            }
            uint8_t* prow = p_s + row * 128;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const float4 ma = *reinterpret_cast<const float4*>(mc + 8 * c);
                const float4 mb = *reinterpret_cast<const float4*>(mc + 8 * c + 4);
                const float mm[8] = {ma.x, ma.y, ma.z, ma.w, mb.x, mb.y, mb.z, mb.w};
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float e = fast_exp2(x[8 * c + j] - mm[j]);   // 0 for rows that are not visible
                    x[8 * c + j] = e;
                    l_thr[8 * c + j] += e;
                }
                uint4 pk;
                pk.x = pack_f16x2(x[8 * c + 0], x[8 * c + 1]);
                pk.y = pack_f16x2(x[8 * c + 2], x[8 * c + 3]);
                pk.z = pack_f16x2(x[8 * c + 4], x[8 * c + 5]);
                pk.w = pack_f16x2(x[8 * c + 6], x[8 * c + 7]);
                *reinterpret_cast<uint4*>(prow + (((4 * set + c) ^ (row & 7)) << 4)) = pk;
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
    if (warp == 16) {
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
    float qc[2][64];
    float ls[2][64];                 // [query parity] the heads' lse in log2
    float acc[kWTiles][2][kRows];    // [tile of the chunk][head group][row]
    Work work;
    long long scratch[kThreads / 32];
    uint64_t full[8];
    uint64_t freed[4];               // the tile's QK has read column blocks 2m, 2m + 1
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

__global__ void __launch_bounds__(kThreads, 1) row_weight_kernel(const AttnFp4Params p) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const int n_cb = p.d / 64;
    const int n_m = (n_cb + 1) / 2;
    uint8_t* q_s = smem;
    uint8_t* t_s = q_s + 2 * n_m * kQBlk;
    WTail* tl = reinterpret_cast<WTail*>(t_s + 2 * n_m * kTBlk);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int groups = p.h > 32 ? 2 : 1;
    const uint32_t n_mma = 32u * (uint32_t)groups;
    volatile int* abort = &tl->abort;
    // this CTA's queries of every sequence, and its piece of the tiles
    const int split = (int)blockIdx.x % p.w_split;
    const int ta = (int)((long long)split * p.s / p.w_split), tb = (int)((long long)(split + 1) * p.s / p.w_split);

    if (warp == 16) {
        tmem_alloc(&tl->tmem_base, 256);
        tmem_relinquish();
    }
    if (tid == 0) {
        for (int j = 0; j < 8; ++j) mbar_init(&tl->full[j], 4);
        for (int m = 0; m < 4; ++m) mbar_init(&tl->freed[m], 1);
        for (int k = 0; k < 2; ++k) {
            mbar_init(&tl->s_full[k], 1);
            mbar_init(&tl->s_free[k], 4 * groups);
        }
        mbar_init(&tl->q_full, 4 * groups);
        tl->abort = 0;
        fence_mbar_init();
    }
    for (int i = tid; i < 2 * n_m * 64 * 8; i += kThreads)
        if (((i >> 3) & 63) >= p.h) reinterpret_cast<uint4*>(q_s)[i] = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
    plan_work(p.B, (int)blockIdx.x / p.w_split, (int)gridDim.x / p.w_split, tl->scratch, &tl->work,
              [&](int b) { return (visible_rows(p, b, p.s - 1) + kRows - 1) / kRows; });
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tl->tmem_base;
    const Work wk = tl->work;
    griddep_wait();   // lse is complete from here on

    // a query's tiles within the chunk: those with a row it sees
    auto last_tile = [&](const Seg& sg, int t) {
        const int nt = (visible_rows(p, sg.b, t) + kRows - 1) / kRows;
        return nt < sg.t1 ? nt : sg.t1;
    };

    if (warp >= 8 && warp < 16) {
        regs_down<kRegsDecode>();
        const int fr = tid & 127, fh = (tid >> 7) & 1;
        uint32_t n = 0;
        bool dead = false;
        WWalk walk(wk);
        Seg sg;
        while (!dead && walk.next(p, sg)) {
            for (int t = ta; t < tb && !dead; ++t) {
                const int end = last_tile(sg, t);
                for (int k = sg.t0; k < end && !dead; ++k, ++n) {
                    const int row = k * kRows + fr;
                    const bool valid = row < sg.vis;
                    RowCodes r;
                    if (valid) load_row(p, sg.b, row, fh, n_cb, r);
#pragma unroll
                    for (int m = 0; m < 4; ++m) {
                        const int j = 2 * m + fh;
                        if (2 * m >= n_cb) break;
                        if (n > 0) {
                            if (!dead) dead = !attn_wait(&tl->freed[m], (n - 1) & 1u, p.status, abort);
                            dead = __any_sync(kWarpFull, dead);
                        }
                        if (dead || j >= n_cb) continue;
                        decode_block(t_s + (size_t)j * kTBlk + fr * 128, fr, valid, r.c[m][0], r.c[m][1], r.s[m]);
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&tl->full[j]);
                    }
                }
            }
        }
    } else if (warp >= 16) {
        regs_down<kRegsMma>();
        const uint32_t idesc_qk = idesc_f16_f32(kRows, (int)n_mma, false, false);
        const uint32_t q0 = smem_u32(q_s), t0 = smem_u32(t_s);
        uint32_t n = 0, qn = 0;
        int have = -1;
        bool ok = warp == 16 && lane == 0;
        WWalk walk(wk);
        Seg sg;
        while (ok && walk.next(p, sg)) {
            for (int t = ta; t < tb && ok; ++t) {
                const int end = last_tile(sg, t);
                if (sg.t0 >= end) continue;
                if (have != sg.b * p.s + t) {   // another query: its Q
                    ok = attn_wait(&tl->q_full, qn & 1u, p.status, abort);
                    ++qn;
                    have = sg.b * p.s + t;
                }
                for (int k = sg.t0; k < end && ok; ++k, ++n) {
                    const uint32_t st = n & 1u;
                    if (n >= 2) ok = attn_wait(&tl->s_free[st], ((n >> 1) - 1) & 1u, p.status, abort);
                    for (int j = 0; j < n_cb && ok; ++j) {
                        ok = attn_wait(&tl->full[j], n & 1u, p.status, abort);
                        if (!ok) break;
                        tc_fence_after();
#pragma unroll
                        for (int kq = 0; kq < 4; ++kq) {
                            const int kk = 4 * j + kq;
                            umma_bf16(tmem + 128u * st + ((kk & 1) ? kTmS1 : kTmS0),
                                      sdesc(t0 + (uint32_t)j * kTBlk + (uint32_t)kq * 32u, 16, 1024, kLayoutSW128),
                                      sdesc(q0 + (uint32_t)j * kQBlk + (uint32_t)kq * 32u, 16, 1024, kLayoutSW128),
                                      idesc_qk, kk >= 2 ? 1u : 0u);
                        }
                        if ((j & 1) || j == n_cb - 1) umma_commit(&tl->freed[j >> 1]);
                    }
                    if (ok) umma_commit(&tl->s_full[st]);
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
                    load_q(p, q, tid, q_s, tl->qc[qbuf]);
                    if (tid < 64) tl->ls[qbuf][tid] = tid < p.h ? __ldcg(p.lse + (int64_t)q * p.h + tid) * kLog2e : 0.f;
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&tl->q_full);
                    named_bar_sync(3, n_soft);
                    have = q;
                }
                const int vis = visible_rows(p, sg.b, t);
                for (int k = sg.t0; k < end; ++k, ++n) {
                    const uint32_t st = n & 1u;
                    if (!dead) dead = !attn_wait(&tl->s_full[st], (n >> 1) & 1u, p.status, abort);
                    dead = __any_sync(kWarpFull, dead);
                    tc_fence_after();
                    uint32_t r0[32], r1[32];
                    tmem_ld32(tmem + lane_base + 128u * st + kTmS0 + 32u * (uint32_t)set, r0);
                    tmem_ld32(tmem + lane_base + 128u * st + kTmS1 + 32u * (uint32_t)set, r1);
                    tmem_ld_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&tl->s_free[st]);
                    if (k * kRows + row < vis && !dead) {
                        float sum = 0.f;
                        const int hn = p.h - 32 * set < 32 ? p.h - 32 * set : 32;
#pragma unroll
                        for (int c = 0; c < 8; ++c) {
                            const float4 q4 = *reinterpret_cast<const float4*>(&tl->qc[qbuf][32 * set + 4 * c]);
                            const float4 l4 = *reinterpret_cast<const float4*>(&tl->ls[qbuf][32 * set + 4 * c]);
                            const float qv[4] = {q4.x, q4.y, q4.z, q4.w}, lv[4] = {l4.x, l4.y, l4.z, l4.w};
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const int i = 4 * c + e;
                                const float x = (__uint_as_float(r0[i]) + __uint_as_float(r1[i])) * qv[e];
                                if (i < hn) sum += fast_exp2(x - lv[e]);
                            }
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
    if (warp == 16) {
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

cudaError_t launch_attn_fp4(const AttnFp4Params& p, cudaStream_t stream) {
    const int nq = p.B * p.s;
    if (nq == 0) return cudaSuccess;
    size_t smem = attn_smem(p.d);
    cudaError_t e = cudaFuncSetAttribute(attn_fp4_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    attn_fp4_kernel<<<p.grid, kThreads, smem, stream>>>(p);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    e = launch_after(merge_kernel, dim3((unsigned)(nq < p.grid ? nq : p.grid), (unsigned)p.h), 128, 0, p, stream);
    if (e != cudaSuccess || !p.row_weight || p.n_rows == 0) return e;
    smem = row_weight_smem(p.d);
    e = cudaFuncSetAttribute(row_weight_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    e = launch_after(row_weight_kernel, dim3((unsigned)p.w_grid), kThreads, smem, p, stream);
    if (e != cudaSuccess || p.w_split == 1) return e;
    return launch_after(row_weight_add_kernel,
                        dim3((unsigned)((p.n_rows + 255) / 256 < 64 ? (p.n_rows + 255) / 256 : 64),
                             (unsigned)(p.B < 65535 ? p.B : 65535)),
                        256, 0, p, stream);
}

}  // namespace sti
