// sti_attn_tiles.cuh -- what the kernels that attend over every row of a cache share: the work as one list of 64-row
// tiles cut between the CTAs, the MMAs of a tile (S^T = tile . Q^T, O^T += V^T . P^T), their bounded waits, and the
// kernel that joins the parts of a query split between CTAs.
#pragma once
#include <cuda_runtime.h>
#include <math.h>
#include <stddef.h>

#include "sti_attn_util.cuh"
#include "sti_ptx.cuh"

namespace sti {

constexpr int kThreads = 640;                  // 8 softmax warps, 8 warps that fill tiles, 4 others: two
                                               // issue MMAs, one prefetches
constexpr int kRows = 64;                      // rows per tile
constexpr uint32_t kQBlk = 64 * 128;           // a Q column block: 64 heads x 64 dims
constexpr uint32_t kTBlk = kRows * 128;        // a tile column block: 64 rows x 64 dims
constexpr uint32_t kPBuf = kRows * 128;        // a P^T buffer: 64 rows x 64 heads
constexpr uint32_t kTmO = 128;                 // TMEM: S^T of tile parity b at columns [64 b, 64 b + 64), O^T d-block
                                               // m at [128 + 64 m, 192 + 64 m)
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.69314718055994531f;

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

struct Work {           // this CTA's piece of the list
    long long lo, hi;   // tiles [lo, hi) of the list
    int q, off;         // the first one: tile `off` of query group q
    long long total;
    int ctas;           // CTAs that have tiles
};

struct Seg {            // a run of one group's tiles
    int q, b, vis, nt, t0, t1;
};

// Walk the piece: group by group, those without a visible row skipped.  P: a kernel's parameters, with
// group_rows(p, b, u), the rows that group u of sequence b goes over.
struct Walk {
    long long pos, hi;
    int q, off;
    __device__ __forceinline__ explicit Walk(const Work& w) : pos(w.lo), hi(w.hi), q(w.q), off(w.off) {}
    template <class P>
    __device__ __forceinline__ bool next(const P& p, Seg& s) {
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
    }
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

// ------------------------------------------------------------------ shared memory

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

// ------------------------------------------------------------------ joining split queries

// P: a kernel's parameters, with group_of(p, u) and head_seen(p, group, head, any), whether the head sees a row; any: a
// part's sum has no minus sign (a kernel may mark with -0 that a head saw none of a part's rows).
// Block (x, head, z): the x-th split query group (there are at most gridDim.x), dims 4 W z .. 4 W (z + 1) - 1; thread
// (g, i), g < G, dims 4 (W z + i) + {0..3} of every G-th part, four parts in flight; their sums join in shared memory
// in a fixed order.  G follows from the parts of a query when all are alike: a single long query (152 parts) needs many loads
// in flight (20 us with G = 8, W = 128), thousands of short ones (two parts each) would spend their time starting wide
// blocks.  A long query among short ones gets the short ones' G: one of 65536 rows x 512 among 59 of 300 takes 58 us for
// the call, alone 29.
template <int G, int W, class P>
__global__ void __launch_bounds__(G * W) merge_kernel(const P p) {
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
    const auto grp = group_of(p, rec.x);
    if (hh >= grp.heads) return;
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
    const float sk_in = p.sink ? __ldg(p.sink + hh % p.h) * kLog2e : -INFINITY;
    const float pl_in = p.prev_lse ? p.prev_lse[at] : -INFINITY, pl = pl_in * kLog2e;
    if (tid < 32) {
        float2 ml[5];   // parts <= 160
#pragma unroll
        for (int k = 0; k < 5; ++k)
            ml[k] = lane + 32 * k < parts ? __ldcg(p.part_ml + slot(lane + 32 * k) * 64 + hh) : make_float2(-INFINITY, 0.f);
        bool any = false;
#pragma unroll
        for (int k = 0; k < 5; ++k) any = any || (lane + 32 * k < parts && !signbit(ml[k].y));
        const bool seen = head_seen(p, grp, hh, __any_sync(kWarpFull, any));
        const float sk = seen ? sk_in : -INFINITY;
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

// ------------------------------------------------------------------ launch

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

}  // namespace sti
