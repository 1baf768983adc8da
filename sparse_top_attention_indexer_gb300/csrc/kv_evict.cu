// kv_evict.cu -- evict the rows of a cache that have received the least attention.
//
// Per sequence with `held` rows above `budget`: the rows are ordered by (protected first, then weight
// descending, then row ascending) and the first `budget` of them stay.  Protected are the first positions
// and the most recent ones (by row_pos).  Freed rows below `budget` (holes) are refilled, in ascending
// order, by the kept rows at or above `budget` (movers), so only as many rows move as were evicted below
// the budget, and no row is both read and written: everything that belongs to a row (weight, position,
// any list of row arrays) moves in one pass without a temporary copy.
//
// One cluster of C CTAs per sequence, each CTA a contiguous piece of the rows, each warp a contiguous
// piece of its CTA's:
//   1. order-preserving 32-bit keys of the rows into shared memory;
//   2. radix select of the budget-th largest key in three passes (11 + 11 + 10 bits): shared-memory
//      histograms per CTA, each CTA sums its slice of the bins over the cluster, every CTA finds the bin;
//   3. rows equal to that key stay in row order until the budget is full: ranks by ballots within warps
//      and prefix sums over warps and CTAs (no atomics whose order could show);
//   4. holes and movers get their ranks the same way and go to two lists in the workspace;
//   5. the cluster copies mover i to hole i, in pieces of up to 16 bytes, over all arrays at once.
// Bound by latency: the chain of barriers (two per pass and four after over the cluster, with C = 8), not by the 8 bytes
// per row it reads: 32 sequences of 2049 rows losing one each 10 us, 8 of 8704 rows losing 512 18 us, one of 52,003
// rows losing 2002 23 us; the same with all weights equal, where every atomic of a pass meets in one bin.  Adding
// equal bins within a warp before the histogram costs more (12, 19, 28 us) than the collisions of its atomics.
// C = 1, 2, 4 or 8 by the rows and the number of sequences (cluster_size).
#include <math.h>

#include "sti_internal.h"
#include "sti_ptx.cuh"

namespace sti {
namespace {

constexpr int kEvThreads = 1024;
constexpr int kEvWarps = kEvThreads / 32;
constexpr int kBins = 2048;
constexpr int kKeyCache = 40960;   // keys a CTA holds in shared memory; rows past it are re-read
constexpr uint32_t kFull = 0xFFFFFFFFu;

struct EvTail {
    uint32_t hist[2][kBins];    // [pass parity]
    uint32_t sum[kBins];        // this CTA's slice of the cluster-wide bins
    uint32_t slice_total;
    uint32_t warp_cnt[2][kEvWarps];
    uint32_t cta_cnt[2][2];     // [call of rank_base]
    uint32_t scratch[kEvWarps];
    uint32_t found[2];          // bin, rows above it
};

template <int C>
__device__ __forceinline__ void ev_sync() {
    __syncwarp();
    if constexpr (C > 1) cluster_sync();
    else __syncthreads();
}
template <int C>
__device__ __forceinline__ uint32_t peer_u32(const uint32_t* local, int rank) {
    if constexpr (C > 1) return ld_dsmem_u32(dsmem_addr(local, (uint32_t)rank));
    else return *local;
}

// Exclusive prefix of v over the block (v of thread 0 first); *total gets the block's sum.
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t* scratch, uint32_t* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t u = __shfl_up_sync(kFull, inc, o);
        if (lane >= o) inc += u;
    }
    __syncthreads();
    if (lane == 31) scratch[warp] = inc;
    __syncthreads();
    uint32_t w = scratch[lane];   // kEvWarps == 32
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t u = __shfl_up_sync(kFull, w, o);
        if (lane >= o) w += u;
    }
    *total = __shfl_sync(kFull, w, 31);
    const uint32_t before = __shfl_sync(kFull, w, (warp + 31) & 31);
    return (warp ? before : 0u) + inc - v;
}

// Counts of two kinds of rows per warp -> the counts in all earlier warps of the cluster.  The two calls have counts of
// their own: nobody waits until they are read.
template <int C, int kCall>
__device__ __forceinline__ void rank_base(EvTail* tl, int rank, uint32_t c0, uint32_t c1, uint32_t& b0, uint32_t& b1) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (lane == 0) {
        tl->warp_cnt[0][warp] = c0;
        tl->warp_cnt[1][warp] = c1;
    }
    __syncthreads();
    uint32_t w0 = tl->warp_cnt[0][lane], w1 = tl->warp_cnt[1][lane];
    const uint32_t t0 = __reduce_add_sync(kFull, w0), t1 = __reduce_add_sync(kFull, w1);
    if (lane >= warp) w0 = w1 = 0u;
    b0 = __reduce_add_sync(kFull, w0);
    b1 = __reduce_add_sync(kFull, w1);
    if (C > 1) {
        if (threadIdx.x == 0) {
            tl->cta_cnt[kCall][0] = t0;
            tl->cta_cnt[kCall][1] = t1;
        }
        ev_sync<C>();
        // one remote read per CTA and warp, all at once
        const bool before = lane < rank;
        b0 += __reduce_add_sync(kFull, before ? peer_u32<C>(&tl->cta_cnt[kCall][0], lane) : 0u);
        b1 += __reduce_add_sync(kFull, before ? peer_u32<C>(&tl->cta_cnt[kCall][1], lane) : 0u);
    } else {
        __syncthreads();
    }
}

__device__ __forceinline__ uint32_t low_bits(int n) { return n >= 32 ? kFull : n <= 0 ? 0u : (1u << n) - 1u; }

template <int BYTES>
struct Piece;
template <> struct Piece<16> { typedef uint4 T; };
template <> struct Piece<8> { typedef uint2 T; };
template <> struct Piece<4> { typedef uint32_t T; };
template <> struct Piece<2> { typedef uint16_t T; };
template <> struct Piece<1> { typedef uint8_t T; };

template <int BYTES>
__device__ __forceinline__ void copy_piece(uint8_t* base, int64_t row_bytes, int64_t to, int64_t of, uint32_t at) {
    typedef typename Piece<BYTES>::T T;
    *reinterpret_cast<T*>(base + to * row_bytes + (int64_t)at * BYTES) =
        *reinterpret_cast<const T*>(base + of * row_bytes + (int64_t)at * BYTES);
}

template <int C>
__global__ void __launch_bounds__(kEvThreads) kv_evict_kernel(const KvEvictParams p) {
    extern __shared__ __align__(16) uint8_t ev_smem[];
    EvTail* tl = reinterpret_cast<EvTail*>(ev_smem);
    uint32_t* keys = reinterpret_cast<uint32_t*>(tl + 1);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = C > 1 ? (int)(blockIdx.x % C) : 0;
    const int b = (int)(blockIdx.x / C);
    const int64_t groups = ((int64_t)__ldg(p.start_pos + b) + p.s) / p.ratio;
    const int gone = p.dropped[b];
    int64_t h64 = groups - gone;
    h64 = h64 < 0 ? 0 : h64 > p.n_rows ? p.n_rows : h64;
    const int held = (int)h64, budget = p.budget;
    if (held <= budget) return;   // the whole cluster

    const float* weight = p.row_weight + (int64_t)b * p.row_weight_bstride;
    const int32_t* pos = p.row_pos + (int64_t)b * p.row_pos_bstride;
    const int64_t recent = groups - p.n_recent;
    // rows of this CTA and of this warp (whole 32-row steps, so that ballots are in row order)
    const int per_warp = (held + 32 * kEvWarps * C - 1) / (32 * kEvWarps * C) * 32;
    const int cta0 = min(held, rank * per_warp * kEvWarps);
    const int w0 = min(held, cta0 + warp * per_warp), w1 = min(held, w0 + per_warp);

    auto key_of = [&](int q, float w) -> uint32_t {
        if (q < p.n_first || q >= recent) return 0xFFFFFFFFu;
        w += 0.f;                          // -0 counts as 0
        if (w != w) return 0xFFFFFFFEu;    // NaN: above every number
        return float_key(w);
    };
    auto make_key = [&](int j) -> uint32_t { return key_of(pos[j], weight[j]); };
    auto key = [&](int j) -> uint32_t { return j - cta0 < kKeyCache ? keys[j - cta0] : make_key(j); };

    for (int i = tid; i < 2 * kBins; i += kEvThreads) tl->hist[0][i] = 0u;
    const int w_cached = min(w1, cta0 + kKeyCache);
    for (int j0 = w0 + lane; j0 < w_cached; j0 += 8 * 32) {   // eight rows' loads in flight
        int q[8];
        float w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int j = min(j0 + 32 * i, w_cached - 1);
            q[i] = pos[j];
            w[i] = weight[j];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (j0 + 32 * i < w_cached) keys[j0 + 32 * i - cta0] = key_of(q[i], w[i]);
    }
    __syncthreads();

    // the budget-th largest key
    uint32_t prefix = 0u, want = (uint32_t)budget;   // want: rows still to take among those matching prefix
    if (budget > 0) {
#pragma unroll 1
        for (int pass = 0; pass < 3; ++pass) {
            const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
            const int bins = pass == 2 ? 1024 : 2048;
            const uint32_t above = pass == 0 ? 0u : 0xFFFFFFFFu << (pass == 1 ? 21 : 10);   // bits already fixed
            uint32_t* hist = tl->hist[pass & 1];
            for (int j = w0 + lane; j < w1; j += 32) {
                const uint32_t k = key(j);
                if ((k & above) == prefix) atomicAdd(&hist[(k >> shift) & (uint32_t)(bins - 1)], 1u);
            }
            ev_sync<C>();   // also: every CTA has read the sums of the pass before
            // this CTA's slice of the bins, summed over the cluster; totals per slice
            const int per = bins / C;
            for (int i = tid; i < per; i += kEvThreads) {
                uint32_t v = 0u;
#pragma unroll
                for (int c = 0; c < C; ++c) v += peer_u32<C>(&hist[rank * per + i], c);
                tl->sum[i] = v;
            }
            if (C > 1) {
                __syncthreads();
                uint32_t t = 0u;
                for (int i = tid; i < per; i += kEvThreads) t += tl->sum[i];
                uint32_t tot;
                block_scan(t, tl->scratch, &tot);
                if (tid == 0) tl->slice_total = tot;
            }
            ev_sync<C>();   // also: every CTA has read this pass's histograms
            // from the top: the slice, then the bin, in which the want-th row lies
            int slice = C - 1;
            if (C > 1) {
                const uint32_t mine = lane < C ? peer_u32<C>(&tl->slice_total, lane) : 0u;
                for (; slice > 0; --slice) {
                    const uint32_t t = __shfl_sync(kFull, mine, slice);
                    if (t >= want) break;
                    want -= t;
                }
            }
            // bins of the slice from the top, two per thread (per <= 2048)
            uint32_t v[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int i = 2 * tid + e;
                v[e] = i < per ? peer_u32<C>(&tl->sum[per - 1 - i], slice) : 0u;
            }
            uint32_t tot;
            const uint32_t before = block_scan(v[0] + v[1], tl->scratch, &tot);
            if (before < want && before + v[0] + v[1] >= want) {
                const int e = before + v[0] >= want ? 0 : 1;
                tl->found[0] = (uint32_t)(slice * per + per - 1 - (2 * tid + e));
                tl->found[1] = before + (e ? v[0] : 0u);
            }
            for (int i = tid; i < kBins; i += kEvThreads) hist[i] = 0u;   // for the pass after the next
            __syncthreads();
            prefix |= tl->found[0] << shift;
            want -= tl->found[1];
            __syncthreads();
        }
    }
    // budget == 0: nothing stays (no key is above 0xFFFFFFFF, and none of the equal ones is wanted)
    const uint32_t T = budget > 0 ? prefix : 0xFFFFFFFFu;
    if (budget == 0) want = 0u;

    // rows equal to T: the first `want` in row order stay
    uint32_t eq_base, unused;
    {
        uint32_t c = 0u;
        for (int j = w0 + lane; j < w1; j += 32) c += key(j) == T ? 1u : 0u;
        rank_base<C, 0>(tl, rank, __reduce_add_sync(kFull, c), 0u, eq_base, unused);
    }
    auto for_rows = [&](auto&& f) {
        uint32_t eq = eq_base;
        for (int j0 = w0; j0 < w1; j0 += 32) {
            const int j = j0 + lane;
            const uint32_t k = j < w1 ? key(j) : 0u;
            const bool is_eq = j < w1 && k == T;
            const uint32_t m = __ballot_sync(kFull, is_eq);
            const bool kept = j < w1 && (k > T || (is_eq && eq + __popc(m & ((1u << lane) - 1u)) < want));
            eq += __popc(m);
            // bits of the step's rows that exist, and of those below the budget
            const uint32_t stay = __ballot_sync(kFull, kept), real = low_bits(w1 - j0), below = low_bits(budget - j0);
            f(j, real & ~stay & below, stay & ~below);
        }
    };
    uint32_t n_hole = 0u, n_move = 0u, hole_base, move_base;
    for_rows([&](int, uint32_t holes, uint32_t movers) {
        n_hole += __popc(holes);
        n_move += __popc(movers);
    });
    rank_base<C, 1>(tl, rank, n_hole, n_move, hole_base, move_base);
    int32_t* to = p.lists + (int64_t)b * 2 * p.most;
    int32_t* of = to + p.most;
    for_rows([&](int j, uint32_t holes, uint32_t movers) {
        const uint32_t lt = (1u << lane) - 1u;
        if ((holes >> lane) & 1u) to[hole_base + __popc(holes & lt)] = j;
        if ((movers >> lane) & 1u) of[move_base + __popc(movers & lt)] = j;
        hole_base += __popc(holes);
        move_base += __popc(movers);
    });
    // the cluster's last warp ends at the number of moves
    if (tid == kEvThreads - 1) tl->cta_cnt[0][0] = move_base;
    ev_sync<C>();   // lists complete, every row's weight and position read
    const uint32_t n = peer_u32<C>(&tl->cta_cnt[0][0], C - 1);

    // move: pieces of every array, one flat index over (array, move, piece)
    int a = 0;
    int64_t a0 = 0;                                   // first index of array a
    int64_t an = (int64_t)n * p.arr[0].pieces;
    for (int64_t idx = rank * kEvThreads + tid;; idx += C * kEvThreads) {
        while (idx >= a0 + an) {
            a0 += an;
            if (++a >= p.n_arr) break;
            an = (int64_t)n * p.arr[a].pieces;
        }
        if (a >= p.n_arr) break;
        const uint32_t off = (uint32_t)(idx - a0), i = off / (uint32_t)p.arr[a].pieces;
        const uint32_t at = off - i * (uint32_t)p.arr[a].pieces;
        uint8_t* base = static_cast<uint8_t*>(p.arr[a].base) + (int64_t)b * p.arr[a].bstride;
        const int64_t rb = p.arr[a].row_bytes;
        const int t = to[i], o = of[i];
        switch (p.arr[a].piece_bytes) {
            case 16: copy_piece<16>(base, rb, t, o, at); break;
            case 8: copy_piece<8>(base, rb, t, o, at); break;
            case 4: copy_piece<4>(base, rb, t, o, at); break;
            case 2: copy_piece<2>(base, rb, t, o, at); break;
            default: copy_piece<1>(base, rb, t, o, at); break;
        }
    }
    if (rank == 0 && tid == 0) p.dropped[b] = gone + (held - budget);
    ev_sync<C>();   // no CTA leaves while another may still read its count
}

template <int C>
cudaError_t launch_c(const KvEvictParams& p, cudaStream_t stream) {
    const int64_t per_cta = ((int64_t)p.n_rows + 32 * kEvWarps * C - 1) / (32 * kEvWarps * C) * 32 * kEvWarps;
    const size_t smem = sizeof(EvTail) + 4 * (size_t)(per_cta < kKeyCache ? per_cta : kKeyCache);
    // the limit belongs to the kernel, not to the call: always the most that any call takes, or a call from another host
    // thread could lower it between this one's two steps
    cudaError_t e = cudaFuncSetAttribute(kv_evict_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)(sizeof(EvTail) + 4 * (size_t)kKeyCache));
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)p.B * C);
    cfg.blockDim = dim3(kEvThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = C;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = C > 1 ? 1 : 0;
    e = cudaLaunchKernelEx(&cfg, kv_evict_kernel<C>, p);
    return e != cudaSuccess ? e : cudaGetLastError();
}

// CTAs per sequence: the C with the least estimate of waves x (start + a step per row of a CTA).  The constants (us) are
// fitted to one row lost of n: C = 1 takes 11 us at n = 2049 and 26 at 16,400 for any number of sequences up to the
// SMs, C = 8 17 and 19 for 8 sequences, but 54 for 32 and 161 for 128, since only 14 such clusters (32 of C = 4, 64 of
// C = 2) are resident at a time; 32 x 32,000 take 39, 30, 23 and 57 us with C = 1, 2, 4 and 8.  Rows past a CTA's
// key cache are read again in every pass, at three times the step.
int cluster_size(int B, int n_rows) {
    const int resident[4] = {device_num_sms(), 64, 32, 14};
    const float start[4] = {9.5f, 15.f, 15.5f, 16.5f};
    int best = 1;
    float least = 0.f;
    for (int i = 0; i < 4; ++i) {
        const float rows = (float)n_rows / (float)(1 << i), waves = (float)((B + resident[i] - 1) / resident[i]);
        const float t = waves * (start[i] + 0.00093f * rows * (rows > (float)kKeyCache ? 3.f : 1.f));
        if (i == 0 || t < least) {
            least = t;
            best = 1 << i;
        }
    }
    return best;
}

}  // namespace

cudaError_t launch_kv_evict(const KvEvictParams& p, cudaStream_t stream) {
    switch (cluster_size(p.B, p.n_rows)) {
        case 1: return launch_c<1>(p, stream);
        case 2: return launch_c<2>(p, stream);
        case 4: return launch_c<4>(p, stream);
        default: return launch_c<8>(p, stream);
    }
}

}  // namespace sti
