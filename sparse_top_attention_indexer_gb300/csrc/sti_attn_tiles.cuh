// sti_attn_tiles.cuh -- what the kernels that attend over every row of a cache share: the sizes of their tiles, descriptors,
// the reading of S^T, bounded waits, and the launch behind a kernel that is still ending.
#pragma once
#include <cuda_runtime.h>
#include <math.h>
#include <stddef.h>

#include "sti_attn_util.cuh"
#include "sti_ptx.cuh"

namespace sti {

constexpr int kRows = 64;                      // rows per tile
constexpr uint32_t kQBlk = 64 * 128;           // a Q column block: 64 heads x 64 dims
constexpr uint32_t kTBlk = kRows * 128;        // a tile column block: 64 rows x 64 dims
constexpr uint32_t kPBuf = kRows * 128;        // a P^T buffer: 64 rows x 64 heads
constexpr uint32_t kTmO = 128;                 // TMEM: S^T of tile parity b at columns [64 b, 64 b + 64), O^T d-block
                                               // m at [128 + 64 m, 192 + 64 m)
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.69314718055994531f;

__device__ __forceinline__ uint32_t lo32(uint64_t v) { return (uint32_t)v; }
__device__ __forceinline__ uint32_t hi32(uint64_t v) { return (uint32_t)(v >> 32); }

// Keep the value from being combined with constants ahead of time: the descriptors of a tile's 64 MMAs, all
// known before the loop, would otherwise be kept (and spilled) as 64 values instead of one and an add each.
__device__ __forceinline__ uint32_t opaque(uint32_t v) {
    asm volatile("" : "+r"(v));
    return v;
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
// kLast: the barrier is looked at once more after `abort`, which says that nobody arrives any more.
template <bool kLast = false>
__device__ __forceinline__ bool tile_wait(uint64_t* bar, uint32_t parity, uint32_t* status, volatile int* abort,
                                          uint64_t limit_ns = STI_WAIT_TIMEOUT_NS) {
    uint64_t t0 = 0;
    for (uint32_t i = 1;; ++i) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((i & 255u) == 0u) {
            if (*abort) return kLast && mbar_try_wait(bar, parity);
            const uint64_t now = global_timer_ns();
            if (t0 == 0) t0 = now;
            else if (now - t0 > limit_ns) {
                if (status) atomicOr(status, 2u /* STI_FLAG_TIMEOUT */);
                *abort = 1;
                return false;
            }
        }
    }
}

// tile_wait for a converged warp.  The vote makes the result visibly warp-uniform; without it the compiler
// treats what follows as divergent, and the MMAs of the issuing warp take three times as long to issue.
template <bool kLast = false>
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, uint32_t* status, volatile int* abort,
                                          uint64_t limit_ns = STI_WAIT_TIMEOUT_NS) {
    return __all_sync(kWarpFull, tile_wait<kLast>(bar, parity, status, abort, limit_ns));
}

// One lane of the (converged) warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
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
