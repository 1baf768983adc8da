// norm_rope.cu -- per-head RMS norm and rotation by position in one pass over the rows, written in place of the heads or
// into the rows of a paged cache.
//
// Row x of d elements at position P:
//   y = x / sqrt(mean(x^2) + eps) * w        (norm; w: optional)
//   (y_a, y_b) of pair i of the rotated range <- gain * (y_a cos t - y_b sin t, y_b cos t + y_a sin t),  t = P f_i
// pairs (2i, 2i + 1) or (i, i + rd / 2) of dims [off, off + rd); the inverse turns by -t.  All in fp32, rounded once.
//
// Angles: f_i comes as turns per position in units of 2^-64, so P f_i mod 1 is one 64-bit integer product, exact for
// every 32-bit position (in fp32 the angle of position 10^6 is off by 2^-5 radians, its rounding).
//
// A block takes the heads of one token, or with few heads several tokens.  It first computes the (cos, sin) of its tokens'
// pairs, spread over its threads, into shared memory, where they serve all heads.  LPR lanes share a row, 8 elements
// (16 bytes) per lane and chunk; U rows per slot are loaded before the first is used, the first ones before the angles.
//
// Many rows are bound by HBM: queries of 4096 tokens, 64 heads x 512, 82 us, 0.97 of the measured copy rate (0.90 to 0.95 for 64
// to 256 dims, 0.85 to 0.95 with 8 heads).  Rows of one head are bound by the way to a block's first row (its place, its position, its
// angles) and by instructions, some 400 per row: 8 x 8192 tokens of which half are padding 20 us (10 at the copy rate).  Steps of that:
// several tokens per block and rows in flight 109 -> 39 us, places looked up once per token -> 32, angles by polynomials -> 23,
// two fp32 per instruction and four blocks per SM -> 20.
#include <cuda_bf16.h>

#include "sti_attn_tiles.cuh"   // launch_after
#include "sti_internal.h"
#include "sti_ptx.cuh"

namespace sti {
namespace {

constexpr int kRowThreads = 256;
constexpr int kPerSlot = 8;        // rows that a block takes per slot, where there are enough (8 heads x 512: 0.92 of the copy rate, 4 0.88,
                                   // 2 0.83, one token per block 0.57)
constexpr int kPad = 2;            // between tokens' angles: whole powers of two would put them all to the same banks
constexpr int kMaxAngles = 4096;   // pairs of a block's tokens: 32 KB

struct Shape {      // a block's rows: `tokens` tokens of `heads` heads each
    int tokens, heads;
    int blocks_h;   // blocks that share a token's heads
    int lanes;      // log2 of the threads that take a token's pairs
};

// (cos, sin) of 2 pi turns / 2^64.  With the nearest quarter turn off, x = 2 pi r is at most pi/4 = 0.786, where the
// Taylor polynomials of degree 9 and 10 are off by x^11 / 11! < 2^-28 and x^12 / 12! < 2^-32.  (sincospif, made for
// every argument, takes four times the instructions, a third of what an appended row took.)
__device__ __forceinline__ float2 cos_sin(uint64_t turns) {
    const uint32_t top = (uint32_t)(turns >> 32);                        // 2^-32 of a turn is 1.5e-9
    const uint32_t q = (top + (1u << 29)) >> 30;                         // nearest quarter, mod 4
    const float x = (float)(int)(top - (q << 30)) * 1.46291808e-9f;      // 2 pi 2^-32
    const float y = x * x;
    const float s = x + x * y * (-1.f / 6 + y * (1.f / 120 + y * (-1.f / 5040 + y * (1.f / 362880))));
    const float c = 1.f + y * (-1.f / 2 + y * (1.f / 24 + y * (-1.f / 720 + y * (1.f / 40320 + y * (-1.f / 3628800)))));
    const float a = q & 1 ? s : c, b = q & 1 ? c : s;                    // cos turns to -sin, sin to cos
    return make_float2((q + 1) & 2 ? -a : a, q & 2 ? -b : b);
}

// Two fp32 at a time, in one instruction each.
__device__ __forceinline__ uint64_t pack2(float x, float y) {
    uint64_t v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(x), "f"(y));
    return v;
}
__device__ __forceinline__ float2 parts2(uint64_t v) {
    float2 f;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
    return f;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t v;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(a), "l"(b));
    return v;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t v;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(v) : "l"(a), "l"(b), "l"(c));
    return v;
}

__device__ __forceinline__ void unpack(const uint4& v, uint64_t (&f)[4]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = pack2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
}

// LPR lanes per row, CH chunks of 8 elements per lane, U rows at a time.  kHalves: pairs (i, i + rd / 2); a lane has both
// chunks of its pairs then (fetched again by the lane of either: 64 heads x 64 0.58 of the copy rate, here 0.86).
template <int LPR, int CH, int U, bool kHalves>
__global__ void __launch_bounds__(kRowThreads, CH <= 2 ? 4 : CH == 3 ? 3 : 2) norm_rope_kernel(const NormRopeParams p, const Shape sh) {
    static_assert(!kHalves || CH % 2 == 0, "");
    constexpr int kSlots = kRowThreads / LPR;
    extern __shared__ __align__(16) float2 cs[];                      // [tokens][rd / 2], then the tokens' places
    const int slot = threadIdx.x / LPR, li = threadIdx.x % LPR;
    const int pairs = p.rd / 2, row_pairs = pairs + kPad;
    int64_t* from = reinterpret_cast<int64_t*>(cs + sh.tokens * row_pairs);   // of its first head in x, -1: padding or past the end
    int64_t* to = from + sh.tokens;                                       // of its first head in y, its row's in the pages (-1: none)
    int* at = reinterpret_cast<int*>(to + sh.tokens);                     // its position
    const uint32_t bt = sh.blocks_h == 1 ? blockIdx.x : blockIdx.x / (uint32_t)sh.blocks_h;
    const uint32_t tok0 = bt * (uint32_t)sh.tokens;
    const int head0 = (int)(blockIdx.x - bt * (uint32_t)sh.blocks_h) * sh.heads;
    const int rows = sh.tokens * sh.heads;
    const int chunks = p.d / 8;
    // Which chunks a lane has, and of which unit of angles: a chunk's four pairs, or the eight of two chunks half a range apart.
    // A unit's angles lie in pieces of two, piece j of all units side by side.
    constexpr int kPieces = kHalves ? 4 : 2;
    const int c_lo = p.off / 8, units = p.rd / (4 * kPieces);
    auto unit_of = [&](int k) { return kHalves ? li + LPR * (k >> 1) : li + LPR * k - c_lo; };
    auto turns_at = [&](int k) { return (uint32_t)unit_of(k) < (uint32_t)units; };   // whether chunk k is rotated
    auto chunk = [&](int k) {
        if (!kHalves) return li + LPR * k;
        const int u = unit_of(k), rest = 2 * (u - units) + (k & 1);   // (of the chunks outside the range)
        return u < units ? c_lo + u + (k & 1) * units : rest < c_lo ? rest : rest + 2 * units;
    };
    // the next kernel may start to be set up, the one before has to be done
    griddep_launch_dependents();
    griddep_wait();
    uint32_t b = 0, t = 0;
    int pos = 0;
    if ((int)threadIdx.x < sh.tokens) {
        const uint32_t tok = tok0 + threadIdx.x;
        int64_t place = -1;
        if (tok < (uint32_t)p.B * (uint32_t)p.s) {      // (below 2^31)
            b = tok / (uint32_t)p.s;
            t = tok - b * (uint32_t)p.s;
            pos = p.pos_per_token ? __ldg(p.pos + tok) : (int)((uint32_t)__ldg(p.pos + b) + t);
            if (!p.n_new || (int)t < __ldg(p.n_new + b)) place = (int64_t)b * p.x_bstride + (int64_t)t * p.x_tstride;
        }
        from[threadIdx.x] = place;
    }
    __syncthreads();
    uint4 v[U][CH];
    const uint16_t* src[U];                             // null: not a row of this block, or a padding token's
    int tk[U];                                          // its token among the block's
    auto load = [&](int i0) {
#pragma unroll
        for (int r = 0; r < U; ++r) {
            const int i = i0 + r * kSlots;
            tk[r] = sh.tokens == 1 ? 0 : sh.heads == 1 ? i : i / sh.heads;
            const int head = head0 + i - tk[r] * sh.heads;
            src[r] = nullptr;
            if (i < rows && head < p.h && from[tk[r]] >= 0) src[r] = p.x + from[tk[r]] + (int64_t)head * p.d;
#pragma unroll
            for (int k = 0; k < CH; ++k) {
                v[r][k] = make_uint4(0, 0, 0, 0);
                if (src[r] && chunk(k) < chunks) v[r][k] = *reinterpret_cast<const uint4*>(src[r] + 8 * chunk(k));
            }
        }
    };
    load(slot);
    if ((int)threadIdx.x < sh.tokens && from[threadIdx.x] >= 0) {
        at[threadIdx.x] = pos;
        int64_t place;
        if (p.y) {
            place = (int64_t)b * p.y_bstride + (int64_t)t * p.y_tstride;
        } else {
            const uint32_t pg = (uint32_t)pos / (uint32_t)p.page_size;
            const int id = pg < (uint32_t)p.max_pages ? __ldg(p.table + (int64_t)b * p.table_stride + pg) : -1;
            const bool good = id >= 0 && id < p.n_pages;
            place = good ? (int64_t)id * p.page_stride + (int64_t)((uint32_t)pos - pg * (uint32_t)p.page_size) * p.d : -1;
            if (!good && p.status) atomicOr(p.status, 1u /* STI_FLAG_INDEX_RANGE */);
        }
        to[threadIdx.x] = place;
    }
    __syncthreads();
    // 2^sh.lanes threads side by side take a token's pairs
    for (int pr = threadIdx.x & ((1 << sh.lanes) - 1); pr < pairs; pr += 1 << sh.lanes) {
        const uint64_t f = __ldg(reinterpret_cast<const unsigned long long*>(p.turns) + pr);
        for (int i = threadIdx.x >> sh.lanes; i < sh.tokens; i += kRowThreads >> sh.lanes) {
            if (from[i] < 0) continue;
            const float2 a = cos_sin((uint64_t)(int64_t)at[i] * f);
            cs[i * row_pairs + ((pr / 2 % kPieces) * units + pr / (2 * kPieces)) * 2 + (pr & 1)] =
                make_float2(a.x * p.gain, (p.inverse ? -a.y : a.y) * p.gain);
        }
    }
    uint64_t weight[CH][4];
#pragma unroll
    for (int k = 0; k < CH; ++k) {
        uint4 w = make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);   // ones
        if (p.weight && chunk(k) < chunks) w = __ldg(reinterpret_cast<const uint4*>(p.weight) + chunk(k));
        unpack(w, weight[k]);
    }
    __syncthreads();
    for (int i0 = slot;;) {
#pragma unroll
        for (int r = 0; r < U; ++r) {
            uint64_t f[CH][4];
#pragma unroll
            for (int k = 0; k < CH; ++k) unpack(v[r][k], f[k]);
            float scale = 1.f;
            if (p.norm) {
                uint64_t sq = 0;
#pragma unroll
                for (int k = 0; k < CH; ++k)
#pragma unroll
                    for (int j = 0; j < 4; ++j) sq = fma2(f[k][j], f[k][j], sq);
                float sum = parts2(sq).x + parts2(sq).y;
#pragma unroll
                for (int o = LPR / 2; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
                scale = rsqrtf(sum * p.inv_d + p.eps);
            }
            if (!src[r]) continue;
            uint16_t* dst = p.y ? p.y : p.pages;        // where the row goes
            if (to[tk[r]] < 0) continue;
            dst += to[tk[r]] + (int64_t)(head0 + i0 + r * kSlots - tk[r] * sh.heads) * p.d;
            const float2* my = cs + tk[r] * row_pairs;
            auto angles = [&](int k, int j) { return *reinterpret_cast<const float4*>(my + 2 * (j * units + unit_of(k))); };
            const uint64_t scale2 = pack2(scale, scale);
            auto write = [&](int k, const float2 (&x)[4]) {
                if (chunk(k) < chunks)
                    *reinterpret_cast<uint4*>(dst + 8 * chunk(k)) = make_uint4(pack_bf16x2(x[0].x, x[0].y), pack_bf16x2(x[1].x, x[1].y),
                                                                              pack_bf16x2(x[2].x, x[2].y), pack_bf16x2(x[3].x, x[3].y));
            };
#pragma unroll
            for (int k = 0; k < CH; k += kHalves ? 2 : 1) {
                float2 x[4], z[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    x[j] = parts2(mul2(mul2(f[k][j], scale2), weight[k][j]));
                    if (kHalves) z[j] = parts2(mul2(mul2(f[k + kHalves][j], scale2), weight[k + kHalves][j]));
                }
                if (turns_at(k)) {
                    if (kHalves) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float4 a = angles(k, j);
                            const float2 u = x[j], w = z[j];
                            x[j] = make_float2(u.x * a.x - w.x * a.y, u.y * a.z - w.y * a.w);
                            z[j] = make_float2(w.x * a.x + u.x * a.y, w.y * a.z + u.y * a.w);
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 4; j += 2) {
                            const float4 a = angles(k, j / 2);
                            const float2 u = x[j], w = x[j + 1];
                            x[j] = make_float2(u.x * a.x - u.y * a.y, u.y * a.x + u.x * a.y);
                            x[j + 1] = make_float2(w.x * a.z - w.y * a.w, w.y * a.z + w.x * a.w);
                        }
                    }
                }
                write(k, x);
                if (kHalves) write(k + kHalves, z);
            }
        }
        i0 += U * kSlots;
        if (i0 - slot >= rows) break;   // (the same for all of the block)
        load(i0);
    }
}

template <int LPR, int CH, int U, bool kHalves>
cudaError_t launch(const NormRopeParams& p, int num_sms, cudaStream_t stream) {
    constexpr int slots = kRowThreads / LPR;
    const int64_t tokens = (int64_t)p.B * p.s;
    auto up = [](int64_t n, int64_t m) { return (n + m - 1) / m; };
    Shape sh;
    sh.heads = p.h;
    sh.tokens = kPerSlot * slots / p.h;
    if (sh.tokens < 1) sh.tokens = 1;
    if (sh.tokens > kRowThreads) sh.tokens = kRowThreads;
    if (p.rd > 0 && sh.tokens > kMaxAngles / (p.rd / 2)) sh.tokens = kMaxAngles / (p.rd / 2);
    // few tokens: fewer per block (two waves of blocks), then their heads to several blocks, as long as every slot has a row
    while (sh.tokens > 1 && sh.tokens * p.h > slots && up(tokens, sh.tokens) < 8 * num_sms) sh.tokens = (sh.tokens + 1) / 2;
    while (sh.tokens == 1 && sh.heads > slots && tokens * up(p.h, sh.heads) < 2 * num_sms) sh.heads = (sh.heads + 1) / 2;
    sh.blocks_h = (int)up(p.h, sh.heads);
    sh.lanes = 0;
    while (1 << sh.lanes < p.rd / 2 && 1 << sh.lanes < kRowThreads) ++sh.lanes;
    const size_t smem = (size_t)sh.tokens * ((p.rd / 2 + kPad) * sizeof(float2) + 2 * sizeof(int64_t) + sizeof(int));
    return launch_after(norm_rope_kernel<LPR, CH, U, kHalves>, dim3((unsigned)(up(tokens, sh.tokens) * sh.blocks_h)), kRowThreads,
                        smem, stream, p, sh);
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeParams& p, int num_sms, cudaStream_t stream) {
    const int chunks = p.d / 8;
    // Two chunks per lane where they fit the row: 8 heads x 128 0.91 of the copy rate, one per lane 0.60; three for what lies between
    // (320 dims leave three lanes in eight idle otherwise: 0.84, with two 0.74).
    if (p.halves) {
        if (chunks <= 8) return launch<4, 2, 2, true>(p, num_sms, stream);
        if (chunks <= 16) return launch<8, 2, 2, true>(p, num_sms, stream);
        if (chunks <= 32) return launch<16, 2, 2, true>(p, num_sms, stream);
        if (chunks <= 64) return launch<32, 2, 2, true>(p, num_sms, stream);
        return launch<32, 4, 1, true>(p, num_sms, stream);
    }
    if (chunks <= 4) return launch<4, 1, 2, false>(p, num_sms, stream);
    if (chunks <= 8) return launch<4, 2, 2, false>(p, num_sms, stream);
    if (chunks <= 16) return launch<8, 2, 2, false>(p, num_sms, stream);
    if (chunks <= 32) return launch<16, 2, 2, false>(p, num_sms, stream);
    if (chunks <= 48) return launch<16, 3, 2, false>(p, num_sms, stream);
    if (chunks <= 64) return launch<32, 2, 2, false>(p, num_sms, stream);
    if (chunks <= 96) return launch<32, 3, 2, false>(p, num_sms, stream);
    return launch<32, 4, 1, false>(p, num_sms, stream);
}

}  // namespace sti
