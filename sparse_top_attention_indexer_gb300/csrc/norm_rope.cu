// norm_rope.cu -- per-head RMS norm and rotation by position in one pass over the rows, written in place of the heads or
// into the rows of a paged cache.
//
// Row x of d elements at position P:
//   y = x / sqrt(mean(x^2) + eps) * w        (norm; w: optional)
//   (y_a, y_b) of pair i of the rotated range <- gain * (y_a cos t - y_b sin t, y_b cos t + y_a sin t),  t = P f_i
// pairs (2i, 2i + 1) or (i, i + rd / 2) of dims [off, off + rd); the inverse turns by -t.  All in fp32, rounded once.
//
// Angles: f_i comes as turns per position in units of 2^-64, so P f_i mod 1 is one 64-bit integer product, exact for
// every 32-bit position (in fp32 the angle of position 10^6 is off by 2^-5 radians, its rounding).  The nearest quarter
// turn is taken off in integers; what is left, at most an eighth of a turn, converts to fp32 and goes to sincospif.
//
// A block first computes the (cos, sin) of its tokens' pairs, one each per thread, into shared memory; they serve
// all heads of the token.  LPR lanes share a row, 8 elements (16 bytes) per lane and chunk; kRowsAhead rows per slot are
// loaded before the first is used.
#include <cuda_bf16.h>

#include "sti_internal.h"
#include "sti_ptx.cuh"

namespace sti {
namespace {

constexpr int kThreads = 256;
constexpr int kRowsAhead = 4;

struct Shape {          // how a block divides its rows
    int heads_at_once;  // row slots that work on one token's heads
    int tokens;         // tokens per block
    int per;            // heads per slot
    int blocks_h;       // blocks that share a token's heads
};

// (cos, sin) of 2 pi turns / 2^64.
__device__ __forceinline__ float2 cos_sin(uint64_t turns) {
    const uint64_t q = (turns + (1ull << 61)) >> 62;                     // nearest quarter, mod 4
    const float r = (float)(int64_t)(turns - (q << 62)) * 0x1p-63f;      // the rest in half turns, [-1/4, 1/4]
    float s, c;
    sincospif(r, &s, &c);
    switch ((int)q & 3) {
        case 0: return make_float2(c, s);
        case 1: return make_float2(-s, c);
        case 2: return make_float2(-c, -s);
        default: return make_float2(s, -c);
    }
}

__device__ __forceinline__ void unpack(const uint4& v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

// LPR lanes per row, CH chunks of 8 elements per lane
template <int LPR, int CH>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(const NormRopeParams p, const Shape sh) {
    extern __shared__ float2 cs[];                      // [tokens][rd / 2]
    const int slot = threadIdx.x / LPR, li = threadIdx.x % LPR;
    const int pairs = p.rd / 2;
    const int64_t tokens = (int64_t)p.B * p.s;
    const int64_t tok0 = (int64_t)(blockIdx.x / (unsigned)sh.blocks_h) * sh.tokens;
    const int tb = slot / sh.heads_at_once, head0 = slot - tb * sh.heads_at_once + (int)(blockIdx.x % (unsigned)sh.blocks_h) * sh.per * sh.heads_at_once;
    auto position = [&](int64_t tok) {
        return p.pos_per_token ? __ldg(p.pos + tok) : (int)((uint32_t)__ldg(p.pos + tok / p.s) + (uint32_t)(tok % p.s));
    };
    const int64_t tok = tok0 + tb;
    const int b = (int)(min(tok, tokens - 1) / p.s), t = (int)(min(tok, tokens - 1) - (int64_t)b * p.s);
    const bool live = tok < tokens && tb < sh.tokens && (!p.n_new || t < __ldg(p.n_new + b));
    const int chunks = p.d / 8;
    const uint16_t* xrow = p.x + (int64_t)b * p.x_bstride + (int64_t)t * p.x_tstride;
    uint4 v[kRowsAhead][CH];
    auto load = [&](int k) {
#pragma unroll
        for (int r = 0; r < kRowsAhead; ++r) {
            const int head = head0 + (k + r) * sh.heads_at_once;
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                const int c = li + LPR * i;
                v[r][i] = make_uint4(0, 0, 0, 0);
                if (live && k + r < sh.per && head < p.h && c < chunks)
                    v[r][i] = *reinterpret_cast<const uint4*>(xrow + (int64_t)head * p.d + 8 * c);
            }
        }
    };
    load(0);
    for (int i = threadIdx.x; i < sh.tokens * pairs; i += kThreads) {
        const int tk = i / pairs, pr = i - tk * pairs;
        if (tok0 + tk < tokens) {
            float2 v2 = cos_sin((uint64_t)(int64_t)position(tok0 + tk) * __ldg(reinterpret_cast<const unsigned long long*>(p.turns) + pr));
            cs[i] = make_float2(v2.x * p.gain, (p.inverse ? -v2.y : v2.y) * p.gain);
        }
    }
    __syncthreads();
    uint16_t* yrow;
    if (p.y) {
        yrow = p.y + (int64_t)b * p.y_bstride + (int64_t)t * p.y_tstride;
    } else {
        yrow = nullptr;
        if (live) {
            const uint32_t at = (uint32_t)position(tok), pg = at / (uint32_t)p.page_size;
            const int id = pg < (uint32_t)p.max_pages ? __ldg(p.table + (int64_t)b * p.table_stride + pg) : -1;
            if (id >= 0 && id < p.n_pages)
                yrow = p.pages + (int64_t)id * p.page_stride + (int64_t)(at - pg * (uint32_t)p.page_size) * p.d;
            else if (li == 0 && p.status)
                atomicOr(p.status, 1u /* STI_FLAG_INDEX_RANGE */);
        }
    }
    const float2* my = cs + tb * pairs;
    const int c_lo = p.off / 8, c_hi = (p.off + p.rd) / 8, half = p.rd / 16;
    for (int k = 0; k < sh.per; k += kRowsAhead) {
#pragma unroll
        for (int r = 0; r < kRowsAhead; ++r) {
            const int head = head0 + (k + r) * sh.heads_at_once;
            const bool on = live && k + r < sh.per && head < p.h;
            // the pairs' other halves, before anything of the row is written
            uint4 other[CH];
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                const int c = li + LPR * i;
                other[i] = make_uint4(0, 0, 0, 0);
                if (p.halves && on && c >= c_lo && c < c_hi)
                    other[i] = *reinterpret_cast<const uint4*>(xrow + (int64_t)head * p.d + 8 * (c < c_lo + half ? c + half : c - half));
            }
            float scale = 1.f;
            if (p.norm) {
                float sum = 0.f;
#pragma unroll
                for (int i = 0; i < CH; ++i) {
                    float f[8];
                    unpack(v[r][i], f);
#pragma unroll
                    for (int j = 0; j < 8; ++j) sum = fmaf(f[j], f[j], sum);
                }
#pragma unroll
                for (int o = LPR / 2; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
                scale = rsqrtf(sum / (float)p.d + p.eps);
            }
            __syncwarp();
            if (!on || !yrow) continue;
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                const int c = li + LPR * i;
                if (c >= chunks) continue;
                float f[8];
                unpack(v[r][i], f);
#pragma unroll
                for (int j = 0; j < 8; ++j) f[j] *= scale;
                if (p.weight) {
                    float w[8];
                    unpack(__ldg(reinterpret_cast<const uint4*>(p.weight) + c), w);
#pragma unroll
                    for (int j = 0; j < 8; ++j) f[j] *= w[j];
                }
                if (c >= c_lo && c < c_hi) {
                    if (p.halves) {
                        const bool low = c < c_lo + half;
                        const int oc = low ? c + half : c - half;
                        float g[8];
                        unpack(other[i], g);
#pragma unroll
                        for (int j = 0; j < 8; ++j) g[j] *= scale;
                        if (p.weight) {
                            float w[8];
                            unpack(__ldg(reinterpret_cast<const uint4*>(p.weight) + oc), w);
#pragma unroll
                            for (int j = 0; j < 8; ++j) g[j] *= w[j];
                        }
                        const float2* a = my + 8 * ((low ? c : oc) - c_lo);
#pragma unroll
                        for (int j = 0; j < 8; ++j) f[j] = low ? f[j] * a[j].x - g[j] * a[j].y : f[j] * a[j].x + g[j] * a[j].y;
                    } else {
                        const float2* a = my + 4 * (c - c_lo);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float x = f[2 * j], z = f[2 * j + 1];
                            f[2 * j] = x * a[j].x - z * a[j].y;
                            f[2 * j + 1] = z * a[j].x + x * a[j].y;
                        }
                    }
                }
                *reinterpret_cast<uint4*>(yrow + (int64_t)head * p.d + 8 * c) =
                    make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
            }
        }
        if (k + kRowsAhead < sh.per) load(k + kRowsAhead);
    }
}

template <int LPR, int CH>
cudaError_t launch(const NormRopeParams& p, int num_sms, cudaStream_t stream) {
    constexpr int slots = kThreads / LPR;
    const int64_t tokens = (int64_t)p.B * p.s;
    Shape sh;
    sh.heads_at_once = 1;
    while (sh.heads_at_once < p.h && sh.heads_at_once < slots) sh.heads_at_once *= 2;
    sh.tokens = slots / sh.heads_at_once;
    sh.per = (p.h + sh.heads_at_once - 1) / sh.heads_at_once;
    const int64_t blocks_t = (tokens + sh.tokens - 1) / sh.tokens;
    auto blocks_h = [&](int per) { return (p.h + per * sh.heads_at_once - 1) / (per * sh.heads_at_once); };
    // few tokens: their heads go to several blocks
    while (sh.per > 1 && blocks_t * blocks_h(sh.per) < num_sms) sh.per = (sh.per + 1) / 2;
    sh.blocks_h = blocks_h(sh.per);
    const size_t smem = (size_t)sh.tokens * (p.rd / 2) * sizeof(float2);
    norm_rope_kernel<LPR, CH><<<(unsigned)(blocks_t * sh.blocks_h), kThreads, smem, stream>>>(p, sh);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeParams& p, int num_sms, cudaStream_t stream) {
    const int chunks = p.d / 8;
    if (chunks <= 4) return launch<4, 1>(p, num_sms, stream);
    if (chunks <= 8) return launch<8, 1>(p, num_sms, stream);
    if (chunks <= 16) return launch<16, 1>(p, num_sms, stream);
    if (chunks <= 32) return launch<32, 1>(p, num_sms, stream);
    if (chunks <= 64) return launch<32, 2>(p, num_sms, stream);
    return launch<32, 4>(p, num_sms, stream);
}

}  // namespace sti
