// kv_append.cu -- quantise new cache rows to 4 bits and write them where the cache expects them.
//
// A group of G consecutive elements shares one scale s; an element x is stored as the E2M1 code of
// x / s (nearest of +-{0, .5, 1, 1.5, 2, 3, 4, 6}, ties to the even code, saturating, no negative zero):
//   G = 16 (compressed KV rows): s = the E4M3 value nearest to max|x| / 6 (0: the group is zeros)
//   G = 32 (MXFP4 index keys):   s = 2^X, X = floor(log2 max|x|) - 2 clamped to [-127, 127]
// A group holding a NaN gets the format's NaN scale and zero codes; infinities saturate.
//
// One thread takes 16 elements (two 16-byte loads, one 8-byte store of codes), so a G = 16 group
// needs no exchange and a G = 32 group one shuffle.  Maxima are taken on the bf16 bit patterns, two
// at a time.
// Rounding: q = x * (1/s) in fp32, with an approximate reciprocal, is off by less than 2^-21 (relative), which
// matters only where x / s is exactly halfway between two codes.  There x = t s with t a border of at most 3 bits and
// s of at most 4, while any other 8-bit x is at least 2^-8 (relative) away; so q is first rounded to
// 12 bits (2^-12 relative), which returns the exact border where x / s is one and moves nothing across
// a border otherwise; the hardware's conversion then breaks the tie to the even code.  (Checked on the CPU for every
// finite x and every s with the reciprocal up to two ulps off: tests/test_append_rounding.py.)
//
// Reads 2 bytes and writes 0.56 (0.53) per element.  65,536 rows of 512: 19.5 us, 4.4 TB/s of the 6.8 that a copy
// reaches; without the quantising arithmetic the same accesses take 14.2 us.  Bound by instruction issue: some 18
// instructions per element, and the schedulers issue in 84 % of their active cycles, with six warps ready on average.
// Two units per thread keep enough loads in flight (one: 25 us).
#include <cuda_bf16.h>
#include <cuda_fp4.h>
#include <cuda_fp8.h>

#include "sti_internal.h"
#include "sti_kvfp4.h"

namespace sti {
namespace {

constexpr int kAppendThreads = 256;
constexpr int kUnits = 2;   // 16-element units per thread, both loaded before either is used

// Rounded to 12 significant bits (ties away; see the header).
__device__ __forceinline__ float round12(float q) {
    return __uint_as_float((__float_as_uint(q) + 0x800u) & 0xFFFFF000u);
}
// x (bf16 pair) times r, rounded to 12 bits.
__device__ __forceinline__ float2 quotient12(uint32_t pair, float r) {
    return make_float2(round12(__uint_as_float(pair << 16) * r), round12(__uint_as_float(pair & 0xFFFF0000u) * r));
}

// Eight elements (four bf16 pairs) -> eight codes, element i in nibble i; negative zeros lose their sign.
__device__ __forceinline__ uint32_t e2m1x8(const uint4& v, float r) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t c = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        c |= (uint32_t)__nv_cvt_float2_to_fp4x2(quotient12(w[i], r), __NV_E2M1, cudaRoundNearest) << (8 * i);
    const uint32_t m = c & 0x77777777u;
    const uint32_t nz = (m | (m >> 1) | (m >> 2)) & 0x11111111u;
    return c & (0x77777777u | (nz << 3));
}

// Sixteen elements (v0, v1) -> codes, and the scale byte of their group.
template <bool MX>   // MX: MXFP4 (groups of 32, E8M0), else groups of 16 with E4M3
__device__ __forceinline__ uint2 quantise16(const uint4& v0, const uint4& v1, uint32_t& sbyte) {
    uint32_t mx = __vmaxu2(__vmaxu2(__vmaxu2(v0.x & 0x7FFF7FFFu, v0.y & 0x7FFF7FFFu),
                                    __vmaxu2(v0.z & 0x7FFF7FFFu, v0.w & 0x7FFF7FFFu)),
                           __vmaxu2(__vmaxu2(v1.x & 0x7FFF7FFFu, v1.y & 0x7FFF7FFFu),
                                    __vmaxu2(v1.z & 0x7FFF7FFFu, v1.w & 0x7FFF7FFFu)));
    mx = max(mx & 0xFFFFu, mx >> 16);   // the largest |x| as a bf16 pattern (NaN patterns are the largest)
    if (MX) mx = max(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 1));
    const bool nan = mx > 0x7F80u;
    float r;
    if (MX) {
        int X = (int)(mx >> 7) - 129;   // exponent field - bias - 2
        X = mx >= 0x7F80u ? 127 : max(X, -127);
        sbyte = nan ? 0xFFu : (uint32_t)(X + 127);
        r = X == 127 ? __uint_as_float(0x00400000u) : __uint_as_float((uint32_t)(127 - X) << 23);   // 2^-X
    } else {
        const float top = __uint_as_float(mx << 16);
        // (a border between two E4M3 values is 5 bits, so 6 of it is 7: the argument of the header holds here too)
        sbyte = nan ? 0x7Fu : (uint32_t)__nv_cvt_float_to_fp8(round12(top * (1.f / 6.f)), __NV_SATFINITE, __NV_E4M3);
        r = (sbyte & 0x7Fu) == 0u ? 0.f : __fdividef(1.f, e4m3_to_float(sbyte));
    }
    return nan ? make_uint2(0u, 0u) : make_uint2(e2m1x8(v0, r), e2m1x8(v1, r));
}

template <bool MX>
__global__ void __launch_bounds__(kAppendThreads) kv_append_kernel(const KvAppendParams p) {
    const uint32_t per_row = (uint32_t)p.dim / 16u;
    const uint32_t total = (uint32_t)p.m * per_row;
    for (int b = blockIdx.y; b < p.B; b += gridDim.y) {
        const uint16_t* xb = p.x + (int64_t)b * p.x_bstride;
        uint4 v[kUnits][2];
        uint32_t idx[kUnits];
#pragma unroll
        for (int k = 0; k < kUnits; ++k) {
            idx[k] = (blockIdx.x * kUnits + k) * kAppendThreads + threadIdx.x;
            const uint4* src = reinterpret_cast<const uint4*>(xb + (int64_t)min(idx[k], total - 1) * 16);   // rows are dense
            v[k][0] = __ldg(src);
            v[k][1] = __ldg(src + 1);
        }
        // 32-bit: start_pos < 2^31, so start_pos + s < 2^32 (64-bit divisions here cost more than the quantising)
        const uint32_t start = (uint32_t)__ldg(p.start_pos + b);
        const uint32_t first = start / (uint32_t)p.ratio;
        const int64_t done = (int64_t)((start + (uint32_t)p.s) / (uint32_t)p.ratio) - first;
        const int64_t row0 = (int64_t)first - (p.dropped ? __ldg(p.dropped + b) : 0);
#pragma unroll
        for (int k = 0; k < kUnits; ++k) {
            uint32_t sbyte;
            const uint2 c = quantise16<MX>(v[k][0], v[k][1], sbyte);
            const uint32_t i = idx[k] / per_row, g = idx[k] - i * per_row;
            if (idx[k] >= total || (int64_t)i >= done) continue;
            const int64_t row = row0 + i;
            if (row < 0 || row >= p.n_rows) {
                if (g == 0 && p.status) atomicOr(p.status, 1u /* STI_FLAG_INDEX_RANGE */);
                continue;
            }
            *reinterpret_cast<uint2*>(p.codes + (int64_t)b * p.codes_bstride + row * (p.dim / 2) + 8 * g) = c;
            uint8_t* sc = p.scales + (int64_t)b * p.scales_bstride;
            if (MX) {
                if ((g & 1u) == 0u) sc[row * (p.dim / 32) + (g >> 1)] = (uint8_t)sbyte;
            } else {
                sc[row * (p.dim / 16) + g] = (uint8_t)sbyte;
            }
            if (g == 0) {
                if (p.row_pos) p.row_pos[(int64_t)b * p.row_pos_bstride + row] = (int32_t)(first + i);
                if (p.row_weight) p.row_weight[(int64_t)b * p.row_weight_bstride + row] = 0.f;
            }
        }
    }
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendParams& p, bool mx, cudaStream_t stream) {
    const int64_t total = (int64_t)p.m * (p.dim / 16);
    const int64_t per_block = (int64_t)kUnits * kAppendThreads;
    const dim3 grid((unsigned)((total + per_block - 1) / per_block), (unsigned)(p.B < 65535 ? p.B : 65535));
    if (mx) kv_append_kernel<true><<<grid, kAppendThreads, 0, stream>>>(p);
    else kv_append_kernel<false><<<grid, kAppendThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace sti
