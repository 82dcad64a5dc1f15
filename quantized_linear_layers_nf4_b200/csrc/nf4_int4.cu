// nf4_int4.cu -- integer 4-bit weights with one scale (and zero point) per group of
// consecutive weights of a row: quantization and dequantization (sm_100a).
//
//   symmetric   s = max|w| / 7,                 q = clamp(rint(w / s) + 8, 0, 15), z = 8
//   asymmetric  s = (max(w,0) - min(w,0)) / 15, z = clamp(rint(-min(w,0) / s), 0, 15),
//               q = clamp(rint(w / s) + z, 0, 15)
//   out = (q - z) s
//
// Every step is one fp32 operation rounded to nearest even; s is rounded to its
// storage type before anything is divided by it, so the codes are the best ones for
// the scale that is kept.  A group of zeros has s = 0 and q = z.
//
// Both are bound by HBM: 2 or 4 bytes of weight and half a byte of code per element.
// Codes are laid out as the NF4 ones are (row-major, element 2i in the high nibble of
// byte i); scales are [k / G, n], so that the 16 rows a matrix product works on have
// their scales of one group in one 32-byte sector.
#include "nf4_common.cuh"
#include "nf4_internal.h"
#include "nf4_ptx.cuh"

namespace nf4 {
namespace int4 {

__device__ __forceinline__ float scale_round(float s, bool f32) { return f32 ? s : __bfloat162float(__float2bfloat16_rn(s)); }

// Scale, divisor and zero point of a group from its extremes.
template <bool kZero>
__device__ __forceinline__ void group_params(float lo, float hi, bool f32, float& s, float& d, float& z) {
    s = scale_round(kZero ? __fdiv_rn(__fsub_rn(hi, lo), 15.0f) : __fdiv_rn(hi, 7.0f), f32);
    d = s > 0.0f ? s : 1.0f;
    z = kZero ? fminf(fmaxf(rintf(__fdiv_rn(-lo, d)), 0.0f), 15.0f) : 8.0f;
}
__device__ __forceinline__ uint32_t code(float w, float d, float z) {
    return static_cast<uint32_t>(fminf(fmaxf(__fadd_rn(rintf(__fdiv_rn(w, d)), z), 0.0f), 15.0f));
}

__device__ __forceinline__ void load8(const void* W, bool bf16, int64_t i, float (&v)[8]) {  // elements 8i .. 8i + 7
    if (bf16) {
        const uint4 r = __ldcs(reinterpret_cast<const uint4*>(W) + i);
        const uint32_t u[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[2 * j] = bf16_bits_to_float(u[j] & 0xffffu);
            v[2 * j + 1] = __uint_as_float(u[j] & 0xffff0000u);
        }
    } else {
        const float4 a = __ldcs(reinterpret_cast<const float4*>(W) + 2 * i), b = __ldcs(reinterpret_cast<const float4*>(W) + 2 * i + 1);
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
}

// `lanes` consecutive lanes of a warp (4 .. 32, a power of two) share a group, each
// with G / lanes elements in chunks of eight `lanes` apart; a group that 32 lanes do
// not hold in one chunk each is read a second time (from L2) for its codes.
template <bool kZero>
__global__ void __launch_bounds__(256) k_int4_quantize(const void* __restrict__ W, bool bf16, int64_t n, int64_t k, int group,
                                                       int lanes, uint32_t* __restrict__ wq, void* __restrict__ scale,
                                                       bool scale_f32, uint8_t* __restrict__ zero) {
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int sub = lane & (lanes - 1);
    const int64_t per_row = k / group, groups = n * per_row;
    const int64_t per_warp = 32 / lanes;
    const int chunks = group / 8;  // of a group
    const int64_t warps = (static_cast<int64_t>(gridDim.x) * blockDim.x) >> 5;
    const int64_t rounds = (groups + warps * per_warp - 1) / (warps * per_warp);
    int64_t gi = ((static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5) * per_warp + lane / lanes;
    for (int64_t it = 0; it < rounds; ++it, gi += warps * per_warp) {
        const bool live = gi < groups;
        const int64_t base = (live ? gi : 0) * chunks;
        float v[8], lo = 0.0f, hi = 0.0f;
        for (int c = sub; c < chunks; c += lanes) {
            load8(W, bf16, base + c, v);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                hi = fmaxf(hi, kZero ? v[j] : fabsf(v[j]));
                if (kZero) lo = fminf(lo, v[j]);
            }
        }
        for (int o = lanes >> 1; o > 0; o >>= 1) {
            hi = fmaxf(hi, __shfl_xor_sync(kFull, hi, o));
            if (kZero) lo = fminf(lo, __shfl_xor_sync(kFull, lo, o));
        }
        float s, d, z;
        group_params<kZero>(lo, hi, scale_f32, s, d, z);
        if (!live) continue;
        for (int c = sub; c < chunks; c += lanes) {
            if (chunks > lanes) load8(W, bf16, base + c, v);
            uint32_t w = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) w |= code(v[j], d, z) << (8 * (j >> 1) + ((j & 1) ? 0 : 4));
            wq[base + c] = w;
        }
        if (sub == 0) {
            const int64_t at = (gi % per_row) * n + gi / per_row;
            if (scale_f32) reinterpret_cast<float*>(scale)[at] = s;
            else reinterpret_cast<__nv_bfloat16*>(scale)[at] = __float2bfloat16_rn(s);
            if (kZero) zero[at] = static_cast<uint8_t>(z);
        }
    }
}

__global__ void __launch_bounds__(256) k_int4_dequantize(const uint32_t* __restrict__ wq, const void* __restrict__ scale,
                                                         bool scale_f32, const uint8_t* __restrict__ zero, int64_t n,
                                                         int64_t k, int group, void* __restrict__ out, bool bf16) {
    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t words = n * k / 8, per_row = k / 8;
    const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.x;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < words; i += step) {
        const uint32_t w = __ldcs(wq + i);
        const int64_t row = i / per_row;
        const int64_t at = ((i - row * per_row) * 8 / group) * n + row;
        const float s = scale_f32 ? __ldg(reinterpret_cast<const float*>(scale) + at)
                                  : __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(scale)[at]);
        const float z = zero ? static_cast<float>(__ldg(zero + at) & 15) : 8.0f;
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = __fmul_rn(static_cast<float>((w >> (8 * (j >> 1) + ((j & 1) ? 0 : 4))) & 15u) - z, s);
        if (bf16) {
            __stcs(reinterpret_cast<uint4*>(out) + i, make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                                pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])));
        } else {
            __stcs(reinterpret_cast<float4*>(out) + 2 * i, make_float4(v[0], v[1], v[2], v[3]));
            __stcs(reinterpret_cast<float4*>(out) + 2 * i + 1, make_float4(v[4], v[5], v[6], v[7]));
        }
    }
}

}  // namespace int4

cudaError_t launch_int4_quantize(const void* W, bool w_bf16, int64_t n, int64_t k, int64_t group, uint8_t* wq, void* scale,
                                 bool scale_f32, uint8_t* zero, const DeviceInfo& dev, cudaStream_t stream) {
    int lanes = 4;
    while (lanes < 32 && group % (lanes * 16) == 0) lanes *= 2;
    const int64_t warps = (n * (k / group) * lanes + 31) / 32;
    int64_t blocks = (warps + 7) / 8;
    const int64_t cap = static_cast<int64_t>(dev.sm_count) * 8;
    if (blocks > cap) blocks = cap;
    const dim3 grid(static_cast<unsigned>(blocks));
    if (zero)
        return launch_pdl(int4::k_int4_quantize<true>, grid, dim3(256), stream, W, w_bf16, n, k, static_cast<int>(group), lanes,
                          reinterpret_cast<uint32_t*>(wq), scale, scale_f32, zero);
    return launch_pdl(int4::k_int4_quantize<false>, grid, dim3(256), stream, W, w_bf16, n, k, static_cast<int>(group), lanes,
                      reinterpret_cast<uint32_t*>(wq), scale, scale_f32, zero);
}

cudaError_t launch_int4_dequantize(const Int4Args& w, void* out, bool out_bf16, const DeviceInfo& dev, cudaStream_t stream) {
    int64_t blocks = (w.n * w.k / 8 + 255) / 256;
    const int64_t cap = static_cast<int64_t>(dev.sm_count) * 8;
    if (blocks > cap) blocks = cap;
    return launch_pdl(int4::k_int4_dequantize, dim3(static_cast<unsigned>(blocks)), dim3(256), stream,
                      reinterpret_cast<const uint32_t*>(w.wq), w.scale, w.scale_f32, w.zero, w.n, w.k, static_cast<int>(w.group),
                      out, out_bf16);
}

}  // namespace nf4
