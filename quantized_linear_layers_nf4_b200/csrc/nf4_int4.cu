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
// the scale that is kept.  A group of zeros has s = 0 and q = z.  A NaN weight gets code 15
// and does not count for the extremes.
//
// Both are bound by HBM: 2 or 4 bytes of weight and half a byte of code per element.
// Codes are laid out as the NF4 ones are (row-major, element 2i in the high nibble of
// byte i); scales are [k / G, n], so that the 16 rows a matrix product works on have
// their scales of one group in one 32-byte sector.
//
// Quantization gives a warp several rows of one group, four loads of a lane in flight, and
// writes the rows' scales together.  Its quotient is Markstein's (nf4_encode.cuh), a clamp
// and an addition of 1.5 * 2^23 round it, and the eight integers of a word, in the low bits
// of those sums, are put together by one multiply-add each, the excess of all taken off
// at the end.  Over 11008 x 4096 in bf16, groups of 128, it takes 32 us (3.5 TB/s of 113 MB, 70 % of the
// issue slots and 62 % of the ALU pipe used; asymmetric 36), and 49 with the restoration behind it, which
// finds codes in L2; with one row a warp and divisions those two took 115.  Groups of no power of two
// (k_int4_quantize_any) read W twice: 68 us over 11008 x 3840 in groups of 192, 29 in groups of 128.
// Dequantization gives a thread the same word of eight rows; a nibble under
// the mantissa of 2^23 needs no shift, since its power of 16 goes into the scale: 21.9 us
// (5.2 TB/s, 81 % of the rate of a copy), with one row a thread 37.
#include "nf4_common.cuh"
#include "nf4_encode.cuh"
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
// The word of eight weights: code 2i in bits 8i + 4 .., code 2i + 1 in bits 8i .., by a divisor d in
// Markstein's range with its rounded reciprocal.  Clamped before it is rounded (the bound is
// an integer), and from above alone: rint(lo / s) + z is 0 or more, since rint is odd and z
// was not cut off (s is within 2^-8 of (hi - lo) / 15), and the symmetric form's quotients
// stay under 7.5.  In that form too the minimum is taken: it makes a NaN quotient the largest code,
// where its sum's bits would reach into the other weights' nibbles.
template <bool kZero>
__device__ __forceinline__ uint32_t encode_fast(const float (&v)[8], float d, float r, float z) {
    const uint64_t rr = f2(r, r), nd = f2(-d, -d), magic = f2(12582912.0f, 12582912.0f);  // 1.5 * 2^23
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint64_t x = f2(v[2 * i], v[2 * i + 1]), q0 = mul2(x, rr);
        const uint64_t q = fma2(fma2(q0, nd, x), rr, q0);
        float a, b;
        asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(q));
        uint64_t t;
        asm("add.rn.f32x2 %0, %1, %2;" : "=l"(t) : "l"(f2(fminf(a, 15.0f - z), fminf(b, 15.0f - z))), "l"(magic));
        w += static_cast<uint32_t>(t) * (16u << (8 * i)) + static_cast<uint32_t>(t >> 32) * (1u << (8 * i));
    }
    return w - (0x4B400000u - static_cast<uint32_t>(z)) * 0x11111111u;
}
template <bool kZero>
__device__ __forceinline__ uint32_t encode(const float (&v)[8], float d, float r, float z) {
    if (markstein_ok(d)) return encode_fast<kZero>(v, d, r, z);
    uint32_t w = 0;  // the same by division, NaN again the largest code
#pragma unroll
    for (int j = 0; j < 8; ++j)
        w |= static_cast<uint32_t>(fmaxf(fminf(__fadd_rn(rintf(__fdiv_rn(v[j], d)), z), 15.0f), 0.0f)) << (8 * (j >> 1) + ((j & 1) ? 0 : 4));
    return w;
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

template <bool kZero>
__device__ __forceinline__ void extremes(const float (&v)[8], float& lo, float& hi) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        hi = fmaxf(hi, kZero ? v[j] : fabsf(v[j]));
        if (kZero) lo = fminf(lo, v[j]);
    }
}
__device__ __forceinline__ void put_scale(void* scale, bool f32, int64_t at, float s) {
    if (f32) reinterpret_cast<float*>(scale)[at] = s;
    else reinterpret_cast<__nv_bfloat16*>(scale)[at] = __float2bfloat16_rn(s);
}

// Eight weights as they are in memory.
template <bool kBf16>
struct Eight {
    uint4 r[kBf16 ? 1 : 2];
    __device__ __forceinline__ void load(const void* W, int64_t i) {
#pragma unroll
        for (int j = 0; j < (kBf16 ? 1 : 2); ++j) r[j] = __ldcs(reinterpret_cast<const uint4*>(W) + (kBf16 ? i : 2 * i + j));
    }
    __device__ __forceinline__ void floats(float (&v)[8]) const {
        const uint32_t u[4] = {r[0].x, r[0].y, r[0].z, r[0].w};
        if (kBf16) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[2 * j] = __uint_as_float(u[j] << 16);
                v[2 * j + 1] = __uint_as_float(u[j] & 0xffff0000u);
            }
        } else {
            const uint32_t x[4] = {r[kBf16 ? 0 : 1].x, r[kBf16 ? 0 : 1].y, r[kBf16 ? 0 : 1].z, r[kBf16 ? 0 : 1].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[j] = __uint_as_float(u[j]);
                v[4 + j] = __uint_as_float(x[j]);
            }
        }
    }
    template <bool kZero>
    __device__ __forceinline__ void extremes(float& lo, float& hi) const {
        lo = hi = 0.0f;
        if (kBf16) {  // two at a time
            const uint32_t u[4] = {r[0].x, r[0].y, r[0].z, r[0].w};
            __nv_bfloat162 top, low;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t m = kZero ? u[j] : u[j] & 0x7fff7fffu;
                const __nv_bfloat162 x = *reinterpret_cast<const __nv_bfloat162*>(&m);
                top = j ? __hmax2(top, x) : x;
                if (kZero) low = j ? __hmin2(low, x) : x;
            }
            hi = fmaxf(0.0f, fmaxf(__low2float(top), __high2float(top)));
            if (kZero) lo = fminf(0.0f, fminf(__low2float(low), __high2float(low)));
        } else {
            float v[8];
            floats(v);
            int4::extremes<kZero>(v, lo, hi);
        }
    }
};

// Four values of each of kLanes lanes to the four results, one in each quarter of the lanes: up1, up0 are
// the bits of its number.
template <int kLanes, typename Op>
__device__ __forceinline__ float quarter_reduce(const float (&x)[4], bool up1, bool up0, Op&& op) {
    const float a = op(up1 ? x[2] : x[0], __shfl_xor_sync(kFull, up1 ? x[0] : x[2], kLanes / 2));
    const float b = op(up1 ? x[3] : x[1], __shfl_xor_sync(kFull, up1 ? x[1] : x[3], kLanes / 2));
    float r = op(up0 ? b : a, __shfl_xor_sync(kFull, up0 ? a : b, kLanes / 4));
#pragma unroll
    for (int o = kLanes / 8; o > 0; o >>= 1) r = op(r, __shfl_xor_sync(kFull, r, o));
    return r;
}

// Groups of 8 kLanes weights (32 .. 256): a warp has kRows rows of one group, 32 / kLanes of
// them at a time.
template <bool kZero, int kLanes, bool kBf16>
__global__ void __launch_bounds__(256) k_int4_quantize(const void* __restrict__ W, int64_t n, int64_t k, uint32_t* __restrict__ wq,
                                                       void* __restrict__ scale, bool scale_f32, uint8_t* __restrict__ zero) {
    constexpr int kAtOnce = 32 / kLanes, kLoads = 4, kRows = kAtOnce * kLoads;
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x & 31, sub = lane % kLanes, mine = lane / kLanes;
    const int64_t groups = k / (8 * kLanes), chunks = k / 8;
    const int64_t tasks = (n + kRows - 1) / kRows * groups;
    const int64_t warps = (static_cast<int64_t>(gridDim.x) * blockDim.x) >> 5;
    for (int64_t task = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5; task < tasks; task += warps) {
        const int64_t block = (task >> 32) == 0 ? static_cast<uint32_t>(task) / static_cast<uint32_t>(groups) : task / groups;
        const int64_t grp = task - block * groups, row0 = block * kRows + mine;
        const int64_t first = row0 * chunks + grp * kLanes + sub;
        Eight<kBf16> v[kLoads];
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            if (row0 + i * kAtOnce < n) v[i].load(W, first + i * kAtOnce * chunks);
            else v[i] = Eight<kBf16>{};
        }
        // Two halvings of the lanes halve the rows each keeps, so a row's extremes end in a quarter of
        // its lanes, which make its scale for all: with all rows reduced in all lanes it took 16
        // shuffles a lane in place of 5, and 3 us more (with a restoration, 11008 x 4096).
        float lo[kLoads], hi[kLoads];
#pragma unroll
        for (int i = 0; i < kLoads; ++i) v[i].template extremes<kZero>(lo[i], hi[i]);
        const bool up1 = (lane & (kLanes / 2)) != 0, up0 = (lane & (kLanes / 4)) != 0;
        const float high = quarter_reduce<kLanes>(hi, up1, up0, [](float x, float y) { return fmaxf(x, y); });
        const float low = kZero ? quarter_reduce<kLanes>(lo, up1, up0, [](float x, float y) { return fminf(x, y); }) : 0.0f;
        float s, d, z;
        group_params<kZero>(low, high, scale_f32, s, d, z);
        const float r = __frcp_rn(d);
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int from = mine * kLanes + (i >> 1) * (kLanes / 2) + (i & 1) * (kLanes / 4);
            const float di = __shfl_sync(kFull, d, from), ri = __shfl_sync(kFull, r, from), zi = kZero ? __shfl_sync(kFull, z, from) : 8.0f;
            float x[8];
            v[i].floats(x);
            if (row0 + i * kAtOnce < n) wq[first + i * kAtOnce * chunks] = encode<kZero>(x, di, ri, zi);
        }
        const int64_t row = row0 + ((up1 ? 2 : 0) + (up0 ? 1 : 0)) * kAtOnce;
        if (lane % (kLanes / 4) == 0 && row < n) {
            put_scale(scale, scale_f32, grp * n + row, s);
            if (kZero) zero[grp * n + row] = static_cast<uint8_t>(z);
        }
    }
}

// Any group: a warp each, read a second time (from L2) for its codes.
template <bool kZero>
__global__ void __launch_bounds__(256) k_int4_quantize_any(const void* __restrict__ W, bool bf16, int64_t n, int64_t k, int group,
                                                           uint32_t* __restrict__ wq, void* __restrict__ scale, bool scale_f32,
                                                           uint8_t* __restrict__ zero) {
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t per_row = k / group, groups = n * per_row;
    const int chunks = group / 8;
    const int64_t warps = (static_cast<int64_t>(gridDim.x) * blockDim.x) >> 5;
    for (int64_t gi = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5; gi < groups; gi += warps) {
        const int64_t base = gi * chunks, row = gi / per_row;
        float v[8], lo = 0.0f, hi = 0.0f, s, d, z;
        for (int c = lane; c < chunks; c += 32) {
            load8(W, bf16, base + c, v);
            extremes<kZero>(v, lo, hi);
        }
        for (int o = 16; o > 0; o >>= 1) {
            hi = fmaxf(hi, __shfl_xor_sync(kFull, hi, o));
            if (kZero) lo = fminf(lo, __shfl_xor_sync(kFull, lo, o));
        }
        group_params<kZero>(lo, hi, scale_f32, s, d, z);
        const float r = __frcp_rn(d);
        for (int c = lane; c < chunks; c += 32) {
            load8(W, bf16, base + c, v);
            wq[base + c] = encode<kZero>(v, d, r, z);
        }
        if (lane == 0) {
            const int64_t at = (gi - row * per_row) * n + row;
            put_scale(scale, scale_f32, at, s);
            if (kZero) zero[at] = static_cast<uint8_t>(z);
        }
    }
}

// (q - z) s of a word's eight codes, each rounded once.
__device__ __forceinline__ void decode8(uint32_t w, float s, float z, float (&v)[8]) {
    if (fabsf(s) >= 0x1p-110f) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t u = h ? w >> 16 : w;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                // nibbles 2i + 1 (first element) and 2i of the half word: 2^23 + 16^p q, less 2^23 + 16^p z,
                // times 16^-p s, whose product rounds as (q - z) s does
                const float p1 = static_cast<float>(1 << (8 * i + 4)), p0 = static_cast<float>(1 << (8 * i));
                const float a = __uint_as_float((u & (0xf0u << (8 * i))) | 0x4B000000u), b = __uint_as_float((u & (0xfu << (8 * i))) | 0x4B000000u);
                const uint64_t off = f2(-__fmaf_rn(z, p1, 8388608.0f), -__fmaf_rn(z, p0, 8388608.0f));
                uint64_t t;
                asm("add.rn.f32x2 %0, %1, %2;" : "=l"(t) : "l"(f2(a, b)), "l"(off));
                t = mul2(t, f2(s * (1.0f / p1), s * (1.0f / p0)));
                asm("mov.b64 {%0, %1}, %2;" : "=f"(v[4 * h + 2 * i]), "=f"(v[4 * h + 2 * i + 1]) : "l"(t));
            }
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = __fmul_rn(static_cast<float>((w >> (8 * (j >> 1) + ((j & 1) ? 0 : 4))) & 15u) - z, s);
}

// A thread has word c of kRows rows: a group's scales of those lie together.
template <bool kBf16>
__global__ void __launch_bounds__(256) k_int4_dequantize(const uint32_t* __restrict__ wq, const void* __restrict__ scale,
                                                         bool scale_f32, const uint8_t* __restrict__ zero, int64_t n,
                                                         int64_t k, int group, void* __restrict__ out) {
    constexpr int kRows = kBf16 ? 8 : 4;
    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t per_row = k / 8, tasks = (n + kRows - 1) / kRows * per_row;
    const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.x;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < tasks; i += step) {
        const int64_t block = (i >> 32) == 0 ? static_cast<uint32_t>(i) / static_cast<uint32_t>(per_row) : i / per_row;
        const uint32_t c = static_cast<uint32_t>(i - block * per_row);
        const int64_t row0 = block * kRows, at = static_cast<int64_t>(c * 8u / static_cast<uint32_t>(group)) * n + row0;
        uint32_t w[kRows];
        float s[kRows], z[kRows];
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            if (row0 + r >= n) break;
            w[r] = __ldcs(wq + (row0 + r) * per_row + c);
            s[r] = scale_f32 ? __ldg(reinterpret_cast<const float*>(scale) + at + r)
                             : __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(scale)[at + r]);
            z[r] = zero ? static_cast<float>(__ldg(zero + at + r) & 15) : 8.0f;
        }
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            if (row0 + r >= n) break;
            float v[8];
            decode8(w[r], s[r], z[r], v);
            const int64_t o = (row0 + r) * per_row + c;
            if (kBf16) {
                __stcs(reinterpret_cast<uint4*>(out) + o, make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                                    pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])));
            } else {
                __stcs(reinterpret_cast<float4*>(out) + 2 * o, make_float4(v[0], v[1], v[2], v[3]));
                __stcs(reinterpret_cast<float4*>(out) + 2 * o + 1, make_float4(v[4], v[5], v[6], v[7]));
            }
        }
    }
}

}  // namespace int4

static dim3 grid_for(int64_t threads, const DeviceInfo& dev) {
    const int64_t blocks = (threads + 255) / 256, cap = static_cast<int64_t>(dev.sm_count) * 8;
    return dim3(static_cast<unsigned>(blocks < cap ? blocks : cap));
}

cudaError_t launch_int4_quantize(const void* W, bool w_bf16, int64_t n, int64_t k, int64_t group, uint8_t* wq, void* scale,
                                 bool scale_f32, uint8_t* zero, const DeviceInfo& dev, cudaStream_t stream) {
    uint32_t* words = reinterpret_cast<uint32_t*>(wq);
#define NF4_INT4_QUANTIZE(Z, L)                                                                                             \
    (w_bf16 ? launch_pdl(int4::k_int4_quantize<Z, L, true>, quantize_grid(L), dim3(256), stream, W, n, k, words, scale, scale_f32, zero) \
            : launch_pdl(int4::k_int4_quantize<Z, L, false>, quantize_grid(L), dim3(256), stream, W, n, k, words, scale, scale_f32, zero))
#define NF4_INT4_QUANTIZE_Z(L) (zero ? NF4_INT4_QUANTIZE(true, L) : NF4_INT4_QUANTIZE(false, L))
    auto quantize_grid = [&](int lanes) { return grid_for((n * lanes + 127) / 128 * (k / group) * 32, dev); };
    switch (group) {
        case 32: return NF4_INT4_QUANTIZE_Z(4);
        case 64: return NF4_INT4_QUANTIZE_Z(8);
        case 128: return NF4_INT4_QUANTIZE_Z(16);
        case 256: return NF4_INT4_QUANTIZE_Z(32);
    }
#undef NF4_INT4_QUANTIZE_Z
#undef NF4_INT4_QUANTIZE
    const dim3 grid = grid_for(n * (k / group) * 32, dev);
    if (zero)
        return launch_pdl(int4::k_int4_quantize_any<true>, grid, dim3(256), stream, W, w_bf16, n, k, static_cast<int>(group), words,
                          scale, scale_f32, zero);
    return launch_pdl(int4::k_int4_quantize_any<false>, grid, dim3(256), stream, W, w_bf16, n, k, static_cast<int>(group), words, scale,
                      scale_f32, zero);
}

cudaError_t launch_int4_dequantize(const Int4Args& w, void* out, bool out_bf16, const DeviceInfo& dev, cudaStream_t stream) {
    const uint32_t* words = reinterpret_cast<const uint32_t*>(w.wq);
    const int rows = out_bf16 ? 8 : 4;
    const dim3 grid = grid_for((w.n + rows - 1) / rows * (w.k / 8), dev);
    if (out_bf16)
        return launch_pdl(int4::k_int4_dequantize<true>, grid, dim3(256), stream, words, w.scale, w.scale_f32, w.zero, w.n, w.k,
                          static_cast<int>(w.group), out);
    return launch_pdl(int4::k_int4_dequantize<false>, grid, dim3(256), stream, words, w.scale, w.scale_f32, w.zero, w.n, w.k,
                      static_cast<int>(w.group), out);
}

}  // namespace nf4
