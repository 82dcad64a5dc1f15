// nf4_few.cuh -- the parts that the few-token kernels share (nf4_int4_gemv.cu,
// nf4_moe.cu): 4-bit weights from global memory straight into the fragments of
// mma.sync, with the group scales applied to the products and not to the weights.
//
// For a row r and a group b of its weights, sum_c x_c w_c = s_b sum_c x_c v_c with
// v_c the unscaled value of the code (an integer q - z, or a codebook level), so
// the scale costs one multiply-add per output and group instead of one multiply
// per weight.  q - z is exact in fp16 and bf16.
//
// One item is 16 rows x 64 k: lane (g, t) = (lane / 4, lane % 4) holds the codes of
// rows g and g + 8, eight bytes each, i.e. the 16 consecutive k from 16 t on; four
// m16n8k16 products consume them.  The order of k inside a product is free as long
// as both operands agree, so nothing is shuffled between lanes: a warp reads 32
// consecutive bytes of each row, whole sectors, and the matching 32 bytes of X.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "nf4_common.cuh"
#include "nf4_decode.cuh"

namespace nf4 {
namespace few {

constexpr int kItemK = 64;  // k of one item

// Codes are read once: no L1 line is kept for them.
__device__ __forceinline__ uint2 ldg_codes(const uint8_t* p) {
    uint2 v;
    asm volatile("ld.global.nc.L1::no_allocate.L2::256B.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
    return v;
}
__device__ __forceinline__ uint32_t ldg_code32(const uint8_t* p) {
    uint32_t v;
    asm volatile("ld.global.nc.L2::256B.u32 %0, [%1];" : "=r"(v) : "l"(p));
    return v;
}

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t m, uint32_t o) {  // (a & m) | o
    uint32_t d;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(a), "r"(m), "r"(o));
    return d;
}
__device__ __forceinline__ uint32_t sub_bf16x2(uint32_t a, uint32_t b) {
    const __nv_bfloat162 r = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t sub_f16x2(uint32_t a, uint32_t b) {
    const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t fma_f16x2(uint32_t a, uint32_t b, uint32_t c) {
    const __half2 r = __hfma2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b),
                              *reinterpret_cast<const __half2*>(&c));
    return *reinterpret_cast<const uint32_t*>(&r);
}

// Eight integer codes of one word (element 2i in the high nibble of byte i) as
// q - z in bf16, pairs (1,5), (0,4), (3,7), (2,6): a nibble under the mantissa of
// 128 is 128 + q, and 128 + z (zoff, both halves) is taken off exactly.
__device__ __forceinline__ void int4_bf16(uint32_t w, uint32_t zoff, uint32_t (&o)[4]) {
    o[0] = sub_bf16x2(and_or(w, 0x000f000fu, 0x43004300u), zoff);
    o[1] = sub_bf16x2(and_or(w >> 4, 0x000f000fu, 0x43004300u), zoff);
    o[2] = sub_bf16x2(and_or(w >> 8, 0x000f000fu, 0x43004300u), zoff);
    o[3] = sub_bf16x2(and_or(w >> 12, 0x000f000fu, 0x43004300u), zoff);
}
__device__ __forceinline__ uint32_t zoff_bf16(uint32_t z) { return (0x4300u + z) * 0x10001u; }  // 128 + z, z <= 15

// The same in fp16, whose ten mantissa bits hold the high nibble in place:
// 1024 + q, and 1024 + 16 q scaled by 1/16; zlo = 1024 + z, zhi = -(64 + z).
__device__ __forceinline__ void int4_f16(uint32_t w, uint32_t zlo, uint32_t zhi, uint32_t (&o)[4]) {
    const uint32_t v = w >> 8;
    o[0] = sub_f16x2(and_or(w, 0x000f000fu, 0x64006400u), zlo);
    o[1] = fma_f16x2(and_or(w, 0x00f000f0u, 0x64006400u), 0x2c002c00u, zhi);
    o[2] = sub_f16x2(and_or(v, 0x000f000fu, 0x64006400u), zlo);
    o[3] = fma_f16x2(and_or(v, 0x00f000f0u, 0x64006400u), 0x2c002c00u, zhi);
}
__device__ __forceinline__ uint32_t zlo_f16(uint32_t z) { return (0x6400u + z) * 0x10001u; }           // 1024 + z
__device__ __forceinline__ uint32_t zhi_f16(uint32_t z) { return (0xd400u + (z << 4)) * 0x10001u; }    // -(64 + z)

// The pairs of X that go with int4_*: (1,5), (0,4) | (3,7), (2,6) from the natural
// pairs (0,1), (2,3), (4,5), (6,7) of eight values.
__device__ __forceinline__ void pair_x(uint32_t x01, uint32_t x23, uint32_t x45, uint32_t x67, uint32_t (&o)[4]) {
    o[0] = prmt(x01, x45, 0x7632);
    o[1] = prmt(x01, x45, 0x5410);
    o[2] = prmt(x23, x67, 0x7632);
    o[3] = prmt(x23, x67, 0x5410);
}

// Integer weights with group scales: scale [k / G, n], zero [k / G, n] or null
// (then 8).  Groups are numbered by 64-k item: item b is in group b / items_per
// (by a multiply: exact while the number of items squared stays under 2^32), or,
// with G = 32, holds groups 2 b and 2 b + 1.
struct Int4Sides {
    const void* scale;
    const uint8_t* zero;
    int64_t n;
    uint32_t magic;  // floor(2^32 / items_per) + 1, 0 when items_per is 1
    int f32;         // scales are fp32 (bf16 otherwise)
};
__host__ __device__ inline uint32_t items_magic(int64_t items_per) {
    return items_per <= 1 ? 0u : static_cast<uint32_t>((1ull << 32) / static_cast<uint64_t>(items_per) + 1);
}
__device__ __forceinline__ uint32_t group_of(const Int4Sides& s, uint32_t item) {
    return s.magic ? __umulhi(item, s.magic) : item;
}
__device__ __forceinline__ uint32_t ldg_scale(const Int4Sides& s, int64_t at) {  // raw bits, widened by scale_f
    return s.f32 ? __ldg(reinterpret_cast<const uint32_t*>(s.scale) + at)
                 : static_cast<uint32_t>(__ldg(reinterpret_cast<const uint16_t*>(s.scale) + at)) << 16;
}
__device__ __forceinline__ uint32_t ldg_zero(const Int4Sides& s, int64_t at) {
    return s.zero ? (__ldg(s.zero + at) & 15u) : 8u;
}

}  // namespace few
}  // namespace nf4
