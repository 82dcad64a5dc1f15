// nf4_few.cuh -- the parts that the few-token kernels share (nf4_int4_gemv.cu,
// nf4_moe.cu): 4-bit weights from global memory straight into the fragments of
// mma.sync, with the group scales applied to the products and not to the weights.
//
// For a row r and a group b of its weights, sum_c x_c w_c = s_b sum_c x_c v_c with
// v_c the unscaled value of the code (an integer q - z, or a codebook level), so
// the scale costs one multiply-add per output and group instead of one multiply
// per weight.  q - z is exact in fp16.
//
// X comes as fp16 times a power of two per token: exact for every bf16 value down to
// 2^-31 of the largest one it is scaled by.  fp16 and not bf16, because its mantissa
// holds a code's high nibble in place (one operation less for half of the codes) and
// a codebook level to 2^-11.
//
// One step is 16 rows x 128 k, 64 bytes of codes a row.  They go from global to shared memory
// by asynchronous copies of 16 bytes, one a lane, kDepth steps ahead in a ring that each warp
// has to itself (registers for that would halve the warps an SM can run), and from there
// to lane (g, t) = (lane / 4, lane % 4), 16 bytes of each of its rows g and g + 8: four words
// of eight codes; a word of all four lanes is 32 k, two m16n8k16 products.  The order of k
// inside a product is free as long as both operands agree, so a lane keeps runs of
// consecutive codes.  What a run may be depends on the groups, since a product must not
// mix two of them:
//   kG128  groups of whole steps: 16 consecutive bytes, one scale a row and step
//   kG64   groups of 64: 8 consecutive bytes of each half
//   kG32   groups of 32: 4 consecutive bytes of each quarter
//   kTable codebook levels with the absmax of each 64: as kG64
// The copies and what feeds them reach 5.4 TB/s without the products; what the products add is
// about 9 instructions a word of codes (integer), or a look-up a byte in a table in shared
// memory (codebook: L1's data pipe is 70 % busy over a whole kernel, 84 % at its best), beside the
// steps' own bookkeeping (all in all 150 to 250 instructions a step).
// Scales go to registers, four groups of a row at a time (a window: kG128 four steps, kG64 and
// kTable two, kG32 one): lane (g, t) loads that of group t for its rows, one window ahead, and a
// shuffle hands it to the other lanes of the row.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include "nf4_common.cuh"
#include "nf4_decode.cuh"

namespace nf4 {
namespace few {

constexpr int kItemK = 64;   // the unit that k is a multiple of
constexpr int kStepK = 128;  // k of a step; its second half may lie past the end of k (see multiply)
constexpr int kStepBytes = 16 * kStepK / 2;

// A kernel's CTA has either W warps, which fill an SM, or half of them where a call gives it
// few steps, so that the next kernel's CTAs find room and start while its last ones run.
constexpr int kFewSteps = 96;  // of a CTA: up to here half the warps

// The warp's number as a value that the compiler sees to be one for all its lanes.
__device__ __forceinline__ int warp_index() { return static_cast<int>(__reduce_max_sync(kFull, threadIdx.x >> 5)); }

enum Fmt { kTable = 0, kG128 = 1, kG64 = 2, kG32 = 3 };

// Codes are read once: past L1.  `bytes` 16, or 0 to fill with zeros and read nothing.
__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t* src, int bytes) {
    asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t* src) {
    asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {  // all but the last N groups of this thread's copies have landed
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                              uint32_t b1) {  // onto zero
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t m, uint32_t o) {  // (a & m) | o
    uint32_t d;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(a), "r"(m), "r"(o));
    return d;
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

// Eight integer codes of one word (element 2i in the high nibble of byte i) as q - z in
// fp16, pairs (1,5), (0,4), (3,7), (2,6): a nibble under the mantissa of 1024 is
// 1024 + q, and four bits higher 1024 + 16 q, brought to q - z by one subtraction
// (zlo = 1024 + z) or one multiply-add (1/16, zhi = -(64 + z)), both exact.
__device__ __forceinline__ void int4_f16(uint32_t w, uint32_t zlo, uint32_t zhi, uint32_t (&o)[4]) {
    const uint32_t v = w >> 8;
    o[0] = sub_f16x2(and_or(w, 0x000f000fu, 0x64006400u), zlo);
    o[1] = fma_f16x2(and_or(w, 0x00f000f0u, 0x64006400u), 0x2c002c00u, zhi);
    o[2] = sub_f16x2(and_or(v, 0x000f000fu, 0x64006400u), zlo);
    o[3] = fma_f16x2(and_or(v, 0x00f000f0u, 0x64006400u), 0x2c002c00u, zhi);
}
// From a zero point in both halves of a word.
__device__ __forceinline__ uint32_t zlo_f16(uint32_t zz) { return zz + 0x64006400u; }         // 1024 + z
__device__ __forceinline__ uint32_t zhi_f16(uint32_t zz) { return zz * 16u + 0xd400d400u; }   // -(64 + z)

// The pairs of X that go with int4_f16, from the natural pairs of eight values.
__device__ __forceinline__ void pair_x(uint32_t x01, uint32_t x23, uint32_t x45, uint32_t x67, uint32_t (&o)[4]) {
    o[0] = prmt(x01, x45, 0x7632);
    o[1] = prmt(x01, x45, 0x5410);
    o[2] = prmt(x23, x67, 0x7632);
    o[3] = prmt(x23, x67, 0x5410);
}

// Two bf16 values times a power of two, as fp16.
__device__ __forceinline__ uint32_t scale_pair(uint32_t x, float factor) {
    const __half2 h = __floats2half2_rn(bf16_bits_to_float(x & 0xffffu) * factor, __uint_as_float(x & 0xffff0000u) * factor);
    return *reinterpret_cast<const uint32_t*>(&h);
}
// The power of two that brings a positive number of biased exponent ex to [2^14, 2^15),
// and its reciprocal; zero, tiny and non-finite ones take the nearest for which both
// are normal numbers.
__device__ __forceinline__ int scale_exponent(int ex) { return min(max(ex, 15), 254); }
__device__ __forceinline__ float scale_up(int ex) { return __int_as_float((127 + 14 + 127 - ex) << 23); }
__device__ __forceinline__ float scale_down(int ex) { return __int_as_float((ex - 14) << 23); }

// What another kernel writes while this one may already run (a programmatic dependent,
// past its wait): not the read-only path.
__device__ __forceinline__ uint4 ld_global16(const void* p) {
    uint4 v;
    asm volatile("ld.global.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
    return v;
}

// ------------------------------- weights -------------------------------
struct Weight {
    const uint8_t* wq;
    int64_t n;
    int k;
    // integer codes: scale [k / group, n], zero the same or null (then 8)
    const void* scale;
    const uint8_t* zero;
    uint32_t scale_row;  // bytes of scales of one group
    int per;         // kG128, kG64: steps, items (of 64 k) of a group; 1
    int units;       // of a row: kG128 steps, kG64 and kTable items, kG32 groups
    int f32;         // scales are fp32 (bf16 otherwise)
    // codebook codes
    const int8_t* absmax_q;
    const float* absmax_scale;
    const float* mu;
    int codebook;
};
// Steps of a window, and groups (kG128: or parts of one) of a step.
template <int F>
constexpr int window_steps() { return F == kG128 ? 4 : (F == kG32 ? 1 : 2); }

// The scales of a lane's two rows.
template <int F, bool Z>
struct Sides {
    const uint8_t* s[2];  // of the rows' first group; absmax codes
    const uint8_t* z[2];
    const float* e[2];    // kTable: scale of the rows' first absmax code, and that code's place under it
    uint32_t at[2];
    uint32_t raw_s[2], raw_z[2];  // of the next window, as loaded: anything done to it would wait for it
    bool past;            // the lane's group of it is past the end of k
    float f[2];           // of this window
    uint32_t zz[2];       // zero points of this window, in both halves

    __device__ __forceinline__ void aim(const Weight& w, const int64_t (&row)[2]) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (F == kTable) {
                const int64_t first = row[i] * w.units;
                s[i] = reinterpret_cast<const uint8_t*>(w.absmax_q) + first;
                e[i] = w.absmax_scale + (first >> 8);
                at[i] = static_cast<uint32_t>(first) & 255u;
            } else {
                s[i] = reinterpret_cast<const uint8_t*>(w.scale) + (w.f32 ? 4 * row[i] : 2 * row[i]);
                if (Z) z[i] = w.zero + row[i];
            }
        }
    }
    __device__ __forceinline__ void load(const Weight& w, int window, int t) {
        past = F != kG128 && 4 * window + t >= w.units;
        const uint32_t unit = min(4 * window + t, w.units - 1);
        if (F == kTable) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                raw_z[i] = static_cast<uint32_t>(static_cast<int32_t>(__ldg(reinterpret_cast<const int8_t*>(s[i] + unit))));
                raw_s[i] = __float_as_uint(__ldg(e[i] + ((at[i] + unit) >> 8)));
            }
            return;
        }
        const uint32_t grp = F == kG32 || w.per == 1 ? unit : unit / static_cast<uint32_t>(w.per);
        const uint64_t to = static_cast<uint64_t>(grp) * w.scale_row;
        if (w.f32) {
#pragma unroll
            for (int i = 0; i < 2; ++i) raw_s[i] = __ldg(reinterpret_cast<const uint32_t*>(s[i] + to));
        } else {
#pragma unroll
            for (int i = 0; i < 2; ++i) raw_s[i] = __ldg(reinterpret_cast<const uint16_t*>(s[i] + to));
        }
        if (Z) {
            const uint64_t tz = static_cast<uint64_t>(grp) * static_cast<uint32_t>(w.n);
#pragma unroll
            for (int i = 0; i < 2; ++i) raw_z[i] = __ldg(z[i] + tz);
        }
    }
    __device__ __forceinline__ void turn(const Weight& w, float mu) {  // the next window becomes this one
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (F == kTable) f[i] = absmax_hat(static_cast<int>(raw_z[i]), __uint_as_float(raw_s[i]), mu);
            else f[i] = __uint_as_float(raw_s[i] << (w.f32 ? 0 : 16));
            if (F != kG128 && past) f[i] = 0.0f;
            if (Z) zz[i] = prmt(raw_z[i], 0u, 0x4040) & 0x000f000fu;
        }
    }
};

// The 16-byte chunk c of row r (0 .. 7) of a step in its ring entry: chunks are permuted so that
// reads of 4, 8 and 16 bytes a lane all find 128 different bytes.
__device__ __forceinline__ uint32_t ring_place(int r, int c) {
    return 64u * r + 16u * (c ^ (((r >> 1) & 1) << 1 | ((r >> 2) & 1)));
}

// The two levels of each byte value as fp16, one copy a bank, 256 bytes an entry (the
// second half of it stays unused), so that a byte above a bank's offset is an address.
constexpr int kTableBytes = 256 * 256;
__device__ __forceinline__ void build_table(uint8_t* tab, int codebook) {
    // a lane holds one level; the two of a byte come by shuffles, and go to 16 bytes of its entry
    const float mine = kCodebook[codebook][threadIdx.x & 15];
    for (int i = threadIdx.x; i < 256 * 8; i += blockDim.x) {  // whole warps
        const int v = i >> 3;
        const __half2 e = __floats2half2_rn(__shfl_sync(kFull, mine, v >> 4), __shfl_sync(kFull, mine, v & 15));
        const uint32_t u = *reinterpret_cast<const uint32_t*>(&e);
        *reinterpret_cast<uint4*>(tab + 256 * v + 16 * (i & 7)) = make_uint4(u, u, u, u);
    }
}

// The four words of a lane's row g (entry + 512: row g + 8) from a ring entry; `at`: the lane's
// offsets in it.
struct Places {
    uint32_t put;     // where the lane's copies go
    uint32_t get[4];  // kG128: one; kG64, kTable: of each half; kG32: of each quarter
};
template <int F>
__device__ __forceinline__ Places places(int g, int t) {
    Places o;
    o.put = ring_place(g, t);
#pragma unroll
    for (int j = 0; j < 4; ++j)
        o.get[j] = F == kG128 ? o.put : (F == kG32 ? ring_place(g, j) + 4 * t : ring_place(g, 2 * (j & 1) + (t >> 1)) + 8 * (t & 1));
    return o;
}
template <int F>
__device__ __forceinline__ void ring_words(const uint8_t* entry, const Places& at, uint32_t (&v)[4]) {
    if (F == kG128) {
        const uint4 u = *reinterpret_cast<const uint4*>(entry + at.get[0]);
        v[0] = u.x; v[1] = u.y; v[2] = u.z; v[3] = u.w;
    } else if (F == kG32) {
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = *reinterpret_cast<const uint32_t*>(entry + at.get[j]);
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint2 u = *reinterpret_cast<const uint2*>(entry + at.get[h]);
            v[2 * h] = u.x;
            v[2 * h + 1] = u.y;
        }
    }
}

// A word as four fp16 pairs; zz: the zero point in both halves; tab: the table, bank: the lane's
// copy of it (4 lane).  Every fourth word decoded by byte permutes instead, to spare the shared
// memory, took a tenth longer.
template <int F>
__device__ __forceinline__ void decode(uint32_t w, uint32_t zz, const uint8_t* tab, uint32_t bank, uint32_t (&o)[4]) {
    if (F == kTable) {
        // byte j of the word above the bank (under 128): the entry's offset by one permute
        o[0] = *reinterpret_cast<const uint32_t*>(tab + prmt(w, bank, 0x5504));
        o[1] = *reinterpret_cast<const uint32_t*>(tab + prmt(w, bank, 0x5514));
        o[2] = *reinterpret_cast<const uint32_t*>(tab + prmt(w, bank, 0x5524));
        o[3] = *reinterpret_cast<const uint32_t*>(tab + prmt(w, bank, 0x5534));
    } else {
        int4_f16(w, zlo_f16(zz), zhi_f16(zz), o);
    }
}

// acc += (16 rows x 128 k of W) x (128 k x 8 NT columns of X); x(j, nt, v) gives the lane's
// eight values of word j, column g of n-tile nt.  `step`: counted from the row's first.  Where k ends
// in the middle of a step, the second half's codes are any, their scales 0 and their X 0.
template <int F, bool Z, int NT, typename XF>
__device__ __forceinline__ void multiply(const Sides<F, Z>& side, const uint8_t* entry, const Places& at, float (&acc)[NT][4],
                                         const uint8_t* tab, uint32_t bank, int step, XF&& x) {
    uint32_t c[2][4];
    ring_words<F>(entry, at, c[0]);
    ring_words<F>(entry + 512, at, c[1]);
    constexpr int kR = window_steps<F>(), kU = 4 / kR;
    const int unit = static_cast<int>(static_cast<unsigned>(step) % kR * kU);  // of the step's first group
    // words j and j + 2 side by side: their sums do not wait for each other's products
    float p[2][NT][4], f[2][2];
    uint32_t zz[2][2] = {{0x00080008u, 0x00080008u}, {0x00080008u, 0x00080008u}};
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        constexpr bool kEach = F == kG32;  // a group ends with every word
        uint32_t a[2][4], b[2][4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (kEach || j == 0) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int from = unit + (j + 2 * h) * kU / 4;
                    if (F == kG128 && h == 1) {
                        f[h][i] = f[0][i];
                        zz[h][i] = zz[0][i];
                    } else {
                        f[h][i] = __shfl_sync(kFull, side.f[i], from, 4);
                        if (Z) zz[h][i] = __shfl_sync(kFull, side.zz[i], from, 4);
                    }
                }
            }
            decode<F>(c[0][j + 2 * h], zz[h][0], tab, bank, a[h]);
            decode<F>(c[1][j + 2 * h], zz[h][1], tab, bank, b[h]);
        }
        uint32_t v[2][NT][4];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) x(j + 2 * h, nt, v[h][nt]);
#pragma unroll
        for (int i = 0; i < 2; ++i)  // the two products of a word
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    if (i == 0 && (kEach || j == 0)) mma_f16_first(p[h][nt], a[h][0], b[h][0], a[h][1], b[h][1], v[h][nt][0], v[h][nt][1]);
                    else mma_f16(p[h][nt], a[h][2 * i], b[h][2 * i], a[h][2 * i + 1], b[h][2 * i + 1], v[h][nt][2 * i], v[h][nt][2 * i + 1]);
                }
        if (kEach || j == 1) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    acc[nt][0] = __fmaf_rn(f[h][0], p[h][nt][0], acc[nt][0]);
                    acc[nt][1] = __fmaf_rn(f[h][0], p[h][nt][1], acc[nt][1]);
                    acc[nt][2] = __fmaf_rn(f[h][1], p[h][nt][2], acc[nt][2]);
                    acc[nt][3] = __fmaf_rn(f[h][1], p[h][nt][3], acc[nt][3]);
                }
        }
    }
}

// ------------------------------ X on chip ------------------------------
// A token's X in shared memory: 16-byte chunks of eight values.  Lane t's chunk j of a step:
//   kG128  chunk 4 t + j, with bit 1 of j flipped for t >= 2 (lanes 0 and 2 would meet in a bank)
//   kG64, kTable  chunk 8 (j / 2) + 2 t + j % 2;   kG32  chunk 4 j + t
// and tokens 16 (kG32: 64) bytes past a multiple of 128 apart, so the eight lanes of two
// tokens that a 16-byte read serves together hit all banks once.
template <int F>
__host__ __device__ constexpr int x_pad() { return F == kG32 ? 64 : 16; }
template <int F>
__device__ __forceinline__ uint32_t x_place(uint32_t chunk) {  // byte of a chunk, counted from the range's first step
    return 16u * (F == kG128 ? chunk ^ ((chunk >> 2) & 2u) : chunk);
}
template <int F>
__device__ __forceinline__ uint32_t x_lane(int t) {  // byte of a lane's chunk 0 inside a step
    return F == kG128 ? 64u * t : (F == kG32 ? 16u * t : 32u * t);
}
template <int F>
__device__ __forceinline__ uint32_t x_chunk(int j, int t) {  // chunk j itself, counted from the step's first
    return F == kG128 ? 4u * t + j : (F == kG32 ? 4u * j + t : 8u * (j >> 1) + 2u * t + (j & 1));
}
// A lane's chunk j of a step lies at x_lane + x_word(j), with x_flip taken off for j >= 2 and added for j < 2.
template <int F>
__device__ __forceinline__ uint32_t x_word(int j) {
    return F == kG128 ? 16u * j : (F == kG32 ? 64u * j : 128u * (j >> 1) + 16u * (j & 1));
}
template <int F>
__device__ __forceinline__ uint32_t x_flip(int t) {
    return F == kG128 ? 16u * (t & 2) : 0u;
}

// X [m] rows of `per` chunks, `row` chunks apart, into shared memory as fp16, each token times the power
// of two that its largest value here asks for (top[token]: that value's bf16 magnitude), in the order of
// int4_f16's pairs.  All threads; m is at most the number of warps, which are dealt out evenly to
// the tokens (1 << lg of them each).  Up to `padded` chunks it is zeros.  Ends with a block barrier.
template <int F>
__device__ __forceinline__ void stage_x(const uint4* x, int row, int per, int padded, int m, int lg, uint8_t* out, int stride, uint32_t* top, int warp,
                                        int lane, int warps) {
    constexpr int kBatch = 8;  // loads in flight
    if (threadIdx.x < warps) top[threadIdx.x] = 0;
    __syncthreads();
    const int tok = warp >> lg, hop = 32 << lg;  // the last warps may have no token
    const int first = (warp & ((1 << lg) - 1)) * 32 + lane;
    const uint4* src = x + static_cast<int64_t>(tok) * row;
    const int end = tok < m ? per : 0;
    uint4 v[kBatch];
    auto load = [&](int c) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            if (c - lane + i * hop >= end) break;
            v[i] = c + i * hop < end ? ld_global16(src + c + i * hop) : make_uint4(0u, 0u, 0u, 0u);
        }
    };
    uint32_t big = 0;  // of both halves
    for (int c = first; c - lane < end; c += kBatch * hop) {
        load(c);
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {  // bf16 magnitudes order as integers
            if (c - lane + i * hop >= end) break;
            big = __vmaxu2(__vmaxu2(big, __vmaxu2(v[i].x & 0x7fff7fffu, v[i].y & 0x7fff7fffu)),
                           __vmaxu2(v[i].z & 0x7fff7fffu, v[i].w & 0x7fff7fffu));
        }
    }
    big = __reduce_max_sync(kFull, max(big & 0xffffu, big >> 16));
    if (lane == 0 && big) atomicMax(&top[tok], big);
    __syncthreads();
    if (tok < m) {
        const float up = scale_up(scale_exponent(static_cast<int>(top[tok] >> 7)));
        const bool again = end > kBatch * hop;  // more than one batch: from L1 this time
        for (int c = per + first; c < padded; c += hop) *reinterpret_cast<uint4*>(out + tok * stride + x_place<F>(c)) = make_uint4(0u, 0u, 0u, 0u);
        for (int c = first; c - lane < end; c += kBatch * hop) {
            if (again) load(c);
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int at = c + i * hop;
                if (at - lane >= end) break;
                uint32_t o[4];
                pair_x(scale_pair(v[i].x, up), scale_pair(v[i].y, up), scale_pair(v[i].z, up), scale_pair(v[i].w, up), o);
                if (at < end) *reinterpret_cast<uint4*>(out + tok * stride + x_place<F>(at)) = make_uint4(o[0], o[1], o[2], o[3]);
            }
        }
    }
    __syncthreads();
}

// `total` things dealt out to `parts` in order, as evenly as they go: part i begins at start(i).
struct Shares {
    int each, more;
    __device__ __forceinline__ int start(int i) const { return i * each + min(i, more); }
};
__host__ __device__ inline Shares shares_of(int total, int parts) {
    const int each = static_cast<int>(static_cast<unsigned>(total) / static_cast<unsigned>(parts));
    return Shares{each, total - each * parts};
}
// Over the warps of a CTA, W or half as many: no division by a variable.
template <int W>
__device__ __forceinline__ Shares shares_of_warps(int total) {
    return blockDim.x == W * 16 ? shares_of(total, W / 2) : shares_of(total, W);
}

// ------------------------------ runs of steps ------------------------------
// The steps of a CTA's tiles, one tile's after the other's, are cut into equal runs for
// its warps.  A tile inside one run is finished from registers; of one that several runs
// share, the warp that begins it adds the others' sums, in warp order, from `slots`.
//   rows(tile, row)      the lane's two rows of a tile
//   begin(tile)          as a tile is entered
//   ahead(step)          before the step's codes are waited for
//   mul(entry, step)     multiplies a step of the tile, counted from the row's first
//   finish(tile)         its sums are complete in acc
// One step at a time: four in a row, with constant windows and offsets, took 1.6 % less over 28672 x 8192
// but 3 to 11 % more over 4096 x 4096 and 1024 x 4096, whose time is in fetching the code, and
// with the experts' registers more throughout.
template <int F, bool Z, int kDepth, int NT>
struct Runner {
    static constexpr int kR = window_steps<F>();
    Sides<F, Z> side;
    Places places;
    float acc[NT][4];
    uint8_t* ring;        // this warp's ring
    uint32_t put;         // the lane's place in it, as an address
    int warp, lane, t;
    int s0, ns;           // steps of a tile: s0 .. s0 + ns of the rows' steps
    int i0, i1;           // the run
    int sent, tile, step;  // steps of the run on their way; the next one
    const uint8_t* c[2];  // the lane's first chunk of the rows of that tile
    int wtile, window;    // the next window

    __device__ __forceinline__ void aim_codes(const Weight& w, const int64_t (&row)[2]) {
#pragma unroll
        for (int i = 0; i < 2; ++i) c[i] = w.wq + row[i] * (w.k >> 1) + 16 * t;
    }
    __device__ __forceinline__ void copy(const Weight& w, uint32_t entry, uint32_t to) const {
        const bool in = F == kG128 || to + 16u * t < static_cast<uint32_t>(w.k >> 1);  // else past the end of k: zeros
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint8_t* p = c[i] + static_cast<uint64_t>(to);
            if (F == kG128) copy16(put + entry + 512 * i, p);
            else copy16(put + entry + 512 * i, p, in ? 16 : 0);
        }
    }
    template <typename Rows>
    __device__ __forceinline__ void send(const Weight& w, uint32_t entry, Rows&& rows) {
        if (sent < i1) {
            copy(w, entry, static_cast<uint32_t>(step) * (kStepK / 2u));
            ++sent;
            if (++step == s0 + ns) {
                step = s0;
                ++tile;
                if (sent < i1) {
                    int64_t row[2];
                    rows(tile, row);
                    aim_codes(w, row);
                }
            }
        }
        copies_commit();
    }
    template <typename Rows>
    __device__ __forceinline__ void next_window(const Weight& w, Rows&& rows) {
        if (wtile * ns >= i1) return;
        side.load(w, window, t);
        if (++window * kR >= s0 + ns) {
            window = s0 / kR;
            ++wtile;
            if (wtile * ns >= i1) return;
            int64_t row[2];
            rows(wtile, row);
            side.aim(w, row);
        }
    }
    // Finds the run; reads nothing of the weight.
    template <typename Rows>
    __device__ __forceinline__ void find(const Weight& w, uint8_t* rings, int warp_, int lane_, const Shares& runs, int s0_, int ns_,
                                          Rows&& rows) {
        warp = warp_;
        lane = lane_;
        t = lane & 3;
        s0 = s0_;
        ns = ns_;
        places = few::places<F>(lane >> 2, t);
        ring = rings + warp * kDepth * kStepBytes;
        put = static_cast<uint32_t>(__cvta_generic_to_shared(ring)) + places.put;
        i0 = sent = runs.start(warp);
        i1 = runs.start(warp + 1);
        tile = wtile = ns ? static_cast<int>(static_cast<unsigned>(i0) / static_cast<unsigned>(ns)) : 0;
        step = s0 + i0 - tile * ns;
        window = step / kR;
        if (i0 < i1) {
            int64_t row[2];
            rows(tile, row);
            aim_codes(w, row);
            side.aim(w, row);
        }
    }
    // Starts its first loads.
    template <typename Rows>
    __device__ __forceinline__ void start(const Weight& w, Rows&& rows) {
#pragma unroll
        for (int d = 0; d < kDepth; ++d) send(w, d * kStepBytes, rows);
        if (i0 < i1) next_window(w, rows);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) acc[nt][0] = acc[nt][1] = acc[nt][2] = acc[nt][3] = 0.0f;
    }
    __device__ __forceinline__ void store(float4* slots) const {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) slots[(warp * NT + nt) * 32 + lane] = make_float4(acc[nt][0], acc[nt][1], acc[nt][2], acc[nt][3]);
    }
    // All threads of the block; ns > 0.
    template <typename Rows, typename Begin, typename Ahead, typename Mul, typename Finish>
    __device__ __forceinline__ void run(const Weight& w, float mu, float4* slots, const Shares& runs, Rows&& rows, Begin&& begin,
                                        Ahead&& ahead, Mul&& mul, Finish&& finish) {
        int tl = static_cast<int>(static_cast<unsigned>(i0) / static_cast<unsigned>(ns)), st = i0 - tl * ns;
        uint32_t entry = 0;
        bool mine = st == 0;  // this warp begins the tile
        for (int i = i0; i < i1;) {
            begin(tl);
            const int n = min(ns - st, i1 - i);
            i += n;
            st += s0;
            auto turn = [&] {
                side.turn(w, mu);
                next_window(w, rows);
            };
            turn();
            for (const int end = st + n;;) {
                ahead(st);
                copies_wait<kDepth - 1>();
                if (F != kG128) __syncwarp();  // else a lane reads what it copied itself
                mul(ring + entry, st);
                if (F != kG128) __syncwarp();
                send(w, entry, rows);
                entry = entry == (kDepth - 1) * kStepBytes ? 0u : entry + kStepBytes;
                ++st;
                if (st == end) break;
                if (st % kR == 0) turn();
            }
            st -= s0;
            if (st < ns) break;
            if (mine) finish(tl);
            else store(slots);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) acc[nt][0] = acc[nt][1] = acc[nt][2] = acc[nt][3] = 0.0f;
            mine = true;
            st = 0;
            ++tl;
        }
        if (!mine && i0 < i1) store(slots);  // neither begun nor ended here
        __syncthreads();
        if (mine && st > 0) {  // begun here, ended by a later warp
            const int end = (tl + 1) * ns;
            for (int v = warp + 1, from = i1; from < end; ++v) {
                const int to = runs.start(v + 1);
                if (to == from) continue;
                from = to;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const float4 u = slots[(v * NT + nt) * 32 + lane];
                    acc[nt][0] += u.x;
                    acc[nt][1] += u.y;
                    acc[nt][2] += u.z;
                    acc[nt][3] += u.w;
                }
            }
            finish(tl);
        }
    }
};

}  // namespace few
}  // namespace nf4
