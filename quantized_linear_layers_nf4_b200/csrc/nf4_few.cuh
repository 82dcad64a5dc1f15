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
// Scales go to registers: lane (g, t) loads that of group t (kG64, kTable: t % 2) of the step
// for its rows, and a shuffle hands it to the other lanes of the row.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include "nf4_common.cuh"
#include "nf4_decode.cuh"

namespace nf4 {
namespace few {

constexpr int kItemK = 64;   // the unit that k is a multiple of
constexpr int kStepK = 128;  // k of a step; its second half may lie past the end of k
constexpr int kStepBytes = 16 * kStepK / 2;

constexpr int kWarps = 24;  // of a CTA, one CTA an SM: 80 registers a thread
constexpr int kThreads = kWarps * 32;

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
    int per;         // kG128, kG64: steps, items (of 64 k) of a group
    int f32;         // scales are fp32 (bf16 otherwise)
    // codebook codes
    const int8_t* absmax_q;
    const float* absmax_scale;
    const float* mu;
    int codebook;
    int pairs;       // items 2 i and 2 i + 1 of a row: one aligned pair of absmax codes, one scale
};
__device__ __forceinline__ uint32_t ldg_scale(const void* scale, int f32, int64_t at) {  // as fp32 bits
    return f32 ? __ldg(reinterpret_cast<const uint32_t*>(scale) + at)
               : static_cast<uint32_t>(__ldg(reinterpret_cast<const uint16_t*>(scale) + at)) << 16;
}

// What goes with a step's codes, as it was loaded: anything done to it before its turn would
// wait for the load.  For rows g, g + 8.
struct Side {
    uint32_t s[2];  // scale; absmax scale
    uint32_t z[2];  // zero point; absmax code
};

// Where a lane's two rows are.
template <int F, bool Z>
struct Cursor {
    const uint8_t* c[2];  // the lane's 16 bytes of the next step
    const uint8_t* s[2];  // its scale; its absmax code
    const uint8_t* z[2];  // its zero point
    int64_t e[2];         // kTable: index of its absmax code
    int left;             // kG128, kG64: steps, items until its next group
};

template <int F, bool Z>
__device__ __forceinline__ void aim(Cursor<F, Z>& o, const Weight& w, int64_t row0, int64_t row1, int step, int t) {
    int grp = 4 * step + t;
    if (F == kG128 || F == kG64) {
        const int unit = F == kG128 ? step : 2 * step + (t & 1);
        grp = static_cast<int>(static_cast<unsigned>(unit) / static_cast<unsigned>(w.per));
        o.left = w.per - (unit - grp * w.per);
    }
    const int items = w.k / kItemK;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int64_t row = i ? row1 : row0;
        o.c[i] = w.wq + row * (w.k >> 1) + step * (kStepK / 2) + 16 * t;
        if (F == kTable) {
            o.e[i] = row * items + 2 * step + (t & 1);
            o.s[i] = reinterpret_cast<const uint8_t*>(w.absmax_q) + o.e[i];
        } else {
            const int64_t at = grp * w.n + row;
            o.s[i] = reinterpret_cast<const uint8_t*>(w.scale) + (w.f32 ? 4 * at : 2 * at);
            if (Z) o.z[i] = w.zero + at;
        }
    }
}

// The 16-byte chunk c of row r (0 .. 7) of a step in its ring entry: chunks are permuted so that
// reads of 4, 8 and 16 bytes a lane all find 128 different bytes.
__device__ __forceinline__ uint32_t ring_place(int r, int c) {
    return 64u * r + 16u * (c ^ (((r >> 1) & 1) << 1 | ((r >> 2) & 1)));
}

// Starts the copies of the cursor's step into a ring entry (`dst`: the lane's place in it),
// loads what goes with it, and moves to the next step.  `two`: the step's second half is not
// past the end of k.
template <int F, bool Z>
__device__ __forceinline__ void load_step(Side& o, uint32_t dst, Cursor<F, Z>& at, const Weight& w, bool two, int t) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        if (F == kG128) copy16(dst + 512 * i, at.c[i]);
        else copy16(dst + 512 * i, at.c[i], two || t < 2 ? 16 : 0);
        at.c[i] += kStepK / 2;
    }
    if (F == kTable) {
        const bool in = two || (t & 1) == 0;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (in) {
                o.z[i] = static_cast<uint32_t>(static_cast<int32_t>(__ldg(reinterpret_cast<const int8_t*>(at.s[i]))));
                o.s[i] = __float_as_uint(__ldg(w.absmax_scale + (at.e[i] >> 8)));
            }
            at.s[i] += 2;
            at.e[i] += 2;
        }
        return;
    }
    const bool in = F == kG128 || two || (F == kG32 ? t < 2 : (t & 1) == 0);
    const int64_t row_s = w.n << (w.f32 ? 2 : 1);
#pragma unroll
    for (int i = 0; i < 2; ++i)
        if (in) {
            o.s[i] = w.f32 ? __ldg(reinterpret_cast<const uint32_t*>(at.s[i])) : __ldg(reinterpret_cast<const uint16_t*>(at.s[i]));
            if (Z) o.z[i] = __ldg(at.z[i]);
        }
    if (F == kG32) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            at.s[i] += 4 * row_s;
            if (Z) at.z[i] += 4 * w.n;
        }
    } else {
        at.left -= F == kG128 ? 1 : 2;
#pragma unroll
        for (int h = 0; h < (F == kG128 ? 1 : 2); ++h)
            if (at.left <= 0) {
                at.left += w.per;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    at.s[i] += row_s;
                    if (Z) at.z[i] += w.n;
                }
            }
    }
}

// The two levels of each byte value as fp16, one copy a bank, 256 bytes an entry (the
// second half of it stays unused), so that a byte in bits 8 .. 15 is an address as it is.
constexpr int kTableBytes = 256 * 256;
__device__ __forceinline__ void build_table(uint8_t* tab, int codebook) {
    for (int i = threadIdx.x; i < 256 * 32; i += blockDim.x) {
        const int v = i >> 5;
        const __half2 e = __floats2half2_rn(kCodebook[codebook][v >> 4], kCodebook[codebook][v & 15]);
        *reinterpret_cast<__half2*>(tab + 256 * v + 4 * (i & 31)) = e;
    }
}
__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
}
__device__ __forceinline__ void lds128(uint32_t addr, uint32_t (&v)[4]) {
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(addr));
}

// The four words of a lane's row g (entry + 512: row g + 8) from a ring entry.
template <int F>
__device__ __forceinline__ void ring_words(uint32_t entry, int g, int t, uint32_t (&v)[4]) {
    if (F == kG128) {
        lds128(entry + ring_place(g, t), v);
    } else if (F == kG32) {
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = lds32(entry + ring_place(g, j) + 4 * t);
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h)
            asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];"
                         : "=r"(v[2 * h]), "=r"(v[2 * h + 1])
                         : "r"(entry + ring_place(g, 2 * h + (t >> 1)) + 8 * (t & 1)));
    }
}

// A word as four fp16 pairs; zz: the zero point in both halves; tab: the lane's copy of the table.
template <int F>
__device__ __forceinline__ void decode(uint32_t w, uint32_t zz, uint32_t tab, uint32_t (&o)[4]) {
    if (F == kTable) {
        const uint32_t v = w >> 16;
        o[0] = lds32((w & 0xffu) * 256u + tab);
        o[1] = lds32((w & 0xff00u) + tab);
        o[2] = lds32((v & 0xffu) * 256u + tab);
        o[3] = lds32((v & 0xff00u) + tab);
    } else {
        int4_f16(w, zlo_f16(zz), zhi_f16(zz), o);
    }
}

// acc += (16 rows x 128 k of W) x (128 k x 8 NT columns of X); x(j, nt, v) gives the lane's
// eight values of word j, column g of n-tile nt; n-tiles without a bit in `live` are left out.
template <int F, bool Z, int NT, typename XF>
__device__ __forceinline__ void multiply(const Side& side, uint32_t entry, const Weight& w, float (&acc)[NT][4], int live, float mu,
                                         uint32_t tab, bool two, int g, int t, XF&& x) {
    uint32_t c[2][4];
    ring_words<F>(entry, g, t, c[0]);
    ring_words<F>(entry + 512, g, t, c[1]);
    float f[2];
    uint32_t zz[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        if (F == kTable) f[i] = absmax_hat(static_cast<int>(side.z[i]), __uint_as_float(side.s[i]), mu);
        else f[i] = __uint_as_float(side.s[i] << (w.f32 ? 0 : 16));
        zz[i] = Z ? prmt(side.z[i], 0u, 0x4040) & 0x000f000fu : 0x00080008u;
    }
    float p[NT][4];
    float fj[2] = {f[0], f[1]};
    uint32_t zj[2] = {zz[0], zz[1]};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (F != kG128 && j == 2 && !two) return;
        const bool first = F == kG128 ? j == 0 : (F == kG32 || (j & 1) == 0);
        const bool last = F == kG128 ? j == 3 : (F == kG32 || (j & 1) == 1);
        if (F != kG128 && first) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                fj[i] = __shfl_sync(kFull, f[i], F == kG32 ? j : j >> 1, 4);
                if (Z) zj[i] = __shfl_sync(kFull, zz[i], F == kG32 ? j : j >> 1, 4);
            }
        }
        uint32_t a[4], b[4];
        decode<F>(c[0][j], zj[0], tab, a);
        decode<F>(c[1][j], zj[1], tab, b);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            if (NT > 1 && !(live >> nt & 1)) continue;
            uint32_t v[4];
            x(j, nt, v);
            if (first) mma_f16_first(p[nt], a[0], b[0], a[1], b[1], v[0], v[1]);
            else mma_f16(p[nt], a[0], b[0], a[1], b[1], v[0], v[1]);
            mma_f16(p[nt], a[2], b[2], a[3], b[3], v[2], v[3]);
        }
        if (last) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                if (NT > 1 && !(live >> nt & 1)) continue;
                acc[nt][0] = __fmaf_rn(fj[0], p[nt][0], acc[nt][0]);
                acc[nt][1] = __fmaf_rn(fj[0], p[nt][1], acc[nt][1]);
                acc[nt][2] = __fmaf_rn(fj[1], p[nt][2], acc[nt][2]);
                acc[nt][3] = __fmaf_rn(fj[1], p[nt][3], acc[nt][3]);
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
template <int F>
__device__ __forceinline__ uint32_t x_word(int j, int t) {  // and of its chunk j from there
    return F == kG128 ? 16u * (j ^ (t & 2)) : (F == kG32 ? 64u * j : 128u * (j >> 1) + 16u * (j & 1));
}
// X [m] rows of `per` chunks, `row` chunks apart, into shared memory as fp16, each token times the power
// of two that its largest value here asks for (top[token]: that value's bf16 magnitude), in the order of
// int4_f16's pairs.  All threads; m is at most the number of warps, which are dealt out evenly to
// the tokens (1 << lg of them each).  Ends with a block barrier.
template <int F>
__device__ __forceinline__ void stage_x(const uint4* x, int row, int per, int m, int lg, uint8_t* out, int stride, uint32_t* top, int warp,
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
__host__ __device__ inline Shares shares_of(int total, int parts) { return Shares{total / parts, total % parts}; }

// ------------------------------ runs of steps ------------------------------
// The steps of a CTA's tiles, one tile's after the other's, are cut into equal runs for
// its warps.  A tile inside one run is finished from registers; of one that several runs
// share, the warp that begins it adds the others' sums, in warp order, from `slots`.
//   next(d)        starts the loads of the run's next step into ring entry d
//   begin(tile)    as a tile is entered
//   mul(d, step)   multiplies a step of the tile, which is in entry d
//   finish(tile)   its sums are complete in acc
// All threads of the block; the first kDepth steps are already on their way.
template <int kDepth, int NT, typename Next, typename Begin, typename Mul, typename Finish>
__device__ __forceinline__ void run(float (&acc)[NT][4], float4* slots, int warp, int lane, const Shares& runs, int ns, Next&& next,
                                    Begin&& begin, Mul&& mul, Finish&& finish) {
    const int i0 = runs.start(warp), i1 = runs.start(warp + 1);
    int tile = static_cast<int>(static_cast<unsigned>(i0) / static_cast<unsigned>(ns)), step = i0 - tile * ns;
    bool mine = step == 0;  // this warp begins the tile
    auto put = [&] {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) slots[(warp * NT + nt) * 32 + lane] = make_float4(acc[nt][0], acc[nt][1], acc[nt][2], acc[nt][3]);
    };
    if (i0 < i1) begin(tile);
    for (int i = i0; i < i1; i += kDepth) {
#pragma unroll
        for (int d = 0; d < kDepth; ++d) {
            if (d > 0 && i + d >= i1) break;
            copies_wait<kDepth - 1>();
            __syncwarp();
            mul(d, step);
            __syncwarp();
            next(d);
            copies_commit();
            if (++step == ns) {
                if (mine) finish(tile);
                else put();
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) acc[nt][0] = acc[nt][1] = acc[nt][2] = acc[nt][3] = 0.0f;
                mine = true;
                step = 0;
                ++tile;
                if (i + d + 1 < i1) begin(tile);
            }
        }
    }
    if (!mine && i0 < i1) put();  // neither begun nor ended here
    __syncthreads();
    if (mine && step > 0) {  // begun here, ended by a later warp
        const int end = (tile + 1) * ns;
        for (int w = warp + 1, from = i1; from < end; ++w) {
            const int to = runs.start(w + 1);
            if (to == from) continue;
            from = to;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const float4 v = slots[(w * NT + nt) * 32 + lane];
                acc[nt][0] += v.x;
                acc[nt][1] += v.y;
                acc[nt][2] += v.z;
                acc[nt][3] += v.w;
            }
        }
        finish(tile);
    }
}

}  // namespace few
}  // namespace nf4
