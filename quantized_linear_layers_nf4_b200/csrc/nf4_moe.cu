// nf4_moe.cu -- a whole mixture-of-experts layer for a few tokens (m <= 16 a pass),
// experts in 4 bits (sm_100a).
//
//   l[t, e] = sum_c X[t, c] R[e, c];  the top_k largest of each row, ties to the lower e
//   p[t, e] = exp(l[t, e] - max) / sum over all (or the chosen) experts
//   a[t, e] = p[t, e] silu(G_e x_t) * (U_e x_t);   Y[t] = sum_e D_e a[t, e]
//
// Bound by HBM: each chosen expert's three matrices are read once, whoever shares it.
// Three launches, each a programmatic dependent of the one before:
//   k_moe_router   one dot product per (expert, token), and X as fp16 times a power of two
//   k_moe_gate_up  every CTA chooses the experts itself from the logits (cheaper than
//                  another launch), then takes its share of the (expert, 8 rows of f)
//                  tiles: 8 gate rows and the 8 up rows that belong to them form the 16
//                  rows of one mma.sync tile, so a lane holds a gate sum and its up sum
//   k_moe_down     16 rows of the output a CTA; the tokens are the columns, so the sum over
//                  experts is the sum over k of all chosen experts one after the other
// The weights' decoding and the tile geometry are in nf4_few.cuh.  No CTA waits for
// another, and every sum is taken in a fixed order.
//
// Roundings.  X (bf16) times a power of two per token is exact in fp16.  Codebook levels
// are rounded to fp16 (within 2^-11 of the value; bf16 would be 2^-8, as much as the rounding
// of the result); integer codes are exact.  The activations a are kept in fp32 and, for the
// products, rounded to fp16 (2^-11); where a token's largest one is outside [2^-6, 2^15)
// they are read from the fp32 copy and scaled by a power of two on the way.
#include <mutex>
#include <type_traits>

#include "nf4_few.cuh"
#include "nf4_internal.h"
#include "nf4_ptx.cuh"

namespace nf4 {
namespace moe {

constexpr int kMaxM = 16;        // tokens of a pass
constexpr int kMaxTop = 16;
constexpr int kMaxE = 512;
constexpr int kMaxPairs = kMaxM * kMaxTop;
constexpr int kWarps = 8;
constexpr int kTableBytes = 256 * 32 * 4;

enum Fmt { kTable = 0, kInt4 = 1, kInt4G32 = 2 };

struct Weight {
    const uint8_t* wq;
    int64_t k;
    const int8_t* absmax_q;  // kTable
    const float* absmax_scale;
    const float* mu;
    int codebook;
    few::Int4Sides sides;  // kInt4, kInt4G32
};

struct Params {
    const __nv_bfloat16* x;
    const __nv_bfloat16* router;
    int m, E, top;
    int h, f;
    int renormalize;
    Weight gate_up, down;
    float* logits;      // [m][E]
    __half* xs;         // [m][h]
    float* xscale;      // [m]
    int* amax;          // [m] bits of the largest |a| of a token
    float* act32;       // [m * top][f], the pairs of an expert together
    __half* act16;
    __nv_bfloat16* y;
    int32_t* ids;       // [m][top] or null
    float* probs;       // [m][top] or null
    int x_paired, act_paired;  // elements in the order of int4_f16's pairs
};

// Position of element j of eight in the order (1,5), (0,4), (3,7), (2,6).
__device__ __forceinline__ int paired(int j) { return (0x57134602u >> (4 * j)) & 7; }

// ------------------------------- router -------------------------------
constexpr int kRouterThreads = 128;
constexpr int kRouterTokens = 4;

__device__ __forceinline__ void dot8(const uint4 a, const uint4 b, float& s) {
    const uint32_t u[4] = {a.x, a.y, a.z, a.w}, v[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        s = __fmaf_rn(bf16_bits_to_float(u[j] & 0xffffu), bf16_bits_to_float(v[j] & 0xffffu), s);
        s = __fmaf_rn(__uint_as_float(u[j] & 0xffff0000u), __uint_as_float(v[j] & 0xffff0000u), s);
    }
}

__global__ void __launch_bounds__(kRouterThreads) k_moe_router(const __grid_constant__ Params p) {
    __shared__ float part[kRouterThreads / 32][kRouterTokens];
    grid_dependency_wait();
    grid_launch_dependents();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int groups = (p.m + kRouterTokens - 1) / kRouterTokens;
    const int chunks = p.h / 8;
    if (static_cast<int>(blockIdx.x) < p.E * groups) {
        const int e = blockIdx.x / groups, t0 = (blockIdx.x % groups) * kRouterTokens;
        const uint4* r = reinterpret_cast<const uint4*>(p.router + static_cast<int64_t>(e) * p.h);
        float s[kRouterTokens] = {};
        for (int c = tid; c < chunks; c += kRouterThreads) {
            const uint4 rv = __ldg(r + c);
#pragma unroll
            for (int j = 0; j < kRouterTokens; ++j)
                if (t0 + j < p.m) dot8(__ldg(reinterpret_cast<const uint4*>(p.x + static_cast<int64_t>(t0 + j) * p.h) + c), rv, s[j]);
        }
#pragma unroll
        for (int j = 0; j < kRouterTokens; ++j) {
            for (int o = 16; o > 0; o >>= 1) s[j] += __shfl_xor_sync(kFull, s[j], o);
            if (lane == 0) part[warp][j] = s[j];
        }
        __syncthreads();
        if (tid < kRouterTokens && t0 + tid < p.m) {
            float v = 0.0f;
            for (int w = 0; w < kRouterThreads / 32; ++w) v += part[w][tid];
            p.logits[(t0 + tid) * p.E + e] = v;
        }
        return;
    }
    // one token's X as fp16: times 2^(14 - e), e the exponent of its largest value
    const int t = blockIdx.x - p.E * groups;
    const uint4* x = reinterpret_cast<const uint4*>(p.x + static_cast<int64_t>(t) * p.h);
    uint32_t top = 0;  // bf16 magnitudes order as integers
    for (int c = tid; c < chunks; c += kRouterThreads) {
        const uint4 v = __ldg(x + c);
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) top = max(top, max(u[j] & 0x7fffu, (u[j] >> 16) & 0x7fffu));
    }
    top = __reduce_max_sync(kFull, top);
    if (lane == 0) part[warp][0] = __uint_as_float(top);
    __syncthreads();
    for (int w = 0; w < kRouterThreads / 32; ++w) top = max(top, __float_as_uint(part[w][0]));
    // biased exponent 127 + e; zero, subnormal and non-finite maxima take the nearest
    // factor that is a normal number both ways
    const int ex = min(max(static_cast<int>(top >> 7), 15), 254);
    const float factor = __uint_as_float(static_cast<uint32_t>(127 + 14 + 127 - ex) << 23);
    if (tid == 0) {
        p.xscale[t] = __uint_as_float(static_cast<uint32_t>(ex - 14) << 23);
        p.amax[t] = 0;
    }
    __half* xs = p.xs + static_cast<int64_t>(t) * p.h;
    for (int c = tid; c < chunks; c += kRouterThreads) {
        const uint4 v = __ldg(x + c);
        uint32_t u[4] = {v.x, v.y, v.z, v.w}, o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const __half2 hh = __floats2half2_rn(bf16_bits_to_float(u[j] & 0xffffu) * factor, __uint_as_float(u[j] & 0xffff0000u) * factor);
            u[j] = *reinterpret_cast<const uint32_t*>(&hh);
        }
        if (p.x_paired) few::pair_x(u[0], u[1], u[2], u[3], o);
        else { o[0] = u[0]; o[1] = u[1]; o[2] = u[2]; o[3] = u[3]; }
        reinterpret_cast<uint4*>(xs)[c] = make_uint4(o[0], o[1], o[2], o[3]);
    }
}

// ------------------------------- routing -------------------------------
struct Route {
    float prob[kMaxM][kMaxTop];
    uint16_t id[kMaxM][kMaxTop];
    uint32_t mask[kMaxE];       // tokens of an expert
    uint16_t pos[kMaxE];        // of an expert in the list of chosen ones
    uint16_t list[kMaxPairs];   // chosen experts, ascending
    uint16_t base[kMaxPairs];   // first pair of a chosen expert
    float pair_prob[kMaxPairs];
    int active;
};

// A key that orders as the logit does; NaN below everything, 0 for "none".
__device__ __forceinline__ uint32_t order_key(float v) {
    if (v != v) return 1u;
    const uint32_t u = __float_as_uint(v + 0.0f);  // -0 as +0
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Every thread of the block; the logits are complete.  A warp per token finds the
// top_k one after the other (the largest key by a warp reduction, among equal ones the
// lowest index by another).
__device__ __forceinline__ void route(const Params& p, Route& R) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, warps = blockDim.x >> 5;
    for (int e = tid; e < p.E; e += blockDim.x) R.mask[e] = 0;
    __syncthreads();
    for (int t = warp; t < p.m; t += warps) {
        float v[kMaxE / 32];
        uint32_t key[kMaxE / 32];
        const float* l = p.logits + t * p.E;
#pragma unroll
        for (int i = 0; i < kMaxE / 32; ++i) {
            const int e = 32 * i + lane;
            key[i] = 0;
            v[i] = 0.0f;
            if (32 * i < p.E && e < p.E) {
                v[i] = __ldcg(l + e);
                key[i] = order_key(v[i]);
            }
        }
        float best = 0.0f, mine = 0.0f, chosen = 0.0f;
        for (int j = 0; j < p.top; ++j) {
            uint32_t k = 0;
#pragma unroll
            for (int i = 0; i < kMaxE / 32; ++i) k = max(k, key[i]);
            const uint32_t kmax = __reduce_max_sync(kFull, k);
            uint32_t at = 0xffffffffu;
#pragma unroll
            for (int i = kMaxE / 32 - 1; i >= 0; --i)
                if (key[i] == kmax) at = 32 * i + lane;
            at = __reduce_min_sync(kFull, at);
            float got = 0.0f;
#pragma unroll
            for (int i = 0; i < kMaxE / 32; ++i)
                if (32 * i + lane == static_cast<int>(at)) {
                    got = v[i];
                    key[i] = 0;
                }
            got = __shfl_sync(kFull, got, at & 31);
            if (j == 0) best = got;
            const float ex = expf(got - best);
            chosen += ex;
            if (lane == j) mine = ex;
            if (lane == 0) {
                R.id[t][j] = static_cast<uint16_t>(at);
                atomicOr(&R.mask[at], 1u << t);
            }
        }
        if (!p.renormalize) {
            chosen = 0.0f;
#pragma unroll
            for (int i = 0; i < kMaxE / 32; ++i)
                if (32 * i + lane < p.E) chosen += expf(v[i] - best);
            for (int o = 16; o > 0; o >>= 1) chosen += __shfl_xor_sync(kFull, chosen, o);
        }
        if (lane < p.top) R.prob[t][lane] = mine / chosen;
    }
    __syncthreads();
    if (warp == 0) {
        int n = 0, pairs = 0;
        for (int e0 = 0; e0 < p.E; e0 += 32) {
            const int e = e0 + lane;
            const int cnt = e < p.E ? __popc(R.mask[e]) : 0;
            const uint32_t any = __ballot_sync(kFull, cnt != 0);
            int sum = cnt;
            for (int o = 1; o < 32; o <<= 1) {
                const int up = __shfl_up_sync(kFull, sum, o);
                if (lane >= o) sum += up;
            }
            if (cnt) {
                const int at = n + __popc(any & ((1u << lane) - 1));
                R.list[at] = static_cast<uint16_t>(e);
                R.base[at] = static_cast<uint16_t>(pairs + sum - cnt);
                R.pos[e] = static_cast<uint16_t>(at);
            }
            n += __popc(any);
            pairs += __shfl_sync(kFull, sum, 31);
        }
        if (lane == 0) R.active = n;
    }
    __syncthreads();
    for (int i = tid; i < p.m * p.top; i += blockDim.x) {
        const int t = i / p.top, j = i % p.top, e = R.id[t][j];
        R.pair_prob[R.base[R.pos[e]] + __popc(R.mask[e] & ((1u << t) - 1))] = R.prob[t][j];
    }
    __syncthreads();
}

// ------------------------------ weight items ------------------------------
template <int FMT>
struct Raw {
    static constexpr int kSides = FMT == kInt4G32 ? 2 : 1;
    uint2 a, b;                                                  // codes of rows g and g + 8
    uint32_t sa[kSides], sb[kSides];                             // scales (absmax scales)
    uint32_t za[kSides], zb[kSides];                             // zero points (absmax codes)
};

template <int FMT>
__device__ __forceinline__ int code_offset(int t) { return FMT == kInt4G32 ? 4 * t : 8 * t; }

template <int FMT>
__device__ __forceinline__ void fetch(const Weight& w, Raw<FMT>& r, const uint8_t* pa, const uint8_t* pb, int64_t ra, int64_t rb,
                                      int blk) {
    const int64_t off = static_cast<int64_t>(blk) * 32;
    if (FMT == kInt4G32) {
        r.a = make_uint2(few::ldg_code32(pa + off), few::ldg_code32(pa + off + 16));
        r.b = make_uint2(few::ldg_code32(pb + off), few::ldg_code32(pb + off + 16));
    } else {
        r.a = few::ldg_codes(pa + off);
        r.b = few::ldg_codes(pb + off);
    }
    if (FMT == kTable) {
        const int64_t ia = ra * (w.k / 64) + blk, ib = rb * (w.k / 64) + blk;
        r.za[0] = static_cast<uint32_t>(static_cast<int32_t>(__ldg(w.absmax_q + ia)));
        r.zb[0] = static_cast<uint32_t>(static_cast<int32_t>(__ldg(w.absmax_q + ib)));
        r.sa[0] = __float_as_uint(__ldg(w.absmax_scale + (ia >> 8)));
        r.sb[0] = __float_as_uint(__ldg(w.absmax_scale + (ib >> 8)));
    } else {
        const int64_t gb = FMT == kInt4G32 ? 2 * static_cast<int64_t>(blk) : few::group_of(w.sides, static_cast<uint32_t>(blk));
#pragma unroll
        for (int i = 0; i < Raw<FMT>::kSides; ++i) {
            const int64_t at = (gb + i) * w.sides.n;
            r.sa[i] = few::ldg_scale(w.sides, at + ra);
            r.sb[i] = few::ldg_scale(w.sides, at + rb);
            r.za[i] = few::ldg_zero(w.sides, at + ra);
            r.zb[i] = few::ldg_zero(w.sides, at + rb);
        }
    }
}

// The two levels of each byte value as fp16, one copy a bank: tab[32 v + lane].
__device__ __forceinline__ void build_table(uint32_t* tab, int codebook) {
    for (int i = threadIdx.x; i < 256 * 32; i += blockDim.x) {
        const int v = i >> 5;
        const __half2 e = __floats2half2_rn(kCodebook[codebook][v >> 4], kCodebook[codebook][v & 15]);
        tab[i] = *reinterpret_cast<const uint32_t*>(&e);
    }
}

// acc += (16 rows x 64 k of W) x (64 k x 8 NT columns); n-tile i is skipped unless bit i of `live`.
template <int FMT, int NT>
__device__ __forceinline__ void multiply(const Raw<FMT>& r, const uint32_t (&x)[NT][8], float (&acc)[NT][4], int live, float mu,
                                         uint32_t tab) {
    float p[NT][4] = {};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t ca = h ? r.a.y : r.a.x, cb = h ? r.b.y : r.b.x;
        const int s = FMT == kInt4G32 ? h : 0;
        uint32_t wa[4], wb[4];
        if (FMT == kTable) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {  // byte j at 128 bytes an entry
                const uint32_t ia = (j == 0 ? ca << 7 : ca >> (8 * j - 7)) & 0x7f80u, ib = (j == 0 ? cb << 7 : cb >> (8 * j - 7)) & 0x7f80u;
                asm volatile("ld.shared.u32 %0, [%1];" : "=r"(wa[j]) : "r"(tab + ia));
                asm volatile("ld.shared.u32 %0, [%1];" : "=r"(wb[j]) : "r"(tab + ib));
            }
        } else {
            few::int4_f16(ca, few::zlo_f16(r.za[s]), few::zhi_f16(r.za[s]), wa);
            few::int4_f16(cb, few::zlo_f16(r.zb[s]), few::zhi_f16(r.zb[s]), wb);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            if (NT > 1 && !(live >> nt & 1)) continue;
            few::mma_f16(p[nt], wa[0], wb[0], wa[1], wb[1], x[nt][4 * h], x[nt][4 * h + 1]);
            few::mma_f16(p[nt], wa[2], wb[2], wa[3], wb[3], x[nt][4 * h + 2], x[nt][4 * h + 3]);
        }
        if (FMT == kInt4G32 || h == 1) {
            float fa = __uint_as_float(r.sa[s]), fb = __uint_as_float(r.sb[s]);
            if (FMT == kTable) {
                fa = absmax_hat(static_cast<int>(r.za[0]), fa, mu);
                fb = absmax_hat(static_cast<int>(r.zb[0]), fb, mu);
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                acc[nt][0] = __fmaf_rn(fa, p[nt][0], acc[nt][0]);
                acc[nt][1] = __fmaf_rn(fa, p[nt][1], acc[nt][1]);
                acc[nt][2] = __fmaf_rn(fb, p[nt][2], acc[nt][2]);
                acc[nt][3] = __fmaf_rn(fb, p[nt][3], acc[nt][3]);
                p[nt][0] = p[nt][1] = p[nt][2] = p[nt][3] = 0.0f;
            }
        }
    }
}

constexpr int kLd = 20;  // floats of a token's 16 rows in the reduction buffer

template <int NT>
__device__ __forceinline__ void put(float (*red)[kLd], const float (&acc)[NT][4], int g, int t) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        red[nt * 8 + 2 * t][g] = acc[nt][0];
        red[nt * 8 + 2 * t + 1][g] = acc[nt][1];
        red[nt * 8 + 2 * t][g + 8] = acc[nt][2];
        red[nt * 8 + 2 * t + 1][g + 8] = acc[nt][3];
    }
}

// The j-th set bit of a mask, or 0 where it has fewer.
__device__ __forceinline__ int nth_bit(uint32_t mask, int j) {
    for (int i = 0; i < j; ++i) mask &= mask - 1;
    return mask ? __ffs(mask) - 1 : 0;
}

// ------------------------------ gate and up ------------------------------
template <int FMT, int NT>
__global__ void __launch_bounds__(kWarps * 32, 2) k_moe_gate_up(const __grid_constant__ Params p) {
    constexpr int kDepth = 4;
    extern __shared__ uint32_t table[];
    __shared__ Route R;
    __shared__ float red[2][kWarps][8 * NT][kLd];

    if (FMT == kTable) build_table(table, p.gate_up.codebook);
    grid_dependency_wait();
    grid_launch_dependents();
    route(p, R);
    if (blockIdx.x == 0)
        for (int i = threadIdx.x; i < p.m * p.top; i += blockDim.x) {
            if (p.ids) p.ids[i] = R.id[i / p.top][i % p.top];
            if (p.probs) p.probs[i] = R.prob[i / p.top][i % p.top];
        }

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const Weight& w = p.gate_up;
    const float mu = FMT == kTable ? __ldg(w.mu) : 0.0f;
    const uint32_t tab = FMT == kTable ? smem_u32(table) + 4 * lane : 0u;
    const int per_e = p.f / 8;
    const int64_t tiles = static_cast<int64_t>(R.active) * per_e;
    const int t0 = static_cast<int>(tiles * blockIdx.x / gridDim.x), t1 = static_cast<int>(tiles * (blockIdx.x + 1) / gridDim.x);
    const int items = p.h / few::kItemK;
    const int b0 = items * warp / kWarps, b1 = items * (warp + 1) / kWarps;
    const int coff = code_offset<FMT>(t);

    // the cursor of the loads, kDepth items ahead of the products
    int ft = t0, fb = b0;
    int64_t fa = 0;
    const uint8_t* fp = nullptr;
    auto aim = [&] {
        const int e = R.list[ft / per_e], r0 = (ft % per_e) * 8;
        fa = static_cast<int64_t>(e) * 2 * p.f + r0 + g;
        fp = w.wq + fa * (w.k / 2) + coff;
    };
    auto fetch_next = [&](Raw<FMT>& r) {
        if (ft >= t1) return;
        fetch<FMT>(w, r, fp, fp + static_cast<int64_t>(p.f) * (w.k / 2), fa, fa + p.f, fb);
        if (++fb == b1) {
            fb = b0;
            if (++ft < t1) aim();
        }
    };

    // what the products of one tile need
    float acc[NT][4] = {};
    const __half* xp[NT];
    bool col[NT];
    int live = 0, e_at = -1, cnt = 0;
    uint32_t mask = 0;
    auto begin = [&](int tile) {
        const int at = tile / per_e;
        if (at == e_at) return;
        e_at = at;
        mask = R.mask[R.list[at]];
        cnt = __popc(mask);
        live = cnt > 8 ? 3 : 1;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int j = nt * 8 + g;
            col[nt] = j < cnt;
            xp[nt] = p.xs + static_cast<int64_t>(nth_bit(mask, j)) * p.h + 2 * coff;
        }
    };
    auto consume = [&](const Raw<FMT>& r, int b) {
        uint32_t x[NT][8];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            uint4 u = make_uint4(0, 0, 0, 0), v = u;
            if (col[nt]) {
                const __half* q = xp[nt] + static_cast<int64_t>(b) * few::kItemK;
                u = *reinterpret_cast<const uint4*>(q);
                v = *reinterpret_cast<const uint4*>(q + (FMT == kInt4G32 ? 32 : 8));
            }
            x[nt][0] = u.x; x[nt][1] = u.y; x[nt][2] = u.z; x[nt][3] = u.w;
            x[nt][4] = v.x; x[nt][5] = v.y; x[nt][6] = v.z; x[nt][7] = v.w;
        }
        multiply<FMT, NT>(r, x, acc, live, mu, tab);
    };
    auto finish = [&](int tile) {
        float(*buf)[8 * NT][kLd] = red[tile & 1];
        put<NT>(buf[warp], acc, g, t);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) acc[nt][0] = acc[nt][1] = acc[nt][2] = acc[nt][3] = 0.0f;
        __syncthreads();  // two buffers: the next tile's sums may be put while these are read
        const int r = threadIdx.x & 7, j = threadIdx.x >> 3;
        if (j < 8 * NT) {  // whole warps
            float ga = 0.0f, up = 0.0f, a = 0.0f;
            const int at = tile / per_e;
            const uint32_t mk = R.mask[R.list[at]];
            const int tok = nth_bit(mk, j);
            if (j < __popc(mk)) {
#pragma unroll
                for (int i = 0; i < kWarps; ++i) {
                    ga += buf[i][j][r];
                    up += buf[i][j][r + 8];
                }
                const float xs = p.xscale[tok];
                const int pair = R.base[at] + j;
                ga *= xs;
                a = ga / (1.0f + expf(-ga)) * (up * xs) * R.pair_prob[pair];
                const int64_t o = static_cast<int64_t>(pair) * p.f + (tile % per_e) * 8 + (p.act_paired ? paired(r) : r);
                p.act32[o] = a;
                p.act16[o] = __float2half_rn(a);
            }
            int top = __float_as_int(fabsf(a));
            for (int o = 4; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(kFull, top, o));
            if (r == 0 && j < __popc(mk)) atomicMax(p.amax + tok, top);
        }
    };

    Raw<FMT> ring[kDepth];
    const int nb = b1 - b0;
    const int total = nb * (t1 - t0);
    if (total > 0) {
        aim();
#pragma unroll
        for (int d = 0; d < kDepth; ++d) fetch_next(ring[d]);
        int tile = t0, b = b0;
        for (int c = 0; c < total; c += kDepth) {
#pragma unroll
            for (int d = 0; d < kDepth; ++d) {
                if (c + d >= total) break;
                if (b == b0) begin(tile);
                consume(ring[d], b);
                fetch_next(ring[d]);
                if (++b == b1) {
                    finish(tile);
                    b = b0;
                    ++tile;
                }
            }
        }
    } else {
        for (int tile = t0; tile < t1; ++tile) finish(tile);  // fewer items than warps
    }
}

// --------------------------------- down ---------------------------------
template <int FMT, int NT>
__global__ void __launch_bounds__(kWarps * 32, 2) k_moe_down(const __grid_constant__ Params p, int splits) {
    constexpr int kDepth = 4;
    extern __shared__ uint32_t table[];
    __shared__ Route R;
    __shared__ float red[kWarps][8 * NT][kLd];
    __shared__ float part[8 * NT][kLd];
    __shared__ float factor[kMaxM];
    __shared__ int wide;

    // The logits are those the previous kernel waited for before it let this one start.
    if (FMT == kTable) build_table(table, p.down.codebook);
    route(p, R);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const Weight& w = p.down;
    const float mu = FMT == kTable ? __ldg(w.mu) : 0.0f;
    const uint32_t tab = FMT == kTable ? smem_u32(table) + 4 * lane : 0u;
    const int rank = splits > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int row0 = static_cast<int>(blockIdx.x / splits) * 16;
    const int per_e = p.f / few::kItemK;
    const int items = R.active * per_e;
    const int c0 = static_cast<int>(static_cast<int64_t>(items) * rank / splits);
    const int c1 = static_cast<int>(static_cast<int64_t>(items) * (rank + 1) / splits);
    const int i0 = c0 + (c1 - c0) * warp / kWarps, i1 = c0 + (c1 - c0) * (warp + 1) / kWarps;
    const int coff = code_offset<FMT>(t);

    int fi = i0, fe = i0 / per_e, fb = i0 % per_e;
    int64_t fa = 0;
    const uint8_t* fp = nullptr;
    auto aim = [&] {
        fa = static_cast<int64_t>(R.list[fe]) * p.h + row0 + g;
        fp = w.wq + fa * (w.k / 2) + coff;
    };
    auto fetch_next = [&](Raw<FMT>& r) {
        if (fi >= i1) return;
        fetch<FMT>(w, r, fp, fp + 4 * w.k, fa, fa + 8, fb);
        ++fi;
        if (++fb == per_e) {
            fb = 0;
            ++fe;
            if (fi < i1) aim();
        }
    };
    Raw<FMT> ring[kDepth];
    if (i0 < i1) {
        aim();
#pragma unroll
        for (int d = 0; d < kDepth; ++d) fetch_next(ring[d]);
    }
    grid_dependency_wait();
    grid_launch_dependents();

    // fp16 activations, or fp32 ones scaled where a token's largest is out of range
    if (threadIdx.x == 0) wide = 0;
    __syncthreads();
    if (threadIdx.x < p.m) {
        const int bits = __ldcg(p.amax + threadIdx.x);
        const int ex = min(max(bits >> 23, 15), 254);
        const bool out = bits != 0 && (bits >= 0x47000000 || bits < 0x3c800000);  // >= 2^15, < 2^-6
        factor[threadIdx.x] = __int_as_float((127 + 14 + 127 - ex) << 23);
        if (out) wide = 1;
    }
    __syncthreads();
    const bool conv = wide != 0;

    float acc[NT][4] = {};
    int at = i0 / per_e, b = i0 % per_e;
    int live = 0;
    bool col[NT];
    int64_t off[NT];
    float fct[NT];
    auto begin = [&] {
        const uint32_t mask = R.mask[R.list[at]];
        live = 0;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int tok = nt * 8 + g;
            if (mask >> (8 * nt) & 0xffu) live |= 1 << nt;
            col[nt] = mask >> tok & 1;
            off[nt] = static_cast<int64_t>(R.base[at] + __popc(mask & ((1u << tok) - 1))) * p.f + 2 * coff;
            fct[nt] = factor[tok < p.m ? tok : 0];
        }
    };
    auto consume = [&](const Raw<FMT>& r) {
        uint32_t x[NT][8];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            uint4 u = make_uint4(0, 0, 0, 0), v = u;
            const int64_t o = off[nt] + b * few::kItemK;
            const int o2 = FMT == kInt4G32 ? 32 : 8;
            if (col[nt]) {
                if (!conv) {
                    u = __ldcg(reinterpret_cast<const uint4*>(p.act16 + o));
                    v = __ldcg(reinterpret_cast<const uint4*>(p.act16 + o + o2));
                } else {
                    uint32_t q[8];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float4 z = __ldcg(reinterpret_cast<const float4*>(p.act32 + o + (i >> 1) * o2) + (i & 1));
                        const __half2 lo = __floats2half2_rn(z.x * fct[nt], z.y * fct[nt]), hi = __floats2half2_rn(z.z * fct[nt], z.w * fct[nt]);
                        q[2 * i] = *reinterpret_cast<const uint32_t*>(&lo);
                        q[2 * i + 1] = *reinterpret_cast<const uint32_t*>(&hi);
                    }
                    u = make_uint4(q[0], q[1], q[2], q[3]);
                    v = make_uint4(q[4], q[5], q[6], q[7]);
                }
            }
            x[nt][0] = u.x; x[nt][1] = u.y; x[nt][2] = u.z; x[nt][3] = u.w;
            x[nt][4] = v.x; x[nt][5] = v.y; x[nt][6] = v.z; x[nt][7] = v.w;
        }
        multiply<FMT, NT>(r, x, acc, live, mu, tab);
        if (++b == per_e) {
            b = 0;
            ++at;
            if (at < R.active) begin();
        }
    };
    if (i0 < i1) begin();
    for (int i = i0; i < i1; i += kDepth) {
#pragma unroll
        for (int d = 0; d < kDepth; ++d) {
            if (i + d >= i1) break;
            consume(ring[d]);
            fetch_next(ring[d]);
        }
    }

    put<NT>(red[warp], acc, g, t);
    __syncthreads();
    auto store = [&](int tok, int r, float v) {
        // the factor is a power of two: so is its reciprocal
        if (tok < p.m) p.y[static_cast<int64_t>(tok) * p.h + row0 + r] = __float2bfloat16_rn(conv ? v / factor[tok] : v);
    };
    for (int i = threadIdx.x; i < 8 * NT * 16; i += blockDim.x) {
        const int tok = i >> 4, r = i & 15;
        float v = 0.0f;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) v += red[k][tok][r];
        if (splits == 1) store(tok, r, v);
        else part[tok][r] = v;
    }
    if (splits == 1) return;
    cluster_sync();
    const uint32_t base = smem_u32(&part[0][0]);
    for (int i = threadIdx.x + rank * blockDim.x; i < 8 * NT * 16; i += blockDim.x * splits) {
        const int tok = i >> 4, r = i & 15;
        float v = 0.0f;
        for (int s = 0; s < splits; ++s)
            v += ld_shared_cluster_f32(map_shared_rank(base + (tok * kLd + r) * 4, static_cast<uint32_t>(s)));
        store(tok, r, v);
    }
    cluster_sync();  // no CTA leaves while another still reads its sums
}

// ------------------------------- host side -------------------------------
static size_t round256(size_t v) { return (v + 255) & ~static_cast<size_t>(255); }

struct Layout {
    size_t logits, xs, xscale, amax, act32, act16, total;
};
static Layout layout(int64_t h, int64_t f, int E, int top) {
    Layout l;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t o = at;
        at += round256(bytes);
        return o;
    };
    l.logits = take(sizeof(float) * kMaxM * E);
    l.xs = take(sizeof(__half) * kMaxM * h);
    l.xscale = take(sizeof(float) * kMaxM);
    l.amax = take(sizeof(int) * kMaxM);
    l.act32 = take(sizeof(float) * kMaxM * top * f);
    l.act16 = take(sizeof(__half) * kMaxM * top * f);
    l.total = at;
    return l;
}

// Dynamic shared memory beside the static one passes 48 KB: allowed once per kernel and device.
template <typename K>
static cudaError_t allow_smem(K kernel, size_t smem, const DeviceInfo& dev) {
    static std::mutex mu;
    static const void* done[64][16] = {};
    if (smem == 0) return cudaSuccess;
    if (dev.device < 0 || dev.device >= 64) return cudaErrorInvalidDevice;
    const void* fn = reinterpret_cast<const void*>(kernel);
    std::lock_guard<std::mutex> lock(mu);
    for (const void*& d : done[dev.device]) {
        if (d == fn) return cudaSuccess;
        if (d) continue;
        const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
        if (e == cudaSuccess) d = fn;
        return e;
    }
    return cudaErrorInvalidConfiguration;
}

template <typename K>
static cudaError_t launch(K kernel, unsigned grid, unsigned threads, size_t smem, int cluster, const DeviceInfo& dev,
                          cudaStream_t stream, const Params& p, int splits) {
    const cudaError_t allowed = allow_smem(kernel, smem, dev);
    if (allowed != cudaSuccess) return allowed;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    if constexpr (std::is_same_v<K, void (*)(const Params)>) return cudaLaunchKernelEx(&cfg, kernel, p);
    else return cudaLaunchKernelEx(&cfg, kernel, p, splits);
}

static int format_of(const MoeWeight& w) { return !w.integer ? kTable : (w.int4.group == 32 ? kInt4G32 : kInt4); }

static Weight weight_of(const MoeWeight& w) {
    Weight o = {};
    o.k = w.k;
    if (w.integer) {
        o.wq = w.int4.wq;
        o.sides = few::Int4Sides{w.int4.scale, w.int4.zero, w.int4.n, few::items_magic(w.int4.group / few::kItemK), w.int4.scale_f32 ? 1 : 0};
    } else {
        o.wq = w.wq;
        o.absmax_q = w.absmax_q;
        o.absmax_scale = w.absmax_scale;
        o.mu = w.absmax_offset;
        o.codebook = w.codebook;
    }
    return o;
}

}  // namespace moe

size_t moe_workspace_bytes(int64_t h, int64_t f, int E, int top) { return moe::layout(h, f, E, top).total; }
int moe_max_experts() { return moe::kMaxE; }
int moe_max_top() { return moe::kMaxTop; }

cudaError_t launch_moe(const void* X, int64_t m, const void* router, int E, const MoeWeight& gate_up, const MoeWeight& down,
                       int top, bool renormalize, void* Y, int32_t* ids, float* probs, void* ws, const DeviceInfo& dev,
                       cudaStream_t stream) {
    using namespace moe;
    const int64_t h = gate_up.k, f = down.k;
    const Layout l = layout(h, f, E, top);
    char* base = static_cast<char*>(ws);
    Params p = {};
    p.router = static_cast<const __nv_bfloat16*>(router);
    p.E = E;
    p.top = top;
    p.h = static_cast<int>(h);
    p.f = static_cast<int>(f);
    p.renormalize = renormalize ? 1 : 0;
    p.gate_up = weight_of(gate_up);
    p.down = weight_of(down);
    p.logits = reinterpret_cast<float*>(base + l.logits);
    p.xs = reinterpret_cast<__half*>(base + l.xs);
    p.xscale = reinterpret_cast<float*>(base + l.xscale);
    p.amax = reinterpret_cast<int*>(base + l.amax);
    p.act32 = reinterpret_cast<float*>(base + l.act32);
    p.act16 = reinterpret_cast<__half*>(base + l.act16);
    p.x_paired = gate_up.integer ? 1 : 0;
    p.act_paired = down.integer ? 1 : 0;
    const int fu = format_of(gate_up), fd = format_of(down);
    for (int64_t t = 0; t < m; t += kMaxM) {
        p.m = static_cast<int>(m - t < kMaxM ? m - t : kMaxM);
        p.x = static_cast<const __nv_bfloat16*>(X) + t * h;
        p.y = static_cast<__nv_bfloat16*>(Y) + t * h;
        p.ids = ids ? ids + t * top : nullptr;
        p.probs = probs ? probs + t * top : nullptr;
        const int groups = (p.m + kRouterTokens - 1) / kRouterTokens;
        cudaError_t e = launch(k_moe_router, static_cast<unsigned>(E * groups + p.m), kRouterThreads, 0, 1, dev, stream, p, 0);
        if (e != cudaSuccess) return e;
        const int64_t chosen = E < p.m * top ? E : p.m * top;
        const int64_t most = chosen * (f / 8), cap = 2 * dev.sm_count;
        const unsigned grid = static_cast<unsigned>(most < cap ? most : cap);
        const bool two = p.m > 8;
#define NF4_MOE_UP(F) (two ? launch(k_moe_gate_up<F, 2>, grid, kWarps * 32, F == kTable ? kTableBytes : 0, 1, dev, stream, p, 0) \
                           : launch(k_moe_gate_up<F, 1>, grid, kWarps * 32, F == kTable ? kTableBytes : 0, 1, dev, stream, p, 0))
        e = fu == kTable ? NF4_MOE_UP(kTable) : fu == kInt4 ? NF4_MOE_UP(kInt4) : NF4_MOE_UP(kInt4G32);
#undef NF4_MOE_UP
        if (e != cudaSuccess) return e;
        const int64_t tiles = h / 16;
        int splits = 1;
        while (splits < 8 && tiles * splits * 2 <= 2 * dev.sm_count) splits *= 2;
        const unsigned dgrid = static_cast<unsigned>(tiles * splits);
#define NF4_MOE_DOWN(F) (two ? launch(k_moe_down<F, 2>, dgrid, kWarps * 32, F == kTable ? kTableBytes : 0, splits, dev, stream, p, splits) \
                             : launch(k_moe_down<F, 1>, dgrid, kWarps * 32, F == kTable ? kTableBytes : 0, splits, dev, stream, p, splits))
        e = fd == kTable ? NF4_MOE_DOWN(kTable) : fd == kInt4 ? NF4_MOE_DOWN(kInt4) : NF4_MOE_DOWN(kInt4G32);
#undef NF4_MOE_DOWN
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace nf4
