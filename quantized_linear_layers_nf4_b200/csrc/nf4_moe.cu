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
//   k_moe_gate_up  every CTA chooses the experts itself from the logits (which saves
//                  another launch), then takes its share of the (expert, 8 rows of f)
//                  tiles: 8 gate rows and the 8 up rows that belong to them form the 16
//                  rows of one mma.sync tile, so a lane holds a gate sum and its up sum
//   k_moe_down     the tokens are the columns, so the sum over experts is the sum over k of
//                  all chosen experts one after the other
// The weights' decoding and the step geometry are in nf4_few.cuh.  Every sum is taken in a
// fixed order.
//
// NF4: one token of 64 experts (6 chosen, 2048 x 1408) takes 25 us, of which the launches and the
// routing are about 10; sixteen tokens of 8 experts (2 chosen, 4096 x 14336) 256 us, 2.8 TB/s: L1's
// data pipe is 70 % busy, about half of that with table look-ups, the rest with X and the codes' way
// through the ring (the copies alone, at 5.4 TB/s, would take 134 us).  Integer codes: 7 tokens of 128
// experts (8 chosen, 2048 x 768) 45 us, 2.5 TB/s; 54 % of the issue slots are used and no pipe more.
// Above sixteen tokens a pass reads its experts again: 32 tokens of those 8 experts 526 us.
//
// Roundings.  X (bf16) times a power of two per token is exact in fp16, but for values below
// 2^-31 of the token's largest.  Codebook levels
// are rounded to fp16 (within 2^-11 of the value; bf16 would be 2^-8, as much as the rounding
// of the result); integer codes are exact.  The activations a are kept in fp32 and, for the
// products, rounded to fp16 (2^-11); where a token's largest one is outside [2^-6, 2^15)
// they are read from the fp32 copy and scaled by a power of two on the way.
#include "nf4.h"
#include "nf4_few.cuh"
#include "nf4_few_host.h"
#include "nf4_ptx.cuh"

namespace nf4 {
namespace moe {

constexpr int kMaxM = 16;  // tokens of a pass
constexpr int kMaxTop = NF4_MOE_MAX_TOP_K;
constexpr int kMaxE = NF4_MOE_MAX_EXPERTS;
// choose: a lane a choice, sixteen logits a lane at most; route: a lane for each 32 experts
static_assert(kMaxTop <= 32 && kMaxE <= 16 * 32 && kMaxE % 32 == 0, "routing tables");
constexpr int kMaxPairs = kMaxM * kMaxTop;
constexpr int kWarps = 20;  // 96 registers a thread; 16 and 24 warps took a few percent longer
constexpr int kDepth = 3;  // steps on their way in a warp, beside the table of levels

struct Params {
    const __nv_bfloat16* x;
    const __nv_bfloat16* router;
    int m, E, top;
    int h, f, hp, fp;
    int renormalize;
    few::Weight gate_up, down;
    float* logits;   // [m][E]
    __half* xs;      // [m][hp], hp = h and fp = f up to whole steps: zeros behind the end
    float* xscale;   // [m]
    int* amax;       // [m] bits of the largest |a| of a token
    float* act32;    // [m * top][fp], the pairs of an expert together
    __half* act16;
    __nv_bfloat16* y;
    int32_t* ids;    // [m][top] or null
    float* probs;    // [m][top] or null
    int x_paired, act_paired;  // eight values in the order of int4_f16's pairs
    int ring_at, slots_at;      // bytes in shared memory: the ring, sums of runs
    few::Shares rows;           // down: 8-row groups of the output over the CTAs
    int part_at, part_rows;     // down: a pair's products with those rows
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
                if (t0 + j < p.m) dot8(few::ld_global16(reinterpret_cast<const uint4*>(p.x + static_cast<int64_t>(t0 + j) * p.h) + c), rv, s[j]);
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
        const uint4 v = few::ld_global16(x + c);
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) top = max(top, max(u[j] & 0x7fffu, (u[j] >> 16) & 0x7fffu));
    }
    top = __reduce_max_sync(kFull, top);
    if (lane == 0) part[warp][0] = __uint_as_float(top);
    __syncthreads();
    for (int w = 0; w < kRouterThreads / 32; ++w) top = max(top, __float_as_uint(part[w][0]));
    const int ex = few::scale_exponent(static_cast<int>(top >> 7));
    const float factor = few::scale_up(ex);
    if (tid == 0) {
        p.xscale[t] = few::scale_down(ex);
        p.amax[t] = 0;
    }
    __half* xs = p.xs + static_cast<int64_t>(t) * p.hp;
    for (int c = chunks + tid; c < p.hp / 8; c += kRouterThreads) reinterpret_cast<uint4*>(xs)[c] = make_uint4(0u, 0u, 0u, 0u);
    // behind the end of f, of the activations to come
    for (int i = tid; i < p.top * (p.fp - p.f); i += kRouterThreads) {
        const int64_t o = (static_cast<int64_t>(t) * p.top + i / (p.fp - p.f)) * p.fp + p.f + i % (p.fp - p.f);
        p.act32[o] = 0.0f;
        p.act16[o] = __float2half_rn(0.0f);
    }
    for (int c = tid; c < chunks; c += kRouterThreads) {
        const uint4 v = few::ld_global16(x + c);
        uint32_t u[4] = {v.x, v.y, v.z, v.w}, o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) u[j] = o[j] = few::scale_pair(u[j], factor);
        if (p.x_paired) few::pair_x(u[0], u[1], u[2], u[3], o);
        reinterpret_cast<uint4*>(xs)[c] = make_uint4(o[0], o[1], o[2], o[3]);
    }
}

// ------------------------------- routing -------------------------------
struct Route {
    uint32_t mask[kMaxE];         // tokens of an expert
    uint16_t pos[kMaxE];          // of an expert's first entry in the list
    uint16_t list[kMaxPairs];     // chosen experts, ascending, once for each eight of their tokens
    uint16_t base[kMaxPairs + 1]; // first pair of an entry; the pairs of an expert are by token
    float prob[kMaxM][kMaxTop];
    uint16_t id[kMaxM][kMaxTop];
    uint16_t pair[kMaxM][kMaxTop];
    float pair_prob[kMaxPairs];
    uint8_t pair_tok[kMaxPairs];
    uint32_t chunk[kMaxE / 32];
    int active;
};

// A key that orders as the logit does; NaN below everything, 0 for "none".
__device__ __forceinline__ uint32_t order_key(float v) {
    if (v != v) return 1u;
    const uint32_t u = __float_as_uint(v + 0.0f);  // -0 as +0
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ float key_value(uint32_t k) {  // and back; NaN for the key of NaN
    return k == 1u ? __int_as_float(0x7fffffff) : __uint_as_float((k & 0x80000000u) ? k & 0x7fffffffu : ~k);
}

// One token's choice, by a warp: C = ceil(E / 32) logits a lane; the largest key by a warp
// reduction, among equal ones the lowest expert by another.  A lone warp's instructions follow
// one another slowly, so there are few: the number of logits is a constant, and what can be
// done for all choices at once is done after the loop.
template <int C>
__device__ __forceinline__ void choose(const Params& p, Route& R, int t, int lane) {
    uint32_t key[C];
    const float* l = p.logits + t * p.E;
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int e = 32 * i + lane;
        key[i] = e < p.E ? order_key(__ldcg(l + e)) : 0u;
    }
    uint32_t all[C];
#pragma unroll
    for (int i = 0; i < C; ++i) all[i] = key[i];
    uint32_t mine = 0, best = 0;
    int id = 0;
    for (int j = 0; j < p.top; ++j) {
        uint32_t k = key[0];
#pragma unroll
        for (int i = 1; i < C; ++i) k = max(k, key[i]);
        k = __reduce_max_sync(kFull, k);
        uint32_t at = 0xffffu;
#pragma unroll
        for (int i = C - 1; i >= 0; --i)
            if (key[i] == k) at = 32 * i + lane;
        at = __reduce_min_sync(kFull, at);
#pragma unroll
        for (int i = 0; i < C; ++i)
            if (at == 32u * i + lane) key[i] = 0;
        if (j == 0) best = k;
        if (lane == j) {
            mine = k;
            id = static_cast<int>(at);
        }
    }
    const float top = key_value(best), ex = lane < p.top ? expf(key_value(mine) - top) : 0.0f;
    float total = 0.0f;
    if (p.renormalize) {
        total = ex;
    } else {
#pragma unroll
        for (int i = 0; i < C; ++i) total += all[i] ? expf(key_value(all[i]) - top) : 0.0f;
    }
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(kFull, total, o);
    if (lane < p.top) {
        R.id[t][lane] = static_cast<uint16_t>(id);
        R.prob[t][lane] = ex / total;
        atomicOr(&R.mask[id], 1u << t);
    }
}

// Every thread of the block; the logits are complete.
__device__ __forceinline__ void route(const Params& p, Route& R) {
    const int tid = threadIdx.x, warp = few::warp_index(), lane = tid & 31, warps = blockDim.x >> 5;
    for (int e = tid; e < p.E; e += blockDim.x) R.mask[e] = 0;
    __syncthreads();
    for (int t = warp; t < p.m; t += warps) {
        if (p.E <= 32) choose<1>(p, R, t, lane);
        else if (p.E <= 64) choose<2>(p, R, t, lane);
        else if (p.E <= 128) choose<4>(p, R, t, lane);
        else if (p.E <= 256) choose<8>(p, R, t, lane);
        else choose<16>(p, R, t, lane);
    }
    __syncthreads();
    // the list: a warp for each 32 experts counts its entries and their pairs, then finds its place
    const int chunks = (p.E + 31) >> 5;
    for (int c = warp; c < chunks; c += warps) {
        const int e = 32 * c + lane;
        const int cnt = e < p.E ? __popc(R.mask[e]) : 0;
        const uint32_t both = __reduce_add_sync(kFull, static_cast<uint32_t>((cnt + 7) >> 3) << 16 | cnt);
        if (lane == 0) R.chunk[c] = both;
    }
    __syncthreads();
    for (int c = warp; c < chunks; c += warps) {
        const int e = 32 * c + lane;
        const int cnt = e < p.E ? __popc(R.mask[e]) : 0;
        const uint32_t before = __reduce_add_sync(kFull, lane < c ? R.chunk[lane] : 0u);
        const uint32_t own = static_cast<uint32_t>((cnt + 7) >> 3) << 16 | cnt;
        uint32_t sum = own;
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t up = __shfl_up_sync(kFull, sum, o);
            if (lane >= o) sum += up;
        }
        const uint32_t first = before + sum - own;
        if (cnt) {
            const int at = static_cast<int>(first >> 16);
            R.pos[e] = static_cast<uint16_t>(at);
            for (int i = 0; 8 * i < cnt; ++i) {
                R.list[at + i] = static_cast<uint16_t>(e);
                R.base[at + i] = static_cast<uint16_t>((first & 0xffffu) + 8 * i);
            }
        }
        if (c == chunks - 1 && lane == 31) {
            R.active = static_cast<int>((before + sum) >> 16);
            R.base[R.active] = static_cast<uint16_t>(before + sum);
        }
    }
    __syncthreads();
    for (int t = warp; t < p.m; t += warps) {
        if (lane >= p.top) continue;
        const int e = R.id[t][lane];
        const int pair = R.base[R.pos[e]] + __popc(R.mask[e] & ((1u << t) - 1));
        R.pair[t][lane] = static_cast<uint16_t>(pair);
        R.pair_prob[pair] = R.prob[t][lane];
        R.pair_tok[pair] = static_cast<uint8_t>(t);
    }
    __syncthreads();
}

// The eight columns of an entry's products are its pairs (token, choice); those past them are not
// used, and their lanes load no X: eight lanes (two columns) less are a pass of L1 less, and
// L1 is what bounds these kernels.  An expert of more than eight tokens comes again for the
// next eight: sums for sixteen at once cost registers and with them warps, on every call,
// and few calls have such an expert.
struct Columns {
    int idx = -1, base = 0, cnt = 0, pair = 0;  // entry of the list; its pairs; the lane's one
    bool mine = false;                          // which is not a repetition
    __device__ __forceinline__ bool enter(const Route& R, int i, int g) {
        if (i == idx) return false;
        idx = i;
        base = R.base[i];
        cnt = R.base[i + 1] - base;
        pair = base + min(g, cnt - 1);
        mine = g < cnt;
        return true;
    }
};

// A lane's X of a step, from global memory through L1, `x` its first chunk: all of it is asked
// for before the first word is decoded.
template <int F>
__device__ __forceinline__ void load_x(uint32_t (&v)[4][4], const __half* x) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint4 u = few::ld_global16(x + (few::x_chunk<F>(i, 0) - few::x_chunk<F>(0, 0)) * 8);
        v[i][0] = u.x; v[i][1] = u.y; v[i][2] = u.z; v[i][3] = u.w;
    }
}

// ------------------------------ gate and up ------------------------------
template <int F, bool Z>
__global__ void __launch_bounds__(kWarps * 32, 1) k_moe_gate_up(const __grid_constant__ Params p) {
    extern __shared__ __align__(128) uint8_t smem[];  // levels, the ring, sums of runs
    __shared__ Route R;

    const int warp = few::warp_index(), lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    if (F == few::kTable) few::build_table(smem, p.gate_up.codebook);
    grid_dependency_wait();
    grid_launch_dependents();
    route(p, R);
    if (blockIdx.x == 0)
        for (int i = threadIdx.x; i < p.m * p.top; i += blockDim.x) {
            if (p.ids) p.ids[i] = R.id[i / p.top][i % p.top];
            if (p.probs) p.probs[i] = R.prob[i / p.top][i % p.top];
        }

    const few::Weight& w = p.gate_up;
    const float mu = F == few::kTable ? __ldg(w.mu) : 0.0f;
    const uint32_t bank = 4 * lane;
    const int per_e = p.f / 8;
    const few::Shares mine = few::shares_of(R.active * per_e, gridDim.x);
    const int t0 = mine.start(blockIdx.x), t1 = mine.start(blockIdx.x + 1);
    const int ns = (p.h + few::kStepK - 1) / few::kStepK;
    const few::Shares runs = few::shares_of_warps<kWarps>((t1 - t0) * ns);

    auto rows_of = [&](int tile, int64_t(&row)[2]) {
        const int idx = (t0 + tile) / per_e;
        row[0] = static_cast<int64_t>(R.list[idx]) * 2 * p.f + (t0 + tile - idx * per_e) * 8 + g;
        row[1] = row[0] + p.f;
    };
    few::Runner<F, Z, kDepth, 1> run;
    run.find(w, smem + p.ring_at, warp, lane, runs, 0, ns, rows_of);
    run.start(w, rows_of);

    Columns col;
    const __half* x = nullptr;  // the lane's first chunk of its column
    auto begin = [&](int tile) {
        if (col.enter(R, (t0 + tile) / per_e, g)) x = p.xs + static_cast<int64_t>(R.pair_tok[col.pair]) * p.hp + few::x_chunk<F>(0, t) * 8;
    };
    uint32_t q[4][4] = {};
    auto ahead = [&](int step) {
        const uint32_t to = static_cast<uint32_t>(step) * few::kStepK;
        if (col.mine) load_x<F>(q, x + to);
    };
    auto mul = [&](const uint8_t* entry, int step) {
        few::multiply<F, Z, 1>(run.side, entry, run.places, run.acc, smem, bank, step, [&](int j, int, uint32_t(&v)[4]) {
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = q[j][i];
        });
    };
    auto finish = [&](int tile) {
        const int r = ((t0 + tile) % per_e) * 8 + g;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const int j = 2 * t + c;
            float a = 0.0f;
            int tok = 0;
            if (j < col.cnt) {
                tok = R.pair_tok[col.base + j];
                const float down = p.xscale[tok];
                const float gate = run.acc[0][c] * down, up = run.acc[0][2 + c] * down;
                a = gate / (1.0f + expf(-gate)) * up * R.pair_prob[col.base + j];
                const int64_t o = static_cast<int64_t>(col.base + j) * p.fp;
                const int place = p.act_paired ? (r & ~7) + paired(g) : r;
                p.act32[o + place] = a;
                p.act16[o + place] = __float2half_rn(a);
            }
            int big = __float_as_int(fabsf(a));
            for (int s = 4; s < 32; s <<= 1) big = max(big, __shfl_xor_sync(kFull, big, s));
            if (g == 0 && j < col.cnt) atomicMax(p.amax + tok, big);
        }
    };
    run.run(w, mu, reinterpret_cast<float4*>(smem + p.slots_at), runs, rows_of, begin, ahead, mul, finish);
}

// --------------------------------- down ---------------------------------
// As load_x, from fp32 and times a token's power of two.
template <int F>
__device__ __forceinline__ void load_wide(uint32_t (&v)[4][4], const float* x, float up) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const uint4 u = few::ld_global16(x + (few::x_chunk<F>(i, 0) - few::x_chunk<F>(0, 0)) * 8 + 4 * k);
            const __half2 lo = __floats2half2_rn(__uint_as_float(u.x) * up, __uint_as_float(u.y) * up);
            const __half2 hi = __floats2half2_rn(__uint_as_float(u.z) * up, __uint_as_float(u.w) * up);
            v[i][2 * k] = *reinterpret_cast<const uint32_t*>(&lo);
            v[i][2 * k + 1] = *reinterpret_cast<const uint32_t*>(&hi);
        }
    }
}

// A CTA has a run of output rows; a tile is 16 of them with one chosen expert's f, its columns that
// expert's pairs.  The products of a pair go to shared memory, and a token's are added there in the
// order of its choices.
template <int F, bool Z>
__global__ void __launch_bounds__(kWarps * 32, 1) k_moe_down(const __grid_constant__ Params p) {
    extern __shared__ __align__(128) uint8_t smem[];  // levels, the ring, sums of runs, the pairs' products
    __shared__ Route R;
    __shared__ float factor[kMaxM];
    __shared__ int wide;
    float* part = reinterpret_cast<float*>(smem + p.part_at);

    const int warp = few::warp_index(), lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    // The logits are those the previous kernel waited for before it let this one start.
    if (F == few::kTable) few::build_table(smem, p.down.codebook);
    route(p, R);

    const few::Weight& w = p.down;
    const float mu = F == few::kTable ? __ldg(w.mu) : 0.0f;
    const uint32_t bank = 4 * lane;
    const int g0 = p.rows.start(blockIdx.x), g1 = p.rows.start(blockIdx.x + 1);
    const int row_tiles = (g1 - g0 + 1) / 2;
    const int ns = (p.f + few::kStepK - 1) / few::kStepK;
    const few::Shares runs = few::shares_of_warps<kWarps>(R.active * row_tiles * ns);

    auto rows_of = [&](int tile, int64_t(&row)[2]) {
        const int idx = tile / row_tiles, grp = g0 + (tile - idx * row_tiles) * 2;
        row[0] = static_cast<int64_t>(R.list[idx]) * p.h + grp * 8 + g;
        // where the second half is another CTA's, the first takes its place and is not stored
        row[1] = row[0] + (grp + 1 < g1 ? 8 : 0);
    };
    few::Runner<F, Z, kDepth, 1> run;
    run.find(w, smem + p.ring_at, warp, lane, runs, 0, ns, rows_of);
    run.start(w, rows_of);
    grid_dependency_wait();
    grid_launch_dependents();

    // fp16 activations, or fp32 ones scaled where a token's largest is out of range
    if (threadIdx.x == 0) wide = 0;
    __syncthreads();
    if (threadIdx.x < p.m) {
        const int bits = __ldcg(p.amax + threadIdx.x);
        factor[threadIdx.x] = few::scale_up(few::scale_exponent(bits >> 23));
        if (bits != 0 && (bits >= 0x47000000 || bits < 0x3c800000)) wide = 1;  // >= 2^15, < 2^-6
    }
    __syncthreads();
    const bool conv = wide != 0;

    Columns col;
    const __half* x = nullptr;  // the lane's first chunk of its column
    auto begin = [&](int tile) {
        if (col.enter(R, tile / row_tiles, g)) x = p.act16 + static_cast<int64_t>(col.pair) * p.fp + few::x_chunk<F>(0, t) * 8;
    };
    uint32_t q[4][4] = {};
    auto ahead = [&](int step) {
        const uint32_t to = static_cast<uint32_t>(step) * few::kStepK;
        if (!col.mine) return;
        if (!conv) load_x<F>(q, x + to);
        else load_wide<F>(q, p.act32 + (x - p.act16) + to, factor[R.pair_tok[col.pair]]);
    };
    auto mul = [&](const uint8_t* entry, int step) {
        few::multiply<F, Z, 1>(run.side, entry, run.places, run.acc, smem, bank, step, [&](int j, int, uint32_t(&v)[4]) {
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = q[j][i];
        });
    };
    auto finish = [&](int tile) {
        const int r0 = (tile % row_tiles) * 16;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const int j = 2 * t + c;
            if (j >= col.cnt) continue;
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (r0 + 8 * i < (g1 - g0) * 8) part[(col.base + j) * p.part_rows + r0 + 8 * i + g] = run.acc[0][2 * i + c];
        }
    };
    run.run(w, mu, reinterpret_cast<float4*>(smem + p.slots_at), runs, rows_of, begin, ahead, mul, finish);
    __syncthreads();
    const int rows = (g1 - g0) * 8;
    for (int i = threadIdx.x; i < p.m * rows; i += blockDim.x) {
        const int tok = i / rows, r = i - tok * rows;
        float v = 0.0f;
        for (int j = 0; j < p.top; ++j) v += part[R.pair[tok][j] * p.part_rows + r];
        // the factor is a power of two: so is its reciprocal
        p.y[static_cast<int64_t>(tok) * p.h + g0 * 8 + r] = __float2bfloat16_rn(conv ? v / factor[tok] : v);
    }
}

// ------------------------------- host side -------------------------------
static size_t round256(size_t v) { return (v + 255) & ~static_cast<size_t>(255); }

struct Layout {
    size_t logits, xs, xscale, amax, act32, act16, total;
};
static int64_t whole_steps(int64_t k) { return (k + few::kStepK - 1) / few::kStepK * few::kStepK; }
static Layout layout(int64_t h, int64_t f, int E, int top) {
    h = whole_steps(h);
    f = whole_steps(f);
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

static few::Weight weight_of(const MoeWeight& w) {
    if (w.integer) return few::int4_weight(w.int4);
    few::Weight o = {};
    o.k = static_cast<int>(w.k);
    o.wq = w.wq;
    o.absmax_q = w.absmax_q;
    o.absmax_scale = w.absmax_scale;
    o.mu = w.absmax_offset;
    o.codebook = w.codebook;
    o.units = static_cast<int>(w.k / few::kItemK);
    return o;
}
// Index of a kernel's instance for a weight: the table form, then three group sizes with and without zero points.
static int form_of(const MoeWeight& w) {
    return w.integer ? 1 + 2 * (few::int4_format(w.int4) - few::kG128) + (w.int4.zero ? 1 : 0) : 0;
}

}  // namespace moe

size_t moe_workspace_bytes(int64_t h, int64_t f, int E, int top) { return moe::layout(h, f, E, top).total; }

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
    p.hp = static_cast<int>(whole_steps(h));
    p.fp = static_cast<int>(whole_steps(f));
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
#define NF4_MOE_FORMS(K)                                                                                        \
    {reinterpret_cast<const void*>(&K<few::kTable, false>), reinterpret_cast<const void*>(&K<few::kG128, false>), \
     reinterpret_cast<const void*>(&K<few::kG128, true>),   reinterpret_cast<const void*>(&K<few::kG64, false>),  \
     reinterpret_cast<const void*>(&K<few::kG64, true>),    reinterpret_cast<const void*>(&K<few::kG32, false>),  \
     reinterpret_cast<const void*>(&K<few::kG32, true>)}
    static const void* const up_fns[7] = NF4_MOE_FORMS(k_moe_gate_up);
    static const void* const down_fns[7] = NF4_MOE_FORMS(k_moe_down);
#undef NF4_MOE_FORMS
    for (int64_t t = 0; t < m; t += kMaxM) {
        p.m = static_cast<int>(m - t < kMaxM ? m - t : kMaxM);
        p.x = static_cast<const __nv_bfloat16*>(X) + t * h;
        p.y = static_cast<__nv_bfloat16*>(Y) + t * h;
        p.ids = ids ? ids + t * top : nullptr;
        p.probs = probs ? probs + t * top : nullptr;
        void* args[1] = {&p};
        const int groups = (p.m + kRouterTokens - 1) / kRouterTokens;
        cudaError_t e = few::launch(reinterpret_cast<const void*>(&k_moe_router), E * groups + p.m, kRouterThreads, 0, 1, stream, args);
        if (e != cudaSuccess) return e;

        int fit = 0;
        const int64_t chosen = E < p.m * top ? E : p.m * top;  // at most, but for experts of more than eight tokens
        auto warps_of = [&](int64_t steps) { return steps <= few::kFewSteps ? kWarps / 2 : kWarps; };
        auto arrange = [&](const MoeWeight& w, int warps) {
            p.ring_at = w.integer ? 0 : few::kTableBytes;
            p.slots_at = p.ring_at + warps * kDepth * few::kStepBytes;
            p.part_at = p.slots_at + warps * 512;
        };
        const void* fn = up_fns[form_of(gate_up)];
        if ((e = few::resident(fn, kWarps * 32, 1, dev, &fit)) != cudaSuccess) return e;
        int64_t grid = chosen * (f / 8) < fit ? chosen * (f / 8) : fit;
        int warps = warps_of((chosen * (f / 8) + grid - 1) / grid * ((h + few::kStepK - 1) / few::kStepK));
        arrange(gate_up, warps);
        if ((e = few::launch(fn, grid, warps * 32, p.part_at, 1, stream, args)) != cudaSuccess) return e;

        // down: so many output rows a CTA that the pairs' products fit
        fn = down_fns[form_of(down)];
        if ((e = few::resident(fn, kWarps * 32, 1, dev, &fit)) != cudaSuccess) return e;
        grid = h / 8 < fit ? h / 8 : fit;
        warps = warps_of(((h / 8 + grid - 1) / grid + 1) / 2 * chosen * ((f + few::kStepK - 1) / few::kStepK));
        arrange(down, warps);
        const int64_t pairs = p.m * top, room = few::kMaxSmem - p.part_at;
        while ((h / 8 + grid - 1) / grid * 8 * pairs * 4 > room) grid += fit;
        p.rows = few::shares_of(static_cast<int>(h / 8), static_cast<int>(grid));
        p.part_rows = static_cast<int>((h / 8 + grid - 1) / grid * 8);
        if ((e = few::launch(fn, grid, warps * 32, p.part_at + pairs * p.part_rows * 4, 1, stream, args)) != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace nf4
