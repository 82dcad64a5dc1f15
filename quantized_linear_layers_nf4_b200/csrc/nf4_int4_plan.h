// nf4_int4_plan.h -- how the linears of integer weights divide a call (nf4_int4_gemv.cu, and
// nf4_gemm.cu with its tile): host arithmetic alone, so that it is tested without a GPU.
// `fit(splits, &clusters)` is few::resident of the kernel: how many clusters of so many CTAs the
// device runs at the same time, 0 where it runs none of that size.
#pragma once

#include "nf4_few_host.h"

namespace nf4 {
namespace int4 {

constexpr int kWarps = 16;  // 128 registers a thread; 24 warps of 80 took a tenth longer

// Steps on their way in a warp: sixteen tokens' X and sums leave room for three.
constexpr int depth_of(int nt) { return nt == 1 ? 4 : 3; }

// Shared memory of a pass: X, the ring, sums of runs, and what is left for the CTA's sums.
struct Room {
    int64_t x_stride, x, ring, slots, left;
};
inline Room room_of(int64_t m, int64_t k, int splits, int fmt, int warps) {
    const int nt = m > 8 ? 2 : 1;
    const int64_t all = (k + few::kStepK - 1) / few::kStepK;
    Room r;
    r.x_stride = (all + splits - 1) / splits * few::kStepK * 2 + (fmt == few::kG32 ? few::x_pad<few::kG32>() : few::x_pad<few::kG64>());
    r.x = (m * r.x_stride + 127) / 128 * 128;
    r.ring = static_cast<int64_t>(warps) * depth_of(nt) * few::kStepBytes;
    r.slots = static_cast<int64_t>(warps) * nt * 512;
    r.left = few::kMaxSmem - r.x - r.ring - r.slots;
    return r;
}

// The largest cluster, up to 8 CTAs, that the device runs.
template <typename Fit>
cudaError_t widest_cluster(Fit&& fit, int* out) {
    for (*out = 8; *out > 1; *out /= 2) {
        int clusters = 0;
        const cudaError_t e = fit(*out, &clusters);
        if (e != cudaSuccess) return e;
        if (clusters > 0) break;
    }
    return cudaSuccess;
}

// Tokens of a pass: so many that an eighth of their X (or what the widest cluster leaves to a CTA)
// leaves room for 16 KB of sums (all sixteen up to k = 33792, eight to 64512, then four).
inline int64_t tokens_of_pass(int64_t m, const Int4Args& w, int widest) {
    int64_t most = kGemvMaxTokens;
    while (most > 1 && room_of(m < most ? m : most, w.k, widest, few::int4_format(w), kWarps).left < 16 * 1024) most /= 2;
    return most;
}

struct Pass {
    int splits, warps;
    int64_t clusters;
    Room at;
    int64_t groups, steps;  // of 8 rows; of k
};
// The pass of m tokens.
template <typename Fit>
cudaError_t plan_pass(int64_t m, const Int4Args& w, int sm_count, int widest, Fit&& fit_of, Pass* out) {
    Pass p = {};
    p.steps = (w.k + few::kStepK - 1) / few::kStepK;
    p.groups = (w.n + 7) / 8;
    // k is split over a cluster where a CTA's share of X would take long to bring in (64 KB),
    // or where there are fewer row groups than SMs and each part still feeds the warps
    p.splits = 1;
    while (p.splits < widest &&
           (m * w.k * 2 / p.splits > 64 * 1024 || (p.groups * p.splits * 2 <= sm_count && p.steps >= p.splits * kWarps)))
        p.splits *= 2;
    int fit = 0;
    const cudaError_t e = fit_of(p.splits, &fit);
    if (e != cudaSuccess) return e;
    if (fit < 1) return cudaErrorInvalidConfiguration;
    p.clusters = fit < p.groups ? fit : p.groups;
    const int64_t steps = ((p.groups + p.clusters - 1) / p.clusters + 1) / 2 * ((p.steps + p.splits - 1) / p.splits);
    // m = 4 is about where what a warp costs at its start outweighs what it adds
    p.warps = steps <= (m > 4 ? 1 : 2) * few::kFewSteps && m <= kWarps / 2 ? kWarps / 2 : kWarps;  // a warp or more a token for X
    p.at = room_of(m, w.k, p.splits, few::int4_format(w), p.warps);
    if (p.at.left < m * 64) return cudaErrorInvalidConfiguration;
    while (p.splits > 1 && (p.groups + p.clusters - 1) / p.clusters * 8 * m * 4 > p.at.left) p.clusters += fit;
    if (p.clusters * p.splits > 0x7fffffff || p.groups > 0x7fffffff) return cudaErrorInvalidConfiguration;
    *out = p;
    return cudaSuccess;
}

}  // namespace int4

namespace gemm {

constexpr int kBM = 256;  // tokens per CTA tile (two 128-row MMA halves)
constexpr int kBN = 256;  // weight rows per CTA tile (MMA N)
constexpr int kBK = 64;   // k per stage: one 128-byte swizzle row of bf16
constexpr int kStagesA = 3;
constexpr int kStagesB = 2;
constexpr int kStagesP = 4;
constexpr int kABytes = kBM * kBK * 2;  // 32768
constexpr int kBBytes = kBN * kBK * 2;  // 32768
constexpr int kPBytes = kBN * kBK / 2;  // 8192
constexpr int kPartPad = 4;  // words between the rows of a CTA's sums in shared memory, for the banks
constexpr int kOffB = kStagesA * kABytes;
constexpr int kOffP = kOffB + kStagesB * kBBytes;
constexpr int kOffBar = kOffP + kStagesP * kPBytes;

// Tiles for integer codes.  A stage takes a time that goes about as 350 + its weight rows, since
// most of it is the decoding warps' latency, so that a few large tiles with k split over a cluster
// beat many small ones, and the waves of tiles over the SMs go in whole numbers.  128 tokens over
// 4096 x 4096 take 14 us with 256 rows and k in eight parts, 25 with 32 rows and k whole, 44 with 256
// and whole; 512 over 11008 x 4096, whose tiles leave no SMs for parts, 45 with 160 rows and 59 with 256.
struct Plan {
    int rows, splits;
    double us;
};
template <typename Fit>
cudaError_t plan_int4(int64_t m, int64_t n, int64_t k, int parts, Fit&& fit_of, Plan* out) {
    const int64_t token_tiles = (m + kBM - 1) / kBM, stages = k / kBK, x_rows = m <= 128 ? 128 : kBM;
    const double stage = 0.95e-3 * (m <= 128 ? 1.0 : 1.15) * parts;
    *out = Plan{kBN, 1, 1e30};
    for (int splits = 1; splits == 1 || (splits <= 8 && stages >= 4 * splits); splits *= 2) {
        int fit = 0;  // clusters at a time
        const cudaError_t e = fit_of(splits, &fit);
        if (e != cudaSuccess) return e;
        if (fit < 1) break;
        for (int rows = kBN; rows >= 32; rows -= 32) {
            if (splits > 1 && x_rows * (rows + kPartPad) * 4 > kOffBar) continue;
            const int64_t waves = ((n + rows - 1) / rows * token_tiles + fit - 1) / fit;
            double us = 5.0 + stage * static_cast<double>(waves * ((stages + splits - 1) / splits) * (350 + rows));
            if (splits > 1) us += 1.5 + 3e-5 * static_cast<double>(x_rows * rows * waves);
            if (us < out->us) *out = Plan{rows, splits, us};
        }
    }
    return cudaSuccess;
}

}  // namespace gemm
}  // namespace nf4
