// nf4_int4_plan.h -- how the few-token kernel of integer weights divides a call
// (nf4_int4_gemv.cu): host arithmetic alone, so that it is tested without a GPU.
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

// Tokens of a pass: so many that an eighth of their X leaves room for 16 KB of sums (all sixteen
// up to k = 33792, eight to 64512, then four).
inline int64_t tokens_of_pass(int64_t m, const Int4Args& w) {
    int64_t most = kGemvMaxTokens;
    while (most > 1 && room_of(m < most ? m : most, w.k, 8, few::int4_format(w), kWarps).left < 16 * 1024) most /= 2;
    return most;
}

}  // namespace int4
}  // namespace nf4
