// nf4_int4_gemv.cu -- Y[t, r] = sum_c X[t, c] (q[r, c] - z) s for few tokens, sixteen
// at a time, integer 4-bit weights with group scales (sm_100a).
//
// Bound by HBM: half a byte of code per weight.  The tensor cores (mma.sync: sixteen
// tokens are too few for a 128-row tcgen05 tile, and the codes would have to pass
// through shared or tensor memory on the way) multiply the exact integers q - z by X,
// and the scale goes onto the fp32 sum of each group or 128 k (nf4_few.cuh), so nothing is
// rounded between the codes and the fp32 sums.
//
// One CTA an SM.  A cluster of S CTAs has a run of rows, each CTA a range of k of them; the
// CTA keeps its part of X in shared memory (as fp16, scaled by a power of two per token)
// and cuts its (16 rows) x (128 k) steps, row tile by row tile, into equal runs for its
// warps (few::Runner).  The CTAs' sums are added in rank order through distributed shared
// memory, so results do not depend on timing.
//
// Groups of 128, bf16 scales: one token over 4096 x 4096 takes 6.2 us, of which a launch and X are
// 4, over 28672 x 8192 27.4 us (4.4 TB/s, 69 % of the rate of a copy); sixteen tokens 44.5 us there
// (48.2 with groups of 64 and zero points).  No unit is full then: a step (16 rows x 128 k) is 202 warp
// instructions (247; one token 151), of which decoding is 72 and products 16, and they fill 57 % (61 %;
// 63 %) of the issue slots with the four warps that a scheduler has.
#include "nf4_few.cuh"
#include "nf4_int4_plan.h"
#include "nf4_ptx.cuh"

namespace nf4 {
namespace int4 {

struct GemvArgs {
    const __nv_bfloat16* x;
    few::Weight w;
    void* y;
    int m, x_lg;            // tokens; warps that bring one token's X in, as a power of two
    few::Shares rows;       // 8-row groups of W over the clusters
    few::Shares ks;         // steps of k over a cluster's CTAs
    int splits;
    int x_stride;           // bytes of a token's part of X in shared memory
    int ring_at, slots_at, part_at;  // byte offsets in shared memory
    int part_rows;
    int bf16_out, early;
};

template <int F, bool Z, int NT>
__global__ void __launch_bounds__(kWarps * 32, 1) k_int4_gemv(const __grid_constant__ GemvArgs a) {
    extern __shared__ __align__(128) uint8_t smem[];  // X, the ring, sums of runs, the CTA's sums
    __shared__ uint32_t top[kWarps];  // bf16 magnitude of a token's largest value in this CTA's range of k
    float* part = reinterpret_cast<float*>(smem + a.part_at);

    const int warp = few::warp_index(), lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int rank = a.splits > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int cl = static_cast<int>(blockIdx.x) >> (31 - __clz(a.splits));
    const int g0 = a.rows.start(cl), g1 = a.rows.start(cl + 1);
    const int s0 = a.ks.start(rank), ns = a.ks.start(rank + 1) - s0;  // steps of a tile
    const int warps = blockDim.x >> 5;
    const few::Shares runs = few::shares_of_warps<kWarps>((g1 - g0 + 1) / 2 * ns);
    auto rows_of = [&](int tile, int64_t(&row)[2]) {
        const int grp = g0 + tile * 2;
        // where a run's last tile has one group, that takes the place of another CTA's, and rows
        // past n are the last one: they are not stored
        row[0] = min(static_cast<int64_t>(grp) * 8 + g, a.w.n - 1);
        row[1] = grp + 1 < g1 ? min(static_cast<int64_t>(grp) * 8 + 8 + g, a.w.n - 1) : row[0];
    };
    few::Runner<F, Z, depth_of(NT), NT> R;
    R.find(a.w, smem + a.ring_at, warp, lane, runs, s0, ns, rows_of);
    if (!a.early) grid_dependency_wait();
    R.start(a.w, rows_of);
    if (a.early) grid_dependency_wait();
    grid_launch_dependents();
    // this CTA's k range of X
    const int first = s0 * (few::kStepK / 8);
    few::stage_x<F>(reinterpret_cast<const uint4*>(a.x) + first, a.w.k / 8, min((s0 + ns) * (few::kStepK / 8), a.w.k / 8) - first,
                    ns * (few::kStepK / 8), a.m, a.x_lg, smem, a.x_stride, top, warp, lane, warps);

    const uint8_t* xb[NT][2];  // columns past m read the last token's: their sums are not stored
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        xb[nt][0] = smem + min(nt * 8 + g, a.m - 1) * a.x_stride + few::x_lane<F>(t) + few::x_flip<F>(t);
        xb[nt][1] = xb[nt][0] - 2 * few::x_flip<F>(t);
    }
    auto mul = [&](const uint8_t* entry, int step) {
        const uint32_t x0 = (step - s0) * (few::kStepK * 2);
        few::multiply<F, Z, NT>(R.side, entry, R.places, R.acc, nullptr, 0u, step, [&](int j, int nt, uint32_t(&v)[4]) {
            const uint4 u = *reinterpret_cast<const uint4*>(xb[nt][j >> 1] + x0 + few::x_word<F>(j));
            v[0] = u.x; v[1] = u.y; v[2] = u.z; v[3] = u.w;
        });
    };
    const int64_t row0 = static_cast<int64_t>(g0) * 8;
    const int rows = static_cast<int>(min(static_cast<int64_t>(g1 - g0) * 8, a.w.n - row0));
    auto finish = [&](int tile) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int tok = nt * 8 + 2 * t + c;
                if (tok >= a.m) continue;
                const float down = few::scale_down(few::scale_exponent(static_cast<int>(top[tok] >> 7)));
                const int64_t o = tok * a.w.n + row0;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int r = tile * 16 + 8 * i + g;
                    if (r >= rows) continue;
                    const float v = R.acc[nt][2 * i + c] * down;
                    if (a.splits > 1) part[tok * a.part_rows + r] = v;
                    else if (a.bf16_out) reinterpret_cast<__nv_bfloat16*>(a.y)[o + r] = __float2bfloat16_rn(v);
                    else reinterpret_cast<float*>(a.y)[o + r] = v;
                }
            }
    };
    R.run(a.w, 0.0f, reinterpret_cast<float4*>(smem + a.slots_at), runs, rows_of, [](int) {}, [](int) {}, mul, finish);
    if (a.splits == 1) return;
    cluster_sync();
    const uint32_t base = smem_u32(part);
    for (int i = threadIdx.x + rank * blockDim.x; i < a.m * rows; i += blockDim.x * a.splits) {
        const int tok = i / rows, r = i - tok * rows;
        float v = 0.0f;
        for (int s = 0; s < a.splits; ++s)
            v += ld_shared_cluster_f32(map_shared_rank(base + (tok * a.part_rows + r) * 4, static_cast<uint32_t>(s)));
        if (a.bf16_out) reinterpret_cast<__nv_bfloat16*>(a.y)[tok * a.w.n + row0 + r] = __float2bfloat16_rn(v);
        else reinterpret_cast<float*>(a.y)[tok * a.w.n + row0 + r] = v;
    }
    cluster_sync();  // no CTA leaves while another still reads its sums
}

}  // namespace int4

static const void* gemv_kernel(int64_t m, const Int4Args& w) {
    using namespace int4;
#define NF4_INT4_GEMV(F, Z) reinterpret_cast<const void*>(&k_int4_gemv<F, Z, 1>), reinterpret_cast<const void*>(&k_int4_gemv<F, Z, 2>)
    static const void* const fns[12] = {NF4_INT4_GEMV(few::kG128, false), NF4_INT4_GEMV(few::kG128, true),
                                        NF4_INT4_GEMV(few::kG64, false),  NF4_INT4_GEMV(few::kG64, true),
                                        NF4_INT4_GEMV(few::kG32, false),  NF4_INT4_GEMV(few::kG32, true)};
#undef NF4_INT4_GEMV
    return fns[(few::int4_format(w) - few::kG128) * 4 + (w.zero ? 2 : 0) + (m > 8 ? 1 : 0)];
}

static cudaError_t launch_int4_gemv_pass(const void* X, int64_t m, const Int4Args& w, void* Y, bool y_bf16, bool early, int widest,
                                         const DeviceInfo& dev, cudaStream_t stream) {
    using namespace int4;
    const void* fn = gemv_kernel(m, w);
    Pass p;
    const cudaError_t e = plan_pass(m, w, dev.sm_count, widest, [&](int splits, int* n) { return few::resident(fn, kWarps * 32, splits, dev, n); }, &p);
    if (e != cudaSuccess) return e;
    GemvArgs a = {};
    a.x = reinterpret_cast<const __nv_bfloat16*>(X);
    a.w = few::int4_weight(w);
    a.y = Y;
    a.m = static_cast<int>(m);
    while ((2 << a.x_lg) * m <= p.warps) ++a.x_lg;
    a.rows = few::shares_of(static_cast<int>(p.groups), static_cast<int>(p.clusters));
    a.ks = few::shares_of(static_cast<int>(p.steps), p.splits);
    a.splits = p.splits;
    a.x_stride = static_cast<int>(p.at.x_stride);
    a.ring_at = static_cast<int>(p.at.x);
    a.slots_at = static_cast<int>(p.at.x + p.at.ring);
    a.part_at = static_cast<int>(p.at.x + p.at.ring + p.at.slots);
    a.part_rows = static_cast<int>((p.groups + p.clusters - 1) / p.clusters * 8);
    a.bf16_out = y_bf16 ? 1 : 0;
    a.early = early ? 1 : 0;
    const size_t smem = static_cast<size_t>(a.part_at + (p.splits > 1 ? m * a.part_rows * 4 : 0));
    void* args[1] = {&a};
    return few::launch(fn, p.clusters * p.splits, p.warps * 32, smem, p.splits, stream, args);
}

static cudaError_t widest_of(int64_t m, const Int4Args& w, const DeviceInfo& dev, int* widest) {
    const void* fn = gemv_kernel(m, w);
    return int4::widest_cluster([&](int splits, int* n) { return few::resident(fn, int4::kWarps * 32, splits, dev, n); }, widest);
}

// A pass takes 7 us over 1024 x 4096, 9 over 4096 x 4096, 14 over 11008 x 4096, 42 over
// 28672 x 8192 and 14 over 512 x 65536: 6 us, 3.2 TB/s and X.  The GEMM (int4_gemm_us) takes 14 us
// over 4096 x 4096, 24 over 11008 x 4096 and 77 over 28672 x 8192 for any number of tokens up to 128.
bool int4_few_tokens(int64_t m, const Int4Args& w, bool y_bf16, const DeviceInfo& dev) {
    if (m <= kGemvMaxTokens) return true;
    const double k = static_cast<double>(w.k), pass = 6.0 + static_cast<double>(w.n) * k * 0.5 / 3.2e6 + k * 5e-5;
    int widest = 1;
    if (widest_of(m, w, dev, &widest) != cudaSuccess) return false;
    const int64_t most = int4::tokens_of_pass(m, w, widest);
    return static_cast<double>((m + most - 1) / most) * pass < int4_gemm_us(m, w.n, w.k, y_bf16, dev);
}

cudaError_t launch_int4_gemv(const void* X, int64_t m, const Int4Args& w, void* Y, bool y_bf16, bool early, const DeviceInfo& dev,
                             cudaStream_t stream) {
    int widest = 1;
    const cudaError_t found = widest_of(m, w, dev, &widest);
    if (found != cudaSuccess) return found;
    const int64_t most = int4::tokens_of_pass(m, w, widest);
    for (int64_t t = 0; t < m; t += most) {
        const cudaError_t e = launch_int4_gemv_pass(static_cast<const char*>(X) + t * w.k * 2, m - t < most ? m - t : most, w,
                                                    static_cast<char*>(Y) + t * w.n * (y_bf16 ? 2 : 4), y_bf16, early, widest, dev, stream);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace nf4
