// nf4_int4_gemv.cu -- Y[t, r] = sum_c X[t, c] (q[r, c] - z) s for few tokens (m <= 16),
// integer 4-bit weights with group scales (sm_100a).
//
// Bound by HBM: half a byte of code per weight.  The tensor cores (mma.sync: sixteen
// tokens are too few for a 128-row tcgen05 tile, and the codes would have to pass
// through shared or tensor memory on the way) multiply the exact integers q - z by X in
// bf16; the scale goes onto the fp32 sum of each 64-k item (nf4_few.cuh), so nothing is
// rounded between the codes and the fp32 sums.
//
// A CTA has 16 RT rows of W and, with a cluster of S CTAs, a range of k; its eight
// warps split that range.  Codes go from global memory to registers, kDepth items
// ahead; X comes through L1.  The warps' sums meet in shared memory and the CTAs' in
// distributed shared memory, both added in rank order: results do not depend on timing.
#include "nf4_few.cuh"
#include "nf4_internal.h"
#include "nf4_ptx.cuh"

namespace nf4 {
namespace int4 {

constexpr int kWarps = 8;

template <bool kG32>
struct Raw {  // what one item of one 16-row tile brings from memory for a lane
    uint2 a, b;  // codes of rows g and g + 8
    uint32_t sa[kG32 ? 2 : 1], sb[kG32 ? 2 : 1], za[kG32 ? 2 : 1], zb[kG32 ? 2 : 1];
};

template <int NT, int RT, bool kG32>
__global__ void __launch_bounds__(kWarps * 32, 2)
k_int4_gemv(const __nv_bfloat16* __restrict__ X, int m, const uint8_t* __restrict__ wq, const few::Int4Sides sides, int64_t n,
            int64_t k, void* __restrict__ Y, bool bf16_out, int splits, int early) {
    constexpr int kDepth = RT >= 4 ? 2 : (RT == 2 ? 3 : 6);
    constexpr int kRows = 16 * RT, kLd = kRows + 4, kTok = 8 * NT;
    __shared__ float red[kWarps][kTok][kLd];
    __shared__ float part[kTok][kLd];

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int rank = splits > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int64_t row0 = static_cast<int64_t>(blockIdx.x / splits) * kRows;
    const int items = static_cast<int>(k / few::kItemK);
    const int c0 = static_cast<int>(static_cast<int64_t>(items) * rank / splits);
    const int c1 = static_cast<int>(static_cast<int64_t>(items) * (rank + 1) / splits);
    const int b0 = c0 + (c1 - c0) * warp / kWarps, b1 = c0 + (c1 - c0) * (warp + 1) / kWarps;

    // byte offset of a lane's codes in a row, and its k, within an item: sixteen k in a
    // run, or with groups of 32 eight of each group
    const int coff = kG32 ? 4 * t : 8 * t;
    const uint8_t* pw[RT][2];
    int64_t rr[RT][2];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int64_t row = row0 + 16 * r + 8 * i + g;
            rr[r][i] = row < n ? row : n - 1;  // rows past n: computed, never stored
            pw[r][i] = wq + rr[r][i] * (k / 2) + coff;
        }
    auto fetch = [&](Raw<kG32>(&raw)[RT], int b) {
        const int64_t off = static_cast<int64_t>(b) * 32;
        const int64_t gb = kG32 ? 2 * static_cast<int64_t>(b) : few::group_of(sides, static_cast<uint32_t>(b));
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            if (kG32) {
                raw[r].a = make_uint2(few::ldg_code32(pw[r][0] + off), few::ldg_code32(pw[r][0] + off + 16));
                raw[r].b = make_uint2(few::ldg_code32(pw[r][1] + off), few::ldg_code32(pw[r][1] + off + 16));
            } else {
                raw[r].a = few::ldg_codes(pw[r][0] + off);
                raw[r].b = few::ldg_codes(pw[r][1] + off);
            }
#pragma unroll
            for (int h = 0; h < (kG32 ? 2 : 1); ++h) {
                raw[r].sa[h] = few::ldg_scale(sides, (gb + h) * n + rr[r][0]);
                raw[r].sb[h] = few::ldg_scale(sides, (gb + h) * n + rr[r][1]);
                raw[r].za[h] = few::ldg_zero(sides, (gb + h) * n + rr[r][0]);
                raw[r].zb[h] = few::ldg_zero(sides, (gb + h) * n + rr[r][1]);
            }
        }
    };
    float acc[RT][NT][4] = {};
    auto consume = [&](const Raw<kG32>(&raw)[RT], int b) {
        uint32_t x[NT][8];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int tok = nt * 8 + g;
            uint4 u = make_uint4(0, 0, 0, 0), v = u;
            if (tok < m) {
                const __nv_bfloat16* xp = X + static_cast<int64_t>(tok) * k + static_cast<int64_t>(b) * few::kItemK + 2 * coff;
                u = __ldg(reinterpret_cast<const uint4*>(xp));
                v = __ldg(reinterpret_cast<const uint4*>(xp + (kG32 ? 32 : 8)));
            }
            few::pair_x(u.x, u.y, u.z, u.w, *reinterpret_cast<uint32_t(*)[4]>(&x[nt][0]));
            few::pair_x(v.x, v.y, v.z, v.w, *reinterpret_cast<uint32_t(*)[4]>(&x[nt][4]));
        }
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            float p[NT][4] = {};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int s = kG32 ? h : 0;
                uint32_t wa[4], wb[4];
                few::int4_bf16(h ? raw[r].a.y : raw[r].a.x, few::zoff_bf16(raw[r].za[s]), wa);
                few::int4_bf16(h ? raw[r].b.y : raw[r].b.x, few::zoff_bf16(raw[r].zb[s]), wb);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    few::mma_bf16(p[nt], wa[0], wb[0], wa[1], wb[1], x[nt][4 * h], x[nt][4 * h + 1]);
                    few::mma_bf16(p[nt], wa[2], wb[2], wa[3], wb[3], x[nt][4 * h + 2], x[nt][4 * h + 3]);
                }
                if (kG32 || h == 1) {
                    const float fa = __uint_as_float(raw[r].sa[s]), fb = __uint_as_float(raw[r].sb[s]);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        acc[r][nt][0] = __fmaf_rn(fa, p[nt][0], acc[r][nt][0]);
                        acc[r][nt][1] = __fmaf_rn(fa, p[nt][1], acc[r][nt][1]);
                        acc[r][nt][2] = __fmaf_rn(fb, p[nt][2], acc[r][nt][2]);
                        acc[r][nt][3] = __fmaf_rn(fb, p[nt][3], acc[r][nt][3]);
                        p[nt][0] = p[nt][1] = p[nt][2] = p[nt][3] = 0.0f;
                    }
                }
            }
        }
    };

    Raw<kG32> ring[kDepth][RT];
    if (!early) grid_dependency_wait();
#pragma unroll
    for (int d = 0; d < kDepth; ++d)
        if (b0 + d < b1) fetch(ring[d], b0 + d);
    if (early) grid_dependency_wait();
    grid_launch_dependents();
    for (int b = b0; b < b1; b += kDepth) {
#pragma unroll
        for (int d = 0; d < kDepth; ++d) {
            if (b + d >= b1) break;
            consume(ring[d], b + d);
            if (b + d + kDepth < b1) fetch(ring[d], b + d + kDepth);
        }
    }

#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float* p0 = &red[warp][nt * 8 + 2 * t][16 * r + g];
            p0[0] = acc[r][nt][0];
            p0[kLd] = acc[r][nt][1];
            p0[8] = acc[r][nt][2];
            p0[kLd + 8] = acc[r][nt][3];
        }
    __syncthreads();
    auto store = [&](int tok, int r, float v) {
        const int64_t row = row0 + r;
        if (tok >= m || row >= n) return;
        if (bf16_out) reinterpret_cast<__nv_bfloat16*>(Y)[tok * n + row] = __float2bfloat16_rn(v);
        else reinterpret_cast<float*>(Y)[tok * n + row] = v;
    };
    for (int i = threadIdx.x; i < kTok * kRows; i += kWarps * 32) {
        const int tok = i / kRows, r = i % kRows;
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) v += red[w][tok][r];
        if (splits == 1) store(tok, r, v);
        else part[tok][r] = v;
    }
    if (splits == 1) return;
    cluster_sync();
    const uint32_t base = smem_u32(&part[0][0]);
    for (int i = threadIdx.x + rank * kWarps * 32; i < kTok * kRows; i += kWarps * 32 * splits) {
        const int tok = i / kRows, r = i % kRows;
        float v = 0.0f;
        for (int s = 0; s < splits; ++s)
            v += ld_shared_cluster_f32(map_shared_rank(base + (tok * kLd + r) * 4, static_cast<uint32_t>(s)));
        store(tok, r, v);
    }
    cluster_sync();  // no CTA leaves while another still reads its sums
}

}  // namespace int4

cudaError_t launch_int4_gemv(const void* X, int64_t m, const Int4Args& w, void* Y, bool y_bf16, bool early, const DeviceInfo& dev,
                             cudaStream_t stream) {
    const int nt = m > 8 ? 2 : 1;
    const bool g32 = w.group == 32;
    int rt = m > 4 ? 2 : 1;
    const int64_t tiles = (w.n + 16 * rt - 1) / (16 * rt);
    const int64_t items = w.k / few::kItemK;
    int splits = 1;
    while (splits < 8 && tiles * splits < dev.sm_count * 2 && items / (splits * 2) >= int4::kWarps * 2) splits *= 2;
    if (tiles * splits > 0x7fffffff) return cudaErrorInvalidConfiguration;
    few::Int4Sides s{w.scale, w.zero, w.n, few::items_magic(w.group / few::kItemK), w.scale_f32 ? 1 : 0};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(tiles * splits));
    cfg.blockDim = dim3(int4::kWarps * 32);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(splits);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = splits > 1 ? 2 : 1;
#define NF4_INT4_GEMV(NT, RT, G32)                                                                                             \
    cudaLaunchKernelEx(&cfg, int4::k_int4_gemv<NT, RT, G32>, reinterpret_cast<const __nv_bfloat16*>(X), static_cast<int>(m),    \
                       w.wq, s, w.n, w.k, Y, y_bf16, splits, early ? 1 : 0)
#define NF4_INT4_GEMV_RT(NT, RT) (g32 ? NF4_INT4_GEMV(NT, RT, true) : NF4_INT4_GEMV(NT, RT, false))
    if (nt == 1) return rt == 1 ? NF4_INT4_GEMV_RT(1, 1) : NF4_INT4_GEMV_RT(1, 2);
    return rt == 1 ? NF4_INT4_GEMV_RT(2, 1) : NF4_INT4_GEMV_RT(2, 2);
#undef NF4_INT4_GEMV
#undef NF4_INT4_GEMV_RT
}

}  // namespace nf4
