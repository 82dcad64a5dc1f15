// nf4_few_host.h -- host side that the few-token kernels share (nf4_few.cuh).
#pragma once

#include "nf4_few.cuh"
#include "nf4_internal.h"

namespace nf4 {
namespace few {

constexpr int kMaxSmem = 216 * 1024;  // dynamic shared memory these kernels may ask for (beside some KB of static)

// Clusters of `splits` (1, 2, 4, 8) CTAs, one CTA an SM, that the current device runs at
// the same time, 0 where it runs none of that size (a part of a GPU may have too few SMs
// together); also allows the kernel its dynamic shared memory.  Asked of the runtime
// once per kernel, device and size.
cudaError_t resident(const void* fn, int threads, int splits, const DeviceInfo& dev, int* out);

inline Weight int4_weight(const Int4Args& w) {
    Weight o = {};
    o.wq = w.wq;
    o.n = w.n;
    o.k = static_cast<int>(w.k);
    o.scale = w.scale;
    o.zero = w.zero;
    o.scale_row = static_cast<uint32_t>(w.n * (w.scale_f32 ? 4 : 2));
    o.units = static_cast<int>(w.group == 32 ? w.k / 32 : (w.group % kStepK == 0 ? w.k / kStepK : w.k / kItemK));
    o.per = static_cast<int>(w.group % kStepK == 0 ? w.group / kStepK : w.group / kItemK);
    o.f32 = w.scale_f32 ? 1 : 0;
    return o;
}
inline Fmt int4_format(const Int4Args& w) { return w.group == 32 ? kG32 : (w.group % kStepK == 0 ? kG128 : kG64); }

// A launch as a programmatic dependent of the preceding kernel, in clusters of `splits`.
inline cudaError_t launch(const void* fn, int64_t grid, int threads, size_t smem, int splits, cudaStream_t stream, void** args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(splits);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = splits > 1 ? 2 : 1;
    return cudaLaunchKernelExC(&cfg, fn, args);
}

}  // namespace few
}  // namespace nf4
