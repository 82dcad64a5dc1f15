// nf4_api.cu -- the extern "C" entry points of libnf4.so (declared in include/nf4.h).
//
// Each entry point validates its arguments on the host, then enqueues kernels
// on the caller's stream.  Nothing is launched when validation fails, nothing
// is allocated, and the host is never synchronized.
#include <cstdint>
#include <cstring>
#include <mutex>

#include "nf4.h"
#include "nf4_internal.h"
#include "nf4_levels.h"

namespace nf4 {

cudaError_t current_device(DeviceInfo* out) {
    static std::mutex mu;
    static DeviceInfo cache[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(mu);
    if (cache[dev].device != dev) {
        DeviceInfo d;
        d.device = dev;
        if ((e = cudaDeviceGetAttribute(&d.sm_count, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
        if ((e = cudaDeviceGetAttribute(&d.major, cudaDevAttrComputeCapabilityMajor, dev)) != cudaSuccess) return e;
        if ((e = cudaDeviceGetAttribute(&d.minor, cudaDevAttrComputeCapabilityMinor, dev)) != cudaSuccess) return e;
        int optin = 0;
        if ((e = cudaDeviceGetAttribute(&optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev)) != cudaSuccess) return e;
        d.smem_optin = static_cast<size_t>(optin);
        cache[dev] = d;
    }
    *out = cache[dev];
    return cudaSuccess;
}

}  // namespace nf4

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Device check shared by every launching entry point.
nf4_status_t device_ok(nf4::DeviceInfo* dev) {
    if (nf4::current_device(dev) != cudaSuccess) {
        cudaGetLastError();
        return NF4_ERR_CUDA;
    }
    if (dev->major != 10) return NF4_ERR_UNSUPPORTED;
    return NF4_OK;
}

nf4_status_t from_cuda(cudaError_t e) { return e == cudaSuccess ? NF4_OK : NF4_ERR_CUDA; }

nf4_status_t check_weight(const nf4_weight_t* w) {
    if (!w) return NF4_ERR_NULL;
    if ((w->magic != NF4_WEIGHT_MAGIC && w->magic != NF4_FP4_WEIGHT_MAGIC) || w->version != NF4_WEIGHT_VERSION ||
        w->blocksize != NF4_BLOCKSIZE || w->blocksize2 != NF4_BLOCKSIZE2)
        return NF4_ERR_STATE;
    if (!w->wq || !w->absmax_q || !w->absmax_scale || !w->absmax_offset) return NF4_ERR_NULL;
    if (w->n <= 0 || w->k <= 0) return NF4_ERR_SHAPE;
    if (w->n > INT64_MAX / w->k) return NF4_ERR_SHAPE;
    if ((w->n * w->k) % NF4_BLOCKSIZE != 0) return NF4_ERR_SHAPE;
    if (!aligned(w->wq, 16) || !aligned(w->absmax_scale, 4) || !aligned(w->absmax_offset, 4))
        return NF4_ERR_ALIGN;
    return NF4_OK;
}

// The codebook a (checked) weight's codes index: its magic says NF4 or FP4.
int codebook_of(const nf4_weight_t* w) { return w->magic == NF4_FP4_WEIGHT_MAGIC ? 1 : 0; }

// Sizes of an integer 4-bit weight; k is limited by what a token slab of X takes on chip.
bool int4_shape_ok(int64_t n, int64_t k, int64_t group) {
    if (n <= 0 || n >= (int64_t{1} << 30) || k <= 0 || k > 65536 || k % 64 != 0) return false;
    return group > 0 && (group == 32 || group % 64 == 0) && k % group == 0;
}

nf4_status_t check_int4(const nf4_int4_weight_t* w, nf4::Int4Args* out) {
    if (!w) return NF4_ERR_NULL;
    if (w->magic != NF4_INT4_WEIGHT_MAGIC || w->version != NF4_WEIGHT_VERSION || w->reserved != 0 ||
        (w->scale_dtype != NF4_F32 && w->scale_dtype != NF4_BF16))
        return NF4_ERR_STATE;
    if (!w->wq || !w->scale) return NF4_ERR_NULL;
    if (!int4_shape_ok(w->n, w->k, w->group)) return NF4_ERR_SHAPE;
    if (!aligned(w->wq, 16) || !aligned(w->scale, w->scale_dtype == NF4_F32 ? 4 : 2)) return NF4_ERR_ALIGN;
    *out = nf4::Int4Args{w->n, w->k, w->group, w->wq, w->scale, w->zero, w->scale_dtype == NF4_F32};
    return NF4_OK;
}

// What both forms of the mixture-of-experts layer share once their weights are checked.
nf4_status_t run_moe(const void* X, int64_t m, const void* router, int32_t E, const nf4::MoeWeight& gate_up, int64_t gate_up_n,
                     const nf4::MoeWeight& down, int64_t down_n, int32_t top_k, void* Y, int32_t* ids, float* probs,
                     uint32_t flags, void* workspace, size_t ws_bytes, nf4_stream_t stream) {
    if (!X || !router || !Y) return NF4_ERR_NULL;
    if ((flags & ~NF4_MOE_RENORMALIZE) != 0) return NF4_ERR_DTYPE;
    const int64_t h = gate_up.k, f = down.k;
    if (m < 1 || m > INT32_MAX || nf4_moe_workspace_bytes(h, f, E, top_k) == 0) return NF4_ERR_SHAPE;
    if (gate_up_n != 2 * f * E || down_n != h * E) return NF4_ERR_SHAPE;
    if (!aligned(X, 16) || !aligned(router, 16) || !aligned(Y, 16) || (ids && !aligned(ids, 4)) || (probs && !aligned(probs, 4)))
        return NF4_ERR_ALIGN;
    if (!workspace || ws_bytes < nf4_moe_workspace_bytes(h, f, E, top_k)) return NF4_ERR_WORKSPACE;
    if (!aligned(workspace, 16)) return NF4_ERR_ALIGN;
    nf4::DeviceInfo dev;
    nf4_status_t st = device_ok(&dev);
    if (st != NF4_OK) return st;
    return from_cuda(nf4::launch_moe(X, m, router, E, gate_up, down, top_k, (flags & NF4_MOE_RENORMALIZE) != 0, Y, ids, probs,
                                     workspace, dev, reinterpret_cast<cudaStream_t>(stream)));
}

nf4::MoeWeight moe_weight(const nf4_weight_t* w) {
    nf4::MoeWeight o;
    o.k = w->k;
    o.wq = w->wq;
    o.absmax_q = w->absmax_q;
    o.absmax_scale = w->absmax_scale;
    o.absmax_offset = w->absmax_offset;
    o.codebook = codebook_of(w);
    return o;
}

}  // namespace

extern "C" {

int nf4_abi_version(void) { return NF4_ABI_VERSION; }

const char* nf4_status_str(int status) {
    switch (status) {
        case NF4_OK: return "NF4_OK";
        case NF4_ERR_NULL: return "NF4_ERR_NULL: a required pointer is NULL";
        case NF4_ERR_SHAPE: return "NF4_ERR_SHAPE: size out of range or not a multiple of the block size";
        case NF4_ERR_ALIGN: return "NF4_ERR_ALIGN: pointer not 16-byte aligned";
        case NF4_ERR_DTYPE: return "NF4_ERR_DTYPE: unsupported dtype";
        case NF4_ERR_STATE: return "NF4_ERR_STATE: bad nf4_weight_t magic, version or block size";
        case NF4_ERR_WORKSPACE: return "NF4_ERR_WORKSPACE: workspace missing or too small";
        case NF4_ERR_CUDA: return "NF4_ERR_CUDA: CUDA runtime error";
        case NF4_ERR_DEVICE_TIMEOUT: return "NF4_ERR_DEVICE_TIMEOUT: a bounded device wait ran out";
        case NF4_ERR_UNSUPPORTED: return "NF4_ERR_UNSUPPORTED: device is not compute capability 10.x";
        default: return "unknown nf4 status";
    }
}

nf4_status_t nf4_codebook(float* levels_out) { return nf4_codebook_typed(NF4_QUANT_NF4, levels_out); }

nf4_status_t nf4_codebook_typed(nf4_quant_type_t quant_type, float* levels_out) {
    if (!levels_out) return NF4_ERR_NULL;
    static const float nf4_levels[16] = NF4_LEVELS_INIT;
    static const float fp4_levels[16] = FP4_LEVELS_INIT;
    if (quant_type == NF4_QUANT_NF4)
        std::memcpy(levels_out, nf4_levels, sizeof nf4_levels);
    else if (quant_type == NF4_QUANT_FP4)
        std::memcpy(levels_out, fp4_levels, sizeof fp4_levels);
    else
        return NF4_ERR_DTYPE;
    return NF4_OK;
}

nf4_status_t nf4_quantize(const void* W, nf4_dtype_t w_dtype, int64_t n, int64_t k, uint8_t* wq,
                          float* absmax, nf4_stream_t stream) {
    return nf4_quantize_typed(W, w_dtype, n, k, NF4_QUANT_NF4, wq, absmax, stream);
}

nf4_status_t nf4_quantize_typed(const void* W, nf4_dtype_t w_dtype, int64_t n, int64_t k,
                                nf4_quant_type_t quant_type, uint8_t* wq, float* absmax, nf4_stream_t stream) {
    if (!W || !wq || !absmax) return NF4_ERR_NULL;
    if (quant_type != NF4_QUANT_NF4 && quant_type != NF4_QUANT_FP4) return NF4_ERR_DTYPE;
    if (w_dtype != NF4_F32 && w_dtype != NF4_BF16) return NF4_ERR_DTYPE;
    if (n <= 0 || k <= 0 || n > INT64_MAX / k || (n * k) % NF4_BLOCKSIZE != 0) return NF4_ERR_SHAPE;
    if (!aligned(W, 16) || !aligned(wq, 16) || !aligned(absmax, 4)) return NF4_ERR_ALIGN;
    nf4::DeviceInfo dev;
    nf4_status_t st = device_ok(&dev);
    if (st != NF4_OK) return st;
    return from_cuda(nf4::launch_quantize(W, w_dtype == NF4_BF16, n * k, wq, absmax,
                                          quant_type == NF4_QUANT_FP4 ? 1 : 0, dev,
                                          reinterpret_cast<cudaStream_t>(stream)));
}

size_t nf4_double_quant_workspace_bytes(int64_t nb) { return nf4::dq_workspace_bytes(nb); }

nf4_status_t nf4_double_quant(const float* absmax, int64_t nb, void* workspace,
                              size_t workspace_bytes, int8_t* absmax_q, float* absmax_scale,
                              float* absmax_offset, nf4_stream_t stream) {
    if (!absmax || !absmax_q || !absmax_scale || !absmax_offset) return NF4_ERR_NULL;
    if (nb <= 0 || nb > nf4::dq_max_nb()) return NF4_ERR_SHAPE;
    if (!workspace || workspace_bytes < nf4::dq_workspace_bytes(nb)) return NF4_ERR_WORKSPACE;
    if (!aligned(absmax, 4) || !aligned(absmax_scale, 4) || !aligned(absmax_offset, 4) ||
        !aligned(workspace, 8))
        return NF4_ERR_ALIGN;
    nf4::DeviceInfo dev;
    nf4_status_t st = device_ok(&dev);
    if (st != NF4_OK) return st;
    return from_cuda(nf4::launch_double_quant(absmax, nb, static_cast<double*>(workspace), absmax_q,
                                              absmax_scale, absmax_offset, dev,
                                              reinterpret_cast<cudaStream_t>(stream)));
}

nf4_status_t nf4_dequantize(const nf4_weight_t* w, void* out, nf4_dtype_t out_dtype,
                            nf4_stream_t stream) {
    nf4_status_t st = check_weight(w);
    if (st != NF4_OK) return st;
    if (!out) return NF4_ERR_NULL;
    if (out_dtype != NF4_F32 && out_dtype != NF4_BF16) return NF4_ERR_DTYPE;
    if (!aligned(out, 16)) return NF4_ERR_ALIGN;
    nf4::DeviceInfo dev;
    if ((st = device_ok(&dev)) != NF4_OK) return st;
    return from_cuda(nf4::launch_dequantize(w->wq, w->absmax_q, w->absmax_scale, w->absmax_offset,
                                            w->n * w->k, out, out_dtype == NF4_BF16, codebook_of(w), dev,
                                            reinterpret_cast<cudaStream_t>(stream)));
}

static_assert(NF4_DEQUANT_BATCH_MAX == nf4::kMaxDequantBatch, "batch bound of the header and the kernel agree");

nf4_status_t nf4_dequantize_batch(const nf4_weight_t* const* w, int32_t count, void* const* out,
                                  nf4_dtype_t out_dtype, nf4_stream_t stream) {
    if (!w || !out) return NF4_ERR_NULL;
    if (count < 1 || count > NF4_DEQUANT_BATCH_MAX) return NF4_ERR_SHAPE;
    if (out_dtype != NF4_F32 && out_dtype != NF4_BF16) return NF4_ERR_DTYPE;
    nf4::DequantItem items[NF4_DEQUANT_BATCH_MAX];
    for (int32_t i = 0; i < count; ++i) {
        if (!w[i] || !out[i]) return NF4_ERR_NULL;
        const nf4_status_t st = check_weight(w[i]);
        if (st != NF4_OK) return st;
        if (!aligned(out[i], 16)) return NF4_ERR_ALIGN;
        items[i] = {w[i]->wq, w[i]->absmax_q, w[i]->absmax_scale, w[i]->absmax_offset, w[i]->n * w[i]->k, out[i],
                    codebook_of(w[i])};
    }
    nf4::DeviceInfo dev;
    nf4_status_t st;
    if ((st = device_ok(&dev)) != NF4_OK) return st;
    return from_cuda(nf4::launch_dequantize_batch(items, count, out_dtype == NF4_BF16, dev,
                                                  reinterpret_cast<cudaStream_t>(stream)));
}

// LoRA workspace: t fp32 [m, r], then its bf16 halves t_hi, t_lo [m, r] (each
// region padded to 256 bytes), then for m > 16 the scratch of the tensor-core
// down-projection, then the split-k area of the decode path.
static size_t lora_t_region(int64_t m, int32_t r, size_t elem) {
    return (static_cast<size_t>(m) * static_cast<size_t>(r) * elem + 255) / 256 * 256;
}
static size_t lora_tc_region(int64_t m, int64_t k, int32_t r) {
    return m > nf4::kGemvMaxTokens ? (nf4::lora_tc_scratch_bytes(m, k, r) + 255) / 256 * 256 : 0;
}
static size_t lora_t_bytes(int64_t m, int64_t k, int32_t r) {
    return lora_t_region(m, r, sizeof(float)) + 2 * lora_t_region(m, r, 2) + lora_tc_region(m, k, r);
}

nf4_status_t nf4_linear_lora(const void* X, int64_t m, const nf4_weight_t* w, const void* lora_down,
                             const void* lora_up, int32_t r, float scale, void* Y, nf4_dtype_t y_dtype,
                             int32_t* dev_status, uint32_t flags, void* workspace, size_t ws_bytes,
                             nf4_stream_t stream) {
    nf4_status_t st = check_weight(w);
    if (st != NF4_OK) return st;
    if (!X || !Y || !lora_down || !lora_up || !workspace) return NF4_ERR_NULL;
    if (y_dtype != NF4_F32 && y_dtype != NF4_BF16) return NF4_ERR_DTYPE;
    if ((flags & ~static_cast<uint32_t>(NF4_LINEAR_WEIGHTS_EARLY)) != 0) return NF4_ERR_DTYPE;
    if (m < 1 || w->k % NF4_BLOCKSIZE != 0 || r < 1 || r > 256) return NF4_ERR_SHAPE;
    if (m > INT64_MAX / w->k || m > INT64_MAX / w->n || m > INT64_MAX / 1024) return NF4_ERR_SHAPE;
    if (!aligned(X, 16) || !aligned(Y, 16) || !aligned(lora_down, 16) || !aligned(lora_up, 16) ||
        !aligned(workspace, 16) || (dev_status && !aligned(dev_status, 4)))
        return NF4_ERR_ALIGN;
    nf4::DeviceInfo dev;
    if ((st = device_ok(&dev)) != NF4_OK) return st;
    const size_t tb = lora_t_bytes(m, w->k, r);
    if (ws_bytes < tb + nf4::linear_workspace_bytes(m, w->n, w->k, dev)) return NF4_ERR_WORKSPACE;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    nf4::LoraArgs lora;
    lora.up = static_cast<const __nv_bfloat16*>(lora_up);
    lora.r = r;
    if (nf4::gemv_fuses_lora(m, w->n, w->k, r, true, dev)) {
        // decode with r = 8 or 16: the dequant-GEMV forms t itself
        lora.down = static_cast<const __nv_bfloat16*>(lora_down);
        lora.scale = scale;
    } else {
        float* t = static_cast<float*>(workspace);
        __nv_bfloat16* t_hi = reinterpret_cast<__nv_bfloat16*>(static_cast<char*>(workspace) + lora_t_region(m, r, 4));
        __nv_bfloat16* t_lo = reinterpret_cast<__nv_bfloat16*>(reinterpret_cast<char*>(t_hi) + lora_t_region(m, r, 2));
        const bool early = (flags & NF4_LINEAR_WEIGHTS_EARLY) != 0;
        if (m > nf4::kGemvMaxTokens) {
            void* scratch = lora_tc_region(m, w->k, r) ? reinterpret_cast<char*>(t_lo) + lora_t_region(m, r, 2) : nullptr;
            st = from_cuda(nf4::launch_lora_down_tc(X, m, w->k, lora_down, r, scale, t, t_hi, t_lo, scratch, early,
                                                    dev, s));
        } else {
            st = from_cuda(nf4::launch_lora_down(X, m, w->k, lora_down, r, scale, t, t_hi, t_lo, early, s));
        }
        if (st != NF4_OK) return st;
        lora.t = t;
        lora.t_hi = t_hi;
        lora.t_lo = t_lo;
    }
    return from_cuda(nf4::launch_linear(X, m, w->wq, w->absmax_q, w->absmax_scale, w->absmax_offset, w->n, w->k,
                                        Y, y_dtype == NF4_BF16, dev_status, (flags & NF4_LINEAR_WEIGHTS_EARLY) != 0,
                                        static_cast<char*>(workspace) + tb, lora, codebook_of(w), dev, s));
}

nf4_status_t nf4_merge_lora(const nf4_weight_t* w, const void* lora_down, const void* lora_up, int32_t r,
                            float scale, void* w_new, uint8_t* wq_out, float* absmax_out,
                            nf4_stream_t stream) {
    nf4_status_t st = check_weight(w);
    if (st != NF4_OK) return st;
    if (!lora_down || !lora_up || !wq_out || !absmax_out) return NF4_ERR_NULL;
    if (w->k % NF4_BLOCKSIZE != 0 || r < 1 || r > 256) return NF4_ERR_SHAPE;
    if (!aligned(lora_down, 16) || !aligned(lora_up, 16) || !aligned(wq_out, 16) || !aligned(absmax_out, 4) ||
        (w_new && !aligned(w_new, 16)))
        return NF4_ERR_ALIGN;
    nf4::DeviceInfo dev;
    if ((st = device_ok(&dev)) != NF4_OK) return st;
    return from_cuda(nf4::launch_merge_lora(w->wq, w->absmax_q, w->absmax_scale, w->absmax_offset, w->n, w->k,
                                            lora_down, lora_up, r, scale, w_new, wq_out, absmax_out,
                                            codebook_of(w), dev,
                                            reinterpret_cast<cudaStream_t>(stream)));
}

size_t nf4_linear_lora_workspace_bytes(int64_t m, int64_t n, int64_t k, int32_t r) {
    if (m < 1 || n < 1 || k < 1 || k % NF4_BLOCKSIZE != 0 || r < 1 || r > 256) return 0;
    nf4::DeviceInfo dev;
    if (device_ok(&dev) != NF4_OK) return 0;
    return lora_t_bytes(m, k, r) + nf4::linear_workspace_bytes(m, n, k, dev);
}

nf4_status_t nf4_linear_group(const void* X, int64_t m, const nf4_weight_t* const* w, int32_t count,
                              void* const* Y, nf4_dtype_t y_dtype, int32_t* dev_status, uint32_t flags,
                              void* workspace, size_t ws_bytes, nf4_stream_t stream) {
    if (!X || !w || !Y) return NF4_ERR_NULL;
    if (count < 1 || count > nf4::kMaxGroup) return NF4_ERR_SHAPE;
    nf4_status_t st;
    for (int32_t i = 0; i < count; ++i) {
        if ((st = check_weight(w[i])) != NF4_OK) return st;
        if (!Y[i]) return NF4_ERR_NULL;
        if (w[i]->k != w[0]->k) return NF4_ERR_SHAPE;
        if (w[i]->magic != w[0]->magic) return NF4_ERR_STATE;
        if (m >= 1 && m > INT64_MAX / w[i]->n) return NF4_ERR_SHAPE;
        if (!aligned(Y[i], 16)) return NF4_ERR_ALIGN;
    }
    const int64_t k = w[0]->k;
    if (y_dtype != NF4_F32 && y_dtype != NF4_BF16) return NF4_ERR_DTYPE;
    if ((flags & ~static_cast<uint32_t>(NF4_LINEAR_WEIGHTS_EARLY | NF4_LINEAR_TEST_TIMEOUT)) != 0)
        return NF4_ERR_DTYPE;
    if (m < 1 || k % NF4_BLOCKSIZE != 0 || m > INT64_MAX / k) return NF4_ERR_SHAPE;
    if (!aligned(X, 16) || (dev_status && !aligned(dev_status, 4))) return NF4_ERR_ALIGN;
    if (workspace && !aligned(workspace, 16)) return NF4_ERR_ALIGN;
    nf4::DeviceInfo dev;
    if ((st = device_ok(&dev)) != NF4_OK) return st;
    nf4::LinearWeight lw[nf4::kMaxGroup];
    for (int32_t i = 0; i < count; ++i) {
        if (workspace && ws_bytes < nf4::linear_workspace_bytes(m, w[i]->n, k, dev)) return NF4_ERR_WORKSPACE;
        lw[i].wq = w[i]->wq;
        lw[i].absmax_q = w[i]->absmax_q;
        lw[i].absmax_scale = w[i]->absmax_scale;
        lw[i].absmax_offset = w[i]->absmax_offset;
        lw[i].n = w[i]->n;
        lw[i].y = Y[i];
    }
    const uint32_t test = (flags & NF4_LINEAR_TEST_TIMEOUT) ? nf4::kTestStall : 0u;
    return from_cuda(nf4::launch_linear_group(X, m, k, lw, count, y_dtype == NF4_BF16, dev_status,
                                              (flags & NF4_LINEAR_WEIGHTS_EARLY) != 0, workspace, nf4::LoraArgs(),
                                              codebook_of(w[0]), test, dev, reinterpret_cast<cudaStream_t>(stream)));
}

int32_t nf4_linear_group_launches(int64_t m, const int64_t* n, int32_t count, int64_t k) {
    if (!n || count < 1 || count > nf4::kMaxGroup || m < 1 || k < 1 || k % NF4_BLOCKSIZE != 0) return -1;
    for (int32_t i = 0; i < count; ++i)
        if (n[i] < 1) return -1;
    nf4::DeviceInfo dev;
    if (device_ok(&dev) != NF4_OK) return -1;
    return nf4::group_in_one_launch(m, n, count, k, false, dev) ? 1 : count;
}

nf4_status_t nf4_linear_ws(const void* X, int64_t m, const nf4_weight_t* w, void* Y,
                           nf4_dtype_t y_dtype, int32_t* dev_status, uint32_t flags, void* workspace,
                           size_t ws_bytes, nf4_stream_t stream) {
    if (!w) return NF4_ERR_NULL;
    return nf4_linear_group(X, m, &w, 1, &Y, y_dtype, dev_status, flags, workspace, ws_bytes, stream);
}

nf4_status_t nf4_linear_ex(const void* X, int64_t m, const nf4_weight_t* w, void* Y,
                           nf4_dtype_t y_dtype, int32_t* dev_status, uint32_t flags, nf4_stream_t stream) {
    return nf4_linear_ws(X, m, w, Y, y_dtype, dev_status, flags, nullptr, 0, stream);
}

nf4_status_t nf4_linear_dx(const void* dY, int64_t m, const nf4_weight_t* w, void* dX,
                           nf4_dtype_t dx_dtype, int32_t* dev_status, nf4_stream_t stream) {
    nf4_status_t st = check_weight(w);
    if (st != NF4_OK) return st;
    if (!dY || !dX) return NF4_ERR_NULL;
    if (dx_dtype != NF4_F32 && dx_dtype != NF4_BF16) return NF4_ERR_DTYPE;
    if (m < 1 || w->k % NF4_BLOCKSIZE != 0 || w->n % 8 != 0) return NF4_ERR_SHAPE;
    if (m > INT64_MAX / w->k || m > INT64_MAX / w->n) return NF4_ERR_SHAPE;
    if (!aligned(dY, 16) || !aligned(dX, 16) || (dev_status && !aligned(dev_status, 4))) return NF4_ERR_ALIGN;
    nf4::DeviceInfo dev;
    if ((st = device_ok(&dev)) != NF4_OK) return st;
    return from_cuda(nf4::launch_gemm_dx(dY, m, w->wq, w->absmax_q, w->absmax_scale, w->absmax_offset, w->n,
                                         w->k, dX, dx_dtype == NF4_BF16, dev_status, codebook_of(w), dev,
                                         reinterpret_cast<cudaStream_t>(stream)));
}

size_t nf4_linear_workspace_bytes(int64_t m, int64_t n, int64_t k) {
    if (m < 1 || n < 1 || k < 1 || k % NF4_BLOCKSIZE != 0) return 0;
    nf4::DeviceInfo dev;
    if (device_ok(&dev) != NF4_OK) return 0;
    return nf4::linear_workspace_bytes(m, n, k, dev);
}

nf4_status_t nf4_linear(const void* X, int64_t m, const nf4_weight_t* w, void* Y,
                        nf4_dtype_t y_dtype, int32_t* dev_status, nf4_stream_t stream) {
    return nf4_linear_ex(X, m, w, Y, y_dtype, dev_status, 0u, stream);
}

nf4_status_t nf4_int4_quantize(const void* W, nf4_dtype_t w_dtype, int64_t n, int64_t k, int64_t group,
                               nf4_dtype_t scale_dtype, uint8_t* wq, void* scale, uint8_t* zero,
                               nf4_stream_t stream) {
    if (!W || !wq || !scale) return NF4_ERR_NULL;
    if ((w_dtype != NF4_F32 && w_dtype != NF4_BF16) || (scale_dtype != NF4_F32 && scale_dtype != NF4_BF16))
        return NF4_ERR_DTYPE;
    if (!int4_shape_ok(n, k, group)) return NF4_ERR_SHAPE;
    if (!aligned(W, 16) || !aligned(wq, 16) || !aligned(scale, scale_dtype == NF4_F32 ? 4 : 2)) return NF4_ERR_ALIGN;
    nf4::DeviceInfo dev;
    nf4_status_t st = device_ok(&dev);
    if (st != NF4_OK) return st;
    return from_cuda(nf4::launch_int4_quantize(W, w_dtype == NF4_BF16, n, k, group, wq, scale, scale_dtype == NF4_F32, zero,
                                               dev, reinterpret_cast<cudaStream_t>(stream)));
}

nf4_status_t nf4_int4_dequantize(const nf4_int4_weight_t* w, void* out, nf4_dtype_t out_dtype, nf4_stream_t stream) {
    nf4::Int4Args a;
    nf4_status_t st = check_int4(w, &a);
    if (st != NF4_OK) return st;
    if (!out) return NF4_ERR_NULL;
    if (out_dtype != NF4_F32 && out_dtype != NF4_BF16) return NF4_ERR_DTYPE;
    if (!aligned(out, 16)) return NF4_ERR_ALIGN;
    nf4::DeviceInfo dev;
    if ((st = device_ok(&dev)) != NF4_OK) return st;
    return from_cuda(nf4::launch_int4_dequantize(a, out, out_dtype == NF4_BF16, dev, reinterpret_cast<cudaStream_t>(stream)));
}

nf4_status_t nf4_int4_linear(const void* X, int64_t m, const nf4_int4_weight_t* w, void* Y, nf4_dtype_t y_dtype,
                             int32_t* dev_status, uint32_t flags, nf4_stream_t stream) {
    nf4::Int4Args a;
    nf4_status_t st = check_int4(w, &a);
    if (st != NF4_OK) return st;
    if (!X || !Y) return NF4_ERR_NULL;
    if (y_dtype != NF4_F32 && y_dtype != NF4_BF16) return NF4_ERR_DTYPE;
    // the few-token kernel has no bounded waits to test: the flag asks for the GEMM
    const bool test = (flags & NF4_LINEAR_TEST_TIMEOUT) != 0;
    if ((flags & ~static_cast<uint32_t>(NF4_LINEAR_WEIGHTS_EARLY | NF4_LINEAR_TEST_TIMEOUT)) != 0 || (test && m <= nf4::kGemvMaxTokens))
        return NF4_ERR_DTYPE;
    if (m < 1 || m > INT32_MAX / 2) return NF4_ERR_SHAPE;
    if (!aligned(X, 16) || !aligned(Y, 16) || (dev_status && !aligned(dev_status, 4))) return NF4_ERR_ALIGN;
    nf4::DeviceInfo dev;
    if ((st = device_ok(&dev)) != NF4_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (!test && nf4::int4_few_tokens(m, a, y_dtype == NF4_BF16, dev))
        return from_cuda(nf4::launch_int4_gemv(X, m, a, Y, y_dtype == NF4_BF16, (flags & NF4_LINEAR_WEIGHTS_EARLY) != 0, dev, s));
    return from_cuda(nf4::launch_gemm(X, m, a.wq, nullptr, nullptr, nullptr, a.n, a.k, Y, y_dtype == NF4_BF16, dev_status,
                                      nf4::LoraArgs(), 0, test ? nf4::kTestStall : 0u, dev, s, &a));
}

size_t nf4_moe_workspace_bytes(int64_t h, int64_t f, int32_t n_experts, int32_t top_k) {
    if (h < 64 || f < 64 || h % 64 != 0 || f % 64 != 0 || h > 65536 || f > 65536) return 0;
    if (n_experts < 1 || n_experts > NF4_MOE_MAX_EXPERTS || top_k < 1 || top_k > NF4_MOE_MAX_TOP_K || top_k > n_experts) return 0;
    return nf4::moe_workspace_bytes(h, f, n_experts, top_k);
}

nf4_status_t nf4_moe(const void* X, int64_t m, const void* router, int32_t n_experts, const nf4_weight_t* gate_up,
                     const nf4_weight_t* down, int32_t top_k, void* Y, int32_t* topk_ids, float* topk_probs, uint32_t flags,
                     void* workspace, size_t ws_bytes, nf4_stream_t stream) {
    nf4_status_t st = check_weight(gate_up);
    if (st == NF4_OK) st = check_weight(down);
    if (st != NF4_OK) return st;
    return run_moe(X, m, router, n_experts, moe_weight(gate_up), gate_up->n, moe_weight(down), down->n, top_k, Y, topk_ids,
                   topk_probs, flags, workspace, ws_bytes, stream);
}

nf4_status_t nf4_int4_moe(const void* X, int64_t m, const void* router, int32_t n_experts, const nf4_int4_weight_t* gate_up,
                          const nf4_int4_weight_t* down, int32_t top_k, void* Y, int32_t* topk_ids, float* topk_probs,
                          uint32_t flags, void* workspace, size_t ws_bytes, nf4_stream_t stream) {
    nf4::MoeWeight gu, dn;
    nf4_status_t st = check_int4(gate_up, &gu.int4);
    if (st == NF4_OK) st = check_int4(down, &dn.int4);
    if (st != NF4_OK) return st;
    gu.integer = dn.integer = true;
    gu.k = gate_up->k;
    dn.k = down->k;
    return run_moe(X, m, router, n_experts, gu, gate_up->n, dn, down->n, top_k, Y, topk_ids, topk_probs, flags, workspace, ws_bytes,
                   stream);
}

}  // extern "C"
