// api.cu -- the extern "C" entry points of libmnb: host-side argument checks,
// then the launchers of the kernel files.  Nothing here touches the device
// before every check has passed.
#include <stdarg.h>
#include <stdio.h>

#include <initializer_list>
#include <mutex>

#include "common.cuh"
#include "internal.h"
#include "raise_limit.h"

namespace mnb {

static thread_local char g_msg[512] = "";

int fail(int code, const char *fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_msg, sizeof(g_msg), fmt, ap);
    va_end(ap);
    return code;
}

void clear_error() { g_msg[0] = 0; }

int check_launch(const char *what) {
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess)
        return fail(MNB_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
    return MNB_OK;
}

EncodeTiledFn tensor_map_encoder() {
    static std::once_flag once;
    static EncodeTiledFn fn = nullptr;
    std::call_once(once, [] {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(ptr);
    });
    return fn;
}

int device_sm_count() {
    static int counts[128] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 128)
        return 148;
    if (counts[dev] <= 0) {
        int n = 0;
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
            n = 148;
        counts[dev] = n;
    }
    return counts[dev];
}

cudaError_t ensure_dynamic_smem(const void *kernel, int bytes, int *cache) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    if (dev < 0 || dev >= kMaxDevices)
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    return (cudaError_t)raise_limit(&cache[dev], bytes, [&](int n) {
        return (int)cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, n);
    });
}

// Limits: sizes fit comfortably in 32-bit element indices of one row and in
// 64-bit byte offsets overall.
static const int64_t kMaxDim = (int64_t)1 << 30;

static int check_weight_shape(const char *fn, int64_t N, int64_t K, int bs) {
    if (N < 0 || K < 0)
        return fail(MNB_ERR_INVALID_ARG, "%s: negative size (N=%lld K=%lld)", fn, (long long)N,
                    (long long)K);
    if (bs != 32 && bs != 64)
        return fail(MNB_ERR_SHAPE, "%s: block size %d not in {32, 64}", fn, bs);
    if (K == 0 || K % bs != 0)
        return fail(MNB_ERR_SHAPE, "%s: K=%lld is not a positive multiple of bs=%d", fn,
                    (long long)K, bs);
    if (N > kMaxDim || K > kMaxDim)
        return fail(MNB_ERR_SHAPE, "%s: N or K above 2^30", fn);
    return MNB_OK;
}

static int check_dtype(const char *fn, const char *what, int t) {
    if (t != MNB_F32 && t != MNB_F16)
        return fail(MNB_ERR_INVALID_ARG, "%s: unknown %s dtype %d", fn, what, t);
    return MNB_OK;
}

static int check_matmul_args(const char *fn, const void *X, int act_t, const uint8_t *packed,
                             const void *scales, int scale_t, void *Y, int64_t M, int64_t N,
                             int64_t K, int bs) {
    int rc;
    if ((rc = check_dtype(fn, "activation", act_t)) || (rc = check_dtype(fn, "scale", scale_t)))
        return rc;
    if ((rc = check_weight_shape(fn, N, K, bs)))
        return rc;
    if (M < 0)
        return fail(MNB_ERR_INVALID_ARG, "%s: negative M", fn);
    if (M > kMaxDim)
        return fail(MNB_ERR_SHAPE, "%s: M above 2^30", fn);
    if (M > 0 && N > 0 && (!X || !packed || !scales || !Y))
        return fail(MNB_ERR_INVALID_ARG, "%s: NULL X, packed, scales or Y", fn);
    if (!aligned(X, 16) || !aligned(packed, 16) || !aligned(Y, 16))
        return fail(MNB_ERR_ALIGN, "%s: X, packed and Y must be 16-byte aligned", fn);
    if (!aligned(scales, scale_t == MNB_F32 ? 4 : 2))
        return fail(MNB_ERR_ALIGN, "%s: scales misaligned", fn);
    return MNB_OK;
}

// Limits of the paged cache: slots and positions are int32 and so is the end of
// the tile that holds the last one, the request scans are one CTA's, and
// page * stride stays far below 2^63.
static const int64_t kMaxSlots = ((int64_t)1 << 31) - 64, kMaxRequests = 4096, kMaxHeads = 4096;
static const int64_t kMaxStride = (int64_t)1 << 31;

static int check_stride(const char *fn, int64_t stride, int dtype) {
    const int64_t unit = dtype == MNB_F16 ? 8 : 4;
    if (stride < 0 || stride > kMaxStride)
        return fail(MNB_ERR_SHAPE, "%s: stride %lld outside [0, 2^31]", fn, (long long)stride);
    if (stride % unit)
        return fail(MNB_ERR_ALIGN, "%s: stride %lld is not a multiple of 16 bytes", fn, (long long)stride);
    return MNB_OK;
}

// Checks *given and copies it to *c, the strides of single extents as 0.
static int check_paged_cache(const char *fn, const mnb_paged_cache *given, mnb_paged_cache *c) {
    int rc;
    *c = *given;
    if (c->num_pages == 1)
        c->page_stride = 0;
    if (c->page_size == 1)
        c->slot_stride = 0;
    if (c->num_heads == 1)
        c->head_stride = 0;
    if (!c->k || !c->v)
        return fail(MNB_ERR_INVALID_ARG, "%s: NULL cache", fn);
    if ((rc = check_dtype(fn, "cache", c->dtype)))
        return rc;
    if (c->page_size < 1 || c->num_pages < 1 || c->page_size > kMaxSlots || c->num_pages > kMaxSlots / c->page_size)
        return fail(MNB_ERR_SHAPE, "%s: %lld pages of %lld tokens (at least one, at most 2^31 - 64 tokens)", fn,
                    (long long)c->num_pages, (long long)c->page_size);
    if (c->num_heads < 1 || c->num_heads > kMaxHeads)
        return fail(MNB_ERR_SHAPE, "%s: %lld KV heads", fn, (long long)c->num_heads);
    if (c->head_dim < 8 || c->head_dim > 256 || c->head_dim % 8)
        return fail(MNB_ERR_SHAPE, "%s: head size %lld is not a multiple of 8 up to 256", fn, (long long)c->head_dim);
    if (!aligned(c->k, 16) || !aligned(c->v, 16))
        return fail(MNB_ERR_ALIGN, "%s: the cache must be 16-byte aligned", fn);
    for (int64_t st : {c->page_stride, c->slot_stride, c->head_stride})
        if ((rc = check_stride(fn, st, c->dtype)))
            return rc;
    return MNB_OK;
}

}  // namespace mnb

using namespace mnb;

extern "C" {

const char *mnb_last_error(void) { return g_msg; }

const char *mnb_version(void) { return "mnb 0.1 (sm_100a)"; }

int mnb_packed_sizes(int64_t N, int64_t K, int bs, mnb_dtype scale_t, int has_zp,
                     size_t *packed_bytes, size_t *scale_bytes, size_t *zp_bytes) {
    clear_error();
    int rc;
    if (!packed_bytes || !scale_bytes || !zp_bytes)
        return fail(MNB_ERR_INVALID_ARG, "mnb_packed_sizes: NULL output pointer");
    if ((rc = check_dtype("mnb_packed_sizes", "scale", scale_t)))
        return rc;
    if ((rc = check_weight_shape("mnb_packed_sizes", N, K, bs)))
        return rc;
    int64_t nb = K / bs;
    *packed_bytes = (size_t)(N * (K / 2));
    *scale_bytes = (size_t)(N * nb * (scale_t == MNB_F32 ? 4 : 2));
    *zp_bytes = has_zp ? (size_t)(N * ((nb + 1) / 2)) : 0;
    return MNB_OK;
}

int mnb_quantize_rtn(const float *W, int64_t N, int64_t K, int bs, int has_zp, uint8_t *packed,
                     void *scales, mnb_dtype scale_t, uint8_t *zp, void *stream) {
    clear_error();
    const char *fn = "mnb_quantize_rtn";
    int rc;
    if ((rc = check_dtype(fn, "scale", scale_t)) || (rc = check_weight_shape(fn, N, K, bs)))
        return rc;
    if (N == 0)
        return MNB_OK;
    if (!W || !packed || !scales || (has_zp && !zp))
        return fail(MNB_ERR_INVALID_ARG, "%s: NULL pointer", fn);
    if (!aligned(W, 16) || !aligned(packed, 16))
        return fail(MNB_ERR_ALIGN, "%s: W and packed must be 16-byte aligned", fn);
    if (!aligned(scales, scale_t == MNB_F32 ? 4 : 2))
        return fail(MNB_ERR_ALIGN, "%s: scales misaligned", fn);
    return launch_quantize_rtn(W, N, K, bs, has_zp ? 1 : 0, packed, scales, scale_t == MNB_F16,
                               has_zp ? zp : nullptr, (cudaStream_t)stream);
}

int mnb_dequantize(const uint8_t *packed, const void *scales, mnb_dtype scale_t, const uint8_t *zp,
                   int64_t N, int64_t K, int bs, void *W_out, mnb_dtype out_t, void *stream) {
    clear_error();
    const char *fn = "mnb_dequantize";
    int rc;
    if ((rc = check_dtype(fn, "scale", scale_t)) || (rc = check_dtype(fn, "output", out_t)) ||
        (rc = check_weight_shape(fn, N, K, bs)))
        return rc;
    if (N == 0)
        return MNB_OK;
    if (!packed || !scales || !W_out)
        return fail(MNB_ERR_INVALID_ARG, "%s: NULL pointer", fn);
    if (!aligned(packed, 16) || !aligned(W_out, 16))
        return fail(MNB_ERR_ALIGN, "%s: packed and W_out must be 16-byte aligned", fn);
    if (!aligned(scales, scale_t == MNB_F32 ? 4 : 2))
        return fail(MNB_ERR_ALIGN, "%s: scales misaligned", fn);
    return launch_dequantize(packed, scales, scale_t == MNB_F16, zp, N, K, bs, W_out,
                             out_t == MNB_F16, (cudaStream_t)stream);
}

int mnb_gemv(const void *X, mnb_dtype act_t, const uint8_t *packed, const void *scales,
             mnb_dtype scale_t, const uint8_t *zp, void *Y, int64_t M, int64_t N, int64_t K,
             int bs, unsigned flags, void *stream) {
    clear_error();
    const char *fn = "mnb_gemv";
    int rc = check_matmul_args(fn, X, act_t, packed, scales, scale_t, Y, M, N, K, bs);
    if (rc)
        return rc;
    if (M > 32 || (M > 16 && act_t != MNB_F16))
        return fail(MNB_ERR_UNSUPPORTED, "%s: M=%lld above %d for %s activations (use mnb_gemm or mnb_matmul)", fn,
                    (long long)M, act_t == MNB_F16 ? 32 : 16, act_t == MNB_F16 ? "fp16" : "fp32");
    if (flags & ~(unsigned)MNB_FLAG_PDL)
        return fail(MNB_ERR_INVALID_ARG, "%s: unknown flags 0x%x", fn, flags);
    if (M == 0 || N == 0)
        return MNB_OK;
    return launch_gemv(X, act_t == MNB_F16, packed, scales, scale_t == MNB_F16, zp, Y, (int)M,
                       (int)N, (int)K, bs, flags, (cudaStream_t)stream);
}

int mnb_gemv_swiglu(const void *X, const uint8_t *packed, const void *scales, mnb_dtype scale_t,
                    const uint8_t *zp, void *Y, int64_t M, int64_t N, int64_t K, int bs, unsigned flags,
                    void *stream) {
    clear_error();
    const char *fn = "mnb_gemv_swiglu";
    int rc = check_matmul_args(fn, X, MNB_F16, packed, scales, scale_t, Y, M, N, K, bs);
    if (rc)
        return rc;
    if (M > 16)
        return fail(MNB_ERR_UNSUPPORTED, "%s: M=%lld > 16", fn, (long long)M);
    if (N % 16 != 0)
        return fail(MNB_ERR_SHAPE, "%s: N=%lld must be a multiple of 16 (8 gate + 8 up rows per group)", fn,
                    (long long)N);
    if (flags & ~(unsigned)MNB_FLAG_PDL)
        return fail(MNB_ERR_INVALID_ARG, "%s: unknown flags 0x%x", fn, flags);
    if (M == 0 || N == 0)
        return MNB_OK;
    return launch_gemv_swiglu(X, packed, scales, scale_t == MNB_F16, zp, Y, (int)M, (int)N, (int)K, bs, flags,
                              (cudaStream_t)stream);
}

size_t mnb_gemv_argmax_workspace_bytes(int64_t M) {
    if (M < 1 || M > 16)
        return 0;
    return mnb::gemv_argmax_workspace_bytes((int)M);
}

int mnb_gemv_argmax(const void *X, const uint8_t *packed, const void *scales, mnb_dtype scale_t,
                    const uint8_t *zp, void *Y, int64_t M, int64_t N, int64_t K, int bs, int32_t *ids,
                    float *max_out, void *workspace, size_t ws_bytes, unsigned flags, void *stream) {
    clear_error();
    const char *fn = "mnb_gemv_argmax";
    int rc = check_matmul_args(fn, X, MNB_F16, packed, scales, scale_t, Y, M, N, K, bs);
    if (rc)
        return rc;
    if (M < 1 || M > 16)
        return fail(MNB_ERR_UNSUPPORTED, "%s: M=%lld outside [1, 16]", fn, (long long)M);
    if (N < 1)
        return fail(MNB_ERR_SHAPE, "%s: N must be positive", fn);
    if (flags & ~(unsigned)MNB_FLAG_PDL)
        return fail(MNB_ERR_INVALID_ARG, "%s: unknown flags 0x%x", fn, flags);
    if (!ids || !workspace)
        return fail(MNB_ERR_INVALID_ARG, "%s: NULL ids or workspace", fn);
    if (!aligned(ids, 4) || !aligned(max_out, 4) || !aligned(workspace, 16))
        return fail(MNB_ERR_ALIGN, "%s: ids / max_out need 4-byte, workspace 16-byte alignment", fn);
    const size_t need = mnb::gemv_argmax_workspace_bytes((int)M);
    if (ws_bytes < need)
        return fail(MNB_ERR_INVALID_ARG, "%s: workspace of %zu bytes, %zu needed", fn, ws_bytes, need);
    return launch_gemv_argmax(X, packed, scales, scale_t == MNB_F16, zp, Y, (int)M, (int)N, (int)K, bs, ids,
                              max_out, workspace, flags, (cudaStream_t)stream);
}

int mnb_gemv_argmax_noalloc(const void *X, const uint8_t *packed, const void *scales, mnb_dtype scale_t,
                            const uint8_t *zp, void *Y, int64_t M, int64_t N, int64_t K, int bs, int32_t *ids,
                            float *max_out, unsigned flags, void *stream) {
    clear_error();
    const char *fn = "mnb_gemv_argmax_noalloc";
    int rc = check_matmul_args(fn, X, MNB_F16, packed, scales, scale_t, Y, M, N, K, bs);
    if (rc)
        return rc;
    if (M < 1 || M > 16)
        return fail(MNB_ERR_UNSUPPORTED, "%s: M=%lld outside [1, 16]", fn, (long long)M);
    if (N < 1)
        return fail(MNB_ERR_SHAPE, "%s: N must be positive", fn);
    if (flags & ~(unsigned)MNB_FLAG_PDL)
        return fail(MNB_ERR_INVALID_ARG, "%s: unknown flags 0x%x", fn, flags);
    if (!ids)
        return fail(MNB_ERR_INVALID_ARG, "%s: NULL ids", fn);
    if (!aligned(ids, 4) || !aligned(max_out, 4))
        return fail(MNB_ERR_ALIGN, "%s: ids and max_out need 4-byte alignment", fn);
    return launch_gemv_argmax_noalloc(X, packed, scales, scale_t == MNB_F16, zp, Y, (int)M, (int)N, (int)K, bs,
                                      ids, max_out, flags, (cudaStream_t)stream);
}

int mnb_gemm(const void *X, mnb_dtype act_t, const uint8_t *packed, const void *scales,
             mnb_dtype scale_t, const uint8_t *zp, void *Y, int64_t M, int64_t N, int64_t K,
             int bs, unsigned flags, void *stream) {
    clear_error();
    const char *fn = "mnb_gemm";
    int rc = check_matmul_args(fn, X, act_t, packed, scales, scale_t, Y, M, N, K, bs);
    if (rc)
        return rc;
    if (act_t != MNB_F16)
        return fail(MNB_ERR_UNSUPPORTED, "%s: the tensor-core path takes fp16 activations", fn);
    if (scale_t != MNB_F16)
        return fail(MNB_ERR_UNSUPPORTED, "%s: the tensor-core path takes fp16 scales (the q4f16 variant)", fn);
    if (N % 128 != 0 || K % 64 != 0)
        return fail(MNB_ERR_SHAPE, "%s: N=%lld must be a multiple of 128 and K=%lld of 64", fn,
                    (long long)N, (long long)K);
    if (flags & ~(unsigned)MNB_FLAG_PDL)
        return fail(MNB_ERR_INVALID_ARG, "%s: unknown flags 0x%x", fn, flags);
    if (M == 0 || N == 0)
        return MNB_OK;
    return launch_gemm(X, packed, scales, scale_t == MNB_F16, zp, Y, (int)M, (int)N, (int)K, bs,
                       flags, (cudaStream_t)stream);
}

// Largest M the dispatcher serves with one decode GEMV launch before switching
// to the tensor-core GEMM (measured on the 1.7B decoder projections, per
// 196-projection pass: GEMV 1.84 / 2.16 / 2.53 ms against GEMM 2.51 / 2.51 /
// 2.51 ms at M = 17 / 24 / 28).
static const int64_t kGemvMaxM = 24;

int mnb_matmul(const void *X, mnb_dtype act_t, const uint8_t *packed, const void *scales, mnb_dtype scale_t,
               const uint8_t *zp, void *Y, int64_t M, int64_t N, int64_t K, int bs, unsigned flags, void *stream) {
    clear_error();
    const char *fn = "mnb_matmul";
    int rc = check_matmul_args(fn, X, act_t, packed, scales, scale_t, Y, M, N, K, bs);
    if (rc)
        return rc;
    if (flags & ~(unsigned)MNB_FLAG_PDL)
        return fail(MNB_ERR_INVALID_ARG, "%s: unknown flags 0x%x", fn, flags);
    if (M == 0 || N == 0)
        return MNB_OK;
    const bool gemm_ok = act_t == MNB_F16 && scale_t == MNB_F16 && N % 128 == 0 && K % 64 == 0;
    if (gemm_ok && M > kGemvMaxM)
        return launch_gemm(X, packed, scales, scale_t == MNB_F16, zp, Y, (int)M, (int)N, (int)K, bs, flags,
                           (cudaStream_t)stream);
    // decode GEMV launches of up to 24 (fp16) or 16 (fp32) tokens; chunk
    // offsets are multiples of 8 rows, so every chunk keeps the 16-byte
    // alignment of X and Y
    const size_t elem = (act_t == MNB_F16) ? 2 : 4;
    const int64_t chunk = (act_t == MNB_F16) ? kGemvMaxM : 16;
    for (int64_t m0 = 0; m0 < M; m0 += chunk) {
        const int mc = (int)((M - m0 < chunk) ? (M - m0) : chunk);
        rc = launch_gemv(static_cast<const unsigned char *>(X) + (size_t)m0 * (size_t)K * elem, act_t == MNB_F16,
                         packed, scales, scale_t == MNB_F16, zp,
                         static_cast<unsigned char *>(Y) + (size_t)m0 * (size_t)N * elem, mc, (int)N, (int)K, bs,
                         flags, (cudaStream_t)stream);
        if (rc)
            return rc;
    }
    return MNB_OK;
}

int mnb_embed_gather(const int8_t *table, const float *row_scales, int64_t V, int64_t D,
                     const int32_t *ids, int64_t T, void *out, mnb_dtype out_t, int *status,
                     void *stream) {
    clear_error();
    const char *fn = "mnb_embed_gather";
    int rc;
    if ((rc = check_dtype(fn, "output", out_t)))
        return rc;
    if (V < 0 || D < 0 || T < 0)
        return fail(MNB_ERR_INVALID_ARG, "%s: negative size", fn);
    if (D % 16 != 0 || D > kMaxDim || V > ((int64_t)1 << 31) - 1 || T > kMaxDim)
        return fail(MNB_ERR_SHAPE, "%s: D must be a multiple of 16; V < 2^31", fn);
    if (T == 0 || D == 0)
        return MNB_OK;
    if (!ids || !out || (V > 0 && (!table || !row_scales)))
        return fail(MNB_ERR_INVALID_ARG, "%s: NULL pointer", fn);
    if (!aligned(table, 16) || !aligned(out, 16) || !aligned(row_scales, 4) || !aligned(ids, 4) ||
        !aligned(status, 4))
        return fail(MNB_ERR_ALIGN, "%s: table and out must be 16-byte aligned", fn);
    return launch_embed_gather(table, row_scales, V, D, ids, T, out, out_t == MNB_F16, status,
                               (cudaStream_t)stream);
}

size_t mnb_gemv_chain_plan_bytes(int ntasks) { return gemv_chain_plan_bytes(ntasks); }

size_t mnb_gemv_chain_workspace_bytes(int ntasks) { return gemv_chain_workspace_bytes(ntasks); }

int mnb_gemv_chain_plan(const mnb_gemv_task *tasks, int ntasks, int64_t M, int bs, void *plan, size_t plan_bytes) {
    clear_error();
    static const char *fn = "mnb_gemv_chain_plan";
    if (!tasks || !plan)
        return fail(MNB_ERR_INVALID_ARG, "%s: NULL tasks or plan", fn);
    if (ntasks < 1 || ntasks > 65536)
        return fail(MNB_ERR_INVALID_ARG, "%s: ntasks=%d outside [1, 65536]", fn, ntasks);
    if (plan_bytes < gemv_chain_plan_bytes(ntasks))
        return fail(MNB_ERR_INVALID_ARG, "%s: plan buffer of %zu bytes, %zu needed", fn, plan_bytes,
                    gemv_chain_plan_bytes(ntasks));
    if (!aligned(plan, 64))
        return fail(MNB_ERR_ALIGN, "%s: plan buffer not 64-byte aligned", fn);
    if (bs != 32 && bs != 64)
        return fail(MNB_ERR_SHAPE, "%s: block size %d not in {32, 64}", fn, bs);
    if (M < 1)
        return fail(MNB_ERR_INVALID_ARG, "%s: M=%lld", fn, (long long)M);
    if (M > 8)
        return fail(MNB_ERR_UNSUPPORTED, "%s: M=%lld above 8", fn, (long long)M);
    return gemv_chain_plan(tasks, ntasks, (int)M, bs, plan, plan_bytes);
}

int mnb_gemv_chain(const void *plan, const void *plan_device, void *workspace, size_t ws_bytes, unsigned flags,
                   void *stream) {
    clear_error();
    static const char *fn = "mnb_gemv_chain";
    if (!plan || !plan_device || !workspace)
        return fail(MNB_ERR_INVALID_ARG, "%s: NULL plan, device plan or workspace", fn);
    if (!aligned(plan, 64) || !aligned(plan_device, 64) || !aligned(workspace, 4))
        return fail(MNB_ERR_ALIGN, "%s: plans must be 64-byte aligned, the workspace 4-byte aligned", fn);
    if (flags & ~(unsigned)MNB_FLAG_PDL)
        return fail(MNB_ERR_INVALID_ARG, "%s: unknown flags 0x%x", fn, flags);
    return launch_gemv_chain(plan, plan_device, workspace, ws_bytes, flags, (cudaStream_t)stream);
}

static const int64_t kGptqMaxK = 8192;

int mnb_gptq_hessian(const void *X, mnb_dtype x_t, int64_t T, int64_t K, float *H, int accumulate, void *stream) {
    clear_error();
    const char *fn = "mnb_gptq_hessian";
    int rc;
    if ((rc = check_dtype(fn, "input", x_t)))
        return rc;
    if (T < 0 || K < 1 || K > kGptqMaxK)
        return fail(MNB_ERR_SHAPE, "%s: T=%lld, K=%lld (K must be in [1, %lld])", fn, (long long)T, (long long)K,
                    (long long)kGptqMaxK);
    if (T > kMaxDim)
        return fail(MNB_ERR_SHAPE, "%s: T above 2^30", fn);
    if (!H || (T > 0 && !X))
        return fail(MNB_ERR_INVALID_ARG, "%s: NULL X or H", fn);
    if (!aligned(H, 4) || !aligned(X, x_t == MNB_F32 ? 4 : 2))
        return fail(MNB_ERR_ALIGN, "%s: X and H need their element alignment", fn);
    return launch_gptq_hessian(X, x_t == MNB_F16, T, K, H, accumulate ? 1 : 0, (cudaStream_t)stream);
}

size_t mnb_gptq_workspace_bytes(int64_t K) {
    if (K < 1 || K > kGptqMaxK)
        return 0;
    return gptq_workspace_bytes(K);
}

int mnb_gptq_prepare(const float *H, int64_t K, float percdamp, float *U, uint8_t *dead, void *workspace,
                     size_t ws_bytes, float *damp_used, void *stream) {
    clear_error();
    const char *fn = "mnb_gptq_prepare";
    if (K < 1 || K > kGptqMaxK)
        return fail(MNB_ERR_SHAPE, "%s: K=%lld outside [1, %lld]", fn, (long long)K, (long long)kGptqMaxK);
    if (!H || !U || !dead || !workspace)
        return fail(MNB_ERR_INVALID_ARG, "%s: NULL H, U, dead or workspace", fn);
    if (!(percdamp >= 0.f) || !(percdamp <= 1.f))
        return fail(MNB_ERR_INVALID_ARG, "%s: percdamp %g outside [0, 1]", fn, (double)percdamp);
    if (!aligned(H, 4) || !aligned(U, 4) || !aligned(workspace, 16))
        return fail(MNB_ERR_ALIGN, "%s: H and U need 4-byte, the workspace 16-byte alignment", fn);
    if (ws_bytes < gptq_workspace_bytes(K))
        return fail(MNB_ERR_INVALID_ARG, "%s: workspace of %zu bytes, %zu needed", fn, ws_bytes,
                    gptq_workspace_bytes(K));
    return launch_gptq_prepare(H, K, percdamp, U, dead, workspace, damp_used, (cudaStream_t)stream);
}

int mnb_gptq_quantize(const float *W, const float *U, const uint8_t *dead, int64_t N, int64_t K, int bs, int has_zp,
                      uint8_t *packed, void *scales, mnb_dtype scale_t, uint8_t *zp, void *stream) {
    clear_error();
    const char *fn = "mnb_gptq_quantize";
    int rc;
    if ((rc = check_dtype(fn, "scale", scale_t)) || (rc = check_weight_shape(fn, N, K, bs)))
        return rc;
    if (K > kGptqMaxK)
        return fail(MNB_ERR_SHAPE, "%s: K=%lld above %lld", fn, (long long)K, (long long)kGptqMaxK);
    if (N == 0)
        return MNB_OK;
    if (!W || !U || !packed || !scales || (has_zp && !zp))
        return fail(MNB_ERR_INVALID_ARG, "%s: NULL pointer", fn);
    if (!aligned(W, 4) || !aligned(U, 4) || !aligned(scales, scale_t == MNB_F32 ? 4 : 2))
        return fail(MNB_ERR_ALIGN, "%s: W, U and scales need their element alignment", fn);
    return launch_gptq_quantize(W, U, dead, N, K, bs, has_zp ? 1 : 0, packed, scales, scale_t == MNB_F16,
                                has_zp ? zp : nullptr, (cudaStream_t)stream);
}

int mnb_paged_tables(const mnb_paged_tables_args *args, unsigned flags, void *stream) {
    clear_error();
    const char *fn = "mnb_paged_tables";
    if (!args)
        return fail(MNB_ERR_INVALID_ARG, "%s: NULL arguments", fn);
    const mnb_paged_tables_args &a = *args;
    if (a.B < 0 || a.T < 0 || a.num_free < 0)
        return fail(MNB_ERR_INVALID_ARG, "%s: negative size (B=%lld T=%lld num_free=%lld)", fn, (long long)a.B,
                    (long long)a.T, (long long)a.num_free);
    if (a.B > kMaxRequests)
        return fail(MNB_ERR_UNSUPPORTED, "%s: B=%lld above %lld", fn, (long long)a.B, (long long)kMaxRequests);
    if (a.page_size < 1 || a.num_pages < 1 || a.page_size > kMaxSlots || a.num_pages > kMaxSlots / a.page_size)
        return fail(MNB_ERR_SHAPE, "%s: %lld pages of %lld tokens (at least one, at most 2^31 - 64 tokens)", fn,
                    (long long)a.num_pages, (long long)a.page_size);
    if (a.max_blocks < 1 || a.max_blocks > kMaxSlots / a.page_size || a.table_stride < a.max_blocks ||
        a.table_stride > kMaxStride)
        return fail(MNB_ERR_SHAPE, "%s: block table of %lld columns, row stride %lld", fn, (long long)a.max_blocks,
                    (long long)a.table_stride);
    if (a.T > kMaxDim || a.num_free > kMaxDim)
        return fail(MNB_ERR_SHAPE, "%s: T or num_free above 2^30", fn);
    if (flags & ~(unsigned)MNB_FLAG_PDL)
        return fail(MNB_ERR_INVALID_ARG, "%s: unknown flags 0x%x", fn, flags);
    if ((a.B > 0 && (!a.ctx_lens || !a.new_lens || !a.block_table || !a.seq_lens)) ||
        (a.num_free > 0 && !a.free_pages) || (a.T > 0 && (!a.slots || !a.positions)) || !a.free_start || !a.free_next || !a.cu_new)
        return fail(MNB_ERR_INVALID_ARG, "%s: NULL pointer", fn);
    for (const void *ptr : {(const void *)a.ctx_lens, (const void *)a.new_lens, (const void *)a.free_pages,
                            (const void *)a.free_start, (const void *)a.block_table, (const void *)a.seq_lens,
                            (const void *)a.cu_new, (const void *)a.slots, (const void *)a.positions,
                            (const void *)a.free_next, (const void *)a.status})
        if (!aligned(ptr, 4))
            return fail(MNB_ERR_ALIGN, "%s: a pointer is not 4-byte aligned", fn);
    if (a.free_next == a.free_start || (a.B > 0 && (a.seq_lens == a.ctx_lens || a.seq_lens == a.new_lens)))
        return fail(MNB_ERR_INVALID_ARG, "%s: an output is an input's buffer", fn);
    return launch_paged_tables(a.ctx_lens, a.new_lens, (int)a.B, (int)a.page_size, (int)a.num_pages, a.free_pages,
                               (int)a.num_free, a.free_start, a.block_table, a.table_stride, (int)a.max_blocks,
                               a.seq_lens, a.cu_new, a.slots, a.positions, (int)a.T, a.free_next, a.status, flags,
                               (cudaStream_t)stream);
}

int mnb_rope_append(const mnb_rope_append_args *args, unsigned flags, void *stream) {
    clear_error();
    const char *fn = "mnb_rope_append";
    if (!args)
        return fail(MNB_ERR_INVALID_ARG, "%s: NULL arguments", fn);
    mnb_paged_cache pool, *cache = &pool;
    int rc = check_paged_cache(fn, &args->cache, cache);
    const void *q = args->q, *k = args->k, *v = args->v;
    void *q_out = args->q_out;
    const int32_t *slots = args->slots, *positions = args->positions;
    const float *cos = args->cos, *sin = args->sin, *q_weight = args->q_weight, *k_weight = args->k_weight;
    int *status = args->status;
    int64_t q_ts = args->q_token_stride, q_hs = args->q_head_stride, k_ts = args->k_token_stride;
    int64_t k_hs = args->k_head_stride, v_ts = args->v_token_stride, v_hs = args->v_head_stride;
    int64_t o_ts = args->o_token_stride, o_hs = args->o_head_stride;
    const int64_t T = args->T, Hq = args->Hq, rot_dim = args->rot_dim, num_pos = args->num_pos;
    const float eps = args->eps;
    if (rc)
        return rc;
    if (T < 0 || Hq < 0 || rot_dim < 0)
        return fail(MNB_ERR_INVALID_ARG, "%s: negative size (T=%lld Hq=%lld rot_dim=%lld)", fn, (long long)T,
                    (long long)Hq, (long long)rot_dim);
    if (T > kMaxDim || Hq > kMaxHeads)
        return fail(MNB_ERR_SHAPE, "%s: T above 2^30 or Hq above %lld", fn, (long long)kMaxHeads);
    if (rot_dim % 8 || rot_dim > cache->head_dim)
        return fail(MNB_ERR_SHAPE, "%s: rot_dim=%lld is not a multiple of 8 up to D=%lld", fn, (long long)rot_dim,
                    (long long)cache->head_dim);
    if (rot_dim && (num_pos < 1 || num_pos > kMaxSlots))
        return fail(MNB_ERR_SHAPE, "%s: num_pos=%lld", fn, (long long)num_pos);
    if (!(eps >= 0.0f) || !(eps <= 3.0e38f))
        return fail(MNB_ERR_INVALID_ARG, "%s: eps is negative or not finite", fn);
    if (flags & ~(unsigned)MNB_FLAG_PDL)
        return fail(MNB_ERR_INVALID_ARG, "%s: unknown flags 0x%x", fn, flags);
    if (T == 0)
        return MNB_OK;
    if (!k || !v || !slots || (Hq && (!q || !q_out)) || (rot_dim && (!positions || !cos || !sin)))
        return fail(MNB_ERR_INVALID_ARG, "%s: NULL pointer", fn);
    for (const void *ptr : {q, k, v, (const void *)q_out, (const void *)cos, (const void *)sin, (const void *)q_weight,
                            (const void *)k_weight})
        if (!aligned(ptr, 16))
            return fail(MNB_ERR_ALIGN, "%s: a pointer is not 16-byte aligned", fn);
    if (!aligned(slots, 4) || !aligned(positions, 4) || !aligned(status, 4))
        return fail(MNB_ERR_ALIGN, "%s: slots, positions and status need 4-byte alignment", fn);
    if (T == 1)
        q_ts = k_ts = v_ts = o_ts = 0;
    if (Hq <= 1)
        q_hs = o_hs = 0;
    if (Hq == 0)
        q_ts = o_ts = 0;
    if (cache->num_heads == 1)
        k_hs = v_hs = 0;
    for (int64_t st : {q_ts, q_hs, k_ts, k_hs, v_ts, v_hs, o_ts, o_hs})
        if ((rc = check_stride(fn, st, cache->dtype)))
            return rc;
    // rows that are written must not lie on one another
    const int64_t D = cache->head_dim;
    if ((cache->num_heads > 1 && cache->head_stride < D) || (cache->page_size > 1 && cache->slot_stride < D) ||
        (cache->num_pages > 1 && cache->page_stride < D) || (Hq > 1 && o_hs < D) || (Hq && T > 1 && o_ts < D))
        return fail(MNB_ERR_SHAPE, "%s: rows of the cache or of q_out overlap", fn);
    if (Hq && q_out == q && ((T > 1 && o_ts != q_ts) || (Hq > 1 && o_hs != q_hs)))
        return fail(MNB_ERR_INVALID_ARG, "%s: q_out is q with other strides", fn);
    return launch_rope_append(q, q_ts, q_hs, k, k_ts, k_hs, v, v_ts, v_hs, cache, slots, positions, T, (int)Hq, cos,
                              sin, (int)rot_dim, (int)num_pos, q_weight, k_weight, eps, q_out, o_ts, o_hs, status,
                              flags, (cudaStream_t)stream);
}

size_t mnb_paged_attention_workspace_bytes(int64_t B, int64_t Hq, int64_t Hkv, int64_t D, mnb_dtype dtype) {
    if (B < 0 || B > kMaxRequests || Hkv < 1 || Hq < Hkv || Hq > kMaxHeads || Hq % Hkv || D < 8 || D > 256 || D % 8 ||
        (dtype != MNB_F16 && dtype != MNB_F32))
        return 0;
    return paged_attention_workspace_bytes((int)Hq, (int)Hkv, (int)D, dtype == MNB_F16);
}

int mnb_paged_attention(const mnb_paged_attention_args *args, unsigned flags, void *stream) {
    clear_error();
    const char *fn = "mnb_paged_attention";
    if (!args)
        return fail(MNB_ERR_INVALID_ARG, "%s: NULL arguments", fn);
    mnb_paged_cache pool, *cache = &pool;
    int rc = check_paged_cache(fn, &args->cache, cache);
    const void *q = args->q;
    void *out = args->out, *workspace = args->workspace;
    float *lse = args->lse;
    const int32_t *block_table = args->block_table, *seq_lens = args->seq_lens;
    int *status = args->status;
    int64_t q_bs = args->q_request_stride, q_hs = args->q_head_stride, o_bs = args->o_request_stride;
    int64_t o_hs = args->o_head_stride;
    const int64_t table_stride = args->table_stride, max_blocks = args->max_blocks, B = args->B, Hq = args->Hq;
    const size_t ws_bytes = args->ws_bytes;
    const float scale = args->scale;
    if (rc)
        return rc;
    if (B < 0 || Hq < 1)
        return fail(MNB_ERR_INVALID_ARG, "%s: B=%lld Hq=%lld", fn, (long long)B, (long long)Hq);
    if (B > kMaxRequests)
        return fail(MNB_ERR_UNSUPPORTED, "%s: B=%lld above %lld", fn, (long long)B, (long long)kMaxRequests);
    if (Hq > kMaxHeads || Hq % cache->num_heads)
        return fail(MNB_ERR_SHAPE, "%s: Hq=%lld is not a multiple of %lld KV heads up to %lld", fn, (long long)Hq,
                    (long long)cache->num_heads, (long long)kMaxHeads);
    if (max_blocks < 1 || max_blocks > kMaxSlots / cache->page_size || table_stride < max_blocks ||
        table_stride > kMaxStride)
        return fail(MNB_ERR_SHAPE, "%s: block table of %lld columns, row stride %lld", fn, (long long)max_blocks,
                    (long long)table_stride);
    if (!(scale >= -2.0e38f && scale <= 2.0e38f))   // times log2 e, as the kernel takes it, it has to be finite
        return fail(MNB_ERR_INVALID_ARG, "%s: scale is not a number of at most 2e38", fn);
    if (flags & ~(unsigned)MNB_FLAG_PDL)
        return fail(MNB_ERR_INVALID_ARG, "%s: unknown flags 0x%x", fn, flags);
    if (B == 0)
        return MNB_OK;
    if (!q || !out || !block_table || !seq_lens || !workspace)
        return fail(MNB_ERR_INVALID_ARG, "%s: NULL pointer", fn);
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(workspace, 16))
        return fail(MNB_ERR_ALIGN, "%s: q, out and workspace must be 16-byte aligned", fn);
    if (!aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(lse, 4) || !aligned(status, 4))
        return fail(MNB_ERR_ALIGN, "%s: block_table, seq_lens, lse and status need 4-byte alignment", fn);
    if (B == 1)
        q_bs = o_bs = 0;
    if (Hq == 1)
        q_hs = o_hs = 0;
    for (int64_t st : {q_bs, q_hs, o_bs, o_hs})
        if ((rc = check_stride(fn, st, cache->dtype)))
            return rc;
    if ((Hq > 1 && o_hs < cache->head_dim) || (B > 1 && o_bs < cache->head_dim))
        return fail(MNB_ERR_SHAPE, "%s: rows of out overlap", fn);
    const size_t need = paged_attention_workspace_bytes((int)Hq, (int)cache->num_heads, (int)cache->head_dim,
                                                        cache->dtype == MNB_F16);
    if (ws_bytes < need)
        return fail(MNB_ERR_INVALID_ARG, "%s: workspace of %zu bytes, %zu needed", fn, ws_bytes, need);
    return launch_paged_attention(q, q_bs, q_hs, cache, block_table, table_stride, (int)max_blocks, seq_lens, (int)B,
                                  (int)Hq, scale, out, o_bs, o_hs, lse, workspace, status, flags,
                                  (cudaStream_t)stream);
}

int mnb_device_status(unsigned *status_out, int clear) {
    clear_error();
    if (!status_out)
        return fail(MNB_ERR_INVALID_ARG, "mnb_device_status: NULL output");
    *status_out = 0;
    const int rc = read_device_status(status_out, clear);
    if (rc)
        return rc;
    if (*status_out & 7u)   // bits 0-2: a bounded wait inside a kernel gave up
        return fail(MNB_ERR_TIMEOUT, "mnb_device_status: a device-side wait timed out (status 0x%x)", *status_out);
    return MNB_OK;
}

}  // extern "C"
