// C-ABI entry points of libw4a16moe: argument checks, workspace layout and
// kernel sequencing. No allocation, no synchronisation (except in
// moe_check_device_error, which exists to synchronise).
#include <math.h>
#include <stdint.h>

#include <mutex>

#include "common.cuh"
#include "kernels.cuh"
#include "kv4_kernels.cuh"
#include "step_kernels.cuh"
#include "w4a16moe.h"

namespace moe {

namespace {
constexpr int kMaxDevices = 64;
int g_sms[kMaxDevices];

struct SmemAttr {
    const void *func;
    int bytes;
    bool done[kMaxDevices];
};
constexpr int kMaxSmemKernels = 64;   // kernels that raise their shared-memory limit (28 today)
SmemAttr g_attrs[kMaxSmemKernels];
int g_nattrs = 0;
std::mutex g_attrs_mu;   // callers may launch from several host threads

int current_device() {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 0;
    return dev;
}
}  // namespace

int sm_count() {
    const int dev = current_device();
    if (g_sms[dev] == 0) {
        int n = 0;
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) n = 1;
        g_sms[dev] = n;
    }
    return g_sms[dev];
}

cudaError_t set_smem_once(const void *func, int bytes) {
    const int dev = current_device();
    std::lock_guard<std::mutex> lock(g_attrs_mu);
    int i = 0;
    for (; i < g_nattrs; ++i)
        if (g_attrs[i].func == func) break;
    if (i == g_nattrs) {
        if (g_nattrs == kMaxSmemKernels)
            return cudaFuncSetAttribute(func, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        g_attrs[i].func = func;
        g_attrs[i].bytes = bytes;
        ++g_nattrs;
    }
    if (g_attrs[i].done[dev]) return cudaSuccess;
    cudaError_t err = cudaFuncSetAttribute(func, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (err == cudaSuccess) g_attrs[i].done[dev] = true;
    return err;
}

// A plain record outside stream capture; inside a capture, an external event
// node, so that the event can still be timed after each graph replay.
cudaError_t record_profile_event(cudaEvent_t ev, cudaStream_t s) {
    if (!ev) return cudaSuccess;
    cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
    const cudaError_t err = cudaStreamIsCapturing(s, &cs);
    if (err != cudaSuccess) return err;
    return cs == cudaStreamCaptureStatusActive ? cudaEventRecordWithFlags(ev, s, cudaEventRecordExternal)
                                               : cudaEventRecord(ev, s);
}

}  // namespace moe

using namespace moe;

namespace {

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Null is allowed only for empty tensors.
bool ptr_ok(const void *p, bool empty) { return empty ? (p == nullptr || aligned16(p)) : (p && aligned16(p)); }

int check_dims(const moe_dims &d) {
    if (d.T < 0 || d.H <= 0 || d.E <= 0 || d.k <= 0 || d.I <= 0) return MOE_ERR_INVALID_ARG;
    if (d.H % kGroup || d.I % kGroup || d.H > 8192 || d.I > 4096) return MOE_ERR_UNSUPPORTED;
    if (d.k > kMaxK || d.k > d.E || d.E > kMaxE) return MOE_ERR_UNSUPPORTED;
    if (d.T > (1 << 20)) return MOE_ERR_UNSUPPORTED;
    // token rows of the fp32 accumulator are addressed by 32-bit offsets t * H
    if ((int64_t)d.T * d.H >= ((int64_t)1 << 32)) return MOE_ERR_UNSUPPORTED;
    if (!prefill_supported(d)) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

int check_ws(const moe_dims &d, const void *ws, size_t ws_bytes) {
    if (!ws || !aligned16(ws)) return MOE_ERR_INVALID_ARG;
    if (ws_bytes < ws_layout(d).total) return MOE_ERR_WORKSPACE;
    return MOE_OK;
}

int cuda_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

cudaEvent_t g_ev_before = nullptr, g_ev_after = nullptr;

int forward_impl(const uint16_t *hidden, const int32_t *topk_ids, const float *topk_w, const int32_t *w1_packed,
                 const uint16_t *w1_scales, const int32_t *w2_packed, const uint16_t *w2_scales, uint16_t *out,
                 uint16_t *next, float eps, moe_dims d, void *ws, size_t ws_bytes, void *stream) {
    int rc = check_dims(d);
    if (rc) return rc;
    const bool empty = d.T == 0;
    if (!ptr_ok(hidden, empty) || !ptr_ok(topk_ids, empty) || !ptr_ok(topk_w, empty)) return MOE_ERR_INVALID_ARG;
    if (!ptr_ok(w1_packed, false) || !ptr_ok(w1_scales, false) || !ptr_ok(w2_packed, false) ||
        !ptr_ok(w2_scales, false))
        return MOE_ERR_INVALID_ARG;
    if (!ptr_ok(next ? (const void *)next : (const void *)out, empty)) return MOE_ERR_INVALID_ARG;
    if (next && !(eps >= 0.f)) return MOE_ERR_INVALID_ARG;
    if ((rc = check_ws(d, ws, ws_bytes))) return rc;
    if (empty) return MOE_OK;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    ExpertArgs a{hidden, topk_ids, topk_w, w1_packed, w1_scales, w2_packed, w2_scales};
    cudaError_t err;
    if (fused_supported(d)) {
        err = record_profile_event(g_ev_before, s);
        if (err == cudaSuccess) err = launch_decode_fused(a, d, ws, out, next, eps, s);
        if (err == cudaSuccess) err = record_profile_event(g_ev_after, s);
        return cuda_status(err);
    }
    err = launch_permute(topk_ids, d, ws, s);
    if (err == cudaSuccess) err = launch_prefill(a, d, ws, out, next, eps, g_ev_before, g_ev_after, s);
    return cuda_status(err);
}

}  // namespace

extern "C" {

const char *moe_status_str(int status) {
    switch (status) {
        case MOE_OK: return "ok";
        case MOE_ERR_INVALID_ARG: return "invalid argument (null or misaligned pointer, bad size)";
        case MOE_ERR_UNSUPPORTED: return "unsupported shape";
        case MOE_ERR_WORKSPACE: return "workspace too small";
        case MOE_ERR_CUDA: return "CUDA runtime or launch error";
        case MOE_ERR_DEVICE: return "a kernel saw an expert id, slot, page, length, token or logit out of range";
        case MOE_ERR_TIMEOUT: return "a kernel's bounded wait gave up";
        default: return "unknown status";
    }
}

int moe_version(void) { return 100; }

int moe_workspace_size(moe_dims d, size_t *bytes) {
    if (!bytes) return MOE_ERR_INVALID_ARG;
    const int rc = check_dims(d);
    if (rc) return rc;
    *bytes = ws_layout(d).total;
    return MOE_OK;
}

int moe_route(const uint16_t *hidden, const uint16_t *router_w, const float *bias, moe_dims d, int32_t *topk_ids,
              float *topk_w, void *ws, size_t ws_bytes, void *stream) {
    int rc = check_dims(d);
    if (rc) return rc;
    const bool empty = d.T == 0;
    if (!ptr_ok(hidden, empty) || !ptr_ok(router_w, false) || !ptr_ok(topk_ids, empty) || !ptr_ok(topk_w, empty))
        return MOE_ERR_INVALID_ARG;
    if (bias && !aligned16(bias)) return MOE_ERR_INVALID_ARG;
    if ((rc = check_ws(d, ws, ws_bytes))) return rc;
    if (empty) return MOE_OK;
    return cuda_status(launch_route(hidden, router_w, bias, d, topk_ids, topk_w, ws,
                                    reinterpret_cast<cudaStream_t>(stream)));
}

int moe_route_shared(const uint16_t *hidden, const uint16_t *router_w, const float *bias, moe_dims d,
                     int32_t *topk_ids, float *topk_w, void *ws, size_t ws_bytes, void *stream) {
    int rc = check_dims(d);
    if (rc) return rc;
    // the forward then runs with one more expert and one more slot per token
    if (d.k + 1 > kMaxK || d.E + 1 > kMaxE) return MOE_ERR_UNSUPPORTED;
    const bool empty = d.T == 0;
    if (!ptr_ok(hidden, empty) || !ptr_ok(router_w, false) || !ptr_ok(topk_ids, empty) || !ptr_ok(topk_w, empty))
        return MOE_ERR_INVALID_ARG;
    if (bias && !aligned16(bias)) return MOE_ERR_INVALID_ARG;
    if ((rc = check_ws(d, ws, ws_bytes))) return rc;
    if (empty) return MOE_OK;
    return cuda_status(launch_route(hidden, router_w, bias, d, topk_ids, topk_w, ws,
                                    reinterpret_cast<cudaStream_t>(stream), true));
}

int moe_w4a16_forward(const uint16_t *hidden, const int32_t *topk_ids, const float *topk_w,
                      const int32_t *w1_packed, const uint16_t *w1_scales, const int32_t *w2_packed,
                      const uint16_t *w2_scales, uint16_t *out, moe_dims d, void *ws, size_t ws_bytes,
                      void *stream) {
    return forward_impl(hidden, topk_ids, topk_w, w1_packed, w1_scales, w2_packed, w2_scales, out, nullptr, 0.f, d,
                        ws, ws_bytes, stream);
}

int moe_w4a16_forward_rms(const uint16_t *hidden, const int32_t *topk_ids, const float *topk_w,
                          const int32_t *w1_packed, const uint16_t *w1_scales, const int32_t *w2_packed,
                          const uint16_t *w2_scales, uint16_t *next, float eps, moe_dims d, void *ws,
                          size_t ws_bytes, void *stream) {
    if (!next && d.T > 0) return MOE_ERR_INVALID_ARG;
    return forward_impl(hidden, topk_ids, topk_w, w1_packed, w1_scales, w2_packed, w2_scales, nullptr, next, eps, d,
                        ws, ws_bytes, stream);
}

int moe_layer_forward(const uint16_t *hidden, const uint16_t *router_w, const float *bias, int32_t shared,
                      const int32_t *w1_packed, const uint16_t *w1_scales, const int32_t *w2_packed,
                      const uint16_t *w2_scales, uint16_t *out, uint16_t *next, float eps, int32_t *topk_ids,
                      float *topk_w, moe_dims d, void *ws, size_t ws_bytes, void *stream) {
    if (shared != 0 && shared != 1) return MOE_ERR_INVALID_ARG;
    int rc = check_dims(d);
    if (rc) return rc;
    if (shared && (d.k + 1 > kMaxK || d.E + 1 > kMaxE)) return MOE_ERR_UNSUPPORTED;
    // the forward's dims: the shared expert is one more expert and one more slot
    const moe_dims df{d.T, d.H, d.E + shared, d.k + shared, d.I};
    if ((rc = check_dims(df))) return rc;
    const bool empty = d.T == 0;
    if (!empty && (out != nullptr) == (next != nullptr)) return MOE_ERR_INVALID_ARG;   // exactly one output
    if (!ptr_ok(hidden, empty) || !ptr_ok(router_w, false) || !ptr_ok(topk_ids, empty) || !ptr_ok(topk_w, empty))
        return MOE_ERR_INVALID_ARG;
    if (!ptr_ok(w1_packed, false) || !ptr_ok(w1_scales, false) || !ptr_ok(w2_packed, false) ||
        !ptr_ok(w2_scales, false))
        return MOE_ERR_INVALID_ARG;
    if (!ptr_ok(next ? (const void *)next : (const void *)out, empty)) return MOE_ERR_INVALID_ARG;
    if (next && !(eps >= 0.f)) return MOE_ERR_INVALID_ARG;
    if (bias && !aligned16(bias)) return MOE_ERR_INVALID_ARG;
    // one workspace serves the router (dims d) and the forward (dims df)
    if ((rc = check_ws(d, ws, ws_bytes)) || (rc = check_ws(df, ws, ws_bytes))) return rc;
    if (empty) return MOE_OK;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (fused_route_supported(df)) {
        const ExpertArgs a{hidden, nullptr, nullptr, w1_packed, w1_scales, w2_packed, w2_scales};
        const RouteArgs r{router_w, bias, topk_ids, topk_w, shared};
        cudaError_t err = record_profile_event(g_ev_before, s);
        if (err == cudaSuccess) err = launch_decode_fused(a, df, ws, out, next, eps, s, &r);
        if (err == cudaSuccess) err = record_profile_event(g_ev_after, s);
        return cuda_status(err);
    }
    // otherwise the router's kernels, then the forward's
    const cudaError_t err = launch_route(hidden, router_w, bias, d, topk_ids, topk_w, ws, s, shared != 0);
    if (err != cudaSuccess) return cuda_status(err);
    return forward_impl(hidden, topk_ids, topk_w, w1_packed, w1_scales, w2_packed, w2_scales, out, next, eps, df, ws,
                        ws_bytes, stream);
}

int moe_permute(const int32_t *topk_ids, moe_dims d, int32_t *offsets, int32_t *perm, void *ws, size_t ws_bytes,
                void *stream) {
    int rc = check_dims(d);
    if (rc) return rc;
    const bool empty = d.T == 0;
    if (!ptr_ok(topk_ids, empty) || !ptr_ok(offsets, false) || !ptr_ok(perm, empty)) return MOE_ERR_INVALID_ARG;
    if ((rc = check_ws(d, ws, ws_bytes))) return rc;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const WsLayout L = ws_layout(d);
    cudaError_t err = launch_permute(topk_ids, d, ws, s);
    if (err == cudaSuccess)
        err = cudaMemcpyAsync(offsets, ws_at<int32_t>(ws, L.offsets), sizeof(int32_t) * (d.E + 1),
                              cudaMemcpyDeviceToDevice, s);
    if (err == cudaSuccess && d.T > 0)
        err = cudaMemcpyAsync(perm, ws_at<int32_t>(ws, L.perm), sizeof(int32_t) * (size_t)d.T * d.k,
                              cudaMemcpyDeviceToDevice, s);
    return cuda_status(err);
}

int moe_pack_int4(const int8_t *q, int64_t N, int64_t K, int32_t *packed, int32_t *bad_count, void *stream) {
    if (N < 0 || K < 0 || K % 8) return MOE_ERR_INVALID_ARG;
    const bool empty = N == 0 || K == 0;
    if (!ptr_ok(q, empty) || !ptr_ok(packed, empty)) return MOE_ERR_INVALID_ARG;
    if (bad_count && (reinterpret_cast<uintptr_t>(bad_count) & 3u)) return MOE_ERR_INVALID_ARG;
    return cuda_status(launch_pack_int4(q, N, K, packed, bad_count, reinterpret_cast<cudaStream_t>(stream)));
}

int moe_forward_plan(moe_dims d, int32_t *plan) {
    if (!plan) return MOE_ERR_INVALID_ARG;
    const int rc = check_dims(d);
    if (rc) return rc;
    *plan = fused_plan(d);
    return MOE_OK;
}

int moe_quantize_int4(const uint16_t *w, int64_t N, int64_t K, int32_t nclip, int32_t *packed, uint16_t *scales,
                      int32_t *choice, void *stream) {
    if (N < 0 || K < 0 || K % kGroup || nclip < 1 || nclip > 100) return MOE_ERR_INVALID_ARG;
    const bool empty = N == 0 || K == 0;
    if (!ptr_ok(w, empty) || !ptr_ok(packed, empty) || !ptr_ok(scales, empty)) return MOE_ERR_INVALID_ARG;
    if (choice && !ptr_ok(choice, empty)) return MOE_ERR_INVALID_ARG;
    return cuda_status(
        launch_quantize_int4(w, N, K, nclip, packed, scales, choice, reinterpret_cast<cudaStream_t>(stream)));
}

int moe_w8a16_linear(const uint16_t *x, const int32_t *w_packed, const uint16_t *scales, int32_t gs, uint16_t *y,
                     int32_t T, int32_t N, int32_t K, void *ws, size_t ws_bytes, void *stream) {
    if (T < 0 || N < 0 || K <= 0 || (gs != 64 && gs != 128) || K % gs) return MOE_ERR_INVALID_ARG;
    if (T > (1 << 20) || K > 65536) return MOE_ERR_UNSUPPORTED;
    const bool empty = T == 0 || N == 0;
    if (!ptr_ok(x, T == 0) || !ptr_ok(w_packed, N == 0) || !ptr_ok(scales, N == 0) || !ptr_ok(y, empty))
        return MOE_ERR_INVALID_ARG;
    if (empty) return MOE_OK;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (T <= 8) {
        if (!w8a16_gemv_supported(T, K)) return MOE_ERR_UNSUPPORTED;
        return cuda_status(launch_w8a16(x, w_packed, scales, gs, y, T, N, K, s));
    }
    // the tensor-core GEMM records a wait that gave up in the workspace's error word, and
    // keeps the partial results of a split over K after it
    if (!ws || !aligned16(ws)) return MOE_ERR_INVALID_ARG;
    size_t need = 0;
    moe_w8a16_workspace_size(T, N, K, gs, &need);
    if (ws_bytes < need) return MOE_ERR_WORKSPACE;
    return cuda_status(launch_w8a16_gemm(x, w_packed, scales, gs, y, T, N, K, reinterpret_cast<Ctrl *>(ws),
                                         ws_at<float>(ws, sizeof(Ctrl)), s));
}

int moe_w8a16_workspace_size(int32_t T, int32_t N, int32_t K, int32_t gs, size_t *bytes) {
    if (!bytes || T < 0 || N < 0 || K <= 0 || (gs != 64 && gs != 128) || K % gs) return MOE_ERR_INVALID_ARG;
    size_t n = sizeof(Ctrl);
    if (T > 8 && N > 0) {
        const int S = w8a16_gemm_splits(T, N, K);
        if (S > 1) n += (size_t)S * T * N * 4;
    }
    *bytes = n;
    return MOE_OK;
}

int moe_w4a16_linear(const uint16_t *x, const int32_t *w_packed, const uint16_t *scales, uint16_t *y, int32_t T,
                     int32_t N, int32_t K, void *ws, size_t ws_bytes, void *stream) {
    size_t need = 0;
    const int rc = moe_w4a16_workspace_size(T, N, K, &need);
    if (rc) return rc;
    if (!ptr_ok(x, T == 0) || !ptr_ok(w_packed, N == 0) || !ptr_ok(scales, N == 0) || !ptr_ok(y, T == 0 || N == 0))
        return MOE_ERR_INVALID_ARG;
    if (!ws || !aligned16(ws)) return MOE_ERR_INVALID_ARG;
    if (ws_bytes < need) return MOE_ERR_WORKSPACE;
    if (T == 0 || N == 0) return MOE_OK;
    return cuda_status(launch_w4a16(x, w_packed, scales, y, T, N, K, ws, reinterpret_cast<cudaStream_t>(stream)));
}

int moe_w4a16_workspace_size(int32_t T, int32_t N, int32_t K, size_t *bytes) {
    if (!bytes || T < 0 || N < 0 || K <= 0) return MOE_ERR_INVALID_ARG;
    if (K % kGroup || T > (1 << 20) || K > 65536 || N > INT32_MAX - 255) return MOE_ERR_UNSUPPORTED;   // (rows of whole CTAs fit 32 bits)
    *bytes = w4a16_workspace_bytes(T, N, K);
    return MOE_OK;
}

}  // extern "C"

namespace {

// [T][heads][D] with D contiguous: 16-byte aligned rows.
bool rows_ok(const void *p, const moe_strides &s, bool empty) {
    return ptr_ok(p, empty) && s.token >= 0 && s.head >= 0 && s.token % 8 == 0 && s.head % 8 == 0;
}

// An output's rows must not overlap one another either.
bool out_rows_ok(const void *p, const moe_strides &s, int T, int heads, int D) {
    const bool empty = T == 0 || heads == 0;
    if (!rows_ok(p, s, empty)) return false;
    if (empty || (T == 1 && heads == 1)) return true;
    if (T == 1) return s.head >= D;
    if (heads == 1) return s.token >= D;
    if (s.token >= s.head) return s.head >= D && s.token >= (heads - 1) * s.head + D;
    return s.token >= D && s.head >= (T - 1) * s.token + D;
}

int check_cache(const moe_kv4_cache &c) {
    if (c.n_pages <= 0 || c.Hkv <= 0 || c.page_size <= 0 || c.D <= 0) return MOE_ERR_INVALID_ARG;
    if (c.D != 64 && c.D != 128) return MOE_ERR_UNSUPPORTED;
    if (c.page_size < 16 || c.page_size > 1024 || (c.page_size & (c.page_size - 1))) return MOE_ERR_UNSUPPORTED;
    if ((int64_t)c.n_pages * c.page_size >= ((int64_t)1 << 31) || c.Hkv > 1024) return MOE_ERR_UNSUPPORTED;
    // row indexes fit 32 bits (more rows than that do not fit the memory)
    if ((int64_t)c.n_pages * c.page_size * c.Hkv >= ((int64_t)1 << 32) - 1) return MOE_ERR_UNSUPPORTED;
    if (!ptr_ok(c.k_codes, false) || !ptr_ok(c.k_scales, false) || !ptr_ok(c.v_codes, false) ||
        !ptr_ok(c.v_scales, false))
        return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

int check_rows_ws(const void *ws, size_t ws_bytes) {
    if (!ws || !aligned16(ws)) return MOE_ERR_INVALID_ARG;
    return ws_bytes < sizeof(Ctrl) ? MOE_ERR_WORKSPACE : MOE_OK;
}

bool aligned4(const void *p) { return p && (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

}  // namespace

extern "C" {

int moe_qk_norm_rope(const uint16_t *q, moe_strides q_strides, const uint16_t *k, moe_strides k_strides,
                     const uint16_t *q_weight, const uint16_t *k_weight, const int32_t *positions,
                     const float *inv_freq, int32_t rot, int32_t interleaved, float eps, uint16_t *q_out,
                     moe_strides q_out_strides, uint16_t *k_out, moe_strides k_out_strides, int32_t T, int32_t Hq,
                     int32_t Hkv, int32_t D, void *stream) {
    if (T < 0 || Hq < 0 || Hkv < 0 || D <= 0 || rot < 0 || rot > D || (interleaved != 0 && interleaved != 1) ||
        !(eps >= 0.f))
        return MOE_ERR_INVALID_ARG;
    if ((D != 64 && D != 128 && D != 256) || rot % 16) return MOE_ERR_UNSUPPORTED;
    if (T > (1 << 20) || Hq > 1024 || Hkv > 1024) return MOE_ERR_UNSUPPORTED;
    const bool no_q = T == 0 || Hq == 0, no_k = T == 0 || Hkv == 0;
    if (!rows_ok(q, q_strides, no_q) || !rows_ok(k, k_strides, no_k) ||
        !out_rows_ok(q_out, q_out_strides, T, Hq, D) || !out_rows_ok(k_out, k_out_strides, T, Hkv, D))
        return MOE_ERR_INVALID_ARG;
    if ((q_weight && !aligned16(q_weight)) || (k_weight && !aligned16(k_weight))) return MOE_ERR_INVALID_ARG;
    if (T > 0 && rot > 0 && (!aligned4(positions) || !aligned4(inv_freq))) return MOE_ERR_INVALID_ARG;
    if (no_q && no_k) return MOE_OK;
    return cuda_status(launch_norm_rope(q, q_strides, k, k_strides, q_weight, k_weight, positions, inv_freq, rot,
                                        interleaved != 0, eps, q_out, q_out_strides, k_out, k_out_strides, T, Hq, Hkv,
                                        D, reinterpret_cast<cudaStream_t>(stream)));
}

int moe_kv4_append(const uint16_t *k, moe_strides k_strides, const uint16_t *v, moe_strides v_strides,
                   const int32_t *slots, int32_t T, moe_kv4_cache cache, void *ws, size_t ws_bytes, void *stream) {
    if (T < 0) return MOE_ERR_INVALID_ARG;
    int rc = check_cache(cache);
    if (rc) return rc;
    if (T > (1 << 20)) return MOE_ERR_UNSUPPORTED;
    if (!rows_ok(k, k_strides, T == 0) || !rows_ok(v, v_strides, T == 0) || (T > 0 && !aligned4(slots)))
        return MOE_ERR_INVALID_ARG;
    if ((rc = check_rows_ws(ws, ws_bytes))) return rc;
    if (T == 0) return MOE_OK;
    return cuda_status(launch_kv4_append(k, k_strides, v, v_strides, slots, T, cache, reinterpret_cast<Ctrl *>(ws),
                                         reinterpret_cast<cudaStream_t>(stream)));
}

int moe_kv4_read(const int32_t *slots, int32_t T, moe_kv4_cache cache, uint16_t *k, uint16_t *v, void *ws,
                 size_t ws_bytes, void *stream) {
    if (T < 0) return MOE_ERR_INVALID_ARG;
    int rc = check_cache(cache);
    if (rc) return rc;
    if (T > (1 << 20)) return MOE_ERR_UNSUPPORTED;
    if (!ptr_ok(k, T == 0) || !ptr_ok(v, T == 0) || (T > 0 && !aligned4(slots))) return MOE_ERR_INVALID_ARG;
    if ((rc = check_rows_ws(ws, ws_bytes))) return rc;
    if (T == 0) return MOE_OK;
    return cuda_status(launch_kv4_read(slots, T, cache, k, v, reinterpret_cast<Ctrl *>(ws),
                                       reinterpret_cast<cudaStream_t>(stream)));
}

int moe_kv4_workspace_size(int32_t T, int32_t Hq, int32_t Hkv, int32_t D, size_t *bytes) {
    if (!bytes || T < 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv) return MOE_ERR_INVALID_ARG;
    if ((D != 64 && D != 128) || Hq / Hkv > 32 || T > (1 << 20) || Hkv > 1024) return MOE_ERR_UNSUPPORTED;
    *bytes = kv4_workspace_bytes(T, Hq, Hkv, D);
    return MOE_OK;
}

int moe_kv4_attention_window(const uint16_t *q, moe_strides q_strides, moe_kv4_cache cache, const int32_t *page_table,
                             int32_t max_pages, const int32_t *lens, const int32_t *cu_q, int32_t B, int32_t T,
                             int32_t Hq, int32_t max_q, float scale, int32_t window, int32_t sinks, uint16_t *out,
                             moe_strides out_strides, float *lse, void *ws, size_t ws_bytes, void *stream) {
    if (window < 1 || sinks < 0) return MOE_ERR_INVALID_ARG;
    int rc = check_cache(cache);
    if (rc) return rc;
    size_t need = 0;
    if ((rc = moe_kv4_workspace_size(T, Hq, cache.Hkv, cache.D, &need))) return rc;
    if (B < 0 || max_pages < 0 || max_q < 0 || (!cu_q && T != B) || (T > 0 && B == 0) || !(fabsf(scale) <= 3.4e38f))
        return MOE_ERR_INVALID_ARG;
    if (B > 4096 || (int64_t)max_pages * cache.page_size >= ((int64_t)1 << 31)) return MOE_ERR_UNSUPPORTED;
    if (!rows_ok(q, q_strides, T == 0) || !out_rows_ok(out, out_strides, T, Hq, cache.D)) return MOE_ERR_INVALID_ARG;
    if (T > 0 && (!aligned4(lens) || (cu_q && !aligned4(cu_q)) || (max_pages > 0 && !aligned4(page_table)) ||
                  (lse && !aligned4(lse))))
        return MOE_ERR_INVALID_ARG;
    if (!ws || !aligned16(ws)) return MOE_ERR_INVALID_ARG;
    if (ws_bytes < need) return MOE_ERR_WORKSPACE;
    if (T == 0) return MOE_OK;
    // a window (or first keys) that every length fits hides nothing
    if (window >= max_pages * cache.page_size || sinks >= max_pages * cache.page_size) window = sinks = 0;
    return cuda_status(launch_kv4_attention(q, q_strides, cache, page_table, max_pages, lens, cu_q, B, T, Hq, max_q,
                                            scale, out, out_strides, lse, ws,
                                            reinterpret_cast<cudaStream_t>(stream), window, sinks));
}

int moe_kv4_attention(const uint16_t *q, moe_strides q_strides, moe_kv4_cache cache, const int32_t *page_table,
                      int32_t max_pages, const int32_t *lens, const int32_t *cu_q, int32_t B, int32_t T, int32_t Hq,
                      int32_t max_q, float scale, uint16_t *out, moe_strides out_strides, float *lse, void *ws,
                      size_t ws_bytes, void *stream) {
    return moe_kv4_attention_window(q, q_strides, cache, page_table, max_pages, lens, cu_q, B, T, Hq, max_q, scale,
                                    INT32_MAX, 0, out, out_strides, lse, ws, ws_bytes, stream);
}

int moe_verify_workspace_size(int32_t B, int32_t T, int32_t V, size_t *bytes) {
    if (!bytes || B < 0 || T < 0 || V <= 0) return MOE_ERR_INVALID_ARG;
    if (B > 4096 || T > 65536 || V > (1 << 20)) return MOE_ERR_UNSUPPORTED;
    *bytes = verify_workspace_bytes(B, T, V);
    return MOE_OK;
}

int moe_verify_drafts(const uint16_t *logits, int64_t logits_stride, const uint16_t *draft_logits, int64_t draft_stride,
                      const int32_t *drafts, const int32_t *cu_rows, const float *temperature, const float *uniform,
                      const float *noise, int64_t noise_stride, int32_t B, int32_t T, int32_t V, int32_t *tokens,
                      int32_t *accepted, void *ws, size_t ws_bytes, void *stream) {
    size_t need = 0;
    const int rc = moe_verify_workspace_size(B, T, V, &need);
    if (rc) return rc;
    // rows of 16-byte pieces, a stride that a row fits
    const auto rows_bad = [](int64_t stride, int rows, int V, int piece) {
        return stride < 0 || stride % piece || (rows > 1 && stride < V);
    };
    if (rows_bad(logits_stride, T, V, 8) || (draft_logits && rows_bad(draft_stride, T, V, 8)) || rows_bad(noise_stride, B, V, 4))
        return MOE_ERR_INVALID_ARG;
    if (!ptr_ok(logits, T == 0) || !ptr_ok(noise, B == 0) || (draft_logits && !aligned16(draft_logits)))
        return MOE_ERR_INVALID_ARG;
    if ((T > 0 && (!aligned4(drafts) || !aligned4(uniform) || !aligned4(tokens))) ||
        (B > 0 && (!aligned4(cu_rows) || !aligned4(accepted))) || (reinterpret_cast<uintptr_t>(temperature) & 3u))
        return MOE_ERR_INVALID_ARG;
    if (!ws || !aligned16(ws)) return MOE_ERR_INVALID_ARG;
    if (ws_bytes < need) return MOE_ERR_WORKSPACE;
    if (B == 0) return MOE_OK;
    const VerifyArgs a{logits, draft_logits, logits_stride, draft_stride, noise_stride, drafts, cu_rows,
                       temperature, uniform, noise, tokens, accepted};
    return cuda_status(launch_verify(a, B, T, V, ws, reinterpret_cast<cudaStream_t>(stream)));
}

int moe_profile_events(void *before_experts, void *after_experts) {
    if ((before_experts == nullptr) != (after_experts == nullptr)) return MOE_ERR_INVALID_ARG;
    g_ev_before = reinterpret_cast<cudaEvent_t>(before_experts);
    g_ev_after = reinterpret_cast<cudaEvent_t>(after_experts);
    return MOE_OK;
}

int moe_check_device_error(void *ws, size_t ws_bytes, void *stream) {
    if (!ws || !aligned16(ws) || ws_bytes < sizeof(Ctrl)) return MOE_ERR_INVALID_ARG;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    uint32_t err_word = 0;
    if (cudaMemcpyAsync(&err_word, ws, sizeof(err_word), cudaMemcpyDeviceToHost, s) != cudaSuccess)
        return MOE_ERR_CUDA;
    if (cudaStreamSynchronize(s) != cudaSuccess) return MOE_ERR_CUDA;
    if (err_word) {
        // A wait that gave up may leave completion counters anywhere in the
        // workspace non-zero; the whole workspace is cleared so that the next
        // call starts from the all-zero state. A bad id leaves the counters
        // consistent: only the error word is cleared.
        const size_t clear = err_word == MOE_ERR_TIMEOUT ? ws_bytes : sizeof(err_word);
        if (cudaMemsetAsync(ws, 0, clear, s) != cudaSuccess) return MOE_ERR_CUDA;
        if (cudaStreamSynchronize(s) != cudaSuccess) return MOE_ERR_CUDA;
        return err_word == MOE_ERR_TIMEOUT ? MOE_ERR_TIMEOUT : MOE_ERR_DEVICE;
    }
    return MOE_OK;
}

}  // extern "C"
