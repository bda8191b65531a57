// Host-side launchers of the attention block's kernels (attn_rows.cu,
// kv4_attention.cu; all enqueue on `s`).
#pragma once
#include "kernels.cuh"

namespace moe {

cudaError_t launch_norm_rope(const uint16_t *q, moe_strides qs, const uint16_t *k, moe_strides ks, const uint16_t *qw,
                             const uint16_t *kw, const int32_t *pos, const float *inv_freq, int rot, bool interleaved,
                             float eps, uint16_t *qo, moe_strides qos, uint16_t *ko, moe_strides kos, int T, int Hq,
                             int Hkv, int D, cudaStream_t s);
cudaError_t launch_kv4_append(const uint16_t *k, moe_strides ks, const uint16_t *v, moe_strides vs,
                              const int32_t *slots, int T, const moe_kv4_cache &c, struct Ctrl *ctrl, cudaStream_t s);
cudaError_t launch_kv4_read(const int32_t *slots, int T, const moe_kv4_cache &c, uint16_t *k, uint16_t *v,
                            struct Ctrl *ctrl, cudaStream_t s);
size_t kv4_workspace_bytes(int T, int Hq, int Hkv, int D);
cudaError_t launch_kv4_attention(const uint16_t *q, moe_strides qs, const moe_kv4_cache &c, const int32_t *table,
                                 int max_pages, const int32_t *lens, const int32_t *cu_q, int B, int T, int Hq,
                                 int max_q, float scale, uint16_t *out, moe_strides os, float *lse, void *ws,
                                 cudaStream_t s);

// A launch that may start while the kernel ahead of it in the stream ends: the
// kernel calls pdl_wait() before it reads or writes anything.
template <typename P>
cudaError_t launch_pdl(void (*kernel)(P), dim3 grid, int threads, size_t smem, cudaStream_t s, const P &p) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace moe
