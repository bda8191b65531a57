// Host-side launchers of the calls that a step with drafted tokens adds to the
// MoE block and the attention block (w4a16.cu, verify.cu; all enqueue on `s`).
#pragma once
#include "common.cuh"
#include "kernels.cuh"

namespace moe {

// What a call keeps in a workspace lies behind the regions that calls leave at
// zero, so that one workspace may serve the experts' and the attention's calls too.
constexpr size_t kBehindZero = 512 + (size_t)kMaxE * kCtrStride * 4;

// y = x . W^T with INT4 weights (w4a16.cu).
size_t w4a16_workspace_bytes(int T, int N, int K);
cudaError_t launch_w4a16(const uint16_t *x, const int32_t *w, const uint16_t *scales, uint16_t *y, int T, int N, int K,
                         void *ws, cudaStream_t s);

// Verification of drafted tokens (verify.cu). Strides of rows in values.
struct VerifyArgs {
    const uint16_t *logits, *draft;
    long long ls, ds, ns;
    const int32_t *drafts, *cu;
    const float *temperature, *uniform, *noise;
    int32_t *tokens, *accepted;
};
size_t verify_workspace_bytes(int B, int T, int V);
cudaError_t launch_verify(const VerifyArgs &a, int B, int T, int V, void *ws, cudaStream_t s);

}  // namespace moe
