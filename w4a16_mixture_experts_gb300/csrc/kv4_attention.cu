// Attention over the paged 4-bit cache: which kernel runs, and its workspace.
//
// Query i of a sequence with nq queries and len keys sits at position
// len - nq + i and sees the keys up to it: out = sum_j softmax(scale q.k_j) v_j,
// lse = log sum_j exp(scale q.k_j); without a key out = 0 and lse = -inf.
#include "kv4_attention.cuh"

namespace moe {

cudaError_t launch_kv4_decode(const kv4::Attn &p, int rows, cudaStream_t s);
cudaError_t launch_kv4_prompt(const kv4::Attn &p, cudaStream_t s);

size_t kv4_workspace_bytes(int T, int Hq, int Hkv, int D) {
    using namespace kv4;
    const bool few = (long long)T * (Hq / Hkv) <= kDecodeRows;
    const size_t stream = 2 * kMaxCtas * sizeof(float) * (size_t)part_floats(kDecodeRows, D);
    const size_t prompt = 2 * kMaxPromptCtas * sizeof(float) * (size_t)part_floats(kPromptRows, D);
    return align_up(kPartOff + (few ? stream : prompt), 256);
}

cudaError_t launch_kv4_attention(const uint16_t *q, moe_strides qs, const moe_kv4_cache &c, const int32_t *table,
                                 int max_pages, const int32_t *lens, const int32_t *cu_q, int B, int T, int Hq,
                                 int max_q, float scale, uint16_t *out, moe_strides os, float *lse, void *ws,
                                 cudaStream_t s) {
    using namespace kv4;
    const int G = Hq / c.Hkv;
    const long long rows = (long long)(max_q < T ? max_q : T) * G;
    const Attn p{{table, lens, cu_q, B, T, max_pages, __builtin_ctz((unsigned)c.page_size)}, q, qs, os, c, out, lse,
                 reinterpret_cast<Ctrl *>(ws), ws_at<uint32_t>(ws, kTicketOff), ws_at<float>(ws, kPartOff), scale, Hq, G};
    return rows <= kDecodeRows ? launch_kv4_decode(p, (int)rows, s) : launch_kv4_prompt(p, s);
}

}  // namespace moe
