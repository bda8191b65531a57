// Attention over the paged 4-bit cache: which kernel runs, its workspace, and
// the join of items that several CTAs worked on.
//
// Query i of a sequence with nq queries and len keys sits at position
// len - nq + i and sees the keys up to it: out = sum_j softmax(scale q.k_j) v_j,
// lse = log sum_j exp(scale q.k_j); without a key out = 0 and lse = -inf.
#include "kv4_attention.cuh"

namespace moe {

cudaError_t launch_kv4_decode(const kv4::Attn &p, int rows, int *rows_at, int *grid, cudaStream_t s);
cudaError_t launch_kv4_prompt(const kv4::Attn &p, int *grid, cudaStream_t s);

namespace {

using namespace kv4;

constexpr int kJoinThreads = 128;

// Block (c, y): rows y of the item that CTA c began. D / 4 lanes have a row, four
// values each; a lane finds the weight of one part of D / 4 at a time, and the
// first parts' values are under way meanwhile.
template <int D>
__global__ void __launch_bounds__(kJoinThreads) kv4_join_kernel(Attn p, int R) {
    constexpr int G = D / 4, kRows = kJoinThreads / G, kAt = 8;   // parts under way at once
    const int c = blockIdx.x, g = threadIdx.x % G, r = blockIdx.y * kRows + threadIdx.x / G;
    pdl_wait();
    pdl_launch_dependents();
    const Begun it = p.begun[c];
    if (it.last == 0 || (int)(blockIdx.y * kRows) >= it.rows) return;
    const int n = it.last - c + 1, row = min(r, it.rows - 1);   // (lanes without a row follow one)
    const size_t N = (size_t)part_floats(R, D);
    const float *const first = p.part + (size_t)(c * 2 + 1) * N, *const rest = p.part + (size_t)c * 2 * N;
    auto part = [&](int i) { return i == 0 ? first : rest + (size_t)i * 2 * N; };
    const size_t value = 2 * R + 4 + (size_t)row * D + g * 4;
    float M = kNoMax, L = 0.f;
    int F = 1;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = 0; i0 < n; i0 += G) {
        float4 v[kAt];
#pragma unroll
        for (int k = 0; k < kAt; ++k) v[k] = __ldcg(reinterpret_cast<const float4 *>(part(min(i0 + k, n - 1)) + value));
        const bool in = i0 + g < n;
        const float *q = part(in ? i0 + g : i0);
        const float m = in ? __ldcg(q + row) : kNoMax, l = in ? __ldcg(q + R + row) : 0.f;
        const int f = in ? __float_as_int(__ldcg(q + 2 * R)) : 1;
        float Mn = fmaxf(M, m);
        int Fn = max(F, f);
#pragma unroll
        for (int o = G / 2; o > 0; o >>= 1) {
            Mn = fmaxf(Mn, __shfl_xor_sync(0xffffffffu, Mn, o));
            Fn = max(Fn, __shfl_xor_sync(0xffffffffu, Fn, o));
        }
        // (halves: a sum of probabilities may be far above 1, its weight below fp32's range)
        const float w2 = exp2_approx(0.5f * (m - Mn)), down2 = exp2_approx(0.5f * (M - Mn)), w = w2 * w2, down = down2 * down2;
        float sum = l * w2 * w2;
#pragma unroll
        for (int o = G / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        L = L * down2 * down2 + sum;
        const float wv = Fn - f > 126 ? 0.f : w * pow2_biased(127 + f - Fn), dv = Fn - F > 126 ? 0.f : down * pow2_biased(127 + F - Fn);
        acc = make_float4(acc.x * dv, acc.y * dv, acc.z * dv, acc.w * dv);
        M = Mn;
        F = Fn;
        const int here = min(G, n - i0);
        for (int k0 = 0;;) {
#pragma unroll
            for (int k = 0; k < kAt; ++k) {
                const float x = __shfl_sync(0xffffffffu, wv, k0 + k, G);
                if (k0 + k < here) {
                    acc.x = fmaf(v[k].x, x, acc.x);
                    acc.y = fmaf(v[k].y, x, acc.y);
                    acc.z = fmaf(v[k].z, x, acc.z);
                    acc.w = fmaf(v[k].w, x, acc.w);
                }
            }
            if ((k0 += kAt) >= here) break;
#pragma unroll
            for (int k = 0; k < kAt; ++k) v[k] = __ldcg(reinterpret_cast<const float4 *>(part(min(i0 + k0 + k, n - 1)) + value));
        }
    }
    if (r >= it.rows) return;
    const int rr = it.qt * R + r, i = rr / p.G, head = it.h * p.G + rr - i * p.G;
    const size_t tok = (size_t)(it.q0 + i);
    const float inv = L == 0.f ? 0.f : 1.f / L, up = pow2_biased(F);
    *reinterpret_cast<uint2 *>(p.out + tok * p.os.token + (size_t)head * p.os.head + g * 4) =
        make_uint2(bf16x2_of(acc.x * inv * up, acc.y * inv * up), bf16x2_of(acc.z * inv * up, acc.w * inv * up));
    if (g == 0 && p.lse) p.lse[tok * p.Hq + head] = L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
}

template <int D>
cudaError_t launch_join(const Attn &p, int R, int grid, cudaStream_t s) {
    constexpr int kRows = kJoinThreads / (D / 4);   // of a block
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid, (unsigned)((R + kRows - 1) / kRows));
    cfg.blockDim = dim3(kJoinThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kv4_join_kernel<D>, p, R);
}

}  // namespace

size_t kv4_workspace_bytes(int T, int Hq, int Hkv, int D) {
    if (T == 0) return sizeof(Ctrl);   // (nothing is launched)
    const bool few = (long long)T * (Hq / Hkv) <= kDecodeRows;
    const size_t stream = 2 * kMaxCtas * sizeof(float) * (size_t)part_floats(kDecodeRows, D);
    const size_t prompt = 2 * kMaxPromptCtas * sizeof(float) * (size_t)part_floats(kPromptRows, D);
    return align_up(kPartOff + kMaxCtas * sizeof(Begun) + (few || stream > prompt ? stream : prompt), 256);
}

cudaError_t launch_kv4_attention(const uint16_t *q, moe_strides qs, const moe_kv4_cache &c, const int32_t *table,
                                 int max_pages, const int32_t *lens, const int32_t *cu_q, int B, int T, int Hq,
                                 int max_q, float scale, uint16_t *out, moe_strides os, float *lse, void *ws,
                                 cudaStream_t s, int window, int sinks) {
    const int G = Hq / c.Hkv;
    const long long rows = (long long)(max_q < T ? max_q : T) * G;
    const Attn p{{table, lens, cu_q, B, T, max_pages, __builtin_ctz((unsigned)c.page_size)}, q, qs, os, c, out, lse,
                 reinterpret_cast<Ctrl *>(ws), ws_at<Begun>(ws, kPartOff), ws_at<float>(ws, kPartOff + kMaxCtas * sizeof(Begun)), scale, Hq, G,
                 window, sinks};
    int R = kPromptRows, grid = 0;
    const cudaError_t err = rows <= kDecodeRows ? launch_kv4_decode(p, (int)rows, &R, &grid, s) : launch_kv4_prompt(p, &grid, s);
    if (err != cudaSuccess) return err;
    return c.D == 64 ? launch_join<64>(p, R, grid, s) : launch_join<128>(p, R, grid, s);
}

}  // namespace moe
