// Attention over the paged 4-bit cache.
//
// Query i of a sequence with nq queries and len keys sits at position
// len - nq + i and sees the keys up to it: out = sum_j softmax(scale q.k_j) v_j,
// lse = log sum_j exp(scale q.k_j); without a key out = 0 and lse = -inf.
#include "kv4_attention.cuh"

namespace moe {

cudaError_t launch_kv4_decode(const kv4::Attn &p, int rows, cudaStream_t s);

namespace {

using kv4::Attn;

// One CTA of 128 threads a row (query, head): a thread scores one key of each
// 128, then adds up one value column.
template <int D>
__global__ void __launch_bounds__(128) attention_rows_kernel(Attn p) {
    __shared__ float s_q[D], s_p[128], s_vs[128], s_red[4];
    __shared__ long long s_at[128];
    __shared__ int s_b;
    const int t = blockIdx.x, hq = blockIdx.y, h = hq / p.G, tid = threadIdx.x;
    pdl_wait();
    pdl_launch_dependents();
    if (tid == 0) {
        int lo = 0;
        if (p.b.cu_q)
            for (int hi = p.b.B; hi - lo > 1;) {
                const int mid = (lo + hi) / 2;
                if (p.b.cu_q[mid] <= t) lo = mid;
                else hi = mid;
            }
        else lo = t;
        s_b = lo;
    }
    if (tid < D) s_q[tid] = bf16_bits_to_f32(p.q[(size_t)t * p.qs.token + (size_t)hq * p.qs.head + tid]);
    __syncthreads();
    const int b = s_b;
    const kv4::Seq sq = kv4::seq_of(p.b, b, p.ctrl);
    if (t < sq.q0 || t >= sq.q0 + sq.nq) return;
    const int keys = sq.len - sq.nq + (t - sq.q0) + 1;
    float m = -INFINITY, l = 0.f, acc = 0.f;
    for (int k0 = 0; k0 < keys; k0 += 128) {
        const int j = k0 + tid;
        float x = -INFINITY, vs = 0.f;
        long long at = -1;
        if (j < keys) {
            const int page = p.b.table[(size_t)b * p.b.max_pages + (j >> p.b.shift)];
            if (page < 0 || page >= p.c.n_pages) {
                set_error(p.ctrl, MOE_ERR_DEVICE);
                x = 0.f;
            } else {
                at = (((long long)page * p.c.Hkv + h) << p.b.shift) + (j & ((1 << p.b.shift) - 1));
                float dot = 0.f;
                for (int w = 0; w < D / 8; ++w) {
                    const uint32_t word = (uint32_t)p.c.k_codes[at * (D / 8) + w];
                    for (int i = 0; i < 8; ++i) dot = fmaf((float)((int)(word >> (4 * i) & 15u) - 8), s_q[w * 8 + i], dot);
                }
                const uint16_t ksb = p.c.k_scales[at], vsb = p.c.v_scales[at];
                x = dot * bf16_bits_to_f32(ksb) * p.scale;
                vs = bf16_bits_to_f32(vsb);
                if (!kv4::finite_bits(ksb) || !kv4::finite_bits(vsb)) {
                    x = NAN;
                    vs = 0.f;
                }
            }
        }
        float mx = x;
        for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        if ((tid & 31) == 0) s_red[tid >> 5] = mx;
        __syncthreads();
        const float mn = fmaxf(m, fmaxf(fmaxf(s_red[0], s_red[1]), fmaxf(s_red[2], s_red[3])));
        const float mu = mn == -INFINITY ? 0.f : mn;
        const float e = __expf(x - mu);
        float sum = e;
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        __syncthreads();
        if ((tid & 31) == 0) s_red[tid >> 5] = sum;
        s_p[tid] = e;
        s_vs[tid] = vs;
        s_at[tid] = at;
        __syncthreads();
        const float f = __expf(m - mu);
        l = l * f + s_red[0] + s_red[1] + s_red[2] + s_red[3];
        m = mn;
        if (tid < D) {
            acc *= f;
            for (int i = 0; i < min(128, keys - k0); ++i)
                if (s_at[i] >= 0 || s_p[i] != s_p[i]) {
                    const float v = s_at[i] >= 0 ? (float)((int)((uint32_t)p.c.v_codes[s_at[i] * (D / 8) + tid / 8] >> (4 * (tid & 7)) & 15u) - 8) : 0.f;
                    acc = fmaf(s_p[i] * s_vs[i], v, acc);
                }
        }
        __syncthreads();
    }
    const bool none = keys <= 0;
    if (tid < D) {
        const __nv_bfloat16 o = __float2bfloat16_rn(none ? 0.f : acc / l);
        p.out[(size_t)t * p.os.token + (size_t)hq * p.os.head + tid] = *reinterpret_cast<const uint16_t *>(&o);
    }
    if (tid == 0 && p.lse) p.lse[(size_t)t * p.Hq + hq] = none ? -INFINITY : m + logf(l);
}

}  // namespace

// The rows that share one pass over their keys decide: up to 32 of a sequence
// go to the streaming kernel.
constexpr int kDecodeRows = 32;

size_t kv4_workspace_bytes(int T, int Hq, int Hkv, int D) {
    (void)T, (void)Hq, (void)Hkv;
    return align_up(kv4::kPartOff + sizeof(float) * 2 * kv4::kMaxCtas * kv4::part_floats(kDecodeRows, D), 256);
}

cudaError_t launch_kv4_attention(const uint16_t *q, moe_strides qs, const moe_kv4_cache &c, const int32_t *table,
                                 int max_pages, const int32_t *lens, const int32_t *cu_q, int B, int T, int Hq,
                                 int max_q, float scale, uint16_t *out, moe_strides os, float *lse, void *ws,
                                 cudaStream_t s) {
    const int G = Hq / c.Hkv;
    Attn p{{table, lens, cu_q, B, T, max_pages, __builtin_ctz((unsigned)c.page_size)}, q, qs, os, c, out, lse,
           reinterpret_cast<Ctrl *>(ws), ws_at<uint32_t>(ws, kv4::kTicketOff), ws_at<float>(ws, kv4::kPartOff), scale, Hq, G};
    if ((long long)max_q * G <= kDecodeRows) return launch_kv4_decode(p, max_q * G, s);
    const dim3 grid(T, Hq);
    return c.D == 64 ? launch_pdl(attention_rows_kernel<64>, grid, 128, 0, s, p)
                     : launch_pdl(attention_rows_kernel<128>, grid, 128, 0, s, p);
}

}  // namespace moe
