// W4A16 linear layers: y = x . W^T with weights in the experts' storage (INT4,
// a bf16 scale per 128 values of a row, q + 8, eight to a word, lowest nibble
// first).
//
//   y[t][n] = sum_g s[n][g] * (sum over the 128 c of group g: q[n][c] x[t][c])
//
// A code is exact in bf16, so the inner sums' products are exact and they add up
// in fp32; a scale multiplies its group's sum in fp32: nothing is rounded to
// fewer bits before y.
//
// A first form for every T: what bounds it is L1, from which every warp takes x again
// (90% busy at 4 x 248320 x 2560, 84 us of a floor of 49; 99.7% at 4001 x 5121 x 4096,
// 1552 us of 85), and where few rows leave SMs idle, each load's latency (7 x 2560 x
// 10240: 35 us of 2). K is not split, and nothing is loaded ahead.
#include "step_kernels.cuh"

namespace moe {

namespace {

constexpr int kWarps = 8;

struct Params {
    const uint16_t *x;     // bf16 [T][K]
    const uint32_t *w;     // [N][K / 8]
    const uint16_t *s;     // bf16 [N][K / 128]
    uint16_t *y;           // bf16 [T][N]
    int T, N, K;
};

__device__ inline uint16_t bf16_of(float v) {
    const __nv_bfloat16 h = __float2bfloat16_rn(v);
    return *reinterpret_cast<const uint16_t *>(&h);
}

// A warp takes 16 rows (M) and 8 tokens (N) through all of K with mma.sync
// m16n8k16. Lane (g, t) reads 16 bytes of rows g and g + 8 of each group: words
// 4 t .. 4 t + 3. A word's pairs (j, j + 4) fill the A fragments of two steps, and
// the B fragments take x's values in the same order.
__global__ void __launch_bounds__(kWarps * 32) w4a16_kernel(Params p) {
    const int lane = threadIdx.x & 31, g = lane >> 2, tig = lane & 3;
    const int blk = blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (blk * 16 >= p.N) return;
    const int G = p.K / kGroup, r0 = blk * 16 + g, r1 = r0 + 8;
    const bool v0 = r0 < p.N, v1 = r1 < p.N;
    const uint4 *w0 = reinterpret_cast<const uint4 *>(p.w + (size_t)(v0 ? r0 : 0) * (p.K / 8)) + tig;
    const uint4 *w1 = reinterpret_cast<const uint4 *>(p.w + (size_t)(v1 ? r1 : 0) * (p.K / 8)) + tig;
    const uint16_t *s0 = p.s + (size_t)(v0 ? r0 : 0) * G, *s1 = p.s + (size_t)(v1 ? r1 : 0) * G;
    for (int t0 = blockIdx.y * 8; t0 < p.T; t0 += gridDim.y * 8) {
        const uint4 *x = reinterpret_cast<const uint4 *>(p.x + (size_t)min(t0 + g, p.T - 1) * p.K) + tig * 4;
        float acc[4] = {0.f, 0.f, 0.f, 0.f};
        for (int k = 0; k < G; ++k) {
            const uint4 a = w0[k * 4], b = w1[k * 4];
            const uint32_t wa[4] = {a.x, a.y, a.z, a.w}, wb[4] = {b.x, b.y, b.z, b.w};
            float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const uint4 v = x[k * 16 + m];
                const uint32_t f0[4] = {int4_pair(wa[m], 0), int4_pair(wb[m], 0), int4_pair(wa[m], 1), int4_pair(wb[m], 1)};
                const uint32_t f1[4] = {int4_pair(wa[m], 2), int4_pair(wb[m], 2), int4_pair(wa[m], 3), int4_pair(wb[m], 3)};
                mma_bf16_16816(c, f0, __byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632));
                mma_bf16_16816(c, f1, __byte_perm(v.y, v.w, 0x5410), __byte_perm(v.y, v.w, 0x7632));
            }
            const float fa = bf16_bits_to_f32(s0[k]), fb = bf16_bits_to_f32(s1[k]);
            acc[0] = fmaf(fa, c[0], acc[0]);
            acc[1] = fmaf(fa, c[1], acc[1]);
            acc[2] = fmaf(fb, c[2], acc[2]);
            acc[3] = fmaf(fb, c[3], acc[3]);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int t = t0 + 2 * tig + i;
            if (t < p.T && v0) p.y[(size_t)t * p.N + r0] = bf16_of(acc[i]);
            if (t < p.T && v1) p.y[(size_t)t * p.N + r1] = bf16_of(acc[2 + i]);
        }
    }
}

}  // namespace

size_t w4a16_workspace_bytes(int, int, int) { return sizeof(Ctrl); }

cudaError_t launch_w4a16(const uint16_t *x, const int32_t *w, const uint16_t *scales, uint16_t *y, int T, int N, int K,
                         void *, cudaStream_t s) {
    const Params p{x, reinterpret_cast<const uint32_t *>(w), scales, y, T, N, K};
    const int blocks = (N + 15) / 16, tiles = (T + 7) / 8;
    w4a16_kernel<<<dim3((unsigned)((blocks + kWarps - 1) / kWarps), (unsigned)(tiles < 65535 ? tiles : 65535)), kWarps * 32, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace moe
