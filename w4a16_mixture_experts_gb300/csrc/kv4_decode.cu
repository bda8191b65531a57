// Attention over the paged 4-bit cache for few query rows a sequence (a decode
// step, or a few draft tokens): up to 32 rows (query, head of the group) share
// one pass over their keys.
//
// What bounds it: a key costs D + 4 bytes of HBM for all its rows, so the
// stream of codes; the dequantisation of its 2 D values is the next (about
// 1.2 instructions a value), so the codes go from global memory to registers in
// the very fragments that mma.sync takes, with the queries as the narrow side:
//   S^T (16 keys x 8 rows) = K (16 keys x D) . Q^T,  O^T (D x 8) += V^T . P^T.
// The lane (g, t) = (lane / 4, lane % 4) of a warp loads 16 consecutive bytes of
// keys g and g + 8 for K, and 8 bytes of keys 2t, 2t+1, 2t+8, 2t+9 for V; the
// order of the D values inside the product is whatever that gives, the same for
// both sides. Codes enter the product exactly, in fp16; a K scale multiplies its
// key's scores in fp32, a V scale its key's probability just before that is
// rounded to fp16, less the exponent F of the largest V scale so far (a whole
// power of two, put back at the end), so that no range of scales is lost. Query
// rows enter as fp16 too, exactly: each less its own exponent.
#include "kv4_attention.cuh"

namespace moe {

namespace {

using namespace kv4;

constexpr int kStep = 16;   // keys of a unit: one warp's step

template <int D, int NT>
struct DecodeCfg {
    static constexpr int kWarps = NT == 1 ? 8 : NT == 2 ? 6 : 4;   // registers: 128, 168, 255 a thread
    static constexpr int kThreads = kWarps * 32;
    static constexpr int kRows = NT * 8;
    static constexpr int kStride = D + 4;                // of a row of partial values in shared memory
    static constexpr int kKW = D / 32, kVW = D / 64;     // words a lane loads of a K row and of a V row
    static constexpr size_t kSmem = sizeof(float) * (size_t)kWarps * kRows * kStride;
};

__device__ inline void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ inline uint32_t transpose8x8(uint32_t v) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

__device__ inline uint32_t half2_of(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

template <int N>
__device__ inline void load_words(uint32_t (&w)[N], const int32_t *p) {
    if constexpr (N == 4) {
        const uint4 v = ld_nc_v4(p);
        w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else if constexpr (N == 2) {
        const uint2 v = __ldg(reinterpret_cast<const uint2 *>(p));
        w[0] = v.x, w[1] = v.y;
    } else {
        w[0] = (uint32_t)__ldg(p);
    }
}

// One step's codes and scales, as loaded.
template <int D>
struct Step {
    uint32_t k[2][D / 32], v[4][D / 64];
    uint16_t scale;   // lanes 0-15: K of key `lane`; 16-31: V of key `lane - 16`
};

template <int D, int NT>
__global__ void __launch_bounds__(DecodeCfg<D, NT>::kThreads, 2) kv4_decode_kernel(Attn p) {
    using Cfg = DecodeCfg<D, NT>;
    constexpr int W = Cfg::kWarps, R = Cfg::kRows, KW = Cfg::kKW, VW = Cfg::kVW;
    extern __shared__ float s_o[];   // [W][R][kStride], then the sequences' prefix
    long long *const s_pre = reinterpret_cast<long long *>(reinterpret_cast<char *>(s_o) + Cfg::kSmem);
    __shared__ uint4 s_q[NT][KW][32];   // query fragments
    __shared__ float s_c[R], s_m[W][R], s_l[W][R];
    __shared__ int s_lim[R], s_F[W];
    __shared__ long long s_sums[W];
    __shared__ int s_last;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;

    pdl_wait();
    pdl_launch_dependents();
    const long long U = scan_units<Cfg::kThreads, kStep>(p, R, s_pre, s_sums);
    // fewer CTAs where there is less than a step for each warp of them
    const int C = (int)min((long long)gridDim.x, max(1LL, (U + W - 1) / W));
    const int c = blockIdx.x;
    if (c >= C) return;
    const long long u_end = U * (c + 1) / C;

    long long u = U * c / C;
    if (u >= u_end) return;
    for (Item it = find_item<kStep>(p, R, s_pre, u); ; next_item<kStep>(p, R, it)) {
        const int st0 = (int)(u - it.first), st1 = (int)min((long long)it.units, u_end - it.first);
        const int rows = min(R, it.s.nq * p.G - it.qt * R);

        // ---- the rows' queries, as the fragments' fp16, and what each row sees
        for (int r = warp; r < R; r += W) {
            const int rr = it.qt * R + r, i = rr / p.G;
            float x[D / 32];
            uint32_t big = 0;
            if (r < rows) {
                const uint16_t *src = p.q + (size_t)(it.s.q0 + i) * p.qs.token + (size_t)(it.h * p.G + rr - i * p.G) * p.qs.head + lane * (D / 32);
#pragma unroll
                for (int j = 0; j < D / 32; j += 2) {
                    const uint32_t v = *reinterpret_cast<const uint32_t *>(src + j);
                    x[j] = __uint_as_float(v << 16);
                    x[j + 1] = __uint_as_float(v & 0xffff0000u);
                    big = max(big, max(v & 0x7FFFu, (v >> 16) & 0x7FFFu));
                }
            } else {
#pragma unroll
                for (int j = 0; j < D / 32; ++j) x[j] = 0.f;
            }
            const int e = norm_exponent(__reduce_max_sync(0xffffffffu, big));
            const float f = pow2_biased(254 - e);
            __half *dst = reinterpret_cast<__half *>(s_q);
#pragma unroll
            for (int j = 0; j < D / 32; ++j) {
                const int d = lane * (D / 32) + j, word = d >> 3, n = d & 7;
                dst[(((r >> 3) * KW + word % KW) * 32 + (r & 7) * 4 + word / KW) * 8 + (n & 3) * 2 + (n >> 2)] = __float2half_rn(x[j] * f);
            }
            if (lane == 0) {
                s_c[r] = p.scale * kLog2e * pow2_biased(e);
                s_lim[r] = r < rows ? it.s.len - it.s.nq + i + 1 : 0;
            }
        }
        __syncthreads();

        float cs[NT][2], m[NT][2], l[NT][2], o[NT][D / 16][4];
        int lim[NT][2], least = 0x7fffffff;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int r = n * 8 + 2 * t + j;
                cs[n][j] = s_c[r];
                lim[n][j] = s_lim[r];
                m[n][j] = kNoMax;
                l[n][j] = 0.f;
                least = min(least, lim[n][j]);
            }
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) o[n][i][j] = 0.f;
        }
        least = __reduce_min_sync(0xffffffffu, least);
        uint4 qf[NT == 1 ? KW : 1];
        if constexpr (NT == 1)
#pragma unroll
            for (int w = 0; w < KW; ++w) qf[w] = s_q[0][w][lane];
        int F = 1;   // biased exponent taken off the V scales

        const int32_t *table = p.b.table + (size_t)it.b * p.b.max_pages;
        const int pmask = (1 << p.b.shift) - 1, keys = it.s.len;
        auto page_of = [&](int st) { return st < st1 && st * kStep < keys ? __ldg(table + (st * kStep >> p.b.shift)) : 0; };
        auto fetch = [&](Step<D> &x, int st, int page) {
            const int key0 = st * kStep;
            const bool ok = key0 < keys && (unsigned)page < (unsigned)p.c.n_pages;
            const size_t row = ((((size_t)(ok ? page : 0) * p.c.Hkv + it.h) << p.b.shift) + (key0 & pmask));
            const int32_t *kp = p.c.k_codes + (row + g) * (D / 8) + t * KW;
            load_words(x.k[0], kp);
            load_words(x.k[1], kp + 8 * (D / 8));
            const int32_t *vp = p.c.v_codes + (row + 2 * t) * (D / 8) + g * VW;
            load_words(x.v[0], vp);
            load_words(x.v[1], vp + D / 8);
            load_words(x.v[2], vp + D);
            load_words(x.v[3], vp + D + D / 8);
            x.scale = __ldg((lane < 16 ? p.c.k_scales : p.c.v_scales) + row + (lane & 15));
            if (!ok || key0 + (lane & 15) >= keys) x.scale = 0;
            if (!ok && key0 < keys && lane == 0) set_error(p.ctrl, MOE_ERR_DEVICE);
        };

        int st = st0 + warp;
        Step<D> cur, nxt;
        if (st < st1) fetch(cur, st, page_of(st));
        int page = page_of(st + W);
        for (; st < st1; st += W) {
            if (st + W < st1) {
                fetch(nxt, st + W, page);
                page = page_of(st + 2 * W);
            }
            // ---- scales
            float f = bf16_bits_to_f32(cur.scale);
            const uint32_t bad = __ballot_sync(0xffffffffu, !finite_bits(cur.scale));
            if (bad) {   // a row that was not finite: its scores become NaN, its values zero
                if ((bad | bad >> 16 | bad << 16) >> lane & 1u) f = lane < 16 ? __uint_as_float(0x7fc00000u) : 0.f;
            }
            const int e = min((int)__reduce_max_sync(0xffffffffu, lane < 16 ? 0u : __float_as_uint(f) >> 23 & 0xFFu), 253);
            if (e > F) {
                const float down = e - F > 126 ? 0.f : pow2_biased(127 + F - e);
                F = e;
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < D / 16; ++i)
#pragma unroll
                        for (int j = 0; j < 4; ++j) o[n][i][j] *= down;
            }
            if (lane >= 16) f *= pow2_biased(254 - F);
            const float ks[2] = {__shfl_sync(0xffffffffu, f, g), __shfl_sync(0xffffffffu, f, g + 8)};
            const float vs[2] = {__shfl_sync(0xffffffffu, f, g + 16), __shfl_sync(0xffffffffu, f, g + 24)};

            // ---- S^T = K . Q^T
            float s[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j) s[n][j] = 0.f;
#pragma unroll
            for (int w = 0; w < KW; ++w) {
                const uint32_t x = cur.k[0][w], y = cur.k[1][w], x8 = x >> 8, y8 = y >> 8;
                const uint32_t a[4] = {nib_lo(x), nib_lo(y), nib_hi(x), nib_hi(y)};
                const uint32_t b[4] = {nib_lo(x8), nib_lo(y8), nib_hi(x8), nib_hi(y8)};
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    uint4 q;
                    if constexpr (NT == 1) q = qf[w];
                    else q = s_q[n][w][lane];
                    mma_f16(s[n], a, q.x, q.y);
                    mma_f16(s[n], b, q.z, q.w);
                }
            }
            // ---- probabilities; the maximum is moved only when a score passes it by 2^8
            const int key = st * kStep + g;
            const bool edge = st * kStep + kStep > least;
            bool over = false;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float x = s[n][j] * ks[j >> 1] * cs[n][j & 1];
                    if (edge && key + (j >> 1) * 8 >= lim[n][j & 1]) x = -INFINITY;
                    s[n][j] = x;
                    over |= x > m[n][j & 1] + 8.f;
                }
            if (__any_sync(0xffffffffu, over)) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        float x = fmaxf(fmaxf(s[n][j], s[n][j + 2]), m[n][j]);
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
                        const float down = exp2_approx(m[n][j] - x);
                        m[n][j] = x;
                        l[n][j] *= down;
#pragma unroll
                        for (int i = 0; i < D / 16; ++i) {
                            o[n][i][j] *= down;
                            o[n][i][j + 2] *= down;
                        }
                    }
            }
            uint32_t b0[NT], b1[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    s[n][j] = exp2_approx(s[n][j] - m[n][j & 1]);
                    l[n][j & 1] += s[n][j];
                    s[n][j] *= vs[j >> 1];
                }
                b0[n] = transpose8x8(half2_of(s[n][0], s[n][1]));
                b1[n] = transpose8x8(half2_of(s[n][2], s[n][3]));
            }
            // ---- O^T += V^T . P^T
#pragma unroll
            for (int w = 0; w < VW; ++w) {
                const uint32_t ab[2] = {__byte_perm(cur.v[0][w], cur.v[1][w], 0x5410), __byte_perm(cur.v[0][w], cur.v[1][w], 0x7632)};
                const uint32_t cd[2] = {__byte_perm(cur.v[2][w], cur.v[3][w], 0x5410), __byte_perm(cur.v[2][w], cur.v[3][w], 0x7632)};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t x = i & 1 ? ab[i >> 1] >> 8 : ab[i >> 1], y = i & 1 ? cd[i >> 1] >> 8 : cd[i >> 1];
                    const uint32_t a[4] = {nib_lo(x), nib_hi(x), nib_lo(y), nib_hi(y)};
#pragma unroll
                    for (int n = 0; n < NT; ++n) mma_f16(o[n][w * 4 + i], a, b0[n], b1[n]);
                }
            }
            cur = nxt;
        }

        // ---- the warps' rows, side by side in shared memory
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float x = l[n][j];
                x += __shfl_xor_sync(0xffffffffu, x, 4);
                x += __shfl_xor_sync(0xffffffffu, x, 8);
                x += __shfl_xor_sync(0xffffffffu, x, 16);
                const int r = n * 8 + 2 * t + j;
                if (g == 0) {
                    s_m[warp][r] = m[n][j];
                    s_l[warp][r] = x;
                }
                float *row = s_o + (warp * R + r) * Cfg::kStride + g * (8 * VW);
#pragma unroll
                for (int i = 0; i < D / 16; i += 2)
                    *reinterpret_cast<float4 *>(row + 2 * i) = make_float4(o[n][i][j], o[n][i][j + 2], o[n][i + 1][j], o[n][i + 1][j + 2]);
            }
        if (lane == 0) s_F[warp] = F;
        __syncthreads();
        int Fm = 1;
#pragma unroll
        for (int w = 0; w < W; ++w) Fm = max(Fm, s_F[w]);
        const bool whole = st0 == 0 && st1 == it.units;
        // a CTA's first part continues an item, its last one may begin one
        float *part = p.part + (size_t)(c * 2 + (st0 == 0)) * part_floats(R, D);
        for (int x = threadIdx.x; x < rows * (D / 4); x += Cfg::kThreads) {
            const int r = x / (D / 4), d = (x % (D / 4)) * 4;
            float M = kNoMax, L = 0.f;
#pragma unroll
            for (int w = 0; w < W; ++w) M = fmaxf(M, s_m[w][r]);
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < W; ++w) {
                const float f = exp2_approx(s_m[w][r] - M);
                L = fmaf(s_l[w][r], f, L);
                const float fv = Fm - s_F[w] > 126 ? 0.f : f * pow2_biased(127 + s_F[w] - Fm);
                const float4 v = *reinterpret_cast<const float4 *>(s_o + (w * R + r) * Cfg::kStride + d);
                acc.x = fmaf(v.x, fv, acc.x);
                acc.y = fmaf(v.y, fv, acc.y);
                acc.z = fmaf(v.z, fv, acc.z);
                acc.w = fmaf(v.w, fv, acc.w);
            }
            if (whole) {
                write_row4(p, it, R, r, d, acc, M, L, Fm);
            } else {
                *reinterpret_cast<float4 *>(part + 2 * R + 4 + r * D + d) = acc;
                if (d == 0) {
                    part[r] = M;
                    part[R + r] = L;
                }
                if (x == 0) part[2 * R] = __int_as_float(Fm);
            }
        }
        __syncthreads();   // (also: the item's shared memory is free)
        if (!whole) {
            const int c0 = cta_of(it.first, U, C), c1 = cta_of(it.first + it.units - 1, U, C);
            if (threadIdx.x == 0) {
                __threadfence();
                const uint32_t n = atom_acq_rel_add_u32(p.ticket + c0, 1u);
                s_last = n == (uint32_t)(c1 - c0);
                if (s_last) p.ticket[c0] = 0;
            }
            __syncthreads();
            if (s_last) {
                __threadfence();
                join_parts<Cfg::kThreads, R, D>(p, it, rows, c0, c1);
            }
            __syncthreads();
        }
        u = it.first + st1;
        if (u >= u_end) break;
    }
}

}  // namespace

template <int D, int NT>
static cudaError_t launch_one(const kv4::Attn &p, cudaStream_t s) {
    using Cfg = DecodeCfg<D, NT>;
    const size_t smem = Cfg::kSmem + sizeof(long long) * ((size_t)p.b.B + 1);
    const cudaError_t err = set_smem_once(reinterpret_cast<const void *>(kv4_decode_kernel<D, NT>), (int)(Cfg::kSmem + sizeof(long long) * 4097));
    if (err != cudaSuccess) return err;
    int grid = 2 * sm_count();
    if (grid > kv4::kMaxCtas) grid = kv4::kMaxCtas;
    return launch_pdl(kv4_decode_kernel<D, NT>, dim3((unsigned)grid), Cfg::kThreads, smem, s, p);
}

cudaError_t launch_kv4_decode(const kv4::Attn &p, int rows, cudaStream_t s) {
    if (p.c.D == 64) return rows <= 8 ? launch_one<64, 1>(p, s) : rows <= 16 ? launch_one<64, 2>(p, s) : launch_one<64, 4>(p, s);
    return rows <= 8 ? launch_one<128, 1>(p, s) : rows <= 16 ? launch_one<128, 2>(p, s) : launch_one<128, 4>(p, s);
}

}  // namespace moe
