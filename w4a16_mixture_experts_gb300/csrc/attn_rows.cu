// The row operators of the attention block: per-head RMS norms with the rotary
// turn in the same pass, and rows written to and read from the 4-bit cache.
// All of them move each value once and are bound by HBM at a prompt's sizes
// and by their launch at a decode step's.
#include "kv4.cuh"

namespace moe {

namespace {

constexpr int kRowThreads = 256;

__device__ inline void unpack8(const uint4 &u, float (&x)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

__device__ inline uint32_t pack2(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// ---------------------------------------------------------------------------
// y = x * w / sqrt(mean(x^2) + eps) over a head's D values, then the pairs of
// the first rot values turned by theta_i = position * inv_freq[i].
//
// The angle. A position times a frequency in fp32 is off by whole radians far
// into a context, so theta is reduced in integers: F_i = frac(inv_freq[i] /
// 2 pi) as a 64-bit fraction of a turn, and position * F_i modulo 2^64 is the
// fraction of a turn exactly (the position is whole, so whole turns drop out).
// F_i costs one fp64 product per thread, an angle three integer products; the
// error is that of F_i, 2^-55 of a turn times the position.
//
// Layout: D / 8 lanes hold a row, 16 bytes each; the sum of squares and the
// other half of a half-split pair come by shuffle. A CTA owns `tb` tokens (all
// heads), whose cosines and sines it puts into shared memory once.
struct NormRope {
    const uint16_t *x[2], *w[2];   // queries, keys
    uint16_t *y[2];
    moe_strides xs[2], ys[2];
    const int32_t *pos;
    const float *inv_freq;
    int T, Hq, H, rot, tb;   // H = Hq + Hkv
    float eps;
};

template <int D, bool kInter>
__global__ void __launch_bounds__(kRowThreads) norm_rope_kernel(NormRope p) {
    constexpr int kLanes = D / 8, kRows = kRowThreads / kLanes;
    extern __shared__ float s_cs[];   // [tb][2][rot / 2]
    const int half = p.rot / 2;
    const int t0 = blockIdx.x * p.tb, nt = min(p.tb, p.T - t0);
    const int lane = threadIdx.x % kLanes, row0 = threadIdx.x / kLanes;
    pdl_wait();
    pdl_launch_dependents();
    for (int i = threadIdx.x; i < half * nt; i += kRowThreads) {
        const int t = i / half, j = i - t * half;
        const double turn = (double)p.inv_freq[j] * 0.15915494309189533577;
        const unsigned long long F = (unsigned long long)((turn - floor(turn)) * 18446744073709551616.0);
        const unsigned long long a = F * (unsigned long long)(long long)p.pos[t0 + t];
        float s, c;
        sincospif((float)(int)(a >> 32) * 4.656612873077393e-10f, &s, &c);   // 2^-31: half turns
        s_cs[(t * 2) * half + j] = c;
        s_cs[(t * 2 + 1) * half + j] = s;
    }
    __syncthreads();
    float w[2][8];
#pragma unroll
    for (int g = 0; g < 2; ++g) {
        if (p.w[g]) unpack8(ld_nc_v4(p.w[g] + lane * 8), w[g]);
        else
            for (int i = 0; i < 8; ++i) w[g][i] = 1.f;
    }
    const int hl = half / 8;   // lanes of half a turn
    const int rows = nt * p.H;
    for (int r = blockIdx.y * kRows + row0; r - row0 < rows; r += kRows * gridDim.y) {
        const bool there = r < rows;   // every lane stays for the shuffles
        const int t = there ? r / p.H : 0, h = there ? r - t * p.H : 0;
        const int g = h >= p.Hq;
        const int hh = g ? h - p.Hq : h;
        float x[8];
        unpack8(there ? *reinterpret_cast<const uint4 *>(p.x[g] + (size_t)(t0 + t) * p.xs[g].token + (size_t)hh * p.xs[g].head + lane * 8)
                      : make_uint4(0, 0, 0, 0), x);
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const float rs = rsqrtf(ss * (1.f / D) + p.eps);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] *= rs * (g ? w[1][i] : w[0][i]);
        const float *cs = s_cs + t * 2 * half;
        if (kInter) {
            if (lane * 8 < p.rot) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float c = cs[lane * 4 + i], s = cs[half + lane * 4 + i];
                    const float a = x[2 * i], b = x[2 * i + 1];
                    x[2 * i] = a * c - b * s;
                    x[2 * i + 1] = fmaf(a, s, b * c);
                }
            }
        } else if (hl) {
            const bool lo = lane < hl;
            const int src = (threadIdx.x & 31) + (lo ? hl : -hl);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float o = __shfl_sync(0xffffffffu, x[i], src & 31);
                if (lane < 2 * hl) {
                    const int j = (lo ? lane : lane - hl) * 8 + i;
                    const float c = cs[j], s = cs[half + j];
                    x[i] = lo ? x[i] * c - o * s : fmaf(x[i], c, o * s);
                }
            }
        }
        if (there)
            *reinterpret_cast<uint4 *>(p.y[g] + (size_t)(t0 + t) * p.ys[g].token + (size_t)hh * p.ys[g].head + lane * 8) =
                make_uint4(pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7]));
    }
}

// ---------------------------------------------------------------------------
// Rows into the cache: s = bf16(max|x| / 7), q = clamp(rint(x / s), -8, 7), the
// quantiser's arithmetic without its clip search (fp32 divisions, so that the
// codes are the same bits wherever they are formed). D / 8 lanes hold a row and
// write a word each. A row with a value that is not finite gets a NaN scale.
struct Rows {
    const uint16_t *x[2];   // append: k, v
    moe_strides xs[2];
    uint16_t *y[2];         // read: k, v
    int32_t *codes[2];
    uint16_t *scales[2];
    const int32_t *slots;
    Ctrl *ctrl;
    int T, Hkv, shift;
    long long n_slots;
};

// The row's place in codes and scales (in rows), or -1.
__device__ inline long long place(const Rows &p, int t, int h) {
    const int sl = p.slots[t];
    if (sl < 0 || sl >= p.n_slots) {
        if (sl != -1) set_error(p.ctrl, MOE_ERR_DEVICE);
        return -1;
    }
    return (((long long)(sl >> p.shift) * p.Hkv + h) << p.shift) + (sl & ((1 << p.shift) - 1));
}

template <int D>
__global__ void __launch_bounds__(kRowThreads) append_kernel(Rows p) {
    constexpr int kLanes = D / 8, kRows = kRowThreads / kLanes;
    const int lane = threadIdx.x % kLanes;
    const long long rows = (long long)p.T * p.Hkv * 2;
    pdl_wait();
    pdl_launch_dependents();
    for (long long r = (long long)blockIdx.x * kRows + threadIdx.x / kLanes; r - threadIdx.x / kLanes < rows; r += (long long)gridDim.x * kRows) {
        const bool there = r < rows;
        const int th = there ? (int)(r >> 1) : 0, g = there ? (int)(r & 1) : 0;
        const int t = th / p.Hkv, h = th - t * p.Hkv;
        float x[8];
        unpack8(there ? *reinterpret_cast<const uint4 *>(p.x[g] + (size_t)t * p.xs[g].token + (size_t)h * p.xs[g].head + lane * 8)
                      : make_uint4(0, 0, 0, 0), x);
        float m = 0.f;
        bool bad = false;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            m = fmaxf(m, fabsf(x[i]));
            bad |= !(fabsf(x[i]) <= 3.402823466e38f);
        }
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        const uint32_t any = __ballot_sync(0xffffffffu, bad);
        bad = (any >> ((threadIdx.x & 31) / kLanes * kLanes)) & ((1u << (kLanes - 1) << 1) - 1u);
        const __nv_bfloat16 sb = __float2bfloat16_rn(__fdiv_rn(m, 7.f));
        const float s = __bfloat162float(sb);
        uint32_t word = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float q = s > 0.f && !bad ? fminf(fmaxf(rintf(__fdiv_rn(x[i], s)), -8.f), 7.f) : 0.f;
            word |= (uint32_t)((int)q + 8) << (4 * i);
        }
        const long long at = there ? place(p, t, h) : -1;
        if (at >= 0) {
            p.codes[g][at * (D / 8) + lane] = (int32_t)word;
            if (lane == 0) p.scales[g][at] = bad ? (uint16_t)0x7FC0u : *reinterpret_cast<const uint16_t *>(&sb);
        }
    }
}

// Rows out of the cache as bf16(q * s); slot -1 reads as zero.
template <int D>
__global__ void __launch_bounds__(kRowThreads) read_kernel(Rows p) {
    constexpr int kLanes = D / 8, kRows = kRowThreads / kLanes;
    const int lane = threadIdx.x % kLanes;
    const long long rows = (long long)p.T * p.Hkv * 2;
    pdl_wait();
    pdl_launch_dependents();
    for (long long r = (long long)blockIdx.x * kRows + threadIdx.x / kLanes; r < rows; r += (long long)gridDim.x * kRows) {
        const int th = (int)(r >> 1), g = (int)(r & 1);
        const int t = th / p.Hkv, h = th - t * p.Hkv;
        const long long at = place(p, t, h);
        uint32_t o[4] = {0, 0, 0, 0};
        if (at >= 0) {
            const uint32_t word = (uint32_t)p.codes[g][at * (D / 8) + lane];
            const float s = bf16_bits_to_f32(p.scales[g][at]);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                o[i] = pack2((float)((int)(word >> (8 * i) & 15u) - 8) * s, (float)((int)(word >> (8 * i + 4) & 15u) - 8) * s);
        }
        *reinterpret_cast<uint4 *>(p.y[g] + ((size_t)t * p.Hkv + h) * D + lane * 8) = make_uint4(o[0], o[1], o[2], o[3]);
    }
}

Rows rows_of(const moe_kv4_cache &c, const int32_t *slots, int T, Ctrl *ctrl) {
    Rows p{};
    p.codes[0] = c.k_codes;
    p.codes[1] = c.v_codes;
    p.scales[0] = c.k_scales;
    p.scales[1] = c.v_scales;
    p.slots = slots;
    p.ctrl = ctrl;
    p.T = T;
    p.Hkv = c.Hkv;
    p.shift = __builtin_ctz((unsigned)c.page_size);
    p.n_slots = (long long)c.n_pages * c.page_size;
    return p;
}

int rows_grid(int T, int Hkv, int D) {
    const long long per = kRowThreads / (D / 8);
    const long long n = ((long long)T * Hkv * 2 + per - 1) / per;
    const long long most = 8LL * sm_count();   // all co-resident, a few rows in turn each
    return (int)(n < most ? n : most);
}

}  // namespace

cudaError_t launch_norm_rope(const uint16_t *q, moe_strides qs, const uint16_t *k, moe_strides ks, const uint16_t *qw,
                             const uint16_t *kw, const int32_t *pos, const float *inv_freq, int rot, bool interleaved,
                             float eps, uint16_t *qo, moe_strides qos, uint16_t *ko, moe_strides kos, int T, int Hq,
                             int Hkv, int D, cudaStream_t s) {
    NormRope p{{q, k}, {qw, kw}, {qo, ko}, {qs, ks}, {qos, kos}, pos, inv_freq, T, Hq, Hq + Hkv, rot, 1, eps};
    const int rows = kRowThreads / (D / 8);
    // a prompt's CTAs own 8 tokens, so that the angles cost little; a decode
    // step's heads go to CTAs of their own
    p.tb = T >= 8 * sm_count() ? 8 : T >= 2 * sm_count() ? 2 : 1;
    const int per = (p.H * p.tb + rows - 1) / rows;
    dim3 grid((T + p.tb - 1) / p.tb, T < 2 * sm_count() ? per : 1);
    const size_t smem = (size_t)p.tb * rot * sizeof(float);
    auto go = [&](auto kernel) { return launch_pdl(kernel, grid, kRowThreads, smem, s, p); };
    switch (D) {
        case 64: return interleaved ? go(norm_rope_kernel<64, true>) : go(norm_rope_kernel<64, false>);
        case 128: return interleaved ? go(norm_rope_kernel<128, true>) : go(norm_rope_kernel<128, false>);
        default: return interleaved ? go(norm_rope_kernel<256, true>) : go(norm_rope_kernel<256, false>);
    }
}

cudaError_t launch_kv4_append(const uint16_t *k, moe_strides ks, const uint16_t *v, moe_strides vs,
                              const int32_t *slots, int T, const moe_kv4_cache &c, Ctrl *ctrl, cudaStream_t s) {
    Rows p = rows_of(c, slots, T, ctrl);
    p.x[0] = k;
    p.x[1] = v;
    p.xs[0] = ks;
    p.xs[1] = vs;
    const int grid = rows_grid(T, c.Hkv, c.D);
    return c.D == 64 ? launch_pdl(append_kernel<64>, grid, kRowThreads, 0, s, p)
                     : launch_pdl(append_kernel<128>, grid, kRowThreads, 0, s, p);
}

cudaError_t launch_kv4_read(const int32_t *slots, int T, const moe_kv4_cache &c, uint16_t *k, uint16_t *v, Ctrl *ctrl,
                            cudaStream_t s) {
    Rows p = rows_of(c, slots, T, ctrl);
    p.y[0] = k;
    p.y[1] = v;
    const int grid = rows_grid(T, c.Hkv, c.D);
    return c.D == 64 ? launch_pdl(read_kernel<64>, grid, kRowThreads, 0, s, p)
                     : launch_pdl(read_kernel<128>, grid, kRowThreads, 0, s, p);
}

}  // namespace moe
