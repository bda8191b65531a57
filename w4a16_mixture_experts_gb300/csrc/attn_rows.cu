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
// fraction of a turn (the position is whole, so whole turns drop out). F_i is a
// 24-bit mantissa times 64 bits of 1 / 2 pi; the error is a unit of its last
// place times the position.
//
// D / 8 lanes hold a row, each both members of four pairs (or eight values that
// do not turn): the turn needs no exchange, the sum of squares a few shuffles.
// They take `chunk` query heads or key heads of a token in a row, kAt of them
// under way at once, and form their coefficients (cosine or sine times weight)
// once for all of them.
// Bound by HBM from some thousand rows on: 16384 tokens of 32 + 8 heads of 128,
// 336 MB, 59.7 us (84% of the copy rate).
struct NormRope {
    const uint16_t *x[2], *w[2];   // queries, keys
    uint16_t *y[2];
    moe_strides xs[2], ys[2];
    const int32_t *pos;
    const float *inv_freq;
    int T, Hq, Hkv, rot, chunk, q_chunks, chunks;   // of a token: of its query heads, of all
    float eps;
};

// frac(f / 2 pi) as a 64-bit fraction; f a finite fp32.
__device__ inline unsigned long long turn_fraction(float f) {
    const uint32_t bits = __float_as_uint(f);
    const int e = max((int)(bits >> 23 & 0xFFu), 1);
    const unsigned long long m = (bits & 0x7FFFFFu) | (bits >> 23 & 0xFFu ? 0x800000u : 0u);
    constexpr unsigned long long kInv2Pi = 0xA2F9836E4E441529ull;   // 2^66 / (2 pi)
    const unsigned long long hi = __umul64hi(m, kInv2Pi), lo = m * kInv2Pi;
    const int down = 152 - e;   // m 2^(e - 150) / 2 pi 2^64
    unsigned long long r = down >= 128 ? 0ull : down >= 64 ? hi >> (down - 64) : down > 0 ? lo >> down | hi << (64 - down) : lo << min(-down, 63);
    return bits >> 31 ? 0ull - r : r;
}

template <int D, bool kInter, int kAt>
__global__ void __launch_bounds__(kRowThreads) norm_rope_kernel(NormRope p) {
    constexpr int kLanes = D / 8, kGroups = kRowThreads / kLanes;
    const int lane = threadIdx.x % kLanes;
    pdl_wait();
    pdl_launch_dependents();
    // the lane's eight values: four at a, four at b
    const int half = p.rot / 2;
    const bool turns = lane * 8 < p.rot;
    const int a = kInter || !turns ? lane * 8 : lane * 4, b = kInter || !turns ? a + 4 : half + a;
    unsigned long long F[4] = {0, 0, 0, 0};
    if (turns)
#pragma unroll
        for (int i = 0; i < 4; ++i) F[i] = turn_fraction(p.inv_freq[lane * 4 + i]);

    const long long tasks = (long long)p.T * p.chunks;
    // every lane of a warp goes as far as its last group, for the shuffles
    for (long long k0 = (long long)blockIdx.x * kGroups; k0 < tasks; k0 += (long long)gridDim.x * kGroups) {
        const long long k = k0 + threadIdx.x / kLanes;
        const bool mine = k < tasks;
        const int t = mine ? (int)(k / p.chunks) : 0, c = mine ? (int)(k - (long long)t * p.chunks) : 0;
        const bool keys = c >= p.q_chunks;
        const int h0 = (keys ? c - p.q_chunks : c) * p.chunk;
        const int rows = mine ? min(p.chunk, (keys ? p.Hkv : p.Hq) - h0) : 0;
        const size_t step = (size_t)(keys ? p.xs[1].head : p.xs[0].head), ystep = (size_t)(keys ? p.ys[1].head : p.ys[0].head);
        const uint16_t *x_at = (keys ? p.x[1] + (size_t)t * p.xs[1].token : p.x[0] + (size_t)t * p.xs[0].token) + h0 * step;
        uint16_t *y_at = (keys ? p.y[1] + (size_t)t * p.ys[1].token : p.y[0] + (size_t)t * p.ys[0].token) + h0 * ystep;
        const uint16_t *const w = keys ? p.w[1] : p.w[0];
        uint2 u[kAt][2];
        auto load = [&](int j0) {
#pragma unroll
            for (int j = 0; j < kAt; ++j) {
                const bool there = j0 + j < rows;
                u[j][0] = there ? *reinterpret_cast<const uint2 *>(x_at + a) : make_uint2(0, 0);
                u[j][1] = there ? *reinterpret_cast<const uint2 *>(x_at + b) : make_uint2(0, 0);
                if (there) x_at += step;
            }
        };
        load(0);
        // out[v] = rs (x[v] cv[v] + x[its partner] cp[v])
        float cv[8], cp[8];
        if (w)
            unpack8(make_uint4(reinterpret_cast<const uint2 *>(w + a)->x, reinterpret_cast<const uint2 *>(w + a)->y,
                               reinterpret_cast<const uint2 *>(w + b)->x, reinterpret_cast<const uint2 *>(w + b)->y), cv);
        else
#pragma unroll
            for (int i = 0; i < 8; ++i) cv[i] = 1.f;
        if (turns) {
            const unsigned long long pos = (unsigned long long)(long long)p.pos[t];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int v = kInter ? 2 * i : i, z = kInter ? 2 * i + 1 : i + 4;
                float sn, cs;
                sincospif((float)(int)(F[i] * pos >> 32) * 4.656612873077393e-10f, &sn, &cs);   // 2^-31: half turns
                cp[v] = -sn * cv[z];
                cp[z] = sn * cv[v];
                cv[v] *= cs;
                cv[z] *= cs;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) cp[i] = 0.f;
        }
        for (int j0 = 0; j0 < p.chunk; j0 += kAt) {
#pragma unroll
            for (int j = 0; j < kAt; ++j) {
                float x[8];
                unpack8(make_uint4(u[j][0].x, u[j][0].y, u[j][1].x, u[j][1].y), x);
                float ss = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
                for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                const float rs = rsqrtf(ss * (1.f / D) + p.eps);
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] *= rs;
                float y[8];
                if (turns) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) y[i] = fmaf(x[i], cv[i], x[kInter ? i ^ 1 : i ^ 4] * cp[i]);
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) y[i] = x[i] * cv[i];
                }
                if (j0 + j < rows) {
                    *reinterpret_cast<uint2 *>(y_at + a) = make_uint2(pack2(y[0], y[1]), pack2(y[2], y[3]));
                    *reinterpret_cast<uint2 *>(y_at + b) = make_uint2(pack2(y[4], y[5]), pack2(y[6], y[7]));
                    y_at += ystep;
                }
            }
            if (j0 + kAt < p.chunk) load(j0 + kAt);
        }
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

// The row's place in codes and scales (in rows), or -1; `bad` where the slot is
// neither in the cache nor -1.
__device__ inline long long place(const Rows &p, int sl, int h, bool &bad) {
    const bool in = (unsigned)sl < (unsigned)p.n_slots;
    bad |= !in && sl != -1;
    return in ? (((long long)(sl >> p.shift) * p.Hkv + h) << p.shift) + (sl & ((1 << p.shift) - 1)) : -1;
}

// The rows of a group of lanes: 2 h + g (g: K or V) of token t, then `step` rows
// on. The step is even, so that g stays; no division or product but the first.
// `at` follows in a tensor with these strides.
struct Walk {
    int t, h2, dt, dh2, n2;
    long long at, dat, wrap;
    __device__ Walk(int row, int step, int Hkv, long long token, long long head) : n2(2 * Hkv) {
        t = row / n2, h2 = row - t * n2;
        dt = step / n2, dh2 = step - dt * n2;
        at = t * token + (h2 >> 1) * head;
        dat = dt * token + (dh2 >> 1) * head;
        wrap = token - Hkv * head;
    }
    __device__ void next() {
        t += dt;
        h2 += dh2;
        at += dat;
        if (h2 >= n2) {
            h2 -= n2;
            ++t;
            at += wrap;
        }
    }
};

__device__ inline void add2(float &a, float &b, float c) {
    asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %2};\n\tadd.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "+f"(a), "+f"(b)
        : "f"(c));
}
__device__ inline void fma2(float &a, float &b, float c, float d) {   // (a, b) = (a, b) * c + d
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %2};\n\tmov.b64 z, {%3, %3};\n\t"
        "fma.rn.f32x2 x, x, y, z;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "+f"(a), "+f"(b)
        : "f"(c), "f"(d));
}

template <int D, int kAt>
__global__ void __launch_bounds__(kRowThreads) append_kernel(Rows p) {
    constexpr int kLanes = D / 8, kRows = kRowThreads / kLanes;
    const int lane = threadIdx.x % kLanes, g = threadIdx.x / kLanes & 1;
    pdl_wait();
    pdl_launch_dependents();
    const uint16_t *const x_at = (g ? p.x[1] : p.x[0]) + lane * 8;
    int32_t *const codes = (g ? p.codes[1] : p.codes[0]) + lane;
    uint16_t *const scales = g ? p.scales[1] : p.scales[0];
    Walk w(blockIdx.x * kRows + threadIdx.x / kLanes, gridDim.x * kRows, p.Hkv, g ? p.xs[1].token : p.xs[0].token, g ? p.xs[1].head : p.xs[0].head);
    bool out = false;   // a slot outside the cache
    // (the lanes of a warp end together: a group beyond the rows goes along)
    uint4 next[kAt];
    int next_sl[kAt], next_h[kAt];
    // kAt rows, under way while the last kAt are worked on (32768 tokens of 8 heads, append and
    // read: 66.0 us with 2, 69.6 with 3, 72.6 with 4, whose registers leave fewer warps; 66.9 with
    // 4 at a time and none under way)
    auto load = [&]() {
#pragma unroll
        for (int j = 0; j < kAt; ++j) {
            const bool there = w.t < p.T;
            next_h[j] = w.h2 >> 1;
            next[j] = there ? *reinterpret_cast<const uint4 *>(x_at + w.at) : make_uint4(0, 0, 0, 0);
            next_sl[j] = there ? p.slots[w.t] : -1;
            w.next();
        }
    };
    bool more = __any_sync(0xffffffffu, w.t < p.T);
    load();
    while (more) {
        uint4 u[kAt];
        long long at[kAt];
#pragma unroll
        for (int j = 0; j < kAt; ++j) {
            u[j] = next[j];
            at[j] = place(p, next_sl[j], next_h[j], out);
        }
        more = __any_sync(0xffffffffu, w.t < p.T);
        if (more) load();
#pragma unroll
        for (int j = 0; j < kAt; ++j) {
            // max|x|; a NaN wins
            auto mag = [](uint32_t v) {
                v &= 0x7FFF7FFFu;
                return *reinterpret_cast<const __nv_bfloat162 *>(&v);
            };
            __nv_bfloat162 m2 = __hmax2_nan(__hmax2_nan(mag(u[j].x), mag(u[j].y)), __hmax2_nan(mag(u[j].z), mag(u[j].w)));
#pragma unroll
            for (int o = kLanes / 2; o > 0; o >>= 1) {
                const uint32_t got = __shfl_xor_sync(0xffffffffu, *reinterpret_cast<const uint32_t *>(&m2), o);
                m2 = __hmax2_nan(m2, *reinterpret_cast<const __nv_bfloat162 *>(&got));
            }
            const float m = __bfloat162float(__hmax_nan(__low2bfloat16(m2), __high2bfloat16(m2)));
            const bool bad = !(m <= 3.402823466e38f);
            // (bf16(m / 7) by the reciprocal: m has 8 bits, so that m / 7 lies 2^-12 from any
            // point between two bf16 at the least)
            const __nv_bfloat16 sb = __float2bfloat16_rn(m * (1.f / 7.f));
            const float s = __bfloat162float(sb);
            // rint(x / s) from x times the approximate reciprocal, which is within 4e-6 of the
            // quotient (|x / s| is at most 7.03). Quotients of 8-bit mantissas are halves exactly,
            // as often as not in a warp's 256, or at least 1 / 1020 away from one; so the product
            // is first rounded to 2^-11 (by adding 1.5 2^12), which makes halves of those and takes
            // no other across. Adding 1.5 2^23 + 8 less that then rounds to whole numbers, ties to
            // even, and leaves the code in the low bits. A scale near the subnormals, which may round far, takes the
            // division and a clamp.
            constexpr float kGrid = 6144.f, kWhole = 12582920.f;   // 1.5 2^12, 1.5 2^23 + 8
            constexpr uint32_t kBits = 0x4B400000u;                // of 1.5 2^23
            float x[8], inv;
            unpack8(u[j], x);
            asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
            uint32_t word = 0x88888888u;
            if (s > 0.f && !bad) {
                word = 0u - kBits * 0x11111111u;
                if (s > 1e-37f) {
#pragma unroll
                    for (int i = 0; i < 8; i += 2) {
                        fma2(x[i], x[i + 1], inv, kGrid);
                        add2(x[i], x[i + 1], kWhole - kGrid);
                        word += __float_as_uint(x[i]) << (4 * i);
                        word += __float_as_uint(x[i + 1]) << (4 * i + 4);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        word += __float_as_uint(fminf(fmaxf(__fdiv_rn(x[i], s), -8.f), 7.f) + kWhole) << (4 * i);
                }
            }
            if (at[j] >= 0) {
                codes[at[j] * (D / 8)] = (int32_t)word;
                if (lane == 0) scales[at[j]] = bad ? (uint16_t)0x7FC0u : *reinterpret_cast<const uint16_t *>(&sb);
            }
        }
    }
    if (out) set_error(p.ctrl, MOE_ERR_DEVICE);
}

// Rows out of the cache as bf16(q * s) (the product of two bf16, rounded once);
// slot -1 reads as zero. A warp reads 512 bytes of codes at a time, 16 a lane
// (8 rows of 128 or 16 of 64), so that enough is under way, and passes them
// through shared memory to the lanes that write 16 bytes of values each, side by
// side: from 4 bytes a lane the loads' latency took 46 us of what moves 25 us'
// worth.
template <int D, int kAt>
__global__ void __launch_bounds__(kRowThreads) read_kernel(Rows p) {
    constexpr int kPieces = D / 32, kRows = 32 / kPieces;   // lanes of a row that read; rows a warp reads at once
    constexpr int kOut = D / 8;                             // lanes of a row that write
    __shared__ uint32_t s_words[kRowThreads / 32][128];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane / kPieces & 1;
    uint32_t *const words = s_words[warp];
    pdl_wait();
    pdl_launch_dependents();
    const int32_t *const codes = (g ? p.codes[1] : p.codes[0]) + lane % kPieces * 4;
    const uint16_t *const scales = g ? p.scales[1] : p.scales[0];
    uint16_t *const y = (lane / kOut & 1 ? p.y[1] : p.y[0]) + lane % kOut * 8;
    Walk w((blockIdx.x * (kRowThreads / 32) + warp) * kRows + lane / kPieces, gridDim.x * (kRowThreads / 32) * kRows, p.Hkv, 2 * p.Hkv, 2);
    bool out = false;
    while (__any_sync(0xffffffffu, w.t < p.T)) {
        uint4 u[kAt];
        uint32_t s2[kAt];
        int sl[kAt], row[kAt];   // row: of K's or V's output, -1: none
#pragma unroll
        for (int j = 0; j < kAt; ++j) {
            row[j] = w.t < p.T ? (int)(w.at >> 1) : -1;
            sl[j] = w.t < p.T ? p.slots[w.t] : -1;
            const long long at = place(p, sl[j], w.h2 >> 1, out);
            u[j] = at >= 0 ? *reinterpret_cast<const uint4 *>(codes + at * (D / 8)) : make_uint4(0x88888888u, 0x88888888u, 0x88888888u, 0x88888888u);
            s2[j] = at >= 0 ? (uint32_t)scales[at] * 0x10001u : 0u;
            w.next();
        }
#pragma unroll
        for (int j = 0; j < kAt; ++j) {
            __syncwarp();
            *reinterpret_cast<uint4 *>(words + lane * 4) = u[j];
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 4; ++i) {   // 32 / kOut rows at a time
                const int from = (i * (32 / kOut) + lane / kOut) * kPieces;
                const uint32_t s = __shfl_sync(0xffffffffu, s2[j], from), word = words[i * 32 + lane];
                const int to = __shfl_sync(0xffffffffu, row[j], from);
                uint32_t q[4];   // pairs (k, k + 4)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t n = int4_pair(word, k);
                    const __nv_bfloat162 x = __hmul2(*reinterpret_cast<const __nv_bfloat162 *>(&n), *reinterpret_cast<const __nv_bfloat162 *>(&s));
                    q[k] = *reinterpret_cast<const uint32_t *>(&x);
                }
                if (to >= 0)
                    *reinterpret_cast<uint4 *>(y + (size_t)to * D) = make_uint4(__byte_perm(q[0], q[1], 0x5410), __byte_perm(q[2], q[3], 0x5410),
                                                                                __byte_perm(q[0], q[1], 0x7632), __byte_perm(q[2], q[3], 0x7632));
            }
        }
    }
    if (out) set_error(p.ctrl, MOE_ERR_DEVICE);
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

// `per` rows a CTA where the card holds them all at once (four times that under
// way are slower there: 3.1 against 4.8 us for 16 tokens written and read), else
// four times.
template <typename One, typename Many>
cudaError_t launch_rows(One one, Many many, const Rows &p, long long per, cudaStream_t s) {
    const long long n = ((long long)p.T * p.Hkv * 2 + per - 1) / per, most = 8LL * sm_count();
    if (n <= most) return launch_pdl(one, dim3((unsigned)n), kRowThreads, 0, s, p);
    return launch_pdl(many, dim3((unsigned)most), kRowThreads, 0, s, p);
}

}  // namespace

cudaError_t launch_norm_rope(const uint16_t *q, moe_strides qs, const uint16_t *k, moe_strides ks, const uint16_t *qw,
                             const uint16_t *kw, const int32_t *pos, const float *inv_freq, int rot, bool interleaved,
                             float eps, uint16_t *qo, moe_strides qos, uint16_t *ko, moe_strides kos, int T, int Hq,
                             int Hkv, int D, cudaStream_t s) {
    const int groups = kRowThreads / (D / 8);
    // a head a task for a decode step's latency; four, or more, where that still leaves the
    // card several tasks for each place (16384 tokens: 8 heads a task 5% faster than 4)
    const long long places = (long long)sm_count() * (2048 / kRowThreads) * groups;
    auto tasks = [&](int n) { return (long long)T * ((Hq + n - 1) / n + (Hkv + n - 1) / n); };
    int chunk = tasks(1) <= places ? 1 : 4;
    while (chunk > 1 && chunk < Hq && tasks(chunk) > 4 * places) chunk *= 2;
    const int qc = (Hq + chunk - 1) / chunk;
    const NormRope p{{q, k}, {qw, kw}, {qo, ko}, {qs, ks}, {qos, kos}, pos, inv_freq, T, Hq, Hkv, rot, chunk, qc, qc + (Hkv + chunk - 1) / chunk, eps};
    const long long blocks = (tasks(chunk) + groups - 1) / groups, most = 8LL * sm_count();
    const dim3 grid((unsigned)(blocks < most ? blocks : most));
    auto go = [&](auto one, auto four) { return chunk == 1 ? launch_pdl(one, grid, kRowThreads, 0, s, p) : launch_pdl(four, grid, kRowThreads, 0, s, p); };
    switch (D) {
        case 64:
            return interleaved ? go(norm_rope_kernel<64, true, 1>, norm_rope_kernel<64, true, 4>) : go(norm_rope_kernel<64, false, 1>, norm_rope_kernel<64, false, 4>);
        case 128:
            return interleaved ? go(norm_rope_kernel<128, true, 1>, norm_rope_kernel<128, true, 4>)
                               : go(norm_rope_kernel<128, false, 1>, norm_rope_kernel<128, false, 4>);
        default:
            return interleaved ? go(norm_rope_kernel<256, true, 1>, norm_rope_kernel<256, true, 4>)
                               : go(norm_rope_kernel<256, false, 1>, norm_rope_kernel<256, false, 4>);
    }
}

cudaError_t launch_kv4_append(const uint16_t *k, moe_strides ks, const uint16_t *v, moe_strides vs,
                              const int32_t *slots, int T, const moe_kv4_cache &c, Ctrl *ctrl, cudaStream_t s) {
    Rows p = rows_of(c, slots, T, ctrl);
    p.x[0] = k;
    p.x[1] = v;
    p.xs[0] = ks;
    p.xs[1] = vs;
    return c.D == 64 ? launch_rows(append_kernel<64, 1>, append_kernel<64, 2>, p, kRowThreads / 8, s)
                     : launch_rows(append_kernel<128, 1>, append_kernel<128, 2>, p, kRowThreads / 16, s);
}

cudaError_t launch_kv4_read(const int32_t *slots, int T, const moe_kv4_cache &c, uint16_t *k, uint16_t *v, Ctrl *ctrl,
                            cudaStream_t s) {
    Rows p = rows_of(c, slots, T, ctrl);
    p.y[0] = k;
    p.y[1] = v;
    return c.D == 64 ? launch_rows(read_kernel<64, 1>, read_kernel<64, 4>, p, kRowThreads / 2, s)
                     : launch_rows(read_kernel<128, 1>, read_kernel<128, 4>, p, kRowThreads / 4, s);
}

}  // namespace moe
