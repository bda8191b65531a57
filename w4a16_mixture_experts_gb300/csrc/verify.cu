// Verification of drafted tokens against the target's probabilities, from given
// random numbers.
//
// Sequence b has the rows [cu[b], cu[b + 1]) of logits: row i predicts what
// follows its drafts 0 .. i - 1, draft i stands at row i, the last row has none.
// With p = softmax(logits / t), q = softmax(draft logits / t) (or 1 at the draft):
//   accepted while u_i q(x_i) < p(x_i); then, at the first row that refuses, the
//   token argmax_v max(p_v - q_v, 0) / e_v, at the last row argmax_v p_v / e_v,
//   with e_v drawn from Exp(1): an exponential race, whose winner v has the
//   probability of v's weight.
// t = 0: accepted while x_i is the row's largest logit (the first of equals).
//
// What bounds it: every logit is read once (2 bytes) for the rows' largest values
// and sums of exponentials, a row of each sequence and its noise once more. Two
// launches: rows' statistics by chunks, over all rows at once (which row decides is
// known only after them), then the decision and the race, by chunks of the
// deciding row; the last CTA of a sequence to finish joins its chunks.
#include <math.h>

#include "step_kernels.cuh"

namespace moe {

namespace {

constexpr int kThreads = 256, kVecs = 4;            // 16-byte loads of a thread in a chunk
constexpr int kChunk = kThreads * 8 * kVecs;        // logits of a chunk
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kMinNoise = 1.17549435e-38f;

struct Stat {       // of a chunk of a row
    float m, s;     // the largest logit, the sum of exp((l - m) / t)
    int arg;        // the first place of m
    int bad;        // a NaN or +inf among them
};

struct Best {
    double score;
    int v, pad;
};

struct Params {
    const uint16_t *logits, *draft;
    long long ls, ds, ns;
    const int32_t *drafts, *cu;
    const float *temperature, *uniform, *noise;
    int32_t *tokens, *accepted;
    int B, T, V, chunks;
    Ctrl *ctrl;
    uint32_t *tickets;   // [B], cleared by the first launch
    Best *best;          // [B][chunks]
    Stat *stats;         // [T][1 or 2][chunks]
};

__device__ inline float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

struct Rows {
    int r0, n;   // first row, rows
};

__device__ inline Rows rows_of(const Params &p, int b) {
    const int a = p.cu[b], e = p.cu[b + 1];
    Rows r;
    r.r0 = min(max(a, 0), p.T);
    const int end = min(max(e, r.r0), p.T);
    r.n = end - r.r0;
    if (r.r0 != a || end != e) set_error(p.ctrl, MOE_ERR_DEVICE);
    return r;
}

// The sequence that row r belongs to, or -1; a whole warp calls it. 32 places at a time.
__device__ inline int sequence_of(const Params &p, int r) {
    const int lane = threadIdx.x & 31;
    int lo = 0, n = p.B;   // the last b in [lo, lo + n) with cu[b] <= r
    while (n > 1) {
        const int step = (n + 31) / 32, b = lo + lane * step;
        const uint32_t m = __ballot_sync(0xffffffffu, b < lo + n && p.cu[b] <= r);
        const int k = m ? 31 - __clz(m) : 0;
        n = min(step, lo + n - (lo + k * step));
        lo += k * step;
    }
    return p.cu[lo] <= r && r < p.cu[lo + 1] ? lo : -1;
}

// 1 / t in units of log 2: finite, so that equal logits stay equal.
__device__ inline float rate_of(float t) { return fminf(kLog2e / t, 1e30f); }

// 8 logits from v on; -inf behind the row's end.
__device__ inline uint4 load8(const uint16_t *row, int v, int V) {
    if (v + 8 <= V) return *reinterpret_cast<const uint4 *>(row + v);
    uint32_t w[4] = {0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u};
    for (int i = 0; v + i < V; ++i) {
        const uint32_t x = row[v + i];
        w[i >> 1] = i & 1 ? (w[i >> 1] & 0xFFFFu) | x << 16 : (w[i >> 1] & 0xFFFF0000u) | x;
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ inline void unpack8(const uint4 &v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

__global__ void __launch_bounds__(kThreads) verify_stats_kernel(const __grid_constant__ Params p) {
    __shared__ float s_m[kThreads / 32], s_s[kThreads / 32];
    __shared__ int s_arg[kThreads / 32], s_bad[kThreads / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (blockIdx.x == 0)
        for (int b = threadIdx.x; b < p.B; b += kThreads) p.tickets[b] = 0;
    if (p.T == 0) return;
    const int c = blockIdx.x % p.chunks, rw = blockIdx.x / p.chunks, sides = p.draft ? 2 : 1;
    const int side = rw / p.T, r = rw - side * p.T;
    const int b = sequence_of(p, r);
    if (b < 0) return;
    const float t = p.temperature ? p.temperature[b] : 1.f;
    if (side && (t == 0.f || r + 1 >= p.cu[b + 1])) return;   // not looked at
    const float rate = t == 0.f ? 0.f : rate_of(t);
    const uint16_t *row = side ? p.draft + r * p.ds : p.logits + r * p.ls;
    uint4 v[kVecs];
    const int v0 = c * kChunk + threadIdx.x * 8;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) v[i] = load8(row, v0 + i * kThreads * 8, p.V);
    float m = -INFINITY;
    int arg = 0x7fffffff, bad = 0;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        float x[8];
        unpack8(v[i], x);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            bad |= !(x[j] < INFINITY);
            if (x[j] > m) {
                m = x[j];
                arg = v0 + i * kThreads * 8 + j;
            }
        }
    }
    float top = m;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float om = __shfl_xor_sync(0xffffffffu, top, o);
        const int oa = __shfl_xor_sync(0xffffffffu, arg, o);
        if (om > top || (om == top && oa < arg)) arg = oa;
        top = fmaxf(top, om);
    }
    float s = 0.f;
    if (top > -INFINITY && rate > 0.f) {
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            float x[8];
            unpack8(v[i], x);
#pragma unroll
            for (int j = 0; j < 8; ++j) s += ex2((x[j] - top) * rate);
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    bad = __any_sync(0xffffffffu, bad);
    if (lane == 0) {
        s_m[warp] = top;
        s_s[warp] = s;
        s_arg[warp] = arg;
        s_bad[warp] = bad;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        Stat st{s_m[0], 0.f, s_arg[0], 0};
        for (int w = 1; w < kThreads / 32; ++w)
            if (s_m[w] > st.m || (s_m[w] == st.m && s_arg[w] < st.arg)) {
                st.m = s_m[w];
                st.arg = s_arg[w];
            }
        for (int w = 0; w < kThreads / 32; ++w) {
            if (s_s[w] > 0.f) st.s += s_s[w] * ex2((s_m[w] - st.m) * rate);
            st.bad |= s_bad[w];
        }
        p.stats[((size_t)r * sides + side) * p.chunks + c] = st;
    }
}

struct Row {
    float m;     // the largest logit
    double z;    // the sum of exp((l - m) / t)
    int arg, bad;
};

__device__ inline Row row_stats(const Params &p, int r, int side, float rate) {
    const Stat *st = p.stats + ((size_t)r * (p.draft ? 2 : 1) + side) * p.chunks;
    Row o{-INFINITY, 0.0, 0, 0};
    for (int c = 0; c < p.chunks; ++c) {
        const Stat s = st[c];
        o.bad |= s.bad;
        if (s.m > o.m) {
            o.m = s.m;
            o.arg = s.arg;
        }
    }
    for (int c = 0; c < p.chunks; ++c)
        if (st[c].s > 0.f) o.z += (double)st[c].s * exp2((double)((st[c].m - o.m) * rate));
    o.bad |= !(o.m > -INFINITY);
    return o;
}

__device__ inline double probability(const Row &o, float l, float t) { return exp(((double)l - (double)o.m) / (double)t) / o.z; }

struct Decision {
    int r0, n, a, state;   // rows of the sequence, accepted drafts; 0: the race decides, 1: `chosen` does
    int chosen, last, x;   // the draft that was refused (its q is 1 without draft logits; -1: none)
    float t, rate, mp, mq;
    double zp, zq;
};

// What becomes of sequence b: a whole warp calls it, a draft a lane.
__device__ inline Decision decide(const Params &p, int b) {
    const int lane = threadIdx.x & 31;
    const Rows rows = rows_of(p, b);
    Decision d;
    d.r0 = rows.r0;
    d.n = rows.n;
    d.t = p.temperature ? p.temperature[b] : 1.f;
    d.a = 0;
    d.state = 1;
    d.chosen = -1;
    d.last = 0;
    d.x = -1;
    d.mp = d.mq = 0.f;
    d.zp = d.zq = 1.0;
    const bool greedy = d.t == 0.f, bad_t = !(d.t >= 0.f && d.t < INFINITY);
    d.rate = greedy ? 0.f : rate_of(d.t);
    if (bad_t && rows.n > 0) set_error(p.ctrl, MOE_ERR_DEVICE);
    if (rows.n == 0 || bad_t) return d;
    for (int i0 = 0;; i0 += 32) {
        const int i = i0 + lane, r = rows.r0 + i;
        const bool there = i < rows.n, last = i == rows.n - 1;
        Row tp{0.f, 1.0, 0, 0}, tq{0.f, 1.0, 0, 0};
        bool stop = !there, fault = false;
        int x = -1;
        if (there) {
            tp = row_stats(p, r, 0, d.rate);
            fault = tp.bad;
            stop = last || fault;
            if (!stop) {
                x = p.drafts[r];
                const bool known = (unsigned)x < (unsigned)p.V;
                if (greedy) {
                    stop = tp.arg != x;
                } else {
                    double q = 1.0;
                    if (p.draft) {
                        tq = row_stats(p, r, 1, d.rate);
                        fault = tq.bad;
                        if (known) q = probability(tq, bf16_bits_to_f32(p.draft[r * p.ds + x]), d.t);
                    }
                    stop = fault || !known || !((double)p.uniform[r] * q < probability(tp, bf16_bits_to_f32(p.logits[r * p.ls + x]), d.t));
                }
                if (!known) x = -2;
            }
        }
        const uint32_t m = __ballot_sync(0xffffffffu, stop);
        // an unknown token that is reached is an error too
        if (m) {
            const int k = __ffs(m) - 1;
            d.a = i0 + k;
            d.last = __shfl_sync(0xffffffffu, (int)last, k);
            d.x = __shfl_sync(0xffffffffu, x, k);
            d.mp = __shfl_sync(0xffffffffu, tp.m, k);
            d.mq = __shfl_sync(0xffffffffu, tq.m, k);
            d.zp = __shfl_sync(0xffffffffu, tp.z, k);
            d.zq = __shfl_sync(0xffffffffu, tq.z, k);
            const bool f = __shfl_sync(0xffffffffu, (int)fault, k);
            if (f || d.x == -2) set_error(p.ctrl, MOE_ERR_DEVICE);
            d.state = f || greedy;
            d.chosen = f ? -1 : __shfl_sync(0xffffffffu, tp.arg, k);
            return d;
        }
    }
}

// Weight of token v with logits l and ld, in 64 bits.
__device__ inline double weight(const Params &p, const Decision &d, int v, float l, float ld, bool residual) {
    const double pv = exp(((double)l - (double)d.mp) / (double)d.t) / d.zp;
    if (!residual) return pv;
    if (!p.draft) return v == d.x ? 0.0 : pv;
    return fmax(pv - exp(((double)ld - (double)d.mq) / (double)d.t) / d.zq, 0.0);
}

__device__ inline float noise_of(float e) { return e >= kMinNoise ? e : kMinNoise; }

// The race over the tokens of chunk c of the deciding row.
__device__ Best race(const Params &p, const Decision &d, int c, bool residual) {
    __shared__ double s_score[kThreads / 32];
    __shared__ int s_v[kThreads / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint16_t *row = p.logits + (d.r0 + d.a) * p.ls, *drow = p.draft ? p.draft + (d.r0 + d.a) * p.ds : nullptr;
    const float *noise = p.noise + blockIdx.y * p.ns;
    double score = 0.0;
    int best = -1;
    for (int i = 0; i < kVecs * 8; ++i) {
        const int v = c * kChunk + i * kThreads + threadIdx.x;
        if (v >= p.V) break;
        const double w = weight(p, d, v, bf16_bits_to_f32(row[v]), drow && residual ? bf16_bits_to_f32(drow[v]) : 0.f, residual);
        const double s = w / (double)noise_of(noise[v]);
        if (w > 0.0 && (best < 0 || s > score)) {
            score = s;
            best = v;
        }
    }
    for (int o = 16; o > 0; o >>= 1) {
        const double os = __shfl_xor_sync(0xffffffffu, score, o);
        const int ov = __shfl_xor_sync(0xffffffffu, best, o);
        if (ov >= 0 && (best < 0 || os > score || (os == score && ov < best))) {
            score = os;
            best = ov;
        }
    }
    __syncthreads();
    if (lane == 0) {
        s_score[warp] = score;
        s_v[warp] = best;
    }
    __syncthreads();
    Best o{s_score[0], s_v[0], 0};
    for (int w = 1; w < kThreads / 32; ++w)
        if (s_v[w] >= 0 && (o.v < 0 || s_score[w] > o.score || (s_score[w] == o.score && s_v[w] < o.v))) {
            o.score = s_score[w];
            o.v = s_v[w];
        }
    return o;
}

__global__ void __launch_bounds__(kThreads) verify_choose_kernel(const __grid_constant__ Params p) {
    __shared__ Decision s_d;
    __shared__ bool s_last;
    const int b = blockIdx.y, c = blockIdx.x;
    if (threadIdx.x < 32) {
        const Decision d = decide(p, b);
        if (threadIdx.x == 0) s_d = d;
    }
    __syncthreads();
    const Decision d = s_d;
    const bool residual = !d.last;
    if (d.state == 0) {
        const Best o = race(p, d, c, residual);
        if (threadIdx.x == 0) p.best[(size_t)b * p.chunks + c] = o;
    }
    if (threadIdx.x == 0) {
        __threadfence();
        s_last = atom_acq_rel_add_u32(p.tickets + b, 1) == (uint32_t)p.chunks - 1;
    }
    __syncthreads();
    if (!s_last) return;
    int chosen = d.chosen;
    if (d.state == 0) {
        Best o{0.0, -1, 0};
        for (int k = 0; k < p.chunks; ++k) {   // (in order of the tokens: ties stay with the first)
            const Best *q = p.best + (size_t)b * p.chunks + k;
            const double s = __ldcg(&q->score);
            const int v = __ldcg(&q->v);
            if (v >= 0 && (o.v < 0 || s > o.score)) o = Best{s, v, 0};
        }
        if (o.v < 0)   // nothing is left of p - q: p itself
            for (int k = 0; k < p.chunks; ++k) {
                const Best x = race(p, d, k, false);
                if (x.v >= 0 && (o.v < 0 || x.score > o.score)) o = x;
            }
        chosen = o.v;
    }
    for (int i = threadIdx.x; i < d.n; i += kThreads) p.tokens[d.r0 + i] = i < d.a ? p.drafts[d.r0 + i] : i == d.a ? chosen : -1;
    if (threadIdx.x == 0) p.accepted[b] = d.a;
}

struct Layout {
    size_t tickets, best, stats, total;
    int chunks;
};
Layout layout(int B, int T, int V, bool draft) {
    Layout L;
    L.chunks = (V + kChunk - 1) / kChunk;
    L.tickets = kBehindZero;
    L.best = align_up(L.tickets + (size_t)B * 4, 256);
    L.stats = align_up(L.best + (size_t)B * L.chunks * sizeof(Best), 256);
    L.total = align_up(L.stats + (size_t)T * (draft ? 2 : 1) * L.chunks * sizeof(Stat), 256);
    return L;
}

}  // namespace

size_t verify_workspace_bytes(int B, int T, int V) { return layout(B, T, V, true).total; }

cudaError_t launch_verify(const VerifyArgs &a, int B, int T, int V, void *ws, cudaStream_t s) {
    const Layout L = layout(B, T, V, a.draft != nullptr);
    const Params p{a.logits, a.draft, a.ls, a.ds, a.ns, a.drafts, a.cu, a.temperature, a.uniform, a.noise, a.tokens, a.accepted,
                   B, T, V, L.chunks, reinterpret_cast<Ctrl *>(ws), ws_at<uint32_t>(ws, L.tickets), ws_at<Best>(ws, L.best), ws_at<Stat>(ws, L.stats)};
    verify_stats_kernel<<<(unsigned)((T > 0 ? T : 1) * (a.draft ? 2 : 1) * L.chunks), kThreads, 0, s>>>(p);
    const cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess) return err;
    verify_choose_kernel<<<dim3((unsigned)L.chunks, (unsigned)B), kThreads, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace moe
