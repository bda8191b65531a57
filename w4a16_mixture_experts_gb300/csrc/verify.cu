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
// and sums of exponentials, a row of each sequence and its noise once more. Three
// launches: rows' statistics by chunks, over all rows at once (which row decides is
// known only after them); the decision, a CTA a sequence; the race, by laps of the
// deciding row, the last CTA of a sequence to finish joining them. (The decision in
// every CTA of the race instead: 77 us for 32 sequences of 4 drafts and 248320
// tokens; in the last CTA of a sequence's statistics: those took 44 us for 31.)
//
// A decision is made with the fewest bits that decide it. The rows' sums are fp32
// and every draft is tested, every race run, in fp32 with bounds on each value
// (kSlack below). What the bounds leave open is weighed in 64 bits, whose values are
// then off by the sums alone (kSum); what that leaves open too, about one draft or
// race in 10^5, with the sums of the one row formed again, first with fp32
// exponentials of exact arguments (kFine), then in 64 bits. (64-bit exponentials for
// all tokens of the deciding rows: 1429 us for 32 sequences of 4 drafts and 248320
// tokens.)
#include <math.h>

#include "kv4_kernels.cuh"
#include "step_kernels.cuh"

namespace moe {

namespace {

constexpr int kThreads = 256;
constexpr int kVecs = 8, kChunk = kThreads * 8 * kVecs;   // 16-byte loads of a thread and logits in a chunk of the statistics
constexpr int kRacePerSm = 4;
constexpr int kLapVecs = 4, kLap = kThreads * 8 * kLapVecs;   // ... and of the race
static_assert(kThreads * kLap >= 1 << 20, "a thread a lap");
constexpr int kList = 1024;   // places for tokens that the bounds leave; where there are more, all of the row are weighed
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kMinNoise = 1.17549435e-38f;
// How far values may be off, relative, with u = 2^-24 for a rounding to fp32.
// A row's sum: the rate is off by 1.3 u, and a difference of logits, its product with
// the rate and what is added to it by u each, so a term 2^-A of the largest by
// 3.3 u A log 2. Weighted with the terms the A are the row's entropy at most, 20 for
// 2^20 tokens: 46 u. Exponentials are off by 4 u and a term passes through 5 (its own,
// the warp's, the block's, two joins of chunks), and 4 products: 24 u. Additions one after
// another: 17 in a thread, 5 in a warp, 7 in a block, 12 over the chunks: 41 u. In all
// 111 u.
constexpr double kSum = 128 * 0x1p-24;
// The sum with fp32 exponentials (off by 2 steps) of exact arguments, added in 64 bits.
constexpr double kFine = 8 * 0x1p-24;
// An fp32 probability: A is 127 at most where it is not zero, so 291 u; the sum's 111 u, its
// logarithm's (up to 20) 22 u, the exponential's and the reciprocals' 4 u each, four products. In all 436 u.
constexpr float kSlack = 512 * 0x1p-24f;
constexpr float kSlackAbs = 2.4e-38f;   // and what fp32 holds as zero

struct alignas(16) Stat {       // of a chunk of a row
    float m, s;     // the largest logit, the sum of exp((l - m) / t): NaN where a logit is NaN or +inf
    int arg, pad;   // (t = 0) the first place of m
};

constexpr int kWritten = -2, kSeveral = -3;
struct Best {           // of a lap: the token ahead, and bounds on its score
    double low, high;
    int v, pad;         // -1: none has a weight; kSeveral: the bounds are of all tokens that may be ahead
};

struct Params {
    const uint16_t *logits, *draft;
    long long ls, ds, ns;
    const int32_t *drafts, *cu;
    const float *temperature, *uniform, *noise;
    int32_t *tokens, *accepted;
    int B, T, V, chunks, laps;
    Ctrl *ctrl;
    uint32_t *tickets;   // [B]: CTAs of a sequence's race done; cleared with the decision
    struct Decision *decisions;   // [B]
    Best *best;          // [B][laps]
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

// Offsets that do not rise within [0, T] bound no rows.
__device__ inline Rows rows_of(const Params &p, int b) {
    const int a = p.cu[b], e = p.cu[b + 1];
    return a < 0 || e > p.T || e < a ? Rows{0, 0} : Rows{a, e - a};
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
constexpr float kMaxRate = 1e30f, kMinRate = 1e-36f;
__device__ inline float rate_of(float t) { return fminf(kLog2e / t, kMaxRate); }
// fp32 bounds nothing where the rate was cut (logits that differ by less than 1e-30 may differ in
// weight) or is so small that logits may count whose difference passes fp32's range.
__device__ inline bool no_bounds(float rate) { return rate >= kMaxRate || rate <= kMinRate; }

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

// Adds the exponentials of two logits, a sum each.
__device__ inline void add_exp2(float &a, float &b, uint32_t w, float rate, float from) {
    asm("{\n\t.reg .b64 x, y, z;\n\t.reg .f32 u, v;\n\t.reg .b32 lo, hi;\n\t"
        "shl.b32 lo, %2, 16;\n\tand.b32 hi, %2, 0xffff0000;\n\t"
        "mov.b64 x, {lo, hi};\n\tmov.b64 y, {%3, %3};\n\tmov.b64 z, {%4, %4};\n\t"
        "fma.rn.f32x2 x, x, y, z;\n\tmov.b64 {u, v}, x;\n\t"
        "ex2.approx.ftz.f32 u, u;\n\tex2.approx.ftz.f32 v, v;\n\t"
        "mov.b64 x, {u, v};\n\tmov.b64 y, {%0, %1};\n\tadd.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "+f"(a), "+f"(b)
        : "r"(w), "f"(rate), "f"(from));
}

__device__ inline float warp_max(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
__device__ inline float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// s * exp2((m - top) * rate), also where both are -inf and s is 0 (or NaN, which stays).
__device__ inline float lowered(float s, float m, float top, float rate) { return m == top ? s : s * ex2((m - top) * rate); }

struct Row {
    float m, z;     // the largest logit, the sum of exp((l - m) / t)
    int arg;        // (t = 0) the first place of m
    bool bad;       // no distribution: a NaN, a +inf, nothing but -inf
};

// A whole warp calls it, a chunk a lane.
__device__ inline Row row_stats(const Params &p, int r, int side, float rate) {
    const Stat *st = p.stats + ((size_t)r * (p.draft ? 2 : 1) + side) * p.chunks;
    const int lane = threadIdx.x & 31;
    Row o{-INFINITY, 0.f, 0x7fffffff, false};
    for (int c0 = 0; c0 < p.chunks; c0 += 32) {
        const bool in = c0 + lane < p.chunks;
        const float4 v = in ? __ldcg(reinterpret_cast<const float4 *>(st + c0 + lane)) : make_float4(-INFINITY, 0.f, __int_as_float(0x7fffffff), 0.f);
        const Stat s{v.x, v.y, __float_as_int(v.z), 0};
        const float m = fmaxf(o.m, warp_max(s.m));
        const int arg = __reduce_min_sync(0xffffffffu, s.m == m ? s.arg : 0x7fffffff);
        o.arg = m > o.m ? arg : min(o.arg, arg);
        o.z = lowered(o.z, o.m, m, rate) + warp_sum(lowered(s.s, s.m, m, rate));
        o.m = m;
    }
    o.bad = !(o.m > -INFINITY && o.z < INFINITY);
    return o;
}

// How well a row's sums are known: not at all (no_bounds), by the statistics (kSum), kFine, 64 bits.
enum Known { kUnknown, kKnown, kKnownFine, kKnownFull };
__device__ inline double off_by(int known) { return known == kKnown ? kSum : kFine; }

struct Decision {
    double zp, zq;      // the deciding row's sums
    int r0, n, a;       // rows of the sequence, accepted drafts
    int chosen;         // the next token where the race does not decide (state 1)
    int state, last;    // the deciding row is the last
    int x;              // the draft that it refused: its q is 1 without draft logits (< 0: none)
    int known;
    float t, rate, mp, mq;
};

// The sum of exp((l - m) / t) over a row's logits l, the largest m: all threads call it and get it.
// 64-bit exponentials: 1.25 ms for 248320 logits in one CTA; fp32 ones: 0.11 ms.
template <bool kFull>
__device__ __noinline__ double row_sum(const uint16_t *row, int V, float m, float t) {
    __shared__ double s_sum[kThreads / 32];
    const double inv = 1.0 / t;
    const float inv_h = (float)inv, inv_l = (float)(inv - inv_h);
    double s = 0.0;
    float sh = 0.f, sl = 0.f;   // the sum and what its roundings left
    for (int v = threadIdx.x * 8; v < V; v += kThreads * 8) {
        float x[8];
        unpack8(load8(row, v, V), x);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (kFull) {
                s += exp(((double)x[i] - m) * inv);
                continue;
            }
            // the argument and its rest: a difference and a product with what their roundings leave
            const float d = x[i] - m, back = d - x[i], dl = (x[i] - (d - back)) - (m + back);
            const float a = d * inv_h, al = fmaf(d, inv_h, -a) + fmaf(d, inv_l, dl * inv_h);
            if (!(a > -100.f)) continue;   // (nothing beside the largest term, 1)
            const float e = expf(a), term = fmaf(e, al, e), sum = sh + term, there = sum - sh;
            sl += (sh - (sum - there)) + (term - there);
            sh = sum;
        }
    }
    if (!kFull) s = (double)sh + sl;
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s_sum[threadIdx.x >> 5] = s;
    __syncthreads();
    s = 0.0;
    for (int w = 0; w < kThreads / 32; ++w) s += s_sum[w];
    return s;
}
// The next better sum.
__device__ inline int better(int known) { return known == kKnown ? kKnownFine : kKnownFull; }
__device__ inline double row_sum(int known, const uint16_t *row, int V, float m, float t) {
    return known == kKnownFine ? row_sum<false>(row, V, m, t) : row_sum<true>(row, V, m, t);
}

// In 64 bits: is u * q(x) < p(x)? 1, 0, or 2: the sums are not known well enough.
__device__ __noinline__ int accepts(float u, float l, float mp, double zp, bool has_q, float ld, float mq, double zq, float t, int known) {
    const double pv = exp(((double)l - mp) / t) / zp, uq = (double)u * (has_q ? exp(((double)ld - mq) / t) / zq : 1.0);
    if (pv > 0.0 && uq > 0.0 && (known == kUnknown || (known != kKnownFull && fabs(pv - uq) <= off_by(known) * (pv + uq)))) return 2;
    return uq < pv;
}

struct Test {   // of a row's draft
    Row p, q;
    int x, stop, fault, last, open;
    float u, l, ld;
};

// A test that the statistics leave open, by better sums: all threads call it.
struct Closed {
    double zp, zq;
    int known, yes;
};
__device__ __noinline__ Closed close(const Params &p, const Test &e, int r, float t, int known) {
    Closed o{1.0, 1.0, known, 2};
    do {
        o.known = better(o.known);
        o.zp = row_sum(o.known, p.logits + r * p.ls, p.V, e.p.m, t);
        if (p.draft) o.zq = row_sum(o.known, p.draft + r * p.ds, p.V, e.q.m, t);
        o.yes = accepts(e.u, e.l, e.p.m, o.zp, p.draft != nullptr, e.ld, e.q.m, o.zq, t, o.known);
    } while (o.yes == 2);
    return o;
}

// What becomes of sequence b, which has rows: all threads call it, a row a warp.
__device__ inline Decision decide(const Params &p, int b, const Rows &rows) {
    __shared__ Test s_test[kThreads / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    Decision d{1.0, 1.0, rows.r0, rows.n, 0, -1, 1, 0, -1, kKnown, p.temperature ? p.temperature[b] : 1.f, 0.f, 0.f, 0.f};
    const bool greedy = d.t == 0.f;
    if (!(d.t >= 0.f && d.t < INFINITY)) {
        if (threadIdx.x == 0) set_error(p.ctrl, MOE_ERR_DEVICE);
        return d;
    }
    d.rate = greedy ? 1.f : rate_of(d.t);
    const int sums = !greedy && no_bounds(d.rate) ? kUnknown : kKnown;   // how well the statistics' are known
    for (int i0 = 0;; i0 += kThreads / 32) {
        const int i = i0 + warp, r = rows.r0 + i;
        Test t{{0.f, 1.f, 0, false}, {0.f, 1.f, 0, false}, -1, 1, 0, 0, 0, 0.f, 0.f, 0.f};
        if (i < rows.n) {
            t.last = i == rows.n - 1;
            const bool has_q = p.draft && !greedy && !t.last;
            const int x = t.last ? -1 : p.drafts[r];
            const bool known = (unsigned)x < (unsigned)p.V;
            const float l = known ? bf16_bits_to_f32(p.logits[r * p.ls + x]) : 0.f;
            const float ld = known && has_q ? bf16_bits_to_f32(p.draft[r * p.ds + x]) : 0.f;
            const float u = t.last ? 0.f : p.uniform[r];
            t.p = row_stats(p, r, 0, d.rate);
            if (has_q) t.q = row_stats(p, r, 1, d.rate);
            t.x = t.last ? -1 : known ? x : -2;
            t.fault = t.p.bad || t.q.bad;
            if (!t.last && !t.fault && known) {
                if (greedy) {
                    t.stop = t.p.arg != x;
                } else {
                    const float pv = ex2((l - t.p.m) * d.rate) / t.p.z, uq = has_q ? u * (ex2((ld - t.q.m) * d.rate) / t.q.z) : u;
                    if (sums == kKnown && fabsf(pv - uq) > kSlack * (pv + fabsf(uq)) && fmaxf(pv, fabsf(uq)) > 1e-30f) {
                        t.stop = !(uq < pv);
                    } else {
                        const int yes = accepts(u, l, t.p.m, t.p.z, has_q, ld, t.q.m, t.q.z, d.t, sums);
                        t.stop = yes != 1;
                        t.open = yes == 2;
                        t.u = u;
                        t.l = l;
                        t.ld = ld;
                    }
                }
            }
        }
        if (i0) __syncthreads();
        if (lane == 0) s_test[warp] = t;
        __syncthreads();
        int k = 0;
        for (; k < kThreads / 32; ++k) {
            const Test &e = s_test[k];
            if (!e.stop) continue;
            d.known = sums;
            d.zp = e.p.z;
            d.zq = e.q.z;
            if (!e.open) break;
            const Closed o = close(p, e, rows.r0 + i0 + k, d.t, sums);
            d.known = o.known;
            d.zp = o.zp;
            d.zq = o.zq;
            if (!o.yes) break;
        }
        if (k == kThreads / 32) continue;
        const Test &e = s_test[k];
        d.a = i0 + k;
        d.last = e.last;
        d.x = e.x;
        d.mp = e.p.m;
        d.mq = e.q.m;
        if ((e.fault || e.x == -2) && threadIdx.x == 0) set_error(p.ctrl, MOE_ERR_DEVICE);
        d.state = e.fault || greedy;
        d.chosen = e.fault ? -1 : e.p.arg;
        return d;
    }
}

__global__ void __launch_bounds__(kThreads) verify_stats_kernel(const __grid_constant__ Params p) {
    __shared__ float s_m[kThreads / 32], s_s[kThreads / 32];
    __shared__ int s_arg;
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = blockIdx.x % p.chunks, rw = blockIdx.x / p.chunks, sides = p.draft ? 2 : 1;
    const int side = rw / p.T, r = rw - side * p.T;
    const int b = sequence_of(p, r);
    if (b < 0) return;
    const Rows rows = rows_of(p, b);
    const float t = p.temperature ? p.temperature[b] : 1.f;
    if (side && (t == 0.f || r == rows.r0 + rows.n - 1)) return;   // not looked at
    const float rate = t == 0.f ? 1.f : rate_of(t);
    const uint16_t *row = side ? p.draft + r * p.ds : p.logits + r * p.ls;
    uint4 v[kVecs];
    const int v0 = c * kChunk + threadIdx.x * 8;
    if ((c + 1) * kChunk <= p.V) {
#pragma unroll
        for (int i = 0; i < kVecs; ++i) v[i] = *reinterpret_cast<const uint4 *>(row + v0 + i * kThreads * 8);
    } else {
#pragma unroll
        for (int i = 0; i < kVecs; ++i) v[i] = load8(row, v0 + i * kThreads * 8, p.V);
    }
    __nv_bfloat162 m2 = __floats2bfloat162_rn(-INFINITY, -INFINITY);
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) m2 = __hmax2(m2, *reinterpret_cast<const __nv_bfloat162 *>(&w[j]));
    }
    const float mine = fmaxf(__low2float(m2), __high2float(m2)), top = warp_max(mine);
    // The sum is taken against the whole number of octaves nearest to the largest (one rounding a
    // term), and brought to the largest itself at the end; where that number is not small, term by term.
    float s, part[4] = {0.f, 0.f, 0.f, 0.f};
    const float octaves = rintf(top * rate);
    if (fabsf(octaves) < 65536.f) {
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) add_exp2(part[j & 2], part[(j & 2) + 1], w[j], rate, -octaves);
        }
        s = ((part[0] + part[1]) + (part[2] + part[3])) * ex2(fmaf(-top, rate, octaves));
    } else {
        const float from = top == -INFINITY ? 0.f : top;
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            float x[8];
            unpack8(v[i], x);
#pragma unroll
            for (int j = 0; j < 8; ++j) part[j & 3] += ex2((x[j] - from) * rate);
        }
        s = (part[0] + part[1]) + (part[2] + part[3]);
    }
    s = warp_sum(s);
    if (lane == 0) {
        s_m[warp] = top;
        s_s[warp] = s;
    }
    if (threadIdx.x == 0) s_arg = 0x7fffffff;
    __syncthreads();
    float all = s_m[0];
#pragma unroll
    for (int w = 1; w < kThreads / 32; ++w) all = fmaxf(all, s_m[w]);
    if (t == 0.f) {
        if (mine == all) {
            int first = 0x7fffffff;
#pragma unroll
            for (int i = kVecs - 1; i >= 0; --i) {
                float x[8];
                unpack8(v[i], x);
#pragma unroll
                for (int j = 7; j >= 0; --j)
                    if (x[j] == all) first = v0 + i * kThreads * 8 + j;
            }
            atomicMin(&s_arg, first);
        }
        __syncthreads();
    }
    if (threadIdx.x == 0) {
        float sum = 0.f;
        for (int w = 0; w < kThreads / 32; ++w) sum += lowered(s_s[w], s_m[w], all, rate);
        p.stats[((size_t)r * sides + side) * p.chunks + c] = Stat{all, sum, s_arg, 0};
    }
}

// The decision for each sequence, and what follows where no race does. Offsets out of
// order anywhere leave rows without statistics: then nothing is accepted.
__global__ void __launch_bounds__(kThreads) verify_decide_kernel(const __grid_constant__ Params p) {
    pdl_wait();
    pdl_launch_dependents();
    const int b = blockIdx.x;
    bool order = true;
    for (int i = threadIdx.x; i < p.B; i += kThreads) order &= p.cu[i] >= 0 && p.cu[i] <= p.cu[i + 1] && p.cu[i + 1] <= p.T;
    order = __syncthreads_and(order);
    const Rows rows = rows_of(p, b);
    Decision d{1.0, 1.0, rows.r0, rows.n, 0, -1, 1, 0, -1, kKnown, 0.f, 0.f, 0.f, 0.f};
    if (!order && threadIdx.x == 0) set_error(p.ctrl, MOE_ERR_DEVICE);
    if (order && rows.n > 0) d = decide(p, b, rows);
    if (threadIdx.x == 0) {
        p.decisions[b] = d;
        p.tickets[b] = 0;
        p.accepted[b] = d.a;
    }
    for (int i = threadIdx.x; i < rows.n; i += kThreads)   // (the race writes the one at d.a where it is run)
        if (i != d.a || d.state) p.tokens[rows.r0 + i] = i < d.a ? p.drafts[rows.r0 + i] : i == d.a ? d.chosen : -1;
}

// The deciding row's values and what a token weighs in it.
struct Weigh {
    const Params &p;
    const Decision &d;
    const uint16_t *row, *drow;   // drow: where q is taken off
    const float *noise;
    int none;                     // a token without weight

    __device__ Weigh(const Params &p_, const Decision &d_, int b, bool residual)
        : p(p_), d(d_), row(p_.logits + (d_.r0 + d_.a) * p_.ls), drow(residual && p_.draft ? p_.draft + (d_.r0 + d_.a) * p_.ds : nullptr),
          noise(p_.noise + b * p_.ns), none(residual && !p_.draft ? d_.x : -1) {}

    __device__ static float noise_of(float e) { return e >= kMinNoise ? e : kMinNoise; }

};

// (score, v) of the token that is ahead of all of the block's: all threads call it.
__device__ inline void ahead(double &score, int &v) {
    __shared__ double s_score[kThreads / 32];
    __shared__ int s_v[kThreads / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    auto join = [&](double os, int ov) {
        if (ov >= 0 && (v < 0 || os > score || (os == score && ov < v))) {
            score = os;
            v = ov;
        }
    };
    for (int o = 16; o > 0; o >>= 1) join(__shfl_xor_sync(0xffffffffu, score, o), __shfl_xor_sync(0xffffffffu, v, o));
    __syncthreads();
    if (lane == 0) {
        s_score[warp] = score;
        s_v[warp] = v;
    }
    __syncthreads();
    for (int w = 0; w < kThreads / 32; ++w) join(s_score[w], s_v[w]);
}

// Whose score is the largest, in 64 bits, of n tokens: those of a list (negative: none), or from
// `first` on? All threads call it and get the answer. The sums are formed again where they leave that
// open, which they can only where q is taken off: else they are one factor of all scores.
__device__ __noinline__ Best settle(const Params &p, int b, bool residual, const int *list, int first, int n) {
    __shared__ Best s_best;
    const Decision d = p.decisions[b];
    const Weigh w(p, d, b, residual);
    double zp = d.zp, zq = d.zq;
    int known = w.drow ? d.known : kKnownFull;
    for (;;) {
        const bool full = known == kKnownFull;
        const double off = full ? 0.0 : off_by(known);
        double low = 0.0, high = 0.0, second = 0.0;   // bounds on the scores: the highest, and the next one after that
        int who = -1;
        if (known != kUnknown) {
            for (int k = threadIdx.x; k < n; k += kThreads) {
                const int v = list ? list[k] : first + k;
                if (v < 0 || v == w.none) continue;
                const double pv = exp(((double)bf16_bits_to_f32(w.row[v]) - d.mp) / d.t) / zp;
                const double qv = w.drow ? exp(((double)bf16_bits_to_f32(w.drow[v]) - d.mq) / d.t) / zq : 0.0;
                const double e = Weigh::noise_of(w.noise[v]), more = pv * (1.0 + off) - qv * (1.0 - off);
                if (!(more > 0.0)) continue;
                low = fmax(low, (pv * (1.0 - off) - qv * (1.0 + off)) / e);
                const double hi = more / e;
                if (who < 0 || hi > high || (hi == high && v < who)) {
                    second = who < 0 ? 0.0 : high;
                    high = hi;
                    who = v;
                } else {
                    second = fmax(second, hi);
                }
            }
            if (full) {
                ahead(high, who);
                return Best{high, high, who, 0};
            }
            int any = 0;
            ahead(low, any);   // (the largest of the lower bounds)
            const bool in = who >= 0 && high >= low;
            const int some = __syncthreads_count(in), many = __syncthreads_or(second >= low);
            if (some == 0) return Best{0.0, 0.0, -1, 0};   // (none can have a weight)
            if (some == 1 && !many && low > 0.0) {
                if (in) s_best = Best{low, high, who, 0};
                __syncthreads();
                const Best o = s_best;
                __syncthreads();
                return o;
            }
        }
        known = better(known);
        zp = row_sum(known, w.row, p.V, d.mp, d.t);
        zq = row_sum(known, w.drow, p.V, d.mq, d.t);
    }
}

__device__ inline void noise8(const float *noise, int v, int V, float (&e)[8]) {
    if (v + 8 <= V) {
        const float4 a = *reinterpret_cast<const float4 *>(noise + v), b = *reinterpret_cast<const float4 *>(noise + v + 4);
        e[0] = a.x, e[1] = a.y, e[2] = a.z, e[3] = a.w, e[4] = b.x, e[5] = b.y, e[6] = b.z, e[7] = b.w;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] = v + i < V ? noise[v + i] : 1.f;
    }
}

// each(v, low, high) for pairs of tokens of lap c of the deciding row and bounds on their scores; high <= 0: no weight
template <class Each>
__device__ inline void pass(const Weigh &w, int c, Each &&each) {
    const Params &p = w.p;
    const Decision &d = w.d;
    const int v0 = c * kLap + threadIdx.x * 8;
    const float lzp = -log2f((float)d.zp), lzq = -log2f((float)d.zq);
    const float2 m2 = make_float2(-d.mp, -d.mp), mq2 = make_float2(-d.mq, -d.mq), rate = make_float2(d.rate, d.rate);
    const float2 zp = make_float2(lzp, lzp), zq = make_float2(lzq, lzq);
    const float2 less = make_float2(1.f - kSlack, 1.f - kSlack), more = make_float2(1.f + kSlack, 1.f + kSlack);
    const float2 neg_less = make_float2(kSlack - 1.f, kSlack - 1.f), neg_more = make_float2(-1.f - kSlack, -1.f - kSlack);
    const float2 off = make_float2(kSlackAbs, kSlackAbs), neg_off = make_float2(-kSlackAbs, -kSlackAbs);
#pragma unroll 2
    for (int i = 0; i < kLapVecs; ++i) {
        const int at = v0 + i * kThreads * 8;
        const uint4 l = load8(w.row, at, p.V), ld = w.drow ? load8(w.drow, at, p.V) : make_uint4(0, 0, 0, 0);
        float e[8];
        noise8(w.noise, at, p.V, e);
        const uint32_t lw[4] = {l.x, l.y, l.z, l.w}, dw[4] = {ld.x, ld.y, ld.z, ld.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float2 x = make_float2(__uint_as_float(lw[j] << 16), __uint_as_float(lw[j] & 0xffff0000u));
            x = __ffma2_rn(__fadd2_rn(x, m2), rate, zp);
            x = make_float2(ex2(x.x), ex2(x.y));
            float2 lo = __ffma2_rn(x, less, neg_off), hi = __ffma2_rn(x, more, off);
            if (w.drow) {
                float2 y = make_float2(__uint_as_float(dw[j] << 16), __uint_as_float(dw[j] & 0xffff0000u));
                y = __ffma2_rn(__fadd2_rn(y, mq2), rate, zq);
                y = make_float2(ex2(y.x), ex2(y.y));
                lo = __ffma2_rn(y, neg_more, lo);
                hi = __ffma2_rn(y, neg_less, hi);
            }
            const float2 inv = make_float2(__fdividef(1.f, Weigh::noise_of(e[2 * j])), __fdividef(1.f, Weigh::noise_of(e[2 * j + 1])));
            // (above 2^126 the quotient is given as zero: there it is a lower bound alone)
            lo = __fmul2_rn(lo, inv);
            hi = __fmul2_rn(hi, make_float2(fmaxf(inv.x, 0x1p-126f), fmaxf(inv.y, 0x1p-126f)));
            if (w.none >> 1 == (at >> 1) + j) {   // (a token without weight)
                if (w.none & 1) lo.y = 0.f, hi.y = -1.f;
                else lo.x = 0.f, hi.x = -1.f;
            }
            each(at + 2 * j, lo, hi);
        }
    }
}

// The race over the tokens of lap c of the deciding row.
__device__ inline Best race(const Weigh &w, int c) {
    __shared__ float s_low[kThreads / 32];
    const Params &p = w.p;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (no_bounds(w.d.rate)) return Best{0.0, INFINITY, kSeveral, 0};   // (no bounds)
    // the two highest bounds of the thread's tokens, and whose the first is
    float low = 0.f, high = -1.f, second = -1.f;
    int who = -1;
    pass(w, c, [&](int v, float2 lo, float2 hi) {
        low = fmaxf(low, fmaxf(lo.x, lo.y));
        second = fmaxf(second, fminf(high, hi.x));
        who = hi.x > high ? v : who;
        high = fmaxf(high, hi.x);
        second = fmaxf(second, fminf(high, hi.y));
        who = hi.y > high ? v + 1 : who;
        high = fmaxf(high, hi.y);
    });
    low = warp_max(low);
    __syncthreads();
    if (lane == 0) s_low[warp] = low;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kThreads / 32; ++k) low = fmaxf(low, s_low[k]);
    // who may be ahead of all: mostly one
    const bool in = high >= low;
    if (!__syncthreads_or(in)) return Best{0.0, 0.0, -1, 0};
    const int some = __syncthreads_count(in), many = __syncthreads_or(second >= low);
    if (some == 1 && !many && low > 0.f) {   // (and it has a weight)
        if (in) p.best[blockIdx.y * (size_t)p.laps + c] = Best{low, high, who, 0};
        return Best{0.0, 0.0, kWritten, 0};
    }
    double top = high;
    ahead(top, who);
    return Best{low, top, kSeveral, 0};
}

__global__ void __launch_bounds__(kThreads, kRacePerSm) verify_race_kernel(const __grid_constant__ Params p) {
    __shared__ bool s_last;
    __shared__ int s_list[kList], s_n;   // tokens that are weighed in 64 bits
    __shared__ bool s_open[kThreads];
    const int b = blockIdx.y, c = blockIdx.x;
    {   // (the noise on its way while the decision is made)
        const int v = c * kLap + threadIdx.x * 32;
        if (v < min((c + 1) * kLap, p.V)) asm volatile("prefetch.global.L2 [%0];" ::"l"(p.noise + b * p.ns + v));
    }
    pdl_wait();
    pdl_launch_dependents();
    const Decision d = p.decisions[b];
    if (d.state) return;
    const Weigh w(p, d, b, !d.last);
    const Best o = race(w, c);
    if (threadIdx.x == 0 && o.v != kWritten) p.best[(size_t)b * p.laps + c] = o;
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();
        s_last = atom_acq_rel_add_u32(p.tickets + b, 1) == (uint32_t)p.laps - 1;
        __threadfence();
    }
    __syncthreads();
    if (!s_last) return;
    // ---- the laps' first ones against one another
    const Best *const best = p.best + (size_t)b * p.laps;
    const bool there = threadIdx.x < p.laps;
    const Best mine{there ? __ldcg(&best[threadIdx.x].low) : 0.0, there ? __ldcg(&best[threadIdx.x].high) : 0.0,
                    there ? __ldcg(&best[threadIdx.x].v) : -1, 0};
    double low = mine.low, none = 0.0;
    int v = 0;
    ahead(low, v);   // (the largest of the lower bounds)
    const bool in = mine.v != -1 && mine.high >= low;
    const int some = __syncthreads_count(in), several = __syncthreads_or(in && mine.v == kSeveral);
    v = in ? mine.v : -1;
    if (some <= 1 && !several) {
        ahead(none, v);
    } else {   // all tokens that reach that bound
        if (threadIdx.x == 0) s_n = 0;
        s_open[threadIdx.x] = v == kSeveral;
        __syncthreads();
        auto take = [&](int at, bool may) {
            if (!may || at >= p.V) return;
            const int i = atomicAdd(&s_n, 1);
            if (i < kList) s_list[i] = at;
        };
        take(v, v >= 0);
        const bool bounds = !no_bounds(d.rate);
        for (int k = 0; bounds && k < p.laps; ++k)
            if (s_open[k])
                pass(w, k, [&](int at, float2, float2 hi) {
                    take(at, hi.x >= low);
                    take(at + 1, hi.y >= low);
                });
        __syncthreads();
        v = bounds && s_n <= kList ? settle(p, b, !d.last, s_list, 0, s_n).v : settle(p, b, !d.last, nullptr, 0, p.V).v;
    }
    if (v < 0) v = settle(p, b, false, nullptr, 0, p.V).v;   // nothing is left of p - q: p itself
    if (threadIdx.x == 0) p.tokens[d.r0 + d.a] = v;
}

struct Layout {
    size_t tickets, decisions, best, stats, total;
    int chunks, laps;
};
Layout layout(int B, int T, int V, bool draft) {
    Layout L;
    L.chunks = (V + kChunk - 1) / kChunk;
    L.laps = (V + kLap - 1) / kLap;
    L.tickets = kBehindZero;
    L.decisions = align_up(L.tickets + (size_t)B * 4, 256);
    L.best = align_up(L.decisions + (size_t)B * sizeof(Decision), 256);
    L.stats = align_up(L.best + (size_t)B * L.laps * sizeof(Best), 256);
    L.total = align_up(L.stats + (size_t)T * (draft ? 2 : 1) * L.chunks * sizeof(Stat), 256);
    return L;
}

}  // namespace

size_t verify_workspace_bytes(int B, int T, int V) { return layout(B, T, V, true).total; }

cudaError_t launch_verify(const VerifyArgs &a, int B, int T, int V, void *ws, cudaStream_t s) {
    const Layout L = layout(B, T, V, a.draft != nullptr);
    const Params p{a.logits, a.draft, a.ls, a.ds, a.ns, a.drafts, a.cu, a.temperature, a.uniform, a.noise, a.tokens, a.accepted,
                   B, T, V, L.chunks, L.laps, reinterpret_cast<Ctrl *>(ws), ws_at<uint32_t>(ws, L.tickets), ws_at<Decision>(ws, L.decisions), ws_at<Best>(ws, L.best), ws_at<Stat>(ws, L.stats)};
    cudaError_t err = T == 0 ? cudaSuccess : launch_pdl(verify_stats_kernel, dim3((unsigned)(T * (a.draft ? 2 : 1) * L.chunks)), kThreads, 0, s, p);
    if (err == cudaSuccess) err = launch_pdl(verify_decide_kernel, dim3((unsigned)B), kThreads, 0, s, p);
    if (err == cudaSuccess && T > 0) err = launch_pdl(verify_race_kernel, dim3((unsigned)L.laps, (unsigned)B), kThreads, 0, s, p);
    return err;
}

}  // namespace moe
