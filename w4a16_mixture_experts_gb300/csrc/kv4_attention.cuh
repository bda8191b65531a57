// What the attention kernels over the 4-bit cache share: their arguments, how
// the work is dealt to the CTAs, and how an item's parts are joined.
//
// An item is up to R query rows of one (sequence, KV head); row r of a sequence
// is query r / G, head r % G of the group. Its work is a number of units, each a
// fixed count of keys, and what beginning and ending it costs, as kLead units
// before those. All items' units lie one after another and CTA c of C takes the
// units [U c / C, U (c + 1) / C), whatever items they belong to: an even share
// for any mix of lengths. (A border among an item's leading units is one before
// it.) The parts of an item that lies in several
// CTAs' shares are joined, in the CTAs' order, by a second kernel, which the
// whole card runs. (The last of the CTAs to finish joining them alone took up to
// 60 us of a prompt chunk's 180, and its fence and ticket 1 us of the others.)
#pragma once

#include <cuda_fp16.h>

#include "kv4.cuh"

namespace moe {
namespace kv4 {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kMaxSeqs = 4096;       // of a call
constexpr float kNoMax = -3e38f;   // below every score: nothing seen yet

// Up to so many rows of a sequence share one streaming pass; calls with more take
// the kernel with two tiles of 128 rows. (4 KV heads x 8, D = 128, us there and here:
// 24 sequences of 1400 to 2780 keys, 32 rows 38 and 52, 40 rows 49 and 52, 72 rows 70 and
// 55; 96 of 400 to 800 keys, 32 rows 58 and 90, 40 rows 97 and 90; 4 of 15000 to 30000
// keys, 32 rows 50 and 62, 40 rows 56 and 62, 72 rows 74 and 62. D = 64: 32 rows 29 and
// 35, 50 and 57, 39 and 46; 40 rows 38 and 35, 85 and 57, 46 and 46.)
constexpr int kDecodeRows = 32;
constexpr int kPromptRows = 256;

// Partial results of at most so many CTAs; fixed figures, so that the
// workspace's size does not depend on the device (152 SMs; the streaming kernel
// runs up to four CTAs on each).
constexpr int kMaxCtas = 640, kMaxPromptCtas = 160;
// The parts and what joins them lie behind the regions that calls leave at
// zero, so that a workspace may serve the experts' calls too.
constexpr size_t kPartOff = 512 + (size_t)kMaxE * kCtrStride * 4;

// What a CTA leaves for the join: the item that it began and did not finish
// goes on to CTA `last` (0: there is none such).
struct Begun {
    int last, q0, h, qt, rows, pad[3];
};

struct Attn {
    Batch b;
    const uint16_t *q;
    moe_strides qs, os;
    moe_kv4_cache c;
    uint16_t *out;
    float *lse;
    Ctrl *ctrl;
    Begun *begun;       // [CTAs]
    float *part;        // [CTAs][2] x part_floats(R, D): a CTA's first part continues an item, its second begins one
    float scale;
    int Hq, G;
    // (instantiations with kWindow only) query at position i sees the keys j <= i with j > i - window or j < sinks
    int window, sinks;
};

// A part of an item: the exponent taken off each row's scores and the sum of its
// probabilities, the exponent taken off all its values, and the rows' values.
__host__ __device__ constexpr int part_floats(int R, int D) { return 2 * R + 4 + R * D; }

// A load that stays where it is written (the compiler would move it down to its
// first use, and its latency with it).
__device__ inline int ld_here(const int32_t *p) {
    int v;
    asm volatile("ld.global.nc.s32 %0, [%1];" : "=r"(v) : "l"(p));
    return v;
}

__device__ inline float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ inline float log2_approx(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 2^(e - 127) for a biased exponent e in [1, 254].
__device__ inline float pow2_biased(int e) { return __uint_as_float((uint32_t)e << 23); }

// The biased exponent that brings a row with the largest magnitude `bits`
// (bf16) to [1, 2) (or near it at the ends of the range): the row is
// multiplied by 2^(127 - e).
__device__ inline int norm_exponent(uint32_t bits) {
    const int e = (int)(bits >> 7) & 0xFF;
    return e == 0xFF ? 127 : min(max(e, 1), 253);
}

// Nibble pairs of a word as fp16x2, exactly. OR-ing a nibble into the mantissa
// of 1024 (bits 0-3) or of 64 (bits 4-7) gives 1024 + n or 64 + n, so two of
// the word's four pairs need no shift.
__device__ inline uint32_t nib_lo(uint32_t w) {   // bits 0-3 of each half, less 8
    uint32_t v;
    asm("lop3.b32 %0, %1, 0x000F000F, %2, 0xEA;" : "=r"(v) : "r"(w), "r"(0x64006400u));
    const __half2 r = __hsub2(*reinterpret_cast<__half2 *>(&v), __float2half2_rn(1032.f));
    return *reinterpret_cast<const uint32_t *>(&r);
}
__device__ inline uint32_t nib_hi(uint32_t w) {   // bits 4-7
    uint32_t v;
    asm("lop3.b32 %0, %1, 0x00F000F0, %2, 0xEA;" : "=r"(v) : "r"(w), "r"(0x54005400u));
    const __half2 r = __hsub2(*reinterpret_cast<__half2 *>(&v), __float2half2_rn(72.f));
    return *reinterpret_cast<const uint32_t *>(&r);
}

// Keys that the last row of row tile qt sees (all rows' keys are a prefix of them).
__device__ inline int tile_keys(const Seq &s, int G, int R, int qt) {
    const int last = (min((qt + 1) * R, s.nq * G) - 1) / G;
    return min(max(s.len - s.nq + last + 1, 0), s.len);
}

// First key that the window of the query at position pos holds.
__device__ inline int window_low(const Attn &p, int pos) { return pos >= p.window ? pos - p.window + 1 : 0; }

// With a window, what lies between the units with first keys (sinks) and the one where
// the window of the tile's first row begins is left out: units [0, head) of keys stay
// where they are, those from head on lie `skip` units further.
struct Gap {
    int head, skip;
    __device__ int key_unit(int u) const { return u < head ? u : u + skip; }
};
template <int kKeys>
__device__ inline Gap tile_gap(const Attn &p, const Seq &s, int R, int qt) {
    const int head = (int)(((unsigned)p.sinks + kKeys - 1) / kKeys);
    return Gap{head, max(window_low(p, s.len - s.nq + qt * R / p.G) / kKeys - head, 0)};
}

// Units of keys of a sequence's row tile: at least one, so that rows that see no
// key are written too.
template <int kKeys, bool kWindow>
__device__ inline int tile_units(const Attn &p, const Seq &s, int R, int qt) {
    const int all = (tile_keys(s, p.G, R, qt) + kKeys - 1) / kKeys;
    return max(1, kWindow ? all - tile_gap<kKeys>(p, s, R, qt).skip : all);
}

// The units of a sequence's row tiles, leading ones included, by a whole warp for
// one sequence.
template <int kKeys, int kLead, bool kWindow>
__device__ long long tiles_units(const Attn &p, const Seq &s, int R) {
    const int tiles = (s.nq * p.G + R - 1) / R;
    long long m = 0;
    for (int qt = threadIdx.x & 31; qt < tiles; qt += 32) m += tile_units<kKeys, kWindow>(p, s, R, qt) + kLead;
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) m += __shfl_xor_sync(0xffffffffu, m, x);
    return m;
}

// The units of one head of each thread's sequence. Sequences of more than two row
// tiles take a warp each: in a CTA of several warpgroups they are shared out over
// all warps through `mid` (12 prompts of up to 1500 queries: 99.2 us with one warp for
// them, 98.0 so).
template <int kThreads, int kKeys, int kLead, bool kWindow>
__device__ long long head_units(const Attn &p, const Seq &s, int R, long long *mid) {
    const int tiles = (s.nq * p.G + R - 1) / R, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long n = 0;
    if (tiles <= 2)
        for (int qt = 0; qt < tiles; ++qt) n += tile_units<kKeys, kWindow>(p, s, R, qt) + kLead;
    if (kThreads <= 128) {
        for (uint32_t many = __ballot_sync(0xffffffffu, tiles > 2); many; many &= many - 1) {
            const int src = __ffs(many) - 1;
            const long long m = tiles_units<kKeys, kLead, kWindow>(p, Seq{0, __shfl_sync(0xffffffffu, s.nq, src), __shfl_sync(0xffffffffu, s.len, src)}, R);
            if (lane == src) n = m;
        }
    } else if (__syncthreads_or(tiles > 2)) {
        mid[threadIdx.x] = tiles > 2 ? (long long)s.nq << 32 | (long long)s.len : -1;
        __syncthreads();
        for (int i = warp; i < kThreads; i += kThreads / 32) {
            const long long x = mid[i];
            if (x < 0) continue;
            const long long m = tiles_units<kKeys, kLead, kWindow>(p, Seq{0, (int)(x >> 32), (int)x}, R);
            if (lane == 0) mid[i] = m;
        }
        __syncthreads();
        if (tiles > 2) n = mid[threadIdx.x];
    }
    return n;
}

// The shares of C CTAs in U units: CTA c begins at floor(U c / C).
struct Shares {
    int U, C, q, r;
    __device__ Shares(int units, int ctas) : U(units), C(ctas), q(units / ctas), r(units % ctas) {}
    __device__ int begin(int c) const { return q * c + r * c / C; }
    __device__ int holder(int u) const {   // the CTA whose share holds unit u
        int c = min((int)((float)u * (float)C / (float)U), C - 1);   // (begin(C + 1) may pass 2^31)
        while (begin(c + 1) <= u) ++c;
        while (begin(c) > u) --c;
        return c;
    }
};

struct Item {
    int b, h, qt;
    int units, first, span;   // units of keys; the first of its units and their number, leading ones included
    Seq s;
};

// The row tile of a sequence and head (whose units begin at `at`) that holds unit u; a
// whole warp calls it.
template <int kKeys, int kLead, bool kWindow>
__device__ void find_tile(const Attn &p, int R, int u, int at, Item &it) {
    const int tiles = (it.s.nq * p.G + R - 1) / R, lane = threadIdx.x & 31;
    for (int q0 = 0;; q0 += 32) {   // 32 at a time
        const int n = q0 + lane < tiles ? tile_units<kKeys, kWindow>(p, it.s, R, q0 + lane) + kLead : 0;
        int inc = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += v;
        }
        const uint32_t here = __ballot_sync(0xffffffffu, u < at + inc);
        if (here || q0 + 32 >= tiles) {
            const int src = here ? __ffs(here) - 1 : 0;
            it.qt = q0 + src;
            it.span = __shfl_sync(0xffffffffu, n, src);
            it.units = it.span - kLead;
            it.first = at + __shfl_sync(0xffffffffu, inc - n, src);
            return;
        }
        at += __shfl_sync(0xffffffffu, inc, 31);
    }
}

// The shares, and the item that CTA c's begins in (where it has a share: c < C).
// All threads call it; it begins and ends with a barrier or more, between which
// `pre` is used where there are more than kThreads sequences. A total of 2^31
// units is refused as a value out of range.
template <int kThreads, int kKeys, int kLead, bool kWindow>
__device__ Shares first_item(const Attn &p, int R, int c, int *pre, long long *warp_sums, Item &shared, Item &it) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long total = 0, before = 0, per_head = 0, n = 0;
    Seq s{0, 0, 0};
    for (int b0 = 0; b0 < p.b.B; b0 += kThreads) {
        const int b = b0 + threadIdx.x;
        s = b < p.b.B ? seq_of(p.b, b, p.ctrl) : Seq{0, 0, 0};
        per_head = head_units<kThreads, kKeys, kLead, kWindow>(p, s, R, reinterpret_cast<long long *>(pre + kMaxSeqs));
        n = per_head * p.c.Hkv;
        long long inc = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long v = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += v;
        }
        if (b0 > 0) __syncthreads();   // (the last round's sums have been read)
        if (lane == 31) warp_sums[warp] = inc;
        __syncthreads();
        before = total + inc - n;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) {
            if (w < warp) before += warp_sums[w];
            total += warp_sums[w];
        }
        if (p.b.B > kThreads && b < p.b.B) pre[b] = (int)before;
    }
    if (total >= (1ll << 31)) {
        set_error(p.ctrl, MOE_ERR_DEVICE);
        total = 0;
    }
    Shares shares((int)total, total == 0 ? 1 : (int)min((long long)gridDim.x, total));
    if (total == 0) shares.C = 0;
    if (p.b.B > kThreads) __syncthreads();
    if (c < shares.C) {
        const int u = shares.begin(c);
        Item x;
        bool look = false;   // this warp looks for the row tile
        int at = 0;
        if (p.b.B <= kThreads) {   // the warp that has the sequence in its registers
            const uint32_t who = __ballot_sync(0xffffffffu, before <= u && u < before + n);
            const int src = who ? __ffs(who) - 1 : 0;
            look = who != 0;
            x.b = (threadIdx.x & ~31) + src;
            x.s = Seq{__shfl_sync(0xffffffffu, s.q0, src), __shfl_sync(0xffffffffu, s.nq, src), __shfl_sync(0xffffffffu, s.len, src)};
            per_head = __shfl_sync(0xffffffffu, per_head, src);
            at = (int)__shfl_sync(0xffffffffu, before, src);
        } else if (warp == 0) {
            int lo = 0;
            for (int hi = p.b.B; hi - lo > 1;) {
                const int mid = (lo + hi) >> 1;
                if (pre[mid] <= u) lo = mid;
                else hi = mid;
            }
            look = true;
            x.b = lo;   // (sequences without units share their successor's pre: the last of them is the one)
            x.s = seq_of(p.b, lo, p.ctrl);
            at = pre[lo];
            per_head = ((lo + 1 < p.b.B ? pre[lo + 1] : (int)total) - at) / p.c.Hkv;
        }
        if (look) {
            x.h = (u - at) / (int)per_head;
            find_tile<kKeys, kLead, kWindow>(p, R, u, at + x.h * (int)per_head, x);
            if (lane == 0) shared = x;
        }
    }
    __syncthreads();
    if (c < shares.C) it = shared;
    return shares;
}

// The item after `it`, where there is one.
template <int kKeys, int kLead, bool kWindow>
__device__ void next_item(const Attn &p, int R, Item &it) {
    it.first += it.span;
    if ((it.qt + 1) * R < it.s.nq * p.G) {
        ++it.qt;
    } else {
        it.qt = 0;
        if (++it.h == p.c.Hkv) {
            it.h = 0;
            do it.s = seq_of(p.b, ++it.b, p.ctrl);
            while (it.s.nq == 0);
        }
    }
    it.units = tile_units<kKeys, kWindow>(p, it.s, R, it.qt);
    it.span = it.units + kLead;
}

// 16 bytes of the cache into shared memory, asynchronously; zeros where there are none.
__device__ inline void copy16(void *dst, const void *src, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ inline void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All of the thread's copies but those of the last N groups have arrived.
template <int N>
__device__ inline void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ inline uint32_t bf16x2_of(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

__device__ inline uint32_t elect() {   // 1 in one lane of the warp, the same each time
    uint32_t lead;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(lead));
    return lead;
}

// The products and their completion, by the threads whose `lead` is set (one of a
// warp). Predicated, not branched around: in a branch of one lane the operands
// cannot be formed in the uniform registers that the instructions take them from.
__device__ inline void mma_ss(uint32_t lead, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %5, 0;\n\tsetp.ne.b32 q, %4, 0;\n\t"
        "@p tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, q;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(lead)
        : "memory");
}
__device__ inline void mma_ts(uint32_t lead, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %5, 0;\n\tsetp.ne.b32 q, %4, 0;\n\t"
        "@p tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, q;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(lead)
        : "memory");
}
__device__ inline void commit(uint32_t lead, uint64_t *bar) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %1, 0;\n\t"
        "@p tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)), "r"(lead)
        : "memory");
}

}  // namespace kv4
}  // namespace moe
