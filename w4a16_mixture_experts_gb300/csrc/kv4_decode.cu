// Attention over the paged 4-bit cache for few query rows a sequence (a decode
// step, or a few draft tokens): up to 32 rows (query, head of the group) share
// one pass over their keys.
//
// What bounds it: a key costs D + 4 bytes of HBM for all its rows, so the
// stream of codes; next come the instructions that make operands of its 2 D
// codes. So keys and values are the wide side (M = 128) of the tensor core's
// products, and a warpgroup takes 128 keys at a time:
//   S^T (128 keys x R rows) = K (128 x D) . Q^T: a thread writes a key's row into
//     its lane of tensor memory as the A operand and finds the key's R scores
//     there, so that its scales are its own and nothing is exchanged;
//   O^T (D x R) += V^T (D x 128 keys) . P^T: V and P go to shared memory as they
//     are, a row a key (MN-major operands).
// The codes come by cp.async, a warp its own 32 keys, a unit ahead of their use.
// (Loads into registers measured 90-125 us where this took 72: the waits for them
// are counted on few scoreboards, so that a shuffle or a shared load behind them
// waited for them too; and a row a lane from global memory visits each cache line
// four times, which had the L1 74% busy.) A warp-level form (mma.sync on fragments
// loaded from global memory) took 770 warp instructions for 32 keys at R = 8, for
// shuffles of scales and maxima, address arithmetic and a transposition of P.
//
// K and V enter as fp16 codes less 8, exactly, and a K scale multiplies its key's
// scores in fp32. A query row enters as fp16 less its own exponent, its largest
// value brought to [2^8, 2^9): exactly, but for values below 2^-25 of the largest,
// which are rounded at 2^-33 of it. (With K as e4m3 codes q + 8, which take a third
// of the instructions, and a query as two e4m3 numbers, what a value far above the
// rest left of them was rounded at 2^-18 of it, and 8 times it passed through the
// sums of keys that hold zeros beside it. That took 71.5 us for two sequences of
// 131072 keys, this 74.5.)
// A V scale multiplies its key's probabilities just before they are rounded to
// fp16, so what is rounded is what the key adds to the row. A row's exponents are
// therefore taken off not against its largest score but against its largest
// product of probability and scale, which is kept between 2^6 and 2^15: a product
// is rounded at 2^-31 of the row's largest at most, whatever the scales of keys
// that the row does not see or that have no probability in it, and a long tail
// of small ones is not lost. (Against the largest score, with the largest V scale
// brought to 1, it was 2^-25 of probability 1 and of that scale.) The sum of the
// probabilities alone follows the same exponent in fp32, up to 2^96 for keys whose
// values are next to nothing.
#include <type_traits>

#include "kv4_attention.cuh"
#include "tcgen05.cuh"

namespace moe {

namespace {

using namespace kv4;

constexpr int kKeys = 128;   // keys of a unit: a warpgroup's turn
// What an item's start and end count for, in units; it moves the balance, never a result. (96 sequences
// of 427 to 3994 keys, 8 rows, D = 128: 44.7, 42.5, 41.7, 42.6 us with 1, 2, 3, 4, D = 64: 36.2, 34.6,
// 34.7, 36.7 with 2, 3, 4, 6; 24 of 905 to 2757 keys, D = 64, 16 rows: 26.0, 25.7, 24.4, 25.5, 32 rows: 44.7,
// 43.9, 42.2, 41.4; D = 128, 16 rows: 32.6, 31.6, 30.6, 29.9, 32 rows: 56.1, 54.9, 53.7, 51.6 with 1, 2, 3, 4.)
template <int D>
constexpr int kLead = D == 128 ? 3 : 4;

template <int D, int R>
struct DecodeCfg {
    static constexpr int kThreads = 128;                  // a warpgroup
    static constexpr int kPerSm = R < 16 ? 4 : 3;         // CTAs an SM
    static constexpr int kNP = R < 16 ? 16 : R;           // columns of S^T and of O^T (R = 8: twice the same)
    static constexpr int kV = 128 * D * 2, kP = R * 256;  // bytes of the operands
    static constexpr int kPs = R < 32 ? 2 : 1;            // of P: two where they fit, one read while the next is written
    static constexpr int kQ = R * D * 2;
    static constexpr int kWarpRaw = 32 * D / 2, kRaw = 4 * kWarpRaw;   // codes of a warp's 32 keys (K or V), of all
    // tensor memory: K's row, scores, values' sums
    static constexpr int kColS = D / 2, kColO = kColS + kNP, kCols = kColO + kNP > 64 ? 128 : 64;
    static_assert(kColO + kNP <= kCols, "tensor memory");
    static constexpr int kSmem = kQ + kV + kPs * kP + 2 * kRaw;
    static constexpr int kChunks = D / 32;                // 16-byte pieces of a row of codes
};

template <int R>
struct DecodeShared {
    alignas(16) float c[R], m[R], wm[4][R];
    alignas(16) uint16_t scales[4][3][2][32];   // of a warp's units in turn: K's, V's
    uint64_t s_full, o_full;                    // scores formed, values added
    long long sums[4];
    Item first;
    int lim[R], we[4];                          // we: exponents of the warps' largest V scales in the item's first unit
    uint32_t tmem;
};

// Bounded wait on a phase. The hint lets a warp sleep through most of a wait (a
// poll returns after 20 us at the latest; the default hint polls about every 40
// clocks, and the other warps pay for it).
__device__ inline bool wait(uint64_t *bar, uint32_t parity) {
    uint32_t ok = 0;
    for (uint32_t i = 0; i < (1u << 15) && !ok; ++i)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 20000;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(smem_u32(bar)), "r"(parity)
            : "memory");
    return ok != 0;
}

// The CTA's barrier, returning the OR of v; and one that all but warp 0 only pass by.
__device__ inline bool bar_or(bool v) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, 0, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)v)
        : "memory");
    return r != 0;
}
__device__ inline void bar_pass(int warp) {
    if (warp == 0) asm volatile("barrier.cta.sync 1, 128;" ::: "memory");
    else asm volatile("barrier.cta.arrive 1, 128;" ::: "memory");
}

__device__ inline uint32_t idesc(int N, bool mn_major) {   // f16 operands, f32 sums
    return (1u << 4) | (mn_major ? 3u << 15 : 0u) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}

// V: rows of 128 swizzled bytes (64 values), 8 rows an atom of 1024; the second
// 64 values 16 KB on. (D = 64: no second block; M's upper half repeats the lower.)
template <int D>
__device__ inline uint64_t v_desc(const void *p) {
    return (uint64_t)((smem_u32(p) >> 4) & 0x3FFFu) | (uint64_t)(D == 128 ? 16384u >> 4 : 0u) << 16 | (uint64_t)(1024u >> 4) << 32 |
           (uint64_t)1u << 46 | (uint64_t)2u << 61;
}

// P: 16 bytes (8 rows) a key, keys side by side, the next 8 rows 2048 bytes on
// (8 rows only: the same again); no swizzle.
template <int R>
__device__ inline uint64_t p_desc(const void *p) {
    return (uint64_t)((smem_u32(p) >> 4) & 0x3FFFu) | (uint64_t)(128u >> 4) << 16 | (uint64_t)(R > 8 ? 2048u >> 4 : 0u) << 32 | (uint64_t)1u << 46;
}

// Q: rows of 128 swizzled bytes (64 values), 8 rows an atom of 1024, the next 8 rows
// behind it (8 rows only: the same again).
template <int R>
__device__ inline uint64_t q_desc(const void *p) {
    return (uint64_t)((smem_u32(p) >> 4) & 0x3FFFu) | (uint64_t)1u << 16 | (uint64_t)(R > 8 ? 1024u >> 4 : 0u) << 32 | (uint64_t)1u << 46 |
           (uint64_t)2u << 61;
}

__device__ inline uint32_t half2_of(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// Two values at a time.
__device__ inline void add2(float &a, float &b, float c, float d) {
    asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %3};\n\t"
        "add.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "+f"(a), "+f"(b)
        : "f"(c), "f"(d));
}
__device__ inline void mul2(float &a, float &b, float c, float d) {
    asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %3};\n\t"
        "mul.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "+f"(a), "+f"(b)
        : "f"(c), "f"(d));
}
__device__ inline void fma2(float &a, float &b, float c, float d, float e, float f) {   // (a, b) * (c, d) + (e, f)
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %3};\n\tmov.b64 z, {%4, %5};\n\t"
        "fma.rn.f32x2 x, x, y, z;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "+f"(a), "+f"(b)
        : "f"(c), "f"(d), "f"(e), "f"(f));
}

// N 32-bit columns of the thread's lane (the values are not to be read before the wait in it).
template <int N>
__device__ inline void ld_cols(uint32_t taddr, float (&v)[N]) {
    static_assert(N % 8 == 0);
    uint32_t r[N];
#pragma unroll
    for (int i = 0; i < N; i += 8)
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3]), "=r"(r[i + 4]), "=r"(r[i + 5]), "=r"(r[i + 6]), "=r"(r[i + 7])
                     : "r"(taddr + i));
#pragma unroll
    for (int i = 0; i < N; i += 8)
        asm volatile("tcgen05.wait::ld.sync.aligned;"
                     : "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]), "+r"(r[i + 5]), "+r"(r[i + 6]), "+r"(r[i + 7])
                     :
                     : "memory");
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = __uint_as_float(r[i]);
}

template <int N>
__device__ inline void st_cols(uint32_t taddr, const uint32_t (&v)[N]) {
    static_assert(N % 8 == 0);
#pragma unroll
    for (int i = 0; i < N; i += 8)
        asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr + i), "r"(v[i]), "r"(v[i + 1]),
                     "r"(v[i + 2]), "r"(v[i + 3]), "r"(v[i + 4]), "r"(v[i + 5]), "r"(v[i + 6]), "r"(v[i + 7])
                     : "memory");
}

// Row by row the maximum (above kNoMax) or the sum of a warp's values, into
// to[0 .. R): the lanes halve their rows at each exchange, so that R rows cost
// about R shuffles and not 5 R.
template <int R, bool kMax>
__device__ inline void reduce_rows(const float (&v)[R], float *to) {
    float x[R];
#pragma unroll
    for (int r = 0; r < R; ++r) x[r] = kMax ? fmaxf(v[r], kNoMax) : v[r];
    const int lane = threadIdx.x & 31;
    int row = 0;
#pragma unroll
    for (int o = 16, n = R; o > 0; o >>= 1) {
        if (n > 1) {
            n >>= 1;
            const bool upper = lane & o;
#pragma unroll
            for (int i = 0; i < R / 2; ++i)
                if (i < n) {
                    const float send = upper ? x[i] : x[i + n], keep = upper ? x[i + n] : x[i];
                    const float got = __shfl_xor_sync(0xffffffffu, send, o);
                    x[i] = kMax ? fmaxf(keep, got) : keep + got;
                }
            row += upper ? n : 0;
        } else {
            const float got = __shfl_xor_sync(0xffffffffu, x[0], o);
            x[0] = kMax ? fmaxf(x[0], got) : x[0] + got;
        }
    }
    if ((lane & (32 / R - 1)) == 0) to[row] = x[0];
}

template <int D, int R>
__global__ void __launch_bounds__(DecodeCfg<D, R>::kThreads, DecodeCfg<D, R>::kPerSm) kv4_decode_kernel(Attn p) {
    using Cfg = DecodeCfg<D, R>;
    extern __shared__ __align__(1024) uint8_t s_dyn[];
    uint8_t *const sQ = s_dyn, *const sV = sQ + Cfg::kQ, *const sP = sV + Cfg::kV;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint8_t *const k_raw = sP + Cfg::kPs * Cfg::kP + warp * Cfg::kWarpRaw, *const v_raw = k_raw + Cfg::kRaw;
    DecodeShared<R> &sh = *reinterpret_cast<DecodeShared<R> *>(s_dyn + Cfg::kSmem);
    // the sequences' prefix: needed only before the first operand is written
    int *const s_pre = reinterpret_cast<int *>(sV);
    static_assert(sizeof(int) * (kMaxSeqs + 1) <= (size_t)(Cfg::kV + Cfg::kPs * Cfg::kP), "prefix");

    if (tid == 0) {
        mbar_init(&sh.s_full, 1);
        mbar_init(&sh.o_full, 1);
        fence_mbar_init();
    }
    pdl_wait();
    pdl_launch_dependents();
    if (warp == 0) {   // (only now: the kernel ahead may hold tensor memory that it has not freed)
        tc::alloc(&sh.tmem, Cfg::kCols);
        tc::relinquish();
    }
    const int c = blockIdx.x;
    Item it;
    const Shares shares = first_item<Cfg::kThreads, kKeys, kLead<D>>(p, R, c, s_pre, sh.sums, sh.first, it);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tcol = sh.tmem, tlane = tcol + ((uint32_t)(warp * 32) << 16);
    // the units of keys of an item in this CTA's share
    const int u_end = c < shares.C ? shares.begin(c + 1) : 0;
    int st0 = 0, st1 = 0;
    if (c < shares.C) {
        st0 = max(shares.begin(c) - it.first - kLead<D>, 0);
        st1 = min(it.units, u_end - it.first - kLead<D>);
    }
    if (st1 <= st0) {   // (a share that ends among leading units has nothing to do)
        if (tid == 0) p.begun[c].last = 0;
        if (warp == 0) tc::dealloc(tcol, Cfg::kCols);
        return;
    }
    uint32_t n_s = 0, n_o = 0;   // products of scores and of values waited for

    // ---- a unit's place in the cache. A warp's 32 keys are two runs of 16, each in one
    // page (page sizes are multiples of 16): lane i knows the run of keys 16 (i / 16) ...
    constexpr uint32_t kNone = 0xffffffffu;   // no such keys, or a page that does not exist: they read as zero
    const int run = warp * 32 + (lane & 16);
    auto page_of = [&](int st) {
        const int key = st * kKeys + run;
        return st < st1 && key < it.s.len ? ld_here(p.b.table + (size_t)it.b * p.b.max_pages + (key >> p.b.shift)) : -1;
    };
    auto place = [&](int st, int page) {   // the run's first row (row indexes are below 2^32 - 1)
        const int key = st * kKeys + run;
        if (st >= st1 || key >= it.s.len) return kNone;
        if ((unsigned)page >= (unsigned)p.c.n_pages) {
            set_error(p.ctrl, MOE_ERR_DEVICE);
            return kNone;
        }
        return (((uint32_t)page * (uint32_t)p.c.Hkv + (uint32_t)it.h) << p.b.shift) + (uint32_t)(key & ((1 << p.b.shift) - 1));
    };
    // The warp's rows, 512 bytes at a time. The 16-byte pieces of a row are turned by the
    // row, so that lanes that read a row each meet no bank twice. Rows that do not exist
    // become zeros.
    auto turned = [](int r) { return D == 128 ? r >> 1 & 3 : r >> 2 & 1; };
    const int copy_to = (lane / Cfg::kChunks * Cfg::kChunks + (lane % Cfg::kChunks ^ turned(lane / Cfg::kChunks))) * 16;
    const char *const k_from = reinterpret_cast<const char *>(p.c.k_codes) + lane * 16, *const v_from = reinterpret_cast<const char *>(p.c.v_codes) + lane * 16;
    struct Runs {
        uint32_t a, b;   // first rows of the warp's two runs
    };
    auto runs_of = [&](uint32_t at) { return Runs{__shfl_sync(0xffffffffu, at, 0), __shfl_sync(0xffffffffu, at, 16)}; };
    auto copy = [&](uint8_t *raw, const char *from, Runs runs) {
        const bool is_a = runs.a != kNone, is_b = runs.b != kNone;
        const char *fa = from + (size_t)(is_a ? runs.a : 0) * (D / 2), *fb = from + (size_t)(is_b ? runs.b : 0) * (D / 2);
#pragma unroll
        for (int k = 0; k < D / 64; ++k) {
            copy16(raw + copy_to + k * 512, fa + k * 512, is_a);
            copy16(raw + copy_to + 8 * D + k * 512, fb + k * 512, is_b);
        }
    };
    // the scales: a run's are 32 bytes; lanes 0-1 and 16-17 copy K's, 2-3 and 18-19 V's
    const uint16_t *const scales_from = ((lane & 2) ? p.c.v_scales : p.c.k_scales) + (lane & 1) * 8;
    uint16_t *const scales_to = &sh.scales[warp][0][lane >> 1 & 1][(lane & 16) + (lane & 1) * 8];
    auto copy_scales = [&](int slot, uint32_t at) {
        if ((lane & 15) < 4) copy16(scales_to + slot * 64, scales_from + (at != kNone ? at : 0), at != kNone);
    };
    auto row_of = [&](const uint8_t *raw, uint4 (&w)[Cfg::kChunks]) {
#pragma unroll
        for (int i = 0; i < Cfg::kChunks; ++i) w[i] = lds_v4(raw + (lane * Cfg::kChunks + (i ^ turned(lane))) * 16);
    };
    auto write_k = [&]() {   // the pairs (k, k + 4) of a word's codes, a column each
        uint4 w[Cfg::kChunks];
        row_of(k_raw, w);
#pragma unroll
        for (int i = 0; i < Cfg::kChunks; ++i) {
            const uint32_t x[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
            uint32_t v[16];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t x8 = x[j] >> 8;
                v[4 * j] = nib_lo(x[j]);
                v[4 * j + 1] = nib_hi(x[j]);
                v[4 * j + 2] = nib_lo(x8);
                v[4 * j + 3] = nib_hi(x8);
            }
            st_cols<16>(tlane + i * 16, v);
        }
    };
    auto write_v = [&]() {
        uint4 w[Cfg::kChunks];
        row_of(v_raw, w);
#pragma unroll
        for (int i = 0; i < Cfg::kChunks; ++i) {
            const uint32_t x[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int chunk = i * 4 + j;
                const uint32_t x8 = x[j] >> 8;
                *reinterpret_cast<uint4 *>(sV + (chunk >> 3) * 16384 + tid * 128 + (((chunk & 7) ^ (tid & 7)) << 4)) =
                    make_uint4(nib_lo(x[j]), nib_hi(x[j]), nib_lo(x8), nib_hi(x8));
            }
        }
    };
    const uint64_t desc_q = q_desc<R>(sQ), desc_v = v_desc<D>(sV), desc_p = p_desc<R>(sP);
    const uint32_t lead = elect();
    auto issue_scores = [&]() {   // (warp 0)
#pragma unroll
        for (int k = 0; k < D / 16; ++k)   // (32 bytes of Q's rows; 64 values a block)
            mma_ts(lead, tcol + Cfg::kColS, tcol + k * 8, desc_q + (uint64_t)((k >> 2) * (R * 128 / 16) + (k & 3) * 2), idesc(Cfg::kNP, false), k > 0);
        commit(lead, &sh.s_full);
    };
    // The first copies of an item (K and scales of its first unit, and V's, in no group
    // yet) and its queries are begun before what else the item's start or the last one's
    // end has to do.
    int page0 = page_of(st0), page1 = page_of(st0 + 1), rows;
    uint32_t at0 = kNone, at1 = kNone;   // where this unit and the next (whose K is under way) lie
    uint2 q_raw[R / 4];                  // the warp's rows r = warp + 4 i, D / 32 values a lane
    auto begin_item = [&]() {
        rows = min(R, it.s.nq * p.G - it.qt * R);
#pragma unroll
        for (int i = 0; i < R / 4; ++i) {
            const int r = warp + 4 * i, rr = it.qt * R + r, qi = rr / p.G;
            q_raw[i] = make_uint2(0, 0);
            if (r < rows) {
                const uint16_t *src = p.q + (size_t)(it.s.q0 + qi) * p.qs.token + (size_t)(it.h * p.G + rr - qi * p.G) * p.qs.head + lane * (D / 32);
                if (D == 128) q_raw[i] = *reinterpret_cast<const uint2 *>(src);
                else q_raw[i].x = *reinterpret_cast<const uint32_t *>(src);
            }
        }
        at0 = place(st0, page0);
        copy(k_raw, k_from, runs_of(at0));
        copy_scales(0, at0);
        copies_commit();
        copy(v_raw, v_from, runs_of(at0));
    };
    begin_item();

    for (;;) {
        // ---- the rows' queries as operands, and what each row sees
#pragma unroll
        for (int i = 0; i < R / 4; ++i) {
            const int r = warp + 4 * i, qi = (it.qt * R + r) / p.G;
            const uint32_t v[2] = {q_raw[i].x, q_raw[i].y};
            float x[D / 32];
            uint32_t big = 0;
#pragma unroll
            for (int j = 0; j < D / 32; j += 2) {
                x[j] = __uint_as_float(v[j / 2] << 16);
                x[j + 1] = __uint_as_float(v[j / 2] & 0xffff0000u);
                big = max(big, max(v[j / 2] & 0x7FFFu, (v[j / 2] >> 16) & 0x7FFFu));
            }
            big = __reduce_max_sync(0xffffffffu, big);
            const int e = norm_exponent(big);
            // the largest to [2^8, 2^9), and signed so that the largest product is the largest
            // score (one by one: the factors' product may be infinite)
            const float f = pow2_biased(254 - e), up = p.scale < 0.f ? -256.f : 256.f;
#pragma unroll
            for (int j = 0; j < D / 32; ++j) {
                // values 0, 4, 1, 5, 2, 6, 3, 7 of eight side by side, as K's
                const int d = lane * (D / 32) + j, at = (d & 56) + (d & 3) * 2 + (d >> 2 & 1);   // of a block of 64
                *reinterpret_cast<__half *>(sQ + (d >> 6) * (R * 128) + r * 128 + (((at >> 3) ^ (r & 7)) << 4) + (at & 7) * 2) = __float2half_rn(x[j] * f * up);
            }
            if (lane == 0) {
                const float cc = fabsf(p.scale) * kLog2e * pow2_biased(e) * (1.f / 256.f);
                sh.c[r] = big < 0x7F80u ? cc : __uint_as_float(0x7fc00000u);   // a query that is not finite: NaN
                sh.lim[r] = r < rows ? it.s.len - it.s.nq + qi + 1 : 0;
            }
        }
        fence_proxy_async_smem();
        __syncthreads();
        if (tid < R) sh.m[tid] = 0.f;   // (the first unit sets it)
        // every row sees the keys below `least`
        const int least = max(it.s.len - it.s.nq + it.qt * R / p.G + 1, 0);

        float l[R];
#pragma unroll
        for (int r = 0; r < R; ++r) l[r] = 0.f;
        int st = st0, slot = 0;   // slot: of this unit's scales
        bool fail = false;        // a wait gave up
        copies_wait<0>();   // (K; V belongs to the next group)
        __syncwarp();
        {
            const float fv = at0 != kNone && st * kKeys + tid < it.s.len ? fabsf(bf16_bits_to_f32(sh.scales[warp][0][1][lane])) : 0.f;
            const uint32_t e = fv > 0.f && fv < INFINITY ? max(__float_as_uint(fv) >> 23, 1u) : 0u, top = __reduce_max_sync(0xffffffffu, e);
            if (lane == 0) sh.we[warp] = (int)top;
        }
        write_k();
        __syncwarp();
        at1 = place(st + 1, page1);
        page1 = page_of(st + 2);
        Runs runs = runs_of(at1);   // of the next unit
        copy(k_raw, k_from, runs);
        copy_scales(1, at1);
        copies_commit();
        copies_commit();   // (in each turn K's group is the last but one where it is waited for)
        tc::wait_st();
        tc::fence_before();
        __syncthreads();
        tc::fence_after();
        if (warp == 0) issue_scores();
        // the biased exponent taken off all V scales, of the largest of the first unit (a middle for
        // their range, nothing more)
        const int we = max(max(sh.we[0], sh.we[1]), max(sh.we[2], sh.we[3])), F = we == 0 ? 127 : min(we, 253);
        for (uint32_t turn = 0; st < st1; ++st, ++turn) {
            const bool more = st + 1 < st1;
            // ---- the key's scores, less the maxima in use. Scales: a row that was not finite
            // makes its scores NaN, its values zero
            const int key = st * kKeys + tid;
            const bool there = at0 != kNone && key < it.s.len;
            float fk = there ? bf16_bits_to_f32(sh.scales[warp][slot][0][lane]) : 0.f;
            float fv = there ? bf16_bits_to_f32(sh.scales[warp][slot][1][lane]) : 0.f;
            if (!(fabsf(fk) < INFINITY) || !(fabsf(fv) < INFINITY)) {
                fk = __uint_as_float(0x7fc00000u);
                fv = 0.f;
            }
            fail |= !wait(&sh.s_full, n_s & 1);
            ++n_s;
            tc::fence_after();
            float s[R];
            {
                ld_cols<R>(tlane + Cfg::kColS, s);
#pragma unroll
                for (int r = 0; r < R; r += 4) {
                    const float4 cs = *reinterpret_cast<const float4 *>(sh.c + r), m = *reinterpret_cast<const float4 *>(sh.m + r);
                    float *x = s + r;
                    mul2(x[0], x[1], fk, fk);
                    mul2(x[2], x[3], fk, fk);
                    fma2(x[0], x[1], cs.x, cs.y, -m.x, -m.y);
                    fma2(x[2], x[3], cs.z, cs.w, -m.z, -m.w);
                }
            }
            // ---- the next unit's K, whose product runs beside what follows
            slot = slot == 2 ? 0 : slot + 1;
            at0 = at1;
            Runs runs_next{kNone, kNone};
            if (more) {
                copies_wait<1>();
                __syncwarp();
                write_k();
                __syncwarp();
                at1 = place(st + 2, page1);
                page1 = page_of(st + 3);
                runs_next = runs_of(at1);
                copy(k_raw, k_from, runs_next);
                copy_scales(slot == 2 ? 0 : slot + 1, at1);
                tc::wait_st();
                tc::fence_before();
                bar_pass(warp);
                if (warp == 0) {
                    tc::fence_after();
                    issue_scores();
                }
            }
            copies_commit();
            if ((st + 1) * kKeys > least) {
#pragma unroll
                for (int r = 0; r < R; ++r)
                    if (key >= sh.lim[r]) s[r] = -INFINITY;
            }
            // ---- probabilities; where one times its V scale would pass 2^15, or itself 2^96, the warp
            // leaves them until the rows' exponents have followed (and in the first unit, which sets them)
            const float f = fminf(fmaxf(fv * pow2_biased(254 - F), -0x1p120f), 0x1p120f), log_f = log2_approx(fabsf(f));
            float top = s[0];
#pragma unroll
            for (int r = 1; r < R; ++r) top = fmaxf(top, s[r]);
            const bool over = __any_sync(0xffffffffu, turn == 0 || top > fminf(15.f - log_f, 96.f));
            const uint32_t p_at = Cfg::kPs == 2 ? (turn & 1) * Cfg::kP : 0;
            auto values_added = [&]() {   // the last unit's values are in the sums, and V and P free
                if (turn > 0) {
                    fail |= !wait(&sh.o_full, n_o & 1);
                    ++n_o;
                }
            };
            auto write_p = [&](bool sum) {
#pragma unroll
                for (int r = 0; r < R; r += 8) {
                    uint32_t h[4];
#pragma unroll
                    for (int j = 0; j < 8; j += 2) {
                        float a = exp2_approx(s[r + j]), b = exp2_approx(s[r + j + 1]);
                        if (sum) add2(l[r + j], l[r + j + 1], a, b);
                        mul2(a, b, f, f);
                        h[j >> 1] = half2_of(a, b);
                    }
                    *reinterpret_cast<uint4 *>(sP + p_at + tid * 16 + (r >> 3) * 2048) = make_uint4(h[0], h[1], h[2], h[3]);
                }
            };
            if (Cfg::kPs == 1) values_added();
            if (!over) write_p(true);
            // ---- the unit's V
            if (Cfg::kPs == 2) values_added();
            copies_wait<1>();
            __syncwarp();
            write_v();
            __syncwarp();
            if (more) copy(v_raw, v_from, runs);
            runs = runs_next;
            copies_commit();
            fence_proxy_async_smem();
            tc::fence_before();
            if (bar_or(over || fail)) {
                tc::fence_after();
                if (bar_or(fail)) break;   // a wait gave up: for all warps at once
                // ---- all follow: the rows' exponents, then the sums
                {
                    float t[R];
                    const float by = fmaxf(log_f - 6.f, -90.f);
#pragma unroll
                    for (int r = 0; r < R; ++r) t[r] = s[r] + by;
                    reduce_rows<R, true>(t, sh.wm[warp]);
                }
                __syncthreads();
                float up[R];   // how far each row's exponent rises, then 2 to half of less that (all of it may be
                               // below fp32's range where the sum of probabilities is far above it)
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const float x = fmaxf(fmaxf(sh.wm[0][r], sh.wm[1][r]), fmaxf(sh.wm[2][r], sh.wm[3][r]));
                    // (a row that sees no key of the first unit sees none of the later ones)
                    up[r] = turn > 0 ? fmaxf(x, 0.f) : x == kNoMax ? 0.f : x;
                    if (tid == r) sh.m[r] += up[r];   // (all have read the old ones before the barriers)
                    s[r] -= up[r];
                    // (turn 0: nothing to rescale, and one far below zero has no power of two)
                    up[r] = turn > 0 ? exp2_approx(-0.5f * up[r]) : 1.f;
                    l[r] = l[r] * up[r] * up[r];
                }
                if (turn > 0) {
                    float o[R];
                    ld_cols<R>(tlane + Cfg::kColO, o);
                    uint32_t w[R];
#pragma unroll
                    for (int r = 0; r < R; ++r) w[r] = __float_as_uint(o[r] * up[r] * up[r]);
                    st_cols<R>(tlane + Cfg::kColO, w);
                    tc::wait_st();
                }
                if (over) write_p(true);
                else write_p(false);   // (its sums hold them already)
                fence_proxy_async_smem();
                tc::fence_before();
                __syncthreads();
            }
            tc::fence_after();
            if (warp == 1) {
#pragma unroll
                for (int k = 0; k < kKeys / 16; ++k)
                    mma_ss(lead, tcol + Cfg::kColO, desc_v + (uint64_t)(k * 128), desc_p + (uint64_t)(p_at / 16 + k * 16), idesc(Cfg::kNP, true),
                           turn > 0 || k > 0);
                commit(lead, &sh.o_full);
            }
        }
        copies_wait<0>();
        if (st < st1) {   // (cut short; the products in flight get a bounded wait)
            wait(&sh.o_full, n_o & 1);
            if (tid == 0) {
                set_error(p.ctrl, MOE_ERR_TIMEOUT);
                p.begun[c].last = 0;
            }
            break;
        }

        // ---- the next item's first copies, then this one's rows
        const Item done = it;
        const bool first_part = st0 == 0, whole = first_part && st1 == it.units;
        bool last_item = it.first + it.span >= u_end;
        if (!last_item) {
            next_item<kKeys, kLead<D>>(p, R, it);
            last_item = u_end - it.first <= kLead<D>;
        }
        if (!last_item) {
            st0 = 0;
            st1 = min(it.units, u_end - it.first - kLead<D>);
            page0 = page_of(0);
            page1 = page_of(1);
        }
        reduce_rows<R, false>(l, sh.wm[warp]);
        fail = !wait(&sh.o_full, n_o & 1);
        ++n_o;
        tc::fence_after();
        float o[R];
        ld_cols<R>(tlane + Cfg::kColO, o);
        const int rows_done = rows;
        if (!last_item) begin_item();
        tc::fence_before();
        if (bar_or(fail)) {
            if (tid == 0) {
                set_error(p.ctrl, MOE_ERR_TIMEOUT);
                p.begun[c].last = 0;
            }
            break;
        }
        // lane x holds place x of the values' order 0, 4, 1, 5, 2, 6, 3, 7
        const int d = (tid & ~7) + ((tid & 7) >> 1) + (tid & 1) * 4;
        float *part = p.part + (size_t)(c * 2 + first_part) * part_floats(R, D);
        const float up = pow2_biased(F);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (r >= rows_done) break;
            const float sum = (sh.wm[0][r] + sh.wm[1][r]) + (sh.wm[2][r] + sh.wm[3][r]);
            if (whole) {
                const int rr = done.qt * R + r, i = rr / p.G, head = done.h * p.G + rr - i * p.G;
                const size_t tok = (size_t)(done.s.q0 + i);
                const float inv = sum == 0.f ? 0.f : 1.f / sum;   // (no key: zero)
                const __nv_bfloat16 x = __float2bfloat16_rn(o[r] * inv * up);
                if (tid < D) p.out[tok * p.os.token + (size_t)head * p.os.head + d] = *reinterpret_cast<const uint16_t *>(&x);
                if (tid == r && p.lse) p.lse[tok * p.Hq + head] = sum == 0.f ? -INFINITY : (sh.m[r] + log2f(sum)) * kLn2;
            } else {
                if (tid < D) part[2 * R + 4 + r * D + d] = o[r];
                if (tid == r) {
                    part[r] = sum == 0.f ? kNoMax : sh.m[r];   // (nothing seen)
                    part[R + r] = sum;
                }
            }
        }
        if (tid == 0) {
            if (!whole) part[2 * R] = __int_as_float(F);
            if (last_item)
                p.begun[c] = Begun{first_part && !whole ? shares.holder(done.first + done.span - 1) : 0, done.s.q0, done.h, done.qt, rows_done, {0, 0, 0}};
        }
        if (last_item) break;
    }
    copies_wait<0>();
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    if (warp == 0) tc::dealloc(sh.tmem, Cfg::kCols);
}

template <int D, int R>
cudaError_t launch_one(const Attn &p, int *rows_at, int *grid_out, cudaStream_t s) {
    using Cfg = DecodeCfg<D, R>;
    constexpr size_t kBytes = Cfg::kSmem + sizeof(DecodeShared<R>);
    static_assert((kBytes + 1024) * Cfg::kPerSm <= 233472, "shared memory");
    const cudaError_t err = set_smem_once(reinterpret_cast<const void *>(kv4_decode_kernel<D, R>), (int)kBytes);
    if (err != cudaSuccess) return err;
    int grid = Cfg::kPerSm * sm_count();
    if (grid > kMaxCtas) grid = kMaxCtas;
    *rows_at = R;
    *grid_out = grid;
    return launch_pdl(kv4_decode_kernel<D, R>, dim3((unsigned)grid), Cfg::kThreads, kBytes, s, p);
}

}  // namespace

cudaError_t launch_kv4_decode(const kv4::Attn &p, int rows, int *rows_at, int *grid, cudaStream_t s) {
    auto pick = [&](auto d) {
        constexpr int D = decltype(d)::value;
        return rows <= 8 ? launch_one<D, 8>(p, rows_at, grid, s) : rows <= 16 ? launch_one<D, 16>(p, rows_at, grid, s) : launch_one<D, 32>(p, rows_at, grid, s);
    };
    return p.c.D == 64 ? pick(std::integral_constant<int, 64>{}) : pick(std::integral_constant<int, 128>{});
}

}  // namespace moe
