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
// (Loads into registers measured 90-125 us where this takes XX: the waits for them
// are counted on few scoreboards, so that a shuffle or a shared load behind them
// waited for them too; and a row a lane from global memory visits each cache line
// four times, which had the L1 74% busy.) A warp-level form (mma.sync on fragments
// loaded from global memory) took 770 warp instructions for 32 keys at R = 8, for
// shuffles of scales and maxima, address arithmetic and a transposition of P.
//
// K enters as e4m3: a code n = q + 8 in the low bits of an e4m3 byte is n 2^-9
// exactly, on both sides of its smallest normal, so two ANDs and a shift make
// operands of 8 codes. A query row enters as the sum of two e4m3 numbers (two
// columns of the product), less its own exponent: 8 bits, all that a bf16 has,
// but for values below 2^-9 of the row's largest, which are rounded at 2^-18 of
// it. The 8 that each code has too many is taken off in fp32: -8 sum q.
// V enters as fp16, exactly. A V scale multiplies its key's probabilities just
// before they are rounded to fp16, less the exponent F of the largest V scale so
// far (a power of two, put back at the end), so that no range of scales is lost.
#include <cuda_fp8.h>

#include "kv4_attention.cuh"
#include "tcgen05.cuh"

namespace moe {

namespace {

using namespace kv4;

constexpr int kKeys = 128;   // keys of a unit: a warpgroup's turn
constexpr uint32_t kNibs = 0x0F0F0F0Fu;

template <int D, int R>
struct DecodeCfg {
    static constexpr int kGroups = 2;                     // warpgroups a CTA
    static constexpr int kPerSm = R < 32 ? 2 : 1;         // CTAs an SM: 128 registers a thread, or 255 for the most rows
    static constexpr int kThreads = kGroups * 128;
    static constexpr int kStride = D + 4;                 // of a row of partial values in shared memory
    static constexpr int kNS = 2 * R, kNP = R < 16 ? 16 : R;   // columns of S^T (two a row) and of O^T (R = 8: twice the same)
    static constexpr int kV = 128 * D * 2, kP = R * 256;  // bytes of a warpgroup's operands
    static constexpr int kPs = R == 16 ? 1 : 2;           // of P: two where they fit, one read while the next is written
    static constexpr int kQ = kNS * 128;
    static constexpr int kWarpRaw = 32 * D / 2, kRaw = 4 * kWarpRaw;   // a warp's codes of 32 keys (K or V), a warpgroup's
    // tensor memory of a warpgroup: K's row, scores, values' sums
    static constexpr int kColS = 32, kColO = kColS + kNS, kCols = R < 16 ? 64 : 128;
    static_assert(kColO + kNP <= kCols, "tensor memory");
    static constexpr int kGroup = kV + kPs * kP + 2 * kRaw, kSmem = kQ + kGroups * kGroup;
    static constexpr int kChunks = D / 32;                // 16-byte pieces of a row of codes
    static_assert(R * kStride * 4 <= kV, "the rows' parts lie where V was");
};

struct Bars {
    uint64_t s_full[2], o_full[2];   // of each warpgroup: scores formed, values added
};

template <int W, int R>
struct DecodeShared {
    alignas(16) float c[R], base[R], m[W][R], l[W][R], wm[W][4][R];
    alignas(16) uint16_t scales[W * 4][3][2][32];   // of a warp's units in turn: K's, V's
    Bars bars;
    long long sums[W * 4];
    int lim[R], F[W], we[W][4], fail[W], last;
    uint32_t tmem;
};

__device__ inline bool wait(uint64_t *bar, uint32_t parity) {
    bool ok = false;
    for (uint32_t i = 0; i < kSpinLimit && !ok; ++i) ok = mbar_try_wait(bar, parity);
    return __all_sync(0xffffffffu, ok);
}

// Named barrier of a warpgroup, and the same returning the OR of v.
__device__ inline void bar_sync(int id) { asm volatile("bar.sync %0, 128;" ::"r"(id) : "memory"); }
__device__ inline bool bar_or(int id, bool v) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, %2, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)v), "r"(id)
        : "memory");
    return r != 0;
}

__device__ inline bool elect() {
    uint32_t pred;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(pred));
    return pred != 0;
}

// kind::f8f6f4 (e4m3 both), A from tensor memory.
__device__ inline void mma_e4m3(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ inline uint32_t idesc(int N, bool mn_major) {   // f32 sums; format 0 is f16 or e4m3, by the kind
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

__device__ inline uint32_t e4m3_of(float x) { return __nv_cvt_float_to_fp8(x, __NV_SATFINITE, __NV_E4M3); }
__device__ inline float of_e4m3(uint32_t b) { return __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)b, __NV_E4M3))); }

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

// 16 bytes of the cache into shared memory, asynchronously.
__device__ inline void copy16(void *dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ inline void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All of the thread's copies but those of the last N groups have arrived.
template <int N>
__device__ inline void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

template <int D, int R>
__global__ void __launch_bounds__(DecodeCfg<D, R>::kThreads, DecodeCfg<D, R>::kPerSm) kv4_decode_kernel(Attn p) {
    using Cfg = DecodeCfg<D, R>;
    constexpr int W = Cfg::kGroups;
    extern __shared__ __align__(1024) uint8_t s_dyn[];
    uint8_t *const sQ = s_dyn, *const s_groups = sQ + Cfg::kQ;
    // the sequences' prefix: needed only before the first operand is written
    int *const s_pre = reinterpret_cast<int *>(s_groups);
    static_assert(sizeof(int) * 4097 <= (size_t)W * Cfg::kGroup, "prefix");
    DecodeShared<W, R> &sh = *reinterpret_cast<DecodeShared<W, R> *>(s_groups + W * Cfg::kGroup);
    Bars &bars = sh.bars;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, wg = warp >> 2, tid = threadIdx.x & 127;
    const int bar = 1 + wg;   // the warpgroup's barrier

    if (threadIdx.x == 0) {
        for (int i = 0; i < W; ++i) {
            mbar_init(&bars.s_full[i], 1);
            mbar_init(&bars.o_full[i], 1);
            sh.fail[i] = 0;
        }
        fence_mbar_init();
    }
    uint8_t *const sV = s_groups + wg * Cfg::kGroup, *const sP = sV + Cfg::kV;
    uint8_t *const k_raw = sP + Cfg::kPs * Cfg::kP + (warp & 3) * Cfg::kWarpRaw, *const v_raw = k_raw + Cfg::kRaw;
    pdl_wait();
    pdl_launch_dependents();
    const int U = scan_units<Cfg::kThreads, kKeys>(p, R, s_pre, sh.sums);
    // fewer CTAs where there is less than a unit for each warpgroup of them
    const Shares shares(U, min((int)gridDim.x, max(1, (U + W - 1) / W)));
    const int c = blockIdx.x;
    if (c >= shares.C || U == 0) return;
    int u = shares.begin(c);
    const int u_end = shares.begin(c + 1);
    if (warp == 0) {
        tc::alloc(&sh.tmem, W * Cfg::kCols);
        tc::relinquish();
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tcol = sh.tmem + wg * Cfg::kCols, tlane = tcol + ((uint32_t)((warp & 3) * 32) << 16);
    uint32_t n_s = 0, n_o = 0;   // products of scores and of values waited for

    // ---- a unit's place in the cache. A warp's 32 keys are two runs of 16, each in one
    // page (page sizes are multiples of 16): lane i knows the run of keys 16 (i / 16) ...
    constexpr uint32_t kNone = 0xffffffffu;   // no such keys, or a page that does not exist: they read as zero
    Item it = find_item<kKeys>(p, R, s_pre, u);
    int st0 = u - it.first, st1 = min(it.units, u_end - it.first);   // the units of the item in this CTA's share
    const int run = (warp & 3) * 32 + (lane & 16);
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
    // keep what was there (codes are finite whatever they are).
    auto turned = [](int r) { return D == 128 ? r >> 1 & 3 : r >> 2 & 1; };
    const int copy_to = (lane / Cfg::kChunks * Cfg::kChunks + (lane % Cfg::kChunks ^ turned(lane / Cfg::kChunks))) * 16;
    auto copy = [&](uint8_t *raw, const int32_t *codes, uint32_t at) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t src = __shfl_sync(0xffffffffu, at, 16 * i);
            if (src != kNone) {
                const char *from = reinterpret_cast<const char *>(codes) + (size_t)src * (D / 2) + lane * 16;
                uint8_t *to = raw + i * (8 * D) + copy_to;
#pragma unroll
                for (int k = 0; k < D / 64; ++k) copy16(to + k * 512, from + k * 512);
            }
        }
    };
    // the scales: a run's are 32 bytes; lanes 0-1 and 16-17 copy K's, 2-3 and 18-19 V's
    auto copy_scales = [&](int slot, uint32_t at) {
        if ((lane & 15) < 4 && at != kNone)
            copy16(&sh.scales[warp][slot][lane >> 1 & 1][(lane & 16) + (lane & 1) * 8],
                   ((lane & 2) ? p.c.v_scales : p.c.k_scales) + at + (lane & 1) * 8);
    };
    auto row_of = [&](const uint8_t *raw, uint4 (&w)[Cfg::kChunks]) {
#pragma unroll
        for (int i = 0; i < Cfg::kChunks; ++i) w[i] = lds_v4(raw + (lane * Cfg::kChunks + (i ^ turned(lane))) * 16);
    };
    auto write_k = [&]() {   // codes 0, 2, 4, 6 of a word are one column, 1, 3, 5, 7 the next
        uint4 w[Cfg::kChunks];
        row_of(k_raw, w);
#pragma unroll
        for (int i = 0; i < Cfg::kChunks; ++i) {
            const uint32_t v[8] = {w[i].x & kNibs, w[i].x >> 4 & kNibs, w[i].y & kNibs, w[i].y >> 4 & kNibs,
                                   w[i].z & kNibs, w[i].z >> 4 & kNibs, w[i].w & kNibs, w[i].w >> 4 & kNibs};
            st_cols<8>(tlane + i * 8, v);
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
    auto issue_scores = [&]() {
        if ((warp & 3) == 0 && elect()) {
#pragma unroll
            for (int k = 0; k < D / 32; ++k)
                mma_e4m3(tcol + Cfg::kColS, tcol + k * 8, tc::sdesc_sw128(sQ) + (uint64_t)(k * 2), idesc(Cfg::kNS, false), k > 0);
            tc::commit(&bars.s_full[wg]);
        }
        __syncwarp();
    };
    // The first copies of an item: K and scales of the warpgroup's first unit, and V's (in
    // no group yet). They are begun before what else the item's start or the last one's
    // end has to do.
    int page0 = page_of(st0 + wg), page1 = page_of(st0 + wg + W);
    uint32_t at0 = kNone;   // the runs of this unit, of the next (whose K is under way)
    auto begin_copies = [&]() {
        at0 = place(st0 + wg, page0);
        copy(k_raw, p.c.k_codes, at0);
        copy_scales(0, at0);
        copies_commit();
        copy(v_raw, p.c.v_codes, at0);
    };
    begin_copies();

    for (;;) {
        const int rows = min(R, it.s.nq * p.G - it.qt * R);

        // ---- the rows' queries as operands, and what each row sees
        for (int r = warp; r < R; r += 4 * W) {
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
            big = __reduce_max_sync(0xffffffffu, big);
            const int e = norm_exponent(big);
            // to [2^7, 2^8), 448 being the largest e4m3, and signed so that the largest
            // product is the largest score (one by one: the factors' product may be infinite)
            const float f = pow2_biased(254 - e), up = p.scale < 0.f ? -128.f : 128.f;
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < D / 32; ++j) {
                // codes 0, 2, 4, 6 of a word are one column of K's row, 1, 3, 5, 7 the next
                const int d = lane * (D / 32) + j, at = (d & ~7) + (d & 1) * 4 + ((d & 7) >> 1);
                const float y = x[j] * f * up;
                const uint32_t q1 = e4m3_of(y), q2 = e4m3_of(y - of_e4m3(q1));
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int n = k * R + r;
                    sQ[(n >> 3) * 1024 + (n & 7) * 128 + (((at >> 4) ^ (n & 7)) << 4) + (at & 15)] = (uint8_t)(k ? q2 : q1);
                }
                sum += of_e4m3(q1) + of_e4m3(q2);
            }
#pragma unroll
            for (int j = 16; j > 0; j >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, j);
            if (lane == 0) {
                // 2^9 of the codes less the 2^7 of the queries
                const float cc = fmaxf(fabsf(p.scale) * kLog2e * pow2_biased(e) * 4.f, 1e-37f);
                sh.c[r] = big < 0x7F80u ? cc : __uint_as_float(0x7fc00000u);   // a query that is not finite: NaN
                sh.base[r] = sum * (-8.f / 512.f);
                sh.lim[r] = r < rows ? it.s.len - it.s.nq + i + 1 : 0;
            }
        }
        if (tid < R) sh.m[wg][tid] = 0.f;   // (the first unit sets it)
        fence_proxy_async_smem();
        __syncthreads();
        // every row sees the keys below `least`
        const int least = max(it.s.len - it.s.nq + it.qt * R / p.G + 1, 0);

        float l[R];
#pragma unroll
        for (int r = 0; r < R; ++r) l[r] = 0.f;
        int F = 1;            // biased exponent taken off the V scales
        float v_top = 0.f;    // 2^(F - 126): they stay below it (0: the first unit takes the branch that sets both)
        int st = st0 + wg, slot = 0;   // slot: of this unit's scales
        const bool any = st < st1;     // (uniform in a warpgroup)
        uint32_t at1 = kNone;
        bool cut = false;     // a wait gave up
        if (any) {
            copies_wait<0>();   // (K; V belongs to the next group)
            __syncwarp();
            write_k();
            __syncwarp();
            at1 = place(st + W, page1);
            page1 = page_of(st + 2 * W);
            copy(k_raw, p.c.k_codes, at1);
            copy_scales(1, at1);
            copies_commit();
            copies_commit();   // (in each turn K's group is the last but one where it is waited for)
            tc::wait_st();
            tc::fence_before();
            bar_sync(bar);
            tc::fence_after();
            issue_scores();
        }
        for (uint32_t turn = 0; st < st1; st += W, ++turn) {
            const bool more = st + W < st1;
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
            bool fail = !wait(&bars.s_full[wg], n_s & 1);
            ++n_s;
            tc::fence_after();
            float s[R];
            {
                float s2[2 * R];
                ld_cols<2 * R>(tlane + Cfg::kColS, s2);
#pragma unroll
                for (int r = 0; r < R; r += 4) {
                    const float4 base = *reinterpret_cast<const float4 *>(sh.base + r), cs = *reinterpret_cast<const float4 *>(sh.c + r),
                                 m = *reinterpret_cast<const float4 *>(sh.m[wg] + r);
                    float *x = s2 + r, *y = s2 + R + r;
                    add2(x[0], x[1], y[0], y[1]);
                    add2(x[2], x[3], y[2], y[3]);
                    add2(x[0], x[1], base.x, base.y);
                    add2(x[2], x[3], base.z, base.w);
                    mul2(x[0], x[1], fk, fk);
                    mul2(x[2], x[3], fk, fk);
                    fma2(x[0], x[1], cs.x, cs.y, -m.x, -m.y);
                    fma2(x[2], x[3], cs.z, cs.w, -m.z, -m.w);
#pragma unroll
                    for (int j = 0; j < 4; ++j) s[r + j] = x[j];
                }
            }
            // ---- the next unit's K, whose product runs beside what follows
            slot = slot == 2 ? 0 : slot + 1;
            at0 = at1;
            if (more) {
                copies_wait<1>();
                __syncwarp();
                write_k();
                __syncwarp();
                at1 = place(st + 2 * W, page1);
                page1 = page_of(st + 3 * W);
                copy(k_raw, p.c.k_codes, at1);
                copy_scales(slot == 2 ? 0 : slot + 1, at1);
            }
            copies_commit();
            if ((st + 1) * kKeys > least) {
#pragma unroll
                for (int r = 0; r < R; ++r)
                    if (key >= sh.lim[r]) s[r] = -INFINITY;
            }
            bool over = fabsf(fv) >= v_top;
#pragma unroll
            for (int r = 0; r < R; ++r) over |= s[r] > 8.f;
            tc::wait_st();
            tc::fence_before();
            const bool move = bar_or(bar, over);
            tc::fence_after();
            if (more) issue_scores();
            bool added = turn == 0;   // the last unit's values are in the sums
            if (move) {
                // ---- a score passed the maximum in use by 2^8, or a V scale its exponent: all follow
                reduce_rows<R, true>(s, sh.wm[wg][warp & 3]);
                const uint32_t e = __reduce_max_sync(0xffffffffu, __float_as_uint(fv) >> 23 & 0xFFu);
                if (lane == 0) sh.we[wg][warp & 3] = (int)e;
                bar_sync(bar);
                int Fn = F;
#pragma unroll
                for (int i = 0; i < 4; ++i) Fn = max(Fn, min(sh.we[wg][i], 253));
                const float fo = Fn - F > 126 ? 0.f : pow2_biased(127 + F - Fn);
                F = Fn;
                v_top = F == 253 ? INFINITY : pow2_biased(F + 1);
                float up[R];   // how far each row's maximum rises, then 2 to less that
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const float x = fmaxf(fmaxf(sh.wm[wg][0][r], sh.wm[wg][1][r]), fmaxf(sh.wm[wg][2][r], sh.wm[wg][3][r]));
                    // (a row that sees no key of the first unit sees none of the later ones)
                    up[r] = turn > 0 ? fmaxf(x, 0.f) : x == kNoMax ? 0.f : x;
                    if (tid == r) sh.m[wg][r] += up[r];   // (all have read the old maxima before the first barrier)
                    s[r] -= up[r];
                    up[r] = exp2_approx(-up[r]);
                    l[r] *= up[r];
                }
                if (turn > 0) {
                    fail |= !wait(&bars.o_full[wg], n_o & 1);
                    ++n_o;
                    added = true;
                    tc::fence_after();
                    float o[R];
                    ld_cols<R>(tlane + Cfg::kColO, o);
                    uint32_t w[R];
#pragma unroll
                    for (int r = 0; r < R; ++r) w[r] = __float_as_uint(o[r] * (up[r] * fo));
                    st_cols<R>(tlane + Cfg::kColO, w);
                    tc::wait_st();
                }
            }
            // ---- probabilities
            fv *= pow2_biased(254 - F);
            uint8_t *const sPn = sP + (Cfg::kPs == 2 ? (turn & 1) * Cfg::kP : 0);
            auto values_added = [&]() {   // the last unit's values are in the sums, and V and P free
                if (!added) {
                    fail |= !wait(&bars.o_full[wg], n_o & 1);
                    ++n_o;
                }
            };
            if (Cfg::kPs == 1) values_added();
#pragma unroll
            for (int r = 0; r < R; r += 8) {
                uint32_t h[4];
#pragma unroll
                for (int j = 0; j < 8; j += 2) {
                    float a = exp2_approx(s[r + j]), b = exp2_approx(s[r + j + 1]);
                    add2(l[r + j], l[r + j + 1], a, b);
                    mul2(a, b, fv, fv);
                    h[j >> 1] = half2_of(a, b);
                }
                *reinterpret_cast<uint4 *>(sPn + (r >> 3) * 2048 + tid * 16) = make_uint4(h[0], h[1], h[2], h[3]);
            }
            // ---- the unit's V
            if (Cfg::kPs == 2) values_added();
            copies_wait<1>();
            __syncwarp();
            write_v();
            __syncwarp();
            if (more) copy(v_raw, p.c.v_codes, at0);
            copies_commit();
            fence_proxy_async_smem();
            tc::fence_before();
            // a wait that gave up ends the warpgroup's turns here, for all its warps at once
            if (bar_or(bar, fail)) {
                sh.fail[wg] = 1;
                cut = true;
                break;
            }
            tc::fence_after();
            if ((warp & 3) == 0 && elect()) {
#pragma unroll
                for (int k = 0; k < kKeys / 16; ++k)
                    tc::mma_ss(tcol + Cfg::kColO, v_desc<D>(sV) + (uint64_t)(k * 128), p_desc<R>(sPn) + (uint64_t)(k * 16),
                               idesc(Cfg::kNP, true), turn > 0 || k > 0);
                tc::commit(&bars.o_full[wg]);
            }
            __syncwarp();
        }

        // ---- the next item's pages
        const Item done = it;
        const bool whole = st0 == 0 && st1 == it.units, first_part = st0 == 0;
        u = it.first + st1;
        const bool last_item = u >= u_end;
        if (!last_item) {
            next_item<kKeys>(p, R, it);
            st0 = 0;
            st1 = min(it.units, u_end - u);
            page0 = page_of(wg);
            page1 = page_of(wg + W);
        }
        // ---- the warpgroups' rows, side by side in shared memory (where V was)
        if (any && !cut) {
            if (!wait(&bars.o_full[wg], n_o & 1)) sh.fail[wg] = 1;
            ++n_o;
            tc::fence_after();
        }
        float *const s_o = reinterpret_cast<float *>(sV);
        {
            float o[R];
            if (any) ld_cols<R>(tlane + Cfg::kColO, o);
            else
#pragma unroll
                for (int r = 0; r < R; ++r) o[r] = 0.f;
            // lane x holds place x of the values' order 0, 4, 1, 5, 2, 6, 3, 7
            const int d = (tid & ~7) + ((tid & 7) >> 1) + (tid & 1) * 4;
            if (tid < D)
#pragma unroll
                for (int r = 0; r < R; ++r) s_o[r * Cfg::kStride + d] = o[r];
        }
        reduce_rows<R, false>(l, sh.wm[wg][warp & 3]);
        if (tid == 0) sh.F[wg] = F;
        copies_wait<0>();
        if (!last_item) begin_copies();
        tc::fence_before();
        __syncthreads();
        tc::fence_after();
        bool failed = false;
#pragma unroll
        for (int w = 0; w < W; ++w) failed |= sh.fail[w] != 0;
        if (failed) {
            if (threadIdx.x == 0) set_error(p.ctrl, MOE_ERR_TIMEOUT);
            break;
        }
        if (tid < R) {
            const float sum = (sh.wm[wg][0][tid] + sh.wm[wg][1][tid]) + (sh.wm[wg][2][tid] + sh.wm[wg][3][tid]);
            sh.l[wg][tid] = sum;
            if (sum == 0.f) sh.m[wg][tid] = kNoMax;   // nothing seen
        }
        __syncthreads();
        int Fm = 1;
#pragma unroll
        for (int w = 0; w < W; ++w) Fm = max(Fm, sh.F[w]);
        // a CTA's first part continues an item, its last one may begin one
        float *part = p.part + (size_t)(c * 2 + first_part) * part_floats(R, D);
        for (int x = threadIdx.x; x < rows * (D / 4); x += Cfg::kThreads) {
            const int r = x / (D / 4), d = (x % (D / 4)) * 4;
            float M = kNoMax, L = 0.f;
#pragma unroll
            for (int w = 0; w < W; ++w) M = fmaxf(M, sh.m[w][r]);
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < W; ++w) {
                const float f = exp2_approx(sh.m[w][r] - M);
                L = fmaf(sh.l[w][r], f, L);
                const float fv = Fm - sh.F[w] > 126 ? 0.f : f * pow2_biased(127 + sh.F[w] - Fm);
                const float4 v = *reinterpret_cast<const float4 *>(s_groups + w * Cfg::kGroup + (r * Cfg::kStride + d) * 4);
                acc.x = fmaf(v.x, fv, acc.x);
                acc.y = fmaf(v.y, fv, acc.y);
                acc.z = fmaf(v.z, fv, acc.z);
                acc.w = fmaf(v.w, fv, acc.w);
            }
            if (whole) {
                write_row4(p, done, R, r, d, acc, M, L, Fm);
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
            const int c0 = shares.holder(done.first), c1 = shares.holder(done.first + done.units - 1);
            if (threadIdx.x == 0) {
                __threadfence();
                const uint32_t n = atom_acq_rel_add_u32(p.ticket + c0, 1u);
                sh.last = n == (uint32_t)(c1 - c0);
                if (sh.last) p.ticket[c0] = 0;
            }
            __syncthreads();
            if (sh.last) {
                __threadfence();
                join_parts<Cfg::kThreads, R, D>(p, done, rows, c0, c1);
            }
            __syncthreads();
        }
        if (last_item) break;
    }
    copies_wait<0>();
    // (after a wait that gave up, the products still in flight get another bounded one)
    if (sh.fail[wg]) wait(&bars.o_full[wg], n_o & 1);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    if (warp == 0) tc::dealloc(sh.tmem, W * Cfg::kCols);
}

template <int D, int R>
cudaError_t launch_one(const Attn &p, cudaStream_t s) {
    using Cfg = DecodeCfg<D, R>;
    constexpr size_t kBase = Cfg::kSmem + sizeof(DecodeShared<Cfg::kGroups, R>);
    static_assert(kBase <= (size_t)(Cfg::kPerSm == 2 ? 115712 : 231424), "shared memory");
    const cudaError_t err = set_smem_once(reinterpret_cast<const void *>(kv4_decode_kernel<D, R>), (int)kBase);
    if (err != cudaSuccess) return err;
    int grid = Cfg::kPerSm * sm_count();
    if (grid > kMaxCtas) grid = kMaxCtas;
    return launch_pdl(kv4_decode_kernel<D, R>, dim3((unsigned)grid), Cfg::kThreads, kBase, s, p);
}

}  // namespace

cudaError_t launch_kv4_decode(const kv4::Attn &p, int rows, cudaStream_t s) {
    if (p.c.D == 64) return rows <= 8 ? launch_one<64, 8>(p, s) : rows <= 16 ? launch_one<64, 16>(p, s) : launch_one<64, 32>(p, s);
    return rows <= 8 ? launch_one<128, 8>(p, s) : rows <= 16 ? launch_one<128, 16>(p, s) : launch_one<128, 32>(p, s);
}

}  // namespace moe
