// Attention over the paged 4-bit cache for many query rows a sequence (prompts
// and prompt chunks), on the tensor core.
//
// What bounds it: 4 D flops per (query row, key), two products of which the
// tensor core does 128 x 128 x D in 4 D clocks (D = 128: 512), against an
// exponential for each score and the dequantisation of each key and value once
// for every 256 rows. A CTA takes 256 rows (query, head of the group) in two
// tiles of 128 that alternate, so that the tensor core works on one while the
// other's softmax runs:
//   warps 0-3, 4-7   a softmax warpgroup for each tile, a thread a row: its 128
//                    scores from tensor memory into registers, probabilities
//                    back as fp16 in the same columns (the A operand of the
//                    second product)
//   warps 8-11       a thread a key: its K row from the cache's pages into shared
//                    memory as fp16, 128 keys a stage, two stages
//   warps 12-15      the same for V (one warpgroup for both was what the tensor
//                    core waited for: 4200 clocks a stage of its 2048)
//   warp 16          issues the products
// The codes come by cp.async, a warp its own 32 keys, a stage ahead of their use.
// The softmax is on a tile's path between its two products, so it is what must be
// short: the scores stay in registers (read twice from tensor memory, with 128
// registers a thread, 4096 queries of 32 heads behind 12288 keys took 875 us, so 766;
// with what follows 716, 71% of the tensor core's rate), and a stage is
// 128 keys wide, because the scores' product reads the queries again for each of
// its parts (64 keys wide, with the other 64 keys' softmax meanwhile: 924 us then).
// S = Q K^T has both operands K-major in the 128-byte swizzle; O += P V takes V
// from the same row-major form as an MN-major operand, so that nothing is
// transposed. Sums stay in tensor memory in fp32 over all keys; they are
// rescaled only when a row's maximum passes the one in use by 2^8.
//
// Precision. A code times its scale has 11 bits, so it is exact in fp16 but for
// its range: K and V rows are less the exponent of the largest K or V scale so far
// (K's put back in fp32 in the scores, V's at the end; the sums are rescaled when
// it grows). From the stage on where the K scales so far lie more than 2^16 apart
// (kKeyRange), or the V scales more than 2^10 (kValueRange; zeros too), the rows are the codes alone,
// and the softmax multiplies scores and probabilities by the keys' scales in fp32: a
// key that a row does not see, or that has no probability in it, takes nothing from
// the others. A query row enters less its own exponent, its largest value brought
// to [2^8, 2^9): values below 2^-25 of that are rounded at 2^-33 of it.
// What is rounded to fp16 for the second product is a probability against the row's
// largest so far, at 2^7 to 2^15, so at 2^-32 of the largest at most (at 1, a tail of
// 2^17 keys below 2^-25 was lost); with codes, its product with the V scale against
// the row's largest such product. (With every stage in codes the chunk of 4096 takes 1486 us.)
#include "kv4_attention.cuh"
#include "tcgen05.cuh"

#include <type_traits>

namespace moe {

namespace {

using namespace kv4;

constexpr int kKeys = 128;       // keys of a unit: one stage
constexpr int kTileRows = 128, kR = kPromptRows;
static_assert(kR == 2 * kTileRows, "two tiles");
constexpr int kThreads = 640;    // (three warps of the last warpgroup only take part in its register split)
constexpr int kWK = 8, kWV = 12, kWMma = 16;
constexpr int kStages = 2;
// registers a thread after the split: 256 x 160 + 256 x 64 + 128 x 32 = 640 x 96
constexpr int kRegsSoft = 160, kRegsDeq = 64, kRegsMma = 32, kRegsLaunch = 96;
static_assert(256 * kRegsSoft + 256 * kRegsDeq + 128 * kRegsMma <= kThreads * kRegsLaunch, "register split");
// What an item's start and end count for, in stages. (Ragged prompts, D = 64: 108.8 us with 2, 102.8
// with 3, 102.9 with 4; the chunk of 4096, D = 128: 719.7, 716.0, 715.6.)
constexpr int kLead = 3;

template <int D>
struct PromptCfg {
    static constexpr int kTile = 128 * D * 2;      // bytes of a fp16 tile of 128 rows: blocks of 64 columns, 16 KB each
    static constexpr int kChunks = D / 32;         // 16-byte pieces of a row of codes
    static constexpr int kRaw = 128 * D / 2;       // bytes of a stage's codes, K or V
    static constexpr int kSmem = (2 + 2 * kStages) * kTile + 2 * kRaw;
    // Shared addresses of the operands, known here so that their descriptors are constants: the
    // kernel's other shared memory lies below (the kernel checks it).
    static constexpr int kAtQ = 10240, kAtK = kAtQ + 2 * kTile, kAtV = kAtK + kStages * kTile;
};

struct Bars {
    uint64_t k_full[kStages], k_empty[kStages], v_full[kStages], v_empty[kStages];
    uint64_t s_full[2], p_full[2], q_full, o_full;
};

__device__ inline bool wait(uint64_t *bar, uint32_t parity, volatile int *abort_flag) {
    bool ok = false;
    for (uint32_t i = 0; i < kSpinLimit; ++i) {
        if ((ok = mbar_try_wait(bar, parity))) break;
        if ((i & 255) == 255 && *abort_flag) break;
    }
    return __all_sync(0xffffffffu, ok);
}

// Named barrier over n threads, returning the AND of v.
__device__ inline bool bar_and(int id, int n, bool v) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.and.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)v), "r"(id), "r"(n)
        : "memory");
    return r != 0;
}

template <int N>
__device__ inline void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ inline void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

// Octaves between the largest scale and the smallest so far up to which scales are
// multiplied into the rows. K's: the products' 11 bits lie above fp16's smallest. V's: a probability's rounding is 2^-22 of what the row's largest adds at most.
constexpr int kKeyRange = 16, kValueRange = 10;

// The exponents of the scales so far, K's or V's of an item.
constexpr int kNoExponent = 1 << 20;
__device__ inline int exponent_of(float s, int zero) {   // (bf16 has 7 octaves below its smallest normal)
    const int e = (int)(__float_as_uint(s) >> 23 & 0xFFu);
    return s == 0.f ? zero : e == 0 ? -7 : e;
}
struct Range {
    int top = 1, low = kNoExponent;
    __device__ bool holds(int e) const { return e == kNoExponent || (e <= top && e >= low); }
    __device__ static void take(int e, int *tops, int *lows, int w4, int lane) {   // a warp's
        const int t = (int)__reduce_max_sync(0xffffffffu, (uint32_t)(e == kNoExponent ? 0 : max(e, 0)));
        const int l = __reduce_min_sync(0xffffffffu, e);
        if (lane == 0) {
            tops[w4] = t;
            lows[w4] = l;
        }
    }
    __device__ void join(const int *tops, const int *lows) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            top = max(top, tops[i]);
            low = min(low, lows[i]);
        }
    }
};

// Descriptor of an operand at a shared address, 128-byte swizzle, 8 rows an atom
// of 1024 bytes. K-major: the leading stride is not used (1). A row-major
// [keys][64-column blocks] tile as an MN-major operand: 64 columns of a row are
// 128 swizzled bytes, atoms follow along K, 64-column blocks lie 16 KB apart (the
// leading stride, 1024 units of 16 bytes).
__host__ __device__ constexpr uint64_t sdesc(uint32_t addr, uint32_t lead) {
    return (uint64_t)((addr >> 4) & 0x3FFFu) | (uint64_t)lead << 16 | (uint64_t)(1024u >> 4) << 32 | (uint64_t)1u << 46 | (uint64_t)2u << 61;
}

// kind::f16, f16 operands, f32 sums; B K-major or MN-major.
__device__ inline uint32_t idesc_f16(int N, bool b_mn) {
    return (1u << 4) | (b_mn ? 1u << 16 : 0u) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}

// 32 columns of the thread's row.
__device__ inline void ld32(uint32_t taddr, float (&v)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
        "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
          "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]),
          "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]),
          "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
        : "r"(taddr)
        : "memory");
}
// The loads' registers are not to be read before the wait: it passes them on.
__device__ inline void wait_ld(float (&v)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                   "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]),
                   "+f"(v[16]), "+f"(v[17]), "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]), "+f"(v[23]),
                   "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]), "+f"(v[29]), "+f"(v[30]), "+f"(v[31])
                 :
                 : "memory");
}

__device__ inline void st16(uint32_t taddr, const uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}

// 16 columns of a thread's row of sums, times f.
__device__ inline void rescale16(uint32_t taddr, float f) {
    uint32_t v[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(taddr)
        : "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * f);
    st16(taddr, v);
}

__device__ inline void fma2(float &a, float &b, float c, float d) {   // (a, b) = (a, b) * c + d
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %2};\n\tmov.b64 z, {%3, %3};\n\t"
        "fma.rn.f32x2 x, x, y, z;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "+f"(a), "+f"(b)
        : "f"(c), "f"(d));
}
__device__ inline void add2(float &a, float &b, float c, float d) {
    asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %3};\n\t"
        "add.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "+f"(a), "+f"(b)
        : "f"(c), "f"(d));
}

// The softmax of a stage whose rows are codes: K's scales, V's less its exponent, and
// what the latter adds to a score to give the exponent of the product, less 7.
struct Scales {
    float k[kKeys], v[kKeys], by[kKeys];
};
struct CodesStage {
    const Scales &scales;
    float c_row;
    int left, up;        // keys of the stage that the row sees; how far V's exponent has risen
    bool sums, codes;    // there are sums so far; they are of stages of codes
    int low, sinks;      // (with a window) keys [sinks, low) of the stage are hidden from the row
};

// A thread's row (m, l0, l1), 32 keys at a time. Such stages come last in an item and have
// a loop of their own: as a branch in the other one they cost all prompts 4-7%, in line or not.
template <int D, bool kWindow>
__device__ inline void codes_stage(float (&row)[3], uint32_t tS, uint32_t tO, const CodesStage &a) {
    float m = row[0], l0 = row[1], l1 = row[2];
    auto scores = [&](int i, float (&x)[32]) {
        ld32(tS + i * 32, x);
        wait_ld(x);
        const int left = a.left - i * 32;
#pragma unroll
        for (int j = 0; j < 32; j += 4) {   // (the factors first: they meet in range)
            const float4 k = *reinterpret_cast<const float4 *>(&a.scales.k[i * 32 + j]);
            x[j] = j < left ? x[j] * (k.x * a.c_row) : -INFINITY;
            x[j + 1] = j + 1 < left ? x[j + 1] * (k.y * a.c_row) : -INFINITY;
            x[j + 2] = j + 2 < left ? x[j + 2] * (k.z * a.c_row) : -INFINITY;
            x[j + 3] = j + 3 < left ? x[j + 3] * (k.w * a.c_row) : -INFINITY;
        }
        if (kWindow) {
            const int low = a.low - i * 32, sinks = a.sinks - i * 32;
#pragma unroll
            for (int j = 0; j < 32; ++j)
                if (j < low && j >= sinks) x[j] = -INFINITY;
        }
    };
    float big = -INFINITY;
#pragma unroll 1
    for (int i = 0; i < 4; ++i) {
        float x[32];
        scores(i, x);
#pragma unroll
        for (int j = 0; j < 32; ++j) big = fmaxf(big, x[j] + a.scales.by[i * 32 + j]);
    }
    if (__any_sync(0xffffffffu, !a.codes || big > m + 8.f || a.up)) {
        // (from probabilities to products: the largest the row has may lie kValueRange below, or anywhere
        // where all V rows were zeros. In halves: a sum of probabilities may lie far above 1, the
        // factor below fp32's range)
        const float mn = fmaxf(a.codes ? m : m - (a.up ? 90.f : (float)kValueRange), big), down = exp2_approx(0.5f * (m - mn));
        m = mn;
        l0 = l0 * down * down;
        l1 = l1 * down * down;
        if (a.sums) {
            const float fo = a.up > 126 ? 0.f : down * down * pow2_biased(127 - a.up);
#pragma unroll 1
            for (int i = 0; i < D / 16; ++i) rescale16(tO + i * 16, fo);
        }
    }
#pragma unroll 1
    for (int i = 0; i < 4; ++i) {   // (the probabilities lie in columns that have been read)
        float x[32];
        uint32_t pr[16];
        scores(i, x);
#pragma unroll
        for (int j = 0; j < 32; j += 2) {
            const float2 f = *reinterpret_cast<const float2 *>(&a.scales.v[i * 32 + j]);
            const float y = exp2_approx(x[j] - m), z = exp2_approx(x[j + 1] - m);
            l0 += y;
            l1 += z;
            const __half2 v = __floats2half2_rn(y * f.x, z * f.y);
            pr[j >> 1] = *reinterpret_cast<const uint32_t *>(&v);
        }
        st16(tS + i * 16, pr);
    }
    row[0] = m;
    row[1] = l0;
    row[2] = l1;
}

// 8 codes of a word, times s, as the chunk of 8 fp16 values in the order
// 0, 4, 1, 5, 2, 6, 3, 7 (queries lie in the same order; the output's columns
// are put back at the end).
__device__ inline uint4 dequant_chunk(uint32_t w, __half2 s) {
    const uint32_t w8 = w >> 8;
    const uint32_t a[4] = {nib_lo(w), nib_hi(w), nib_lo(w8), nib_hi(w8)};
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 r = __hmul2(*reinterpret_cast<const __half2 *>(&a[i]), s);
        o[i] = *reinterpret_cast<const uint32_t *>(&r);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

template <int D>
__device__ inline uint8_t *chunk_at(uint8_t *tile, int row, int chunk) {   // 8 values of a row of a swizzled tile
    return tile + (chunk >> 3) * 16384 + row * 128 + (((chunk & 7) ^ (row & 7)) << 4);
}

template <int D, bool kWindow>
__global__ void __launch_bounds__(kThreads, 1) kv4_prompt_kernel(Attn p) {
    using Cfg = PromptCfg<D>;
    extern __shared__ uint8_t s_dyn[];
    uint8_t *const sQ = s_dyn + (Cfg::kAtQ - smem_u32(s_dyn));
    uint8_t *const sK = sQ + 2 * Cfg::kTile, *const sV = sK + kStages * Cfg::kTile, *const s_raw = sV + kStages * Cfg::kTile;
    int *const s_pre = reinterpret_cast<int *>(sK);   // (needed only before the first operand is written)
    static_assert(sizeof(int) * kMaxSeqs + sizeof(long long) * kThreads <= kStages * Cfg::kTile, "prefix");
    __shared__ Bars bars;
    __shared__ long long s_sums[kThreads / 32];
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort;
    __shared__ Item s_first;
    __shared__ alignas(16) int s_E[4], s_F[4], s_red[2][2][4][4];   // the K exponent (0: the rows are codes) and V exponent of a stage (rings of 4)
    // Scales of a stage of codes. A ring of 3: the stage three on is written after the scores of the next
    // have been formed, and those after this one's have been used.
    __shared__ alignas(16) Scales s_scale[3];
    __shared__ alignas(16) uint16_t s_scales[8][3][2][32];   // of a warp's stages in turn: K's, V's
    volatile int *const abort_flag = &s_abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    {
        uint32_t size;
        asm("mov.u32 %0, %%dynamic_smem_size;" : "=r"(size));
        if (smem_u32(s_dyn) > Cfg::kAtQ || smem_u32(s_dyn) + size < Cfg::kAtQ + Cfg::kSmem) {   // (the whole card: the same for every CTA)
            pdl_wait();
            if (threadIdx.x == 0) {
                set_error(p.ctrl, MOE_ERR_DEVICE);
                p.begun[blockIdx.x].last = 0;
            }
            return;
        }
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&bars.k_full[i], 4);
            mbar_init(&bars.k_empty[i], 1);
            mbar_init(&bars.v_full[i], 4);
            mbar_init(&bars.v_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars.s_full[i], 1);
            mbar_init(&bars.p_full[i], 4);
        }
        mbar_init(&bars.q_full, 8);
        mbar_init(&bars.o_full, 1);
        s_abort = 0;
        fence_mbar_init();
    }
    pdl_wait();
    pdl_launch_dependents();
    const int c = blockIdx.x;
    Item it;
    const Shares shares = first_item<kThreads, kKeys, kLead, kWindow>(p, kR, c, s_pre, s_sums, s_first, it);
    const int u_begin = c < shares.C ? shares.begin(c) : 0, u_end = c < shares.C ? shares.begin(c + 1) : 0;
    // the stages of an item in this CTA's share: [st0, st1)
    auto stages_of = [&](const Item &x, int &st0, int &st1) {
        st0 = max(u_begin - x.first - kLead, 0);
        st1 = min(x.units, u_end - x.first - kLead);
        return st1 > st0;
    };
    int st0, st1;
    if (c >= shares.C || !stages_of(it, st0, st1)) {   // (the whole CTA; a share that ends among leading units has nothing to do)
        if (threadIdx.x == 0) p.begun[c].last = 0;
        return;
    }
    // the next item with stages in the share; false: there is none
    auto go_on = [&]() {
        if (it.first + it.span >= u_end) return false;
        next_item<kKeys, kLead, kWindow>(p, kR, it);
        return stages_of(it, st0, st1);
    };
    if (warp == kWMma) {
        tc::alloc(&s_tmem, 512);
        tc::relinquish();
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    constexpr uint32_t tmem = 0;   // (all 512 columns: they begin at 0) columns: S0/P0 0-127, S1/P1 128-255, O0 from 256, O1 from 256 + D

    if (warp < kWK) {
        // ------------------------------------------------------------ softmax, a thread a row
        regs_inc<kRegsSoft>();
        const int wg = warp >> 2, r = threadIdx.x;   // row of the item
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t tS = tmem + lanes + wg * 128, tO = tmem + lanes + 256 + wg * D;
        uint32_t g = 0, gs = 0, n_item = 0;   // stages so far (all items; of this tile's), items
        bool ok = true;
        for (;; ++n_item) {
            const int rows = min(kR, it.s.nq * p.G - it.qt * kR);
            const int rr = it.qt * kR + r, qi = rr / p.G, head = it.h * p.G + rr - qi * p.G;
            const bool mine = wg * kTileRows < rows;   // (the whole warpgroup) this tile has rows
            // ---- the row's query
            float c_row = 0.f, l0 = 0.f, l1 = 0.f;
            int lim = 0, low = 0;
            const Gap gap = kWindow ? tile_gap<kKeys>(p, it.s, kR, it.qt) : Gap{0, 0};
            auto first_key = [&](int st) { return (kWindow ? gap.key_unit(st) : st) * kKeys; };
            {
                // whole rows at a time into the warp's part of the tile, then each thread its own
                constexpr int kPieces = D / 8, kAtOnce = 32 / kPieces;
                const long long at = (long long)(it.s.q0 + qi) * p.qs.token + (long long)head * p.qs.head;
                const bool there = r < rows;
#pragma unroll
                for (int i = 0; i < kPieces; ++i) {
                    const int row = i * kAtOnce + lane / kPieces, piece = lane % kPieces;
                    const long long src = __shfl_sync(0xffffffffu, there ? at : -1, row);
                    copy16(chunk_at<D>(sQ + wg * Cfg::kTile, (r & 96) + row, piece), p.q + (src < 0 ? 0 : src) + piece * 8, src >= 0);
                }
                copies_commit();
                copies_wait<0>();
                __syncwarp();
                uint4 x[D / 8];
                uint32_t big = 0;
#pragma unroll
                for (int i = 0; i < D / 8; ++i) {
                    x[i] = lds_v4(chunk_at<D>(sQ + wg * Cfg::kTile, r & 127, i));
                    const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) big = max(big, max(w[j] & 0x7FFFu, w[j] >> 16 & 0x7FFFu));
                }
                const int e = max(norm_exponent(big), 9);
                float f = pow2_biased(262 - e);   // the largest to [2^8, 2^9)
                if (p.scale < 0.f) f = -f;   // so that the largest product is the largest score
                if (there) lim = it.s.len - it.s.nq + qi + 1;
                if (kWindow && there) low = window_low(p, lim - 1);
                c_row = fabsf(p.scale) * kLog2e * pow2_biased(e - 8);
                if (big >= 0x7F80u && lim > 0) l0 = __uint_as_float(0x7fc00000u);   // a query that is not finite: NaN, where it sees a key
                uint8_t *const tile = sQ + wg * Cfg::kTile;
#pragma unroll
                for (int i = 0; i < D / 8; ++i) {
                    const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
                    uint32_t h[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {   // the pair (j, j + 4)
                        const uint32_t a = w[j >> 1], b = w[2 + (j >> 1)];
                        const __half2 v = __floats2half2_rn(__uint_as_float(j & 1 ? a & 0xffff0000u : a << 16) * f,
                                                            __uint_as_float(j & 1 ? b & 0xffff0000u : b << 16) * f);
                        h[j] = *reinterpret_cast<const uint32_t *>(&v);
                    }
                    *reinterpret_cast<uint4 *>(chunk_at<D>(tile, r & 127, i)) = make_uint4(h[0], h[1], h[2], h[3]);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars.q_full);
            }
            const int least = __reduce_min_sync(0xffffffffu, lim);
            const int low_last = kWindow ? __reduce_max_sync(0xffffffffu, low) : 0;
            float m = kNoMax;   // the exponent taken off: that of the largest probability (or product), less 7 to 15
            int F = 1;
            int st = st0;
            for (; st < st1 && ok; ++st, ++g) {
                if (!mine) continue;
                if (!(ok = wait(&bars.s_full[wg], gs & 1, abort_flag))) break;
                ++gs;
                tc::fence_after();
                const int E = s_E[g & 3], Fn = s_F[g & 3];
                if (E == 0) break;
                float x[128];
#pragma unroll
                for (int i = 0; i < 4; ++i) ld32(tS + i * 32, *reinterpret_cast<float(*)[32]>(x + i * 32));
#pragma unroll
                for (int i = 0; i < 4; ++i) wait_ld(*reinterpret_cast<float(*)[32]>(x + i * 32));
                const float ct = fmaxf(c_row * pow2_biased(E), 1e-37f);
                float mx[4];
                const int key0 = first_key(st);
                if (key0 + kKeys > least) {
                    const int left = lim - key0;   // keys of the stage that the row sees
#pragma unroll
                    for (int j = 0; j < 128; ++j)
                        if (j >= left) x[j] = -INFINITY;
                }
                if (kWindow && key0 < low_last && key0 + kKeys > p.sinks) {
                    const int before = low - key0, sinks = p.sinks - key0;   // keys [sinks, before) are hidden
#pragma unroll
                    for (int j = 0; j < 128; ++j)
                        if (j < before && j >= sinks) x[j] = -INFINITY;
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) mx[i] = x[i];
#pragma unroll
                for (int j = 4; j < 128; ++j) mx[j & 3] = fmaxf(mx[j & 3], x[j]);
                const float big = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * ct;
                if (__any_sync(0xffffffffu, big > m + 15.f || Fn != F)) {
                    // a new exponent (or V's): the row's sums so far follow it
                    const float mn = fmaxf(m, big - 7.f);
                    const float down = exp2_approx(m - mn);
                    m = mn;
                    l0 *= down;
                    l1 *= down;
                    const float fo = Fn - F > 126 ? 0.f : down * pow2_biased(127 + F - Fn);
                    F = Fn;
                    if (st > st0) {   // (all earlier products are complete: this stage's scores came after them)
#pragma unroll 1
                        for (int i = 0; i < D / 16; ++i) rescale16(tO + i * 16, fo);
                    }
                }
#pragma unroll
                for (int i = 0; i < 128; i += 32) {
                    uint32_t pr[16];
#pragma unroll
                    for (int j = 0; j < 32; j += 2) {
                        float &y = x[i + j], &z = x[i + j + 1];
                        fma2(y, z, ct, -m);
                        y = exp2_approx(y);
                        z = exp2_approx(z);
                        add2(l0, l1, y, z);
                        const __half2 v = __floats2half2_rn(y, z);
                        pr[j >> 1] = *reinterpret_cast<const uint32_t *>(&v);
                    }
                    st16(tS + (i >> 1), pr);
                }
                tc::wait_st();
                tc::fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars.p_full[wg]);
            }
            // ---- codes from here on
            for (bool codes = false; st < st1 && ok; ++st, ++g) {
                if (codes) {   // (the first one's scores have been waited for)
                    if (!(ok = wait(&bars.s_full[wg], gs & 1, abort_flag))) break;
                    ++gs;
                    tc::fence_after();
                }
                const int Fn = s_F[g & 3];
                float state[3] = {m, l0, l1};
                codes_stage<D, kWindow>(state, tS, tO, CodesStage{s_scale[g % 3], c_row, lim - first_key(st), Fn - F, st > st0, codes,
                                                                  low - first_key(st), p.sinks - first_key(st)});
                m = state[0];
                l0 = state[1];
                l1 = state[2];
                F = Fn;
                codes = true;
                tc::wait_st();
                tc::fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars.p_full[wg]);
            }
            // ---- the item's sums
            ok = ok && wait(&bars.o_full, n_item & 1, abort_flag);
            tc::fence_after();
            const bool whole = st0 == 0 && st1 == it.units;
            float *part = p.part + (size_t)(c * 2 + (st0 == 0)) * part_floats(kR, D);
            const float l = l0 + l1;
            if (ok && mine) {
                // 128 bytes of each of the warp's rows at a time through its part of the query tile (no
                // product reads it any more), so that 8 lanes write a row
                const float inv = l == 0.f ? 0.f : 1.f / l, up = pow2_biased(F);
                const long long at = (long long)(it.s.q0 + qi) * p.os.token + (long long)head * p.os.head;
                uint8_t *const mid = sQ + wg * Cfg::kTile + (warp & 3) * 4096;
                auto put = [&](int chunk, uint4 v) { *reinterpret_cast<uint4 *>(mid + lane * 128 + ((chunk ^ (lane & 7)) << 4)) = v; };
                auto rows_out = [&](auto &&store) {
                    __syncwarp();
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const int row = k * 4 + (lane >> 3);
                        store(row, lane & 7, lds_v4(mid + row * 128 + (((lane & 7) ^ (row & 7)) << 4)));
                    }
                    __syncwarp();
                };
#pragma unroll
                for (int i = 0; i < D / 32; ++i) {
                    float o[32];
                    ld32(tO + i * 32, o);
                    wait_ld(o);
#pragma unroll
                    for (int j = 0; j < 32; j += 8) {
                        const float v[8] = {o[j], o[j + 2], o[j + 4], o[j + 6], o[j + 1], o[j + 3], o[j + 5], o[j + 7]};
                        if (whole) {
                            put((i & 1) * 4 + j / 8, make_uint4(bf16x2_of(v[0] * inv * up, v[1] * inv * up), bf16x2_of(v[2] * inv * up, v[3] * inv * up),
                                                                bf16x2_of(v[4] * inv * up, v[5] * inv * up), bf16x2_of(v[6] * inv * up, v[7] * inv * up)));
                        } else {
                            put(j / 4, make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])));
                            put(j / 4 + 1, make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7])));
                        }
                    }
                    if (!whole) {
                        rows_out([&](int row, int piece, uint4 v) {
                            const int y = (r & ~31) + row;
                            if (y < rows) *reinterpret_cast<uint4 *>(part + 2 * kR + 4 + y * D + i * 32 + piece * 4) = v;
                        });
                    } else if (i & 1) {
                        rows_out([&](int row, int piece, uint4 v) {
                            const long long dst = __shfl_sync(0xffffffffu, at, row);
                            if ((r & ~31) + row < rows) *reinterpret_cast<uint4 *>(p.out + dst + (i >> 1) * 64 + piece * 8) = v;
                        });
                    }
                }
                if (r < rows) {
                    if (whole) {
                        if (p.lse) p.lse[(size_t)(it.s.q0 + qi) * p.Hq + head] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
                    } else {
                        part[r] = m;
                        part[kR + r] = l;
                        if (r == 0) part[2 * kR] = __int_as_float(F);
                    }
                }
            }
            tc::fence_before();
            if (!ok) {
                *abort_flag = 1;
                if (lane == 0) set_error(p.ctrl, MOE_ERR_TIMEOUT);
            }
            const Begun begun{ok && st0 == 0 && !whole ? shares.holder(it.first + it.span - 1) : 0, it.s.q0, it.h, it.qt, rows, {0, 0, 0}};
            if (!ok || !go_on()) {
                if (threadIdx.x == 0) p.begun[c] = begun;
                break;
            }
        }
    } else if (warp < kWMma) {
        // ------------------------------------------------------------ keys (warps 8-11) or values, a thread a key
        regs_dec<kRegsDeq>();
        const bool keys = warp < kWV;
        const int r = threadIdx.x & 127, w4 = warp & 3, run = w4 * 32 + (lane & 16);
        uint8_t *const raw = s_raw + (keys ? 0 : Cfg::kRaw) + w4 * (32 * D / 2), *const tiles = keys ? sK : sV;
        uint64_t *const full = keys ? bars.k_full : bars.v_full, *const empty = keys ? bars.k_empty : bars.v_empty;
        uint16_t(*const scales)[2][32] = s_scales[warp - kWK];
        // A warp's 32 keys are two runs of 16, each in one page: lane i knows the run of keys
        // 16 (i / 16) ... and the warp copies 512 bytes at a time, the 16-byte pieces of a row
        // turned by the row, so that lanes that read a row each meet no bank twice.
        constexpr uint32_t kNone = 0xffffffffu;   // no such keys, or a page that does not exist: they read as zero
        auto turned = [](int x) { return D == 128 ? x >> 1 & 3 : x >> 2 & 1; };
        const int copy_to = (lane / Cfg::kChunks * Cfg::kChunks + (lane % Cfg::kChunks ^ turned(lane / Cfg::kChunks))) * 16;
        const char *const from = reinterpret_cast<const char *>(keys ? p.c.k_codes : p.c.v_codes) + lane * 16;
        const uint16_t *const scales_from = ((lane & 2) ? p.c.v_scales : p.c.k_scales) + (lane & 1) * 8;
        uint32_t g = 0;
        bool ok = true;
        for (;;) {
            const int len = it.s.len;
            const int32_t *table = p.b.table + (size_t)it.b * p.b.max_pages;
            const Gap gap = kWindow ? tile_gap<kKeys>(p, it.s, kR, it.qt) : Gap{0, 0};
            const int low = kWindow ? window_low(p, len - it.s.nq + it.qt * kR / p.G) : 0;   // of the item's first row
            auto first_key = [&](int st) { return (kWindow ? gap.key_unit(st) : st) * kKeys; };
            // (a run that no row sees is not read: its page may be gone)
            auto in_reach = [&](int key) { return key < len && (!kWindow || key < p.sinks || key > low - 16); };
            // a key that no row sees, of a run that is read, is as one that is not there: it counts for no exponent,
            // and what would be out of their range does not enter the products
            const int end = kWindow ? tile_keys(it.s, p.G, kR, it.qt) : len;
            auto seen = [&](int key) { return key < end && (!kWindow || key < p.sinks || key >= low); };
            auto page_of = [&](int st) {
                const int key = first_key(st) + run;
                return st < st1 && in_reach(key) ? ld_here(table + (key >> p.b.shift)) : -1;
            };
            auto place = [&](int st, int page) {   // the run's first row (row indexes are below 2^32 - 1)
                const int key = first_key(st) + run;
                if (st >= st1 || !in_reach(key)) return kNone;
                if ((unsigned)page >= (unsigned)p.c.n_pages) {
                    set_error(p.ctrl, MOE_ERR_DEVICE);
                    return kNone;
                }
                return (((uint32_t)page * (uint32_t)p.c.Hkv + (uint32_t)it.h) << p.b.shift) + (uint32_t)(key & ((1 << p.b.shift) - 1));
            };
            auto copy = [&](uint32_t at, int slot) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t src = __shfl_sync(0xffffffffu, at, 16 * i);
                    const bool there = src != kNone;
                    const char *x = from + (size_t)(there ? src : 0) * (D / 2);
#pragma unroll
                    for (int k = 0; k < D / 64; ++k) copy16(raw + copy_to + i * (8 * D) + k * 512, x + k * 512, there);
                }
                // a run's scales are 32 bytes: lanes 0-1 and 16-17 copy K's, 2-3 and 18-19 V's
                if ((lane & 15) < 4)
                    copy16(&scales[slot][lane >> 1 & 1][(lane & 16) + (lane & 1) * 8], scales_from + (at != kNone ? at : 0), at != kNone);
                copies_commit();
            };
            uint32_t at0 = place(st0, page_of(st0)), at1 = kNone;
            int page = page_of(st0 + 1), slot = 0, E = 1, F = 1;
            Range k_range, v_range;
            bool codes = false;   // the scales so far lie too far apart
            copy(at0, 0);
            for (int st = st0; st < st1; ++st, ++g) {
                const int b = g % kStages;
                copies_wait<0>();
                __syncwarp();
                uint4 w[Cfg::kChunks];
#pragma unroll
                for (int i = 0; i < Cfg::kChunks; ++i) w[i] = lds_v4(raw + (lane * Cfg::kChunks + (i ^ turned(lane))) * 16);
                const int key = first_key(st) + r;
                const bool there = at0 != kNone && seen(key);
                const uint16_t ks = there ? scales[slot][0][lane] : (uint16_t)0, vs = there ? scales[slot][1][lane] : (uint16_t)0;
                __syncwarp();
                slot = slot == 2 ? 0 : slot + 1;
                if (st + 1 < st1) {
                    at1 = place(st + 1, page);
                    page = page_of(st + 2);
                    copy(at1, slot);
                }
                at0 = at1;
                ok = wait(&empty[b], ((g / kStages) & 1) ^ 1, abort_flag);
                // ---- the exponents; a row that was not finite: K becomes NaN, V zero
                const bool bad = !finite_bits(ks) || !finite_bits(vs);
                const float kf = bad ? 0.f : bf16_bits_to_f32(ks), vf = bad ? 0.f : bf16_bits_to_f32(vs);
                // (a row of zeros in V lies far below the others: its key may have all the probability)
                const int ke = exponent_of(kf, kNoExponent), ve = exponent_of(vf, seen(key) && !bad ? -100 : kNoExponent);
                // (most stages change nothing: that is seen at the barrier alone. With four reductions a warp
                // for each stage's own exponents the prompt chunk took 756 us, so 732; with the first stage's
                // before the wait 850)
                if (st == st0 || !bar_and(keys ? 2 : 3, 128, ok && k_range.holds(ke) && v_range.holds(ve))) {
                    int(&red)[4][4] = s_red[!keys][g & 1];   // (a stage has a barrier at least: the last stage's may still be read)
                    Range::take(ke, red[0], red[1], w4, lane);
                    Range::take(ve, red[2], red[3], w4, lane);
                    if (!(ok = bar_and(keys ? 2 : 3, 128, ok))) break;   // (for all warps of the role at once)
                    k_range.join(red[0], red[1]);
                    v_range.join(red[2], red[3]);
                    // (with codes V's exponent stays, as a middle for their range)
                    if (!codes) {
                        // (V all zeros so far: none is lost to another)
                        codes = k_range.low < k_range.top - kKeyRange || (v_range.top > 1 && v_range.low < v_range.top - kValueRange);
                        if (!codes || F == 1) F = min(v_range.top, 253);
                        E = codes ? 0 : min(k_range.top, 253);
                    }
                }
                if (keys) {
                    if (codes) {
                        const float f = fminf(fmaxf(vf * pow2_biased(254 - F), -0x1p120f), 0x1p120f);
                        Scales &to = s_scale[g % 3];
                        to.k[r] = kf;
                        to.v[r] = f;
                        to.by[r] = fmaxf(log2_approx(fabsf(f)) - 7.f, -90.f);
                    }
                    if (r == 0) {
                        s_E[g & 3] = E;
                        s_F[g & 3] = F;
                    }
                }
                const float factor = keys && bad ? NAN : codes ? 1.f : keys ? kf * pow2_biased(254 - E) : vf * pow2_biased(254 - F);
                const __half2 s2 = __float2half2_rn(factor);
#pragma unroll
                for (int i = 0; i < Cfg::kChunks; ++i) {
                    const uint32_t x[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        *reinterpret_cast<uint4 *>(chunk_at<D>(tiles + b * Cfg::kTile, r, i * 4 + j)) = dequant_chunk(x[j], s2);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&full[b]);
            }
            if (!ok) {
                *abort_flag = 1;
                if (lane == 0) set_error(p.ctrl, MOE_ERR_TIMEOUT);
                break;
            }
            if (!go_on()) break;
        }
        copies_wait<0>();
    } else {
        regs_dec<kRegsMma>();
        if (warp == kWMma) {
            // -------------------------------------------------------- the products
            const uint32_t id_s = idesc_f16(128, false), id_o = idesc_f16(D, true);
            uint32_t g = 0, gp[2] = {0, 0}, n_item = 0;
            bool ok = true;
            const std::integral_constant<int, 0> c0;
            const std::integral_constant<int, 1> c1;
            static_assert(kStages == 2, "buffers");
            // Tile, stage and addresses are constants here: descriptors made from registers were kept
            // in too many of them, and moved to where the instructions take them from each time
            // (the figure above: 766 -> 715 us).
            const uint32_t lead = elect();
            auto scores = [&](auto wg_c, auto b_c) {
                constexpr int wg = decltype(wg_c)::value, b = decltype(b_c)::value;
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint64_t x = sdesc(Cfg::kAtQ + wg * Cfg::kTile + (k >> 2) * 16384 + (k & 3) * 32, 1);
                    const uint64_t y = sdesc(Cfg::kAtK + b * Cfg::kTile + (k >> 2) * 16384 + (k & 3) * 32, 1);
                    mma_ss(lead, tmem + wg * 128, x, y, id_s, k > 0);
                }
                commit(lead, &bars.s_full[wg]);
            };
            auto values = [&](auto wg_c, auto b_c, bool first) {
                constexpr int wg = decltype(wg_c)::value, b = decltype(b_c)::value;
#pragma unroll
                for (int k = 0; k < kKeys / 16; ++k)
                    mma_ts(lead, tmem + 256 + wg * D, tmem + wg * 128 + k * 8, sdesc(Cfg::kAtV + b * Cfg::kTile + k * 2048, 1024), id_o, !first || k > 0);
            };
            auto done = [&](uint64_t *bar) { commit(lead, bar); };
            for (;; ++n_item) {
                const bool two = it.s.nq * p.G - it.qt * kR > kTileRows;
                // scores of the item's first stage, in buffer b
                auto start = [&](auto b_c) {
                    constexpr int b = decltype(b_c)::value;
                    if (!(ok = wait(&bars.q_full, n_item & 1, abort_flag) && wait(&bars.k_full[b], (g / kStages) & 1, abort_flag))) return;
                    tc::fence_after();
                    scores(c0, b_c);
                    if (two) scores(c1, b_c);
                    done(&bars.k_empty[b]);
                };
                // values of a stage in buffer b, scores of the next
                auto step = [&](auto b_c, auto bn_c, bool first, bool more) {
                    constexpr int b = decltype(b_c)::value, bn = decltype(bn_c)::value;
                    ok = wait(&bars.v_full[b], (g / kStages) & 1, abort_flag) && wait(&bars.p_full[0], gp[0] & 1, abort_flag);
                    if (!ok) return;
                    ++gp[0];
                    tc::fence_after();
                    values(c0, b_c, first);
                    if (more) {
                        if (!(ok = wait(&bars.k_full[bn], ((g + 1) / kStages) & 1, abort_flag))) return;
                        tc::fence_after();
                        scores(c0, bn_c);
                    }
                    if (two) {
                        if (!(ok = wait(&bars.p_full[1], gp[1] & 1, abort_flag))) return;
                        ++gp[1];
                        tc::fence_after();
                        values(c1, b_c, first);
                    }
                    done(&bars.v_empty[b]);
                    if (more) {
                        if (two) scores(c1, bn_c);
                        done(&bars.k_empty[bn]);
                    }
                };
                if (g & 1) start(c1); else start(c0);
                for (int st = st0; st < st1 && ok; ++st, ++g) {
                    if (g & 1) step(c1, c0, st == st0, st + 1 < st1);
                    else step(c0, c1, st == st0, st + 1 < st1);
                }
                done(&bars.o_full);
                if (!ok) {
                    // the products in flight end by themselves: give them a bounded wait before the CTA exits
                    for (uint32_t i = 0; i < kSpinLimit && !mbar_try_wait(&bars.o_full, n_item & 1); ++i) {}
                    *abort_flag = 1;
                    if (lane == 0) set_error(p.ctrl, MOE_ERR_TIMEOUT);
                    break;
                }
                if (!go_on()) break;
            }
        }
    }
    __syncwarp();
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    if (warp == kWMma) tc::dealloc(tmem, 512);
}

template <int D, bool kWindow>
cudaError_t launch_one(const Attn &p, int *grid_out, cudaStream_t s) {
    const void *fn = reinterpret_cast<const void *>(kv4_prompt_kernel<D, kWindow>);
    // The register split takes what the launch reserves: it must be the whole of it.
    static const bool split_ok = [fn] {
        cudaFuncAttributes a;
        return cudaFuncGetAttributes(&a, fn) == cudaSuccess && a.numRegs >= kRegsLaunch;
    }();
    if (!split_ok) return cudaErrorInvalidConfiguration;
    constexpr size_t kBase = PromptCfg<D>::kSmem + PromptCfg<D>::kAtQ - 1024;   // (what comes first: the system's 1 KB)
    const cudaError_t err = set_smem_once(fn, (int)kBase);
    if (err != cudaSuccess) return err;
    int grid = sm_count();
    if (grid > kMaxPromptCtas) grid = kMaxPromptCtas;
    *grid_out = grid;
    return launch_pdl(kv4_prompt_kernel<D, kWindow>, dim3((unsigned)grid), kThreads, kBase, s, p);
}

}  // namespace

cudaError_t launch_kv4_prompt(const kv4::Attn &p, int *grid, cudaStream_t s) {
    if (p.window) return p.c.D == 64 ? launch_one<64, true>(p, grid, s) : launch_one<128, true>(p, grid, s);
    return p.c.D == 64 ? launch_one<64, false>(p, grid, s) : launch_one<128, false>(p, grid, s);
}

}  // namespace moe
