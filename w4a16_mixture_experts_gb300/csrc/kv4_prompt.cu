// Attention over the paged 4-bit cache for many query rows a sequence (prompts
// and prompt chunks), on the tensor core.
//
// What bounds it: 4 D flops per (query row, key), two products of which the
// tensor core does 128 x 128 x D in 64 D clocks (D = 128: 512), against an
// exponential for each score and the dequantisation of each key and value once
// for every 256 rows. A CTA takes 256 rows (query, head of the group) in two
// tiles of 128 that alternate, so that the tensor core works on one while the
// other's softmax runs:
//   warps 0-3, 4-7   a softmax warpgroup for each tile, a thread a row: scores
//                    from tensor memory into registers, probabilities back as
//                    fp16 in the same columns (the A operand of the second product)
//   warps 8-11       a thread a key: its K and V row from the cache's pages into
//                    shared memory as fp16, 128 keys a stage, two stages each
//   warp 12          issues the products
// S = Q K^T has both operands K-major in the 128-byte swizzle; O += P V takes V
// from the same row-major form as an MN-major operand, so that nothing is
// transposed. Sums stay in tensor memory in fp32 over all keys; they are
// rescaled only when a row's maximum passes the one in use by 2^8.
//
// Precision. A code times its scale has 11 bits, so it is exact in fp16 but for
// its range: a stage's K rows are less the exponent of the stage's largest K
// scale (put back in fp32 in the scores), V rows less that of the largest V
// scale so far (put back at the end; the sums are rescaled when it grows), and a
// query row less its own. Rows more than 2^14 below the largest lose bits that
// are below 2^-24 of it. Probabilities are rounded to fp16.
#include "kv4_attention.cuh"
#include "tcgen05.cuh"

namespace moe {

namespace {

using namespace kv4;

constexpr int kKeys = 128;       // keys of a unit: one stage
constexpr int kTileRows = 128, kR = kPromptRows;
static_assert(kR == 2 * kTileRows, "two tiles");
constexpr int kThreads = 512;    // (three warps of the last warpgroup only take part in its register split)
constexpr int kWK = 8, kWMma = 12;
constexpr int kStages = 2;
// registers a thread after the split: 256 x 176 + 128 x 80 + 128 x 80 = 512 x 128
constexpr int kRegsSoft = 176, kRegsDeq = 80, kRegsMma = 80, kRegsLaunch = 128;
static_assert(256 * kRegsSoft + 128 * kRegsDeq + 128 * kRegsMma <= kThreads * kRegsLaunch, "register split");

template <int D>
struct PromptCfg {
    static constexpr int kTile = 128 * D * 2;      // bytes of a fp16 tile of 128 rows: blocks of 64 columns, 16 KB each
    static constexpr int kSmem = (2 + 2 * kStages) * kTile;
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

__device__ inline bool elect() {
    uint32_t pred;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(pred));
    return pred != 0;
}

template <int N>
__device__ inline void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ inline void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

// A row-major [keys][64-column blocks] tile as an MN-major operand: 64 columns
// of a row are 128 swizzled bytes, 8 rows an atom of 1024 (the stride along K),
// 64-column blocks 16 KB apart (the leading stride).
__device__ inline uint64_t sdesc_mn_sw128(const void *smem_ptr) {
    const uint32_t addr = smem_u32(smem_ptr);
    return (uint64_t)((addr >> 4) & 0x3FFFu) | (uint64_t)(16384u >> 4) << 16 | (uint64_t)(1024u >> 4) << 32 |
           (uint64_t)1u << 46 | (uint64_t)2u << 61;
}

// kind::f16, f16 operands, f32 sums; B K-major or MN-major.
__device__ inline uint32_t idesc_f16(int N, bool b_mn) {
    return (1u << 4) | (b_mn ? 1u << 16 : 0u) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
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
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
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

template <int D>
__global__ void __launch_bounds__(kThreads, 1) kv4_prompt_kernel(Attn p) {
    using Cfg = PromptCfg<D>;
    extern __shared__ uint8_t s_dyn[];
    uint8_t *const sQ = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(s_dyn) + 1023) & ~(uintptr_t)1023);
    uint8_t *const sK = sQ + 2 * Cfg::kTile, *const sV = sK + kStages * Cfg::kTile;
    int *const s_pre = reinterpret_cast<int *>(sV + kStages * Cfg::kTile);
    __shared__ Bars bars;
    __shared__ long long s_sums[kThreads / 32];
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort;
    __shared__ int s_E[4], s_F[4], s_red[2][2][4];   // a stage's K exponent, V exponent so far (rings of 4 stages)
    volatile int *const abort_flag = &s_abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

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
    const int U = scan_units<kThreads, kKeys>(p, kR, s_pre, s_sums);
    const Shares shares(U, min((int)gridDim.x, max(1, U)));
    const int c = blockIdx.x;
    if (c >= shares.C || U == 0) {   // (the whole CTA)
        if (threadIdx.x == 0) p.begun[c].last = 0;
        return;
    }
    const int u_begin = shares.begin(c), u_end = shares.begin(c + 1);
    if (warp == kWMma) {
        tc::alloc(&s_tmem, 512);
        tc::relinquish();
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = s_tmem;   // columns: S0/P0 0-127, S1/P1 128-255, O0 from 256, O1 from 256 + D

    if (warp < kWK) {
        // ------------------------------------------------------------ softmax, a thread a row
        regs_inc<kRegsSoft>();
        const int wg = warp >> 2, r = threadIdx.x;   // row of the item
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t tS = tmem + lanes + wg * 128, tO = tmem + lanes + 256 + wg * D;
        uint32_t g = 0, gs = 0, n_item = 0;   // stages so far (all items; of this tile's), items
        bool ok = true;
        Item it = find_item<kKeys>(p, kR, s_pre, u_begin);
        for (int u = u_begin;; next_item<kKeys>(p, kR, it), ++n_item) {
            const int st0 = u - it.first, st1 = min(it.units, u_end - it.first);
            const int rows = min(kR, it.s.nq * p.G - it.qt * kR);
            const int rr = it.qt * kR + r, qi = rr / p.G, head = it.h * p.G + rr - qi * p.G;
            const bool mine = wg * kTileRows < rows;   // (the whole warpgroup) this tile has rows
            // ---- the row's query
            float c_row = 0.f;
            int lim = 0;
            {
                uint4 x[D / 8];
                uint32_t big = 0;
                const bool there = r < rows;
                const uint16_t *src = p.q + (size_t)(it.s.q0 + qi) * p.qs.token + (size_t)head * p.qs.head;
#pragma unroll
                for (int i = 0; i < D / 8; ++i) {
                    x[i] = there ? *reinterpret_cast<const uint4 *>(src + i * 8) : make_uint4(0, 0, 0, 0);
                    const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) big = max(big, max(w[j] & 0x7FFFu, w[j] >> 16 & 0x7FFFu));
                }
                const int e = norm_exponent(big);
                float f = pow2_biased(254 - e);
                if (p.scale < 0.f) f = -f;   // so that the largest product is the largest score
                if (there) lim = it.s.len - it.s.nq + qi + 1;
                c_row = fabsf(p.scale) * kLog2e * pow2_biased(e);
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
            float m = kNoMax, l0 = 0.f, l1 = 0.f;
            int F = 1;
            for (int st = st0; st < st1 && ok; ++st, ++g) {
                if (!mine) continue;
                if (!(ok = wait(&bars.s_full[wg], gs & 1, abort_flag))) break;
                ++gs;
                tc::fence_after();
                float s[4][32];
#pragma unroll
                for (int i = 0; i < 4; ++i) tc::ld_32x32b_x32(tS + i * 32, s[i]);
#pragma unroll
                for (int i = 0; i < 4; ++i) wait_ld(s[i]);
                const int E = s_E[g & 3], Fn = s_F[g & 3];
                const float ct = fmaxf(c_row * pow2_biased(E), 1e-37f);
                if (st * kKeys + kKeys > least) {
                    const int left = lim - st * kKeys;   // keys of the stage that the row sees
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (i * 32 + j >= left) s[i][j] = -INFINITY;
                }
                float mx[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    mx[i] = s[i][0];
#pragma unroll
                    for (int j = 1; j < 32; ++j) mx[i] = fmaxf(mx[i], s[i][j]);
                }
                const float big = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * ct;
                if (__any_sync(0xffffffffu, big > m + 8.f || Fn != F)) {
                    // a new maximum (or exponent of V): the row's sums so far follow it
                    const float mn = fmaxf(m, big);
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
                for (int h = 0; h < 2; ++h) {   // 64 keys at a time
                    uint32_t pr[32];
#pragma unroll
                    for (int j = 0; j < 64; j += 2) {
                        float &x = s[h * 2 + (j >> 5)][j & 31], &y = s[h * 2 + (j >> 5)][(j & 31) + 1];
                        fma2(x, y, ct, -m);
                        x = exp2_approx(x);
                        y = exp2_approx(y);
                        add2(l0, l1, x, y);
                        const __half2 v = __floats2half2_rn(x, y);
                        pr[j >> 1] = *reinterpret_cast<const uint32_t *>(&v);
                    }
                    tc::st_32x32b_x32(tS + h * 32, pr);
                }
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
                const float inv = l == 0.f ? 0.f : 1.f / l, up = pow2_biased(F);
                uint16_t *dst = p.out + (size_t)(it.s.q0 + qi) * p.os.token + (size_t)head * p.os.head;
#pragma unroll
                for (int i = 0; i < D / 32; ++i) {
                    float o[32];
                    tc::ld_32x32b_x32(tO + i * 32, o);
                    wait_ld(o);
                    if (r < rows) {
#pragma unroll
                        for (int j = 0; j < 32; j += 8) {
                            const float v[8] = {o[j], o[j + 2], o[j + 4], o[j + 6], o[j + 1], o[j + 3], o[j + 5], o[j + 7]};
                            if (whole) {
                                *reinterpret_cast<uint4 *>(dst + i * 32 + j) =
                                    make_uint4(bf16x2_of(v[0] * inv * up, v[1] * inv * up), bf16x2_of(v[2] * inv * up, v[3] * inv * up),
                                               bf16x2_of(v[4] * inv * up, v[5] * inv * up), bf16x2_of(v[6] * inv * up, v[7] * inv * up));
                            } else {
                                float4 *d = reinterpret_cast<float4 *>(part + 2 * kR + 4 + r * D + i * 32 + j);
                                d[0] = make_float4(v[0], v[1], v[2], v[3]);
                                d[1] = make_float4(v[4], v[5], v[6], v[7]);
                            }
                        }
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
            u = it.first + st1;
            if (threadIdx.x == 0 && (!ok || u >= u_end)) {
                const bool goes_on = ok && st0 == 0 && !whole;
                p.begun[c] = Begun{goes_on ? shares.holder(it.first + it.units - 1) : 0, it.s.q0, it.h, it.qt, rows, {0, 0, 0}};
            }
            if (!ok) {
                *abort_flag = 1;
                if (lane == 0) set_error(p.ctrl, MOE_ERR_TIMEOUT);
                break;
            }
            if (u >= u_end) break;
        }
    } else if (warp < kWMma) {
        // ------------------------------------------------------------ keys and values, a thread a key
        regs_dec<kRegsDeq>();
        const int r = threadIdx.x & 127, w4 = warp & 3;
        uint32_t g = 0;
        bool ok = true;
        Item it = find_item<kKeys>(p, kR, s_pre, u_begin);
        for (int u = u_begin; ok; next_item<kKeys>(p, kR, it)) {
            const int st0 = u - it.first, st1 = min(it.units, u_end - it.first);
            const int32_t *table = p.b.table + (size_t)it.b * p.b.max_pages;
            const int len = it.s.len, pmask = (1 << p.b.shift) - 1;
            auto page_of = [&](int st) {
                const int key = st * kKeys + r;
                return st < st1 && key < len ? __ldg(table + (key >> p.b.shift)) : -1;
            };
            uint4 kw[D / 32], vw[D / 32];
            uint16_t ks = 0, vs = 0;
            size_t row = 0;
            auto place = [&](int st, int page) {   // the thread's row of stage st; its scales
                const int key = st * kKeys + r;
                const bool in = st < st1 && key < len, fine = in && (unsigned)page < (unsigned)p.c.n_pages;
                if (in && !fine) set_error(p.ctrl, MOE_ERR_DEVICE);
                row = fine ? (((size_t)page * p.c.Hkv + it.h) << p.b.shift) + (key & pmask) : 0;
                ks = fine ? __ldg(p.c.k_scales + row) : 0;
                vs = fine ? __ldg(p.c.v_scales + row) : 0;
            };
            auto load = [&](uint4 (&w)[D / 32], const int32_t *codes) {
#pragma unroll
                for (int i = 0; i < D / 32; ++i) w[i] = ld_nc_v4(codes + row * (D / 8) + i * 4);
            };
            auto store = [&](uint8_t *tile, const uint4 (&w)[D / 32], __half2 s) {
#pragma unroll
                for (int i = 0; i < D / 32; ++i) {
                    const uint32_t x[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        *reinterpret_cast<uint4 *>(chunk_at<D>(tile, r, i * 4 + j)) = dequant_chunk(x[j], s);
                }
            };
            place(st0, page_of(st0));
            load(kw, p.c.k_codes);
            load(vw, p.c.v_codes);
            int page = page_of(st0 + 1);
            int F = 1;
            for (int st = st0; st < st1; ++st, ++g) {
                const int b = g % kStages;
                const uint32_t ph = (g / kStages) & 1;
                ok = ok && wait(&bars.k_empty[b], ph ^ 1, abort_flag);
                // ---- the stage's exponents; a row that was not finite: K becomes NaN, V zero
                const bool bad = !finite_bits(ks) || !finite_bits(vs);
                const float kf = bad ? 0.f : bf16_bits_to_f32(ks), vf = bad ? 0.f : bf16_bits_to_f32(vs);
                const uint32_t ek = __reduce_max_sync(0xffffffffu, __float_as_uint(kf) >> 23 & 0xFFu);
                const uint32_t ev = __reduce_max_sync(0xffffffffu, __float_as_uint(vf) >> 23 & 0xFFu);
                if (lane == 0) {
                    s_red[g & 1][0][w4] = (int)ek;
                    s_red[g & 1][1][w4] = (int)ev;
                }
                if (!(ok = bar_and(2, 128, ok))) break;
                int E = 1;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    E = max(E, s_red[g & 1][0][i]);
                    F = max(F, s_red[g & 1][1][i]);
                }
                E = min(E, 253);
                F = min(F, 253);
                if (r == 0) {
                    s_E[g & 3] = E;
                    s_F[g & 3] = F;
                }
                const __half2 k2 = bad ? __float2half2_rn(NAN) : __float2half2_rn(kf * pow2_biased(254 - E));
                const __half2 v2 = __float2half2_rn(vf * pow2_biased(254 - F));
                store(sK + b * Cfg::kTile, kw, k2);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars.k_full[b]);
                const bool more = st + 1 < st1;
                if (more) {
                    place(st + 1, page);
                    load(kw, p.c.k_codes);
                    page = page_of(st + 2);
                }
                ok = wait(&bars.v_empty[b], ph ^ 1, abort_flag);
                if (ok) store(sV + b * Cfg::kTile, vw, v2);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars.v_full[b]);
                if (more) load(vw, p.c.v_codes);
            }
            u = it.first + st1;
            if (!ok) {
                *abort_flag = 1;
                if (lane == 0) set_error(p.ctrl, MOE_ERR_TIMEOUT);
                break;
            }
            if (u >= u_end) break;
        }
    } else {
        regs_dec<kRegsMma>();
        if (warp == kWMma) {
            // -------------------------------------------------------- the products
            const uint32_t id_s = idesc_f16(128, false), id_o = idesc_f16(D, true);
            uint32_t g = 0, gp[2] = {0, 0}, n_item = 0;
            bool ok = true;
            auto scores = [&](int wg, int b) {
                if (elect()) {
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        const uint64_t a = tc::sdesc_sw128(sQ + wg * Cfg::kTile + (k >> 2) * 16384) + (uint64_t)((k & 3) * 2);
                        const uint64_t d = tc::sdesc_sw128(sK + b * Cfg::kTile + (k >> 2) * 16384) + (uint64_t)((k & 3) * 2);
                        tc::mma_ss(tmem + wg * 128, a, d, id_s, k > 0);
                    }
                    tc::commit(&bars.s_full[wg]);
                }
                __syncwarp();
            };
            auto values = [&](int wg, int b, bool first) {
                if (elect()) {
                    const uint64_t d = sdesc_mn_sw128(sV + b * Cfg::kTile);
#pragma unroll
                    for (int k = 0; k < kKeys / 16; ++k)
                        tc::mma_ts(tmem + 256 + wg * D, tmem + wg * 128 + k * 8, d + (uint64_t)(k * 128), id_o, !first || k > 0);
                }
                __syncwarp();
            };
            auto done = [&](uint64_t *bar) {
                if (elect()) tc::commit(bar);
                __syncwarp();
            };
            Item it = find_item<kKeys>(p, kR, s_pre, u_begin);
            for (int u = u_begin;; next_item<kKeys>(p, kR, it), ++n_item) {
                const int st0 = u - it.first, st1 = min(it.units, u_end - it.first);
                const bool two = it.s.nq * p.G - it.qt * kR > kTileRows;
                ok = wait(&bars.q_full, n_item & 1, abort_flag) && wait(&bars.k_full[g % kStages], (g / kStages) & 1, abort_flag);
                if (ok) {
                    tc::fence_after();
                    scores(0, g % kStages);
                    if (two) scores(1, g % kStages);
                    done(&bars.k_empty[g % kStages]);
                }
                for (int st = st0; st < st1 && ok; ++st, ++g) {
                    const int b = g % kStages, bn = (g + 1) % kStages;
                    const bool more = st + 1 < st1;
                    ok = wait(&bars.v_full[b], (g / kStages) & 1, abort_flag) && wait(&bars.p_full[0], gp[0] & 1, abort_flag);
                    if (!ok) break;
                    ++gp[0];
                    tc::fence_after();
                    values(0, b, st == st0);
                    if (more) {
                        if (!(ok = wait(&bars.k_full[bn], ((g + 1) / kStages) & 1, abort_flag))) break;
                        tc::fence_after();
                        scores(0, bn);
                    }
                    if (two) {
                        if (!(ok = wait(&bars.p_full[1], gp[1] & 1, abort_flag))) break;
                        ++gp[1];
                        tc::fence_after();
                        values(1, b, st == st0);
                    }
                    done(&bars.v_empty[b]);
                    if (more) {
                        if (two) scores(1, bn);
                        done(&bars.k_empty[bn]);
                    }
                }
                done(&bars.o_full);
                if (!ok) {
                    // the products in flight end by themselves: give them a bounded wait before the CTA exits
                    for (uint32_t i = 0; i < kSpinLimit && !mbar_try_wait(&bars.o_full, n_item & 1); ++i) {}
                    *abort_flag = 1;
                    if (lane == 0) set_error(p.ctrl, MOE_ERR_TIMEOUT);
                    break;
                }
                u = it.first + st1;
                if (u >= u_end) break;
            }
        }
    }
    __syncwarp();
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    if (warp == kWMma) tc::dealloc(tmem, 512);
}

template <int D>
cudaError_t launch_one(const Attn &p, int *grid_out, cudaStream_t s) {
    const void *fn = reinterpret_cast<const void *>(kv4_prompt_kernel<D>);
    // The register split takes what the launch reserves: it must be the whole of it.
    static const bool split_ok = [fn] {
        cudaFuncAttributes a;
        return cudaFuncGetAttributes(&a, fn) == cudaSuccess && a.numRegs >= kRegsLaunch;
    }();
    if (!split_ok) return cudaErrorInvalidConfiguration;
    constexpr size_t kBase = PromptCfg<D>::kSmem + 1024;
    const cudaError_t err = set_smem_once(fn, (int)(kBase + sizeof(int) * 4097));
    if (err != cudaSuccess) return err;
    int grid = sm_count();
    if (grid > kMaxPromptCtas) grid = kMaxPromptCtas;
    *grid_out = grid;
    return launch_pdl(kv4_prompt_kernel<D>, dim3((unsigned)grid), kThreads, kBase + sizeof(int) * ((size_t)p.b.B + 1), s, p);
}

}  // namespace

cudaError_t launch_kv4_prompt(const kv4::Attn &p, int *grid, cudaStream_t s) {
    return p.c.D == 64 ? launch_one<64>(p, grid, s) : launch_one<128>(p, grid, s);
}

}  // namespace moe
