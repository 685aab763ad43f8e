// chunk_tc.cu -- attention of chunks of new tokens over the paged cache (bf16, head_dim 128,
// 5th-generation tensor cores).
//
//     out[r] = sum_{t <= L + i} p_t V_t / sum p_t,   p_t = 2^(scale log2(e) q_r . K_t - m_r)
//
// for row i of a sequence, in one pass over its keys. A CTA goes through the tiles of its
// share of the call (chunk.cuh): up to two halves of 128 rows (token, head) against 128 tokens.
// S = Q K^T and O += P V run on the tensor cores, S, P (bf16) and O in tensor memory:
//     columns 0..127 S, 128..191 P of half 0, 192..255 P of half 1, 256 + 128 h.. O of half h.
// One S serves both halves in turn: the softmax warps of a half take it into registers at
// once and give it back, so that the next product never waits for their arithmetic. In the
// steady state one thread issues
//     QK_1(j)  PV_0(j-1)  QK_0(j+1)  PV_1(j-1) ...
// so that a half finds its next scores ready when it is through with a tile. A thread sustains
// N = 128 products at the tensor cores' full rate (64 cycles for M = N = 128, K = 16), so one
// issuing thread is enough; N = 64 takes nearly as long (59), hence 128 tokens to a tile.
//
// Warps: K producer, V producer, the issuer, the planner (which lays out the CTA's parts ahead of the
// others, in a ring in shared memory, and loads their Q), and four softmax warps per half,
// which also write the results. A part of at most 128 rows uses half 0 alone.
//
// The running maximum m moves only when it grows by more than 2^8 (O is rescaled then); sums
// and O are fp32. P is rounded to bf16 for the second product, at most half a step each.
//
// A token that a row does not see has p = 0, but 0 * V is no zero where V holds an infinity or
// a NaN. Rows behind the block's last token are zeroed in shared memory; tokens inside the block can
// only be masked. So a row that comes out with a value that is not finite, and that has masked tokens
// among its tiles, is computed again from its visible tokens alone, by its warp in fp32.
//
// Bound: with few rows a sequence HBM (64 tokens over 32768 each, 64/8 heads: 6.44 GB in 961 us, 6.7
// TB/s, a copy's rate). With many the softmax warps: a tile of 256 rows by 128 tokens takes
// them about 2700 cycles, of which the tensor cores have work for 2048, and a unit's end (the
// last product, O out of tensor memory, the pieces that wait to be joined) 8 to 9 thousand.
// A prompt of 8192 tokens, 32/8 heads: 424 to 433 us, 1280 TFLOP/s of its visible scores (67 %
// of the measured burst rate); 8185 tokens after 24576, 64/8 heads: 4.9 to 5.4 ms (75 to 82 %), where the
// power limit lowers the clock. One token over 2049: 21.5 us, all of it latency (layout 3.5, first
// page numbers and K 2.2, tile 2, pieces 1.5, join 6).
// Registers: 384 threads start with 168 each; the four warps of the first group keep 56 and the softmax
// warps take 224 (128 x 56 + 256 x 224 is the launch's total). A thread holds a row of 128
// scores; at 208 registers they spill and the long case takes 18 % more.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <math.h>

#include "attn_tc_common.cuh"
#include "chunk.cuh"

namespace svf {

namespace {

namespace ct {
constexpr int BN = 128;                  // tokens per tile
constexpr int HD = 128;                  // head_dim
constexpr int COL = 128 * 128;           // one 64-dim block of 128 rows (bytes)
constexpr int TILE = 2 * COL;            // 128 rows of Q, K or V
constexpr int KS = 2, VS = 3;            // ring stages
constexpr int NR = 4;                    // parts in the planner's ring
constexpr int NT = 384;
constexpr int SW0 = 4;                   // first softmax warp
constexpr uint32_t tS = 0, tP = 128, tO = 256;
constexpr unsigned long long kLongWaitNs = 60000000000ull;  // waits as long as a part may take
constexpr int kBarBoth = 1, kBarHalf = 2;  // named barriers: all softmax warps, half 0's
}  // namespace ct

struct TcPart {
    int b, head, row, tok0, ntok;  // row: q row of the block's first token
    int L;
    int x0, n, t;                  // first tile, tiles of the part, tiles of the unit
    int cf, cl, slot;              // groups that share the unit; this part's place in the workspace
    int first_slot;                // piece 0's: 1 if the unit is not the first of its group
    int two;                       // both halves have rows
    int bad;                       // first token whose page is not in the cache
    int clear;                     // the last tile reaches behind the block's last token
};

struct TcSmem {
    static constexpr int kQ = 0;
    static constexpr int kK = kQ + 2 * ct::TILE;
    static constexpr int kV = kK + ct::KS * ct::TILE;
    static constexpr int kBar = kV + ct::VS * ct::TILE;
    static constexpr int kNumBars = 2 * ct::KS + 2 * ct::VS + 2 * ct::NR + 3 + 4 * 2 + ct::VS + 1;
    static constexpr int kMisc = kBar + ((kNumBars * 8 + 127) / 128) * 128;
    static constexpr int kSpace = kMisc + 64;
    static constexpr int kParts = kSpace + 64;
    static constexpr int kJoin = kParts + ct::NR * (int)sizeof(TcPart);
    static constexpr int kBytes = kJoin + 256 * 4;
    static constexpr int kDynamic = kBytes + 1024;  // slack to align the base to 1 KB
    static_assert(sizeof(ChunkSpace) <= 64, "space");
    static_assert(kDynamic <= 227 * 1024, "shared memory budget");
};

__device__ __forceinline__ int bar_or(int id, int n, int pred) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.s32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, %2, %3, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(pred), "r"(id), "r"(n)
        : "memory");
    return (int)r;
}

// Products with the operands' descriptors as their low words (start address and leading offset; the
// high word is the same for all: 1024 bytes between groups of eight rows, 128-byte swizzle):
// the issuer has no register to spare either.
constexpr uint32_t kDescHigh = (1024 >> 4) | 1u << 14 | 2u << 29;
__device__ __forceinline__ uint32_t desc_low(uint32_t start, uint32_t lbo) {
    return start >> 4 | (lbo >> 4) << 16;
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "mov.b64 a, {%1, %5};\n\tmov.b64 b, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(acc), "r"(kDescHigh)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "mov.b64 b, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(acc), "r"(kDescHigh)
        : "memory");
}

// Barriers by their 32-bit addresses: the softmax warps have no register to spare.
__device__ __forceinline__ bool try_wait_at(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ bool test_wait_at(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ void arrive_at(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
// A warp's wait, as mbar_wait_for; the clock is read in units of 1.024 us, in 32 bits.
__device__ __forceinline__ bool warp_wait_at(uint32_t bar, uint32_t parity, volatile int *abort,
                                             unsigned long long ns) {
    if (__all_sync(0xffffffffu, test_wait_at(bar, parity))) return true;
    const bool quick = ns < 1000000ull;
    const uint32_t t0 = (uint32_t)(globaltimer_ns() >> 10), limit = (uint32_t)(ns >> 10);
    for (uint32_t it = 1;; ++it) {
        const bool ok = quick ? test_wait_at(bar, parity) : try_wait_at(bar, parity);
        if (__all_sync(0xffffffffu, ok)) return true;
        if (quick || (it & 63u) == 0) {
            if ((uint32_t)(globaltimer_ns() >> 10) - t0 > limit) *abort = 1;
            if (__any_sync(0xffffffffu, *abort)) return false;
        }
    }
}

// A wait of the roles that need few registers.
__device__ __forceinline__ bool role_wait(uint64_t *bar, uint32_t parity, volatile int *abort,
                                          unsigned long long ns) {
    return mbar_wait_for(bar, parity, abort, ns);
}

// Eight floats (as bits) as bf16.
__device__ __forceinline__ uint4 eight_bf16(const uint32_t *o) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = pack_bf16x2(__uint_as_float(o[2 * i]), __uint_as_float(o[2 * i + 1]));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// 32 bytes in one store: a lane of a warp that writes a row each fills whole sectors.
__device__ __forceinline__ void store32(void *p, uint4 a, uint4 b) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(a.x),
                 "r"(a.y), "r"(a.z), "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
                 : "memory");
}

__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(p));
    return p != 0;
}

template <int N>
__device__ __forceinline__ void regs_dec() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_inc() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// The row of a part again, from its visible tokens in [t0, t1) alone, by a warp: 4 of the head's
// elements per lane. Sums in fp32; returns the normalised elements and the log2-sum-exp.
__device__ __noinline__ float4 row_again(const ChunkParams &p, int b, int head, size_t qrow, int t0,
                                         int t1, float *lse2) {
    const int lane = threadIdx.x & 31;
    auto four = [&](const void *base, size_t row) {
        const uint2 w = __ldg(reinterpret_cast<const uint2 *>(
                                  static_cast<const __nv_bfloat16 *>(base) + row * ct::HD) + lane);
        return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u),
                           __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u));
    };
    const float4 q = four(p.q, qrow);
    const int32_t *table = p.page_table + (size_t)b * p.max_pages;
    float m = -INFINITY, l = 0.0f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int t = t0; t < t1; ++t) {
        const int id = __ldg(table + t / p.ps);
        float4 k = make_float4(0.f, 0.f, 0.f, 0.f), v = k;
        if (id >= 0 && id < p.num_pages) {
            const size_t at = ((size_t)id * p.ps + t % p.ps) * p.Hkv + head;
            k = four(p.k_cache, at);
            v = four(p.v_cache, at);
        }
        const float s = warp_sum(fmaf(q.x, k.x, fmaf(q.y, k.y, fmaf(q.z, k.z, q.w * k.w)))) *
                        p.scale_log2;
        const float nm = fmaxf(m, s);
        const float base = nm == -INFINITY ? 0.0f : nm;
        const float a = ex2_approx(m - base), e = ex2_approx(s - base);
        m = nm;
        l = fmaf(l, a, e);
        o.x = fmaf(e, v.x, o.x * a);
        o.y = fmaf(e, v.y, o.y * a);
        o.z = fmaf(e, v.z, o.z * a);
        o.w = fmaf(e, v.w, o.w * a);
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    *lse2 = l == 0.0f ? -INFINITY : m + __log2f(l);
    return make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
}

// The thread that fills the ring of K or of V.
struct Producer {
    const CUtensorMap *map;
    uint8_t *ring;
    uint64_t *full, *empty;
    int stages, st, issued;
    uint32_t ph;  // parity of the stage's last release; the first round passes
    unsigned long long ns;
    volatile int *abort;
    bool ok;
};

// The tiles of a part, each in boxes of a page (at most 128 tokens). Page-table entries are read a
// tile ahead. `bad` gets the first token of the part whose page is not in the cache.
__device__ __forceinline__ void load_part(const ChunkParams &p, Producer &w, const TcPart &pt, int *bad) {
    using namespace ct;
    constexpr int MAXB = BN / 16;
    const int n = pt.n, x0 = pt.x0, head = pt.head, end = pt.L + pt.tok0 + pt.ntok, ps = p.ps;
    const int box = ps < BN ? ps : BN, bpt = BN / box;
    const int32_t *table = p.page_table + (size_t)pt.b * p.max_pages;
    const int oob = p.num_pages * ps;  // a slot past the cache: TMA fills zeros
    // slots of tile x's boxes
    auto fetch = [&](int x, int *slot) {
        const unsigned t0 = (unsigned)(x0 + x) * BN;
        const unsigned page = bpt > 1 ? (unsigned)(x0 + x) * bpt : t0 / (unsigned)ps;
        const int off = bpt > 1 ? 0 : (int)(t0 - page * (unsigned)ps);
#pragma unroll
        for (int i = 0; i < MAXB; ++i) {
            slot[i] = oob;
            if (i < bpt && x < n && t0 + i * box < (unsigned)end) {
                const int id = __ldg(table + page + i);
                if (id >= 0 && id < p.num_pages) slot[i] = id * ps + off;
                else if (bad) atomicMin(bad, (int)(t0 + i * box));
            }
        }
    };
    int slot[MAXB], next[MAXB];
    fetch(0, slot);
    for (int j = 0; w.ok && j < n; ++j) {
        fetch(j + 1, next);
        if (!(w.ok = mbar_wait_for(&w.empty[w.st], w.ph, w.abort, w.ns))) break;
        uint64_t *full = &w.full[w.st];
        uint8_t *stage = w.ring + w.st * TILE;
        mbar_arrive_expect_tx(full, TILE);
#pragma unroll
        for (int i = 0; i < MAXB; ++i) {
            if (i < bpt) {
                tma_load_3d(stage + i * box * 128, w.map, 0, head, slot[i], full);
                tma_load_3d(stage + COL + i * box * 128, w.map, 64, head, slot[i], full);
            }
            slot[i] = next[i];
        }
        ++w.issued;
        if (++w.st == w.stages) {
            w.st = 0;
            w.ph ^= 1;
        }
    }
}

__global__ void __launch_bounds__(ct::NT, 1)
    chunk_tc_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
                    const __grid_constant__ CUtensorMap tmq, ChunkParams p) {
    using namespace ct;
    using S = TcSmem;
    constexpr unsigned FULL = 0xffffffffu;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint8_t *sQ = smem + S::kQ, *sK = smem + S::kK, *sV = smem + S::kV;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + S::kBar);
    uint64_t *k_full = bars, *k_empty = k_full + KS;
    uint64_t *v_full = k_empty + KS, *v_empty = v_full + VS;
    uint64_t *part_full = v_empty + VS;       // [NR] the planner wrote the part
    uint64_t *part_empty = part_full + NR;    // [NR] everybody is through with it
    uint64_t *q_full = part_empty + NR;       // the part's Q landed
    uint64_t *q_free = q_full + 1;            // its products are done: Q may be replaced
    uint64_t *s_free = q_free + 1;            // S was taken into registers
    uint64_t *s_full = s_free + 1;            // [2] Q K^T of the half is in S
    uint64_t *p_full = s_full + 2;            // [2] P of the half is written
    uint64_t *o_done = p_full + 2;            // [2] P V of the half is done
    uint64_t *o_free = o_done + 2;            // [2] O of the half was read out
    uint64_t *v_clear = o_free + 2;           // [VS] rows of the stage behind a block's last token are cleared
    uint64_t *drain = v_clear + VS;           // the issuer's products done, after an abort
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + S::kMisc);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + S::kMisc + 4);
    int *s_last = reinterpret_cast<int *>(smem + S::kMisc + 8);
    ChunkSpace *space = reinterpret_cast<ChunkSpace *>(smem + S::kSpace);
    TcPart *parts = reinterpret_cast<TcPart *>(smem + S::kParts);
    float *join = reinterpret_cast<float *>(smem + S::kJoin);  // [256] the rows' joined log2-sum-exp

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int hl = blockIdx.x % p.S;  // this CTA's head of a head block

    if (threadIdx.x == 0) {
        for (int i = 0; i < KS; ++i) {
            mbar_init(&k_full[i], 1);
            mbar_init(&k_empty[i], 1);
        }
        for (int i = 0; i < VS; ++i) {
            mbar_init(&v_full[i], 1);
            mbar_init(&v_empty[i], 1);
            mbar_init(&v_clear[i], 1);
        }
        for (int i = 0; i < NR; ++i) {
            mbar_init(&part_full[i], 1);
            mbar_init(&part_empty[i], 3 + 8);
        }
        mbar_init(q_full, 1);
        mbar_init(q_free, 1);
        mbar_init(s_free, 128);
        for (int h = 0; h < 2; ++h) {
            mbar_init(&s_full[h], 1);
            mbar_init(&p_full[h], 128);
            mbar_init(&o_done[h], 1);
            mbar_init(&o_free[h], 128);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        mbar_fence_init();
    }
    if (warp == 1 && lane == 0) {
        tma_prefetch_desc(&tmk);
        tma_prefetch_desc(&tmv);
        tma_prefetch_desc(&tmq);
    }
    if (warp == 2) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    const uint32_t tmem = *tmem_slot;
    tc_fence_after();
    pdl_wait();
    pdl_launch_dependents();
    if (p.B > kChunkWarpBatch) chunk_layout<BN, NT>(p, space, reinterpret_cast<ChunkCount *>(join));

    // Waits of the ring of parts: they go on after an abort, when every role still goes through
    // the parts (without work), so that the pieces of split units are all counted.
    volatile int never = 0;
    auto ring_wait = [&](uint64_t *bar, int use) {
        return __all_sync(FULL, mbar_wait_for(bar, (uint32_t)(use & 1), &never, kLongWaitNs));
    };
    const unsigned long long long_ns = p.wait_ns < kWaitDeadlineNs ? p.wait_ns : kLongWaitNs;

    if (warp < SW0) {
        regs_dec<56>();
        auto role_ring_wait = [&](uint64_t *bar, int use) {
            return __all_sync(FULL, role_wait(bar, (uint32_t)(use & 1), &never, kLongWaitNs));
        };
        auto role_wait_long = [&](uint64_t *bar, uint32_t parity) {
            return __all_sync(FULL, role_wait(bar, parity, abort_flag, long_ns));
        };
        if (warp <= 1) {
            // -------------------------------------------------------- producers of K and V
            // one elected thread each, as for the issuer: a box takes a third of what it
            // takes a lane of several
            if (elect_one()) {
                const bool is_k = warp == 0;
                Producer w = {is_k ? &tmk : &tmv, is_k ? sK : sV, is_k ? k_full : v_full,
                              is_k ? k_empty : v_empty, is_k ? KS : VS, 0, 0, 1u, long_ns, abort_flag, true};
                for (int i = 0; role_wait(&part_full[i % NR], (uint32_t)(i / NR & 1), &never, kLongWaitNs);
                     ++i) {
                    TcPart *pt = &parts[i % NR];
                    if (pt->n == 0) break;
                    load_part(p, w, *pt, is_k ? &pt->bad : nullptr);
                    mbar_arrive(&part_empty[i % NR]);
                }
                // never leave with copies in flight: the last fill of every stage
                for (int s = 0; s < w.stages && s < w.issued; ++s)
                    role_wait(&w.full[s], (uint32_t)(((w.issued - 1 - s) / w.stages) & 1), &never,
                                  kWaitDeadlineNs);
            }
            __syncwarp();
        } else if (warp == 2) {
            // -------------------------------------------------------- the issuer
            // one elected thread: the compiler sees that it is alone and issues a product in
            // 64 cycles (under `lane == 0` each takes about 100, whatever its size)
            if (elect_one()) {
                constexpr uint32_t idesc_qk = idesc_bf16_f32(128, BN, false, false);
                constexpr uint32_t idesc_pv = idesc_bf16_f32(128, HD, false, true);
                const uint32_t dQ = desc_low(smem_u32(sQ), 16), dK = desc_low(smem_u32(sK), 16);
                const uint32_t dV = desc_low(smem_u32(sV), COL);
                uint32_t ks = 0, vs = 0;              // stages of the next QK and the next PV
                uint32_t kph = 0, vph = 0, sph = 1;
                uint32_t zph = 0;                // bit s: parity of the stage's next clearing
                uint32_t pph = 0;
                uint32_t oph = 3;     // bit h: the half had a part; parity of O's release
                bool ok = true;
                auto one = [&](uint64_t *bar, uint32_t parity) {
                    return role_wait(bar, parity, abort_flag, long_ns);
                };
            // S = Q_h K^T of the tile in K's stage ks, once S was taken
            auto issue_qk = [&](const uint32_t h, bool last_of_tile, bool last_of_part) {
                if (!(ok = ok && one(s_free, sph))) return;
                sph ^= 1;
                tc_fence_after();
                const uint32_t q = dQ + h * (TILE >> 4), k = dK + ks * (TILE >> 4);
#pragma unroll
                for (int kk = 0; kk < 8; ++kk) {
                    const uint32_t o = ((kk >> 2) * COL + (kk & 3) * 32) >> 4;
                    mma_ss(tmem + tS, q + o, k + o, idesc_qk, kk > 0);
                }
                umma_commit(&s_full[h]);
                if (last_of_tile) {
                    umma_commit(&k_empty[ks]);
                    if (last_of_part) umma_commit(q_free);
                    if (++ks == KS) {
                        ks = 0;
                        kph ^= 1;
                    }
                }
            };
            // O_h (+)= P_h V of the tile in V's stage vs, once P is written; `cleared`: once the
            // rows behind the block's end are cleared too
            auto issue_pv = [&](const uint32_t h, bool first, bool last_of_tile, bool cleared, bool last) {
                if (h == 0) {
                    if (!(ok = ok && one(&v_full[vs], vph))) return;
                    if (cleared) {
                        if (!(ok = one(&v_clear[vs], zph >> vs & 1))) return;
                        zph ^= 1u << vs;
                    }
                }
                if (first) {  // O of the half's last part was read out
                    if (!(ok = ok && one(&o_free[h], oph >> h & 1))) return;
                    oph ^= 1u << h;
                }
                // (the half gave back S of its next tile after it wrote P)
                if (!(ok = ok && (!last || one(&p_full[h], pph >> h & 1)))) return;
                pph ^= 1u << h;
                tc_fence_after();
                const uint32_t d = tmem + tO + h * 128, a = tmem + tP + h * 64;
                const uint32_t v = dV + vs * (TILE >> 4);
                mma_ts(d, a, v, idesc_pv, first ? 0u : 1u);
#pragma unroll
                for (int kk = 1; kk < 8; ++kk)
                    mma_ts(d, a + kk * 8, v + (kk * 2048 >> 4), idesc_pv, 1u);
                umma_commit(&o_done[h]);
                if (last_of_tile) {
                    umma_commit(&v_empty[vs]);
                    if (++vs == VS) {
                        vs = 0;
                        vph ^= 1;
                    }
                }
            };
            for (int i = 0; role_wait(&part_full[i % NR], (uint32_t)(i / NR & 1), &never, kLongWaitNs); ++i) {
                const int n = parts[i % NR].n, two = parts[i % NR].two;
                const bool clear = parts[i % NR].clear;
                if (n == 0) break;
                mbar_arrive(&part_empty[i % NR]);
                if (!(ok = ok && one(q_full, (uint32_t)(i & 1)))) continue;
                // A half that takes its next S has written P: the PV of that tile follows, behind
                // the other half's next product.
                if (two) {
                    ok = one(&k_full[ks], kph);
                    issue_qk(0, false, false);
                    for (int j = 0; ok && j < n; ++j) {
                        issue_qk(1, true, j == n - 1);
                        if (j > 0) issue_pv(0, j == 1, false, false, false);
                        if (j + 1 < n) {
                            ok = ok && one(&k_full[ks], kph);
                            issue_qk(0, false, false);
                        }
                        if (j > 0) issue_pv(1, j == 1, true, false, j + 1 == n);
                    }
                    issue_pv(0, n == 1, false, clear, true);
                    issue_pv(1, n == 1, true, false, true);
                } else {
                    for (int j = 0; ok && j < n + 2; ++j) {
                        if (j < n) {
                            ok = one(&k_full[ks], kph);
                            issue_qk(0, true, j == n - 1);
                        }
                        if (j > 1) issue_pv(0, j == 2, true, clear && j == n + 1, j >= n);
                    }
                }
            }
            }
            __syncwarp();
        } else {
            // -------------------------------------------------------- the planner
            // a batch that one warp can lay out the others need not wait for
            const ChunkSpace sp = p.B > kChunkWarpBatch ? *space : chunk_layout_warp<BN>(p, lane);
            if (lane == 0 && p.B <= kChunkWarpBatch) *space = sp;
            ChunkSeg g;
            // (a part that ends in its unit's lead has no tiles and is none)
            auto with_tiles = [&](bool more) {
                int first;
                while (more && chunk_part(sp, g, first) == 0) more = chunk_next<BN>(p, sp, g);
                return more;
            };
            bool more = with_tiles(chunk_first<BN>(p, sp, g)), ended = false, ok = true;
            int posted = 0, loaded = 0, q_loads = 0, tiles = 0;
            // The rows of V behind the last token of a part, whose last tile is the tiles-th: up
            // to the end of their page they may hold anything. Called when the part's QKs
            // are done: then the softmax has taken the scores of the tile before, after the PV
            // of the tile VS before the last, so v_full's phase is that tile's or the last's.
            auto clear = [&](const TcPart *pt) {
                tiles += pt->n;
                if (!pt->clear) return;
                const int vs = (tiles - 1) % VS, use = (tiles - 1) / VS;
                if (ok && (ok = role_wait_long(&v_full[vs], (uint32_t)(use & 1)))) {
                    const int ps = p.ps, box = ps < BN ? ps : BN;
                    const int r0 = (int)((long long)pt->L + pt->tok0 + pt->ntok - (long long)(pt->t - 1) * BN);
                    const int r1 = (r0 + box - 1) / box * box;
                    uint8_t *vsm = sV + vs * TILE;
                    for (int i = r0 * 16 + lane; i < r1 * 16; i += 32)
                        *reinterpret_cast<uint4 *>(vsm + ((i & 15) >> 3) * COL + (i >> 4) * 128 +
                                                   (i & 7) * 16) = make_uint4(0, 0, 0, 0);
                    fence_proxy_async_smem();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&v_clear[vs]);
            };
            for (;;) {
                while (!ended && posted < loaded + NR - 1) {
                    TcPart *pt = &parts[posted % NR];
                    if (posted >= NR && !role_ring_wait(&part_empty[posted % NR], posted / NR - 1)) {
                        ended = true;
                        break;
                    }
                    if (lane == 0) {
                        TcPart w = {};
                        if (more) {
                            w.b = g.b;
                            w.head = g.hb * p.S + hl;
                            w.tok0 = g.k * p.TB;
                            w.row = g.row0 + w.tok0;
                            w.ntok = min(p.TB, g.n - w.tok0);
                            w.L = g.L;
                            w.n = chunk_part(sp, g, w.x0);
                            w.t = g.t;
                            chunk_groups(sp, g, w.cf, w.cl);
                            w.slot = 2 * blockIdx.x + (g.x0 == sp.s ? 0 : 1);
                            w.first_slot = chunk_start(w.cf, sp.T, sp.C) < g.pu ? 1 : 0;
                            w.two = w.ntok > p.TB / 2;
                            w.bad = kPieceFine;
                            w.clear = w.x0 + w.n == w.t &&
                                      (long long)w.t * BN > (long long)w.L + w.tok0 + w.ntok;
                        }
                        *pt = w;
                        mbar_arrive(&part_full[posted % NR]);
                    }
                    __syncwarp();
                    ++posted;
                    if (!more) ended = true;
                    else more = with_tiles(chunk_next<BN>(p, sp, g));
                }
                if (loaded >= posted - (ended ? 1 : 0)) break;
                const TcPart *pt = &parts[loaded % NR];
                if (ok && loaded > 0) ok = role_wait_long(q_free, (uint32_t)((loaded - 1) & 1));
                if (ok && lane == 0) {
                    const int half = p.TB / 2;
                    mbar_arrive_expect_tx(q_full, (pt->two ? 2u : 1u) * 2u * 128u * (uint32_t)(half * p.G));
                    for (int h = 0; h <= pt->two; ++h)
#pragma unroll
                        for (int dh = 0; dh < 2; ++dh)
                            tma_load_3d(sQ + h * TILE + dh * COL, &tmq, dh * 64, pt->head * p.G,
                                        pt->row + h * half, q_full);
                }
                __syncwarp();
                q_loads += ok;
                // (the part before is still in the ring: at most NR - 1 are ahead of it)
                if (loaded > 0) clear(&parts[(loaded - 1) % NR]);
                ++loaded;
            }
            if (loaded > 0) {
                if (ok) ok = role_wait_long(q_free, (uint32_t)((loaded - 1) & 1));
                clear(&parts[(loaded - 1) % NR]);
            }
            // (after an abort nobody may have waited for the last Q)
            if (q_loads > 0 && lane == 0)
                role_wait(q_full, (uint32_t)((q_loads - 1) & 1), &never, kWaitDeadlineNs);
            __syncwarp();
        }
    } else {
        regs_inc<224>();
        // ------------------------------------------------------------ softmax
        const int h = (warp - SW0) >> 2, quarter = warp & 3;
        const int r = quarter * 32 + lane;           // row of the half
        const int st = threadIdx.x - 32 * SW0;       // 0 .. 255
        const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
        const uint32_t aS = tmem + lane_off + tS, aP = tmem + lane_off + tP + h * 64;
        const uint32_t aO = tmem + lane_off + tO + h * 128;
        const float sl2 = p.scale_log2;
        const int half_tok = p.TB / 2, half_rows = half_tok * p.G;
        __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(p.out);
        const bool wide_out = (reinterpret_cast<uintptr_t>(p.out) & 31) == 0;
        const int tok = h * half_tok + r / p.G;      // token of the row in its block
        // the half's barriers
        const uint32_t bH = smem_u32(bars) + h * 8;
        constexpr int kSFree = (2 * KS + 2 * VS + 2 * NR + 2) * 8, kSFull = kSFree + 8,
                      kPFull = kSFull + 16, kODone = kPFull + 16;
        auto wait_at = [&](uint32_t bar, uint32_t parity) {
            return warp_wait_at(bar, parity, abort_flag, p.wait_ns);
        };

        chunk_status<HD, __nv_bfloat16>(p, st, 256,
                                        [&](bool v) { return bar_or(kBarBoth, 256, v) != 0; });

        bool ok = true;
        int cnt = 0;    // tiles of this half so far
        for (int i = 0; ring_wait(&part_full[i % NR], i / NR); ++i) {
            const volatile TcPart *pt = &parts[i % NR];
            const int n = pt->n;
            if (n == 0) break;
            const int two = pt->two;
            if (h == 1 && !two) {
                __syncwarp();
                if (lane == 0) mbar_arrive(&part_empty[i % NR]);
                continue;
            }
            // (what the tiles do not need is read again behind them)
            const bool live = __any_sync(FULL, r < half_rows && tok < pt->ntok);
            // columns of the part up to it are visible (rows of padding see them all)
            int lim = r < half_rows && tok < pt->ntok ? pt->L + pt->tok0 + tok - pt->x0 * BN : 0x7fffffff;
            float m_ref = -INFINITY, l = 0.0f;
            for (int jl = 0; ok && jl < n; ++jl, ++cnt, lim -= BN) {
                if (!(ok = wait_at(bH + kSFull, (uint32_t)(cnt & 1)))) break;
                if (!live) {  // padding of the half: its rows are not looked at
                    arrive_at(bH - h * 8 + kSFree);
                    if (cnt > 0 && !(ok = wait_at(bH + kODone, (uint32_t)((cnt - 1) & 1)))) break;
                    arrive_at(bH + kPFull);
                    continue;
                }
                tc_fence_after();
                uint32_t v[BN];
                tmem_ld32(aS, v);
                tmem_ld32(aS + 32, v + 32);
                tmem_ld32(aS + 64, v + 64);
                tmem_ld32(aS + 96, v + 96);
                tmem_wait_ld();
                tc_fence_before();
                arrive_at(bH - h * 8 + kSFree);
                if (__any_sync(FULL, lim < BN - 1)) {
#pragma unroll
                    for (int c = 0; c < BN; ++c) v[c] = c <= lim ? v[c] : 0xff800000u;
                }
                float m0 = -INFINITY, m1 = -INFINITY, m2 = -INFINITY, m3 = -INFINITY;
#pragma unroll
                for (int c = 0; c < BN; c += 8) {
                    m0 = fmax3(m0, __uint_as_float(v[c]), __uint_as_float(v[c + 1]));
                    m1 = fmax3(m1, __uint_as_float(v[c + 2]), __uint_as_float(v[c + 3]));
                    m2 = fmax3(m2, __uint_as_float(v[c + 4]), __uint_as_float(v[c + 5]));
                    m3 = fmax3(m3, __uint_as_float(v[c + 6]), __uint_as_float(v[c + 7]));
                }
                const float mx = fmax3(m0, m1, fmaxf(m2, m3)) * sl2;
                // lazy rescale: move the reference only when the maximum grows by > 2^8
                const bool need = mx > m_ref + tc::kRescaleThreshold;
                const float alpha = need ? ex2_approx(m_ref - mx) : 1.0f;
                if (need) {
                    l *= alpha;
                    m_ref = mx;
                }
                const float mneg = m_ref == -INFINITY ? 0.0f : -m_ref;
                const float2 sc2 = make_float2(sl2, sl2), mn2 = make_float2(mneg, mneg);
                float2 rs = make_float2(0.0f, 0.0f);
#pragma unroll
                for (int c = 0; c < BN / 2; ++c) {  // P takes the place of S
                    const float2 y = ffma2(make_float2(__uint_as_float(v[2 * c]),
                                                       __uint_as_float(v[2 * c + 1])), sc2, mn2);
                    const float2 pp = make_float2(ex2_approx(y.x), ex2_approx(y.y));
                    rs = fadd2(rs, pp);
                    v[c] = pack_bf16x2(pp.x, pp.y);
                }
                l += rs.x + rs.y;
                // P of the tile before was read, O is final up to it
                if (cnt > 0 && !(ok = wait_at(bH + kODone, (uint32_t)((cnt - 1) & 1)))) break;
                if (jl > 0 && __any_sync(FULL, need)) {
                    tc_fence_after();
#pragma unroll 1
                    for (int c = 0; c < 8; ++c) {
                        uint32_t o[16];
                        tmem_ld16(aO + c * 16, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                        tmem_st16(aO + c * 16, o);
                    }
                }
                tmem_st16(aP, v);
                tmem_st16(aP + 16, v + 16);
                tmem_st16(aP + 32, v + 32);
                tmem_st16(aP + 48, v + 48);
                tmem_wait_st();
                tc_fence_before();
                arrive_at(bH + kPFull);
            }
            // ---- the end of the part: O after its last PV
            if (ok) ok = wait_at(bH + kODone, (uint32_t)((cnt - 1) & 1));
            tc_fence_after();
            const int L = pt->L, x0 = pt->x0, tok0 = pt->tok0, ntok = pt->ntok;
            const bool row_valid = r < half_rows && tok < ntok;
            const int see = row_valid ? L + tok0 + tok : 0x7fffffff;
            const int head = pt->head, cf = pt->cf, cl = pt->cl, slot = pt->slot;
            const int first_slot = pt->first_slot, bad = pt->bad, b = pt->b, qrow0 = pt->row;
            const bool split = cf != cl;
            const float inv = l == 0.0f ? 0.0f : 1.0f / l;
            const float ls = l == 0.0f ? -INFINITY : m_ref + __log2f(l);
            const size_t row = ((size_t)(qrow0 + tok)) * p.Hq + (size_t)head * p.G + r % p.G;
            const int lr = h * 128 + r;
            // tokens of this part that the row does not see?
            const int seen_to = (int)min((long long)(x0 + n) * BN, (long long)L + tok0 + ntok);
            const bool masked = row_valid && seen_to > see + 1;
            float odd = 0.0f;  // NaN if the row holds a value that is not finite
            if (!split) {
                const bool zero = !ok || see >= bad;
#pragma unroll 1
                for (int c64 = 0; c64 < 2; ++c64) {
                    uint32_t o[64];
                    if (ok) {
                        tmem_ld32(aO + c64 * 64, o);
                        tmem_ld32(aO + c64 * 64 + 32, o + 32);
                        tmem_wait_ld();
                    }
                    if (zero) {
#pragma unroll
                        for (int e = 0; e < 64; ++e) o[e] = 0;
                    }
                    if (row_valid) {
#pragma unroll
                        for (int e = 0; e < 64; ++e) {
                            odd = fmaf(__uint_as_float(o[e]), 0.0f, odd);
                            o[e] = __float_as_uint(__uint_as_float(o[e]) * inv);
                        }
                        __nv_bfloat16 *op = out + row * HD + c64 * 64;
                        if (wide_out) {
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                store32(op + 16 * k, eight_bf16(o + 16 * k), eight_bf16(o + 16 * k + 8));
                        } else {
#pragma unroll
                            for (int k = 0; k < 8; ++k)
                                reinterpret_cast<uint4 *>(op)[k] = eight_bf16(o + 8 * k);
                        }
                    }
                }
                if (row_valid && p.lse) p.lse[row] = zero ? 0.0f : ls * 0.69314718055994531f;
            } else {
                float4 *dst = p.part + (size_t)slot * (HD / 4) * p.slot_rows;
#pragma unroll 1
                for (int c32 = 0; c32 < 4; ++c32) {
                    uint32_t o[32];
                    if (ok) {
                        tmem_ld32(aO + c32 * 32, o);
                        tmem_wait_ld();
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = 0;
                    }
                    if (row_valid) {
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            float f[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                f[e] = __uint_as_float(o[4 * k + e]);
                                odd = fmaf(f[e], 0.0f, odd);
                                f[e] *= inv;
                            }
                            __stcg(dst + (size_t)(c32 * 8 + k) * p.slot_rows + lr,
                                   make_float4(f[0], f[1], f[2], f[3]));
                        }
                    }
                }
                if (row_valid) __stcg(p.part_lse + (size_t)slot * p.slot_rows + lr, ok ? ls : -INFINITY);
            }
            // O may restart
            tc_fence_before();
            mbar_arrive(&o_free[h]);
            // rows that a masked token may have reached: again, without it
            unsigned again = __ballot_sync(FULL, ok && masked && odd != 0.0f && see < bad);
            __syncwarp();
            while (again) {
                const int rl = __ffs(again) - 1;
                again &= again - 1;
                const size_t at = __shfl_sync(FULL, (unsigned long long)row, rl);
                const int last = __shfl_sync(FULL, see, rl);
                float lse2;
                const float4 o = row_again(p, b, head, at, x0 * BN, min(seen_to, last + 1), &lse2);
                if (!split) {
                    *reinterpret_cast<uint2 *>(out + at * HD + lane * 4) =
                        make_uint2(pack_bf16x2(o.x, o.y), pack_bf16x2(o.z, o.w));
                    if (lane == 0 && p.lse) p.lse[at] = lse2 * 0.69314718055994531f;
                } else {
                    const int lr2 = h * 128 + quarter * 32 + rl;
                    __stcg(p.part + ((size_t)slot * (HD / 4) + lane) * p.slot_rows + lr2, o);
                    if (lane == 0) __stcg(p.part_lse + (size_t)slot * p.slot_rows + lr2, lse2);
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&part_empty[i % NR]);
            if (!split) continue;
            // ---- a piece: count it, and join the unit's pieces if it was the last
            const int nthr = two ? 256 : 128, id = two ? kBarBoth : kBarHalf;
            const int F = cl - cf + 1;
            if (r == 0) __stcg(p.part_bad + 2 * slot + h, ok ? bad : kPieceLost);
            bar_or(id, nthr, 0);
            if (st == 0) {
                __threadfence();  // what the barrier made visible to this thread, too
                int *counter = p.counters + cf * p.S + hl;
                const int before = atomicAdd(counter, 1);
                if (before == F - 1) *counter = 0;
                *s_last = before == F - 1;
                __threadfence();
            }
            if (!bar_or(id, nthr, st == 0 && *s_last)) continue;
            const ChunkJoin jn = {F, cf, hl, first_slot, ntok * p.G, half_rows, 1 + two,
                                  qrow0, head, L + tok0, st, nthr, id};
            chunk_join<HD, __nv_bfloat16>(p, jn, join);
        }
    }

    tc_fence_before();
    __syncthreads();
    if (*abort_flag) {
        // Some role gave up, the issuer perhaps through before: its products finish before tensor
        // memory and shared memory go. (elect.sync elects the same thread each time, the one
        // that issued them.)
        if (warp == 2 && elect_one()) {
            umma_commit(drain);
            mbar_wait_for(drain, 0, &never, kWaitDeadlineNs);
        }
        __syncwarp();
        tc_fence_before();
        __syncthreads();
    }
    if (warp == 2) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
    // ---- CTAs that gave up: the last CTA of the call, to which every status word is visible,
    // adds the bit for the sequences they had tiles of
    if (threadIdx.x == 0) {
        if (*abort_flag && space->s < space->e) {
            ChunkSeg g;
            chunk_first<BN>(p, *space, g);
            const int b0 = g.b;
            while (chunk_next<BN>(p, *space, g)) {}
            p.gave_up[2 * blockIdx.x] = b0;
            p.gave_up[2 * blockIdx.x + 1] = g.b < p.B ? g.b : p.B - 1;
            atomicOr(p.done + 2 + blockIdx.x / 32, 1 << (blockIdx.x & 31));
            atomicOr(p.done + 1, 1);
        }
        __threadfence();
        if (atomicAdd(p.done, 1) == (int)gridDim.x - 1) {
            __threadfence();
            p.done[0] = 0;
            if (atomicExch(p.done + 1, 0)) {
                for (int c = 0; c < (int)gridDim.x; ++c)
                    if (atomicAnd(p.done + 2 + c / 32, ~(1 << (c & 31))) >> (c & 31) & 1)
                        for (int b = __ldcg(p.gave_up + 2 * c); b <= __ldcg(p.gave_up + 2 * c + 1); ++b)
                            atomicOr(p.status + b, SVF_DEV_TIMEOUT);
            }
        }
    }
}

// K or V cache [num_pages * page_size tokens][Hkv][128] as a 3-D map; boxes of 64 dims x 1 head
// x one page (at most 128 tokens), 128-byte swizzle.
bool make_cache_map(CUtensorMap *map, const void *base, int num_pages, int page_size, int Hkv) {
    auto enc = tensor_map_encoder();
    if (!enc) return false;
    cuuint64_t dims[3] = {(cuuint64_t)ct::HD, (cuuint64_t)Hkv,
                          (cuuint64_t)num_pages * (cuuint64_t)page_size};
    cuuint64_t strides[2] = {(cuuint64_t)ct::HD * 2, (cuuint64_t)Hkv * ct::HD * 2};
    cuuint32_t box[3] = {64, 1, (cuuint32_t)(page_size < ct::BN ? page_size : ct::BN)};
    cuuint32_t estr[3] = {1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box,
               estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// q [rows][Hq][128]: boxes of 64 dims x G heads x floor(128 / G) tokens, the rows (token, head) of
// a half.
bool make_rows_map(CUtensorMap *map, const void *q, int rows, int Hq, int G) {
    auto enc = tensor_map_encoder();
    if (!enc) return false;
    cuuint64_t dims[3] = {(cuuint64_t)ct::HD, (cuuint64_t)Hq, (cuuint64_t)rows};
    cuuint64_t strides[2] = {(cuuint64_t)ct::HD * 2, (cuuint64_t)Hq * ct::HD * 2};
    cuuint32_t box[3] = {64, (cuuint32_t)G, (cuuint32_t)(128 / G)};
    cuuint32_t estr[3] = {1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(q), dims, strides, box,
               estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

cudaError_t launch_chunk_tc(const ChunkParams &p, int ctas, cudaStream_t stream) {
    CUtensorMap tmk, tmv, tmq;
    if (!make_cache_map(&tmk, p.k_cache, p.num_pages, p.ps, p.Hkv) ||
        !make_cache_map(&tmv, p.v_cache, p.num_pages, p.ps, p.Hkv) ||
        !make_rows_map(&tmq, p.q, p.rows, p.Hq, p.G))
        return cudaErrorInvalidValue;
    const cudaError_t e = cudaFuncSetAttribute(
        chunk_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, TcSmem::kDynamic);
    if (e != cudaSuccess) return e;
    return launch_pdl(chunk_tc_kernel, dim3((unsigned)ctas), dim3(ct::NT), (size_t)TcSmem::kDynamic,
                      stream, 0u, tmk, tmv, tmq, p);
}

}  // namespace svf
