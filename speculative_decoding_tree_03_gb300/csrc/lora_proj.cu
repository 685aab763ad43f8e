// lora_proj.cu -- a shared projection with a low-rank adapter per request:
//     y[r] = W x[r] + s_a B_a (A_a x[r]),   a = ids[r / rows_per_id]
// (a = -1: y[r] = W x[r]), bf16 operands and result, fp32 sums.
//
// lora_shrink.cu leaves t[r] = s_a A_a x[r]. Here the rest is ONE matrix product
// with a longer inner axis: to the H columns of x and W come, for every
// distinct adapter a of the row tile, rank columns that hold t on the rows of a
// (zero on the others) and B_a. So the adapters ride in the same tensor-memory
// accumulator as the shared product, and y is written once.
//   - t is kept as two bf16 terms, hi + lo (16 bits of significand, error
//     2^-16 of t): one rounding to bf16 would add an error as large as the
//     result's own when the adapter's part dominates.
//   - A product of a zero of t with an infinity or NaN of another request's
//     B_a would be NaN. Every B_a tile is looked over in shared memory before
//     its products: non-finite elements are replaced by tiny numbers of their
//     sign there, and their terms are added to the rows of a alone, in the
//     epilogue. Not by zero: an infinite t times the tiny number is the
//     infinity that it is times the element, where zero would make it NaN; on
//     the rows of a the sum is infinite or NaN by the added terms whatever a
//     tiny number leaves, on all others it meets a zero of t.
//   - B_a and t come by 16-byte asynchronous copies of the adapter warps, which
//     place the chunks as the MMA's swizzle wants them, leave t's rows of other
//     adapters zero, and bring a warp's first B_a before t is there. TMA boxes
//     of 32-byte rows took 3.6 us from t's end to the first adapter's products
//     (64 requests, 56 adapters of rank 16, 4096 -> 4096: 22.7 us; 20.0 with the copies).
//   - The tensor-core work of an adapter is confined to the window of the tile
//     that holds its rows (the MMA's N: steps of 16 rows, of 32 for a pair of
//     CTAs), and a 64-column block carries as many adapters as fit: 4 of rank
//     <= 16 (tiles of 32-byte rows), 2 of rank <= 32 (64 bytes), else one (128
//     bytes).
//
// W's rows are the MMA's M axis (128 per CTA), the rows of x its N axis (tiles
// of BN <= 256), K in blocks of 64 staged by TMA with 128-byte swizzle.
// CG = 2: two CTAs of a cluster work on one tile of 256 rows of W
// (cta_group::2), each loads its own 128 rows of W and half of the x tile, and
// the first one issues the products for both. One CTA alone would have to
// bring 48 KB into shared memory per 128 x 256 x 64 block, and shared memory
// would be what bounds it; the pair brings 32 KB each. CG = 1 serves few rows
// (bound by the bytes of W).
// Roles of a CTA (320 threads):
//   warp 0      producer: TMA of W and x blocks; then it hands free stages on;
//   warp 1      MMA issuer (of the pair's first CTA);
//   warps 2-5   epilogue (tensor memory -> y; in pairs warps 6-9 take half of
//               the last tile's);
//   warps 6-9   adapters: warp 6 lists the tile's distinct adapters; each of
//               the four fills the adapter blocks of every fourth stage and
//               looks over their B_a.
// The t columns come last, so the shared product runs while lora_shrink still
// does (the launches overlap; only the adapter warps wait for it, before t).
//
// Few rows leave too few tiles for the SMs: CK CTAs (or pairs) of a cluster
// then share a tile, each with an equal part of K and every CK-th adapter
// block, and their sums meet over distributed shared memory in a fixed order.
//
// Bound and measured (graph replays, three sets of inputs in turn): 1984 rows,
// 8192 -> 10240, 24 adapters of rank 16: the tensor cores under the power cap,
// 202-221 us from one run to the next, 1.51 to 1.66 PFLOP/s, 88 to 97 % of the
// measured sustained rate of a library product, whose own product of this shape
// without adapters takes 210 (341 us with one CTA per tile and lane-predicated
// issue); in a stream of eager calls 230. Few rows: HBM and the call's own
// latency: one row, 4096 -> 6144: 14.5 us, of which 2.2 pass until this kernel
// starts, 2.6 to the first product, 6.6 while W streams (50 MB), 3.1 in the
// adapter's products, the cluster's sum and the exit; 64 requests 18.1 us, an
// EAGLE-2 batch of 4 x 60 rows (rank 64, 4096 -> 6144) 22.4.
// Tried and dropped: adapter blocks spread among the last blocks of K
// (70B-shaped batch 222 against 200 us: their checks and the products share
// shared memory's bandwidth), one polling lane per warp (one row 19.2
// against 18.3), two CTAs per SM (19.8 against 16.9), a warp's next B_a on
// its way before the last one is looked over (no gain in any shape), all
// four adapter warps on each block where there are one or two (EAGLE-2 batch
// 23.9 against 23.6), B_a brought to the L2 while W streams (128 rows, 100
// adapters of rank 64: 142 against 129), 88 registers per thread (64
// requests 22.2 against 19.9: the CTAs start later beside lora_shrink's).
#include <cuda.h>
#include <cudaTypedefs.h>

#include <atomic>
#include <map>
#include <mutex>
#include <tuple>

#include "common.cuh"
#include "internal.h"
#include "lora.h"

namespace svf {

namespace lp {
constexpr int BM = 128;                 // rows of W per CTA (MMA M per CTA)
constexpr int BK = 64;                  // K per stage: one 128-byte swizzle row
constexpr int A_BYTES = BM * BK * 2;
constexpr int MAX_STAGES = 12;
constexpr int THREADS = 320;
constexpr int MAX_BN = 256;
constexpr int MAX_LIST = 3 * MAX_BN / 2; // adapter windows of one row tile
constexpr int HASH = 2 * MAX_BN;        // slots for the distinct adapters of a row tile
constexpr int SMEM_BUDGET = 192 * 1024; // stage ring; leaves lora_shrink room beside it
}  // namespace lp

struct LpParams {
    int R, H, O, rank, adapters, per;
    int BN, CK, n_tiles, tiles, kblocks, stages;
    int kchunks;    // 64-column blocks of one adapter: 1, or 2 (rank > 64)
    int lpack;      // log2 of the adapters of one block: 2, 1 or 0 (0 when kchunks is 2)
    uint32_t tmem_cols;
    unsigned long long wait_ns;
    const __nv_bfloat16 *t;  // [hi and lo, R, rank]
    const int32_t *ids;
    const __nv_bfloat16 *lora_b;
    __nv_bfloat16 *y;
    long long y_stride;
    int32_t *status;
};

// Shared memory behind the stage ring.
struct LpShared {
    uint64_t full[lp::MAX_STAGES];   // a block of W and x has landed (in the pair's first CTA)
    uint64_t ready[lp::MAX_STAGES];  // a stage is free for an adapter block
    uint64_t ext[lp::MAX_STAGES];    // the block's B_a and t are there (first CTA: both CTAs')
    uint64_t empty[lp::MAX_STAGES];
    uint64_t recv;                   // the other CTAs' sums of this CTA's rows of y
    uint64_t acc_full[2], acc_empty[2], list_full[2], list_empty[2], ext_done[2];
    int ids[2][lp::MAX_BN];     // adapter of each row of the tile; -1 none, -2 a bad id
    uint32_t list[2][lp::MAX_LIST]; // an adapter's window: lp_window's fields
    int n_list[2];
    int nonfinite[2];           // some B_a tile held an infinity or NaN
    int bad_id[2];              // some row's id is bad
    // the list's hash table: adapter id and number, and each one's first and last row
    int hash_id[lp::HASH], hash_no[lp::HASH], span[lp::MAX_BN];
    uint32_t tmem;
    int committed;  // stages whose products were issued
    uint32_t par_main, any_main;  // the producer's, at its end
    int abort;
};

// A list entry: the adapter (below 2^16), the first row of its window and its
// row count, in units of 16 rows.
__device__ __forceinline__ uint32_t lp_window(int id, int w0, int len) {
    return (uint32_t)id | (uint32_t)(w0 >> 4) << 16 | (uint32_t)(len >> 4) << 24;
}
__device__ __forceinline__ int lp_adapter(uint32_t w) { return (int)(w & 0xffffu); }
__device__ __forceinline__ int lp_first(uint32_t w) { return (int)(w >> 16 & 0xffu) << 4; }
__device__ __forceinline__ int lp_rows(uint32_t w) { return (int)(w >> 24) << 4; }

__device__ __forceinline__ bool lp_wait(uint64_t *bar, uint32_t parity, volatile int *abort,
                                        unsigned long long ns) {
    const bool ok = mbar_wait_for(bar, parity, abort, ns);
    return __all_sync(0xffffffffu, ok);
}

// A thread's wait for a barrier that threads of another CTA arrive on.
__device__ __forceinline__ bool lp_wait_cluster(uint64_t *bar, uint32_t parity,
                                                volatile int *abort, unsigned long long ns) {
    if (mbar_try_wait_cluster(bar, parity)) return true;
    const unsigned long long t0 = globaltimer_ns();
    for (uint32_t it = 1;; ++it) {
        if (mbar_try_wait_cluster(bar, parity)) return true;
        if ((it & 63u) == 0) {
            if (*abort) return false;
            if (globaltimer_ns() - t0 > ns) {
                *abort = 1;
                return false;
            }
        }
    }
}

// One lane of a converged warp. tcgen05 and TMA instructions take their
// operands from uniform registers; under this predicate the compiler knows that
// one thread runs them and needs no loop over lanes around each (under
// `lane == 0` every block of K took 0.43 us whatever its size).
__device__ __forceinline__ bool lp_elect() {
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(p));
    return p != 0;
}

// Arrive on a barrier of another CTA of the cluster (an address from cluster_map).
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t remote) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(remote)
                 : "memory");
}

// A bulk copy from this CTA's shared memory to the same object `dst` of CTA `to`
// of the cluster, whose bytes count on that CTA's `bar`.
__device__ __forceinline__ void bulk_copy_peer(void *dst, const void *src, uint32_t bytes,
                                               uint64_t *bar, uint32_t to) {
    asm volatile(
        "cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, "
        "[%3];" ::"r"(cluster_map(dst, to)),
        "r"(smem_u32(src)), "r"(bytes), "r"(cluster_map(bar, to))
        : "memory");
}

// ---------------------------------------------------------------- CTA pairs
// A TMA load into this CTA whose bytes count on a barrier of the pair's first
// CTA (bar: its shared::cluster address).
__device__ __forceinline__ void tma_load_2d_pair(void *dst, const void *tmap, int c0, int c1,
                                                 uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile"
        ".mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(c0), "r"(c1), "r"(bar)
        : "memory");
}
template <int CG>
__device__ __forceinline__ void lp_tmem_alloc(uint32_t *dst, uint32_t ncols) {
    if constexpr (CG == 1) {
        tmem_alloc(dst, ncols);
        tmem_relinquish();
    } else {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(dst)),
                     "r"(ncols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
}
template <int CG>
__device__ __forceinline__ void lp_tmem_dealloc(uint32_t taddr, uint32_t ncols) {
    if constexpr (CG == 1)
        tmem_dealloc(taddr, ncols);
    else
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr),
                     "r"(ncols)
                     : "memory");
}
template <int CG>
__device__ __forceinline__ void lp_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       uint32_t accumulate) {
    if constexpr (CG == 1) {
        umma_ss(d, a, b, idesc, accumulate);
    } else {
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
            : "memory");
    }
}
// Arrive on `bar` (in both CTAs of a pair, mask) once the products issued so far are done.
template <int CG>
__device__ __forceinline__ void lp_commit(uint64_t *bar, uint16_t mask) {
    if constexpr (CG == 1)
        umma_commit(bar);
    else
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster"
            ".multicast::cluster.b64 [%0], %1;" ::"r"(smem_u32(bar)),
            "h"(mask)
            : "memory");
}

// Matrix descriptor of a K-major tile with rows of row_bytes (32, 64 or 128,
// swizzled over as many bytes).
__device__ __forceinline__ uint64_t lp_desc(uint32_t start, uint32_t row_bytes) {
    const uint64_t layout = row_bytes == 128 ? 2u : row_bytes == 64 ? 4u : 6u;
    uint64_t d = (uint64_t)((start >> 4) & 0x3FFFu);
    d |= (uint64_t)1 << 16;                         // leading offset: not used, K within a row
    d |= (uint64_t)((8 * row_bytes) >> 4) << 32;    // 8-row groups
    d |= (uint64_t)1 << 46;
    d |= layout << 61;
    return d;
}
// The distinct adapters of rows [n0, n0 + BN), in order of first appearance,
// each with the window of the tile that holds its rows (16 CG rows aligned),
// in pieces of at most BN / 2 rows: at most 3 pieces for an adapter of two
// rows or more and one for the others, 1.5 BN in all. One warp, 32 rows at a
// time: lanes with the same id are matched, the first of each looks the id up
// in a hash table in shared memory (about 1 us for 256 rows; looking at the
// rows one after the other took 0.35 us a row).
template <int CG>
__device__ void lp_build_list(const LpParams &p, LpShared *sh, int buf, int n0, int lane) {
    constexpr int G = 16 * CG;
    for (int k = lane; k < lp::HASH; k += 32) sh->hash_id[k] = -1;
    __syncwarp();
    int n = 0;  // distinct adapters so far
    bool any_bad = false;
    for (int c = 0; c < p.BN; c += 32) {
        const int row = n0 + c + lane;
        int id = -1;
        if (row < p.R) {
            id = p.ids[row / p.per];
            if (id < -1 || id >= p.adapters) id = -2;
        }
        sh->ids[buf][c + lane] = id;
        any_bad |= id == -2;
        const unsigned same = __match_any_sync(0xffffffffu, id);
        bool fresh = false;
        int slot = 0;
        if (id >= 0 && lane == __ffs(same) - 1) {
            slot = (int)((unsigned)id * 2654435761u >> 23);  // 512 slots
            while (true) {
                const int was = atomicCAS(&sh->hash_id[slot], -1, id);
                fresh = was == -1;
                if (fresh || was == id) break;
                slot = (slot + 1) & (lp::HASH - 1);  // at most 256 ids: a slot is free
            }
            const int last = c + 31 - __clz(same);
            if (!fresh) {
                const int no = sh->hash_no[slot];
                sh->span[no] = (sh->span[no] & 0xffff) | last << 16;
            }
        }
        const unsigned m = __ballot_sync(0xffffffffu, fresh);
        if (fresh) {
            const int no = n + __popc(m & ((1u << lane) - 1u));
            sh->hash_no[slot] = no;
            sh->span[no] = (c + lane) | (c + 31 - __clz(same)) << 16;
            sh->list[buf][no] = (uint32_t)id;  // spread out to its pieces below
        }
        n += __popc(m);
        __syncwarp();
    }
    any_bad = __any_sync(0xffffffffu, any_bad);
    // the windows, from the last 32 adapters to the first, so that no piece is
    // written over an adapter that is still to be read
    const int most = (p.BN / 2) & ~(G - 1);
    int total = 0;
    for (int e = lane; e < n; e += 32) {
        const int w0 = (sh->span[e] & 0xffff) & ~(G - 1), w1 = ((sh->span[e] >> 16) + G) & ~(G - 1);
        total += (w1 - w0 + most - 1) / most;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    int end = total;
    for (int e0 = (n - 1) & ~31; e0 >= 0 && n > 0; e0 -= 32) {
        const int e = e0 + lane;
        int id = 0, w0 = 0, w1 = 0, pieces = 0;
        if (e < n) {
            id = (int)sh->list[buf][e];
            w0 = (sh->span[e] & 0xffff) & ~(G - 1);
            w1 = ((sh->span[e] >> 16) + G) & ~(G - 1);
            pieces = (w1 - w0 + most - 1) / most;
        }
        int after = pieces;  // pieces of this lane's adapter and the later ones
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_down_sync(0xffffffffu, after, o);
            if (lane + o < 32) after += v;
        }
        __syncwarp();
        for (int k = 0; k < pieces; ++k, w0 += most)
            sh->list[buf][end - after + k] = lp_window(id, w0, min(w1 - w0, most));
        end -= __shfl_sync(0xffffffffu, after, 0);
        __syncwarp();
    }
    if (lane == 0) {
        sh->n_list[buf] = total;
        sh->nonfinite[buf] = 0;
        sh->bad_id[buf] = any_bad;
    }
    __syncwarp();
}

// The terms of non-finite elements of the row's own B_a, from memory.
__device__ __noinline__ float lp_nonfinite_terms(const LpParams &p, int id, int row, int o) {
    const __nv_bfloat16 *b = p.lora_b + ((size_t)id * p.O + o) * (size_t)p.rank;
    const __nv_bfloat16 *hi = p.t + (size_t)row * p.rank, *lo = hi + (size_t)p.R * p.rank;
    float v = 0.f;
    for (int j = 0; j < p.rank; ++j) {
        const float f = __bfloat162float(b[j]);
        if (!isfinite(f)) v += (__bfloat162float(hi[j]) + __bfloat162float(lo[j])) * f;
    }
    return v;
}

// 32 columns of a tile that has bad ids or met non-finite elements of some B_a
// (patch).
__device__ __noinline__ void lp_store_checked(const LpParams &p, const int *ids, const uint32_t *r,
                                              bool patch, int rows_left, int row0, int o) {
    for (int j = 0; j < 32 && j < rows_left; ++j) {
        float v = ids[j] == -2 ? 0.f : __uint_as_float(r[j]);
        if (patch && ids[j] >= 0) v += lp_nonfinite_terms(p, ids[j], row0 + j, o);
        p.y[(long long)(row0 + j) * p.y_stride + o] = __float2bfloat16(v);
    }
}

// acc + 0 * v on pairs of bf16.
__device__ __forceinline__ void add_zero_times(uint32_t &acc, uint32_t v) {
    asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(acc) : "r"(v), "r"(0u));
}

// Replaces the non-finite elements of 8 bf16 values by numbers of their sign
// between 2^-126 and 2^-125 (the largest exponent becomes the smallest).
__device__ __forceinline__ void lp_clean(uint4 *at) {
    const uint4 b = *at;
    uint32_t wd[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if ((wd[k] & 0x7f80u) == 0x7f80u) wd[k] &= ~0x7f00u;
        if ((wd[k] & 0x7f800000u) == 0x7f800000u) wd[k] &= ~0x7f000000u;
    }
    *at = make_uint4(wd[0], wd[1], wd[2], wd[3]);
}

// 16 bytes to shared memory, zeros unless ok (src is not read then).
__device__ __forceinline__ void lp_copy16(uint32_t dst, const void *src, bool ok) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(ok ? 16 : 0)
                 : "memory");
}

// Chunk c of row `row` of a tile with rows of 16 NCH bytes, swizzled over as many.
template <int NCH>
__device__ __forceinline__ uint32_t lp_chunk(uint32_t tile, int row, int c) {
    const uint32_t at = tile + (uint32_t)(row * NCH + c) * 16u;
    return at ^ ((at >> 7 & (uint32_t)(NCH - 1)) << 4);
}

// An adapter block: up to PACK adapters, entries from e0 on of list buf, columns
// from 64 kx on.
struct LpBlock {
    int buf, e0, kx;
    int m0, row0;    // the tile's first row of W (this CTA's) and of x
    int half, slot;  // as in the kernel
};

// Copies the block's rows of t, hi and lo; zeros on rows of other adapters.
template <int CG, int PACK>
__device__ __forceinline__ void lp_copy_t(const LpParams &p, const LpShared *sh, const LpBlock &b,
                                          uint32_t hi, int lane) {
    constexpr int NCH = 8 / PACK;  // 16-byte chunks of a row
    const int ne = min(PACK, sh->n_list[b.buf] - b.e0);
    const int c = lane % NCH;
    const bool inside = b.kx * 8 + c < p.rank / 8;
    for (int e = 0; e < ne; ++e, hi += (uint32_t)b.slot) {
        const uint32_t w = sh->list[b.buf][b.e0 + e], lo = hi + (uint32_t)(b.slot / 2);
        // this CTA's rows of the window: all, or its half of them
        const int rows = lp_rows(w) / CG, first = lp_first(w) + b.half * rows;
        for (int row = lane / NCH; row < rows; row += 32 / NCH) {
            const bool ok = inside && sh->ids[b.buf][first + row] == lp_adapter(w);
            const size_t at =
                ok ? (size_t)(b.row0 + first + row) * p.rank + b.kx * lp::BK + c * 8 : 0;
            lp_copy16(lp_chunk<NCH>(hi, row, c), p.t + at, ok);
            lp_copy16(lp_chunk<NCH>(lo, row, c), p.t + (size_t)p.R * p.rank + at, ok);
        }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
}

// Fills a stage with an adapter block, by one warp. True if B_a held an infinity
// or NaN; they are replaced (lp_clean).
template <int CG, int PACK>
__device__ __forceinline__ bool lp_load_block(const LpParams &p, const LpShared *sh,
                                              const LpBlock &b, uint8_t *tiles_b, uint8_t *hi,
                                              int lane) {
    constexpr int NCH = 8 / PACK;
    const int ne = min(PACK, sh->n_list[b.buf] - b.e0);
    const int c = lane % NCH;
    const bool inside = b.kx * 8 + c < p.rank / 8;
    for (int e = 0; e < ne; ++e) {
        const uint32_t tile = smem_u32(tiles_b) + (uint32_t)(e * lp::BM * NCH * 16);
        const int id = lp_adapter(sh->list[b.buf][b.e0 + e]);
        const __nv_bfloat16 *src = p.lora_b + ((size_t)id * p.O + b.m0) * (size_t)p.rank;
#pragma unroll 8
        for (int row = lane / NCH; row < lp::BM; row += 32 / NCH) {
            const bool ok = inside && b.m0 + row < p.O;
            lp_copy16(lp_chunk<NCH>(tile, row, c),
                      src + (ok ? row * p.rank + b.kx * lp::BK + c * 8 : 0), ok);
        }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    pdl_wait();  // t is complete
    lp_copy_t<CG, PACK>(p, sh, b, smem_u32(hi), lane);
    asm volatile("cp.async.wait_group 1;" ::: "memory");  // B_a is there
    __syncwarp();
    // 0 times an infinity or NaN is NaN, and stays in the sum
    uint4 *tiles = reinterpret_cast<uint4 *>(tiles_b) + lane;
    uint32_t seen[4] = {0, 0, 0, 0};
    for (int k = 0; k < ne * lp::BM * NCH; k += 8 * 32) {
        uint4 v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) v[u] = tiles[k + u * 32];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            add_zero_times(seen[0], v[u].x);
            add_zero_times(seen[1], v[u].y);
            add_zero_times(seen[2], v[u].z);
            add_zero_times(seen[3], v[u].w);
        }
    }
    const bool bad =
        __any_sync(0xffffffffu, ((seen[0] | seen[1] | seen[2] | seen[3]) & 0x7fff7fffu) != 0);
    if (bad)
        for (int k = 0; k < ne * lp::BM * NCH; k += 32) lp_clean(tiles + k);
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    return bad;
}

// The parameters stay where the launch puts them (__grid_constant__): functions
// that are not inlined take their address, for which every thread would else
// make a copy in local memory and read all of them from there (one row, 4096 ->
// 6144: 15.1 against 14.4 us; EAGLE-2 batch 23.5 against 22.5; 128 rows, 100
// adapters of rank 16, in single CTAs 30.8 against 30.0; of ten larger shapes
// 768 rows of 24 adapters of rank 16 lost most, 33.7 to 34.7).
template <int CG>
__global__ void __maxnreg__(80)
    lora_proj_kernel(const __grid_constant__ CUtensorMap tmw,
                     const __grid_constant__ CUtensorMap tmx,
                     const __grid_constant__ LpParams p) {
    using namespace lp;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const int S = p.stages;
    const int b_bytes = p.BN / CG * 128;
    uint8_t *sA = smem;
    uint8_t *sB = smem + S * A_BYTES;
    LpShared *sh = reinterpret_cast<LpShared *>(sB + S * b_bytes);
    volatile int *abort_flag = &sh->abort;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int cluster = CG * p.CK;
    if (!cluster_shape_is((uint32_t)cluster, 1u, 1u)) {
        // not the cluster that pairs and sums address: the whole cluster leaves
        pdl_wait();
        if (tid == 0) atomicOr(p.status, SVF_DEV_BAD_CLUSTER);
        return;
    }
    const int crank = cluster > 1 ? (int)cluster_ctarank() : 0;
    const int half = CG == 2 ? crank & 1 : 0;  // which 128 of the tile's rows of W
    const int lead = crank - half;             // the pair's first CTA
    const int rank = crank / CG;               // which part of K
    const uint16_t pair_mask = (uint16_t)(3u << lead);
    const int first_tile = blockIdx.x / cluster, tile_step = gridDim.x / cluster;
    const int kb0 = (int)((long long)p.kblocks * rank / p.CK);
    const int nkb = (int)((long long)p.kblocks * (rank + 1) / p.CK) - kb0;
    const int row_bytes = 128 >> p.lpack, tile_bytes = BM * row_bytes;
    const int pack = 1 << p.lpack, deep = p.kchunks - 1;
    // A stage's x area is shared out among the block's adapters; each part
    // holds the rows of t's hi, and from its middle on those of lo.
    const int slot = b_bytes >> p.lpack;

    const int rot = (int)((long long)first_tile * nkb / tile_step) % nkb;
    // One CTA's first loads need no more than its own barriers, so they go out
    // before tensor memory is there (one row, 4096 -> 6144: 15.9 against 16.2 us).
    const int pre = CG == 1 ? min(S, nkb) : 0;

    if (warp == 0 && lp_elect()) {
        for (int s = 0; s < S; ++s) {
            mbar_init(&sh->full[s], 1);
            mbar_init(&sh->ready[s], 1);
            mbar_init(&sh->ext[s], CG);
            mbar_init(&sh->empty[s], 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(&sh->acc_full[a], 1);
            mbar_init(&sh->acc_empty[a], 4 * CG);
            mbar_init(&sh->list_full[a], 1);
            mbar_init(&sh->list_empty[a], 10);  // warps 0, 1, 2-5, 6-9
            mbar_init(&sh->ext_done[a], 4);
        }
        mbar_init(&sh->recv, 1);
        sh->committed = 0;
        sh->abort = 0;
        mbar_fence_init();
        if constexpr (CG == 1) {
            const int m0 = first_tile / p.n_tiles * BM, n0 = first_tile % p.n_tiles * p.BN;
            int kc = (kb0 + rot) * BK;
            for (int s = 0; s < pre; ++s) {
                mbar_arrive_expect_tx(&sh->full[s], (uint32_t)(A_BYTES + b_bytes));
                tma_load_2d(sA + s * A_BYTES, &tmw, kc, m0, &sh->full[s]);
                tma_load_2d(sB + s * b_bytes, &tmx, kc, n0, &sh->full[s]);
                kc = kc + BK == (kb0 + nkb) * BK ? kb0 * BK : kc + BK;
            }
        }
    }
    if (CG == 2 && warp == 2 && lane == 0) {
        tma_prefetch_desc(&tmw);
        tma_prefetch_desc(&tmx);
    }
    if (warp == 1) lp_tmem_alloc<CG>(&sh->tmem, p.tmem_cols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (CG == 2) {  // the other CTA's barriers exist before anything arrives on them
        cluster_arrive();
        cluster_wait();
    }
    // Only t waits for the kernel before this one (in the adapter warps): that
    // kernel lets this one start after its own wait, so what this call reads
    // besides t was complete by then.
    if (tile_step >= p.tiles) pdl_launch_dependents();  // one tile each
    const uint32_t tmem = sh->tmem;
    // A stage's full barrier counts its W and x blocks, its ready and ext
    // barriers its adapter blocks; who waits for one keeps the parity of its
    // next phase, one bit per stage.
    uint32_t par_main = 0, par_ext = 0;
    uint32_t any_main = 0;

    // Columns from .. to - 1 of a finished tile (rows of y): the work of warps 2
    // to 5. In pairs, whose tiles are wide, warps 6 to 9 take the second half of
    // a CTA's last tile; their adapter blocks are done by then (EAGLE-2 batch
    // 23.1 us against 23.5; the 32 to 64 columns of single CTAs lost 1 to 4 %). One
    // code for both sizes costs single CTAs of many adapters 3 % (128 rows, 100
    // adapters of rank 16: 30.0 us against 29.1 with a copy of their own).
    const int split = CG == 2 ? (p.BN / 32 + 1) / 2 * 32 : p.BN;
    auto drain = [&](int buf, int m0, int n0, int from, int to) {
        const int q = warp & 3;  // tensor-memory lanes 32 q .. 32 q + 31
        const uint32_t lane_base = (uint32_t)(q * 32) << 16;
        const bool pairs = (p.y_stride & 1) == 0 && (reinterpret_cast<uintptr_t>(p.y) & 3) == 0;
        const int o = m0 + q * 32 + lane;
        const bool patch = sh->nonfinite[buf] != 0;
        if (p.CK > 1) {
            // The ring is idle: the others may send once all say so. Partial
            // sums into it, [column][128] fp32.
            cluster_arrive();
            float *part = reinterpret_cast<float *>(smem) + q * 32 + lane;
            for (int c = from; c < to; c += 32) {
                uint32_t r[32];
                tmem_ld32(tmem + lane_base + (uint32_t)(buf * p.BN + c), r);
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 32; ++j) part[(c + j) * BM] = __uint_as_float(r[j]);
            }
            fence_proxy_async_smem();  // the bulk copies below read them
        } else {
            const bool plain = !patch && !sh->bad_id[buf];
            for (int c = from; c < to; c += 32) {
                uint32_t r[32];
                tmem_ld32(tmem + lane_base + (uint32_t)(buf * p.BN + c), r);
                tmem_wait_ld();
                const int rows_left = p.R - (n0 + c);
                if (plain && !pairs) {
                    __nv_bfloat16 *at = p.y + (long long)(n0 + c) * p.y_stride + o;
                    if (o < p.O) {
#pragma unroll
                        for (int j = 0; j < 32; ++j) {
                            if (j < rows_left) *at = __float2bfloat16(__uint_as_float(r[j]));
                            at += p.y_stride;
                        }
                    }
                    continue;
                }
                if (!plain) {
                    uint32_t v[32];
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] = r[j];
                    if (o < p.O)
                        lp_store_checked(p, sh->ids[buf] + c, v, patch, rows_left, n0 + c, o);
                    continue;
                }
                // two lanes swap a value each, so that a lane stores two
                // neighbours of one row: even lanes of row j, odd of j + 1
                const int odd = lane & 1;
                __nv_bfloat16 *dst =
                    p.y + (long long)(n0 + c + odd) * p.y_stride + (o - odd);
                const bool both = o - odd + 1 < p.O, one = o - odd < p.O;
                if (rows_left >= 32 && m0 + q * 32 + 32 <= p.O) {
#pragma unroll
                    for (int j = 0; j < 32; j += 2) {
                        const float a = __uint_as_float(r[j]), b = __uint_as_float(r[j + 1]);
                        const float got = __shfl_xor_sync(0xffffffffu, odd ? a : b, 1);
                        *reinterpret_cast<uint32_t *>(dst) =
                            odd ? pack_bf16x2(got, b) : pack_bf16x2(a, got);
                        dst += 2 * p.y_stride;
                    }
                    continue;
                }
#pragma unroll
                for (int j = 0; j < 32; j += 2) {
                    const float a = __uint_as_float(r[j]), b = __uint_as_float(r[j + 1]);
                    const float got = __shfl_xor_sync(0xffffffffu, odd ? a : b, 1);
                    const uint32_t w = odd ? pack_bf16x2(got, b) : pack_bf16x2(a, got);
                    if (j + odd < rows_left) {
                        if (both)
                            *reinterpret_cast<uint32_t *>(dst) = w;
                        else if (one)
                            *reinterpret_cast<uint16_t *>(dst) = (uint16_t)w;
                    }
                    dst += 2 * p.y_stride;
                }
            }
        }
    };

    if (warp == 0) {
        // ------------------------------------------------------------ producer
        if (lp_elect()) {
            bool ok = true;
            int i = 0, s = pre == S ? 0 : pre, done = pre;
            uint32_t turn = pre == S ? 0u : 1u;  // parity of the phase that frees stage s
            par_main = any_main = (1u << pre) - 1u;
            for (int tile = first_tile; tile < p.tiles && ok; tile += tile_step, ++i) {
                const int m0 = (tile / p.n_tiles * CG + half) * BM;
                const int n0 = tile % p.n_tiles * p.BN + half * (p.BN / 2);
                // tiles that start together start at different columns
                int kc = (kb0 + (rot + done) % nkb) * BK;
                for (int kb = done; kb < nkb; ++kb) {
                    if (!(ok = mbar_wait_for(&sh->empty[s], turn, abort_flag, p.wait_ns))) break;
                    if (half == 0)
                        mbar_arrive_expect_tx(&sh->full[s], (uint32_t)(CG * (A_BYTES + b_bytes)));
                    if constexpr (CG == 1) {
                        tma_load_2d(sA + s * A_BYTES, &tmw, kc, m0, &sh->full[s]);
                        tma_load_2d(sB + s * b_bytes, &tmx, kc, n0, &sh->full[s]);
                    } else {
                        const uint32_t bar = cluster_map(&sh->full[s], (uint32_t)lead);
                        tma_load_2d_pair(sA + s * A_BYTES, &tmw, kc, m0, bar);
                        tma_load_2d_pair(sB + s * b_bytes, &tmx, kc, n0, bar);
                    }
                    par_main ^= 1u << s;
                    any_main |= 1u << s;
                    kc = kc + BK == (kb0 + nkb) * BK ? kb0 * BK : kc + BK;
                    if (++s == S) {
                        s = 0;
                        turn ^= 1u;
                    }
                }
                if (!ok) break;
                done = 0;
                const int buf = i & 1;
                if (!(ok = mbar_wait_for(&sh->list_full[buf], (uint32_t)(i >> 1 & 1), abort_flag,
                                         p.wait_ns)))
                    break;
                const int n_list = sh->n_list[buf];
                const int blocks = ((n_list + pack - 1) >> p.lpack) << deep;
                for (int x = rank; x < blocks; x += p.CK) {
                    if (!(ok = mbar_wait_for(&sh->empty[s], turn, abort_flag, p.wait_ns))) break;
                    mbar_arrive(&sh->ready[s]);
                    if (++s == S) {
                        s = 0;
                        turn ^= 1u;
                    }
                }
                mbar_arrive(&sh->list_empty[buf]);
            }
            pdl_wait();  // this grid ends after the one before it
            sh->par_main = par_main;
            sh->any_main = any_main;
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer
        if (lp_elect()) {
            bool ok = true;
            int i = 0, s = 0, it = 0;
            const uint32_t idesc = idesc_bf16_f32(BM * CG, p.BN, false, false);
            const uint64_t desc_a = smem_desc_sw128(smem_u32(sA), 16, 1024);
            const uint64_t desc_b = smem_desc_sw128(smem_u32(sB), 16, 1024);
            for (int tile = first_tile; tile < p.tiles && ok; tile += tile_step, ++i) {
                const int buf = i & 1, ause = i >> 1;
                const uint32_t d = tmem + (uint32_t)(buf * p.BN);
                if (half == 0) {
                    if (ause > 0 &&
                        !(ok = lp_wait_cluster(&sh->acc_empty[buf], (uint32_t)((ause - 1) & 1),
                                               abort_flag, p.wait_ns)))
                        break;
                    tc_fence_after();
                    for (int kb = 0; kb < nkb; ++kb, ++it) {
                        if (!(ok = mbar_wait_for(&sh->full[s], par_main >> s & 1u, abort_flag,
                                                 p.wait_ns)))
                            break;
                        par_main ^= 1u << s;
                        tc_fence_after();
                        const uint64_t a = desc_a + (uint32_t)(s * (A_BYTES >> 4));
                        const uint64_t b = desc_b + (uint32_t)(s * (b_bytes >> 4));
#pragma unroll
                        for (int k = 0; k < BK / 16; ++k)
                            lp_mma<CG>(d, a + 2 * k, b + 2 * k, idesc, (kb > 0 || k > 0) ? 1u : 0u);
                        lp_commit<CG>(&sh->empty[s], pair_mask);
                        if (++s == S) s = 0;
                    }
                    if (!ok) break;
                }
                if (!(ok = mbar_wait_for(&sh->list_full[buf], (uint32_t)(ause & 1), abort_flag,
                                         p.wait_ns)))
                    break;
                if (half == 0) {
                    const int n_list = sh->n_list[buf];
                    const int blocks = ((n_list + pack - 1) >> p.lpack) << deep;
                    const uint64_t ext_a = lp_desc(smem_u32(sA), row_bytes);
                    const uint64_t ext_t = lp_desc(smem_u32(sB), row_bytes);
                    for (int x = rank; x < blocks; x += p.CK, ++it) {
                        const int e0 = (x >> deep) << p.lpack;
                        const int ne = min(pack, n_list - e0);
                        if (!(ok = lp_wait_cluster(&sh->ext[s], par_ext >> s & 1u, abort_flag,
                                                   p.wait_ns)))
                            break;
                        par_ext ^= 1u << s;
                        tc_fence_after();
                        const int ksteps = (min(p.rank - (x & deep) * BK, BK) + 15) >> 4;
                        for (int e = 0; e < ne; ++e) {
                            const uint32_t w = sh->list[buf][e0 + e];
                            const uint32_t dw = d + (uint32_t)lp_first(w);
                            const uint32_t idw = idesc_bf16_f32(BM * CG, lp_rows(w), false, false);
                            const uint64_t da =
                                ext_a + (uint32_t)((s * A_BYTES + e * tile_bytes) >> 4);
                            const uint64_t hi = ext_t + (uint32_t)((s * b_bytes + e * slot) >> 4);
                            const uint64_t lo = hi + (uint32_t)(slot / 2 >> 4);
                            for (int k = 0; k < ksteps; ++k) {
                                lp_mma<CG>(dw, da + 2 * k, hi + 2 * k, idw, 1u);
                                lp_mma<CG>(dw, da + 2 * k, lo + 2 * k, idw, 1u);
                            }
                        }
                        lp_commit<CG>(&sh->empty[s], pair_mask);
                        if (++s == S) s = 0;
                    }
                    if (!ok) break;
                    lp_commit<CG>(&sh->acc_full[buf], pair_mask);
                }
                mbar_arrive(&sh->list_empty[buf]);
            }
            sh->committed = it;
        }
        __syncwarp();
    } else if (warp < 6) {
        // ------------------------------------------------------------ epilogue
        bool ok = true;
        int i = 0;
        for (int tile = first_tile; tile < p.tiles && ok; tile += tile_step, ++i) {
            const int m0 = (tile / p.n_tiles * CG + half) * BM, n0 = tile % p.n_tiles * p.BN;
            const int buf = i & 1, ause = i >> 1;
            if (!(ok = lp_wait(&sh->acc_full[buf], (uint32_t)(ause & 1), abort_flag, p.wait_ns)))
                break;
            // the adapter warps are done with the tile: its ids and flag stand
            if (!(ok = lp_wait(&sh->ext_done[buf], (uint32_t)(ause & 1), abort_flag, p.wait_ns)))
                break;
            tc_fence_after();
            drain(buf, m0, n0, 0, tile + tile_step < p.tiles ? p.BN : split);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (half == 0)
                    mbar_arrive(&sh->acc_empty[buf]);
                else
                    mbar_arrive_cluster(cluster_map(&sh->acc_empty[buf], (uint32_t)lead));
                mbar_arrive(&sh->list_empty[buf]);
            }
        }
        if (p.CK > 1 && !ok) cluster_arrive();
    } else {
        // ------------------------------------------------------------ adapters
        // a stage's adapter blocks are always the same warp's, so that it sees
        // every phase of the stage's barrier
        const int w = warp - 6;
        bool ok = true;
        int s = 0, i = 0;
        for (int tile = first_tile; tile < p.tiles && ok; tile += tile_step, ++i) {
            const int n0 = tile % p.n_tiles * p.BN;
            const int m0 = (tile / p.n_tiles * CG + half) * BM;
            const int buf = i & 1, ause = i >> 1;
            if (warp == 6) {
                if (ause > 0 && !(ok = lp_wait(&sh->list_empty[buf], (uint32_t)((ause - 1) & 1),
                                               abort_flag, p.wait_ns)))
                    break;
                lp_build_list<CG>(p, sh, buf, n0, lane);
                if (lane == 0) mbar_arrive(&sh->list_full[buf]);
            }
            if (!(ok = lp_wait(&sh->list_full[buf], (uint32_t)(ause & 1), abort_flag, p.wait_ns)))
                break;
            s = (s + nkb) % S;
            const int n_list = sh->n_list[buf];
            const int blocks = ((n_list + pack - 1) >> p.lpack) << deep;
            for (int x = rank; x < blocks; x += p.CK, s = s + 1 == S ? 0 : s + 1) {
                if ((s & 3) != w) continue;
                if (!(ok = lp_wait(&sh->ready[s], par_ext >> s & 1u, abort_flag, p.wait_ns))) break;
                par_ext ^= 1u << s;
                const int e0 = (x >> deep) << p.lpack, kx = x & deep;
                uint8_t *tb = sA + s * A_BYTES, *hi = sB + s * b_bytes;
                const LpBlock b = {buf, e0, kx, m0, n0, half, slot};
                const bool bad =
                    p.lpack == 2   ? lp_load_block<CG, 4>(p, sh, b, tb, hi, lane)
                    : p.lpack == 1 ? lp_load_block<CG, 2>(p, sh, b, tb, hi, lane)
                                   : lp_load_block<CG, 1>(p, sh, b, tb, hi, lane);
                if (bad) sh->nonfinite[buf] = 1;
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    if (half == 0)
                        mbar_arrive(&sh->ext[s]);
                    else
                        mbar_arrive_cluster(cluster_map(&sh->ext[s], (uint32_t)lead));
                }
            }
            if (!ok) break;
            if (lane == 0) {
                mbar_arrive(&sh->ext_done[buf]);
                mbar_arrive(&sh->list_empty[buf]);
            }
            __syncwarp();
            if constexpr (CG == 2) {
                if (tile + tile_step < p.tiles) continue;
                // (A list of this tile says that the uses of its buffer before are
                // over, so the parity is of this one.)
                if (!(ok = lp_wait(&sh->acc_full[buf], (uint32_t)(ause & 1), abort_flag,
                                   p.wait_ns)) ||
                    !(ok = lp_wait(&sh->ext_done[buf], (uint32_t)(ause & 1), abort_flag,
                                   p.wait_ns)))
                    break;
                tc_fence_after();
                drain(buf, m0, n0, split, p.BN);
            }
        }
        if (CG == 2 && p.CK > 1 && !ok) cluster_arrive();
    }

    if (p.CK > 1 && (warp < 2 || (CG == 1 && warp > 5))) cluster_arrive();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (p.CK > 1) {
        // ------------------------------------------------------------ cluster sum
        // Each CTA adds up an equal part of the tile's columns (rows of y) from
        // the CK partial tiles of its rows of W, in order of K. Every CTA came
        // to the barrier before it read its tensor memory (one after that cost
        // 0.4 us more). The parts move by bulk copies from shared memory to
        // shared memory, one per pair of CTAs, behind the receiver's own
        // partial tile (128 rows of y of a tile of 256, two CTAs: loads from
        // the other CTA's shared memory took 4.5 us, at 7 bytes a cycle).
        cluster_wait();
        const int m0 = (first_tile / p.n_tiles * CG + half) * BM;
        const int n0 = first_tile % p.n_tiles * p.BN;
        const int cols = min(p.BN, p.R - n0);
        const int c0 = cols * rank / p.CK, c1 = cols * (rank + 1) / p.CK;
        const int most = (p.BN + p.CK - 1) / p.CK;
        float *part = reinterpret_cast<float *>(smem), *recv = part + p.BN * BM;
        if (tid == 0) {
            mbar_arrive_expect_tx(&sh->recv, (uint32_t)((p.CK - 1) * (c1 - c0) * BM * 4));
            for (int d = 1; d < p.CK; ++d) {
                const int k = rank + d < p.CK ? rank + d : rank + d - p.CK;
                const int b0 = cols * k / p.CK, b1 = cols * (k + 1) / p.CK;
                if (b1 > b0)
                    bulk_copy_peer(recv + (rank < k ? rank : rank - 1) * most * BM, part + b0 * BM,
                                   (uint32_t)((b1 - b0) * BM * 4), &sh->recv,
                                   (uint32_t)(k * CG + half));
            }
        }
        int patch = 0;
        for (int k = 0; k < p.CK; ++k)
            patch |= ld_dsmem_s32(cluster_map(&sh->nonfinite[0], (uint32_t)(k * CG + half)));
        lp_wait(&sh->recv, 0, abort_flag, p.wait_ns);
        const bool quads = (p.y_stride & 3) == 0 && (reinterpret_cast<uintptr_t>(p.y) & 7) == 0;
        // a warp takes a row of y, a lane 4 neighbouring columns of it (where
        // rows are 8-byte aligned, else every 32nd)
        const int step = quads ? 1 : 32, o2 = quads ? lane * 4 : lane;
        const int o = m0 + o2;
        for (int c = c0 + warp; c < c1; c += THREADS / 32) {
            float v[4] = {0.f, 0.f, 0.f, 0.f};
            for (int k = 0; k < p.CK; ++k) {
                const float *from = (k == rank ? part + c * BM
                                               : recv + ((k < rank ? k : k - 1) * most + c - c0) * BM) + o2;
                if (quads) {
                    const float4 t = *reinterpret_cast<const float4 *>(from);
                    v[0] += t.x, v[1] += t.y, v[2] += t.z, v[3] += t.w;
                } else {
#pragma unroll
                    for (int u = 0; u < 4; ++u) v[u] += from[u * 32];
                }
            }
            if (o >= p.O) continue;
            const int id = sh->ids[0][c], row = n0 + c;
            if (id == -2) v[0] = v[1] = v[2] = v[3] = 0.f;
            if (patch && id >= 0) {
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    if (o + u * step < p.O) v[u] += lp_nonfinite_terms(p, id, row, o + u * step);
            }
            __nv_bfloat16 *dst = p.y + (long long)row * p.y_stride + o;
            if (quads && o + 3 < p.O) {
                *reinterpret_cast<uint2 *>(dst) =
                    make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
            } else {
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    if (o + u * step < p.O) dst[u * step] = __float2bfloat16(v[u]);
            }
        }
    }
    // Leave only when every load that this CTA issued has landed, every commit
    // that frees one of its stages has arrived, and the others' partial sums,
    // which every CTA sends whatever became of them, are here. A tile that was
    // finished implies all three (its products are done, in both CTAs of a
    // pair); after a wait that gave up the barriers are waited for with a
    // limit, and 20 ms are left for what counts elsewhere: the loads of a
    // pair's second CTA (on the first one's barriers) and the last commit (on
    // acc_full). No CTA of a cluster leaves before the others have done this.
    if (*abort_flag && warp == 0 && lane == 0) {
        volatile int never = 0;
        for (int s = 0; s < S; ++s) {
            if (half == 0 && (sh->any_main >> s & 1u))
                mbar_wait_for(&sh->full[s], (sh->par_main >> s & 1u) ^ 1u, &never, 20000000ull);
            if (s < sh->committed)
                mbar_wait_for(&sh->empty[s], (uint32_t)((sh->committed - 1 - s) / S & 1), &never,
                              20000000ull);
        }
        if (p.CK > 1) mbar_wait_for(&sh->recv, 0, &never, 20000000ull);
        const unsigned long long t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 20000000ull) {
        }
    }
    __syncthreads();
    if (cluster > 1) {
        cluster_arrive();
        cluster_wait();
    }
    if (warp == 1) lp_tmem_dealloc<CG>(tmem, p.tmem_cols);
    if (tid == 0 && *abort_flag) atomicOr(p.status, SVF_DEV_TIMEOUT);
}

// ---------------------------------------------------------------- host side

static PFN_cuTensorMapEncodeTiled_v12000 lp_encoder() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000,
                                             cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
    });
    return fn;
}

// [rows, cols] bf16 with rows row_stride elements apart, in boxes of 64 columns
// x box_rows rows.
static bool lp_map(CUtensorMap *map, const void *base, long long rows, long long cols,
                   long long row_stride, int box_rows) {
    auto enc = lp_encoder();
    if (!enc) return false;
    cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)row_stride * 2};
    cuuint32_t box[2] = {(cuuint32_t)lp::BK, (cuuint32_t)box_rows};
    cuuint32_t estr[2] = {1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(base), dims, strides,
               box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool lora_proj_supported(int R, int H, int O, int adapters, int rank) {
    return R >= 1 && R <= (1 << 17) && H >= 8 && H % 8 == 0 && H <= (1 << 16) && O >= 1 &&
           O <= (1 << 20) && adapters >= 1 && adapters <= (1 << 16) && rank >= 8 &&
           rank % 8 == 0 && rank <= 128;
}

static size_t lp_smem(const LpParams &p, int cg) {
    return 1024 + (size_t)p.stages * (lp::A_BYTES + p.BN / cg * 128) + sizeof(LpShared);
}

// The limit that every call sets, so that calls of several host threads agree.
static constexpr size_t kLpMaxSmem = 1024 + lp::SMEM_BUDGET + sizeof(LpShared);

static void lp_stages(LpParams *p, int cg) {
    p->stages = lp::SMEM_BUDGET / (lp::A_BYTES + p->BN / cg * 128);
    if (p->stages > lp::MAX_STAGES) p->stages = lp::MAX_STAGES;
}

// What the kernel takes for granted of a way to cut a call into tiles: a ring
// within its budget that holds, where CTAs share K, a partial tile and the
// other CTAs' parts of one; adapter windows of half a tile; whole clusters.
static bool lp_fits(const LpParams &p, int cg) {
    if ((cg != 1 && cg != 2) || p.BN < 32 || p.BN > lp::MAX_BN || p.BN % 32 != 0 ||
        p.BN / 2 < 16 * cg || p.CK < 1 || p.CK > p.kblocks || p.CK * cg > 8 || p.stages < 2 ||
        p.stages > lp::MAX_STAGES)
        return false;
    const size_t ring = (size_t)p.stages * (lp::A_BYTES + p.BN / cg * 128);
    const size_t sums = (size_t)lp::BM * 4 * (p.BN + (p.CK - 1) * ((p.BN + p.CK - 1) / p.CK));
    return ring <= lp::SMEM_BUDGET && (p.CK == 1 || sums <= ring) &&
           (long long)p.n_tiles * p.BN >= p.R &&
           (long long)(p.tiles / p.n_tiles) * cg * lp::BM >= p.O;
}

// How a call is cut into tiles.
struct LpPlan {
    int cg, BN, n_tiles, tiles, stages, CK;
    int resident;  // clusters that fit at once
};

// Tiles of one CTA or a pair, rows of x per tile and CTAs (pairs) per tile: the
// least of a model of the call in ns. A block of K takes a CTA the longest of
// its products (1900 MHz), its share of what the L2 hands to the SMs (19 TB/s
// measured, 130 GB/s to one) and of HBM (7 TB/s), and the latency of a load
// (1.7 us) over the stages of its ring; an adapter block about 0.5 us, 0.8 in a
// pair (128 rows, 100 adapters of rank 16, 4096 -> 6144: single CTAs 29.9 us,
// pairs 33.5; 100 of rank 64, 8192 -> 10240: single CTAs 138, pairs 118). A tile
// begins with about 3.5 us and ends with its stores (12 ns a row of x), or with
// the sum over the cluster (30 ns a row); and a CTA costs 12 ns, as it leaves
// less of the GPU to lora_shrink (240 rows, 4096 -> 6144, rank 64: 96 CTAs 22.5
// us, 144 CTAs 26.1; without adapters 20.1 and 19.8).
static bool lp_make_plan(LpParams c, int groups, LpPlan *plan) {
    double least = 0;
    for (int cg = 1; cg <= 2; ++cg) {
        if (cg == 2 && (c.R <= 64 || c.O <= lp::BM)) break;
        auto kern = cg == 2 ? lora_proj_kernel<2> : lora_proj_kernel<1>;
        // one CTA alone takes more than 64 rows of x only where W has no second
        // tile for a pair
        const int widest = cg == 1 && c.O > lp::BM ? 64 : lp::MAX_BN;
        const int m_tiles = (c.O + cg * lp::BM - 1) / (cg * lp::BM);
        const int n_min = (c.R + widest - 1) / widest;
        for (int n = n_min; n <= n_min + (cg == 2 ? 3 : 0) && n <= 512; ++n) {
            c.BN = ((c.R + n - 1) / n + 31) / 32 * 32;
            if (n > n_min && c.BN < 96) break;
            c.n_tiles = (c.R + c.BN - 1) / c.BN;
            c.tiles = m_tiles * c.n_tiles;
            lp_stages(&c, cg);
            int most = groups < c.adapters ? groups : c.adapters;
            if (most > c.BN) most = c.BN;
            const int blocks = (((most - 1) >> c.lpack) + 1) * c.kchunks;
            const double bytes = lp::A_BYTES + c.BN / cg * 128;
            for (c.CK = 1; c.CK * cg <= 8 && c.CK <= c.kblocks; ++c.CK) {
                const int fit = resident_clusters(kern, lp::THREADS, kLpMaxSmem, c.CK * cg);
                if (fit < 1) continue;
                const int waves = (c.tiles + fit - 1) / fit;
                if (c.CK > 1 && waves > 1) continue;
                if (!lp_fits(c, cg)) continue;
                const double ctas = (double)(c.tiles < fit ? c.tiles : fit) * c.CK * cg;
                double kb = c.BN * 1.05;
                const double l2 = bytes * ctas / 19000, sm = bytes / 130;
                const double hbm = lp::A_BYTES * ctas / 7000 / c.n_tiles;
                if (l2 > kb) kb = l2;
                if (sm > kb) kb = sm;
                if (hbm > kb) kb = hbm;
                if (1700.0 / c.stages > kb) kb = 1700.0 / c.stages;
                const double t =
                    waves * ((c.kblocks * kb + blocks * (cg == 2 ? 800.0 : 500.0)) / c.CK + 3500) +
                    (c.CK > 1 ? 1500 + 30.0 * c.BN : 12.0 * c.BN) + 12 * ctas;
                if (least == 0 || t < least) {
                    least = t;
                    *plan = {cg, c.BN, c.n_tiles, c.tiles, c.stages, c.CK, fit};
                }
            }
        }
    }
    return least > 0;
}

// The plan of a shape on the current device, worked out once.
static bool lp_plan(const LpParams &p, int groups, LpPlan *plan) {
    static std::mutex mu;
    static std::map<std::tuple<int, int, int, int, int, int, int>, LpPlan> cache;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    const auto key = std::make_tuple(dev, p.R, p.H, p.O, p.rank, p.adapters, groups);
    std::lock_guard<std::mutex> lock(mu);
    const auto it = cache.find(key);
    if (it != cache.end()) {
        *plan = it->second;
        return true;
    }
    if (!lp_make_plan(p, groups, plan)) return false;
    if (cache.size() >= 4096) cache.clear();
    cache[key] = *plan;
    return true;
}

// A call's sizes and the way that it is cut into tiles; false if there is none,
// or one that the kernel does not take.
static bool lp_shape(int R, int per, int H, int O, int adapters, int rank, LpParams *p,
                     LpPlan *plan) {
    p->R = R;
    p->H = H;
    p->O = O;
    p->rank = rank;
    p->adapters = adapters;
    p->per = per;
    p->kblocks = (H + lp::BK - 1) / lp::BK;
    p->kchunks = (rank + lp::BK - 1) / lp::BK;
    p->lpack = rank <= 16 ? 2 : rank <= 32 ? 1 : 0;
    try {
        if (!lp_plan(*p, R / per, plan)) return false;
    } catch (...) {  // no host memory: no exception leaves a C entry
        return false;
    }
    p->BN = plan->BN;
    p->n_tiles = plan->n_tiles;
    p->tiles = plan->tiles;
    p->stages = plan->stages;
    p->CK = plan->CK;
    return lp_fits(*p, plan->cg) && plan->resident >= 1;
}

bool lora_proj_plan(int R, int per, int H, int O, int adapters, int rank, int32_t *plan) {
    LpParams p;
    LpPlan c;
    if (!lp_shape(R, per, H, O, adapters, rank, &p, &c)) return false;
    const int32_t v[6] = {c.cg, c.BN, c.CK, c.tiles, c.stages, c.resident};
    for (int i = 0; i < 6; ++i) plan[i] = v[i];
    return true;
}

static std::atomic<long long> g_lora_wait_ns{0};

void lora_proj_set_wait_ns(long long ns) { g_lora_wait_ns.store(ns > 0 ? ns : 0); }

int launch_lora_proj(const LoraArgs &a, cudaStream_t stream) {
    LpParams p;
    LpPlan plan;
    if (!lp_shape(a.R, a.rows_per_id, a.H, a.O, a.adapters, a.rank, &p, &plan))
        return SVF_ERR_LAUNCH;
    const int cg = plan.cg;
    auto kern = cg == 2 ? lora_proj_kernel<2> : lora_proj_kernel<1>;
    const size_t smem = lp_smem(p, cg);
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kLpMaxSmem) !=
        cudaSuccess)
        return SVF_ERR_LAUNCH;
    uint32_t cols = 32;
    while (cols < (uint32_t)((p.CK > 1 ? 1 : 2) * p.BN)) cols <<= 1;
    p.tmem_cols = cols;
    const long long wns = g_lora_wait_ns.load();
    p.wait_ns = wns > 0 ? (unsigned long long)wns : kWaitDeadlineNs;
    p.t = static_cast<const __nv_bfloat16 *>(a.workspace);
    p.ids = a.ids;
    p.lora_b = static_cast<const __nv_bfloat16 *>(a.lora_b);
    p.y = static_cast<__nv_bfloat16 *>(a.y);
    p.y_stride = a.y_stride;
    p.status = a.status;
    CUtensorMap tmw, tmx;
    if (!lp_map(&tmw, a.weight, a.O, a.H, a.H, lp::BM) ||
        !lp_map(&tmx, a.x, a.R, a.H, a.x_stride, p.BN / cg))
        return SVF_ERR_LAUNCH;
    if (launch_lora_shrink(a, p.wait_ns, stream) != cudaSuccess) return SVF_ERR_LAUNCH;
    int clusters = p.tiles;
    if (p.CK == 1 && clusters > plan.resident) clusters = plan.resident;  // persistent
    const int cluster = cg * p.CK;
    if (launch_pdl(kern, dim3((unsigned)(clusters * cluster)), dim3(lp::THREADS), smem, stream,
                   cluster > 1 ? (unsigned)cluster : 0u, tmw, tmx, p) != cudaSuccess)
        return SVF_ERR_LAUNCH;
    return SVF_OK;
}

}  // namespace svf
