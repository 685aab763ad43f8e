// lora_proj.cu -- a shared projection with a low-rank adapter per request:
//     y[r] = W x[r] + s_a B_a (A_a x[r]),   a = ids[r / rows_per_id]
// (a = -1: y[r] = W x[r]), bf16 operands and result, fp32 sums.
//
// lora_shrink.cu leaves t[r] = s_a A_a x[r] in fp32. Here the rest is ONE
// matrix product with a longer inner axis: to the H columns of x and W come,
// for every distinct adapter a of the row tile, rank columns that hold t on
// the rows of a (zero on the others) and B_a. So the adapters ride in the same
// tensor-memory accumulator as the shared product, and y is written once.
//   - t enters as two bf16 terms, hi + lo (16 bits of significand, error
//     2^-16 of t): one rounding to bf16 would add an error as large as the
//     result's own when the adapter's part dominates.
//   - A product of a zero of t with an infinity or NaN of another request's
//     B_a would be NaN. Every B_a tile is looked over in shared memory before
//     its products: non-finite elements are replaced by zero there, and their
//     terms are added to the rows of a alone, in the epilogue.
//   - The tensor-core work of an adapter is confined to the window of the tile
//     that holds its rows (the MMA's N: steps of 16 rows, of 32 for a pair of
//     CTAs), and a 64-column
//     block carries as many adapters as fit: 4 of rank <= 16 (tiles of 32-byte
//     rows), 2 of rank <= 32 (64 bytes), else one (128 bytes).
//
// W's rows are the MMA's M axis (128 per CTA), the rows of x its N axis (tiles
// of BN <= 256), K in blocks of 64 staged by TMA with 128-byte swizzle.
// CG = 2: two CTAs of a cluster work on one tile of 256 rows of W
// (cta_group::2), each loads its own 128 rows of W and half of the x tile, and
// the first one issues the products for both. One CTA alone would have to
// bring 48 KB into shared memory per 128 x 256 x 64 block, and shared memory
// would be what bounds it; the pair brings 32 KB each. CG = 1 serves few rows
// (bound by the bytes of W), where two CTAs per SM keep more loads in flight.
// Roles of a CTA (320 threads):
//   warp 0      producer: TMA of W and x blocks, then of B_a blocks;
//   warp 1      MMA issuer (of the pair's first CTA);
//   warps 2-5   epilogue (tensor memory -> y);
//   warps 6-9   adapters: warp 6 lists the tile's distinct adapters; all four
//               wait for a block's B_a tiles, look them over, and write t's hi
//               and lo next to them.
// The t columns come last, so the shared product runs while lora_shrink still
// does (the launches overlap; only warps 6-9 wait for it).
//
// Few rows leave too few tiles for the SMs: CK CTAs (or pairs) of a cluster
// then share a tile, each with an equal part of K and every CK-th adapter
// block, and their sums meet over distributed shared memory in a fixed order.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <mutex>

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
constexpr int ADAPTER_THREADS = 128;
constexpr int MAX_BN = 256;
constexpr int MAX_LIST = 2 * MAX_BN;    // adapter windows of one row tile
constexpr int SMEM_ONE = 192 * 1024;    // stage ring of a CTA that has its SM alone
constexpr int SMEM_TWO = 88 * 1024;     // ... that shares its SM with another
}  // namespace lp

struct LpParams {
    int R, H, O, rank, adapters, per;
    int BN, CK, n_tiles, tiles, kblocks, stages;
    int kchunks;    // 64-column blocks of one adapter (rank > 64: 2)
    int pack;       // adapters of one block: 4, 2 or 1
    uint32_t tmem_cols;
    unsigned long long wait_ns;
    const float *t;
    const int32_t *ids;
    const __nv_bfloat16 *lora_b;
    __nv_bfloat16 *y;
    long long y_stride;
    int32_t *status;
};

// Shared memory behind the stage ring.
struct LpShared {
    uint64_t full[lp::MAX_STAGES];   // a block of W and x has landed (in the pair's first CTA)
    uint64_t bfull[lp::MAX_STAGES];  // a block of B_a has landed
    uint64_t ext[lp::MAX_STAGES];    // ... is looked over, and t stands next to it (first CTA)
    uint64_t empty[lp::MAX_STAGES];
    uint64_t acc_full[2], acc_empty[2], list_full[2], list_empty[2], ext_done[2];
    int ids[2][lp::MAX_BN];     // adapter of each row of the tile; -1 none, -2 a bad id
    int2 list[2][lp::MAX_LIST]; // adapter; first row and row count of its window
    int n_list[2];
    int nonfinite[2];
    uint32_t tmem;
    int committed;  // stages whose products were issued
    int abort;
};

__device__ __forceinline__ bool lp_wait(uint64_t *bar, uint32_t parity, volatile int *abort,
                                        unsigned long long ns) {
    const bool ok = mbar_wait_for(bar, parity, abort, ns);
    return __all_sync(0xffffffffu, ok);
}

// The same for a barrier that another CTA's threads arrive on.
__device__ __forceinline__ bool lp_wait_cluster(uint64_t *bar, uint32_t parity,
                                                volatile int *abort, unsigned long long ns) {
    bool ok = mbar_try_wait_cluster(bar, parity);
    if (!ok) {
        const unsigned long long t0 = globaltimer_ns();
        for (uint32_t it = 1;; ++it) {
            if ((ok = mbar_try_wait_cluster(bar, parity))) break;
            if ((it & 63u) == 0) {
                if (*abort) break;
                if (globaltimer_ns() - t0 > ns) {
                    *abort = 1;
                    break;
                }
            }
        }
    }
    return __all_sync(0xffffffffu, ok);
}

// Arrive on a barrier of another CTA of the cluster (an address from cluster_map).
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t remote) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(remote)
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
// Byte offset of 16-byte chunk c of row `row` in such a tile.
__device__ __forceinline__ int lp_swizzled(int row, int c, int row_bytes) {
    const int sh = row_bytes == 128 ? 0 : row_bytes == 64 ? 1 : 2;
    return row * row_bytes + ((c ^ ((row >> sh) & (row_bytes / 16 - 1))) << 4);
}

__device__ __forceinline__ bool bf16_nonfinite2(uint32_t w) {
    return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
}

// The distinct adapters of rows [n0, n0 + BN), in order of first appearance,
// each with the window of the tile that holds its rows (16 CG rows aligned),
// in pieces of at most BN / 2 rows. One warp. At most 3 pieces for an adapter
// of two rows or more and one for the others: 1.5 BN in all.
template <int CG>
__device__ void lp_build_list(const LpParams &p, LpShared *sh, int buf, int n0, int lane) {
    constexpr int G = 16 * CG;
    int v[lp::MAX_BN / 32];
    const int chunks = p.BN / 32;
#pragma unroll
    for (int c = 0; c < lp::MAX_BN / 32; ++c) {
        v[c] = -1;
        if (c < chunks) {
            const int row = n0 + c * 32 + lane;
            if (row < p.R) {
                const int id = p.ids[row / p.per];
                v[c] = id < -1 || id >= p.adapters ? -2 : id;
            }
            sh->ids[buf][c * 32 + lane] = v[c];
        }
    }
    __syncwarp();
    int n = 0;
    // only the first row of a group can be the first of an adapter
    int i = 0;
    while (i < p.BN && n0 + i < p.R) {
        const int id = sh->ids[buf][i];
        if (id >= 0) {
            int first = -1, last = -1;
#pragma unroll
            for (int c = 0; c < lp::MAX_BN / 32; ++c) {
                const unsigned m = __ballot_sync(0xffffffffu, v[c] == id);
                if (m) {
                    if (first < 0) first = c * 32 + __ffs(m) - 1;
                    last = c * 32 + 31 - __clz(m);
                }
            }
            if (first == i) {
                int w0 = first & ~(G - 1);
                const int w1 = (last + G) & ~(G - 1);
                const int most = (p.BN / 2) & ~(G - 1);
                while (w0 < w1) {
                    const int len = min(w1 - w0, most);
                    if (lane == 0) sh->list[buf][n] = make_int2(id, w0 | len << 16);
                    ++n;
                    w0 += len;
                }
            }
        }
        i += p.per - (n0 + i) % p.per;
    }
    if (lane == 0) {
        sh->n_list[buf] = n;
        sh->nonfinite[buf] = 0;
    }
    __syncwarp();
}

// The terms of non-finite elements of the row's own B_a, from memory.
__device__ __noinline__ float lp_nonfinite_terms(const LpParams &p, int id, int row, int o) {
    const __nv_bfloat16 *b = p.lora_b + ((size_t)id * p.O + o) * (size_t)p.rank;
    const float *t = p.t + (size_t)row * p.rank;
    float v = 0.f;
    for (int j = 0; j < p.rank; ++j) {
        const float f = __bfloat162float(b[j]);
        if (!isfinite(f)) v += __ldcg(t + j) * f;
    }
    return v;
}

// 32 columns of a tile that met non-finite elements of some B_a.
__device__ __noinline__ void lp_store_patched(const LpParams &p, const int *ids, const uint32_t *r,
                                              int rows_left, int row0, int o) {
    for (int j = 0; j < 32 && j < rows_left; ++j) {
        float v = ids[j] == -2 ? 0.f : __uint_as_float(r[j]);
        if (ids[j] >= 0) v += lp_nonfinite_terms(p, ids[j], row0 + j, o);
        p.y[(long long)(row0 + j) * p.y_stride + o] = __float2bfloat16(v);
    }
}

// Replaces the non-finite elements of 8 bf16 values by zero; true if there were any.
__device__ __forceinline__ bool lp_clean(uint4 *at) {
    const uint4 b = *at;
    if (!(bf16_nonfinite2(b.x) | bf16_nonfinite2(b.y) | bf16_nonfinite2(b.z) |
          bf16_nonfinite2(b.w)))
        return false;
    uint32_t wd[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if ((wd[k] & 0x7f80u) == 0x7f80u) wd[k] &= 0xffff0000u;
        if ((wd[k] & 0x7f800000u) == 0x7f800000u) wd[k] &= 0xffffu;
    }
    *at = make_uint4(wd[0], wd[1], wd[2], wd[3]);
    return true;
}

template <int CG>
__global__ void __launch_bounds__(lp::THREADS, CG == 1 ? 2 : 1)
    lora_proj_kernel(const __grid_constant__ CUtensorMap tmw, const __grid_constant__ CUtensorMap tmx,
                     const __grid_constant__ CUtensorMap tmb, LpParams p) {
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
    const int row_bytes = 128 / p.pack, tile_bytes = BM * row_bytes;

    if (tid == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(&sh->full[s], 1);
            mbar_init(&sh->bfull[s], 1);
            mbar_init(&sh->ext[s], 4 * CG);
            mbar_init(&sh->empty[s], 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(&sh->acc_full[a], 1);
            mbar_init(&sh->acc_empty[a], 4 * CG);
            mbar_init(&sh->list_full[a], 1);
            mbar_init(&sh->list_empty[a], 10);  // warps 0, 1, 2-5, 6-9
            mbar_init(&sh->ext_done[a], 4);
        }
        sh->committed = 0;
        sh->abort = 0;
        mbar_fence_init();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&tmw);
        tma_prefetch_desc(&tmx);
        tma_prefetch_desc(&tmb);
    }
    if (warp == 1) lp_tmem_alloc<CG>(&sh->tmem, p.tmem_cols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (CG == 2) {  // the other CTA's barriers exist before anything arrives on them
        cluster_arrive();
        cluster_wait();
    }
    // Only t waits for the kernel before this one (warps 6-9 below): that
    // kernel lets this one start after its own wait, so what this call reads
    // besides t was complete by then.
    pdl_launch_dependents();
    const uint32_t tmem = sh->tmem;
    int issued = 0;  // producer: stages loaded
    // A stage's full barrier counts its W and x blocks, its bfull barrier its
    // B_a blocks; who waits for one keeps the parity of its next phase, one
    // bit per stage.
    uint32_t par_main = 0, par_ext = 0;
    uint32_t any_main = 0, any_ext = 0;

    if (warp == 0) {
        // ------------------------------------------------------------ producer
        bool ok = true;
        int i = 0;
        const int rot = (int)((long long)first_tile * nkb / tile_step) % nkb;
        for (int tile = first_tile; tile < p.tiles && ok; tile += tile_step, ++i) {
            const int m0 = (tile / p.n_tiles * CG + half) * BM;
            const int n0 = tile % p.n_tiles * p.BN + half * (p.BN / 2);
            for (int kb = 0; kb < nkb; ++kb, ++issued) {
                const int s = issued % S, use = issued / S;
                // tiles that start together start at different columns
                const int kc = (kb0 + (kb + rot < nkb ? kb + rot : kb + rot - nkb)) * BK;
                if (use > 0 && !(ok = lp_wait(&sh->empty[s], (uint32_t)((use - 1) & 1),
                                              abort_flag, p.wait_ns)))
                    break;
                if (lane == 0) {
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
                }
                par_main ^= 1u << s;
                any_main |= 1u << s;
                __syncwarp();
            }
            if (!ok) break;
            const int buf = i & 1;
            if (!(ok = lp_wait(&sh->list_full[buf], (uint32_t)(i >> 1 & 1), abort_flag,
                               p.wait_ns)))
                break;
            const int n_list = sh->n_list[buf];
            const int blocks = (n_list + p.pack - 1) / p.pack * p.kchunks;
            for (int x = rank; x < blocks; x += p.CK, ++issued) {
                const int e0 = x / p.kchunks * p.pack, kc = x % p.kchunks;
                const int ne = min(p.pack, n_list - e0);
                const int s = issued % S, use = issued / S;
                if (use > 0 && !(ok = lp_wait(&sh->empty[s], (uint32_t)((use - 1) & 1),
                                              abort_flag, p.wait_ns)))
                    break;
                if (lane == 0) {
                    mbar_arrive_expect_tx(&sh->bfull[s], (uint32_t)(ne * tile_bytes));
                    for (int e = 0; e < ne; ++e)
                        tma_load_3d(sA + s * A_BYTES + e * tile_bytes, &tmb, kc * BK, m0,
                                    sh->list[buf][e0 + e].x, &sh->bfull[s]);
                }
                par_ext ^= 1u << s;
                any_ext |= 1u << s;
                __syncwarp();
            }
            if (lane == 0) mbar_arrive(&sh->list_empty[buf]);
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer
        bool ok = true;
        int it = 0, i = 0;
        const uint32_t idesc = idesc_bf16_f32(BM * CG, p.BN, false, false);
        for (int tile = first_tile; tile < p.tiles && ok; tile += tile_step, ++i) {
            const int buf = i & 1, ause = i >> 1;
            if (half == 0) {
                if (ause > 0 &&
                    !(ok = lp_wait_cluster(&sh->acc_empty[buf], (uint32_t)((ause - 1) & 1),
                                           abort_flag, p.wait_ns)))
                    break;
                tc_fence_after();
                const uint32_t d = tmem + (uint32_t)(buf * p.BN);
                for (int kb = 0; kb < nkb; ++kb, ++it) {
                    const int s = it % S;
                    if (!(ok = lp_wait(&sh->full[s], par_main >> s & 1u, abort_flag, p.wait_ns)))
                        break;
                    par_main ^= 1u << s;
                    tc_fence_after();
                    if (lane == 0) {
                        const uint32_t a = smem_u32(sA + s * A_BYTES);
                        const uint32_t b = smem_u32(sB + s * b_bytes);
#pragma unroll
                        for (int k = 0; k < BK / 16; ++k)
                            lp_mma<CG>(d, smem_desc_sw128(a + k * 32, 16, 1024),
                                       smem_desc_sw128(b + k * 32, 16, 1024), idesc,
                                       (kb > 0 || k > 0) ? 1u : 0u);
                        lp_commit<CG>(&sh->empty[s], pair_mask);
                    }
                    __syncwarp();
                }
                if (!ok) break;
            }
            if (!(ok = lp_wait(&sh->list_full[buf], (uint32_t)(ause & 1), abort_flag, p.wait_ns)))
                break;
            if (half == 0) {
                const uint32_t d = tmem + (uint32_t)(buf * p.BN);
                const int n_list = sh->n_list[buf];
                const int blocks = (n_list + p.pack - 1) / p.pack * p.kchunks;
                const uint32_t slot_bytes = (uint32_t)(b_bytes / 2 / p.pack);
                for (int x = rank; x < blocks; x += p.CK, ++it) {
                    const int e0 = x / p.kchunks * p.pack, kc = x % p.kchunks;
                    const int ne = min(p.pack, n_list - e0);
                    const int s = it % S;
                    if (!(ok = lp_wait_cluster(&sh->ext[s], par_ext >> s & 1u, abort_flag,
                                               p.wait_ns)))
                        break;
                    par_ext ^= 1u << s;
                    tc_fence_after();
                    if (lane == 0) {
                        const int ksteps = (min(p.rank - kc * BK, BK) + 15) / 16;
                        for (int e = 0; e < ne; ++e) {
                            const int w = sh->list[buf][e0 + e].y;
                            const uint32_t dw = d + (uint32_t)(w & 0xffff);
                            const uint32_t idw = idesc_bf16_f32(BM * CG, w >> 16, false, false);
                            const uint32_t a = smem_u32(sA + s * A_BYTES + e * tile_bytes);
                            const uint32_t hi = smem_u32(sB + s * b_bytes) + e * slot_bytes;
                            const uint32_t lo = hi + (uint32_t)b_bytes / 2;
                            for (int k = 0; k < ksteps; ++k) {
                                const uint64_t da = lp_desc(a + k * 32, row_bytes);
                                lp_mma<CG>(dw, da, lp_desc(hi + k * 32, row_bytes), idw, 1u);
                                lp_mma<CG>(dw, da, lp_desc(lo + k * 32, row_bytes), idw, 1u);
                            }
                        }
                        lp_commit<CG>(&sh->empty[s], pair_mask);
                    }
                    __syncwarp();
                }
                if (!ok) break;
                if (lane == 0) lp_commit<CG>(&sh->acc_full[buf], pair_mask);
            }
            if (lane == 0) mbar_arrive(&sh->list_empty[buf]);
            __syncwarp();
        }
        if (lane == 0) sh->committed = it;
    } else if (warp < 6) {
        // ------------------------------------------------------------ epilogue
        const int q = warp & 3;  // tensor-memory lanes 32 q .. 32 q + 31
        const uint32_t lane_base = (uint32_t)(q * 32) << 16;
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
            const int o = m0 + q * 32 + lane;
            const bool o_ok = o < p.O;
            const bool patch = sh->nonfinite[buf] != 0;
            if (p.CK > 1) {
                // partial sums into the (now idle) stage ring, [column][128] fp32
                float *part = reinterpret_cast<float *>(smem) + q * 32 + lane;
                for (int c = 0; c < p.BN; c += 32) {
                    uint32_t r[32];
                    tmem_ld32(tmem + lane_base + (uint32_t)(buf * p.BN + c), r);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 32; ++j) part[(c + j) * BM] = __uint_as_float(r[j]);
                }
            } else {
                __nv_bfloat16 *col = p.y + o;
                for (int c = 0; c < p.BN; c += 32) {
                    uint32_t r[32];
                    tmem_ld32(tmem + lane_base + (uint32_t)(buf * p.BN + c), r);
                    tmem_wait_ld();
                    const int rows_left = p.R - (n0 + c);
                    if (!o_ok) continue;
                    if (patch) {
                        uint32_t v[32];
#pragma unroll
                        for (int j = 0; j < 32; ++j) v[j] = r[j];
                        lp_store_patched(p, sh->ids[buf] + c, v, rows_left, n0 + c, o);
                        continue;
                    }
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (j < rows_left) {
                            const float v =
                                sh->ids[buf][c + j] == -2 ? 0.f : __uint_as_float(r[j]);
                            col[(long long)(n0 + c + j) * p.y_stride] = __float2bfloat16(v);
                        }
                }
            }
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
    } else {
        // ------------------------------------------------------------ adapters
        const int at = tid - (THREADS - ADAPTER_THREADS);
        // a block's adapters are shared out among 4 / pack warps each
        const int group = ADAPTER_THREADS / p.pack, e = at / group, ti = at % group;
        bool ok = true;
        int it = 0, i = 0;
        bool waited = false;
        for (int tile = first_tile; tile < p.tiles && ok; tile += tile_step, ++i) {
            const int n0 = tile % p.n_tiles * p.BN;
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
            const int n_list = sh->n_list[buf];
            if (!waited) {
                pdl_wait();  // t is complete
                waited = true;
            }
            it += nkb;
            const int blocks = (n_list + p.pack - 1) / p.pack * p.kchunks;
            for (int x = rank; x < blocks; x += p.CK, ++it) {
                const int e0 = x / p.kchunks * p.pack, kc = x % p.kchunks;
                const bool mine = e0 + e < n_list;
                const int2 entry = sh->list[buf][mine ? e0 + e : e0];
                // this CTA's rows of the window: all, or its half of them
                const int rows = (entry.y >> 16) / CG;
                const int w0 = (entry.y & 0xffff) + half * rows;
                const int rc = min(p.rank - kc * BK, BK);  // columns, a multiple of 8
                const int nch = (rc + 15) / 16 * 2;        // 16-byte chunks of a row of t
                const int units = mine ? rows * nch : 0;
                auto load_t = [&](int u, float *f) {
                    const int row = u / nch, c = u % nch;
#pragma unroll
                    for (int k = 0; k < 8; ++k) f[k] = 0.f;
                    if (u < units && c * 8 < rc && sh->ids[buf][w0 + row] == entry.x) {
                        const float4 *src = reinterpret_cast<const float4 *>(
                            p.t + (size_t)(n0 + w0 + row) * p.rank + kc * BK + c * 8);
                        *reinterpret_cast<float4 *>(f) = __ldcg(src);
                        *reinterpret_cast<float4 *>(f + 4) = __ldcg(src + 1);
                    }
                };
                float f[2][8];
                load_t(ti, f[0]);
                load_t(ti + group, f[1]);
                const int s = it % S;
                if (!(ok = lp_wait(&sh->bfull[s], par_ext >> s & 1u, abort_flag, p.wait_ns)))
                    break;
                par_ext ^= 1u << s;
                if (mine) {
                    uint8_t *tile_b = sA + s * A_BYTES + e * tile_bytes;
                    bool bad = false;
                    for (int row = ti; row < BM; row += group)
                        for (int c = 0; c < rc / 8; ++c)
                            bad |= lp_clean(reinterpret_cast<uint4 *>(
                                tile_b + lp_swizzled(row, c, row_bytes)));
                    if (bad) sh->nonfinite[buf] = 1;
                }
                // t of the window: hi in the first half of the stage's x area,
                // lo in the second
                uint8_t *hi = sB + s * b_bytes + e * (b_bytes / 2 / p.pack);
                uint8_t *lo = hi + b_bytes / 2;
                for (int u = ti; u < units; u += 2 * group) {
                    if (u != ti) {
                        load_t(u, f[0]);
                        load_t(u + group, f[1]);
                    }
#pragma unroll
                    for (int v = 0; v < 2; ++v) {
                        if (u + v * group >= units) break;
                        uint32_t h[4], l[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            h[k] = pack_bf16x2(f[v][2 * k], f[v][2 * k + 1]);
                            const float h0 = __uint_as_float(h[k] << 16);
                            const float h1 = __uint_as_float(h[k] & 0xffff0000u);
                            // an infinite hi has no remainder
                            l[k] = pack_bf16x2(isfinite(h0) ? f[v][2 * k] - h0 : 0.f,
                                               isfinite(h1) ? f[v][2 * k + 1] - h1 : 0.f);
                        }
                        const int off = lp_swizzled((u + v * group) / nch, (u + v * group) % nch,
                                                    row_bytes);
                        *reinterpret_cast<uint4 *>(hi + off) = make_uint4(h[0], h[1], h[2], h[3]);
                        *reinterpret_cast<uint4 *>(lo + off) = make_uint4(l[0], l[1], l[2], l[3]);
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    if (half == 0)
                        mbar_arrive(&sh->ext[s]);
                    else
                        mbar_arrive_cluster(cluster_map(&sh->ext[s], (uint32_t)lead));
                }
            }
            if (lane == 0) {
                mbar_arrive(&sh->ext_done[buf]);
                mbar_arrive(&sh->list_empty[buf]);
            }
            __syncwarp();
        }
        if (!waited) pdl_wait();
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (p.CK > 1) {
        // ------------------------------------------------------------ cluster sum
        // Each CTA adds up an equal part of the tile's columns (rows of y)
        // from the CK partial tiles of its rows of W, in order of K.
        cluster_arrive();
        cluster_wait();
        const int m0 = (first_tile / p.n_tiles * CG + half) * BM;
        const int n0 = first_tile % p.n_tiles * p.BN;
        const int c0 = p.BN * rank / p.CK, c1 = p.BN * (rank + 1) / p.CK;
        int patch = 0;
        for (int k = 0; k < p.CK; ++k)
            patch |= ld_dsmem_s32(cluster_map(&sh->nonfinite[0], (uint32_t)(k * CG + half)));
        const bool pair = (p.y_stride & 1) == 0 &&
                          (reinterpret_cast<uintptr_t>(p.y) & 3) == 0;
        const float *part = reinterpret_cast<const float *>(smem);
        for (int u = tid; u < (c1 - c0) * (BM / 2); u += THREADS) {
            const int c = c0 + u / (BM / 2), o2 = u % (BM / 2) * 2;
            const int row = n0 + c, o = m0 + o2;
            if (row >= p.R || o >= p.O) continue;
            float a = 0.f, b = 0.f;
            for (int k = 0; k < p.CK; ++k) {
                const uint32_t src = cluster_map(part + c * BM + o2, (uint32_t)(k * CG + half));
                a += ld_dsmem_f32(src);
                b += ld_dsmem_f32(src + 4);
            }
            const int id = sh->ids[0][c];
            if (id == -2) a = b = 0.f;
            if (patch && id >= 0) {
                a += lp_nonfinite_terms(p, id, row, o);
                if (o + 1 < p.O) b += lp_nonfinite_terms(p, id, row, o + 1);
            }
            __nv_bfloat16 *dst = p.y + (long long)row * p.y_stride + o;
            if (pair && o + 1 < p.O) {
                *reinterpret_cast<uint32_t *>(dst) = pack_bf16x2(a, b);
            } else {
                dst[0] = __float2bfloat16(a);
                if (o + 1 < p.O) dst[1] = __float2bfloat16(b);
            }
        }
    }
    // Leave only when every load that this CTA issued has landed and every
    // commit that frees one of its stages has arrived. A tile that was
    // finished implies both (its products are done, in both CTAs of a pair);
    // after a wait that gave up the barriers are waited for with a limit, and
    // a pair, whose loads count on the first CTA's barriers, leaves 20 ms for
    // them to land.
    if (*abort_flag && warp == 0 && lane == 0) {
        volatile int never = 0;
        for (int s = 0; s < S; ++s) {
            if (half == 0 && (any_main >> s & 1u))
                mbar_wait_for(&sh->full[s], (par_main >> s & 1u) ^ 1u, &never, 20000000ull);
            if (any_ext >> s & 1u)
                mbar_wait_for(&sh->bfull[s], (par_ext >> s & 1u) ^ 1u, &never, 20000000ull);
            if (s < sh->committed)
                mbar_wait_for(&sh->empty[s], (uint32_t)((sh->committed - 1 - s) / S & 1), &never,
                              20000000ull);
        }
        const unsigned long long t0 = globaltimer_ns();
        while (CG == 2 && globaltimer_ns() - t0 < 20000000ull) {
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

// [planes, rows, cols] bf16 with the given strides (elements); boxes of
// box_cols columns (32, 64 or 128 bytes, swizzled over as many) x box_rows
// rows of one plane. dims == 2: one plane.
static bool lp_map(CUtensorMap *map, const void *base, int dims, long long planes, long long rows,
                   long long cols, long long row_stride, long long plane_stride, int box_cols,
                   int box_rows) {
    auto enc = lp_encoder();
    if (!enc) return false;
    cuuint64_t d[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)planes};
    cuuint64_t strides[2] = {(cuuint64_t)row_stride * 2, (cuuint64_t)plane_stride * 2};
    cuuint32_t box[3] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows, 1};
    cuuint32_t estr[3] = {1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)dims, const_cast<void *>(base), d,
               strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               box_cols == 64   ? CU_TENSOR_MAP_SWIZZLE_128B
               : box_cols == 32 ? CU_TENSOR_MAP_SWIZZLE_64B
                                : CU_TENSOR_MAP_SWIZZLE_32B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool lora_proj_supported(int R, int H, int O, int adapters, int rank) {
    return R >= 1 && R <= (1 << 20) && H >= 8 && H % 8 == 0 && H <= (1 << 16) && O >= 1 &&
           O <= (1 << 20) && adapters >= 1 && adapters <= (1 << 16) && rank >= 8 &&
           rank % 8 == 0 && rank <= 128;
}

static size_t lp_smem(const LpParams &p, int cg) {
    return 1024 + (size_t)p.stages * (lp::A_BYTES + p.BN / cg * 128) + sizeof(LpShared);
}

static void lp_stages(LpParams *p, int cg, int budget) {
    p->stages = budget / (lp::A_BYTES + p->BN / cg * 128);
    if (p->stages > lp::MAX_STAGES) p->stages = lp::MAX_STAGES;
}

int launch_lora_proj(const LoraArgs &a, cudaStream_t stream) {
    LpParams p;
    p.R = a.R;
    p.H = a.H;
    p.O = a.O;
    p.rank = a.rank;
    p.adapters = a.adapters;
    p.per = a.rows_per_id;
    p.kblocks = (a.H + lp::BK - 1) / lp::BK;
    p.kchunks = (a.rank + lp::BK - 1) / lp::BK;
    p.pack = a.rank <= 16 ? 4 : a.rank <= 32 ? 2 : 1;
    const int sms = num_sms();
    const int cg = a.R > 64 && a.O > lp::BM ? 2 : 1;
    const int m_tiles = (a.O + cg * lp::BM - 1) / (cg * lp::BM);
    // rows of x per tile: the fewest waves of tiles over the SMs, each as
    // long as its rows (and a constant share)
    const int n_min = (a.R + lp::MAX_BN - 1) / lp::MAX_BN;
    long long best = 0;
    for (int n = n_min; n <= n_min + 3; ++n) {
        const int bn = ((a.R + n - 1) / n + 31) / 32 * 32;
        const int nt = (a.R + bn - 1) / bn;
        const long long waves = ((long long)m_tiles * nt * cg + sms - 1) / sms;
        const long long cost = waves * (bn + 16);
        if (n == n_min || cost < best) {
            best = cost;
            p.BN = bn;
            p.n_tiles = nt;
        }
        if (bn <= 128) break;
    }
    p.tiles = m_tiles * p.n_tiles;
    lp_stages(&p, cg, cg == 1 && p.BN <= 64 ? lp::SMEM_TWO : lp::SMEM_ONE);
    const size_t smem = lp_smem(p, cg);
    // CTAs (pairs) per tile, from the clusters that can be resident at once:
    // the waves, each as long as a CTA's blocks of K and of adapters, about 8
    // blocks' time from launch to the first product and to the last store, and
    // about 4 for the sum over the cluster
    auto kern = cg == 2 ? lora_proj_kernel<2> : lora_proj_kernel<1>;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) !=
        cudaSuccess)
        return SVF_ERR_LAUNCH;
    const int groups = a.R / a.rows_per_id;
    int most = groups < a.adapters ? groups : a.adapters;
    if (most > p.BN) most = p.BN;
    const int work = p.kblocks + most / p.pack * p.kchunks;
    double least = 0;
    int resident = 1;
    p.CK = 1;
    for (int c = 1; c * cg <= 8 && c <= p.kblocks; ++c) {
        int fit = resident_clusters(kern, lp::THREADS, smem, c * cg);
        if (fit < 1) fit = c == 1 ? sms / cg : 0;
        if (fit < 1) continue;
        const double waves = (p.tiles + fit - 1) / fit;
        const double t = waves * ((double)work / c + 8 + (c > 1 ? 4 : 0));
        if (c == 1 || t < least) {
            least = t;
            p.CK = c;
            resident = fit;
        }
    }
    uint32_t cols = 32;
    while (cols < (uint32_t)(2 * p.BN)) cols <<= 1;
    p.tmem_cols = cols;
    p.wait_ns = kWaitDeadlineNs;
    p.t = static_cast<const float *>(a.workspace);
    p.ids = a.ids;
    p.lora_b = static_cast<const __nv_bfloat16 *>(a.lora_b);
    p.y = static_cast<__nv_bfloat16 *>(a.y);
    p.y_stride = a.y_stride;
    p.status = a.status;
    CUtensorMap tmw, tmx, tmb;
    if (!lp_map(&tmw, a.weight, 2, 1, a.O, a.H, a.H, 0, 64, lp::BM) ||
        !lp_map(&tmx, a.x, 2, 1, a.R, a.H, a.x_stride, 0, 64, p.BN / cg) ||
        !lp_map(&tmb, a.lora_b, 3, a.adapters, a.O, a.rank, a.rank, (long long)a.O * a.rank,
                64 / p.pack, lp::BM))
        return SVF_ERR_LAUNCH;
    if (launch_lora_shrink(a, stream) != cudaSuccess) return SVF_ERR_LAUNCH;
    int clusters = p.tiles;
    if (p.CK == 1 && clusters > resident) clusters = resident;  // persistent
    const int cluster = cg * p.CK;
    if (launch_pdl(kern, dim3((unsigned)(clusters * cluster)), dim3(lp::THREADS), smem, stream,
                   cluster > 1 ? (unsigned)cluster : 0u, tmw, tmx, tmb, p) != cudaSuccess)
        return SVF_ERR_LAUNCH;
    return SVF_OK;
}

}  // namespace svf
