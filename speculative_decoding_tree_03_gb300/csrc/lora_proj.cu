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
//     2^-17 of t): one rounding to bf16 would add an error as large as the
//     result's own when the adapter's part dominates.
//   - A product of a zero of t with an infinity or NaN of another request's
//     B_a would be NaN. Every B_a tile is looked over in shared memory before
//     its products: non-finite elements are replaced by zero there, and their
//     terms are added to the rows of a alone, in the epilogue.
//
// W's rows are the MMA's M axis (tiles of 128), the rows of x its N axis
// (tiles of BN <= 256), K in blocks of 64 staged by TMA with 128-byte swizzle.
// Roles of a CTA (320 threads):
//   warp 0      producer: TMA of W and x blocks, then of B_a blocks;
//   warp 1      MMA issuer;
//   warps 2-5   epilogue (tensor memory -> y);
//   warps 6-9   adapters: warp 6 lists the tile's distinct adapters; each of
//               the four takes the adapter blocks of every fourth stage: it
//               waits for the B_a tile, looks it over, and writes t's hi and lo
//               next to it.
// The t columns come last, so the shared product runs while lora_shrink still
// does (the launches overlap; only warps 6-9 wait for it).
//
// Few rows leave too few tiles for the SMs: CK CTAs (a cluster) then share a
// tile, each with an equal part of K and every CK-th adapter, and their sums
// meet over distributed shared memory in a fixed order.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <mutex>

#include "common.cuh"
#include "internal.h"
#include "lora.h"

namespace svf {

namespace lp {
constexpr int BM = 128;                 // rows of W per tile (MMA M)
constexpr int BK = 64;                  // K per stage: one 128-byte swizzle row
constexpr int A_BYTES = BM * BK * 2;
constexpr int MAX_STAGES = 12;
constexpr int THREADS = 320;
constexpr int MAX_BN = 256;
constexpr int MAX_LIST = 2 * MAX_BN;    // adapter windows of one row tile
constexpr int SMEM_BUDGET = 188 * 1024; // stage ring; lora_shrink keeps room beside it
}  // namespace lp

struct LpParams {
    int R, H, O, rank, adapters, per;
    int BN, CK, n_tiles, tiles, kblocks, kchunks, stages;
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
    uint64_t full[lp::MAX_STAGES];   // a block of W and x has landed
    uint64_t bfull[lp::MAX_STAGES];  // a block of B_a has landed
    uint64_t ext[lp::MAX_STAGES];    // ... is looked over, and t stands next to it
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

__device__ __forceinline__ bool bf16_nonfinite2(uint32_t w) {
    return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
}

// The distinct adapters of rows [n0, n0 + BN), in order of first appearance,
// each with the 16-row aligned window of the tile that holds its rows, in
// pieces of at most BN / 2 rows. One warp.
__device__ void lp_build_list(const LpParams &p, LpShared *sh, int buf, int n0, int lane) {
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
                int w0 = first & ~15;
                const int w1 = (last + 16) & ~15;
                const int most = p.BN / 2;
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
__device__ float lp_nonfinite_terms(const LpParams &p, int id, int row, int o) {
    const __nv_bfloat16 *b = p.lora_b + ((size_t)id * p.O + o) * (size_t)p.rank;
    const float *t = p.t + (size_t)row * p.rank;
    float v = 0.f;
    for (int j = 0; j < p.rank; ++j) {
        const float f = __bfloat162float(b[j]);
        if (!isfinite(f)) v += __ldcg(t + j) * f;
    }
    return v;
}

__global__ void __launch_bounds__(lp::THREADS, 1)
    lora_proj_kernel(const __grid_constant__ CUtensorMap tmw, const __grid_constant__ CUtensorMap tmx,
                     const __grid_constant__ CUtensorMap tmb, LpParams p) {
    using namespace lp;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const int S = p.stages;
    const int b_bytes = p.BN * 128;
    uint8_t *sA = smem;
    uint8_t *sB = smem + S * A_BYTES;
    LpShared *sh = reinterpret_cast<LpShared *>(sB + S * b_bytes);
    volatile int *abort_flag = &sh->abort;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (!cluster_shape_is((uint32_t)p.CK, 1u, 1u)) {
        // not the cluster that the sums address: the whole cluster leaves
        pdl_wait();
        if (tid == 0) atomicOr(p.status, SVF_DEV_BAD_CLUSTER);
        return;
    }
    const int rank = p.CK > 1 ? (int)cluster_ctarank() : 0;
    const int first_tile = blockIdx.x / p.CK, tile_step = gridDim.x / p.CK;
    const int kb0 = (int)((long long)p.kblocks * rank / p.CK);
    const int nkb = (int)((long long)p.kblocks * (rank + 1) / p.CK) - kb0;

    if (tid == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(&sh->full[s], 1);
            mbar_init(&sh->bfull[s], 1);
            mbar_init(&sh->ext[s], 1);
            mbar_init(&sh->empty[s], 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(&sh->acc_full[a], 1);
            mbar_init(&sh->acc_empty[a], 4);
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
    if (warp == 1) {
        tmem_alloc(&sh->tmem, p.tmem_cols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // Only t waits for the kernel before this one (warps 6-9 below): that
    // kernel lets this one start after its own wait, so what this call reads
    // besides t was complete by then.
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
        for (int tile = first_tile; tile < p.tiles && ok; tile += tile_step, ++i) {
            const int m0 = tile / p.n_tiles * BM, n0 = tile % p.n_tiles * p.BN;
            // tiles that start together start at different columns
            const int rot = (int)((long long)first_tile * nkb / tile_step) % nkb;
            for (int kb = 0; kb < nkb; ++kb, ++issued) {
                const int s = issued % S, use = issued / S;
                const int kc = (kb0 + (kb + rot < nkb ? kb + rot : kb + rot - nkb)) * BK;
                if (use > 0 && !(ok = lp_wait(&sh->empty[s], (uint32_t)((use - 1) & 1),
                                              abort_flag, p.wait_ns)))
                    break;
                if (lane == 0) {
                    mbar_arrive_expect_tx(&sh->full[s], (uint32_t)(A_BYTES + b_bytes));
                    tma_load_2d(sA + s * A_BYTES, &tmw, kc, m0, &sh->full[s]);
                    tma_load_2d(sB + s * b_bytes, &tmx, kc, n0, &sh->full[s]);
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
            for (int e = rank; e < n_list && ok; e += p.CK) {
                const int id = sh->list[buf][e].x;
                for (int kc = 0; kc < p.kchunks; ++kc, ++issued) {
                    const int s = issued % S, use = issued / S;
                    if (use > 0 && !(ok = lp_wait(&sh->empty[s], (uint32_t)((use - 1) & 1),
                                                  abort_flag, p.wait_ns)))
                        break;
                    if (lane == 0) {
                        mbar_arrive_expect_tx(&sh->bfull[s], (uint32_t)A_BYTES);
                        tma_load_3d(sA + s * A_BYTES, &tmb, kc * BK, m0, id, &sh->bfull[s]);
                    }
                    par_ext ^= 1u << s;
                    any_ext |= 1u << s;
                    __syncwarp();
                }
            }
            if (lane == 0) mbar_arrive(&sh->list_empty[buf]);
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer
        bool ok = true;
        int it = 0, i = 0;
        const uint32_t idesc = idesc_bf16_f32(128, p.BN, false, false);
        for (int tile = first_tile; tile < p.tiles && ok; tile += tile_step, ++i) {
            const int buf = i & 1, ause = i >> 1;
            if (ause > 0 && !(ok = lp_wait(&sh->acc_empty[buf], (uint32_t)((ause - 1) & 1),
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
                        umma_ss(d, smem_desc_sw128(a + k * 32, 16, 1024),
                                smem_desc_sw128(b + k * 32, 16, 1024), idesc,
                                (kb > 0 || k > 0) ? 1u : 0u);
                    umma_commit(&sh->empty[s]);
                }
                __syncwarp();
            }
            if (!ok) break;
            if (!(ok = lp_wait(&sh->list_full[buf], (uint32_t)(ause & 1), abort_flag, p.wait_ns)))
                break;
            const int n_list = sh->n_list[buf];
            for (int e = rank; e < n_list && ok; e += p.CK) {
                const int w = sh->list[buf][e].y;
                const int w0 = w & 0xffff, len = w >> 16;
                const uint32_t idw = idesc_bf16_f32(128, len, false, false);
                for (int kc = 0; kc < p.kchunks; ++kc, ++it) {
                    const int s = it % S;
                    if (!(ok = lp_wait(&sh->ext[s], par_ext >> s & 1u, abort_flag, p.wait_ns)))
                        break;
                    par_ext ^= 1u << s;
                    tc_fence_after();
                    if (lane == 0) {
                        const uint32_t a = smem_u32(sA + s * A_BYTES);
                        const uint32_t hi = smem_u32(sB + s * b_bytes);
                        const uint32_t lo = hi + (uint32_t)b_bytes / 2;
                        const int ksteps = (min(p.rank - kc * BK, BK) + 15) / 16;
                        for (int k = 0; k < ksteps; ++k) {
                            const uint64_t da = smem_desc_sw128(a + k * 32, 16, 1024);
                            umma_ss(d + (uint32_t)w0, da, smem_desc_sw128(hi + k * 32, 16, 1024),
                                    idw, 1u);
                            umma_ss(d + (uint32_t)w0, da, smem_desc_sw128(lo + k * 32, 16, 1024),
                                    idw, 1u);
                        }
                        umma_commit(&sh->empty[s]);
                    }
                    __syncwarp();
                }
            }
            if (!ok) break;
            if (lane == 0) {
                umma_commit(&sh->acc_full[buf]);
                mbar_arrive(&sh->list_empty[buf]);
            }
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
            const int m0 = tile / p.n_tiles * BM, n0 = tile % p.n_tiles * p.BN;
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
                    if (o_ok) {
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (j < rows_left) {
                                const int id = sh->ids[buf][c + j];
                                float v = id == -2 ? 0.f : __uint_as_float(r[j]);
                                if (patch && id >= 0)
                                    v += lp_nonfinite_terms(p, id, n0 + c + j, o);
                                col[(long long)(n0 + c + j) * p.y_stride] = __float2bfloat16(v);
                            }
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&sh->acc_empty[buf]);
                mbar_arrive(&sh->list_empty[buf]);
            }
        }
    } else {
        // ------------------------------------------------------------ adapters
        const int w = warp - 6;
        bool ok = true;
        int it = 0, i = 0;
        bool waited = false;
        for (int tile = first_tile; tile < p.tiles && ok; tile += tile_step, ++i) {
            const int n0 = tile % p.n_tiles * p.BN;
            const int buf = i & 1, ause = i >> 1;
            if (w == 0) {
                if (ause > 0 && !(ok = lp_wait(&sh->list_empty[buf], (uint32_t)((ause - 1) & 1),
                                               abort_flag, p.wait_ns)))
                    break;
                lp_build_list(p, sh, buf, n0, lane);
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
            for (int e = rank; e < n_list && ok; e += p.CK) {
                const int2 entry = sh->list[buf][e];
                const int id = entry.x, w0 = entry.y & 0xffff, len = entry.y >> 16;
                for (int kc = 0; kc < p.kchunks; ++kc, ++it) {
                    const int s = it % S;
                    if ((s & 3) != w) continue;  // a stage is always the same warp's
                    if (!(ok = lp_wait(&sh->bfull[s], par_ext >> s & 1u, abort_flag, p.wait_ns)))
                        break;
                    par_ext ^= 1u << s;
                    const int rc = min(p.rank - kc * BK, BK);  // a multiple of 8
                    uint8_t *tA = sA + s * A_BYTES;
                    bool bad = false;
                    for (int c = 0; c < rc / 8; ++c)
#pragma unroll
                        for (int u = 0; u < BM / 32; ++u) {
                            const int row = u * 32 + lane;
                            uint4 *at = reinterpret_cast<uint4 *>(
                                tA + row * 128 + ((c ^ (row & 7)) << 4));
                            uint4 b = *at;
                            if (bf16_nonfinite2(b.x) | bf16_nonfinite2(b.y) |
                                bf16_nonfinite2(b.z) | bf16_nonfinite2(b.w)) {
                                uint32_t wd[4] = {b.x, b.y, b.z, b.w};
                                for (int k = 0; k < 4; ++k) {
                                    if ((wd[k] & 0x7f80u) == 0x7f80u) wd[k] &= 0xffff0000u;
                                    if ((wd[k] & 0x7f800000u) == 0x7f800000u) wd[k] &= 0xffffu;
                                }
                                *at = make_uint4(wd[0], wd[1], wd[2], wd[3]);
                                bad = true;
                            }
                        }
                    if (bad) sh->nonfinite[buf] = 1;
                    // t of the window: hi in the first half of the stage's x
                    // area, lo in the second; 16-byte chunks of 8 columns
                    uint8_t *hi = sB + s * b_bytes, *lo = hi + b_bytes / 2;
                    const int nch = (rc + 15) / 16 * 2;
                    for (int u = lane; u < len * nch; u += 32) {
                        const int row = u / nch, c = u % nch;
                        float f[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k) f[k] = 0.f;
                        if (c * 8 < rc && sh->ids[buf][w0 + row] == id) {
                            const float4 *src = reinterpret_cast<const float4 *>(
                                p.t + (size_t)(n0 + w0 + row) * p.rank + kc * BK + c * 8);
                            *reinterpret_cast<float4 *>(f) = __ldcg(src);
                            *reinterpret_cast<float4 *>(f + 4) = __ldcg(src + 1);
                        }
                        uint32_t h[4], l[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            h[k] = pack_bf16x2(f[2 * k], f[2 * k + 1]);
                            const float h0 = __uint_as_float(h[k] << 16);
                            const float h1 = __uint_as_float(h[k] & 0xffff0000u);
                            // an infinite hi has no remainder
                            l[k] = pack_bf16x2(isfinite(h0) ? f[2 * k] - h0 : 0.f,
                                               isfinite(h1) ? f[2 * k + 1] - h1 : 0.f);
                        }
                        const int off = row * 128 + ((c ^ (row & 7)) << 4);
                        *reinterpret_cast<uint4 *>(hi + off) = make_uint4(h[0], h[1], h[2], h[3]);
                        *reinterpret_cast<uint4 *>(lo + off) = make_uint4(l[0], l[1], l[2], l[3]);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sh->ext[s]);
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
        // from the CK partial tiles, in rank order.
        cluster_arrive();
        cluster_wait();
        const int m0 = first_tile / p.n_tiles * BM, n0 = first_tile % p.n_tiles * p.BN;
        const int c0 = p.BN * rank / p.CK, c1 = p.BN * (rank + 1) / p.CK;
        int patch = 0;
        for (int c = 0; c < p.CK; ++c) patch |= ld_dsmem_s32(cluster_map(&sh->nonfinite[0], c));
        const bool pair = (p.y_stride & 1) == 0 &&
                          (reinterpret_cast<uintptr_t>(p.y) & 3) == 0;
        const float *part = reinterpret_cast<const float *>(smem);
        for (int u = tid; u < (c1 - c0) * (BM / 2); u += THREADS) {
            const int c = c0 + u / (BM / 2), o2 = u % (BM / 2) * 2;
            const int row = n0 + c, o = m0 + o2;
            if (row >= p.R || o >= p.O) continue;
            float a = 0.f, b = 0.f;
            for (int k = 0; k < p.CK; ++k) {
                const uint32_t at = cluster_map(part + c * BM + o2, (uint32_t)k);
                a += ld_dsmem_f32(at);
                b += ld_dsmem_f32(at + 4);
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
    // leave only when every load that this CTA issued has landed and every
    // commit that frees one of its stages has arrived
    if (warp == 0 && lane == 0) {
        volatile int never = 0;
        for (int s = 0; s < S; ++s) {
            if (any_main >> s & 1u)
                mbar_wait_for(&sh->full[s], (par_main >> s & 1u) ^ 1u, &never, kWaitDeadlineNs);
            if (any_ext >> s & 1u)
                mbar_wait_for(&sh->bfull[s], (par_ext >> s & 1u) ^ 1u, &never, kWaitDeadlineNs);
            if (s < sh->committed)
                mbar_wait_for(&sh->empty[s], (uint32_t)((sh->committed - 1 - s) / S & 1), &never,
                              kWaitDeadlineNs);
        }
    }
    __syncthreads();
    if (p.CK > 1) {
        cluster_arrive();
        cluster_wait();
    }
    if (warp == 1) tmem_dealloc(tmem, p.tmem_cols);
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

// [planes, rows, cols] bf16 with the given strides (elements); boxes of 64
// columns x box_rows rows of one plane, 128-byte swizzle. dims == 2: one plane.
static bool lp_map(CUtensorMap *map, const void *base, int dims, long long planes, long long rows,
                   long long cols, long long row_stride, long long plane_stride, int box_rows) {
    auto enc = lp_encoder();
    if (!enc) return false;
    cuuint64_t d[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)planes};
    cuuint64_t strides[2] = {(cuuint64_t)row_stride * 2, (cuuint64_t)plane_stride * 2};
    cuuint32_t box[3] = {64, (cuuint32_t)box_rows, 1};
    cuuint32_t estr[3] = {1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)dims, const_cast<void *>(base), d,
               strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool lora_proj_supported(int R, int H, int O, int adapters, int rank) {
    return R >= 1 && R <= (1 << 20) && H >= 8 && H % 8 == 0 && H <= (1 << 16) && O >= 1 &&
           O <= (1 << 20) && adapters >= 1 && adapters <= (1 << 16) && rank >= 8 &&
           rank % 8 == 0 && rank <= 128;
}

int launch_lora_proj(const LoraArgs &a, cudaStream_t stream) {
    LpParams p;
    p.R = a.R;
    p.H = a.H;
    p.O = a.O;
    p.rank = a.rank;
    p.adapters = a.adapters;
    p.per = a.rows_per_id;
    p.n_tiles = (a.R + lp::MAX_BN - 1) / lp::MAX_BN;
    p.BN = ((a.R + p.n_tiles - 1) / p.n_tiles + 31) / 32 * 32;
    p.n_tiles = (a.R + p.BN - 1) / p.BN;
    const int m_tiles = (a.O + lp::BM - 1) / lp::BM;
    p.tiles = m_tiles * p.n_tiles;
    p.kblocks = (a.H + lp::BK - 1) / lp::BK;
    p.kchunks = (a.rank + lp::BK - 1) / lp::BK;
    // CTAs per tile: as many as fill the SMs once, each with at least four
    // blocks of K
    const int sms = num_sms();
    p.CK = 1;
    for (int c = 2; c <= 8; ++c)
        if (p.tiles * c <= sms && p.kblocks >= 4 * c) p.CK = c;
    const int stage_bytes = lp::A_BYTES + p.BN * 128;
    p.stages = lp::SMEM_BUDGET / stage_bytes;
    if (p.stages > lp::MAX_STAGES) p.stages = lp::MAX_STAGES;
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
    if (!lp_map(&tmw, a.weight, 2, 1, a.O, a.H, a.H, 0, lp::BM) ||
        !lp_map(&tmx, a.x, 2, 1, a.R, a.H, a.x_stride, 0, p.BN) ||
        !lp_map(&tmb, a.lora_b, 3, a.adapters, a.O, a.rank, a.rank, (long long)a.O * a.rank,
                lp::BM))
        return SVF_ERR_LAUNCH;
    const size_t smem = 1024 + (size_t)p.stages * stage_bytes + sizeof(LpShared);
    if (cudaFuncSetAttribute(lora_proj_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)smem) != cudaSuccess)
        return SVF_ERR_LAUNCH;
    if (launch_lora_shrink(a, stream) != cudaSuccess) return SVF_ERR_LAUNCH;
    int clusters = p.tiles;
    if (p.CK == 1 && clusters > sms) clusters = sms;  // persistent
    if (launch_pdl(lora_proj_kernel, dim3((unsigned)(clusters * p.CK)), dim3(lp::THREADS), smem,
                   stream, p.CK > 1 ? (unsigned)p.CK : 0u, tmw, tmx, tmb, p) != cudaSuccess)
        return SVF_ERR_LAUNCH;
    return SVF_OK;
}

}  // namespace svf
