// lora_shrink.cu -- the low-rank inner products of lora_proj: for every row r
// with adapter a = ids[r / rows_per_id],
//     t[r][j] = scale_a * sum_k x[r][k] A_a[j][k],   j < rank,
// summed in fp32 and kept as two bf16 terms, hi + lo, for the tensor cores, and
// the per-group status words.
//
// Bound: the bytes of x and of the used A matrices (HBM or L2), and the
// latency of a short call; the products are a few percent of the projection's.
// So nothing is staged: the rows of x and of A are K-major, and the order of
// the terms of a sum over k is free, so a warp feeds mma.sync fragments
// straight from 16-byte global loads by letting lane (g, q) of a fragment hold
// the 8 consecutive k of its quarter of a 32-wide block (the same permutation
// of k on both operands), with the loads of the next DEPTH blocks in flight in
// registers. The tcgen05 path would have to stage both operands through shared
// memory and tensor memory for N = rank columns.
//
// A CTA takes a block of 16 MT rows and one of the distinct adapters in it;
// its 4 warps, and the KS CTAs of its cluster, share the 32-wide blocks of
// K. The warps' sums meet in shared memory; every CTA sends each of the
// others its share of them (asynchronous stores that count on the receiver's
// barrier) and adds up the terms of its own share, both in a fixed order (64
// requests with 56 adapters, the whole call: 18.5 us; 19.4 where they read
// each other's sums between two barriers). Rows of other adapters in the
// block are not stored, so an infinity or NaN in one request's adapter or
// hidden state stays with it.
//
// The kernel is small (128 threads of 128 registers, two CTAs per SM; 96
// where ranks above 16 fill many CTAs: 128 rows of 100 adapters of rank 64,
// 8192 -> 10240, took 134 us with 128 and deeper loads, 122 with 96), so
// that the CTAs of the projection kernel start beside it (the cap of 128 makes
// the instance of rank 8 spill 52 bytes, and 32-row tiles of rank 16 20): its
// first products
// need no t, which is there (after 5 to 12 us) before their last. Alone it
// takes 5.5 us for one row, 7.5 us for 64 rows of 56 adapters of rank 16
// (4096 columns).
#include "common.cuh"
#include "internal.h"
#include "lora.h"

namespace svf {

namespace {

constexpr int kShrinkWarps = 4;
constexpr int kShrinkThreads = 32 * kShrinkWarps;

struct ShrinkArgs {
    const __nv_bfloat16 *x, *la;
    const float *scales;
    const int32_t *ids;
    __nv_bfloat16 *t;  // [hi and lo, R, rank]
    int32_t *status;
    long long x_stride;
    int R, H, rank, adapters, per;
    int KS, slots, ngroups;
    unsigned long long wait_ns;
};

__device__ __forceinline__ void mma_bf16(float *c, uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 ld16(const __nv_bfloat16 *p, bool ok) {
    return ok ? __ldg(reinterpret_cast<const uint4 *>(p)) : make_uint4(0, 0, 0, 0);
}

// MT: 16-row tiles of x of a block; NT: 8-row tiles of A that a CTA takes
// (rank in groups of 8 NT)
template <int MT, int NT, int DEPTH>
__global__ void __maxnreg__(MT == 1 && NT == 4 ? 96 : 128) lora_shrink_kernel(ShrinkArgs p) {
    constexpr int ROWS = 16 * MT;
    constexpr int TILE = ROWS * NT * 8;
    __shared__ __align__(16) float s_acc[kShrinkWarps][TILE];
    // Every CTA of the cluster sums up an equal share of the tile: s_recv
    // [KS][TILE / KS] gets the CTAs' terms of it.
    __shared__ __align__(16) float s_recv[TILE];
    __shared__ __align__(8) uint64_t s_full;
    __shared__ int s_ids[32];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int ks = blockIdx.x % p.KS;
    int rest = blockIdx.x / p.KS;
    const int ng = rest % p.ngroups;
    rest /= p.ngroups;
    const int slot = rest % p.slots, blk = rest / p.slots;
    const int row0 = blk * ROWS;
    const bool shaped = cluster_shape_is((uint32_t)p.KS, 1u, 1u);
    const bool shared = shaped && p.KS > 1;
    if (shared) {
        if (tid == 0) {
            mbar_init(&s_full, 1);
            mbar_fence_init();
            mbar_arrive_expect_tx(&s_full, TILE * 4);
        }
        cluster_arrive();  // the others may send
    }
    pdl_wait();
    // The projection kernel starts when every CTA here has come to this call,
    // so after the wait above: what it reads besides t is complete by then.
    pdl_launch_dependents();
    if (tid < 32) {
        const int row = row0 + tid;
        int id = -1;
        if (tid < ROWS && row < p.R) {
            const int g = row / p.per;
            id = p.ids[g];
            const bool bad = id < -1 || id >= p.adapters;
            if (slot == 0 && ng == 0 && ks == 0 && row % p.per == 0)
                p.status[g] = (bad ? SVF_DEV_BAD_ADAPTER : 0) | (shaped ? 0 : SVF_DEV_BAD_CLUSTER);
            if (bad) id = -1;
        }
        s_ids[tid] = id;
    }
    __syncthreads();
    if (!shaped) return;  // not the cluster that the sums address: touch no peer
    const int my = s_ids[lane];
    const unsigned same = __match_any_sync(0xffffffffu, my);
    unsigned todo = __ballot_sync(0xffffffffu, my >= 0 && lane == __ffs(same) - 1);
    for (int i = 0; i < slot && todo; ++i) todo &= todo - 1;
    const int kchunks = (p.H + 31) / 32, kstep = p.KS * kShrinkWarps;
    const int g = lane >> 2, q = lane & 3;
    bool sent = false, lost = false;
    const int n0 = ng * NT * 8;
    const int nt = min(NT, (p.rank - n0) / 8);
    while (todo) {  // the slot-th distinct adapter, then every slots-th after it
        const int id = s_ids[__ffs(todo) - 1];
        for (int i = 0; i < p.slots && todo; ++i) todo &= todo - 1;
        bool mine[2 * MT];
        const __nv_bfloat16 *xr[2 * MT];
#pragma unroll
        for (int m = 0; m < 2 * MT; ++m) {
            mine[m] = s_ids[m * 8 + g] == id;
            xr[m] = p.x + (long long)(row0 + (mine[m] ? m * 8 + g : 0)) * p.x_stride + q * 8;
        }
        const __nv_bfloat16 *ar = p.la + ((size_t)id * p.rank + n0 + g) * (size_t)p.H + q * 8;
        float acc[MT][NT][4];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n)
                acc[m][n][0] = acc[m][n][1] = acc[m][n][2] = acc[m][n][3] = 0.f;
        uint4 xv[DEPTH][2 * MT], av[DEPTH][NT];
        auto load = [&](int kc, uint4 *x, uint4 *a) {
            const int k = kc * 32;
            const bool ok = k + q * 8 < p.H;
#pragma unroll
            for (int m = 0; m < 2 * MT; ++m) x[m] = ld16(xr[m] + k, mine[m] && ok);
#pragma unroll
            for (int n = 0; n < NT; ++n) a[n] = ld16(ar + (size_t)(n * 8) * p.H + k, n < nt && ok);
        };
        const int kc0 = ks * kShrinkWarps + warp;
#pragma unroll
        for (int d = 0; d < DEPTH; ++d) load(kc0 + d * kstep, xv[d], av[d]);
        for (int kc = kc0; kc < kchunks; kc += DEPTH * kstep) {
#pragma unroll
            for (int d = 0; d < DEPTH; ++d) {
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    const uint4 u0 = xv[d][2 * m], u1 = xv[d][2 * m + 1];
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const uint4 b = av[d][n];
                        mma_bf16(acc[m][n], u0.x, u1.x, u0.y, u1.y, b.x, b.y);
                        mma_bf16(acc[m][n], u0.z, u1.z, u0.w, u1.w, b.z, b.w);
                    }
                }
                load(kc + (d + DEPTH) * kstep, xv[d], av[d]);
            }
        }
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float *d = &s_acc[warp][(m * 16 + g) * NT * 8 + n * 8 + q * 2];
                *reinterpret_cast<float2 *>(d) = make_float2(acc[m][n][0], acc[m][n][1]);
                *reinterpret_cast<float2 *>(d + 8 * NT * 8) = make_float2(acc[m][n][2], acc[m][n][3]);
            }
        __syncthreads();
        const int share = TILE / p.KS;  // KS is a power of two
        if (p.KS > 1) {
            // The host gives a cluster one adapter only, so nothing is sent twice.
            cluster_wait();
            for (int i = 4 * tid; i < TILE; i += 4 * kShrinkThreads) {
                float4 v = *reinterpret_cast<const float4 *>(&s_acc[0][i]);
#pragma unroll
                for (int w = 1; w < kShrinkWarps; ++w) {
                    const float4 u = *reinterpret_cast<const float4 *>(&s_acc[w][i]);
                    v.x += u.x, v.y += u.y, v.z += u.z, v.w += u.w;
                }
                const uint32_t to = (uint32_t)(i / share);
                st_async_v4(cluster_map(&s_recv[ks * share + i % share], to), v,
                            cluster_map(&s_full, to));
            }
            sent = true;
            lost = !mbar_wait_cluster_for(&s_full, 0, p.wait_ns);
        }
        const float scale = p.scales ? p.scales[id] : 1.f;
        for (int i = ks * share + tid; i < (ks + 1) * share; i += kShrinkThreads) {
            const int row = i / (NT * 8), j = i % (NT * 8);
            if (s_ids[row] != id || n0 + j >= p.rank) continue;
            float v = 0.f;
            if (p.KS > 1) {
                for (int c = 0; c < p.KS; ++c) v += s_recv[c * share + i - ks * share];
            } else {
#pragma unroll
                for (int w = 0; w < kShrinkWarps; ++w) v += s_acc[w][i];
            }
            v *= scale;
            const __nv_bfloat16 hi = __float2bfloat16(v);
            const float h = __bfloat162float(hi);
            __nv_bfloat16 *t = p.t + (size_t)(row0 + row) * p.rank + n0 + j;
            t[0] = hi;
            // an infinite hi has no remainder
            t[(size_t)p.R * p.rank] = __float2bfloat16(isfinite(h) ? v - h : 0.f);
        }
        if (p.KS > 1) break;
        __syncthreads();
    }
    if (shared && !sent) cluster_wait();
    if (shared && __syncthreads_or(lost)) {
        // Terms may still be on their way here. Every other CTA has sent its own
        // once it comes to this barrier too, or has left; then they land.
        cluster_arrive();
        cluster_wait();
        if (tid == 0) {
            mbar_wait_cluster_for(&s_full, 0, 20000000ull);
            atomicOr(p.status, SVF_DEV_TIMEOUT);
        }
        __syncthreads();
    }
}

template <int MT, int NT, int DEPTH>
cudaError_t launch_tiled(ShrinkArgs p, cudaStream_t stream) {
    p.ngroups = (p.rank + NT * 8 - 1) / (NT * 8);
    const int rows = 16 * MT;
    const int blocks = (p.R + rows - 1) / rows;
    // distinct adapters that a block's consecutive rows can meet
    int most = p.per >= rows ? 2 : (rows - 2) / p.per + 2;
    const int groups = p.R / p.per;
    if (most > groups) most = groups;
    if (most > rows) most = rows;
    // As many CTAs as hold an adapter of a block each, but at most so many per SM:
    // two while what is read is small, so that the projection's CTAs fit beside
    // them (64 rows, 56 adapters of rank 16, 4096 -> 4096: 18.5 us, 20.2 with
    // six); six where it would take longer than the projection's first products
    // (then the sooner it is over the better: 512 rows in groups of 4, 100
    // adapters of rank 64, 4096 -> 6144: 74.5 us, 89 with two).
    const int used = groups < p.adapters ? groups : p.adapters;
    const double bytes = 2.0 * p.H * (p.R + (double)used * p.rank);
    const bool large = bytes > 16e6;
    const long long room = (large ? 6ll : 2ll) * num_sms();
    int slots = most;
    while (slots > 1 && (long long)blocks * slots * p.ngroups > room) slots = (slots + 1) / 2;
    p.slots = slots;
    // Then up to 8 CTAs over K, each warp with a block of its own (a cluster takes
    // one adapter, so only where there are slots for all). Of the six per SM this
    // fills three for ranks up to 32 and fewer than 1024 rows: 256 rows of 200
    // adapters of rank 16, 4096 -> 4096: 31.3 us, 37.3 with six; 64 rows, 40
    // adapters of rank 16, 14336 -> 4096: 32.0, 34.0; 640 rows in groups of 4, 160
    // adapters of rank 32: 46.8, 44.6. All six else: 32 rows of 32 adapters of rank
    // 64: 22.7, 25.1 with two; 4096 rows in groups of 64, 60 adapters of rank 16:
    // 101, 105 to 117 with two.
    const long long room_k =
        large && p.rank <= 32 && p.R < 1024 ? 3ll * num_sms() : room;
    const int kchunks = (p.H + 31) / 32;
    p.KS = 1;
    while (slots == most && p.KS < 8 && 2ll * p.KS * blocks * slots * p.ngroups <= room_k &&
           p.KS * kShrinkWarps < kchunks)
        p.KS *= 2;
    return launch_pdl(lora_shrink_kernel<MT, NT, DEPTH>,
                      dim3((unsigned)(p.KS * blocks * slots * p.ngroups)), dim3(kShrinkThreads), 0,
                      stream, p.KS > 1 ? (unsigned)p.KS : 0u, p);
}

template <int NT, int D1, int D2>
cudaError_t launch_ranked(const ShrinkArgs &p, cudaStream_t stream) {
    // Tiles of 32 rows, which a tile of A serves at once, where they meet at most
    // two groups (4096 columns; tiles of 16 in brackets: 1024 rows in groups of 32,
    // 9 adapters of rank 32: 38.8 us [40.4]; 4096 in groups of 128, rank 8: 97
    // [102]; 1984 in groups of 31, rank 16: 75.6 [74.4]; but 1024 in groups of 16,
    // rank 16: 41.5 [37.2]) and are many (512 in groups of 32, rank 16, 4096 ->
    // 6144: 30.3 [27.9]; -> 4096: 22.2 [22.8]; 256 in groups of 64, rank 64: 22.1
    // [21.0]).
    return p.per >= 31 && p.R >= 1024 ? launch_tiled<2, NT, D2>(p, stream)
                                     : launch_tiled<1, NT, D1>(p, stream);
}

}  // namespace

cudaError_t launch_lora_shrink(const LoraArgs &a, unsigned long long wait_ns,
                               cudaStream_t stream) {
    ShrinkArgs p;
    p.x = static_cast<const __nv_bfloat16 *>(a.x);
    p.la = static_cast<const __nv_bfloat16 *>(a.lora_a);
    p.scales = a.scales;
    p.ids = a.ids;
    p.t = static_cast<__nv_bfloat16 *>(a.workspace);
    p.status = a.status;
    p.x_stride = a.x_stride;
    p.R = a.R;
    p.H = a.H;
    p.rank = a.rank;
    p.adapters = a.adapters;
    p.per = a.rows_per_id;
    p.wait_ns = wait_ns;
    if (a.rank <= 8) return launch_ranked<1, 4, 4>(p, stream);
    if (a.rank <= 16) return launch_ranked<2, 4, 3>(p, stream);
    return launch_ranked<4, 2, 2>(p, stream);
}

}  // namespace svf
