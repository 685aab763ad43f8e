// lora_shrink.cu -- the low-rank inner products of lora_proj: for every row r
// with adapter a = ids[r / rows_per_id],
//     t[r][j] = scale_a * sum_k x[r][k] A_a[j][k],   j < rank   (fp32)
// and the per-group status words.
//
// Bound: the bytes of x and of the used A matrices (HBM or L2), and the
// latency of a short call; the products are a few percent of the projection's.
// So nothing is staged: the rows of x and of A are K-major, and the order of
// the terms of a sum over k is free, so a warp feeds mma.sync fragments
// straight from 16-byte global loads by letting lane (g, q) of a fragment hold
// the 16 consecutive k of its quarter of a 64-wide block (the same permutation
// of k on both operands). The tcgen05 path would have to stage both operands
// through shared memory and tensor memory for N = rank columns.
//
// A CTA takes a block of 16 rows and one of the distinct adapters in it; its
// 4 warps, and the KS CTAs of its cluster, share the 64-wide blocks of K. The
// warps' sums meet in shared memory, the CTAs' over distributed shared memory,
// in a fixed order. Rows of other adapters in the block are not stored, so an
// infinity or NaN in one request's adapter or hidden state stays with it.
#include "common.cuh"
#include "internal.h"
#include "lora.h"

namespace svf {

namespace {

constexpr int kShrinkWarps = 4;
constexpr int kShrinkThreads = 32 * kShrinkWarps;
constexpr int kShrinkRows = 16;

struct ShrinkArgs {
    const __nv_bfloat16 *x, *la;
    const float *scales;
    const int32_t *ids;
    float *t;
    int32_t *status;
    long long x_stride;
    int R, H, rank, adapters, per;
    int KS, slots, ngroups;
};

__device__ __forceinline__ void mma_bf16(float *c, const uint32_t *a, uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 ld16(const __nv_bfloat16 *p, bool ok) {
    return ok ? __ldg(reinterpret_cast<const uint4 *>(p)) : make_uint4(0, 0, 0, 0);
}

// NT: 8-row tiles of A that a CTA takes (rank in groups of 8 NT)
template <int NT>
__global__ void __launch_bounds__(kShrinkThreads, 5) lora_shrink_kernel(ShrinkArgs p) {
    __shared__ float s_acc[kShrinkWarps][kShrinkRows][NT * 8];
    __shared__ int s_ids[kShrinkRows];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int ks = blockIdx.x % p.KS;  // the CTA's rank in its cluster
    int rest = blockIdx.x / p.KS;
    const int ng = rest % p.ngroups;
    rest /= p.ngroups;
    const int slot = rest % p.slots, blk = rest / p.slots;
    const int row0 = blk * kShrinkRows;
    const bool shaped = cluster_shape_is((uint32_t)p.KS, 1u, 1u);
    pdl_wait();
    // the projection kernel starts when every CTA here has passed the wait
    // above, so that what it reads besides t is complete
    pdl_launch_dependents();
    if (tid < kShrinkRows) {
        const int row = row0 + tid;
        int id = -1;
        if (row < p.R) {
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
    const int my = s_ids[lane & 15];
    bool first = my >= 0 && lane < 16;
    for (int i = 0; i < (lane & 15); ++i) first &= s_ids[i] != my;
    unsigned todo = __ballot_sync(0xffffffffu, first);
    for (int i = 0; i < slot && todo; ++i) todo &= todo - 1;
    const int kchunks = (p.H + 63) / 64;
    const int g = lane >> 2, q = lane & 3;
    const int n0 = ng * NT * 8;
    const int nt = min(NT, (p.rank - n0) / 8);
    while (todo) {  // the slot-th distinct adapter, then every slots-th after it
        const int id = s_ids[__ffs(todo) - 1];
        for (int i = 0; i < p.slots && todo; ++i) todo &= todo - 1;
        const bool r0 = s_ids[g] == id, r1 = s_ids[g + 8] == id;
        const __nv_bfloat16 *x0 = p.x + (long long)(row0 + (r0 ? g : 0)) * p.x_stride;
        const __nv_bfloat16 *x1 = p.x + (long long)(row0 + (r1 ? g + 8 : 0)) * p.x_stride;
        const __nv_bfloat16 *a0 = p.la + ((size_t)id * p.rank + n0 + g) * (size_t)p.H;
        float acc[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
            acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.f;
#pragma unroll 2
        for (int kc = ks * kShrinkWarps + warp; kc < kchunks; kc += p.KS * kShrinkWarps) {
            const int k = kc * 64 + q * 16;
            const bool ok0 = k < p.H, ok1 = k + 8 < p.H;
            uint4 xv[4], av[NT][2];
            xv[0] = ld16(x0 + k, r0 && ok0);
            xv[1] = ld16(x0 + k + 8, r0 && ok1);
            xv[2] = ld16(x1 + k, r1 && ok0);
            xv[3] = ld16(x1 + k + 8, r1 && ok1);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const __nv_bfloat16 *an = a0 + (size_t)(n * 8) * p.H + k;
                av[n][0] = ld16(an, n < nt && ok0);
                av[n][1] = ld16(an + 8, n < nt && ok1);
            }
            const uint32_t *u0 = reinterpret_cast<const uint32_t *>(xv);
            const uint32_t *u1 = reinterpret_cast<const uint32_t *>(xv + 2);
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const uint32_t a[4] = {u0[2 * s], u1[2 * s], u0[2 * s + 1], u1[2 * s + 1]};
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const uint32_t *b = reinterpret_cast<const uint32_t *>(av[n]);
                    mma_bf16(acc[n], a, b[2 * s], b[2 * s + 1]);
                }
            }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float *d = &s_acc[warp][g][n * 8 + q * 2];
            *reinterpret_cast<float2 *>(d) = make_float2(acc[n][0], acc[n][1]);
            *reinterpret_cast<float2 *>(d + 8 * NT * 8) = make_float2(acc[n][2], acc[n][3]);
        }
        __syncthreads();
        // the warps' sums, into the first one's place
        for (int i = tid; i < kShrinkRows * NT * 8; i += kShrinkThreads) {
            float v = 0.f;
#pragma unroll
            for (int w = 0; w < kShrinkWarps; ++w) v += (&s_acc[w][0][0])[i];
            (&s_acc[0][0][0])[i] = v;
        }
        if (p.KS > 1) {
            cluster_arrive();
            cluster_wait();
        } else {
            __syncthreads();
        }
        const float scale = p.scales ? p.scales[id] : 1.f;
        const int per_cta = kShrinkRows * NT * 8 / p.KS;  // KS is a power of two
        for (int i = ks * per_cta + tid; i < (ks + 1) * per_cta; i += kShrinkThreads) {
            float v = 0.f;
            if (p.KS > 1) {
                for (int c = 0; c < p.KS; ++c)
                    v += ld_dsmem_f32(cluster_map(&s_acc[0][0][0] + i, (uint32_t)c));
            } else {
                v = (&s_acc[0][0][0])[i];
            }
            const int row = i / (NT * 8), j = i % (NT * 8);
            if (s_ids[row] == id && n0 + j < p.rank)
                p.t[(size_t)(row0 + row) * p.rank + n0 + j] = v * scale;
        }
        if (p.KS > 1) {
            cluster_arrive();
            cluster_wait();
        } else {
            __syncthreads();
        }
    }
}

template <int NT>
cudaError_t launch_nt(ShrinkArgs p, cudaStream_t stream) {
    p.ngroups = (p.rank + NT * 8 - 1) / (NT * 8);
    const int blocks = (p.R + kShrinkRows - 1) / kShrinkRows;
    // distinct adapters that 16 consecutive rows can meet
    int most = p.per >= kShrinkRows ? 2 : (kShrinkRows - 2) / p.per + 2;
    const int groups = (p.R + p.per - 1) / p.per;
    if (most > groups) most = groups;
    if (most > kShrinkRows) most = kShrinkRows;
    // One CTA per adapter of a block, up to two CTAs per SM, so that the CTAs
    // of the projection kernel find room beside them and start at once; then
    // up to 8 CTAs (a cluster) over K while the two per SM are not used up and
    // each warp still has a 64-wide block of its own.
    const long long room = 2ll * num_sms();
    int slots = most;
    while (slots > 1 && (long long)blocks * slots * p.ngroups > room) slots = (slots + 1) / 2;
    const int kchunks = (p.H + 63) / 64;
    int KS = 1;
    while (KS < 8 && 2ll * KS * blocks * slots * p.ngroups <= room && KS * kShrinkWarps < kchunks)
        KS *= 2;
    p.slots = slots;
    p.KS = KS;
    return launch_pdl(lora_shrink_kernel<NT>,
                      dim3((unsigned)(KS * blocks * slots * p.ngroups)), dim3(kShrinkThreads), 0, stream, KS > 1 ? (unsigned)KS : 0u, p);
}

}  // namespace

cudaError_t launch_lora_shrink(const LoraArgs &a, cudaStream_t stream) {
    ShrinkArgs p;
    p.x = static_cast<const __nv_bfloat16 *>(a.x);
    p.la = static_cast<const __nv_bfloat16 *>(a.lora_a);
    p.scales = a.scales;
    p.ids = a.ids;
    p.t = static_cast<float *>(a.workspace);
    p.status = a.status;
    p.x_stride = a.x_stride;
    p.R = a.R;
    p.H = a.H;
    p.rank = a.rank;
    p.adapters = a.adapters;
    p.per = a.rows_per_id;
    if (a.rank <= 8) return launch_nt<1>(p, stream);
    if (a.rank <= 16) return launch_nt<2>(p, stream);
    return launch_nt<4>(p, stream);
}

}  // namespace svf
