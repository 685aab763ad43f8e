// chunk_simt.cu -- attention of chunks of new tokens over the paged cache, on CUDA cores.
//
//     out[r] = sum_{t <= L + i} p_t V_t / sum p_t,   p_t = 2^(scale log2(e) q_r . K_t - m_r)
//
// for row i of a sequence, in one pass over its keys with the running maximum m and sum of
// each row. All arithmetic is fp32; this is the path of fp32 tensors.
//
// A CTA goes through the tiles of its share of the call (chunk.cuh): 64 rows (token, head)
// against 64 tokens at a time. 256 threads as 16 x 16: thread (y, x) has rows 4 y .. + 3 and
// tokens x, x + 16, .. of the scores, and the same rows of O with elements 4 x + 64 c ..; so a
// row's sums stay inside 16 neighbouring lanes. The next K comes while P is made and
// multiplied with V, the next V while the next scores are made.
//
// Bound: fp32 FMA issue and shared-memory reads of the two products (2 D FMAs per score).
// Measured, 32/8 heads: 20 tokens over 20000 each of 20 sequences 2420 us (D = 128; 2970 with K and V
// through registers, whose loads wait for one another); 2048 tokens over themselves 3240 us at
// D = 128 (3035 through registers: the only case that loses) and 1490 at D = 64 (1510).
#include <math.h>

#include "chunk.cuh"

namespace svf {

namespace {

constexpr int BN = 64, BM = 64, NT = 256;

template <int D>
struct ChunkSmem {
    static constexpr int LDK = D + 4;   // 16 rows apart: 16 bytes skew
    static constexpr int LDP = BM + 4;
    float q[BM][LDK];
    float k[BN][LDK];
    float v[BN][LDK];
    float p[BN][LDP];  // P transposed: [token][row]
    float w[BM];       // the join: a row's log2-sum-exp
    int bad;           // first token of the part whose page is not in the cache
    int last;
    ChunkSpace space;
    ChunkCount sums[NT / 32];
};

__device__ __forceinline__ float ex2(float x) { return exp2f(x); }

template <int D>
__global__ void __launch_bounds__(NT) chunk_simt_kernel(ChunkParams p) {
    using Sm = ChunkSmem<D>;
    extern __shared__ __align__(16) uint8_t raw[];
    Sm &sm = *reinterpret_cast<Sm *>(raw);
    const int tid = threadIdx.x, x = tid & 15, y = tid >> 4;
    constexpr int NC = D / 64;  // column groups of O
    pdl_wait();
    pdl_launch_dependents();
    chunk_status<D, float>(p, tid, NT, [](bool v) { return __syncthreads_or(v) != 0; });
    chunk_layout<BN, NT>(p, &sm.space, sm.sums);
    const float *Q = static_cast<const float *>(p.q);
    const float *K = static_cast<const float *>(p.k_cache);
    const float *V = static_cast<const float *>(p.v_cache);
    float *out = static_cast<float *>(p.out);
    ChunkSeg g;
    for (bool more = chunk_first<BN>(p, sm.space, g); more;
         more = chunk_next<BN>(p, sm.space, g)) {
        int x0;
        const int tiles = chunk_part(sm.space, g, x0);
        if (tiles == 0) continue;
        const int head = g.hb * p.S + blockIdx.x % p.S;
        const int tok0 = g.k * p.TB, ntok = min(p.TB, g.n - tok0);
        const int M = ntok * p.G;  // rows of the block
        const int32_t *table = p.page_table + (size_t)g.b * p.max_pages;
        __syncthreads();  // the part before is through with shared memory
        if (tid == 0) sm.bad = kPieceFine;
        for (int i = tid; i < BM * (D / 4); i += NT) {
            const int r = i / (D / 4), c = i % (D / 4);
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < M)
                v = __ldg(reinterpret_cast<const float4 *>(
                              Q + ((size_t)(g.row0 + tok0 + r / p.G) * p.Hq + head * p.G + r % p.G) * D) +
                          c);
            *reinterpret_cast<float4 *>(&sm.q[r][4 * c]) = v;
        }
        float m[4], l[4], o[4][4 * NC];
        int see[4];  // the last token that the row sees
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            m[i] = -INFINITY;
            l[i] = 0.0f;
            const int r = 4 * y + i;
            see[i] = r < M ? g.L + tok0 + r / p.G : -1;
#pragma unroll
            for (int c = 0; c < 4 * NC; ++c) o[i][c] = 0.0f;
        }
        // Tiles come by asynchronous copies: 16 bytes a lane, R rows of K or V a warp. A row without
        // a token of the block, or without a page, is zeros.
        constexpr int R = D / 16;
        const int tend = g.L + tok0 + ntok;  // tokens that the block sees
        const int crow = tid / (D / 4), cc = tid % (D / 4);  // rows crow + (NT / (D / 4)) q
        int at[R];
        auto lookup = [&](int xt) {
#pragma unroll
            for (int q = 0; q < R; ++q) {
                const unsigned t = (unsigned)xt * BN + crow + q * (NT / (D / 4));
                at[q] = -1;
                if (xt < x0 + tiles && t < (unsigned)tend) {
                    const unsigned page = t / (unsigned)p.ps;
                    const int id = __ldg(table + page);
                    if (id >= 0 && id < p.num_pages) at[q] = id * p.ps + (int)(t - page * (unsigned)p.ps);
                    else if (cc == 0) atomicMin(&sm.bad, (int)t);
                }
            }
        };
        auto copy = [&](float (*dst)[Sm::LDK], const float *base) {
#pragma unroll
            for (int q = 0; q < R; ++q) {
                const float *src = base + ((size_t)max(at[q], 0) * p.Hkv + head) * D + 4 * cc;
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                                 smem_u32(&dst[crow + q * (NT / (D / 4))][4 * cc])),
                             "l"(src), "r"(at[q] >= 0 ? 16 : 0)
                             : "memory");
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        __syncthreads();  // sm.bad is set
        lookup(x0);
        copy(sm.k, K);
        copy(sm.v, V);
        for (int xt = x0; xt < x0 + tiles; ++xt) {
            const int t0 = xt * BN;
            asm volatile("cp.async.wait_group 1;" ::: "memory");  // K is there
            __syncthreads();
            float s[4][4];  // rows 4 y + i, tokens x + 16 j
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) s[i][j] = 0.0f;
#pragma unroll 4
            for (int d = 0; d < D; d += 4) {
                float4 a[4], b[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) a[i] = *reinterpret_cast<const float4 *>(&sm.q[4 * y + i][d]);
#pragma unroll
                for (int j = 0; j < 4; ++j) b[j] = *reinterpret_cast<const float4 *>(&sm.k[x + 16 * j][d]);
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        s[i][j] = fmaf(a[i].x, b[j].x, s[i][j]);
                        s[i][j] = fmaf(a[i].y, b[j].y, s[i][j]);
                        s[i][j] = fmaf(a[i].z, b[j].z, s[i][j]);
                        s[i][j] = fmaf(a[i].w, b[j].w, s[i][j]);
                    }
            }
            __syncthreads();  // K may be replaced, while P is made and multiplied
            lookup(xt + 1);
            copy(sm.k, K);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float mx = -INFINITY;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    s[i][j] = x + 16 * j <= see[i] - t0 ? s[i][j] * p.scale_log2 : -INFINITY;
                    mx = fmaxf(mx, s[i][j]);
                }
#pragma unroll
                for (int h = 8; h > 0; h >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, h));
                const float nm = fmaxf(m[i], mx);
                const float base = nm == -INFINITY ? 0.0f : nm;
                const float alpha = ex2(m[i] - base);  // 0 at the first visible token
                m[i] = nm;
                float sum = 0.0f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    s[i][j] = ex2(s[i][j] - base);
                    sum += s[i][j];
                }
                l[i] = fmaf(l[i], alpha, sum);  // this lane's tokens only
#pragma unroll
                for (int c = 0; c < 4 * NC; ++c) o[i][c] *= alpha;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
                *reinterpret_cast<float4 *>(&sm.p[x + 16 * j][4 * y]) =
                    make_float4(s[0][j], s[1][j], s[2][j], s[3][j]);
            asm volatile("cp.async.wait_group 1;" ::: "memory");  // V is there
            __syncthreads();
            const bool inner = BN - 1 <= g.L + tok0 - t0;  // every row sees the whole tile
#pragma unroll 4
            for (int t = 0; t < BN; ++t) {
                const float4 a = *reinterpret_cast<const float4 *>(&sm.p[t][4 * y]);
                const float pr[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    const float4 b = *reinterpret_cast<const float4 *>(&sm.v[t][4 * x + 64 * c]);
                    const float vv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        // a token that a row does not see adds nothing, whatever its V holds
                        if (inner || t <= see[i] - t0)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                o[i][4 * c + e] = fmaf(pr[i], vv[e], o[i][4 * c + e]);
                    }
                }
            }
            __syncthreads();  // V may be replaced, while the next S is made
            copy(sm.v, V);
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncthreads();
        // ---- the end of the part
        const int first_bad = sm.bad;
        float inv[4], ls[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int h = 8; h > 0; h >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], h);
            inv[i] = l[i] == 0.0f ? 0.0f : 1.0f / l[i];
            ls[i] = l[i] == 0.0f ? -INFINITY : m[i] + log2f(l[i]);
        }
        const ChunkSpace &sp = sm.space;
        int cf, cl;
        chunk_groups(sp, g, cf, cl);
        auto row_at = [&](int r) {
            return (size_t)(g.row0 + tok0 + r / p.G) * p.Hq + head * p.G + r % p.G;
        };
        if (cf == cl) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = 4 * y + i;
                if (r >= M) continue;
                const bool zero = see[i] >= first_bad;
                const size_t row = row_at(r);
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    float4 w = make_float4(o[i][4 * c] * inv[i], o[i][4 * c + 1] * inv[i],
                                           o[i][4 * c + 2] * inv[i], o[i][4 * c + 3] * inv[i]);
                    if (zero) w = make_float4(0.f, 0.f, 0.f, 0.f);
                    *reinterpret_cast<float4 *>(out + row * D + 4 * x + 64 * c) = w;
                }
                if (x == 0 && p.lse) p.lse[row] = zero ? 0.0f : ls[i] * 0.69314718055994531f;
            }
            continue;
        }
        const int slot = 2 * blockIdx.x + (g.x0 == sp.s ? 0 : 1);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = 4 * y + i;
            if (r >= M) continue;
#pragma unroll
            for (int c = 0; c < NC; ++c)
                __stcg(p.part + ((size_t)slot * (D / 4) + x + 16 * c) * p.slot_rows + r,
                       make_float4(o[i][4 * c] * inv[i], o[i][4 * c + 1] * inv[i],
                                   o[i][4 * c + 2] * inv[i], o[i][4 * c + 3] * inv[i]));
            if (x == 0) __stcg(p.part_lse + (size_t)slot * p.slot_rows + r, ls[i]);
        }
        if (tid == 0) __stcg(p.part_bad + 2 * slot, first_bad);
        __syncthreads();
        int *counter = p.counters + cf * p.S + blockIdx.x % p.S;
        const int F = cl - cf + 1;
        if (tid == 0) {
            __threadfence();  // what the barrier made visible to this thread, too
            const int before = atomicAdd(counter, 1);
            sm.last = before == F - 1;
            if (before == F - 1) *counter = 0;
            __threadfence();
        }
        __syncthreads();
        if (!sm.last) continue;
        const ChunkJoin jn = {F, cf, (int)(blockIdx.x % p.S), chunk_start(cf, sp.T, sp.C) < g.pu ? 1 : 0,
                              M, M, 1, g.row0 + tok0, head, g.L + tok0, tid, NT, 0};
        chunk_join<D, float>(p, jn, sm.w);
    }
}

template <int D>
cudaError_t launch_d(const ChunkParams &p, int ctas, cudaStream_t stream) {
    const int smem = (int)sizeof(ChunkSmem<D>);
    const cudaError_t e = cudaFuncSetAttribute(chunk_simt_kernel<D>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    return launch_pdl(chunk_simt_kernel<D>, dim3((unsigned)ctas), dim3(NT), (size_t)smem, stream, 0u,
                      p);
}

}  // namespace

cudaError_t launch_chunk_simt(const ChunkParams &p, int D, int ctas, cudaStream_t stream) {
    return D == 64 ? launch_d<64>(p, ctas, stream) : launch_d<128>(p, ctas, stream);
}

}  // namespace svf
