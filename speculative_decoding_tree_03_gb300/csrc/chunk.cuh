// chunk.cuh -- how the two chunk-attention kernels divide a call, and how they join it.
//
// Sequence b has n_b new rows on top of L_b cached tokens; row i of it sees the tokens
// t <= L_b + i. Rows are taken together with the G query heads of a KV head (token-major),
// in blocks of TB tokens; block k needs the key tiles of BN tokens
//     tiles(b, k) = ceil((L_b + min((k + 1) TB, n_b)) / BN).
// A unit is (sequence, KV head, block). The CTAs form groups of S, one CTA per KV head of a
// head block (S = Hkv where that fills the GPU), whose CTAs go through the same token ranges
// side by side: a token's row of the cache holds all heads. The units' tiles, with `lead` more in
// front of each for what a unit costs besides (its Q, its output), are laid end to
// end, sequence by sequence (its head blocks, their row blocks), T in all, and group c of C
// takes [cT/C, (c+1)T/C): every CTA the same work, whether the call is one token after a long
// context or a prompt of thousands. The lengths are on the device only, so
// every CTA lays the space out by itself: the sum over a sequence's blocks has the closed
// form floor_sum, and sequences are summed by all threads.
//
// A unit inside one group is written as final output. Of a unit split between groups each
// piece is written as normalised fp32 rows with their log2-sum-exp to the workspace and
// counted (a piece has tiles: one that ends in the lead is none); whoever counts last joins the
// pieces in their order,
//     out = sum_f w_f O_f,  w_f = 2^(lse_f - max) / sum,
// so nobody waits for another CTA, and the result does not depend on who it was. A split unit
// is the last of the group that holds its first tile, so one counter per CTA is enough;
// the joining CTA puts it back to zero.
#pragma once

#include "common.cuh"
#include "internal.h"

namespace svf {

constexpr int kChunkMaxCtas = 512;   // counters in the workspace
constexpr int kChunkHeadBytes = kChunkMaxCtas * 4 + 256;

struct ChunkParams {
    const void *q, *k_cache, *v_cache;
    void *out;
    float *lse;
    const int32_t *page_table, *seq_lens, *row_offsets;
    int32_t *status;
    int B, rows, Hq, Hkv, G, ps, num_pages, max_pages;
    int TB;        // tokens of a row block
    int S, NHB;    // heads of a group; head blocks (S * NHB = Hkv)
    int groups;    // groups of the grid
    int min_tiles; // a group has at least this many tiles, or there are fewer groups
    int lead;      // tiles that a unit's beginning and end are worth
    float scale_log2;
    unsigned long long wait_ns;
    int *counters;     // [kChunkMaxCtas] zero between calls
    int *done;         // [2] CTAs that are through; some CTA gave up (both zero between calls)
    int *gave_up;      // [2 CTAs] first and last sequence of a CTA that gave up
    int *part_bad;     // [2 CTAs] first token of a piece whose page is not in the cache, or a flag
    float *part_lse;   // [2 CTAs][slot_rows]
    float4 *part;      // [2 CTAs][D / 4][slot_rows]
    int slot_rows;
};

constexpr int kPieceFine = 0x7fffffff;  // part_bad: every page was there
constexpr int kPieceLost = -1;          // part_bad: a wait gave up

struct ChunkSeq {
    int L, n, row0;
    bool rows_ok;  // its rows are inside the call's
    bool ok;       // and its lengths fit
};

__device__ __forceinline__ ChunkSeq chunk_seq(const ChunkParams &p, int b) {
    ChunkSeq s;
    s.L = __ldg(p.seq_lens + b);
    s.row0 = __ldg(p.row_offsets + b);
    const int end = __ldg(p.row_offsets + b + 1);
    s.rows_ok = s.row0 >= 0 && end >= s.row0 && end <= p.rows;
    s.n = s.rows_ok ? end - s.row0 : 0;
    s.ok = s.rows_ok && s.L >= 0 && (long long)s.L + s.n <= (long long)p.max_pages * p.ps;
    return s;
}

// sum_{i < n} floor((a i + b) / m), by Euclid's steps on (a, m)
__device__ __forceinline__ long long floor_sum(long long n, unsigned m, unsigned a,
                                               unsigned long long b) {
    long long r = 0;
    while (n > 0) {
        r += (long long)(a / m) * (n * (n - 1) / 2) + (long long)(b / m) * n;
        a %= m;
        b %= m;
        const unsigned long long y = (unsigned long long)a * (unsigned long long)n + b;
        if (y < m) break;
        n = (long long)(y / m);
        b = y % m;
        const unsigned t = m;
        m = a;
        a = t;
    }
    return r;
}

__device__ __forceinline__ int chunk_blocks(const ChunkParams &p, int n) {
    return (n + p.TB - 1) / p.TB;
}

template <int BN>
__device__ __forceinline__ int chunk_tiles(const ChunkParams &p, const ChunkSeq &s, int k) {
    const long long end = (long long)s.L + min((long long)(k + 1) * p.TB, (long long)s.n);
    return (int)((end + BN - 1) / BN);
}

// Length of the first k row blocks of a sequence in the tile space, for one head.
template <int BN>
__device__ __forceinline__ long long chunk_tiles_before(const ChunkParams &p, const ChunkSeq &s,
                                                        int k) {
    const int full = min(k, s.n / p.TB);
    long long t = (long long)k * p.lead;
    if (full > 0)
        t += floor_sum(full, BN, (unsigned)p.TB,
                      (unsigned long long)s.L + (unsigned)p.TB + (unsigned)(BN - 1));
    if (k > full) t += ((long long)s.L + s.n + BN - 1) / BN;
    return t;
}

template <int BN>
__device__ __forceinline__ long long chunk_seq_tiles(const ChunkParams &p, const ChunkSeq &s) {
    if (!s.ok || s.n == 0) return 0;
    return chunk_tiles_before<BN>(p, s, chunk_blocks(p, s.n)) * p.NHB;
}

// The tile space of the call as a CTA sees it.
struct ChunkSpace {
    long long T, s, e;  // all tiles; this group's
    long long pu;       // first tile of the unit that holds s
    int C, grp;
    int b, hb, k;       // that unit
};

// A part [x0, x1) of one unit's length, the unit beginning at pu: `lead` and then its t tiles.
struct ChunkSeg {
    long long pu, x0, x1;
    int b, hb, k, t;
    int L, n, row0;
};

// First tile of group c's share and the group whose share holds tile x.
__device__ __forceinline__ long long chunk_start(int c, long long T, int C) {
    return (long long)c * T / C;
}
__device__ __forceinline__ int chunk_group_of(long long x, long long T, int C) {
    return (int)(((x + 1) * (long long)C - 1) / T);
}

// The part's first tile, and how many it has (0: it ends in the unit's lead, nothing to do).
__device__ __forceinline__ int chunk_part(const ChunkParams &p, const ChunkSeg &g, int &first) {
    const long long at = g.pu + p.lead;
    first = (int)max(g.x0 - at, 0ll);
    return (int)max(g.x1 - at, 0ll) - first;
}

// The groups with the first and the last tile of a unit.
__device__ __forceinline__ void chunk_groups(const ChunkParams &p, const ChunkSpace &sp,
                                             const ChunkSeg &g, int &cf, int &cl) {
    cf = chunk_group_of(g.pu + p.lead, sp.T, sp.C);
    cl = chunk_group_of(g.pu + p.lead + g.t - 1, sp.T, sp.C);
}

// Lays out the tile space; all NT threads of the CTA, which meet in it. `wsum` is
// shared memory for NT / 32 sums.
template <int BN, int NT>
__device__ void chunk_layout(const ChunkParams &p, ChunkSpace *sp, long long *wsum) {
    constexpr unsigned FULL = 0xffffffffu;
    constexpr int NW = NT / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long lo = (long long)p.B * threadIdx.x / NT;
    const long long hi = (long long)p.B * (threadIdx.x + 1) / NT;
    long long mine = 0;
    for (long long b = lo; b < hi; ++b) mine += chunk_seq_tiles<BN>(p, chunk_seq(p, (int)b));
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(FULL, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) wsum[warp] = incl;
    __syncthreads();
    if (warp == 0) {
        const long long w = lane < NW ? wsum[lane] : 0;
        long long wi = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long v = __shfl_up_sync(FULL, wi, o);
            if (lane >= o) wi += v;
        }
        __syncwarp();
        if (lane < NW) wsum[lane] = wi - w;
        if (lane == 31) sp->T = wi;
    }
    __syncthreads();
    const long long T = sp->T;
    const long long first = wsum[warp] + incl - mine;
    long long Cl = T / p.min_tiles;
    Cl = Cl < 1 ? 1 : (Cl > p.groups ? p.groups : Cl);
    const int C = (int)Cl;
    const int grp = blockIdx.x / p.S;
    const long long s = grp < C && T > 0 ? chunk_start(grp, T, C) : T;
    const long long e = grp < C && T > 0 ? chunk_start(grp + 1, T, C) : T;
    if (s < e && first <= s && s < first + mine) {
        // this thread's sequences hold tile s
        long long pb = first;
        for (long long b = lo; b < hi; ++b) {
            const long long tb = chunk_seq_tiles<BN>(p, chunk_seq(p, (int)b));
            if (s < pb + tb) {
                sp->pu = pb;  // of the sequence, so far
                sp->b = (int)b;
                break;
            }
            pb += tb;
        }
    }
    __syncthreads();
    if (warp == 0) {
        if (s < e) {
            // the head block, and the row block by a search with 32 probes a step
            const ChunkSeq q = chunk_seq(p, sp->b);
            const int nb = chunk_blocks(p, q.n);
            const long long F = chunk_tiles_before<BN>(p, q, nb);
            const long long off = s - sp->pu;
            const int hb = (int)(off / F);
            const long long x = off - (long long)hb * F;
            int a = 0, z = nb;  // before(a) <= x < before(z)
            while (z - a > 1) {
                const int step = (z - a + 31) / 32;
                const int at = min(a + step * lane, z);
                const bool le = at < z && chunk_tiles_before<BN>(p, q, at) <= x;
                const unsigned m = __ballot_sync(FULL, le);
                const int last = 31 - __clz(m);  // lane 0 is always in
                z = min(a + step * (last + 1), z);
                a = a + step * last;
            }
            __syncwarp();
            if (lane == 0) {
                sp->hb = hb;
                sp->k = a;
                sp->pu += (long long)hb * F + chunk_tiles_before<BN>(p, q, a);
            }
        }
        if (lane == 0) {
            sp->s = s;
            sp->e = e;
            sp->C = C;
            sp->grp = grp;
        }
    }
    __syncthreads();
}

template <int BN>
__device__ __forceinline__ bool chunk_first(const ChunkParams &p, const ChunkSpace &sp,
                                            ChunkSeg &g) {
    if (sp.s >= sp.e) return false;
    const ChunkSeq q = chunk_seq(p, sp.b);
    g.b = sp.b;
    g.hb = sp.hb;
    g.k = sp.k;
    g.L = q.L;
    g.n = q.n;
    g.row0 = q.row0;
    g.pu = sp.pu;
    g.t = chunk_tiles<BN>(p, q, g.k);
    g.x0 = sp.s;
    g.x1 = min(g.pu + p.lead + g.t, sp.e);
    return true;
}

// The next part of this group's share; false behind the last.
template <int BN>
__device__ __forceinline__ bool chunk_next(const ChunkParams &p, const ChunkSpace &sp,
                                           ChunkSeg &g) {
    if (g.x1 >= sp.e) return false;
    ChunkSeq q;
    q.L = g.L;
    q.n = g.n;
    if (++g.k >= chunk_blocks(p, g.n)) {
        g.k = 0;
        if (++g.hb >= p.NHB) {
            g.hb = 0;
            do {
                if (++g.b >= p.B) return false;
                q = chunk_seq(p, g.b);
            } while (!q.ok || q.n == 0);
            g.L = q.L;
            g.n = q.n;
            g.row0 = q.row0;
        }
    }
    g.pu = g.x1;
    g.x0 = g.x1;
    g.t = chunk_tiles<BN>(p, q, g.k);
    g.x1 = min(g.pu + p.lead + g.t, sp.e);
    return true;
}

// Status words, and zero outputs of a sequence whose lengths do not fit; `nt` threads,
// thread `tid`, of one CTA (b = blockIdx.x, + gridDim.x, ..). `any` is an or over them.
template <int D, typename T, typename Any>
__device__ void chunk_status(const ChunkParams &p, int tid, int nt, Any any) {
    for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
        const ChunkSeq s = chunk_seq(p, b);
        bool bad = false;
        if (s.ok && s.n > 0) {
            const int pages = (int)(((long long)s.L + s.n + p.ps - 1) / p.ps);
            const int32_t *row = p.page_table + (size_t)b * p.max_pages;
#pragma unroll 4
            for (int i = tid; i < pages; i += nt) {
                const int id = __ldg(row + i);
                bad |= id < 0 || id >= p.num_pages;
            }
        }
        bad = any(bad);
        if (tid == 0) p.status[b] = !s.ok ? SVF_DEV_BAD_LENGTH : bad ? SVF_DEV_BAD_PAGE : 0;
        if (!s.ok && s.n > 0) {
            T *out = static_cast<T *>(p.out) + (size_t)s.row0 * p.Hq * D;
            const long long all = (long long)s.n * p.Hq * (D * (int)sizeof(T) / 16);
            for (long long i = tid; i < all; i += nt)
                reinterpret_cast<uint4 *>(out)[i] = make_uint4(0, 0, 0, 0);
            if (p.lse)
                for (long long i = tid; i < (long long)s.n * p.Hq; i += nt)
                    p.lse[(size_t)s.row0 * p.Hq + i] = 0.0f;
        }
    }
}

}  // namespace svf
