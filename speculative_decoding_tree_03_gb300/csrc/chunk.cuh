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
    int *part_bad;     // [2 CTAs][2 halves] first token of a piece whose page is not in the cache, or a flag
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

// Quotient of what is mostly below 2^32 (a 64-bit division takes ten times as long). Not inlined, as
// other things here that a part needs once: the kernels' code is to stay in the instruction
// cache (a call of one token spends more time fetching code than on anything else).
static __device__ __noinline__ long long quot(long long a, long long b) {
    if (((unsigned long long)(a | b) >> 32) == 0) return (long long)((unsigned)a / (unsigned)b);
    return a / b;
}

// sum_{i < n} floor((a i + b) / m), by Euclid's steps on (a, m)
static __device__ __noinline__ long long floor_sum(long long n, unsigned m, unsigned a,
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
    const unsigned end = (unsigned)s.L + (unsigned)min((long long)(k + 1) * p.TB, (long long)s.n);
    return (int)((end + BN - 1) / BN);  // end is below 2^31
}

// Tiles of the first k row blocks of a sequence, for one head.
template <int BN>
__device__ __forceinline__ long long chunk_tiles_before(const ChunkParams &p, const ChunkSeq &s,
                                                        int k) {
    const int full = min(k, s.n / p.TB);
    long long t = 0;
    if (full > 0)
        t = floor_sum(full, BN, (unsigned)p.TB,
                      (unsigned long long)s.L + (unsigned)p.TB + (unsigned)(BN - 1));
    if (k > full) t += ((unsigned)s.L + (unsigned)s.n + BN - 1) / BN;
    return t;
}

// The tile space of the call as a CTA sees it.
struct ChunkSpace {
    long long T, s, e;  // its length; this group's share
    long long pu;       // where the unit begins that holds s
    int C, grp, lead;
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
    return quot((long long)c * T, C);
}
__device__ __forceinline__ int chunk_group_of(long long x, long long T, int C) {
    return (int)quot((x + 1) * (long long)C - 1, T);
}

// The part's first tile, and how many it has (0: it ends in the unit's lead, nothing to do).
__device__ __forceinline__ int chunk_part(const ChunkSpace &sp, const ChunkSeg &g, int &first) {
    const long long at = g.pu + sp.lead;
    first = (int)max(g.x0 - at, 0ll);
    return (int)max(g.x1 - at, 0ll) - first;
}

// The groups with the first and the last tile of a unit.
__device__ __forceinline__ void chunk_groups(const ChunkSpace &sp, const ChunkSeg &g, int &cf,
                                             int &cl) {
    cf = chunk_group_of(g.pu + sp.lead, sp.T, sp.C);
    cl = chunk_group_of(g.pu + sp.lead + g.t - 1, sp.T, sp.C);
}

// Tiles and units of the sequences lo .. hi - 1.
struct ChunkCount {
    long long tiles, units;
};
template <int BN>
__device__ __noinline__ ChunkCount chunk_count(const ChunkParams &p, int lo, int hi) {
    ChunkCount c = {0, 0};
    for (int b = lo; b < hi; ++b) {
        const ChunkSeq s = chunk_seq(p, b);
        if (!s.ok || s.n == 0) continue;
        const int nb = chunk_blocks(p, s.n);
        c.tiles += chunk_tiles_before<BN>(p, s, nb) * p.NHB;
        c.units += (long long)nb * p.NHB;
    }
    return c;
}
__device__ __forceinline__ ChunkCount chunk_scan(ChunkCount c, int lane) {  // inclusive, of a warp
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long t = __shfl_up_sync(0xffffffffu, c.tiles, o);
        const long long u = __shfl_up_sync(0xffffffffu, c.units, o);
        if (lane >= o) {
            c.tiles += t;
            c.units += u;
        }
    }
    return c;
}

// The space of a call with these totals: what the group's share is.
__device__ __forceinline__ ChunkSpace chunk_share(const ChunkParams &p, ChunkCount all) {
    ChunkSpace sp;
    // With no more units than groups every group has about one of them at most, and a lead in
    // front of each would leave groups without tiles.
    sp.lead = all.units <= p.groups ? 0 : p.lead;
    sp.T = all.tiles + all.units * sp.lead;
    const long long C = quot(sp.T, p.min_tiles);
    sp.C = (int)(C < 1 ? 1 : (C > p.groups ? p.groups : C));
    sp.grp = blockIdx.x / p.S;
    sp.s = sp.e = sp.T;
    if (sp.grp < sp.C && sp.T > 0) {
        sp.s = chunk_start(sp.grp, sp.T, sp.C);
        sp.e = chunk_start(sp.grp + 1, sp.T, sp.C);
    }
    sp.pu = 0;
    sp.b = sp.hb = sp.k = 0;
    return sp;
}

// Finds the sequence of lo .. hi - 1, which begin at pb, that holds sp.s.
template <int BN>
__device__ __forceinline__ void chunk_find(const ChunkParams &p, ChunkSpace &sp, int lo, int hi,
                                           long long pb) {
    for (int b = lo; b < hi; ++b) {
        const ChunkCount c = chunk_count<BN>(p, b, b + 1);
        const long long len = c.tiles + c.units * sp.lead;
        if (sp.s < pb + len) {
            sp.pu = pb;  // of the sequence, so far
            sp.b = b;
            return;
        }
        pb += len;
    }
}

// By a warp: the head block, and the row block by a search with 32 probes a step.
template <int BN>
__device__ __forceinline__ void chunk_locate(const ChunkParams &p, ChunkSpace &sp, int lane) {
    const ChunkSeq q = chunk_seq(p, sp.b);
    const int nb = chunk_blocks(p, q.n);
    auto before = [&](int k) { return chunk_tiles_before<BN>(p, q, k) + (long long)k * sp.lead; };
    const long long off = sp.s - sp.pu;
    if (nb == 1 && p.NHB == 1) return;
    const long long F = before(nb);
    sp.hb = (int)quot(off, F);
    const long long x = off - (long long)sp.hb * F;
    int a = 0, z = nb;  // before(a) <= x < before(z)
    while (z - a > 1) {
        const int step = (z - a + 31) / 32;
        const int at = min(a + step * lane, z);
        const bool le = at < z && before(at) <= x;
        const int last = 31 - __clz(__ballot_sync(0xffffffffu, le));  // lane 0 is always in
        z = min(a + step * (last + 1), z);
        a = a + step * last;
    }
    sp.k = a;
    sp.pu += (long long)sp.hb * F + before(a);
}

constexpr int kChunkWarpBatch = 128;  // sequences that one warp lays out (four a lane)

// Lays out the tile space, by one warp (B <= kChunkWarpBatch).
template <int BN>
__device__ __noinline__ ChunkSpace chunk_layout_warp(const ChunkParams &p, int lane) {
    constexpr unsigned FULL = 0xffffffffu;
    const int per = (p.B + 31) / 32, lo = min(lane * per, p.B), hi = min(lo + per, p.B);
    const ChunkCount mine = chunk_count<BN>(p, lo, hi), incl = chunk_scan(mine, lane);
    const ChunkCount all = {__shfl_sync(FULL, incl.tiles, 31), __shfl_sync(FULL, incl.units, 31)};
    ChunkSpace sp = chunk_share(p, all);
    if (sp.s >= sp.e) return sp;
    const long long len = mine.tiles + mine.units * sp.lead;
    const long long first = incl.tiles + incl.units * sp.lead - len;
    const bool holds = first <= sp.s && sp.s < first + len;
    if (holds) chunk_find<BN>(p, sp, lo, hi, first);
    const int who = __ffs(__ballot_sync(FULL, holds)) - 1;
    sp.pu = __shfl_sync(FULL, sp.pu, who);
    sp.b = __shfl_sync(FULL, sp.b, who);
    chunk_locate<BN>(p, sp, lane);
    return sp;
}

// The same by all NT threads of the CTA, which meet in it. `sums` is shared memory.
template <int BN, int NT>
__device__ __noinline__ void chunk_layout(const ChunkParams &p, ChunkSpace *out, ChunkCount *sums) {
    constexpr int NW = NT / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int lo = (int)((unsigned)p.B * threadIdx.x / NT);  // B <= 2^20
    const int hi = (int)((unsigned)p.B * (threadIdx.x + 1) / NT);
    const ChunkCount mine = chunk_count<BN>(p, lo, hi), incl = chunk_scan(mine, lane);
    if (lane == 31) sums[warp] = incl;
    __syncthreads();
    ChunkCount before = {0, 0}, all = {0, 0};
    for (int w = 0; w < NW; ++w) {
        const ChunkCount c = sums[w];
        if (w < warp) {
            before.tiles += c.tiles;
            before.units += c.units;
        }
        all.tiles += c.tiles;
        all.units += c.units;
    }
    ChunkSpace sp = chunk_share(p, all);
    const long long len = mine.tiles + mine.units * sp.lead;
    const long long first =
        before.tiles + incl.tiles + (before.units + incl.units) * sp.lead - len;
    if (threadIdx.x == 0 && sp.s >= sp.e) *out = sp;
    if (sp.s < sp.e && first <= sp.s && sp.s < first + len) {
        chunk_find<BN>(p, sp, lo, hi, first);
        *out = sp;
    }
    __syncthreads();
    if (warp == 0 && sp.s < sp.e) {
        sp = *out;
        chunk_locate<BN>(p, sp, lane);
        __syncwarp();
        if (lane == 0) *out = sp;
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
    g.x1 = min(g.pu + sp.lead + g.t, sp.e);
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
    g.x1 = min(g.pu + sp.lead + g.t, sp.e);
    return true;
}

// The join of the pieces of a unit.
struct ChunkJoin {
    int F, cf, lane_cta, first_slot;  // pieces; their first group; the CTA's place in a group
    int M, half_rows;  // rows of the block; row m is at m, or from half_rows on at 128 + m - half_rows
    int halves;        // part_bad entries of a piece
    int qrow0, head, see0;  // the block's first row of q, the KV head, the last token of its first row
    int tid, nt, bar;       // the threads (whole warps) and a named barrier for them
};

template <typename T>
__device__ __forceinline__ void store4(T *p, float4 v);
template <>
__device__ __forceinline__ void store4<float>(float *p, float4 v) {
    *reinterpret_cast<float4 *>(p) = v;
}
template <>
__device__ __forceinline__ void store4<__nv_bfloat16>(__nv_bfloat16 *p, float4 v) {
    *reinterpret_cast<uint2 *>(p) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
}

// Few rows: a warp to a row, its lanes the pieces' log-sum-exps and then the row's chunks of
// 16 bytes. Many: a thread to a chunk of a row, rows next to each other, which reads whole
// lines. Loads go out several at a time: a round trip takes about 0.6 us. `all` is shared
// memory for M floats.
template <int D, typename T>
__device__ __noinline__ void chunk_join(const ChunkParams &p, const ChunkJoin &j, float *all) {
    constexpr unsigned FULL = 0xffffffffu;
    constexpr int C = D / 4, U = 4;
    const int lane = j.tid & 31, F = j.F, M = j.M;
    T *out = static_cast<T *>(p.out);
    auto slot_of = [&](int f) {
        return 2 * ((j.cf + f) * p.S + j.lane_cta) + (f == 0 ? j.first_slot : 0);
    };
    auto place = [&](int m) { return m < j.half_rows ? m : 128 + m - j.half_rows; };
    auto lse_at = [&](int f, int at) {
        return f < F ? __ldcg(p.part_lse + slot_of(f) * p.slot_rows + at) : -INFINITY;
    };
    const unsigned piece = (unsigned)(C * p.slot_rows);  // float4s of a piece
    auto part_at = [&](int f, int c, int at) {
        return f < F ? __ldcg(p.part + ((size_t)slot_of(f) * piece + (unsigned)(c * p.slot_rows + at)))
                     : make_float4(0.f, 0.f, 0.f, 0.f);
    };
    auto out_row = [&](int m) {
        return (size_t)(j.qrow0 + m / p.G) * p.Hq + (size_t)j.head * p.G + m % p.G;
    };
    auto fma4 = [](float4 &acc, float w, const float4 &a) {
        acc.x = fmaf(w, a.x, acc.x);
        acc.y = fmaf(w, a.y, acc.y);
        acc.z = fmaf(w, a.z, acc.z);
        acc.w = fmaf(w, a.w, acc.w);
    };
    // rows that see a token without a page (all of them, where a piece was lost) are 0
    auto first_bad = [&] {
        int lost = kPieceFine;
        for (int i = lane; i < F * j.halves; i += 32) {
            const int f = i / j.halves;
            lost = min(lost, __ldcg(p.part_bad + 2 * slot_of(f) + i - f * j.halves));
        }
        return lost;
    };
    int lost = kPieceFine;
    auto put = [&](int m, int c, float4 v) {
        if (j.see0 + m / p.G >= lost) v = make_float4(0.f, 0.f, 0.f, 0.f);
        store4(out + out_row(m) * D + c * 4, v);
    };
    auto put_lse = [&](int m, float lse2) {
        if (p.lse) p.lse[out_row(m)] = j.see0 + m / p.G >= lost ? 0.0f : lse2 * 0.69314718055994531f;
    };
    if (M * 8 <= j.nt && F <= 32) {
        for (int m = j.tid >> 5; m < M; m += j.nt >> 5) {
            const int at = place(m), c = lane < C ? lane : 0;
            const float v = lse_at(lane, at);
            float4 a[U];
#pragma unroll
            for (int u = 0; u < U; ++u) a[u] = part_at(u, c, at);
            lost = __reduce_min_sync(FULL, first_bad());
            const float mx = warp_max(v);
            const float sum = warp_sum(v == -INFINITY ? 0.0f : exp2f(v - mx));
            const float lse = mx + log2f(sum);
            const float w = v == -INFINITY ? 0.0f : exp2f(v - lse);
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
            for (int f0 = 0;;) {
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const float vu = __shfl_sync(FULL, v, (f0 + u) & 31);
                    const float wu = __shfl_sync(FULL, w, (f0 + u) & 31);
                    if (f0 + u < F && vu != -INFINITY) fma4(acc, wu, a[u]);
                }
                if ((f0 += U) >= F) break;
#pragma unroll
                for (int u = 0; u < U; ++u) a[u] = part_at(f0 + u, c, at);
            }
            if (lane < C) put(m, lane, acc);
            if (lane == 0) put_lse(m, lse);
        }
        return;
    }
    lost = __reduce_min_sync(FULL, first_bad());
    auto sync = [&] { asm volatile("barrier.cta.sync %0, %1;" ::"r"(j.bar), "r"(j.nt) : "memory"); };
    for (int m = j.tid; m < M; m += j.nt) {
        const int at = place(m);
        float mx = -INFINITY, sum = 0.0f;
        for (int f0 = 0; f0 < F; f0 += U) {
            float v[U], nm = mx;
#pragma unroll
            for (int u = 0; u < U; ++u) v[u] = lse_at(f0 + u, at);
#pragma unroll
            for (int u = 0; u < U; ++u) nm = fmaxf(nm, v[u]);
            if (mx != -INFINITY) sum *= exp2f(mx - nm);
#pragma unroll
            for (int u = 0; u < U; ++u) sum += v[u] == -INFINITY ? 0.0f : exp2f(v[u] - nm);
            mx = nm;
        }
        all[m] = mx + log2f(sum);
        put_lse(m, all[m]);
    }
    sync();
    // bf16: four chunks at once, two pieces of each, since a unit of many rows is mostly split between
    // two groups (a mixed batch of 5003 rows 297 us, a prompt of 8192 424; one chunk, four
    // pieces 311 and 436; two and four 304 and 430, four and four 315 and 442, eight and two 300 and 428).
    // fp32: one chunk, four pieces, whose units are split into more (333 rows of 5 sequences 48.2 us;
    // four and two 50.4, and more loads take registers from the tiles).
    if constexpr (sizeof(T) == 2) {
        constexpr int IT = 4, UP = 2;
        for (int it0 = j.tid; it0 < M * C; it0 += IT * j.nt) {
            int c[IT], m[IT];
            float lse[IT];
            float4 acc[IT];
#pragma unroll
            for (int i = 0; i < IT; ++i) {
                const int it = min(it0 + i * j.nt, M * C - 1);
                c[i] = it / M;
                m[i] = it - c[i] * M;
                lse[i] = all[m[i]];
                acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            }
            for (int f0 = 0; f0 < F; f0 += UP) {
                float v[IT][UP];
                float4 a[IT][UP];
#pragma unroll
                for (int i = 0; i < IT; ++i)
#pragma unroll
                    for (int u = 0; u < UP; ++u) {
                        v[i][u] = lse_at(f0 + u, place(m[i]));
                        a[i][u] = part_at(f0 + u, c[i], place(m[i]));
                    }
#pragma unroll
                for (int i = 0; i < IT; ++i)
#pragma unroll
                    for (int u = 0; u < UP; ++u)
                        if (v[i][u] != -INFINITY) fma4(acc[i], exp2f(v[i][u] - lse[i]), a[i][u]);
            }
#pragma unroll
            for (int i = 0; i < IT; ++i)
                if (it0 + i * j.nt < M * C) put(m[i], c[i], acc[i]);
        }
    } else {
        for (int it = j.tid; it < M * C; it += j.nt) {
            const int c = it / M, m = it - c * M, at = place(m);
            const float lse = all[m];
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int f0 = 0; f0 < F; f0 += 4) {
                float v[4];
                float4 a[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    v[u] = lse_at(f0 + u, at);
                    a[u] = part_at(f0 + u, c, at);
                }
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    if (v[u] != -INFINITY) fma4(acc, exp2f(v[u] - lse), a[u]);
            }
            put(m, c, acc);
        }
    }
    sync();  // `all` is used again
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
