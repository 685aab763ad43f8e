// pages_shared.cu -- sequences that share pages of the paged KV cache: forks, the
// copies of their last pages, and the release of pages that others still hold.
//
// A page that h sequences hold has shares = h - 1 (0 for a page of one sequence and
// for a free one, so that page_reserve needs to know nothing of it). A fork of a
// sequence of L tokens holds the source's floor(L / ps) full pages too (shares + 1
// each; full pages are never written again) and, where L % ps > 0, a page of its own
// from the stack, into which the first L % ps tokens of the source's last page are
// copied in every layer. A release takes one holder away from each page; a page
// without any goes back onto the stack.
//
// Forks are served in order, as page_reserve serves sequences: fork f lacks
// need_f = [L % ps > 0] pages, I_f = sum_{f' <= f} need_f', and it is served when
// need_f = 0 or I_f <= F; its page is free[F - I_f].
//
// The order of the stack after a release must not depend on the order of atomics.
// With c holders of a page leaving in one call, after the counts are lowered
// shares = h - 1 - c < 0 says that nobody is left; among those c sequences the last
// one (by index) puts the page back, found by atomicMin(shares, kClaim - b). So the
// pages come in the order of a release without shares, sequence by sequence in table
// order, and a release of what nobody shares leaves the same stack as page_release.
#include "common.cuh"
#include "internal.h"
#include "page_math.cuh"

namespace svf {

namespace {

constexpr int kForkThreads = 256;
constexpr int kShareThreads = 1024;
constexpr int kCopyThreads = 256;
constexpr int kClaim = -(1 << 30);  // below any count: at most 2^30 holders leave in a call
constexpr int kMostGifts = (1 << 30) - 1;

struct ForkArgs {
    int32_t *table;
    const int32_t *free_pages;
    int32_t *state, *shares, *seq_lens;
    const int32_t *src, *dst;
    int32_t *copy_src, *copy_dst, *copy_len, *status;
    int B, F, max_pages, ps, num_pages;
};

// grid (forks, chunks): the row of fork blockIdx.x in gridDim.y parts. Every CTA looks
// at all forks by itself (which rows are used twice, how many pages the forks before
// its own take), as the page-reserve kernel does with the sequences.
__global__ void __launch_bounds__(kForkThreads) page_fork_kernel(ForkArgs a) {
    extern __shared__ unsigned s_row[];  // [B]: how many forks write the row; bit 31: one reads it
    __shared__ int s_part[kForkThreads / 32];
    __shared__ int s_free;
    const int f = blockIdx.x, c = blockIdx.y, C = gridDim.y, tid = threadIdx.x;
    for (int i = tid; i < a.B; i += kForkThreads) s_row[i] = 0;
    pdl_wait();
    pdl_launch_dependents();
    if (tid == 0) s_free = min(max(*(volatile int32_t *)a.state, 0), a.num_pages);
    __syncthreads();
    auto is_row = [&](int r) { return r >= 0 && r < a.B; };
    for (int i = tid; i < a.F; i += kForkThreads) {
        const int s = a.src[i], d = a.dst[i];
        if (is_row(s)) atomicOr(&s_row[s], 1u << 31);
        if (is_row(d)) atomicAdd(&s_row[d], 1u);
    }
    __syncthreads();
    // a fork's rows are fine: nobody else writes its destination, nobody reads that,
    // and nobody writes its source
    auto rows_ok = [&](int s, int d) {
        return is_row(s) && is_row(d) && s_row[d] == 1u && s_row[s] == (1u << 31);
    };
    // the source's length; -1 where it cannot be
    auto length = [&](int s) {
        const int L = a.seq_lens[s];
        return L >= 0 && (long long)L <= (long long)a.max_pages * a.ps ? L : -1;
    };
    int before = 0;
    for (int i = tid; i < f; i += kForkThreads) {
        const int s = a.src[i], d = a.dst[i];
        if (rows_ok(s, d)) {
            const int L = length(s);
            before += L > 0 && L % a.ps != 0;
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
    if ((tid & 31) == 0) s_part[tid >> 5] = before;
    __syncthreads();
    before = 0;
#pragma unroll
    for (int i = 0; i < kForkThreads / 32; ++i) before += s_part[i];
    const int F = s_free;
    const int s = a.src[f], d = a.dst[f];
    const bool fine = rows_ok(s, d);
    const int L = fine ? length(s) : -1;
    const int full = L >= 0 ? L / a.ps : 0, part = L >= 0 ? L % a.ps : 0;
    const int incl = before + (part > 0);
    const bool served = L >= 0 && (part == 0 || incl <= F);
    const int32_t *from = a.table + (size_t)(fine ? s : 0) * a.max_pages;
    auto is_page = [&](int p) { return p >= 0 && p < a.num_pages; };
    const int fresh = served && part > 0 ? a.free_pages[F - incl] : -1;
    bool bad = false;  // a page id outside the cache
    if (L >= 0) {
        int32_t *to = a.table + (size_t)d * a.max_pages;
        const int i0 = (int)((long long)a.max_pages * c / C);
        const int i1 = (int)((long long)a.max_pages * (c + 1) / C);
#pragma unroll 4
        for (int i = i0 + tid; i < i1; i += kForkThreads) {
            int p = -1;
            if (served && i < full) {
                p = from[i];
                if (is_page(p)) atomicAdd(&a.shares[p], 1);
                else p = -1;
            } else if (served && i == full && part > 0 && is_page(fresh)) {
                p = fresh;
            }
            to[i] = p;
        }
    }
    if (c == 0) {
        const int old = served && part > 0 ? from[full] : 0;
        if (served) {
#pragma unroll 4
            for (int i = tid; i < full; i += kForkThreads) bad |= !is_page(from[i]);
            if (part > 0) bad |= !is_page(old) || !is_page(fresh);
        }
        bad = __syncthreads_or(bad);
        if (tid == 0) {
            int st = 0;
            if (!fine) st = SVF_DEV_BAD_ROW;
            else if (L < 0) st = SVF_DEV_BAD_LENGTH;
            else if (!served) st = SVF_DEV_NO_PAGES;
            else if (bad) st = SVF_DEV_BAD_PAGE;
            const bool copy = served && part > 0 && is_page(old) && is_page(fresh);
            a.copy_src[f] = copy ? old : -1;
            a.copy_dst[f] = copy ? fresh : -1;
            a.copy_len[f] = copy ? part : 0;
            a.status[f] = st;
            if (L >= 0) a.seq_lens[d] = served ? L : 0;
        }
    }
    if (tid == 0) {  // s_free was read before a barrier; the last CTA writes the new count
        const int taken = served && part > 0 ? incl : 0;
        if (gridDim.x * gridDim.y == 1) {
            a.state[0] = F - taken;
        } else {
            if (c == 0 && taken > 0) atomicMax(&a.state[2], taken);
            __threadfence();
            if (atomicAdd(&a.state[1], 1) == (int)(gridDim.x * gridDim.y) - 1) {
                __threadfence();
                a.state[0] = F - atomicExch(&a.state[2], 0);
                atomicExch(&a.state[1], 0);
            }
        }
    }
}

// grid (copies, layers, 2 parts): the first `len` tokens of page src over those of page
// dst, K (z = 0) or V (z = 1): contiguous bytes of a page.
__global__ void __launch_bounds__(kCopyThreads) page_copy_kernel(
    uint8_t *__restrict__ k_cache, uint8_t *__restrict__ v_cache, long long layer_bytes,
    int num_pages, int ps, int row_chunks, const int32_t *__restrict__ src,
    const int32_t *__restrict__ dst, const int32_t *__restrict__ lens,
    int32_t *__restrict__ status) {
    const int i = blockIdx.x, layer = blockIdx.y;
    pdl_wait();
    pdl_launch_dependents();
    const int s = src[i], d = dst[i], n = lens ? lens[i] : ps;
    int st = 0;
    const bool none = s == -1 && d == -1;
    if (!none) {
        if (s < 0 || s >= num_pages || d < 0 || d >= num_pages) st |= SVF_DEV_BAD_PAGE;
        if (n < 0 || n > ps) st |= SVF_DEV_BAD_LENGTH;
    }
    if (layer == 0 && blockIdx.z == 0 && threadIdx.x == 0) status[i] = st;
    if (none || st || s == d) return;
    uint8_t *base = (blockIdx.z ? v_cache : k_cache) + (size_t)layer * layer_bytes;
    const size_t page = (size_t)ps * row_chunks * 16;
    const uint4 *from = reinterpret_cast<const uint4 *>(base + s * page);
    uint4 *to = reinterpret_cast<uint4 *>(base + d * page);
    const long long all = (long long)n * row_chunks;
    for (long long j0 = threadIdx.x; j0 < all; j0 += 8 * kCopyThreads) {
        uint4 x[8];
#pragma unroll
        for (int u = 0; u < 8; ++u)
            if (j0 + u * kCopyThreads < all) x[u] = from[j0 + u * kCopyThreads];
#pragma unroll
        for (int u = 0; u < 8; ++u)
            if (j0 + u * kCopyThreads < all) to[j0 + u * kCopyThreads] = x[u];
    }
}

__device__ __forceinline__ void or_cluster(uint32_t at, unsigned bits) {
    asm volatile("red.shared::cluster.or.b32 [%0], %1;" ::"r"(at), "r"(bits) : "memory");
}

struct SharedReleaseArgs {
    int32_t *table;
    const int32_t *old_lens, *keep_lens;
    int32_t *free_pages, *state, *shares;
    int32_t *n_released, *status;
    int B, max_pages, ps, num_pages;
};

// One cluster. The pages that the sequences leave have ranks 0 .. total - 1, sequence by
// sequence in table order; a warp of the cluster takes an equal run of them. Passes over
// the ranks, the cluster meeting in between: look at the ids (a sequence with a bad one
// leaves nothing), lower the counts, claim the pages that nobody holds, count them (per
// warp, so that every page has its place), put them back. Up to kKeep ranks a thread stay
// in registers, so that the ids are read once and a pass has all of its reads in
// flight. Bound: the passes, each a round trip to the L2 and a meeting. 56 forks of 2049 pages, with
// fork and copy: 31.8 us with 16 CTAs, 42.3 with 8 (63.5 with every pass reading the table again);
// 34 where a thread goes through all 16 ranks though it has 7. Small tables take 8 CTAs and a rank
// a thread, whose code is shorter.
template <int kKeep, int kCtas>
__global__ void __launch_bounds__(kShareThreads) page_release_shared_kernel(SharedReleaseArgs a) {
    extern __shared__ int s_off[];   // [B + 1] the running sum of the pages
    int *s_first = s_off + a.B + 1;  // [B]
    unsigned *s_bad = reinterpret_cast<unsigned *>(s_first + a.B);  // a bit per sequence
    __shared__ int s_warp[kShareThreads / 32];
    __shared__ int s_total;  // pages that this CTA puts back
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = blockIdx.x;
    constexpr unsigned FULL = 0xffffffffu;
    if (!cluster_shape_is((uint32_t)kCtas, 1u, 1u)) {
        pdl_wait();
        for (int b = rank * kShareThreads + tid; b < a.B; b += kCtas * kShareThreads) {
            a.n_released[b] = 0;
            a.status[b] = SVF_DEV_BAD_CLUSTER;
        }
        return;
    }
    for (int i = tid; i < (a.B + 31) / 32; i += kShareThreads) s_bad[i] = 0;
    cluster_arrive();  // the others may set bits of s_bad
    pdl_wait();
    pdl_launch_dependents();
    const int F = min(max(*(volatile int32_t *)a.state, 0), a.num_pages);
    auto gift = [&](int b, int &first, int &n) {
        const int old = a.old_lens[b], keep = a.keep_lens[b];
        const bool ok = keep >= 0 && old >= keep &&
                        (long long)old <= (long long)a.max_pages * a.ps;
        first = ok ? pages_of(keep, a.ps) : 0;
        n = ok ? pages_of(old, a.ps) - first : 0;
        return ok;
    };
    int total = 0;
    for (int i0 = 0; i0 < a.B; i0 += kShareThreads) {
        const int i = i0 + tid;
        int v = 0, first = 0;
        if (i < a.B) {
            gift(i, first, v);
            s_first[i] = first;
            v = min(v, kMostGifts);
        }
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(FULL, v, o);
            if (lane >= o) v = sat_add(v, u, kMostGifts);
        }
        if (lane == 31) s_warp[warp] = v;
        __syncthreads();
        int w = s_warp[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(FULL, w, o);
            if (lane >= o) w = sat_add(w, u, kMostGifts);
        }
        const int below = __shfl_sync(FULL, w, warp - 1 < 0 ? 0 : warp - 1);
        if (i < a.B)
            s_off[i + 1] = sat_add(sat_add(total, warp > 0 ? below : 0, kMostGifts), v, kMostGifts);
        total = sat_add(total, __shfl_sync(FULL, w, 31), kMostGifts);
        __syncthreads();
    }
    if (tid == 0) s_off[0] = 0;
    __syncthreads();
    cluster_wait();
    const bool many = total >= kMostGifts;  // more than can be counted: nothing is taken
    if (many) total = 0;
    constexpr int kWarps = kCtas * kShareThreads / 32;
    const int per = ((total + kWarps - 1) / kWarps + 31) & ~31;
    const int k0 = (int)min((long long)(rank * (kShareThreads / 32) + warp) * per, (long long)total);
    const int k1 = min(k0 + per, total);
    auto owner = [&](int k) {  // the sequence of rank k < total
        int lo = 0, hi = a.B;  // s_off[lo] <= k < s_off[hi]
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (s_off[mid] <= k) lo = mid;
            else hi = mid;
        }
        return lo;
    };
    auto entry = [&](int b, int k) {
        return a.table + (size_t)b * a.max_pages + s_first[b] + (k - s_off[b]);
    };
    auto is_bad = [&](int b) { return (s_bad[b >> 5] >> (b & 31) & 1u) != 0; };
    auto meet = [&] {
        __threadfence();
        cluster_arrive();
        cluster_wait();
    };
    // f(k, b, p) for this thread's ranks: page p of sequence b
    const bool kept = per <= 32 * kKeep;
    int seq[kKeep], id[kKeep];
    if (kept) {
#pragma unroll
        for (int u = 0; u < kKeep && 32 * u < per; ++u) {
            const int k = k0 + lane + 32 * u;
            seq[u] = k < k1 ? owner(k) : -1;
            if (k < k1) id[u] = *entry(seq[u], k);
        }
    }
    auto each = [&](auto f) {
        if (kept) {
#pragma unroll
            for (int u = 0; u < kKeep && 32 * u < per; ++u)
                if (seq[u] >= 0) f(k0 + lane + 32 * u, seq[u], id[u]);
        } else {
            for (int k = k0 + lane; k < k1; k += 32) {
                const int b = owner(k);
                f(k, b, *entry(b, k));
            }
        }
    };
    each([&](int, int b, int p) {
        if ((p < 0 || p >= a.num_pages) && !is_bad(b))
            for (int c = 0; c < kCtas; ++c)
                or_cluster(cluster_map(&s_bad[b >> 5], (uint32_t)c), 1u << (b & 31));
    });
    meet();
    for (int b = rank * kShareThreads + tid; b < a.B; b += kCtas * kShareThreads) {
        int first, n;
        const bool ok = gift(b, first, n);
        a.n_released[b] = 0;
        a.status[b] = !ok ? SVF_DEV_BAD_LENGTH : (n > 0 && (many || is_bad(b))) ? SVF_DEV_BAD_PAGE : 0;
    }
    if (kept) {  // the ranks of sequences that leave nothing are out
#pragma unroll
        for (int u = 0; u < kKeep && 32 * u < per; ++u)
            if (seq[u] >= 0 && is_bad(seq[u])) seq[u] = -1;
    }
    each([&](int k, int b, int p) {
        if (is_bad(b)) return;
        atomicSub(&a.shares[p], 1);
        if (kept) *entry(b, k) = -1;  // (else it is read again)
    });
    meet();
    int now[kKeep];
    if (kept) {
#pragma unroll
        for (int u = 0; u < kKeep && 32 * u < per; ++u) now[u] = seq[u] >= 0 ? __ldcg(&a.shares[id[u]]) : 0;
#pragma unroll
        for (int u = 0; u < kKeep && 32 * u < per; ++u)
            if (now[u] < 0) atomicMin(&a.shares[id[u]], kClaim - seq[u]);
    } else {
        each([&](int, int b, int p) {
            if (!is_bad(b) && __ldcg(&a.shares[p]) < 0) atomicMin(&a.shares[p], kClaim - b);
        });
    }
    meet();
    // back: the page has its last holder in this sequence
    auto back = [&](int k, int &b, int &p) {
        if (k >= k1) return false;
        b = owner(k);
        if (is_bad(b)) return false;
        p = *entry(b, k);
        return __ldcg(&a.shares[p]) == kClaim - b;
    };
    int mine = 0;
    unsigned mask = 0;  // bit u: the page of kept rank u goes back
    if (kept) {
#pragma unroll
        for (int u = 0; u < kKeep && 32 * u < per; ++u) now[u] = seq[u] >= 0 ? __ldcg(&a.shares[id[u]]) : 0;
#pragma unroll
        for (int u = 0; u < kKeep && 32 * u < per; ++u) {
            const bool yes = seq[u] >= 0 && now[u] == kClaim - seq[u];
            mask |= yes ? 1u << u : 0u;
            mine += __popc(__ballot_sync(FULL, yes));
        }
    } else {
        for (int k = k0 + lane; k - lane < k1; k += 32) {
            int b = -1, p = -1;
            mine += __popc(__ballot_sync(FULL, back(k, b, p)));
        }
    }
    if (lane == 0) s_warp[warp] = mine;
    __syncthreads();
    int incl = s_warp[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(FULL, incl, o);
        if (lane >= o) incl += u;
    }
    int at = __shfl_sync(FULL, incl, warp) - mine;  // before this warp, in this CTA
    if (tid == 31) s_total = incl;
    meet();  // (the counts above were read by everybody before a page goes back, too)
    int all = 0;
    for (int c = 0; c < kCtas; ++c) {
        const int t = ld_dsmem_s32(cluster_map(&s_total, (uint32_t)c));
        if (c < rank) at += t;
        all += t;
    }
    auto put = [&](bool yes, int b, int p) {
        const unsigned who = __ballot_sync(FULL, yes);
        if (yes) {
            // a stack that is full already holds pages that it should not: no more go on it
            const long long to = (long long)F + all - 1 - (at + __popc(who & ((1u << lane) - 1)));
            if (to < a.num_pages) a.free_pages[to] = p;
            else atomicOr(&a.status[b], SVF_DEV_BAD_PAGE);
            a.shares[p] = 0;
        }
        at += __popc(who);
        if (who) {
            const unsigned same = __match_any_sync(FULL, yes ? b : -1);
            if (yes && lane == __ffs(same) - 1) atomicAdd(&a.n_released[b], __popc(same));
        }
    };
    if (kept) {
#pragma unroll
        for (int u = 0; u < kKeep && 32 * u < per; ++u) put(mask >> u & 1u, seq[u], id[u]);
    } else {
        for (int k = k0 + lane; k - lane < k1; k += 32) {
            int b = -1, p = -1;
            const bool yes = back(k, b, p);
            put(yes, b, p);
        }
    }
    if (!kept)
        each([&](int k, int b, int) {
            if (!is_bad(b)) *entry(b, k) = -1;
        });
    // nobody leaves while another may read its count; every CTA read the old one at the start
    cluster_arrive();
    cluster_wait();
    if (rank == 0 && tid == 0)
        a.state[0] = (int)min((long long)F + all, (long long)a.num_pages);
}

template <int kKeep, int kCtas>
cudaError_t launch_release(const SharedReleaseArgs &a, size_t bytes, cudaStream_t stream) {
    auto kernel = page_release_shared_kernel<kKeep, kCtas>;
    constexpr int kMost = (2 * kMaxPageSequences + 1 + (kMaxPageSequences + 31) / 32) * (int)sizeof(int);
    cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
    if (e == cudaSuccess && kCtas > 8)
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    return launch_pdl(kernel, dim3(kCtas), dim3(kShareThreads), bytes, stream, (unsigned)kCtas, a);
}

}  // namespace

cudaError_t launch_page_fork(const PageForkArgs &p, cudaStream_t stream) {
    ForkArgs a;
    a.table = p.page_table;
    a.free_pages = p.free_pages;
    a.state = p.pool_state;
    a.shares = p.shares;
    a.seq_lens = p.seq_lens;
    a.src = p.src;
    a.dst = p.dst;
    a.copy_src = p.copy_src;
    a.copy_dst = p.copy_dst;
    a.copy_len = p.copy_len;
    a.status = p.status;
    a.B = p.B;
    a.F = p.F;
    a.max_pages = p.max_pages;
    a.ps = p.page_size;
    a.num_pages = p.num_pages;
    // four entries a thread, at most eight CTAs per SM
    const int most = 8 * num_sms() / p.F, want = p.max_pages / (4 * kForkThreads);
    const int chunks = want < most ? want : most;
    return launch_pdl(page_fork_kernel, dim3((unsigned)p.F, (unsigned)(chunks < 1 ? 1 : chunks)),
                      dim3(kForkThreads), (size_t)p.B * sizeof(unsigned), stream, 0u, a);
}

cudaError_t launch_page_copy(const PageCopyArgs &p, cudaStream_t stream) {
    const int row_chunks = (int)((size_t)p.Hkv * p.D * p.elem_size / 16);
    return launch_pdl(page_copy_kernel, dim3((unsigned)p.n, (unsigned)p.num_layers, 2),
                      dim3(kCopyThreads), 0, stream, 0u, static_cast<uint8_t *>(p.k_cache),
                      static_cast<uint8_t *>(p.v_cache), p.layer_stride * (long long)p.elem_size,
                      p.num_pages, p.page_size, row_chunks, p.src, p.dst, p.lens, p.status);
}

cudaError_t launch_page_release_shared(const PageReleaseArgs &p, int32_t *shares,
                                       cudaStream_t stream) {
    SharedReleaseArgs a;
    a.table = p.page_table;
    a.old_lens = p.old_lens;
    a.keep_lens = p.keep_lens;
    a.free_pages = p.free_pages;
    a.state = p.pool_state;
    a.shares = shares;
    a.n_released = p.n_released;
    a.status = p.status;
    a.B = p.B;
    a.max_pages = p.max_pages;
    a.ps = p.page_size;
    a.num_pages = p.num_pages;
    const size_t bytes = (size_t)(2 * p.B + 1 + (p.B + 31) / 32) * sizeof(int);
    // A table whose every page fits one rank a thread of 8 CTAs has the kernel for that; from 16
    // thousand entries on 16 CTAs, where such a cluster fits the device. Forks, copies and release of
    // 56 rows of 64, with 16 and with 8 CTAs (us): 145 entries a row 18.7 and 17.5, 252 20.0 and
    // 20.1, 502 22.5 and 23.0, 1002 26.7 and 29.6, 2050 30.8 and 39.5.
    if ((long long)p.B * p.max_pages > 16 * kShareThreads &&
        resident_clusters(page_release_shared_kernel<16, 16>, kShareThreads, bytes, 16) > 0)
        return launch_release<16, 16>(a, bytes, stream);
    return (long long)p.B * p.max_pages > 8 * kShareThreads ? launch_release<16, 8>(a, bytes, stream)
                                                            : launch_release<1, 8>(a, bytes, stream);
}

}  // namespace svf
