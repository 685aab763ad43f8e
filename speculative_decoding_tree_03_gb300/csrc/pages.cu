// pages.cu -- page tables and slot maps of the paged KV cache, kept on the device.
//
// A pool is a stack of free page ids, free[0 .. F), and a sequence of L tokens
// holds ceil(L / ps) pages, whose ids stand at the front of its page-table row.
// svf_page_reserve makes room for n_b new tokens of every sequence:
//     need_b = ceil((L_b + n_b) / ps) - ceil(L_b / ps),   I_b = sum_{b' <= b} need_b',
//     the k-th page handed out is free[F - 1 - k], and sequence b gets the
//     ranks I_b - need_b .. I_b - 1;
// it is served when need_b = 0 or I_b <= F. I is monotone, so the ranks handed
// out are 0 .. max{I_b : I_b <= F} - 1 whatever the order the CTAs run in, and
// the result does not depend on that order. svf_page_release is its inverse:
// the pages go back so that a release of exactly what a reserve took restores
// the stack entry by entry.
//
// Bound: latency. The 70B-shaped batch (64 trees of 31 nodes) moves 28 KB; the
// time is the launch, three dependent reads (lengths, top of the stack, page
// id) and the stores. So every CTA sums the lengths of all sequences before
// its own instead of waiting for a scan by somebody else, and only the counter
// of the pool needs an order: the CTAs take tickets after they have read it, and
// the last one writes the new count (no CTA waits). That is a few loads per
// thread, all from L2, for batches of some hundred sequences; its cost grows
// with the square of the batch (trees of 31 nodes, reserve alone: 64 sequences
// 4 us, 1024 9 us, 4096 50 us, 8192, the most, 167 us).
#include "common.cuh"
#include "internal.h"
#include "page_math.cuh"

namespace svf {

namespace {

constexpr int kPageThreads = 256;
constexpr int kReleaseThreads = 1024;
constexpr int kKept = 4;  // ids that a thread of a release keeps in registers

// state[0] free pages; state[1] tickets and state[2] the largest served I_b of
// the call in flight (both zero between calls).
struct ReserveArgs {
    int32_t *table;
    const int32_t *seq_lens, *new_lens, *depth;
    const int32_t *free_pages;
    int32_t *state;
    int32_t *slots, *positions, *row_offsets, *status;
    int B, max_pages, ps, num_pages, T;
};

struct Want {
    int L, n, rows, need;
    bool ok;
};

__device__ __forceinline__ Want want_of(const ReserveArgs &a, int b) {
    Want w;
    w.L = a.seq_lens[b];
    w.n = a.new_lens[b];
    w.rows = min(max(w.n, 0), a.T + 1);
    w.ok = w.L >= 0 && w.n >= 0 && (long long)w.L + w.n <= (long long)a.max_pages * a.ps;
    w.need = w.ok ? min(pages_of(w.L + w.n, a.ps) - pages_of(w.L, a.ps), a.num_pages + 1) : 0;
    return w;
}

// grid (B, chunks): the rows and pages of sequence blockIdx.x in gridDim.y equal parts
__global__ void __launch_bounds__(kPageThreads) page_reserve_kernel(ReserveArgs a) {
    __shared__ int s_part[3][kPageThreads / 32];
    __shared__ int s_free;
    const int b = blockIdx.x, c = blockIdx.y, C = gridDim.y, tid = threadIdx.x;
    pdl_wait();
    pdl_launch_dependents();
    const Want w = want_of(a, b);
    if (tid == 0) s_free = min(max(*(volatile int32_t *)a.state, 0), a.num_pages);
    const int rcap = a.T + 1, pcap = a.num_pages + 1;
    int sum[3] = {0, 0, 0};  // rows before b, all rows, pages before b
    for (int i = tid; i < a.B; i += kPageThreads) {
        const Want v = want_of(a, i);
        sum[1] = sat_add(sum[1], v.rows, rcap);
        if (i < b) {
            sum[0] = sat_add(sum[0], v.rows, rcap);
            sum[2] = sat_add(sum[2], v.need, pcap);
        }
    }
    const int cap[3] = {rcap, rcap, pcap};
#pragma unroll
    for (int k = 0; k < 3; ++k) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            sum[k] = sat_add(sum[k], __shfl_xor_sync(0xffffffffu, sum[k], o), cap[k]);
        if ((tid & 31) == 0) s_part[k][tid >> 5] = sum[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        sum[k] = 0;
#pragma unroll
        for (int i = 0; i < kPageThreads / 32; ++i) sum[k] = sat_add(sum[k], s_part[k][i], cap[k]);
    }
    const int rows_before = sum[0], rows_all = sum[1], need_before = sum[2];
    const int F = s_free;
    const bool over = rows_all > a.T;  // the rows of the call do not fit: nothing is taken
    const int incl = sat_add(need_before, w.need, pcap);
    const bool live = w.ok && !(over && w.n > 0);
    const bool served = live && (w.need == 0 || incl <= F);
    const int held = w.ok ? pages_of(w.L, a.ps) : 0;
    int32_t *row = a.table + (size_t)b * a.max_pages;
    // the id of page-table index i of this sequence, -1 if it has none or a bad one
    auto page_at = [&](int i) {
        const int p = i < held ? row[i]
                      : served ? a.free_pages[F - 1 - (need_before + i - held)]
                               : -1;
        return p >= 0 && p < a.num_pages ? p : -1;
    };
    if (live && w.need > 0) {
        const int j0 = (int)((long long)w.need * c / C), j1 = (int)((long long)w.need * (c + 1) / C);
#pragma unroll 2
        for (int j = j0 + tid; j < j1; j += kPageThreads) row[held + j] = page_at(held + j);
    }
    const int r0 = min(rows_before, a.T), r1 = min(rows_before + w.rows, a.T);
    const int n = r1 - r0;
    const int i0 = (int)((long long)n * c / C), i1 = (int)((long long)n * (c + 1) / C);
#pragma unroll 4
    for (int i = i0 + tid; i < i1; i += kPageThreads) {
        int slot = -1, pos = 0;
        if (live) {
            const unsigned t = (unsigned)w.L + (unsigned)i;
            if (served) {
                const int p = page_at((int)(t / (unsigned)a.ps));
                if (p >= 0) slot = p * a.ps + (int)(t % (unsigned)a.ps);
            }
            pos = a.depth ? w.L + a.depth[r0 + i] : (int)t;
        }
        a.slots[r0 + i] = slot;
        if (a.positions) a.positions[r0 + i] = pos;
    }
    // rows behind the last sequence
    for (int i = min(rows_all, a.T) + (b * C + c) * kPageThreads + tid; i < a.T;
         i += a.B * C * kPageThreads) {
        a.slots[i] = -1;
        if (a.positions) a.positions[i] = 0;
    }
    int st = 0;
    if (c == 0) {
        if (served && w.n > 0) {  // every page that its new tokens fall into
            bool bad = false;
#pragma unroll 4
            for (int i = w.L / a.ps + tid; i < held + w.need; i += kPageThreads)
                bad |= page_at(i) < 0;
            if (__syncthreads_or(bad)) st = SVF_DEV_BAD_PAGE;
        }
        if (tid == 0) {
            if (!live) st = SVF_DEV_BAD_LENGTH;
            else if (!served) st = SVF_DEV_NO_PAGES;
            a.status[b] = st;
            a.row_offsets[b] = r0;
            if (b == a.B - 1) a.row_offsets[a.B] = min(rows_all, a.T);
        }
    }
    if (tid == 0) {  // s_free was read before the barrier
        const int taken = served ? incl * (w.need > 0) : 0;
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

__device__ __forceinline__ void or_cluster(uint32_t at, unsigned bits) {
    asm volatile("red.shared::cluster.or.b32 [%0], %1;" ::"r"(at), "r"(bits) : "memory");
}

struct ReleaseArgs {
    int32_t *table;
    const int32_t *old_lens, *keep_lens;
    int32_t *free_pages, *state;
    int32_t *n_released, *status;
    int B, max_pages, ps, num_pages;
};

// What sequence b gives back: n pages from entry `first` of its row on.
struct Gift {
    int first, n;
    bool ok;
};

__device__ __forceinline__ Gift gift_of(const ReleaseArgs &a, int b) {
    const int old = a.old_lens[b], keep = a.keep_lens[b];
    Gift g;
    g.ok = keep >= 0 && old >= keep && (long long)old <= (long long)a.max_pages * a.ps;
    g.first = g.ok ? pages_of(keep, a.ps) : 0;
    g.n = g.ok ? pages_of(old, a.ps) - g.first : 0;
    return g;
}

// One cluster of `ctas` CTAs, or its first alone. Every CTA sums up by itself
// how many pages each sequence gives back, so that the pages of the call have
// ranks 0 .. total - 1, sequence by sequence in table order; thread t of all
// takes the ranks t, t + threads, .. (their sequence by a search in the sums),
// looks at the ids, and once nobody found a bad one puts rank k at
// free[F + total - 1 - k]. So the chain is two reads, lengths and ids (and the
// lengths once more where bad sequences are left out), whatever the lengths are
// like (200 ragged prompts of 16 thousand pages, reserve and release: 15.3 us;
// 20.7 with a warp to a sequence and long ones by whole CTAs one after the
// other).
__global__ void __launch_bounds__(kReleaseThreads) page_release_kernel(ReleaseArgs a, int ctas) {
    extern __shared__ int s_off[];  // [B + 1] the running sum of the pages
    int *s_first = s_off + a.B + 1;  // [B]
    unsigned *s_bad = reinterpret_cast<unsigned *>(s_first + a.B);  // a bit per sequence
    __shared__ int s_warp[kReleaseThreads / 32];
    __shared__ int s_any;  // some bit of s_bad is set
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (!cluster_shape_is((uint32_t)ctas, 1u, 1u)) {
        pdl_wait();
        for (int b = blockIdx.x * kReleaseThreads + tid; b < a.B; b += ctas * kReleaseThreads) {
            a.n_released[b] = 0;
            a.status[b] = SVF_DEV_BAD_CLUSTER;
        }
        return;
    }
    const int rank = blockIdx.x;
    for (int i = tid; i < (a.B + 31) / 32; i += kReleaseThreads) s_bad[i] = 0;
    if (tid == 0) s_any = 0;
    if (ctas > 1) cluster_arrive();  // the others may set bits of s_bad
    pdl_wait();
    pdl_launch_dependents();
    int F = rank == 0 ? *(volatile int32_t *)a.state : 0;
    auto is_bad = [&](int b) { return (s_bad[b >> 5] >> (b & 31) & 1u) != 0; };
    const int cap = a.num_pages + 1;
    // the running sum of the pages of all sequences but the bad ones
    auto scan = [&](bool checked) {
        int carry = 0;
        for (int i0 = 0; i0 < a.B; i0 += kReleaseThreads) {
            const int i = i0 + tid;
            int v = 0;
            if (i < a.B) {
                const Gift g = gift_of(a, i);
                s_first[i] = g.first;
                v = checked && is_bad(i) ? 0 : min(g.n, cap);
            }
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, v, o);
                if (lane >= o) v = sat_add(v, u, cap);
            }
            if (lane == 31) s_warp[warp] = v;
            __syncthreads();
            int w = s_warp[lane];  // 32 warps: every warp scans their sums
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, w, o);
                if (lane >= o) w = sat_add(w, u, cap);
            }
            const int below = __shfl_sync(0xffffffffu, w, warp - 1 < 0 ? 0 : warp - 1);
            if (i < a.B) s_off[i + 1] = sat_add(sat_add(carry, warp > 0 ? below : 0, cap), v, cap);
            carry = sat_add(carry, __shfl_sync(0xffffffffu, w, 31), cap);
            __syncthreads();
        }
        if (tid == 0) s_off[0] = 0;
        __syncthreads();
        return carry;
    };
    auto owner = [&](int k) {  // the sequence of rank k < s_off[B]
        int lo = 0, hi = a.B;  // s_off[lo] <= k < s_off[hi]
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (s_off[mid] <= k) lo = mid;
            else hi = mid;
        }
        return lo;
    };
    auto entry = [&](int b, int j) {  // the j-th page that b gives back
        return a.table + (size_t)b * a.max_pages + s_first[b] + j;
    };
    int total = scan(false);
    if (ctas > 1) cluster_wait();
    // Few pages are the first CTA's (64 trees of 31 nodes, reserve and release:
    // 8.6 us, 8.9 with all CTAs).
    const bool alone = ctas == 1 || total <= kKept * kReleaseThreads;
    if (alone && rank > 0) return;
    if (rank > 0) F = *(volatile int32_t *)a.state;
    F = min(max(F, 0), a.num_pages);
    const int threads = alone ? kReleaseThreads : ctas * kReleaseThreads;
    const int me = rank * kReleaseThreads + tid;
    auto mark = [&](int b) {  // in every CTA, once from each
        if (is_bad(b) || (atomicOr(&s_bad[b >> 5], 1u << (b & 31)) >> (b & 31) & 1u)) return;
        s_any = 1;
        for (int c = 0; !alone && c < ctas; ++c) {
            or_cluster(cluster_map(&s_bad[b >> 5], (uint32_t)c), 1u << (b & 31));
            or_cluster(cluster_map(&s_any, (uint32_t)c), 1u);
        }
    };
    auto is_page = [&](int p) { return p >= 0 && p < a.num_pages; };
    // a thread's first pages: the id, the sequence and the number in it
    int id[kKept], seq[kKept], num[kKept];
    const bool counted = total < cap, fits = counted && total <= kKept * threads;
    if (counted) {
#pragma unroll
        for (int u = 0; u < kKept; ++u) {
            const int k = me + u * threads;
            seq[u] = -1;
            if (k < total) {
                seq[u] = owner(k);
                num[u] = k - s_off[seq[u]];
                id[u] = *entry(seq[u], num[u]);
            }
        }
#pragma unroll
        for (int u = 0; u < kKept; ++u)
            if (seq[u] >= 0 && !is_page(id[u])) mark(seq[u]);
        for (int k = me + kKept * threads; k < total; k += threads) {
            const int b = owner(k);
            if (!is_page(*entry(b, k - s_off[b]))) mark(b);
        }
    } else {  // more than the cache has: without the bad sequences it may be less
        for (int b = me >> 5; b < a.B; b += threads >> 5) {
            const Gift g = gift_of(a, b);
            const int32_t *row = a.table + (size_t)b * a.max_pages + g.first;
            bool bad = false;
            for (int i = lane; i < g.n; i += 32) bad |= !is_page(row[i]);
            if (__any_sync(0xffffffffu, bad) && lane == 0) mark(b);
        }
    }
    if (alone) {
        __syncthreads();
    } else {
        cluster_arrive();
        cluster_wait();
    }
    const bool again = !counted || s_any != 0;
    if (again) total = scan(true);
    // more pages than the cache has: some were given back before; take none
    const bool none = F + total > a.num_pages;
    for (int b = me; b < a.B; b += threads) {
        const Gift g = gift_of(a, b);
        int st = g.ok ? 0 : SVF_DEV_BAD_LENGTH, n = g.n;
        if (n > 0 && (none || is_bad(b))) {
            st = SVF_DEV_BAD_PAGE;
            n = 0;
        }
        a.n_released[b] = n;
        a.status[b] = st;
    }
    if (none) return;
    int32_t *top = a.free_pages + (F + total - 1);
    const bool kept = !again || fits;  // else the ranks are others now
    if (kept) {
#pragma unroll
        for (int u = 0; u < kKept; ++u)
            if (seq[u] >= 0 && !is_bad(seq[u])) {
                top[-(s_off[seq[u]] + num[u])] = id[u];
                *entry(seq[u], num[u]) = -1;
            }
    }
    for (int k = me + (kept ? kKept * threads : 0); k < total; k += threads) {
        const int b = owner(k);
        int32_t *at = entry(b, k - s_off[b]);
        top[-k] = *at;
        *at = -1;
    }
    // every CTA read the count before the cluster met
    if (me == 0) a.state[0] = F + total;
}

__global__ void __launch_bounds__(kPageThreads)
    page_pool_init_kernel(int32_t *free_pages, int32_t *state, int num_pages) {
    pdl_wait();
    pdl_launch_dependents();
    for (int i = blockIdx.x * kPageThreads + threadIdx.x; i < num_pages;
         i += gridDim.x * kPageThreads)
        free_pages[i] = num_pages - 1 - i;  // page 0 is handed out first
    if (blockIdx.x == 0 && threadIdx.x < 4) state[threadIdx.x] = threadIdx.x == 0 ? num_pages : 0;
}

// Parts per sequence: one row a thread on average (ragged lengths make some
// sequences several times as long), at most eight CTAs per SM in all.
int chunks_for(long long items, int B) {
    const long long want = items / ((long long)B * kPageThreads);
    const int most = 8 * num_sms() / B;
    const long long c = want < most ? want : most;
    return c < 1 ? 1 : (int)c;
}

}  // namespace

cudaError_t launch_page_pool_init(int32_t *free_pages, int32_t *state, int num_pages,
                                  cudaStream_t stream) {
    const int blocks = (num_pages + kPageThreads - 1) / kPageThreads;
    const int most = 2 * num_sms();
    return launch_pdl(page_pool_init_kernel, dim3((unsigned)(blocks < most ? blocks : most)),
                      dim3(kPageThreads), 0, stream, 0u, free_pages, state, num_pages);
}

cudaError_t launch_page_reserve(const PageReserveArgs &p, cudaStream_t stream) {
    ReserveArgs a;
    a.table = p.page_table;
    a.seq_lens = p.seq_lens;
    a.new_lens = p.new_lens;
    a.depth = p.depth;
    a.free_pages = p.free_pages;
    a.state = p.pool_state;
    a.slots = p.slots;
    a.positions = p.positions;
    a.row_offsets = p.row_offsets;
    a.status = p.status;
    a.B = p.B;
    a.max_pages = p.max_pages;
    a.ps = p.page_size;
    a.num_pages = p.num_pages;
    a.T = p.rows;
    return launch_pdl(page_reserve_kernel, dim3((unsigned)p.B, (unsigned)chunks_for(p.rows, p.B)),
                      dim3(kPageThreads), 0, stream, 0u, a);
}

cudaError_t launch_page_release(const PageReleaseArgs &p, cudaStream_t stream) {
    ReleaseArgs a;
    a.table = p.page_table;
    a.old_lens = p.old_lens;
    a.keep_lens = p.keep_lens;
    a.free_pages = p.free_pages;
    a.state = p.pool_state;
    a.n_released = p.n_released;
    a.status = p.status;
    a.B = p.B;
    a.max_pages = p.max_pages;
    a.ps = p.page_size;
    a.num_pages = p.num_pages;
    const int ctas = p.B == 1 ? 1 : 8;
    const size_t smem = (size_t)(2 * p.B + 1 + (p.B + 31) / 32) * sizeof(int);
    // The kernel's static arrays count towards the default limit of 48 KB too
    // (sums of 6032 to 6048 sequences fit it, but not together with them), and
    // calls of several host threads agree on one limit.
    const cudaError_t e = cudaFuncSetAttribute(
        page_release_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
        (2 * kMaxPageSequences + 1 + kMaxPageSequences / 32) * (int)sizeof(int));
    if (e != cudaSuccess) return e;
    return launch_pdl(page_release_kernel, dim3((unsigned)ctas), dim3(kReleaseThreads), smem, stream,
                      ctas > 1 ? (unsigned)ctas : 0u, a, ctas);
}

}  // namespace svf
