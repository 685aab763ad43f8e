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
// its own (a few loads per thread, all from L2) instead of waiting for a scan
// by somebody else, and only the counter of the pool needs an order: the CTAs
// take tickets after they have read it, and the last one writes the new count
// (no CTA waits).
#include "common.cuh"
#include "internal.h"

namespace svf {

namespace {

constexpr int kPageThreads = 256;

// state[0] free pages; state[1] tickets and state[2] the largest served I_b of
// the call in flight (both zero between calls).
__device__ __forceinline__ int sat_add(int a, int b, int cap) {
    // 0 <= a, b <= cap < 2^30: associative, so the order of a sum does not matter
    return min(a + b, cap);
}

__device__ __forceinline__ int block_sat_sum(int v, int cap, int *s_part) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = sat_add(v, __shfl_xor_sync(0xffffffffu, v, o), cap);
    __syncthreads();  // s_part may still be read from the previous sum
    if ((threadIdx.x & 31) == 0) s_part[threadIdx.x >> 5] = v;
    __syncthreads();
    int t = 0;
    for (int w = 0; w < kPageThreads / 32; ++w) t = sat_add(t, s_part[w], cap);
    return t;
}

__device__ __forceinline__ int pages_of(int tokens, int ps) {
    return tokens / ps + (tokens % ps != 0);
}

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
    __shared__ int s_part[kPageThreads / 32];
    __shared__ int s_free;
    const int b = blockIdx.x, c = blockIdx.y, C = gridDim.y, tid = threadIdx.x;
    pdl_wait();
    pdl_launch_dependents();
    if (tid == 0) s_free = min(max(*(volatile int32_t *)a.state, 0), a.num_pages);
    const int rcap = a.T + 1, pcap = a.num_pages + 1;
    int rows_before = 0, rows_all = 0, need_before = 0;
    for (int i = tid; i < a.B; i += kPageThreads) {
        const Want w = want_of(a, i);
        rows_all = sat_add(rows_all, w.rows, rcap);
        if (i < b) {
            rows_before = sat_add(rows_before, w.rows, rcap);
            need_before = sat_add(need_before, w.need, pcap);
        }
    }
    rows_before = block_sat_sum(rows_before, rcap, s_part);
    rows_all = block_sat_sum(rows_all, rcap, s_part);
    need_before = block_sat_sum(need_before, pcap, s_part);
    const int F = s_free;
    const Want w = want_of(a, b);
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
        for (int j = j0 + tid; j < j1; j += kPageThreads) row[held + j] = page_at(held + j);
    }
    const int r0 = min(rows_before, a.T), r1 = min(rows_before + w.rows, a.T);
    const int n = r1 - r0;
    const int i0 = (int)((long long)n * c / C), i1 = (int)((long long)n * (c + 1) / C);
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
    if (tid == 0) {  // s_free was read before the sums' barriers
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

struct ReleaseArgs {
    int32_t *table;
    const int32_t *old_lens, *keep_lens;
    int32_t *free_pages, *state;
    int32_t *n_released, *status;
    int B, max_pages, ps, num_pages;
};

// How many pages sequence b gives back (every thread of the CTA gets the
// answer): 0 when its lengths or one of its page ids are bad.
__device__ __forceinline__ int release_count(const ReleaseArgs &a, int b, int *lo, int *st) {
    const int old = a.old_lens[b], keep = a.keep_lens[b];
    *st = 0;
    *lo = 0;
    if (keep < 0 || old < keep || (long long)old > (long long)a.max_pages * a.ps) {
        *st = SVF_DEV_BAD_LENGTH;
        return 0;
    }
    const int first = pages_of(keep, a.ps), end = pages_of(old, a.ps);
    *lo = first;
    const int32_t *row = a.table + (size_t)b * a.max_pages;
    bool bad = false;
    for (int i = first + (int)threadIdx.x; i < end; i += kPageThreads)
        bad |= row[i] < 0 || row[i] >= a.num_pages;
    if (__syncthreads_or(bad)) {
        *st = SVF_DEV_BAD_PAGE;
        return 0;
    }
    return end - first;
}

__global__ void __launch_bounds__(kPageThreads) page_release_check_kernel(ReleaseArgs a) {
    pdl_wait();
    pdl_launch_dependents();
    int lo, st;
    const int n = release_count(a, blockIdx.x, &lo, &st);
    if (threadIdx.x == 0) {
        a.n_released[blockIdx.x] = n;
        a.status[blockIdx.x] = st;
    }
}

// grid (B, chunks). Rank k of all the pages given back (sequence by sequence,
// in table order) goes to free[F + total - 1 - k]. A single sequence checks
// its own pages here; otherwise the kernel before this one has.
template <bool ALONE>
__global__ void __launch_bounds__(kPageThreads) page_release_kernel(ReleaseArgs a) {
    __shared__ int s_part[kPageThreads / 32];
    __shared__ int s_free;
    const int b = blockIdx.x, c = blockIdx.y, C = gridDim.y, tid = threadIdx.x;
    pdl_wait();
    pdl_launch_dependents();
    if (tid == 0) s_free = min(max(*(volatile int32_t *)a.state, 0), a.num_pages);
    int before = 0, total = 0, n, lo, st = 0;
    const int cap = a.num_pages + 1;
    if (ALONE) {
        n = release_count(a, b, &lo, &st);
        total = min(n, cap);
        __syncthreads();
    } else {
        for (int i = tid; i < a.B; i += kPageThreads) {
            const int m = min(a.n_released[i], cap);
            total = sat_add(total, m, cap);
            if (i < b) before = sat_add(before, m, cap);
        }
        before = block_sat_sum(before, cap, s_part);
        total = block_sat_sum(total, cap, s_part);
        n = a.n_released[b];
        lo = n > 0 ? pages_of(a.keep_lens[b], a.ps) : 0;
    }
    const int F = s_free;
    // more pages than the cache has: some were given back before, take none
    const bool over = F + total > a.num_pages;
    if (!over && n > 0) {
        int32_t *row = a.table + (size_t)b * a.max_pages + lo;
        const int j0 = (int)((long long)n * c / C), j1 = (int)((long long)n * (c + 1) / C);
        for (int j = j0 + tid; j < j1; j += kPageThreads) {
            a.free_pages[F + total - 1 - (before + j)] = row[j];
            row[j] = -1;
        }
    }
    if (tid == 0) {
        if (ALONE) {
            a.n_released[b] = over ? 0 : n;
            a.status[b] = over ? SVF_DEV_BAD_PAGE : st;
        } else if (c == 0 && over && n > 0) {
            a.status[b] = SVF_DEV_BAD_PAGE;
        }
    }
    if (ALONE) {
        if (tid == 0 && !over) a.state[0] = F + total;
        return;
    }
    __shared__ int s_last;
    if (tid == 0) {
        __threadfence();
        s_last = atomicAdd(&a.state[1], 1) == (int)(gridDim.x * gridDim.y) - 1;
    }
    __syncthreads();
    if (!s_last) return;
    __threadfence();
    // every CTA has read the count and the n_released that it needs
    if (over)
        for (int i = tid; i < a.B; i += kPageThreads) a.n_released[i] = 0;
    if (tid == 0) {
        if (!over) a.state[0] = F + total;
        atomicExch(&a.state[1], 0);
    }
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

// Parts per sequence: enough CTAs for about four rows (or pages) a thread,
// at most two CTAs per SM in all.
int chunks_for(long long items, int B) {
    const long long want = items / ((long long)B * kPageThreads * 4);
    const int most = 2 * num_sms() / B;
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
    if (p.B == 1)  // one CTA checks and gives back
        return launch_pdl(page_release_kernel<true>, dim3(1u, 1u), dim3(kPageThreads), 0, stream,
                          0u, a);
    const cudaError_t e = launch_pdl(page_release_check_kernel, dim3((unsigned)p.B),
                                     dim3(kPageThreads), 0, stream, 0u, a);
    if (e != cudaSuccess) return e;
    return launch_pdl(page_release_kernel<false>,
                      dim3((unsigned)p.B, (unsigned)chunks_for((long long)p.B * 256, p.B)),
                      dim3(kPageThreads), 0, stream, 0u, a);
}

}  // namespace svf
