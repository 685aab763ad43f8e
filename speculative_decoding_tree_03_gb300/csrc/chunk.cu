// chunk.cu -- the host's side of the chunk attention: which kernel, how many CTAs, and where
// things are in the workspace.
#include <math.h>

#include <atomic>

#include "chunk.cuh"

namespace svf {

namespace {

std::atomic<long long> g_wait_ns{0};

struct Plan {
    int ctas, S, rows_per_block, TB, min_tiles, lead, slot_rows;
    size_t done, gave_up, part_bad, part_lse, part, total;
};

// Heads of a group: the divisor of Hkv that leaves the fewest SMs without work, the largest of
// those (its CTAs read the same token rows side by side).
int group_heads(int Hkv, int ctas) {
    int best = 1, used = 0;
    for (int s = 1; s <= Hkv && s <= ctas; ++s)
        if (Hkv % s == 0 && ctas / s * s >= used) {
            used = ctas / s * s;
            best = s;
        }
    return best;
}

Plan plan_of(int rows, int Hq, int Hkv, int D, int dtype) {
    Plan c;
    const int G = Hq / Hkv;
    int most;
    // min_tiles: the least tiles that a CTA's share is cut to. bf16: one (a token over 2049: 21.5 us with 1
    // to 3). fp32: two (333 rows of 5 sequences 46.3 us; one, with twice the pieces to join, 59.8;
    // three 49.1, four 55.8).
    // lead: tiles that a unit's end costs (chunk.cuh); bf16 prompt of 8192 tokens: 0 535 us, 2 483,
    // 4 469, 6 459, 8 463.
    if (dtype == SVF_BF16) {
        most = num_sms();
        c.TB = 2 * (128 / G);
        c.rows_per_block = 256;
        c.min_tiles = 1;
        c.lead = 6;
    } else {
        most = num_sms() * (D == 64 ? 3 : 1);  // CTAs whose shared memory fits an SM
        c.TB = 64 / G;
        c.rows_per_block = 64;
        c.min_tiles = 2;
        c.lead = 1;
    }
    if (most > kChunkMaxCtas) most = kChunkMaxCtas;
    c.S = group_heads(Hkv, most);
    c.ctas = most / c.S * c.S;
    auto up = [](size_t x, size_t to) { return (x + to - 1) / to * to; };
    const size_t want = up((size_t)(rows > 0 ? rows : 1) * G, 32);
    c.slot_rows = want < (size_t)c.rows_per_block ? (int)want : c.rows_per_block;
    const size_t slots = 2 * (size_t)c.ctas;
    c.done = kChunkMaxCtas * sizeof(int);  // the counters, and what else begins at zero, stay in place
    c.gave_up = kChunkHeadBytes;
    c.part_bad = up(c.gave_up + slots * sizeof(int), 256);
    c.part_lse = up(c.part_bad + 2 * slots * sizeof(int), 256);
    c.part = up(c.part_lse + slots * c.slot_rows * sizeof(float), 256);
    c.total = c.part + slots * c.slot_rows * (size_t)D * sizeof(float);
    return c;
}

}  // namespace

bool chunk_supported(int rows, int B, int Hq, int Hkv, int D, int dtype, int page_size) {
    if (rows > (1 << 24) || B > (1 << 20) || Hq < 1 || Hkv < 1 || Hkv > 1024 || Hq % Hkv != 0 ||
        Hq / Hkv > 64)
        return false;
    if (dtype == SVF_F32) return D == 64 || D == 128;
    return dtype == SVF_BF16 && D == 128 &&
           (page_size == 16 || page_size == 32 || page_size == 64 || page_size % 128 == 0);
}

size_t chunk_workspace_bytes(int rows, int Hq, int Hkv, int D, int dtype) {
    return plan_of(rows, Hq, Hkv, D, dtype).total;
}

void chunk_set_wait_ns(long long ns) { g_wait_ns.store(ns); }

int launch_chunk(const ChunkArgs &a, cudaStream_t stream) {
    const Plan c = plan_of(a.rows, a.Hq, a.Hkv, a.D, a.dtype);
    if (!a.workspace || a.workspace_bytes < c.total) return SVF_ERR_WORKSPACE;
    uint8_t *ws = static_cast<uint8_t *>(a.workspace);
    ChunkParams p;
    p.q = a.q;
    p.k_cache = a.k_cache;
    p.v_cache = a.v_cache;
    p.out = a.out;
    p.lse = a.lse;
    p.page_table = a.page_table;
    p.seq_lens = a.seq_lens;
    p.row_offsets = a.row_offsets;
    p.status = a.status;
    p.B = a.B;
    p.rows = a.rows;
    p.Hq = a.Hq;
    p.Hkv = a.Hkv;
    p.G = a.Hq / a.Hkv;
    p.ps = a.page_size;
    p.num_pages = a.num_pages;
    p.max_pages = a.max_pages;
    p.TB = c.TB;
    p.S = c.S;
    p.NHB = a.Hkv / c.S;
    p.groups = c.ctas / c.S;
    p.min_tiles = c.min_tiles;
    p.lead = c.lead;
    const float scale = a.sm_scale > 0.0f ? a.sm_scale : 1.0f / sqrtf((float)a.D);
    p.scale_log2 = scale * 1.4426950408889634f;
    const long long ns = g_wait_ns.load();
    p.wait_ns = ns > 0 ? (unsigned long long)ns : kWaitDeadlineNs;
    p.counters = reinterpret_cast<int *>(ws);
    p.done = reinterpret_cast<int *>(ws + c.done);
    p.gave_up = reinterpret_cast<int *>(ws + c.gave_up);
    p.part_bad = reinterpret_cast<int *>(ws + c.part_bad);
    p.part_lse = reinterpret_cast<float *>(ws + c.part_lse);
    p.part = reinterpret_cast<float4 *>(ws + c.part);
    p.slot_rows = c.slot_rows;
    // (a call without rows has status words to write, which either kernel does)
    const cudaError_t e = a.dtype == SVF_BF16 && a.rows > 0
                              ? launch_chunk_tc(p, c.ctas, stream)
                              : launch_chunk_simt(p, a.D, c.ctas, stream);
    return e == cudaSuccess ? SVF_OK : SVF_ERR_LAUNCH;
}

}  // namespace svf
