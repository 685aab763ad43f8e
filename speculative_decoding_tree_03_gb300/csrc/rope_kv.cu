// rope_kv.cu -- rotary positions of a step's rows, and their K/V into the cache.
//
// Row t of the step (a tree node, or a prompt token) has position pos and slot
// s. With c_i = rope[pos][i], s_i = rope[pos][rot/2 + i] (the cosine and sine
// of the position's i-th angle), every pair of a q or k head turns by its
// angle:
//     (x_a, x_b) -> (x_a c_i - x_b s_i,  x_b c_i + x_a s_i),
// a, b = i, i + rot/2 (or 2i, 2i + 1 when interleaved); elements from rot on
// stay. q rows go to q_out, k rows to the cache's slot s, and v rows are
// copied there. The products and their sum are taken in fp32 and rounded once
// to the element type (bf16: half a unit in the last place, what the cache
// holds anyway).
//
// Bound: HBM: each q, k and v element is read once and written once, plus one
// table row of 4 rot bytes per token. So no staging: a thread takes 16 bytes
// of either half of a pair block (32 contiguous bytes when interleaved), reads
// its cosines and sines once and takes HEADS heads with them, all of its loads
// issued before the first is used; nothing is read twice, so loads and stores
// are marked for early eviction. Measured for 16391 rows of 32 + 8 + 8 heads of
// 128 (bf16, 407 MB): 59.7 us, the rate of a plain copy; 73.2 us with 256
// threads and four heads each, 60.7 us with 128, 67.7 us with two heads each. For
// 1984 rows of 64 + 8 + 8 heads (82 MB) 14.1 us, 86 % of a copy.
#include "common.cuh"
#include "internal.h"

namespace svf {

namespace {

constexpr int kRopeThreads = 128;

struct RopeArgs {
    const uint8_t *q, *k, *v;
    long long q_stride, k_stride, v_stride;  // bytes between rows
    uint8_t *q_out, *k_cache, *v_cache;
    const float *rope;
    const int32_t *positions, *slots;
    int32_t *status;
    int T, Hq, Hkv, rot, max_pos, num_slots;
    int head_bytes;  // D * element size
    int J;           // items of a head: two 16-byte vectors each
    int pairs;       // the first `pairs` of them are rotated
    int HG;          // heads that a block covers at once
};

template <typename T>
struct Vec;
template <>
struct Vec<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void load(uint4 r, float *f) {
        f[0] = __uint_as_float(r.x);
        f[1] = __uint_as_float(r.y);
        f[2] = __uint_as_float(r.z);
        f[3] = __uint_as_float(r.w);
    }
    static __device__ __forceinline__ uint4 store(const float *f) {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                          __float_as_uint(f[3]));
    }
};
template <>
struct Vec<__nv_bfloat16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void load(uint4 r, float *f) {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ uint4 store(const float *f) {
        return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                          pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
    }
};

// block: J * HG threads, thread (j, hs) = item j of heads hs, hs + HG, ...;
// grid (rows, head blocks of HG * HEADS)
template <typename T, bool INTER, int HEADS>
__global__ void __launch_bounds__(kRopeThreads) rope_kv_kernel(RopeArgs a) {
    constexpr int N = Vec<T>::N;
    const int t = blockIdx.x;
    const int j = threadIdx.x % a.J, hs = threadIdx.x / a.J;
    pdl_wait();
    pdl_launch_dependents();
    const int slot = a.slots[t];
    const int pos = a.positions[t];
    int st = 0;
    if (slot != -1) {
        if (slot < 0 || slot >= a.num_slots) st |= SVF_DEV_BAD_PAGE;
        if (pos < 0 || pos >= a.max_pos) st |= SVF_DEV_BAD_LENGTH;
    }
    if (a.status && blockIdx.y == 0 && threadIdx.x == 0) a.status[t] = st;
    if (slot == -1) return;  // a row behind the last sequence, or one without a page
    const bool turn = j < a.pairs;
    // byte offsets of the item's two vectors inside a head; the tail of an
    // odd number of vectors ends with a single one
    const int va = (INTER || !turn) ? (turn ? 2 * j : 2 * a.pairs + 2 * (j - a.pairs)) : j;
    const int vb = (INTER || !turn) ? va + 1 : j + a.pairs;
    const int oa = va * 16, ob = vb * 16;
    const bool has_b = ob < a.head_bytes;
    float cs[N], sn[N];
    if (turn && !st) {
        const float *row = a.rope + (size_t)pos * a.rot + j * N;
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            *reinterpret_cast<float4 *>(cs + i) = __ldg(reinterpret_cast<const float4 *>(row + i));
            *reinterpret_cast<float4 *>(sn + i) =
                __ldg(reinterpret_cast<const float4 *>(row + a.rot / 2 + i));
        }
    }
    const int H = a.Hq + 2 * a.Hkv;
    const int h0 = blockIdx.y * a.HG * HEADS + hs;
    const size_t kv_row = (size_t)(st ? 0 : slot) * (size_t)(a.Hkv * a.head_bytes);
    uint4 xa[HEADS], xb[HEADS];
#pragma unroll
    for (int u = 0; u < HEADS; ++u) {
        const int h = h0 + u * a.HG;
        xa[u] = xb[u] = make_uint4(0, 0, 0, 0);
        if (h < H && !st) {
            const uint8_t *src =
                h < a.Hq ? a.q + t * a.q_stride + (size_t)h * a.head_bytes
                : h < a.Hq + a.Hkv
                    ? a.k + t * a.k_stride + (size_t)(h - a.Hq) * a.head_bytes
                    : a.v + t * a.v_stride + (size_t)(h - a.Hq - a.Hkv) * a.head_bytes;
            xa[u] = __ldcs(reinterpret_cast<const uint4 *>(src + oa));
            if (has_b) xb[u] = __ldcs(reinterpret_cast<const uint4 *>(src + ob));
        }
    }
#pragma unroll
    for (int u = 0; u < HEADS; ++u) {
        const int h = h0 + u * a.HG;
        if (h >= H || (st && h >= a.Hq)) break;  // a flagged row's q is zero, its K/V unwritten
        if (turn && !st && h < a.Hq + a.Hkv) {
            float x[2 * N], y[2 * N];
            Vec<T>::load(xa[u], x);
            Vec<T>::load(xb[u], x + N);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int p = INTER ? 2 * i : i, q = INTER ? 2 * i + 1 : N + i;
                y[p] = fmaf(x[p], cs[i], -(x[q] * sn[i]));
                y[q] = fmaf(x[q], cs[i], x[p] * sn[i]);
            }
            xa[u] = Vec<T>::store(y);
            xb[u] = Vec<T>::store(y + N);
        }
        uint8_t *dst = h < a.Hq ? a.q_out + ((size_t)t * a.Hq + h) * a.head_bytes
                       : h < a.Hq + a.Hkv
                           ? a.k_cache + kv_row + (size_t)(h - a.Hq) * a.head_bytes
                           : a.v_cache + kv_row + (size_t)(h - a.Hq - a.Hkv) * a.head_bytes;
        __stcs(reinterpret_cast<uint4 *>(dst + oa), xa[u]);
        if (has_b) __stcs(reinterpret_cast<uint4 *>(dst + ob), xb[u]);
    }
}

template <typename T, bool INTER>
cudaError_t launch_typed(const RopeArgs &a, cudaStream_t stream) {
    const int H = a.Hq + 2 * a.Hkv;
    const dim3 block((unsigned)(a.J * a.HG));
    // few rows: one head per thread, so that every load of the call is in
    // flight at once; many rows: three, which amortises the table row
    const long long blocks1 = (long long)a.T * ((H + a.HG - 1) / a.HG);
    if (blocks1 <= 2ll * num_sms())
        return launch_pdl(rope_kv_kernel<T, INTER, 1>,
                          dim3((unsigned)a.T, (unsigned)((H + a.HG - 1) / a.HG)), block, 0, stream,
                          0u, a);
    const int per = a.HG * 3;
    return launch_pdl(rope_kv_kernel<T, INTER, 3>,
                      dim3((unsigned)a.T, (unsigned)((H + per - 1) / per)), block, 0, stream, 0u,
                      a);
}

}  // namespace

bool rope_kv_supported(int T, int Hq, int Hkv, int D, int rot, int elem_size) {
    const int N = 16 / elem_size;
    return T <= (1 << 24) && Hq >= 0 && Hkv >= 1 && Hq <= 1024 && Hkv <= 1024 && D >= N &&
           D <= 512 && D % N == 0 && rot >= 2 * N && rot <= D && rot % (2 * N) == 0;
}

cudaError_t launch_rope_kv(const RopeKvArgs &p, cudaStream_t stream) {
    RopeArgs a;
    const int es = p.elem_size;
    a.q = static_cast<const uint8_t *>(p.q);
    a.k = static_cast<const uint8_t *>(p.k);
    a.v = static_cast<const uint8_t *>(p.v);
    a.q_stride = p.q_stride * es;
    a.k_stride = p.k_stride * es;
    a.v_stride = p.v_stride * es;
    a.q_out = static_cast<uint8_t *>(p.q_out);
    a.k_cache = static_cast<uint8_t *>(p.k_cache);
    a.v_cache = static_cast<uint8_t *>(p.v_cache);
    a.rope = p.rope;
    a.positions = p.positions;
    a.slots = p.slots;
    a.status = p.status;
    a.T = p.T;
    a.Hq = p.Hq;
    a.Hkv = p.Hkv;
    a.rot = p.rot;
    a.max_pos = p.max_pos;
    a.num_slots = p.num_slots;
    a.head_bytes = p.D * es;
    const int N = 16 / es;
    a.pairs = p.rot / (2 * N);
    const int tail = (p.D - p.rot) / N;
    a.J = a.pairs + (tail + 1) / 2;
    a.HG = kRopeThreads / a.J;
    const int H = p.Hq + 2 * p.Hkv;
    if (a.HG > H) a.HG = H;
    if (es == 2)
        return p.interleaved ? launch_typed<__nv_bfloat16, true>(a, stream)
                             : launch_typed<__nv_bfloat16, false>(a, stream);
    return p.interleaved ? launch_typed<float, true>(a, stream)
                         : launch_typed<float, false>(a, stream);
}

}  // namespace svf
