// norm_rope.cu -- per-head norms of a step's q and k rows, their rotary positions on one
// or several axes, and their K/V into the cache, in one pass.
//
// A q or k head x of D elements becomes
//     y = x * w / sqrt(sum x^2 / D + eps)         (no norm where its weights are absent)
//     (y_a, y_b) -> (y_a c_i - y_b s_i,  y_b c_i + y_a s_i)      for its pairs i < rot / 2,
// a, b = i, i + rot/2 (or 2i, 2i + 1 when interleaved), with c_i = rope[pos][i],
// s_i = rope[pos][rot/2 + i] at the position of the pair's own axis:
// pos = positions[axis_i][t] (time, height and width of an image's token, say; one axis:
// positions[t]). Elements from rot on keep y. q goes to q_out, k to the cache's slot,
// v is copied there. Everything is fp32 between the one read and the one rounding to the
// element type: y is not rounded before it is turned, so the result is off by half a step
// of its type and no more than a few 2^-24 besides.
//
// Bound: HBM, as rope_kv.cu: each element is read once and written once. A head's items
// (two 16-byte vectors each) belong to a power of two of neighbouring lanes; the sums of squares
// of a thread's heads meet in the same shuffles, and neighbouring elements are multiplied in
// pairs. Measured for 16391 rows of 32 + 8 + 8 heads of 128 (bf16, 411 MB): 64.5 us on one
// axis (the rotary write alone takes 59.7, a copy 60.6), 82 with the heads' sums one after the
// other; 74.5 us on three axes, whose cosines a block first gathers to shared memory (81.6 with every
// thread gathering its own). Seven blocks an SM: six 66 and 78 us, eight spill (92 and 78).
#include "common.cuh"
#include "internal.h"
#include "vec16.cuh"

namespace svf {

namespace {

constexpr int kNormRopeThreads = 128;
constexpr int kMostPairs = 128;  // D <= 256

struct NormRopeDev {
    const uint8_t *q, *k, *v;
    long long q_stride, k_stride, v_stride;  // bytes between rows
    uint8_t *q_out, *k_cache, *v_cache;
    const uint8_t *q_norm, *k_norm;
    const float *rope;
    const int32_t *positions, *pair_axis, *slots;
    int32_t *status;
    int T, Hq, Hkv, rot, max_pos, num_slots, axes;
    int head_bytes;  // D * element size
    int J;           // items of a head: two 16-byte vectors each
    int lanes;       // lanes of a head: the power of two from J on
    int pairs;       // the first `pairs` items are rotated
    int HG;          // heads that a block covers at once
    float eps, inv_d;
};

__device__ __forceinline__ float2 fmul2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 ra, rb, rd;\n\t"
        "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
        "mul.rn.f32x2 rd, ra, rb;\n\t"
        "mov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

// block: lanes * HG threads, thread (j, hs) = item j of heads hs, hs + HG, ...;
// grid (rows, head blocks of HG * HEADS)
template <typename T, bool INTER, bool MULTI, int HEADS>
__global__ void __launch_bounds__(kNormRopeThreads, 7) norm_rope_kernel(NormRopeDev a) {
    constexpr int N = Vec<T>::N;
    const int t = blockIdx.x;
    const int j = threadIdx.x % a.lanes, hs = threadIdx.x / a.lanes;
    pdl_wait();
    pdl_launch_dependents();
    // what the addresses of a row depend on, in one round trip
    const int slot = a.slots[t];
    int pos[MULTI ? 4 : 1];
#pragma unroll
    for (int x = 0; x < (MULTI ? 4 : 1); ++x)
        pos[x] = x < a.axes ? a.positions[(size_t)x * a.T + t] : 0;
    int axis = 0;
    if (MULTI && threadIdx.x < a.rot / 2) axis = __ldg(a.pair_axis + threadIdx.x);
    int st = 0;
    if (slot != -1) {
        if (slot < 0 || slot >= a.num_slots) st |= SVF_DEV_BAD_PAGE;
#pragma unroll
        for (int x = 0; x < (MULTI ? 4 : 1); ++x)
            if (x < a.axes && (pos[x] < 0 || pos[x] >= a.max_pos)) st |= SVF_DEV_BAD_LENGTH;
    }
    const bool turn = j < a.pairs;
    __shared__ __align__(16) float s_cs[MULTI ? 2 * kMostPairs : 4];  // cosines, then sines
    const int H = a.Hq + 2 * a.Hkv;
    const int h0 = blockIdx.y * a.HG * HEADS + hs;
    const bool item = j < a.J;
    // byte offsets of the item's two vectors inside a head; the tail of an
    // odd number of vectors ends with a single one
    const int va = (INTER || !turn) ? (turn ? 2 * j : 2 * a.pairs + 2 * (j - a.pairs)) : j;
    const int vb = (INTER || !turn) ? va + 1 : j + a.pairs;
    const int oa = va * 16, ob = vb * 16;
    const bool has_b = item && ob < a.head_bytes;
    const bool left_out = slot == -1;  // a row behind the last sequence, or one without a page
    uint4 xa[HEADS], xb[HEADS];
#pragma unroll
    for (int u = 0; u < HEADS; ++u) {
        const int h = h0 + u * a.HG;
        xa[u] = xb[u] = make_uint4(0, 0, 0, 0);
        if (item && h < H && !st && !left_out) {
            const uint8_t *src =
                h < a.Hq ? a.q + t * a.q_stride + (size_t)h * a.head_bytes
                : h < a.Hq + a.Hkv
                    ? a.k + t * a.k_stride + (size_t)(h - a.Hq) * a.head_bytes
                    : a.v + t * a.v_stride + (size_t)(h - a.Hq - a.Hkv) * a.head_bytes;
            xa[u] = __ldcs(reinterpret_cast<const uint4 *>(src + oa));
            if (has_b) xb[u] = __ldcs(reinterpret_cast<const uint4 *>(src + ob));
        }
    }
    if (MULTI) {
        // the row's cosines and sines, each pair's by its own axis, once for all heads
        bool bad = false;
        for (int i = threadIdx.x; i < a.rot / 2; i += (int)blockDim.x) {
            const int ax = i == threadIdx.x ? axis : __ldg(a.pair_axis + i);
            if (ax < 0 || ax >= a.axes) {
                bad = true;
            } else if (!st && !left_out) {
                const int at = ax == 0 ? pos[0] : ax == 1 ? pos[MULTI] : ax == 2 ? pos[2 * MULTI] : pos[3 * MULTI];
                const float *row = a.rope + (size_t)at * a.rot + i;
                s_cs[i] = __ldg(row);
                s_cs[kMostPairs + i] = __ldg(row + a.rot / 2);
            }
        }
        // (every block looks at all pairs, so all agree)
        if (__syncthreads_or(bad) && !left_out) {
            st |= SVF_DEV_BAD_LENGTH;
#pragma unroll
            for (int u = 0; u < HEADS; ++u) xa[u] = xb[u] = make_uint4(0, 0, 0, 0);
        }
    }
    if (a.status && blockIdx.y == 0 && threadIdx.x == 0) a.status[t] = st;
    if (left_out) return;
    float cs[N], sn[N];
    if (turn && !st) {
        const float *row = MULTI ? s_cs + j * N : a.rope + (size_t)pos[0] * a.rot + j * N;
        const int sines = MULTI ? kMostPairs : a.rot / 2;
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            *reinterpret_cast<float4 *>(cs + i) = *reinterpret_cast<const float4 *>(row + i);
            *reinterpret_cast<float4 *>(sn + i) = *reinterpret_cast<const float4 *>(row + sines + i);
        }
    }
    const size_t kv_row = (size_t)(st ? 0 : slot) * (size_t)(a.Hkv * a.head_bytes);
    // the heads' sums of squares, all of them through the same shuffles
    float ss[HEADS];
#pragma unroll
    for (int u = 0; u < HEADS; ++u) {
        float x[2 * N];
        Vec<T>::load(xa[u], x);
        Vec<T>::load(xb[u], x + N);
        float2 s2 = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float2 v = make_float2(x[2 * i], x[2 * i + 1]);
            s2 = ffma2(v, v, s2);
        }
        ss[u] = s2.x + s2.y;
    }
    if (a.q_norm || a.k_norm)
        for (int o = a.lanes >> 1; o > 0; o >>= 1)
#pragma unroll
            for (int u = 0; u < HEADS; ++u) ss[u] += __shfl_xor_sync(0xffffffffu, ss[u], o);
#pragma unroll
    for (int u = 0; u < HEADS; ++u) {
        const int h = h0 + u * a.HG;
        const bool is_q = h < a.Hq;
        if (!st) {
            float x[2 * N];
            Vec<T>::load(xa[u], x);
            Vec<T>::load(xb[u], x + N);
            // in pairs of neighbouring elements, which one instruction takes
            float2 x2[N];
#pragma unroll
            for (int i = 0; i < N; ++i) x2[i] = make_float2(x[2 * i], x[2 * i + 1]);
            if (item && h < a.Hq + a.Hkv) {
                const uint8_t *w = is_q ? a.q_norm : a.k_norm;
                const bool normed = w != nullptr;
                if (normed) {
                    const float r = rsqrtf(fmaf(ss[u], a.inv_d, a.eps));
                    const float2 r2 = make_float2(r, r);
                    float g[2 * N];
                    Vec<T>::load(__ldg(reinterpret_cast<const uint4 *>(w + oa)), g);
                    Vec<T>::load(__ldg(reinterpret_cast<const uint4 *>(w + (has_b ? ob : oa))), g + N);
#pragma unroll
                    for (int i = 0; i < N; ++i)
                        x2[i] = fmul2(fmul2(x2[i], r2), make_float2(g[2 * i], g[2 * i + 1]));
                }
                if (turn) {
                    if (INTER) {
#pragma unroll
                        for (int i = 0; i < N; ++i)
                            x2[i] = ffma2(x2[i], make_float2(cs[i], cs[i]),
                                          fmul2(make_float2(x2[i].y, x2[i].x), make_float2(-sn[i], sn[i])));
                    } else {
#pragma unroll
                        for (int i = 0; i < N / 2; ++i) {
                            const float2 c2 = make_float2(cs[2 * i], cs[2 * i + 1]);
                            const float2 n2 = make_float2(sn[2 * i], sn[2 * i + 1]);
                            const float2 p = x2[i], q = x2[N / 2 + i];
                            x2[i] = ffma2(p, c2, fmul2(q, make_float2(-n2.x, -n2.y)));
                            x2[N / 2 + i] = ffma2(q, c2, fmul2(p, n2));
                        }
                    }
                }
                if (normed || turn) {  // (what is only copied keeps its bits, a NaN's too)
#pragma unroll
                    for (int i = 0; i < N; ++i) {
                        x[2 * i] = x2[i].x;
                        x[2 * i + 1] = x2[i].y;
                    }
                    xa[u] = Vec<T>::store(x);
                    xb[u] = Vec<T>::store(x + N);
                }
            }
        }
        if (!item || h >= H || (st && !is_q)) continue;  // a flagged row's q is zero, its K/V unwritten
        uint8_t *dst = is_q ? a.q_out + ((size_t)t * a.Hq + h) * a.head_bytes
                       : h < a.Hq + a.Hkv
                           ? a.k_cache + kv_row + (size_t)(h - a.Hq) * a.head_bytes
                           : a.v_cache + kv_row + (size_t)(h - a.Hq - a.Hkv) * a.head_bytes;
        __stcs(reinterpret_cast<uint4 *>(dst + oa), xa[u]);
        if (has_b) __stcs(reinterpret_cast<uint4 *>(dst + ob), xb[u]);
    }
}

template <typename T, bool INTER, bool MULTI>
cudaError_t launch_typed(const NormRopeDev &a, cudaStream_t stream) {
    const int H = a.Hq + 2 * a.Hkv;
    const dim3 block((unsigned)(a.lanes * a.HG));
    // few rows: one head per thread, so that every load of the call is in
    // flight at once; many rows: three, which amortises the table row
    const long long blocks1 = (long long)a.T * ((H + a.HG - 1) / a.HG);
    if (blocks1 <= 2ll * num_sms())
        return launch_pdl(norm_rope_kernel<T, INTER, MULTI, 1>,
                          dim3((unsigned)a.T, (unsigned)((H + a.HG - 1) / a.HG)), block, 0, stream,
                          0u, a);
    const int per = a.HG * 3;
    return launch_pdl(norm_rope_kernel<T, INTER, MULTI, 3>,
                      dim3((unsigned)a.T, (unsigned)((H + per - 1) / per)), block, 0, stream, 0u,
                      a);
}

template <typename T>
cudaError_t launch_type(const NormRopeDev &a, bool inter, cudaStream_t stream) {
    if (a.axes > 1)
        return inter ? launch_typed<T, true, true>(a, stream)
                     : launch_typed<T, false, true>(a, stream);
    return inter ? launch_typed<T, true, false>(a, stream)
                 : launch_typed<T, false, false>(a, stream);
}

}  // namespace

bool norm_rope_supported(int T, int Hq, int Hkv, int D, int rot, int axes, int elem_size) {
    return rope_kv_supported(T, Hq, Hkv, D, rot, elem_size) && D <= 256 && axes >= 1 && axes <= 4;
}

cudaError_t launch_norm_rope(const NormRopeArgs &n, cudaStream_t stream) {
    const RopeKvArgs &p = n.rope;
    NormRopeDev a;
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
    a.q_norm = static_cast<const uint8_t *>(n.q_norm);
    a.k_norm = static_cast<const uint8_t *>(n.k_norm);
    a.rope = p.rope;
    a.positions = p.positions;
    a.pair_axis = n.pair_axis;
    a.slots = p.slots;
    a.status = p.status;
    a.T = p.T;
    a.Hq = p.Hq;
    a.Hkv = p.Hkv;
    a.rot = p.rot;
    a.max_pos = p.max_pos;
    a.num_slots = p.num_slots;
    a.axes = n.axes;
    a.eps = n.eps;
    a.inv_d = 1.0f / (float)p.D;
    a.head_bytes = p.D * es;
    const int N = 16 / es;
    a.pairs = p.rot / (2 * N);
    const int tail = (p.D - p.rot) / N;
    a.J = a.pairs + (tail + 1) / 2;
    a.lanes = 1;
    while (a.lanes < a.J) a.lanes *= 2;
    a.HG = kNormRopeThreads / a.lanes;
    // whole warps, for the shuffles: lanes and 128 are powers of two
    const int H = p.Hq + 2 * p.Hkv;
    while (a.HG * a.lanes > 32 && a.HG / 2 >= H) a.HG /= 2;
    return es == 2 ? launch_type<__nv_bfloat16>(a, p.interleaved, stream)
                   : launch_type<float>(a, p.interleaved, stream);
}

}  // namespace svf
