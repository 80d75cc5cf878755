// Norm of every query and key head with the position rotation in the same pass,
// and its gradient.
//
//   n = x r w,  r = 1 / sqrt(sum x^2 [/ d] + eps);  pairs (n_p, n_{p + R}), p < R, turned by the
//   angle position * inv_freq[p]; the channels behind 2 R pass through.
//
// Backward, with dn the gradient turned back: dw = sum dn x r, and with u = dn w
//   dx = r (u - x r^2 (sum u x) [/ d]).
//
// Bound by its bytes: x in, y out (backward: x and dy in, dx out). A row's
// channels are split into units of V: unit i is channels [i V, i V + V) together
// with the V at distance R that they turn with (behind 2 R: with the next half of
// the rest), so that a lane holds both halves of its pairs and a row needs no
// exchange but the sum of squares. A CTA takes one position and turns all images
// and heads of it by one set of angles: sines and cosines are computed once a
// position, from float64 angles (a float32 product is off by whole radians at
// positions of 2^24).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "vscan_common.cuh"

namespace vscan {

constexpr int QN_THREADS = 256;
constexpr int QN_MAX_PAIRS = 128;  // d <= 256

struct QkNormParams {
    int batch, tokens, heads_q, heads_k, d, pairs, axes;
    int rms;             // 1: mean of squares, 0: sum
    int pos_img;         // elements between images of positions (0: shared)
    int groups;          // CTAs that share one position's images
    int lanes;           // lanes of a row: a power of two
    int units;           // units of a row
    float eps;
    const void *q, *k;
    const float *wq, *wk, *inv_freq;
    const int* positions;
    void *yq, *yk;
    long long q_tok, q_img, k_tok, k_img, yq_tok, yq_img, yk_tok, yk_img;
    // backward: dyq, dyk at the y strides, dense dq, dk
    const void *dyq, *dyk;
    void *dq, *dk;
    float* part;         // [CTAs][2][d] sums for the weights, or null
    int blocks;
};

// First channels of the two halves of unit i, or -1 where it has no second (first) half.
__device__ __forceinline__ void qn_unit(const QkNormParams& p, int V, int i, int& lo, int& hi)
{
    const int turned = p.pairs / V;  // units that are rotated; the host picks V to divide pairs
    if (i < turned) {
        lo = i * V;
        hi = lo + p.pairs;
        return;
    }
    const int rest = (p.d - 2 * p.pairs) / V, first = (rest + 1) / 2, j = i - turned;
    lo = j < first ? 2 * p.pairs + j * V : -1;
    hi = j < first && j + first < rest ? lo + first * V : -1;
}

// Plain loads: the output may be the input's own memory, which the read-only path excludes.
template <typename T, int V>
__device__ __forceinline__ void qn_load(const T* p, float (&x)[V])
{
    if constexpr (sizeof(T) == 2 && V >= 2) {
        uint32_t a[V / 2];
        if constexpr (V == 8) {
            const uint4 u = *reinterpret_cast<const uint4*>(p);
            a[0] = u.x; a[1] = u.y; a[2] = u.z; a[3] = u.w;
        } else if constexpr (V == 4) {
            const uint2 u = *reinterpret_cast<const uint2*>(p);
            a[0] = u.x; a[1] = u.y;
        } else {
            a[0] = *reinterpret_cast<const uint32_t*>(p);
        }
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            x[2 * i] = __uint_as_float(a[i] << 16);
            x[2 * i + 1] = __uint_as_float(a[i] & 0xffff0000u);
        }
    } else if constexpr (sizeof(T) == 4 && V == 4) {
        const float4 u = *reinterpret_cast<const float4*>(p);
        x[0] = u.x; x[1] = u.y; x[2] = u.z; x[3] = u.w;
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = to_float(p[i]);
    }
}

template <typename T, int V>
__device__ __forceinline__ void qn_store(T* p, const float (&x)[V])
{
    if constexpr (V == 8) {
        uint4 u;
        __nv_bfloat162 a[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        u.x = *reinterpret_cast<uint32_t*>(&a[0]);
        u.y = *reinterpret_cast<uint32_t*>(&a[1]);
        u.z = *reinterpret_cast<uint32_t*>(&a[2]);
        u.w = *reinterpret_cast<uint32_t*>(&a[3]);
        *reinterpret_cast<uint4*>(p) = u;
    } else if constexpr (V == 4) {
        store4(p, make_float4(x[0], x[1], x[2], x[3]));
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) store_elem(p + i, x[i]);
    }
}

// Cosine and sine of every pair's angle at one position, by the whole CTA.
__device__ __forceinline__ void qn_angles(const QkNormParams& p, const int* pos, float2* cs)
{
    const int per = p.pairs / p.axes;
    for (int i = threadIdx.x; i < p.pairs; i += QN_THREADS) {
        // the product is exact in float64 (31 + 24 bits round to 53: 2^-53 of it); whole turns come off there
        const double turn = (double)pos[i / per] * (double)p.inv_freq[i];
        const double two_pi = 6.283185307179586476925;
        const double r = fma(-rint(turn / two_pi), two_pi, turn);
        float s, c;
        sincosf((float)r, &s, &c);
        cs[i] = make_float2(c, s);
    }
}

// Rows of one position: (image of the group) x (query heads, then key heads).
template <typename T, int V, int U, bool BACK>
__global__ void __launch_bounds__(QN_THREADS) qk_norm_kernel(const QkNormParams p)
{
    __shared__ float2 cs[QN_MAX_PAIRS];
    extern __shared__ float wsum[];  // backward with weights: [warps][2][d]
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int sub = lane & (p.lanes - 1), per_warp = 32 / p.lanes;
    const int heads = p.heads_q + p.heads_k;
    const int row_slot = warp * per_warp + lane / p.lanes, row_slots = (QN_THREADS / 32) * per_warp;
    int lo[U], hi[U];
    float w[2][U][2 * V];
    float acc[BACK ? 2 : 1][U][2 * V];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int i = u * p.lanes + sub;
        lo[u] = hi[u] = -1;
        if (i < p.units) qn_unit(p, V, i, lo[u], hi[u]);
#pragma unroll
        for (int e = 0; e < V; ++e)
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const float* src = t ? p.wk : p.wq;
                w[t][u][e] = src && lo[u] >= 0 ? src[lo[u] + e] : 1.f;
                w[t][u][V + e] = src && hi[u] >= 0 ? src[hi[u] + e] : 1.f;
            }
    }
    if (BACK) {
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int e = 0; e < 2 * V; ++e) acc[t][u][e] = 0.f;
    }
    const long long work = (long long)p.tokens * p.groups;
    for (long long item = blockIdx.x; item < work; item += gridDim.x) {
        const int token = (int)(item / p.groups), group = (int)(item - (long long)token * p.groups);
        if (p.pairs) {
            __syncthreads();
            qn_angles(p, p.positions + (long long)group * p.pos_img + (long long)token * p.axes, cs);
            __syncthreads();
        }
        const int images = (p.batch - group + p.groups - 1) / p.groups;  // group, group + groups, ..
        const int rows = images * heads;
        for (int first = 0; first < rows; first += row_slots) {
            const int row = first + row_slot;
            const bool live = row < rows;
            const int image = group + (row / heads) * p.groups, h = row - (row / heads) * heads;
            const bool key = h >= p.heads_q;
            const int head = key ? h - p.heads_q : h;
            const T* src = key ? reinterpret_cast<const T*>(p.k) + image * p.k_img + token * p.k_tok
                               : reinterpret_cast<const T*>(p.q) + image * p.q_img + token * p.q_tok;
            const long long yat = key ? image * p.yk_img + token * p.yk_tok : image * p.yq_img + token * p.yq_tok;
            src += (long long)head * p.d;
            float x[U][2 * V], dy[BACK ? U : 1][2 * V];
            float sq = 0.f;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float a[V] = {}, b[V] = {};
                if (live && lo[u] >= 0) qn_load<T, V>(src + lo[u], a);
                if (live && hi[u] >= 0) qn_load<T, V>(src + hi[u], b);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    x[u][e] = a[e];
                    x[u][V + e] = b[e];
                    sq += a[e] * a[e] + b[e] * b[e];
                }
            }
            if (BACK) {
                const T* g = reinterpret_cast<const T*>(key ? p.dyk : p.dyq) + yat + (long long)head * p.d;
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    float a[V] = {}, b[V] = {};
                    if (live && lo[u] >= 0) qn_load<T, V>(g + lo[u], a);
                    if (live && hi[u] >= 0) qn_load<T, V>(g + hi[u], b);
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        dy[u][e] = a[e];
                        dy[u][V + e] = b[e];
                    }
                }
            }
            for (int o = p.lanes >> 1; o > 0; o >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
            const float r = 1.f / sqrtf((p.rms ? sq / p.d : sq) + p.eps);
            if (!BACK) {
                T* dst = reinterpret_cast<T*>(key ? p.yk : p.yq) + yat + (long long)head * p.d;
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    float a[V], b[V];
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        a[e] = x[u][e] * r * (key ? w[1][u][e] : w[0][u][e]);
                        b[e] = x[u][V + e] * r * (key ? w[1][u][V + e] : w[0][u][V + e]);
                        if (lo[u] >= 0 && lo[u] < p.pairs) {
                            const float2 t = cs[lo[u] + e];
                            const float y = a[e] * t.x - b[e] * t.y;
                            b[e] = a[e] * t.y + b[e] * t.x;
                            a[e] = y;
                        }
                    }
                    if (live && lo[u] >= 0) qn_store<T, V>(dst + lo[u], a);
                    if (live && hi[u] >= 0) qn_store<T, V>(dst + hi[u], b);
                }
            } else {
                float inner = 0.f;
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        float a = dy[u][e], b = dy[u][V + e];
                        if (lo[u] >= 0 && lo[u] < p.pairs) {  // turned back
                            const float2 t = cs[lo[u] + e];
                            const float y = a * t.x + b * t.y;
                            b = b * t.x - a * t.y;
                            a = y;
                        }
                        const float ga = a * x[u][e] * r, gb = b * x[u][V + e] * r;
                        if (key) {
                            acc[BACK ? 1 : 0][u][e] += ga;
                            acc[BACK ? 1 : 0][u][V + e] += gb;
                        } else {
                            acc[0][u][e] += ga;
                            acc[0][u][V + e] += gb;
                        }
                        a *= key ? w[1][u][e] : w[0][u][e];
                        b *= key ? w[1][u][V + e] : w[0][u][V + e];
                        inner += a * x[u][e] + b * x[u][V + e];
                        dy[u][e] = a;
                        dy[u][V + e] = b;
                    }
                for (int o = p.lanes >> 1; o > 0; o >>= 1) inner += __shfl_xor_sync(0xffffffffu, inner, o);
                const float f = (p.rms ? inner / p.d : inner) * r * r;
                T* dst = reinterpret_cast<T*>(key ? p.dk : p.dq);
                if (dst) {
                    dst += (((long long)image * p.tokens + token) * (key ? p.heads_k : p.heads_q) + head) * p.d;
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        float a[V], b[V];
#pragma unroll
                        for (int e = 0; e < V; ++e) {
                            a[e] = r * (dy[u][e] - x[u][e] * f);
                            b[e] = r * (dy[u][V + e] - x[u][V + e] * f);
                        }
                        if (live && lo[u] >= 0) qn_store<T, V>(dst + lo[u], a);
                        if (live && hi[u] >= 0) qn_store<T, V>(dst + hi[u], b);
                    }
                }
            }
        }
    }
    if (BACK && p.part) {
        // the rows of a warp hold the same channels: add them up, then the warps, in a fixed order
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int e = 0; e < 2 * V; ++e) {
                    float a = acc[BACK ? t : 0][u][e];
                    for (int o = p.lanes; o < 32; o <<= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
                    const int base = e < V ? lo[u] : hi[u];
                    if (lane < p.lanes && base >= 0) wsum[(warp * 2 + t) * p.d + base + (e < V ? e : e - V)] = a;
                }
        __syncthreads();
        for (int i = tid; i < 2 * p.d; i += QN_THREADS) {
            float a = 0.f;
            for (int wp = 0; wp < QN_THREADS / 32; ++wp) a += wsum[wp * 2 * p.d + i];
            p.part[(long long)blockIdx.x * 2 * p.d + i] = a;
        }
    }
}

// dwq, dwk: the CTAs' sums added in a fixed order, in float64. One warp a channel.
__global__ void __launch_bounds__(QN_THREADS) qk_norm_weight_kernel(const float* part, int blocks, int d, float* dwq, float* dwk)
{
    const int i = blockIdx.x * (QN_THREADS / 32) + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (i >= 2 * d) return;
    float* dst = i < d ? dwq : dwk;
    if (!dst) return;
    double a = 0.0;
    for (int b = lane; b < blocks; b += 32) a += (double)part[(long long)b * 2 * d + i];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a += __shfl_down_sync(0xffffffffu, a, o);
    if (lane == 0) dst[i < d ? i : i - d] = (float)a;
}

}  // namespace vscan
