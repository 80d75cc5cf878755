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
// exchange but the sum of squares. A CTA takes one position of q or of k and turns
// its images and heads by one set of angles: sines and cosines are computed once a
// position, from float64 angles (a float32 product is off by whole radians at
// positions of 2^24). Two rows a lane are in flight where a row takes one unit a lane
// (one row where the registers end: gradients at V = 8, rows of several units a lane), and
// weights wait in shared memory, for more CTAs an SM. Registers are capped at 64 forward and
// 80 backward; at V = 8 the forward pass spills 48 bytes a thread there, at V = 4 the passes
// 8 to 24. On 64 images of 4097 tokens, 6 + 6 heads of 128, bf16, forward: 308 us, 5.2 TB/s, 80 %
// of the copy rate, the issue slots half used (329 us with scalar products and a division for
// every row's head). Gradients of 16 images of 3136 tokens, 12 + 4 heads of 72: 136 us, 2.5
// times their bytes: 72 channels fill five of a row's eight lanes, q's CTAs have three times the
// rows of k's, and one row a lane is in flight.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "vscan_common.cuh"
#include "vscan_tc.cuh"

namespace vscan {

constexpr int QN_THREADS = 256, QN_SUM_THREADS = 1024;
constexpr int QN_MAX_PAIRS = 128;  // d <= 256

struct QkNormSide {  // q or k
    int heads;
    const void* x;
    const float* w;
    void* y;             // backward: dense gradient of x
    const void* dy;
    long long x_tok, x_img, y_tok, y_img;  // y's (backward: dy's) strides
};

struct QkNormParams {
    int batch, tokens, d, pairs, axes;
    int rms;             // 1: mean of squares, 0: sum
    int pos_img;         // elements between images of positions (0: shared)
    int groups;          // CTAs that share one position's images
    int lanes;           // lanes of a row: a power of two
    int units;           // units of a row
    float eps;
    const float* inv_freq;
    const int* positions;
    QkNormSide side[2];
    float* part;         // backward: [2][blocks][d] sums for the weights, or null
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

// V neighbouring values from shared memory, 16 bytes at a time where V allows.
template <int V>
__device__ __forceinline__ void qn_shared(const float* s, float (&v)[V])
{
    if constexpr (V >= 4) {
#pragma unroll
        for (int i = 0; i < V; i += 4) *reinterpret_cast<float4*>(v + i) = *reinterpret_cast<const float4*>(s + i);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = s[i];
    }
}

// Two values an instruction, where there are two: v *= s; s += x y; a turn of pairs, x = a c + m d and
// y = b c + n d with (m, n) = (-b, a), or back with (b, -a).
template <int V>
__device__ __forceinline__ void qn_scale(float (&v)[V], const float (&s)[V])
{
    if constexpr (V == 1) {
        v[0] *= s[0];
    } else {
#pragma unroll
        for (int e = 0; e < V; e += 2) {
            const float2 y = __fmul2_rn(make_float2(v[e], v[e + 1]), make_float2(s[e], s[e + 1]));
            v[e] = y.x;
            v[e + 1] = y.y;
        }
    }
}
template <int V>
__device__ __forceinline__ void qn_add(float (&s)[V], const float (&x)[V], const float (&y)[V])
{
    if constexpr (V == 1) {
        s[0] += x[0] * y[0];
    } else {
#pragma unroll
        for (int e = 0; e < V; e += 2) {
            const float2 z = __ffma2_rn(make_float2(x[e], x[e + 1]), make_float2(y[e], y[e + 1]), make_float2(s[e], s[e + 1]));
            s[e] = z.x;
            s[e + 1] = z.y;
        }
    }
}
template <bool BACK, int V>
__device__ __forceinline__ void qn_turn(float (&a)[V], float (&b)[V], const float (&c)[V], const float (&d)[V])
{
    float m[V], n[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
        m[e] = BACK ? b[e] : -b[e];
        n[e] = BACK ? -a[e] : a[e];
    }
    qn_scale(a, c);
    qn_scale(b, c);
    qn_add(a, m, d);
    qn_add(b, n, d);
}

// Cosine and sine of every pair's angle at one position, by the whole CTA.
__device__ __forceinline__ void qn_angles(const QkNormParams& p, const int* pos, float* cosine, float* sine)
{
    const int per = p.pairs / p.axes;
    for (int i = threadIdx.x; i < p.pairs; i += QN_THREADS) {
        // the product rounds to 2^-53 of itself; whole turns come off in float64
        const double angle = (double)pos[i / per] * (double)p.inv_freq[i];
        constexpr double two_pi = 6.283185307179586476925, per_turn = 0.15915494309189533577;
        const double rest = fma(-rint(angle * per_turn), two_pi, angle);
        sincospif((float)(rest * (2.0 * per_turn)), sine + i, cosine + i);
    }
}

// Rows of one position: (image of the group) x head. blockIdx.y: q or k.
template <typename T, int V, int U, bool BACK>
__global__ void __launch_bounds__(QN_THREADS, BACK ? 3 : 4) qk_norm_kernel(const QkNormParams p)
{
    constexpr int R = U == 1 && (!BACK || V <= 4) ? 2 : 1;  // rows a lane has in flight
    __shared__ __align__(16) float cosine[QN_MAX_PAIRS], sine[QN_MAX_PAIRS], weight[2 * QN_MAX_PAIRS];
    extern __shared__ float wsum[];  // backward with weights: [warps][d]
    const QkNormSide& side = p.side[blockIdx.y];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int sub = lane & (p.lanes - 1), per_warp = 32 / p.lanes;
    const int row_slot = warp * per_warp + lane / p.lanes, row_slots = (QN_THREADS / 32) * per_warp;
    const bool weighted = side.w != nullptr;
    if (weighted)
        for (int i = tid; i < p.d; i += QN_THREADS) weight[i] = side.w[i];
    int lo[U], hi[U];
    float acc[BACK ? U : 1][2 * V];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int i = u * p.lanes + sub;
        lo[u] = hi[u] = -1;
        if (i < p.units) qn_unit(p, V, i, lo[u], hi[u]);
    }
    if (BACK) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int e = 0; e < 2 * V; ++e) acc[u][e] = 0.f;
    }
    const long long work = (long long)p.tokens * p.groups;
    // a lane's rows are R * row_slots apart: so many images and heads
    const int hop = R * row_slots /* <= 512 */, hop_at = hop / side.heads, hop_head = hop - hop_at * side.heads;
    for (long long item = blockIdx.x; item < work; item += gridDim.x) {
        const int token = (int)(item / p.groups), group = (int)(item - (long long)token * p.groups);
        __syncthreads();
        if (p.pairs) qn_angles(p, p.positions + (long long)group * p.pos_img + (long long)token * p.axes, cosine, sine);
        __syncthreads();
        const int images = (p.batch - group + p.groups - 1) / p.groups;  // group, group + groups, ..
        const int rows = images * side.heads;
        const T* x_item = reinterpret_cast<const T*>(side.x) + group * side.x_img + token * side.x_tok;
        const long long y_item = group * side.y_img + token * side.y_tok, x_hop = p.groups * side.x_img, y_hop = p.groups * side.y_img;
        int at[R], head[R];
#pragma unroll
        for (int k = 0; k < R; ++k) {
            at[k] = (k * row_slots + row_slot) / side.heads;
            head[k] = k * row_slots + row_slot - at[k] * side.heads;
        }
        for (int first = 0; first < rows; first += hop) {
            float x[R][U][2 * V], dy[BACK ? R : 1][U][2 * V];
            long long yat[R], dense[BACK ? R : 1];
            bool live[R];
#pragma unroll
            for (int k = 0; k < R; ++k) {
                live[k] = at[k] < images;
                const long long in_token = (long long)head[k] * p.d;
                const T* src = x_item + at[k] * x_hop + in_token;
                yat[k] = y_item + at[k] * y_hop + in_token;
                if (BACK) dense[k] = ((long long)(group + at[k] * p.groups) * p.tokens + token) * side.heads * p.d + in_token;
                at[k] += hop_at;
                head[k] += hop_head;
                if (head[k] >= side.heads) {
                    head[k] -= side.heads;
                    ++at[k];
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    float a[V] = {}, b[V] = {};
                    if (live[k] && lo[u] >= 0) qn_load<T, V>(src + lo[u], a);
                    if (live[k] && hi[u] >= 0) qn_load<T, V>(src + hi[u], b);
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        x[k][u][e] = a[e];
                        x[k][u][V + e] = b[e];
                    }
                    if (BACK) {
                        const T* g = reinterpret_cast<const T*>(side.dy) + yat[k];
                        float c[V] = {}, d[V] = {};
                        if (live[k] && lo[u] >= 0) qn_load<T, V>(g + lo[u], c);
                        if (live[k] && hi[u] >= 0) qn_load<T, V>(g + hi[u], d);
#pragma unroll
                        for (int e = 0; e < V; ++e) {
                            dy[k][u][e] = c[e];
                            dy[k][u][V + e] = d[e];
                        }
                    }
                }
            }
#pragma unroll
            for (int k = 0; k < R; ++k) {
                float squares[2] = {};
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int e = 0; e < 2 * V; e += 2) {
                        const float x2[2] = {x[k][u][e], x[k][u][e + 1]};
                        qn_add(squares, x2, x2);
                    }
                float sq = squares[0] + squares[1];
                for (int o = p.lanes >> 1; o > 0; o >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
                const float square = (p.rms ? sq / p.d : sq) + p.eps;
                float r = rsqrtf(square);  // good to 2 units of the last place: enough for what leaves in bf16
                if ((BACK || sizeof(T) == 4) && r > 0.f && r < __int_as_float(0x7f800000))  // else one step of Newton's
                    r = fmaf(0.5f * r, fmaf(-square * r, r, 1.f), r);
                // a row that is not there has no length: without eps its r is infinite, and 0 r NaN in the weights'
                // sums. Asked by its index: any further use of live[k], the loads' flag, costs (56x56 gradients: 135 -> 200 us)
                if (BACK && first + k * row_slots + row_slot >= rows) r = 0.f;
                if (!BACK) {
                    T* dst = reinterpret_cast<T*>(side.y) + yat[k];
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        float a[V], b[V], c[V], d[V];
#pragma unroll
                        for (int e = 0; e < V; ++e) {
                            a[e] = x[k][u][e];
                            b[e] = x[k][u][V + e];
                            c[e] = r;
                        }
                        qn_scale(a, c);
                        qn_scale(b, c);
                        if (weighted) {
                            qn_shared<V>(weight + max(lo[u], 0), c);
                            qn_shared<V>(weight + max(hi[u], 0), d);
                            qn_scale(a, c);
                            qn_scale(b, d);
                        }
                        if (lo[u] >= 0 && lo[u] < p.pairs) {  // turned
                            qn_shared<V>(cosine + lo[u], c);
                            qn_shared<V>(sine + lo[u], d);
                            qn_turn<false>(a, b, c, d);
                        }
                        if (live[k] && lo[u] >= 0) qn_store<T, V>(dst + lo[u], a);
                        if (live[k] && hi[u] >= 0) qn_store<T, V>(dst + hi[u], b);
                    }
                } else {
                    float inner = 0.f;
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        float a[V], b[V], c[V], d[V];
#pragma unroll
                        for (int e = 0; e < V; ++e) {
                            a[e] = dy[k][u][e];
                            b[e] = dy[k][u][V + e];
                        }
                        if (lo[u] >= 0 && lo[u] < p.pairs) {  // turned back
                            qn_shared<V>(cosine + lo[u], c);
                            qn_shared<V>(sine + lo[u], d);
                            qn_turn<true>(a, b, c, d);
                        }
                        float dn[2 * V], n[2 * V];
#pragma unroll
                        for (int e = 0; e < 2 * V; ++e) {
                            dn[e] = e < V ? a[e] : b[e - V];
                            n[e] = r;
                        }
                        qn_scale(n, x[k][u]);
                        qn_add(acc[u], dn, n);
                        if (weighted) {
                            qn_shared<V>(weight + max(lo[u], 0), c);
                            qn_shared<V>(weight + max(hi[u], 0), d);
#pragma unroll
                            for (int e = 0; e < 2 * V; ++e) n[e] = e < V ? c[e] : d[e - V];
                            qn_scale(dn, n);
                        }
                        float part[2] = {};
#pragma unroll
                        for (int e = 0; e < 2 * V; e += 2) {
                            const float u2[2] = {dn[e], dn[e + 1]}, x2[2] = {x[k][u][e], x[k][u][e + 1]};
                            qn_add(part, u2, x2);
                        }
                        inner += part[0] + part[1];
#pragma unroll
                        for (int e = 0; e < 2 * V; ++e) dy[k][u][e] = dn[e];
                    }
                    for (int o = p.lanes >> 1; o > 0; o >>= 1) inner += __shfl_xor_sync(0xffffffffu, inner, o);
                    const float f = (p.rms ? inner / p.d : inner) * r * r;
                    if (side.y) {
                        T* dst = reinterpret_cast<T*>(side.y) + dense[k];
#pragma unroll
                        for (int u = 0; u < U; ++u) {
                            float out[2 * V], s[2 * V], a[V], b[V];
#pragma unroll
                            for (int e = 0; e < 2 * V; ++e) {
                                out[e] = dy[k][u][e];
                                s[e] = -f;
                            }
                            qn_add(out, x[k][u], s);
#pragma unroll
                            for (int e = 0; e < 2 * V; ++e) s[e] = r;
                            qn_scale(out, s);
#pragma unroll
                            for (int e = 0; e < V; ++e) {
                                a[e] = out[e];
                                b[e] = out[V + e];
                            }
                            if (live[k] && lo[u] >= 0) qn_store<T, V>(dst + lo[u], a);
                            if (live[k] && hi[u] >= 0) qn_store<T, V>(dst + hi[u], b);
                        }
                    }
                }
            }
        }
    }
    if (BACK && p.part) {
        // the rows of a warp hold the same channels: add them up, then the warps, in a fixed order
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int e = 0; e < 2 * V; ++e) {
                float a = acc[u][e];
                for (int o = p.lanes; o < 32; o <<= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
                const int base = e < V ? lo[u] : hi[u];
                if (lane < p.lanes && base >= 0) wsum[warp * p.d + base + (e < V ? e : e - V)] = a;
            }
        start_next();
        __syncthreads();
        for (int i = tid; i < p.d; i += QN_THREADS) {
            float a = 0.f;
            for (int wp = 0; wp < QN_THREADS / 32; ++wp) a += wsum[wp * p.d + i];
            p.part[((long long)blockIdx.y * p.blocks + blockIdx.x) * p.d + i] = a;
        }
    }
}

// dwq, dwk: the CTAs' sums added in a fixed order, in float64. A CTA takes 32 channels of one of
// the two, a warp every 32nd sum of them.
__global__ void __launch_bounds__(QN_SUM_THREADS) qk_norm_weight_kernel(const float* part, int blocks, int d, float* dwq, float* dwk)
{
    __shared__ double sum[QN_SUM_THREADS / 32][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, i = blockIdx.x * 32 + lane;
    wait_previous();
    float* dst = blockIdx.y ? dwk : dwq;
    double a = 0.0;
    if (i < d && dst) {
#pragma unroll 4
        for (int b = warp; b < blocks; b += QN_SUM_THREADS / 32) a += (double)part[((long long)blockIdx.y * blocks + b) * d + i];
    }
    sum[warp][lane] = a;
    __syncthreads();
    if (warp == 0 && i < d && dst) {
        for (int w = 1; w < QN_SUM_THREADS / 32; ++w) a += sum[w][lane];
        dst[i] = (float)a;
    }
}

}  // namespace vscan
