// Gated delta rule: device code of the chunked forward and backward passes and
// of the single-token step.
//
// Per value head, with log decay g and write strength beta,
//
//   S_t = e^{g_t} S_{t-1} + beta_t k_t (v_t - e^{g_t} S_{t-1}^T k_t)^T,   y_t = scale S_t^T q_t.
//
// Inside a chunk of 64 steps with entering state S0 and G the running sum of g,
// substituting the recurrence into itself gives
//
//   (I + L) W = X,   L_ij = beta_i e^{G_i - G_j} k_i.k_j (j < i),   X_i = beta_i (v_i - e^{G_i} S0^T k_i)
//   y_i = scale e^{G_i} S0^T q_i + sum_{j<=i} P_ij w_j,             P_ij = scale e^{G_i - G_j} q_i.k_j
//   S_C = e^{G_C} S0 + sum_j e^{G_C - G_j} k_j w_j^T
//
// so a chunk is matrix products plus the inverse T = (I + L)^-1 of a 64 x 64
// unit lower triangle. delta_prep_kernel computes T, P and the decays of every
// chunk in parallel; delta_scan_kernel walks the chunks of one head in order
// and holds the state in registers; delta_rscan_kernel walks them backwards for
// the gradients; delta_grad_kernel turns both walks into dq, dk, da, db chunk
// by chunk in parallel.
//
// Precision. Products run on the bf16 tensor-core path with float32
// accumulation. A bf16 input is exact there; every float32 operand (the state,
// W, T, P) is split into three bf16 terms of 8 bits each (x = x0 + x1 + x2) and
// the products of total order up to 2 are summed, so that states and gradients
// keep float32 accuracy: one cut term alone would leave up to 2^-7 and two 2^-15 in a
// carried state. The one product whose result leaves in bf16 at once, W P in y, has two
// terms of each, rounded: 2^-17 of each operand, and 2^-16 for the product of both second
// terms that is left out, so at most 2^-15 of sum_j |P_ij w_j| before the rounding of y,
// which is 2^-8 of y. By the rms it is 4.4e-6 of y, against the rounding's 1.65e-3, and y is as
// far from float64 (to four digits) with three terms. Those cost 206 -> 214 us at 56x56 (16
// images, 3 heads of 64 x 64), 156 -> 167 us for 24 packed sequences and 1390 -> 1480 us at
// 64x64 + CLS (64 images, 6 heads of 128 x 128). The state itself is float32 throughout, in
// registers, and is only ever added to with rounding.
//
// Measured on one B200 (one kernel at a time): 64 images of 4097 tokens, 6 heads of 128 x 128,
// bf16: triangles 545 us, walk 768 us; 16 images of 56x56, 3 heads of 64 x 64: 52 and 150 us; one
// float32 image of 197 tokens, 6 heads of 64 x 64: 13 and 23 us. The backward pass of 16 images of
// 4097 tokens, 6 heads of 128 x 128: triangles 157 us, walk 281 us, reverse walk 336 us, per-chunk
// gradients 828 us.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "vscan_common.cuh"
#include "vscan_params.cuh"
#include "vscan_route.cuh"
#include "vscan_tc.cuh"

namespace vscan {

constexpr int DL_C = 64;          // steps per chunk
// Floats per chunk in the workspace: e^{G_i}, e^{G_C - G_i}, beta_i, {e^{G_C}}, G_i rounded and the rest of it (two
// each), -beta_i e^{G_i}.
constexpr int DL_VECS = 8 * DL_C;  // 2048 bytes, so that the planes behind them keep their alignment
constexpr int DL_PLANE = DL_C * DL_C;

struct DeltaParams {
    RouteGeom g;
    int has_route, dir;
    int batch;        // images, or packed sequences
    int tokens;       // rows per image, or rows of the packed arrays
    int heads_k, heads_v, group;
    int dk, dv;
    const int* offsets;  // [batch + 1] or null
    int chunks;          // chunks per image (no offsets)
    long long slots;     // chunk slots in the workspace
    int tplanes;         // bf16 planes of P in the workspace (T always has 3)
    const void *q, *k, *v, *a, *b;
    const float *A, *bias;
    const float* s_in;
    float* s_out;
    void* y;
    float scale, beta_scale;
    long long q_tok, q_img, k_tok, k_img, v_tok, v_img, a_tok, a_img, b_tok, b_img, y_tok, y_img;
    // workspace, indexed by slot * heads_v + head
    unsigned char* wrec; // records: DL_VECS floats, three planes of T, tplanes planes of P, in float32 also three
                         // planes each of K and Q; each plane [64][64] the image of a swizzled tile, so that a walk
                         // copies a record as it is
    float* wL;           // [..][64][64]: e^{G_i - G_j} k_i.k_j below the diagonal (backward, else null)
    float* wS;           // [..][DKP][dv]: state entering the chunk (backward)
    float* wW;           // [..][64][dv]: W of the chunk (backward)
    // backward
    const void* dy;      // like y
    const float* ds_in;  // gradient of the final state or null
    float* ds_out;       // gradient of the initial state or null
    float* wdS;          // [..][DKP][dv]: gradient of the state leaving the chunk
    float* wdX;          // [..][64][dv]: gradient of X
    float* wpart;        // [..][2]: per-chunk sums for dA and dbias
    float *wdq, *wdk;    // [images][tokens][heads_v][dk]: per value head where key heads are shared, else null
    void *dq, *dkey, *dvalue, *da, *db;  // dense, in the I/O type
    float *dA, *dbias;
    int* status;  // device word or null
};

// The steps of one image or packed sequence: its length, its first workspace
// slot, and the token row of a step. Offsets come from device memory: they are
// clamped into the arrays so that no value of theirs leads outside.
struct DeltaSeq {
    int len, first;
    long long slot;
};

__device__ __forceinline__ DeltaSeq delta_seq(const DeltaParams& p, int b)
{
    DeltaSeq s;
    if (p.offsets) {
        const int o0 = min(max(p.offsets[b], 0), p.tokens);
        const int o1 = min(max(p.offsets[b + 1], o0), p.tokens);
        s.len = o1 - o0;
        s.first = o0;
        s.slot = o0 / DL_C + b;
    } else {
        s.len = p.has_route ? p.g.L : p.tokens;
        s.first = 0;
        s.slot = (long long)b * p.chunks;
    }
    return s;
}

// Row of step t in the token arrays of its image; -1 for a padding step of the
// atrous route, whose token is zero, and behind the sequence's end.
__device__ __forceinline__ int delta_row(const DeltaParams& p, const DeltaSeq& s, int t)
{
    if (t >= s.len) return -1;
    if (!p.has_route) return s.first + t;
    return route_token_any(p.g, p.dir, t);
}

__device__ __forceinline__ long long delta_img(const DeltaParams& p, int b) { return p.offsets ? 0 : b; }

// Parts of a record.
template <typename T, int DKP>
__host__ __device__ constexpr size_t delta_record_bytes(int tplanes)
{
    return DL_VECS * 4 + (size_t)(3 + tplanes + (sizeof(T) == 4 ? 6 * (DKP / 64) : 0)) * DL_PLANE * 2;
}
template <typename T, int DKP>
__device__ __forceinline__ float* record_vec(const DeltaParams& p, size_t rec)
{
    return reinterpret_cast<float*>(p.wrec + rec * delta_record_bytes<T, DKP>(p.tplanes));
}
template <typename T, int DKP>
__device__ __forceinline__ __nv_bfloat16* record_P(const DeltaParams& p, size_t rec)
{
    return reinterpret_cast<__nv_bfloat16*>(record_vec<T, DKP>(p, rec) + DL_VECS) + 3 * DL_PLANE;
}

// ---- tensor-core fragments ------------------------------------------------------
// m16n8k16: lane (g, t) = (lane / 4, lane % 4) holds of A the pairs of columns
// 2t and 2t + 8 of rows g and g + 8; of B the pairs of rows 2t and 2t + 8 of
// column g; of C columns 2t, 2t + 1 of rows g and g + 8. (Only the two small
// products per chunk of delta_prep_kernel use these; the others run on tcgen05,
// which has eight times the rate.)
struct Frag4 { uint32_t x[4]; };

__device__ __forceinline__ void mma_bf16(float (&c)[4], const Frag4& a, uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a.x[0]), "r"(a.x[1]), "r"(a.x[2]), "r"(a.x[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ Frag4 ldsm4(const __nv_bfloat16* p)
{
    Frag4 f;
    const unsigned s = static_cast<unsigned>(__cvta_generic_to_shared(p));
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];\n"
                 : "=r"(f.x[0]), "=r"(f.x[1]), "=r"(f.x[2]), "=r"(f.x[3]) : "r"(s));
    return f;
}

// A fragment of the 16 x 16 block at (m0, k0) of a row-major [m][k] tile.
__device__ __forceinline__ Frag4 load_a(const __nv_bfloat16* t, int pitch, int m0, int k0, int lane)
{
    return ldsm4(t + (m0 + (lane & 7) + ((lane >> 3) & 1) * 8) * pitch + k0 + (lane >> 4) * 8);
}
// B fragments of two neighbouring 8-wide column tiles (x[0..1] at n0, x[2..3] at
// n0 + 8) of a [n][k] tile.
__device__ __forceinline__ Frag4 load_b(const __nv_bfloat16* t, int pitch, int n0, int k0, int lane)
{
    return ldsm4(t + (n0 + (lane & 7) + (lane >> 4) * 8) * pitch + k0 + ((lane >> 3) & 1) * 8);
}

// x = h + r for a pair: h the upper 16 bits (packed, x in the low half), r exact. Cut instead of
// rounded, three terms hold the 24 bits of a float32 exactly, and a byte permutation takes the
// place of a conversion (56x56 cross-scan walk, batch 16: 197 us rounding, 185 cutting).
__device__ __forceinline__ uint32_t split_bf16(float& x, float& y)
{
    const uint32_t a = __float_as_uint(x), b = __float_as_uint(y);
    // a packed subtraction, as a product with -1: a packed sum has no sign of its own for an operand
    const float2 r = __ffma2_rn(make_float2(__uint_as_float(a & 0xffff0000u), __uint_as_float(b & 0xffff0000u)),
                                make_float2(-1.f, -1.f), make_float2(x, y));
    x = r.x;
    y = r.y;
    return __byte_perm(a, b, 0x7632);
}

// The rounded pair, for fewer than three terms.
__device__ __forceinline__ uint32_t round_bf16(float x, float y)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// c += sum over terms a[x] b[y], x + y <= ORD, b from NB planes of one pair of column tiles.
// The tensor core truncates what it adds to its accumulator. Small terms go first, so that
// they truncate little; six products in a row would still cut six times into the running sum,
// so those are summed on their own and added with rounding (relative error of the float32
// gradients of 777 steps, dk 48, dv 80: 1.4e-6 in one sum, 2e-7 apart).
template <int NA, int NB, int ORD = 2>
__device__ __forceinline__ void mma_terms(float (&c0)[4], float (&c1)[4], const Frag4 (&a)[NA], const Frag4 (&b)[NB])
{
    constexpr bool apart = NA == 3 && NB == 3 && ORD == 2;
    float t0[4] = {}, t1[4] = {};
#pragma unroll
    for (int o = ORD; o >= 0; --o)
#pragma unroll
        for (int y = 0; y < NB; ++y) {
            const int x = o - y;
            if (x >= 0 && x < NA) {
                mma_bf16(apart ? t0 : c0, a[x], b[y].x[0], b[y].x[1]);
                mma_bf16(apart ? t1 : c1, a[x], b[y].x[2], b[y].x[3]);
            }
        }
    if (apart) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            c0[i] += t0[i];
            c1[i] += t1[i];
        }
    }
}

// e^{G_i - G_j} from running sums held as a rounded value and the rest of it. FAST: by ex2, good
// to 2^-22, for what leaves in bf16.
template <bool FAST>
__device__ __forceinline__ float decay_between(float2 gi, float2 gj)
{
    const float d = (gi.x - gj.x) + (gi.y - gj.y);
    return FAST ? fast_exp2(d * LOG2E) : expf(d);
}

// ---- tiles ------------------------------------------------------------------------
template <typename T> struct DeltaIo;
template <> struct DeltaIo<__nv_bfloat16> { static constexpr int planes = 1; };
template <> struct DeltaIo<float> { static constexpr int planes = 3; };

// Log decay of a step. It is clamped at -120 (e^-120 is 0 in float32 with or
// without the clamp), which keeps differences of its sums free of inf - inf.
__device__ __forceinline__ float delta_softplus(float x) { return fmaxf(x, 0.f) + log1pf(expf(-fabsf(x))); }
__device__ __forceinline__ float delta_decay(float A, float x)
{
    const float g = A * delta_softplus(x);
    return g < -120.f ? -120.f : g;
}
__device__ __forceinline__ float delta_sigmoid(float x) { return 1.f / (1.f + expf(-x)); }

// e^x of a difference of running sums held in float64: the float32 rounding of a
// far-away sum would be an error of the exponent.
__device__ __forceinline__ float exp_diff(double d)
{
    const float h = (float)d;
    const float e = expf(h);
    return e + e * (float)(d - (double)h);
}

// Element (i, j) of a 64 x 64 plane of the workspace: the image of a swizzled tile.
__device__ __forceinline__ int plane_at(int i, int j) { return tc_swizzle(i, j >> 3) / 2 + (j & 7); }

// THREADS threads move the 64 rows of VECS 16-byte pieces of a chunk; a thread keeps to one piece
// and to every (THREADS / VECS)-th row, four rows at a time: their token rows are read before the
// first of the four copies, which those reads could not pass. Not unrolled further: in the walks
// this code runs once a chunk between the computing warps' long one, and unrolled it spent its
// time on instruction-cache misses (70 to 140 cycles a piece).
template <int VECS, int THREADS, typename F>
__device__ __forceinline__ void copy_rows(const int* rows, int tid, F copy)
{
    constexpr int step = THREADS / VECS, B = 4;
    if (THREADS % VECS != 0 && tid >= step * VECS) return;
#pragma unroll 1
    for (int r = tid / VECS; r < DL_C; r += B * step) {
        int row[B];
#pragma unroll
        for (int i = 0; i < B; ++i) row[i] = rows[min(r + i * step, DL_C - 1)];
#pragma unroll
        for (int i = 0; i < B; ++i)
            if (r + i * step < DL_C) copy(r + i * step, row[i]);
    }
}

// ---- per-chunk triangle: T, P, decays -----------------------------------------------
// One CTA of eight warps per chunk and value head, bound by the latency of its chain, so
// the chain is kept short and several CTAs share an SM: warps 0-3 form K K^T, L and T,
// warps 4-7 Q K^T and P at the same time, row block by row block of 16. T comes from
// the inverses of the four diagonal 16 x 16 blocks (one column a lane, each known
// entry subtracted from all later ones at once), merged twice:
//   [A 0; C B]^-1 = [A^-1 0; -B^-1 C A^-1 B^-1].
// L and T's blocks lie transposed as well, so that four rows of a left factor are one
// 16-byte read. The decays and T are assembled in shared memory, in the walks' swizzled
// layout, and leave in one bulk copy; P goes out directly. What shared memory holds is
// packed so that four CTAs share an SM (bf16): L^T's rows begin at their diagonal block,
// the part of T^T that nothing reads has no place, and the merges' first factors lie in
// T's own rows. Blocks above the diagonal hold nothing, and nothing reads them.
constexpr int DP_THREADS = 256;
constexpr int DP_TP = 36;  // row pitch of the 32 x 32 blocks of T
// L^T: rows of block b hold the steps from 16 b on.
__host__ __device__ constexpr int prep_lt_pitch(int b) { return 68 - 16 * b; }
__host__ __device__ constexpr int prep_lt(int j)  // L_ij at prep_lt(j) + i
{
    return (j >> 4) * (1088 - 128 * ((j >> 4) - 1)) + (j & 15) * prep_lt_pitch(j >> 4) - (j & ~15);
}
static_assert(prep_lt(16) + 16 == prep_lt(15) + 68 && prep_lt(48) + 48 == prep_lt(47) + 68, "rows follow one another");

template <typename T, int DKP>
struct PrepShape {
    static constexpr int NP = DeltaIo<T>::planes;
    static constexpr int pitch = DKP + 8;  // an odd multiple of 16 bytes
    static constexpr int plane = DL_C * pitch;
    static constexpr int tiles = 2 * NP * plane * 2;                      // bytes of K and Q, until the products are done:
    static constexpr int image = DL_VECS * 4 + 3 * DL_PLANE * 2;          // then decays and T's planes,
    static constexpr int later = image + DL_C * DP_TP * 4;                // and T by rows
    static constexpr int front = (tiles > later ? tiles : later);
    static constexpr int oL = front, oTt = oL + (prep_lt(63) + 68) * 4, oGates = oTt + (DL_C - 16) * DP_TP * 4;
    static constexpr size_t smem = oGates + DL_C * (8 + 4 * 7);
};

// A value's three bf16 terms, one in each plane of T's image; `at` is its plane_at.
__device__ __forceinline__ void image_put(__nv_bfloat16* img, int at, float x)
{
    uint16_t* o = reinterpret_cast<uint16_t*>(img) + at;
#pragma unroll
    for (int n = 0; n < 3; ++n) {
        const uint32_t u = __float_as_uint(x);
        o[n * DL_PLANE] = (uint16_t)(u >> 16);
        x -= __uint_as_float(u & 0xffff0000u);
    }
}

// The rows of K or Q to padded rows in bf16 planes, by all warps but the first; float32 ones, split,
// to the record as well.
template <int DKP>
__device__ __forceinline__ void prep_load(__nv_bfloat16* dst, unsigned char*, const __nv_bfloat16* src, long long tok,
                                          const int* rows, int have, int tid)
{
    constexpr int vecs = DKP / 8;
    const int c = tid % vecs * 8;
    const __nv_bfloat16* at = c < have ? src + c : src;
    copy_rows<vecs, DP_THREADS - 32>(rows, tid, [&](int r, int row) {
        const bool ok = c < have && row >= 0;
        copy16(dst + r * (DKP + 8) + c, at + (ok ? row * tok : 0), ok);
    });
}
template <int DKP>
__device__ __forceinline__ void prep_load(__nv_bfloat16* dst, unsigned char* image, const float* src, long long tok,
                                          const int* rows, int have, int tid)
{
    constexpr int vecs = DKP / 8;
    const int c = tid % vecs * 8;
    copy_rows<vecs, DP_THREADS - 32>(rows, tid, [&](int r, int row) {
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f), z = x;
        if (row >= 0 && c < have) x = __ldg(reinterpret_cast<const float4*>(src + c + row * tok));
        if (row >= 0 && c + 4 < have) z = __ldg(reinterpret_cast<const float4*>(src + c + 4 + row * tok));
#pragma unroll
        for (int n = 0; n < 3; ++n) {
            uint4 u;
            u.x = split_bf16(x.x, x.y);
            u.y = split_bf16(x.z, x.w);
            u.z = split_bf16(z.x, z.y);
            u.w = split_bf16(z.z, z.w);
            *reinterpret_cast<uint4*>(dst + n * (DL_C * (DKP + 8)) + r * (DKP + 8) + c) = u;
            *reinterpret_cast<uint4*>(image + n * (DKP / 64 * TC_TILE) + tc_swizzle(r, c / 8)) = u;
        }
    });
}

template <typename T, int DKP, int PP>  // PP planes of P
__global__ void __launch_bounds__(DP_THREADS, DeltaIo<T>::planes == 1 ? 4 : 3) delta_prep_kernel(const DeltaParams p)
{
    using Sh = PrepShape<T, DKP>;
    constexpr int NP = Sh::NP, PITCH = Sh::pitch, PLANE = Sh::plane;
    extern __shared__ __align__(128) unsigned char smem[];
    __nv_bfloat16* K = reinterpret_cast<__nv_bfloat16*>(smem);
    __nv_bfloat16* Q = K + NP * PLANE;
    float* vec = reinterpret_cast<float*>(smem);
    __nv_bfloat16* imgT = reinterpret_cast<__nv_bfloat16*>(vec + DL_VECS);
    float* Tr = reinterpret_cast<float*>(smem + Sh::image);                 // T_ij at [i][j mod 32]
    float* Lt = reinterpret_cast<float*>(smem + Sh::oL);                // L_ij at prep_lt(j) + i
    float* Tt = reinterpret_cast<float*>(smem + Sh::oTt) - 16 * DP_TP;  // T_ij at [j][i mod 32], j from 16 on
    float2* G = reinterpret_cast<float2*>(smem + Sh::oGates);           // running sum, rounded and rest
    float* beta = reinterpret_cast<float*>(G + DL_C);
    float *onward = beta + DL_C, *upto = onward + DL_C;                     // [64]; [4][64], row block 0 unused
    int* rows = reinterpret_cast<int*>(upto + 4 * DL_C);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, head = blockIdx.y;
    const int group = warp >> 2, m0 = (warp & 3) * 16;
    start_next();

    // the sequence of this slot
    int b;
    if (p.offsets) {
        int lo = 0, hi = p.batch;  // last b whose first slot is <= blockIdx.x
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (delta_seq(p, mid).slot <= (long long)blockIdx.x) lo = mid; else hi = mid;
        }
        b = lo;
    } else {
        b = blockIdx.x / p.chunks;
    }
    const DeltaSeq s = delta_seq(p, b);
    const long long c = (long long)blockIdx.x - s.slot;
    if (c < 0 || c * DL_C >= s.len) return;
    const int t0 = (int)c * DL_C;
    const long long img = delta_img(p, b);
    const int hk = head / p.group;
    const size_t rec = (size_t)blockIdx.x * p.heads_v + head;

    unsigned char* out = p.wrec + rec * delta_record_bytes<T, DKP>(PP);
    __nv_bfloat16* imgP = reinterpret_cast<__nv_bfloat16*>(out + Sh::image);
    double g[2];
    if (warp == 0) {  // running sum of the log decay: two steps a lane, then a scan over the lanes
        const float A = p.A[head], bias = p.bias ? p.bias[head] : 0.f;
        float a[2], bb[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int row = delta_row(p, s, t0 + 2 * lane + i);
            a[i] = row >= 0 ? to_float(reinterpret_cast<const T*>(p.a)[img * p.a_img + row * p.a_tok + head]) : 0.f;
            bb[i] = row >= 0 ? to_float(reinterpret_cast<const T*>(p.b)[img * p.b_img + row * p.b_tok + head]) : 0.f;
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const bool in = t0 + 2 * lane + i < s.len;
            g[i] = in ? (double)delta_decay(A, a[i] + bias) : 0.0;
            beta[2 * lane + i] = in ? p.beta_scale * delta_sigmoid(bb[i]) : 0.f;
        }
        double sum = g[0] + g[1];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const double other = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += other;
        }
        g[0] = sum - g[1];
        g[1] = sum;
#pragma unroll
        for (int i = 0; i < 2; ++i) G[2 * lane + i] = make_float2((float)g[i], (float)(g[i] - (double)(float)g[i]));
    } else {  // the other warps fetch K and Q
        const int ht = tid - 32;
        if (ht < DL_C) rows[ht] = delta_row(p, s, t0 + ht);
        bar_sync(3, DP_THREADS - 32);
        unsigned char* kq = out + DL_VECS * 4 + (3 + PP) * TC_TILE;
        prep_load<DKP>(K, kq, reinterpret_cast<const T*>(p.k) + img * p.k_img + (long long)hk * p.dk, p.k_tok, rows, p.dk, ht);
        prep_load<DKP>(Q, kq + 3 * (DKP / 64) * TC_TILE, reinterpret_cast<const T*>(p.q) + img * p.q_img + (long long)hk * p.dk, p.q_tok, rows, p.dk, ht);
        cp_async_commit();
        cp_async_wait<0>();
    }
    __syncthreads();
    // Decays between blocks of 16 steps, in two factors of at most 1: from step j to the first of
    // row block B, and on from there to step i. Inside a block each pair has its own.
    if (tid < DL_C) {
        const float2 x = G[tid], r = G[tid & ~15];
        onward[tid] = expf((x.x - r.x) + (x.y - r.y));
    } else {
        const int bi = tid >> 6, j = tid & 63;  // 1 .. 3
        const float2 x = G[j], r = G[bi * 16];
        if (j < bi * 16) upto[bi * DL_C + j] = expf((r.x - x.x) + (r.y - x.y));
    }

    // K K^T (warps 0-3) and Q K^T, the lower triangle of a row block
    float acc[8][4] = {};
    {
        const __nv_bfloat16* left = group ? Q : K;
#pragma unroll 2
        for (int k0 = 0; k0 < DKP; k0 += 16) {
            Frag4 a[NP];
#pragma unroll
            for (int n = 0; n < NP; ++n) a[n] = load_a(left + n * PLANE, PITCH, m0, k0, lane);
#pragma unroll
            for (int nt = 0; nt < 8; nt += 2) {
                if (nt * 8 <= m0) {
                    Frag4 bk[NP];
#pragma unroll
                    for (int n = 0; n < NP; ++n) bk[n] = load_b(K + n * PLANE, PITCH, nt * 8, k0, lane);
                    mma_terms<NP, NP>(acc[nt], acc[nt + 1], a, bk);
                }
            }
        }
    }
    __syncthreads();  // K and Q are read: their place is the record's now
    {
        const int r0 = m0 + (lane >> 2), tc = (lane & 3) * 2;
        const float beta0 = beta[r0], beta1 = beta[r0 + 8];
        // one pair of columns of one row, decayed: to P's planes, or to L
        auto put = [&](int i, int half, int nt, float v0, float v1) {
            const int j = nt * 8 + tc;
            if (group) {
                v0 *= p.scale;
                v1 *= p.scale;
                __nv_bfloat16* o = imgP + i * 64 + ((nt ^ (lane >> 2)) << 3) + tc;  // plane_at(i, j)
                if (PP == 2) {  // rounded, both: what the product of the second terms would add is left out
                    const uint32_t u = round_bf16(v0, v1);
                    *reinterpret_cast<uint32_t*>(o) = u;
                    *reinterpret_cast<uint32_t*>(o + DL_PLANE) =
                        round_bf16(v0 - __uint_as_float(u << 16), v1 - __uint_as_float(u & 0xffff0000u));
                } else {
#pragma unroll
                    for (int n = 0; n < 3; ++n) *reinterpret_cast<uint32_t*>(o + n * DL_PLANE) = split_bf16(v0, v1);
                }
            } else {
                if (PP == 3 && p.wL) *reinterpret_cast<float2*>(p.wL + rec * DL_PLANE + i * DL_C + j) = make_float2(v0, v1);
                const float be = half ? beta1 : beta0;
                Lt[prep_lt(j) + i] = be * v0;
                Lt[prep_lt(j + 1) + i] = be * v1;
            }
        };
        const float f0 = onward[r0], f1 = onward[r0 + 8];
        float diag[2][4];  // the block on the diagonal, moved to fixed registers: its code is there once
#pragma unroll
        for (int nt = 0; nt < 8; nt += 2) {
            if (nt * 8 == m0) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    diag[0][e] = acc[nt][e];
                    diag[1][e] = acc[nt + 1][e];
                }
            } else if (nt * 8 < m0) {
#pragma unroll
                for (int n = nt; n < nt + 2; ++n) {
                    const float2 h = *reinterpret_cast<const float2*>(upto + (m0 / 16) * DL_C + n * 8 + tc);
                    put(r0, 0, n, f0 * h.x * acc[n][0], f0 * h.y * acc[n][1]);
                    put(r0 + 8, 1, n, f1 * h.x * acc[n][2], f1 * h.y * acc[n][3]);
                }
            }
        }
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            const int j = m0 + n * 8 + tc;
            const float2 gj0 = G[j], gj1 = G[j + 1];
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int i = r0 + half * 8;
                const float2 gi = G[i];
                // selected, not multiplied by zero: what lies above the diagonal is not looked at
                const float d0 = decay_between<false>(gi, gj0), d1 = decay_between<false>(gi, gj1);
                put(i, half, m0 / 8 + n, j < i + group ? d0 * diag[n][half * 2] : 0.f,
                    j + 1 < i + group ? d1 * diag[n][half * 2 + 1] : 0.f);
            }
        }
    }
    if (group) return;
    if (warp == 0) {
        const double last = __shfl_sync(0xffffffffu, g[1], 31);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = 2 * lane + i;
            const float e = exp_diff(g[i]);
            vec[r] = e;
            vec[6 * DL_C + r] = -beta[r] * e;
            vec[DL_C + r] = exp_diff(last - g[i]);
            vec[2 * DL_C + r] = beta[r];
        }
        if (lane == 0) vec[3 * DL_C] = exp_diff(last);
        *reinterpret_cast<float4*>(vec + 4 * DL_C + 4 * lane) = *reinterpret_cast<const float4*>(G + 2 * lane);
    }
    bar_sync(1, 128);
    if (lane < 16) {  // inverse of diagonal block m0, column `lane`
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = i == lane ? 1.f : 0.f;
        const float* L = Lt + prep_lt(m0) + m0;
        const int pitch = prep_lt_pitch(m0 >> 4);
#pragma unroll
        for (int j = 0; j < 15; ++j) {
            float l[16];
#pragma unroll
            for (int q = (j + 1) / 4; q < 4; ++q) *reinterpret_cast<float4*>(l + 4 * q) = *reinterpret_cast<const float4*>(L + j * pitch + 4 * q);
#pragma unroll
            for (int i = j + 1; i < 16; ++i) x[i] -= l[i] * x[j];
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            Tr[(m0 + i) * DP_TP + (m0 & 31) + lane] = x[i];
            if (m0) Tt[(m0 + lane) * DP_TP + (m0 & 31) + i] = x[i];
            image_put(imgT, (m0 + i) * 64 + ((((m0 + lane) >> 3) ^ (i & 7)) << 3) + (lane & 7), x[i]);
        }
    }
    bar_sync(1, 128);
    {  // 16 x 16 blocks below the diagonal of both 32 x 32 ones: four rows of a column a thread
        const int b0 = (tid >> 6) * 32, col = tid & 15, r = (tid >> 4 & 3) * 4;
        float m[4] = {}, o[4] = {};
        float* Mb = Tr + (b0 + 16) * DP_TP;  // where o goes in the end
        const float* L = Lt + prep_lt(b0) + b0 + 16 + r;
        const int pitch = prep_lt_pitch(b0 >> 4);
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            const float4 l = *reinterpret_cast<const float4*>(L + k * pitch);
            const float x = Tr[(b0 + k) * DP_TP + col];
            m[0] += l.x * x; m[1] += l.y * x; m[2] += l.z * x; m[3] += l.w * x;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) Mb[(r + i) * DP_TP + col] = m[i];
        bar_sync(1, 128);
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            const float4 l = *reinterpret_cast<const float4*>(Tt + (b0 + 16 + k) * DP_TP + 16 + r);
            const float x = Mb[k * DP_TP + col];
            o[0] -= l.x * x; o[1] -= l.y * x; o[2] -= l.z * x; o[3] -= l.w * x;
        }
        bar_sync(1, 128);
#pragma unroll
        for (int i = 0; i < 4; ++i) image_put(imgT, plane_at(b0 + 16 + r + i, b0 + col), o[i]);
        // The next products read the first block by rows and the second one by columns, above
        // the diagonal too.
        if (b0) {
            *reinterpret_cast<float4*>(Tt + (32 + col) * DP_TP + 16 + r) = make_float4(o[0], o[1], o[2], o[3]);
            *reinterpret_cast<float4*>(Tt + (48 + col) * DP_TP + r) = make_float4(0.f, 0.f, 0.f, 0.f);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                Tr[(16 + r + i) * DP_TP + col] = o[i];
                Tr[(r + i) * DP_TP + 16 + col] = 0.f;
            }
        }
    }
    bar_sync(1, 128);
    {  // the 32 x 32 block below the diagonal: four rows of two columns a thread
        const int col = (tid & 15) * 2, r = (tid >> 4) * 4;
        float m[4][2] = {}, o[4][2] = {};
        float* M = Tr + 32 * DP_TP;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll 8
            for (int k = 0; k < 16; ++k) {
                const float4 l = *reinterpret_cast<const float4*>(Lt + prep_lt(h * 16) + k * prep_lt_pitch(h) + 32 + r);
                const float2 x = *reinterpret_cast<const float2*>(Tr + (h * 16 + k) * DP_TP + col);
                m[0][0] += l.x * x.x; m[1][0] += l.y * x.x; m[2][0] += l.z * x.x; m[3][0] += l.w * x.x;
                m[0][1] += l.x * x.y; m[1][1] += l.y * x.y; m[2][1] += l.z * x.y; m[3][1] += l.w * x.y;
            }
#pragma unroll
        for (int i = 0; i < 4; ++i) *reinterpret_cast<float2*>(M + (r + i) * DP_TP + col) = make_float2(m[i][0], m[i][1]);
        bar_sync(1, 128);
#pragma unroll 8
        for (int k = 0; k < 32; ++k) {
            const float4 l = *reinterpret_cast<const float4*>(Tt + (32 + k) * DP_TP + r);
            const float2 x = *reinterpret_cast<const float2*>(M + k * DP_TP + col);
            o[0][0] -= l.x * x.x; o[1][0] -= l.y * x.x; o[2][0] -= l.z * x.x; o[3][0] -= l.w * x.x;
            o[0][1] -= l.x * x.y; o[1][1] -= l.y * x.y; o[2][1] -= l.z * x.y; o[3][1] -= l.w * x.y;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int n = 0; n < 3; ++n)
                *reinterpret_cast<uint32_t*>(imgT + n * DL_PLANE + plane_at(32 + r + i, col)) = split_bf16(o[i][0], o[i][1]);
    }
    tc_fence_smem();
    bar_sync(1, 128);
    if (tid == 0) {
        bulk_out(out, vec, Sh::image);
        bulk_out_read();
    }
}

// ---- the walk over the chunks -----------------------------------------------------
// One CTA per image (sequence), value head and slice of 128 value channels. The
// products are formed transposed, with the value channel as the row of the 128-row
// tensor-core tile, so that a thread holds half a row of everything in registers: of
// S^T[128][DKP] (float32, for the whole walk), and in turn of (K S)^T, X^T, W^T and
// y^T[128][64]. Between two products it rescales its values, splits them into bf16
// terms and stores them to tensor memory as the next left operand; no value crosses
// threads. Per chunk:
//
//   1. KS = S K^T, QS = S Q^T                 B = K, Q    (K-major)
//   2. X = beta (V - e^G KS);  W = X T^T      B = T       (K-major)
//   3. dS = (e^{G_C - G} W) K, O = W P^T      B = K (MN-major: the same tile), P (K-major)
//   4. S = e^{G_C} S + dS (float32, in registers);  y = scale e^G QS + O
//
// The chain KS -> W -> dS -> S bounds the walk, so everything else is off it: eight
// warps compute, one thread issues the products (the ones of the chain first), three
// warps copy the next chunks' tiles in, and a computing thread never waits for
// another one, only for products. y of a chunk is finished while the next one waits for W. T and P are lower triangles: slice ks of their summed
// index touches the columns from 16 ks on only.
// Tensor-memory columns: S terms (over them dS, once step 1 is done), KS (W, then W's
// terms for O), QS, X's terms (then those of e^{G_C - G} W), O.
constexpr int DW_COMPUTE = 256, DW_HELP = 96, DW_THREADS = 384;  // warps 0-7, 9-11, all (warp 8 issues)
// Registers a thread: 384 x 168 at launch, split 200 / 96: 256 x 200 + 128 x 96 = 63488 of 64512.
constexpr int DW_REGS_COMPUTE = 200, DW_REGS_HELP = 96;

constexpr int WALK_FRONT = 2048;  // bytes in front of the stages, of WalkShared

template <typename T, int DKP>
struct WalkShape {
    static constexpr int NP = DeltaIo<T>::planes;
    static constexpr int PP = NP == 1 ? 2 : 3;   // terms of P and W in O: a bf16 y needs two
    static constexpr int STAGES = NP == 1 || DKP == 64 ? 2 : 1;
    static constexpr int KB = DKP / 64;          // 64-wide tiles of K
    static constexpr int plane = KB * TC_TILE;   // bytes
    static constexpr int vpitch = 128 + 16 / (int)sizeof(T);
    // a stage: the chunk's record (decays, T, P), K, Q, and V where it is bf16. Float32 K and Q come
    // split, as a part of the record; float32 values go straight to registers and back
    static constexpr int oT = DL_VECS * 4, oP = oT + 3 * TC_TILE;
    static __host__ __device__ constexpr int oK(int pplanes) { return oP + pplanes * TC_TILE; }
    static __host__ __device__ constexpr int oQ(int pplanes) { return oK(pplanes) + NP * plane; }
    static __host__ __device__ constexpr int oV(int pplanes) { return oQ(pplanes) + NP * plane; }
    static __host__ __device__ constexpr int stage(int pplanes)
    {
        return (oV(pplanes) + (NP == 1 ? DL_C * vpitch * (int)sizeof(T) : 0) + 1023) / 1024 * 1024;
    }
    static constexpr int out = NP == 1 ? DL_C * vpitch * (int)sizeof(T) : 0;  // behind the stages: y's (dV's) way out
    // at least half of the SM's shared memory: one CTA an SM, which owns all tensor memory
    static __host__ __device__ constexpr size_t smem(int pplanes)
    {
        const size_t n = 1024 + WALK_FRONT + (size_t)STAGES * stage(pplanes) + out;
        return n < 120 * 1024 ? 120 * 1024 : n;
    }
    // tensor-memory columns of one term of half a row of S (DKP / 2 values)
    static constexpr int SC = DKP / 4;
};

// The 64 rows of a token array into swizzled shared memory in bf16 planes, zero where there is
// no token and from column `have` on.
template <int COLS>
__device__ __forceinline__ void walk_load(unsigned char* dst, const __nv_bfloat16* src, long long tok, const int* rows, int have,
                                          int tid)
{
    constexpr int vecs = COLS / 8;
    const int c = tid % vecs;
    const bool in = c * 8 < have;
    const __nv_bfloat16* at = in ? src + c * 8 : src;
    copy_rows<vecs, DW_HELP>(rows, tid, [&](int r, int row) {
        const bool ok = in && row >= 0;
        copy16(dst + tc_swizzle(r, c), at + (ok ? row * tok : 0), ok);
    });
}
// The rows of a value-shaped token array (up to 128 channels of them), unsplit, in and out. A
// bulk copy a row would be fewer instructions, but they issue one after the other: 64 of them
// took 2600 cycles.
template <typename T>
__device__ __forceinline__ void walk_load_values(T* dst, int pitch, const T* src, long long tok, const int* rows, int have, int tid)
{
    constexpr int V = 16 / sizeof(T), vecs = 128 / V;
    const int c = tid % vecs * V;
    const bool in = c < have;
    const T* at = in ? src + c : src;
    copy_rows<vecs, DW_HELP>(rows, tid, [&](int r, int row) {
        const bool ok = in && row >= 0;
        copy16(dst + r * pitch + c, at + (ok ? row * tok : 0), ok);
    });
}
// 32 steps of a float32 value channel, neighbouring lanes neighbouring channels.
__device__ __forceinline__ void walk_fetch(float (&x)[32], const float* src, long long tok, const int* rows, bool live)
{
#pragma unroll
    for (int i = 0; i < 32; i += 4) {
        const int4 r = *reinterpret_cast<const int4*>(rows + i);
        x[i] = live && r.x >= 0 ? __ldg(src + r.x * tok) : 0.f;
        x[i + 1] = live && r.y >= 0 ? __ldg(src + r.y * tok) : 0.f;
        x[i + 2] = live && r.z >= 0 ? __ldg(src + r.z * tok) : 0.f;
        x[i + 3] = live && r.w >= 0 ? __ldg(src + r.w * tok) : 0.f;
    }
}
__device__ __forceinline__ void walk_put(float* dst, long long tok, const int* rows, bool live, const float (&x)[32])
{
#pragma unroll
    for (int i = 0; i < 32; i += 4) {
        const int4 r = *reinterpret_cast<const int4*>(rows + i);
        if (live && r.x >= 0) dst[r.x * tok] = x[i];
        if (live && r.y >= 0) dst[r.y * tok] = x[i + 1];
        if (live && r.z >= 0) dst[r.z * tok] = x[i + 2];
        if (live && r.w >= 0) dst[r.w * tok] = x[i + 3];
    }
}

// 32 steps of a warp's 32 value channels to their token rows, through the warp's own corner of the
// stage's value tile (whose values it alone has read): one value at a time from the registers,
// 32 stores a lane took 2100 cycles a chunk, this takes 500. `mine` is this thread's value of
// step 0 in the tile, `dst` the channel of lane 0.
__device__ __forceinline__ void stage_two(float* p, int pitch, float x, float y)
{
    p[0] = x;
    p[pitch] = y;
}
__device__ __forceinline__ void stage_two(__nv_bfloat16* p, int pitch, float x, float y)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);  // one conversion for both
    p[0] = __low2bfloat16(h);
    p[pitch] = __high2bfloat16(h);
}
template <typename T, int N>
__device__ __forceinline__ void walk_stage(T* mine, int pitch, const float (&x)[N])
{
#pragma unroll
    for (int i = 0; i < N; i += 2) stage_two(mine + i * pitch, pitch, x[i], x[i + 1]);
}
template <int N = 32, typename T>
__device__ __forceinline__ void walk_flush(T* dst, long long tok, const int* rows, const T* mine, int pitch, int have, int lane)
{
    __syncwarp();
    constexpr int V = 16 / sizeof(T), vecs = 32 / V, per = 32 / vecs;  // pieces of a row, rows at a time
    const int c = lane % vecs * V;
    const T* src = mine - lane + c;
    if (c < have)
#pragma unroll
        for (int i = 0; i < N; i += per) {
            const int r = i + lane / vecs, row = rows[r];
            if (row >= 0) *reinterpret_cast<uint4*>(dst + row * tok + c) = *reinterpret_cast<const uint4*>(src + r * pitch);
        }
    __syncwarp();
}
template <typename T, int N>
__device__ __forceinline__ void walk_store(T* dst, long long tok, const int* rows, T* mine, int pitch, int have, int lane,
                                           const float (&x)[N])
{
    walk_stage(mine, pitch, x);
    walk_flush<N>(dst, tok, rows, mine, pitch, have, lane);
}

// NT bf16 terms of 32 values of a row, term n in the 16 columns from addr + n * step on. Three
// are cut (exact); one or two are rounded (2^-17 for two, cut ones would leave 2^-15), unless
// CUT says that more follow elsewhere.
template <int NT, bool CUT = NT == 3>
__device__ __forceinline__ void put_terms(uint32_t addr, int step, float (&v)[32])
{
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        uint32_t u[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            if (CUT) {
                u[i] = split_bf16(v[2 * i], v[2 * i + 1]);
            } else {
                u[i] = round_bf16(v[2 * i], v[2 * i + 1]);
                v[2 * i] -= __uint_as_float(u[i] << 16);
                v[2 * i + 1] -= __uint_as_float(u[i] & 0xffff0000u);
            }
        }
        tc_st16(addr + n * step, u);
    }
}

// What the first two of three terms hold.
__device__ __forceinline__ float upper_terms(float x)
{
    const float h = __uint_as_float(__float_as_uint(x) & 0xffff0000u);
    return h + __uint_as_float(__float_as_uint(x - h) & 0xffff0000u);
}

// x * s and x * s + z, two values at a time; s in shared memory.
__device__ __forceinline__ void scale_row(float (&x)[32], const float* s)
{
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
        const float2 r = __fmul2_rn(make_float2(x[i], x[i + 1]), *reinterpret_cast<const float2*>(s + i));
        x[i] = r.x;
        x[i + 1] = r.y;
    }
}
__device__ __forceinline__ void scale_add_row(float (&x)[32], const float* s, const float (&z)[32])
{
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
        const float2 r = __ffma2_rn(make_float2(x[i], x[i + 1]), *reinterpret_cast<const float2*>(s + i), make_float2(z[i], z[i + 1]));
        x[i] = r.x;
        x[i + 1] = r.y;
    }
}
// S = e S + half a row in the tensor-memory columns from `from` on.
template <int HS>
__device__ __forceinline__ void advance_state(float (&S)[HS], float e, uint32_t from)
{
    float x[HS];
#pragma unroll
    for (int i = 0; i < HS; i += 32) tc_ld32(from + i, x + i);
    tc_wait_ld();
#pragma unroll
    for (int i = 0; i < HS; i += 2) {
        const float2 r = __ffma2_rn(make_float2(S[i], S[i + 1]), make_float2(e, e), make_float2(x[i], x[i + 1]));
        S[i] = r.x;
        S[i + 1] = r.y;
    }
}

// S's (dS's) terms: half a row's lie side by side, three of SC columns.
template <int HS, int SC>
__device__ __forceinline__ void put_state(uint32_t addr, const float (&S)[HS])
{
#pragma unroll
    for (int i = 0; i < HS; i += 32) {
        float x[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) x[e] = S[i + e];
        put_terms<3>(addr + i / 2, SC, x);
    }
}

// All products of orders ORD down to LEAST of an operand of NA terms in tensor memory with
// NB planes in shared memory, small ones first: they add up before the large ones
// truncate the accumulator at their own size. mma(x, y, k, add) issues slice k (from
// FIRST on, cyclically) of term x with plane y.
template <int NA, int NB, int ORD, int KS, int FIRST, int LEAST = 0, typename F>
__device__ __forceinline__ void tc_product(bool add, F mma)
{
    // unrolled, constants and all: a product issues in its 32 cycles or less; rolled it took 70
#pragma unroll
    for (int o = ORD; o >= LEAST; --o)
#pragma unroll 1
        for (int y = o < NA ? 0 : o - NA + 1; y <= o && y < NB; ++y) {
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                mma(o - y, y, (k + FIRST) % KS, add);
                add = true;
            }
        }
}

// What a walk's CTA keeps in shared memory besides the stages.
struct WalkShared {
    unsigned long long full[2], empty[2], done[5];
    uint32_t tmem;
    int dead;
    alignas(16) int rows[4][DL_C];  // token rows of chunk c in slot c mod 4
};
static_assert(sizeof(WalkShared) <= WALK_FRONT, "shared memory in front of the stages");

struct WalkBars {
    uint32_t full, empty, done;  // shared addresses; 8 bytes apart
    __device__ __forceinline__ explicit WalkBars(WalkShared* w)
    {
        full = static_cast<uint32_t>(__cvta_generic_to_shared(w->full));
        empty = static_cast<uint32_t>(__cvta_generic_to_shared(w->empty));
        done = static_cast<uint32_t>(__cvta_generic_to_shared(w->done));
    }
};

// Tensor memory and barriers of a walk; all threads. A stage is free again after `releases` arrivals:
// the computing threads', who have then waited for every product of theirs that reads it, and one more
// where the issuing warp waits for a product that they do not wait for.
__device__ __forceinline__ uint32_t walk_begin(WalkShared* w, const WalkBars& bar, int releases)
{
    if (threadIdx.x < 32) tc_alloc(static_cast<uint32_t>(__cvta_generic_to_shared(&w->tmem)));
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar.full + 8 * i, DW_HELP);  // the copying threads, each with the bytes of its bulk copies
            mbar_init(bar.empty + 8 * i, releases);
        }
        for (int i = 0; i < 5; ++i) mbar_init(bar.done + 8 * i, 1);
        w->dead = 0;
        mbar_fence_init();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    return w->tmem;
}

__device__ __forceinline__ void walk_end(WalkShared* w, uint32_t tm, int* status)
{
    tc_wait_st();
    tc_fence_before();
    __syncthreads();
    start_next();
    if (threadIdx.x == 0 && status && w->dead) atomicOr(status, DEV_STATUS_TIMEOUT);
    if (threadIdx.x < 32) tc_free(tm, &w->dead);
}

// The copying warps' part: chunk n of `chunks` into stage n mod STAGES. `in` returns the bytes of
// its thread's bulk copies.
template <int STAGES, typename ROWS, typename IN>
__device__ __forceinline__ void walk_copy(WalkShared* w, const WalkBars& bar, int chunks, int tid, ROWS row_of, IN in)
{
    for (int n = 0; n < chunks; ++n) {
        const int st = STAGES == 2 ? n & 1 : 0;
        // chunk n - 4, the last user of this slot, has left: its y goes before chunk n - 3 is done, for
        // which the last round waited
        if (tid < DL_C) w->rows[n % 4][tid] = row_of(n, tid);
        bar_sync(7, DW_HELP);
        if (n >= STAGES) mbar_wait(bar.empty + 8 * st, ((n - STAGES) / STAGES) & 1, &w->dead);
        const uint32_t bytes = in(n, st, w->rows[n % 4]);
        cp_async_commit();
        cp_async_wait<0>();
        tc_fence_smem();
        mbar_expect(bar.full + 8 * st, bytes);
    }
}

__device__ __forceinline__ void walk_ready(int id)  // this thread's part of an operand is in tensor memory
{
    tc_wait_st();
    tc_fence_before();
    bar_arrive(id, DW_COMPUTE + 32);
}

template <typename T, int DKP, bool SAVE>
__global__ void __launch_bounds__(DW_THREADS, 1) delta_scan_kernel(const DeltaParams p)
{
    using Sh = WalkShape<T, DKP>;
    constexpr int NP = Sh::NP, PP = Sh::PP, HS = DKP / 2, KT = DKP / 16, STAGES = Sh::STAGES;
    // tensor-memory columns
    constexpr int cS = 0, cKS = cS + 6 * Sh::SC, cQS = cKS + 64, cX = cQS + 64, cO = cX + 96;
    constexpr int cDS = DKP == 128 ? cS : cO + 64;
    static_assert(cO + (DKP == 128 ? 64 : 128) <= 512, "tensor memory");
    extern __shared__ unsigned char smem_raw[];
    unsigned char* smem = smem_raw + (1024 - (__cvta_generic_to_shared(smem_raw) & 1023)) % 1024;
    WalkShared* ws = reinterpret_cast<WalkShared*>(smem);
    unsigned char* stages = smem + WALK_FRONT;
    constexpr int STAGE = Sh::stage(PP);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int head = blockIdx.y, b = blockIdx.z;
    const int slice = blockIdx.x * 128;
    const DeltaSeq s = delta_seq(p, b);
    const int chunks = (s.len + DL_C - 1) / DL_C;
    const size_t sbase = ((size_t)b * p.heads_v + head) * p.dk * p.dv;
    const WalkBars bar(ws);
    const uint32_t tm = walk_begin(ws, bar, DW_COMPUTE + (SAVE ? 0 : 1));
    wait_previous();

    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(DW_REGS_HELP));
        if (warp == 8) {
            auto aS = [&](int x, int ks) { return tm + cS + (ks / (KT / 2)) * 3 * Sh::SC + x * Sh::SC + (ks % (KT / 2)) * 8; };
            auto aX = [&](int x, int ks) { return tm + cX + (ks >> 1) * 48 + x * 16 + (ks & 1) * 8; };
            // W's terms for O lie over W itself and QS, each half of a row over the columns that its own thread has read
            auto aW = [&](int x, int ks) { return tm + (x < 2 ? cKS + x * 16 : cQS) + (ks >> 1) * 32 + (ks & 1) * 8; };
            for (int c = 0; c < chunks; ++c) {
                const int st = STAGES == 2 ? c & 1 : 0;
                const uint32_t par = c & 1;
                const uint32_t bK = static_cast<uint32_t>(__cvta_generic_to_shared(stages + st * STAGE));
                const uint64_t dK = tc_desc(bK + Sh::oK(PP)), dQ = tc_desc(bK + Sh::oQ(PP));
                const uint64_t dT = tc_desc(bK + Sh::oT), dP = tc_desc(bK + Sh::oP);
                mbar_wait(bar.full + 8 * st, (c / STAGES) & 1, &ws->dead);
                bar_sync(1, DW_COMPUTE + 32);
                tc_fence_after();
                if (tc_elect()) {  // 1
                    auto rows_of = [&](uint32_t d, uint64_t t) {
                        return [=](int x, int y, int ks, bool add) {
                            tc_mma(tm + d, aS(x, ks), t + (y * Sh::plane + (ks >> 2) * TC_TILE + (ks & 3) * 32) / 16,
                                   tc_idesc(64, false), add);
                        };
                    };
                    tc_product<3, NP, 2, KT, 0>(false, rows_of(cKS, dK));
                    tc_commit(bar.done);
                    if (!SAVE) {
                        tc_product<3, NP, 2, KT, 0>(false, rows_of(cQS, dQ));
                        tc_commit(bar.done + 8);
                    }
                }
                __syncwarp();
                bar_sync(2, DW_COMPUTE + 32);
                tc_fence_after();
                if (tc_elect()) {  // 2
                    tc_product<3, 3, 2, 4, 0>(false, [&](int x, int y, int ks, bool add) {
                        tc_mma(tm + cKS + 16 * ks, aX(x, ks), dT + (y * TC_TILE + ks * (2048 + 32)) / 16,
                               tc_idesc(64 - 16 * ks, false), add);
                    });
                    tc_commit(bar.done + 16);
                }
                __syncwarp();
                bar_sync(3, DW_COMPUTE + 32);
                tc_fence_after();
                if (tc_elect()) {  // 3
#pragma unroll
                    for (int nb = 0; nb < Sh::KB; ++nb)
                        tc_product<3, NP, 2, 4, 0>(false, [&](int x, int y, int ks, bool add) {
                            tc_mma(tm + cDS + nb * (3 * Sh::SC), aX(x, ks),
                                   dK + (y * Sh::plane + nb * TC_TILE + ks * 2048) / 16, tc_idesc(64, true), add);
                        });
                    tc_commit(bar.done + 24);
                }
                __syncwarp();
                if (!SAVE) {
                    bar_sync(4, DW_COMPUTE + 32);
                    tc_fence_after();
                    if (tc_elect()) {
                        tc_product<PP, PP, PP - 1, 4, 0>(false, [&](int x, int y, int ks, bool add) {
                            tc_mma(tm + cO + 16 * ks, aW(x, ks), dP + (y * TC_TILE + ks * (2048 + 32)) / 16,
                                   tc_idesc(64 - 16 * ks, false), add);
                        });
                        tc_commit(bar.done + 32);
                    }
                    __syncwarp();
                    // O has read W's terms, over which the next KS lies, and P, over which the stage's next record
                    // comes; the computing threads, which wait for O a chunk later, have not seen that
                    mbar_wait(bar.done + 32, par, &ws->dead);
                    if (lane == 0) mbar_arrive(bar.empty + 8 * st);
                }
            }
        } else {
            const int ht = tid - 288, hk = head / p.group;
            const long long img = delta_img(p, b);
            const T* q = reinterpret_cast<const T*>(p.q) + img * p.q_img + (long long)hk * p.dk;
            const T* k = reinterpret_cast<const T*>(p.k) + img * p.k_img + (long long)hk * p.dk;
            const T* v = reinterpret_cast<const T*>(p.v) + img * p.v_img + (long long)head * p.dv + slice;
            const int dvs = min(128, p.dv - slice);
            walk_copy<STAGES>(
                ws, bar, chunks, ht, [&](int c, int r) { return delta_row(p, s, c * DL_C + r); },
                [&](int c, int st, const int* rows) {
                    unsigned char* base = stages + st * STAGE;
                    const uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(base)), full = bar.full + 8 * st;
                    const size_t rec = (size_t)(s.slot + c) * p.heads_v + head;
                    if constexpr (NP == 1) {
                        walk_load<DKP>(base + Sh::oK(PP), k, p.k_tok, rows, p.dk, ht);
                        if (!SAVE) walk_load<DKP>(base + Sh::oQ(PP), q, p.q_tok, rows, p.dk, ht);
                        walk_load_values(reinterpret_cast<T*>(base + Sh::oV(PP)), Sh::vpitch, v, p.v_tok, rows, dvs, ht);
                    }
                    uint32_t bytes = 0;
                    if (ht == 0) {
                        bytes = DL_VECS * 4 + (NP == 1 ? (3 + (SAVE ? 0 : PP)) * TC_TILE : (3 + PP) * TC_TILE + 2 * NP * Sh::plane);
                        bulk_in(at, record_vec<T, DKP>(p, rec), bytes, full);
                    }
                    return bytes;
                });
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(DW_REGS_COMPUTE));
        const int half = warp >> 2, row = (warp & 3) * 32 + lane, vc = slice + row;  // this thread's value channel
        const bool live = vc < p.dv;
        const uint32_t tl = tm + ((uint32_t)(warp & 3) << 21);  // this warp's 32 rows
        const T* v = reinterpret_cast<const T*>(p.v) + delta_img(p, b) * p.v_img + (long long)head * p.dv + vc;
        T* y = reinterpret_cast<T*>(p.y) + delta_img(p, b) * p.y_img + (long long)head * p.dv + vc - lane;
        float S[HS];  // S^T[row][half * HS + i]
#pragma unroll
        for (int i = 0; i < HS; ++i) {
            const int kc = half * HS + i;
            S[i] = p.s_in && live && kc < p.dk ? p.s_in[sbase + (size_t)kc * p.dv + vc] : 0.f;
        }
        if (chunks > 0) {
            put_state<HS, Sh::SC>(tl + cS + half * 3 * Sh::SC, S);
            walk_ready(1);
        }
        // y of chunk c, which waits in `o` (its part from the entering state) and O: a chunk later, while the
        // chain waits for W and then for dS, so that it delays little
        float o[SAVE ? 1 : 32];
        T* corner = reinterpret_cast<T*>(stages + STAGES * STAGE) + half * 32 * Sh::vpitch + row;
        auto put_y = [&](int c) {
            float x[32];
            mbar_wait(bar.done + 32, c & 1, &ws->dead);
            tc_fence_after();
            tc_ld32(tl + cO + half * 32, x);
            tc_wait_ld();
            if constexpr (!SAVE) {
#pragma unroll
                for (int i = 0; i < 32; ++i) x[i] += o[i];
                if constexpr (NP == 1)
                    walk_stage(corner, Sh::vpitch, x);
                else
                    walk_put(y + lane, p.y_tok, ws->rows[c % 4] + half * 32, live, x);
            }
        };
        auto flush_y = [&](int c) {
            if constexpr (!SAVE && NP == 1)
                walk_flush(y, p.y_tok, ws->rows[c % 4] + half * 32, corner, Sh::vpitch, p.dv - vc + lane, lane);
        };
        for (int c = 0; c < chunks; ++c) {
            const int st = STAGES == 2 ? c & 1 : 0;
            const uint32_t par = c & 1;
            const T* vd = reinterpret_cast<const T*>(stages + st * STAGE + Sh::oV(PP)) + half * 32 * Sh::vpitch + row;
            const float* vec = reinterpret_cast<const float*>(stages + st * STAGE) + half * 32;
            const size_t rec = (size_t)(s.slot + c) * p.heads_v + head;
            if (SAVE && live) {  // the state entering the chunk, for the gradients
                float* o = p.wS + rec * p.dv * DKP + vc;
#pragma unroll
                for (int i = 0; i < HS; ++i) o[(size_t)(half * HS + i) * p.dv] = S[i];
            }
            float x[32];
            mbar_wait(bar.full + 8 * st, (c / STAGES) & 1, &ws->dead);
            {
                float u[32];
                if constexpr (NP == 1) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) u[i] = to_float(vd[i * Sh::vpitch]);
                } else {
                    walk_fetch(u, v, p.v_tok, ws->rows[c % 4] + half * 32, live);
                }
                mbar_wait(bar.done, par, &ws->dead);
                tc_fence_after();
                tc_ld32(tl + cKS + half * 32, x);
                tc_wait_ld();
#pragma unroll
                for (int i = 0; i < 32; ++i) x[i] = vec[2 * DL_C + i] * (u[i] - vec[i] * x[i]);  // X^T = beta (V - e^G K S)^T
            }
            put_terms<3>(tl + cX + half * 48, 16, x);
            walk_ready(2);
            if constexpr (!SAVE) {
                if (c > 0) put_y(c - 1);
                mbar_wait(bar.done + 8, par, &ws->dead);
                tc_fence_after();
                tc_ld32(tl + cQS + half * 32, o);
                tc_wait_ld();
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] *= p.scale * vec[i];
            }
            mbar_wait(bar.done + 16, par, &ws->dead);
            tc_fence_after();
            tc_ld32(tl + cKS + half * 32, x);
            tc_wait_ld();
            {
                float w[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) w[i] = x[i];
                scale_row(w, vec + DL_C);
                put_terms<3>(tl + cX + half * 48, 16, w);
                walk_ready(3);
            }
            if constexpr (SAVE) {
                if (live) {
                    float* ow = p.wW + (rec * DL_C + half * 32) * p.dv + vc;
#pragma unroll
                    for (int i = 0; i < 32; ++i) ow[(size_t)i * p.dv] = x[i];
                }
            } else {
                if constexpr (PP == 2) {
                    put_terms<2>(tl + cKS + half * 32, 16, x);
                } else {  // the third term lies apart
                    float w[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i) w[i] = x[i] - upper_terms(x[i]);
                    put_terms<1>(tl + cQS + half * 32, 16, w);
                    put_terms<2, true>(tl + cKS + half * 32, 16, x);
                }
                walk_ready(4);
            }
            if (c > 0) flush_y(c - 1);
            const float eC = vec[3 * DL_C - half * 32];
            mbar_wait(bar.done + 24, par, &ws->dead);
            tc_fence_after();
            advance_state(S, eC, tl + cDS + half * (DKP == 128 ? 3 * Sh::SC : 32));
            mbar_arrive(bar.empty + 8 * st);
            if (c + 1 < chunks) {
                put_state<HS, Sh::SC>(tl + cS + half * 3 * Sh::SC, S);
                walk_ready(1);
            }
        }
        if (!SAVE && chunks > 0) {
            put_y(chunks - 1);
            flush_y(chunks - 1);
        }
        if (p.s_out && live)
#pragma unroll
            for (int i = 0; i < HS; ++i)
                if (half * HS + i < p.dk) p.s_out[sbase + (size_t)(half * HS + i) * p.dv + vc] = S[i];
    }
    walk_end(ws, tm, p.status);
}

// ---- one token ----------------------------------------------------------------------
// One CTA per row, value head and 32 value channels: 8 lanes hold four channels
// each of a state row, 16 such groups share the dk rows. The state is read once
// into registers and written once: bound by those bytes (256 rows of 6 heads of 128 x 128:
// 203 MB in 33 us, 6.1 TB/s).
constexpr int DS_COLS = 32, DS_GROUPS = 16, DS_ROWS = 8;  // dk <= 128

template <typename T>
__global__ void __launch_bounds__(128) delta_step_kernel(const DeltaParams p)
{
    __shared__ float kq[2][128];
    __shared__ float4 part[4][8];
    const int tid = threadIdx.x, lane8 = tid & 7, grp = tid >> 3, warp = tid >> 5;
    const int head = blockIdx.y, b = blockIdx.z, hk = head / p.group;
    const int vc = blockIdx.x * DS_COLS + lane8 * 4;
    const bool live = vc < p.dv;
    const size_t sbase = ((size_t)b * p.heads_v + head) * p.dk * p.dv + vc;
    float4 S[DS_ROWS];
#pragma unroll
    for (int i = 0; i < DS_ROWS; ++i) {
        const int r = i * DS_GROUPS + grp;
        S[i] = live && r < p.dk ? *reinterpret_cast<const float4*>(p.s_in + sbase + (size_t)r * p.dv)
                                : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    if (tid < p.dk) {
        kq[0][tid] = to_float(reinterpret_cast<const T*>(p.k)[(long long)b * p.k_img + (long long)hk * p.dk + tid]);
        kq[1][tid] = to_float(reinterpret_cast<const T*>(p.q)[(long long)b * p.q_img + (long long)hk * p.dk + tid]);
    }
    const float x = to_float(reinterpret_cast<const T*>(p.a)[(long long)b * p.a_img + head]) + (p.bias ? p.bias[head] : 0.f);
    const float decay = expf(delta_decay(p.A[head], x));
    const float beta = p.beta_scale * delta_sigmoid(to_float(reinterpret_cast<const T*>(p.b)[(long long)b * p.b_img + head]));
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (live) v = load4(reinterpret_cast<const T*>(p.v) + (long long)b * p.v_img + (long long)head * p.dv + vc);
    __syncthreads();

    // sum over the rows: over the registers, the four groups of a warp, the four warps
    auto rows_dot = [&](const float* vec) {
        float4 d = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int i = 0; i < DS_ROWS; ++i) {
            const int r = i * DS_GROUPS + grp;
            const float c = r < p.dk ? vec[r] : 0.f;
            d.x += c * S[i].x; d.y += c * S[i].y; d.z += c * S[i].z; d.w += c * S[i].w;
        }
#pragma unroll
        for (int o = 8; o < 32; o <<= 1) {
            d.x += __shfl_xor_sync(0xffffffffu, d.x, o);
            d.y += __shfl_xor_sync(0xffffffffu, d.y, o);
            d.z += __shfl_xor_sync(0xffffffffu, d.z, o);
            d.w += __shfl_xor_sync(0xffffffffu, d.w, o);
        }
        if ((tid & 31) < 8) part[warp][lane8] = d;
        __syncthreads();
        d = part[0][lane8];
#pragma unroll
        for (int w = 1; w < 4; ++w) {
            const float4 e = part[w][lane8];
            d.x += e.x; d.y += e.y; d.z += e.z; d.w += e.w;
        }
        return d;
    };
#pragma unroll
    for (int i = 0; i < DS_ROWS; ++i) { S[i].x *= decay; S[i].y *= decay; S[i].z *= decay; S[i].w *= decay; }
    const float4 d = rows_dot(kq[0]);
    const float4 w = make_float4(beta * (v.x - d.x), beta * (v.y - d.y), beta * (v.z - d.z), beta * (v.w - d.w));
    __syncthreads();  // part is read before the second sum writes it
#pragma unroll
    for (int i = 0; i < DS_ROWS; ++i) {
        const int r = i * DS_GROUPS + grp;
        if (r < p.dk) {
            const float c = kq[0][r];
            S[i].x += c * w.x; S[i].y += c * w.y; S[i].z += c * w.z; S[i].w += c * w.w;
            if (live) *reinterpret_cast<float4*>(p.s_out + sbase + (size_t)r * p.dv) = S[i];
        }
    }
    float4 o = rows_dot(kq[1]);
    if (tid < 8 && live) {
        o.x *= p.scale; o.y *= p.scale; o.z *= p.scale; o.w *= p.scale;
        store4(reinterpret_cast<T*>(p.y) + (long long)b * p.y_img + (long long)head * p.dv + vc, o);
    }
}

}  // namespace vscan
