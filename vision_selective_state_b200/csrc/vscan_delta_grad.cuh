// Gated delta rule: device code of the backward pass.
//
// With dO the gradient of y and dS that of the state leaving a chunk, the chunk's
// forward (see vscan_delta.cuh) turned round is
//
//   dW = P^T dO + (e^{G_C - G_j} k_j) dS          dX = T^T dW          dV = beta dX
//   dS0 = e^{G_C} dS + sum_i scale e^{G_i} q_i dO_i^T - sum_i e^{G_i} k_i dV_i^T
//   E_ij = scale e^{G_i - G_j} dO_i.w_j (j <= i)   M_ij = -e^{G_i - G_j} dV_i.w_j (j < i)
//   dq_i  = scale e^{G_i} S0 dO_i + sum_j E_ij k_j
//   dkr_i = -e^{G_i} S0 dV_i + sum_j M_ij k_j                        (k_i as the key that reads)
//   dkc_j = e^{G_C - G_j} dS w_j + sum_i E_ij q_i + sum_i M_ij k_i   (k_j as the key that writes)
//   dg_i  = sum_{r >= i > j} H_rj + sum_{r >= i} U_r + sum_{j < i} V_j + e^{G_C} <dS, S0>
//           H_rj = E_rj q_r.k_j + M_rj k_r.k_j
//           U_r = scale e^{G_r} q_r.S0 dO_r - e^{G_r} k_r.S0 dV_r      V_j = e^{G_C - G_j} k_j.dS w_j
//   db_i  = (dX_i.w_i)(1 - sigmoid(b_i))
//
// The first two lines need the chunks in order and only this head's slice of the
// value channels (delta_rscan_kernel); the rest is independent chunk by chunk
// (delta_grad_kernel). dg_i gathers the terms whose decay factor spans step i; the
// pairs (r, j) that do are the row sums of H from i on less its column sums from i
// on, in which a pair that lies wholly behind i cancels: both sums run in float64
// over the same rounded H, so it cancels to 2^-53 of itself. (q.dq + k.dk over the
// finished gradients has the same value, but its cancelling parts are rounded
// apart, which strong decays - dg small, A large - turn into an error of da.)
#pragma once

#include "vscan_delta.cuh"

namespace vscan {

// ---- the walk backwards ---------------------------------------------------------------
// As the walk forwards, with dS^T[128][DKP] in registers:
//
//   1. D1 = dS K^T, D2 = dO P                        B = K (K-major), P (MN-major)
//   2. dW = e^{G_C - G} D1 + D2;  dX = dW T          B = T (MN-major)
//   3. ddS = (scale e^G dO) Q - (e^G beta dX) K      B = Q, K (MN-major)
//   4. dS = e^{G_C} dS + ddS
//
// Tensor-memory columns: dS's terms (over them ddS), D1 (then dX), D2 and dO's terms
// (then those of scale e^G dO), dW's terms (then those of e^G dV).
template <typename T, int DKP>
__global__ void __launch_bounds__(DW_THREADS, 1) delta_rscan_kernel(const DeltaParams p)
{
    using Sh = WalkShape<T, DKP>;
    constexpr int NP = Sh::NP, HS = DKP / 2, KT = DKP / 16, STAGE = Sh::stage(3), STAGES = Sh::STAGES;
    constexpr int cS = 0, c1 = cS + 6 * Sh::SC, c2 = c1 + 64, cA = c2 + 64, cW = cA + NP * 32;
    constexpr int cDS = DKP == 128 ? cS : cW + 96;
    static_assert(cW + (DKP == 128 ? 96 : 160) <= 512, "tensor memory");
    extern __shared__ unsigned char smem_raw[];
    unsigned char* smem = smem_raw + (1024 - (__cvta_generic_to_shared(smem_raw) & 1023)) % 1024;
    WalkShared* ws = reinterpret_cast<WalkShared*>(smem);
    unsigned char* stages = smem + WALK_FRONT;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int head = blockIdx.y, b = blockIdx.z;
    const int slice = blockIdx.x * 128;
    const DeltaSeq s = delta_seq(p, b);
    const int chunks = (s.len + DL_C - 1) / DL_C;
    const size_t sbase = ((size_t)b * p.heads_v + head) * p.dk * p.dv;
    const WalkBars bar(ws);
    const uint32_t tm = walk_begin(ws, bar, DW_COMPUTE);  // they wait for the last product
    wait_previous();
    // n counts the chunks in the order of the walk, from the last to the first

    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(DW_REGS_HELP));
        if (warp == 8) {
            auto aS = [&](int x, int ks) { return tm + cS + (ks / (KT / 2)) * 3 * Sh::SC + x * Sh::SC + (ks % (KT / 2)) * 8; };
            auto aO = [&](int x, int ks) { return tm + cA + (ks >> 1) * (NP * 16) + x * 16 + (ks & 1) * 8; };
            auto aQ = [&](int x, int ks) { return tm + c2 + (ks >> 1) * 48 + x * 16 + (ks & 1) * 8; };
            auto aW = [&](int x, int ks) { return tm + cW + (ks >> 1) * 48 + x * 16 + (ks & 1) * 8; };
            for (int n = 0; n < chunks; ++n) {
                const int st = STAGES == 2 ? n & 1 : 0;
                const uint32_t bK = static_cast<uint32_t>(__cvta_generic_to_shared(stages + st * STAGE));
                const uint64_t dK = tc_desc(bK + Sh::oK(3)), dQ = tc_desc(bK + Sh::oQ(3)), dT = tc_desc(bK + Sh::oT), dP = tc_desc(bK + Sh::oP);
                mbar_wait(bar.full + 8 * st, (n / STAGES) & 1, &ws->dead);
                bar_sync(1, DW_COMPUTE + 32);
                tc_fence_after();
                if (tc_elect())  // 1
                    tc_product<3, NP, 2, KT, 0>(false, [&](int x, int y, int ks, bool add) {
                        tc_mma(tm + c1, aS(x, ks), dK + (y * Sh::plane + (ks >> 2) * TC_TILE + (ks & 3) * 32) / 16,
                               tc_idesc(64, false), add);
                    });
                __syncwarp();
                bar_sync(2, DW_COMPUTE + 32);
                tc_fence_after();
                if (tc_elect()) {  // slice ks of the rows i reaches the columns j up to 16 ks + 15: the last one covers all
                    tc_product<NP, 3, 2, 4, 3>(false, [&](int x, int y, int ks, bool add) {
                        tc_mma(tm + c2, aO(x, ks), dP + (y * TC_TILE + ks * 2048) / 16, tc_idesc(16 * ks + 16, true), add);
                    });
                    tc_commit(bar.done);
                }
                __syncwarp();
                bar_sync(3, DW_COMPUTE + 32);
                tc_fence_after();
                if (tc_elect()) {  // 2
                    tc_product<3, 3, 2, 4, 3>(false, [&](int x, int y, int ks, bool add) {
                        tc_mma(tm + c1, aW(x, ks), dT + (y * TC_TILE + ks * 2048) / 16, tc_idesc(16 * ks + 16, true), add);
                    });
                    tc_commit(bar.done + 8);
                }
                __syncwarp();
                // small terms of both parts before the large ones of either
                auto part = [&](auto a, uint64_t t, int nb) {
                    return [=](int x, int y, int ks, bool add) {
                        tc_mma(tm + cDS + nb * (3 * Sh::SC), a(x, ks), t + (y * Sh::plane + nb * TC_TILE + ks * 2048) / 16,
                               tc_idesc(64, true), add);
                    };
                };
                bar_sync(4, DW_COMPUTE + 32);
                tc_fence_after();
                if (tc_elect())  // 3
#pragma unroll
                    for (int nb = 0; nb < Sh::KB; ++nb) tc_product<3, NP, 2, 4, 0, 1>(false, part(aQ, dQ, nb));
                __syncwarp();
                bar_sync(5, DW_COMPUTE + 32);
                tc_fence_after();
                if (tc_elect()) {
#pragma unroll
                    for (int nb = 0; nb < Sh::KB; ++nb) {
                        tc_product<3, NP, 2, 4, 0, 1>(true, part(aW, dK, nb));
                        tc_product<3, NP, 0, 4, 0>(true, part(aQ, dQ, nb));
                        tc_product<3, NP, 0, 4, 0>(true, part(aW, dK, nb));
                    }
                    tc_commit(bar.done + 16);
                }
                __syncwarp();
            }
        } else {
            const int ht = tid - 288, hk = head / p.group;
            const long long img = delta_img(p, b);
            const T* q = reinterpret_cast<const T*>(p.q) + img * p.q_img + (long long)hk * p.dk;
            const T* k = reinterpret_cast<const T*>(p.k) + img * p.k_img + (long long)hk * p.dk;
            const T* dy = reinterpret_cast<const T*>(p.dy) + img * p.y_img + (long long)head * p.dv + slice;
            const int dvs = min(128, p.dv - slice);
            walk_copy<STAGES>(
                ws, bar, chunks, ht, [&](int n, int r) { return delta_row(p, s, (chunks - 1 - n) * DL_C + r); },
                [&](int n, int st, const int* rows) {
                    unsigned char* base = stages + st * STAGE;
                    const uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(base)), full = bar.full + 8 * st;
                    const size_t rec = (size_t)(s.slot + chunks - 1 - n) * p.heads_v + head;
                    if constexpr (NP == 1) {
                        walk_load<DKP>(base + Sh::oK(3), k, p.k_tok, rows, p.dk, ht);
                        walk_load<DKP>(base + Sh::oQ(3), q, p.q_tok, rows, p.dk, ht);
                        walk_load_values(reinterpret_cast<T*>(base + Sh::oV(3)), Sh::vpitch, dy, p.y_tok, rows, dvs, ht);
                    }
                    uint32_t bytes = 0;
                    if (ht == 0) {
                        bytes = DL_VECS * 4 + 6 * TC_TILE + (NP == 1 ? 0 : 2 * NP * Sh::plane);
                        bulk_in(at, record_vec<T, DKP>(p, rec), bytes, full);
                    }
                    return bytes;
                });
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(DW_REGS_COMPUTE));
        const int half = warp >> 2, row = (warp & 3) * 32 + lane, vc = slice + row;
        const bool live = vc < p.dv;
        const uint32_t tl = tm + ((uint32_t)(warp & 3) << 21);
        const T* dy = reinterpret_cast<const T*>(p.dy) + delta_img(p, b) * p.y_img + (long long)head * p.dv + vc;
        T* dvalue = reinterpret_cast<T*>(p.dvalue);
        if (dvalue) dvalue += (delta_img(p, b) * p.tokens * p.heads_v + head) * (long long)p.dv + vc - lane;
        float S[HS];  // dS^T[row][half * HS + i]
#pragma unroll
        for (int i = 0; i < HS; ++i) {
            const int kc = half * HS + i;
            S[i] = p.ds_in && live && kc < p.dk ? p.ds_in[sbase + (size_t)kc * p.dv + vc] : 0.f;
        }
        if (chunks > 0) {
            put_state<HS, Sh::SC>(tl + cS + half * 3 * Sh::SC, S);
            walk_ready(1);
        }
        for (int n = 0; n < chunks; ++n) {
            const int st = STAGES == 2 ? n & 1 : 0;
            const uint32_t par = n & 1;
            T* vd = reinterpret_cast<T*>(stages + st * STAGE + Sh::oV(3)) + half * 32 * Sh::vpitch + row;
            const float* vec = reinterpret_cast<const float*>(stages + st * STAGE) + half * 32;
            const size_t rec = (size_t)(s.slot + chunks - 1 - n) * p.heads_v + head;
            float o[32], x[32];
            mbar_wait(bar.full + 8 * st, (n / STAGES) & 1, &ws->dead);
            if constexpr (NP == 1) {
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] = to_float(vd[i * Sh::vpitch]);
            } else {
                walk_fetch(o, dy, p.y_tok, ws->rows[n % 4] + half * 32, live);
            }
#pragma unroll
            for (int i = 0; i < 32; ++i) x[i] = o[i];
            put_terms<NP>(tl + cA + half * (NP * 16), 16, x);
            walk_ready(2);
            if (live) {  // the gradient of the state leaving the chunk
                float* g = p.wdS + rec * p.dv * DKP + vc;
#pragma unroll
                for (int i = 0; i < HS; ++i) g[(size_t)(half * HS + i) * p.dv] = S[i];
            }
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] *= p.scale * vec[i];
            mbar_wait(bar.done, par, &ws->dead);
            tc_fence_after();
            {
                float z[32];
                tc_ld32(tl + c1 + half * 32, x);
                tc_ld32(tl + c2 + half * 32, z);
                tc_wait_ld();
                scale_add_row(x, vec + DL_C, z);
            }
            put_terms<3>(tl + cW + half * 48, 16, x);
            walk_ready(3);
            // over D2, which both halves of a row have to have read
            mbar_wait(bar.done + 8, par, &ws->dead);
            put_terms<3>(tl + c2 + half * 48, 16, o);
            walk_ready(4);
            tc_fence_after();
            tc_ld32(tl + c1 + half * 32, x);
            tc_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = x[i];
            scale_row(x, vec + 6 * DL_C);
            put_terms<3>(tl + cW + half * 48, 16, x);  // -e^G dV
            walk_ready(5);
            if (live) {
                float* ox = p.wdX + (rec * DL_C + half * 32) * p.dv + vc;
#pragma unroll
                for (int i = 0; i < 32; ++i) ox[(size_t)i * p.dv] = o[i];
            }
            if (dvalue) {
#pragma unroll
                for (int i = 0; i < 32; ++i) x[i] = o[i];
                scale_row(x, vec + 2 * DL_C);
                if constexpr (NP == 1)
                    walk_store(dvalue, (long long)p.heads_v * p.dv, ws->rows[n % 4] + half * 32, vd, Sh::vpitch, p.dv - vc + lane,
                               lane, x);
                else
                    walk_put(dvalue + lane, (long long)p.heads_v * p.dv, ws->rows[n % 4] + half * 32, live, x);
            }
            const float eC = vec[3 * DL_C - half * 32];
            mbar_wait(bar.done + 16, par, &ws->dead);
            tc_fence_after();
            advance_state(S, eC, tl + cDS + half * (DKP == 128 ? 3 * Sh::SC : 32));
            mbar_arrive(bar.empty + 8 * st);
            if (n + 1 < chunks) {
                put_state<HS, Sh::SC>(tl + cS + half * 3 * Sh::SC, S);
                walk_ready(1);
            }
        }
        if (p.ds_out && live)
#pragma unroll
            for (int i = 0; i < HS; ++i)
                if (half * HS + i < p.dk) p.ds_out[sbase + (size_t)(half * HS + i) * p.dv + vc] = S[i];
    }
    walk_end(ws, tm, p.status);
}

// ---- per-chunk gradients -------------------------------------------------------------
// One CTA per chunk and value head. As in the walks the products stand
// transposed, with the key channel as the row of the 128-row tile, so that a thread
// holds a quarter of the steps of one key channel:
//
//   D1[dk][i | i] = S0 [dO | dV]^T      D2[i | i][j] = [dO | dV] W^T      D3[dk][j] = dS W^T
//   (dq | dkr)^T = (scale e^G | -e^G) D1 + K^T [E | M]^T       dkc^T = e^{G_C - G} D3 + Q^T E + K^T M
//
// D1 .. D3 take both operands from shared memory, where everything float32 lies split in
// bf16 planes, in slabs of 64 value channels; dO and dV share their tiles' rows, so that
// they are one operand. E and M come from D2 through registers and back to shared memory,
// [i][j], where the same tile is E (M) and its transpose; K^T and Q^T lie in tensor memory.
// One CTA an SM, whose phases follow one another: of the 34,000 cycles of a chunk and head
// at dk = dv = 128 the products take 12,000, splitting the operands (S0 and dS are 32,768
// values) and waiting for them 10,000, E and M 2,400, the scaled results with their part of dg
// 3,200. Sixteen computing warps instead of eight: 57 -> 44 us for 3 float32 images of 777 tokens
// (dk 48, dv 80), 31 us instead of 35 for 8 bf16 ones of 197, and no change at 128 x 128, where
// the tensor core and the loads bound the slabs. 544 threads leave 96 registers each, too few for
// all pieces fetched ahead: 4 and 84 bytes a thread spill in bf16 (DKP 64, 128), 52 and 140 in float32.
constexpr int DG_COMPUTE = 512, DG_THREADS = 544;  // sixteen warps and one that issues the products

template <typename T> struct GradRaw;  // four values of dy
template <> struct GradRaw<__nv_bfloat16> { using type = uint2; };
template <> struct GradRaw<float> { using type = float4; };

template <typename T, int DKP>
struct GradShape {
    static constexpr int NP = DeltaIo<T>::planes;
    static constexpr int KB = DKP / 64;
    static constexpr int plane = KB * TC_TILE;    // of K or Q; of a slab of a state: [DKP][64]
    static constexpr int oK = 0, oQ = NP * plane, oS = 2 * NP * plane, oW = oS + 3 * plane;
    static constexpr int oX = oW + 3 * TC_TILE;   // three pairs of tiles: dO's and dV's terms; later E's and M's
    static constexpr int oEnd = oX + 6 * TC_TILE;
    static constexpr int oSums = oW + 2 * TC_TILE;  // GradSums, once W is read
    static constexpr int front = 4096;  // GradShared
    static constexpr size_t smem = 1024 + front + oEnd;
};

struct GradShared {
    unsigned long long done;
    uint32_t tmem;
    int dead;
    alignas(16) int rows[DL_C];
    float xw[DL_C];                // dX.w
    float red[DG_COMPUTE / 32];    // <dS, S0>
    alignas(16) float vec[DL_VECS];
};
struct GradSums {
    double hrow[2][4][DL_C];       // row sums of H: E's and M's part, quarters of the columns
    double hcol[4][DL_C];          // column sums, by quarters of the 128 rows of D2
    float U[4][DL_C], V[4][DL_C];  // by quarters of the key channels
};
static_assert(sizeof(GradShared) <= 4096, "shared memory in front of the tiles");
static_assert(sizeof(GradSums) <= TC_TILE, "in the place of W's third plane");

// Sum over the warp of each of 32 values; lane l gets the l-th.
__device__ __forceinline__ float reduce_columns(float (&v)[32], int lane)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const bool up = lane & o;
#pragma unroll
        for (int i = 0; i < o; ++i) {
            const float send = up ? v[i] : v[i + o], keep = up ? v[i + o] : v[i];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
        }
    }
    return v[0];
}

// Four values of a row into three planes of a swizzled tile (planes `plane` bytes apart).
__device__ __forceinline__ void put_planes(unsigned char* dst, int plane, int r, int c, float4 x)
{
    unsigned char* o = dst + r * 128 + (((c >> 3) ^ (r & 7)) << 4) + (c & 7) * 2;
#pragma unroll
    for (int n = 0; n < 3; ++n) {
        uint2 u;
        u.x = split_bf16(x.x, x.y);
        u.y = split_bf16(x.z, x.w);
        *reinterpret_cast<uint2*>(o + n * plane) = u;
    }
}

// N values of a row, NP bf16 terms, from a column of a [64][DKP] tile of K or Q.
template <int NP, int DKP, int N>
__device__ __forceinline__ void column_of(const unsigned char* tile, int plane, int col, int first, float (&v)[N])
{
#pragma unroll
    for (int i = 0; i < N; ++i) {
        float x = 0.f;
        const unsigned char* at = tile + tc_swizzle(first + i, col >> 3) + (col & 7) * 2;
#pragma unroll
        for (int n = NP - 1; n >= 0; --n) x += __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(at + n * plane));
        v[i] = x;
    }
}

// Rows of K or Q into swizzled tiles, by all threads.
template <int DKP>
__device__ __forceinline__ void grad_load(unsigned char* dst, const __nv_bfloat16* src, long long tok, const int* rows, int have, int tid)
{
    constexpr int vecs = DKP / 8;
    const int c = tid % vecs;
    const bool in = c * 8 < have;
    const __nv_bfloat16* at = in ? src + c * 8 : src;
    copy_rows<vecs, DG_COMPUTE>(rows, tid, [&](int r, int row) {
        const bool ok = in && row >= 0;
        copy16(dst + tc_swizzle(r, c), at + (ok ? row * tok : 0), ok);
    });
}
template <int DKP>
__device__ __forceinline__ void grad_load(unsigned char* dst, const float* src, long long tok, const int* rows, int have, int tid)
{
    constexpr int vecs = DKP / 4;
    const int c = tid % vecs * 4;
    copy_rows<vecs, DG_COMPUTE>(rows, tid, [&](int r, int row) {
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (row >= 0 && c < have) x = __ldg(reinterpret_cast<const float4*>(src + c + row * tok));
        put_planes(dst + (c >> 6) * TC_TILE, DKP / 64 * TC_TILE, r, c & 63, x);
    });
}

template <typename T, int DKP>
__global__ void __launch_bounds__(DG_THREADS, 1) delta_grad_kernel(const DeltaParams p)
{
    using Sh = GradShape<T, DKP>;
    constexpr int NP = Sh::NP;
    // tensor-memory columns; what D1 .. D3 get from the smaller terms is summed apart, cSmall further on
    // (one accumulator over several slabs would be truncated by each of them), and K^T and Q^T follow there
    constexpr int c1 = 0, c2 = 128, c3 = 192, cSmall = 256, cKT = 256, cQT = cKT + NP * 32;
    extern __shared__ unsigned char smem_raw[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, quarter = warp >> 2;
    const int head = blockIdx.y, hk = head / p.group;
    wait_previous();

    int b;
    if (p.offsets) {
        int lo = 0, hi = p.batch;
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
    const size_t rec = (size_t)blockIdx.x * p.heads_v + head;
    const float* wS = p.wS + rec * p.dv * DKP;
    const float* wdS = p.wdS + rec * p.dv * DKP;
    const float* wW = p.wW + rec * DL_C * p.dv;
    const float* wdX = p.wdX + rec * DL_C * p.dv;
    const T* dy = reinterpret_cast<const T*>(p.dy) + img * p.y_img + (long long)head * p.dv;

    GradShared* sh = reinterpret_cast<GradShared*>(smem_raw);
    unsigned char* tiles = smem_raw + Sh::front;
    tiles += (1024 - (__cvta_generic_to_shared(tiles) & 1023)) % 1024;
    GradSums* sums = reinterpret_cast<GradSums*>(tiles + Sh::oSums);
    const uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(tiles));
    const uint32_t done = static_cast<uint32_t>(__cvta_generic_to_shared(&sh->done));
    // A slab of everything else passes through registers, fetched ahead: a state is NS pieces of
    // four channels a thread, W, dX and dO NW each (a row's sixteen pieces are in half a warp).
    constexpr int STEP = DG_COMPUTE / 16, NS = DKP / STEP, NW = DL_C / STEP;
    using Raw = typename GradRaw<T>::type;
    const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
    const int pr = tid >> 4, pc = (tid & 15) * 4;  // first row of this thread's pieces, STEP apart, and their columns
    float4 s0[NS], ds[NS], w[NW], x[NW];
    Raw o[NW];
    auto fetch_state = [&](float4 (&v)[NS], const float* src, int slab) {
        const bool in = slab + pc < p.dv;
#pragma unroll
        for (int i = 0; i < NS; ++i)
            v[i] = in ? __ldg(reinterpret_cast<const float4*>(src + (size_t)(pr + STEP * i) * p.dv + slab + pc)) : zero;
    };
    auto fetch = [&](int slab) {
        fetch_state(s0, wS, slab);
        fetch_state(ds, wdS, slab);
        const bool in = slab + pc < p.dv;
#pragma unroll
        for (int i = 0; i < NW; ++i) {
            const int r = pr + STEP * i;
            w[i] = in ? __ldg(reinterpret_cast<const float4*>(wW + (size_t)r * p.dv + slab + pc)) : zero;
            x[i] = in ? __ldg(reinterpret_cast<const float4*>(wdX + (size_t)r * p.dv + slab + pc)) : zero;
        }
    };
    auto fetch_dy = [&](int slab) {
#pragma unroll
        for (int i = 0; i < NW; ++i) {
            const int row = sh->rows[pr + STEP * i];
            o[i] = Raw{};
            if (slab + pc < p.dv && row >= 0) o[i] = __ldg(reinterpret_cast<const Raw*>(dy + row * p.y_tok + slab + pc));
        }
    };
    if (warp < DG_COMPUTE / 32) fetch(0);

    if (warp == 0) tc_alloc(static_cast<uint32_t>(__cvta_generic_to_shared(&sh->tmem)));
    if (tid == 0) {
        mbar_init(done, 1);
        sh->dead = 0;
        mbar_fence_init();
    }
    if (tid < DL_C) sh->rows[tid] = delta_row(p, s, t0 + tid);
    if (tid < DL_VECS / 4) reinterpret_cast<float4*>(sh->vec)[tid] = __ldg(reinterpret_cast<const float4*>(record_vec<T, DKP>(p, rec)) + tid);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = sh->tmem, tl = tm + ((uint32_t)(warp & 3) << 21);
    uint32_t phase = 0;
    const float* vec = sh->vec;
    const uint64_t aS = tc_desc(at + Sh::oS), aX = tc_desc(at + Sh::oX), bW = tc_desc(at + Sh::oW);
    auto aK = [&](int x, int ks) { return tm + cKT + x * 32 + ks * 8; };

    if (warp == DG_COMPUTE / 32) {  // issues the products
        // what dg, da and db need of a and b, two steps a lane, ahead of the sums
        const float A = p.A[head], bias = p.bias ? p.bias[head] : 0.f;
        float soft[2], slope[2], open[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int row = sh->rows[2 * lane + i];
            const float a = (row >= 0 ? to_float(reinterpret_cast<const T*>(p.a)[img * p.a_img + row * p.a_tok + head]) : 0.f) + bias;
            const float bb = row >= 0 ? to_float(reinterpret_cast<const T*>(p.b)[img * p.b_img + row * p.b_tok + head]) : 0.f;
            soft[i] = delta_softplus(a);
            slope[i] = A * delta_sigmoid(a);
            open[i] = delta_sigmoid(-bb);
        }
        for (int slab = 0; slab < p.dv; slab += 64) {
            const bool more = slab > 0;
            bar_sync(1, DG_THREADS);
            tc_fence_after();
            if (tc_elect()) {
                auto d1 = [&](int x, int y, int ks, bool add) {  // S0 [dO | dV]^T
                    const uint32_t d = tm + c1 + (x + y ? cSmall : 0);
                    const uint64_t a = aS + (x * Sh::plane + ks * 32) / 16;
                    if (NP == 1 && y > 0)
                        tc_mma_ss(d + 64, a, aX + ((2 * y + 1) * TC_TILE + ks * 32) / 16, tc_idesc(64, false), add);
                    else
                        tc_mma_ss(d, a, aX + (2 * y * TC_TILE + ks * 32) / 16, tc_idesc(128, false), add);
                };
                tc_product<3, 3, 2, 4, 0, 1>(more, d1);
                tc_product<3, 3, 0, 4, 0>(more, d1);
                tc_commit(done);
                auto d2 = [&](int x, int y, int ks, bool add) {  // [dO | dV] W^T
                    tc_mma_ss(tm + c2 + (x + y ? cSmall : 0), aX + (2 * x * TC_TILE + ks * 32) / 16, bW + (y * TC_TILE + ks * 32) / 16, tc_idesc(64, false),
                              add);
                };
                tc_product<3, 3, 2, 4, 0, 1>(more, d2);
                tc_product<3, 3, 0, 4, 0>(more, d2);
            }
            __syncwarp();
            bar_sync(2, DG_THREADS);
            tc_fence_after();
            if (tc_elect()) {
                auto d3 = [&](int x, int y, int ks, bool add) {  // dS W^T
                    tc_mma_ss(tm + c3 + (x + y ? cSmall : 0), aS + (x * Sh::plane + ks * 32) / 16,
                              bW + (y * TC_TILE + ks * 32) / 16, tc_idesc(64, false), add);
                };
                tc_product<3, 3, 2, 4, 0, 1>(more, d3);
                tc_product<3, 3, 0, 4, 0>(more, d3);
                tc_commit(done);
            }
            __syncwarp();
        }
        bar_sync(3, DG_THREADS);
        tc_fence_after();
        if (tc_elect()) {
            tc_product<NP, 3, 2, 4, 0>(false, [&](int x, int y, int ks, bool add) {  // K^T [E | M]^T
                tc_mma(tm + c1, aK(x, ks), aX + (2 * y * TC_TILE + ks * 32) / 16, tc_idesc(128, false), add);
            });
            auto qe = [&](int x, int y, int ks, bool add) {  // Q^T E
                tc_mma(tm + c3, tm + cQT + x * 32 + ks * 8, aX + (2 * y * TC_TILE + ks * 2048) / 16, tc_idesc(64, true), add);
            };
            auto km = [&](int x, int y, int ks, bool add) {  // K^T M
                tc_mma(tm + c3, aK(x, ks), aX + ((2 * y + 1) * TC_TILE + ks * 2048) / 16, tc_idesc(64, true), add);
            };
            tc_product<NP, 3, 2, 4, 0, 1>(false, qe);
            tc_product<NP, 3, 2, 4, 0, 1>(true, km);
            tc_product<NP, 3, 0, 4, 0>(true, qe);
            tc_product<NP, 3, 0, 4, 0>(true, km);
            tc_commit(done);
        }
        __syncwarp();
        // dg, two steps a lane; then a, b and the sums for A and bias
        double x[2], v[2], base = 0.0;
        for (int w = 0; w < DG_COMPUTE / 32; ++w) base += (double)sh->red[w];
        base *= (double)vec[3 * DL_C];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = 2 * lane + i;
            x[i] = v[i] = 0.0;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                x[i] += sums->hrow[0][q][r] + sums->hrow[1][q][r] - sums->hcol[q][r] + (double)sums->U[q][r];
                v[i] += (double)sums->V[q][r];
            }
        }
        double sum = x[0] + x[1], before = v[0] + v[1];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const double other = __shfl_down_sync(0xffffffffu, sum, o), prior = __shfl_up_sync(0xffffffffu, before, o);
            if (lane + o < 32) sum += other;
            if (lane >= o) before += prior;
        }
        before -= v[0] + v[1];
        const double dg[2] = {base + sum + before, base + (sum - x[0]) + (before + v[0])};
        double sA = 0.0, sb = 0.0;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = 2 * lane + i;
            if (t0 + r >= s.len) continue;
            const int row = sh->rows[r];
            const float da = (float)dg[i] * slope[i];
            sA += dg[i] * (double)soft[i];
            sb += (double)da;
            if (row >= 0) {
                const size_t o = (size_t)(img * p.tokens + row) * p.heads_v + head;
                if (p.da) store_elem(reinterpret_cast<T*>(p.da) + o, da);
                if (p.db) store_elem(reinterpret_cast<T*>(p.db) + o, sh->xw[r] * open[i]);
            }
        }
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            sA += __shfl_xor_sync(0xffffffffu, sA, o);
            sb += __shfl_xor_sync(0xffffffffu, sb, o);
        }
        if (lane == 0) {
            p.wpart[2 * rec] = (float)sA;
            p.wpart[2 * rec + 1] = (float)sb;
        }
        __syncthreads();
        return;
    }
    auto ready = [&](int id) {  // this thread's part of the operands lies in shared (tensor) memory
        tc_fence_smem();
        tc_fence_before();
        bar_arrive(id, DG_THREADS);
    };

    fetch_dy(0);
    // K and Q
    {
        const T* k = reinterpret_cast<const T*>(p.k) + img * p.k_img + (long long)hk * p.dk;
        const T* q = reinterpret_cast<const T*>(p.q) + img * p.q_img + (long long)hk * p.dk;
        grad_load<DKP>(tiles + Sh::oK, k, p.k_tok, sh->rows, p.dk, tid);
        grad_load<DKP>(tiles + Sh::oQ, q, p.q_tok, sh->rows, p.dk, tid);
        cp_async_commit();
    }
    if (NP == 1)  // an exact dO has no second and third term
        for (int i = tid; i < 2 * TC_TILE / 16; i += DG_COMPUTE)
            *reinterpret_cast<uint4*>(tiles + Sh::oX + 2 * TC_TILE + (i >> 9) * 2 * TC_TILE + (i & 511) * 16) = make_uint4(0, 0, 0, 0);

    // what E (P, in its planes) and M (L) are multiplied with for dg: this thread's quarter of a row, fetched ahead as well
    const int part = (warp >> 1) & 1, step = (warp & 1) * 32 + lane, j0 = quarter * 16;
    uint4 factor[6];
    auto fetch_factors = [&]() {
        if (part == 0) {
            const __nv_bfloat16* wP = record_P<T, DKP>(p, rec);
#pragma unroll
            for (int q = 0; q < 6; ++q)
                factor[q] = __ldg(reinterpret_cast<const uint4*>(wP + (q >> 1) * DL_PLANE + plane_at(step, j0 + (q & 1) * 8)));
        } else {
            const uint4* wL = reinterpret_cast<const uint4*>(p.wL + rec * DL_PLANE + step * DL_C + j0);
#pragma unroll
            for (int q = 0; q < 4; ++q) factor[q] = __ldg(wL + q);
        }
    };
    float dots = 0.f;
    float xw[NW] = {};
    for (int slab = 0; slab < p.dv; slab += 64) {
        const bool more = slab > 0;
#pragma unroll
        for (int i = 0; i < NS; ++i) put_planes(tiles + Sh::oS, Sh::plane, pr + STEP * i, pc, s0[i]);
#pragma unroll
        for (int i = 0; i < NW; ++i) {
            const int r = pr + STEP * i;
            xw[i] += w[i].x * x[i].x + w[i].y * x[i].y + w[i].z * x[i].z + w[i].w * x[i].w;
            put_planes(tiles + Sh::oW, TC_TILE, r, pc, w[i]);
            const float beta = vec[2 * DL_C + r];
            put_planes(tiles + Sh::oX + TC_TILE, 2 * TC_TILE, r, pc, make_float4(beta * x[i].x, beta * x[i].y, beta * x[i].z, beta * x[i].w));
            if constexpr (NP == 1)
                *reinterpret_cast<uint2*>(tiles + Sh::oX + r * 128 + (((pc >> 3) ^ (r & 7)) << 4) + (pc & 7) * 2) = o[i];
            else
                put_planes(tiles + Sh::oX, 2 * TC_TILE, r, pc, o[i]);
        }
        if (!more) cp_async_wait<0>();
        ready(1);
        // the gradient of the state leaving the chunk, over the one entering it once D1 has read that
#pragma unroll
        for (int i = 0; i < NS; ++i) dots += ds[i].x * s0[i].x + ds[i].y * s0[i].y + ds[i].z * s0[i].z + ds[i].w * s0[i].w;
        mbar_wait(done, phase, &sh->dead);
        phase ^= 1;
#pragma unroll
        for (int i = 0; i < NS; ++i) put_planes(tiles + Sh::oS, Sh::plane, pr + STEP * i, pc, ds[i]);
        ready(2);
        if (slab + 64 < p.dv) {
            fetch(slab + 64);
            fetch_dy(slab + 64);
        } else {
            fetch_factors();
        }
        mbar_wait(done, phase, &sh->dead);
        phase ^= 1;
    }
#pragma unroll
    for (int i = 0; i < NW; ++i) {
#pragma unroll
        for (int q = 1; q < 16; q <<= 1) xw[i] += __shfl_xor_sync(0xffffffffu, xw[i], q);
        if ((lane & 15) == 0) sh->xw[pr + STEP * i] = xw[i];
    }
    tc_fence_after();
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) dots += __shfl_xor_sync(0xffffffffu, dots, o);
    if (lane == 0) sh->red[warp] = dots;

    // E and M: rows 0-63 of D2 and rows 64-127, columns 16 quarter .. of this thread's step i
    {
        const int i = step;
        float e[16], f[16];
        tc_ld16(tl + c2 + j0, e);
        tc_ld16(tl + c2 + cSmall + j0, f);
        tc_wait_ld();
#pragma unroll
        for (int k = 0; k < 16; ++k) e[k] += f[k];
        if (part == 0) {  // P, whole again
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                float z = 0.f;
#pragma unroll
                for (int n = 2; n >= 0; --n) {
                    const uint4& u = factor[n * 2 + (k >> 3)];
                    const uint32_t a = (k >> 1 & 3) == 0 ? u.x : (k >> 1 & 3) == 1 ? u.y : (k >> 1 & 3) == 2 ? u.z : u.w;
                    z += __uint_as_float(k & 1 ? a & 0xffff0000u : a << 16);
                }
                f[k] = z;
            }
        } else {
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                const uint4& u = factor[k >> 2];
                f[k] = -__uint_as_float((k & 3) == 0 ? u.x : (k & 3) == 1 ? u.y : (k & 3) == 2 ? u.z : u.w);
            }
        }
        // a step's own product carries no decay: it is no part of dg. Blocks above the diagonal
        // hold nothing: selected, not multiplied by zero
        double sum = 0.0, col = 0.0;
        float* h = reinterpret_cast<float*>(tiles + Sh::oS) + warp * (32 * 17);  // this warp's [row][column], over the states
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            f[k] = j0 + k < i ? e[k] * f[k] : 0.f;
            h[lane * 17 + k] = f[k];
            sum += (double)f[k];
        }
        sums->hrow[part][quarter][i] = sum;
        __syncwarp();
#pragma unroll 8
        for (int k = 0; k < 16; ++k) col += (double)h[((lane & 16) + k) * 17 + (lane & 15)];  // half the rows a lane
        col += __shfl_xor_sync(0xffffffffu, col, 16);
        if (lane < 16) sums->hcol[warp & 3][j0 + lane] = col;
        const float2* G = reinterpret_cast<const float2*>(vec + 4 * DL_C);
        const float2 gi = G[i];
        const float sign = part == 0 ? p.scale : -1.f;
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            const float2 gj = G[j0 + k];
            const float d = decay_between<NP == 1>(gi, gj);
            e[k] = j0 + k <= i - part ? sign * (d * e[k]) : 0.f;
        }
        unsigned char* o = tiles + Sh::oX + part * TC_TILE;
#pragma unroll
        for (int k = 0; k < 16; k += 4) put_planes(o, 2 * TC_TILE, i, j0 + k, make_float4(e[k], e[k + 1], e[k + 2], e[k + 3]));
    }
    // D1 and D3, scaled, and their part of dg
    const int dk = (warp & 3) * 32 + lane;
    const bool live = dk < DKP;  // DKP = 64: the upper two warps of each four idle here
    float dq[16], dkr[16], dkc[16];
    {
        float u[32], x[16];  // U's and V's parts
        tc_ld16(tl + c1 + j0, dq);
        tc_ld16(tl + c1 + cSmall + j0, x);
        tc_wait_ld();
#pragma unroll
        for (int i = 0; i < 16; ++i) dq[i] += x[i];
        tc_ld16(tl + c1 + 64 + j0, dkr);
        tc_ld16(tl + c1 + cSmall + 64 + j0, x);
        tc_wait_ld();
#pragma unroll
        for (int i = 0; i < 16; ++i) dkr[i] += x[i];
        tc_ld16(tl + c3 + j0, dkc);
        tc_ld16(tl + c3 + cSmall + j0, x);
        tc_wait_ld();
#pragma unroll
        for (int i = 0; i < 16; ++i) dkc[i] += x[i];
        if (live) column_of<NP, DKP>(tiles + Sh::oQ, Sh::plane, dk, j0, x);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float eG = vec[j0 + i];
            dq[i] *= p.scale * eG;
            dkr[i] *= -eG;
            dkc[i] *= vec[DL_C + j0 + i];
            u[i] = live ? x[i] * dq[i] : 0.f;
        }
        if (live) column_of<NP, DKP>(tiles + Sh::oK, Sh::plane, dk, j0, x);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            u[i] += live ? x[i] * dkr[i] : 0.f;
            u[16 + i] = live ? x[i] * dkc[i] : 0.f;
        }
        (lane < 16 ? sums->U : sums->V)[warp & 3][j0 + (lane & 15)] = reduce_columns(u, lane);
    }
    tc_fence_before();
    bar_sync(4, DG_COMPUTE);  // the parts of dg are there, and the columns behind cSmall read
    tc_fence_after();
    // K^T and Q^T: this thread's key channel, half the steps of one of them
    {
        const int which = quarter & 1, h = quarter >> 1;
        if ((warp & 3) * 32 < DKP) {
            float x[32];
            column_of<NP, DKP>(tiles + (which ? Sh::oQ : Sh::oK), Sh::plane, dk, h * 32, x);
            put_terms<NP, NP == 3>(tl + (which ? cQT : cKT) + h * 16, 32, x);
        }
    }
    tc_wait_st();
    ready(3);
    mbar_wait(done, phase, &sh->dead);
    tc_fence_after();
    {
        float x[16];
        tc_ld16(tl + c1 + j0, x);
        tc_wait_ld();
#pragma unroll
        for (int i = 0; i < 16; ++i) dq[i] += x[i];
        tc_ld16(tl + c1 + 64 + j0, x);
        tc_wait_ld();
#pragma unroll
        for (int i = 0; i < 16; ++i) dkr[i] += x[i];
        tc_ld16(tl + c3 + j0, x);
        tc_wait_ld();
#pragma unroll
        for (int i = 0; i < 16; ++i) dkc[i] += dkr[i] + x[i];
    }
    start_next();
    // rows out, over the states' place
    const int* rows = sh->rows + j0;
    const size_t first = (size_t)img * p.tokens;
    if ((warp & 3) * 32 < DKP) {
        const int have = p.dk - (warp & 3) * 32;
        if (p.wdq) {
            float* mine = reinterpret_cast<float*>(tiles + Sh::oS) + warp * (16 * 36) + lane;
            const long long tok = (long long)p.heads_v * p.dk;
            const size_t o = (first * p.heads_v + head) * p.dk + (warp & 3) * 32;
            walk_store(p.wdq + o, tok, rows, mine, 36, have, lane, dq);
            __syncwarp();
            walk_store(p.wdk + o, tok, rows, mine, 36, have, lane, dkc);
        } else {
            constexpr int pitch = 32 + 16 / (int)sizeof(T);
            T* mine = reinterpret_cast<T*>(tiles + Sh::oS) + warp * (16 * pitch) + lane;
            const long long tok = (long long)p.heads_k * p.dk;
            const size_t o = (first * p.heads_k + hk) * p.dk + (warp & 3) * 32;
            if (p.dq) walk_store(reinterpret_cast<T*>(p.dq) + o, tok, rows, mine, pitch, have, lane, dq);
            __syncwarp();
            if (p.dkey) walk_store(reinterpret_cast<T*>(p.dkey) + o, tok, rows, mine, pitch, have, lane, dkc);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (tid == 0 && p.status && sh->dead) atomicOr(p.status, DEV_STATUS_TIMEOUT);
    if (warp == 0) tc_free(tm, &sh->dead);
}

// dA and dbias of one head: its chunks' sums added in a fixed order.
__global__ void __launch_bounds__(256) delta_param_grad_kernel(const DeltaParams p)
{
    __shared__ double part[2][8];
    const int head = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    wait_previous();
    double sA = 0.0, sb = 0.0;
    for (long long i = tid; i < p.slots; i += 256) {
        const float2 x = *reinterpret_cast<const float2*>(p.wpart + 2 * ((size_t)i * p.heads_v + head));
        sA += x.x;
        sb += x.y;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        sA += __shfl_down_sync(0xffffffffu, sA, o);
        sb += __shfl_down_sync(0xffffffffu, sb, o);
    }
    if (lane == 0) { part[0][warp] = sA; part[1][warp] = sb; }
    __syncthreads();
    if (tid == 0) {
        sA = sb = 0.0;
        for (int w = 0; w < 8; ++w) { sA += part[0][w]; sb += part[1][w]; }
        if (p.dA) p.dA[head] = (float)sA;
        if (p.dbias) p.dbias[head] = (float)sb;
    }
}

// dq and dk of a shared key head: its value heads' parts added in order.
template <typename T>
__global__ void __launch_bounds__(256) delta_group_kernel(const DeltaParams p, long long vecs)
{
    wait_previous();
    start_next();
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;  // four channels of one row and key head
    if (i >= vecs) return;
    const int per = p.dk / 4;
    const long long rh = i / per;
    const int c = (int)(i - rh * per) * 4;
    const float* src = blockIdx.y ? p.wdk : p.wdq;
    T* dst = reinterpret_cast<T*>(blockIdx.y ? p.dkey : p.dq);
    if (!dst) return;
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int g = 0; g < p.group; ++g) {
        const float4 x = __ldg(reinterpret_cast<const float4*>(src + (rh * p.group + g) * p.dk + c));
        sum.x += x.x; sum.y += x.y; sum.z += x.z; sum.w += x.w;
    }
    store4(dst + rh * p.dk + c, sum);
}

}  // namespace vscan
