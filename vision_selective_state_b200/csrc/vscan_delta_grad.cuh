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
    unsigned char* stages = smem + 1024;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int head = blockIdx.y, b = blockIdx.z;
    const int slice = blockIdx.x * 128;
    const DeltaSeq s = delta_seq(p, b);
    const int chunks = (s.len + DL_C - 1) / DL_C;
    const size_t sbase = ((size_t)b * p.heads_v + head) * p.dk * p.dv;
    const WalkBars bar(ws);
    const uint32_t tm = walk_begin(ws, bar);
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
                const uint64_t dK = tc_desc(bK), dQ = tc_desc(bK + Sh::oQ), dT = tc_desc(bK + Sh::oT), dP = tc_desc(bK + Sh::oP);
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
                auto state = [&](auto a, uint64_t t, bool more) {
#pragma unroll
                    for (int nb = 0; nb < Sh::KB; ++nb)
                        tc_product<3, NP, 2, 4, 0>(more, [&](int x, int y, int ks, bool add) {
                            tc_mma(tm + cDS + nb * (3 * Sh::SC), a(x, ks),
                                   t + (y * Sh::plane + nb * TC_TILE + ks * 2048) / 16, tc_idesc(64, true), add);
                        });
                };
                bar_sync(4, DW_COMPUTE + 32);
                tc_fence_after();
                if (tc_elect()) state(aQ, dQ, false);  // 3
                __syncwarp();
                bar_sync(5, DW_COMPUTE + 32);
                tc_fence_after();
                if (tc_elect()) {
                    state(aW, dK, true);
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
                    walk_load<DKP>(base, k, p.k_tok, rows, p.dk, ht);
                    walk_load<DKP>(base + Sh::oQ, q, p.q_tok, rows, p.dk, ht);
                    walk_load_values(reinterpret_cast<T*>(base + Sh::oV(3)), Sh::vpitch, dy, p.y_tok, rows, dvs, ht);
                    uint32_t bytes = 0;
                    if (ht == 0) {
                        bytes = DL_VECS * 4 + 6 * TC_TILE;
                        bulk_in(at + Sh::oVec, record_vec(p, rec), bytes, full);
                    }
                    return bytes;
                });
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(DW_REGS_COMPUTE));
        const int half = warp >> 2, row = (warp & 3) * 32 + lane, vc = slice + row;
        const bool live = vc < p.dv;
        const uint32_t tl = tm + ((uint32_t)(warp & 3) << 21);
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
            const float* vec = reinterpret_cast<const float*>(stages + st * STAGE + Sh::oVec) + half * 32;
            const size_t rec = (size_t)(s.slot + chunks - 1 - n) * p.heads_v + head;
            float o[32], x[32];
            mbar_wait(bar.full + 8 * st, (n / STAGES) & 1, &ws->dead);
#pragma unroll
            for (int i = 0; i < 32; ++i) x[i] = o[i] = to_float(vd[i * Sh::vpitch]);
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
#pragma unroll
                for (int i = 0; i < 32; ++i) x[i] = vec[DL_C + i] * x[i] + z[i];
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
            if (live) {
                float* ox = p.wdX + (rec * DL_C + half * 32) * p.dv + vc;
#pragma unroll
                for (int i = 0; i < 32; ++i) ox[(size_t)i * p.dv] = x[i];
            }
#pragma unroll
            for (int i = 0; i < 32; ++i) x[i] *= vec[2 * DL_C + i];  // dV
            {
                float u[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) u[i] = x[i] * -vec[i];
                put_terms<3>(tl + cW + half * 48, 16, u);
            }
            walk_ready(5);
            if (dvalue)
                walk_store(dvalue, (long long)p.heads_v * p.dv, ws->rows[n % 3] + half * 32, vd, Sh::vpitch, p.dv - vc + lane, lane, x);
            const float eC = vec[3 * DL_C - half * 32];
            mbar_wait(bar.done + 16, par, &ws->dead);
            tc_fence_after();
#pragma unroll
            for (int i = 0; i < HS; i += 32) {
                tc_ld32(tl + cDS + (DKP == 128 ? half * 3 * Sh::SC : half * 32) + i, x);
                tc_wait_ld();
#pragma unroll
                for (int e = 0; e < 32; ++e) S[i + e] = eC * S[i + e] + x[e];
            }
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
// One CTA of eight warps per chunk and value head: four row blocks of 16 steps
// times two halves of the key channels (of the steps j for E and M). The states
// pass through shared memory in slabs of 64 value channels, split into bf16
// terms once for all warps; dO, X's gradient and W go to registers directly.
template <typename T, int DKP>
struct GradShape {
    static constexpr int NP = DeltaIo<T>::planes;
    static constexpr int pitch = DKP + 8;
    static constexpr int plane = DL_C * pitch;
    static constexpr int splane = DKP * DL_TPITCH;  // a slab of a state: [DKP][64 value channels]
    // K, Q; a slab of a state, E and M in three planes each; row sums
    static constexpr size_t smem = (size_t)2 * NP * plane * 2 + (size_t)3 * splane * 2 + (size_t)6 * DL_C * DL_TPITCH * 2 +
                                   6 * DL_C * 8 + (5 * DL_C + 16) * 4;
};

__device__ __forceinline__ float2 load_pair(const float* p) { return __ldg(reinterpret_cast<const float2*>(p)); }
__device__ __forceinline__ float2 load_pair(const __nv_bfloat16* p)
{
    const uint32_t u = __ldg(reinterpret_cast<const uint32_t*>(p));
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}
__device__ __forceinline__ void store_pair(float* p, float x, float y) { *reinterpret_cast<float2*>(p) = make_float2(x, y); }
__device__ __forceinline__ void store_pair(__nv_bfloat16* p, float x, float y)
{
    *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(x, y);
}

template <typename T, int DKP>
__global__ void __launch_bounds__(256) delta_grad_kernel(const DeltaParams p)
{
    using Sh = GradShape<T, DKP>;
    constexpr int NP = Sh::NP, PITCH = Sh::pitch, PLANE = Sh::plane;
    constexpr int NH = DKP / 16;  // 8-wide tiles in half of the key channels (2 at DKP = 32)
    extern __shared__ __align__(16) unsigned char smem[];
    double* hrow = reinterpret_cast<double*>(smem);  // [2 halves][64] row sums of H
    double* hcol = hrow + 2 * DL_C;                  // [4 row blocks][64] column sums of H
    float* rows = reinterpret_cast<float*>(hcol + 4 * DL_C);  // [2 halves][64] U, then V; [64] dX.w
    float* red = rows + 5 * DL_C;                    // [8] <dS, S0>
    __nv_bfloat16* K = reinterpret_cast<__nv_bfloat16*>(red + 16);
    __nv_bfloat16* Q = K + NP * PLANE;
    __nv_bfloat16* St = Q + NP * PLANE;
    __nv_bfloat16* E = St + 3 * Sh::splane;
    __nv_bfloat16* M = E + 3 * DL_C * DL_TPITCH;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gr = lane >> 2, tc = (lane & 3) * 2;
    const int head = blockIdx.y, hk = head / p.group;
    const int m0 = (warp & 3) * 16, half = warp >> 2, n0 = half * (DKP / 2);

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
    const float* vec = record_vec(p, rec);
    const float* wS = p.wS + rec * p.dv * DKP;
    const float* wdS = p.wdS + rec * p.dv * DKP;
    const float* wW = p.wW + rec * DL_C * p.dv;
    const float* wdX = p.wdX + rec * DL_C * p.dv;

    load_tile(K, PITCH, PLANE, reinterpret_cast<const T*>(p.k) + img * p.k_img + (long long)hk * p.dk, p.k_tok, p, s, t0,
              DKP, p.dk, tid, 256);
    load_tile(Q, PITCH, PLANE, reinterpret_cast<const T*>(p.q) + img * p.q_img + (long long)hk * p.dk, p.q_tok, p, s, t0,
              DKP, p.dk, tid, 256);
    cp_async_commit();

    // this thread's two rows of the chunk
    const int r0 = m0 + gr, r1 = r0 + 8;
    const int row0 = delta_row(p, s, t0 + r0), row1 = delta_row(p, s, t0 + r1);
    const T* dy = reinterpret_cast<const T*>(p.dy) + img * p.y_img + (long long)head * p.dv;
    const float eG0 = vec[r0], eG1 = vec[r1], eD0 = vec[DL_C + r0], eD1 = vec[DL_C + r1];
    const float beta0 = vec[2 * DL_C + r0], beta1 = vec[2 * DL_C + r1];

    float dq[NH][4] = {}, dkr[NH][4] = {}, dkc[NH][4] = {}, e[4][4] = {}, m[4][4] = {};
    float xw0 = 0.f, xw1 = 0.f, dots = 0.f;
    for (int slab = 0; slab < p.dv; slab += DL_C) {
        const int cols = min(DL_C, p.dv - slab);
        auto load_state = [&](const float* src, const float* other) {
            for (int i = tid; i < DKP * (DL_C / 4); i += 256) {
                const int r = i / (DL_C / 4), cc = (i - r * (DL_C / 4)) * 4;
                float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
                if (cc < cols) {
                    x = __ldg(reinterpret_cast<const float4*>(src + (size_t)r * p.dv + slab + cc));
                    if (other) {
                        const float4 z = __ldg(reinterpret_cast<const float4*>(other + (size_t)r * p.dv + slab + cc));
                        dots += x.x * z.x + x.y * z.y + x.z * z.z + x.w * z.w;
                    }
                }
#pragma unroll
                for (int n = 0; n < 3; ++n) {
                    uint2 u;
                    u.x = split_bf16(x.x, x.y);
                    u.y = split_bf16(x.z, x.w);
                    *reinterpret_cast<uint2*>(St + n * Sh::splane + r * DL_TPITCH + cc) = u;
                }
            }
        };
        // rows r0, r1 at columns col and col + 8 of a [64][dv] array, as two C tiles
        auto rows_of = [&](const float* src, int col, float (&lo)[4], float (&hi)[4]) {
            const float2 z = make_float2(0.f, 0.f);
            const float2 a = col < p.dv ? load_pair(src + (size_t)r0 * p.dv + col) : z;
            const float2 bb = col < p.dv ? load_pair(src + (size_t)r1 * p.dv + col) : z;
            const float2 cc = col + 8 < p.dv ? load_pair(src + (size_t)r0 * p.dv + col + 8) : z;
            const float2 d = col + 8 < p.dv ? load_pair(src + (size_t)r1 * p.dv + col + 8) : z;
            lo[0] = a.x; lo[1] = a.y; lo[2] = bb.x; lo[3] = bb.y;
            hi[0] = cc.x; hi[1] = cc.y; hi[2] = d.x; hi[3] = d.y;
        };
        load_state(wS, nullptr);
        cp_async_wait<0>();
        __syncthreads();
        for (int kt = 0; kt * 16 < cols; ++kt) {
            const int col = slab + kt * 16 + tc;
            float lo[4], hi[4], wl[4], wh[4];
            Frag4 oa[NP], va[3];
            {
                const float2 z = make_float2(0.f, 0.f);
                const float2 a = row0 >= 0 && col < p.dv ? load_pair(dy + row0 * p.y_tok + col) : z;
                const float2 bb = row1 >= 0 && col < p.dv ? load_pair(dy + row1 * p.y_tok + col) : z;
                const float2 cc = row0 >= 0 && col + 8 < p.dv ? load_pair(dy + row0 * p.y_tok + col + 8) : z;
                const float2 d = row1 >= 0 && col + 8 < p.dv ? load_pair(dy + row1 * p.y_tok + col + 8) : z;
                lo[0] = a.x; lo[1] = a.y; lo[2] = bb.x; lo[3] = bb.y;
                hi[0] = cc.x; hi[1] = cc.y; hi[2] = d.x; hi[3] = d.y;
            }
            split_tiles<NP>(lo, hi, oa);
            rows_of(wdX, col, lo, hi);
            rows_of(wW, col, wl, wh);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                xw0 += lo[i] * wl[i] + hi[i] * wh[i];
                xw1 += lo[2 + i] * wl[2 + i] + hi[2 + i] * wh[2 + i];
                lo[i] *= beta0; hi[i] *= beta0;
                lo[2 + i] *= beta1; hi[2 + i] *= beta1;
            }
            split_tiles<3>(lo, hi, va);
            // dO S0^T and dV S0^T
#pragma unroll
            for (int nt = 0; nt < NH; nt += 2) {
                Frag4 f[3];
#pragma unroll
                for (int n = 0; n < 3; ++n) f[n] = load_b(St + n * Sh::splane, DL_TPITCH, n0 + nt * 8, kt * 16, lane);
                mma_terms<NP, 3>(dq[nt], dq[nt + 1], oa, f);
                mma_terms<3, 3>(dkr[nt], dkr[nt + 1], va, f);
            }
            // dO W^T and dV W^T, columns 32 half .. of the steps j up to this row block
#pragma unroll
            for (int nt = 0; nt < 4; nt += 2) {
                const int j = half * 32 + nt * 8;
                if (j <= m0 + 15) {
                    float b0[4], b1[4];  // step j + gr, then j + 8 + gr: channels col.. and col + 8..
                    const float2 z = make_float2(0.f, 0.f);
                    const float2 w00 = col < p.dv ? load_pair(wW + (size_t)(j + gr) * p.dv + col) : z;
                    const float2 w01 = col + 8 < p.dv ? load_pair(wW + (size_t)(j + gr) * p.dv + col + 8) : z;
                    const float2 w10 = col < p.dv ? load_pair(wW + (size_t)(j + 8 + gr) * p.dv + col) : z;
                    const float2 w11 = col + 8 < p.dv ? load_pair(wW + (size_t)(j + 8 + gr) * p.dv + col + 8) : z;
                    b0[0] = w00.x; b0[1] = w00.y; b0[2] = w01.x; b0[3] = w01.y;
                    b1[0] = w10.x; b1[1] = w10.y; b1[2] = w11.x; b1[3] = w11.y;
                    Frag4 f[3];
                    split_tiles<3>(b0, b1, f);
                    mma_terms<NP, 3>(e[nt], e[nt + 1], oa, f);
                    mma_terms<3, 3>(m[nt], m[nt + 1], va, f);
                }
            }
        }
        __syncthreads();
        load_state(wdS, wS);
        __syncthreads();
        for (int kt = 0; kt * 16 < cols; ++kt) {  // W dS^T
            float lo[4], hi[4];
            rows_of(wW, slab + kt * 16 + tc, lo, hi);
            Frag4 wa[3];
            split_tiles<3>(lo, hi, wa);
#pragma unroll
            for (int nt = 0; nt < NH; nt += 2) {
                Frag4 f[3];
#pragma unroll
                for (int n = 0; n < 3; ++n) f[n] = load_b(St + n * Sh::splane, DL_TPITCH, n0 + nt * 8, kt * 16, lane);
                mma_terms<3, 3>(dkc[nt], dkc[nt + 1], wa, f);
            }
        }
        __syncthreads();
    }

    // the decays, and E and M to shared memory
    auto k_at = [&](const __nv_bfloat16* t, int r, int col) {  // a pair of the tile's values
        float2 x = make_float2(0.f, 0.f);
#pragma unroll
        for (int n = NP - 1; n >= 0; --n) {
            const __nv_bfloat162 h = *reinterpret_cast<const __nv_bfloat162*>(t + n * PLANE + r * PITCH + col);
            x.x += __low2float(h);
            x.y += __high2float(h);
        }
        return x;
    };
    float u0 = 0.f, u1 = 0.f, v0 = 0.f, v1 = 0.f;  // this thread's part of U and V of its rows
#pragma unroll
    for (int nt = 0; nt < NH; ++nt) {
        const int col = n0 + nt * 8 + tc;
        const float2 k0 = k_at(K, r0, col), k1 = k_at(K, r1, col), q0 = k_at(Q, r0, col), q1 = k_at(Q, r1, col);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            dq[nt][i] *= p.scale * (i < 2 ? eG0 : eG1);
            dkr[nt][i] *= -(i < 2 ? eG0 : eG1);
            dkc[nt][i] *= i < 2 ? eD0 : eD1;
        }
        u0 += q0.x * dq[nt][0] + q0.y * dq[nt][1] + k0.x * dkr[nt][0] + k0.y * dkr[nt][1];
        u1 += q1.x * dq[nt][2] + q1.y * dq[nt][3] + k1.x * dkr[nt][2] + k1.y * dkr[nt][3];
        v0 += k0.x * dkc[nt][0] + k0.y * dkc[nt][1];
        v1 += k1.x * dkc[nt][2] + k1.y * dkc[nt][3];
    }
    {
        const double* G = reinterpret_cast<const double*>(vec + 4 * DL_C);
        const double g0 = G[r0], g1 = G[r1];
        const __nv_bfloat16* wP = record_P(p, rec);
        const float* wL = p.wL + rec * DL_PLANE;
        double hr0 = 0.0, hr1 = 0.0;
#pragma unroll
        for (int nt = 0; nt < 4; ++nt) {
            const int j = half * 32 + nt * 8 + tc;
            float ev[4], mv[4];
            double hc[2] = {0.0, 0.0};
            if (j <= r1) {
                float pv[4] = {}, lv[4];
#pragma unroll
                for (int n = 2; n >= 0; --n) {
                    const float2 x = load_pair(wP + n * DL_PLANE + plane_at(r0, j));
                    const float2 z = load_pair(wP + n * DL_PLANE + plane_at(r1, j));
                    pv[0] += x.x; pv[1] += x.y; pv[2] += z.x; pv[3] += z.y;
                }
                const float2 l0 = load_pair(wL + r0 * DL_C + j), l1 = load_pair(wL + r1 * DL_C + j);
                lv[0] = l0.x; lv[1] = l0.y; lv[2] = l1.x; lv[3] = l1.y;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int r = i < 2 ? r0 : r1, jj = j + (i & 1);
                    // a step's own product carries no decay: it is no part of dg
                    const float h = jj < r ? e[nt][i] * pv[i] - m[nt][i] * lv[i] : 0.f;
                    (i < 2 ? hr0 : hr1) += (double)h;
                    hc[i & 1] += (double)h;
                }
            }
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) {
                hc[0] += __shfl_xor_sync(0xffffffffu, hc[0], o);
                hc[1] += __shfl_xor_sync(0xffffffffu, hc[1], o);
            }
            if (gr == 0) {
                hcol[(warp & 3) * DL_C + j] = hc[0];
                hcol[(warp & 3) * DL_C + j + 1] = hc[1];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = i < 2 ? r0 : r1, jj = j + (i & 1);
                const float d = jj <= r ? exp_diff((i < 2 ? g0 : g1) - G[jj]) : 0.f;
                ev[i] = jj <= r ? p.scale * (d * e[nt][i]) : 0.f;
                mv[i] = jj < r ? -d * m[nt][i] : 0.f;
            }
#pragma unroll
            for (int n = 0; n < 3; ++n) {
                __nv_bfloat16 *eo = E + n * DL_C * DL_TPITCH, *mo = M + n * DL_C * DL_TPITCH;
                *reinterpret_cast<uint32_t*>(eo + r0 * DL_TPITCH + j) = split_bf16(ev[0], ev[1]);
                *reinterpret_cast<uint32_t*>(eo + r1 * DL_TPITCH + j) = split_bf16(ev[2], ev[3]);
                *reinterpret_cast<uint32_t*>(mo + r0 * DL_TPITCH + j) = split_bf16(mv[0], mv[1]);
                *reinterpret_cast<uint32_t*>(mo + r1 * DL_TPITCH + j) = split_bf16(mv[2], mv[3]);
            }
        }
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
            hr0 += __shfl_xor_sync(0xffffffffu, hr0, o);
            hr1 += __shfl_xor_sync(0xffffffffu, hr1, o);
            u0 += __shfl_xor_sync(0xffffffffu, u0, o);
            u1 += __shfl_xor_sync(0xffffffffu, u1, o);
            v0 += __shfl_xor_sync(0xffffffffu, v0, o);
            v1 += __shfl_xor_sync(0xffffffffu, v1, o);
            xw0 += __shfl_xor_sync(0xffffffffu, xw0, o);
            xw1 += __shfl_xor_sync(0xffffffffu, xw1, o);
        }
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) dots += __shfl_xor_sync(0xffffffffu, dots, o);
        if ((lane & 3) == 0) {
            hrow[half * DL_C + r0] = hr0;
            hrow[half * DL_C + r1] = hr1;
            rows[half * DL_C + r0] = u0;
            rows[half * DL_C + r1] = u1;
            rows[(2 + half) * DL_C + r0] = v0;
            rows[(2 + half) * DL_C + r1] = v1;
            if (half == 0) {
                rows[4 * DL_C + r0] = xw0;
                rows[4 * DL_C + r1] = xw1;
            }
        }
        if (lane == 0) red[warp] = dots;
    }
    __syncthreads();
    // dq += E K, dkr += M K over the steps up to the row block
    for (int kt = 0; kt * 16 <= m0; ++kt) {
        Frag4 ea[3], ma[3];
#pragma unroll
        for (int n = 0; n < 3; ++n) {
            ea[n] = load_a(E + n * DL_C * DL_TPITCH, DL_TPITCH, m0, kt * 16, lane);
            ma[n] = load_a(M + n * DL_C * DL_TPITCH, DL_TPITCH, m0, kt * 16, lane);
        }
#pragma unroll
        for (int nt = 0; nt < NH; nt += 2) {
            Frag4 f[NP];
#pragma unroll
            for (int n = 0; n < NP; ++n) f[n] = load_b_t(K + n * PLANE, PITCH, n0 + nt * 8, kt * 16, lane);
            mma_terms<3, NP>(dq[nt], dq[nt + 1], ea, f);
            mma_terms<3, NP>(dkr[nt], dkr[nt + 1], ma, f);
        }
    }
    // dkc += E^T Q + M^T K over the steps from the row block on
    for (int kt = m0 / 16; kt < 4; ++kt) {
        Frag4 ea[3], ma[3];
#pragma unroll
        for (int n = 0; n < 3; ++n) {
            ea[n] = load_a_t(E + n * DL_C * DL_TPITCH, DL_TPITCH, m0, kt * 16, lane);
            ma[n] = load_a_t(M + n * DL_C * DL_TPITCH, DL_TPITCH, m0, kt * 16, lane);
        }
#pragma unroll
        for (int nt = 0; nt < NH; nt += 2) {
            Frag4 f[NP];
#pragma unroll
            for (int n = 0; n < NP; ++n) f[n] = load_b_t(Q + n * PLANE, PITCH, n0 + nt * 8, kt * 16, lane);
            mma_terms<3, NP>(dkc[nt], dkc[nt + 1], ea, f);
#pragma unroll
            for (int n = 0; n < NP; ++n) f[n] = load_b_t(K + n * PLANE, PITCH, n0 + nt * 8, kt * 16, lane);
            mma_terms<3, NP>(dkc[nt], dkc[nt + 1], ma, f);
        }
    }
    // rows out
#pragma unroll
    for (int nt = 0; nt < NH; ++nt) {
        const int col = n0 + nt * 8 + tc;
        if (col < p.dk) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int row = h ? row1 : row0;
                if (row < 0) continue;
                const float x0 = dkr[nt][2 * h] + dkc[nt][2 * h], x1 = dkr[nt][2 * h + 1] + dkc[nt][2 * h + 1];
                const size_t at = (size_t)(img * p.tokens + row);
                if (p.wdq) {
                    const size_t o = (at * p.heads_v + head) * p.dk + col;
                    store_pair(p.wdq + o, dq[nt][2 * h], dq[nt][2 * h + 1]);
                    store_pair(p.wdk + o, x0, x1);
                } else {
                    const size_t o = (at * p.heads_k + hk) * p.dk + col;
                    if (p.dq) store_pair(reinterpret_cast<T*>(p.dq) + o, dq[nt][2 * h], dq[nt][2 * h + 1]);
                    if (p.dkey) store_pair(reinterpret_cast<T*>(p.dkey) + o, x0, x1);
                }
            }
        }
    }
    if (warp == 0) {  // dg, two steps a lane; then a, b and the sums for A and bias
        double x[2], v[2], base = 0.0;
        for (int w = 0; w < 8; ++w) base += (double)red[w];
        base *= (double)vec[3 * DL_C];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = 2 * lane + i;
            x[i] = hrow[r] + hrow[DL_C + r] - (hcol[r] + hcol[DL_C + r] + hcol[2 * DL_C + r] + hcol[3 * DL_C + r]) +
                   (double)rows[r] + (double)rows[DL_C + r];
            v[i] = (double)rows[2 * DL_C + r] + (double)rows[3 * DL_C + r];
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
        const float A = p.A[head], bias = p.bias ? p.bias[head] : 0.f;
        double sA = 0.0, sb = 0.0;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = 2 * lane + i;
            if (t0 + r >= s.len) continue;
            const int row = delta_row(p, s, t0 + r);
            const float a = row >= 0 ? to_float(reinterpret_cast<const T*>(p.a)[img * p.a_img + row * p.a_tok + head]) : 0.f;
            const float da = (float)dg[i] * A * delta_sigmoid(a + bias);
            sA += dg[i] * (double)delta_softplus(a + bias);
            sb += (double)da;
            if (row >= 0) {
                const size_t o = (size_t)(img * p.tokens + row) * p.heads_v + head;
                const float bb = to_float(reinterpret_cast<const T*>(p.b)[img * p.b_img + row * p.b_tok + head]);
                if (p.da) store_elem(reinterpret_cast<T*>(p.da) + o, da);
                if (p.db) store_elem(reinterpret_cast<T*>(p.db) + o, rows[4 * DL_C + r] * delta_sigmoid(-bb));
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
    }
}

// dA and dbias of one head: its chunks' sums added in a fixed order.
__global__ void __launch_bounds__(256) delta_param_grad_kernel(const DeltaParams p)
{
    __shared__ double part[2][8];
    const int head = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
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
