// C ABI of the query/key norm with position rotation (declared in include/vscan.h):
// argument checks, variant selection and launch. Every check runs before the
// first CUDA call, so a rejected call launches nothing.
#include <algorithm>
#include <cmath>

#include "vscan.h"
#include "vscan_host.h"
#include "vscan_qknorm.cuh"

namespace {

using vscan::QkNormParams;
using vscan_host::aligned16;
using vscan_host::cuda_fail;
using vscan_host::fail;
using vscan_host::launch_after;
using vscan_host::NvtxRange;

// CTAs of q and as many of k. Forward two rounds of the four CTAs of 256 threads that an SM holds: 64
// images of 4097 tokens, 6 + 6 heads of 128, bf16: 308 us (one round: 318). Backward half as many, since
// every CTA pays for its sums of the weights' gradients; the kernel's 70 to 80 registers let three CTAs
// share an SM, so that 444 of the 592 run at once, and those of the side with fewer heads end early.
// The best of what was measured on 16 images of 3136 tokens, 12 + 4 heads of 72: 136 us (262 CTAs a
// side: 154; 370: 147; 740: 155).
int most_blocks(bool back) { return 148 * (back ? 2 : 4); }

vscan_status check_stride(const char* name, int64_t tok, int64_t img, int64_t width, int vec)
{
    if (tok < 0 || img < 0) return fail(VSCAN_ERR_INVALID_ARGUMENT, "%s strides must be >= 0 (0 = dense)", name);
    if ((tok != 0 && tok < width) || tok % vec != 0 || img % vec != 0)
        return fail(VSCAN_ERR_ALIGNMENT, "%s strides %lld, %lld: at least %lld a token, multiples of %d", name, (long long)tok,
                    (long long)img, (long long)width, vec);
    return VSCAN_OK;
}

vscan_status check_shape(const vscan_qknorm_args* a)
{
    if (!a) return fail(VSCAN_ERR_INVALID_ARGUMENT, "args is NULL");
    if (a->dtype != VSCAN_F32 && a->dtype != VSCAN_BF16)
        return fail(VSCAN_ERR_INVALID_ARGUMENT, "unknown dtype %d", a->dtype);
    if (a->norm != VSCAN_NORM_L2 && a->norm != VSCAN_NORM_RMS)
        return fail(VSCAN_ERR_INVALID_ARGUMENT, "unknown norm %d", a->norm);
    if (a->batch < 0 || a->tokens < 0)
        return fail(VSCAN_ERR_INVALID_ARGUMENT, "batch %d and tokens %d must be >= 0", a->batch, a->tokens);
    if (a->heads_q < 1 || a->heads_k < 1 || a->dim < 1)
        return fail(VSCAN_ERR_INVALID_ARGUMENT, "heads_q %d, heads_k %d and dim %d must be >= 1", a->heads_q, a->heads_k, a->dim);
    const int vec = a->dtype == VSCAN_F32 ? 4 : 8;
    if (a->dim % vec != 0)
        return fail(VSCAN_ERR_ALIGNMENT, "dim %d is not a multiple of %d (16-byte rows)", a->dim, vec);
    if (a->dim > 2 * vscan::QN_MAX_PAIRS) return fail(VSCAN_ERR_UNSUPPORTED, "dim %d > %d", a->dim, 2 * vscan::QN_MAX_PAIRS);
    // rows of a position, which a lane counts in steps of at most 512, in 32 bits
    if ((int64_t)a->batch * ((int64_t)a->heads_q + a->heads_k) > 0x7fffffffLL - 1024)
        return fail(VSCAN_ERR_UNSUPPORTED, "batch x (heads_q + heads_k) must be below 2^31 - 1024");
    if (!(a->eps >= 0.f) || !std::isfinite(a->eps)) return fail(VSCAN_ERR_INVALID_ARGUMENT, "eps must be finite and >= 0");
    if (a->reserved != 0) return fail(VSCAN_ERR_INVALID_ARGUMENT, "args.reserved must be 0");
    if (a->pos_per_image != 0 && a->pos_per_image != 1)
        return fail(VSCAN_ERR_INVALID_ARGUMENT, "pos_per_image must be 0 or 1");
    if (a->pairs < 0 || a->pairs > a->dim / 2)
        return fail(VSCAN_ERR_SHAPE, "pairs %d is not within 0 .. dim / 2 = %d", a->pairs, a->dim / 2);
    if (a->axes != 1 && a->axes != 2) return fail(VSCAN_ERR_SHAPE, "axes %d is not 1 or 2", a->axes);
    if (a->pairs % a->axes != 0) return fail(VSCAN_ERR_SHAPE, "pairs %d is not a multiple of axes %d", a->pairs, a->axes);
    if ((int64_t)a->tokens * a->axes > 0x7fffffffLL)
        return fail(VSCAN_ERR_UNSUPPORTED, "tokens x axes must be below 2^31");
    if (a->pairs && (!a->inv_freq || !a->positions))
        return fail(VSCAN_ERR_INVALID_ARGUMENT, "pairs %d without inv_freq and positions", a->pairs);
    const int64_t wq = (int64_t)a->heads_q * a->dim, wk = (int64_t)a->heads_k * a->dim;
    vscan_status st;
    if ((st = check_stride("q", a->q_tok_stride, a->q_batch_stride, wq, vec)) != VSCAN_OK) return st;
    if ((st = check_stride("k", a->k_tok_stride, a->k_batch_stride, wk, vec)) != VSCAN_OK) return st;
    if ((st = check_stride("yq", a->yq_tok_stride, a->yq_batch_stride, wq, vec)) != VSCAN_OK) return st;
    if ((st = check_stride("yk", a->yk_tok_stride, a->yk_batch_stride, wk, vec)) != VSCAN_OK) return st;
    if (((uintptr_t)a->wq & 3) || ((uintptr_t)a->wk & 3) || ((uintptr_t)a->inv_freq & 3) || ((uintptr_t)a->positions & 3))
        return fail(VSCAN_ERR_ALIGNMENT, "wq, wk, inv_freq or positions is not 4-byte aligned");
    return VSCAN_OK;
}

// Channels a lane loads at once: the widest whose units fall on whole pairs, 16
// bytes unless the number of pairs is odd in it.
int unit_width(const vscan_qknorm_args* a)
{
    int v = a->dtype == VSCAN_F32 ? 4 : 8;
    while (a->pairs % v != 0 || (a->dim - 2 * a->pairs) % v != 0) v /= 2;
    return v;
}

// CTAs: one for each position and group of images. Images share a position's angles; they are
// spread over groups until every CTA slot has several items (so that the last round costs
// little), as long as an item keeps 32 rows of the smaller side.
int groups_of(const vscan_qknorm_args* a, bool back)
{
    if (a->pairs && a->pos_per_image) return std::max(a->batch, 1);
    const long long heads = std::min(a->heads_q, a->heads_k);
    const long long want = (6LL * most_blocks(back) + a->tokens - 1) / std::max(a->tokens, 1);
    const long long most = std::max(1LL, std::max(a->batch * heads / 32, (long long)most_blocks(back) / std::max(a->tokens, 1)));
    return (int)std::max(1LL, std::min(std::min(want, most), (long long)a->batch));
}

int blocks_of(const vscan_qknorm_args* a, bool back)
{
    return (int)std::min<long long>((long long)a->tokens * groups_of(a, back), most_blocks(back));
}

QkNormParams make_params(const vscan_qknorm_args* a, int v, bool back)
{
    QkNormParams p{};
    p.batch = a->batch; p.tokens = a->tokens;
    p.d = a->dim; p.pairs = a->pairs; p.axes = a->axes;
    p.rms = a->norm == VSCAN_NORM_RMS;
    p.pos_img = a->pos_per_image ? a->tokens * a->axes : 0;
    p.groups = groups_of(a, back);
    p.units = a->pairs / v + ((a->dim - 2 * a->pairs) / v + 1) / 2;
    p.lanes = 1;
    while (p.lanes < 32 && p.lanes < p.units) p.lanes *= 2;
    p.eps = a->eps;
    p.inv_freq = a->inv_freq; p.positions = a->positions;
    auto stride = [&](int64_t tok, int64_t img, int heads, long long& t, long long& i) {
        t = tok ? tok : (long long)heads * a->dim;
        i = img ? img : t * a->tokens;
    };
    vscan::QkNormSide &q = p.side[0], &k = p.side[1];
    q.heads = a->heads_q; q.x = a->q; q.w = a->wq; q.y = a->yq;
    k.heads = a->heads_k; k.x = a->k; k.w = a->wk; k.y = a->yk;
    stride(a->q_tok_stride, a->q_batch_stride, a->heads_q, q.x_tok, q.x_img);
    stride(a->k_tok_stride, a->k_batch_stride, a->heads_k, k.x_tok, k.x_img);
    stride(a->yq_tok_stride, a->yq_batch_stride, a->heads_q, q.y_tok, q.y_img);
    stride(a->yk_tok_stride, a->yk_batch_stride, a->heads_k, k.y_tok, k.y_img);
    p.blocks = blocks_of(a, back);
    return p;
}

template <typename T, int V, bool BACK>
void launch_units(const QkNormParams& p, size_t smem, cudaStream_t s)
{
    const int per_lane = (p.units + p.lanes - 1) / p.lanes;
    if (per_lane == 1)
        vscan::qk_norm_kernel<T, V, 1, BACK><<<dim3(p.blocks, 2), vscan::QN_THREADS, smem, s>>>(p);
    else if constexpr (V <= 2) {
        if (per_lane == 2)
            vscan::qk_norm_kernel<T, V, 2, BACK><<<dim3(p.blocks, 2), vscan::QN_THREADS, smem, s>>>(p);
        else if constexpr (V == 1)
            vscan::qk_norm_kernel<T, V, 4, BACK><<<dim3(p.blocks, 2), vscan::QN_THREADS, smem, s>>>(p);
    }
}

template <bool BACK>
cudaError_t launch(const vscan_qknorm_args* a, const QkNormParams& p, int v, cudaStream_t s)
{
    const size_t smem = BACK && p.part ? (size_t)(vscan::QN_THREADS / 32) * p.d * 4 : 0;
    if (a->dtype == VSCAN_F32) {
        if (v == 4) launch_units<float, 4, BACK>(p, smem, s);
        else if (v == 2) launch_units<float, 2, BACK>(p, smem, s);
        else launch_units<float, 1, BACK>(p, smem, s);
    } else {
        if (v == 8) launch_units<__nv_bfloat16, 8, BACK>(p, smem, s);
        else if (v == 4) launch_units<__nv_bfloat16, 4, BACK>(p, smem, s);
        else if (v == 2) launch_units<__nv_bfloat16, 2, BACK>(p, smem, s);
        else launch_units<__nv_bfloat16, 1, BACK>(p, smem, s);
    }
    return cudaGetLastError();
}

bool empty(const vscan_qknorm_args* a) { return a->batch == 0 || a->tokens == 0; }

}  // namespace

extern "C" {

vscan_status vscan_qknorm_forward(const vscan_qknorm_args* args, void* stream)
{
    const vscan_status st = check_shape(args);
    if (st != VSCAN_OK) return st;
    if (empty(args)) return VSCAN_OK;
    if (!args->q || !args->k || !args->yq || !args->yk)
        return fail(VSCAN_ERR_INVALID_ARGUMENT, "q, k, yq and yk must not be NULL");
    if (!aligned16(args->q) || !aligned16(args->k) || !aligned16(args->yq) || !aligned16(args->yk))
        return fail(VSCAN_ERR_ALIGNMENT, "q, k, yq and yk must be 16-byte aligned");
    NvtxRange range("vscan_qknorm_forward");
    const int v = unit_width(args);
    const cudaError_t e = launch<false>(args, make_params(args, v, false), v, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? VSCAN_OK : cuda_fail(e, "vscan_qknorm_forward");
}

vscan_status vscan_qknorm_backward_workspace_size(const vscan_qknorm_args* args, uint64_t* bytes)
{
    if (!bytes) return fail(VSCAN_ERR_INVALID_ARGUMENT, "bytes is NULL");
    const vscan_status st = check_shape(args);
    if (st != VSCAN_OK) return st;
    *bytes = empty(args) ? 0 : (uint64_t)blocks_of(args, true) * 2 * args->dim * 4;
    return VSCAN_OK;
}

vscan_status vscan_qknorm_backward(const vscan_qknorm_args* args, const vscan_qknorm_grads* grads, void* stream)
{
    const vscan_status st = check_shape(args);
    if (st != VSCAN_OK) return st;
    if (!grads) return fail(VSCAN_ERR_INVALID_ARGUMENT, "grads is NULL");
    if (((uintptr_t)grads->dwq & 3) || ((uintptr_t)grads->dwk & 3) || ((uintptr_t)grads->workspace & 3))
        return fail(VSCAN_ERR_ALIGNMENT, "dwq, dwk or the workspace is not 4-byte aligned");
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool weights = grads->dwq || grads->dwk;
    cudaError_t e = cudaSuccess;
    if (empty(args)) {
        NvtxRange range("vscan_qknorm_backward");
        if (grads->dwq) e = cudaMemsetAsync(grads->dwq, 0, (size_t)args->dim * 4, s);
        if (grads->dwk && e == cudaSuccess) e = cudaMemsetAsync(grads->dwk, 0, (size_t)args->dim * 4, s);
        return e == cudaSuccess ? VSCAN_OK : cuda_fail(e, "vscan_qknorm_backward");
    }
    if (!args->q || !args->k || !grads->dyq || !grads->dyk)
        return fail(VSCAN_ERR_INVALID_ARGUMENT, "q, k, dyq and dyk must not be NULL");
    if (!aligned16(args->q) || !aligned16(args->k) || !aligned16(grads->dyq) || !aligned16(grads->dyk) ||
        !aligned16(grads->dq) || !aligned16(grads->dk))
        return fail(VSCAN_ERR_ALIGNMENT, "q, k, dyq, dyk, dq and dk must be 16-byte aligned");
    const int v = unit_width(args);
    QkNormParams p = make_params(args, v, true);
    const uint64_t need = (uint64_t)p.blocks * 2 * args->dim * 4;
    if (weights && (!grads->workspace || grads->workspace_bytes < need))
        return fail(VSCAN_ERR_WORKSPACE, "workspace of %llu bytes, %llu needed", (unsigned long long)grads->workspace_bytes,
                    (unsigned long long)need);
    NvtxRange range("vscan_qknorm_backward");
    p.side[0].dy = grads->dyq; p.side[0].y = grads->dq;
    p.side[1].dy = grads->dyk; p.side[1].y = grads->dk;
    p.part = weights ? static_cast<float*>(grads->workspace) : nullptr;
    e = launch<true>(args, p, v, s);
    if (e == cudaSuccess && weights) {
        e = launch_after(true, vscan::qk_norm_weight_kernel, dim3((args->dim + 31) / 32, 2), vscan::QN_SUM_THREADS, 0, s,
                         (const float*)p.part, p.blocks, (int)args->dim, grads->dwq, grads->dwk);
    }
    return e == cudaSuccess ? VSCAN_OK : cuda_fail(e, "vscan_qknorm_backward");
}

}  // extern "C"
