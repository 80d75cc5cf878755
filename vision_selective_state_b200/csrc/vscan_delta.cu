// C ABI of the gated delta rule (declared in include/vscan.h): argument checks,
// workspace layout, kernel selection and launch. Every check runs before the
// first CUDA call, so a rejected call launches nothing.
#include <cmath>

#include "vscan.h"
#include "vscan_delta.cuh"
#include "vscan_delta_grad.cuh"
#include "vscan_host.h"

namespace {

using vscan_host::aligned16;
using vscan_host::cuda_fail;
using vscan_host::fail;
using vscan_host::NvtxRange;
using vscan_host::round256;
using vscan_host::launch_after;
using vscan_host::set_smem_once;
using vscan::DeltaParams;
using vscan::DL_C;

constexpr int kAttrDevices = 64;
constexpr int kMaxDimK = 128, kMaxDimV = 256, kMaxGrid = 65535;

// Widths the kernels are built for: dim_k is rounded up to one of them.
int padded_dim_k(int dk) { return dk <= 64 ? 64 : 128; }

struct Stride { int64_t tok, img; };

Stride resolve(int64_t tok, int64_t img, int64_t width, int64_t tokens)
{
    Stride s;
    s.tok = tok ? tok : width;
    s.img = img ? img : s.tok * tokens;
    return s;
}

vscan_status check_stride(const char* name, int64_t tok, int64_t img, int64_t width, int64_t tokens, int vec)
{
    if (tok < 0 || img < 0) return fail(VSCAN_ERR_INVALID_ARGUMENT, "%s strides must be >= 0 (0 = dense)", name);
    const Stride s = resolve(tok, img, width, tokens);
    if (s.tok < width || s.tok % vec != 0)
        return fail(VSCAN_ERR_ALIGNMENT, "%s token stride %lld must be >= %lld and a multiple of %d", name, (long long)s.tok,
                    (long long)width, vec);
    if (s.img % vec != 0)
        return fail(VSCAN_ERR_ALIGNMENT, "%s batch stride %lld is not a multiple of %d", name, (long long)s.img, vec);
    return VSCAN_OK;
}

// Checks that do not depend on where the tensors live.
vscan_status check_shape(const vscan_route* r, const vscan_delta_args* a)
{
    if (!a) return fail(VSCAN_ERR_INVALID_ARGUMENT, "args is NULL");
    if (a->dtype != VSCAN_F32 && a->dtype != VSCAN_BF16)
        return fail(VSCAN_ERR_INVALID_ARGUMENT, "unknown dtype %d", a->dtype);
    if (a->batch < 0) return fail(VSCAN_ERR_INVALID_ARGUMENT, "batch %d < 0", a->batch);
    if (a->tokens < 0) return fail(VSCAN_ERR_INVALID_ARGUMENT, "tokens %d < 0", a->tokens);
    if (a->heads_k < 1 || a->heads_v < 1)
        return fail(VSCAN_ERR_INVALID_ARGUMENT, "heads_k %d and heads_v %d must be >= 1", a->heads_k, a->heads_v);
    if (a->heads_v % a->heads_k != 0)
        return fail(VSCAN_ERR_SHAPE, "heads_v %d is not a multiple of heads_k %d", a->heads_v, a->heads_k);
    if (a->dim_k < 1 || a->dim_v < 1)
        return fail(VSCAN_ERR_INVALID_ARGUMENT, "dim_k %d and dim_v %d must be >= 1", a->dim_k, a->dim_v);
    const int vec = a->dtype == VSCAN_F32 ? 4 : 8;
    if (a->dim_k % vec != 0 || a->dim_v % vec != 0)
        return fail(VSCAN_ERR_ALIGNMENT, "dim_k %d and dim_v %d must be multiples of %d (16-byte rows)", a->dim_k, a->dim_v, vec);
    if (a->dim_k > kMaxDimK || a->dim_v > kMaxDimV)
        return fail(VSCAN_ERR_UNSUPPORTED, "dim_k %d > %d or dim_v %d > %d", a->dim_k, kMaxDimK, a->dim_v, kMaxDimV);
    if (a->tokens > 0x7fffffff - (DL_C - 1))  // rounded up to chunks in 32 bits
        return fail(VSCAN_ERR_UNSUPPORTED, "tokens %d > 2^31 - %d", a->tokens, DL_C);
    if (a->batch > kMaxGrid || a->heads_v > kMaxGrid)
        return fail(VSCAN_ERR_UNSUPPORTED, "batch %d or heads_v %d > %d", a->batch, a->heads_v, kMaxGrid);
    if (!std::isfinite(a->scale) || !std::isfinite(a->beta_scale))
        return fail(VSCAN_ERR_INVALID_ARGUMENT, "scale and beta_scale must be finite");
    if (r) {
        if (r->g.kind != vscan::RK_BIDIR && r->g.kind != vscan::RK_CROSS4 && r->g.kind != vscan::RK_ATROUS2)
            return fail(VSCAN_ERR_UNSUPPORTED, "the delta rule runs over BIDIR, CROSS4 and ATROUS2 routes");
        if (a->seq_offsets) return fail(VSCAN_ERR_UNSUPPORTED, "seq_offsets needs plain sequences, not a route");
        if (a->direction < 0 || a->direction >= r->g.K)
            return fail(VSCAN_ERR_SHAPE, "direction %d, the route has %d", a->direction, r->g.K);
        if (a->tokens != r->g.tokens)
            return fail(VSCAN_ERR_SHAPE, "tokens %d, the route has %d per image", a->tokens, r->g.tokens);
    } else if (a->direction != 0) {
        return fail(VSCAN_ERR_SHAPE, "direction %d without a route", a->direction);
    }
    const int64_t wk = (int64_t)a->heads_k * a->dim_k, wv = (int64_t)a->heads_v * a->dim_v;
    vscan_status st;
    if ((st = check_stride("q", a->q_tok_stride, a->q_batch_stride, wk, a->tokens, vec)) != VSCAN_OK) return st;
    if ((st = check_stride("k", a->k_tok_stride, a->k_batch_stride, wk, a->tokens, vec)) != VSCAN_OK) return st;
    if ((st = check_stride("v", a->v_tok_stride, a->v_batch_stride, wv, a->tokens, vec)) != VSCAN_OK) return st;
    if ((st = check_stride("y", a->y_tok_stride, a->y_batch_stride, wv, a->tokens, vec)) != VSCAN_OK) return st;
    if ((st = check_stride("a", a->a_tok_stride, a->a_batch_stride, 1, a->tokens, 1)) != VSCAN_OK) return st;
    if ((st = check_stride("b", a->b_tok_stride, a->b_batch_stride, 1, a->tokens, 1)) != VSCAN_OK) return st;
    return VSCAN_OK;
}

// y (or, for the gradients, dy) is the last tensor: the only one some calls lack.
vscan_status check_pointers(const vscan_delta_args* a, const void* y)
{
    if (!a->q || !a->k || !a->v || !a->a || !a->b || !y || !a->A)
        return fail(VSCAN_ERR_INVALID_ARGUMENT, "q, k, v, a, b, A and y (dy) must not be NULL");
    if (!aligned16(a->q) || !aligned16(a->k) || !aligned16(a->v) || !aligned16(y) || !aligned16(a->initial_state) ||
        !aligned16(a->final_state))
        return fail(VSCAN_ERR_ALIGNMENT, "q, k, v, y (dy) and the states must be 16-byte aligned");
    const uintptr_t el = a->dtype == VSCAN_F32 ? 3 : 1;
    if (((uintptr_t)a->a & el) || ((uintptr_t)a->b & el) || ((uintptr_t)a->A & 3) || ((uintptr_t)a->bias & 3) ||
        ((uintptr_t)a->seq_offsets & 3) || ((uintptr_t)a->status & 3))
        return fail(VSCAN_ERR_ALIGNMENT, "a, b, A, bias, seq_offsets or status is not aligned to its element");
    return VSCAN_OK;
}

int chunks_of(const vscan_route* r, const vscan_delta_args* a)
{
    return ((r ? r->g.L : a->tokens) + DL_C - 1) / DL_C;
}

// Chunk slots of the workspace. A packed sequence's slots start at
// floor(first row / 64) + its index: sequences never share one.
long long slots_of(const vscan_route* r, const vscan_delta_args* a)
{
    if (a->seq_offsets) return (long long)a->tokens / DL_C + a->batch + 1;
    return (long long)a->batch * chunks_of(r, a);
}

bool empty(const vscan_delta_args* a) { return a->batch == 0; }

struct Layout {
    size_t total;  // the records
    size_t L, S, dS, W, dX, part, dq, dk, grad_total;  // backward
};

Layout forward_layout(const vscan_route* r, const vscan_delta_args* a, int pplanes)
{
    const size_t n = (size_t)slots_of(r, a) * a->heads_v;
    Layout l;
    const bool wide = padded_dim_k(a->dim_k) == 128;
    l.total = round256(n * (a->dtype == VSCAN_F32
                                ? (wide ? vscan::delta_record_bytes<float, 128>(pplanes) : vscan::delta_record_bytes<float, 64>(pplanes))
                                : vscan::delta_record_bytes<__nv_bfloat16, 64>(pplanes)));
    return l;
}

// The forward's scratch with P in three planes, and what the walks leave for the
// per-chunk gradients.
Layout backward_layout(const vscan_route* r, const vscan_delta_args* a)
{
    Layout l = forward_layout(r, a, 3);
    const size_t n = (size_t)slots_of(r, a) * a->heads_v, state = (size_t)a->dim_v * padded_dim_k(a->dim_k) * 4;
    const size_t rows = (size_t)DL_C * a->dim_v * 4;
    l.L = l.total;
    l.S = l.L + round256(n * vscan::DL_PLANE * 4);
    l.dS = l.S + round256(n * state);
    l.W = l.dS + round256(n * state);
    l.dX = l.W + round256(n * rows);
    l.part = l.dX + round256(n * rows);
    l.dq = l.part + round256(n * 8);
    const size_t images = a->seq_offsets ? 1 : a->batch;
    const size_t shared = a->heads_v == a->heads_k ? 0 : round256(images * a->tokens * a->heads_v * a->dim_k * 4);
    l.dk = l.dq + shared;
    l.grad_total = l.dk + shared;
    return l;
}

int forward_planes(const vscan_delta_args* a) { return a->dtype == VSCAN_F32 ? 3 : 2; }

DeltaParams make_params(const vscan_route* r, const vscan_delta_args* a)
{
    DeltaParams p{};
    if (r) { p.g = r->g; p.has_route = 1; }
    p.dir = a->direction;
    p.batch = a->batch;
    p.tokens = a->tokens;
    p.heads_k = a->heads_k;
    p.heads_v = a->heads_v;
    p.group = a->heads_v / a->heads_k;
    p.dk = a->dim_k;
    p.dv = a->dim_v;
    p.offsets = a->seq_offsets;
    p.chunks = chunks_of(r, a);
    p.slots = slots_of(r, a);
    p.q = a->q; p.k = a->k; p.v = a->v; p.a = a->a; p.b = a->b; p.y = a->y;
    p.A = a->A; p.bias = a->bias;
    p.s_in = a->initial_state;
    p.s_out = a->final_state;
    p.status = a->status;
    p.scale = a->scale;
    p.beta_scale = a->beta_scale;
    const int64_t wk = (int64_t)a->heads_k * a->dim_k, wv = (int64_t)a->heads_v * a->dim_v;
    Stride s;
    s = resolve(a->q_tok_stride, a->q_batch_stride, wk, a->tokens); p.q_tok = s.tok; p.q_img = s.img;
    s = resolve(a->k_tok_stride, a->k_batch_stride, wk, a->tokens); p.k_tok = s.tok; p.k_img = s.img;
    s = resolve(a->v_tok_stride, a->v_batch_stride, wv, a->tokens); p.v_tok = s.tok; p.v_img = s.img;
    s = resolve(a->y_tok_stride, a->y_batch_stride, wv, a->tokens); p.y_tok = s.tok; p.y_img = s.img;
    s = resolve(a->a_tok_stride, a->a_batch_stride, a->heads_v, a->tokens); p.a_tok = s.tok; p.a_img = s.img;
    s = resolve(a->b_tok_stride, a->b_batch_stride, a->heads_v, a->tokens); p.b_tok = s.tok; p.b_img = s.img;
    return p;
}

template <typename T, int DKP, int PP>
cudaError_t launch_prep(const DeltaParams& p, cudaStream_t stream)
{
    if (p.slots == 0 || p.tokens == 0) return cudaSuccess;
    static int done[kAttrDevices];
    constexpr size_t smem = vscan::PrepShape<T, DKP>::smem;
    cudaError_t e = set_smem_once(vscan::delta_prep_kernel<T, DKP, PP>, (int)smem, done, kAttrDevices);
    if (e != cudaSuccess) return e;
    return launch_after(false, vscan::delta_prep_kernel<T, DKP, PP>, dim3((unsigned)p.slots, p.heads_v), vscan::DP_THREADS, smem,
                        stream, p);
}

dim3 walk_grid(const DeltaParams& p) { return dim3((p.dv + 127) / 128, p.heads_v, p.batch); }

template <typename T, int DKP, bool SAVE>
cudaError_t launch_scan(const DeltaParams& p, cudaStream_t stream)
{
    using Sh = vscan::WalkShape<T, DKP>;
    static int done[kAttrDevices];
    constexpr size_t smem = Sh::smem(Sh::PP);
    const cudaError_t e = set_smem_once(vscan::delta_scan_kernel<T, DKP, SAVE>, (int)smem, done, kAttrDevices);
    if (e != cudaSuccess) return e;
    return launch_after(p.slots > 0 && p.tokens > 0, vscan::delta_scan_kernel<T, DKP, SAVE>, walk_grid(p), vscan::DW_THREADS, smem,
                        stream, p);
}

template <typename T, int DKP>
cudaError_t run_forward(const DeltaParams& p, cudaStream_t stream)
{
    cudaError_t e = launch_prep<T, DKP, vscan::WalkShape<T, DKP>::PP>(p, stream);
    if (e != cudaSuccess) return e;
    return launch_scan<T, DKP, false>(p, stream);
}

template <typename T, int DKP>
cudaError_t run_backward(const DeltaParams& p, cudaStream_t stream)
{
    static int done_r[kAttrDevices], done_g[kAttrDevices];
    cudaError_t e;
    const bool any = p.tokens > 0 && p.slots > 0;
    // The walk backwards and the per-chunk gradients of a long call come later: their blocks would
    // take their places while the last walks still run, unevenly (gradients of 16 images of 4097
    // tokens, 6 heads of 128 x 128: 1620 us early, 1600 after the end; of 8 images of 197 tokens, 64 x 64:
    // 75.5 and 77.7 us).
    const bool early = any && p.slots * p.heads_v <= 4 * 148;
    if (any) {
        if ((e = launch_prep<T, DKP, 3>(p, stream)) != cudaSuccess) return e;
        if ((e = launch_scan<T, DKP, true>(p, stream)) != cudaSuccess) return e;
    }
    constexpr size_t walk = vscan::WalkShape<T, DKP>::smem(3);
    if ((e = set_smem_once(vscan::delta_rscan_kernel<T, DKP>, (int)walk, done_r, kAttrDevices)) != cudaSuccess) return e;
    if ((e = launch_after(early, vscan::delta_rscan_kernel<T, DKP>, walk_grid(p), vscan::DW_THREADS, walk, stream, p)) != cudaSuccess) return e;
    if (any) {
        constexpr size_t smem = vscan::GradShape<T, DKP>::smem;
        if ((e = set_smem_once(vscan::delta_grad_kernel<T, DKP>, (int)smem, done_g, kAttrDevices)) != cudaSuccess) return e;
        e = launch_after(early, vscan::delta_grad_kernel<T, DKP>, dim3((unsigned)p.slots, p.heads_v), vscan::DG_THREADS, smem, stream, p);
        if (e != cudaSuccess) return e;
        if (p.wdq && (p.dq || p.dkey)) {
            const long long vecs = (long long)(p.offsets ? 1 : p.batch) * p.tokens * p.heads_k * (p.dk / 4);
            e = launch_after(true, vscan::delta_group_kernel<T>, dim3((unsigned)((vecs + 255) / 256), 2), 256, 0, stream, p, vecs);
            if (e != cudaSuccess) return e;
        }
    }
    return p.dA || p.dbias ? launch_after(true, vscan::delta_param_grad_kernel, dim3(p.heads_v), 256, 0, stream, p) : cudaSuccess;
}

// f(width) with the I/O type and the padded key width as template arguments.
#define DELTA_DISPATCH(FN, a, ...)                                                                             \
    (a->dtype == VSCAN_F32 ? (padded_dim_k(a->dim_k) == 64 ? FN<float, 64>(__VA_ARGS__) : FN<float, 128>(__VA_ARGS__)) \
                           : (padded_dim_k(a->dim_k) == 64 ? FN<__nv_bfloat16, 64>(__VA_ARGS__)                 \
                                                           : FN<__nv_bfloat16, 128>(__VA_ARGS__)))

}  // namespace

extern "C" {

vscan_status vscan_delta_workspace_size(const vscan_route* route, const vscan_delta_args* args, uint64_t* bytes)
{
    if (!bytes) return fail(VSCAN_ERR_INVALID_ARGUMENT, "bytes is NULL");
    const vscan_status st = check_shape(route, args);
    if (st != VSCAN_OK) return st;
    *bytes = empty(args) ? 0 : forward_layout(route, args, forward_planes(args)).total;
    return VSCAN_OK;
}

vscan_status vscan_delta_forward(const vscan_route* route, const vscan_delta_args* args, void* stream)
{
    vscan_status st = check_shape(route, args);
    if (st != VSCAN_OK) return st;
    if (empty(args) || (args->tokens == 0 && !args->final_state)) return VSCAN_OK;
    if (args->tokens > 0 && (st = check_pointers(args, args->y)) != VSCAN_OK) return st;
    if (!aligned16(args->initial_state) || !aligned16(args->final_state))
        return fail(VSCAN_ERR_ALIGNMENT, "the states must be 16-byte aligned");
    const Layout l = forward_layout(route, args, forward_planes(args));
    if (l.total && (!args->workspace || args->workspace_bytes < l.total))
        return fail(VSCAN_ERR_WORKSPACE, "workspace of %llu bytes, %llu needed", (unsigned long long)args->workspace_bytes,
                    (unsigned long long)l.total);
    if (!aligned16(args->workspace)) return fail(VSCAN_ERR_ALIGNMENT, "workspace is not 16-byte aligned");
    if (slots_of(route, args) > 0x7fffffffLL)
        return fail(VSCAN_ERR_UNSUPPORTED, "more than 2^31 chunks of %d steps", DL_C);
    NvtxRange range("vscan_delta_forward");
    DeltaParams p = make_params(route, args);
    char* ws = static_cast<char*>(args->workspace);
    p.tplanes = forward_planes(args);
    p.wrec = reinterpret_cast<unsigned char*>(ws);
    const cudaError_t e = DELTA_DISPATCH(run_forward, args, p, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? VSCAN_OK : cuda_fail(e, "vscan_delta_forward");
}

vscan_status vscan_delta_backward_workspace_size(const vscan_route* route, const vscan_delta_args* args, uint64_t* bytes)
{
    if (!bytes) return fail(VSCAN_ERR_INVALID_ARGUMENT, "bytes is NULL");
    const vscan_status st = check_shape(route, args);
    if (st != VSCAN_OK) return st;
    *bytes = empty(args) ? 0 : backward_layout(route, args).grad_total;
    return VSCAN_OK;
}

vscan_status vscan_delta_backward(const vscan_route* route, const vscan_delta_args* args, const void* dy,
                                  const vscan_delta_grads* grads, void* stream)
{
    vscan_status st = check_shape(route, args);
    if (st != VSCAN_OK) return st;
    if (!grads) return fail(VSCAN_ERR_INVALID_ARGUMENT, "grads is NULL");
    const bool none = empty(args) || args->tokens == 0;
    if (!none && (st = check_pointers(args, dy)) != VSCAN_OK) return st;
    if (!aligned16(grads->dq) || !aligned16(grads->dk) || !aligned16(grads->dv) || !aligned16(grads->d_initial_state) ||
        !aligned16(grads->d_final_state) || !aligned16(grads->workspace))
        return fail(VSCAN_ERR_ALIGNMENT, "dq, dk, dv, the states' gradients and the workspace must be 16-byte aligned");
    const uintptr_t el = args->dtype == VSCAN_F32 ? 3 : 1;
    if (((uintptr_t)grads->da & el) || ((uintptr_t)grads->db & el) || ((uintptr_t)grads->dA & 3) ||
        ((uintptr_t)grads->dbias & 3))
        return fail(VSCAN_ERR_ALIGNMENT, "da, db, dA or dbias is not aligned to its element");
    if (grads->d_final_state && grads->d_final_state == grads->d_initial_state)
        return fail(VSCAN_ERR_INVALID_ARGUMENT, "d_final_state and d_initial_state must not be the same memory");
    const Layout l = backward_layout(route, args);
    if (!none && (!grads->workspace || grads->workspace_bytes < l.grad_total))
        return fail(VSCAN_ERR_WORKSPACE, "workspace of %llu bytes, %llu needed", (unsigned long long)grads->workspace_bytes,
                    (unsigned long long)l.grad_total);
    if (slots_of(route, args) > 0x7fffffffLL)
        return fail(VSCAN_ERR_UNSUPPORTED, "more than 2^31 chunks of %d steps", DL_C);
    NvtxRange range("vscan_delta_backward");
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e = cudaSuccess;
    auto zero = [&](void* ptr, size_t bytes) {
        if (ptr && bytes && e == cudaSuccess) e = cudaMemsetAsync(ptr, 0, bytes, s);
    };
    // every token row's gradients, for rows that no step visits
    auto zero_rows = [&] {
        const size_t el_bytes = vscan_host::elem_bytes(args->dtype);
        const size_t rows = (size_t)(args->seq_offsets ? 1 : args->batch) * args->tokens;
        zero(grads->dq, rows * args->heads_k * args->dim_k * el_bytes);
        zero(grads->dk, rows * args->heads_k * args->dim_k * el_bytes);
        zero(grads->dv, rows * args->heads_v * args->dim_v * el_bytes);
        zero(grads->da, rows * args->heads_v * el_bytes);
        zero(grads->db, rows * args->heads_v * el_bytes);
    };
    if (none) {  // no step: the state's gradient passes through
        zero_rows();  // packed rows without a sequence; otherwise there are none
        zero(grads->dA, (size_t)args->heads_v * 4);
        zero(grads->dbias, (size_t)args->heads_v * 4);
        const size_t bytes = (size_t)args->batch * args->heads_v * args->dim_k * args->dim_v * 4;
        if (grads->d_initial_state && grads->d_final_state && bytes && e == cudaSuccess)
            e = cudaMemcpyAsync(grads->d_initial_state, grads->d_final_state, bytes, cudaMemcpyDeviceToDevice, s);
        else
            zero(grads->d_initial_state, bytes);
        return e == cudaSuccess ? VSCAN_OK : cuda_fail(e, "vscan_delta_backward");
    }
    DeltaParams p = make_params(route, args);
    char* ws = static_cast<char*>(grads->workspace);
    p.s_out = nullptr;
    p.tplanes = 3;
    p.wrec = reinterpret_cast<unsigned char*>(ws);
    p.wL = reinterpret_cast<float*>(ws + l.L);
    p.wS = reinterpret_cast<float*>(ws + l.S);
    p.wdS = reinterpret_cast<float*>(ws + l.dS);
    p.wW = reinterpret_cast<float*>(ws + l.W);
    p.wdX = reinterpret_cast<float*>(ws + l.dX);
    p.wpart = reinterpret_cast<float*>(ws + l.part);
    if (p.group > 1) {
        p.wdq = reinterpret_cast<float*>(ws + l.dq);
        p.wdk = reinterpret_cast<float*>(ws + l.dk);
    }
    p.dy = dy;
    p.ds_in = grads->d_final_state;
    p.ds_out = grads->d_initial_state;
    p.dq = grads->dq; p.dkey = grads->dk; p.dvalue = grads->dv;
    p.da = grads->da; p.db = grads->db;
    p.dA = grads->dA; p.dbias = grads->dbias;
    if (args->seq_offsets || (route && route->g.kind == vscan::RK_ATROUS2)) {
        zero_rows();  // rows without a step, and chunk slots without a chunk
        zero(p.wpart, (size_t)p.slots * p.heads_v * 8);
        if (p.wdq) zero(p.wdq, l.grad_total - l.dq);
        if (e != cudaSuccess) return cuda_fail(e, "vscan_delta_backward");
    }
    e = DELTA_DISPATCH(run_backward, args, p, s);
    return e == cudaSuccess ? VSCAN_OK : cuda_fail(e, "vscan_delta_backward");
}

vscan_status vscan_delta_step(const vscan_delta_args* args, void* stream)
{
    vscan_status st = check_shape(nullptr, args);
    if (st != VSCAN_OK) return st;
    if (args->tokens != 1) return fail(VSCAN_ERR_SHAPE, "vscan_delta_step takes one token a row, not %d", args->tokens);
    if (args->seq_offsets) return fail(VSCAN_ERR_UNSUPPORTED, "vscan_delta_step takes no seq_offsets");
    if (empty(args)) return VSCAN_OK;
    if ((st = check_pointers(args, args->y)) != VSCAN_OK) return st;
    if (!args->initial_state || !args->final_state)
        return fail(VSCAN_ERR_INVALID_ARGUMENT, "initial_state and final_state must not be NULL");
    NvtxRange range("vscan_delta_step");
    const DeltaParams p = make_params(nullptr, args);
    const dim3 grid((p.dv + vscan::DS_COLS - 1) / vscan::DS_COLS, p.heads_v, p.batch);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (args->dtype == VSCAN_F32)
        vscan::delta_step_kernel<float><<<grid, 128, 0, s>>>(p);
    else
        vscan::delta_step_kernel<__nv_bfloat16><<<grid, 128, 0, s>>>(p);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? VSCAN_OK : cuda_fail(e, "vscan_delta_step");
}

}  // extern "C"
