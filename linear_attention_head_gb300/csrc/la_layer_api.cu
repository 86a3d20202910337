// la_layer_api.cu -- the C entry points of the operators beside the attention
// (include/la.h): the gated linear recurrence and the norms of queries and
// keys with the position rotation.  Argument checks, then the launches of
// la_scan.cu and la_qk_rope.cu.

#include <climits>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <exception>
#include <new>
#include <vector>

#include "../../include/la.h"
#include "la_internal.h"

namespace {

la_status fail(la_status st, const char *fmt, ...)
{
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    la::set_last_error(buf);
    return st;
}

la_status launched(cudaError_t e, const char *what)
{
    if (e == cudaSuccess)
        return LA_OK;
    if (e == cudaErrorNotSupported)
        return fail(LA_ERR_UNSUPPORTED, "%s: sizes beyond what the kernels handle", what);
    return fail(LA_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

la_status need(const void *p, const char *name)
{
    return p ? LA_OK : fail(LA_ERR_INVALID_ARG, "%s is NULL", name);
}

bool known_dtype(int32_t t) { return t == LA_DTYPE_BF16 || t == LA_DTYPE_F32; }

la_status check_rows(int32_t batch, int32_t seq_len, int32_t dim)
{
    if (batch < 0 || seq_len < 0)
        return fail(LA_ERR_INVALID_ARG, "negative batch (%d) or seq_len (%d)", batch, seq_len);
    if (batch > (1 << 30))
        return fail(LA_ERR_INVALID_ARG, "batch = %d", batch);
    if (dim < 1 || dim > 256)
        return fail(LA_ERR_UNSUPPORTED, "dim = %d: supported range is 1..256", dim);
    return LA_OK;
}

la_status check_in(const int64_t *st, const char *name)
{
    for (int i = 0; i < 3; ++i)
        if (st[i] < 0)
            return fail(LA_ERR_INVALID_ARG, "negative stride of %s", name);
    return LA_OK;
}

// Outputs: every element in a place of its own (a stride may still be too
// small to tell rows apart; only repeats are refused).
la_status check_out(const int64_t *st, const char *name, int32_t B, int32_t T, int32_t H)
{
    la_status e = check_in(st, name);
    const int32_t n[3] = {B, T, H};
    const bool empty = !B || !T || !H;
    for (int i = 0; i < 3 && !e && !empty; ++i)
        if (st[i] == 0 && n[i] > 1)
            e = fail(LA_ERR_INVALID_ARG, "stride 0 of %s: an output cannot repeat rows", name);
    return e;
}

// The packed-sequence table, as la_fwd takes it, and what it says (without one:
// `batch` sequences of seq_len tokens).
struct Sequences {
    int n = 0;              // of states
    int some_empty = 0;     // sequences without tokens are among them
    int64_t tiles = 0;      // of la::SCAN_TILE tokens, of all sequences together
    int64_t longest = 0;
};
la_status check_packed(int32_t batch, int32_t seq_len, int32_t num_seqs, const int32_t *cu,
                       const int32_t *cu_host, cudaStream_t stream, Sequences *q)
{
    q->n = batch;
    q->some_empty = batch > 0 && seq_len == 0;
    q->longest = seq_len;
    q->tiles = (int64_t)batch * (((int64_t)seq_len + la::SCAN_TILE - 1) / la::SCAN_TILE);
    if (!cu)
        return cu_host ? fail(LA_ERR_INVALID_ARG, "cu_seqlens_host given without cu_seqlens")
                       : LA_OK;
    if (batch != 1)
        return fail(LA_ERR_INVALID_ARG,
                    "with cu_seqlens the sequences are packed in one batch row: "
                    "batch must be 1, got %d",
                    batch);
    if (num_seqs < 0 || num_seqs > (1 << 30))
        return fail(LA_ERR_INVALID_ARG, "num_seqs = %d", num_seqs);
    *q = Sequences{};
    q->n = num_seqs;
    std::vector<int32_t> copy;
    if (!cu_host) {
        copy.resize((size_t)num_seqs + 1);
        cudaError_t e = cudaMemcpyAsync(copy.data(), cu, sizeof(int32_t) * copy.size(),
                                        cudaMemcpyDeviceToHost, stream);
        if (e == cudaSuccess)
            e = cudaStreamSynchronize(stream);
        if (e != cudaSuccess)
            return launched(e, "copying cu_seqlens to the host");
        cu_host = copy.data();
    }
    if (cu_host[0] != 0)
        return fail(LA_ERR_INVALID_ARG, "cu_seqlens[0] = %d, expected 0", cu_host[0]);
    for (int n = 0; n < num_seqs; ++n) {
        const int64_t len = (int64_t)cu_host[n + 1] - cu_host[n];
        if (len < 0)
            return fail(LA_ERR_INVALID_ARG, "cu_seqlens decreases at %d (%d -> %d)", n,
                        cu_host[n], cu_host[n + 1]);
        q->some_empty |= len == 0;
        q->longest = len > q->longest ? len : q->longest;
        q->tiles += (len + la::SCAN_TILE - 1) / la::SCAN_TILE;
    }
    if (cu_host[num_seqs] != seq_len)
        return fail(LA_ERR_INVALID_ARG, "cu_seqlens[%d] = %d but seq_len = %d", num_seqs,
                    cu_host[num_seqs], seq_len);
    return LA_OK;
}

la_status check_workspace(const void *ws, size_t bytes, size_t want)
{
    if (!want)
        return LA_OK;
    if (!ws || bytes < want)
        return fail(LA_ERR_INVALID_ARG, "this call needs a workspace of %zu bytes, got %zu", want,
                    ws ? bytes : (size_t)0);
    if (reinterpret_cast<uintptr_t>(ws) & 255)
        return fail(LA_ERR_INVALID_ARG, "workspace is not 256-byte aligned");
    return LA_OK;
}

// An exception (no memory for the host copy of cu_seqlens) must not leave a C
// entry point.
template <typename F> la_status guarded(F f)
{
    la::set_last_error("");
    try {
        return f();
    } catch (const std::bad_alloc &) {
        return fail(LA_ERR_INVALID_ARG, "no host memory to check the arguments");
    } catch (const std::exception &e) {
        return fail(LA_ERR_INVALID_ARG, "%s", e.what());
    }
}

la::Tok tok(const void *p, const int64_t *st) { return la::Tok{p, st[0], st[1], st[2], 1}; }
la::TokOut tok_out(void *p, const int64_t *st) { return la::TokOut{p, st[0], st[1], st[2]}; }

// ---- gated linear recurrence ------------------------------------------------

la_status scan_sizes(const la_scan_dims *d, int32_t dtype)
{
    if (!d)
        return fail(LA_ERR_INVALID_ARG, "dims is NULL");
    if (!known_dtype(dtype))
        return fail(LA_ERR_INVALID_ARG, "dtype %d is neither LA_DTYPE_BF16 nor LA_DTYPE_F32",
                    dtype);
    if (d->gate_dtype != dtype && d->gate_dtype != LA_DTYPE_F32)
        return fail(LA_ERR_INVALID_ARG, "gate_dtype %d is neither the token dtype nor LA_DTYPE_F32",
                    d->gate_dtype);
    if (d->heads < 1 || d->heads > 65535)
        return fail(LA_ERR_INVALID_ARG, "heads = %d outside 1..65535", d->heads);
    return check_rows(d->batch, d->seq_len, d->dim);
}

size_t states_bytes(const la_scan_dims *d)
{
    return la::scan_states_bytes(d->batch, d->seq_len, d->num_seqs, d->heads, d->dim);
}

// A copy of the initial states (final_state being initial_state itself: the
// kernel reads a sequence's initial state twice).
size_t init_bytes(const la_scan_dims *d)
{
    const int32_t n = d->batch > d->num_seqs ? d->batch : d->num_seqs;
    return (size_t)n * d->heads * d->dim * sizeof(float);
}

bool scan_sized(const la_scan_dims *d)
{
    return d && d->batch >= 0 && d->seq_len >= 0 && d->heads >= 1 && d->heads <= 65535 &&
           d->dim >= 1 && d->dim <= 256;
}

size_t round256(size_t x) { return (x + 255) / 256 * 256; }

la_status scan_args(const la_scan_dims *d, int32_t dtype, const void *x, const void *g,
                    const float *init, int32_t reverse, const int32_t *cu,
                    const int32_t *cu_host, cudaStream_t s, la::ScanArgs *a)
{
    la_status e;
    if ((e = scan_sizes(d, dtype)) || (e = check_in(d->x_strides, "x")) ||
        (e = check_in(d->g_strides, "g")))
        return e;
    *a = la::ScanArgs{};
    Sequences q;
    if ((e = check_packed(d->batch, d->seq_len, d->num_seqs, cu, cu_host, s, &q)))
        return e;
    a->N = q.n;
    a->some_empty = q.some_empty;
    a->B = d->batch;
    a->T = d->seq_len;
    a->H = d->heads;
    a->D = d->dim;
    a->cu = cu;
    a->reverse = reverse ? 1 : 0;
    a->bf16 = dtype == LA_DTYPE_BF16;
    a->gate_bf16 = d->gate_dtype == LA_DTYPE_BF16;
    a->x = tok(x, d->x_strides);
    a->g = tok(g, d->g_strides);
    a->init = init;
    la::scan_plan(a, q.tiles, q.longest);
    if ((int64_t)a->B * a->T > 0 && ((e = need(x, "x")) || (e = need(g, "g"))))
        return e;
    return LA_OK;
}

// ---- norms and rotation -------------------------------------------------------

la_status rope_sizes(const la_rope_dims *d, int32_t dtype)
{
    if (!d)
        return fail(LA_ERR_INVALID_ARG, "dims is NULL");
    if (!known_dtype(dtype) || !known_dtype(d->weight_dtype))
        return fail(LA_ERR_INVALID_ARG,
                    "dtype %d or weight_dtype %d is neither LA_DTYPE_BF16 nor LA_DTYPE_F32", dtype,
                    d->weight_dtype);
    if (d->q_heads < 0 || d->q_heads > 65535 || d->k_heads < 0 || d->k_heads > 65535 ||
        d->q_heads + d->k_heads == 0)
        return fail(LA_ERR_INVALID_ARG, "q_heads = %d, k_heads = %d: 0..65535, not both 0",
                    d->q_heads, d->k_heads);
    la_status e = check_rows(d->batch, d->seq_len, d->dim);
    if (e)
        return e;
    if (d->rotary_dim < 0 || d->rotary_dim > d->dim || d->rotary_dim % 2)
        return fail(LA_ERR_INVALID_ARG, "rotary_dim = %d must be even, 0..dim = %d", d->rotary_dim,
                    d->dim);
    if (d->num_axes < 1 || d->num_axes > 4)
        return fail(LA_ERR_INVALID_ARG, "num_axes = %d outside 1..4", d->num_axes);
    for (int j = 0; j < d->rotary_dim / 2; ++j)
        if (d->pair_axis[j] >= d->num_axes)
            return fail(LA_ERR_INVALID_ARG, "pair_axis[%d] = %d, but num_axes = %d", j,
                        d->pair_axis[j], d->num_axes);
    return LA_OK;
}

la_status rope_args(const la_rope_dims *d, int32_t dtype, const void *qw, const void *kw,
                    float eps, const double *inv_freq, const void *positions,
                    const int32_t *offset, const int32_t *cu, const int32_t *cu_host,
                    cudaStream_t s, la::RopeArgs *a)
{
    la_status e = rope_sizes(d, dtype);
    if (e)
        return e;
    *a = la::RopeArgs{};
    Sequences q;
    if ((e = check_packed(d->batch, d->seq_len, d->num_seqs, cu, cu_host, s, &q)))
        return e;
    a->N = q.n;
    if (d->normalize && !(eps >= 0.f && std::isfinite(eps)))
        return fail(LA_ERR_INVALID_ARG, "eps = %g must be finite and not negative", (double)eps);
    if (!d->normalize && (qw || kw))
        return fail(LA_ERR_INVALID_ARG, "weights given without normalize");
    if (d->rotary_dim && (e = need(inv_freq, "inv_freq")))
        return e;
    if (positions) {
        if (d->position_bytes != 4 && d->position_bytes != 8)
            return fail(LA_ERR_INVALID_ARG, "position_bytes = %d must be 4 or 8",
                        d->position_bytes);
        if (offset)
            return fail(LA_ERR_INVALID_ARG, "position_offset goes with positions = NULL only");
        if ((e = check_in(d->position_strides, "positions")))
            return e;
    } else if (d->num_axes != 1 && d->rotary_dim) {
        return fail(LA_ERR_INVALID_ARG, "num_axes = %d needs positions", d->num_axes);
    }
    a->B = d->batch;
    a->T = d->seq_len;
    a->D = d->dim;
    a->R = d->rotary_dim;
    a->axes = d->num_axes;
    a->bf16 = dtype == LA_DTYPE_BF16;
    a->w_bf16 = d->weight_dtype == LA_DTYPE_BF16;
    a->normalize = d->normalize ? 1 : 0;
    a->interleaved = d->interleaved ? 1 : 0;
    a->pos64 = d->position_bytes == 8;
    a->eps = eps;
    a->inv_freq = inv_freq;
    a->pos = positions;
    a->offset = offset;
    a->cu = positions ? nullptr : cu;
    for (int i = 0; i < 3; ++i)
        a->ps[i] = d->position_strides[i];
    for (int j = 0; j < d->rotary_dim / 2; ++j)
        a->axis[j] = d->pair_axis[j];
    a->t[0].heads = d->q_heads;
    a->t[1].heads = d->k_heads;
    a->t[0].w = qw;
    a->t[1].w = kw;
    return LA_OK;
}

void put(int64_t *to, const int64_t *from)
{
    for (int i = 0; i < 3; ++i)
        to[i] = from[i];
}

bool same(const int64_t *x, const int64_t *y)
{
    return x[0] == y[0] && x[1] == y[1] && x[2] == y[2];
}

}  // namespace

extern "C" {

size_t la_gated_scan_states_size(const la_scan_dims *dims)
{
    return scan_sized(dims) ? states_bytes(dims) : 0;
}

size_t la_gated_scan_workspace_size(const la_scan_dims *dims, int32_t dtype, int32_t backward)
{
    (void)dtype;
    if (!scan_sized(dims))
        return 0;
    return round256(la::scan_maps_bytes(dims->seq_len)) +
           (backward == 3   ? round256(init_bytes(dims))
            : backward == 2 ? round256(states_bytes(dims))
                            : 0);
}

la_status la_gated_scan_fwd(const la_scan_dims *dims, int32_t dtype, const void *x,
                            const void *g, const float *initial_state, int32_t reverse,
                            const int32_t *cu_seqlens, const int32_t *cu_seqlens_host, void *o,
                            float *final_state, float *states, void *workspace,
                            size_t workspace_bytes, void *stream)
{
    return guarded([&]() -> la_status {
        cudaStream_t s = (cudaStream_t)stream;
        la::ScanArgs a;
        la_status e = scan_args(dims, dtype, x, g, initial_state, reverse, cu_seqlens,
                                cu_seqlens_host, s, &a);
        if (e || (e = check_out(dims->o_strides, "o", a.B, a.T, a.H)))
            return e;
        if ((int64_t)a.B * a.T > 0 && (e = need(o, "o")))
            return e;
        const bool in_place = final_state && final_state == initial_state;
        if ((e = check_workspace(workspace, workspace_bytes,
                                 la_gated_scan_workspace_size(dims, dtype, in_place ? 3 : 0))))
            return e;
        if (a.N == 0)
            return LA_OK;
        a.o = tok_out(o, dims->o_strides);
        a.fin = final_state;
        a.states = states;
        if (in_place && (int64_t)a.B * a.T > 0) {
            float *copy = reinterpret_cast<float *>(
                static_cast<uint8_t *>(workspace) +
                round256(la::scan_maps_bytes(a.T)));
            if ((e = launched(cudaMemcpyAsync(copy, initial_state,
                                              (size_t)a.N * a.H * a.D * sizeof(float),
                                              cudaMemcpyDeviceToDevice, s),
                              "initial state")))
                return e;
            a.init = copy;
        }
        return launched(la::scan_forward(a, workspace, s), "gated scan");
    });
}

la_status la_gated_scan_bwd(const la_scan_dims *dims, int32_t dtype, const void *x,
                            const void *g, const void *d_o, const float *initial_state,
                            const float *d_final_state, int32_t reverse,
                            const int32_t *cu_seqlens, const int32_t *cu_seqlens_host,
                            const float *states, void *dx, void *dg, float *d_initial_state,
                            void *workspace, size_t workspace_bytes, void *stream)
{
    return guarded([&]() -> la_status {
        cudaStream_t s = (cudaStream_t)stream;
        la::ScanArgs a;
        la_status e = scan_args(dims, dtype, x, g, initial_state, reverse, cu_seqlens,
                                cu_seqlens_host, s, &a);
        if (e || (e = check_in(dims->do_strides, "d_o")) ||
            (e = check_out(dims->dx_strides, "dx", a.B, a.T, a.H)) ||
            (e = check_out(dims->dg_strides, "dg", a.B, a.T, a.H)))
            return e;
        if ((int64_t)a.B * a.T > 0 &&
            ((e = need(d_o, "d_o")) || (e = need(dx, "dx")) || (e = need(dg, "dg"))))
            return e;
        if ((e = check_workspace(workspace, workspace_bytes,
                                 la_gated_scan_workspace_size(dims, dtype, states ? 1 : 2))))
            return e;
        if (a.N == 0)
            return LA_OK;
        a.states = const_cast<float *>(states);
        if (!states && states_bytes(dims)) {
            a.states = reinterpret_cast<float *>(
                static_cast<uint8_t *>(workspace) +
                round256(la::scan_maps_bytes(a.T)));
            if ((e = launched(la::scan_forward(a, workspace, s), "gated scan states")))
                return e;
        }
        a.d_o = tok(d_o, dims->do_strides);
        a.dx = tok_out(dx, dims->dx_strides);
        a.dg = tok_out(dg, dims->dg_strides);
        a.dfin = d_final_state;
        a.dinit = d_initial_state;
        return launched(la::scan_backward(a, workspace, s), "gated scan backward");
    });
}

la_status la_qk_norm_rope_fwd(const la_rope_dims *dims, int32_t dtype, const void *q,
                              const void *k, const void *q_weight, const void *k_weight,
                              float eps, const double *inv_freq, const void *positions,
                              const int32_t *position_offset, const int32_t *cu_seqlens,
                              const int32_t *cu_seqlens_host, void *qo, void *ko, void *stream)
{
    return guarded([&]() -> la_status {
        cudaStream_t s = (cudaStream_t)stream;
        la::RopeArgs a;
        la_status e = rope_args(dims, dtype, q_weight, k_weight, eps, inv_freq, positions,
                                position_offset, cu_seqlens, cu_seqlens_host, s, &a);
        if (e)
            return e;
        const bool some = (int64_t)a.B * a.T > 0;
        const void *in[2] = {q, k};
        void *out[2] = {qo, ko};
        const int64_t *is[2] = {dims->q_strides, dims->k_strides};
        const int64_t *os[2] = {dims->qo_strides, dims->ko_strides};
        for (int i = 0; i < 2; ++i) {
            la::RopeTensor &t = a.t[i];
            if (!t.heads)
                continue;
            if ((e = check_in(is[i], i ? "k" : "q")) ||
                (e = check_out(os[i], i ? "ko" : "qo", a.B, a.T, t.heads)))
                return e;
            if (some && ((e = need(in[i], i ? "k" : "q")) || (e = need(out[i], i ? "ko" : "qo"))))
                return e;
            if (some && in[i] == out[i] && !same(is[i], os[i]))
                return fail(LA_ERR_INVALID_ARG, "%s in place needs the input's strides",
                            i ? "ko" : "qo");
            t.x = in[i];
            t.y = out[i];
            put(t.xs, is[i]);
            put(t.ys, os[i]);
        }
        return some ? launched(la::rope_run(false, a, s), "norm and rotation") : LA_OK;
    });
}

size_t la_qk_norm_rope_workspace_size(const la_rope_dims *dims, int32_t dtype)
{
    if (!dims || rope_sizes(dims, dtype) != LA_OK || !dims->normalize)
        return 0;
    return la::rope_partial_bytes(dims->dim);
}

la_status la_qk_norm_rope_bwd(const la_rope_dims *dims, int32_t dtype, const void *q,
                              const void *k, const void *d_qo, const void *d_ko,
                              const void *q_weight, const void *k_weight, float eps,
                              const double *inv_freq, const void *positions,
                              const int32_t *position_offset, const int32_t *cu_seqlens,
                              const int32_t *cu_seqlens_host, void *dq, void *dk,
                              void *d_q_weight, void *d_k_weight, void *workspace,
                              size_t workspace_bytes, void *stream)
{
    return guarded([&]() -> la_status {
        cudaStream_t s = (cudaStream_t)stream;
        la::RopeArgs a;
        la_status e = rope_args(dims, dtype, q_weight, k_weight, eps, inv_freq, positions,
                                position_offset, cu_seqlens, cu_seqlens_host, s, &a);
        if (e)
            return e;
        const bool some = (int64_t)a.B * a.T > 0;
        const void *in[2] = {q, k}, *dy[2] = {d_qo, d_ko};
        void *out[2] = {dq, dk}, *dw[2] = {d_q_weight, d_k_weight};
        const int64_t *is[2] = {dims->q_strides, dims->k_strides};
        const int64_t *gs[2] = {dims->qo_strides, dims->ko_strides};
        const int64_t *os[2] = {dims->dq_strides, dims->dk_strides};
        bool weights = false;
        for (int i = 0; i < 2; ++i) {
            la::RopeTensor &t = a.t[i];
            if (dw[i] && (!dims->normalize || !t.heads))
                return fail(LA_ERR_INVALID_ARG, "%s needs normalize and the tensor itself",
                            i ? "d_k_weight" : "d_q_weight");
            if (!t.heads)
                continue;
            if ((a.normalize && (e = check_in(is[i], i ? "k" : "q"))) ||
                (e = check_in(gs[i], i ? "d_ko" : "d_qo")) ||
                (e = check_out(os[i], i ? "dk" : "dq", a.B, a.T, t.heads)))
                return e;
            if (some && ((a.normalize && (e = need(in[i], i ? "k" : "q"))) ||
                         (e = need(dy[i], i ? "d_ko" : "d_qo")) ||
                         (e = need(out[i], i ? "dk" : "dq"))))
                return e;
            t.x = in[i];
            t.dy = dy[i];
            t.y = out[i];
            t.dw = dw[i];
            weights |= dw[i] != nullptr;
            put(t.xs, is[i]);
            put(t.dys, gs[i]);
            put(t.ys, os[i]);
        }
        if (weights && (e = check_workspace(workspace, workspace_bytes,
                                            la_qk_norm_rope_workspace_size(dims, dtype))))
            return e;
        if (!some) {   // no rows: the weights' gradients are zero
            for (int i = 0; i < 2; ++i)
                if (dw[i] &&
                    (e = launched(cudaMemsetAsync(dw[i], 0, (size_t)a.D * (a.w_bf16 ? 2 : 4), s),
                                  "weight gradient")))
                    return e;
            return LA_OK;
        }
        a.partial = static_cast<float *>(workspace);
        return launched(la::rope_run(true, a, s), "norm and rotation backward");
    });
}

}  // extern "C"
