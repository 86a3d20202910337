// la_layer_api.cu -- the C entry points of the operators beside the attention
// (include/la.h): the gated linear recurrence, the norms of queries and keys
// with the position rotation, the gated delta rule, and the norms around a block.
// Argument checks, then the launches of la_scan.cu, la_qk_rope.cu,
// la_delta_token.cu, la_delta_tc.cu and la_block_norm.cu.

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

// ---- gated delta rule --------------------------------------------------------

la_status delta_sizes(const la_delta_dims *d, int32_t dtype)
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
    if (d->qk_heads < 1 || d->qk_heads > d->heads || d->heads % d->qk_heads)
        return fail(LA_ERR_INVALID_ARG, "qk_heads = %d does not divide heads = %d", d->qk_heads,
                    d->heads);
    if (d->dim_v < 1 || d->dim_v > 256)
        return fail(LA_ERR_UNSUPPORTED, "dim_v = %d: supported range is 1..256", d->dim_v);
    return check_rows(d->batch, d->seq_len, d->dim_qk);
}

// Sizes and strides; q.longest as check_packed found it.
la::DeltaArgs delta_args(const la_delta_dims *d, int32_t dtype, const Sequences &q)
{
    la::DeltaArgs a{};
    a.B = d->batch;
    a.T = d->seq_len;
    a.H = d->heads;
    a.HK = d->qk_heads;
    a.D = d->dim_qk;
    a.E = d->dim_v;
    a.N = q.n;
    a.longest = q.longest;
    a.bf16 = dtype == LA_DTYPE_BF16;
    a.gate_bf16 = d->gate_dtype == LA_DTYPE_BF16;
    a.q = tok(nullptr, d->q_strides);
    a.k = tok(nullptr, d->k_strides);
    a.v = tok(nullptr, d->v_strides);
    a.q.hdiv = a.k.hdiv = a.H / a.HK;
    a.g = tok(nullptr, d->g_strides);
    a.beta = tok(nullptr, d->beta_strides);
    return a;
}

// The sequences as a size query sees them; false: not a valid table.
bool delta_query(const la_delta_dims *d, int32_t dtype, const int32_t *cu_host, la::DeltaArgs *a)
{
    if (delta_sizes(d, dtype) != LA_OK)
        return false;
    Sequences q;
    if (cu_host) {
        // cu_host stands for both tables: only the host's is read
        if (check_packed(d->batch, d->seq_len, d->num_seqs, cu_host, cu_host, nullptr, &q) != LA_OK)
            return false;
    } else {
        q.n = d->batch;
        q.longest = d->seq_len;
    }
    *a = delta_args(d, dtype, q);
    a->cu = cu_host;
    return true;
}

size_t delta_workspace(const la::DeltaArgs &a, int backward)
{
    const bool tc = la::delta_tc_sized(a);
    if (backward == 0 || backward == 3)
        return tc ? round256(la::delta_tc_fwd_bytes(a, backward == 3)) : 0;
    if (!tc)
        return round256(la::delta_token_bwd_bytes(a));
    const size_t again = round256(la::delta_tc_saved_bytes(a)) +
                         round256(la::delta_tc_fwd_bytes(a, true));
    return round256(la::delta_tc_bwd_bytes(a)) + (backward == 2 ? again : 0);
}

la_status delta_inputs(const la_delta_dims *d, int32_t dtype, const void *q, const void *k,
                       const void *v, const void *g, const void *beta, float scale,
                       const float *init, const int32_t *cu, const int32_t *cu_host,
                       cudaStream_t s, la::DeltaArgs *a)
{
    la_status e = delta_sizes(d, dtype);
    Sequences sq;
    if (e || (e = check_in(d->q_strides, "q")) || (e = check_in(d->k_strides, "k")) ||
        (e = check_in(d->v_strides, "v")) || (e = check_in(d->g_strides, "g")) ||
        (e = check_in(d->beta_strides, "beta")))
        return e;
    if (!std::isfinite(scale))
        return fail(LA_ERR_INVALID_ARG, "scale is not finite");
    if ((e = check_packed(d->batch, d->seq_len, d->num_seqs, cu, cu_host, s, &sq)))
        return e;
    if ((int64_t)d->batch * d->seq_len > 0 &&
        ((e = need(q, "q")) || (e = need(k, "k")) || (e = need(v, "v")) || (e = need(g, "g")) ||
         (e = need(beta, "beta"))))
        return e;
    *a = delta_args(d, dtype, sq);
    a->cu = cu;
    a->scale = scale;
    a->q.p = q;
    a->k.p = k;
    a->v.p = v;
    a->g.p = g;
    a->beta.p = beta;
    a->init = init;
    return LA_OK;
}

bool delta_row(const void *p, const int64_t *st, const la::DeltaArgs &a, int heads)
{
    return la::delta_tc_row_ok(p, st, a.B, a.T, heads);
}

// ---- norms around a block ------------------------------------------------------

la_status norm_sizes(const la_block_norm_dims *d, int32_t dtype)
{
    if (!d)
        return fail(LA_ERR_INVALID_ARG, "dims is NULL");
    if (!known_dtype(dtype))
        return fail(LA_ERR_INVALID_ARG, "dtype %d is neither LA_DTYPE_BF16 nor LA_DTYPE_F32",
                    dtype);
    if (!known_dtype(d->weight_dtype))
        return fail(LA_ERR_INVALID_ARG, "weight_dtype = %d", d->weight_dtype);
    if (d->batch < 0 || d->seq_len < 0)
        return fail(LA_ERR_INVALID_ARG, "negative batch (%d) or seq_len (%d)", d->batch,
                    d->seq_len);
    if (d->heads < 1 || d->heads > 65535)
        return fail(LA_ERR_INVALID_ARG, "heads = %d outside 1..65535", d->heads);
    if (d->dim < 1 || d->dim > la::NORM_MOST_DIM)
        return fail(LA_ERR_UNSUPPORTED, "dim = %d: supported range is 1..%d", d->dim,
                    la::NORM_MOST_DIM);
    if (d->activation < 0 || d->activation > 2)
        return fail(LA_ERR_INVALID_ARG, "activation = %d outside 0..2", d->activation);
    if ((double)d->batch * d->seq_len * d->heads > INT_MAX)
        return fail(LA_ERR_UNSUPPORTED, "more than 2^31 - 1 rows");
    return LA_OK;
}

la::NormRows norm_rows(const void *p, const int64_t *st)
{
    return la::NormRows{p, {st[0], st[1], st[2]}};
}

la_status norm_args(const la_block_norm_dims *d, int32_t dtype, const void *x, const void *gate,
                    const void *residual, const void *post, const void *pre, float eps,
                    float scale, la::BlockNormArgs *a)
{
    la_status e = norm_sizes(d, dtype);
    if (e || (e = check_in(d->x_strides, "x")) ||
        (gate && (e = check_in(d->gate_strides, "gate"))) ||
        (residual && (e = check_in(d->residual_strides, "residual"))))
        return e;
    if (!(eps >= 0.f) || !std::isfinite(eps) || !std::isfinite(scale))
        return fail(LA_ERR_INVALID_ARG, "eps must be finite and not negative, scale finite");
    *a = la::BlockNormArgs{};
    a->B = d->batch;
    a->T = d->seq_len;
    a->H = d->heads;
    a->D = d->dim;
    a->rows = (int64_t)d->batch * d->seq_len * d->heads;
    if (a->rows > 0 && (e = need(x, "x")))
        return e;
    a->bf16 = dtype == LA_DTYPE_BF16;
    a->w_bf16 = d->weight_dtype == LA_DTYPE_BF16;
    a->activation = d->activation;
    a->eps = eps;
    a->scale = scale;
    a->x = norm_rows(x, d->x_strides);
    a->gate = norm_rows(gate, d->gate_strides);
    a->residual = norm_rows(residual, d->residual_strides);
    a->post = post;
    a->pre = pre;
    return LA_OK;
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

size_t la_gated_delta_workspace_size(const la_delta_dims *dims, int32_t dtype,
                                     const int32_t *cu_seqlens_host, int32_t backward)
{
    la::DeltaArgs a;
    return delta_query(dims, dtype, cu_seqlens_host, &a) ? delta_workspace(a, backward) : 0;
}

size_t la_gated_delta_saved_size(const la_delta_dims *dims, int32_t dtype,
                                 const int32_t *cu_seqlens_host)
{
    la::DeltaArgs a;
    if (!delta_query(dims, dtype, cu_seqlens_host, &a) || !la::delta_tc_sized(a))
        return 0;
    return round256(la::delta_tc_saved_bytes(a));
}

la_status la_gated_delta_fwd(const la_delta_dims *dims, int32_t dtype, const void *q,
                             const void *k, const void *v, const void *g, const void *beta,
                             float scale, const float *initial_state, const int32_t *cu_seqlens,
                             const int32_t *cu_seqlens_host, void *o, float *final_state,
                             void *saved, void *workspace, size_t workspace_bytes, void *stream)
{
    return guarded([&]() -> la_status {
        cudaStream_t s = (cudaStream_t)stream;
        la::DeltaArgs a;
        la_status e = delta_inputs(dims, dtype, q, k, v, g, beta, scale, initial_state,
                                   cu_seqlens, cu_seqlens_host, s, &a);
        if (e || (e = check_out(dims->o_strides, "o", a.B, a.T, a.H)))
            return e;
        if ((int64_t)a.B * a.T > 0 && (e = need(o, "o")))
            return e;
        bool tc = la::delta_tc_sized(a);
        if (tc && !(delta_row(q, dims->q_strides, a, a.HK) &&
                    delta_row(k, dims->k_strides, a, a.HK) &&
                    delta_row(v, dims->v_strides, a, a.H) &&
                    delta_row(o, dims->o_strides, a, a.H))) {
            if (saved)
                return fail(LA_ERR_INVALID_ARG, "with saved, q, k, v and o must start on 16-byte "
                                                "boundaries, with strides of whole 16 bytes");
            tc = false;
        }
        if ((e = check_workspace(workspace, workspace_bytes,
                                 delta_workspace(a, saved ? 3 : 0))))
            return e;
        if (saved && (reinterpret_cast<uintptr_t>(saved) & 255))
            return fail(LA_ERR_INVALID_ARG, "saved is not 256-byte aligned");
        a.o = tok_out(o, dims->o_strides);
        a.fin = final_state;
        a.saved = static_cast<uint8_t *>(saved);
        a.ws = static_cast<uint8_t *>(workspace);
        if (tc) {
            a.withhold_handoff = la::take_withheld();
            return launched(la::delta_tc_forward(a, s), "gated delta rule");
        }
        return launched(la::delta_token_forward(a, s), "gated delta rule");
    });
}

la_status la_gated_delta_bwd(const la_delta_dims *dims, int32_t dtype, const void *q,
                             const void *k, const void *v, const void *g, const void *beta,
                             const void *d_o, float scale, const float *initial_state,
                             const float *d_final_state, const int32_t *cu_seqlens,
                             const int32_t *cu_seqlens_host, const void *saved, void *dq,
                             void *dk, void *dv, void *dg, void *dbeta, float *d_initial_state,
                             void *workspace, size_t workspace_bytes, void *stream)
{
    return guarded([&]() -> la_status {
        cudaStream_t s = (cudaStream_t)stream;
        la::DeltaArgs a;
        la_status e = delta_inputs(dims, dtype, q, k, v, g, beta, scale, initial_state,
                                   cu_seqlens, cu_seqlens_host, s, &a);
        if (e || (e = check_in(dims->do_strides, "d_o")) ||
            (e = check_out(dims->dq_strides, "dq", a.B, a.T, a.HK)) ||
            (e = check_out(dims->dk_strides, "dk", a.B, a.T, a.HK)) ||
            (e = check_out(dims->dv_strides, "dv", a.B, a.T, a.H)))
            return e;
        if ((int64_t)a.B * a.T > 0 &&
            ((e = need(d_o, "d_o")) || (e = need(dq, "dq")) || (e = need(dk, "dk")) ||
             (e = need(dv, "dv")) || (e = need(dg, "dg")) || (e = need(dbeta, "dbeta"))))
            return e;
        const bool tc = la::delta_tc_sized(a);
        if (tc && !(delta_row(q, dims->q_strides, a, a.HK) &&
                    delta_row(k, dims->k_strides, a, a.HK) &&
                    delta_row(v, dims->v_strides, a, a.H) &&
                    delta_row(d_o, dims->do_strides, a, a.H) &&
                    delta_row(dq, dims->dq_strides, a, a.HK) &&
                    delta_row(dk, dims->dk_strides, a, a.HK) &&
                    delta_row(dv, dims->dv_strides, a, a.H)))
            return fail(LA_ERR_INVALID_ARG,
                        "q, k, v, d_o, dq, dk and dv must start on 16-byte boundaries, with "
                        "strides of whole 16 bytes");
        if ((e = check_workspace(workspace, workspace_bytes, delta_workspace(a, saved ? 1 : 2))))
            return e;
        if (saved && (reinterpret_cast<uintptr_t>(saved) & 255))
            return fail(LA_ERR_INVALID_ARG, "saved is not 256-byte aligned");
        a.d_o = tok(d_o, dims->do_strides);
        a.dq = tok_out(dq, dims->dq_strides);
        a.dk = tok_out(dk, dims->dk_strides);
        a.dv = tok_out(dv, dims->dv_strides);
        a.dg = dg;
        a.dbeta = dbeta;
        a.dfin = d_final_state;
        a.dinit = d_initial_state;
        a.ws = static_cast<uint8_t *>(workspace);
        if (!tc)
            return launched(la::delta_token_backward(a, s), "gated delta rule backward");
        a.withhold_handoff = la::take_withheld();
        a.saved = static_cast<uint8_t *>(const_cast<void *>(saved));
        if (!saved) {   // the forward again, without its outputs
            la::DeltaArgs f = a;
            const size_t own = round256(la::delta_tc_bwd_bytes(a));
            f.withhold_handoff = 0;
            f.saved = a.saved = a.ws + own;
            f.ws = f.saved + round256(la::delta_tc_saved_bytes(a));
            if ((e = launched(la::delta_tc_forward(f, s), "gated delta rule states")))
                return e;
        }
        return launched(la::delta_tc_backward(a, s), "gated delta rule backward");
    });
}

la_status la_block_norm_fwd(const la_block_norm_dims *dims, int32_t dtype, const void *x,
                            const void *gate, const void *residual, const void *post_weight,
                            const void *pre_weight, float eps, float scale, void *h, void *y,
                            void *stream)
{
    return guarded([&]() -> la_status {
        la::BlockNormArgs a;
        la_status e = norm_args(dims, dtype, x, gate, residual, post_weight, pre_weight, eps,
                                scale, &a);
        if (e || (e = check_out(dims->h_strides, "h", a.B, a.T, a.H)) ||
            (y && (e = check_out(dims->y_strides, "y", a.B, a.T, a.H))))
            return e;
        if (y && !pre_weight)
            return fail(LA_ERR_INVALID_ARG, "y needs pre_weight");
        if (a.rows == 0)
            return LA_OK;
        if ((e = need(h, "h")) || (pre_weight && (e = need(y, "y"))))
            return e;
        if (y == h || y == x || (gate && (y == gate || h == gate)) || (residual && y == residual))
            return fail(LA_ERR_INVALID_ARG, "an output overlaps an input or the other output");
        if ((h == x && !same(dims->h_strides, dims->x_strides)) ||
            (h == residual && !same(dims->h_strides, dims->residual_strides)))
            return fail(LA_ERR_INVALID_ARG, "h in place needs the input's strides");
        a.h = norm_rows(h, dims->h_strides);
        a.y = norm_rows(y, dims->y_strides);
        return launched(la::block_norm_run(false, a, (cudaStream_t)stream), "block norm");
    });
}

size_t la_block_norm_workspace_size(const la_block_norm_dims *dims, int32_t dtype)
{
    return norm_sizes(dims, dtype) == LA_OK ? la::block_norm_partial_bytes(dims->dim) : 0;
}

la_status la_block_norm_bwd(const la_block_norm_dims *dims, int32_t dtype, const void *x,
                            const void *gate, const void *residual, const void *post_weight,
                            const void *pre_weight, float eps, float scale, const void *d_h,
                            const void *d_y, void *dx, void *d_gate, void *d_residual,
                            void *d_post_weight, void *d_pre_weight, void *workspace,
                            size_t workspace_bytes, void *stream)
{
    return guarded([&]() -> la_status {
        cudaStream_t s = (cudaStream_t)stream;
        la::BlockNormArgs a;
        la_status e = norm_args(dims, dtype, x, gate, residual, post_weight, pre_weight, eps,
                                scale, &a);
        if (e || (d_h && (e = check_in(dims->dh_strides, "d_h"))) ||
            (d_y && (e = check_in(dims->dy_strides, "d_y"))) ||
            (e = check_out(dims->dx_strides, "dx", a.B, a.T, a.H)) ||
            (d_gate && (e = check_out(dims->dgate_strides, "d_gate", a.B, a.T, a.H))) ||
            (d_residual &&
             (e = check_out(dims->dresidual_strides, "d_residual", a.B, a.T, a.H))))
            return e;
        if ((d_y || d_pre_weight) && !pre_weight)
            return fail(LA_ERR_INVALID_ARG, "d_y and d_pre_weight need pre_weight");
        if (d_post_weight && !post_weight)
            return fail(LA_ERR_INVALID_ARG, "d_post_weight needs post_weight");
        if (d_gate && !gate)
            return fail(LA_ERR_INVALID_ARG, "d_gate needs gate");
        const size_t wide = a.w_bf16 ? 2 : 4;
        if (a.rows == 0) {  // no rows: the weights' gradients are zero
            for (void *w : {d_post_weight, d_pre_weight})
                if (w && (e = launched(cudaMemsetAsync(w, 0, a.D * wide, s), "weight gradient")))
                    return e;
            return LA_OK;
        }
        if ((e = need(dx, "dx")) || (gate && (e = need(d_gate, "d_gate"))) ||
            (pre_weight ? (e = need(d_y, "d_y")) : (e = need(d_h, "d_h"))))
            return e;
        if ((d_post_weight || d_pre_weight) &&
            (e = check_workspace(workspace, workspace_bytes,
                                 la_block_norm_workspace_size(dims, dtype))))
            return e;
        a.dh = norm_rows(d_h, dims->dh_strides);
        a.dy = norm_rows(d_y, dims->dy_strides);
        a.dx = norm_rows(dx, dims->dx_strides);
        a.dgate = norm_rows(d_gate, dims->dgate_strides);
        a.dresidual = norm_rows(d_residual, dims->dresidual_strides);
        a.dpost = d_post_weight;
        a.dpre = d_pre_weight;
        a.partial = static_cast<float *>(workspace);
        return launched(la::block_norm_run(true, a, s), "block norm backward");
    });
}

}  // extern "C"
