// abi_layers.hip -- the extern "C" boundary of the RMS norm, linear attention and token log probabilities: argument
// validation and dispatch, with the rules of abi_recurrent.hip (every check before the first HIP call, scratch from the
// caller).
#include <limits.h>

#include <algorithm>

#include "abi_checks.hpp"
#include "mamba_scan.h"
#include "mss_internal.hpp"

namespace {

using namespace mss::abi;

int status(hipError_t e) { return e == hipSuccess ? MSS_OK : MSS_ERR_HIP; }

// t has the extents of `like` but its last one, and then, with last >= 0, `last`.
bool lead_is(const mss_tensor_t* t, const mss_tensor_t& like, int64_t last = -1) {
    if (!t) return true;
    const int lead = like.ndim - 1;
    if (t->ndim != lead + (last >= 0 ? 1 : 0)) return false;
    for (int i = 0; i < lead; ++i)
        if (t->shape[i] != like.shape[i]) return false;
    return last < 0 || t->shape[lead] == last;
}
bool same_shape(const mss_tensor_t* t, const mss_tensor_t& like) { return lead_is(t, like, like.shape[like.ndim - 1]); }

bool in_place(const mss_tensor_t* out, const mss_tensor_t* in) { return out && in && out->data == in->data; }

// Sizes of an attention call; MSS_OK, or what is wrong with them.
int check_sizes(int64_t Bt, int64_t L, int64_t H, int64_t Hq, int64_t Hk, int64_t Hv, int64_t K, int64_t V) {
    if (Bt < 0 || L < 0 || H < 1 || Hq < 1 || Hk < 1 || Hv < 1 || K < 1 || V < 1) return MSS_ERR_SHAPE;
    if (H % Hq || H % Hk || H % Hv) return MSS_ERR_SHAPE;
    if (H > 32768) return MSS_ERR_UNSUPPORTED;  // a chunk's offsets are 32 bits
    if (K % 16 || V % 16 || K > mss::kAttnMostDim || V > mss::kAttnMostDim) return MSS_ERR_UNSUPPORTED;
    int64_t n = 0;
    if (L > INT32_MAX) return MSS_ERR_UNSUPPORTED;
    if (__builtin_mul_overflow(Bt, H, &n) || n > (int64_t{1} << 20)) return MSS_ERR_UNSUPPORTED;  // 2^32 threads a launch
    if (__builtin_mul_overflow(n, L, &n) || n > (int64_t{1} << 40)) return MSS_ERR_UNSUPPORTED;
    return MSS_OK;
}

bool all_aligned(Ts ts) {
    for (const mss_tensor_t* t : ts)
        if (t && numel(*t) > 0 && !aligned(*t, 16)) return false;
    return true;
}

}  // namespace

extern "C" {

int mss_rms_norm_fwd(const mss_tensor_t* x, const mss_tensor_t* residual, const mss_tensor_t* weight, float eps,
                     const mss_tensor_t* out, const mss_tensor_t* residual_out, const mss_tensor_t* rstd,
                     const mss_tensor_t* scales, void* stream) {
    try {
        const mss_tensor_t* const req[] = {x, weight, out};
        int st = check_descs(req, {residual, residual_out, rstd, scales});
        if (st != MSS_OK) return st;
        if (!residual != !residual_out) return MSS_ERR_NULL_ARG;
        if (!scales && out->dtype == MSS_F8E4M3) return MSS_ERR_NULL_ARG;
        if (x->ndim < 2) return MSS_ERR_SHAPE;
        const int64_t W = x->shape[x->ndim - 1], parts = (W + 127) / 128;
        if (W < 1 || !shape_is(*weight, 1, W) || !(eps >= 0.0f)) return MSS_ERR_SHAPE;
        for (const mss_tensor_t* t : {residual, out, residual_out})
            if (t && !same_shape(t, *x)) return MSS_ERR_SHAPE;
        if (!lead_is(rstd, *x) || (!lead_is(scales, *x, 1) && !lead_is(scales, *x, parts))) return MSS_ERR_SHAPE;
        if (!act_dtype(x->dtype) || (residual && !act_dtype(residual->dtype)) ||
            (residual && residual_out->dtype != residual->dtype) || !all_dtype({weight, rstd, scales}, MSS_F32) ||
            out->dtype != (scales ? static_cast<int32_t>(MSS_F8E4M3) : x->dtype))
            return MSS_ERR_DTYPE;
        if (!laid_out({x, residual, weight, out, residual_out, rstd, scales})) return MSS_ERR_LAYOUT;
        if (!apart({x, weight}, {out, residual_out, rstd, scales}) ||
            !apart({residual}, {out, in_place(residual_out, residual) ? nullptr : residual_out, rstd, scales}))
            return MSS_ERR_ALIAS;
        if (W > mss::kNormWidest) return MSS_ERR_UNSUPPORTED;
        mss::NormLaunch a;
        a.x = x->data; a.residual = residual ? residual->data : nullptr; a.weight = static_cast<const float*>(weight->data);
        a.out = out->data; a.residual_out = residual ? residual_out->data : nullptr; a.rstd = ptr<float>(rstd);
        a.scales = ptr<float>(scales);
        a.W = W; a.R = numel(*x) / W; a.eps = eps;
        a.G = scales ? static_cast<int>(scales->shape[scales->ndim - 1]) : 1;
        a.x_bf16 = x->dtype == MSS_BF16; a.residual_bf16 = residual && residual->dtype == MSS_BF16;
        a.vec_ok = whole_vectors(W, x->dtype, {x, scales ? nullptr : out}) &&
                   (!residual || whole_vectors(W, residual->dtype, {residual, residual_out})) &&
                   (!scales || (W % 8 == 0 && aligned(*out, 8)));
        if (a.R == 0) return MSS_OK;
        return status(mss::launch_rms_norm_fwd(a, static_cast<hipStream_t>(stream)));
    } catch (...) {
        return MSS_ERR_HIP;
    }
}

int mss_rms_norm_bwd_scratch(int64_t rows, int64_t width, int64_t* floats) {
    if (!floats) return MSS_ERR_NULL_ARG;
    int64_t n = 0;
    if (rows < 0 || width < 1 || __builtin_mul_overflow(rows, width, &n) || n > (int64_t{1} << 48)) return MSS_ERR_SHAPE;
    if (width > mss::kNormWidest) return MSS_ERR_UNSUPPORTED;
    *floats = mss::rms_norm_bwd_scratch(rows, width);
    return MSS_OK;
}

int mss_rms_norm_bwd(const mss_tensor_t* z, const mss_tensor_t* weight, const mss_tensor_t* rstd,
                     const mss_tensor_t* dout, const mss_tensor_t* dresidual_out, const mss_tensor_t* dx,
                     const mss_tensor_t* dresidual, const mss_tensor_t* dweight, const mss_tensor_t* scratch,
                     void* stream) {
    try {
        const mss_tensor_t* const req[] = {z, weight, rstd, dout, dx};
        int st = check_descs(req, {dresidual_out, dresidual, dweight});
        if (st != MSS_OK) return st;
        if (z->ndim < 2) return MSS_ERR_SHAPE;
        const int64_t W = z->shape[z->ndim - 1];
        if (W < 1 || !shape_is(*weight, 1, W) || (dweight && !shape_is(*dweight, 1, W)) || !lead_is(rstd, *z))
            return MSS_ERR_SHAPE;
        for (const mss_tensor_t* t : {dout, dresidual_out, dx, dresidual})
            if (t && !same_shape(t, *z)) return MSS_ERR_SHAPE;
        if (!act_dtype(z->dtype) || !act_dtype(dout->dtype) || dx->dtype != dout->dtype ||
            !all_dtype({dresidual_out, dresidual}, z->dtype) || !all_dtype({weight, rstd, dweight}, MSS_F32))
            return MSS_ERR_DTYPE;
        if (!laid_out({z, weight, rstd, dout, dresidual_out, dx, dresidual, dweight})) return MSS_ERR_LAYOUT;
        if (W > mss::kNormWidest) return MSS_ERR_UNSUPPORTED;
        const int64_t R = numel(*z) / W;
        if (dweight && (st = check_scratch(scratch, mss::rms_norm_bwd_scratch(R, W))) != MSS_OK) return st;
        if (!apart({z, weight, rstd, dout, dresidual_out}, {dx, dresidual, dweight, dweight ? scratch : nullptr}))
            return MSS_ERR_ALIAS;
        mss::NormBwdLaunch a;
        a.z = z->data; a.weight = static_cast<const float*>(weight->data); a.rstd = static_cast<const float*>(rstd->data);
        a.dout = dout->data; a.dresidual_out = ptr<const void>(dresidual_out); a.dx = dx->data;
        a.dresidual = ptr<void>(dresidual); a.dweight = ptr<float>(dweight); a.scratch = dweight ? ptr<float>(scratch) : nullptr;
        a.R = R; a.W = W;
        a.x_bf16 = dout->dtype == MSS_BF16; a.z_bf16 = z->dtype == MSS_BF16;
        a.vec_ok = whole_vectors(W, z->dtype, {z, dresidual_out, dresidual}) && whole_vectors(W, dout->dtype, {dout, dx});
        if (R == 0 && !dweight) return MSS_OK;  // with no rows dweight is still written (zeros)
        return status(mss::launch_rms_norm_bwd(a, static_cast<hipStream_t>(stream)));
    } catch (...) {
        return MSS_ERR_HIP;
    }
}

int mss_linear_attention_scratch(int64_t batch, int64_t L, int64_t heads, int64_t q_heads, int64_t k_heads,
                                 int64_t v_heads, int64_t key_dim, int64_t value_dim, int64_t* fwd, int64_t* bwd) {
    if (!fwd || !bwd) return MSS_ERR_NULL_ARG;
    const int st = check_sizes(batch, L, heads, q_heads, k_heads, v_heads, key_dim, value_dim);
    if (st != MSS_OK) return st;
    const auto n = [](int64_t v) { return static_cast<int>(v); };
    *fwd = *bwd = 0;
    for (const bool bf16 : {false, true}) {  // what either type needs
        *fwd = std::max(*fwd, mss::attn_fwd_scratch(batch, L, n(heads), n(key_dim), n(value_dim), bf16));
        *bwd = std::max(*bwd, mss::attn_bwd_scratch(batch, L, n(heads), n(q_heads), n(k_heads), n(v_heads), n(key_dim),
                                                    n(value_dim), bf16));
    }
    return MSS_OK;
}

int mss_linear_attention_fwd(const mss_tensor_t* q, const mss_tensor_t* k, const mss_tensor_t* v,
                             const mss_tensor_t* rate, float scale, const mss_tensor_t* initial_state,
                             const mss_tensor_t* seq_lens, const mss_tensor_t* out, const mss_tensor_t* last_state,
                             const mss_tensor_t* scratch, void* stream) {
    try {
        const mss_tensor_t* const req[] = {q, k, v, rate, out};
        int st = check_descs(req, {initial_state, seq_lens, last_state});
        if (st != MSS_OK) return st;
        if (q->ndim != 4 || k->ndim != 4 || v->ndim != 4 || rate->ndim != 1) return MSS_ERR_SHAPE;
        const int64_t Bt = q->shape[0], L = q->shape[1], Hq = q->shape[2], K = q->shape[3], Hk = k->shape[2],
                      Hv = v->shape[2], V = v->shape[3], H = rate->shape[0];
        if (!shape_is(*k, 4, Bt, L, Hk, K) || !shape_is(*v, 4, Bt, L, Hv, V) || !shape_is(*out, 4, Bt, L, H, V))
            return MSS_ERR_SHAPE;
        for (const mss_tensor_t* t : {initial_state, last_state})
            if (t && !shape_is(*t, 4, Bt, H, K, V)) return MSS_ERR_SHAPE;
        if (seq_lens && !shape_is(*seq_lens, 1, Bt)) return MSS_ERR_SHAPE;
        st = check_sizes(Bt, L, H, Hq, Hk, Hv, K, V);
        if (st == MSS_ERR_SHAPE) return st;
        if (!act_dtype(q->dtype) || !all_dtype({k, v, out}, q->dtype) ||
            !all_dtype({rate, initial_state, last_state}, MSS_F32) || !all_dtype({seq_lens}, MSS_I32))
            return MSS_ERR_DTYPE;
        if (!laid_out({q, k, v, rate, initial_state, seq_lens, out, last_state}) ||
            !all_aligned({q, k, v, initial_state, out, last_state}))
            return MSS_ERR_LAYOUT;
        if (st != MSS_OK) return st;
        const int h = static_cast<int>(H);
        st = check_scratch(scratch, mss::attn_fwd_scratch(Bt, L, h, static_cast<int>(K), static_cast<int>(V),
                                                           q->dtype == MSS_BF16));
        if (st != MSS_OK) return st;
        if (!apart({q, k, v, rate, initial_state, seq_lens}, {out, last_state, scratch})) return MSS_ERR_ALIAS;
        mss::AttnLaunch a;
        a.q = q->data; a.k = k->data; a.v = v->data; a.rate = static_cast<const float*>(rate->data);
        a.h0 = ptr<const float>(initial_state); a.lens = ptr<const int32_t>(seq_lens); a.out = out->data;
        a.last_state = ptr<float>(last_state); a.scratch = ptr<float>(scratch);
        a.Bt = Bt; a.L = L; a.H = h; a.Hq = static_cast<int>(Hq); a.Hk = static_cast<int>(Hk);
        a.Hv = static_cast<int>(Hv); a.K = static_cast<int>(K); a.V = static_cast<int>(V);
        a.scale = scale;
        a.bf16 = q->dtype == MSS_BF16;
        if (Bt == 0 || (L == 0 && !last_state)) return MSS_OK;
        return status(mss::launch_attn_fwd(a, static_cast<hipStream_t>(stream)));
    } catch (...) {
        return MSS_ERR_HIP;
    }
}

int mss_linear_attention_bwd(const mss_tensor_t* q, const mss_tensor_t* k, const mss_tensor_t* v,
                             const mss_tensor_t* rate, float scale, const mss_tensor_t* initial_state,
                             const mss_tensor_t* seq_lens, const mss_tensor_t* dout, const mss_tensor_t* dlast_state,
                             const mss_tensor_t* dq, const mss_tensor_t* dk, const mss_tensor_t* dv,
                             const mss_tensor_t* dinitial_state, const mss_tensor_t* scratch, void* stream) {
    try {
        const mss_tensor_t* const req[] = {q, k, v, rate, dout, dq, dk, dv};
        int st = check_descs(req, {initial_state, seq_lens, dlast_state, dinitial_state});
        if (st != MSS_OK) return st;
        if (q->ndim != 4 || k->ndim != 4 || v->ndim != 4 || rate->ndim != 1) return MSS_ERR_SHAPE;
        const int64_t Bt = q->shape[0], L = q->shape[1], Hq = q->shape[2], K = q->shape[3], Hk = k->shape[2],
                      Hv = v->shape[2], V = v->shape[3], H = rate->shape[0];
        if (!shape_is(*k, 4, Bt, L, Hk, K) || !shape_is(*v, 4, Bt, L, Hv, V) || !shape_is(*dout, 4, Bt, L, H, V) ||
            !shape_is(*dq, 4, Bt, L, Hq, K) || !shape_is(*dk, 4, Bt, L, Hk, K) || !shape_is(*dv, 4, Bt, L, Hv, V))
            return MSS_ERR_SHAPE;
        for (const mss_tensor_t* t : {initial_state, dlast_state, dinitial_state})
            if (t && !shape_is(*t, 4, Bt, H, K, V)) return MSS_ERR_SHAPE;
        if (seq_lens && !shape_is(*seq_lens, 1, Bt)) return MSS_ERR_SHAPE;
        st = check_sizes(Bt, L, H, Hq, Hk, Hv, K, V);
        if (st == MSS_ERR_SHAPE) return st;
        if (!act_dtype(q->dtype) || !all_dtype({k, v, dout, dq, dk, dv}, q->dtype) ||
            !all_dtype({rate, initial_state, dlast_state, dinitial_state}, MSS_F32) || !all_dtype({seq_lens}, MSS_I32))
            return MSS_ERR_DTYPE;
        if (!laid_out({q, k, v, rate, initial_state, seq_lens, dout, dlast_state, dq, dk, dv, dinitial_state}) ||
            !all_aligned({q, k, v, initial_state, dout, dlast_state, dq, dk, dv, dinitial_state}))
            return MSS_ERR_LAYOUT;
        if (st != MSS_OK) return st;
        mss::AttnLaunch a;
        a.q = q->data; a.k = k->data; a.v = v->data; a.rate = static_cast<const float*>(rate->data);
        a.h0 = ptr<const float>(initial_state); a.lens = ptr<const int32_t>(seq_lens); a.dout = dout->data;
        a.dlast = ptr<const float>(dlast_state); a.dq = dq->data; a.dk = dk->data; a.dv = dv->data;
        a.dh0 = ptr<float>(dinitial_state);
        a.Bt = Bt; a.L = L; a.H = static_cast<int>(H); a.Hq = static_cast<int>(Hq); a.Hk = static_cast<int>(Hk);
        a.Hv = static_cast<int>(Hv); a.K = static_cast<int>(K); a.V = static_cast<int>(V);
        a.scale = scale;
        a.bf16 = q->dtype == MSS_BF16;
        st = check_scratch(scratch, mss::attn_bwd_scratch(Bt, L, a.H, a.Hq, a.Hk, a.Hv, a.K, a.V, a.bf16));
        if (st != MSS_OK) return st;
        a.scratch = ptr<float>(scratch);
        if (!apart({q, k, v, rate, initial_state, seq_lens, dout, dlast_state}, {dq, dk, dv, dinitial_state, scratch}))
            return MSS_ERR_ALIAS;
        if (Bt == 0 || (L == 0 && !dinitial_state)) return MSS_OK;
        return status(mss::launch_attn_bwd(a, static_cast<hipStream_t>(stream)));
    } catch (...) {
        return MSS_ERR_HIP;
    }
}

int mss_linear_attention_update(const mss_tensor_t* state, const mss_tensor_t* q, const mss_tensor_t* k,
                                const mss_tensor_t* v, const mss_tensor_t* rate, float scale, const mss_tensor_t* out,
                                void* stream) {
    try {
        const mss_tensor_t* const req[] = {state, q, k, v, rate, out};
        int st = check_descs(req, {});
        if (st != MSS_OK) return st;
        if (state->ndim != 4 || q->ndim != 3 || k->ndim != 3 || v->ndim != 3) return MSS_ERR_SHAPE;
        const int64_t Bt = state->shape[0], H = state->shape[1], K = state->shape[2], V = state->shape[3],
                      Hq = q->shape[1], Hk = k->shape[1], Hv = v->shape[1];
        if (!shape_is(*q, 3, Bt, Hq, K) || !shape_is(*k, 3, Bt, Hk, K) || !shape_is(*v, 3, Bt, Hv, V) ||
            !shape_is(*rate, 1, H) || !shape_is(*out, 3, Bt, H, V))
            return MSS_ERR_SHAPE;
        st = check_sizes(Bt, 1, H, Hq, Hk, Hv, K, V);
        if (st == MSS_ERR_SHAPE) return st;
        if (!act_dtype(q->dtype) || !all_dtype({k, v, out}, q->dtype) || !all_dtype({state, rate}, MSS_F32))
            return MSS_ERR_DTYPE;
        if (!laid_out({state, q, k, v, rate, out}) || !all_aligned({state})) return MSS_ERR_LAYOUT;
        if (st != MSS_OK) return st;
        if (!apart({q, k, v, rate}, {state, out})) return MSS_ERR_ALIAS;
        mss::AttnUpdateLaunch a;
        a.state = static_cast<float*>(state->data); a.q = q->data; a.k = k->data; a.v = v->data;
        a.rate = static_cast<const float*>(rate->data); a.out = out->data;
        a.Bt = Bt; a.H = static_cast<int>(H); a.Hq = static_cast<int>(Hq); a.Hk = static_cast<int>(Hk);
        a.Hv = static_cast<int>(Hv); a.K = static_cast<int>(K); a.V = static_cast<int>(V);
        a.scale = scale;
        a.bf16 = q->dtype == MSS_BF16;
        if (Bt == 0) return MSS_OK;
        return status(mss::launch_attn_update(a, static_cast<hipStream_t>(stream)));
    } catch (...) {
        return MSS_ERR_HIP;
    }
}

int mss_token_logprobs_scratch(int64_t rows, int64_t vocab, int64_t top, int64_t* floats) {
    if (!floats) return MSS_ERR_NULL_ARG;
    int64_t n = 0;
    if (rows < 0 || vocab < 1 || top < 0 || __builtin_mul_overflow(rows, vocab, &n) || n > (int64_t{1} << 48))
        return MSS_ERR_SHAPE;
    if (vocab > INT32_MAX || top > mss::kBeamMost) return MSS_ERR_UNSUPPORTED;
    *floats = mss::logprob_scratch(rows, vocab, top);
    return MSS_OK;
}

int mss_token_logprobs_fwd(const mss_tensor_t* logits, const mss_tensor_t* tokens, const mss_tensor_t* logprobs,
                           const mss_tensor_t* entropy, const mss_tensor_t* top_logprobs,
                           const mss_tensor_t* top_tokens, const mss_tensor_t* saved, const mss_tensor_t* scratch,
                           void* stream) {
    try {
        const mss_tensor_t* const req[] = {logits, tokens, logprobs};
        int st = check_descs(req, {entropy, top_logprobs, top_tokens, saved});
        if (st != MSS_OK) return st;
        if (!top_logprobs != !top_tokens) return MSS_ERR_NULL_ARG;
        if (logits->ndim < 2) return MSS_ERR_SHAPE;
        const int64_t V = logits->shape[logits->ndim - 1], K = top_tokens ? top_tokens->shape[top_tokens->ndim - 1] : 0;
        if (V < 1 || (top_tokens && K < 1)) return MSS_ERR_SHAPE;
        if (!lead_is(tokens, *logits) || !lead_is(logprobs, *logits) || !lead_is(entropy, *logits) ||
            !lead_is(top_logprobs, *logits, K) || !lead_is(top_tokens, *logits, K) || !lead_is(saved, *logits, 3))
            return MSS_ERR_SHAPE;
        if (!act_dtype(logits->dtype) || !all_dtype({logprobs, entropy, top_logprobs, saved}, MSS_F32) ||
            !all_dtype({tokens, top_tokens}, MSS_I32))
            return MSS_ERR_DTYPE;
        if (!laid_out({logits, tokens, logprobs, entropy, top_logprobs, top_tokens, saved})) return MSS_ERR_LAYOUT;
        if (V > INT32_MAX || K > mss::kBeamMost) return MSS_ERR_UNSUPPORTED;
        const int64_t R = numel(*logits) / V;
        if ((st = check_scratch(scratch, mss::logprob_scratch(R, V, K))) != MSS_OK) return st;
        if (!apart({logits, tokens}, {logprobs, entropy, top_logprobs, top_tokens, saved, scratch})) return MSS_ERR_ALIAS;
        mss::LogprobLaunch a;
        a.logits = logits->data; a.tokens = static_cast<const int32_t*>(tokens->data);
        a.logprobs = static_cast<float*>(logprobs->data); a.entropy = ptr<float>(entropy);
        a.top_logprobs = ptr<float>(top_logprobs); a.top_tokens = ptr<int32_t>(top_tokens); a.saved = ptr<float>(saved);
        a.scratch = ptr<float>(scratch);
        a.R = R; a.V = V; a.K = static_cast<int>(K);
        a.bf16 = logits->dtype == MSS_BF16;
        if (R == 0) return MSS_OK;
        return status(mss::launch_logprob_fwd(a, static_cast<hipStream_t>(stream)));
    } catch (...) {
        return MSS_ERR_HIP;
    }
}

int mss_token_logprobs_bwd(const mss_tensor_t* logits, const mss_tensor_t* tokens, const mss_tensor_t* saved,
                           const mss_tensor_t* dlogprobs, const mss_tensor_t* dentropy, const mss_tensor_t* dlogits,
                           void* stream) {
    try {
        const mss_tensor_t* const req[] = {logits, tokens, saved, dlogprobs, dlogits};
        int st = check_descs(req, {dentropy});
        if (st != MSS_OK) return st;
        if (logits->ndim < 2) return MSS_ERR_SHAPE;
        const int64_t V = logits->shape[logits->ndim - 1];
        if (V < 1 || !lead_is(tokens, *logits) || !lead_is(saved, *logits, 3) || !lead_is(dlogprobs, *logits) ||
            !lead_is(dentropy, *logits) || !same_shape(dlogits, *logits))
            return MSS_ERR_SHAPE;
        if (!act_dtype(logits->dtype) || dlogits->dtype != logits->dtype ||
            !all_dtype({saved, dlogprobs, dentropy}, MSS_F32) || !all_dtype({tokens}, MSS_I32))
            return MSS_ERR_DTYPE;
        if (!laid_out({logits, tokens, saved, dlogprobs, dentropy, dlogits})) return MSS_ERR_LAYOUT;
        if (V > INT32_MAX) return MSS_ERR_UNSUPPORTED;
        if (!apart({tokens, saved, dlogprobs, dentropy, in_place(dlogits, logits) ? nullptr : logits}, {dlogits}))
            return MSS_ERR_ALIAS;
        mss::LogprobBwdLaunch a;
        a.logits = logits->data; a.tokens = static_cast<const int32_t*>(tokens->data);
        a.saved = static_cast<const float*>(saved->data); a.dlogprobs = static_cast<const float*>(dlogprobs->data);
        a.dentropy = ptr<const float>(dentropy); a.dlogits = dlogits->data;
        a.V = V; a.R = numel(*logits) / V;
        a.bf16 = logits->dtype == MSS_BF16;
        a.vec_ok = whole_vectors(V, logits->dtype, {logits, dlogits});
        if (a.R == 0) return MSS_OK;
        return status(mss::launch_logprob_bwd(a, static_cast<hipStream_t>(stream)));
    } catch (...) {
        return MSS_ERR_HIP;
    }
}

}  // extern "C"
