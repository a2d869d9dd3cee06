// abi_recurrent.hip -- the extern "C" boundary of the gated scan, the conv's gradients and beam
// search: argument validation and dispatch.  Every check runs before the first HIP call.  These
// entry points own no workspace: scratch comes from the caller, so calls on any streams, host
// threads and captured graphs are independent as long as their scratch is.
#include <algorithm>
#include <vector>

#include "abi_checks.hpp"
#include "mamba_scan.h"
#include "mss_internal.hpp"

namespace {

using namespace mss::abi;

int status(hipError_t e) { return e == hipSuccess ? MSS_OK : MSS_ERR_HIP; }

}  // namespace

extern "C" {

int mss_gated_scan_scratch(int64_t batch, int64_t d_inner, int64_t L, int64_t* fwd, int64_t* bwd) {
    if (!fwd || !bwd) return MSS_ERR_NULL_ARG;
    int64_t n = 0;
    if (batch < 0 || d_inner < 0 || L < 0) return MSS_ERR_SHAPE;
    if (__builtin_mul_overflow(batch, d_inner, &n) || __builtin_mul_overflow(n, L, &n) || n > (int64_t{1} << 48) ||
        batch * d_inner > (int64_t{1} << 48))
        return MSS_ERR_SHAPE;
    *fwd = mss::gated_fwd_scratch(batch, d_inner, L);
    *bwd = mss::gated_bwd_scratch(batch, d_inner, L);
    return MSS_OK;
}

int mss_gated_scan_fwd(const mss_tensor_t* x, const mss_tensor_t* fgate, const mss_tensor_t* igate,
                       const mss_tensor_t* rate, const mss_tensor_t* initial_state, const mss_tensor_t* seq_lens,
                       const mss_tensor_t* out, const mss_tensor_t* last_state, const mss_tensor_t* saved_states,
                       const mss_tensor_t* scratch, void* stream) {
    try {
        const mss_tensor_t* const req[] = {x, fgate, igate, rate};
        int st = check_descs(req, {initial_state, seq_lens, out, last_state, saved_states});
        if (st != MSS_OK) return st;
        if (!out && !last_state && !saved_states) return MSS_ERR_NULL_ARG;  // nothing to write
        if (x->ndim != 3) return MSS_ERR_SHAPE;
        const int64_t Bt = x->shape[0], Dn = x->shape[1], L = x->shape[2];
        for (const mss_tensor_t* t : {fgate, igate, out})
            if (t && !shape_is(*t, 3, Bt, Dn, L)) return MSS_ERR_SHAPE;
        if (!shape_is(*rate, 1, Dn)) return MSS_ERR_SHAPE;
        for (const mss_tensor_t* t : {initial_state, last_state})
            if (t && !shape_is(*t, 2, Bt, Dn)) return MSS_ERR_SHAPE;
        if (seq_lens && !shape_is(*seq_lens, 1, Bt)) return MSS_ERR_SHAPE;
        if (saved_states && !shape_is(*saved_states, 3, Bt, Dn, (L + mss::kGatedTile - 1) / mss::kGatedTile))
            return MSS_ERR_SHAPE;
        if (!act_dtype(x->dtype) || !all_dtype({fgate, igate, out}, x->dtype) ||
            !all_dtype({rate, initial_state, last_state, saved_states}, MSS_F32) || !all_dtype({seq_lens}, MSS_I32))
            return MSS_ERR_DTYPE;
        if (!laid_out({x, fgate, igate, rate, initial_state, seq_lens, out, last_state, saved_states}))
            return MSS_ERR_LAYOUT;
        if ((st = check_scratch(scratch, mss::gated_fwd_scratch(Bt, Dn, L))) != MSS_OK) return st;
        if (!apart({x, fgate, igate, rate, initial_state, seq_lens}, {out, last_state, saved_states, scratch}))
            return MSS_ERR_ALIAS;
        mss::GatedLaunch a;
        a.x = x->data; a.f = fgate->data; a.i = igate->data; a.rate = ptr<const float>(rate);
        a.h0 = ptr<const float>(initial_state); a.lens = ptr<const int32_t>(seq_lens); a.out = ptr<void>(out);
        a.last_state = ptr<float>(last_state); a.saved = ptr<float>(saved_states); a.scratch = ptr<float>(scratch);
        a.Bt = Bt; a.Dn = Dn; a.L = L;
        a.bf16 = x->dtype == MSS_BF16;
        a.vec_ok = whole_vectors(L, x->dtype, {x, fgate, igate, out});
        if (Bt * Dn == 0) return MSS_OK;
        return status(mss::launch_gated_fwd(a, static_cast<hipStream_t>(stream)));
    } catch (...) {
        return MSS_ERR_HIP;
    }
}

int mss_gated_scan_bwd(const mss_tensor_t* x, const mss_tensor_t* fgate, const mss_tensor_t* igate,
                       const mss_tensor_t* rate, const mss_tensor_t* seq_lens, const mss_tensor_t* saved_states,
                       const mss_tensor_t* dout, const mss_tensor_t* dlast_state, const mss_tensor_t* dx,
                       const mss_tensor_t* dfgate, const mss_tensor_t* digate, const mss_tensor_t* drate,
                       const mss_tensor_t* dinitial_state, const mss_tensor_t* scratch, void* stream) {
    try {
        const mss_tensor_t* const req[] = {x, fgate, igate, rate, saved_states, dout, dx, dfgate, digate, drate};
        int st = check_descs(req, {seq_lens, dlast_state, dinitial_state});
        if (st != MSS_OK) return st;
        if (x->ndim != 3) return MSS_ERR_SHAPE;
        const int64_t Bt = x->shape[0], Dn = x->shape[1], L = x->shape[2];
        for (const mss_tensor_t* t : {fgate, igate, dout, dx, dfgate, digate})
            if (!shape_is(*t, 3, Bt, Dn, L)) return MSS_ERR_SHAPE;
        if (!shape_is(*rate, 1, Dn) || !shape_is(*drate, 1, Dn)) return MSS_ERR_SHAPE;
        for (const mss_tensor_t* t : {dlast_state, dinitial_state})
            if (t && !shape_is(*t, 2, Bt, Dn)) return MSS_ERR_SHAPE;
        if (seq_lens && !shape_is(*seq_lens, 1, Bt)) return MSS_ERR_SHAPE;
        if (!shape_is(*saved_states, 3, Bt, Dn, (L + mss::kGatedTile - 1) / mss::kGatedTile)) return MSS_ERR_SHAPE;
        if (!act_dtype(x->dtype) || !all_dtype({fgate, igate, dout, dx, dfgate, digate}, x->dtype) ||
            !all_dtype({rate, drate, saved_states, dlast_state, dinitial_state}, MSS_F32) ||
            !all_dtype({seq_lens}, MSS_I32))
            return MSS_ERR_DTYPE;
        if (!laid_out({x, fgate, igate, rate, seq_lens, saved_states, dout, dlast_state, dx, dfgate, digate, drate,
                       dinitial_state}))
            return MSS_ERR_LAYOUT;
        if ((st = check_scratch(scratch, mss::gated_bwd_scratch(Bt, Dn, L))) != MSS_OK) return st;
        if (!apart({x, fgate, igate, rate, seq_lens, saved_states, dout, dlast_state},
                   {dx, dfgate, digate, drate, dinitial_state, scratch}))
            return MSS_ERR_ALIAS;
        mss::GatedLaunch a;
        a.x = x->data; a.f = fgate->data; a.i = igate->data; a.rate = ptr<const float>(rate);
        a.lens = ptr<const int32_t>(seq_lens); a.saved = ptr<float>(saved_states); a.dout = dout->data;
        a.dlast = ptr<const float>(dlast_state); a.dx = dx->data; a.df = dfgate->data; a.di = digate->data;
        a.drate = ptr<float>(drate); a.dh0 = ptr<float>(dinitial_state); a.scratch = ptr<float>(scratch);
        a.Bt = Bt; a.Dn = Dn; a.L = L;
        a.bf16 = x->dtype == MSS_BF16;
        a.vec_ok = whole_vectors(L, x->dtype, {x, fgate, igate, dout, dx, dfgate, digate});
        if (Dn == 0) return MSS_OK;  // with an empty batch drate is still written (zeros)
        return status(mss::launch_gated_bwd(a, static_cast<hipStream_t>(stream)));
    } catch (...) {
        return MSS_ERR_HIP;
    }
}

int mss_gated_state_update(const mss_tensor_t* state, const mss_tensor_t* x, const mss_tensor_t* fgate,
                           const mss_tensor_t* igate, const mss_tensor_t* rate, const mss_tensor_t* out,
                           void* stream) {
    try {
        const mss_tensor_t* const req[] = {state, x, fgate, igate, rate, out};
        const int st = check_descs(req, {});
        if (st != MSS_OK) return st;
        if (state->ndim != 2) return MSS_ERR_SHAPE;
        const int64_t Bt = state->shape[0], Dn = state->shape[1];
        for (const mss_tensor_t* t : {x, fgate, igate, out})
            if (!shape_is(*t, 2, Bt, Dn)) return MSS_ERR_SHAPE;
        if (!shape_is(*rate, 1, Dn)) return MSS_ERR_SHAPE;
        if (!act_dtype(x->dtype) || !all_dtype({fgate, igate, out}, x->dtype) || !all_dtype({state, rate}, MSS_F32))
            return MSS_ERR_DTYPE;
        if (!laid_out({state, x, fgate, igate, rate, out})) return MSS_ERR_LAYOUT;
        if (!apart({x, fgate, igate, rate}, {state, out})) return MSS_ERR_ALIAS;
        mss::GatedUpdateLaunch a;
        a.state = static_cast<float*>(state->data);
        a.x = x->data; a.f = fgate->data; a.i = igate->data; a.rate = static_cast<const float*>(rate->data);
        a.out = out->data;
        a.Dn = Dn; a.R = Bt * Dn;
        a.bf16 = x->dtype == MSS_BF16;
        if (a.R == 0) return MSS_OK;
        return status(mss::launch_gated_update(a, static_cast<hipStream_t>(stream)));
    } catch (...) {
        return MSS_ERR_HIP;
    }
}

int mss_causal_conv1d_bwd_scratch(int64_t batch, int64_t d_inner, int64_t L, int64_t K, int64_t* floats) {
    if (!floats) return MSS_ERR_NULL_ARG;
    int64_t n = 0;
    if (batch < 0 || d_inner < 0 || L < 0 || K < 1) return MSS_ERR_SHAPE;
    if (__builtin_mul_overflow(batch, d_inner, &n) || n > (int64_t{1} << 44) || L > (int64_t{1} << 48))
        return MSS_ERR_SHAPE;
    if (K > 4) return MSS_ERR_UNSUPPORTED;
    *floats = mss::conv1d_bwd_scratch(batch, d_inner, L, K);
    return MSS_OK;
}

int mss_causal_conv1d_bwd(const mss_tensor_t* x, const mss_tensor_t* weight, const mss_tensor_t* bias,
                          const mss_tensor_t* initial_state, int silu_flag, const mss_tensor_t* dout,
                          const mss_tensor_t* dfinal_state, const mss_tensor_t* dx, const mss_tensor_t* dweight,
                          const mss_tensor_t* dbias, const mss_tensor_t* dinitial_state,
                          const mss_tensor_t* scratch, void* stream) {
    try {
        const mss_tensor_t* const req[] = {x, weight, dout, dx, dweight};
        int st = check_descs(req, {bias, initial_state, dfinal_state, dbias, dinitial_state});
        if (st != MSS_OK) return st;
        if (x->ndim != 3 || weight->ndim != 2) return MSS_ERR_SHAPE;
        const int64_t Bt = x->shape[0], Dn = x->shape[1], L = x->shape[2], K = weight->shape[1];
        if (K < 1) return MSS_ERR_SHAPE;
        if (!shape_is(*dout, 3, Bt, Dn, L) || !shape_is(*dx, 3, Bt, Dn, L)) return MSS_ERR_SHAPE;
        if (!shape_is(*weight, 2, Dn, K) || !shape_is(*dweight, 2, Dn, K)) return MSS_ERR_SHAPE;
        for (const mss_tensor_t* t : {bias, dbias})
            if (t && !shape_is(*t, 1, Dn)) return MSS_ERR_SHAPE;
        for (const mss_tensor_t* t : {initial_state, dfinal_state, dinitial_state})
            if (t && !shape_is(*t, 3, Bt, Dn, K - 1)) return MSS_ERR_SHAPE;
        if (!act_dtype(x->dtype) || !all_dtype({dout, dx, initial_state, dfinal_state, dinitial_state}, x->dtype) ||
            !all_dtype({weight, bias, dweight, dbias}, MSS_F32))
            return MSS_ERR_DTYPE;
        if (!laid_out({x, weight, bias, initial_state, dout, dfinal_state, dx, dweight, dbias, dinitial_state}))
            return MSS_ERR_LAYOUT;
        if (K > 4) return MSS_ERR_UNSUPPORTED;
        if ((st = check_scratch(scratch, mss::conv1d_bwd_scratch(Bt, Dn, L, K))) != MSS_OK) return st;
        if (!apart({x, weight, bias, initial_state, dout, dfinal_state}, {dx, dweight, dbias, dinitial_state, scratch}))
            return MSS_ERR_ALIAS;
        mss::ConvBwdLaunch a;
        a.x = x->data; a.w = static_cast<const float*>(weight->data); a.bias = ptr<const float>(bias);
        a.state_in = ptr<const void>(initial_state); a.dout = dout->data; a.dfinal = ptr<const void>(dfinal_state);
        a.dx = dx->data; a.dw = static_cast<float*>(dweight->data); a.db = ptr<float>(dbias);
        a.dstate = ptr<void>(dinitial_state); a.scratch = ptr<float>(scratch);
        a.Dn = Dn; a.L = L; a.R = Bt * Dn;
        a.K = static_cast<int>(K);
        a.silu = silu_flag != 0;
        a.bf16 = x->dtype == MSS_BF16;
        a.vec_ok = whole_vectors(L, x->dtype, {x, dout, dx});
        if (Dn == 0) return MSS_OK;  // with an empty batch the sums are still written (zeros)
        return status(mss::launch_conv1d_bwd(a, static_cast<hipStream_t>(stream)));
    } catch (...) {
        return MSS_ERR_HIP;
    }
}

int mss_beam_select_scratch(int64_t batch, int64_t beams, int64_t vocab, int64_t k, int64_t* floats) {
    if (!floats) return MSS_ERR_NULL_ARG;
    if (batch < 0 || beams < 1 || vocab < 1 || k < 1) return MSS_ERR_SHAPE;
    if (beams > mss::kBeamMost || k > mss::kBeamMost || vocab > INT32_MAX || batch > (int64_t{1} << 24))
        return MSS_ERR_UNSUPPORTED;
    *floats = mss::beam_select_scratch(batch, beams, vocab, k);
    return MSS_OK;
}

int mss_beam_select(const mss_tensor_t* logits, const mss_tensor_t* scores, const mss_tensor_t* finished,
                    int end_token, const mss_tensor_t* next_scores, const mss_tensor_t* parents,
                    const mss_tensor_t* tokens, const mss_tensor_t* next_finished, const mss_tensor_t* scratch,
                    void* stream) {
    try {
        const mss_tensor_t* const req[] = {logits, scores, next_scores, parents, tokens};
        int st = check_descs(req, {finished, next_finished});
        if (st != MSS_OK) return st;
        if (logits->ndim != 3 || next_scores->ndim != 2) return MSS_ERR_SHAPE;
        const int64_t Bt = logits->shape[0], N = logits->shape[1], V = logits->shape[2], K = next_scores->shape[1];
        if (N < 1 || V < 1 || K < 1) return MSS_ERR_SHAPE;
        if (!shape_is(*scores, 2, Bt, N) || (finished && !shape_is(*finished, 2, Bt, N))) return MSS_ERR_SHAPE;
        for (const mss_tensor_t* t : {next_scores, parents, tokens, next_finished})
            if (t && !shape_is(*t, 2, Bt, K)) return MSS_ERR_SHAPE;
        // a finished beam needs the end token it goes on with
        if (end_token < -1 || end_token >= V || (finished && end_token < 0)) return MSS_ERR_SHAPE;
        if (!act_dtype(logits->dtype) || !all_dtype({scores, next_scores}, MSS_F32) ||
            !all_dtype({finished, parents, tokens, next_finished}, MSS_I32))
            return MSS_ERR_DTYPE;
        if (!laid_out({logits, scores, finished, next_scores, parents, tokens, next_finished})) return MSS_ERR_LAYOUT;
        if (N > mss::kBeamMost || K > mss::kBeamMost || V > INT32_MAX || Bt > (int64_t{1} << 24))
            return MSS_ERR_UNSUPPORTED;
        if ((st = check_scratch(scratch, mss::beam_select_scratch(Bt, N, V, K))) != MSS_OK) return st;
        // scores and finished may be their own successors; any other overlap is refused
        const auto same = [](const mss_tensor_t* a, const mss_tensor_t* b) {
            return a && b && a->data == b->data && a->shape[1] == b->shape[1];
        };
        if (!apart({logits, same(next_scores, scores) ? nullptr : scores}, {next_scores}) ||
            !apart({logits, same(next_finished, finished) ? nullptr : finished}, {next_finished}) ||
            !apart({logits, scores, finished}, {parents, tokens, scratch}) ||
            overlap(next_scores, finished) || overlap(next_finished, scores) ||
            !apart({}, {next_scores, next_finished, parents, tokens, scratch}))
            return MSS_ERR_ALIAS;
        mss::BeamSelectLaunch a;
        a.logits = logits->data; a.scores = static_cast<const float*>(scores->data);
        a.finished = ptr<const int32_t>(finished); a.next_scores = static_cast<float*>(next_scores->data);
        a.parents = static_cast<int32_t*>(parents->data); a.tokens = static_cast<int32_t*>(tokens->data);
        a.next_finished = ptr<int32_t>(next_finished); a.scratch = ptr<float>(scratch);
        a.Bt = Bt; a.N = N; a.V = V; a.K = K; a.end = end_token;
        a.bf16 = logits->dtype == MSS_BF16;
        a.vec_ok = whole_vectors(V, logits->dtype, {logits});
        if (Bt == 0) return MSS_OK;
        return status(mss::launch_beam_select(a, static_cast<hipStream_t>(stream)));
    } catch (...) {
        return MSS_ERR_HIP;
    }
}

int mss_beam_reorder(const mss_tensor_t* const* states, int count, const mss_tensor_t* parents, void* stream) {
    try {
        if (count < 0) return MSS_ERR_SHAPE;
        if (!parents || (count > 0 && !states)) return MSS_ERR_NULL_ARG;
        int st = check_desc(parents, true);
        if (st != MSS_OK) return st;
        for (int t = 0; t < count; ++t)
            if ((st = check_desc(states[t], true)) != MSS_OK) return st;
        if (parents->ndim != 2) return MSS_ERR_SHAPE;
        const int64_t Bt = parents->shape[0], N = parents->shape[1];
        for (int t = 0; t < count; ++t)
            if (states[t]->shape[0] != Bt * N) return MSS_ERR_SHAPE;
        if (parents->dtype != MSS_I32) return MSS_ERR_DTYPE;
        for (int t = 0; t < count; ++t)
            if (!act_dtype(states[t]->dtype) && states[t]->dtype != MSS_I32) return MSS_ERR_DTYPE;
        if (!laid_out({parents})) return MSS_ERR_LAYOUT;
        for (int t = 0; t < count; ++t)
            if (!laid_out({states[t]})) return MSS_ERR_LAYOUT;
        std::vector<Range> used;
        used.reserve(static_cast<size_t>(count) + 1);
        for (int t = -1; t < count; ++t) {
            const Range r = range_of(t < 0 ? parents : states[t]);
            if (r.lo != r.hi) used.push_back(r);
        }
        std::sort(used.begin(), used.end(), [](const Range& a, const Range& b) { return a.lo < b.lo; });
        for (size_t t = 1; t < used.size(); ++t)
            if (used[t].lo < used[t - 1].hi) return MSS_ERR_ALIAS;
        if (N > mss::kBeamMost) return MSS_ERR_UNSUPPORTED;
        if (Bt * N == 0 || count == 0) return MSS_OK;
        std::vector<mss::BeamReorderLaunch> l(static_cast<size_t>(count));
        for (int t = 0; t < count; ++t)
            l[t] = {states[t]->data, numel(*states[t]) / (Bt * N) * static_cast<int64_t>(elem_size(states[t]->dtype))};
        return status(mss::launch_beam_reorder(l.data(), count, static_cast<const int32_t*>(parents->data), Bt,
                                               static_cast<int>(N), static_cast<hipStream_t>(stream)));
    } catch (...) {
        return MSS_ERR_HIP;
    }
}

}  // extern "C"
