// Host side of the training operators' entry points: argument checks, workspace
// checks and the launches.  Everything is checked before anything is enqueued.
#include <algorithm>
#include <cmath>
#include <initializer_list>

#include "api_common.h"
#include "muon.h"
#include "train_internal.h"

using namespace muon;

namespace {

size_t elem_size(int32_t dtype) { return dtype == MUON_BF16 ? 2 : 4; }

// The buffers of one call.  Their number is small, so the overlap check is pairwise.
struct Buffers {
    struct Buf {
        uintptr_t lo, hi;
        size_t pitch, width;   // of a matrix's rows, in bytes; a vector is one row
        bool out;
        const char* name;
        size_t pitch2, width2;   // the same bytes, or more, as other rows (a head each); 0: none
        // No byte in common.  Matrices of one pitch may lie in each other's gaps (column ranges of one buffer).
        bool apart(const Buf& o) const {
            if (lo >= o.hi || o.lo >= hi) return true;
            return in_gaps(o, pitch, width, o.pitch, o.width) || (pitch2 && in_gaps(o, pitch2, width2, o.pitch2, o.width2));
        }
        bool in_gaps(const Buf& o, size_t p, size_t w, size_t op, size_t ow) const {
            if (p != op || w > p || ow > p) return false;
            const size_t after = (o.lo >= lo ? o.lo - lo : p - (lo - o.lo) % p) % p;
            return after >= w && after + ow <= p;
        }
    };
    Buf b[24];
    int n = 0;
    const char* bad = nullptr;   // first problem found by add()
    const char* why = nullptr;

    // `optional`: NULL is fine.  Buffers of no elements need no pointer.
    void add(const char* name, const void* p, size_t bytes, size_t align, bool out, bool optional = false) {
        rows(name, p, bytes, bytes, bytes, align, out, optional);
    }
    void rows(const char* name, const void* p, size_t bytes, size_t pitch, size_t width, size_t align, bool out, bool optional) {
        if (bad || bytes == 0) return;
        if (!p) {
            if (!optional) { bad = name; why = "is NULL"; }
            return;
        }
        const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
        if (lo % align) { bad = name; why = "is misaligned"; return; }
        b[n++] = {lo, lo + bytes, pitch, width, out, name, 0, 0};
    }
    // rows x heads x width with pitches ld and hs: an input's may be anything (0: broadcast), an output's elements are apart.
    void heads(const char* name, const void* p, int64_t rows, int64_t heads, int64_t width, int64_t ld, int64_t hs, size_t es, bool out,
               bool optional = false) {
        if (bad || rows == 0 || (optional && !p)) return;
        constexpr int64_t MOST = int64_t{1} << 40;
        if (rows == 1) ld = 0;
        if (heads == 1) hs = 0;
        if (ld < 0 || hs < 0 || ld > MOST || hs > MOST) { bad = name; why = "has a negative pitch or one beyond 2^40"; return; }
        const __int128 span = static_cast<__int128>(rows - 1) * ld + static_cast<__int128>(heads - 1) * hs + width;
        if (span > MOST * 65536) { bad = name; why = "spans more than 2^56 elements"; return; }
        const bool by_row = (heads == 1 || hs >= width) && (rows == 1 || ld >= (heads - 1) * hs + width);
        const bool by_head = (rows == 1 || ld >= width) && (heads == 1 || static_cast<__int128>(hs) >= static_cast<__int128>(rows - 1) * ld + width);
        if (out && !by_row && !by_head) { bad = name; why = "has overlapping rows or heads"; return; }
        const size_t bytes = static_cast<size_t>(span) * es;
        const int before = n;
        if (by_row && rows > 1) this->rows(name, p, bytes, ld * es, ((heads - 1) * hs + width) * es, es, out, false);
        else if (by_head && heads > 1) this->rows(name, p, bytes, hs * es, ((rows - 1) * ld + width) * es, es, out, false);
        else this->rows(name, p, bytes, bytes, bytes, es, out, false);
        if (n > before && heads > 1 && rows > 1 && hs >= width && ld % hs == 0) {
            b[n - 1].pitch2 = hs * es;
            b[n - 1].width2 = width * es;
        }
    }
    void matrix(const char* name, const void* p, int64_t rows, int64_t cols, int64_t ld, size_t es, bool out,
                bool optional = false) {
        if (bad || rows == 0 || (optional && !p)) return;
        if (ld < cols || ld > (int64_t{1} << 40)) { bad = name; why = "has a row pitch below its columns or beyond 2^40"; return; }
        this->rows(name, p, (static_cast<size_t>(rows - 1) * ld + cols) * es, ld * es, cols * es, es, out, false);
    }
    // The same buffer as input and output, with the same pitch, is an in-place call.
    muon_status check(const void* in_place_in = nullptr, const void* in_place_out = nullptr) const {
        if (bad) return fail(MUON_ERR_INVALID_ARG, "%s %s", bad, why);
        for (int i = 0; i < n; ++i)
            for (int j = i + 1; j < n; ++j) {
                if (!(b[i].out || b[j].out) || b[i].apart(b[j])) continue;
                const uintptr_t pi = reinterpret_cast<uintptr_t>(in_place_in), po = reinterpret_cast<uintptr_t>(in_place_out);
                if (pi && pi == po && b[i].lo == pi && b[j].lo == pi && b[i].hi == b[j].hi && b[i].out != b[j].out) continue;
                return fail(MUON_ERR_INVALID_ARG, "%s and %s overlap", b[i].name, b[j].name);
            }
        return MUON_OK;
    }
    muon_status check_against(const char* name, const void* p, size_t bytes) const {
        const uintptr_t lo = reinterpret_cast<uintptr_t>(p), hi = lo + bytes;
        for (int i = 0; i < n && bytes; ++i)
            if (b[i].lo < hi && lo < b[i].hi) return fail(MUON_ERR_INVALID_ARG, "%s and %s overlap", b[i].name, name);
        return MUON_OK;
    }
};

muon_status check_workspace(const void* ws, size_t have, size_t need) {
    if (need == 0) return MUON_OK;
    if (!ws) return fail(MUON_ERR_WORKSPACE, "workspace is NULL");
    if (reinterpret_cast<uintptr_t>(ws) % ALIGN) return fail(MUON_ERR_WORKSPACE, "workspace is not %zu-byte aligned", ALIGN);
    if (have < need) return fail(MUON_ERR_WORKSPACE, "workspace has %zu bytes, %zu needed", have, need);
    return MUON_OK;
}

muon_status check_dtype(int32_t dtype, const char* what) {
    if (dtype != MUON_F32 && dtype != MUON_BF16) return fail(MUON_ERR_INVALID_ARG, "unknown %s %d", what, dtype);
    return MUON_OK;
}

muon_status check_finite(std::initializer_list<float> vs, const char* what) {
    for (float v : vs)
        if (!std::isfinite(v)) return fail(MUON_ERR_INVALID_ARG, "%s must be finite", what);
    return MUON_OK;
}

#define MUON_TRY(expr)                          \
    do {                                        \
        const muon_status st_ = (expr);         \
        if (st_ != MUON_OK) return st_;         \
    } while (0)

// ---- block norm ---------------------------------------------------------------

muon_status check_norm_shape(int64_t rows, int64_t cols, int32_t dtype, int32_t weight_dtype, int32_t gate_kind) {
    MUON_TRY(check_dtype(dtype, "dtype"));
    MUON_TRY(check_dtype(weight_dtype, "weight_dtype"));
    if (gate_kind < MUON_GATE_NONE || gate_kind > MUON_GATE_FULL)
        return fail(MUON_ERR_INVALID_ARG, "unknown gate_kind %d", gate_kind);
    if (rows < 0 || cols < 1) return fail(MUON_ERR_INVALID_ARG, "shape %lld x %lld", (long long)rows, (long long)cols);
    if (rows > MUON_MAX_TOKENS || cols > MUON_MAX_NORM_COLS)
        return fail(MUON_ERR_UNSUPPORTED, "shape %lld x %lld is beyond %lld x %d", (long long)rows, (long long)cols,
                    (long long)MUON_MAX_TOKENS, MUON_MAX_NORM_COLS);
    return MUON_OK;
}

muon_status check_norm(const muon_block_norm_args* a, Buffers& buf) {
    if (!a) return fail(MUON_ERR_INVALID_ARG, "args is NULL");
    MUON_TRY(check_norm_shape(a->rows, a->cols, a->dtype, a->weight_dtype, a->gate_kind));
    MUON_TRY(check_finite({a->residual_scale, a->eps}, "residual_scale and eps"));
    if (a->eps < 0.0f) return fail(MUON_ERR_INVALID_ARG, "eps must be >= 0");
    // a matrix of no rows needs no pointer
    if (a->rows > 0 && (a->gate != nullptr) != (a->gate_kind != MUON_GATE_NONE))
        return fail(MUON_ERR_INVALID_ARG, "gate and gate_kind disagree");
    if (a->rows > 0 && (a->pre_weight != nullptr) != (a->out_norm != nullptr))
        return fail(MUON_ERR_INVALID_ARG, "pre_weight and out_norm go together");
    const size_t es = elem_size(a->dtype), ws = elem_size(a->weight_dtype), d = static_cast<size_t>(a->cols);
    buf.matrix("x", a->x, a->rows, a->cols, a->ld_x, es, false);
    buf.matrix("residual", a->residual, a->rows, a->cols, a->ld_residual, es, false);
    buf.add("post_weight", a->post_weight, d * ws, ws, false, true);
    buf.add("pre_weight", a->pre_weight, d * ws, ws, false, true);
    if (a->gate_kind == MUON_GATE_CHANNEL) buf.add("gate", a->gate, d * ws, ws, false);
    if (a->gate_kind == MUON_GATE_FULL) buf.matrix("gate", a->gate, a->rows, a->cols, a->ld_gate, es, false);
    buf.matrix("out_residual", a->out_residual, a->rows, a->cols, a->ld_out_residual, es, true);
    buf.matrix("out_norm", a->out_norm, a->rows, a->cols, a->ld_out_norm, es, true, true);
    buf.add("rstd", a->rstd, 2 * static_cast<size_t>(a->rows) * sizeof(float), sizeof(float), true, true);
    const bool in_place = a->ld_residual == a->ld_out_residual;
    return buf.check(in_place ? a->residual : nullptr, a->out_residual);
}

muon_status check_norm_backward(const muon_block_norm_backward_args* a, Buffers& buf) {
    if (!a) return fail(MUON_ERR_INVALID_ARG, "args is NULL");
    MUON_TRY(check_norm_shape(a->rows, a->cols, a->dtype, a->weight_dtype, a->gate_kind));
    MUON_TRY(check_finite({a->residual_scale}, "residual_scale"));
    if (a->rows > 0) {
        if ((a->gate != nullptr) != (a->gate_kind != MUON_GATE_NONE))
            return fail(MUON_ERR_INVALID_ARG, "gate and gate_kind disagree");
        if (!a->grad_norm && !a->grad_out_residual)
            return fail(MUON_ERR_INVALID_ARG, "grad_norm and grad_out_residual are both NULL");
        if (a->grad_norm && !a->pre_weight) return fail(MUON_ERR_INVALID_ARG, "grad_norm needs pre_weight");
    }
    if ((a->post_weight != nullptr) != (a->grad_post_weight != nullptr) || (a->gate != nullptr) != (a->grad_gate != nullptr) ||
        (a->pre_weight != nullptr) != (a->grad_pre_weight != nullptr))
        return fail(MUON_ERR_INVALID_ARG, "a weight and its gradient go together");
    const size_t es = elem_size(a->dtype), ws = elem_size(a->weight_dtype), d = static_cast<size_t>(a->cols);
    buf.matrix("x", a->x, a->rows, a->cols, a->ld_x, es, false);
    buf.matrix("out_residual", a->out_residual, a->rows, a->cols, a->ld_out_residual, es, false);
    buf.add("rstd", a->rstd, 2 * static_cast<size_t>(a->rows) * sizeof(float), sizeof(float), false);
    buf.matrix("grad_norm", a->grad_norm, a->rows, a->cols, a->ld_grad_norm, es, false, true);
    buf.matrix("grad_out_residual", a->grad_out_residual, a->rows, a->cols, a->ld_grad_out_residual, es, false, true);
    buf.add("post_weight", a->post_weight, d * ws, ws, false, true);
    buf.add("pre_weight", a->pre_weight, d * ws, ws, false, true);
    buf.add("grad_post_weight", a->grad_post_weight, d * ws, ws, true, true);
    buf.add("grad_pre_weight", a->grad_pre_weight, d * ws, ws, true, true);
    if (a->gate_kind == MUON_GATE_CHANNEL) {
        buf.add("gate", a->gate, d * ws, ws, false);
        buf.add("grad_gate", a->grad_gate, d * ws, ws, true);
    }
    if (a->gate_kind == MUON_GATE_FULL) {
        buf.matrix("gate", a->gate, a->rows, a->cols, a->ld_gate, es, false);
        buf.matrix("grad_gate", a->grad_gate, a->rows, a->cols, a->ld_grad_gate, es, true);
    }
    buf.matrix("grad_x", a->grad_x, a->rows, a->cols, a->ld_grad_x, es, true);
    buf.matrix("grad_residual", a->grad_residual, a->rows, a->cols, a->ld_grad_residual, es, true);
    const bool in_place = a->ld_grad_out_residual == a->ld_grad_residual;
    return buf.check(in_place ? a->grad_out_residual : nullptr, a->grad_residual);
}

// ---- token log-probabilities ----------------------------------------------------

muon_status check_logp_shape(int64_t tokens, int64_t cols, int64_t vocab, int32_t dtype, float scale) {
    MUON_TRY(check_dtype(dtype, "dtype"));
    MUON_TRY(check_finite({scale}, "scale"));
    if (tokens < 0 || cols < 1 || vocab < 1)
        return fail(MUON_ERR_INVALID_ARG, "%lld tokens, %lld columns, vocabulary of %lld", (long long)tokens, (long long)cols,
                    (long long)vocab);
    if (tokens > MUON_MAX_TOKENS || cols > MUON_MAX_DIM || vocab > MUON_MAX_VOCAB)
        return fail(MUON_ERR_UNSUPPORTED, "%lld tokens, %lld columns, vocabulary of %lld: beyond %lld, %d, %d",
                    (long long)tokens, (long long)cols, (long long)vocab, (long long)MUON_MAX_TOKENS, MUON_MAX_DIM,
                    MUON_MAX_VOCAB);
    return MUON_OK;
}

muon_status check_logp(const muon_token_logp_args* a, Buffers& buf) {
    if (!a) return fail(MUON_ERR_INVALID_ARG, "args is NULL");
    MUON_TRY(check_logp_shape(a->tokens, a->cols, a->vocab, a->dtype, a->scale));
    const size_t es = elem_size(a->dtype), t = static_cast<size_t>(a->tokens);
    buf.matrix("hidden", a->hidden, a->tokens, a->cols, a->ld_hidden, es, false);
    buf.matrix("head", a->head, a->vocab, a->cols, a->ld_head, es, false);
    buf.add("targets", a->targets, t * 8, 8, false);
    buf.add("logp", a->logp, t * 4, 4, true);
    buf.add("lse", a->lse, t * 4, 4, true);
    if (a->saved) buf.add("saved", a->saved, token_logp_saved_bytes(*a), ALIGN, true);
    return buf.check();
}

muon_token_logp_args forward_shape(const muon_token_logp_backward_args& a) {
    muon_token_logp_args f{};
    f.tokens = a.tokens;
    f.cols = a.cols;
    f.vocab = a.vocab;
    f.dtype = a.dtype;
    return f;
}

muon_status check_logp_backward(const muon_token_logp_backward_args* a, Buffers& buf) {
    if (!a) return fail(MUON_ERR_INVALID_ARG, "args is NULL");
    MUON_TRY(check_logp_shape(a->tokens, a->cols, a->vocab, a->dtype, a->scale));
    if (!a->grad_hidden && !a->grad_head && a->tokens > 0)
        return fail(MUON_ERR_INVALID_ARG, "grad_hidden and grad_head are both NULL");
    const size_t es = elem_size(a->dtype), t = static_cast<size_t>(a->tokens);
    buf.matrix("hidden", a->hidden, a->tokens, a->cols, a->ld_hidden, es, false);
    buf.matrix("head", a->head, a->vocab, a->cols, a->ld_head, es, false);
    buf.add("targets", a->targets, t * 8, 8, false);
    buf.add("lse", a->lse, t * 4, 4, false);
    buf.add("grad_logp", a->grad_logp, t * 4, 4, false);
    if (a->saved) buf.add("saved", a->saved, token_logp_saved_bytes(forward_shape(*a)), ALIGN, false);
    buf.matrix("grad_hidden", a->grad_hidden, a->tokens, a->cols, a->ld_grad_hidden, es, true, true);
    buf.matrix("grad_head", a->grad_head, a->vocab, a->cols, a->ld_grad_head, es, true, true);
    return buf.check();
}

// ---- losses -----------------------------------------------------------------------

muon_status check_sequences(int64_t tokens, int64_t sequences, int32_t dtype) {
    MUON_TRY(check_dtype(dtype, "dtype"));
    if (tokens < 0 || sequences < 0)
        return fail(MUON_ERR_INVALID_ARG, "%lld tokens in %lld sequences", (long long)tokens, (long long)sequences);
    if (tokens > MUON_MAX_TOKENS || sequences > MUON_MAX_TOKENS)
        return fail(MUON_ERR_UNSUPPORTED, "%lld tokens in %lld sequences: beyond %lld", (long long)tokens,
                    (long long)sequences, (long long)MUON_MAX_TOKENS);
    return MUON_OK;
}

muon_status check_preference(const muon_preference_args* a, Buffers& buf) {
    if (!a) return fail(MUON_ERR_INVALID_ARG, "args is NULL");
    MUON_TRY(check_sequences(a->tokens, a->sequences, a->dtype));
    if (a->sequences % 2) return fail(MUON_ERR_INVALID_ARG, "%lld sequences are not pairs", (long long)a->sequences);
    MUON_TRY(check_finite({a->beta, a->margin, a->label_smoothing, a->grad_scale}, "beta, margin, label_smoothing and grad_scale"));
    if (a->label_smoothing < 0.0f || a->label_smoothing > 1.0f)
        return fail(MUON_ERR_INVALID_ARG, "label_smoothing outside [0, 1]");
    if (a->kind < MUON_PREFERENCE_SIGMOID || a->kind > MUON_PREFERENCE_SQUARED)
        return fail(MUON_ERR_INVALID_ARG, "unknown preference kind %d", a->kind);
    if (a->kind == MUON_PREFERENCE_SQUARED && a->beta == 0.0f)
        return fail(MUON_ERR_INVALID_ARG, "the squared preference loss needs beta != 0");
    const size_t es = elem_size(a->dtype), n = static_cast<size_t>(a->tokens), q = static_cast<size_t>(a->sequences);
    buf.add("logp", a->logp, n * es, es, false);
    buf.add("ref_logp", a->ref_logp, n * es, es, false, true);
    buf.add("mask", a->mask, n, 1, false, true);
    buf.add("offsets", a->offsets, (q + 1) * 8, 8, false);
    buf.add("loss", a->loss, 4, 4, true);
    buf.add("rewards", a->rewards, q * 4, 4, true, true);
    buf.add("grad_logp", a->grad_logp, n * es, es, true, true);
    return buf.check();
}

muon_status check_policy(const muon_policy_args* a, Buffers& buf) {
    if (!a) return fail(MUON_ERR_INVALID_ARG, "args is NULL");
    MUON_TRY(check_sequences(a->tokens, a->sequences, a->dtype));
    MUON_TRY(check_finite({a->clip_low, a->clip_high, a->dual_clip, a->kl_coef, a->grad_scale},
                          "clip_low, clip_high, dual_clip, kl_coef and grad_scale"));
    if (a->clip_low < 0.0f || a->clip_high < 0.0f) return fail(MUON_ERR_INVALID_ARG, "clip_low and clip_high must be >= 0");
    if (a->dual_clip != 0.0f && a->dual_clip < 1.0f) return fail(MUON_ERR_INVALID_ARG, "dual_clip must be 0 or >= 1");
    if (a->kl < MUON_KL_NONE || a->kl > MUON_KL_K3) return fail(MUON_ERR_INVALID_ARG, "unknown kl %d", a->kl);
    if (a->reduction != MUON_REDUCE_TOKEN && a->reduction != MUON_REDUCE_SEQUENCE)
        return fail(MUON_ERR_INVALID_ARG, "unknown reduction %d", a->reduction);
    if (a->kl == MUON_KL_NONE ? a->ref_logp != nullptr : (!a->ref_logp && a->tokens > 0))
        return fail(MUON_ERR_INVALID_ARG, "ref_logp and kl go together");
    const size_t es = elem_size(a->dtype), n = static_cast<size_t>(a->tokens), q = static_cast<size_t>(a->sequences);
    buf.add("logp", a->logp, n * es, es, false);
    buf.add("old_logp", a->old_logp, n * es, es, false);
    buf.add("ref_logp", a->ref_logp, n * es, es, false, true);
    buf.add("advantages", a->advantages, (a->advantage_per_sequence ? q : n) * 4, 4, false);
    buf.add("mask", a->mask, n, 1, false, true);
    buf.add("offsets", a->offsets, (q + 1) * 8, 8, false);
    buf.add("loss", a->loss, 4, 4, true);
    buf.add("stats", a->stats, 16, 4, true, true);
    buf.add("grad_logp", a->grad_logp, n * es, es, true, true);
    return buf.check();
}

// ---- attention ------------------------------------------------------------------

// A and the backward pass's arguments share the fields that are looked at here.
template <typename A> muon_status check_attention_shape(const A* a) {
    MUON_TRY(check_dtype(a->dtype, "dtype"));
    MUON_TRY(check_finite({a->scale}, "scale"));
    if (a->queries < 0 || a->keys < 0 || a->sequences < 1 || a->width < 1 || a->heads < 1 || a->kv_heads < 1 || a->window < 0)
        return fail(MUON_ERR_INVALID_ARG, "%lld queries and %lld keys in %lld sequences, %d and %d heads of width %d, window %lld",
                    (long long)a->queries, (long long)a->keys, (long long)a->sequences, a->heads, a->kv_heads, a->width, (long long)a->window);
    if (a->heads % a->kv_heads) return fail(MUON_ERR_INVALID_ARG, "%d heads are not a multiple of %d", a->heads, a->kv_heads);
    if (!a->offsets && (a->sequences != 1 || a->key_offsets))
        return fail(MUON_ERR_INVALID_ARG, "without offsets there is one sequence, and no key_offsets");
    if (a->queries > MUON_MAX_TOKENS || a->keys > MUON_MAX_TOKENS || a->sequences > MUON_MAX_TOKENS || a->heads > MUON_MAX_HEADS ||
        a->width > MUON_MAX_HEAD_WIDTH)
        return fail(MUON_ERR_UNSUPPORTED, "%lld queries, %lld keys, %lld sequences, %d heads of width %d: beyond %lld, %d, %d", (long long)a->queries,
                    (long long)a->keys, (long long)a->sequences, a->heads, a->width, (long long)MUON_MAX_TOKENS, MUON_MAX_HEADS, MUON_MAX_HEAD_WIDTH);
    if ((a->bias != nullptr) != (a->bucket_map != nullptr)) return fail(MUON_ERR_INVALID_ARG, "bias and bucket_map go together");
    if (a->bias) {
        if (a->buckets < 1 || a->reach < 0) return fail(MUON_ERR_INVALID_ARG, "%d buckets, reach %d", a->buckets, a->reach);
        if (a->buckets > MUON_MAX_BUCKETS || a->reach > MUON_MAX_REACH)
            return fail(MUON_ERR_UNSUPPORTED, "%d buckets, reach %d: beyond %d, %d", a->buckets, a->reach, MUON_MAX_BUCKETS, MUON_MAX_REACH);
    }
    return MUON_OK;
}

template <typename A> void attention_inputs(const A* a, Buffers& buf) {
    const size_t es = elem_size(a->dtype);
    buf.heads("q", a->q, a->queries, a->heads, a->width, a->ld_q, a->hs_q, es, false);
    buf.heads("k", a->k, a->keys, a->kv_heads, a->width, a->ld_k, a->hs_k, es, false);
    buf.heads("v", a->v, a->keys, a->kv_heads, a->width, a->ld_v, a->hs_v, es, false);
    buf.add("offsets", a->offsets, (static_cast<size_t>(a->sequences) + 1) * 8, 8, false, true);
    buf.add("key_offsets", a->key_offsets, (static_cast<size_t>(a->sequences) + 1) * 8, 8, false, true);
    buf.add("key_mask", a->key_mask, static_cast<size_t>(a->keys), 1, false, true);
    if (a->bias) {
        buf.add("bias", a->bias, static_cast<size_t>(a->buckets) * a->heads * es, es, false);
        buf.add("bucket_map", a->bucket_map, (2 * static_cast<size_t>(a->reach) + 1) * 4, 4, false);
    }
}

muon_status check_attention(const muon_attention_args* a, Buffers& buf, const float* lse_low = nullptr) {
    if (!a) return fail(MUON_ERR_INVALID_ARG, "args is NULL");
    MUON_TRY(check_attention_shape(a));
    const size_t es = elem_size(a->dtype);
    attention_inputs(a, buf);
    buf.heads("out", a->out, a->queries, a->heads, a->width, a->ld_out, a->hs_out, es, true);
    buf.add("lse", a->lse, static_cast<size_t>(a->queries) * a->heads * 4, 4, true);
    buf.heads("out_low", a->out_low, a->queries, a->heads, a->width, a->ld_out_low, a->hs_out_low, es, true, true);
    buf.add("lse_low", lse_low, static_cast<size_t>(a->queries) * a->heads * 4, 4, true, true);
    return buf.check();
}

muon_status check_attention_backward(const muon_attention_backward_args* a, Buffers& buf, const float* lse_low = nullptr) {
    if (!a) return fail(MUON_ERR_INVALID_ARG, "args is NULL");
    MUON_TRY(check_attention_shape(a));
    if ((a->bias != nullptr) != (a->grad_bias != nullptr)) return fail(MUON_ERR_INVALID_ARG, "bias and its gradient go together");
    const size_t es = elem_size(a->dtype);
    attention_inputs(a, buf);
    buf.heads("out", a->out, a->queries, a->heads, a->width, a->ld_out, a->hs_out, es, false);
    buf.add("lse", a->lse, static_cast<size_t>(a->queries) * a->heads * 4, 4, false);
    buf.add("lse_low", lse_low, static_cast<size_t>(a->queries) * a->heads * 4, 4, false, true);
    buf.heads("out_low", a->out_low, a->queries, a->heads, a->width, a->ld_out_low, a->hs_out_low, es, false, true);
    buf.heads("grad_out", a->grad_out, a->queries, a->heads, a->width, a->ld_grad_out, a->hs_grad_out, es, false);
    buf.heads("grad_q", a->grad_q, a->queries, a->heads, a->width, a->ld_grad_q, a->hs_grad_q, es, true);
    buf.heads("grad_k", a->grad_k, a->keys, a->kv_heads, a->width, a->ld_grad_k, a->hs_grad_k, es, true);
    buf.heads("grad_v", a->grad_v, a->keys, a->kv_heads, a->width, a->ld_grad_v, a->hs_grad_v, es, true);
    if (a->bias) buf.add("grad_bias", a->grad_bias, static_cast<size_t>(a->buckets) * a->heads * es, es, true);
    return buf.check();
}

// ---- tokens to experts and back -----------------------------------------------------

muon_status check_expert_shape(int64_t tokens, int64_t cols, int32_t chosen, int32_t num_experts, int32_t dtype) {
    MUON_TRY(check_dtype(dtype, "dtype"));
    if (tokens < 0 || cols < 1 || chosen < 1 || num_experts < 1)
        return fail(MUON_ERR_INVALID_ARG, "%lld tokens of %lld columns to %d of %d experts", (long long)tokens, (long long)cols, chosen, num_experts);
    if (chosen > MUON_MAX_CHOSEN || num_experts > MUON_MAX_EXPERTS || cols > MUON_MAX_DIM || tokens > MUON_MAX_TOKENS / chosen)
        return fail(MUON_ERR_UNSUPPORTED, "%lld tokens of %lld columns to %d of %d experts: beyond %lld choices, %d, %d, %d", (long long)tokens,
                    (long long)cols, chosen, num_experts, (long long)MUON_MAX_TOKENS, MUON_MAX_DIM, MUON_MAX_CHOSEN, MUON_MAX_EXPERTS);
    return MUON_OK;
}

muon_status check_expert_sort(const muon_expert_sort_args* a, Buffers& buf) {
    if (!a) return fail(MUON_ERR_INVALID_ARG, "args is NULL");
    MUON_TRY(check_expert_shape(a->tokens, a->cols, a->chosen, a->num_experts, a->dtype));
    const size_t es = elem_size(a->dtype), n = static_cast<size_t>(a->tokens) * a->chosen;
    buf.matrix("x", a->x, a->tokens, a->cols, a->ld_x, es, false);
    buf.add("experts", a->experts, n * 8, 8, false);
    buf.matrix("sorted", a->sorted, n, a->cols, a->ld_sorted, es, true);
    buf.add("slots", a->slots, n * 4, 4, true);
    buf.add("offsets", a->offsets, (static_cast<size_t>(a->num_experts) + 1) * 8, 8, true);
    return buf.check();
}

muon_status check_expert_sort_backward(const muon_expert_sort_backward_args* a, Buffers& buf) {
    if (!a) return fail(MUON_ERR_INVALID_ARG, "args is NULL");
    MUON_TRY(check_expert_shape(a->tokens, a->cols, a->chosen, 1, a->dtype));
    const size_t es = elem_size(a->dtype), n = static_cast<size_t>(a->tokens) * a->chosen;
    buf.matrix("grad_sorted", a->grad_sorted, n, a->cols, a->ld_grad_sorted, es, false);
    buf.add("slots", a->slots, n * 4, 4, false);
    buf.matrix("grad_x", a->grad_x, a->tokens, a->cols, a->ld_grad_x, es, true);
    return buf.check();
}

muon_status check_expert_combine(const muon_expert_combine_args* a, Buffers& buf) {
    if (!a) return fail(MUON_ERR_INVALID_ARG, "args is NULL");
    MUON_TRY(check_expert_shape(a->tokens, a->cols, a->chosen, 1, a->dtype));
    const size_t es = elem_size(a->dtype), n = static_cast<size_t>(a->tokens) * a->chosen;
    buf.matrix("y", a->y, n, a->cols, a->ld_y, es, false);
    buf.add("slots", a->slots, n * 4, 4, false);
    buf.add("weights", a->weights, n * 4, 4, false);
    buf.matrix("out", a->out, a->tokens, a->cols, a->ld_out, es, true);
    return buf.check();
}

muon_status check_expert_combine_backward(const muon_expert_combine_backward_args* a, Buffers& buf) {
    if (!a) return fail(MUON_ERR_INVALID_ARG, "args is NULL");
    MUON_TRY(check_expert_shape(a->tokens, a->cols, a->chosen, a->num_experts, a->dtype));
    const size_t es = elem_size(a->dtype), n = static_cast<size_t>(a->tokens) * a->chosen;
    buf.matrix("grad_out", a->grad_out, a->tokens, a->cols, a->ld_grad_out, es, false);
    buf.matrix("y", a->y, n, a->cols, a->ld_y, es, false);
    buf.add("slots", a->slots, n * 4, 4, false);
    buf.add("weights", a->weights, n * 4, 4, false);
    buf.add("offsets", a->offsets, (static_cast<size_t>(a->num_experts) + 1) * 8, 8, false);
    buf.matrix("grad_y", a->grad_y, n, a->cols, a->ld_grad_y, es, true);
    buf.add("grad_weights", a->grad_weights, n * 4, 4, true);
    return buf.check();
}

// One launch sequence without a workspace.
template <typename F> muon_status run_plain(int cls, const char* what, void* stream, F launch) {
    int dev = 0, cus = 0;
    MUON_TRY(check_device(&dev, &cus));
    const hipStream_t s = static_cast<hipStream_t>(stream);
    MUON_TRY(timed_launch(cls, s, what, [&] { return launch(s); }));
    clear_error();
    return MUON_OK;
}

// Runs one operator: workspace and device checks, then the launches.
template <typename F>
muon_status run_op(Buffers& buf, size_t need, void* ws, size_t ws_bytes, F launch) {
    MUON_TRY(check_workspace(ws, ws_bytes, need));
    MUON_TRY(buf.check_against("the workspace", ws, need));
    int dev = 0, cus = 0;
    MUON_TRY(check_device(&dev, &cus));
    MUON_TRY(launch());
    clear_error();
    return MUON_OK;
}

size_t at_least_one(size_t bytes) { return std::max(align_up(bytes, ALIGN), ALIGN); }

}  // namespace

extern "C" {

muon_status muon_block_norm(const muon_block_norm_args* a, void* stream) {
    Buffers buf;
    MUON_TRY(check_norm(a, buf));
    int dev = 0, cus = 0;
    MUON_TRY(check_device(&dev, &cus));
    const hipStream_t s = static_cast<hipStream_t>(stream);
    MUON_TRY(timed_launch(9, s, "block norm kernel", [&] { return launch_block_norm(*a, s); }));
    clear_error();
    return MUON_OK;
}

size_t muon_block_norm_backward_workspace_bytes(const muon_block_norm_backward_args* a) {
    Buffers buf;
    return check_norm_backward(a, buf) == MUON_OK ? at_least_one(block_norm_backward_bytes(*a)) : 0;
}

muon_status muon_block_norm_backward(const muon_block_norm_backward_args* a, void* ws, size_t ws_bytes, void* stream) {
    Buffers buf;
    MUON_TRY(check_norm_backward(a, buf));
    const hipStream_t s = static_cast<hipStream_t>(stream);
    return run_op(buf, block_norm_backward_bytes(*a), ws, ws_bytes, [&] {
        return timed_launch(9, s, "block norm backward kernels", [&] { return launch_block_norm_backward(*a, ws, s); });
    });
}

size_t muon_token_logp_saved_bytes(const muon_token_logp_args* a) {
    if (!a) return fail(MUON_ERR_INVALID_ARG, "args is NULL"), 0;
    if (check_logp_shape(a->tokens, a->cols, a->vocab, a->dtype, a->scale) != MUON_OK) return 0;
    return at_least_one(token_logp_saved_bytes(*a));
}

size_t muon_token_logp_workspace_bytes(const muon_token_logp_args* a) {
    Buffers buf;
    return check_logp(a, buf) == MUON_OK ? at_least_one(token_logp_bytes(*a)) : 0;
}

muon_status muon_token_logp(const muon_token_logp_args* a, void* ws, size_t ws_bytes, void* stream) {
    Buffers buf;
    MUON_TRY(check_logp(a, buf));
    const hipStream_t s = static_cast<hipStream_t>(stream);
    return run_op(buf, token_logp_bytes(*a), ws, ws_bytes, [&] {
        return timed_launch(10, s, "token log-probability kernels", [&] { return launch_token_logp(*a, ws, s); });
    });
}

size_t muon_token_logp_backward_workspace_bytes(const muon_token_logp_backward_args* a) {
    Buffers buf;
    return check_logp_backward(a, buf) == MUON_OK ? at_least_one(token_logp_backward_bytes(*a)) : 0;
}

muon_status muon_token_logp_backward(const muon_token_logp_backward_args* a, void* ws, size_t ws_bytes, void* stream) {
    Buffers buf;
    MUON_TRY(check_logp_backward(a, buf));
    const hipStream_t s = static_cast<hipStream_t>(stream);
    return run_op(buf, token_logp_backward_bytes(*a), ws, ws_bytes, [&] {
        return timed_launch(10, s, "token log-probability backward kernels",
                            [&] { return launch_token_logp_backward(*a, ws, s); });
    });
}

size_t muon_preference_loss_workspace_bytes(const muon_preference_args* a) {
    Buffers buf;
    return check_preference(a, buf) == MUON_OK ? at_least_one(preference_bytes(*a)) : 0;
}

muon_status muon_preference_loss(const muon_preference_args* a, void* ws, size_t ws_bytes, void* stream) {
    Buffers buf;
    MUON_TRY(check_preference(a, buf));
    const hipStream_t s = static_cast<hipStream_t>(stream);
    return run_op(buf, preference_bytes(*a), ws, ws_bytes, [&] {
        return timed_launch(11, s, "preference loss kernels", [&] { return launch_preference(*a, ws, s); });
    });
}

size_t muon_policy_loss_workspace_bytes(const muon_policy_args* a) {
    Buffers buf;
    return check_policy(a, buf) == MUON_OK ? at_least_one(policy_bytes(*a)) : 0;
}

muon_status muon_policy_loss(const muon_policy_args* a, void* ws, size_t ws_bytes, void* stream) {
    Buffers buf;
    MUON_TRY(check_policy(a, buf));
    const hipStream_t s = static_cast<hipStream_t>(stream);
    return run_op(buf, policy_bytes(*a), ws, ws_bytes, [&] {
        return timed_launch(12, s, "policy loss kernels", [&] { return launch_policy(*a, ws, s); });
    });
}

size_t muon_attention_workspace_bytes(const muon_attention_args* a) {
    Buffers buf;
    return check_attention(a, buf) == MUON_OK ? at_least_one(attention_bytes(*a)) : 0;
}

muon_status muon_attention_two_part(const muon_attention_args* a, float* lse_low, void* ws, size_t ws_bytes, void* stream) {
    Buffers buf;
    MUON_TRY(check_attention(a, buf, lse_low));
    const hipStream_t s = static_cast<hipStream_t>(stream);
    return run_op(buf, attention_bytes(*a), ws, ws_bytes, [&] {
        return timed_launch(13, s, "attention kernels", [&] { return launch_attention(*a, lse_low, ws, s); });
    });
}

muon_status muon_attention(const muon_attention_args* a, void* ws, size_t ws_bytes, void* stream) {
    return muon_attention_two_part(a, nullptr, ws, ws_bytes, stream);
}

size_t muon_attention_backward_workspace_bytes(const muon_attention_backward_args* a) {
    Buffers buf;
    return check_attention_backward(a, buf) == MUON_OK ? at_least_one(attention_backward_bytes(*a)) : 0;
}

muon_status muon_attention_backward_two_part(const muon_attention_backward_args* a, const float* lse_low, void* ws, size_t ws_bytes,
                                             void* stream) {
    Buffers buf;
    MUON_TRY(check_attention_backward(a, buf, lse_low));
    const hipStream_t s = static_cast<hipStream_t>(stream);
    return run_op(buf, attention_backward_bytes(*a), ws, ws_bytes, [&] {
        return timed_launch(13, s, "attention backward kernels", [&] { return launch_attention_backward(*a, lse_low, ws, s); });
    });
}

muon_status muon_attention_backward(const muon_attention_backward_args* a, void* ws, size_t ws_bytes, void* stream) {
    return muon_attention_backward_two_part(a, nullptr, ws, ws_bytes, stream);
}

size_t muon_expert_sort_workspace_bytes(const muon_expert_sort_args* a) {
    Buffers buf;
    return check_expert_sort(a, buf) == MUON_OK ? at_least_one(expert_sort_bytes(*a)) : 0;
}

muon_status muon_expert_sort(const muon_expert_sort_args* a, void* ws, size_t ws_bytes, void* stream) {
    Buffers buf;
    MUON_TRY(check_expert_sort(a, buf));
    const hipStream_t s = static_cast<hipStream_t>(stream);
    return run_op(buf, expert_sort_bytes(*a), ws, ws_bytes, [&] {
        return timed_launch(14, s, "expert sort kernels", [&] { return launch_expert_sort(*a, ws, s); });
    });
}

muon_status muon_expert_sort_backward(const muon_expert_sort_backward_args* a, void* stream) {
    Buffers buf;
    MUON_TRY(check_expert_sort_backward(a, buf));
    return run_plain(14, "expert sort backward kernel", stream, [&](hipStream_t s) { return launch_expert_sort_backward(*a, s); });
}

muon_status muon_expert_combine(const muon_expert_combine_args* a, void* stream) {
    Buffers buf;
    MUON_TRY(check_expert_combine(a, buf));
    return run_plain(14, "expert combine kernel", stream, [&](hipStream_t s) { return launch_expert_combine(*a, s); });
}

muon_status muon_expert_combine_backward(const muon_expert_combine_backward_args* a, void* stream) {
    Buffers buf;
    MUON_TRY(check_expert_combine_backward(a, buf));
    return run_plain(14, "expert combine backward kernel", stream, [&](hipStream_t s) { return launch_expert_combine_backward(*a, s); });
}

}  // extern "C"
