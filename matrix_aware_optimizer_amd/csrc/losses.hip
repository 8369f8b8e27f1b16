// Losses over per-token log-probabilities, with their gradients: the preference loss over
// pairs of sequences and the clipped policy loss with a KL term (formulas in muon.h).
//
// Both are sums over ragged sequences followed by an elementwise gradient.  A first launch
// reduces each sequence (one workgroup per sequence), one workgroup joins the sequences
// into the loss and each one's gradient factor, and a last launch writes the gradient.
#include "train_internal.h"

namespace muon {

namespace {

constexpr int LS_THREADS = 256;

// Tokens of sequence s, clamped to [0, tokens).
struct Span {
    int64_t lo, hi;
    __device__ Span(const int64_t* offsets, int64_t s, int64_t tokens) {
        lo = min(max(offsets[s], static_cast<int64_t>(0)), tokens);
        hi = max(min(max(offsets[s + 1], static_cast<int64_t>(0)), tokens), lo);
    }
};

__device__ __forceinline__ bool counted(const uint8_t* mask, int64_t t) { return !mask || mask[t] != 0; }

// Zeros before the first and after the last sequence (workgroup 0 and the last one).
__device__ void zero_uncovered(void* grad, int dt, const int64_t* offsets, int64_t sequences, int64_t tokens) {
    if (!grad) return;
    const int64_t lo = sequences ? min(max(offsets[0], static_cast<int64_t>(0)), tokens) : tokens;
    const int64_t hi = sequences ? Span(offsets, sequences - 1, tokens).hi : tokens;
    const int64_t n = static_cast<int64_t>(gridDim.x) * LS_THREADS, i0 = static_cast<int64_t>(blockIdx.x) * LS_THREADS + threadIdx.x;
    for (int64_t t = i0; t < lo; t += n) st_dt(grad, t, 0.0f, dt);
    for (int64_t t = hi + i0; t < tokens; t += n) st_dt(grad, t, 0.0f, dt);
}

// ---- preference -------------------------------------------------------------

// sums[s] = { sum of counted log ratios, counted tokens }
__global__ __launch_bounds__(LS_THREADS) void preference_sums_kernel(muon_preference_args a, float* sums) {
    __shared__ float red[LS_THREADS / 64];
    const int64_t s = blockIdx.x;
    const Span sp(a.offsets, s, a.tokens);
    float v = 0.0f, c = 0.0f;
    for (int64_t t = sp.lo + threadIdx.x; t < sp.hi; t += LS_THREADS) {
        if (!counted(a.mask, t)) continue;
        v += ld_dt(a.logp, t, a.dtype) - (a.ref_logp ? ld_dt(a.ref_logp, t, a.dtype) : 0.0f);
        c += 1.0f;
    }
    v = block_sum<LS_THREADS>(v, red);
    c = block_sum<LS_THREADS>(c, red);
    if (threadIdx.x == 0) { sums[2 * s] = v; sums[2 * s + 1] = c; }
}

// log(1 + exp(x)) and 1 / (1 + exp(-x)) for any x
__device__ __forceinline__ float softplus(float x) { return fmaxf(x, 0.0f) + log1pf(expf(-fabsf(x))); }
__device__ __forceinline__ float sigmoid(float x) { return 1.0f / (1.0f + expf(-x)); }

// The loss and, in place of sums[2 s], the gradient factor of sequence s's counted tokens.
__global__ __launch_bounds__(LS_THREADS) void preference_pairs_kernel(muon_preference_args a, float* sums) {
    __shared__ float red[LS_THREADS / 64];
    const int64_t pairs = a.sequences / 2;
    float loss = 0.0f;
    for (int64_t p = threadIdx.x; p < pairs; p += LS_THREADS) {
        float w[2], r[2];
        for (int k = 0; k < 2; ++k) {
            w[k] = a.average ? 1.0f / fmaxf(sums[4 * p + 2 * k + 1], 1.0f) : 1.0f;
            r[k] = sums[4 * p + 2 * k] * w[k];
            if (a.rewards) a.rewards[2 * p + k] = a.beta * r[k];
        }
        const float u = r[0] - r[1], h = a.beta * u - a.margin, e = a.label_smoothing;
        float l, du;
        if (a.kind == MUON_PREFERENCE_SIGMOID) {
            l = (1.0f - e) * softplus(-h) + e * softplus(h);
            du = a.beta * (e * sigmoid(h) - (1.0f - e) * sigmoid(-h));
        } else if (a.kind == MUON_PREFERENCE_HINGE) {
            l = fmaxf(1.0f - h, 0.0f);
            du = h < 1.0f ? -a.beta : 0.0f;
        } else {
            const float q = u - 0.5f / a.beta;
            l = q * q;
            du = 2.0f * q;
        }
        loss += l;
        du *= a.grad_scale / static_cast<float>(pairs);
        sums[4 * p] = du * w[0];
        sums[4 * p + 2] = -du * w[1];
    }
    loss = block_sum<LS_THREADS>(loss, red);
    if (threadIdx.x == 0) *a.loss = pairs ? loss / static_cast<float>(pairs) : 0.0f;
}

__global__ __launch_bounds__(LS_THREADS) void preference_grad_kernel(muon_preference_args a, const float* sums) {
    zero_uncovered(a.grad_logp, a.dtype, a.offsets, a.sequences, a.tokens);
    if (static_cast<int64_t>(blockIdx.x) >= a.sequences) return;
    const Span sp(a.offsets, blockIdx.x, a.tokens);
    const float f = sums[2 * static_cast<int64_t>(blockIdx.x)];
    for (int64_t t = sp.lo + threadIdx.x; t < sp.hi; t += LS_THREADS)
        st_dt(a.grad_logp, t, counted(a.mask, t) ? f : 0.0f, a.dtype);
}

// ---- policy -----------------------------------------------------------------

struct PolicyToken { float loss, grad, kl, held, rho; };

__device__ __forceinline__ PolicyToken policy_token(const muon_policy_args& a, int64_t t, float adv) {
    const float lp = ld_dt(a.logp, t, a.dtype), lo = 1.0f - a.clip_low, hi = 1.0f + a.clip_high;
    PolicyToken o;
    o.rho = expf(lp - ld_dt(a.old_logp, t, a.dtype));
    float gain = fminf(o.rho * adv, fminf(fmaxf(o.rho, lo), hi) * adv);
    bool held = (adv > 0.0f && o.rho > hi) || (adv < 0.0f && o.rho < lo);
    if (a.dual_clip > 0.0f && adv < 0.0f && o.rho > a.dual_clip) {
        gain = a.dual_clip * adv;
        held = true;
    }
    o.held = held ? 1.0f : 0.0f;
    o.loss = -gain;
    o.grad = held ? 0.0f : -o.rho * adv;
    o.kl = 0.0f;
    if (a.kl != MUON_KL_NONE) {
        const float q = ld_dt(a.ref_logp, t, a.dtype) - lp;
        float dk;
        if (a.kl == MUON_KL_K1) { o.kl = -q; dk = 1.0f; }
        else if (a.kl == MUON_KL_K2) { o.kl = 0.5f * q * q; dk = -q; }
        else { const float em = expm1f(q); o.kl = em - q; dk = -em; }
        o.loss += a.kl_coef * o.kl;
        o.grad += a.kl_coef * dk;
    }
    return o;
}

constexpr int PL_SUMS = 5;   // loss, KL, held, rho, counted tokens

__global__ __launch_bounds__(LS_THREADS) void policy_sums_kernel(muon_policy_args a, float* sums) {
    __shared__ float red[LS_THREADS / 64];
    const int64_t s = blockIdx.x;
    const Span sp(a.offsets, s, a.tokens);
    float v[PL_SUMS] = {};
    for (int64_t t = sp.lo + threadIdx.x; t < sp.hi; t += LS_THREADS) {
        if (!counted(a.mask, t)) continue;
        const PolicyToken o = policy_token(a, t, a.advantages[a.advantage_per_sequence ? s : t]);
        v[0] += o.loss; v[1] += o.kl; v[2] += o.held; v[3] += o.rho; v[4] += 1.0f;
    }
    for (int k = 0; k < PL_SUMS; ++k) {
        const float x = block_sum<LS_THREADS>(v[k], red);
        if (threadIdx.x == 0) sums[PL_SUMS * s + k] = x;
    }
}

// The loss and the statistics; a sequence's weight replaces its loss sum.
__global__ __launch_bounds__(LS_THREADS) void policy_join_kernel(muon_policy_args a, float* sums) {
    __shared__ float red[LS_THREADS / 64];
    float v[PL_SUMS] = {};
    for (int64_t s = threadIdx.x; s < a.sequences; s += LS_THREADS) {
        const float* q = sums + PL_SUMS * s;
        v[0] += a.reduction == MUON_REDUCE_SEQUENCE ? q[0] / fmaxf(q[4], 1.0f) : q[0];
        for (int k = 1; k < PL_SUMS; ++k) v[k] += q[k];
    }
    for (int k = 0; k < PL_SUMS; ++k) v[k] = block_sum<LS_THREADS>(v[k], red);
    const float per_token = 1.0f / fmaxf(v[4], 1.0f), per_seq = 1.0f / fmaxf(static_cast<float>(a.sequences), 1.0f);
    if (threadIdx.x == 0) {
        *a.loss = v[0] * (a.reduction == MUON_REDUCE_SEQUENCE ? per_seq : per_token);
        if (a.stats) {
            a.stats[0] = v[1] * per_token;
            a.stats[1] = v[2] * per_token;
            a.stats[2] = v[3] * per_token;
            a.stats[3] = v[4];
        }
    }
    for (int64_t s = threadIdx.x; s < a.sequences; s += LS_THREADS)
        sums[PL_SUMS * s] = a.grad_scale *
                            (a.reduction == MUON_REDUCE_SEQUENCE ? per_seq / fmaxf(sums[PL_SUMS * s + 4], 1.0f) : per_token);
}

__global__ __launch_bounds__(LS_THREADS) void policy_grad_kernel(muon_policy_args a, const float* sums) {
    zero_uncovered(a.grad_logp, a.dtype, a.offsets, a.sequences, a.tokens);
    const int64_t s = blockIdx.x;
    if (s >= a.sequences) return;
    const Span sp(a.offsets, s, a.tokens);
    const float f = sums[PL_SUMS * s];
    for (int64_t t = sp.lo + threadIdx.x; t < sp.hi; t += LS_THREADS) {
        float g = 0.0f;
        if (counted(a.mask, t)) g = f * policy_token(a, t, a.advantages[a.advantage_per_sequence ? s : t]).grad;
        st_dt(a.grad_logp, t, g, a.dtype);
    }
}

unsigned seq_grid(int64_t sequences) { return static_cast<unsigned>(sequences > 0 ? sequences : 1); }

}  // namespace

size_t preference_bytes(const muon_preference_args& a) { return 2 * sizeof(float) * static_cast<size_t>(a.sequences); }

hipError_t launch_preference(const muon_preference_args& a, void* workspace, hipStream_t s) {
    float* sums = static_cast<float*>(workspace);
    if (a.sequences > 0)
        hipLaunchKernelGGL(preference_sums_kernel, dim3(seq_grid(a.sequences)), dim3(LS_THREADS), 0, s, a, sums);
    hipLaunchKernelGGL(preference_pairs_kernel, dim3(1), dim3(LS_THREADS), 0, s, a, sums);
    if (a.grad_logp)
        hipLaunchKernelGGL(preference_grad_kernel, dim3(seq_grid(a.sequences)), dim3(LS_THREADS), 0, s, a, sums);
    return hipGetLastError();
}

size_t policy_bytes(const muon_policy_args& a) { return PL_SUMS * sizeof(float) * static_cast<size_t>(a.sequences); }

hipError_t launch_policy(const muon_policy_args& a, void* workspace, hipStream_t s) {
    float* sums = static_cast<float*>(workspace);
    if (a.sequences > 0)
        hipLaunchKernelGGL(policy_sums_kernel, dim3(seq_grid(a.sequences)), dim3(LS_THREADS), 0, s, a, sums);
    hipLaunchKernelGGL(policy_join_kernel, dim3(1), dim3(LS_THREADS), 0, s, a, sums);
    if (a.grad_logp)
        hipLaunchKernelGGL(policy_grad_kernel, dim3(seq_grid(a.sequences)), dim3(LS_THREADS), 0, s, a, sums);
    return hipGetLastError();
}

}  // namespace muon
