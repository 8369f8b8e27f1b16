// Losses over per-token log-probabilities, with their gradients: the preference loss over
// pairs of sequences and the clipped policy loss with a KL term (formulas in muon.h).
//
// A few bytes and operations a token: HBM-bound for millions of tokens, launch- and
// latency-bound for thousands.  The work is cut by tokens, not by sequences, so that one long
// sequence among short ones spreads like any other: a wave takes a unit of 512 tokens, 8 a lane
// (one 32-byte access each), and walks over the pieces of sequences in its unit.
//
// A sequence's sum is put together from its units' in token order, so results do not depend
// on scheduling.  Per unit u: head[u] is the sum of the piece that starts at the unit's first
// token, tail[u] that of the piece that starts inside and goes on past its end; a sequence
// that lies inside a unit, past its first token, has its sum in own[s].  So sequence [lo, hi) is
//   (lo at a unit's start ? head : hi in the same unit ? own[s] : tail)[its first unit] + head[every later unit].
//
// Preference: units -> pairs (loss terms and each sequence's gradient factor) -> gradient.
// Policy: the number of counted tokens first (1 byte a token, only with a mask), then loss and
// gradient in one pass over the rest, then the partial sums.  Up to LS_SMALL tokens all steps run in one
// workgroup and one launch: a wave keeps its unit's tokens in registers, the offsets and sums sit in LDS.  (The state that
// the steps pass on, arguments and LDS addresses, lies in scratch there: 168 and 184 bytes a lane.)
//
// Preference, 1.18 M tokens in 256 pairs (15 MB): three launches of 4.9, 5.5 and 4.5 us, each little more than its latency; 8 sequences
// in one launch 9.4 us (three: 16).  Policy, 2.36 M tokens in 2048 sequences (42 MB): 18 us (2.3 TB/s) after 4 - 5 us of counting and
// before 4 us of sums: the search for a unit's sequences, their offsets and advantages, then its tokens are loads that wait for each
// other.  1.35 M tokens in 6 sequences: 13 us + 3.9 + 3.8.
#include <algorithm>

#include "train_internal.h"

namespace muon {

namespace {

constexpr int UNIT = 512, PER = 8;       // tokens of a wave's unit, of a lane
constexpr int LS_THREADS = 256;          // workgroups of the launches over many units: 4 waves
constexpr int LS_ONE = 1024;             // the workgroup that does everything, at most: 16 waves
// Tokens up to which it does: one unit a wave (6 pairs of up to 1024 tokens: 12.8 us, 16 with the launches over many units; 12
// policy sequences of up to 1000: 16.6 us, 18).
constexpr int64_t LS_SMALL = LS_ONE / 64 * UNIT;
constexpr int LS_SMALL_SEQS = 1024;      // sequences up to which it does: their offsets and sums in LDS
// Workgroups of the other launches, at most: 5 a CU, what the registers hold (policy, 2048 sequences: 26 us; 2 a CU: 29).
constexpr int LS_GRID = 1280;
constexpr int LS_COUNTS = 1024;          // workgroups that count, at most: one partial each (256: 1 us more)
// Units beyond which the counts of sequences are joined by a launch of their own; up to it each unit adds up the others of its
// sequence itself, at most 64 loads a lane, which grows with the square of a sequence (one sequence of 1.0, 2.1, 4.2, 16.9 million
// tokens: 23, 36, 86, 897 us; joined 20, 28, 39, 111; six of 1.35 million in all: 19, joined 28).
constexpr int64_t LS_JOIN = 4096;

__device__ __forceinline__ int lane_id() { return threadIdx.x & 63; }

// Tokens t .. t + 7 of a vector of n, zero past its end.
template <typename T> __device__ __forceinline__ void load_tokens(const void* p, int t, int n, float (&o)[PER]) {
    Run<T> r;
    const auto* q = G(static_cast<const T*>(p));
    if (t + PER <= n) r.load(q, t);
    else if (t < n) r.load(q, t, n - t);
#pragma unroll
    for (int e = 0; e < PER; ++e) o[e] = r.get(e);
}
template <typename T> __device__ __forceinline__ void store_tokens(void* p, int t, int n, const float (&o)[PER]) {
    auto* q = G(static_cast<T*>(p));
    if (t + PER <= n) {
        st_run(q, t, o);
    } else {
#pragma unroll
        for (int e = 0; e < PER - 1; ++e)
            if (t + e < n) st_el<T>(p, t + e, o[e]);
    }
}
// Bit e: token t + e exists and its mask counts it.
__device__ __forceinline__ unsigned load_mask(const uint8_t* mask, int t, int n) {
    const unsigned there = t + PER <= n ? 0xffu : t < n ? (1u << (n - t)) - 1u : 0u;
    if (!mask) return there;
    unsigned m = 0;
    typedef u32x2_t u32x2_el1 __attribute__((aligned(1)));
    if (t + PER <= n) {
        const u32x2_t w = *(const global_t<u32x2_el1>*)(G(mask) + t);
#pragma unroll
        for (int e = 0; e < PER; ++e) m |= ((w[e >> 2] >> (8 * (e & 3))) & 0xffu) ? 1u << e : 0u;
    } else {
#pragma unroll
        for (int e = 0; e < PER - 1; ++e)
            if (t + e < n && G(mask)[t + e]) m |= 1u << e;
    }
    return m;
}

// The sequences, as offsets clamped to the tokens there are (so no offset makes an access stray).
// OFF: int64_t as the caller has them, or int where a workgroup keeps them clamped in LDS.
template <typename OFF> struct Sequences {
    const OFF* offsets;
    int count, tokens;
    __device__ __forceinline__ int at(int k) const {
        const OFF v = offsets[k];
        return static_cast<int>(v < 0 ? 0 : v > tokens ? tokens : v);
    }
    // The last k with at(k) <= t, or -1: 64 probes at a time.
    __device__ __forceinline__ int last_at_most(int t) const {
        int lo = 0, hi = count + 1;   // the number of such k lies in [lo, hi]
        while (lo < hi) {
            const int step = (hi - lo + 63) / 64, k = lo + lane_id() * step;
            const int c = __popcll(__ballot(k < hi && at(k) <= t));
            if (c == 0) break;
            const int next = lo + (c - 1) * step + 1;
            hi = min(hi, lo + c * step);
            lo = next;
        }
        return lo - 1;
    }
    // f(s, a, b, lo, hi, side) for every sequence s = [lo, hi) with a piece [a, b) in [t0, t1).  `side`: value
    // of extra(s) of that sequence, loaded 63 sequences at a time with the offsets.
    template <typename E, typename F> __device__ __forceinline__ void pieces(int t0, int t1, E extra, F f) const {
        for (int s0 = max(last_at_most(t0), 0); s0 < count; s0 += 63) {
            const int k = min(s0 + lane_id(), count);
            const int off = at(k);
            const float ex = extra(min(k, count - 1));
            const int n = min(63, count - s0);
            for (int i = 0; i < n; ++i) {
                const int lo = __builtin_amdgcn_readlane(off, i), hi = max(__builtin_amdgcn_readlane(off, i + 1), lo);
                if (lo >= t1) return;
                const int a = max(lo, t0), b = min(hi, t1);
                if (a < b) f(s0 + i, a, b, lo, hi, __int_as_float(__builtin_amdgcn_readlane(__float_as_int(ex), i)));
            }
        }
    }
};

// Bit e: token t + e lies in [a, b).
__device__ __forceinline__ unsigned in_piece(int t, int a, int b) {
    const int l = min(max(a - t, 0), PER), h = min(max(b - t, 0), PER);
    return (1u << h) - (1u << l) & (h > l ? ~0u : 0u);
}

// Sums of sequences by unit: V = float or double2.
template <typename V> struct UnitSums {
    V *head, *tail, *own;
    __device__ __forceinline__ void put(int s, int a, int lo, int hi, V v) const {
        const int u = a / UNIT;
        if (a == u * UNIT) head[u] = v;
        else if (hi <= (u + 1) * UNIT) own[s] = v;
        else tail[u] = v;
    }
    __device__ __forceinline__ V first(int s, int lo, int hi) const {
        const int u = lo / UNIT;
        return lo == u * UNIT ? head[u] : hi <= (u + 1) * UNIT ? own[s] : tail[u];
    }
};
__device__ __forceinline__ float add(float a, float b) { return a + b; }
__device__ __forceinline__ double2 add(double2 a, double2 b) { return make_double2(a.x + b.x, a.y + b.y); }
__device__ __forceinline__ float wave_total(float v) { return wave_sum(v); }
__device__ __forceinline__ double2 wave_total(double2 v) { return make_double2(wave_sum(v.x), wave_sum(v.y)); }

// head[first .. last] summed by the wave.
template <typename V> __device__ __forceinline__ V heads(const UnitSums<V>& q, int first, int last) {
    V v = {};
#pragma unroll 8
    for (int u = first + lane_id(); u <= last; u += 64) v = add(v, q.head[u]);
    return wave_total(v);
}

// ---- preference -------------------------------------------------------------

// Log ratios are summed and subtracted in fp64: without a reference a pair's difference may be a millionth of its two sums
// (60000 tokens each: fp32 sums were off by 4e-3 of a log-probability).

template <typename OFF> struct PreferenceState {
    typedef double2 Sum;
    muon_preference_args a;
    Sequences<OFF> seqs;
    UnitSums<double2> q;    // { sum of counted log ratios, counted tokens }
    float* factor;          // gradient factor by sequence
    float* losses;          // by pair
    __device__ int units() const { return static_cast<int>((a.tokens + UNIT - 1) / UNIT); }
};

// What a lane reads of its 8 tokens.
struct PreferenceTokens {
    float lp[PER], ref[PER] = {};
    unsigned live;
    template <typename T> __device__ __forceinline__ void load(const muon_preference_args& a, int t) {
        const int n = static_cast<int>(a.tokens);
        load_tokens<T>(a.logp, t, n, lp);
        if (a.ref_logp) load_tokens<T>(a.ref_logp, t, n, ref);
        live = load_mask(a.mask, t, n);
    }
};

template <typename S> __device__ __forceinline__ void preference_unit(const S& st, int u, const PreferenceTokens& k) {
    const int t0 = u * UNIT, t = t0 + PER * lane_id();
    st.seqs.pieces(t0, t0 + UNIT, [](int) { return 0.0f; }, [&](int s, int a, int b, int lo, int hi, float) {
        const unsigned on = k.live & in_piece(t, a, b);
        double v = 0.0;
#pragma unroll
        for (int e = 0; e < PER; ++e) v += (on >> e & 1u) ? static_cast<double>(k.lp[e]) - static_cast<double>(k.ref[e]) : 0.0;
        v = wave_sum(v);
        const float c = wave_sum(static_cast<float>(__popc(on)));
        if (lane_id() == 0) st.q.put(s, a, lo, hi, make_double2(v, c));
    });
}

// Sum of the sequence that each lane asks for (s < 0: none), short ones lane by lane, long ones by the wave.
template <typename S> __device__ __forceinline__ typename S::Sum lane_sequence_sums(const S& st, int s) {
    typedef typename S::Sum Sum;
    int lo = 0, hi = 0;
    if (s >= 0) {
        lo = st.seqs.at(s);
        hi = max(st.seqs.at(s + 1), lo);
    }
    Sum v = {};
    constexpr int NEAR = 8;   // units past the first, whose sums a lane loads at once
    const int u0 = lo / UNIT, u1 = hi > lo ? (hi - 1) / UNIT : u0;
    const bool far = u1 - u0 > NEAR;
    if (hi > lo) {
        v = st.q.first(s, lo, hi);
        if (!far && u1 > u0) {
            Sum h[NEAR];
#pragma unroll
            for (int k = 0; k < NEAR; ++k) h[k] = st.q.head[min(u0 + 1 + k, u1)];
#pragma unroll
            for (int k = 0; k < NEAR; ++k)
                if (u0 + 1 + k <= u1) v = add(v, h[k]);
        }
    }
    for (unsigned long long todo = __ballot(far); todo; todo &= todo - 1) {
        const int l = __ffsll(todo) - 1;
        const Sum h = heads(st.q, __builtin_amdgcn_readlane(u0, l) + 1, __builtin_amdgcn_readlane(u1, l));
        if (lane_id() == l) v = add(v, h);
    }
    return v;
}

// log(1 + exp(x)) and 1 / (1 + exp(-x)) for any x
__device__ __forceinline__ float softplus(float x) { return fmaxf(x, 0.0f) + log1pf(expf(-fabsf(x))); }
__device__ __forceinline__ float sigmoid(float x) { return 1.0f / (1.0f + expf(-x)); }

// A pair a lane: its loss term and its sequences' gradient factors.
template <typename S> __device__ __forceinline__ void preference_pairs(const S& st, int wave, int waves) {
    const muon_preference_args& a = st.a;
    const int pairs = static_cast<int>(a.sequences / 2);
    for (int p0 = wave * 64; p0 < pairs; p0 += waves * 64) {
        const int p = p0 + lane_id();
        const bool on = p < pairs;
        float w[2];
        double r[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const double2 v = lane_sequence_sums(st, on ? 2 * p + k : -1);
            const double n = fmax(v.y, 1.0);
            w[k] = a.average ? 1.0f / static_cast<float>(n) : 1.0f;
            r[k] = a.average ? v.x / n : v.x;
            if (on && a.rewards) a.rewards[2 * p + k] = static_cast<float>(a.beta * r[k]);
        }
        const double u = r[0] - r[1];
        const float h = static_cast<float>(a.beta * u - a.margin), e = a.label_smoothing;
        float l, du;
        if (a.kind == MUON_PREFERENCE_SIGMOID) {
            // a share of 0 counts for nothing, also where its term is infinite
            l = (e < 1.0f ? (1.0f - e) * softplus(-h) : 0.0f) + (e > 0.0f ? e * softplus(h) : 0.0f);
            du = a.beta * (e * sigmoid(h) - (1.0f - e) * sigmoid(-h));
        } else if (a.kind == MUON_PREFERENCE_HINGE) {
            l = fmaxf(1.0f - h, 0.0f);
            du = h < 1.0f ? -a.beta : 0.0f;
        } else {
            const float q = static_cast<float>(u - 0.5 / a.beta);
            l = q * q;
            du = 2.0f * q;
        }
        du *= a.grad_scale / static_cast<float>(pairs);
        if (on) {
            st.losses[p] = l;
            st.factor[2 * p] = du * w[0];
            st.factor[2 * p + 1] = -du * w[1];
        }
    }
}

template <typename S> __device__ __forceinline__ void preference_loss(const S& st, float* red) {
    const int pairs = static_cast<int>(st.a.sequences / 2);
    float v = 0.0f;
#pragma unroll 4
    for (int p = threadIdx.x; p < pairs; p += blockDim.x) v += st.losses[p];
    v = block_sum(v, red);
    if (threadIdx.x == 0) *st.a.loss = pairs ? v / static_cast<float>(pairs) : 0.0f;
}

template <typename T, typename S> __device__ __forceinline__ void preference_grad(const S& st, int u, unsigned live) {
    const int t0 = u * UNIT, t = t0 + PER * lane_id();
    float g[PER] = {};
    st.seqs.pieces(t0, t0 + UNIT, [&](int s) { return st.factor[s]; }, [&](int, int a, int b, int, int, float f) {
        const unsigned on = live & in_piece(t, a, b);
#pragma unroll
        for (int e = 0; e < PER; ++e)
            if (on >> e & 1u) g[e] = f;
    });
    store_tokens<T>(st.a.grad_logp, t, static_cast<int>(st.a.tokens), g);
}

__device__ __forceinline__ int wave_index() { return __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6)); }

enum PreferenceStep { PF_UNITS = 0, PF_PAIRS = 1, PF_GRAD = 2 };

template <typename T, int STEP> __global__ __launch_bounds__(LS_THREADS) void preference_kernel(PreferenceState<int64_t> st) {
    __shared__ float red[LS_THREADS / 64];
    constexpr int W = LS_THREADS / 64;
    if (STEP == PF_UNITS) {
        for (int u = blockIdx.x * W + wave_index(); u < st.units(); u += gridDim.x * W) {
            PreferenceTokens k;
            k.load<T>(st.a, u * UNIT + PER * lane_id());
            preference_unit(st, u, k);
        }
    } else if (STEP == PF_PAIRS) {
        preference_pairs(st, blockIdx.x * W + wave_index(), gridDim.x * W);
    } else if (blockIdx.x == 0) {
        preference_loss(st, red);
    } else {
        for (int u = (blockIdx.x - 1) * W + wave_index(); u < st.units(); u += (gridDim.x - 1) * W)
            preference_grad<T>(st, u, load_mask(st.a.mask, u * UNIT + PER * lane_id(), static_cast<int>(st.a.tokens)));
    }
}

// Offsets, clamped, into LDS; a barrier follows.
__device__ __forceinline__ void offsets_to_lds(const int64_t* offsets, int64_t sequences, int64_t tokens, int* lds) {
    const Sequences<int64_t> sq{offsets, static_cast<int>(sequences), static_cast<int>(tokens)};
    for (int k = threadIdx.x; k <= sq.count; k += blockDim.x) lds[k] = sq.at(k);
}

template <typename T> __global__ __launch_bounds__(LS_ONE) void preference_one_kernel(muon_preference_args a) {
    constexpr int W = LS_ONE / 64;
    __shared__ float red[W];
    __shared__ int offsets[LS_SMALL_SEQS + 1];
    __shared__ double2 head[W], tail[W], own[LS_SMALL_SEQS];
    __shared__ float factor[LS_SMALL_SEQS], losses[LS_SMALL_SEQS / 2];
    const int u = wave_index();
    const PreferenceState<int> st{a, {offsets, static_cast<int>(a.sequences), static_cast<int>(a.tokens)}, {head, tail, own}, factor, losses};
    PreferenceTokens k;
    k.load<T>(a, u * UNIT + PER * lane_id());
    offsets_to_lds(a.offsets, a.sequences, a.tokens, offsets);
    __syncthreads();
    if (u < st.units()) preference_unit(st, u, k);
    __syncthreads();
    preference_pairs(st, u, blockDim.x / 64);
    __syncthreads();
    if (a.grad_logp && u < st.units()) preference_grad<T>(st, u, k.live);
    preference_loss(st, red);
}

// ---- policy -----------------------------------------------------------------

// Weighted loss, KL, held, rho, counted tokens.  Summed in fp64: gains of both signs cancel, and fp32 sums
// of 32616 tokens lost 1.3e-6 of a loss near 0.
constexpr int PL_SUMS = 5;

template <typename OFF> struct PolicyState {
    typedef float Sum;
    muon_policy_args a;
    Sequences<OFF> seqs;
    UnitSums<float> q;      // counted tokens by unit: sequence means with a mask
    bool joined = false;    // own[s] holds the whole count of every sequence that goes beyond a unit
    __device__ int units() const { return static_cast<int>((a.tokens + UNIT - 1) / UNIT); }
    __device__ bool by_sequence() const { return a.reduction == MUON_REDUCE_SEQUENCE; }
    // Nothing about a token depends on its sequence.
    __device__ bool flat() const { return !by_sequence() && !a.advantage_per_sequence; }
    __device__ unsigned covered(int t) const { return seqs.count ? in_piece(t, seqs.at(0), seqs.at(seqs.count)) : 0u; }
};

// Counted tokens of a unit's sequences that go on beyond it (the others are counted where they are used).
template <typename S> __device__ __forceinline__ void policy_unit_counts(const S& st, int u, unsigned live) {
    const int t0 = u * UNIT, t = t0 + PER * lane_id();
    st.seqs.pieces(t0, t0 + UNIT, [](int) { return 0.0f; }, [&](int s, int a, int b, int lo, int hi, float) {
        if (lo >= t0 && hi <= t0 + UNIT) return;
        const float c = wave_sum(static_cast<float>(__popc(live & in_piece(t, a, b))));
        if (lane_id() == 0) st.q.put(s, a, lo, hi, c);
    });
}

struct PolicyToken { double loss; float grad, kl, rho; bool held; };

// The ratio is taken as 1 + expm1, put together in fp64: near 1 a rounded ratio alone would cost a loss that is small against
// its terms its last digits.
__device__ __forceinline__ PolicyToken policy_token(const muon_policy_args& a, float lp, float old, float ref, float adv) {
    const float lo = 1.0f - a.clip_low, hi = 1.0f + a.clip_high;
    PolicyToken o;
    float em = expm1f(lp - old);
    o.rho = 1.0f + em;
    const bool above = adv > 0.0f && o.rho > hi, below = adv < 0.0f && o.rho < lo;
    const bool dual = a.dual_clip > 0.0f && adv < 0.0f && o.rho > a.dual_clip;
    em = above ? a.clip_high : below ? -a.clip_low : em;
    o.held = above || below || dual;
    o.loss = -(dual ? static_cast<double>(a.dual_clip) : 1.0 + static_cast<double>(em)) * static_cast<double>(adv);
    o.grad = o.held ? 0.0f : -o.rho * adv;
    o.kl = 0.0f;
    if (a.kl != MUON_KL_NONE) {
        const float q = ref - lp;
        float dk;
        if (a.kl == MUON_KL_K1) { o.kl = -q; dk = 1.0f; }
        else if (a.kl == MUON_KL_K2) { o.kl = 0.5f * q * q; dk = -q; }
        else { const float em = expm1f(q); o.kl = em - q; dk = -em; }
        o.loss = fma(static_cast<double>(a.kl_coef), static_cast<double>(o.kl), o.loss);
        o.grad = fmaf(a.kl_coef, dk, o.grad);
    }
    return o;
}

// What a lane reads of its 8 tokens, then their weights.
struct PolicyTokens {
    float lp[PER], old[PER], ref[PER] = {}, adv[PER] = {}, wt[PER] = {};
    unsigned live, counted = 0;
    template <typename T> __device__ __forceinline__ void load(const muon_policy_args& a, int t) {
        const int n = static_cast<int>(a.tokens);
        load_tokens<T>(a.logp, t, n, lp);
        load_tokens<T>(a.old_logp, t, n, old);
        if (a.kl != MUON_KL_NONE) load_tokens<T>(a.ref_logp, t, n, ref);
        if (!a.advantage_per_sequence) load_tokens<float>(a.advantages, t, n, adv);
        live = load_mask(a.mask, t, n);
    }
};

// Which of the tokens count, their advantages and weights (1 under a token mean, whose weight comes later).  `advantages`: by
// sequence, if they are.
template <typename S>
__device__ __forceinline__ void policy_weights(const S& st, int u, const float* advantages, PolicyTokens& k) {
    const int t0 = u * UNIT, t = t0 + PER * lane_id();
    if (st.flat()) {
        k.counted = k.live & st.covered(t);
#pragma unroll
        for (int e = 0; e < PER; ++e) k.wt[e] = 1.0f;
        return;
    }
    const bool per_seq = st.a.advantage_per_sequence != 0;
    st.seqs.pieces(t0, t0 + UNIT, [&](int s) { return per_seq ? advantages[s] : 0.0f; },
                   [&](int s, int a, int b, int lo, int hi, float side) {
                       const unsigned on = k.live & in_piece(t, a, b);
                       float w = 1.0f;
                       if (st.by_sequence()) {
                           float c;
                           if (!st.a.mask) c = static_cast<float>(hi - lo);
                           else if (lo >= t0 && hi <= t0 + UNIT) c = wave_sum(static_cast<float>(__popc(on)));
                           else if (st.joined) c = st.q.own[s];
                           else c = st.q.first(s, lo, hi) + heads(st.q, lo / UNIT + 1, (hi - 1) / UNIT);
                           w = 1.0f / (fmaxf(c, 1.0f) * static_cast<float>(st.seqs.count));
                       }
                       k.counted |= on;
#pragma unroll
                       for (int e = 0; e < PER; ++e)
                           if (on >> e & 1u) {
                               k.wt[e] = w;
                               if (per_seq) k.adv[e] = side;
                           }
                   });
}

// The tokens' sums, and their gradients before the common factor.
__device__ __forceinline__ void policy_tokens(const muon_policy_args& a, const PolicyTokens& k, double (&v)[PL_SUMS], float (&g)[PER]) {
    float kl = 0.0f, rho = 0.0f;
    int held = 0;
#pragma unroll
    for (int e = 0; e < PER; ++e) {
        g[e] = 0.0f;
        if (!(k.counted >> e & 1u)) continue;
        const PolicyToken o = policy_token(a, k.lp[e], k.old[e], k.ref[e], k.adv[e]);
        v[0] = fma(static_cast<double>(k.wt[e]), o.loss, v[0]);
        kl += o.kl;
        rho += o.rho;
        held += o.held;
        g[e] = k.wt[e] * o.grad;
    }
    v[1] += kl;
    v[2] += held;
    v[3] += rho;
    v[4] += __popc(k.counted);
}
template <typename T>
__device__ __forceinline__ void policy_store(const muon_policy_args& a, int u, float factor, float (&g)[PER]) {
#pragma unroll
    for (int e = 0; e < PER; ++e) g[e] *= factor;
    store_tokens<T>(a.grad_logp, u * UNIT + PER * lane_id(), static_cast<int>(a.tokens), g);
}

// v: the sums over everything.
__device__ __forceinline__ void policy_write(const muon_policy_args& a, const double (&v)[PL_SUMS]) {
    const double per = 1.0 / fmax(v[4], 1.0);
    *a.loss = static_cast<float>(a.reduction == MUON_REDUCE_SEQUENCE ? v[0] : v[0] * per);
    if (!a.stats) return;
    a.stats[0] = static_cast<float>(v[1] * per);
    a.stats[1] = static_cast<float>(v[2] * per);
    a.stats[2] = static_cast<float>(v[3] * per);
    a.stats[3] = static_cast<float>(v[4]);
}

// With a mask: the counted tokens of all sequences, one partial a workgroup, or of each one's units.
__global__ __launch_bounds__(LS_THREADS) void policy_counts_kernel(PolicyState<int64_t> st, float* counts) {
    __shared__ float red[LS_THREADS / 64];
    constexpr int W = LS_THREADS / 64;
    const int n = static_cast<int>(st.a.tokens);
    float total = 0.0f;
    for (int u = blockIdx.x * W + wave_index(); u < st.units(); u += gridDim.x * W) {
        const int t = u * UNIT + PER * lane_id();
        const unsigned live = load_mask(st.a.mask, t, n);
        if (st.by_sequence()) policy_unit_counts(st, u, live);
        else total += static_cast<float>(__popc(live & st.covered(t)));
    }
    if (st.by_sequence()) return;
    total = block_sum(total, red);
    if (threadIdx.x == 0) counts[blockIdx.x] = total;
}

// The counts of the sequences that go beyond a unit, each put together once.
__global__ __launch_bounds__(LS_THREADS) void policy_join_kernel(PolicyState<int64_t> st) {
    constexpr int W = LS_THREADS / 64;
    for (int s0 = (blockIdx.x * W + wave_index()) * 64; s0 < st.seqs.count; s0 += gridDim.x * W * 64) {
        const int s = s0 + lane_id(), lo = st.seqs.at(min(s, st.seqs.count - 1)), hi = st.seqs.at(min(s, st.seqs.count - 1) + 1);
        const bool on = s < st.seqs.count && hi > lo && hi > (lo / UNIT + 1) * UNIT;
        const float c = lane_sequence_sums(st, on ? s : -1);
        if (on) st.q.own[s] = c;
    }
}

// counts: `parts` partial counts (token mean with a mask).  sums: PL_SUMS by workgroup.
template <typename T>
__global__ __launch_bounds__(LS_THREADS, LS_GRID / 256) void policy_main_kernel(PolicyState<int64_t> st, const float* counts, int parts, double* sums) {
    constexpr int W = LS_THREADS / 64;
    __shared__ double red[PL_SUMS * W];
    const muon_policy_args& a = st.a;
    float factor = 0.0f;
    bool known = false;
    double v[PL_SUMS] = {};
    for (int u = blockIdx.x * W + wave_index(); u < st.units(); u += gridDim.x * W) {
        PolicyTokens k;
        k.load<T>(a, u * UNIT + PER * lane_id());
        if (!known) {   // once, behind the first unit's loads
            factor = a.grad_scale;
            if (!st.by_sequence()) {
                float total;
                if (a.mask) {
                    float c = 0.0f;
                    for (int p = lane_id(); p < parts; p += 64) c += counts[p];
                    total = wave_sum(c);
                } else {
                    total = st.seqs.count ? static_cast<float>(max(st.seqs.at(st.seqs.count) - st.seqs.at(0), 0)) : 0.0f;
                }
                factor /= fmaxf(total, 1.0f);
            }
            known = true;
        }
        policy_weights(st, u, a.advantages, k);
        float g[PER];
        policy_tokens(a, k, v, g);
        if (a.grad_logp) policy_store<T>(a, u, factor, g);
    }
    block_sums(v, red);
    if (threadIdx.x == 0)
#pragma unroll
        for (int k = 0; k < PL_SUMS; ++k) sums[PL_SUMS * blockIdx.x + k] = v[k];
}

__global__ __launch_bounds__(LS_THREADS) void policy_final_kernel(muon_policy_args a, const double* sums, int blocks) {
    __shared__ double red[PL_SUMS * LS_THREADS / 64];
    double v[PL_SUMS] = {};
#pragma unroll 4
    for (int b = threadIdx.x; b < blocks; b += LS_THREADS)
#pragma unroll
        for (int k = 0; k < PL_SUMS; ++k) v[k] += sums[PL_SUMS * b + k];
    block_sums(v, red);
    if (threadIdx.x == 0) policy_write(a, v);
}

template <typename T> __global__ __launch_bounds__(LS_ONE) void policy_one_kernel(muon_policy_args a) {
    constexpr int W = LS_ONE / 64;
    __shared__ double red[PL_SUMS * W];
    __shared__ int offsets[LS_SMALL_SEQS + 1];
    __shared__ float head[W], tail[W], own[LS_SMALL_SEQS], adv[LS_SMALL_SEQS];
    const int u = wave_index();
    const PolicyState<int> st{a, {offsets, static_cast<int>(a.sequences), static_cast<int>(a.tokens)}, {head, tail, own}};
    PolicyTokens k;
    k.load<T>(a, u * UNIT + PER * lane_id());
    offsets_to_lds(a.offsets, a.sequences, a.tokens, offsets);
    if (a.advantage_per_sequence)
        for (int s = threadIdx.x; s < st.seqs.count; s += blockDim.x) adv[s] = a.advantages[s];
    __syncthreads();
    if (st.by_sequence() && a.mask) {
        if (u < st.units()) policy_unit_counts(st, u, k.live);
        __syncthreads();
    }
    double v[PL_SUMS] = {};
    float g[PER] = {};
    if (u < st.units()) {
        policy_weights(st, u, adv, k);
        policy_tokens(a, k, v, g);
    }
    block_sums(v, red);
    if (a.grad_logp && u < st.units()) policy_store<T>(a, u, st.by_sequence() ? a.grad_scale : a.grad_scale / fmaxf(static_cast<float>(v[4]), 1.0f), g);
    if (threadIdx.x == 0) policy_write(a, v);
}

// ---- host ---------------------------------------------------------------------

int64_t units_of(int64_t tokens) { return (tokens + UNIT - 1) / UNIT; }
unsigned one_block(int64_t tokens) { return static_cast<unsigned>(64 * std::max<int64_t>(1, units_of(tokens))); }
// Workgroups for so many waves' units: at most `most`, each wave with as many units as any other (or one less).
unsigned grid_for(int64_t units, int most) {
    const int64_t rounds = std::max<int64_t>(1, (units + 4 * most - 1) / (4 * most));
    return static_cast<unsigned>(std::max<int64_t>(1, (units + 4 * rounds - 1) / (4 * rounds)));
}

}  // namespace

size_t preference_bytes(const muon_preference_args& a) {
    const size_t q = static_cast<size_t>(a.sequences), u = static_cast<size_t>(units_of(a.tokens));
    return (2 * u + q) * sizeof(double2) + (q + q / 2) * sizeof(float);
}

hipError_t launch_preference(const muon_preference_args& a, void* workspace, hipStream_t s) {
    const bool bf = a.dtype == MUON_BF16;
    if (a.tokens <= LS_SMALL && a.sequences <= LS_SMALL_SEQS) {
        if (bf) hipLaunchKernelGGL(preference_one_kernel<uint16_t>, dim3(1), dim3(one_block(a.tokens)), 0, s, a);
        else hipLaunchKernelGGL(preference_one_kernel<float>, dim3(1), dim3(one_block(a.tokens)), 0, s, a);
        return hipGetLastError();
    }
    const size_t q = static_cast<size_t>(a.sequences), u = static_cast<size_t>(units_of(a.tokens));
    double2* f2 = static_cast<double2*>(workspace);
    float* f = reinterpret_cast<float*>(f2 + 2 * u + q);
    const PreferenceState<int64_t> st{a, {a.offsets, static_cast<int>(a.sequences), static_cast<int>(a.tokens)},
                                      {f2, f2 + u, f2 + 2 * u}, f, f + q};
    auto launch = [&](auto kernel, unsigned grid) {
        hipLaunchKernelGGL(kernel, dim3(grid), dim3(LS_THREADS), 0, s, st);
        return hipGetLastError();
    };
    const unsigned grid = grid_for(u, LS_GRID);
    hipError_t e = launch(bf ? preference_kernel<uint16_t, PF_UNITS> : preference_kernel<float, PF_UNITS>, grid);
    if (e == hipSuccess) e = launch(preference_kernel<float, PF_PAIRS>, grid_for((a.sequences / 2 + 63) / 64, LS_GRID));
    if (e == hipSuccess)
        e = launch(bf ? preference_kernel<uint16_t, PF_GRAD> : preference_kernel<float, PF_GRAD>, a.grad_logp ? grid + 1 : 1);
    return e;
}

size_t policy_bytes(const muon_policy_args& a) {
    const size_t q = static_cast<size_t>(a.sequences), u = static_cast<size_t>(units_of(a.tokens));
    return PL_SUMS * LS_GRID * sizeof(double) + (2 * u + q + LS_COUNTS) * sizeof(float);
}

hipError_t launch_policy(const muon_policy_args& a, void* workspace, hipStream_t s) {
    const bool bf = a.dtype == MUON_BF16;
    if (a.tokens <= LS_SMALL && a.sequences <= LS_SMALL_SEQS) {
        if (bf) hipLaunchKernelGGL(policy_one_kernel<uint16_t>, dim3(1), dim3(one_block(a.tokens)), 0, s, a);
        else hipLaunchKernelGGL(policy_one_kernel<float>, dim3(1), dim3(one_block(a.tokens)), 0, s, a);
        return hipGetLastError();
    }
    const size_t q = static_cast<size_t>(a.sequences), u = static_cast<size_t>(units_of(a.tokens));
    double* sums = static_cast<double*>(workspace);
    float* f = reinterpret_cast<float*>(sums + PL_SUMS * LS_GRID);
    float* counts = f + 2 * u + q;
    PolicyState<int64_t> st{a, {a.offsets, static_cast<int>(a.sequences), static_cast<int>(a.tokens)}, {f, f + u, f + 2 * u}};
    hipError_t e = hipSuccess;
    int parts = 0;
    if (a.mask) {
        // by sequence every unit has work that waits; counting alone is a byte a token
        parts = static_cast<int>(grid_for(u, a.reduction == MUON_REDUCE_SEQUENCE ? LS_GRID : LS_COUNTS));
        hipLaunchKernelGGL(policy_counts_kernel, dim3(parts), dim3(LS_THREADS), 0, s, st, counts);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
        st.joined = a.reduction == MUON_REDUCE_SEQUENCE && static_cast<int64_t>(u) > LS_JOIN;
        if (st.joined) {
            hipLaunchKernelGGL(policy_join_kernel, dim3(grid_for((a.sequences + 63) / 64, LS_GRID)), dim3(LS_THREADS), 0, s, st);
            e = hipGetLastError();
            if (e != hipSuccess) return e;
        }
    }
    const unsigned grid = grid_for(u, LS_GRID);
    if (bf) hipLaunchKernelGGL(policy_main_kernel<uint16_t>, dim3(grid), dim3(LS_THREADS), 0, s, st, counts, parts, sums);
    else hipLaunchKernelGGL(policy_main_kernel<float>, dim3(grid), dim3(LS_THREADS), 0, s, st, counts, parts, sums);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(policy_final_kernel, dim3(1), dim3(LS_THREADS), 0, s, a, sums, static_cast<int>(grid));
    return hipGetLastError();
}

}  // namespace muon
