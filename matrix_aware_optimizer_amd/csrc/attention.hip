// Attention over packed sequences, forward and backward (formulas: muon.h), on the matrix cores.
//
// Forward and grad_q: a workgroup of 4 waves takes 128 queries of one head, a wave 32 of them, and walks over the keys a tile
// at a time.  The scores are formed transposed, S^T = K Q^T: a lane then holds one query's scores, so the softmax's maximum and
// sum are a lane's own business but for one exchange with lane l ^ 32, a rescale is a factor a lane, and the
// probabilities are at once the operand of O^T = V^T P^T (attention_tile.h).
// grad_k and grad_v: a workgroup takes 128 keys of one key head, a wave 32 of them, and walks over the queries of every head that
// shares it; S = Q K^T comes out with one key a lane, ready for dV^T = dO^T P and dK^T = Q^T dS.  Two kernels form the
// scores twice (7 products where one kernel would need 5), but no sum is shared between workgroups: no atomics, the
// same bits on every run, and shared key heads add up in registers.
//
// Both tiles of a walk are double-buffered in LDS; a step's loads are issued before the step before it is computed, with
// one barrier a step.  Two workgroups run on a CU in bf16, but one of grad_q where a bias meets heads wider than 64 (LDS) and one of what makes
// all gradients at once; in fp32 one, two of the forward and grad_q kernels up to 64 wide.
//
// Measured (16384 tokens, causal, 16 heads of 128 over 4, bf16): forward 1.45 to 1.54 ms, 710 to 760 TFLOP/s by the operator's own count; grad_q 2.0
// to 2.1 ms and grad_k with grad_v 3.1 to 3.4 ms, 770 to 830 and 650 to 710 by the three and four products that they form, second parts not counted.  The matrix cores are busy 60, 59 and 53 % of the time, half
// of it or a third with the second parts of probabilities and dz, and the vector units 58, 50 and 44 %: a lane's exponentials, maxima and
// roundings take about as long as its products, and of two waves a SIMD the one's products cover only part of the other's.
#include <algorithm>
#include <numeric>

#include "attention_tile.h"

namespace muon {

namespace {

using namespace at;

constexpr int AT_THREADS = 256, AT_WAVES = 4, AT_SHIFT = 7, AT_ROWS = 1 << AT_SHIFT;   // rows (queries or keys) a workgroup
constexpr int AT_MAX_SPLITS = 64;
constexpr int AT_FINISH = 1024;                                 // threads of the sums' workgroups
constexpr int64_t AT_CUS = 256;
// The bias's slots are added up a distance at a time in a launch of its own, and buckets from those sums, where there are more slots or more
// distances a bucket; else by bucket at once.  Both passes, bf16, at once and in two: 8192 tokens, 16 heads of 64, 304 slots 349 and 346 us, reach 1024
// 398 and 382; 2 sequences, 8 heads, reach 4096 960 and 912; 77 tokens, 8 heads 29.0 and 29.8, 512 tokens 47.6 and 50.4, 4 x 512
// tokens 104.1 and 105.1.  With 75 distances a bucket (300 queries over 900 keys) 51.9 and 50.1, with 32 (2 x 512 tokens) 80.2 and 82.0.
constexpr int64_t AT_FEW_SLOTS = 256, AT_FEW_DISTANCES = 64;
// Slots take 4 (2 reach + 1) bytes a wave and head.  Where those of all units pass this many bytes (4000 sequences of 40 tokens, 16 heads, reach
// 1024: 2.8 GB, both passes 5.25 ms in one go and 5.38 so), grad_q goes over the units in batches, and each batch's slots are added to the
// distances' sums before the next.
constexpr int64_t AT_SLOT_BYTES = int64_t{1} << 29;

// fp32 products take 16 times as long as bf16's: steps and blocks of columns that a narrow head does not have are left out (72 of
// 128: 4 of 11 of a tile's products).
template <typename T> __device__ __forceinline__ bool beyond(int column, int width) { return sizeof(T) == 4 && column >= width; }

// Rows of a walked tile: of keys, and of queries for grad_k and grad_v.
template <typename T> constexpr int walk_rows() { return sizeof(T) == 2 ? 64 : 32; }
constexpr int KV_ROWS = 32;

struct Common {
    muon_attention_args a;
    float* lse_low;       // queries x heads, or NULL
    int64_t unit0;        // first unit of this launch
    int64_t units;        // of the whole call: units of an axis x heads x splits
    int64_t q_axis, q_stride, k_axis, k_stride;   // units of the two axes, and the stride through them
    int splits;
    int window;           // 0: none
    int gqa;              // heads / kv_heads
    int pack;             // the heads of a workgroup's rows: 2^pack heads that share a key head, row by row for each query (forward)
};
struct ForwardArgs {
    Common c;
    float* part;          // splits > 1: out before its division, [split][query][head][width], then maximum and sum, [split][query][head]
};
struct BackwardArgs {
    Common c;             // c.a.out, out_low: the forward call's
    const void* grad_out;
    void* grad_q;
    void* grad_k;
    void* grad_v;
    int64_t ld_do, hs_do, ld_dq, hs_dq, ld_dk, hs_dk, ld_dv, hs_dv;
    float* delta;         // query x head; NULL where one launch does all
    int q_splits, kv_splits;
    float* q_part;        // splits > 1: sums of each split
    float* kv_part;
    float* bias_part;     // [head][slot][2 reach + 1], a slot per wave of a batch of units
    int64_t slots;
    int64_t first_unit;   // of the batch
    int64_t q_blocks;     // one launch for all: its first blocks make grad_q
};

// Which unit of the axis, head and split a workgroup has.  Heads go fastest, and where they allow it in runs that share an XCD
// (workgroups go to XCDs in turn), so that a key head's rows stay in one L2.
// stride: how to go through the units (unit_stride).  Returns the unit's turn on that way.
__device__ __forceinline__ int64_t decode(int64_t id, int heads, int splits, int64_t axis, int64_t stride, int& u, int& head, int& split) {
    const int hs = heads * splits;
    const int64_t r = id / hs;
    u = static_cast<int>(stride == 1 ? r : r * stride % axis);
    int k = static_cast<int>(id - r * hs);
    if (hs % 8 == 0) k = (k % 8) * (hs / 8) + k / 8;
    head = k / splits;
    split = k - head * splits;
    return r;
}

// A negative scale goes into the sign of one factor of the scores and a scale of 0 into its values: then a score that is hidden, at
// -infinity, stays there under the (positive) factor that remains.
template <typename T> __device__ __forceinline__ void negate(Frag<T>& f) {
    if constexpr (sizeof(T) == 2) f.w ^= 0x80008000u;
    else { f.w[0] = -f.w[0]; f.w[1] = -f.w[1]; }
}
__device__ __forceinline__ float size_of(float scale) { return scale == 0.0f ? 1.0f : fabsf(scale); }

// A row's lse in two parts, L = hi + low, from its reference m (natural units with a bias, else powers of two) and the sum l of its terms.
// Whole powers of two of l are added as they are, so that the logarithm is one between sqrt(1/2) and sqrt(2), within 2^-24.
template <bool BIAS> __device__ __forceinline__ void store_lse(const Common& c, int64_t at, float m, float l) {
    float hi = NEG_INF, low = 0.0f;
    if (l != 0.0f) {
        float x = __builtin_amdgcn_frexp_mantf(l);
        int e = __builtin_amdgcn_frexp_expf(l);
        if (x < 0.70710678f) {
            x *= 2.0f;
            --e;
        }
        const double n = LN2_64 * (static_cast<double>(e) + static_cast<double>(__builtin_amdgcn_logf(x))), at_m = BIAS ? m : LN2_64 * m;
        hi = static_cast<float>(at_m + n);
        low = fabsf(hi) < -NEG_INF ? static_cast<float>((at_m - hi) + n) : 0.0f;      // a low m takes all of n out of their sum
    }
    G(c.a.lse)[at] = hi;
    if (c.lse_low) G(c.lse_low)[at] = low;
}
// What a row's probabilities are formed again with: p = 2^low2 exp(score - ref), the score times log2 e in `ref`'s place and a power of two
// where there is no bias.  low2 is what lse and its product with log2 e lose in 32 bits: without it a row's probabilities would all be
// off by up to |lse| 2^-23, and with a bias so low that the logarithm of the sum is lost in lse by a factor of the keys' number.
struct RowRef {
    float ref, low2;
    template <bool BIAS> __device__ __forceinline__ void set(float lse, float low) {
        ref = BIAS ? lse : lse * LOG2E;
        low2 = -LOG2E * low - (BIAS ? 0.0f : fmaf(lse, LOG2E, -ref) + lse * LOG2E_LOW);
    }
};

// Bias of a head at distance j - a.
template <typename T> __device__ __forceinline__ int bucket_at(const muon_attention_args& a, int dist) {
    const int r = a.reach, d = dist < -r ? -r : dist > r ? r : dist;
    return G(a.bucket_map)[d + r];
}
template <typename T> __device__ __forceinline__ float bias_value(const muon_attention_args& a, int bucket, int head) {
    const bool ok = static_cast<unsigned>(bucket) < static_cast<unsigned>(a.buckets);
    return ok ? ld_el<T>(static_cast<const T*>(a.bias), static_cast<size_t>(bucket) * a.heads + head) : 0.0f;
}

// Bias over the distances between a tile of rows and one of keys, a buffer of it a tile.  The bucket of the tile after next
// and the value of the next one are under way while a tile is computed.
template <typename T, int N> struct BiasWindow {
    static_assert(N <= AT_THREADS, "one distance a thread");
    int bucket = 0;
    float value = 0.0f;
    __device__ __forceinline__ void ask(const muon_attention_args& a, int first) { if (static_cast<int>(threadIdx.x) < N) bucket = bucket_at<T>(a, first + static_cast<int>(threadIdx.x)); }
    __device__ __forceinline__ void fetch(const muon_attention_args& a, int head) { if (static_cast<int>(threadIdx.x) < N) value = bias_value<T>(a, bucket, head); }
    __device__ __forceinline__ void put(lds_float_t* buf) const { if (static_cast<int>(threadIdx.x) < N) buf[threadIdx.x] = value; }
};

// Keys that a lane's query sees are lo .. lo + span - 1; how a wave's 32 queries stand to a tile of keys.
struct Sight {
    int lo;
    unsigned span;
    __device__ __forceinline__ void set(int l, int h) { lo = l; span = h > l ? h - l : 0; }
};
enum { NOTHING = 0, SOME = 1, ALL = 2 };
// Queries at key positions a0 .. a1, keys j0 .. j1, all of them within the sequence or less than a tile behind it.  Positions and window
// reach 2^30: their differences stay within 32 bits, a sum of the two does not.
__device__ __forceinline__ int tile_sight(int a0, int a1, int j0, int j1, bool causal, int window) {
    if (causal && j0 > a1) return NOTHING;
    if (window && (j1 - a0 <= -window || j0 - a1 >= window)) return NOTHING;
    if (causal && j1 > a0) return SOME;
    if (window && (j0 - a1 <= -window || j1 - a0 >= window)) return SOME;
    return ALL;
}
// Scores outside a lane's sight to -infinity: register i stands for place at + 8 (i / 4) + i % 4 (4 h is in `at`); bits: the
// key mask of those places.
__device__ __forceinline__ void hide(f32x16_t& s, const Sight& v, int at) {
    const int t = at - v.lo;
#pragma unroll
    for (int i = 0; i < 16; ++i) s[i] = static_cast<unsigned>(t + 8 * (i >> 2) + (i & 3)) < v.span ? s[i] : NEG_INF;
}
__device__ __forceinline__ void hide_masked(f32x16_t& s, uint32_t bits) {
#pragma unroll
    for (int i = 0; i < 16; ++i) s[i] = (bits >> (8 * (i >> 2) + (i & 3))) & 1u ? s[i] : NEG_INF;
}

// Walk of a wave's 32 queries over tiles of keys: what the forward and the grad_q kernel share.
template <typename T, int DP> struct KeyWalk {
    static constexpr int BN = walk_rows<T>(), NB = BN / 32, KS = DP / 16;
    static constexpr int TILE = BN * Row<T, DP>::BYTES;
    static constexpr int WIN = AT_ROWS + BN;          // distances between 128 queries and a tile of keys (one to spare)
    const muon_attention_args& a;
    Span sp;
    int head, pack, wave_at;                          // (first) head, this wave's first query in its sequence
    int off;                                          // key position of query 0
    int first, last;                                  // tiles
    const T* kbase;
    const T* vbase;

    __device__ __forceinline__ KeyWalk(const Common& c, const Span& s, int h, int split, int splits, int p) : a(c.a), sp(s), head(h), pack(p) {
        wave_at = sp.at + (32 * wave_id() >> pack);
        off = sp.other_len - sp.len;
        const int a0 = sp.at + off, a1 = sp.at + min(sp.rows, AT_ROWS >> pack) - 1 + off;
        int lo = 0, hi = sp.other_len;
        if (a.causal) hi = min(hi, a1 + 1);
        if (c.window) { lo = max(lo, a0 - c.window + 1); hi = min(hi, a1 + c.window); }
        const int t0 = lo / BN, n = hi > lo ? (hi + BN - 1) / BN - t0 : 0;
        first = t0 + static_cast<int>(static_cast<int64_t>(n) * split / splits);
        last = t0 + static_cast<int>(static_cast<int64_t>(n) * (split + 1) / splits);
        const int kv = head / c.gqa;
        kbase = static_cast<const T*>(a.k) + static_cast<int64_t>(sp.other) * a.ld_k + static_cast<int64_t>(kv) * a.hs_k;
        vbase = static_cast<const T*>(a.v) + static_cast<int64_t>(sp.other) * a.ld_v + static_cast<int64_t>(kv) * a.hs_v;
    }
    // What this lane's key of tile t is worth: its mask byte.
    __device__ __forceinline__ unsigned key_byte(int t) const {
        const int j = t * BN + static_cast<int>(threadIdx.x & 63);
        const bool in = j < sp.other_len && static_cast<int>(threadIdx.x & 63) < BN;
        return in ? (a.key_mask ? G(a.key_mask)[sp.other + j] : 1u) : 0u;
    }
    __device__ __forceinline__ void load(int t, lds_byte_t* k, lds_byte_t* v, uint64_t live) const {
        const int64_t j = static_cast<int64_t>(t) * BN;
        load_tile<T, DP, BN, AT_THREADS>(k, kbase + j * a.ld_k, a.ld_k, a.width, live);
        load_tile<T, DP, BN, AT_THREADS>(v, vbase + j * a.ld_v, a.ld_v, a.width, live);
    }
    __device__ __forceinline__ Sight sight(const Common& c, int at) const {      // of the query at place `at`
        const int p = min(at, sp.len - 1) + off;
        int lo = 0, hi = sp.other_len;
        if (a.causal) hi = min(hi, p + 1);
        if (c.window) { lo = max(lo, p - c.window + 1); hi = min(hi, p + c.window); }
        Sight s;
        s.set(lo, at < sp.len ? hi : lo);
        return s;
    }
    // Scores of tile t (raw products) with what the wave sees of it; false if nothing.
    __device__ __forceinline__ int seen(const Common& c, int t, uint64_t live) const {
        const int j0 = t * BN, a0 = wave_at + off, a1 = a0 + (31 >> pack);
        constexpr uint64_t full = BN == 64 ? ~0ull : (1ull << (BN & 63)) - 1;
        const int s = wave_at >= sp.len ? NOTHING : tile_sight(a0, a1, j0, j0 + BN - 1, a.causal, c.window);
        return s == ALL && live != full ? SOME : s;
    }
    // Distance of the window's first entry for tile t.
    __device__ __forceinline__ int window_first(int t) const { return t * BN - (sp.at + AT_ROWS - 1 + off); }
    // z = scale x + bias (natural units) for one block; w: the tile's window; near == 0: `far` everywhere.
    __device__ __forceinline__ void add_bias(f32x16_t& s, float scale, const lds_float_t* w, bool near, float far, int nb) const {
        const int lane = threadIdx.x & 63;
        if (near) {
            // entry of key 32 nb + 8 (i / 4) + 4 h + i % 4 and query 32 wave + l % 32
            const lds_float_t* p = w + (AT_ROWS - 1 - 32 * wave_id() - (lane & 31)) + 32 * nb + 4 * (lane >> 5);
#pragma unroll
            for (int i = 0; i < 16; ++i) s[i] = fmaf(s[i], scale, p[8 * (i >> 2) + (i & 3)]);
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) s[i] = fmaf(s[i], scale, far);
        }
    }
    // Is the bias one value over this wave's part of tile t?  -1 / 1: the one below / above, 0: no.
    __device__ __forceinline__ int far(int t) const {
        const int j0 = t * BN, a0 = wave_at + off;
        if (j0 + BN - 1 - a0 <= -a.reach) return -1;
        return j0 - (a0 + 31) >= a.reach ? 1 : 0;
    }
};

// ---- forward --------------------------------------------------------------------

template <typename T, int DP, bool BIAS>
__global__ __launch_bounds__(AT_THREADS, sizeof(T) == 2 ? 2 : 1) void attention_forward_kernel(ForwardArgs f) {
    typedef KeyWalk<T, DP> W;
    constexpr int NB = W::NB, KS = W::KS, DB = DP / 32;
    __shared__ __attribute__((aligned(512))) u32x4_t lds[4 * W::TILE / 16];
    __shared__ float win[BIAS ? 2 * W::WIN : 1];
    const Common& c = f.c;
    const muon_attention_args& a = c.a;
    int u, head, split;
    decode(c.unit0 + blockIdx.x, a.heads >> c.pack, c.splits, c.q_axis, c.q_stride, u, head, split);
    head <<= c.pack;
    Span sp;
    if (!find_span<false>(AT_SHIFT - c.pack, a.offsets, a.key_offsets, static_cast<int>(a.sequences), static_cast<int>(a.queries), static_cast<int>(a.keys), a.causal, u, sp)) return;
    const W w(c, sp, head, split, c.splits, c.pack);
    const int lane = threadIdx.x & 63, place = w.wave_at + ((lane & 31) >> c.pack), own = head + (lane & ((1 << c.pack) - 1));   // this lane's query and head
    const bool row_ok = place < sp.len;
    const int64_t row = sp.start - sp.at + place;
    const Sight sight = w.sight(c, place);
    lds_byte_t* buf = (lds_byte_t*)lds;
    Lanes<T, DP> lanes;
    lds_float_t* wbuf = (lds_float_t*)win;

    Frag<T> qf[KS];
    {
        const T* q = static_cast<const T*>(a.q) + row * a.ld_q + static_cast<int64_t>(own) * a.hs_q;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            qf[ks] = global_frag<T>(q, 16 * ks + 8 * (lane >> 5), a.width, row_ok && a.scale != 0.0f);
            if (a.scale < 0.0f) negate<T>(qf[ks]);
        }
    }
    const float scale = size_of(a.scale), unit = BIAS ? LOG2E : scale * LOG2E;     // from what s holds to powers of two
    const float slack = 8.0f / LOG2E * (BIAS ? 1.0f : LOG2E);                    // 8 powers of two, in m's units

    f32x16_t o[DB] = {};
    float m = NEG_INF, l = 0.0f;      // BIAS: natural units, else powers of two; l: this lane's half of the row
    BiasWindow<T, W::WIN> bw;
    float far_lo = 0.0f, far_hi = 0.0f;
    unsigned byte = 0;
    uint64_t live = 0, next = 0;
    if (w.first < w.last) {
        // loads come back in order: what others wait for goes first
        const unsigned first_byte = w.key_byte(w.first);
        byte = w.key_byte(w.first + 1);
        int lo_bucket = 0, hi_bucket = 0;
        if constexpr (BIAS) {
            bw.ask(a, w.window_first(w.first));
            lo_bucket = bucket_at<T>(a, -a.reach);
            hi_bucket = bucket_at<T>(a, a.reach);
        }
        next = __ballot(first_byte != 0);
        if constexpr (BIAS) {
            bw.fetch(a, head);
            far_lo = bias_value<T>(a, lo_bucket, head);
            far_hi = bias_value<T>(a, hi_bucket, head);
            bw.ask(a, w.window_first(w.first + 1));
        }
        w.load(w.first, buf, buf + W::TILE, next);
        if constexpr (BIAS) bw.put(wbuf);
    }
    for (int t = w.first; t < w.last; ++t) {
        const int b = (t - w.first) & 1;
        tile_barrier();
        live = next;
        if (t + 1 < w.last) {
            next = __ballot(byte != 0);
            w.load(t + 1, buf + 2 * W::TILE * (b ^ 1), buf + 2 * W::TILE * (b ^ 1) + W::TILE, next);
            byte = w.key_byte(t + 2);
            if constexpr (BIAS) {
                bw.fetch(a, head);
                bw.ask(a, w.window_first(t + 2));
            }
        }
        const int seen = w.seen(c, t, live);
        if (seen != NOTHING) {
            const unsigned kt = lds_at(buf) + 2 * W::TILE * b, vt = kt + W::TILE;
            lanes.fresh();
            f32x16_t s[NB] = {};
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
                if (!beyond<T>(16 * ks, a.width))
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb) mma(s[nb], row_frag<T, DP>(kt, lanes, 32 * nb, ks), qf[ks]);
            if constexpr (BIAS) {
                const int far = w.far(t);
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) w.add_bias(s[nb], scale, wbuf + b * W::WIN, far == 0, far < 0 ? far_lo : far_hi, nb);
            }
            if (seen == SOME) {
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) {
                    hide(s[nb], sight, t * W::BN + 32 * nb + 4 * (lane >> 5));
                    if (a.key_mask) hide_masked(s[nb], static_cast<uint32_t>(live >> (32 * nb + 4 * (lane >> 5))));
                }
            }
            float top = NEG_INF;
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int i = 0; i < 16; ++i) top = fmaxf(top, s[nb][i]);
            top = half_max(top);
            if constexpr (!BIAS) top *= unit;
            // The reference goes 2^8 above the maximum and moves only when that passes it: the terms stay at or below 1, and most
            // tiles need no rescale.
            if (__any(top > m)) {
                const float r = top > m ? top + slack : m;
                const float f2 = r == m ? 1.0f : exp2_((m - r) * (BIAS ? LOG2E : 1.0f));
                m = r;
                l *= f2;
#pragma unroll
                for (int db = 0; db < DB; ++db) o[db] *= f2;
            }
            const float ref = m == NEG_INF ? 0.0f : m;
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    s[nb][i] = BIAS ? exp2_((s[nb][i] - ref) * unit) : exp2_(fmaf(s[nb][i], unit, -ref));
                    l += s[nb][i];
                }
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    const Parts<T> p(s[nb], g);
#pragma unroll
                    for (int db = 0; db < DB; ++db)
                        if (!beyond<T>(32 * db, a.width)) p.mma_to(o[db], col_frag<T, DP>(vt, lanes, 32 * nb + 16 * g, db));
                }
        }
        if constexpr (BIAS)
            if (t + 1 < w.last) bw.put(wbuf + (b ^ 1) * W::WIN);
    }
    l = half_sum(l);
    if (!row_ok) return;
    if (c.splits > 1) {
        const int64_t at = row * a.heads + own, n = a.queries * a.heads;
        float* o_part = f.part + (split * n + at) * a.width;
        float* ml = f.part + c.splits * n * a.width + (split * n + at) * 2;
        store_rows<float>(o, 1.0f, o_part, static_cast<float*>(nullptr), a.width);
        if (lane < 32) {
            G(ml)[0] = m;
            G(ml)[1] = l;
        }
        return;
    }
    T* out = static_cast<T*>(a.out) + row * a.ld_out + static_cast<int64_t>(own) * a.hs_out;
    T* low = a.out_low ? static_cast<T*>(a.out_low) + row * a.ld_out_low + static_cast<int64_t>(own) * a.hs_out_low : nullptr;
    store_rows<T>(o, l == 0.0f ? 0.0f : 1.0f / l, out, low, a.width);
    if (lane < 32) store_lse<BIAS>(c, row * a.heads + own, m, l);
}

// Joins the splits of a row: a wave each.
template <typename T, bool BIAS> __global__ __launch_bounds__(256) void attention_join_kernel(ForwardArgs f, int64_t row0) {
    const Common& c = f.c;
    const muon_attention_args& a = c.a;
    const int64_t n = a.queries * a.heads, at = row0 + static_cast<int64_t>(blockIdx.x) * 4 + wave_id();
    if (at >= n) return;
    const int lane = threadIdx.x & 63;
    const float* ml = f.part + c.splits * n * a.width;
    float m = NEG_INF, l = 0.0f;
    if (lane < c.splits) {
        m = G(ml)[(lane * n + at) * 2];
        l = G(ml)[(lane * n + at) * 2 + 1];
    }
    float top = m;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) top = fmaxf(top, __shfl_xor(top, d));
    const float unit = BIAS ? LOG2E : 1.0f;
    const float f2 = m == top || l == 0.0f ? (l == 0.0f ? 0.0f : 1.0f) : exp2_((m - top) * unit);
    const float sum = wave_sum(l * f2);
    // eight splits' values are asked for before the first is added; a split of no key holds zeros
    float v[2] = {};
    const int d0 = min(lane, a.width - 1), d1 = min(lane + 64, a.width - 1);
    for (int s0 = 0; s0 < c.splits; s0 += 8) {
        float x[8][2];
#pragma unroll
        for (int s = 0; s < 8; ++s) {
            const float* p = f.part + (min(s0 + s, c.splits - 1) * n + at) * a.width;
            x[s][0] = G(p)[d0];
            x[s][1] = G(p)[d1];
        }
#pragma unroll
        for (int s = 0; s < 8; ++s) {
            const float fs = s0 + s < c.splits ? __shfl(f2, s0 + s) : 0.0f;
            v[0] = fmaf(x[s][0], fs, v[0]);
            v[1] = fmaf(x[s][1], fs, v[1]);
        }
    }
    const int64_t row = at / a.heads;
    const int head = static_cast<int>(at - row * a.heads);
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
    for (int k = 0; k < 2; ++k)
        if (lane + 64 * k < a.width) {
            const float x = v[k] * inv;
            st_el<T>(a.out, row * a.ld_out + static_cast<int64_t>(head) * a.hs_out + lane + 64 * k, x);
            if (a.out_low)
                st_el<T>(a.out_low, row * a.ld_out_low + static_cast<int64_t>(head) * a.hs_out_low + lane + 64 * k,
                         sizeof(T) == 2 ? x - bf16_to_f32(f32_to_bf16(x)) : 0.0f);
        }
    if (lane == 0) store_lse<BIAS>(c, at, top, sum);
}

// ---- grad_q, and the bias's gradient --------------------------------------------

// Sums of dz over the distances that a wave meets.  A 32 x 32 block of dz goes to LDS with query q's row moved right by 31 - q, so
// that a distance is a column: lane c adds up column c (what a row does not reach stays 0).  The next block's distances
// begin 32 further on, so 32 sums are complete after a block and go to the wave's slot; the others move down by 32 lanes.  Distances
// beyond the reach have one bucket a side and add up in registers.  The order of the additions is fixed.  (Adding to LDS
// by its float atomics: 363 us for grad_q at 8192 x 16 x 64, 135 so.)
struct BiasSums {
    static constexpr int ROWS = 32 * 64, ROOM = ROWS + 32;   // floats a wave
    lds_float_t* room;       // [query][64], and a place that is never read
    lds_float_t* mine;       // where this lane's part of a block goes
    float* slot;             // 2 reach + 1
    int reach, begin, next;  // distances written to the slot: begin .. next - 1
    bool any;
    float carry, below, above;
    __device__ __forceinline__ void start(lds_float_t* p, float* s, int r) {
        room = p;
        slot = s;
        reach = r;
        begin = next = 0;
        any = false;
        carry = below = above = 0.0f;
        for (int i = 0; i < 32; ++i) room[64 * i + (threadIdx.x & 63)] = 0.0f;
    }
    // A query that sees nothing, or a place behind the last one, stays out of the sums: its part of a block may hold anything (a bias of no pair).
    __device__ __forceinline__ void set_row(bool ok) {
        const int lane = threadIdx.x & 63, q = lane & 31;
        mine = room + (ok ? 64 * q + 31 - q + 4 * (lane >> 5) : ROWS);
    }
    // lanes 0 .. 31 hold the sums of distances next ..
    __device__ __forceinline__ void flush(float v) {
        const int lane = threadIdx.x & 63, dist = next + lane;
        if (lane < 32) {
            if (dist <= -reach) below += v;
            else if (dist >= reach) above += v;
            else G(slot)[dist + reach] = v;
        }
        next += 32;
    }
    // one block of dz; dist: the distance of its first key from its last query
    __device__ __forceinline__ void add(const f32x16_t& dz, int dist) {
        const int lane = threadIdx.x & 63;
        if (!any) {
            any = true;
            begin = next = dist;
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) mine[8 * (i >> 2) + (i & 3)] = dz[i];
        // a wave's LDS accesses come in order; the compiler has to leave them so, since lanes read what others wrote
        asm volatile("" ::: "memory");
        float v[4] = {};
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i & 3] += room[64 * i + lane];
        asm volatile("" ::: "memory");
        const float sum = (v[0] + v[1]) + (v[2] + v[3]) + carry;
        flush(sum);
        const float up = __shfl_xor(sum, 32);
        carry = lane < 32 ? up : 0.0f;
    }
    __device__ __forceinline__ void finish() {
        if (any) flush(carry);
        const int lane = threadIdx.x & 63;
        for (int i = 1 + lane; i < 2 * reach; i += 64)
            if (!any || i - reach < begin || i - reach >= next) G(slot)[i] = 0.0f;
        below = wave_sum(below);
        above = wave_sum(above);
        if (lane == 0) {
            if (reach == 0) {
                G(slot)[0] = below + above;
            } else {
                G(slot)[0] = below;
                G(slot)[2 * reach] = above;
            }
        }
    }
};

// LDS of a workgroup: the tiles, then the bias's windows and rooms.
template <typename T, int DP, bool BIAS> constexpr int grad_q_lds() {
    return 4 * KeyWalk<T, DP>::TILE + (BIAS ? (2 * KeyWalk<T, DP>::WIN + AT_WAVES * BiasSums::ROOM) * 4 : 0);
}

template <typename T, int DP, bool BIAS> __device__ __forceinline__ void grad_q_block(const BackwardArgs& f, int64_t block, lds_byte_t* buf) {
    typedef KeyWalk<T, DP> W;
    constexpr int NB = W::NB, KS = W::KS, DB = DP / 32;
    const Common& c = f.c;
    const muon_attention_args& a = c.a;
    int u, head, split;
    const int64_t turn = decode(block, a.heads, f.q_splits, c.q_axis, c.q_stride, u, head, split);
    lds_float_t* wbuf = (lds_float_t*)(buf + 4 * W::TILE);
    BiasSums sums;
    if constexpr (BIAS) {
        const int64_t slot = head * f.slots + ((turn - f.first_unit) * f.q_splits + split) * AT_WAVES + wave_id();
        sums.start(wbuf + 2 * W::WIN + BiasSums::ROOM * wave_id(), f.bias_part + slot * (2 * a.reach + 1), a.reach);
    }
    Span sp;
    if (!find_span<false>(AT_SHIFT, a.offsets, a.key_offsets, static_cast<int>(a.sequences), static_cast<int>(a.queries), static_cast<int>(a.keys), a.causal, u, sp)) {
        if constexpr (BIAS) sums.finish();
        return;
    }
    const W w(c, sp, head, split, f.q_splits, 0);
    const int lane = threadIdx.x & 63, place = w.wave_at + (lane & 31);
    const int64_t row = sp.start - sp.at + place;
    const Sight sight = w.sight(c, place);
    Lanes<T, DP> lanes;

    // a query that sees no key takes no part, whatever its rows hold
    const bool in = place < sp.len;
    const int64_t stat = in ? row * a.heads + head : 0;
    const float lse_there = G(a.lse)[stat], low_there = G(c.lse_low ? c.lse_low : a.lse)[stat];      // both at once, with no branch between
    const float lse = in ? lse_there : NEG_INF;
    const bool row_ok = lse != NEG_INF;
    if constexpr (BIAS) sums.set_row(row_ok);
    const float lse_low = c.lse_low && row_ok ? low_there : 0.0f;
    Frag<T> qf[KS], df[KS];
    float delta = 0.0f;
    {
        const int h = lane >> 5;
        const T* q = static_cast<const T*>(a.q) + row * a.ld_q + static_cast<int64_t>(head) * a.hs_q;
        const T* d = static_cast<const T*>(f.grad_out) + row * f.ld_do + static_cast<int64_t>(head) * f.hs_do;
        const T* out = static_cast<const T*>(a.out) + row * a.ld_out + static_cast<int64_t>(head) * a.hs_out;
        const T* low = static_cast<const T*>(a.out_low) + row * a.ld_out_low + static_cast<int64_t>(head) * a.hs_out_low;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            const int e0 = 16 * ks + 8 * h;
            qf[ks] = global_frag<T>(q, e0, a.width, row_ok && a.scale != 0.0f);
            if (a.scale < 0.0f) negate<T>(qf[ks]);
            df[ks] = global_frag<T>(d, e0, a.width, row_ok);
            const Frag<T> of = global_frag<T>(out, e0, a.width, row_ok);
#pragma unroll
            for (int e = 0; e < 8; ++e) delta = fmaf(frag_get(df[ks], e), frag_get(of, e), delta);
            if (a.out_low) {
                const Frag<T> lf = global_frag<T>(low, e0, a.width, row_ok);
#pragma unroll
                for (int e = 0; e < 8; ++e) delta = fmaf(frag_get(df[ks], e), frag_get(lf, e), delta);
            }
        }
        delta = half_sum(delta);
        if (f.delta && place < sp.len && lane < 32 && split == 0) G(f.delta)[row * a.heads + head] = delta;
    }
    const float scale = size_of(a.scale), unit = BIAS ? LOG2E : scale * LOG2E;
    // With a bias +infinity, so that p is 0, where nothing is seen: from 89 on a bias alone would make an infinite one.
    RowRef r{BIAS ? -NEG_INF : 0.0f, 0.0f};
    if (row_ok) r.set<BIAS>(lse, lse_low);
    const float ref = r.ref, norm = exp2_(r.low2), delta_norm = delta * norm;

    f32x16_t o[DB] = {};
    BiasWindow<T, W::WIN> bw;
    float far_lo = 0.0f, far_hi = 0.0f;
    unsigned byte = 0;
    uint64_t live = 0, next = 0;
    if (w.first < w.last) {
        // loads come back in order: what others wait for goes first
        const unsigned first_byte = w.key_byte(w.first);
        byte = w.key_byte(w.first + 1);
        int lo_bucket = 0, hi_bucket = 0;
        if constexpr (BIAS) {
            bw.ask(a, w.window_first(w.first));
            lo_bucket = bucket_at<T>(a, -a.reach);
            hi_bucket = bucket_at<T>(a, a.reach);
        }
        next = __ballot(first_byte != 0);
        if constexpr (BIAS) {
            bw.fetch(a, head);
            far_lo = bias_value<T>(a, lo_bucket, head);
            far_hi = bias_value<T>(a, hi_bucket, head);
            bw.ask(a, w.window_first(w.first + 1));
        }
        w.load(w.first, buf, buf + W::TILE, next);
        if constexpr (BIAS) bw.put(wbuf);
    }
    for (int t = w.first; t < w.last; ++t) {
        const int b = (t - w.first) & 1;
        tile_barrier();
        live = next;
        if (t + 1 < w.last) {
            next = __ballot(byte != 0);
            w.load(t + 1, buf + 2 * W::TILE * (b ^ 1), buf + 2 * W::TILE * (b ^ 1) + W::TILE, next);
            byte = w.key_byte(t + 2);
            if constexpr (BIAS) {
                bw.fetch(a, head);
                bw.ask(a, w.window_first(t + 2));
            }
        }
        const int seen = w.seen(c, t, live);
        if (seen != NOTHING) {
            const unsigned kt = lds_at(buf) + 2 * W::TILE * b;
            const int far = BIAS ? w.far(t) : 0;
            // a block of 32 keys at a time: all of a tile at once does not fit the registers of two waves a SIMD
#pragma unroll DP == 64 ? NB : 1
            for (int nb = 0; nb < NB; ++nb) {
                const unsigned kb = kt + 32 * nb * Row<T, DP>::BYTES, vb = kb + W::TILE;
                lanes.fresh();
                f32x16_t s = {}, dp = {};
#pragma unroll
                for (int ks = 0; ks < KS; ++ks)
                    if (!beyond<T>(16 * ks, a.width)) {
                        mma(s, row_frag<T, DP>(kb, lanes, 0, ks), qf[ks]);
                        mma(dp, row_frag<T, DP>(vb, lanes, 0, ks), df[ks]);
                    }
                if constexpr (BIAS) w.add_bias(s, scale, wbuf + b * W::WIN, far == 0, far < 0 ? far_lo : far_hi, nb);
                if (seen == SOME) {
                    hide(s, sight, t * W::BN + 32 * nb + 4 * (lane >> 5));
                    if (a.key_mask) hide_masked(s, static_cast<uint32_t>(live >> (32 * nb + 4 * (lane >> 5))));
                }
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float p = BIAS ? exp2_((s[i] - ref) * unit) : exp2_(fmaf(s[i], unit, -ref));
                    s[i] = p * fmaf(dp[i], norm, -delta_norm);
                }
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    const Parts<T> p(s, g);
#pragma unroll
                    for (int db = 0; db < DB; ++db)
                        if (!beyond<T>(32 * db, a.width)) p.mma_to(o[db], col_frag<T, DP>(kb, lanes, 16 * g, db));
                }
                if constexpr (BIAS) {
                    if (far == 0) {
                        sums.add(s, t * W::BN + 32 * nb - (w.wave_at + 31 + w.off));
                    } else {
                        float v = 0.0f;
#pragma unroll
                        for (int i = 0; i < 16; ++i) v += s[i];
                        v = row_ok ? v : 0.0f;
                        if (far < 0) sums.below += v;
                        else sums.above += v;
                    }
                }
            }
        }
        if constexpr (BIAS)
            if (t + 1 < w.last) bw.put(wbuf + (b ^ 1) * W::WIN);
    }
    if constexpr (BIAS) sums.finish();
    if (place >= sp.len) return;
    if (f.q_splits > 1) {
        const int64_t at = row * a.heads + head, n = a.queries * a.heads;
        store_rows<float>(o, 1.0f, f.q_part + (split * n + at) * a.width, static_cast<float*>(nullptr), a.width);
        return;
    }
    store_rows<T>(o, a.scale, static_cast<T*>(f.grad_q) + row * f.ld_dq + static_cast<int64_t>(head) * f.hs_dq, static_cast<T*>(nullptr), a.width);
}

template <typename T, int DP, bool BIAS>
__global__ __launch_bounds__(AT_THREADS, sizeof(T) == 2 && !(BIAS && DP == 128) ? 2 : 1) void attention_grad_q_kernel(BackwardArgs f) {
    __shared__ __attribute__((aligned(512))) char lds[grad_q_lds<T, DP, BIAS>()];
    grad_q_block<T, DP, BIAS>(f, f.c.unit0 + blockIdx.x, (lds_byte_t*)lds);
}

// ---- grad_k and grad_v ------------------------------------------------------------

// Two waves a SIMD, of workgroups that share no barrier, fill each other's waits.  In bf16 with DP 128 that takes v's fragments out of
// LDS (both accumulators, k's fragments and a block's scores fill 256 registers; 1 is spilled, with a bias 16), and tiles of 32 queries, so that two
// workgroups fit a CU's LDS (8192 tokens, 16 heads of 128: 265 us; one workgroup of 8 waves and tiles of 64 queries 285).
template <typename T, int DP> struct KvShape {
    static constexpr bool V_LDS = sizeof(T) == 2 && DP == 128;
    static constexpr int WAVES = sizeof(T) == 2 ? 2 : 1;      // a SIMD
};

// LDS of a workgroup: the tiles, v, [buffer][ref; low2 (fp32: 2^low2); delta][query], a zero for each query, the bias's windows.
template <typename T, int DP, bool BIAS> constexpr int grad_kv_lds() {
    return (4 * KV_ROWS + (KvShape<T, DP>::V_LDS ? AT_ROWS : 0)) * Row<T, DP>::BYTES + 7 * KV_ROWS * 4 + (BIAS ? 2 * (AT_ROWS + KV_ROWS) * 4 : 0);
}

// SELF: delta is formed here, tile by tile, for a launch that does not wait for grad_q's: a wave takes 8 of a tile's 32 queries,
// 8 lanes a query.
template <typename T, int DP, bool BIAS, bool SELF>
__device__ __forceinline__ void grad_kv_block(const BackwardArgs& f, int64_t block, lds_byte_t* buf) {
    constexpr int BQ = KV_ROWS;
    constexpr int KS = DP / 16, DB = DP / 32, TILE = BQ * Row<T, DP>::BYTES, WIN = AT_ROWS + BQ;
    constexpr bool V_LDS = KvShape<T, DP>::V_LDS;
    constexpr int VTILE = V_LDS ? AT_ROWS * Row<T, DP>::BYTES : 0;
    const Common& c = f.c;
    const muon_attention_args& a = c.a;
    int u, kv, split;
    decode(block, a.kv_heads, f.kv_splits, c.k_axis, c.k_stride, u, kv, split);
    Span sp;
    if (!find_span<true>(AT_SHIFT, a.key_offsets, a.offsets, static_cast<int>(a.sequences), static_cast<int>(a.keys), static_cast<int>(a.queries), a.causal, u, sp)) return;
    const int lane = threadIdx.x & 63, wave = wave_id(), h = lane >> 5;
    const int wave_at = sp.at + 32 * wave, place = wave_at + (lane & 31), nq = sp.other_len, off = sp.len - nq;
    const int64_t row = sp.start - sp.at + place;
    const bool in = place < sp.len, key_ok = in && (!a.key_mask || G(a.key_mask)[in ? row : 0] != 0);
    Lanes<T, DP> lanes;
    lds_float_t* stats = (lds_float_t*)(buf + 4 * TILE + VTILE);
    lds_float_t* zeros = stats + 6 * BQ;
    lds_float_t* wbuf = stats + 7 * BQ;

    // queries that see this lane's key: places lo .. lo + span - 1
    Sight sight;
    {
        int lo = 0, hi = nq;
        const int p = min(place, sp.len - 1) - off;
        if (a.causal) lo = max(lo, p);
        if (c.window) { lo = max(lo, p - c.window + 1); hi = min(hi, p + c.window); }
        sight.set(lo, key_ok ? hi : lo);
    }
    const bool keys_all = __all(key_ok);
    Frag<T> kf[KS], vf[V_LDS ? 1 : KS];
    const unsigned vt = lds_at(buf) + 4 * TILE + 32 * wave * Row<T, DP>::BYTES;
    if constexpr (V_LDS) {
        for (int b = 0; b < AT_ROWS; b += 64) {
            const int j = sp.at + b + lane;
            const int64_t first = sp.start + b;
            const uint64_t live = __ballot(j < sp.len && (!a.key_mask || G(a.key_mask)[j < sp.len ? first + lane : 0] != 0));
            load_tile<T, DP, 64, AT_THREADS>(buf + 4 * TILE + b * Row<T, DP>::BYTES,
                                          static_cast<const T*>(a.v) + first * a.ld_v + static_cast<int64_t>(kv) * a.hs_v, a.ld_v, a.width, live);
        }
    }
    {
        const T* k = static_cast<const T*>(a.k) + row * a.ld_k + static_cast<int64_t>(kv) * a.hs_k;
        const T* v = static_cast<const T*>(a.v) + row * a.ld_v + static_cast<int64_t>(kv) * a.hs_v;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            kf[ks] = global_frag<T>(k, 16 * ks + 8 * h, a.width, key_ok && a.scale != 0.0f);
            if (a.scale < 0.0f) negate<T>(kf[ks]);
            if constexpr (!V_LDS) vf[ks] = global_frag<T>(v, 16 * ks + 8 * h, a.width, key_ok);
        }
    }
    // the walk: tiles first .. first + n - 1 of the queries, for every head that shares this key head
    int lo = 0, hi = nq;
    {
        const int j1 = sp.at + min(sp.rows, AT_ROWS) - 1;
        if (a.causal) lo = max(lo, sp.at - off);
        if (c.window) { lo = max(lo, sp.at - off - c.window + 1); hi = min(hi, j1 - off + c.window); }
    }
    const int first = lo / BQ, n = hi > lo ? (hi + BQ - 1) / BQ - first : 0;
    const int64_t steps = static_cast<int64_t>(n) * c.gqa;
    const int64_t it0 = steps * split / f.kv_splits, it1 = steps * (split + 1) / f.kv_splits;
    struct At {
        int head, t;
        int64_t left;             // steps from here on
    };
    auto after = [&](At w) {
        --w.left;
        if (++w.t == first + n) {
            w.t = first;
            ++w.head;
        }
        return w;
    };
    At now{kv * c.gqa, first, it1 - it0};
    if (it1 > it0) {
        const int g = static_cast<int>(it0 / n);
        now.head += g;
        now.t += static_cast<int>(it0 - static_cast<int64_t>(g) * n);
    }
    Frag<T> own_d[SELF ? DP / 64 : 1], own_o[SELF ? DP / 64 : 1], own_l[SELF ? DP / 64 : 1];
    float own_lse = NEG_INF;
    // lse of this lane's row of a step (and its delta, or what that is formed of): -infinity where there is nothing to see
    auto ask = [&](const At& w, float& l, float& low, float& d) {
        l = NEG_INF;
        low = d = 0.0f;
        if (w.left <= 0) return;
        const int i = w.t * BQ + lane;
        if (lane < BQ && i < nq) {
            const int64_t at = static_cast<int64_t>(sp.other + i) * a.heads + w.head;
            l = G(a.lse)[at];
            if (c.lse_low) low = G(c.lse_low)[at];
            if constexpr (!SELF) d = G(f.delta)[at];
        }
        if constexpr (SELF) {
            const int own = 8 * wave + (lane >> 3);
            const int64_t r = static_cast<int64_t>(sp.other) + w.t * BQ + own, at = r * a.heads + w.head;
            const bool ok = w.t * BQ + own < nq;
            own_lse = G(a.lse)[ok ? at : 0];           // looked at where delta is formed: nothing waits for it here
            if (!ok) own_lse = NEG_INF;
            const T* dr = static_cast<const T*>(f.grad_out) + r * f.ld_do + static_cast<int64_t>(w.head) * f.hs_do;
            const T* outr = static_cast<const T*>(a.out) + r * a.ld_out + static_cast<int64_t>(w.head) * a.hs_out;
            const T* low = static_cast<const T*>(a.out_low) + r * a.ld_out_low + static_cast<int64_t>(w.head) * a.hs_out_low;
#pragma unroll
            for (int k = 0; k < DP / 64; ++k) {
                const int e0 = 64 * k + 8 * (lane & 7);
                own_d[k] = global_frag<T>(dr, e0, a.width, ok);
                own_o[k] = global_frag<T>(outr, e0, a.width, ok);
                if (a.out_low) own_l[k] = global_frag<T>(low, e0, a.width, ok);
            }
        }
    };
    // Loads a step's tiles; returns whether its probabilities take low2.  fp32: a factor for each.  In bf16 it is left out up to an lse of 2^10,
    // where it is below 2^-13; a factor for each, as in fp32, costs 16 products a block and registers that 128 wide does not have (8192
    // tokens, 16 heads: 426 -> 467 us both passes).
    auto load = [&](const At& w, int b, float l, float low, float d) {
        const uint64_t live = __ballot(l != NEG_INF);
        const int64_t i0 = static_cast<int64_t>(sp.other) + static_cast<int64_t>(w.t) * BQ;
        load_tile<T, DP, BQ, AT_THREADS>(buf + 2 * TILE * b, static_cast<const T*>(a.q) + i0 * a.ld_q + static_cast<int64_t>(w.head) * a.hs_q, a.ld_q, a.width, live);
        load_tile<T, DP, BQ, AT_THREADS>(buf + 2 * TILE * b + TILE, static_cast<const T*>(f.grad_out) + i0 * f.ld_do + static_cast<int64_t>(w.head) * f.hs_do, f.ld_do, a.width, live);
        if (wave == 0 && lane < BQ) {
            RowRef r{BIAS ? -NEG_INF : 0.0f, 0.0f};       // as in grad_q_block
            if (l != NEG_INF) r.set<BIAS>(l, low);
            stats[3 * BQ * b + lane] = r.ref;
            stats[3 * BQ * b + BQ + lane] = sizeof(T) == 2 ? r.low2 : exp2_(r.low2);
            if constexpr (!SELF) stats[3 * BQ * b + 2 * BQ + lane] = l == NEG_INF ? 0.0f : d;
        }
        if constexpr (SELF) {
            float v = 0.0f;
#pragma unroll
            for (int k = 0; k < DP / 64; ++k)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    v = fmaf(frag_get(own_d[k], e), frag_get(own_o[k], e), v);
                    if (a.out_low) v = fmaf(frag_get(own_d[k], e), frag_get(own_l[k], e), v);
                }
#pragma unroll
            for (int k = 1; k < 8; k <<= 1) v += __shfl_xor(v, k);
            if ((lane & 7) == 0) stats[3 * BQ * b + 2 * BQ + 8 * wave + (lane >> 3)] = own_lse == NEG_INF ? 0.0f : v;
        }
        if (BIAS && !c.lse_low) return false;
        return (sizeof(T) == 4 ? __any(l != NEG_INF) : __any(l >= 1024.0f || (l <= -1024.0f && l != NEG_INF))) != 0;
    };
    // distance of the window's first entry for tile t: that of this workgroup's first key and the tile's last query
    auto window_first = [&](int t) { return sp.at - (t * BQ + BQ - 1 + off); };

    const float scale = size_of(a.scale), unit = BIAS ? LOG2E : scale * LOG2E;
    f32x16_t dk[DB] = {}, dv[DB] = {};
    BiasWindow<T, WIN> bw;
    float lse = 0.0f, lse_low = 0.0f, delta = 0.0f;
    bool take_low = false, take_low_next = false;
    if (wave == 0 && lane < BQ) zeros[lane] = 0.0f;
    if (now.left > 0) {
        ask(now, lse, lse_low, delta);
        take_low_next = load(now, 0, lse, lse_low, delta);
        ask(after(now), lse, lse_low, delta);
        if constexpr (BIAS) {
            bw.ask(a, window_first(now.t));
            bw.fetch(a, now.head);
            bw.put(wbuf);
            bw.ask(a, window_first(after(now).t));
        }
    }
    int b = 0;
    for (; now.left > 0; now = after(now), b ^= 1) {
        const At next = after(now);
        tile_barrier();
        take_low = take_low_next;
        if (next.left > 0) {
            take_low_next = load(next, b ^ 1, lse, lse_low, delta);
            ask(after(next), lse, lse_low, delta);
            if constexpr (BIAS) {
                bw.fetch(a, next.head);
                bw.ask(a, window_first(after(next).t));
            }
        }
        const unsigned qt = lds_at(buf) + 2 * TILE * b, dt = qt + TILE;
        lanes.fresh();
        const lds_float_t* st = stats + 3 * BQ * b;
        const int i0 = now.t * BQ;
        int seen = wave_at >= sp.len ? NOTHING : tile_sight(i0 + off, i0 + off + 31, wave_at, wave_at + 31, a.causal, c.window);
        if (seen != NOTHING) {
            if (i0 + 31 >= nq || !keys_all) seen = SOME;
            f32x16_t s = {}, dp = {};
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                if (beyond<T>(16 * ks, a.width)) continue;
                mma(s, row_frag<T, DP>(qt, lanes, 0, ks), kf[ks]);
                if constexpr (V_LDS) mma(dp, row_frag<T, DP>(dt, lanes, 0, ks), row_frag<T, DP>(vt, lanes, 0, ks));
                else mma(dp, row_frag<T, DP>(dt, lanes, 0, ks), vf[ks]);
            }
            if constexpr (BIAS) {
                // entry of key 32 wave + l % 32 and query 8 (i / 4) + 4 h + i % 4 of the tile
                const lds_float_t* p = wbuf + b * WIN + (BQ - 1 - 4 * h) + 32 * wave + (lane & 31);
#pragma unroll
                for (int i = 0; i < 16; ++i) s[i] = fmaf(s[i], scale, p[-(8 * (i >> 2) + (i & 3))]);
            }
            const lds_float_t* refs = st;
            float factor = unit;
            if (sizeof(T) == 4 ? seen == SOME : __builtin_expect(seen == SOME || take_low, 0)) {
                if (seen == SOME) hide(s, sight, i0 + 4 * h);
                if (sizeof(T) == 2 && take_low) {
                    // the whole exponent, so that what follows has nothing to take from it
                    refs = zeros;
                    factor = 1.0f;
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const f32x4_t ref = *(const lds_f32x4_t*)(st + 8 * q + 4 * h), low = *(const lds_f32x4_t*)(st + BQ + 8 * q + 4 * h);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float z = s[4 * q + e];
                            s[4 * q + e] = (BIAS ? (z - ref[e]) * unit : fmaf(z, unit, -ref[e])) + low[e];
                        }
                    }
                }
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const f32x4_t ref = *(const lds_f32x4_t*)(refs + 8 * q + 4 * h), dl = *(const lds_f32x4_t*)(st + 2 * BQ + 8 * q + 4 * h);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float z = s[4 * q + e];
                    s[4 * q + e] = BIAS ? exp2_((z - ref[e]) * factor) : exp2_(fmaf(z, factor, -ref[e]));
                    if (sizeof(T) == 2) dp[4 * q + e] = s[4 * q + e] * (dp[4 * q + e] - dl[e]);
                }
            }
            if (sizeof(T) == 4 && take_low) {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const f32x4_t norm = *(const lds_f32x4_t*)(st + BQ + 8 * q + 4 * h);
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[4 * q + e] *= norm[e];
                }
            }
            if (sizeof(T) == 4)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const f32x4_t dl = *(const lds_f32x4_t*)(st + 2 * BQ + 8 * q + 4 * h);
#pragma unroll
                for (int e = 0; e < 4; ++e) dp[4 * q + e] = s[4 * q + e] * (dp[4 * q + e] - dl[e]);
            }
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                const Parts<T> p(s, g), d(dp, g);
#pragma unroll
                for (int db = 0; db < DB; ++db) {
                    if (beyond<T>(32 * db, a.width)) continue;
                    p.mma_to(dv[db], col_frag<T, DP>(dt, lanes, 16 * g, db));
                    d.mma_to(dk[db], col_frag<T, DP>(qt, lanes, 16 * g, db));
                }
            }
        }
        if constexpr (BIAS)
            if (next.left > 0) bw.put(wbuf + (b ^ 1) * WIN);
    }
    if (!in) return;
    if (f.kv_splits > 1) {
        const int64_t at = row * a.kv_heads + kv, total = a.keys * a.kv_heads;
        float* p = f.kv_part + (2 * split * total + at) * a.width;
        store_rows<float>(dk, 1.0f, p, static_cast<float*>(nullptr), a.width);
        store_rows<float>(dv, 1.0f, p + total * a.width, static_cast<float*>(nullptr), a.width);
        return;
    }
    store_rows<T>(dk, a.scale, static_cast<T*>(f.grad_k) + row * f.ld_dk + static_cast<int64_t>(kv) * f.hs_dk, static_cast<T*>(nullptr), a.width);
    store_rows<T>(dv, 1.0f, static_cast<T*>(f.grad_v) + row * f.ld_dv + static_cast<int64_t>(kv) * f.hs_dv, static_cast<T*>(nullptr), a.width);
}

template <typename T, int DP, bool BIAS>
__global__ __launch_bounds__(AT_THREADS, (KvShape<T, DP>::WAVES)) void attention_grad_kv_kernel(BackwardArgs f) {
    __shared__ __attribute__((aligned(512))) char lds[grad_kv_lds<T, DP, BIAS>()];
    grad_kv_block<T, DP, BIAS, false>(f, f.c.unit0 + blockIdx.x, (lds_byte_t*)lds);
}

// All of a small call at once.
template <typename T, int DP, bool BIAS> __global__ __launch_bounds__(AT_THREADS, 1) void attention_grad_all_kernel(BackwardArgs f) {
    constexpr int Q = grad_q_lds<T, DP, BIAS>(), KV = grad_kv_lds<T, DP, BIAS>();
    __shared__ __attribute__((aligned(512))) char lds[Q > KV ? Q : KV];
    if (blockIdx.x < f.q_blocks) grad_q_block<T, DP, BIAS>(f, blockIdx.x, (lds_byte_t*)lds);
    else grad_kv_block<T, DP, BIAS, true>(f, blockIdx.x - f.q_blocks, (lds_byte_t*)lds);
}

// ---- what splits and slots add up to ----------------------------------------------------

// One matrix's sum over the splits: out[row][head][d] = scale * sum of part[split][row][head][d].
struct SumJob {
    const float* part;
    void* out;
    int64_t pitch, count, ld, hs;   // count: rows x heads x width, 0: nothing to do
    int splits, heads;
    float scale;
};
struct FinishArgs {
    SumJob job[3];
    int64_t first[4];               // blocks of the jobs: first[k] .. first[k + 1) - 1
    int64_t block0;
    const float* bias_part;
    const double* bias_sums;        // of the distances, or NULL: each bucket adds up its distances' slots
    const int32_t* bucket_map;
    void* grad_bias;
    int64_t slots;
    int entries, buckets, bias_heads, width;
};

// Sum over `count` slots for 64 distances of one head, added to what the batches before left (`more`).  The orders are fixed; sums in fp64:
// they have up to millions of terms of either sign.
__global__ __launch_bounds__(1024) void attention_bias_slots_kernel(const float* part, int64_t slots, int64_t count, int entries, double* sums, int more) {
    __shared__ double red[16][64];
    const int lane = threadIdx.x & 63, wave = wave_id(), head = blockIdx.y;
    const int d = min(static_cast<int>(blockIdx.x) * 64 + lane, entries - 1);
    double v = 0.0;
    const float* p = part + head * slots * entries + d;
    int64_t s = wave;
    for (; s + 7 * 16 < count; s += 8 * 16) {
        float x[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = G(p)[(s + 16 * k) * entries];
#pragma unroll
        for (int k = 0; k < 8; ++k) v += x[k];
    }
    for (; s < count; s += 16) v += G(p)[s * entries];
    red[wave][lane] = v;
    __syncthreads();
    if (wave == 0) {
        for (int k = 1; k < 16; ++k) v += red[k][lane];
        MUON_GLOBAL double* sum = G(sums) + static_cast<int64_t>(head) * entries + d;
        if (more) v += *sum;
        if (static_cast<int>(blockIdx.x) * 64 + lane < entries) *sum = v;
    }
}

// The sums that are left, in one launch: a workgroup for each bucket and head, then AT_FINISH values of a matrix each.
template <typename T> __global__ __launch_bounds__(AT_FINISH) void attention_finish_kernel(FinishArgs f) {
    __shared__ double red[AT_FINISH / 64];
    __shared__ int mine[2 * MUON_MAX_REACH + 1];
    __shared__ int count;
    const int64_t block = f.block0 + blockIdx.x;
    if (block < f.first[0]) {
        const int bucket = static_cast<int>(block / f.bias_heads), head = static_cast<int>(block - static_cast<int64_t>(bucket) * f.bias_heads);
        const int lane = threadIdx.x & 63, wave = wave_id();
        double v = 0.0;
        if (f.bias_sums) {
            for (int d = threadIdx.x; d < f.entries; d += AT_FINISH)
                if (G(f.bucket_map)[d] == bucket) v += G(f.bias_sums)[static_cast<int64_t>(head) * f.entries + d];
        } else {
            // the bucket's distances, in order, found by the first wave
            if (wave == 0) {
                int n = 0;
                for (int d0 = 0; d0 < f.entries; d0 += 16 * 64) {
                    int of[16];
#pragma unroll
                    for (int k = 0; k < 16; ++k) of[k] = G(f.bucket_map)[min(d0 + 64 * k + lane, f.entries - 1)];
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        const bool in = d0 + 64 * k + lane < f.entries && of[k] == bucket;
                        const uint64_t set = __ballot(in);
                        if (in) mine[n + __popcll(set & ((1ull << lane) - 1))] = d0 + 64 * k + lane;
                        n += __popcll(set);
                    }
                }
                if (lane == 0) count = n;
            }
            __syncthreads();
            // 32 slots at once, 32 lanes a slot
            const int n = count;
            for (int64_t slot = threadIdx.x >> 5; slot < f.slots; slot += AT_FINISH / 32) {
                const float* p = f.bias_part + (head * f.slots + slot) * f.entries;
#pragma unroll 4
                for (int i = threadIdx.x & 31; i < n; i += 32) v += G(p)[mine[i]];
            }
        }
        double s[1] = {v};
        block_sums(s, red);
        if (threadIdx.x == 0) st_el<T>(f.grad_bias, static_cast<size_t>(bucket) * f.bias_heads + head, static_cast<float>(s[0]));
        return;
    }
    const int k = block >= f.first[2] ? 2 : block >= f.first[1] ? 1 : 0;
    const SumJob& j = f.job[k];
    const int64_t i = (block - f.first[k]) * AT_FINISH + threadIdx.x;
    if (i >= j.count) return;
    float v = 0.0f;
    int s = 0;
    for (; s + 7 < j.splits; s += 8) {
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = G(j.part)[(s + e) * j.pitch + i];
#pragma unroll
        for (int e = 0; e < 8; ++e) v += x[e];
    }
    for (; s < j.splits; ++s) v += G(j.part)[s * j.pitch + i];
    const int64_t at = i / f.width, row = at / j.heads;
    st_el<T>(j.out, row * j.ld + (at - row * j.heads) * j.hs + (i - at * f.width), v * j.scale);
}

// ---- rows to whole chunks -----------------------------------------------------------------

struct PackJob {
    const void* src;
    void* dst;
    int64_t ld, hs, count, heads;   // count: rows x heads
    int64_t first;                  // chunk of the whole launch
};
struct PackArgs {
    PackJob job[6];
    int64_t total;                  // chunks
    int64_t base;
    int jobs, width, chunks;        // chunks a row
};
template <typename T> __global__ __launch_bounds__(256) void attention_pack_kernel(PackArgs p) {
    const int64_t i = p.base + static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (i >= p.total) return;
    int k = 0;
#pragma unroll
    for (int n = 1; n < 6; ++n) k = n < p.jobs && i >= p.job[n].first ? n : k;
    const PackJob& j = p.job[k];
    const int64_t c = i - j.first, row = c / p.chunks, t = row / j.heads;
    const int e0 = static_cast<int>(c - row * p.chunks) * (16 / static_cast<int>(sizeof(T)));
    const T* src = static_cast<const T*>(j.src) + t * j.ld + (row - t * j.heads) * j.hs;
    G(static_cast<u32x4_t*>(j.dst))[c] = ld_part<T>(src + e0, p.width - e0);
}

// ---- host -------------------------------------------------------------------------

// Few units of an axis leave CUs idle: their walks are split until the workgroups fill the chip once (`target`: as many as it holds at
// once; a second round for a few of them costs as much as a full one), while a part keeps two tiles on average, one in fp32 if there are
// more than four (a join costs as much as one).  Under a causal
// mask walks so long that a part keeps 64 tiles are split until there are eight workgroups a CU, so that the longest do not end alone
// (16384 tokens, 4 key heads, grad_k and grad_v: 5.8 ms in one part).
int64_t axis_units(int64_t rows, int64_t sequences, int heads, int pack = 0) {
    return std::max<int64_t>(1, ((rows >> (AT_SHIFT - pack)) + sequences) * (heads >> pack));
}
int plan_splits(int64_t rows, int64_t sequences, int heads, int64_t walk, int tile, int dtype, bool causal, int64_t target, int pack = 0) {
    const int64_t n = axis_units(rows, sequences, heads, pack), tiles = std::max<int64_t>(1, walk / sequences / tile);
    const int64_t want = std::max(std::min((target + n / 2) / n, dtype == MUON_F32 && tiles > 4 ? tiles : tiles / 2), causal ? std::min(2048 / n, tiles / 64) : 0);
    return static_cast<int>(std::min<int64_t>(std::max<int64_t>(1, want), AT_MAX_SPLITS));
}
int tile_rows(int dtype) { return dtype == MUON_BF16 ? walk_rows<uint16_t>() : walk_rows<float>(); }
// Workgroups at once: two a CU, but one where fp32 takes all registers.  grad_q of a bias runs one a CU beyond 64 wide and is split as if two ran: split
// for one, 4096 causal tokens in 2 sequences, 4 heads, take 250 us for 237 (both passes), 2048 tokens, 8 heads 208 for 202, 1100 tokens, 4 heads 99 for 102.
int64_t at_once(int dtype, int width) { return dtype == MUON_F32 && width > 64 ? AT_CUS : 2 * AT_CUS; }

// Sequences of fewer queries than a workgroup has rows: heads that share a key head fill them (a bias is one head's), so that
// keys are read once for all of them (one query over 4096 keys, 4 heads each of 4 key heads: 10.0 us, 14.2 with a workgroup a head).
int forward_pack(const muon_attention_args& a) {
    int pack = 0;
    if (!a.bias && a.queries / a.sequences < AT_ROWS)
        while (pack < 5 && (a.heads / a.kv_heads) % (2 << pack) == 0) ++pack;
    return pack;
}
int forward_splits(const muon_attention_args& a) {
    return plan_splits(a.queries, a.sequences, a.heads, a.keys, tile_rows(a.dtype), a.dtype, a.causal, at_once(a.dtype, a.width), forward_pack(a));
}
struct BackwardPlan {
    int q_splits, kv_splits;
    int64_t q_blocks, kv_blocks;
    bool all;                                       // one launch for the three gradients
    bool two_step;                                  // the bias's slots are added up by distance first
    int64_t slots, batch;                           // of the bias's partial sums, per head, for a batch of so many units
    size_t delta, q_part, kv_part, bias_part, bias_sums, bytes;   // offsets
};
BackwardPlan plan_backward(const muon_attention_backward_args& a) {
    BackwardPlan p{};
    const int64_t qu = axis_units(a.queries, a.sequences, a.heads), ku = axis_units(a.keys, a.sequences, a.kv_heads);
    // As long as both find room on the chip at once, and walk over about 1024 keys at most, one launch takes as long as the longer of two
    // (3 sequences of 167 tokens, 16 heads of 64: 34 us the forward and backward pass, 43 in two launches; one of 1024 tokens, 2 heads: 39 and
    // 46).  Beyond that the registers of both parts together cost more, one workgroup a CU (4096 tokens, 4 heads of 128 over one key head: 282
    // and 224; 3 sequences of 683, 8 heads of 64: 104 and 90).  Its room goes to them by their products, 3 and 4.
    p.all = a.queries && a.keys && qu + ku <= AT_CUS && a.keys / a.sequences <= 1024;
    const int64_t kv_walk = a.queries * (a.heads / a.kv_heads);
    p.q_splits = plan_splits(a.queries, a.sequences, a.heads, a.keys, tile_rows(a.dtype), a.dtype, a.causal, p.all ? AT_CUS * 3 / 7 : at_once(a.dtype, a.width));
    p.kv_splits = plan_splits(a.keys, a.sequences, a.kv_heads, kv_walk, KV_ROWS, a.dtype, a.causal, p.all ? AT_CUS * 4 / 7 : at_once(a.dtype, 128));
    p.q_blocks = a.queries ? span_units(a.queries, a.sequences, AT_ROWS) * a.heads * p.q_splits : 0;
    p.kv_blocks = a.keys ? span_units(a.keys, a.sequences, AT_ROWS) * a.kv_heads * p.kv_splits : 0;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t here = at;
        at += (bytes + 255) / 256 * 256;
        return here;
    };
    const size_t q = static_cast<size_t>(a.queries) * a.heads, k = static_cast<size_t>(a.keys) * a.kv_heads;
    p.delta = take(p.all ? 0 : q * 4);
    p.q_part = take(p.q_splits > 1 ? p.q_splits * q * a.width * 4 : 0);
    p.kv_part = take(p.kv_splits > 1 ? 2 * p.kv_splits * k * a.width * 4 : 0);
    if (a.bias) {
        const size_t entries = 2 * static_cast<size_t>(a.reach) + 1;
        const int64_t units = a.queries ? span_units(a.queries, a.sequences, AT_ROWS) : 0, of_unit = static_cast<int64_t>(p.q_splits) * AT_WAVES;
        const int64_t fit = std::max<int64_t>(1, AT_SLOT_BYTES / static_cast<int64_t>(of_unit * a.heads * entries * 4)), batches = (units + fit - 1) / fit;
        p.batch = p.all || batches <= 1 ? units : (units + batches - 1) / batches;
        p.slots = p.batch * of_unit;
        p.two_step = p.batch < units || p.slots > AT_FEW_SLOTS || static_cast<int64_t>(entries) > AT_FEW_DISTANCES * a.buckets;
        p.bias_part = take(p.slots * a.heads * entries * 4);
        p.bias_sums = take(p.two_step ? a.heads * entries * 8 : 0);
    }
    p.bytes = at;
    return p;
}

int64_t elem(int dtype) { return dtype == MUON_BF16 ? 2 : 4; }
bool whole(const void* p, int64_t ld, int64_t hs, int64_t es) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * es % 16 == 0 && hs * es % 16 == 0;
}

// Inputs whose rows do not come in whole 16-byte chunks (odd widths, pitches or starts) are copied into the workspace first, one
// launch for all, rows of the next whole width with zeros behind: the walks read every row many times, and loads that go through
// registers wait for each other (2048 tokens, 8 heads of 101, both passes: 322 us without the copy, 142 with it, 120 at 104).
struct Packer {
    PackArgs args{};
    int64_t es;
    int width, padded;
    size_t at = 0;            // bytes of the workspace taken so far
    char* ws;
    Packer(int dtype, int w, void* workspace) : es(elem(dtype)), width(w), padded(static_cast<int>((w * es + 15) / 16 * 16 / es)), ws(static_cast<char*>(workspace)) {
        args.width = width;
        args.chunks = static_cast<int>(padded * es / 16);
    }
    // Puts the copy in place of a tensor that needs one.
    void operator()(const void*& p, int64_t& ld, int64_t& hs, int64_t rows, int64_t heads) {
        if (!p || rows == 0 || (width == padded && whole(p, ld, hs, es))) return;
        PackJob& j = args.job[args.jobs++];
        j = {p, ws + at, ld, hs, rows * heads, heads, args.total};
        args.total += j.count * args.chunks;
        p = ws + at;
        at += (static_cast<size_t>(j.count) * padded * es + 255) / 256 * 256;
        ld = heads * padded;
        hs = padded;
    }
};

// 1, or for sequences beyond find_span's orders a stride of about 0.618 units that meets every one of them once (units are odd, so that
// the stride mixes odd and even ones too).
int64_t unit_stride(int64_t units, int64_t sequences) {
    if (sequences <= SPAN_SCAN) return 1;
    int64_t k = units * 309 / 500;
    while (std::gcd(k, units) != 1) ++k;
    return k;
}

Common common_args(const muon_attention_args& a, int splits, int pack) {
    Common c{};
    c.a = a;
    c.pack = pack;
    c.q_axis = span_units(a.queries, a.sequences, AT_ROWS >> pack);
    c.k_axis = span_units(a.keys, a.sequences, AT_ROWS);
    c.q_stride = unit_stride(c.q_axis, a.sequences);
    c.k_stride = unit_stride(c.k_axis, a.sequences);
    if (!c.a.key_offsets) c.a.key_offsets = c.a.offsets;
    c.splits = splits;
    c.window = static_cast<int>(std::min<int64_t>(a.window, (1 << 30) - 1));
    c.gqa = a.heads / a.kv_heads;
    return c;
}

// A launch holds at most 2^32 - 1 threads.
template <typename F> hipError_t in_launches(int64_t blocks, F launch) {
    constexpr int64_t MOST = int64_t{1} << 21;      // of up to 1024
    for (int64_t b = 0; b < blocks; b += MOST) {
        const hipError_t e = launch(b, static_cast<unsigned>(std::min(MOST, blocks - b)));
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

template <typename T, int DP, bool BIAS> hipError_t run_forward(ForwardArgs f, hipStream_t s) {
    hipError_t e = in_launches(f.c.units, [&](int64_t base, unsigned n) {
        f.c.unit0 = base;
        hipLaunchKernelGGL((attention_forward_kernel<T, DP, BIAS>), dim3(n), dim3(AT_THREADS), 0, s, f);
        return hipGetLastError();
    });
    if (e != hipSuccess || f.c.splits == 1) return e;
    return in_launches((f.c.a.queries * f.c.a.heads + 3) / 4, [&](int64_t base, unsigned n) {
        hipLaunchKernelGGL((attention_join_kernel<T, BIAS>), dim3(n), dim3(256), 0, s, f, base * 4);
        return hipGetLastError();
    });
}

template <typename T, int DP, bool BIAS>
hipError_t run_backward(BackwardArgs f, const BackwardPlan& p, const muon_attention_backward_args& b, char* ws, hipStream_t s) {
    const muon_attention_args& a = f.c.a;
    hipError_t e = hipSuccess;
    auto add_slots = [&](int64_t units, bool more) {
        const int entries = 2 * a.reach + 1;
        hipLaunchKernelGGL(attention_bias_slots_kernel, dim3((entries + 63) / 64, a.heads), dim3(1024), 0, s, f.bias_part, p.slots,
                           units * p.q_splits * AT_WAVES, entries, reinterpret_cast<double*>(ws + p.bias_sums), more ? 1 : 0);
        return hipGetLastError();
    };
    if (p.all) {
        hipLaunchKernelGGL((attention_grad_all_kernel<T, DP, BIAS>), dim3(static_cast<unsigned>(p.q_blocks + p.kv_blocks)), dim3(AT_THREADS), 0, s, f);
        e = hipGetLastError();
        if (e == hipSuccess && BIAS && p.two_step) e = add_slots(p.batch, false);
    } else {
        const int64_t of_unit = static_cast<int64_t>(a.heads) * p.q_splits, units = p.q_blocks / of_unit, batch = BIAS && units ? p.batch : units;
        for (int64_t u = 0; u < units; u += batch) {
            const int64_t n_units = std::min(batch, units - u);
            f.first_unit = u;
            e = in_launches(n_units * of_unit, [&](int64_t base, unsigned n) {
                f.c.unit0 = u * of_unit + base;
                hipLaunchKernelGGL((attention_grad_q_kernel<T, DP, BIAS>), dim3(n), dim3(AT_THREADS), 0, s, f);
                return hipGetLastError();
            });
            if (e == hipSuccess && BIAS && p.two_step) e = add_slots(n_units, u > 0);
            if (e != hipSuccess) return e;
        }
        if (BIAS && p.two_step && units == 0) e = add_slots(0, false);
        if (e != hipSuccess) return e;
        e = in_launches(p.kv_blocks, [&](int64_t base, unsigned n) {
            f.c.unit0 = base;
            hipLaunchKernelGGL((attention_grad_kv_kernel<T, DP, BIAS>), dim3(n), dim3(AT_THREADS), 0, s, f);
            return hipGetLastError();
        });
    }
    if (e != hipSuccess) return e;
    FinishArgs g{};
    g.width = a.width;
    if constexpr (BIAS) {
        g.bias_part = f.bias_part;
        g.bucket_map = a.bucket_map;
        g.grad_bias = b.grad_bias;
        g.slots = p.slots;
        g.entries = 2 * a.reach + 1;
        g.buckets = a.buckets;
        g.bias_heads = a.heads;
        g.first[0] = static_cast<int64_t>(a.buckets) * a.heads;
        if (p.two_step) g.bias_sums = reinterpret_cast<const double*>(ws + p.bias_sums);
    }
    const int64_t q = a.queries * a.heads * a.width, k = a.keys * a.kv_heads * a.width;
    if (p.q_splits > 1) g.job[0] = {f.q_part, f.grad_q, q, q, f.ld_dq, f.hs_dq, p.q_splits, a.heads, a.scale};
    if (p.kv_splits > 1) {
        g.job[1] = {f.kv_part, f.grad_k, 2 * k, k, f.ld_dk, f.hs_dk, p.kv_splits, a.kv_heads, a.scale};
        g.job[2] = {f.kv_part + k, f.grad_v, 2 * k, k, f.ld_dv, f.hs_dv, p.kv_splits, a.kv_heads, 1.0f};
    }
    for (int i = 0; i < 3; ++i) g.first[i + 1] = g.first[i] + (g.job[i].count + AT_FINISH - 1) / AT_FINISH;
    return in_launches(g.first[3], [&](int64_t base, unsigned n) {
        g.block0 = base;
        hipLaunchKernelGGL((attention_finish_kernel<T>), dim3(n), dim3(AT_FINISH), 0, s, g);
        return hipGetLastError();
    });
}

// Calls f with the tile width and whether there is a bias, as types.
template <typename F> hipError_t dispatch(int dtype, int width, bool bias, F f) {
    auto by_bias = [&](auto t, auto dp) { return bias ? f(t, dp, std::true_type{}) : f(t, dp, std::false_type{}); };
    auto by_width = [&](auto t) {
        return width <= 64 ? by_bias(t, std::integral_constant<int, 64>{}) : by_bias(t, std::integral_constant<int, 128>{});
    };
    return dtype == MUON_BF16 ? by_width(uint16_t{}) : by_width(float{});
}

}  // namespace

namespace {

template <typename T> hipError_t run_pack_as(PackArgs p, hipStream_t s) {
    return in_launches((p.total + 255) / 256, [&](int64_t base, unsigned n) {
        p.base = base * 256;
        hipLaunchKernelGGL((attention_pack_kernel<T>), dim3(n), dim3(256), 0, s, p);
        return hipGetLastError();
    });
}
hipError_t run_pack(const Packer& p, int dtype, hipStream_t s) {
    return dtype == MUON_BF16 ? run_pack_as<uint16_t>(p.args, s) : run_pack_as<float>(p.args, s);
}

// The forward call with its packed inputs; the workspace: copies, then the splits' sums.
Packer pack_forward(muon_attention_args& a, void* workspace) {
    Packer p(a.dtype, a.width, workspace);
    p(a.q, a.ld_q, a.hs_q, a.queries, a.heads);
    p(a.k, a.ld_k, a.hs_k, a.keys, a.kv_heads);
    p(a.v, a.ld_v, a.hs_v, a.keys, a.kv_heads);
    return p;
}
Packer pack_backward(muon_attention_backward_args& b, void* workspace) {
    Packer p(b.dtype, b.width, workspace);
    p(b.q, b.ld_q, b.hs_q, b.queries, b.heads);
    p(b.k, b.ld_k, b.hs_k, b.keys, b.kv_heads);
    p(b.v, b.ld_v, b.hs_v, b.keys, b.kv_heads);
    p(b.grad_out, b.ld_grad_out, b.hs_grad_out, b.queries, b.heads);
    p(b.out, b.ld_out, b.hs_out, b.queries, b.heads);
    p(b.out_low, b.ld_out_low, b.hs_out_low, b.queries, b.heads);
    return p;
}

}  // namespace

size_t attention_bytes(const muon_attention_args& args) {
    muon_attention_args a = args;
    const int s = forward_splits(a);
    return pack_forward(a, nullptr).at + (s > 1 ? static_cast<size_t>(s) * a.queries * a.heads * (a.width + 2) * sizeof(float) : 0);
}

hipError_t launch_attention(const muon_attention_args& args, float* lse_low, void* workspace, hipStream_t s) {
    if (args.queries == 0) return hipSuccess;
    muon_attention_args a = args;
    const Packer pack = pack_forward(a, workspace);
    const hipError_t e = run_pack(pack, a.dtype, s);
    if (e != hipSuccess) return e;
    ForwardArgs f{};
    f.c = common_args(a, forward_splits(a), forward_pack(a));
    f.c.units = f.c.q_axis * (a.heads >> f.c.pack) * f.c.splits;
    f.c.lse_low = lse_low;
    f.part = reinterpret_cast<float*>(static_cast<char*>(workspace) + pack.at);
    return dispatch(a.dtype, a.width, a.bias != nullptr, [&](auto t, auto dp, auto bias) {
        return run_forward<decltype(t), decltype(dp)::value, decltype(bias)::value>(f, s);
    });
}

size_t attention_backward_bytes(const muon_attention_backward_args& args) {
    muon_attention_backward_args b = args;
    return pack_backward(b, nullptr).at + plan_backward(b).bytes;
}

hipError_t launch_attention_backward(const muon_attention_backward_args& args, const float* lse_low, void* workspace, hipStream_t s) {
    muon_attention_backward_args b = args;
    const Packer pack = pack_backward(b, workspace);
    hipError_t e = run_pack(pack, b.dtype, s);
    if (e != hipSuccess) return e;
    const BackwardPlan p = plan_backward(b);
    muon_attention_args a{};
    a.q = b.q; a.k = b.k; a.v = b.v;
    a.offsets = b.offsets; a.key_offsets = b.key_offsets; a.key_mask = b.key_mask;
    a.bias = b.bias; a.bucket_map = b.bucket_map;
    a.out = const_cast<void*>(b.out); a.lse = const_cast<float*>(b.lse); a.out_low = const_cast<void*>(b.out_low);
    a.queries = b.queries; a.keys = b.keys; a.sequences = b.sequences;
    a.ld_q = b.ld_q; a.hs_q = b.hs_q; a.ld_k = b.ld_k; a.hs_k = b.hs_k; a.ld_v = b.ld_v; a.hs_v = b.hs_v;
    a.ld_out = b.ld_out; a.hs_out = b.hs_out; a.ld_out_low = b.ld_out_low; a.hs_out_low = b.hs_out_low;
    a.window = b.window; a.scale = b.scale;
    a.heads = b.heads; a.kv_heads = b.kv_heads; a.width = b.width;
    a.buckets = b.buckets; a.reach = b.reach; a.causal = b.causal; a.dtype = b.dtype;
    BackwardArgs f{};
    f.c = common_args(a, 1, 0);
    f.c.lse_low = const_cast<float*>(lse_low);
    f.grad_out = b.grad_out;
    f.grad_q = b.grad_q; f.grad_k = b.grad_k; f.grad_v = b.grad_v;
    f.ld_do = b.ld_grad_out; f.hs_do = b.hs_grad_out;
    f.ld_dq = b.ld_grad_q; f.hs_dq = b.hs_grad_q;
    f.ld_dk = b.ld_grad_k; f.hs_dk = b.hs_grad_k;
    f.ld_dv = b.ld_grad_v; f.hs_dv = b.hs_grad_v;
    char* ws = static_cast<char*>(workspace) + pack.at;
    f.delta = p.all ? nullptr : reinterpret_cast<float*>(ws + p.delta);
    f.bias_part = reinterpret_cast<float*>(ws + p.bias_part);
    f.slots = p.slots;
    f.q_splits = p.q_splits;
    f.kv_splits = p.kv_splits;
    f.q_part = reinterpret_cast<float*>(ws + p.q_part);
    f.kv_part = reinterpret_cast<float*>(ws + p.kv_part);
    f.q_blocks = p.q_blocks;
    return dispatch(a.dtype, a.width, a.bias != nullptr, [&](auto t, auto dp, auto bias) {
        return run_backward<decltype(t), decltype(dp)::value, decltype(bias)::value>(f, p, b, ws, s);
    });
}

}  // namespace muon
