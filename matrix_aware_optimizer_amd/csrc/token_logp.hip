// Log-probabilities of target tokens under a vocabulary head, and their gradients.
//
//   z = scale hidden head^T,  lse_i = log sum_j exp(z_ij),  logp_i = z_i,target_i - lse_i
//   dz_ij = scale grad_logp_i ([j = target_i] - exp(z_ij - lse_i))
//   grad_hidden = dz head,  grad_head = dz^T hidden
// The work is the three products (2 tokens vocab cols operations each), bound by the matrix
// cores; everything else is arranged around the 256 x 256 tile of product_tile.h:
//
//  - Only scored tokens are worked on: scan_kernel lists them on the GPU, the products
//    gather their rows of hidden, and workgroups beyond the list end at once.
//  - Logits: C = head hidden^T, vocabulary along the accumulator rows, so that a lane holds 64
//    logits of one token and the softmax's running maximum and sum need one exchange between
//    lanes and one between two waves.  Only (maximum, sum) per token and tile leave the tile;
//    combine_kernel joins them.  With `saved` the tile's exp(z - tile maximum) goes out too: in fp16 in
//    bf16 calls (values of at most 1: 11 bits where bf16 keeps 8, fewer below 2^-14 of the tile's maximum, 0 below 2^-25), else
//    in fp32.  Neither maximum nor sum counts the token's target: beside a certain target the other entries of its tile keep
//    their bits, and the target's own gradient comes from logp.
//  - Backward: dz comes from `saved` by an elementwise pass; without `saved` the logits' product comes first again, for a
//    chunk of tokens at a time.  The target's own dz is -c expm1(logp): 1 - exp(z - lse) from a rounded lse would be off by
//    1e-6, all there is of a certain token's gradient.
//    dz is written both token-major and vocabulary-major, and head and hidden are transposed
//    once, so that both gradients are k-contiguous products (C rows = columns of the gradient,
//    C columns = its rows).  Few tiles: the sum over k is split over workgroups that leave fp32
//    tiles, added in order by slab_sum_kernel.
//  - fp32 operands travel as two fp16 parts under a scale (product_tile.h): scan_kernel finds the largest values, and the
//    kernels that make the copies the scales.  dz does so too, in bf16 calls in one part: 11 bits of it where bf16 would keep 8
//    (6144 x 2048 x 32000: a gradient's error with its own rounding 0.0017 of its norm, as if dz were exact; 0.0024 in bf16).  The
//    matrix cores take one type, so the transposed copies of bf16 operands are fp16 under a scale as well, exact down to
//    2^-29 of the operand's largest value; what that costs is a look through head for it.  dz has a scale for each token, that its own
//    largest entry gives, -c expm1(logp) of the target: a token's gradient keeps its bits beside tokens with larger ones.
//    grad_hidden takes the tokens' scales out of its columns; for grad_head they are taken out of hidden's copy before the product.
//  - Few tokens: what counts is the head's way through memory, so each step reads (or writes) it once where it is,
//    with 16 x 16 MFMAs and no staging (fp32 as three bf16 parts there: exact down to 2^-109, so that only hidden, which
//    is small and quickly looked through, gets a scale).
//
// The softmax works in base 2: with k' = |scale| log2(e) and acc the product (negated if scale is negative) a tile keeps
// M = k' max acc, rounded, and sums 2^(k' acc - M), the exponent formed by one fused operation: what M is rounded to
// cancels, where a rounded k' acc would lose a unit of its own size.  A target's acc is kept as it is and its own term
// stays out of M and the sum S of its token, logp = -log(1 + S 2^(M - k' acc_target)), which keeps its relative precision as
// logp goes to 0.
#include <algorithm>
#include <type_traits>

#include "product_tile.h"
#include "train_internal.h"

namespace muon {

namespace {

using pt::u32x4;

constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;
// Most tokens of the few_ kernels (forward and backward, 48 tokens x 2048 x 32000 bf16: 142 us,
// 224 with the tiles' kernels; 64: 147, 229; 40 tokens in fp32: 378, 574; 12 tokens x 2048 x 65536 in fp32: 404, 1217).
constexpr int64_t FEW_TOKENS = 64;
constexpr int FEW_ROWS = 32;                // vocabulary entries per workgroup of few_kernel
constexpr int64_t DZ_BYTES = int64_t{4} << 30;   // both layouts of dz (without `saved`: and e), at most: more tokens go in chunks
constexpr int CUS = 256;
// 256 x 256 tiles below which the smaller tile serves a product: some 3/4 of the CUs.  2000 x 1024 x 8192, both passes: 188 us, at a
// bound of 96 198; 8192 (6144 scored) x 2048 x 32000: 2556, at 512 2930; 777 x 1000 x 32003: 296, at 512 330.
constexpr int64_t FEW_TILES = 192;
constexpr int PAD = 256;                    // every buffer of dz, e and their statistics is padded to the larger tile
// Runs of k of a product with few tiles, at most, and k-steps of one, at least: 300 x 512 x 8000, both passes, 69 us; 67 with 8
// runs or 16 steps, 69 with 32 runs or 4 steps.
constexpr int MAX_SPLITS = 16, MIN_SPLIT_STEPS = 8;

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline int64_t up(int64_t a, int64_t b) { return ceil_div(a, b) * b; }

// x times its operand's scale as fp16 parts (product_tile.h), patterns of 16 bits.  What is not finite is all in the first.
__device__ __forceinline__ void split2(float x, uint16_t (&p)[2]) {
    const _Float16 hi = static_cast<_Float16>(x);
    const float h = static_cast<float>(hi);
    const _Float16 lo = static_cast<_Float16>(fabsf(h) < INFINITY ? (x - h) * (1.0f / pt::LO_STEP) : 0.0f);
    p[0] = __builtin_bit_cast(uint16_t, hi);
    p[1] = __builtin_bit_cast(uint16_t, lo);
}
// A value, scaled, as the fp16 parts that the gradients' products take.
template <int PARTS> __device__ __forceinline__ void half_parts(float x, uint16_t (&p)[2]) {
    if constexpr (PARTS == 1) p[0] = __builtin_bit_cast(uint16_t, static_cast<_Float16>(x));
    else split2(x, p);
}

// k' of the comment above; scale 0 as a number so small that it makes no difference, so that k' times minus infinity stays so.
__device__ __forceinline__ float rate_of(float scale2) { return fmaxf(fabsf(scale2), 1.17549435e-38f); }
__device__ __forceinline__ float shown(float m) { return m == -INFINITY ? 0.0f : m; }   // an M to subtract

// Workgroups in a row, whatever their number: a launch holds fewer than 2^32 threads along x, so the row goes on along y.
__device__ __forceinline__ int64_t block_in_row() { return static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x; }
dim3 row_of_blocks(int64_t blocks, int threads) {
    const int64_t x = std::max<int64_t>(1, std::min(blocks, (int64_t{1} << 31) / threads));
    return dim3(static_cast<unsigned>(x), static_cast<unsigned>(std::max<int64_t>(1, (blocks + x - 1) / x)));
}

// ---------------------------------------------------------------------------
// The scored tokens, in order
// ---------------------------------------------------------------------------

constexpr int LIVE_THREADS = 1024, LIVE_PER = 4;

// idx[0 .. count): the tokens with a target >= 0.  logp and lse (forward) of the others are
// set to 0.  One workgroup: 8 bytes a token, a few microseconds for 8192.
__device__ __forceinline__ void list_live(const int64_t* targets, int64_t tokens, int32_t* idx, int32_t* count, float* logp, float* lse) {
    __shared__ int sums[LIVE_THREADS / 64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int base = 0;
    for (int64_t t0 = 0; t0 < tokens; t0 += LIVE_THREADS * LIVE_PER) {
        bool on[LIVE_PER];
        int n = 0;
#pragma unroll
        for (int e = 0; e < LIVE_PER; ++e) {
            const int64_t t = t0 + threadIdx.x * LIVE_PER + e;
            on[e] = t < tokens && targets[t] >= 0;
            n += on[e];
            if (logp && t < tokens && !on[e]) { logp[t] = 0.0f; lse[t] = 0.0f; }
        }
        int pre = n;   // inclusive prefix in the wave
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int v = __shfl_up(pre, o, 64);
            if (lane >= o) pre += v;
        }
        __syncthreads();
        if (lane == 63) sums[wave] = pre;
        __syncthreads();
        int before = base;
        for (int w = 0; w < LIVE_THREADS / 64; ++w) {
            if (w < wave) before += sums[w];
            base += sums[w];
        }
        before += pre - n;
#pragma unroll
        for (int e = 0; e < LIVE_PER; ++e)
            if (on[e]) idx[before++] = static_cast<int32_t>(t0 + threadIdx.x * LIVE_PER + e);
    }
    if (threadIdx.x == 0) *count = base;
}

// The rows of one call's products along the tokens: entries [first, first + most) of the list.
struct Live {
    const int32_t* idx;
    const int32_t* count;
    int32_t first, most;
    __device__ int rows() const { return max(0, min(*count - first, most)); }
};

// ---------------------------------------------------------------------------
// Scales of operands in fp16
// ---------------------------------------------------------------------------

// Bits of the largest finite |x| over the rows of head and the scored rows of hidden, one partial a workgroup: the first
// ABS_HEAD of them for head, the others for hidden.
constexpr int ABS_HEAD = 512, ABS_HIDDEN = 128, ABS_ROWS = 4;   // ABS_ROWS: rows a wave has in flight
struct AbsMaxArgs {
    const void *head, *hidden;
    size_t ld_head, ld_hidden;
    int64_t vocab, tokens, cols;
    const int64_t* targets;
    uint32_t* part;
};
__device__ __forceinline__ uint32_t block_max(uint32_t m, uint32_t* red) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), o, 64)));
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
    __syncthreads();
    for (int w = 0; w < static_cast<int>(blockDim.x >> 6); ++w) m = max(m, red[w]);
    return m;
}
__device__ __forceinline__ uint32_t finite_bits(float x) {
    const uint32_t b = __float_as_uint(x) & 0x7fffffffu;
    return b < 0x7f800000u ? b : 0u;
}
// The largest magnitude of a run so far, as bits (bf16: of two values a word), infinities and NaN included.
__device__ __forceinline__ uint32_t largest_bits(const Run<uint16_t>& x, uint32_t m) {
    typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));
#pragma unroll
    for (int e = 0; e < 4; ++e)
        m = __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2_t, m), __builtin_bit_cast(u16x2_t, x.w[e] & 0x7fff7fffu)));
    return m;
}
__device__ __forceinline__ uint32_t largest_bits(const Run<float>& x, uint32_t m) {
#pragma unroll
    for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(x.get(e)) & 0x7fffffffu);
    return m;
}
template <typename T> __device__ __forceinline__ void find_absmax(const AbsMaxArgs& a, int block, uint32_t* red) {
    const bool head = block < ABS_HEAD;
    const int b = head ? block : block - ABS_HEAD, blocks = head ? ABS_HEAD : ABS_HIDDEN;
    const int waves = blockDim.x >> 6, wave = pt::wave_id();
    const int64_t rows = head ? a.vocab : a.tokens, runs = (a.cols + 7) / 8;
    const size_t ld = head ? a.ld_head : a.ld_hidden;
    const auto* base = G(static_cast<const T*>(head ? a.head : a.hidden));
    // rows from `wave` on, f(run) on each run of 8 columns of those that count
    auto over = [&](auto f) {
        for (int64_t r = ABS_ROWS * (static_cast<int64_t>(waves) * b + wave); r < rows; r += ABS_ROWS * static_cast<int64_t>(waves) * blocks) {
            bool on[ABS_ROWS];
#pragma unroll
            for (int i = 0; i < ABS_ROWS; ++i) on[i] = r + i < rows && (head || a.targets[r + i] >= 0);
            for (int64_t k = threadIdx.x & 63; k < runs; k += 64) {
                Run<T> x[ABS_ROWS];
#pragma unroll
                for (int i = 0; i < ABS_ROWS; ++i) {
                    if (!on[i]) continue;
                    const auto* q = base + static_cast<size_t>(r + i) * ld;
                    if (8 * k + 8 <= a.cols) x[i].load(q, static_cast<unsigned>(8 * k));
                    else x[i].load(q, static_cast<unsigned>(8 * k), static_cast<unsigned>(a.cols - 8 * k));
                }
#pragma unroll
                for (int i = 0; i < ABS_ROWS; ++i) f(x[i]);
            }
        }
    };
    uint32_t m = 0;
    over([&](const Run<T>& x) { m = largest_bits(x, m); });
    if constexpr (sizeof(T) == 2) m = max(m << 16, m & 0xffff0000u);
    if (__any(m >= 0x7f800000u)) {   // not finite: again, with a look at each value
        m = 0;
        over([&](const Run<T>& x) {
#pragma unroll
            for (int e = 0; e < 8; ++e) m = max(m, finite_bits(x.get(e)));
        });
    }
    m = block_max(m, red);
    if (threadIdx.x == 0) a.part[block] = m;
}
// What the products wait for, side by side: the list (the first workgroup, if wanted) and the largest values.
struct ScanArgs {
    int list;               // 1: with the list
    const int64_t* targets;
    int64_t tokens;
    int32_t *idx, *count;
    float *logp, *lse;
    int first, blocks;      // workgroups for the largest values, from `first` on (ABS_HEAD: hidden alone)
    AbsMaxArgs absmax;
};
template <typename T> __global__ __launch_bounds__(LIVE_THREADS) void scan_kernel(ScanArgs a) {
    __shared__ uint32_t red[LIVE_THREADS / 64];
    if (a.list && blockIdx.x == 0) list_live(a.targets, a.tokens, a.idx, a.count, a.logp, a.lse);
    else find_absmax<T>(a.absmax, a.first + static_cast<int>(blockIdx.x) - a.list, red);
}
// The power of two that brings the largest value to 2^14 .. 2^15.
__device__ __forceinline__ float scale_of(uint32_t bits) {
    if (bits == 0) return 1.0f;
    const int s = min(14 - (static_cast<int>(bits >> 23) - 127), 126);   // at least -113: a normal number both ways
    return __uint_as_float(static_cast<uint32_t>(s + 127) << 23);
}
__device__ __forceinline__ int exponent_of(float scale) { return static_cast<int>(__float_as_uint(scale) >> 23) - 127; }
// An operand's scale from scan_kernel's partials, by a workgroup that is about to use it.
__device__ __forceinline__ float operand_scale(const uint32_t* part, bool head, uint32_t* red) {
    const int first = head ? 0 : ABS_HEAD, n = head ? ABS_HEAD : ABS_HIDDEN;
    uint32_t m = 0;
    for (int k = threadIdx.x; k < n; k += blockDim.x) m = max(m, part[first + k]);
    m = block_max(m, red);
    __syncthreads();   // `red` may be used again
    return scale_of(m);
}
// Exponent of the smallest scale that dz of any token can get: no value exceeds |scale grad_logp| of its token.
struct DzScaleArgs {
    Live live;
    const float* grad_logp;
    float scale;
    int32_t* out;
};
__device__ __forceinline__ void dz_scale(const DzScaleArgs& a, uint32_t* red) {
    uint32_t m = 0;
    const int n = a.live.rows();
#pragma unroll 8
    for (int r = threadIdx.x; r < n; r += blockDim.x) m = max(m, finite_bits(a.scale * a.grad_logp[a.live.idx[a.live.first + r]]));
    m = block_max(m, red);
    if (threadIdx.x == 0) *a.out = exponent_of(scale_of(m));
}

// What dz of a list entry takes.  dz_y = -c expm1(logp) of the target is minus the sum of the entry's other values, so none is larger.
struct DzTokenArgs {
    Live live;
    const int64_t* targets;
    const float *logp, *grad_logp;   // logp: by list entry
    float scale;
    int vocab;
    const int32_t* least;            // dz_scale's
};
struct DzToken {
    int64_t target;
    float c, logp;
    __device__ __forceinline__ void load(const DzTokenArgs& a, int tok, int entry) {
        target = a.targets[tok];
        c = a.scale * a.grad_logp[tok];
        logp = a.logp[entry];
    }
    __device__ __forceinline__ bool valid(const DzTokenArgs& a) const { return target < a.vocab; }
    __device__ __forceinline__ float dy() const { return -c * expm1f(logp); }
    // Exponent of the token's scale.
    __device__ __forceinline__ int exponent(const DzTokenArgs& a) const {
        const uint32_t largest = finite_bits(valid(a) ? dy() : c);   // 0 also where it is not finite
        return largest ? max(*a.least, exponent_of(scale_of(largest))) : *a.least;
    }
};

// ---------------------------------------------------------------------------
// Operand copies
// ---------------------------------------------------------------------------

struct PackArgs {
    const void* src;
    size_t ld;             // elements
    int64_t rows, cols;    // of src (rows: an upper bound where `live` gives them)
    int use_live;
    Live live;
    uint16_t* dst;
    size_t dst_ld, part;   // elements
    const float* scale;    // transposes: the operand's scale
};

// Copies for the logits' product, dst[part][r][0 .. dst_ld) = parts of src[row r], zero past its columns: of head (the first
// head_blocks workgroups) and of hidden.
struct PackBothArgs {
    PackArgs head, hidden;
    int head_blocks, hidden_blocks;
    const uint32_t* absmax;   // two parts: scan_kernel's partials
    float* scales;            // and where the scales of hidden and head are left
};
template <typename T, int PARTS>
__global__ __launch_bounds__(256) void pack_kernel(PackBothArgs both) {
    __shared__ uint32_t red[4];
    const bool head = static_cast<int>(blockIdx.x) < both.head_blocks;
    const PackArgs& a = head ? both.head : both.hidden;
    const int block = head ? blockIdx.x : blockIdx.x - both.head_blocks, blocks = head ? both.head_blocks : both.hidden_blocks;
    const int64_t rows = a.use_live ? a.live.rows() : a.rows;
    const int64_t per = a.dst_ld / 8, n = rows * per;
    float scale = 1.0f;
    if constexpr (PARTS == 2) {
        scale = operand_scale(both.absmax, head, red);
        if (block == 0 && threadIdx.x == 0) both.scales[head] = scale;
    }
    for (int64_t q = static_cast<int64_t>(block) * 256 + threadIdx.x; q < n; q += static_cast<int64_t>(blocks) * 256) {
        const int64_t r = q / per, c = (q - r * per) * 8;
        const size_t s = static_cast<size_t>(a.use_live ? a.live.idx[a.live.first + r] : r) * a.ld + c;
        uint16_t v[8][2];
        Run<T> x;
        const auto* q8 = G(static_cast<const T*>(a.src) + s);
        if (c + 8 <= a.cols) x.load(q8, 0);
        else if (c < a.cols) x.load(q8, 0, static_cast<unsigned>(a.cols - c));
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if constexpr (PARTS == 1) v[e][0] = f32_to_bf16(x.get(e));
            else split2(x.get(e) * scale, v[e]);
        }
#pragma unroll
        for (int p = 0; p < PARTS; ++p) {
            u32x4 w;
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = v[2 * e][p] | static_cast<uint32_t>(v[2 * e + 1][p]) << 16;
            G(reinterpret_cast<u32x4*>(a.dst + p * a.part + r * a.dst_ld + c))[0] = w;
        }
    }
}

// dst[part][c][r] = fp16 parts of src[row r][c] for c < cols, zero for rows past the last up to a multiple of 64: the
// 64 x 64 tile at (r0, c0), through LDS as fp32, 16-byte accesses on both sides.
template <typename T, int PARTS> __device__ __forceinline__ void transpose_tile(const PackArgs& a, int64_t r0, int64_t c0, float (&tile)[64][65]) {
    const float scale = *a.scale;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        const int k = (threadIdx.x >> 3) + 32 * half, x = 8 * (threadIdx.x & 7);
        const int64_t r = r0 + k, left = a.cols - c0 - x;
        Run<T> w;
        if (r < a.rows && left > 0) {
            const auto* q = G(static_cast<const T*>(a.src) + static_cast<size_t>(r) * a.ld + c0);
            if (left >= 8) w.load(q, x);
            else w.load(q, x, static_cast<unsigned>(left));
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) tile[k][x + e] = w.get(e);
    }
    __syncthreads();
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        const int c = (threadIdx.x >> 3) + 32 * half, r = 8 * (threadIdx.x & 7);
        if (c0 + c >= a.cols) continue;
        uint16_t v[8][2];
#pragma unroll
        for (int e = 0; e < 8; ++e) half_parts<PARTS>(tile[r + e][c] * scale, v[e]);
#pragma unroll
        for (int p = 0; p < PARTS; ++p) {
            u32x4 w;
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = v[2 * e][p] | static_cast<uint32_t>(v[2 * e + 1][p]) << 16;
            G(reinterpret_cast<u32x4*>(a.dst + p * a.part + (c0 + c) * a.dst_ld + r0 + r))[0] = w;
        }
    }
}

// One launch for what comes before dz: the transpose of head, the least scale of dz and, for grad_hidden, zeros in
// the rows of tokens that are not scored.  Each is a run of workgroups.
struct PrepareArgs {
    PackArgs head;
    int head_blocks, head_rows;       // 64 x 64 tiles, along the rows first; of them along the rows
    Live live;
    const int64_t* targets;
    int64_t tokens, cols;
    void* zero;
    size_t zero_ld;
    int zero_blocks;
    DzScaleArgs dz;                   // one workgroup, if out is not NULL
};
template <typename T, int PARTS> __global__ __launch_bounds__(256) void prepare_kernel(PrepareArgs a) {
    __shared__ float tile[64][65];
    int b = blockIdx.x;
    if (a.dz.out && b-- == 0) {   // first: it takes the longest
        dz_scale(a.dz, reinterpret_cast<uint32_t*>(tile));
        return;
    }
    if (b < a.head_blocks) {
        if (a.live.rows() == 0) return;   // nothing will read it
        transpose_tile<T, PARTS>(a.head, static_cast<int64_t>(b % a.head_rows) * 64, static_cast<int64_t>(b / a.head_rows) * 64, tile);
        return;
    }
    b -= a.head_blocks;
    for (int64_t t = static_cast<int64_t>(b) * 4 + (threadIdx.x >> 6); t < a.tokens; t += 4 * static_cast<int64_t>(a.zero_blocks))
        if (a.targets[t] < 0)
            for (int64_t c = threadIdx.x & 63; c < a.cols; c += 64) st_el<T>(a.zero, t * a.zero_ld + c, 0.0f);
}

// ---------------------------------------------------------------------------
// Logits, tile by tile
// ---------------------------------------------------------------------------

enum LogitsMode { LG_STATS = 0, LG_SAVE = 1 };

struct LogitsArgs {
    const char* a;          // head rows (bytes pitch a_ld, parts a_part apart)
    size_t a_ld, a_part;
    const char* b;          // hidden rows, by token (gather) or packed by list entry
    size_t b_ld, b_part;
    int gather;
    Live live;
    const int64_t* targets;
    int vocab, steps, tail, ta, tb;   // tail: 16-byte chunks of the last k-step
    float scale2;           // scale log2(e)
    const float* scales;    // two parts: of hidden and head
    float *m, *s;           // M and S: tile x list entry from live.first on (pitch rows_pitch)
    float* zt;              // target's acc by list entry
    size_t rows_pitch;
    void* e;                // LG_SAVE: 2^(k' acc - M), list entry from live.first on x vocabulary (pitch vp), fp16 (bf16 operands) or fp32
    size_t vp;
};

// The staged tile's first `rows` columns as rows of `dst` (from its column v0), column c at row r0 + c.
template <typename TL>
__device__ __forceinline__ void store_cols(const pt::lds_byte_t* L, uint16_t* dst, size_t ld, size_t r0, size_t v0, int rows) {
    constexpr int Q = TL::SIZE / 8, PER = TL::THREADS / Q;   // chunks of a column, columns at a time
#pragma unroll 4
    for (int k = 0; k < TL::SIZE / PER; ++k) {
        const int c = PER * k + static_cast<int>(threadIdx.x) / Q, q = threadIdx.x % Q;
        if (c >= rows) return;
        __builtin_nontemporal_store(TL::stage_col8(L, c, q), G(reinterpret_cast<u32x4*>(dst + (r0 + c) * ld + v0 + 8 * q)));
    }
}

// 6144 scored tokens x 2048 x 32000 bf16, keeping e: 755 - 790 us, 1020 - 1066 TFLOP/s (a library product of 8192^3 reaches 1534): 32 k-steps
// a tile, and nothing runs under a tile's first loads, statistics and 0.4 GB of e, since a workgroup takes the CU's LDS.  512 x 1024 x 8192
// fp32 (128-tile): 42 us, 3 x 205 TFLOP/s: 256 tiles, one round, bound by LDS reads.
template <int EDGE, int PARTS, int MODE, bool KTAIL>
__global__ __launch_bounds__(pt::Tile<EDGE>::THREADS, 2) void logits_kernel(LogitsArgs a) {
    typedef pt::Tile<EDGE> TL;
    __shared__ u32x4 lds[TL::LDS_CHUNKS];
    pt::lds_byte_t* L = (pt::lds_byte_t*)lds;
    const int n = a.live.rows();
    const int tb = (n + EDGE - 1) / EDGE, nb = a.ta * tb;
    const int64_t block = block_in_row();
    if (block >= nb) return;
    int ia, ib;
    pt::tile_of(pt::xcd_remap(static_cast<int>(block), nb), a.ta, tb, ia, ib);
    const int v0 = ia * EDGE, r0 = ib * EDGE;
    const char *sa[TL::HL], *sb[TL::HL];
#pragma unroll
    for (int j = 0; j < TL::HL; ++j) {
        const int row = TL::load_row(j);
        sa[j] = a.a + static_cast<size_t>(min(v0 + row, a.vocab - 1)) * a.a_ld + TL::load_chunk(j) * 16;
        int r = min(r0 + row, n - 1);
        if (a.gather) r = a.live.idx[a.live.first + r];
        sb[j] = a.b + static_cast<size_t>(r) * a.b_ld + TL::load_chunk(j) * 16;
    }
    typename TL::Acc acc = {};
    typedef std::conditional_t<PARTS == 1, pt::bf16x8_t, pt::f16x8_t> Of;
    TL::template run<Of, PARTS, KTAIL>(sa, sb, a.a_part, a.b_part, 0, a.steps, a.tail, lds, acc);

    const int place = TL::stack_place(), h = (threadIdx.x >> 5) & 1;
    const int vl = v0 + TL::first_row();              // this lane's first vocabulary entry
    const bool edge = v0 + EDGE > a.vocab;            // uniform: entries past the vocabulary
    const float k = rate_of(a.scale2);
    if constexpr (PARTS == 2) {
        int e[TL::SN];
#pragma unroll
        for (int j = 0; j < TL::SN; ++j) e[j] = -exponent_of(a.scales[0]) - exponent_of(a.scales[1]);
        pt::unscale<TL>(acc, e);
    }
    if (a.scale2 < 0.0f) {
#pragma unroll
        for (int i = 0; i < TL::SM; ++i)
#pragma unroll
            for (int j = 0; j < TL::SN; ++j) acc[i][j] = -acc[i][j];
    }
    lds_barrier();                                    // every wave is done with the operand slabs

    float* smax = reinterpret_cast<float*>(lds);          // [STACKED][EDGE]
    float* ssum = smax + TL::STACKED * EDGE;              // [STACKED][EDGE]
    int col[TL::SN];
    float mx[TL::SN];
#pragma unroll
    for (int j = 0; j < TL::SN; ++j) {
        col[j] = TL::column(j);
        const int r = min(r0 + col[j], n - 1);
        const int64_t t = a.targets[a.live.idx[a.live.first + r]];
        const int y = t < a.vocab ? static_cast<int>(t) - vl : -1;
        // this lane holds entries 8 n .. 8 n + 3 of its share
        const bool mine = y >= 0 && y < 32 * TL::SM && (y & 4) == 0 && r0 + col[j] < n;
        float zt = 0.0f;
        mx[j] = -INFINITY;
        if (edge) {
#pragma unroll
            for (int i = 0; i < TL::SM; ++i)
#pragma unroll
                for (int q = 0; q < 16; ++q)
                    if (vl + 32 * i + 8 * (q >> 2) + (q & 3) >= a.vocab) acc[i][j][q] = -INFINITY;
        }
#pragma unroll
        for (int i = 0; i < TL::SM; ++i)
#pragma unroll
            for (int q = 0; q < 16; ++q) {
                const bool target = 32 * i + 8 * (q >> 2) + (q & 3) == y;   // goes out by itself
                zt = target ? acc[i][j][q] : zt;
                acc[i][j][q] = target ? -INFINITY : acc[i][j][q];
                mx[j] = fmaxf(mx[j], acc[i][j][q]);
                if (q % 4 == 3) __builtin_amdgcn_sched_barrier(0);          // else the compares' masks pile up
            }
        mx[j] = fmaxf(mx[j], __shfl_xor(mx[j], 32, 64));
        if (h == 0) smax[EDGE * place + col[j]] = mx[j];
        if (mine) a.zt[a.live.first + r0 + col[j]] = zt;
    }
    lds_barrier();
#pragma unroll
    for (int j = 0; j < TL::SN; ++j) {
#pragma unroll
        for (int p = 0; p < TL::STACKED; ++p) mx[j] = fmaxf(mx[j], smax[EDGE * p + col[j]]);
        mx[j] *= k;
        const float base = shown(mx[j]);
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < TL::SM; ++i)
#pragma unroll
            for (int q = 0; q < 16; ++q) {
                const float ex = __builtin_amdgcn_exp2f(fmaf(acc[i][j][q], k, -base));
                sum += ex;
                if (MODE == LG_SAVE) acc[i][j][q] = ex;
            }
        sum += __shfl_xor(sum, 32, 64);
        if (h == 0) ssum[EDGE * place + col[j]] = sum;
    }
    lds_barrier();
#pragma unroll
    for (int j = 0; j < TL::SN; ++j)
        if (place == 0 && h == 0) {
            const size_t o = ia * a.rows_pitch + r0 + col[j];
            float sum = ssum[col[j]];
#pragma unroll
            for (int p = 1; p < TL::STACKED; ++p) sum += ssum[EDGE * p + col[j]];
            a.m[o] = mx[j];
            a.s[o] = sum;
        }
    if constexpr (MODE == LG_SAVE) {
        if constexpr (PARTS == 1) {
            lds_barrier();
            const typename TL::Stage st;
            st.put_all_f16(L, acc);
            lds_barrier();
            store_cols<TL>(L, static_cast<uint16_t*>(a.e), a.vp, r0, v0, n - r0);
        } else {
            float* e = static_cast<float*>(a.e);
            for (int pass = 0; pass < TL::F32_PASSES; ++pass) {
                lds_barrier();
                TL::put_f32(L, acc, pass);
                lds_barrier();
                constexpr int Q = EDGE / 4, PER = TL::THREADS / Q;
#pragma unroll 4
                for (int k = 0; k < 128 / PER; ++k) {
                    const int c = 128 * pass + PER * k + static_cast<int>(threadIdx.x) / Q, q = threadIdx.x % Q;
                    if (r0 + c >= n) break;
                    __builtin_nontemporal_store(TL::stage_f32(L, c, q),
                                                G(reinterpret_cast<u32x4*>(e + (static_cast<size_t>(r0) + c) * a.vp + v0 + 4 * q)));
                }
            }
        }
    }
}

// ---------------------------------------------------------------------------
// dz from the kept exp(z - m)
// ---------------------------------------------------------------------------

// e of entry r of a run
__device__ __forceinline__ float e_of(const Run<uint16_t>& x, int r) {
    return static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(x.w[r >> 1] >> (16 * (r & 1)))));
}
__device__ __forceinline__ float e_of(const Run<float>& x, int r) { return x.get(r); }

struct DzArgs {
    const void* e;          // list entry from `kept` on x vocabulary, pitch vp
    const float* m;         // tile x list entry from `kept` on
    int kept;
    const float *ref, *shift;   // list entry: p = e 2^(M - k' ref + shift)
    float scale2;
    size_t m_pitch;
    int m_edge;             // vocabulary entries per tile
    DzTokenArgs tok;
    size_t vp, rows_pitch;
    uint16_t *dz, *dzt;     // rows relative to live.first
    size_t dz_part, dzt_part;
    int32_t* exponents;     // of the tokens' scales, by row of dz
    PackArgs hidden;        // the transpose of hidden for grad_head, by workgroups past the vocabulary's
};

// 64 tokens x 64 entries a workgroup, or 64 tokens x 64 columns of hidden.  Reads 2 (fp32: 4) bytes an element and writes 2 x 2
// (fp32: 2 x 4), HBM-bound (6144 x 32000 bf16 and 2048 columns of hidden: 1.28 GB in 250 us, 5.1 TB/s).  E: what e is kept in.
template <typename E, int PARTS>
__global__ __launch_bounds__(256) void dz_kernel(DzArgs a) {
    __shared__ __attribute__((aligned(16))) uint16_t tile[PARTS][64][72];   // [entry or column][token]
    const int n = a.tok.live.rows();
    // dz's tiles along the vocabulary first, then hidden's along the tokens first (neighbours write one run of a row)
    const int across = static_cast<int>(a.vp / 64), down = static_cast<int>(a.rows_pitch / 64);
    const int past = static_cast<int>(blockIdx.x) - across * down;
    const int r0 = 64 * (past < 0 ? static_cast<int>(blockIdx.x) / across : past % down);
    const int v0 = 64 * (static_cast<int>(blockIdx.x) % across), c0 = past < 0 ? 0 : 64 * (past / down);
    if (r0 >= n) return;
    const int vb = threadIdx.x & 7;            // 8 entries each
    const float k = rate_of(a.scale2);
    // everything that comes from far first: it waits for nothing
    Run<E> x[2];
    int tok[2];
    DzToken t[2];
    float m[2], ref[2], shift[2];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        const int r = min(r0 + static_cast<int>(threadIdx.x >> 3) + 32 * half, n - 1), entry = a.tok.live.first + r;
        tok[half] = a.tok.live.idx[entry];
        if (past < 0) {
            x[half].load(G(static_cast<const E*>(a.e)) + static_cast<size_t>(entry - a.kept) * a.vp, v0 + 8 * vb);
            m[half] = a.m[(v0 / a.m_edge) * a.m_pitch + entry - a.kept];
            ref[half] = a.ref[entry];
            shift[half] = a.shift[entry];
        }
    }
#pragma unroll
    for (int half = 0; half < 2; ++half)
        t[half].load(a.tok, tok[half], a.tok.live.first + min(r0 + static_cast<int>(threadIdx.x >> 3) + 32 * half, n - 1));
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        const int rt = (threadIdx.x >> 3) + 32 * half, r = r0 + rt;
        uint16_t v[8][2];
        const int exponent = t[half].exponent(a.tok);
        if (past >= 0) {   // hidden under its scale, times the least of dz over the token's own: at most 1
            const int up = exponent_of(*a.hidden.scale) + *a.tok.least - exponent;
            const int64_t left = r < n ? a.hidden.cols - c0 - 8 * vb : 0;
            const auto* q = G(static_cast<const E*>(a.hidden.src) + static_cast<size_t>(tok[half]) * a.hidden.ld + c0);
            if (left >= 8) x[half].load(q, 8 * vb);
            else if (left > 0) x[half].load(q, 8 * vb, static_cast<unsigned>(left));
#pragma unroll
            for (int q = 0; q < 8; ++q) half_parts<PARTS>(__builtin_amdgcn_ldexpf(x[half].get(q), up), v[q]);
        } else {
            const int y = t[half].valid(a.tok) ? static_cast<int>(t[half].target) - v0 - 8 * vb : -1;
            const float c = t[half].c;
            // under the token's scale
            const float f = __builtin_amdgcn_ldexpf(c * __builtin_amdgcn_exp2f(fmaf(-ref[half], k, m[half]) + shift[half]), exponent);
            const float dy = __builtin_amdgcn_ldexpf(t[half].dy(), exponent);
            if (v0 == 0 && vb == 0 && r < n) a.exponents[r] = exponent;
            const bool none = r >= n || c == 0.0f;
#pragma unroll
            for (int q = 0; q < 8; ++q)
                half_parts<PARTS>(none || v0 + 8 * vb + q >= a.tok.vocab ? 0.0f : q == y ? dy : -e_of(x[half], q) * f, v[q]);
        }
#pragma unroll
        for (int p = 0; p < PARTS; ++p) {
            if (a.dz && r < n && past < 0) {
                u32x4 w;
#pragma unroll
                for (int k = 0; k < 4; ++k) w[k] = v[2 * k][p] | static_cast<uint32_t>(v[2 * k + 1][p]) << 16;
                G(reinterpret_cast<u32x4*>(a.dz + p * a.dz_part + static_cast<size_t>(r) * a.vp + v0 + 8 * vb))[0] = w;
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) tile[p][8 * vb + k][rt] = v[k][p];
        }
    }
    if (!a.dzt) return;
    uint16_t* out = past < 0 ? a.dzt + static_cast<size_t>(v0) * a.rows_pitch : a.hidden.dst + static_cast<size_t>(c0) * a.rows_pitch;
    const size_t part = past < 0 ? a.dzt_part : a.hidden.part;
    const int64_t rows = past < 0 ? 64 : a.hidden.cols - c0;
    __syncthreads();
#pragma unroll
    for (int p = 0; p < PARTS; ++p)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int v = (threadIdx.x >> 3) + 32 * half, q = 8 * (threadIdx.x & 7);
            if (v >= rows) continue;
            const u32x4 w = *reinterpret_cast<const u32x4*>(&tile[p][v][q]);
            G(reinterpret_cast<u32x4*>(out + p * part + static_cast<size_t>(v) * a.rows_pitch + r0 + q))[0] = w;
        }
}

// ---------------------------------------------------------------------------
// Gradients: C rows = columns of the gradient, C columns = its rows
// ---------------------------------------------------------------------------

struct GradArgs {
    const char* a;          // transposed operand: one row per gradient column
    size_t a_ld, a_part;
    // dz (rows = list entries, whatever memory holds past the last: those columns of C are not stored) or its transpose (rows =
    // vocabulary, zeros from the last list entry to a whole k-step)
    const char* b;
    size_t b_ld, b_part;
    Live live;
    int cols, rows;         // rows: vocabulary; for grad_hidden the list gives them
    int by_token;           // grad_hidden: rows from the list, out rows are its tokens
    int steps;              // k-steps (by_token: over the vocabulary), else the list gives them
    int ta, tb, splits;
    void* out;
    size_t ld;
    float* slab;            // fp32 tiles in accumulator layout, [split][tile][quads][threads] x 16 bytes, or NULL: write out
    int add;                // add to what the slab holds (later chunks of tokens)
    const float* scale;              // of the transposed operand
    const int32_t* exponents;        // of dz's scales: by row (by_token), or the least
};

// A whole 16-byte piece of the output at any element alignment, or the first `left` of its elements.
__device__ __forceinline__ void st_piece(uint16_t* p, const u32x4& v, int left) {
    if (left >= 8) {
        *(global_t<u32x4_el2>*)G(p) = v;
    } else {
#pragma unroll
        for (int e = 0; e < 7; ++e)
            if (e < left) G(p)[e] = static_cast<uint16_t>(v[e >> 1] >> (16 * (e & 1)));
    }
}
__device__ __forceinline__ void st_piece(float* p, const u32x4& v, int left) {
    if (left >= 4) {
        *(global_t<f32x4_el4>*)G(p) = __builtin_bit_cast(f32x4_t, v);
    } else {
#pragma unroll
        for (int e = 0; e < 3; ++e)
            if (e < left) G(p)[e] = __uint_as_float(v[e]);
    }
}

// T: the gradient's type.  6144 tokens x 2048 x 32000 bf16: 795 us (grad_hidden: 24 x 8 tiles of 500 steps, a quarter of the CUs without
// one) and 690 us (grad_head: 125 x 8 tiles of 96 steps, 665 with bf16 operands: the clock), 1013 and 1167 TFLOP/s.
template <int EDGE, int PARTS, typename T>
__global__ __launch_bounds__(pt::Tile<EDGE>::THREADS, 2) void grad_kernel(GradArgs a) {
    typedef pt::Tile<EDGE> TL;
    __shared__ u32x4 lds[TL::LDS_CHUNKS];
    pt::lds_byte_t* L = (pt::lds_byte_t*)lds;
    const int n = a.live.rows();
    const int rows = a.by_token ? n : a.rows, all = a.by_token ? a.steps : (n + pt::KS - 1) / pt::KS;
    const int tb = (rows + EDGE - 1) / EDGE, nb = a.ta * tb;
    if (static_cast<int>(blockIdx.x) >= nb) return;
    const int tile = pt::xcd_remap(blockIdx.x, nb);
    int ia, ib;
    pt::tile_of(tile, a.ta, tb, ia, ib);
    const int c0 = ia * EDGE, r0 = ib * EDGE;
    const int split = blockIdx.y;
    const int k_first = static_cast<int>(static_cast<int64_t>(all) * split / a.splits);
    const int steps = static_cast<int>(static_cast<int64_t>(all) * (split + 1) / a.splits) - k_first;
    typename TL::Acc acc = {};
    if (steps > 0) {
        const char *sa[TL::HL], *sb[TL::HL];
#pragma unroll
        for (int j = 0; j < TL::HL; ++j) {
            const int row = TL::load_row(j);
            sa[j] = a.a + static_cast<size_t>(min(c0 + row, a.cols - 1)) * a.a_ld + TL::load_chunk(j) * 16;
            sb[j] = a.b + static_cast<size_t>(r0 + row) * a.b_ld + TL::load_chunk(j) * 16;   // padded to the tile
        }
        TL::template run<pt::f16x8_t, PARTS, false>(sa, sb, a.a_part, a.b_part, static_cast<size_t>(k_first) * (pt::KS * 2), steps, 0, lds, acc);
    }
    const int up = exponent_of(*a.scale);
    int down[TL::SN];
#pragma unroll
    for (int j = 0; j < TL::SN; ++j) down[j] = -up - a.exponents[a.by_token ? min(r0 + TL::column(j), n - 1) : 0];
    pt::unscale<TL>(acc, down);
    if (a.slab) {
        float* s = a.slab + (static_cast<size_t>(split) * a.ta * a.tb + tile) * (EDGE * EDGE) + threadIdx.x * 4;
#pragma unroll
        for (int i = 0; i < TL::SM; ++i)
#pragma unroll
            for (int j = 0; j < TL::SN; ++j)
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    float* p = s + static_cast<size_t>((i * TL::SN + j) * 4 + g) * (TL::THREADS * 4);
                    float4 v = make_float4(acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2], acc[i][j][4 * g + 3]);
                    if (a.add) {
                        const float4 o = ld_f4(p);
                        v = make_float4(v.x + o.x, v.y + o.y, v.z + o.z, v.w + o.w);
                    }
                    st_f4(p, v);
                }
        return;
    }
    T* out = static_cast<T*>(a.out);
    constexpr int E = 16 / sizeof(T), Q = EDGE / E, PER = TL::THREADS / Q;   // elements of a piece, pieces of a row, rows at a time
    constexpr int PASSES = sizeof(T) == 2 ? 1 : TL::F32_PASSES, COLS = EDGE / PASSES;
    for (int pass = 0; pass < PASSES; ++pass) {
        lds_barrier();
        if constexpr (sizeof(T) == 2) {
            const typename TL::Stage st;
            st.put_all(L, acc);
        } else {
            TL::put_f32(L, acc, pass);
        }
        lds_barrier();
#pragma unroll 4
        for (int k = 0; k < COLS / PER; ++k) {
            const int c = COLS * pass + PER * k + static_cast<int>(threadIdx.x) / Q, q = threadIdx.x % Q;
            if (r0 + c >= rows) continue;
            const size_t row = a.by_token ? a.live.idx[a.live.first + r0 + c] : r0 + c;
            u32x4 v;
            if constexpr (sizeof(T) == 2) v = TL::stage_col8(L, c, q);
            else v = TL::stage_f32(L, c, q);
            st_piece(out + row * a.ld + c0 + E * q, v, a.cols - c0 - E * q);
        }
    }
}

// Sums the splits' tiles in order and writes the gradient; one wave per 32 x 32 block.
template <int EDGE> __global__ __launch_bounds__(256) void slab_sum_kernel(GradArgs a, int dt) {
    typedef pt::Tile<EDGE> TL;
    constexpr int BLOCKS = (EDGE / 32) * (EDGE / 32), PER = TL::SM * TL::SN;   // blocks of a tile, of a wave's share
    __shared__ float tile[4][32][33];   // [wave][gradient row][gradient column]
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int block = blockIdx.x * 4 + wave, t = block / BLOCKS, b = block % BLOCKS;
    const int rows = a.by_token ? a.live.rows() : a.rows;
    const int tb = (rows + EDGE - 1) / EDGE;
    if (t >= a.ta * tb) return;
    int ia, ib;
    pt::tile_of(t, a.ta, tb, ia, ib);
    const int w = b / PER, i = (b % PER) / TL::SN, j = b % TL::SN;
    const int c0 = ia * EDGE + TL::share_row(w) + 32 * i, r0 = ib * EDGE + TL::share_col(w) + 32 * j;
    if (c0 >= a.cols || r0 >= rows) return;
    float4 v[4] = {};
#pragma unroll 4
    for (int s = 0; s < a.splits; ++s) {
        const float* p = a.slab + (static_cast<size_t>(s) * a.ta * a.tb + t) * (EDGE * EDGE) + (64 * w + lane) * 4;
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const float4 x = ld_f4(p + static_cast<size_t>((i * TL::SN + j) * 4 + g) * (TL::THREADS * 4));
            v[g] = make_float4(v[g].x + x.x, v[g].y + x.y, v[g].z + x.z, v[g].w + x.w);
        }
    }
#pragma unroll
    for (int g = 0; g < 4; ++g) {
        float* q = &tile[wave][lane & 31][8 * g + 4 * (lane >> 5)];
        q[0] = v[g].x; q[1] = v[g].y; q[2] = v[g].z; q[3] = v[g].w;
    }
    __builtin_amdgcn_wave_barrier();   // one wave's LDS: its writes come before its reads
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    const int c = c0 + (lane & 31);
    if (c >= a.cols) return;
#pragma unroll 4
    for (int k = 0; k < 16; ++k) {
        const int r = 2 * k + (lane >> 5);
        if (r0 + r >= rows) continue;
        const size_t row = a.by_token ? a.live.idx[a.live.first + r0 + r] : r0 + r;
        st_dt(a.out, row * a.ld + c, tile[wave][r][lane & 31], dt);
    }
}

// ---------------------------------------------------------------------------
// Few tokens: the head is read once
// ---------------------------------------------------------------------------

typedef float f32x4m_t __attribute__((ext_vector_type(4)));

// x as three bf16 parts, exact to 24 bits: the first two truncated (so nothing overflows), the last rounded.
__device__ __forceinline__ void split3(float x, uint16_t (&p)[3]) {
    const uint32_t hi = __float_as_uint(x) & 0xffff0000u;
    const bool fin = (hi & 0x7f800000u) != 0x7f800000u;
    p[0] = static_cast<uint16_t>((fin ? hi : hi | (x != x ? 0x00400000u : 0u)) >> 16);
    const float r = fin ? x - __uint_as_float(hi) : 0.0f;
    const uint32_t mid = __float_as_uint(r) & 0xffff0000u;
    p[1] = static_cast<uint16_t>(mid >> 16);
    p[2] = f32_to_bf16(r - __uint_as_float(mid));
}
// The products of parts that few_kernel sums, small ones first, two bits each: those whose indexes add to at most 2.
template <int PARTS> struct FewOrder;
template <> struct FewOrder<1> { static constexpr int N = 1; static constexpr unsigned W = 0, H = 0; };
template <> struct FewOrder<3> {
    static constexpr int N = 6;                       // (2,0) (0,2) (1,1) (1,0) (0,1) (0,0)
    static constexpr unsigned W = 2u | 0u << 2 | 1u << 4 | 1u << 6, H = 0u | 2u << 2 | 1u << 4 | 0u << 6 | 1u << 8;
};

// 8 values of k of one row from column k, zero past the last column, as bf16 parts (of x scale in fp32).
template <typename T, int PARTS> __device__ __forceinline__ void few_load(const void* base, size_t off, int k, int cols, float scale, u32x4 (&out)[PARTS]) {
    Run<T> x;
    const auto* row = G(static_cast<const T*>(base) + off);
    if (k + 8 <= cols) x.load(row, k);
    else if (k < cols) x.load(row, k, cols - k);
    if constexpr (PARTS == 1) {
        out[0] = x.w;
    } else {
        uint16_t v[8][3];
#pragma unroll
        for (int e = 0; e < 8; ++e) split3(x.get(e) * scale, v[e]);
#pragma unroll
        for (int p = 0; p < PARTS; ++p)
#pragma unroll
            for (int e = 0; e < 4; ++e) out[p][e] = v[2 * e][p] | static_cast<uint32_t>(v[2 * e + 1][p]) << 16;
    }
}

struct FewArgs {
    const void *head, *hidden;
    size_t ld_head, ld_hidden;
    const int64_t* targets;
    int tokens, cols, vocab, tiles;
    float scale2;
    float *m, *s, *zt;      // M and S: token x tile; target's acc by token
    void* e;                // 2^(k' acc - M), token x vocabulary (pitch vp), fp16 in bf16 calls, else fp32; or NULL
    size_t vp;
    const uint32_t* absmax; // fp32: scan_kernel's partials for hidden, or NULL: hidden as it is
};

// FEW_ROWS entries x up to 16 NT tokens a workgroup; its four waves take 64 values of k in turn.  Vocabulary
// along the accumulator rows, tokens along the columns (16 x 16 MFMA).  HBM-bound: the head once,
// cols x vocab elements (one token x 2048 x 32000: 25.6 us, 5.1 TB/s); hidden comes from the caches, and for 64 tokens
// that is what it waits for (52 us).
template <typename T, int PARTS, int NT>
__global__ __launch_bounds__(256, NT == 1 ? 4 : 1) void few_kernel(FewArgs a) {
    constexpr int TOK = 16 * NT, GROUPS = 256 / TOK, PER = FEW_ROWS / GROUPS;   // at the end: threads a token, entries a thread
    __shared__ float red[4][FEW_ROWS][TOK + 1];
    __shared__ float part[2][GROUPS][TOK];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int v0 = blockIdx.x * FEW_ROWS, ln = lane & 15, kg = 8 * (lane >> 4);
    size_t wo[2], ho[NT];
#pragma unroll
    for (int r = 0; r < 2; ++r) wo[r] = static_cast<size_t>(min(v0 + 16 * r + ln, a.vocab - 1)) * a.ld_head;
#pragma unroll
    for (int t = 0; t < NT; ++t) ho[t] = static_cast<size_t>(min(16 * t + ln, a.tokens - 1)) * a.ld_hidden;
    const float hs = PARTS == 1 || !a.absmax ? 1.0f : operand_scale(a.absmax, false, reinterpret_cast<uint32_t*>(red));
    f32x4m_t acc[2][NT] = {};
    constexpr int DEEP = PARTS == 1 ? 2 : 1;   // 64-value runs of k in flight (4: 31.7 us for one token and 32000 x 2048, 2: 29.1)
    for (int k0 = 64 * wave; k0 < a.cols; k0 += 256 * DEEP) {
        u32x4 w[2 * DEEP][2][PARTS], h[2 * DEEP][NT][PARTS];
#pragma unroll
        for (int b = 0; b < 2 * DEEP; ++b) {
            const int k = k0 + 256 * (b >> 1) + 32 * (b & 1) + kg;
#pragma unroll
            for (int r = 0; r < 2; ++r) few_load<T, PARTS>(a.head, wo[r], k, a.cols, 1.0f, w[b][r]);
#pragma unroll
            for (int t = 0; t < NT; ++t) few_load<T, PARTS>(a.hidden, ho[t], k, a.cols, hs, h[b][t]);
        }
#pragma unroll
        for (int b = 0; b < 2 * DEEP; ++b) {
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int q = 0; q < FewOrder<PARTS>::N; ++q)
                        acc[r][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                            __builtin_bit_cast(pt::bf16x8_t, w[b][r][(FewOrder<PARTS>::W >> 2 * q) & 3u]),
                            __builtin_bit_cast(pt::bf16x8_t, h[b][t][(FewOrder<PARTS>::H >> 2 * q) & 3u]), acc[r][t], 0, 0, 0);
        }
    }
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) red[wave][16 * r + 4 * (lane >> 4) + e][16 * t + ln] = acc[r][t][e];
    __syncthreads();
    const float k = rate_of(a.scale2);
    const int t = threadIdx.x % TOK, g = threadIdx.x / TOK, v = v0 + PER * g;   // this thread's entries from v on
    const int64_t y = t < a.tokens ? a.targets[t] - v : -1;
    float z[PER], m = -INFINITY, sum = 0.0f;
#pragma unroll
    for (int r = 0; r < PER; ++r) {
        z[r] = red[0][PER * g + r][t] + red[1][PER * g + r][t] + red[2][PER * g + r][t] + red[3][PER * g + r][t];
        if constexpr (PARTS == 3) z[r] = __builtin_amdgcn_ldexpf(z[r], -exponent_of(hs));
        if (a.scale2 < 0.0f) z[r] = -z[r];
        if (v + r >= a.vocab) {
            z[r] = -INFINITY;
        } else if (r == y) {   // the target goes out by itself
            a.zt[t] = z[r];
            z[r] = -INFINITY;
        }
        m = fmaxf(m, z[r]);
    }
    part[0][g][t] = m;
    __syncthreads();
#pragma unroll
    for (int h = 0; h < GROUPS; ++h) m = fmaxf(m, part[0][h][t]);
    m *= k;
    uint16_t e16[PER];
#pragma unroll
    for (int r = 0; r < PER; ++r) {
        const float e = __builtin_amdgcn_exp2f(fmaf(z[r], k, -shown(m)));
        if constexpr (sizeof(T) == 2) e16[r] = __builtin_bit_cast(uint16_t, static_cast<_Float16>(e));
        else if (a.e && t < a.tokens) static_cast<float*>(a.e)[t * a.vp + v + r] = e;
        sum += e;
    }
    part[1][g][t] = sum;
    __syncthreads();
    if (t >= a.tokens) return;
    if (sizeof(T) == 2 && a.e) {
        uint32_t w[PER / 2];
#pragma unroll
        for (int r = 0; r < PER / 2; ++r) w[r] = e16[2 * r] | static_cast<uint32_t>(e16[2 * r + 1]) << 16;
        __builtin_memcpy(__builtin_assume_aligned(static_cast<uint16_t*>(a.e) + t * a.vp + v, 2 * PER), w, sizeof(w));
    }
    if (g == 0) {
        sum = part[1][0][t];
#pragma unroll
        for (int h = 1; h < GROUPS; ++h) sum += part[1][h][t];
        a.m[static_cast<size_t>(t) * a.tiles + blockIdx.x] = m;
        a.s[static_cast<size_t>(t) * a.tiles + blockIdx.x] = sum;
    }
}

// ---------------------------------------------------------------------------
// Few tokens: gradients
// ---------------------------------------------------------------------------
// Both have gradient columns along the accumulator rows and k (vocabulary entries, or tokens) across rows of an operand that
// lies k-major.  A lane reads 8 columns (16 bytes in bf16) of 8 rows of k, which transposed in its registers are the A
// fragments of 8 MFMAs: MFMA j takes column 8 p + j of lane group p.  Lane i of 16 takes the run p = 4 (i & 3) + (i >> 2), so
// that of C row 4 q + e, run 4 e + q, the four lanes q that share a C column hold adjacent runs.
// dz is formed from e where it is used.  One token's rounded dz would be its whole gradient's error, so dz goes as two
// bf16 parts, hi + lo (fp32: three, as everything here; there hidden is scaled).

constexpr int FEW_STRIP = 128;       // gradient columns of a wave

struct FewGradArgs {
    const void *head, *hidden;
    size_t ld_head, ld_hidden;
    const int64_t* targets;
    int tokens, cols, vocab, tiles, strips, splits;
    float scale2, scale;
    const void* e;                     // token x vocabulary, pitch vp (FewArgs)
    size_t vp;
    const float* m;                    // token x tile
    const float *logp, *ref, *shift;   // by token, as in DzArgs
    const float* grad_logp;
    float* slab;                       // [split][strip][j][4 registers of every 16 tokens][lane]
    void *grad_hidden, *grad_head;     // or NULL
    size_t ld_grad_hidden, ld_grad_head;
    const uint32_t* absmax;            // fp32: scan_kernel's partials for hidden
};

// What dz of a token takes.
struct FewToken {
    float c = 0.0f, ref = 0.0f, shift = 0.0f, dy = 0.0f;
    int y = -1;
    __device__ __forceinline__ void load(const FewGradArgs& a, int t) {
        if (t >= a.tokens) return;
        const int64_t target = a.targets[t];
        if (target < 0) return;
        y = target < a.vocab ? static_cast<int>(target) : -1;
        c = a.scale * a.grad_logp[t];
        ref = a.ref[t];
        shift = a.shift[t];
        dy = -c * expm1f(a.logp[t]);
    }
    __device__ __forceinline__ float factor(float m, float k) const { return c * __builtin_amdgcn_exp2f(fmaf(-ref, k, m) + shift); }
    // e of entry v, times the factor of its tile
    __device__ __forceinline__ float dz(float e, float f, int v, int vocab) const {
        return c == 0.0f || v >= vocab ? 0.0f : v == y ? dy : -e * f;
    }
};
// Parts of dz: hi + lo, or three.
template <int PARTS> struct DzParts { static constexpr int N = PARTS == 1 ? 2 : 3; };
__device__ __forceinline__ void dz_parts(float x, uint16_t (&p)[2]) {
    p[0] = f32_to_bf16(x);
    p[1] = f32_to_bf16(x - bf16_to_f32(p[0]));
}
__device__ __forceinline__ void dz_parts(float x, uint16_t (&p)[3]) { split3(x, p); }

// Column j of 8 rows (times scale, in fp32) as an A fragment.
__device__ __forceinline__ void few_fragment(const Run<uint16_t> (&r)[8], int j, float, u32x4 (&out)[1]) {
#pragma unroll
    for (int p = 0; p < 4; ++p)
        out[0][p] = __builtin_amdgcn_perm(r[2 * p + 1].w[j >> 1], r[2 * p].w[j >> 1], (j & 1) ? 0x07060302u : 0x05040100u);
}
__device__ __forceinline__ void few_fragment(const Run<float> (&r)[8], int j, float scale, u32x4 (&out)[3]) {
    uint16_t v[8][3];
#pragma unroll
    for (int k = 0; k < 8; ++k) split3(r[k].get(j) * scale, v[k]);
#pragma unroll
    for (int p = 0; p < 3; ++p)
#pragma unroll
        for (int e = 0; e < 4; ++e) out[p][e] = v[2 * e][p] | static_cast<uint32_t>(v[2 * e + 1][p]) << 16;
}
// a times b over their parts, small products first.
template <int PARTS>
__device__ __forceinline__ void few_mfma(f32x4m_t& acc, const u32x4 (&a)[PARTS], const u32x4 (&b)[DzParts<PARTS>::N]) {
    constexpr int N = PARTS == 1 ? 2 : FewOrder<3>::N;
#pragma unroll
    for (int q = 0; q < N; ++q) {
        const int pa = PARTS == 1 ? 0 : (FewOrder<3>::W >> 2 * q) & 3u, pb = PARTS == 1 ? 1 - q : (FewOrder<3>::H >> 2 * q) & 3u;
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(pt::bf16x8_t, a[pa]), __builtin_bit_cast(pt::bf16x8_t, b[pb]),
                                                      acc, 0, 0, 0);
    }
}
__device__ __forceinline__ int few_column(int lane) { return 8 * (4 * (lane & 3) + ((lane & 15) >> 2)); }   // of the strip
template <typename T> __device__ __forceinline__ void few_row(Run<T>& r, const T* row, int col, int cols) {
    if (col + 8 <= cols) r.load(G(row), col);
    else if (col < cols) r.load(G(row), col, cols - col);
}

// grad_hidden: a strip of columns and a run of vocabulary tiles a workgroup, its four waves taking tiles in turn; their sums
// are put together in LDS.  HBM-bound: head once (2 tokens x 2048 x 32000: 24 us, 5.5 TB/s, from the
// last-level cache in part; 6 x 3176 x 52257: 127 us, 2.6 TB/s, where few_kernel's plain rows reach 2.8).  16 NT tokens, the
// registers allowing; blockIdx.y: which of them.
template <typename T, int PARTS, int NT>
__global__ __launch_bounds__(256, NT == 1 ? 3 : 2) void few_hidden_kernel(FewGradArgs a) {
    constexpr int REGS = 4 * NT, DP = DzParts<PARTS>::N;
    constexpr bool AHEAD = PARTS == 1 && NT <= 2;   // registers for the next tile's rows
    const int t0 = 16 * NT * blockIdx.y;
    __shared__ float red[4][REGS][64];
    const int lane = threadIdx.x & 63, wave = pt::wave_id(), q = lane >> 4;
    const int strip = blockIdx.x % a.strips, split = blockIdx.x / a.strips;
    const int col = FEW_STRIP * strip + few_column(lane);
    const int first = static_cast<int>(static_cast<int64_t>(a.tiles) * split / a.splits);
    const int last = static_cast<int>(static_cast<int64_t>(a.tiles) * (split + 1) / a.splits);
    const float k = rate_of(a.scale2);
    const T* head = static_cast<const T*>(a.head);
    const T* e = static_cast<const T*>(a.e);
    FewToken tok[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) tok[n].load(a, t0 + 16 * n + (lane & 15));
    struct Chunk {
        Run<T> rows[8], e[NT];
        float m[NT];
    };
    auto load = [&](Chunk& c, int tile) {
        const int v = FEW_ROWS * tile + 8 * q;
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            c.rows[r] = Run<T>{};
            few_row(c.rows[r], head + static_cast<size_t>(min(v + r, a.vocab - 1)) * a.ld_head, col, a.cols);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int t = min(t0 + 16 * n + (lane & 15), a.tokens - 1);
            c.e[n].load(G(e + t * a.vp), v);
            c.m[n] = a.m[static_cast<size_t>(t) * a.tiles + tile];
        }
    };
    f32x4m_t acc[8][NT] = {};
    Chunk now, next;
    if (AHEAD && first + wave < last) load(now, first + wave);
    for (int tile = first + wave; tile < last; tile += 4) {
        if (!AHEAD) load(now, tile);
        else if (tile + 4 < last) load(next, tile + 4);
        u32x4 b[NT][DP];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const float f = tok[n].factor(now.m[n], k);
            uint16_t v[8][DP];
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                dz_parts(tok[n].dz(e_of(now.e[n], r), f, FEW_ROWS * tile + 8 * q + r, a.vocab), v[r]);
            }
#pragma unroll
            for (int p = 0; p < DP; ++p)
#pragma unroll
                for (int r = 0; r < 4; ++r) b[n][p][r] = v[2 * r][p] | static_cast<uint32_t>(v[2 * r + 1][p]) << 16;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            u32x4 w[PARTS];
            few_fragment(now.rows, j, 1.0f, w);
#pragma unroll
            for (int n = 0; n < NT; ++n) few_mfma<PARTS>(acc[j][n], w, b[n]);
        }
        if (AHEAD) now = next;
    }
    const int all = REGS * gridDim.y;
    float* slab = a.slab + (static_cast<size_t>(split) * a.strips + strip) * (8 * all * 64) + REGS * blockIdx.y * 64;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        __syncthreads();
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int r = 0; r < 4; ++r) red[wave][4 * n + r][lane] = acc[j][n][r];
        __syncthreads();
        for (int x = wave; x < REGS; x += 4)
            slab[(j * all + x) * 64 + lane] = red[0][x][lane] + red[1][x][lane] + red[2][x][lane] + red[3][x][lane];
    }
}

// The splits' sums, in order, to grad_hidden; zeros for tokens that are not scored.  An element a thread.
template <typename T, int BLOCKS> __global__ __launch_bounds__(256) void few_sum_kernel(FewGradArgs a) {
    constexpr int REGS = 4 * BLOCKS;
    const int i = blockIdx.x * 256 + threadIdx.x, lane = i & 63, x = (i >> 6) % REGS, js = (i >> 6) / REGS;
    const int t = 16 * (x >> 2) + (lane & 15), col = FEW_STRIP * (js >> 3) + 8 * (4 * (x & 3) + (lane >> 4)) + (js & 7);
    if (t >= a.tokens || col >= a.cols) return;
    const size_t step = static_cast<size_t>(a.strips) * (8 * REGS * 64);
    float v = 0.0f;
#pragma unroll 8
    for (int s = 0; s < a.splits; ++s) v += a.slab[s * step + i];
    st_el<T>(a.grad_hidden, t * a.ld_grad_hidden + col, a.targets[t] < 0 ? 0.0f : v);
}

// grad_head: a tile of FEW_ROWS entries a workgroup, whose dz is formed once in LDS; its waves take strips of columns in turn.
// Bound by the writes: head's size once (2 tokens x 2048 x 32000: 31 us, 4.2 TB/s; 6 x 3176 x 52257: 66 us, 5 TB/s).  KS: runs
// of 32 tokens (64 tokens: 51 us, the products and their operands' way through L2).
template <typename T, int PARTS, int KS> __global__ __launch_bounds__(256, 2) void few_head_kernel(FewGradArgs a) {
    constexpr int DP = DzParts<PARTS>::N, VB = FEW_ROWS / 16;
    __shared__ __attribute__((aligned(16))) uint16_t tile[DP][FEW_ROWS][32 * KS + 8];   // [entry][token]
    const int lane = threadIdx.x & 63, wave = pt::wave_id(), q = lane >> 4;
    const int v0 = blockIdx.x * FEW_ROWS;
    const float k = rate_of(a.scale2);
    const T* e = static_cast<const T*>(a.e);
    const float hs = PARTS == 1 ? 1.0f : operand_scale(a.absmax, false, reinterpret_cast<uint32_t*>(tile));
    const unsigned long long live = __ballot(lane < a.tokens && a.targets[min(lane, max(a.tokens - 1, 0))] >= 0);
    const int t = threadIdx.x % (32 * KS), r0 = 8 * (threadIdx.x / (32 * KS));   // a token and 8 entries a thread
    if (r0 < FEW_ROWS) {
        FewToken tok;
        Run<T> x;
        float f = 0.0f;
        if (live >> t & 1u) {
            x.load(G(e + t * a.vp), v0 + r0);
            tok.load(a, t);
            f = tok.factor(a.m[static_cast<size_t>(t) * a.tiles + blockIdx.x], k);
        }
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            uint16_t p[DP];
            dz_parts(tok.dz(e_of(x, r), f, v0 + r0 + r, a.vocab), p);
#pragma unroll
            for (int d = 0; d < DP; ++d) tile[d][r0 + r][t] = p[d];
        }
    }
    __syncthreads();
    const T* hidden = static_cast<const T*>(a.hidden);
    T* out = static_cast<T*>(a.grad_head);
    for (int strip = blockIdx.y * 4 + wave; strip < a.strips; strip += 4 * gridDim.y) {
        const int col = FEW_STRIP * strip + few_column(lane);
        f32x4m_t acc[8][VB] = {};
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            Run<T> rows[8];
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                const int t = 32 * s + 8 * q + r;
                if (live >> t & 1u) few_row(rows[r], hidden + t * a.ld_hidden, col, a.cols);   // whatever others hold counts for nothing
            }
            u32x4 b[VB][DP];
#pragma unroll
            for (int n = 0; n < VB; ++n)
#pragma unroll
                for (int d = 0; d < DP; ++d) b[n][d] = *reinterpret_cast<const u32x4*>(&tile[d][16 * n + (lane & 15)][32 * s + 8 * q]);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                u32x4 w[PARTS];
                few_fragment(rows, j, hs, w);
#pragma unroll
                for (int n = 0; n < VB; ++n) few_mfma<PARTS>(acc[j][n], w, b[n]);
            }
        }
#pragma unroll
        for (int n = 0; n < VB; ++n) {
            const int v = v0 + 16 * n + (lane & 15);
            if (v >= a.vocab) continue;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int c = FEW_STRIP * strip + 8 * (4 * r + q);
                T* p = out + static_cast<size_t>(v) * a.ld_grad_head + c;
                if constexpr (sizeof(T) == 2) {
                    u32x4 w;
#pragma unroll
                    for (int j = 0; j < 4; ++j) w[j] = pack_bf16x2(acc[2 * j][n][r], acc[2 * j + 1][n][r]);
                    st_piece(p, w, a.cols - c);
                } else {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        u32x4 w;
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            w[j] = __float_as_uint(__builtin_amdgcn_ldexpf(acc[4 * h + j][n][r], -exponent_of(hs)));
                        st_piece(p + 4 * h, w, a.cols - c - 4 * h);
                    }
                }
            }
        }
    }
}

// ---------------------------------------------------------------------------
// lse and logp from the tiles' statistics
// ---------------------------------------------------------------------------

struct CombineArgs {
    const float *m, *s, *zt;
    size_t tile_stride, row_stride;
    int tiles;
    const int64_t* targets;
    int64_t vocab;
    float *logp, *lse;            // or NULL: what is kept is enough
    Live live;                    // no list: every token, in order (then unscored ones are zeroed here)
    int64_t tokens;
    float scale2;
    float *kept_logp, *kept_ref, *kept_shift;   // by list entry, for the backward pass (DzArgs), or NULL
    const uint32_t* absmax;       // scan_kernel's partials, or NULL: the scales of hidden and head are known or not needed
    float* scales;
};

// 2^(a - b) for a <= b, with equal infinities taken as equal
__device__ __forceinline__ float pow2_diff(float a, float b) { return a == b ? 1.0f : __builtin_amdgcn_exp2f(a - b); }

// TOK tokens a workgroup, 256 / TOK threads each.
template <int TOK>
__global__ __launch_bounds__(256) void combine_kernel(CombineArgs a) {
    constexpr int NP = 256 / TOK;
    __shared__ float sm[NP][TOK], ss[NP][TOK];
    const int tk = threadIdx.x % TOK, part = threadIdx.x / TOK;
    const int64_t row = block_in_row() * TOK + tk;
    if (a.absmax && block_in_row() < 2) {   // there are at least PAD / TOK
        const bool head = block_in_row() == 1;
        const float scale = operand_scale(a.absmax, head, reinterpret_cast<uint32_t*>(&sm[0][0]));
        if (threadIdx.x == 0) a.scales[head] = scale;
    }
    const int64_t n = a.live.idx ? a.live.rows() : a.tokens;
    const float k = rate_of(a.scale2);
    float m = -INFINITY, s = 0.0f;
    if (row < n)
#pragma unroll 4
        for (int t = part; t < a.tiles; t += NP) {
            const size_t o = t * a.tile_stride + row * a.row_stride;
            const float mt = a.m[o], st = a.s[o], up = fmaxf(m, mt);
            s = s * pow2_diff(m, up) + st * pow2_diff(mt, up);
            m = up;
        }
    sm[part][tk] = m;
    ss[part][tk] = s;
    for (int o = NP / 2; o > 0; o >>= 1) {
        __syncthreads();
        if (part < o) {
            const float m2 = sm[part + o][tk], s2 = ss[part + o][tk], up = fmaxf(m, m2);
            s = s * pow2_diff(m, up) + s2 * pow2_diff(m2, up);
            m = up;
            sm[part][tk] = m;
            ss[part][tk] = s;
        }
    }
    if (part != 0 || row >= n) return;
    const int64_t entry = a.live.first + row, tok = a.live.idx ? a.live.idx[entry] : row, y = a.targets[tok];
    // s is the sum without the target, if there is one
    float logp, lse = (m + log2f(s)) * LN2, ref = 0.0f, shift = -(m + log2f(s));
    if (y < 0) {
        logp = lse = 0.0f;
    } else if (y >= a.vocab) {
        logp = NAN;
    } else {
        const float zt = a.zt[entry], d = fmaf(-zt, k, m);
        if (d < 80.0f) {
            logp = 0.0f - log1pf(s * __builtin_amdgcn_exp2f(d));
            lse = zt * k * LN2 - logp;
            ref = zt;
            shift = logp * LOG2E;
        } else {
            logp = -(d + log2f(s)) * LN2;     // here 1 is nothing beside the sum
        }
    }
    if (a.logp) {
        a.logp[tok] = logp;
        a.lse[tok] = lse;
    }
    if (a.kept_logp) {
        a.kept_logp[entry] = logp;
        a.kept_ref[entry] = ref;
        a.kept_shift[entry] = shift;
    }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

#define TL_TRY(expr)                       \
    do {                                   \
        const hipError_t e_ = (expr);      \
        if (e_ != hipSuccess) return e_;   \
    } while (0)

struct Bump {
    size_t at = 0;
    size_t take(size_t bytes) {
        const size_t o = at;
        at += (bytes + 255) / 256 * 256;
        return o;
    }
};

// Which tile serves a product of so many 256 x 256 tiles.
int edge_for(int64_t tiles) { return tiles < FEW_TILES ? 128 : 256; }

// What both directions derive from the shape.
struct Shape {
    int64_t tokens, cols, vocab;
    int parts;
    int64_t tp, vp, dp;      // padded to PAD, PAD, the k-step
    int edge;                // tile of the logits' product
    bool few;                // forward and backward as for few tokens; a forward pass that keeps nothing has its own rule
    int few_tiles;           // of FEW_ROWS entries
    bool direct_hidden, direct_head;   // operands that the products can read where they are: bf16 in whole 16-byte chunks
    Shape(int64_t t, int64_t d, int64_t v, int dtype, const void* hidden, int64_t ld_hidden, const void* head, int64_t ld_head)
        : tokens(t), cols(d), vocab(v), parts(dtype == MUON_BF16 ? 1 : 2), tp(up(std::max<int64_t>(t, 1), PAD)), vp(up(v, PAD)),
          dp(up(d, pt::KS)), edge(edge_for(tp / PAD * (vp / PAD))), few(t <= FEW_TOKENS),
          few_tiles(static_cast<int>(ceil_div(v, FEW_ROWS))) {
        const bool ok = dtype == MUON_BF16 && d % 8 == 0;
        direct_hidden = ok && reinterpret_cast<uintptr_t>(hidden) % 16 == 0 && ld_hidden % 8 == 0;
        direct_head = ok && reinterpret_cast<uintptr_t>(head) % 16 == 0 && ld_head % 8 == 0;
    }
    int ta() const { return static_cast<int>(vp / edge); }
};

// The buffer that the forward pass keeps: e, the tiles' M, what combine_kernel keeps by token, and (many tokens) the list.
struct SavedPlan {
    size_t e, m, logp, ref, shift, idx, count, scales, bytes;
    explicit SavedPlan(const Shape& sh) {
        Bump b;
        const size_t rows = static_cast<size_t>(sh.few ? sh.tokens : sh.tp);
        e = b.take((sh.parts == 1 ? 2 : 4) * rows * sh.vp);
        m = b.take(sizeof(float) * rows * (sh.few ? sh.few_tiles : sh.ta()));
        logp = b.take(sizeof(float) * rows);
        ref = b.take(sizeof(float) * rows);
        shift = b.take(sizeof(float) * rows);
        idx = b.take(sh.few ? 0 : sizeof(int32_t) * rows);
        count = b.take(sizeof(int32_t));
        scales = b.take(2 * sizeof(float));
        bytes = b.at;
    }
};

struct ForwardPlan {
    Shape sh;
    bool few;
    size_t idx, count, hidden, head, m, s, zt, absmax, scales, bytes;
    explicit ForwardPlan(const muon_token_logp_args& a)
        : sh(a.tokens, a.cols, a.vocab, a.dtype, a.hidden, a.ld_hidden, a.head, a.ld_head) {
        // Beyond 32 tokens few_kernel waits more on hidden than on a head of many tiles, and the large tile takes over where it
        // can read both in place (48 tokens x 2048 bf16: 32000 entries 50 against 35 us, 16000 29 against 29, 8000 19
        // against 27; fp32 or copies: 126 against 234 us)
        const bool large = sh.direct_head && sh.direct_hidden && a.tokens > 32 && sh.few_tiles > 2 * CUS;
        few = a.saved ? sh.few : a.tokens <= FEW_TOKENS && !large;
        Bump b;
        const size_t part = sizeof(uint16_t) * sh.parts * sh.dp;
        idx = b.take(few || a.saved ? 0 : sizeof(int32_t) * sh.tp);
        count = b.take(sizeof(int32_t));
        hidden = b.take(few || sh.direct_hidden ? 0 : part * sh.tp);
        head = b.take(few || sh.direct_head ? 0 : part * sh.vocab);
        const size_t stats = few ? static_cast<size_t>(a.tokens) * sh.few_tiles : static_cast<size_t>(sh.ta()) * sh.tp;
        m = b.take(a.saved ? 0 : stats * sizeof(float));
        s = b.take(stats * sizeof(float));
        zt = b.take(sizeof(float) * sh.tp);
        absmax = b.take(sh.parts == 2 || (a.saved && !few) ? sizeof(uint32_t) * (ABS_HEAD + ABS_HIDDEN) : 0);
        scales = b.take(few || sh.parts == 1 ? 0 : 2 * sizeof(float));
        bytes = b.at;
    }
};

// The backward pass for few tokens: workgroups over the columns and, for grad_hidden, over runs of vocabulary tiles, as
// many as the chip holds at once (registers).  Without `saved` a forward pass comes first, into the workspace.
struct FewPlan {
    Shape sh;
    int strips, splits;
    muon_token_logp_args forward;
    size_t slab, absmax, logp, lse, saved, workspace, bytes;
    explicit FewPlan(const muon_token_logp_backward_args& a)
        : sh(a.tokens, a.cols, a.vocab, a.dtype, a.hidden, a.ld_hidden, a.head, a.ld_head), forward{} {
        // (6 tokens x 3176 x 52257: 302 us for both passes, 322 with two workgroups a CU, 394 with one; 2 x 2048 x 32000: 90, 88, 91)
        strips = static_cast<int>(ceil_div(a.cols, FEW_STRIP));
        splits = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>((blocks() == 1 ? 3 : 2) * CUS / strips, sh.few_tiles / 8)));
        Bump b;
        slab = b.take(a.grad_hidden ? sizeof(float) * FEW_STRIP * static_cast<size_t>(strips) * splits * 16 * blocks() : 0);
        absmax = b.take(sh.parts == 1 ? 0 : sizeof(uint32_t) * (ABS_HEAD + ABS_HIDDEN));
        if (!a.saved) {
            forward.hidden = a.hidden;
            forward.head = a.head;
            forward.targets = a.targets;
            forward.tokens = a.tokens;
            forward.cols = a.cols;
            forward.vocab = a.vocab;
            forward.ld_hidden = a.ld_hidden;
            forward.ld_head = a.ld_head;
            forward.scale = a.scale;
            forward.dtype = a.dtype;
            forward.saved = const_cast<void*>(a.head);   // any: there is one
            logp = b.take(sizeof(float) * a.tokens);
            lse = b.take(sizeof(float) * a.tokens);
            saved = b.take(SavedPlan(sh).bytes);
            workspace = b.take(ForwardPlan(forward).bytes);
        }
        bytes = b.at;
    }
    int blocks() const { return sh.tokens <= 16 ? 1 : sh.tokens <= 32 ? 2 : 4; }   // of 16 tokens
};

// How a gradient's product is tiled and spread: the small tile where the large ones are too few, then
// the sum over k over enough workgroups for the chip, each with a worthwhile run of k.
struct GradPlan {
    int edge, ta, tb, splits;
    bool slab;
    GradPlan(int64_t cols, int64_t rows, int64_t k, bool later_chunks) {
        edge = edge_for(ceil_div(cols, 256) * ceil_div(rows, 256));
        ta = static_cast<int>(ceil_div(cols, edge));
        tb = static_cast<int>(ceil_div(rows, edge));
        const int64_t tiles = static_cast<int64_t>(ta) * tb;
        splits = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({CUS / tiles, MAX_SPLITS, k / pt::KS / MIN_SPLIT_STEPS})));
        slab = splits > 1 || later_chunks;
    }
    size_t slab_bytes() const { return slab ? sizeof(float) * edge * edge * static_cast<size_t>(splits) * ta * tb : 0; }
};

struct BackwardPlan {
    Shape sh;
    int64_t chunk;          // list entries at a time
    int chunks;
    GradPlan gh, gw;
    size_t idx, count, hidden, head, head_t, hidden_t, dz, dzt, slab, slab_w, absmax, scales, exponents, bytes;
    size_t e, m, s, zt, logp, ref, shift;   // without `saved`: e, M and S of a chunk, the rest by list entry
    static int64_t chunk_of(const Shape& sh, bool saved) {
        const int64_t row = sizeof(uint16_t) * sh.parts * (saved ? 2 : 3) * sh.vp;   // e takes as much as dz
        return std::min(sh.tp, std::max<int64_t>(PAD, DZ_BYTES / row / PAD * PAD));
    }
    explicit BackwardPlan(const muon_token_logp_backward_args& a)
        : sh(a.tokens, a.cols, a.vocab, a.dtype, a.hidden, a.ld_hidden, a.head, a.ld_head),
          chunk(chunk_of(sh, a.saved != nullptr)), chunks(static_cast<int>(ceil_div(sh.tp, chunk))), gh(sh.cols, chunk, sh.vp, false),
          gw(sh.cols, sh.vocab, chunk, chunks > 1) {
        Bump b;
        const size_t el = sizeof(uint16_t) * sh.parts;
        idx = b.take(a.saved ? 0 : sizeof(int32_t) * sh.tp);
        count = b.take(sizeof(int32_t));
        hidden = b.take(a.saved || sh.direct_hidden ? 0 : el * sh.dp * chunk);
        head = b.take(a.saved || sh.direct_head ? 0 : el * sh.dp * sh.vocab);
        head_t = b.take(a.grad_hidden ? el * sh.cols * sh.vp : 0);
        hidden_t = b.take(a.grad_head ? el * sh.cols * chunk : 0);
        dz = b.take(a.grad_hidden ? el * chunk * sh.vp : 0);
        dzt = b.take(a.grad_head ? el * chunk * sh.vp : 0);
        // the slab of grad_head lives through the chunks, so the two do not share one
        slab = b.take(a.grad_hidden ? gh.slab_bytes() : 0);
        slab_w = b.take(a.grad_head ? gw.slab_bytes() : 0);
        absmax = b.take(a.saved ? 0 : sizeof(uint32_t) * (ABS_HEAD + ABS_HIDDEN));
        scales = b.take(3 * sizeof(float));
        exponents = b.take(sizeof(int32_t) * chunk);
        const size_t by_chunk = a.saved ? 0 : static_cast<size_t>(chunk), by_entry = a.saved ? 0 : sizeof(float) * sh.tp;
        e = b.take(el * by_chunk * sh.vp);
        m = b.take(sizeof(float) * by_chunk * sh.ta());
        s = b.take(sizeof(float) * by_chunk * sh.ta());
        zt = b.take(by_entry);
        logp = b.take(by_entry);
        ref = b.take(by_entry);
        shift = b.take(by_entry);
        bytes = b.at;
    }
};

bool few_backward(const muon_token_logp_backward_args& a) { return a.tokens <= FEW_TOKENS; }
Shape shape_of(const muon_token_logp_args& a) { return Shape(a.tokens, a.cols, a.vocab, a.dtype, a.hidden, a.ld_hidden, a.head, a.ld_head); }

// The list of scored tokens and, with `part`, the largest values of both operands.
hipError_t launch_scan(int dtype, const void* hidden, int64_t ld_hidden, const void* head, int64_t ld_head, const Shape& sh,
                       const int64_t* targets, int32_t* idx, int32_t* count, float* logp, float* lse, uint32_t* part, hipStream_t s) {
    const ScanArgs a{1, targets, sh.tokens, idx, count, logp, lse, 0, part ? ABS_HEAD + ABS_HIDDEN : 0,
                     {head, hidden, static_cast<size_t>(ld_head), static_cast<size_t>(ld_hidden), sh.vocab, sh.tokens, sh.cols, targets, part}};
    if (dtype == MUON_BF16) hipLaunchKernelGGL(scan_kernel<uint16_t>, dim3(1 + a.blocks), dim3(LIVE_THREADS), 0, s, a);
    else hipLaunchKernelGGL(scan_kernel<float>, dim3(1 + a.blocks), dim3(LIVE_THREADS), 0, s, a);
    return hipGetLastError();
}

// The largest value of hidden's scored rows alone (few tokens).
hipError_t launch_hidden_absmax(const void* hidden, int64_t ld_hidden, const Shape& sh, const int64_t* targets, uint32_t* part, hipStream_t s) {
    const ScanArgs a{0, nullptr, 0, nullptr, nullptr, nullptr, nullptr, ABS_HEAD, ABS_HIDDEN,
                     {nullptr, hidden, 0, static_cast<size_t>(ld_hidden), 0, sh.tokens, sh.cols, targets, part}};
    hipLaunchKernelGGL(scan_kernel<float>, dim3(a.blocks), dim3(LIVE_THREADS), 0, s, a);
    return hipGetLastError();
}

template <int EDGE, int MODE> hipError_t launch_logits_edge(const LogitsArgs& l, int parts, hipStream_t s) {
    const dim3 grid = row_of_blocks(static_cast<int64_t>(l.ta) * l.tb, pt::Tile<EDGE>::THREADS), block(pt::Tile<EDGE>::THREADS);
    if (parts == 2) hipLaunchKernelGGL((logits_kernel<EDGE, 2, MODE, false>), grid, block, 0, s, l);
    else if (l.tail < pt::CHUNKS) hipLaunchKernelGGL((logits_kernel<EDGE, 1, MODE, true>), grid, block, 0, s, l);
    else hipLaunchKernelGGL((logits_kernel<EDGE, 1, MODE, false>), grid, block, 0, s, l);
    return hipGetLastError();
}
template <int MODE> hipError_t launch_logits(const LogitsArgs& l, int edge, int parts, hipStream_t s) {
    return edge == 256 ? launch_logits_edge<256, MODE>(l, parts, s) : launch_logits_edge<128, MODE>(l, parts, s);
}

template <int EDGE> hipError_t launch_grad_edge(const GradArgs& g, int parts, int dtype, bool last, hipStream_t s) {
    const dim3 grid(static_cast<unsigned>(g.ta) * g.tb, g.splits), block(pt::Tile<EDGE>::THREADS);
    if (parts == 1) hipLaunchKernelGGL((grad_kernel<EDGE, 1, uint16_t>), grid, block, 0, s, g);
    else hipLaunchKernelGGL((grad_kernel<EDGE, 2, float>), grid, block, 0, s, g);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !g.slab || !last) return e;
    const unsigned blocks = static_cast<unsigned>(g.ta) * g.tb * (EDGE / 32 * (EDGE / 32) / 4);
    hipLaunchKernelGGL(slab_sum_kernel<EDGE>, dim3(blocks), dim3(256), 0, s, g, dtype);
    return hipGetLastError();
}
hipError_t launch_grad(GradArgs g, const GradPlan& pl, float* slab, int parts, int dtype, bool last, hipStream_t s) {
    g.ta = pl.ta;
    g.tb = pl.tb;
    g.splits = pl.splits;
    g.slab = pl.slab ? slab : nullptr;
    return pl.edge == 256 ? launch_grad_edge<256>(g, parts, dtype, last, s) : launch_grad_edge<128>(g, parts, dtype, last, s);
}

// The logits' operands: packed copies where the products cannot read the caller's rows.  absmax: two parts.
hipError_t logits_operands(const Shape& sh, const void* hidden, int64_t ld_hidden, const void* head, int64_t ld_head,
                           int dtype, char* hidden_copy, char* head_copy, bool pack_head, const uint32_t* absmax, float* scales,
                           LogitsArgs& l, hipStream_t s) {
    const size_t row = sizeof(uint16_t) * sh.dp;
    l.steps = static_cast<int>(sh.dp / pt::KS);
    // copies have zeros past the last column; a row read in place has none, so its last step stops there (in both)
    l.tail = sh.direct_head || sh.direct_hidden ? static_cast<int>(ceil_div(sh.cols - (sh.dp - pt::KS), 8)) : pt::CHUNKS;
    l.vocab = static_cast<int>(sh.vocab);
    l.ta = sh.ta();
    l.scales = scales;
    l.a = sh.direct_head ? static_cast<const char*>(head) : head_copy;
    l.a_ld = sh.direct_head ? 2 * static_cast<size_t>(ld_head) : row;
    l.a_part = row * sh.vocab;
    l.gather = sh.direct_hidden;
    l.b = sh.direct_hidden ? static_cast<const char*>(hidden) : hidden_copy;
    l.b_ld = sh.direct_hidden ? 2 * static_cast<size_t>(ld_hidden) : row;
    l.b_part = row * l.live.most;
    const size_t dp = static_cast<size_t>(sh.dp);
    auto blocks = [&](int64_t rows) { return static_cast<int>(std::min<int64_t>(ceil_div(rows * sh.dp / 8, 256), 8 * CUS)); };
    const PackBothArgs p{{head, static_cast<size_t>(ld_head), sh.vocab, sh.cols, 0, {}, reinterpret_cast<uint16_t*>(head_copy), dp, dp * sh.vocab, nullptr},
                         {hidden, static_cast<size_t>(ld_hidden), l.live.most, sh.cols, 1, l.live, reinterpret_cast<uint16_t*>(hidden_copy), dp,
                          dp * l.live.most, nullptr},
                         sh.direct_head || !pack_head ? 0 : blocks(sh.vocab), sh.direct_hidden ? 0 : blocks(l.live.most), absmax, scales};
    if (p.head_blocks + p.hidden_blocks == 0) return hipSuccess;
    const dim3 grid(p.head_blocks + p.hidden_blocks);
    if (dtype == MUON_BF16) hipLaunchKernelGGL((pack_kernel<uint16_t, 1>), grid, dim3(256), 0, s, p);
    else hipLaunchKernelGGL((pack_kernel<float, 2>), grid, dim3(256), 0, s, p);
    return hipGetLastError();
}

template <typename T, int PARTS> hipError_t launch_few(const muon_token_logp_args& a, const ForwardPlan& pl, char* ws, hipStream_t s) {
    const Shape& sh = pl.sh;
    char* keep = static_cast<char*>(a.saved);
    const SavedPlan sv(sh);
    auto kept = [&](size_t o) { return keep ? reinterpret_cast<float*>(keep + o) : nullptr; };
    FewArgs f{a.head, a.hidden, static_cast<size_t>(a.ld_head), static_cast<size_t>(a.ld_hidden), a.targets,
                 static_cast<int>(a.tokens), static_cast<int>(a.cols), static_cast<int>(a.vocab), sh.few_tiles, a.scale * LOG2E,
                 keep ? kept(sv.m) : reinterpret_cast<float*>(ws + pl.m), reinterpret_cast<float*>(ws + pl.s),
                 reinterpret_cast<float*>(ws + pl.zt), kept(sv.e), static_cast<size_t>(sh.vp),
                 keep ? reinterpret_cast<uint32_t*>(ws + pl.absmax) : nullptr};
    // for the gradients' sake; without them its launch (4 us of 51) costs more than values below 2^-109 are worth
    if (PARTS == 3 && keep) TL_TRY(launch_hidden_absmax(a.hidden, a.ld_hidden, sh, a.targets, reinterpret_cast<uint32_t*>(ws + pl.absmax), s));
    const dim3 grid(static_cast<unsigned>(f.tiles));
    if (f.tokens <= 16) hipLaunchKernelGGL((few_kernel<T, PARTS, 1>), grid, dim3(256), 0, s, f);
    else if (f.tokens <= 32) hipLaunchKernelGGL((few_kernel<T, PARTS, 2>), grid, dim3(256), 0, s, f);
    else hipLaunchKernelGGL((few_kernel<T, PARTS, 4>), grid, dim3(256), 0, s, f);
    TL_TRY(hipGetLastError());
    const CombineArgs c{f.m, f.s, f.zt, 1, static_cast<size_t>(sh.few_tiles), sh.few_tiles, a.targets, a.vocab, a.logp, a.lse,
                        {}, a.tokens, f.scale2, kept(sv.logp), kept(sv.ref), kept(sv.shift), nullptr, nullptr};
    hipLaunchKernelGGL(combine_kernel<1>, dim3(static_cast<unsigned>(a.tokens)), dim3(256), 0, s, c);
    return hipGetLastError();
}

template <typename T, int PARTS, int NT>
hipError_t launch_few_grads_nt(const FewGradArgs& g, const FewPlan& pl, hipStream_t s) {
    if (g.grad_hidden) {
        constexpr int AT_ONCE = PARTS == 3 && NT == 4 ? 2 : NT;
        hipLaunchKernelGGL((few_hidden_kernel<T, PARTS, AT_ONCE>), dim3(static_cast<unsigned>(pl.strips) * pl.splits, NT / AT_ONCE),
                           dim3(256), 0, s, g);
        TL_TRY(hipGetLastError());
        hipLaunchKernelGGL((few_sum_kernel<T, NT>), dim3(static_cast<unsigned>(pl.strips) * (FEW_STRIP * 16 * NT / 256)), dim3(256), 0, s, g);
        TL_TRY(hipGetLastError());
    }
    if (g.grad_head) {
        // enough workgroups over the columns to fill the chip
        const int by = std::max(1, std::min((4 * CUS + g.tiles - 1) / g.tiles, (pl.strips + 3) / 4));
        hipLaunchKernelGGL((few_head_kernel<T, PARTS, NT == 4 ? 2 : 1>), dim3(g.tiles, by), dim3(256), 0, s, g);
        TL_TRY(hipGetLastError());
    }
    return hipSuccess;
}
template <typename T, int PARTS>
hipError_t launch_few_grads(const muon_token_logp_backward_args& a, const FewPlan& pl, const char* saved, float* slab, uint32_t* absmax, hipStream_t s) {
    const SavedPlan sv(pl.sh);
    auto kept = [&](size_t o) { return reinterpret_cast<const float*>(saved + o); };
    const FewGradArgs g{a.head, a.hidden, static_cast<size_t>(a.ld_head), static_cast<size_t>(a.ld_hidden), a.targets,
                        static_cast<int>(a.tokens), static_cast<int>(a.cols), static_cast<int>(a.vocab), pl.sh.few_tiles,
                        pl.strips, pl.splits, a.scale * LOG2E, a.scale, saved + sv.e, static_cast<size_t>(pl.sh.vp), kept(sv.m),
                        kept(sv.logp), kept(sv.ref), kept(sv.shift), a.grad_logp, slab,
                        a.tokens > 0 ? a.grad_hidden : nullptr, a.grad_head, static_cast<size_t>(a.ld_grad_hidden),
                        static_cast<size_t>(a.ld_grad_head), absmax};
    switch (pl.blocks()) {
        case 1: return launch_few_grads_nt<T, PARTS, 1>(g, pl, s);
        case 2: return launch_few_grads_nt<T, PARTS, 2>(g, pl, s);
        default: return launch_few_grads_nt<T, PARTS, 4>(g, pl, s);
    }
}

}  // namespace

size_t token_logp_saved_bytes(const muon_token_logp_args& a) { return SavedPlan(shape_of(a)).bytes; }
size_t token_logp_bytes(const muon_token_logp_args& a) { return ForwardPlan(a).bytes; }
size_t token_logp_backward_bytes(const muon_token_logp_backward_args& a) {
    return few_backward(a) ? FewPlan(a).bytes : BackwardPlan(a).bytes;
}

hipError_t launch_token_logp(const muon_token_logp_args& a, void* workspace, hipStream_t s) {
    if (a.tokens == 0) return hipSuccess;
    const ForwardPlan pl(a);
    const Shape& sh = pl.sh;
    char* ws = static_cast<char*>(workspace);
    float* m = reinterpret_cast<float*>(ws + pl.m);
    float* sums = reinterpret_cast<float*>(ws + pl.s);
    float* zt = reinterpret_cast<float*>(ws + pl.zt);
    const float scale2 = a.scale * LOG2E;
    if (pl.few) return a.dtype == MUON_BF16 ? launch_few<uint16_t, 1>(a, pl, ws, s) : launch_few<float, 3>(a, pl, ws, s);
    LogitsArgs l{};
    int32_t* idx = reinterpret_cast<int32_t*>(ws + pl.idx);
    int32_t* count = reinterpret_cast<int32_t*>(ws + pl.count);
    float *kept_logp = nullptr, *kept_ref = nullptr, *kept_shift = nullptr;
    if (a.saved) {
        const SavedPlan sv(sh);
        char* p = static_cast<char*>(a.saved);
        l.e = p + sv.e;
        m = reinterpret_cast<float*>(p + sv.m);
        kept_logp = reinterpret_cast<float*>(p + sv.logp);
        kept_ref = reinterpret_cast<float*>(p + sv.ref);
        kept_shift = reinterpret_cast<float*>(p + sv.shift);
        idx = reinterpret_cast<int32_t*>(p + sv.idx);
        count = reinterpret_cast<int32_t*>(p + sv.count);
    }
    uint32_t* absmax = sh.parts == 2 || a.saved ? reinterpret_cast<uint32_t*>(ws + pl.absmax) : nullptr;
    TL_TRY(launch_scan(a.dtype, a.hidden, a.ld_hidden, a.head, a.ld_head, sh, a.targets, idx, count, a.logp, a.lse, absmax, s));
    l.live = {idx, count, 0, static_cast<int32_t>(sh.tp)};
    float* scales = reinterpret_cast<float*>(a.saved ? static_cast<char*>(a.saved) + SavedPlan(sh).scales : ws + pl.scales);
    TL_TRY(logits_operands(sh, a.hidden, a.ld_hidden, a.head, a.ld_head, a.dtype, ws + pl.hidden, ws + pl.head, true, absmax, scales, l, s));
    l.targets = a.targets;
    l.tb = static_cast<int>(sh.tp / sh.edge);
    l.scale2 = scale2;
    l.m = m;
    l.s = sums;
    l.zt = zt;
    l.rows_pitch = sh.tp;
    l.vp = sh.vp;
    TL_TRY(a.saved ? launch_logits<LG_SAVE>(l, sh.edge, sh.parts, s) : launch_logits<LG_STATS>(l, sh.edge, sh.parts, s));
    const CombineArgs c{m, sums, zt, static_cast<size_t>(sh.tp), 1, sh.ta(), a.targets, a.vocab, a.logp, a.lse, l.live, a.tokens,
                        scale2, kept_logp, kept_ref, kept_shift, sh.parts == 1 ? absmax : nullptr, scales};
    hipLaunchKernelGGL(combine_kernel<32>, row_of_blocks(sh.tp / 32, 256), dim3(256), 0, s, c);
    return hipGetLastError();
}

namespace {
hipError_t launch_few_backward(const muon_token_logp_backward_args& a, char* ws, hipStream_t s) {
    FewPlan pl(a);
    const char* saved = static_cast<const char*>(a.saved);
    if (!saved) {
        pl.forward.logp = reinterpret_cast<float*>(ws + pl.logp);
        pl.forward.lse = reinterpret_cast<float*>(ws + pl.lse);
        pl.forward.saved = ws + pl.saved;
        TL_TRY(launch_token_logp(pl.forward, ws + pl.workspace, s));
        saved = ws + pl.saved;
    }
    float* slab = reinterpret_cast<float*>(ws + pl.slab);
    uint32_t* absmax = reinterpret_cast<uint32_t*>(ws + pl.absmax);
    if (a.dtype == MUON_BF16) return launch_few_grads<uint16_t, 1>(a, pl, saved, slab, absmax, s);
    TL_TRY(launch_hidden_absmax(a.hidden, a.ld_hidden, pl.sh, a.targets, absmax, s));
    return launch_few_grads<float, 3>(a, pl, saved, slab, absmax, s);
}
}  // namespace

hipError_t launch_token_logp_backward(const muon_token_logp_backward_args& a, void* workspace, hipStream_t s) {
    if (few_backward(a)) return launch_few_backward(a, static_cast<char*>(workspace), s);
    const BackwardPlan pl(a);
    const Shape& sh = pl.sh;
    const SavedPlan sv(sh);
    char* ws = static_cast<char*>(workspace);
    const char* saved = static_cast<const char*>(a.saved);
    const int32_t* idx = reinterpret_cast<const int32_t*>(saved ? saved + sv.idx : ws + pl.idx);
    const int32_t* count = reinterpret_cast<const int32_t*>(saved ? saved + sv.count : ws + pl.count);
    // scales of hidden and head: as the forward pass left them, or found again; the least of dz: over all tokens, since chunks add up
    float* own = reinterpret_cast<float*>(ws + pl.scales);
    uint32_t* absmax = reinterpret_cast<uint32_t*>(ws + pl.absmax);
    const float* scales = saved ? reinterpret_cast<const float*>(saved + sv.scales) : own;
    int32_t* least = reinterpret_cast<int32_t*>(own + 2);
    const Live everyone{idx, count, 0, static_cast<int32_t>(sh.tp)};
    if (!saved)
        TL_TRY(launch_scan(a.dtype, a.hidden, a.ld_hidden, a.head, a.ld_head, sh, a.targets, const_cast<int32_t*>(idx),
                           const_cast<int32_t*>(count), nullptr, nullptr, absmax, s));
    const size_t vp = sh.vp, dz_part = static_cast<size_t>(pl.chunk) * vp;
    auto at = [&](size_t o) { return reinterpret_cast<float*>(ws + o); };
    uint16_t* dz = a.grad_hidden ? reinterpret_cast<uint16_t*>(ws + pl.dz) : nullptr;
    uint16_t* dzt = a.grad_head ? reinterpret_cast<uint16_t*>(ws + pl.dzt) : nullptr;
    for (int c = 0; c < pl.chunks; ++c) {
        const Live live{idx, count, static_cast<int32_t>(c * pl.chunk), static_cast<int32_t>(pl.chunk)};
        LogitsArgs l{};
        l.live = live;
        if (!saved) {
            TL_TRY(logits_operands(sh, a.hidden, a.ld_hidden, a.head, a.ld_head, a.dtype, ws + pl.hidden, ws + pl.head, c == 0, absmax, own, l, s));
            l.targets = a.targets;
            l.tb = static_cast<int>(pl.chunk / sh.edge);
            l.scale2 = a.scale * LOG2E;
            l.m = at(pl.m);
            l.s = at(pl.s);
            l.zt = at(pl.zt);
            l.rows_pitch = pl.chunk;
            l.e = ws + pl.e;
            l.vp = vp;
            TL_TRY(launch_logits<LG_SAVE>(l, sh.edge, sh.parts, s));
            const CombineArgs f{l.m, l.s, l.zt, static_cast<size_t>(pl.chunk), 1, sh.ta(), a.targets, a.vocab, nullptr, nullptr, live,
                                a.tokens, l.scale2, at(pl.logp), at(pl.ref), at(pl.shift), sh.parts == 1 ? absmax : nullptr, own};
            hipLaunchKernelGGL(combine_kernel<32>, row_of_blocks(pl.chunk / 32, 256), dim3(256), 0, s, f);
            TL_TRY(hipGetLastError());
        }
        PrepareArgs p{};
        p.live = live;
        if (c == 0) p.dz = {everyone, a.grad_logp, a.scale, least};
        const int col_tiles = static_cast<int>(ceil_div(sh.cols, 64));
        if (a.grad_hidden && c == 0) {
            p.head = {a.head, static_cast<size_t>(a.ld_head), sh.vocab, sh.cols, 0, live, reinterpret_cast<uint16_t*>(ws + pl.head_t),
                      vp, vp * sh.cols, scales + 1};
            p.head_rows = static_cast<int>(ceil_div(sh.vocab, 64));
            p.head_blocks = p.head_rows * col_tiles;
            p.targets = a.targets;
            p.tokens = a.tokens;
            p.cols = sh.cols;
            p.zero = a.grad_hidden;
            p.zero_ld = a.ld_grad_hidden;
            p.zero_blocks = static_cast<int>(std::min<int64_t>(ceil_div(a.tokens, 4), 4 * CUS));
        }
        const int prepare = p.head_blocks + p.zero_blocks + (p.dz.out ? 1 : 0);
        if (prepare > 0) {
            if (sh.parts == 1) hipLaunchKernelGGL((prepare_kernel<uint16_t, 1>), dim3(prepare), dim3(256), 0, s, p);
            else hipLaunchKernelGGL((prepare_kernel<float, 2>), dim3(prepare), dim3(256), 0, s, p);
            TL_TRY(hipGetLastError());
        }
        auto kept = [&](size_t o, size_t without) { return reinterpret_cast<const float*>(saved ? saved + o : ws + without); };
        const PackArgs hidden_t{a.hidden, static_cast<size_t>(a.ld_hidden), pl.chunk, sh.cols, 1, live, reinterpret_cast<uint16_t*>(ws + pl.hidden_t),
                                static_cast<size_t>(pl.chunk), static_cast<size_t>(pl.chunk) * sh.cols, scales};
        const DzTokenArgs tok{live, a.targets, kept(sv.logp, pl.logp), a.grad_logp, a.scale, static_cast<int>(a.vocab), least};
        int32_t* exponents = reinterpret_cast<int32_t*>(ws + pl.exponents);
        const DzArgs d{kept(sv.e, pl.e), kept(sv.m, pl.m), saved ? 0 : live.first, kept(sv.ref, pl.ref), kept(sv.shift, pl.shift),
                       a.scale * LOG2E, static_cast<size_t>(saved ? sh.tp : pl.chunk), sh.edge, tok, vp, static_cast<size_t>(pl.chunk),
                       dz, dzt, dz_part, dz_part, exponents, hidden_t};
        const dim3 grid(static_cast<unsigned>(vp / 64 + (a.grad_head ? col_tiles : 0)) * static_cast<unsigned>(pl.chunk / 64));
        if (sh.parts == 1) hipLaunchKernelGGL((dz_kernel<uint16_t, 1>), grid, dim3(256), 0, s, d);
        else hipLaunchKernelGGL((dz_kernel<float, 2>), grid, dim3(256), 0, s, d);
        TL_TRY(hipGetLastError());
        GradArgs g{};
        g.live = live;
        g.cols = static_cast<int>(sh.cols);
        if (a.grad_hidden) {
            g.exponents = exponents;
            g.scale = scales + 1;
            g.a = ws + pl.head_t;
            g.a_ld = 2 * vp;
            g.a_part = 2 * vp * sh.cols;
            g.b = reinterpret_cast<const char*>(dz);
            g.b_ld = 2 * vp;
            g.b_part = 2 * dz_part;
            g.by_token = 1;
            g.steps = static_cast<int>(ceil_div(sh.vocab, pt::KS));
            g.out = a.grad_hidden;
            g.ld = a.ld_grad_hidden;
            TL_TRY(launch_grad(g, pl.gh, reinterpret_cast<float*>(ws + pl.slab), sh.parts, a.dtype, true, s));
        }
        if (a.grad_head) {
            g.exponents = least;
            g.scale = scales;
            g.a = ws + pl.hidden_t;
            g.a_ld = 2 * static_cast<size_t>(pl.chunk);
            g.a_part = g.a_ld * sh.cols;
            g.b = reinterpret_cast<const char*>(dzt);
            g.b_ld = g.a_ld;
            g.b_part = 2 * dz_part;
            g.by_token = 0;
            g.rows = static_cast<int>(sh.vocab);
            g.out = a.grad_head;
            g.ld = a.ld_grad_head;
            g.add = c > 0;
            TL_TRY(launch_grad(g, pl.gw, reinterpret_cast<float*>(ws + pl.slab_w), sh.parts, a.dtype, c + 1 == pl.chunks, s));
        }
    }
    return hipSuccess;
}

}  // namespace muon
