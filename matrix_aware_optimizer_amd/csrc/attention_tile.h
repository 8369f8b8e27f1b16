// Fragments and tiles shared by the attention kernels (attention.hip).
//
// All products go through 32 x 32 blocks, C[m][n] += sum_k A[m][k] B[k][n], 16 values of k a step.  In a step, lane
// l holds 8 values of A's row l % 32 and of B's column l % 32 ("slots" 8 h + 0 .. 7, h = l / 32); C's column is l % 32
// and its rows are 8 (i / 4) + 4 h + i % 4 for register i.  bf16: one v_mfma_f32_32x32x16_bf16 a step; fp32: eight
// v_mfma_f32_32x32x2_f32, each over one slot of both halves, exact products, so both types share one layout.
//
// Which k a slot stands for is free as long as A and B agree.  The probabilities come out of one product as C and go into
// the next as B without leaving their registers: slot 8 h + j of the step over rows 16 g .. 16 g + 15 of C is
// register 8 g + j, that is row 16 g + 8 (j / 4) + 4 h + j % 4.  A is then read from a tile whose rows are k, transposed on
// the way (col_frag), at the same rows.
//
// A tile is ROWS x DP values in LDS, loaded straight from global memory in 16-byte chunks; chunk c of a row stands at
// c ^ swizzle(row).  The swizzles keep both ways of reading free of bank conflicts: 16 rows at one chunk, and 4 + 4
// rows (bf16: 4 chunks each, fp32: 8) for the transposed reads.
#pragma once

#include "train_internal.h"

namespace muon {
namespace at {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef short i16x4_t __attribute__((ext_vector_type(4)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) void* lds_ptr_t;
typedef __attribute__((address_space(3))) char lds_byte_t;
typedef __attribute__((address_space(3))) u32x4_t lds_u32x4_t;
typedef __attribute__((address_space(3))) f32x4_t lds_f32x4_t;
typedef __attribute__((address_space(3))) i16x4_t lds_i16x4_t;
typedef __attribute__((address_space(3))) float lds_float_t;

constexpr double LOG2E_64 = 1.44269504088896340736, LN2_64 = 0.69314718055994530942;
constexpr float LOG2E = static_cast<float>(LOG2E_64), LOG2E_LOW = static_cast<float>(LOG2E_64 - static_cast<double>(LOG2E));
constexpr float NEG_INF = -__builtin_inff();

static __device__ const u32x4_t zero_chunk = {};   // what a load reads in place of a row or column that is not there

__device__ __forceinline__ int wave_id() { return __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6)); }
__device__ __forceinline__ float exp2_(float v) { return __builtin_amdgcn_exp2f(v); }

// Between lanes l and l ^ 32.
__device__ __forceinline__ float half_max(float v) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float half_sum(float v) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

template <typename T> struct Frag;   // 8 values
template <> struct Frag<uint16_t> { u32x4_t w; };
template <> struct Frag<float> { f32x4_t w[2]; };

__device__ __forceinline__ void mma(f32x16_t& acc, const Frag<uint16_t>& a, const Frag<uint16_t>& b) {
    acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a.w), __builtin_bit_cast(bf16x8_t, b.w), acc, 0, 0, 0);
}
__device__ __forceinline__ void mma(f32x16_t& acc, const Frag<float>& a, const Frag<float>& b) {
#pragma unroll
    for (int j = 0; j < 8; ++j) acc = __builtin_amdgcn_mfma_f32_32x32x2f32(a.w[j >> 2][j & 3], b.w[j >> 2][j & 3], acc, 0, 0, 0);
}

// Registers 8 g .. 8 g + 7 of C as B of the next product.  bf16: two parts, hi = bf16(v) and lo = bf16(v - hi), 16 bits;
// one part (8 bits) would add as much error to an output as its own rounding.
template <typename T> struct Parts;
template <> struct Parts<uint16_t> {
    Frag<uint16_t> hi, lo;
    __device__ __forceinline__ Parts(const f32x16_t& c, int g) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float x = c[8 * g + 2 * e], y = c[8 * g + 2 * e + 1];
            const uint32_t h = pack_bf16x2(x, y);
            hi.w[e] = h;
            lo.w[e] = pack_bf16x2(x - __uint_as_float(h << 16), y - __uint_as_float(h & 0xffff0000u));
        }
    }
    __device__ __forceinline__ void mma_to(f32x16_t& acc, const Frag<uint16_t>& a) const {
        mma(acc, a, hi);
        mma(acc, a, lo);
    }
};
template <> struct Parts<float> {
    Frag<float> v;
    __device__ __forceinline__ Parts(const f32x16_t& c, int g) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v.w[e >> 2][e & 3] = c[8 * g + e];
    }
    __device__ __forceinline__ void mma_to(f32x16_t& acc, const Frag<float>& a) const { mma(acc, a, v); }
};

// Geometry of a tile row of DP values of T.
template <typename T, int DP> struct Row {
    static constexpr int ES = sizeof(T);
    static constexpr int PER = 16 / ES;            // values a chunk
    static constexpr int CH = DP / PER;            // chunks a row
    static constexpr int BYTES = DP * ES;
    static __device__ __forceinline__ int swizzle(int row) {
        if constexpr (CH == 8) return (((row >> 1) & 1) << 2) | ((row >> 2) & 3);          // two rows share 256 bytes
        else if constexpr (ES == 2) return ((row & 3) << 2) | ((row >> 2) & 3);
        else return (row & 3) | (((row >> 3) & 1) << 2) | (((row >> 2) & 1) << 3);
    }
};

// Where a lane reads in a tile: byte addresses for step 0 of row_frag and block 0 of col_frag.  A tile starts at a multiple
// of 512 bytes, so the chunk of another step or block is one exclusive or away.  fresh() keeps the compiler from holding every such
// address in a register of its own through the whole loop.
template <typename T, int DP> struct Lanes {
    unsigned row, col;
    __device__ __forceinline__ Lanes() {
        typedef Row<T, DP> R;
        const int lane = threadIdx.x & 63, r = lane & 31, h = lane >> 5;
        if constexpr (R::ES == 2) {
            row = r * R::BYTES + ((h ^ R::swizzle(r)) << 4);
            // ds_read_b64_tr_b16: 16 lanes read 4 rows of 16 values, lane i gets column i of them
            const int i16 = lane & 15, g16 = lane >> 4, cr = 4 * (g16 >> 1) + (i16 >> 2);
            col = cr * R::BYTES + (((2 * (g16 & 1) + ((i16 & 3) >> 1)) ^ R::swizzle(cr)) << 4) + (i16 & 1) * 8;
        } else {
            row = r * R::BYTES + (((2 * h) ^ R::swizzle(r)) << 4);
            col = 4 * h * R::BYTES + (((r >> 2) ^ (h << 3)) << 4) + (r & 3) * 4;
        }
    }
    __device__ __forceinline__ void fresh() { asm volatile("" : "+v"(row), "+v"(col)); }
};
__device__ __forceinline__ unsigned lds_at(const lds_byte_t* p) { return static_cast<unsigned>(reinterpret_cast<uintptr_t>(p)); }
template <typename V> __device__ __forceinline__ V ld_lds(unsigned at) { return *(const __attribute__((address_space(3))) V*)static_cast<uintptr_t>(at); }

// A operand: rows row0 + l % 32 of the tile at `tile`, step ks along them.  row0 a multiple of 32.
template <typename T, int DP> __device__ __forceinline__ Frag<T> row_frag(unsigned tile, const Lanes<T, DP>& w, int row0, int ks) {
    typedef Row<T, DP> R;
    Frag<T> f;
    if constexpr (R::ES == 2) {
        f.w = ld_lds<u32x4_t>(((tile + w.row) ^ (ks << 5)) + row0 * R::BYTES);
    } else {
        f.w[0] = ld_lds<f32x4_t>(((tile + w.row) ^ (ks << 6)) + row0 * R::BYTES);
        f.w[1] = ld_lds<f32x4_t>(((tile + w.row) ^ (ks << 6) ^ 16) + row0 * R::BYTES);
    }
    return f;
}

// A operand, transposed: column 32 db + l % 32 of the tile at the rows row0 + 8 (j / 4) + 4 h + j % 4.  row0 a multiple of 16.
template <typename T, int DP> __device__ __forceinline__ Frag<T> col_frag(unsigned tile, const Lanes<T, DP>& w, int row0, int db) {
    typedef Row<T, DP> R;
    Frag<T> f;
    if constexpr (R::ES == 2) {
        const unsigned p = (tile + w.col) ^ (db << 6);
        const i16x4_t a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4_t*)static_cast<uintptr_t>(p + row0 * R::BYTES));
        const i16x4_t b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4_t*)static_cast<uintptr_t>((p ^ 32) + (row0 + 8) * R::BYTES));
        const u32x2_t a2 = __builtin_bit_cast(u32x2_t, a), b2 = __builtin_bit_cast(u32x2_t, b);
        f.w = u32x4_t{a2.x, a2.y, b2.x, b2.y};
    } else {
        // swizzle(row) of the row of slot j is j + 8 h
#pragma unroll
        for (int j = 0; j < 8; ++j)
            f.w[j >> 2][j & 3] = ld_lds<float>(((tile + w.col) ^ (db << 7) ^ (j << 4)) + (row0 + 8 * (j >> 2) + (j & 3)) * R::BYTES);
    }
    return f;
}

template <typename T> __device__ __forceinline__ float to_f32(T v);
template <> __device__ __forceinline__ float to_f32<uint16_t>(uint16_t v) { return bf16_to_f32(v); }
template <> __device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <typename T> __device__ __forceinline__ float ld_el(const T* p, size_t i) { return to_f32<T>(G(p)[i]); }

// n <= 16 / sizeof(T) values from p on, any alignment, zeros behind them.
template <typename T> __device__ __forceinline__ u32x4_t ld_part(const T* p, int n) {
    u32x4_t w = {};
    constexpr int PER = 16 / sizeof(T);
    if (n >= PER) {
        if constexpr (sizeof(T) == 2) return *(const MUON_GLOBAL u32x4_el2*)G(p);
        else return __builtin_bit_cast(u32x4_t, static_cast<f32x4_t>(*(const MUON_GLOBAL f32x4_el4*)G(p)));
    }
#pragma unroll
    for (int e = 0; e < PER - 1; ++e)
        if (e < n) {
            if constexpr (sizeof(T) == 2) w[e >> 1] |= static_cast<uint32_t>(G(p)[e]) << (16 * (e & 1));
            else w[e] = __float_as_uint(G(p)[e]);
        }
    return w;
}

// B operand straight from global memory: values e0 .. e0 + 7 of a row of `width`, zeros behind it; rows come in whole 16-byte
// chunks.  A load is one unconditional access, so a row's loads are all in flight at once.
template <typename T> __device__ __forceinline__ Frag<T> global_frag(const T* row, int e0, int width, bool ok) {
    Frag<T> f;
    constexpr int N = sizeof(T) / 2, PER = 16 / sizeof(T);
    u32x4_t w[N];
#pragma unroll
    for (int k = 0; k < N; ++k) {
        const int e = e0 + PER * k;
        w[k] = *(const MUON_GLOBAL u32x4_t*)G(ok && e < width ? static_cast<const void*>(row + e) : static_cast<const void*>(&zero_chunk));
    }
    if constexpr (sizeof(T) == 2) f.w = w[0];
    else
#pragma unroll
        for (int k = 0; k < 2; ++k) f.w[k] = __builtin_bit_cast(f32x4_t, w[k]);
    return f;
}
__device__ __forceinline__ float frag_get(const Frag<uint16_t>& f, int e) {
    return __uint_as_float((e & 1) ? (f.w[e >> 1] & 0xffff0000u) : (f.w[e >> 1] << 16));
}
__device__ __forceinline__ float frag_get(const Frag<float>& f, int e) { return f.w[e >> 2][e & 3]; }

// Loads rows 0 .. ROWS - 1 at `base` (pitch ld), in whole 16-byte chunks, into a tile: rows whose bit of `live` is 0 and columns
// from `width` on as zeros.  The loads go straight into LDS and are under way when this returns (vmcnt).
template <typename T, int DP, int ROWS, int THREADS>
__device__ __forceinline__ void load_tile(lds_byte_t* tile, const T* base, int64_t ld, int width, uint64_t live) {
    typedef Row<T, DP> R;
    constexpr int N = ROWS * R::CH / THREADS;
    static_assert(N * THREADS == ROWS * R::CH && THREADS % R::CH == 0, "whole passes of whole rows");
    const int tid = threadIdx.x, wave = wave_id();
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int row = (i * THREADS + tid) / R::CH, e0 = ((tid % R::CH) ^ R::swizzle(row)) * R::PER;
        const bool ok = ((live >> row) & 1) && e0 < width;
        const void* src = ok ? static_cast<const void*>(base + row * ld + e0) : static_cast<const void*>(&zero_chunk);
        __builtin_amdgcn_global_load_lds(src, (lds_ptr_t)(tile + (i * THREADS + wave * 64) * 16), 16, 0, 0);
    }
}

// Everything this wave has asked for is in LDS, and every wave of the workgroup is here.
__device__ __forceinline__ void tile_barrier() { asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// C (rows: width, column: this lane's row of the output) times f, to row pointer `out` of type T and, where wanted, what
// rounding took to `low`.  Four values at once at any alignment, the last ones of an odd width one by one.
typedef u32x2_t u32x2_el2 __attribute__((aligned(2)));
template <typename T, int NB> __device__ __forceinline__ void store_rows(const f32x16_t (&c)[NB], float f, T* out, T* low, int width) {
    const int h = (threadIdx.x & 63) >> 5;
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int d = 32 * b + 8 * q + 4 * h;
            const float v[4] = {c[b][4 * q] * f, c[b][4 * q + 1] * f, c[b][4 * q + 2] * f, c[b][4 * q + 3] * f};
            if (d + 4 <= width) {
                if constexpr (sizeof(T) == 2) {
                    const u32x2_t w = {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
                    *(MUON_GLOBAL u32x2_el2*)G(out + d) = w;
                    if (low) {
                        const u32x2_t l = {pack_bf16x2(v[0] - __uint_as_float(w.x << 16), v[1] - __uint_as_float(w.x & 0xffff0000u)),
                                           pack_bf16x2(v[2] - __uint_as_float(w.y << 16), v[3] - __uint_as_float(w.y & 0xffff0000u))};
                        *(MUON_GLOBAL u32x2_el2*)G(low + d) = l;
                    }
                } else {
                    *(MUON_GLOBAL f32x4_el4*)G(out + d) = f32x4_t{v[0], v[1], v[2], v[3]};
                    if (low) *(MUON_GLOBAL f32x4_el4*)G(low + d) = f32x4_t{};
                }
            } else {
#pragma unroll
                for (int e = 0; e < 3; ++e)
                    if (d + e < width) {
                        st_el<T>(out, d + e, v[e]);
                        if (low) st_el<T>(low, d + e, sizeof(T) == 2 ? v[e] - bf16_to_f32(f32_to_bf16(v[e])) : 0.0f);
                    }
            }
        }
}

// A unit of one axis: `rows` rows of a sequence from `start` on, `at` of them before it, and the sequence's rows of the
// other axis.  Row 0 .. offsets[0) and those from offsets[sequences) on count as two more sequences, which see nothing:
// every row belongs to exactly one unit.
struct Span {
    int start, at, rows;      // first row (of the whole axis), its place in the sequence, rows left of the sequence
    int len, other, other_len;
};
// Without a causal mask units come sequence by sequence.  Under one they come in the order of what they walk, the longest first, so
// that none of those runs alone at the end (8192 tokens in 6 sequences, 16 heads: grad_k and grad_v 262 -> 240 us, grad_q 189 ->
// 181; without a mask that order would only part the tiles of a sequence, 166 -> 189 us at 12 sequences): unit (s, r) of sequence s is the one with r units of s behind it (HEAD: before it) in that respect, and all units of a larger r
// come first.  A wave does that for up to 61 sequences, one a lane: C(r) = sum over s of max(0, units of s - r) units have a rank
// of r or more.  For more sequences, up to SPAN_SCAN, it adds units up in order, 4 x 63 sequences a trip to memory.  For more still unit u is rows BM j .. of sequence s with bound(s) / BM + s + j = u: distinct for distinct
// (s, j), since a sequence has at most bound(s + 1) / BM - bound(s) / BM + 1 units; a wave looks at 64 sequences at once.  Units
// without rows then stand between the others, every second one where sequences have up to BM rows, and XCDs and shader engines, which take
// workgroups in turn, would leave half the chip without work (200 sequences of 128 rows: 188 us, 95 in order): the caller
// goes through the units by a stride that mixes them.
// (4000 sequences of 40 tokens, forward: 119 us in order, 36 by the stride; 240 of 128: 95 in order.)
constexpr int SPAN_LANES = 61, SPAN_SCAN = 512;   // sequences that find_span handles a lane each, and in order
__host__ __device__ inline int64_t span_units(int64_t rows, int64_t sequences, int bm) { return (rows / bm + sequences + 3) | 1; }
__device__ __forceinline__ int bound(const int64_t* offsets, int sequences, int rows, int s) {
    if (s <= 0) return 0;
    if (s > sequences + 1) return rows;
    if (!offsets) return s == 1 ? 0 : rows;
    const int64_t v = G(offsets)[s - 1];
    return static_cast<int>(v < 0 ? 0 : v > rows ? rows : v);
}
// HEAD: the first rows of a sequence walk the longest (keys), else the last (queries).  BM = 2^shift.
template <bool HEAD>
__device__ __forceinline__ bool find_span(int shift, const int64_t* offsets, const int64_t* others, int sequences, int rows, int other_rows, bool causal, int u, Span& sp) {
    const int lane = threadIdx.x & 63;
    int s, b0, o0, o1, j;
    if (sequences <= SPAN_LANES) {
        // every bound of both axes at once, one trip to memory
        const int mine = bound(offsets, sequences, rows, lane), other = bound(others, sequences, other_rows, lane);
        const int len = __shfl(mine, lane + 1) - mine, units = lane <= sequences + 1 && len > 0 ? ((len - 1) >> shift) + 1 : 0;
        auto ranked = [&](int r) { return static_cast<int>(wave_sum(static_cast<float>(units > r ? units - r : 0))); };     // below 2^24
        if (u >= ranked(0)) return false;
        if (causal) {
            int most = units;
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) most = max(most, __shfl_xor(most, d));
            int lo = 0, hi = __builtin_amdgcn_readfirstlane(most), above = 0;     // C(lo) > u >= C(hi) = above
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1, n = ranked(mid);
                if (n > u) lo = mid;
                else {
                    hi = mid;
                    above = n;
                }
            }
            const uint64_t in = __ballot(units > lo);
            s = __builtin_ctzll(__ballot(units > lo && __popcll(in & ((1ull << lane) - 1)) == u - above));
            j = HEAD ? __builtin_amdgcn_readlane(units, s) - 1 - lo : lo;
        } else {
            int upto = units;
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {
                const int v = __shfl_up(upto, d);
                upto += lane >= d ? v : 0;
            }
            s = __popcll(__ballot(upto <= u));
            j = u - __builtin_amdgcn_readlane(upto - units, s);
        }
        b0 = __builtin_amdgcn_readlane(mine, s);
        sp.len = __builtin_amdgcn_readlane(len, s);
        o0 = __builtin_amdgcn_readlane(other, s);
        o1 = __builtin_amdgcn_readlane(other, s + 1);
    } else if (sequences <= SPAN_SCAN) {
        int c = 0, base = 0;
        bool found = false;
        s = j = b0 = 0;
        while (!found && c < sequences + 2) {
            int mine[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) mine[k] = bound(offsets, sequences, rows, c + 63 * k + lane);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int at = c + 63 * k + lane, len = __shfl(mine[k], lane + 1) - mine[k];
                const int units = lane < 63 && at <= sequences + 1 && len > 0 ? ((len - 1) >> shift) + 1 : 0;
                const int total = static_cast<int>(wave_sum(static_cast<float>(units)));
                if (!found && u < base + total) {
                    found = true;
                    int upto = units;
#pragma unroll
                    for (int d = 1; d < 64; d <<= 1) {
                        const int v = __shfl_up(upto, d);
                        upto += lane >= d ? v : 0;
                    }
                    const int l = __popcll(__ballot(base + upto <= u));
                    s = c + 63 * k + l;
                    j = u - base - __builtin_amdgcn_readlane(upto - units, l);
                    b0 = __builtin_amdgcn_readlane(mine[k], l);
                    sp.len = __builtin_amdgcn_readlane(len, l);
                }
                base += found ? 0 : total;
            }
            c += 4 * 63;
        }
        if (!found) return false;
        o0 = bound(others, sequences, other_rows, s);
        o1 = bound(others, sequences, other_rows, s + 1);
    } else {
        int lo = 0, hi = sequences + 1;
        while (hi > lo) {
            const int step = (hi - lo + 63) / 64;
            const int64_t at = lo + static_cast<int64_t>(lane + 1) * step;
            const bool below = at <= hi && (bound(offsets, sequences, rows, static_cast<int>(at)) >> shift) + at <= u;
            const int n = __popcll(__ballot(below));
            lo += n * step;
            hi = hi < lo + step - 1 ? hi : lo + step - 1;
        }
        s = __builtin_amdgcn_readfirstlane(lo);
        b0 = bound(offsets, sequences, rows, s);
        sp.len = bound(offsets, sequences, rows, s + 1) - b0;
        o0 = bound(others, sequences, other_rows, s);
        o1 = bound(others, sequences, other_rows, s + 1);
        j = u - ((b0 >> shift) + s);
        if (j < 0 || sp.len <= 0 || (static_cast<int64_t>(j) << shift) >= sp.len) return false;
    }
    sp.at = j << shift;
    sp.start = b0 + sp.at;
    sp.rows = sp.len - sp.at;
    sp.other = 0;
    sp.other_len = 0;
    if (s >= 1 && s <= sequences) {
        sp.other = o0;
        sp.other_len = o1 > o0 ? o1 - o0 : 0;
    }
    return true;
}

}  // namespace at
}  // namespace muon
