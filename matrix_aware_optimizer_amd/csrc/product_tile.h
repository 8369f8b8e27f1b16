// Square tiles of C = A B^T on the gfx950 matrix cores, for the products of the
// vocabulary head (token_logp.hip): both operands of 16-bit values, k-contiguous.
//
//   C[r][c] = sum_k A[r][k] B[c][k]
// Tile<256>: 8 waves (2 x 4, two a SIMD); a wave owns 128 x 64 of the tile as 4 x 2 blocks of
// 32 x 32 (v_mfma_f32_32x32x16, fp32 sums).
// Tile<128>: 8 waves, of which 4 (2 x 2 of 64 x 64) take the first half of every k-step and 4 the
// second; at the end the two sums of each 64 x 64 are exchanged so that each wave keeps 32 x 64.
// It reads LDS twice as much per product (as long as its MFMAs take), so it serves products with too few
// 256-tiles for the chip.
// Either takes a CU's whole LDS.  A k-step is 64 values of k: 128 bytes of each row of both
// operands, loaded straight into LDS (16 bytes a lane).  Tile<256> keeps a ring of five
// slabs, A's slab two steps ahead and B's one; a step lasts longer than a load takes.  A step of
// Tile<128> is a quarter as long, so it loads both operands four steps ahead.  The loads are spread over the step's MFMA groups, fragments are double-buffered in
// registers, and the barrier that opens a step stands before the last quarter of the one before
// it, whose MFMAs then cover the new step's first fragment reads.  Rows are XOR-swizzled by
// 16-byte chunks against bank conflicts.  Each lane's source rows are fixed for the whole tile, so any row may
// come from anywhere (gathered tokens, rows clamped at an edge).  k is a multiple of 64, or (KTAIL) of 8:
// then the last step's missing chunks come from 16 bytes of zeros.
//
// fp32 operands come as two fp16 parts of 11 bits each, x = (hi + 2^-11 lo) / scale with one power-of-two scale an operand
// that brings its largest value to 2^14 .. 2^15 (values below 2^-28 of it lose bits: fp16 ends at 2^-24).
// The tile sums lo hi + hi lo first, multiplies by 2^-11, and goes on with hi hi; lo lo, below 2^-22 of
// the product of the magnitudes, is left out.  Three fp16 products take 3 / 2517 of the time unit against
// 1 / 157 for the fp32 MFMA: 5 times less.  (Subnormal fp16 inputs of the MFMA are taken at their value.)
#pragma once

#include "muon_internal.h"

namespace muon {

namespace pt {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void* lds_ptr_t;
typedef __attribute__((address_space(3))) char lds_byte_t;
typedef __attribute__((address_space(3))) u32x2_t lds_u32x2_t;
typedef __attribute__((address_space(3))) u32x4 lds_u32x4_t;

constexpr int KS = 64;               // k per step
constexpr int CHUNKS = 8;            // 16-byte chunks per row and step
constexpr int SUB = CHUNKS / 2;      // MFMA k-slices per step

static __device__ const u32x4 zero_chunk = {};   // what a KTAIL product reads past the last column

__device__ __forceinline__ int wave_id() { return __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6)); }
__device__ __forceinline__ int swz(int row, int c) { return row * CHUNKS + (c ^ ((row >> 1) & 7)); }

// Parts of the operands (one: the value itself; fp32: hi and lo, pitch a_part / b_part bytes) in the
// order in which their products are summed, two bits a product.
template <int PARTS> struct Order;
template <> struct Order<1> { static constexpr int N = 1; static constexpr unsigned A = 0, B = 0; };
template <> struct Order<2> { static constexpr int N = 3; static constexpr unsigned A = 1u, B = 1u << 2; };   // lo hi, hi lo, hi hi
constexpr float LO_STEP = 1.0f / 2048.0f;   // what lo counts against hi

// V: bf16x8_t or f16x8_t, what the operands hold.
template <typename V> __device__ __forceinline__ void mfma(f32x16_t& acc, const u32x4& a, const u32x4& b) {
    if constexpr (__is_same(V, bf16x8_t))
        acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), acc, 0, 0, 0);
    else
        acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b), acc, 0, 0, 0);
}
// Between the cross products and hi hi.
template <int PARTS, int M, int N> __device__ __forceinline__ void scale_cross(f32x16_t (&acc)[M][N], int kt, int steps) {
    if constexpr (PARTS == 2) {
        if (kt == 2 * steps) {
#pragma unroll
            for (int i = 0; i < M; ++i)
#pragma unroll
                for (int j = 0; j < N; ++j) acc[i][j] *= LO_STEP;
        }
    }
}

// Byte offset of successive k-steps of one operand over the parts' products.
template <int PARTS> struct Walk {
    unsigned order;
    size_t part;
    int per, left;      // steps per product, steps left in this one
    size_t off;
    __device__ Walk(unsigned o, size_t p, size_t k0, int per_) : order(o), part(p), per(per_), left(per_), off(0), base(k0) { begin(); }
    __device__ __forceinline__ void begin() { off = base + (PARTS > 1 ? (order & 3u) * part : 0); }
    __device__ __forceinline__ void next() {
        off += CHUNKS * 16;
        if constexpr (PARTS > 1) {
            if (--left == 0) { order >>= 2; left = per; begin(); }
        }
    }
    size_t base;
};

template <int EDGE> struct Tile {
    static constexpr int SIZE = EDGE;                        // rows and columns of C
    static constexpr int NWAVES = 8, THREADS = 64 * NWAVES;
    static constexpr int KGROUPS = EDGE == 256 ? 1 : 2;      // waves that share a part of C, by halves of the k-step
    static constexpr int WAVES_N = EDGE / 64;
    static constexpr int WM = EDGE / 2, WN = 64;             // a wave's part of C while it multiplies
    static constexpr int SM = WM / 32 / KGROUPS, SN = WN / 32;   // blocks of it that the wave ends up with
    static constexpr int SLAB = EDGE * CHUNKS;               // chunks of one operand's step
    static constexpr int SLOTS = 5;                          // of the ring; Tile<128>: of each operand's
    static constexpr int DEPTH = SLOTS - 1;                  // Tile<128>: steps loaded ahead
    static constexpr int LDS_CHUNKS = (EDGE == 256 ? 1 : 2) * SLOTS * SLAB;
    static constexpr int HL = SLAB / 64 / NWAVES;            // loads a wave issues per slab
    // loads of A(kt + 2) issued before the barrier that opens step kt + 1
    static constexpr int PB = ((SUB - 1) * SM < 2 * HL ? (SUB - 1) * SM : 2 * HL) - HL;
    static_assert(EDGE == 128 || (EDGE == 256 && 2 * HL <= SUB * SM && PB >= 0 && SM >= SN), "tile geometry");

    typedef f32x16_t Acc[SM][SN];

    // Which row of the slab, and which of its 16-byte chunks, this lane's load j fetches.
    static __device__ __forceinline__ int load_row(int j) {
        return ((wave_id() * HL + j) * 64 + static_cast<int>(threadIdx.x & 63)) / CHUNKS;
    }
    static __device__ __forceinline__ int load_chunk(int j) { return (static_cast<int>(threadIdx.x) & 7) ^ ((load_row(j) >> 1) & 7); }

    // acc += the tile's product over `steps` k-steps (per part product) from byte offset k0 of
    // the rows.  srca[j], srcb[j]: this lane's row of load j, already moved to its chunk (load_row,
    // load_chunk).  steps >= 1.  KTAIL: the last step has `tail` chunks.  Ends with every LDS read
    // of this wave done; other waves may still read, so a barrier comes before the LDS is used again.
    template <typename V, int PARTS, bool KTAIL>
    static __device__ __attribute__((always_inline)) void run(const char* const (&srca)[HL], const char* const (&srcb)[HL],
                                                              size_t a_part, size_t b_part, size_t k0, int steps, int tail,
                                                              u32x4* lds, Acc& acc) {
        static_assert(PARTS == 1 || (!KTAIL && __is_same(V, f16x8_t)), "two parts are fp16, packed to whole steps");
        if constexpr (EDGE == 128) {
            run_deep<V, PARTS, KTAIL>(srca, srcb, a_part, b_part, k0, steps, tail, lds, acc);
            return;
        }
        const int lane = threadIdx.x & 63, wave = wave_id();
        const int wm = wave / WAVES_N, wn = wave % WAVES_N;
        const int total = steps * Order<PARTS>::N;
        Walk<PARTS> wa(Order<PARTS>::A, a_part, k0, steps), wb(Order<PARTS>::B, b_part, k0, steps);
        auto issue = [&](const char* s, size_t off, int kt, int slot, int j) {
            const char* from = s + off;
            if (KTAIL && kt == total - 1) from = load_chunk(j) < tail ? from : reinterpret_cast<const char*>(&zero_chunk);
            __builtin_amdgcn_global_load_lds((const void*)from, (lds_ptr_t)(lds + slot * SLAB + (wave * HL + j) * 64), 16, 0, 0);
        };
#pragma unroll
        for (int j = 0; j < HL; ++j) issue(srca[j], wa.off, 0, 0, j);
        wa.next();
#pragma unroll
        for (int j = 0; j < HL; ++j) issue(srcb[j], wb.off, 0, 1, j);
        wb.next();
        if (total > 1) {
#pragma unroll
            for (int j = 0; j < HL; ++j) issue(srca[j], wa.off, 1, 2, j);
            wa.next();
        }
        const int half = lane >> 5;
        const int arow = wm * WM + (lane & 31), brow = wn * WN + (lane & 31);
        u32x4 fa[2][SM], fb[2][SN];
        if (total > 1)
            asm volatile("s_waitcnt vmcnt(%0)" ::"n"(HL) : "memory");
        else
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        asm volatile("s_barrier" ::: "memory");
#pragma unroll
        for (int i = 0; i < SM; ++i) fa[0][i] = lds[swz(arow + i * 32, half)];
#pragma unroll
        for (int j = 0; j < SN; ++j) fb[0][j] = lds[SLAB + swz(brow + j * 32, half)];

        int sa = 0;   // slot of A(kt); B(kt) is in the next one
        for (int kt = 0; kt < total; ++kt) {
            const int sb = sa + 1 == SLOTS ? 0 : sa + 1;
            const int s3 = sa >= 2 ? sa - 2 : sa + 3;   // slot of B(kt + 1)
            const int s4 = sa >= 1 ? sa - 1 : sa + 4;   // slot of A(kt + 2)
            const int na = sa >= 3 ? sa - 3 : sa + 2;   // slot of A(kt + 1)
            const u32x4* LA = lds + sa * SLAB;
            const u32x4* LB = lds + sb * SLAB;
            const bool more1 = kt + 1 < total, more2 = kt + 2 < total;
            const size_t offa = wa.off, offb = wb.off;
            scale_cross<PARTS>(acc, kt, steps);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int s = 0; s < SUB; ++s) {
                if (s == SUB - 1 && more1) {
                    // step kt's slabs have been read, this wave's loads of B(kt + 1) and A(kt + 1)
                    // are done, only A(kt + 2) may be in flight
                    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
                    if (more2)
                        asm volatile("s_waitcnt vmcnt(%0)" ::"n"(PB) : "memory");
                    else
                        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
                    asm volatile("s_barrier" ::: "memory");
                    __builtin_amdgcn_sched_barrier(0);
                }
                const int cn = 2 * (s + 1) + half;
#pragma unroll
                for (int i = 0; i < SM; ++i) {
#pragma unroll
                    for (int j = 0; j < SN; ++j)
                        mfma<V>(acc[i][j], fa[s & 1][i], fb[s & 1][j]);
                    if (s + 1 < SUB) {
                        fa[(s + 1) & 1][i] = LA[swz(arow + i * 32, cn)];
                        if (i < SN) fb[(s + 1) & 1][i] = LB[swz(brow + i * 32, cn)];
                    } else if (more1) {
                        fa[0][i] = lds[na * SLAB + swz(arow + i * 32, half)];
                        if (i < SN) fb[0][i] = lds[s3 * SLAB + swz(brow + i * 32, half)];
                    }
                    const int g = s * SM + i;
                    if (g < HL && more1) issue(srcb[g], offb, kt + 1, s3, g);
                    if (g >= HL && g < 2 * HL && more2) issue(srca[g - HL], offa, kt + 2, s4, g - HL);
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
            wa.next();
            wb.next();
            sa = na;
        }
    }

    // Tile<128>: both operands DEPTH steps ahead.  Step kt lives in slot kt % SLOTS of each operand's ring, and while it
    // is worked on the slots of step kt - 1 take step kt + DEPTH.
    template <typename V, int PARTS, bool KTAIL>
    static __device__ __attribute__((always_inline)) void run_deep(const char* const (&srca)[HL], const char* const (&srcb)[HL],
                                                                   size_t a_part, size_t b_part, size_t k0, int steps, int tail,
                                                                   u32x4* lds, Acc& out) {
        constexpr int BM = WM / 32, SLICES = SUB / KGROUPS;       // blocks of rows, k-slices of a step for this wave
        constexpr int BEFORE = (SLICES - 1) * BM;                  // loads of step kt + DEPTH issued before its barrier
        static_assert(2 * HL == SLICES * BM && BM == SN && SM == 1, "one load per group of MFMAs");
        const int lane = threadIdx.x & 63, wave = wave_id();
        const int pos = wave % (NWAVES / KGROUPS), kg = wave / (NWAVES / KGROUPS);
        const int wm = pos / WAVES_N, wn = pos % WAVES_N;
        const int total = steps * Order<PARTS>::N;
        Walk<PARTS> wa(Order<PARTS>::A, a_part, k0, steps), wb(Order<PARTS>::B, b_part, k0, steps);
        // load j of step kt: 0 .. HL - 1 of A, HL .. 2 HL - 1 of B
        auto issue = [&](int kt, int slot, int j) {
            const bool b = j >= HL;
            const char* from = b ? srcb[j - HL] + wb.off : srca[j] + wa.off;
            if (KTAIL && kt == total - 1)
                from = load_chunk(b ? j - HL : j) < tail ? from : reinterpret_cast<const char*>(&zero_chunk);
            __builtin_amdgcn_global_load_lds((const void*)from,
                                             (lds_ptr_t)(lds + ((b ? SLOTS : 0) + slot) * SLAB + (wave * HL + (b ? j - HL : j)) * 64),
                                             16, 0, 0);
        };
#pragma unroll
        for (int kt = 0; kt < DEPTH; ++kt)
            if (kt < total) {
#pragma unroll
                for (int j = 0; j < 2 * HL; ++j) issue(kt, kt, j);
                wa.next();
                wb.next();
            }
        const int arow = wm * WM + (lane & 31), brow = wn * WN + (lane & 31);
        const int c0 = 2 * SLICES * kg + (lane >> 5);   // this lane's first chunk of a step's rows
        const u32x4* ldsb = lds + SLOTS * SLAB;
        f32x16_t acc[BM][SN] = {};
        u32x4 fa[2][BM], fb[2][SN];
        if (total >= DEPTH)
            asm volatile("s_waitcnt vmcnt(%0)" ::"n"((DEPTH - 1) * 2 * HL) : "memory");
        else
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        asm volatile("s_barrier" ::: "memory");
#pragma unroll
        for (int i = 0; i < BM; ++i) {
            fa[0][i] = lds[swz(arow + i * 32, c0)];
            fb[0][i] = ldsb[swz(brow + i * 32, c0)];
        }
        int sl = 0;   // slot of step kt
        for (int kt = 0; kt < total; ++kt) {
            const int nx = sl + 1 == SLOTS ? 0 : sl + 1, fill = sl == 0 ? SLOTS - 1 : sl - 1;
            const bool more1 = kt + 1 < total, more = kt + DEPTH < total;
            scale_cross<PARTS>(acc, kt, steps);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int s = 0; s < SLICES; ++s) {
                if (s == SLICES - 1 && more1) {
                    // this step's slabs have been read and this wave's loads of step kt + 1 are done; those of
                    // the DEPTH - 2 steps after it, and of step kt + DEPTH so far, may be in flight (the
                    // last steps, which load nothing, wait for all)
                    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
                    if (more)
                        asm volatile("s_waitcnt vmcnt(%0)" ::"n"((DEPTH - 2) * 2 * HL + BEFORE) : "memory");
                    else
                        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
                    asm volatile("s_barrier" ::: "memory");
                    __builtin_amdgcn_sched_barrier(0);
                }
                const bool in = s + 1 < SLICES;
                const u32x4 *LA = lds + (in ? sl : nx) * SLAB, *LB = ldsb + (in ? sl : nx) * SLAB;
                const int cn = in ? c0 + 2 * (s + 1) : c0;
#pragma unroll
                for (int i = 0; i < BM; ++i) {
                    if (in || more1) {
                        fa[(s + 1) & 1][i] = LA[swz(arow + i * 32, cn)];
                        fb[(s + 1) & 1][i] = LB[swz(brow + i * 32, cn)];
                    }
#pragma unroll
                    for (int j = 0; j < SN; ++j)
                        mfma<V>(acc[i][j], fa[s & 1][i], fb[s & 1][j]);
                    if (more) issue(kt + DEPTH, fill, s * BM + i);
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
            wa.next();
            wb.next();
            sl = nx;
        }
        // block row kg of the pair's sum stays here, the other goes to the partner: [wave][register][lane]
        lds_barrier();
        float* x = reinterpret_cast<float*>(lds);
#pragma unroll
        for (int j = 0; j < SN; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) x[((wave * SN + j) * 16 + r) * 64 + lane] = kg ? acc[0][j][r] : acc[1][j][r];
        lds_barrier();
        const int partner = wave ^ (NWAVES / KGROUPS);
#pragma unroll
        for (int j = 0; j < SN; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r)
                out[0][j][r] += (kg ? acc[1][j][r] : acc[0][j][r]) + x[((partner * SN + j) * 16 + r) * 64 + lane];
    }

    // Accumulator register 4 g + p of block (i, j) holds, in lane l of wave (wm, wn), C element
    //   row share_row(w) + 32 i + 8 g + 4 (l >> 5) + p,  column share_col(w) + 32 j + (l & 31).
    static __device__ __forceinline__ int share_row(int wave) {
        constexpr int POS = NWAVES / KGROUPS;
        return WM * (wave % POS / WAVES_N) + 32 * SM * (wave / POS);
    }
    static __device__ __forceinline__ int share_col(int wave) { return WN * (wave % (NWAVES / KGROUPS) % WAVES_N); }
    static __device__ __forceinline__ int column(int j) { return share_col(wave_id()) + 32 * j + (static_cast<int>(threadIdx.x) & 31); }
    static __device__ __forceinline__ int first_row() { return share_row(wave_id()) + 4 * ((static_cast<int>(threadIdx.x) >> 5) & 1); }
    // Waves whose shares lie on top of each other in the same columns, and this wave's place among them.
    static constexpr int STACKED = EDGE / (32 * SM);
    static __device__ __forceinline__ int stack_place() { return share_row(wave_id()) / (32 * SM); }

    // Staging as 16-bit values: column c at 2 EDGE c bytes, its rows in units of 4 (8 bytes), unit u at
    // position u ^ csw(c): a lane's 4 rows are one write, free of bank conflicts, and a column is read
    // back in order (16 bytes = 8 rows).
    static __device__ __forceinline__ int csw(int c) { return (c & 31) ^ (((c >> 5) & 1) << 2); }
    struct Stage {
        int wbase[SN];
        __device__ Stage() {
#pragma unroll
            for (int j = 0; j < SN; ++j) {
                const int c = column(j);
                wbase[j] = c * (2 * EDGE) + ((2 * first_row()) ^ (8 * csw(c)));
            }
        }
        __device__ __forceinline__ void put(lds_byte_t* L, int i, int j, int g, unsigned w0, unsigned w1) const {
            *(lds_u32x2_t*)(L + (wbase[j] ^ (64 * i + 16 * g))) = u32x2_t{w0, w1};
        }
        __device__ __forceinline__ void put_all(lds_byte_t* L, const Acc& acc) const {
#pragma unroll
            for (int i = 0; i < SM; ++i)
#pragma unroll
                for (int j = 0; j < SN; ++j)
#pragma unroll
                    for (int g = 0; g < 4; ++g)
                        put(L, i, j, g, pack_bf16x2(acc[i][j][4 * g], acc[i][j][4 * g + 1]),
                            pack_bf16x2(acc[i][j][4 * g + 2], acc[i][j][4 * g + 3]));
        }
        __device__ __forceinline__ void put_all_f16(lds_byte_t* L, const Acc& acc) const {
            typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
            auto two = [](float a, float b) {
                return __builtin_bit_cast(unsigned, f16x2_t{static_cast<_Float16>(a), static_cast<_Float16>(b)});
            };
#pragma unroll
            for (int i = 0; i < SM; ++i)
#pragma unroll
                for (int j = 0; j < SN; ++j)
#pragma unroll
                    for (int g = 0; g < 4; ++g)
                        put(L, i, j, g, two(acc[i][j][4 * g], acc[i][j][4 * g + 1]), two(acc[i][j][4 * g + 2], acc[i][j][4 * g + 3]));
        }
    };
    // Rows 8 q .. 8 q + 7 of column c.
    static __device__ __forceinline__ u32x4 stage_col8(const lds_byte_t* L, int c, int q) {
        const int s = csw(c);
        const u32x4 v = *(const lds_u32x4_t*)(L + (c * (2 * EDGE) + 16 * (q ^ (s >> 1))));
        return (s & 1) ? u32x4{v.z, v.w, v.x, v.y} : v;
    }
    // Staging as fp32, 128 columns at a time (pass = c / 128): column c at 4 EDGE (c % 128) bytes, its rows in
    // units of 4 (16 bytes), unit u at position u ^ (c & 31).
    static constexpr int F32_PASSES = EDGE / 128;
    static __device__ __forceinline__ void put_f32(lds_byte_t* L, const Acc& acc, int pass) {
#pragma unroll
        for (int j = 0; j < SN; ++j) {
            const int c = column(j);
            if (c / 128 != pass) continue;   // the same for a whole wave
#pragma unroll
            for (int i = 0; i < SM; ++i)
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const int u = (first_row() + 32 * i + 8 * g) / 4;
                    *(lds_u32x4_t*)(L + ((c % 128) * (4 * EDGE) + 16 * (u ^ (c & 31)))) =
                        u32x4{__float_as_uint(acc[i][j][4 * g]), __float_as_uint(acc[i][j][4 * g + 1]),
                              __float_as_uint(acc[i][j][4 * g + 2]), __float_as_uint(acc[i][j][4 * g + 3])};
                }
        }
    }
    static __device__ __forceinline__ u32x4 stage_f32(const lds_byte_t* L, int c, int u) {
        return *(const lds_u32x4_t*)(L + ((c % 128) * (4 * EDGE) + 16 * (u ^ (c & 31))));
    }
};

// The accumulators of column j times 2^e[j]: both operands' scales, powers of two, at once (either alone might leave fp32's range).
template <typename TL> __device__ __forceinline__ void unscale(typename TL::Acc& acc, const int (&e)[TL::SN]) {
#pragma unroll
    for (int i = 0; i < TL::SM; ++i)
#pragma unroll
        for (int j = 0; j < TL::SN; ++j)
#pragma unroll
            for (int q = 0; q < 16; ++q) {
                acc[i][j][q] = __builtin_amdgcn_ldexpf(acc[i][j][q], e[j]);
                asm volatile("" : "+v"(acc[i][j][q]));   // here and in place
            }
}

// Tiles in runs of 32 on one XCD (the hardware deals workgroups round-robin over the 8), a
// bijection on [0, nb): a run is a 4 x 8 block of tiles whose operand panels share an L2.
constexpr int XCDS = 8, XCD_RUN = 32, GROUP = 4;
__device__ __forceinline__ int xcd_remap(int b, int nb) {
    const int full = (nb / (XCDS * XCD_RUN)) * (XCDS * XCD_RUN);
    if (b >= full) return b;
    const int xcd = b % XCDS, slot = b / XCDS;
    return ((slot / XCD_RUN) * XCDS + xcd) * XCD_RUN + slot % XCD_RUN;
}
// Tile t of ta x tb tiles, in groups of GROUP tiles of b, a-major inside a group.
__device__ __forceinline__ void tile_of(int t, int ta, int tb, int& ia, int& ib) {
    const int per = GROUP * ta, g = t / per, r = t - g * per, first = g * GROUP;
    const int size = min(tb - first, GROUP);
    ia = r / size;
    ib = first + r - ia * size;
}

}  // namespace pt

}  // namespace muon
