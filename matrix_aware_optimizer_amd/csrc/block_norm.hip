// Norms around a block with its gate and residual scale, forward and backward.
//
//   a = x rstd0 wp,  r' = alpha r + g a,  n = r' rstd1 wq,  rstd = 1 / sqrt(mean(v^2) + eps)
// and, from dn and dr' (with h = r' rstd1, xh = x rstd0):
//   dh = dn wq,  R = dr' + rstd1 (dh - h mean(dh h)),  dr = alpha R,  dg = R a,
//   da = R g,  dxh = da wp,  dx = rstd0 (dxh - xh mean(dxh xh)),
//   dwq = sum dn h,  dwp = sum da xh  over the rows.
//
// HBM-bound: the forward pass reads x and r and writes r' and n, the backward pass reads
// x, r', dn and dr' and writes dx and dr (a full gate adds one each way); a few operations
// per byte.  So a row is read once and kept, as fp32, by the NT threads that share it, in registers but for 16385 columns and
// more (6 to 116 values a thread go through scratch there):
// one wave for rows up to 1024 columns (forward; its sums need no barrier), 256 or 1024 threads
// for longer ones (1003 x 1407 fp32, both passes: 31.5 us, 34.2 with one wave a row; 8192 x 2048 bf16 the same with
// either).  The weights are read again for every row: they come from L2.
// 8192 x 2048 bf16: forward 24 - 26 us (134 MB, 5.4 TB/s), backward 45 us (201 MB, 4.5 TB/s) and 5.7 us for the weights' partials; fp32
// 55 (4.9 TB/s), 85 (4.8) and 6.5; one row: 2.7 - 3.8 us, a launch's length.  The backward kernel is held to 128 registers, 4 waves a
// SIMD: its forms for odd widths, for 2049 to 4096 columns and most in fp32 keep 2 to 19 values a thread in scratch (8192 x 4096 bf16: 105
// us, 3.8 TB/s).  Odd widths cost more than that, in both passes, by accesses that are not aligned: 1003 x 1407 fp32 31 us, x 1408 25;
// 8192 x 2047 bf16 168 us, x 2048 78.
//
// The backward pass needs mean(dxh xh), and dxh needs mean(dh h) first.  With q = g wp xh,
//   sum dxh xh = sum (dr' + rstd1 dh) q - rstd1 mean(dh h) sum h q,
// so the three sums sum dh h, sum (dr' + rstd1 dh) q and sum h q are taken together, one
// exchange per row instead of two.  Weight gradients stay in registers over a workgroup's rows (a
// thread keeps its columns) and end in one fp32 partial per workgroup, summed in a fixed order by
// block_norm_weights_kernel.
#include <algorithm>

#include "train_internal.h"

namespace muon {

namespace {

// Waves of the backward pass's workgroups, at most: 16 a CU (8192 x 2048 bf16, both passes: 78 us; 8 a CU 83, 32 a CU 89).
constexpr int64_t BN_WAVES = 4096;
// Rows of a workgroup, at least: each leaves a partial weight gradient to sum (1003 x 1407 fp32: 34 us; one row 36, eight 52).
constexpr int64_t BN_ROWS = 2;
constexpr int64_t BN_LONG = 8192;   // longest row that one workgroup's registers hold in the backward pass
constexpr int BN_CHUNK = 2048;      // columns of a longer row a workgroup takes at a time

// Which of the workgroup's rows this thread works on: the same for a whole wave, so that row addresses are
// scalar.
template <int NT> __device__ __forceinline__ int row_of_thread() {
    return __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x / NT));
}

// The 8 VPT columns of a row that one of its NT threads keeps: VPT runs of 8, NT runs apart.  TAIL: the last
// run of the row may be short.
template <int NT, int VPT, bool TAIL> struct Cols {
    static constexpr int N = 8 * VPT;
    unsigned cols, t;   // t: the thread's first run
    __device__ unsigned run(int v) const { return (v * NT + t) * 8; }
    __device__ bool has(int k) const { return TAIL ? run(k / 8) + k % 8 < cols : run(k / 8) < cols; }
    template <typename T> __device__ __forceinline__ void load(const void* p, size_t off, float (&o)[N]) const {
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const auto* q = G(static_cast<const T*>(p) + off);
            Run<T> w;
            if (TAIL ? run(v) + 8 <= cols : run(v) < cols) w.load(q, run(v));
            else if (TAIL && run(v) < cols) w.load(q, run(v), cols - run(v));
#pragma unroll
            for (int e = 0; e < 8; ++e) o[8 * v + e] = w.get(e);
        }
    }
    template <typename T> __device__ __forceinline__ void store(void* p, size_t off, const float (&o)[N]) const {
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            auto* q = G(static_cast<T*>(p) + off);
            float w[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e] = o[8 * v + e];
            if (TAIL ? run(v) + 8 <= cols : run(v) < cols) st_run(q, run(v), w);
            else if (TAIL && run(v) < cols)
#pragma unroll
                for (int e = 0; e < 7; ++e)
                    if (run(v) + e < cols) st_el<T>(p, off + run(v) + e, w[e]);
        }
    }
    // a weight vector; 1 where there is none
    __device__ __forceinline__ void weight(const void* p, int dt, float (&o)[N]) const {
        if (!p) {
#pragma unroll
            for (int k = 0; k < N; ++k) o[k] = 1.0f;
        } else if (dt == DT_BF16) {
            load<uint16_t>(p, 0, o);
        } else {
            load<float>(p, 0, o);
        }
    }
    template <typename T>
    __device__ __forceinline__ void gate(const void* p, int kind, int wdt, size_t off, float (&o)[N]) const {
        if (kind == MUON_GATE_FULL) load<T>(p, off, o);
        else weight(kind == MUON_GATE_CHANNEL ? p : nullptr, wdt, o);
    }
};

// Sums over the NT threads of one row, NS at a time, given to all of them.  `red` holds NS floats per
// wave of the workgroup, twice: rows take the two halves in turn, so one barrier per call is enough.
template <int NT, int NS, int WAVES>
__device__ __forceinline__ void row_sums(float (&v)[NS], float* red, int turn) {
#pragma unroll
    for (int k = 0; k < NS; ++k) v[k] = wave_sum(v[k]);
    if constexpr (NT > 64) {
        float* r = red + (turn & 1) * NS * WAVES;
        const int wave = threadIdx.x >> 6, first = wave / (NT / 64) * (NT / 64);
        if ((threadIdx.x & 63) == 0)
#pragma unroll
            for (int k = 0; k < NS; ++k) r[k * WAVES + wave] = v[k];
        lds_barrier();
#pragma unroll
        for (int k = 0; k < NS; ++k) {
            v[k] = r[k * WAVES + first];
#pragma unroll
            for (int w = 1; w < NT / 64; ++w) v[k] += r[k * WAVES + first + w];
        }
    }
}

// row0: the launch's first row.
template <typename T, int NT, int VPT, bool TAIL>
__global__ __launch_bounds__(NT < 256 ? 256 : NT) void block_norm_kernel(muon_block_norm_args a, int64_t row0) {
    constexpr int BLOCK = NT < 256 ? 256 : NT, PER = BLOCK / NT, N = 8 * VPT;
    __shared__ float red[2 * BLOCK / 64];
    const int64_t row = row0 + static_cast<int64_t>(blockIdx.x) * PER + row_of_thread<NT>();
    if (NT == 64 && row >= a.rows) return;   // longer rows: one per workgroup, none past the last
    const Cols<NT, VPT, TAIL> c{static_cast<unsigned>(a.cols), threadIdx.x % NT};
    const float inv = 1.0f / static_cast<float>(a.cols);
    float x[N], y[N], w[N], gt[N];
    c.template load<T>(a.x, row * a.ld_x, x);
    c.template load<T>(a.residual, row * a.ld_residual, y);
    c.template gate<T>(a.gate, a.gate_kind, a.weight_dtype, row * a.ld_gate, gt);
    c.weight(a.post_weight, a.weight_dtype, w);
    float s0 = 1.0f, s1 = 1.0f;
    if (a.post_weight) {
        float s[1] = {0.0f};
#pragma unroll
        for (int k = 0; k < N; ++k) s[0] = fmaf(x[k], x[k], s[0]);
        row_sums<NT, 1, BLOCK / 64>(s, red, 0);
        s0 = 1.0f / sqrtf(fmaf(s[0], inv, a.eps));
    }
#pragma unroll
    for (int k = 0; k < N; ++k) y[k] = fmaf(gt[k], x[k] * s0 * w[k], a.residual_scale * y[k]);
    c.template store<T>(a.out_residual, row * a.ld_out_residual, y);
    if (a.out_norm) {
        c.weight(a.pre_weight, a.weight_dtype, w);
        float s[1] = {0.0f};
#pragma unroll
        for (int k = 0; k < N; ++k) s[0] += c.has(k) ? y[k] * y[k] : 0.0f;
        row_sums<NT, 1, BLOCK / 64>(s, red, 1);
        s1 = 1.0f / sqrtf(fmaf(s[0], inv, a.eps));
#pragma unroll
        for (int k = 0; k < N; ++k) y[k] = y[k] * s1 * w[k];
        c.template store<T>(a.out_norm, row * a.ld_out_norm, y);
    }
    if (a.rstd && threadIdx.x % NT == 0) {
        a.rstd[row] = s0;
        a.rstd[a.rows + row] = s1;
    }
}

constexpr int bwd_block(int nt) { return nt < 256 ? 256 : nt; }

// What the backward pass reads of one row, and the sums it needs of it.
template <typename T, typename C> struct BackwardRow {
    static constexpr int N = C::N;
    float x[N], h[N], dn[N], tot[N], gt[N], wp[N];   // xh, h, dn, dr' (then dr' + rstd1 dh), gate, wp
    float s0, s1;
    __device__ __forceinline__ void load(const muon_block_norm_backward_args& a, const C& c, int64_t row) {
        c.template load<T>(a.x, row * a.ld_x, x);
        c.template load<T>(a.out_residual, row * a.ld_out_residual, h);
        if (a.grad_norm) {
            c.template load<T>(a.grad_norm, row * a.ld_grad_norm, dn);
        } else {
#pragma unroll
            for (int k = 0; k < N; ++k) dn[k] = 0.0f;
        }
        if (a.grad_out_residual) {
            c.template load<T>(a.grad_out_residual, row * a.ld_grad_out_residual, tot);
        } else {
#pragma unroll
            for (int k = 0; k < N; ++k) tot[k] = 0.0f;
        }
        c.template gate<T>(a.gate, a.gate_kind, a.weight_dtype, row * a.ld_gate, gt);
        c.weight(a.post_weight, a.weight_dtype, wp);
        s0 = a.rstd[row];
        s1 = a.rstd[a.rows + row];
    }
    // adds this thread's share of sum dh h, sum (dr' + rstd1 dh) q, sum h q
    __device__ __forceinline__ void sums(const muon_block_norm_backward_args& a, const C& c, float (&s)[3]) {
        float wq[N];
        c.weight(a.pre_weight, a.weight_dtype, wq);
#pragma unroll
        for (int k = 0; k < N; ++k) {
            x[k] *= s0;
            h[k] *= s1;
            const float dh = dn[k] * wq[k], q = gt[k] * wp[k] * x[k];
            s[0] = fmaf(dh, h[k], s[0]);
            tot[k] = fmaf(s1, dh, tot[k]);
            s[1] = fmaf(tot[k], q, s[1]);
            s[2] = fmaf(h[k], q, s[2]);
        }
    }
    // m1 = rstd1 mean(dh h), m0 = mean(dxh xh)
    static __device__ __forceinline__ void means(const float (&s)[3], float s1, float inv, float& m1, float& m0) {
        m1 = s1 * (s[0] * inv);
        m0 = (s[1] - m1 * s[2]) * inv;
    }
};

// Rows beyond BN_LONG: m1 and m0 of each, one workgroup a row, from row0 on.
template <typename T, bool TAIL>
__global__ __launch_bounds__(1024) void block_norm_means_kernel(muon_block_norm_backward_args a, float* means, int64_t row0) {
    __shared__ float red[2 * 3 * 16];
    const int64_t row = row0 + blockIdx.x;
    float s[3] = {0.0f, 0.0f, 0.0f}, s1 = 1.0f;
    for (unsigned c0 = 0; c0 < a.cols; c0 += 8192) {
        const Cols<1024, 1, TAIL> c{static_cast<unsigned>(a.cols), threadIdx.x + c0 / 8};
        BackwardRow<T, Cols<1024, 1, TAIL>> r;
        r.load(a, c, row);
        r.sums(a, c, s);
        s1 = r.s1;
    }
    row_sums<1024, 3, 16>(s, red, 0);
    if (threadIdx.x == 0) {
        float m1, m0;
        BackwardRow<T, Cols<1024, 1, TAIL>>::means(s, s1, 1.0f / static_cast<float>(a.cols), m1, m0);
        means[row] = m1;
        means[a.rows + row] = m0;
    }
}

// GIVEN: the rows' means come from block_norm_means_kernel and blockIdx.y is the run of BN_CHUNK columns.
template <typename T, int NT, bool TAIL, bool GIVEN>
__global__ __launch_bounds__(bwd_block(NT), 4) void block_norm_backward_kernel(
    muon_block_norm_backward_args a, float* part, const float* means) {
    constexpr int BLOCK = bwd_block(NT), PER = BLOCK / NT, WAVES = BLOCK / 64, N = 8;
    typedef Cols<NT, 1, TAIL> C;
    __shared__ float red[2 * 3 * WAVES];
    __shared__ float join[PER > 1 ? PER * NT * N : 1];
    const int g = row_of_thread<NT>();
    const C c{static_cast<unsigned>(a.cols), threadIdx.x % NT + (GIVEN ? blockIdx.y * (BN_CHUNK / 8) : 0)};
    const float inv = 1.0f / static_cast<float>(a.cols);
    float swp[N] = {}, sg[N] = {}, swq[N] = {};   // this thread's columns of the weight gradients
    int turn = 0;
    for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * PER; r0 < a.rows; r0 += static_cast<int64_t>(gridDim.x) * PER, ++turn) {
        const bool on = r0 + g < a.rows;
        const int64_t row = on ? r0 + g : a.rows - 1;
        BackwardRow<T, C> r;
        r.load(a, c, row);
        float s[3] = {0.0f, 0.0f, 0.0f}, m1, m0;
        r.sums(a, c, s);
        if constexpr (GIVEN) {
            m1 = means[row];
            m0 = means[a.rows + row];
        } else {
            row_sums<NT, 3, WAVES>(s, red, turn);
            r.means(s, r.s1, inv, m1, m0);
        }
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const float tot = fmaf(-m1, r.h[k], r.tot[k]), da = tot * r.gt[k], xw = r.x[k] * r.wp[k];
            if (on) {
                swq[k] = fmaf(r.dn[k], r.h[k], swq[k]);
                swp[k] = fmaf(da, r.x[k], swp[k]);
                sg[k] = fmaf(tot, xw, sg[k]);
            }
            r.h[k] = a.post_weight ? r.s0 * (da * r.wp[k] - r.x[k] * m0) : da;   // dx
            r.x[k] = tot * xw;                                                  // dg of this row
            r.tot[k] = a.residual_scale * tot;
        }
        if (on) {
            c.template store<T>(a.grad_x, row * a.ld_grad_x, r.h);
            c.template store<T>(a.grad_residual, row * a.ld_grad_residual, r.tot);
            if (a.gate_kind == MUON_GATE_FULL) c.template store<T>(a.grad_gate, row * a.ld_grad_gate, r.x);
        }
    }
    // the workgroup's rows share its columns: their sums are joined in LDS, in order
    float* out = part + static_cast<size_t>(blockIdx.x) * 3 * a.cols;
#pragma unroll
    for (int which = 0; which < 3; ++which) {
        float (&s)[N] = which == 0 ? swp : which == 1 ? sg : swq;
        if (which == 1 && a.gate_kind != MUON_GATE_CHANNEL) continue;
        if constexpr (PER > 1) {
            __syncthreads();
#pragma unroll
            for (int k = 0; k < N; ++k) join[(g * N + k) * NT + threadIdx.x % NT] = s[k];
            __syncthreads();
            if (g == 0)
#pragma unroll
                for (int k = 0; k < N; ++k)
#pragma unroll
                    for (int p = 1; p < PER; ++p) s[k] += join[(p * N + k) * NT + threadIdx.x % NT];
        }
        if (g == 0) c.template store<float>(out, which * a.cols, s);
    }
}

// Sums the workgroups' partial weight gradients in order: 64 columns x 16 runs of partials a workgroup.
__global__ __launch_bounds__(1024) void block_norm_weights_kernel(muon_block_norm_backward_args a, const float* part,
                                                                  int parts) {
    __shared__ float run[16][64];
    const int which = blockIdx.y;
    void* out = which == 0 ? a.grad_post_weight
                           : which == 1 ? (a.gate_kind == MUON_GATE_CHANNEL ? a.grad_gate : nullptr) : a.grad_pre_weight;
    if (!out) return;
    const int64_t c = static_cast<int64_t>(blockIdx.x) * 64 + (threadIdx.x & 63);
    const int r = threadIdx.x >> 6, per = (parts + 15) / 16;
    float s = 0.0f;
    if (c < a.cols) {
        const float* p = part + which * a.cols + c;
#pragma unroll 8
        for (int k = r * per; k < min(parts, (r + 1) * per); ++k) s += p[static_cast<size_t>(k) * 3 * a.cols];
    }
    run[r][threadIdx.x & 63] = s;
    __syncthreads();
    if (r != 0 || c >= a.cols) return;
#pragma unroll
    for (int k = 1; k < 16; ++k) s += run[k][threadIdx.x];
    st_dt(out, c, s, a.weight_dtype);
}

// launch(first row, grid) for `per` rows a workgroup of `threads`: as many launches as it takes, since one holds fewer than 2^32
// threads (at 64 columns beyond 2^26 rows, at 8192 beyond 2^22).
template <typename F> hipError_t in_launches(int64_t rows, int per, int threads, F launch) {
    const int64_t most = (int64_t{1} << 31) / threads * per;
    for (int64_t row0 = 0; row0 < rows; row0 += most) {
        launch(row0, dim3(static_cast<unsigned>((std::min(rows - row0, most) + per - 1) / per)));
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

template <typename T, int NT, int VPT> hipError_t forward(const muon_block_norm_args& a, hipStream_t s) {
    constexpr int BLOCK = NT < 256 ? 256 : NT;
    return in_launches(a.rows, BLOCK / NT, BLOCK, [&](int64_t row0, dim3 grid) {
        if (a.cols % 8) hipLaunchKernelGGL((block_norm_kernel<T, NT, VPT, true>), grid, dim3(BLOCK), 0, s, a, row0);
        else hipLaunchKernelGGL((block_norm_kernel<T, NT, VPT, false>), grid, dim3(BLOCK), 0, s, a, row0);
    });
}

template <typename T> hipError_t forward_by_cols(const muon_block_norm_args& a, hipStream_t s) {
    if (a.cols <= 512) return forward<T, 64, 1>(a, s);
    if (a.cols <= 1024) return forward<T, 64, 2>(a, s);
    if (a.cols <= 2048) return forward<T, 256, 1>(a, s);
    if (a.cols <= 4096) return forward<T, 256, 2>(a, s);
    if (a.cols <= 8192) return forward<T, 1024, 1>(a, s);
    if (a.cols <= 16384) return forward<T, 1024, 2>(a, s);
    return forward<T, 1024, 4>(a, s);
}

// Threads per row of the backward pass.
int backward_threads(int64_t cols) { return cols <= 512 ? 64 : cols <= 2048 || cols > BN_LONG ? 256 : cols <= 4096 ? 512 : 1024; }
int64_t backward_chunks(int64_t cols) { return cols > BN_LONG ? (cols + BN_CHUNK - 1) / BN_CHUNK : 1; }
int64_t backward_parts(const muon_block_norm_backward_args& a) {
    const int block = bwd_block(backward_threads(a.cols));
    const int64_t per = BN_ROWS * (block / backward_threads(a.cols));
    return std::min((a.rows + per - 1) / per, std::max<int64_t>(1, BN_WAVES / (block / 64) / backward_chunks(a.cols)));
}
size_t backward_part_floats(const muon_block_norm_backward_args& a) { return static_cast<size_t>(backward_parts(a)) * 3 * a.cols; }

template <typename T, int NT, bool GIVEN = false>
hipError_t backward(const muon_block_norm_backward_args& a, float* part, const float* means, hipStream_t s) {
    const dim3 grid(static_cast<unsigned>(backward_parts(a)), static_cast<unsigned>(backward_chunks(a.cols))), block(bwd_block(NT));
    if (a.cols % 8) hipLaunchKernelGGL((block_norm_backward_kernel<T, NT, true, GIVEN>), grid, block, 0, s, a, part, means);
    else hipLaunchKernelGGL((block_norm_backward_kernel<T, NT, false, GIVEN>), grid, block, 0, s, a, part, means);
    return hipGetLastError();
}

template <typename T>
hipError_t backward_by_cols(const muon_block_norm_backward_args& a, float* part, hipStream_t s) {
    if (a.cols <= 512) return backward<T, 64>(a, part, nullptr, s);
    if (a.cols <= 2048) return backward<T, 256>(a, part, nullptr, s);
    if (a.cols <= 4096) return backward<T, 512>(a, part, nullptr, s);
    if (a.cols <= BN_LONG) return backward<T, 1024>(a, part, nullptr, s);
    // a row's accumulators and data no longer fit: its means first, then runs of columns (x, r', dn and dr' read twice)
    float* means = part + backward_part_floats(a);
    const hipError_t e = in_launches(a.rows, 1, 1024, [&](int64_t row0, dim3 grid) {
        if (a.cols % 8) hipLaunchKernelGGL((block_norm_means_kernel<T, true>), grid, dim3(1024), 0, s, a, means, row0);
        else hipLaunchKernelGGL((block_norm_means_kernel<T, false>), grid, dim3(1024), 0, s, a, means, row0);
    });
    return e != hipSuccess ? e : backward<T, 256, true>(a, part, means, s);
}

}  // namespace

hipError_t launch_block_norm(const muon_block_norm_args& a, hipStream_t s) {
    if (a.rows == 0) return hipSuccess;
    return a.dtype == MUON_BF16 ? forward_by_cols<uint16_t>(a, s) : forward_by_cols<float>(a, s);
}

size_t block_norm_backward_bytes(const muon_block_norm_backward_args& a) {
    return sizeof(float) * (backward_part_floats(a) + (a.cols > BN_LONG ? 2 * static_cast<size_t>(a.rows) : 0));
}

hipError_t launch_block_norm_backward(const muon_block_norm_backward_args& a, void* workspace, hipStream_t s) {
    float* part = static_cast<float*>(workspace);
    const int64_t parts = backward_parts(a);
    if (parts > 0) {
        const hipError_t e = a.dtype == MUON_BF16 ? backward_by_cols<uint16_t>(a, part, s)
                                                  : backward_by_cols<float>(a, part, s);
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL(block_norm_weights_kernel, dim3(static_cast<unsigned>((a.cols + 63) / 64), 3), dim3(1024), 0, s, a, part,
                       static_cast<int>(parts));
    return hipGetLastError();
}

}  // namespace muon
