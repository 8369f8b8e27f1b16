// Norms around a block with its gate and residual scale, forward and backward.
//
//   a = x rstd0 wp,  r' = alpha r + g a,  n = r' rstd1 wq,  rstd = 1 / sqrt(mean(v^2) + eps)
// and, from dn and dr' (with h = r' rstd1, xh = x rstd0):
//   dh = dn wq,  R = dr' + rstd1 (dh - h mean(dh h)),  dr = alpha R,  dg = R a,
//   da = R g,  dxh = da wp,  dx = rstd0 (dxh - xh mean(dxh xh)),
//   dwq = sum dn h,  dwp = sum da xh  over the rows.
// One workgroup per row (forward) or per run of rows (backward), every pass over the
// row reading it again.
#include "train_internal.h"

namespace muon {

namespace {

constexpr int BN_THREADS = 256;
constexpr int BN_MAX_PARTS = 256;   // row runs of the backward pass, one partial weight gradient each

struct RowIo {
    int dt, wdt;
    __device__ float mat(const void* p, size_t i) const { return ld_dt(p, i, dt); }
    __device__ float wt(const void* p, size_t i) const { return p ? ld_dt(p, i, wdt) : 1.0f; }
    __device__ float gate(const void* p, int kind, size_t row_off, int c) const {
        return kind == MUON_GATE_NONE ? 1.0f : kind == MUON_GATE_CHANNEL ? ld_dt(p, c, wdt) : ld_dt(p, row_off + c, dt);
    }
};

__global__ __launch_bounds__(BN_THREADS) void block_norm_kernel(muon_block_norm_args a) {
    __shared__ float red[BN_THREADS / 64];
    const RowIo io{a.dtype, a.weight_dtype};
    const size_t row = blockIdx.x;
    const int d = static_cast<int>(a.cols);
    const size_t xo = row * a.ld_x, ro = row * a.ld_residual, go = row * a.ld_gate;
    float s0 = 1.0f;
    if (a.post_weight) {
        float s = 0.0f;
        for (int c = threadIdx.x; c < d; c += BN_THREADS) {
            const float v = io.mat(a.x, xo + c);
            s += v * v;
        }
        s0 = 1.0f / sqrtf(block_sum<BN_THREADS>(s, red) / d + a.eps);
    }
    auto joined = [&](int c) {
        return a.residual_scale * io.mat(a.residual, ro + c) +
               io.gate(a.gate, a.gate_kind, go, c) * (io.mat(a.x, xo + c) * s0 * io.wt(a.post_weight, c));
    };
    float s1 = 1.0f;
    if (a.out_norm) {
        float s = 0.0f;
        for (int c = threadIdx.x; c < d; c += BN_THREADS) {
            const float v = joined(c);
            s += v * v;
        }
        s1 = 1.0f / sqrtf(block_sum<BN_THREADS>(s, red) / d + a.eps);
    }
    for (int c = threadIdx.x; c < d; c += BN_THREADS) {
        const float v = joined(c);
        st_dt(a.out_residual, row * a.ld_out_residual + c, v, a.dtype);
        if (a.out_norm) st_dt(a.out_norm, row * a.ld_out_norm + c, v * s1 * io.wt(a.pre_weight, c), a.dtype);
    }
    if (a.rstd && threadIdx.x == 0) {
        a.rstd[row] = s0;
        a.rstd[a.rows + row] = s1;
    }
}

__global__ __launch_bounds__(BN_THREADS) void block_norm_backward_kernel(muon_block_norm_backward_args a, float* part) {
    __shared__ float red[BN_THREADS / 64];
    const RowIo io{a.dtype, a.weight_dtype};
    const int d = static_cast<int>(a.cols);
    float* pp = part + static_cast<size_t>(blockIdx.x) * 3 * d;   // post weight, gate, pre weight
    for (int c = threadIdx.x; c < 3 * d; c += BN_THREADS) pp[c] = 0.0f;
    __syncthreads();
    for (size_t row = blockIdx.x; row < static_cast<size_t>(a.rows); row += gridDim.x) {
        const float s0 = a.rstd[row], s1 = a.rstd[a.rows + row];
        const size_t xo = row * a.ld_x, ho = row * a.ld_out_residual, no = row * a.ld_grad_norm,
                     uo = row * a.ld_grad_out_residual, go = row * a.ld_gate;
        auto hat = [&](int c) { return io.mat(a.out_residual, ho + c) * s1; };
        auto dhat = [&](int c) { return io.mat(a.grad_norm, no + c) * io.wt(a.pre_weight, c); };
        float m1 = 0.0f;
        if (a.grad_norm) {
            for (int c = threadIdx.x; c < d; c += BN_THREADS) m1 += dhat(c) * hat(c);
            m1 = block_sum<BN_THREADS>(m1, red) / d;
        }
        auto total = [&](int c) {
            float v = a.grad_out_residual ? io.mat(a.grad_out_residual, uo + c) : 0.0f;
            if (a.grad_norm) v += s1 * (dhat(c) - hat(c) * m1);
            return v;
        };
        float m0 = 0.0f;
        if (a.post_weight) {
            for (int c = threadIdx.x; c < d; c += BN_THREADS)
                m0 += total(c) * io.gate(a.gate, a.gate_kind, go, c) * io.wt(a.post_weight, c) * (io.mat(a.x, xo + c) * s0);
            m0 = block_sum<BN_THREADS>(m0, red) / d;
        }
        for (int c = threadIdx.x; c < d; c += BN_THREADS) {
            const float r = total(c), xh = io.mat(a.x, xo + c) * s0, w = io.wt(a.post_weight, c);
            const float da = r * io.gate(a.gate, a.gate_kind, go, c);
            if (a.grad_norm && a.grad_pre_weight) pp[2 * d + c] += io.mat(a.grad_norm, no + c) * hat(c);
            pp[c] += da * xh;
            if (a.gate_kind == MUON_GATE_CHANNEL) pp[d + c] += r * xh * w;
            if (a.gate_kind == MUON_GATE_FULL) st_dt(a.grad_gate, row * a.ld_grad_gate + c, r * xh * w, a.dtype);
            st_dt(a.grad_x, row * a.ld_grad_x + c, a.post_weight ? s0 * (da * w - xh * m0) : da, a.dtype);
            st_dt(a.grad_residual, row * a.ld_grad_residual + c, a.residual_scale * r, a.dtype);
        }
    }
}

// Sums the runs' partial weight gradients in run order.
__global__ __launch_bounds__(BN_THREADS) void block_norm_weights_kernel(muon_block_norm_backward_args a,
                                                                        const float* part, int parts) {
    const int d = static_cast<int>(a.cols);
    const int c = blockIdx.x * BN_THREADS + threadIdx.x;
    if (c >= d) return;
    void* outs[3] = {a.grad_post_weight, a.gate_kind == MUON_GATE_CHANNEL ? a.grad_gate : nullptr, a.grad_pre_weight};
    for (int k = 0; k < 3; ++k) {
        if (!outs[k]) continue;
        float s = 0.0f;
        for (int p = 0; p < parts; ++p) s += part[(static_cast<size_t>(p) * 3 + k) * d + c];
        st_dt(outs[k], c, s, a.weight_dtype);
    }
}

int backward_parts(const muon_block_norm_backward_args& a) {
    return static_cast<int>(a.rows < BN_MAX_PARTS ? a.rows : BN_MAX_PARTS);
}

}  // namespace

hipError_t launch_block_norm(const muon_block_norm_args& a, hipStream_t s) {
    if (a.rows == 0) return hipSuccess;
    hipLaunchKernelGGL(block_norm_kernel, dim3(static_cast<unsigned>(a.rows)), dim3(BN_THREADS), 0, s, a);
    return hipGetLastError();
}

size_t block_norm_backward_bytes(const muon_block_norm_backward_args& a) {
    return static_cast<size_t>(backward_parts(a)) * 3 * a.cols * sizeof(float);
}

hipError_t launch_block_norm_backward(const muon_block_norm_backward_args& a, void* workspace, hipStream_t s) {
    float* part = static_cast<float*>(workspace);
    const int parts = backward_parts(a);
    if (parts > 0) {
        hipLaunchKernelGGL(block_norm_backward_kernel, dim3(parts), dim3(BN_THREADS), 0, s, a, part);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    const unsigned grid = static_cast<unsigned>((a.cols + BN_THREADS - 1) / BN_THREADS);
    hipLaunchKernelGGL(block_norm_weights_kernel, dim3(grid), dim3(BN_THREADS), 0, s, a, part, parts);
    return hipGetLastError();
}

}  // namespace muon
