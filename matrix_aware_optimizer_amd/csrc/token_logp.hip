// Log-probabilities of target tokens under a vocabulary head, and their gradients.
//
//   z = scale hidden head^T,  lse_i = log sum_j exp(z_ij),  logp_i = z_i,target_i - lse_i
//   dz_ij = scale grad_logp_i ([j = target_i] - exp(z_ij - lse_i))
//   grad_hidden = dz head,  grad_head = dz^T hidden
// z (tokens x vocab, fp32) is formed by a plain tiled product; dz replaces it in place.
#include "train_internal.h"

namespace muon {

namespace {

constexpr int TL_THREADS = 256;
constexpr int TL_TILE = 64, TL_K = 16;

// C[m][n] = scale sum_k A(m, k) B(k, n), A(m, k) at m * am + k * ak (likewise B and C).
// Rows m (live_m) or terms k (live_k) of a token that is not scored count as zero.
struct ProductArgs {
    const void *a, *b;
    void* c;
    size_t am, ak, bn, bk, cm;
    int adt, bdt, cdt;
    int64_t m, n, k;
    float scale;
    const int64_t *live_m, *live_k;
};

__global__ __launch_bounds__(TL_THREADS) void product_kernel(ProductArgs p) {
    __shared__ float as[TL_K][TL_TILE + 1], bs[TL_K][TL_TILE + 1];
    const int64_t m0 = static_cast<int64_t>(blockIdx.y) * TL_TILE, n0 = static_cast<int64_t>(blockIdx.x) * TL_TILE;
    const int tm = threadIdx.x / 16, tn = threadIdx.x % 16;
    float acc[4][4] = {};
    for (int64_t k0 = 0; k0 < p.k; k0 += TL_K) {
        for (int e = threadIdx.x; e < TL_TILE * TL_K; e += TL_THREADS) {
            const int64_t r = e / TL_K, k = k0 + e % TL_K;
            const bool lk = k < p.k && (!p.live_k || p.live_k[k] >= 0);
            as[e % TL_K][r] = lk && m0 + r < p.m ? ld_dt(p.a, (m0 + r) * p.am + k * p.ak, p.adt) : 0.0f;
            bs[e % TL_K][r] = lk && n0 + r < p.n ? ld_dt(p.b, (n0 + r) * p.bn + k * p.bk, p.bdt) : 0.0f;
        }
        __syncthreads();
        for (int k = 0; k < TL_K; ++k)
            for (int i = 0; i < 4; ++i)
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(as[k][tm + 16 * i], bs[k][tn + 16 * j], acc[i][j]);
        __syncthreads();
    }
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const int64_t m = m0 + tm + 16 * i, n = n0 + tn + 16 * j;
            if (m >= p.m || n >= p.n) continue;
            const bool live = !p.live_m || p.live_m[m] >= 0;
            st_dt(p.c, m * p.cm + n, live ? p.scale * acc[i][j] : 0.0f, p.cdt);
        }
}

hipError_t launch_product(const ProductArgs& p, hipStream_t s) {
    if (p.m == 0 || p.n == 0) return hipSuccess;
    const dim3 grid(static_cast<unsigned>((p.n + TL_TILE - 1) / TL_TILE), static_cast<unsigned>((p.m + TL_TILE - 1) / TL_TILE));
    hipLaunchKernelGGL(product_kernel, grid, dim3(TL_THREADS), 0, s, p);
    return hipGetLastError();
}

// One workgroup per token.  The target's own term is kept out of the sum:
// logp = -log(1 + sum_{j != target} exp(z_j - z_target)), which keeps its relative
// precision as logp goes to 0.
__global__ __launch_bounds__(TL_THREADS) void logp_rows_kernel(muon_token_logp_args a, const float* z) {
    __shared__ float red[TL_THREADS / 64], redm[TL_THREADS / 64];
    const int64_t row = blockIdx.x, y = a.targets[row];
    if (y < 0) {
        if (threadIdx.x == 0) { a.logp[row] = 0.0f; a.lse[row] = 0.0f; }
        return;
    }
    const float* zr = z + static_cast<size_t>(row) * a.vocab;
    float m = -INFINITY;
    for (int64_t j = threadIdx.x; j < a.vocab; j += TL_THREADS)
        if (j != y) m = fmaxf(m, zr[j]);
    for (int o = 32; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor(m, o, 64));
    if ((threadIdx.x & 63) == 0) redm[threadIdx.x >> 6] = m;
    __syncthreads();
    for (int w = 0; w < TL_THREADS / 64; ++w) m = fmaxf(m, redm[w]);
    float s = 0.0f;
    for (int64_t j = threadIdx.x; j < a.vocab; j += TL_THREADS)
        if (j != y && m > -INFINITY) s += expf(zr[j] - m);
    s = block_sum<TL_THREADS>(s, red);
    if (threadIdx.x != 0) return;
    if (y >= a.vocab) {
        a.logp[row] = NAN;
        a.lse[row] = m + logf(s);
        return;
    }
    const float zy = zr[y], d = m - zy;
    // s exp(d) overflows for a far-off target: there 1 is nothing beside it
    const float logp = s == 0.0f ? 0.0f : d < 60.0f ? -log1pf(s * expf(d)) : -(d + logf(s));
    a.logp[row] = logp;
    a.lse[row] = zy - logp;
}

__global__ __launch_bounds__(TL_THREADS) void dlogits_kernel(muon_token_logp_backward_args a, const float* z, float* dz) {
    const int64_t row = blockIdx.x, y = a.targets[row];
    const size_t off = static_cast<size_t>(row) * a.vocab;
    const float c = a.scale * a.grad_logp[row], lse = a.lse[row];
    for (int64_t j = threadIdx.x; j < a.vocab; j += TL_THREADS)
        dz[off + j] = y < 0 || c == 0.0f ? 0.0f : c * ((j == y ? 1.0f : 0.0f) - expf(z[off + j] - lse));
}

size_t logits_bytes(int64_t tokens, int64_t vocab) { return static_cast<size_t>(tokens) * vocab * sizeof(float); }

}  // namespace

size_t token_logp_saved_bytes(const muon_token_logp_args& a) { return logits_bytes(a.tokens, a.vocab); }
size_t token_logp_bytes(const muon_token_logp_args& a) { return logits_bytes(a.tokens, a.vocab); }
size_t token_logp_backward_bytes(const muon_token_logp_backward_args& a) { return logits_bytes(a.tokens, a.vocab); }

hipError_t launch_token_logp(const muon_token_logp_args& a, void* workspace, int cu_count, hipStream_t s) {
    if (a.tokens == 0) return hipSuccess;
    float* z = static_cast<float*>(a.saved ? a.saved : workspace);
    const ProductArgs p{a.hidden, a.head, z, static_cast<size_t>(a.ld_hidden), 1, static_cast<size_t>(a.ld_head), 1,
                        static_cast<size_t>(a.vocab), a.dtype, a.dtype, DT_F32, a.tokens, a.vocab, a.cols, a.scale,
                        nullptr, nullptr};
    const hipError_t e = launch_product(p, s);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(logp_rows_kernel, dim3(static_cast<unsigned>(a.tokens)), dim3(TL_THREADS), 0, s, a, z);
    return hipGetLastError();
}

hipError_t launch_token_logp_backward(const muon_token_logp_backward_args& a, void* workspace, int cu_count,
                                      hipStream_t s) {
    float* dz = static_cast<float*>(workspace);
    const float* z = static_cast<const float*>(a.saved ? a.saved : workspace);
    const size_t ldh = a.ld_hidden, ldw = a.ld_head, v = a.vocab;
    hipError_t e = hipSuccess;
    if (!a.saved) {
        const ProductArgs p{a.hidden, a.head, dz, ldh, 1, ldw, 1, v, a.dtype, a.dtype, DT_F32, a.tokens, a.vocab,
                            a.cols, a.scale, nullptr, nullptr};
        e = launch_product(p, s);
        if (e != hipSuccess) return e;
    }
    if (a.tokens > 0) {
        hipLaunchKernelGGL(dlogits_kernel, dim3(static_cast<unsigned>(a.tokens)), dim3(TL_THREADS), 0, s, a, z, dz);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (a.grad_hidden) {
        const ProductArgs p{dz, a.head, a.grad_hidden, v, 1, 1, ldw, static_cast<size_t>(a.ld_grad_hidden), DT_F32, a.dtype,
                            a.dtype, a.tokens, a.cols, a.vocab, 1.0f, a.targets, nullptr};
        e = launch_product(p, s);
        if (e != hipSuccess) return e;
    }
    if (a.grad_head) {
        const ProductArgs p{dz, a.hidden, a.grad_head, 1, v, 1, ldh, static_cast<size_t>(a.ld_grad_head), DT_F32, a.dtype,
                            a.dtype, a.vocab, a.cols, a.tokens, 1.0f, nullptr, a.targets};
        e = launch_product(p, s);
    }
    return e;
}

}  // namespace muon
