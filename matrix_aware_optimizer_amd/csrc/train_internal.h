// Internal types of the training operators (block_norm.hip, token_logp.hip,
// losses.hip) and their host side (train_api.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "muon.h"
#include "muon_internal.h"

namespace muon {

// One element, from fp32, of a buffer of float or bf16 (uint16_t) values.
template <typename T> __device__ __forceinline__ void st_el(void* p, size_t i, float v);
template <> __device__ __forceinline__ void st_el<float>(void* p, size_t i, float v) { G(static_cast<float*>(p))[i] = v; }
template <> __device__ __forceinline__ void st_el<uint16_t>(void* p, size_t i, float v) {
    G(static_cast<uint16_t*>(p))[i] = f32_to_bf16(v);
}
// The same with the dtype as a (uniform) value.
__device__ __forceinline__ void st_dt(void* p, size_t i, float v, int dt) {
    if (dt == DT_BF16) st_el<uint16_t>(p, i, v);
    else st_el<float>(p, i, v);
}

// 8 consecutive elements at any element alignment: the hardware takes such accesses whole, so odd widths and
// pitches cost only the cache lines that a run crosses.
typedef u32x4_t u32x4_el2 __attribute__((aligned(2)));
typedef f32x4_t f32x4_el4 __attribute__((aligned(4)));
template <typename T> using global_t = MUON_GLOBAL T;
// A run as loaded: converted only where it is used, so that a row's loads are all in flight at once.
template <typename T> struct Run;
template <> struct Run<uint16_t> {
    u32x4_t w = {};
    __device__ __forceinline__ void load(const global_t<uint16_t>* p, unsigned i) { w = *(const global_t<u32x4_el2>*)(p + i); }
    __device__ __forceinline__ void load(const global_t<uint16_t>* p, unsigned i, unsigned n) {
#pragma unroll
        for (int e = 0; e < 7; ++e)
            if (e < static_cast<int>(n)) w[e >> 1] |= static_cast<uint32_t>(p[i + e]) << (16 * (e & 1));
    }
    __device__ __forceinline__ float get(int e) const {
        return __uint_as_float((e & 1) ? (w[e >> 1] & 0xffff0000u) : (w[e >> 1] << 16));
    }
};
template <> struct Run<float> {
    f32x4_t w[2] = {};
    __device__ __forceinline__ void load(const global_t<float>* p, unsigned i) {
        w[0] = *(const global_t<f32x4_el4>*)(p + i);
        w[1] = *(const global_t<f32x4_el4>*)(p + i + 4);
    }
    __device__ __forceinline__ void load(const global_t<float>* p, unsigned i, unsigned n) {
#pragma unroll
        for (int e = 0; e < 7; ++e)
            if (e < static_cast<int>(n)) w[e >> 2][e & 3] = p[i + e];
    }
    __device__ __forceinline__ float get(int e) const { return w[e >> 2][e & 3]; }
};
__device__ __forceinline__ void st_run(global_t<uint16_t>* p, unsigned i, const float (&o)[8]) {
    u32x4_t w;
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = pack_bf16x2(o[2 * e], o[2 * e + 1]);
    *(global_t<u32x4_el2>*)(p + i) = w;
}
__device__ __forceinline__ void st_run(global_t<float>* p, unsigned i, const float (&o)[8]) {
    *(global_t<f32x4_el4>*)(p + i) = f32x4_t{o[0], o[1], o[2], o[3]};
    *(global_t<f32x4_el4>*)(p + i + 4) = f32x4_t{o[4], o[5], o[6], o[7]};
}

// Sum over a wave, the same in every lane, through the lanes' data paths (a few cycles a step, where a shuffle goes through
// LDS): within rows of 16 lanes, then row 0 to 1 and 2 to 3, then row 1 to 2 and 3; lane 63 ends with all.
template <int CTRL, int ROWS> __device__ __forceinline__ float dpp_add(float v) {
    return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, ROWS, 0xF, false));
}
__device__ __forceinline__ float wave_sum(float v) {
    v = dpp_add<0x111, 0xF>(v);   // row_shr:1
    v = dpp_add<0x112, 0xF>(v);
    v = dpp_add<0x114, 0xF>(v);
    v = dpp_add<0x118, 0xF>(v);
    v = dpp_add<0x142, 0xA>(v);   // row_bcast:15 into rows 1 and 3
    v = dpp_add<0x143, 0xC>(v);   // row_bcast:31 into rows 2 and 3
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}

template <int CTRL, int ROWS> __device__ __forceinline__ double dpp_add(double v) {
    const unsigned long long b = __double_as_longlong(v);
    const int lo = __builtin_amdgcn_update_dpp(0, static_cast<int>(b), CTRL, ROWS, 0xF, false);
    const int hi = __builtin_amdgcn_update_dpp(0, static_cast<int>(b >> 32), CTRL, ROWS, 0xF, false);
    return v + __hiloint2double(hi, lo);
}
__device__ __forceinline__ double wave_sum(double v) {
    v = dpp_add<0x111, 0xF>(v);
    v = dpp_add<0x112, 0xF>(v);
    v = dpp_add<0x114, 0xF>(v);
    v = dpp_add<0x118, 0xF>(v);
    v = dpp_add<0x142, 0xA>(v);
    v = dpp_add<0x143, 0xC>(v);
    const unsigned long long b = __double_as_longlong(v);
    return __hiloint2double(__builtin_amdgcn_readlane(static_cast<int>(b >> 32), 63), __builtin_amdgcn_readlane(static_cast<int>(b), 63));
}

// Sums over a workgroup, given to every thread; `red` holds a value of each sum per wave.  The order of the
// additions is fixed.  Safe to call again at once with the same `red`.
template <int N, typename V> __device__ __forceinline__ void block_sums(V (&v)[N], V* red) {
    const int waves = blockDim.x >> 6;
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = wave_sum(v[k]);
    if (waves == 1) return;
    lds_barrier();
    if ((threadIdx.x & 63) == 0)
#pragma unroll
        for (int k = 0; k < N; ++k) red[k * waves + (threadIdx.x >> 6)] = v[k];
    lds_barrier();
#pragma unroll
    for (int k = 0; k < N; ++k) {
        v[k] = red[k * waves];
        for (int w = 1; w < waves; ++w) v[k] += red[k * waves + w];
    }
}
__device__ __forceinline__ float block_sum(float v, float* red) {
    float s[1] = {v};
    block_sums(s, red);
    return s[0];
}

hipError_t launch_block_norm(const muon_block_norm_args& a, hipStream_t s);
size_t block_norm_backward_bytes(const muon_block_norm_backward_args& a);
hipError_t launch_block_norm_backward(const muon_block_norm_backward_args& a, void* workspace, hipStream_t s);

size_t token_logp_saved_bytes(const muon_token_logp_args& a);
size_t token_logp_bytes(const muon_token_logp_args& a);
hipError_t launch_token_logp(const muon_token_logp_args& a, void* workspace, hipStream_t s);
size_t token_logp_backward_bytes(const muon_token_logp_backward_args& a);
hipError_t launch_token_logp_backward(const muon_token_logp_backward_args& a, void* workspace, hipStream_t s);

size_t preference_bytes(const muon_preference_args& a);
hipError_t launch_preference(const muon_preference_args& a, void* workspace, hipStream_t s);
size_t policy_bytes(const muon_policy_args& a);
hipError_t launch_policy(const muon_policy_args& a, void* workspace, hipStream_t s);

}  // namespace muon
