// Tokens sorted by expert and back (formulas: muon.h).  All four calls move rows; wide ones come near a copy's rate, or past it.
//
// Sort: a counting sort of tokens x chosen choices, stable, without atomics on what it returns.  The choices are cut
// into chunks; one launch counts each chunk's experts, the next ranks every choice within its chunk (a wave finds the lanes
// with the same expert bit by bit, by ballots) and copies the rows.  Several workgroups share a chunk: each ranks all of it and
// copies its part, which costs less than a launch in between.  A call of one chunk needs no count.
// The rows' runs of 8 values go at any alignment (Run, st_run).
//
// Measured (8192 x 2048 bf16 to 6 of 64 experts; a copy moves 5.05 TB/s): sort 4.6 + 46 us (5.1 TB/s), its gradient and the weighted
// sum 60 - 66 us each (3.6 - 3.9 TB/s, what holds them there was not found; 35 us, 6.7 TB/s, where the rows are in cache), the weighted sum's gradient 74 us (5.9 TB/s).
// Narrow rows are far from it: the sort and the weighted sum's gradient give a row to a whole wave, one after the other (65536 x 64 to 2 of 64: 69 and
// 70 us for 25 and 42 MB; the sums, which take as many lanes a row as it fills, 6).
#include <algorithm>

#include "train_internal.h"

namespace muon {

namespace {

constexpr int EX_THREADS = 256, EX_WAVES = 4;
constexpr int EX_CHUNK = 512, EX_PER = EX_CHUNK / EX_THREADS;   // choices a chunk, a lane
constexpr int EX_MOST_SHARES = EX_CHUNK / EX_WAVES, EX_WORKGROUPS = 1024;   // workgroups a chunk; as many in all, where they have rows
// (8192 x 2048 to 6 of 64: 45 us; with 256 and 4096 51 and 50; 2048 tokens 18, 21 and 22)
// Up to so many chunks and experts every workgroup adds up the chunks' counts by itself; for more a launch in between does it once.  64 wide,
// bf16, direct and scanned: 64 experts 8.5 and 10.0 us (4 chunks), 68 and 72 (256); 128 experts 9.1 and 10.4, 71 and 73, 408 and 308 (1536
// chunks); 256 experts 10.2 and 10.8 (4), 15.8 and 14.1 (16), 78 and 73 (256); 1024 experts 35 and 16.5 (16).
constexpr int EX_DIRECT_CHUNKS = 256, EX_DIRECT_EXPERTS = 128;

__device__ __forceinline__ int wave_id() { return __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6)); }

// The expert of choice i, num_experts for a dropped one and behind the end.
__device__ __forceinline__ int expert_of(const muon_expert_sort_args& a, int64_t i, int64_t n) {
    if (i >= n) return a.num_experts;
    const int64_t e = G(a.experts)[i];
    return e >= 0 && e < a.num_experts ? static_cast<int>(e) : a.num_experts;
}

template <typename T> __device__ __forceinline__ void zero_row(T* row, int64_t cols, int lane) {
    for (int64_t i = 8 * lane; i < cols; i += 512) {
        if (i + 8 <= cols) {
            const float z[8] = {};
            st_run(G(row) + i, 0, z);
        } else {
            for (int64_t e = i; e < cols; ++e) st_el<T>(row, e, 0.0f);
        }
    }
}

// Columns at .. at + 7 of a row of `cols`, as many as there are.
template <typename T> __device__ __forceinline__ void load_run(Run<T>& r, const global_t<T>* row, int64_t at, int64_t cols) {
    if (at + 8 <= cols) r.load(row + at, 0);
    else if (at < cols) r.load(row + at, 0, static_cast<unsigned>(cols - at));
}

struct SortArgs {
    muon_expert_sort_args a;
    int32_t* counts;      // [chunk][expert]; scanned: choices of the expert in the chunks before
    int32_t* totals;      // scanned: [expert]
    int chunks, scanned;
    int64_t block0;
};

__global__ __launch_bounds__(EX_THREADS) void expert_count_kernel(SortArgs s) {
    extern __shared__ int hist[];
    const muon_expert_sort_args& a = s.a;
    const int64_t n = a.tokens * a.chosen, chunk = s.block0 + blockIdx.x;
    for (int e = threadIdx.x; e <= a.num_experts; e += EX_THREADS) hist[e] = 0;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < EX_PER; ++k) atomicAdd(&hist[expert_of(a, chunk * EX_CHUNK + k * EX_THREADS + threadIdx.x, n)], 1);
    __syncthreads();
    for (int e = threadIdx.x; e < a.num_experts; e += EX_THREADS) G(s.counts)[chunk * a.num_experts + e] = hist[e];
}

// Counts to counts of the chunks before, for 64 experts a workgroup, 16 runs of chunks at once.
__global__ __launch_bounds__(1024) void expert_scan_kernel(SortArgs s) {
    __shared__ int run[16][64];
    const int lane = threadIdx.x & 63, wave = wave_id(), e = blockIdx.x * 64 + lane, per = (s.chunks + 15) / 16;
    const int c0 = min(wave * per, s.chunks), c1 = min(c0 + per, s.chunks);
    const bool ok = e < s.a.num_experts;
    int sum = 0;
    for (int c = c0; c < c1 && ok; ++c) sum += G(s.counts)[static_cast<int64_t>(c) * s.a.num_experts + e];
    run[wave][lane] = sum;
    __syncthreads();
    int before = 0, total = 0;
    for (int w = 0; w < 16; ++w) {
        before += w < wave ? run[w][lane] : 0;
        total += run[w][lane];
    }
    for (int c = c0; c < c1 && ok; ++c) {
        MUON_GLOBAL int32_t* p = G(s.counts) + static_cast<int64_t>(c) * s.a.num_experts + e;
        const int v = *p;
        *p = before;
        before += v;
    }
    if (wave == 0 && ok) G(s.totals)[e] = total;
}

template <typename T> __global__ __launch_bounds__(EX_THREADS) void expert_place_kernel(SortArgs s, int shares) {
    extern __shared__ int lds[];
    const muon_expert_sort_args& a = s.a;
    const int E = a.num_experts, lane = threadIdx.x & 63, wave = wave_id();
    const int64_t n = a.tokens * a.chosen, block = s.block0 + blockIdx.x, chunk = block / shares;
    const int share = static_cast<int>(block - chunk * shares), span = EX_CHUNK / shares;
    if (block != 0 && chunk * EX_CHUNK + share * span >= n) return;
    int* hist = lds;                         // [wave][E + 1], then the choices of the waves before
    int* first = hist + EX_WAVES * (E + 1);  // E + 1: where the expert's choices of this chunk begin
    int* totals = first + E + 1;             // E + 1
    int* place = totals + E + 1;             // EX_CHUNK
    int* red = place + EX_CHUNK;             // EX_WAVES
    for (int i = threadIdx.x; i < (EX_WAVES + 2) * (E + 1); i += EX_THREADS) hist[i] = 0;
    __syncthreads();

    // totals of all experts, and what the chunks before this one hold: chunks in turn to the waves
    if (s.chunks > 1 && !s.scanned)
        for (int e = lane; e < E; e += 64) {
            int before = 0, total = 0;
#pragma unroll 8
            for (int c = wave; c < s.chunks; c += EX_WAVES) {
                const int v = G(s.counts)[static_cast<int64_t>(c) * E + e];
                before += c < chunk ? v : 0;
                total += v;
            }
            atomicAdd(&first[e], before);
            atomicAdd(&totals[e], total);
        }

    // each wave ranks its own choices, in order
    int expert[EX_PER], rank[EX_PER];
    const int bits = 32 - __builtin_clz(E);          // dropped choices are expert E
    int* mine = hist + wave * (E + 1);
#pragma unroll
    for (int k = 0; k < EX_PER; ++k) {
        const int id = expert_of(a, chunk * EX_CHUNK + (wave * EX_PER + k) * 64 + lane, n);
        uint64_t same = ~0ull;
        for (int b = 0; b < bits; ++b) {
            const uint64_t set = __ballot((id >> b) & 1);
            same &= (id >> b) & 1 ? set : ~set;
        }
        const int before = __popcll(same & ((1ull << lane) - 1));
        expert[k] = id;
        rank[k] = mine[id] + before;
        __syncthreads();
        if (before == 0) mine[id] += __popcll(same);
        __syncthreads();
    }

    // the running sum of the totals
    const int per = (E + EX_THREADS - 1) / EX_THREADS, e0 = threadIdx.x * per;
    int sum = 0;
    for (int e = e0; e < min(e0 + per, E); ++e) {
        int own = 0;
#pragma unroll
        for (int w = 0; w < EX_WAVES; ++w) {
            const int v = hist[w * (E + 1) + e];
            hist[w * (E + 1) + e] = own;
            own += v;
        }
        const int before = s.scanned ? G(s.counts)[chunk * E + e] : first[e];
        const int total = s.chunks == 1 ? own : s.scanned ? G(s.totals)[e] : totals[e];
        first[e] = sum + before;
        sum += total;
    }
    // running sum over the threads
    int scan = sum;
    for (int d = 1; d < 64; d <<= 1) {
        const int v = __shfl_up(scan, d);
        scan += lane >= d ? v : 0;
    }
    if (lane == 63) red[wave] = scan;
    __syncthreads();
    int base = scan - sum, all = 0;
#pragma unroll
    for (int w = 0; w < EX_WAVES; ++w) {
        base += w < wave ? red[w] : 0;
        all += red[w];
    }
    for (int e = e0; e < min(e0 + per, E); ++e) {
        first[e] += base;
        if (block == 0) G(a.offsets)[e] = first[e];      // nothing comes before chunk 0
    }
    if (block == 0 && threadIdx.x == 0) G(a.offsets)[E] = all;
    __syncthreads();

#pragma unroll
    for (int k = 0; k < EX_PER; ++k) {
        const int64_t i = chunk * EX_CHUNK + (wave * EX_PER + k) * 64 + lane;
        const int slot = expert[k] < E ? first[expert[k]] + hist[wave * (E + 1) + expert[k]] + rank[k] : -1;
        place[(wave * EX_PER + k) * 64 + lane] = slot;
        if (share == 0 && i < n) G(a.slots)[i] = slot;
    }
    __syncthreads();

    // this workgroup's share of the rows; of row i itself, if it lies behind the last one taken
    for (int k = wave; k < span; k += EX_WAVES) {
        const int64_t i = chunk * EX_CHUNK + share * span + k;
        if (i >= n) break;
        if (i >= all) zero_row<T>(static_cast<T*>(a.sorted) + i * a.ld_sorted, a.cols, lane);
        const int slot = __builtin_amdgcn_readfirstlane(place[share * span + k]);
        if (slot < 0) continue;
        const global_t<T>* src = G(static_cast<const T*>(a.x) + i / a.chosen * a.ld_x);
        global_t<T>* dst = G(static_cast<T*>(a.sorted) + slot * a.ld_sorted);
        for (int64_t c = 8 * lane; c < a.cols; c += 4 * 512) {
            Run<T> r[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) load_run(r[q], src, c + 512 * q, a.cols);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int64_t at = c + 512 * q;
                if (at + 8 <= a.cols) {
                    r[q].store(dst + at);
                } else {
#pragma unroll
                    for (int e = 0; e < 7; ++e)
                        if (at + e < a.cols) st_el<T>(static_cast<T*>(a.sorted) + slot * a.ld_sorted, at + e, r[q].get(e));
                }
            }
        }
    }
}

// ---- sums over a token's rows ----------------------------------------------------

struct GatherArgs {
    const void* rows;       // tokens * chosen x cols
    const int32_t* slots;
    const float* weights;   // or NULL: 1
    void* out;
    int64_t tokens, cols, ld_rows, ld_out;
    int chosen, lanes;      // threads a token: a power of two that covers cols / 8 where it can
    int64_t token0;
};

// out[t] = sum over c of weights[t][c] rows[slots[t][c]], in fp32 in the order of c, rounded once.  EX_AHEAD rows' runs are
// loaded before the first is added (2: 2 % faster at 6 rows a token in cache; 8: 5 to 20 % slower).
constexpr int EX_AHEAD = 4;
template <typename T> __global__ __launch_bounds__(EX_THREADS) void expert_gather_kernel(GatherArgs g) {
    const int per = EX_THREADS / g.lanes;
    const int64_t t = g.token0 + static_cast<int64_t>(blockIdx.x) * per + threadIdx.x / g.lanes;
    if (t >= g.tokens) return;
    const int64_t n = g.tokens * g.chosen;
    const global_t<T>* rows = G(static_cast<const T*>(g.rows));
    global_t<T>* out = G(static_cast<T*>(g.out)) + t * g.ld_out;
    for (int64_t c = 8 * static_cast<int64_t>(threadIdx.x % g.lanes); c < g.cols; c += 8 * g.lanes) {
        const unsigned left = static_cast<unsigned>(g.cols - c < 8 ? g.cols - c : 8);
        float sum[8] = {};
        for (int k0 = 0; k0 < g.chosen; k0 += EX_AHEAD) {
            Run<T> r[EX_AHEAD];
            float w[EX_AHEAD];
#pragma unroll
            for (int k = 0; k < EX_AHEAD; ++k) {
                const int64_t at = t * g.chosen + k0 + k;
                const int slot = k0 + k < g.chosen ? G(g.slots)[at] : -1;
                w[k] = 0.0f;
                if (slot >= 0 && slot < n) {
                    w[k] = g.weights ? G(g.weights)[at] : 1.0f;
                    const global_t<T>* p = rows + slot * g.ld_rows + c;
                    if (left == 8) r[k].load(p, 0);
                    else r[k].load(p, 0, left);
                }
            }
#pragma unroll
            for (int k = 0; k < EX_AHEAD; ++k)
#pragma unroll
                for (int e = 0; e < 8; ++e) sum[e] = fmaf(w[k], r[k].get(e), sum[e]);
        }
        if (left == 8) st_run(out + c, 0, sum);
        else
#pragma unroll
            for (int e = 0; e < 7; ++e)
                if (e < static_cast<int>(left)) st_el<T>(static_cast<T*>(g.out), t * g.ld_out + c + e, sum[e]);
    }
}

// ---- gradients of the weighted sum -------------------------------------------------

// A wave a choice: grad_y's row and the choice's dot product from one pass over the two rows.  The wave of choice i also
// clears row i if no choice has it.
template <typename T> __global__ __launch_bounds__(EX_THREADS) void expert_scatter_kernel(muon_expert_combine_backward_args a, int64_t block0) {
    const int lane = threadIdx.x & 63;
    const int64_t n = a.tokens * a.chosen, i = (block0 + blockIdx.x) * EX_WAVES + wave_id();
    if (i >= n) return;
    if (i >= G(a.offsets)[a.num_experts]) zero_row<T>(static_cast<T*>(a.grad_y) + i * a.ld_grad_y, a.cols, lane);
    const int slot = __builtin_amdgcn_readfirstlane(G(a.slots)[i]);
    float dot = 0.0f;
    if (slot >= 0 && slot < n) {
        const float w = G(a.weights)[i];
        const global_t<T>* g = G(static_cast<const T*>(a.grad_out) + i / a.chosen * a.ld_grad_out);
        const global_t<T>* y = G(static_cast<const T*>(a.y) + slot * a.ld_y);
        T* out = static_cast<T*>(a.grad_y) + slot * a.ld_grad_y;
        for (int64_t c = 8 * lane; c < a.cols; c += 4 * 512) {
            Run<T> gr[4], yr[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                load_run(gr[q], g, c + 512 * q, a.cols);
                load_run(yr[q], y, c + 512 * q, a.cols);
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int64_t at = c + 512 * q;
                float o[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float v = gr[q].get(e);
                    dot = fmaf(v, yr[q].get(e), dot);
                    o[e] = w * v;
                }
                if (at + 8 <= a.cols) st_run(G(out) + at, 0, o);
                else
#pragma unroll
                    for (int e = 0; e < 7; ++e)
                        if (at + e < a.cols) st_el<T>(out, at + e, o[e]);
            }
        }
    }
    dot = wave_sum(dot);
    if (lane == 0) G(a.grad_weights)[i] = dot;
}

// ---- host --------------------------------------------------------------------------

int64_t sort_chunks(int64_t n) { return std::max<int64_t>(1, (n + EX_CHUNK - 1) / EX_CHUNK); }

// A launch holds at most 2^32 - 1 threads.
template <typename F> hipError_t in_launches(int64_t blocks, F launch) {
    constexpr int64_t MOST = int64_t{1} << 22;
    for (int64_t b = 0; b < blocks; b += MOST) {
        launch(b, static_cast<unsigned>(std::min(MOST, blocks - b)));
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

template <typename T> hipError_t run_gather(GatherArgs g, hipStream_t s) {
    g.lanes = 8;
    while (g.lanes < EX_THREADS && g.lanes * 8 < g.cols) g.lanes *= 2;
    const int per = EX_THREADS / g.lanes;
    return in_launches((g.tokens + per - 1) / per, [&](int64_t b, unsigned n) {
        g.token0 = b * per;
        hipLaunchKernelGGL((expert_gather_kernel<T>), dim3(n), dim3(EX_THREADS), 0, s, g);
    });
}

}  // namespace

size_t expert_sort_bytes(const muon_expert_sort_args& a) {
    const int64_t chunks = sort_chunks(a.tokens * a.chosen);
    return chunks == 1 ? 0 : static_cast<size_t>(chunks + 1) * a.num_experts * sizeof(int32_t);
}

hipError_t launch_expert_sort(const muon_expert_sort_args& a, void* workspace, hipStream_t s) {
    const int64_t n = a.tokens * a.chosen;
    SortArgs g{};
    g.a = a;
    g.chunks = static_cast<int>(sort_chunks(n));
    g.scanned = g.chunks > 1 && (g.chunks > EX_DIRECT_CHUNKS || a.num_experts > EX_DIRECT_EXPERTS);
    g.counts = static_cast<int32_t*>(workspace);
    g.totals = g.counts + static_cast<size_t>(g.chunks) * a.num_experts;
    hipError_t e;
    if (g.chunks > 1) {
        e = in_launches(g.chunks, [&](int64_t b, unsigned blocks) {
            g.block0 = b;
            hipLaunchKernelGGL(expert_count_kernel, dim3(blocks), dim3(EX_THREADS), (a.num_experts + 1) * sizeof(int), s, g);
        });
        if (e != hipSuccess) return e;
        if (g.scanned) {
            hipLaunchKernelGGL(expert_scan_kernel, dim3((a.num_experts + 63) / 64), dim3(1024), 0, s, g);
            e = hipGetLastError();
            if (e != hipSuccess) return e;
        }
    }
    int shares = 4;
    while (shares < EX_MOST_SHARES && shares * g.chunks < EX_WORKGROUPS) shares *= 2;
    const size_t lds = ((EX_WAVES + 2) * (a.num_experts + 1) + EX_CHUNK + EX_WAVES) * sizeof(int);
    return in_launches(static_cast<int64_t>(g.chunks) * shares, [&](int64_t b, unsigned blocks) {
        g.block0 = b;
        if (a.dtype == MUON_BF16) hipLaunchKernelGGL((expert_place_kernel<uint16_t>), dim3(blocks), dim3(EX_THREADS), lds, s, g, shares);
        else hipLaunchKernelGGL((expert_place_kernel<float>), dim3(blocks), dim3(EX_THREADS), lds, s, g, shares);
    });
}

hipError_t launch_expert_sort_backward(const muon_expert_sort_backward_args& a, hipStream_t s) {
    const GatherArgs g{a.grad_sorted, a.slots, nullptr, a.grad_x, a.tokens, a.cols, a.ld_grad_sorted, a.ld_grad_x, a.chosen, 0, 0};
    return a.dtype == MUON_BF16 ? run_gather<uint16_t>(g, s) : run_gather<float>(g, s);
}

hipError_t launch_expert_combine(const muon_expert_combine_args& a, hipStream_t s) {
    const GatherArgs g{a.y, a.slots, a.weights, a.out, a.tokens, a.cols, a.ld_y, a.ld_out, a.chosen, 0, 0};
    return a.dtype == MUON_BF16 ? run_gather<uint16_t>(g, s) : run_gather<float>(g, s);
}

hipError_t launch_expert_combine_backward(const muon_expert_combine_backward_args& a, hipStream_t s) {
    return in_launches((a.tokens * a.chosen + EX_WAVES - 1) / EX_WAVES, [&](int64_t b, unsigned n) {
        if (a.dtype == MUON_BF16) hipLaunchKernelGGL((expert_scatter_kernel<uint16_t>), dim3(n), dim3(EX_THREADS), 0, s, a, b);
        else hipLaunchKernelGGL((expert_scatter_kernel<float>), dim3(n), dim3(EX_THREADS), 0, s, a, b);
    });
}

}  // namespace muon
