// Layer norm over the channels of each row, and its VJP.
//
//   mean = sum(x) / C, rstd = 1 / sqrt(sum((x - mean)^2) / C + eps), out = (x - mean) rstd w + b
//   xh = (x - mean) rstd, gw = g w
//   grad_x = rstd (gw - sum(gw) / C - xh sum(gw xh) / C), grad_w = sum_rows g xh, grad_b = sum_rows g
//
// Bound by memory: each element is read once and written once. A row is held in the
// registers of one team of lanes (a power of two up to a warp for up to 32 element
// groups, then a warp with several groups per lane, a whole block for wide rows), so the second pass over it costs no further read. That pass takes the
// deviations d from the rounded mean and both sum(d) and sum(d^2): the first corrects
// the mean for its own rounding, the variance is sum(d^2) / C minus that correction
// squared, so a large common offset of a row costs the forward no accuracy. The backward is
// the formula at the mean that it is given, which float32 has rounded: xh is off by up to
// 2^-24 |mean| rstd. Channel c always belongs to the
// same lane, so the weight gradients are summed in registers over all rows a block
// visits; each block leaves one partial row in the workspace, and a second launch
// adds the partial rows in block order.
#include "etp_dense.cuh"

namespace etp {
namespace dense {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// Sum over a team of lanes (power of two <= 32), or over the block.
template <bool BLOCK>
__device__ __forceinline__ float team_sum(float v, int team, float* red) {
    if (BLOCK) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        __syncthreads();  // the previous sum has been read
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
        __syncthreads();
        float t = red[0];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) t += red[w];
        return t;
    }
    for (int o = team >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// One row's share of a lane: NV groups of V channels, zeros past C. Addresses are clamped
// into the row and the loads unconditional: a branch around each would wait for each.
template <typename T, int V, int NV>
__device__ __forceinline__ void load_row(const T* p, int C, int lane, int step, float (&v)[NV][V]) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (lane + i * step) * V;
        Pack<T, V>::load(p + (c < C ? c : 0), v[i]);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if ((lane + i * step) * V >= C)
#pragma unroll
            for (int j = 0; j < V; ++j) v[i][j] = 0.f;
}
template <typename T, int V, int NV>
__device__ __forceinline__ void load_param(const T* p, float none, int C, int lane, int step, float (&v)[NV][V]) {
    if (p) {
        load_row<T, V, NV>(p, C, lane, step, v);
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) v[i][j] = none;
    }
}

// Rows that a team has in flight at once.
template <int V, int NV>
constexpr int kRowsAtOnce = V * NV <= 4 ? 4 : V * NV <= 8 ? 2 : 1;

template <typename T, int V, int NV, bool BLOCK>
__global__ void __launch_bounds__(kThreads)
    etp_norm_fwd_kernel(RowMap map, int C, int team, float eps, Rows x, const T* __restrict__ weight,
                        const T* __restrict__ bias, Rows out, float* __restrict__ mean, float* __restrict__ rstd) {
    __shared__ float red[kWarps];
    constexpr int U = kRowsAtOnce<V, NV>;
    const int step = BLOCK ? kThreads : team;
    const int lane = threadIdx.x & (step - 1);
    const int rows_per_block = kThreads / step;
    const int sub = threadIdx.x / step;
    float wv[NV][V], bv[NV][V];
    load_param<T, V, NV>(weight, 1.f, C, lane, step, wv);
    load_param<T, V, NV>(bias, 0.f, C, lane, step, bv);
    const long long stride = (long long)gridDim.x * rows_per_block;
    // every lane of a warp runs the same number of steps: the sums are warp-collective
    for (long long r0 = (long long)blockIdx.x * rows_per_block; r0 < map.M; r0 += U * stride) {
        float v[U][NV][V];
        int row[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const long long r = r0 + u * stride + sub;
            row[u] = r < map.M ? (int)r : -1;
            load_row<T, V, NV>(static_cast<const T*>(x.p) + x.offset(map, row[u] < 0 ? 0 : row[u]), C, lane, step, v[u]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int j = 0; j < V; ++j) s += v[u][i][j];
            const float mu = __fdiv_rn(team_sum<BLOCK>(s, team, red), (float)C);
            // deviations from the rounded mean; what rounding took from it is their own mean
            float q = 0.f, e = 0.f;
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if ((lane + i * step) * V < C)
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        v[u][i][j] -= mu;
                        e += v[u][i][j];
                        q = fmaf(v[u][i][j], v[u][i][j], q);
                    }
            const float rest = __fdiv_rn(team_sum<BLOCK>(e, team, red), (float)C);
            const float var = __fdiv_rn(team_sum<BLOCK>(q, team, red), (float)C) - rest * rest;
            // (rounding may leave it below zero; a NaN stays one)
            const float rs = 1.f / sqrtf((var < 0.f ? 0.f : var) + eps);
            if (row[u] < 0) continue;
            T* os = static_cast<T*>(out.p) + out.offset(map, row[u]);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (lane + i * step) * V;
                if (c < C) {
#pragma unroll
                    for (int j = 0; j < V; ++j) v[u][i][j] = fmaf((v[u][i][j] - rest) * rs, wv[i][j], bv[i][j]);
                    Pack<T, V>::store(os + c, v[u][i]);
                }
            }
            if (lane == 0) {
                if (mean) mean[row[u]] = mu + rest;
                if (rstd) rstd[row[u]] = rs;
            }
        }
    }
}

// part: [gridDim.x][2][C] partial sums (grad_w, grad_b) when PARAMS.
template <typename T, int V, int NV, bool BLOCK, bool PARAMS>
__global__ void __launch_bounds__(kThreads)
    etp_norm_bwd_kernel(RowMap map, int C, int team, Rows x, const T* __restrict__ weight,
                        const float* __restrict__ mean, const float* __restrict__ rstd, Rows g, Rows gx,
                        float* __restrict__ part) {
    __shared__ float red[kWarps];
    extern __shared__ float acc[];  // [2][C], warp teams with PARAMS
    constexpr int U = kRowsAtOnce<V, NV> > 2 ? 2 : kRowsAtOnce<V, NV>;
    if (PARAMS) launch_dependents();
    const int step = BLOCK ? kThreads : team;
    const int lane = threadIdx.x & (step - 1);
    const int rows_per_block = kThreads / step;
    const int sub = threadIdx.x / step;
    float wv[NV][V], gws[NV][V], gbs[NV][V];
    load_param<T, V, NV>(weight, 1.f, C, lane, step, wv);
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) gws[i][j] = 0.f, gbs[i][j] = 0.f;
    const float inv = 1.f / (float)C;
    const long long stride = (long long)gridDim.x * rows_per_block;
    for (long long r0 = (long long)blockIdx.x * rows_per_block; r0 < map.M; r0 += U * stride) {
        float xv[U][NV][V], gv[U][NV][V], mu[U], rs[U];
        int row[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const long long r = r0 + u * stride + sub;
            row[u] = r < map.M ? (int)r : -1;
            const int at = row[u] < 0 ? 0 : row[u];
            load_row<T, V, NV>(static_cast<const T*>(x.p) + x.offset(map, at), C, lane, step, xv[u]);
            load_row<T, V, NV>(static_cast<const T*>(g.p) + g.offset(map, at), C, lane, step, gv[u]);
            mu[u] = mean[at], rs[u] = rstd[at];
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float s1 = 0.f, s2 = 0.f;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const bool on = row[u] >= 0 && (lane + i * step) * V < C;
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float xh = (xv[u][i][j] - mu[u]) * rs[u];
                    xv[u][i][j] = xh;
                    if (PARAMS && on) {
                        gws[i][j] = fmaf(gv[u][i][j], xh, gws[i][j]);
                        gbs[i][j] += gv[u][i][j];
                    }
                    if (on) {
                        gv[u][i][j] *= wv[i][j];
                        s1 += gv[u][i][j];
                        s2 = fmaf(gv[u][i][j], xh, s2);
                    }
                }
            }
            if (!gx.p) continue;  // the same for every thread
            s1 = team_sum<BLOCK>(s1, team, red) * inv;
            s2 = team_sum<BLOCK>(s2, team, red) * inv;
            if (row[u] < 0) continue;
            T* os = static_cast<T*>(gx.p) + gx.offset(map, row[u]);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (lane + i * step) * V;
                if (c < C) {
#pragma unroll
                    for (int j = 0; j < V; ++j) gv[u][i][j] = rs[u] * (gv[u][i][j] - s1 - xv[u][i][j] * s2);
                    Pack<T, V>::store(os + c, gv[u][i]);
                }
            }
        }
    }
    if (!PARAMS) return;
    float* row = part + (size_t)blockIdx.x * 2 * C;
    if (BLOCK) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int c = (lane + i * step) * V + j;
                if (c < C) row[c] = gws[i][j], row[C + c] = gbs[i][j];
            }
        return;
    }
    // the teams of a warp, then the warps in order
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j)
            for (int o = step; o < 32; o <<= 1) {
                gws[i][j] += __shfl_xor_sync(0xffffffffu, gws[i][j], o);
                gbs[i][j] += __shfl_xor_sync(0xffffffffu, gbs[i][j], o);
            }
    for (int w = 0; w < kWarps; ++w) {
        if ((int)(threadIdx.x >> 5) == w && (int)(threadIdx.x & 31) < step)
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const int c = (lane + i * step) * V + j;
                    if (c < C) {
                        acc[c] = w ? acc[c] + gws[i][j] : gws[i][j];
                        acc[C + c] = w ? acc[C + c] + gbs[i][j] : gbs[i][j];
                    }
                }
        __syncthreads();
    }
    for (int c = threadIdx.x; c < 2 * C; c += kThreads) row[c] = acc[c];
}

// grad_w, grad_b (either may be null) from [n][2][C] partial rows in a fixed order: 8
// columns (a sector) by 64 row lanes per block, then the 64 sums in order. Started while
// the partial rows are still being written: waits for them itself.
constexpr int kJoinCols = 8, kJoinRows = 64;
template <typename T>
__global__ void __launch_bounds__(kJoinCols* kJoinRows)
    etp_norm_params_kernel(int n, int C, const float* __restrict__ part, T* __restrict__ gw, T* __restrict__ gb) {
    __shared__ float red[kJoinRows][kJoinCols + 1];
    const int col = blockIdx.x * kJoinCols + threadIdx.x % kJoinCols, sub = threadIdx.x / kJoinCols;
    wait_for_previous();
    float s = 0.f;
    if (col < 2 * C)
#pragma unroll 8
        for (int i = sub; i < n; i += kJoinRows) s += part[(size_t)i * 2 * C + col];
    red[sub][threadIdx.x % kJoinCols] = s;
    __syncthreads();
    if (sub != 0 || col >= 2 * C) return;
#pragma unroll 16
    for (int w = 1; w < kJoinRows; ++w) s += red[w][threadIdx.x];
    T* o = col < C ? gw : gb;
    if (o) o[col < C ? col : col - C] = from_float<T>(s);
}

int pow2_at_least(int n) {
    int p = 1;
    while (p < n) p <<= 1;
    return p;
}

// Channels above which a whole block takes a row. Single elements (V = 1) reach it sooner:
// a warp would hold so many that few rows fit an SM. bfloat16 backward, 2^24 elements, block /
// warp a row: 193 channels 129 / 61 us, 225 114 / 55, 257 101 / 142, 321 85 / 127, 511 57 / 103.
// The forward holds less and would rather have warps on the other side of the limit too
// (257 channels 129 / 67 us, 511 68 / 43); one limit serves both.
__host__ __device__ constexpr int block_above(int V) { return V == 1 ? 256 : 1024; }

// Teams and blocks of a launch: lanes per row, and as many blocks as keep the SMs full.
struct Shape {
    int team, rows_per_block, grid;
};
Shape norm_shape(int M, int C, int V, int per_sm) {
    const int vecs = (C + V - 1) / V;
    const bool block = C > block_above(V);
    if (block && V == 1) per_sm = 8;
    Shape s;
    s.team = block ? kThreads : (vecs < 32 ? pow2_at_least(vecs) : 32);
    s.rows_per_block = kThreads / s.team;
    const long long want = ((long long)M + s.rows_per_block - 1) / s.rows_per_block;
    const long long cap = (long long)sm_count() * per_sm;
    s.grid = (int)(want < cap ? want : cap);
    return s;
}

constexpr int kFwdPerSm = 8, kBwdPerSm = 4;

template <typename T, int V, int NV, bool BLOCK>
struct FwdLaunch {
    static cudaError_t run(const RowMap& map, int C, float eps, const Rows& x, const void* w, const void* b,
                           const Rows& out, float* mean, float* rstd, cudaStream_t s) {
        const Shape sh = norm_shape(map.M, C, V, kFwdPerSm);
        etp_norm_fwd_kernel<T, V, NV, BLOCK><<<sh.grid, kThreads, 0, s>>>(
            map, C, sh.team, eps, x, static_cast<const T*>(w), static_cast<const T*>(b), out, mean, rstd);
        return cudaGetLastError();
    }
};

template <typename T, int V, int NV, bool BLOCK>
struct BwdLaunch {
    static cudaError_t run(const RowMap& map, int C, const Rows& x, const void* w, const float* mean,
                           const float* rstd, const Rows& g, const Rows& gx, float* part, int* grid, cudaStream_t s) {
        const Shape sh = norm_shape(map.M, C, V, kBwdPerSm);
        *grid = sh.grid;
        const T* wt = static_cast<const T*>(w);
        if (part)
            etp_norm_bwd_kernel<T, V, NV, BLOCK, true>
                <<<sh.grid, kThreads, BLOCK ? 0 : 2 * C * sizeof(float), s>>>(map, C, sh.team, x, wt, mean, rstd, g,
                                                                             gx, part);
        else
            etp_norm_bwd_kernel<T, V, NV, BLOCK, false>
                <<<sh.grid, kThreads, 0, s>>>(map, C, sh.team, x, wt, mean, rstd, g, gx, nullptr);
        return cudaGetLastError();
    }
};

// The instance whose NV groups per lane cover C channels.
template <template <typename, int, int, bool> class L, typename T, int V, typename... A>
cudaError_t pick(int C, A&&... a) {
    const int vecs = (C + V - 1) / V;
    if (C <= block_above(V)) {
        const int nv = (vecs + 31) / 32;
        if (nv <= 1) return L<T, V, 1, false>::run(a...);
        if (nv <= 2) return L<T, V, 2, false>::run(a...);
        if (nv <= 4) return L<T, V, 4, false>::run(a...);
        if constexpr (V <= 4) {
            if (nv <= 8) return L<T, V, 8, false>::run(a...);
        }
        return cudaErrorInvalidValue;
    }
    const int nv = (vecs + kThreads - 1) / kThreads;
    if constexpr (V == 8) {
        if (nv <= 1) return L<T, V, 1, true>::run(a...);
    }
    if (nv <= 2) return L<T, V, 2, true>::run(a...);
    if (nv <= 4) return L<T, V, 4, true>::run(a...);
    if constexpr (V <= 4) {
        if (nv <= 8) return L<T, V, 8, true>::run(a...);
    }
    if constexpr (V == 1) {
        if (nv <= 16) return L<T, V, 16, true>::run(a...);
        if (nv <= 32) return L<T, V, 32, true>::run(a...);
    }
    return cudaErrorInvalidValue;
}

template <template <typename, int, int, bool> class L, typename... A>
cudaError_t pick_type(bool bf16, bool v16, int C, A&&... a) {
    if (bf16) return v16 ? pick<L, __nv_bfloat16, 8>(C, a...) : pick<L, __nv_bfloat16, 1>(C, a...);
    return v16 ? pick<L, float, 4>(C, a...) : pick<L, float, 1>(C, a...);
}

}  // namespace

cudaError_t norm_forward(bool bf16, bool v16, const RowMap& map, int C, float eps, const Rows& x, const void* weight,
                         const void* bias, const Rows& out, float* mean, float* rstd, cudaStream_t s) {
    if (map.M == 0) return cudaSuccess;
    return pick_type<FwdLaunch>(bf16, v16, C, map, C, eps, x, weight, bias, out, mean, rstd, s);
}

size_t norm_workspace_bytes(int M, int C) {
    // the larger grid of the vector and the scalar form
    const int g1 = norm_shape(M, C, 1, kBwdPerSm).grid, g8 = norm_shape(M, C, 8, kBwdPerSm).grid;
    const int g4 = norm_shape(M, C, 4, kBwdPerSm).grid;
    const int g = g1 > g8 ? (g1 > g4 ? g1 : g4) : (g8 > g4 ? g8 : g4);
    return (size_t)g * 2 * C * sizeof(float);
}

cudaError_t norm_backward(bool bf16, bool v16, const RowMap& map, int C, const Rows& x, const void* weight,
                          const float* mean, const float* rstd, const Rows& g, const Rows& gx, void* gweight,
                          void* gbias, void* ws, cudaStream_t s) {
    float* part = gweight || gbias ? static_cast<float*>(ws) : nullptr;
    int grid = 0;
    if (map.M > 0) {
        const cudaError_t e = pick_type<BwdLaunch>(bf16, v16, C, map, C, x, weight, mean, rstd, g, gx, part, &grid, s);
        if (e != cudaSuccess) return e;
    }
    if (!gweight && !gbias) return cudaSuccess;
    const int blocks = (2 * C + kJoinCols - 1) / kJoinCols, threads = kJoinCols * kJoinRows;
    if (bf16)
        return launch_after(etp_norm_params_kernel<__nv_bfloat16>, blocks, threads, 0, s, grid, C, part,
                            static_cast<__nv_bfloat16*>(gweight), static_cast<__nv_bfloat16*>(gbias));
    return launch_after(etp_norm_params_kernel<float>, blocks, threads, 0, s, grid, C, part,
                        static_cast<float*>(gweight), static_cast<float*>(gbias));
}

}  // namespace dense
}  // namespace etp
