// Layer norm over the channels of each row, and its VJP.
//
//   mean = sum(x) / C, rstd = 1 / sqrt(sum((x - mean)^2) / C + eps), out = (x - mean) rstd w + b
//   xh = (x - mean) rstd, gw = g w
//   grad_x = rstd (gw - sum(gw) / C - xh sum(gw xh) / C), grad_w = sum_rows g xh, grad_b = sum_rows g
//
// Bound by memory: each element is read once and written once. A row is held in the
// registers of one team of lanes (a power of two up to a warp for up to 32 element
// groups, then a warp with several groups per lane, a whole block above 1024
// channels), so the second pass over it costs no further read. That pass takes the
// deviations d from the rounded mean and both sum(d) and sum(d^2): the first corrects
// the mean for its own rounding, the variance is sum(d^2) / C minus that correction
// squared, so a large common offset of a row costs no accuracy. Channel c always belongs to the
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

template <typename T, int V, int NV, bool BLOCK>
__global__ void __launch_bounds__(kThreads)
    etp_norm_fwd_kernel(RowMap map, int C, int team, float eps, Rows x, const T* __restrict__ weight,
                        const T* __restrict__ bias, Rows out, float* __restrict__ mean, float* __restrict__ rstd) {
    __shared__ float red[kWarps];
    const int step = BLOCK ? kThreads : team;
    const int lane = threadIdx.x & (step - 1);
    const int rows_per_block = kThreads / step;
    const int sub = threadIdx.x / step;
    float wv[NV][V], bv[NV][V];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (lane + i * step) * V;
#pragma unroll
        for (int j = 0; j < V; ++j) wv[i][j] = 1.f, bv[i][j] = 0.f;
        if (c < C) {
            if (weight) Pack<T, V>::load(weight + c, wv[i]);
            if (bias) Pack<T, V>::load(bias + c, bv[i]);
        }
    }
    // every lane of a warp runs the same number of steps: the sums are warp-collective
    for (long long r0 = (long long)blockIdx.x * rows_per_block; r0 < map.M; r0 += (long long)gridDim.x * rows_per_block) {
        const bool live = r0 + sub < map.M;
        const int r = live ? (int)(r0 + sub) : 0;
        const T* xs = static_cast<const T*>(x.p) + x.offset(map, r);
        float v[NV][V];
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (lane + i * step) * V;
#pragma unroll
            for (int j = 0; j < V; ++j) v[i][j] = 0.f;
            if (live && c < C) Pack<T, V>::load(xs + c, v[i]);
#pragma unroll
            for (int j = 0; j < V; ++j) s += v[i][j];
        }
        const float mu = __fdiv_rn(team_sum<BLOCK>(s, team, red), (float)C);
        // deviations from the rounded mean; what rounding took from it is their own mean
        float q = 0.f, e = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if ((lane + i * step) * V < C)
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    v[i][j] -= mu;
                    e += v[i][j];
                    q = fmaf(v[i][j], v[i][j], q);
                }
        const float rest = __fdiv_rn(team_sum<BLOCK>(e, team, red), (float)C);
        const float var = fmaxf(__fdiv_rn(team_sum<BLOCK>(q, team, red), (float)C) - rest * rest, 0.f);
        const float rs = 1.f / sqrtf(var + eps);
        if (!live) continue;
        T* os = static_cast<T*>(out.p) + out.offset(map, r);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (lane + i * step) * V;
            if (c < C) {
#pragma unroll
                for (int j = 0; j < V; ++j) v[i][j] = fmaf((v[i][j] - rest) * rs, wv[i][j], bv[i][j]);
                Pack<T, V>::store(os + c, v[i]);
            }
        }
        if (lane == 0) {
            if (mean) mean[r] = mu + rest;
            if (rstd) rstd[r] = rs;
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
    const int step = BLOCK ? kThreads : team;
    const int lane = threadIdx.x & (step - 1);
    const int rows_per_block = kThreads / step;
    const int sub = threadIdx.x / step;
    float wv[NV][V], gws[NV][V], gbs[NV][V];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (lane + i * step) * V;
#pragma unroll
        for (int j = 0; j < V; ++j) wv[i][j] = 1.f, gws[i][j] = 0.f, gbs[i][j] = 0.f;
        if (weight && c < C) Pack<T, V>::load(weight + c, wv[i]);
    }
    const float inv = 1.f / (float)C;
    for (long long r0 = (long long)blockIdx.x * rows_per_block; r0 < map.M; r0 += (long long)gridDim.x * rows_per_block) {
        const bool live = r0 + sub < map.M;
        const int r = live ? (int)(r0 + sub) : 0;
        const T* xs = static_cast<const T*>(x.p) + x.offset(map, r);
        const T* gs = static_cast<const T*>(g.p) + g.offset(map, r);
        const float mu = live ? mean[r] : 0.f, rs = live ? rstd[r] : 0.f;
        float xv[NV][V], gv[NV][V];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (lane + i * step) * V;
#pragma unroll
            for (int j = 0; j < V; ++j) xv[i][j] = mu, gv[i][j] = 0.f;
            if (live && c < C) {
                Pack<T, V>::load(xs + c, xv[i]);
                Pack<T, V>::load(gs + c, gv[i]);
            }
        }
        float s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float xh = (xv[i][j] - mu) * rs;
                xv[i][j] = xh;
                if (PARAMS) {
                    gws[i][j] = fmaf(gv[i][j], xh, gws[i][j]);
                    gbs[i][j] += gv[i][j];
                }
                gv[i][j] *= wv[i][j];
                s1 += gv[i][j];
                s2 = fmaf(gv[i][j], xh, s2);
            }
        if (!gx.p) continue;  // the same for every thread
        s1 = team_sum<BLOCK>(s1, team, red) * inv;
        s2 = team_sum<BLOCK>(s2, team, red) * inv;
        if (!live) continue;
        T* os = static_cast<T*>(gx.p) + gx.offset(map, r);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (lane + i * step) * V;
            if (c < C) {
#pragma unroll
                for (int j = 0; j < V; ++j) gv[i][j] = rs * (gv[i][j] - s1 - xv[i][j] * s2);
                Pack<T, V>::store(os + c, gv[i]);
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

// grad_w, grad_b (either may be null) from [n][2][C] partial rows, in row order: 32
// columns by 8 row lanes per block, then the 8 sums in order.
template <typename T>
__global__ void __launch_bounds__(kThreads)
    etp_norm_params_kernel(int n, int C, const float* __restrict__ part, T* __restrict__ gw, T* __restrict__ gb) {
    __shared__ float red[kWarps][33];
    const int col = blockIdx.x * 32 + (threadIdx.x & 31), sub = threadIdx.x >> 5;
    float s = 0.f;
    if (col < 2 * C)
#pragma unroll 8
        for (int i = sub; i < n; i += kWarps) s += part[(size_t)i * 2 * C + col];
    red[sub][threadIdx.x & 31] = s;
    __syncthreads();
    if (sub != 0 || col >= 2 * C) return;
#pragma unroll
    for (int w = 1; w < kWarps; ++w) s += red[w][threadIdx.x & 31];
    T* o = col < C ? gw : gb;
    if (o) o[col < C ? col : col - C] = from_float<T>(s);
}

int pow2_at_least(int n) {
    int p = 1;
    while (p < n) p <<= 1;
    return p;
}

// Teams and blocks of a launch: lanes per row, and as many blocks as keep the SMs full.
struct Shape {
    int team, rows_per_block, grid;
};
Shape norm_shape(int M, int C, int V, int per_sm) {
    const int vecs = (C + V - 1) / V;
    const bool block = C > 1024;
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
    if (C <= 1024) {
        const int nv = (vecs + 31) / 32;
        if (nv <= 1) return L<T, V, 1, false>::run(a...);
        if (nv <= 2) return L<T, V, 2, false>::run(a...);
        if (nv <= 4) return L<T, V, 4, false>::run(a...);
        if constexpr (V <= 4) {
            if (nv <= 8) return L<T, V, 8, false>::run(a...);
        }
        if constexpr (V == 1) {
            if (nv <= 16) return L<T, V, 16, false>::run(a...);
            return L<T, V, 32, false>::run(a...);
        }
        return cudaErrorInvalidValue;
    }
    const int nv = (vecs + kThreads - 1) / kThreads;
    if constexpr (V == 8) {
        if (nv <= 1) return L<T, V, 1, true>::run(a...);
    }
    if constexpr (V >= 4) {
        if (nv <= 2) return L<T, V, 2, true>::run(a...);
    }
    if constexpr (V >= 4) {
        if (nv <= 4) return L<T, V, 4, true>::run(a...);
    }
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
    const int blocks = (2 * C + 31) / 32;
    if (bf16)
        etp_norm_params_kernel<__nv_bfloat16><<<blocks, kThreads, 0, s>>>(
            grid, C, part, static_cast<__nv_bfloat16*>(gweight), static_cast<__nv_bfloat16*>(gbias));
    else
        etp_norm_params_kernel<float><<<blocks, kThreads, 0, s>>>(grid, C, part, static_cast<float*>(gweight),
                                                                  static_cast<float*>(gbias));
    return cudaGetLastError();
}

}  // namespace dense
}  // namespace etp
