// C ABI of the dense row operators (declared in include/etp_dense.h): host-side
// argument checks and launches on the caller's stream.
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>

#include "etp_dense.cuh"

namespace etp {
namespace dense {

int sm_count() {
    // a device's multiprocessors do not change; 0: not asked for yet
    static std::atomic<int> known[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        cudaGetLastError();
        return 148;
    }
    int n = dev < 64 ? known[dev].load(std::memory_order_relaxed) : 0;
    if (n > 0) return n;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) {
        cudaGetLastError();
        return 148;
    }
    if (dev < 64) known[dev].store(n, std::memory_order_relaxed);
    return n;
}

}  // namespace dense
}  // namespace etp

namespace {

using etp::dense::LinearArgs;
using etp::dense::RowMap;
using etp::dense::Rows;

etp_status cuda_status(cudaError_t e) { return e == cudaSuccess ? ETP_OK : ETP_ERR_CUDA; }
bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

etp_status check_workspace(const void* p, size_t have, size_t need) {
    if (need == 0) return ETP_OK;
    if (!p || !aligned(p, 16)) return ETP_ERR_INVALID_ARG;
    return have < need ? ETP_ERR_WORKSPACE : ETP_OK;
}

// The rows of a call in the fewest groups: one group of many rows counts as many groups of one row.
struct Call {
    RowMap map;
    bool merged = false;  // groups = 1: the row stride is the only one
    size_t elem = 4;
    etp_status status = ETP_OK;
    Call(etp_dtype dtype, int groups, int per_group) {
        if (groups < 0 || per_group < 0) {
            status = ETP_ERR_INVALID_ARG;
            return;
        }
        if (dtype != ETP_F32 && dtype != ETP_BF16) {
            status = ETP_ERR_UNSUPPORTED;
            return;
        }
        elem = dtype == ETP_F32 ? 4 : 2;
        const long long m = (long long)groups * per_group;
        if (m >= (1ll << 31) - 128) {
            status = ETP_ERR_TOO_LARGE;
            return;
        }
        map.M = (int)m;
        merged = groups == 1;
        map.per = etp::dense::FastDiv(merged || per_group < 1 ? 1 : per_group);
        groups_ = groups, per_ = per_group;
    }
    // The operand's strides in that form; false when it is not acceptable.
    bool rows(const etp_rows* r, int channels, bool output, Rows* o) const {
        if (!r || !r->data || !aligned(r->data, elem)) return false;
        const int64_t gs = groups_ > 1 ? r->group_stride : 0, rs = per_ > 1 ? r->row_stride : 0;
        if (gs < 0 || rs < 0) return false;
        if (gs > INT32_MAX || rs > INT32_MAX) return false;
        if (output) {
            const int64_t G = groups_, P = per_;
            const bool in_group = P == 1 || rs >= channels, across = G == 1 || gs >= channels;
            if (!in_group || !across) return false;
            if (G > 1 && P > 1 && gs < (P - 1) * rs + channels && rs < (G - 1) * gs + channels) return false;
        }
        o->p = r->data;
        o->gs = (unsigned)(merged ? rs : gs);
        o->rs = (unsigned)(merged ? 0 : rs);
        return true;
    }
    // Whether every row of the operand starts on a 16-byte boundary.
    bool v16(const Rows& r) const {
        const unsigned n = 16 / (unsigned)elem;
        return !r.p || (aligned(r.p, 16) && r.gs % n == 0 && r.rs % n == 0);
    }

private:
    int groups_ = 0, per_ = 0;
};

}  // namespace

extern "C" {

etp_status etp_linear_forward(etp_dtype dtype, int groups, int per_group, int K, int N, const etp_rows* x,
                              const void* W, const void* bias, etp_activation act, const etp_rows* residual,
                              const etp_rows* z, const etp_rows* out, void* workspace, size_t workspace_bytes,
                              etp_stream_t stream) {
    const Call c(dtype, groups, per_group);
    if (c.status != ETP_OK) return c.status;
    if (K < 1 || N < 1 || K > ETP_LINEAR_MAX_CHANNELS || N > ETP_LINEAR_MAX_CHANNELS) return ETP_ERR_INVALID_ARG;
    if (act != ETP_ACT_NONE && act != ETP_ACT_SILU) return ETP_ERR_UNSUPPORTED;
    if (c.map.M == 0) return ETP_OK;
    LinearArgs a{};
    a.map = c.map;
    a.K = K, a.N = N;
    if (!c.rows(x, K, false, &a.x) || !c.rows(out, N, true, &a.out)) return ETP_ERR_INVALID_ARG;
    if (residual && !c.rows(residual, N, false, &a.residual)) return ETP_ERR_INVALID_ARG;
    if (z && !c.rows(z, N, true, &a.z)) return ETP_ERR_INVALID_ARG;
    if (!W || !aligned(W, c.elem) || !aligned(bias, c.elem)) return ETP_ERR_INVALID_ARG;
    a.W = W, a.bias = bias;
    const etp_status ws =
        check_workspace(workspace, workspace_bytes,
                        etp::dense::linear_workspace_bytes(dtype == ETP_BF16, c.map.M, K, N, true, false, false, false));
    if (ws != ETP_OK) return ws;
    a.ws = static_cast<float*>(workspace);
    a.silu = act == ETP_ACT_SILU;
    return cuda_status(etp::dense::linear_forward(dtype == ETP_BF16, a, reinterpret_cast<cudaStream_t>(stream)));
}

etp_status etp_linear_workspace_size(etp_dtype dtype, int groups, int per_group, int K, int N, int backward,
                                     size_t* bytes) {
    const Call c(dtype, groups, per_group);
    if (c.status != ETP_OK) return c.status;
    if (!bytes || K < 1 || N < 1 || K > ETP_LINEAR_MAX_CHANNELS || N > ETP_LINEAR_MAX_CHANNELS ||
        (backward != 0 && backward != 1))
        return ETP_ERR_INVALID_ARG;
    const bool bf16 = dtype == ETP_BF16, b = backward != 0;
    *bytes = etp::dense::linear_workspace_bytes(bf16, c.map.M, K, N, !b, b, b, b);
    // grad_bias alone takes ranges of its own
    if (b) {
        const size_t bias = etp::dense::linear_workspace_bytes(bf16, c.map.M, K, N, false, true, false, true);
        if (bias > *bytes) *bytes = bias;
    }
    return ETP_OK;
}

etp_status etp_linear_backward(etp_dtype dtype, int groups, int per_group, int K, int N, const etp_rows* x,
                               const void* W, etp_activation act, const etp_rows* z, const etp_rows* grad_out,
                               const etp_rows* grad_x, void* grad_W, void* grad_bias, void* workspace,
                               size_t workspace_bytes, etp_stream_t stream) {
    const Call c(dtype, groups, per_group);
    if (c.status != ETP_OK) return c.status;
    if (K < 1 || N < 1 || K > ETP_LINEAR_MAX_CHANNELS || N > ETP_LINEAR_MAX_CHANNELS) return ETP_ERR_INVALID_ARG;
    if (act != ETP_ACT_NONE && act != ETP_ACT_SILU) return ETP_ERR_UNSUPPORTED;
    if (!aligned(grad_W, c.elem) || !aligned(grad_bias, c.elem)) return ETP_ERR_INVALID_ARG;
    if (!grad_x && !grad_W && !grad_bias) return ETP_OK;
    LinearArgs a{};
    a.map = c.map;
    a.K = K, a.N = N;
    if (c.map.M > 0) {
        if (!c.rows(grad_out, N, false, &a.g)) return ETP_ERR_INVALID_ARG;
        if (act == ETP_ACT_SILU && !c.rows(z, N, false, &a.z)) return ETP_ERR_INVALID_ARG;
        if (grad_x && (!c.rows(grad_x, K, true, &a.gx) || !W || !aligned(W, c.elem))) return ETP_ERR_INVALID_ARG;
        if (grad_W && !c.rows(x, K, false, &a.x)) return ETP_ERR_INVALID_ARG;
    }
    const etp_status ws = check_workspace(
        workspace, workspace_bytes,
        etp::dense::linear_workspace_bytes(dtype == ETP_BF16, c.map.M, K, N, false, grad_x != nullptr,
                                           grad_W != nullptr, grad_bias != nullptr));
    if (ws != ETP_OK) return ws;
    a.W = W;
    a.gW = grad_W, a.gbias = grad_bias;
    a.ws = static_cast<float*>(workspace);
    a.silu = act == ETP_ACT_SILU;
    return cuda_status(etp::dense::linear_backward(dtype == ETP_BF16, a, reinterpret_cast<cudaStream_t>(stream)));
}

etp_status etp_layer_norm_forward(etp_dtype dtype, int groups, int per_group, int C, float eps, const etp_rows* x,
                                  const void* weight, const void* bias, const etp_rows* out, float* mean, float* rstd,
                                  etp_stream_t stream) {
    const Call c(dtype, groups, per_group);
    if (c.status != ETP_OK) return c.status;
    if (C < 1 || !(eps >= 0.f) || !std::isfinite(eps)) return ETP_ERR_INVALID_ARG;
    if (C > ETP_NORM_MAX_CHANNELS) return ETP_ERR_UNSUPPORTED;
    if (c.map.M == 0) return ETP_OK;
    Rows xr, orow;
    if (!c.rows(x, C, false, &xr) || !c.rows(out, C, true, &orow)) return ETP_ERR_INVALID_ARG;
    if (!aligned(weight, c.elem) || !aligned(bias, c.elem) || !aligned(mean, 4) || !aligned(rstd, 4))
        return ETP_ERR_INVALID_ARG;
    const bool v16 = c.v16(xr) && c.v16(orow) && aligned(weight, 16) && aligned(bias, 16) && (C * c.elem) % 16 == 0;
    return cuda_status(etp::dense::norm_forward(dtype == ETP_BF16, v16, c.map, C, eps, xr, weight, bias, orow, mean,
                                                rstd, reinterpret_cast<cudaStream_t>(stream)));
}

etp_status etp_layer_norm_workspace_size(etp_dtype dtype, int groups, int per_group, int C, size_t* bytes) {
    const Call c(dtype, groups, per_group);
    if (c.status != ETP_OK) return c.status;
    if (!bytes || C < 1) return ETP_ERR_INVALID_ARG;
    if (C > ETP_NORM_MAX_CHANNELS) return ETP_ERR_UNSUPPORTED;
    *bytes = etp::dense::norm_workspace_bytes(c.map.M, C);
    return ETP_OK;
}

etp_status etp_layer_norm_backward(etp_dtype dtype, int groups, int per_group, int C, const etp_rows* x,
                                   const void* weight, const float* mean, const float* rstd, const etp_rows* grad_out,
                                   const etp_rows* grad_x, void* grad_weight, void* grad_bias, void* workspace,
                                   size_t workspace_bytes, etp_stream_t stream) {
    const Call c(dtype, groups, per_group);
    if (c.status != ETP_OK) return c.status;
    if (C < 1) return ETP_ERR_INVALID_ARG;
    if (C > ETP_NORM_MAX_CHANNELS) return ETP_ERR_UNSUPPORTED;
    if (!aligned(weight, c.elem) || !aligned(grad_weight, c.elem) || !aligned(grad_bias, c.elem))
        return ETP_ERR_INVALID_ARG;
    if (!grad_x && !grad_weight && !grad_bias) return ETP_OK;
    Rows xr, gr, gx;
    if (c.map.M > 0) {
        if (!c.rows(x, C, false, &xr) || !c.rows(grad_out, C, false, &gr)) return ETP_ERR_INVALID_ARG;
        if (grad_x && !c.rows(grad_x, C, true, &gx)) return ETP_ERR_INVALID_ARG;
        if (!mean || !rstd || !aligned(mean, 4) || !aligned(rstd, 4)) return ETP_ERR_INVALID_ARG;
    }
    if (grad_weight || grad_bias) {
        const etp_status ws = check_workspace(workspace, workspace_bytes, etp::dense::norm_workspace_bytes(c.map.M, C));
        if (ws != ETP_OK) return ws;
    }
    const bool v16 = c.v16(xr) && c.v16(gr) && c.v16(gx) && aligned(weight, 16) && (C * c.elem) % 16 == 0;
    return cuda_status(etp::dense::norm_backward(dtype == ETP_BF16, v16, c.map, C, xr, weight, mean, rstd, gr, gx,
                                                 grad_weight, grad_bias, workspace,
                                                 reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
