// What the dense row operators (linear layers, layer norm) share: the addressing of
// rows, element types, 16-byte element groups.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "etp_dense.h"

namespace etp {
namespace dense {

// Quotient by a divisor d fixed at launch, for 0 <= n < 2^31 (round-up reciprocal of
// Granlund and Montgomery: p = 31 + ceil(log2 d), q = n ceil(2^p / d) >> p).
struct FastDiv {
    unsigned mul = 0, shift = 0;
    int d = 1;
    FastDiv() = default;
    explicit FastDiv(int div) : d(div) {
        if (div <= 1) return;
        unsigned lg = 0;
        while ((1ull << lg) < (unsigned long long)div) ++lg;
        const unsigned p = 31 + lg;
        mul = (unsigned)(((1ull << p) + div - 1) / div);
        shift = p - 32;
    }
    __device__ __forceinline__ unsigned quot(unsigned n) const {
        return d == 1 ? n : (__umulhi(n, mul) >> shift);
    }
};

// M rows in groups: row r of an operand starts at p + offset(map, r) elements. Strides
// are below 2^31 elements, so that an offset is two 32 x 32 -> 64 bit products.
struct RowMap {
    int M = 0;
    FastDiv per;
};
struct Rows {
    void* p = nullptr;
    unsigned gs = 0, rs = 0;
    __device__ __forceinline__ unsigned long long offset(const RowMap& m, int r) const {
        const unsigned g = m.per.quot((unsigned)r);
        return (unsigned long long)g * gs + (unsigned long long)((unsigned)r - g * (unsigned)m.per.d) * rs;
    }
};

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_float(float v);
template <>
__device__ __forceinline__ float from_float<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

__device__ __forceinline__ float bf16_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// V consecutive elements as floats: V = 1, or the 16 bytes of V = 4 floats or 8 bf16.
template <typename T, int V>
struct Pack;
template <typename T>
struct Pack<T, 1> {
    static __device__ __forceinline__ void load(const T* p, float (&v)[1]) { v[0] = to_float(*p); }
    static __device__ __forceinline__ void store(T* p, const float (&v)[1]) { *p = from_float<T>(v[0]); }
};
template <>
struct Pack<float, 4> {
    static __device__ __forceinline__ void load(const float* p, float (&v)[4]) {
        const float4 q = *reinterpret_cast<const float4*>(p);
        v[0] = q.x, v[1] = q.y, v[2] = q.z, v[3] = q.w;
    }
    static __device__ __forceinline__ void store(float* p, const float (&v)[4]) {
        *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    }
};
template <>
struct Pack<__nv_bfloat16, 8> {
    static __device__ __forceinline__ void load(const __nv_bfloat16* p, float (&v)[8]) {
        const uint4 q = *reinterpret_cast<const uint4*>(p);
        v[0] = bf16_lo(q.x), v[1] = bf16_hi(q.x), v[2] = bf16_lo(q.y), v[3] = bf16_hi(q.y);
        v[4] = bf16_lo(q.z), v[5] = bf16_hi(q.z), v[6] = bf16_lo(q.w), v[7] = bf16_hi(q.w);
    }
    static __device__ __forceinline__ void store(__nv_bfloat16* p, const float (&v)[8]) {
        *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                                                  pack_bf16(v[6], v[7]));
    }
};

// SiLU and its derivative in float32: s = 1 / (1 + exp(-z)), silu = z s,
// silu' = s (1 + z (1 - s)), with exp(-z) = 2^(-z log2(e)) and the approximate 2^x and 1/x of
// the special function unit (2 ulp and 1 ulp of their own results). The product z log2(e) is
// rounded before 2^x, so exp is off by up to 1.25 |z| 2^-24 of itself more (the rounding, and
// that of log2(e)): s keeps (1.25 |z| + 8) 2^-24 of its own size, which for z > 0 is mostly the
// 1 beside exp, and for z = -20, where silu is -4e-8, 33 units of 2^-24. Carrying the low part
// of the product along would cost four more instructions an element, for an absolute error
// that stays below 2^-24 (1 + |z|). Subnormal intermediates go to zero, which
// only exp(-z) for z > 87 and 1/x for z < -87 reach: s is then 1 or 0 within 2^-126.
__device__ __forceinline__ float sigmoid(float z) {
    float e, s;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(z * -1.4426950408889634f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(1.f + e));
    return s;
}
// (a product of its own: never contracted with a sum, so a layer's result does not depend on what else it stores)
__device__ __forceinline__ float silu(float z) { return __fmul_rn(z, sigmoid(z)); }
__device__ __forceinline__ float silu_grad(float z) {
    const float s = sigmoid(z);
    return s * fmaf(z, 1.f - s, 1.f);
}

// Programmatic dependent launch: a kernel launched by launch_after may start once every
// block of the kernel before it on the stream has called launch_dependents (or ended), and
// calls wait_for_previous before it reads that kernel's results or writes anything. Its
// launch overlaps with the other's run.
__device__ __forceinline__ void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
template <typename... P, typename... A>
cudaError_t launch_after(void (*kernel)(P...), int blocks, int threads, size_t smem, cudaStream_t s, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

int sm_count();  // multiprocessors of the current device

// Launches (arguments checked by the C ABI). V16: every row of every operand and every
// channel vector starts on a 16-byte boundary and C is a multiple of 16 bytes.
cudaError_t norm_forward(bool bf16, bool v16, const RowMap& map, int C, float eps, const Rows& x, const void* weight,
                         const void* bias, const Rows& out, float* mean, float* rstd, cudaStream_t s);
size_t norm_workspace_bytes(int M, int C);
cudaError_t norm_backward(bool bf16, bool v16, const RowMap& map, int C, const Rows& x, const void* weight,
                          const float* mean, const float* rstd, const Rows& g, const Rows& gx, void* gweight,
                          void* gbias, void* ws, cudaStream_t s);

struct LinearArgs {
    RowMap map;
    int K, N;
    Rows x, residual, z, out;  // forward; null p: absent
    Rows g, gx;                // backward
    const void *W, *bias;
    void *gW, *gbias;
    float* ws;
    bool silu;
};
cudaError_t linear_forward(bool bf16, const LinearArgs& a, cudaStream_t s);
// Workspace of a forward, or of a backward with these outputs.
size_t linear_workspace_bytes(bool bf16, int M, int K, int N, bool fwd, bool gx, bool gw, bool gb);
cudaError_t linear_backward(bool bf16, const LinearArgs& a, cudaStream_t s);
int linear_read_and_clear_fault();

}  // namespace dense
}  // namespace etp
