// Linear layers with a fused epilogue, and their VJP, on the tensor cores (tcgen05).
//
//   forward   z = x W + bias, out = act(z) + residual
//   backward  dz = g act'(z);  grad_x = dz W^T;  grad_W = x^T dz;  grad_bias = sum of dz over the rows
//
// Each of the three products is D[m][n] = sum_k A[m][k] B[k][n] in tiles of 128 x BN
// outputs, 64 k per stage. One persistent CTA per SM:
//   - loader warps read a stage of both operands from global memory into registers
//     (the next one is in flight while the current one is converted), form dz where it
//     is an operand, and store bfloat16 operands in the 128-byte-swizzled layouts of
//     the tensor core: an operand whose contraction index is contiguous in memory
//     K-major, one whose other index is contiguous MN-major, so nothing is transposed;
//   - one warp issues the MMAs into a ring of accumulators in tensor memory;
//   - epilogue warps add the accumulators up in registers and apply the epilogue.
// Float32 operands are split by truncation into three bfloat16 parts x = x0 + x1 + x2
// (8 bits each: exact), and a product is the sum of the six part products x0 w0, x0 w1,
// x1 w0, x1 w1, x0 w2, x2 w0: what is left out is below 2^-22 of it. That is as many
// MMAs as three TF32 products, at twice the mantissa of the smallest terms kept and in
// three quarters of the shared memory, and both layouts are available to 16-bit types.
// The tensor core truncates when it adds to its accumulator; so a float32 stage starts
// a new accumulator, adds the small products first and the x0 w0 ones last (four
// truncated additions of full size), and stages are added up in registers, rounded to
// nearest. bfloat16 operands are one part (dz is rounded to it: the tensor core reads
// nothing wider beside bf16 weights without a second product); their accumulator holds
// 16 stages, whose truncations stay far below the result's own rounding.
//
// grad_W contracts over the rows: the rows are cut into as many ranges as leave every
// SM one, each range's sums go to the workspace, and a second launch adds them up in
// range order. grad_bias is summed by the loaders of dz on the way.
#include "etp_dense.cuh"
#include "etp_tcgen05.cuh"

namespace etp {
namespace dense {
namespace {

enum class Product { kForward, kGradX, kGradW };

constexpr int kRowsTile = 128, kStageK = 64;
// Warps: 8 of the epilogue, the loaders, one for the MMAs. Four loader warps leave 128
// registers a thread (13 warps) for the epilogue's sums and the loads in flight; the
// backward products, whose loaders have dz to compute and whose epilogue is plain, have
// eight (17 warps, 96).
constexpr int kEpiWarps = 8;
template <Product P>
struct Warps {
    static constexpr int kLoad = P == Product::kForward ? 4 : 8;
    static constexpr int kLoaders = 32 * kLoad;
    static constexpr int kMma = kEpiWarps + kLoad;
    static constexpr int kThreads = 32 * (kMma + 1);
};
constexpr int kBiasRows = Warps<Product::kGradW>::kLoad;  // partial sums of dz per range: one per loader warp
constexpr int kWaitLimit = 1 << 22;
constexpr int kRing = 4;               // accumulators in tensor memory
constexpr uint32_t kSmemMost = 232448;

__device__ int g_fault;

template <int V>
struct Int {
    static constexpr int value = V;
};

template <typename T>
constexpr int kParts = sizeof(T) == 4 ? 3 : 1;
// Stages that one accumulator holds.
template <typename T>
constexpr int kChunk = sizeof(T) == 4 ? 1 : 16;

// Shared memory of one instance: slots of A and B parts, barriers.
template <typename T, Product P, int BN>
struct Layout {
    static constexpr bool kAMn = P == Product::kGradW;   // A is MN-major (contraction over rows)
    static constexpr bool kBMn = P != Product::kGradX;   // B likewise
    static constexpr uint32_t kAPart = kRowsTile * kStageK * 2;
    static constexpr uint32_t kBPart = kBMn && BN < 64 ? 64u * kStageK * 2 : (uint32_t)BN * kStageK * 2;
    static constexpr uint32_t kSlot = kParts<T> * (kAPart + kBPart);
    static constexpr uint32_t kTail = 256;  // barriers
    static constexpr int kFit = (int)((kSmemMost - kTail) / kSlot);
    static constexpr int kSlots = kFit < 6 ? kFit : 6;
    static constexpr uint32_t kOffBars = kSlots * kSlot;
    static constexpr uint32_t kBytes = kOffBars + kTail;
    static constexpr uint32_t kTmemCols = kRing * BN;
    static_assert(kSlots >= 2 && kBytes <= kSmemMost && kTmemCols <= 512, "linear layer shared memory");
};

// An operand as the loaders see it: source rows of ncols contiguous elements.
struct Operand {
    Rows rows;
    RowMap map;
    int nrows = 0, ncols = 0;
    int vec = 0;  // rows and columns in whole 16-byte groups
};

struct Job {
    Operand A, B, Z;  // Z: the pre-activation beside dz
    int silu = 0;
    int m = 0, n = 0, k = 0;  // extents of the product
    int ntn = 1, items = 1;   // tiles along n; work items
    int tiles = 1, range = 0; // grad_W: tiles of the output, rows per range
    RowMap map;               // rows of the output operands
    Rows out, z, residual;
    const void* bias = nullptr;
    int vec_out = 0;  // the epilogue's operands move 2 elements at a time
    void* gW = nullptr;
    float *part = nullptr, *bias_part = nullptr;
    const unsigned char* image = nullptr;  // B as tiles of operand parts, or null
};

// Loads under a predicate, zeros where it is false. The predicate is inside the
// instruction: a branch around a load would make the warp wait for it at the join.
__device__ __forceinline__ uint4 ldg16(const void* p, bool on) {
    uint4 v;
    asm volatile(
        "{\n .reg .pred pp;\n setp.ne.b32 pp, %5, 0;\n mov.u32 %0, 0;\n mov.u32 %1, 0;\n mov.u32 %2, 0;\n"
        " mov.u32 %3, 0;\n @pp ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];\n}"
        : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w)
        : "l"(p), "r"((int)on));
    return v;
}
__device__ __forceinline__ uint32_t ldg_elem(const float* p, bool on) {
    uint32_t v;
    asm volatile("{\n .reg .pred pp;\n setp.ne.b32 pp, %2, 0;\n mov.u32 %0, 0;\n @pp ld.global.nc.u32 %0, [%1];\n}"
                 : "=&r"(v)
                 : "l"(p), "r"((int)on));
    return v;
}
__device__ __forceinline__ uint32_t ldg_elem(const __nv_bfloat16* p, bool on) {
    uint32_t v;
    asm volatile(
        "{\n .reg .pred pp;\n .reg .u16 h;\n setp.ne.b32 pp, %2, 0;\n mov.u16 h, 0;\n @pp ld.global.nc.u16 h, [%1];\n"
        " cvt.u32.u16 %0, h;\n}"
        : "=&r"(v)
        : "l"(p), "r"((int)on));
    return v;
}

// 16 bytes of global memory into shared memory asynchronously, zeros where `on` is false.
__device__ __forceinline__ void copy16(void* dst, const void* src, bool on) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(tc::smem_u32(dst)), "l"(src), "r"(on ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Eight consecutive elements of a row as they lie in memory, zeros past the `left` that remain.
template <typename T>
struct Unit;
template <>
struct Unit<float> {
    uint4 a, b;
    template <bool VEC>
    __device__ __forceinline__ void load(const float* p, int left) {
        if constexpr (VEC) {
            a = ldg16(p, left >= 4);
            b = ldg16(p + 4, left >= 8);
        } else {
            a = make_uint4(ldg_elem(p, left > 0), ldg_elem(p + 1, left > 1), ldg_elem(p + 2, left > 2),
                           ldg_elem(p + 3, left > 3));
            b = make_uint4(ldg_elem(p + 4, left > 4), ldg_elem(p + 5, left > 5), ldg_elem(p + 6, left > 6),
                           ldg_elem(p + 7, left > 7));
        }
    }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        v[0] = __uint_as_float(a.x), v[1] = __uint_as_float(a.y), v[2] = __uint_as_float(a.z);
        v[3] = __uint_as_float(a.w), v[4] = __uint_as_float(b.x), v[5] = __uint_as_float(b.y);
        v[6] = __uint_as_float(b.z), v[7] = __uint_as_float(b.w);
    }
};
template <>
struct Unit<__nv_bfloat16> {
    uint4 a;
    template <bool VEC>
    __device__ __forceinline__ void load(const __nv_bfloat16* p, int left) {
        if constexpr (VEC) {
            a = ldg16(p, left >= 8);
        } else {
            a = make_uint4(ldg_elem(p, left > 0) | ldg_elem(p + 1, left > 1) << 16,
                           ldg_elem(p + 2, left > 2) | ldg_elem(p + 3, left > 3) << 16,
                           ldg_elem(p + 4, left > 4) | ldg_elem(p + 5, left > 5) << 16,
                           ldg_elem(p + 6, left > 6) | ldg_elem(p + 7, left > 7) << 16);
        }
    }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        v[0] = bf16_lo(a.x), v[1] = bf16_hi(a.x), v[2] = bf16_lo(a.y), v[3] = bf16_hi(a.y);
        v[4] = bf16_lo(a.z), v[5] = bf16_hi(a.z), v[6] = bf16_lo(a.w), v[7] = bf16_hi(a.w);
    }
};

// High halves of two floats as a bf16 pair (truncation).
__device__ __forceinline__ uint32_t high_pair(float a, float b) {
    return __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
}
__device__ __forceinline__ float high_part(float v) { return __uint_as_float(__float_as_uint(v) & 0xffff0000u); }

// Eight floats into the operand parts at `dst` (part stride bytes): three truncated
// parts of a float32 operand, one rounded part of a bf16 one.
template <typename T>
__device__ __forceinline__ void store_parts(unsigned char* dst, uint32_t part, float (&v)[8]) {
    if constexpr (sizeof(T) == 2) {
        *reinterpret_cast<uint4*>(dst) = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]),
                                                    pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
    } else {
#pragma unroll
        for (int p = 0; p < 3; ++p) {
            *reinterpret_cast<uint4*>(dst + p * part) = make_uint4(high_pair(v[0], v[1]), high_pair(v[2], v[3]),
                                                                   high_pair(v[4], v[5]), high_pair(v[6], v[7]));
            if (p < 2)
#pragma unroll
                for (int j = 0; j < 8; j += 2) {  // packed: v - high_part(v)
                    const float2 r = __fadd2_rn(make_float2(v[j], v[j + 1]),
                                                make_float2(-high_part(v[j]), -high_part(v[j + 1])));
                    v[j] = r.x, v[j + 1] = r.y;
                }
        }
    }
}

// Descriptors of the 128-byte-swizzled bf16 layouts. Atoms of 8 rows x 128 bytes, the
// 16-byte chunk index XORed with the row. K-major: rows are m (n), 64 k across, SBO =
// 1024 bytes between groups of 8 rows. MN-major: rows are k, 64 m (n) across; SBO =
// 1024 between groups of 8 k, LBO between panels of 64 m (n).
constexpr uint32_t kPanel = kStageK * 128;  // MN-major panel: 64 k rows of 128 bytes
template <bool MN>
__device__ __forceinline__ uint64_t desc128(uint32_t saddr) {
    const uint64_t lbo = MN ? (kPanel >> 4) : 1;
    return (uint64_t)((saddr >> 4) & 0x3FFFu) | (lbo << 16) | ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) |
           ((uint64_t)2 << 61);
}
// D f32, A and B bf16, shape 128 x n.
template <bool AMN, bool BMN>
constexpr uint32_t idesc_bf16(int n) {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((AMN ? 1u : 0u) << 15) | ((BMN ? 1u : 0u) << 16) |
           ((uint32_t)(n >> 3) << 17) | ((uint32_t)(kRowsTile >> 4) << 24);
}
__device__ __forceinline__ void mma_bf16(uint32_t d, uint64_t da, uint64_t db, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n .reg .pred pp;\n setp.ne.b32 pp, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, pp;\n}" ::"r"(d),
        "l"(da), "l"(db), "r"(idesc), "r"(acc)
        : "memory");
}

// Two elements of a row, zeros past the `left` that remain. V: both at once (they are
// aligned and `left` is not 1). The statements are volatile, so that they stay in order:
// a residual that is the output is read before it is written, and one row at a time.
template <bool V>
__device__ __forceinline__ float2 load2(const float* p, int left) {
    float a, b;
    if constexpr (V)
        asm volatile("{\n .reg .pred pp;\n setp.gt.s32 pp, %3, 0;\n mov.f32 %0, 0f00000000;\n mov.f32 %1, 0f00000000;\n"
            " @pp ld.global.v2.f32 {%0, %1}, [%2];\n}"
            : "=&f"(a), "=&f"(b)
            : "l"(p), "r"(left));
    else
        asm volatile("{\n .reg .pred p0, p1;\n setp.gt.s32 p0, %3, 0;\n setp.gt.s32 p1, %3, 1;\n mov.f32 %0, 0f00000000;\n"
            " mov.f32 %1, 0f00000000;\n @p0 ld.global.f32 %0, [%2];\n @p1 ld.global.f32 %1, [%2+4];\n}"
            : "=&f"(a), "=&f"(b)
            : "l"(p), "r"(left));
    return make_float2(a, b);
}
template <bool V>
__device__ __forceinline__ float2 load2(const __nv_bfloat16* p, int left) {
    uint32_t a;
    if constexpr (V)
        asm volatile("{\n .reg .pred pp;\n setp.gt.s32 pp, %2, 0;\n mov.u32 %0, 0;\n @pp ld.global.u32 %0, [%1];\n}"
            : "=&r"(a)
            : "l"(p), "r"(left));
    else
        asm volatile("{\n .reg .pred p0, p1;\n .reg .u16 h0, h1;\n setp.gt.s32 p0, %2, 0;\n setp.gt.s32 p1, %2, 1;\n"
            " mov.u16 h0, 0;\n mov.u16 h1, 0;\n @p0 ld.global.u16 h0, [%1];\n @p1 ld.global.u16 h1, [%1+2];\n"
            " mov.b32 %0, {h0, h1};\n}"
            : "=&r"(a)
            : "l"(p), "r"(left));
    return make_float2(bf16_lo(a), bf16_hi(a));
}
template <bool V>
__device__ __forceinline__ void store2(float* p, float2 v, int left) {
    if constexpr (V)
        asm volatile("{\n .reg .pred pp;\n setp.gt.s32 pp, %3, 0;\n @pp st.global.v2.f32 [%0], {%1, %2};\n}" ::"l"(p),
                     "f"(v.x), "f"(v.y), "r"(left));
    else
        asm volatile("{\n .reg .pred p0, p1;\n setp.gt.s32 p0, %3, 0;\n setp.gt.s32 p1, %3, 1;\n"
                     " @p0 st.global.f32 [%0], %1;\n @p1 st.global.f32 [%0+4], %2;\n}" ::"l"(p),
                     "f"(v.x), "f"(v.y), "r"(left));
}
template <bool V>
__device__ __forceinline__ void store2(__nv_bfloat16* p, float2 v, int left) {
    const uint32_t a = pack_bf16(v.x, v.y);
    if constexpr (V)
        asm volatile("{\n .reg .pred pp;\n setp.gt.s32 pp, %2, 0;\n @pp st.global.u32 [%0], %1;\n}" ::"l"(p), "r"(a),
                     "r"(left));
    else
        asm volatile("{\n .reg .pred p0, p1;\n .reg .u16 h0, h1;\n setp.gt.s32 p0, %2, 0;\n setp.gt.s32 p1, %2, 1;\n"
                     " mov.b32 {h0, h1}, %1;\n @p0 st.global.u16 [%0], h0;\n @p1 st.global.u16 [%0+2], h1;\n}" ::"l"(p),
                     "r"(a), "r"(left));
}

// One work item: an output tile, and the range of the contraction it covers.
struct Item {
    int m0, n0, k0, k1, split, stages;
};
template <Product P>
__device__ __forceinline__ Item item_of(const Job& j, int i, int bn) {
    Item it;
    int tile = i;
    it.split = 0, it.k0 = 0, it.k1 = j.k;
    if (P == Product::kGradW) {
        it.split = i / j.tiles;
        tile = i - it.split * j.tiles;
        it.k0 = it.split * j.range;
        it.k1 = min(j.k, it.k0 + j.range);
    }
    const int mt = tile / j.ntn;
    it.m0 = mt * kRowsTile;
    it.n0 = (tile - mt * j.ntn) * bn;
    it.stages = (it.k1 - it.k0 + kStageK - 1) / kStageK;
    return it;
}

// The epilogue of a tile on one warp's 32 rows x BN / 2 columns, in the accumulator's
// fragment layout: a lane holds 4 rows, of each 2 neighbouring columns in every 8. The 4
// lanes of a row make whole 32-byte sectors of float32, so loads and stores go straight
// between registers and memory, and a lane has 4 row addresses, not one per element.
// V: every operand of the epilogue moves 2 elements at a time.
template <typename T, Product P, int BN, bool V>
__device__ __forceinline__ void finish(const Job& job, const Item& it, float (&acc)[2][BN / 4], int quad, int half,
                                       int lane) {
    constexpr int kGroups = BN / 16;  // groups of 8 columns
    const int n0 = it.n0 + half * (BN / 2) + 2 * (lane & 3);
    const bool has_res = P == Product::kForward && job.residual.p != nullptr;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int m = it.m0 + quad * 32 + 8 * r + (lane >> 2);
        const int left = m < job.m ? job.n - n0 : 0;
        float2 v[kGroups];
#pragma unroll
        for (int c = 0; c < kGroups; ++c)
            v[c] = make_float2(acc[r >> 1][4 * c + 2 * (r & 1)], acc[r >> 1][4 * c + 2 * (r & 1) + 1]);
        if constexpr (P == Product::kForward) {
            float2 res[kGroups];
            if (has_res) {
                const T* p = static_cast<const T*>(job.residual.p) + job.residual.offset(job.map, m) + n0;
#pragma unroll
                for (int c = 0; c < kGroups; ++c) res[c] = load2<V>(p + 8 * c, left - 8 * c);
            }
            if (job.bias) {
                const T* p = static_cast<const T*>(job.bias) + n0;
#pragma unroll
                for (int c = 0; c < kGroups; ++c) {
                    const float2 b = load2<V>(p + 8 * c, job.n - n0 - 8 * c);
                    v[c].x += b.x, v[c].y += b.y;
                }
            }
            if (job.z.p) {
                T* p = static_cast<T*>(job.z.p) + job.z.offset(job.map, m) + n0;
#pragma unroll
                for (int c = 0; c < kGroups; ++c) store2<V>(p + 8 * c, v[c], left - 8 * c);
            }
            if (job.silu)
#pragma unroll
                for (int c = 0; c < kGroups; ++c) v[c].x = silu(v[c].x), v[c].y = silu(v[c].y);
            if (has_res)
#pragma unroll
                for (int c = 0; c < kGroups; ++c) v[c].x += res[c].x, v[c].y += res[c].y;
        }
        if (P == Product::kGradW && job.part) {
            float* p = job.part + ((size_t)it.split * job.m + m) * job.n + n0;
#pragma unroll
            for (int c = 0; c < kGroups; ++c) store2<V>(p + 8 * c, v[c], left - 8 * c);
        } else {
            T* p = P == Product::kGradW ? static_cast<T*>(job.gW) + (size_t)m * job.n + n0
                                        : static_cast<T*>(job.out.p) + job.out.offset(job.map, m) + n0;
#pragma unroll
            for (int c = 0; c < kGroups; ++c) store2<V>(p + 8 * c, v[c], left - 8 * c);
        }
    }
}

// A loader's share of an operand tile of ROWS source rows by COLS columns: units of 8
// columns, unit u = t + 256 i at row u / (COLS / 8).
template <int ROWS, int COLS, int kLoaders>
struct Share {
    static constexpr int kPerRow = COLS / 8;
    static constexpr int kIters = ROWS * kPerRow / kLoaders;
    static_assert(kIters >= 1 && ROWS * kPerRow % kLoaders == 0, "loader share");
    static __device__ __forceinline__ int row(int t, int i) { return (t + kLoaders * i) / kPerRow; }
    static __device__ __forceinline__ int col(int t) { return t % kPerRow; }
    static __device__ __forceinline__ uint32_t offset(int t, int i) {
        const int r = row(t, i), c = col(t);
        return (uint32_t)(c >> 3) * kPanel + (uint32_t)(r >> 3) * 1024 + (uint32_t)(r & 7) * 128 +
               (uint32_t)(((c & 7) ^ (r & 7)) << 4);
    }
};

// IMAGE: B arrives as ready tiles (etp_linear_image_kernel) by bulk copies.
template <typename T, Product P, int BN, bool VEC, bool IMAGE>
__global__ void __launch_bounds__(Warps<P>::kThreads, 1) etp_linear_kernel(const __grid_constant__ Job job) {
    using Lay = Layout<T, P, BN>;
    constexpr int NP = kParts<T>;
    constexpr int kLoadWarps = Warps<P>::kLoad, kLoaders = Warps<P>::kLoaders, kMmaWarp = Warps<P>::kMma;
    constexpr bool kDzA = P == Product::kGradX, kDzB = P == Product::kGradW;
    // bfloat16 operands that need no arithmetic are copied straight to shared memory
    constexpr bool kCopyA = sizeof(T) == 2 && VEC && !kDzA, kCopyB = sizeof(T) == 2 && VEC && !kDzB && !IMAGE;
    constexpr bool kCopies = kCopyA || kCopyB;
    constexpr bool kRegA = !kCopyA, kRegB = !kCopyB && !IMAGE;
    constexpr int kDepth = Lay::kSlots - 1;  // stages of copies in flight
    // parts of a stage that a loader holds in flight in turn, as registers allow
    constexpr int kHalves = IMAGE || sizeof(T) == 2 ? (P == Product::kForward ? 1 : 2) : P == Product::kGradX ? 4 : 2;
    using ShareA = Share<Lay::kAMn ? kStageK : kRowsTile, Lay::kAMn ? kRowsTile : kStageK, kLoaders>;
    using ShareB = Share<Lay::kBMn ? kStageK : BN, Lay::kBMn ? BN : kStageK, kLoaders>;
    constexpr int IA = ShareA::kIters, IB = ShareB::kIters;
    constexpr int HA = (IA + kHalves - 1) / kHalves, HB = (IB + kHalves - 1) / kHalves;  // units of a part

    extern __shared__ __align__(1024) unsigned char smem[];
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + Lay::kOffBars);  // a slot's operands are written
    uint64_t* bfull = full + Lay::kSlots;                                 // its image tile has arrived
    uint64_t* empty = bfull + Lay::kSlots;                                // its MMAs are done
    uint64_t* tfull = empty + Lay::kSlots;                                // an accumulator is complete
    uint64_t* tempty = tfull + kRing;                                     // and has been read
    uint64_t* drain = tempty + kRing;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31;

    if (warp == kMmaWarp) tc::tmem_alloc(tmem_slot, Lay::kTmemCols);
    if (t == 0) {
        for (int i = 0; i < Lay::kSlots; ++i) {
            tc::mbar_init(&full[i], kLoadWarps);
            tc::mbar_init(&bfull[i], 1);
            tc::mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < kRing; ++i) {
            tc::mbar_init(&tfull[i], 1);
            tc::mbar_init(&tempty[i], kEpiWarps);
        }
        tc::mbar_init(drain, 1);
        *abort_flag = 0;
        tc::mbar_fence_init();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    // A bounded wait; false: leave the loops. wait(): the same answer for the whole warp.
    auto wait1 = [&](uint64_t* bar, unsigned parity) {
        const bool ok = !*abort_flag && tc::mbar_wait(bar, parity, kWaitLimit);
        if (!ok) *abort_flag = 1;
        return ok;
    };
    auto wait = [&](uint64_t* bar, unsigned parity) { return __all_sync(0xffffffffu, wait1(bar, parity)) != 0; };
    int images = 0;  // (loader thread 0) image tiles asked for

    if (warp >= kEpiWarps && warp < kMmaWarp) {  // loaders
        const int lt = t - 32 * kEpiWarps;
        Unit<T> ra[kRegA ? HA : 1], rb[kRegB ? HB : 1], rz[kDzA ? HA : kDzB ? HB : 1];
        // Two cursors: the stage that is stored now, and the one that is fetched into registers.
        struct Cursor {
            int i, ks;
            Item it;
        } now{(int)blockIdx.x, 0, item_of<P>(job, blockIdx.x, BN)}, next = now;
        auto advance = [&](Cursor& c) {  // true: another item
            if (++c.ks < c.it.stages) return false;
            c.ks = 0;
            c.i += gridDim.x;
            if (c.i >= job.items) return false;
            c.it = item_of<P>(job, c.i, BN);
            return true;
        };
        // addresses of a K-major A's rows, for the cursor that reads it
        const T *arow[Lay::kAMn ? 1 : IA], *zrow[kDzA ? IA : 1];
        auto set_rows = [&](const Item& it) {
            if constexpr (!Lay::kAMn) {
#pragma unroll
                for (int i = 0; i < IA; ++i) {
                    const int r = it.m0 + ShareA::row(lt, i);
                    arow[i] = static_cast<const T*>(job.A.rows.p) + job.A.rows.offset(job.A.map, r) + 8 * ShareA::col(lt);
                    if constexpr (kDzA) {
                        zrow[i] =
                            static_cast<const T*>(job.Z.rows.p) + job.Z.rows.offset(job.Z.map, r) + 8 * ShareA::col(lt);
                    }
                }
            }
        };
        // unit i of a stage's A (B) tile: its address, and how many of its elements exist
        auto unit_a = [&](const Cursor& c, int i, const T*& p) {
            const int kk = c.it.k0 + c.ks * kStageK;
            if constexpr (Lay::kAMn) {
                const int r = kk + ShareA::row(lt, i), col = c.it.m0 + 8 * ShareA::col(lt);
                p = static_cast<const T*>(job.A.rows.p) + job.A.rows.offset(job.A.map, r) + col;
                return r < c.it.k1 ? job.A.ncols - col : 0;
            } else {
                p = arow[i] + kk;
                return c.it.m0 + ShareA::row(lt, i) < job.A.nrows ? job.A.ncols - kk - 8 * ShareA::col(lt) : 0;
            }
        };
        auto unit_b = [&](const Cursor& c, int i, const T*& p, const T*& pz) {
            const int kk = c.it.k0 + c.ks * kStageK;
            const int r = (Lay::kBMn ? kk : c.it.n0) + ShareB::row(lt, i);
            const int col = (Lay::kBMn ? c.it.n0 : kk) + 8 * ShareB::col(lt);
            p = static_cast<const T*>(job.B.rows.p) + job.B.rows.offset(job.B.map, r) + col;
            if (kDzB) pz = static_cast<const T*>(job.Z.rows.p) + job.Z.rows.offset(job.Z.map, r) + col;
            return r < (kDzB ? c.it.k1 : job.B.nrows) ? job.B.ncols - col : 0;
        };
        auto fetch_a = [&](const Cursor& c, int h, int q) {  // unit q of part h (and its pre-activation)
            if constexpr (kRegA) {
                if (h * HA + q >= IA) return;
                const T* p;
                const int left = unit_a(c, h * HA + q, p);
                ra[q].template load<VEC>(p, left);
                if constexpr (kDzA) {
                    if (job.silu) rz[q].template load<VEC>(zrow[h * HA + q] + c.it.k0 + c.ks * kStageK, left);
                }
            }
        };
        auto fetch_b = [&](const Cursor& c, int h, int q) {
            if constexpr (kRegB) {
                if (h * HB + q >= IB) return;
                const T *p, *pz = nullptr;
                const int left = unit_b(c, h * HB + q, p, pz);
                rb[q].template load<VEC>(p, left);
                if constexpr (kDzB) {
                    if (job.silu) rz[q].template load<VEC>(pz, left);
                }
            }
        };
        auto dz = [&](float (&v)[8], const Unit<T>& z) {
            if (!job.silu) return;
            float zv[8];
            z.get(zv);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] *= silu_grad(zv[j]);
        };
        auto arrive = [&](int slot) {  // this warp's part of the slot is written
            tc::fence_proxy_async();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&full[slot]);
        };
        float bsum[8];
        int n = 0;
        set_rows(now.it);
#pragma unroll
        for (int q = 0; q < HA; ++q) fetch_a(now, 0, q);
#pragma unroll
        for (int q = 0; q < HB; ++q) fetch_b(now, 0, q);
        for (; now.i < job.items; ++n) {
            const int slot = n % Lay::kSlots;
            if (n >= Lay::kSlots && !wait(&empty[slot], (n / Lay::kSlots - 1) & 1)) break;
            unsigned char* sa = smem + slot * Lay::kSlot;
            unsigned char* sb = sa + NP * Lay::kAPart;
            if (IMAGE && lt == 0) {
                const int nks = (job.k + kStageK - 1) / kStageK;
                tc::mbar_expect_tx(&bfull[slot], NP * Lay::kBPart);
                tc::bulk_g2s(sb, job.image + (size_t)((now.it.n0 / BN) * nks + now.ks) * (NP * Lay::kBPart),
                             NP * Lay::kBPart, &bfull[slot]);
                images = n + 1;
            }
            if constexpr (kCopyA) {
#pragma unroll
                for (int q = 0; q < IA; ++q) {
                    const T* p;
                    const int left = unit_a(now, q, p);
                    copy16(sa + ShareA::offset(lt, q), left > 0 ? p : static_cast<const T*>(job.A.rows.p), left > 0);
                }
            }
            if constexpr (kCopyB) {
#pragma unroll
                for (int q = 0; q < IB; ++q) {
                    const T *p, *pz = nullptr;
                    const int left = unit_b(now, q, p, pz);
                    copy16(sb + ShareB::offset(lt, q), left > 0 ? p : static_cast<const T*>(job.B.rows.p), left > 0);
                }
            }
            if (kCopies) copy_commit();
            if (kDzB && now.ks == 0)
#pragma unroll
                for (int j = 0; j < 8; ++j) bsum[j] = 0.f;
            // a unit's registers are refilled as soon as it is stored: it is in flight while the others are converted
#pragma unroll
            for (int h = 0; h < kHalves; ++h) {
                const bool here = h + 1 < kHalves;
                if (!here && advance(next) && kRegA) set_rows(next.it);
                const bool more = next.i < job.items;
                if constexpr (kRegA) {
#pragma unroll
                    for (int q = 0; q < HA; ++q) {
                        if (h * HA + q < IA) {
                            float v[8];
                            ra[q].get(v);
                            if constexpr (kDzA) {
                                dz(v, rz[q]);
                            }
                            store_parts<T>(sa + ShareA::offset(lt, h * HA + q), Lay::kAPart, v);
                        }
                        if (here)
                            fetch_a(now, h + 1, q);
                        else if (more)
                            fetch_a(next, 0, q);
                    }
                }
                if constexpr (kRegB) {
#pragma unroll
                    for (int q = 0; q < HB; ++q) {
                        if (h * HB + q < IB) {
                            float v[8];
                            rb[q].get(v);
                            if constexpr (kDzB) {
                                dz(v, rz[q]);
#pragma unroll
                                for (int j = 0; j < 8; ++j) bsum[j] += v[j];
                            }
                            store_parts<T>(sb + ShareB::offset(lt, h * HB + q), Lay::kBPart, v);
                        }
                        if (here)
                            fetch_b(now, h + 1, q);
                        else if (more)
                            fetch_b(next, 0, q);
                    }
                }
            }
            if (!kCopies) {
                arrive(slot);
            } else if (n >= kDepth) {
                copy_wait<kDepth>();
                arrive((n - kDepth) % Lay::kSlots);
            }
            if (kDzB && now.ks + 1 >= now.it.stages && job.bias_part && now.it.m0 == 0) {
                // the item's sums of dz over its rows: the lanes of a warp that share columns, one row per warp
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    for (int o = ShareB::kPerRow; o < 32; o <<= 1) bsum[j] += __shfl_xor_sync(0xffffffffu, bsum[j], o);
                if (lane < ShareB::kPerRow) {
                    float* row = job.bias_part + (size_t)(now.it.split * kLoadWarps + (warp - kEpiWarps)) * job.n;
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const int c = now.it.n0 + 8 * ShareB::col(lt) + j;
                        if (c < job.n) row[c] = bsum[j];
                    }
                }
            }
            now = next;
            if (kCopyA && now.ks == 0) set_rows(now.it);
        }
        if (kCopies) {
            copy_wait<0>();
            for (int m = n > kDepth ? n - kDepth : 0; m < n; ++m) arrive(m % Lay::kSlots);
        }
    } else if (warp == kMmaWarp && lane == 0) {
        constexpr uint32_t idesc = idesc_bf16<Lay::kAMn, Lay::kBMn>(BN);
        // one K step of 16, one part: descriptor units of 16 bytes
        constexpr uint32_t kStepA = (Lay::kAMn ? 2048 : 32) >> 4, kStepB = (Lay::kBMn ? 2048 : 32) >> 4;
        constexpr int kPairs = NP == 3 ? 6 : 1;
        constexpr int pa[6] = {NP == 3 ? 1 : 0, 0, 2, 0, 1, 0}, pb[6] = {NP == 3 ? 1 : 0, 2, 0, 1, 0, 0};
        const uint64_t base_a = desc128<Lay::kAMn>(tc::smem_u32(smem));
        const uint64_t base_b = desc128<Lay::kBMn>(tc::smem_u32(smem + NP * Lay::kAPart));
        // the stage's MMAs, unrolled: descriptors are the slot's plus constants
        auto issue = [&](auto steps_c, uint32_t d, uint64_t da, uint64_t db, bool first) {
            constexpr int S = decltype(steps_c)::value;
#pragma unroll
            for (int q = 0; q < kPairs; ++q)
#pragma unroll
                for (int s = 0; s < S; ++s)
                    mma_bf16(d, da + (uint64_t)(pa[q] * (Lay::kAPart >> 4) + s * kStepA),
                             db + (uint64_t)(pb[q] * (Lay::kBPart >> 4) + s * kStepB), idesc,
                             q == 0 && s == 0 ? (first ? 0u : 1u) : 1u);
        };
        int n = 0, chunk = 0;
        bool ok = true;
        for (int i = blockIdx.x; i < job.items && ok; i += gridDim.x) {
            const Item it = item_of<P>(job, i, BN);
            for (int ks = 0; ks < it.stages; ++ks, ++n) {
                const int slot = n % Lay::kSlots, buf = chunk % kRing;
                const bool first = ks % kChunk<T> == 0;
                if ((first && chunk >= kRing && !wait1(&tempty[buf], (chunk / kRing - 1) & 1)) ||
                    !wait1(&full[slot], (n / Lay::kSlots) & 1) ||
                    (IMAGE && !wait1(&bfull[slot], (n / Lay::kSlots) & 1))) {
                    ok = false;
                    break;
                }
                tc::fence_after_sync();
                const int left = it.k1 - it.k0 - ks * kStageK;
                const uint32_t d = tmem + buf * BN;
                const uint64_t da = base_a + (uint64_t)(slot * (Lay::kSlot >> 4));
                const uint64_t db = base_b + (uint64_t)(slot * (Lay::kSlot >> 4));
                if (left > 48) issue(Int<4>{}, d, da, db, first);
                else if (left > 32) issue(Int<3>{}, d, da, db, first);
                else if (left > 16) issue(Int<2>{}, d, da, db, first);
                else issue(Int<1>{}, d, da, db, first);
                tc::mma_commit(&empty[slot]);
                if (ks + 1 == it.stages || (ks + 1) % kChunk<T> == 0) {
                    tc::mma_commit(&tfull[buf]);
                    ++chunk;
                }
            }
        }
    } else if (warp < kEpiWarps) {
        constexpr int NR = BN / 4;  // registers of a warp's 16 lanes x BN / 2 columns
        constexpr int kPiece = NR < 16 ? NR : 16;
        const int quad = warp & 3, half = warp >> 2;
        const uint32_t base = tmem + ((uint32_t)(quad * 32) << 16) + half * (BN / 2);
        int chunk = 0;
        bool ok = true;
        for (int i = blockIdx.x; i < job.items && ok; i += gridDim.x) {
            const Item it = item_of<P>(job, i, BN);
            float acc[2][NR];
#pragma unroll
            for (int j = 0; j < NR; ++j) acc[0][j] = acc[1][j] = 0.f;
            for (int ks = 0; ks < it.stages; ks += kChunk<T>, ++chunk) {
                const int buf = chunk % kRing;
                if (!wait(&tfull[buf], (chunk / kRing) & 1)) {
                    ok = false;
                    break;
                }
                tc::fence_after_sync();
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int c = 0; c < NR; c += kPiece) {
                        float v[kPiece];
                        tc::tmem_ld_frag<kPiece>(base + ((uint32_t)(16 * h) << 16) + buf * BN + 2 * c, v);
                        tc::tmem_wait_ld(v);
#pragma unroll
                        for (int j = 0; j < kPiece; ++j) acc[h][c + j] += v[j];
                    }
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&tempty[buf]);
            }
            if (!ok) break;
            if (job.vec_out)
                finish<T, P, BN, true>(job, it, acc, quad, half, lane);
            else
                finish<T, P, BN, false>(job, it, acc, quad, half, lane);
        }
    }
    __syncthreads();
    if (*abort_flag) {  // leave no MMA or copy in flight on the freed memory
        if (t == 32 * kMmaWarp) {
            atomicOr(&g_fault, 1);
            tc::mma_commit(drain);
            tc::mbar_wait(drain, 0, kWaitLimit);
        }
        if (IMAGE && t == 32 * kEpiWarps)
            for (int m = images > Lay::kSlots ? images - Lay::kSlots : 0; m < images; ++m)
                tc::mbar_wait(&bfull[m % Lay::kSlots], (m / Lay::kSlots) & 1, kWaitLimit);
        __syncthreads();
    }
    tc::fence_before_sync();
    __syncthreads();
    if (warp == kMmaWarp) tc::tmem_dealloc(tmem, Lay::kTmemCols);
}

// W as tiles of operand parts in the layout of a slot's B, tile (nt, ks) after tile:
// converted once here instead of once per row tile by every CTA. A thread converts
// units of 8 consecutive elements of W.
template <typename T, Product P, int BN>
__global__ void __launch_bounds__(256) etp_linear_image_kernel(const T* __restrict__ W, int rows, int cols, bool vec,
                                                               unsigned char* __restrict__ image) {
    using Lay = Layout<T, P, BN>;
    constexpr int R = Lay::kBMn ? kStageK : BN, C = Lay::kBMn ? BN : kStageK;  // W's rows and columns in a tile
    constexpr int kPerRow = C / 8, kUnits = R * kPerRow;
    const int ct = (cols + C - 1) / C, rt = (rows + R - 1) / R;
    const int u = blockIdx.x * 256 + threadIdx.x, tile = u / kUnits, w = u % kUnits;
    if (tile >= ct * rt) return;
    // tiles along the contraction are adjacent: it runs over W's rows (MN-major) or columns
    const int rti = Lay::kBMn ? tile % rt : tile / ct, cti = Lay::kBMn ? tile / rt : tile % ct;
    const int r = w / kPerRow, c = w % kPerRow, gr = rti * R + r, gc = cti * C + 8 * c;
    const T* p = W + (size_t)gr * cols + gc;
    const int left = gr < rows ? cols - gc : 0;
    Unit<T> q;
    if (vec)
        q.template load<true>(p, left);
    else
        q.template load<false>(p, left);
    float v[8];
    q.get(v);
    store_parts<T>(image + (size_t)tile * kParts<T> * Lay::kBPart + (uint32_t)(c >> 3) * kPanel +
                       (uint32_t)(r >> 3) * 1024 + (uint32_t)(r & 7) * 128 + (uint32_t)(((c & 7) ^ (r & 7)) << 4),
                   Lay::kBPart, v);
}

// grad_W from the ranges' sums [splits][count] and grad_bias from [bias_rows][N], both in
// order: 32 columns of up to 4 elements by 8 row lanes per block, then the 8 sums in order.
template <typename T>
__global__ void __launch_bounds__(256)
    etp_linear_join_kernel(const float* __restrict__ part, int splits, size_t count, T* __restrict__ gW,
                           const float* __restrict__ bias_part, int bias_rows, int N, T* __restrict__ gbias,
                           int blocks_w) {
    __shared__ float red[8][32];
    const int sub = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const bool is_bias = (int)blockIdx.x >= blocks_w;
    const size_t cols = is_bias ? (size_t)N : count;
    const size_t col = (size_t)(is_bias ? blockIdx.x - blocks_w : blockIdx.x) * 32 + lane;
    const int rows = is_bias ? bias_rows : splits;
    const float* src = is_bias ? bias_part : part;
    float s = 0.f;
    if (col < cols)
#pragma unroll 8
        for (int r = sub; r < rows; r += 8) s += src[(size_t)r * cols + col];
    red[sub][lane] = s;
    __syncthreads();
    if (sub != 0 || col >= cols) return;
#pragma unroll
    for (int w = 1; w < 8; ++w) s += red[w][lane];
    (is_bias ? gbias : gW)[col] = from_float<T>(s);
}

bool rows_aligned(const Rows& r, int elem, int bytes) {
    const unsigned n = bytes / elem;
    return (reinterpret_cast<uintptr_t>(r.p) % bytes) == 0 && r.gs % n == 0 && r.rs % n == 0;
}

Operand operand(const Rows& r, const RowMap& map, int nrows, int ncols, int elem) {
    Operand o;
    o.rows = r, o.map = map, o.nrows = nrows, o.ncols = ncols;
    o.vec = rows_aligned(r, elem, 16) && ncols % (16 / elem) == 0;
    return o;
}

Operand matrix(const void* p, int nrows, int ncols, int elem) {
    Rows r;
    r.p = const_cast<void*>(p), r.gs = (unsigned)ncols;
    RowMap map;
    map.M = nrows;
    return operand(r, map, nrows, ncols, elem);
}

template <typename T, Product P, int BN, bool VEC, bool IMAGE>
cudaError_t launch_kernel(const Job& j, cudaStream_t s) {
    using Lay = Layout<T, P, BN>;
    const cudaError_t e = cudaFuncSetAttribute(etp_linear_kernel<T, P, BN, VEC, IMAGE>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Lay::kBytes);
    if (e != cudaSuccess) return e;
    const int sms = sm_count();
    etp_linear_kernel<T, P, BN, VEC, IMAGE><<<j.items < sms ? j.items : sms, Warps<P>::kThreads, Lay::kBytes, s>>>(j);
    return cudaGetLastError();
}

// VEC: the operands' rows move in 16-byte groups.
template <typename T, Product P, int BN>
cudaError_t launch_bn(Job& j, unsigned char* image, cudaStream_t s) {
    const bool z = !j.Z.rows.p || j.Z.vec;
    if constexpr (P != Product::kGradW) {
        if (image) {
            using Lay = Layout<T, P, BN>;
            const int rows = j.B.nrows, cols = j.B.ncols;
            const int R = Lay::kBMn ? kStageK : BN, C = Lay::kBMn ? BN : kStageK;
            const long long units = (long long)((rows + R - 1) / R) * ((cols + C - 1) / C) * (R * C / 8);
            etp_linear_image_kernel<T, P, BN><<<(unsigned)((units + 255) / 256), 256, 0, s>>>(
                static_cast<const T*>(j.B.rows.p), rows, cols, j.B.vec, image);
            const cudaError_t e = cudaGetLastError();
            if (e != cudaSuccess) return e;
            j.image = image;
            return j.A.vec && z ? launch_kernel<T, P, BN, true, true>(j, s)
                                : launch_kernel<T, P, BN, false, true>(j, s);
        }
    }
    return j.A.vec && j.B.vec && z ? launch_kernel<T, P, BN, true, false>(j, s)
                                   : launch_kernel<T, P, BN, false, false>(j, s);
}

// How the forward and grad_x products of M rows, k contracted and n output columns are
// tiled: the widest tile that still gives every SM one, or the narrowest; and whether W
// is converted ahead (an image), which pays once several row tiles share it.
struct Tiling {
    int bn;
    bool image;
    size_t image_bytes;
};
Tiling tiling(bool bf16, Product p, int M, int k, int n) {
    const long long mt = ((long long)M + kRowsTile - 1) / kRowsTile;
    const int sms = sm_count();
    Tiling t;
    t.bn = n > 64 && mt * ((n + 127) / 128) >= sms ? 128 : n > 32 && mt * ((n + 63) / 64) >= sms ? 64 : 32;
    t.image = mt >= sms;
    const size_t part = (size_t)(p == Product::kForward && t.bn < 64 ? 64 : t.bn) * kStageK * 2;
    t.image_bytes =
        t.image ? (size_t)((n + t.bn - 1) / t.bn) * ((k + kStageK - 1) / kStageK) * (bf16 ? 1 : 3) * part : 0;
    return t;
}

template <typename T, Product P>
cudaError_t launch(Job& j, int bn, int splits, unsigned char* image, cudaStream_t s) {
    j.ntn = (j.n + bn - 1) / bn;
    const long long tiles = (long long)((j.m + kRowsTile - 1) / kRowsTile) * j.ntn;
    if (tiles > 0x7fff0000LL) return cudaErrorInvalidValue;
    j.tiles = j.items = (int)tiles;
    if (P == Product::kGradW) {  // a tile of no rows still is one tile
        if (j.m == 0) j.tiles = j.ntn;
        j.items = j.tiles * splits;
    }
    switch (bn) {
        case 128: return launch_bn<T, P, 128>(j, image, s);
        case 64: return launch_bn<T, P, 64>(j, image, s);
        default: return launch_bn<T, P, 32>(j, image, s);
    }
}

// grad_W: tile width and ranges of the rows. Ranges are whole stages, and at least four
// of them, so that the partial sums stay small beside the operands.
struct Ranges {
    int bn, tiles, splits, range;
};
Ranges ranges(int M, int K, int N) {
    Ranges r;
    r.bn = N > 64 ? 128 : N > 32 ? 64 : 32;
    r.tiles = ((K + kRowsTile - 1) / kRowsTile) * ((N + r.bn - 1) / r.bn);
    const int sms = sm_count();
    const int stages = (M + kStageK - 1) / kStageK;
    int want = r.tiles < sms ? sms / r.tiles : 1;
    const int most = (stages + 3) / 4;
    want = want < most ? want : most;
    const int per = want > 0 ? (stages + want - 1) / want : 1;
    r.range = per * kStageK;
    r.splits = stages > 0 ? (stages + per - 1) / per : 0;
    return r;
}

template <typename T>
cudaError_t forward(const LinearArgs& a, cudaStream_t s) {
    constexpr int elem = sizeof(T);
    Job j;
    j.A = operand(a.x, a.map, a.map.M, a.K, elem);
    j.B = matrix(a.W, a.K, a.N, elem);
    j.silu = a.silu;
    j.m = a.map.M, j.n = a.N, j.k = a.K;
    j.map = a.map;
    j.out = a.out, j.z = a.z, j.residual = a.residual;
    j.bias = a.bias;
    j.vec_out = a.N % 2 == 0 && rows_aligned(a.out, elem, 2 * elem) && rows_aligned(a.z, elem, 2 * elem) &&
                rows_aligned(a.residual, elem, 2 * elem) && (reinterpret_cast<uintptr_t>(a.bias) % (2 * elem)) == 0;
    const Tiling t = tiling(elem == 2, Product::kForward, j.m, j.k, j.n);
    return launch<T, Product::kForward>(j, t.bn, 1, t.image ? reinterpret_cast<unsigned char*>(a.ws) : nullptr, s);
}

template <typename T>
cudaError_t backward(const LinearArgs& a, cudaStream_t s) {
    constexpr int elem = sizeof(T);
    if (a.gx.p && a.map.M > 0) {
        Job j;
        j.A = operand(a.g, a.map, a.map.M, a.N, elem);
        if (a.silu) j.Z = operand(a.z, a.map, a.map.M, a.N, elem);
        j.B = matrix(a.W, a.K, a.N, elem);
        j.silu = a.silu;
        j.m = a.map.M, j.n = a.K, j.k = a.N;
        j.map = a.map;
        j.out = a.gx;
        j.vec_out = a.K % 2 == 0 && rows_aligned(a.gx, elem, 2 * elem);
        const Tiling t = tiling(elem == 2, Product::kGradX, j.m, j.k, j.n);
        const cudaError_t e = launch<T, Product::kGradX>(
            j, t.bn, 1, t.image ? reinterpret_cast<unsigned char*>(a.ws) : nullptr, s);
        if (e != cudaSuccess) return e;
    }
    if (!a.gW && !a.gbias) return cudaSuccess;
    // without grad_W the tile has no rows: only the loaders' sums of dz are wanted
    const int K = a.gW ? a.K : 0;
    const Ranges r = ranges(a.map.M, a.gW ? a.K : 1, a.N);
    const bool join = r.splits != 1;
    float* bias_part = a.gbias ? a.ws : nullptr;
    float* part = a.ws + (size_t)r.splits * kBiasRows * a.N;
    if (r.splits > 0) {
        Job j;
        j.A = operand(a.gW ? a.x : a.g, a.map, a.map.M, K, elem);  // without grad_W: no columns, nothing read
        j.B = operand(a.g, a.map, a.map.M, a.N, elem);
        if (a.silu) j.Z = operand(a.z, a.map, a.map.M, a.N, elem);
        j.silu = a.silu;
        j.m = K, j.n = a.N, j.k = a.map.M;
        j.range = r.range;
        j.gW = a.gW;
        j.part = join && a.gW ? part : nullptr;
        j.bias_part = bias_part;
        j.vec_out = a.N % 2 == 0 && (j.part || (reinterpret_cast<uintptr_t>(a.gW) % (2 * elem)) == 0);
        const cudaError_t e = launch<T, Product::kGradW>(j, r.bn, r.splits, nullptr, s);
        if (e != cudaSuccess) return e;
    }
    const size_t count = a.gW && join ? (size_t)a.K * a.N : 0;
    const int blocks_w = (int)((count + 31) / 32), blocks_b = a.gbias ? (a.N + 31) / 32 : 0;
    if (blocks_w + blocks_b == 0) return cudaSuccess;
    etp_linear_join_kernel<T><<<blocks_w + blocks_b, 256, 0, s>>>(part, r.splits, count, static_cast<T*>(a.gW),
                                                                  bias_part, r.splits * kBiasRows, a.N,
                                                                  static_cast<T*>(a.gbias), blocks_w);
    return cudaGetLastError();
}

}  // namespace

cudaError_t linear_forward(bool bf16, const LinearArgs& a, cudaStream_t s) {
    if (a.map.M == 0) return cudaSuccess;
    return bf16 ? forward<__nv_bfloat16>(a, s) : forward<float>(a, s);
}

// The backward's two products use the workspace one after the other.
size_t linear_workspace_bytes(bool bf16, int M, int K, int N, bool fwd, bool gx, bool gw, bool gb) {
    size_t most = 0;
    auto at_least = [&](size_t v) { most = v > most ? v : most; };
    if (fwd) at_least(tiling(bf16, Product::kForward, M, K, N).image_bytes);
    if (gx) at_least(tiling(bf16, Product::kGradX, M, N, K).image_bytes);
    if (gw || gb) {
        const Ranges r = ranges(M, gw ? K : 1, N);  // as backward() asks for them
        at_least(((gw && r.splits > 1 ? (size_t)r.splits * K * N : 0) + (size_t)r.splits * kBiasRows * N) *
                 sizeof(float));
    }
    return most;
}

cudaError_t linear_backward(bool bf16, const LinearArgs& a, cudaStream_t s) {
    return bf16 ? backward<__nv_bfloat16>(a, s) : backward<float>(a, s);
}

int linear_read_and_clear_fault() {
    int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_fault, sizeof(int)) != cudaSuccess) return -1;
    const int zero = 0;
    cudaMemcpyToSymbol(g_fault, &zero, sizeof(int));
    return v;
}

}  // namespace dense
}  // namespace etp
