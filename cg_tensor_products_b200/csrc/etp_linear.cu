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
//   - epilogue warps add the accumulators up in registers and apply the epilogue:
//     through a swizzled patch of shared memory per warp, so that global loads and
//     stores run along the rows.
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
constexpr int kEpiWarps = 8, kLoadWarps = 8;
constexpr int kLoaders = 32 * kLoadWarps;
constexpr int kMmaWarp = kEpiWarps + kLoadWarps;
constexpr int kThreads = 32 * (kMmaWarp + 1);
constexpr int kWaitLimit = 1 << 22;
constexpr int kRing = 4;               // accumulators in tensor memory
constexpr int kStageBytes = 32 * 32 * 4;  // epilogue patch of a warp
constexpr uint32_t kSmemMost = 232448;

__device__ int g_fault;

template <typename T>
constexpr int kParts = sizeof(T) == 4 ? 3 : 1;
// Stages that one accumulator holds.
template <typename T>
constexpr int kChunk = sizeof(T) == 4 ? 1 : 16;

// Shared memory of one instance: `stages` slots of A and B parts, the epilogue patches, barriers.
template <typename T, Product P, int BN>
struct Layout {
    static constexpr bool kAMn = P == Product::kGradW;   // A is MN-major (contraction over rows)
    static constexpr bool kBMn = P != Product::kGradX;   // B likewise
    static constexpr uint32_t kAPart = kRowsTile * kStageK * 2;
    static constexpr uint32_t kBPart = kBMn && BN < 64 ? 64u * kStageK * 2 : (uint32_t)BN * kStageK * 2;
    static constexpr uint32_t kSlot = kParts<T> * (kAPart + kBPart);
    static constexpr uint32_t kTail = kEpiWarps * kStageBytes + 256;
    static constexpr int kFit = (int)((kSmemMost - kTail) / kSlot);
    static constexpr int kSlots = kFit < 4 ? kFit : 4;
    static constexpr uint32_t kOffStage = kSlots * kSlot;
    static constexpr uint32_t kOffBars = kOffStage + kEpiWarps * kStageBytes;
    static constexpr uint32_t kBytes = kOffStage + kTail;
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
    int vec_out = 0, vec_z = 0, vec_res = 0;
    void* gW = nullptr;
    float *part = nullptr, *bias_part = nullptr;
};

__device__ __forceinline__ uint4 ldg16(const void* p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// Eight consecutive elements of a row as they lie in memory, zeros past ncols.
template <typename T>
struct Unit;
template <>
struct Unit<float> {
    uint4 a, b;
    __device__ __forceinline__ void clear() { a = b = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void load(const float* p, int left, bool vec) {
        clear();
        if (vec) {
            if (left >= 4) a = ldg16(p);
            if (left >= 8) b = ldg16(p + 4);
            return;
        }
        uint32_t v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = j < left ? __float_as_uint(__ldg(p + j)) : 0u;
        a = make_uint4(v[0], v[1], v[2], v[3]);
        b = make_uint4(v[4], v[5], v[6], v[7]);
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
    __device__ __forceinline__ void clear() { a = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void load(const __nv_bfloat16* p, int left, bool vec) {
        clear();
        if (vec) {
            if (left >= 8) a = ldg16(p);
            return;
        }
        uint32_t v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[j] = j < left ? (uint32_t)__ldg(reinterpret_cast<const unsigned short*>(p) + j) : 0u;
        a = make_uint4(v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16);
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
                for (int j = 0; j < 8; ++j) v[j] -= high_part(v[j]);
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

template <typename T>
__device__ __forceinline__ float4 load4(const T* p, int left, bool vec) {
    if constexpr (sizeof(T) == 4) {
        if (vec) return *reinterpret_cast<const float4*>(p);
    } else {
        if (vec) {
            const uint2 q = *reinterpret_cast<const uint2*>(p);
            return make_float4(bf16_lo(q.x), bf16_hi(q.x), bf16_lo(q.y), bf16_hi(q.y));
        }
    }
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    v.x = to_float(p[0]);
    if (left > 1) v.y = to_float(p[1]);
    if (left > 2) v.z = to_float(p[2]);
    if (left > 3) v.w = to_float(p[3]);
    return v;
}
template <typename T>
__device__ __forceinline__ void store4(T* p, float4 v, int left, bool vec) {
    if constexpr (sizeof(T) == 4) {
        if (vec) {
            *reinterpret_cast<float4*>(p) = v;
            return;
        }
    } else {
        if (vec) {
            *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
            return;
        }
    }
    p[0] = from_float<T>(v.x);
    if (left > 1) p[1] = from_float<T>(v.y);
    if (left > 2) p[2] = from_float<T>(v.z);
    if (left > 3) p[3] = from_float<T>(v.w);
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

// A loader's share of an operand tile of ROWS source rows by COLS columns: units of 8
// columns, unit u = t + 256 i at row u / (COLS / 8).
template <int ROWS, int COLS>
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

template <typename T, Product P, int BN>
__global__ void __launch_bounds__(kThreads, 1) etp_linear_kernel(const __grid_constant__ Job job) {
    using Lay = Layout<T, P, BN>;
    constexpr int NP = kParts<T>;
    constexpr bool kDzA = P == Product::kGradX, kDzB = P == Product::kGradW;
    // what a loader holds in flight: whole shares, or halves of them beside the pre-activation
    constexpr int kHalves = P == Product::kForward ? 1 : 2;
    using ShareA = Share<Lay::kAMn ? kStageK : kRowsTile, Lay::kAMn ? kRowsTile : kStageK>;
    using ShareB = Share<Lay::kBMn ? kStageK : BN, Lay::kBMn ? BN : kStageK>;
    constexpr int IA = ShareA::kIters, IB = ShareB::kIters;
    constexpr int HA = (IA + kHalves - 1) / kHalves, HB = (IB + kHalves - 1) / kHalves;

    extern __shared__ __align__(1024) unsigned char smem[];
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + Lay::kOffBars);
    uint64_t* empty = full + Lay::kSlots;
    uint64_t* tfull = empty + Lay::kSlots;
    uint64_t* tempty = tfull + kRing;
    uint64_t* drain = tempty + kRing;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31;

    if (warp == kMmaWarp) tc::tmem_alloc(tmem_slot, Lay::kTmemCols);
    if (t == 0) {
        for (int i = 0; i < Lay::kSlots; ++i) {
            tc::mbar_init(&full[i], kLoadWarps);
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
    // A bounded wait, the same answer for the whole warp; false: leave the loops.
    auto wait = [&](uint64_t* bar, unsigned parity) {
        const bool ok = !*abort_flag && tc::mbar_wait(bar, parity, kWaitLimit);
        if (!ok) *abort_flag = 1;
        return __all_sync(0xffffffffu, ok) != 0;
    };

    if (warp >= kEpiWarps && warp < kMmaWarp) {  // loaders
        const int lt = t - 32 * kEpiWarps;
        Unit<T> ra[HA], rb[HB], rz[kDzA ? HA : kDzB ? HB : 1];
        auto load_a = [&](const Item& it, int ks, int h) {
            const int kk = it.k0 + ks * kStageK;
            const int row0 = Lay::kAMn ? kk : it.m0, col0 = Lay::kAMn ? it.m0 : kk;
            const int rlim = Lay::kAMn ? it.k1 : job.A.nrows;
            const int c = col0 + 8 * ShareA::col(lt), left = job.A.ncols - c;
#pragma unroll
            for (int i = 0; i < HA; ++i) {
                const int r = row0 + ShareA::row(lt, h * HA + i);
                ra[i].clear();
                if (kDzA) rz[i].clear();
                if (h * HA + i < IA && r < rlim && left > 0) {
                    ra[i].load(static_cast<const T*>(job.A.rows.p) + job.A.rows.offset(job.A.map, r) + c, left, job.A.vec);
                    if (kDzA && job.silu)
                        rz[i].load(static_cast<const T*>(job.Z.rows.p) + job.Z.rows.offset(job.Z.map, r) + c, left,
                                   job.Z.vec);
                }
            }
        };
        auto load_b = [&](const Item& it, int ks, int h) {
            const int kk = it.k0 + ks * kStageK;
            const int row0 = Lay::kBMn ? kk : it.n0, col0 = Lay::kBMn ? it.n0 : kk;
            const int rlim = kDzB ? it.k1 : job.B.nrows;
            const int c = col0 + 8 * ShareB::col(lt), left = job.B.ncols - c;
#pragma unroll
            for (int i = 0; i < HB; ++i) {
                const int r = row0 + ShareB::row(lt, h * HB + i);
                rb[i].clear();
                if (kDzB) rz[i].clear();
                if (h * HB + i < IB && r < rlim && left > 0) {
                    rb[i].load(static_cast<const T*>(job.B.rows.p) + job.B.rows.offset(job.B.map, r) + c, left, job.B.vec);
                    if (kDzB && job.silu)
                        rz[i].load(static_cast<const T*>(job.Z.rows.p) + job.Z.rows.offset(job.Z.map, r) + c, left,
                                   job.Z.vec);
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
        float bsum[8];
        int i = blockIdx.x, ks = 0;
        Item it = item_of<P>(job, i, BN);
        load_a(it, 0, 0);
        load_b(it, 0, 0);
        for (int n = 0; i < job.items; ++n) {
            const int slot = n % Lay::kSlots;
            if (n >= Lay::kSlots && !wait(&empty[slot], (n / Lay::kSlots - 1) & 1)) break;
            unsigned char* sa = smem + slot * Lay::kSlot;
            unsigned char* sb = sa + NP * Lay::kAPart;
            if (kDzB && ks == 0)
#pragma unroll
                for (int j = 0; j < 8; ++j) bsum[j] = 0.f;
            // the stage after this one
            int ni = i, nks = ks + 1;
            Item nit = it;
            if (nks >= it.stages) {
                nks = 0;
                ni = i + gridDim.x;
                if (ni < job.items) nit = item_of<P>(job, ni, BN);
            }
            const bool more = ni < job.items;
#pragma unroll
            for (int h = 0; h < kHalves; ++h) {
#pragma unroll
                for (int q = 0; q < HA; ++q)
                    if (h * HA + q < IA) {
                        float v[8];
                        ra[q].get(v);
                        if (kDzA) dz(v, rz[q]);
                        store_parts<T>(sa + ShareA::offset(lt, h * HA + q), Lay::kAPart, v);
                    }
                if (h + 1 < kHalves)
                    load_a(it, ks, h + 1);
                else if (more)
                    load_a(nit, nks, 0);
#pragma unroll
                for (int q = 0; q < HB; ++q)
                    if (h * HB + q < IB) {
                        float v[8];
                        rb[q].get(v);
                        if (kDzB) {
                            dz(v, rz[q]);
#pragma unroll
                            for (int j = 0; j < 8; ++j) bsum[j] += v[j];
                        }
                        store_parts<T>(sb + ShareB::offset(lt, h * HB + q), Lay::kBPart, v);
                    }
                if (h + 1 < kHalves)
                    load_b(it, ks, h + 1);
                else if (more)
                    load_b(nit, nks, 0);
            }
            tc::fence_proxy_async();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&full[slot]);
            if (kDzB && ks + 1 >= it.stages && job.bias_part && it.m0 == 0) {
                // the item's sums of dz over its rows: the lanes of a warp that share columns, one row per warp
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    for (int o = ShareB::kPerRow; o < 32; o <<= 1) bsum[j] += __shfl_xor_sync(0xffffffffu, bsum[j], o);
                if (lane < ShareB::kPerRow) {
                    float* row = job.bias_part + (size_t)(it.split * kLoadWarps + (warp - kEpiWarps)) * job.n;
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const int c = it.n0 + 8 * ShareB::col(lt) + j;
                        if (c < job.n) row[c] = bsum[j];
                    }
                }
            }
            i = ni, ks = nks, it = nit;
        }
    } else if (warp == kMmaWarp) {
        constexpr uint32_t idesc = idesc_bf16<Lay::kAMn, Lay::kBMn>(BN);
        constexpr uint32_t kStepA = Lay::kAMn ? 2048 : 32, kStepB = Lay::kBMn ? 2048 : 32;  // 16 k
        constexpr int kPairs = NP == 3 ? 6 : 1;
        constexpr int pa[6] = {NP == 3 ? 1 : 0, 0, 2, 0, 1, 0}, pb[6] = {NP == 3 ? 1 : 0, 2, 0, 1, 0, 0};
        int n = 0, chunk = 0;
        bool ok = true;
        for (int i = blockIdx.x; i < job.items && ok; i += gridDim.x) {
            const Item it = item_of<P>(job, i, BN);
            for (int ks = 0; ks < it.stages; ++ks, ++n) {
                const int slot = n % Lay::kSlots, buf = chunk % kRing;
                const bool first = ks % kChunk<T> == 0;
                if (first && chunk >= kRing && !wait(&tempty[buf], (chunk / kRing - 1) & 1)) {
                    ok = false;
                    break;
                }
                if (!wait(&full[slot], (n / Lay::kSlots) & 1)) {
                    ok = false;
                    break;
                }
                tc::fence_after_sync();
                const int left = it.k1 - it.k0 - ks * kStageK;
                const int steps = left >= kStageK ? kStageK / 16 : (left + 15) / 16;
                const bool last = ks + 1 == it.stages || (ks + 1) % kChunk<T> == 0;
                if (lane == 0) {
                    const uint32_t sa = tc::smem_u32(smem + slot * Lay::kSlot), sb = sa + NP * Lay::kAPart;
#pragma unroll
                    for (int q = 0; q < kPairs; ++q)
                        for (int s = 0; s < steps; ++s)
                            mma_bf16(tmem + buf * BN, desc128<Lay::kAMn>(sa + pa[q] * Lay::kAPart + s * kStepA),
                                     desc128<Lay::kBMn>(sb + pb[q] * Lay::kBPart + s * kStepB), idesc,
                                     first && q == 0 && s == 0 ? 0u : 1u);
                    tc::mma_commit(&empty[slot]);
                    if (last) tc::mma_commit(&tfull[buf]);
                }
                __syncwarp();
                if (last) ++chunk;
            }
        }
    } else {  // epilogue
        constexpr int NC = BN / 2;                  // columns of a warp
        constexpr int CW = NC < 32 ? NC : 32;       // columns at a time
        constexpr int LPR = CW / 4, RPI = 32 / LPR;  // lanes per row, rows per pass
        const int quad = warp & 3, half = warp >> 2;
        float* st = reinterpret_cast<float*>(smem + Lay::kOffStage + warp * kStageBytes);
        const uint32_t lane_base = tmem + ((uint32_t)(quad * 32) << 16) + half * NC;
        auto swz = [](int row, int j) { return LPR == 8 ? (j ^ (row & 7)) : (j ^ ((row >> 1) & 3)); };
        int chunk = 0;
        bool ok = true;
        for (int i = blockIdx.x; i < job.items && ok; i += gridDim.x) {
            const Item it = item_of<P>(job, i, BN);
            float acc[NC];
#pragma unroll
            for (int c = 0; c < NC; ++c) acc[c] = 0.f;
            for (int ks = 0; ks < it.stages; ks += kChunk<T>, ++chunk) {
                const int buf = chunk % kRing;
                if (!wait(&tfull[buf], (chunk / kRing) & 1)) {
                    ok = false;
                    break;
                }
                tc::fence_after_sync();
#pragma unroll
                for (int c = 0; c < NC; c += 16) {
                    float v[16];
                    tc::tmem_ld<16>(lane_base + buf * BN + c, v);
                    tc::tmem_wait_ld(v);
#pragma unroll
                    for (int j = 0; j < 16; ++j) acc[c + j] += v[j];
                }
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&tempty[buf]);
            }
            if (!ok) break;
#pragma unroll
            for (int c = 0; c < NC; c += CW) {
#pragma unroll
                for (int j = 0; j < LPR; ++j)
                    *reinterpret_cast<float4*>(st + lane * CW + 4 * swz(lane, j)) =
                        make_float4(acc[c + 4 * j], acc[c + 4 * j + 1], acc[c + 4 * j + 2], acc[c + 4 * j + 3]);
                __syncwarp();
                const int jj = lane % LPR;
                const int n = it.n0 + half * NC + c + 4 * jj, left = job.n - n;
                float4 bias = make_float4(0.f, 0.f, 0.f, 0.f);
                if (P == Product::kForward && job.bias && left > 0)
                    bias = load4(static_cast<const T*>(job.bias) + n, left, false);
#pragma unroll
                for (int rr = 0; rr < LPR; ++rr) {
                    const int row = RPI * rr + lane / LPR, m = it.m0 + quad * 32 + row;
                    if (m >= job.m || left <= 0) continue;
                    float4 v = *reinterpret_cast<const float4*>(st + row * CW + 4 * swz(row, jj));
                    if (P == Product::kForward) {
                        v.x += bias.x, v.y += bias.y, v.z += bias.z, v.w += bias.w;
                        if (job.z.p)
                            store4(static_cast<T*>(job.z.p) + job.z.offset(job.map, m) + n, v, left, job.vec_z);
                        if (job.silu) v.x = silu(v.x), v.y = silu(v.y), v.z = silu(v.z), v.w = silu(v.w);
                        if (job.residual.p) {
                            const float4 r = load4(
                                static_cast<const T*>(job.residual.p) + job.residual.offset(job.map, m) + n, left,
                                job.vec_res);
                            v.x += r.x, v.y += r.y, v.z += r.z, v.w += r.w;
                        }
                    }
                    if (P != Product::kGradW) {
                        store4(static_cast<T*>(job.out.p) + job.out.offset(job.map, m) + n, v, left, job.vec_out);
                    } else if (job.part) {
                        store4(job.part + ((size_t)it.split * job.m + m) * job.n + n, v, left, job.vec_out);
                    } else {
                        store4(static_cast<T*>(job.gW) + (size_t)m * job.n + n, v, left, job.vec_out);
                    }
                }
                __syncwarp();
            }
        }
    }
    __syncthreads();
    if (*abort_flag) {  // leave no MMA in flight on the freed memory
        if (t == 32 * kMmaWarp) {
            atomicOr(&g_fault, 1);
            tc::mma_commit(drain);
            tc::mbar_wait(drain, 0, kWaitLimit);
        }
        __syncthreads();
    }
    tc::fence_before_sync();
    __syncthreads();
    if (warp == kMmaWarp) tc::tmem_dealloc(tmem, Lay::kTmemCols);
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
    const long long n = bytes / elem;
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
    r.p = const_cast<void*>(p), r.gs = ncols;
    RowMap map;
    map.M = nrows;
    return operand(r, map, nrows, ncols, elem);
}

template <typename T, Product P, int BN>
cudaError_t launch_bn(Job& j, cudaStream_t s) {
    using Lay = Layout<T, P, BN>;
    const cudaError_t e = cudaFuncSetAttribute(etp_linear_kernel<T, P, BN>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)Lay::kBytes);
    if (e != cudaSuccess) return e;
    const int sms = sm_count();
    etp_linear_kernel<T, P, BN><<<j.items < sms ? j.items : sms, kThreads, Lay::kBytes, s>>>(j);
    return cudaGetLastError();
}

// Columns of a tile: the widest that still gives every SM a tile, or the narrowest.
int tile_cols(int M, int N) {
    const long long mt = (M + kRowsTile - 1) / kRowsTile;
    const int sms = sm_count();
    if (N > 64 && mt * ((N + 127) / 128) >= sms) return 128;
    if (N > 32 && mt * ((N + 63) / 64) >= sms) return 64;
    return 32;
}

template <typename T, Product P>
cudaError_t launch(Job& j, int bn, int splits, cudaStream_t s) {
    j.ntn = (j.n + bn - 1) / bn;
    const long long tiles = (long long)((j.m + kRowsTile - 1) / kRowsTile) * j.ntn;
    if (tiles > 0x7fff0000LL) return cudaErrorInvalidValue;
    j.tiles = j.items = (int)tiles;
    if (P == Product::kGradW) {  // a tile of no rows still is one tile
        if (j.m == 0) j.tiles = j.ntn;
        j.items = j.tiles * splits;
    }
    switch (bn) {
        case 128: return launch_bn<T, P, 128>(j, s);
        case 64: return launch_bn<T, P, 64>(j, s);
        default: return launch_bn<T, P, 32>(j, s);
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
    const bool n4 = a.N % 4 == 0;
    j.vec_out = n4 && rows_aligned(a.out, elem, 4 * elem);
    j.vec_z = n4 && rows_aligned(a.z, elem, 4 * elem);
    j.vec_res = n4 && rows_aligned(a.residual, elem, 4 * elem);
    return launch<T, Product::kForward>(j, tile_cols(j.m, j.n), 1, s);
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
        j.vec_out = a.K % 4 == 0 && rows_aligned(a.gx, elem, 4 * elem);
        const cudaError_t e = launch<T, Product::kGradX>(j, tile_cols(j.m, j.n), 1, s);
        if (e != cudaSuccess) return e;
    }
    if (!a.gW && !a.gbias) return cudaSuccess;
    // without grad_W the tile has no rows: only the loaders' sums of dz are wanted
    const int K = a.gW ? a.K : 0;
    const Ranges r = ranges(a.map.M, a.gW ? a.K : 1, a.N);
    const bool join = r.splits != 1;
    float* bias_part = a.gbias ? a.ws : nullptr;
    float* part = a.ws + (size_t)r.splits * kLoadWarps * a.N;
    if (r.splits > 0) {
        Job j;
        j.A = operand(a.x, a.map, a.map.M, K, elem);
        j.B = operand(a.g, a.map, a.map.M, a.N, elem);
        if (a.silu) j.Z = operand(a.z, a.map, a.map.M, a.N, elem);
        j.silu = a.silu;
        j.m = K, j.n = a.N, j.k = a.map.M;
        j.range = r.range;
        j.gW = a.gW;
        j.part = join && a.gW ? part : nullptr;
        j.bias_part = bias_part;
        j.vec_out = a.N % 4 == 0 && (j.part ? (reinterpret_cast<uintptr_t>(part) % 16) == 0
                                            : (reinterpret_cast<uintptr_t>(a.gW) % (4 * elem)) == 0);
        const cudaError_t e = launch<T, Product::kGradW>(j, r.bn, r.splits, s);
        if (e != cudaSuccess) return e;
    }
    const size_t count = a.gW && join ? (size_t)a.K * a.N : 0;
    const int blocks_w = (int)((count + 31) / 32), blocks_b = a.gbias ? (a.N + 31) / 32 : 0;
    if (blocks_w + blocks_b == 0) return cudaSuccess;
    etp_linear_join_kernel<T><<<blocks_w + blocks_b, 256, 0, s>>>(part, r.splits, count, static_cast<T*>(a.gW),
                                                                  bias_part, r.splits * kLoadWarps, a.N,
                                                                  static_cast<T*>(a.gbias), blocks_w);
    return cudaGetLastError();
}

}  // namespace

cudaError_t linear_forward(bool bf16, const LinearArgs& a, cudaStream_t s) {
    if (a.map.M == 0) return cudaSuccess;
    return bf16 ? forward<__nv_bfloat16>(a, s) : forward<float>(a, s);
}

size_t linear_workspace_bytes(int M, int K, int N) {
    const Ranges r = ranges(M, K, N), b = ranges(M, 1, N);  // grad_bias alone takes the second
    const size_t sums = r.splits > 1 ? (size_t)r.splits * K * N : 0;
    const int most = r.splits > b.splits ? r.splits : b.splits;
    return (sums + (size_t)most * kLoadWarps * N) * sizeof(float);
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
