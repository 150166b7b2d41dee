// Linear layers with a fused epilogue, and their VJP, on the tensor cores (tcgen05).
//
//   forward   z = x W + bias, out = act(z) + residual
//   backward  dz = g act'(z);  grad_x = dz W^T;  grad_W = x^T dz;  grad_bias = sum of dz over the rows
//
// Each of the three products is D[m][n] = sum_k A[m][k] B[k][n] in tiles of 128 x BN
// outputs, 32 or 64 k per stage. One persistent CTA per SM:
//   - loader warps bring a stage's elements into shared memory by asynchronous copies, a
//     few stages ahead, form dz where it is an operand, and hand over bfloat16 operands.
//     A that has to be converted goes to tensor memory (lane = m), where the tensor core
//     reads it without using shared memory's bandwidth, which bounds these kernels: a
//     128 x 128 x 16 product reads 4 KB of B in its 64 cycles, with A in shared memory
//     too all that there is. For grad_W the lane is a column of x, so its transposition
//     is in the reading. B, and a bfloat16 A that is used as it is, lie in shared memory
//     in the swizzled layouts of the tensor core: an operand whose contraction index is
//     contiguous in memory K-major, one whose other index is contiguous MN-major;
//   - W is converted ahead once where many row tiles share it, and its tiles arrive by
//     bulk copies;
//   - one warp issues the MMAs into a ring of accumulators in tensor memory;
//   - epilogue warps add the accumulators up in registers and apply the epilogue.
// Float32 operands are split into three bfloat16 parts x = x0 + x1 + x2 of 8 bits, and a
// product is the sum of the six part products x0 w0, x0 w1, x1 w0, x1 w1, x0 w2, x2 w0.
// x0 is x truncated (rounding would turn the largest floats into infinities), x1 the rest
// rounded, x2 what is left. For x in [1, 2): x1 <= 2^-7, |x2| <= 2^-16 and a multiple of
// 2^-23, so the three are exact, and what is left out, x1 w2 + x2 w1 + x2 w2, is below 2^-22
// of the product and of either sign (with x1 truncated: up to 2^-21 and always towards
// zero). Exact holds from |x| = 2^-110 up; below it x2 ends at bfloat16's smallest
// subnormal, and the parts are within 2^-133 of x. The six are as many
// MMAs as three TF32 products, at twice the mantissa of the smallest terms kept and in
// three quarters of the space, and both layouts are available to 16-bit types.
// The tensor core truncates when it adds to its accumulator; so a float32 stage starts
// a new accumulator, adds the small products first and the x0 w0 ones last (up to four
// truncated additions of full size), and stages are added up in registers, rounded to
// nearest. bfloat16 operands are one part. dz of a bfloat16 layer with an activation is not
// a bfloat16 value: it enters as two rounded parts, its upper 16 bits (one part alone, 2^-8
// of each dz, takes grad_x from 58.7 to 56.3 us at 131072 x 256 -> 256 and lifts the
// gradients' error from 1.65e-3, that of storing them, to 2.35e-3). A bfloat16
// accumulator holds a whole tile: up to 2^16 k in 4096 truncated additions (8192 with dz's
// low part), each 2^-24 of the sum on average, stay below an eighth of the result's own
// rounding.
//
// grad_W contracts over the rows: the rows are cut into as many ranges as leave every
// SM one, each range's sums go to the workspace, and a second launch adds them up in
// range order. grad_bias is summed by the loaders of dz on the way.
#include <atomic>

#include "etp_dense.cuh"
#include "etp_tcgen05.cuh"

namespace etp {
namespace dense {
namespace {

enum class Product { kForward, kGradX, kGradW };

constexpr int kRowsTile = 128;
constexpr int kRangeK = 64;  // ranges of rows are whole multiples of it
// Warps: the epilogue's (a quarter of the rows each, by a half or a quarter of the
// columns), the loaders, one for the MMAs. The float32 forward's epilogue has most to do
// and its loaders least; the backward products have dz to compute in the loaders.
template <typename T, Product P>
struct Warps {
    static constexpr int kEpi = P == Product::kForward && sizeof(T) == 4 ? 16 : 8;
    static constexpr int kLoad = P == Product::kForward ? (sizeof(T) == 4 ? 4 : 8) : sizeof(T) == 4 ? 8 : 16;
    static constexpr int kMma = kEpi + kLoad;
    static constexpr int kThreads = 32 * (kMma + 1);
    static constexpr int kLoaders = 32 * kLoad;
};
constexpr int kBiasRows = 16;  // most partial sums of dz per range: one per loader warp
constexpr int kWaitLimit = 1 << 22;
// Accumulators in tensor memory. One of 256 columns: the loaders' stages ahead cover its epilogue.
template <int COLS>
constexpr int kRingOf = COLS == 256 ? 1 : 2;
constexpr uint32_t kSmemMost = 232448;

__device__ int g_fault;

template <int V>
struct Int {
    static constexpr int value = V;
};

// bfloat16 parts of an operand: three of a float32 one, two of the dz of bfloat16 layers
// (computed in float32; two parts are within 2^-17 of it, one within 2^-8), one of the rest.
template <typename T, Product P>
constexpr int kPartsA = sizeof(T) == 4 ? 3 : P == Product::kGradX ? 2 : 1;
template <typename T, Product P>
constexpr int kPartsB = sizeof(T) == 4 ? 3 : P == Product::kGradW ? 2 : 1;
// k of a stage. grad_W's float32 stages are half as long: they hold three operands.
template <typename T, Product P>
constexpr int kStageK = sizeof(T) == 4 && P == Product::kGradW ? 32 : 64;
// Stages that one accumulator holds: one of float32, a whole item's of bfloat16.
template <typename T>
constexpr int kChunk = sizeof(T) == 4 ? 1 : 1 << 20;
constexpr int kMostRange = 1 << 16;  // rows of a range: bounds the truncations of a bfloat16 accumulator

// Swizzled bf16 operand layouts in shared memory: rows of 128 bytes, the 16-byte chunk
// index XORed with the row mod 8. MN-major: rows are k, 64 m (n) across; groups of 8 k
// 1024 bytes apart (SBO), panels of 64 m (n) K * 128 bytes apart (LBO). K-major: rows are
// m (n), 64 k across, groups of 8 rows 1024 bytes apart.
template <bool MN, int K>
__device__ __forceinline__ uint64_t operand_desc(uint32_t saddr) {
    static_assert(MN || K == 64, "K-major rows of 128 bytes");
    constexpr uint64_t lbo = MN ? (K * 128 >> 4) : 1, sbo = 1024 >> 4;
    return (uint64_t)((saddr >> 4) & 0x3FFFu) | (lbo << 16) | (sbo << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
// Byte offset of the 16-byte chunk c of source row r in an operand part.
template <int K>
__host__ __device__ constexpr uint32_t chunk_offset(int r, int c) {
    return (uint32_t)(c >> 3) * (K * 128) + (uint32_t)(r >> 3) * 1024 + (uint32_t)(r & 7) * 128 +
           (uint32_t)(((c & 7) ^ (r & 7)) << 4);
}

// A loader's share of an operand tile of ROWS source rows by COLS columns: units of 8
// columns, unit u = t + THREADS i at row u / (COLS / 8).
template <int ROWS, int COLS, int K, int THREADS>
struct Share {
    static constexpr int kPerRow = COLS / 8;
    static constexpr int kIters = (ROWS * kPerRow + THREADS - 1) / THREADS;
    static constexpr bool kEven = ROWS * kPerRow % THREADS == 0;  // or the last threads have none
    static __device__ __forceinline__ int row(int t, int i) { return (t + THREADS * i) / kPerRow; }
    static __device__ __forceinline__ int col(int t) { return t % kPerRow; }
    static __device__ __forceinline__ bool has(int t, int i) { return kEven || t + THREADS * i < ROWS * kPerRow; }
    static __device__ __forceinline__ uint32_t offset(int t, int i) { return chunk_offset<K>(row(t, i), col(t)); }
};

// The tile shapes and memory of one instance. VEC: the operands' rows move in 16-byte
// groups. IMAGE: B arrives as ready tiles. MT: tiles of 128 m that share a stage's B.
template <typename T, Product P, int BN, bool VEC, bool IMAGE, int MT = 1>
struct Layout {
    using W = Warps<T, P>;
    static constexpr int kK = kStageK<T, P>;
    static constexpr bool kAMn = P == Product::kGradW;  // A is MN-major (contraction over rows)
    static constexpr bool kBMn = P != Product::kGradX;  // B likewise
    static constexpr bool kDzA = P == Product::kGradX, kDzB = P == Product::kGradW;
    static constexpr bool kTmemA = sizeof(T) == 4 || kDzA;  // A is converted
    static constexpr bool kConvB = !IMAGE && (sizeof(T) == 4 || kDzB);  // B is converted here
    static constexpr bool kCopyB = !IMAGE && !kConvB;                   // or used as it is
    using ShareA = Share<kAMn ? kK : kRowsTile, kAMn ? kRowsTile * MT : kK, kK, W::kLoaders>;
    static_assert(MT == 1 || (kAMn && !kTmemA), "tall tiles");
    using ShareB = Share<kBMn ? kK : BN, kBMn ? BN : kK, kK, W::kLoaders>;
    // A slot: B's parts and an A that is used as it is; a converted A's parts have columns in tensor memory
    static constexpr uint32_t kAPart = kTmemA ? 0 : MT * kRowsTile * kK * 2;
    static constexpr uint32_t kBPart = (kBMn && BN < 64 ? 64u : (uint32_t)BN) * kK * 2;
    static constexpr int kPA = kPartsA<T, P>, kPB = kPartsB<T, P>;
    static constexpr uint32_t kSlot = kPB * kBPart + kAPart;
    static constexpr uint32_t kACols = kTmemA ? kPA * kK / 2 : 0;
    // Elements on their way, per stage: of A, of the pre-activation beside dz, of B
    static constexpr uint32_t kRawA = kTmemA ? kRowsTile * kK * sizeof(T) : 0;
    static constexpr uint32_t kRawB = kConvB ? ShareB::kIters * W::kLoaders * 8 * sizeof(T) : 0;
    static constexpr uint32_t kRawZ = kDzA ? kRawA : kDzB ? kRawB : 0;
    static constexpr uint32_t kRaw = kRawA + kRawZ + kRawB;
    static constexpr int kAcc = MT * BN, kRing = kRingOf<kAcc>;  // columns of an accumulator, accumulators
    static constexpr uint32_t kTail = 256;  // barriers
    static constexpr int kWant = 3;         // slots, where there is room
    static constexpr int kTmemSlots = kACols ? (int)((512 - kRing * kAcc) / kACols) : 8;
    static constexpr int kSome = 2 + (kSlot <= 32768 || sizeof(T) == 2);
    static constexpr int kFew = kTmemSlots < kSome ? kTmemSlots : kSome;
    // Stages in flight. Copies straight into a slot share their groups, and the slot's hand-over lags behind by
    // as many; without other elements on their way they use the slots themselves.
    // grad_W of bfloat16 has large slots (two parts of dz): one stage ahead and three slots are fastest (131072 x 128 ->
    // 128 38 us, with four slots 44 us, two stages ahead 48 us; 256 -> 256 with stages of half the length 83 us, 67 us so).
    static constexpr bool kBig = kDzB && sizeof(T) == 2;
    static constexpr int kMost = kBig ? 1 : !kTmemA || kCopyB ? kFew - 1 : 3;
    static constexpr int kRoom = kRaw ? (int)((kSmemMost - kTail - kFew * kSlot) / kRaw) : 1;
    static constexpr int kDepth = kRoom < kMost ? kRoom : kMost;
    static constexpr int kFit = (int)((kSmemMost - kTail - kDepth * kRaw) / kSlot);
    static constexpr int kMostSlots = kBig ? kWant : kRaw ? kWant + 1 : 6;
    static constexpr int kCap = kTmemSlots < kMostSlots ? kTmemSlots : kMostSlots;
    static constexpr int kSlots = kFit < kCap ? kFit : kCap;
    static constexpr int kLag = kTmemA && !kCopyB ? 0 : kRaw ? kDepth : kSlots / 2;  // the rest: ready for the MMAs
    static constexpr uint32_t kOffRaw = kSlots * kSlot;
    static constexpr uint32_t kOffBars = kOffRaw + kDepth * kRaw;
    static constexpr uint32_t kBytes = kOffBars + kTail;
    static constexpr uint32_t kTmemCols = kRing * kAcc + kSlots * kACols <= 128   ? 128
                                          : kRing * kAcc + kSlots * kACols <= 256 ? 256
                                                                                : 512;
    static_assert(kSlots >= 2 && kDepth >= 1 && kLag < kSlots && kBytes <= kSmemMost, "linear layer memory");
    static_assert(kRing * kAcc + kSlots * kACols <= 512, "linear layer tensor memory");
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
    FastDiv ntn;              // tiles along n
    int items = 1;            // work items
    FastDiv tiles;            // grad_W: tiles of the output
    int range = 0;            // and rows per range
    RowMap map;               // rows of the output operands
    Rows out, z, residual;
    const void* bias = nullptr;
    int vec_out = 0;  // the epilogue's operands move 1 (0), 2 (1) or 4 (2) elements at a time
    void* gW = nullptr;
    float *part = nullptr, *bias_part = nullptr;
    const unsigned char* image = nullptr;  // B as tiles of operand parts, or null
};

// Asynchronous copies into shared memory, zeros where `on` is false.
__device__ __forceinline__ void copy16(void* dst, const void* src, bool on) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(tc::smem_u32(dst)), "l"(src), "r"(on ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void copy4(void* dst, const void* src, bool on) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(tc::smem_u32(dst)), "l"(src), "r"(on ? 4 : 0)
                 : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// 16 bytes of a row of which `left` elements remain: one copy, or element by element where
// rows are not aligned (float32 still asynchronously; bfloat16 elements are narrower than
// the narrowest asynchronous copy and pass through registers).
template <typename T, bool VEC>
__device__ __forceinline__ void copy_chunk(unsigned char* dst, const T* p, int left) {
    if constexpr (VEC) {
        copy16(dst, p, left > 0);
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int j = 0; j < 4; ++j) copy4(dst + 4 * j, p + j, left > j);
    } else {
        uint32_t v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            asm volatile(
                "{\n .reg .pred pp;\n .reg .u16 h;\n setp.ne.b32 pp, %2, 0;\n mov.u16 h, 0;\n"
                " @pp ld.global.nc.u16 h, [%1];\n cvt.u32.u16 %0, h;\n}"
                : "=&r"(v[j])
                : "l"(p + j), "r"((int)(left > j)));
        *reinterpret_cast<uint4*>(dst) =
            make_uint4(v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16);
    }
}

// Copies of one operand tile: `n` chunks a lane, chunk i (DR i) rows below the lane's
// first and in the same columns. On one row stride that is a fixed distance in memory.
template <typename T, bool VEC, int N, int DR, typename Dst>
__device__ __forceinline__ void copy_column(const Operand& o, int r0, int rlim, int c, Dst&& dst) {
    const int left = o.ncols - c;
    if (o.map.per.d == 1) {
        const T* p = static_cast<const T*>(o.rows.p) + (unsigned long long)(unsigned)r0 * o.rows.gs + c;
#pragma unroll
        for (int i = 0; i < N; ++i)
            copy_chunk<T, VEC>(dst(i), p + (unsigned long long)(DR * i) * o.rows.gs, r0 + DR * i < rlim ? left : 0);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int r = r0 + DR * i;
            copy_chunk<T, VEC>(dst(i), static_cast<const T*>(o.rows.p) + o.rows.offset(o.map, r) + c,
                               r < rlim ? left : 0);
        }
    }
}

// 16 bytes of shared memory as floats.
template <typename T>
__device__ __forceinline__ void read16(const unsigned char* p, float* v) {
    const uint4 q = *reinterpret_cast<const uint4*>(p);
    if constexpr (sizeof(T) == 4) {
        v[0] = __uint_as_float(q.x), v[1] = __uint_as_float(q.y), v[2] = __uint_as_float(q.z), v[3] = __uint_as_float(q.w);
    } else {
        v[0] = bf16_lo(q.x), v[1] = bf16_hi(q.x), v[2] = bf16_lo(q.y), v[3] = bf16_hi(q.y);
        v[4] = bf16_lo(q.z), v[5] = bf16_hi(q.z), v[6] = bf16_lo(q.w), v[7] = bf16_hi(q.w);
    }
}

// High halves of two floats as a bf16 pair (truncation).
__device__ __forceinline__ uint32_t high_pair(float a, float b) {
    return __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
}

// The parts of N floats, part after part, as bf16 pairs: emit(p, pairs). NP rounded parts,
// each of what is left by those before it; a float32 operand's first is truncated, and its
// last has nothing to round.
template <typename T, int NP, int N, typename Emit>
__device__ __forceinline__ void split_parts(float (&v)[N], Emit&& emit) {
    uint32_t w[N / 2];
#pragma unroll
    for (int p = 0; p < NP; ++p) {
#pragma unroll
        for (int j = 0; j < N; j += 2)
            w[j / 2] = sizeof(T) == 4 && p != 1 ? high_pair(v[j], v[j + 1]) : pack_bf16(v[j], v[j + 1]);
        emit(p, w);
        if (p + 1 < NP)
#pragma unroll
            for (int j = 0; j < N; j += 2) {  // packed: v - part, exact
                const float2 r = __ffma2_rn(make_float2(bf16_lo(w[j / 2]), bf16_hi(w[j / 2])), make_float2(-1.f, -1.f),
                                            make_float2(v[j], v[j + 1]));
                v[j] = r.x, v[j + 1] = r.y;
            }
    }
}
template <typename T, int NP>
__device__ __forceinline__ void store_parts(unsigned char* dst, uint32_t part, float (&v)[8], bool low = true) {
    split_parts<T, NP, 8>(v, [&](int p, const uint32_t(&w)[4]) {
        if (p == 0 || low) *reinterpret_cast<uint4*>(dst + p * part) = make_uint4(w[0], w[1], w[2], w[3]);
    });
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
__device__ __forceinline__ void mma_bf16_ta(uint32_t d, uint32_t a, uint64_t db, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n .reg .pred pp;\n setp.ne.b32 pp, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, pp;\n}" ::"r"(d),
        "r"(a), "l"(db), "r"(idesc), "r"(acc)
        : "memory");
}

// How an epilogue moves two elements of a row: whole pairs inside a tile that has all its
// rows (at one stride) and columns, whole pairs under a predicate (an even number of columns), or single
// elements. Zeros are read past the `left` that remain. The predicated statements are
// volatile, so that they stay in order: a residual that is the output is read before it
// is written.
enum class Pairs { kFull, kEven, kAny };
template <Pairs V>
__device__ __forceinline__ float2 load2(const float* p, int left) {
    float a, b;
    if constexpr (V == Pairs::kFull) return *reinterpret_cast<const float2*>(p);
    if constexpr (V == Pairs::kEven)
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
template <Pairs V>
__device__ __forceinline__ float2 load2(const __nv_bfloat16* p, int left) {
    uint32_t a;
    if constexpr (V == Pairs::kFull)
        a = *reinterpret_cast<const uint32_t*>(p);
    else if constexpr (V == Pairs::kEven)
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
template <Pairs V>
__device__ __forceinline__ void store2(float* p, float2 v, int left) {
    if constexpr (V == Pairs::kFull)
        *reinterpret_cast<float2*>(p) = v;
    else if constexpr (V == Pairs::kEven)
        asm volatile("{\n .reg .pred pp;\n setp.gt.s32 pp, %3, 0;\n @pp st.global.v2.f32 [%0], {%1, %2};\n}" ::"l"(p),
                     "f"(v.x), "f"(v.y), "r"(left));
    else
        asm volatile("{\n .reg .pred p0, p1;\n setp.gt.s32 p0, %3, 0;\n setp.gt.s32 p1, %3, 1;\n"
                     " @p0 st.global.f32 [%0], %1;\n @p1 st.global.f32 [%0+4], %2;\n}" ::"l"(p),
                     "f"(v.x), "f"(v.y), "r"(left));
}
template <Pairs V>
__device__ __forceinline__ void store2(__nv_bfloat16* p, float2 v, int left) {
    const uint32_t a = pack_bf16(v.x, v.y);
    if constexpr (V == Pairs::kFull)
        *reinterpret_cast<uint32_t*>(p) = a;
    else if constexpr (V == Pairs::kEven)
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
template <typename T, Product P, int MT>
__device__ __forceinline__ Item item_of(const Job& j, int i, int bn) {
    Item it;
    int tile = i;
    it.split = 0, it.k0 = 0, it.k1 = j.k;
    if (P == Product::kGradW) {
        it.split = (int)j.tiles.quot(i);
        tile = i - it.split * j.tiles.d;
        it.k0 = it.split * j.range;
        it.k1 = j.k - it.k0 < j.range ? j.k : it.k0 + j.range;  // k0 + range may pass 2^31
    }
    const int mt = (int)j.ntn.quot(tile);
    it.m0 = mt * kRowsTile * MT;
    it.n0 = (tile - mt * j.ntn.d) * bn;
    it.stages = (it.k1 - it.k0 + kStageK<T, P> - 1) / kStageK<T, P>;
    return it;
}

// The epilogue of a tile on one warp's 32 rows x COLS columns, in the accumulator's
// fragment layout: a lane holds 4 rows, of each 2 neighbouring columns in every 8. The 4
// lanes of a row make whole 32-byte sectors of float32, so loads and stores go straight
// between registers and memory.
template <Pairs V>
__device__ __forceinline__ unsigned long long row_offset(const Job& job, const Rows& r, int m) {
    return V == Pairs::kFull ? (unsigned long long)(unsigned)m * r.gs : r.offset(job.map, m);
}
// bfloat16 pairs of a row's groups c, c + 1 (16 columns, one sector): traded between the
// row's 4 lanes so that each stores 4 neighbouring columns and the sector is written whole
// (grad_x: 131072 x 256 bf16 66 -> 58 us; the forward's longer epilogue loses by it, 112 -> 171 us
// at 166517 x 512).
template <int G>
__device__ __forceinline__ void store_quads(__nv_bfloat16* row, const float2 (&v)[G], int lane) {
    const int q = lane & 3, src = (lane & ~3) + 2 * (q & 1);
#pragma unroll
    for (int c = 0; c < G; c += 2) {
        const uint32_t a = pack_bf16(v[c].x, v[c].y), b = pack_bf16(v[c + 1].x, v[c + 1].y);
        const uint32_t a0 = __shfl_sync(0xffffffffu, a, src), b0 = __shfl_sync(0xffffffffu, b, src);
        const uint32_t a1 = __shfl_sync(0xffffffffu, a, src + 1), b1 = __shfl_sync(0xffffffffu, b, src + 1);
        *reinterpret_cast<uint2*>(row + 8 * c + 4 * q) = make_uint2(q < 2 ? a0 : b0, q < 2 ? a1 : b1);
    }
}
template <typename T, Product P, int COLS, Pairs V>
__device__ __forceinline__ void finish(const Job& job, const Item& it, float (&acc)[2][COLS / 2],
                                       int quad, int n0, int lane) {
    constexpr int kGroups = COLS / 8 < 4 ? COLS / 8 : 4;  // groups of 8 columns at a time
    const bool has_res = P == Product::kForward && job.residual.p != nullptr;
#pragma unroll
    for (int g = 0; g < COLS / 8; g += kGroups) {
        const int n = it.n0 + n0 + 8 * g + 2 * (lane & 3);
        float2 bias[kGroups];
        if constexpr (P == Product::kForward) {
#pragma unroll
            for (int c = 0; c < kGroups; ++c) {
                bias[c] = make_float2(0.f, 0.f);
                if (job.bias) bias[c] = load2<V>(static_cast<const T*>(job.bias) + n + 8 * c, job.n - n - 8 * c);
            }
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {  // a row at a time: two spill, which costs more than their overlap gives
            const int m = it.m0 + quad * 32 + 8 * r + (lane >> 2);
            const int left = V == Pairs::kFull || m < job.m ? job.n - n : 0;
            float2 res[kGroups];
            if (has_res) {
                const T* p = static_cast<const T*>(job.residual.p) + row_offset<V>(job, job.residual, m) + n;
#pragma unroll
                for (int c = 0; c < kGroups; ++c) res[c] = load2<V>(p + 8 * c, left - 8 * c);
            }
            float2 v[kGroups];
#pragma unroll
            for (int c = 0; c < kGroups; ++c)
                v[c] = make_float2(acc[r >> 1][4 * (g + c) + 2 * (r & 1)], acc[r >> 1][4 * (g + c) + 2 * (r & 1) + 1]);
            if constexpr (P == Product::kForward) {
#pragma unroll
                for (int c = 0; c < kGroups; ++c) v[c].x += bias[c].x, v[c].y += bias[c].y;
                if (job.z.p) {
                    T* p = static_cast<T*>(job.z.p) + row_offset<V>(job, job.z, m) + n;
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
            if constexpr (sizeof(T) == 2 && V == Pairs::kFull && P == Product::kGradX && kGroups % 2 == 0) {
                store_quads<kGroups>(static_cast<T*>(job.out.p) + row_offset<V>(job, job.out, m) + n - 2 * (lane & 3), v,
                                     lane);
            } else if (P == Product::kGradW && job.part) {
                float* p = job.part + ((size_t)it.split * job.m + m) * job.n + n;
#pragma unroll
                for (int c = 0; c < kGroups; ++c) store2<V>(p + 8 * c, v[c], left - 8 * c);
            } else {
                T* p = P == Product::kGradW ? static_cast<T*>(job.gW) + (size_t)m * job.n + n
                                            : static_cast<T*>(job.out.p) + row_offset<V>(job, job.out, m) + n;
#pragma unroll
                for (int c = 0; c < kGroups; ++c) store2<V>(p + 8 * c, v[c], left - 8 * c);
            }
        }
    }
}

template <typename T, Product P, int BN, bool VEC, bool IMAGE, int MT = 1>
__global__ void __launch_bounds__(Warps<T, P>::kThreads, 1) etp_linear_kernel(const __grid_constant__ Job job) {
    using Lay = Layout<T, P, BN, VEC, IMAGE, MT>;
    using W = Warps<T, P>;
    using ShareA = typename Lay::ShareA;
    using ShareB = typename Lay::ShareB;
    constexpr int K = Lay::kK, kSlots = Lay::kSlots, kRing = Lay::kRing;
    constexpr bool kDzA = Lay::kDzA, kDzB = Lay::kDzB;

    extern __shared__ __align__(1024) unsigned char smem[];
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + Lay::kOffBars);  // a slot's operands are written
    uint64_t* bfull = full + kSlots;                                      // its image tile has arrived
    uint64_t* empty = bfull + kSlots;                                     // its MMAs are done
    uint64_t* tfull = empty + kSlots;                                     // an accumulator is complete
    uint64_t* tempty = tfull + kRing;                                     // and has been read
    uint64_t* drain = tempty + kRing;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31;

    if (warp == W::kMma) tc::tmem_alloc(tmem_slot, Lay::kTmemCols);
    if (t == 0) {
        for (int i = 0; i < kSlots; ++i) {
            tc::mbar_init(&full[i], W::kLoad);
            tc::mbar_init(&bfull[i], 1);
            tc::mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < kRing; ++i) {
            tc::mbar_init(&tfull[i], 1);
            tc::mbar_init(&tempty[i], W::kEpi);
        }
        tc::mbar_init(drain, 1);
        *abort_flag = 0;
        tc::mbar_fence_init();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    const uint32_t tmem_a = tmem + kRing * Lay::kAcc;  // converted A: per slot, part after part
    // A bounded wait; false: leave the loops. wait(): the same answer for the whole warp.
    auto wait1 = [&](uint64_t* bar, unsigned parity) {
        if (tc::mbar_wait(bar, parity, 1)) return true;  // mostly it is there
        const bool ok = !*abort_flag && tc::mbar_wait(bar, parity, kWaitLimit);
        if (!ok) *abort_flag = 1;
        return ok;
    };
    auto wait = [&](uint64_t* bar, unsigned parity) { return __all_sync(0xffffffffu, wait1(bar, parity)) != 0; };
    int images = 0;  // (first loader thread) image tiles asked for
    // Where a whole contraction is one stage, its converted A serves all column tiles of a row block: the A
    // columns in tensor memory then change with the row block, not with the stage (16384 x 64 -> 4352: 95 us
    // without, 80 us with).
    const bool keep_a = Lay::kTmemA && !Lay::kConvB && !Lay::kCopyB && job.k <= K;
    // This CTA's items lo, lo + step, .. below hi: one after another then, else taken in turn with the other CTAs,
    // so that those that run together share a row block in L2.
    const int step = keep_a ? 1 : gridDim.x;
    const int lo = keep_a ? (int)((long long)job.items * blockIdx.x / gridDim.x) : blockIdx.x;
    const int hi = keep_a ? (int)((long long)job.items * (blockIdx.x + 1) / gridDim.x) : job.items;
    if (P == Product::kGradW && (job.part || job.bias_part)) launch_dependents();
    if (IMAGE) wait_for_previous();  // for the image

    if (warp >= W::kEpi && warp < W::kMma) {  // loaders
        const int lt = t - 32 * W::kEpi, lw = lt >> 5;
        // Two cursors: the stage that is handed over now, and the one that is fetched, kDepth ahead.
        struct Cursor {
            int i, ks;
            Item it;
        } now{lo, 0, item_of<T, P, MT>(job, lo, BN)}, next = now;
        auto advance = [&](Cursor& c) {
            if (++c.ks < c.it.stages) return;
            c.ks = 0;
            c.i += step;
            if (c.i < hi) c.it = item_of<T, P, MT>(job, c.i, BN);
        };
        int ring = 0;  // the stage's place among the kDepth in flight
        constexpr int kChunkElems = 16 / sizeof(T);
        // -- A that is converted. A warp serves the 32 TMEM lanes that it may write (its index mod 4) and its share
        // of the k; it copies just what it reads, so that no other warp has to be waited for.
        constexpr int kShareK = 4 * K / W::kLoad;          // k of a warp
        constexpr int kRowBytes = Lay::kAMn ? 32 * (int)sizeof(T) : kShareK * (int)sizeof(T);  // of its block
        constexpr int kRows = Lay::kAMn ? kShareK : 32, kRowChunks = kRowBytes / 16;
        constexpr int kBlock = kRows * kRowBytes;
        const int quad = warp & 3, kshare = lw >> 2;
        auto block_a = [&](int z) {  // (z = 1: the pre-activation's)
            return smem + Lay::kOffRaw + ring * Lay::kRaw + z * Lay::kRawA + lw * kBlock;
        };
        auto chunk_a = [&](int r, int c) {  // chunk c of the block's row r: no two of 8 neighbouring rows in one bank
            const int x = kRowChunks >= 8 ? r & 7 : kRowChunks == 4 ? (r >> 1) & 3 : (r >> 2) & 1;
            return (uint32_t)(r * kRowBytes + (((c & ~7) | ((c ^ x) & 7)) << 4));
        };
        auto fetch_a = [&](const Cursor& c, const Operand& o, int z) {
            constexpr int kPer = 32 / kRowChunks > 0 ? 32 / kRowChunks : 1;  // rows side by side in a warp's copies
            constexpr int kCols = kRowChunks < 32 ? kRowChunks : 32;
            const int kk = c.it.k0 + c.ks * K + kshare * kShareK;
            const int row0 = Lay::kAMn ? kk : c.it.m0 + 32 * quad, col0 = Lay::kAMn ? c.it.m0 + 32 * quad : kk;
            const int rlim = Lay::kAMn ? c.it.k1 : o.nrows;
            unsigned char* blk = block_a(z);
            copy_column<T, VEC, kRows / kPer, kPer>(
                o, row0 + lane / kCols, rlim, col0 + (lane % kCols) * kChunkElems,
                [&](int i) { return blk + chunk_a(lane / kCols + kPer * i, lane % kCols); });
        };
        auto convert_a = [&](int slot) {
            constexpr int kB = kShareK < 16 ? kShareK : 16;  // k at a time
            const uint32_t col = tmem_a + ((uint32_t)(quad * 32) << 16) + slot * Lay::kACols + kshare * (kShareK / 2);
            const unsigned char *blk = block_a(0), *zb = block_a(1);
#pragma unroll
            for (int b = 0; b < kShareK / kB; ++b) {
                float v[kB];
                if constexpr (Lay::kAMn) {
                    // (float32) the lane's column, k after k
#pragma unroll
                    for (int j = 0; j < kB; ++j) {
                        const int r = b * kB + j;
                        v[j] = *reinterpret_cast<const float*>(blk + chunk_a(r, lane / 4) + 4 * (lane % 4));
                    }
                } else {
#pragma unroll
                    for (int c = 0; c < kB / kChunkElems; ++c)
                        read16<T>(blk + chunk_a(lane, b * (kB / kChunkElems) + c), v + c * kChunkElems);
                    if constexpr (kDzA) {
                        if (job.silu) {
                            float zv[kB];
#pragma unroll
                            for (int c = 0; c < kB / kChunkElems; ++c)
                                read16<T>(zb + chunk_a(lane, b * (kB / kChunkElems) + c), zv + c * kChunkElems);
#pragma unroll
                            for (int j = 0; j < kB; ++j) v[j] *= silu_grad(zv[j]);
                        }
                    }
                }
                split_parts<T, Lay::kPA, kB>(v, [&](int p, const uint32_t(&w)[kB / 2]) {
                    if (sizeof(T) == 4 || p == 0 || job.silu) tc::tmem_st(col + p * (K / 2) + b * (kB / 2), w);
                });
            }
        };
        // -- B that is converted: units of 8 columns; a warp's 32 units of one index lie together in planes of their
        // first and their second 16 bytes (one plane of bfloat16). The lanes copy the warp's units together, so
        // that neighbouring lanes read neighbouring 16 bytes.
        constexpr int kPlanes = sizeof(T) / 2;
        auto unit_b = [&](int z, int i) {
            return smem + Lay::kOffRaw + ring * Lay::kRaw + Lay::kRawA + (kDzA ? Lay::kRawZ : 0) + z * Lay::kRawB +
                   (i * W::kLoad + lw) * (512 * kPlanes);
        };
        auto fetch_b = [&](const Cursor& c, const Operand& o, int z) {
            const int kk = c.it.k0 + c.ks * K;
            const int row0 = Lay::kBMn ? kk : c.it.n0, col0 = Lay::kBMn ? c.it.n0 : kk;
            const int rlim = kDzB ? c.it.k1 : o.nrows;
#pragma unroll
            for (int h = 0; h < kPlanes; ++h) {
                const int w = (lt & ~31) + 32 / kPlanes * h + lane / kPlanes, sub = lane % kPlanes;
                const int lim = ShareB::kEven || ShareB::has(w, 0) ? rlim : 0;  // (one unit a thread at most then)
                copy_column<T, VEC, ShareB::kIters, W::kLoaders / ShareB::kPerRow>(
                    o, row0 + ShareB::row(w, 0), lim, col0 + 8 * ShareB::col(w) + sub * kChunkElems,
                    [&](int i) { return unit_b(z, i) + sub * 512 + (32 / kPlanes * h + lane / kPlanes) * 16; });
            }
        };
        float bsum[8];
        auto convert_b = [&](unsigned char* sb) {
#pragma unroll
            for (int i = 0; i < ShareB::kIters; ++i) {
                float v[8];
#pragma unroll
                for (int h = 0; h < kPlanes; ++h) read16<T>(unit_b(0, i) + h * 512 + lane * 16, v + h * kChunkElems);
                if constexpr (kDzB) {
                    if (job.silu) {
                        float zv[8];
#pragma unroll
                        for (int h = 0; h < kPlanes; ++h)
                            read16<T>(unit_b(1, i) + h * 512 + lane * 16, zv + h * kChunkElems);
#pragma unroll
                        for (int j = 0; j < 8; ++j) v[j] *= silu_grad(zv[j]);
                    }
#pragma unroll
                    for (int j = 0; j < 8; ++j) bsum[j] += v[j];
                }
                if (ShareB::has(lt, i))  // (a bfloat16 cotangent without an activation has no low part)
                    store_parts<T, Lay::kPB>(sb + ShareB::offset(lt, i), Lay::kBPart, v, sizeof(T) == 4 || job.silu);
            }
        };
        // -- operands used as they are, straight into the slot
        auto copy_tile = [&](auto share_c, const Operand& o, unsigned char* dst, int row0, int rlim, int col0) {
            using S = decltype(share_c);
            const int lim = S::kEven || S::has(lt, 0) ? rlim : 0;
            if (S::kEven || S::has(lt, 0))
                copy_column<T, VEC, S::kIters, W::kLoaders / S::kPerRow>(o, row0 + S::row(lt, 0), lim,
                                                                         col0 + 8 * S::col(lt),
                                                                         [&](int i) { return dst + S::offset(lt, i); });
        };
        auto fetch = [&]() {  // the fetch cursor's stage, one group of copies
            if (next.i < hi) {
                if constexpr (Lay::kTmemA) {
                    fetch_a(next, job.A, 0);
                    if constexpr (kDzA) {
                        if (job.silu) fetch_a(next, job.Z, 1);
                    }
                }
                if constexpr (Lay::kConvB) {
                    fetch_b(next, job.B, 0);
                    if constexpr (kDzB) {
                        if (job.silu) fetch_b(next, job.Z, 1);
                    }
                }
            }
            copy_commit();
            if (Lay::kTmemA && keep_a) next.i += job.ntn.d - 1 - (next.i - (next.it.m0 / kRowsTile) * job.ntn.d);
            advance(next);
        };
        auto arrive = [&](int slot) {  // this warp's part of the slot is written
            if (Lay::kTmemA) tc::tmem_wait_st();
            tc::fence_proxy_async();
            if (Lay::kTmemA) tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&full[slot]);
        };
        int n = 0;
        if constexpr (Lay::kRaw > 0) {
            for (ring = 0; ring < Lay::kDepth; ++ring) fetch();
            ring = 0;
        }
        int blocks = 0;  // row blocks converted (keep_a)
        for (; now.i < hi; ++n) {
            const int slot = n % kSlots;
            if (n >= kSlots && !wait(&empty[slot], (n / kSlots - 1) & 1)) break;
            if (Lay::kTmemA) tc::fence_after_sync();
            unsigned char* sb = smem + slot * Lay::kSlot;
            unsigned char* sa = sb + Lay::kPB * Lay::kBPart;
            if (IMAGE && lt == 0) {
                const int nks = (job.k + K - 1) / K;
                tc::mbar_expect_tx(&bfull[slot], Lay::kPB * Lay::kBPart);
                tc::bulk_g2s(sb, job.image + (size_t)((now.it.n0 / BN) * nks + now.ks) * (Lay::kPB * Lay::kBPart),
                             Lay::kPB * Lay::kBPart, &bfull[slot]);
                images = n + 1;
            }
            const int kk = now.it.k0 + now.ks * K;
            if constexpr (!Lay::kTmemA) {
                copy_tile(ShareA{}, job.A, sa, Lay::kAMn ? kk : now.it.m0, Lay::kAMn ? now.it.k1 : job.A.nrows,
                          Lay::kAMn ? now.it.m0 : kk);
            }
            if constexpr (Lay::kCopyB) {
                copy_tile(ShareB{}, job.B, sb, Lay::kBMn ? kk : now.it.n0, job.B.nrows, Lay::kBMn ? now.it.n0 : kk);
            }
            if constexpr (Lay::kRaw > 0) {
                const bool fresh = !(Lay::kTmemA && keep_a) || now.i == lo || now.it.n0 == 0;
                if (fresh) {
                    copy_wait<Lay::kDepth - 1>();
                    __syncwarp();
                    if constexpr (Lay::kTmemA) convert_a(keep_a ? blocks % kSlots : slot);
                    if constexpr (Lay::kConvB) {
                        if (kDzB && now.ks == 0)
#pragma unroll
                            for (int j = 0; j < 8; ++j) bsum[j] = 0.f;
                        convert_b(sb);
                    }
                    __syncwarp();  // read by all lanes
                    fetch();       // its group takes in the copies into the slot
                    ring = ring + 1 == Lay::kDepth ? 0 : ring + 1;
                    ++blocks;
                }
            } else {
                copy_commit();
            }
            if constexpr (Lay::kLag == 0) {
                arrive(slot);
            } else if (n >= Lay::kLag) {
                if (Lay::kRaw == 0) copy_wait<Lay::kLag>();  // else the wait above has passed that stage's copies
                arrive((n - Lay::kLag) % kSlots);
            }
            if (kDzB && now.ks + 1 >= now.it.stages && job.bias_part && now.it.m0 == 0) {
                // the item's sums of dz over its rows: the lanes of a warp that share columns, one row per warp
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    for (int o = ShareB::kPerRow; o < 32; o <<= 1) bsum[j] += __shfl_xor_sync(0xffffffffu, bsum[j], o);
                if (lane < ShareB::kPerRow) {
                    float* row = job.bias_part + (size_t)(now.it.split * W::kLoad + lw) * job.n;
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const int c = now.it.n0 + 8 * ShareB::col(lt) + j;
                        if (c < job.n) row[c] = bsum[j];
                    }
                }
            }
            advance(now);
        }
        copy_wait<0>();
        for (int m = n > Lay::kLag ? n - Lay::kLag : 0; m < n; ++m) arrive(m % kSlots);
    } else if (warp == W::kMma && lane == 0) {
        constexpr uint32_t idesc = idesc_bf16<Lay::kAMn && !Lay::kTmemA, Lay::kBMn>(BN);
        // one K step of 16, one part: descriptor units of 16 bytes
        constexpr uint32_t kStepA = (Lay::kAMn ? 2048 : 32) >> 4, kStepB = (Lay::kBMn ? 2048 : 32) >> 4;
        // the part products, smallest first: six of float32; the low and the high part of a bfloat16 layer's dz
        constexpr bool kF32 = sizeof(T) == 4;
        constexpr int kPairs = kF32 ? 6 : kDzA || kDzB ? 2 : 1;
        constexpr int pa[6] = {kF32 || kDzA ? 1 : 0, 0, 2, 0, 1, 0}, pb[6] = {kF32 || kDzB ? 1 : 0, kF32 ? 2 : 0, 0, 1, 0, 0};
        uint64_t base_a = 0;
        if constexpr (!Lay::kTmemA) base_a = operand_desc<Lay::kAMn, K>(tc::smem_u32(smem + Lay::kPB * Lay::kBPart));
        const uint64_t base_b = operand_desc<Lay::kBMn, K>(tc::smem_u32(smem));
        // the stage's MMAs, unrolled: operand addresses are the slot's plus constants
        auto issue = [&](auto steps_c, auto from_c, uint32_t d, int slot, int aslot, bool first) {
            constexpr int S = decltype(steps_c)::value, kFrom = decltype(from_c)::value;
            const uint64_t db = base_b + (uint64_t)(slot * (Lay::kSlot >> 4));
            [[maybe_unused]] const uint64_t da = base_a + (uint64_t)(slot * (Lay::kSlot >> 4));
            [[maybe_unused]] const uint32_t ta = tmem_a + aslot * Lay::kACols;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int q = kFrom; q < kPairs; ++q)
#pragma unroll
                    for (int s = 0; s < S; ++s) {
                        const uint32_t acc = q == kFrom && s == 0 ? (first ? 0u : 1u) : 1u;
                        const uint64_t b = db + (uint64_t)(pb[q] * (Lay::kBPart >> 4) + s * kStepB);
                        if constexpr (Lay::kTmemA)
                            mma_bf16_ta(d, ta + pa[q] * (K / 2) + s * 8, b, idesc, acc);
                        else  // a tile of 128 m: two panels
                            mma_bf16(d + mt * BN, da + (uint64_t)(mt * (2 * K * 128 >> 4) + s * kStepA), b, idesc, acc);
                    }
        };
        int n = 0, chunk = 0;
        bool ok = true;
        int block = -1;
        for (int i = lo; i < hi && ok; i += step) {
            const Item it = item_of<T, P, MT>(job, i, BN);
            if (i == lo || it.n0 == 0) ++block;
            for (int ks = 0; ks < it.stages; ++ks, ++n) {
                const int slot = n % kSlots, buf = chunk % kRing;
                const bool first = ks % kChunk<T> == 0;
                if ((first && chunk >= kRing && !wait1(&tempty[buf], (chunk / kRing - 1) & 1)) ||
                    !wait1(&full[slot], (n / kSlots) & 1) || (IMAGE && !wait1(&bfull[slot], (n / kSlots) & 1))) {
                    ok = false;
                    break;
                }
                tc::fence_after_sync();
                const int left = it.k1 - it.k0 - ks * K;
                const uint32_t d = tmem + buf * Lay::kAcc;
                const int aslot = keep_a ? block % kSlots : slot;
                auto steps = [&](auto from_c) {
                    if (left > K - 16)
                        issue(Int<K / 16>{}, from_c, d, slot, aslot, first);
                    else if (K == 64 && left > 32)
                        issue(Int<K == 64 ? 3 : 1>{}, from_c, d, slot, aslot, first);
                    else if (K == 64 && left > 16)
                        issue(Int<K == 64 ? 2 : 1>{}, from_c, d, slot, aslot, first);
                    else
                        issue(Int<1>{}, from_c, d, slot, aslot, first);
                };
                if (kPairs == 2 && !job.silu)  // dz is the bfloat16 cotangent itself: no low part
                    steps(Int<kPairs == 2 ? 1 : 0>{});
                else
                    steps(Int<0>{});
                tc::mma_commit(&empty[slot]);
                if (ks + 1 == it.stages || (ks + 1) % kChunk<T> == 0) {
                    tc::mma_commit(&tfull[buf]);
                    ++chunk;
                }
            }
        }
    } else if (warp < W::kEpi) {
        constexpr int kCols = 4 * BN / W::kEpi;  // columns of a warp
        const int quad = warp & 3, n0 = (warp >> 2) * kCols;
        const uint32_t base = tmem + ((uint32_t)(quad * 32) << 16) + n0;
        auto read = [&](int buf, int c, auto& v) {  // 16 lanes by NC columns from column c, both halves
            constexpr int NC = sizeof(v) / (2 * sizeof(float)) * 2;
#pragma unroll
            for (int h = 0; h < 2; ++h)
                tc::tmem_ld_frag<NC / 2>(base + ((uint32_t)(16 * h) << 16) + buf * Lay::kAcc + c, v[h]);
            tc::tmem_wait_ld(v[0]);
            tc::tmem_wait_ld(v[1]);
        };
        auto release = [&](int buf) {  // the accumulator has been read
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&tempty[buf]);
        };
        constexpr int kFullVec = sizeof(T) == 2 && P == Product::kGradX ? 2 : 1;
        auto end = [&](const Item& it, int at, auto cols_c, auto& acc) {
            constexpr int NC = decltype(cols_c)::value;
            if (job.vec_out >= kFullVec && job.map.per.d == 1 && it.m0 + kRowsTile <= job.m && it.n0 + BN <= job.n)
                finish<T, P, NC, Pairs::kFull>(job, it, acc, quad, n0 + at, lane);
            else if (job.vec_out)
                finish<T, P, NC, Pairs::kEven>(job, it, acc, quad, n0 + at, lane);
            else
                finish<T, P, NC, Pairs::kAny>(job, it, acc, quad, n0 + at, lane);
        };
        int chunk = 0;
        bool ok = true;
        for (int i = lo; i < hi && ok; i += step) {
            const Item it = item_of<T, P, MT>(job, i, BN);
            if constexpr (sizeof(T) == 2) {  // one accumulator: pieces of it, read and finished in turn
                constexpr int NC = kCols < 32 ? kCols : 32;
                const int buf = chunk % kRing;
                ok = wait(&tfull[buf], (chunk / kRing) & 1);
                if (!ok) break;
                tc::fence_after_sync();
#pragma unroll 1
                for (int mt = 0; mt < MT; ++mt) {
                    Item sub = it;
                    sub.m0 += mt * kRowsTile;
#pragma unroll 1
                    for (int c = 0; c < kCols; c += NC) {
                        float v[2][NC / 2];
                        read(buf, mt * BN + c, v);
                        if (mt + 1 == MT && c + NC == kCols) release(buf);
                        end(sub, c, Int<NC>{}, v);
                    }
                }
                ++chunk;
            } else {
                constexpr int NR = kCols / 2, NP2 = NR < 16 ? NR : P == Product::kForward ? 16 : 8;
                float acc[2][NR];
#pragma unroll
                for (int j = 0; j < NR; ++j) acc[0][j] = acc[1][j] = 0.f;
                for (int ks = 0; ks < it.stages; ks += kChunk<T>, ++chunk) {
                    const int buf = chunk % kRing;
                    ok = wait(&tfull[buf], (chunk / kRing) & 1);
                    if (!ok) break;
                    tc::fence_after_sync();
#pragma unroll
                    for (int c = 0; c < NR; c += NP2) {  // as many columns at once as registers allow
                        float v[2][NP2];
                        read(buf, 2 * c, v);
#pragma unroll
                        for (int h = 0; h < 2; ++h)
#pragma unroll
                            for (int j = 0; j < NP2; j += 2) {
                                const float2 a = __fadd2_rn(make_float2(acc[h][c + j], acc[h][c + j + 1]),
                                                            make_float2(v[h][j], v[h][j + 1]));
                                acc[h][c + j] = a.x, acc[h][c + j + 1] = a.y;
                            }
                    }
                    release(buf);
                }
                if (!ok) break;
                end(it, 0, Int<kCols>{}, acc);
            }
        }
    }
    __syncthreads();
    if (*abort_flag) {  // leave no MMA or copy in flight on the freed memory
        if (t == 32 * W::kMma) {
            atomicOr(&g_fault, 1);
            tc::mma_commit(drain);
            tc::mbar_wait(drain, 0, kWaitLimit);
        }
        if (IMAGE && t == 32 * W::kEpi)
            for (int m = images > kSlots ? images - kSlots : 0; m < images; ++m)
                tc::mbar_wait(&bfull[m % kSlots], (m / kSlots) & 1, kWaitLimit);
        __syncthreads();
    }
    tc::fence_before_sync();
    __syncthreads();
    if (warp == W::kMma) tc::tmem_dealloc(tmem, Lay::kTmemCols);
}

// W as tiles of operand parts in the layout of a slot's B, tile (nt, ks) after tile:
// converted once here instead of once per row tile by every CTA. A thread converts
// units of 8 consecutive elements of W.
template <typename T, Product P, int BN>
__global__ void __launch_bounds__(256) etp_linear_image_kernel(const T* __restrict__ W, int rows, int cols,
                                                               unsigned char* __restrict__ image) {
    using Lay = Layout<T, P, BN, true, true>;
    constexpr int R = Lay::kBMn ? Lay::kK : BN, C = Lay::kBMn ? BN : Lay::kK;  // W's rows and columns in a tile
    constexpr int kPerRow = C / 8, kUnits = R * kPerRow;
    const int ct = (cols + C - 1) / C, rt = (rows + R - 1) / R;
    launch_dependents();
    const int u = blockIdx.x * 256 + threadIdx.x, tile = u / kUnits, w = u % kUnits;
    if (tile >= ct * rt) return;
    // tiles along the contraction are adjacent: it runs over W's rows (MN-major) or columns
    const int rti = Lay::kBMn ? tile % rt : tile / ct, cti = Lay::kBMn ? tile / rt : tile % ct;
    const int r = w / kPerRow, c = w % kPerRow, gr = rti * R + r, gc = cti * C + 8 * c;
    const T* p = W + (size_t)gr * cols + gc;
    const int left = gr < rows ? cols - gc : 0;
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = j < left ? to_float(p[j]) : 0.f;
    store_parts<T, Lay::kPB>(image + (size_t)tile * Lay::kPB * Lay::kBPart + chunk_offset<Lay::kK>(r, c),
                             Lay::kBPart, v);
}

// grad_W from the ranges' sums [splits][count] and grad_bias from [bias_rows][N], both in
// a fixed order. A block: 128 elements of grad_W (V = 4 a thread, 16 row lanes) or 8 of
// grad_bias (64 row lanes), then the row lanes' sums in order. Started while the sums are
// still being written: waits for them itself.
constexpr int kJoinThreads = 512;
template <typename T, int V>
__global__ void __launch_bounds__(kJoinThreads)
    etp_linear_join_kernel(const float* __restrict__ part, int splits, size_t count, T* __restrict__ gW,
                           const float* __restrict__ bias_part, int bias_rows, int N, T* __restrict__ gbias,
                           int blocks_w) {
    __shared__ float red[kJoinThreads * V];
    wait_for_previous();
    const int t = threadIdx.x;
    if ((int)blockIdx.x < blocks_w) {
        constexpr int kCols = 32, kRows = kJoinThreads / kCols;
        const size_t col = ((size_t)blockIdx.x * kCols + t % kCols) * V;
        const int sub = t / kCols;
        float s[V];
#pragma unroll
        for (int j = 0; j < V; ++j) s[j] = 0.f;
        if (col < count)
#pragma unroll 4
            for (int r = sub; r < splits; r += kRows) {
                float v[V];
                Pack<float, V>::load(part + (size_t)r * count + col, v);
#pragma unroll
                for (int j = 0; j < V; ++j) s[j] += v[j];
            }
#pragma unroll
        for (int j = 0; j < V; ++j) red[t * V + j] = s[j];
        __syncthreads();
        if (t >= kCols * V) return;
        const size_t at = (size_t)blockIdx.x * kCols * V + t;
        if (at >= count) return;
        float sum = red[t];
#pragma unroll
        for (int w = 1; w < kRows; ++w) sum += red[w * kCols * V + t];
        gW[at] = from_float<T>(sum);
        return;
    }
    constexpr int kCols = 8, kRows = kJoinThreads / kCols;
    const int col = ((int)blockIdx.x - blocks_w) * kCols + t % kCols, sub = t / kCols;
    float s = 0.f;
    if (col < N)
#pragma unroll 8
        for (int r = sub; r < bias_rows; r += kRows) s += bias_part[(size_t)r * N + col];
    red[t] = s;
    __syncthreads();
    if (t >= kCols || col >= N) return;
#pragma unroll 16
    for (int w = 1; w < kRows; ++w) s += red[w * kCols + t];
    gbias[col] = from_float<T>(s);
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

template <typename T, Product P, int BN, bool VEC, bool IMAGE, int MT = 1>
cudaError_t launch_kernel(const Job& j, cudaStream_t s) {
    using Lay = Layout<T, P, BN, VEC, IMAGE, MT>;
    // the shared memory limit of this kernel is raised once per device (a bit of the mask)
    static std::atomic<unsigned long long> raised{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = dev < 64 ? 1ull << dev : 0;
    if (!(raised.load(std::memory_order_relaxed) & bit)) {
        e = cudaFuncSetAttribute(etp_linear_kernel<T, P, BN, VEC, IMAGE, MT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)Lay::kBytes);
        if (e != cudaSuccess) return e;
        raised.fetch_or(bit, std::memory_order_relaxed);
    }
    const int sms = sm_count();
    const int grid = j.items < sms ? j.items : sms;
    if (IMAGE)
        return launch_after(etp_linear_kernel<T, P, BN, VEC, IMAGE, MT>, grid, Warps<T, P>::kThreads, Lay::kBytes, s, j);
    etp_linear_kernel<T, P, BN, VEC, IMAGE, MT><<<grid, Warps<T, P>::kThreads, Lay::kBytes, s>>>(j);
    return cudaGetLastError();
}

// VEC: the operands' rows move in 16-byte groups.
template <typename T, Product P, int BN, int MT = 1>
cudaError_t launch_bn(Job& j, unsigned char* image, cudaStream_t s) {
    const bool z = !j.Z.rows.p || j.Z.vec;
    if constexpr (P != Product::kGradW) {
        if (image) {
            using Lay = Layout<T, P, BN, true, true>;
            const int rows = j.B.nrows, cols = j.B.ncols;
            const int R = Lay::kBMn ? Lay::kK : BN, C = Lay::kBMn ? BN : Lay::kK;
            const long long units = (long long)((rows + R - 1) / R) * ((cols + C - 1) / C) * (R * C / 8);
            etp_linear_image_kernel<T, P, BN><<<(unsigned)((units + 255) / 256), 256, 0, s>>>(
                static_cast<const T*>(j.B.rows.p), rows, cols, image);
            const cudaError_t e = cudaGetLastError();
            if (e != cudaSuccess) return e;
            j.image = image;
            return j.A.vec && z ? launch_kernel<T, P, BN, true, true>(j, s)
                                : launch_kernel<T, P, BN, false, true>(j, s);
        }
    }
    return j.A.vec && j.B.vec && z ? launch_kernel<T, P, BN, true, false, MT>(j, s)
                                   : launch_kernel<T, P, BN, false, false, MT>(j, s);
}

// How the forward and grad_x products of M rows, k contracted and n output columns are
// tiled: the widest tile that still gives every SM one, or the narrowest (256 columns
// with bfloat16 alone: A is then read, and dz formed, half as often; 131072 x 256 -> 256
// grad_x 89 us with 128, 58 us with 256; float32 parts leave no tensor memory for it).
// float32 takes 128 columns once every SM gets two such tiles: below that its one or two
// rounds wait for whole conversions (forward with 128 / 64 columns, on the device alone:
// 20480 x 128 -> 128 18.8 / 13.0 us, 37000 rows 19.8 / 15.8, 40000 rows 15.0 / 18.5; bfloat16
// 12.3 / 13.3 at 20480). The rule counts SMs without a tile, not rounds, and loses where a
// wider tile would take fewer of them, float32 forward: 8192 x 128 -> 128 10.6 us with the 32
// columns that it takes (64: 8.3), 2048 x 128 -> 512 10.6 (64: 8.3), 4096 x 256 -> 256 15.9 (64:
// 12.1), 12288 x 128 -> 128 12.3 with 64 (128: 11.4), 2048 x 256 -> 1024 18.6 with 64 (128:
// 16.6); it gains at 1024 x 128 -> 512 6.8 with 32 (64: 8.0) and 4096 x 128 -> 128 7.0 (8.2). And whether W
// is converted ahead (an image), which pays once a CTA would convert it more than once and
// enough row tiles share it. float32, with the image / without: 64 x 256 -> 65536 64 / 51 us,
// 256 x 1024 -> 32768 155 / 170, 4096 x 512 -> 4096 90 / 156. bfloat16, whose image is only a
// copy in another order: 64 x 2048 -> 40960 120 / 57 us, 1024 x 1024 -> 8192 49 / 43,
// 4096 x 512 -> 4096 43 / 43, 16384 x 256 -> 2048 47 / 49.
struct Tiling {
    int bn;
    bool image;
    size_t image_bytes;
};
Tiling tiling(bool bf16, Product p, int M, int k, int n) {
    const long long mt = ((long long)M + kRowsTile - 1) / kRowsTile;
    const int sms = sm_count();
    Tiling t;
    auto enough = [&](int bn, int each) { return n > bn / 2 && mt * ((n + bn - 1) / bn) >= (long long)each * sms; };
    t.bn = bf16 && p == Product::kGradX && enough(256, 1) ? 256
           : enough(128, bf16 ? 1 : 2)                    ? 128
           : enough(64, 1)                                ? 64
                                                          : 32;
    t.image = mt >= (bf16 ? 32 : 2) && mt * ((n + t.bn - 1) / t.bn) >= 2 * sms;
    constexpr int K = 64;  // k of a stage of either
    static_assert(kStageK<float, Product::kForward> == K && kStageK<float, Product::kGradX> == K, "image tiles");
    const size_t part = (size_t)(p == Product::kForward && t.bn < 64 ? 64 : t.bn) * K * 2;
    t.image_bytes = t.image ? (size_t)((n + t.bn - 1) / t.bn) * ((k + K - 1) / K) * (bf16 ? 1 : 3) * part : 0;
    return t;
}

template <typename T, Product P>
cudaError_t launch(Job& j, int bn, int tall, int splits, unsigned char* image, cudaStream_t s) {
    j.ntn = FastDiv((j.n + bn - 1) / bn);
    const int mtn = P == Product::kGradW && j.m == 0 ? 1 : (j.m + tall * kRowsTile - 1) / (tall * kRowsTile);  // no rows: still a tile
    const long long tiles = (long long)mtn * j.ntn.d;
    if (tiles * splits > 0x7fff0000LL) return cudaErrorInvalidValue;
    j.tiles = FastDiv((int)tiles);
    j.items = (int)tiles * splits;
    if constexpr (sizeof(T) == 2 && P == Product::kGradW) {
        if (tall == 2) return launch_bn<T, P, 128, 2>(j, image, s);
    }
    switch (bn) {
        case 256:
            if constexpr (sizeof(T) == 2 && P == Product::kGradX) return launch_bn<T, P, 256>(j, image, s);
            return cudaErrorInvalidValue;
        case 128: return launch_bn<T, P, 128>(j, image, s);
        case 64: return launch_bn<T, P, 64>(j, image, s);
        default: return launch_bn<T, P, 32>(j, image, s);
    }
}

// grad_W: tile shape and ranges of the rows, whole stages, one range per SM and tile.
struct Ranges {
    int bn, tall, tiles, splits, range;  // tall: tiles of 256 x 128, so that dz is formed for two row tiles at once
};
Ranges ranges(bool bf16, int M, int K, int N) {
    Ranges r;
    r.bn = N > 64 ? 128 : N > 32 ? 64 : 32;
    r.tall = bf16 && K > 128 && r.bn == 128 ? 2 : 1;  // (131072 x 256 -> 256: 90 us with 1, 66 us with 2)
    r.tiles = ((K + r.tall * kRowsTile - 1) / (r.tall * kRowsTile)) * ((N + r.bn - 1) / r.bn);
    const int sms = sm_count();
    const int stages = (M + kRangeK - 1) / kRangeK;
    int want = r.tiles < sms ? sms / r.tiles : 1;
    want = want < stages ? want : stages;
    const int least = bf16 ? (int)(((long long)M + kMostRange - 1) / kMostRange) : 1;
    want = want > least ? want : least;
    const int per = want > 0 ? (stages + want - 1) / want : 1;
    // a multiple of kRangeK that an int holds (M is below 2^31 - 128)
    const long long range = (long long)per * kRangeK, most = (1ll << 31) - kRangeK;
    r.range = (int)(range < most ? range : most);
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
    return launch<T, Product::kForward>(j, t.bn, 1, 1, t.image ? reinterpret_cast<unsigned char*>(a.ws) : nullptr, s);
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
        for (int v = 2; v <= 4; v *= 2)
            if (a.K % v == 0 && rows_aligned(a.gx, elem, v * elem)) j.vec_out = v / 2;
        const Tiling t = tiling(elem == 2, Product::kGradX, j.m, j.k, j.n);
        const cudaError_t e = launch<T, Product::kGradX>(
            j, t.bn, 1, 1, t.image ? reinterpret_cast<unsigned char*>(a.ws) : nullptr, s);
        if (e != cudaSuccess) return e;
    }
    if (!a.gW && !a.gbias) return cudaSuccess;
    // without grad_W the tile has no rows: only the loaders' sums of dz are wanted
    const int K = a.gW ? a.K : 0;
    const Ranges r = ranges(elem == 2, a.map.M, a.gW ? a.K : 1, a.N);
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
        const cudaError_t e = launch<T, Product::kGradW>(j, r.bn, r.tall, r.splits, nullptr, s);
        if (e != cudaSuccess) return e;
    }
    const size_t count = a.gW && join ? (size_t)a.K * a.N : 0;
    const bool v4 = count % 4 == 0;
    const int per = v4 ? 128 : 32;
    const int blocks_w = (int)((count + per - 1) / per), blocks_b = a.gbias ? (a.N + 7) / 8 : 0;
    if (blocks_w + blocks_b == 0) return cudaSuccess;
    return launch_after(v4 ? etp_linear_join_kernel<T, 4> : etp_linear_join_kernel<T, 1>, blocks_w + blocks_b,
                        kJoinThreads, 0, s, part, r.splits, count, static_cast<T*>(a.gW), bias_part,
                        r.splits * Warps<T, Product::kGradW>::kLoad, a.N, static_cast<T*>(a.gbias), blocks_w);
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
        const Ranges r = ranges(bf16, M, gw ? K : 1, N);  // as backward() asks for them
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
