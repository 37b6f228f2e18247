// loss_device.h - device helpers of the row kernels (k_topk.hip,
// k_distill.hip, k_balance.hip): the three logit types as 16-byte granules,
// and reductions over a wave and a workgroup.
#pragma once

#include <type_traits>

#include "loss_internal.h"
#include "scape_device.h"

namespace scape {

typedef uint32_t gran __attribute__((ext_vector_type(4)));  // 16 bytes of a row

constexpr float kNegInf = -__builtin_inff();
constexpr float kLog2e = 1.44269504088896340736f;
constexpr double kLn2 = 0.693147180559945309417, kLog2e64 = 1.44269504088896340736;

// A logit type: its storage, its elements per granule, and the conversions
// of element j (a compile-time constant after unrolling) of a granule.
struct F32 {
    using raw = uint32_t;
    static constexpr int kN = 4;
    static constexpr uint32_t kNegInfBits = 0xFF800000u;
    static __device__ __forceinline__ float up(const gran& g, int j) { return __uint_as_float(g[j]); }
    static __device__ __forceinline__ float up1(raw r) { return __uint_as_float(r); }
    static __device__ __forceinline__ void set(gran& g, int j, raw r) { g[j] = r; }
    static __device__ __forceinline__ raw down1(float f) { return __float_as_uint(f); }
    static __device__ __forceinline__ gran down(const float (&f)[kN]) {
        return gran{__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3])};
    }
};

struct BF16 {
    using raw = uint16_t;
    static constexpr int kN = 8;
    static constexpr uint32_t kNegInfBits = 0xFF80u;
    typedef __bf16 pair __attribute__((ext_vector_type(2)));
    typedef float fpair __attribute__((ext_vector_type(2)));
    static __device__ __forceinline__ float up(const gran& g, int j) {
        return __uint_as_float((j & 1) ? (g[j >> 1] & 0xFFFF0000u) : (g[j >> 1] << 16));
    }
    static __device__ __forceinline__ float up1(raw r) { return __uint_as_float((uint32_t)r << 16); }
    static __device__ __forceinline__ void set(gran& g, int j, raw r) {
        g[j >> 1] = (j & 1) ? (g[j >> 1] & 0x0000FFFFu) | ((uint32_t)r << 16) : (g[j >> 1] & 0xFFFF0000u) | r;
    }
    // one rounding, to nearest even: the gradient's type holds 8 bits
    static __device__ __forceinline__ uint32_t down2(float a, float b) {
        return __builtin_bit_cast(uint32_t, __builtin_convertvector((fpair{a, b}), pair));
    }
    static __device__ __forceinline__ raw down1(float f) { return (raw)(down2(f, f) & 0xFFFFu); }
    static __device__ __forceinline__ gran down(const float (&f)[kN]) {
        return gran{down2(f[0], f[1]), down2(f[2], f[3]), down2(f[4], f[5]), down2(f[6], f[7])};
    }
};

struct F16 {
    using raw = uint16_t;
    static constexpr int kN = 8;
    static constexpr uint32_t kNegInfBits = 0xFC00u;
    typedef _Float16 pair __attribute__((ext_vector_type(2)));
    static __device__ __forceinline__ float up(const gran& g, int j) {
        const uint32_t two = g[j >> 1];  // a bit_cast straight from the vector's element takes element 0
        return (float)__builtin_bit_cast(pair, two)[j & 1];
    }
    static __device__ __forceinline__ float up1(raw r) { return (float)__builtin_bit_cast(_Float16, r); }
    static __device__ __forceinline__ void set(gran& g, int j, raw r) { BF16::set(g, j, r); }
    // one rounding, to nearest even: the gradient's type holds 11 bits
    static __device__ __forceinline__ raw down1(float f) { return __builtin_bit_cast(raw, (_Float16)f); }
    static __device__ __forceinline__ uint32_t down2(float a, float b) {
        return (uint32_t)down1(a) | ((uint32_t)down1(b) << 16);
    }
    static __device__ __forceinline__ gran down(const float (&f)[kN]) {
        return gran{down2(f[0], f[1]), down2(f[2], f[3]), down2(f[4], f[5]), down2(f[6], f[7])};
    }
};

// One element of an array whose type is known at run time (the teacher's
// values, k of them a row): the bits, which take no instruction that would
// wait for the load, and what they are.
__device__ __forceinline__ uint32_t load_bits(const void* p, int32_t dtype, int64_t i) {
    if (dtype == SCAPE_DTYPE_F32) return static_cast<const uint32_t*>(p)[i];
    return static_cast<const uint16_t*>(p)[i];
}
__device__ __forceinline__ float value_of(uint32_t bits, int32_t dtype) {
    if (dtype == SCAPE_DTYPE_F32) return __uint_as_float(bits);
    return dtype == SCAPE_DTYPE_BF16 ? BF16::up1((uint16_t)bits) : F16::up1((uint16_t)bits);
}

// A row starts anywhere; its granules lie on 16-byte boundaries.  The `head`
// elements before the first boundary and the `tail` elements after the last
// whole granule are fewer than a granule each, and are taken one a thread
// beside the granules, so nothing outside the row is touched.  Granule i
// holds elements head + i N ...
struct RowShape {
    int32_t head, granules, tail;
};
template <class T>
__device__ __forceinline__ RowShape row_shape(const void* row, int32_t n) {
    RowShape r;
    r.head = (int32_t)(((16u - ((uint32_t)(uintptr_t)row & 15u)) & 15u) / sizeof(typename T::raw));
    if (r.head > n) r.head = n;
    r.granules = (n - r.head) / T::kN;
    r.tail = n - r.head - r.granules * T::kN;
    return r;
}
// What a row without a whole granule reads instead, so that the loads of a
// kernel's first granules stand under no condition.
__device__ gran g_no_granule = {0u, 0u, 0u, 0u};

// Granule i of a run, and 16 bytes at it: a uniform base and a 32-bit offset.
// Read once, written once: non-temporal both ways (loss and gradient of
// 4096x32000 bf16 109 -> 101 us, gradient of 1024x50304 f32 90 -> 81 us).
__device__ __forceinline__ gran granule_at(const void* body, int32_t i) {
    return __builtin_nontemporal_load(
        reinterpret_cast<const gran*>(static_cast<const char*>(body) + (size_t)((uint32_t)i * 16u)));
}

// The element a thread takes beside its granules in the first or the last
// part of a row, or -1.
__device__ __forceinline__ int32_t lone_element(const RowShape& r, int32_t n, bool first, bool last) {
    const int32_t tid = (int32_t)threadIdx.x;
    if (first && tid < r.head) return tid;
    if (last && tid >= 64 && tid - 64 < r.tail) return n - r.tail + tid - 64;
    return -1;
}

// 16 bytes to granule i of a run of any alignment: one store (the target's
// memory mode takes them; the compiler picks the instruction).
typedef uint32_t loose_gran __attribute__((ext_vector_type(4), aligned(2)));
__device__ __forceinline__ void store_loose(void* run, int32_t i, const gran& g) {
    __builtin_nontemporal_store((loose_gran)g, reinterpret_cast<loose_gran*>(static_cast<char*>(run) +
                                                                             (size_t)((uint32_t)i * 16u)));
}

template <class T>
__device__ __forceinline__ gran no_entries() {  // a granule of -inf
    return T::kN == 4 ? gran{T::kNegInfBits, T::kNegInfBits, T::kNegInfBits, T::kNegInfBits}
                      : gran{T::kNegInfBits * 0x10001u, T::kNegInfBits * 0x10001u, T::kNegInfBits * 0x10001u,
                             T::kNegInfBits * 0x10001u};
}

// Between two passes over registers: the compiler would keep a first pass's
// unpacked 16-bit elements, two registers for one, for the second, and spill.
__device__ __forceinline__ void forget_unpacked(gran& g) { asm volatile("" : "+v"(g)); }
// A thread's index anew, so that the addresses made from it in one pass are
// not kept for the next.
__device__ __forceinline__ int32_t again(int32_t tid) {
    asm volatile("" : "+v"(tid));
    return tid;
}

// The larger of two, NaN if either is: v_maximum3_f32 takes three at once.
__device__ __forceinline__ float max_nan(float a, float b) { return __builtin_elementwise_maximum(a, b); }
template <class T>
__device__ __forceinline__ float granule_max(const gran& g) {
    if constexpr (std::is_same<T, F16>::value) {  // two at once, unpacked at the end
        typedef _Float16 pair __attribute__((ext_vector_type(2)));
        const uint32_t w0 = g[0], w1 = g[1], w2 = g[2], w3 = g[3];
        const pair m = __builtin_elementwise_maximum(
            __builtin_elementwise_maximum(__builtin_bit_cast(pair, w0), __builtin_bit_cast(pair, w1)),
            __builtin_elementwise_maximum(__builtin_bit_cast(pair, w2), __builtin_bit_cast(pair, w3)));
        return max_nan((float)m[0], (float)m[1]);
    }
    float m = T::up(g, 0);
#pragma unroll
    for (int j = 1; j < T::kN; ++j) m = max_nan(m, T::up(g, j));
    return m;
}

__device__ __forceinline__ float fast_exp2(float x) { return __builtin_amdgcn_exp2f(x); }  // v_exp_f32

// Element j minus r.  fp16: as a multiply-add by a one that the compiler does
// not see, which takes the element unpacked and converted in the same
// instruction (v_fma_mix_f32).
template <class T>
__device__ __forceinline__ float less(const gran& g, int j, float r) {
    if constexpr (std::is_same<T, F16>::value) {
        float one = 1.0f;
        asm("" : "+v"(one));
        return __builtin_fmaf(T::up(g, j), one, -r);
    }
    return T::up(g, j) - r;
}

// A running sum of 2^(c2 (x - ref)), ref the largest x so far.  The difference
// is taken before the product: a product's rounding against a reference that
// was rounded as well is off by as much as the logits are large, and a row of
// the type's lowest value would leave the range.  It follows the loads as they
// arrive: no pass for the maximum first.  -inf adds nothing; NaN and +inf make
// the sum NaN.
constexpr float kLowest = -3.402823466e38f;
struct RunningSum {
    float ref, sum;
    static __device__ __forceinline__ RunningSum none() { return RunningSum{kLowest, 0.0f}; }
    // B granules whose largest element is m
    template <class T, int B>
    __device__ __forceinline__ void add(const gran (&g)[B], float m, float c2) {
        const float r = fmaxf(ref, m);
        float s0 = sum * fast_exp2((ref - r) * c2), s1 = 0.0f;  // two chains, for the adders
        ref = r;
#pragma unroll
        for (int b = 0; b < B; ++b)
#pragma unroll
            for (int j = 0; j < T::kN; j += 2) {
                s0 += fast_exp2(less<T>(g[b], j, r) * c2);
                s1 += fast_exp2(less<T>(g[b], j + 1, r) * c2);
            }
        sum = s0 + s1;
    }
    __device__ __forceinline__ void add1(float x, float c2) {
        const float r = fmaxf(ref, x);
        sum = sum * fast_exp2((ref - r) * c2) + fast_exp2((x - r) * c2);
        ref = r;
    }
};

// ---------------------------------------------------------------------------
// Reductions.  Over a wave without LDS: quads and rows of 16 by DPP
// permutations, then rows against rows with the gfx950 row swaps (both
// results hold one row of each pair, so adding them is the pair's sum in
// every lane).  Every lane gets the same bits.
template <int kCtrl>
__device__ __forceinline__ uint32_t dpp32(uint32_t x) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, kCtrl, 0xF, 0xF, false);
}

struct OpMaxF {
    static __device__ __forceinline__ float f(float a, float b) { return max_nan(a, b); }
};
struct OpMaxNum {  // NaN left out
    static __device__ __forceinline__ float f(float a, float b) { return fmaxf(a, b); }
};
struct OpSumF {
    static __device__ __forceinline__ float f(float a, float b) { return a + b; }
};
struct OpMaxU {
    static __device__ __forceinline__ uint32_t f(uint32_t a, uint32_t b) { return a > b ? a : b; }
};

// All-reduce of a 32-bit value over groups of kLanes consecutive lanes.
template <class Op, int kLanes, class V>
__device__ __forceinline__ V group_reduce(V x) {
    static_assert(sizeof(V) == 4, "32-bit values");
#define SCAPE_DPP_STEP(ctrl) x = Op::f(x, __builtin_bit_cast(V, dpp32<ctrl>(__builtin_bit_cast(uint32_t, x))))
    if constexpr (kLanes >= 2) SCAPE_DPP_STEP(0xB1);    // quad_perm [1,0,3,2]
    if constexpr (kLanes >= 4) SCAPE_DPP_STEP(0x4E);    // quad_perm [2,3,0,1]
    if constexpr (kLanes >= 8) SCAPE_DPP_STEP(0x141);   // row_half_mirror
    if constexpr (kLanes >= 16) SCAPE_DPP_STEP(0x140);  // row_mirror
#undef SCAPE_DPP_STEP
    if constexpr (kLanes >= 32) {
        const auto r = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, x),
                                                        __builtin_bit_cast(uint32_t, x), false, false);
        x = Op::f(__builtin_bit_cast(V, (uint32_t)r[0]), __builtin_bit_cast(V, (uint32_t)r[1]));
    }
    if constexpr (kLanes >= 64) {
        const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, x),
                                                        __builtin_bit_cast(uint32_t, x), false, false);
        x = Op::f(__builtin_bit_cast(V, (uint32_t)r[0]), __builtin_bit_cast(V, (uint32_t)r[1]));
    }
    return x;
}

template <int kCtrl>
__device__ __forceinline__ double dpp64(double x) {
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    return __builtin_bit_cast(double, (uint64_t)dpp32<kCtrl>((uint32_t)u) | (uint64_t)dpp32<kCtrl>((uint32_t)(u >> 32)) << 32);
}

// Sum over the kWaves (4 or 8) values that each group of as many lanes holds
// alike: the workgroup's waves' partial sums, read by lane % kWaves.
template <int kWaves>
__device__ __forceinline__ double sum_waves_f64(double x) {
    static_assert(kWaves == 4 || kWaves == 8, "quads or half rows");
    x += dpp64<0xB1>(x);
    x += dpp64<0x4E>(x);
    if constexpr (kWaves == 8) x += dpp64<0x141>(x);
    return x;
}

__device__ __forceinline__ double wave_sum_f64(double x) {
    x = sum_waves_f64<8>(x);
    x += dpp64<0x140>(x);
    {
        const uint64_t u = __builtin_bit_cast(uint64_t, x);
        const auto lo = __builtin_amdgcn_permlane16_swap((uint32_t)u, (uint32_t)u, false, false);
        const auto hi = __builtin_amdgcn_permlane16_swap((uint32_t)(u >> 32), (uint32_t)(u >> 32), false, false);
        x = __builtin_bit_cast(double, (uint64_t)(uint32_t)lo[0] | (uint64_t)(uint32_t)hi[0] << 32) +
            __builtin_bit_cast(double, (uint64_t)(uint32_t)lo[1] | (uint64_t)(uint32_t)hi[1] << 32);
    }
    {
        const uint64_t u = __builtin_bit_cast(uint64_t, x);
        const auto lo = __builtin_amdgcn_permlane32_swap((uint32_t)u, (uint32_t)u, false, false);
        const auto hi = __builtin_amdgcn_permlane32_swap((uint32_t)(u >> 32), (uint32_t)(u >> 32), false, false);
        x = __builtin_bit_cast(double, (uint64_t)(uint32_t)lo[0] | (uint64_t)(uint32_t)hi[0] << 32) +
            __builtin_bit_cast(double, (uint64_t)(uint32_t)lo[1] | (uint64_t)(uint32_t)hi[1] << 32);
    }
    return x;
}

// x of one lane (a constant) in every lane.
__device__ __forceinline__ double from_lane(double x, int lane) {
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    return __builtin_bit_cast(double, (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)u, lane) |
                                          (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), lane)
                                              << 32);
}

// x of lane base + lane % kWaves (a power of two).
template <int kWaves>
__device__ __forceinline__ double from_lane_of(double x, int base) {
    return __shfl(x, base + (int)(lane_id() & (kWaves - 1)), 64);
}

// Joins the lanes' running sums: every lane gets the wave's.
__device__ __forceinline__ void wave_join(RunningSum& r, float c2) {
    const float ref = group_reduce<OpMaxNum, 64>(r.ref);
    r.sum = group_reduce<OpSumF, 64>(r.sum * fast_exp2((r.ref - ref) * c2));
    r.ref = ref;
}
// Joins the waves' sums, that of wave w in the lanes w, w + kWaves, ...
template <int kWaves>
__device__ __forceinline__ void join_waves(RunningSum& r, float c2) {
    const float ref = group_reduce<OpMaxNum, kWaves>(r.ref);
    r.sum = group_reduce<OpSumF, kWaves>(r.sum * fast_exp2((r.ref - ref) * c2));
    r.ref = ref;
}

}  // namespace scape
