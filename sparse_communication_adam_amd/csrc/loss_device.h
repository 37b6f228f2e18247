// loss_device.h - device helpers of the row kernels (k_topk.hip,
// k_distill.hip, k_balance.hip): the three logit types as 16-byte granules,
// and reductions over a wave and a workgroup.
#pragma once

#include "loss_internal.h"
#include "scape_device.h"

namespace scape {

typedef uint32_t gran __attribute__((ext_vector_type(4)));  // 16 bytes of a row

constexpr float kNegInf = -__builtin_inff();
constexpr float kLog2e = 1.44269504088896340736f;
constexpr double kLn2 = 0.693147180559945309417;

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
// values, k of them a row).
__device__ __forceinline__ float load_any(const void* p, int32_t dtype, int64_t i) {
    if (dtype == SCAPE_DTYPE_F32) return static_cast<const float*>(p)[i];
    const uint16_t r = static_cast<const uint16_t*>(p)[i];
    return dtype == SCAPE_DTYPE_BF16 ? BF16::up1(r) : F16::up1(r);
}

// A row starts anywhere, its granules lie on 16-byte boundaries: element e of
// the row is element (e + lead) % N of granule (e + lead) / N.  Only the first
// and the last granule can reach past the row; those are read and written
// element by element, so nothing outside the row is touched.
template <class T>
__device__ __forceinline__ int row_lead(const void* row) {
    return (int)(((uintptr_t)row & 15u) / sizeof(typename T::raw));
}

template <class T>
__device__ __forceinline__ gran load_granule(const typename T::raw* row, int64_t e0, int64_t n) {
    if (e0 >= 0 && e0 + T::kN <= n) return *reinterpret_cast<const gran*>(row + e0);
    gran g = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int j = 0; j < T::kN; ++j) {
        const int64_t e = e0 + j;
        T::set(g, j, (e >= 0 && e < n) ? row[e] : (typename T::raw)T::kNegInfBits);
    }
    return g;
}

// vec: the destination row has the source row's lead.
template <class T>
__device__ __forceinline__ void store_granule(typename T::raw* row, int64_t e0, int64_t n, bool vec, const gran& g) {
    if (vec && e0 >= 0 && e0 + T::kN <= n) {
        *reinterpret_cast<gran*>(row + e0) = g;
        return;
    }
#pragma unroll
    for (int j = 0; j < T::kN; ++j) {
        const int64_t e = e0 + j;
        if (e >= 0 && e < n)
            row[e] = sizeof(typename T::raw) == 4 ? (typename T::raw)g[j & 3]
                                                  : (typename T::raw)((j & 1) ? g[(j >> 1) & 3] >> 16 : g[(j >> 1) & 3]);
    }
}

__device__ __forceinline__ float fast_exp2(float x) { return __builtin_amdgcn_exp2f(x); }  // v_exp_f32

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
    static __device__ __forceinline__ float f(float a, float b) { return fmaxf(a, b); }
};
struct OpSumF {
    static __device__ __forceinline__ float f(float a, float b) { return a + b; }
};
struct OpMaxU {
    static __device__ __forceinline__ uint32_t f(uint32_t a, uint32_t b) { return a > b ? a : b; }
};
struct OpSumU {
    static __device__ __forceinline__ uint32_t f(uint32_t a, uint32_t b) { return a + b; }
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

__device__ __forceinline__ double wave_sum_f64(double x) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) x += __shfl_xor(x, d, 64);
    return x;
}

}  // namespace scape
