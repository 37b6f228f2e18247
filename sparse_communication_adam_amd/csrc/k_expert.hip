// k_expert.hip - a router's choices sorted by expert, tokens laid out in that
// order, and the way back with weights and its gradient.
//
//   row[t][j]: the place of choice (t, j) in a stable sort of all by expert
//   y[row[t][j]] = x[t];  out[t] = sum_j w[t][j] y[row[t][j]]
//   dy[row[t][j]] = w[t][j] dout[t];  dw[t][j] = y[row[t][j]] . dout[t]
//
// The moves are bound by their bytes: a wave takes a token, reads its row once
// and goes through its k places, whose numbers are scalars to it.
#include "loss_device.h"

namespace scape {

namespace {

// ---------------------------------------------------------------------------
// The sort: a count, a scan over experts and blocks, and the places.  A wave
// goes through a run of choices 64 at a time; lanes of equal expert find each
// other by ballots over the expert's bits.

__device__ __forceinline__ uint64_t alike(int32_t e, bool on, int bits) {
    uint64_t m = wave_ballot(on);
    for (int b = 0; b < bits; ++b) {
        const uint64_t v = wave_ballot((e >> b) & 1);
        m &= (e >> b) & 1 ? v : ~v;
    }
    return m;
}

// Choice p, or -1 where it is none.
__device__ __forceinline__ int32_t choice(const SortArgs& a, int64_t p, int64_t end) {
    if (p >= end) return -1;
    const int32_t e = a.idx[p];
    return e >= 0 && e < a.experts ? e : -1;
}

// Counts of a wave's run, into its row of LDS.
__device__ __forceinline__ void count_run(const SortArgs& a, uint32_t* row, int64_t p0, int64_t p1) {
    for (int64_t p = p0; p < p1; p += 64) {
        const int32_t e = choice(a, p + lane_id(), p1);
        if (e >= 0) atomicAdd(&row[e], 1u);
    }
}
// The places of a wave's run; row holds each expert's next place.
__device__ __forceinline__ void place_run(const SortArgs& a, volatile uint32_t* row, int64_t p0, int64_t p1) {
    for (int64_t p = p0; p < p1; p += 64) {
        const int64_t at = p + lane_id();
        const int32_t e = choice(a, at, p1);
        const uint64_t m = alike(e, e >= 0, a.bits);
        const uint32_t rank = lanes_below(m);
        // LDS serves a wave in order: all lanes have read before the first of
        // each expert writes
        const uint32_t base = e >= 0 ? row[e] : 0u;
        __builtin_amdgcn_wave_barrier();
        if (e >= 0 && rank == 0) row[e] = base + (uint32_t)__popcll(m);
        __builtin_amdgcn_wave_barrier();
        if (at < p1) a.row[at] = e >= 0 ? (int32_t)(base + rank) : -1;
    }
}

__global__ __launch_bounds__(kBlock) void k_expert_count(SortArgs a) {
    __shared__ uint32_t hist[kMaxExperts];
    for (int32_t e = threadIdx.x; e < a.experts; e += kBlock) hist[e] = 0;
    __syncthreads();
    const int64_t b0 = (int64_t)blockIdx.x * a.run, p0 = b0 + (threadIdx.x >> 6) * (a.run / kWaves);
    int64_t p1 = p0 + a.run / kWaves;
    if (p1 > a.choices) p1 = a.choices;
    count_run(a, hist, p0, p1);
    __syncthreads();
    for (int32_t e = threadIdx.x; e < a.experts; e += kBlock) a.counts[(int64_t)blockIdx.x * a.experts + e] = hist[e];
}

// Counts become first places: of the experts before, and of the blocks before
// within an expert.  One workgroup, a thread an expert.
__global__ __launch_bounds__(kMaxExperts) void k_expert_scan(SortArgs a) {
    __shared__ uint32_t scratch[kMaxExperts / 64];
    const int32_t e = (int32_t)threadIdx.x;
    uint32_t n = 0;
    if (e < a.experts)
        for (int32_t b = 0; b < a.blocks; ++b) n += a.counts[(int64_t)b * a.experts + e];
    uint32_t total, at = block_exclusive_scan_t<kMaxExperts>(n, scratch, &total);
    if (e < a.experts) {
        a.offsets[e] = (int32_t)at;
        for (int32_t b = 0; b < a.blocks; ++b) {
            uint32_t* const c = &a.counts[(int64_t)b * a.experts + e];
            const uint32_t k = *c;
            *c = at;
            at += k;
        }
    }
    if (e == 0) a.offsets[a.experts] = (int32_t)total;
}

__global__ __launch_bounds__(kBlock) void k_expert_place(SortArgs a) {
    __shared__ uint32_t next[kWaves][kMaxExperts];
    const uint32_t wave = threadIdx.x >> 6;
    for (int32_t e = threadIdx.x; e < a.experts; e += kBlock)
        for (int w = 0; w < kWaves; ++w) next[w][e] = 0;
    __syncthreads();
    const int64_t p0 = (int64_t)blockIdx.x * a.run + wave * (a.run / kWaves);
    int64_t p1 = p0 + a.run / kWaves;
    if (p1 > a.choices) p1 = a.choices;
    count_run(a, next[wave], p0, p1);
    __syncthreads();
    for (int32_t e = threadIdx.x; e < a.experts; e += kBlock) {
        uint32_t at = a.counts[(int64_t)blockIdx.x * a.experts + e];
        for (int w = 0; w < kWaves; ++w) {
            const uint32_t n = next[w][e];
            next[w][e] = at;
            at += n;
        }
    }
    __syncthreads();
    place_run(a, next[wave], p0, p1);
}

// ---------------------------------------------------------------------------
// The moves.  Rows lie anywhere: 16 bytes at a time from their first element,
// at whatever alignment, and the rest one element a lane.

typedef uint32_t loose __attribute__((ext_vector_type(4), aligned(2)));
__device__ __forceinline__ gran read16(const char* row, int64_t i) {
    return (gran) * reinterpret_cast<const loose*>(row + i * 16);
}
__device__ __forceinline__ void write16(char* row, int64_t i, const gran& g) {
    *reinterpret_cast<loose*>(row + i * 16) = (loose)g;
}

// Where choice j of token t lies, or -1.
__device__ __forceinline__ int64_t place(const MoveArgs& a, int64_t t, int32_t j) {
    const int32_t r = __builtin_amdgcn_readfirstlane(a.row[t * a.k + j]);
    return r >= 0 && r < a.rows ? r : -1;
}

template <class T>
__global__ __launch_bounds__(kBlock) void k_expert_gather(MoveArgs a) {
    using raw = typename T::raw;
    const uint32_t lane = lane_id();
    const int64_t t = (int64_t)blockIdx.x * kWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (t >= a.tokens) return;
    const char* const x = (const char*)a.x + t * a.ld_x * sizeof(raw);
    const int64_t whole = a.dim / T::kN, rest = whole * T::kN + lane;
    for (int64_t i = lane; i < whole; i += 64) {
        const gran g = read16(x, i);
        for (int32_t j = 0; j < a.k; ++j) {
            const int64_t r = place(a, t, j);
            if (r >= 0) write16((char*)a.y + r * a.ld_y * sizeof(raw), i, g);
        }
    }
    if (rest < a.dim) {
        const raw v = reinterpret_cast<const raw*>(x)[rest];
        for (int32_t j = 0; j < a.k; ++j) {
            const int64_t r = place(a, t, j);
            if (r >= 0) reinterpret_cast<raw*>(a.y)[r * a.ld_y + rest] = v;
        }
    }
}

// Sums in float32 in the order of the choices, rounded once.
template <class T>
__global__ __launch_bounds__(kBlock) void k_expert_combine(MoveArgs a) {
    using raw = typename T::raw;
    const uint32_t lane = lane_id();
    const int64_t t = (int64_t)blockIdx.x * kWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (t >= a.tokens) return;
    char* const out = (char*)a.out + t * a.ld_out * sizeof(raw);
    const int64_t whole = a.dim / T::kN, rest = whole * T::kN + lane;
    for (int64_t i = lane; i < whole; i += 64) {
        float s[T::kN];
#pragma unroll
        for (int e = 0; e < T::kN; ++e) s[e] = 0.0f;
        for (int32_t j = 0; j < a.k; ++j) {
            const int64_t r = place(a, t, j);
            const float w = a.weight ? a.weight[t * a.k + j] : 1.0f;
            if (r < 0 || w == 0.0f) continue;
            const gran g = read16((const char*)a.y + r * a.ld_y * sizeof(raw), i);
#pragma unroll
            for (int e = 0; e < T::kN; ++e) s[e] = __builtin_fmaf(w, T::up(g, e), s[e]);
        }
        write16(out, i, T::down(s));
    }
    if (rest < a.dim) {
        float s = 0.0f;
        for (int32_t j = 0; j < a.k; ++j) {
            const int64_t r = place(a, t, j);
            const float w = a.weight ? a.weight[t * a.k + j] : 1.0f;
            if (r < 0 || w == 0.0f) continue;
            s = __builtin_fmaf(w, T::up1(reinterpret_cast<const raw*>(a.y)[r * a.ld_y + rest]), s);
        }
        reinterpret_cast<raw*>(out)[rest] = T::down1(s);
    }
}

template <class T>
__global__ __launch_bounds__(kBlock) void k_expert_combine_back(MoveArgs a) {
    using raw = typename T::raw;
    const uint32_t lane = lane_id();
    const int64_t t = (int64_t)blockIdx.x * kWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (t >= a.tokens) return;
    const char* const dout = (const char*)a.x + t * a.ld_x * sizeof(raw);
    const int64_t whole = a.dim / T::kN, rest = whole * T::kN + lane;
    for (int32_t j = 0; j < a.k; ++j) {
        const int64_t r = place(a, t, j);
        if (r < 0) {
            if (a.dweight && lane == 0) a.dweight[t * a.k + j] = 0.0f;
            continue;
        }
        const float w = a.weight ? a.weight[t * a.k + j] : 1.0f;
        const char* const y = (const char*)a.y_in + r * a.ld_y_in * sizeof(raw);
        char* const dy = (char*)a.y + r * a.ld_y * sizeof(raw);
        float dot = 0.0f;
        for (int64_t i = lane; i < whole; i += 64) {
            const gran d = read16(dout, i);
            if (a.dweight) {
                const gran g = read16(y, i);
#pragma unroll
                for (int e = 0; e < T::kN; ++e) dot = __builtin_fmaf(T::up(g, e), T::up(d, e), dot);
            }
            float v[T::kN];
#pragma unroll
            for (int e = 0; e < T::kN; ++e) v[e] = w != 0.0f ? w * T::up(d, e) : 0.0f;
            if (a.y) write16(dy, i, T::down(v));
        }
        if (rest < a.dim) {
            const float d = T::up1(reinterpret_cast<const raw*>(dout)[rest]);
            if (a.dweight) dot = __builtin_fmaf(T::up1(reinterpret_cast<const raw*>(y)[rest]), d, dot);
            if (a.y) reinterpret_cast<raw*>(dy)[rest] = T::down1(w != 0.0f ? w * d : 0.0f);
        }
        if (a.dweight) {
            dot = group_reduce<OpSumF, 64>(dot);
            if (lane == 0) a.dweight[t * a.k + j] = dot;
        }
    }
}

#define SCAPE_BY_TYPE(kernel)                                                                                   \
    do {                                                                                                        \
        const dim3 grid((uint32_t)((a.tokens + kWaves - 1) / kWaves)), block(kBlock);                           \
        if (a.dtype == SCAPE_DTYPE_F32) hipLaunchKernelGGL(kernel<F32>, grid, block, 0, s, a);                  \
        else if (a.dtype == SCAPE_DTYPE_BF16) hipLaunchKernelGGL(kernel<BF16>, grid, block, 0, s, a);           \
        else hipLaunchKernelGGL(kernel<F16>, grid, block, 0, s, a);                                             \
        return hipGetLastError();                                                                               \
    } while (0)

}  // namespace

hipError_t launch_expert_sort(hipStream_t s, const SortArgs& a) {
    const dim3 blocks((uint32_t)a.blocks);
    if (a.blocks) hipLaunchKernelGGL(k_expert_count, blocks, dim3(kBlock), 0, s, a);
    hipLaunchKernelGGL(k_expert_scan, dim3(1), dim3(kMaxExperts), 0, s, a);  // offsets are written in any case
    if (a.blocks) hipLaunchKernelGGL(k_expert_place, blocks, dim3(kBlock), 0, s, a);
    return hipGetLastError();
}
hipError_t launch_expert_gather(hipStream_t s, const MoveArgs& a) { SCAPE_BY_TYPE(k_expert_gather); }
hipError_t launch_expert_combine(hipStream_t s, const MoveArgs& a) { SCAPE_BY_TYPE(k_expert_combine); }
hipError_t launch_expert_combine_back(hipStream_t s, const MoveArgs& a) { SCAPE_BY_TYPE(k_expert_combine_back); }

}  // namespace scape
