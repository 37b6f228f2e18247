// k_balance.hip - a router's balance loss and per-expert counts, with the
// gradient of its logits, for gfx950.
//
// Token t has a score p_te for each of E experts: softmax of its logits, or
// their sigmoids s_te over the sum of them.  Over a segment's n valid tokens,
// c_e selections and P_e = sum_t p_te:
//   loss      = alpha E / (k n^2) sum_e c_e P_e
//   d/dl_te   = G p_te (c_e - sum_j p_tj c_j) [(1 - s_te) for sigmoids]
//   G         = dloss alpha E / (k n^2)
// The counts do not depend on the logits' values (a choice has no gradient).
//
// A group of lanes holds a token's logits, each lane 16-byte granules of it,
// so a wave reads a run of tokens as one contiguous piece and the sums over
// experts stay inside the group.  What bounds the kernels is the read of the
// logits (and the write of the gradient) and, as the arrays are small, what a
// launch and a chain of dependent loads take: the loss of 131072x64 f32 (38 MB,
// 5.6 us at the copy's rate) takes 11.6 us and 5.9 for joining the runs, 10.4
// without any arithmetic; the gradient of 65536x256 bf16 (67 MB, 10 us) 17.0 with
// sigmoids, of which the vector units issue for 9; that of 4096x60 f32 4.8.  Sums
// over tokens are held in float32 inside a workgroup's run (off by 4e-8 of the
// loss at 131072x64, half a step being 6e-8) and in float64 across runs, in a
// fixed order.
#include <float.h>

#include "loss_device.h"

namespace scape {

static_assert(SCAPE_BALANCE_MAX_EXPERTS <= 1024, "a thread for each expert in k_balance_finish");

struct Run {
    int32_t seg, t0, t1;  // tokens [t0, t1) of segment seg
};

// Offsets are read clamped to the tokens there are: a wrong one gives wrong
// sums but no access outside.
__device__ __forceinline__ int32_t offset_at(const BalanceArgs& a, int32_t s) {
    if (!a.offsets) return s == 0 ? 0 : (int32_t)a.in.rows;
    const int32_t o = a.offsets[s];
    return o < 0 ? 0 : (o > (int32_t)a.in.rows ? (int32_t)a.in.rows : o);
}
__device__ __forceinline__ int32_t first_slot(const BalanceArgs& a, int32_t s) { return offset_at(a, s) / a.run + s; }

// The run of a slot: the last segment that starts at or before it, found by a
// whole wave, 64 segments (or strides of segments) a step.
__device__ __forceinline__ Run run_of(const BalanceArgs& a, int32_t slot) {
    int32_t lo = 0;
    if (a.offsets) {
        for (int32_t n = a.segments; n > 1;) {
            const int32_t step = (n + 63) / 64, s = lo + (int32_t)lane_id() * step;
            const int32_t at = s < lo + n ? first_slot(a, s) : 0x7FFFFFFF;
            const int32_t below = (int32_t)__popcll(wave_ballot(at <= slot));
            const int32_t k = below > 0 ? below - 1 : 0;
            lo += k * step;
            n -= k * step;
            n = n < step ? n : step;
        }
    }
    const int32_t f = first_slot(a, lo);
    const int64_t t0 = offset_at(a, lo) + (int64_t)(slot - f) * a.run;
    const int64_t end = offset_at(a, lo + 1), t1 = t0 + a.run;
    if (slot < f || t0 >= end) return Run{lo, 0, 0};
    return Run{lo, (int32_t)t0, (int32_t)(t1 < end ? t1 : end)};
}

// A token's logits lie in a group of lanes, lane l with the granules l, l +
// kLanes, ...  The last granule of a row whose length is no multiple of one is
// the row's last 16 bytes, so it overlaps the one before: what it repeats, and
// all of a lane past the row's end, does not count (`keep` has 0 there).  Rows
// and granules may begin anywhere.  kTiny: a row shorter than a granule, one
// lane's, element by element.
template <class T, int kLanes, int kGran, bool kTiny>
struct Lane {
    using raw = typename T::raw;
    int32_t at[kGran], skip[kGran];  // column of element 0, elements that do not count
    gran keep[kGran];
    bool whole;  // all of them do
    __device__ __forceinline__ Lane(uint32_t l, int32_t E) {
        whole = !kTiny;
#pragma unroll
        for (int c = 0; c < kGran; ++c) {
            const int32_t e0 = (int32_t)(l + c * kLanes) * T::kN;
            at[c] = kTiny ? 0 : min(e0, E - T::kN);
            skip[c] = kTiny ? 0 : min(e0 - at[c], T::kN);
            whole = whole && skip[c] == 0;
            keep[c] = gran{0u, 0u, 0u, 0u};
#pragma unroll
            for (int j = 0; j < T::kN; ++j)
                if (kTiny ? j < E : j >= skip[c]) T::set(keep[c], j, (raw)~raw(0));
        }
    }
    __device__ __forceinline__ bool has(int c, int j, int32_t E) const { return kTiny ? j < E : j >= skip[c]; }
    __device__ __forceinline__ void load(const BalanceArgs& a, int32_t t, gran (&g)[kGran]) const {
        const raw* z = static_cast<const raw*>(a.in.z) + (int64_t)t * a.in.ld;
        if constexpr (kTiny) {
#pragma unroll
            for (int j = 0; j < T::kN; ++j) T::set(g[0], j, z[min(j, (int32_t)a.in.cols - 1)]);
        } else {
#pragma unroll
            for (int c = 0; c < kGran; ++c) g[c] = *reinterpret_cast<const loose_gran*>(z + at[c]);
        }
    }
    // -inf where nothing counts; a token that does not count has nothing.
    __device__ __forceinline__ void settle(bool live, gran (&g)[kGran]) const {
        if (!wave_ballot(!live || !whole)) return;
#pragma unroll
        for (int c = 0; c < kGran; ++c)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const uint32_t m = live ? keep[c][q] : 0u;
                g[c][q] = (g[c][q] & m) | (no_entries<T>()[q] & ~m);
            }
    }
};

// Tokens t of a run that a group takes together, their loads all on the way
// before the first is worked on and under no condition: past the run's end
// its last token, which then does not count.
template <int kBatch, class L, int kGran>
__device__ __forceinline__ void load_batch(const BalanceArgs& a, const Run& r, const L& lane, int32_t t, int32_t step,
                                           gran (&g)[kBatch][kGran], bool (&live)[kBatch]) {
    const uint8_t* mask = a.mask ? a.mask : static_cast<const uint8_t*>(a.in.z);  // any byte there is
    uint8_t m[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
        const int32_t at = min(t + i * step, r.t1 - 1);
        m[i] = mask[a.mask ? at : 0];
        lane.load(a, at, g[i]);
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) live[i] = t + i * step < r.t1 && (!a.mask || m[i] != 0);
}

// A token's scores, not yet divided by their sum: w[i], and 1 / sum.  A token
// whose logits are all -inf has 0 for both, and so has one that is not live.
// For sigmoids grad[i] is s (1 - s), the slope of the score.  v_exp_f32 and
// v_rcp_f32 are good to a step of float32.
//
// Sigmoids leave float32's range below about -87.  A token whose sigmoids
// add up to less than 2^-64 has logits below -44: 1 + exp(x) is 1 there to
// float32, so its scores are a softmax and its slopes the scores themselves.
// Above that, what is lost is 2^-62 of the sum at most.
constexpr float kLowSum = 0x1p-64f;
template <class T, int kLanes, int kGran, bool kSoftmax, bool kGrad>
__device__ __forceinline__ float scores(bool live, const gran (&g)[kGran], float (&w)[kGran * T::kN],
                                        float (&grad)[kGran * T::kN]) {
    float sum = 0.0f;
    if constexpr (kSoftmax) {
        float m = granule_max<T>(g[0]);
#pragma unroll
        for (int c = 1; c < kGran; ++c) m = max_nan(m, granule_max<T>(g[c]));
        m = group_reduce<OpMaxF, kLanes>(m);
        const float ref = m == kNegInf ? 0.0f : m;
#pragma unroll
        for (int i = 0; i < kGran * T::kN; ++i) {
            w[i] = fast_exp2(less<T>(g[i / T::kN], i % T::kN, ref) * kLog2e);
            if constexpr (kGrad) grad[i] = w[i];
            sum += w[i];
        }
        sum = group_reduce<OpSumF, kLanes>(sum);
    } else {
#pragma unroll
        for (int i = 0; i < kGran * T::kN; ++i) {
            const float e = fast_exp2(T::up(g[i / T::kN], i % T::kN) * -kLog2e);  // inf for -inf: a score of 0
            w[i] = __builtin_amdgcn_rcpf(1.0f + e);
            if constexpr (kGrad) grad[i] = w[i] * (fminf(e, FLT_MAX) * w[i]);  // 0 for -inf, not inf times 0
            sum += w[i];
        }
        sum = group_reduce<OpSumF, kLanes>(sum);
        if (__builtin_expect(wave_ballot(live && sum < kLowSum) != 0, 0)) {
            const bool low = sum < kLowSum;
            gran x[kGran];
#pragma unroll
            for (int c = 0; c < kGran; ++c) forget_unpacked(x[c] = g[c]);
            float m = granule_max<T>(x[0]), of = 0.0f;
#pragma unroll
            for (int c = 1; c < kGran; ++c) m = max_nan(m, granule_max<T>(x[c]));
            m = group_reduce<OpMaxF, kLanes>(m);
            const float ref = m == kNegInf ? 0.0f : m;
#pragma unroll
            for (int i = 0; i < kGran * T::kN; ++i) {
                const float y = fast_exp2((T::up(x[i / T::kN], i % T::kN) - ref) * kLog2e);
                w[i] = low ? y : w[i];
                if constexpr (kGrad) grad[i] = low ? y : grad[i];
                of += y;
            }
            of = group_reduce<OpSumF, kLanes>(of);
            sum = low ? of : sum;
        }
    }
    return sum == 0.0f ? 0.0f : __builtin_amdgcn_rcpf(sum);
}

__device__ __forceinline__ float balance_loss_of(double dot, int32_t n, int32_t E, int32_t k, float alpha) {
    if (n <= 0) return 0.0f;
    return (float)((double)alpha * E / ((double)k * n * n) * dot);
}

// The sums over a run of tokens.  kWhole: a run is a segment, and what is left
// to do for it is done here (2000x8 bf16 in 7 segments: 8.8 us; the two
// launches took 11.5).  1024 threads, one workgroup a CU: with 512 and twice
// the runs it takes as long, but the join of twice the runs 1.3 us more.
template <class T, int kLanes, int kGran, bool kTiny, bool kSoftmax, bool kWhole>
__global__ __launch_bounds__(kForwardThreads) void k_balance_runs(BalanceArgs a) {
    constexpr int kV = kGran * T::kN, kTokens = 64 / kLanes, kNW = kForwardThreads / 64, kStep = kNW * kTokens;
    constexpr int kBatch = kGran == 1 ? 8 : kV == 8 ? 4 : 2;
    __shared__ float part[kNW / 2][SCAPE_BALANCE_MAX_EXPERTS];
    __shared__ int32_t hist[SCAPE_BALANCE_MAX_EXPERTS];
    __shared__ int32_t s_tok;
    __shared__ double wd[kNW];
    const uint32_t tid = threadIdx.x, lane = lane_id(), wave = tid / 64, l = lane % kLanes;
    const int32_t E = (int32_t)a.in.cols;
    Run r;
    if constexpr (kWhole)
        r = Run{(int32_t)blockIdx.x, offset_at(a, (int32_t)blockIdx.x), offset_at(a, (int32_t)blockIdx.x + 1)};
    else
        r = run_of(a, (int32_t)blockIdx.x);
    if (r.t0 >= r.t1 && !kWhole) return;
    for (int32_t e = (int32_t)tid; e < E; e += kForwardThreads) hist[e] = 0;
    if (tid == 0) s_tok = 0;
    __syncthreads();

    // the choices, four a thread at a time; the first four are on their way
    // before the logits are
    const int64_t c0 = (int64_t)r.t0 * a.k;
    const uint32_t choices = r.t1 > r.t0 ? (uint32_t)((int64_t)(r.t1 - r.t0) * a.k) : 0u;
    int32_t chosen[4];
    uint8_t counted[4];
    auto load_choices = [&](uint32_t f0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t f = min(f0 + i * kForwardThreads, choices - 1);
            chosen[i] = a.idx[c0 + f];
            counted[i] = a.mask ? a.mask[r.t0 + (int32_t)(f / (uint32_t)a.k)] : 1;
        }
    };
    if (choices > 0) load_choices(tid);

    float acc[kV];
#pragma unroll
    for (int i = 0; i < kV; ++i) acc[i] = 0.0f;
    const Lane<T, kLanes, kGran, kTiny> mine(l, E);
    uint32_t tokens = 0;
    for (int32_t b = r.t0 + (int32_t)(wave * kTokens + lane / kLanes); b < r.t1; b += kStep * kBatch) {
        gran g[kBatch][kGran];
        bool live[kBatch];
        load_batch<kBatch>(a, r, mine, b, kStep, g, live);
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            mine.settle(live[i], g[i]);
            float w[kV], none[kV];
            // a token that does not count: 0
            const float inv = scores<T, kLanes, kGran, kSoftmax, false>(live[i], g[i], w, none);
#pragma unroll
            for (int v = 0; v < kV; ++v) acc[v] = __builtin_fmaf(w[v], inv, acc[v]);
            tokens += live[i] && l == 0 ? 1u : 0u;
        }
    }
    for (uint32_t f0 = tid; f0 < choices;) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (f0 + i * kForwardThreads < choices && chosen[i] >= 0 && chosen[i] < E && counted[i] != 0)
                atomicAdd(&hist[chosen[i]], 1);
        f0 += kForwardThreads * 4;
        if (f0 < choices) load_choices(f0);
    }
    // the wave's groups, then the waves, one half of them onto the other first
#pragma unroll
    for (int i = 0; i < kV; ++i)
#pragma unroll
        for (int d = kLanes; d < 64; d <<= 1) acc[i] += __shfl_xor(acc[i], d, 64);
    tokens = wave_sum(tokens);
    if (lane == 0 && tokens) atomicAdd(&s_tok, (int32_t)tokens);
    auto columns = [&](auto f) {
        if (lane < kLanes) {
#pragma unroll
            for (int i = 0; i < kV; ++i)
                if (mine.has(i / T::kN, i % T::kN, E)) f(mine.at[i / T::kN] + i % T::kN, acc[i]);
        }
    };
    if (wave >= kNW / 2) columns([&](int32_t e, float x) { part[wave - kNW / 2][e] = x; });
    __syncthreads();
    if (wave < kNW / 2) columns([&](int32_t e, float x) { part[wave][e] += x; });
    __syncthreads();
    const int64_t o = (int64_t)blockIdx.x * E;
    double dot = 0.0;
    for (int32_t e = (int32_t)tid; e < E; e += kForwardThreads) {
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < kNW / 2; ++w) s += part[w][e];
        if constexpr (kWhole) {
            a.counts[o + e] = hist[e];
            a.psum[o + e] = s;
            dot = (double)hist[e] * (double)s;
        } else {
            a.part[o + e] = make_float2(s, __int_as_float(hist[e]));
        }
    }
    if constexpr (kWhole) {
        dot = wave_sum_f64(dot);
        if (lane == 0) wd[wave] = dot;
        __syncthreads();
        if (tid == 0) {
            a.n_tok[blockIdx.x] = s_tok;
            double t = 0.0;
            for (int w = 0; w < kNW; ++w) t += wd[w];
            if (a.loss) a.loss[blockIdx.x] = balance_loss_of(t, s_tok, E, a.k, a.alpha);
        }
    } else if (tid == 0) {
        a.part_tok[blockIdx.x] = s_tok;
    }
}

// One workgroup a segment: the sums over its runs, and the loss.  A column's
// runs are dealt out over as many threads as there are columns to spare, sixteen
// loads of each in flight, and joined in order.
constexpr int kFinishThreads = 1024;
__global__ __launch_bounds__(kFinishThreads) void k_balance_finish(BalanceArgs a) {
    __shared__ double ps[kFinishThreads];
    __shared__ int32_t cs[kFinishThreads];
    __shared__ double wd[kFinishThreads / 64];
    __shared__ int32_t s_tok;
    const int32_t tid = (int32_t)threadIdx.x, E = (int32_t)a.in.cols, s = (int32_t)blockIdx.x;
    const int32_t len = offset_at(a, s + 1) - offset_at(a, s);
    const int32_t base = first_slot(a, s);
    int32_t runs = len > 0 ? (len + a.run - 1) / a.run : 0;
    if (runs > a.slots - base) runs = a.slots - base;
    if (tid == 0) s_tok = 0;
    __syncthreads();
    int32_t tok = 0;
    for (int32_t c = tid; c < runs; c += kFinishThreads) tok += a.part_tok[base + c];
    if (tok) atomicAdd(&s_tok, tok);
    const int32_t deep = kFinishThreads / E;  // E <= kFinishThreads
    const int32_t e = tid % E, d = tid / E;
    double p = 0.0, dot = 0.0;
    int32_t n = 0;
    if (d < deep) {
        constexpr int kBatch = 16;
        for (int32_t c0 = d; c0 < runs; c0 += deep * kBatch) {
            float2 x[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int32_t c = c0 + i * deep;
                x[i] = a.part[(int64_t)(base + (c < runs ? c : c0)) * E + e];
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
                if (c0 + i * deep < runs) {
                    p += (double)x[i].x;
                    n += __float_as_int(x[i].y);
                }
        }
    }
    ps[tid] = p;
    cs[tid] = n;
    __syncthreads();
    if (d == 0) {
        for (int32_t i = 1; i < deep; ++i) {
            p += ps[i * E + e];
            n += cs[i * E + e];
        }
        a.counts[(int64_t)s * E + e] = n;
        a.psum[(int64_t)s * E + e] = (float)p;
        dot = (double)n * p;
    }
    dot = wave_sum_f64(dot);
    if ((tid & 63) == 0) wd[tid / 64] = dot;
    __syncthreads();
    if (tid == 0) {
        a.n_tok[s] = s_tok;
        double t = 0.0;
        for (int w = 0; w < kFinishThreads / 64; ++w) t += wd[w];
        if (a.loss) a.loss[s] = balance_loss_of(t, s_tok, E, a.k, a.alpha);
    }
}

__global__ __launch_bounds__(kBlock) void k_balance_loss(const int32_t* counts, const float* psum,
                                                         const int32_t* n_tok, int32_t E, int32_t k, float alpha,
                                                         float* loss) {
    __shared__ double wd[kWaves];
    const int64_t o = (int64_t)blockIdx.x * E;
    double dot = 0.0;
    for (int32_t e = (int32_t)threadIdx.x; e < E; e += kBlock) dot += (double)counts[o + e] * (double)psum[o + e];
    dot = wave_sum_f64(dot);
    if ((threadIdx.x & 63) == 0) wd[threadIdx.x / 64] = dot;
    __syncthreads();
    if (threadIdx.x == 0) {
        double t = 0.0;
        for (int w = 0; w < kWaves; ++w) t += wd[w];
        loss[blockIdx.x] = balance_loss_of(t, n_tok[blockIdx.x], E, k, alpha);
    }
}

// The gradient: a batch of four tokens a group, all loads first (65536x256 bf16
// with two 17.6 us, four 17.5, eight 19.4).
template <class T, int kLanes, int kGran, bool kTiny, bool kSoftmax>
__global__ __launch_bounds__(kBackwardThreads) void k_balance_grad(BalanceArgs a) {
    using raw = typename T::raw;
    constexpr int kV = kGran * T::kN, kTokens = 64 / kLanes, kStep = kBackwardThreads / 64 * kTokens;
    constexpr int kBatch = kGran == 1 ? kBackwardBatch : kGran == 2 ? kBackwardBatch / 2 : 1;
    const uint32_t lane = lane_id(), wave = threadIdx.x / 64, l = lane % kLanes;
    const int32_t E = (int32_t)a.in.cols;
    const Run r = run_of(a, (int32_t)blockIdx.x);
    if (r.t0 >= r.t1) return;
    const Lane<T, kLanes, kGran, kTiny> mine(l, E);
    float c[kV];
#pragma unroll
    for (int i = 0; i < kV; ++i) {
        const int32_t e = min(mine.at[i / T::kN] + i % T::kN, E - 1);
        c[i] = (float)a.counts[(int64_t)r.seg * E + e];
    }
    const int32_t n = a.n_tok[r.seg];
    const float up = a.dloss ? a.dloss[r.seg] : 1.0f;
    const float G = n > 0 ? (float)((double)up * (double)a.alpha * E / ((double)a.k * n * n)) : 0.0f;
    for (int32_t b = r.t0 + (int32_t)(wave * kTokens + lane / kLanes); b < r.t1; b += kStep * kBatch) {
        gran g[kBatch][kGran];
        bool live[kBatch];
        load_batch<kBatch>(a, r, mine, b, kStep, g, live);
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int32_t t = b + i * kStep;
            mine.settle(live[i], g[i]);
            float w[kV], grad[kV];
            const float inv = scores<T, kLanes, kGran, kSoftmax, true>(live[i], g[i], w, grad);
            float dot = 0.0f;
#pragma unroll
            for (int v = 0; v < kV; ++v) dot = __builtin_fmaf(w[v], c[v], dot);
            dot = group_reduce<OpSumF, kLanes>(dot) * inv;
            const float up1 = live[i] ? G * inv : 0.0f, less = up1 * dot;
            if (t < r.t1) {
                raw* dz = static_cast<raw*>(a.dz) + (int64_t)t * a.ld_dz;
#pragma unroll
                for (int q = 0; q < kGran; ++q) {
                    float v[T::kN];
#pragma unroll
                    for (int j = 0; j < T::kN; ++j) {
                        const int x = q * T::kN + j;
                        v[j] = grad[x] * __builtin_fmaf(c[x], up1, -less);
                    }
                    if (!kTiny && mine.skip[q] == 0) {
                        *reinterpret_cast<loose_gran*>(dz + mine.at[q]) = (loose_gran)T::down(v);
                    } else {
#pragma unroll
                        for (int j = 0; j < T::kN; ++j)
                            if (mine.has(q, j, E)) dz[mine.at[q] + j] = T::down1(v[j]);
                    }
                }
            }
        }
    }
}

// A kernel for each score: with both in one, the sigmoids' low tokens cost the
// softmax too (gradient of 65536x256 f16, replayed: 14.2 us before there were
// any, 14.8 in one kernel, 13.8 in one of its own).
template <class T, int kLanes, int kGran, bool kTiny, bool kSoftmax>
static void runs_or_grad_of(hipStream_t s, const BalanceArgs& a) {
    const dim3 grid((uint32_t)a.slots);
    if (a.dz)
        hipLaunchKernelGGL((k_balance_grad<T, kLanes, kGran, kTiny, kSoftmax>), grid, dim3(kBackwardThreads), 0, s, a);
    else if (a.whole)
        hipLaunchKernelGGL((k_balance_runs<T, kLanes, kGran, kTiny, kSoftmax, true>), grid, dim3(kForwardThreads), 0, s, a);
    else
        hipLaunchKernelGGL((k_balance_runs<T, kLanes, kGran, kTiny, kSoftmax, false>), grid, dim3(kForwardThreads), 0, s, a);
}
template <class T, int kLanes, int kGran, bool kTiny>
static void runs_or_grad(hipStream_t s, const BalanceArgs& a) {
    if (a.score == SCAPE_SCORE_SOFTMAX)
        runs_or_grad_of<T, kLanes, kGran, kTiny, true>(s, a);
    else
        runs_or_grad_of<T, kLanes, kGran, kTiny, false>(s, a);
}

template <class T>
static hipError_t balance_typed(hipStream_t s, const BalanceArgs& a) {
    const int64_t g = (a.in.cols + T::kN - 1) / T::kN;  // granules a token
    constexpr int kTwo = T::kN == 4 ? 2 : 1;  // eight elements a lane, where there are as many
    if (a.in.cols < T::kN) runs_or_grad<T, 1, 1, true>(s, a);
    else switch (balance_lanes(a.in.dtype, a.in.cols)) {
        case 1: runs_or_grad<T, 1, 1, false>(s, a); break;
        case 4: runs_or_grad<T, 4, 1, false>(s, a); break;
        case 8: runs_or_grad<T, 8, kTwo, false>(s, a); break;
        case 16: runs_or_grad<T, 16, kTwo, false>(s, a); break;
        case 32: runs_or_grad<T, 32, kTwo, false>(s, a); break;
        default:
            if (g <= 64 * kTwo) runs_or_grad<T, 64, kTwo, false>(s, a);
            else runs_or_grad<T, 64, 2 * kTwo, false>(s, a);
    }
    return hipGetLastError();
}

static hipError_t balance_any(hipStream_t s, const BalanceArgs& a) {
    if (a.in.dtype == SCAPE_DTYPE_F32) return balance_typed<F32>(s, a);
    if (a.in.dtype == SCAPE_DTYPE_BF16) return balance_typed<BF16>(s, a);
    return balance_typed<F16>(s, a);
}

hipError_t launch_balance_forward(hipStream_t s, const BalanceArgs& a) {
    if (a.in.rows > 0) {
        const hipError_t e = balance_any(s, a);
        if (e != hipSuccess || a.whole) return e;
    }
    hipLaunchKernelGGL(k_balance_finish, dim3((uint32_t)a.segments), dim3(kFinishThreads), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_balance_loss(hipStream_t s, const int32_t* counts, const float* psum, const int32_t* n_tok,
                               int32_t segments, int32_t experts, int32_t k, float alpha, float* loss) {
    hipLaunchKernelGGL(k_balance_loss, dim3((uint32_t)segments), dim3(kBlock), 0, s, counts, psum, n_tok, experts, k,
                       alpha, loss);
    return hipGetLastError();
}

hipError_t launch_balance_backward(hipStream_t s, const BalanceArgs& a) { return balance_any(s, a); }

}  // namespace scape
