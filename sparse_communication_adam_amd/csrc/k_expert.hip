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
// The sort: a count for each block, and the places.  A wave goes through a run
// of choices 64 at a time; lanes of equal expert find each other by ballots over
// the expert's bits.

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

// Counts of a wave's run, into its row of LDS; kAhead loads are on their way.
constexpr int kAhead = 8;
__device__ __forceinline__ void count_run(const SortArgs& a, uint32_t* row, int64_t p0, int64_t p1) {
    for (int64_t p = p0; p < p1; p += 64 * kAhead) {
        int32_t e[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) e[i] = choice(a, p + i * 64 + lane_id(), p1);
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (e[i] >= 0) atomicAdd(&row[e[i]], 1u);
    }
}
// The places of a wave's run; row holds each expert's next place.
__device__ __forceinline__ void place_run(const SortArgs& a, volatile uint32_t* row, int64_t p0, int64_t p1) {
    for (int64_t p = p0; p < p1; p += 64 * kAhead) {
        int32_t e[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) e[i] = choice(a, p + i * 64 + lane_id(), p1);
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (p + i * 64 >= p1) break;
            const int64_t at = p + i * 64 + lane_id();
            const uint64_t m = alike(e[i], e[i] >= 0, a.bits);
            const uint32_t rank = lanes_below(m);
            // LDS serves a wave in order: all lanes have read before the first of
            // each expert writes
            const uint32_t base = e[i] >= 0 ? row[e[i]] : 0u;
            __builtin_amdgcn_wave_barrier();
            if (e[i] >= 0 && rank == 0) row[e[i]] = base + (uint32_t)__popcll(m);
            __builtin_amdgcn_wave_barrier();
            if (at < p1) a.row[at] = e[i] >= 0 ? (int32_t)(base + rank) : -1;
        }
    }
}

// A wave's run of choices: a quarter of the block's.
__device__ __forceinline__ void run_of(const SortArgs& a, int64_t& p0, int64_t& p1) {
    p0 = (int64_t)blockIdx.x * a.run + (threadIdx.x >> 6) * (a.run / kWaves);
    p1 = p0 + a.run / kWaves;
    if (p1 > a.choices) p1 = a.choices;
}

__global__ __launch_bounds__(kBlock) void k_expert_count(SortArgs a) {
    __shared__ uint32_t hist[kMaxExperts];
    for (int32_t e = threadIdx.x; e < a.experts; e += kBlock) hist[e] = 0;
    __syncthreads();
    int64_t p0, p1;
    run_of(a, p0, p1);
    count_run(a, hist, p0, p1);
    __syncthreads();
    for (int32_t e = threadIdx.x; e < a.experts; e += kBlock) a.counts[(int64_t)blockIdx.x * a.experts + e] = hist[e];
}

// The places.  Each block sums the counts of all blocks, and of those before
// it, for itself: they are few (a block for 2048 choices) and in the caches,
// and a launch between the count and this costs more.  131072 choices of 64
// experts take 5.0 + 8.3 us in a trace: two launches, and in each a chain of the
// choices' load, LDS and the counts; the bytes (1 MB) are nothing.  One block
// alone needs no count before it (one token: 3.2 us, a launch).  Of very many
// choices and experts the counts are what takes the time: 1200000 choices of 512
// experts 5.8 + 44 us, 469 blocks reading 469 x 512 counts each.
__global__ __launch_bounds__(kBlock) void k_expert_place(SortArgs a) {
    __shared__ uint32_t next[kWaves][kMaxExperts], before[kMaxExperts], total[kMaxExperts], scratch[kWaves];
    const uint32_t tid = threadIdx.x, wave = tid >> 6;
    for (int32_t e = tid; e < a.experts; e += kBlock) {
        for (int w = 0; w < kWaves; ++w) next[w][e] = 0;
        before[e] = total[e] = 0;
    }
    __syncthreads();
    int64_t p0, p1;
    run_of(a, p0, p1);
    count_run(a, next[wave], p0, p1);
    if (a.blocks > 1) {
        // few experts: several threads share one's blocks
        const int32_t parts = a.experts <= kBlock / 4 ? 4 : a.experts <= kBlock / 2 ? 2 : 1, lanes = kBlock / parts;
        const int32_t part = (int32_t)tid / lanes;
        for (int32_t e = (int32_t)tid % lanes; e < a.experts; e += lanes) {
            uint32_t all = 0, here = 0;
#pragma unroll 16
            for (int32_t b = part; b < a.blocks; b += parts) {
                const uint32_t n = a.counts[(int64_t)b * a.experts + e];
                all += n;
                here += b < (int32_t)blockIdx.x ? n : 0u;
            }
            atomicAdd(&total[e], all);
            atomicAdd(&before[e], here);
        }
    }
    __syncthreads();
    // first places: a thread has kMaxExperts / kBlock experts in a row
    constexpr int kEach = kMaxExperts / kBlock;
    uint32_t n[kEach], sum = 0;
    for (int i = 0; i < kEach; ++i) {
        const int32_t e = (int32_t)tid * kEach + i;
        n[i] = 0;
        if (e < a.experts) {
            n[i] = total[e];
            if (a.blocks == 1)
                for (int w = 0; w < kWaves; ++w) n[i] += next[w][e];
        }
        sum += n[i];
    }
    uint32_t all, at = block_exclusive_scan(sum, scratch, &all);
    for (int i = 0; i < kEach; ++i) {
        const int32_t e = (int32_t)tid * kEach + i;
        if (e < a.experts) {
            if (blockIdx.x == 0) a.offsets[e] = (int32_t)at;
            uint32_t place = at + before[e];
            for (int w = 0; w < kWaves; ++w) {
                const uint32_t c = next[w][e];
                next[w][e] = place;
                place += c;
            }
        }
        at += n[i];
    }
    if (blockIdx.x == 0 && tid == 0) a.offsets[a.experts] = (int32_t)all;
    __syncthreads();
    place_run(a, next[wave], p0, p1);
}

// ---------------------------------------------------------------------------
// The moves.  A wave takes a token.  Its places and weights are loaded once, a
// lane each, and handed round as scalars.  Rows lie anywhere: 16 bytes at a time
// from their first element, at whatever alignment.  Of a row that is no whole
// number of granules the last one ends with the row and repeats elements of the
// one before it, which get the same values twice (16384x257 f16, k = 8, one
// element a lane instead: combine 29 us).  Lanes behind a row's last granule load
// it again and store nothing.  Rows of less than a granule go an element a lane.

typedef uint32_t loose __attribute__((ext_vector_type(4), aligned(2)));
__device__ __forceinline__ gran read16(const void* row, uint32_t byte) {
    return (gran)__builtin_nontemporal_load(reinterpret_cast<const loose*>(static_cast<const char*>(row) + byte));
}
__device__ __forceinline__ gran read16_again(const void* row, uint32_t byte) {  // a row that is read more than once
    return (gran)*reinterpret_cast<const loose*>(static_cast<const char*>(row) + byte);
}
__device__ __forceinline__ void write16(void* row, uint32_t byte, const gran& g) {
    __builtin_nontemporal_store((loose)g, reinterpret_cast<loose*>(static_cast<char*>(row) + byte));
}

// Up to 64 choices of a token from j0 on, a lane each: the place (-1: none) and
// the weight.
struct Held {
    int32_t row;
    float weight;
    __device__ __forceinline__ void load(const MoveArgs& a, int64_t t, int32_t j0) {
        const int32_t j = j0 + (int32_t)lane_id();
        row = -1;
        weight = 1.0f;
        if (j < a.k) {
            row = a.row[t * a.k + j];
            if (a.weight) weight = a.weight[t * a.k + j];
        }
        if (row < 0 || row >= a.rows) row = -1;
    }
    __device__ __forceinline__ int32_t place(int j) const { return __builtin_amdgcn_readlane(row, j); }
    __device__ __forceinline__ float factor(int j) const {
        return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, weight), j));
    }
};
__device__ __forceinline__ int64_t token_of_wave() {
    return (int64_t)blockIdx.x * kWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
}

// A row's granules: how many, and where the last one begins.
struct Span {
    int64_t granules;
    uint32_t last;
};
template <class T>
__device__ __forceinline__ Span span_of(const MoveArgs& a) {
    constexpr uint32_t kSize = 16 / T::kN;
    return a.dim < T::kN ? Span{0, 0} : Span{(a.dim + T::kN - 1) / T::kN, (uint32_t)a.dim * kSize - 16u};
}
// kB granules at a time for each lane.
template <class T, int kB>
struct Row {
    static __device__ __forceinline__ uint32_t byte(const Span& s, int64_t i) {  // of granule i, or of the last
        const uint32_t b = (uint32_t)i * 16u;
        return b < s.last ? b : s.last;
    }
    static __device__ __forceinline__ void load(gran (&g)[kB], const void* row, const Span& s, int64_t i0) {
#pragma unroll
        for (int b = 0; b < kB; ++b) g[b] = read16(row, byte(s, i0 + b * 64));
    }
    static __device__ __forceinline__ void load_again(gran (&g)[kB], const void* row, const Span& s, int64_t i0) {
#pragma unroll
        for (int b = 0; b < kB; ++b) g[b] = read16_again(row, byte(s, i0 + b * 64));
    }
    static __device__ __forceinline__ void store(const gran (&g)[kB], void* row, const Span& s, int64_t i0) {
#pragma unroll
        for (int b = 0; b < kB; ++b)
            if (i0 + b * 64 < s.granules) write16(row, byte(s, i0 + b * 64), g[b]);
    }
};
// g . d of granule i, without what the granule before the last has of it.
template <class T>
__device__ __forceinline__ float dot_of(const gran& g, const gran& d, const Span& s, int64_t i) {
    float part = 0.0f;
    if (s.last + 16u == (uint32_t)s.granules * 16u) {
#pragma unroll
        for (int e = 0; e < T::kN; ++e) part = __builtin_fmaf(T::up(g, e), T::up(d, e), part);
    } else {
        const uint32_t back = i + 1 == s.granules ? (uint32_t)i * 16u - s.last : 0u;
#pragma unroll
        for (int e = 0; e < T::kN; ++e) {
            const bool first = (uint32_t)e * (16 / T::kN) >= back;
            part = __builtin_fmaf(first ? T::up(g, e) : 0.0f, first ? T::up(d, e) : 0.0f, part);
        }
    }
    return i < s.granules ? part : 0.0f;
}

// kB granules of the token are in registers while they go to its places.  Bound
// by the writes: 16384x2048 bf16, k = 8, 102 us in a trace, 5.9 TB/s of 6.7 that a
// copy reaches; the workgroups' rows lie all over y.
template <class T, int kB>
__global__ __launch_bounds__(kBlock) void k_expert_gather(MoveArgs a) {
    using raw = typename T::raw;
    const uint32_t lane = lane_id();
    const int64_t t = token_of_wave();
    if (t >= a.tokens) return;
    const raw* const x = static_cast<const raw*>(a.x) + t * a.ld_x;
    raw* const y = static_cast<raw*>(a.y);
    const Span s = span_of<T>(a);
    Held h;
    for (int32_t j0 = 0; j0 < a.k; j0 += 64) {
        h.load(a, t, j0);
        const int n = a.k - j0 < 64 ? a.k - j0 : 64;
        for (int64_t i = lane; i - lane < s.granules; i += 64 * kB) {
            gran g[kB];
            Row<T, kB>::load_again(g, x, s, i);
            for (int j = 0; j < n; ++j) {
                const int64_t r = h.place(j);
                if (r >= 0) Row<T, kB>::store(g, y + r * a.ld_y, s, i);
            }
        }
        if (s.granules == 0 && lane < a.dim) {
            const raw v = x[lane];
            for (int j = 0; j < n; ++j) {
                const int64_t r = h.place(j);
                if (r >= 0) y[r * a.ld_y + lane] = v;
            }
        }
    }
}

// Sums in float32 in the order of the choices, rounded once.  kJ rows are on
// their way at a time; a place that is none, or has weight 0, reads a granule of
// zeros instead, so that no load stands under a condition.  Bound by the reads of
// rows all over y: 16384x2048 bf16, k = 8, 102 us in a trace, 5.9 TB/s.
template <class T, int kB, int kJ>
__global__ __launch_bounds__(kBlock) void k_expert_combine(MoveArgs a) {
    using raw = typename T::raw;
    const uint32_t lane = lane_id();
    const int64_t t = token_of_wave();
    if (t >= a.tokens) return;
    raw* const out = static_cast<raw*>(a.out) + t * a.ld_out;
    const raw* const y = static_cast<const raw*>(a.y);
    const Span span = span_of<T>(a);
    Held h;
    if (a.k <= 64) h.load(a, t, 0);
    for (int64_t i = lane; i - lane < span.granules; i += 64 * kB) {
        float s[kB][T::kN];
#pragma unroll
        for (int b = 0; b < kB; ++b)
#pragma unroll
            for (int e = 0; e < T::kN; ++e) s[b][e] = 0.0f;
        for (int32_t j0 = 0; j0 < a.k; j0 += kJ) {
            if (a.k > 64 && (j0 & 63) == 0) h.load(a, t, j0);
            gran g[kJ][kB];
            float w[kJ];
#pragma unroll
            for (int j = 0; j < kJ; ++j) {  // lanes behind the last choice hold none
                const int64_t r = h.place((j0 + j) & 63);
                w[j] = h.factor((j0 + j) & 63);
                const bool on = r >= 0 && w[j] != 0.0f && j0 + j < a.k;
                const void* const row = on ? static_cast<const void*>(y + r * a.ld_y) : &g_no_granule;
                if (!on) w[j] = 0.0f;
#pragma unroll
                for (int b = 0; b < kB; ++b) g[j][b] = read16(row, on ? Row<T, kB>::byte(span, i + b * 64) : 0u);
            }
#pragma unroll
            for (int j = 0; j < kJ; ++j)
#pragma unroll
                for (int b = 0; b < kB; ++b)
#pragma unroll
                    for (int e = 0; e < T::kN; ++e) s[b][e] = __builtin_fmaf(w[j], T::up(g[j][b], e), s[b][e]);
        }
#pragma unroll
        for (int b = 0; b < kB; ++b)
            if (i + b * 64 < span.granules) write16(out, Row<T, kB>::byte(span, i + b * 64), T::down(s[b]));
    }
    if (span.granules == 0) {
        float s = 0.0f;
        for (int32_t j = 0; j < a.k; ++j) {
            if ((a.k > 64 && (j & 63) == 0)) h.load(a, t, j);
            const int64_t r = h.place(j & 63);
            const float w = h.factor(j & 63);
            if (r < 0 || w == 0.0f || lane >= a.dim) continue;
            s = __builtin_fmaf(w, T::up1(y[r * a.ld_y + lane]), s);
        }
        if (lane < a.dim) out[lane] = T::down1(s);
    }
}

// A workgroup takes a token and its waves the token's choices in turn (a wave
// for a token is slower for few tokens: 2000x1536 f16, k = 4, 12.9 us and 15.5).
// Bound by reading y and writing dy: 8192x4096 bf16, k = 8, 208 us in a trace, 5.5
// TB/s.
// dout is in registers where kB granules a lane hold it all, else it is read for
// every place; the waves' reads of it meet in the L1.  A grid's axis counts its
// threads in 32 bits, so more tokens than that lie along the other axis.
constexpr int64_t kTokensAcross = int64_t(1) << 22;
template <class T, int kB>
__global__ __launch_bounds__(kBlock) void k_expert_combine_back(MoveArgs a) {
    using raw = typename T::raw;
    const uint32_t lane = lane_id();
    const int64_t t = (int64_t)blockIdx.y * kTokensAcross + blockIdx.x;
    if (t >= a.tokens) return;
    const raw* const dout = static_cast<const raw*>(a.x) + t * a.ld_x;
    const raw* const y = static_cast<const raw*>(a.y_in);
    raw* const dy = static_cast<raw*>(a.y);
    const Span s = span_of<T>(a);
    const bool held = s.granules <= 64 * kB, tiny = s.granules == 0 && lane < a.dim;
    gran d[kB];
    if (held && s.granules) Row<T, kB>::load_again(d, dout, s, lane);
    const float last = tiny ? T::up1(dout[lane]) : 0.0f;
    Held h;
    const int32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    for (int32_t j = wave; j < a.k; j += kWaves) {
        if (j == wave || (j & 63) == wave) h.load(a, t, j & ~63);
        const int64_t r = h.place(j & 63);
        if (r < 0) {
            if (a.dweight && lane == 0) a.dweight[t * a.k + j] = 0.0f;
            continue;
        }
        const float w = h.factor(j & 63);
        float dot = 0.0f;
        for (int64_t i = lane; i - lane < s.granules; i += 64 * kB) {
            gran g[kB];
            if (a.dweight) Row<T, kB>::load(g, y + r * a.ld_y_in, s, i);
            if (!held) Row<T, kB>::load_again(d, dout, s, i);
            if (dy) {
                gran v[kB];
#pragma unroll
                for (int b = 0; b < kB; ++b) {
                    float f[T::kN];
#pragma unroll
                    for (int e = 0; e < T::kN; ++e) f[e] = w != 0.0f ? w * T::up(d[b], e) : 0.0f;
                    v[b] = T::down(f);
                }
                Row<T, kB>::store(v, dy + r * a.ld_y, s, i);
            }
            if (a.dweight) {
#pragma unroll
                for (int b = 0; b < kB; ++b) dot += dot_of<T>(g[b], d[b], s, i + b * 64);
            }
        }
        if (tiny) {
            if (a.dweight) dot = T::up1(y[r * a.ld_y_in + lane]) * last;
            if (dy) dy[r * a.ld_y + lane] = T::down1(w != 0.0f ? w * last : 0.0f);
        }
        if (a.dweight) {
            dot = group_reduce<OpSumF, 64>(dot);
            if (lane == 0) a.dweight[t * a.k + j] = dot;
        }
    }
}

// Short rows: kL lanes take a choice, so that a wave has several on their way
// (16384x128 bf16, k = 8: gradient 16 us, 4.5 TB/s).
template <class T, int kL>
struct Choice {
    int64_t c, t, r;  // the choice, its token and its place
    uint32_t lane, byte;
    float weight;
    bool in, on, mine;  // in: there is one; on: it has a place; mine: the lane has a granule of it
    __device__ __forceinline__ Choice(const MoveArgs& a, const Span& s) {
        lane = threadIdx.x % kL;
        c = (int64_t)blockIdx.x * (kBlock / kL) + threadIdx.x / kL;
        in = c < a.tokens * a.k;
        t = in ? (uint32_t)c / (uint32_t)a.k : 0;
        r = in ? a.row[c] : -1;
        weight = in && a.weight ? a.weight[c] : 1.0f;
        on = r >= 0 && r < a.rows;
        mine = on && lane < s.granules;
        byte = Row<T, 1>::byte(s, lane);
    }
};
template <class T, int kL>
__global__ __launch_bounds__(kBlock) void k_expert_gather_rows(MoveArgs a) {
    using raw = typename T::raw;
    const Span s = span_of<T>(a);
    const Choice<T, kL> q(a, s);
    if (!q.mine) return;
    const gran g = read16_again(static_cast<const raw*>(a.x) + q.t * a.ld_x, q.byte);
    write16(static_cast<raw*>(a.y) + q.r * a.ld_y, q.byte, g);
}
template <class T, int kL>
__global__ __launch_bounds__(kBlock) void k_expert_back_rows(MoveArgs a) {
    using raw = typename T::raw;
    const Span s = span_of<T>(a);
    const Choice<T, kL> q(a, s);
    gran g = gran{0, 0, 0, 0}, d = g;
    if (q.mine) {
        d = read16_again(static_cast<const raw*>(a.x) + q.t * a.ld_x, q.byte);
        if (a.dweight) g = read16(static_cast<const raw*>(a.y_in) + q.r * a.ld_y_in, q.byte);
        if (a.y) {
            float f[T::kN];
#pragma unroll
            for (int e = 0; e < T::kN; ++e) f[e] = q.weight != 0.0f ? q.weight * T::up(d, e) : 0.0f;
            write16(static_cast<raw*>(a.y) + q.r * a.ld_y, q.byte, T::down(f));
        }
    }
    if (!a.dweight) return;
    const float dot = group_reduce<OpSumF, kL>(dot_of<T>(g, d, s, q.lane));
    if (q.in && q.lane == 0) a.dweight[q.c] = dot;
}

// Granules a lane: as many as a row has for it, up to four or eight.
int granules_of(const MoveArgs& a) {
    const int64_t n = 16 / dtype_size(a.dtype);
    return (int)(((a.dim + n - 1) / n + 63) / 64);
}
// Lanes for a choice of a short row, 0 where it is none (or where the choices'
// threads do not fit a grid's axis).  The gradient of 16384 tokens, k =
// 8, takes a wave a choice and so: 128 bf16 38.5 and 16.7 us, 100 f16 60 and 21,
// 256 bf16 44.7 and 30.8; with all 64 lanes no less (512 bf16 54.5 and 58.2).
int lanes_of(const MoveArgs& a) {
    const int64_t n = 16 / dtype_size(a.dtype), granules = a.dim < n ? 33 : (a.dim + n - 1) / n;
    for (int lanes = 8; lanes <= 32; lanes *= 2)
        if (granules <= lanes) return a.tokens * a.k <= (int64_t(1) << 31) / lanes ? lanes : 0;
    return 0;
}
#define SCAPE_RUN_ROWS(lanes, ...)                                                                                      \
    hipLaunchKernelGGL((__VA_ARGS__), dim3((uint32_t)((a.tokens * a.k * lanes + kBlock - 1) / kBlock)), dim3(kBlock), 0, s, a)

#define SCAPE_RUN(...) \
    hipLaunchKernelGGL((__VA_ARGS__), dim3((uint32_t)((a.tokens + kWaves - 1) / kWaves)), dim3(kBlock), 0, s, a)
#define SCAPE_RUN_TOKEN(...)                                                                                            \
    hipLaunchKernelGGL((__VA_ARGS__), dim3((uint32_t)(a.tokens < kTokensAcross ? a.tokens : kTokensAcross),             \
                                           (uint32_t)((a.tokens + kTokensAcross - 1) / kTokensAcross)), dim3(kBlock), 0, s, a)

template <class T>
hipError_t gather_of(hipStream_t s, const MoveArgs& a) {
    const int n = granules_of(a), lanes = lanes_of(a);
    if (lanes == 8) SCAPE_RUN_ROWS(8, k_expert_gather_rows<T, 8>);
    else if (lanes == 16) SCAPE_RUN_ROWS(16, k_expert_gather_rows<T, 16>);
    else if (lanes == 32) SCAPE_RUN_ROWS(32, k_expert_gather_rows<T, 32>);
    else if (n <= 1) SCAPE_RUN(k_expert_gather<T, 1>);
    else if (n <= 2) SCAPE_RUN(k_expert_gather<T, 2>);
    else SCAPE_RUN(k_expert_gather<T, 4>);
    return hipGetLastError();
}
template <class T>
hipError_t combine_of(hipStream_t s, const MoveArgs& a) {
    const int n = granules_of(a);
    if (a.k <= 2) {
        if (n <= 1) SCAPE_RUN(k_expert_combine<T, 1, 2>);
        else SCAPE_RUN(k_expert_combine<T, 2, 2>);
    } else if (a.k <= 4) {
        if (n <= 1) SCAPE_RUN(k_expert_combine<T, 1, 4>);
        else SCAPE_RUN(k_expert_combine<T, 2, 4>);
    } else {
        if (n <= 1) SCAPE_RUN(k_expert_combine<T, 1, 8>);
        else SCAPE_RUN(k_expert_combine<T, 2, 8>);
    }
    return hipGetLastError();
}
template <class T>
hipError_t back_of(hipStream_t s, const MoveArgs& a) {
    const int n = granules_of(a), lanes = lanes_of(a);
    if (lanes == 8) SCAPE_RUN_ROWS(8, k_expert_back_rows<T, 8>);
    else if (lanes == 16) SCAPE_RUN_ROWS(16, k_expert_back_rows<T, 16>);
    else if (lanes == 32) SCAPE_RUN_ROWS(32, k_expert_back_rows<T, 32>);
    else if (n <= 1) SCAPE_RUN_TOKEN(k_expert_combine_back<T, 1>);
    else if (n <= 2) SCAPE_RUN_TOKEN(k_expert_combine_back<T, 2>);
    else if (n <= 4) SCAPE_RUN_TOKEN(k_expert_combine_back<T, 4>);
    else SCAPE_RUN_TOKEN(k_expert_combine_back<T, 8>);
    return hipGetLastError();
}
#define SCAPE_BY_TYPE(run) \
    return a.dtype == SCAPE_DTYPE_F32 ? run<F32>(s, a) : a.dtype == SCAPE_DTYPE_BF16 ? run<BF16>(s, a) : run<F16>(s, a)

}  // namespace

hipError_t launch_expert_sort(hipStream_t s, const SortArgs& a) {
    const dim3 blocks((uint32_t)a.blocks), threads(kBlock);
    if (a.blocks > 1) hipLaunchKernelGGL(k_expert_count, blocks, threads, 0, s, a);
    hipLaunchKernelGGL(k_expert_place, blocks, threads, 0, s, a);
    return hipGetLastError();
}
hipError_t launch_expert_gather(hipStream_t s, const MoveArgs& a) { SCAPE_BY_TYPE(gather_of); }
hipError_t launch_expert_combine(hipStream_t s, const MoveArgs& a) { SCAPE_BY_TYPE(combine_of); }
hipError_t launch_expert_combine_back(hipStream_t s, const MoveArgs& a) { SCAPE_BY_TYPE(back_of); }

}  // namespace scape
