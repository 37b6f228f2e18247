// k_topk.hip - the k largest entries of each row of a logit matrix, in order
// (larger value first, equal values by the lower column), and the row's
// log-sum-exp: the per-layer mask's tie rule on rows.  For gfx950.
//
// An entry's rank is one unsigned 64-bit number, (ordered value bits) << 32 |
// ~column, so no two entries of a row are equal and the result does not
// depend on the order in which candidates are found.
//
// Each kernel reads a row once, so what bounds the long rows is the read of the
// logits.
//  - k_topk_small: rows of up to 1024 columns (a router's experts), a group
//    of lanes per row.
//  - k_topk_rows: longer rows, a workgroup per row or part of one, the row in
//    registers.
//  - k_topk_merge: joins the parts of a split row.
#include <float.h>

#include <type_traits>

#include "loss_device.h"

namespace scape {

// Unsigned order of floats: -inf < ... < -0 = +0 < ... < +inf < NaN.
__device__ __forceinline__ uint32_t order_key(float f) {
    uint32_t b = __float_as_uint(f + 0.0f);  // -0 becomes +0
    if (f != f) return 0xFFFFFFFFu;
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
    if (k == 0xFFFFFFFFu) return __uint_as_float(0x7FC00000u);
    return __uint_as_float((k & 0x80000000u) ? k ^ 0x80000000u : ~k);
}
constexpr uint32_t kKeyNegInf = 0x007FFFFFu;  // order_key(-inf): no entry

// Entry `r` of the row's result.
template <class T>
__device__ __forceinline__ void write_entry(const TopkArgs& a, int64_t row, int32_t r, uint64_t comp) {
    const int64_t o = row * a.k + r;
    const bool none = comp == 0;
    const float v = none ? kNegInf : key_value((uint32_t)(comp >> 32));
    static_cast<typename T::raw*>(a.val)[o] = T::down1(v);  // exact: v came from this type
    a.idx[o] = none ? -1 : (int32_t)~(uint32_t)comp;
}

// log-sum-exp from sum = sum 2^(c2 (x - ref)); only the last step rounds.
__device__ __forceinline__ float lse_of(const TopkArgs& a, float ref, double sum) {
    return (float)((double)ref * a.scale + kLn2 * log2(sum));
}

// ---------------------------------------------------------------------------
// Long rows

// Ranks the n candidates in list (n <= kTopkList, all different) and hands
// the first k, in order, to emit(r, composite); slots past n get 0.
template <int kThreads, class Emit>
__device__ void emit_sorted(uint64_t* list, uint32_t n, int32_t k, Emit emit) {
    const uint32_t tid = threadIdx.x;
    if (n <= 512) {
        // each candidate counts those above it, eight at a time (the row
        // kernel over 1021x50257 f32 47 -> 43 us)
        constexpr uint32_t kAt = 8;
        const uint32_t n8 = (n + kAt - 1) / kAt * kAt;
        if (tid < n8 - n) list[n + tid] = 0;
        __syncthreads();
        for (uint32_t i = tid; i < n; i += kThreads) {
            const uint64_t mine = list[i];
            uint32_t r = 0;
            for (uint32_t j = 0; j < n8; j += kAt) {
                uint64_t x[kAt];
#pragma unroll
                for (uint32_t u = 0; u < kAt; ++u) x[u] = list[j + u];
#pragma unroll
                for (uint32_t u = 0; u < kAt; ++u) r += x[u] > mine ? 1u : 0u;
            }
            if (r < (uint32_t)k) emit((int32_t)r, mine);
        }
    } else {
        uint32_t p = 1024;
        while (p < n) p <<= 1;
        for (uint32_t i = n + tid; i < p; i += kThreads) list[i] = 0;
        for (uint32_t size = 2; size <= p; size <<= 1)
            for (uint32_t d = size >> 1; d > 0; d >>= 1) {
                __syncthreads();
                for (uint32_t t = tid; t < p / 2; t += kThreads) {
                    const uint32_t i = 2 * t - (t & (d - 1)), j = i + d;
                    const uint64_t x = list[i], y = list[j];
                    if ((x < y) == ((i & size) == 0)) {
                        list[i] = y;
                        list[j] = x;
                    }
                }
            }
        __syncthreads();
        for (uint32_t i = tid; i < (uint32_t)k && i < n; i += kThreads) emit((int32_t)i, list[i]);
    }
    for (uint32_t i = n + tid; i < (uint32_t)k; i += kThreads) emit((int32_t)i, 0ull);
}

// A workgroup takes `per` granules of a row into registers and makes the
// row's k largest, or its part's, from them.  4096x32000 bf16, k = 64: 49 us,
// 5.3 TB/s (a plain read of as much 38 us): four workgroups of a CU load while
// others choose, and the choice alone, from the threshold on, costs the 9 us
// that this does not hide.  1021x50257 f32, k = 100, in four parts: 44 us, 4.7
// TB/s, and 6 for the merge.
//
// Candidates: of disjoint groups of entries, two a thread, the k-th largest of
// the groups' maxima is at most the k-th largest entry, and for k well below
// the number of groups only a few more than k entries reach it.  Granules
// whose maximum reaches it are copied to LDS and gone through there, so a
// thread with such a granule does not hold up its wave.  Where there are more
// than the lists hold (ties, or k near the number of groups), the exact
// threshold comes from a radix selection that reads the row again, from the
// caches, for each 8-bit digit.
constexpr int kTopkHits = 768;  // granules, an equal share for each wave
template <class T, int kThreads, int kGran>
__global__ __launch_bounds__(kThreads, 4) void k_topk_rows(TopkArgs a) {
    constexpr int kNW = kThreads / 64;
    __shared__ __align__(16) uint64_t list[kTopkList];
    __shared__ gran hit[kTopkHits];
    __shared__ int32_t hit_at[kTopkHits];
    __shared__ uint32_t hist[256];
    __shared__ uint32_t gmax[2 * kThreads];
    __shared__ float2 wsum[kNW];
    __shared__ uint32_t s_n, s_over, s_bin, s_need, s_tau;
    using raw = typename T::raw;
    const int32_t tid = (int32_t)threadIdx.x, wave = tid / 64;
    const int64_t row = blockIdx.x / (uint32_t)a.splits;
    const int32_t sp = (int32_t)(blockIdx.x % (uint32_t)a.splits);
    const raw* z = static_cast<const raw*>(a.in.z) + row * a.in.ld;
    const int32_t n = (int32_t)a.in.cols, k = a.k;
    const RowShape sh = row_shape<T>(z, n);
    const int32_t g0 = sp * a.per;
    const int32_t cnt = min(a.per, sh.granules - g0);  // may be <= 0 in the last split
    const gran* body = cnt > 0 ? reinterpret_cast<const gran*>(z + sh.head) + g0 : &g_no_granule;
    const int32_t first = sh.head + g0 * T::kN;  // column of granule 0's first element

    // loads under no condition, so that the first are worked on while the
    // last are on their way; past the end the last granule again, taken out
    // below
    gran g[kGran];
#pragma unroll
    for (int c = 0; c < kGran; ++c) g[c] = granule_at(body, max(min(tid + c * kThreads, cnt - 1), 0));
    const int32_t lone = lone_element(sh, n, sp == 0, sp == a.splits - 1);
    float lx = T::up1(z[lone >= 0 ? lone : 0]);
    if (lone < 0) lx = kNegInf;
    if (tid == 0) s_n = s_over = 0;

    constexpr int kBatch = kGran / 2 < 4 ? kGran / 2 : 4;
    float gm[kGran], m0 = kNegInf, m1 = kNegInf;
    RunningSum rs = RunningSum::none();
#pragma unroll
    for (int c = 0; c < kGran; c += kBatch)
        if (c * kThreads < cnt || c == 0) {
            if ((c + kBatch) * kThreads > cnt) {
#pragma unroll
                for (int b = 0; b < kBatch; ++b)
                    if (tid + (c + b) * kThreads >= cnt) g[c + b] = no_entries<T>();
            }
            gran x[kBatch];
            float bm = kNegInf;
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                x[b] = g[c + b];
                gm[c + b] = granule_max<T>(x[b]);
                bm = max_nan(bm, gm[c + b]);
            }
            (c & kBatch ? m1 : m0) = max_nan(c & kBatch ? m1 : m0, bm);
            rs.template add<T, kBatch>(x, bm, a.c2);
        } else {
#pragma unroll
            for (int b = 0; b < kBatch; ++b) gm[c + b] = kNegInf;
        }
    rs.add1(lx, a.c2);
    m0 = max_nan(m0, lx);
    gmax[tid] = order_key(m0) >> 16;
    gmax[tid + kThreads] = order_key(m1) >> 16;
    wave_join(rs, a.c2);
    if ((tid & 63) == 0) wsum[wave] = make_float2(rs.ref, rs.sum);
    __syncthreads();

    // wave 0: the k-th largest of the maxima, to the top 16 bits of its key
    if (wave == 0) {
        uint32_t mk[2 * kNW];
#pragma unroll
        for (int w = 0; w < 2 * kNW; ++w) mk[w] = gmax[w * 64 + tid];
        // the bits that all maxima share are the threshold's too (where there
        // are k of them), so the search begins at the first that differs
        uint32_t hi = mk[0], lo = mk[0], t = 0;
#pragma unroll
        for (int w = 1; w < 2 * kNW; ++w) {
            hi = mk[w] > hi ? mk[w] : hi;
            lo = mk[w] < lo ? mk[w] : lo;
        }
        hi = group_reduce<OpMaxU, 64>(hi);
        lo = ~group_reduce<OpMaxU, 64>(~lo);
        const int top = k <= 2 * kThreads ? 31 - (int)__builtin_clz((hi ^ lo) | 1u) : 15;
        if (k <= 2 * kThreads) t = hi & ~((2u << top) - 1u);
        for (int b = __builtin_amdgcn_readfirstlane(top); b >= 0; --b) {
            const uint32_t x = t | (1u << b);
            uint32_t count = 0;
#pragma unroll
            for (int w = 0; w < 2 * kNW; ++w) count += (uint32_t)__popcll(wave_ballot(mk[w] >= x));
            if (count >= (uint32_t)k) t = x;
        }
        if (tid == 0) s_tau = t;
    } else if (wave == kNW - 1) {
        RunningSum r{wsum[tid & (kNW - 1)].x, wsum[tid & (kNW - 1)].y};
        join_waves<kNW>(r, a.c2);
        if (tid == kThreads - 1) {
            if (a.splits > 1)
                a.part[row * a.splits + sp] = make_float2(r.ref, r.sum);
            else if (a.lse)
                a.lse[row] = lse_of(a, r.ref, (double)r.sum);
        }
    }
    __syncthreads();

    // candidates: entries not below the threshold, which is finite (so -inf
    // is never one, and NaN, which compares false, always is)
    const float tau = fmaxf(key_value(s_tau << 16), -FLT_MAX);
    auto take = [&](float f, int32_t col) {
        if (!(f < tau)) {
            const uint32_t at = atomicAdd(&s_n, 1u);
            if (at < kTopkList) list[at] = ((uint64_t)order_key(f) << 32) | (uint32_t)~(uint32_t)col;
        }
    };
    take(lx, lone);
    constexpr uint32_t kShare = kTopkHits / kNW;
    const uint32_t share = (uint32_t)wave * kShare;
    uint32_t hits = 0;  // of the wave
#pragma unroll
    for (int c = 0; c < kGran; ++c) {
        const bool reaches = !(gm[c] < tau);
        const uint64_t lanes = wave_ballot(reaches);
        if (lanes) {
            const uint32_t at = hits + lanes_below(lanes);
            if (reaches && at < kShare) {
                hit[share + at] = g[c];
                hit_at[share + at] = first + (tid + c * kThreads) * T::kN;
            }
            hits += (uint32_t)__popcll(lanes);
        }
    }
    if (hits <= kShare) {
        // the wave's own hits: its LDS writes are done before it reads
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        const raw* elems = reinterpret_cast<const raw*>(hit + share);
        for (uint32_t i = (uint32_t)tid & 63u; i < hits * T::kN; i += 64)
            take(T::up1(elems[i]), hit_at[share + i / T::kN] + (int32_t)(i % T::kN));
    } else if ((tid & 63) == 0) {
        s_over = 1;
    }
    __syncthreads();
    uint32_t found = s_n;
    if (s_over || found > kTopkList) {
        // radix selection over 8-bit digits of the composite, largest first;
        // every part of the row by its granules, then the lone elements
        auto each = [&](auto f) {
            for (int32_t i0 = 0; i0 < cnt; i0 += kThreads) {
                const int32_t i = i0 + tid;
                const gran x = i < cnt ? granule_at(body, i) : no_entries<T>();
#pragma unroll
                for (int j = 0; j < T::kN; ++j) f(T::up(x, j), first + i * T::kN + j);
            }
            f(lx, lone);
        };
        uint64_t prefix = 0;
        uint32_t need = (uint32_t)k;
        int shift = 56;
        __syncthreads();
        for (;; shift -= 8) {
            if (shift == 24) {  // ~column >> 24 is 0xFF: columns are below 2^24
                prefix = (prefix << 8) | 0xFFu;
                continue;
            }
            for (int32_t i = tid; i < 256; i += kThreads) hist[i] = 0;
            __syncthreads();
            each([&](float f, int32_t col) {
                const uint64_t comp = ((uint64_t)order_key(f) << 32) | (uint32_t)~(uint32_t)col;
                const bool in = f != kNegInf && (shift == 56 || (comp >> (shift + 8)) == prefix);
                hist_add_wave(hist, (uint32_t)(comp >> shift) & 255u, in);
            });
            __syncthreads();
            if (wave == 0) {
                // bins from the top, four a lane: the one that holds the
                // need-th, or the lowest where there are fewer
                uint32_t h[4], own = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) own += h[i] = hist[255 - (4 * tid + i)];
                const uint32_t upto = wave_inclusive_scan(own);
                const uint64_t reach = wave_ballot(upto >= need);
                if (tid == (reach ? (int)__builtin_ctzll(reach) : 63)) {
                    uint32_t above = upto - own, i = 0;
#pragma unroll
                    for (uint32_t u = 0; u < 3; ++u)
                        if (i == u && above + h[u] < need) {
                            above += h[u];
                            i = u + 1;
                        }
                    s_bin = 255 - (4 * (uint32_t)tid + i);
                    s_need = need - above;
                }
            }
            __syncthreads();
            prefix = (prefix << 8) | s_bin;
            need = s_need;
            if ((uint32_t)k - need + hist[s_bin] <= kTopkList || shift == 0) break;
            __syncthreads();
        }
        __syncthreads();
        if (tid == 0) s_n = 0;
        __syncthreads();
        each([&](float f, int32_t col) {
            const uint64_t comp = ((uint64_t)order_key(f) << 32) | (uint32_t)~(uint32_t)col;
            if (f != kNegInf && (comp >> shift) >= prefix) list[atomicAdd(&s_n, 1u)] = comp;
        });
        __syncthreads();
        found = s_n;
    }

    if (a.splits == 1) {
        emit_sorted<kThreads>(list, found, k, [&](int32_t r, uint64_t comp) { write_entry<T>(a, row, r, comp); });
    } else {
        uint64_t* out = a.cand + (row * a.splits + sp) * k;
        emit_sorted<kThreads>(list, found, k, [&](int32_t r, uint64_t comp) { out[r] = comp; });
    }
}

// Joins a row's parts.  Each part's candidates are sorted, so of the first
// ceil(k / splits) of every part at least k are in the row: only entries that
// reach the smallest of those can be among the row's k largest.
constexpr int kMergeThreads = 256;
template <class T>
__global__ __launch_bounds__(kMergeThreads) void k_topk_merge(TopkArgs a) {
    __shared__ __align__(16) uint64_t list[kTopkList];
    __shared__ uint64_t s_low;
    __shared__ uint32_t s_n;
    const int32_t tid = (int32_t)threadIdx.x;
    const int64_t row = blockIdx.x;
    const uint32_t k = (uint32_t)a.k, all = (uint32_t)a.splits * k;
    const uint64_t* cand = a.cand + row * all;
    if (tid < 64) {
        const uint32_t at = (k + (uint32_t)a.splits - 1) / (uint32_t)a.splits - 1;
        uint64_t low = ~0ull;
        if (tid < a.splits) low = cand[(uint32_t)tid * k + at];
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const uint64_t o = __shfl_xor((unsigned long long)low, d, 64);
            low = o < low ? o : low;
        }
        if (tid == 0) {
            s_low = low;
            s_n = 0;
        }
    } else if (tid < 128 && a.lse) {
        RunningSum r = RunningSum::none();
        if (tid - 64 < a.splits) {
            const float2 p = a.part[row * a.splits + (tid - 64)];
            r = RunningSum{p.x, p.y};
        }
        wave_join(r, a.c2);
        if (tid == 64) a.lse[row] = lse_of(a, r.ref, (double)r.sum);
    }
    __syncthreads();
    const uint64_t low = s_low;
    for (uint32_t i = (uint32_t)tid; i < all; i += kMergeThreads) {
        const uint64_t x = cand[i];
        if (x >= low && x != 0) {
            const uint32_t at = atomicAdd(&s_n, 1u);
            if (at < kTopkList) list[at] = x;
        }
    }
    __syncthreads();
    const uint32_t found = s_n;
    if (found <= kTopkList) {
        emit_sorted<kMergeThreads>(list, found, a.k, [&](int32_t r, uint64_t comp) { write_entry<T>(a, row, r, comp); });
        return;
    }
    // too many (one part holds most of them): an entry's rank is its place in
    // its own part plus, by binary search, the entries above it in the others
    for (uint32_t i = (uint32_t)tid; i < all; i += kMergeThreads) {
        const uint64_t x = cand[i];
        if (x == 0) continue;
        const uint32_t own = i / k;
        uint32_t r = i - own * k;
        for (uint32_t s = 0; s < (uint32_t)a.splits && r < k; ++s) {
            if (s == own) continue;
            uint32_t lo = 0, hi = k;
            while (lo < hi) {
                const uint32_t mid = (lo + hi) / 2;
                if (cand[s * k + mid] > x)
                    lo = mid + 1;
                else
                    hi = mid;
            }
            r += lo;
        }
        if (r < k) write_entry<T>(a, row, (int32_t)r, x);
    }
}

// ---------------------------------------------------------------------------
// Short rows: kLanes lanes a row, kGran granules a lane; lane l holds the
// granules l, l + kLanes, ...  (vec: rows on 16-byte boundaries; otherwise
// element by element).  A lane sorts its entries; in each of k rounds the
// largest head of the group leaves its lane's list, and lane r keeps the r-th
// until a whole group's worth is written at once.  What bounds it is the
// instructions: 65536x64 f32, k = 6, takes 10.5 us, 5.5 of them the vector
// units' and 3 the memory's; a scan of each lane's entries in every round took 15.

// An entry: value and column as one number, larger for an earlier rank.  A
// 16-bit value and its column share a word; 0 is no entry.
template <class T>
struct Ranked {
    static constexpr uint32_t kNan = std::is_same<T, BF16>::value ? 0x7FC0u : 0x7E00u;
    static constexpr uint32_t kKeyNegInf = 0x8000u - (T::kNegInfBits & 0x7FFFu);
    uint32_t w;
    static __device__ __forceinline__ Ranked of(const gran& g, int j, uint32_t col) {
        const uint32_t b = (g[j >> 1] >> (16 * (j & 1))) & 0xFFFFu, mag = b & 0x7FFFu;
        uint32_t key = (b & 0x8000u) ? 0x8000u - mag : 0x8000u + mag;  // -0 is +0
        key = mag > (T::kNegInfBits & 0x7FFFu) ? 0xFFFFu : key;
        return Ranked{(key << 16) | (0xFFFFu - col)};
    }
    static __device__ __forceinline__ void order(Ranked& a, Ranked& b) {
        const uint32_t hi = a.w > b.w ? a.w : b.w;
        b.w = a.w > b.w ? b.w : a.w;
        a.w = hi;
    }
    template <int kLanes>
    __device__ __forceinline__ Ranked best() const { return Ranked{group_reduce<OpMaxU, kLanes>(w)}; }
    __device__ __forceinline__ bool is(const Ranked& o) const { return w == o.w; }
    __device__ __forceinline__ bool none() const { return (w >> 16) <= kKeyNegInf; }
    __device__ __forceinline__ typename T::raw value() const {
        const uint32_t key = w >> 16;
        if (none()) return (typename T::raw)T::kNegInfBits;
        return (typename T::raw)(key == 0xFFFFu ? kNan : key >= 0x8000u ? key - 0x8000u : 0x10000u - key);
    }
    __device__ __forceinline__ int32_t column() const { return none() ? -1 : (int32_t)(0xFFFFu - (w & 0xFFFFu)); }
    static __device__ __forceinline__ Ranked empty() { return Ranked{0u}; }
    __device__ __forceinline__ void take(bool which, const Ranked& o) { w = which ? o.w : w; }
};
template <>
struct Ranked<F32> {
    uint32_t key, ncol;  // ncol = ~column
    static __device__ __forceinline__ Ranked of(const gran& g, int j, uint32_t col) {
        return Ranked{order_key(F32::up(g, j)), ~col};
    }
    static __device__ __forceinline__ void order(Ranked& a, Ranked& b) {
        const bool up = (((uint64_t)b.key << 32) | b.ncol) > (((uint64_t)a.key << 32) | a.ncol);
        const Ranked x = a;
        a.take(up, b);
        b.take(up, x);
    }
    template <int kLanes>
    __device__ __forceinline__ Ranked best() const {
        const uint32_t top = group_reduce<OpMaxU, kLanes>(key);
        return Ranked{top, group_reduce<OpMaxU, kLanes>(key == top ? ncol : 0u)};
    }
    __device__ __forceinline__ bool is(const Ranked& o) const { return key == o.key && ncol == o.ncol; }
    __device__ __forceinline__ bool none() const { return key <= kKeyNegInf; }
    __device__ __forceinline__ uint32_t value() const { return none() ? F32::kNegInfBits : __float_as_uint(key_value(key)); }
    __device__ __forceinline__ int32_t column() const { return none() ? -1 : (int32_t)~ncol; }
    static __device__ __forceinline__ Ranked empty() { return Ranked{0u, 0u}; }
    __device__ __forceinline__ void take(bool which, const Ranked& o) {
        key = which ? o.key : key;
        ncol = which ? o.ncol : ncol;
    }
};

// Batcher's merge exchange over a lane's kV entries, largest first.
template <int kV, class E>
__device__ __forceinline__ void sort_lane(E (&e)[kV]) {
#pragma unroll
    for (int p = 1; p < kV; p *= 2)
#pragma unroll
        for (int q = p; q >= 1; q /= 2)
#pragma unroll
            for (int i = 0; i + q < kV; ++i)
                if (i >= q % p && (i - q % p) % (2 * q) < q && i / (2 * p) == (i + q) / (2 * p)) E::order(e[i], e[i + q]);
}

template <class T, int kLanes, int kGran, bool kVec>
__global__ __launch_bounds__(kBlock) void k_topk_small(TopkArgs a) {
    using raw = typename T::raw;
    constexpr int kRowsPerWave = 64 / kLanes, kV = kGran * T::kN;
    const uint32_t lane = lane_id(), l = lane % kLanes;
    const int64_t row = ((int64_t)blockIdx.x * kWaves + threadIdx.x / 64) * kRowsPerWave + lane / kLanes;
    const bool live = row < a.in.rows;
    const raw* z = static_cast<const raw*>(a.in.z) + (live ? row : 0) * a.in.ld;
    const int32_t n = live ? (int32_t)a.in.cols : 0;
    gran g[kGran];
#pragma unroll
    for (int c = 0; c < kGran; ++c) {
        const int32_t e0 = (int32_t)(l + c * kLanes) * T::kN;
        g[c] = no_entries<T>();
        if (kVec && e0 + T::kN <= n) {
            g[c] = *reinterpret_cast<const gran*>(z + e0);
        } else {
#pragma unroll
            for (int j = 0; j < T::kN; ++j)
                if (e0 + j < n) T::set(g[c], j, z[e0 + j]);
        }
    }
    if (a.lse) {
        float m = granule_max<T>(g[0]);
#pragma unroll
        for (int c = 1; c < kGran; ++c) m = max_nan(m, granule_max<T>(g[c]));
        m = group_reduce<OpMaxF, kLanes>(m);
        const float ref = m == kNegInf ? 0.0f : m;
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < kV; ++i) sum += fast_exp2(less<T>(g[i / T::kN], i % T::kN, ref) * a.c2);
        sum = group_reduce<OpSumF, kLanes>(sum);
        // v_log_f32: the sum is 1 to 1024, so a step of it is less than what the sum is off by
        if (l == 0 && live) a.lse[row] = (float)((double)ref * a.scale + kLn2 * (double)__builtin_amdgcn_logf(sum));
    }
    Ranked<T> e[kV];
#pragma unroll
    for (int i = 0; i < kV; ++i)
        e[i] = Ranked<T>::of(g[i / T::kN], i % T::kN, (l + (uint32_t)(i / T::kN) * kLanes) * T::kN + (uint32_t)(i % T::kN));
    sort_lane<kV>(e);
    Ranked<T> kept = Ranked<T>::empty();
    for (int32_t r = 0; r < a.k; ++r) {
        const Ranked<T> top = e[0].template best<kLanes>();
        const bool mine = e[0].is(top);
#pragma unroll
        for (int i = 0; i + 1 < kV; ++i) e[i].take(mine, e[i + 1]);
        e[kV - 1].take(mine, Ranked<T>::empty());
        const int32_t at = r % kLanes;
        kept.take((int32_t)l == at, top);
        if (at == kLanes - 1 || r == a.k - 1) {
            if (live && (int32_t)l <= at) {
                const int64_t o = row * a.k + (r - at) + (int32_t)l;
                static_cast<raw*>(a.val)[o] = kept.value();
                a.idx[o] = kept.column();
            }
        }
    }
}

template <class T, int kLanes, int kGran>
static void topk_small(hipStream_t s, const TopkArgs& a, bool vec) {
    constexpr int rows = kWaves * (64 / kLanes);
    const dim3 grid((uint32_t)((a.in.rows + rows - 1) / rows));
    if (vec)
        hipLaunchKernelGGL((k_topk_small<T, kLanes, kGran, true>), grid, dim3(kBlock), 0, s, a);
    else
        hipLaunchKernelGGL((k_topk_small<T, kLanes, kGran, false>), grid, dim3(kBlock), 0, s, a);
}

template <class T>
static hipError_t topk_typed(hipStream_t s, const TopkArgs& a) {
    if (topk_small(a.in.cols, a.k)) {
        const bool vec = (uintptr_t)a.in.z % 16 == 0 && a.in.ld * sizeof(typename T::raw) % 16 == 0;
        const int64_t g = (a.in.cols + T::kN - 1) / T::kN;  // granules a row
        // fewer lanes a row, each with more to sort, make the rounds cheaper (65536 rows, k = 8, replayed: 256 f32
        // columns on 64 lanes 48 us, on 16 lanes of four granules 38; 256 bf16 on 64 lanes 48, on 16 of two 25)
        constexpr int kFour = T::kN == 4 ? 4 : 2;
        if (g <= 4) topk_small<T, 4, 1>(s, a, vec);
        else if (g <= 16) topk_small<T, 8, 2>(s, a, vec);
        else if (g <= 16 * kFour) topk_small<T, 16, kFour>(s, a, vec);
        else if (g <= 32 * kFour) topk_small<T, 32, kFour>(s, a, vec);
        else topk_small<T, 64, kFour>(s, a, vec);
        return hipGetLastError();
    }
    const dim3 grid((uint32_t)(a.in.rows * a.splits));
    if (a.per <= 256 * 4) hipLaunchKernelGGL((k_topk_rows<T, 256, 4>), grid, dim3(256), 0, s, a);
    else if (a.per <= 256 * 8) hipLaunchKernelGGL((k_topk_rows<T, 256, 8>), grid, dim3(256), 0, s, a);
    else if (a.per <= 256 * 16) hipLaunchKernelGGL((k_topk_rows<T, 256, 16>), grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((k_topk_rows<T, 512, 16>), grid, dim3(512), 0, s, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.splits == 1) return e;
    hipLaunchKernelGGL((k_topk_merge<T>), dim3((uint32_t)a.in.rows), dim3(kMergeThreads), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_topk(hipStream_t s, const TopkArgs& a) {
    if (a.in.dtype == SCAPE_DTYPE_F32) return topk_typed<F32>(s, a);
    if (a.in.dtype == SCAPE_DTYPE_BF16) return topk_typed<BF16>(s, a);
    return topk_typed<F16>(s, a);
}

}  // namespace scape
