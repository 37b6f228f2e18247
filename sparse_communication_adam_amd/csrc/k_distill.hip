// k_distill.hip - distillation from a teacher's top logits, for gfx950.
//
// A row has student logits z (n columns) and k teacher entries (value t_j,
// column i_j).  With s = 1 / temperature, p = softmax(s z), the entries'
// teacher probabilities q_j, the teacher's mass outside them q_T and the
// student's p_T:
//   KL   = sum_j q_j (log q_j - log p_{i_j}) + q_T (log q_T - log p_T)
//   d/dz = s (Q p_v - q_T p_v / p_T)      outside the entries, Q = sum q_j + q_T
//        = s (Q p_{i_j} - q_j)            at an entry
//
// The logits are read once.  The entries' columns are marked in an LDS bitmap
// and struck out of the granules as they arrive (-inf), so the sums that
// follow are the tail's own, never a difference of two large ones; the k
// entries are gathered and their terms summed in 64 bits meanwhile.
//  - k_distill_loss: streams a row, or a part of one, through a workgroup.
//  - k_distill_fused: loss and gradient; the row stays in the registers of
//    its workgroup, so it is read once for both.
//  - k_distill_join: joins the parts of a row where few rows are split.
//  - k_distill_grad: streams the gradient of a row, or a part of one, from the
//    statistics.
// What bounds them is the read of the logits and the write of the gradient.
//
// Statistics kept for a later backward pass: L = log sum exp(s z) and
// log p_T.  The latter is near 0 where the entries hold little of the
// student's mass, and the gradient's tail factor (Q - q_T / p_T) p_T =
// sum q_j p_T + q_T (p_T - 1) is then made of two small terms.
#include "loss_device.h"

namespace scape {

static_assert(kRowWaves == 8, "the waves' partial sums are joined by eight lanes");
constexpr int kEntries = SCAPE_DISTILL_MAX_K / kRowThreads;  // entries a thread
static_assert(SCAPE_DISTILL_MAX_K % kRowThreads == 0, "entries are dealt out evenly");

// The bitmap: column v is bit v + 8 - head, so that a granule's columns are a
// byte of it, or half of one.
inline uint32_t bitmap_words(int64_t cols) { return (uint32_t)((cols + 8 + 31) / 32); }
template <class T>
__device__ __forceinline__ uint32_t granule_bits(const uint32_t* bitmap, int32_t i) {
    const uint8_t* bytes = reinterpret_cast<const uint8_t*>(bitmap);
    return T::kN == 8 ? bytes[1 + i] : ((uint32_t)bytes[1 + (i >> 1)] >> (4 * (i & 1))) & 15u;
}

// A row's teacher entries, thread t holding entries t, t + kRowThreads, ...
struct Entries {
    int32_t col[kEntries];  // -1: none
    float t[kEntries];      // the teacher's value
    float z[kEntries];      // the student's logit
    // kept for the gradient in float32 (the sums are over float64): each is
    // rounded once more, a step of a float32 gradient
    float q[kEntries];  // exp of the teacher's log-probability (against the wave's largest where its lse is not given)
    float p[kEntries];  // 2^x_j against the wave's largest, x_j = z_j c2
};

// Reads the row's columns; one outside the row is no entry.
__device__ __forceinline__ void read_columns(const DistillArgs& a, int64_t row, Entries& en) {
#pragma unroll
    for (int i = 0; i < kEntries; ++i) {
        const int32_t slot = (int32_t)threadIdx.x + i * kRowThreads;
        int32_t c = -1;
        if (slot < a.k) c = a.t_idx[row * a.k + slot];
        en.col[i] = c >= 0 && c < (int32_t)a.in.cols ? c : -1;
    }
}

// Reads the entries' values, and their logits for columns in [lo, hi).
template <class T>
__device__ __forceinline__ void read_values(const DistillArgs& a, int64_t row, const typename T::raw* z, int32_t lo,
                                            int32_t hi, Entries& en) {
#pragma unroll
    for (int i = 0; i < kEntries; ++i) {
        en.t[i] = en.z[i] = 0.0f;
        if (en.col[i] >= 0) {
            en.t[i] = load_any(a.t_val, a.t_dtype, row * a.k + (int32_t)threadIdx.x + i * kRowThreads);
            if (en.col[i] >= lo && en.col[i] < hi) en.z[i] = T::up1(z[en.col[i]]);
        }
    }
}

// Marks the entries' columns in the bitmap, which the workgroup has cleared
// (a barrier ago).  An entry whose column a lower slot has is dropped.
// Returns whether the row has any entry.  The bitmap is complete after it.
__device__ __forceinline__ bool mark_columns(const DistillArgs& a, int64_t row, int32_t head, uint32_t* bitmap,
                                             Entries& en) {
    uint32_t seen = 0;  // bit 0: some entry; bit 1: some column twice
#pragma unroll
    for (int i = 0; i < kEntries; ++i)
        if (en.col[i] >= 0) {
            const uint32_t at = (uint32_t)(en.col[i] + 8 - head), bit = 1u << (at & 31u);
            seen |= (atomicOr(&bitmap[at >> 5], bit) & bit) ? 3u : 1u;
        }
    const bool any = __syncthreads_or(seen != 0);
    if (!any) return false;
    if (__syncthreads_or((seen & 2u) != 0)) {
        // which of two threads came first is chance, so every entry looks for
        // its column in the slots below its own
#pragma unroll
        for (int i = 0; i < kEntries; ++i)
            if (en.col[i] >= 0) {
                const int32_t slot = (int32_t)threadIdx.x + i * kRowThreads;
                for (int32_t j = 0; j < slot; ++j)
                    if (a.t_idx[row * a.k + j] == en.col[i]) {
                        en.col[i] = -1;
                        break;
                    }
            }
    }
    return true;
}

// s t_j, minus the teacher's lse where it is given.
__device__ __forceinline__ double log_q(const DistillArgs& a, double lse, float t) {
    return t == kNegInf ? (double)t : (double)t * (double)a.scale - lse;
}

// A wave's entries summed, against the wave's own references; the row's are
// put together in finish_row.
struct WaveSums {
    double top;  // sum 2^(x_j - mt)
    double q;    // sum q_j, q_j = exp(lq_j), lq_j the teacher's log-probability less mq
    double qt;   // sum q_j lq_j
    double qx;   // sum q_j x_j
    float mt;    // the largest x_j
    float mq;    // 0 where the teacher's lse is given, else the largest s t_j
};
constexpr float kLowest = -3.402823466e38f;

// kStudent: also the student's terms.  en.q and en.p are set.
template <bool kStudent>
__device__ __forceinline__ WaveSums entry_sums(const DistillArgs& a, double lse, Entries& en) {
    WaveSums s{0.0, 0.0, 0.0, 0.0, kLowest, a.t_lse ? 0.0f : kLowest};
    bool some = false;
#pragma unroll
    for (int i = 0; i < kEntries; ++i) {
        en.q[i] = en.p[i] = 0.0f;
        if (en.col[i] >= 0) {
            some = true;
            if (kStudent) s.mt = fmaxf(s.mt, en.z[i] * a.c2);
            if (!a.t_lse) s.mq = fmaxf(s.mq, en.t[i] * a.scale);
        }
    }
    if (wave_ballot(some) == 0) return s;
    if (kStudent) s.mt = group_reduce<OpMaxNum, 64>(s.mt);
    if (!a.t_lse) s.mq = group_reduce<OpMaxNum, 64>(s.mq);
#pragma unroll
    for (int i = 0; i < kEntries; ++i)
        if (en.col[i] >= 0) {
            const double lq = log_q(a, lse, en.t[i]) - (double)s.mq, q = exp(lq);
            en.q[i] = (float)q;
            s.q += q;
            if (kStudent) {
                const double x = (double)en.z[i] * (double)a.c2, p = exp2(x - (double)s.mt);
                en.p[i] = (float)p;
                s.top += p;
                if (q != 0.0) {
                    s.qt += q * lq;
                    s.qx += q * x;
                }
            }
        }
    s.q = wave_sum_f64(s.q);
    if (kStudent) {
        s.top = wave_sum_f64(s.top);
        s.qt = wave_sum_f64(s.qt);
        s.qx = wave_sum_f64(s.qx);
    }
    return s;
}

// The row's loss, statistics and gradient factors.
struct RowResult {
    float loss;          // KL
    float stat0, stat1;  // L, log p_T
    float vref, tail;    // the tail's gradient is tail 2^(x_v - vref)
    double p, q;         // an entry's gradient is p en.p - q en.q, for the entries of this lane's wave (lane % 8)
    bool dead;           // no student mass at all: nothing to learn
};

// A whole wave calls it; lane l brings the entries' sums of wave l % 8 and
// the tail's running sum of the row.  The four logarithms of the row are one,
// on four lanes.
__device__ __forceinline__ RowResult finish_row(const DistillArgs& a, const RunningSum& tail, const WaveSums& w) {
    RowResult r;
    const double t = (double)tail.sum;
    const bool has_tail = !(t == 0.0);
    const double tref = (double)tail.ref;
    const double ref = fmax(has_tail ? tref : (double)kLowest, (double)group_reduce<OpMaxNum, 8>(w.mt));
    const double fp = exp2((double)w.mt - ref);
    const double top = sum8_f64(w.top * fp);
    double fq = 1.0, qt = w.qt;
    if (!a.t_lse) {
        const double d = (double)w.mq - (double)group_reduce<OpMaxNum, 8>(w.mq);
        fq = exp(d);
        qt += w.q != 0.0 ? w.q * d : 0.0;
    }
    const double q = sum8_f64(w.q * fq);
    qt = sum8_f64(qt * fq);
    const double qx = sum8_f64(w.qx * fq);
    const double far = has_tail ? exp2(tref - ref) : 0.0;  // 0 too where the tail is out of range
    const double sum = t * far + top;
    double qsum, rest = 0.0;
    if (a.t_lse) {
        qsum = q;
        rest = has_tail && 1.0 - qsum > 0.0 ? 1.0 - qsum : 0.0;  // no tail: its term is left out
    } else {
        qsum = q == 0.0 ? 0.0 : 1.0;  // 0: every entry's value is -inf
    }
    const uint32_t lane = lane_id();
    const double logs = log(lane == 0 ? sum : lane == 1 ? t : lane == 2 ? q : rest);
    const double log_sum = from_lane(logs, 0), log_t = from_lane(logs, 1), log_q = from_lane(logs, 2),
                 log_rest = from_lane(logs, 3);
    const double qnorm = qsum == 0.0 ? 0.0 : a.t_lse ? 1.0 : 1.0 / q;
    const double lpt = has_tail ? log_t + (tref - ref) * kLn2 - log_sum : -__builtin_inf();
    const double lse = ref * kLn2 + log_sum;
    double kl = 0.0;
    if (qsum != 0.0) {
        kl = (qt - qx * kLn2) * qnorm + qsum * lse;
        if (!a.t_lse) kl -= log_q;
    }
    if (rest > 0.0) kl += rest * (log_rest - lpt);
    const double inv = 1.0 / sum;
    r.loss = (float)kl;
    r.stat0 = (float)lse;
    r.stat1 = (float)lpt;
    r.vref = tail.ref;
    // (Q - q_T / p_T) p_v with q_T / p_T = q_T + q_T top / (t far)
    r.tail = has_tail ? (float)(inv * (qsum * far - rest * top / t)) : 0.0f;
    r.p = fp * inv * (qsum + rest);
    r.q = fq * qnorm;
    r.dead = sum == 0.0;
    return r;
}

__device__ __forceinline__ void write_row(const DistillArgs& a, int64_t row, float w, const RowResult& r) {
    a.loss[row] = r.dead ? 0.0f : w * r.loss;
    a.stats[2 * row] = r.stat0;
    a.stats[2 * row + 1] = r.stat1;
}
__device__ __forceinline__ void write_no_row(const DistillArgs& a, int64_t row) {
    a.loss[row] = 0.0f;
    a.stats[2 * row] = 0.0f;
    a.stats[2 * row + 1] = 0.0f;
}

// A workgroup's part of a row.
template <class T>
struct Part {
    using raw = typename T::raw;
    int64_t row;
    int32_t sp, n;
    const raw* z;
    RowShape sh;
    int32_t g0, cnt, first;  // first granule, granules, column of the first granule's first element
    const gran* body;
    int32_t lone;
    int32_t col0, col1;  // its columns
    __device__ __forceinline__ explicit Part(const DistillArgs& a) {
        row = blockIdx.x / (uint32_t)a.splits;
        sp = (int32_t)(blockIdx.x % (uint32_t)a.splits);
        n = (int32_t)a.in.cols;
        z = static_cast<const raw*>(a.in.z) + row * a.in.ld;
        sh = row_shape<T>(z, n);
        g0 = sp * a.per;
        cnt = max(min(a.per, sh.granules - g0), 0);
        const bool last = sp == a.splits - 1;
        first = sh.head + g0 * T::kN;
        body = reinterpret_cast<const gran*>(z + sh.head) + g0;
        lone = lone_element(sh, n, sp == 0, last);
        col0 = sp == 0 ? 0 : first;
        col1 = last ? n : first + cnt * T::kN;
    }
    __device__ __forceinline__ gran load(int32_t i) const { return i < cnt ? body[i] : no_entries<T>(); }
};

__device__ __forceinline__ void clear_bitmap(uint32_t* bitmap, int32_t n) {
    const uint32_t words = (uint32_t)(n + 8 + 31) / 32u;
    for (uint32_t i = threadIdx.x; i < words; i += kRowThreads) bitmap[i] = 0;
}

// Granule g, number i of the row, without the entries' columns.
template <class T>
__device__ __forceinline__ void strike(const uint32_t* bitmap, int32_t i, gran& g) {
    const uint32_t b = granule_bits<T>(bitmap, i);
    if (b) {
#pragma unroll
        for (int j = 0; j < T::kN; ++j)
            if (b & (1u << j)) T::set(g, j, (typename T::raw)T::kNegInfBits);
    }
}
__device__ __forceinline__ bool struck(const uint32_t* bitmap, int32_t head, int32_t col) {
    const uint32_t at = (uint32_t)(col + 8 - head);
    return (bitmap[at >> 5] >> (at & 31u)) & 1u;
}

// A row that is not read: zeros.
template <class T>
__device__ __forceinline__ void zero_part(const Part<T>& p, typename T::raw* dz) {
    for (int32_t i = (int32_t)threadIdx.x; i < p.cnt; i += kRowThreads)
        store_loose(dz + p.first + i * T::kN, gran{0u, 0u, 0u, 0u});
    if (p.lone >= 0) dz[p.lone] = 0;
}

// kPart: only the part's running sum of the tail, for k_distill_join.
// Four granules a thread are worked on while the next four are on their way.
template <class T, bool kPart>
__global__ __launch_bounds__(kRowThreads, 8) void k_distill_loss(DistillArgs a) {
    extern __shared__ uint32_t bitmap[];
    __shared__ float2 wsum[kRowWaves];
    __shared__ WaveSums wrec[kRowWaves];
    constexpr int kBatch = 4, kStep = kBatch * kRowThreads;
    const int32_t tid = (int32_t)threadIdx.x, wave = tid / 64;
    const Part<T> p(a);
    const float w = a.weight ? a.weight[p.row] : 1.0f;
    gran g[kBatch], next[kBatch];
    float lx = kNegInf;
    Entries en;
    double t_lse = 0.0;
    bool alive = false;
    if (w != 0.0f) {
        read_columns(a, p.row, en);
#pragma unroll
        for (int b = 0; b < kBatch; ++b) g[b] = p.load(tid + b * kRowThreads);
        if (p.lone >= 0) lx = T::up1(p.z[p.lone]);
        read_values<T>(a, p.row, p.z, 0, kPart ? 0 : p.n, en);
        if (!kPart && a.t_lse) t_lse = (double)a.t_lse[p.row];
        clear_bitmap(bitmap, p.n);
        __syncthreads();
        alive = mark_columns(a, p.row, p.sh.head, bitmap, en);
    }
    if (!alive) {  // the same for the whole workgroup
        if (tid == 0) {
            if (kPart)
                a.part[p.row * a.splits + p.sp] = make_float2(0.0f, 0.0f);
            else
                write_no_row(a, p.row);
        }
        return;
    }
    RunningSum rs = RunningSum::none();
    if (p.lone >= 0 && !struck(bitmap, p.sh.head, p.lone)) rs.add1(lx, a.c2);
    for (int32_t base = 0; base < p.cnt; base += kStep) {
        const int32_t i = base + tid;
        if (base + kStep < p.cnt) {
#pragma unroll
            for (int b = 0; b < kBatch; ++b) next[b] = p.load(i + kStep + b * kRowThreads);
        }
        float m = kNegInf;
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            if (i + b * kRowThreads < p.cnt) strike<T>(bitmap, p.g0 + i + b * kRowThreads, g[b]);
            m = max_nan(m, granule_max<T>(g[b]));
        }
        rs.template add<T, kBatch>(g, m, a.c2);
#pragma unroll
        for (int b = 0; b < kBatch; ++b) g[b] = next[b];
    }
    wave_join(rs);
    if ((tid & 63) == 0) wsum[wave] = make_float2(rs.ref, rs.sum);
    if constexpr (!kPart) {
        const WaveSums ws = entry_sums<true>(a, t_lse, en);
        if ((tid & 63) == 0) wrec[wave] = ws;
    }
    __syncthreads();
    if (wave == 0) {
        RunningSum r{wsum[tid & 7].x, wsum[tid & 7].y};
        join8(r);
        if constexpr (kPart) {
            if (tid == 0) a.part[p.row * a.splits + p.sp] = make_float2(r.ref, r.sum);
        } else {
            const RowResult res = finish_row(a, r, wrec[tid & 7]);
            if (tid == 0) write_row(a, p.row, w, res);
        }
    }
}

// Writes the entries' columns: d_j = fp en.p - fq en.q.
template <class T>
__device__ __forceinline__ void write_entries(const Part<T>& p, const Entries& en, float gs, double fp, double fq,
                                              typename T::raw* dz) {
#pragma unroll
    for (int i = 0; i < kEntries; ++i)
        if (en.col[i] >= p.col0 && en.col[i] < p.col1)
            dz[en.col[i]] = gs == 0.0f ? (typename T::raw)0
                                       : T::down1((float)((double)gs * (fp * (double)en.p[i] - fq * (double)en.q[i])));
}

// Loss and gradient of whole rows, kGran granules a thread.
template <class T, int kGran>
__global__ __launch_bounds__(kRowThreads, row_waves(kGran)) void k_distill_fused(DistillArgs a) {
    extern __shared__ uint32_t bitmap[];
    __shared__ float2 wsum[kRowWaves];
    __shared__ WaveSums wrec[kRowWaves];
    __shared__ double s_p[kRowWaves], s_q[kRowWaves];
    __shared__ float s_vref, s_tail, s_gs;
    constexpr int kBatch = kGran < 4 ? kGran : 4;
    using raw = typename T::raw;
    const int32_t tid = (int32_t)threadIdx.x, wave = tid / 64;
    const Part<T> p(a);
    raw* dz = static_cast<raw*>(a.dz) + p.row * a.ld_dz;
    const float w = a.weight ? a.weight[p.row] : 1.0f;
    gran g[kGran];
    float lx = kNegInf;
    Entries en;
    double t_lse = 0.0;
    bool alive = false;
    if (w != 0.0f) {
        read_columns(a, p.row, en);
#pragma unroll
        for (int c = 0; c < kGran; ++c) g[c] = p.load(tid + c * kRowThreads);
        if (p.lone >= 0) lx = T::up1(p.z[p.lone]);
        read_values<T>(a, p.row, p.z, 0, p.n, en);
        if (a.t_lse) t_lse = (double)a.t_lse[p.row];
        clear_bitmap(bitmap, p.n);
        __syncthreads();
        alive = mark_columns(a, p.row, p.sh.head, bitmap, en);
    }
    if (!alive) {  // the same for the whole workgroup
        if (tid == 0) write_no_row(a, p.row);
        zero_part(p, dz);
        return;
    }
    RunningSum rs = RunningSum::none();
    if (p.lone >= 0 && !struck(bitmap, p.sh.head, p.lone)) rs.add1(lx, a.c2);
    const int32_t tid1 = again(tid);
#pragma unroll
    for (int c = 0; c < kGran; c += kBatch)
        if (c * kRowThreads < p.cnt) {
            gran x[kBatch];
            float m = kNegInf;
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                const int32_t i = tid1 + (c + b) * kRowThreads;
                if (i < p.cnt) strike<T>(bitmap, i, g[c + b]);
                x[b] = g[c + b];
                m = max_nan(m, granule_max<T>(x[b]));
            }
            rs.template add<T, kBatch>(x, m, a.c2);
        }
    wave_join(rs);
    if ((tid & 63) == 0) wsum[wave] = make_float2(rs.ref, rs.sum);
    {
        const WaveSums ws = entry_sums<true>(a, t_lse, en);
        if ((tid & 63) == 0) wrec[wave] = ws;
    }
    __syncthreads();
    if (wave == 0) {
        RunningSum r{wsum[tid & 7].x, wsum[tid & 7].y};
        join8(r);
        const RowResult res = finish_row(a, r, wrec[tid & 7]);
        if (tid < kRowWaves) {
            s_p[tid] = res.p;
            s_q[tid] = res.q;
        }
        if (tid == 0) {
            write_row(a, p.row, w, res);
            const float gs = res.dead ? 0.0f : w * a.scale;
            s_gs = gs;
            s_tail = gs == 0.0f ? 0.0f : gs * res.tail;
            s_vref = gs == 0.0f ? -kNegInf : res.vref;  // nothing to learn: exponents of -inf
        }
    }
    __syncthreads();
    const float f = s_tail, vref = s_vref;
    const int32_t tid2 = again(tid);
#pragma unroll
    for (int c = 0; c < kGran; ++c) {
        const int32_t i = tid2 + c * kRowThreads;
        forget_unpacked(g[c]);
        if (i < p.cnt) {
            float d[T::kN];
#pragma unroll
            for (int j = 0; j < T::kN; ++j) d[j] = f * fast_exp2(__builtin_fmaf(T::up(g[c], j), a.c2, -vref));
            store_loose(dz + p.first + i * T::kN, T::down(d));
        }
    }
    if (p.lone >= 0) dz[p.lone] = T::down1(f * fast_exp2(__builtin_fmaf(lx, a.c2, -vref)));
    __syncthreads();  // the entries' columns are written over the tail's values
    write_entries(p, en, s_gs, s_p[wave], s_q[wave], dz);
}

// The gradient of a row or a part of one, from the statistics.
template <class T>
__global__ __launch_bounds__(kRowThreads, 8) void k_distill_grad(DistillArgs a) {
    extern __shared__ uint32_t bitmap[];
    __shared__ WaveSums wrec[kRowWaves];
    __shared__ double s_p, s_q[kRowWaves];
    __shared__ float s_vref, s_tail, s_gs;
    constexpr int kBatch = 4, kStep = kBatch * kRowThreads;
    using raw = typename T::raw;
    const int32_t tid = (int32_t)threadIdx.x, wave = tid / 64;
    const Part<T> p(a);
    raw* dz = static_cast<raw*>(a.dz) + p.row * a.ld_dz;
    float w = a.weight ? a.weight[p.row] : 1.0f;
    if (a.dloss) w = w == 0.0f ? 0.0f : w * a.dloss[p.row];
    gran g[kBatch], next[kBatch];
    float lx = kNegInf;
    Entries en;
    double t_lse = 0.0;
    bool alive = false;
    if (w != 0.0f) {
        read_columns(a, p.row, en);
#pragma unroll
        for (int b = 0; b < kBatch; ++b) g[b] = p.load(tid + b * kRowThreads);
        if (p.lone >= 0) lx = T::up1(p.z[p.lone]);
        // dz may be z, and other workgroups write their parts of it: only
        // this part's logits are read
        read_values<T>(a, p.row, p.z, p.col0, p.col1, en);
        if (a.t_lse) t_lse = (double)a.t_lse[p.row];
        clear_bitmap(bitmap, p.n);
        __syncthreads();
        alive = mark_columns(a, p.row, p.sh.head, bitmap, en);
    }
    if (!alive) {  // the same for the whole workgroup
        zero_part(p, dz);
        return;
    }
    {
        const WaveSums ws = entry_sums<false>(a, t_lse, en);
        if ((tid & 63) == 0) wrec[wave] = ws;
    }
    const float l = a.stats[2 * p.row], lpt = a.stats[2 * p.row + 1];
#pragma unroll
    for (int i = 0; i < kEntries; ++i)
        if (en.col[i] >= 0) en.p[i] = (float)exp((double)en.z[i] * (double)a.scale - (double)l);
    __syncthreads();
    if (wave == 0) {
        const WaveSums r = wrec[tid & 7];
        const double fq = a.t_lse ? 1.0 : exp((double)r.mq - (double)group_reduce<OpMaxNum, 8>(r.mq));
        const double q = sum8_f64(r.q * fq);
        const double qsum = a.t_lse ? q : q == 0.0 ? 0.0 : 1.0;
        const double rest = a.t_lse && 1.0 - q > 0.0 && lpt != kNegInf ? 1.0 - q : 0.0;
        // (Q - q_T / p_T) p_v, against L, or where 1 / p_T could leave the
        // range against the tail's own log-sum-exp
        float v = l, tail = (float)qsum;
        if (rest > 0.0) {
            const double pt = exp((double)lpt), c = qsum * pt + rest * (pt - 1.0);
            const bool near = lpt > -30.0f;
            tail = (float)(near ? c / pt : c);
            if (!near) v = (float)((double)l + (double)lpt);
        }
        if (tid < kRowWaves) s_q[tid] = fq * (qsum == 0.0 ? 0.0 : a.t_lse ? 1.0 : 1.0 / q);
        if (tid == 0) {
            const float gs = l == kNegInf ? 0.0f : w * a.scale;
            s_p = qsum + rest;
            s_gs = gs;
            s_tail = gs == 0.0f ? 0.0f : gs * tail;
            s_vref = gs == 0.0f ? -kNegInf : v;  // nothing to learn: exponents of -inf
        }
    }
    __syncthreads();
    const float f = s_tail, vref = s_vref;
    // A float32 gradient takes the difference from L first: it would see the
    // rounding of L log2(e), which a 16-bit one does not.
    const float vref2 = vref * kLog2e;
    auto grad = [&](float x) {
        const float e = T::kN == 4 ? __builtin_fmaf(x, a.scale, -vref) * kLog2e : __builtin_fmaf(x, a.c2, -vref2);
        return f * fast_exp2(e);
    };
    for (int32_t base = 0; base < p.cnt; base += kStep) {
        const int32_t i = base + tid;
        if (base + kStep < p.cnt) {
#pragma unroll
            for (int b = 0; b < kBatch; ++b) next[b] = p.load(i + kStep + b * kRowThreads);
        }
#pragma unroll
        for (int b = 0; b < kBatch; ++b)
            if (i + b * kRowThreads < p.cnt) {
                float d[T::kN];
#pragma unroll
                for (int j = 0; j < T::kN; ++j) d[j] = grad(T::up(g[b], j));
                store_loose(dz + p.first + (i + b * kRowThreads) * T::kN, T::down(d));
            }
#pragma unroll
        for (int b = 0; b < kBatch; ++b) g[b] = next[b];
    }
    if (p.lone >= 0) dz[p.lone] = T::down1(grad(lx));
    __syncthreads();  // the entries' columns are written over the tail's values
    write_entries(p, en, s_gs, s_p, s_q[wave], dz);
}

// Joins the parts of a split row: the loss and the statistics.
template <class T>
__global__ __launch_bounds__(kRowThreads) void k_distill_join(DistillArgs a) {
    extern __shared__ uint32_t bitmap[];
    __shared__ WaveSums wrec[kRowWaves];
    using raw = typename T::raw;
    const int32_t tid = (int32_t)threadIdx.x, wave = tid / 64, n = (int32_t)a.in.cols;
    const int64_t row = blockIdx.x;
    const raw* z = static_cast<const raw*>(a.in.z) + row * a.in.ld;
    const float w = a.weight ? a.weight[row] : 1.0f;
    Entries en;
    double t_lse = 0.0;
    bool alive = false;
    RunningSum r = RunningSum::none();  // of lane s: part s
    if (w != 0.0f) {
        read_columns(a, row, en);
        read_values<T>(a, row, z, 0, n, en);
        if (a.t_lse) t_lse = (double)a.t_lse[row];
        if ((tid & 63) < a.splits) {
            const float2 p = a.part[row * a.splits + (tid & 63)];
            r = RunningSum{p.x, p.y};
        }
        clear_bitmap(bitmap, n);
        __syncthreads();
        alive = mark_columns(a, row, 0, bitmap, en);
    }
    if (!alive) {
        if (tid == 0) write_no_row(a, row);
        return;
    }
    const WaveSums ws = entry_sums<true>(a, t_lse, en);
    if ((tid & 63) == 0) wrec[wave] = ws;
    __syncthreads();
    if (wave == 0) {
        wave_join(r);
        const RowResult res = finish_row(a, r, wrec[tid & 7]);
        if (tid == 0) write_row(a, row, w, res);
    }
}

static size_t bitmap_bytes(const DistillArgs& a) { return bitmap_words(a.in.cols) * sizeof(uint32_t); }
static dim3 parts(const DistillArgs& a) { return dim3((uint32_t)(a.in.rows * a.splits)); }

template <class T>
static hipError_t backward_typed(hipStream_t s, const DistillArgs& a) {
    hipLaunchKernelGGL((k_distill_grad<T>), parts(a), dim3(kRowThreads), bitmap_bytes(a), s, a);
    return hipGetLastError();
}

template <class T>
static hipError_t forward_typed(hipStream_t s, const DistillArgs& a) {
    const size_t lds = bitmap_bytes(a);
    const int32_t each = (a.per + kRowThreads - 1) / kRowThreads;
    if (a.splits > 1) {
        hipLaunchKernelGGL((k_distill_loss<T, true>), parts(a), dim3(kRowThreads), lds, s, a);
        hipLaunchKernelGGL((k_distill_join<T>), dim3((uint32_t)a.in.rows), dim3(kRowThreads), lds, s, a);
    } else if (a.dz && each <= kRowGranules) {
        if (each <= 4) hipLaunchKernelGGL((k_distill_fused<T, 4>), parts(a), dim3(kRowThreads), lds, s, a);
        else if (each <= 8) hipLaunchKernelGGL((k_distill_fused<T, 8>), parts(a), dim3(kRowThreads), lds, s, a);
        else hipLaunchKernelGGL((k_distill_fused<T, kRowGranules>), parts(a), dim3(kRowThreads), lds, s, a);
        return hipGetLastError();
    } else {
        hipLaunchKernelGGL((k_distill_loss<T, false>), parts(a), dim3(kRowThreads), lds, s, a);
    }
    const hipError_t e = hipGetLastError();
    return e != hipSuccess || !a.dz ? e : backward_typed<T>(s, a);
}

hipError_t launch_distill_forward(hipStream_t s, const DistillArgs& a) {
    if (a.in.dtype == SCAPE_DTYPE_F32) return forward_typed<F32>(s, a);
    if (a.in.dtype == SCAPE_DTYPE_BF16) return forward_typed<BF16>(s, a);
    return forward_typed<F16>(s, a);
}

hipError_t launch_distill_backward(hipStream_t s, const DistillArgs& a) {
    if (a.in.dtype == SCAPE_DTYPE_F32) return backward_typed<F32>(s, a);
    if (a.in.dtype == SCAPE_DTYPE_BF16) return backward_typed<BF16>(s, a);
    return backward_typed<F16>(s, a);
}

}  // namespace scape
