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
#include <type_traits>

#include "loss_device.h"

namespace scape {

// LDS of a workgroup: a bitmap of the row's columns, then the row's k slots:
// column (-1: no entry), teacher's value and student's logit.
//
// The bitmap lies as a thread's granules do, four of them (tid, tid + threads,
// ...) in one cell: whether a thread's next four granules hold an entry is one
// read and one test.  The lone elements beside the granules have 16 bits of
// their own behind the cells.
template <class T, int kThreads>
struct Bitmap {
    using Cell = std::conditional_t<T::kN == 8, uint32_t, uint16_t>;
    static constexpr int kCellBits = 4 * T::kN, kCellGranules = 4 * kThreads;
    Cell* cells;
    RowShape sh;
    int32_t n;
    static __host__ __device__ int32_t cell_count(int32_t granules) {
        return (granules + kCellGranules - 1) / kCellGranules * kThreads;
    }
    // for rows of at most this many granules
    static __host__ __device__ int32_t bytes(int32_t granules) {
        return (cell_count(granules) * (int32_t)sizeof(Cell) + 4 + 15) / 16 * 16;
    }
    __device__ __forceinline__ uint32_t bit_of(int32_t col) const {
        const int32_t e = col - sh.head, i = e / T::kN;
        if (e >= 0 && i < sh.granules) {
            const int32_t cell = i / kCellGranules * kThreads + i % kThreads;
            return (uint32_t)(cell * kCellBits + (i / kThreads & 3) * T::kN + e % T::kN);
        }
        return (uint32_t)(cell_count(sh.granules) * kCellBits + (e < 0 ? col : 8 + col - (n - sh.tail)));
    }
    __device__ __forceinline__ void clear() const {
        const int32_t words = bytes(sh.granules) / 4;
        uint32_t* w = reinterpret_cast<uint32_t*>(cells);
        for (int32_t i = (int32_t)threadIdx.x; i < words; i += kThreads) w[i] = 0;
    }
    // whether it was set before
    __device__ __forceinline__ bool set(int32_t col) const {
        const uint32_t at = bit_of(col), bit = 1u << (at & 31u);
        return (atomicOr(reinterpret_cast<uint32_t*>(cells) + (at >> 5), bit) & bit) != 0;
    }
    __device__ __forceinline__ bool has(int32_t col) const {
        const uint32_t at = bit_of(col);
        return (reinterpret_cast<const uint32_t*>(cells)[at >> 5] >> (at & 31u)) & 1u;
    }
    // Strikes the entries out of the thread's granules tid + (b + 4 c) kThreads, b < 4, c = cell_row.
    __device__ __forceinline__ void strike(int32_t cell_row, gran (&g)[4]) const {
        const uint32_t bits = cells[cell_row * kThreads + (int32_t)threadIdx.x];
        if (bits) {
#pragma unroll
            for (int b = 0; b < 4; ++b)
#pragma unroll
                for (int j = 0; j < T::kN; ++j)
                    if (bits & (1u << (b * T::kN + j))) T::set(g[b], j, (typename T::raw)T::kNegInfBits);
        }
    }
};

// The k slots of a row.  Slot tid's values wait in registers until the row's
// logits have gone by; t and z hold the entry's terms q and p afterwards.
struct Slots {
    int32_t* col;
    float* t;
    float* z;
    float t0, z0;
};
inline int32_t slot_bytes(int32_t k) { return 12 * k; }

// Column of a slot; one outside the row is no entry.
__device__ __forceinline__ int32_t slot_column(const DistillArgs& a, int64_t row, int32_t slot) {
    const int32_t c = slot < a.k ? a.t_idx[row * a.k + slot] : -1;
    return c >= 0 && c < (int32_t)a.in.cols ? c : -1;
}

// Reads the slots' values, logits for columns in [lo, hi) only (hi = 0: no
// values at all), and marks the columns.  c0 is slot tid's column.  An entry
// whose column a lower slot has is dropped.  The bitmap has been cleared, by
// this workgroup, without a barrier since; it is complete afterwards.  Returns
// whether the row has any entry.
template <class T, int kThreads>
__device__ __forceinline__ bool read_slots(const DistillArgs& a, int64_t row, const typename T::raw* z, int32_t lo,
                                           int32_t hi, int32_t c0, const Bitmap<T, kThreads>& bitmap, Slots& s) {
    const int32_t tid = (int32_t)threadIdx.x;
    __syncthreads();
    uint32_t seen = 0;  // bit 0: some entry; bit 1: some column twice
    s.t0 = s.z0 = 0.0f;
    for (int32_t slot = tid; slot < a.k; slot += kThreads) {
        const int32_t c = slot == tid ? c0 : slot_column(a, row, slot);
        s.col[slot] = c;
        if (c < 0) continue;
        float t = 0.0f, x = 0.0f;
        if (hi > 0) t = load_any(a.t_val, a.t_dtype, row * a.k + slot);
        if (c >= lo && c < hi) x = T::up1(z[c]);
        if (slot == tid) {
            s.t0 = t;
            s.z0 = x;
        } else {
            s.t[slot] = t;
            s.z[slot] = x;
        }
        seen |= bitmap.set(c) ? 3u : 1u;
    }
    if (!__syncthreads_or((int)seen)) return false;
    if (__syncthreads_or((int)(seen & 2u))) {
        // which of two threads came first is chance, so every entry looks for
        // its column in the slots below its own
        for (int32_t slot = tid; slot < a.k; slot += kThreads) {
            const int32_t c = s.col[slot];
            for (int32_t j = 0; j < slot && c >= 0; ++j)
                if (a.t_idx[row * a.k + j] == c) {
                    s.col[slot] = -1;
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

// kStudent: also the student's terms.  Slots' t and z become q and p, for the
// gradient, in float32: each is rounded once more, a step of a float32
// gradient (the sums are over float64).
template <int kThreads, bool kStudent>
__device__ __forceinline__ WaveSums entry_sums(const DistillArgs& a, double lse, Slots& sl) {
    const int32_t tid = (int32_t)threadIdx.x;
    WaveSums s{0.0, 0.0, 0.0, 0.0, kLowest, a.t_lse ? 0.0f : kLowest};
    if (tid < a.k) {
        sl.t[tid] = sl.t0;
        sl.z[tid] = sl.z0;
    }
    bool some = false;
    for (int32_t slot = tid; slot < a.k; slot += kThreads)
        if (sl.col[slot] >= 0) {
            some = true;
            if (kStudent) s.mt = fmaxf(s.mt, sl.z[slot] * a.c2);
            if (!a.t_lse) s.mq = fmaxf(s.mq, sl.t[slot] * a.scale);
        }
    if (wave_ballot(some) == 0) return s;
    if (kStudent) s.mt = group_reduce<OpMaxNum, 64>(s.mt);
    if (!a.t_lse) s.mq = group_reduce<OpMaxNum, 64>(s.mq);
    for (int32_t slot = tid; slot < a.k; slot += kThreads)
        if (sl.col[slot] >= 0) {
            const double lq = log_q(a, lse, sl.t[slot]) - (double)s.mq, q = exp(lq);
            sl.t[slot] = (float)q;
            s.q += q;
            if (kStudent) {
                const double x = (double)sl.z[slot] * (double)a.c2, p = exp2(x - (double)s.mt);
                sl.z[slot] = (float)p;
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
    double p, q;         // an entry's gradient is p p_j - q q_j, for the entries of this lane's wave (lane % kWaves)
    bool dead;           // no student mass at all: nothing to learn
};

// A whole wave calls it; lane l brings the entries' sums of wave l % kWaves
// and the tail's running sum of the row.  The four logarithms of the row are
// one, on four lanes.
template <int kWaves>
__device__ __forceinline__ RowResult finish_row(const DistillArgs& a, const RunningSum& tail, const WaveSums& w) {
    RowResult r;
    const double t = (double)tail.sum;
    const bool has_tail = !(t == 0.0);
    const double tref = (double)tail.ref;
    const double ref = fmax(has_tail ? tref : (double)kLowest, (double)group_reduce<OpMaxNum, kWaves>(w.mt));
    const double fp = exp2((double)w.mt - ref);
    const double top = sum_waves_f64<kWaves>(w.top * fp);
    double fq = 1.0, qt = w.qt;
    if (!a.t_lse) {
        const double d = (double)w.mq - (double)group_reduce<OpMaxNum, kWaves>(w.mq);
        fq = exp(d);
        qt += w.q != 0.0 ? w.q * d : 0.0;
    }
    const double q = sum_waves_f64<kWaves>(w.q * fq);
    qt = sum_waves_f64<kWaves>(qt * fq);
    const double qx = sum_waves_f64<kWaves>(w.qx * fq);
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
    // four granules of a thread, from number base + tid on
    template <int kThreads>
    __device__ __forceinline__ void load(int32_t base, gran (&g)[4]) const {
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const int32_t i = base + (int32_t)threadIdx.x + b * kThreads;
            g[b] = no_entries<T>();
            if (i < cnt) g[b] = granule_at(body, i);
        }
    }
};

// A row that is not read: zeros.
template <class T, int kThreads>
__device__ __forceinline__ void zero_part(const Part<T>& p, typename T::raw* dz) {
    for (int32_t i = (int32_t)threadIdx.x; i < p.cnt; i += kThreads)
        store_loose(dz + p.first, i, gran{0u, 0u, 0u, 0u});
    if (p.lone >= 0) dz[p.lone] = 0;
}

template <class T, int kThreads>
__device__ __forceinline__ void lds_layout(const DistillArgs& a, const RowShape& sh, uint8_t* lds,
                                           Bitmap<T, kThreads>& bitmap, Slots& s) {
    bitmap.cells = reinterpret_cast<typename Bitmap<T, kThreads>::Cell*>(lds);
    bitmap.sh = sh;
    bitmap.n = (int32_t)a.in.cols;
    s.col = reinterpret_cast<int32_t*>(lds + Bitmap<T, kThreads>::bytes(sh.granules));
    s.t = reinterpret_cast<float*>(s.col + a.k);
    s.z = s.t + a.k;
}

// kPart: only the part's running sum of the tail, for k_distill_join.
// Four granules a thread are worked on while the next four are on their way.
template <class T, bool kPart>
__global__ __launch_bounds__(kStreamThreads, 8) void k_distill_loss(DistillArgs a) {
    constexpr int kThreads = kStreamThreads, kNW = kThreads / 64, kStep = 4 * kThreads;
    extern __shared__ __align__(16) uint8_t lds[];
    __shared__ float2 wsum[kNW];
    __shared__ WaveSums wrec[kNW];
    const int32_t tid = (int32_t)threadIdx.x, wave = tid / 64;
    const Part<T> p(a);
    const float w = a.weight ? a.weight[p.row] : 1.0f;
    Bitmap<T, kThreads> bitmap;
    Slots slots;
    lds_layout(a, p.sh, lds, bitmap, slots);
    gran g[4], next[4];
    float lx = kNegInf;
    double t_lse = 0.0;
    bool alive = false;
    if (w != 0.0f) {
        const int32_t c0 = slot_column(a, p.row, tid);
        p.template load<kThreads>(0, g);
        if (p.lone >= 0) lx = T::up1(p.z[p.lone]);
        if (!kPart && a.t_lse) t_lse = (double)a.t_lse[p.row];
        bitmap.clear();
        alive = read_slots<T, kThreads>(a, p.row, p.z, 0, kPart ? 0 : p.n, c0, bitmap, slots);
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
    if (p.lone >= 0 && !bitmap.has(p.lone)) rs.add1(lx, a.c2);
    for (int32_t base = 0; base < p.cnt; base += kStep) {
        if (base + kStep < p.cnt) p.template load<kThreads>(base + kStep, next);
        bitmap.strike((p.g0 + base) / kStep, g);
        float m = granule_max<T>(g[0]);
#pragma unroll
        for (int b = 1; b < 4; ++b) m = max_nan(m, granule_max<T>(g[b]));
        rs.template add<T, 4>(g, m, a.c2);
#pragma unroll
        for (int b = 0; b < 4; ++b) g[b] = next[b];
    }
    wave_join(rs);
    if ((tid & 63) == 0) wsum[wave] = make_float2(rs.ref, rs.sum);
    if constexpr (!kPart) {
        const WaveSums ws = entry_sums<kThreads, true>(a, t_lse, slots);
        if ((tid & 63) == 0) wrec[wave] = ws;
    }
    __syncthreads();
    if (wave == 0) {
        RunningSum r{wsum[tid & (kNW - 1)].x, wsum[tid & (kNW - 1)].y};
        join_waves<kNW>(r);
        if constexpr (kPart) {
            if (tid == 0) a.part[p.row * a.splits + p.sp] = make_float2(r.ref, r.sum);
        } else {
            const RowResult res = finish_row<kNW>(a, r, wrec[tid & (kNW - 1)]);
            if (tid == 0) write_row(a, p.row, w, res);
        }
    }
}

// Writes the entries' columns: d_j = gs (fp p_j - fq q_j).
template <class T, int kThreads>
__device__ __forceinline__ void write_entries(const DistillArgs& a, const Part<T>& p, const Slots& s, float gs,
                                              double fp, double fq, typename T::raw* dz) {
    for (int32_t slot = (int32_t)threadIdx.x; slot < a.k; slot += kThreads) {
        const int32_t c = s.col[slot];
        if (c < 0 || c < p.col0 || c >= p.col1) continue;
        const double d = (double)gs * (fp * (double)s.z[slot] - fq * (double)s.t[slot]);
        dz[c] = gs == 0.0f ? (typename T::raw)0 : T::down1((float)d);
    }
}

// Loss and gradient of whole rows, kGran granules a thread.
template <class T, int kThreads, int kGran>
__global__ __launch_bounds__(kThreads, 4) void k_distill_fused(DistillArgs a) {
    constexpr int kNW = kThreads / 64;
    extern __shared__ __align__(16) uint8_t lds[];
    __shared__ float2 wsum[kNW];
    __shared__ WaveSums wrec[kNW];
    __shared__ double s_p[kNW], s_q[kNW];
    __shared__ float s_vref, s_tail, s_gs;
    using raw = typename T::raw;
    const int32_t tid = (int32_t)threadIdx.x, wave = tid / 64;
    const Part<T> p(a);
    raw* dz = static_cast<raw*>(a.dz) + p.row * a.ld_dz;
    const float w = a.weight ? a.weight[p.row] : 1.0f;
    Bitmap<T, kThreads> bitmap;
    Slots slots;
    lds_layout(a, p.sh, lds, bitmap, slots);
    gran g[kGran / 4][4];
    float lx = kNegInf;
    double t_lse = 0.0;
    bool alive = false;
    if (w != 0.0f) {
        const int32_t c0 = slot_column(a, p.row, tid);
#pragma unroll
        for (int c = 0; c < kGran / 4; ++c) p.template load<kThreads>(c * 4 * kThreads, g[c]);
        if (p.lone >= 0) lx = T::up1(p.z[p.lone]);
        if (a.t_lse) t_lse = (double)a.t_lse[p.row];
        bitmap.clear();
        alive = read_slots<T, kThreads>(a, p.row, p.z, 0, p.n, c0, bitmap, slots);
    }
    if (!alive) {  // the same for the whole workgroup
        if (tid == 0) write_no_row(a, p.row);
        zero_part<T, kThreads>(p, dz);
        return;
    }
    RunningSum rs = RunningSum::none();
    if (p.lone >= 0 && !bitmap.has(p.lone)) rs.add1(lx, a.c2);
#pragma unroll
    for (int c = 0; c < kGran / 4; ++c)
        if (c * 4 * kThreads < p.cnt) {
            bitmap.strike(c, g[c]);
            float m = granule_max<T>(g[c][0]);
#pragma unroll
            for (int b = 1; b < 4; ++b) m = max_nan(m, granule_max<T>(g[c][b]));
            rs.template add<T, 4>(g[c], m, a.c2);
        }
    wave_join(rs);
    if ((tid & 63) == 0) wsum[wave] = make_float2(rs.ref, rs.sum);
    {
        const WaveSums ws = entry_sums<kThreads, true>(a, t_lse, slots);
        if ((tid & 63) == 0) wrec[wave] = ws;
    }
    __syncthreads();
    if (wave == 0) {
        RunningSum r{wsum[tid & (kNW - 1)].x, wsum[tid & (kNW - 1)].y};
        join_waves<kNW>(r);
        const RowResult res = finish_row<kNW>(a, r, wrec[tid & (kNW - 1)]);
        if (tid < kNW) {
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
        const int32_t i = tid2 + c * kThreads;
        gran& x = g[c / 4][c % 4];
        forget_unpacked(x);
        if (i < p.cnt) {
            float d[T::kN];
#pragma unroll
            for (int j = 0; j < T::kN; ++j) d[j] = f * fast_exp2(__builtin_fmaf(T::up(x, j), a.c2, -vref));
            store_loose(dz + p.first, i, T::down(d));
        }
    }
    if (p.lone >= 0) dz[p.lone] = T::down1(f * fast_exp2(__builtin_fmaf(lx, a.c2, -vref)));
    __syncthreads();  // the entries' columns are written over the tail's values
    write_entries<T, kThreads>(a, p, slots, s_gs, s_p[wave], s_q[wave], dz);
}

// The gradient of a row or a part of one, from the statistics.
template <class T>
__global__ __launch_bounds__(kStreamThreads, 8) void k_distill_grad(DistillArgs a) {
    constexpr int kThreads = kStreamThreads, kNW = kThreads / 64, kStep = 4 * kThreads;
    extern __shared__ __align__(16) uint8_t lds[];
    __shared__ WaveSums wrec[kNW];
    __shared__ double s_p, s_q[kNW];
    __shared__ float s_vref, s_tail, s_gs;
    using raw = typename T::raw;
    const int32_t tid = (int32_t)threadIdx.x, wave = tid / 64;
    const Part<T> p(a);
    raw* dz = static_cast<raw*>(a.dz) + p.row * a.ld_dz;
    float w = a.weight ? a.weight[p.row] : 1.0f;
    if (a.dloss) w = w == 0.0f ? 0.0f : w * a.dloss[p.row];
    Bitmap<T, kThreads> bitmap;
    Slots slots;
    lds_layout(a, p.sh, lds, bitmap, slots);
    gran g[4], next[4];
    float lx = kNegInf;
    double t_lse = 0.0;
    bool alive = false;
    if (w != 0.0f) {
        const int32_t c0 = slot_column(a, p.row, tid);
        p.template load<kThreads>(0, g);
        if (p.lone >= 0) lx = T::up1(p.z[p.lone]);
        if (a.t_lse) t_lse = (double)a.t_lse[p.row];
        bitmap.clear();
        // dz may be z, and other workgroups write their parts of it: only
        // this part's logits are read
        alive = read_slots<T, kThreads>(a, p.row, p.z, p.col0, p.col1, c0, bitmap, slots);
    }
    if (!alive) {  // the same for the whole workgroup
        zero_part<T, kThreads>(p, dz);
        return;
    }
    const float l = a.stats[2 * p.row], lpt = a.stats[2 * p.row + 1];
    {
        const WaveSums ws = entry_sums<kThreads, false>(a, t_lse, slots);
        if ((tid & 63) == 0) wrec[wave] = ws;
    }
    for (int32_t slot = tid; slot < a.k; slot += kThreads)
        slots.z[slot] = (float)exp((double)slots.z[slot] * (double)a.scale - (double)l);
    __syncthreads();
    if (wave == 0) {
        const WaveSums r = wrec[tid & (kNW - 1)];
        const double fq = a.t_lse ? 1.0 : exp((double)r.mq - (double)group_reduce<OpMaxNum, kNW>(r.mq));
        const double q = sum_waves_f64<kNW>(r.q * fq);
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
        if (tid < kNW) s_q[tid] = fq * (qsum == 0.0 ? 0.0 : a.t_lse ? 1.0 : 1.0 / q);
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
        if (base + kStep < p.cnt) p.template load<kThreads>(base + kStep, next);
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const int32_t i = base + tid + b * kThreads;
            if (i < p.cnt) {
                float d[T::kN];
#pragma unroll
                for (int j = 0; j < T::kN; ++j) d[j] = grad(T::up(g[b], j));
                store_loose(dz + p.first, i, T::down(d));
            }
        }
#pragma unroll
        for (int b = 0; b < 4; ++b) g[b] = next[b];
    }
    if (p.lone >= 0) dz[p.lone] = T::down1(grad(lx));
    __syncthreads();  // the entries' columns are written over the tail's values
    write_entries<T, kThreads>(a, p, slots, s_gs, s_p, s_q[wave], dz);
}

// Joins the parts of a split row: the loss and the statistics.
template <class T>
__global__ __launch_bounds__(kStreamThreads) void k_distill_join(DistillArgs a) {
    constexpr int kThreads = kStreamThreads, kNW = kThreads / 64;
    extern __shared__ __align__(16) uint8_t lds[];
    __shared__ WaveSums wrec[kNW];
    using raw = typename T::raw;
    const int32_t tid = (int32_t)threadIdx.x, wave = tid / 64;
    const int64_t row = blockIdx.x;
    const raw* z = static_cast<const raw*>(a.in.z) + row * a.in.ld;
    const float w = a.weight ? a.weight[row] : 1.0f;
    Bitmap<T, kThreads> bitmap;
    Slots slots;
    lds_layout(a, row_shape<T>(z, (int32_t)a.in.cols), lds, bitmap, slots);
    double t_lse = 0.0;
    bool alive = false;
    RunningSum r = RunningSum::none();  // of lane s: part s
    if (w != 0.0f) {
        const int32_t c0 = slot_column(a, row, tid);
        if (a.t_lse) t_lse = (double)a.t_lse[row];
        if ((tid & 63) < a.splits) {
            const float2 p = a.part[row * a.splits + (tid & 63)];
            r = RunningSum{p.x, p.y};
        }
        bitmap.clear();
        alive = read_slots<T, kThreads>(a, row, z, 0, (int32_t)a.in.cols, c0, bitmap, slots);
    }
    if (!alive) {
        if (tid == 0) write_no_row(a, row);
        return;
    }
    const WaveSums ws = entry_sums<kThreads, true>(a, t_lse, slots);
    if ((tid & 63) == 0) wrec[wave] = ws;
    __syncthreads();
    if (wave == 0) {
        wave_join(r);
        const RowResult res = finish_row<kNW>(a, r, wrec[tid & (kNW - 1)]);
        if (tid == 0) write_row(a, row, w, res);
    }
}

template <class T, int kThreads>
static size_t lds_bytes(const DistillArgs& a) {
    return (size_t)(Bitmap<T, kThreads>::bytes((int32_t)row_granules(a.in.dtype, a.in.cols)) + slot_bytes(a.k));
}
static dim3 parts(const DistillArgs& a) { return dim3((uint32_t)(a.in.rows * a.splits)); }

template <class T>
static hipError_t backward_typed(hipStream_t s, const DistillArgs& a) {
    hipLaunchKernelGGL((k_distill_grad<T>), parts(a), dim3(kStreamThreads), (lds_bytes<T, kStreamThreads>(a)), s, a);
    return hipGetLastError();
}

template <class T, int kThreads, int kGran>
static void fused(hipStream_t s, const DistillArgs& a) {
    hipLaunchKernelGGL((k_distill_fused<T, kThreads, kGran>), parts(a), dim3(kThreads), (lds_bytes<T, kThreads>(a)), s,
                       a);
}

template <class T>
static hipError_t forward_typed(hipStream_t s, const DistillArgs& a) {
    const size_t lds = lds_bytes<T, kStreamThreads>(a);
    if (a.splits > 1) {
        hipLaunchKernelGGL((k_distill_loss<T, true>), parts(a), dim3(kStreamThreads), lds, s, a);
        hipLaunchKernelGGL((k_distill_join<T>), dim3((uint32_t)a.in.rows), dim3(kStreamThreads), lds, s, a);
    } else if (a.dz && a.per <= kRowCapacity) {
        if (a.per <= 256 * 4) fused<T, 256, 4>(s, a);
        else if (a.per <= 256 * 8) fused<T, 256, 8>(s, a);
        else if (a.per <= 256 * 16) fused<T, 256, 16>(s, a);
        else fused<T, 512, 16>(s, a);
        return hipGetLastError();
    } else {
        hipLaunchKernelGGL((k_distill_loss<T, false>), parts(a), dim3(kStreamThreads), lds, s, a);
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
