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
// The logits are read once.
// The entries' columns are marked in an LDS bitmap and struck out of the
// granules as they go by (-inf), so that the running sum is the tail's own,
// never a difference of two large ones.  The entries' terms are summed in 64
// bits.
//  - k_distill_loss: streams a row, or a part of one, through a workgroup.
//  - k_distill_fused: loss and gradient; the row stays in the registers of
//    its workgroup, so it is read once for both.
//  - k_distill_join: joins the parts of a row where few rows are split.
//  - k_distill_grad: streams the gradient of a row, or a part of one, from the
//    statistics.
// What bounds them is the read of the logits and the write of the gradient:
//   loss, 2048x50257 f16               44 us, 4.6 TB/s (a plain read 30 us)
//   loss, 7x50304 bf16                 11 us: a row's chain of latencies
//   loss and gradient, 4096x32000 bf16 101 us, 5.2 TB/s read and written (a
//                                      copy 79 us)
//   the same, 1024x50304 f32           117 us: rows past 8192 granules are read
//                                      for the loss and again for the gradient
//   gradient, 1024x50304 f32           82 us, 5.0 TB/s (a copy 62 us)
// A reading kernel keeps 6 waves a SIMD and eight granules a thread in flight;
// of the gradient's excess over a copy 3 to 5 us are the entries' columns,
// which are partial writes over lines that have left.
//
// Statistics kept for a later backward pass: L = log sum exp(s z) and
// log p_T.  The latter is near 0 where the entries hold little of the
// student's mass, and the gradient's tail factor (Q - q_T / p_T) p_T =
// sum q_j p_T + q_T (p_T - 1) is then made of two small terms.  Where the
// student holds almost nothing outside the entries, the tail is summed again.
#include <type_traits>

#include "loss_device.h"

namespace scape {

// LDS of a workgroup: a bitmap of the row's columns, then the k slots: col
// (-1: no entry), t (the teacher's value, then q), z (the student's logit,
// then p).
//
// The bitmap lies as a thread's granules do, four of them (tid, tid + threads,
// ...) in one cell: whether its next four granules hold an entry is one read
// and one test.  Some lane of a wave nearly always has one, so what counts is
// the striking: of 16-bit types a cell's low half has the bits of the even
// elements and its high half those of the odd ones, so that two packed shifts
// make the mask of two elements (1.5 instructions an element; testing bit by
// bit took 5.6, as much as all the rest).  The elements beside the granules
// have 16 bits of their own behind the cells.
template <class T, int kThreads>
struct Lds {
    using Cell = std::conditional_t<T::kN == 8, uint32_t, uint16_t>;
    static constexpr int kCellBits = 4 * T::kN, kCellGranules = 4 * kThreads;
    Cell* cells;
    int32_t* col;
    float* t;
    float* z;
    RowShape sh;
    int32_t n, k;

    static __host__ __device__ int32_t cell_count(int32_t granules) {
        return (granules + kCellGranules - 1) / kCellGranules * kThreads;
    }
    static __host__ __device__ int32_t cell_bytes(int32_t granules) {
        return cell_count(granules) * (int32_t)sizeof(Cell) + 4;
    }
    static int32_t bytes(int32_t granules, int32_t k) { return cell_bytes(granules) + 12 * k; }
    __device__ __forceinline__ Lds(uint8_t* at, const RowShape& shape, int32_t cols, int32_t slots) {
        sh = shape;
        n = cols;
        k = slots;
        col = reinterpret_cast<int32_t*>(at);
        t = reinterpret_cast<float*>(col + k);
        z = t + k;
        cells = reinterpret_cast<Cell*>(z + k);
    }
    __device__ __forceinline__ uint32_t* words() const { return reinterpret_cast<uint32_t*>(cells); }
    __device__ __forceinline__ void clear() const {
        const int32_t m = cell_bytes(sh.granules) / 4;
        for (int32_t i = (int32_t)threadIdx.x; i < m; i += kThreads) words()[i] = 0;
    }
    __device__ __forceinline__ uint32_t bit_of(int32_t c) const {
        const int32_t e = c - sh.head, i = e / T::kN, j = e % T::kN;
        if (e >= 0 && i < sh.granules) {
            const int32_t cell = i / kCellGranules * kThreads + i % kThreads, b = i / kThreads & 3;
            return (uint32_t)(cell * kCellBits + (T::kN == 8 ? b * 4 + j / 2 + 16 * (j & 1) : b * 4 + j));
        }
        return (uint32_t)(cell_count(sh.granules) * kCellBits + (e < 0 ? c : 8 + c - (n - sh.tail)));
    }
    // Marks a column; whether it was marked before.
    __device__ __forceinline__ bool mark(int32_t c) const {
        const uint32_t at = bit_of(c), bit = 1u << (at & 31u);
        return (atomicOr(words() + (at >> 5), bit) & bit) != 0;
    }
    __device__ __forceinline__ bool marked(int32_t c) const {
        const uint32_t at = bit_of(c);
        return (words()[at >> 5] >> (at & 31u)) & 1u;
    }
    // Strikes the entries out of the thread's granules
    // tid + (b + 4 cell_row) kThreads, b < 4.
    __device__ __forceinline__ void strike(int32_t cell_row, gran (&g)[4]) const {
        const uint32_t bits = cells[cell_row * kThreads + (int32_t)threadIdx.x];
        uint32_t none = no_entries<T>()[0];
        asm("" : "+s"(none));  // in a register: one v_bfi_b32 a word, where a literal takes two instructions
        if (bits) {
#pragma unroll
            for (int b = 0; b < 4; ++b)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    uint32_t m;
                    if constexpr (T::kN == 8) {
                        typedef int16_t pair __attribute__((ext_vector_type(2)));
                        m = __builtin_bit_cast(uint32_t, (pair)(__builtin_bit_cast(pair, bits) << (int16_t)(15 - 4 * b - q)));
                        asm("" : "+v"(m));
                        m = __builtin_bit_cast(uint32_t, (pair)(__builtin_bit_cast(pair, m) >> (int16_t)15));
                    } else {
                        m = (uint32_t)((int32_t)(bits << (31 - 4 * b - q)) >> 31);
                    }
                    asm("" : "+v"(m));  // a mask: else each element becomes a test and a select
                    g[b][q] = (g[b][q] & ~m) | (none & m);
                }
        }
    }
};

// A slot's column and teacher's value as they are read; a column outside the
// row is no entry.
struct Slot {
    int32_t c;
    uint32_t t;  // bits
};
__device__ __forceinline__ Slot read_slot(const DistillArgs& a, int64_t row, int32_t slot) {
    const int64_t at = row * a.k + (slot < a.k ? slot : a.k - 1);
    Slot s{a.t_idx[at], load_bits(a.t_val, a.t_dtype, at)};
    if (slot >= a.k) s.c = -1;
    return s;
}

// Marks the row's entries; s0 is slot tid.  An entry whose column a lower slot
// has is dropped.  The bitmap has been cleared by this workgroup, s_flags too,
// without a barrier since; both are complete afterwards.  Returns whether the
// row has any entry.
template <class T, int kThreads>
__device__ __forceinline__ bool mark_entries(const DistillArgs& a, int64_t row, Slot s0, const Lds<T, kThreads>& lds,
                                             uint32_t* s_flags) {
    const int32_t tid = (int32_t)threadIdx.x;
    __syncthreads();
    uint32_t seen = 0;  // bit 0: some entry; bit 1: some column twice
    for (int32_t slot = tid; slot < a.k; slot += kThreads) {
        const Slot s = slot == tid ? s0 : read_slot(a, row, slot);
        const bool there = s.c >= 0 && s.c < lds.n;
        lds.col[slot] = there ? s.c : -1;
        lds.t[slot] = value_of(s.t, a.t_dtype);
        if (!there) continue;
        seen |= 1u;
        if (lds.mark(s.c)) seen |= 2u;
    }
    if (seen) atomicOr(s_flags, seen);
    __syncthreads();
    seen = *s_flags;
    if (seen & 2u) {
        // which of two threads came first is chance, so every entry looks for
        // its column in the slots below its own
        for (int32_t slot = tid; slot < a.k; slot += kThreads) {
            const int32_t c = lds.col[slot];
            for (int32_t j = 0; j < slot && c >= 0; ++j)
                if (a.t_idx[row * a.k + j] == c) {
                    lds.col[slot] = -1;
                    break;
                }
        }
    }
    return seen != 0;
}

// log q_j: s t_j minus the teacher's lse where it is given, else against mq.
__device__ __forceinline__ double log_q(const DistillArgs& a, double lse, float t, float mq) {
    if (t == kNegInf) return (double)t;
    return a.t_lse ? (double)t * (double)a.scale - lse : ((double)t - (double)mq) * (double)a.scale;
}

// A wave's entries summed, against the wave's own references; the row's are
// put together in finish_row.
struct WaveSums {
    double top;  // sum 2^(c2 (x_j - mt))
    double q;    // sum q_j, q_j = exp(lq_j), lq_j the teacher's log-probability (against mq)
    double qt;   // sum q_j lq_j
    double qx;   // sum q_j c2 (x_j - mt), entries at a column of -inf left out
    float mt;    // the largest x_j
    float mq;    // 0 where the teacher's lse is given, else the largest t_j
    float mi;    // the largest t_j with q_j > 0 at a column of -inf; -inf: none
};

// kStudent: also the student's terms.  Slots' t and z become q and p, for the
// gradient, in float32: each is rounded once more, a step of a float32
// gradient (the sums are over float64).
template <class T, int kThreads, bool kStudent>
__device__ __forceinline__ WaveSums entry_sums(const DistillArgs& a, double lse, const Lds<T, kThreads>& l) {
    const int32_t tid = (int32_t)threadIdx.x;
    WaveSums s{0.0, 0.0, 0.0, 0.0, kLowest, a.t_lse ? 0.0f : kLowest, kNegInf};
    bool some = false;
    for (int32_t slot = tid; slot < a.k; slot += kThreads)
        if (l.col[slot] >= 0) {
            some = true;
            if (kStudent) s.mt = fmaxf(s.mt, l.z[slot]);
            if (!a.t_lse) s.mq = fmaxf(s.mq, l.t[slot]);
        }
    if (wave_ballot(some) == 0) return s;
    if (kStudent) s.mt = group_reduce<OpMaxNum, 64>(s.mt);
    if (!a.t_lse) s.mq = group_reduce<OpMaxNum, 64>(s.mq);
    for (int32_t slot = tid; slot < a.k; slot += kThreads)
        if (l.col[slot] >= 0) {
            const float t = l.t[slot];
            const double lq = log_q(a, lse, t, s.mq), q = exp(lq);
            l.t[slot] = (float)q;
            s.q += q;
            if (kStudent) {
                const double x = ((double)l.z[slot] - (double)s.mt) * (double)a.c2, p = exp2(x);
                l.z[slot] = (float)p;
                s.top += p;
                if (q != 0.0) {
                    s.qt += q * lq;
                    if (x == -__builtin_inf())
                        s.mi = fmaxf(s.mi, t);
                    else
                        s.qx += q * x;
                }
            }
        }
    s.q = wave_sum_f64(s.q);
    if (kStudent) {
        s.top = wave_sum_f64(s.top);
        s.qt = wave_sum_f64(s.qt);
        s.qx = wave_sum_f64(s.qx);
        s.mi = group_reduce<OpMaxNum, 64>(s.mi);
    }
    return s;
}

// The row's loss, statistics and gradient factors.
struct RowResult {
    float loss;          // KL
    float stat0, stat1;  // L, log p_T
    float2 anchor;       // L = scale * x + y
    float vref, tail;    // the tail's gradient is tail 2^(c2 (x_v - vref))
    double p, q;         // an entry's gradient is p p_j - q q_j, for the entries of this lane's wave (lane % kWaves)
    bool dead;           // no student mass at all: nothing to learn
};

// A whole wave calls it; lane l brings the entries' sums of wave l % kWaves
// and the tail's running sum of the row.  The row's powers, its logarithms and
// its divisions are one each, on as many lanes.
template <int kWaves>
__device__ __forceinline__ RowResult finish_row(const DistillArgs& a, const RunningSum& tail, const WaveSums& w) {
    RowResult r;
    const uint32_t lane = lane_id();
    const double t = (double)tail.sum, tref = (double)tail.ref, c2 = (double)a.c2;
    const bool has_tail = !(t == 0.0);
    const double ref = fmax(has_tail ? tref : (double)kLowest, (double)group_reduce<OpMaxNum, kWaves>(w.mt));
    const double mq = (double)group_reduce<OpMaxNum, kWaves>(w.mq), mi = (double)group_reduce<OpMaxNum, kWaves>(w.mi);
    const double dq = a.t_lse ? 0.0 : ((double)w.mq - mq) * (double)a.scale;
    // lanes 0..: the waves' references against the row's; 16..: the teacher's
    // likewise; 32: the tail's (0 too where the tail is out of range); 48: the
    // entry of most mass at a column of -inf against the teacher's reference
    const double powers = exp2(lane < 16   ? ((double)w.mt - ref) * c2
                               : lane < 32 ? dq * kLog2e64
                               : lane < 48 ? (tref - ref) * c2
                                           : (mi - mq) * (double)a.scale * kLog2e64);
    const double fp = from_lane_of<kWaves>(powers, 0), fq = from_lane_of<kWaves>(powers, 16);
    const double far = has_tail ? from_lane(powers, 32) : 0.0;
    const double top = sum_waves_f64<kWaves>(w.top * fp);
    const double q = sum_waves_f64<kWaves>(w.q * fq);
    const double qt = sum_waves_f64<kWaves>((w.qt + (w.q != 0.0 ? w.q * dq : 0.0)) * fq);
    const double qx = sum_waves_f64<kWaves>((w.qx + (w.q != 0.0 ? w.q * (((double)w.mt - ref) * c2) : 0.0)) * fq);
    const double sum = t * far + top;
    double qsum, rest = 0.0;
    if (a.t_lse) {
        qsum = q;
        rest = has_tail && 1.0 - qsum > 0.0 ? 1.0 - qsum : 0.0;  // no tail: its term is left out
    } else {
        qsum = q == 0.0 ? 0.0 : 1.0;  // 0: every entry's value is -inf
    }
    const double of = lane == 0 ? sum : lane == 1 ? t : lane == 2 ? q : rest;
    const double logs = log(of), inverses = 1.0 / of;
    const double log_sum = from_lane(logs, 0), log_t = from_lane(logs, 1), log_q = from_lane(logs, 2),
                 log_rest = from_lane(logs, 3);
    const double inv = from_lane(inverses, 0);
    const double qnorm = qsum == 0.0 ? 0.0 : a.t_lse ? 1.0 : from_lane(inverses, 2);
    const double lpt = has_tail ? log_t + (tref - ref) * (c2 * kLn2) - log_sum : -__builtin_inf();
    const double lse = ref * (double)a.scale + log_sum;
    double kl = 0.0;
    if (qsum != 0.0) {
        kl = (qt - qx * kLn2) * qnorm + qsum * log_sum;  // against ref, which cancels
        if (!a.t_lse) kl -= log_q;
    }
    if (rest > 0.0) kl += rest * (log_rest - lpt);
    // mass where the student has none: judged by the entry's probability in the
    // row, as a wave whose entries are all faint has it too large against its own
    // reference.  With the teacher's lse the two are the same.
    if (a.t_lse ? mi > -__builtin_inf() : from_lane(powers, 48) > 0.0) kl += __builtin_inf();
    r.loss = (float)kl;
    r.stat0 = (float)lse;
    r.anchor = make_float2((float)ref, (float)log_sum);  // ref is a logit
    r.stat1 = (float)lpt;
    r.vref = tail.ref;
    // (Q - q_T / p_T) p_v with q_T / p_T = q_T + q_T top / (t far)
    r.tail = has_tail ? (float)(inv * (qsum * far - rest * top * from_lane(inverses, 1))) : 0.0f;
    r.p = fp * inv * (qsum + rest);
    r.q = fq * qnorm;
    r.dead = sum == 0.0;
    return r;
}

__device__ __forceinline__ void write_row(const DistillArgs& a, int64_t row, float w, const RowResult& r) {
    a.loss[row] = r.dead ? 0.0f : w * r.loss;
    a.stats[2 * row] = r.stat0;
    a.stats[2 * row + 1] = r.stat1;
    if (a.anchor) a.anchor[row] = r.anchor;
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
        take(a.per, sp == a.splits - 1);
    }
    // The whole row in the place of its first part.
    __device__ __forceinline__ void take_whole() { take(sh.granules, true); }
    __device__ __forceinline__ void take(int32_t per, bool last) {
        g0 = sp * per;
        cnt = max(min(per, sh.granules - g0), 0);
        first = sh.head + g0 * T::kN;
        body = cnt > 0 ? reinterpret_cast<const gran*>(z + sh.head) + g0 : &g_no_granule;
        lone = lone_element(sh, n, sp == 0, last);
        // a last part may begin past the granules: what is left is its lone columns
        col0 = sp == 0 ? 0 : min(first, sh.head + sh.granules * T::kN);
        col1 = last ? n : first + cnt * T::kN;
    }
    // Four granules of a thread, from number base + tid on; past the last one
    // the last one again (trim takes it out).  A load under a condition, were
    // it one that is always true, would cost the prefetch: the compiler then
    // cannot count the loads in flight and waits for all of them.
    template <int kThreads>
    __device__ __forceinline__ void load(int32_t base, gran (&g)[4]) const {
#pragma unroll
        for (int b = 0; b < 4; ++b)
            g[b] = granule_at(body, max(min(base + (int32_t)threadIdx.x + b * kThreads, cnt - 1), 0));
    }
    template <int kThreads>
    __device__ __forceinline__ void trim(int32_t base, gran (&g)[4]) const {
#pragma unroll
        for (int b = 0; b < 4; ++b)
            if (base + (int32_t)threadIdx.x + b * kThreads >= cnt) g[b] = no_entries<T>();
    }
    // The lone element, -inf if there is none, and an entry's logit, 0 outside
    // the part's columns: loads without a condition too (a part may have no
    // column of its own to read instead).
    __device__ __forceinline__ float element(int32_t c, bool there, float other) const {
        const float x = T::up1(*(there ? z + c : reinterpret_cast<const raw*>(&g_no_granule)));
        return there ? x : other;
    }
    __device__ __forceinline__ float lone_logit() const { return element(lone, lone >= 0, kNegInf); }
    __device__ __forceinline__ float entry_logit(int32_t c) const { return element(c, c >= col0 && c < col1, 0.0f); }
};

// Streams the part through two sets of four granules a thread: one is on its
// way while the other is worked on.  `first` is loaded already.  whole(base,
// x) takes granules base + tid + b threads that are all there, last(base, x)
// the ones of which some are past the end.
template <class T, int kThreads, class Whole, class Last>
__device__ __forceinline__ void stream_row(const Part<T>& p, gran (&first)[4], Whole whole, Last last) {
    constexpr int kStep = 4 * kThreads;
    gran second[4];
    int32_t base = 0;
    for (; base + 2 * kStep <= p.cnt; base += 2 * kStep) {
        p.template load<kThreads>(base + kStep, second);
        whole(base, first);
        p.template load<kThreads>(base + 2 * kStep, first);
        whole(base + kStep, second);
    }
    if (base + kStep <= p.cnt) {
        p.template load<kThreads>(base + kStep, second);
        whole(base, first);
        if (base + kStep < p.cnt) last(base + kStep, second);
    } else if (base < p.cnt) {
        last(base, first);
    }
}

// A row that is not read: zeros.
template <class T, int kThreads>
__device__ __forceinline__ void zero_part(const Part<T>& p, typename T::raw* dz) {
    for (int32_t i = (int32_t)threadIdx.x; i < p.cnt; i += kThreads)
        store_loose(dz + p.first, i, gran{0u, 0u, 0u, 0u});
    if (p.lone >= 0) dz[p.lone] = 0;
}

// The entries' logits: slot tid's comes in a register (it was asked for when
// its column was known, and is not waited for before the row has gone by), the
// others are read here.
template <class T, int kThreads>
__device__ __forceinline__ void take_logits(const DistillArgs& a, const Part<T>& p, float z0,
                                            const Lds<T, kThreads>& l) {
    for (int32_t slot = (int32_t)threadIdx.x; slot < a.k; slot += kThreads)
        l.z[slot] = slot == (int32_t)threadIdx.x ? z0 : p.entry_logit(l.col[slot]);
}

// kPart: only the part's running sum of the tail, for k_distill_join.
// Four granules a thread are worked on while the next four are on their way.
template <class T, bool kPart, int kThreads>
__global__ __launch_bounds__(kThreads, 6) void k_distill_loss(DistillArgs a) {
    constexpr int kNW = kThreads / 64, kStep = 4 * kThreads;
    extern __shared__ __align__(16) uint8_t lds_bytes[];
    __shared__ float2 wsum[kNW];
    __shared__ WaveSums wrec[kNW];
    __shared__ uint32_t s_flags;
    const int32_t tid = (int32_t)threadIdx.x, wave = tid / 64;
    const Part<T> p(a);
    const Lds<T, kThreads> l(lds_bytes, p.sh, p.n, a.k);
    const float w = a.weight ? a.weight[p.row] : 1.0f;
    const double t_lse = !kPart && a.t_lse ? (double)a.t_lse[p.row] : 0.0;
    const Slot s0 = read_slot(a, p.row, tid);
    gran g[4];
    p.template load<kThreads>(0, g);
    const float lx = p.lone_logit();
    const float z0 = kPart ? 0.0f : p.entry_logit(s0.c);
    if (tid == 0) s_flags = 0;
    l.clear();
    if (!mark_entries(a, p.row, s0, l, &s_flags) || w == 0.0f) {
        if (tid == 0) {
            if (kPart)
                a.part[p.row * a.splits + p.sp] = make_float2(0.0f, 0.0f);
            else
                write_no_row(a, p.row);
        }
        return;
    }
    RunningSum rs = RunningSum::none();
    if (p.lone >= 0 && !l.marked(p.lone)) rs.add1(lx, a.c2);
    auto take = [&](int32_t base, gran (&x)[4]) {
        l.strike((p.g0 + base) / kStep, x);
        float m = granule_max<T>(x[0]);
#pragma unroll
        for (int b = 1; b < 4; ++b) m = max_nan(m, granule_max<T>(x[b]));
        rs.template add<T, 4>(x, m, a.c2);
    };
    stream_row<T, kThreads>(p, g, take, [&](int32_t base, gran (&x)[4]) {
        p.template trim<kThreads>(base, x);
        take(base, x);
    });
    wave_join(rs, a.c2);
    if ((tid & 63) == 0) wsum[wave] = make_float2(rs.ref, rs.sum);
    if constexpr (!kPart) {
        take_logits<T, kThreads>(a, p, z0, l);
        const WaveSums ws = entry_sums<T, kThreads, true>(a, t_lse, l);
        if ((tid & 63) == 0) wrec[wave] = ws;
    }
    __syncthreads();
    if (wave == 0) {
        RunningSum r{wsum[tid & (kNW - 1)].x, wsum[tid & (kNW - 1)].y};
        join_waves<kNW>(r, a.c2);
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
__device__ __forceinline__ void write_entries(const DistillArgs& a, const Part<T>& p, const Lds<T, kThreads>& l,
                                              float gs, double fp, double fq, typename T::raw* dz) {
    for (int32_t slot = (int32_t)threadIdx.x; slot < a.k; slot += kThreads) {
        const int32_t c = l.col[slot];
        if (c < 0 || c < p.col0 || c >= p.col1) continue;
        const double d = (double)gs * (fp * (double)l.z[slot] - fq * (double)l.t[slot]);
        dz[c] = gs == 0.0f ? (typename T::raw)0 : T::down1((float)d);
    }
}

// Loss and gradient of whole rows, kGran granules a thread.
template <class T, int kThreads, int kGran>
__global__ __launch_bounds__(kThreads, 4) void k_distill_fused(DistillArgs a) {
    constexpr int kNW = kThreads / 64;
    extern __shared__ __align__(16) uint8_t lds_bytes[];
    __shared__ float2 wsum[kNW];
    __shared__ WaveSums wrec[kNW];
    __shared__ double s_p[kNW], s_q[kNW];
    __shared__ float s_vref, s_tail, s_gs;
    __shared__ uint32_t s_flags;
    using raw = typename T::raw;
    const int32_t tid = (int32_t)threadIdx.x, wave = tid / 64;
    const Part<T> p(a);
    const Lds<T, kThreads> l(lds_bytes, p.sh, p.n, a.k);
    raw* dz = static_cast<raw*>(a.dz) + p.row * a.ld_dz;
    const float w = a.weight ? a.weight[p.row] : 1.0f;
    const double t_lse = a.t_lse ? (double)a.t_lse[p.row] : 0.0;
    if (w == 0.0f) {
        if (tid == 0) write_no_row(a, p.row);
        zero_part<T, kThreads>(p, dz);
        return;
    }
    const Slot s0 = read_slot(a, p.row, tid);
    gran g[kGran / 4][4];
#pragma unroll
    for (int c = 0; c < kGran / 4; ++c) p.template load<kThreads>(c * 4 * kThreads, g[c]);
    const float lx = p.lone_logit();
    const float z0 = p.entry_logit(s0.c);
    if (tid == 0) s_flags = 0;
    l.clear();
    if (!mark_entries(a, p.row, s0, l, &s_flags)) {
        if (tid == 0) write_no_row(a, p.row);
        zero_part<T, kThreads>(p, dz);
        return;
    }
    RunningSum rs = RunningSum::none();
    if (p.lone >= 0 && !l.marked(p.lone)) rs.add1(lx, a.c2);
#pragma unroll
    for (int c = 0; c < kGran / 4; ++c)
        if (c * 4 * kThreads < p.cnt) {
            if ((c + 1) * 4 * kThreads > p.cnt) p.template trim<kThreads>(c * 4 * kThreads, g[c]);
            l.strike(c, g[c]);
            float m = granule_max<T>(g[c][0]);
#pragma unroll
            for (int b = 1; b < 4; ++b) m = max_nan(m, granule_max<T>(g[c][b]));
            rs.template add<T, 4>(g[c], m, a.c2);
        }
    wave_join(rs, a.c2);
    if ((tid & 63) == 0) wsum[wave] = make_float2(rs.ref, rs.sum);
    {
        take_logits<T, kThreads>(a, p, z0, l);
        const WaveSums ws = entry_sums<T, kThreads, true>(a, t_lse, l);
        if ((tid & 63) == 0) wrec[wave] = ws;
    }
    __syncthreads();
    if (wave == 0) {
        RunningSum r{wsum[tid & (kNW - 1)].x, wsum[tid & (kNW - 1)].y};
        join_waves<kNW>(r, a.c2);
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
            for (int j = 0; j < T::kN; ++j) d[j] = f * fast_exp2(less<T>(x, j, vref) * a.c2);
            store_loose(dz + p.first, i, T::down(d));
        }
    }
    if (p.lone >= 0) dz[p.lone] = T::down1(f * fast_exp2((lx - vref) * a.c2));
    __syncthreads();  // the entries' columns are written over what is there
    write_entries(a, p, l, s_gs, s_p[wave], s_q[wave], dz);
}

// The gradient of a row or a part of one, from the statistics.  A tail of less
// than exp(-30) of the student's mass is a faint one: log p_T has too few bits
// for it (a step of float32 is 64 where the other columns are masked with -1e9),
// so its sum is made again, against its own largest logit.  The row's first
// part then takes the whole row and the other parts leave: dz may lie over z.
// (1024x50304 f32, every row a faint one: 138 us instead of 82; 64x131072 bf16
// 40 instead of 14.)
constexpr float kFaint = -30.0f;
template <class T>
__global__ __launch_bounds__(kRowThreads, 6) void k_distill_grad(DistillArgs a) {
    constexpr int kThreads = kRowThreads, kNW = kThreads / 64;
    extern __shared__ __align__(16) uint8_t lds_bytes[];
    __shared__ float2 wsum[kNW];
    __shared__ WaveSums wrec[kNW];
    __shared__ double s_p, s_q[kNW];
    __shared__ float s_xref, s_vref, s_tail, s_gs;
    __shared__ uint32_t s_flags;
    using raw = typename T::raw;
    const int32_t tid = (int32_t)threadIdx.x, wave = tid / 64;
    Part<T> p(a);
    const Lds<T, kThreads> l(lds_bytes, p.sh, p.n, a.k);
    raw* dz = static_cast<raw*>(a.dz) + p.row * a.ld_dz;
    float w = a.weight ? a.weight[p.row] : 1.0f;
    const float up = a.dloss ? a.dloss[p.row] : 1.0f;
    const double t_lse = a.t_lse ? (double)a.t_lse[p.row] : 0.0;
    const float lse = a.stats[2 * p.row], lpt = a.stats[2 * p.row + 1];
    const float2 at = a.anchor ? a.anchor[p.row] : make_float2(0.0f, lse);  // L = scale * at.x + at.y
    const Slot s0 = read_slot(a, p.row, tid);
    gran g[4];
    p.template load<kThreads>(0, g);
    // dz may be z, and other workgroups write their parts of it: only this
    // part's logits are read
    float lx = p.lone_logit();
    float z0 = p.entry_logit(s0.c);
    w = w == 0.0f ? 0.0f : w * up;
    if (tid == 0) s_flags = 0;
    l.clear();
    if (!mark_entries(a, p.row, s0, l, &s_flags) || w == 0.0f) {
        zero_part<T, kThreads>(p, dz);
        return;
    }
    const bool faint = a.t_lse && lpt <= kFaint;
    if (faint) {
        if (p.sp != 0) return;
        p.take_whole();
        lx = p.lone_logit();
        z0 = p.entry_logit(s0.c);
        RunningSum rs = RunningSum::none();
        if (p.lone >= 0 && !l.marked(p.lone)) rs.add1(lx, a.c2);
        // one set of granules, so that rows that are none keep their registers
        for (int32_t base = 0; base < p.cnt; base += 4 * kThreads) {
            p.template load<kThreads>(base, g);
            p.template trim<kThreads>(base, g);
            l.strike(base / (4 * kThreads), g);
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const gran one[1] = {g[b]};
                rs.template add<T, 1>(one, granule_max<T>(g[b]), a.c2);
            }
        }
        wave_join(rs, a.c2);
        if ((tid & 63) == 0) wsum[wave] = make_float2(rs.ref, rs.sum);
        p.template load<kThreads>(0, g);
    }
    // before any other thread may write over z
    for (int32_t slot = tid + kThreads; slot < a.k; slot += kThreads)
        l.z[slot] = p.entry_logit(l.col[slot]);
    {
        const WaveSums ws = entry_sums<T, kThreads, false>(a, t_lse, l);
        if ((tid & 63) == 0) wrec[wave] = ws;
    }
    __syncthreads();
    if (wave == 0) {
        const WaveSums r = wrec[tid & (kNW - 1)];
        const double fq = a.t_lse ? 1.0 : exp(((double)r.mq - (double)group_reduce<OpMaxNum, kNW>(r.mq)) * (double)a.scale);
        const double q = sum_waves_f64<kNW>(r.q * fq);
        const double qsum = a.t_lse ? q : q == 0.0 ? 0.0 : 1.0;
        RunningSum own{0.0f, 1.0f};
        if (faint) {
            own = RunningSum{wsum[tid & (kNW - 1)].x, wsum[tid & (kNW - 1)].y};
            join_waves<kNW>(own, a.c2);
        }
        const double rest = a.t_lse && 1.0 - q > 0.0 && own.sum != 0.0f ? 1.0 - q : 0.0;  // sum 0: no tail
        // (Q - q_T / p_T) p_v, against L, or a faint tail's against its own sum
        float xref = at.x, v = at.y, tail = (float)qsum;
        if (rest > 0.0) {
            const double pt = exp((double)lpt), c = qsum * pt + rest * (pt - 1.0);
            tail = (float)(c / (faint ? (double)own.sum : pt));
            if (faint) {
                xref = own.ref;
                v = 0.0f;
            }
        }
        if (tid < kNW) s_q[tid] = fq * (qsum == 0.0 ? 0.0 : a.t_lse ? 1.0 : 1.0 / q);
        if (tid == 0) {
            const float gs = lse == kNegInf ? 0.0f : w * a.scale;
            s_p = qsum + rest;
            s_gs = gs;
            s_tail = gs == 0.0f ? 0.0f : gs * tail;
            s_xref = xref;
            s_vref = gs == 0.0f ? -kNegInf : v;  // nothing to learn: exponents of -inf
        }
    }
    __syncthreads();
    const float f = s_tail, xref = s_xref, vref = s_vref;
    // the difference from L first: neither rounds L log2(e) nor leaves the range
    auto grad = [&](float x) { return f * fast_exp2(__builtin_fmaf(x - xref, a.scale, -vref) * kLog2e); };
    auto write = [&](int32_t i, const gran& x) {
        float d[T::kN];
#pragma unroll
        for (int j = 0; j < T::kN; ++j) d[j] = grad(T::up(x, j));
        store_loose(dz + p.first, i, T::down(d));
    };
    stream_row<T, kThreads>(
        p, g,
        [&](int32_t base, const gran (&x)[4]) {
#pragma unroll
            for (int b = 0; b < 4; ++b) write(base + tid + b * kThreads, x[b]);
        },
        [&](int32_t base, const gran (&x)[4]) {
#pragma unroll
            for (int b = 0; b < 4; ++b)
                if (base + tid + b * kThreads < p.cnt) write(base + tid + b * kThreads, x[b]);
        });
    if (p.lone >= 0) dz[p.lone] = T::down1(grad(lx));
    if (tid < a.k) l.z[tid] = z0;
    for (int32_t slot = tid; slot < a.k; slot += kThreads)
        l.z[slot] = (float)exp(((double)l.z[slot] - (double)at.x) * (double)a.scale - (double)at.y);
    __syncthreads();  // the entries' columns are written over the tail's values
    write_entries(a, p, l, s_gs, s_p, s_q[wave], dz);
}

// Joins the parts of a split row: the loss and the statistics.
template <class T>
__global__ __launch_bounds__(kRowThreads) void k_distill_join(DistillArgs a) {
    constexpr int kThreads = kRowThreads, kNW = kThreads / 64;
    extern __shared__ __align__(16) uint8_t lds_bytes[];
    __shared__ WaveSums wrec[kNW];
    __shared__ uint32_t s_flags;
    const int32_t tid = (int32_t)threadIdx.x, wave = tid / 64, n = (int32_t)a.in.cols;
    const int64_t row = blockIdx.x;
    const typename T::raw* z = static_cast<const typename T::raw*>(a.in.z) + row * a.in.ld;
    const Lds<T, kThreads> l(lds_bytes, row_shape<T>(z, n), n, a.k);
    const float w = a.weight ? a.weight[row] : 1.0f;
    const double t_lse = a.t_lse ? (double)a.t_lse[row] : 0.0;
    const Slot s0 = read_slot(a, row, tid);
    RunningSum r = RunningSum::none();  // of lane s: part s
    if ((tid & 63) < a.splits) {
        const float2 p = a.part[row * a.splits + (tid & 63)];
        r = RunningSum{p.x, p.y};
    }
    if (tid == 0) s_flags = 0;
    l.clear();
    if (!mark_entries(a, row, s0, l, &s_flags) || w == 0.0f) {
        if (tid == 0) write_no_row(a, row);
        return;
    }
    for (int32_t slot = tid; slot < a.k; slot += kThreads)
        if (l.col[slot] >= 0) l.z[slot] = T::up1(z[l.col[slot]]);
    const WaveSums ws = entry_sums<T, kThreads, true>(a, t_lse, l);
    if ((tid & 63) == 0) wrec[wave] = ws;
    __syncthreads();
    if (wave == 0) {
        wave_join(r, a.c2);
        const RowResult res = finish_row<kNW>(a, r, wrec[tid & (kNW - 1)]);
        if (tid == 0) write_row(a, row, w, res);
    }
}

// At most 34 KB of bitmap (2^18 columns) and 12 KB of slots (k = 1024).
template <class T, int kThreads>
static size_t lds_size(const DistillArgs& a) {
    return (size_t)Lds<T, kThreads>::bytes((int32_t)row_granules(a.in.dtype, a.in.cols), a.k);
}
static dim3 parts(const DistillArgs& a) { return dim3((uint32_t)(a.in.rows * a.splits)); }

template <class T>
static hipError_t backward_typed(hipStream_t s, const DistillArgs& a) {
    DistillArgs b = a;
    b.splits = a.grad_splits;
    b.per = a.grad_per;
    hipLaunchKernelGGL((k_distill_grad<T>), parts(b), dim3(kRowThreads), (lds_size<T, kRowThreads>(b)), s, b);
    return hipGetLastError();
}

template <class T, int kThreads, int kGran>
static void fused(hipStream_t s, const DistillArgs& a) {
    hipLaunchKernelGGL((k_distill_fused<T, kThreads, kGran>), parts(a), dim3(kThreads), (lds_size<T, kThreads>(a)), s,
                       a);
}

template <class T>
static hipError_t forward_typed(hipStream_t s, const DistillArgs& a) {
    const size_t lds = lds_size<T, kRowThreads>(a);
    if (a.splits > 1) {
        hipLaunchKernelGGL((k_distill_loss<T, true, kRowThreads>), parts(a), dim3(kRowThreads), lds, s, a);
        hipLaunchKernelGGL((k_distill_join<T>), dim3((uint32_t)a.in.rows), dim3(kRowThreads), lds, s, a);
    } else if (a.dz && a.per <= kFusedCapacity) {
        if (a.per <= 256 * 4) fused<T, 256, 4>(s, a);
        else if (a.per <= 256 * 8) fused<T, 256, 8>(s, a);
        else if (a.per <= 256 * 16) fused<T, 256, 16>(s, a);
        else fused<T, 512, 16>(s, a);
        return hipGetLastError();
    } else if (a.per <= kTopkCapacity || a.in.rows > 512) {
        hipLaunchKernelGGL((k_distill_loss<T, false, 256>), parts(a), dim3(256), lds, s, a);
    } else {  // few long rows (7x131072 bf16 19 us instead of 21, replayed; 2048x50257 f16 would take 49 instead of 44)
        hipLaunchKernelGGL((k_distill_loss<T, false, 512>), parts(a), dim3(512), (lds_size<T, 512>(a)), s, a);
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
