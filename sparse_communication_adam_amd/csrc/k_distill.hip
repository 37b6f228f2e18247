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
// One workgroup takes a row, or a part of one, into registers and reads the
// logits once: the entries' columns are marked in an LDS bitmap and struck
// out of the registers (-inf), so the sums that follow are the tail's own,
// never a difference of two large ones; the k entries are gathered and their
// terms summed in 64 bits.  The gradient is then made from the same
// registers.  What bounds it is the read of the logits and the write of the
// gradient.
//
// Statistics kept for a later backward pass: L = log sum exp(s z) and
// log p_T.  The latter is near 0 where the entries hold little of the
// student's mass, and the gradient's tail factor (Q - q_T / p_T) p_T =
// sum q_j p_T + q_T (p_T - 1) is then made of two small terms.
#include "loss_device.h"

namespace scape {

// What a launch of k_distill_row does.
enum DistillMode : int {
    kLoss = 0,      // loss and statistics of whole rows
    kLossGrad = 1,  // those and the gradient
    kPart = 2,      // a part's tail sum, for k_distill_join
    kGrad = 3,      // the gradient of a row or part, from the statistics
};

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
    // kept for the gradient in float32 (its own sums are over float64): each
    // is rounded once more, a step of a float32 gradient
    float q[kEntries];  // exp of the teacher's log-probability, not normalised where the teacher's lse is not given
    float p[kEntries];  // 2^(x_j - ref)
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

struct RowSums {  // over the row's entries
    double top;   // sum 2^(x_j - ref), x_j = z_j c2
    double q;     // sum q_j (not normalised where the teacher's lse is not given)
    double qt;    // sum q_j log q_j (likewise)
    double qx;    // sum q_j x_j
};

// The entries' terms, against ref and, where the teacher's lse is not given,
// tmax.  en.q and en.p are set.
__device__ __forceinline__ RowSums entry_sums(const DistillArgs& a, double lse, double tmax, double ref, Entries& en) {
    RowSums s{0.0, 0.0, 0.0, 0.0};
#pragma unroll
    for (int i = 0; i < kEntries; ++i) {
        en.q[i] = en.p[i] = 0.0f;
        if (en.col[i] >= 0) {
            const double x = (double)en.z[i] * (double)a.c2, lq = log_q(a, lse, en.t[i]) - tmax, q = exp(lq);
            const double p = exp2(x - ref);
            en.q[i] = (float)q;
            en.p[i] = (float)p;
            s.top += p;
            if (q != 0.0) {
                s.q += q;
                s.qt += q * lq;
                s.qx += q * x;
            }
        }
    }
    if (wave_ballot(s.top != 0.0 || s.q != 0.0) != 0) {
        s.top = wave_sum_f64(s.top);
        s.q = wave_sum_f64(s.q);
        s.qt = wave_sum_f64(s.qt);
        s.qx = wave_sum_f64(s.qx);
    }
    return s;
}

// The row's loss, statistics and gradient factors from the tail's sum
// t = sum 2^(x - tref) and the entries' sums, against ref.  A whole wave
// calls it with the same arguments: the four logarithms are one, on four
// lanes.
struct RowResult {
    float loss;          // KL
    float stat0, stat1;  // L, log p_T
    float tail;          // the tail's gradient is tail 2^(x_v - tref)
    double inv;          // 1 / sum 2^(x - ref): p_v = inv 2^(x_v - ref)
    double whole;        // Q
    double qnorm;        // q_j = qnorm en.q
    bool dead;           // no student mass at all: nothing to learn
};
__device__ __forceinline__ RowResult finish_row(const DistillArgs& a, double ref, double tref, double t,
                                                const RowSums& s) {
    RowResult r;
    const bool has_tail = !(t == 0.0);
    const double far = has_tail ? exp2(tref - ref) : 0.0;  // 0 too where the tail is out of range
    const double sum = t * far + s.top;
    double qsum, rest = 0.0;
    if (a.t_lse) {
        qsum = s.q;
        rest = has_tail && 1.0 - qsum > 0.0 ? 1.0 - qsum : 0.0;  // no tail: its term is left out
    } else {
        qsum = s.q == 0.0 ? 0.0 : 1.0;  // 0: every entry's value is -inf
    }
    const uint32_t lane = lane_id();
    const double logs = log(lane == 0 ? sum : lane == 1 ? t : lane == 2 ? s.q : rest);
    const double log_sum = from_lane(logs, 0), log_t = from_lane(logs, 1), log_s = from_lane(logs, 2),
                 log_rest = from_lane(logs, 3);
    r.qnorm = a.t_lse ? 1.0 : qsum / s.q;
    if (qsum == 0.0) r.qnorm = 0.0;
    const double lpt = has_tail ? log_t + (tref - ref) * kLn2 - log_sum : -__builtin_inf();
    const double lse = ref * kLn2 + log_sum;
    double kl = 0.0;
    if (qsum != 0.0) {
        kl = (s.qt - s.qx * kLn2) * r.qnorm + qsum * lse;
        if (!a.t_lse) kl -= qsum * log_s;  // q_j = exp(lq_j) / sum
    }
    if (rest > 0.0) kl += rest * (log_rest - lpt);
    r.whole = qsum + rest;
    r.loss = (float)kl;
    r.stat0 = (float)lse;
    r.stat1 = (float)lpt;
    r.inv = 1.0 / sum;
    // (Q - q_T / p_T) p_v with q_T / p_T = q_T + q_T top / tail
    r.tail = has_tail ? (float)(r.inv * (qsum * far - rest * s.top / t)) : 0.0f;
    r.dead = sum == 0.0;
    return r;
}

template <class T, int kGran, int kMode>
__global__ __launch_bounds__(kRowThreads, row_waves(kGran)) void k_distill_row(DistillArgs a) {
    extern __shared__ uint32_t bitmap[];
    __shared__ float wmax[3][kRowWaves];
    __shared__ float wsum[kRowWaves];
    __shared__ double wd[4][kRowWaves];
    __shared__ RowResult s_res;
    __shared__ float s_vref;
    using raw = typename T::raw;
    const int32_t tid = (int32_t)threadIdx.x, wave = tid / 64;
    const int64_t row = blockIdx.x / (uint32_t)a.splits;
    const int32_t sp = (int32_t)(blockIdx.x % (uint32_t)a.splits);
    const raw* z = static_cast<const raw*>(a.in.z) + row * a.in.ld;
    const int32_t n = (int32_t)a.in.cols;
    const RowShape sh = row_shape<T>(z, n);
    const int32_t g0 = sp * a.per;
    const int32_t cnt = max(min(a.per, sh.granules - g0), 0);
    const bool last = sp == a.splits - 1;
    const gran* body = reinterpret_cast<const gran*>(z + sh.head) + g0;
    const int32_t first = sh.head + g0 * T::kN;  // column of granule 0's first element
    const int32_t lone = lone_element(sh, n, sp == 0, last);
    // the columns of this part
    const int32_t col0 = sp == 0 ? 0 : first, col1 = last ? n : first + cnt * T::kN;
    raw* dz = nullptr;
    if constexpr (kMode == kLossGrad || kMode == kGrad) dz = static_cast<raw*>(a.dz) + row * a.ld_dz;

    float w = a.weight ? a.weight[row] : 1.0f;
    if (kMode == kGrad && a.dloss) w = w == 0.0f ? 0.0f : w * a.dloss[row];
    gran g[kGran];
    float lx = kNegInf;
    Entries en;
    double t_lse = 0.0;
    bool alive = false;
    if (w != 0.0f) {
        read_columns(a, row, en);
#pragma unroll
        for (int c = 0; c < kGran; ++c) {
            const int32_t i = tid + c * kRowThreads;
            g[c] = no_entries<T>();
            if (i < cnt) g[c] = body[i];
        }
        if (lone >= 0) lx = T::up1(z[lone]);
        // the gradient may overwrite the logits, part by part: only this
        // part's are read
        read_values<T>(a, row, z, kMode == kGrad ? col0 : 0, kMode == kPart ? 0 : kMode == kGrad ? col1 : n, en);
        if (a.t_lse) t_lse = (double)a.t_lse[row];
        const uint32_t words = (uint32_t)(n + 8 + 31) / 32u;
        for (uint32_t i = (uint32_t)tid; i < words; i += kRowThreads) bitmap[i] = 0;
        __syncthreads();
        alive = mark_columns(a, row, sh.head, bitmap, en);
    }
    if (!alive) {  // the same for the whole workgroup
        if constexpr (kMode == kLoss || kMode == kLossGrad)
            if (tid == 0) {
                a.loss[row] = 0.0f;
                a.stats[2 * row] = 0.0f;
                a.stats[2 * row + 1] = 0.0f;
            }
        if constexpr (kMode == kPart)
            if (tid == 0) a.part[row * a.splits + sp] = make_float2(0.0f, 0.0f);
        if constexpr (kMode == kLossGrad || kMode == kGrad) {
            for (int32_t i = tid; i < cnt; i += kRowThreads) store_loose(dz + first + i * T::kN, gran{0u, 0u, 0u, 0u});
            if (lone >= 0) dz[lone] = 0;
        }
        return;
    }

    float vref = 0.0f, tail = 0.0f;  // the tail's gradient: tail 2^(x - vref)
    double ref = 0.0, inv = 0.0, whole = 0.0, qnorm = 0.0;
    if constexpr (kMode != kGrad) {
        // strike the entries out; maxima of the tail, the entries and the teacher
        if (lone >= 0) {
            const uint32_t at = (uint32_t)(lone + 8 - sh.head);
            if (bitmap[at >> 5] & (1u << (at & 31u))) lx = kNegInf;
        }
        float m = lx, mt = kNegInf, mq = kNegInf;
        const int32_t tid1 = again(tid);
#pragma unroll
        for (int c = 0; c < kGran; ++c) {
            const int32_t i = tid1 + c * kRowThreads;
            const uint32_t b = i < cnt ? granule_bits<T>(bitmap, g0 + i) : 0u;
            if (b) {
#pragma unroll
                for (int j = 0; j < T::kN; ++j)
                    if (b & (1u << j)) T::set(g[c], j, (raw)T::kNegInfBits);
            }
            m = max_nan(m, granule_max<T>(g[c]));
        }
        m = group_reduce<OpMaxF, 64>(m);
        if constexpr (kMode != kPart) {
#pragma unroll
            for (int i = 0; i < kEntries; ++i)
                if (en.col[i] >= 0) {
                    mt = max_nan(mt, en.z[i]);
                    mq = max_nan(mq, (float)log_q(a, t_lse, en.t[i]));
                }
            mt = group_reduce<OpMaxF, 64>(mt);
            mq = group_reduce<OpMaxF, 64>(mq);
        }
        if ((tid & 63) == 0) {
            wmax[0][wave] = m;
            wmax[1][wave] = mt;
            wmax[2][wave] = mq;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kRowWaves; ++i) {
            m = max_nan(m, wmax[0][i]);
            mt = max_nan(mt, wmax[1][i]);
            mq = max_nan(mq, wmax[2][i]);
        }
        // The tail is summed against its own maximum: it may lie far below
        // the entries.  (Two chains, for the adders.)
        vref = m == kNegInf ? 0.0f : m * a.c2;
        float sum = fast_exp2(__builtin_fmaf(lx, a.c2, -vref)), sum1 = 0.0f;
#pragma unroll
        for (int c = 0; c < kGran; ++c)
            if (c * kRowThreads < cnt) {
                forget_unpacked(g[c]);
#pragma unroll
                for (int j = 0; j < T::kN; j += 2) {
                    sum += fast_exp2(__builtin_fmaf(T::up(g[c], j), a.c2, -vref));
                    sum1 += fast_exp2(__builtin_fmaf(T::up(g[c], j + 1), a.c2, -vref));
                }
            }
        sum = group_reduce<OpSumF, 64>(sum + sum1);
        if ((tid & 63) == 0) wsum[wave] = sum;
        if constexpr (kMode == kPart) {
            __syncthreads();
            if (tid == 0) {
                float t = wsum[0];
                for (int i = 1; i < kRowWaves; ++i) t += wsum[i];
                a.part[row * a.splits + sp] = make_float2(vref, t);
            }
            return;
        } else {
            const float both = max_nan(m, mt);
            ref = both == kNegInf ? 0.0 : (double)(both * a.c2);
            const RowSums s = entry_sums(a, t_lse, a.t_lse || mq == kNegInf ? 0.0 : (double)mq, ref, en);
            if ((tid & 63) == 0) {
                wd[0][wave] = s.top;
                wd[1][wave] = s.q;
                wd[2][wave] = s.qt;
                wd[3][wave] = s.qx;
            }
            __syncthreads();
            if (wave == 0) {
                const int32_t v = tid & 7;
                const double t = sum8_f64((double)wsum[v]);
                const RowSums r{sum8_f64(wd[0][v]), sum8_f64(wd[1][v]), sum8_f64(wd[2][v]), sum8_f64(wd[3][v])};
                const RowResult res = finish_row(a, ref, (double)vref, t, r);
                if (tid == 0) {
                    a.loss[row] = res.dead ? 0.0f : w * res.loss;
                    a.stats[2 * row] = res.stat0;
                    a.stats[2 * row + 1] = res.stat1;
                    s_res = res;
                }
            }
            if constexpr (kMode == kLoss) return;
            __syncthreads();
            if (s_res.dead) w = 0.0f;
            inv = s_res.inv;
            tail = s_res.tail;
            whole = s_res.whole;
            qnorm = s_res.qnorm;
        }
    } else {
        // the teacher's sum, as in the forward pass
        double tmax = 0.0;
        if (!a.t_lse) {
            float mq = kNegInf;
#pragma unroll
            for (int i = 0; i < kEntries; ++i)
                if (en.col[i] >= 0) mq = max_nan(mq, (float)log_q(a, t_lse, en.t[i]));
            mq = group_reduce<OpMaxF, 64>(mq);
            if ((tid & 63) == 0) wmax[0][wave] = mq;
            __syncthreads();
#pragma unroll
            for (int i = 0; i < kRowWaves; ++i) mq = max_nan(mq, wmax[0][i]);
            if (mq != kNegInf) tmax = (double)mq;
        }
        double q = 0.0;
#pragma unroll
        for (int i = 0; i < kEntries; ++i) {
            const double x = en.col[i] >= 0 ? exp(log_q(a, t_lse, en.t[i]) - tmax) : 0.0;
            en.q[i] = (float)x;
            q += x;
        }
        if (wave_ballot(q != 0.0) != 0) q = wave_sum_f64(q);
        if ((tid & 63) == 0) wd[0][wave] = q;
        __syncthreads();
        if (wave == 0) {
            const float l = a.stats[2 * row], lpt = a.stats[2 * row + 1];
            q = sum8_f64(wd[0][tid & 7]);
            RowResult r{};
            r.qnorm = a.t_lse ? 1.0 : q == 0.0 ? 0.0 : 1.0 / q;
            const double qsum = a.t_lse ? q : q == 0.0 ? 0.0 : 1.0;
            const double rest = a.t_lse && 1.0 - q > 0.0 && lpt != kNegInf ? 1.0 - q : 0.0;
            r.whole = qsum + rest;
            // (Q - q_T / p_T) p_v, against L, or where 1 / p_T could leave the
            // range against the tail's own log-sum-exp
            r.stat0 = l;
            float v = l;
            if (rest == 0.0) {
                r.tail = (float)qsum;
            } else {
                const double pt = exp((double)lpt), c = qsum * pt + rest * (pt - 1.0);
                const bool near = lpt > -30.0f;
                r.tail = (float)(near ? c / pt : c);
                if (!near) v = (float)((double)l + (double)lpt);
            }
            r.dead = l == kNegInf;
            if (tid == 0) {
                s_res = r;
                s_vref = v;
            }
        }
        __syncthreads();
        if (s_res.dead) w = 0.0f;
        ref = (double)s_res.stat0;
        tail = s_res.tail;
        whole = s_res.whole;
        qnorm = s_res.qnorm;
        vref = s_vref;
    }

    if constexpr (kMode == kLossGrad || kMode == kGrad) {
        const float gs = w * a.scale;
        const float f = gs == 0.0f ? 0.0f : gs * tail;
        if (gs == 0.0f) vref = -kNegInf;  // the whole row is -inf, or its factor vanishes: exponents of -inf
        // From the statistics, float32 gradients take the difference first:
        // they would see the rounding of L log2(e).
        auto grad = [&](float x) {
            float e;
            if constexpr (kMode == kLossGrad)
                e = __builtin_fmaf(x, a.c2, -vref);
            else
                e = __builtin_fmaf(x, a.scale, -vref) * kLog2e;
            return f * fast_exp2(e);
        };
        if (lone >= 0) dz[lone] = T::down1(grad(lx));
        const int32_t tid2 = again(tid);
#pragma unroll
        for (int c = 0; c < kGran; ++c) {
            const int32_t i = tid2 + c * kRowThreads;
            forget_unpacked(g[c]);
            if (i < cnt) {
                float d[T::kN];
#pragma unroll
                for (int j = 0; j < T::kN; ++j) d[j] = grad(T::up(g[c], j));
                store_loose(dz + first + i * T::kN, T::down(d));
            }
        }
        __syncthreads();  // the entries' columns are written over the tail's values
#pragma unroll
        for (int i = 0; i < kEntries; ++i)
            if (en.col[i] >= col0 && en.col[i] < col1) {
                double p;
                if constexpr (kMode == kLossGrad)
                    p = (double)en.p[i] * inv;
                else
                    p = exp((double)en.z[i] * (double)a.scale - ref);
                dz[en.col[i]] = gs == 0.0f ? (raw)0 : T::down1((float)((double)gs * (p * whole - (double)en.q[i] * qnorm)));
            }
    }
}

// Joins the parts of a split row: the loss and the statistics.
template <class T>
__global__ __launch_bounds__(kRowThreads) void k_distill_join(DistillArgs a) {
    extern __shared__ uint32_t bitmap[];
    __shared__ float wmax[2][kRowWaves];
    __shared__ double wd[4][kRowWaves];
    using raw = typename T::raw;
    const int32_t tid = (int32_t)threadIdx.x, wave = tid / 64;
    const int64_t row = blockIdx.x;
    const raw* z = static_cast<const raw*>(a.in.z) + row * a.in.ld;
    const float w = a.weight ? a.weight[row] : 1.0f;
    Entries en;
    double t_lse = 0.0;
    bool alive = false;
    float2 part = make_float2(0.0f, 0.0f);  // of lane s: part s
    if (w != 0.0f) {
        read_columns(a, row, en);
        read_values<T>(a, row, z, 0, (int32_t)a.in.cols, en);
        if (a.t_lse) t_lse = (double)a.t_lse[row];
        const uint32_t words = (uint32_t)(a.in.cols + 8 + 31) / 32u;
        for (uint32_t i = (uint32_t)tid; i < words; i += kRowThreads) bitmap[i] = 0;
        if ((tid & 63) < a.splits) part = a.part[row * a.splits + (tid & 63)];
        __syncthreads();
        alive = mark_columns(a, row, 0, bitmap, en);
    }
    if (!alive) {
        if (tid == 0) {
            a.loss[row] = 0.0f;
            a.stats[2 * row] = 0.0f;
            a.stats[2 * row + 1] = 0.0f;
        }
        return;
    }
    float mt = kNegInf, mq = kNegInf;
#pragma unroll
    for (int i = 0; i < kEntries; ++i)
        if (en.col[i] >= 0) {
            mt = max_nan(mt, en.z[i]);
            mq = max_nan(mq, (float)log_q(a, t_lse, en.t[i]));
        }
    mt = group_reduce<OpMaxF, 64>(mt);
    mq = group_reduce<OpMaxF, 64>(mq);
    if ((tid & 63) == 0) {
        wmax[0][wave] = mt;
        wmax[1][wave] = mq;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kRowWaves; ++i) {
        mt = max_nan(mt, wmax[0][i]);
        mq = max_nan(mq, wmax[1][i]);
    }
    float tref = group_reduce<OpMaxF, 64>(part.y != 0.0f ? part.x : kNegInf);
    const float both = max_nan(tref, mt == kNegInf ? kNegInf : mt * a.c2);
    if (tref == kNegInf) tref = 0.0f;
    const double ref = both == kNegInf ? 0.0 : (double)both;
    const RowSums s = entry_sums(a, t_lse, a.t_lse || mq == kNegInf ? 0.0 : (double)mq, ref, en);
    if ((tid & 63) == 0) {
        wd[0][wave] = s.top;
        wd[1][wave] = s.q;
        wd[2][wave] = s.qt;
        wd[3][wave] = s.qx;
    }
    __syncthreads();
    if (wave == 0) {
        const int32_t v = tid & 7;
        const RowSums r{sum8_f64(wd[0][v]), sum8_f64(wd[1][v]), sum8_f64(wd[2][v]), sum8_f64(wd[3][v])};
        const double t = wave_sum_f64(part.y != 0.0f ? (double)part.y * exp2((double)part.x - (double)tref) : 0.0);
        const RowResult res = finish_row(a, ref, (double)tref, t, r);
        if (tid == 0) {
            a.loss[row] = res.dead ? 0.0f : w * res.loss;
            a.stats[2 * row] = res.stat0;
            a.stats[2 * row + 1] = res.stat1;
        }
    }
}

template <class T, int kMode>
static hipError_t distill_rows(hipStream_t s, const DistillArgs& a) {
    const dim3 grid((uint32_t)(a.in.rows * a.splits));
    const size_t lds = bitmap_words(a.in.cols) * sizeof(uint32_t);
    const int32_t each = (a.per + kRowThreads - 1) / kRowThreads;
    if (each <= 4) hipLaunchKernelGGL((k_distill_row<T, 4, kMode>), grid, dim3(kRowThreads), lds, s, a);
    else if (each <= 8) hipLaunchKernelGGL((k_distill_row<T, 8, kMode>), grid, dim3(kRowThreads), lds, s, a);
    else hipLaunchKernelGGL((k_distill_row<T, kRowGranules, kMode>), grid, dim3(kRowThreads), lds, s, a);
    return hipGetLastError();
}

template <class T>
static hipError_t forward_typed(hipStream_t s, const DistillArgs& a) {
    if (a.splits == 1) return a.dz ? distill_rows<T, kLossGrad>(s, a) : distill_rows<T, kLoss>(s, a);
    hipError_t e = distill_rows<T, kPart>(s, a);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((k_distill_join<T>), dim3((uint32_t)a.in.rows), dim3(kRowThreads),
                       bitmap_words(a.in.cols) * sizeof(uint32_t), s, a);
    if ((e = hipGetLastError()) != hipSuccess || !a.dz) return e;
    return distill_rows<T, kGrad>(s, a);
}

hipError_t launch_distill_forward(hipStream_t s, const DistillArgs& a) {
    if (a.in.dtype == SCAPE_DTYPE_F32) return forward_typed<F32>(s, a);
    if (a.in.dtype == SCAPE_DTYPE_BF16) return forward_typed<BF16>(s, a);
    return forward_typed<F16>(s, a);
}

hipError_t launch_distill_backward(hipStream_t s, const DistillArgs& a) {
    if (a.in.dtype == SCAPE_DTYPE_F32) return distill_rows<F32, kGrad>(s, a);
    if (a.in.dtype == SCAPE_DTYPE_BF16) return distill_rows<BF16, kGrad>(s, a);
    return distill_rows<F16, kGrad>(s, a);
}

}  // namespace scape
