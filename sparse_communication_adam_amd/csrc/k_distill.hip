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

constexpr int kEntries = SCAPE_DISTILL_MAX_K / kRowThreads;  // entries a thread
static_assert(SCAPE_DISTILL_MAX_K % kRowThreads == 0, "entries are dealt out evenly");

// The bitmap: bit v is column v.  Byte-addressed reads of eight columns from
// any column on: two words around it.
__device__ __forceinline__ uint32_t bits_from(const uint32_t* bitmap, int32_t e) {
    const uint32_t w = (uint32_t)e >> 5, sh = (uint32_t)e & 31u;
    const uint64_t two = (uint64_t)bitmap[w] | ((uint64_t)bitmap[w + 1] << 32);
    return (uint32_t)(two >> sh);
}
inline uint32_t bitmap_words(int64_t cols) { return (uint32_t)((cols + 31) / 32 + 1); }

// A row's teacher entries, thread t holding entries t, t + kRowThreads, ...
struct Entries {
    int32_t col[kEntries];  // -1: none
    double lt[kEntries];    // s t_j (minus the teacher's lse where it is given)
};

// Reads the row's entries and marks their columns.  An entry whose column is
// outside the row is none, and so is one whose column a lower slot has.
// Returns whether the row has any entry.  Holds four barriers at most; the
// bitmap is complete after it.
__device__ __forceinline__ bool read_entries(const DistillArgs& a, int64_t row, uint32_t* bitmap, Entries& en) {
    const uint32_t tid = threadIdx.x;
    const int32_t n = (int32_t)a.in.cols;
    const uint32_t words = (uint32_t)((n + 31) / 32 + 1);
    for (uint32_t i = tid; i < words; i += kRowThreads) bitmap[i] = 0;
    const double lse = a.t_lse ? (double)a.t_lse[row] : 0.0;
#pragma unroll
    for (int i = 0; i < kEntries; ++i) {
        const int32_t slot = (int32_t)tid + i * kRowThreads;
        en.col[i] = -1;
        en.lt[i] = 0.0;
        if (slot < a.k) {
            const int64_t at = row * a.k + slot;
            const int32_t c = a.t_idx[at];
            if (c >= 0 && c < n) {
                en.col[i] = c;
                const float t = load_any(a.t_val, a.t_dtype, at);
                en.lt[i] = t == kNegInf ? (double)t : (double)t * (double)a.scale - lse;
            }
        }
    }
    __syncthreads();
    bool again = false, any = false;
#pragma unroll
    for (int i = 0; i < kEntries; ++i)
        if (en.col[i] >= 0) {
            const uint32_t bit = 1u << (en.col[i] & 31);
            again |= (atomicOr(&bitmap[en.col[i] >> 5], bit) & bit) != 0;
            any = true;
        }
    if (__syncthreads_or(again)) {
        // some column twice: which thread came first is chance, so every
        // entry looks for its column in the slots below its own
#pragma unroll
        for (int i = 0; i < kEntries; ++i)
            if (en.col[i] >= 0) {
                const int32_t slot = (int32_t)tid + i * kRowThreads;
                for (int32_t j = 0; j < slot; ++j)
                    if (a.t_idx[row * a.k + j] == en.col[i]) {
                        en.col[i] = -1;
                        break;
                    }
            }
    }
    return __syncthreads_or(any);
}

struct RowSums {  // of the entries, over the row
    double top;   // sum 2^(x_j - ref), x_j = z_j c2
    double q;     // sum q'_j  (q' is not normalised where the teacher is renormalised)
    double qt;    // sum q'_j lt_j
    double qx;    // sum q'_j x_j
};

// The row's loss, statistics and gradient factors from the tail's sum t =
// sum 2^(x - tref) and the entries' sums, against ref.
struct RowResult {
    float loss;          // KL
    float stat0, stat1;  // L, log p_T
    float tail;          // the tail's gradient is tail 2^(x_v - tref)
    double inv;          // 1 / sum 2^(x - ref): p_v = inv 2^(x_v - ref)
    double whole;        // Q
    double qnorm;        // q_j = qnorm q'_j
    bool dead;           // no student mass at all: nothing to learn
};
__device__ RowResult finish_row(const DistillArgs& a, double ref, double tref, double t, const RowSums& s,
                                double tmax) {
    RowResult r;
    const bool has_tail = !(t == 0.0);
    const double far = has_tail ? exp2(tref - ref) : 0.0;  // 0 too where the tail is out of range
    const double sum = t * far + s.top;
    const double log2sum = log2(sum);
    double qsum, log_shift = 0.0, rest = 0.0;
    if (a.t_lse) {
        r.qnorm = 1.0;
        qsum = s.q;
        rest = has_tail && 1.0 - qsum > 0.0 ? 1.0 - qsum : 0.0;  // no tail: its term is left out
    } else if (s.q > 0.0 || s.q != s.q) {
        r.qnorm = 1.0 / s.q;
        qsum = 1.0;
        log_shift = tmax + log(s.q);  // log q_j = lt_j - log_shift
    } else {
        r.qnorm = qsum = 0.0;  // every entry's value is -inf
    }
    const double tail = t * far;
    double lpt = -__builtin_inf();
    if (tail > 1e-290)
        lpt = -log1p(s.top / tail);
    else if (has_tail)
        lpt = (log2(t) + (tref - ref) - log2sum) * kLn2;
    double kl = 0.0;
    if (qsum != 0.0) kl = s.qt * r.qnorm - qsum * log_shift - (s.qx * r.qnorm - qsum * (ref + log2sum)) * kLn2;
    if (rest > 0.0) kl += rest * (log(rest) - lpt);
    r.whole = qsum + rest;
    r.loss = (float)kl;
    r.stat0 = (float)((ref + log2sum) * kLn2);
    r.stat1 = (float)lpt;
    r.inv = 1.0 / sum;
    // (Q - q_T / p_T) p_v with q_T / p_T = q_T + q_T top / tail
    r.tail = has_tail ? (float)(qsum * far / sum - rest * (s.top / sum) / t) : 0.0f;
    r.dead = sum == 0.0;
    return r;
}

__device__ __forceinline__ double block_sum_f64(double x, double* lds) {
    const double w = wave_sum_f64(x);
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x / 64] = w;
    __syncthreads();
    double t = 0.0;
#pragma unroll
    for (int i = 0; i < kRowWaves; ++i) t += lds[i];
    return t;
}

// The entries' terms: q'_j = exp(lt_j - tmax) (tmax 0 where the teacher's lse
// is given), x_j from the row itself.
template <class T>
__device__ __forceinline__ void entry_terms(const DistillArgs& a, const Entries& en, const float* zc, double tmax,
                                            double ref, RowSums& s) {
    s = RowSums{0.0, 0.0, 0.0, 0.0};
#pragma unroll
    for (int i = 0; i < kEntries; ++i)
        if (en.col[i] >= 0) {
            const double x = (double)zc[i] * (double)a.c2, q = exp(en.lt[i] - tmax);
            s.top += exp2(x - ref);
            if (q > 0.0) {
                s.q += q;
                s.qt += q * en.lt[i];
                s.qx += q * x;
            }
        }
}

template <class T, int kGran, int kMode>
__global__ __launch_bounds__(kRowThreads) void k_distill_row(DistillArgs a) {
    extern __shared__ uint32_t bitmap[];
    __shared__ float wmax[3][kRowWaves];
    __shared__ float wsum[kRowWaves];
    __shared__ double wd[4][kRowWaves];
    __shared__ RowResult s_res;
    using raw = typename T::raw;
    const uint32_t tid = threadIdx.x, wave = tid / 64;
    const int64_t row = blockIdx.x / (uint32_t)a.splits;
    const int32_t sp = (int32_t)(blockIdx.x % (uint32_t)a.splits);
    const raw* z = static_cast<const raw*>(a.in.z) + row * a.in.ld;
    const int lead = row_lead<T>(z);
    const int32_t total = (int32_t)((lead + a.in.cols + T::kN - 1) / T::kN);
    const int32_t g0 = sp * a.per;
    const int32_t cnt = min(a.per, total - g0);
    const int64_t n = a.in.cols;
    raw* dz = nullptr;
    bool vec = false;
    if constexpr (kMode == kLossGrad || kMode == kGrad) {
        dz = static_cast<raw*>(a.dz) + row * a.ld_dz;
        vec = row_lead<T>(dz) == lead;
    }

    float w = a.weight ? a.weight[row] : 1.0f;
    if (kMode == kGrad && a.dloss) w = w == 0.0f ? 0.0f : w * a.dloss[row];
    gran g[kGran];
    if (w != 0.0f) {
#pragma unroll
        for (int c = 0; c < kGran; ++c) {
            const int32_t gi = (int32_t)tid + c * kRowThreads;
            const int64_t e0 = gi < cnt ? (int64_t)(g0 + gi) * T::kN - lead : n;
            if (c * kRowThreads < cnt || c == 0) g[c] = load_granule<T>(z, e0, n);
        }
    }
    Entries en;
    const bool alive = w != 0.0f && read_entries(a, row, bitmap, en);
    if (!alive) {  // the same for the whole workgroup
        if constexpr (kMode == kLoss || kMode == kLossGrad)
            if (tid == 0) {
                a.loss[row] = 0.0f;
                a.stats[2 * row] = 0.0f;
                a.stats[2 * row + 1] = 0.0f;
            }
        if constexpr (kMode == kLossGrad || kMode == kGrad)
            for (int32_t gi = (int32_t)tid; gi < cnt; gi += kRowThreads)
                store_granule<T>(dz, (int64_t)(g0 + gi) * T::kN - lead, n, vec, gran{0u, 0u, 0u, 0u});
        return;
    }

    // the entries' logits (of this part only where the gradient may
    // overwrite the logits part by part)
    float zc[kEntries];
#pragma unroll
    for (int i = 0; i < kEntries; ++i) {
        zc[i] = 0.0f;
        if (en.col[i] >= 0) {
            const int32_t gi = (en.col[i] + lead) / T::kN - g0;
            if (kMode == kLoss || kMode == kLossGrad || (kMode == kGrad && gi >= 0 && gi < cnt))
                zc[i] = T::up1(z[en.col[i]]);
        }
    }

    float ref = 0.0f, vref = 0.0f, tail = 0.0f;  // references of the entries and of the tail, the tail's factor
    double inv = 0.0, whole = 0.0, qnorm = 0.0, tmax = 0.0;
    if constexpr (kMode != kGrad) {
        // strike the entries out; maxima of the tail, the entries and the teacher
        float m = kNegInf, mt = kNegInf, mq = kNegInf;
#pragma unroll
        for (int c = 0; c < kGran; ++c)
            if (c * kRowThreads < cnt || c == 0) {
                const int32_t gi = (int32_t)tid + c * kRowThreads;
                const int32_t e0 = (g0 + gi) * T::kN - lead;
                if (gi < cnt) {
                    uint32_t b = e0 >= 0 ? bits_from(bitmap, e0) : bits_from(bitmap, 0) << -e0;
                    b &= (1u << T::kN) - 1u;
                    if (b) {
#pragma unroll
                        for (int j = 0; j < T::kN; ++j)
                            if (b & (1u << j)) T::set(g[c], j, (raw)T::kNegInfBits);
                    }
                }
#pragma unroll
                for (int j = 0; j < T::kN; ++j) m = fmaxf(m, T::up(g[c], j));
            }
        if constexpr (kMode != kPart) {
#pragma unroll
            for (int i = 0; i < kEntries; ++i)
                if (en.col[i] >= 0) {
                    mt = fmaxf(mt, zc[i]);
                    mq = fmaxf(mq, (float)en.lt[i]);
                }
        }
        m = group_reduce<OpMaxF, 64>(m);
        if constexpr (kMode != kPart) {
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
            m = fmaxf(m, wmax[0][i]);
            mt = fmaxf(mt, wmax[1][i]);
            mq = fmaxf(mq, wmax[2][i]);
        }
        // The tail is summed against its own maximum: it may lie far below the entries.
        const float tref = m == kNegInf ? 0.0f : m * a.c2;
        float sum = 0.0f;
#pragma unroll
        for (int c = 0; c < kGran; ++c)
            if (c * kRowThreads < cnt || c == 0) {
#pragma unroll
                for (int j = 0; j < T::kN; ++j) sum += fast_exp2(__builtin_fmaf(T::up(g[c], j), a.c2, -tref));
            }
        sum = group_reduce<OpSumF, 64>(sum);
        if ((tid & 63) == 0) wsum[wave] = sum;
        if constexpr (kMode == kPart) {
            __syncthreads();
            if (tid == 0) {
                double t = 0.0;
                for (int i = 0; i < kRowWaves; ++i) t += (double)wsum[i];
                a.part[row * a.splits + sp] = make_float2(tref, (float)t);
            }
            return;
        } else {
            const float both = fmaxf(m, mt);
            ref = both == kNegInf ? 0.0f : both * a.c2;
            tmax = a.t_lse ? 0.0 : (mq == kNegInf ? 0.0 : (double)mq);
            RowSums s;
            entry_terms<T>(a, en, zc, tmax, (double)ref, s);
            s.top = wave_sum_f64(s.top);
            s.q = wave_sum_f64(s.q);
            s.qt = wave_sum_f64(s.qt);
            s.qx = wave_sum_f64(s.qx);
            if ((tid & 63) == 0) {
                wd[0][wave] = s.top;
                wd[1][wave] = s.q;
                wd[2][wave] = s.qt;
                wd[3][wave] = s.qx;
            }
            __syncthreads();
            if (tid == 0) {
                RowSums r{0.0, 0.0, 0.0, 0.0};
                double t = 0.0;
                for (int i = 0; i < kRowWaves; ++i) {
                    t += (double)wsum[i];
                    r.top += wd[0][i];
                    r.q += wd[1][i];
                    r.qt += wd[2][i];
                    r.qx += wd[3][i];
                }
                const RowResult res = finish_row(a, (double)ref, (double)tref, t, r, tmax);
                a.loss[row] = res.dead ? 0.0f : w * res.loss;
                a.stats[2 * row] = res.stat0;
                a.stats[2 * row + 1] = res.stat1;
                s_res = res;
            }
            if constexpr (kMode == kLoss) return;
            __syncthreads();
            const RowResult res = s_res;
            if (res.dead) w = 0.0f;
            inv = res.inv;
            tail = res.tail;
            vref = tref;
            whole = res.whole;
            qnorm = res.qnorm;
        }
    } else {
        const float l = a.stats[2 * row], lpt = a.stats[2 * row + 1];
        // the teacher's sums, as in the forward pass
        if (!a.t_lse) {
            float mq = kNegInf;
#pragma unroll
            for (int i = 0; i < kEntries; ++i)
                if (en.col[i] >= 0) mq = fmaxf(mq, (float)en.lt[i]);
            mq = group_reduce<OpMaxF, 64>(mq);
            if ((tid & 63) == 0) wmax[0][wave] = mq;
            __syncthreads();
#pragma unroll
            for (int i = 0; i < kRowWaves; ++i) mq = fmaxf(mq, wmax[0][i]);
            tmax = mq == kNegInf ? 0.0 : (double)mq;
        }
        double q = 0.0;
#pragma unroll
        for (int i = 0; i < kEntries; ++i)
            if (en.col[i] >= 0) q += exp(en.lt[i] - tmax);
        q = block_sum_f64(q, wd[0]);
        double rest = 0.0;
        if (a.t_lse) {
            qnorm = 1.0;
            rest = 1.0 - q > 0.0 && lpt != kNegInf ? 1.0 - q : 0.0;
        } else {
            qnorm = q == 0.0 ? 0.0 : 1.0 / q;
            q = q == 0.0 ? 0.0 : 1.0;
        }
        whole = q + rest;
        // (Q - q_T / p_T) p_v, against L, or where exp(-log p_T) could leave
        // the range against the tail's own log-sum-exp
        const double t = q * exp((double)lpt) + rest * expm1((double)lpt);
        ref = vref = l;
        if (rest == 0.0) {
            tail = (float)q;
        } else if (lpt > -30.0f) {
            tail = (float)(t * exp(-(double)lpt));
        } else {
            tail = (float)t;
            vref = (float)((double)l + (double)lpt);
        }
        if (l == kNegInf) w = 0.0f;
    }

    if constexpr (kMode == kLossGrad || kMode == kGrad) {
        const float gs = w * a.scale;
        if (gs == 0.0f) {  // the whole row is -inf: no gradient
#pragma unroll
            for (int c = 0; c < kGran; ++c) {
                const int32_t gi = (int32_t)tid + c * kRowThreads;
                if (gi < cnt) store_granule<T>(dz, (int64_t)(g0 + gi) * T::kN - lead, n, vec, gran{0u, 0u, 0u, 0u});
            }
            return;
        }
        const float f = gs * tail;
#pragma unroll
        for (int c = 0; c < kGran; ++c) {
            const int32_t gi = (int32_t)tid + c * kRowThreads;
            if (gi < cnt) {
                float d[T::kN];
#pragma unroll
                for (int j = 0; j < T::kN; ++j) {
                    const float x = T::up(g[c], j);
                    // from the statistics: the difference first, as float32
                    // gradients would see the error of L log2(e)
                    const float e = kMode == kLossGrad ? __builtin_fmaf(x, a.c2, -vref)
                                                       : __builtin_fmaf(x, a.scale, -vref) * kLog2e;
                    d[j] = f * fast_exp2(e);
                }
                store_granule<T>(dz, (int64_t)(g0 + gi) * T::kN - lead, n, vec, T::down(d));
            }
        }
        __syncthreads();  // the entries' columns are written over the tail's values
#pragma unroll
        for (int i = 0; i < kEntries; ++i)
            if (en.col[i] >= 0) {
                const int32_t gi = (en.col[i] + lead) / T::kN - g0;
                if (gi >= 0 && gi < cnt) {
                    double p;
                    if constexpr (kMode == kLossGrad)
                        p = exp2((double)zc[i] * (double)a.c2 - (double)ref) * inv;
                    else
                        p = exp((double)zc[i] * (double)a.scale - (double)ref);
                    const double q = exp(en.lt[i] - tmax) * qnorm;
                    dz[en.col[i]] = T::down1((float)((double)gs * (p * whole - q)));
                }
            }
    }
}

// Joins the parts of a split row: the loss and the statistics.
template <class T>
__global__ __launch_bounds__(kRowThreads) void k_distill_join(DistillArgs a) {
    extern __shared__ uint32_t bitmap[];
    __shared__ float wmax[2][kRowWaves];
    __shared__ double wd[kRowWaves], we[kRowWaves], wf[kRowWaves], wg[kRowWaves];
    using raw = typename T::raw;
    const uint32_t tid = threadIdx.x, wave = tid / 64;
    const int64_t row = blockIdx.x;
    const raw* z = static_cast<const raw*>(a.in.z) + row * a.in.ld;
    const float w = a.weight ? a.weight[row] : 1.0f;
    Entries en;
    const bool alive = w != 0.0f && read_entries(a, row, bitmap, en);
    if (!alive) {
        if (tid == 0) {
            a.loss[row] = 0.0f;
            a.stats[2 * row] = 0.0f;
            a.stats[2 * row + 1] = 0.0f;
        }
        return;
    }
    float zc[kEntries], mt = kNegInf, mq = kNegInf;
#pragma unroll
    for (int i = 0; i < kEntries; ++i) {
        zc[i] = 0.0f;
        if (en.col[i] >= 0) {
            zc[i] = T::up1(z[en.col[i]]);
            mt = fmaxf(mt, zc[i]);
            mq = fmaxf(mq, (float)en.lt[i]);
        }
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
        mt = fmaxf(mt, wmax[0][i]);
        mq = fmaxf(mq, wmax[1][i]);
    }
    const float2* p = a.part + row * a.splits;
    float tref = kNegInf;
    for (int s = 0; s < a.splits; ++s)
        if (p[s].y != 0.0f) tref = fmaxf(tref, p[s].x);
    float ref = fmaxf(tref, mt == kNegInf ? kNegInf : mt * a.c2);
    if (tref == kNegInf) tref = 0.0f;
    if (ref == kNegInf) ref = 0.0f;
    const double tmax = a.t_lse ? 0.0 : (mq == kNegInf ? 0.0 : (double)mq);
    RowSums s;
    entry_terms<T>(a, en, zc, tmax, (double)ref, s);
    s.top = block_sum_f64(s.top, wd);
    s.q = block_sum_f64(s.q, we);
    s.qt = block_sum_f64(s.qt, wf);
    s.qx = block_sum_f64(s.qx, wg);
    if (tid == 0) {
        double t = 0.0;
        for (int i = 0; i < a.splits; ++i)
            if (p[i].y != 0.0f) t += (double)p[i].y * exp2((double)p[i].x - (double)tref);
        const RowResult res = finish_row(a, (double)ref, (double)tref, t, s, tmax);
        a.loss[row] = res.dead ? 0.0f : w * res.loss;
        a.stats[2 * row] = res.stat0;
        a.stats[2 * row + 1] = res.stat1;
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
