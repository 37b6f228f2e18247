// k_vocab.hip - softmax cross entropy over a vocabulary from hidden states
// h [rows][dim] and head weights w [cols][dim], without the logits: their
// products live in registers, tile by tile.
//
//   z = scale * h w^T;  lse = log sum exp z;  loss = weight (lse - z[label])
//   P = g (exp(z - lse) - onehot), g = weight * dloss * scale
//   dh = P w;  dw = P^T h
//
// Three matrix products over one tile loop.  The logits' tile has the words as
// MFMA rows and the tokens as its columns, so a lane holds words of one token
// and the row statistics are sums in registers.  The backward pass takes the
// vocabulary in pieces: P of a piece goes to the workspace in 16 bits, and both
// gradients read it from there.
//
// What bounds it: of many tokens the matrix cores, which at this load run below
// their top clock; of few the reading of w and the writing of dw.  8192x32000x2048
// bf16, us in a trace (averages of 43 passes, here and below), and PFLOP/s: sums 828
// (1.30), P 2 x 427 (1.26), dh 2 x 398 (1.35), dw 2 x 450 (1.19); the library's plain
// products of these shapes take 834, 856 and 1129.  7x50304x1024: sums 21 us, 4.9
// TB/s of w.
#include "loss_device.h"

namespace scape {

namespace {

typedef float f4 __attribute__((ext_vector_type(4)));
typedef uint32_t u2 __attribute__((ext_vector_type(2)));
typedef short s4 __attribute__((ext_vector_type(4)));
typedef short s8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) char lds_t;
typedef __attribute__((address_space(3))) void lds_void;

template <class T>
__device__ __forceinline__ f4 mfma(const s8& a, const s8& b, const f4& c) {
    if constexpr (std::is_same<T, BF16>::value) {
        typedef __bf16 v8 __attribute__((ext_vector_type(8)));
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8, a), __builtin_bit_cast(v8, b), c, 0, 0, 0);
    } else {
        typedef _Float16 v8 __attribute__((ext_vector_type(8)));
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8, a), __builtin_bit_cast(v8, b), c, 0, 0, 0);
    }
}

constexpr uint32_t kOutside = 0x80000000u;      // an offset that the resource's bound turns into zeros
constexpr uint32_t kRawBuffer = 0x00027000u;

// One operand of a product: rows of 16-bit elements, ld apart.  Along: the
// summed axis lies along the rows (extent rows of them); else it runs over
// rows of `extent` elements.  A blocked one lies in blocks of 64 elements of its
// rows, which are `block` apart; it has nothing but whole tiles.
// All sizes are below 2^21 (the call checks that), so their sums are 32-bit.
struct Side {
    const void* p;
    int32_t ld, extent, depth;  // depth: elements of the summed axis
    int32_t block = 0;
};

// Moves a tile of kR x kDepth from memory to LDS, 16 bytes a lane, and reads MFMA
// fragments of it.  The load writes LDS in lane order, so the lanes' addresses
// are permuted instead: the 16-byte pieces of a row are exchanged by an XOR
// that spreads what one fragment read touches over all banks.
constexpr int kDepth = 64;  // elements of the summed axis in a slot
template <bool kAlong, int kR, int kThreads, bool kBlocked>
struct Stage {
    static constexpr int kBytes = kR * 2 * kDepth;
    static constexpr int kPieces = kBytes / 16;
    // Every wave issues as many loads, so that they can be counted: of a tile
    // with fewer pieces than threads some are loaded twice.
    static constexpr int kLoads = kPieces > kThreads ? kPieces / kThreads : 1;
    static constexpr int kLanes = kPieces < kThreads ? kPieces : kThreads;
    static constexpr int kRow = kAlong ? kDepth * 2 : kR * 2;  // bytes
    static constexpr int kRowPieces = kRow / 16;
    // Rows that one load of all threads covers.  Where the exchange is the same
    // from one load to the next, a lane's offset is one register and a multiple
    // of the row distance.
    static constexpr int kRowsALoad = kLanes / kRowPieces;
    static constexpr bool kSteady = kLoads == 1 || kRowsALoad % 16 == 0;
    static_assert(kPieces % 64 == 0 && (kPieces % kThreads == 0 || kThreads % kPieces == 0), "whole waves");
    static_assert(kAlong || (kR & (kR - 1)) == 0, "rows of pieces that an XOR stays in");
    uint32_t off[kSteady ? 1 : kLoads], pitch;  // a lane's
    int32_t piece;                              // a lane's first element along the depth
    uint32_t wave;                              // where a wave's share of a load begins in the slot
    const char* at;                             // the next tile, and what is left of the depth there
    int32_t left, bytes, ld, block;

    // what the pieces of row k are exchanged by; the same for k + 4 (k % 8 < 4)
    // and k + 16, which a fragment's reads and a lane's loads are apart
    static __device__ __forceinline__ uint32_t turn(uint32_t k) {
        if constexpr (kAlong) return k & 7u;
        if constexpr (kR >= 128) return ((k & 3u) | ((k >> 3) & 1u) << 2) << 1;
        if constexpr (kR == 64) return (((k >> 1) & 1u) | ((k >> 3) & 1u) << 1) << 1;
        if constexpr (kR == 32) return ((k >> 3) & 1u) << 1;
        return 0;
    }

    // The tile at row (or column) r0 and depth k is the first.
    __device__ __forceinline__ void init(const Side& s, int32_t r0, int32_t k) {
        const uint32_t tid = threadIdx.x % kLanes;
        ld = kBlocked ? kDepth : s.ld;
        block = s.block;
        pitch = (uint32_t)(ld * 2);
#pragma unroll
        for (int i = 0; i < (kSteady ? 1 : kLoads); ++i) {
            const uint32_t q = (uint32_t)i * kThreads + tid, row = q / kRowPieces, pos = q % kRowPieces;
            const uint32_t at16 = pos ^ turn(row);
            off[i] = row * pitch + (kBlocked ? (at16 >> 3) * (uint32_t)(block * 2) + ((at16 & 7) << 4) : at16 << 4);
            if (i == 0) piece = (int32_t)(at16 * 8);
        }
        wave = __builtin_amdgcn_readfirstlane(tid >> 6) * 1024;
        left = s.depth - k;
        const int32_t rows = s.extent - r0 < kR ? s.extent - r0 : kR;
        if constexpr (kBlocked) {
            bytes = kAlong ? rows * ld * 2 : (kR / 64 - 1) * block * 2 + 128;  // of all rows, or of a last one
            at = static_cast<const char*>(s.p) +
                 (kAlong ? (int64_t)r0 * ld + (int64_t)(k / 64) * block : (int64_t)k * ld + (int64_t)(r0 / 64) * block) * 2;
        } else {
            bytes = kAlong ? ((rows - 1) * ld + left) * 2 : (s.extent - r0) * 2;  // the same
            at = static_cast<const char*>(s.p) + (kAlong ? (int64_t)r0 * ld + k : (int64_t)k * ld + r0) * 2;
        }
    }

    // The next tile to a slot.  Behind the end of the depth there are zeros.
    __device__ __forceinline__ void load(lds_t* to) {
        const int32_t rows = left < kDepth ? left : kDepth;
        const int32_t held = kAlong ? bytes : (rows - 1) * ld * 2 + bytes, some = left > 0 ? held : 0;
        const auto rsrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(at), 0, some, kRawBuffer);
        // one register, not one for each load: the sums need them
        asm volatile("" : "+v"(off[0]));
        const uint32_t kill = kAlong && piece >= left ? kOutside : 0u;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const uint32_t o = kSteady ? (off[0] | kill) + (uint32_t)(i * kRowsALoad) * pitch : off[kSteady ? 0 : i] | kill;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_void*)(to + wave + i * kThreads * 16), 16, o, 0, 0, 0);
        }
        at += !kAlong ? (int64_t)kDepth * 2 * ld : kBlocked ? (int64_t)block * 2 : kDepth * 2;
        if (kAlong && !kBlocked) bytes -= kDepth * 2;
        left -= kDepth;
    }

    // Where a lane reads the first fragment of the wave's rows (from r0, a
    // multiple of the wave's share), and from there fragment f of the h-th 32
    // of the depth.
    static __device__ __forceinline__ uint32_t first(uint32_t lane, uint32_t r0) {
        if constexpr (kAlong) {
            const uint32_t row = r0 + (lane & 15u);
            return row * kRow + (((lane >> 4) ^ turn(row)) << 4);
        } else {
            const uint32_t k = (lane >> 4) * 8 + ((lane & 15u) >> 2), c = lane & 3u;
            return k * kRow + (((r0 / 8 + (c >> 1)) ^ turn(k)) << 4) + (c & 1u) * 8;
        }
    }
    static __device__ __forceinline__ s8 read(const lds_t* tile, uint32_t first, int f, int h) {
        if constexpr (kAlong) {
            return *reinterpret_cast<const __attribute__((address_space(3))) s8*>(tile + (first ^ (uint32_t)(h * 64)) + f * 16 * kRow);
        } else {
            typedef __attribute__((address_space(3))) s4 lds_s4;
            lds_t* const p = const_cast<lds_t*>(tile) + (first ^ (uint32_t)(f * 32)) + h * 32 * kRow;
            const s4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4*)p);
            const s4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4*)(p + 4 * kRow));
            return s8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
        }
    }
};

// A workgroup's tile of a product: kM x kN over kWM x kWN waves.  The operands
// come through slots of 64 deep, kSlotsA of the one and kSlotsB of the other.  A
// wave holds the fragments of a slot's two halves: while one half is multiplied
// the other is read, and when both are in registers the slots are loaded anew,
// the other slots' products ahead of their use.
template <class T, bool kAlongA, bool kAlongB, int kM, int kN, int kWM, int kWN, int kSlotsA, int kSlotsB, bool kBlockedB = false>
struct Tile {
    static constexpr int kThreads = kWM * kWN * 64;
    static constexpr int kTM = kM / kWM, kTN = kN / kWN;  // a wave's part, powers of two
    static constexpr int kFM = kTM / 16, kFN = kTN / 16;
    using A = Stage<kAlongA, kM, kThreads, false>;
    using B = Stage<kAlongB, kN, kThreads, kBlockedB>;
    static constexpr int kLoads = A::kLoads + B::kLoads;
    static_assert(kWM * kWN * 16 * kTM * 2 <= A::kBytes, "hand_out's rows");
    static constexpr int kLdsA = kSlotsA * A::kBytes, kLds = kLdsA + kSlotsB * B::kBytes;
    // Loads that may be on their way when the next slots have to be there: those
    // issued behind the last of them (of a step's loads B's are first).
    static constexpr int kAhead = (kSlotsB - 2) * kLoads + (kSlotsA > kSlotsB ? A::kLoads : 0);
    static_assert(kSlotsA >= kSlotsB && kSlotsB >= 2, "");
    // A half's fragments.
    struct Half {
        s8 a[kFM], b[kFN];
        __device__ __forceinline__ void read(const lds_t* from_a, const lds_t* from_b, uint32_t& fa, uint32_t& fb, int h) {
            asm volatile("" : "+v"(fa), "+v"(fb));  // addresses are made from these two here, and not kept
#pragma unroll
            for (int j = 0; j < kFN; ++j) b[j] = B::read(from_b, fb, j, h);
#pragma unroll
            for (int i = 0; i < kFM; ++i) a[i] = A::read(from_a, fa, i, h);
        }
    };
    f4 acc[kFM][kFN];
    A la;
    B lb;
    uint32_t fa, fb;

    __device__ __forceinline__ void start(const Side& a, const Side& b, int32_t m0, int32_t n0, int32_t k0) {
        la.init(a, m0, k0);
        lb.init(b, n0, k0);
        fa = A::first(lane_id(), wave_m());
        fb = B::first(lane_id(), wave_n());
#pragma unroll
        for (int i = 0; i < kFM; ++i)
#pragma unroll
            for (int j = 0; j < kFN; ++j) acc[i][j] = f4{0, 0, 0, 0};
    }

    // Both operands along the depth from k0 to k1; what is loaded behind the end
    // of it is zeros.
    __device__ __forceinline__ void run(const Side& a, const Side& b, int32_t m0, int32_t n0, int32_t k0, int32_t k1,
                                        lds_t* lds) {
        static_assert(kAlongA && kAlongB, "the compiler waits for every load before a transposing read of the same object");
        start(a, b, m0, n0, k0);
#pragma unroll
        for (int i = -kSlotsA; i < 0; ++i) {
            if (i + kSlotsB >= 0) lb.load(lds + kLdsA + (i + kSlotsB) * B::kBytes);
            asm volatile("" ::: "memory");
            la.load(lds + (i + kSlotsA) * A::kBytes);
        }
        wait<kAhead + kLoads>();
        Half x, y;
        x.read(lds, lds + kLdsA, fa, fb, 0);
        uint32_t ia = 0, ib = kLdsA, ja = A::kBytes, jb = kLdsA + B::kBytes;  // this step's slots and the next one's
        for (int32_t k = k0; k < k1; k += kDepth) {
            slot(lds + ia, lds + ib, lds + ja, lds + jb, x, y);
            ia = ja;
            ib = jb;
            ja = ja == kLdsA - A::kBytes ? 0 : ja + A::kBytes;
            jb = jb == kLds - B::kBytes ? kLdsA : jb + B::kBytes;
        }
        wait<0>();  // what was loaded behind the end is in LDS, too
    }
    // The same for any operands.  Every slot is an object of its own and the loop
    // goes through them by name, so that the compiler knows what is read to be
    // none of what is loaded meanwhile.
    struct Slots {
        lds_t *a[3], *b[3];
    };
    static constexpr int kTurn = kSlotsA == kSlotsB ? kSlotsA : kSlotsA * kSlotsB;
    __device__ __forceinline__ void run(const Side& a, const Side& b, int32_t m0, int32_t n0, int32_t k0, int32_t k1,
                                        const Slots& s) {
        start(a, b, m0, n0, k0);
#pragma unroll
        for (int i = -kSlotsA; i < 0; ++i) {
            if (i + kSlotsB >= 0) lb.load(s.b[i + kSlotsB]);
            asm volatile("" ::: "memory");
            la.load(s.a[i + kSlotsA]);
        }
        wait<kAhead + kLoads>();
        Half x, y;
        x.read(s.a[0], s.b[0], fa, fb, 0);
        int32_t k = k0;
        for (; k + (kTurn - 1) * kDepth < k1; k += kTurn * kDepth) turn<0>(s, x, y);
        rest<0>(s, x, y, k, k1);
        wait<0>();
    }
    template <int i>
    __device__ __forceinline__ void turn(const Slots& s, Half& x, Half& y) {
        if constexpr (i < kTurn) {
            slot(s.a[i % kSlotsA], s.b[i % kSlotsB], s.a[(i + 1) % kSlotsA], s.b[(i + 1) % kSlotsB], x, y);
            turn<i + 1>(s, x, y);
        }
    }
    template <int i>
    __device__ __forceinline__ void rest(const Slots& s, Half& x, Half& y, int32_t k, int32_t k1) {
        if constexpr (i < kTurn - 1)
            if (k < k1) {
                slot(s.a[i % kSlotsA], s.b[i % kSlotsB], s.a[(i + 1) % kSlotsA], s.b[(i + 1) % kSlotsB], x, y);
                rest<i + 1>(s, x, y, k + kDepth, k1);
            }
    }
    __device__ __forceinline__ void slot(lds_t* now_a, lds_t* now_b, const lds_t* next_a, const lds_t* next_b, Half& x, Half& y) {
        y.read(now_a, now_b, fa, fb, 1);
        multiply(x);
        mix<false>();
        wait<kAhead>();
        x.read(next_a, next_b, fa, fb, 0);
        lb.load(now_b);
        asm volatile("" ::: "memory");  // in this order: kAhead counts on it
        la.load(now_a);
        multiply(y);
        mix<true>();
        __builtin_amdgcn_sched_barrier(0);
    }
    // All but the last n loads of every wave are in LDS, and every wave has the
    // fragments that it was reading.
    template <int n>
    static __device__ __forceinline__ void wait() {
        static_assert(n < 64, "what the counter holds");
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_waitcnt((n & 15) | 7 << 4 | 0 << 8 | (n >> 4) << 14);
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
    }
    __device__ __forceinline__ void multiply(const Half& f) {
#pragma unroll
        for (int i = 0; i < kFM; ++i)
#pragma unroll
            for (int j = 0; j < kFN; ++j) acc[i][j] = mfma<T>(f.a[i], f.b[j], acc[i][j]);
    }
    // The order of a half: a product for each read (of 16 bytes a lane) first, so
    // that the rest of the products covers the last read's way, and the loads
    // between those.
    static constexpr int kReadsA = kAlongA ? 1 : 2, kReadsB = kAlongB ? 1 : 2, kProducts = kFM * kFN;
    template <bool kFetch>
    static __device__ __forceinline__ void mix() {
        constexpr int kPlain = kProducts - kFM - kFN;
        static_assert(kFM + kFN <= 2 * kProducts, "");
        mix_reads<kFN, kReadsB>();
        mix_reads<kFM, kReadsA>();
        if constexpr (kFetch) mix_loads<kLoads, kPlain>();
    }
    template <int n, int each>
    static __device__ __forceinline__ void mix_reads() {
        if constexpr (n > 0) {
            __builtin_amdgcn_sched_group_barrier(0x100, each, 0);
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            mix_reads<n - 1, each>();
        }
    }
    template <int n, int products>
    static __device__ __forceinline__ void mix_loads() {
        if constexpr (n > 0) {
            constexpr int m = products > 0 ? (products + n - 1) / n : 0;
            __builtin_amdgcn_sched_group_barrier(0x010, 1, 0);
            if constexpr (m > 0) __builtin_amdgcn_sched_group_barrier(0x008, m, 0);
            mix_loads<n - 1, products - m>();
        }
    }
    // The wave's part of the tile as rows of the n axis: put(i, j) gives the four
    // 16-bit elements of the lane's place in fragment (i, j), out(n, m, granule)
    // takes eight of them of row n from m on, both counted within the wave's part.
    // A lane's own four are 8 bytes of a row and 16 lanes are 16 rows; through LDS
    // (behind the products, which are done with it) a row's 2 kTM bytes lie beside
    // each other.  16 rows at a time, LDS serving a wave in order.
    template <class Put, class Out>
    static __device__ __forceinline__ void hand_out(lds_t* lds, const Put& put, const Out& out) {
        constexpr int kPitch = kTM * 2, kRowPieces = kTM / 8;  // pieces are exchanged as the operands' are
        lds_t* const mine = lds + (threadIdx.x >> 6) * (16 * kPitch);
        const uint32_t lane = lane_id();
#pragma unroll
        for (int j = 0; j < kFN; ++j) {
#pragma unroll
            for (int i = 0; i < kFM; ++i) {
                const uint32_t piece = ((uint32_t)i * 2 + lane_m() / 8) ^ (lane_n() % kRowPieces);
                *reinterpret_cast<__attribute__((address_space(3))) u2*>(mine + lane_n() * kPitch + piece * 16 + lane_m() % 8 * 2) =
                    put(i, j);
            }
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
            for (int q = 0; q < (16 * kRowPieces + 63) / 64; ++q) {
                const uint32_t at = (uint32_t)q * 64 + lane, row = at / kRowPieces, piece = at % kRowPieces;
                if (16 * kRowPieces % 64 && at >= 16 * kRowPieces) break;
                const gran g = *reinterpret_cast<const __attribute__((address_space(3))) gran*>(
                    mine + row * kPitch + (piece ^ (row % kRowPieces)) * 16);
                out(j * 16 + row, piece * 8, g);
            }
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        }
    }
    // The wave's first row and column in the tile, and the lane's of a fragment.
    static __device__ __forceinline__ uint32_t wave_m() { return ((threadIdx.x >> 6) % kWM) * kTM; }
    static __device__ __forceinline__ uint32_t wave_n() { return ((threadIdx.x >> 6) / kWM) * kTN; }
    static __device__ __forceinline__ uint32_t lane_m() { return (lane_id() >> 4) * 4; }
    static __device__ __forceinline__ uint32_t lane_n() { return lane_id() & 15u; }
};

// Block b of a grid of nm x nn tiles.  Workgroups of one XCD, which share an
// L2, take runs of blocks (xcd_block); a run walks bands of kBand tiles of the n
// axis, all of the m axis for each.
constexpr uint32_t kBand = 8;
__device__ __forceinline__ void tile_of(uint32_t b, uint32_t nm, uint32_t nn, uint32_t& m, uint32_t& n) {
    const uint32_t band = b / (kBand * nm), first = band * kBand, in = b - band * kBand * nm;
    const uint32_t wide = nn - first < kBand ? nn - first : kBand;
    n = __builtin_amdgcn_readfirstlane(first + in % wide);  // divisions are made in vector registers
    m = __builtin_amdgcn_readfirstlane(in / wide);
}

// ---------------------------------------------------------------------------
// The loss: each tile's reference and sum of a token, and the label's logit.
// 2048x50257x1024 f16 takes 218 us (198 at the least): 1576 tiles on 256 CUs are seven rounds where
// 6.2 would do, and a tile's exponentials are not hidden behind products.

template <class T, int kM, int kN, int kWM, int kWN, int kSlotsA, int kSlotsB>
__global__ __launch_bounds__(kWM * kWN * 64) void k_vocab_sums(VocabArgs a) {
    using G = Tile<T, true, true, kM, kN, kWM, kWN, kSlotsA, kSlotsB>;
    __shared__ __attribute__((aligned(16))) char lds[G::kLds];
    uint32_t tm, tn;
    tile_of(xcd_block(blockIdx.x, gridDim.x), a.tiles_v, a.tiles_n, tm, tn);
    const int32_t m0 = (int32_t)tm * kM, n0 = (int32_t)tn * kN;
    const uint32_t lm = G::wave_m() + G::lane_m(), ln = G::wave_n() + G::lane_n();
    int32_t label[G::kFN];  // loaded ahead of the products
#pragma unroll
    for (int j = 0; j < G::kFN; ++j) label[j] = n0 + (int32_t)ln + j * 16 < a.rows ? a.label[n0 + (int32_t)ln + j * 16] : -1;
    G g;
    g.run(Side{a.w, (int32_t)a.ld_w, (int32_t)a.cols, (int32_t)a.dim}, Side{a.h, (int32_t)a.ld_h, (int32_t)a.rows, (int32_t)a.dim}, m0, n0, 0,
          (int32_t)a.dim, (lds_t*)lds);
    // the loop's last barrier is behind every read of the tiles
    float2* const red = reinterpret_cast<float2*>(lds);  // [kWM][kN]
    const int32_t left = (int32_t)a.cols - m0 - (int32_t)lm;  // words from the lane's first on
    const bool ragged = a.cols - m0 < kM;
#pragma unroll
    for (int j = 0; j < G::kFN; ++j) {
        const int32_t lab = label[j] - m0 - (int32_t)lm;  // of the lane's words
        if (ragged) {
#pragma unroll
            for (int i = 0; i < G::kFM; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (i * 16 + e >= left) g.acc[i][j][e] = kNegInf;
        }
        float top = kNegInf;
#pragma unroll
        for (int i = 0; i < G::kFM; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) top = fmaxf(top, g.acc[i][j][e]);
        // In base 2, against a reference that is a rounded product itself: the
        // fused multiply-add rounds each exponent once, and whatever the
        // reference's own rounding was stands in the reference.
        top = fmaxf(top, __shfl_xor(top, 16, 64));
        top = fmaxf(top, __shfl_xor(top, 32, 64));
        // Words that are none leave the lowest reference, which no sum gives way to.
        const float ref = top == kNegInf ? kLowest : top * a.c2;
        float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
        for (int i = 0; i < G::kFM; ++i) {
            s0 += fast_exp2(__builtin_fmaf(g.acc[i][j][0], a.c2, -ref));
            s1 += fast_exp2(__builtin_fmaf(g.acc[i][j][1], a.c2, -ref));
            s0 += fast_exp2(__builtin_fmaf(g.acc[i][j][2], a.c2, -ref));
            s1 += fast_exp2(__builtin_fmaf(g.acc[i][j][3], a.c2, -ref));
        }
        float sum = s0 + s1;
        sum += __shfl_xor(sum, 16, 64);
        sum += __shfl_xor(sum, 32, 64);
        if (lane_id() < 16) red[(G::wave_m() / G::kTM) * kN + ln + j * 16] = float2{ref, sum};
        if (label[j] >= 0 && lab >= 0 && lab < G::kTM && (lab & 15) < 4 && lab < left) {
            float at = 0.0f;
#pragma unroll
            for (int i = 0; i < G::kFM; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) at = lab == i * 16 + e ? g.acc[i][j][e] : at;
            a.at_label[n0 + (int64_t)ln + j * 16] = at;
        }
    }
    __syncthreads();
    for (uint32_t t = threadIdx.x; t < (uint32_t)kN; t += G::kThreads) {
        float2 r = red[t];
#pragma unroll
        for (int w = 1; w < kWM; ++w) {
            const float2 q = red[w * kN + t];
            const float ref = fmaxf(r.x, q.x);
            r.y = r.y * fast_exp2(r.x - ref) + q.y * fast_exp2(q.x - ref);
            r.x = ref;
        }
        if (n0 + t < a.rows) a.part[(int64_t)tm * a.rows + n0 + t] = r;
    }
}

// Joins a token's tiles: 16 tokens a workgroup, 64 threads each, four tiles on
// their way to a thread.  A launch and a chain of loads: 4.5 us in a trace for 7
// tokens and 786 tiles, 4.8 for 8192 and 125.
constexpr int kJoinTokens = 16, kJoinParts = 64, kJoinEach = 4;
__device__ __forceinline__ void join_sums(float2& r, const float2& p) {
    const float ref = fmaxf(r.x, p.x);
    r.y = r.y * fast_exp2(r.x - ref) + p.y * fast_exp2(p.x - ref);
    r.x = ref;
}
__global__ __launch_bounds__(kJoinTokens* kJoinParts) void k_vocab_join(VocabArgs a) {
    __shared__ float2 red[kJoinParts / 4][kJoinTokens];
    const uint32_t t = threadIdx.x % kJoinTokens, q = threadIdx.x / kJoinTokens;
    const int64_t n = (int64_t)blockIdx.x * kJoinTokens + t;
    float2 r = float2{kLowest, 0.0f};
    if (n < a.rows)
        for (uint32_t v = q; v < a.tiles_v; v += kJoinParts * kJoinEach) {
            float2 p[kJoinEach];
#pragma unroll
            for (int i = 0; i < kJoinEach; ++i) {
                const uint32_t at = v + i * kJoinParts;
                p[i] = at < a.tiles_v ? a.part[(int64_t)at * a.rows + n] : float2{kLowest, 0.0f};
            }
#pragma unroll
            for (int i = 0; i < kJoinEach; ++i) join_sums(r, p[i]);
        }
    // a wave holds four threads of each token
    join_sums(r, float2{__shfl_xor(r.x, 16, 64), __shfl_xor(r.y, 16, 64)});
    join_sums(r, float2{__shfl_xor(r.x, 32, 64), __shfl_xor(r.y, 32, 64)});
    if (lane_id() < kJoinTokens) red[threadIdx.x >> 6][t] = r;
    __syncthreads();
    if (q >= 4) return;
    r = red[q * 4][t];
#pragma unroll
    for (int i = 1; i < 4; ++i) join_sums(r, red[q * 4 + i][t]);
    join_sums(r, float2{__shfl_xor(r.x, 16, 64), __shfl_xor(r.y, 16, 64)});
    join_sums(r, float2{__shfl_xor(r.x, 32, 64), __shfl_xor(r.y, 32, 64)});
    if (q != 0 || n >= a.rows) return;
    const double lse2 = (double)r.x + log2((double)r.y);  // in base 2
    a.lse[n] = (float)(lse2 * kLn2);
    const int32_t lab = a.label[n];
    const float w = a.weight ? a.weight[n] : 1.0f;
    const bool on = lab >= 0 && lab < a.cols && w != 0.0f;
    a.loss[n] = on ? (float)((double)w * kLn2 * (lse2 - (double)a.at_label[n] * (double)a.c2)) : 0.0f;
}

// ---------------------------------------------------------------------------
// The gradient.

// Per row: the factor of its P, its log-sum-exp in base 2, and the power of two
// that stands beside an fp16 P.  bf16 has float32's range, so P takes the whole
// factor; an fp16 P is (p - onehot) times a mantissa in [2^14, 2^15), so that p
// keeps its bits down to 2^-28, and the power of two is put on dh exactly and on
// the copy of h that dw takes.
__device__ __forceinline__ float row_factor(const VocabArgs& a, int64_t n) {
    const int32_t lab = a.label[n];
    if (lab < 0 || lab >= a.cols) return 0.0f;
    const float w = a.weight ? a.weight[n] : 1.0f, d = a.dloss ? a.dloss[n] : 1.0f;
    return w == 0.0f || d == 0.0f ? 0.0f : (float)((double)w * (double)d * (double)a.scale);
}
__device__ __forceinline__ bool has_exponent(float f) { return f != 0.0f && __builtin_isfinite(f); }
__device__ __forceinline__ int exponent_of(float f) {  // |f| < 2^e
    int e;
    (void)frexpf(f, &e);
    return e;
}
__device__ __forceinline__ VocabRow row_of(const VocabArgs& a, int64_t n) {
    VocabRow r{0.0f, 0.0f, -1, 0.0f};
    const float f = n < a.rows ? row_factor(a, n) : 0.0f;
    if (f != 0.0f) {
        r.lse2 = a.lse[n] * kLog2e;
        r.f = f;
        r.label = a.label[n];
        r.dh = 1.0f;
        if (a.dtype == SCAPE_DTYPE_F16 && __builtin_isfinite(f)) {
            int e;
            r.f = frexpf(f, &e) * 32768.0f;
            r.dh = ldexpf(1.0f, e - 15);
        }
    }
    return r;
}
// One workgroup: 8192 rows take 14 us, beside 2.5 ms of products.
__global__ __launch_bounds__(1024) void k_vocab_rows(VocabArgs a) {
    if (threadIdx.x == 0) a.dw_scale[0] = 1.0f;
    for (int64_t n = threadIdx.x; n < a.rows_pad; n += 1024) a.row[n] = row_of(a, n);
}

// The same where fp16 rows go to dw.  Their sum has one power of two, so row n's
// copy of h is h 2^(e - E + 15), e of its factor and E the largest e + x of all
// rows, |h| < 2^x in a row: the largest element of all lies in [2^14, 2^15), and
// every copy is exact down to 2^-14, 2^-28 of that.  Below, its rounding is 2^-25
// at most, in dw |p - onehot| 2^(E-40) a term; 2^E is at most four times the
// largest |factor h|.  (With h against the largest factor alone, the top half of
// the type's range was left unused, and of a row whose factor is 2^20 below it
// 4 of 11 bits.)  A wave a row; each workgroup leaves its largest e + x.
// A reading of h: 8192x2048 15 us.
constexpr int kNoExponent = -10000;
__device__ __forceinline__ int wave_max(int x) {
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) {
        const int o = __shfl_xor(x, d, 64);
        x = o > x ? o : x;
    }
    return x;
}
__global__ __launch_bounds__(kRowThreads) void k_vocab_tops(VocabArgs a) {
    __shared__ int tops[kWaves];
    const uint32_t lane = lane_id(), wave = threadIdx.x >> 6;
    int top = kNoExponent;
    for (int64_t n = (int64_t)blockIdx.x * kWaves + wave; n < a.rows_pad; n += (int64_t)gridDim.x * kWaves) {
        if (lane == 0) a.row[n] = row_of(a, n);
        const float f = n < a.rows ? row_factor(a, n) : 0.0f;
        if (!has_exponent(f)) continue;
        const gran* const from = reinterpret_cast<const gran*>((const char*)a.h + n * a.ld_h * 2);
        int most = 0;  // the bits of the largest finite magnitude
        for (int64_t i = lane; i < a.dim / 8; i += 64) {
            const gran g = from[i];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int bits = (int)(g[j >> 1] >> (16 * (j & 1)) & 0x7fffu);
                most = bits < 0x7c00 && bits > most ? bits : most;
            }
        }
        most = wave_max(most);
        if (most == 0) continue;
        const int x = exponent_of((float)__builtin_bit_cast(_Float16, (uint16_t)most)) + exponent_of(f);
        top = x > top ? x : top;
    }
    if (lane == 0) tops[wave] = top;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < kWaves; ++w) top = tops[w] > top ? tops[w] : top;
        a.top[blockIdx.x] = top;
    }
}

// The rows of h that dw takes: zeros where a row does not count, whatever it
// holds, and times the row's power of two (fp16).  A copy: 8192x2048 14 us (fp16 17).
template <class T, int kThreads>
__device__ __forceinline__ void copy_row(const VocabArgs& a, int64_t n, float c) {
    const gran* from = reinterpret_cast<const gran*>((const char*)a.h + n * a.ld_h * 2);
    gran* to = reinterpret_cast<gran*>((char*)a.h_copy + n * a.dim * 2);
    for (int64_t i = threadIdx.x; i < a.dim / 8; i += kThreads) {
        gran g = gran{0, 0, 0, 0};
        if (c != 0.0f) {
            g = from[i];
            if constexpr (std::is_same<T, F16>::value) {
                float f[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) f[j] = T::up(g, j) * c;
                g = T::down(f);
            }
        }
        to[i] = g;
    }
}
__global__ __launch_bounds__(kRowThreads) void k_vocab_copy(VocabArgs a) {
    copy_row<BF16, kRowThreads>(a, blockIdx.x, a.row[blockIdx.x].f != 0.0f ? 1.0f : 0.0f);
}
template <int kThreads>
__device__ __forceinline__ void copy_scaled(const VocabArgs& a, int64_t n, int32_t tops, int* scratch) {
    int top = kNoExponent;
    for (int32_t i = (int32_t)threadIdx.x; i < tops; i += kThreads) top = a.top[i] > top ? a.top[i] : top;
    top = wave_max(top);
    if ((threadIdx.x & 63u) == 0) scratch[threadIdx.x >> 6] = top;
    __syncthreads();
    for (int w = 0; w < kThreads / 64; ++w) top = scratch[w] > top ? scratch[w] : top;
    const bool none = top == kNoExponent;  // no row has both a factor and a finite element
    if (n == 0 && threadIdx.x == 0) a.dw_scale[0] = none ? 1.0f : ldexpf(1.0f, top - 30);
    const float f = row_factor(a, n);
    int shift = 0;
    if (!none && has_exponent(f)) {
        shift = exponent_of(f) - top + 15;
        // A number becomes 0 far below and a NaN stays one; only a row of zeros or
        // of no numbers, which has no part in E, lies far above.
        shift = shift < -100 ? -100 : shift > 100 ? 100 : shift;
    }
    copy_row<F16, kThreads>(a, n, f != 0.0f ? ldexpf(1.0f, shift) : 0.0f);
}
__global__ __launch_bounds__(kRowThreads) void k_vocab_copy_scaled(VocabArgs a, int32_t tops) {
    __shared__ int scratch[kWaves];
    copy_scaled<kRowThreads>(a, blockIdx.x, tops, scratch);
}
// Few rows: they are copied without a launch for it, bf16 with the rows' factors,
// fp16 by workgroups behind the tiles of the first piece's P (gradient with a
// launch for it and so: 7x50304x1024 68.7 and 65.6 us, 64x32000x2048 100.3 and 98.4).
constexpr int64_t kFewRows = 512;
template <class T>
__global__ __launch_bounds__(kRowThreads) void k_vocab_rows_copy(VocabArgs a) {
    const int64_t n = blockIdx.x;
    const VocabRow r = row_of(a, n);
    if (threadIdx.x == 0) {
        a.row[n] = r;
        if (n == 0) a.dw_scale[0] = 1.0f;
    }
    if constexpr (std::is_same<T, BF16>::value)
        if (a.dw && n < a.rows) copy_row<T, kRowThreads>(a, n, r.f != 0.0f ? 1.0f : 0.0f);
}

// P of a piece of the vocabulary, rounded once to the operands' type: half a
// step of its 8 (bf16) or 11 bits, as each gradient's own rounding is.
// 333x50257x1536 f16 takes 82 us: 394 tiles are two rounds of 256 CUs.
template <class T, int kM, int kN, int kWM, int kWN, int kSlotsA, int kSlotsB>
__global__ __launch_bounds__(kWM * kWN * 64) void k_vocab_p(VocabArgs a, int32_t v0, int32_t v1, uint32_t tiles, int32_t tops) {
    using G = Tile<T, true, true, kM, kN, kWM, kWN, kSlotsA, kSlotsB>;
    __shared__ __attribute__((aligned(16))) char lds[G::kLds];
    if constexpr (std::is_same<T, F16>::value)
        if (blockIdx.x >= tiles) {  // a row of h for dw
            copy_scaled<G::kThreads>(a, blockIdx.x - tiles, tops, reinterpret_cast<int*>(lds));
            return;
        }
    uint32_t tm, tn;
    tile_of(xcd_block(blockIdx.x, tiles), (uint32_t)(v1 - v0 + kM - 1) / kM, a.tiles_n, tm, tn);
    const int32_t m0 = (int32_t)tm * kM, n0 = (int32_t)tn * kN;
    const int32_t lm = m0 + (int32_t)(G::wave_m() + G::lane_m()), left = v1 - v0 - lm;
    const int32_t n1 = n0 + (int32_t)G::wave_n();
    VocabRow r[G::kFN];  // loaded ahead of the products
#pragma unroll
    for (int j = 0; j < G::kFN; ++j) r[j] = a.row[n1 + j * 16 + (int32_t)G::lane_n()];
    G g;
    g.run(Side{(const char*)a.w + v0 * a.ld_w * 2, (int32_t)a.ld_w, v1 - v0, (int32_t)a.dim},
          Side{a.h, (int32_t)a.ld_h, (int32_t)a.rows, (int32_t)a.dim}, m0, n0, 0, (int32_t)a.dim, (lds_t*)lds);
    const bool ragged = v1 - v0 - m0 < kM;
#pragma unroll
    for (int j = 0; j < G::kFN; ++j) {
        const int32_t lab = r[j].label - v0 - lm;  // of the lane's words
        const bool on = r[j].f != 0.0f;            // else the row may hold anything
#pragma unroll
        for (int i = 0; i < G::kFM; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float x = fast_exp2(__builtin_fmaf(g.acc[i][j][e], a.c2, -r[j].lse2));
                g.acc[i][j][e] = on ? x : 0.0f;
            }
        if (on && lab >= 0 && lab < G::kTM && (lab & 15) < 4) {
#pragma unroll
            for (int i = 0; i < G::kFM; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) g.acc[i][j][e] -= lab == i * 16 + e ? 1.0f : 0.0f;
        }
        if (ragged) {
#pragma unroll
            for (int i = 0; i < G::kFM; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (i * 16 + e >= left) g.acc[i][j][e] = 0.0f;
        }
    }
    G::hand_out(
        (lds_t*)lds,
        [&](int i, int j) {
            const f4 p = g.acc[i][j] * r[j].f;
            return u2{T::down2(p[0], p[1]), T::down2(p[2], p[3])};
        },
        [&](uint32_t n, uint32_t m, const gran& q) {
            const int64_t v = m0 + G::wave_m() + m, row = n1 + (int64_t)n;
            const int64_t at = kN >= kDepth ? (v >> 6) * a.block_p + row * kDepth + (v & 63) : row * a.ld_p + v;
            *reinterpret_cast<gran*>((char*)a.p + at * 2) = q;
        });
}

// dw of a piece.  It is stored past the caches, 256 bytes of a row at a time: with
// 64 or 32 at a time, exchanged between the lanes without LDS, the gradient of
// 7x50304x1024 took 82 and 104 us instead of 78.  333x50257x1536 f16 takes 86 us, of
// which the six steps of a tile are half: all CUs multiply and then all write.
// Loading the next tile's operands meanwhile gained nothing (75.4 us for 75.8 then).
template <class T, class G, int kM, int kN>
__device__ __forceinline__ void dw_tile(const VocabArgs& a, const typename G::Slots& slots, uint32_t b, int32_t v0, int32_t v1) {
    const uint32_t nm = (uint32_t)((a.dim + kM - 1) / kM), nn = (uint32_t)(v1 - v0 + kN - 1) / kN;
    uint32_t tm, tn;
    tile_of(b, nm, nn, tm, tn);
    const int32_t m0 = (int32_t)tm * kM, n0 = (int32_t)tn * kN;
    G g;
    g.run(Side{a.h_copy, (int32_t)a.dim, (int32_t)a.dim, (int32_t)a.rows},
          Side{a.p, (int32_t)a.ld_p, (int32_t)a.piece, (int32_t)a.rows_pad, (int32_t)a.block_p}, m0, n0, 0, (int32_t)a.rows, slots);
    const float c = a.dw_scale[0];
    G::hand_out(
        slots.a[0],
        [&](int i, int j) {
            const f4 x = g.acc[i][j] * c;
            return u2{T::down2(x[0], x[1]), T::down2(x[2], x[3])};
        },
        [&](uint32_t n, uint32_t d, const gran& q) {
            const int64_t v = v0 + n0 + (int64_t)(G::wave_n() + n), col = m0 + G::wave_m() + d;
            if (v < v1 && col < a.dim)
                __builtin_nontemporal_store(q, reinterpret_cast<gran*>((char*)a.dw + (v * a.ld_dw + col) * 2));
        });
}

// The slots are objects of their own, so that the compiler knows what is read to
// be none of what is loaded meanwhile (one that is not there is next to nothing).
template <class T, int kM, int kN, int kWM, int kWN>
__global__ __launch_bounds__(kWM * kWN * 64) void k_vocab_dw(VocabArgs a, int32_t v0, int32_t v1) {
    using G = Tile<T, false, false, kM, kN, kWM, kWN, 2, 2, true>;
    __shared__ __attribute__((aligned(16))) char a0[G::A::kBytes], a1[G::A::kBytes], b0[G::B::kBytes], b1[G::B::kBytes];
    const typename G::Slots slots{{(lds_t*)a0, (lds_t*)a1, nullptr}, {(lds_t*)b0, (lds_t*)b1, nullptr}};
    dw_tile<T, G, kM, kN>(a, slots, xcd_block(blockIdx.x, gridDim.x), v0, v1);
}

// dh of a piece: [split][rows][dim] sums in float32, split over the words.
// Where one split sums them all, the last piece's launch writes dh itself.
// kBoth: and dw, for few tokens, eight workgroups of the one (one an XCD) and
// eight of the other in turn: dh reads the head's weights while dw writes as much
// (bf16 us, in two launches and in one: 7x50304x1024 77 and 64, 24x32000x2048 100
// and 87, 64x50304x1024 91 and 73; from 65 tokens on the two take each other's
// caches, 512x32000x2048 212 and 236).
template <class T, int kM, int kN, int kWM, int kWN, int kSlotsA, int kSlotsB, bool kBoth>
__global__ __launch_bounds__(kWM * kWN * 64) void k_vocab_dh(VocabArgs a, int32_t v0, int32_t v1, bool first, bool last, uint32_t n_dh,
                                                             uint32_t n_dw) {
    using G = Tile<T, false, true, kM, kN, kWM, kWN, kSlotsA, kSlotsB, (kN >= kDepth)>;
    __shared__ __attribute__((aligned(16))) char a0[G::A::kBytes], a1[G::A::kBytes], b0[kBoth ? G::A::kBytes : G::B::kBytes], b1[G::B::kBytes];
    __shared__ __attribute__((aligned(16))) char a2[kSlotsA > 2 ? G::A::kBytes : 16], b2[kSlotsB > 2 ? G::B::kBytes : 16];
    const typename G::Slots slots{{(lds_t*)a0, (lds_t*)a1, (lds_t*)a2}, {(lds_t*)b0, (lds_t*)b1, (lds_t*)b2}};
    uint32_t at = blockIdx.x, of_them = gridDim.x;
    if constexpr (kBoth) {
        using W = Tile<T, false, false, kM, kM, 2, 2, 2, 2, (kN >= kDepth)>;
        static_assert(W::kThreads == G::kThreads && W::A::kBytes == G::A::kBytes && W::B::kBytes == G::A::kBytes && kSlotsA == 3, "");
        const uint32_t g = at / kXcds, gh = (n_dh + kXcds - 1) / kXcds, gw = (n_dw + kXcds - 1) / kXcds, both = gh < gw ? gh : gw;
        const bool of_dh = g < 2 * both ? (g & 1) == 0 : gh > gw;
        at = (g < 2 * both ? g / 2 : g - both) * kXcds + at % kXcds;
        of_them = of_dh ? n_dh : n_dw;
        if (at >= of_them) return;
        if (!of_dh) {
            const typename W::Slots w{{(lds_t*)a0, (lds_t*)a1, nullptr}, {(lds_t*)b0, (lds_t*)a2, nullptr}};
            dw_tile<T, W, kM, kM>(a, w, xcd_block(at, of_them), v0, v1);
            return;
        }
    }
    // a split's tiles, which share its words, on one XCD
    const uint32_t b = xcd_block(at, of_them);
    uint32_t tm, tn;
    const uint32_t nm = (uint32_t)((a.dim + kM - 1) / kM), tiles = nm * a.tiles_n;
    const uint32_t split = __builtin_amdgcn_readfirstlane(b / tiles);
    tile_of(b - split * tiles, nm, a.tiles_n, tm, tn);
    const int32_t m0 = (int32_t)tm * kM, n0 = (int32_t)tn * kN;
    const int32_t part = (int32_t)a.split_words, k0 = (int32_t)split * part, all = v1 - v0;
    const int32_t k1 = k0 + part < all ? k0 + part : all;
    if (k0 >= k1 && !first) return;
    G g;
    if (k0 < k1) {
        g.run(Side{(const char*)a.w + v0 * a.ld_w * 2, (int32_t)a.ld_w, (int32_t)a.dim, all},
              Side{a.p, (int32_t)a.ld_p, (int32_t)a.rows_pad, (int32_t)a.piece, (int32_t)a.block_p}, m0, n0, k0, k1, slots);
    } else {
#pragma unroll
        for (int i = 0; i < G::kFM; ++i)
#pragma unroll
            for (int j = 0; j < G::kFN; ++j) g.acc[i][j] = f4{0, 0, 0, 0};
    }
    const int64_t m = m0 + G::wave_m() + G::lane_m(), n1 = n0 + G::wave_n() + G::lane_n();
    if (last && a.splits == 1) {
        G::hand_out(
            slots.a[0],
            [&](int i, int j) {
                const int64_t n = n1 + j * 16;
                f4 x = g.acc[i][j];
                float c = 0.0f;
                if (n < a.rows && m + i * 16 < a.dim) {
                    c = a.row[n].dh;
                    if (!first) x += *reinterpret_cast<const f4*>(a.dh_sum + n * a.dim + m + i * 16);
                }
                x = c != 0.0f ? x * c : f4{0, 0, 0, 0};
                return u2{T::down2(x[0], x[1]), T::down2(x[2], x[3])};
            },
            [&](uint32_t n, uint32_t d, const gran& q) {
                const int64_t row = n0 + G::wave_n() + n, col = m0 + G::wave_m() + d;
                if (row < a.rows && col < a.dim) *reinterpret_cast<gran*>((char*)a.dh + (row * a.ld_dh + col) * 2) = q;
            });
        return;
    }
#pragma unroll
    for (int j = 0; j < G::kFN; ++j) {
        const int64_t n = n1 + j * 16;
        if (n >= a.rows) continue;
        float* const to = a.dh_sum + ((int64_t)split * a.rows + n) * a.dim + m;
#pragma unroll
        for (int i = 0; i < G::kFM; ++i)
            if (m + i * 16 < a.dim) {
                f4* const q = reinterpret_cast<f4*>(to + i * 16);
                *q = first ? g.acc[i][j] : *q + g.acc[i][j];
            }
    }
}

// dh: the splits' sums, times the row's power of two, rounded once (21 splits of
// 333x1536: 8.9 us in a trace, 43 MB at 4.8 TB/s).  A workgroup
// takes 512 elements of a row, each wave a quarter of the splits, in an order
// that the sizes alone decide.
constexpr int kJoinWidth = 512;
template <class T>
__global__ __launch_bounds__(kRowThreads) void k_vocab_dh_join(VocabArgs a) {
    __shared__ f4 part[kWaves][2][64];
    const uint32_t lane = lane_id(), wave = threadIdx.x >> 6, chunks = (uint32_t)((a.dim + kJoinWidth - 1) / kJoinWidth);
    const int64_t n = blockIdx.x / chunks, at = (int64_t)(blockIdx.x % chunks) * kJoinWidth + lane * 8;
    f4 lo = f4{0, 0, 0, 0}, hi = lo;
    if (at < a.dim) {
        const float* p = a.dh_sum + ((int64_t)wave * a.rows + n) * a.dim + at;
#pragma unroll 4
        for (int32_t s = (int32_t)wave; s < a.splits; s += kWaves, p += kWaves * a.rows * a.dim) {
            lo += reinterpret_cast<const f4*>(p)[0];
            hi += reinterpret_cast<const f4*>(p)[1];
        }
    }
    part[wave][0][lane] = lo;
    part[wave][1][lane] = hi;
    __syncthreads();
    if (wave != 0 || at >= a.dim) return;
    for (int w = 1; w < kWaves; ++w) {
        lo += part[w][0][lane];
        hi += part[w][1][lane];
    }
    const float c = a.row[n].dh;
    if (c == 0.0f) lo = hi = f4{0, 0, 0, 0};
    const float f[8] = {lo[0] * c, lo[1] * c, lo[2] * c, lo[3] * c, hi[0] * c, hi[1] * c, hi[2] * c, hi[3] * c};
    *reinterpret_cast<gran*>((char*)a.dh + (n * a.ld_dh + at) * 2) = T::down(f);
}

template <class T>
__global__ __launch_bounds__(kRowThreads) void k_vocab_zero(VocabArgs a) {  // dw of no rows
    gran* to = reinterpret_cast<gran*>((char*)a.dw + (int64_t)blockIdx.x * a.ld_dw * 2);
    for (int64_t i = threadIdx.x; i < a.dim / 8; i += kRowThreads) to[i] = gran{0, 0, 0, 0};
}

#define SCAPE_RUN(kernel, blocks, threads, ...) \
    hipLaunchKernelGGL(HIP_KERNEL_NAME(kernel), dim3((uint32_t)(blocks)), dim3(threads), 0, s, __VA_ARGS__)

// The tiles by the tokens of one (a.tile_n): words or columns of h and w on one
// side, tokens on the other.  Few tokens are a matter of reading w: small tiles,
// so that a CU holds several and every CU has some.  From 129 tokens on the tile
// is as large as two waves a SIMD hold: what a product moves through the caches
// goes with 1 / kM + 1 / kN (8192x32000x2048 bf16, before later steps: loss 837 us
// with 256x256, 1005 with 128x256 and two workgroups a CU).
// The logits' operands are read along their rows and take as many slots as LDS
// holds beside the other workgroups of the CU: w comes from memory, and a tile's
// time for one slot is shorter than its way.
#define SCAPE_LOGITS_BY_TILE(kernel, blocks, ...)                                                          \
    switch (a.tile_n) {                                                                                    \
        case 16: SCAPE_RUN((kernel<T, kSmallWords, 16, 4, 1, 4, 4>), blocks, 256, __VA_ARGS__); break;      \
        case 32: SCAPE_RUN((kernel<T, kSmallWords, 32, 4, 1, 4, 4>), blocks, 256, __VA_ARGS__); break;      \
        case 64: SCAPE_RUN((kernel<T, kSmallWords, 64, 2, 2, 3, 3>), blocks, 256, __VA_ARGS__); break;      \
        case 128: SCAPE_RUN((kernel<T, kSmallWords, 128, 2, 2, 3, 3>), blocks, 256, __VA_ARGS__); break;    \
        case 192: SCAPE_RUN((kernel<T, 256, 192, 2, 4, 3, 2>), blocks, 512, __VA_ARGS__); break;            \
        default: SCAPE_RUN((kernel<T, 256, 256, 2, 4, 3, 2>), blocks, 512, __VA_ARGS__); break;             \
    }
// Both gradients of a piece.
template <class T>
void back_of(hipStream_t s, const VocabArgs& a, int32_t v0, int32_t v1, bool first, bool last) {
    const int64_t across = (a.dim + a.dh_tile - 1) / a.dh_tile;
    const int64_t n_dh = a.dh ? across * a.tiles_n * a.splits : 0;
    const int64_t n_dw = a.dw ? across * ((v1 - v0 + a.dh_tile - 1) / a.dh_tile) : 0;
    const uint32_t nh = (uint32_t)n_dh, nw = (uint32_t)n_dw;
    if (a.tile_n <= 64) {
        const int64_t n = ((n_dh + kXcds - 1) / kXcds + (n_dw + kXcds - 1) / kXcds) * kXcds;
        if (n == 0) return;
        if (a.tile_n == 16) SCAPE_RUN((k_vocab_dh<T, kSmallDims, 16, 4, 1, 3, 3, true>), n, 256, a, v0, v1, first, last, nh, nw);
        else if (a.tile_n == 32) SCAPE_RUN((k_vocab_dh<T, kSmallDims, 32, 4, 1, 3, 3, true>), n, 256, a, v0, v1, first, last, nh, nw);
        else SCAPE_RUN((k_vocab_dh<T, kSmallDims, 64, 2, 2, 3, 3, true>), n, 256, a, v0, v1, first, last, nh, nw);
        return;
    }
    if (n_dh) {
        if (a.tile_n == 128) SCAPE_RUN((k_vocab_dh<T, kSmallDims, 128, 2, 2, 2, 2, false>), n_dh, 256, a, v0, v1, first, last, nh, nw);
        else if (a.tile_n == 192) SCAPE_RUN((k_vocab_dh<T, 256, 192, 2, 4, 3, 2, false>), n_dh, 512, a, v0, v1, first, last, nh, nw);
        else SCAPE_RUN((k_vocab_dh<T, 256, 256, 2, 4, 3, 2, false>), n_dh, 512, a, v0, v1, first, last, nh, nw);
    }
    if (n_dw) {
        if (a.tile_n == 128) SCAPE_RUN((k_vocab_dw<T, kSmallDims, kSmallDims, 2, 2>), n_dw, 256, a, v0, v1);
        else SCAPE_RUN((k_vocab_dw<T, 256, 256, 2, 4>), n_dw, 512, a, v0, v1);
    }
}

template <class T>
hipError_t sums_of(hipStream_t s, const VocabArgs& a) {
    const int64_t tiles = (int64_t)a.tiles_v * a.tiles_n;
    SCAPE_LOGITS_BY_TILE(k_vocab_sums, tiles, a);
    SCAPE_RUN(k_vocab_join, (a.rows + kJoinTokens - 1) / kJoinTokens, kJoinTokens * kJoinParts, a);
    return hipGetLastError();
}

template <class T>
hipError_t grad_of(hipStream_t s, const VocabArgs& a) {
    if (a.rows == 0) {
        if (a.dw) SCAPE_RUN(k_vocab_zero<T>, a.cols, kRowThreads, a);
        return hipGetLastError();
    }
    const int64_t groups = (a.rows_pad + kWaves - 1) / kWaves;
    const int32_t tops = (int32_t)(groups < kVocabTops ? groups : kVocabTops);
    int64_t copies = 0;  // of rows beside the first piece's P
    if (std::is_same<T, F16>::value && a.dw) {
        SCAPE_RUN(k_vocab_tops, tops, kRowThreads, a);
        if (a.rows <= kFewRows) copies = a.rows;
        else SCAPE_RUN(k_vocab_copy_scaled, a.rows, kRowThreads, a, tops);
    } else if (a.rows <= kFewRows) {
        SCAPE_RUN(k_vocab_rows_copy<T>, a.rows_pad, kRowThreads, a);
    } else {
        SCAPE_RUN(k_vocab_rows, 1, 1024, a);
        if (a.dw) SCAPE_RUN(k_vocab_copy, a.rows, kRowThreads, a);
    }
    const int32_t piece = (int32_t)a.piece, cols = (int32_t)a.cols;
    for (int32_t v0 = 0; v0 < cols; v0 += piece) {
        const int32_t v1 = v0 + piece < cols ? v0 + piece : cols;
        const bool first = v0 == 0, last = v1 == cols;
        const int64_t tiles = (int64_t)((v1 - v0 + a.tile_m - 1) / a.tile_m) * a.tiles_n;
        SCAPE_LOGITS_BY_TILE(k_vocab_p, tiles + (first ? copies : 0), a, v0, v1, (uint32_t)tiles, tops);
        back_of<T>(s, a, v0, v1, first, last);
    }
    if (a.dh && a.splits > 1) SCAPE_RUN(k_vocab_dh_join<T>, a.rows * ((a.dim + kJoinWidth - 1) / kJoinWidth), kRowThreads, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_vocab_loss(hipStream_t s, const VocabArgs& a) {
    return a.dtype == SCAPE_DTYPE_BF16 ? sums_of<BF16>(s, a) : sums_of<F16>(s, a);
}

hipError_t launch_vocab_grad(hipStream_t s, const VocabArgs& a) {
    return a.dtype == SCAPE_DTYPE_BF16 ? grad_of<BF16>(s, a) : grad_of<F16>(s, a);
}

}  // namespace scape
