// k_gradnorm.hip - the workers' gradient norms over all layers, and the
// gradients clipped by them, in a context's layout.
//
//   norm_i = sqrt(sum_l sum_j g_i[j]^2), norm_W = sqrt(mean_i norm_i^2)
//   out = f g, f = max_norm / norm where norm > max_norm, 0 where it is not finite
//
// Both read every gradient once (2 bytes an element) and are bound by that.
// Squares are summed in float64: no square of a bf16 leaves its range, and the
// sums of 2^31 of them keep more bits than the norm's own type has.
#include "loss_device.h"

namespace scape {

namespace {

// A workgroup's share: one tile of one worker, its elements inside the layer.
struct Share {
    const char* g;     // first byte of the tile's first word of this worker
    int64_t at;        // and its offset from the worker's first
    uint32_t pitch;    // bytes from a word to the next
    int32_t elements;  // of the tile that are inside the layer (kTileWords * 64 at most)
};
__device__ __forceinline__ Share share_of(const GradArgs& a, uint32_t tile, uint32_t worker) {
    const TileDesc t = a.tiles[tile];
    const LayerDesc l = a.layers[t.layer];
    Share s;
    s.pitch = a.ws * 2;
    s.at = (int64_t)t.w0 * s.pitch;
    s.g = reinterpret_cast<const char*>(a.g[worker]) + s.at;
    const uint32_t end = l.off + l.n, stop = t.w1 * 64 < end ? t.w1 * 64 : end;
    s.elements = (int32_t)(stop - t.w0 * 64);
    return s;
}

constexpr int kTileGranules = kTileWords * 8, kPerThread = kTileGranules / kBlock;

// A workgroup a tile of a worker, 16 bytes a load, all of a thread's on their way.
// Bound by the read: two workers of 355M elements 203 us in a trace, 7.0 TB/s.
__global__ __launch_bounds__(kBlock) void k_grad_squares(GradArgs a) {
    __shared__ double waves[kWaves];
    const uint32_t tid = threadIdx.x, b = xcd_block(blockIdx.x, gridDim.x);
    const uint32_t worker = b % a.workers, tile = b / a.workers;
    const Share s = share_of(a, tile, worker);
    const int32_t whole = s.elements / 8;
    double sum[2] = {0.0, 0.0};
    const auto add = [&](const gran& g, int count) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const double x = j < count ? (double)BF16::up(g, j) : 0.0;
            sum[j & 1] = __builtin_fma(x, x, sum[j & 1]);
        }
    };
    gran g[kPerThread];
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
        const int32_t q = i * kBlock + (int32_t)tid;
        g[i] = gran{0, 0, 0, 0};
        if (q < whole)
            g[i] = __builtin_nontemporal_load(reinterpret_cast<const gran*>(s.g + (int64_t)(q >> 3) * s.pitch + (q & 7) * 16));
    }
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) add(g[i], 8);
    if (tid == 0 && (s.elements & 7)) {
        const gran last = *reinterpret_cast<const gran*>(s.g + (int64_t)(whole >> 3) * s.pitch + (whole & 7) * 16);
        add(last, s.elements & 7);
    }
    const double w = wave_sum_f64(sum[0] + sum[1]);
    if ((tid & 63u) == 0) waves[tid >> 6] = w;
    __syncthreads();
    if (tid == 0) a.part[(int64_t)worker * a.n_tiles + tile] = (waves[0] + waves[1]) + (waves[2] + waves[3]);
}

// A layer's tiles, a wave each layer and worker in turn.
__device__ __forceinline__ void join_layers(const GradArgs& a, uint32_t wave, uint32_t waves) {
    const uint32_t lane = lane_id(), layers = a.n_layers * a.workers;
    for (uint32_t i = wave; i < layers; i += waves) {
        const uint32_t worker = i / a.n_layers, layer = i - worker * a.n_layers;
        const uint32_t t0 = a.layer_tile0[layer], t1 = a.layer_tile0[layer + 1];
        double x = 0.0;
#pragma unroll 16
        for (uint32_t t = t0 + lane; t < t1; t += 64) x += a.part[(int64_t)worker * a.n_tiles + t];
        x = wave_sum_f64(x);
        if (lane == 0) {
            if (a.layer_norm) a.layer_norm[i] = (float)sqrt(x);
            a.layer_sum[i] = x;
        }
    }
}
// The layers of a worker, in their order, by a wave each; then the workers.
__device__ __forceinline__ void join_workers(const GradArgs& a, uint32_t wave, uint32_t waves) {
    __shared__ double sums[SCAPE_MAX_WORKERS];
    const uint32_t lane = lane_id();
    for (uint32_t i = wave; i < a.workers; i += waves) {
        double x = 0.0;
#pragma unroll 8
        for (uint32_t l = lane; l < a.n_layers; l += 64) x += a.layer_sum[i * a.n_layers + l];
        x = wave_sum_f64(x);
        if (lane == 0) {
            a.norm[i] = (float)sqrt(x);
            sums[i] = x;
        }
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        double all = 0.0;
        for (uint32_t i = 0; i < a.workers; ++i) all += sums[i];
        a.norm[a.workers] = (float)sqrt(all / (double)a.workers);
    }
}
// Few layers: one workgroup joins all.  Else a launch for the layers and one for
// the workers: a ticket that the last workgroup finds would have to be ordered
// behind the others' sums across the XCDs' caches, which takes longer than a
// launch (2x292 layers 12-17 us, in two launches 10.2 in a trace).
constexpr int kJoinThreads = 1024, kJoinWaves = kJoinThreads / 64;
__global__ __launch_bounds__(kJoinThreads) void k_grad_join(GradArgs a) {
    join_layers(a, threadIdx.x >> 6, kJoinWaves);
    __syncthreads();
    join_workers(a, threadIdx.x >> 6, kJoinWaves);
}
__global__ __launch_bounds__(kBlock) void k_grad_layers(GradArgs a) {
    join_layers(a, blockIdx.x * kWaves + (threadIdx.x >> 6), gridDim.x * kWaves);
}
__global__ __launch_bounds__(kJoinThreads) void k_grad_workers(GradArgs a) {
    join_workers(a, threadIdx.x >> 6, kJoinWaves);
}

// 16 bytes a thread, as a plain copy does best (two workers of 355M elements in a
// trace: 497 us with four a thread, 460 so, 6.2 TB/s; bound by read and write).
constexpr int kClipParts = kPerThread;
__global__ __launch_bounds__(kBlock) void k_grad_clip(GradArgs a) {
    const uint32_t tid = threadIdx.x, b = xcd_block(blockIdx.x, gridDim.x), part = b % kClipParts, c = b / kClipParts;
    const uint32_t worker = c % a.workers, tile = c / a.workers;
    const float norm = a.norm[a.shared ? a.workers : worker];
    // One rounding of the factor, one of the product to 8 bits.
    const float f = norm > a.max_norm ? a.max_norm / norm : 1.0f;
    const bool drop = !(norm <= kMaxFloat);  // infinite or NaN
    if (f == 1.0f && !drop && a.out[worker] == a.g[worker]) return;
    const Share s = share_of(a, tile, worker);
    const int32_t q = (int32_t)(part * kBlock + tid), whole = s.elements / 8, rest = s.elements - q * 8;
    if (q > whole || rest <= 0) return;
    const int64_t at = (int64_t)(q >> 3) * s.pitch + (q & 7) * 16;
    const gran* const from = reinterpret_cast<const gran*>(s.g + at);
    gran* const to = reinterpret_cast<gran*>(reinterpret_cast<char*>(a.out[worker]) + s.at + at);
    const gran g = __builtin_nontemporal_load(from);
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = drop ? 0.0f : BF16::up(g, j) * f;
    const gran r = BF16::down(v);
    if (q < whole) {
        __builtin_nontemporal_store(r, to);
    } else {  // what lies behind the layer's end stays as it is
        uint16_t* const last = reinterpret_cast<uint16_t*>(to);
        for (int j = 0; j < rest; ++j) last[j] = (uint16_t)(r[j >> 1] >> (16 * (j & 1)));
    }
}

}  // namespace

hipError_t launch_grad_norm(hipStream_t s, const GradArgs& a) {
    if (a.n_tiles) hipLaunchKernelGGL(k_grad_squares, dim3(a.n_tiles * a.workers), dim3(kBlock), 0, s, a);
    const uint32_t layers = a.n_layers * a.workers;
    if (layers <= 4 * kJoinWaves) {
        hipLaunchKernelGGL(k_grad_join, dim3(1), dim3(kJoinThreads), 0, s, a);
    } else {
        const uint32_t n = (layers + kWaves - 1) / kWaves;
        hipLaunchKernelGGL(k_grad_layers, dim3(n < 65536 ? n : 65536), dim3(kBlock), 0, s, a);
        hipLaunchKernelGGL(k_grad_workers, dim3(1), dim3(kJoinThreads), 0, s, a);
    }
    return hipGetLastError();
}

hipError_t launch_grad_clip(hipStream_t s, const GradArgs& a) {
    if (!a.n_tiles) return hipSuccess;
    hipLaunchKernelGGL(k_grad_clip, dim3(a.n_tiles * a.workers * kClipParts), dim3(kBlock), 0, s, a);
    return hipGetLastError();
}

}  // namespace scape
