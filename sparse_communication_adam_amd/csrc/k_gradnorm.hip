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

__global__ __launch_bounds__(kBlock) void k_grad_squares(GradArgs a) {
    __shared__ double waves[kWaves];
    const uint32_t tid = threadIdx.x, worker = blockIdx.x % a.workers, tile = blockIdx.x / a.workers;
    if (blockIdx.x == 0 && tid == 0) *a.ticket = 0;  // for the join, which is a launch behind
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

// First tile of the layers from l on.
__device__ __forceinline__ uint32_t first_tile(const GradArgs& a, int32_t l) {
    uint32_t lo = 0, hi = a.n_tiles;
    while (lo < hi) {
        const uint32_t m = (lo + hi) / 2;
        if (a.tiles[m].layer < l) lo = m + 1;
        else hi = m;
    }
    return lo;
}

__device__ __forceinline__ double block_sum_f64(double x, double* waves) {
    x = wave_sum_f64(x);
    if ((threadIdx.x & 63u) == 0) waves[threadIdx.x >> 6] = x;
    __syncthreads();
    x = (waves[0] + waves[1]) + (waves[2] + waves[3]);
    __syncthreads();
    return x;
}

// A layer's tiles, one workgroup each layer and worker; the last workgroup to
// finish sums the layers, in their order.
__global__ __launch_bounds__(kBlock) void k_grad_join(GradArgs a) {
    __shared__ double waves[kWaves];
    __shared__ uint32_t turn;
    const uint32_t tid = threadIdx.x;
    const int32_t layer = (int32_t)(blockIdx.x % a.n_layers);
    const uint32_t worker = blockIdx.x / a.n_layers;
    const uint32_t t0 = first_tile(a, layer), t1 = first_tile(a, layer + 1);
    double x = 0.0;
    for (uint32_t t = t0 + tid; t < t1; t += kBlock) x += a.part[(int64_t)worker * a.n_tiles + t];
    x = block_sum_f64(x, waves);
    if (tid == 0) {
        if (a.layer_norm) a.layer_norm[(int64_t)worker * a.n_layers + layer] = (float)sqrt(x);
        __hip_atomic_store(&a.layer_sum[(int64_t)worker * a.n_layers + layer], x, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        turn = __hip_atomic_fetch_add(a.ticket, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT);
    }
    __syncthreads();
    if (turn != gridDim.x - 1) return;
    double all = 0.0;
    for (uint32_t i = 0; i < a.workers; ++i) {
        x = 0.0;
        for (uint32_t l = tid; l < a.n_layers; l += kBlock)
            x += __hip_atomic_load(&a.layer_sum[(int64_t)i * a.n_layers + l], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        x = block_sum_f64(x, waves);
        all += x;
        if (tid == 0) a.norm[i] = (float)sqrt(x);
    }
    if (tid == 0) a.norm[a.workers] = (float)sqrt(all / (double)a.workers);
}

__global__ __launch_bounds__(kBlock) void k_grad_clip(GradArgs a) {
    const uint32_t tid = threadIdx.x, worker = blockIdx.x % a.workers, tile = blockIdx.x / a.workers;
    const float norm = a.norm[a.shared ? a.workers : worker];
    // One rounding of the factor, one of the product to 8 bits.
    const float f = norm > a.max_norm ? a.max_norm / norm : 1.0f;
    const bool drop = !(norm <= kMaxFloat);  // infinite or NaN
    if (f == 1.0f && !drop && a.out[worker] == a.g[worker]) return;
    const Share s = share_of(a, tile, worker);
    char* const out = reinterpret_cast<char*>(a.out[worker]) + s.at;
    const int32_t whole = s.elements / 8;
    const auto scaled = [&](const gran& g) {
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = drop ? 0.0f : BF16::up(g, j) * f;
        return BF16::down(v);
    };
    gran g[kPerThread];
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
        const int32_t q = i * kBlock + (int32_t)tid;
        if (q < whole)
            g[i] = __builtin_nontemporal_load(reinterpret_cast<const gran*>(s.g + (int64_t)(q >> 3) * s.pitch + (q & 7) * 16));
    }
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
        const int32_t q = i * kBlock + (int32_t)tid;
        if (q < whole)
            __builtin_nontemporal_store(scaled(g[i]), reinterpret_cast<gran*>(out + (int64_t)(q >> 3) * s.pitch + (q & 7) * 16));
    }
    if (tid == 0 && (s.elements & 7)) {  // what lies behind the layer's end stays as it is
        const int64_t at = (int64_t)(whole >> 3) * s.pitch + (whole & 7) * 16;
        const gran last = scaled(*reinterpret_cast<const gran*>(s.g + at));
        uint16_t* const to = reinterpret_cast<uint16_t*>(out + at);
        for (int j = 0; j < (s.elements & 7); ++j) to[j] = (uint16_t)(last[j >> 1] >> (16 * (j & 1)));
    }
}

}  // namespace

hipError_t launch_grad_norm(hipStream_t s, const GradArgs& a) {
    if (a.n_tiles) hipLaunchKernelGGL(k_grad_squares, dim3(a.n_tiles * a.workers), dim3(kBlock), 0, s, a);
    else if (hipError_t e = launch_fill_u32(s, a.ticket, 1, 0)) return e;
    hipLaunchKernelGGL(k_grad_join, dim3(a.n_layers * a.workers), dim3(kBlock), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_grad_clip(hipStream_t s, const GradArgs& a) {
    if (!a.n_tiles) return hipSuccess;
    hipLaunchKernelGGL(k_grad_clip, dim3(a.n_tiles * a.workers), dim3(kBlock), 0, s, a);
    return hipGetLastError();
}

}  // namespace scape
