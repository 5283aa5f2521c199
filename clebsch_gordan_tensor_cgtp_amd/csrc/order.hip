// The lists that the experts' products and gradients go by (gfx950): rows by the pair of their lowest
// experts, slots (row * K + choice) by expert, and each expert's first slot.  Both are stable counting
// sorts over at most 4,097 keys, so every list has one right answer.
//
// A wave counts and places the items of one stretch, in their order: inside 64 items the rank among
// equal keys comes from ballots over the key's bits, so no atomic decides a place (those of the
// counts add integers).
#include <hip/hip_runtime.h>

#include <algorithm>

#include "route.h"

namespace cgtp {

namespace {

// what is sorted: the rows (slots false), or the slots
struct Items {
    const int32_t *experts;
    int64_t N, count;
    int K, E, second, bins;  // bins of the second expert; keys
    bool slots;
};

__device__ __forceinline__ int valid(int e, int E) { return e >= 0 && e < E ? e : E; }

__device__ __forceinline__ int key_of(const Items &s, int64_t i)
{
    if (s.slots) return valid(s.experts[i], s.E);
    int a = s.E, b = s.E;
    for (int j = 0; j < s.K; ++j) {
        const int e = valid(s.experts[i * s.K + j], s.E), high = e > a ? e : a;
        a = e < a ? e : a;
        b = high < b ? high : b;
    }
    if (a == s.E) return s.bins - 1;  // a row without an expert comes last
    if (s.second == 1) return a;
    return a * s.second + (b == s.E ? a : b) * s.second / s.E;
}

// lanes of the wave that hold the same key (those without an item hold -1)
__device__ __forceinline__ unsigned long long same_key(int key, int bits)
{
    unsigned long long m = __ballot(key >= 0);
    for (int b = 0; b < bits; ++b) {
        const unsigned long long set = __ballot((key >> b) & 1);
        m &= (key >> b) & 1 ? set : ~set;
    }
    return m;
}

__device__ __forceinline__ int bits_of(int bins) { return 32 - __clz(bins); }

// exclusive prefix over the wave's lanes
__device__ __forceinline__ int wave_scan(int v, int lane)
{
    int sum = v;
    for (int off = 1; off < 64; off *= 2) {
        const int o = __shfl_up(sum, off);
        sum += lane >= off ? o : 0;
    }
    return sum - v;
}

__global__ void __launch_bounds__(64) count_keys(Items a, Items b, int64_t per_a, int64_t per_b, int32_t *counts_a,
                                                 int32_t *counts_b)
{
    __shared__ int32_t hist[kOrderBins];
    const Items s = blockIdx.y ? b : a;
    const int64_t per = blockIdx.y ? per_b : per_a, lo = blockIdx.x * per, hi = lo + per < s.count ? lo + per : s.count;
    for (int k = threadIdx.x; k < s.bins; k += 64) hist[k] = 0;
    __syncthreads();
    for (int64_t i = lo + threadIdx.x; i < hi; i += 64) atomicAdd(&hist[key_of(s, i)], 1);
    __syncthreads();
    int32_t *out = (blockIdx.y ? counts_b : counts_a) + (int64_t)blockIdx.x * s.bins;
    for (int k = threadIdx.x; k < s.bins; k += 64) out[k] = hist[k];
}

// counts [waves][bins] become, for each key, the items of earlier waves; totals [bins]
__global__ void __launch_bounds__(64) scan_waves(int waves, int bins_a, int bins_b, int32_t *counts_a, int32_t *counts_b)
{
    const int bins = blockIdx.y ? bins_b : bins_a, k = blockIdx.x * 64 + threadIdx.x;
    int32_t *c = blockIdx.y ? counts_b : counts_a;
    if (k >= bins) return;
    int32_t run = 0;
    for (int w0 = 0; w0 < waves; w0 += 16) {
        int32_t v[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = w0 + i < waves ? c[(int64_t)(w0 + i) * bins + k] : 0;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            if (w0 + i < waves) c[(int64_t)(w0 + i) * bins + k] = run;
            run += v[i];
        }
    }
    c[(int64_t)waves * bins + k] = run;
}

__global__ void __launch_bounds__(64) place_items(Items a, Items b, int64_t per_a, int64_t per_b, int waves,
                                                  const int32_t *counts_a, const int32_t *counts_b, int32_t *rows,
                                                  int32_t *slots, int32_t *offsets)
{
    __shared__ int32_t next[kOrderBins];
    const Items s = blockIdx.y ? b : a;
    const int32_t *counts = blockIdx.y ? counts_b : counts_a, *totals = counts + (int64_t)waves * s.bins;
    const int lane = threadIdx.x;
    for (int k = lane; k < s.bins; k += 64) next[k] = totals[k];
    __syncthreads();
    // each lane sums a run of neighbouring keys, then writes their starts
    const int run = (s.bins + 63) / 64, k0 = lane * run, k1 = k0 + run < s.bins ? k0 + run : s.bins;
    int sum = 0;
    for (int k = k0; k < k1; ++k) sum += next[k];
    int start = wave_scan(sum, lane);
    for (int k = k0; k < k1; ++k) {
        const int n = next[k];
        next[k] = start;
        start += n;
    }
    __syncthreads();
    if (s.slots && blockIdx.x == 0)
        for (int k = lane; k < s.bins; k += 64) offsets[k] = next[k];
    for (int k = lane; k < s.bins; k += 64) next[k] += counts[(int64_t)blockIdx.x * s.bins + k];
    __syncthreads();
    const int64_t per = blockIdx.y ? per_b : per_a, lo = blockIdx.x * per, hi = lo + per < s.count ? lo + per : s.count;
    int32_t *out = s.slots ? slots : rows;
    const int bits = bits_of(s.bins);
    for (int64_t i0 = lo; i0 < hi; i0 += 64) {
        const int64_t i = i0 + lane;
        const int key = i < hi ? key_of(s, i) : -1;
        const unsigned long long peers = same_key(key, bits);
        const int rank = __popcll(peers & ((1ull << lane) - 1));
        int at = 0;
        if (key >= 0) at = next[key] + rank;
        __syncthreads();
        if (key >= 0) {
            out[at] = (int32_t)i;
            if (rank == 0) next[key] += __popcll(peers);
        }
        __syncthreads();
    }
}

// Few items: one workgroup counts, scans and places; a wave's counts are 16 bits wide.
__global__ void __launch_bounds__(1024) order_small(Items a, Items b, int32_t *rows, int32_t *slots, int32_t *offsets)
{
    __shared__ uint16_t hist[16 * kOrderBins];
    __shared__ int32_t total[kOrderBins];
    __shared__ int32_t part[16];
    const Items s = blockIdx.x ? b : a;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int per = ((int)s.count + 15) / 16, lo = wave * per, hi = lo + per < s.count ? lo + per : (int)s.count;
    uint16_t *mine = hist + wave * s.bins;
    const int bits = bits_of(s.bins);
    for (int k = threadIdx.x; k < 16 * s.bins; k += 1024) hist[k] = 0;
    __syncthreads();
    for (int i0 = lo; i0 < hi; i0 += 64) {
        const int key = i0 + lane < hi ? key_of(s, i0 + lane) : -1;
        const unsigned long long peers = same_key(key, bits);
        // one lane of each key adds, and the wave's LDS operations keep their order
        if (key >= 0 && (peers & ((1ull << lane) - 1)) == 0) mine[key] += (uint16_t)__popcll(peers);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "workgroup");
        __builtin_amdgcn_wave_barrier();
    }
    __syncthreads();
    // a key's items of earlier waves; the thread's keys are neighbours, so that the scan below is one of threads
    const int run = (s.bins + 1023) / 1024, k0 = threadIdx.x * run, k1 = k0 + run < s.bins ? k0 + run : s.bins;
    int sum = 0;
    for (int k = k0; k < k1; ++k) {
        int before = 0;
        for (int w = 0; w < 16; ++w) {
            const int n = hist[w * s.bins + k];
            hist[w * s.bins + k] = (uint16_t)before;
            before += n;
        }
        total[k] = before;
        sum += before;
    }
    const int inside = wave_scan(sum, lane);
    if (lane == 63) part[wave] = inside + sum;
    __syncthreads();
    int start = inside;
    for (int w = 0; w < wave; ++w) start += part[w];
    for (int k = k0; k < k1; ++k) {
        const int n = total[k];
        total[k] = start;
        if (s.slots) offsets[k] = start;
        start += n;
    }
    __syncthreads();
    int32_t *out = s.slots ? slots : rows;
    for (int i0 = lo; i0 < hi; i0 += 64) {
        const int i = i0 + lane, key = i < hi ? key_of(s, i) : -1;
        const unsigned long long peers = same_key(key, bits);
        const int rank = __popcll(peers & ((1ull << lane) - 1));
        int at = 0;
        if (key >= 0) at = total[key] + mine[key] + rank;
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "workgroup");
        __builtin_amdgcn_wave_barrier();
        if (key >= 0) {
            out[at] = i;
            if (rank == 0) mine[key] += (uint16_t)__popcll(peers);
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "workgroup");
        __builtin_amdgcn_wave_barrier();
    }
}

Items items(const int32_t *experts, int64_t N, int K, int E, bool slots)
{
    Items s{experts, N, slots ? N * K : N, K, E, 1, E + 1, slots};
    if (!slots && K > 1) {
        s.second = std::min(E, (kOrderBins - 1) / E);
        s.bins = E * s.second + 1;
    }
    return s;
}

bool small(int64_t N, int K) { return N * K <= 16384; }

}  // namespace

size_t order_workspace(int64_t N, int K, int E)
{
    if (small(N, K)) return 0;
    const Items a = items(nullptr, N, K, E, false), b = items(nullptr, N, K, E, true);
    return (size_t)(kOrderWaves + 1) * (a.bins + b.bins) * 4;
}

hipError_t launch_order(int64_t N, int K, int E, const int32_t *experts, int32_t *rows, int32_t *slots, int32_t *offsets,
                        void *workspace, hipStream_t st)
{
    const Items a = items(experts, N, K, E, false), b = items(experts, N, K, E, true);
    if (small(N, K)) {
        hipLaunchKernelGGL(order_small, dim3(2), dim3(1024), 0, st, a, b, rows, slots, offsets);
        return hipGetLastError();
    }
    int32_t *ca = static_cast<int32_t *>(workspace), *cb = ca + (size_t)(kOrderWaves + 1) * a.bins;
    const int64_t pa = (a.count + kOrderWaves - 1) / kOrderWaves, pb = (b.count + kOrderWaves - 1) / kOrderWaves;
    hipLaunchKernelGGL(count_keys, dim3(kOrderWaves, 2), dim3(64), 0, st, a, b, pa, pb, ca, cb);
    hipLaunchKernelGGL(scan_waves, dim3((std::max(a.bins, b.bins) + 63) / 64, 2), dim3(64), 0, st, kOrderWaves, a.bins,
                       b.bins, ca, cb);
    hipLaunchKernelGGL(place_items, dim3(kOrderWaves, 2), dim3(64), 0, st, a, b, pa, pb, kOrderWaves, ca, cb, rows,
                       slots, offsets);
    return hipGetLastError();
}

}  // namespace cgtp
