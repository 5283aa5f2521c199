// The lists that the experts' products and gradients go by (gfx950): rows by the pair of their lowest
// experts, slots (row * K + choice) by expert, and each expert's first slot.  Both are stable counting
// sorts over at most 4,097 keys, so every list has one right answer.
//
// A workgroup of 16 waves places one stretch of up to 8,192 items: each wave counts its share per key, the counts
// are summed over the waves and keys, and inside 64 items the rank among equal keys comes from ballots over the key's
// bits, so no atomic decides a place (those of the first launch's counts add integers).  A list of one stretch
// takes one launch, longer ones three: counts, their sums over the stretches, places.
//
// What bounds it is the number of separate writes: 64 lanes writing to 64 places take a wave 0.75 us.  Slots, which have
// few keys, are therefore sorted within the stretch in LDS and written in runs.  (200,000 rows with 6 of 64 experts:
// 1.2 million slots and 200,000 rows.)
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

constexpr int kNone = -2147483647 - 1;  // no item

__device__ __forceinline__ int key_of(const Items &s, int64_t i)
{
    if (s.slots) {
        const int e = s.experts[i];  // checked where it is used, so that its load may be in flight until then
        return e == kNone ? -1 : e;
    }
    int a = s.E, b = s.E;
    for (int j0 = 0; j0 < s.K; j0 += 8) {
        int e[8];  // eight loads in flight
#pragma unroll
        for (int j = 0; j < 8; ++j) e[j] = j0 + j < s.K ? s.experts[i * s.K + j0 + j] : s.E;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int v = valid(e[j], s.E), high = v > a ? v : a;
            a = v < a ? v : a;
            b = high < b ? high : b;
        }
    }
    if (a == s.E) return s.bins - 1;  // a row without an expert comes last
    if (s.second == 1) return a;
    return a * s.second + (b == s.E ? a : b) * s.second / s.E;
}

__device__ __forceinline__ int checked(const Items &s, int key)
{
    return key == kNone ? -1 : s.slots ? valid(key, s.E) : key;
}

// lanes of the wave that hold the same key of BITS bits (those without an item hold -1)
template <int BITS> __device__ __forceinline__ unsigned long long same_key(int key)
{
    unsigned long long m = __ballot(key >= 0);
#pragma unroll
    for (int b = 0; b < BITS; ++b) {
        const int s = (int)((unsigned)key << (31 - b)) >> 31;  // the bit in every place
        m &= ~(__ballot(s != 0) ^ (unsigned long long)(long long)s);
    }
    return m;
}

// Keys of a list have up to 7, 10 or 13 bits: a loop over as many as there are takes three times as long as one unrolled.
#define WITH_BITS(bins, call)      \
    if ((bins) <= 128) {           \
        constexpr int BITS = 7;    \
        call;                      \
    } else if ((bins) <= 1024) {   \
        constexpr int BITS = 10;   \
        call;                      \
    } else {                       \
        constexpr int BITS = 13;   \
        call;                      \
    }

// Between accesses of one wave to its own LDS: they keep their order in the hardware, so the compiler alone has to be
// held to it.  A barrier would wait for the stores to memory as well, about 1 us each time.
__device__ __forceinline__ void keep_order()
{
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

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

// a list, its stretches and their counts
struct List {
    Items s;
    int stretches;
    int64_t per;
    int32_t *counts;  // none of one stretch; [stretches + 1][bins]: a stretch's items of each key, later those of the stretches before it; then all
};

__global__ void __launch_bounds__(1024) count_keys(List a, List b)
{
    __shared__ int32_t hist[kOrderBins];
    const List l = blockIdx.y ? b : a;
    if (l.stretches == 1 || (int)blockIdx.x >= l.stretches) return;
    const int64_t lo = blockIdx.x * l.per, hi = lo + l.per < l.s.count ? lo + l.per : l.s.count;
    int key[kStretch / 1024];
#pragma unroll
    for (int u = 0; u < kStretch / 1024; ++u) {
        const int64_t i = lo + u * 1024 + threadIdx.x;
        key[u] = i < hi ? key_of(l.s, i) : kNone;
    }
    for (int k = threadIdx.x; k < l.s.bins; k += 1024) hist[k] = 0;
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kStretch / 1024; ++u) {
        const int k = checked(l.s, key[u]);
        if (k >= 0) atomicAdd(&hist[k], 1);
    }
    __syncthreads();
    int32_t *out = l.counts + (int64_t)blockIdx.x * l.s.bins;
    for (int k = threadIdx.x; k < l.s.bins; k += 1024) out[k] = hist[k];
}

// KEYS keys of a list; the 1024 / KEYS threads to each sum neighbouring stretches, 16 at a time
template <int KEYS> __device__ __forceinline__ void scan_list(const List &l, int32_t (&part)[1024])
{
    constexpr int SEGS = 1024 / KEYS, AT_ONCE = 16;
    const int bins = l.s.bins, lane = threadIdx.x % KEYS, seg = threadIdx.x / KEYS, k = blockIdx.x * KEYS + lane;
    if (l.stretches == 1 || (int)blockIdx.x * KEYS >= bins) return;
    const int per = (l.stretches + SEGS - 1) / SEGS, w0 = seg * per, w1 = w0 + per < l.stretches ? w0 + per : l.stretches;
    int32_t *c = l.counts + k, v[AT_ONCE], sum = 0;
    for (int w = w0; w < w1; w += AT_ONCE) {
#pragma unroll
        for (int i = 0; i < AT_ONCE; ++i) v[i] = k < bins && w + i < w1 ? c[(int64_t)(w + i) * bins] : 0;
#pragma unroll
        for (int i = 0; i < AT_ONCE; ++i) sum += v[i];
    }
    part[threadIdx.x] = sum;
    __syncthreads();
    if (k >= bins) return;
    int32_t run = 0;
#pragma unroll 8
    for (int i = 0; i < seg; ++i) run += part[i * KEYS + lane];
    if (seg == SEGS - 1) c[(int64_t)l.stretches * bins] = run + sum;
    for (int w = w0; w < w1; w += AT_ONCE) {
        if (per > AT_ONCE) {
#pragma unroll
            for (int i = 0; i < AT_ONCE; ++i) v[i] = w + i < w1 ? c[(int64_t)(w + i) * bins] : 0;
        }
#pragma unroll
        for (int i = 0; i < AT_ONCE; ++i) {
            if (w + i < w1) c[(int64_t)(w + i) * bins] = run;
            run += v[i];
        }
    }
}

// 64 keys of a wide table, whose rows are read in whole cache lines, 16 of a narrow one, for more workgroups
constexpr int kRowKeys = 64, kSlotKeys = 16;

__global__ void __launch_bounds__(1024) scan_stretches(List a, List b)
{
    __shared__ int32_t part[1024];
    if (blockIdx.y)
        scan_list<kSlotKeys>(b, part);
    else
        scan_list<kRowKeys>(a, part);
}

// LDS of a workgroup that places a stretch
struct Stretch {
    union {
        uint16_t hist[16 * (kOrderBins + 1)];  // rows: a wave's counts of each key, then the stretch's before it
        struct {
            uint16_t hist[16 * (kMaxExperts + 2)];
            uint16_t item[kStretch], key[kStretch];  // the stretch's items by key
        } by_key;
    };
    int32_t first[kOrderBins];  // a key's first place: in the list (rows), in the stretch (slots)
    int32_t shift[kMaxExperts + 1];  // slots: from the place in the stretch to that in the list
    int32_t part[16];
};

// sums over threads before this one
__device__ __forceinline__ int group_scan(int v, int32_t (&part)[16])
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, inside = wave_scan(v, lane);
    __syncthreads();
    if (lane == 63) part[wave] = inside + v;
    __syncthreads();
    int start = inside;
#pragma unroll
    for (int w = 0; w < 15; ++w) start += w < wave ? part[w] : 0;
    return start;
}

// One stretch of a list into `out`.  totals [bins] (NULL: the stretch is the list) and before [bins], the items of
// earlier stretches.
template <int BITS, bool SLOTS>
__device__ __forceinline__ void place(const Items &s, int64_t lo, int count, const int32_t *totals, const int32_t *before,
                                      Stretch &l, int32_t *out, int32_t *offsets)
{
    constexpr int STEPS = kStretch / 1024;  // of 64 items to a wave
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, per = (count + 15) / 16;
    const int i0 = wave * per, i1 = i0 + per < count ? i0 + per : count;
    const int pitch = (s.bins + 1) & ~1;  // of a wave's counts, which are added to in pairs
    uint16_t *const hist = SLOTS ? l.by_key.hist : l.hist, *const mine = hist + wave * pitch;
    int key[STEPS];
#pragma unroll
    for (int u = 0; u < STEPS; ++u) key[u] = i0 + u * 64 + lane < i1 ? key_of(s, lo + i0 + u * 64 + lane) : kNone;
    // the thread's keys are neighbours, so that a scan over threads is one over keys
    const int run = (s.bins + 1023) / 1024, k0 = threadIdx.x * run, k1 = k0 + run < s.bins ? k0 + run : s.bins;
    for (int k = threadIdx.x; k < 8 * pitch; k += 1024) reinterpret_cast<uint32_t *>(hist)[k] = 0;
    __syncthreads();
#pragma unroll
    for (int u = 0; u < STEPS; ++u) {
        key[u] = checked(s, key[u]);
        // no count passes 512, so none reaches into its neighbour's bits
        if (key[u] >= 0) atomicAdd(reinterpret_cast<uint32_t *>(mine) + (key[u] >> 1), key[u] & 1 ? 65536u : 1u);
    }
    __syncthreads();
    int sum = 0, all = 0;
    for (int k = k0; k < k1; ++k) {
        int n = 0;
#pragma unroll
        for (int w = 0; w < 16; ++w) {
            const int c = hist[w * pitch + k];
            hist[w * pitch + k] = (uint16_t)n;
            n += c;
        }
        l.first[k] = n;
        sum += n;
        all += totals ? totals[k] : n;
    }
    int at = group_scan(all, l.part), inside = SLOTS ? group_scan(sum, l.part) : 0;
    for (int k = k0; k < k1; ++k) {
        const int n = l.first[k];
        if (SLOTS) {
            if (offsets) offsets[k] = at;
            l.first[k] = inside;
            l.shift[k] = at + (before ? before[k] : 0) - inside;
            inside += n;
        } else {
            l.first[k] = at + (before ? before[k] : 0);
        }
        at += totals ? totals[k] : n;
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < STEPS; ++u) {
        if (i0 + u * 64 >= i1) break;
        const int k = key[u], i = i0 + u * 64 + lane;
        const unsigned long long peers = same_key<BITS>(k);
        const int rank = __popcll(peers & ((1ull << lane) - 1));
        int place = 0;
        if (k >= 0) place = l.first[k] + mine[k] + rank;
        keep_order();
        if (k >= 0) {
            if (SLOTS) {
                l.by_key.item[place] = (uint16_t)i;
                l.by_key.key[place] = (uint16_t)k;
            } else {
                out[place] = (int32_t)(lo + i);
            }
            if (rank == 0) mine[k] += (uint16_t)__popcll(peers);
        }
        keep_order();
    }
    if (SLOTS) {
        __syncthreads();
        for (int p = threadIdx.x; p < count; p += 1024) out[p + l.shift[l.by_key.key[p]]] = (int32_t)(lo + l.by_key.item[p]);
    }
}

__global__ void __launch_bounds__(1024) place_items(List a, List b, int32_t *rows, int32_t *slots, int32_t *offsets)
{
    __shared__ Stretch l;
    const List q = blockIdx.y ? b : a;
    const int w = blockIdx.x;
    if (w >= q.stretches) return;
    const int64_t lo = w * q.per;
    const int count = (int)(lo + q.per < q.s.count ? q.per : lo < q.s.count ? q.s.count - lo : 0);
    const int32_t *totals = q.stretches > 1 ? q.counts + (int64_t)q.stretches * q.s.bins : nullptr;
    const int32_t *before = q.stretches > 1 ? q.counts + (int64_t)w * q.s.bins : nullptr;
    if (blockIdx.y) {
        WITH_BITS(q.s.bins, (place<BITS, true>(q.s, lo, count, totals, before, l, slots, w == 0 ? offsets : nullptr)))
    } else {
        WITH_BITS(q.s.bins, (place<BITS, false>(q.s, lo, count, totals, before, l, rows, nullptr)))
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

// A workgroup takes nearly all LDS of a CU, so the two lists have 80 and 160 of them, at most one for each of the
// 256 CUs, and more where stretches would be too long (20,000 rows with 2 of 8 experts, in 253 and 255 stretches: 11 us).
List list_of(const Items &s, int32_t *counts)
{
    List l{s, 1, s.count, counts};
    if (s.count > kStretch) {
        const int most = s.slots ? 160 : 80;
        l.per = std::min<int64_t>(kStretch, std::max<int64_t>(1024, (s.count + most - 1) / most));
        l.stretches = (int)((s.count + l.per - 1) / l.per);
    }
    return l;
}

size_t table_bytes(const List &l) { return l.stretches > 1 ? (size_t)(l.stretches + 1) * l.s.bins * 4 : 0; }

}  // namespace

size_t order_workspace(int64_t N, int K, int E)
{
    return table_bytes(list_of(items(nullptr, N, K, E, false), nullptr)) + table_bytes(list_of(items(nullptr, N, K, E, true), nullptr));
}

hipError_t launch_order(int64_t N, int K, int E, const int32_t *experts, int32_t *rows, int32_t *slots, int32_t *offsets,
                        void *workspace, hipStream_t st)
{
    List a = list_of(items(experts, N, K, E, false), static_cast<int32_t *>(workspace));
    List b = list_of(items(experts, N, K, E, true), static_cast<int32_t *>(workspace));
    b.counts += table_bytes(a) / 4;
    const dim3 grid(std::max(a.stretches, b.stretches), 2);
    if (grid.x > 1) {
        hipLaunchKernelGGL(count_keys, grid, dim3(1024), 0, st, a, b);
        hipLaunchKernelGGL(scan_stretches, dim3(std::max((a.s.bins + kRowKeys - 1) / kRowKeys, (b.s.bins + kSlotKeys - 1) / kSlotKeys), 2),
                           dim3(1024), 0, st, a, b);
    }
    hipLaunchKernelGGL(place_items, grid, dim3(1024), 0, st, a, b, rows, slots, offsets);
    return hipGetLastError();
}

}  // namespace cgtp
