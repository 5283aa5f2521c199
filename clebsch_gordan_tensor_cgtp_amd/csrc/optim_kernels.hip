// The AdamW step over many tensors, its 8-bit moments, and the gradient's global norm (gfx950).
//
// With f the clipping factor and g = f grad:
//   m <- b1 m + (1 - b1) g,   v <- b2 v + (1 - b2) g^2,
//   p <- p (1 - lr wd) - (lr / (1 - b1^t)) m / (sqrt(v) / sqrt(1 - b2^t) + eps).
//
// One workgroup takes one unit of 2048 elements of one tensor; it finds the tensor by comparing
// its number with the table's unit starts, one per lane.  The table is a kernel argument, so
// nothing about the tensors is kept from one call for the next, and a captured graph replays the
// pointers it was captured with.
//
// 8-bit moments.  A block of 64 values shares a float scale, its largest magnitude a; a value x
// is held as the code round(c sqrt(|x| / a)), which stands for a (code / c)^2.  The first
// moment has c = 127 and a sign; of the second its root s = sqrt(v) is held, c = 255, and a
// nonzero s never gets the code 0: rounded down it would leave eps alone under a first moment
// that is not 0.  Near the largest value the step is 2 / c of it (0.8% of s), and the smallest code
// stands for a / 65025, so that v spans nine decades within a block.  The scale is a float
// and not a power of two: s decays by sqrt(b2) a step, far less than half a code's step, and a block
// whose gradients have ceased would otherwise stay where it is.
//
// Products and sums are rounded one by one (no contraction), so that a code does not depend on
// which of them the compiler fuses.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "optim.h"

#pragma clang fp contract(off)

namespace cgtp {

namespace {

template <Elem E> struct Types;
template <> struct Types<Elem::f32> { typedef float T; typedef float R; };
template <> struct Types<Elem::f64> { typedef double T; typedef double R; };
template <> struct Types<Elem::bf16> { typedef __bf16 T; typedef float R; };
template <> struct Types<Elem::f16> { typedef _Float16 T; typedef float R; };

template <typename S, int N> struct VecOf { typedef S type __attribute__((ext_vector_type(N), aligned(sizeof(S)))); };

// n of the N values at p; the others are 0
template <int N, typename S, typename R> __device__ __forceinline__ void load_some(const S *p, int64_t n, R (&x)[N])
{
    typedef typename VecOf<S, N>::type V;
    if (n >= N) {
        const V r = *reinterpret_cast<const V *>(p);
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = (R)r[i];
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = i < n ? (R)p[i] : (R)0;
    }
}

template <int N, typename S, typename R> __device__ __forceinline__ void store_some(S *p, int64_t n, const R (&x)[N])
{
    typedef typename VecOf<S, N>::type V;
    if (n >= N) {
        V r;
#pragma unroll
        for (int i = 0; i < N; ++i) r[i] = (S)x[i];
        __builtin_nontemporal_store(r, reinterpret_cast<V *>(p));
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i < n) p[i] = (S)x[i];
    }
}

template <bool ONCE = false, int N, typename S, typename R>
__device__ __forceinline__ void load_vec(const S *p, R (&x)[N])
{
    typedef S V __attribute__((ext_vector_type(N)));
    const V *at = reinterpret_cast<const V *>(p);
    const V r = ONCE ? __builtin_nontemporal_load(at) : *at;
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = (R)r[i];
}

template <int N, typename S, typename R> __device__ __forceinline__ void store_vec(S *p, const R (&x)[N])
{
    typedef S V __attribute__((ext_vector_type(N)));
    V r;
#pragma unroll
    for (int i = 0; i < N; ++i) r[i] = (S)x[i];
    __builtin_nontemporal_store(r, reinterpret_cast<V *>(p));
}

// the table's tensor that unit `u` of the launch belongs to
__device__ __forceinline__ int tensor_of(const TensorTable &t, int u)
{
    const int lane = threadIdx.x & 63;
    int at = 0;
#pragma unroll
    for (int k = 0; k < kTableTensors; k += 64) {
        const int i = k + lane;
        const bool before = i < kTableTensors && i < t.n && t.unit[i < kTableTensors ? i : 0] <= u;
        at += __popcll(__ballot(before));
    }
    return __builtin_amdgcn_readfirstlane(at - 1);
}

// ------------------------------------------------------------------------------------------
// 8-bit codes

template <int CTRL> __device__ __forceinline__ unsigned dpp_max(unsigned v)
{
    return max(v, (unsigned)__builtin_amdgcn_mov_dpp((int)v, CTRL, 15, 15, false));
}

// Largest magnitude of the values of `LANES` neighbouring lanes, NaN where one of them is not finite:
// the scale is NaN then, the codes are 0 and the block reads as NaN.  (An infinite scale would not do: a
// second moment's codes above 0 would read as infinite, and their weights stop without a sign.)
// Compared as bit patterns, in which an infinity is above every number and a NaN above that.
template <int LANES, int N> __device__ __forceinline__ float block_most(const float (&x)[N])
{
    unsigned most = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) most = max(most, __float_as_uint(x[i]) & 0x7fffffffu);
    static_assert(LANES == 8 || LANES == 16, "a block is 8 or 16 lanes");
    most = dpp_max<0xB1>(most);   // quad_perm 1,0,3,2
    most = dpp_max<0x4E>(most);   // quad_perm 2,3,0,1
    most = dpp_max<0x141>(most);  // row_half_mirror
    if (LANES == 16) most = dpp_max<0x140>(most);  // row_mirror
    if (most >= 0x7f800000u) return __builtin_nanf("");
    const float a = __uint_as_float(most);
    return a < 1.17549435e-38f ? 0.0f : a;  // below it 1 / a is infinite
}

// Codes of N values.  The code is defined by the correctly rounded root; the hardware's is off by up to a
// step of its last bit, which matters only where the scaled root lies next to the middle between two
// codes (255 times 1.5 steps of 2^-24, and a rounding of the product: 4e-5): a wave in which any
// does takes the exact root.  About one wave in ten does; the exact root everywhere is 16 instructions more a
// code, of some 75 an element.
template <bool SIGNED, int N> __device__ __forceinline__ void codes_of(const float (&x)[N], float most, float (&q)[N])
{
    constexpr float top = SIGNED ? 127.0f : 255.0f;
    const float inv = most > 0.0f ? 1.0f / most : 0.0f;
    float middle = 0.0f;
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const float t = __builtin_amdgcn_sqrtf(fabsf(x[j]) * inv) * top;
        q[j] = rintf(t);
        middle = fmaxf(middle, fabsf(t - q[j]));
    }
    if (__any(middle > 0.5f - 6e-5f)) {
#pragma unroll
        for (int j = 0; j < N; ++j) q[j] = rintf(__builtin_sqrtf(fabsf(x[j]) * inv) * top);
    }
#pragma unroll
    for (int j = 0; j < N; ++j) {
        // NaN becomes 0: the block's scale is NaN then
        q[j] = fminf(fmaxf(q[j], !SIGNED && x[j] > 0.0f && most > 0.0f ? 1.0f : 0.0f), top);
        if (SIGNED && x[j] < 0.0f) q[j] = -q[j];
    }
}

template <bool SIGNED> __device__ __forceinline__ float value_of(float code, float most)
{
    const float t = code * (1.0f / (SIGNED ? 127.0f : 255.0f));
    return (SIGNED ? t * fabsf(t) : t * t) * most;
}

// ------------------------------------------------------------------------------------------
// the step

// What decides whether a step is taken, for the step and for the schedule that counts it.
__device__ __forceinline__ double scaled_norm(const double *norm, double grad_scale) { return fabs(grad_scale) * *norm; }
__device__ __forceinline__ bool is_finite(double n) { return fabs(n) < __builtin_inf(); }

// Bounded by HBM: 28 bytes an element in 32 bits, 16.25 in 8 bits (f32 tensors).  What is read and
// written once bypasses the last-level cache, and the units are taken from the last one down, so that of
// the gradients, which the norm has just read from the first one up, the end is still there: 111.6M f32
// weights with clipping, moments in 32 bits 692 -> 635 us, in 8 bits (decoded too) 671 -> 648 us.  A lane
// takes as many elements as make 16 bytes of the widest of the buffers, so that each load of a wave
// covers whole cache lines, which loads past the cache need (62.5M bf16 weights with copies, no
// clipping, 433 -> 385 us).  In 8 bits the arithmetic weighs as much as the memory; with the hardware's
// roots and reciprocals (codes_of; for the quotient an error of 2^-23 of a step that is itself a
// thousandth of the weight) 648 -> 602 us.
template <Elem E, bool CODES, bool MASTER>
__global__ void __launch_bounds__(256) adamw_kernel(const TensorTable t, const MomentBuffers mb, const StepScalars s,
                                                    const double *norm, const double *schedule)
{
    typedef typename Types<E>::T T;
    typedef typename Types<E>::R R;
    constexpr int N = 16 / (CODES && !MASTER ? sizeof(T) : sizeof(R));
    constexpr int PASSES = kUnit / (256 * N);
    static_assert(PASSES >= 1 && PASSES * 256 * N == kUnit, "a unit is whole passes of the workgroup");

    double factor = s.grad_scale;
    if (norm) {
        const double n = scaled_norm(norm, s.grad_scale);
        if (!is_finite(n)) return;  // a gradient is not finite: nothing is changed
        if (s.max_norm > 0 && n > s.max_norm) factor *= s.max_norm / n;
    }
    double lr = s.lr, bias1 = s.bias1, bias2 = s.bias2;
    if (schedule) {
        lr = schedule[1];
        bias1 = schedule[2];
        bias2 = schedule[3];
    }
    const R f = (R)factor, b1 = (R)s.beta1, c1 = (R)(1 - s.beta1), b2 = (R)s.beta2, c2 = (R)(1 - s.beta2);
    const R keep = (R)(1 - lr * s.weight_decay), rate = (R)(lr / bias1), root = (R)(1 / __builtin_sqrt(bias2));
    const R eps = (R)s.eps;

    const int u = t.unit[t.n] - 1 - (int)blockIdx.x;
    const int i = tensor_of(t, u);
    const int64_t first = (int64_t)(u - t.unit[i]) * kUnit;                 // in the tensor
    const int64_t base = ((int64_t)t.state[i] + (u - t.unit[i])) * kUnit;  // in the moments
    const int64_t left = t.numel[i] - first;
    T *param = static_cast<T *>(t.param[i]) + first;
    const T *grad = static_cast<const T *>(t.grad[i]) + first;

    R p[PASSES][N], g[PASSES][N], m[PASSES][N], v[PASSES][N];
    float am[PASSES], as[PASSES];
#pragma unroll
    for (int k = 0; k < PASSES; ++k) {
        const int at = (k * 256 + (int)threadIdx.x) * N;
        load_some(grad + at, left - at, g[k]);
        if constexpr (MASTER)
            load_vec<true>(static_cast<const float *>(mb.master) + base + at, p[k]);
        else
            load_some(param + at, left - at, p[k]);
        if constexpr (CODES) {
            load_vec(static_cast<const signed char *>(mb.m) + base + at, m[k]);
            load_vec(static_cast<const unsigned char *>(mb.v) + base + at, v[k]);
            am[k] = mb.scales[(base + at) / kScaleBlock];
            as[k] = mb.scales[mb.blocks + (base + at) / kScaleBlock];
        } else {
            load_vec<true>(static_cast<const R *>(mb.m) + base + at, m[k]);
            load_vec<true>(static_cast<const R *>(mb.v) + base + at, v[k]);
        }
    }
#pragma unroll
    for (int k = 0; k < PASSES; ++k) {
        const int at = (k * 256 + (int)threadIdx.x) * N;
        R sv[N];
#pragma unroll
        for (int j = 0; j < N; ++j) {
            if constexpr (CODES) {
                m[k][j] = value_of<true>(m[k][j], am[k]);
                const float old = value_of<false>(v[k][j], as[k]);
                v[k][j] = old * old;
            }
            const R gj = g[k][j] * f;
            m[k][j] = m[k][j] * b1 + gj * c1;
            v[k][j] = v[k][j] * b2 + gj * gj * c2;
            if constexpr (sizeof(R) == 8)
                sv[j] = __builtin_sqrt(v[k][j]);
            else
                sv[j] = __builtin_sqrtf(v[k][j]);
            p[k][j] = p[k][j] * keep;
            if constexpr (CODES)
                p[k][j] = p[k][j] - m[k][j] * rate * __builtin_amdgcn_rcpf(sv[j] * root + eps);
            else
                p[k][j] = p[k][j] - m[k][j] * rate / (sv[j] * root + eps);
        }
        if constexpr (MASTER) store_vec(static_cast<float *>(mb.master) + base + at, p[k]);
        store_some(param + at, left - at, p[k]);
        if constexpr (CODES) {
            constexpr int LANES = kScaleBlock / N;
            const float mm = block_most<LANES>(m[k]), ms = block_most<LANES>(sv);
            float cm[N], cs[N];
            codes_of<true>(m[k], mm, cm);
            codes_of<false>(sv, ms, cs);
            store_vec(static_cast<signed char *>(mb.m) + base + at, cm);
            store_vec(static_cast<unsigned char *>(mb.v) + base + at, cs);
            if (threadIdx.x % LANES == 0) {
                mb.scales[(base + at) / kScaleBlock] = mm;
                mb.scales[mb.blocks + (base + at) / kScaleBlock] = ms;
            }
        } else {
            store_vec(static_cast<R *>(mb.m) + base + at, m[k]);
            store_vec(static_cast<R *>(mb.v) + base + at, v[k]);
        }
    }
}

// ------------------------------------------------------------------------------------------
// the gradient's norm: squares and sums in double, in a fixed order

__device__ __forceinline__ double wave_total(double x)
{
#pragma unroll
    for (int k = 32; k >= 1; k /= 2) x += __shfl_xor(x, k);
    return x;
}

template <int THREADS> __device__ __forceinline__ double group_total(double x)
{
    __shared__ double part[THREADS / 64];
    x = wave_total(x);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = x;
    __syncthreads();
    x = 0;
    for (int w = 0; w < THREADS / 64; ++w) x += part[w];
    return x;
}

template <Elem E> __global__ void __launch_bounds__(256) square_sums_kernel(const TensorTable t, double *partial)
{
    typedef typename Types<E>::T T;
    constexpr int N = 16 / sizeof(T);
    constexpr int PASSES = kUnit / (256 * N);
    double sum = 0;
    const int units = t.unit[t.n];
    for (int u = (int)blockIdx.x; u < units; u += (int)gridDim.x) {
        const int i = tensor_of(t, u);
        const int64_t first = (int64_t)(u - t.unit[i]) * kUnit, left = t.numel[i] - first;
        const T *grad = static_cast<const T *>(t.grad[i]) + first;
        double g[PASSES][N];
#pragma unroll
        for (int k = 0; k < PASSES; ++k) {
            const int at = (k * 256 + (int)threadIdx.x) * N;
            load_some(grad + at, left - at, g[k]);
        }
#pragma unroll
        for (int k = 0; k < PASSES; ++k)
#pragma unroll
            for (int j = 0; j < N; ++j) sum += g[k][j] * g[k][j];
    }
    sum = group_total<256>(sum);
    if (threadIdx.x == 0) partial[blockIdx.x] = sum;
}

__global__ void __launch_bounds__(1024) norm_kernel(const double *partial, int64_t n, double *norm)
{
    double s = 0;
    for (int64_t i = threadIdx.x; i < n; i += 1024) s += partial[i];
    s = group_total<1024>(s);
    if (threadIdx.x == 0) *norm = __builtin_sqrt(s);
}

// ------------------------------------------------------------------------------------------
// 8-bit moments to and from single precision

__global__ void __launch_bounds__(256) state_read_kernel(const signed char *m, const unsigned char *v,
                                                         const float *scales, int64_t elements, float *m_out,
                                                         float *v_out)
{
    for (int64_t at = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4; at < elements; at += (int64_t)gridDim.x * 1024) {
        const float am = scales[at / kScaleBlock], as = scales[(elements + at) / kScaleBlock];
        float x[4];
        if (m_out) {
            load_vec(m + at, x);
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] = value_of<true>(x[j], am);
            store_vec(m_out + at, x);
        }
        if (v_out) {
            load_vec(v + at, x);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float s = value_of<false>(x[j], as);
                x[j] = s * s;
            }
            store_vec(v_out + at, x);
        }
    }
}

// elements is a multiple of a unit, so every lane of a block's 16 is in range or none
__global__ void __launch_bounds__(256) state_write_kernel(const float *m_in, const float *v_in, int64_t elements,
                                                          signed char *m, unsigned char *v, float *scales)
{
    for (int64_t at = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4; at < elements; at += (int64_t)gridDim.x * 1024) {
        float x[4], c[4];
        load_vec(m_in + at, x);
        float most = block_most<16>(x);
        codes_of<true>(x, most, c);
        store_vec(m + at, c);
        if (threadIdx.x % 16 == 0) scales[at / kScaleBlock] = most;
        load_vec(v_in + at, x);
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = __builtin_sqrtf(x[j]);
        most = block_most<16>(x);
        codes_of<false>(x, most, c);
        store_vec(v + at, c);
        if (threadIdx.x % 16 == 0) scales[(elements + at) / kScaleBlock] = most;
    }
}

// {step, lr, 1 - b1^step, 1 - b2^step}: one more step, if it is one that the moments take
__global__ void schedule_kernel(double *schedule, double beta1, double beta2, const double *norm, double grad_scale)
{
    if (threadIdx.x != 0) return;
    if (norm && !is_finite(scaled_norm(norm, grad_scale))) return;
    const double step = schedule[0] + 1;
    schedule[0] = step;
    schedule[2] = 1 - pow(beta1, step);
    schedule[3] = 1 - pow(beta2, step);
}

template <Elem E>
hipError_t launch_adamw_as(bool codes, const TensorTable &t, const MomentBuffers &mb, const StepScalars &s,
                           const double *norm, const double *schedule, hipStream_t st)
{
    const dim3 grid((unsigned)t.unit[t.n]), block(256);
    constexpr bool half = E == Elem::bf16 || E == Elem::f16;
    if constexpr (E == Elem::f64) {
        if (codes || mb.master) return hipErrorInvalidValue;
        adamw_kernel<E, false, false><<<grid, block, 0, st>>>(t, mb, s, norm, schedule);
    } else if constexpr (half) {
        if (codes && mb.master)
            adamw_kernel<E, true, true><<<grid, block, 0, st>>>(t, mb, s, norm, schedule);
        else if (codes)
            adamw_kernel<E, true, false><<<grid, block, 0, st>>>(t, mb, s, norm, schedule);
        else if (mb.master)
            adamw_kernel<E, false, true><<<grid, block, 0, st>>>(t, mb, s, norm, schedule);
        else
            adamw_kernel<E, false, false><<<grid, block, 0, st>>>(t, mb, s, norm, schedule);
    } else {
        if (mb.master) return hipErrorInvalidValue;
        if (codes)
            adamw_kernel<E, true, false><<<grid, block, 0, st>>>(t, mb, s, norm, schedule);
        else
            adamw_kernel<E, false, false><<<grid, block, 0, st>>>(t, mb, s, norm, schedule);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_adamw(Elem elem, bool codes, const TensorTable &t, const MomentBuffers &mb, const StepScalars &s,
                        const double *norm, const double *schedule, hipStream_t st)
{
    if (t.n == 0 || t.unit[t.n] == 0) return hipSuccess;
    switch (elem) {
    case Elem::f32: return launch_adamw_as<Elem::f32>(codes, t, mb, s, norm, schedule, st);
    case Elem::f64: return launch_adamw_as<Elem::f64>(codes, t, mb, s, norm, schedule, st);
    case Elem::bf16: return launch_adamw_as<Elem::bf16>(codes, t, mb, s, norm, schedule, st);
    case Elem::f16: return launch_adamw_as<Elem::f16>(codes, t, mb, s, norm, schedule, st);
    }
    return hipErrorInvalidValue;
}

int grad_norm_groups(int64_t units) { return (int)std::min<int64_t>(units, kNormGroups); }

hipError_t launch_square_sums(Elem elem, const TensorTable &t, double *partial, hipStream_t st)
{
    const int groups = grad_norm_groups(t.unit[t.n]);
    if (groups == 0) return hipSuccess;
    const dim3 grid((unsigned)groups), block(256);
    switch (elem) {
    case Elem::f32: square_sums_kernel<Elem::f32><<<grid, block, 0, st>>>(t, partial); break;
    case Elem::f64: square_sums_kernel<Elem::f64><<<grid, block, 0, st>>>(t, partial); break;
    case Elem::bf16: square_sums_kernel<Elem::bf16><<<grid, block, 0, st>>>(t, partial); break;
    case Elem::f16: square_sums_kernel<Elem::f16><<<grid, block, 0, st>>>(t, partial); break;
    }
    return hipGetLastError();
}

hipError_t launch_norm(const double *partial, int64_t n, double *norm, hipStream_t st)
{
    norm_kernel<<<dim3(1), dim3(1024), 0, st>>>(partial, n, norm);
    return hipGetLastError();
}

// 1024 elements to a workgroup, and more to each where a launch's threads would not fit 32 bits
static dim3 flat_grid(int64_t elements) { return dim3((unsigned)std::min<int64_t>(elements / 1024, 1 << 23)); }

hipError_t launch_state_read(const void *m, const void *v, const float *scales, int64_t elements, float *m_out,
                             float *v_out, hipStream_t st)
{
    if (elements == 0) return hipSuccess;
    state_read_kernel<<<flat_grid(elements), dim3(256), 0, st>>>(
        static_cast<const signed char *>(m), static_cast<const unsigned char *>(v), scales, elements, m_out, v_out);
    return hipGetLastError();
}

hipError_t launch_state_write(const float *m_in, const float *v_in, int64_t elements, void *m, void *v, float *scales,
                              hipStream_t st)
{
    if (elements == 0) return hipSuccess;
    state_write_kernel<<<flat_grid(elements), dim3(256), 0, st>>>(
        m_in, v_in, elements, static_cast<signed char *>(m), static_cast<unsigned char *>(v), scales);
    return hipGetLastError();
}

hipError_t launch_schedule(double *schedule, double beta1, double beta2, const double *norm, double grad_scale,
                           hipStream_t st)
{
    schedule_kernel<<<dim3(1), dim3(64), 0, st>>>(schedule, beta1, beta2, norm, grad_scale);
    return hipGetLastError();
}

}  // namespace cgtp
