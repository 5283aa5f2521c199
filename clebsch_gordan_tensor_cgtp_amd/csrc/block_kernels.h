// HIP source of the block kernels: the norm at a block's entry and the join at its end (norm,
// gate, residual sum and the next block's norm), forward and backward.  block.cpp puts a
// plan's constants in front of this text and compiles it for gfx950.
//
// Constants of a plan:
//   T, R         element type in memory; type of statistics, weights and sums (float, or double)
//   D, C         columns and channels of a row
//   VEC          elements of 16 bytes
//   G, BLOCK     lanes that share a row; threads of a workgroup
//   CV           neighbouring channels that a lane takes together
//   GATE, ACT    0 none, 1 one logit per row, 2 one per channel; 0 identity 1 sigmoid 2 silu 3 tanh
//   POST, NEXT   norm after the block; norm of the next block
//   NSLOT, S_*   a lane's slots, each CV channels of one irrep (neighbouring irreps of equal degree are
//                one): S_COL, S_CH the irrep's first column and channel, S_K = 2l+1, S_MUL its channels,
//                S_UNIT lane 0's first group of CV channels, S_AT the slot's first element in the lane
//   EPL, E_C     elements of a lane; the lane's channel (of NSLOT x CV) that each belongs to
//   FLAT         the slots are over columns, as if each were a channel (S_K = 1, S_MUL = D): rows without a
//                gate per channel.  NSEG, G_*: the irreps themselves, of which weights are gathered
#pragma once

namespace cgtp {

static const char kBlockKernels[] = R"HIP(
#define DEV static __device__ __forceinline__

constexpr int NC = NSLOT * CV;
constexpr int NW = G > 64 ? G / 64 : 1;            // waves that share a row
constexpr int RPB = BLOCK / G;                     // rows of a workgroup at a time (1 when NW > 1)

// ---------------------------------------------------------------- rows in registers
// With a gate per channel, a lane holds whole channels, all components of each: CV neighbouring
// channels of 2l+1 components are one run of memory, the runs of the row's lanes follow one another, and
// what is per channel (weights, gates, their gradients) meets its components in the lane's own
// registers.  Dealing columns to the lanes and passing gates and their gradients through LDS took 775
// us for the join's backward on 200,000 rows of 64x(0e,1o,2e) in bf16, this 285 us.  Without such a
// gate columns are dealt (FLAT): every load is as wide as it can be, and weights are spread over columns once
// per workgroup (norm, 20,000 rows of 128x(0e,1o,2e,3o) in fp64: 113 us, 136 us by channels).
// Rows start at any element, so the vector types claim no more than the element's alignment.
// Channels past an irrep's end read as 0 and are not written.

template <int N, typename S> DEV void load_run(const S *p, R *x)
{
    if constexpr (N > 0) {
        constexpr int W = 16 / sizeof(S);
        constexpr int n = N >= W ? W : N >= 8 ? 8 : N >= 4 ? 4 : N >= 2 ? 2 : 1;
        typedef S V __attribute__((ext_vector_type(n), aligned(sizeof(S))));
        if constexpr (n == 1) {
            x[0] = (R)p[0];
        } else {
            const V r = *reinterpret_cast<const V *>(p);
#pragma unroll
            for (int i = 0; i < n; ++i) x[i] = (R)r[i];
        }
        load_run<N - n>(p + n, x + n);
    }
}

template <int N, typename S> DEV void store_run(S *p, const R *x)
{
    if constexpr (N > 0) {
        constexpr int W = 16 / sizeof(S);
        constexpr int n = N >= W ? W : N >= 8 ? 8 : N >= 4 ? 4 : N >= 2 ? 2 : 1;
        typedef S V __attribute__((ext_vector_type(n), aligned(sizeof(S))));
        if constexpr (n == 1) {
            p[0] = (S)x[0];
        } else {
            V r;
#pragma unroll
            for (int i = 0; i < n; ++i) r[i] = (S)x[i];
            *reinterpret_cast<V *>(p) = r;
        }
        store_run<N - n>(p + n, x + n);
    }
}

// slot J of a row of K-component channels (columns), or of one value per channel (K = 1)
template <int J, int K, typename S> DEV void load_slot(const S *irrep, int lane, R *x)
{
    const int unit = S_UNIT[J] + lane, left = S_MUL[J] - unit * CV;
    const S *p = irrep + unit * (CV * K);
    constexpr int LAST = S_MUL[J] % CV;  // channels of an irrep's short last group
    if ((S_UNIT[J] + G) * CV <= S_MUL[J] || left >= CV) {
        load_run<CV * K>(p, x);
    } else {
#pragma unroll
        for (int i = 0; i < CV * K; ++i) x[i] = (R)0;
        if (LAST > 0 && left > 0) load_run<LAST * K>(p, x);
    }
}

template <int J, int K, typename S> DEV void store_slot(S *irrep, int lane, const R *x)
{
    const int unit = S_UNIT[J] + lane, left = S_MUL[J] - unit * CV;
    S *p = irrep + unit * (CV * K);
    constexpr int LAST = S_MUL[J] % CV;
    if ((S_UNIT[J] + G) * CV <= S_MUL[J] || left >= CV)
        store_run<CV * K>(p, x);
    else if (LAST > 0 && left > 0)
        store_run<LAST * K>(p, x);
}

template <int J = 0> DEV void load_cols(const T *row, int lane, R (&x)[EPL])
{
    if constexpr (J < NSLOT) {
        load_slot<J, S_K[J]>(row + S_COL[J], lane, x + S_AT[J]);
        load_cols<J + 1>(row, lane, x);
    }
}

template <int J = 0> DEV void store_cols(T *row, int lane, const R (&x)[EPL])
{
    if constexpr (J < NSLOT) {
        store_slot<J, S_K[J]>(row + S_COL[J], lane, x + S_AT[J]);
        store_cols<J + 1>(row, lane, x);
    }
}

template <int J = 0, typename S> DEV void load_channels(const S *row, int lane, R (&c)[NC])
{
    if constexpr (J < NSLOT) {
        load_slot<J, 1>(row + S_CH[J], lane, c + J * CV);
        load_channels<J + 1>(row, lane, c);
    }
}

template <int J = 0, typename S> DEV void store_channels(S *row, int lane, const R (&c)[NC])
{
    if constexpr (J < NSLOT) {
        store_slot<J, 1>(row + S_CH[J], lane, c + J * CV);
        store_channels<J + 1>(row, lane, c);
    }
}

#define EACH_E(i) _Pragma("unroll") for (int i = 0; i < EPL; ++i)
#define EACH_C(c) _Pragma("unroll") for (int c = 0; c < NC; ++c)

// channel of a column; first column and columns of a channel
DEV int channel_of(int col)
{
    int ch = 0;
#pragma unroll
    for (int s = 0; s < NSEG; ++s)
        if (col >= G_COL[s]) ch = G_CH[s] + (col - G_COL[s]) / G_K[s];
    return ch;
}

DEV void columns_of(int c, int &col, int &k)
{
#pragma unroll
    for (int s = 0; s < NSEG; ++s)
        if (c >= G_CH[s]) {
            k = G_K[s];
            col = G_COL[s] + (c - G_CH[s]) * k;
        }
}

// w of the lane's channels (columns where FLAT), 1 without weights
DEV void load_weights(const R *w, int lane, R (&x)[NC])
{
    if (w && FLAT) {
#pragma unroll
        for (int j = 0; j < NSLOT; ++j)
#pragma unroll
            for (int v = 0; v < CV; ++v) {
                const int col = (S_UNIT[j] + lane) * CV + v;
                x[j * CV + v] = col < D ? w[channel_of(col)] : (R)0;
            }
    } else if (w) {
        load_channels(w, lane, x);
    } else {
        EACH_C(c) x[c] = (R)1;
    }
}

// scale[c] w_post[c], each 1 where it is not given
DEV void load_scale(const R *scale, const R *w_post, int lane, R (&x)[NC])
{
    load_weights(scale, lane, x);
    if (POST && w_post) {
        R y[NC];
        load_weights(w_post, lane, y);
        EACH_C(c) x[c] *= y[c];
    }
}

// ---------------------------------------------------------------- sums over a row
// Exchanges of a butterfly: inside 16 lanes by DPP (quads, then mirrored halves and rows, whose
// values are equal by then), across them by the permlane swaps.  Every lane ends with the same bits.
// A swap's results are copied into plain variables first: bit-casting the elements of the builtin's
// vector made the front end read element 0 for both.

template <int CTRL> DEV float dpp(float v)
{
    return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 15, 15, false));
}
template <int CTRL> DEV double dpp(double v)
{
    const unsigned long long b = __builtin_bit_cast(unsigned long long, v);
    const unsigned lo = __builtin_amdgcn_mov_dpp((int)b, CTRL, 15, 15, false);
    const unsigned hi = __builtin_amdgcn_mov_dpp((int)(b >> 32), CTRL, 15, 15, false);
    return __builtin_bit_cast(double, (unsigned long long)hi << 32 | lo);
}
DEV float swap16(float v)
{
    const unsigned a = __builtin_bit_cast(unsigned, v);
    const auto r = __builtin_amdgcn_permlane16_swap(a, a, false, false);
    const unsigned r0 = r[0], r1 = r[1];
    return __builtin_bit_cast(float, r0) + __builtin_bit_cast(float, r1);
}
DEV float swap32(float v)
{
    const unsigned a = __builtin_bit_cast(unsigned, v);
    const auto r = __builtin_amdgcn_permlane32_swap(a, a, false, false);
    const unsigned r0 = r[0], r1 = r[1];
    return __builtin_bit_cast(float, r0) + __builtin_bit_cast(float, r1);
}
DEV double join64(unsigned lo, unsigned hi)
{
    return __builtin_bit_cast(double, (unsigned long long)hi << 32 | lo);
}
DEV double swap16(double v)
{
    const unsigned long long b = __builtin_bit_cast(unsigned long long, v);
    const auto lo = __builtin_amdgcn_permlane16_swap((unsigned)b, (unsigned)b, false, false);
    const auto hi = __builtin_amdgcn_permlane16_swap((unsigned)(b >> 32), (unsigned)(b >> 32), false, false);
    return join64(lo[0], hi[0]) + join64(lo[1], hi[1]);
}
DEV double swap32(double v)
{
    const unsigned long long b = __builtin_bit_cast(unsigned long long, v);
    const auto lo = __builtin_amdgcn_permlane32_swap((unsigned)b, (unsigned)b, false, false);
    const auto hi = __builtin_amdgcn_permlane32_swap((unsigned)(b >> 32), (unsigned)(b >> 32), false, false);
    return join64(lo[0], hi[0]) + join64(lo[1], hi[1]);
}

DEV R lane_sum(R v)
{
    if (G >= 2) v += dpp<0xB1>(v);    // quad_perm 1,0,3,2
    if (G >= 4) v += dpp<0x4E>(v);    // quad_perm 2,3,0,1
    if (G >= 8) v += dpp<0x141>(v);   // row_half_mirror
    if (G >= 16) v += dpp<0x140>(v);  // row_mirror
    if (G >= 32) v = swap16(v);
    if (G >= 64) v = swap32(v);
    return v;
}

// Sum over the row's lanes, the same in all of them.  Waves that share a row exchange theirs
// through LDS with one barrier: consecutive sums take alternate halves of `red`, and a half is
// written again only after the other half's barrier, which every wave reaches after its reads.
DEV R row_sum(R v, R *red, int &turn)
{
    v = lane_sum(v);
    if (NW == 1) return v;
    R *slot = red + turn * NW;
    turn ^= 1;
    if ((threadIdx.x & 63) == 0) slot[threadIdx.x >> 6] = v;
    __syncthreads();
    R s = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) s += slot[w];
    return s;
}

// ---------------------------------------------------------------- partial weight gradients
// A workgroup's sums per channel into out[C]: a wave's row groups are added by lane exchanges, its
// waves one after the other through LDS; where waves share a row each lane has the whole sum of its
// channels already.  FLAT: a channel's columns are added on the way out of LDS.
// Up to the partials the sums are held in R, a lane's rows one after the other: each lane takes N over the rows that
// the workgroups take at once, 98 for 200,000 rows of 576 in fp32, whose weight gradient is then off by 2e-7 of its
// norm (6e-8 with rows summed in double).  Doubles would be one more register a channel, two in the join's
// backward, which has up to 248 of them in use.
constexpr int SUMS = NW > 1 ? 1 : BLOCK / 64;
constexpr int WIDTH = FLAT ? D : C;
constexpr int SUM_LDS = SUMS == 1 && !FLAT ? 1 : SUMS * WIDTH;

// v summed over the lanes of a wave that agree in lane % G: halves and rows by the swaps, then rotations
// inside a row of 16, whose halves, quarters and eighths are equal by then
DEV R group_sum(R v)
{
    if (G < 64) v = swap32(v);
    if (G < 32) v = swap16(v);
    if (G < 16) v += dpp<0x128>(v);  // row_ror:8
    if (G < 8) v += dpp<0x124>(v);
    if (G < 4) v += dpp<0x122>(v);
    if (G < 2) v += dpp<0x121>(v);
    return v;
}

DEV void write_partial(R (&acc)[NC], int lane, R *lds, R *out)
{
    EACH_C(c) acc[c] = group_sum(acc[c]);
    if (SUMS == 1 && !FLAT) {
        store_channels(out, lane, acc);
        return;
    }
    __syncthreads();
    if (NW > 1)
        store_channels(lds, lane, acc);
    else if ((threadIdx.x & 63) < G)
        store_channels(lds + (threadIdx.x >> 6) * WIDTH, lane, acc);
    __syncthreads();
    for (int c = threadIdx.x; c < C; c += BLOCK) {
        int col = c, k = 1;
        if (FLAT) columns_of(c, col, k);
        R s = 0;
        for (int m = 0; m < k; ++m)
#pragma unroll
            for (int w = 0; w < SUMS; ++w) s += lds[w * WIDTH + col + m];
        out[c] = s;
    }
}

// ---------------------------------------------------------------- the gate
// Rows of 16 bits take the hardware's exponential and reciprocal: their errors, |g| 2^-23 and 2^-23 of the
// result, are far below a rounding to 16 bits; the weight gradients, which are float, have them in every row's
// term, as large as a few of float's own roundings (the join's backward, 8,192 scalar rows
// of 4,096 in bf16 with a SiLU gate: 131 us with expf and a division, 116 us).
DEV float exp_of(float v) { return sizeof(T) == 2 ? __builtin_amdgcn_exp2f(v * 1.44269504f) : expf(v); }
DEV float inverse(float v) { return sizeof(T) == 2 ? __builtin_amdgcn_rcpf(v) : 1.0f / v; }
DEV double inverse(double v) { return 1.0 / v; }
DEV double exp_of(double v) { return exp(v); }
DEV float tanh_of(float v) { return tanhf(v); }
DEV double tanh_of(double v) { return tanh(v); }
DEV float root_inverse(float v) { return 1.0f / __builtin_sqrtf(v); }
DEV double root_inverse(double v) { return 1.0 / __builtin_sqrt(v); }

DEV R gate_value(R g)
{
    if (ACT == 0) return g;
    if (ACT == 3) return tanh_of(g);
    const R s = inverse((R)1 + exp_of(-g));
    return ACT == 1 ? s : g * s;
}

// tanh(g) from e = exp(-2 |g|) and r = 1 / (1 + e); below 1/4, where 1 - e would cancel, its series to g^9 (what
// follows is under 2^-26 of it there).  Doubles take the function itself.
DEV float tanh_from(float g, float e, float r)
{
    const float t = (1.0f - e) * r, g2 = g * g;
    const float small = g * (1.0f + g2 * (-1.0f / 3 + g2 * (2.0f / 15 + g2 * (-17.0f / 315 + g2 * (62.0f / 2835)))));
    return g2 < 0.0625f ? small : g < 0 ? -t : t;
}
DEV double tanh_from(double g, double, double) { return tanh(g); }

// act'(g) and act(g).  The sigmoid and its complement are q = e / (1 + e) and 1 - q, e = exp(-|g|), and the slope
// their product; with 1 - s from s it would carry a rounding of 1 (17% of it at 15, all of it at 17).  tanh's
// slope is 4 e / (1 + e)^2 with e = exp(-2 |g|), not 1 - tanh^2.  SiLU's complement is a small term beside 1 there.
DEV R gate_slope(R g, R &value)
{
    if (ACT == 0) {
        value = g;
        return (R)1;
    }
    if (ACT == 3) {
        const R e = exp_of(g < 0 ? 2 * g : -2 * g), r = inverse((R)1 + e);
        value = tanh_from(g, e, r);
        return 4 * (e * r * r);
    }
    if (ACT == 1) {
        const R e = exp_of(g < 0 ? g : -g), q = e * inverse((R)1 + e);
        value = g < 0 ? q : (R)1 - q;
        return q * ((R)1 - q);
    }
    const R s = inverse((R)1 + exp_of(-g));
    value = g * s;
    return s * ((R)1 + g * ((R)1 - s));
}

#define ROW_SETUP                                                       \
    const int lane = threadIdx.x % G, group = threadIdx.x / G;          \
    __shared__ R red[2 * NW];                                           \
    int turn = 0;

// rows n of this row group; lanes of a group past the last row work on that row and write nothing
#define EACH_ROW(n, on)                                                                                  \
    for (long n##0 = (long)blockIdx.x * RPB; n##0 < N; n##0 += (long)gridDim.x * RPB)                    \
        if (const bool on = n##0 + group < N; true)                                                      \
            if (const long n = on ? n##0 + group : N - 1; true)

// ---------------------------------------------------------------- norm
// u = x rstd w,  rstd = (sum x^2 / D + eps)^(-1/2).  One read of x, one write of u.
extern "C" __global__ void __launch_bounds__(BLOCK)
cgtp_norm_fwd(const T *__restrict__ x, long x_ld, const R *__restrict__ w, T *__restrict__ u, R *__restrict__ rstd,
              long N, R eps)
{
    ROW_SETUP
    R wc[NC];
    load_weights(w, lane, wc);
    EACH_ROW(n, on)
    {
        R v[EPL], ss = 0;
        load_cols(x + n * x_ld, lane, v);
        EACH_E(i) ss += v[i] * v[i];
        const R r = root_inverse(row_sum(ss, red, turn) / (R)D + eps);
        EACH_E(i) v[i] = v[i] * r * wc[E_C[i]];
        if (on) {
            store_cols(u + n * D, lane, v);
            if (rstd && lane == 0) rstd[n] = r;
        }
    }
}

// With q = w du and y = x rstd:  dx = rstd (q - y mean(q y)) (+ add),  dw[c] = sum_n sum_m du y.
extern "C" __global__ void __launch_bounds__(BLOCK)
cgtp_norm_bwd(const T *__restrict__ x, long x_ld, const R *__restrict__ w, const R *__restrict__ rstd,
              const T *__restrict__ du, const T *__restrict__ add, T *__restrict__ dx, R *__restrict__ part, long N)
{
    ROW_SETUP
    R wc[NC], acc[NC];
    load_weights(w, lane, wc);
    EACH_C(c) acc[c] = 0;
    EACH_ROW(n, on)
    {
        R y[EPL], q[EPL], t[NC], dot = 0;
        load_cols(x + n * x_ld, lane, y);
        load_cols(du + n * D, lane, q);
        const R r = rstd[n];
        EACH_C(c) t[c] = 0;
        EACH_E(i)
        {
            y[i] *= r;
            t[E_C[i]] += q[i] * y[i];
            q[i] *= wc[E_C[i]];
        }
        EACH_C(c)
        {
            if (part && on) acc[c] += t[c];
            dot += t[c] * wc[c];
        }
        if (!dx) continue;
        dot = row_sum(dot, red, turn) / (R)D;
        EACH_E(i) q[i] = r * (q[i] - y[i] * dot);
        if (add) {
            load_cols(add + n * D, lane, y);
            EACH_E(i) q[i] += y[i];
        }
        if (on) store_cols(dx + n * D, lane, q);
    }
    if (!part) return;
    __shared__ R lds[SUM_LDS];
    write_partial(acc, lane, lds, part + (long)blockIdx.x * C);
}

// ---------------------------------------------------------------- join
// h = alpha r + b[c] y with y = f (rstd_f) and b = act(gate) scale w_post;  u = h rstd_h w_next.
// u comes from h before its rounding.
extern "C" __global__ void __launch_bounds__(BLOCK)
cgtp_join_fwd(const T *__restrict__ res, const T *__restrict__ f, long f_ld, const T *__restrict__ gate, long gate_ld,
              const R *__restrict__ w_post, const R *__restrict__ scale, const R *__restrict__ w_next,
              T *__restrict__ h, T *__restrict__ u, R *__restrict__ rstd_f, R *__restrict__ rstd_h, long N, R alpha,
              R eps)
{
    ROW_SETUP
    R ws[NC], wn[NC];
    load_scale(scale, w_post, lane, ws);
    if (NEXT) load_weights(w_next, lane, wn);
    EACH_ROW(n, on)
    {
        R v[EPL], rv[EPL], b[NC], ss = 0, rf = 1;
        load_cols(f + n * f_ld, lane, v);
        load_cols(res + n * D, lane, rv);
        if (GATE == 2) {
            load_channels(gate + n * gate_ld, lane, b);
            EACH_C(c) b[c] = gate_value(b[c]) * ws[c];
        } else {
            const R a = GATE == 1 ? gate_value((R)gate[n * gate_ld]) : (R)1;
            EACH_C(c) b[c] = a * ws[c];
        }
        if (POST) {
            EACH_E(i) ss += v[i] * v[i];
            rf = root_inverse(row_sum(ss, red, turn) / (R)D + eps);
        }
        EACH_E(i) v[i] = alpha * rv[i] + v[i] * rf * b[E_C[i]];
        if (on) {
            store_cols(h + n * D, lane, v);
            if (POST && rstd_f && lane == 0) rstd_f[n] = rf;
        }
        if (NEXT) {
            ss = 0;
            EACH_E(i) ss += v[i] * v[i];
            const R rh = root_inverse(row_sum(ss, red, turn) / (R)D + eps);
            EACH_E(i) v[i] = v[i] * rh * wn[E_C[i]];
            if (on) {
                store_cols(u + n * D, lane, v);
                if (rstd_h && lane == 0) rstd_h[n] = rh;
            }
        }
    }
}

// Where 1,024 lanes share a row a lane has 128 registers, and the slope of such a gate is one more a channel to
// hold: there the gate and f are loaded after the next norm's sum.  Wide rows, gate and f before the sum and after
// it: 8,192 x 8,192 fp32 sigmoid 508, 479 us, tanh 521, 500; 4,096 x 8,192 fp64 sigmoid 1,146, 999, tanh 1,331, 1,144;
// 4,096 x 16,384 fp32 1,032, 1,012 and 1,237, 1,049; bf16 sigmoid 705, 695.  (By 1 - s and 1 - tanh^2, which are wrong
// for open gates: 496, 490, 921, 1,144, 945, 903, 572.)
constexpr bool LATE = BLOCK == 1024 && NEXT && GATE == 2 && (ACT == 1 || ACT == 3);

// With z = h rstd_h, q = w_next du:  e = dh + rstd_h (q - z mean(q z)) is the whole gradient of h,
//   dr = alpha e,  t[c] = sum_m e y,  P[c] = sum_n act t,  dgate = act' scale w_post t,
//   p = e b,  df = rstd_f (p - y mean(p y)) (p without the norm),  Q[c] = sum_n sum_m du z.
// dscale = w_post P, dw_post = scale P and dw_next = Q come from the workgroups' partials.
extern "C" __global__ void __launch_bounds__(BLOCK)
cgtp_join_bwd(const T *__restrict__ dh, const T *__restrict__ du, const T *__restrict__ h, const T *__restrict__ f,
              long f_ld, const T *__restrict__ gate, long gate_ld, const R *__restrict__ w_post,
              const R *__restrict__ scale, const R *__restrict__ w_next, const R *__restrict__ rstd_f,
              const R *__restrict__ rstd_h, T *__restrict__ dres, T *__restrict__ df, long df_ld,
              T *__restrict__ dgate, long dgate_ld, R *__restrict__ part, long N, R alpha)
{
    ROW_SETUP
    R ws[NC], wn[NC], P[NC], Q[NC];
    load_scale(scale, w_post, lane, ws);
    if (NEXT) load_weights(w_next, lane, wn);
    EACH_C(c) P[c] = Q[c] = 0;
    EACH_ROW(n, on)
    {
        R e[EPL], y[EPL], g[NC], t[NC], a = 1, slope = 0, dot = 0;
        if (GATE == 2 && !LATE) load_channels(gate + n * gate_ld, lane, g);
        if (GATE == 1) slope = gate_slope((R)gate[n * gate_ld], a);
        if (!LATE) load_cols(f + n * f_ld, lane, y);
        if (dh) {
            load_cols(dh + n * D, lane, e);
        } else {
            EACH_E(i) e[i] = 0;
        }
        if (NEXT) {
            R z[EPL], q[EPL];
            load_cols(h + n * D, lane, z);
            load_cols(du + n * D, lane, q);
            const R rh = rstd_h[n];
            EACH_C(c) t[c] = 0;
            EACH_E(i)
            {
                z[i] *= rh;
                t[E_C[i]] += q[i] * z[i];
                q[i] *= wn[E_C[i]];
            }
            EACH_C(c)
            {
                if (part && on) Q[c] += t[c];
                dot += t[c] * wn[c];
            }
            dot = row_sum(dot, red, turn) / (R)D;
            EACH_E(i) e[i] += rh * (q[i] - z[i] * dot);
        }
        if (dres && on) {
            R o[EPL];
            EACH_E(i) o[i] = alpha * e[i];
            store_cols(dres + n * D, lane, o);
        }
        if (LATE) {
            load_channels(gate + n * gate_ld, lane, g);
            load_cols(f + n * f_ld, lane, y);
        }
        const R rf = POST ? rstd_f[n] : (R)1;
        dot = 0;
        EACH_C(c) t[c] = 0;
        EACH_E(i)
        {
            y[i] *= rf;
            t[E_C[i]] += e[i] * y[i];
        }
        EACH_C(c)
        {
            R value = a;
            if (GATE == 2) {
                const R s = gate_slope(g[c], value);
                g[c] = s * (t[c] * ws[c]);
            }
            if (part && on) P[c] += t[c] * value;
            dot += t[c] * ws[c] * (GATE == 2 ? value : (R)1);
            t[c] = ws[c] * value;
        }
        if (GATE == 2 && dgate && on) store_channels(dgate + n * dgate_ld, lane, g);
        if (POST || GATE == 1) dot = row_sum(dot, red, turn);
        if (GATE == 1 && dgate && on && lane == 0) dgate[n * dgate_ld] = (T)(slope * dot);
        EACH_E(i) e[i] *= t[E_C[i]];
        if (POST) {
            dot = dot * a / (R)D;
            EACH_E(i) e[i] = rf * (e[i] - y[i] * dot);
        }
        if (df && on) store_cols(df + n * df_ld, lane, e);
    }
    if (!part) return;
    __shared__ R lds[SUM_LDS];
    R *out = part + (long)blockIdx.x * (NEXT ? 2 : 1) * C;
    write_partial(P, lane, lds, out);
    if (NEXT) write_partial(Q, lane, lds, out + C);
}

// ---------------------------------------------------------------- sums of the partials
// rows of `width` elements, one per workgroup of the pass before, added in a fixed order in double:
// a workgroup takes 16 columns, 64 rows at a time (four to a wave, whose sums the lanes exchange).
// join: the first C are P, the next C are Q; else they are the norm's weight gradient.
extern "C" __global__ void __launch_bounds__(1024)
cgtp_block_reduce(const R *__restrict__ part, long rows, int width, int join, const R *__restrict__ w_post,
                  const R *__restrict__ scale, R *__restrict__ g_post, R *__restrict__ g_scale, R *__restrict__ g_next)
{
    __shared__ double sums[16][16];
    const int col = threadIdx.x & 15, at = blockIdx.x * 16 + col, wave = threadIdx.x >> 6;
    double s = 0;
    if (at < width) {
#pragma unroll 8
        for (long r = threadIdx.x >> 4; r < rows; r += 64) s += (double)part[r * width + at];
    }
    s = swap32(swap16(s));
    if ((threadIdx.x & 63) < 16) sums[wave][col] = s;
    __syncthreads();
    if (threadIdx.x >= 16 || at >= width) return;
    s = 0;
#pragma unroll
    for (int k = 0; k < 16; ++k) s += sums[k][col];
    if (join && at < C) {
        if (g_scale) g_scale[at] = (R)(POST && w_post ? s * (double)w_post[at] : s);
        if (POST && g_post) g_post[at] = (R)(scale ? s * (double)scale[at] : s);
    } else if (g_next) {
        g_next[join ? at - C : at] = (R)s;
    }
}
)HIP";

}  // namespace cgtp
