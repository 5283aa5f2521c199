// HIP source of the block kernels: the norm at a block's entry and the join at its end (norm,
// gate, residual sum and the next block's norm), forward and backward.  block.cpp puts a
// plan's constants in front of this text and compiles it for gfx950.
//
// Constants of a plan:
//   T, R        element type in memory; type of statistics, weights and sums (float, or double)
//   D, C        columns and channels of a row
//   VEC, G, NV  elements of a 16-byte chunk; lanes that share a row; chunks of a lane
//   BLOCK       threads of a workgroup
//   NSEG, SEG_COL, SEG_CH, SEG_K   irreps of equal degree: first column, first channel, 2l+1
//   GATE, ACT   0 none, 1 one logit per row, 2 one per channel; 0 identity 1 sigmoid 2 silu 3 tanh
//   POST, NEXT  norm after the block; norm of the next block
#pragma once

namespace cgtp {

static const char kBlockKernels[] = R"HIP(
#define DEV static __device__ __forceinline__

constexpr int CHUNKS = (D + VEC - 1) / VEC;        // chunks of a row, the last one perhaps short
constexpr int FULL = D / VEC, TAIL = D % VEC;
constexpr int CCHUNKS = (C + VEC - 1) / VEC;       // the same of a row of channels
constexpr int CFULL = C / VEC, CTAIL = C % VEC;
constexpr int NVC = (CCHUNKS + G - 1) / G;
constexpr int NW = G > 64 ? G / 64 : 1;            // waves that share a row
constexpr int RPB = BLOCK / G;                     // rows of a workgroup at a time (1 when NW > 1)
constexpr int DP = CHUNKS * VEC, CP = CCHUNKS * VEC;
constexpr bool SCALAR = D == C;                    // every irrep has l = 0: a column is a channel
constexpr bool STAGED = GATE == 2 && !SCALAR;      // the gate goes through LDS

typedef T Raw __attribute__((ext_vector_type(VEC), aligned(sizeof(T))));
typedef R RawR __attribute__((ext_vector_type(VEC), aligned(sizeof(R))));

// ---------------------------------------------------------------- rows in registers
// Lane `lane` of a row's G lanes holds chunks lane, lane + G, ...: every load is 16 bytes and the
// row's lanes read consecutive ones.  Rows start at any element, so the vector types claim no
// more than the element's alignment.  Columns past the row's end read as 0 and are not written.

template <int N, int NFULL, int NTAIL, typename S> DEV void load_row(const S *row, int lane, R (&x)[N][VEC])
{
    typedef S V __attribute__((ext_vector_type(VEC), aligned(sizeof(S))));
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const int k = lane + G * j;
        if (G * (j + 1) <= NFULL || k < NFULL) {
            const V r = *reinterpret_cast<const V *>(row + k * VEC);
#pragma unroll
            for (int i = 0; i < VEC; ++i) x[j][i] = (R)r[i];
        } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i) x[j][i] = (NTAIL > i && k == NFULL) ? (R)row[k * VEC + i] : (R)0;
        }
    }
}

template <int N, int NFULL, int NTAIL> DEV void store_row(T *row, int lane, const R (&x)[N][VEC])
{
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const int k = lane + G * j;
        if (G * (j + 1) <= NFULL || k < NFULL) {
            Raw r;
#pragma unroll
            for (int i = 0; i < VEC; ++i) r[i] = (T)x[j][i];
            *reinterpret_cast<Raw *>(row + k * VEC) = r;
        } else if (NTAIL > 0 && k == NFULL) {
#pragma unroll
            for (int i = 0; i < NTAIL; ++i) row[k * VEC + i] = (T)x[j][i];
        }
    }
}

#define LOAD_COLS(p, x) load_row<NV, FULL, TAIL>(p, lane, x)
#define STORE_COLS(p, x) store_row<NV, FULL, TAIL>(p, lane, x)
#define LOAD_CHANNELS(p, x) load_row<NVC, CFULL, CTAIL>(p, lane, x)
#define STORE_CHANNELS(p, x) store_row<NVC, CFULL, CTAIL>(p, lane, x)
#define EACH(N, j, i) _Pragma("unroll") for (int j = 0; j < (N); ++j) _Pragma("unroll") for (int i = 0; i < VEC; ++i)

// channel of a column (of the last one for columns past the end), first column of a channel
DEV int channel_of(int col)
{
    col = col < D ? col : D - 1;
    int ch = 0;
#pragma unroll
    for (int s = 0; s < NSEG; ++s)
        if (col >= SEG_COL[s]) ch = SEG_CH[s] + (col - SEG_COL[s]) / SEG_K[s];
    return ch;
}

DEV void columns_of(int c, int &col, int &k)
{
    col = 0;
    k = 1;
#pragma unroll
    for (int s = 0; s < NSEG; ++s)
        if (c >= SEG_CH[s]) {
            k = SEG_K[s];
            col = SEG_COL[s] + (c - SEG_CH[s]) * k;
        }
}

// w[channel of the column], 1 without weights
DEV void load_weights(const R *w, int lane, R (&x)[NV][VEC])
{
    if (!w) {
        EACH(NV, j, i) x[j][i] = (R)1;
    } else if (SCALAR) {
        LOAD_COLS(w, x);
    } else {
        EACH(NV, j, i) x[j][i] = w[channel_of((lane + G * j) * VEC + i)];
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

// LDS written by this row's lanes becomes readable by them
DEV void row_sync()
{
    if (NW > 1) {
        __syncthreads();
    } else {
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    }
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
// acc (per column) of the workgroup's row groups, summed group by group and over each channel's
// columns into out[C]; lds holds RPB x DP elements.
DEV void partial_from_columns(const R (&acc)[NV][VEC], int lane, int group, R *lds, R *out)
{
    if (SCALAR && RPB == 1) {
        EACH(NV, j, i)
        {
            const int col = (lane + G * j) * VEC + i;
            if (col < C) out[col] = acc[j][i];
        }
        return;
    }
    __syncthreads();
    EACH(NV, j, i)
    {
        const int col = (lane + G * j) * VEC + i;
        if (col < DP) lds[group * DP + col] = acc[j][i];
    }
    __syncthreads();
    for (int c = threadIdx.x; c < C; c += BLOCK) {
        int col, k;
        columns_of(c, col, k);
        R s = 0;
        for (int g = 0; g < RPB; ++g)
            for (int m = 0; m < k; ++m) s += lds[g * DP + col + m];
        out[c] = s;
    }
}

// the same for sums that are per channel already; lds holds RPB x CP elements
DEV void partial_from_channels(const R (&acc)[NVC][VEC], int lane, int group, R *lds, R *out)
{
    __syncthreads();
    EACH(NVC, j, i)
    {
        const int c = (lane + G * j) * VEC + i;
        if (c < CP) lds[group * CP + c] = acc[j][i];
    }
    __syncthreads();
    for (int c = threadIdx.x; c < C; c += BLOCK) {
        R s = 0;
        for (int g = 0; g < RPB; ++g) s += lds[g * CP + c];
        out[c] = s;
    }
}

// ---------------------------------------------------------------- the gate
DEV float exp_of(float v) { return expf(v); }
DEV double exp_of(double v) { return exp(v); }
DEV float tanh_of(float v) { return tanhf(v); }
DEV double tanh_of(double v) { return tanh(v); }
DEV float root_inverse(float v) { return 1.0f / __builtin_sqrtf(v); }
DEV double root_inverse(double v) { return 1.0 / __builtin_sqrt(v); }

DEV R gate_value(R g)
{
    if (ACT == 0) return g;
    if (ACT == 3) return tanh_of(g);
    const R s = (R)1 / ((R)1 + exp_of(-g));
    return ACT == 1 ? s : g * s;
}

DEV R gate_slope(R g, R &value)
{
    if (ACT == 0) {
        value = g;
        return (R)1;
    }
    if (ACT == 3) {
        value = tanh_of(g);
        return (R)1 - value * value;
    }
    const R s = (R)1 / ((R)1 + exp_of(-g));
    value = ACT == 1 ? s : g * s;
    return ACT == 1 ? s * ((R)1 - s) : s * ((R)1 + g * ((R)1 - s));
}

// scale[c] * w_post[c], each 1 where it is not given
DEV void load_channel_scale(const R *scale, const R *w_post, int lane, R (&x)[NVC][VEC])
{
    EACH(NVC, j, i)
    {
        const int c = (lane + G * j) * VEC + i;
        x[j][i] = c < C ? (scale ? scale[c] : (R)1) * (POST && w_post ? w_post[c] : (R)1) : (R)0;
    }
}

DEV void load_column_scale(const R *scale, const R *w_post, int lane, R (&x)[NV][VEC])
{
    load_weights(scale, lane, x);
    if (POST && w_post) {
        R y[NV][VEC];
        load_weights(w_post, lane, y);
        EACH(NV, j, i) x[j][i] *= y[j][i];
    }
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
    R wc[NV][VEC];
    load_weights(w, lane, wc);
    EACH_ROW(n, on)
    {
        R v[NV][VEC], ss = 0;
        LOAD_COLS(x + n * x_ld, v);
        EACH(NV, j, i) ss += v[j][i] * v[j][i];
        const R r = root_inverse(row_sum(ss, red, turn) / (R)D + eps);
        EACH(NV, j, i) v[j][i] = v[j][i] * r * wc[j][i];
        if (on) {
            STORE_COLS(u + n * D, v);
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
    R wc[NV][VEC], acc[NV][VEC];
    load_weights(w, lane, wc);
    EACH(NV, j, i) acc[j][i] = 0;
    EACH_ROW(n, on)
    {
        R y[NV][VEC], q[NV][VEC], dot = 0;
        LOAD_COLS(x + n * x_ld, y);
        LOAD_COLS(du + n * D, q);
        const R r = rstd[n];
        EACH(NV, j, i)
        {
            y[j][i] *= r;
            if (part && on) acc[j][i] += q[j][i] * y[j][i];
            q[j][i] *= wc[j][i];
            dot += q[j][i] * y[j][i];
        }
        if (!dx) continue;
        dot = row_sum(dot, red, turn) / (R)D;
        EACH(NV, j, i) q[j][i] = r * (q[j][i] - y[j][i] * dot);
        if (add) {
            LOAD_COLS(add + n * D, y);
            EACH(NV, j, i) q[j][i] += y[j][i];
        }
        if (on) STORE_COLS(dx + n * D, q);
    }
    if (!part) return;
    __shared__ R lds[SCALAR && RPB == 1 ? 1 : RPB * DP];
    partial_from_columns(acc, lane, group, lds, part + (long)blockIdx.x * C);
}

// ---------------------------------------------------------------- join
// h = alpha r + b[c] y with y = f (rstd_f) and b = act(gate) scale w_post;  u = h rstd_h w_next.
// u comes from h before its rounding.  Per-channel gates are evaluated once per channel and
// shared through LDS where a channel has several components.
extern "C" __global__ void __launch_bounds__(BLOCK)
cgtp_join_fwd(const T *__restrict__ res, const T *__restrict__ f, long f_ld, const T *__restrict__ gate, long gate_ld,
              const R *__restrict__ w_post, const R *__restrict__ scale, const R *__restrict__ w_next,
              T *__restrict__ h, T *__restrict__ u, R *__restrict__ rstd_f, R *__restrict__ rstd_h, long N, R alpha,
              R eps)
{
    ROW_SETUP
    __shared__ R staged[STAGED ? RPB * CP : 1];
    R *b = staged + group * CP;
    R ws[NV][VEC], wsc[NVC][VEC], wn[NV][VEC];
    if constexpr (STAGED)
        load_channel_scale(scale, w_post, lane, wsc);
    else
        load_column_scale(scale, w_post, lane, ws);
    if constexpr (NEXT) load_weights(w_next, lane, wn);
    EACH_ROW(n, on)
    {
        R v[NV][VEC], rv[NV][VEC], ss = 0, rf = 1;
        LOAD_COLS(f + n * f_ld, v);
        LOAD_COLS(res + n * D, rv);
        if constexpr (STAGED) {
            R g[NVC][VEC];
            LOAD_CHANNELS(gate + n * gate_ld, g);
            EACH(NVC, j, i)
            {
                const int c = (lane + G * j) * VEC + i;
                if (c < CP) b[c] = gate_value(g[j][i]) * wsc[j][i];
            }
            row_sync();
        }
        if constexpr (POST) {
            EACH(NV, j, i) ss += v[j][i] * v[j][i];
            rf = root_inverse(row_sum(ss, red, turn) / (R)D + eps);
        }
        if constexpr (STAGED) {
            EACH(NV, j, i)
            v[j][i] = alpha * rv[j][i] + v[j][i] * rf * b[channel_of((lane + G * j) * VEC + i)];
            row_sync();
        } else if constexpr (GATE == 2) {
            R g[NV][VEC];
            LOAD_COLS(gate + n * gate_ld, g);
            EACH(NV, j, i) v[j][i] = alpha * rv[j][i] + v[j][i] * rf * ws[j][i] * gate_value(g[j][i]);
        } else {
            const R a = GATE == 1 ? gate_value((R)gate[n * gate_ld]) : (R)1;
            EACH(NV, j, i) v[j][i] = alpha * rv[j][i] + v[j][i] * rf * ws[j][i] * a;
        }
        if constexpr (TAIL > 0 || CHUNKS % G != 0) {
            EACH(NV, j, i) if ((lane + G * j) * VEC + i >= D) v[j][i] = 0;
        }
        if (on) {
            STORE_COLS(h + n * D, v);
            if (POST && rstd_f && lane == 0) rstd_f[n] = rf;
        }
        if constexpr (NEXT) {
            ss = 0;
            EACH(NV, j, i) ss += v[j][i] * v[j][i];
            const R rh = root_inverse(row_sum(ss, red, turn) / (R)D + eps);
            EACH(NV, j, i) v[j][i] = v[j][i] * rh * wn[j][i];
            if (on) {
                STORE_COLS(u + n * D, v);
                if (rstd_h && lane == 0) rstd_h[n] = rh;
            }
        }
    }
}

// With z = h rstd_h, q = w_next du:  e = dh + rstd_h (q - z mean(q z)) is the whole gradient of h,
//   dr = alpha e,  t = e y,  P[c] = sum_n act sum_m t,  dgate = act' scale w_post sum_m t,
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
    constexpr int LDS = (SCALAR && RPB == 1) ? 1 : RPB * DP;
    __shared__ R lds[LDS];
    __shared__ R staged[STAGED ? RPB * CP : 1];
    R *b = staged + group * CP;
    R ws[NV][VEC], wsc[NVC][VEC], wn[NV][VEC];
    R P[NV][VEC], PC[NVC][VEC], Q[NV][VEC];
    if constexpr (STAGED) {
        load_channel_scale(scale, w_post, lane, wsc);
        EACH(NVC, j, i) PC[j][i] = 0;
    } else {
        load_column_scale(scale, w_post, lane, ws);
        EACH(NV, j, i) P[j][i] = 0;
    }
    if constexpr (NEXT) {
        load_weights(w_next, lane, wn);
        EACH(NV, j, i) Q[j][i] = 0;
    }
    EACH_ROW(n, on)
    {
        R e[NV][VEC], y[NV][VEC], dot = 0;
        R ga[NVC][VEC], gs[NVC][VEC];
        LOAD_COLS(f + n * f_ld, y);
        if (dh) {
            LOAD_COLS(dh + n * D, e);
        } else {
            EACH(NV, j, i) e[j][i] = 0;
        }
        if constexpr (STAGED) {
            R g[NVC][VEC];
            LOAD_CHANNELS(gate + n * gate_ld, g);
            EACH(NVC, j, i)
            {
                const int c = (lane + G * j) * VEC + i;
                gs[j][i] = gate_slope(g[j][i], ga[j][i]);
                if (c < CP) b[c] = ga[j][i] * wsc[j][i];
            }
        }
        if constexpr (NEXT) {
            R z[NV][VEC], q[NV][VEC];
            LOAD_COLS(h + n * D, z);
            LOAD_COLS(du + n * D, q);
            const R rh = rstd_h[n];
            EACH(NV, j, i)
            {
                z[j][i] *= rh;
                if (part && on) Q[j][i] += q[j][i] * z[j][i];
                q[j][i] *= wn[j][i];
                dot += q[j][i] * z[j][i];
            }
            dot = row_sum(dot, red, turn) / (R)D;
            EACH(NV, j, i) e[j][i] += rh * (q[j][i] - z[j][i] * dot);
        }
        if (dres && on) {
            R o[NV][VEC];
            EACH(NV, j, i) o[j][i] = alpha * e[j][i];
            STORE_COLS(dres + n * D, o);
        }
        const R rf = POST ? rstd_f[n] : (R)1;
        EACH(NV, j, i) y[j][i] *= rf;
        dot = 0;
        if constexpr (STAGED) {
            R *t = lds + group * DP;
            EACH(NV, j, i)
            {
                const int col = (lane + G * j) * VEC + i;
                if (col < DP) t[col] = e[j][i] * y[j][i];
            }
            row_sync();
            EACH(NV, j, i)
            {
                e[j][i] *= b[channel_of((lane + G * j) * VEC + i)];
                dot += e[j][i] * y[j][i];
            }
            EACH(NVC, j, i)
            {
                const int c = (lane + G * j) * VEC + i;
                R s = 0;
                if (c < C) {
                    int col, k;
                    columns_of(c, col, k);
                    for (int m = 0; m < k; ++m) s += t[col + m];
                }
                if (part && on) PC[j][i] += s * ga[j][i];
                gs[j][i] *= s * wsc[j][i];
            }
            row_sync();
            if (dgate && on) STORE_CHANNELS(dgate + n * dgate_ld, gs);
        } else if constexpr (GATE == 2) {
            R g[NV][VEC];
            LOAD_COLS(gate + n * gate_ld, g);
            EACH(NV, j, i)
            {
                R a;
                const R sl = gate_slope(g[j][i], a);
                const R t = e[j][i] * y[j][i];
                if (part && on) P[j][i] += t * a;
                g[j][i] = sl * (t * ws[j][i]);
                e[j][i] *= ws[j][i] * a;
                dot += e[j][i] * y[j][i];
            }
            if (dgate && on) STORE_COLS(dgate + n * dgate_ld, g);
        } else {
            R a = 1, sl = 0;
            if constexpr (GATE == 1) sl = gate_slope((R)gate[n * gate_ld], a);
            EACH(NV, j, i)
            {
                if (part && on) P[j][i] += e[j][i] * y[j][i] * a;
                e[j][i] *= ws[j][i];
                dot += e[j][i] * y[j][i];
                e[j][i] *= a;
            }
        }
        if constexpr (POST || GATE == 1) dot = row_sum(dot, red, turn);
        if constexpr (GATE == 1 || GATE == 0) {
            R a = 1, sl = 0;
            if constexpr (GATE == 1) {
                sl = gate_slope((R)gate[n * gate_ld], a);
                if (dgate && on && lane == 0) dgate[n * dgate_ld] = (T)(sl * dot);
            }
            dot *= a;
        }
        if constexpr (POST) {
            dot /= (R)D;
            EACH(NV, j, i) e[j][i] = rf * (e[j][i] - y[j][i] * dot);
        }
        if (df && on) STORE_COLS(df + n * df_ld, e);
    }
    if (!part) return;
    R *out = part + (long)blockIdx.x * (NEXT ? 2 : 1) * C;
    if constexpr (STAGED)
        partial_from_channels(PC, lane, group, staged, out);
    else
        partial_from_columns(P, lane, group, lds, out);
    if constexpr (NEXT) partial_from_columns(Q, lane, group, lds, out + C);
}

// ---------------------------------------------------------------- sums of the partials
// rows of `width` elements, one per workgroup of the pass before, added in a fixed order in double.
// join: the first C are P, the next C are Q; else they are the norm's weight gradient.
extern "C" __global__ void __launch_bounds__(1024)
cgtp_block_reduce(const R *__restrict__ part, long rows, int width, int join, const R *__restrict__ w_post,
                  const R *__restrict__ scale, R *__restrict__ g_post, R *__restrict__ g_scale, R *__restrict__ g_next)
{
    __shared__ double sums[16][64];
    const int at = blockIdx.x * 64 + (threadIdx.x & 63), slice = threadIdx.x >> 6;
    double s = 0;
    if (at < width)
        for (long r = slice; r < rows; r += 16) s += (double)part[r * width + at];
    sums[slice][threadIdx.x & 63] = s;
    __syncthreads();
    if (slice != 0 || at >= width) return;
#pragma unroll
    for (int k = 1; k < 16; ++k) s += sums[k][threadIdx.x & 63];
    if (join && at < C) {
        if (g_scale) g_scale[at] = (R)(POST && w_post ? s * (double)w_post[at] : s);
        if (POST && g_post) g_post[at] = (R)(scale ? s * (double)scale[at] : s);
    } else if (g_next) {
        g_next[join ? at - C : at] = (R)s;
    }
}
)HIP";

}  // namespace cgtp
