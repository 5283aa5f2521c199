// HIP source of the experts' products over irreps rows, out[n] = sum_j p[n][j] W[e(n, j)] x[n], and of
// their gradients.  linear.cpp puts a plan's constants and the shared text (row_kernels.h) in front of
// this text and compiles it for gfx950.
//
// Constants of a plan, beside T, R and ACT:
//   E, K          experts; experts of a row (0: the one expert of every row, with weight 1)
//   NUMEL         weights of an expert
//   Forward, Backward, and for few rows ForwardFew, BackwardFew: the product's two directions, each a struct of
//     NPARTS, IN_PITCH, OUT_PITCH, LDS_BYTES  parts, worked on one after the other: pitches of their rows in LDS
//     NS, S_PART, S_COL, S_LEN, S_LDS, S_PAD  input irreps: part, first column, columns; where they begin in LDS and
//                                             columns there (whole steps)
//     NOUT, O_PART, O_COL, O_MUL, O_K, O_LDS, O_P0, O_PN   output irreps: first column, channels, 2l+1, place in LDS,
//                                             first path, paths
//     P_LDS, P_MUL, P_W                       paths: the input irrep's place in LDS and channels, the matrix
//                                             [O_MUL][P_MUL] (row major) in the expert's weights
//     NU, U_PART, U_OUT, U_N0, U_NN, U_WAVE, WAVES  units: output irrep, first and number of its blocks of 16
//                                             channels, the wave that takes it; waves of a workgroup
//     DOT, SIMD_WAVES                         1: the weights p have a gradient; waves that registers are kept few enough for
//   NPATH, W_*    for the weight gradients, per path: W_XC, W_MI the input's first column and channels, W_GC, W_MO
//                 the output's, W_K, W_OFF the first weight
//   NT, T_PATH, T_V, T_U, T_BV, T_BU          tiles of the gradients: path, first output and input channel, 16-blocks
//   T_WV, T_WU, T_NODES, MAX_STRETCH          of each; waves along each, nodes in LDS at a time; most slots of a stretch
#pragma once

namespace cgtp {

static const char kLinearKernels[] = R"HIP(
typedef R V4 __attribute__((ext_vector_type(4)));
constexpr bool HALF = sizeof(T) == 2;
constexpr int KL = HALF ? 8 : 4;  // input channels that a lane holds of a step
constexpr int STEP = 4 * KL;      // input channels of a step
constexpr int BIG = 0x7fffffff;

// ---------------------------------------------------------------- matrix instructions
// 16x16 blocks.  Lane l holds row (or column) l % 16 of an operand and, of the summed index, the values
// of its quarter l / 16: which ones they are does not matter as long as both operands agree, so a lane takes
// KL neighbouring channels, all 2l+1 components of each: one run of its row, straight into registers.  The
// product is formed transposed (rows: output channels, columns: nodes), which leaves a lane with four
// neighbouring channels of one node, one run again, and with the node's own weight.
// Of the result, lane l has column l % 16 and rows 4 (l / 16) + i (f64: l / 16 + 4 i).
DEV int row_channel(int row) { return sizeof(T) == 8 ? row / 4 + 4 * (row % 4) : row; }

#if defined(BITS16)
typedef T V8 __attribute__((ext_vector_type(8)));
DEV V4 mfma(V8 a, V8 b, V4 c)
{
#if BITS16 == 1
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
#else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
#endif
}
#endif
)HIP"
R"HIP(
// N neighbouring elements as they are
template <int N> DEV void load_raw(const T *p, T *x)
{
    if constexpr (N > 0) {
        constexpr int W = 16 / sizeof(T);
        constexpr int n = N >= W ? W : N >= 8 ? 8 : N >= 4 ? 4 : N >= 2 ? 2 : 1;
        typedef T V __attribute__((ext_vector_type(n), aligned(sizeof(T))));
        if constexpr (n == 1) {
            x[0] = p[0];
        } else {
            const V r = *reinterpret_cast<const V *>(p);
#pragma unroll
            for (int i = 0; i < n; ++i) x[i] = r[i];
        }
        load_raw<N - n>(p + n, x + n);
    }
}

// `count` of N channels of KC elements, zeros for the others; ALL: every one is there
template <int N, int KC, bool ALL> DEV void load_channels(const T *p, int count, T *x)
{
    if (ALL || count >= N) {
        load_raw<N * KC>(p, x);
    } else {
#pragma unroll
        for (int i = 0; i < N * KC; ++i) x[i] = i < count * KC ? p[i] : (T)0;
    }
}

// acc[n][m] += A[n] B[m] over a step of STEP channels; a: KL per block, b: KL channels of KC components
template <int NN, int KC> DEV void step(const T (&a)[NN][KL], const T (&b)[KL * KC], V4 (&acc)[NN][KC])
{
#if defined(BITS16)
    V8 bv[KC];
#pragma unroll
    for (int m = 0; m < KC; ++m)
#pragma unroll
        for (int i = 0; i < 8; ++i) bv[m][i] = b[i * KC + m];
#pragma unroll
    for (int n = 0; n < NN; ++n) {
        V8 av;
#pragma unroll
        for (int i = 0; i < 8; ++i) av[i] = a[n][i];
#pragma unroll
        for (int m = 0; m < KC; ++m) acc[n][m] = mfma(av, bv[m], acc[n][m]);
    }
#else
#pragma unroll
    for (int i = 0; i < KL; ++i)
#pragma unroll
        for (int n = 0; n < NN; ++n)
#pragma unroll
            for (int m = 0; m < KC; ++m) acc[n][m] = MFMA(a[n][i], b[i * KC + m], acc[n][m]);
#endif
}

// ---------------------------------------------------------------- tiles of 16 rows
// A workgroup takes 16 rows, one part of their irreps after the other: a part's input columns come into LDS by
// loads of neighbouring lanes along the rows, and its results leave it the same way.  Operands read straight
// from memory are runs of 16 (2l+1) bytes per lane, each instruction touching 64 cache lines for 16 bytes each.
// A part that would leave a CU one workgroup (OUT_PITCH 0) stores its results from registers all the same: two workgroups
// that overlap are worth more there (20,000 rows of 128x(0e,1o,2e,3o) in fp32, forward: 304 us through LDS, 265 us).
// In LDS an irrep starts at 16 bytes and is padded with zeros to whole steps; a row's pitch is an odd multiple
// of 16 bytes, so that the eight lanes of an LDS access (eight nodes) meet different banks.
constexpr int VEC = 16 / sizeof(T);
typedef T V16 __attribute__((ext_vector_type(VEC)));

template <class D, int S> DEV void copy_in(T *lds, int pitch, const T *in, long ld, const int *node)
{
    constexpr int LEN = D::S_LEN[S], CHUNKS = D::S_PAD[S] / VEC, TOTAL = 16 * CHUNKS, THREADS = D::WAVES * 64;
#pragma unroll 8
    for (int at = threadIdx.x; at < TOTAL; at += THREADS) {
        const int r = at / CHUNKS, e = at % CHUNKS * VEC, n = node[r];
        T v[VEC];
        // whole runs are loaded without a branch: a node that is none takes row 0, and its results are not stored
        if constexpr (LEN % VEC == 0 && LEN == D::S_PAD[S])
            load_raw<VEC>(in + (n < 0 ? 0 : n) * ld + D::S_COL[S] + e, v);
        else
            load_channels<VEC, 1, false>(in + (n < 0 ? 0 : n) * ld + D::S_COL[S] + e, n < 0 ? 0 : LEN - e, v);
        V16 q;
#pragma unroll
        for (int i = 0; i < VEC; ++i) q[i] = v[i];
        *reinterpret_cast<V16 *>(lds + r * pitch + D::S_LDS[S] + e) = q;
    }
}

// rows of the part's output irreps: into LDS (the row of x), or out of it
template <class D, int O, bool OUT> DEV void copy_rows(T *lds, int pitch, T *rows, long ld, const int *node)
{
    constexpr int LEN = D::O_MUL[O] * D::O_K[O], CHUNKS = (LEN + VEC - 1) / VEC, TOTAL = 16 * CHUNKS, THREADS = D::WAVES * 64;
#pragma unroll 8
    for (int at = threadIdx.x; at < TOTAL; at += THREADS) {
        const int r = at / CHUNKS, e = at % CHUNKS * VEC, n = node[r];
        T *p = rows + (n < 0 ? 0 : n) * ld + D::O_COL[O] + e;
        V16 *q = reinterpret_cast<V16 *>(lds + r * pitch + D::O_LDS[O] + e);
        T v[VEC];
        if (OUT) {
            const V16 w = *q;
#pragma unroll
            for (int i = 0; i < VEC; ++i) v[i] = w[i];
            if (n < 0) continue;
            typedef T V __attribute__((ext_vector_type(VEC), aligned(sizeof(T))));
            if (LEN % VEC == 0 || e + VEC <= LEN) {
                // past the caches, which keep the matrices and the rows instead: 200,000 rows of 64x(0e,1o,2e) in bf16 by one
                // matrix 123 us, this way 95 us (93 us now); of 5,000 rows there is no difference
                __builtin_nontemporal_store((V)w, reinterpret_cast<V *>(p));
            } else {
#pragma unroll
                for (int i = 0; i < VEC; ++i)
                    if (e + i < LEN) p[i] = v[i];
            }
        } else {
            if constexpr (LEN % VEC == 0)
                load_raw<VEC>(p, v);
            else
                load_channels<VEC, 1, false>(p, n < 0 ? 0 : LEN - e, v);
            V16 w;
#pragma unroll
            for (int i = 0; i < VEC; ++i) w[i] = v[i];
            *q = w;
        }
    }
}

template <class D, int PART, int S = 0> DEV void part_in(T *lds, const T *in, long ld, const int *node)
{
    if constexpr (S < D::NS) {
        if constexpr (D::S_PART[S] == PART) copy_in<D, S>(lds, D::IN_PITCH[PART], in, ld, node);
        part_in<D, PART, S + 1>(lds, in, ld, node);
    }
}

template <class D, int PART, bool OUT, int O = 0> DEV void part_rows(T *lds, T *rows, long ld, const int *node)
{
    if constexpr (O < D::NOUT) {
        if constexpr (D::O_PART[O] == PART) copy_rows<D, O, OUT>(lds, D::OUT_PITCH[PART], rows, ld, node);
        part_rows<D, PART, OUT, O + 1>(lds, rows, ld, node);
    }
}

// `count` elements of LDS, 16 bytes at a time where there are as many
template <int N> DEV void read_lds(const T *p, T *x)
{
    constexpr int n = N >= VEC ? VEC : N;
    typedef T V __attribute__((ext_vector_type(n)));
    const V r = *reinterpret_cast<const V *>(p);
#pragma unroll
    for (int i = 0; i < n; ++i) x[i] = r[i];
    if constexpr (N > n) read_lds<N - n>(p + n, x + n);
}

// One path's product of an expert: w its matrix, x the node's row in LDS
template <class D, int U, int P> DEV void path(const T *w, const T *x, int lane, V4 (&acc)[D::U_NN[U]][D::O_K[D::U_OUT[U]]])
{
    constexpr int O = D::U_OUT[U], N0 = D::U_N0[U], NN = D::U_NN[U], KC = D::O_K[O], MI = D::P_MUL[P], MO = D::O_MUL[O];
    const int v = N0 * 16 + row_channel(lane & 15), k = (lane >> 4) * KL;
    x += D::P_LDS[P] + k * KC;
    w += D::P_W[P] + k;
    // channels past the irrep's end: their products are not stored, so any row of the matrix does for them
    int row[NN];
#pragma unroll
    for (int n = 0; n < NN; ++n) row[n] = ((N0 + n + 1) * 16 <= MO || v + n * 16 < MO ? v + n * 16 : MO - 1) * MI;
#pragma unroll 4
    for (int s = 0; s < MI / STEP; ++s) {
        T a[NN][KL], b[KL * KC];
#pragma unroll
        for (int n = 0; n < NN; ++n) load_raw<KL>(w + row[n] + s * STEP, a[n]);
        read_lds<KL * KC>(x + s * STEP * KC, b);
        step<NN, KC>(a, b, acc);
    }
    if constexpr (MI % STEP != 0) {
        constexpr int s = MI / STEP;
        T a[NN][KL], b[KL * KC];
#pragma unroll
        for (int n = 0; n < NN; ++n) load_channels<KL, 1, false>(w + row[n] + s * STEP, MI - s * STEP - k, a[n]);
        read_lds<KL * KC>(x + s * STEP * KC, b);
        step<NN, KC>(a, b, acc);
    }
}

template <class D, int U, int P, int END> DEV void paths(const T *w, const T *x, int lane,
                                                         V4 (&acc)[D::U_NN[U]][D::O_K[D::U_OUT[U]]])
{
    if constexpr (P < END) {
        path<D, U, P>(w, x, lane, acc);
        paths<D, U, P + 1, END>(w, x, lane, acc);
    }
}

// the smallest over the 16 nodes, the same in every lane of the wave
DEV int wave_min(int v)
{
    int o = __builtin_amdgcn_mov_dpp(v, 0xB1, 15, 15, false);
    v = o < v ? o : v;
    o = __builtin_amdgcn_mov_dpp(v, 0x4E, 15, 15, false);
    v = o < v ? o : v;
    o = __builtin_amdgcn_mov_dpp(v, 0x141, 15, 15, false);
    v = o < v ? o : v;
    o = __builtin_amdgcn_mov_dpp(v, 0x140, 15, 15, false);
    v = o < v ? o : v;
    return __builtin_amdgcn_readfirstlane(v);
}

constexpr int KS = K > 0 ? K : 1;

struct Node {
    const T *in;  // its row of the part's input, in LDS
    T *out;       // and of its output, which first holds x where the weights' gradient is wanted
    T *row;       // its rows in memory: of the output (NULL: none), and of x
    const T *x;
    int e[KS];    // its experts, BIG where there is none
    R p[KS];
};

// A wave's 16 nodes take the experts that any of them has in rising order.  A node's sum is of its own
// experts alone, each product scaled in R and added to it (others are not added, so what they hold cannot
// reach it), and so depends neither on its neighbours nor on the order of the rows.
template <class D, int U> DEV void unit(const Node &node, const T *w, int lane, bool dot, R (&dp)[KS])
{
    constexpr int O = D::U_OUT[U], N0 = D::U_N0[U], NN = D::U_NN[U], KC = D::O_K[O], MO = D::O_MUL[O];
    constexpr int P0 = D::O_P0[O], PN = D::O_PN[O];
    constexpr bool DIRECT = D::OUT_PITCH[D::U_PART[U]] == 0;
    const int v0 = N0 * 16 + 4 * (lane >> 4);  // the lane's first channel
    T *out = node.out + D::O_LDS[O] + v0 * KC;
    V4 total[NN][KC];
#pragma unroll
    for (int n = 0; n < NN; ++n)
#pragma unroll
        for (int m = 0; m < KC; ++m) total[n][m] = (V4)(R)0;
    if constexpr (PN > 0) {
        // a direct part's x stays in registers from one expert to the next
        T xr[DIRECT && D::DOT ? NN : 1][4 * KC];
        if constexpr (DIRECT && D::DOT) {
#pragma unroll
            for (int n = 0; n < NN; ++n)
                load_channels<4, KC, false>(node.x + D::O_COL[O] + (v0 + n * 16) * KC, node.x ? MO - v0 - n * 16 : 0, xr[n]);
        }
        int last = -1;
        for (;;) {
            int next = BIG;
            if (K > 0) {
#pragma unroll
                for (int j = 0; j < K; ++j) next = node.e[j] > last && node.e[j] < next ? node.e[j] : next;
                next = wave_min(next);
                if (next == BIG) break;
            }
            const T *we = w + (K > 0 ? (long)next * NUMEL : 0);
            V4 acc[NN][KC];
#pragma unroll
            for (int n = 0; n < NN; ++n)
#pragma unroll
                for (int m = 0; m < KC; ++m) acc[n][m] = (V4)(R)0;
            paths<D, U, P0, P0 + PN>(we, node.in, lane, acc);
            if (K == 0) {
#pragma unroll
                for (int n = 0; n < NN; ++n)
#pragma unroll
                    for (int m = 0; m < KC; ++m) total[n][m] = acc[n][m];
                break;
            }
            R p = 0;
            bool has = false;
#pragma unroll
            for (int j = 0; j < K; ++j)
                if (node.e[j] == next) {
                    p += node.p[j];
                    has = true;
                }
            if (has) {
#pragma unroll
                for (int n = 0; n < NN; ++n)
#pragma unroll
                    for (int m = 0; m < KC; ++m)
#pragma unroll
                        for (int i = 0; i < 4; ++i) total[n][m][i] = fma(p, acc[n][m][i], total[n][m][i]);
            }
            if (D::DOT && dot) {
                R s = 0;
#pragma unroll
                for (int n = 0; n < NN; ++n) {
                    T x[4 * KC];
                    if constexpr (DIRECT) {
#pragma unroll
                        for (int i = 0; i < 4 * KC; ++i) x[i] = xr[n][i];
                    } else {
                        read_lds<4 * KC>(out + n * 16 * KC, x);
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int m = 0; m < KC; ++m)
                            if ((N0 + n + 1) * 16 <= MO || v0 + n * 16 + i < MO) s = fma(acc[n][m][i], (R)x[i * KC + m], s);
                }
                s = swap32(swap16(s));
#pragma unroll
                for (int j = 0; j < K; ++j) dp[j] += node.e[j] == next ? s : (R)0;
            }
            last = next;
        }
    }
    if constexpr (DIRECT) {
        if (!node.row) return;
#pragma unroll
        for (int n = 0; n < NN; ++n) {
            R v[4 * KC];
#pragma unroll
            for (int i = 0; i < 4 * KC; ++i) v[i] = total[n][i % KC][i / KC];
            T *row = node.row + D::O_COL[O] + (v0 + n * 16) * KC;
            const int left = MO - v0 - n * 16;
            if ((N0 + n + 1) * 16 <= MO || left >= 4) {
                store_run<4 * KC>(row, v);
            } else {
#pragma unroll
                for (int i = 0; i < 4 * KC; ++i)
                    if (i < left * KC) row[i] = (T)v[i];
            }
        }
        return;
    }
#pragma unroll
    for (int n = 0; n < NN; ++n) {
        constexpr int n4 = 4 * KC >= VEC ? VEC : 4 * KC;
        typedef T V __attribute__((ext_vector_type(n4)));
#pragma unroll
        for (int q = 0; q < 4 * KC / n4; ++q) {
            V r;
#pragma unroll
            for (int i = 0; i < n4; ++i) r[i] = (T)total[n][(q * n4 + i) % KC][(q * n4 + i) / KC];
            *reinterpret_cast<V *>(out + n * 16 * KC + q * n4) = r;
        }
        if constexpr (4 * KC % n4 != 0) {
#pragma unroll
            for (int i = 4 * KC / n4 * n4; i < 4 * KC; ++i) out[n * 16 * KC + i] = (T)total[n][i % KC][i / KC];
        }
    }
}

template <class D, int PART, int U = 0> DEV void units(const Node &node, const T *w, int wave, int lane, bool dot, R (&dp)[KS])
{
    if constexpr (U < D::NU) {
        if constexpr (D::U_PART[U] == PART) {
            if (D::U_WAVE[U] == wave) unit<D, U>(node, w, lane, dot, dp);
        }
        units<D, PART, U + 1>(node, w, wave, lane, dot, dp);
    }
}

template <class D, int PART = 0>
DEV void parts(Node &node, T *tile, const int *rows, const T *in, long in_ld, const T *w, T *out, long out_ld, const T *x,
               long x_ld, int wave, int lane, R (&dp)[KS])
{
    if constexpr (PART < D::NPARTS) {
        constexpr bool DIRECT = D::OUT_PITCH[PART] == 0;
        T *results = tile + 16 * D::IN_PITCH[PART];
        if (PART > 0) __syncthreads();  // the part before has left LDS
        part_in<D, PART>(tile, in, in_ld, rows);
        if (D::DOT && x && !DIRECT) part_rows<D, PART, false>(results, const_cast<T *>(x), x_ld, rows);
        __syncthreads();
        node.in = tile + (lane & 15) * D::IN_PITCH[PART];
        node.out = results + (lane & 15) * D::OUT_PITCH[PART];
        units<D, PART>(node, w, wave, lane, x != nullptr, dp);
        if (out && !DIRECT) {
            __syncthreads();
            part_rows<D, PART, true>(results, out, out_ld, rows);
        }
        parts<D, PART + 1>(node, tile, rows, in, in_ld, w, out, out_ld, x, x_ld, wave, lane, dp);
    }
}

template <class D>
DEV void product(const T *in, long in_ld, const T *w, const int *experts, const R *weights, const int *order, long N,
                 T *out, long out_ld, const T *x, long x_ld, R *grad_weights)
{
    __shared__ V16 tile[D::LDS_BYTES / 16];
    __shared__ int rows[16];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const long at = (long)blockIdx.x * 16 + (lane & 15);
    long n = at < N ? at : -1;
    if (order && n >= 0) n = order[n];
    if (n >= N || n < 0) n = -1;
    if (threadIdx.x < 16) rows[threadIdx.x] = (int)n;
    Node node;
    node.row = out && n >= 0 ? out + n * out_ld : nullptr;
    node.x = x && n >= 0 ? x + n * x_ld : nullptr;
    R dp[KS];
#pragma unroll
    for (int j = 0; j < KS; ++j) {
        const int e = K > 0 && n >= 0 ? experts[n * K + j] : -1;
        const bool has = e >= 0 && e < E;
        node.e[j] = has ? e : BIG;
        node.p[j] = has ? weights[n * K + j] : (R)0;
        dp[j] = 0;
    }
    __syncthreads();
    parts<D>(node, reinterpret_cast<T *>(tile), rows, in, in_ld, w, out, out_ld, x, x_ld, wave, lane, dp);
    if (K > 0 && D::DOT && grad_weights) {
        // the waves' shares of a node's sum, in the waves' order
        __shared__ R lds[D::DOT ? D::WAVES * 16 * KS : 1];
#pragma unroll
        for (int j = 0; j < K; ++j)
            if (lane < 16) lds[(wave * 16 + lane) * KS + j] = dp[j];
        __syncthreads();
        for (int t = threadIdx.x; t < 16 * K; t += D::WAVES * 64) {
            const int i = t / KS, j = t % KS, row = rows[i];
            R s = 0;
#pragma unroll
            for (int v = 0; v < D::WAVES; ++v) s += lds[(v * 16 + i) * KS + j];
            if (row >= 0) grad_weights[(long)row * K + j] = s;
        }
    }
}

#define FORWARD(name, D)                                                                                            \
    extern "C" __global__ void __launch_bounds__(D::WAVES * 64, D::SIMD_WAVES)                                      \
    name(const T *__restrict__ x, long x_ld, const T *__restrict__ w, const int *__restrict__ experts,              \
         const R *__restrict__ weights, const int *__restrict__ order, long N, T *__restrict__ out, long out_ld)    \
    {                                                                                                               \
        product<D>(x, x_ld, w, experts, weights, order, N, out, out_ld, nullptr, 0, nullptr);                       \
    }
FORWARD(cgtp_linear_fwd, Forward)
FORWARD(cgtp_linear_fwd_few, ForwardFew)

// grad_x and the gradient of the weights p: dp[n][j] = <x[n], W^T g[n]>.  w holds the transposed matrices.
#define BACKWARD(name, D)                                                                                           \
    extern "C" __global__ void __launch_bounds__(D::WAVES * 64, D::SIMD_WAVES)                                      \
    name(const T *__restrict__ g, long g_ld, const T *__restrict__ w, const int *__restrict__ experts,              \
         const R *__restrict__ weights, const int *__restrict__ order, long N, T *__restrict__ grad_x,              \
         long grad_x_ld, const T *__restrict__ x, long x_ld, R *__restrict__ grad_weights)                          \
    {                                                                                                               \
        product<D>(g, g_ld, w, experts, weights, order, N, grad_x, grad_x_ld, grad_weights ? x : nullptr, x_ld,     \
                   grad_weights);                                                                                   \
    }
BACKWARD(cgtp_linear_bwd_x, Backward)
BACKWARD(cgtp_linear_bwd_x_few, BackwardFew)

// every matrix [mul_out][mul_in] transposed, in its place
extern "C" __global__ void __launch_bounds__(256) cgtp_linear_transpose(const T *__restrict__ w, T *__restrict__ wt)
{
    const int i = blockIdx.x * 256 + threadIdx.x;
    if (i >= NUMEL) return;
    int p = 0;
    for (int k = 1; k < NPATH; ++k) p = i >= W_OFF[k] ? k : p;
    const int at = i - W_OFF[p], u = at / W_MO[p], v = at % W_MO[p];
    const long base = (long)blockIdx.y * NUMEL;
    wt[base + i] = w[base + W_OFF[p] + v * W_MI[p] + u];
}
)HIP"
R"HIP(
// ---------------------------------------------------------------- weight gradients
// dW[e][v][u] = sum over the expert's slots of p sum_m g[v][m] x[u][m].  A workgroup takes a stretch of one
// expert's slots and one tile of a path; nodes are the summed index.  Its rows come into LDS along the rows, NODES at a
// time, the next ones on their way in registers while the present ones are multiplied, and p is put to g on the way.
// 16-bit operands take g p rounded to T: one rounding more of each term.

struct Stretch {
    int expert;
    long begin, end;
};

// Stretches are numbered floor(offsets[e] / len) + e upwards for expert e: there is room for each one's
// ceil(count / len), since floor((o + c) / len) - floor(o / len) + 1 is at least that.
DEV Stretch stretch_of(const int *offsets, long count, long len, long number, int lane)
{
    if (!offsets) {
        const long b = number * len;
        return {0, b, b + len < count ? b + len : count};
    }
    int below = 0;
    for (int e0 = 0; e0 < E; e0 += 64) {
        const int e = e0 + lane;
        bool is = false;
        if (e < E) {
            const long o = offsets[e];
            is = (o < 0 ? 0 : o > count ? count : o) / len + e <= number;
        }
        below += __popcll(__ballot(is));
    }
    const int e = below > 0 ? below - 1 : 0;
    long lo = offsets[e], hi = offsets[e + 1];
    lo = lo < 0 ? 0 : lo > count ? count : lo;
    hi = hi < lo ? lo : hi > count ? count : hi;
    const long b = lo + (number - (lo / len + e)) * len;
    return {e, b < lo ? hi : b, b + len < hi ? b + len : hi};
}

// LDS of a workgroup: rows and weights of its stretch's slots, then the nodes at hand
struct Table {
    int row[MAX_STRETCH];  // -1 where a slot has none
    R p[MAX_STRETCH];
};

#if defined(BITS16)
constexpr int OCTET = 8;  // nodes that an operand's lane holds; in LDS a column's eight lie side by side
#else
constexpr int OCTET = 1;
#endif

template <int I> struct Shape {
    static constexpr int P = T_PATH[I], KC = W_K[P], WV = T_WV[I], WU = T_WU[I];
    static constexpr int NV = (T_BV[I] + WV - 1) / WV, NU = (T_BU[I] + WU - 1) / WU;  // blocks of a wave
    static constexpr int V = T_V[I], U = T_U[I], MO = W_MO[P], MI = W_MI[P];
    static constexpr int GC = (MO - V < T_BV[I] * 16 ? MO - V : T_BV[I] * 16) * KC;   // columns of the tile
    static constexpr int XC = (MI - U < T_BU[I] * 16 ? MI - U : T_BU[I] * 16) * KC;
    static constexpr int GP = NV * WV * 16 * KC, XP = NU * WU * 16 * KC;               // and in LDS
    // a node's row in LDS begins 16 banks after the one before, so that a wave's four nodes meet different ones
    static constexpr int PITCH = ((GP + XP) * (int)sizeof(T) + 255) / 256 * 256 / (int)sizeof(T) + 64 / (int)sizeof(T);
    static constexpr int NODES = T_NODES[I], CG = (GC + VEC - 1) / VEC, CX = (XC + VEC - 1) / VEC;
    // No run of columns is cut short: every load is made, of row 0 where there is no node, and what it brought is a zero
    // in LDS.  With a branch around each load 200,000 rows of 64x(0e,1o,2e) in bf16, 2 of 16 experts, took 593 us, this way 347 us.
    static constexpr bool WHOLE = GC % VEC == 0 && XC % VEC == 0;
    static constexpr int UNITS = NODES / OCTET * (CG + CX), ROUNDS = (UNITS + 255) / 256;
};

// What a thread brings of the nodes from `first` on: ROUNDS runs of VEC columns, of OCTET nodes each.
template <int I> DEV void fetch(const T *x, long x_ld, const T *g, long g_ld, const Table &tab, int first, int count,
                                V16 (&v)[Shape<I>::ROUNDS][OCTET])
{
    typedef Shape<I> S;
#pragma unroll
    for (int r = 0; r < S::ROUNDS; ++r) {
        const int at = r * 256 + threadIdx.x, c = at % (S::CG + S::CX);
        const bool out = c < S::CG;
        const int col = (out ? c : c - S::CG) * VEC, left = (out ? S::GC : S::XC) - col;
        const T *base = out ? g + W_GC[S::P] + S::V * S::KC + col : x + W_XC[S::P] + S::U * S::KC + col;
        const long ld = out ? g_ld : x_ld;
#pragma unroll
        for (int o = 0; o < OCTET; ++o) {
            const int node = first + at / (S::CG + S::CX) * OCTET + o;
            const int row = at < S::UNITS && node < count ? tab.row[node] : -1;
            T q[VEC];
            if constexpr (S::WHOLE)
                load_raw<VEC>(base + (row < 0 ? 0 : row) * ld, q);
            else
                load_channels<VEC, 1, false>(base + (row < 0 ? 0 : row) * ld, row < 0 ? 0 : left, q);
#pragma unroll
            for (int i = 0; i < VEC; ++i) v[r][o][i] = q[i];
        }
    }
}

template <int I> DEV void keep(T *lds, const Table &tab, int first, int count, const V16 (&v)[Shape<I>::ROUNDS][OCTET])
{
    typedef Shape<I> S;
#pragma unroll
    for (int r = 0; r < S::ROUNDS; ++r) {
        const int at = r * 256 + threadIdx.x, c = at % (S::CG + S::CX), node = at / (S::CG + S::CX) * OCTET;
        if (at >= S::UNITS) break;
        const bool out = c < S::CG;
        V16 q[OCTET];
#pragma unroll
        for (int o = 0; o < OCTET; ++o) {
            q[o] = v[r][o];
            const bool in = first + node + o < count && (!S::WHOLE || tab.row[first + node + o] >= 0);
            if (S::WHOLE && !(K > 0 && out)) {
#pragma unroll
                for (int i = 0; i < VEC; ++i) q[o][i] = in ? q[o][i] : (T)0;
            }
            if (K > 0 && out) {
                const R p = in ? tab.p[first + node + o] : (R)0;
#pragma unroll
                for (int i = 0; i < VEC; ++i) q[o][i] = in ? (T)((R)v[r][o][i] * p) : (T)0;
            }
        }
        const int col = out ? c * VEC : S::GP + (c - S::CG) * VEC;
        if (OCTET == 1) {
            *reinterpret_cast<V16 *>(lds + node * S::PITCH + col) = q[0];
        } else {
            // columns of eight nodes, eight of them: turned over in registers
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                V16 t;
#pragma unroll
                for (int o = 0; o < OCTET; ++o) t[o % VEC] = q[o][i];
                *reinterpret_cast<V16 *>(lds + node * S::PITCH + (col + i) * OCTET) = t;
            }
        }
    }
}

template <int I> DEV void tile(const T *x, long x_ld, const T *g, long g_ld, const Table &tab, int count, R *part, T *lds)
{
    typedef Shape<I> S;
    constexpr int NV = S::NV, NU = S::NU, KC = S::KC;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int a = lane & 15, quarter = lane >> 4, wv = wave / S::WU, wu = wave % S::WU;
    const bool works = wave < S::WV * S::WU;
    V4 acc[NV][NU];
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int k = 0; k < NU; ++k) acc[j][k] = (V4)(R)0;
    V16 v[S::ROUNDS][OCTET];
    fetch<I>(x, x_ld, g, g_ld, tab, 0, count, v);
    for (int first = 0; first < count; first += S::NODES) {
        __syncthreads();
        keep<I>(lds, tab, first, count, v);
        __syncthreads();
        if (first + S::NODES < count) fetch<I>(x, x_ld, g, g_ld, tab, first + S::NODES, count, v);
        if (!works) continue;
#pragma unroll 1
        for (int n = 0; n < S::NODES; n += 4 * OCTET) {
            const T *row = lds + (n + quarter * OCTET) * S::PITCH;
            const T *gr = row + (wv * NV * 16 + a) * KC * OCTET, *xr = row + (S::GP + (wu * NU * 16 + a) * KC) * OCTET;
#pragma unroll
            for (int m = 0; m < KC; ++m) {
#if defined(BITS16)
                V8 ga[NV], xa[NU];
#pragma unroll
                for (int j = 0; j < NV; ++j) ga[j] = *reinterpret_cast<const V8 *>(gr + (j * 16 * KC + m) * OCTET);
#pragma unroll
                for (int k = 0; k < NU; ++k) xa[k] = *reinterpret_cast<const V8 *>(xr + (k * 16 * KC + m) * OCTET);
#pragma unroll
                for (int j = 0; j < NV; ++j)
#pragma unroll
                    for (int k = 0; k < NU; ++k) acc[j][k] = mfma(ga[j], xa[k], acc[j][k]);
#else
                T ga[NV], xa[NU];
#pragma unroll
                for (int j = 0; j < NV; ++j) ga[j] = gr[j * 16 * KC + m];
#pragma unroll
                for (int k = 0; k < NU; ++k) xa[k] = xr[k * 16 * KC + m];
#pragma unroll
                for (int j = 0; j < NV; ++j)
#pragma unroll
                    for (int k = 0; k < NU; ++k) acc[j][k] = MFMA(ga[j], xa[k], acc[j][k]);
#endif
            }
        }
    }
    if (!works) return;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int k = 0; k < NU; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = sizeof(T) == 8 ? quarter + 4 * i : 4 * quarter + i;
                const int vo = S::V + (wv * NV + j) * 16 + row, uo = S::U + (wu * NU + k) * 16 + a;
                // blocks past the tile belong to the next one
                if ((wv * NV + j) < T_BV[I] && (wu * NU + k) < T_BU[I] && vo < S::MO && uo < S::MI)
                    part[W_OFF[S::P] + vo * S::MI + uo] = acc[j][k][i];
            }
}

template <int I = 0> DEV void tiles(int which, const T *x, long x_ld, const T *g, long g_ld, const Table &tab, int count, R *part,
                                    T *lds)
{
    if constexpr (I < NT) {
        if (which == I)
            tile<I>(x, x_ld, g, g_ld, tab, count, part, lds);
        else
            tiles<I + 1>(which, x, x_ld, g, g_ld, tab, count, part, lds);
    }
}

template <int I = 0> constexpr int tile_elements()
{
    if constexpr (I < NT) {
        constexpr int mine = Shape<I>::NODES * Shape<I>::PITCH, rest = tile_elements<I + 1>();
        return mine > rest ? mine : rest;
    }
    return 0;
}

extern "C" __global__ void __launch_bounds__(256, 2)
cgtp_linear_bwd_w(const T *__restrict__ x, long x_ld, const T *__restrict__ g, long g_ld, const R *__restrict__ weights,
                  const int *__restrict__ slots, const int *__restrict__ offsets, long N, long count, long len,
                  R *__restrict__ part)
{
    __shared__ Table tab;
    __shared__ V16 lds[tile_elements() / VEC];
    // All stretches of the tile that takes longest come first.  With the tiles of a stretch side by side a CU got the same
    // tile every time (four tiles, 32 CUs to an XCD): 378 us for 20,000 rows of 128x(0e,1o,2e,3o) in fp32, this way 255 us, now 229 us (its products
    // alone: 142).
    const long stretches = gridDim.x / NT, number = blockIdx.x % stretches;
    const int which = (int)(blockIdx.x / stretches);
    const Stretch s = stretch_of(offsets, count, len, number, threadIdx.x & 63);
    if (s.begin >= s.end) return;
    const int n = (int)(s.end - s.begin);
    for (int i = threadIdx.x; i < n; i += 256) {
        const long slot = slots ? slots[s.begin + i] : s.begin + i;
        const bool in = slot >= 0 && slot < count;
        tab.row[i] = in ? (int)(slot / KS) : -1;
        tab.p[i] = K > 0 && in ? weights[slot] : (R)1;
    }
    __syncthreads();
    tiles(which, x, x_ld, g, g_ld, tab, n, part + number * NUMEL, reinterpret_cast<T *>(lds));
}

// the stretches of each expert, in their order; zeros for an expert without slots
extern "C" __global__ void __launch_bounds__(256)
cgtp_linear_reduce(const R *__restrict__ part, const int *__restrict__ offsets, long count, long len, T *__restrict__ grad_w)
{
    const int i = blockIdx.x * 256 + threadIdx.x, e = blockIdx.y;
    if (i >= NUMEL) return;
    long lo = offsets ? offsets[e] : 0, hi = offsets ? offsets[e + 1] : count;
    lo = lo < 0 ? 0 : lo > count ? count : lo;
    hi = hi < lo ? lo : hi > count ? count : hi;
    const long first = lo / len + e, n = (hi - lo + len - 1) / len;
    double sum = 0;
#pragma unroll 8
    for (long c = 0; c < n; ++c) sum += (double)part[(first + c) * NUMEL + i];
    grad_w[(long)e * NUMEL + i] = (T)(R)sum;
}
)HIP";

}  // namespace cgtp
