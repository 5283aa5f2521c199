// HIP source of the group norm with its activation over a batch of graphs, channels last: forward and
// backward.  gnorm.cpp puts a configuration's constants and the shared text (row_kernels.h) in front
// of this text and compiles it for gfx950.
//
// Constants of a configuration, beside T, R and ACT:
//   C, GROUPS, W  channels of a row, groups, channels of a group
//   CV            neighbouring channels that a lane takes together
//   P, RW, NS     lanes of a row; rows that a wave takes at once; a lane's slots of CV channels, 64 CV apart
//   GP            the power of two that holds the groups
//   BF, BB        rows that a lane holds in the forward, in the backward
//   NWMAX         most waves of a workgroup
#pragma once

namespace cgtp {

static const char kGroupNormKernels[] = R"HIP(
constexpr int EPL = NS * CV;                 // channels of a lane
constexpr int ES = W % CV == 0 ? CV : 1;     // channels of a group that a lane adds before it hands them on
constexpr int CE = (C + ES - 1) / ES, WE = W / ES, EE = EPL / ES;  // a row's, a group's and a lane's such sums
constexpr int BATCH = EPL <= 4 ? 4 : 2;      // rows that a lane has in flight along a chunk

#define EACH(i) _Pragma("unroll") for (int i = 0; i < EPL; ++i)

// Two ways over the rows, in the same launches, since the graphs' sizes are known on the device alone.
//
// A graph of up to `cap` rows (waves x RW x a lane's rows) is one workgroup's: its rows stay in registers from
// the statistics to the result, so they are read once.  Larger graphs are dealt out in chunks of `rows`
// neighbouring rows whatever graphs they are of: a chunk's share of a graph is a piece, the first launch leaves each
// piece's sums and the second joins a graph's pieces, every workgroup for itself (at most 1,024 of them, from
// the L2), and finishes its rows.  Piece numbers chunk + graph are all different, since from one piece to the next the
// chunk or the graph goes up.

DEV long clamped(long v, long n) { return v < 0 ? 0 : v > n ? n : v; }

// The first graph that ends behind `row` (S where none does), by 64 probes at a time.
DEV int find_graph(const int *ptr, int S, long row)
{
    const int lane = threadIdx.x & 63;
    int lo = -1, hi = S;
    while (hi - lo > 1) {
        const int step = (hi - lo + 63) / 64;
        const long p = lo + (lane + 1L) * step;
        const bool ends = p < hi && (long)ptr[p + 1] <= row;
        lo += __popcll(__ballot(ends)) * step;
        hi = hi < lo + step ? hi : lo + step;
    }
    return hi;
}

// The first graph from s on with more than `cap` rows, S where none begins before row `end`.
DEV int find_large(const int *ptr, int S, long N, long cap, int s, long end)
{
    const int lane = threadIdx.x & 63;
    for (; s < S; s += 64) {
        const int g = s + lane;
        const long lo = g < S ? clamped(ptr[g], N) : N, hi = g < S ? clamped(ptr[g + 1], N) : 0;
        const unsigned long long large = __ballot(lo < end && hi - lo > cap), past = __ballot(lo >= end);
        if (large) return s + __ffsll((long long)large) - 1;
        if (past) break;
    }
    return S;
}

// the rows [a, b) of chunk [c0, c1) in each large graph
#define EACH_PIECE(chunk)                                                                 \
    const long c0 = (long)(chunk) * rows, c1 = c0 + rows < N ? c0 + rows : N;             \
    for (int graph = find_large(ptr, S, N, cap, find_graph(ptr, S, c0), c1); graph < S;   \
         graph = find_large(ptr, S, N, cap, graph + 1, c1))                               \
        if (const long lo = clamped(ptr[graph], N), hi = clamped(ptr[graph + 1], N), a = lo > c0 ? lo : c0, b = hi < c1 ? hi : c1; b > a)

// a thread's place: its lane along the row, its row of those that the workgroup takes at once (RG), whether it has one
struct Place {
    int lane, row, RG;
    bool on;
};
DEV Place place()
{
    const int l = threadIdx.x & 63, wave = threadIdx.x >> 6;
    return {l % P, wave * RW + l / P, (int)(blockDim.x >> 6) * RW, l / P < RW};
}

// The lane's channels of slot J: a row's last CV channels where its own would reach past the end.  Two lanes then
// hold some channels both, with the same values, and write the same where they write.
DEV int first_channel(int lane, int slot)
{
    const int at = (slot * 64 + lane) * CV;
    return C % CV == 0 && (NS == 1 || C % (64 * CV) == 0) ? at : at < C - CV ? at : C - CV;
}
DEV int channel(int lane, int i) { return first_channel(lane, i / CV) + i % CV; }

template <int J = 0, typename S, typename X> DEV void load_row(const S *row, int lane, X *x)
{
    if constexpr (J < NS) {
        load_run<CV>(row + first_channel(lane, J), x + J * CV);
        load_row<J + 1>(row, lane, x);
    }
}

template <int J = 0, typename S> DEV void store_row(S *row, int lane, const R *x)
{
    if constexpr (J < NS) {
        store_run<CV>(row + first_channel(lane, J), x + J * CV);
        store_row<J + 1>(row, lane, x);
    }
}

// a row's channels of a lane as they are in memory
struct Raw {
    typedef T V __attribute__((ext_vector_type(CV)));
    V v[NS];
    __device__ __forceinline__ R at(int i) const { return (R)v[i / CV][i % CV]; }
};
DEV void load_raw(const T *row, int lane, Raw &x)
{
    typedef T V __attribute__((ext_vector_type(CV), aligned(sizeof(T))));
#pragma unroll
    for (int j = 0; j < NS; ++j) x.v[j] = *reinterpret_cast<const V *>(row + first_channel(lane, j));
}

// one value per channel, `none` where there are none
DEV void load_channels(const R *w, int lane, R none, R (&x)[EPL])
{
    if (w)
        load_row(w, lane, x);
    else
        EACH(i) x[i] = none;
}

// one value per group, of the lane's channels
DEV void load_groups(const R *v, int lane, R (&x)[EPL])
{
    EACH(i) x[i] = v[channel(lane, i) / W];
}

// (n, m, q) and (k, km, kq): counts, means and sums of squared distances from them, joined into the first
DEV void merge(R &n, R &m, R &q, R k, R km, R kq)
{
    const R all = n + k;
    if (all > (R)0) {
        const R share = k / all, d = km - m;
        m += d * share;
        q += kq + d * d * (n * share);
        n = all;
    }
}

// sum over the first `width` lanes (a power of two up to 64) that a lane is one of
DEV R lanes_sum(R v, int width)
{
    if (width >= 2) v += dpp<0xB1>(v);    // quad_perm 1,0,3,2
    if (width >= 4) v += dpp<0x4E>(v);    // quad_perm 2,3,0,1
    if (width >= 8) v += dpp<0x141>(v);   // row_half_mirror
    if (width >= 16) v += dpp<0x140>(v);  // row_mirror
    if (width >= 32) v = swap16(v);
    if (width >= 64) v = swap32(v);
    return v;
}

// LDS of a workgroup: `sums` holds a lane's sums (NW x 64 x EE for each of NV quantities), `total` [NV][GROUPS] the
// groups', `part` those of the waves that share one.
extern __shared__ double shared[];

// The groups' totals of NV quantities that lanes hold per channel.  Threads share out the groups, or the
// groups the threads; sums run in a fixed order.  `total` may be read until the next call, whose first barrier comes
// before it is written again.
template <int NV> DEV void group_totals(const Place &at, const R (&v)[NV][EPL], R *sums, R *part, R *total)
{
    const int threads = blockDim.x, entries = at.RG * CE;
    if (at.on) {
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int i = 0; i < EE; ++i) {
                R s = v[k][i * ES];
#pragma unroll
                for (int j = 1; j < ES; ++j) s += v[k][i * ES + j];
                sums[k * entries + at.row * CE + channel(at.lane, i * ES) / ES] = s;
            }
    }
    __syncthreads();
    const int tg = threads >= GP ? threads / GP : 1, q = threadIdx.x % tg, pw = tg > 64 ? tg / 64 : 1;
    for (int g = threadIdx.x / tg; g < GP; g += threads / tg) {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            R s = 0;
            if (g < GROUPS)
                for (int e = q; e < at.RG * WE; e += tg) s += sums[k * entries + e / WE * CE + g * WE + e % WE];
            s = lanes_sum(s, tg < 64 ? tg : 64);
            if (g < GROUPS && (q & 63) == 0) (pw > 1 ? part : total)[(k * GROUPS + g) * pw + (q >> 6)] = s;
        }
    }
    __syncthreads();
    if (pw > 1) {
        for (int i = threadIdx.x; i < NV * GROUPS; i += threads) {
            R s = 0;
            for (int j = 0; j < pw; ++j) s += part[i * pw + j];
            total[i] = s;
        }
        __syncthreads();
    }
}

#define SHARED_SETUP(NV)                                            \
    R *const sums = reinterpret_cast<R *>(shared);                  \
    R *const total = sums + (NV) * (int)(blockDim.x >> 6) * RW * CE; \
    R *const part_sums = total + (NV) * GROUPS;

// zeros into the chunk's rows of no graph
DEV void clear_rest(T *y, long ld, const int *ptr, int S, long N, long rows, long chunk)
{
    const Place at = place();
    const long c0 = chunk * rows, c1 = c0 + rows < N ? c0 + rows : N;
    const long head = clamped(ptr[0], N), tail = clamped(ptr[S], N);
    R none[EPL];
    EACH(i) none[i] = (R)0;
    if (!at.on || (c0 >= head && c1 <= tail)) return;
    for (long row = c0 + at.row; row < c1; row += at.RG)
        if (row < head || row >= tail) store_row(y + row * ld, at.lane, none);
}

// ---------------------------------------------------------------- forward
DEV R inverse_root(R v) { return (R)1 / sqrt(v); }

// The first S workgroups take a graph each; the others leave mean and sum of squared distances of the large graphs'
// pieces.
extern "C" __global__ void __launch_bounds__(64 * NWMAX)
cgtp_gnorm_fwd(const T *__restrict__ x, long ld, const int *__restrict__ ptr, int S, long N, long rows, long cap,
               const R *__restrict__ w, const R *__restrict__ bias, T *__restrict__ y, long y_ld, int fill,
               R *__restrict__ mean, R *__restrict__ rstd, R *__restrict__ piece, R eps)
{
    SHARED_SETUP(1)
    const Place at = place();
    if ((int)blockIdx.x >= S) {
        const int chunk = (int)blockIdx.x - S;
        if (fill) clear_rest(y, y_ld, ptr, S, N, rows, chunk);
        EACH_PIECE(chunk)
        {
            // A lane takes the mean and the squared distances of a batch of rows and joins them with those before:
            // no squares of values far from their mean are summed, so a mean much larger than the spread costs no digits.
            R m[EPL], d[1][EPL], n = 0;
            EACH(i) m[i] = d[0][i] = (R)0;
            if (at.on)
                for (long row = a + at.row; row < b; row += at.RG * BATCH) {
                    R v[BATCH][EPL];
                    int k = 0;
#pragma unroll
                    for (int t = 0; t < BATCH; ++t) {
                        const bool in = row + t * at.RG < b;
                        k += in;
                        load_row(x + (in ? row + t * at.RG : row) * ld, at.lane, v[t]);
                    }
                    const R inv = (R)1 / (R)k, all = n + (R)k, share = (R)k / all, both = n * share;
                    EACH(i)
                    {
                        R bm = v[0][i], bq = 0;
#pragma unroll
                        for (int t = 1; t < BATCH; ++t) bm += t < k ? v[t][i] : (R)0;
                        bm *= inv;
#pragma unroll
                        for (int t = 0; t < BATCH; ++t) {
                            const R o = t < k ? v[t][i] - bm : (R)0;
                            bq = fma(o, o, bq);
                        }
                        const R o = bm - m[i];
                        m[i] = fma(o, share, m[i]);
                        d[0][i] += fma(o * o, both, bq);
                    }
                    n = all;
                }
            R s[1][EPL], gm[EPL];
            EACH(i) s[0][i] = n * m[i];
            group_totals<1>(at, s, sums, part_sums, total);
            const R inv = (R)1 / (R)((b - a) * W);
            load_groups(total, at.lane, gm);
            R *out = piece + ((long)chunk + graph) * GROUPS * 2;
            EACH(i)
            {
                gm[i] *= inv;
                const R o = m[i] - gm[i];
                d[0][i] = n > (R)0 ? fma(n * o, o, d[0][i]) : (R)0;
            }
            for (int g = threadIdx.x; g < GROUPS; g += blockDim.x) out[g * 2] = total[g] * inv;
            group_totals<1>(at, d, sums, part_sums, total);
            for (int g = threadIdx.x; g < GROUPS; g += blockDim.x) out[g * 2 + 1] = total[g];
        }
        return;
    }
    const long g0 = blockIdx.x;
    const long lo = clamped(ptr[g0], N), hi = clamped(ptr[g0 + 1], N), n = hi - lo;
    if (n > cap) return;
    if (n <= 0) {
        for (int g = threadIdx.x; g < GROUPS; g += blockDim.x) {
            mean[g0 * GROUPS + g] = (R)0;
            rstd[g0 * GROUPS + g] = inverse_root(eps);
        }
        return;
    }
    // The rows stay as they are in memory, 16-bit ones in half the registers: more graphs fit a CU at once.
    Raw v[BF];
    R s[1][EPL], m[EPL];
    const int left = at.on ? (int)n - at.row : 0;  // of its rows and those behind them
    const T *px = x + (lo + at.row) * ld;
#pragma unroll
    for (int t = 0; t < BF; ++t, px += at.RG * ld) {
        if (t * at.RG < left)
            load_raw(px, at.lane, v[t]);
        else
#pragma unroll
            for (int j = 0; j < NS; ++j) v[t].v[j] = (Raw::V)(T)0;
    }
    EACH(i) s[0][i] = (R)0;
#pragma unroll
    for (int t = 0; t < BF; ++t) EACH(i) s[0][i] += v[t].at(i);
    group_totals<1>(at, s, sums, part_sums, total);
    const R inv = (R)1 / (R)(n * W);
    load_groups(total, at.lane, m);
    EACH(i)
    {
        m[i] *= inv;
        s[0][i] = (R)0;
    }
#pragma unroll
    for (int t = 0; t < BF; ++t)
        if (t * at.RG < left) EACH(i)
        {
            const R o = v[t].at(i) - m[i];
            s[0][i] = fma(o, o, s[0][i]);
        }
    for (int g = threadIdx.x; g < GROUPS; g += blockDim.x) mean[g0 * GROUPS + g] = total[g] * inv;
    group_totals<1>(at, s, sums, part_sums, total);
    R k[EPL], wc[EPL], bc[EPL];
    load_groups(total, at.lane, k);
    load_channels(w, at.lane, (R)1, wc);
    load_channels(bias, at.lane, (R)0, bc);
    EACH(i) k[i] = inverse_root(fma(k[i], inv, eps)) * wc[i];
    for (int g = threadIdx.x; g < GROUPS; g += blockDim.x) rstd[g0 * GROUPS + g] = inverse_root(fma(total[g], inv, eps));
    T *py = y + (lo + at.row) * y_ld;
#pragma unroll
    for (int t = 0; t < BF; ++t, py += at.RG * y_ld) {
        if (t * at.RG >= left) continue;
        R o[EPL];
        EACH(i) o[i] = act_value(fma(v[t].at(i) - m[i], k[i], bc[i]));
        store_row(py, at.lane, o);
    }
}

// The large graphs' chunks: a graph's pieces joined, in lanes that take pieces in turn and then by a tree, and its
// rows finished.  The workgroup that has a graph's first row stores its statistics.
extern "C" __global__ void __launch_bounds__(64 * NWMAX)
cgtp_gnorm_fwd_large(const T *__restrict__ x, long ld, const int *__restrict__ ptr, int S, long N, long rows, long cap,
                     const R *__restrict__ w, const R *__restrict__ bias, const R *__restrict__ piece,
                     T *__restrict__ y, long y_ld, R *__restrict__ mean, R *__restrict__ rstd, R eps)
{
    R *const ln = reinterpret_cast<R *>(shared), *const lm = ln + blockDim.x, *const lq = lm + blockDim.x;
    R *const gm = lq + blockDim.x, *const gr = gm + GROUPS;
    const Place at = place();
    EACH_PIECE(blockIdx.x)
    {
        const int threads = blockDim.x, tg = threads >= GP ? threads / GP : 1, j = threadIdx.x / (threads / tg);
        const long first = lo / rows, last = (hi - 1) / rows;
        for (int g = threadIdx.x % (threads / tg); g < GP; g += threads / tg) {
            R n = 0, m = 0, q = 0;
            if (g < GROUPS) {
#pragma unroll 4
                for (long c = first + j; c <= last; c += tg) {
                    const long pa = lo > c * rows ? lo : c * rows, pb = hi < (c + 1) * rows ? hi : (c + 1) * rows;
                    const R *in = piece + ((c + graph) * GROUPS + g) * 2;
                    merge(n, m, q, (R)((pb - pa) * W), in[0], in[1]);
                }
            }
            for (int half = tg / 2; half > 0; half /= 2) {
                __syncthreads();
                ln[threadIdx.x] = n;
                lm[threadIdx.x] = m;
                lq[threadIdx.x] = q;
                __syncthreads();
                if (j < half) {
                    const int o = threadIdx.x + half * (threads / tg);
                    merge(n, m, q, ln[o], lm[o], lq[o]);
                }
            }
            if (j == 0 && g < GROUPS) {
                gm[g] = m;
                gr[g] = inverse_root(q / n + eps);
                if (a == lo) {
                    mean[(long)graph * GROUPS + g] = m;
                    rstd[(long)graph * GROUPS + g] = gr[g];
                }
            }
        }
        __syncthreads();
        R m[EPL], k[EPL], wc[EPL], bc[EPL];
        load_groups(gm, at.lane, m);
        load_groups(gr, at.lane, k);
        load_channels(w, at.lane, (R)1, wc);
        load_channels(bias, at.lane, (R)0, bc);
        EACH(i) k[i] *= wc[i];
        if (at.on)
            for (long row = a + at.row; row < b; row += at.RG * BATCH) {
                R v[BATCH][EPL];
#pragma unroll
                for (int t = 0; t < BATCH; ++t)
                    load_row(x + (row + t * at.RG < b ? row + t * at.RG : row) * ld, at.lane, v[t]);
#pragma unroll
                for (int t = 0; t < BATCH; ++t) {
                    EACH(i) v[t][i] = act_value(fma(v[t][i] - m[i], k[i], bc[i]));
                    if (row + t * at.RG < b) store_row(y + (row + t * at.RG) * y_ld, at.lane, v[t]);
                }
            }
        __syncthreads();
    }
}

// ---------------------------------------------------------------- backward
// dz = dy act'(z), q = dz w, with k = rstd w:  o = x - mean and dz of a row, from its x and dy.  xh = o rstd is left to the
// sums, which are multiplied by rstd once.
DEV void slopes(int lane, const R (&m)[EPL], const R (&k)[EPL], const R (&bc)[EPL], R (&o)[EPL], R (&dz)[EPL])
{
    EACH(i)
    {
        R value;
        o[i] -= m[i];
        dz[i] *= act_slope(fma(o[i], k[i], bc[i]), value);
    }
}

// m, k and the bias of the lane's channels in graph s
DEV void load_graph(const R *mean, const R *rstd, const R *w, const R *bias, long s, int lane, R (&m)[EPL], R (&k)[EPL], R (&bc)[EPL])
{
    R rs[EPL];
    load_groups(mean + s * GROUPS, lane, m);
    load_groups(rstd + s * GROUPS, lane, rs);
    load_channels(w, lane, (R)1, k);
    load_channels(bias, lane, (R)0, bc);
    EACH(i) k[i] *= rs[i];
}

// Sums v of dz and dz o over a graph's rows: into the weights' (which are of dz xh), then q's and q xh's.
DEV void through_weights(const R *rstd, const R *w, long s, int lane, R (&tw)[EPL], R (&tb)[EPL], R (&v)[2][EPL])
{
    R rs[EPL], wc[EPL];
    load_groups(rstd + s * GROUPS, lane, rs);
    load_channels(w, lane, (R)1, wc);
    EACH(i)
    {
        v[1][i] *= rs[i];
        tb[i] += v[0][i];
        tw[i] += v[1][i];
        v[0][i] *= wc[i];
        v[1][i] *= wc[i];
    }
}

// dx = rstd (q - mean q - xh mean(q xh)) = dz k - c0 - o c1, from the means in v
DEV void dx_terms(const R *rstd, long s, int lane, R (&v)[2][EPL])
{
    R rs[EPL];
    load_groups(rstd + s * GROUPS, lane, rs);
    EACH(i)
    {
        v[0][i] *= rs[i];
        v[1][i] *= rs[i] * rs[i];
    }
}

// the workgroup's sums of dz xh and dz per channel, of all its rows
DEV void channel_sums(const Place &at, const R (&tw)[EPL], const R (&tb)[EPL], R *lds, R *out)
{
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        __syncthreads();
        if (at.on) EACH(i) lds[at.row * C + channel(at.lane, i)] = k == 0 ? tw[i] : tb[i];
        __syncthreads();
        for (int c = threadIdx.x; c < C; c += blockDim.x) {
            R s = 0;
            for (int r = 0; r < at.RG; ++r) s += lds[r * C + c];
            out[k * C + c] = s;
        }
    }
}

// The first `graphs` workgroups take graphs in turn; the others leave the sums of q and q xh of the large graphs'
// pieces.  Each leaves its sums of dz xh and dz per channel in wpart.
extern "C" __global__ void __launch_bounds__(64 * NWMAX)
cgtp_gnorm_bwd(const T *__restrict__ x, long ld, const T *__restrict__ dy, long dy_ld, const int *__restrict__ ptr, int S,
               long N, long rows, int graphs, long cap, const R *__restrict__ w, const R *__restrict__ bias,
               const R *__restrict__ mean, const R *__restrict__ rstd, T *__restrict__ dx, long dx_ld, int fill,
               R *__restrict__ piece, R *__restrict__ wpart)
{
    SHARED_SETUP(2)
    const Place at = place();
    R tw[EPL], tb[EPL];
    EACH(i) tw[i] = tb[i] = (R)0;
    if ((int)blockIdx.x >= graphs) {
        const int chunk = (int)blockIdx.x - graphs;
        if (dx && fill) clear_rest(dx, dx_ld, ptr, S, N, rows, chunk);
        EACH_PIECE(chunk)
        {
            R m[EPL], k[EPL], bc[EPL], v[2][EPL];
            load_graph(mean, rstd, w, bias, graph, at.lane, m, k, bc);
            EACH(i) v[0][i] = v[1][i] = (R)0;
            if (at.on)
                for (long row = a + at.row; row < b; row += at.RG * BATCH) {
                    R o[BATCH][EPL], dz[BATCH][EPL];
#pragma unroll
                    for (int t = 0; t < BATCH; ++t) {
                        const long n = row + t * at.RG < b ? row + t * at.RG : row;
                        load_row(x + n * ld, at.lane, o[t]);
                        load_row(dy + n * dy_ld, at.lane, dz[t]);
                    }
#pragma unroll
                    for (int t = 0; t < BATCH; ++t) {
                        slopes(at.lane, m, k, bc, o[t], dz[t]);
                        if (row + t * at.RG < b) EACH(i)
                        {
                            v[0][i] += dz[t][i];
                            v[1][i] = fma(dz[t][i], o[t][i], v[1][i]);
                        }
                    }
                }
            through_weights(rstd, w, graph, at.lane, tw, tb, v);
            if (dx) {
                group_totals<2>(at, v, sums, part_sums, total);
                R *out = piece + ((long)chunk + graph) * GROUPS * 2;
                for (int g = threadIdx.x; g < GROUPS; g += blockDim.x) {
                    out[g * 2] = total[g];
                    out[g * 2 + 1] = total[GROUPS + g];
                }
            }
        }
    } else {
        for (long g0 = blockIdx.x; g0 < S; g0 += graphs) {
            const long lo = clamped(ptr[g0], N), hi = clamped(ptr[g0 + 1], N), n = hi - lo;
            if (n > cap || n <= 0) continue;
            R m[EPL], k[EPL], bc[EPL], v[2][EPL], o[BB][EPL], dz[BB][EPL];
            const int left = at.on ? (int)n - at.row : 0;  // of its rows and those behind them
            const T *px = x + (lo + at.row) * ld, *pd = dy + (lo + at.row) * dy_ld;
#pragma unroll
            for (int t = 0; t < BB; ++t, px += at.RG * ld, pd += at.RG * dy_ld) {
                if (t * at.RG < left) {
                    load_row(px, at.lane, o[t]);
                    load_row(pd, at.lane, dz[t]);
                } else {
                    EACH(i) o[t][i] = dz[t][i] = (R)0;
                }
            }
            load_graph(mean, rstd, w, bias, g0, at.lane, m, k, bc);
            EACH(i) v[0][i] = v[1][i] = (R)0;
#pragma unroll
            for (int t = 0; t < BB; ++t)
                if (t * at.RG < left) {
                    slopes(at.lane, m, k, bc, o[t], dz[t]);
                    EACH(i)
                    {
                        v[0][i] += dz[t][i];
                        v[1][i] = fma(dz[t][i], o[t][i], v[1][i]);
                    }
                }
            through_weights(rstd, w, g0, at.lane, tw, tb, v);
            if (!dx) continue;
            group_totals<2>(at, v, sums, part_sums, total);
            const R inv = (R)1 / (R)(n * W);
            load_groups(total, at.lane, v[0]);
            load_groups(total + GROUPS, at.lane, v[1]);
            EACH(i)
            {
                v[0][i] *= inv;
                v[1][i] *= inv;
            }
            dx_terms(rstd, g0, at.lane, v);
            T *po = dx + (lo + at.row) * dx_ld;
#pragma unroll
            for (int t = 0; t < BB; ++t, po += at.RG * dx_ld) {
                if (t * at.RG >= left) continue;
                EACH(i) dz[t][i] = dz[t][i] * k[i] - v[0][i] - o[t][i] * v[1][i];
                store_row(po, at.lane, dz[t]);
            }
        }
    }
    if (wpart) channel_sums(at, tw, tb, sums, wpart + (long)blockIdx.x * 2 * C);
}

// The workgroups' sums per channel, added in double: 16 columns of [count][2C].
DEV void add_columns(int block, const R *wpart, long count, R *gw, R *gb)
{
    double *const lds = shared;
    const int col = block * 16 + threadIdx.x % 16, j = threadIdx.x / 16, step = blockDim.x / 16;
    double sum = 0;
    if (col < 2 * C) {
#pragma unroll 8
        for (long c = j; c < count; c += step) sum += (double)wpart[c * 2 * C + col];
    }
    lds[threadIdx.x] = sum;
    for (int half = step / 2; half > 0; half /= 2) {
        __syncthreads();
        if (j < half) lds[threadIdx.x] += lds[threadIdx.x + half * 16];
    }
    if (j == 0 && col < 2 * C) {
        if (col < C && gw) gw[col] = (R)lds[threadIdx.x];
        if (col >= C && gb) gb[col - C] = (R)lds[threadIdx.x];
    }
}

// The first `columns` workgroups add the weights' gradients; the others finish the large graphs' chunks:
// dx = rstd (q - mean q - xh mean(q xh)).
extern "C" __global__ void __launch_bounds__(64 * NWMAX)
cgtp_gnorm_bwd_large(const T *__restrict__ x, long ld, const T *__restrict__ dy, long dy_ld, const int *__restrict__ ptr,
                     int S, long N, long rows, long cap, const R *__restrict__ w, const R *__restrict__ bias,
                     const R *__restrict__ mean, const R *__restrict__ rstd, const R *__restrict__ piece, T *__restrict__ dx,
                     long dx_ld, int columns, const R *__restrict__ wpart, long count, R *__restrict__ gw, R *__restrict__ gb)
{
    if ((int)blockIdx.x < columns) {
        add_columns(blockIdx.x, wpart, count, gw, gb);
        return;
    }
    R *const l0 = reinterpret_cast<R *>(shared), *const l1 = l0 + blockDim.x, *const g0s = l1 + blockDim.x, *const g1s = g0s + GROUPS;
    const Place at = place();
    EACH_PIECE((int)blockIdx.x - columns)
    {
        const int threads = blockDim.x, tg = threads >= GP ? threads / GP : 1, j = threadIdx.x / (threads / tg);
        const long first = lo / rows, last = (hi - 1) / rows;
        const R inv = (R)1 / (R)((hi - lo) * W);
        for (int g = threadIdx.x % (threads / tg); g < GP; g += threads / tg) {
            R a0 = 0, a1 = 0;
            if (g < GROUPS) {
#pragma unroll 8
                for (long c = first + j; c <= last; c += tg) {
                    const R *in = piece + ((c + graph) * GROUPS + g) * 2;
                    a0 += in[0];
                    a1 += in[1];
                }
            }
            for (int half = tg / 2; half > 0; half /= 2) {
                __syncthreads();
                l0[threadIdx.x] = a0;
                l1[threadIdx.x] = a1;
                __syncthreads();
                if (j < half) {
                    a0 += l0[threadIdx.x + half * (threads / tg)];
                    a1 += l1[threadIdx.x + half * (threads / tg)];
                }
            }
            if (j == 0 && g < GROUPS) {
                g0s[g] = a0 * inv;
                g1s[g] = a1 * inv;
            }
        }
        __syncthreads();
        R m[EPL], k[EPL], bc[EPL], v[2][EPL];
        load_graph(mean, rstd, w, bias, graph, at.lane, m, k, bc);
        load_groups(g0s, at.lane, v[0]);
        load_groups(g1s, at.lane, v[1]);
        dx_terms(rstd, graph, at.lane, v);
        if (at.on)
            for (long row = a + at.row; row < b; row += at.RG * BATCH) {
                R o[BATCH][EPL], dz[BATCH][EPL];
#pragma unroll
                for (int t = 0; t < BATCH; ++t) {
                    const long n = row + t * at.RG < b ? row + t * at.RG : row;
                    load_row(x + n * ld, at.lane, o[t]);
                    load_row(dy + n * dy_ld, at.lane, dz[t]);
                }
#pragma unroll
                for (int t = 0; t < BATCH; ++t) {
                    slopes(at.lane, m, k, bc, o[t], dz[t]);
                    EACH(i) dz[t][i] = dz[t][i] * k[i] - v[0][i] - o[t][i] * v[1][i];
                    if (row + t * at.RG < b) store_row(dx + (row + t * at.RG) * dx_ld, at.lane, dz[t]);
                }
            }
        __syncthreads();
    }
}
)HIP";

}  // namespace cgtp
