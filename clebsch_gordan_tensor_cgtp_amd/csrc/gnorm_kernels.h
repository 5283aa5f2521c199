// HIP source of the group norm with its activation over a batch of graphs, channels last: forward and
// backward.  gnorm.cpp puts a configuration's constants and the shared text (row_kernels.h) in front
// of this text and compiles it for gfx950.
//
// Constants of a configuration, beside T, R and ACT:
//   C, GROUPS, W  channels of a row, groups, channels of a group
//   CV            neighbouring channels that a lane takes together
//   P, RW, NS     lanes of a row; rows that a wave takes at once; a lane's slots of CV channels, 64 CV apart
//   GL            groups reduced at a time: the power of two that holds them, at most 64
//   CHUNK_LDS     elements of a workgroup's LDS sums
#pragma once

namespace cgtp {

static const char kGroupNormKernels[] = R"HIP(
constexpr int EPL = NS * CV;       // channels of a lane
constexpr int LG = 64 / GL;        // lanes that reduce a group
constexpr int ENTRIES = RW * W;    // lane sums of a group
constexpr int BATCH = EPL <= 8 ? 4 : 2;  // rows that a lane has in flight

#define EACH(i) _Pragma("unroll") for (int i = 0; i < EPL; ++i)

// A wave is a workgroup and takes `rows` neighbouring rows, whatever graphs they belong to: no wave waits for
// another, and a batch of one huge graph is shared as evenly as one of thousands of small ones.  A
// wave's share of a graph is a piece; piece numbers chunk + graph are all different, since from one piece to
// the next the chunk or the graph goes up.

// The first graph that ends behind `row` (S where none does), by 64 probes at a time.
DEV int find_graph(const int *ptr, int S, long row, int lane)
{
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

DEV long clamped(long v, long n) { return v < 0 ? 0 : v > n ? n : v; }

// the rows [a, b) of chunk [c0, c1) in graph s; empty ones are passed over
#define EACH_PIECE                                                                        \
    const int lane = threadIdx.x % P, r = threadIdx.x / P;                                \
    const long c0 = (long)blockIdx.x * rows, c1 = c0 + rows < N ? c0 + rows : N;          \
    for (int s = find_graph(ptr, S, c0, threadIdx.x); s < S; ++s)                         \
        if (const long lo = clamped(ptr[s], N); lo >= c1)                                 \
            break;                                                                        \
        else if (const long hi = clamped(ptr[s + 1], N), a = lo > c0 ? lo : c0, b = hi < c1 ? hi : c1; b > a)

template <int J = 0, typename S> DEV void load_row(const S *row, int lane, R *x)
{
    if constexpr (J < NS) {
        const int at = (J * 64 + lane) * CV;
        constexpr int LAST = C % CV;
        if ((J + 1) * 64 * CV <= C || at + CV <= C) {
            load_run<CV>(row + at, x + J * CV);
        } else {
#pragma unroll
            for (int i = 0; i < CV; ++i) x[J * CV + i] = (R)0;
            if (LAST > 0 && at < C) load_run<LAST>(row + at, x + J * CV);
        }
        load_row<J + 1>(row, lane, x);
    }
}

template <int J = 0, typename S> DEV void store_row(S *row, int lane, const R *x)
{
    if constexpr (J < NS) {
        const int at = (J * 64 + lane) * CV;
        constexpr int LAST = C % CV;
        if ((J + 1) * 64 * CV <= C || at + CV <= C)
            store_run<CV>(row + at, x + J * CV);
        else if (LAST > 0 && at < C)
            store_run<LAST>(row + at, x + J * CV);
        store_row<J + 1>(row, lane, x);
    }
}

DEV int channel(int lane, int i) { return ((i / CV) * 64 + lane) * CV + i % CV; }

// one value per channel, `none` where there are none or past the row's end
DEV void load_channels(const R *w, int lane, R none, R (&x)[EPL])
{
    EACH(i)
    {
        const int c = channel(lane, i);
        x[i] = w && c < C ? w[c] : none;
    }
}

// one value per group, of the lane's channels; every `stride`-th
DEV void load_groups(const R *v, int stride, int lane, R (&x)[EPL])
{
    EACH(i)
    {
        const int c = channel(lane, i);
        x[i] = v[(c < C ? c / W : 0) * stride];
    }
}

DEV void keep(R *lds, int r, int lane, const R (&x)[EPL])
{
    if (r < RW) EACH(i)
    {
        const int c = channel(lane, i);
        if (c < C) lds[r * C + c] = x[i];
    }
}

// sum over the LG lanes of a group
DEV R lanes_sum(R v)
{
    if (LG >= 2) v += dpp<0xB1>(v);    // quad_perm 1,0,3,2
    if (LG >= 4) v += dpp<0x4E>(v);    // quad_perm 2,3,0,1
    if (LG >= 8) v += dpp<0x141>(v);   // row_half_mirror
    if (LG >= 16) v += dpp<0x140>(v);  // row_mirror
    if (LG >= 32) v = swap16(v);
    if (LG >= 64) v = swap32(v);
    return v;
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

// zeros into the chunk's rows of no graph
DEV void clear_rest(T *y, long ld, const int *ptr, int S, long N, long rows)
{
    const int lane = threadIdx.x % P, r = threadIdx.x / P;
    const long c0 = (long)blockIdx.x * rows, c1 = c0 + rows < N ? c0 + rows : N;
    const long head = clamped(ptr[0], N), tail = clamped(ptr[S], N);
    R none[EPL];
    EACH(i) none[i] = (R)0;
    if (r >= RW) return;
    for (long row = c0 + r; row < c1; row += RW)
        if (row < head || row >= tail) store_row(y + row * ld, lane, none);
}

// ---------------------------------------------------------------- forward
// Mean and sum of squared distances of every piece and group.  A lane takes the mean and the distances of a
// batch of rows and joins them with those before: no squares of values far from their mean are ever
// summed, so a mean much larger than the spread costs no digits.
extern "C" __global__ void __launch_bounds__(64)
cgtp_gnorm_stats(const T *__restrict__ x, long ld, const int *__restrict__ ptr, int S, long N, long rows,
                 R *__restrict__ part)
{
    __shared__ R lmean[CHUNK_LDS], ldist[CHUNK_LDS];
    EACH_PIECE
    {
        R mean[EPL], dist[EPL], n = 0;
        EACH(i) mean[i] = dist[i] = (R)0;
        if (r < RW)
            for (long row = a + r; row < b; row += RW * BATCH) {
                R v[BATCH][EPL];
                int m = 0;
#pragma unroll
                for (int k = 0; k < BATCH; ++k) {
                    const bool in = row + k * RW < b;
                    m += in;
                    load_row(x + (in ? row + k * RW : row) * ld, lane, v[k]);
                }
                const R inv = (R)1 / (R)m, all = n + (R)m, share = (R)m / all, both = n * share;
                EACH(i)
                {
                    R bm = v[0][i], bq = 0;
#pragma unroll
                    for (int k = 1; k < BATCH; ++k) bm += k < m ? v[k][i] : (R)0;
                    bm *= inv;
#pragma unroll
                    for (int k = 0; k < BATCH; ++k) {
                        const R d = k < m ? v[k][i] - bm : (R)0;
                        bq = fma(d, d, bq);
                    }
                    const R d = bm - mean[i];
                    mean[i] = fma(d, share, mean[i]);
                    dist[i] += fma(d * d, both, bq);
                }
                n = all;
            }
        keep(lmean, r, lane, mean);
        keep(ldist, r, lane, dist);
        __syncthreads();
        const int q = threadIdx.x % LG;
        for (int g0 = 0; g0 < GROUPS; g0 += GL) {
            const int g = g0 + threadIdx.x / LG;
            R sum = 0, ss = 0;
            if (g < GROUPS)
                for (int e = q; e < ENTRIES; e += LG) {
                    const int er = e / W, left = (int)(b - a) - er;
                    const R k = left > 0 ? (R)((left + RW - 1) / RW) : (R)0;
                    sum = fma(k, lmean[er * C + g * W + e % W], sum);
                }
            const R m = lanes_sum(sum) / (R)((b - a) * W);
            if (g < GROUPS)
                for (int e = q; e < ENTRIES; e += LG) {
                    const int er = e / W, left = (int)(b - a) - er;
                    if (left <= 0) continue;
                    const R k = (R)((left + RW - 1) / RW), d = lmean[er * C + g * W + e % W] - m;
                    ss += fma(k * d, d, ldist[er * C + g * W + e % W]);
                }
            ss = lanes_sum(ss);
            if (q == 0 && g < GROUPS) {
                R *out = part + (((long)blockIdx.x + s) * GROUPS + g) * 2;
                out[0] = m;
                out[1] = ss;
            }
        }
        __syncthreads();
    }
}

// The pieces of a graph, one workgroup each graph: lanes take pieces in turn, GL groups side by side, and
// are joined by a tree.
#define JOIN_SETUP                                                                            \
    const int s = blockIdx.x, gl = threadIdx.x % GL, j = threadIdx.x / GL, nj = blockDim.x / GL; \
    const long lo = clamped(ptr[s], N), hi = clamped(ptr[s + 1], N);                          \
    const long first = lo / rows, last = hi > lo ? (hi - 1) / rows : first - 1;

extern "C" __global__ void __launch_bounds__(256)
cgtp_gnorm_join(const int *__restrict__ ptr, long N, long rows, const R *__restrict__ part, R *__restrict__ mean,
                R *__restrict__ rstd, R eps)
{
    __shared__ R ln[256], lm[256], lq[256];
    JOIN_SETUP
    for (int g0 = 0; g0 < GROUPS; g0 += GL) {
        const int g = g0 + gl;
        R n = 0, m = 0, q = 0;
        if (g < GROUPS)
            for (long c = first + j; c <= last; c += nj) {
                const long a = lo > c * rows ? lo : c * rows, b = hi < (c + 1) * rows ? hi : (c + 1) * rows;
                const R *in = part + ((c + s) * GROUPS + g) * 2;
                merge(n, m, q, (R)((b - a) * W), in[0], in[1]);
            }
        for (int half = nj / 2; half > 0; half /= 2) {
            __syncthreads();
            ln[threadIdx.x] = n;
            lm[threadIdx.x] = m;
            lq[threadIdx.x] = q;
            __syncthreads();
            if (j < half) {
                const int o = threadIdx.x + half * GL;
                merge(n, m, q, ln[o], lm[o], lq[o]);
            }
        }
        if (j == 0 && g < GROUPS) {
            if (mean) mean[(long)s * GROUPS + g] = m;
            rstd[(long)s * GROUPS + g] = (R)1 / sqrt((n > (R)0 ? q / n : (R)0) + eps);
        }
    }
}

extern "C" __global__ void __launch_bounds__(64)
cgtp_gnorm_apply(const T *__restrict__ x, long ld, const int *__restrict__ ptr, int S, long N, long rows,
                 const R *__restrict__ w, const R *__restrict__ bias, const R *__restrict__ mean,
                 const R *__restrict__ rstd, T *__restrict__ y, long y_ld, int fill)
{
    if (fill) clear_rest(y, y_ld, ptr, S, N, rows);
    R wc[EPL], bc[EPL];
    load_channels(w, threadIdx.x % P, (R)1, wc);
    load_channels(bias, threadIdx.x % P, (R)0, bc);
    EACH_PIECE
    {
        R m[EPL], k[EPL];
        load_groups(mean + (long)s * GROUPS, 1, lane, m);
        load_groups(rstd + (long)s * GROUPS, 1, lane, k);
        EACH(i) k[i] *= wc[i];
        if (r < RW)
            for (long row = a + r; row < b; row += RW * BATCH) {
                R v[BATCH][EPL];
#pragma unroll
                for (int t = 0; t < BATCH; ++t) load_row(x + (row + t * RW < b ? row + t * RW : row) * ld, lane, v[t]);
#pragma unroll
                for (int t = 0; t < BATCH; ++t) {
                    EACH(i) v[t][i] = act_value(fma(v[t][i] - m[i], k[i], bc[i]));
                    if (row + t * RW < b) store_row(y + (row + t * RW) * y_ld, lane, v[t]);
                }
            }
    }
}

// ---------------------------------------------------------------- backward
// dz = dy act'(z),  q = dz w:  every piece's and group's sums of q and q xh, and the chunk's sums of dz xh
// and dz per channel.
DEV void slopes(const T *x, const T *dy, int lane, const R (&m)[EPL], const R (&rs)[EPL], const R (&wc)[EPL],
                const R (&bc)[EPL], R (&xh)[EPL], R (&dz)[EPL])
{
    load_row(x, lane, xh);
    load_row(dy, lane, dz);
    EACH(i)
    {
        xh[i] = (xh[i] - m[i]) * rs[i];
        R value;
        dz[i] *= act_slope(fma(xh[i], wc[i], bc[i]), value);
    }
}

extern "C" __global__ void __launch_bounds__(64)
cgtp_gnorm_bwd_sums(const T *__restrict__ x, long ld, const T *__restrict__ dy, long dy_ld, const int *__restrict__ ptr,
                    int S, long N, long rows, const R *__restrict__ w, const R *__restrict__ bias,
                    const R *__restrict__ mean, const R *__restrict__ rstd, R *__restrict__ part, R *__restrict__ wpart)
{
    __shared__ R lq[CHUNK_LDS], lx[CHUNK_LDS];
    R wc[EPL], bc[EPL], tw[EPL], tb[EPL];
    load_channels(w, threadIdx.x % P, (R)1, wc);
    load_channels(bias, threadIdx.x % P, (R)0, bc);
    EACH(i) tw[i] = tb[i] = (R)0;
    EACH_PIECE
    {
        R m[EPL], rs[EPL], sq[EPL], sx[EPL];
        load_groups(mean + (long)s * GROUPS, 1, lane, m);
        load_groups(rstd + (long)s * GROUPS, 1, lane, rs);
        EACH(i) sq[i] = sx[i] = (R)0;
        if (r < RW)
            for (long row = a + r; row < b; row += RW * BATCH) {
                R xh[BATCH][EPL], dz[BATCH][EPL];
#pragma unroll
                for (int t = 0; t < BATCH; ++t) {
                    const long n = row + t * RW < b ? row + t * RW : row;
                    slopes(x + n * ld, dy + n * dy_ld, lane, m, rs, wc, bc, xh[t], dz[t]);
                }
#pragma unroll
                for (int t = 0; t < BATCH; ++t)
                    if (row + t * RW < b) EACH(i)
                    {
                        sq[i] += dz[t][i];
                        sx[i] = fma(dz[t][i], xh[t][i], sx[i]);
                    }
            }
        EACH(i)
        {
            tb[i] += sq[i];
            tw[i] += sx[i];
            sq[i] *= wc[i];
            sx[i] *= wc[i];
        }
        keep(lq, r, lane, sq);
        keep(lx, r, lane, sx);
        __syncthreads();
        const int q = threadIdx.x % LG;
        for (int g0 = 0; g0 < GROUPS; g0 += GL) {
            const int g = g0 + threadIdx.x / LG;
            R a0 = 0, a1 = 0;
            if (g < GROUPS)
                for (int e = q; e < ENTRIES; e += LG) {
                    const int at = (e / W) * C + g * W + e % W;
                    a0 += lq[at];
                    a1 += lx[at];
                }
            a0 = lanes_sum(a0);
            a1 = lanes_sum(a1);
            if (q == 0 && g < GROUPS) {
                R *out = part + (((long)blockIdx.x + s) * GROUPS + g) * 2;
                out[0] = a0;
                out[1] = a1;
            }
        }
        __syncthreads();
    }
    if (!wpart) return;
    keep(lq, threadIdx.x / P, threadIdx.x % P, tw);
    keep(lx, threadIdx.x / P, threadIdx.x % P, tb);
    __syncthreads();
    R *out = wpart + (long)blockIdx.x * 2 * C;
    for (int c = threadIdx.x; c < C; c += 64) {
        R a0 = 0, a1 = 0;
#pragma unroll
        for (int k = 0; k < RW; ++k) {
            a0 += lq[k * C + c];
            a1 += lx[k * C + c];
        }
        out[c] = a0;
        out[C + c] = a1;
    }
}

// stat [graphs][GROUPS][2]: means of q and of q xh
extern "C" __global__ void __launch_bounds__(256)
cgtp_gnorm_bwd_join(const int *__restrict__ ptr, long N, long rows, const R *__restrict__ part, R *__restrict__ stat)
{
    __shared__ R l0[256], l1[256];
    JOIN_SETUP
    for (int g0 = 0; g0 < GROUPS; g0 += GL) {
        const int g = g0 + gl;
        R a0 = 0, a1 = 0;
        if (g < GROUPS)
            for (long c = first + j; c <= last; c += nj) {
                const R *in = part + ((c + s) * GROUPS + g) * 2;
                a0 += in[0];
                a1 += in[1];
            }
        for (int half = nj / 2; half > 0; half /= 2) {
            __syncthreads();
            l0[threadIdx.x] = a0;
            l1[threadIdx.x] = a1;
            __syncthreads();
            if (j < half) {
                a0 += l0[threadIdx.x + half * GL];
                a1 += l1[threadIdx.x + half * GL];
            }
        }
        if (j == 0 && g < GROUPS && hi > lo) {
            const R inv = (R)1 / (R)((hi - lo) * W);
            R *out = stat + ((long)s * GROUPS + g) * 2;
            out[0] = a0 * inv;
            out[1] = a1 * inv;
        }
    }
}

// dx = rstd (q - mean q - xh mean(q xh))
extern "C" __global__ void __launch_bounds__(64)
cgtp_gnorm_bwd_apply(const T *__restrict__ x, long ld, const T *__restrict__ dy, long dy_ld,
                     const int *__restrict__ ptr, int S, long N, long rows, const R *__restrict__ w,
                     const R *__restrict__ bias, const R *__restrict__ mean, const R *__restrict__ rstd,
                     const R *__restrict__ stat, T *__restrict__ dx, long dx_ld, int fill)
{
    if (fill) clear_rest(dx, dx_ld, ptr, S, N, rows);
    R wc[EPL], bc[EPL];
    load_channels(w, threadIdx.x % P, (R)1, wc);
    load_channels(bias, threadIdx.x % P, (R)0, bc);
    EACH_PIECE
    {
        R m[EPL], rs[EPL], mq[EPL], mx[EPL];
        load_groups(mean + (long)s * GROUPS, 1, lane, m);
        load_groups(rstd + (long)s * GROUPS, 1, lane, rs);
        load_groups(stat + (long)s * GROUPS * 2, 2, lane, mq);
        load_groups(stat + (long)s * GROUPS * 2 + 1, 2, lane, mx);
        if (r < RW)
            for (long row = a + r; row < b; row += RW * BATCH) {
                R xh[BATCH][EPL], dz[BATCH][EPL];
#pragma unroll
                for (int t = 0; t < BATCH; ++t) {
                    const long n = row + t * RW < b ? row + t * RW : row;
                    slopes(x + n * ld, dy + n * dy_ld, lane, m, rs, wc, bc, xh[t], dz[t]);
                }
#pragma unroll
                for (int t = 0; t < BATCH; ++t) {
                    EACH(i) dz[t][i] = rs[i] * (dz[t][i] * wc[i] - mq[i] - xh[t][i] * mx[i]);
                    if (row + t * RW < b) store_row(dx + (row + t * RW) * dx_ld, lane, dz[t]);
                }
            }
    }
}

// The chunks' sums per channel, added in double: 16 columns of [chunks][2C] to a workgroup, 64 lanes each.
extern "C" __global__ void __launch_bounds__(1024)
cgtp_gnorm_columns(const R *__restrict__ wpart, long chunks, R *__restrict__ gw, R *__restrict__ gb)
{
    __shared__ double lds[1024];
    const int col = blockIdx.x * 16 + threadIdx.x % 16, j = threadIdx.x / 16;
    double sum = 0;
    if (col < 2 * C) {
#pragma unroll 8
        for (long c = j; c < chunks; c += 64) sum += (double)wpart[c * 2 * C + col];
    }
    lds[threadIdx.x] = sum;
    for (int half = 32; half > 0; half /= 2) {
        __syncthreads();
        if (j < half) lds[threadIdx.x] += lds[threadIdx.x + half * 16];
    }
    if (j == 0 && col < 2 * C) {
        if (col < C && gw) gw[col] = (R)lds[threadIdx.x];
        if (col >= C && gb) gb[col - C] = (R)lds[threadIdx.x];
    }
}
)HIP";

}  // namespace cgtp
