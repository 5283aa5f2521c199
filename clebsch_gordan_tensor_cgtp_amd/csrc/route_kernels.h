// HIP source of the routing of rows to experts: scores, choice and weights, and their backward.
// route.cpp puts a configuration's constants and the shared text (row_kernels.h) in front of this text
// and compiles it for gfx950.
//
// Constants of a configuration, beside T, R and ACT:
//   E, K          experts, choices of a row
//   L, EPL        lanes of a row, neighbouring experts of a lane
//   NGRP, GW, LPG groups of experts (1 where every group is taken), experts and lanes of a group
//   TOPG          groups that are taken
//   SIGMOID, RENORM
#pragma once

namespace cgtp {

static const char kRouteKernels[] = R"HIP(
constexpr int RPB = 256 / L;  // rows of a workgroup
#define EACH(i) _Pragma("unroll") for (int i = 0; i < EPL; ++i)

DEV double inf() { return __builtin_huge_val(); }
DEV float lowest(float) { return -__builtin_huge_valf(); }
DEV double lowest(double) { return -__builtin_huge_val(); }

// the value of another lane: inside 16 lanes by DPP (row_kernels.h), across them by the LDS's crossbar
template <int CTRL> DEV int dpp_int(int v) { return __builtin_amdgcn_mov_dpp(v, CTRL, 15, 15, false); }
DEV int from_lane(int v, int lane) { return __builtin_amdgcn_ds_bpermute(lane * 4, v); }
DEV float from_lane(float v, int lane) { return __builtin_bit_cast(float, from_lane(__builtin_bit_cast(int, v), lane)); }
DEV double from_lane(double v, int lane)
{
    const unsigned long long b = __builtin_bit_cast(unsigned long long, v);
    return join64((unsigned)from_lane((int)b, lane), (unsigned)from_lane((int)(b >> 32), lane));
}

// STEP of a butterfly over lanes; each step's partner holds the other half's result
template <int STEP> DEV int other(int v)
{
    if constexpr (STEP == 1) return dpp_int<0xB1>(v);
    if constexpr (STEP == 2) return dpp_int<0x4E>(v);
    if constexpr (STEP == 4) return dpp_int<0x141>(v);
    if constexpr (STEP == 8) return dpp_int<0x140>(v);
    return from_lane(v, (int)(threadIdx.x & 63) ^ STEP);
}
template <int STEP> DEV float other(float v) { return __builtin_bit_cast(float, other<STEP>(__builtin_bit_cast(int, v))); }
template <int STEP> DEV double other(double v)
{
    const unsigned long long b = __builtin_bit_cast(unsigned long long, v);
    return join64((unsigned)other<STEP>((int)b), (unsigned)other<STEP>((int)(b >> 32)));
}

template <int LANES, int STEP = 1, typename V> DEV V lanes_sum(V v)
{
    if constexpr (STEP < LANES) return lanes_sum<LANES, STEP * 2>(v + other<STEP>(v));
    return v;
}
template <int LANES, int STEP = 1, typename V> DEV V lanes_max(V v)
{
    if constexpr (STEP < LANES) {
        const V o = other<STEP>(v);
        return lanes_max<LANES, STEP * 2>(o > v ? o : v);
    }
    return v;
}

// the larger score, of equal ones the lower expert
template <int STEP = 1, typename V> DEV void lanes_best(V &c, int &e)
{
    if constexpr (STEP < L) {
        const V oc = other<STEP>(c);
        const int oe = other<STEP>(e);
        const bool take = oc > c || (oc == c && oe < e);
        c = take ? oc : c;
        e = take ? oe : e;
        lanes_best<STEP * 2>(c, e);
    }
}

// the two largest of a group's lanes
template <int STEP = 1, typename V> DEV void group_best(V &b1, V &b2)
{
    if constexpr (STEP < LPG) {
        const V o1 = other<STEP>(b1), o2 = other<STEP>(b2);
        const V low = o1 > b1 ? b1 : o1, high = o1 > b1 ? o1 : b1, next = o2 > b2 ? o2 : b2;
        b1 = high;
        b2 = low > next ? low : next;
        group_best<STEP * 2>(b1, b2);
    }
}

// a lane's experts: the first, and how many there are
struct Share {
    int first, count;
};
DEV Share share_of(int q)
{
    const int g = q / LPG, at = (q % LPG) * EPL;
    const int count = g < NGRP ? GW - at : 0;
    return {g * GW + at, count < 0 ? 0 : count > EPL ? EPL : count};
}

template <typename S, typename V> DEV void load_share(const S *row, Share sh, V none, V (&x)[EPL])
{
    if (sh.count == EPL) {
        R v[EPL];
        load_run<EPL>(row + sh.first, v);
        EACH(i) x[i] = (V)v[i];
    } else {
        EACH(i) x[i] = i < sh.count ? (V)(R)row[sh.first + i] : none;
    }
}

// Scores, choice and weights of a row by L lanes.  Scores are doubles whatever the logits' type: which of
// two neighbours is chosen does not depend on a rounding of the exponential.  An expert whose logit
// or whose biased score is -inf is masked: it is not chosen, and has no score.
extern "C" __global__ void __launch_bounds__(256)
cgtp_route_fwd(const T *__restrict__ logits, long ld, const R *__restrict__ bias, int *__restrict__ experts,
               R *__restrict__ weights, long N, double scale)
{
    const int q = threadIdx.x % L;
    const long at = (long)blockIdx.x * RPB + threadIdx.x / L, row = at < N ? at : N - 1;
    const Share sh = share_of(q);
    double s[EPL], c[EPL], b[EPL];
    load_share(logits + row * ld, sh, lowest(0.0), s);
    if (bias)
        load_share(bias, sh, 0.0, b);
    else
        EACH(i) b[i] = 0;
    double most = lowest(0.0);
    EACH(i) most = s[i] > most ? s[i] : most;
    if (!SIGMOID) most = lanes_max<L>(most);
    double total = 0;
    EACH(i)
    {
        const bool masked = s[i] == lowest(0.0);
        if (SIGMOID)
            s[i] = masked ? 0.0 : 1.0 / (1.0 + exp(-s[i]));
        else
            s[i] = masked ? 0.0 : exp(s[i] - most);
        total += s[i];
        c[i] = masked ? lowest(0.0) : 0.0;
    }
    if (!SIGMOID) {
        total = lanes_sum<L>(total);
        EACH(i) s[i] = c[i] == 0.0 ? s[i] / total : 0.0;
    }
    EACH(i)
    {
        if (c[i] == 0.0) {
            c[i] = s[i] + b[i];
            if (c[i] != c[i]) c[i] = -1.7976931348623157e308;  // not a number: after every other one
        }
    }
    if (TOPG < NGRP) {
        double b1 = lowest(0.0), b2 = lowest(0.0);
        EACH(i)
        {
            const double low = c[i] > b1 ? b1 : c[i];
            b1 = c[i] > b1 ? c[i] : b1;
            b2 = low > b2 ? low : b2;
        }
        group_best(b1, b2);
        const double mine = b2 > lowest(0.0) ? b1 + b2 : b1;
        const int g = q / LPG, base = (threadIdx.x & 63) - q;
        int rank = 0;
        for (int o = 0; o < NGRP; ++o) {
            const double theirs = from_lane(mine, base + o * LPG);
            rank += theirs > mine || (theirs == mine && o < g);
        }
        EACH(i) c[i] = rank < TOPG ? c[i] : lowest(0.0);
    }
    int chosen[K];
    double score[K], sum = 0;
#pragma unroll
    for (int j = 0; j < K; ++j) {
        double best = lowest(0.0);
        int e = E;
        EACH(i)
        {
            const bool take = c[i] > best;
            best = take ? c[i] : best;
            e = take ? sh.first + i : e;
        }
        lanes_best(best, e);
        const bool some = best > lowest(0.0);
        double v = 0;
        EACH(i)
        {
            const bool it = sh.first + i == e;
            v = it ? s[i] : v;
            c[i] = it ? lowest(0.0) : c[i];
        }
        const int owner = (threadIdx.x & 63) - q + (e / GW) * LPG + (e % GW) / EPL;
        v = from_lane(v, some ? owner : (int)(threadIdx.x & 63));
        chosen[j] = some ? e : -1;
        score[j] = some ? v : 0.0;
        sum += score[j];
    }
    if (at >= N) return;
    if (RENORM && sum < 1e-290) {
        // scores near or below a double's range (far under an unchosen logit, or sigmoids of under -660): their shares
        // with the largest exponential taken out, as in the backward
        double x[K], top = lowest(0.0);
#pragma unroll
        for (int j = 0; j < K; ++j) {
            x[j] = chosen[j] < 0 ? lowest(0.0) : (double)(R)logits[row * ld + chosen[j]];
            top = x[j] > top ? x[j] : top;
        }
        if (SIGMOID && top > 0.0) top = 0.0;
        sum = 0;
#pragma unroll
        for (int j = 0; j < K; ++j) {
            score[j] = chosen[j] < 0 ? 0.0 : SIGMOID ? 1.0 / (exp(top) + exp(top - x[j])) : exp(x[j] - top);
            sum += score[j];
        }
    }
    const double f = RENORM ? (sum == 0.0 ? 0.0 : scale / sum) : scale;
#pragma unroll
    for (int j = 0; j < K; ++j)
        if (q == j % L) {
            experts[row * K + j] = chosen[j];
            weights[row * K + j] = (R)(score[j] * f);
        }
}

// d/dlogits of <grad_weights, weights>, the choice held fixed.  L lanes share a row and each takes its
// chosen logits itself.  Shares of the chosen sum are formed with their largest exponential
// taken out, so they hold where every score of a row is below the type's range.
extern "C" __global__ void __launch_bounds__(256)
cgtp_route_bwd(const T *__restrict__ logits, long ld, const int *__restrict__ experts, const R *__restrict__ grad,
               T *__restrict__ out, long N, R scale)
{
    const int q = threadIdx.x % L;
    const long at = (long)blockIdx.x * RPB + threadIdx.x / L, row = at < N ? at : N - 1;
    const Share sh = share_of(q);
    const T *l = logits + row * ld;
    int e[K];
    R d[K], x[K], most = lowest((R)0);
#pragma unroll
    for (int j = 0; j < K; ++j) {
        e[j] = experts[row * K + j];
        const bool in = e[j] >= 0 && e[j] < E;
        e[j] = in ? e[j] : -1;
        d[j] = in ? grad[row * K + j] * scale : (R)0;
        x[j] = in ? (R)l[e[j]] : lowest((R)0);
        most = x[j] > most ? x[j] : most;
    }
    R v[EPL];
    EACH(i) v[i] = (R)0;
    if (SIGMOID || RENORM) {
        if (RENORM) {
            R total = 0, dot = 0, r[K];
            const R top = SIGMOID && most > (R)0 ? (R)0 : most;
#pragma unroll
            for (int j = 0; j < K; ++j) {
                // softmax: exp(x - top); sigmoid: exp(-top) / (1 + exp(-x))
                r[j] = e[j] < 0 ? (R)0 : SIGMOID ? (R)1 / (exp(top) + exp(top - x[j])) : exp(x[j] - top);
                total += r[j];
                dot += r[j] * d[j];
            }
            const R inv = total > (R)0 || total != total ? (R)1 / total : (R)0;
            dot *= inv;
#pragma unroll
            for (int j = 0; j < K; ++j) d[j] = r[j] * inv * (d[j] - dot);
        }
        if (SIGMOID) {
#pragma unroll
            for (int j = 0; j < K; ++j) {
                const R u = exp(x[j] < (R)0 ? x[j] : -x[j]), inv = (R)1 / ((R)1 + u);
                const R rest = x[j] < (R)0 ? inv : u * inv;  // 1 - s
                d[j] = e[j] < 0 ? (R)0 : RENORM ? d[j] * rest : d[j] * (u * inv * inv);
            }
        }
#pragma unroll
        for (int j = 0; j < K; ++j) EACH(i) v[i] += sh.first + i == e[j] ? d[j] : (R)0;
    } else {
        R s[EPL], total = 0, dot = 0;
        load_share(l, sh, lowest((R)0), s);
        most = lowest((R)0);
        EACH(i) most = s[i] > most ? s[i] : most;
        most = lanes_max<L>(most);
        EACH(i)
        {
            s[i] = s[i] == lowest((R)0) ? (R)0 : exp(s[i] - most);
            total += s[i];
        }
        total = lanes_sum<L>(total);
        const R inv = total == (R)0 ? (R)0 : (R)1 / total;
#pragma unroll
        for (int j = 0; j < K; ++j) {
            if (e[j] >= 0) dot += exp(x[j] - most) * inv * d[j];
            EACH(i) v[i] += sh.first + i == e[j] ? d[j] : (R)0;
        }
        EACH(i) v[i] = s[i] * inv * (v[i] - dot);
    }
    if (at >= N) return;
    T *o = out + row * E + sh.first;
    if (sh.count == EPL) {
        store_run<EPL>(o, v);
    } else {
        EACH(i)
            if (i < sh.count) o[i] = (T)v[i];
    }
}
)HIP";

}  // namespace cgtp
