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

template <int LANES, int STEP = 1> DEV int lanes_min(int v)
{
    if constexpr (STEP < LANES) {
        const int o = other<STEP>(v);
        return lanes_min<LANES, STEP * 2>(o < v ? o : v);
    }
    return v;
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

// ---------------------------------------------------------------- choice
// A row is L lanes'.  Which of two neighbouring experts is chosen is a matter of their scores in double, whatever the
// logits' type.  An expert whose logit or whose biased score is -inf is masked: it is not chosen, and has no score.
struct Row {
    Share sh;
    int q, base;  // the lane's number in the row, the wave's lane of the row's first
    const T *logits;
    const R *bias;
};

// the row's groups that are taken: c of the others masked.  Returns whether a group's sum lies so close to another's
// (`close` times their size) that the order of the two is not sure.
template <typename V> DEV bool take_groups(const Row &row, V (&c)[EPL], const V (&score)[EPL], V close)
{
    V b1 = lowest((V)0), b2 = lowest((V)0);
    EACH(i)
    {
        const V v = c[i] > lowest((V)0) ? score[i] : lowest((V)0), low = v > b1 ? b1 : v;
        b1 = v > b1 ? v : b1;
        b2 = low > b2 ? low : b2;
    }
    group_best(b1, b2);
    const V mine = b2 > lowest((V)0) ? b1 + b2 : b1, near = close * ((V)1 + (mine < (V)0 ? -mine : mine));
    const int g = row.q / LPG;
    int rank = 0;
    bool unsure = false;
#pragma unroll
    for (int o = 0; o < NGRP; ++o) {
        const V theirs = from_lane(mine, row.base + o * LPG), gap = theirs - mine;
        rank += theirs > mine || (theirs == mine && o < g);
        unsure = unsure || (o != g && gap >= -near && gap <= near);
    }
    EACH(i) c[i] = rank < TOPG ? c[i] : lowest((V)0);
    return close > (V)0 && unsure;
}

// The K largest c in falling order, of equal ones the lowest expert first: -1 where none is left.  They are masked in c.
template <typename V> DEV void pick(const Row &row, V (&c)[EPL], int (&chosen)[K], V (&best)[K])
{
#pragma unroll
    for (int j = 0; j < K; ++j) {
        V most = c[0];
#pragma unroll
        for (int i = 1; i < EPL; ++i) most = c[i] > most ? c[i] : most;
        most = lanes_max<L>(most);
        int e = E;
#pragma unroll
        for (int i = EPL - 1; i >= 0; --i) e = c[i] == most ? row.sh.first + i : e;
        e = lanes_min<L>(e);
        EACH(i) c[i] = row.sh.first + i == e ? lowest((V)0) : c[i];
        chosen[j] = most > lowest((V)0) ? e : -1;
        best[j] = most;
    }
}

// The choice in double.
DEV void choose(const Row &row, int (&chosen)[K])
{
    double s[EPL], c[EPL], b[EPL], most = lowest(0.0), total = 0;
    load_share(row.logits, row.sh, lowest(0.0), s);
    if (row.bias)
        load_share(row.bias, row.sh, 0.0, b);
    else
        EACH(i) b[i] = 0;
    EACH(i)
    {
        most = s[i] > most ? s[i] : most;
        c[i] = s[i] == lowest(0.0) ? lowest(0.0) : 0.0;
    }
    if (!SIGMOID) most = lanes_max<L>(most);
    EACH(i)
    {
        s[i] = c[i] < 0.0 ? 0.0 : SIGMOID ? 1.0 / (1.0 + exp(-s[i])) : exp(s[i] - most);
        total += s[i];
    }
    if (!SIGMOID) {
        total = lanes_sum<L>(total);
        EACH(i) s[i] = c[i] < 0.0 ? 0.0 : s[i] / total;
    }
    EACH(i)
    {
        if (c[i] == 0.0) {
            c[i] = s[i] + b[i];
            if (c[i] != c[i]) c[i] = -1.7976931348623157e308;  // not a number: after every other one
        }
    }
    if (TOPG < NGRP) {
        EACH(i) b[i] = c[i];
        take_groups(row, c, b, 0.0);
    }
    double best[K];
    pick(row, c, chosen, best);
}

// The choice in float, and whether it is surely the one in double.  Without a bias experts go by their logits, whose
// order is the scores' but where these are equal as doubles: logits that differ by next to nothing, or scores near 1
// or 0.  With one, a score is off by less than 2^-20 of 1 (a rounding of the exponent's argument, |x| exp(-|x|) of it, the
// exponential, a sum of up to 512 and a quotient), so c in neighbouring places have to be further apart than twice
// that, or of equal logits and biases.
DEV bool choose_fast(const Row &row, int (&chosen)[K])
{
    constexpr float CLOSE = 4e-6f;
    float x[EPL], c[EPL], s[EPL], most = lowest(0.0f);
    load_share(row.logits, row.sh, lowest(0.0f), x);
    EACH(i) most = x[i] > most ? x[i] : most;
    most = lanes_max<L>(most);
    bool sure = most < (SIGMOID ? 18.0f : 1e4f);
    EACH(i) c[i] = x[i];
    if (row.bias || TOPG < NGRP) {
        float total = 0, b[EPL];
        if (row.bias)
            load_share(row.bias, row.sh, 0.0f, b);
        else
            EACH(i) b[i] = 0;
        EACH(i)
        {
            const float e = __builtin_amdgcn_exp2f((SIGMOID ? -x[i] : x[i] - most) * 1.44269504f);
            s[i] = SIGMOID ? __builtin_amdgcn_rcpf(1.0f + e) : e;
            total += x[i] > lowest(0.0f) ? s[i] : 0.0f;
        }
        if (!SIGMOID) {
            const float inv = __builtin_amdgcn_rcpf(lanes_sum<L>(total));
            EACH(i) s[i] *= inv;
        }
        EACH(i)
        {
            s[i] += b[i];
            if (row.bias) c[i] = x[i] > lowest(0.0f) ? s[i] : lowest(0.0f);
            sure = sure && (x[i] == lowest(0.0f) || s[i] - s[i] == 0.0f);  // finite
        }
        if (TOPG < NGRP) sure = !take_groups(row, c, s, 2 * CLOSE) && sure;
    } else {
        EACH(i) sure = sure && (x[i] == lowest(0.0f) || x[i] - x[i] == 0.0f);
    }
    float best[K], rest = lowest(0.0f);
    pick(row, c, chosen, best);
    EACH(i) rest = c[i] > rest ? c[i] : rest;
    rest = lanes_max<L>(rest);  // the best that is left shows whether the last one is sure
#pragma unroll
    for (int j = 0; j < K; ++j) {
        if (j % L != row.q) continue;  // a lane looks at some places and the next ones
        if (chosen[j] < 0) continue;
        const float next = j + 1 < K ? best[j + 1] : rest, gap = best[j] - next;
        if (!row.bias) {
            // far below 1 (a sigmoid) or the largest (a softmax) scores may be too small for a double
            sure = sure && (gap == 0.0f || gap > 1e-10f * (1.0f + fabsf(best[j]) + fabsf(most))) &&
                   (SIGMOID ? best[j] : best[j] - most) > -600.0f;
        } else if (gap <= CLOSE * (1.0f + fabsf(best[j]))) {
            const int e0 = chosen[j], e1 = j + 1 < K ? chosen[j + 1] : -1;
            sure = sure && e1 >= 0 && row.logits[e0] == row.logits[e1] && row.bias[e0] == row.bias[e1];
        }
    }
    return lanes_min<L>(sure ? 1 : 0) != 0;
}

// Choice and weights of a row by L lanes.  A weight is formed in double from the chosen logits, each by one lane.
extern "C" __global__ void __launch_bounds__(256)
cgtp_route_fwd(const T *__restrict__ logits, long ld, const R *__restrict__ bias, int *__restrict__ experts,
               R *__restrict__ weights, long N, double scale)
{
    const long at = (long)blockIdx.x * RPB + threadIdx.x / L, n = at < N ? at : N - 1;
    Row row;
    row.q = threadIdx.x % L;
    row.base = (threadIdx.x & 63) - row.q;
    row.sh = share_of(row.q);
    row.logits = logits + n * ld;
    row.bias = bias;
    int chosen[K];
    bool sure = false;
    if constexpr (sizeof(R) == 4) sure = choose_fast(row, chosen);
    if (!sure) choose(row, chosen);
    double total = 1, most = 0;
    if (!SIGMOID && !RENORM) {
        double x[EPL];
        load_share(row.logits, row.sh, lowest(0.0), x);
        most = lowest(0.0);
        EACH(i) most = x[i] > most ? x[i] : most;
        most = lanes_max<L>(most);
        total = 0;
        EACH(i) total += x[i] == lowest(0.0) ? 0.0 : exp(x[i] - most);
        total = lanes_sum<L>(total);
    }
    // the lane's places, K / L of them
    constexpr int PLACES = (K + L - 1) / L;
    int e[PLACES];
    double x[PLACES], top = lowest(0.0), sum = 0;
#pragma unroll
    for (int p = 0; p < PLACES; ++p) {
        e[p] = -1;
#pragma unroll
        for (int j = p * L; j < K && j < (p + 1) * L; ++j) e[p] = j % L == row.q ? chosen[j] : e[p];
        x[p] = e[p] < 0 ? lowest(0.0) : (double)(R)row.logits[e[p]];
        top = x[p] > top ? x[p] : top;
    }
    if (RENORM) {
        // with the largest exponential taken out: scores too small for a double have shares
        top = lanes_max<L>(top);
        if (SIGMOID && top > 0.0) top = 0.0;
    }
#pragma unroll
    for (int p = 0; p < PLACES; ++p) {
        if (RENORM)
            x[p] = e[p] < 0 ? 0.0 : SIGMOID ? 1.0 / (exp(top) + exp(top - x[p])) : exp(x[p] - top);
        else
            x[p] = e[p] < 0 ? 0.0 : SIGMOID ? 1.0 / (1.0 + exp(-x[p])) : exp(x[p] - most) / total;
        sum += x[p];
    }
    if (RENORM) {
        sum = lanes_sum<L>(sum);
        scale = sum == 0.0 ? 0.0 : scale / sum;
    }
    if (at >= N) return;
#pragma unroll
    for (int p = 0; p < PLACES; ++p)
        if (p * L + row.q < K) {
            experts[n * K + p * L + row.q] = e[p];
            weights[n * K + p * L + row.q] = (R)(x[p] * scale);
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
