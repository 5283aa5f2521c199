// Group norm plans: row layout, the generated source's constants, and the entry points
// cgtp_group_norm_* (documented in include/cgtp.h).
#include <algorithm>
#include <cmath>
#include <memory>

#include "config_module.h"
#include "gnorm_kernels.h"
#include "row_kernels.h"
#include "rows.h"

struct cgtp_group_norm {
    cgtp_group_norm_config cfg{};
    int elem = 4, real = 4;              // bytes of an element; of a statistic or weight
    int cv = 1, p = 1, rw = 1, ns = 1;   // channels a lane takes together, lanes of a row, rows at once, slots
    cgtp::ConfigModule mod;
    int held_fwd = 1, held_bwd = 1, waves = 1;  // rows that a lane holds; most waves of a workgroup
    enum { fwd, fwd_large, bwd, bwd_large };
    int groups_pow2 = 1;
};

namespace cgtp {

namespace {

int pow2_at_least(int n)
{
    int p = 1;
    while (p < n) p *= 2;
    return p;
}

// A lane takes up to 16 bytes of a row at a time; short rows lie side by side in a wave.  In the forward it holds 128
// bytes of its graph's rows as they are in memory; in the backward rows of x and dy in the statistics' type, in what
// registers the waves of a workgroup leave beside seven values per channel.  Wide rows, of which a lane holds more
// channels, get fewer waves.
void lay_out(cgtp_group_norm &g)
{
    const int c = g.cfg.channels;
    g.elem = elem_bytes(g.cfg.dtype);
    g.real = real_bytes(g.cfg.dtype);
    g.cv = 16 / g.elem;
    while (g.cv > c) g.cv /= 2;
    const int units = (c + g.cv - 1) / g.cv;
    g.p = std::min(units, 64);
    g.ns = (units + 63) / 64;
    g.rw = 64 / g.p;
    g.groups_pow2 = pow2_at_least(g.cfg.groups);
    const int channels = g.ns * g.cv, regs = channels * g.real / 4;
    g.held_fwd = std::max(1, 128 / (channels * g.elem));
    g.waves = regs <= 8 ? 16 : regs <= 16 ? 8 : 4;
    g.held_bwd = regs <= 4 ? 8 : 2;
}

std::string constants(const cgtp_group_norm &g)
{
    std::string s = "// group norm of " + std::to_string(g.cfg.channels) + " channels\n";
    auto num = [&](const char *n, long v) { s += std::string("constexpr int ") + n + " = " + std::to_string(v) + ";\n"; };
    s += "#define FAST_EXP (sizeof(T) <= 4)\n";
    s += std::string("typedef ") + type_name(g.cfg.dtype) + " T;\n";
    s += std::string("typedef ") + (g.cfg.dtype == CGTP_F64 ? "double" : "float") + " R;\n";
    num("ACT", g.cfg.act);
    num("C", g.cfg.channels);
    num("GROUPS", g.cfg.groups);
    num("W", g.cfg.channels / g.cfg.groups);
    num("CV", g.cv);
    num("P", g.p);
    num("RW", g.rw);
    num("NS", g.ns);
    num("GP", g.groups_pow2);
    num("BF", g.held_fwd);
    num("BB", g.held_bwd);
    num("NWMAX", g.waves);
    return s;
}

// How a pass over N rows in S graphs is launched (gnorm_kernels.h has the two ways over the rows).
struct Split {
    int waves;       // of a workgroup
    int64_t cap;     // rows of a graph that one workgroup takes
    int64_t rows;    // of a chunk
    int64_t chunks, graphs;  // workgroups of the first launch
    bool large;      // whether a graph can have more than cap rows
};

// Where a workgroup of the most waves holds all N rows, as few waves as do: no graph is large, and the second
// launch is left out.  Else 2.5 mean graphs: of graphs of uneven sizes most are one workgroup's then, and
// waves that a smaller one leaves idle are few; where that is far more than a workgroup's, nearly all are large, and four
// waves share them out more evenly.  (4,000 graphs of 50 rows on average, 64 channels in bf16.)
// Chunks: at most 1,024, whose pieces each workgroup of the second launch joins for itself; a backward's
// workgroups take graphs in turn, since each leaves its partial sums of the weights' gradients: 1,024 of them, or 8,192 where
// each would have more than 16.
Split split(const cgtp_group_norm &g, int64_t N, int64_t S, bool backward)
{
    Split p{};
    const int64_t held = (int64_t)g.rw * (backward ? g.held_bwd : g.held_fwd);
    const int64_t want = N <= held * g.waves ? N : (int64_t)(2.5 * (double)N / (double)std::max<int64_t>(1, S));
    p.waves = want > 4 * held * g.waves ? std::min(4, g.waves) : 1;
    if (want <= 4 * held * g.waves)
        while (p.waves < g.waves && held * p.waves < want) p.waves *= 2;
    p.cap = held * p.waves;
    p.large = N > p.cap;
    const int64_t step = (int64_t)g.rw * p.waves * (g.ns * g.cv <= 4 ? 4 : 2);
    p.rows = std::max<int64_t>(1, (N + 1024 * step - 1) / (1024 * step)) * step;
    p.chunks = (N + p.rows - 1) / p.rows;
    p.graphs = backward ? std::min<int64_t>(S, S <= 16384 ? 1024 : 8192) : S;
    return p;
}

// bytes of LDS: a lane's sums of `quantities`, the groups' and their parts (or a column per channel)
int lds_bytes(const cgtp_group_norm &g, int waves, int quantities, bool columns)
{
    const int w = g.cfg.channels / g.cfg.groups, es = w % g.cv == 0 ? g.cv : 1, ce = (g.cfg.channels + es - 1) / es;
    const int per_group = std::max(1, 64 * waves / g.groups_pow2 / 64);
    const int sums = quantities * (waves * g.rw * ce + g.cfg.groups * (1 + per_group));
    return std::max(sums, columns ? waves * g.rw * g.cfg.channels : 0) * g.real;
}

int lds_bytes_large(const cgtp_group_norm &g, int threads)
{
    return std::max((3 * threads + 2 * g.cfg.groups) * g.real, threads * 8);
}

size_t aligned(size_t n) { return (n + 255) / 256 * 256; }

struct Workspace {
    size_t part, stat, wpart;  // bytes
    size_t bytes() const { return aligned(part) + aligned(stat) + aligned(wpart); }
};

Workspace workspace_of(const cgtp_group_norm &g, int64_t N, int64_t S, bool backward)
{
    const Split sp = split(g, N, S, backward);
    Workspace w{};
    if (S == 0) return w;
    if (sp.large) w.part = (size_t)(sp.chunks + S) * g.cfg.groups * 2 * g.real;
    if (!backward) w.stat = (size_t)S * g.cfg.groups * 2 * g.real;  // where the caller wants no statistics
    if (backward) w.wpart = (size_t)(sp.chunks + sp.graphs) * 2 * g.cfg.channels * g.real;
    return w;
}

void run_lds(hipFunction_t f, int64_t groups, int threads, int lds, void **args, void *stream)
{
    check_hip(hipModuleLaunchKernel(f, (unsigned)groups, 1, 1, (unsigned)threads, 1, 1, (unsigned)lds,
                                    static_cast<hipStream_t>(stream), args, nullptr),
              "hipModuleLaunchKernel");
}

void check_graphs(int64_t S, const int32_t *ptr)
{
    require(S >= 0 && S < INT_MAX, "S must be in [0, 2^31-1)");
    require_ptr(ptr, "ptr", 4);
}

}  // namespace

}  // namespace cgtp

using namespace cgtp;

extern "C" {

cgtp_status cgtp_group_norm_create(const cgtp_group_norm_config *config, cgtp_group_norm **norm_out)
{
    return guarded([&] {
        require(config && norm_out, "NULL argument to cgtp_group_norm_create");
        *norm_out = nullptr;
        const cgtp_group_norm_config &c = *config;
        require(c.dtype == CGTP_F32 || c.dtype == CGTP_F64 || c.dtype == CGTP_BF16 || c.dtype == CGTP_F16,
                "dtype must be CGTP_F32, CGTP_F64, CGTP_BF16 or CGTP_F16");
        require(c.channels >= 1 && c.groups >= 1 && c.channels % c.groups == 0,
                "channels must be a positive multiple of groups");
        require(c.act >= CGTP_ACT_IDENTITY && c.act <= CGTP_ACT_TANH, "act must be a cgtp_act");
        require(std::isfinite(c.eps) && c.eps > 0 && (c.dtype == CGTP_F64 || (float)c.eps >= 1e-30f),
                "eps must be finite and positive (at least 1e-30 where statistics are float)");
        if (c.channels > 2048) throw Error(CGTP_ERR_UNSUPPORTED, "group norm: more than 2048 channels");
        auto h = std::make_unique<cgtp_group_norm>();
        h->cfg = c;
        lay_out(*h);
        h->mod.build(constants(*h) + kRowKernels + kGroupNormKernels,
                     {"cgtp_gnorm_fwd", "cgtp_gnorm_fwd_large", "cgtp_gnorm_bwd", "cgtp_gnorm_bwd_large"});
        *norm_out = h.release();
    });
}

cgtp_status cgtp_group_norm_destroy(cgtp_group_norm *norm)
{
    return guarded([&] {
        if (!norm) return;
        norm->mod.unload();
        delete norm;
    });
}

const char *cgtp_group_norm_source(const cgtp_group_norm *norm) { return norm ? norm->mod.source.c_str() : nullptr; }

cgtp_status cgtp_group_norm_workspace_size(const cgtp_group_norm *norm, int64_t N, int64_t S, int32_t backward,
                                           size_t *bytes)
{
    return guarded([&] {
        require(norm && bytes, "NULL argument to cgtp_group_norm_workspace_size");
        check_count(N);
        require(S >= 0 && S < INT_MAX, "S must be in [0, 2^31-1)");
        *bytes = workspace_of(*norm, N, S, backward != 0).bytes();
    });
}

cgtp_status cgtp_group_norm_forward(const cgtp_group_norm *norm, int64_t N, int64_t S, const int32_t *ptr, const void *x,
                                    int64_t x_ld, const void *w, const void *bias, void *y, int64_t y_ld, int32_t fill,
                                    void *mean, void *rstd, void *workspace, size_t workspace_bytes, void *stream)
{
    return guarded([&] {
        require(norm != nullptr, "norm is NULL");
        auto &g = *const_cast<cgtp_group_norm *>(norm);
        check_count(N);
        check_graphs(S, ptr);
        if (S == 0) return;
        require(!mean == !rstd, "mean and rstd are given together");
        const int c = g.cfg.channels;
        const Rows X{x, c, x_ld, "x"}, Y{y, c, y_ld, "y"};
        if (N > 0) {
            check_rows(g.elem, N, X);
            check_rows(g.elem, N, Y);
        }
        const size_t nw = (size_t)c * g.real, ns = (size_t)S * g.cfg.groups * g.real;
        for (const auto &a : {std::make_pair((const void *)w, "w"), {bias, "bias"}, {mean, "mean"}, {rstd, "rstd"}})
            if (a.first) require_ptr(a.first, a.second, g.real);
        const Workspace ws = workspace_of(g, N, S, false);
        require_ptr(workspace, "workspace", 256);
        require(workspace_bytes >= ws.bytes(), "workspace too small (see cgtp_group_norm_workspace_size)");
        Arguments all(g.elem, N);
        all.rows(X, false);
        all.rows(Y, true);
        all.flat(ptr, (size_t)(S + 1) * 4, "ptr", false);
        all.flat(w, nw, "w", false);
        all.flat(bias, nw, "bias", false);
        all.flat(mean, ns, "mean", true);
        all.flat(rstd, ns, "rstd", true);
        all.flat(workspace, ws.bytes(), "workspace", true);
        all.check();
        const auto &F = g.mod.here();
        const Split sp = split(g, N, S, false);
        require(S + sp.chunks < INT_MAX, "too many graphs");
        void *piece = workspace;
        if (!mean) {
            mean = static_cast<char *>(workspace) + aligned(ws.part);
            rstd = static_cast<char *>(mean) + ns;
        }
        long xl = (long)x_ld, yl = (long)y_ld, n = (long)N, rows = (long)sp.rows, cap = (long)sp.cap;
        int s = (int)S;
        float ef = (float)g.cfg.eps;
        double ed = g.cfg.eps;
        void *eps = g.real == 8 ? (void *)&ed : (void *)&ef;
        void *args[] = {&x, &xl, &ptr, &s, &n, &rows, &cap, &w, &bias, &y, &yl, &fill, &mean, &rstd, &piece, eps};
        run_lds(F[cgtp_group_norm::fwd], sp.chunks + sp.graphs, 64 * sp.waves, lds_bytes(g, sp.waves, 1, false), args, stream);
        if (sp.large) {
            const int threads = 64 * std::min(std::max(sp.waves, 4), g.waves);
            void *largs[] = {&x, &xl, &ptr, &s, &n, &rows, &cap, &w, &bias, &piece, &y, &yl, &mean, &rstd, eps};
            run_lds(F[cgtp_group_norm::fwd_large], sp.chunks, threads, lds_bytes_large(g, threads), largs, stream);
        }
    });
}

cgtp_status cgtp_group_norm_backward(const cgtp_group_norm *norm, int64_t N, int64_t S, const int32_t *ptr,
                                     const void *x, int64_t x_ld, const void *w, const void *bias, const void *mean,
                                     const void *rstd, const void *grad_y, int64_t grad_y_ld, void *grad_x,
                                     int64_t grad_x_ld, int32_t fill, void *grad_w, void *grad_bias,
                                     void *workspace, size_t workspace_bytes, void *stream)
{
    return guarded([&] {
        require(norm != nullptr, "norm is NULL");
        auto &g = *const_cast<cgtp_group_norm *>(norm);
        check_count(N);
        check_graphs(S, ptr);
        if (!grad_x && !grad_w && !grad_bias) return;
        const int c = g.cfg.channels;
        const size_t nw = (size_t)c * g.real, ns = (size_t)S * g.cfg.groups * g.real;
        for (const auto &a : {std::make_pair((const void *)w, "w"), {bias, "bias"}, {grad_w, "grad_w"},
                              {grad_bias, "grad_bias"}})
            if (a.first) require_ptr(a.first, a.second, g.real);
        const bool weights = grad_w || grad_bias, work = N > 0 && S > 0;
        const Rows X{x, c, x_ld, "x"}, DY{grad_y, c, grad_y_ld, "grad_y"}, DX{grad_x, c, grad_x_ld, "grad_x"};
        const Workspace ws = workspace_of(g, N, S, true);
        Arguments all(g.elem, N);
        if (work) {
            check_rows(g.elem, N, X);
            check_rows(g.elem, N, DY);
            if (grad_x) check_rows(g.elem, N, DX);
            require_ptr(mean, "mean", g.real);
            require_ptr(rstd, "rstd", g.real);
            require_ptr(workspace, "workspace", 256);
            require(workspace_bytes >= ws.bytes(), "workspace too small (see cgtp_group_norm_workspace_size)");
            all.rows(X, false);
            all.rows(DY, false);
            all.rows(DX, true);
            all.flat(ptr, (size_t)(S + 1) * 4, "ptr", false);
            all.flat(mean, ns, "mean", false);
            all.flat(rstd, ns, "rstd", false);
            all.flat(workspace, ws.bytes(), "workspace", true);
        }
        all.flat(w, nw, "w", false);
        all.flat(bias, nw, "bias", false);
        all.flat(grad_w, nw, "grad_w", true);
        all.flat(grad_bias, nw, "grad_bias", true);
        all.check();
        const auto &F = g.mod.here();
        const Split sp = split(g, N, S, true);
        char *at = static_cast<char *>(workspace);
        void *piece = at, *wpart = weights ? at + aligned(ws.part) + aligned(ws.stat) : nullptr;
        long xl = (long)x_ld, dyl = (long)grad_y_ld, dxl = (long)grad_x_ld, n = (long)N, rows = (long)sp.rows, cap = (long)sp.cap;
        long count = work ? (long)(sp.chunks + sp.graphs) : 0;
        int s = (int)S, graphs = (int)sp.graphs, columns = weights ? (2 * c + 15) / 16 : 0;
        if (work) {
            void *args[] = {&x, &xl, &grad_y, &dyl, &ptr, &s, &n, &rows, &graphs, &cap, &w, &bias, &mean, &rstd, &grad_x, &dxl,
                            &fill, &piece, &wpart};
            run_lds(F[cgtp_group_norm::bwd], sp.chunks + sp.graphs, 64 * sp.waves, lds_bytes(g, sp.waves, 2, true), args, stream);
        }
        const int64_t finish = work && grad_x && sp.large ? sp.chunks : 0;
        if (columns + finish > 0) {
            const int threads = 64 * std::min(std::max(sp.waves, 8), g.waves);
            void *args[] = {&x, &xl, &grad_y, &dyl, &ptr, &s, &n, &rows, &cap, &w, &bias, &mean, &rstd, &piece, &grad_x, &dxl,
                            &columns, &wpart, &count, &grad_w, &grad_bias};
            run_lds(F[cgtp_group_norm::bwd_large], columns + finish, threads, lds_bytes_large(g, threads), args, stream);
        }
    });
}

}  // extern "C"
