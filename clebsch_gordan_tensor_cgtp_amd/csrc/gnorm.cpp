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
    enum { stats, join, apply, bwd_sums, bwd_join, bwd_apply, columns };
    int width() const { return cfg.channels / cfg.groups; }
    int batch() const { return ns * cv <= 8 ? 4 : 2; }
};

namespace cgtp {

namespace {

int pow2_at_least(int n)
{
    int p = 1;
    while (p < n) p *= 2;
    return p;
}

// A lane takes up to 16 bytes of a row at a time; short rows lie side by side in a wave.
void lay_out(cgtp_group_norm &g)
{
    const int c = g.cfg.channels;
    g.elem = elem_bytes(g.cfg.dtype);
    g.real = real_bytes(g.cfg.dtype);
    g.cv = std::min(16 / g.elem, pow2_at_least(c));
    const int units = (c + g.cv - 1) / g.cv;
    g.p = std::min(units, 64);
    g.ns = (units + 63) / 64;
    g.rw = 64 / g.p;
}

std::string constants(const cgtp_group_norm &g)
{
    std::string s = "// group norm of " + std::to_string(g.cfg.channels) + " channels\n";
    auto num = [&](const char *n, long v) { s += std::string("constexpr int ") + n + " = " + std::to_string(v) + ";\n"; };
    s += std::string("typedef ") + type_name(g.cfg.dtype) + " T;\n";
    s += std::string("typedef ") + (g.cfg.dtype == CGTP_F64 ? "double" : "float") + " R;\n";
    num("ACT", g.cfg.act);
    num("C", g.cfg.channels);
    num("GROUPS", g.cfg.groups);
    num("W", g.width());
    num("CV", g.cv);
    num("P", g.p);
    num("RW", g.rw);
    num("NS", g.ns);
    num("GL", std::min(64, pow2_at_least(g.cfg.groups)));
    num("CHUNK_LDS", (long)g.rw * g.cfg.channels);
    return s;
}

// Rows of a wave: whole batches, and no more waves than `most`.
int64_t chunk_rows(const cgtp_group_norm &g, int64_t N, int64_t most)
{
    const int64_t step = (int64_t)g.rw * g.batch();
    return std::max<int64_t>(1, (N + most * step - 1) / (most * step)) * step;
}

constexpr int64_t kForwardWaves = 4096, kBackwardWaves = 2048;

struct Split {
    int64_t rows, chunks;
};

Split split(const cgtp_group_norm &g, int64_t N, bool backward)
{
    const int64_t rows = chunk_rows(g, N, backward ? kBackwardWaves : kForwardWaves);
    return {rows, (N + rows - 1) / rows};
}

size_t aligned(size_t n) { return (n + 255) / 256 * 256; }

struct Workspace {
    size_t part, stat, wpart;  // bytes
    size_t bytes() const { return aligned(part) + aligned(stat) + aligned(wpart); }
};

Workspace workspace_of(const cgtp_group_norm &g, int64_t N, int64_t S, bool backward)
{
    const Split sp = split(g, N, backward);
    Workspace w{};
    if (S == 0) return w;
    w.part = (size_t)(sp.chunks + S) * g.cfg.groups * 2 * g.real;
    // the forward's statistics, where the caller wants none; the backward's means
    w.stat = (size_t)S * g.cfg.groups * 2 * g.real;
    if (backward) w.wpart = (size_t)sp.chunks * 2 * g.cfg.channels * g.real;
    return w;
}

int join_threads(int64_t S) { return S > 8192 ? 64 : 256; }

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
                     {"cgtp_gnorm_stats", "cgtp_gnorm_join", "cgtp_gnorm_apply", "cgtp_gnorm_bwd_sums",
                      "cgtp_gnorm_bwd_join", "cgtp_gnorm_bwd_apply", "cgtp_gnorm_columns"});
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
        const Split sp = split(g, N, false);
        void *part = workspace;
        if (!mean) {
            mean = static_cast<char *>(workspace) + aligned(ws.part);
            rstd = static_cast<char *>(mean) + ns;
        }
        long xl = (long)x_ld, yl = (long)y_ld, n = (long)N, rows = (long)sp.rows;
        int s = (int)S;
        float ef = (float)g.cfg.eps;
        double ed = g.cfg.eps;
        void *eps = g.real == 8 ? (void *)&ed : (void *)&ef;
        if (sp.chunks) {
            void *args[] = {&x, &xl, &ptr, &s, &n, &rows, &part};
            run(F[cgtp_group_norm::stats], sp.chunks, 64, args, stream);
        }
        void *jargs[] = {&ptr, &n, &rows, &part, &mean, &rstd, eps};
        run(F[cgtp_group_norm::join], S, join_threads(S), jargs, stream);
        if (sp.chunks) {
            void *args[] = {&x, &xl, &ptr, &s, &n, &rows, &w, &bias, &mean, &rstd, &y, &yl, &fill};
            run(F[cgtp_group_norm::apply], sp.chunks, 64, args, stream);
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
        const Split sp = split(g, N, true);
        char *at = static_cast<char *>(workspace);
        void *part = at, *stat = at + aligned(ws.part), *wpart = at + aligned(ws.part) + aligned(ws.stat);
        if (!weights) wpart = nullptr;
        long xl = (long)x_ld, dyl = (long)grad_y_ld, dxl = (long)grad_x_ld, n = (long)N, rows = (long)sp.rows;
        long chunks = work ? (long)sp.chunks : 0;
        int s = (int)S;
        if (work) {
            void *args[] = {&x, &xl, &grad_y, &dyl, &ptr, &s, &n, &rows, &w, &bias, &mean, &rstd, &part, &wpart};
            run(F[cgtp_group_norm::bwd_sums], sp.chunks, 64, args, stream);
            if (grad_x) {
                void *jargs[] = {&ptr, &n, &rows, &part, &stat};
                run(F[cgtp_group_norm::bwd_join], S, join_threads(S), jargs, stream);
                void *aargs[] = {&x, &xl, &grad_y, &dyl, &ptr, &s, &n, &rows, &w, &bias, &mean, &rstd, &stat, &grad_x, &dxl,
                                 &fill};
                run(F[cgtp_group_norm::bwd_apply], sp.chunks, 64, aargs, stream);
            }
        }
        if (weights) {
            void *args[] = {&wpart, &chunks, &grad_w, &grad_bias};
            run(F[cgtp_group_norm::columns], (2 * c + 15) / 16, 1024, args, stream);
        }
    });
}

}  // extern "C"
