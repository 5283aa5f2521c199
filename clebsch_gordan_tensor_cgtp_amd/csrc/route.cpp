// Routers: lane layout, the generated source's constants, and the entry points cgtp_router_* and
// cgtp_route_* (documented in include/cgtp.h).
#include "route.h"

#include <algorithm>
#include <cmath>
#include <memory>

#include "config_module.h"
#include "route_kernels.h"
#include "row_kernels.h"
#include "rows.h"

struct cgtp_router {
    cgtp_router_config cfg{};
    int elem = 4, real = 4;
    int groups = 1, lanes_per_group = 1, lanes = 1, epl = 1;  // groups: 1 where every one is taken
    cgtp::ConfigModule mod;
    enum { fwd, bwd };
};

namespace cgtp {

namespace {

int pow2_at_least(int n)
{
    int p = 1;
    while (p < n) p *= 2;
    return p;
}

// A lane holds at most 8 neighbouring experts of one group, 16 where a wave has no more lanes (512 experts in g
// groups, fewer than 2 g of them with the power of two's empty ones, on 64 lanes).
void lay_out(cgtp_router &r)
{
    r.elem = elem_bytes(r.cfg.dtype);
    r.real = real_bytes(r.cfg.dtype);
    r.groups = r.cfg.top_groups < r.cfg.groups ? r.cfg.groups : 1;
    const int width = r.cfg.experts / r.groups, slots = pow2_at_least(r.groups);
    if (slots > 64) throw Error(CGTP_ERR_UNSUPPORTED, "router: more than 64 groups");
    r.lanes_per_group = std::min(pow2_at_least((width + 7) / 8), 64 / slots);
    r.lanes = slots * r.lanes_per_group;
    r.epl = (width + r.lanes_per_group - 1) / r.lanes_per_group;
}

std::string constants(const cgtp_router &r)
{
    std::string s = "// routing to " + std::to_string(r.cfg.experts) + " experts\n";
    auto num = [&](const char *n, long v) { s += std::string("constexpr int ") + n + " = " + std::to_string(v) + ";\n"; };
    s += std::string("typedef ") + type_name(r.cfg.dtype) + " T;\n";
    s += std::string("typedef ") + (r.cfg.dtype == CGTP_F64 ? "double" : "float") + " R;\n";
    num("ACT", 0);
    num("E", r.cfg.experts);
    num("K", r.cfg.top_k);
    num("L", r.lanes);
    num("EPL", r.epl);
    num("NGRP", r.groups);
    num("GW", r.cfg.experts / r.groups);
    num("LPG", r.lanes_per_group);
    num("TOPG", r.groups == 1 ? 1 : r.cfg.top_groups);
    num("SIGMOID", r.cfg.score == CGTP_SCORE_SIGMOID);
    num("RENORM", r.cfg.renormalise ? 1 : 0);
    return s;
}

void check_slots(const cgtp_router &r, int64_t N)
{
    check_count(N);
    require(N <= (int64_t)INT_MAX / r.cfg.top_k, "N * top_k must be below 2^31");
}

}  // namespace

}  // namespace cgtp

using namespace cgtp;

extern "C" {

cgtp_status cgtp_router_create(const cgtp_router_config *config, cgtp_router **router_out)
{
    return guarded([&] {
        require(config && router_out, "NULL argument to cgtp_router_create");
        *router_out = nullptr;
        const cgtp_router_config &c = *config;
        require(c.dtype == CGTP_F32 || c.dtype == CGTP_F64 || c.dtype == CGTP_BF16 || c.dtype == CGTP_F16,
                "dtype must be CGTP_F32, CGTP_F64, CGTP_BF16 or CGTP_F16");
        require(c.score == CGTP_SCORE_SOFTMAX || c.score == CGTP_SCORE_SIGMOID, "score must be a cgtp_score");
        require(c.experts >= 1, "experts must be positive");
        require(c.groups >= 1 && c.experts % c.groups == 0, "groups must divide experts");
        require(c.top_groups >= 1 && c.top_groups <= c.groups, "top_groups must be in [1, groups]");
        require(c.top_k >= 1 && c.top_k <= c.experts / c.groups * c.top_groups,
                "top_k must be in [1, the experts of top_groups groups]");
        require(std::isfinite(c.scale), "scale must be finite");
        if (c.experts > kMaxExperts) throw Error(CGTP_ERR_UNSUPPORTED, "router: more than 512 experts");
        if (c.top_k > 32) throw Error(CGTP_ERR_UNSUPPORTED, "router: more than 32 experts of a row");
        auto h = std::make_unique<cgtp_router>();
        h->cfg = c;
        lay_out(*h);
        h->mod.build(constants(*h) + kRowKernels + kRouteKernels, {"cgtp_route_fwd", "cgtp_route_bwd"});
        *router_out = h.release();
    });
}

cgtp_status cgtp_router_destroy(cgtp_router *router)
{
    return guarded([&] {
        if (!router) return;
        router->mod.unload();
        delete router;
    });
}

const char *cgtp_router_source(const cgtp_router *router) { return router ? router->mod.source.c_str() : nullptr; }

cgtp_status cgtp_route_forward(const cgtp_router *router, int64_t N, const void *logits, int64_t logits_ld,
                               const void *bias, int32_t *experts, void *weights, void *stream)
{
    return guarded([&] {
        require(router != nullptr, "router is NULL");
        auto &r = *const_cast<cgtp_router *>(router);
        check_slots(r, N);
        if (N == 0) return;
        const int e = r.cfg.experts, k = r.cfg.top_k;
        const Rows X{logits, e, logits_ld, "logits"};
        check_rows(r.elem, N, X);
        if (bias) require_ptr(bias, "bias", r.real);
        require_ptr(experts, "experts", 4);
        require_ptr(weights, "weights", r.real);
        Arguments all(r.elem, N);
        all.rows(X, false);
        all.flat(bias, (size_t)e * r.real, "bias", false);
        all.flat(experts, (size_t)N * k * 4, "experts", true);
        all.flat(weights, (size_t)N * k * r.real, "weights", true);
        all.check();
        const auto &F = r.mod.here();
        long ld = (long)logits_ld, n = (long)N;
        double scale = r.cfg.scale;
        void *args[] = {&logits, &ld, &bias, &experts, &weights, &n, &scale};
        const int rows = 256 / r.lanes;
        run(F[cgtp_router::fwd], (N + rows - 1) / rows, 256, args, stream);
    });
}

cgtp_status cgtp_route_backward(const cgtp_router *router, int64_t N, const void *logits, int64_t logits_ld,
                                const int32_t *experts, const void *grad_weights, void *grad_logits, void *stream)
{
    return guarded([&] {
        require(router != nullptr, "router is NULL");
        auto &r = *const_cast<cgtp_router *>(router);
        check_slots(r, N);
        if (N == 0) return;
        const int e = r.cfg.experts, k = r.cfg.top_k;
        const Rows X{logits, e, logits_ld, "logits"}, G{grad_logits, e, e, "grad_logits"};
        check_rows(r.elem, N, X);
        check_rows(r.elem, N, G);
        require_ptr(experts, "experts", 4);
        require_ptr(grad_weights, "grad_weights", r.real);
        Arguments all(r.elem, N);
        all.rows(X, false);
        all.rows(G, true);
        all.flat(experts, (size_t)N * k * 4, "experts", false);
        all.flat(grad_weights, (size_t)N * k * r.real, "grad_weights", false);
        all.check();
        const auto &F = r.mod.here();
        long ld = (long)logits_ld, n = (long)N;
        double sd = r.cfg.scale;
        float sf = (float)sd;
        void *scale = r.real == 8 ? (void *)&sd : (void *)&sf;
        void *args[] = {&logits, &ld, &experts, &grad_weights, &grad_logits, &n, scale};
        const int rows = 256 / r.lanes;
        run(F[cgtp_router::bwd], (N + rows - 1) / rows, 256, args, stream);
    });
}

cgtp_status cgtp_route_order_workspace_size(const cgtp_router *router, int64_t N, size_t *bytes)
{
    return guarded([&] {
        require(router && bytes, "NULL argument to cgtp_route_order_workspace_size");
        check_slots(*router, N);
        *bytes = order_workspace(N, router->cfg.top_k, router->cfg.experts);
    });
}

cgtp_status cgtp_route_order(const cgtp_router *router, int64_t N, const int32_t *experts, int32_t *rows, int32_t *slots,
                             int32_t *offsets, void *workspace, size_t workspace_bytes, void *stream)
{
    return guarded([&] {
        require(router != nullptr, "router is NULL");
        check_slots(*router, N);
        const int e = router->cfg.experts, k = router->cfg.top_k;
        require_ptr(offsets, "offsets", 4);
        const size_t need = order_workspace(N, k, e);
        Arguments all(4, N);
        if (N > 0) {
            require_ptr(experts, "experts", 4);
            require_ptr(rows, "rows", 4);
            require_ptr(slots, "slots", 4);
            if (need) require_ptr(workspace, "workspace", 256);
            require(workspace_bytes >= need, "workspace too small (see cgtp_route_order_workspace_size)");
            all.flat(experts, (size_t)N * k * 4, "experts", false);
            all.flat(rows, (size_t)N * 4, "rows", true);
            all.flat(slots, (size_t)N * k * 4, "slots", true);
            all.flat(workspace, need, "workspace", true);
        }
        all.flat(offsets, (size_t)(e + 1) * 4, "offsets", true);
        all.check();
        check_hip(launch_order(N, k, e, experts, rows, slots, offsets, workspace, static_cast<hipStream_t>(stream)),
                  "cgtp_route_order");
    });
}

}  // extern "C"
