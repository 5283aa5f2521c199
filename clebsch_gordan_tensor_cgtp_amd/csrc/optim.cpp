// Entry points of the optimizer step: cgtp_adamw_*, cgtp_grad_norm (documented in include/cgtp.h).
#include "optim.h"

#include <algorithm>
#include <climits>
#include <cmath>
#include <iterator>
#include <memory>
#include <vector>

#include "abi_util.h"

struct cgtp_adamw {
    std::vector<int64_t> sizes;
    std::vector<int64_t> first;  // first unit of each tensor
    int64_t units = 0;
    cgtp_adamw_config cfg{};
    size_t elem = 4, real = 4;
};

using namespace cgtp;

namespace {

size_t moment_bytes(const cgtp_adamw &o) { return o.cfg.state_bits == 8 ? 1 : o.real; }

int64_t elements(const cgtp_adamw &o) { return o.units * kUnit; }

// Units of one launch: 256 threads each, and a launch's threads are counted in 32 bits.
constexpr int64_t kLaunchUnits = (int64_t)1 << 23;

// Calls `use` with tables of at most kTableTensors tensors and kLaunchUnits units, longer tensors in
// parts, the ones without a gradient and the empty ones left out.
template <class F> void each_table(const cgtp_adamw &o, void *const *params, const void *const *grads, F &&use)
{
    TensorTable t;
    int64_t units = 0;
    auto flush = [&] {
        if (t.n == 0) return;
        t.unit[t.n] = (int32_t)units;
        use(t);
        t.n = 0;
        units = 0;
    };
    for (size_t i = 0; i < o.sizes.size(); ++i) {
        if (!grads[i]) continue;
        for (int64_t done = 0; done < o.sizes[i];) {
            const int64_t part = std::min(o.sizes[i] - done, (kLaunchUnits - units) * kUnit);
            t.unit[t.n] = (int32_t)units;
            t.state[t.n] = (int32_t)(o.first[i] + done / kUnit);
            t.numel[t.n] = part;
            t.param[t.n] = params ? static_cast<char *>(params[i]) + done * o.elem : nullptr;
            t.grad[t.n] = static_cast<const char *>(grads[i]) + done * o.elem;
            units += (part + kUnit - 1) / kUnit;
            done += part;
            if (++t.n == kTableTensors || units == kLaunchUnits) flush();
        }
    }
    flush();
}

Elem elem_of(const cgtp_adamw &o) { return (Elem)o.cfg.dtype; }

void check_grads(const cgtp_adamw &o, const void *const *grads)
{
    require(grads != nullptr || o.sizes.empty(), "grads is NULL");
    for (size_t i = 0; i < o.sizes.size(); ++i)
        if (grads[i] && reinterpret_cast<uintptr_t>(grads[i]) % o.elem)
            require(false, "grads[" + std::to_string(i) + "] is not aligned to its elements");
}

// Memory that a call reads, or also writes.
struct Extent {
    const void *p;
    size_t n;
    bool written;
    const char *name;
};

// What is written overlaps nothing else: in the order of their starts, each extent begins after the
// end of every written one before it, a written one after the end of all.
// Each of the lists mostly comes in that order (tensors of one buffer): it is sorted only if not.
void check_extents(std::vector<Extent> &state, std::vector<Extent> &params, std::vector<Extent> &grads)
{
    auto at = [](const Extent &e) { return reinterpret_cast<uintptr_t>(e.p); };
    auto before = [&](const Extent &a, const Extent &b) { return at(a) < at(b); };
    std::vector<Extent> both, all;
    for (auto *list : {&state, &params, &grads})
        if (!std::is_sorted(list->begin(), list->end(), before)) std::sort(list->begin(), list->end(), before);
    both.reserve(params.size() + grads.size());
    all.reserve(both.capacity() + state.size());
    std::merge(params.begin(), params.end(), grads.begin(), grads.end(), std::back_inserter(both), before);
    std::merge(both.begin(), both.end(), state.begin(), state.end(), std::back_inserter(all), before);
    const Extent *any = nullptr, *written = nullptr;  // the ones that reach furthest
    auto ends = [&](const Extent *e) { return at(*e) + e->n; };
    for (const Extent &e : all) {
        if (!e.p || !e.n) continue;
        const Extent *last = e.written ? any : written;
        if (last && ends(last) > at(e)) require(false, std::string(e.name) + " overlaps " + last->name);
        if (!any || ends(&e) > ends(any)) any = &e;
        if (e.written && (!written || ends(&e) > ends(written))) written = &e;
    }
}

// one partial per workgroup of each launch; a launch ends at a full table or at kLaunchUnits
size_t norm_workspace(const cgtp_adamw &o)
{
    const int64_t launches = ((int64_t)o.sizes.size() + kTableTensors - 1) / kTableTensors + o.units / kLaunchUnits;
    return (size_t)launches * kNormGroups * sizeof(double);
}

}  // namespace

extern "C" {

cgtp_status cgtp_adamw_create(int32_t n_tensors, const int64_t *sizes, const cgtp_adamw_config *config,
                              cgtp_adamw **opt_out)
{
    return guarded([&] {
        require(config && opt_out && (sizes || n_tensors == 0), "NULL argument to cgtp_adamw_create");
        *opt_out = nullptr;
        require(n_tensors >= 0, "n_tensors is negative");
        const cgtp_adamw_config &c = *config;
        require(c.dtype == CGTP_F32 || c.dtype == CGTP_F64 || c.dtype == CGTP_BF16 || c.dtype == CGTP_F16,
                "dtype must be CGTP_F32, CGTP_F64, CGTP_BF16 or CGTP_F16");
        require(c.state_bits == 32 || c.state_bits == 8, "state_bits must be 32 or 8");
        require(c.master == 0 || c.dtype == CGTP_BF16 || c.dtype == CGTP_F16,
                "master copies belong to 16-bit tensors");
        if (c.state_bits == 8 && c.dtype == CGTP_F64)
            throw Error(CGTP_ERR_UNSUPPORTED, "double precision tensors have no 8-bit moments");
        auto o = std::make_unique<cgtp_adamw>();
        o->cfg = c;
        o->elem = c.dtype == CGTP_F64 ? 8 : c.dtype == CGTP_F32 ? 4 : 2;
        o->real = c.dtype == CGTP_F64 ? 8 : 4;
        for (int32_t i = 0; i < n_tensors; ++i) {
            require(sizes[i] >= 0 && sizes[i] < ((int64_t)1 << 40), "a tensor's size is out of range");
            o->sizes.push_back(sizes[i]);
            o->first.push_back(o->units);
            o->units += (sizes[i] + kUnit - 1) / kUnit;
            require(o->units < INT_MAX / 2, "the tensors hold more than 2^41 elements");
        }
        *opt_out = o.release();
    });
}

cgtp_status cgtp_adamw_destroy(cgtp_adamw *opt)
{
    delete opt;
    return CGTP_OK;
}

cgtp_status cgtp_adamw_info_get(const cgtp_adamw *opt, cgtp_adamw_info *info)
{
    return guarded([&] {
        require(opt && info, "NULL argument to cgtp_adamw_info_get");
        info->n_tensors = (int32_t)opt->sizes.size();
        info->elements = elements(*opt);
        info->blocks = elements(*opt) / kScaleBlock;
        info->norm_workspace = (int64_t)norm_workspace(*opt);
    });
}

cgtp_status cgtp_adamw_offset(const cgtp_adamw *opt, int32_t tensor, int64_t *offset)
{
    return guarded([&] {
        require(opt && offset, "NULL argument to cgtp_adamw_offset");
        require(tensor >= 0 && (size_t)tensor < opt->sizes.size(), "tensor out of range");
        *offset = opt->first[tensor] * kUnit;
    });
}

cgtp_status cgtp_grad_norm(const cgtp_adamw *opt, const void *const *grads, double *norm, void *workspace,
                           size_t workspace_bytes, void *stream)
{
    return guarded([&] {
        require(opt != nullptr, "opt is NULL");
        const cgtp_adamw &o = *opt;
        check_grads(o, grads);
        require_ptr(norm, "norm", 8);
        const size_t need = norm_workspace(o);
        if (need) require_ptr(workspace, "workspace", 256);
        require(workspace_bytes >= need, "workspace too small (see cgtp_adamw_info)");
        require_disjoint(norm, 8, "norm", workspace, need, "workspace");
        for (size_t i = 0; i < o.sizes.size(); ++i) {
            require_disjoint(grads[i], o.sizes[i] * o.elem, "a gradient", norm, 8, "norm");
            require_disjoint(grads[i], o.sizes[i] * o.elem, "a gradient", workspace, need, "workspace");
        }
        hipStream_t st = static_cast<hipStream_t>(stream);
        double *part = static_cast<double *>(workspace);
        int64_t n = 0;
        each_table(o, nullptr, grads, [&](const TensorTable &t) {
            check_hip(launch_square_sums(elem_of(o), t, part + n, st), "gradient norm launch");
            n += grad_norm_groups(t.unit[t.n]);
        });
        check_hip(launch_norm(part, n, norm, st), "gradient norm launch");
    });
}

cgtp_status cgtp_adamw_step(const cgtp_adamw *opt, void *const *params, const void *const *grads, void *m, void *v,
                            float *scales, float *master, const cgtp_adamw_hyper *hyper, const double *norm,
                            const double *schedule, void *stream)
{
    return guarded([&] {
        require(opt && hyper, "opt or hyper is NULL");
        const cgtp_adamw &o = *opt;
        const cgtp_adamw_hyper &h = *hyper;
        require(std::isfinite(h.lr) && h.lr >= 0, "lr must be finite and not negative");
        require(h.beta1 >= 0 && h.beta1 < 1 && h.beta2 >= 0 && h.beta2 < 1, "betas must lie in [0, 1)");
        require(std::isfinite(h.eps) && h.eps > 0 && (o.real == 8 || h.eps >= 1e-30),
                "eps must be finite and positive (at least 1e-30 where arithmetic is float)");
        require(std::isfinite(h.weight_decay) && h.weight_decay >= 0, "weight_decay must be finite and not negative");
        require(h.max_norm >= 0, "max_norm must not be negative or NaN (0: no clipping)");
        require(std::isfinite(h.grad_scale), "grad_scale must be finite");
        require(h.max_norm == 0 || norm != nullptr, "max_norm needs norm");
        require(schedule != nullptr || h.step >= 1, "step counts from 1");
        if (norm) require_ptr(norm, "norm", 8);
        if (schedule) require_ptr(schedule, "schedule", 8);
        check_grads(o, grads);
        require(params != nullptr || o.sizes.empty(), "params is NULL");
        const size_t el = (size_t)elements(o);
        if (el == 0) return;
        const size_t mbytes = el * moment_bytes(o);
        const bool codes = o.cfg.state_bits == 8;
        require_ptr(m, "m", 16);
        require_ptr(v, "v", 16);
        if (codes) require_ptr(scales, "scales", 4);
        require(codes || !scales, "scales given to moments in 32 bits");
        if (o.cfg.master) require_ptr(master, "master", 16);
        require(o.cfg.master || !master, "master given to an optimizer without master copies");
        std::vector<Extent> state = {{m, mbytes, true, "m"},
                                     {v, mbytes, true, "v"},
                                     {scales, codes ? el / kScaleBlock * 8 : 0, true, "scales"},
                                     {master, master ? el * 4 : 0, true, "master"},
                                     {norm, norm ? (size_t)8 : 0, false, "norm"},
                                     {schedule, schedule ? (size_t)32 : 0, false, "schedule"}};
        std::vector<Extent> tensors, gradients;
        tensors.reserve(o.sizes.size());
        gradients.reserve(o.sizes.size());
        for (size_t i = 0; i < o.sizes.size(); ++i) {
            if (o.sizes[i] == 0 || !grads[i]) continue;
            const size_t bytes = (size_t)o.sizes[i] * o.elem;
            if (!params[i] || reinterpret_cast<uintptr_t>(params[i]) % o.elem)
                require(false, "params[" + std::to_string(i) + "] is NULL or not aligned to its elements");
            tensors.push_back({params[i], bytes, true, "a tensor"});
            gradients.push_back({grads[i], bytes, false, "a gradient"});
        }
        check_extents(state, tensors, gradients);
        StepScalars s{h.max_norm, h.grad_scale, h.lr, h.beta1, h.beta2, h.eps, h.weight_decay, 1, 1};
        if (!schedule) {
            s.bias1 = 1 - std::pow(h.beta1, (double)h.step);
            s.bias2 = 1 - std::pow(h.beta2, (double)h.step);
        }
        const MomentBuffers mb{m, v, scales, master, (int64_t)(el / kScaleBlock)};
        each_table(o, params, grads, [&](const TensorTable &t) {
            check_hip(launch_adamw(elem_of(o), codes, t, mb, s, norm, schedule, static_cast<hipStream_t>(stream)),
                      "adamw launch");
        });
    });
}

cgtp_status cgtp_adamw_schedule(double *schedule, double beta1, double beta2, void *stream)
{
    return cgtp_adamw_schedule_norm(schedule, beta1, beta2, nullptr, 1, stream);
}

cgtp_status cgtp_adamw_schedule_norm(double *schedule, double beta1, double beta2, const double *norm,
                                     double grad_scale, void *stream)
{
    return guarded([&] {
        require_ptr(schedule, "schedule", 8);
        require(beta1 >= 0 && beta1 < 1 && beta2 >= 0 && beta2 < 1, "betas must lie in [0, 1)");
        require(std::isfinite(grad_scale), "grad_scale must be finite");
        if (norm) require_ptr(norm, "norm", 8);
        require_disjoint(schedule, 32, "schedule", norm, 8, "norm");
        check_hip(launch_schedule(schedule, beta1, beta2, norm, grad_scale, static_cast<hipStream_t>(stream)),
                  "schedule launch");
    });
}

cgtp_status cgtp_adamw_state_read(const cgtp_adamw *opt, const void *m, const void *v, const float *scales,
                                  float *m_out, float *v_out, void *stream)
{
    return guarded([&] {
        require(opt != nullptr, "opt is NULL");
        if (opt->cfg.state_bits != 8) throw Error(CGTP_ERR_UNSUPPORTED, "moments in 32 bits are read as they are");
        const size_t el = (size_t)elements(*opt);
        if (el == 0 || (!m_out && !v_out)) return;
        require_ptr(m, "m", 16);
        require_ptr(v, "v", 16);
        require_ptr(scales, "scales", 4);
        if (m_out) require_ptr(m_out, "m_out", 16);
        if (v_out) require_ptr(v_out, "v_out", 16);
        struct { const void *p; size_t n; const char *name; } io[] = {
            {m_out, m_out ? el * 4 : 0, "m_out"}, {v_out, v_out ? el * 4 : 0, "v_out"}, {m, el, "m"}, {v, el, "v"},
            {scales, el / kScaleBlock * 8, "scales"}};
        for (int i = 0; i < 2; ++i)
            for (int j = i + 1; j < 5; ++j) require_disjoint(io[i].p, io[i].n, io[i].name, io[j].p, io[j].n, io[j].name);
        check_hip(launch_state_read(m, v, scales, (int64_t)el, m_out, v_out, static_cast<hipStream_t>(stream)),
                  "state read launch");
    });
}

cgtp_status cgtp_adamw_state_write(const cgtp_adamw *opt, const float *m_in, const float *v_in, void *m, void *v,
                                   float *scales, void *stream)
{
    return guarded([&] {
        require(opt != nullptr, "opt is NULL");
        if (opt->cfg.state_bits != 8) throw Error(CGTP_ERR_UNSUPPORTED, "moments in 32 bits are written as they are");
        const size_t el = (size_t)elements(*opt);
        if (el == 0) return;
        require_ptr(m, "m", 16);
        require_ptr(v, "v", 16);
        require_ptr(scales, "scales", 4);
        require_ptr(m_in, "m_in", 16);
        require_ptr(v_in, "v_in", 16);
        struct { const void *p; size_t n; const char *name; } io[] = {
            {m, el, "m"}, {v, el, "v"}, {scales, el / kScaleBlock * 8, "scales"}, {m_in, el * 4, "m_in"},
            {v_in, el * 4, "v_in"}};
        for (int i = 0; i < 3; ++i)
            for (int j = i + 1; j < 5; ++j) require_disjoint(io[i].p, io[i].n, io[i].name, io[j].p, io[j].n, io[j].name);
        check_hip(launch_state_write(m_in, v_in, (int64_t)el, m, v, scales, static_cast<hipStream_t>(stream)),
                  "state write launch");
    });
}

}  // extern "C"
