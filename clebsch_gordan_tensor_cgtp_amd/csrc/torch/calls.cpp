// The block, group norm, routing, experts' and optimizer calls from Python, for the ordinary call, whose outputs are all new: checks,
// outputs, the current stream and the C entry point in compiled code (a small join takes 5.9 us
// here and 11.9 us through ctypes, of which the launch is 3).  Each function returns None where an
// argument is not as its entry point wants it; binding.py then goes its own way, through ctypes, and
// says what is wrong.  A status that is not CGTP_OK is returned as a number.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <vector>

#include "cgtp.h"

namespace {

struct BlockMeta {
    const cgtp_block *block;
    int64_t d, channels, gate_width;
    bool post, next;
    at::ScalarType rows, real;
};

struct AdamWMeta {
    const cgtp_adamw *opt;
    std::vector<int64_t> sizes;
    int64_t elements, blocks, norm_workspace;
    bool codes;
    at::ScalarType elem, real;
};

struct GroupNormMeta {
    const cgtp_group_norm *norm;
    int64_t channels, groups;
    at::ScalarType rows, real;
};

struct RouterMeta {
    const cgtp_router *router;
    int64_t experts, top_k;
    at::ScalarType rows, real;
};

struct LinearMeta {
    const cgtp_linear *linear;
    int64_t d_in, d_out, experts, top_k, numel;
    at::ScalarType rows, real;
};

const char *const kBlock = "cgtp.block", *const kAdamW = "cgtp.adamw", *const kGroupNorm = "cgtp.group_norm",
           *const kRouter = "cgtp.router", *const kLinear = "cgtp.linear";

at::ScalarType elem_type(long dtype)
{
    return dtype == CGTP_F64 ? at::kDouble : dtype == CGTP_BF16 ? at::kBFloat16 : dtype == CGTP_F16 ? at::kHalf : at::kFloat;
}

const at::Tensor *tensor(PyObject *o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

// Addresses of a call's tensors; `fine` while every one is as it has to be, on the device that is the
// current one, where launches go (binding.py makes another device the current one).
struct Args {
    int64_t device;
    bool fine = true;

    explicit Args(const at::Tensor *first) : device(first && first->is_cuda() ? first->get_device() : -1)
    {
        fine = device >= 0 && device == c10::hip::current_device();
    }

    bool here(const at::Tensor *x, at::ScalarType t) const
    {
        return x && x->is_cuda() && x->get_device() == device && x->scalar_type() == t;
    }

    // a contiguous tensor of this type and shape; None where it may be absent
    void *at(PyObject *o, at::ScalarType t, at::IntArrayRef shape, bool optional = false)
    {
        if (o == Py_None) {
            fine = fine && optional;
            return nullptr;
        }
        const at::Tensor *x = tensor(o);
        if (!here(x, t) || x->sizes() != shape || !x->is_contiguous()) {
            fine = false;
            return nullptr;
        }
        return x->data_ptr();
    }

    // n rows of `width` consecutive elements, `ld` elements apart; None where the width is 0
    void *rows(PyObject *o, at::ScalarType t, int64_t n, int64_t width, int64_t *ld)
    {
        *ld = width;
        if (width == 0) {
            fine = fine && o == Py_None;
            return nullptr;
        }
        const at::Tensor *x = tensor(o);
        if (!here(x, t) || x->dim() != 2 || x->size(0) != n || x->size(1) != width || (width > 1 && x->stride(1) != 1)) {
            fine = false;
            return nullptr;
        }
        if (n > 1) *ld = x->stride(0);
        fine = fine && *ld >= width;
        return x->data_ptr();
    }

    void *stream() const { return c10::hip::getCurrentHIPStream((c10::DeviceIndex)device).stream(); }
};

void *address(const at::Tensor &t) { return t.defined() ? t.data_ptr() : nullptr; }

PyObject *answer(cgtp_status status, std::initializer_list<const at::Tensor *> tensors)
{
    if (status != CGTP_OK) return PyLong_FromLong(status);
    PyObject *out = PyTuple_New((Py_ssize_t)tensors.size());
    if (!out) return nullptr;
    Py_ssize_t i = 0;
    for (const at::Tensor *t : tensors) {
        PyObject *o = t->defined() ? THPVariable_Wrap(*t) : Py_None;
        if (!o) {
            Py_DECREF(out);
            return nullptr;
        }
        if (o == Py_None) Py_INCREF(o);
        PyTuple_SET_ITEM(out, i++, o);
    }
    return out;
}

bool takes(Py_ssize_t given, Py_ssize_t wanted)
{
    if (given != wanted) PyErr_Format(PyExc_TypeError, "%zd arguments given, %zd wanted", given, wanted);
    return given == wanted;
}

// ------------------------------------------------------------------------------------------ blocks

// (handle, d, channels, gate_width, post_norm, next_norm, dtype)
PyObject *block(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (!takes(n, 7)) return nullptr;
    const long dtype = PyLong_AsLong(a[6]);
    auto *m = new BlockMeta{static_cast<const cgtp_block *>(PyLong_AsVoidPtr(a[0])),
                            PyLong_AsLongLong(a[1]), PyLong_AsLongLong(a[2]), PyLong_AsLongLong(a[3]),
                            PyObject_IsTrue(a[4]) == 1, PyObject_IsTrue(a[5]) == 1, elem_type(dtype),
                            dtype == CGTP_F64 ? at::kDouble : at::kFloat};
    if (PyErr_Occurred()) {
        delete m;
        return nullptr;
    }
    return PyCapsule_New(m, kBlock,
                         [](PyObject *o) { delete static_cast<BlockMeta *>(PyCapsule_GetPointer(o, kBlock)); });
    END_HANDLE_TH_ERRORS
}

const BlockMeta *block_of(PyObject *o) { return static_cast<const BlockMeta *>(PyCapsule_GetPointer(o, kBlock)); }

// (block, x, w, need_rstd) -> (u, rstd)
PyObject *norm_forward(PyObject *, PyObject *const *a, Py_ssize_t n_args)
{
    HANDLE_TH_ERRORS
    if (!takes(n_args, 4)) return nullptr;
    if (a[0] == Py_None) Py_RETURN_NONE;  // closed
    const BlockMeta *m = block_of(a[0]);
    if (!m) return nullptr;
    const at::Tensor *x = tensor(a[1]);
    Args in(x);
    if (!in.fine || x->dim() != 2) Py_RETURN_NONE;
    const int64_t n = x->size(0);
    int64_t ld;
    const void *xp = in.rows(a[1], m->rows, n, m->d, &ld), *w = in.at(a[2], m->real, {m->channels}, true);
    if (!in.fine) Py_RETURN_NONE;
    at::Tensor u = at::empty({n, m->d}, x->options()), rstd;
    if (PyObject_IsTrue(a[3]) == 1) rstd = at::empty({n}, x->options().dtype(m->real));
    return answer(cgtp_norm_forward(m->block, n, xp, ld, w, address(u), address(rstd), in.stream()), {&u, &rstd});
    END_HANDLE_TH_ERRORS
}

// a workspace of the block's size for n rows
cgtp_status workspace_for(const BlockMeta *m, int64_t n, const at::Tensor &like, at::Tensor *ws, size_t *bytes)
{
    const cgtp_status st = cgtp_block_workspace_size(m->block, n, bytes);
    if (st == CGTP_OK && *bytes) *ws = at::empty({(int64_t)*bytes}, like.options().dtype(at::kByte));
    return st;
}

// (block, x, w, rstd, grad_u, grad_add, need_x, need_w) -> (grad_x, grad_w)
PyObject *norm_backward(PyObject *, PyObject *const *a, Py_ssize_t n_args)
{
    HANDLE_TH_ERRORS
    if (!takes(n_args, 8)) return nullptr;
    if (a[0] == Py_None) Py_RETURN_NONE;  // closed
    const BlockMeta *m = block_of(a[0]);
    if (!m) return nullptr;
    const at::Tensor *x = tensor(a[1]);
    Args in(x);
    if (!in.fine || x->dim() != 2) Py_RETURN_NONE;
    const int64_t n = x->size(0);
    int64_t ld;
    const void *xp = in.rows(a[1], m->rows, n, m->d, &ld), *w = in.at(a[2], m->real, {m->channels}, true),
               *rstd = in.at(a[3], m->real, {n}), *du = in.at(a[4], m->rows, {n, m->d}),
               *add = in.at(a[5], m->rows, {n, m->d}, true);
    if (!in.fine) Py_RETURN_NONE;
    at::Tensor gx, gw, ws;
    size_t bytes = 0;
    if (PyObject_IsTrue(a[6]) == 1) gx = at::empty({n, m->d}, x->options());
    cgtp_status st = CGTP_OK;
    if (PyObject_IsTrue(a[7]) == 1) {
        gw = at::empty({m->channels}, x->options().dtype(m->real));
        st = workspace_for(m, n, *x, &ws, &bytes);
    }
    if (st == CGTP_OK)
        st = cgtp_norm_backward(m->block, n, xp, ld, w, rstd, du, add, address(gx), address(gw), address(ws), bytes,
                                in.stream());
    return answer(st, {&gx, &gw});
    END_HANDLE_TH_ERRORS
}

// (block, res, f, gate, w_post, scale, w_next, need_rstd) -> (h, u, rstd_f, rstd_h)
PyObject *join_forward(PyObject *, PyObject *const *a, Py_ssize_t n_args)
{
    HANDLE_TH_ERRORS
    if (!takes(n_args, 8)) return nullptr;
    if (a[0] == Py_None) Py_RETURN_NONE;  // closed
    const BlockMeta *m = block_of(a[0]);
    if (!m) return nullptr;
    const at::Tensor *f = tensor(a[2]);
    Args in(f);
    if (!in.fine || f->dim() != 2) Py_RETURN_NONE;
    const int64_t n = f->size(0);
    int64_t f_ld, g_ld;
    const void *fp = in.rows(a[2], m->rows, n, m->d, &f_ld), *gp = in.rows(a[3], m->rows, n, m->gate_width, &g_ld),
               *res = in.at(a[1], m->rows, {n, m->d}), *wp = in.at(a[4], m->real, {m->channels}, true),
               *sc = in.at(a[5], m->real, {m->channels}, true), *wn = in.at(a[6], m->real, {m->channels}, true);
    if (!in.fine) Py_RETURN_NONE;
    const bool stats = PyObject_IsTrue(a[7]) == 1;
    const auto real = f->options().dtype(m->real);
    at::Tensor h = at::empty({n, m->d}, f->options()), u, rf, rh;
    if (m->next) u = at::empty({n, m->d}, f->options());
    if (m->post && stats) rf = at::empty({n}, real);
    if (m->next && stats) rh = at::empty({n}, real);
    return answer(cgtp_join_forward(m->block, n, res, fp, f_ld, gp, g_ld, wp, sc, wn, address(h), address(u),
                                    address(rf), address(rh), in.stream()),
                  {&h, &u, &rf, &rh});
    END_HANDLE_TH_ERRORS
}

// (block, grad_h, grad_u, h, f, gate, w_post, scale, w_next, rstd_f, rstd_h, need of the six) ->
// (grad_res, grad_f, grad_gate, grad_w_post, grad_scale, grad_w_next)
PyObject *join_backward(PyObject *, PyObject *const *a, Py_ssize_t n_args)
{
    HANDLE_TH_ERRORS
    if (!takes(n_args, 12)) return nullptr;
    if (a[0] == Py_None) Py_RETURN_NONE;  // closed
    const BlockMeta *m = block_of(a[0]);
    if (!m) return nullptr;
    const at::Tensor *f = tensor(a[4]);
    Args in(f);
    if (!in.fine || f->dim() != 2 || !PyTuple_Check(a[11]) || PyTuple_GET_SIZE(a[11]) != 6) Py_RETURN_NONE;
    const int64_t n = f->size(0);
    int64_t f_ld, g_ld;
    const void *fp = in.rows(a[4], m->rows, n, m->d, &f_ld), *gp = in.rows(a[5], m->rows, n, m->gate_width, &g_ld),
               *dh = in.at(a[1], m->rows, {n, m->d}, true), *du = in.at(a[2], m->rows, {n, m->d}, true),
               *h = in.at(a[3], m->rows, {n, m->d}, true), *wp = in.at(a[6], m->real, {m->channels}, true),
               *sc = in.at(a[7], m->real, {m->channels}, true), *wn = in.at(a[8], m->real, {m->channels}, true),
               *rf = in.at(a[9], m->real, {n}, true), *rh = in.at(a[10], m->real, {n}, true);
    if (!in.fine) Py_RETURN_NONE;
    const bool has[6] = {true, true, m->gate_width > 0, m->post, true, m->next};
    at::Tensor g[6], ws;
    const auto rows = f->options(), real = f->options().dtype(m->real);
    for (int i = 0; i < 6; ++i) {
        if (!has[i] || PyObject_IsTrue(PyTuple_GET_ITEM(a[11], i)) != 1) continue;
        if (i < 3)
            g[i] = at::empty({n, i == 2 ? m->gate_width : m->d}, rows);
        else
            g[i] = at::empty({m->channels}, real);
    }
    size_t bytes = 0;
    cgtp_status st = CGTP_OK;
    if (g[3].defined() || g[4].defined() || g[5].defined()) st = workspace_for(m, n, *f, &ws, &bytes);
    if (st == CGTP_OK)
        st = cgtp_join_backward(m->block, n, dh, du, h, fp, f_ld, gp, g_ld, wp, sc, wn, rf, rh, address(g[0]),
                                address(g[1]), m->d, address(g[2]), m->gate_width, address(g[3]), address(g[4]),
                                address(g[5]), address(ws), bytes, in.stream());
    return answer(st, {&g[0], &g[1], &g[2], &g[3], &g[4], &g[5]});
    END_HANDLE_TH_ERRORS
}

// ------------------------------------------------------------------------------------------ experts

template <class M> PyObject *capsule(M *m, const char *name, PyCapsule_Destructor drop)
{
    if (PyErr_Occurred()) {
        delete m;
        return nullptr;
    }
    return PyCapsule_New(m, name, drop);
}

at::ScalarType real_type(long dtype) { return dtype == CGTP_F64 ? at::kDouble : at::kFloat; }

// (handle, channels, groups, dtype)
PyObject *group_norm(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (!takes(n, 4)) return nullptr;
    const long dtype = PyLong_AsLong(a[3]);
    return capsule(new GroupNormMeta{static_cast<const cgtp_group_norm *>(PyLong_AsVoidPtr(a[0])), PyLong_AsLongLong(a[1]),
                                     PyLong_AsLongLong(a[2]), elem_type(dtype), real_type(dtype)},
                   kGroupNorm, [](PyObject *o) { delete static_cast<GroupNormMeta *>(PyCapsule_GetPointer(o, kGroupNorm)); });
    END_HANDLE_TH_ERRORS
}

// the graphs of row pointers ptr; -1 where they are none
int64_t graphs_of(const Args &in, PyObject *o, const int32_t **ptr)
{
    const at::Tensor *t = tensor(o);
    if (!in.here(t, at::kInt) || t->dim() != 1 || t->size(0) < 1 || !t->is_contiguous()) return -1;
    *ptr = static_cast<const int32_t *>(t->data_ptr());
    return t->size(0) - 1;
}

// (norm, x, ptr, w, bias, need_stats) -> (y, mean, rstd)
PyObject *group_norm_forward(PyObject *, PyObject *const *a, Py_ssize_t n_args)
{
    HANDLE_TH_ERRORS
    if (!takes(n_args, 6)) return nullptr;
    if (a[0] == Py_None) Py_RETURN_NONE;  // closed
    const auto *m = static_cast<const GroupNormMeta *>(PyCapsule_GetPointer(a[0], kGroupNorm));
    if (!m) return nullptr;
    const at::Tensor *x = tensor(a[1]);
    Args in(x);
    if (!in.fine || x->dim() != 2) Py_RETURN_NONE;
    const int64_t n = x->size(0);
    int64_t ld;
    const int32_t *ptr = nullptr;
    const int64_t s = graphs_of(in, a[2], &ptr);
    const void *xp = in.rows(a[1], m->rows, n, m->channels, &ld), *w = in.at(a[3], m->real, {m->channels}, true),
               *bias = in.at(a[4], m->real, {m->channels}, true);
    if (!in.fine || s < 0) Py_RETURN_NONE;
    const auto real = x->options().dtype(m->real);
    at::Tensor y = at::empty({n, m->channels}, x->options()), mean, rstd, ws;
    if (PyObject_IsTrue(a[5]) == 1) {
        mean = at::empty({s, m->groups}, real);
        rstd = at::empty({s, m->groups}, real);
    }
    size_t bytes = 0;
    cgtp_status st = cgtp_group_norm_workspace_size(m->norm, n, s, 0, &bytes);
    if (st == CGTP_OK && bytes) ws = at::empty({(int64_t)bytes}, x->options().dtype(at::kByte));
    if (st == CGTP_OK)
        st = cgtp_group_norm_forward(m->norm, n, s, ptr, xp, ld, w, bias, address(y), m->channels, 1, address(mean),
                                     address(rstd), address(ws), bytes, in.stream());
    return answer(st, {&y, &mean, &rstd});
    END_HANDLE_TH_ERRORS
}

// (norm, x, ptr, w, bias, mean, rstd, grad_y, need of the three) -> (grad_x, grad_w, grad_bias)
PyObject *group_norm_backward(PyObject *, PyObject *const *a, Py_ssize_t n_args)
{
    HANDLE_TH_ERRORS
    if (!takes(n_args, 11)) return nullptr;
    if (a[0] == Py_None) Py_RETURN_NONE;  // closed
    const auto *m = static_cast<const GroupNormMeta *>(PyCapsule_GetPointer(a[0], kGroupNorm));
    if (!m) return nullptr;
    const at::Tensor *x = tensor(a[1]);
    Args in(x);
    if (!in.fine || x->dim() != 2) Py_RETURN_NONE;
    const int64_t n = x->size(0), c = m->channels;
    int64_t ld, dy_ld;
    const int32_t *ptr = nullptr;
    const int64_t s = graphs_of(in, a[2], &ptr);
    if (s < 0) Py_RETURN_NONE;
    const void *xp = in.rows(a[1], m->rows, n, c, &ld), *w = in.at(a[3], m->real, {c}, true),
               *bias = in.at(a[4], m->real, {c}, true), *mean = in.at(a[5], m->real, {s, m->groups}),
               *rstd = in.at(a[6], m->real, {s, m->groups}), *dy = in.rows(a[7], m->rows, n, c, &dy_ld);
    if (!in.fine) Py_RETURN_NONE;
    const auto real = x->options().dtype(m->real);
    at::Tensor gx, gw, gb, ws;
    if (PyObject_IsTrue(a[8]) == 1) gx = at::empty({n, c}, x->options());
    if (PyObject_IsTrue(a[9]) == 1) gw = at::empty({c}, real);
    if (PyObject_IsTrue(a[10]) == 1) gb = at::empty({c}, real);
    size_t bytes = 0;
    cgtp_status st = cgtp_group_norm_workspace_size(m->norm, n, s, 1, &bytes);
    if (st == CGTP_OK && bytes) ws = at::empty({(int64_t)bytes}, x->options().dtype(at::kByte));
    if (st == CGTP_OK)
        st = cgtp_group_norm_backward(m->norm, n, s, ptr, xp, ld, w, bias, mean, rstd, dy, dy_ld, address(gx), c, 1,
                                      address(gw), address(gb), address(ws), bytes, in.stream());
    return answer(st, {&gx, &gw, &gb});
    END_HANDLE_TH_ERRORS
}

// (handle, experts, top_k, dtype)
PyObject *router(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (!takes(n, 4)) return nullptr;
    const long dtype = PyLong_AsLong(a[3]);
    return capsule(new RouterMeta{static_cast<const cgtp_router *>(PyLong_AsVoidPtr(a[0])), PyLong_AsLongLong(a[1]),
                                  PyLong_AsLongLong(a[2]), elem_type(dtype), real_type(dtype)},
                   kRouter, [](PyObject *o) { delete static_cast<RouterMeta *>(PyCapsule_GetPointer(o, kRouter)); });
    END_HANDLE_TH_ERRORS
}

const RouterMeta *router_of(PyObject *o) { return static_cast<const RouterMeta *>(PyCapsule_GetPointer(o, kRouter)); }

// (router, logits, bias) -> (experts, weights)
PyObject *route_forward(PyObject *, PyObject *const *a, Py_ssize_t n_args)
{
    HANDLE_TH_ERRORS
    if (!takes(n_args, 3)) return nullptr;
    if (a[0] == Py_None) Py_RETURN_NONE;  // closed
    const RouterMeta *m = router_of(a[0]);
    if (!m) return nullptr;
    const at::Tensor *l = tensor(a[1]);
    Args in(l);
    if (!in.fine || l->dim() != 2) Py_RETURN_NONE;
    const int64_t n = l->size(0);
    int64_t ld;
    const void *lp = in.rows(a[1], m->rows, n, m->experts, &ld), *bias = in.at(a[2], m->real, {m->experts}, true);
    if (!in.fine) Py_RETURN_NONE;
    at::Tensor experts = at::empty({n, m->top_k}, l->options().dtype(at::kInt)),
               weights = at::empty({n, m->top_k}, l->options().dtype(m->real));
    return answer(cgtp_route_forward(m->router, n, lp, ld, bias, static_cast<int32_t *>(address(experts)), address(weights),
                                     in.stream()),
                  {&experts, &weights});
    END_HANDLE_TH_ERRORS
}

// (router, logits, experts, grad_weights) -> (grad_logits,)
PyObject *route_backward(PyObject *, PyObject *const *a, Py_ssize_t n_args)
{
    HANDLE_TH_ERRORS
    if (!takes(n_args, 4)) return nullptr;
    if (a[0] == Py_None) Py_RETURN_NONE;  // closed
    const RouterMeta *m = router_of(a[0]);
    if (!m) return nullptr;
    const at::Tensor *l = tensor(a[1]);
    Args in(l);
    if (!in.fine || l->dim() != 2) Py_RETURN_NONE;
    const int64_t n = l->size(0);
    int64_t ld;
    const void *lp = in.rows(a[1], m->rows, n, m->experts, &ld), *e = in.at(a[2], at::kInt, {n, m->top_k}),
               *g = in.at(a[3], m->real, {n, m->top_k});
    if (!in.fine) Py_RETURN_NONE;
    at::Tensor out = at::empty({n, m->experts}, l->options());
    return answer(cgtp_route_backward(m->router, n, lp, ld, static_cast<const int32_t *>(e), g, address(out), in.stream()), {&out});
    END_HANDLE_TH_ERRORS
}

// (router, experts) -> (rows, slots, offsets)
PyObject *route_order(PyObject *, PyObject *const *a, Py_ssize_t n_args)
{
    HANDLE_TH_ERRORS
    if (!takes(n_args, 2)) return nullptr;
    if (a[0] == Py_None) Py_RETURN_NONE;  // closed
    const RouterMeta *m = router_of(a[0]);
    if (!m) return nullptr;
    const at::Tensor *x = tensor(a[1]);
    Args in(x);
    if (!in.fine || x->dim() != 2) Py_RETURN_NONE;
    const int64_t n = x->size(0);
    const void *e = in.at(a[1], at::kInt, {n, m->top_k});
    if (!in.fine) Py_RETURN_NONE;
    at::Tensor rows = at::empty({n}, x->options()), slots = at::empty({n * m->top_k}, x->options()),
               offsets = at::empty({m->experts + 1}, x->options()), ws;
    size_t bytes = 0;
    cgtp_status st = cgtp_route_order_workspace_size(m->router, n, &bytes);
    if (st == CGTP_OK && bytes) ws = at::empty({(int64_t)bytes}, x->options().dtype(at::kByte));
    if (st == CGTP_OK)
        st = cgtp_route_order(m->router, n, static_cast<const int32_t *>(e), static_cast<int32_t *>(address(rows)),
                              static_cast<int32_t *>(address(slots)), static_cast<int32_t *>(address(offsets)), address(ws),
                              bytes, in.stream());
    return answer(st, {&rows, &slots, &offsets});
    END_HANDLE_TH_ERRORS
}

// (handle, d_in, d_out, experts, top_k, weight_numel, dtype)
PyObject *linear(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (!takes(n, 7)) return nullptr;
    const long dtype = PyLong_AsLong(a[6]);
    return capsule(new LinearMeta{static_cast<const cgtp_linear *>(PyLong_AsVoidPtr(a[0])), PyLong_AsLongLong(a[1]),
                                  PyLong_AsLongLong(a[2]), PyLong_AsLongLong(a[3]), PyLong_AsLongLong(a[4]),
                                  PyLong_AsLongLong(a[5]), elem_type(dtype), real_type(dtype)},
                   kLinear, [](PyObject *o) { delete static_cast<LinearMeta *>(PyCapsule_GetPointer(o, kLinear)); });
    END_HANDLE_TH_ERRORS
}

// a linear's choice of experts: experts, weights, and of the order rows, slots and offsets
struct Choice {
    const int32_t *experts = nullptr;
    const void *weights = nullptr;
    const int32_t *rows = nullptr, *slots = nullptr, *offsets = nullptr;
};

// from the two tensors and the order (None or a tuple of three), `fine` cleared where they are not as they have to be
Choice choice(Args &in, const LinearMeta *m, int64_t n, PyObject *experts, PyObject *weights, PyObject *order)
{
    Choice c;
    if (m->top_k == 0) {
        in.fine = in.fine && experts == Py_None && weights == Py_None && order == Py_None;
        return c;
    }
    c.experts = static_cast<const int32_t *>(in.at(experts, at::kInt, {n, m->top_k}));
    c.weights = in.at(weights, m->real, {n, m->top_k});
    if (order == Py_None) return c;
    if (!PyTuple_Check(order) || PyTuple_GET_SIZE(order) != 3) {
        in.fine = false;
        return c;
    }
    c.rows = static_cast<const int32_t *>(in.at(PyTuple_GET_ITEM(order, 0), at::kInt, {n}, true));
    c.slots = static_cast<const int32_t *>(in.at(PyTuple_GET_ITEM(order, 1), at::kInt, {n * m->top_k}, true));
    c.offsets = static_cast<const int32_t *>(in.at(PyTuple_GET_ITEM(order, 2), at::kInt, {m->experts + 1}, true));
    return c;
}

// (linear, x, w, experts, weights, order) -> (out,)
PyObject *linear_forward(PyObject *, PyObject *const *a, Py_ssize_t n_args)
{
    HANDLE_TH_ERRORS
    if (!takes(n_args, 6)) return nullptr;
    if (a[0] == Py_None) Py_RETURN_NONE;  // closed
    const auto *m = static_cast<const LinearMeta *>(PyCapsule_GetPointer(a[0], kLinear));
    if (!m) return nullptr;
    const at::Tensor *x = tensor(a[1]);
    Args in(x);
    if (!in.fine || x->dim() != 2) Py_RETURN_NONE;
    const int64_t n = x->size(0);
    int64_t ld;
    const void *xp = in.rows(a[1], m->rows, n, m->d_in, &ld), *w = in.at(a[2], m->rows, {m->experts, m->numel});
    const Choice c = choice(in, m, n, a[3], a[4], a[5]);
    if (!in.fine) Py_RETURN_NONE;
    at::Tensor out = at::empty({n, m->d_out}, x->options());
    return answer(cgtp_linear_forward(m->linear, n, xp, ld, w, c.experts, c.weights, c.rows, address(out), m->d_out, in.stream()),
                  {&out});
    END_HANDLE_TH_ERRORS
}

// (linear, x, w, grad_out, experts, weights, order, need of the three) -> (grad_x, grad_w, grad_weights)
PyObject *linear_backward(PyObject *, PyObject *const *a, Py_ssize_t n_args)
{
    HANDLE_TH_ERRORS
    if (!takes(n_args, 10)) return nullptr;
    if (a[0] == Py_None) Py_RETURN_NONE;  // closed
    const auto *m = static_cast<const LinearMeta *>(PyCapsule_GetPointer(a[0], kLinear));
    if (!m) return nullptr;
    const at::Tensor *x = tensor(a[1]);
    Args in(x);
    if (!in.fine || x->dim() != 2) Py_RETURN_NONE;
    const int64_t n = x->size(0);
    int64_t ld, g_ld;
    const void *xp = in.rows(a[1], m->rows, n, m->d_in, &ld), *w = in.at(a[2], m->rows, {m->experts, m->numel}),
               *g = in.rows(a[3], m->rows, n, m->d_out, &g_ld);
    const Choice c = choice(in, m, n, a[4], a[5], a[6]);
    const bool need_w = PyObject_IsTrue(a[8]) == 1;
    if (!in.fine || (need_w && m->top_k && (!a[6] || a[6] == Py_None))) Py_RETURN_NONE;
    at::Tensor gx, gw, gp, ws;
    if (PyObject_IsTrue(a[7]) == 1) gx = at::empty({n, m->d_in}, x->options());
    if (need_w) gw = at::empty({m->experts, m->numel}, x->options());
    if (PyObject_IsTrue(a[9]) == 1 && m->top_k) gp = at::empty({n, m->top_k}, x->options().dtype(m->real));
    size_t bytes = 0;
    cgtp_status st = cgtp_linear_workspace_size(m->linear, n, &bytes);
    if (st == CGTP_OK && bytes) ws = at::empty({(int64_t)bytes}, x->options().dtype(at::kByte));
    if (st == CGTP_OK)
        st = cgtp_linear_backward(m->linear, n, xp, ld, w, c.experts, c.weights, c.rows, c.slots, c.offsets, g, g_ld,
                                  address(gx), m->d_in, address(gw), address(gp), address(ws), bytes, in.stream());
    return answer(st, {&gx, &gw, &gp});
    END_HANDLE_TH_ERRORS
}

// ------------------------------------------------------------------------------------------ optimizer

// (handle, sizes, elements, blocks, norm_workspace, state_bits, dtype)
PyObject *adamw(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (!takes(n, 7)) return nullptr;
    if (!PyTuple_Check(a[1])) return PyErr_Format(PyExc_TypeError, "sizes must be a tuple");
    auto m = std::make_unique<AdamWMeta>();
    m->opt = static_cast<const cgtp_adamw *>(PyLong_AsVoidPtr(a[0]));
    for (Py_ssize_t i = 0; i < PyTuple_GET_SIZE(a[1]); ++i) m->sizes.push_back(PyLong_AsLongLong(PyTuple_GET_ITEM(a[1], i)));
    m->elements = PyLong_AsLongLong(a[2]);
    m->blocks = PyLong_AsLongLong(a[3]);
    m->norm_workspace = PyLong_AsLongLong(a[4]);
    m->codes = PyLong_AsLong(a[5]) == 8;
    const long dtype = PyLong_AsLong(a[6]);
    m->elem = elem_type(dtype);
    m->real = dtype == CGTP_F64 ? at::kDouble : at::kFloat;
    if (PyErr_Occurred()) return nullptr;
    return PyCapsule_New(m.release(), kAdamW,
                         [](PyObject *o) { delete static_cast<AdamWMeta *>(PyCapsule_GetPointer(o, kAdamW)); });
    END_HANDLE_TH_ERRORS
}

const AdamWMeta *adamw_of(PyObject *o) { return static_cast<const AdamWMeta *>(PyCapsule_GetPointer(o, kAdamW)); }

const at::Tensor *first_of(PyObject *tuple)
{
    if (!PyTuple_Check(tuple)) return nullptr;
    for (Py_ssize_t i = 0; i < PyTuple_GET_SIZE(tuple); ++i)
        if (PyTuple_GET_ITEM(tuple, i) != Py_None) return tensor(PyTuple_GET_ITEM(tuple, i));
    return nullptr;
}

// addresses of the layout's tensors, null for None where that may be
bool addresses(const AdamWMeta *m, const Args &in, PyObject *tuple, bool optional, std::vector<void *> *out)
{
    const size_t n = m->sizes.size();
    if (!PyTuple_Check(tuple) || (size_t)PyTuple_GET_SIZE(tuple) != n) return false;
    out->resize(n);
    for (size_t i = 0; i < n; ++i) {
        PyObject *o = PyTuple_GET_ITEM(tuple, (Py_ssize_t)i);
        if (o == Py_None && optional) {
            (*out)[i] = nullptr;
            continue;
        }
        const at::Tensor *x = tensor(o);
        if (!in.here(x, m->elem) || x->numel() != m->sizes[i] || !x->is_contiguous()) return false;
        (*out)[i] = x->data_ptr();
    }
    return true;
}

// (layout, tensors, None among them allowed) -> whether the layout's calls take them
PyObject *takes_tensors(PyObject *, PyObject *const *a, Py_ssize_t n_args)
{
    HANDLE_TH_ERRORS
    if (!takes(n_args, 2)) return nullptr;
    if (a[0] == Py_None) Py_RETURN_NONE;  // closed
    const AdamWMeta *m = adamw_of(a[0]);
    if (!m) return nullptr;
    Args in(first_of(a[1]));
    std::vector<void *> at;
    return PyBool_FromLong(in.fine && addresses(m, in, a[1], true, &at));
    END_HANDLE_TH_ERRORS
}

// (layout, gradients) -> (norm,)
PyObject *grad_norm(PyObject *, PyObject *const *a, Py_ssize_t n_args)
{
    HANDLE_TH_ERRORS
    if (!takes(n_args, 2)) return nullptr;
    if (a[0] == Py_None) Py_RETURN_NONE;  // closed
    const AdamWMeta *m = adamw_of(a[0]);
    if (!m) return nullptr;
    const at::Tensor *first = first_of(a[1]);
    Args in(first);
    std::vector<void *> grads;
    if (!in.fine || !addresses(m, in, a[1], true, &grads)) Py_RETURN_NONE;
    at::Tensor norm = at::empty({1}, first->options().dtype(at::kDouble));
    at::Tensor ws = at::empty({m->norm_workspace}, first->options().dtype(at::kByte));
    return answer(cgtp_grad_norm(m->opt, grads.data(), static_cast<double *>(norm.data_ptr()), address(ws),
                                 (size_t)m->norm_workspace, in.stream()),
                  {&norm});
    END_HANDLE_TH_ERRORS
}

// (layout, parameters, gradients, m, v, scales, master, norm, schedule, step, lr, beta1, beta2, eps,
// weight_decay, max_norm, grad_scale) -> ()
PyObject *adamw_step(PyObject *, PyObject *const *a, Py_ssize_t n_args)
{
    HANDLE_TH_ERRORS
    if (!takes(n_args, 17)) return nullptr;
    if (a[0] == Py_None) Py_RETURN_NONE;  // closed
    const AdamWMeta *m = adamw_of(a[0]);
    if (!m) return nullptr;
    Args in(first_of(a[1]));
    std::vector<void *> params, grads;
    if (!in.fine || !addresses(m, in, a[1], false, &params) || !addresses(m, in, a[2], true, &grads)) Py_RETURN_NONE;
    void *mp = in.at(a[3], m->codes ? at::kChar : m->real, {m->elements}),
         *vp = in.at(a[4], m->codes ? at::kByte : m->real, {m->elements}),
         *sc = in.at(a[5], at::kFloat, {2, m->blocks}, true), *ma = in.at(a[6], at::kFloat, {m->elements}, true),
         *norm = in.at(a[7], at::kDouble, {1}, true), *sch = in.at(a[8], at::kDouble, {4}, true);
    if (!in.fine) Py_RETURN_NONE;
    cgtp_adamw_hyper hy;
    hy.step = PyLong_AsLongLong(a[9]);
    double *scalars[] = {&hy.lr, &hy.beta1, &hy.beta2, &hy.eps, &hy.weight_decay, &hy.max_norm, &hy.grad_scale};
    for (int i = 0; i < 7; ++i) *scalars[i] = PyFloat_AsDouble(a[10 + i]);
    if (PyErr_Occurred()) return nullptr;
    return answer(cgtp_adamw_step(m->opt, params.data(), grads.data(), mp, vp, static_cast<float *>(sc),
                                  static_cast<float *>(ma), &hy, static_cast<const double *>(norm),
                                  static_cast<const double *>(sch), in.stream()),
                  {});
    END_HANDLE_TH_ERRORS
}

// (layout, m, v, scales) -> (m, v) in float
PyObject *adamw_state_read(PyObject *, PyObject *const *a, Py_ssize_t n_args)
{
    HANDLE_TH_ERRORS
    if (!takes(n_args, 4)) return nullptr;
    if (a[0] == Py_None) Py_RETURN_NONE;  // closed
    const AdamWMeta *m = adamw_of(a[0]);
    if (!m) return nullptr;
    const at::Tensor *first = tensor(a[1]);
    Args in(first);
    if (!in.fine || !m->codes) Py_RETURN_NONE;
    const void *mp = in.at(a[1], at::kChar, {m->elements}), *vp = in.at(a[2], at::kByte, {m->elements});
    const void *sc = in.at(a[3], at::kFloat, {2, m->blocks});
    if (!in.fine) Py_RETURN_NONE;
    at::Tensor mo = at::empty({m->elements}, first->options().dtype(at::kFloat)), vo = at::empty_like(mo);
    return answer(cgtp_adamw_state_read(m->opt, mp, vp, static_cast<const float *>(sc), static_cast<float *>(address(mo)),
                                        static_cast<float *>(address(vo)), in.stream()),
                  {&mo, &vo});
    END_HANDLE_TH_ERRORS
}

#define CGTP_CALL(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, nullptr}
PyMethodDef kMethods[] = {CGTP_CALL(block),        CGTP_CALL(norm_forward),  CGTP_CALL(norm_backward),
                          CGTP_CALL(join_forward), CGTP_CALL(join_backward), CGTP_CALL(adamw),
                          CGTP_CALL(grad_norm),    CGTP_CALL(adamw_step),    CGTP_CALL(takes_tensors),
                          CGTP_CALL(adamw_state_read), CGTP_CALL(group_norm),
                          CGTP_CALL(group_norm_forward), CGTP_CALL(group_norm_backward), CGTP_CALL(router),
                          CGTP_CALL(route_forward), CGTP_CALL(route_backward), CGTP_CALL(route_order), CGTP_CALL(linear),
                          CGTP_CALL(linear_forward), CGTP_CALL(linear_backward),
                          {nullptr, nullptr, 0, nullptr}};
#undef CGTP_CALL

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls(void) { return PyModule_Create(&kModule); }
