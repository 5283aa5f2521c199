// Block plans: row layout, launch geometry, the generated source's constants, and the entry points
// cgtp_block_*, cgtp_norm_* and cgtp_join_* (documented in include/cgtp.h).
#include "block.h"

#include <algorithm>
#include <climits>
#include <cmath>
#include <memory>

#include "abi_util.h"
#include "block_kernels.h"

struct cgtp_block {
    cgtp::Block b;
};

namespace cgtp {

namespace {

constexpr int kLds = 160 * 1024;  // bytes of a workgroup

const char *type_name(int dtype)
{
    switch (dtype) {
    case CGTP_F64: return "double";
    case CGTP_BF16: return "__bf16";
    case CGTP_F16: return "_Float16";
    default: return "float";
    }
}

// The lanes' share of a row: G lanes, CV neighbouring channels (columns in a flat layout) to a slot.
// Of every pair, the cost of a row in lane operations is taken: its lanes times a lane's elements,
// which idle lanes and channels past an irrep's end raise, more where loads are narrow (below 16 bytes
// in a flat layout, below 8 in runs of channels, which are neighbours in the same cache lines), where a
// lane holds over 48 bytes of the row as it is stored (fewer waves fit a SIMD; 16-bit elements take twice
// that in registers, which the rule does not count: a flat 16-bit row of 576 gets 24 elements a lane, and the
// join's backward then 248 registers), and where waves must meet at barriers; the most
// lanes of equal cost.  One rule serves all four passes; its weights are fitted to times of 14 shapes at 2 to 9
// pairs each.  The
// join's backward, fp32: 20,000 rows of 128x(0e,1o,2e,3o), 64 lanes of 32 elements 210 us, 128 of 16 201
// us, 512 of 16, half idle, 216 us; 5,000 rows of 32x(0e,1o,2e), 32 lanes of 9 13.3 us, 16 of 18 15.9 us.
// The norm: backward, 200,000 flat rows of 576 in fp32, 32 lanes of 20 elements 356 us, 64 of 12, a
// quarter idle, 340 us; 200,000 rows of 65 in fp16, 4 lanes of 9 loads of 4 bytes 25.7 us, of 3 loads of 16
// 12.3 us.
void pick_lanes(Block &b)
{
    double best = 0;
    const int64_t most = 128;  // elements of a lane
    b.lanes = 0;
    for (int cv = 1; cv <= b.vec; cv *= 2)
        for (int g = 1; g <= 1024; g *= 2) {
            int64_t elems = 0, bytes = 0;
            for (const Block::Segment &s : b.slots_over()) {
                const int64_t slots = ((s.mul + cv - 1) / cv + g - 1) / g;
                const int run = cv * s.k;
                elems += slots * run;
                bytes += slots * (run / b.vec) * 16;  // by loads, none below 8 bytes
                for (int piece = b.vec / 2; piece >= 1; piece /= 2)
                    if (run & piece) bytes += slots * std::max(b.flat ? 16 : 8, piece * b.elem);
            }
            if (elems > most) continue;
            const double held = (double)elems * b.elem;
            double cost = (double)g * elems / b.d;
            cost *= 1 + 0.01 * std::max(0.0, held - 48);
            cost *= 1 + (b.flat ? 0.3 : 0.1) * ((double)bytes / (elems * b.elem) - 1);
            if (g > 64) cost *= 1 + 0.04 * std::log2(g / 64);
            if (b.lanes == 0 || cost <= best) {
                best = cost;
                b.lanes = g;
                b.cv = cv;
                b.elems = (int)elems;
            }
        }
    if (b.lanes == 0)
        throw Error(CGTP_ERR_UNSUPPORTED, "block: a lane would hold more than 128 elements of a row (too many columns, "
                                          "or too many changes of degree)");
    b.block = b.lanes > 64 ? b.lanes : 256;
    const long sums = b.lanes > 64 ? 1 : b.block / 64;
    const long bytes = 2L * std::max(1, b.lanes / 64) * b.real + (sums > 1 || b.flat ? sums * (b.flat ? b.d : b.c) * b.real : 0);
    if (bytes > kLds)
        throw Error(CGTP_ERR_UNSUPPORTED, "block: the sums over a row's channels need " + std::to_string(bytes) +
                                              " bytes of LDS, a workgroup has 163840");
}

std::string constants(const Block &b)
{
    std::string s = "// row norm and block join: " + std::to_string(b.d) + " columns, " + std::to_string(b.c) +
                    " channels\n";
    auto line = [&](const std::string &t) { s += t + "\n"; };
    line(std::string("typedef ") + type_name(b.cfg.dtype) + " T;");
    line(std::string("typedef ") + (b.cfg.dtype == CGTP_F64 ? "double" : "float") + " R;");
    auto num = [&](const char *n, long v) { line(std::string("constexpr int ") + n + " = " + std::to_string(v) + ";"); };
    num("D", b.d);
    num("C", b.c);
    num("VEC", b.vec);
    num("G", b.lanes);
    num("CV", b.cv);
    num("BLOCK", b.block);
    num("GATE", b.cfg.gate);
    num("ACT", b.cfg.act);
    num("POST", b.cfg.post_norm ? 1 : 0);
    num("NEXT", b.cfg.next_norm ? 1 : 0);
    std::string col, ch, k, mul, unit, at, of;
    int slots = 0, elems = 0;
    auto add = [](std::string &t, int v) { t += (t.empty() ? "" : ", ") + std::to_string(v); };
    for (const Block::Segment &g : b.slots_over())
        for (int u = 0; u * b.cv < g.mul; u += b.lanes, ++slots) {
            add(col, g.col);
            add(ch, g.ch);
            add(k, g.k);
            add(mul, g.mul);
            add(unit, u);
            add(at, elems);
            for (int i = 0; i < b.cv * g.k; ++i) add(of, slots * b.cv + i / g.k);
            elems += b.cv * g.k;
        }
    num("NSLOT", slots);
    num("EPL", elems);
    auto list = [&](const char *n, const char *len, const std::string &v) {
        line(std::string("constexpr int ") + n + "[" + len + "] = {" + v + "};");
    };
    list("S_COL", "NSLOT", col);
    list("S_CH", "NSLOT", ch);
    list("S_K", "NSLOT", k);
    list("S_MUL", "NSLOT", mul);
    list("S_UNIT", "NSLOT", unit);
    list("S_AT", "NSLOT", at);
    list("E_C", "EPL", of);
    line(std::string("constexpr bool FLAT = ") + (b.flat ? "true;" : "false;"));
    num("NSEG", (long)b.segs.size());
    std::string gcol, gch, gk;
    for (const Block::Segment &g : b.segs) {
        add(gcol, g.col);
        add(gch, g.ch);
        add(gk, g.k);
    }
    list("G_COL", "NSEG", gcol);
    list("G_CH", "NSEG", gch);
    list("G_K", "NSEG", gk);
    return s;
}

}  // namespace

void build_block(Block &b, const std::string &irreps)
{
    int64_t col = 0, ch = 0;
    for (const Irrep &ir : parse_irreps(irreps, "block")) {
        const int k = 2 * ir.l + 1;
        if (b.segs.empty() || b.segs.back().k != k) b.segs.push_back({(int)col, (int)ch, k, 0});
        b.segs.back().mul += ir.mul;
        col += (int64_t)ir.mul * k;
        ch += ir.mul;
        if (col > (1 << 20)) throw Error(CGTP_ERR_UNSUPPORTED, "block: a row of more than 1048576 columns");
    }
    if (b.segs.size() > 128)
        throw Error(CGTP_ERR_UNSUPPORTED, "block: more than 128 runs of equal degrees along a row");
    b.d = (int)col;
    b.c = (int)ch;
    b.elem = b.cfg.dtype == CGTP_F64 ? 8 : b.cfg.dtype == CGTP_F32 ? 4 : 2;
    b.real = b.cfg.dtype == CGTP_F64 ? 8 : 4;
    b.vec = 16 / b.elem;
    b.flat = b.d != b.c && b.cfg.gate != CGTP_GATE_CHANNEL;
    pick_lanes(b);
    b.source = constants(b) + kBlockKernels;
    b.code = compile_source(b.source);
}

const Block::Fns &block_for_current_device(Block &b)
{
    int dev = 0;
    check_hip(hipGetDevice(&dev), "hipGetDevice");
    std::lock_guard<std::mutex> lock(b.mu);
    auto it = b.loaded.find(dev);
    if (it != b.loaded.end()) return it->second;
    Block::Fns F;
    check_hip(hipModuleLoadData(&F.module, b.code.data()), "hipModuleLoadData");
    check_hip(hipModuleGetFunction(&F.norm_fwd, F.module, "cgtp_norm_fwd"), "hipModuleGetFunction(norm_fwd)");
    check_hip(hipModuleGetFunction(&F.norm_bwd, F.module, "cgtp_norm_bwd"), "hipModuleGetFunction(norm_bwd)");
    check_hip(hipModuleGetFunction(&F.join_fwd, F.module, "cgtp_join_fwd"), "hipModuleGetFunction(join_fwd)");
    check_hip(hipModuleGetFunction(&F.join_bwd, F.module, "cgtp_join_bwd"), "hipModuleGetFunction(join_bwd)");
    check_hip(hipModuleGetFunction(&F.reduce, F.module, "cgtp_block_reduce"), "hipModuleGetFunction(block_reduce)");
    return b.loaded.emplace(dev, F).first->second;
}

void unload_block(Block &b)
{
    if (b.loaded.empty()) return;
    int prev = 0;
    const bool have_prev = hipGetDevice(&prev) == hipSuccess;
    for (auto &kv : b.loaded)
        if (kv.second.module && hipSetDevice(kv.first) == hipSuccess) (void)hipModuleUnload(kv.second.module);
    b.loaded.clear();
    if (have_prev) (void)hipSetDevice(prev);
}

// At most 2,048 waves, two for each of the 1,024 SIMDs, which then take rows in turn: the weights are read and
// the partial sums written once by each (the join's backward, 200,000 rows of 64x(0e,1o,2e) bf16: 345, 289,
// 304, 313 us at 1, 2, 4, 8 waves to a SIMD; the norm's, 8,192 rows of 4,096 bf16: 54, 43, 45, 53 us).
// A workgroup stays on one CU: where 1,024 lanes share a row these are 128 workgroups, on half of the 256 CUs
// (8,192 rows of 8,192 fp32, the norm's backward 185 us, 4.3 TB/s, where 576 columns reach 5.5).
int64_t block_groups(const Block &b, int64_t N, int waves_per_simd)
{
    const int64_t need = (N + b.rows_per_group() - 1) / b.rows_per_group();
    return std::max<int64_t>(1, std::min<int64_t>(need, 1024 * waves_per_simd / (b.block / 64)));
}

// A forward pass has no partial sums: rows that twice as many waves take at once are taken at once
// (the join, 5,000 rows of 32x(0e,1o,2e) fp32: 7.6 us in turns, 7.25).
int64_t forward_groups(const Block &b, int64_t N, int waves_per_simd)
{
    const int64_t at_once = block_groups(b, N, 2 * waves_per_simd), in_turns = block_groups(b, N, waves_per_simd);
    return at_once * b.rows_per_group() >= N ? at_once : in_turns;
}

// The norm's forward has one row to wait for at a time and no partial sums: four waves where a barrier
// makes several wait together, or where 16-bit elements take more arithmetic by the byte (20,000 rows
// of 2,048 fp64 113 us against 120 with two, 200,000 of 576 bf16 87 against 108; but fp32 176 against 161).
int norm_waves(const Block &b) { return b.lanes > 64 || b.elem == 2 ? 4 : 2; }

namespace {

// Rows of `width` elements every `ld` elements.
struct Rows {
    const void *p;
    int64_t width, ld;
    const char *name;
};

void check_rows(const Block &b, int64_t N, const Rows &r)
{
    require_ptr(r.p, r.name, b.elem);
    require(r.ld >= r.width && r.ld < INT_MAX,
            std::string(r.name) + ": row pitch " + std::to_string(r.ld) + " is below the row's " +
                std::to_string(r.width) + " elements or above 2^31-1");
    require(N <= ((int64_t)1 << 56) / (r.ld * b.elem), std::string(r.name) + ": more than 2^56 bytes");
}

// No row of one may overlap a row of the other: their ranges are apart, or both have the same
// pitch and lie side by side inside it (a block's output and its gates in one buffer).
void rows_apart(const Block &b, int64_t N, const Rows &x, const Rows &y)
{
    if (!x.p || !y.p || !N || !x.width || !y.width) return;
    const int64_t es = b.elem;
    const uint64_t a = reinterpret_cast<uintptr_t>(x.p), c = reinterpret_cast<uintptr_t>(y.p);
    const uint64_t na = (uint64_t)((N - 1) * x.ld + x.width) * es, nc = (uint64_t)((N - 1) * y.ld + y.width) * es;
    if (a + na <= c || c + nc <= a) return;
    if (x.ld == y.ld) {
        const int64_t pitch = x.ld * es;
        int64_t m = (int64_t)(c - a) % pitch;
        if (m < 0) m += pitch;
        if (m >= x.width * es && m + y.width * es <= pitch) return;
    }
    throw Error(CGTP_ERR_INVALID_ARG, std::string(x.name) + " overlaps " + y.name);
}

void rows_apart(const Block &b, int64_t N, const Rows &x, const void *p, size_t bytes, const char *name)
{
    if (!x.p || !p || !N) return;
    require_disjoint(x.p, (size_t)((N - 1) * x.ld + x.width) * b.elem, x.name, p, bytes, name);
}

void check_count(int64_t N)
{
    require(N >= 0 && N < INT_MAX, "N must be in [0, 2^31-1)");
}

void run(hipFunction_t f, int64_t groups, int threads, void **args, void *stream)
{
    check_hip(hipModuleLaunchKernel(f, (unsigned)groups, 1, 1, (unsigned)threads, 1, 1, 0,
                                    static_cast<hipStream_t>(stream), args, nullptr),
              "hipModuleLaunchKernel");
}

void reduce_partials(const Block &b, const Block::Fns &F, const void *part, int64_t parts, bool join, const void *w_post,
                     const void *scale, void *g_post, void *g_scale, void *g_next, void *stream)
{
    long rows = (long)parts;
    int is_join = join ? 1 : 0;
    int width = b.c * (join && b.cfg.next_norm ? 2 : 1);
    void *args[] = {&part, &rows, &width, &is_join, &w_post, &scale, &g_post, &g_scale, &g_next};
    run(F.reduce, (width + 15) / 16, 1024, args, stream);
}

size_t workspace_bytes_of(const Block &b, int64_t N)
{
    return N == 0 ? 0 : (size_t)block_groups(b, N) * b.c * (b.cfg.next_norm ? 2 : 1) * b.real;
}

// scalars passed to a kernel as its statistics' type
struct Real {
    float f;
    double d;
    bool wide;
    Real(const Block &b, double v) : f((float)v), d(v), wide(b.real == 8) {}
    void *arg() { return wide ? (void *)&d : (void *)&f; }
};

}  // namespace

}  // namespace cgtp

using namespace cgtp;

extern "C" {

cgtp_status cgtp_block_create(const char *irreps, const cgtp_block_config *config, cgtp_block **block_out)
{
    return guarded([&] {
        require(irreps && config && block_out, "NULL argument to cgtp_block_create");
        *block_out = nullptr;
        const cgtp_block_config &c = *config;
        require(c.dtype == CGTP_F32 || c.dtype == CGTP_F64 || c.dtype == CGTP_BF16 || c.dtype == CGTP_F16,
                "dtype must be CGTP_F32, CGTP_F64, CGTP_BF16 or CGTP_F16");
        require(c.gate >= CGTP_GATE_NONE && c.gate <= CGTP_GATE_CHANNEL, "gate must be a cgtp_gate");
        require(c.act >= CGTP_ACT_IDENTITY && c.act <= CGTP_ACT_TANH, "act must be a cgtp_act");
        require(std::isfinite(c.eps) && c.eps > 0 && (c.dtype == CGTP_F64 || (float)c.eps >= 1e-30f),
                "eps must be finite and positive (at least 1e-30 where statistics are float)");
        require(std::isfinite(c.alpha), "alpha must be finite");
        auto h = std::make_unique<cgtp_block>();
        h->b.cfg = c;
        build_block(h->b, irreps);
        *block_out = h.release();
    });
}

cgtp_status cgtp_block_destroy(cgtp_block *block)
{
    return guarded([&] {
        if (!block) return;
        unload_block(block->b);
        delete block;
    });
}

cgtp_status cgtp_block_info_get(const cgtp_block *block, cgtp_block_info *info)
{
    return guarded([&] {
        require(block && info, "NULL argument to cgtp_block_info_get");
        const Block &b = block->b;
        info->d = b.d;
        info->channels = b.c;
        info->gate_width = b.gate_width();
        info->dtype = b.cfg.dtype;
        info->lanes = b.lanes;
        info->elements = b.elems;
    });
}

const char *cgtp_block_source(const cgtp_block *block) { return block ? block->b.source.c_str() : nullptr; }

cgtp_status cgtp_block_workspace_size(const cgtp_block *block, int64_t N, size_t *bytes)
{
    return guarded([&] {
        require(block && bytes, "NULL argument to cgtp_block_workspace_size");
        check_count(N);
        *bytes = workspace_bytes_of(block->b, N);
    });
}

cgtp_status cgtp_norm_forward(const cgtp_block *block, int64_t N, const void *x, int64_t x_ld, const void *w, void *u,
                              void *rstd, void *stream)
{
    return guarded([&] {
        require(block != nullptr, "block is NULL");
        Block &b = const_cast<cgtp_block *>(block)->b;
        check_count(N);
        if (N == 0) return;
        const Rows X{x, b.d, x_ld, "x"}, U{u, b.d, b.d, "u"};
        check_rows(b, N, X);
        check_rows(b, N, U);
        if (w) require_ptr(w, "w", b.real);
        if (rstd) require_ptr(rstd, "rstd", b.real);
        const size_t nw = (size_t)b.c * b.real, ns = (size_t)N * b.real;
        rows_apart(b, N, U, X);
        rows_apart(b, N, U, w, nw, "w");
        rows_apart(b, N, U, rstd, ns, "rstd");
        rows_apart(b, N, X, rstd, ns, "rstd");
        require_disjoint(rstd, rstd ? ns : 0, "rstd", w, w ? nw : 0, "w");
        const auto &F = block_for_current_device(b);
        long ld = (long)x_ld, rows = (long)N;
        Real eps(b, b.cfg.eps);
        void *args[] = {&x, &ld, &w, &u, &rstd, &rows, eps.arg()};
        run(F.norm_fwd, forward_groups(b, N, norm_waves(b)), b.block, args, stream);
    });
}

cgtp_status cgtp_norm_backward(const cgtp_block *block, int64_t N, const void *x, int64_t x_ld, const void *w,
                               const void *rstd, const void *grad_u, const void *grad_add, void *grad_x, void *grad_w,
                               void *workspace, size_t workspace_bytes, void *stream)
{
    return guarded([&] {
        require(block != nullptr, "block is NULL");
        Block &b = const_cast<cgtp_block *>(block)->b;
        check_count(N);
        if (!grad_x && !grad_w) return;
        if (grad_w) require_ptr(grad_w, "grad_w", b.real);
        const size_t nw = (size_t)b.c * b.real, ns = (size_t)N * b.real;
        if (N == 0) {
            if (grad_w)
                reduce_partials(b, block_for_current_device(b), nullptr, 0, false, nullptr, nullptr, nullptr, nullptr,
                                grad_w, stream);
            return;
        }
        const Rows X{x, b.d, x_ld, "x"}, DU{grad_u, b.d, b.d, "grad_u"}, ADD{grad_add, b.d, b.d, "grad_add"},
            DX{grad_x, b.d, b.d, "grad_x"};
        check_rows(b, N, X);
        check_rows(b, N, DU);
        if (grad_add) check_rows(b, N, ADD);
        if (grad_x) check_rows(b, N, DX);
        if (w) require_ptr(w, "w", b.real);
        require_ptr(rstd, "rstd", b.real);
        size_t need = 0;
        if (grad_w) {
            need = (size_t)block_groups(b, N) * nw;
            require_ptr(workspace, "workspace", 256);
            require(workspace_bytes >= need, "workspace too small (see cgtp_block_workspace_size)");
        }
        struct { void *p; size_t n; const char *name; } outs[] = {
            {grad_x, grad_x ? (size_t)N * b.d * b.elem : 0, "grad_x"},
            {grad_w, grad_w ? nw : 0, "grad_w"},
            {need ? workspace : nullptr, need, "workspace"}};
        struct { const void *p; size_t n; const char *name; } ins[] = {
            {x, (size_t)((N - 1) * x_ld + b.d) * b.elem, "x"}, {grad_u, (size_t)N * b.d * b.elem, "grad_u"},
            {grad_add, grad_add ? (size_t)N * b.d * b.elem : 0, "grad_add"}, {w, w ? nw : 0, "w"}, {rstd, ns, "rstd"}};
        for (int i = 0; i < 3; ++i) {
            for (auto &in : ins) require_disjoint(outs[i].p, outs[i].n, outs[i].name, in.p, in.n, in.name);
            for (int j = i + 1; j < 3; ++j)
                require_disjoint(outs[i].p, outs[i].n, outs[i].name, outs[j].p, outs[j].n, outs[j].name);
        }
        const auto &F = block_for_current_device(b);
        long ld = (long)x_ld, rows = (long)N;
        void *part = grad_w ? workspace : nullptr;
        void *args[] = {&x, &ld, &w, &rstd, &grad_u, &grad_add, &grad_x, &part, &rows};
        const int64_t groups = block_groups(b, N);
        run(F.norm_bwd, groups, b.block, args, stream);
        if (grad_w)
            reduce_partials(b, F, part, groups, false, nullptr, nullptr, nullptr, nullptr, grad_w, stream);
    });
}

cgtp_status cgtp_join_forward(const cgtp_block *block, int64_t N, const void *res, const void *f, int64_t f_ld,
                              const void *gate, int64_t gate_ld, const void *w_post, const void *scale,
                              const void *w_next, void *h, void *u, void *rstd_f, void *rstd_h, void *stream)
{
    return guarded([&] {
        require(block != nullptr, "block is NULL");
        Block &b = const_cast<cgtp_block *>(block)->b;
        check_count(N);
        if (N == 0) return;
        const int gw = b.gate_width();
        const bool next = b.cfg.next_norm != 0, post = b.cfg.post_norm != 0;
        require(gw > 0 || !gate, "gate given to a block without one");
        require(next || (!u && !w_next && !rstd_h), "u, w_next or rstd_h given to a block without a next norm");
        require(post || (!w_post && !rstd_f), "w_post or rstd_f given to a block without a post norm");
        const Rows RES{res, b.d, b.d, "res"}, F_{f, b.d, f_ld, "f"}, GT{gate, gw, gate_ld, "gate"}, H{h, b.d, b.d, "h"},
            U{u, b.d, b.d, "u"};
        check_rows(b, N, RES);
        check_rows(b, N, F_);
        if (gw) check_rows(b, N, GT);
        check_rows(b, N, H);
        if (next) check_rows(b, N, U);
        struct { const void *p; size_t n; const char *name; bool out; } reals[] = {
            {w_post, (size_t)b.c * b.real, "w_post", false}, {scale, (size_t)b.c * b.real, "scale", false},
            {w_next, (size_t)b.c * b.real, "w_next", false}, {rstd_f, (size_t)N * b.real, "rstd_f", true},
            {rstd_h, (size_t)N * b.real, "rstd_h", true}};
        for (auto &r : reals) {
            if (r.p) require_ptr(r.p, r.name, b.real);
            rows_apart(b, N, H, r.p, r.n, r.name);
            if (next) rows_apart(b, N, U, r.p, r.n, r.name);
            if (!r.out) continue;
            for (const Rows *in : {&RES, &F_, &GT}) rows_apart(b, N, *in, r.p, r.n, r.name);
            for (auto &o : reals)
                if (&o != &r) require_disjoint(r.p, r.p ? r.n : 0, r.name, o.p, o.p ? o.n : 0, o.name);
        }
        for (const Rows *in : {&RES, &F_, &GT}) {
            rows_apart(b, N, H, *in);
            if (next) rows_apart(b, N, U, *in);
        }
        if (next) rows_apart(b, N, H, U);
        const auto &F = block_for_current_device(b);
        long fl = (long)f_ld, gl = (long)gate_ld, rows = (long)N;
        Real alpha(b, b.cfg.alpha), eps(b, b.cfg.eps);
        void *args[] = {&res, &f, &fl, &gate, &gl, &w_post, &scale, &w_next, &h, &u, &rstd_f, &rstd_h, &rows,
                        alpha.arg(), eps.arg()};
        run(F.join_fwd, forward_groups(b, N, 2), b.block, args, stream);
    });
}

cgtp_status cgtp_join_backward(const cgtp_block *block, int64_t N, const void *grad_h, const void *grad_u,
                               const void *h, const void *f, int64_t f_ld, const void *gate, int64_t gate_ld,
                               const void *w_post, const void *scale, const void *w_next, const void *rstd_f,
                               const void *rstd_h, void *grad_res, void *grad_f, int64_t grad_f_ld, void *grad_gate,
                               int64_t grad_gate_ld, void *grad_w_post, void *grad_scale, void *grad_w_next,
                               void *workspace, size_t workspace_bytes, void *stream)
{
    return guarded([&] {
        require(block != nullptr, "block is NULL");
        Block &b = const_cast<cgtp_block *>(block)->b;
        check_count(N);
        const int gw = b.gate_width();
        const bool next = b.cfg.next_norm != 0, post = b.cfg.post_norm != 0;
        require(gw > 0 || (!gate && !grad_gate), "gate or grad_gate given to a block without one");
        require(next || (!grad_u && !w_next && !rstd_h && !grad_w_next),
                "grad_u, w_next, rstd_h or grad_w_next given to a block without a next norm");
        require(post || (!w_post && !rstd_f && !grad_w_post),
                "w_post, rstd_f or grad_w_post given to a block without a post norm");
        const bool weights = grad_w_post || grad_scale || grad_w_next;
        if (!grad_res && !grad_f && !grad_gate && !weights) return;
        const size_t nw = (size_t)b.c * b.real, ns = (size_t)N * b.real;
        if (w_post) require_ptr(w_post, "w_post", b.real);
        if (scale) require_ptr(scale, "scale", b.real);
        if (w_next) require_ptr(w_next, "w_next", b.real);
        if (grad_w_post) require_ptr(grad_w_post, "grad_w_post", b.real);
        if (grad_scale) require_ptr(grad_scale, "grad_scale", b.real);
        if (grad_w_next) require_ptr(grad_w_next, "grad_w_next", b.real);
        if (N == 0) {
            if (weights)
                reduce_partials(b, block_for_current_device(b), nullptr, 0, true, nullptr, nullptr, grad_w_post,
                                grad_scale, grad_w_next, stream);
            return;
        }
        const Rows DH{grad_h, b.d, b.d, "grad_h"}, DU{grad_u, b.d, b.d, "grad_u"}, H{h, b.d, b.d, "h"},
            F_{f, b.d, f_ld, "f"}, GT{gate, gw, gate_ld, "gate"};
        const Rows DR{grad_res, b.d, b.d, "grad_res"}, DF{grad_f, b.d, grad_f_ld, "grad_f"},
            DG{grad_gate, gw, grad_gate_ld, "grad_gate"};
        require(grad_h || next, "grad_h is NULL");
        if (grad_h) check_rows(b, N, DH);
        if (next) {
            check_rows(b, N, DU);
            check_rows(b, N, H);
            require_ptr(rstd_h, "rstd_h", b.real);
        }
        check_rows(b, N, F_);
        if (gw) check_rows(b, N, GT);
        if (post) require_ptr(rstd_f, "rstd_f", b.real);
        for (const Rows *o : {&DR, &DF, &DG})
            if (o->p) check_rows(b, N, *o);
        size_t need = 0;
        if (weights) {
            need = workspace_bytes_of(b, N);
            require_ptr(workspace, "workspace", 256);
            require(workspace_bytes >= need, "workspace too small (see cgtp_block_workspace_size)");
        }
        const Rows NH = next ? H : Rows{nullptr, 0, 0, "h"};
        const Rows *row_in[] = {&DH, &DU, &NH, &F_, &GT}, *row_out[] = {&DR, &DF, &DG};
        struct { const void *p; size_t n; const char *name; bool out; } reals[] = {
            {w_post, nw, "w_post", false}, {scale, nw, "scale", false}, {w_next, nw, "w_next", false},
            {rstd_f, ns, "rstd_f", false}, {rstd_h, ns, "rstd_h", false}, {grad_w_post, nw, "grad_w_post", true},
            {grad_scale, nw, "grad_scale", true}, {grad_w_next, nw, "grad_w_next", true},
            {weights ? workspace : nullptr, need, "workspace", true}};
        for (int i = 0; i < 3; ++i) {
            for (const Rows *in : row_in) rows_apart(b, N, *row_out[i], *in);
            for (int j = i + 1; j < 3; ++j) rows_apart(b, N, *row_out[i], *row_out[j]);
            for (auto &r : reals) rows_apart(b, N, *row_out[i], r.p, r.n, r.name);
        }
        for (auto &r : reals) {
            if (!r.out || !r.p) continue;
            for (const Rows *in : row_in) rows_apart(b, N, *in, r.p, r.n, r.name);
            for (auto &o : reals)
                if (&o != &r) require_disjoint(r.p, r.n, r.name, o.p, o.p ? o.n : 0, o.name);
        }
        const auto &F = block_for_current_device(b);
        long fl = (long)f_ld, gl = (long)gate_ld, dfl = (long)grad_f_ld, dgl = (long)grad_gate_ld, rows = (long)N;
        void *part = weights ? workspace : nullptr;
        Real alpha(b, b.cfg.alpha);
        void *args[] = {&grad_h, &grad_u, &h, &f, &fl, &gate, &gl, &w_post, &scale, &w_next, &rstd_f, &rstd_h, &grad_res,
                        &grad_f, &dfl, &grad_gate, &dgl, &part, &rows, alpha.arg()};
        const int64_t groups = block_groups(b, N);
        run(F.join_bwd, groups, b.block, args, stream);
        if (weights)
            reduce_partials(b, F, part, groups, true, w_post, scale, grad_w_post, grad_scale, grad_w_next, stream);
    });
}

}  // extern "C"
