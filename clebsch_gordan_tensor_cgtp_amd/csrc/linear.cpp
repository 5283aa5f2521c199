// Plans of the experts' products: paths, units and tiles, the generated source's constants, and the entry
// points cgtp_linear_* (documented in include/cgtp.h).
#include <algorithm>
#include <memory>

#include "config_module.h"
#include "linear_kernels.h"
#include "route.h"
#include "row_kernels.h"
#include "rows.h"

namespace {

struct LinearPath {
    int in_col, mul_in, out_col, mul_out, k, in, out;  // first columns, channels, 2l+1, irreps
    int64_t w;                                         // first weight
};

struct Unit {
    int part, out, first, count, wave;  // output irrep, 16-blocks of channels
};

// an input irrep of a direction, as it lies in LDS
struct Segment {
    int part, col, len, lds, pad;
};

// one direction of the product
struct Direction {
    std::vector<int> col, mul, k, part, lds, p0, pn;  // output irreps
    std::vector<int> p_lds, p_mul;                    // paths, by output irrep
    std::vector<int64_t> p_w;
    std::vector<Segment> segments;
    std::vector<int> in_pitch, out_pitch;             // parts, in elements
    std::vector<Unit> units;
    int waves = 1, simd_waves = 2, lds_bytes = 0;
};

struct Tile {
    int path, v, u, bv, bu, wv, wu, nodes;
};

}  // namespace

struct cgtp_linear {
    cgtp_linear_config cfg{};
    int elem = 4, real = 4;
    int d_in = 0, d_out = 0;
    int64_t numel = 0;
    std::vector<LinearPath> paths;
    Direction fwd, bwd, fwd_few, bwd_few;  // and of few rows
    std::vector<Tile> tiles;
    cgtp::ConfigModule mod;
    enum { forward, backward_x, transpose, backward_w, reduce, forward_few, backward_x_few };
};

namespace cgtp {

namespace {

constexpr int kMaxPaths = 64, kMaxUnits = 128, kLds = 160 * 1024, kMaxStretch = 512;

void find_paths(cgtp_linear &l, const std::vector<Irrep> &ins, const std::vector<Irrep> &outs)
{
    int64_t d_in = 0, d_out = 0;
    std::vector<int> out_col;
    for (const Irrep &o : outs) {
        out_col.push_back((int)d_out);
        d_out += o.dim();
    }
    for (size_t i = 0; i < ins.size(); ++i) {
        for (size_t j = 0; j < outs.size(); ++j)
            if (ins[i].l == outs[j].l && ins[i].p == outs[j].p) {
                l.paths.push_back({(int)d_in, ins[i].mul, out_col[j], outs[j].mul, 2 * ins[i].l + 1, (int)i, (int)j, l.numel});
                l.numel += (int64_t)ins[i].mul * outs[j].mul;
            }
        d_in += ins[i].dim();
    }
    if (d_in > (1 << 20) || d_out > (1 << 20))
        throw Error(CGTP_ERR_UNSUPPORTED, "linear: a row of more than 1048576 columns");
    l.d_in = (int)d_in;
    l.d_out = (int)d_out;
    if (l.paths.empty()) throw Error(CGTP_ERR_IRREPS, "linear: no irrep of the input is one of the output");
    if (l.paths.size() > (size_t)kMaxPaths) throw Error(CGTP_ERR_UNSUPPORTED, "linear: more than 64 pairs of equal irreps");
    if (l.numel > (1 << 26)) throw Error(CGTP_ERR_UNSUPPORTED, "linear: more than 2^26 weights of an expert");
}

int round_up(int n, int to) { return (n + to - 1) / to * to; }

// an odd number of 16 bytes
int odd_pitch(int elements, int vec) { return (round_up(elements, vec) / vec | 1) * vec; }

// Irreps of one degree and parity belong to one part: no others read what they read.  Parts are filled up to
// 64 KB of LDS for their rows in and out, so that two workgroups or more share a CU; where one degree's alone take over
// 76 KB, results do not go through LDS.
void plan_direction(cgtp_linear &l, Direction &d, const std::vector<Irrep> &ins, const std::vector<Irrep> &outs, bool backward, bool few)
{
    const int vec = 16 / l.elem, step = l.elem == 2 ? 32 : 16;
    struct Class {
        int l, p, in, out, part;
    };
    std::vector<Class> classes;
    auto class_of = [&](const Irrep &ir) -> Class & {
        for (Class &c : classes)
            if (c.l == ir.l && c.p == ir.p) return c;
        classes.push_back({ir.l, ir.p, 0, 0, 0});
        return classes.back();
    };
    for (const Irrep &o : outs) class_of(o).out += round_up(round_up(o.mul, 16) * (2 * o.l + 1), vec);
    for (const Irrep &i : ins)
        for (Class &c : classes)
            if (c.l == i.l && c.p == i.p) c.in += round_up(i.mul, step) * (2 * i.l + 1);
    const int budget = 64 * 1024;
    int part = -1;
    for (Class &c : classes) {
        auto bytes = [&](int in, int out) { return 16 * l.elem * (odd_pitch(in, vec) + odd_pitch(out, vec)); };
        if (part < 0 || bytes(d.in_pitch[part] + c.in, d.out_pitch[part] + c.out) > budget) {
            d.in_pitch.push_back(0);
            d.out_pitch.push_back(0);
            ++part;
        }
        c.part = part;
        d.in_pitch[part] += c.in;
        d.out_pitch[part] += c.out;
        if (bytes(d.in_pitch[part], 0) > kLds - 8 * 1024)
            throw Error(CGTP_ERR_UNSUPPORTED, "linear: 16 rows of one degree and parity need " +
                                                  std::to_string(bytes(d.in_pitch[part], 0)) +
                                                  " bytes of LDS, a workgroup has 155648 for them");
    }
    const int parts = part + 1;
    std::vector<bool> direct;
    for (int p = 0; p < parts; ++p)
        direct.push_back(16 * l.elem * (odd_pitch(d.in_pitch[p], vec) + odd_pitch(d.out_pitch[p], vec)) > 76 * 1024);
    std::vector<int> in_at(parts, 0), out_at(parts, 0);
    std::vector<int> in_lds;
    int at = 0;
    for (const Irrep &i : ins) {
        const int len = i.dim(), pad = round_up(i.mul, step) * (2 * i.l + 1);
        in_lds.push_back(-1);
        for (const Class &c : classes)
            if (c.l == i.l && c.p == i.p) {
                d.segments.push_back({c.part, at, len, in_at[c.part], pad});
                in_lds.back() = in_at[c.part];
                in_at[c.part] += pad;
            }
        at += len;
    }
    at = 0;
    for (size_t o = 0; o < outs.size(); ++o) {
        const int k = 2 * outs[o].l + 1, mul = outs[o].mul, in = class_of(outs[o]).part;
        d.col.push_back(at);
        d.mul.push_back(mul);
        d.k.push_back(k);
        d.part.push_back(in);
        d.lds.push_back(out_at[in]);
        out_at[in] += round_up(round_up(mul, 16) * k, vec);
        d.p0.push_back((int)d.p_lds.size());
        for (const LinearPath &p : l.paths)
            if ((backward ? p.in : p.out) == (int)o) {
                d.p_lds.push_back(in_lds[backward ? p.out : p.in]);
                d.p_mul.push_back(backward ? p.mul_out : p.mul_in);
                d.p_w.push_back(p.w);
            }
        d.pn.push_back((int)d.p_lds.size() - d.p0.back());
        at += mul * k;
    }
    for (int p = 0; p < parts; ++p) {
        d.in_pitch[p] = odd_pitch(d.in_pitch[p], vec);
        d.out_pitch[p] = direct[p] ? 0 : odd_pitch(d.out_pitch[p], vec);
        d.lds_bytes = std::max(d.lds_bytes, 16 * l.elem * (d.in_pitch[p] + d.out_pitch[p]));
    }
    // Four waves; eight where results do not go through LDS, of which parts are wide (20,000 rows of 128x(0e,1o,2e,3o) in
    // fp32, forward: 300 us with four, 265 us).  For few rows, a workgroup or less to each CU, up to twelve: what
    // counts then is the way through one tile (21 rows of 64x(0e,1o,2e) in bf16: 10.1 us with four, 8.2 us; 200,000 of
    // them 181 us, with eight 225 us).
    d.waves = few ? 12 : std::count(direct.begin(), direct.end(), true) ? 8 : 4;
    if (d.waves == 8) d.simd_waves = 4;  // two such workgroups on a CU (the backward: 352 us with one, 303 us)
    int most_units = 1;
    for (int p = 0; p < parts; ++p) {
        // Units: a wave's even share of the part's 16-blocks times components, no more than 20 (10 in double), since
        // their sums are held twice (of the expert at hand, and of all): 160 registers of a lane.
        int64_t work = 0;
        for (size_t o = 0; o < outs.size(); ++o)
            if (d.part[o] == p) work += (int64_t)((d.mul[o] + 15) / 16) * d.k[o];
        const int most = (int)std::min<int64_t>(l.elem == 8 ? 10 : 20, (work + d.waves - 1) / d.waves);
        std::vector<Unit> units;
        for (size_t o = 0; o < outs.size(); ++o) {
            if (d.part[o] != p) continue;
            const int blocks = (d.mul[o] + 15) / 16, n = std::max(1, most / d.k[o]), pieces = (blocks + n - 1) / n;
            for (int i = 0; i < pieces; ++i) {
                const int first = (int)((int64_t)blocks * i / pieces), end = (int)((int64_t)blocks * (i + 1) / pieces);
                units.push_back({p, (int)o, first, end - first, 0});
            }
        }
        // the costliest first, each to the wave with the least to do
        std::stable_sort(units.begin(), units.end(), [&](const Unit &a, const Unit &b) { return a.count * d.k[a.out] > b.count * d.k[b.out]; });
        std::vector<int> load(d.waves, 0);
        for (Unit &u : units) {
            u.wave = (int)(std::min_element(load.begin(), load.end()) - load.begin());
            load[u.wave] += u.count * d.k[u.out];
        }
        most_units = std::max<int>(most_units, (int)units.size());
        d.units.insert(d.units.end(), units.begin(), units.end());
    }
    d.waves = std::min(d.waves, most_units);
    if (d.units.size() > (size_t)kMaxUnits) throw Error(CGTP_ERR_UNSUPPORTED, "linear: too many channels");
}

// Tiles of the gradients: four waves, two along each side where there are blocks for them, hold up to 4 x 4 16-blocks
// each (2 x 2 in double, and in 16 bits for many components, whose rows fill LDS); the nodes at hand take up to 32 KB of
// LDS, 64 KB of 16-bit rows, of which a matrix instruction takes 32.  Tiles of many components come first: they take longest.
void plan_tiles(cgtp_linear &l)
{
    for (size_t p = 0; p < l.paths.size(); ++p) {
        const LinearPath &q = l.paths[p];
        const int bv = (q.mul_out + 15) / 16, bu = (q.mul_in + 15) / 16;
        const int most = l.elem == 8 || (l.elem == 2 && q.k > 3) ? 2 : 4;
        int wv = std::min(2, bv), wu = std::min(2, bu);
        if (wv == 1) wu = std::min(4, bu);
        if (wu == 1) wv = std::min(4, bv);
        for (int v = 0; v < bv; v += most * wv)
            for (int u = 0; u < bu; u += most * wu) {
                Tile t{(int)p, 16 * v, 16 * u, std::min(bv - v, most * wv), std::min(bu - u, most * wu), wv, wu, 0};
                const int step = l.elem == 2 ? 32 : 4, row = 16 * (t.bv + t.bu) * q.k * l.elem;
                t.nodes = step * std::max(1, std::min(l.elem == 2 ? 2 : 8, (l.elem == 2 ? 65536 : 32768) / (row * step)));
                l.tiles.push_back(t);
            }
    }
    std::stable_sort(l.tiles.begin(), l.tiles.end(), [&](const Tile &a, const Tile &b) { return l.paths[a.path].k > l.paths[b.path].k; });
}

struct Text {
    std::string s;
    void num(const std::string &n, int64_t v, const char *in = "") { s += std::string(in) + "constexpr int " + n + " = " + std::to_string(v) + ";\n"; }
    template <class F> void list(const std::string &n, size_t len, F &&f, const char *in = "")
    {
        s += std::string(in) + "constexpr int " + n + "[" + std::to_string(std::max<size_t>(1, len)) + "] = {";
        for (size_t i = 0; i < len; ++i) s += (i ? ", " : "") + std::to_string(f(i));
        s += "};\n";
    }
};

void direction_text(Text &t, const char *name, const Direction &d, bool dot)
{
    const char *st = "    static ";
    t.s += std::string("struct ") + name + " {\n";
    t.num("DOT", dot ? 1 : 0, st);
    t.num("SIMD_WAVES", d.simd_waves, st);
    t.num("NPARTS", (int64_t)d.in_pitch.size(), st);
    t.num("LDS_BYTES", d.lds_bytes, st);
    t.list("IN_PITCH", d.in_pitch.size(), [&](size_t i) { return d.in_pitch[i]; }, st);
    t.list("OUT_PITCH", d.out_pitch.size(), [&](size_t i) { return d.out_pitch[i]; }, st);
    t.num("NS", (int64_t)d.segments.size(), st);
    t.list("S_PART", d.segments.size(), [&](size_t i) { return d.segments[i].part; }, st);
    t.list("S_COL", d.segments.size(), [&](size_t i) { return d.segments[i].col; }, st);
    t.list("S_LEN", d.segments.size(), [&](size_t i) { return d.segments[i].len; }, st);
    t.list("S_LDS", d.segments.size(), [&](size_t i) { return d.segments[i].lds; }, st);
    t.list("S_PAD", d.segments.size(), [&](size_t i) { return d.segments[i].pad; }, st);
    t.num("NOUT", (int64_t)d.col.size(), st);
    t.list("O_PART", d.part.size(), [&](size_t i) { return d.part[i]; }, st);
    t.list("O_COL", d.col.size(), [&](size_t i) { return d.col[i]; }, st);
    t.list("O_MUL", d.mul.size(), [&](size_t i) { return d.mul[i]; }, st);
    t.list("O_K", d.k.size(), [&](size_t i) { return d.k[i]; }, st);
    t.list("O_LDS", d.lds.size(), [&](size_t i) { return d.lds[i]; }, st);
    t.list("O_P0", d.p0.size(), [&](size_t i) { return d.p0[i]; }, st);
    t.list("O_PN", d.pn.size(), [&](size_t i) { return d.pn[i]; }, st);
    t.list("P_LDS", d.p_lds.size(), [&](size_t i) { return d.p_lds[i]; }, st);
    t.list("P_MUL", d.p_mul.size(), [&](size_t i) { return d.p_mul[i]; }, st);
    t.list("P_W", d.p_w.size(), [&](size_t i) { return d.p_w[i]; }, st);
    t.num("NU", (int64_t)d.units.size(), st);
    t.num("WAVES", d.waves, st);
    t.list("U_PART", d.units.size(), [&](size_t i) { return d.units[i].part; }, st);
    t.list("U_OUT", d.units.size(), [&](size_t i) { return d.units[i].out; }, st);
    t.list("U_N0", d.units.size(), [&](size_t i) { return d.units[i].first; }, st);
    t.list("U_NN", d.units.size(), [&](size_t i) { return d.units[i].count; }, st);
    t.list("U_WAVE", d.units.size(), [&](size_t i) { return d.units[i].wave; }, st);
    t.s += "};\n";
}

std::string constants(const cgtp_linear &l)
{
    Text t;
    t.s = "// experts' products: " + std::to_string(l.d_in) + " columns into " + std::to_string(l.d_out) + "\n";
    t.s += std::string("typedef ") + type_name(l.cfg.dtype) + " T;\n";
    t.s += std::string("typedef ") + (l.cfg.dtype == CGTP_F64 ? "double" : "float") + " R;\n";
    if (l.elem == 2)
        t.s += std::string("#define BITS16 ") + (l.cfg.dtype == CGTP_BF16 ? "1" : "2") + "\n";
    else
        t.s += std::string("#define MFMA(a, b, c) __builtin_amdgcn_mfma_") +
               (l.elem == 8 ? "f64_16x16x4f64" : "f32_16x16x4f32") + "(a, b, c, 0, 0, 0)\n";
    t.num("ACT", 0);
    t.num("E", l.cfg.experts);
    t.num("K", l.cfg.top_k);
    t.num("NUMEL", l.numel);
    direction_text(t, "Forward", l.fwd, false);
    direction_text(t, "Backward", l.bwd, l.cfg.top_k > 0);
    direction_text(t, "ForwardFew", l.fwd_few, false);
    direction_text(t, "BackwardFew", l.bwd_few, l.cfg.top_k > 0);
    t.num("NPATH", (int64_t)l.paths.size());
    t.list("W_XC", l.paths.size(), [&](size_t i) { return l.paths[i].in_col; });
    t.list("W_MI", l.paths.size(), [&](size_t i) { return l.paths[i].mul_in; });
    t.list("W_GC", l.paths.size(), [&](size_t i) { return l.paths[i].out_col; });
    t.list("W_MO", l.paths.size(), [&](size_t i) { return l.paths[i].mul_out; });
    t.list("W_K", l.paths.size(), [&](size_t i) { return l.paths[i].k; });
    t.list("W_OFF", l.paths.size(), [&](size_t i) { return l.paths[i].w; });
    t.num("NT", (int64_t)l.tiles.size());
    t.list("T_PATH", l.tiles.size(), [&](size_t i) { return l.tiles[i].path; });
    t.list("T_V", l.tiles.size(), [&](size_t i) { return l.tiles[i].v; });
    t.list("T_U", l.tiles.size(), [&](size_t i) { return l.tiles[i].u; });
    t.list("T_BV", l.tiles.size(), [&](size_t i) { return l.tiles[i].bv; });
    t.list("T_BU", l.tiles.size(), [&](size_t i) { return l.tiles[i].bu; });
    t.list("T_WV", l.tiles.size(), [&](size_t i) { return l.tiles[i].wv; });
    t.list("T_WU", l.tiles.size(), [&](size_t i) { return l.tiles[i].wu; });
    t.list("T_NODES", l.tiles.size(), [&](size_t i) { return l.tiles[i].nodes; });
    t.num("MAX_STRETCH", kMaxStretch);
    return t.s;
}

bool few_rows(int64_t N) { return N <= 16 * 256; }

int64_t slots_of(const cgtp_linear &l, int64_t N) { return N * std::max(1, l.cfg.top_k); }

// Slots of a stretch of the weight gradients: enough workgroups for some to each of the 256 CUs, but no shorter than
// 64 slots, each stretch writing a partial sum of every weight.
int64_t stretch_len(const cgtp_linear &l, int64_t N)
{
    const int64_t slots = slots_of(l, N), groups = std::max<int64_t>(1, 1024 / (int64_t)l.tiles.size());
    const int64_t len = std::max<int64_t>(64, (slots + groups - 1) / groups);
    return std::min<int64_t>(kMaxStretch, (len + 31) / 32 * 32);
}

int64_t stretches(const cgtp_linear &l, int64_t N)
{
    const int64_t len = stretch_len(l, N);
    return (slots_of(l, N) / len + l.cfg.experts + 7) / 8 * 8;  // a whole number to each of the 8 XCDs
}

size_t aligned(size_t n) { return (n + 255) / 256 * 256; }

size_t weight_bytes(const cgtp_linear &l) { return (size_t)l.cfg.experts * l.numel * l.elem; }

size_t backward_bytes(const cgtp_linear &l, int64_t N)
{
    return N == 0 ? 0 : aligned(weight_bytes(l)) + aligned((size_t)stretches(l, N) * l.numel * l.real);
}

void run2(hipFunction_t f, int64_t x, int64_t y, int threads, void **args, void *stream)
{
    check_hip(hipModuleLaunchKernel(f, (unsigned)x, (unsigned)y, 1, (unsigned)threads, 1, 1, 0,
                                    static_cast<hipStream_t>(stream), args, nullptr),
              "hipModuleLaunchKernel");
}

void check_linear(const cgtp_linear &l, int64_t N)
{
    check_count(N);
    require(N <= (int64_t)INT_MAX / std::max(1, l.cfg.top_k), "N * top_k must be below 2^31");
}

// what a product without a choice of experts does not take
void check_choice(const cgtp_linear &l, const void *experts, const void *weights, int64_t N)
{
    if (l.cfg.top_k == 0) {
        require(!experts && !weights, "experts or weights given to a linear without a choice of experts");
        return;
    }
    if (N == 0) return;
    require_ptr(experts, "experts", 4);
    require_ptr(weights, "weights", l.real);
}

}  // namespace

}  // namespace cgtp

using namespace cgtp;

extern "C" {

cgtp_status cgtp_linear_create(const char *in_irreps, const char *out_irreps, const cgtp_linear_config *config,
                               cgtp_linear **linear_out)
{
    return guarded([&] {
        require(in_irreps && out_irreps && config && linear_out, "NULL argument to cgtp_linear_create");
        *linear_out = nullptr;
        const cgtp_linear_config &c = *config;
        require(c.dtype == CGTP_F32 || c.dtype == CGTP_F64 || c.dtype == CGTP_BF16 || c.dtype == CGTP_F16,
                "dtype must be CGTP_F32, CGTP_F64, CGTP_BF16 or CGTP_F16");
        require(c.experts >= 1, "experts must be positive");
        require(c.top_k >= 0 && c.top_k <= c.experts, "top_k must be in [0, experts]");
        require(c.top_k > 0 || c.experts == 1, "a linear without a choice (top_k 0) has one expert");
        if (c.experts > kMaxExperts) throw Error(CGTP_ERR_UNSUPPORTED, "linear: more than 512 experts");
        if (c.top_k > 32) throw Error(CGTP_ERR_UNSUPPORTED, "linear: more than 32 experts of a row");
        auto h = std::make_unique<cgtp_linear>();
        h->cfg = c;
        h->elem = elem_bytes(c.dtype);
        h->real = real_bytes(c.dtype);
        const std::vector<Irrep> ins = parse_irreps(in_irreps, "input"), outs = parse_irreps(out_irreps, "output");
        find_paths(*h, ins, outs);
        plan_direction(*h, h->fwd, ins, outs, false, false);
        plan_direction(*h, h->bwd, outs, ins, true, false);
        plan_direction(*h, h->fwd_few, ins, outs, false, true);
        plan_direction(*h, h->bwd_few, outs, ins, true, true);
        plan_tiles(*h);
        h->mod.build(constants(*h) + kRowKernels + kLinearKernels,
                     {"cgtp_linear_fwd", "cgtp_linear_bwd_x", "cgtp_linear_transpose", "cgtp_linear_bwd_w",
                      "cgtp_linear_reduce", "cgtp_linear_fwd_few", "cgtp_linear_bwd_x_few"});
        *linear_out = h.release();
    });
}

cgtp_status cgtp_linear_destroy(cgtp_linear *linear)
{
    return guarded([&] {
        if (!linear) return;
        linear->mod.unload();
        delete linear;
    });
}

cgtp_status cgtp_linear_info_get(const cgtp_linear *linear, cgtp_linear_info *info)
{
    return guarded([&] {
        require(linear && info, "NULL argument to cgtp_linear_info_get");
        info->d_in = linear->d_in;
        info->d_out = linear->d_out;
        info->num_paths = (int32_t)linear->paths.size();
        info->dtype = linear->cfg.dtype;
        info->weight_numel = linear->numel;
    });
}

const char *cgtp_linear_source(const cgtp_linear *linear) { return linear ? linear->mod.source.c_str() : nullptr; }

cgtp_status cgtp_linear_forward(const cgtp_linear *linear, int64_t N, const void *x, int64_t x_ld, const void *w,
                                const int32_t *experts, const void *weights, const int32_t *rows, void *out,
                                int64_t out_ld, void *stream)
{
    return guarded([&] {
        require(linear != nullptr, "linear is NULL");
        auto &l = *const_cast<cgtp_linear *>(linear);
        check_linear(l, N);
        check_choice(l, experts, weights, N);
        if (N == 0) return;
        const Rows X{x, l.d_in, x_ld, "x"}, O{out, l.d_out, out_ld, "out"};
        check_rows(l.elem, N, X);
        check_rows(l.elem, N, O);
        require_ptr(w, "w", l.elem);
        if (rows) require_ptr(rows, "rows", 4);
        const size_t slots = (size_t)N * l.cfg.top_k;
        Arguments all(l.elem, N);
        all.rows(X, false);
        all.rows(O, true);
        all.flat(w, weight_bytes(l), "w", false);
        all.flat(experts, slots * 4, "experts", false);
        all.flat(weights, slots * l.real, "weights", false);
        all.flat(rows, (size_t)N * 4, "rows", false);
        all.check();
        const auto &F = l.mod.here();
        long xl = (long)x_ld, ol = (long)out_ld, n = (long)N;
        void *args[] = {&x, &xl, &w, &experts, &weights, &rows, &n, &out, &ol};
        const bool few = few_rows(N);
        run(F[few ? cgtp_linear::forward_few : cgtp_linear::forward], (N + 15) / 16, (few ? l.fwd_few : l.fwd).waves * 64, args,
            stream);
    });
}

cgtp_status cgtp_linear_workspace_size(const cgtp_linear *linear, int64_t N, size_t *bytes)
{
    return guarded([&] {
        require(linear && bytes, "NULL argument to cgtp_linear_workspace_size");
        check_linear(*linear, N);
        *bytes = backward_bytes(*linear, N);
    });
}

cgtp_status cgtp_linear_backward(const cgtp_linear *linear, int64_t N, const void *x, int64_t x_ld, const void *w,
                                 const int32_t *experts, const void *weights, const int32_t *rows, const int32_t *slots,
                                 const int32_t *offsets, const void *grad_out, int64_t grad_out_ld, void *grad_x,
                                 int64_t grad_x_ld, void *grad_w, void *grad_weights, void *workspace,
                                 size_t workspace_bytes, void *stream)
{
    return guarded([&] {
        require(linear != nullptr, "linear is NULL");
        auto &l = *const_cast<cgtp_linear *>(linear);
        check_linear(l, N);
        check_choice(l, experts, weights, N);
        require(l.cfg.top_k > 0 || (!slots && !offsets && !grad_weights),
                "slots, offsets or grad_weights given to a linear without a choice of experts");
        if (!grad_x && !grad_w && !grad_weights) return;
        if (grad_w) require_ptr(grad_w, "grad_w", l.elem);
        const bool routed = l.cfg.top_k > 0;
        long len = (long)stretch_len(l, N), count = (long)slots_of(l, N);
        if (N == 0) {
            if (!grad_w) return;
            const void *none = nullptr;
            const int32_t *no_offsets = nullptr;
            void *args[] = {&none, &no_offsets, &count, &len, &grad_w};
            run2(l.mod.here()[cgtp_linear::reduce], (l.numel + 255) / 256, l.cfg.experts, 256, args, stream);
            return;
        }
        const Rows X{x, l.d_in, x_ld, "x"}, G{grad_out, l.d_out, grad_out_ld, "grad_out"},
            GX{grad_x, l.d_in, grad_x_ld, "grad_x"};
        const bool to_x = grad_x || grad_weights;
        if (grad_w || grad_weights) check_rows(l.elem, N, X);
        check_rows(l.elem, N, G);
        if (grad_x) check_rows(l.elem, N, GX);
        if (to_x) require_ptr(w, "w", l.elem);
        if (grad_weights) require_ptr(grad_weights, "grad_weights", l.real);
        if (rows) require_ptr(rows, "rows", 4);
        if (grad_w && routed) {
            require_ptr(slots, "slots", 4);
            require_ptr(offsets, "offsets", 4);
        }
        const size_t need = backward_bytes(l, N), ns = (size_t)N * l.cfg.top_k;
        require_ptr(workspace, "workspace", 256);
        require(workspace_bytes >= need, "workspace too small (see cgtp_linear_workspace_size)");
        Arguments all(l.elem, N);
        if (grad_w || grad_weights) all.rows(X, false);
        all.rows(G, false);
        all.rows(GX, true);
        if (to_x) all.flat(w, weight_bytes(l), "w", false);
        all.flat(experts, ns * 4, "experts", false);
        all.flat(weights, ns * l.real, "weights", false);
        all.flat(rows, (size_t)N * 4, "rows", false);
        all.flat(slots, ns * 4, "slots", false);
        all.flat(offsets, (size_t)(l.cfg.experts + 1) * 4, "offsets", false);
        all.flat(grad_w, weight_bytes(l), "grad_w", true);
        all.flat(grad_weights, ns * l.real, "grad_weights", true);
        all.flat(workspace, need, "workspace", true);
        all.check();
        const auto &F = l.mod.here();
        long xl = (long)x_ld, gl = (long)grad_out_ld, gxl = (long)grad_x_ld, n = (long)N;
        void *turned = workspace, *part = static_cast<char *>(workspace) + aligned(weight_bytes(l));
        if (to_x) {
            void *targs[] = {&w, &turned};
            run2(F[cgtp_linear::transpose], (l.numel + 255) / 256, l.cfg.experts, 256, targs, stream);
            void *args[] = {&grad_out, &gl, &turned, &experts, &weights, &rows, &n, &grad_x, &gxl, &x, &xl, &grad_weights};
            const bool few = few_rows(N);
            run(F[few ? cgtp_linear::backward_x_few : cgtp_linear::backward_x], (N + 15) / 16,
                (few ? l.bwd_few : l.bwd).waves * 64, args, stream);
        }
        if (grad_w) {
            void *args[] = {&x, &xl, &grad_out, &gl, &weights, &slots, &offsets, &n, &count, &len, &part};
            run(F[cgtp_linear::backward_w], (int64_t)l.tiles.size() * stretches(l, N), 256, args, stream);
            void *rargs[] = {&part, &offsets, &count, &len, &grad_w};
            run2(F[cgtp_linear::reduce], (l.numel + 255) / 256, l.cfg.experts, 256, rargs, stream);
        }
    });
}

}  // extern "C"
