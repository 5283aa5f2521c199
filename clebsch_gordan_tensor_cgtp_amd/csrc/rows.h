// Checks of row arguments and the launch of a compiled kernel, for the entry points whose rows may
// have a pitch.
#pragma once

#include <climits>
#include <vector>

#include "abi_util.h"

namespace cgtp {

// Rows of `width` elements every `ld` elements.
struct Rows {
    const void *p;
    int64_t width, ld;
    const char *name;
};

inline void check_rows(int elem, int64_t N, const Rows &r)
{
    require_ptr(r.p, r.name, elem);
    require(r.ld >= r.width && r.ld < INT_MAX,
            std::string(r.name) + ": row pitch " + std::to_string(r.ld) + " is below the row's " +
                std::to_string(r.width) + " elements or above 2^31-1");
    require(N <= ((int64_t)1 << 56) / (r.ld * elem), std::string(r.name) + ": more than 2^56 bytes");
}

// No row of one may overlap a row of the other: their ranges are apart, or both have the same
// pitch and lie side by side inside it (a block's output and its gates in one buffer).
inline void rows_apart(int elem, int64_t N, const Rows &x, const Rows &y)
{
    if (!x.p || !y.p || !N || !x.width || !y.width) return;
    const int64_t es = elem;
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

inline void rows_apart(int elem, int64_t N, const Rows &x, const void *p, size_t bytes, const char *name)
{
    if (!x.p || !p || !N) return;
    require_disjoint(x.p, (size_t)((N - 1) * x.ld + x.width) * elem, x.name, p, bytes, name);
}

// Every argument of a call with what it covers; no output may overlap any other.
class Arguments {
public:
    Arguments(int elem, int64_t N) : elem(elem), N(N) {}
    void rows(const Rows &r, bool out)
    {
        if (r.p) all.push_back({r, 0, out, true});
    }
    void flat(const void *p, size_t bytes, const char *name, bool out)
    {
        if (p && bytes) all.push_back({Rows{p, 0, 0, name}, bytes, out, false});
    }
    void check() const
    {
        for (size_t i = 0; i < all.size(); ++i)
            for (size_t j = 0; j < all.size(); ++j)
                if (all[i].out && i != j && (!all[j].out || j > i)) apart(all[i], all[j]);
    }

private:
    struct Item {
        Rows r;
        size_t bytes;
        bool out, is_rows;
    };
    void apart(const Item &a, const Item &b) const
    {
        if (a.is_rows && b.is_rows)
            rows_apart(elem, N, a.r, b.r);
        else if (a.is_rows)
            rows_apart(elem, N, a.r, b.r.p, b.bytes, b.r.name);
        else if (b.is_rows)
            rows_apart(elem, N, b.r, a.r.p, a.bytes, a.r.name);
        else
            require_disjoint(a.r.p, a.bytes, a.r.name, b.r.p, b.bytes, b.r.name);
    }
    int elem;
    int64_t N;
    std::vector<Item> all;
};

inline void check_count(int64_t N)
{
    require(N >= 0 && N < INT_MAX, "N must be in [0, 2^31-1)");
}

inline void run(hipFunction_t f, int64_t groups, int threads, void **args, void *stream)
{
    check_hip(hipModuleLaunchKernel(f, (unsigned)groups, 1, 1, (unsigned)threads, 1, 1, 0,
                                    static_cast<hipStream_t>(stream), args, nullptr),
              "hipModuleLaunchKernel");
}

}  // namespace cgtp
