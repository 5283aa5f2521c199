// What every extern "C" entry point of libcgtp shares: the calling thread's last message, the
// guard that turns an exception into a status, and the argument checks made before any HIP call.
#pragma once

#include <hip/hip_runtime_api.h>

#include <cstdint>
#include <new>
#include <string>

#include "plan.h"

namespace cgtp {

inline std::string &last_error_message()
{
    static thread_local std::string msg;
    return msg;
}

inline cgtp_status fail(cgtp_status code, const std::string &msg)
{
    last_error_message() = msg;
    return code;
}

template <class F> cgtp_status guarded(F &&f)
{
    try {
        f();
        return CGTP_OK;
    } catch (const Error &e) {
        return fail(e.code, e.what());
    } catch (const std::bad_alloc &) {
        return fail(CGTP_ERR_INTERNAL, "host out of memory");
    } catch (const std::exception &e) {
        return fail(CGTP_ERR_INTERNAL, e.what());
    } catch (...) {
        return fail(CGTP_ERR_INTERNAL, "unknown failure");
    }
}

inline void require(bool ok, const std::string &msg)
{
    if (!ok) throw Error(CGTP_ERR_INVALID_ARG, msg);
}

inline void require_ptr(const void *p, const char *name, size_t align)
{
    if (!p) throw Error(CGTP_ERR_INVALID_ARG, std::string(name) + " is NULL");
    if (reinterpret_cast<uintptr_t>(p) % align)
        throw Error(CGTP_ERR_INVALID_ARG,
                    std::string(name) + " is not aligned to " + std::to_string(align) + " bytes");
}

// [a, a+na) and [b, b+nb) in bytes must not overlap
inline void require_disjoint(const void *a, size_t na, const char *an, const void *b, size_t nb, const char *bn)
{
    if (!a || !b || !na || !nb) return;
    auto x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    if (!(x + na <= y || y + nb <= x))
        throw Error(CGTP_ERR_INVALID_ARG, std::string(an) + " overlaps " + bn);
}

inline void check_hip(hipError_t e, const char *what)
{
    if (e != hipSuccess) throw Error(CGTP_ERR_HIP, std::string(what) + ": " + hipGetErrorString(e));
}

}  // namespace cgtp
