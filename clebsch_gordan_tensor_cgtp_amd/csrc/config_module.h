// A module compiled for one configuration of an operator, loaded on each device at its first use there.
#pragma once

#include <hip/hip_runtime_api.h>

#include <map>
#include <mutex>
#include <string>
#include <vector>

#include "abi_util.h"

namespace cgtp {

inline const char *type_name(int dtype)
{
    switch (dtype) {
    case CGTP_F64: return "double";
    case CGTP_BF16: return "__bf16";
    case CGTP_F16: return "_Float16";
    default: return "float";
    }
}

inline int elem_bytes(int dtype) { return dtype == CGTP_F64 ? 8 : dtype == CGTP_F32 ? 4 : 2; }
inline int real_bytes(int dtype) { return dtype == CGTP_F64 ? 8 : 4; }

class ConfigModule {
public:
    // compiles the source; `kernels` are the functions that here() lists, in this order
    void build(const std::string &text, std::vector<const char *> kernels)
    {
        source = text;
        names = std::move(kernels);
        code = compile_source(source);
    }

    // the kernels on the current device
    const std::vector<hipFunction_t> &here()
    {
        int dev = 0;
        check_hip(hipGetDevice(&dev), "hipGetDevice");
        std::lock_guard<std::mutex> lock(mu);
        auto it = loaded.find(dev);
        if (it != loaded.end()) return it->second.fns;
        Loaded l;
        check_hip(hipModuleLoadData(&l.module, code.data()), "hipModuleLoadData");
        for (const char *name : names) {
            hipFunction_t f = nullptr;
            check_hip(hipModuleGetFunction(&f, l.module, name), name);
            l.fns.push_back(f);
        }
        return loaded.emplace(dev, std::move(l)).first->second.fns;
    }

    void unload()
    {
        if (loaded.empty()) return;
        int prev = 0;
        const bool have_prev = hipGetDevice(&prev) == hipSuccess;
        for (auto &kv : loaded)
            if (kv.second.module && hipSetDevice(kv.first) == hipSuccess) (void)hipModuleUnload(kv.second.module);
        loaded.clear();
        if (have_prev) (void)hipSetDevice(prev);
    }

    std::string source;

private:
    struct Loaded {
        hipModule_t module = nullptr;
        std::vector<hipFunction_t> fns;
    };
    std::vector<char> code;
    std::vector<const char *> names;
    std::mutex mu;  // guards `loaded`
    std::map<int, Loaded> loaded;
};

}  // namespace cgtp
