// Launchers of the lists by expert (order.hip).
#pragma once

#include <hip/hip_runtime_api.h>

#include <cstdint>

namespace cgtp {

constexpr int kOrderBins = 4097;   // keys of a list, one of them for what has no expert
constexpr int kStretch = 8192;     // most items of a list that one workgroup places
constexpr int kMaxExperts = 512;

size_t order_workspace(int64_t N, int K, int E);
hipError_t launch_order(int64_t N, int K, int E, const int32_t *experts, int32_t *rows, int32_t *slots, int32_t *offsets,
                        void *workspace, hipStream_t st);

}  // namespace cgtp
