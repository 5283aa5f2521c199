// The optimizer step's kernels (optim_kernels.hip) and the table of tensors they take.
#pragma once

#include <hip/hip_runtime_api.h>

#include <cstdint>

namespace cgtp {

// Moments lie in flat buffers in which every tensor starts at a whole unit: a workgroup's work.
constexpr int kUnit = 2048;
// Values that share a scale in the 8-bit form.
constexpr int kScaleBlock = 64;
// Most workgroups of a launch of the gradients' norm, and so partial sums of it.
constexpr int kNormGroups = 2048;
// Tensors of one launch: their table is a kernel argument, which may take 4 KB.
constexpr int kTableTensors = 112;

struct TensorTable {
    int32_t n = 0;
    int32_t unit[kTableTensors + 1];   // first unit of the launch, the launch's units at the end
    int32_t state[kTableTensors];      // first unit in the moments' buffers
    int64_t numel[kTableTensors];
    void *param[kTableTensors];
    const void *grad[kTableTensors];
};

struct StepScalars {
    double max_norm, grad_scale;  // max_norm 0: no clipping
    double lr, beta1, beta2, eps, weight_decay, bias1, bias2;
};

struct MomentBuffers {
    void *m, *v;     // 32 bits (64 for f64 tensors), or 8-bit codes
    float *scales;   // [2][blocks], 8-bit codes only
    void *master;    // single precision weights of 16-bit tensors, or NULL
    int64_t blocks;
};

enum class Elem { f32 = 0, f64 = 1, bf16 = 2, f16 = 3 };

hipError_t launch_adamw(Elem elem, bool codes, const TensorTable &t, const MomentBuffers &mb, const StepScalars &s,
                        const double *norm, const double *schedule, hipStream_t st);
// partial[workgroup] = sum of squares over that workgroup's units, in double; returns the workgroups
int grad_norm_groups(int64_t units);
hipError_t launch_square_sums(Elem elem, const TensorTable &t, double *partial, hipStream_t st);
hipError_t launch_norm(const double *partial, int64_t n, double *norm, hipStream_t st);
hipError_t launch_state_read(const void *m, const void *v, const float *scales, int64_t elements, float *m_out,
                             float *v_out, hipStream_t st);
hipError_t launch_state_write(const float *m_in, const float *v_in, int64_t elements, void *m, void *v, float *scales,
                              hipStream_t st);
hipError_t launch_schedule(double *schedule, double beta1, double beta2, const double *norm, double grad_scale,
                           hipStream_t st);

}  // namespace cgtp
