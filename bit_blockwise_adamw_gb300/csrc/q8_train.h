// q8_train.h -- declarations shared by the training-step operators' translation
// units (include/q8train.h): launchers, and small device helpers.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "q8train.h"

namespace q8 {

// Launch configurations of each unit's kernels, worked out ahead of the first
// call (q8_prepare_device).
cudaError_t prepare_ff();
cudaError_t prepare_norm();
cudaError_t prepare_distill();

// The current device's SM count, and the host-mapped word that a kernel sets
// when one of its waits ran out.
struct DeviceInfo {
    int sms = 0;
    int32_t* fault = nullptr;
};
cudaError_t device_info(DeviceInfo* out);

// A launch that gave up waiting is reported by the next call on its device.
cudaError_t earlier_fault(int32_t* fault);

// Launchers: arguments already checked.
struct FfBackward {
    const uint16_t* dh;
    int64_t dh_stride;
    const float* saved;
    uint16_t* dx;
    int64_t dx_stride;
    uint16_t* dw_gate;
    uint16_t* dw_up;
};
int64_t ff_workspace(const q8_gated_ff& f, bool backward);
cudaError_t launch_ff_forward(const q8_gated_ff& f, uint16_t* h, int64_t h_stride, float* saved, cudaStream_t st);
cudaError_t launch_ff_backward(const q8_gated_ff& f, const FfBackward& b, cudaStream_t st);

cudaError_t launch_norm_forward(const q8_block_norm& n, void* residual_out, int64_t residual_out_stride, uint16_t* z,
                                int64_t z_stride, cudaStream_t st);
int64_t norm_workspace(const q8_block_norm& n, const q8_block_norm_grads& g);
cudaError_t launch_norm_backward(const q8_block_norm& n, const q8_block_norm_grads& g, cudaStream_t st);

// forward: loss non-NULL; backward alone: loss NULL, stats read.
cudaError_t launch_distill(const q8_distill_topk& d, float* loss, float* stats_out, const float* stats_in,
                           void* dlogits, int64_t dlogits_stride, cudaStream_t st);

__device__ __forceinline__ float bf16_to_float(uint16_t b) { return __uint_as_float(static_cast<uint32_t>(b) << 16); }

__device__ __forceinline__ uint16_t float_to_bf16(float x)
{
    return __bfloat16_as_ushort(__float2bfloat16_rn(x));
}

}  // namespace q8
