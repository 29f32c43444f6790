// linear_q4.hip -- few-token products with packed int4 weights and group scales.
//
// The simplest form: one wave per output column, its lanes along K.
#include "moe_device.h"
#include "moe_launch.h"

namespace moe {

__global__ __launch_bounds__(256) void k_linear_q4_col(LinearQ4 a, int t0)
{
    const int lane = threadIdx.x & 63;
    const int n = blockIdx.x * 4 + (threadIdx.x >> 6), t = t0 + blockIdx.y;
    if (n >= a.N) return;
    const int groups = a.K / a.group;
    float y = 0.f;
    for (int k = lane * 2; k < a.K; k += 128) {
        const uint8_t b = a.q[(int64_t)n * (a.K / 2) + k / 2];
        const int64_t g = (int64_t)n * groups + k / a.group;
        const float s = a.scales_bf16 ? bf16_to_f32(((const uint16_t *)a.scales)[g]) : ((const float *)a.scales)[g];
        const uint16_t *x = a.x + t * a.x_stride + k;
        y += s * (bf16_to_f32(x[0]) * (float)((int)((b & 15u) ^ 8u) - 8) +
                  bf16_to_f32(x[1]) * (float)((int)((b >> 4) ^ 8u) - 8));
    }
    y = wave_sum_f32(y);
    if (lane) return;
    const int64_t at = (int64_t)t * a.N + n;
    if (a.residual) y += bf16_to_f32(a.residual[at]);
    if (a.out_f32) ((float *)a.out)[at] = y;
    else ((__bf16 *)a.out)[at] = (__bf16)y;
}

size_t linear_q4_workspace(int, int, int) { return 256; }

hipError_t launch_linear_q4(const LinearQ4 &a, hipStream_t st)
{
    for (int t = 0; t < a.T; t += 65535) {
        hipLaunchKernelGGL(k_linear_q4_col, dim3((a.N + 3) / 4, a.T - t < 65535 ? a.T - t : 65535), dim3(256), 0, st, a, t);
    }
    return hipGetLastError();
}

}  // namespace moe
