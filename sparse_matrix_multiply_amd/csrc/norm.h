// RMS norm (include/mmac_norm.h): parameters of the kernels and their launchers.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mmac {

// Pitches in bytes.
struct NormParams {
    const uint8_t *X;
    int64_t x_pitch;
    const uint8_t *R;        // NULL, or what is added to X
    int64_t r_pitch;
    const void *w;
    uint8_t *H;              // NULL, or X + R as rounded to X's type
    int64_t h_pitch;
    uint8_t *Y;              // X's type, or 8-bit elements
    int64_t y_pitch;
    uint32_t *SY;            // scale words of 8-bit elements
    int64_t lds;
    float *rstd;             // NULL, or one per row
    int64_t M;
    int N;
    float eps;
};

struct NormGradParams {
    const uint8_t *dY;
    int64_t dy_pitch;
    const uint8_t *H;
    int64_t h_pitch;
    const void *w;
    const float *rstd;
    const uint8_t *dH;       // NULL, or what is added to the gradient
    int64_t dh_pitch;
    uint8_t *dX;
    int64_t dx_pitch;
    float *dW;               // NULL, or N sums
    float *partials;         // norm_grad_parts(M) rows of N sums
    int64_t M;
    int N;
};

// Workgroups of the backward kernel, each with a row of partial sums.
int norm_grad_parts(int64_t M, int64_t N);

// y_type: X's type or DT_E4M3 / DT_E5M2.
hipError_t launch_rmsnorm(int x_type, int w_type, int y_type, const NormParams &p, hipStream_t s);
hipError_t launch_rmsnorm_grad(int x_type, int w_type, const NormGradParams &p, hipStream_t s);

}  // namespace mmac
