// norm_bwd.cuh -- parameters of the gated norm's gradient (gated_norm_bwd.cu).
#pragma once

#include "ssd_common.cuh"

namespace ssd {

struct NormBwdParams {
    const void *y, *z, *dout;
    int64_t yrs, zrs, dors;
    const float *w;
    float eps;
    int group;
    void *dy, *dz;
    int64_t dyrs, dzrs;
    float *dw;
    float *ws;                  // [grid * teams][d]
    int64_t rows;
    int d;
};

struct NormBwdPlan {
    int teams, threads, grid;
};
NormBwdPlan norm_bwd_plan(int64_t rows, int d, int sms);
int launch_gated_norm_backward(const NormBwdParams &p, int dtype, int sms, cudaStream_t st);

}  // namespace ssd
