// slots.cuh -- parameters of the single-token step over a pool of slots (decode_slots.cu).
#pragma once

#include "ssd_common.cuh"

namespace ssd {

struct SlotDecodeParams {
    int b, H, P, N, G;
    int n_slots;
    const int *slots;           // [b], -1 = an empty row
    const void *u;
    int64_t ubs;
    const float *w, *bias;
    const void *tail_in;        // [n_slots][3][C_ch]
    void *tail_out;
    const float *dt, *A, *D;
    const float *h_in;          // [n_slots][H][P][N]
    float *h_out;
    void *y;
    int64_t ybs;
    const float *dt_bias;
    int dt_softplus;
    float dt_min, dt_max;
    int heads_per_cta, stages;  // set by the launcher
    unsigned int *status;
    uint64_t wait_limit_ns;
    int64_t test_drop_unit;     // the CTA whose copies are never issued (test hook), or -1
};

int launch_slot_decode(const SlotDecodeParams &p, int dtype, int sms, cudaStream_t st);

}  // namespace ssd
