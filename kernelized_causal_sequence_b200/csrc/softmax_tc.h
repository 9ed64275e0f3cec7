// softmax_tc.h — host entry of the tensor-core softmax prefill.
#pragma once
#include "softmax_simt.cuh"
#include "tc_launch.h"

namespace la {

inline bool softmax_tc_supported(la_dtype in) { return in != LA_F32; }
la_status softmax_tc(const SoftmaxParams &sp, la_dtype in, la_dtype out, int d, int *status,
                     unsigned long long wait_ns, cudaStream_t st);
unsigned long long wait_limit_ns();   // la_set_wait_limit_ns

}  // namespace la
