#pragma once
// The tensor-core form of the scan over packed prompts (ssd_packed.cu), for the per-head layout
// with head dim 64, dstate 128 and bf16 I/O.
#include <cuda_runtime.h>

#include "ssm_scan.h"

namespace ssm {
namespace packed {

struct PackedParams;
bool ssd_packed_covers(const ssm_dims_t& d);
int ssd_packed_launch(PackedParams& p, cudaStream_t s);

}  // namespace packed
}  // namespace ssm
