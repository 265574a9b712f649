// The scan over packed prompts with dstate 32.
#include "scan_packed.cuh"

template int ssm::packed::launch_n<__nv_bfloat16, 32>(PackedParams&, bool, cudaStream_t);
template int ssm::packed::launch_n<float, 32>(PackedParams&, bool, cudaStream_t);
