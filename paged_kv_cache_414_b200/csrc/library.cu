// The library's one translation unit: the 16-bit pool's kernels and entry
// points, then the operators around the 8-bit pool and the prompt pass, which
// use the former's helpers and its device error word.
#include "pa_kernels.cu"

#include "fp8_cache.cuh"
#include "decode_fp8.cuh"
#include "prompt_attention.cuh"

#include "serving_api.cuh"
