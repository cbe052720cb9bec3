// host_api.cuh -- what the translation units with entry points share on the
// host: the muon_last_error() text, the device check, the profiler's launch
// bracket and the tensor-map encoder (all defined in muon_api.cu).
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <functional>

#include "../../include/muon_b200.h"

namespace muon {

// Kernel kinds the profiler sums by (names in muon_api.cu, same order).
enum Kind {
  K_MOMENTUM = 0, K_NORM, K_GRAM, K_POLY, K_AXPY, K_AXPY_UPDATE, K_UPDATE, K_EMIT, K_ADAMW,
  K_GRAM_F32, K_POLY_F32, K_AXPY_F32, K_AXPY_UPDATE_F32, K_NORMUON_UPDATE, K_MOMENTUM_ROWEQ,
  K_EMBED, K_EMBED_SORT, K_EMBED_GRAD, K_LAYER_NORM, K_LAYER_NORM_GRAD, K_CKPT_PACK, K_CKPT_UNPACK,
  K_WEIGHT_GRAD, K_COUNT
};

void api_clear_error();
muon_status api_fail(muon_status st, const char* fmt, ...);
muon_status api_cuda_fail(cudaError_t e, const char* what);
// The current device's SM count; fails unless it is compute capability 10.0.
muon_status api_device(int* sms);
cudaError_t api_timed_launch(int kind, cudaStream_t s, const std::function<cudaError_t()>& f);
// 2-D to 5-D tiled tensor map over `base` (dims and box innermost first,
// strides in bytes of dims 1..); out-of-range elements load as zeros.
muon_status api_tensor_map(CUtensorMap* map, CUtensorMapDataType type, int rank, void* base,
                           const cuuint64_t* dims, const cuuint64_t* strides, const cuuint32_t* box,
                           CUtensorMapSwizzle swizzle);

}  // namespace muon
