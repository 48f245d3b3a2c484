// ex_router.cuh -- the launchers of ex_router.cu.
#pragma once

#include "ex_common.cuh"
#include "zc_router.h"

namespace zc {
namespace ex {

struct RouterShape {
  size_t tokens;
  int experts, k, type, score, normalize;
  float scale;
};

cudaError_t launch_route(const RouterShape& s, const void* logits, size_t pitch, float* weights, int* ids,
                         cudaStream_t stream);
cudaError_t launch_route_grad(const RouterShape& s, const float* d_weights, const int* ids, const float* d_loss,
                              const float* slope, const void* logits, size_t pitch, void* d_logits, size_t d_pitch,
                              const DeviceInfo& dev, cudaStream_t stream);
size_t balance_workspace(size_t tokens, int experts);
cudaError_t launch_balance(const RouterShape& s, const void* logits, size_t pitch, const int* ids, float* loss, int* counts,
                           float* slope, void* workspace, cudaStream_t stream);

}  // namespace ex
}  // namespace zc
