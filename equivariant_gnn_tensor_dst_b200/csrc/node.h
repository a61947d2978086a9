// Node-feature operators (include/tpconv_node.h): what the plan, the launch code and the
// kernels share.
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

#include "internal.h"

namespace tpc {

// One irrep block of a row: C channels of d = 2l+1 components, S = C d elements.
struct NodeBlock {
  int off, C, d, S;
  int chan0;   // first channel of the row's channel numbering (weight)
  int bias0;   // first channel of the bias numbering; < 0: not a 0e block (no centring, no bias)
  int grp0;    // first dropout group (four channels) of the row's group numbering
};

struct NodeDesc {
  int n_blocks, dim, channels, biases, groups;
  int mul_ir;  // 0: blocks [d][C], 1: blocks [C][d]
  float eps;
  NodeBlock b[MAX_BLOCKS];
};

// Dropout of one call as the kernels see it.
struct Drop {
  uint32_t key[10][2];    // the seed's words, and what each round makes of them
  uint64_t offset;
  const long long* step;  // device, added to offset; may be NULL
  uint32_t threshold;     // dropped iff word < threshold
  int mode;               // 0: all kept, nothing to draw (p = 0), 1: drawn, 2: all dropped (p = 1)
  float scale;            // 1 / (1 - p), 0 at p = 1
};

// Arguments of the norm passes.  Element type T is the launcher's `dtype`.
struct NormArgs {
  const void* x;          // input; z in the fused backward
  const float *weight, *bias;
  // forward
  const void* residual;
  void *y, *z;
  // backward
  const void *grad_y, *grad_z;
  void *grad_x, *grad_residual;
  // double backward
  const void* gg_x;
  const float *gg_weight, *gg_bias;
  void* grad_grad_y;
  // sums over rows
  float *grad_weight, *grad_bias;
  float* partial;         // workspace; NULL when neither sum is wanted
};

enum NormPass { NORM_FORWARD = 0, NORM_BACKWARD = 1, NORM_DOUBLE_BACKWARD = 2 };

// drop != NULL: the fused dropout + residual variants of forward and backward.
cudaError_t launch_norm(NormPass pass, int dtype, const NodeDesc& D, long long N, const NormArgs& A, const Drop* drop,
                        cudaStream_t s);
size_t norm_partial_floats(const NodeDesc& D, long long N, int esize);  // elements of esize bytes
cudaError_t launch_dropout(int dtype, const NodeDesc& D, long long N, const void* x, const void* residual,
                           const Drop& drop, void* out, cudaStream_t s);

}  // namespace tpc
