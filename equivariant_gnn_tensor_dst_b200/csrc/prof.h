// The library's launch profiling (tpconv_profile_begin / _end), as seen by the launch code.
#pragma once
#include <cuda_runtime.h>

namespace tpc {

enum ProfCat {
  PC_UVW_STATE = 0, PC_UVW_STATE_TAN, PC_UVW_RECV_BWD, PC_UVW_SRC, PC_UVW_SRC_TAN, PC_GEMM,
  PC_UVU_FWD, PC_UVU_RECV_BWD, PC_UVU_GRADW, PC_UVU_SRC, PC_POS, PC_GRAPH, PC_RECV_TAN, PC_NODE, PC_COUNT
};

int prof_open(int category, int launches, cudaStream_t s);  // slot, or -1 while profiling is off
void prof_close(int slot, cudaStream_t s);
void prof_count(int category, int launches);                // launches known only as they are made

// Brackets one library call that launches `nk` kernels on stream s.
struct ProfScope {
  int slot;
  cudaStream_t s;
  ProfScope(int c, int nk, cudaStream_t st) : slot(prof_open(c, nk, st)), s(st) {}
  ~ProfScope() { prof_close(slot, s); }
};

}  // namespace tpc
