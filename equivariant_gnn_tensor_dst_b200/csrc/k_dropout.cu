// Equivariant dropout with a counter-based mask (include/tpconv_node.h).
#include "node.cuh"

namespace tpc {
namespace {

constexpr int kThreads = 256;

// One thread per channel of a row, all its components.
template <class T>
__global__ void __launch_bounds__(kThreads) k_dropout_any(const NodeDesc D, const Drop drop, const T* x, const T* res,
                                                          T* out, const long long N) {
  const NodeBlock B = D.b[blockIdx.y];
  const uint64_t off = drop_offset(drop);
  for (long long n = blockIdx.x; n < N; n += gridDim.x)
    for (int c = threadIdx.x; c < B.C; c += kThreads)
      for (int m = 0; m < B.d; ++m) {
        const long long i = n * D.dim + B.off + (D.mul_ir ? c * B.d + m : m * B.C + c);
        float v = drop_one(drop, off, B, c, (uint32_t)n, to_f32(x[i]));
        if (res) v += to_f32(res[i]);
        out[i] = from_f32<T>(v);
      }
}

template <class T>
cudaError_t run_dropout(const NodeDesc& D, long long N, const void* x, const void* residual, const Drop& drop,
                        void* out, cudaStream_t s) {
  const dim3 grid((unsigned)(N < 65535 ? N : 65535), D.n_blocks);
  k_dropout_any<T><<<grid, kThreads, 0, s>>>(D, drop, (const T*)x, (const T*)residual, (T*)out, N);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_dropout(int dtype, const NodeDesc& D, long long N, const void* x, const void* residual,
                           const Drop& drop, void* out, cudaStream_t s) {
  if (dtype == 0) return run_dropout<float>(D, N, x, residual, drop, out, s);
  if (dtype == 1) return run_dropout<__nv_bfloat16>(D, N, x, residual, drop, out, s);
  return run_dropout<__half>(D, N, x, residual, drop, out, s);
}

}  // namespace tpc
