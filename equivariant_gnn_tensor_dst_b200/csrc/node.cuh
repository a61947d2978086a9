// Device helpers of the node-feature kernels: storage types, the dropout generator, sums.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "node.h"

namespace tpc {

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
template <class T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

// Philox4x32-10: ten rounds of two 32 x 32 -> 64 products on a 128-bit counter (Salmon et al. 2011,
// section 4.3); the rounds' keys come with the call.
__device__ __forceinline__ uint4 philox10(uint32_t c0, uint32_t c1, uint32_t c2, uint32_t c3, const Drop& D) {
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const uint64_t a = (uint64_t)c0 * 0xD2511F53u, b = (uint64_t)c2 * 0xCD9E8D57u;
    c0 = (uint32_t)(b >> 32) ^ c1 ^ D.key[i][0];
    c1 = (uint32_t)b;
    c2 = (uint32_t)(a >> 32) ^ c3 ^ D.key[i][1];
    c3 = (uint32_t)a;
  }
  return make_uint4(c0, c1, c2, c3);
}

__device__ __forceinline__ uint32_t word_of(const uint4& w, int i) {
  return i == 0 ? w.x : i == 1 ? w.y : i == 2 ? w.z : w.w;
}

// offset + *step of a call
__device__ __forceinline__ uint64_t drop_offset(const Drop& D) {
  return D.offset + (D.step ? (uint64_t)*D.step : 0ull);
}

// Words of a row's channel group.
__device__ __forceinline__ uint4 drop_words(const Drop& D, uint64_t off, uint32_t group, uint32_t row) {
  return philox10(group, row, (uint32_t)off, (uint32_t)(off >> 32), D);
}

// kept ? v * scale : 0 for one channel, drawing its group's words
__device__ __forceinline__ float drop_one(const Drop& D, uint64_t off, const NodeBlock& B, int c, uint32_t row,
                                          float v) {
  if (D.mode == 0) return v;
  if (D.mode == 2) return 0.f;
  const uint4 w = drop_words(D, off, B.grp0 + (c >> 2), row);
  return word_of(w, c & 3) >= D.threshold ? __fmul_rn(v, D.scale) : 0.f;
}

// Two 16-bit elements of a word, lower address first.
template <class T>
__device__ __forceinline__ void unpack(uint32_t w, float& x, float& y);
template <>
__device__ __forceinline__ void unpack<__nv_bfloat16>(uint32_t w, float& x, float& y) {
  x = __uint_as_float(w << 16);
  y = __uint_as_float(w & 0xffff0000u);
}
template <>
__device__ __forceinline__ void unpack<__half>(uint32_t w, float& x, float& y) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
  x = f.x;
  y = f.y;
}
template <class T>
__device__ __forceinline__ uint32_t pack(float x, float y);
template <>
__device__ __forceinline__ uint32_t pack<__nv_bfloat16>(float x, float y) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&v);
}
template <>
__device__ __forceinline__ uint32_t pack<__half>(float x, float y) {
  const __half2 v = __floats2half2_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Which channels of a block the elements s (block-relative) belong to.
struct Channels {
  int mul_ir, C, d;
  uint32_t inv;  // ceil(2^32 / (mul_ir ? d : C)): exact quotients for s, C < 2^15
  __device__ __forceinline__ Channels(const NodeDesc& D, const NodeBlock& B) : mul_ir(D.mul_ir), C(B.C), d(B.d) {
    const uint32_t q = mul_ir ? d : C;
    inv = q > 1 ? (uint32_t)((0x100000000ull + q - 1) / q) : 0;
  }
  __device__ __forceinline__ int of(int s) const {
    if (mul_ir) return d == 1 ? s : (int)__umulhi((uint32_t)s, inv);
    return C == 1 ? 0 : s - C * (int)__umulhi((uint32_t)s, inv);
  }
  __device__ __forceinline__ int at(int c, int m) const { return mul_ir ? c * d + m : m * C + c; }
};

// Sums of K values over groups of G lanes (a power of two, at most 32), to all lanes of a group.  One
// branch on G: one a step, and what it takes to bring the lanes together again, cost as much as it
// saved.
template <int K>
__device__ __forceinline__ void group_step(float (&v)[K], int G, int o) {
  const bool in = G > o;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const float w = __shfl_xor_sync(0xffffffffu, v[k], o);
    v[k] += in ? w : 0.f;
  }
}
template <int K>
__device__ __forceinline__ void group_sum(float (&v)[K], int G) {
  if (G > 8) {
    group_step(v, G, 16);
    group_step(v, G, 8);
  }
  group_step(v, G, 4);
  group_step(v, G, 2);
  group_step(v, G, 1);
}

}  // namespace tpc
