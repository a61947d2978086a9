// Irreps layer norm: forward, backward, double backward, and the forward and backward fused
// with dropout and the residual sum (include/tpconv_node.h has the formulas).
#include "node.cuh"

namespace tpc {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxParts = 296;  // row ranges with partial sums of their own (weight and bias gradients)

// Sums of K values over the CTA, to all its threads.
template <int K>
__device__ __forceinline__ void cta_sum(float (&v)[K]) {
  __shared__ float part[kThreads / 32][K];
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
  __syncthreads();  // the previous call's readers are done
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int k = 0; k < K; ++k) part[threadIdx.x >> 5][k] = v[k];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < K; ++k) {
    v[k] = 0.f;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) v[k] += part[w][k];
  }
}

// Floats of one row range's partial sums: channels, then the 0e channels again (bias).
__host__ __device__ inline int part_width(const NodeDesc& D) { return D.channels + D.biases; }

// ---- any block size: one CTA per row of a block, a thread owning whole channels ----

struct Elem {  // element (component m, channel c) of a block
  int mul_ir, C, d;
  __device__ __forceinline__ int at(int c, int m) const { return mul_ir ? c * d + m : m * C + c; }
};

template <class T, bool FUSED>
__global__ void __launch_bounds__(kThreads) k_norm_fwd_any(const NodeDesc D, const Drop drop, const NormArgs A,
                                                           const long long N) {
  const NodeBlock B = D.b[blockIdx.y];
  const Elem E{D.mul_ir, B.C, B.d};
  const bool centred = B.bias0 >= 0;
  const float inv = 1.f / (float)B.S;
  const uint64_t off = FUSED ? drop_offset(drop) : 0;
  for (long long n = blockIdx.x; n < N; n += gridDim.x) {
    const T* x = (const T*)A.x + n * D.dim + B.off;
    const T* res = FUSED && A.residual ? (const T*)A.residual + n * D.dim + B.off : nullptr;
    auto value = [&](int c, int s) {
      float v = to_f32(x[s]);
      if (FUSED) {
        v = drop_one(drop, off, B, c, (uint32_t)n, v);
        if (res) v += to_f32(res[s]);
      }
      return v;
    };
    float mu[1] = {0.f}, q[1] = {0.f};
    if (centred) {
      for (int c = threadIdx.x; c < B.C; c += kThreads)
        for (int m = 0; m < B.d; ++m) mu[0] += value(c, E.at(c, m));
      cta_sum(mu);
      mu[0] *= inv;
    }
    for (int c = threadIdx.x; c < B.C; c += kThreads)
      for (int m = 0; m < B.d; ++m) {
        const float u = value(c, E.at(c, m)) - mu[0];
        q[0] += u * u;
      }
    cta_sum(q);
    const float r = 1.f / sqrtf(q[0] * inv + D.eps);
    for (int c = threadIdx.x; c < B.C; c += kThreads) {
      const float w = A.weight ? A.weight[B.chan0 + c] : 1.f;
      const float b = centred && A.bias ? A.bias[B.bias0 + c] : 0.f;
      for (int m = 0; m < B.d; ++m) {
        const int s = E.at(c, m);
        const float v = value(c, s);
        if (FUSED) ((T*)A.z)[n * D.dim + B.off + s] = from_f32<T>(v);
        ((T*)A.y)[n * D.dim + B.off + s] = from_f32<T>((v - mu[0]) * r * w + b);
      }
    }
  }
}

template <class T, bool FUSED>
__global__ void __launch_bounds__(kThreads) k_norm_bwd_any(const NodeDesc D, const Drop drop, const NormArgs A,
                                                           const long long N) {
  const NodeBlock B = D.b[blockIdx.y];
  const Elem E{D.mul_ir, B.C, B.d};
  const bool centred = B.bias0 >= 0;
  const float inv = 1.f / (float)B.S;
  const uint64_t off = FUSED ? drop_offset(drop) : 0;
  float* pw = A.partial ? A.partial + (long long)blockIdx.x * part_width(D) + B.chan0 : nullptr;
  float* pb = A.partial && centred ? A.partial + (long long)blockIdx.x * part_width(D) + D.channels + B.bias0 : nullptr;
  for (long long n = blockIdx.x; n < N; n += gridDim.x) {
    const long long row = n * D.dim + B.off;
    const T *x = (const T*)A.x + row, *g = (const T*)A.grad_y + row;
    float m1[2] = {0.f, 0.f};
    if (centred) {
      for (int c = threadIdx.x; c < B.C; c += kThreads) {
        const float w = A.weight ? A.weight[B.chan0 + c] : 1.f;
        for (int m = 0; m < B.d; ++m) {
          const int s = E.at(c, m);
          m1[0] += to_f32(x[s]);
          m1[1] += w * to_f32(g[s]);
        }
      }
      cta_sum(m1);
    }
    const float mu = m1[0] * inv, ma = m1[1] * inv;
    float m2[2] = {0.f, 0.f};
    for (int c = threadIdx.x; c < B.C; c += kThreads) {
      const float w = A.weight ? A.weight[B.chan0 + c] : 1.f;
      for (int m = 0; m < B.d; ++m) {
        const int s = E.at(c, m);
        const float u = to_f32(x[s]) - mu;
        m2[0] += u * u;
        m2[1] += u * (w * to_f32(g[s]) - ma);
      }
    }
    cta_sum(m2);
    const float r = 1.f / sqrtf(m2[0] * inv + D.eps), mh = r * m2[1] * inv;
    for (int c = threadIdx.x; c < B.C; c += kThreads) {
      const float w = A.weight ? A.weight[B.chan0 + c] : 1.f;
      float sw = 0.f, sb = 0.f;
      for (int m = 0; m < B.d; ++m) {
        const int s = E.at(c, m);
        const float gv = to_f32(g[s]), h = (to_f32(x[s]) - mu) * r;
        float t = r * (w * gv - ma - h * mh);
        sw += gv * h;
        sb += gv;
        if (FUSED) {
          if (A.grad_z) t += to_f32(((const T*)A.grad_z)[row + s]);
          if (A.grad_residual) ((T*)A.grad_residual)[row + s] = from_f32<T>(t);
          if (A.grad_x) ((T*)A.grad_x)[row + s] = from_f32<T>(drop_one(drop, off, B, c, (uint32_t)n, t));
        } else if (A.grad_x) {
          ((T*)A.grad_x)[row + s] = from_f32<T>(t);
        }
      }
      // the range's sums live in the workspace; the same thread owns channel c in every row
      const bool first = n == blockIdx.x;
      if (pw) pw[c] = first ? sw : pw[c] + sw;
      if (pb) pb[c] = first ? sb : pb[c] + sb;
    }
  }
}

template <class T>
__global__ void __launch_bounds__(kThreads) k_norm_dbl_any(const NodeDesc D, const NormArgs A, const long long N) {
  const NodeBlock B = D.b[blockIdx.y];
  const Elem E{D.mul_ir, B.C, B.d};
  const bool centred = B.bias0 >= 0;
  const float inv = 1.f / (float)B.S;
  float* pw = A.partial ? A.partial + (long long)blockIdx.x * part_width(D) + B.chan0 : nullptr;
  for (long long n = blockIdx.x; n < N; n += gridDim.x) {
    const long long row = n * D.dim + B.off;
    const T *x = (const T*)A.x + row, *g = (const T*)A.grad_y + row;
    const T* p = A.gg_x ? (const T*)A.gg_x + row : nullptr;
    auto weight = [&](int c) { return A.weight ? A.weight[B.chan0 + c] : 1.f; };
    auto tangent = [&](int c) { return A.gg_weight ? A.gg_weight[B.chan0 + c] : 0.f; };
    auto pv = [&](int s) { return p ? to_f32(p[s]) : 0.f; };
    float s1[4] = {0.f, 0.f, 0.f, 0.f};  // x, p, a, w
    if (centred) {
      for (int c = threadIdx.x; c < B.C; c += kThreads)
        for (int m = 0; m < B.d; ++m) {
          const int s = E.at(c, m);
          s1[0] += to_f32(x[s]);
          s1[1] += pv(s);
          s1[2] += weight(c) * to_f32(g[s]);
          s1[3] += tangent(c) * to_f32(g[s]);
        }
      cta_sum(s1);
    }
    const float mx = s1[0] * inv, mp = s1[1] * inv, ma = s1[2] * inv, mw = s1[3] * inv;
    float s2[5] = {0.f, 0.f, 0.f, 0.f, 0.f};  // u u, u p', u a', p' a', u w'
    for (int c = threadIdx.x; c < B.C; c += kThreads)
      for (int m = 0; m < B.d; ++m) {
        const int s = E.at(c, m);
        const float u = to_f32(x[s]) - mx, gv = to_f32(g[s]);
        const float pp = pv(s) - mp, aa = weight(c) * gv - ma, ww = tangent(c) * gv - mw;
        s2[0] += u * u;
        s2[1] += u * pp;
        s2[2] += u * aa;
        s2[3] += pp * aa;
        s2[4] += u * ww;
      }
    cta_sum(s2);
    const float r = 1.f / sqrtf(s2[0] * inv + D.eps);
    const float P = r * s2[1] * inv, Q = r * s2[2] * inv, R = s2[3] * inv, V = r * s2[4] * inv;
    for (int c = threadIdx.x; c < B.C; c += kThreads) {
      const float w = weight(c), t = tangent(c);
      const float b = centred && A.gg_bias ? A.gg_bias[B.bias0 + c] : 0.f;
      float sw = 0.f;
      for (int m = 0; m < B.d; ++m) {
        const int s = E.at(c, m);
        const float h = (to_f32(x[s]) - mx) * r, gv = to_f32(g[s]);
        const float pp = pv(s) - mp, aa = w * gv - ma, ww = t * gv - mw;
        const float k = r * (pp - h * P);
        sw += gv * k;
        if (A.grad_grad_y) ((T*)A.grad_grad_y)[row + s] = from_f32<T>(w * k + t * h + b);
        if (A.grad_x)
          ((T*)A.grad_x)[row + s] =
              from_f32<T>(r * r * (h * (3.f * P * Q - R) - Q * pp - P * aa) + r * (ww - h * V));
      }
      if (pw) pw[c] = n == blockIdx.x ? sw : pw[c] + sw;
    }
  }
}

// ---- sums of the partials over the row ranges, in range order ----

__global__ void k_norm_reduce(const NodeDesc D, const float* __restrict__ partial, int parts, float* grad_weight,
                              float* grad_bias) {
  const int i = blockIdx.x * blockDim.x + threadIdx.x, width = part_width(D);
  if (i >= width) return;
  float* out = i < D.channels ? (grad_weight ? grad_weight + i : nullptr)
                              : (grad_bias ? grad_bias + (i - D.channels) : nullptr);
  if (!out) return;
  float v = 0.f;
  for (int k = 0; k < parts; ++k) v += partial[(long long)k * width + i];
  *out = v;
}

inline int row_parts(long long N) { return (int)(N < kMaxParts ? N : kMaxParts); }

template <class T>
cudaError_t run_norm(NormPass pass, const NodeDesc& D, long long N, const NormArgs& A, const Drop* drop,
                     cudaStream_t s) {
  const Drop none{};
  const dim3 grid(pass == NORM_FORWARD ? (unsigned)(N < 65535 ? N : 65535) : (unsigned)row_parts(N), D.n_blocks);
  if (pass == NORM_FORWARD) {
    if (drop) k_norm_fwd_any<T, true><<<grid, kThreads, 0, s>>>(D, *drop, A, N);
    else k_norm_fwd_any<T, false><<<grid, kThreads, 0, s>>>(D, none, A, N);
  } else if (pass == NORM_BACKWARD) {
    if (drop) k_norm_bwd_any<T, true><<<grid, kThreads, 0, s>>>(D, *drop, A, N);
    else k_norm_bwd_any<T, false><<<grid, kThreads, 0, s>>>(D, none, A, N);
  } else {
    k_norm_dbl_any<T><<<grid, kThreads, 0, s>>>(D, A, N);
  }
  if (A.partial)
    k_norm_reduce<<<(part_width(D) + 127) / 128, 128, 0, s>>>(D, A.partial, row_parts(N), A.grad_weight, A.grad_bias);
  return cudaGetLastError();
}

}  // namespace

size_t norm_partial_floats(const NodeDesc& D, long long N) { return (size_t)row_parts(N) * part_width(D); }

cudaError_t launch_norm(NormPass pass, int dtype, const NodeDesc& D, long long N, const NormArgs& A, const Drop* drop,
                        cudaStream_t s) {
  if (dtype == 0) return run_norm<float>(pass, D, N, A, drop, s);
  if (dtype == 1) return run_norm<__nv_bfloat16>(pass, D, N, A, drop, s);
  return run_norm<__half>(pass, D, N, A, drop, s);
}

}  // namespace tpc
