// Irreps layer norm and dropout on node rows: forward, backward, double backward, and the forward
// and backward fused with dropout and the residual sum (include/tpconv_node.h has the formulas).
//
// Every (row, block) segment of S = (2l+1) C elements is a norm of its own.  The passes are bound
// by HBM traffic (a few flops per byte): each array is read once into registers, the statistics
// are sums over the lanes that hold a segment, and outputs are written from the same registers.
//
//  * k_fwd / k_bwd / k_dbl<WIDE = false>: a segment is held by a group of G lanes (a power of two,
//    at most a warp), lane l holding the packs l, l + G, ... of V elements, J packs at most.  A CTA
//    serves one block of the irreps and strides over rows; the blocks share the CTAs in proportion
//    to their sizes, so that all of them walk through the rows at the same pace in one wave.
//    A lane's columns are the same in every row: weights stay in registers, and the sums over rows
//    are per-lane registers until the rows are done.  The next row's packs are loaded while the
//    current row is computed.
//  * WIDE = true: the CTA is the group (segments beyond a warp's registers).
//  * k_*_any: any width, the segment read again from cache for each sum.
//
// Sums over rows (weight and bias gradients) have no atomics: each CTA writes its partial sums to
// the workspace and k_norm_reduce adds them in CTA order; a launch with one CTA per block writes
// the gradients itself.
#include "node.cuh"

namespace tpc {
namespace {

constexpr int kThreads = 256;
constexpr int kSms = 148;
constexpr int kWideMax = 512;      // threads of a WIDE CTA
constexpr int kAnyParts = 296;     // row ranges of the any-width kernels
constexpr int kAnyFloats = 1 << 22;  // bound on their partial sums

enum Kind { KIND_GROUP, KIND_WIDE, KIND_ANY };

// Blocks served by one launch: CTAs [cta0[k], cta0[k + 1]) serve block blk[k].
struct RowMap {
  int n;
  int blk[MAX_BLOCKS];
  int cta0[MAX_BLOCKS + 1];
  int lg[MAX_BLOCKS];              // log2 of the group's lanes (KIND_GROUP)
  long long part0[MAX_BLOCKS];     // first float of the block's partial sums
  int direct;                      // one CTA per block: sums go to the gradients themselves
};

// The partial sums of one block: `parts` rows of weight sums (per channel, or per element of
// which `comps` belong to a channel) followed by bias sums.
struct PartMap {
  int n;
  int blk[MAX_BLOCKS];
  int parts[MAX_BLOCKS], comps[MAX_BLOCKS];
  long long part0[MAX_BLOCKS];
};

__host__ __device__ inline long long part_stride(const NodeBlock& B, int comps) {
  return (long long)B.C * comps + (B.bias0 >= 0 ? B.C : 0);
}

// Sums of K values over the CTA (any number of warps), to all its threads.
template <int K>
__device__ __forceinline__ void cta_sum(float (&v)[K]) {
  __shared__ float part[K][32];
  group_sum(v, 32);
  __syncthreads();  // the previous call's readers are done
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int k = 0; k < K; ++k) part[k][threadIdx.x >> 5] = v[k];
  __syncthreads();
  const int warps = blockDim.x >> 5;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    v[k] = 0.f;
    for (int w = 0; w < warps; ++w) v[k] += part[k][w];
  }
}

// ---- segments in registers ----

// A thread's place: its block, its lane of a group and the rows it serves.
template <bool WIDE>
struct Place {
  NodeBlock B;
  int k, G, lane, group, rows;   // rows served by the CTA per step
  long long n, stride;
  __device__ __forceinline__ Place(const NodeDesc& D, const RowMap& M) {
    k = 0;
    while (k + 1 < M.n && (int)blockIdx.x >= M.cta0[k + 1]) ++k;
    B = D.b[M.blk[k]];
    const int lg = M.lg[k];
    G = WIDE ? (int)blockDim.x : 1 << lg;
    lane = WIDE ? (int)threadIdx.x : (int)threadIdx.x & (G - 1);
    group = WIDE ? 0 : (int)threadIdx.x >> lg;
    rows = WIDE ? 1 : kThreads >> lg;
    n = (long long)((int)blockIdx.x - M.cta0[k]) * rows + group;
    stride = (long long)(M.cta0[k + 1] - M.cta0[k]) * rows;
  }
  // whether any lane of the warp has a row left (groups share shuffles)
  __device__ __forceinline__ bool more(long long row, long long N) const {
    return row - (WIDE ? 0 : group - (((int)threadIdx.x & ~31) / G)) < N;
  }
  template <int K>
  __device__ __forceinline__ void sum(float (&v)[K]) const {
    if (WIDE) cta_sum(v);
    else group_sum(v, G);
  }
  __device__ __forceinline__ void sync() const {
    if (WIDE) __syncthreads();
    else __syncwarp();
  }
};

template <class T, int V, int J>
struct Segment {
  Pack<T, V> p[J];
  // packs of a segment at `base` (element 0 of the block in this row); ok: the row exists
  __device__ __forceinline__ void load(const T* base, int lane, int G, int S, bool ok) {
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int s = (j * G + lane) * V;
      if (ok && s < S) p[j] = *reinterpret_cast<const Pack<T, V>*>(base + s);
    }
  }
};

template <class T, int V, int J>
__device__ __forceinline__ void store(T* base, const float (&v)[J * V], int lane, int G, int S, bool ok) {
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int s = (j * G + lane) * V;
    if (!ok || s >= S) continue;
    Pack<T, V> p;
#pragma unroll
    for (int i = 0; i < V; ++i) p.v[i] = from_f32<T>(v[j * V + i]);
    *reinterpret_cast<Pack<T, V>*>(base + s) = p;
  }
}

// Values of a channel vector at a lane's elements (fill beyond the segment is not read).
template <int V, int J>
__device__ __forceinline__ void gather(float (&w)[J * V], const float* vec, const Channels& ch, int lane, int G, int S,
                                       float missing) {
#pragma unroll
  for (int j = 0; j < J; ++j)
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int s = (j * G + lane) * V + i;
      w[j * V + i] = vec && s < S ? vec[ch.of(s)] : missing;
    }
}

// Keep bits of a segment's channel groups (four channels each, one byte per group) in shared
// memory: each group's counter is drawn once, whatever the layout and the number of components.
template <int BYTES>
struct Mask {
  unsigned char* m;   // this group's bytes
  int quads;          // packs lie inside one component and start on a multiple of four channels
  __device__ __forceinline__ Mask(unsigned char* all, int slot, const NodeDesc& D, const NodeBlock& B, int V) {
    m = all + slot * ((B.C + 3) / 4);
    quads = V % 4 == 0 && (B.d == 1 || (!D.mul_ir && B.C % V == 0));
  }
  template <class P>
  __device__ __forceinline__ void draw(const Drop& drop, uint64_t off, const P& at, uint32_t row) {
    at.sync();  // the previous row's readers are done
    const int groups = (at.B.C + 3) / 4;
    for (int g = at.lane; g < groups; g += at.G) {
      const uint4 w = drop_words(drop, off, at.B.grp0 + g, row);
      m[g] = (w.x >= drop.threshold ? 1 : 0) | (w.y >= drop.threshold ? 2 : 0) | (w.z >= drop.threshold ? 4 : 0) |
             (w.w >= drop.threshold ? 8 : 0);
    }
    at.sync();
  }
  // v -> kept ? v * scale : 0
  template <int V, int J>
  __device__ __forceinline__ void apply(float (&v)[J * V], const Drop& drop, const Channels& ch, int lane, int G,
                                        int S) const {
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int s = (j * G + lane) * V;
      if (s >= S) continue;
      if (quads) {
        const int c = ch.of(s) >> 2;
#pragma unroll
        for (int i = 0; i < V; ++i) v[j * V + i] = (m[c + i / 4] >> (i & 3)) & 1 ? __fmul_rn(v[j * V + i], drop.scale) : 0.f;
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const int c = ch.of(s + i);
          v[j * V + i] = (m[c >> 2] >> (c & 3)) & 1 ? __fmul_rn(v[j * V + i], drop.scale) : 0.f;
        }
      }
    }
  }
};

template <int V, int J, bool WIDE>
constexpr int mask_bytes() { return (WIDE ? kWideMax : kThreads) * (V * J) / 4 + kThreads + 4; }

template <class T, int V, int J>
__device__ __forceinline__ void convert(float (&v)[J * V], const Segment<T, V, J>& a, int lane, int G, int S, bool ok) {
#pragma unroll
  for (int j = 0; j < J; ++j)
#pragma unroll
    for (int i = 0; i < V; ++i) v[j * V + i] = ok && (j * G + lane) * V < S ? to_f32(a.p[j].v[i]) : 0.f;
}

// Dropout (DROP) and norm (NORM) of x, either or both; with DROP the sum with the residual is z.
template <class T, int V, int J, bool WIDE, bool DROP, bool NORM>
__global__ void __launch_bounds__(WIDE ? kWideMax : kThreads)
    k_fwd(const __grid_constant__ NodeDesc D, const __grid_constant__ RowMap M, const __grid_constant__ Drop drop,
          const __grid_constant__ NormArgs A, const long long N) {
  constexpr int E = V * J;
  __shared__ unsigned char keep[DROP ? mask_bytes<V, J, WIDE>() : 1];
  const Place<WIDE> at(D, M);
  const NodeBlock& B = at.B;
  const int S = B.S, G = at.G, lane = at.lane;
  const Channels ch(D, B);
  const bool centred = NORM && B.bias0 >= 0;
  const float inv = 1.f / (float)S;
  Mask<mask_bytes<V, J, WIDE>()> mask(keep, at.group, D, B, V);
  const uint64_t off = DROP ? drop_offset(drop) : 0;
  float w[NORM ? E : 1], b[NORM ? E : 1];
  if constexpr (NORM) {
    gather<V, J>(w, A.weight ? A.weight + B.chan0 : nullptr, ch, lane, G, S, 1.f);
    gather<V, J>(b, centred && A.bias ? A.bias + B.bias0 : nullptr, ch, lane, G, S, 0.f);
  }
  const T *x = (const T*)A.x + B.off, *res = DROP && A.residual ? (const T*)A.residual + B.off : nullptr;
  T *y = NORM ? (T*)A.y + B.off : nullptr, *z = DROP ? (T*)A.z + B.off : nullptr;

  Segment<T, V, J> cx, cr;
  long long n = at.n;
  cx.load(x + n * D.dim, lane, G, S, n < N);
  if (DROP && res) cr.load(res + n * D.dim, lane, G, S, n < N);
  for (; at.more(n, N); n += at.stride) {
    const bool ok = n < N;
    float v[E];
    convert(v, cx, lane, G, S, ok);
    if constexpr (DROP) {
      float r[E];
      if (res) convert(r, cr, lane, G, S, ok);
      const long long next = n + at.stride;
      cx.load(x + next * D.dim, lane, G, S, next < N);
      if (res) cr.load(res + next * D.dim, lane, G, S, next < N);
      if (drop.mode == 1) {
        mask.draw(drop, off, at, (uint32_t)n);
        mask.template apply<V, J>(v, drop, ch, lane, G, S);
      } else if (drop.mode == 2) {
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = 0.f;
      }
      if (res) {
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] += r[e];
      }
      store<T, V, J>(z + n * D.dim, v, lane, G, S, ok);
    } else {
      const long long next = n + at.stride;
      cx.load(x + next * D.dim, lane, G, S, next < N);
    }
    if constexpr (NORM) {
      if (centred) {
        float mu[1] = {0.f};
#pragma unroll
        for (int e = 0; e < E; ++e) mu[0] += v[e];
        at.sum(mu);
        mu[0] *= inv;
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = (e / V * G + lane) * V < S ? v[e] - mu[0] : 0.f;
      }
      float q[1] = {0.f};
#pragma unroll
      for (int e = 0; e < E; ++e) q[0] += v[e] * v[e];
      at.sum(q);
      const float r = __frsqrt_rn(q[0] * inv + D.eps);
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] = v[e] * r * w[e] + b[e];
      store<T, V, J>(y + n * D.dim, v, lane, G, S, ok);
    }
  }
}

// Adds the lanes' sums over rows of a CTA and writes them per channel (per element if WIDE).
template <int V, int J, bool WIDE>
__device__ __forceinline__ void write_sums(float (&acc)[J * V], float* smem, float* out, const Place<WIDE>& at,
                                           const Channels& ch) {
  constexpr int E = V * J;
  const int S = at.B.S, G = at.G;
  if constexpr (WIDE) {
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int s = (e / V * G + at.lane) * V + e % V;
      if (s < S) out[s] = acc[e];
    }
  } else {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      if (G <= o) {
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] += __shfl_xor_sync(0xffffffffu, acc[e], o);
      }
    __syncthreads();  // earlier readers of smem are done
    const int warp = threadIdx.x >> 5;
    if (((int)threadIdx.x & 31) < G) {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int s = (e / V * G + at.lane) * V + e % V;
        if (s < S) smem[warp * S + s] = acc[e];
      }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < at.B.C; c += kThreads) {
      float v = 0.f;
      for (int m = 0; m < at.B.d; ++m)
        for (int k = 0; k < kThreads / 32; ++k) v += smem[k * S + ch.at(c, m)];
      out[c] = v;
    }
  }
}

// Where a CTA's weight (or bias) sums go.
__device__ __forceinline__ float* sums_out(const RowMap& M, const NodeBlock& B, int k, int comps, const float* partial,
                                           float* grad, int first, bool bias) {
  if (M.direct) return grad ? grad + first : nullptr;
  if (!partial) return nullptr;
  return const_cast<float*>(partial) + M.part0[k] + ((int)blockIdx.x - M.cta0[k]) * part_stride(B, comps) +
         (bias ? (long long)B.C * comps : 0);
}

template <class T, int V, int J, bool WIDE, bool DROP>
__global__ void __launch_bounds__(WIDE ? kWideMax : kThreads)
    k_bwd(const __grid_constant__ NodeDesc D, const __grid_constant__ RowMap M, const __grid_constant__ Drop drop,
          const __grid_constant__ NormArgs A, const long long N) {
  constexpr int E = V * J;
  __shared__ unsigned char keep[DROP ? mask_bytes<V, J, WIDE>() : 1];
  __shared__ float smem[WIDE ? 1 : kThreads * E];
  const Place<WIDE> at(D, M);
  const NodeBlock& B = at.B;
  const int S = B.S, G = at.G, lane = at.lane;
  const Channels ch(D, B);
  const bool centred = B.bias0 >= 0;
  const float inv = 1.f / (float)S;
  Mask<mask_bytes<V, J, WIDE>()> mask(keep, at.group, D, B, V);
  const uint64_t off = DROP ? drop_offset(drop) : 0;
  float w[E], sw[E], sb[E];
  gather<V, J>(w, A.weight ? A.weight + B.chan0 : nullptr, ch, lane, G, S, 1.f);
#pragma unroll
  for (int e = 0; e < E; ++e) sw[e] = sb[e] = 0.f;
  const T *x = (const T*)A.x + B.off, *gy = (const T*)A.grad_y + B.off;
  const T* gz = DROP && A.grad_z ? (const T*)A.grad_z + B.off : nullptr;
  T *gx = A.grad_x ? (T*)A.grad_x + B.off : nullptr, *gr = DROP && A.grad_residual ? (T*)A.grad_residual + B.off : nullptr;

  Segment<T, V, J> cx, cg, cz;
  long long n = at.n;
  cx.load(x + n * D.dim, lane, G, S, n < N);
  cg.load(gy + n * D.dim, lane, G, S, n < N);
  for (; at.more(n, N); n += at.stride) {
    const bool ok = n < N;
    float u[E], g[E];
    convert(u, cx, lane, G, S, ok);
    convert(g, cg, lane, G, S, ok);
    const long long next = n + at.stride;
    if (DROP && gz) cz.load(gz + n * D.dim, lane, G, S, ok);
    cx.load(x + next * D.dim, lane, G, S, next < N);
    cg.load(gy + next * D.dim, lane, G, S, next < N);
    float ma = 0.f;
    if (centred) {
      float m[2] = {0.f, 0.f};
#pragma unroll
      for (int e = 0; e < E; ++e) {
        m[0] += u[e];
        m[1] += w[e] * g[e];
      }
      at.sum(m);
      const float mu = m[0] * inv;
      ma = m[1] * inv;
#pragma unroll
      for (int e = 0; e < E; ++e) u[e] = (e / V * G + lane) * V < S ? u[e] - mu : 0.f;
    }
    float q[2] = {0.f, 0.f};
#pragma unroll
    for (int e = 0; e < E; ++e) {
      q[0] += u[e] * u[e];
      q[1] += u[e] * (w[e] * g[e] - ma);
    }
    at.sum(q);
    const float r = __frsqrt_rn(q[0] * inv + D.eps), mh = r * q[1] * inv;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float h = u[e] * r;
      sw[e] += g[e] * h;  // a row beyond the last one adds zeros
      sb[e] += g[e];
      u[e] = r * (w[e] * g[e] - ma - h * mh);
    }
    if constexpr (DROP) {
      if (gz) {
        float t[E];
        convert(t, cz, lane, G, S, ok);
#pragma unroll
        for (int e = 0; e < E; ++e) u[e] += t[e];
      }
      if (gr) store<T, V, J>(gr + n * D.dim, u, lane, G, S, ok);
      if (gx && drop.mode == 1) {
        mask.draw(drop, off, at, (uint32_t)n);
        mask.template apply<V, J>(u, drop, ch, lane, G, S);
      } else if (drop.mode == 2) {
#pragma unroll
        for (int e = 0; e < E; ++e) u[e] = 0.f;
      }
    }
    if (gx) store<T, V, J>(gx + n * D.dim, u, lane, G, S, ok);
  }
  const int comps = WIDE ? B.d : 1;
  if (float* out = sums_out(M, B, at.k, comps, A.partial, A.grad_weight, B.chan0, false))
    write_sums<V, J, WIDE>(sw, smem, out, at, ch);
  if (centred)
    if (float* out = sums_out(M, B, at.k, comps, A.partial, A.grad_bias, B.bias0, true))
      write_sums<V, J, WIDE>(sb, smem, out, at, ch);
}

template <class T, int V, int J, bool WIDE>
__global__ void __launch_bounds__(WIDE ? kWideMax : kThreads)
    k_dbl(const __grid_constant__ NodeDesc D, const __grid_constant__ RowMap M, const __grid_constant__ NormArgs A,
          const long long N) {
  constexpr int E = V * J;
  __shared__ float smem[WIDE ? 1 : kThreads * E];
  const Place<WIDE> at(D, M);
  const NodeBlock& B = at.B;
  const int S = B.S, G = at.G, lane = at.lane;
  const Channels ch(D, B);
  const bool centred = B.bias0 >= 0;
  const float inv = 1.f / (float)S;
  float w[E], t[E], sw[E];
  gather<V, J>(w, A.weight ? A.weight + B.chan0 : nullptr, ch, lane, G, S, 1.f);
  gather<V, J>(t, A.gg_weight ? A.gg_weight + B.chan0 : nullptr, ch, lane, G, S, 0.f);
  const float* tb = centred && A.gg_bias ? A.gg_bias + B.bias0 : nullptr;
#pragma unroll
  for (int e = 0; e < E; ++e) sw[e] = 0.f;
  const T *x = (const T*)A.x + B.off, *gy = (const T*)A.grad_y + B.off;
  const T* px = A.gg_x ? (const T*)A.gg_x + B.off : nullptr;
  T *gx = A.grad_x ? (T*)A.grad_x + B.off : nullptr, *gg = A.grad_grad_y ? (T*)A.grad_grad_y + B.off : nullptr;

  Segment<T, V, J> cx, cg, cp;
  long long n = at.n;
  cx.load(x + n * D.dim, lane, G, S, n < N);
  cg.load(gy + n * D.dim, lane, G, S, n < N);
  cp.load(px + n * D.dim, lane, G, S, px && n < N);
  for (; at.more(n, N); n += at.stride) {
    const bool ok = n < N;
    float u[E], g[E], p[E];
    convert(u, cx, lane, G, S, ok);
    convert(g, cg, lane, G, S, ok);
    convert(p, cp, lane, G, S, ok && px);
    const long long next = n + at.stride;
    cx.load(x + next * D.dim, lane, G, S, next < N);
    cg.load(gy + next * D.dim, lane, G, S, next < N);
    cp.load(px + next * D.dim, lane, G, S, px && next < N);
    float ma = 0.f, mw = 0.f;
    if (centred) {
      float m[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int e = 0; e < E; ++e) {
        m[0] += u[e];
        m[1] += p[e];
        m[2] += w[e] * g[e];
        m[3] += t[e] * g[e];
      }
      at.sum(m);
      ma = m[2] * inv;
      mw = m[3] * inv;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const bool in = (e / V * G + lane) * V < S;
        u[e] = in ? u[e] - m[0] * inv : 0.f;
        p[e] = in ? p[e] - m[1] * inv : 0.f;
      }
    }
    float q[5] = {0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float a = w[e] * g[e] - ma;
      q[0] += u[e] * u[e];
      q[1] += u[e] * p[e];
      q[2] += u[e] * a;
      q[3] += p[e] * a;
      q[4] += u[e] * (t[e] * g[e] - mw);
    }
    at.sum(q);
    const float r = __frsqrt_rn(q[0] * inv + D.eps);
    const float P = r * q[1] * inv, Q = r * q[2] * inv, R = q[3] * inv, W = r * q[4] * inv;
    float o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float h = u[e] * r, a = w[e] * g[e] - ma, k = r * (p[e] - h * P);
      sw[e] += g[e] * k;
      o[e] = r * r * (h * (3.f * P * Q - R) - Q * p[e] - P * a) + r * (t[e] * g[e] - mw - h * W);
      const int s = (e / V * G + lane) * V + e % V;
      u[e] = w[e] * k + t[e] * h + (tb && s < S ? tb[s] : 0.f);  // a 0e block's channels are its elements
    }
    if (gx) store<T, V, J>(gx + n * D.dim, o, lane, G, S, ok);
    if (gg) store<T, V, J>(gg + n * D.dim, u, lane, G, S, ok);
  }
  if (float* out = sums_out(M, B, at.k, WIDE ? B.d : 1, A.partial, A.grad_weight, B.chan0, false))
    write_sums<V, J, WIDE>(sw, smem, out, at, ch);
}

// ---- any width: one CTA per segment, read again for each sum; a thread owns whole channels ----

// The CTA's block and rows, as Place.
struct AnyPlace {
  NodeBlock B;
  int k;
  long long n, stride;
  __device__ __forceinline__ AnyPlace(const NodeDesc& D, const RowMap& M) {
    k = 0;
    while (k + 1 < M.n && (int)blockIdx.x >= M.cta0[k + 1]) ++k;
    B = D.b[M.blk[k]];
    n = (int)blockIdx.x - M.cta0[k];
    stride = M.cta0[k + 1] - M.cta0[k];
  }
};

// f(channel, element) over the thread's elements of a block
template <class F>
__device__ __forceinline__ void each(const NodeBlock& B, int mul_ir, F f) {
  for (int c = threadIdx.x; c < B.C; c += kThreads)
    for (int m = 0; m < B.d; ++m) f(c, mul_ir ? c * B.d + m : m * B.C + c);
}

template <class T, bool DROP, bool NORM>
__global__ void __launch_bounds__(kThreads)
    k_fwd_any(const __grid_constant__ NodeDesc D, const __grid_constant__ RowMap M, const __grid_constant__ Drop drop,
              const __grid_constant__ NormArgs A, const long long N) {
  const AnyPlace at(D, M);
  const NodeBlock& B = at.B;
  const bool centred = B.bias0 >= 0;
  const float inv = 1.f / (float)B.S;
  const uint64_t off = DROP ? drop_offset(drop) : 0;
  for (long long n = at.n; n < N; n += at.stride) {
    const long long row = n * D.dim + B.off;
    const T* x = (const T*)A.x + row;
    const T* res = DROP && A.residual ? (const T*)A.residual + row : nullptr;
    auto value = [&](int c, int s) {
      float v = to_f32(x[s]);
      if (DROP) {
        v = drop_one(drop, off, B, c, (uint32_t)n, v);
        if (res) v += to_f32(res[s]);
      }
      return v;
    };
    float mu = 0.f, r = 1.f;
    if constexpr (NORM) {
      if (centred) {
        float m[1] = {0.f};
        each(B, D.mul_ir, [&](int c, int s) { m[0] += value(c, s); });
        cta_sum(m);
        mu = m[0] * inv;
      }
      float q[1] = {0.f};
      each(B, D.mul_ir, [&](int c, int s) {
        const float u = value(c, s) - mu;
        q[0] += u * u;
      });
      cta_sum(q);
      r = __frsqrt_rn(q[0] * inv + D.eps);
    }
    each(B, D.mul_ir, [&](int c, int s) {
      const float v = value(c, s);
      if (DROP) ((T*)A.z)[row + s] = from_f32<T>(v);
      if (NORM)
        ((T*)A.y)[row + s] = from_f32<T>((v - mu) * r * (A.weight ? A.weight[B.chan0 + c] : 1.f) +
                                         (centred && A.bias ? A.bias[B.bias0 + c] : 0.f));
    });
  }
}

template <class T, bool DROP>
__global__ void __launch_bounds__(kThreads)
    k_bwd_any(const __grid_constant__ NodeDesc D, const __grid_constant__ RowMap M, const __grid_constant__ Drop drop,
              const __grid_constant__ NormArgs A, const long long N) {
  const AnyPlace at(D, M);
  const NodeBlock& B = at.B;
  const bool centred = B.bias0 >= 0;
  const float inv = 1.f / (float)B.S;
  const uint64_t off = DROP ? drop_offset(drop) : 0;
  float* pw = sums_out(M, B, at.k, 1, A.partial, A.grad_weight, B.chan0, false);
  float* pb = centred ? sums_out(M, B, at.k, 1, A.partial, A.grad_bias, B.bias0, true) : nullptr;
  for (long long n = at.n; n < N; n += at.stride) {
    const long long row = n * D.dim + B.off;
    const T *x = (const T*)A.x + row, *g = (const T*)A.grad_y + row;
    auto a = [&](int c, int s) { return (A.weight ? A.weight[B.chan0 + c] : 1.f) * to_f32(g[s]); };
    float m[2] = {0.f, 0.f}, q[2] = {0.f, 0.f};
    if (centred) {
      each(B, D.mul_ir, [&](int c, int s) {
        m[0] += to_f32(x[s]);
        m[1] += a(c, s);
      });
      cta_sum(m);
    }
    const float mu = m[0] * inv, ma = m[1] * inv;
    each(B, D.mul_ir, [&](int c, int s) {
      const float u = to_f32(x[s]) - mu;
      q[0] += u * u;
      q[1] += u * (a(c, s) - ma);
    });
    cta_sum(q);
    const float r = __frsqrt_rn(q[0] * inv + D.eps), mh = r * q[1] * inv;
    for (int c = threadIdx.x; c < B.C; c += kThreads) {
      float sw = 0.f, sb = 0.f;
      for (int k = 0; k < B.d; ++k) {
        const int s = D.mul_ir ? c * B.d + k : k * B.C + c;
        const float gv = to_f32(g[s]), h = (to_f32(x[s]) - mu) * r;
        float t = r * (a(c, s) - ma - h * mh);
        sw += gv * h;
        sb += gv;
        if (DROP) {
          if (A.grad_z) t += to_f32(((const T*)A.grad_z)[row + s]);
          if (A.grad_residual) ((T*)A.grad_residual)[row + s] = from_f32<T>(t);
          if (A.grad_x) t = drop_one(drop, off, B, c, (uint32_t)n, t);
        }
        if (A.grad_x) ((T*)A.grad_x)[row + s] = from_f32<T>(t);
      }
      // the CTA's sums so far live in memory; the same thread owns channel c in every row
      const bool first = n == at.n;
      if (pw) pw[c] = first ? sw : pw[c] + sw;
      if (pb) pb[c] = first ? sb : pb[c] + sb;
    }
  }
}

template <class T>
__global__ void __launch_bounds__(kThreads)
    k_dbl_any(const __grid_constant__ NodeDesc D, const __grid_constant__ RowMap M, const __grid_constant__ NormArgs A,
              const long long N) {
  const AnyPlace at(D, M);
  const NodeBlock& B = at.B;
  const bool centred = B.bias0 >= 0;
  const float inv = 1.f / (float)B.S;
  float* pw = sums_out(M, B, at.k, 1, A.partial, A.grad_weight, B.chan0, false);
  auto weight = [&](int c) { return A.weight ? A.weight[B.chan0 + c] : 1.f; };
  auto tangent = [&](int c) { return A.gg_weight ? A.gg_weight[B.chan0 + c] : 0.f; };
  for (long long n = at.n; n < N; n += at.stride) {
    const long long row = n * D.dim + B.off;
    const T *x = (const T*)A.x + row, *g = (const T*)A.grad_y + row;
    auto pv = [&](int s) { return A.gg_x ? to_f32(((const T*)A.gg_x)[row + s]) : 0.f; };
    float m[4] = {0.f, 0.f, 0.f, 0.f}, q[5] = {0.f, 0.f, 0.f, 0.f, 0.f};
    if (centred) {
      each(B, D.mul_ir, [&](int c, int s) {
        const float gv = to_f32(g[s]);
        m[0] += to_f32(x[s]);
        m[1] += pv(s);
        m[2] += weight(c) * gv;
        m[3] += tangent(c) * gv;
      });
      cta_sum(m);
    }
    const float mx = m[0] * inv, mp = m[1] * inv, ma = m[2] * inv, mw = m[3] * inv;
    each(B, D.mul_ir, [&](int c, int s) {
      const float u = to_f32(x[s]) - mx, gv = to_f32(g[s]), p = pv(s) - mp, a = weight(c) * gv - ma;
      q[0] += u * u;
      q[1] += u * p;
      q[2] += u * a;
      q[3] += p * a;
      q[4] += u * (tangent(c) * gv - mw);
    });
    cta_sum(q);
    const float r = __frsqrt_rn(q[0] * inv + D.eps);
    const float P = r * q[1] * inv, Q = r * q[2] * inv, R = q[3] * inv, W = r * q[4] * inv;
    for (int c = threadIdx.x; c < B.C; c += kThreads) {
      const float w = weight(c), t = tangent(c), b = centred && A.gg_bias ? A.gg_bias[B.bias0 + c] : 0.f;
      float sw = 0.f;
      for (int j = 0; j < B.d; ++j) {
        const int s = D.mul_ir ? c * B.d + j : j * B.C + c;
        const float h = (to_f32(x[s]) - mx) * r, gv = to_f32(g[s]), p = pv(s) - mp, a = w * gv - ma;
        const float k = r * (p - h * P);
        sw += gv * k;
        if (A.grad_grad_y) ((T*)A.grad_grad_y)[row + s] = from_f32<T>(w * k + t * h + b);
        if (A.grad_x)
          ((T*)A.grad_x)[row + s] =
              from_f32<T>(r * r * (h * (3.f * P * Q - R) - Q * p - P * a) + r * (t * gv - mw - h * W));
      }
      if (pw) pw[c] = n == at.n ? sw : pw[c] + sw;
    }
  }
}

// ---- sums of the partials over the CTAs, in CTA order: 32 channels x 8 shares of the parts ----

__global__ void __launch_bounds__(256) k_norm_reduce(const __grid_constant__ NodeDesc D, const __grid_constant__ PartMap M,
                                                     const float* __restrict__ partial, float* grad_weight,
                                                     float* grad_bias) {
  __shared__ float share[8][32];
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const int i = blockIdx.x * 32 + tx;
  const bool bias = i >= D.channels;
  const int c = bias ? i - D.channels : i;
  float* out = bias ? grad_bias : grad_weight;
  bool wanted = out && i < D.channels + D.biases;
  float v = 0.f;
  if (wanted) {
    int k = 0;
    for (; k < M.n; ++k) {
      const NodeBlock& B = D.b[M.blk[k]];
      const int first = bias ? B.bias0 : B.chan0;
      if (first >= 0 && c >= first && c < first + B.C) break;
    }
    wanted = k < M.n;  // else the block's only CTA has written the gradient
    if (wanted) {
      const NodeBlock& B = D.b[M.blk[k]];
      const int comps = M.comps[k];
      const long long stride = part_stride(B, comps);
      const float* p = partial + M.part0[k] + (bias ? (long long)B.C * comps : 0);
      const int own = c - (bias ? B.bias0 : B.chan0);
      for (int t = ty; t < M.parts[k]; t += 8)
        for (int m = 0; m < (bias ? 1 : comps); ++m)
          v += p[t * stride + (D.mul_ir ? own * comps + m : m * B.C + own)];
    }
  }
  share[ty][tx] = v;
  __syncthreads();
  if (ty == 0 && wanted) {
    v = 0.f;
#pragma unroll
    for (int t = 0; t < 8; ++t) v += share[t][tx];
    out[c] = v;
  }
}

// ---- launch plan ----

struct Launch {
  Kind kind;
  int J, ctas, threads;
  RowMap M;
};

struct LaunchPlan {
  int V = 1, n = 0;
  Launch l[3];
  PartMap parts{};
  size_t floats = 0;   // partial sums
};

// Elements of one access: 16 bytes where every block starts and ends on that boundary (rows then do,
// too), else pairs of 16-bit values, else single elements.
int pack_width(const NodeDesc& D, int esize) {
  for (int V : {16 / esize, 2, 1}) {
    if (V * esize > 16 || (esize == 4 && V == 2)) continue;
    bool fits = true;
    for (int b = 0; b < D.n_blocks; ++b) fits = fits && D.b[b].S % V == 0;
    if (fits) return V;
  }
  return 1;
}

enum Pass { PASS_FWD = NORM_FORWARD, PASS_BWD = NORM_BACKWARD, PASS_DBL = NORM_DOUBLE_BACKWARD };

// Packs per lane that the kernels are built for (run_width), ascending, ending with 0.
const int* pack_counts(Pass pass, int V) {
  static const int f4[] = {1, 2, 3, 4, 5, 0}, f8[] = {1, 2, 3, 0}, f2[] = {4, 8, 0}, f1[] = {4, 8, 16, 0};
  static const int d4[] = {1, 2, 3, 0}, d8[] = {1, 2, 0}, d2[] = {4, 0}, d1[] = {4, 8, 0};
  if (pass == PASS_DBL) return V == 4 ? d4 : V == 8 ? d8 : V == 2 ? d2 : d1;
  return V == 4 ? f4 : V == 8 ? f8 : V == 2 ? f2 : f1;
}
constexpr int wide_packs(bool dbl, int V) { return (dbl ? 8 : 16) / V; }

int log2_lanes(int S, int per_lane) {
  int lg = 0;
  while ((per_lane << lg) < S) ++lg;
  return lg;
}

LaunchPlan plan_launches(Pass pass, const NodeDesc& D, long long N, int esize) {
  LaunchPlan P;
  P.V = pack_width(D, esize);
  const int* js = pack_counts(pass, P.V);
  int jmax = 0;
  for (const int* j = js; *j; ++j) jmax = *j;
  const int jw = wide_packs(pass == PASS_DBL, P.V);
  Kind kind[MAX_BLOCKS];
  for (int b = 0; b < D.n_blocks; ++b)
    kind[b] = D.b[b].S <= 32 * P.V * jmax ? KIND_GROUP : D.b[b].S <= kWideMax * P.V * jw ? KIND_WIDE : KIND_ANY;
  for (Kind kd : {KIND_GROUP, KIND_WIDE, KIND_ANY}) {
    Launch L{};
    L.kind = kd;
    long long total = 0;
    int widest = 0;
    for (int b = 0; b < D.n_blocks; ++b)
      if (kind[b] == kd) {
        L.M.blk[L.M.n++] = b;
        total += D.b[b].S;
        widest = D.b[b].S > widest ? D.b[b].S : widest;
      }
    if (L.M.n == 0) continue;
    long long resident;   // CTAs that run at a time
    L.threads = kThreads;
    if (kd == KIND_GROUP) {
      // fewest lane-packs per row; a segment's lanes are a power of two
      long long best = -1;
      for (const int* j = js; *j; ++j) {
        if (widest > 32 * P.V * *j) continue;
        long long cost = 0;
        for (int k = 0; k < L.M.n; ++k) cost += (long long)*j << log2_lanes(D.b[L.M.blk[k]].S, P.V * *j);
        if (best < 0 || cost < best) {
          best = cost;
          L.J = *j;
        }
      }
      for (int k = 0; k < L.M.n; ++k) L.M.lg[k] = log2_lanes(D.b[L.M.blk[k]].S, P.V * L.J);
      resident = kSms * (pass == PASS_FWD ? 4 : 2);
    } else if (kd == KIND_WIDE) {
      L.J = jw;
      L.threads = (widest + 32 * P.V * jw - 1) / (32 * P.V * jw) * 32;
      resident = kSms * (kWideMax / L.threads);
    } else {
      resident = pass == PASS_FWD ? kSms * 8 : kAnyParts;
    }
    bool direct = pass != PASS_FWD;
    for (int k = 0; k < L.M.n; ++k) {
      const NodeBlock& B = D.b[L.M.blk[k]];
      const long long rows = kd == KIND_GROUP ? kThreads >> L.M.lg[k] : 1;
      const long long most = (N + rows - 1) / rows;
      long long ctas = resident * B.S / total;
      if (pass != PASS_FWD) {
        if (kd == KIND_ANY && ctas > kAnyFloats / part_stride(B, 1)) ctas = kAnyFloats / part_stride(B, 1);
        if (most <= 8) ctas = 1;
      }
      ctas = ctas < 1 ? 1 : ctas > most ? most : ctas;
      L.M.cta0[k + 1] = L.M.cta0[k] + (int)ctas;
      direct = direct && ctas == 1 && (kd != KIND_WIDE || B.d == 1);  // WIDE sums are per element
    }
    L.ctas = L.M.cta0[L.M.n];
    L.M.direct = direct;
    if (pass != PASS_FWD && !direct)
      for (int k = 0; k < L.M.n; ++k) {
        const NodeBlock& B = D.b[L.M.blk[k]];
        const int i = P.parts.n++, comps = kd == KIND_WIDE ? B.d : 1;
        P.parts.blk[i] = L.M.blk[k];
        P.parts.parts[i] = L.M.cta0[k + 1] - L.M.cta0[k];
        P.parts.comps[i] = comps;
        P.parts.part0[i] = L.M.part0[k] = (long long)P.floats;
        P.floats += (size_t)(P.parts.parts[i] * part_stride(B, comps));
      }
    P.l[P.n++] = L;
  }
  return P;
}

// One pass over the rows.
struct Call {
  Pass pass;
  bool drop, norm;
  const NodeDesc& D;
  const Drop& d;
  const NormArgs& A;
  long long N;
  cudaStream_t s;
};

template <class T, int V, int J, bool WIDE, bool DBL>
void run_packs(const Call& c, const Launch& L) {
  const dim3 grid(L.ctas), block(L.threads);
  if constexpr (DBL) {
    k_dbl<T, V, J, WIDE><<<grid, block, 0, c.s>>>(c.D, L.M, c.A, c.N);
  } else if (c.pass == PASS_FWD) {
    if (c.drop && c.norm) k_fwd<T, V, J, WIDE, true, true><<<grid, block, 0, c.s>>>(c.D, L.M, c.d, c.A, c.N);
    else if (c.drop) k_fwd<T, V, J, WIDE, true, false><<<grid, block, 0, c.s>>>(c.D, L.M, c.d, c.A, c.N);
    else k_fwd<T, V, J, WIDE, false, true><<<grid, block, 0, c.s>>>(c.D, L.M, c.d, c.A, c.N);
  } else {
    if (c.drop) k_bwd<T, V, J, WIDE, true><<<grid, block, 0, c.s>>>(c.D, L.M, c.d, c.A, c.N);
    else k_bwd<T, V, J, WIDE, false><<<grid, block, 0, c.s>>>(c.D, L.M, c.d, c.A, c.N);
  }
}

// the kernel of a launch's pack count, out of pack_counts
template <class T, int V, bool DBL, int... Js>
void run_counts(const Call& c, const Launch& L) {
  ((L.J == Js ? run_packs<T, V, Js, false, DBL>(c, L) : void()), ...);
}

template <class T, int V>
void run_width(const Call& c, const Launch& L) {
  const bool dbl = c.pass == PASS_DBL;
  if (L.kind == KIND_WIDE) {
    if (dbl) run_packs<T, V, wide_packs(true, V), true, true>(c, L);
    else run_packs<T, V, wide_packs(false, V), true, false>(c, L);
  } else if constexpr (V == 4) {
    if (dbl) run_counts<T, V, true, 1, 2, 3>(c, L);
    else run_counts<T, V, false, 1, 2, 3, 4, 5>(c, L);
  } else if constexpr (V == 8) {
    if (dbl) run_counts<T, V, true, 1, 2>(c, L);
    else run_counts<T, V, false, 1, 2, 3>(c, L);
  } else if constexpr (V == 2) {
    if (dbl) run_counts<T, V, true, 4>(c, L);
    else run_counts<T, V, false, 4, 8>(c, L);
  } else {
    if (dbl) run_counts<T, V, true, 4, 8>(c, L);
    else run_counts<T, V, false, 4, 8, 16>(c, L);
  }
}

template <class T>
void run_any(const Call& c, const Launch& L) {
  const dim3 grid(L.ctas), block(kThreads);
  if (c.pass == PASS_FWD) {
    if (c.drop && c.norm) k_fwd_any<T, true, true><<<grid, block, 0, c.s>>>(c.D, L.M, c.d, c.A, c.N);
    else if (c.drop) k_fwd_any<T, true, false><<<grid, block, 0, c.s>>>(c.D, L.M, c.d, c.A, c.N);
    else k_fwd_any<T, false, true><<<grid, block, 0, c.s>>>(c.D, L.M, c.d, c.A, c.N);
  } else if (c.pass == PASS_BWD) {
    if (c.drop) k_bwd_any<T, true><<<grid, block, 0, c.s>>>(c.D, L.M, c.d, c.A, c.N);
    else k_bwd_any<T, false><<<grid, block, 0, c.s>>>(c.D, L.M, c.d, c.A, c.N);
  } else {
    k_dbl_any<T><<<grid, block, 0, c.s>>>(c.D, L.M, c.A, c.N);
  }
}

template <class T>
cudaError_t run_node(const Call& c) {
  const LaunchPlan P = plan_launches(c.pass, c.D, c.N, sizeof(T));
  for (int i = 0; i < P.n; ++i) {
    const Launch& L = P.l[i];
    if (L.kind == KIND_ANY) run_any<T>(c, L);
    else if (P.V == 16 / (int)sizeof(T)) run_width<T, 16 / (int)sizeof(T)>(c, L);
    else if (P.V == 1) run_width<T, 1>(c, L);
    else if constexpr (sizeof(T) == 2) run_width<T, 2>(c, L);
  }
  if (c.A.partial && P.parts.n)
    k_norm_reduce<<<(c.D.channels + c.D.biases + 31) / 32, 256, 0, c.s>>>(c.D, P.parts, c.A.partial, c.A.grad_weight,
                                                                          c.A.grad_bias);
  return cudaGetLastError();
}

}  // namespace

// One build unit per storage type.
#define TPC_NODE_ARGS int pass, bool norm, const NodeDesc &D, long long N, const NormArgs &A, const Drop *drop, cudaStream_t s
cudaError_t run_node_f32(TPC_NODE_ARGS);
cudaError_t run_node_bf16(TPC_NODE_ARGS);
cudaError_t run_node_f16(TPC_NODE_ARGS);

#if TPC_UNIT_T == 0
#define TPC_RUN run_node_f32
#define TPC_T float
#elif TPC_UNIT_T == 1
#define TPC_RUN run_node_bf16
#define TPC_T __nv_bfloat16
#else
#define TPC_RUN run_node_f16
#define TPC_T __half
#endif
cudaError_t TPC_RUN(TPC_NODE_ARGS) {
  const Drop none{};
  return run_node<TPC_T>(Call{(Pass)pass, drop != nullptr, norm, D, drop ? *drop : none, A, N, s});
}

#if TPC_UNIT_T == 0
static cudaError_t run_typed(int dtype, TPC_NODE_ARGS) {
  return dtype == 0   ? run_node_f32(pass, norm, D, N, A, drop, s)
         : dtype == 1 ? run_node_bf16(pass, norm, D, N, A, drop, s)
                      : run_node_f16(pass, norm, D, N, A, drop, s);
}

cudaError_t launch_norm(NormPass pass, int dtype, const NodeDesc& D, long long N, const NormArgs& A, const Drop* drop,
                        cudaStream_t s) {
  return run_typed(dtype, pass, true, D, N, A, drop, s);
}

cudaError_t launch_dropout(int dtype, const NodeDesc& D, long long N, const void* x, const void* residual,
                           const Drop& drop, void* out, cudaStream_t s) {
  NormArgs A{};
  A.x = x;
  A.residual = residual;
  A.z = out;
  return run_typed(dtype, PASS_FWD, false, D, N, A, &drop, s);
}

size_t norm_partial_floats(const NodeDesc& D, long long N, int esize) {
  if (N == 0) return 0;
  const size_t b = plan_launches(PASS_BWD, D, N, esize).floats, d = plan_launches(PASS_DBL, D, N, esize).floats;
  return b > d ? b : d;
}
#endif

}  // namespace tpc
