// Irreps layer norm and dropout on node rows: forward, backward, double backward, and the forward
// and backward fused with dropout and the residual sum (include/tpconv_node.h has the formulas).
//
// Every (row, block) segment of S = (2l+1) C elements is a norm of its own.  The passes are bound
// by HBM traffic (a few flops per byte), in 16 bits nearly as much by instruction issue: each array
// is read once, the statistics are sums over the lanes that hold a segment, and outputs are
// written from the same registers; arithmetic is two float32 values an instruction (f32x2).
//
//  * k_fwd / k_bwd / k_dbl<WIDE = false>: a segment is held by a group of G lanes (a power of two,
//    at most a warp), lane l holding the packs l, l + G, ... of V elements, J packs at most.  A CTA
//    serves one block of the irreps and strides over rows; the blocks share the CTAs in proportion
//    to their sizes, so that all of them walk through the rows at the same pace in one wave.
//    A lane's columns are the same in every row: the sums over rows are per-lane registers until
//    the rows are done, weights are expanded per element in shared memory once.
//  * Rows are copied ahead with cp.async into a ring of shared memory slots that belong to the
//    thread alone (no barriers, no registers held by loads in flight).
//  * WIDE = true: the CTA is the group (segments beyond a warp's registers).
//  * k_*_any: any width, the segment read again from cache for each sum.
//
// Sums over rows (weight and bias gradients) have no atomics: each CTA writes its partial sums to
// the workspace and k_norm_reduce adds them in CTA order; a launch with one CTA per block writes
// the gradients itself.
#include <atomic>

#include "node.cuh"

namespace tpc {
namespace {

constexpr int kThreads = 256;
constexpr int kSms = 148;
constexpr int kWideMax = 512;      // threads of a WIDE CTA
constexpr int kMaxSmem = 231 * 1000;  // dynamic shared memory of a CTA (the rest of 227 KB is static)
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

// ---- pairs of float32 ----

typedef unsigned long long f2;  // two float32, the lower one first

__device__ __forceinline__ f2 pack2(float a, float b) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ f2 both(float a) { return pack2(a, a); }
__device__ __forceinline__ float lo(f2 v) { return __uint_as_float((uint32_t)v); }
__device__ __forceinline__ float hi(f2 v) { return __uint_as_float((uint32_t)(v >> 32)); }
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
  f2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
template <int P>
__device__ __forceinline__ float total(const f2 (&v)[P]) {
  f2 s = v[0];
#pragma unroll
  for (int p = 1; p < P; ++p) s = add2(s, v[p]);
  return lo(s) + hi(s);
}

// Sums of K values over the CTA (any number of warps), to all its threads.
template <int K>
__device__ __forceinline__ void cta_sum(float (&v)[K]) {
  __shared__ float part[32][K];
  group_sum(v, 32);
  __syncthreads();  // the previous call's readers are done
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int k = 0; k < K; ++k) part[threadIdx.x >> 5][k] = v[k];
  __syncthreads();
  const int warps = blockDim.x >> 5;
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = 0.f;
  for (int w = 0; w < warps; ++w)
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] += part[w][k];
}

// ---- segments in registers ----

// A thread's place: its block, its lane of a group and the rows it serves.
template <bool WIDE>
struct Place {
  NodeBlock B;
  int k, G, lane, group;
  int warp_group;                // the group of the warp's first lane
  long long n, stride;
  __device__ __forceinline__ Place(const NodeDesc& D, const RowMap& M) {
    k = 0;
    while (k + 1 < M.n && (int)blockIdx.x >= M.cta0[k + 1]) ++k;
    B = D.b[M.blk[k]];
    const int lg = M.lg[k];
    G = WIDE ? (int)blockDim.x : 1 << lg;
    lane = WIDE ? (int)threadIdx.x : (int)threadIdx.x & (G - 1);
    group = WIDE ? 0 : (int)threadIdx.x >> lg;
    warp_group = WIDE ? 0 : ((int)threadIdx.x & ~31) >> lg;
    const int rows = WIDE ? 1 : kThreads >> lg;
    n = (long long)((int)blockIdx.x - M.cta0[k]) * rows + group;
    stride = (long long)(M.cta0[k + 1] - M.cta0[k]) * rows;
  }
  // whether any group of the warp has a row left (groups share shuffles)
  __device__ __forceinline__ bool more(long long row, long long N) const { return row - (group - warp_group) < N; }
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

template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t to, const void* from, int bytes) {
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(bytes) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(to), "l"(from), "n"(BYTES), "r"(bytes) : "memory");
}

// Slots of the copy ring: enough that a CTA has 16 KB or more on the way (as measured, more gains
// nothing), two at least.
__host__ __device__ constexpr int ring_slots(int esize, int elems, int arrays) {
  const int bytes = arrays * elems * esize * kThreads;
  return bytes >= 16384 ? 2 : bytes >= 8192 ? 3 : 4;
}

// A thread's own packs of A arrays, copied ahead row by row.  Lanes beyond the segment and rows
// beyond the last one read zeros (a copy of no bytes, from an address inside the array).  Packs
// narrower than cp.async's four bytes are loaded when they are wanted.
template <class T, int V, int J, int A>
struct Ring {
  static constexpr int kBytes = V * (int)sizeof(T), kSlots = ring_slots(sizeof(T), V * J, A);
  static constexpr bool kAsync = kBytes >= 4;
  const T* base[A];
  char* mine;                // this thread's pack 0 of slot 0
  int slot_bytes, pack_bytes;
  int S, step, first;        // elements between packs, first element
  long long dim, N, stride, ahead;
  int fill, read;

  __device__ __forceinline__ void start(char* smem, const NodeDesc& D, const NodeBlock& B, int lane, int G,
                                        long long n, long long stride_, long long N_) {
    pack_bytes = kBytes * (int)blockDim.x;
    slot_bytes = A * J * pack_bytes;
    mine = smem + kBytes * threadIdx.x;
    S = B.S;
    first = lane * V;
    step = G * V;
    dim = D.dim;
    N = N_;
    stride = stride_;
    ahead = n;
    fill = read = 0;
    if constexpr (kAsync) {
#pragma unroll
      for (int i = 0; i < kSlots - 1; ++i) issue();
    }
  }
  // copies of the row `ahead` into the next slot
  __device__ __forceinline__ void issue() {
    const bool ok = ahead < N;
    const long long row = (ok ? ahead : N - 1) * dim;
    const uint32_t to = (uint32_t)__cvta_generic_to_shared(mine + fill * slot_bytes);
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int s = first + j * step;
      const bool in = s < S;
#pragma unroll
      for (int a = 0; a < A; ++a)
        if (base[a])
          copy_async<kBytes>(to + (a * J + j) * pack_bytes, base[a] + row + (in ? s : 0), ok && in ? kBytes : 0);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    ahead += stride;
    fill = fill + 1 == kSlots ? 0 : fill + 1;
  }
  // makes the next row readable and starts the copies of a later one
  __device__ __forceinline__ void next() {
    if constexpr (kAsync) {
      issue();
      asm volatile("cp.async.wait_group %0;" ::"n"(kSlots - 1) : "memory");
    }
  }
  // pairs of array a of the current row
  __device__ __forceinline__ void get(int a, f2 (&v)[V * J / 2]) const {
    Pack<T, V> p[J];
#pragma unroll
    for (int j = 0; j < J; ++j) {
      if constexpr (kAsync) {
        p[j] = *reinterpret_cast<const Pack<T, V>*>(mine + read * slot_bytes + (a * J + j) * pack_bytes);
      } else {
        const int s = first + j * step;
#pragma unroll
        for (int i = 0; i < V; ++i) p[j].v[i] = from_f32<T>(0.f);
        if (ahead < N && s < S) p[j] = *reinterpret_cast<const Pack<T, V>*>(base[a] + ahead * dim + s);
      }
    }
#pragma unroll
    for (int e = 0; e < V * J; e += 2)
      v[e / 2] = pack2(to_f32(p[e / V].v[e % V]), to_f32(p[(e + 1) / V].v[(e + 1) % V]));
  }
  __device__ __forceinline__ void done() {
    if constexpr (kAsync) read = read + 1 == kSlots ? 0 : read + 1;
    else ahead += stride;
  }
  __device__ __forceinline__ void finish() const {
    if constexpr (kAsync) asm volatile("cp.async.wait_all;" ::: "memory");
  }
};

template <class T, int V, int J>
__device__ __forceinline__ void store(T* row, const f2 (&v)[V * J / 2], int lane, int G, int S, bool ok) {
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int s = (j * G + lane) * V;
    if (!ok || s >= S) continue;
    Pack<T, V> p;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = j * V + i;
      p.v[i] = from_f32<T>(e % 2 ? hi(v[e / 2]) : lo(v[e / 2]));
    }
    *reinterpret_cast<Pack<T, V>*>(row + s) = p;
  }
}

// A channel vector expanded per element in shared memory (`missing` where there is none).
__device__ __forceinline__ void expand(float* to, const float* vec, const Channels& ch, int S, float missing) {
  for (int s = threadIdx.x; s < S; s += blockDim.x) to[s] = vec ? vec[ch.of(s)] : missing;
}

// Pairs of an expanded vector at a lane's elements (anything beyond the segment).
template <int V, int J>
__device__ __forceinline__ void lookup(f2 (&w)[V * J / 2], const float* vec, int lane, int G, int S) {
#pragma unroll
  for (int j = 0; j < J; ++j) {
    int s = (j * G + lane) * V;
    s = s < S ? s : 0;
    if constexpr (V % 4 == 0) {
#pragma unroll
      for (int i = 0; i < V; i += 4) {
        const float4 q = *reinterpret_cast<const float4*>(vec + s + i);
        w[(j * V + i) / 2] = pack2(q.x, q.y);
        w[(j * V + i) / 2 + 1] = pack2(q.z, q.w);
      }
    } else if constexpr (V == 2) {
      const float2 q = *reinterpret_cast<const float2*>(vec + s);
      w[j] = pack2(q.x, q.y);
    } else {
      const float q = vec[s];
      w[j / 2] = j % 2 ? pack2(lo(w[j / 2]), q) : pack2(q, 0.f);
    }
  }
}

// Keep bits of a segment's channel groups (four channels each, one byte per group) in shared
// memory: each group's counter is drawn once, whatever the layout and the number of components.
template <int V, int J>
struct Mask {
  unsigned char* m;   // this group's bytes
  bool quads;         // packs lie inside one component and start on a multiple of four channels
  uint64_t off;
  __device__ __forceinline__ Mask(unsigned char* all, int slot, const NodeDesc& D, const NodeBlock& B,
                                  const Drop& drop) {
    m = all + slot * ((B.C + 3) / 4);
    quads = V % 4 == 0 && (B.d == 1 || (!D.mul_ir && B.C % V == 0));
    off = drop.mode == 1 ? drop_offset(drop) : 0;
  }
  // keep bits of a lane's elements in a row, lowest first
  template <class P>
  __device__ __forceinline__ uint32_t bits(const Drop& drop, const P& at, const Channels& ch, uint32_t row) {
    if (drop.mode != 1) return drop.mode == 0 ? ~0u : 0u;
    at.sync();  // the previous row's readers are done
    const int groups = (at.B.C + 3) / 4;
    for (int g = at.lane; g < groups; g += at.G) {
      const uint4 w = drop_words(drop, off, at.B.grp0 + g, row);
      m[g] = (w.x >= drop.threshold ? 1 : 0) | (w.y >= drop.threshold ? 2 : 0) | (w.z >= drop.threshold ? 4 : 0) |
             (w.w >= drop.threshold ? 8 : 0);
    }
    at.sync();
    uint32_t keep = 0;
    if (quads) {
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const int s = (j * at.G + at.lane) * V;
        const int c = s < at.B.S ? ch.of(s) >> 2 : 0;
#pragma unroll
        for (int i = 0; i < V / 4; ++i) keep |= (uint32_t)m[c + i] << (j * V + 4 * i);
      }
    } else {
#pragma unroll 1
      for (int j = 0; j < J; ++j) {
        const int s = (j * at.G + at.lane) * V;
        if (s >= at.B.S) break;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const int c = ch.of(s + i);
          keep |= ((uint32_t)m[c >> 2] >> (c & 3) & 1u) << (j * V + i);
        }
      }
    }
    return keep;
  }
};

// v -> kept ? v * scale : 0
template <int P>
__device__ __forceinline__ void apply_mask(f2 (&v)[P], uint32_t keep, float scale) {
  const f2 q = both(scale);
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const f2 t = mul2(v[p], q);
    v[p] = pack2(keep >> (2 * p) & 1 ? lo(t) : 0.f, keep >> (2 * p + 1) & 1 ? hi(t) : 0.f);
  }
}

// v + m at the lane's elements inside the segment (the others hold zeros)
template <int V, int J>
__device__ __forceinline__ void shift(f2 (&v)[V * J / 2], float m, int lane, int G, int S) {
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const float t = (j * G + lane) * V < S ? m : 0.f;
    if constexpr (V == 1) {
      v[j / 2] = j % 2 ? pack2(lo(v[j / 2]), hi(v[j / 2]) + t) : pack2(lo(v[j / 2]) + t, hi(v[j / 2]));
    } else {
#pragma unroll
      for (int i = 0; i < V; i += 2) v[(j * V + i) / 2] = add2(v[(j * V + i) / 2], both(t));
    }
  }
}

// Shared memory of a CTA: the ring (after the rows: the sums over them), then vectors expanded per
// element, then keep bits.
__host__ __device__ constexpr int rows_bytes(int esize, int V, int elems, int arrays, bool sums, int threads) {
  const int ring = V * esize < 4 ? 0 : ring_slots(esize, elems, arrays) * arrays * elems * esize * threads;
  const int acc = sums ? threads * elems * 4 : 0;
  return ring > acc ? ring : acc;
}
__host__ __device__ constexpr int vector_bytes(int S) { return (S + 3) / 4 * 16; }
constexpr int mask_bytes(int elems, int threads) { return threads * elems / 4 + threads + 4; }

extern __shared__ __align__(16) char g_smem[];

// Dropout (DROP) and norm (NORM) of x, either or both; with DROP the sum with the residual is z.
template <class T, int V, int J, bool WIDE, bool DROP, bool NORM>
__global__ void __launch_bounds__(WIDE ? kWideMax : kThreads, WIDE ? 1 : 2)
    k_fwd(const __grid_constant__ NodeDesc D, const __grid_constant__ RowMap M, const __grid_constant__ Drop drop,
          const __grid_constant__ NormArgs A, const long long N) {
  constexpr int P = V * J / 2, R = DROP ? 2 : 1;
  const Place<WIDE> at(D, M);
  const NodeBlock& B = at.B;
  const int S = B.S, G = at.G, lane = at.lane;
  const Channels ch(D, B);
  const bool centred = NORM && B.bias0 >= 0;
  const float inv = 1.f / (float)S;
  float* sw = reinterpret_cast<float*>(g_smem + rows_bytes(sizeof(T), V, V * J, R, false, blockDim.x));
  float* sb = sw + (S + 3) / 4 * 4;
  unsigned char* bytes = reinterpret_cast<unsigned char*>(sw + (NORM ? 2 * ((S + 3) / 4 * 4) : 0));
  Ring<T, V, J, R> ring;
  ring.base[0] = (const T*)A.x + B.off;
  if constexpr (DROP) ring.base[R - 1] = A.residual ? (const T*)A.residual + B.off : nullptr;
  ring.start(g_smem, D, B, lane, G, at.n, at.stride, N);
  if constexpr (NORM) {
    expand(sw, A.weight ? A.weight + B.chan0 : nullptr, ch, S, 1.f);
    expand(sb, centred && A.bias ? A.bias + B.bias0 : nullptr, ch, S, 0.f);
    __syncthreads();
  }
  Mask<V, J> mask(bytes, at.group, D, B, drop);
  const bool res = DROP && A.residual;
  T *y = NORM ? (T*)A.y + B.off : nullptr, *z = DROP ? (T*)A.z + B.off : nullptr;
  for (long long n = at.n; at.more(n, N); n += at.stride) {
    const bool ok = n < N;
    ring.next();
    f2 v[P];
    ring.get(0, v);
    if constexpr (DROP) {
      apply_mask(v, mask.bits(drop, at, ch, (uint32_t)n), drop.scale);
      if (res) {
        f2 r[P];
        ring.get(R - 1, r);
#pragma unroll
        for (int p = 0; p < P; ++p) v[p] = add2(v[p], r[p]);
      }
      store<T, V, J>(z + n * D.dim, v, lane, G, S, ok);
    }
    if constexpr (NORM) {
      if (centred) {
        float mu[1] = {total(v)};
        at.sum(mu);
        shift<V, J>(v, -mu[0] * inv, lane, G, S);
      }
      f2 q2[P];
#pragma unroll
      for (int p = 0; p < P; ++p) q2[p] = mul2(v[p], v[p]);
      float q[1] = {total(q2)};
      at.sum(q);
      const f2 r = both(__frsqrt_rn(q[0] * inv + D.eps));
      f2 w[P], b[P];
      lookup<V, J>(w, sw, lane, G, S);
      lookup<V, J>(b, sb, lane, G, S);
#pragma unroll
      for (int p = 0; p < P; ++p) v[p] = fma2(mul2(v[p], r), w[p], b[p]);
      store<T, V, J>(y + n * D.dim, v, lane, G, S, ok);
    }
    ring.done();
  }
  ring.finish();
}

// Adds the lanes' sums over rows of a CTA and writes them per channel (per element if WIDE).
template <int V, int J, bool WIDE>
__device__ __forceinline__ void write_sums(const f2 (&sums)[V * J / 2], float* smem, float* out,
                                           const Place<WIDE>& at, const Channels& ch) {
  constexpr int E = V * J;
  const int S = at.B.S, G = at.G;
  if constexpr (WIDE) {
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int s = (e / V * G + at.lane) * V + e % V;
      if (s < S) out[s] = e % 2 ? hi(sums[e / 2]) : lo(sums[e / 2]);
    }
  } else {
    float acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = e % 2 ? hi(sums[e / 2]) : lo(sums[e / 2]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      if (G <= o) {
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] += __shfl_xor_sync(0xffffffffu, acc[e], o);
      }
    __syncthreads();  // the ring, or earlier sums, have been read
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
#pragma unroll
        for (int k = 0; k < kThreads / 32; ++k) v += smem[k * S + ch.at(c, m)];
      out[c] = v;
    }
  }
}

// Where a CTA's weight (or bias) sums go.
__device__ __forceinline__ float* sums_out(const RowMap& M, const NodeBlock& B, int k, int comps, float* partial,
                                           float* grad, int first, bool bias) {
  if (M.direct) return grad ? grad + first : nullptr;
  if (!partial) return nullptr;
  return partial + M.part0[k] + ((int)blockIdx.x - M.cta0[k]) * part_stride(B, comps) +
         (bias ? (long long)B.C * comps : 0);
}

template <class T, int V, int J, bool WIDE, bool DROP>
__global__ void __launch_bounds__(WIDE ? kWideMax : kThreads, WIDE ? 1 : 2)
    k_bwd(const __grid_constant__ NodeDesc D, const __grid_constant__ RowMap M, const __grid_constant__ Drop drop,
          const __grid_constant__ NormArgs A, const long long N) {
  constexpr int P = V * J / 2, R = DROP ? 3 : 2;
  const Place<WIDE> at(D, M);
  const NodeBlock& B = at.B;
  const int S = B.S, G = at.G, lane = at.lane;
  const Channels ch(D, B);
  const bool centred = B.bias0 >= 0;
  const float inv = 1.f / (float)S;
  float* ws = reinterpret_cast<float*>(g_smem + rows_bytes(sizeof(T), V, V * J, R, !WIDE, blockDim.x));
  unsigned char* bytes = reinterpret_cast<unsigned char*>(ws + (S + 3) / 4 * 4);
  Ring<T, V, J, R> ring;
  ring.base[0] = (const T*)A.x + B.off;
  ring.base[1] = (const T*)A.grad_y + B.off;
  if constexpr (DROP) ring.base[R - 1] = A.grad_z ? (const T*)A.grad_z + B.off : nullptr;
  ring.start(g_smem, D, B, lane, G, at.n, at.stride, N);
  expand(ws, A.weight ? A.weight + B.chan0 : nullptr, ch, S, 1.f);
  __syncthreads();
  Mask<V, J> mask(bytes, at.group, D, B, drop);
  f2 sw[P], sb[P];
#pragma unroll
  for (int p = 0; p < P; ++p) sw[p] = sb[p] = 0;
  const bool gz = DROP && A.grad_z;
  T *gx = A.grad_x ? (T*)A.grad_x + B.off : nullptr, *gr = DROP && A.grad_residual ? (T*)A.grad_residual + B.off : nullptr;
  for (long long n = at.n; at.more(n, N); n += at.stride) {
    const bool ok = n < N;
    ring.next();
    f2 u[P], a[P];
    ring.get(0, u);
    {
      f2 w[P];
      ring.get(1, a);
      lookup<V, J>(w, ws, lane, G, S);
#pragma unroll
      for (int p = 0; p < P; ++p) {
        sb[p] = add2(sb[p], a[p]);
        a[p] = mul2(a[p], w[p]);
      }
    }
    if (centred) {
      float m[2] = {total(u), total(a)};
      at.sum(m);
      shift<V, J>(u, -m[0] * inv, lane, G, S);
      shift<V, J>(a, -m[1] * inv, lane, G, S);
    }
    f2 q0 = mul2(u[0], u[0]), q1 = mul2(u[0], a[0]);
#pragma unroll
    for (int p = 1; p < P; ++p) {
      q0 = fma2(u[p], u[p], q0);
      q1 = fma2(u[p], a[p], q1);
    }
    float q[2] = {lo(q0) + hi(q0), lo(q1) + hi(q1)};
    at.sum(q);
    const float r = __frsqrt_rn(q[0] * inv + D.eps);
    {
      f2 g[P];
      ring.get(1, g);   // read again instead of held: the registers carry the sums
      const f2 r2 = both(r), mh = both(-(r * q[1] * inv));
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const f2 h = mul2(u[p], r2);
        sw[p] = fma2(g[p], h, sw[p]);
        u[p] = mul2(r2, fma2(h, mh, a[p]));
      }
    }
    if constexpr (DROP) {
      if (gz) {
        f2 t[P];
        ring.get(R - 1, t);
#pragma unroll
        for (int p = 0; p < P; ++p) u[p] = add2(u[p], t[p]);
      }
      if (gr) store<T, V, J>(gr + n * D.dim, u, lane, G, S, ok);
      if (gx) apply_mask(u, mask.bits(drop, at, ch, (uint32_t)n), drop.scale);
    }
    if (gx) store<T, V, J>(gx + n * D.dim, u, lane, G, S, ok);
    ring.done();
  }
  ring.finish();
  const int comps = WIDE ? B.d : 1;
  float* smem = reinterpret_cast<float*>(g_smem);
  if (float* out = sums_out(M, B, at.k, comps, A.partial, A.grad_weight, B.chan0, false))
    write_sums<V, J, WIDE>(sw, smem, out, at, ch);
  if (centred)
    if (float* out = sums_out(M, B, at.k, comps, A.partial, A.grad_bias, B.bias0, true))
      write_sums<V, J, WIDE>(sb, smem, out, at, ch);
}

template <class T, int V, int J, bool WIDE>
__global__ void __launch_bounds__(WIDE ? kWideMax : kThreads, WIDE ? 1 : 2)
    k_dbl(const __grid_constant__ NodeDesc D, const __grid_constant__ RowMap M, const __grid_constant__ NormArgs A,
          const long long N) {
  constexpr int P = V * J / 2;
  const Place<WIDE> at(D, M);
  const NodeBlock& B = at.B;
  const int S = B.S, G = at.G, lane = at.lane, S4 = (S + 3) / 4 * 4;
  const Channels ch(D, B);
  const bool centred = B.bias0 >= 0;
  const float inv = 1.f / (float)S;
  float* ws = reinterpret_cast<float*>(g_smem + rows_bytes(sizeof(T), V, V * J, 3, !WIDE, blockDim.x));
  float *ts = ws + S4, *bs = ts + S4;
  Ring<T, V, J, 3> ring;
  ring.base[0] = (const T*)A.x + B.off;
  ring.base[1] = (const T*)A.grad_y + B.off;
  ring.base[2] = A.gg_x ? (const T*)A.gg_x + B.off : nullptr;
  ring.start(g_smem, D, B, lane, G, at.n, at.stride, N);
  expand(ws, A.weight ? A.weight + B.chan0 : nullptr, ch, S, 1.f);
  expand(ts, A.gg_weight ? A.gg_weight + B.chan0 : nullptr, ch, S, 0.f);
  expand(bs, centred && A.gg_bias ? A.gg_bias + B.bias0 : nullptr, ch, S, 0.f);
  __syncthreads();
  f2 sw[P];
#pragma unroll
  for (int p = 0; p < P; ++p) sw[p] = 0;
  T *gx = A.grad_x ? (T*)A.grad_x + B.off : nullptr, *gg = A.grad_grad_y ? (T*)A.grad_grad_y + B.off : nullptr;
  for (long long n = at.n; at.more(n, N); n += at.stride) {
    const bool ok = n < N;
    ring.next();
    // u, p, a = weight g, e = gg_weight g; less their means in a 0e block
    f2 u[P], pt[P], a[P], e[P], w[P], t[P];
    ring.get(0, u);
    if (A.gg_x) {
      ring.get(2, pt);
    } else {
#pragma unroll
      for (int p = 0; p < P; ++p) pt[p] = 0;
    }
    ring.get(1, a);
    lookup<V, J>(w, ws, lane, G, S);
    lookup<V, J>(t, ts, lane, G, S);
#pragma unroll
    for (int p = 0; p < P; ++p) {
      e[p] = mul2(a[p], t[p]);
      a[p] = mul2(a[p], w[p]);
    }
    if (centred) {
      float m[4] = {total(u), total(pt), total(a), total(e)};
      at.sum(m);
      shift<V, J>(u, -m[0] * inv, lane, G, S);
      shift<V, J>(pt, -m[1] * inv, lane, G, S);
      shift<V, J>(a, -m[2] * inv, lane, G, S);
      shift<V, J>(e, -m[3] * inv, lane, G, S);
    }
    f2 q2[5];
#pragma unroll
    for (int k = 0; k < 5; ++k) q2[k] = 0;
#pragma unroll
    for (int p = 0; p < P; ++p) {
      q2[0] = fma2(u[p], u[p], q2[0]);
      q2[1] = fma2(u[p], pt[p], q2[1]);
      q2[2] = fma2(u[p], a[p], q2[2]);
      q2[3] = fma2(pt[p], a[p], q2[3]);
      q2[4] = fma2(u[p], e[p], q2[4]);
    }
    float q[5];
#pragma unroll
    for (int k = 0; k < 5; ++k) q[k] = lo(q2[k]) + hi(q2[k]);
    at.sum(q);
    const float r = __frsqrt_rn(q[0] * inv + D.eps);
    const float mp = r * q[1] * inv, ma = r * q[2] * inv, mpa = q[3] * inv, me = r * q[4] * inv;
    // grad_x = h (r^2 (3 mp ma - mpa) - r me) - r^2 ma p - r^2 mp a + r e,  k = r (p - h mp)
    const f2 r2 = both(r), ch_ = both(r * r * (3.f * mp * ma - mpa) - r * me), cp = both(-(r * r * ma)),
             ca = both(-(r * r * mp)), nmp = both(-mp);
    f2 g[P], b[P];
    ring.get(1, g);
    lookup<V, J>(w, ws, lane, G, S);
    lookup<V, J>(t, ts, lane, G, S);
    lookup<V, J>(b, bs, lane, G, S);
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const f2 h = mul2(u[p], r2), k = mul2(r2, fma2(h, nmp, pt[p]));
      sw[p] = fma2(g[p], k, sw[p]);
      u[p] = fma2(h, ch_, fma2(cp, pt[p], fma2(ca, a[p], mul2(r2, e[p]))));
      e[p] = fma2(w[p], k, fma2(t[p], h, b[p]));
    }
    if (gx) store<T, V, J>(gx + n * D.dim, u, lane, G, S, ok);
    if (gg) store<T, V, J>(gg + n * D.dim, e, lane, G, S, ok);
    ring.done();
  }
  ring.finish();
  if (float* out = sums_out(M, B, at.k, WIDE ? B.d : 1, A.partial, A.grad_weight, B.chan0, false))
    write_sums<V, J, WIDE>(sw, reinterpret_cast<float*>(g_smem), out, at, ch);
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

// ---- sums of the partials over the CTAs: 32 channels x 32 shares of the parts, each share and then
// the shares in order ----

constexpr int kShares = 32;

__global__ void __launch_bounds__(32 * kShares)
    k_norm_reduce(const __grid_constant__ NodeDesc D, const __grid_constant__ PartMap M,
                  const float* __restrict__ partial, float* grad_weight, float* grad_bias) {
  __shared__ float share[kShares][33];
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
      const int comps = bias ? 1 : M.comps[k], parts = M.parts[k];
      const long long stride = part_stride(B, M.comps[k]);
      const float* p = partial + M.part0[k] + (bias ? (long long)B.C * M.comps[k] : 0);
      const int own = c - (bias ? B.bias0 : B.chan0);
      for (int m = 0; m < comps; ++m) {
        const float* q = p + (D.mul_ir ? own * comps + m : m * B.C + own);
#pragma unroll 4
        for (int t = ty; t < parts; t += kShares) v += q[t * stride];
      }
    }
  }
  share[ty][tx] = v;
  __syncthreads();
  // warp ty adds channel ty's shares
  v = share[tx][ty];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (tx == 0) share[0][ty] = v;  // column ty: read by this warp alone, before
  __syncthreads();
  if (ty == 0 && wanted) out[c] = share[0][tx];
}

// ---- launch plan ----

struct Launch {
  Kind kind;
  int J, ctas, threads, smem;
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

// Dynamic shared memory of a CTA whose widest segment has S elements.
int smem_bytes(Pass pass, bool drop, bool norm, int esize, int V, int J, int threads, bool wide, int S) {
  const int arrays = pass == PASS_FWD ? (drop ? 2 : 1) : pass == PASS_BWD ? (drop ? 3 : 2) : 3;
  const int vectors = pass == PASS_FWD ? (norm ? 2 : 0) : pass == PASS_BWD ? 1 : 3;
  return rows_bytes(esize, V, V * J, arrays, pass != PASS_FWD && !wide, threads) + vectors * vector_bytes(S) +
         (drop ? mask_bytes(V * J, threads) : 0);
}

// CTAs that an SM holds: by registers (launch bounds; more where the kernels use fewer) and by
// shared memory (227 KB, 1 KB of it per CTA for the system).
int ctas_per_sm(int by_registers, int smem) {
  const int by_smem = 232448 / (smem + 1024 + 512);
  return by_smem < 1 ? 1 : by_smem < by_registers ? by_smem : by_registers;
}

LaunchPlan plan_launches(Pass pass, bool drop, bool norm, const NodeDesc& D, long long N, int esize) {
  LaunchPlan P;
  P.V = pack_width(D, esize);
  const int* js = pack_counts(pass, P.V);
  int jmax = 0;
  for (const int* j = js; *j; ++j) jmax = *j;
  const int jw = wide_packs(pass == PASS_DBL, P.V);
  Kind kind[MAX_BLOCKS];
  const auto wide_threads = [&](int S) { return (S + 32 * P.V * jw - 1) / (32 * P.V * jw) * 32; };
  const auto wide_smem = [&](int S) { return smem_bytes(pass, drop, norm, esize, P.V, jw, wide_threads(S), true, S); };
  for (int b = 0; b < D.n_blocks; ++b) {
    const int S = D.b[b].S;
    kind[b] = S <= 32 * P.V * jmax                                           ? KIND_GROUP
              : S <= kWideMax * P.V * jw && wide_smem(S) <= kMaxSmem ? KIND_WIDE
                                                                             : KIND_ANY;
  }
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
        if (best < 0 || cost <= best) {
          best = cost;
          L.J = *j;
        }
      }
      for (int k = 0; k < L.M.n; ++k) L.M.lg[k] = log2_lanes(D.b[L.M.blk[k]].S, P.V * L.J);
      L.smem = smem_bytes(pass, drop, norm, esize, P.V, L.J, L.threads, false, widest);
      resident = kSms * ctas_per_sm(pass == PASS_FWD ? 4 : 2, L.smem);
    } else if (kd == KIND_WIDE) {
      L.J = jw;
      L.threads = wide_threads(widest);
      L.smem = wide_smem(widest);
      resident = kSms * ctas_per_sm(kWideMax / L.threads, L.smem);
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

// Launches one kernel.  Dynamic shared memory beyond 48 KB has to be allowed once per kernel and
// device (not a stream operation, so a capture may do it).
template <class... Ps, class... As>
void launch(void (*kernel)(Ps...), std::atomic<uint64_t>& allowed, const Call& c, const Launch& L, const As&... args) {
  if (L.smem > 44 * 1024) {  // static shared memory counts, too
    int dev = 0;
    cudaGetDevice(&dev);
    const uint64_t bit = 1ull << (dev & 63);
    if (dev > 63 || !(allowed.load(std::memory_order_acquire) & bit)) {
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
      allowed.fetch_or(bit, std::memory_order_release);
    }
  }
  kernel<<<L.ctas, L.threads, L.smem, c.s>>>(args...);
}

template <class T, int V, int J, bool WIDE, bool DBL>
void run_packs(const Call& c, const Launch& L) {
  static std::atomic<uint64_t> ok[5];  // devices, by kernel
  if constexpr (DBL) {
    launch(k_dbl<T, V, J, WIDE>, ok[0], c, L, c.D, L.M, c.A, c.N);
  } else if (c.pass == PASS_FWD) {
    if (c.drop && c.norm) launch(k_fwd<T, V, J, WIDE, true, true>, ok[0], c, L, c.D, L.M, c.d, c.A, c.N);
    else if (c.drop) launch(k_fwd<T, V, J, WIDE, true, false>, ok[1], c, L, c.D, L.M, c.d, c.A, c.N);
    else launch(k_fwd<T, V, J, WIDE, false, true>, ok[2], c, L, c.D, L.M, c.d, c.A, c.N);
  } else {
    if (c.drop) launch(k_bwd<T, V, J, WIDE, true>, ok[3], c, L, c.D, L.M, c.d, c.A, c.N);
    else launch(k_bwd<T, V, J, WIDE, false>, ok[4], c, L, c.D, L.M, c.d, c.A, c.N);
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
  const LaunchPlan P = plan_launches(c.pass, c.drop, c.norm, c.D, c.N, sizeof(T));
  for (int i = 0; i < P.n; ++i) {
    const Launch& L = P.l[i];
    if (L.kind == KIND_ANY) run_any<T>(c, L);
    else if (P.V == 16 / (int)sizeof(T)) run_width<T, 16 / (int)sizeof(T)>(c, L);
    else if (P.V == 1) run_width<T, 1>(c, L);
    else if constexpr (sizeof(T) == 2) run_width<T, 2>(c, L);
  }
  if (c.A.partial && P.parts.n)
    k_norm_reduce<<<(c.D.channels + c.D.biases + 31) / 32, 32 * kShares, 0, c.s>>>(c.D, P.parts, c.A.partial, c.A.grad_weight,
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
  size_t most = 0;
  for (const LaunchPlan& P :
       {plan_launches(PASS_BWD, false, true, D, N, esize), plan_launches(PASS_BWD, true, true, D, N, esize),
        plan_launches(PASS_DBL, false, true, D, N, esize)})
    most = P.floats > most ? P.floats : most;
  return most;
}
#endif

}  // namespace tpc
