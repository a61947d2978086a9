// Irreps layer norm and dropout on node rows: forward, backward, double backward, and the forward
// and backward fused with dropout and the residual sum (include/tpconv_node.h has the formulas).
//
// Every (row, block) segment of S = (2l+1) C elements is a norm of its own.  The passes are bound
// by HBM traffic (a few flops per byte), in 16 bits nearly as much by instruction issue: each array
// is read once, the statistics are sums over the lanes that hold a segment, and outputs are
// written from the same registers; arithmetic is two float32 values an instruction (f32x2).
//
//  * k_fwd / k_bwd / k_dbl: a segment is held by a group of G lanes (a power of two, up to the
//    CTA), lane l holding the 16-byte packs l, l + G, ..., J packs at most.  A CTA serves one block
//    of the irreps and strides over rows; the blocks share one wave of CTAs so that all make about
//    the same number of steps.  A lane's columns are the same in every row: the sums over rows are
//    per-lane registers until the rows are done, weights are expanded per element in shared memory
//    once.
//  * Rows are copied ahead with cp.async into a ring of shared memory slots that belong to the
//    thread alone (no barriers, no registers held by loads in flight).
//  * EDGE = true: rows or blocks that start off a 16-byte boundary.  A CTA serves the rows n of one
//    residue class (n mod R), in which a block has one offset from the boundary, so packs stay
//    aligned and columns stay fixed; the first and last pack of a segment hold neighbours'
//    elements, which are masked and not written.
//  * k_*_any: segments beyond a CTA's registers, read again from cache for each sum.
//
// Sums over rows (weight and bias gradients) have no atomics: each CTA writes its partial sums to
// the workspace and k_norm_reduce adds them in CTA order; a launch with one CTA per block writes
// the gradients itself.
//
// Launches are programmatic: a kernel may start while the one before it in the stream drains, and
// waits for that one's end (cudaGridDependencySynchronize) before it touches memory.  Measured times
// are of inputs larger than L2, on a B200.
#include <algorithm>
#include <atomic>

#include "node.cuh"
#include "prof.h"

namespace tpc {
namespace {

constexpr int kThreads = 256;
constexpr int kWide = 512;         // threads of a CTA for the widest segments
constexpr int kSms = 148;
constexpr int kMostSums = 5;       // sums over a segment taken together
constexpr int kDropCtas = 4;       // CTAs per SM of k_drop
constexpr int kMaxSmem = 231 * 1000;  // dynamic shared memory of a CTA (the rest of 227 KB is static)
constexpr int kAnyParts = 296;     // row ranges of the any-width kernels
constexpr int kAnyFloats = 1 << 22;  // bound on their partial sums

// Blocks served by one launch: CTAs [cta0[k], cta0[k + 1]) serve block blk[k].
struct RowMap {
  int n;
  int classes;                     // residue classes of rows (R), 1 unless EDGE
  int direct;                      // one CTA per block: sums go to the gradients themselves
  int blk[MAX_BLOCKS];
  int cta0[MAX_BLOCKS + 1];
  int lg[MAX_BLOCKS];              // log2 of the group's lanes
  long long part0[MAX_BLOCKS];     // first float of the block's partial sums
};

// The partial sums of one block: `parts` rows of channel sums (weight, then bias of a 0e block).
struct PartMap {
  int n;
  int blk[MAX_BLOCKS];
  int parts[MAX_BLOCKS];
  long long part0[MAX_BLOCKS];
};

__host__ __device__ inline long long part_stride(const NodeBlock& B) { return (long long)B.C * (B.bias0 >= 0 ? 2 : 1); }

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
  f2 s[P];
#pragma unroll
  for (int p = 0; p < P; ++p) s[p] = v[p];
#pragma unroll
  for (int n = P; n > 1; n = (n + 1) / 2)
#pragma unroll
    for (int p = 0; p < n / 2; ++p) s[p] = add2(s[p], s[n - 1 - p]);
  return lo(s[0]) + hi(s[0]);
}

// Sums of K values over W (a power of two) consecutive warps, to all their threads, by way of
// part[2][warps of the CTA][each] in shared memory: calls alternate between the two halves, and none
// can be two calls ahead of another warp, so one barrier a call is enough.  A warp's place does not
// depend on K: other groups of the CTA may be at a call with another K.  (Values folded over the lanes
// for half the shuffles, and the warps' sums read as vectors, took longer: 4096x0e bf16 68 us, 60 us.)
template <int K, class Sync>
__device__ __forceinline__ void warps_sum(float (&v)[K], float* part, int each, int warps, int& flip, int first, int W,
                                          Sync sync) {
  group_sum(v, 32);
  float* to = part + flip * warps * each;
  flip ^= 1;
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int k = 0; k < K; ++k) to[(threadIdx.x >> 5) * each + k] = v[k];
  sync();
  const int w = first + ((int)threadIdx.x & (W - 1));
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = to[w * each + k];
  group_sum(v, W);
}

// ---- segments in registers ----

// A thread's place: its block, its lane of a group and the rows it serves.
template <int TH, bool EDGE>
struct Place {
  NodeBlock B;
  int k, lg, G, lane, group;
  int shift;                     // EDGE: elements between the 16-byte boundary and the segment
  uint32_t n, stride, warp_rows; // warp_rows: the thread's row minus that of the warp's first lane
  uint32_t step;                 // elements between a lane's packs
  float* part;                   // exchange between the warps of a group
  mutable int flip;
  __device__ __forceinline__ Place(const NodeDesc& D, const RowMap& M, int V, float* part_) : part(part_), flip(0) {
    k = 0;
    while (k + 1 < M.n && (int)blockIdx.x >= M.cta0[k + 1]) ++k;
    B = D.b[M.blk[k]];
    lg = M.lg[k];
    G = 1 << lg;
    lane = (int)threadIdx.x & (G - 1);
    group = (int)threadIdx.x >> lg;
    step = G * V;
    const uint32_t rows = TH >> lg, cta = blockIdx.x - M.cta0[k], ctas = M.cta0[k + 1] - M.cta0[k];
    const uint32_t R = EDGE ? M.classes : 1, cls = EDGE ? cta % R : 0;
    n = R * (cta / R * rows + group) + cls;
    stride = ctas * rows;
    warp_rows = G < 32 ? R * (((int)threadIdx.x & 31) >> lg) : 0;
    shift = EDGE ? (int)(((long long)cls * D.dim + B.off) % V) : 0;
  }
  // whether any group of the warp has a row left (groups share shuffles)
  __device__ __forceinline__ bool more(uint32_t row, uint32_t N) const { return row - warp_rows < N; }
  __device__ __forceinline__ void sync() const {
    if (G <= 32) __syncwarp();
    else asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(G) : "memory");
  }
  template <int K>
  __device__ __forceinline__ void sum(float (&v)[K]) const {
    if (G <= 32) {
      group_sum(v, G);
    } else {
      const int W = G >> 5;
      warps_sum(v, part, kMostSums, TH / 32, flip, ((int)threadIdx.x >> 5) & ~(W - 1), W, [&] { sync(); });
    }
  }
  // element of a lane's pack j (negative or >= S: not in the segment)
  template <int V>
  __device__ __forceinline__ int elem(int j) const { return (j * G + lane) * V - shift; }
};

// Slots of the copy ring: the row that is computed, and as many rows on the way as make up 12 KB or more
// for 256 threads in float32 (forward 50000 x 592: 41 us, 47 us with 24 KB or more), 24 KB in 16 bits,
// where a row is half as long and takes as many instructions (the same in bf16: 31 us with one row ahead,
// 26 us with 12 KB, 25 us with 24 KB).  One row on the way at least, which for three arrays of four packs
// is 48 KB; CTAs of 512 threads have twice as much on the way.
__host__ __device__ constexpr int ring_slots(int esize, int pack_bytes) {
  return ((esize == 4 ? 12288 : 24576) + pack_bytes * kThreads - 1) / (pack_bytes * kThreads) + 1;
}

// A thread's own packs of A arrays, copied ahead row by row.  Packs beyond the segment hold zeros
// from the start; slots of rows beyond the last one hold anything (such rows are computed, by
// groups that share a warp with others, but neither stored nor summed).
template <class T, int J, int A, int TH, bool EDGE>
struct Ring {
  static constexpr int V = 16 / sizeof(T), kSlots = ring_slots(sizeof(T), 16 * A * J);
  static constexpr int kPack = 16 * TH, kSlot = A * J * kPack;
  const char* p[A];          // this lane's pack 0 in the row `ahead`; NULL: no such array
  uint32_t mine, fill, read; // shared addresses: slot 0, next slot to fill, current slot
  uint32_t ahead, N, stride;
  uint32_t inside;           // bit j: pack j has elements of the segment
  long long row_step;
  uint32_t pack_step;        // bytes between a lane's packs
  long long left;            // EDGE: bytes from p[] to the end of the arrays

  __device__ __forceinline__ void start(char* smem, const NodeDesc& D, const Place<TH, EDGE>& at, uint32_t N_,
                                        const void* const (&arrays)[A]) {
    mine = fill = read = (uint32_t)__cvta_generic_to_shared(smem) + 16 * threadIdx.x;
    ahead = at.n;
    N = N_;
    stride = at.stride;
    const long long first = (long long)ahead * D.dim + at.B.off + at.template elem<V>(0);
    row_step = (long long)stride * D.dim * (int)sizeof(T);
    pack_step = at.step * (uint32_t)sizeof(T);
    left = ((long long)N * D.dim - first) * (int)sizeof(T);
#pragma unroll
    for (int a = 0; a < A; ++a) p[a] = arrays[a] ? (const char*)arrays[a] + first * (int)sizeof(T) : nullptr;
    inside = 0;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      if (at.template elem<V>(j) < at.B.S) {
        inside |= 1u << j;
      } else {
#pragma unroll
        for (int i = 0; i < kSlots * A; ++i)
          *reinterpret_cast<uint4*>(smem + 16 * threadIdx.x + (i * J + j) * kPack) = make_uint4(0, 0, 0, 0);
      }
    }
#pragma unroll
    for (int i = 0; i < kSlots - 1; ++i) issue();
  }
  // copies of the row `ahead` into the next slot
  __device__ __forceinline__ void issue() {
    if (ahead < N) {
#pragma unroll
      for (int a = 0; a < A; ++a) {
        if (!p[a]) continue;
#pragma unroll
        for (int j = 0; j < J; ++j) {
          if (!(inside >> j & 1)) continue;
          const char* from = p[a] + j * pack_step;
          int bytes = 16;  // the arrays' last pack may be cut short
          if (EDGE && left - j * pack_step < 16) bytes = (int)(left - j * pack_step);
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(fill + (a * J + j) * kPack), "l"(from),
                       "r"(bytes)
                       : "memory");
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    ahead += stride;
    left -= row_step;
#pragma unroll
    for (int a = 0; a < A; ++a)
      if (p[a]) p[a] += row_step;
    fill = fill == mine + (kSlots - 1) * kSlot ? mine : fill + kSlot;
  }
  // makes the next row readable and starts the copies of a later one
  __device__ __forceinline__ void next() {
    issue();
    asm volatile("cp.async.wait_group %0;" ::"n"(kSlots - 1) : "memory");
  }
  // pack j of array a of the current row
  __device__ __forceinline__ uint4 word(int a, int j) const {
    uint4 w;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
                 : "r"(read + (a * J + j) * kPack)
                 : "memory");
    return w;
  }
  __device__ __forceinline__ void done() { read = read == mine + (kSlots - 1) * kSlot ? mine : read + kSlot; }
  __device__ __forceinline__ void finish() const { asm volatile("cp.async.wait_all;" ::: "memory"); }
};

// Pairs of array a of the current row.  EDGE: `inner` masks the words of the packs to the elements
// of the segment.
template <class T, int J, bool EDGE>
struct Inner {
  static constexpr int V = 16 / sizeof(T);
  uint4 m[EDGE ? J : 1];
  __device__ __forceinline__ explicit Inner(uint32_t valid) {
    if constexpr (EDGE) {
#pragma unroll
      for (int j = 0; j < J; ++j) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if constexpr (sizeof(T) == 4) w[i] = valid >> (j * V + i) & 1 ? ~0u : 0u;
          else w[i] = (valid >> (j * V + 2 * i) & 1 ? 0xffffu : 0u) | (valid >> (j * V + 2 * i + 1) & 1 ? 0xffff0000u : 0u);
        }
        m[j] = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
  }
  template <class Source>
  __device__ __forceinline__ void get(const Source& rows, int a, f2 (&v)[V * J / 2]) const {
#pragma unroll
    for (int j = 0; j < J; ++j) {
      uint4 q = rows.word(a, j);
      if constexpr (EDGE) {
        q.x &= m[j].x;
        q.y &= m[j].y;
        q.z &= m[j].z;
        q.w &= m[j].w;
      }
      const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int i = 0; i < V; i += 2) {
        float x, y;
        if constexpr (sizeof(T) == 4) {
          x = __uint_as_float(w[i]);
          y = __uint_as_float(w[i + 1]);
        } else {
          unpack<T>(w[i / 2], x, y);
        }
        v[(j * V + i) / 2] = pack2(x, y);
      }
    }
  }
};

// A thread's packs of an output, row by row.
template <class T, int J, int TH, bool EDGE>
struct Out {
  static constexpr int V = 16 / sizeof(T);
  char* p;                   // this lane's pack 0 in the current row; NULL: not wanted
  long long row_step;
  uint32_t pack_step;
  __device__ __forceinline__ Out(void* array, const NodeDesc& D, const Place<TH, EDGE>& at) {
    const long long first = (long long)at.n * D.dim + at.B.off + at.template elem<V>(0);
    p = array ? (char*)array + first * (int)sizeof(T) : nullptr;
    row_step = (long long)at.stride * D.dim * (int)sizeof(T);
    pack_step = at.step * (uint32_t)sizeof(T);
  }
  __device__ __forceinline__ explicit operator bool() const { return p != nullptr; }
  __device__ __forceinline__ void put(const f2 (&v)[V * J / 2], uint32_t valid) const {
#pragma unroll
    for (int j = 0; j < J; ++j) {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < V; i += 2) {
        const f2 q = v[(j * V + i) / 2];
        if constexpr (sizeof(T) == 4) {
          w[i] = __float_as_uint(lo(q));
          w[i + 1] = __float_as_uint(hi(q));
        } else {
          w[i / 2] = pack<T>(lo(q), hi(q));
        }
      }
      const uint32_t all = (1u << V) - 1, bits = valid >> (j * V) & all;
      if (EDGE ? bits == all : bits != 0) {
        *reinterpret_cast<uint4*>(p + j * pack_step) = make_uint4(w[0], w[1], w[2], w[3]);
      } else if (EDGE && bits) {
        // a cut pack in the widest pieces that it has (single elements: twice the time, 50000 x 145 f16)
        char* to = p + j * pack_step;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t half = (1u << (V / 2)) - 1, bh = bits >> (h * (V / 2)) & half;
          if (bh == half) {
            *reinterpret_cast<uint2*>(to + 8 * h) = make_uint2(w[2 * h], w[2 * h + 1]);
            continue;
          }
#pragma unroll
          for (int q = 2 * h; q < 2 * h + 2; ++q) {
            if constexpr (sizeof(T) == 4) {
              if (bits >> q & 1) reinterpret_cast<uint32_t*>(to)[q] = w[q];
            } else {
              const uint32_t bq = bits >> (2 * q) & 3u;
              if (bq == 3u) reinterpret_cast<uint32_t*>(to)[q] = w[q];
              else if (bq == 1u) reinterpret_cast<uint16_t*>(to)[2 * q] = (uint16_t)w[q];
              else if (bq == 2u) reinterpret_cast<uint16_t*>(to)[2 * q + 1] = (uint16_t)(w[q] >> 16);
            }
          }
        }
      }
    }
  }
  __device__ __forceinline__ void next() {
    if (p) p += row_step;
  }
};

// Bits of the lane's elements that belong to the segment, lowest first.
template <int V, int J, class P>
__device__ __forceinline__ uint32_t valid_bits(const P& at) {
  uint32_t bits = 0;
#pragma unroll
  for (int j = 0; j < J; ++j)
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int s = at.template elem<V>(j) + i;
      if (s >= 0 && s < at.B.S) bits |= 1u << (j * V + i);
    }
  return bits;
}

// K channel vectors expanded per element in shared memory, one behind the other, element s at [shift +
// s] of n (`missing` where there is no vector, zeros outside the segment).  All loads of a batch are on
// the way together: this is a CTA's first wait for memory.
template <int K>
__device__ __forceinline__ void expand(float* to, int n, const float* const (&vec)[K], const float (&missing)[K],
                                       const Channels& ch, int S, int shift) {
  if (ch.d == 1 && shift == 0 && S % 4 == 0) {  // channels are elements: four at a time
    bool aligned = true;
#pragma unroll
    for (int k = 0; k < K; ++k) aligned = aligned && (reinterpret_cast<uintptr_t>(vec[k]) & 15u) == 0;
    if (aligned) {
      for (int i = 4 * threadIdx.x; i < n; i += 4 * blockDim.x)
#pragma unroll
        for (int k = 0; k < K; ++k) {
          float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
          if (i < S)
            v = vec[k] ? *reinterpret_cast<const float4*>(vec[k] + i)
                       : make_float4(missing[k], missing[k], missing[k], missing[k]);
          *reinterpret_cast<float4*>(to + k * n + i) = v;
        }
      return;
    }
  }
  constexpr int U = 16 / K;
  for (int i0 = threadIdx.x; i0 < n; i0 += U * blockDim.x) {
    float v[U][K];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int s = i0 + u * (int)blockDim.x - shift;
      const bool in = s >= 0 && s < S;
      const int c = in ? ch.of(s) : 0;
#pragma unroll
      for (int k = 0; k < K; ++k) v[u][k] = !in ? 0.f : vec[k] ? vec[k][c] : missing[k];
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (i0 + u * (int)blockDim.x < n) to[k * n + i0 + u * blockDim.x] = v[u][k];
  }
}

// A parameter vector from a block's first channel on.
__device__ __forceinline__ const float* from_channel(const float* v, int first) {
  return v && first >= 0 ? v + first : nullptr;
}

// Pairs of an expanded vector at a lane's elements.
template <int V, int J, class P>
__device__ __forceinline__ void lookup(f2 (&w)[V * J / 2], const float* vec, const P& at) {
#pragma unroll
  for (int j = 0; j < J; ++j)
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      const int s = (j * at.G + at.lane) * V + i;
      const float4 q = *reinterpret_cast<const float4*>(vec + s);
      w[(j * V + i) / 2] = pack2(q.x, q.y);
      w[(j * V + i) / 2 + 1] = pack2(q.z, q.w);
    }
}

// What is kept of a segment's channels, in shared memory: each group of four channels is drawn once,
// whatever the layout and the number of components.  Where packs lie inside one component and start
// on a multiple of four channels, a byte holds a group's four bits; else a byte stands for a channel,
// and the lanes know the channels of their elements.
template <int V, int J>
struct Mask {
  unsigned char* m;   // this group's bytes
  bool quads;
  uint64_t off;
  uint32_t of[J * V / 2];  // channels of the lane's elements, two per word (quads: of the packs)
  template <class P>
  __device__ __forceinline__ Mask(unsigned char* all, const P& at, const NodeDesc& D, const Drop& drop,
                                  const Channels& ch, uint32_t valid) {
    m = all + at.group * ((at.B.C + 3) / 4 * 4);
    quads = at.shift == 0 && (at.B.d == 1 || (!D.mul_ir && at.B.C % V == 0));
    off = drop.mode == 1 ? drop_offset(drop) : 0;
#pragma unroll
    for (int e = 0; e < J * V; e += 2) {
      uint32_t c[2];
#pragma unroll
      for (int i = 0; i < 2; ++i)
        c[i] = valid >> (e + i) & 1 ? ch.of(at.template elem<V>((e + i) / V) + (e + i) % V) : 0;
      of[e / 2] = c[0] | c[1] << 16;
    }
  }
  // keep bits of a lane's elements in a row, lowest first
  template <class P>
  __device__ __forceinline__ uint32_t bits(const Drop& drop, const P& at, uint32_t row) {
    if (drop.mode != 1) return drop.mode == 0 ? ~0u : 0u;
    at.sync();  // the previous row's readers are done
    const int groups = (at.B.C + 3) / 4;
    for (int g = at.lane; g < groups; g += at.G) {
      const uint4 w = drop_words(drop, off, at.B.grp0 + g, row);
      const uint32_t k0 = w.x >= drop.threshold, k1 = w.y >= drop.threshold, k2 = w.z >= drop.threshold,
                     k3 = w.w >= drop.threshold;
      if (quads) m[g] = (unsigned char)(k0 | k1 << 1 | k2 << 2 | k3 << 3);
      else *reinterpret_cast<uint32_t*>(m + 4 * g) = k0 | k1 << 8 | k2 << 16 | k3 << 24;
    }
    at.sync();
    uint32_t keep = 0;
    if (quads) {
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const uint32_t g = (of[j * V / 2] & 0xffffu) >> 2;
        // a cut last pack reads bytes of groups that are not there: its bits are not used
#pragma unroll
        for (int i = 0; i < V / 4; ++i) keep |= (uint32_t)m[g + i] << (j * V + 4 * i);
      }
    } else {
#pragma unroll
      for (int e = 0; e < J * V; ++e)
        keep |= (uint32_t)m[e % 2 ? of[e / 2] >> 16 : of[e / 2] & 0xffffu] << e;
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

// Whether the sum of squares about the mean, taken as a difference (sum of squares less mean times
// sum), has to be taken again around the mean: the difference is exact to a few 2^-24 of itself while
// the mean is at most twice the spread (and the sum of products with a to a few 2^-24 of |a|, which
// the product in a has lost already).  Also where it is no number, and where `raw`, the sums that the
// differences are taken of, has left float32's range: about the mean they may be within it (0 * raw is no
// number then; as a test of its own: forward 4096x0e bf16 29.2 us).  All warps of a group have read the
// same values and added them in the same order, so all take the same way (and meet at its barrier).
__device__ __forceinline__ bool sums_again(float raw, float mu, float S, float q) {
  return !(mu * mu * S <= fmaf(4.f, q, 0.f * raw));
}

// v + m at the lane's elements inside the segment (the others hold zeros)
template <int V, int J, bool EDGE>
__device__ __forceinline__ void shift_by(f2 (&v)[V * J / 2], float m, uint32_t valid) {
#pragma unroll
  for (int j = 0; j < J; ++j) {
    if constexpr (EDGE) {
#pragma unroll
      for (int i = 0; i < V; i += 2)
        v[(j * V + i) / 2] = add2(v[(j * V + i) / 2], pack2(valid >> (j * V + i) & 1 ? m : 0.f,
                                                            valid >> (j * V + i + 1) & 1 ? m : 0.f));
    } else {
      const f2 t = both(valid >> (j * V) & 1 ? m : 0.f);
#pragma unroll
      for (int i = 0; i < V; i += 2) v[(j * V + i) / 2] = add2(v[(j * V + i) / 2], t);
    }
  }
}

// Shared memory of a CTA: the ring (after the rows: the sums over them), vectors expanded per
// element, the exchange between warps, keep bits.
__host__ __device__ constexpr int rows_bytes(int elems, int arrays, int packs, bool sums, int threads) {
  const int ring = ring_slots(16 / (elems / packs), 16 * arrays * packs) * 16 * arrays * packs * threads, acc = sums ? threads * elems * 4 : 0;
  return ring > acc ? ring : acc;
}
// a vector's elements as far as any lane reads them
__host__ __device__ constexpr int vector_bytes(int elems, int lg) { return (elems << lg) * 4; }
constexpr int kPartBytes = 2 * (kWide / 32) * kMostSums * 4;
constexpr int mask_bytes(int elems, int threads) { return threads * elems + 4 * threads; }

extern __shared__ __align__(16) char g_smem[];

enum Pass { PASS_FWD = NORM_FORWARD, PASS_BWD = NORM_BACKWARD, PASS_DBL = NORM_DOUBLE_BACKWARD };

// CTAs of 256 threads that an SM is to hold (a bound on the registers).
// (Three in the forward up to 8 elements, two else: more are not faster, the backward's of 8
// elements are slower by 5 to 15 %.)
constexpr int min_ctas(Pass pass, int elems) { return pass == PASS_FWD && elems <= 8 ? 3 : 2; }

#define TPC_NODE_KERNEL(TH, PASS, ELEMS) \
  __global__ void __launch_bounds__(TH, (TH) == kThreads ? min_ctas(PASS, ELEMS) : 1)

// Dropout (DROP) and norm (NORM) of x, either or both; with DROP the sum with the residual is z.
template <class T, int J, int TH, bool EDGE, bool DROP, bool NORM>
TPC_NODE_KERNEL(TH, PASS_FWD, 16 / sizeof(T) * J)
    k_fwd(const __grid_constant__ NodeDesc D, const __grid_constant__ RowMap M, const __grid_constant__ Drop drop,
          const __grid_constant__ NormArgs A, const uint32_t N) {
  constexpr int V = 16 / sizeof(T), E = V * J, P = E / 2, R = DROP ? 2 : 1;
  float* part = reinterpret_cast<float*>(g_smem + rows_bytes(E, R, J, false, TH));
  const Place<TH, EDGE> at(D, M, V, part);
  const NodeBlock& B = at.B;
  const Channels ch(D, B);
  const bool centred = NORM && B.bias0 >= 0;
  const float inv = 1.f / (float)B.S;
  float* sw = reinterpret_cast<float*>(reinterpret_cast<char*>(part) + kPartBytes);
  float* sb = sw + (E << at.lg);
  Ring<T, J, R, TH, EDGE> rows;
  cudaGridDependencySynchronize();  // nothing before this reads what an earlier kernel may write
  if constexpr (DROP) rows.start(g_smem, D, at, N, {A.x, A.residual});
  else rows.start(g_smem, D, at, N, {A.x});
  if constexpr (NORM) {
    expand<2>(sw, E << at.lg, {from_channel(A.weight, B.chan0), from_channel(A.bias, B.bias0)}, {1.f, 0.f}, ch, B.S,
              at.shift);
    __syncthreads();
  }
  const uint32_t valid = valid_bits<V, J>(at);
  Mask<V, J> mask(reinterpret_cast<unsigned char*>(NORM ? sb + (E << at.lg) : sw), at, D, drop, ch, valid);
  const Inner<T, J, EDGE> inner(valid);
  Out<T, J, TH, EDGE> y(NORM ? A.y : nullptr, D, at), z(DROP ? A.z : nullptr, D, at);
  f2 w[NORM ? P : 1], b[NORM ? P : 1];
  if constexpr (NORM) {
    lookup<V, J>(w, sw, at);
    lookup<V, J>(b, sb, at);
  }
  for (uint32_t n = at.n; at.more(n, N); n += at.stride) {
    const bool ok = n < N;
    rows.next();
    f2 v[P];
    inner.get(rows, 0, v);
    if constexpr (DROP) {
      apply_mask(v, mask.bits(drop, at, n), drop.scale);
      if (A.residual) {
        f2 r[P];
        inner.get(rows, R - 1, r);
#pragma unroll
        for (int p = 0; p < P; ++p) v[p] = add2(v[p], r[p]);
      }
      if (ok) z.put(v, valid);
      z.next();
    }
    if constexpr (NORM) {
      float q[1];
      bool second = true;
      if (centred) {
        float mu;
        if (at.G > 32) {  // one exchange between the warps instead of two: see k_bwd
          f2 vv = mul2(v[0], v[0]);
#pragma unroll
          for (int p = 1; p < P; ++p) vv = fma2(v[p], v[p], vv);
          float m[2] = {total(v), lo(vv) + hi(vv)};
          at.sum(m);
          mu = m[0] * inv;
          q[0] = m[1] - m[0] * mu;
          second = sums_again(m[1], mu, (float)B.S, q[0]);
        } else {
          float m[1] = {total(v)};
          at.sum(m);
          mu = m[0] * inv;
        }
        shift_by<V, J, EDGE>(v, -mu, valid);
      }
      if (second) {
        f2 q2 = mul2(v[0], v[0]);
#pragma unroll
        for (int p = 1; p < P; ++p) q2 = fma2(v[p], v[p], q2);
        q[0] = lo(q2) + hi(q2);
        at.sum(q);
      }
      const f2 r = both(rsqrtf(q[0] * inv + D.eps));
#pragma unroll
      for (int p = 0; p < P; ++p) v[p] = fma2(mul2(v[p], r), w[p], b[p]);
      if (ok) y.put(v, valid);
      y.next();
    }
    rows.done();
  }
  rows.finish();
  cudaTriggerProgrammaticLaunchCompletion();
}

// Adds the lanes' sums over rows of a CTA and writes them per channel.  Short code: it runs once, and
// is waited for as it is fetched (12,700 cycles with shuffles unrolled over the elements, 4096x0e).
template <int V, int J, int TH, bool EDGE>
__device__ __forceinline__ void write_sums(const f2 (&sums)[V * J / 2], float* smem, float* out,
                                           const Place<TH, EDGE>& at, const Channels& ch) {
  constexpr int E = V * J;
  const int lanes_e = E << at.lg, copies = TH >> at.lg;  // a group's elements, groups
  __syncthreads();  // the ring, or earlier sums, have been read
#pragma unroll
  for (int j = 0; j < J; ++j)
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      const f2 a = sums[(j * V + i) / 2], b = sums[(j * V + i) / 2 + 1];
      *reinterpret_cast<float4*>(smem + at.group * lanes_e + (j * at.G + at.lane) * V + i) =
          make_float4(lo(a), hi(a), lo(b), hi(b));
    }
  __syncthreads();
  if (at.B.d == 1 && at.shift == 0 && at.B.C % 4 == 0 && (reinterpret_cast<uintptr_t>(out) & 15u) == 0) {
    for (int c = 4 * threadIdx.x; c < at.B.C; c += 4 * TH) {  // channels are elements: four at a time
      float4 v = *reinterpret_cast<const float4*>(smem + c);
#pragma unroll 4
      for (int k = 1; k < copies; ++k) {
        const float4 q = *reinterpret_cast<const float4*>(smem + k * lanes_e + c);
        v = make_float4(v.x + q.x, v.y + q.y, v.z + q.z, v.w + q.w);
      }
      *reinterpret_cast<float4*>(out + c) = v;
    }
    return;
  }
  if (copies > 1) {
    for (int i = threadIdx.x; i < lanes_e; i += TH) {
      float v = 0.f;
#pragma unroll 8
      for (int k = 0; k < copies; ++k) v += smem[k * lanes_e + i];
      smem[i] = v;  // copy 0: read by this thread alone
    }
    __syncthreads();
  }
#pragma unroll 1
  for (int c = threadIdx.x; c < at.B.C; c += TH) {
    float v = 0.f;
    for (int m = 0; m < at.B.d; ++m) v += smem[at.shift + ch.at(c, m)];
    out[c] = v;
  }
}

// Where a CTA's weight (or bias) sums go.
__device__ __forceinline__ float* sums_out(const RowMap& M, const NodeBlock& B, int k, float* partial, float* grad,
                                           int first, bool bias) {
  if (M.direct) return grad ? grad + first : nullptr;
  if (!partial) return nullptr;
  return partial + M.part0[k] + ((int)blockIdx.x - M.cta0[k]) * part_stride(B) + (bias ? B.C : 0);
}

template <class T, int J, int TH, bool EDGE, bool DROP>
TPC_NODE_KERNEL(TH, PASS_BWD, 16 / sizeof(T) * J)
    k_bwd(const __grid_constant__ NodeDesc D, const __grid_constant__ RowMap M, const __grid_constant__ Drop drop,
          const __grid_constant__ NormArgs A, const uint32_t N) {
  constexpr int V = 16 / sizeof(T), E = V * J, P = E / 2, R = DROP ? 3 : 2;
  float* part = reinterpret_cast<float*>(g_smem + rows_bytes(E, R, J, true, TH));
  const Place<TH, EDGE> at(D, M, V, part);
  const NodeBlock& B = at.B;
  const Channels ch(D, B);
  const bool centred = B.bias0 >= 0;
  const float inv = 1.f / (float)B.S;
  float* ws = reinterpret_cast<float*>(reinterpret_cast<char*>(part) + kPartBytes);
  Ring<T, J, R, TH, EDGE> rows;
  cudaGridDependencySynchronize();
  if constexpr (DROP) rows.start(g_smem, D, at, N, {A.x, A.grad_y, A.grad_z});
  else rows.start(g_smem, D, at, N, {A.x, A.grad_y});
  expand<1>(ws, E << at.lg, {from_channel(A.weight, B.chan0)}, {1.f}, ch, B.S, at.shift);
  __syncthreads();
  const uint32_t valid = valid_bits<V, J>(at);
  Mask<V, J> mask(reinterpret_cast<unsigned char*>(ws + (E << at.lg)), at, D, drop, ch, valid);
  const Inner<T, J, EDGE> inner(valid);
  constexpr bool HOLD = E <= 8;  // as the registers allow (16 elements spill: 4096x0e bf16 74 us, 69 us without)
  f2 w[P], sw[P], sb[P];
  if constexpr (HOLD) lookup<V, J>(w, ws, at);
#pragma unroll
  for (int p = 0; p < P; ++p) sw[p] = sb[p] = 0;
  Out<T, J, TH, EDGE> gx(A.grad_x, D, at), gr(DROP ? A.grad_residual : nullptr, D, at);
  float* const sums_w = sums_out(M, B, at.k, A.partial, A.grad_weight, B.chan0, false);
  float* const sums_b = centred ? sums_out(M, B, at.k, A.partial, A.grad_bias, B.bias0, true) : nullptr;
  for (uint32_t n = at.n; at.more(n, N); n += at.stride) {
    const bool ok = n < N;
    rows.next();
    // HOLD: grad_y and the weights stay in registers; else their product, and grad_y is read again
    f2 u[P], a[P];
    inner.get(rows, 0, u);
    inner.get(rows, 1, a);
    if (centred && ok) {
#pragma unroll
      for (int p = 0; p < P; ++p) sb[p] = add2(sb[p], a[p]);
    }
    if constexpr (!HOLD) {
      lookup<V, J>(w, ws, at);
#pragma unroll
      for (int p = 0; p < P; ++p) a[p] = mul2(w[p], a[p]);
    }
    const auto product = [&](int p) { return HOLD ? mul2(w[p], a[p]) : a[p]; };  // weight grad_y
    float ma = 0.f, q[2];
    bool second = true;
    if (centred) {
      // Groups of several warps wait for one another in a sum: theirs has the second moments as well
      // (4096x0e bf16: 54 us, 57 us with two sums; forward 29 us, 33 us).
      const bool once = at.G > 32;
      f2 t[P], uu = mul2(u[0], u[0]), ut = mul2(u[0], product(0));
#pragma unroll
      for (int p = 0; p < P; ++p) t[p] = product(p);
      float mu;
      if (once) {
#pragma unroll
        for (int p = 1; p < P; ++p) {
          uu = fma2(u[p], u[p], uu);
          ut = fma2(u[p], t[p], ut);
        }
        float m[4] = {total(u), total(t), lo(uu) + hi(uu), lo(ut) + hi(ut)};
        at.sum(m);
        mu = m[0] * inv;
        ma = m[1] * inv;
        q[0] = m[2] - m[0] * mu;
        q[1] = m[3] - m[1] * mu;
        second = sums_again(m[2] + m[3], mu, (float)B.S, q[0]);
      } else {
        float m[2] = {total(u), total(t)};
        at.sum(m);
        mu = m[0] * inv;
        ma = m[1] * inv;
      }
      shift_by<V, J, EDGE>(u, -mu, valid);
    }
    if (second) {
      // mean(a) would drop out of mean(a h) in a 0e block if h had no mean, but u keeps the rounding of mu:
      // with a less its mean, neither counts (means of 1000 in both, spreads of 1: grad_x to 3e-3, 0.2
      // with mean(a) left in)
      const f2 nma = both(-ma);
      const auto rest = [&](int p) { return HOLD ? fma2(w[p], a[p], nma) : add2(a[p], nma); };
      f2 q0 = mul2(u[0], u[0]), q1 = mul2(u[0], rest(0));
#pragma unroll
      for (int p = 1; p < P; ++p) {
        q0 = fma2(u[p], u[p], q0);
        q1 = fma2(u[p], rest(p), q1);
      }
      q[0] = lo(q0) + hi(q0);
      q[1] = lo(q1) + hi(q1);
      at.sum(q);
    }
    const float r = rsqrtf(q[0] * inv + D.eps);
    {
      f2 g[P];
      if constexpr (!HOLD) inner.get(rows, 1, g);
      const f2 r2 = both(r), mh = both(-(r * r * q[1] * inv)), c0 = both(-(r * ma));
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const f2 h = mul2(u[p], r2);
        if (ok) sw[p] = fma2(HOLD ? a[p] : g[p], h, sw[p]);
        u[p] = fma2(h, mh, fma2(product(p), r2, c0));
      }
    }
    if constexpr (DROP) {
      if (A.grad_z) {
        f2 t[P];
        inner.get(rows, R - 1, t);
#pragma unroll
        for (int p = 0; p < P; ++p) u[p] = add2(u[p], t[p]);
      }
      if (gr && ok) gr.put(u, valid);
      gr.next();
      if (gx) apply_mask(u, mask.bits(drop, at, n), drop.scale);
    }
    if (gx && ok) gx.put(u, valid);
    gx.next();
    rows.done();
  }
  rows.finish();
  cudaTriggerProgrammaticLaunchCompletion();
  float* smem = reinterpret_cast<float*>(g_smem);
  if (sums_w) write_sums<V, J>(sw, smem, sums_w, at, ch);
  if (sums_b) write_sums<V, J>(sb, smem, sums_b, at, ch);
}

template <class T, int J, int TH, bool EDGE>
TPC_NODE_KERNEL(TH, PASS_DBL, 16 / sizeof(T) * J)
    k_dbl(const __grid_constant__ NodeDesc D, const __grid_constant__ RowMap M, const __grid_constant__ NormArgs A,
          const uint32_t N) {
  constexpr int V = 16 / sizeof(T), E = V * J, P = E / 2;
  float* part = reinterpret_cast<float*>(g_smem + rows_bytes(E, 3, J, true, TH));
  const Place<TH, EDGE> at(D, M, V, part);
  const NodeBlock& B = at.B;
  const Channels ch(D, B);
  const bool centred = B.bias0 >= 0;
  const float inv = 1.f / (float)B.S;
  float* ws = reinterpret_cast<float*>(reinterpret_cast<char*>(part) + kPartBytes);
  float *ts = ws + (E << at.lg), *bs = ts + (E << at.lg);
  Ring<T, J, 3, TH, EDGE> rows;
  cudaGridDependencySynchronize();
  rows.start(g_smem, D, at, N, {A.x, A.grad_y, A.gg_x});
  expand<3>(ws, E << at.lg,
            {from_channel(A.weight, B.chan0), from_channel(A.gg_weight, B.chan0), from_channel(A.gg_bias, B.bias0)},
            {1.f, 0.f, 0.f}, ch, B.S, at.shift);
  __syncthreads();
  const uint32_t valid = valid_bits<V, J>(at);
  const Inner<T, J, EDGE> inner(valid);
  f2 sw[P];
#pragma unroll
  for (int p = 0; p < P; ++p) sw[p] = 0;
  Out<T, J, TH, EDGE> gx(A.grad_x, D, at), gg(A.grad_grad_y, D, at);
  float* const sums_w = sums_out(M, B, at.k, A.partial, A.grad_weight, B.chan0, false);
  for (uint32_t n = at.n; at.more(n, N); n += at.stride) {
    const bool ok = n < N;
    rows.next();
    // u, p, a = weight g, e = gg_weight g; less their means in a 0e block
    f2 u[P], pt[P], a[P], e[P], w[P], t[P];
    inner.get(rows, 0, u);
    if (A.gg_x) {
      inner.get(rows, 2, pt);
    } else {
#pragma unroll
      for (int p = 0; p < P; ++p) pt[p] = 0;
    }
    inner.get(rows, 1, a);
    lookup<V, J>(w, ws, at);
    lookup<V, J>(t, ts, at);
#pragma unroll
    for (int p = 0; p < P; ++p) {
      e[p] = mul2(a[p], t[p]);
      a[p] = mul2(a[p], w[p]);
    }
    if (centred) {
      float m[4] = {total(u), total(pt), total(a), total(e)};
      at.sum(m);
      shift_by<V, J, EDGE>(u, -m[0] * inv, valid);
      shift_by<V, J, EDGE>(pt, -m[1] * inv, valid);
      shift_by<V, J, EDGE>(a, -m[2] * inv, valid);
      shift_by<V, J, EDGE>(e, -m[3] * inv, valid);
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
    const float r = rsqrtf(q[0] * inv + D.eps);
    const float mp = r * q[1] * inv, ma = r * q[2] * inv, mpa = q[3] * inv, me = r * q[4] * inv;
    // grad_x = h (r^2 (3 mp ma - mpa) - r me) - r^2 ma p - r^2 mp a + r e,  k = r (p - h mp)
    const f2 r2 = both(r), c_h = both(r * r * (3.f * mp * ma - mpa) - r * me), c_p = both(-(r * r * ma)),
             c_a = both(-(r * r * mp)), nmp = both(-mp);
    f2 g[P], b[P];
    inner.get(rows, 1, g);
    lookup<V, J>(w, ws, at);
    lookup<V, J>(t, ts, at);
    lookup<V, J>(b, bs, at);
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const f2 h = mul2(u[p], r2), k = mul2(r2, fma2(h, nmp, pt[p]));
      if (ok) sw[p] = fma2(g[p], k, sw[p]);
      u[p] = fma2(h, c_h, fma2(c_p, pt[p], fma2(c_a, a[p], mul2(r2, e[p]))));
      e[p] = fma2(w[p], k, fma2(t[p], h, b[p]));
    }
    if (gx && ok) gx.put(u, valid);
    if (gg && ok) gg.put(e, valid);
    gx.next();
    gg.next();
    rows.done();
  }
  rows.finish();
  cudaTriggerProgrammaticLaunchCompletion();
  if (sums_w) write_sums<V, J>(sw, reinterpret_cast<float*>(g_smem), sums_w, at, ch);
}

// ---- dropout alone in 16 bits, blocks whose channels come in whole packs: a thread owns V channels of
// a row ----
//
// Bound by loads' latency and the generator's instructions.  With all 2l+1 components of its channels
// in one thread, a counter is drawn once for them and needs no exchange between lanes: 16384 x 1152
// bf16 14 us (82 % of the copy bandwidth), 27 us by k_fwd.  Four CTAs an SM and one row a step (two
// for scalars) measured best.  In float32 k_fwd's ring is faster (50000 x 592 with residual: 57 us, 65
// us here).

// Rows a step.
__host__ __device__ constexpr int drop_rows(int d) { return d == 1 ? 2 : 1; }

template <class T, int DC, bool MUL_IR>
__device__ __forceinline__ void drop_block(const NodeDesc& D, const NodeBlock& B, const Drop& drop, const T* x,
                                           const T* res, T* out, uint32_t N, uint32_t cta, uint32_t ctas) {
  constexpr int V = 16 / sizeof(T), U = drop_rows(DC);
  const uint32_t packs = B.C / V, lanes = packs < kThreads ? packs : kThreads, rows = kThreads / lanes;
  const uint32_t slot = threadIdx.x / lanes, lane = threadIdx.x - slot * lanes;
  if (slot >= rows) return;
  const uint64_t off = drop.mode == 1 ? drop_offset(drop) : 0;
  const int step = MUL_IR ? V : B.C;  // elements between a thread's packs
  for (uint32_t n0 = cta * rows * U + slot; n0 < N; n0 += ctas * rows * U)
    for (uint32_t q = lane; q < packs; q += lanes) {
      const uint32_t first = B.off + q * (MUL_IR ? V * DC : V);
      uint4 a[U][DC], b[U][DC];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const uint32_t n = n0 + u * rows;
        if (n >= N) break;
        const long long at = (long long)n * D.dim + first;
#pragma unroll
        for (int k = 0; k < DC; ++k) {
          a[u][k] = *reinterpret_cast<const uint4*>(x + at + k * step);
          if (res) b[u][k] = *reinterpret_cast<const uint4*>(res + at + k * step);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const uint32_t n = n0 + u * rows;
        if (n >= N) break;
        uint32_t keep = drop.mode == 0 ? ~0u : 0u;
        if (drop.mode == 1) {
#pragma unroll
          for (int g = 0; g < V / 4; ++g) {
            const uint4 w = drop_words(drop, off, B.grp0 + q * (V / 4) + g, n);
            keep |= ((w.x >= drop.threshold ? 1u : 0u) | (w.y >= drop.threshold ? 2u : 0u) |
                     (w.z >= drop.threshold ? 4u : 0u) | (w.w >= drop.threshold ? 8u : 0u))
                    << (4 * g);
          }
        }
        uint32_t m[V];  // all ones where a channel is kept: one AND an element
#pragma unroll
        for (int i = 0; i < V; ++i) m[i] = keep >> i & 1 ? ~0u : 0u;
        T* to = out + (long long)n * D.dim + first;
#pragma unroll
        for (int k = 0; k < DC; ++k) {
          const uint32_t wa[4] = {a[u][k].x, a[u][k].y, a[u][k].z, a[u][k].w};
          const uint32_t wb[4] = {b[u][k].x, b[u][k].y, b[u][k].z, b[u][k].w};
          uint32_t o[4];
#pragma unroll
          for (int i = 0; i < V; i += 2) {
            const int c0 = MUL_IR ? (k * V + i) / DC : i, c1 = MUL_IR ? (k * V + i + 1) / DC : i + 1;
            float v0, v1;
            unpack<T>(wa[i / 2], v0, v1);
            const f2 t = mul2(pack2(v0, v1), both(drop.scale));
            v0 = __uint_as_float(__float_as_uint(lo(t)) & m[c0]);
            v1 = __uint_as_float(__float_as_uint(hi(t)) & m[c1]);
            if (res) {
              float r0, r1;
              unpack<T>(wb[i / 2], r0, r1);
              v0 += r0;
              v1 += r1;
            }
            o[i / 2] = pack<T>(v0, v1);
          }
          *reinterpret_cast<uint4*>(to + k * step) = make_uint4(o[0], o[1], o[2], o[3]);
        }
      }
    }
}

template <class T, bool MUL_IR>
__global__ void __launch_bounds__(kThreads, kDropCtas)
    k_drop(const __grid_constant__ NodeDesc D, const __grid_constant__ RowMap M, const __grid_constant__ Drop drop,
           const T* x, const T* res, T* out, const uint32_t N) {
  int k = 0;
  while (k + 1 < M.n && (int)blockIdx.x >= M.cta0[k + 1]) ++k;
  const NodeBlock& B = D.b[M.blk[k]];
  const uint32_t cta = blockIdx.x - M.cta0[k], ctas = M.cta0[k + 1] - M.cta0[k];
  cudaGridDependencySynchronize();
  switch (B.d) {
    case 1: return drop_block<T, 1, false>(D, B, drop, x, res, out, N, cta, ctas);
    case 3: return drop_block<T, 3, MUL_IR>(D, B, drop, x, res, out, N, cta, ctas);
    case 5: return drop_block<T, 5, MUL_IR>(D, B, drop, x, res, out, N, cta, ctas);
    default: return drop_block<T, 7, MUL_IR>(D, B, drop, x, res, out, N, cta, ctas);
  }
}

// ---- any width: one CTA per segment, read again for each sum; a thread owns whole channels ----

template <int K>
__device__ __forceinline__ void cta_sum(float (&v)[K], int& flip) {
  __shared__ __align__(16) float part[2 * (kThreads / 32) * K];
  warps_sum(v, part, K, kThreads / 32, flip, 0, kThreads / 32, [] { __syncthreads(); });
}

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
              const __grid_constant__ NormArgs A, const uint32_t N) {
  const AnyPlace at(D, M);
  int flip = 0;
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
        cta_sum(m, flip);
        mu = m[0] * inv;
      }
      float q[1] = {0.f};
      each(B, D.mul_ir, [&](int c, int s) {
        const float u = value(c, s) - mu;
        q[0] += u * u;
      });
      cta_sum(q, flip);
      r = rsqrtf(q[0] * inv + D.eps);
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
              const __grid_constant__ NormArgs A, const uint32_t N) {
  const AnyPlace at(D, M);
  int flip = 0;
  const NodeBlock& B = at.B;
  const bool centred = B.bias0 >= 0;
  const float inv = 1.f / (float)B.S;
  const uint64_t off = DROP ? drop_offset(drop) : 0;
  float* pw = sums_out(M, B, at.k, A.partial, A.grad_weight, B.chan0, false);
  float* pb = centred ? sums_out(M, B, at.k, A.partial, A.grad_bias, B.bias0, true) : nullptr;
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
      cta_sum(m, flip);
    }
    const float mu = m[0] * inv, ma = m[1] * inv;
    each(B, D.mul_ir, [&](int c, int s) {
      const float u = to_f32(x[s]) - mu;
      q[0] += u * u;
      q[1] += u * (a(c, s) - ma);
    });
    cta_sum(q, flip);
    const float r = rsqrtf(q[0] * inv + D.eps), mh = r * q[1] * inv;
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
              const uint32_t N) {
  const AnyPlace at(D, M);
  int flip = 0;
  const NodeBlock& B = at.B;
  const bool centred = B.bias0 >= 0;
  const float inv = 1.f / (float)B.S;
  float* pw = sums_out(M, B, at.k, A.partial, A.grad_weight, B.chan0, false);
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
      cta_sum(m, flip);
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
    cta_sum(q, flip);
    const float r = rsqrtf(q[0] * inv + D.eps);
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
                  const float* partial, float* grad_weight, float* grad_bias) {
  __shared__ float share[kShares][33];
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const int i = blockIdx.x * 32 + tx;
  const bool bias = i >= D.channels;
  const int c = bias ? i - D.channels : i;
  float* out = bias ? grad_bias : grad_weight;
  bool wanted = out && i < D.channels + D.biases;
  const float* q = nullptr;
  int parts = 0;
  long long stride = 0;
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
      parts = M.parts[k];
      stride = part_stride(B);
      q = partial + M.part0[k] + (bias ? B.C + c - B.bias0 : c - B.chan0);
    }
  }
  cudaGridDependencySynchronize();  // the partial sums are complete (read past L1: written meanwhile)
  float v = 0.f;
  constexpr int kBatch = 10;  // loads on the way at a time: one wait for the CTAs of one wave
  for (int t = ty; t < parts; t += kBatch * kShares) {
    float w[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) w[i] = t + i * kShares < parts ? __ldcg(q + (t + i * kShares) * stride) : 0.f;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) v += w[i];
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

enum Kind { KIND_GROUP, KIND_WIDE, KIND_ANY };  // 256 threads, 512 threads, any width

struct Launch {
  Kind kind;
  int J, ctas, threads, smem;
  RowMap M;
};

struct LaunchPlan {
  bool edge = false;
  int n = 0;
  Launch l[3];
  PartMap parts{};
  size_t floats = 0;   // partial sums
};

// Most packs per lane: 16 elements, 12 (8 in 16 bits) in the double backward, whose five values per
// element fill the registers.  CTAs of 512 threads have that many always.
constexpr int most_packs(bool dbl, int esize) { return dbl ? (esize == 4 ? 3 : 1) : (esize == 4 ? 4 : 2); }
// CTAs of 256 threads have 1 up to this: 8 elements in the passes with sums off the boundary, whose masks
// take registers (backward 50000 x 145 f32: 28 us, 31 us with 12; f16: 26 us, 29 us with 16).
constexpr int most_narrow_packs(Pass pass, bool edge, int esize) {
  const int most = most_packs(pass == PASS_DBL, esize), eight = 8 * esize / 16;
  return edge && pass != PASS_FWD && most > eight ? eight : most;
}

int log2_lanes(int elems, int per_lane) {
  int lg = 0;
  while ((per_lane << lg) < elems) ++lg;
  return lg;
}

struct Shape {
  Pass pass;
  bool drop, norm;
  int esize, V;
  int arrays() const { return pass == PASS_FWD ? (drop ? 2 : 1) : pass == PASS_BWD ? (drop ? 3 : 2) : 3; }
  // Dynamic shared memory of a CTA whose widest group has 2^lg lanes.
  int smem(int J, int threads, int lg) const {
    const int vectors = pass == PASS_FWD ? (norm ? 2 : 0) : pass == PASS_BWD ? 1 : 3;
    return rows_bytes(V * J, arrays(), J, pass != PASS_FWD, threads) + kPartBytes +
           vectors * vector_bytes(V * J, lg) + (drop ? mask_bytes(V * J, threads) : 0);
  }
};

// CTAs that an SM holds: by registers and by shared memory (227 KB, 1 KB of it per CTA for the
// system).
int ctas_per_sm(int by_registers, int smem) {
  const int by_smem = 232448 / (smem + 1024);
  return by_smem < 1 ? 1 : by_smem < by_registers ? by_smem : by_registers;
}

LaunchPlan plan_launches(const Shape& sh, const NodeDesc& D, long long N) {
  LaunchPlan P;
  const int V = sh.V;
  const bool sums = sh.pass != PASS_FWD;
  for (int b = 0; b < D.n_blocks; ++b) P.edge = P.edge || D.b[b].S % V != 0;
  int R = 1;  // rows after which a row starts on the same offset from a 16-byte boundary
  while (P.edge && (long long)R * D.dim % V != 0) R *= 2;
  const int pad = P.edge ? V - 1 : 0;
  const int jmax = most_packs(sh.pass == PASS_DBL, sh.esize);
  // Most lanes of a segment in CTAs of 256 threads.  Wider ones share CTAs of 512 in the passes with
  // sums: half the partial sums (backward 8192 x 4096 bf16: 63 us, 65 us).
  const int narrow = sums ? 128 : kThreads;
  Kind kind[MAX_BLOCKS];
  for (int b = 0; b < D.n_blocks; ++b) {
    const int S = D.b[b].S + pad;
    kind[b] = S <= narrow * V * jmax                                                  ? KIND_GROUP
              : S <= kWide * V * jmax && sh.smem(jmax, kWide, log2_lanes(S, V * jmax)) <= kMaxSmem ? KIND_WIDE
                                                                                                  : KIND_ANY;
  }
  for (Kind kd : {KIND_GROUP, KIND_WIDE, KIND_ANY}) {
    Launch L{};
    L.kind = kd;
    RowMap& M = L.M;
    for (int b = 0; b < D.n_blocks; ++b)
      if (kind[b] == kd) M.blk[M.n++] = b;
    if (M.n == 0) continue;
    L.threads = kd == KIND_WIDE ? kWide : kThreads;
    M.classes = kd == KIND_ANY ? 1 : R;
    long long resident;   // CTAs that run at a time
    if (kd == KIND_ANY) {
      resident = sums ? kAnyParts : kSms * 8;
      for (int k = 0; k < M.n; ++k) M.lg[k] = log2_lanes(kThreads, 1);
    } else {
      // Fewest lane-packs per row (a segment's lanes are a power of two); of equal ones the most
      // packs per lane, but 12 elements in the passes with sums and in dropout alone (fused backward
      // 50000 x 592 f32: 104 us, 112 us with 16), 8 in the double backward (the same rows: 105 us, 110
      // us with 12).
      const int lg_max = log2_lanes(L.threads, 1), few = sh.pass == PASS_DBL ? 8 : !P.edge && (sums || !sh.norm) ? 12 : 16;
      const int most = kd == KIND_WIDE ? jmax : most_narrow_packs(sh.pass, P.edge, sh.esize);
      long long best = -1;
      for (int j = kd == KIND_WIDE ? jmax : 1; j <= most; ++j) {
        long long cost = 0;
        bool fits = true;
        for (int k = 0; k < M.n; ++k) {
          const int lg = log2_lanes(D.b[M.blk[k]].S + pad, V * j);
          fits = fits && lg <= lg_max;
          cost += (long long)j << lg;
        }
        int lanes = 0;
        for (int k = 0; k < M.n; ++k) lanes = std::max(lanes, 1 << log2_lanes(D.b[M.blk[k]].S + pad, V * j));
        if (fits && (best < 0 || cost < best || (cost == best && (V * j <= few || lanes > 32)))) {
          best = cost;
          L.J = j;
        }
      }
      int widest = 0;
      for (int k = 0; k < M.n; ++k) {
        M.lg[k] = log2_lanes(D.b[M.blk[k]].S + pad, V * L.J);
        widest = M.lg[k] > widest ? M.lg[k] : widest;
      }
      L.smem = sh.smem(L.J, L.threads, widest);
      resident = kSms * ctas_per_sm(kd == KIND_WIDE ? 1 : min_ctas(sh.pass, V * L.J), L.smem);
    }
    // CTAs that run at a time, shared out in proportion to the blocks' steps.  Few rows: one CTA per
    // block, whose sums need no second launch (64 x 288 f32 backward: 4.4 us; 6 us in two launches).
    long long rows[MAX_BLOCKS], total = 0, most = 0;   // rows[k]: CTA steps of block k in a residue class
    for (int k = 0; k < M.n; ++k) {
      const int per_step = kd == KIND_ANY ? 1 : L.threads >> M.lg[k];
      rows[k] = ((N + M.classes - 1) / M.classes + per_step - 1) / per_step;
      total += rows[k] * M.classes;
      most = rows[k] > most ? rows[k] : most;
    }
    const bool few_rows = sums && M.classes == 1 && most <= 4;
    const auto ctas = [&](int k) -> long long {
      if (few_rows) return 1;
      const long long share = total <= resident ? rows[k] : rows[k] * resident / total;
      return (share < 1 ? 1 : share) * M.classes;
    };
    M.direct = sums;
    for (int k = 0; k < M.n; ++k) {
      long long c = ctas(k);
      const long long room = kAnyFloats / part_stride(D.b[M.blk[k]]);
      if (sums && kd == KIND_ANY && c > room) c = room < 1 ? 1 : room;
      M.cta0[k + 1] = M.cta0[k] + (int)c;
      M.direct = M.direct && c == 1;
    }
    L.ctas = M.cta0[M.n];
    if (sums && !M.direct)
      for (int k = 0; k < M.n; ++k) {
        const int i = P.parts.n++;
        P.parts.blk[i] = M.blk[k];
        P.parts.parts[i] = M.cta0[k + 1] - M.cta0[k];
        P.parts.part0[i] = M.part0[k] = (long long)P.floats;
        P.floats += ((size_t)(P.parts.parts[i] * part_stride(D.b[M.blk[k]])) + 3) / 4 * 4;
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
  uint32_t N;
  cudaStream_t s;
};

// A launch that may start while the kernel before it in the stream drains.
template <class... Ps, class... As>
cudaError_t launch_early(void (*kernel)(Ps...), int ctas, int threads, int smem, cudaStream_t s, const As&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  prof_count(PC_NODE, 1);
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Launches a rows' kernel.  Dynamic shared memory beyond 48 KB has to be allowed once per kernel and
// device (not a stream operation, so a capture may do it).  Errors are seen by cudaGetLastError.
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
  launch_early(kernel, L.ctas, L.threads, L.smem, c.s, args...);
}

// Only kernels that some rows reach are built: dropout alone in 16 bits has rows off the boundary here
// (k_drop has the others).
template <class T, int J, int TH, bool EDGE, Pass PASS>
void run_kernel(const Call& c, const Launch& L) {
  static std::atomic<uint64_t> ok[3];  // devices, by kernel
  if constexpr (PASS == PASS_FWD) {
    if (!c.drop) {
      launch(k_fwd<T, J, TH, EDGE, false, true>, ok[0], c, L, c.D, L.M, c.d, c.A, c.N);
    } else if (c.norm) {
      launch(k_fwd<T, J, TH, EDGE, true, true>, ok[1], c, L, c.D, L.M, c.d, c.A, c.N);
    } else if constexpr (sizeof(T) == 4 || EDGE) {
      launch(k_fwd<T, J, TH, EDGE, true, false>, ok[2], c, L, c.D, L.M, c.d, c.A, c.N);
    }
  } else if constexpr (PASS == PASS_BWD) {
    if (c.drop) launch(k_bwd<T, J, TH, EDGE, true>, ok[0], c, L, c.D, L.M, c.d, c.A, c.N);
    else launch(k_bwd<T, J, TH, EDGE, false>, ok[1], c, L, c.D, L.M, c.d, c.A, c.N);
  } else {
    launch(k_dbl<T, J, TH, EDGE>, ok[0], c, L, c.D, L.M, c.A, c.N);
  }
}

template <class T, bool EDGE, Pass PASS, int J = 1>
void run_packs(const Call& c, const Launch& L) {
  if (L.kind == KIND_WIDE) {
    if constexpr (J == 1) run_kernel<T, most_packs(PASS == PASS_DBL, sizeof(T)), kWide, EDGE, PASS>(c, L);
  } else if (L.J == J) {
    run_kernel<T, J, kThreads, EDGE, PASS>(c, L);
  } else if constexpr (J < most_narrow_packs(PASS, EDGE, sizeof(T))) {
    run_packs<T, EDGE, PASS, J + 1>(c, L);
  }
}

template <class T, bool EDGE>
void run_pass(const Call& c, const Launch& L) {
  if (c.pass == PASS_FWD) run_packs<T, EDGE, PASS_FWD>(c, L);
  else if (c.pass == PASS_BWD) run_packs<T, EDGE, PASS_BWD>(c, L);
  else run_packs<T, EDGE, PASS_DBL>(c, L);
}

template <class T>
void run_any(const Call& c, const Launch& L) {
  const dim3 grid(L.ctas), block(kThreads);
  prof_count(PC_NODE, 1);
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

// Dropout alone where every block's channels come in whole packs; false: not such rows.
template <class T>
bool run_drop(const Call& c) {
  constexpr int V = 16 / sizeof(T);
  for (int b = 0; b < c.D.n_blocks; ++b)
    if (c.D.b[b].C % V != 0) return false;
  // CTAs in proportion to what the blocks' steps take: a load's latency and the packs.  The latency as 8
  // packs, 2 with a residual (twice the loads on the way): 16384 x 1152 bf16 14.1 us, 15.3 us with 2
  // (16.9 us by bytes alone); 50000 x 592 bf16 with residual 33.4 us, 36.0 us with 8.
  RowMap M{};
  M.n = c.D.n_blocks;
  long long work[MAX_BLOCKS], most[MAX_BLOCKS], total = 0;
  for (int b = 0; b < M.n; ++b) {
    const NodeBlock& B = c.D.b[b];
    const long long packs = B.C / V, lanes = packs < kThreads ? packs : kThreads;
    const long long rows = kThreads / lanes * drop_rows(B.d);
    most[b] = (c.N + rows - 1) / rows;
    const int loads = drop_rows(B.d) * B.d * (c.A.residual ? 2 : 1);
    work[b] = most[b] * ((packs + lanes - 1) / lanes) * ((c.A.residual ? 2 : 8) + loads);
    total += work[b];
  }
  for (int b = 0; b < M.n; ++b) {
    const long long share = work[b] * kSms * kDropCtas / total;
    M.blk[b] = b;
    M.cta0[b + 1] = M.cta0[b] + (int)(share < 1 ? 1 : share > most[b] ? most[b] : share);
  }
  launch_early(c.D.mul_ir ? k_drop<T, true> : k_drop<T, false>, M.cta0[M.n], kThreads, 0, c.s, c.D, M, c.d,
               (const T*)c.A.x, (const T*)c.A.residual, (T*)c.A.z, c.N);
  return true;
}

template <class T>
cudaError_t run_node(const Call& c) {
  if constexpr (sizeof(T) == 2)
    if (!c.norm && run_drop<T>(c)) return cudaGetLastError();
  const LaunchPlan P = plan_launches(Shape{c.pass, c.drop, c.norm, sizeof(T), 16 / sizeof(T)}, c.D, c.N);
  for (int i = 0; i < P.n; ++i) {
    const Launch& L = P.l[i];
    if (L.kind == KIND_ANY) run_any<T>(c, L);
    else if (P.edge) run_pass<T, true>(c, L);
    else run_pass<T, false>(c, L);
  }
  if (c.A.partial && P.parts.n)
    launch_early(k_norm_reduce, (c.D.channels + c.D.biases + 31) / 32, 32 * kShares, 0, c.s, c.D, P.parts,
                 (const float*)c.A.partial, c.A.grad_weight, c.A.grad_bias);
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
  return run_node<TPC_T>(Call{(Pass)pass, drop != nullptr, norm, D, drop ? *drop : none, A, (uint32_t)N, s});
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
  for (const Shape& sh : {Shape{PASS_BWD, false, true, esize, 16 / esize}, Shape{PASS_BWD, true, true, esize, 16 / esize},
                          Shape{PASS_DBL, false, true, esize, 16 / esize}}) {
    const size_t f = plan_launches(sh, D, N).floats;
    most = f > most ? f : most;
  }
  return most;
}
#endif

}  // namespace tpc
