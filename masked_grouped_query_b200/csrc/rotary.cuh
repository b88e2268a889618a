// rotary.cuh -- rotary positions with one or several axes.
//
// Pair p of a head belongs to axis a(p) and turns by angle
//   position[a(p)][b][l] * f(p),
// (x, z) -> (x cos - z sin, z cos + x sin); the inverse turns back, which is
// also the gradient (the rotation is orthogonal).  Elements past the last
// pair pass through.
//
// The angle is kept in turns: position * (f / 2 pi) in fp64, whose fraction
// is exact to 2^-20 of a turn or better for every 32-bit position (an fp32
// product would lose the fraction at positions of some thousands), then
// sincospi of the fp32 fraction.
//
// Bound by memory: q and k are read and written once.  A thread computes the
// sine and cosine of V pairs of one token once and applies them to a run of
// heads, so the fp64 work is one multiplication per pair and token for all
// heads of the run; the host cuts the heads into runs only as far as it needs
// threads (single-token calls).
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

namespace gqa {

constexpr int kRotMaxPairs = 128;
constexpr int kRotMaxAxes = 8;
constexpr int kRotThreads = 256;

struct RotaryParams {
  const void *q, *k;
  void *q_out, *k_out;
  const void* positions;   // [axes][batch][length], int32 or int64
  int pos64, inverse;
  int batch, length, head_dim, q_heads, kv_heads;
  int pairs;               // rotated pairs per head
  int vecs;                // threads per (token, head run): pairs / V + passed-through vectors
  int heads_per_thread;
  // Elements between batch rows, heads and tokens: input and output, q then k.
  long long in_b[2], in_h[2], in_l[2];
  long long out_b[2], out_h[2], out_l[2];
  double turn[kRotMaxPairs];     // frequency / (2 pi)
  unsigned char axis[kRotMaxPairs];
};

// V elements as they lie in memory (one access), and as floats.
template <typename T, int V>
struct __align__(sizeof(T) * V > 16 ? 16 : sizeof(T) * V) RotVec {
  T x[V];
};
__device__ __forceinline__ float rot_float(float x) { return x; }
__device__ __forceinline__ float rot_float(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T rot_round(float x);
template <>
__device__ __forceinline__ float rot_round<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 rot_round<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <typename T, int V>
__device__ __forceinline__ void rot_store(T* p, const float (&f)[V]) {
  RotVec<T, V> v;
#pragma unroll
  for (int i = 0; i < V; ++i) v.x[i] = rot_round<T>(f[i]);
  *reinterpret_cast<RotVec<T, V>*>(p) = v;
}

template <int V, typename TI, typename TO, bool kInterleaved>
__global__ void __launch_bounds__(kRotThreads) rotary_kernel(const __grid_constant__ RotaryParams p) {
  const long long tokens = (long long)p.batch * p.length;
  const long long idx = (long long)blockIdx.x * kRotThreads + threadIdx.x;
  const long long tok = idx / p.vecs;
  if (tok >= tokens) return;
  const int vec = (int)(idx - tok * p.vecs);
  const int b = (int)(tok / p.length), l = (int)(tok - (long long)b * p.length);
  const int h0 = blockIdx.y * p.heads_per_thread;
  const int h1 = min(h0 + p.heads_per_thread, p.q_heads + p.kv_heads);
  const bool turns = vec * V < p.pairs;
  float cs[V], sn[V];
  int off0, off1;
  if (turns) {
    const int p0 = vec * V;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const long long at = (long long)p.axis[p0 + i] * tokens + tok;
      const long long pos = p.pos64 ? static_cast<const long long*>(p.positions)[at]
                                    : static_cast<const int*>(p.positions)[at];
      const double t = (double)pos * p.turn[p0 + i];
      sincospif(2.f * (float)(t - rint(t)), &sn[i], &cs[i]);
      if (p.inverse) sn[i] = -sn[i];
    }
    off0 = kInterleaved ? 2 * p0 : p0;
    off1 = kInterleaved ? 2 * p0 + V : p0 + p.pairs;
  } else {
    off0 = off1 = 2 * p.pairs + (vec * V - p.pairs);
  }
  // Heads in flight per thread: their vectors stay as loaded until they are
  // turned, 16 or 32 bytes a head.
  constexpr int U = sizeof(TI) * V >= 16 ? 4 : 8;
  // A batch of heads lies in q or in k, never across.
  for (int hb = h0; hb < h1;) {
    const int w = hb >= p.q_heads;
    const int base = w ? p.q_heads : 0, end = w ? h1 : min(h1, p.q_heads);
    const int n = min(U, end - hb);
    const TI* src = static_cast<const TI*>(w ? p.k : p.q) + b * p.in_b[w] +
                    (hb - base) * p.in_h[w] + l * p.in_l[w];
    TO* dst = static_cast<TO*>(w ? p.k_out : p.q_out) + b * p.out_b[w] + (hb - base) * p.out_h[w] +
              l * p.out_l[w];
    const long long ih = p.in_h[w], oh = p.out_h[w];
    RotVec<TI, V> x[U], z[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (u >= n) break;
      x[u] = *reinterpret_cast<const RotVec<TI, V>*>(src + u * ih + off0);
      if (turns) z[u] = *reinterpret_cast<const RotVec<TI, V>*>(src + u * ih + off1);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (u >= n) break;
      float a[V], c[V];
      if (!turns) {
#pragma unroll
        for (int i = 0; i < V; ++i) a[i] = rot_float(x[u].x[i]);
        rot_store<TO, V>(dst + u * oh + off0, a);
        continue;
      }
      if constexpr (kInterleaved) {
        // The 2 V elements x | z hold pairs (0, 1), (2, 3), ...
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float e = rot_float(2 * i < V ? x[u].x[2 * i % V] : z[u].x[2 * i % V]);
          const float f = rot_float(2 * i + 1 < V ? x[u].x[(2 * i + 1) % V] : z[u].x[(2 * i + 1) % V]);
          const float re = e * cs[i] - f * sn[i], im = f * cs[i] + e * sn[i];
          if (2 * i < V) a[2 * i % V] = re; else c[2 * i % V] = re;
          if (2 * i + 1 < V) a[(2 * i + 1) % V] = im; else c[(2 * i + 1) % V] = im;
        }
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float e = rot_float(x[u].x[i]), f = rot_float(z[u].x[i]);
          a[i] = e * cs[i] - f * sn[i];
          c[i] = f * cs[i] + e * sn[i];
        }
      }
      rot_store<TO, V>(dst + u * oh + off0, a);
      rot_store<TO, V>(dst + u * oh + off1, c);
    }
    hb += n;
  }
}

}  // namespace gqa
