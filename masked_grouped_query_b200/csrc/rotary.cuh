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

template <typename T, int V>
struct RotVec;
template <int V>
struct __align__(2 * V) RotBf {
  __nv_bfloat16 x[V];
};
template <int V>
struct __align__(V >= 4 ? 16 : 4 * V) RotF {
  float x[V];
};
template <int V>
__device__ __forceinline__ void rot_load(const __nv_bfloat16* p, float (&f)[V]) {
  const RotBf<V> v = *reinterpret_cast<const RotBf<V>*>(p);
#pragma unroll
  for (int i = 0; i < V; ++i) f[i] = __bfloat162float(v.x[i]);
}
template <int V>
__device__ __forceinline__ void rot_load(const float* p, float (&f)[V]) {
  const RotF<V> v = *reinterpret_cast<const RotF<V>*>(p);
#pragma unroll
  for (int i = 0; i < V; ++i) f[i] = v.x[i];
}
template <int V>
__device__ __forceinline__ void rot_store(__nv_bfloat16* p, const float (&f)[V]) {
  RotBf<V> v;
#pragma unroll
  for (int i = 0; i < V; ++i) v.x[i] = __float2bfloat16_rn(f[i]);
  *reinterpret_cast<RotBf<V>*>(p) = v;
}
template <int V>
__device__ __forceinline__ void rot_store(float* p, const float (&f)[V]) {
  RotF<V> v;
#pragma unroll
  for (int i = 0; i < V; ++i) v.x[i] = f[i];
  *reinterpret_cast<RotF<V>*>(p) = v;
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
  constexpr int U = 4;  // heads in flight per thread
  for (int hb = h0; hb < h1; hb += U) {
    float x[U][V], z[U][V];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = hb + u;
      if (h >= h1) break;
      const int w = h >= p.q_heads;
      const TI* src = static_cast<const TI*>(w ? p.k : p.q) + b * p.in_b[w] +
                      (h - (w ? p.q_heads : 0)) * p.in_h[w] + l * p.in_l[w];
      rot_load<V>(src + off0, x[u]);
      if (turns) rot_load<V>(src + off1, z[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = hb + u;
      if (h >= h1) break;
      const int w = h >= p.q_heads;
      TO* dst = static_cast<TO*>(w ? p.k_out : p.q_out) + b * p.out_b[w] +
                (h - (w ? p.q_heads : 0)) * p.out_h[w] + l * p.out_l[w];
      if (!turns) {
        rot_store<V>(dst + off0, x[u]);
        continue;
      }
      float a[V], c[V];
      if constexpr (kInterleaved) {
        // The 2 V elements x | z hold pairs (0, 1), (2, 3), ...
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float e = 2 * i < V ? x[u][2 * i % V] : z[u][2 * i % V];
          const float f = 2 * i + 1 < V ? x[u][(2 * i + 1) % V] : z[u][(2 * i + 1) % V];
          const float re = e * cs[i] - f * sn[i], im = f * cs[i] + e * sn[i];
          if (2 * i < V) a[2 * i % V] = re; else c[2 * i % V] = re;
          if (2 * i + 1 < V) a[(2 * i + 1) % V] = im; else c[(2 * i + 1) % V] = im;
        }
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          a[i] = x[u][i] * cs[i] - z[u][i] * sn[i];
          c[i] = z[u][i] * cs[i] + x[u][i] * sn[i];
        }
      }
      rot_store<V>(dst + off0, a);
      rot_store<V>(dst + off1, c);
    }
  }
}

}  // namespace gqa
