// rotary.cuh -- rotary positions with one or several axes.
//
// Pair p of a head belongs to axis a(p) and turns by angle
//   position[a(p)][b][l] * f(p),
// (x, z) -> (x cos - z sin, z cos + x sin); the inverse turns back, which is
// also the gradient (the rotation is orthogonal).  Elements past the last
// pair pass through.
//
// The angle is kept in turns: position * (f / 2 pi) in fp64, two roundings of
// 2^-53 relative, then sincospi of the fraction in fp32 (2^-25 of a turn).  For
// 32-bit positions and frequencies up to 1 that is 7e-7 radians (an fp32
// product would lose the fraction at positions of some thousands).
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
__global__ void __launch_bounds__(kRotThreads, V == 8 ? 4 : 6) rotary_kernel(const __grid_constant__ RotaryParams p) {
  // The pairs' frequencies and axes go through shared memory: read from the
  // parameters by every thread at its own index, they would be fetched one
  // distinct address at a time.
  __shared__ double s_turn[kRotMaxPairs];
  __shared__ int s_axis[kRotMaxPairs];
  for (int i = threadIdx.x; i < p.pairs; i += kRotThreads) {
    s_turn[i] = p.turn[i];
    s_axis[i] = p.axis[i];
  }
  __syncthreads();
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
      const long long at = s_axis[p0 + i] * tokens + tok;
      const long long pos = p.pos64 ? static_cast<const long long*>(p.positions)[at]
                                    : static_cast<const int*>(p.positions)[at];
      const double t = (double)pos * s_turn[p0 + i];
      sincospif(2.f * (float)(t - rint(t)), &sn[i], &cs[i]);
      if (p.inverse) sn[i] = -sn[i];
    }
    off0 = kInterleaved ? 2 * p0 : p0;
    off1 = kInterleaved ? 2 * p0 + V : p0 + p.pairs;
  } else {
    off0 = off1 = 2 * p.pairs + (vec * V - p.pairs);
  }
  const int d1 = off1 - off0;
#pragma unroll 1
  for (int w = 0; w < 2; ++w) {  // q, then k
    const int first = w ? max(h0 - p.q_heads, 0) : h0;
    const int end = w ? h1 - p.q_heads : min(h1, p.q_heads);
    if (first >= end) continue;
    const long long ih = p.in_h[w], oh = p.out_h[w];
    const TI* src = static_cast<const TI*>(w ? p.k : p.q) + b * p.in_b[w] + first * ih + l * p.in_l[w] + off0;
    TO* dst = static_cast<TO*>(w ? p.k_out : p.q_out) + b * p.out_b[w] + first * oh + l * p.out_l[w] + off0;
    auto turn = [&](const RotVec<TI, V>& x, const RotVec<TI, V>& z, TO* to) {
      float a[V], c[V];
      if (!turns) {
#pragma unroll
        for (int i = 0; i < V; ++i) a[i] = rot_float(x.x[i]);
        rot_store<TO, V>(to, a);
        return;
      }
      if constexpr (kInterleaved) {
        // The 2 V elements x | z hold pairs (0, 1), (2, 3), ...
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float e = rot_float(2 * i < V ? x.x[2 * i % V] : z.x[2 * i % V]);
          const float f = rot_float(2 * i + 1 < V ? x.x[(2 * i + 1) % V] : z.x[(2 * i + 1) % V]);
          const float re = e * cs[i] - f * sn[i], im = f * cs[i] + e * sn[i];
          if (2 * i < V) a[2 * i % V] = re; else c[2 * i % V] = re;
          if (2 * i + 1 < V) a[(2 * i + 1) % V] = im; else c[(2 * i + 1) % V] = im;
        }
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float e = rot_float(x.x[i]), f = rot_float(z.x[i]);
          a[i] = e * cs[i] - f * sn[i];
          c[i] = f * cs[i] + e * sn[i];
        }
      }
      rot_store<TO, V>(to, a);
      rot_store<TO, V>(to + d1, c);
    };
    // Two heads in flight per thread (the elements as loaded), and four to
    // six blocks per SM.  Measured on the long prompt (2 x 16384 tokens, 32 +
    // 8 heads of 128): 5.3 TB/s; four heads in flight and two blocks, 4.0.
    int n = end - first;
#pragma unroll 1
    for (; n >= 2; n -= 2, src += 2 * ih, dst += 2 * oh) {
      const RotVec<TI, V> x0 = *reinterpret_cast<const RotVec<TI, V>*>(src);
      const RotVec<TI, V> z0 = *reinterpret_cast<const RotVec<TI, V>*>(src + d1);
      const RotVec<TI, V> x1 = *reinterpret_cast<const RotVec<TI, V>*>(src + ih);
      const RotVec<TI, V> z1 = *reinterpret_cast<const RotVec<TI, V>*>(src + ih + d1);
      turn(x0, z0, dst);
      turn(x1, z1, dst + oh);
    }
    if (n > 0) {
      const RotVec<TI, V> x0 = *reinterpret_cast<const RotVec<TI, V>*>(src);
      const RotVec<TI, V> z0 = *reinterpret_cast<const RotVec<TI, V>*>(src + d1);
      turn(x0, z0, dst);
    }
  }
}

}  // namespace gqa
