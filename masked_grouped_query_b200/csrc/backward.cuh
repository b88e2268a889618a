// backward.cuh -- the backward pass of masked GQA attention: what its two
// kernels share, and the pass over the rows that prepares their statistics.
//
// With s = q k^T, x = s / sqrt(D) (or cap * tanh(s / (sqrt(D) cap))) and the
// forward's row statistics, the probabilities are recomputed,
//   P = exp(x - lse),  0 where the mask hides the key,
// and with dP = dO V^T and delta = rowsum(dO * O) - dlse
//   dS = P * (dP - delta) * (1 - tanh^2 with a cap),
//   dV = P^T dO,  dK = dS^T Q / sqrt(D),  dQ = dS K / sqrt(D).
// The gradient of a kv head sums over the q heads of its group.
//
// dK and dV are sums over rows, dQ is a sum over keys.  One pass that made
// all three would have to add dQ (or dK, dV) across CTAs; doing that in no
// fixed order changes the result from run to run, and this library's results
// do not change.  So two kernels each own their outputs: one walks the rows
// of a key tile (four products: S, dP, dV, dK), the other the keys of a row
// tile (three: S, dP, dQ).  Seven products instead of five, but no atomics,
// no fp32 dQ buffer and no conversion pass.
//
// When there are far fewer tiles than SMs (few keys under many rows, few rows
// over many keys), the walk of each tile is cut into `splits` parts that leave
// fp32 partials, which bwd_join_kernel adds in their order.
#pragma once

#include "mask.cuh"
#include "ptx.cuh"

namespace gqa {

constexpr float kLog2e32 = 1.4426950408889634f;

// Rows as the backward kernels see them: `runs` runs of `run` consecutive
// rows (row r of a run is query r % q_len), cut into tiles of 128 that do not
// cross runs.  A run is a q head when a mask makes most tiles of a head
// skippable (q_len >= 256), else the whole group of a kv head, which wastes
// no part of a tile at head boundaries.
struct BwdShape {
  int q_len, kv_len, head_dim, causal, window;
  int run;            // rows per run
  int runs_per_unit;  // runs of one (batch, kv head): group, or 1
  int tiles;          // 128-row tiles per run
  long long runs;     // batch * kv heads * runs_per_unit
  long long units;    // batch * kv heads
};

struct BwdParams {
  BwdShape sh;
  const __nv_bfloat16 *q, *k, *v, *dout;
  __nv_bfloat16 *dq, *dk, *dv;
  const float* stats;  // [run][tile]: 128 times -lse (log2 units, -inf: no key), then 128 delta
  int softcap;
  float scale;         // 1 / sqrt(D)
  float logit_scale;   // log2(e) / sqrt(D)
  float cap_in;        // 1 / (sqrt(D) * cap)
  float cap_out;       // cap * log2(e)
  float poly_most;     // largest |x * cap_in| for the degree-7 polynomial (tcgen05)
  // Parts of a tile's walk; with more than one, their fp32 partials: part i is
  // [columns rounded up to 16, by 4][tile rows][4].
  int kv_splits, q_splits;
  float *part_dk, *part_dv, *part_dq;
};

// Part sp of splits of n steps: [begin, end).
__device__ __forceinline__ void bwd_part(int n, int sp, int splits, int& begin, int& end) {
  begin = 0;
  end = n;
  if (splits > 1) {  // 64-bit divisions that the usual walk is spared
    begin = (int)((long long)n * sp / splits);
    end = (int)((long long)n * (sp + 1) / splits);
  }
}

// Adds the partials of dK, dV (jobs 0, 1) and dQ (job 2) in their order and
// rounds the sums; a block per tile, rows fastest (coalesced reads).
struct BwdJoin {
  struct Job {
    const float* part;
    __nv_bfloat16* out;
    float scale;
    int splits, rows;  // parts per tile; rows of a run of tiles
    long long outers, items;
  } job[3];
  int tile_rows, head_dim;
};
__global__ void __launch_bounds__(256) bwd_join_kernel(const __grid_constant__ BwdJoin j) {
  const BwdJoin::Job& job = j.job[blockIdx.y];
  const long long item = blockIdx.x;
  if (job.splits <= 1 || item >= job.items) return;
  const int R = j.tile_rows, pad = (j.head_dim + 15) / 16 * 16;
  const long long outer = item % job.outers;
  const int row0 = (int)(item / job.outers) * R;
  const float4* src = reinterpret_cast<const float4*>(job.part) + item * job.splits * (R * pad / 4);
  for (int e = threadIdx.x; e < R * (j.head_dim / 8); e += 256) {
    const int row = e % R, c = e / R;
    if (row0 + row >= job.rows) continue;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
    for (int sp = 0; sp < job.splits; ++sp) {
      const float4* q = src + (long long)sp * (R * pad / 4) + (2 * c) * R + row;
      const float4 x = q[0], y = q[R];
      a.x += x.x; a.y += x.y; a.z += x.z; a.w += x.w;
      b.x += y.x; b.y += y.y; b.z += y.z; b.w += y.w;
    }
    const float f = job.scale;
    *reinterpret_cast<uint4*>(job.out + (outer * job.rows + row0 + row) * j.head_dim + 8 * c) =
        make_uint4(pack_bf16(a.x * f, a.y * f), pack_bf16(a.z * f, a.w * f),
                   pack_bf16(b.x * f, b.y * f), pack_bf16(b.z * f, b.w * f));
  }
}

__host__ __device__ __forceinline__ MaskSpec bwd_mask(const BwdShape& s) {
  return MaskSpec{s.q_len, s.kv_len, s.causal, s.window};
}

// The queries [lo, hi] (indexes into q_len, clamped) that see any key of
// [k0, k1]; empty when hi < lo.
__host__ __device__ __forceinline__ void bwd_query_range(const BwdShape& s, int k0, int k1, int& lo,
                                                         int& hi) {
  const long long base = (long long)s.kv_len - s.q_len;
  long long a = 0, b = (long long)s.q_len - 1;
  if (s.causal || s.window > 0) a = k0 - base > 0 ? k0 - base : 0;
  if (s.window > 0) {
    const long long e = (long long)k1 + s.window - 1 - base;
    b = e < b ? e : b;
  }
  if (a > s.q_len) a = s.q_len;
  if (b < -1) b = -1;
  lo = (int)a;
  hi = (int)b;
}

// Row tiles [first, first + count) of each run that a key tile has to visit.
__host__ __device__ __forceinline__ void bwd_row_tiles(const BwdShape& s, int k0, int k1, int tile,
                                                       int& first, int& count) {
  int lo, hi;
  bwd_query_range(s, k0, k1, lo, hi);
  first = 0;
  count = 0;
  if (hi < lo) return;
  if (s.run == s.q_len) {
    first = lo / tile;
    count = hi / tile - first + 1;
  } else {
    count = (s.run + tile - 1) / tile;
  }
}

// Whether any row of a row tile fails to see any of the `keys` keys from k0 on:
// only then are scores masked one by one.
__device__ __forceinline__ bool bwd_need_mask(const BwdShape& s, const MaskSpec& ms, int r0, int nr,
                                              int k0, int keys) {
  if (!(s.causal || s.window > 0)) return k0 + keys > s.kv_len;
  int i0 = r0, i1 = r0 + nr - 1;
  if (s.run != s.q_len) {
    if (nr >= s.q_len) {
      i0 = 0;
      i1 = s.q_len - 1;
    } else {
      i0 = (int)((unsigned)i0 % (unsigned)s.q_len);
      i1 = (int)((unsigned)i1 % (unsigned)s.q_len);
      if (i1 < i0) {
        i0 = 0;
        i1 = s.q_len - 1;
      }
    }
  }
  const int base = s.kv_len - s.q_len;
  return !(k0 >= first_key(ms, base + i1) && k0 + keys - 1 <= last_key(ms, base + i0));
}

// delta and lse of every row into the tiled statistics, one block per tile.
// A tile's rows are one contiguous stretch of dO and of O, read in 16-byte
// pieces whatever head_dim is; the pieces' dot products meet in shared memory
// (rows padded by one word against bank conflicts) and two threads add up a
// row.  Rows that pad a run's last tile get -lse = -inf and delta = 0, so that
// their P and dS are zero.  Bound by the reads: 16 threads a row, a pass per
// row, reached 2.9 TB/s at head_dim 128 and 1.8 TB/s at 72.
constexpr int kBwStatThreads = 256;
__global__ void __launch_bounds__(kBwStatThreads)
    bwd_stats_kernel(const __nv_bfloat16* __restrict__ dout, const __nv_bfloat16* __restrict__ o,
                     const float* __restrict__ lse, const float* __restrict__ dlse,
                     float* __restrict__ stats, const BwdShape s) {
  __shared__ float part[128 * 33];
  const long long tile = blockIdx.x;
  const long long run = tile / s.tiles;
  const int r0 = (int)(tile - run * s.tiles) * 128;
  const int nr = min(128, s.run - r0);
  const long long row0 = run * s.run + r0;
  const unsigned per_row = (unsigned)s.head_dim / 8, pieces = nr * per_row;
  const uint4* a = reinterpret_cast<const uint4*>(dout + row0 * s.head_dim);
  const uint4* b = reinterpret_cast<const uint4*>(o + row0 * s.head_dim);
  constexpr int U = 4;  // pieces in flight per thread
  for (unsigned i0 = threadIdx.x; i0 < pieces; i0 += U * kBwStatThreads) {
    uint4 x[U], y[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const unsigned i = i0 + u * kBwStatThreads;
      if (i < pieces) {
        x[u] = __ldg(a + i);
        y[u] = __ldg(b + i);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const unsigned i = i0 + u * kBwStatThreads;
      if (i >= pieces) break;
      const uint32_t xs[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
      const uint32_t ys[4] = {y[u].x, y[u].y, y[u].z, y[u].w};
      float sum = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&xs[e]));
        const float2 g = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&ys[e]));
        sum = fmaf(f.x, g.x, sum);
        sum = fmaf(f.y, g.y, sum);
      }
      const unsigned row = i / per_row;
      part[row * (per_row + 1) + (i - row * per_row)] = sum;
    }
  }
  __syncthreads();
  const int r = threadIdx.x >> 1, half = threadIdx.x & 1;
  float sum = 0.f;
  if (r < nr)
    for (unsigned c = half; c < per_row; c += 2) sum += part[r * (per_row + 1) + c];
  sum += __shfl_xor_sync(0xffffffffu, sum, 1);
  if (half == 0) {
    float l2 = -INFINITY;
    if (r < nr) {
      const float l = lse[row0 + r];
      l2 = l == -INFINITY ? -INFINITY : -l * kLog2e32;
      if (dlse) sum -= dlse[row0 + r];
    }
    stats[tile * 256 + r] = l2;
    stats[tile * 256 + 128 + r] = r < nr ? sum : 0.f;
  }
}

// ------------------------------------------------------------------ mma.sync
// Both kernels as 64 x 64 tiles on mma.sync m16n8k16, for every head_dim up
// to 256; the tcgen05 kernels take over up to 128 (with wider heads their
// accumulators alone would fill TMEM, and two operand tiles shared memory).
//
// One CTA keeps the 64 rows of its own two operands in shared memory (K, V
// for dK/dV; Q, dO for dQ) and streams 64-row tiles of the other two through
// two buffers (cp.async: the next tiles load under this one's products).  Eight
// warps: warp w computes the 16 x 32 piece (16 own rows from w % 4, 32
// streamed rows from w / 4) of S and dP, leaves P and dS as bf16 in shared
// memory, and accumulates 16 own rows x half of the columns of its outputs in
// registers (fp32).
constexpr int kBmTile = 64;
constexpr int kBmThreads = 256;

template <int KS>
struct BwdMmaCfg {
  static constexpr int kPitch = KS * 16 + 8;  // elements: rows 16 bytes off a multiple of 128
  static constexpr int kTileElems = kBmTile * kPitch;
  static constexpr int kPPitch = kBmTile + 8;
  static constexpr int kSmemBytes = (6 * kTileElems + 2 * kBmTile * kPPitch) * 2 + 6 * kBmTile * 4;
};

// n rows x D of a [rows][D] matrix into a padded tile, zeros elsewhere
// (asynchronously: part of the thread's next committed group).
template <int KS>
__device__ __forceinline__ void bwd_load_tile(__nv_bfloat16* dst, const __nv_bfloat16* src, int D,
                                              int n) {
  using C = BwdMmaCfg<KS>;
#pragma unroll 4
  for (int i = threadIdx.x; i < kBmTile * KS * 2; i += kBmThreads) {
    const int r = i / (KS * 2), c = (i - r * (KS * 2)) * 8;
    const bool in = r < n && c < D;
    cp_async16(dst + r * C::kPitch + c, in ? src + (long long)r * D + c : src, in);
  }
}

// Two values as a bf16 pair; with kFine they keep what the rounding left.
template <bool kFine>
__device__ __forceinline__ uint32_t bwd_take_bf16(float& a, float& b) {
  const uint32_t w = pack_bf16(a, b);
  if constexpr (kFine) {
    a -= __uint_as_float(w << 16);
    b -= __uint_as_float(w & 0xffff0000u);
  }
  return w;
}

template <int KS, bool kDQ, bool kFine>
__global__ void __launch_bounds__(kBmThreads, 1) bwd_mma_kernel(const BwdParams p) {
  using C = BwdMmaCfg<KS>;
  const BwdShape& s = p.sh;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  __nv_bfloat16* own1 = (__nv_bfloat16*)smem_raw;  // K (dK/dV) or Q (dQ)
  __nv_bfloat16* own2 = own1 + C::kTileElems;      // V or dO
  __nv_bfloat16* str = own2 + C::kTileElems;       // two buffers of Q, dO or K, V
  __nv_bfloat16* pm = str + 4 * C::kTileElems;     // P  [own row][streamed row]
  __nv_bfloat16* dm = pm + kBmTile * C::kPPitch;   // dS
  // Two buffers for the query rows: 64 times -lse, 64 delta, 64 positions.
  float* st2 = (float*)(dm + kBmTile * C::kPPitch);
  if (threadIdx.x == 0 && !kDQ) {  // the statistics; then dQ may start (see backward_sm100.cuh)
    grid_wait();
    grid_launch_dependents();
  }
  __syncthreads();

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t4 = lane & 3, mi = lane >> 3, rr = lane & 7;
  const int m0 = (warp & 3) * 16, half = warp >> 2, n0 = half * 32;
  const int D = s.head_dim;
  const MaskSpec ms = bwd_mask(s);

  // Own tile, and the steps [begin, end) of the walk over the streamed ones:
  // step i is tile first + i % count of run i / count.
  const int splits = kDQ ? p.q_splits : p.kv_splits;
  const int u = (int)(blockIdx.x / (unsigned)splits), sp = (int)(blockIdx.x % (unsigned)splits);
  long long run0, unit;
  int own_row0, own_n, first, count, begin, end;
  if (kDQ) {
    run0 = u % (int)s.runs;
    own_row0 = u / (int)s.runs * kBmTile;
    own_n = min(kBmTile, s.run - own_row0);
    unit = run0 / s.runs_per_unit;
    const KeyRange kr = key_range(ms, own_row0, own_n, kBmTile);
    first = kr.t_first;
    count = kr.t_count;
    bwd_part(count, sp, splits, begin, end);
    bwd_load_tile<KS>(own1, p.q + (run0 * s.run + own_row0) * D, D, own_n);
    bwd_load_tile<KS>(own2, p.dout + (run0 * s.run + own_row0) * D, D, own_n);
  } else {
    unit = u % (int)s.units;
    own_row0 = u / (int)s.units * kBmTile;
    own_n = min(kBmTile, s.kv_len - own_row0);
    run0 = unit * s.runs_per_unit;
    bwd_row_tiles(s, own_row0, own_row0 + own_n - 1, kBmTile, first, count);
    bwd_part(count * s.runs_per_unit, sp, splits, begin, end);
    bwd_load_tile<KS>(own1, p.k + (unit * s.kv_len + own_row0) * D, D, own_n);
    bwd_load_tile<KS>(own2, p.v + (unit * s.kv_len + own_row0) * D, D, own_n);
  }

  float acc1[KS][4], acc2[kDQ ? 1 : KS][4];  // dK or dQ; dV
#pragma unroll
  for (int i = 0; i < KS; ++i) acc1[i][0] = acc1[i][1] = acc1[i][2] = acc1[i][3] = 0.f;
#pragma unroll
  for (int i = 0; i < (kDQ ? 1 : KS); ++i) acc2[i][0] = acc2[i][1] = acc2[i][2] = acc2[i][3] = 0.f;

  // What thread t (< 192) brings of the query rows' 192 numbers.  dQ's CTAs read
  // past L1 (see the head of backward_sm100.cuh), once: the rows are their own.
  auto row_stat = [&](long long run, int q_row0) {
    const int w = threadIdx.x >> 6, r = threadIdx.x & 63;
    const float* at = p.stats + (run * s.tiles + (q_row0 >> 7)) * 256 + w * 128 + (q_row0 & 127) + r;
    return w == 2 ? __int_as_float(s.kv_len - s.q_len + (q_row0 + r) % s.q_len) : kDQ ? __ldcg(at) : *at;
  };
  if (kDQ && threadIdx.x < 192) st2[threadIdx.x] = st2[192 + threadIdx.x] = row_stat(run0, own_row0);
  // Tile `it` of the walk into its buffer.
  auto fetch = [&](int it) {
    const long long run = run0 + (kDQ ? 0 : it / count);
    const int row0 = (first + it % count) * kBmTile;
    const int n = min(kBmTile, (kDQ ? s.kv_len : s.run) - row0);
    __nv_bfloat16* s1 = str + ((it - begin) & 1) * 2 * C::kTileElems;
    const long long off = (kDQ ? unit * s.kv_len + row0 : run * s.run + row0) * (long long)D;
    bwd_load_tile<KS>(s1, (kDQ ? p.k : p.q) + off, D, n);
    bwd_load_tile<KS>(s1 + C::kTileElems, (kDQ ? p.v : p.dout) + off, D, n);
    if (!kDQ && threadIdx.x < 192) st2[((it - begin) & 1) * 192 + threadIdx.x] = row_stat(run, row0);
    cp_async_commit();
  };
  if (begin < end) {
    fetch(begin);
  } else {  // never leave with copies in flight
    cp_async_commit();
    cp_async_wait<0>();
  }
  for (int it = begin; it < end; ++it) {
    const int str_row0 = (first + it % count) * kBmTile;
    const int q_row0 = kDQ ? own_row0 : str_row0, k_row0 = kDQ ? str_row0 : own_row0;
    const bool need_mask =
        bwd_need_mask(s, ms, q_row0, min(kBmTile, s.run - q_row0), k_row0, kBmTile);
    const __nv_bfloat16* str1 = str + ((it - begin) & 1) * 2 * C::kTileElems;
    const __nv_bfloat16* str2 = str1 + C::kTileElems;
    const float* st = st2 + ((it - begin) & 1) * 192;
    if (it + 1 < end) {  // its buffer was last read before the loop's closing barrier
      fetch(it + 1);
      cp_async_wait<1>();
    } else {
      cp_async_wait<0>();
    }
    __syncthreads();

    // S (or S^T) and dP (or dP^T): 16 own rows x 32 streamed rows.
    float sc[4][4], dp[4][4];
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) sc[n][e] = dp[n][e] = 0.f;
    {
      const uint32_t aoff = ((m0 + (lane & 15)) * C::kPitch + (lane >> 4) * 8) * 2;
      const uint32_t boff = ((n0 + (mi >> 1) * 8 + rr) * C::kPitch + (mi & 1) * 8) * 2;
      const uint32_t a1 = smem_u32(own1) + aoff, a2 = smem_u32(own2) + aoff;
      const uint32_t b1 = smem_u32(str1) + boff, b2 = smem_u32(str2) + boff;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        uint32_t x0, x1, x2, x3, y0, y1, y2, y3;
        ldsm_x4(a1 + ks * 32, x0, x1, x2, x3);
        ldsm_x4(a2 + ks * 32, y0, y1, y2, y3);
#pragma unroll
        for (int n = 0; n < 4; n += 2) {
          uint32_t c0, c1, c2, c3;
          ldsm_x4(b1 + n * 8 * C::kPitch * 2 + ks * 32, c0, c1, c2, c3);
          mma_16816(sc[n], x0, x1, x2, x3, c0, c1);
          mma_16816(sc[n + 1], x0, x1, x2, x3, c2, c3);
          ldsm_x4(b2 + n * 8 * C::kPitch * 2 + ks * 32, c0, c1, c2, c3);
          mma_16816(dp[n], y0, y1, y2, y3, c0, c1);
          mma_16816(dp[n + 1], y0, y1, y2, y3, c2, c3);
        }
      }
    }
    // P and dS in place of S and dP; hidden pairs become zeros, whatever they
    // were.  Element e of piece n: own row m0 + g + 8 (e / 2), streamed row
    // n0 + 8 n + 2 t4 + e % 2.
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int qr = kDQ ? m0 + g + 8 * (e >> 1) : n0 + n * 8 + 2 * t4 + (e & 1);
        float slope = 1.f, y;
        if (p.softcap) {
          y = p.cap_out * tanh_accurate(sc[n][e] * p.cap_in, slope);
        } else {
          y = sc[n][e] * p.logit_scale;
        }
        sc[n][e] = ex2(y + st[qr]);
        dp[n][e] = sc[n][e] * (dp[n][e] - st[64 + qr]) * slope;
      }
    if (need_mask) {
#pragma unroll
      for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int own = m0 + g + 8 * (e >> 1), col = n0 + n * 8 + 2 * t4 + (e & 1);
          const int key = k_row0 + (kDQ ? col : own), qpos = __float_as_int(st[128 + (kDQ ? own : col)]);
          if (key < first_key(ms, qpos) || key > last_key(ms, qpos)) sc[n][e] = dp[n][e] = 0.f;
        }
    }
    // Rounded to bf16 for the tensor cores as the forward's P is; when fine, a
    // second round with what the first rounding left.
    auto products = [&]() {
#pragma unroll
      for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int off = (m0 + g + 8 * h) * C::kPPitch + n0 + n * 8 + 2 * t4;
          if (!kDQ) *(uint32_t*)(pm + off) = bwd_take_bf16<kFine>(sc[n][2 * h], sc[n][2 * h + 1]);
          *(uint32_t*)(dm + off) = bwd_take_bf16<kFine>(dp[n][2 * h], dp[n][2 * h + 1]);
        }
      __syncthreads();
      // Outputs: 16 own rows x half of the columns, over the 64 streamed rows.
      {
        const uint32_t aoff = ((m0 + (lane & 15)) * C::kPPitch + (lane >> 4) * 8) * 2;
        const uint32_t ad = smem_u32(dm) + aoff, ap = smem_u32(pm) + aoff;
        const uint32_t boff = (((mi & 1) * 8 + rr) * C::kPitch + half * KS * 8 + (mi >> 1) * 8) * 2;
        const uint32_t b1 = smem_u32(str1) + boff, b2 = smem_u32(str2) + boff;
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
          uint32_t x0, x1, x2, x3, y0 = 0, y1 = 0, y2 = 0, y3 = 0;
          ldsm_x4(ad + ks * 32, x0, x1, x2, x3);
          if (!kDQ) ldsm_x4(ap + ks * 32, y0, y1, y2, y3);
#pragma unroll
          for (int n = 0; n < KS; n += 2) {
            uint32_t c0, c1, c2, c3;
            ldsm_x4_t(b1 + (ks * 16 * C::kPitch + n * 8) * 2, c0, c1, c2, c3);
            mma_16816(acc1[n], x0, x1, x2, x3, c0, c1);
            mma_16816(acc1[n + 1], x0, x1, x2, x3, c2, c3);
            if constexpr (!kDQ) {
              ldsm_x4_t(b2 + (ks * 16 * C::kPitch + n * 8) * 2, c0, c1, c2, c3);
              mma_16816(acc2[n], y0, y1, y2, y3, c0, c1);
              mma_16816(acc2[n + 1], y0, y1, y2, y3, c2, c3);
            }
          }
        }
      }
    };
    products();
    if constexpr (kFine) {
      __syncthreads();  // the first terms are no longer read
      products();
    }
    __syncthreads();  // the buffer, P and dS are no longer read
  }

  const long long out0 = kDQ ? run0 * s.run + own_row0 : unit * s.kv_len + own_row0;
#pragma unroll
  for (int n = 0; n < KS; ++n)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = m0 + g + 8 * h, c = half * KS * 8 + n * 8 + 2 * t4;
      if (r >= own_n || c >= D) continue;
      if (splits > 1) {
        const long long at = blockIdx.x * (long long)(kBmTile * ((D + 15) / 16 * 16)) +
                             ((c >> 2) * kBmTile + r) * 4 + (c & 3);
        *(float2*)((kDQ ? p.part_dq : p.part_dk) + at) = make_float2(acc1[n][2 * h], acc1[n][2 * h + 1]);
        if constexpr (!kDQ)
          *(float2*)(p.part_dv + at) = make_float2(acc2[n][2 * h], acc2[n][2 * h + 1]);
        continue;
      }
      const long long off = (out0 + r) * D + c;
      *(uint32_t*)((kDQ ? p.dq : p.dk) + off) =
          pack_bf16(acc1[n][2 * h] * p.scale, acc1[n][2 * h + 1] * p.scale);
      if constexpr (!kDQ)
        *(uint32_t*)(p.dv + off) = pack_bf16(acc2[n][2 * h], acc2[n][2 * h + 1]);
    }
  // One CTA is enough: the kernel has not ended before it has.
  if (kDQ && blockIdx.x == gridDim.x - 1 && threadIdx.x == 0) grid_wait();
}

}  // namespace gqa
