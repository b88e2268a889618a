// backward_sm100.cuh -- the backward pass on the 5th-generation tensor cores
// (head_dim up to 128); backward.cuh has the formulas and the row layout.
//
// Two kernels with the same frame, one CTA of 12 warps per tile of 128 and
// per SM:
//   warp 0      TMA loader (and the statistics' bulk copies);
//   warp 1      TMEM allocator; its lane 0 issues every tcgen05.mma;
//   warps 2-3   idle (they complete warpgroup 0 for the register split);
//   warps 4-11  elementwise work: warpgroup h takes columns [64 h, 64 h + 64)
//               of the 128 x 128 tiles, a thread one lane (row) of them.
//
// bwd_dkdv_kernel: one key tile.  K and V stay in shared memory, the row
// tiles of every q head of the group stream by (Q through three slots, dO
// through two).  Scores are computed transposed, keys as lanes:
//   S^T = K Q^T, dP^T = V dO^T    (both operands from shared memory)
//   dV += P^T dO, dK += dS^T Q    (A = P^T, dS^T as bf16 from TMEM, written
//                                  over the scores they came from)
// so that P^T and dS^T never leave TMEM.  TMEM is full: S^T [0, 128), dP^T
// [128, 256), dV [256, 384), dK [384, 512).  The elementwise warps alternate
// between P^T (from S^T) and dS^T (from dP^T); while they make one, the
// tensor core runs the two products that the other one feeds and frees:
//   P^T_j done  -> dV += P^T_j dO_j,  S^T_{j+1}
//   dS^T_j done -> dK += dS^T_j Q_j,  dP^T_{j+1}
//
// bwd_dq_kernel: one row tile.  Q and dO stay, key tiles stream (K through
// three slots, V through two), rows are lanes:
//   S = Q K^T (two buffers), dP = dO V^T, dQ += dS K (A = dS from TMEM).
// TMEM: S [0, 256), dP [256, 384), dQ [384, 512).
//
// P is recomputed as 2^(x - lse) with both in log2 units: the statistics are
// known, so there is no running maximum and nothing to rescale.  The fp32 P
// stays in registers between the two elementwise halves of a tile.
// All waits are bounded.
#pragma once

#include "backward.cuh"
#include "ptx.cuh"

namespace gqa {

constexpr int kBwThreads = 384;
// Registers: 4 * 32 * 88 + 8 * 32 * 208 = 64,512 = 384 threads x 168 at launch
// (checked by the host before the first launch).
constexpr int kBwRegsLow = 88;
constexpr int kBwRegsHigh = 208;
constexpr int kBwRegTotal = 4 * 32 * kBwRegsLow + 8 * 32 * kBwRegsHigh;

template <int DCH>
struct BwdCfg {
  static constexpr int kBoxBytes = 128 * 128;         // 128 rows x 64 bf16
  static constexpr int kTileBytes = DCH * kBoxBytes;  // one 128-row operand tile
  // Two resident tiles, three slots of one streamed operand, two of the other.
  static constexpr int kRing3 = 2 * kTileBytes;
  static constexpr int kRing2 = kRing3 + 3 * kTileBytes;
  static constexpr int kStats = kRing2 + 2 * kTileBytes;  // two slots of 256 floats
  static constexpr int kBars = kStats + 2 * 1024;
  static constexpr int kNumBars = 24;
  static constexpr int kSmemBytes = kBars + kNumBars * 8 + 16;
};

// Whether any row of a row tile fails to see any key of a key tile: only then
// are scores masked one by one.
__device__ __forceinline__ bool bwd_need_mask(const BwdShape& s, const MaskSpec& ms, int r0, int nr,
                                              int k0) {
  if (!(s.causal || s.window > 0)) return k0 + 127 >= s.kv_len;
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
  return !(k0 >= first_key(ms, base + i1) && k0 + 127 <= last_key(ms, base + i0));
}

// P of 32 columns from 32 raw scores (nl: -lse of their rows, in pairs), and
// with a softcap the factors 1 - tanh^2 that dS takes.  The last pairs of
// every 16 take 2^x from the FMA pipe: MUFU alone would need 1024 cycles for
// a 128 x 128 tile, half of the tensor core's time for the tile's products.
constexpr int kBwEmuFrom = 13;
template <bool kCap>
__device__ __forceinline__ void bwd_probs(const BwdParams& p, const uint32_t (&s)[32],
                                          const f2 (&nl)[16], f2 (&pr)[16], f2 (&fac)[16]) {
  if constexpr (!kCap) {
    const f2 sc = f2_pack(p.logit_scale, p.logit_scale);
#pragma unroll
    for (int c = 0; c < 16; ++c) {
      const f2 y = f2_fma(f2_pack(__uint_as_float(s[2 * c]), __uint_as_float(s[2 * c + 1])), sc, nl[c]);
      pr[c] = c >= kBwEmuFrom ? exp2_poly_x2(y) : exp2_mufu_x2(y);
    }
  } else {
    float am = 0.f;
#pragma unroll
    for (int c = 0; c < 32; c += 2)
      am = fmax3(am, fabsf(__uint_as_float(s[c])), fabsf(__uint_as_float(s[c + 1])));
    const bool small = __all_sync(0xffffffffu, am * p.cap_in <= 0.5f);
    const f2 co = f2_pack(p.cap_out, p.cap_out), one = f2_pack(1.f, 1.f);
    if (small) {
      const f2 ci = f2_pack(p.cap_in, p.cap_in), nci = f2_pack(-p.cap_in, -p.cap_in);
      const f2 c3 = f2_pack(kTanh9C3, kTanh9C3), c5 = f2_pack(kTanh9C5, kTanh9C5);
      const f2 c7 = f2_pack(kTanh9C7, kTanh9C7), c9 = f2_pack(kTanh9C9, kTanh9C9);
#pragma unroll
      for (int c = 0; c < 16; ++c) {
        const f2 x = f2_pack(__uint_as_float(s[2 * c]), __uint_as_float(s[2 * c + 1]));
        const f2 y = f2_mul(x, ci), y2 = f2_mul(y, y);
        const f2 q = f2_fma(f2_fma(f2_fma(f2_fma(c9, y2, c7), y2, c5), y2, c3), y2, one);
        const f2 t = f2_mul(y, q);
        pr[c] = exp2_mufu_x2(f2_fma(co, t, nl[c]));
        fac[c] = f2_fma(t, f2_mul(f2_mul(x, nci), q), one);
      }
    } else {
#pragma unroll
      for (int c = 0; c < 16; ++c) {
        const float a = tanh_accurate(__uint_as_float(s[2 * c]) * p.cap_in);
        const float b = tanh_accurate(__uint_as_float(s[2 * c + 1]) * p.cap_in);
        pr[c] = exp2_mufu_x2(f2_fma(co, f2_pack(a, b), nl[c]));
        fac[c] = f2_pack(fmaf(-a, a, 1.f), fmaf(-b, b, 1.f));
      }
    }
  }
}

// dS of 32 columns as bf16 from what bwd_probs left (p times the factor), dP
// and the rows' delta.  A hidden score is an exact zero whatever dP is.
__device__ __forceinline__ void bwd_ds(const f2* keep, const uint32_t (&dp)[32], const f2 (&dl)[16],
                                       bool masked, uint32_t (&pk)[16]) {
  f2 d[16];
#pragma unroll
  for (int c = 0; c < 16; ++c)
    d[c] = f2_mul(keep[c], f2_sub(f2_pack(__uint_as_float(dp[2 * c]), __uint_as_float(dp[2 * c + 1])),
                                  dl[c]));
  if (masked) {
#pragma unroll
    for (int c = 0; c < 16; ++c) {
      float k0, k1, a, b;
      f2_unpack(keep[c], k0, k1);
      f2_unpack(d[c], a, b);
      d[c] = f2_pack(k0 == 0.f ? 0.f : a, k1 == 0.f ? 0.f : b);
    }
  }
#pragma unroll
  for (int c = 0; c < 16; ++c) pk[c] = pack_bf16_f2(d[c]);
}

// 32 floats of shared memory, the same for every lane, as pairs.
__device__ __forceinline__ void bwd_load32(const float* src, f2 (&v)[16]) {
#pragma unroll
  for (int c = 0; c < 16; c += 2) {
    const ulonglong2 w = *reinterpret_cast<const ulonglong2*>(src + 2 * c);
    v[c] = w.x;
    v[c + 1] = w.y;
  }
}

// One 128 x 64-column piece of TMEM (this warp's 32 lanes) scaled, rounded to
// bf16 and stored through a swizzled 32-row box and TMA; rows and columns
// outside the tensor are not written.
__device__ __forceinline__ void bwd_store_box(const CUtensorMap* map, uint8_t* stage, uint32_t tm,
                                              int c0, int cols, int row, int outer, float scale,
                                              bool zero, int lane) {
  if (lane == 0) bulk_wait_read();
  __syncwarp();
  for (int c1 = 0; c1 < cols; c1 += 16) {
    uint32_t v[16];
    if (zero) {
#pragma unroll
      for (int e = 0; e < 16; ++e) v[e] = 0u;
    } else {
      tmem_ld16(tm + c0 + c1, v);
      tmem_ld_wait();
    }
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        w[e] = pack_bf16(__uint_as_float(v[8 * g + 2 * e]) * scale,
                         __uint_as_float(v[8 * g + 2 * e + 1]) * scale);
      *reinterpret_cast<uint4*>(stage + sw128(lane, (c1 >> 3) + g)) =
          make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) {
    tma_store_3d(map, stage, c0, row, outer);
    bulk_commit();
  }
}

// The products, 8 K-steps of 16 unless K is head_dim.  Shared memory lies
// below 256 KB, so a descriptor's 14-bit address field never carries out and
// a K-step is one addition to its low word.
// A and B K-major from shared memory (128 x 128, K = head_dim):
template <int DCH>
__device__ __forceinline__ void bwd_issue_ss(uint32_t leader, uint32_t d, uint64_t ad, uint64_t bd,
                                             uint32_t idesc, int ksteps) {
  using C = BwdCfg<DCH>;
#pragma unroll
  for (int ks = 0; ks < 4 * DCH; ++ks) {
    if (ks >= ksteps) break;
    const uint32_t off = ((ks >> 2) * C::kBoxBytes + (ks & 3) * 32) >> 4;
    mma_bf16_ss_warp(leader, d, ad + off, bd + off, idesc, ks > 0);
  }
}
// A (128 x 128 bf16) from TMEM: columns 0..63 of the tile at a, 64..127 at
// a + 64; B (128 x N) from shared memory, N contiguous.  K-steps [k0, k1) of
// both halves.
__device__ __forceinline__ void bwd_issue_ts(uint32_t leader, uint32_t d, uint32_t a, uint64_t bd,
                                             uint32_t idesc, bool first, int k0, int k1) {
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int ks = k0; ks < k1; ++ks)
      mma_bf16_ts_warp(leader, d, a + h * 64 + ks * 8, bd + (4 * h + ks) * (2048 >> 4), idesc,
                       !(first && h == 0 && ks == 0));
}
// Descriptors of a tile as either operand of bwd_issue_ss, and as the B of
// bwd_issue_ts.
__device__ __forceinline__ uint64_t bwd_desc_k(uint32_t tile) { return sdesc_sw128(tile, 16, 1024); }
template <int DCH>
__device__ __forceinline__ uint64_t bwd_desc_n(uint32_t tile) {
  return sdesc_sw128(tile, BwdCfg<DCH>::kBoxBytes, 1024);
}

// ------------------------------------------------------------------ dK, dV
template <int DCH, bool kCap>
__global__ void __launch_bounds__(kBwThreads, 1)
    bwd_dkdv_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_do,
                    const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                    const __grid_constant__ CUtensorMap tm_dk, const __grid_constant__ CUtensorMap tm_dv,
                    const BwdParams p) {
  using C = BwdCfg<DCH>;
  const BwdShape& s = p.sh;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* sk = smem;
  uint8_t* sv = smem + C::kTileBytes;
  uint8_t* sq = smem + C::kRing3;
  uint8_t* sdo = smem + C::kRing2;
  float* stats = (float*)(smem + C::kStats);
  uint64_t* bars = (uint64_t*)(smem + C::kBars);
  uint64_t* kv_full = bars;
  uint64_t* q_full = bars + 1;    // [3]
  uint64_t* q_empty = bars + 4;   // [3]
  uint64_t* do_full = bars + 7;   // [2]
  uint64_t* do_empty = bars + 9;  // [2]
  uint64_t* st_full = bars + 11;  // [2]
  uint64_t* st_empty = bars + 13; // [2]
  uint64_t* s_full = bars + 15;
  uint64_t* dp_full = bars + 16;
  uint64_t* p_full = bars + 17;
  uint64_t* ds_full = bars + 18;
  uint64_t* o_done = bars + 19;
  uint64_t* p_half = bars + 20;
  uint32_t* tmem_slot = (uint32_t*)(bars + C::kNumBars);

  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    mbar_init(kv_full, 1);
    for (int i = 0; i < 3; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&do_full[i], 1);
      mbar_init(&do_empty[i], 1);
      mbar_init(&st_full[i], 1);
      mbar_init(&st_empty[i], 8);
    }
    mbar_init(s_full, 1);
    mbar_init(dp_full, 1);
    mbar_init(p_half, 8);
    mbar_init(p_full, 8);
    mbar_init(ds_full, 8);
    mbar_init(o_done, 1);
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // Key tiles in ascending order: under a causal mask the first ones have the
  // most rows, so the light ones fill the last wave.
  const int unit = (int)(blockIdx.x % (unsigned)s.units);
  const int k0 = (int)(blockIdx.x / (unsigned)s.units) * 128;
  int first, count;
  bwd_row_tiles(s, k0, min(k0 + 127, s.kv_len - 1), 128, first, count);
  const int n = count * s.runs_per_unit;
  const int run0 = unit * s.runs_per_unit;

  if (warp < 4) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kBwRegsLow));
  if (warp == 0) {
    if (lane == 0 && n > 0) {
      tma_prefetch_map(&tm_q);
      tma_prefetch_map(&tm_do);
      mbar_arrive_expect_tx(kv_full, 2 * C::kTileBytes);
      for (int c = 0; c < DCH; ++c)
        tma_load_3d(sk + c * C::kBoxBytes, &tm_k, kv_full, c * 64, k0, unit);
      for (int c = 0; c < DCH; ++c)
        tma_load_3d(sv + c * C::kBoxBytes, &tm_v, kv_full, c * 64, k0, unit);
      int jq = 0, jd = 0, js = 0;  // loads issued
      int run = run0, t = first;
      for (int j = 0; j < n; ++j) {
        if (j >= 3 && !mbar_wait(&q_empty[j % 3], (j / 3 - 1) & 1, kStatusTimeoutProducer)) break;
        mbar_arrive_expect_tx(&q_full[j % 3], C::kTileBytes);
        for (int c = 0; c < DCH; ++c)
          tma_load_3d(sq + (j % 3) * C::kTileBytes + c * C::kBoxBytes, &tm_q, &q_full[j % 3], c * 64,
                      t * 128, run);
        ++jq;
        if (j >= 2 && !mbar_wait(&do_empty[j & 1], (j / 2 - 1) & 1, kStatusTimeoutProducer)) break;
        mbar_arrive_expect_tx(&do_full[j & 1], C::kTileBytes);
        for (int c = 0; c < DCH; ++c)
          tma_load_3d(sdo + (j & 1) * C::kTileBytes + c * C::kBoxBytes, &tm_do, &do_full[j & 1],
                      c * 64, t * 128, run);
        ++jd;
        if (j >= 2 && !mbar_wait(&st_empty[j & 1], (j / 2 - 1) & 1, kStatusTimeoutProducer)) break;
        mbar_arrive_expect_tx(&st_full[j & 1], 1024);
        bulk_load(stats + (j & 1) * 256, p.stats + ((long long)run * s.tiles + t) * 256, 1024,
                  &st_full[j & 1]);
        ++js;
        if (++t == first + count) {
          t = first;
          ++run;
        }
      }
      // Never leave with copies in flight.
      mbar_wait(kv_full, 0, kStatusTimeoutProducer);
      for (int j = max(0, jq - 3); j < jq; ++j)
        mbar_wait(&q_full[j % 3], (j / 3) & 1, kStatusTimeoutProducer);
      for (int j = max(0, jd - 2); j < jd; ++j)
        mbar_wait(&do_full[j & 1], (j / 2) & 1, kStatusTimeoutProducer);
      for (int j = max(0, js - 2); j < js; ++j)
        mbar_wait(&st_full[j & 1], (j / 2) & 1, kStatusTimeoutProducer);
    }
  } else if (warp == 1) {
    // The whole warp walks the loop, lane 0 issues (see mma_bf16_ss_warp).
    if (n > 0) {
      const uint32_t leader = lane == 0;
      const int d_pad = (s.head_dim + 15) / 16 * 16, ksteps = d_pad / 16;
      const uint32_t idesc_s = idesc_bf16_f32(128, 128, 0);
      const uint32_t idesc_o = idesc_bf16_f32(128, d_pad, 1);
      const uint64_t kd = bwd_desc_k(smem_u32(sk)), vd = bwd_desc_k(smem_u32(sv));
      const uint64_t qk = bwd_desc_k(smem_u32(sq)), qn = bwd_desc_n<DCH>(smem_u32(sq));
      const uint64_t dk = bwd_desc_k(smem_u32(sdo)), dn = bwd_desc_n<DCH>(smem_u32(sdo));
      constexpr uint32_t kTile = C::kTileBytes >> 4;  // a slot, in descriptor units
      // Uniform over the warp, so that it stays converged.
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        return __all_sync(0xffffffffu, mbar_wait(bar, parity, kStatusTimeoutMma)) != 0;
      };
      bool ok = wait(kv_full, 0) && wait(&q_full[0], 0);
      if (ok) {
        tc_fence_after();
        bwd_issue_ss<DCH>(leader, tmem, kd, qk, idesc_s, ksteps);
        mma_commit_warp(leader, s_full);
      }
      int sq_j = 0, sq_n = 1;  // Q slots of tiles j and j + 1
      ok = ok && wait(&do_full[0], 0);
      for (int j = 0; j < n && ok; ++j) {
        const uint32_t doj = (j & 1) * kTile;
        const bool more = j + 1 < n;
        tc_fence_after();
        bwd_issue_ss<DCH>(leader, tmem + 128, vd, dk + doj, idesc_s, ksteps);
        mma_commit_warp(leader, dp_full);
        // dV in two parts: rows 0..31 and 64..95 of the tile first.
        if (!(ok = wait(p_half, j & 1))) break;
        tc_fence_after();
        bwd_issue_ts(leader, tmem + 256, tmem, dn + doj, idesc_o, j == 0, 0, 2);
        // The next tile's operands are waited for ahead of their turn.
        if (more && !(ok = wait(&q_full[sq_n], ((j + 1) / 3) & 1))) break;
        if (!(ok = wait(p_full, j & 1))) break;
        tc_fence_after();
        bwd_issue_ts(leader, tmem + 256, tmem, dn + doj, idesc_o, false, 2, 4);
        mma_commit_warp(leader, &do_empty[j & 1]);
        if (more) {
          bwd_issue_ss<DCH>(leader, tmem, kd, qk + sq_n * kTile, idesc_s, ksteps);
          mma_commit_warp(leader, s_full);
          if (!(ok = wait(&do_full[(j + 1) & 1], ((j + 1) / 2) & 1))) break;
        }
        if (!(ok = wait(ds_full, j & 1))) break;
        tc_fence_after();
        bwd_issue_ts(leader, tmem + 384, tmem + 128, qn + sq_j * kTile, idesc_o, j == 0, 0, 4);
        mma_commit_warp(leader, &q_empty[sq_j]);
        sq_j = sq_n;
        if (++sq_n == 3) sq_n = 0;
      }
      // Every product finished before the epilogue, and before TMEM is freed.
      mma_commit_warp(leader, o_done);
      wait(o_done, 0);
    }
  } else if (warp >= 4) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kBwRegsHigh));
    const int h = (warp - 4) >> 2, quarter = warp & 3;
    const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
    const uint32_t s_tm = tmem + lane_base + 64 * h, dp_tm = s_tm + 128;
    const int key = k0 + quarter * 32 + lane;
    const MaskSpec ms = bwd_mask(s);
    // Queries that see this lane's key: [qlo, qlo + qspan] (none past kv_len).
    int qlo, qhi;
    bwd_query_range(s, key, key, qlo, qhi);
    if (key >= s.kv_len || qhi < qlo) {
      qlo = 0x7fffffff;
      qhi = 0x7fffffff;
    }
    const unsigned qspan = (unsigned)(qhi - qlo);
    bool ok = true;
    int run = run0, t = first;
    for (int j = 0; j < n; ++j) {
      const int r0 = t * 128, nr = min(128, s.run - r0);
      const bool need_mask = bwd_need_mask(s, ms, r0, nr, k0);
      f2 keep[32];
      const float* st = stats + (j & 1) * 256 + 64 * h;
      ok = mbar_wait(&st_full[j & 1], (j / 2) & 1, kStatusTimeoutSoftmax) &&
           mbar_wait(s_full, j & 1, kStatusTimeoutSoftmax);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      uint32_t b0[32], b1[32];
      tmem_ld32(s_tm, b0);
      int qi = need_mask ? (r0 + 64 * h) % s.q_len : 0;  // query of the next column
      // P of columns 32 g .. 32 g + 31 of this half, into TMEM columns
      // [16 g, 16 g + 16) of it, whose scores have been read.
      auto probs = [&](const uint32_t(&sv32)[32], int g) {
        f2 nl[16], pr[16], fac[16];
        bwd_load32(st + 32 * g, nl);
        bwd_probs<kCap>(p, sv32, nl, pr, fac);
        if (need_mask) {
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            float a, b;
            f2_unpack(pr[c], a, b);
            if ((unsigned)(qi - qlo) > qspan) a = 0.f;
            if (++qi == s.q_len) qi = 0;
            if ((unsigned)(qi - qlo) > qspan) b = 0.f;
            if (++qi == s.q_len) qi = 0;
            pr[c] = f2_pack(a, b);
          }
        }
        uint32_t pk[16];
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          pk[c] = pack_bf16_f2(pr[c]);
          keep[16 * g + c] = kCap ? f2_mul(pr[c], fac[c]) : pr[c];
        }
        tmem_st16(s_tm + 16 * g, pk);
      };
      tmem_ld_wait();
      tmem_ld32(s_tm + 32, b1);
      probs(b0, 0);
      tmem_ld_wait();  // the second half is read before the first part is handed over
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(p_half);
      probs(b1, 1);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(p_full);

      f2 dl[16];
      bwd_load32(st + 128, dl);
      ok = __all_sync(0xffffffffu, mbar_wait(dp_full, j & 1, kStatusTimeoutSoftmax));
      if (!ok) break;
      tc_fence_after();
      uint32_t pk[16];
      tmem_ld32(dp_tm, b0);
      tmem_ld32(dp_tm + 32, b1);
      tmem_ld_wait();
      bwd_ds(keep, b0, dl, need_mask, pk);
      tmem_st16(dp_tm, pk);
      bwd_load32(st + 160, dl);
      bwd_ds(keep + 16, b1, dl, need_mask, pk);
      tmem_st16(dp_tm + 16, pk);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(ds_full);
        mbar_arrive(&st_empty[j & 1]);
      }
      if (++t == first + count) {
        t = first;
        ++run;
      }
    }
    if (n > 0 && ok)
      ok = __all_sync(0xffffffffu, mbar_wait(o_done, 0, kStatusTimeoutEpilogue));
    if (ok) {
      tc_fence_after();
      // Warpgroup 0 stores dV, warpgroup 1 dK, through boxes in the Q ring
      // (every load into it has been consumed).
      uint8_t* stage = sq + (warp - 4) * 4096;
      const int d_pad = (s.head_dim + 15) / 16 * 16;
      for (int c0 = 0; c0 < d_pad && k0 + quarter * 32 < s.kv_len; c0 += 64)
        bwd_store_box(h ? &tm_dk : &tm_dv, stage, tmem + lane_base + 256 + 128 * h, c0,
                      min(64, d_pad - c0), k0 + quarter * 32, unit, h ? p.scale : 1.f, n == 0, lane);
      if (lane == 0) bulk_wait_all();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------------ dQ
template <int DCH, bool kCap>
__global__ void __launch_bounds__(kBwThreads, 1)
    bwd_dq_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_do,
                  const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                  const __grid_constant__ CUtensorMap tm_dq, const BwdParams p) {
  using C = BwdCfg<DCH>;
  const BwdShape& s = p.sh;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* sq = smem;
  uint8_t* sdo = smem + C::kTileBytes;
  uint8_t* sk = smem + C::kRing3;
  uint8_t* sv = smem + C::kRing2;
  uint64_t* bars = (uint64_t*)(smem + C::kBars);
  uint64_t* q_full = bars;
  uint64_t* k_full = bars + 1;   // [3]
  uint64_t* k_empty = bars + 4;  // [3]
  uint64_t* v_full = bars + 7;   // [2]
  uint64_t* v_empty = bars + 9;  // [2]
  uint64_t* s_full = bars + 11;  // [2]
  uint64_t* dp_full = bars + 13;
  uint64_t* ds_full = bars + 14;
  uint64_t* o_done = bars + 15;
  uint32_t* tmem_slot = (uint32_t*)(bars + C::kNumBars);

  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    for (int i = 0; i < 3; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&k_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&v_full[i], 1);
      mbar_init(&v_empty[i], 1);
      mbar_init(&s_full[i], 1);
    }
    mbar_init(dp_full, 1);
    mbar_init(ds_full, 8);
    mbar_init(o_done, 1);
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // Row tiles in descending order: under a causal mask the last ones have the
  // most keys.  Runs of one kv head follow each other and share K and V in L2.
  const int run = (int)(blockIdx.x % (unsigned)s.runs);
  const int t = s.tiles - 1 - (int)(blockIdx.x / (unsigned)s.runs);
  const int r0 = t * 128, nr = min(128, s.run - r0);
  const int unit = run / s.runs_per_unit;
  const MaskSpec ms = bwd_mask(s);
  const KeyRange kr = key_range(ms, r0, nr, 128);
  const int n = kr.t_count;

  if (warp < 4) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kBwRegsLow));
  if (warp == 0) {
    if (lane == 0 && n > 0) {
      tma_prefetch_map(&tm_k);
      tma_prefetch_map(&tm_v);
      mbar_arrive_expect_tx(q_full, 2 * C::kTileBytes);
      for (int c = 0; c < DCH; ++c)
        tma_load_3d(sq + c * C::kBoxBytes, &tm_q, q_full, c * 64, r0, run);
      for (int c = 0; c < DCH; ++c)
        tma_load_3d(sdo + c * C::kBoxBytes, &tm_do, q_full, c * 64, r0, run);
      int jk = 0, jv = 0;
      for (int j = 0; j < n; ++j) {
        const int key0 = (kr.t_first + j) * 128;
        if (j >= 3 && !mbar_wait(&k_empty[j % 3], (j / 3 - 1) & 1, kStatusTimeoutProducer)) break;
        mbar_arrive_expect_tx(&k_full[j % 3], C::kTileBytes);
        for (int c = 0; c < DCH; ++c)
          tma_load_3d(sk + (j % 3) * C::kTileBytes + c * C::kBoxBytes, &tm_k, &k_full[j % 3], c * 64,
                      key0, unit);
        ++jk;
        if (j >= 2 && !mbar_wait(&v_empty[j & 1], (j / 2 - 1) & 1, kStatusTimeoutProducer)) break;
        mbar_arrive_expect_tx(&v_full[j & 1], C::kTileBytes);
        for (int c = 0; c < DCH; ++c)
          tma_load_3d(sv + (j & 1) * C::kTileBytes + c * C::kBoxBytes, &tm_v, &v_full[j & 1], c * 64,
                      key0, unit);
        ++jv;
      }
      mbar_wait(q_full, 0, kStatusTimeoutProducer);
      for (int j = max(0, jk - 3); j < jk; ++j)
        mbar_wait(&k_full[j % 3], (j / 3) & 1, kStatusTimeoutProducer);
      for (int j = max(0, jv - 2); j < jv; ++j)
        mbar_wait(&v_full[j & 1], (j / 2) & 1, kStatusTimeoutProducer);
    }
  } else if (warp == 1) {
    // The whole warp walks the loop, lane 0 issues (see mma_bf16_ss_warp).
    if (n > 0) {
      const uint32_t leader = lane == 0;
      const int d_pad = (s.head_dim + 15) / 16 * 16, ksteps = d_pad / 16;
      const uint32_t idesc_s = idesc_bf16_f32(128, 128, 0);
      const uint32_t idesc_o = idesc_bf16_f32(128, d_pad, 1);
      const uint64_t qd = bwd_desc_k(smem_u32(sq)), dd = bwd_desc_k(smem_u32(sdo));
      const uint64_t kk = bwd_desc_k(smem_u32(sk)), kn = bwd_desc_n<DCH>(smem_u32(sk));
      const uint64_t vk = bwd_desc_k(smem_u32(sv));
      constexpr uint32_t kTile = C::kTileBytes >> 4;
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        return __all_sync(0xffffffffu, mbar_wait(bar, parity, kStatusTimeoutMma)) != 0;
      };
      auto wait_k = [&](int j) { return wait(&k_full[j % 3], (j / 3) & 1); };
      auto wait_v = [&](int j) { return wait(&v_full[j & 1], (j / 2) & 1); };
      auto issue_s = [&](int j) {
        bwd_issue_ss<DCH>(leader, tmem + 128 * (j & 1), qd, kk + j % 3 * kTile, idesc_s, ksteps);
        mma_commit_warp(leader, &s_full[j & 1]);
      };
      auto issue_dp = [&](int j) {
        bwd_issue_ss<DCH>(leader, tmem + 256, dd, vk + (j & 1) * kTile, idesc_s, ksteps);
        mma_commit_warp(leader, dp_full);
        mma_commit_warp(leader, &v_empty[j & 1]);
      };
      bool ok = wait(q_full, 0) && wait_k(0);
      if (ok) {
        tc_fence_after();
        issue_s(0);
        ok = wait_v(0);
      }
      if (ok) {
        tc_fence_after();
        issue_dp(0);
        ok = n < 2 || wait_k(1);
      }
      if (ok && n > 1) {
        tc_fence_after();
        issue_s(1);
      }
      for (int j = 0; j < n && ok; ++j) {
        // V of the next turn is waited for ahead of it.
        if (j + 1 < n && !(ok = wait_v(j + 1))) break;
        // dS_j written: dP_j and S_j have been read.
        if (!(ok = wait(ds_full, j & 1))) break;
        tc_fence_after();
        if (j + 1 < n) issue_dp(j + 1);
        bwd_issue_ts(leader, tmem + 384, tmem + 128 * (j & 1), kn + j % 3 * kTile, idesc_o, j == 0, 0, 4);
        mma_commit_warp(leader, &k_empty[j % 3]);
        if (j + 2 < n) {
          if (!(ok = wait_k(j + 2))) break;
          tc_fence_after();
          issue_s(j + 2);
        }
      }
      mma_commit_warp(leader, o_done);
      wait(o_done, 0);
    }
  } else if (warp >= 4) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kBwRegsHigh));
    const int h = (warp - 4) >> 2, quarter = warp & 3;
    const int r = quarter * 32 + lane;
    const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
    const float* st = p.stats + ((long long)run * s.tiles + t) * 256;
    const float nlse = st[r], delta = st[128 + r];
    int lo = 0, hi = -1;
    if (r < nr) {
      const int qpos = s.kv_len - s.q_len + (r0 + r) % s.q_len;
      lo = first_key(ms, qpos);
      hi = last_key(ms, qpos);
    }
    bool ok = true;
    for (int j = 0; j < n; ++j) {
      const int key0 = (kr.t_first + j) * 128;
      const bool need_mask = !(key0 >= kr.all_lo && key0 + 127 <= kr.all_hi);
      const int clo = max(lo - key0, 0), chi = min(hi - key0, 127);
      const int vlo = chi >= clo ? clo : 128;
      const unsigned vspan = chi >= clo ? (unsigned)(chi - clo) : 0u;
      const uint32_t s_tm = tmem + lane_base + 128 * (j & 1) + 64 * h;
      f2 keep[32];
      ok = __all_sync(0xffffffffu, mbar_wait(&s_full[j & 1], (j / 2) & 1, kStatusTimeoutSoftmax));
      if (!ok) break;
      tc_fence_after();
      uint32_t b0[32], b1[32];
      f2 row[16];
      auto probs = [&](const uint32_t(&sv32)[32], int g) {
        f2 pr[16], fac[16];
#pragma unroll
        for (int c = 0; c < 16; ++c) row[c] = f2_pack(nlse, nlse);
        bwd_probs<kCap>(p, sv32, row, pr, fac);
        if (need_mask) {
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            const int col = 64 * h + 32 * g + 2 * c;
            float a, b;
            f2_unpack(pr[c], a, b);
            pr[c] = f2_pack((unsigned)(col - vlo) > vspan ? 0.f : a,
                            (unsigned)(col + 1 - vlo) > vspan ? 0.f : b);
          }
        }
#pragma unroll
        for (int c = 0; c < 16; ++c) keep[16 * g + c] = kCap ? f2_mul(pr[c], fac[c]) : pr[c];
      };
      tmem_ld32(s_tm, b0);
      tmem_ld_wait();
      tmem_ld32(s_tm + 32, b1);
      probs(b0, 0);
      tmem_ld_wait();
      probs(b1, 1);
      ok = __all_sync(0xffffffffu, mbar_wait(dp_full, j & 1, kStatusTimeoutSoftmax));
      if (!ok) break;
      tc_fence_after();
      uint32_t pk[16];
      tmem_ld32(tmem + lane_base + 256 + 64 * h, b0);
      tmem_ld32(tmem + lane_base + 288 + 64 * h, b1);
#pragma unroll
      for (int c = 0; c < 16; ++c) row[c] = f2_pack(delta, delta);
      tmem_ld_wait();
      bwd_ds(keep, b0, row, need_mask, pk);
      tmem_st16(s_tm, pk);
      bwd_ds(keep + 16, b1, row, need_mask, pk);
      tmem_st16(s_tm + 16, pk);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(ds_full);
    }
    if (n > 0 && ok)
      ok = __all_sync(0xffffffffu, mbar_wait(o_done, 0, kStatusTimeoutEpilogue));
    if (ok) {
      tc_fence_after();
      uint8_t* stage = sk + (warp - 4) * 4096;
      const int d_pad = (s.head_dim + 15) / 16 * 16, c0 = 64 * h;
      if (c0 < d_pad && quarter * 32 < nr)
        bwd_store_box(&tm_dq, stage, tmem + lane_base + 384, c0, min(64, d_pad - c0),
                      r0 + quarter * 32, run, p.scale, n == 0, lane);
      if (lane == 0) bulk_wait_all();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace gqa
