// backward_sm100.cuh -- the backward pass on the 5th-generation tensor cores
// (head_dim up to 128); backward.cuh has the formulas and the row layout.
//
// Two kernels with the same frame, one CTA of 12 warps per tile of 128 and
// per SM:
//   warp 0      TMA loader (and the statistics' bulk copies);
//   warp 1      TMEM allocator, and the thread that issues every tcgen05.mma;
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

// P of 32 columns from 32 raw scores: 2^(x - lse), and with a softcap the
// factor (1 - tanh^2) for dS folded into `keep` (else keep = p).
template <bool kCap>
__device__ __forceinline__ void bwd_probs(const BwdParams& p, const uint32_t (&s)[32],
                                          const float (&lse)[32], float (&pr)[32], float* keep) {
  if constexpr (!kCap) {
    const f2 sc = f2_pack(p.logit_scale, p.logit_scale);
#pragma unroll
    for (int c = 0; c < 32; c += 2) {
      const f2 y = f2_fma(f2_pack(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), sc,
                          f2_pack(-lse[c], -lse[c + 1]));
      f2_unpack(exp2_mufu_x2(y), pr[c], pr[c + 1]);
      keep[c] = pr[c];
      keep[c + 1] = pr[c + 1];
    }
  } else {
    float am = 0.f;
#pragma unroll
    for (int c = 0; c < 32; c += 2)
      am = fmax3(am, fabsf(__uint_as_float(s[c])), fabsf(__uint_as_float(s[c + 1])));
    const bool small = __all_sync(0xffffffffu, am * p.cap_in <= 0.5f);
    if (small) {
#pragma unroll
      for (int c = 0; c < 32; ++c) {
        const float t = tanh_poly9_small(__uint_as_float(s[c]) * p.cap_in);
        pr[c] = ex2(fmaf(p.cap_out, t, -lse[c]));
        keep[c] = pr[c] * fmaf(-t, t, 1.f);
      }
    } else {
#pragma unroll
      for (int c = 0; c < 32; ++c) {
        const float t = tanh_accurate(__uint_as_float(s[c]) * p.cap_in);
        pr[c] = ex2(fmaf(p.cap_out, t, -lse[c]));
        keep[c] = pr[c] * fmaf(-t, t, 1.f);
      }
    }
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

// The products' issue loops.  A and B K-major from shared memory (128 x 128,
// K = head_dim):
template <int DCH>
__device__ __forceinline__ void bwd_issue_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc,
                                             int ksteps) {
  using C = BwdCfg<DCH>;
  const uint64_t ad = sdesc_sw128(a, 16, 1024), bd = sdesc_sw128(b, 16, 1024);
#pragma unroll
  for (int ks = 0; ks < 4 * DCH; ++ks) {
    if (ks >= ksteps) break;
    const uint32_t off = (ks >> 2) * C::kBoxBytes + (ks & 3) * 32;
    mma_bf16_ss(d, sdesc_advance(ad, off), sdesc_advance(bd, off), idesc, ks > 0);
  }
}
// A (128 x 128 bf16) from TMEM: columns 0..63 of the tile at a, 64..127 at
// a + 64; B (128 x N) from shared memory, N contiguous.
template <int DCH>
__device__ __forceinline__ void bwd_issue_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc,
                                             bool first) {
  using C = BwdCfg<DCH>;
  const uint64_t bd = sdesc_sw128(b, C::kBoxBytes, 1024);
#pragma unroll
  for (int ks = 0; ks < 8; ++ks)
    mma_bf16_ts(d, a + (ks >> 2) * 64 + (ks & 3) * 8, sdesc_advance(bd, ks * 2048), idesc,
                !(first && ks == 0));
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
  uint32_t* tmem_slot = (uint32_t*)(bars + C::kNumBars);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
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
    if (lane == 0 && n > 0) {
      const int d_pad = (s.head_dim + 15) / 16 * 16, ksteps = d_pad / 16;
      const uint32_t idesc_s = idesc_bf16_f32(128, 128, 0);
      const uint32_t idesc_o = idesc_bf16_f32(128, d_pad, 1);
      const uint32_t ka = smem_u32(sk), va = smem_u32(sv), qa = smem_u32(sq), da = smem_u32(sdo);
      constexpr uint32_t code = kStatusTimeoutMma;
      bool ok = mbar_wait(kv_full, 0, code) && mbar_wait(&q_full[0], 0, code);
      if (ok) {
        tc_fence_after();
        bwd_issue_ss<DCH>(tmem, ka, qa, idesc_s, ksteps);
        mma_commit(s_full);
      }
      for (int j = 0; j < n && ok; ++j) {
        const uint32_t doj = da + (j & 1) * C::kTileBytes;
        if (!(ok = mbar_wait(&do_full[j & 1], (j / 2) & 1, code))) break;
        tc_fence_after();
        bwd_issue_ss<DCH>(tmem + 128, va, doj, idesc_s, ksteps);
        mma_commit(dp_full);
        if (!(ok = mbar_wait(p_full, j & 1, code))) break;
        tc_fence_after();
        bwd_issue_ts<DCH>(tmem + 256, tmem, doj, idesc_o, j == 0);
        mma_commit(&do_empty[j & 1]);
        if (j + 1 < n) {
          if (!(ok = mbar_wait(&q_full[(j + 1) % 3], ((j + 1) / 3) & 1, code))) break;
          tc_fence_after();
          bwd_issue_ss<DCH>(tmem, ka, qa + (j + 1) % 3 * C::kTileBytes, idesc_s, ksteps);
          mma_commit(s_full);
        }
        if (!(ok = mbar_wait(ds_full, j & 1, code))) break;
        tc_fence_after();
        bwd_issue_ts<DCH>(tmem + 384, tmem + 128, qa + j % 3 * C::kTileBytes, idesc_o, j == 0);
        mma_commit(&q_empty[j % 3]);
      }
      // Every product finished before the epilogue, and before TMEM is freed.
      mma_commit(o_done);
      mbar_wait(o_done, 0, code);
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
      float pr[64];
      const float* st = stats + (j & 1) * 256 + 64 * h;
      ok = mbar_wait(&st_full[j & 1], (j / 2) & 1, kStatusTimeoutSoftmax) &&
           mbar_wait(s_full, j & 1, kStatusTimeoutSoftmax);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      int qi = need_mask ? (r0 + 64 * h) % s.q_len : 0;  // query of the next column
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        uint32_t sv32[32];
        float lse[32], pc[32];
        tmem_ld32(s_tm + 32 * g, sv32);
#pragma unroll
        for (int c = 0; c < 32; c += 4) {
          const float4 f = *reinterpret_cast<const float4*>(st + 32 * g + c);
          lse[c] = f.x;
          lse[c + 1] = f.y;
          lse[c + 2] = f.z;
          lse[c + 3] = f.w;
        }
        tmem_ld_wait();
        bwd_probs<kCap>(p, sv32, lse, pc, &pr[32 * g]);
        if (need_mask) {
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            if ((unsigned)(qi - qlo) > qspan) pc[c] = pr[32 * g + c] = 0.f;
            if (++qi == s.q_len) qi = 0;
          }
        }
        uint32_t pk[16];
#pragma unroll
        for (int c = 0; c < 16; ++c) pk[c] = pack_bf16(pc[2 * c], pc[2 * c + 1]);
        // Columns [16 g, 16 g + 16) of this half: read already (g = 0: scores
        // 0..31 of the half; g = 1: still within them).
        tmem_st16(s_tm + 16 * g, pk);
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(p_full);

      ok = __all_sync(0xffffffffu, mbar_wait(dp_full, j & 1, kStatusTimeoutSoftmax));
      if (!ok) break;
      tc_fence_after();
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        uint32_t dv32[32];
        tmem_ld32(dp_tm + 32 * g, dv32);
        float dl[32];
#pragma unroll
        for (int c = 0; c < 32; c += 4) {
          const float4 f = *reinterpret_cast<const float4*>(st + 128 + 32 * g + c);
          dl[c] = f.x;
          dl[c + 1] = f.y;
          dl[c + 2] = f.z;
          dl[c + 3] = f.w;
        }
        tmem_ld_wait();
        uint32_t pk[16];
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          const float p0 = pr[32 * g + 2 * c], p1 = pr[32 * g + 2 * c + 1];
          const f2 d = f2_mul(f2_pack(p0, p1),
                              f2_sub(f2_pack(__uint_as_float(dv32[2 * c]), __uint_as_float(dv32[2 * c + 1])),
                                     f2_pack(dl[2 * c], dl[2 * c + 1])));
          float a, b;
          f2_unpack(d, a, b);
          if (need_mask) {  // a hidden score is an exact zero whatever dP is
            a = p0 == 0.f ? 0.f : a;
            b = p1 == 0.f ? 0.f : b;
          }
          pk[c] = pack_bf16(a, b);
        }
        tmem_st16(dp_tm + 16 * g, pk);
      }
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

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
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
    if (lane == 0 && n > 0) {
      const int d_pad = (s.head_dim + 15) / 16 * 16, ksteps = d_pad / 16;
      const uint32_t idesc_s = idesc_bf16_f32(128, 128, 0);
      const uint32_t idesc_o = idesc_bf16_f32(128, d_pad, 1);
      const uint32_t qa = smem_u32(sq), da = smem_u32(sdo), ka = smem_u32(sk), va = smem_u32(sv);
      constexpr uint32_t code = kStatusTimeoutMma;
      auto issue_s = [&](int j) {
        if (!mbar_wait(&k_full[j % 3], (j / 3) & 1, code)) return false;
        tc_fence_after();
        bwd_issue_ss<DCH>(tmem + 128 * (j & 1), qa, ka + j % 3 * C::kTileBytes, idesc_s, ksteps);
        mma_commit(&s_full[j & 1]);
        return true;
      };
      auto issue_dp = [&](int j) {
        if (!mbar_wait(&v_full[j & 1], (j / 2) & 1, code)) return false;
        tc_fence_after();
        bwd_issue_ss<DCH>(tmem + 256, da, va + (j & 1) * C::kTileBytes, idesc_s, ksteps);
        mma_commit(dp_full);
        mma_commit(&v_empty[j & 1]);
        return true;
      };
      bool ok = mbar_wait(q_full, 0, code) && issue_s(0) && issue_dp(0) && (n < 2 || issue_s(1));
      for (int j = 0; j < n && ok; ++j) {
        // dS_j written: dP_j and S_j have been read.
        if (!(ok = mbar_wait(ds_full, j & 1, code))) break;
        if (j + 1 < n && !(ok = issue_dp(j + 1))) break;
        tc_fence_after();
        bwd_issue_ts<DCH>(tmem + 384, tmem + 128 * (j & 1), ka + j % 3 * C::kTileBytes, idesc_o, j == 0);
        mma_commit(&k_empty[j % 3]);
        if (j + 2 < n && !(ok = issue_s(j + 2))) break;
      }
      mma_commit(o_done);
      mbar_wait(o_done, 0, code);
    }
  } else if (warp >= 4) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kBwRegsHigh));
    const int h = (warp - 4) >> 2, quarter = warp & 3;
    const int r = quarter * 32 + lane;
    const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
    const float* st = p.stats + ((long long)run * s.tiles + t) * 256;
    const float lse = st[r], delta = st[128 + r];
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
      float pr[64];
      ok = __all_sync(0xffffffffu, mbar_wait(&s_full[j & 1], (j / 2) & 1, kStatusTimeoutSoftmax));
      if (!ok) break;
      tc_fence_after();
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        uint32_t sv32[32];
        float l32[32], pc[32];
        tmem_ld32(s_tm + 32 * g, sv32);
#pragma unroll
        for (int c = 0; c < 32; ++c) l32[c] = lse;
        tmem_ld_wait();
        bwd_probs<kCap>(p, sv32, l32, pc, &pr[32 * g]);
        if (need_mask) {
#pragma unroll
          for (int c = 0; c < 32; ++c)
            if ((unsigned)(64 * h + 32 * g + c - vlo) > vspan) pr[32 * g + c] = 0.f;
        }
      }
      ok = __all_sync(0xffffffffu, mbar_wait(dp_full, j & 1, kStatusTimeoutSoftmax));
      if (!ok) break;
      tc_fence_after();
      const f2 dl = f2_pack(delta, delta);
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        uint32_t dv32[32], pk[16];
        tmem_ld32(tmem + lane_base + 256 + 64 * h + 32 * g, dv32);
        tmem_ld_wait();
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          const float p0 = pr[32 * g + 2 * c], p1 = pr[32 * g + 2 * c + 1];
          const f2 d = f2_mul(f2_pack(p0, p1),
                              f2_sub(f2_pack(__uint_as_float(dv32[2 * c]), __uint_as_float(dv32[2 * c + 1])), dl));
          float a, b;
          f2_unpack(d, a, b);
          if (need_mask) {
            a = p0 == 0.f ? 0.f : a;
            b = p1 == 0.f ? 0.f : b;
          }
          pk[c] = pack_bf16(a, b);
        }
        tmem_st16(s_tm + 16 * g, pk);
      }
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
