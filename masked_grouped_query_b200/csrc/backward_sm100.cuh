// backward_sm100.cuh -- the backward pass on the 5th-generation tensor cores
// (head_dim up to 128); backward.cuh has the formulas and the row layout.
//
// Two kernels with the same frame, one CTA of 12 warps per SM that walks work
// items (a key tile, or a row tile, of 128) in rounds of the grid; barriers,
// TMEM and the rings live across items, so the next item's loads and first
// products run under the current one's last steps and its stores:
//   warps 0, 3  TMA loaders (warp 0 the statistics' bulk copies too);
//   warp 1      TMEM allocator; warps 1 and 2 issue the tcgen05.mma (a lane each);
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
//
// The dQ kernel does not wait for the other one: both need the statistics
// alone.  Each launch may start when the kernel before it has started
// everywhere, so on small problems the two run side by side, and on large ones
// dQ's CTAs take each SM as it becomes free.  The chain: the dK/dV kernel
// waits for the statistics, then lets dQ's CTAs start (the statistics are
// therefore complete for them too; they read them past L1, since without a
// wait of their own nothing promises that L1 holds no older ones); dQ's last
// CTA waits for the dK/dV kernel before it ends, so that whatever follows in
// the stream finds both done.
//
// kFine: P and dS go to the tensor core as two bf16 terms each, the rounded
// value and the rounded rest, so that the gradients' only rounding that counts
// is their own.  Three more products in ten: only small problems take it
// (kBwFineSteps).
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
  static constexpr int kNumBars = 26;
  // Output boxes, 4 KB for each of the eight elementwise warps: with 64
  // columns there is room for them, with 128 they take the two-slot ring's
  // slot of the item's last tile.  Its next load, the second tile of the next
  // item, then waits for them; the first one does not.
  static constexpr int kStage = (kBars + kNumBars * 8 + 16 + 1023) / 1024 * 1024;
  static constexpr int kSmemBytes = DCH == 1 ? kStage + 8 * 4096 : kBars + kNumBars * 8 + 16;
  static __device__ __forceinline__ uint8_t* stage(uint8_t* smem, int last_tile) {
    return DCH == 1 ? smem + kStage : smem + kRing2 + (last_tile & 1) * kTileBytes;
  }
};

// P of 32 columns from 32 raw scores (nl: -lse of their rows, in pairs), and
// with a softcap the factors 1 - tanh^2 that dS takes.  Every 2^x is MUFU's:
// moving 2 to 6 of 16 pairs to the FMA pipe, as the forward kernel does with
// 2, measured from 1% faster to 2% slower.
template <bool kCap>
__device__ __forceinline__ void bwd_probs(const BwdParams& p, const uint32_t (&s)[32],
                                          const f2 (&nl)[16], f2 (&pr)[16], f2 (&fac)[16]) {
  if constexpr (!kCap) {
    const f2 sc = f2_pack(p.logit_scale, p.logit_scale);
#pragma unroll
    for (int c = 0; c < 16; ++c) {
      const f2 y = f2_fma(f2_pack(__uint_as_float(s[2 * c]), __uint_as_float(s[2 * c + 1])), sc, nl[c]);
      pr[c] = exp2_mufu_x2(y);
    }
  } else {
    float am = 0.f;
#pragma unroll
    for (int c = 0; c < 32; c += 2)
      am = fmax3(am, fabsf(__uint_as_float(s[c])), fabsf(__uint_as_float(s[c + 1])));
    const bool small = __all_sync(0xffffffffu, am * p.cap_in <= p.poly_most);
    const f2 co = f2_pack(p.cap_out, p.cap_out), one = f2_pack(1.f, 1.f);
    if (small) {
      // tanh(x cap_in) as x Q(x^2), cap_in folded into the coefficients.
      const float i2 = p.cap_in * p.cap_in;
      const float q1 = kTanhC1 * p.cap_in, q3 = kTanhC3 * p.cap_in * i2;
      const float q5 = kTanhC5 * p.cap_in * i2 * i2, q7 = kTanhC7 * p.cap_in * i2 * i2 * i2;
      const f2 c1 = f2_pack(q1, q1), c3 = f2_pack(q3, q3), c5 = f2_pack(q5, q5), c7 = f2_pack(q7, q7);
#pragma unroll
      for (int c = 0; c < 16; ++c) {
        const f2 x = f2_pack(__uint_as_float(s[2 * c]), __uint_as_float(s[2 * c + 1]));
        const f2 x2 = f2_mul(x, x);
        const f2 t = f2_mul(x, f2_fma(f2_fma(f2_fma(c7, x2, c5), x2, c3), x2, c1));
        pr[c] = exp2_mufu_x2(f2_fma(co, t, nl[c]));
        fac[c] = f2_fma(t, t ^ 0x8000000080000000ull, one);
      }
    } else {
      // Two of tanh_large at a time.
      const float in = p.cap_in * 2.8853900817779268f;
      const f2 half = f2_pack(0.5f, 0.5f), ci = f2_pack(in, in);
#pragma unroll
      for (int c = 0; c < 16; ++c) {
        float a, b;
        f2_unpack(f2_mul(f2_pack(__uint_as_float(s[2 * c]), __uint_as_float(s[2 * c + 1])), ci), a, b);
        const f2 u = exp2_mufu_x2(f2_pack(min_nan(a, 100.f), min_nan(b, 100.f)));
        f2_unpack(f2_fma(u, half, half), a, b);
        const f2 h = f2_pack(rcp(a), rcp(b));
        pr[c] = exp2_mufu_x2(f2_fma(co, f2_sub(one, h), nl[c]));
        fac[c] = f2_mul(f2_mul(u, h), h);
      }
    }
  }
}

// 32 fp32 values rounded to bf16 into TMEM columns [0, 16) at tm, and with
// kFine what the rounding left into columns [32, 48).
template <bool kFine>
__device__ __forceinline__ void bwd_store_bf16(uint32_t tm, const f2 (&v)[16]) {
  uint32_t w[16];
#pragma unroll
  for (int c = 0; c < 16; ++c) w[c] = pack_bf16_f2(v[c]);
  tmem_st16(tm, w);
  if constexpr (kFine) {
#pragma unroll
    for (int c = 0; c < 16; ++c)
      w[c] = pack_bf16_f2(f2_sub(v[c], f2_pack(__uint_as_float(w[c] << 16),
                                               __uint_as_float(w[c] & 0xffff0000u))));
    tmem_st16(tm + 32, w);
  }
}

// Zeros in the columns whose bit is not set.
__device__ __forceinline__ void bwd_hide(f2 (&pr)[16], uint32_t seen) {
#pragma unroll
  for (int c = 0; c < 16; ++c) {
    float a, b;
    f2_unpack(pr[c], a, b);
    pr[c] = f2_pack(seen & (1u << (2 * c)) ? a : 0.f, seen & (2u << (2 * c)) ? b : 0.f);
  }
}

// dS of 32 columns from what bwd_probs left (p times the factor), dP and the
// rows' delta.  A hidden score is an exact zero whatever dP is; a visible one
// whose p has underflowed is not: with an infinite dP it is NaN.
__device__ __forceinline__ void bwd_ds(const f2* keep, const uint32_t (&dp)[32], const f2 (&dl)[16],
                                       bool masked, uint32_t seen, f2 (&d)[16]) {
#pragma unroll
  for (int c = 0; c < 16; ++c)
    d[c] = f2_mul(keep[c], f2_sub(f2_pack(__uint_as_float(dp[2 * c]), __uint_as_float(dp[2 * c + 1])),
                                  dl[c]));
  if (masked) bwd_hide(d, seen);
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

// 64 columns of a warp's 32 rows of an fp32 accumulator at tm, scaled and
// rounded to bf16, through a swizzled 32-row box in shared memory and one TMA
// store (rows and columns outside the tensor are not written; columns of the
// accumulator past head_dim hold whatever TMEM held).  `again`: the box's
// previous store, of this item, may still be reading it.  Items of one length
// finish together on all SMs, and their stores then wait for L2: TMA stores
// leave these warps free meanwhile (from registers, in whole lines or not,
// they took 1.5 to 2 times as long on the encoder shape).
__device__ __forceinline__ void bwd_store_box(const CUtensorMap* map, uint8_t* stage, uint32_t tm,
                                              int x, int row, int outer, float scale, bool again,
                                              int lane) {
  uint32_t a[32], b[32], w[32];
  tmem_ld32(tm, a);
  tmem_ld32(tm + 32, b);
  tmem_ld_wait();
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    w[e] = pack_bf16(__uint_as_float(a[2 * e]) * scale, __uint_as_float(a[2 * e + 1]) * scale);
    w[16 + e] = pack_bf16(__uint_as_float(b[2 * e]) * scale, __uint_as_float(b[2 * e + 1]) * scale);
  }
  if (again) {
    if (lane == 0) bulk_wait_read();
    __syncwarp();
  }
#pragma unroll
  for (int g = 0; g < 8; ++g)
    *reinterpret_cast<uint4*>(stage + sw128(lane, g)) =
        make_uint4(w[4 * g], w[4 * g + 1], w[4 * g + 2], w[4 * g + 3]);
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) {
    tma_store_3d(map, stage, x, row, outer);
    bulk_commit();
  }
}

// Zeros for a warp's rows (contiguous in memory) of an item without a step.
// Not through a box: the loader, which skips such items, may have filled it.
__device__ __forceinline__ void bwd_store_zeros(__nv_bfloat16* dst, int rows, int head_dim, int lane) {
  const int pieces = rows * (head_dim / 8);
  for (int i = lane; i < pieces; i += 32)
    reinterpret_cast<uint4*>(dst)[i] = make_uint4(0u, 0u, 0u, 0u);
}

// The same rows as a part's fp32 partial: columns [0, cols) of the accumulator
// at tm (lane = row), or zeros for a part without a step.
__device__ __forceinline__ void bwd_store_part(float* dst, uint32_t tm, int c0, int c1, int row, bool zero) {
  for (int c = c0; c < c1; c += 16) {
    uint32_t v[16];
    tmem_ld16(tm + c, v);
    tmem_ld_wait();
#pragma unroll
    for (int g = 0; g < 4; ++g)
      reinterpret_cast<float4*>(dst)[(c / 4 + g) * 128 + row] =
          zero ? make_float4(0.f, 0.f, 0.f, 0.f)
               : make_float4(__uint_as_float(v[4 * g]), __uint_as_float(v[4 * g + 1]),
                             __uint_as_float(v[4 * g + 2]), __uint_as_float(v[4 * g + 3]));
  }
}

// Bits lo..hi of a word (none when hi < lo, or outside 0..31).
__device__ __forceinline__ uint32_t bwd_bits(int lo, int hi) {
  lo = max(lo, 0);
  hi = min(hi, 31);
  return hi < lo ? 0u : (0xffffffffu >> (31 - hi)) & (0xffffffffu << lo);
}
// The k-th item of this CTA: items go out in rounds of the grid, every other
// round backwards when they are sorted heavy first, so that no CTA takes the
// heaviest of every round.
__device__ __forceinline__ int bwd_item(const BwdShape& s, int k) {
  const int G = (int)gridDim.x, c = (int)blockIdx.x;
  return k * G + (((s.causal || s.window > 0) && (k & 1)) ? G - 1 - c : c);
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
template <int k0, int k1>
__device__ __forceinline__ void bwd_issue_ts(uint32_t leader, uint32_t d, uint32_t a, uint64_t bd,
                                             uint32_t idesc, bool first) {
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
template <int DCH, bool kCap, bool kFine>
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
  uint64_t* k_full = bars;
  uint64_t* q_full = bars + 1;    // [3]
  uint64_t* q_empty = bars + 4;   // [3]
  uint64_t* do_full = bars + 7;   // [2]
  uint64_t* do_empty = bars + 9;  // [2]
  uint64_t* st_full = bars + 11;  // [2]
  uint64_t* st_empty = bars + 13; // [2]
  uint64_t* s_full = bars + 15;   // [2], by tile: two roles wait for it, a step apart
  uint64_t* dp_full = bars + 17;
  uint64_t* p_half = bars + 18;
  uint64_t* p_full = bars + 19;
  uint64_t* ds_full = bars + 20;
  uint64_t* o_done = bars + 21;
  uint64_t* k_empty = bars + 22;
  uint64_t* v_full = bars + 23;
  uint64_t* v_empty = bars + 24;
  uint64_t* drain = bars + 25;
  uint32_t* tmem_slot = (uint32_t*)(bars + C::kNumBars);

  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    mbar_init(k_full, 1);
    mbar_init(k_empty, 1);
    mbar_init(drain, 2);
    mbar_init(v_full, 1);
    mbar_init(v_empty, 1);
    for (int i = 0; i < 3; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&do_full[i], 1);
      mbar_init(&do_empty[i], 2 + 8);  // both issuers, the elementwise warps
      mbar_init(&st_full[i], 1);
      mbar_init(&st_empty[i], 8);
    }
    mbar_init(&s_full[0], 1);
    mbar_init(&s_full[1], 1);
    mbar_init(p_half, 8);
    mbar_init(dp_full, 1);
    mbar_init(p_full, 8);
    mbar_init(ds_full, 8);
    mbar_init(o_done, 2);
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  if (threadIdx.x == 0) {
    grid_wait();
    grid_launch_dependents();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // Item i: part i % splits of unit and key tile u = i / splits: unit u % units,
  // tile u / units, in ascending order: under a causal mask the first ones
  // have the most rows.  Step j of an item is row tile t + j, wrapping inside
  // [first, first + count), from run `run` on.
  const int units = (int)s.units, splits = p.kv_splits;
  const int items = units * ((s.kv_len + 127) / 128) * splits;
  struct Item {
    int unit, k0, first, count, n, run, t;
  };
  auto item_at = [&](int i) {
    const int u = splits > 1 ? i / splits : i;
    Item t;
    t.unit = u % units;
    t.k0 = u / units * 128;
    bwd_row_tiles(s, t.k0, min(t.k0 + 127, s.kv_len - 1), 128, t.first, t.count);
    int begin, end;
    bwd_part(t.count * s.runs_per_unit, i - u * splits, splits, begin, end);
    t.n = end - begin;
    const int skip = begin > 0 ? begin / t.count : 0;
    t.run = t.unit * s.runs_per_unit + skip;
    t.t = t.first + begin - skip * t.count;
    return t;
  };

  if (warp < 4) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kBwRegsLow));
  if (warp == 0 || warp == 3) {
    // Two loaders: warp 0 K, Q and the statistics, warp 3 V and dO (whose
    // slots also hold the output boxes).
    if (lane == 0) {
      constexpr uint32_t code = kStatusTimeoutProducer;
      auto load = [&](uint8_t* dst, const CUtensorMap* map, uint64_t* bar, int row, int outer) {
        mbar_arrive_expect_tx(bar, C::kTileBytes);
        for (int c = 0; c < DCH; ++c)
          tma_load_3d(dst + c * C::kBoxBytes, map, bar, c * 64, row, outer);
      };
      const bool first = warp == 0;
      tma_prefetch_map(first ? &tm_q : &tm_do);
      tma_prefetch_map(first ? &tm_k : &tm_v);
      int J = 0, busy = 0;        // row tiles and items so far
      int n1 = 0, n2 = 0, n3 = 0;  // loads issued: K or V, Q or dO, statistics
      bool ok = true;
      for (int kk = 0, i = bwd_item(s, 0); i < items && ok; i = bwd_item(s, ++kk)) {
        const Item it = item_at(i);
        if (it.n == 0) continue;
        uint64_t* const free1 = first ? k_empty : v_empty;
        if (busy > 0 && !(ok = mbar_wait(free1, (busy - 1) & 1, code))) break;
        if (first) load(sk, &tm_k, k_full, it.k0, it.unit);
        else load(sv, &tm_v, v_full, it.k0, it.unit);
        ++n1;
        int run = it.run, t = it.t;
        for (int j = 0; j < it.n; ++j, ++J) {
          const int q3 = J % 3, d2 = J & 1;
          if (first) {
            if (J >= 3 && !(ok = mbar_wait(&q_empty[q3], (J / 3 - 1) & 1, code))) break;
            load(sq + q3 * C::kTileBytes, &tm_q, &q_full[q3], t * 128, run);
            ++n2;
            if (J >= 2 && !(ok = mbar_wait(&st_empty[d2], (J / 2 - 1) & 1, code))) break;
            mbar_arrive_expect_tx(&st_full[d2], 1024);
            bulk_load(stats + d2 * 256, p.stats + ((long long)run * s.tiles + t) * 256, 1024,
                      &st_full[d2]);
            ++n3;
          } else {
            if (J >= 2 && !(ok = mbar_wait(&do_empty[d2], (J / 2 - 1) & 1, code))) break;
            load(sdo + d2 * C::kTileBytes, &tm_do, &do_full[d2], t * 128, run);
            ++n2;
          }
          if (++t == it.first + it.count) {
            t = it.first;
            ++run;
          }
        }
        ++busy;
      }
      // Never leave with copies in flight.
      if (n1 > 0) mbar_wait(first ? k_full : v_full, (n1 - 1) & 1, code);
      if (first)
        for (int j = max(0, n2 - 3); j < n2; ++j) mbar_wait(&q_full[j % 3], (j / 3) & 1, code);
      else
        for (int j = max(0, n2 - 2); j < n2; ++j) mbar_wait(&do_full[j & 1], (j / 2) & 1, code);
      for (int j = max(0, n3 - 2); j < n3; ++j) mbar_wait(&st_full[j & 1], (j / 2) & 1, code);
    }
  } else if (warp == 1 || warp == 2) {
    // Two issuers: warp 1 the products S^T and dV, warp 2 dP^T and dK.  While
    // one waits for its next operand, the other one's products fill the
    // tensor core; each writes its own TMEM columns, in its own order.  The
    // whole warp walks the loop, lane 0 issues (see mma_bf16_ss_warp).
    const uint32_t leader = lane == 0;
    const int d_pad = (s.head_dim + 15) / 16 * 16, ksteps = d_pad / 16;
    const uint32_t idesc_s = idesc_bf16_f32(128, 128, 0);
    const uint32_t idesc_o = idesc_bf16_f32(128, d_pad, 1);
    const uint64_t kd = bwd_desc_k(smem_u32(sk)), vd = bwd_desc_k(smem_u32(sv));
    const uint64_t qk = bwd_desc_k(smem_u32(sq)), qn = bwd_desc_n<DCH>(smem_u32(sq));
    const uint64_t dk = bwd_desc_k(smem_u32(sdo)), dn = bwd_desc_n<DCH>(smem_u32(sdo));
    constexpr uint32_t kTile = C::kTileBytes >> 4;  // a slot, in descriptor units
    // Waits are uniform over the warp, so that it stays converged.
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      return __all_sync(0xffffffffu, mbar_wait(bar, parity, kStatusTimeoutMma)) != 0;
    };
    int J = 0, busy = 0;
    int sq_j = 0, sq_n = 1;  // Q slots of row tiles J and J + 1
    bool ok = true;
    for (int kk = 0, i = bwd_item(s, 0); i < items && ok; i = bwd_item(s, ++kk)) {
      const int n = item_at(i).n;
      if (n == 0) continue;
      if (warp == 1) {
        if (!(ok = wait(k_full, busy & 1) && wait(&q_full[sq_j], (J / 3) & 1))) break;
        tc_fence_after();
        bwd_issue_ss<DCH>(leader, tmem, kd, qk + sq_j * kTile, idesc_s, ksteps);
        mma_commit_warp(leader, &s_full[J & 1]);
        if (n == 1) mma_commit_warp(leader, k_empty);
        for (int j = 0; j < n; ++j, ++J) {
          const bool more = j + 1 < n;
          // Loads first: they are there long before P is.
          if (!(ok = wait(&do_full[J & 1], (J / 2) & 1))) break;
          if (more && !(ok = wait(&q_full[sq_n], ((J + 1) / 3) & 1))) break;
          // dV in two parts: rows 0..31 and 64..95 of the tile first, so that
          // the next S^T waits for half a product only once P^T is complete.
          if (!(ok = wait(p_half, J & 1))) break;
          tc_fence_after();
          bwd_issue_ts<0, 2>(leader, tmem + 256, tmem, dn + (J & 1) * kTile, idesc_o, j == 0);
          if (kFine) bwd_issue_ts<0, 2>(leader, tmem + 256, tmem + 32, dn + (J & 1) * kTile, idesc_o, false);
          if (!(ok = wait(p_full, J & 1))) break;
          tc_fence_after();
          bwd_issue_ts<2, 4>(leader, tmem + 256, tmem, dn + (J & 1) * kTile, idesc_o, false);
          if (kFine) bwd_issue_ts<2, 4>(leader, tmem + 256, tmem + 32, dn + (J & 1) * kTile, idesc_o, false);
          mma_commit_warp(leader, &do_empty[J & 1]);
          if (more) {
            bwd_issue_ss<DCH>(leader, tmem, kd, qk + sq_n * kTile, idesc_s, ksteps);
            mma_commit_warp(leader, &s_full[(J + 1) & 1]);
            if (j + 2 == n) mma_commit_warp(leader, k_empty);
          }
          sq_j = sq_n;
          if (++sq_n == 3) sq_n = 0;
        }
      } else {
        if (!(ok = wait(v_full, busy & 1))) break;
        for (int j = 0; j < n; ++j, ++J) {
          if (!(ok = wait(&do_full[J & 1], (J / 2) & 1))) break;
          tc_fence_after();
          bwd_issue_ss<DCH>(leader, tmem + 128, vd, dk + (J & 1) * kTile, idesc_s, ksteps);
          mma_commit_warp(leader, dp_full);
          mma_commit_warp(leader, &do_empty[J & 1]);
          if (j + 1 == n) mma_commit_warp(leader, v_empty);
          if (!(ok = wait(&q_full[sq_j], (J / 3) & 1) && wait(ds_full, J & 1))) break;
          // The next S^T goes first: P^T waits for it, nothing waits for dK.
          if (j + 1 < n && !(ok = wait(&s_full[(J + 1) & 1], ((J + 1) / 2) & 1))) break;
          tc_fence_after();
          bwd_issue_ts<0, 4>(leader, tmem + 384, tmem + 128, qn + sq_j * kTile, idesc_o, j == 0);
          if (kFine)
            bwd_issue_ts<0, 4>(leader, tmem + 384, tmem + 160, qn + sq_j * kTile, idesc_o, false);
          mma_commit_warp(leader, &q_empty[sq_j]);
          if (++sq_j == 3) sq_j = 0;
        }
      }
      if (!ok) break;
      mma_commit_warp(leader, o_done);
      ++busy;
    }
    // Every product finished before TMEM is freed.
    mma_commit_warp(leader, drain);
    wait(drain, 0);
  } else if (warp >= 4) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kBwRegsHigh));
    const int h = (warp - 4) >> 2, quarter = warp & 3;
    const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
    const uint32_t s_tm = tmem + lane_base + 64 * h, dp_tm = s_tm + 128;
    const MaskSpec ms = bwd_mask(s);
    int J = 0, busy = 0;
    bool ok = true;
    int i = bwd_item(s, 0);
    Item it = item_at(i);
    for (int kk = 1; i < items && ok; ++kk) {
      const int key = it.k0 + quarter * 32 + lane;
      // Queries that see this lane's key: [qlo, qhi] (none past kv_len).
      int qlo, qhi;
      bwd_query_range(s, key, key, qlo, qhi);
      if (key >= s.kv_len) qhi = -1;
      int t = it.t;
      for (int j = 0; j < it.n; ++j, ++J) {
        const int r0 = t * 128, nr = min(128, s.run - r0);
        const bool need_mask = bwd_need_mask(s, ms, r0, nr, it.k0, 128);
        const uint32_t par = J & 1, dpar = (J / 2) & 1;
        f2 keep[32];
        const float* st = stats + par * 256 + 64 * h;
        f2 nl[16];
        ok = __all_sync(0xffffffffu, mbar_wait(&st_full[par], dpar, kStatusTimeoutSoftmax));
        if (!ok) break;
        bwd_load32(st, nl);
        ok = __all_sync(0xffffffffu, mbar_wait(&s_full[par], dpar, kStatusTimeoutSoftmax));
        if (!ok) break;
        tc_fence_after();
        uint32_t b0[32], b1[32];
        tmem_ld32(s_tm, b0);
        uint32_t seen[2] = {0u, 0u};  // this lane's key by the columns of its half
        if (need_mask) {
          const int c0 = r0 + 64 * h;
          if (s.run == s.q_len) {
            seen[0] = bwd_bits(qlo - c0, qhi - c0);
            seen[1] = bwd_bits(qlo - c0 - 32, qhi - c0 - 32);
          } else {  // several heads in the tile: query by query
            int qi = c0 % s.q_len;
#pragma unroll 1
            for (int c = 0; c < 32; ++c) {
              if (qi >= qlo && qi <= qhi) seen[0] |= 1u << c;
              if (++qi == s.q_len) qi = 0;
            }
#pragma unroll 1
            for (int c = 0; c < 32; ++c) {
              if (qi >= qlo && qi <= qhi) seen[1] |= 1u << c;
              if (++qi == s.q_len) qi = 0;
            }
            seen[0] &= bwd_bits(0, nr - 1 - 64 * h);  // rows that pad the tile see nothing
            seen[1] &= bwd_bits(0, nr - 1 - 64 * h - 32);
          }
        }
        // P of columns 32 g .. 32 g + 31 of this half, into TMEM columns
        // [16 g, 16 g + 16) of it, whose scores have been read.
        auto probs = [&](const uint32_t(&sv32)[32], int g) {
          f2 pr[16], fac[16];
          bwd_probs<kCap>(p, sv32, nl, pr, fac);
          if (need_mask) bwd_hide(pr, seen[g]);
#pragma unroll
          for (int c = 0; c < 16; ++c) keep[16 * g + c] = kCap ? f2_mul(pr[c], fac[c]) : pr[c];
          bwd_store_bf16<kFine>(s_tm + 16 * g, pr);
        };
        if (kFine) tmem_ld32(s_tm + 32, b1);  // the rests go over these scores
        tmem_ld_wait();
        if (!kFine) tmem_ld32(s_tm + 32, b1);
        probs(b0, 0);
        tmem_ld_wait();
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_half);
        bwd_load32(st + 32, nl);
        probs(b1, 1);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full);

        f2 dl[16];
        bwd_load32(st + 128, dl);
        ok = __all_sync(0xffffffffu, mbar_wait(dp_full, par, kStatusTimeoutSoftmax));
        if (!ok) break;
        tc_fence_after();
        f2 ds[16];
        tmem_ld32(dp_tm, b0);
        tmem_ld32(dp_tm + 32, b1);
        tmem_ld_wait();
        bwd_ds(keep, b0, dl, need_mask, seen[0], ds);
        bwd_store_bf16<kFine>(dp_tm, ds);
        bwd_load32(st + 160, dl);
        bwd_ds(keep + 16, b1, dl, need_mask, seen[1], ds);
        bwd_store_bf16<kFine>(dp_tm + 16, ds);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(ds_full);
          mbar_arrive(&st_empty[par]);
          if (j + 1 < it.n) mbar_arrive(&do_empty[par]);  // the last slot holds the output boxes first
        }
        if (++t == it.first + it.count) t = it.first;
      }
      if (!ok) break;
      const int next = bwd_item(s, kk);
      const Item next_it = item_at(next);  // ahead of the wait: divisions
      if (it.n > 0) {
        ok = __all_sync(0xffffffffu, mbar_wait(o_done, busy & 1, kStatusTimeoutEpilogue));
        if (!ok) break;
        ++busy;
        tc_fence_after();
      }
      // Warpgroup 0 stores dV, warpgroup 1 dK.  The next item's first products
      // into them follow this thread's next P and dS arrivals.
      const int row0 = it.k0 + quarter * 32;
      if (splits > 1) {
        const int d_pad = (s.head_dim + 15) / 16 * 16;
        bwd_store_part((h ? p.part_dk : p.part_dv) + (long long)i * 128 * d_pad,
                       tmem + lane_base + 256 + 128 * h, 0, d_pad, quarter * 32 + lane, it.n == 0);
        if (lane == 0 && it.n > 0) mbar_arrive(&do_empty[(J - 1) & 1]);
      } else if (it.n == 0) {
        if (row0 < s.kv_len)
          bwd_store_zeros((h ? p.dk : p.dv) + ((long long)it.unit * s.kv_len + row0) * s.head_dim,
                          min(32, s.kv_len - row0), s.head_dim, lane);
      } else {
        uint8_t* stage = C::stage(smem, J - 1) + (warp - 4) * 4096;
#pragma unroll 1
        for (int c0 = 0; c0 < s.head_dim && row0 < s.kv_len; c0 += 64)
          bwd_store_box(h ? &tm_dk : &tm_dv, stage, tmem + lane_base + 256 + 128 * h + c0, c0, row0,
                        it.unit, h ? p.scale : 1.f, c0 > 0, lane);
        if (lane == 0) {
          bulk_wait_read();  // the slot goes back to the loader
          mbar_arrive(&do_empty[(J - 1) & 1]);
        }
      }
      i = next;
      it = next_it;
    }
    if (lane == 0) bulk_wait_all();  // stores done before the CTA exits
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------------ dQ
template <int DCH, bool kCap, bool kFine>
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
  // [2], by tile: with one barrier, the issuer of dQ could find the phase
  // after its own complete as well and take it for none.
  uint64_t* ds_full = bars + 14;
  uint64_t* o_done = bars + 16;
  uint64_t* q_empty = bars + 17;
  uint64_t* do_full = bars + 18;
  uint64_t* do_empty = bars + 19;
  uint64_t* drain = bars + 20;
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
      mbar_init(&v_empty[i], 1 + 8);  // dP, the elementwise warps
      mbar_init(&s_full[i], 1);
      mbar_init(&ds_full[i], 8);
    }
    mbar_init(dp_full, 1);
    mbar_init(o_done, 1);
    mbar_init(q_empty, 1);
    mbar_init(do_full, 1);
    mbar_init(do_empty, 1);
    mbar_init(drain, 2);
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

  // Item i: part i % splits of run and row tile u = i / splits: run u % runs,
  // tiles from the last down: under a causal mask the last ones have the most
  // keys.  Runs of one kv head follow each other and share K and V in L2.
  const MaskSpec ms = bwd_mask(s);
  const int runs = (int)s.runs, splits = p.q_splits, items = runs * s.tiles * splits;
  struct Item {
    int run, unit, r0, nr, tile, part;
    KeyRange kr;
  };
  auto item_at = [&](int i) {
    const int u = splits > 1 ? i / splits : i, sp = i - u * splits;
    Item t;
    t.run = u % runs;
    t.tile = s.tiles - 1 - u / runs;
    t.part = (t.tile * runs + t.run) * splits + sp;
    t.r0 = t.tile * 128;
    t.nr = min(128, s.run - t.r0);
    t.unit = t.run / s.runs_per_unit;
    t.kr = key_range(ms, t.r0, t.nr, 128);
    int begin, end;
    bwd_part(t.kr.t_count, sp, splits, begin, end);
    t.kr.t_first += begin;
    t.kr.t_count = end - begin;
    return t;
  };

  if (warp < 4) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kBwRegsLow));
  if (warp == 0 || warp == 3) {
    // Two loaders: warp 0 Q and K, warp 3 dO and V (whose slots also hold the
    // output boxes).
    if (lane == 0) {
      constexpr uint32_t code = kStatusTimeoutProducer;
      auto load = [&](uint8_t* dst, const CUtensorMap* map, uint64_t* bar, int row, int outer) {
        mbar_arrive_expect_tx(bar, C::kTileBytes);
        for (int c = 0; c < DCH; ++c)
          tma_load_3d(dst + c * C::kBoxBytes, map, bar, c * 64, row, outer);
      };
      const bool first = warp == 0;
      tma_prefetch_map(first ? &tm_q : &tm_do);
      tma_prefetch_map(first ? &tm_k : &tm_v);
      int J = 0, busy = 0, n1 = 0, n2 = 0;
      bool ok = true;
      for (int kk = 0, i = bwd_item(s, 0); i < items && ok; i = bwd_item(s, ++kk)) {
        const Item it = item_at(i);
        if (it.kr.t_count == 0) continue;
        uint64_t* const free1 = first ? q_empty : do_empty;
        if (busy > 0 && !(ok = mbar_wait(free1, (busy - 1) & 1, code))) break;
        if (first) load(sq, &tm_q, q_full, it.r0, it.run);
        else load(sdo, &tm_do, do_full, it.r0, it.run);
        ++n1;
        for (int j = 0; j < it.kr.t_count; ++j, ++J) {
          const int key0 = (it.kr.t_first + j) * 128, k3 = J % 3, v2 = J & 1;
          if (first) {
            if (J >= 3 && !(ok = mbar_wait(&k_empty[k3], (J / 3 - 1) & 1, code))) break;
            load(sk + k3 * C::kTileBytes, &tm_k, &k_full[k3], key0, it.unit);
          } else {
            if (J >= 2 && !(ok = mbar_wait(&v_empty[v2], (J / 2 - 1) & 1, code))) break;
            load(sv + v2 * C::kTileBytes, &tm_v, &v_full[v2], key0, it.unit);
          }
          ++n2;
        }
        ++busy;
      }
      // Never leave with copies in flight.
      if (n1 > 0) mbar_wait(first ? q_full : do_full, (n1 - 1) & 1, code);
      if (first)
        for (int j = max(0, n2 - 3); j < n2; ++j) mbar_wait(&k_full[j % 3], (j / 3) & 1, code);
      else
        for (int j = max(0, n2 - 2); j < n2; ++j) mbar_wait(&v_full[j & 1], (j / 2) & 1, code);
    }
  } else if (warp == 1 || warp == 2) {
    // Two issuers as above: warp 1 S and dQ, warp 2 dP.
    const uint32_t leader = lane == 0;
    const int d_pad = (s.head_dim + 15) / 16 * 16, ksteps = d_pad / 16;
    const uint32_t idesc_s = idesc_bf16_f32(128, 128, 0);
    const uint32_t idesc_o = idesc_bf16_f32(128, d_pad, 1);
    const uint64_t qd = bwd_desc_k(smem_u32(sq)), dd = bwd_desc_k(smem_u32(sdo));
    const uint64_t kd = bwd_desc_k(smem_u32(sk)), kn = bwd_desc_n<DCH>(smem_u32(sk));
    const uint64_t vd = bwd_desc_k(smem_u32(sv));
    constexpr uint32_t kTile = C::kTileBytes >> 4;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      return __all_sync(0xffffffffu, mbar_wait(bar, parity, kStatusTimeoutMma)) != 0;
    };
    int J = 0, busy = 0;
    int k_j = 0, k_s = 0, x = 0;  // K slots of dQ's tile J and of S's tile x
    bool ok = true;
    for (int kk = 0, i = bwd_item(s, 0); i < items && ok; i = bwd_item(s, ++kk)) {
      const int n = item_at(i).kr.t_count;
      if (n == 0) continue;
      if (warp == 1) {
        const int x_end = J + n;
        // S of the next tile into its buffer; the last one frees Q.
        auto issue_s = [&]() {
          if (!wait(&k_full[k_s], (x / 3) & 1)) return false;
          tc_fence_after();
          bwd_issue_ss<DCH>(leader, tmem + 128 * (x & 1), qd, kd + k_s * kTile, idesc_s, ksteps);
          mma_commit_warp(leader, &s_full[x & 1]);
          ++x;
          if (++k_s == 3) k_s = 0;
          if (x == x_end) mma_commit_warp(leader, q_empty);
          return true;
        };
        if (!(ok = wait(q_full, busy & 1) && issue_s())) break;
        if (n > 1 && !(ok = issue_s())) break;
        for (int j = 0; j < n; ++j, ++J) {
          // dS_j written: S_j has been read.
          if (!(ok = wait(&ds_full[J & 1], (J / 2) & 1))) break;
          tc_fence_after();
          bwd_issue_ts<0, 4>(leader, tmem + 384, tmem + 128 * (J & 1), kn + k_j * kTile, idesc_o, j == 0);
          if (kFine)
            bwd_issue_ts<0, 4>(leader, tmem + 384, tmem + 128 * (J & 1) + 32, kn + k_j * kTile, idesc_o, false);
          mma_commit_warp(leader, &k_empty[k_j]);
          if (++k_j == 3) k_j = 0;
          if (x < x_end && !(ok = issue_s())) break;
        }
        if (!ok) break;
        mma_commit_warp(leader, o_done);
      } else {
        if (!(ok = wait(do_full, busy & 1))) break;
        for (int j = 0; j < n; ++j, ++J) {
          if (!(ok = wait(&v_full[J & 1], (J / 2) & 1))) break;
          // The previous tile's dP has been read.
          if (J > 0 && !(ok = wait(&ds_full[(J - 1) & 1], ((J - 1) / 2) & 1))) break;
          tc_fence_after();
          bwd_issue_ss<DCH>(leader, tmem + 256, dd, vd + (J & 1) * kTile, idesc_s, ksteps);
          mma_commit_warp(leader, dp_full);
          mma_commit_warp(leader, &v_empty[J & 1]);
        }
        if (!ok) break;
        mma_commit_warp(leader, do_empty);
      }
      ++busy;
    }
    // Every product finished before TMEM is freed.
    mma_commit_warp(leader, drain);
    wait(drain, 0);
  } else if (warp >= 4) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kBwRegsHigh));
    const int h = (warp - 4) >> 2, quarter = warp & 3;
    const int r = quarter * 32 + lane;
    const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
    int J = 0, busy = 0;
    bool ok = true;
    int i = bwd_item(s, 0);
    Item it = item_at(i);
    for (int kk = 1; i < items && ok; ++kk) {
      const float* st = p.stats + ((long long)it.run * s.tiles + it.tile) * 256;
      const float nlse = __ldcg(st + r), delta = __ldcg(st + 128 + r);  // from L2 (see the head)
      int lo = 0, hi = -1;
      if (r < it.nr) {
        const int qpos = s.kv_len - s.q_len + (it.r0 + r) % s.q_len;
        lo = first_key(ms, qpos);
        hi = last_key(ms, qpos);
      }
      for (int j = 0; j < it.kr.t_count; ++j, ++J) {
        const int key0 = (it.kr.t_first + j) * 128;
        const bool need_mask = !(key0 >= it.kr.all_lo && key0 + 127 <= it.kr.all_hi);
        const int c0 = key0 + 64 * h;
        const uint32_t s_tm = tmem + lane_base + 128 * (J & 1) + 64 * h;
        f2 keep[32];
        ok = __all_sync(0xffffffffu, mbar_wait(&s_full[J & 1], (J / 2) & 1, kStatusTimeoutSoftmax));
        if (!ok) break;
        tc_fence_after();
        uint32_t b0[32], b1[32];
        f2 row[16];
        auto probs = [&](const uint32_t(&sv32)[32], int g) {
          f2 pr[16], fac[16];
#pragma unroll
          for (int c = 0; c < 16; ++c) row[c] = f2_pack(nlse, nlse);
          bwd_probs<kCap>(p, sv32, row, pr, fac);
          if (need_mask) bwd_hide(pr, bwd_bits(lo - c0 - 32 * g, hi - c0 - 32 * g));
#pragma unroll
          for (int c = 0; c < 16; ++c) keep[16 * g + c] = kCap ? f2_mul(pr[c], fac[c]) : pr[c];
        };
        tmem_ld32(s_tm, b0);
        tmem_ld_wait();
        tmem_ld32(s_tm + 32, b1);
        probs(b0, 0);
        tmem_ld_wait();
        probs(b1, 1);
        ok = __all_sync(0xffffffffu, mbar_wait(dp_full, J & 1, kStatusTimeoutSoftmax));
        if (!ok) break;
        tc_fence_after();
        f2 ds[16];
        tmem_ld32(tmem + lane_base + 256 + 64 * h, b0);
        tmem_ld32(tmem + lane_base + 288 + 64 * h, b1);
#pragma unroll
        for (int c = 0; c < 16; ++c) row[c] = f2_pack(delta, delta);
        tmem_ld_wait();
        bwd_ds(keep, b0, row, need_mask, bwd_bits(lo - c0, hi - c0), ds);
        bwd_store_bf16<kFine>(s_tm, ds);
        bwd_ds(keep + 16, b1, row, need_mask, bwd_bits(lo - c0 - 32, hi - c0 - 32), ds);
        bwd_store_bf16<kFine>(s_tm + 16, ds);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&ds_full[J & 1]);
          // The last slot holds the output boxes first.
          if (j + 1 < it.kr.t_count) mbar_arrive(&v_empty[J & 1]);
        }
      }
      if (!ok) break;
      const int next = bwd_item(s, kk);
      const Item next_it = item_at(next);  // ahead of the wait: divisions
      if (it.kr.t_count > 0) {
        ok = __all_sync(0xffffffffu, mbar_wait(o_done, busy & 1, kStatusTimeoutEpilogue));
        if (!ok) break;
        ++busy;
        tc_fence_after();
      }
      // Each warpgroup stores its half of the columns.
      const int rows = it.nr - quarter * 32;
      if (splits > 1) {
        const int d_pad = (s.head_dim + 15) / 16 * 16;
        bwd_store_part(p.part_dq + (long long)it.part * 128 * d_pad, tmem + lane_base + 384, 64 * h,
                       min(64 * h + 64, d_pad), r, it.kr.t_count == 0);
        if (lane == 0 && it.kr.t_count > 0) mbar_arrive(&v_empty[(J - 1) & 1]);
      } else if (it.kr.t_count == 0) {
        if (rows > 0 && h == 0)
          bwd_store_zeros(p.dq + ((long long)it.run * s.run + it.r0 + quarter * 32) * s.head_dim,
                          min(32, rows), s.head_dim, lane);
      } else {
        if (rows > 0 && 64 * h < s.head_dim)
          bwd_store_box(&tm_dq, C::stage(smem, J - 1) + (warp - 4) * 4096, tmem + lane_base + 384 + 64 * h,
                        64 * h, it.r0 + quarter * 32, it.run, p.scale, false, lane);
        if (lane == 0) {
          bulk_wait_read();  // the slot goes back to the loader
          mbar_arrive(&v_empty[(J - 1) & 1]);
        }
      }
      i = next;
      it = next_it;
    }
    if (lane == 0) bulk_wait_all();  // stores done before the CTA exits
  }
  // One CTA is enough: the kernel has not ended before it has.
  if (blockIdx.x == gridDim.x - 1 && threadIdx.x == 0) grid_wait();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace gqa
