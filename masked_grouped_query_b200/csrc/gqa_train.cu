// gqa_train.cu -- host side of the backward pass and of the rotary positions
// in libgqa_attn.so: argument checks, plans and launches behind the C ABI of
// gqa_attn.h.  The kernels are included below; gqa_attn.cu holds the rest of
// the library.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <mutex>

#include "gqa_attn.h"
#include "host.h"
#include "status.cuh"
#include "ptx.cuh"
#include "mask.cuh"
#include "backward.cuh"
#include "backward_sm100.cuh"
#include "rotary.cuh"

namespace {

using namespace gqa;
using gqa_host::cuda_fail;
using gqa_host::detail;
using gqa_host::overlaps;

std::mutex g_attr_mu;
constexpr int kMaxDevices = 64;

inline long long ceil_div(long long a, long long b) { return (a + b - 1) / b; }

// Sets a kernel's dynamic shared memory limit once per device.
template <typename K>
int allow_smem(K kernel, int bytes, int device, bool* done) {
  std::lock_guard<std::mutex> lk(g_attr_mu);
  if (done[device]) return GQA_ATTN_OK;
  const cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return cuda_fail("cudaFuncSetAttribute(backward)", e, GQA_ATTN_ERR_LAUNCH);
  done[device] = true;
  return GQA_ATTN_OK;
}

int launched(const char* where) {
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? GQA_ATTN_OK : cuda_fail(where, e, GQA_ATTN_ERR_LAUNCH);
}

// ------------------------------------------------------------------ backward
// Sizes and the row layout of a backward call (see BwdShape).
int bwd_shape(int batch, int q_len, int kv_len, int hq, int hkv, int d, int causal, int window,
              BwdShape* s) {
  if (batch < 0 || q_len < 0 || kv_len < 0 || hq < 1 || hkv < 1) return GQA_ATTN_ERR_BAD_SHAPE;
  if (hq % hkv != 0) return GQA_ATTN_ERR_HEAD_RATIO;
  if (d < 8 || d > 256 || d % 8 != 0) return GQA_ATTN_ERR_HEAD_DIM;
  const int group = hq / hkv;
  // Row and key indexes are 32-bit, with room for the last tile's padding.
  constexpr long long kMost = 0x7fff0000LL;
  if ((long long)group * q_len > kMost || kv_len > kMost || (long long)batch * hq > kMost)
    return GQA_ATTN_ERR_TOO_LARGE;
  s->q_len = q_len;
  s->kv_len = kv_len;
  s->head_dim = d;
  s->causal = causal ? 1 : 0;
  s->window = window > 0 ? window : 0;
  const bool per_head = (s->causal || s->window) && q_len >= 256;
  s->runs_per_unit = per_head ? group : 1;
  s->run = per_head ? q_len : group * q_len;
  s->tiles = (int)ceil_div(s->run, 128);
  s->units = (long long)batch * hkv;
  s->runs = s->units * s->runs_per_unit;
  // One block per row tile and per key tile (64 rows at the least), and the
  // statistics' bytes in a size_t with room to spare.
  if (s->runs * s->tiles * 2 > kMost || s->units * ceil_div(kv_len, 64) > kMost)
    return GQA_ATTN_ERR_TOO_LARGE;
  return GQA_ATTN_OK;
}

// How the walks are cut, and where the scratch holds what.
struct BwdPlan {
  int tile;  // rows of a key or row tile: 128 (tcgen05) or 64
  long long key_tiles, row_tiles;
  int kv_splits, q_splits;
  bool fine;
  size_t off_dk, off_dv, off_dq, bytes;
};

// Parts of a walk of `steps` steps, `items` walks in all.  A part's start and
// its share of the join cost about as much as four steps, so no part is
// shorter, and walks under twelve steps (of the mma.sync kernels: eight, whose
// step is the longer one) stay whole; the parts fill one CTA per SM of the
// full GPU at most (a fixed number: the scratch size is host arithmetic).
// Measured, microseconds whole and cut (batch, queries, keys, heads, width):
//   3, 3352, 64, 12:4, 32:  248 and 78     1, 1, 32768, 8:1, 128: 295 and 82
//   1, 2048, 2048, 4:1, 128: 115 and 48    2, 1, 4096, 32:8, 128: 60 and 49
//   1, 2048, 2048, 1:1, 128: 36 and 27     1, 2048, 2048, 1:1, 256: 161 and 92
// and with 8 steps (1, 1024, 1024, 8:8, 64) 21 and 26, or in parts of one or
// two steps 27 to 41 where parts of four take 23 to 27; mma.sync with 10 steps
// (1, 600, 600, 2:1, 256) 60 and 41.
constexpr int kBwSplitCtas = 148;
int bwd_splits(long long items, long long steps, int tile) {
  if (items <= 0 || steps < (tile == 64 ? 8 : 12) || 2 * items > kBwSplitCtas) return 1;
  const long long fit = kBwSplitCtas / items, most = steps / 4;
  return (int)(fit < most ? fit : most);
}

// Problems of at most this many steps (one per SM) take P and dS in two bf16
// terms.  Their gradients' error, in the 2-norm, then is the outputs' rounding
// alone, 1.7e-3; with one term it is 2.4e-3, and where few products make a
// gradient up to twice the rounding.  So the same rows may give gradients that
// differ by that rounding in a larger batch.  Measured, microseconds with one
// and two terms (captured calls): 23 and 27 (1, 128, 128, 4:1, 128), 16 and 20
// (1, 512, 512, 2:2, 128), where an uncaptured call takes 28 for its launches
// anyhow; but 21 and 27 for 512 steps (1, 1024, 1024, 8:8, 64), 1519 and 2159
// for the largest case.
constexpr long long kBwFineSteps = 148;

BwdPlan bwd_plan(const BwdShape& s, bool may_split) {
  BwdPlan pl;
  pl.tile = s.head_dim > 128 ? 64 : 128;
  pl.key_tiles = s.units * ceil_div(s.kv_len, pl.tile);
  pl.row_tiles = s.runs * ceil_div(s.run, pl.tile);
  // The longest walk: every tile of the other side, or what a window shows.
  long long rows = ceil_div(s.run, pl.tile), keys = ceil_div(s.kv_len, pl.tile);
  if (s.window > 0) {
    const long long span = s.run == s.q_len ? pl.tile : s.q_len;  // positions in a row tile
    const long long seen = ((long long)s.window + span + pl.tile - 2) / pl.tile + 1;
    if (s.run == s.q_len && seen < rows) rows = seen;
    if (seen < keys) keys = seen;
  }
  const long long steps = pl.key_tiles * (rows * s.runs_per_unit);
  pl.fine = steps <= kBwFineSteps;
  pl.kv_splits = may_split ? bwd_splits(pl.key_tiles, rows * s.runs_per_unit, pl.tile) : 1;
  pl.q_splits = may_split ? bwd_splits(pl.row_tiles, keys, pl.tile) : 1;
  auto align = [](size_t x) { return (x + 255) & ~(size_t)255; };
  const size_t part = (size_t)pl.tile * ((s.head_dim + 15) / 16 * 16) * sizeof(float);
  const size_t kv = pl.kv_splits > 1 ? align((size_t)pl.key_tiles * pl.kv_splits * part) : 0;
  const size_t q = pl.q_splits > 1 ? align((size_t)pl.row_tiles * pl.q_splits * part) : 0;
  pl.off_dk = (size_t)s.runs * (size_t)s.tiles * 256 * sizeof(float);
  pl.off_dv = pl.off_dk + kv;
  pl.off_dq = pl.off_dv + kv;
  pl.bytes = pl.off_dq + q;
  return pl;
}

// A launch that may start before the kernel ahead of it in the stream ends
// (see the head of backward_sm100.cuh).
template <typename... P, typename... A>
int launch_after(const char* where, void (*kernel)(P...), long long grid, int threads, int smem,
                 cudaStream_t st, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
  return e == cudaSuccess ? GQA_ATTN_OK : cuda_fail(where, e, GQA_ATTN_ERR_LAUNCH);
}

template <int KS, bool kFine>
int launch_bwd_mma(const BwdParams& p, int device, cudaStream_t st) {
  using C = BwdMmaCfg<KS>;
  static bool done_kv[kMaxDevices], done_q[kMaxDevices];
  int rc = allow_smem(bwd_mma_kernel<KS, false, kFine>, C::kSmemBytes, device, done_kv);
  if (rc == GQA_ATTN_OK) rc = allow_smem(bwd_mma_kernel<KS, true, kFine>, C::kSmemBytes, device, done_q);
  if (rc != GQA_ATTN_OK) return rc;
  const long long key_tiles = p.sh.units * ceil_div(p.sh.kv_len, kBmTile);
  if ((rc = launch_after("launch(backward dK dV)", bwd_mma_kernel<KS, false, kFine>, key_tiles * p.kv_splits, kBmThreads,
                         C::kSmemBytes, st, p)) != GQA_ATTN_OK)
    return rc;
  const long long row_tiles = p.sh.runs * ceil_div(p.sh.run, kBmTile);
  return launch_after("launch(backward dQ)", bwd_mma_kernel<KS, true, kFine>, row_tiles * p.q_splits, kBmThreads,
                      C::kSmemBytes, st, p);
}

// Shared memory limit of a tcgen05 backward kernel, and the check that its
// register split fits what the block is launched with (setmaxnreg.inc could
// never be granted otherwise).
template <typename K>
int bwd_sm100_setup(K kernel, int bytes, int device, bool* done) {
  {
    std::lock_guard<std::mutex> lk(g_attr_mu);
    if (done[device]) return GQA_ATTN_OK;
  }
  cudaFuncAttributes fa;
  const cudaError_t e = cudaFuncGetAttributes(&fa, kernel);
  if (e != cudaSuccess) return cuda_fail("cudaFuncGetAttributes(backward)", e, GQA_ATTN_ERR_LAUNCH);
  if (fa.numRegs * kBwThreads < kBwRegTotal)
    return detail(GQA_ATTN_ERR_LAUNCH, "backward kernel built with %d registers/thread: register "
                  "split needs %d", fa.numRegs, kBwRegTotal);
  return allow_smem(kernel, bytes, device, done);
}

template <int DCH, bool kCap, bool kFine>
int launch_bwd_sm100(const BwdParams& p, int device, int sms, cudaStream_t st) {
  using C = BwdCfg<DCH>;
  static bool done_kv[kMaxDevices], done_q[kMaxDevices];
  int rc = bwd_sm100_setup(bwd_dkdv_kernel<DCH, kCap, kFine>, C::kSmemBytes, device, done_kv);
  if (rc == GQA_ATTN_OK) rc = bwd_sm100_setup(bwd_dq_kernel<DCH, kCap, kFine>, C::kSmemBytes, device, done_q);
  if (rc != GQA_ATTN_OK) return rc;
  const BwdShape& s = p.sh;
  CUtensorMap q, dout, k, v, dq, dk, dv;
  const struct {
    CUtensorMap* map;
    const void* base;
    bool rows;
    int box;
  } maps[7] = {{&q, p.q, true, 128},  {&dout, p.dout, true, 128}, {&k, p.k, false, 128},
               {&v, p.v, false, 128}, {&dq, p.dq, true, 32},      {&dk, p.dk, false, 32},
               {&dv, p.dv, false, 32}};
  for (const auto& m : maps)
    if ((rc = gqa_host::tensor_map(m.map, m.base, s.head_dim, m.rows ? s.run : s.kv_len,
                                   m.rows ? s.runs : s.units, m.box)) != GQA_ATTN_OK)
      return rc;
  const long long key_tiles = s.units * ceil_div(s.kv_len, 128) * p.kv_splits;
  const long long row_tiles = s.runs * s.tiles * p.q_splits;
  if ((rc = launch_after("launch(backward dK dV)", bwd_dkdv_kernel<DCH, kCap, kFine>,
                         key_tiles < sms ? key_tiles : sms, kBwThreads, C::kSmemBytes, st, q, dout, k,
                         v, dk, dv, p)) != GQA_ATTN_OK)
    return rc;
  // Four CTAs per SM, one after the other, even out what the key tiles left
  // uneven (one SM's share at a time would keep it).
  const long long q_grid = row_tiles < 4LL * sms ? row_tiles : 4LL * sms;
  return launch_after("launch(backward dQ)", bwd_dq_kernel<DCH, kCap, kFine>, q_grid, kBwThreads,
                      C::kSmemBytes, st, q, dout, k, v, dq, p);
}

template <int DCH>
int launch_bwd_sm100_d(const BwdParams& p, bool fine, int device, int sms, cudaStream_t st) {
  if (fine)
    return p.softcap ? launch_bwd_sm100<DCH, true, true>(p, device, sms, st)
                     : launch_bwd_sm100<DCH, false, true>(p, device, sms, st);
  return p.softcap ? launch_bwd_sm100<DCH, true, false>(p, device, sms, st)
                   : launch_bwd_sm100<DCH, false, false>(p, device, sms, st);
}

// ------------------------------------------------------------------ rotary
template <int V, typename TI, typename TO>
int launch_rotary(const RotaryParams& p, bool interleaved, dim3 grid, cudaStream_t st) {
  if (interleaved)
    rotary_kernel<V, TI, TO, true><<<grid, kRotThreads, 0, st>>>(p);
  else
    rotary_kernel<V, TI, TO, false><<<grid, kRotThreads, 0, st>>>(p);
  return launched("launch(rotary)");
}

template <int V>
int launch_rotary_types(const RotaryParams& p, bool in32, bool out32, bool interleaved, dim3 grid,
                        cudaStream_t st) {
  using B = __nv_bfloat16;
  if (in32)
    return out32 ? launch_rotary<V, float, float>(p, interleaved, grid, st)
                 : launch_rotary<V, float, B>(p, interleaved, grid, st);
  return out32 ? launch_rotary<V, B, float>(p, interleaved, grid, st)
               : launch_rotary<V, B, B>(p, interleaved, grid, st);
}

}  // namespace

namespace gqa_host {

cudaError_t train_status(uint32_t* word) {
  return cudaMemcpyFromSymbol(word, gqa::g_gqa_status, sizeof *word);
}
cudaError_t train_clear_status() {
  const uint32_t z = 0;
  return cudaMemcpyToSymbol(gqa::g_gqa_status, &z, sizeof z);
}

}  // namespace gqa_host

extern "C" {

int gqa_attn_bwd_scratch(int batch, int q_len, int kv_len, int num_q_heads, int num_kv_heads,
                         int head_dim, int causal, int window, size_t* bytes) {
  BwdShape s;
  const int rc = bwd_shape(batch, q_len, kv_len, num_q_heads, num_kv_heads, head_dim, causal,
                           window, &s);
  if (rc != GQA_ATTN_OK) return rc;
  if (bytes) *bytes = bwd_plan(s, true).bytes;
  return GQA_ATTN_OK;
}

int gqa_attn_bwd(const void* dout, const void* q, const void* k, const void* v, const void* o,
                 const float* lse, const float* dlse, void* dq, void* dk, void* dv, void* scratch,
                 size_t scratch_bytes, int batch, int q_len, int kv_len, int num_q_heads,
                 int num_kv_heads, int head_dim, int causal, int window, float softcap,
                 void* stream) {
  BwdParams p;
  BwdShape& s = p.sh;
  int rc = bwd_shape(batch, q_len, kv_len, num_q_heads, num_kv_heads, head_dim, causal, window, &s);
  if (rc != GQA_ATTN_OK) return rc;
  if (!(softcap >= 0.0f) || std::isinf(softcap)) return GQA_ATTN_ERR_SOFTCAP;
  const size_t rows = (size_t)batch * num_q_heads * (size_t)q_len;
  const size_t q_bytes = rows * head_dim * 2, stat_bytes = rows * 4;
  const size_t kv_bytes = (size_t)batch * num_kv_heads * (size_t)kv_len * head_dim * 2;
  if (q_bytes && (!dout || !q || !o || !lse || !dq)) return GQA_ATTN_ERR_NULL_POINTER;
  if (kv_bytes && (!k || !v || !dk || !dv)) return GQA_ATTN_ERR_NULL_POINTER;
  if (((uintptr_t)dout | (uintptr_t)q | (uintptr_t)k | (uintptr_t)v | (uintptr_t)o |
       (uintptr_t)lse | (uintptr_t)dlse | (uintptr_t)dq | (uintptr_t)dk | (uintptr_t)dv |
       (uintptr_t)scratch) & 15u)
    return GQA_ATTN_ERR_MISALIGNED;
  const bool work = q_bytes && kv_bytes;
  softcap = std::min(softcap, gqa_host::kSoftcapMost);
  p.softcap = softcap > 0.f;
  p.scale = 1.0f / std::sqrt((float)head_dim);
  p.cap_in = p.softcap ? gqa_host::softcap_in(p.scale, softcap) : 0.f;
  constexpr float k7[4] = {kTanhC1, kTanhC3, kTanhC5, kTanhC7};
  p.poly_most = p.softcap ? gqa_host::softcap_fold_most(k7, p.cap_in, 1.f, 0.5f) : 0.f;
  // (force_path 1 takes the mma.sync kernels for narrow heads too, uncut.)
  const bool narrow_mma = head_dim <= 128 && gqa_host::forced_path() == 1;
  const BwdPlan pl = bwd_plan(s, !narrow_mma);
  const size_t need = work ? pl.bytes : 0;
  if (need && !scratch) return GQA_ATTN_ERR_NULL_POINTER;
  if (scratch_bytes < need)
    return detail(GQA_ATTN_ERR_ARG, "backward scratch of %zu bytes, needs %zu", scratch_bytes, need);
  const void* outs[4] = {dq, dk, dv, scratch};
  const size_t out_bytes[4] = {q_bytes, kv_bytes, kv_bytes, need};
  const void* ins[7] = {dout, q, k, v, o, lse, dlse};
  const size_t in_bytes[7] = {q_bytes, q_bytes, kv_bytes, kv_bytes, q_bytes, stat_bytes, stat_bytes};
  for (int i = 0; i < 4; ++i) {
    for (int j = 0; j < 7; ++j)
      if (overlaps(outs[i], out_bytes[i], ins[j], in_bytes[j])) return GQA_ATTN_ERR_ALIAS;
    for (int j = 0; j < i; ++j)
      if (overlaps(outs[i], out_bytes[i], outs[j], out_bytes[j])) return GQA_ATTN_ERR_ALIAS;
  }
  if (!q_bytes && !kv_bytes) return GQA_ATTN_OK;
  int device = 0, sms = 0;
  if ((rc = gqa_host::device(&device, &sms)) != GQA_ATTN_OK) return rc;
  cudaStream_t st = (cudaStream_t)stream;
  if (!work) {  // no queries or no keys: every gradient that exists is zero
    cudaError_t e = cudaSuccess;
    if (q_bytes) e = cudaMemsetAsync(dq, 0, q_bytes, st);
    if (kv_bytes) e = cudaMemsetAsync(dk, 0, kv_bytes, st);
    if (kv_bytes && e == cudaSuccess) e = cudaMemsetAsync(dv, 0, kv_bytes, st);
    return e == cudaSuccess ? GQA_ATTN_OK : cuda_fail("cudaMemsetAsync(gradient)", e, GQA_ATTN_ERR_LAUNCH);
  }
  p.q = (const __nv_bfloat16*)q;
  p.k = (const __nv_bfloat16*)k;
  p.v = (const __nv_bfloat16*)v;
  p.dout = (const __nv_bfloat16*)dout;
  p.dq = (__nv_bfloat16*)dq;
  p.dk = (__nv_bfloat16*)dk;
  p.dv = (__nv_bfloat16*)dv;
  p.stats = (const float*)scratch;
  p.kv_splits = pl.kv_splits;
  p.q_splits = pl.q_splits;
  p.part_dk = (float*)((char*)scratch + pl.off_dk);
  p.part_dv = (float*)((char*)scratch + pl.off_dv);
  p.part_dq = (float*)((char*)scratch + pl.off_dq);
  p.logit_scale = kLog2e32 * p.scale;
  p.cap_out = p.softcap ? softcap * kLog2e32 : 0.f;
  bwd_stats_kernel<<<(unsigned)(s.runs * s.tiles), kBwStatThreads, 0, st>>>(
      p.dout, (const __nv_bfloat16*)o, lse, dlse, (float*)scratch, s);
  if ((rc = launched("launch(backward statistics)")) != GQA_ATTN_OK) return rc;
  // The tcgen05 kernels hold dK and dV of 128 columns each in TMEM next to the
  // scores: wider heads stay on mma.sync.
  if (head_dim > 128)
    rc = (pl.fine ? launch_bwd_mma<16, true> : launch_bwd_mma<16, false>)(p, device, st);
  else if (narrow_mma)
    rc = (pl.fine ? launch_bwd_mma<8, true> : launch_bwd_mma<8, false>)(p, device, st);
  else
    rc = (head_dim <= 64 ? launch_bwd_sm100_d<1> : launch_bwd_sm100_d<2>)(p, pl.fine, device, sms, st);
  if (rc != GQA_ATTN_OK || (pl.kv_splits == 1 && pl.q_splits == 1)) return rc;
  BwdJoin j;
  j.job[0] = {p.part_dk, p.dk, p.scale, pl.kv_splits, kv_len, s.units, pl.key_tiles};
  j.job[1] = {p.part_dv, p.dv, 1.0f, pl.kv_splits, kv_len, s.units, pl.key_tiles};
  j.job[2] = {p.part_dq, p.dq, p.scale, pl.q_splits, s.run, s.runs, pl.row_tiles};
  j.tile_rows = pl.tile;
  j.head_dim = head_dim;
  const long long most = (pl.kv_splits > 1 ? pl.key_tiles : 0) > (pl.q_splits > 1 ? pl.row_tiles : 0)
                             ? pl.key_tiles : pl.row_tiles;
  bwd_join_kernel<<<dim3((unsigned)most, 3), 256, 0, st>>>(j);
  return launched("launch(backward join)");
}

int gqa_attn_rotary(const void* q, const void* k, void* q_out, void* k_out, const void* positions,
                    int batch, int length, int num_q_heads, int num_kv_heads, int head_dim,
                    int num_axes, const int* sections, double theta, unsigned int flags,
                    void* stream) {
  if (flags & ~0xffu) return GQA_ATTN_ERR_ARG;
  if (batch < 0 || length < 0 || num_q_heads < 0 || num_kv_heads < 0 ||
      num_q_heads + (long long)num_kv_heads < 1)
    return GQA_ATTN_ERR_BAD_SHAPE;
  if (head_dim < 8 || head_dim > 256 || head_dim % 8 != 0) return GQA_ATTN_ERR_HEAD_DIM;
  if (num_axes < 1 || num_axes > kRotMaxAxes || !sections)
    return detail(GQA_ATTN_ERR_ARG, "rotary: %d axes, takes 1 to %d", num_axes, kRotMaxAxes);
  if (!(theta > 0.0) || std::isinf(theta)) return detail(GQA_ATTN_ERR_ARG, "rotary: theta %g", theta);
  long long pairs = 0;
  for (int a = 0; a < num_axes; ++a) {
    if (sections[a] < 1) return detail(GQA_ATTN_ERR_ARG, "rotary: section of %d pairs", sections[a]);
    pairs += sections[a];
  }
  if (2 * pairs > head_dim)
    return detail(GQA_ATTN_ERR_ARG, "rotary: %lld pairs in a head of %d", pairs, head_dim);
  const bool in32 = flags & GQA_ROTARY_IN_F32, out32 = flags & GQA_ROTARY_OUT_F32;
  const bool in_seq = flags & GQA_ROTARY_IN_SEQ_MAJOR, out_seq = flags & GQA_ROTARY_OUT_SEQ_MAJOR;
  const bool interleaved = flags & GQA_ROTARY_INTERLEAVED;
  const long long tokens = (long long)batch * length;
  const long long heads = (long long)num_q_heads + num_kv_heads;
  if (heads > 65535 || tokens > (1LL << 38)) return GQA_ATTN_ERR_TOO_LARGE;
  const size_t n[2] = {(size_t)tokens * num_q_heads * head_dim, (size_t)tokens * num_kv_heads * head_dim};
  const void* in[2] = {q, k};
  void* out[2] = {q_out, k_out};
  if (tokens && !positions) return GQA_ATTN_ERR_NULL_POINTER;
  uintptr_t bits = (uintptr_t)positions;
  if (num_q_heads) bits |= (uintptr_t)q | (uintptr_t)q_out;
  if (num_kv_heads) bits |= (uintptr_t)k | (uintptr_t)k_out;
  if (bits & 15u) return GQA_ATTN_ERR_MISALIGNED;
  const size_t ie = in32 ? 4 : 2, oe = out32 ? 4 : 2;
  const size_t pos_bytes = (size_t)num_axes * (size_t)tokens * ((flags & GQA_ROTARY_POS_I64) ? 8 : 4);
  for (int w = 0; w < 2; ++w) {
    if (n[w] && (!in[w] || !out[w])) return GQA_ATTN_ERR_NULL_POINTER;
    if (overlaps(out[w], n[w] * oe, positions, pos_bytes)) return GQA_ATTN_ERR_ALIAS;
    // In place is fine where every element stays where it is.
    if (!(out[w] == in[w] && in32 == out32 && in_seq == out_seq) &&
        overlaps(out[w], n[w] * oe, in[w], n[w] * ie))
      return GQA_ATTN_ERR_ALIAS;
    if (overlaps(out[w], n[w] * oe, in[1 - w], n[1 - w] * ie)) return GQA_ATTN_ERR_ALIAS;
  }
  if (overlaps(q_out, n[0] * oe, k_out, n[1] * oe)) return GQA_ATTN_ERR_ALIAS;
  if (tokens == 0) return GQA_ATTN_OK;
  int device = 0, sms = 0;
  const int rc = gqa_host::device(&device, &sms);
  if (rc != GQA_ATTN_OK) return rc;
  RotaryParams p;
  p.q = q;
  p.k = k;
  p.q_out = q_out;
  p.k_out = k_out;
  p.positions = positions;
  p.pos64 = (flags & GQA_ROTARY_POS_I64) ? 1 : 0;
  p.inverse = (flags & GQA_ROTARY_INVERSE) ? 1 : 0;
  p.batch = batch;
  p.length = length;
  p.head_dim = head_dim;
  p.q_heads = num_q_heads;
  p.kv_heads = num_kv_heads;
  p.pairs = (int)pairs;
  // Strides of the dense [batch][length][heads][d] and [batch][heads][length][d].
  for (int w = 0; w < 2; ++w) {
    const long long h = w ? num_kv_heads : num_q_heads, d = head_dim;
    p.in_b[w] = p.out_b[w] = h * length * d;
    p.in_h[w] = in_seq ? d : (long long)length * d;
    p.in_l[w] = in_seq ? h * d : d;
    p.out_h[w] = out_seq ? d : (long long)length * d;
    p.out_l[w] = out_seq ? h * d : d;
  }
  // Frequency of pair i: theta^(-i / pairs), or theta^(-j / section) for the
  // j-th pair of its axis, as turns per position.  A running product in the
  // wider type: ratio's own rounding enters every power, 128 of them lose seven
  // bits, of which fp64 has none to spare at positions of 2^31.  128 pairs take
  // a host core 0.6 us so; 1.7 with a power for each, 0.2 in fp64.
  const long double pi2 = 6.283185307179586476925286766559L;
  const bool per_axis = flags & GQA_ROTARY_PER_AXIS;
  long double ratio = std::pow((long double)theta, -1.0L / pairs), f = 1.0L;
  int at = 0;
  for (int a = 0; a < num_axes; ++a) {
    if (per_axis) {
      ratio = std::pow((long double)theta, -1.0L / sections[a]);
      f = 1.0L;
    }
    for (int j = 0; j < sections[a]; ++j, ++at, f *= ratio) {
      p.turn[at] = (double)(f / pi2);
      p.axis[at] = (unsigned char)a;
    }
  }
  // The widest vector that keeps every access aligned: 8 bf16 (16 bytes) or
  // 4 elements when the pairs divide by it, else single elements.
  const int v = pairs % 8 == 0 && !in32 && !out32 && !interleaved ? 8 : pairs % 4 == 0 ? 4 : 1;
  p.vecs = ((int)pairs + (head_dim - 2 * (int)pairs)) / v;
  // All heads of a token in one thread, unless that leaves an SM with less
  // than its 2048 threads: then runs of heads, down to a single one.  (At 1024
  // or 4096 threads the measured cases take up to 10% longer.)
  const long long threads = tokens * p.vecs;
  const long long runs = ceil_div((long long)sms * 2048, threads);
  p.heads_per_thread = (int)(runs >= heads ? 1 : ceil_div(heads, runs));
  const long long gx = ceil_div(threads, kRotThreads);
  if (gx > 0x7fffffffLL) return GQA_ATTN_ERR_TOO_LARGE;
  const dim3 grid((unsigned)gx, (unsigned)ceil_div(heads, p.heads_per_thread));
  cudaStream_t st = (cudaStream_t)stream;
  if (v == 8) {
    rotary_kernel<8, __nv_bfloat16, __nv_bfloat16, false><<<grid, kRotThreads, 0, st>>>(p);
    return launched("launch(rotary)");
  }
  if (v == 4) return launch_rotary_types<4>(p, in32, out32, interleaved, grid, st);
  return launch_rotary_types<1>(p, in32, out32, interleaved, grid, st);
}

}  // extern "C"
