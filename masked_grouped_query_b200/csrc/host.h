// host.h -- host-side pieces that gqa_attn.cu offers to the library's other
// translation unit.
#pragma once

#include <cfloat>
#include <cmath>

#include <algorithm>

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace gqa_host {

// The current device: checked for compute capability 10.x (GQA_ATTN_ERR_DEVICE
// otherwise); *index gets its number, *sms its SM count.
int device(int* index, int* sms);

// 3-D bf16 tensor map over [outer][rows][cols] with a (64 cols x box_rows x 1)
// box and 128-byte swizzle; out-of-range elements read as zero.
int tensor_map(CUtensorMap* map, const void* base, int cols, long long rows, long long outer,
               int box_rows);

// Value of the force_path override (0 automatic, 1 mma.sync, 2 tcgen05).
int forced_path();

// Remember a failed CUDA call for gqa_attn_last_error_detail; returns `code`.
int cuda_fail(const char* where, cudaError_t e, int code);
// The same for a message of this library.
int detail(int code, const char* fmt, ...);

// The training operators take softcaps above this one as this one: neither
// changes a logit up to 1e26 in fp32 (by (x / cap)^2 / 3 of itself), and with
// this one the scales derived from it stay normal numbers.
constexpr float kSoftcapMost = 1e30f;
// 1 / (sqrt(head_dim) * softcap), finite (and so with log2(e) etc.) for every softcap.
inline float softcap_in(float scale, float softcap) { return std::min(scale / softcap, 1e37f); }

// The kernels evaluate scale * tanh(x * cap_in) as x Q(x^2), with scale and
// cap_in's powers folded into the coefficients k of tanh's odd polynomial on
// [0, most] (one product per pair of scores less than scaling x first).  The
// largest |x * cap_in| for which that is good to 2e-8: `most`, less where a term
// underflows, so that what is lost of it stays below; none (-1) where powers
// could overflow, for softcaps below 1e-3.  Past it they take an exponential.
template <int N>
float softcap_fold_most(const float (&k)[N], float cap_in, float scale, float most) {
  if (cap_in > 1e3f) return -1.f;
  double f = (double)scale * cap_in;
  for (int i = 0; i < N; ++i, f *= (double)cap_in * cap_in)
    if (std::fabs(f * k[i]) < FLT_MIN)
      most = std::min(most, (float)std::pow(2e-8 / std::fabs(k[i]), 1.0 / (2 * i + 1)));
  return most;
}

bool overlaps(const void* a, size_t na, const void* b, size_t nb);

// Defined in gqa_train.cu: its status word (returns a CUDA error).
cudaError_t train_status(uint32_t* word);
cudaError_t train_clear_status();

}  // namespace gqa_host
