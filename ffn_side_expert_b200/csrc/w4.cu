// w4.cu -- rows grouped by expert times 4-bit weights with group scales, and the whole expert
// (gate/up, SwiGLU, down) on such weights, for the few rows an expert gets in a decode
// micro-batch.
//
//   W[n][k] = (q[n][k] - z[n][k / G]) * scale[n][k / G],  q, z in 0..15 (z = 8 without zero points)
//   y[r][n] = sum_k x[r][k] W[n][k]                         per expert, fp32 sums
//   act = silu(x Wg^T) * (x Wu^T),  Y = act W2^T
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "afd_ffn.h"
#include "common.cuh"
#include "internal.h"

namespace afd {
namespace {

constexpr int kW4MaxExperts = 256;

struct W4Args {
  const uint8_t* codes;
  const void* scale;
  const uint8_t* zero;
  const __nv_bfloat16* x;   // [n_rows][K]; with planes = 2 a second plane of low parts follows
  const int32_t* counts;    // [E], or nullptr: one expert, every row
  void* y;
  int E, N, K, G, n_rows, scale_f32, y_f32, planes;
  int* err;
};

// The expert's first row and its rows, from counts: negative counts are flagged and taken as
// 0, rows past n_rows are flagged and cut off.
__device__ __forceinline__ void expert_rows(const W4Args& a, int e, int* first, int* rows) {
  int at = 0, mine = a.n_rows;
  if (a.counts) {
    long long sum = 0;
    int bad = 0;
    for (int f = 0; f < e; ++f) {
      const int c = a.counts[f];
      sum += max(c, 0);
      bad |= c < 0;
    }
    const int c = a.counts[e];
    bad |= c < 0;
    at = static_cast<int>(min(sum, static_cast<long long>(a.n_rows)));
    mine = min(max(c, 0), a.n_rows - at);
    bad |= sum + max(c, 0) > a.n_rows;
    if (bad && threadIdx.x == 0) atomicOr(a.err, kErrBadOffsets);
  }
  *first = at;
  *rows = mine;
}

__device__ __forceinline__ void w4_dot(const W4Args& a, int e, int n, int first, int m, int lane, float (&acc)[8]) {
  const uint32_t* q = reinterpret_cast<const uint32_t*>(a.codes + (static_cast<size_t>(e) * a.N + n) * (a.K / 2));
  const size_t gp = (static_cast<size_t>(e) * a.N + n) * (a.K / a.G);
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = 0.f;
  for (int w = lane; w < a.K / 8; w += 32) {
    const uint32_t word = q[w];
    const size_t g = gp + w * 8 / a.G;
    const float sc = a.scale_f32 ? static_cast<const float*>(a.scale)[g]
                                 : __bfloat162float(static_cast<const __nv_bfloat16*>(a.scale)[g]);
    const float z = a.zero ? static_cast<float>(a.zero[g] & 15) : 8.f;
    for (int i = 0; i < m; ++i) {
      float d = 0.f;
      for (int p = 0; p < a.planes; ++p) {
        const __nv_bfloat16* x = a.x + (static_cast<size_t>(p) * a.n_rows + first + i) * a.K + w * 8;
        for (int j = 0; j < 8; ++j)
          d = fmaf(__bfloat162float(x[j]), static_cast<float>((word >> (4 * j)) & 15u) - z, d);
      }
      acc[i] = fmaf(d, sc, acc[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = warp_sum(acc[i]);
}

template <bool SWIGLU>
__global__ void __launch_bounds__(256) w4_rows_kernel(const W4Args a) {
  const int e = blockIdx.y, lane = threadIdx.x & 31, n = blockIdx.x * 8 + (threadIdx.x >> 5);
  const int outs = SWIGLU ? a.N / 2 : a.N;
  int first, rows;
  expert_rows(a, e, &first, &rows);
  if (n >= outs) return;
  for (int r0 = 0; r0 < rows; r0 += 8) {
    const int m = min(8, rows - r0);
    float v[8];
    w4_dot(a, e, n, first + r0, m, lane, v);
    if constexpr (SWIGLU) {
      float u[8];
      w4_dot(a, e, n + outs, first + r0, m, lane, u);
      for (int i = 0; i < m; ++i) {
        const float act = v[i] / (1.f + expf(-v[i])) * u[i];
        const __nv_bfloat16 hi = __float2bfloat16_rn(act);
        const size_t at = static_cast<size_t>(first + r0 + i) * outs + n;
        if (lane == 0) {
          static_cast<__nv_bfloat16*>(a.y)[at] = hi;
          static_cast<__nv_bfloat16*>(a.y)[static_cast<size_t>(a.n_rows) * outs + at] =
              __float2bfloat16_rn(act - __bfloat162float(hi));
        }
      }
    } else if (lane == 0) {
      for (int i = 0; i < m; ++i) {
        const size_t at = static_cast<size_t>(first + r0 + i) * outs + n;
        if (a.y_f32) static_cast<float*>(a.y)[at] = v[i];
        else static_cast<__nv_bfloat16*>(a.y)[at] = __float2bfloat16_rn(v[i]);
      }
    }
  }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int check_w4(const afd_ffn_w4* w, int32_t E) {
  if (!w || E < 1 || w->N < 1 || w->K < 32 || w->K % 32 != 0 || w->group < 32 || w->group % 32 != 0 ||
      w->K % w->group != 0)
    return AFD_ERR_INVALID_ARG;
  if (w->scale_dtype != AFD_DT_BF16 && w->scale_dtype != AFD_DT_F32) return AFD_ERR_INVALID_ARG;
  if (E > kW4MaxExperts || static_cast<long long>(E) * w->N > (1LL << 30) || w->K > (1 << 20)) return AFD_ERR_UNSUPPORTED;
  return AFD_OK;
}

int check_w4_pointers(const afd_ffn_w4* w) {
  const uintptr_t size = w->scale_dtype == AFD_DT_F32 ? 4 : 2;
  if (!w->codes || !w->scale || !aligned16(w->codes) || reinterpret_cast<uintptr_t>(w->scale) % size != 0)
    return AFD_ERR_INVALID_ARG;
  return AFD_OK;
}

template <bool SWIGLU>
void launch_w4(const afd_ffn_w4& w, int E, const void* x, int planes, const int32_t* counts, int n_rows, void* y,
               int y_f32, int* err, cudaStream_t s) {
  W4Args a{static_cast<const uint8_t*>(w.codes), w.scale, w.zero, static_cast<const __nv_bfloat16*>(x), counts, y,
           E, w.N, w.K, w.group, n_rows, w.scale_dtype == AFD_DT_F32, y_f32, planes, err};
  const int outs = SWIGLU ? w.N / 2 : w.N;
  w4_rows_kernel<SWIGLU><<<dim3((outs + 7) / 8, E), 256, 0, s>>>(a);
}

}  // namespace
}  // namespace afd

using namespace afd;

extern "C" int afd_ffn_w4_rows(const afd_ffn_w4* w, int32_t E, const void* x, const int32_t* counts, int32_t n_rows,
                               void* y, int32_t y_dtype, void* stream) {
  int st = check_w4(w, E);
  if (st != AFD_OK) return st;
  if (n_rows < 0 || (y_dtype != AFD_DT_BF16 && y_dtype != AFD_DT_F32)) return AFD_ERR_INVALID_ARG;
  if ((!counts && E != 1) || (reinterpret_cast<uintptr_t>(counts) & 3u)) return AFD_ERR_INVALID_ARG;
  if (n_rows > (1 << 24)) return AFD_ERR_UNSUPPORTED;
  if (n_rows == 0) return AFD_OK;
  if ((st = check_w4_pointers(w)) != AFD_OK) return st;
  if (!x || !y || !aligned16(x) || !aligned16(y)) return AFD_ERR_INVALID_ARG;
  int* err = nullptr;
  if ((st = rows_err_word(&err)) != AFD_OK) return st;
  launch_w4<false>(*w, E, x, 1, counts, n_rows, y, y_dtype == AFD_DT_F32, err, static_cast<cudaStream_t>(stream));
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? AFD_OK : rows_cuda_fail(e);
}

extern "C" int64_t afd_ffn_w4_scratch_bytes(int32_t n_rows, int32_t I) {
  return n_rows < 0 || I < 0 ? 0 : 4LL * n_rows * I;
}

extern "C" int afd_ffn_w4_expert_rows(const afd_ffn_w4* w13, const afd_ffn_w4* w2, int32_t E, const void* rows,
                                      const int32_t* counts, int32_t n_rows, void* Y, int32_t y_dtype, void* scratch,
                                      void* stream) {
  int st = check_w4(w13, E);
  if (st != AFD_OK) return st;
  if ((st = check_w4(w2, E)) != AFD_OK) return st;
  if (n_rows < 0 || (y_dtype != AFD_DT_BF16 && y_dtype != AFD_DT_F32)) return AFD_ERR_INVALID_ARG;
  if (w13->N != 2 * w2->K || w13->K != w2->N) return AFD_ERR_INVALID_ARG;
  if ((!counts && E != 1) || (reinterpret_cast<uintptr_t>(counts) & 3u)) return AFD_ERR_INVALID_ARG;
  if (n_rows > (1 << 24)) return AFD_ERR_UNSUPPORTED;
  if (n_rows == 0) return AFD_OK;
  if ((st = check_w4_pointers(w13)) != AFD_OK || (st = check_w4_pointers(w2)) != AFD_OK) return st;
  if (!rows || !Y || !scratch || !aligned16(rows) || !aligned16(Y) || !aligned16(scratch)) return AFD_ERR_INVALID_ARG;
  int* err = nullptr;
  if ((st = rows_err_word(&err)) != AFD_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  launch_w4<true>(*w13, E, rows, 1, counts, n_rows, scratch, 0, err, s);
  launch_w4<false>(*w2, E, scratch, 2, counts, n_rows, Y, y_dtype == AFD_DT_F32, err, s);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? AFD_OK : rows_cuda_fail(e);
}
