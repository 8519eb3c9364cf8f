// norm.cu -- residual addition and root-mean-square norm in front of the FFN, with bf16 rows
// for the router and the layer, and e4m3 rows with one scale each for a W8A8 expert that takes every row.
//
//   s = x + residual (fp32)      sum = s in the residual's type
//   y = s * (mean(s^2) + eps)^(-1/2) * gamma (fp32, from s before its rounding)
//   out = bf16(y)      row_scale = max |y| / 448 (1 for a zero row, at least 2^-149)      codes = e4m3(y / row_scale)
//
// Bound by HBM: every byte is read and written once.  One CTA holds a row in registers between
// the loads and the stores; its one reduction carries both sum(s^2) and max |s gamma|, since
// max |y| is the latter times the row's factor.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "afd_ffn.h"
#include "common.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace afd {
namespace {

constexpr int kNormMaxH = 32768;

struct NormArgs {
  const void *x, *residual, *gamma;
  void *sum, *out;
  uint8_t* codes;
  float* row_scale;
  long long ldx, ldr, lds, ldo;
  int H;
  float eps;
};

// V elements from p (V = 8: 16-byte aligned)
template <int V>
__device__ __forceinline__ void load_row(const __nv_bfloat16* p, float (&f)[V]) {
  if constexpr (V == 8) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    const __nv_bfloat162* b = reinterpret_cast<const __nv_bfloat162*>(&u);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 g = __bfloat1622float2(b[i]);
      f[2 * i] = g.x;
      f[2 * i + 1] = g.y;
    }
  } else {
    f[0] = __bfloat162float(*p);
  }
}
template <int V>
__device__ __forceinline__ void load_row(const float* p, float (&f)[V]) {
  if constexpr (V == 8) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  } else {
    f[0] = *p;
  }
}
template <int V>
__device__ __forceinline__ void store_row(__nv_bfloat16* p, const float (&f)[V]) {
  if constexpr (V == 8) {
    uint4 u;
    __nv_bfloat162* b = reinterpret_cast<__nv_bfloat162*>(&u);
#pragma unroll
    for (int i = 0; i < 4; ++i) b[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    *reinterpret_cast<uint4*>(p) = u;
  } else {
    *p = __float2bfloat16_rn(f[0]);
  }
}
template <int V>
__device__ __forceinline__ void store_row(float* p, const float (&f)[V]) {
  if constexpr (V == 8) {
    reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
  } else {
    *p = f[0];
  }
}

// a / b rounded to nearest, from the correctly rounded reciprocal r of b: one Newton step on the
// quotient with an exact remainder (P. Markstein, "Computation of elementary functions on the IBM RISC
// System/6000 processor", 1990).  Holds while neither the quotient nor the remainder leaves the normal
// range, or the result is far below the last e4m3 code.
__device__ __forceinline__ float divide(float a, float b, float r) {
  const float q = a * r;
  return fmaf(fmaf(-q, b, a), r, q);
}

// Scale of a row's codes.  A quotient that rounds to zero would make the codes those of y / 0, and NaN at the
// row's zeros: the smallest fp32 number stands for it.
__device__ __forceinline__ float row_scale_of(float amax) {
  return amax > 0.f ? fmaxf(__fdiv_rn(amax, kE4m3Max), 0x1p-149f) : 1.0f;
}

// One CTA per row; thread i takes the pieces of V elements i, i + blockDim, ... (N at most) and keeps
// s gamma in registers; sum is written on the way.  The sum of squares goes through shuffles, the
// maximum through redux.sync on its bits; then every warp adds the warps' sums in the same order.
template <int V, int N, int MAXT, int MINB, typename RT, typename GT>
__global__ void __launch_bounds__(MAXT, MINB)
add_rmsnorm_kernel(const NormArgs a) {
  launch_dependents();
  wait_dependency();
  __shared__ float red_sum[32];
  __shared__ unsigned red_top[32];
  const long long t = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(a.x) + t * a.ldx;
  const RT* r = static_cast<const RT*>(a.residual) + t * a.ldr;
  const GT* g = static_cast<const GT*>(a.gamma);
  const int pieces = a.H / V;
  float s[N][V];
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const int p = tid + n * blockDim.x;
    if (p < pieces) load_row<V>(x + static_cast<size_t>(p) * V, s[n]);
  }
  if (a.residual) {
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int p = tid + n * blockDim.x;
      if (p < pieces) {
        float rv[V];
        load_row<V>(r + static_cast<size_t>(p) * V, rv);
#pragma unroll
        for (int i = 0; i < V; ++i) s[n][i] += rv[i];
      }
    }
  }
  float ss = 0.f, top = 0.f;
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const int p = tid + n * blockDim.x;
    if (p < pieces) {
      if (a.sum) store_row<V>(static_cast<RT*>(a.sum) + t * a.lds + static_cast<size_t>(p) * V, s[n]);
      float gv[V];
      load_row<V>(g + static_cast<size_t>(p) * V, gv);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        ss = fmaf(s[n][i], s[n][i], ss);
        s[n][i] *= gv[i];
        top = fmaxf(top, fabsf(s[n][i]));
      }
    }
  }
  ss = warp_sum(ss);
  const unsigned wtop = __reduce_max_sync(0xffffffffu, __float_as_uint(top));  // bits of numbers >= 0 are in their order
  if (lane == 0) {
    red_sum[warp] = ss;
    red_top[warp] = wtop;
  }
  __syncthreads();
  const int warps = blockDim.x >> 5;
  ss = warp_sum(lane < warps ? red_sum[lane] : 0.f);
  top = __uint_as_float(__reduce_max_sync(0xffffffffu, lane < warps ? red_top[lane] : 0u));
  const float factor = __frsqrt_rn(ss / static_cast<float>(a.H) + a.eps);
  const float amax = top * factor;
  const float scale = row_scale_of(amax);
  const float inv = __frcp_rn(scale);
  const bool plain = scale > 1e-30f && scale < 1e30f;  // where divide() holds
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const int p = tid + n * blockDim.x;
    if (p < pieces) {
      float y[V];
#pragma unroll
      for (int i = 0; i < V; ++i) y[i] = s[n][i] * factor;
      if (a.out) store_row<V>(static_cast<__nv_bfloat16*>(a.out) + t * a.ldo + static_cast<size_t>(p) * V, y);
      if (a.codes) {
#pragma unroll
        for (int i = 0; i < V; ++i) y[i] = plain ? divide(y[i], scale, inv) : __fdiv_rn(y[i], scale);
        uint8_t* c = a.codes + t * a.H + static_cast<size_t>(p) * V;
        if constexpr (V == 8) {
          uint32_t q[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float* v = y + 4 * i;
            const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[0], v[1]), __NV_SATFINITE, __NV_E4M3);
            const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v[2], v[3]), __NV_SATFINITE, __NV_E4M3);
            q[i] = lo | (hi << 16);
          }
          *reinterpret_cast<uint2*>(c) = make_uint2(q[0], q[1]);
        } else {
          *c = __nv_cvt_float_to_fp8(y[0], __NV_SATFINITE, __NV_E4M3);
        }
      }
    }
  }
  if (a.codes && tid == 0) a.row_scale[t] = scale;
}

// Eight elements from p, which has its type's alignment only: the aligned 16-byte pieces that hold them,
// shifted together.  Only where those lie inside [begin, end), the row; else element by element, where
// element i counts if first <= i < last.
__device__ __forceinline__ void shift_words(uint32_t* w, int n, int by) {  // by 0..3 words; n words stay valid
#pragma unroll
  for (int i = 0; i < 10; ++i)
    if (i < n + 2) w[i] = by & 1 ? w[i + 1] : w[i];
#pragma unroll
  for (int i = 0; i < 9; ++i)
    if (i < n) w[i] = by & 2 ? w[i + 2] : w[i];
}
template <typename T>
__device__ __forceinline__ void load_shifted(const T* p, const T* begin, const T* end, int first, int last, float (&f)[8]) {
  constexpr int kPieces = sizeof(T) == 2 ? 2 : 3;  // that eight elements can touch
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), from = a & ~static_cast<uintptr_t>(15);
  const int off = static_cast<int>(a & 15);
  if (from >= reinterpret_cast<uintptr_t>(begin) &&
      from + 16 * (off ? kPieces : kPieces - 1) <= reinterpret_cast<uintptr_t>(end)) {
    uint32_t w[13];
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      if (i == kPieces - 1 && !off) break;
      const uint4 v = reinterpret_cast<const uint4*>(from)[i];
      w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
    }
    if constexpr (sizeof(T) == 2) {
      shift_words(w, 5, off >> 2);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t v = __funnelshift_r(w[i], w[i + 1], (off & 2) * 8);
        f[2 * i] = __uint_as_float(v << 16);
        f[2 * i + 1] = __uint_as_float(v & 0xffff0000u);
      }
    } else {
      shift_words(w, 8, off >> 2);
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(w[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = i >= first && i < last ? static_cast<float>(p[i]) : 0.f;
  }
}

// Rows that do not start on 16-byte boundaries, written to contiguous tensors: thread i takes the aligned
// pieces of eight of the outputs, i, i + blockDim, ..., which are aligned pieces of each of them (the flat
// index is a multiple of eight), and reads its inputs shifted.  A row's first and last piece can reach
// into its neighbours: those elements are left out.
template <int N, int MAXT, int MINB, typename RT, typename GT>
__global__ void __launch_bounds__(MAXT, MINB)
add_rmsnorm_shifted_kernel(const NormArgs a) {
  launch_dependents();
  wait_dependency();
  __shared__ float red_sum[32];
  __shared__ unsigned red_top[32];
  const long long t = blockIdx.x, flat = t * a.H;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(a.x) + t * a.ldx;
  const RT* r = static_cast<const RT*>(a.residual) + t * a.ldr;
  const GT* g = static_cast<const GT*>(a.gamma);
  const int lead = static_cast<int>(flat & 7), pieces = (lead + a.H + 7) >> 3;
  float s[N][8];
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const int p = tid + n * blockDim.x;
    if (p < pieces) {
      const int e = p * 8 - lead, first = max(0, -e), last = min(8, a.H - e);
      load_shifted(x + e, x, x + a.H, first, last, s[n]);
      if (a.residual) {
        float rv[8];
        load_shifted(r + e, r, r + a.H, first, last, rv);
#pragma unroll
        for (int i = 0; i < 8; ++i) s[n][i] += rv[i];
      }
    }
  }
  if (a.sum) __syncthreads();  // sum may be the residual's buffer, whose pieces are read by neighbours too
  // piece p of a row's outputs to v's buffer
  auto store = [&](auto* to, int p, const float (&v)[8]) {
    const int e = p * 8 - lead;
    if (e >= 0 && e + 8 <= a.H) {
      store_row<8>(to + flat + e, v);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (e + i >= 0 && e + i < a.H) {
          const float one[1] = {v[i]};
          store_row<1>(to + flat + e + i, one);
        }
    }
  };
  float ss = 0.f, top = 0.f;
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const int p = tid + n * blockDim.x;
    if (p < pieces) {
      const int e = p * 8 - lead;
      if (a.sum) store(static_cast<RT*>(a.sum), p, s[n]);
      float gv[8];
      load_shifted(g + e, g, g + a.H, max(0, -e), min(8, a.H - e), gv);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        ss = fmaf(s[n][i], s[n][i], ss);
        s[n][i] *= gv[i];
        top = fmaxf(top, fabsf(s[n][i]));
      }
    }
  }
  ss = warp_sum(ss);
  const unsigned wtop = __reduce_max_sync(0xffffffffu, __float_as_uint(top));
  if (lane == 0) {
    red_sum[warp] = ss;
    red_top[warp] = wtop;
  }
  __syncthreads();
  const int warps = blockDim.x >> 5;
  ss = warp_sum(lane < warps ? red_sum[lane] : 0.f);
  top = __uint_as_float(__reduce_max_sync(0xffffffffu, lane < warps ? red_top[lane] : 0u));
  const float factor = __frsqrt_rn(ss / static_cast<float>(a.H) + a.eps);
  const float amax = top * factor;
  const float scale = row_scale_of(amax);
  const float inv = __frcp_rn(scale);
  const bool plain = scale > 1e-30f && scale < 1e30f;
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const int p = tid + n * blockDim.x;
    if (p < pieces) {
      float y[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = s[n][i] * factor;
      if (a.out) store(static_cast<__nv_bfloat16*>(a.out), p, y);
      if (a.codes) {
        uint32_t q[2] = {0u, 0u};
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          const float v0 = plain ? divide(y[i], scale, inv) : __fdiv_rn(y[i], scale);
          const float v1 = plain ? divide(y[i + 1], scale, inv) : __fdiv_rn(y[i + 1], scale);
          q[i >> 2] |= static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(make_float2(v0, v1), __NV_SATFINITE, __NV_E4M3)) << (i & 2) * 8;
        }
        const int e = p * 8 - lead;
        uint8_t* c = a.codes + flat + e;
        if (e >= 0 && e + 8 <= a.H) {
          *reinterpret_cast<uint2*>(c) = make_uint2(q[0], q[1]);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (e + i >= 0 && e + i < a.H) c[i] = static_cast<uint8_t>(q[i >> 2] >> (i & 3) * 8);
        }
      }
    }
  }
  if (a.codes && tid == 0) a.row_scale[t] = scale;
}

template <int V, int N, int MAXT, int MINB, typename RT, typename GT>
void launch_norm_kernel(const NormArgs& a, int T, cudaStream_t s) {
  const int threads = (a.H / V + N * 32 - 1) / (N * 32) * 32;
  launch_dependent(add_rmsnorm_kernel<V, N, MAXT, MINB, RT, GT>, T, threads, 0, s, a);
}

// Pieces per thread and CTAs per SM.  Few rows: one piece, the shortest way through a row.  Rows that
// fill the SMs many times: two, so that a row's reduction is paid by fewer warps, in few enough
// registers that four rows are in flight on an SM.  8192 rows of 7168 (bf16 residual, both outputs):
// 98 us so (82 % of the copy rate); 1 piece 118 to 122 us, 4 pieces 112 to 139 us, 2 pieces in more
// registers 110 us.  Single elements, which rows of any start take where an output has gaps between its
// rows: 515 rows of 4097 at 6 a thread 9.1 us, 5 10.7, 8 10.1, 16 13.9 us.
constexpr int kManyRows = 256;

template <int V, typename RT, typename GT>
void launch_norm(const NormArgs& a, int T, cudaStream_t s) {
  const int pieces = a.H / V;
  const bool many = T >= kManyRows;
  if constexpr (V == 8) {
    if (pieces <= (many ? 128 : 1024)) launch_norm_kernel<V, 1, 1024, 1, RT, GT>(a, T, s);
    else if (many && pieces <= 1024) launch_norm_kernel<V, 2, 512, 4, RT, GT>(a, T, s);
    else launch_norm_kernel<V, 4, 1024, 1, RT, GT>(a, T, s);
  } else {
    if (pieces <= (many ? 256 : 1024)) launch_norm_kernel<V, 1, 1024, 1, RT, GT>(a, T, s);
    else if (many && pieces <= 4224) launch_norm_kernel<V, 6, 704, 2, RT, GT>(a, T, s);
    else if (many && pieces <= 8192) launch_norm_kernel<V, 8, 1024, 2, RT, GT>(a, T, s);
    else if (pieces <= 8192) launch_norm_kernel<V, 8, 1024, 1, RT, GT>(a, T, s);
    else launch_norm_kernel<V, 32, 1024, 1, RT, GT>(a, T, s);
  }
}

// Shifted pieces against single elements: 4000 rows of 7001 (fp32 residual, both outputs) 88 us and 150 us,
// 515 rows of 4097 8.7 and 10.4, 3000 rows of 2345 22 and 29; 8000 rows of 301 13.5 and 10.8.  Four rows on
// an SM rather than two: 88 against 107 us.
constexpr int kShiftedMinH = 512;

template <typename RT, typename GT>
void launch_shifted(const NormArgs& a, int T, cudaStream_t s) {
  const int pieces = (a.H + 14) / 8;  // at most
  // At most 32 elements a thread, as in the other forms, so that a row's sum of squares is as exact: a thread has a
  // fifth piece only in rows of more than 4096 pieces, whose first and last are parts.  Five whole ones took 210 us
  // for 2000 rows of 24001, four take 198; 4000 rows of 9001 126 and 130.
  const int per = pieces <= 256 ? 1 : pieces <= 1024 ? 2 : 4, threads = std::min(1024, (pieces + per * 32 - 1) / (per * 32) * 32);
  if (per == 1) launch_dependent(add_rmsnorm_shifted_kernel<1, 256, 4, RT, GT>, T, threads, 0, s, a);
  else if (per == 2) launch_dependent(add_rmsnorm_shifted_kernel<2, 512, 4, RT, GT>, T, threads, 0, s, a);
  else launch_dependent(add_rmsnorm_shifted_kernel<5, 1024, 1, RT, GT>, T, threads, 0, s, a);
}

// How rows move: 16-byte pieces, shifted pieces, single elements.
enum NormForm { kPieces, kShifted, kElements };

template <typename RT, typename GT>
void launch_norm_form(const NormArgs& a, int T, NormForm form, cudaStream_t s) {
  if (form == kPieces) launch_norm<8, RT, GT>(a, T, s);
  else if (form == kShifted) launch_shifted<RT, GT>(a, T, s);
  else launch_norm<1, RT, GT>(a, T, s);
}

void launch_norm_types(const NormArgs& a, const afd_ffn_norm_cfg& c, NormForm form, cudaStream_t s) {
  const bool rf = c.residual_dtype == AFD_DT_F32, gf = c.gamma_dtype == AFD_DT_F32;
  if (rf && gf) launch_norm_form<float, float>(a, c.T, form, s);
  else if (rf) launch_norm_form<float, __nv_bfloat16>(a, c.T, form, s);
  else if (gf) launch_norm_form<__nv_bfloat16, float>(a, c.T, form, s);
  else launch_norm_form<__nv_bfloat16, __nv_bfloat16>(a, c.T, form, s);
}

bool elem_dtype(int32_t d) { return d == AFD_DT_BF16 || d == AFD_DT_F32; }
bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

}  // namespace
}  // namespace afd

using namespace afd;

extern "C" int afd_ffn_add_rmsnorm(const afd_ffn_norm_cfg* cfg, const void* x, const void* residual,
                                   const void* gamma, void* sum, void* out, void* codes, float* row_scale,
                                   void* stream) {
  if (!cfg) return AFD_ERR_INVALID_ARG;
  const afd_ffn_norm_cfg& c = *cfg;
  if (c.T < 0 || c.H < 1 || !elem_dtype(c.residual_dtype) || !elem_dtype(c.gamma_dtype)) return AFD_ERR_INVALID_ARG;
  if (!(c.eps >= 0.f) || !(c.eps <= 3.4e38f)) return AFD_ERR_INVALID_ARG;
  if (c.H > kNormMaxH) return AFD_ERR_UNSUPPORTED;
  NormArgs a{x, residual, gamma, sum, out, static_cast<uint8_t*>(codes), row_scale, c.x_stride, c.residual_stride,
             c.sum_stride, c.out_stride, c.H, c.eps};
  for (long long* ld : {&a.ldx, &a.ldr, &a.lds, &a.ldo}) {
    if (*ld == 0) *ld = c.H;
    if (*ld < c.H) return AFD_ERR_INVALID_ARG;
  }
  if (c.T == 0) return AFD_OK;
  if (!x || !gamma || (sum && !residual) || (!out && !codes) || (!codes != !row_scale)) return AFD_ERR_INVALID_ARG;
  const uintptr_t rsize = c.residual_dtype == AFD_DT_F32 ? 4 : 2, gsize = c.gamma_dtype == AFD_DT_F32 ? 4 : 2;
  if (!aligned(x, 2) || !aligned(residual, rsize) || !aligned(sum, rsize) || !aligned(gamma, gsize) ||
      !aligned(out, 2) || !aligned(row_scale, 4))
    return AFD_ERR_INVALID_ARG;
  // 16-byte pieces where every row of every tensor starts on a 16-byte boundary
  const uintptr_t rper = 16 / rsize;
  const bool wide = c.H % 8 == 0 && aligned(x, 16) && a.ldx % 8 == 0 && aligned(gamma, 16) &&
                    (!residual || (aligned(residual, 16) && a.ldr % rper == 0)) &&
                    (!sum || (aligned(sum, 16) && a.lds % rper == 0)) &&
                    (!out || (aligned(out, 16) && a.ldo % 8 == 0)) && (!codes || aligned(codes, 8));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  // Outputs without gaps between their rows, from a 16-byte boundary on.
  const bool flat = (!sum || (a.lds == c.H && aligned(sum, 16))) && (!out || (a.ldo == c.H && aligned(out, 16))) &&
                    (!codes || aligned(codes, 8));
  launch_norm_types(a, c, wide ? kPieces : flat && c.H >= kShiftedMinH ? kShifted : kElements, s);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? AFD_OK : rows_cuda_fail(e);
}
