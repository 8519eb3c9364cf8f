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
#include <atomic>

#include "afd_ffn.h"
#include "common.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace afd {
namespace {

constexpr int kW4MaxExperts = 256;
constexpr int kW4MaxRows = 1 << 22;
constexpr int kWarps = 8, kThreads = kWarps * 32;
constexpr int kSliceK = 128;       // inputs a warp takes in one step
constexpr int kUnitRows = 32;      // weight rows of a unit: two m16 tiles (gate and up rows for SwiGLU)
constexpr int kTileBytes = kUnitRows * kSliceK / 2;
constexpr int kTokens = 16;        // tokens of a unit: two n8 tiles
constexpr int kRedPitch = kUnitRows + 4;

struct W4Args {
  const uint8_t* codes;
  const void* scale;
  const uint8_t* zero;
  const __nv_bfloat16* x;   // [n_rows][K]; with planes = 2 a second plane of low parts follows
  const int32_t* counts;    // [E], or nullptr: one expert, every row
  void* y;
  int E, N, K, G, n_rows, scale_f32, y_f32, planes;
  int scale_words, zero_words;  // 4-byte words a row's scales / zero points of one step can touch
  int slot_bytes;           // one step of one warp in the ring
  unsigned long long group_inv;  // ceil(2^32 / (G / 32))
  int* err;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool full) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(full ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}

// D (16 x 8, fp32) += A (16 x 16, bf16) B (16 x 8, bf16)
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Codes i and i + 4 of a word as bf16 q - z: 0x4300 | q is 128 + q exactly, and so is the difference
// with 128 + z (zz: both halves).
__device__ __forceinline__ uint32_t unpack_pair(uint32_t shifted, uint32_t zz) {
  const uint32_t v = (shifted & 0x000f000fu) | 0x43004300u;
  const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&v), *reinterpret_cast<const __nv_bfloat162*>(&zz));
  return *reinterpret_cast<const uint32_t*>(&d);
}

struct UnitTables {
  int first[kW4MaxExperts], rows[kW4MaxExperts], unit_base[kW4MaxExperts + 1];
};

// Rows and unit bases of every expert from counts: negative counts are flagged and taken as 0,
// rows past n_rows are flagged and cut off.  Expert e has ceil(rows / kTokens) * blocks units.
__device__ __forceinline__ void build_tables(const W4Args& a, int blocks, UnitTables& tb, int* wsum) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int c = 0;
  bool bad = false;
  if (tid < a.E) {
    c = a.counts ? a.counts[tid] : a.n_rows;
    bad = c < 0 || c > a.n_rows;
    c = min(max(c, 0), a.n_rows);
  }
  int incl = warp_incl_scan(c, lane);
  if (lane == 31) wsum[warp] = incl;
  __syncthreads();
  int before = 0;
  for (int w = 0; w < warp; ++w) before += wsum[w];
  incl += before;
  bad |= incl > a.n_rows;
  const int first = min(incl - c, a.n_rows);
  const int rows = min(c, a.n_rows - first);
  if (bad && blockIdx.x == 0) atomicOr(a.err, kErrBadOffsets);
  const int units = (rows + kTokens - 1) / kTokens * blocks;
  int uincl = warp_incl_scan(units, lane);
  __syncthreads();
  if (lane == 31) wsum[warp] = uincl;
  __syncthreads();
  for (int w = 0; w < warp; ++w) uincl += wsum[w];
  tb.first[tid] = first;
  tb.rows[tid] = rows;
  tb.unit_base[tid + 1] = uincl;
  if (tid == 0) tb.unit_base[0] = 0;
  __syncthreads();
}

// One unit: an expert, 32 weight rows (SwiGLU: 16 gate rows and their 16 up rows) and up to 16 of
// its tokens, over the whole of K.
struct Unit {
  int e, first, m, row0;  // first token row, tokens, first output column
};

template <bool SWIGLU>
__device__ __forceinline__ Unit unit_at(int u, int* e, const UnitTables& tb) {
  while (u >= tb.unit_base[*e + 1]) ++*e;
  Unit r;
  r.e = *e;
  const int tiles = (tb.rows[r.e] + kTokens - 1) / kTokens;
  const int at = u - tb.unit_base[r.e];
  const int block = at / tiles, tile = at - block * tiles;
  r.first = tb.first[r.e] + tile * kTokens;
  r.m = min(kTokens, tb.rows[r.e] - tile * kTokens);
  r.row0 = block * (SWIGLU ? kUnitRows / 2 : kUnitRows);
  return r;
}

// Weight row (inside the expert) of unit row i; rows past the end repeat the last one.
template <bool SWIGLU>
__device__ __forceinline__ int weight_row(const W4Args& a, int row0, int i) {
  if (SWIGLU) {
    const int half = a.N / 2;
    return (i < 16 ? 0 : half) + min(row0 + (i & 15), half - 1);
  }
  return min(row0 + i, a.N - 1);
}

template <bool SWIGLU, bool WIDE, int STAGES>
__global__ void __launch_bounds__(kThreads, 2) w4_rows_kernel(const W4Args a) {
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ UnitTables tb;
  __shared__ int wsum[kWarps];
  __shared__ float red[kWarps][kTokens][kRedPitch];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int outs = SWIGLU ? a.N / 2 : a.N;
  constexpr int kOut = SWIGLU ? kUnitRows / 2 : kUnitRows;
  build_tables(a, (outs + kOut - 1) / kOut, tb, wsum);
  const int total = tb.unit_base[a.E];
  const int KG = a.K / a.G;
  const int rounds = (a.K + kWarps * kSliceK - 1) / (kWarps * kSliceK);
  const int active = min(kWarps, (a.K + kSliceK - 1) / kSliceK);  // warps with a slice of K

  const uint32_t my_ring = smem_u32(ring) + warp * STAGES * a.slot_bytes;
  const int cps = a.scale_f32 ? 4 : 2;

  // ---- loads: a step is 32 rows x 128 inputs of one round of one unit
  int lu = blockIdx.x, lr = 0, le = 0, lslot = 0;
  const uint8_t* wp[4];
  long long srow = 0;  // scale index of group 0 of this lane's row
  auto load_unit = [&]() {
    const Unit un = unit_at<SWIGLU>(lu, &le, tb);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = weight_row<SWIGLU>(a, un.row0, i * 8 + g);
      wp[i] = a.codes + (static_cast<size_t>(un.e) * a.N + r) * (a.K / 2) + t * 16;
    }
    srow = (static_cast<long long>(un.e) * a.N + weight_row<SWIGLU>(a, un.row0, lane)) * KG;
  };
  auto load_step = [&]() {
    if (lu < total) {
      if (lr == 0) load_unit();
      const int k = (lr * kWarps + warp) * kSliceK;
      if (k < a.K) {
        const uint32_t slot = my_ring + lslot * a.slot_bytes;
        const bool in = k + t * 32 < a.K;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = i * 8 + g;
          cp_async16(slot + r * 64 + ((t ^ ((r >> 1) & 3)) * 16), in ? wp[i] + k / 2 : a.codes, in);
        }
        const int kq = k / 32;
        const int g0 = static_cast<int>((kq * a.group_inv) >> 32);
        const long long at = srow + g0, end = static_cast<long long>(a.E) * a.N * KG;
        // the words that hold scales at .. at + 3 (as many as a step can need), cut at the tensor's end
        const long long sb = at * cps & ~3LL, send = end * cps;
        const uint32_t sdst = slot + kTileBytes + lane * a.scale_words * 4;
        for (int w = 0; w < a.scale_words; ++w) {
          const long long o = sb + w * 4;
          const int n = static_cast<int>(min(4LL, max(0LL, send - o)));
          cp_async4(sdst + w * 4, static_cast<const uint8_t*>(a.scale) + (n ? o : 0), n);
        }
        const long long zb = at & ~3LL;
        const uint32_t zdst = slot + kTileBytes + 32 * a.scale_words * 4 + lane * a.zero_words * 4;
        for (int w = 0; w < a.zero_words; ++w) {
          const long long o = zb + w * 4;
          const int n = static_cast<int>(min(4LL, max(0LL, end - o)));
          cp_async4(zdst + w * 4, a.zero + (n ? o : 0), n);
        }
      }
      if (++lr == rounds) {
        lr = 0;
        lu += gridDim.x;
      }
    }
    cp_async_commit();
    lslot = lslot + 1 == STAGES ? 0 : lslot + 1;
  };

#pragma unroll 1
  for (int i = 0; i < STAGES - 1; ++i) load_step();
  asm volatile("griddepcontrol.wait;" ::: "memory");

  int ce = 0, cslot = 0;
  for (int u = blockIdx.x; u < total; u += gridDim.x) {
    const Unit un = unit_at<SWIGLU>(u, &ce, tb);
    const bool two = un.m > 8;
    // parity / byte phase of each row's first scale in its words
    int phase[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      phase[i] = static_cast<int>(((static_cast<long long>(un.e) * a.N + weight_row<SWIGLU>(a, un.row0, i * 8 + g)) * KG) & 3);
    const __nv_bfloat16* xr[2];
    bool have[2];
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      have[n] = n * 8 + g < un.m;
      xr[n] = a.x + static_cast<size_t>(un.first + (have[n] ? n * 8 + g : 0)) * a.K;
    }
    float acc[2][2][4];
#pragma unroll
    for (int i = 0; i < 16; ++i) (&acc[0][0][0])[i] = 0.f;

    for (int r = 0; r < rounds; ++r) {
      cp_async_wait<STAGES - 2>();
      __syncwarp();
      load_step();
      const uint32_t slot = my_ring + cslot * a.slot_bytes;
      cslot = cslot + 1 == STAGES ? 0 : cslot + 1;
      const int k = (r * kWarps + warp) * kSliceK;
      if (k >= a.K) continue;
      const int steps = WIDE ? 4 : min(4, (a.K - k) / 32);
      const int kq = k / 32;
      const int g0 = static_cast<int>((kq * a.group_inv) >> 32);
      uint4 wide[4];
      if (WIDE) {
#pragma unroll
        for (int i = 0; i < 4; ++i) wide[i] = lds128(slot + (i * 8 + g) * 64 + ((t ^ (((i * 8 + g) >> 1) & 3)) * 16));
      }
      float part[2][2][4];
      uint32_t zz[4];
      float sc[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (!WIDE && j >= steps) break;
        if (j == 0 || !WIDE) {
          const int d = WIDE ? 0 : static_cast<int>(((kq + j) * a.group_inv) >> 32) - g0;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int row = i * 8 + g, ph = phase[i] + g0;
            const uint32_t sa = slot + kTileBytes + row * a.scale_words * 4;
            if (a.scale_f32) {
              sc[i] = __uint_as_float(lds32(sa + d * 4));
            } else {
              const int h = (ph & 1) + d;
              const uint32_t w = lds32(sa + (h >> 1) * 4);
              sc[i] = __uint_as_float((h & 1) ? (w & 0xffff0000u) : (w << 16));
            }
            uint32_t z = 8;
            if (a.zero_words) {
              const int b = (ph & 3) + d;
              z = lds32(slot + kTileBytes + 32 * a.scale_words * 4 + row * a.zero_words * 4 + (b >> 2) * 4) >> ((b & 3) * 8) & 15u;
            }
            zz[i] = (z << 16 | z) | 0x43004300u;
          }
#pragma unroll
          for (int i = 0; i < 16; ++i) (&part[0][0][0])[i] = 0.f;
        }
        uint32_t word[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          word[i] = WIDE ? (j == 0 ? wide[i].x : j == 1 ? wide[i].y : j == 2 ? wide[i].z : wide[i].w)
                         : lds32(slot + (i * 8 + g) * 64 + ((j ^ (((i * 8 + g) >> 1) & 3)) * 16) + t * 4);
        uint32_t A[2][2][4];  // [m tile][half of the word]
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            A[mt][h][0] = unpack_pair(word[2 * mt] >> (8 * h), zz[2 * mt]);
            A[mt][h][1] = unpack_pair(word[2 * mt + 1] >> (8 * h), zz[2 * mt + 1]);
            A[mt][h][2] = unpack_pair(word[2 * mt] >> (8 * h + 4), zz[2 * mt]);
            A[mt][h][3] = unpack_pair(word[2 * mt + 1] >> (8 * h + 4), zz[2 * mt + 1]);
          }
        const int kx = k + (WIDE ? t * 32 + j * 8 : j * 32 + t * 8);
        for (int p = 0; p < a.planes; ++p) {
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            if (n == 1 && !two) break;
            uint4 v = make_uint4(0u, 0u, 0u, 0u);
            if (have[n]) v = *reinterpret_cast<const uint4*>(xr[n] + static_cast<size_t>(p) * a.n_rows * a.K + kx);
            const uint32_t b0 = __byte_perm(v.x, v.z, 0x5410), b1 = __byte_perm(v.x, v.z, 0x7632);
            const uint32_t b2 = __byte_perm(v.y, v.w, 0x5410), b3 = __byte_perm(v.y, v.w, 0x7632);
#pragma unroll
            for (int mt = 0; mt < 2; ++mt) {
              mma_bf16(part[mt][n], A[mt][0], b0, b1);
              mma_bf16(part[mt][n], A[mt][1], b2, b3);
            }
          }
        }
        if (j == 3 || !WIDE) {
#pragma unroll
          for (int mt = 0; mt < 2; ++mt)
#pragma unroll
            for (int n = 0; n < 2; ++n) {
              acc[mt][n][0] = fmaf(sc[2 * mt], part[mt][n][0], acc[mt][n][0]);
              acc[mt][n][1] = fmaf(sc[2 * mt], part[mt][n][1], acc[mt][n][1]);
              acc[mt][n][2] = fmaf(sc[2 * mt + 1], part[mt][n][2], acc[mt][n][2]);
              acc[mt][n][3] = fmaf(sc[2 * mt + 1], part[mt][n][3], acc[mt][n][3]);
            }
        }
      }
    }

    // the warps' sums, joined in warp order
    if (warp < active) {
#pragma unroll
      for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          if (n == 1 && !two) break;
#pragma unroll
          for (int c = 0; c < 4; ++c) red[warp][n * 8 + t * 2 + (c & 1)][mt * 16 + (c >> 1) * 8 + g] = acc[mt][n][c];
        }
    }
    __syncthreads();
    for (int o = tid; o < un.m * kOut; o += kThreads) {
      const int tok = o / kOut, col = o % kOut;
      float v = 0.f, up = 0.f;
      for (int w = 0; w < active; ++w) {
        v += red[w][tok][col];
        if (SWIGLU) up += red[w][tok][16 + col];
      }
      if (un.row0 + col < outs) {
        const size_t at = static_cast<size_t>(un.first + tok) * outs + un.row0 + col;
        if (SWIGLU) {
          const float act = v / (1.f + expf(-v)) * up;
          const __nv_bfloat16 hi = __float2bfloat16_rn(act);
          static_cast<__nv_bfloat16*>(a.y)[at] = hi;
          static_cast<__nv_bfloat16*>(a.y)[static_cast<size_t>(a.n_rows) * outs + at] =
              __float2bfloat16_rn(act - __bfloat162float(hi));
        } else if (a.y_f32) {
          static_cast<float*>(a.y)[at] = v;
        } else {
          static_cast<__nv_bfloat16*>(a.y)[at] = __float2bfloat16_rn(v);
        }
      }
    }
    __syncthreads();  // red is free again
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

// Units are counted in 32 bits.
bool units_fit(int n_rows, int E, int outs, int unit_outs) {
  const long long units = (static_cast<long long>(n_rows) / kTokens + E) * ((outs + unit_outs - 1) / unit_outs);
  return units < (1LL << 31) - 65536;
}

int check_w4_pointers(const afd_ffn_w4* w) {
  // scales and zero points are fetched in 4-byte words
  const uintptr_t mis = (reinterpret_cast<uintptr_t>(w->scale) | reinterpret_cast<uintptr_t>(w->zero)) & 3u;
  if (!w->codes || !w->scale || !aligned16(w->codes) || mis) return AFD_ERR_INVALID_ARG;
  return AFD_OK;
}

constexpr int kStages = 4;
constexpr int kMaxSlotBytes = kTileBytes + 32 * 4 * (4 + 2);
constexpr int kMaxDevices = 64;

template <bool SWIGLU, bool WIDE>
cudaError_t launch_w4_kernel(const W4Args& a, bool after_gate_up, cudaStream_t s) {
  auto kernel = w4_rows_kernel<SWIGLU, WIDE, kStages>;
  // per device and kernel, once: the SM count, and leave for the largest ring
  static std::atomic<int> sm_count[kMaxDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  int sms = dev < kMaxDevices ? sm_count[dev].load(std::memory_order_relaxed) : 0;
  if (sms == 0) {
    e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kWarps * kStages * kMaxSlotBytes);
    if (e != cudaSuccess) return e;
    if (dev < kMaxDevices) sm_count[dev].store(sms, std::memory_order_relaxed);
  }
  const int smem = kWarps * kStages * a.slot_bytes;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(2 * sms);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = after_gate_up ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <bool SWIGLU>
cudaError_t launch_w4(const afd_ffn_w4& w, int E, const void* x, int planes, const int32_t* counts, int n_rows, void* y,
                      int y_f32, int* err, cudaStream_t s) {
  W4Args a{static_cast<const uint8_t*>(w.codes), w.scale, w.zero, static_cast<const __nv_bfloat16*>(x), counts, y,
           E, w.N, w.K, w.group, n_rows, w.scale_dtype == AFD_DT_F32, y_f32, planes, 0, 0, 0, 0, err};
  // groups that 128 inputs can reach, in 4-byte words that may start inside one
  const int reach = w.group % kSliceK == 0 ? 1 : w.group == 32 ? 4 : 2;
  a.scale_words = a.scale_f32 ? reach : reach / 2 + 1;
  a.zero_words = w.zero ? (reach == 1 ? 1 : 2) : 0;
  a.slot_bytes = kTileBytes + 32 * 4 * (a.scale_words + a.zero_words);
  const unsigned q = w.group / 32;
  a.group_inv = ((1ull << 32) + q - 1) / q;
  return w.group % kSliceK == 0 ? launch_w4_kernel<SWIGLU, true>(a, planes == 2, s)
                                : launch_w4_kernel<SWIGLU, false>(a, planes == 2, s);
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
  if (n_rows > kW4MaxRows || !units_fit(n_rows, E, w->N, kUnitRows)) return AFD_ERR_UNSUPPORTED;
  if (n_rows == 0) return AFD_OK;
  if ((st = check_w4_pointers(w)) != AFD_OK) return st;
  if (!x || !y || !aligned16(x) || !aligned16(y)) return AFD_ERR_INVALID_ARG;
  int* err = nullptr;
  if ((st = rows_err_word(&err)) != AFD_OK) return st;
  const cudaError_t e = launch_w4<false>(*w, E, x, 1, counts, n_rows, y, y_dtype == AFD_DT_F32, err,
                                         static_cast<cudaStream_t>(stream));
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
  if (n_rows > kW4MaxRows || !units_fit(n_rows, E, w2->K, kUnitRows / 2) || !units_fit(n_rows, E, w2->N, kUnitRows))
    return AFD_ERR_UNSUPPORTED;
  if (n_rows == 0) return AFD_OK;
  if ((st = check_w4_pointers(w13)) != AFD_OK || (st = check_w4_pointers(w2)) != AFD_OK) return st;
  if (!rows || !Y || !scratch || !aligned16(rows) || !aligned16(Y) || !aligned16(scratch)) return AFD_ERR_INVALID_ARG;
  int* err = nullptr;
  if ((st = rows_err_word(&err)) != AFD_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = launch_w4<true>(*w13, E, rows, 1, counts, n_rows, scratch, 0, err, s);
  if (e == cudaSuccess) e = launch_w4<false>(*w2, E, scratch, 2, counts, n_rows, Y, y_dtype == AFD_DT_F32, err, s);
  return e == cudaSuccess ? AFD_OK : rows_cuda_fail(e);
}
