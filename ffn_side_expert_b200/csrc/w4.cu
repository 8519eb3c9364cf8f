// w4.cu -- rows grouped by expert times 4-bit weights with group scales, and the whole expert
// (gate/up, SwiGLU, down) on such weights, for the few rows an expert gets in a decode
// micro-batch.
//
//   W[n][k] = (q[n][k] - z[n][k / G]) * scale[n][k / G],  q, z in 0..15 (z = 8 without zero points)
//   y[r][n] = sum_k x[r][k] W[n][k]                         per expert, fp32 sums
//   act = silu(x Wg^T) * (x Wu^T),  Y = act W2^T
//
// The products are bf16 with fp32 sums: (q - z) / 4 is exact in bf16, the sum over a group's inputs
// is scaled in fp32, the factor 4 comes back at the end.  The SwiGLU rows are kept as two bf16
// terms (hi + lo, 2^-17 relative), which are two columns of the down product.
//
// What bounds it.  At the HBM rate an SM gets 46 codes a clock, and its integer pipe does 64 lane
// operations; so the unpacking decides.  A word of eight codes takes nine instructions, five of
// them integer: one shift, four masks and four bf16x2 FMAs that take the zero point off
// (unpack_word).  Weights come through a cp.async ring per warp, straight from HBM; the inputs,
// few, from L1 and L2.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

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
constexpr int kBlockRows = 16;     // weight rows of a block (SwiGLU: 8 gate rows and their 8 up rows); a unit is one or two
constexpr int kTileBytes = 2 * kBlockRows * kSliceK / 2;
constexpr int kCols = 8;           // columns of a unit: 8 tokens, or 4 of two planes
constexpr int kRedPitch = 2 * kBlockRows + 4;
constexpr int kStages = 4;

struct W4Args {
  const uint8_t* codes;
  const void* scale;
  const uint8_t* zero;
  const __nv_bfloat16* x;   // [n_rows * planes][K]
  const int32_t* counts;    // [E], or nullptr: one expert, every row
  void* y;
  int E, N, K, G, n_rows, scale_f32, y_f32;
  unsigned group_inv;       // ceil(2^32 / (G / 32)), 0 for groups of 32
  int windows;              // rows of scales (and zero points) that whole 16-byte pieces cover
  int* err;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool full) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(full ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async8(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
// This kernel's dependents may start; wait for the kernel this one depends on (nothing outside a
// programmatic launch).
__device__ __forceinline__ void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_dependency() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// D (16 x 8, fp32) = A (16 x 16, bf16) B (16 x 8, bf16) + C
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1, const float (&c)[4]) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %11, %12, %13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}

__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}

// (q - z) / 4 of a word's eight codes as bf16 pairs: codes i and i + 4 in p[i], or in their own order
// (OWN_ORDER) codes 2 i and 2 i + 1.  A code in the low four bits of a half, under the exponent of
// 128, reads 128 + q.  One four bits up reads q 2^-129 as it stands: subnormal up to 7, and the first
// normal numbers go on in the same steps.  Both are exact, and so are the FMAs.  c0 = -(128 + z) / 4
// and c1 = -z / 4, in both halves.  Nine instructions, or twelve.
template <bool OWN_ORDER = false>
__device__ __forceinline__ void unpack_word(uint32_t w, uint32_t c0, uint32_t c1, uint32_t (&p)[4]) {
  constexpr uint32_t kQuarter = 0x3E803E80u, k2to127 = 0x7F007F00u;
  if (OWN_ORDER) {  // a byte in both halves: its low code from the low half, its high code from the high one
    const uint32_t c = __byte_perm(c0, c1, 0x5410);
    p[0] = fma_bf16x2((__byte_perm(w, 0, 0x4040) & 0x00f0000fu) | 0x00004300u, 0x7F003E80u, c);
    p[1] = fma_bf16x2((__byte_perm(w, 0, 0x4141) & 0x00f0000fu) | 0x00004300u, 0x7F003E80u, c);
    p[2] = fma_bf16x2((__byte_perm(w, 0, 0x4242) & 0x00f0000fu) | 0x00004300u, 0x7F003E80u, c);
    p[3] = fma_bf16x2((__byte_perm(w, 0, 0x4343) & 0x00f0000fu) | 0x00004300u, 0x7F003E80u, c);
  } else {
    const uint32_t s = w >> 8;
    p[0] = fma_bf16x2((w & 0x000f000fu) | 0x43004300u, kQuarter, c0);
    p[1] = fma_bf16x2(w & 0x00f000f0u, k2to127, c1);
    p[2] = fma_bf16x2((s & 0x000f000fu) | 0x43004300u, kQuarter, c0);
    p[3] = fma_bf16x2(s & 0x00f000f0u, k2to127, c1);
  }
}

// ---------------------------------------------------------------------- the product
struct UnitTables {
  int first[kW4MaxExperts], rows[kW4MaxExperts], unit_base[kW4MaxExperts + 1];
};

// Rows and unit bases of every expert from counts: negative counts are flagged and taken as 0,
// rows past n_rows are flagged and cut off.  units_of(rows): an expert's units.
template <typename F>
__device__ __forceinline__ void build_tables(const W4Args& a, F units_of, UnitTables& tb, int* wsum) {
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
  const int units = tid < a.E ? units_of(rows) : 0;
  int uincl = warp_incl_scan(units, lane);
  __syncthreads();
  if (lane == 31) wsum[warp] = uincl;
  __syncthreads();
  for (int w = 0; w < warp; ++w) uincl += wsum[w];
  if (tid < kW4MaxExperts) {
    tb.first[tid] = first;
    tb.rows[tid] = rows;
    tb.unit_base[tid + 1] = uincl;
  }
  if (tid == 0) tb.unit_base[0] = 0;
  __syncthreads();
}

// One unit: an expert with its m tokens from row `first`, and mt blocks of its weight rows from
// output row0 on, over the whole of K.
struct Unit {
  int e, first, m, row0, mt;
};

// The unit at block b of a team's blocks, which end at `end`.
template <bool SWIGLU>
__device__ __forceinline__ Unit unit_at(int b, int end, int* e, const UnitTables& tb) {
  while (b >= tb.unit_base[*e + 1]) ++*e;
  Unit r;
  r.e = *e;
  r.first = tb.first[r.e];
  r.m = tb.rows[r.e];
  r.row0 = (b - tb.unit_base[r.e]) * (SWIGLU ? kBlockRows / 2 : kBlockRows);
  r.mt = b + 1 < min(end, tb.unit_base[r.e + 1]) ? 2 : 1;
  return r;
}

// Weight row (inside the expert) of row i * 8 + g of a unit; rows past the end repeat the last one.
template <bool SWIGLU>
__device__ __forceinline__ int weight_row(const W4Args& a, int row0, int i, int g) {
  if (SWIGLU) {
    const int half = a.N / 2;
    return ((i & 1) ? half : 0) + min(row0 + (i >> 1) * 8 + g, half - 1);
  }
  return min(row0 + i * 8 + g, a.N - 1);
}

// Group of the 32 inputs kq: kq / (G / 32).
__device__ __forceinline__ int group_of(const W4Args& a, int kq) {
  return a.group_inv ? static_cast<int>(__umulhi(static_cast<unsigned>(kq), a.group_inv)) : kq;
}

// What a product is for.  kGateUp: gate and up rows, the SwiGLU rows out as two bf16 terms; kDown: from
// those to the results; kRows: one product on its own.
enum W4Mode { kRows, kGateUp, kDown };

// Place of input i of eight in the SwiGLU rows: the order in which unpack_word pairs the codes.
__device__ __forceinline__ int paired_place(int i) { return (i & ~7) | ((i & 3) << 1) | (i >> 2 & 1); }

// One result: of kGateUp, from a gate and an up value, the SwiGLU value as two bf16 terms.
template <int MODE>
__device__ __forceinline__ void store_out(const W4Args& a, int row, int out, int outs, float v, float up) {
  if (MODE == kGateUp) {
    const float act = v / (1.f + expf(-v)) * up;
    const __nv_bfloat16 hi = __float2bfloat16_rn(act);
    // an infinite or NaN value is its own high term alone
    const __nv_bfloat16 lo = __float2bfloat16_rn(fabsf(act) < INFINITY ? act - __bfloat162float(hi) : 0.f);
    __nv_bfloat16* y = static_cast<__nv_bfloat16*>(a.y) + static_cast<size_t>(row) * 2 * outs + paired_place(out);
    y[0] = hi;
    y[outs] = lo;
  } else {
    const size_t at = static_cast<size_t>(row) * outs + out;
    if (a.y_f32)
      static_cast<float*>(a.y)[at] = v;
    else
      static_cast<__nv_bfloat16*>(a.y)[at] = __float2bfloat16_rn(v);
  }
}

}  // namespace
}  // namespace afd

#include "w4_wide.cuh"

namespace afd {
namespace {

// Warps that share a unit.  A team's cost: its units, two blocks at 10 or one at 6, times the steps
// of a warp and about 0.8 of a step for the join.  The smallest wins, the wider split on a tie.
__device__ __forceinline__ int choose_split(int blocks, int slices, int ctas) {
  int best = 8, least = 0x7fffffff;
  for (int split = 8; split >= 1; split >>= 1) {
    const int teams = ctas * (kWarps / split);
    const int n = (blocks + teams - 1) / teams;
    const long long cost = static_cast<long long>((n >> 1) * 10 + (n & 1) * 6) * ((slices + split - 1) / split * 10 + 8);
    if (cost < least) {
      least = static_cast<int>(cost);
      best = split;
    }
  }
  return best;
}

// The experts with few rows: at most kCols columns.
// PARTS: groups of a slice with a scale each (1, 2 or 4).
template <int MODE, int PARTS, bool ZERO>
__global__ void __launch_bounds__(kThreads, 2) w4_rows_kernel(const W4Args a) {
  constexpr bool SWIGLU = MODE == kGateUp, WIDE = PARTS == 1;
  constexpr int kPlanes = MODE == kDown ? 2 : 1;
  constexpr int kOut = SWIGLU ? kBlockRows / 2 : kBlockRows;  // outputs of a block
  extern __shared__ __align__(16) uint8_t ring[];             // [kWarps][kStages][kTileBytes]
  __shared__ float red[2][kWarps][kCols][kRedPitch];
  __shared__ UnitTables tb;
  __shared__ int wsum[kWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3;
  launch_dependents();
  const int outs = SWIGLU ? a.N / 2 : a.N;
  const int per_expert = (outs + kOut - 1) / kOut;
  build_tables(a, [&](int rows) { return rows > 0 && rows * kPlanes <= kCols ? per_expert : 0; }, tb, wsum);
  const int total = tb.unit_base[a.E];
  const int KG = a.K / a.G;
  // split warps share a unit, each with every split-th slice of K; a team takes consecutive blocks
  const int slices = (a.K + kSliceK - 1) / kSliceK;
  const int split = choose_split(total, slices, gridDim.x);
  const int sub = warp & (split - 1), team = warp / split;
  const int active = min(split, slices);                     // warps of a team with a slice
  const int steps = (slices - sub + split - 1) / split;      // this warp's slices of a unit
  const int teams = gridDim.x * (kWarps / split), me = blockIdx.x * (kWarps / split) + team;
  const int b0 = static_cast<int>(static_cast<long long>(total) * me / teams);
  const int b1 = static_cast<int>(static_cast<long long>(total) * (me + 1) / teams);
  const int cps = a.scale_f32 ? 4 : 2;

  // ---- loads: a step is the unit's rows x 128 inputs
  // Row r's 16 bytes c are kept at place c ^ (r / 2 % 4), so that neither side's accesses conflict.
  const int swizzle = (g >> 1) & 3;
  uint8_t* const my_ring = ring + warp * kStages * kTileBytes + g * 64;
  const uint32_t put = smem_u32(my_ring) + (t ^ swizzle) * 16;
  int lb = steps > 0 ? b0 : b1, ls = 0, le = 0, lmt = 0, lslot = 0;
  const uint8_t* wp[4];
  auto load_step = [&]() {
    if (lb < b1) {
      if (ls == 0) {
        const Unit un = unit_at<SWIGLU>(lb, b1, &le, tb);
        lmt = un.mt;
        const size_t row = static_cast<size_t>(un.e) * a.N;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          wp[i] = a.codes + (row + weight_row<SWIGLU>(a, un.row0, i, g)) * (a.K / 2) + sub * 64 + t * 16;
        // the scales and zero points of row `lane`, which the products read: in L2 by then
        const size_t at = (row + weight_row<SWIGLU>(a, un.row0, lane >> 3, lane & 7)) * KG;
        const uint8_t* sp = static_cast<const uint8_t*>(a.scale) + at * cps;
        if (lane < un.mt * kBlockRows) {
          for (int o = sub * 32; o < KG * cps; o += split * 32) prefetch_l2(sp + o);
          if (ZERO)
            for (int o = sub * 32; o < KG; o += split * 32) prefetch_l2(a.zero + at + o);
        }
      }
      const uint32_t dst = put + lslot;
      const bool in = WIDE || (ls * split + sub) * kSliceK + t * 32 < a.K;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (i == 2 && lmt == 1) break;
        if (WIDE)
          cp_async16(dst + i * 512, wp[i]);
        else
          cp_async16(dst + i * 512, in ? wp[i] : a.codes, in);
        wp[i] += split * 64;
      }
      if (++ls == steps) {
        ls = 0;
        lb += lmt;
      }
    }
    cp_async_commit();
    lslot = lslot == (kStages - 1) * kTileBytes ? 0 : lslot + kTileBytes;
  };

#pragma unroll 1
  for (int i = 0; i < kStages - 1; ++i) load_step();
  if (MODE == kDown) wait_dependency();

  int ce = 0, cslot = 0, buf = 0;
  for (int b = b0; b < b1; buf ^= 1) {
    const Unit un = unit_at<SWIGLU>(b, b1, &ce, tb);
    b += un.mt;
    const int cols = un.m * kPlanes;
    auto products = [&](auto blocks) {
      constexpr int MT = decltype(blocks)::value;
      // columns past the last one repeat it; their results are not used
      const __nv_bfloat16* col = a.x + (static_cast<size_t>(un.first) * kPlanes + min(g, cols - 1)) * a.K + sub * kSliceK + t * (WIDE ? 32 : 8);
      // scales of rows i * 8 + g
      const uint8_t* sp[2 * MT];
      const uint8_t* zp[ZERO ? 2 * MT : 1];
#pragma unroll
      for (int i = 0; i < 2 * MT; ++i) {
        const size_t at = (static_cast<size_t>(un.e) * a.N + weight_row<SWIGLU>(a, un.row0, i, g)) * KG;
        sp[i] = static_cast<const uint8_t*>(a.scale) + at * cps;
        if (ZERO) zp[i] = a.zero + at;
      }
      float acc[MT][4];
#pragma unroll
      for (int i = 0; i < MT * 4; ++i) (&acc[0][0])[i] = 0.f;

#pragma unroll 1
      for (int s = 0, k = sub * kSliceK; s < steps; ++s, k += split * kSliceK) {
        const uint8_t* slot = my_ring + cslot;
        cslot = cslot == (kStages - 1) * kTileBytes ? 0 : cslot + kTileBytes;
        const int parts = WIDE ? 4 : min(4, (a.K - k) / 32);
        uint4 x[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (WIDE || j < parts) x[j] = *reinterpret_cast<const uint4*>(col + j * (WIDE ? 8 : 32));
        col += split * kSliceK;
        float sc[2 * MT];
        uint32_t z[2 * MT];
        auto load_scales = [&](int j) {
          const int d = group_of(a, k / 32 + j);
          if (a.scale_f32) {
#pragma unroll
            for (int i = 0; i < 2 * MT; ++i) sc[i] = __ldg(reinterpret_cast<const float*>(sp[i]) + d);
          } else {
#pragma unroll
            for (int i = 0; i < 2 * MT; ++i)
              sc[i] = __uint_as_float(static_cast<uint32_t>(__ldg(reinterpret_cast<const unsigned short*>(sp[i]) + d)) << 16);
          }
          if (ZERO) {
#pragma unroll
            for (int i = 0; i < 2 * MT; ++i) z[i] = __ldg(zp[i] + d);
          }
        };
        load_scales(0);
        cp_async_wait<kStages - 2>();
        __syncwarp();
        load_step();
        uint4 wide[2 * MT];
        if (WIDE) {
#pragma unroll
          for (int i = 0; i < 2 * MT; ++i) wide[i] = *reinterpret_cast<const uint4*>(slot + i * 512 + (t ^ swizzle) * 16);
        }
        float part[MT][4], f[2 * MT];
        const float none[4] = {0.f, 0.f, 0.f, 0.f};
        uint32_t c0[2 * MT], c1[2 * MT];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (!WIDE && j >= parts) break;
          constexpr int kSpan = 4 / PARTS;  // words of a part
          const bool starts = j % kSpan == 0, ends = j % kSpan == kSpan - 1;
          if (starts) {
#pragma unroll
            for (int i = 0; i < 2 * MT; ++i) {
              c0[i] = 0xC208C208u;  // -(128 + 8) / 4
              c1[i] = 0xC000C000u;  // -8 / 4
              if (ZERO) {
                const uint32_t q = ((z[i] & 15u) | 0x4300u) * 0x10001u;  // 128 + z
                c0[i] = fma_bf16x2(q, 0xBE80BE80u, 0x80008000u);
                c1[i] = fma_bf16x2(q, 0xBE80BE80u, 0x42004200u);
              }
              f[i] = sc[i];
            }
            if (j + kSpan < 4 && j + kSpan < parts) load_scales(j + kSpan);
          }
          uint32_t p[2 * MT][4];
#pragma unroll
          for (int i = 0; i < 2 * MT; ++i) {
            const uint32_t w = WIDE ? (j == 0 ? wide[i].x : j == 1 ? wide[i].y : j == 2 ? wide[i].z : wide[i].w)
                                    : *reinterpret_cast<const uint32_t*>(slot + i * 512 + (j ^ swizzle) * 16 + t * 4);
            unpack_word(w, c0[i], c1[i], p[i]);
          }
          const uint4 v = x[j];
          uint32_t x0 = v.x, x1 = v.y, x2 = v.z, x3 = v.w;
          if (MODE != kDown) {  // inputs i and i + 4 side by side, as the codes
            x0 = __byte_perm(v.x, v.z, 0x5410);
            x1 = __byte_perm(v.x, v.z, 0x7632);
            x2 = __byte_perm(v.y, v.w, 0x5410);
            x3 = __byte_perm(v.y, v.w, 0x7632);
          }
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            float(&d)[4] = part[mt];
            if (starts)
              mma_bf16(d, p[2 * mt][0], p[2 * mt + 1][0], p[2 * mt][1], p[2 * mt + 1][1], x0, x1, none);
            else
              mma_bf16(d, p[2 * mt][0], p[2 * mt + 1][0], p[2 * mt][1], p[2 * mt + 1][1], x0, x1, d);
            mma_bf16(d, p[2 * mt][2], p[2 * mt + 1][2], p[2 * mt][3], p[2 * mt + 1][3], x2, x3, d);
            if (ends) {
#pragma unroll
              for (int c = 0; c < 4; ++c) acc[mt][c] = fmaf(f[2 * mt + (c >> 1)], d[c], acc[mt][c]);
            }
          }
        }
      }
      if (sub < active) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int c = 0; c < 4; ++c) red[buf][warp][t * 2 + (c & 1)][mt * 16 + (c >> 1) * 8 + g] = acc[mt][c];
      }
    };
    if (un.mt == 2) products(std::integral_constant<int, 2>());
    else products(std::integral_constant<int, 1>());

    // The warps' sums, joined in warp order.  One barrier a unit: a warp that writes this buffer
    // again has passed the next unit's barrier, and so have all that read it here.
    asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "r"(split * 32) : "memory");
    const int w0 = team * split;
    auto sum = [&](int tok, int row) {
      float v = 0.f;
      for (int w = 0; w < active; ++w) {
#pragma unroll
        for (int p = 0; p < kPlanes; ++p) v += red[buf][w0 + w][tok * kPlanes + p][row];
      }
      return v * 4.f;
    };
    const int unit_outs = un.mt * kOut;
    for (int o = sub * 32 + lane; o < un.m * 2 * kOut; o += split * 32) {
      const int tok = o / (2 * kOut), out = o % (2 * kOut);
      if (out >= unit_outs || un.row0 + out >= outs) continue;
      store_out<MODE>(a, un.first + tok, un.row0 + out, outs, sum(tok, SWIGLU ? (out >> 3) * 16 + (out & 7) : out),
                      SWIGLU ? sum(tok, (out >> 3) * 16 + 8 + (out & 7)) : 0.f);
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

// Units are counted in 32 bits: blocks of at least 8 outputs of every expert, and tiles of at least 32
// tokens by 64 outputs.
bool units_fit(int n_rows, int E, int outs) {
  const long long few = static_cast<long long>(E) * (outs / 8 + 1);
  const long long wide = (static_cast<long long>(n_rows) / 32 + E) * (outs / 64 + 1);
  return few < (1LL << 31) - 65536 && wide < (1LL << 31) - 65536;
}

int check_w4_pointers(const afd_ffn_w4* w) {
  // scales and zero points are fetched in 4-byte words
  const uintptr_t mis = (reinterpret_cast<uintptr_t>(w->scale) | reinterpret_cast<uintptr_t>(w->zero)) & 3u;
  if (!w->codes || !w->scale || !aligned16(w->codes) || mis) return AFD_ERR_INVALID_ARG;
  return AFD_OK;
}

constexpr int kRingBytes = kWarps * kStages * kTileBytes;
constexpr int kMaxDevices = 64;

// A kernel's launch on the current device; at most one of the stream's kernels may still run when it
// starts (programmatic), which it waits for before it reads what that one writes.
template <typename... Args>
cudaError_t launch_on_device(void (*kernel)(Args...), std::atomic<int>* sm_count, int ctas_per_sm, int threads, int smem,
                             bool programmatic, cudaStream_t s, const Args&... args) {
  // per device and kernel, once: the SM count, and leave for the shared memory
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  int sms = dev < kMaxDevices ? sm_count[dev].load(std::memory_order_relaxed) : 0;
  if (sms == 0) {
    e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    if (dev < kMaxDevices) sm_count[dev].store(sms, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(ctas_per_sm * sms);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = programmatic ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int MODE, int PARTS, bool ZERO>
cudaError_t launch_few(const W4Args& a, bool programmatic, cudaStream_t s) {
  static std::atomic<int> sm_count[kMaxDevices];
  return launch_on_device(w4_rows_kernel<MODE, PARTS, ZERO>, sm_count, 2, kThreads, kRingBytes, programmatic, s, a);
}

template <int MODE, int PARTS>
cudaError_t launch_wide(const CUtensorMap& codes, const W4Args& a, bool programmatic, cudaStream_t s) {
  static std::atomic<int> sm_count[kMaxDevices];
  return launch_on_device(w4_wide_kernel<MODE, PARTS>, sm_count, 1, kWideThreads, kWideSmem, programmatic, s, codes, a);
}

template <int MODE, int PARTS>
cudaError_t launch_parts(const W4Args& a, bool few, const CUtensorMap* more, bool after, cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  if (few) e = a.zero ? launch_few<MODE, PARTS, true>(a, after, s) : launch_few<MODE, PARTS, false>(a, after, s);
  if (more && e == cudaSuccess) e = launch_wide<MODE, PARTS>(*more, a, after || few, s);
  return e;
}

// One product: the experts with few rows, then those with more.  Only a call that can have such
// rows launches a kernel for them.  after: the product reads what the stream's last kernel writes.
template <int MODE>
int launch_w4(const afd_ffn_w4& w, int E, const void* x, const int32_t* counts, int n_rows, void* y, int y_f32, int* err,
              bool after, cudaStream_t s) {
  constexpr int kPlanes = MODE == kDown ? 2 : 1;
  W4Args a{};
  a.codes = static_cast<const uint8_t*>(w.codes);
  a.scale = w.scale;
  a.zero = w.zero;
  a.x = static_cast<const __nv_bfloat16*>(x);
  a.counts = counts;
  a.y = y;
  a.E = E; a.N = w.N; a.K = w.K; a.G = w.group; a.n_rows = n_rows;
  a.scale_f32 = w.scale_dtype == AFD_DT_F32;
  a.y_f32 = y_f32;
  const unsigned q = w.group / 32;
  a.group_inv = q == 1 ? 0u : static_cast<unsigned>(((1ull << 32) + q - 1) / q);
  // groups that 16 bytes of scales hold; a slice's groups lie in one such piece where slices and groups nest
  const int piece = a.scale_f32 ? 4 : 8;
  a.windows = a.K / a.G % piece == 0 && (w.group % kSliceK == 0 || kSliceK % w.group == 0) && aligned16(w.scale) &&
              (reinterpret_cast<uintptr_t>(w.zero) & (piece - 1)) == 0;
  a.err = err;
  const bool more = static_cast<long long>(n_rows) * kPlanes > kCols;
  CUtensorMap map;
  if (more && !encode_byte_rows(&map, w.codes, w.K / 2, static_cast<uint64_t>(E) * w.N, kSliceK / 2, kWideRows / 2))
    return AFD_ERR_NO_DEVICE;
  const bool few = !more || counts;
  const CUtensorMap* m = more ? &map : nullptr;
  const cudaError_t e = w.group % 128 == 0  ? launch_parts<MODE, 1>(a, few, m, after, s)
                        : w.group % 64 == 0 ? launch_parts<MODE, 2>(a, few, m, after, s)
                                            : launch_parts<MODE, 4>(a, few, m, after, s);
  return e == cudaSuccess ? AFD_OK : rows_cuda_fail(e);
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
  if (n_rows > kW4MaxRows || !units_fit(n_rows, E, w->N)) return AFD_ERR_UNSUPPORTED;
  if (n_rows == 0) return AFD_OK;
  if ((st = check_w4_pointers(w)) != AFD_OK) return st;
  if (!x || !y || !aligned16(x) || !aligned16(y)) return AFD_ERR_INVALID_ARG;
  int* err = nullptr;
  if ((st = rows_err_word(&err)) != AFD_OK) return st;
  return launch_w4<kRows>(*w, E, x, counts, n_rows, y, y_dtype == AFD_DT_F32, err, false, static_cast<cudaStream_t>(stream));
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
  if (n_rows > kW4MaxRows || !units_fit(n_rows, E, w2->K) || !units_fit(n_rows, E, w2->N))
    return AFD_ERR_UNSUPPORTED;
  if (n_rows == 0) return AFD_OK;
  if ((st = check_w4_pointers(w13)) != AFD_OK || (st = check_w4_pointers(w2)) != AFD_OK) return st;
  if (!rows || !Y || !scratch || !aligned16(rows) || !aligned16(Y) || !aligned16(scratch)) return AFD_ERR_INVALID_ARG;
  int* err = nullptr;
  if ((st = rows_err_word(&err)) != AFD_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if ((st = launch_w4<kGateUp>(*w13, E, rows, counts, n_rows, scratch, 0, err, false, s)) != AFD_OK) return st;
  return launch_w4<kDown>(*w2, E, scratch, counts, n_rows, Y, y_dtype == AFD_DT_F32, err, true, s);
}
