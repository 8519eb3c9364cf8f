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
constexpr int kCols = 16;          // columns of a unit, two n8 tiles: 16 tokens, or 8 of two planes
constexpr int kRedPitch = kUnitRows + 4;

struct W4Args {
  const uint8_t* codes;
  const void* scale;
  const uint8_t* zero;
  const __nv_bfloat16* x;   // [n_rows * planes][K]
  const int32_t* counts;    // [E], or nullptr: one expert, every row
  void* y;
  int E, N, K, G, n_rows, scale_f32, y_f32;
  int scale_words, zero_words;  // 4-byte words a row's scales / zero points of one step can touch
  int slot_bytes;           // one step of one warp in the ring
  int split;                // warps that share a unit, each with its own slices of K: 1, 2, 4 or 8
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
// This kernel's dependents may start; wait for the kernel this one depends on (nothing outside a
// programmatic launch).
__device__ __forceinline__ void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_dependency() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// D (16 x 8, fp32) += A (16 x 16, bf16) B (16 x 8, bf16)
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}

// (q - z) / 4 of a word's codes i and i + 4 as bf16 pairs p[i].  A code in the low four bits of a
// half, under the exponent of 128, reads 128 + q.  One four bits up reads q 2^-129 as it stands:
// subnormal up to 7, and the first normal numbers go on in the same steps.  Both are exact, and so
// are the FMAs.  c0 = -(128 + z) / 4, c1 = -z / 4, in both halves.
__device__ __forceinline__ void unpack_word(uint32_t w, uint32_t c0, uint32_t c1, uint32_t (&p)[4]) {
  constexpr uint32_t kQuarter = 0x3E803E80u, k2to127 = 0x7F007F00u;
  const uint32_t s = w >> 8;
  p[0] = fma_bf16x2((w & 0x000f000fu) | 0x43004300u, kQuarter, c0);
  p[1] = fma_bf16x2(w & 0x00f000f0u, k2to127, c1);
  p[2] = fma_bf16x2((s & 0x000f000fu) | 0x43004300u, kQuarter, c0);
  p[3] = fma_bf16x2(s & 0x00f000f0u, k2to127, c1);
}

// ---------------------------------------------------------------------- the product
struct UnitTables {
  int first[kW4MaxExperts], rows[kW4MaxExperts], unit_base[kW4MaxExperts + 1];
};

// Rows and unit bases of every expert from counts: negative counts are flagged and taken as 0,
// rows past n_rows are flagged and cut off.  Expert e has ceil(rows / kTokens) * blocks units.
template <int kTokens>
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

// One unit: an expert, 32 weight rows (SwiGLU: 16 gate rows and their 16 up rows) and up to kTokens
// of its tokens, over the whole of K.
struct Unit {
  int e, first, m, row0;  // first token row, tokens, first output column
};

template <bool SWIGLU, int kTokens>
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

// A row group's scales and zero points in one step (WIDE: one group, else one per 32 inputs).
template <bool WIDE, bool ZERO>
struct Scales {
  float sc[WIDE ? 1 : 4][4];
  uint32_t z0[ZERO ? (WIDE ? 1 : 4) : 1][ZERO ? 4 : 1], z1[ZERO ? (WIDE ? 1 : 4) : 1][ZERO ? 4 : 1];

  __device__ __forceinline__ void load(const W4Args& a, const uint8_t* slot, const int (&phase)[4], int kq, int g0, int g,
                                       int steps) {
    if (!ZERO) {
      z0[0][0] = 0xC208C208u;  // -(128 + 8) / 4
      z1[0][0] = 0xC000C000u;  // -8 / 4
    }
#pragma unroll
    for (int j = 0; j < (WIDE ? 1 : 4); ++j) {
      if (!WIDE && j >= steps) break;
      const int d = WIDE ? 0 : static_cast<int>(((kq + j) * a.group_inv) >> 32) - g0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = i * 8 + g, ph = phase[i] + g0;
        const uint8_t* sa = slot + kTileBytes + row * a.scale_words * 4;
        if (a.scale_f32)
          sc[j][i] = *reinterpret_cast<const float*>(sa + d * 4);
        else
          sc[j][i] = __uint_as_float(static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(sa + ((ph & 1) + d) * 2)) << 16);
        if (ZERO) {
          const uint32_t z = slot[kTileBytes + 32 * a.scale_words * 4 + row * a.zero_words * 4 + (ph & 3) + d] & 15u;
          const uint32_t b = (z | 0x4300u) * 0x10001u;            // 128 + z
          z0[j][i] = fma_bf16x2(b, 0xBE80BE80u, 0x80008000u);     // -(128 + z) / 4
          z1[j][i] = fma_bf16x2(b, 0xBE80BE80u, 0x42004200u);     // 32 - (128 + z) / 4
        }
      }
    }
  }
  __device__ __forceinline__ void unpack(uint32_t w, int j, int i, uint32_t (&p)[4]) const {
    unpack_word(w, z0[ZERO && !WIDE ? j : 0][ZERO ? i : 0], z1[ZERO && !WIDE ? j : 0][ZERO ? i : 0], p);
  }
};

constexpr int kStages = 4;

// What a product is for.  kGateUp: gate and up rows, the SwiGLU rows out as two bf16 terms; kDown: from
// those to the results; kRows: one product on its own.
enum W4Mode { kRows, kGateUp, kDown };

// Place of input i of eight in the SwiGLU rows: the order in which unpack_word pairs the codes.
__device__ __forceinline__ int paired_place(int i) { return (i & ~7) | ((i & 3) << 1) | (i >> 2 & 1); }

template <int MODE, bool WIDE, bool ZERO>
__global__ void __launch_bounds__(kThreads, 2) w4_rows_kernel(const W4Args a) {
  constexpr bool SWIGLU = MODE == kGateUp;
  constexpr int kPlanes = MODE == kDown ? 2 : 1, kTokens = kCols / kPlanes;
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ UnitTables tb;
  __shared__ int wsum[kWarps];
  __shared__ float red[kWarps][kCols][kRedPitch];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3;
  if (MODE == kGateUp) launch_dependents();
  const int outs = SWIGLU ? a.N / 2 : a.N;
  constexpr int kOut = SWIGLU ? kUnitRows / 2 : kUnitRows;
  build_tables<kTokens>(a, (outs + kOut - 1) / kOut, tb, wsum);
  const int total = tb.unit_base[a.E];
  const int KG = a.K / a.G;
  // split warps share a unit; each team of them takes every teams-th unit
  const int sub = warp % a.split, team = warp / a.split;
  const int rounds = (a.K + a.split * kSliceK - 1) / (a.split * kSliceK);
  const int active = min(a.split, (a.K + kSliceK - 1) / kSliceK);  // warps of a team with a slice of K
  const int u0 = team * gridDim.x + blockIdx.x, teams = gridDim.x * (kWarps / a.split);

  uint8_t* const my_slots = ring + warp * kStages * a.slot_bytes;
  const uint32_t my_ring = smem_u32(my_slots);
  const int cps = a.scale_f32 ? 4 : 2;

  // ---- loads: a step is 32 rows x 128 inputs of one round of one unit
  int lu = u0, lr = 0, le = 0, lslot = 0;
  const uint8_t* wp[4];
  const uint8_t *sp = nullptr, *zp = nullptr;  // the word that holds the first scale / zero point of this lane's row
  int sleft = 0, zleft = 0, sphase = 0;  // bytes from there to the tensor's end (at most 2^30), scales before it in the word
  auto load_unit = [&]() {
    const Unit un = unit_at<SWIGLU, kTokens>(lu, &le, tb);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = weight_row<SWIGLU>(a, un.row0, i * 8 + g);
      wp[i] = a.codes + (static_cast<size_t>(un.e) * a.N + r) * (a.K / 2) + t * 16;
    }
    const long long at = (static_cast<long long>(un.e) * a.N + weight_row<SWIGLU>(a, un.row0, lane)) * KG;
    const long long end = static_cast<long long>(a.E) * a.N * KG;
    const long long sb = at * cps & ~3LL;
    sp = static_cast<const uint8_t*>(a.scale) + sb;
    sleft = static_cast<int>(min(end * cps - sb, 1LL << 30));
    sphase = static_cast<int>(at & 3);
    if (ZERO) {
      zp = a.zero + (at & ~3LL);
      zleft = static_cast<int>(min(end - (at & ~3LL), 1LL << 30));
    }
  };
  auto load_step = [&]() {
    if (lu < total) {
      if (lr == 0) load_unit();
      const int k = (lr * a.split + sub) * kSliceK;
      if (k < a.K) {
        const uint32_t slot = my_ring + lslot * a.slot_bytes;
        const bool in = WIDE || k + t * 32 < a.K;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = i * 8 + g;
          cp_async16(slot + r * 64 + ((t ^ ((r >> 1) & 3)) * 16), in ? wp[i] + k / 2 : a.codes, in);
        }
        const int g0 = static_cast<int>((k / 32 * a.group_inv) >> 32);
        // the words that hold the scales from g0 on (as many as a step can need), cut at the tensor's end
        const int so = a.scale_f32 ? g0 * 4 : ((sphase & 1) + g0) * 2 & ~3;
        const uint32_t sdst = slot + kTileBytes + lane * a.scale_words * 4;
        for (int w = 0; w < a.scale_words; ++w) {
          const int n = min(4, max(0, sleft - so - w * 4));
          cp_async4(sdst + w * 4, n ? sp + so + w * 4 : sp, n);
        }
        if (ZERO) {
          const int zo = (sphase + g0) & ~3;
          const uint32_t zdst = slot + kTileBytes + 32 * a.scale_words * 4 + lane * a.zero_words * 4;
          for (int w = 0; w < a.zero_words; ++w) {
            const int n = min(4, max(0, zleft - zo - w * 4));
            cp_async4(zdst + w * 4, n ? zp + zo + w * 4 : zp, n);
          }
        }
      }
      if (++lr == rounds) {
        lr = 0;
        lu += teams;
      }
    }
    cp_async_commit();
    lslot = lslot + 1 == kStages ? 0 : lslot + 1;
  };

#pragma unroll 1
  for (int i = 0; i < kStages - 1; ++i) load_step();
  if (MODE == kDown) wait_dependency();

  int ce = 0, cslot = 0;
  for (int u = u0; u < total; u += teams) {
    const Unit un = unit_at<SWIGLU, kTokens>(u, &ce, tb);
    // phase of each row's first scale in its words
    int phase[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      phase[i] = static_cast<int>(((static_cast<long long>(un.e) * a.N + weight_row<SWIGLU>(a, un.row0, i * 8 + g)) * KG) & 3);
    // columns past the last one repeat it; their results are not used
    const int cols = un.m * kPlanes;
    const __nv_bfloat16* col[2];
#pragma unroll
    for (int n = 0; n < 2; ++n)
      col[n] = a.x + (static_cast<size_t>(un.first) * kPlanes + min(n * 8 + g, cols - 1)) * a.K + t * (WIDE ? 32 : 8);
    const bool two = cols > 8;
    float acc[2][2][4];
#pragma unroll
    for (int i = 0; i < 16; ++i) (&acc[0][0][0])[i] = 0.f;

    for (int r = 0; r < rounds; ++r) {
      const int k = (r * a.split + sub) * kSliceK;
      const bool mine = k < a.K;
      const uint8_t* slot = my_slots + cslot * a.slot_bytes;
      cslot = cslot + 1 == kStages ? 0 : cslot + 1;
      const int steps = WIDE ? 4 : min(4, (a.K - k) / 32);
      uint4 b[4];
      if (mine) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (WIDE || j < steps) b[j] = *reinterpret_cast<const uint4*>(col[0] + k + j * (WIDE ? 8 : 32));
      }
      cp_async_wait<kStages - 2>();
      __syncwarp();
      load_step();
      if (!mine) continue;
      const int kq = k / 32, g0 = static_cast<int>((kq * a.group_inv) >> 32);
      Scales<WIDE, ZERO> s;
      s.load(a, slot, phase, kq, g0, g, steps);
      uint4 wide[4];
      if (WIDE) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          wide[i] = *reinterpret_cast<const uint4*>(slot + (i * 8 + g) * 64 + ((t ^ ((g >> 1) & 3)) * 16));
      }
      float part[2][2][4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (!WIDE && j >= steps) break;
        if (!WIDE || j == 0) {
#pragma unroll
          for (int i = 0; i < 16; ++i) (&part[0][0][0])[i] = 0.f;
        }
        uint32_t p[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t w = WIDE ? (j == 0 ? wide[i].x : j == 1 ? wide[i].y : j == 2 ? wide[i].z : wide[i].w)
                                  : *reinterpret_cast<const uint32_t*>(slot + (i * 8 + g) * 64 + ((j ^ ((g >> 1) & 3)) * 16) + t * 4);
          s.unpack(w, j, i, p[i]);
        }
        auto products = [&](const uint4& v, float (&d)[2][4]) {
          uint32_t b0 = v.x, b1 = v.y, b2 = v.z, b3 = v.w;
          if (MODE != kDown) {  // inputs i and i + 4 side by side, as the codes
            b0 = __byte_perm(v.x, v.z, 0x5410);
            b1 = __byte_perm(v.x, v.z, 0x7632);
            b2 = __byte_perm(v.y, v.w, 0x5410);
            b3 = __byte_perm(v.y, v.w, 0x7632);
          }
#pragma unroll
          for (int mt = 0; mt < 2; ++mt) {
            mma_bf16(d[mt], p[2 * mt][0], p[2 * mt + 1][0], p[2 * mt][1], p[2 * mt + 1][1], b0, b1);
            mma_bf16(d[mt], p[2 * mt][2], p[2 * mt + 1][2], p[2 * mt][3], p[2 * mt + 1][3], b2, b3);
          }
        };
        products(b[j], part[0]);
        if (two) products(*reinterpret_cast<const uint4*>(col[1] + k + j * (WIDE ? 8 : 32)), part[1]);
        if (!WIDE || j == 3) {
#pragma unroll
          for (int mt = 0; mt < 2; ++mt)
#pragma unroll
            for (int c = 0; c < 4; ++c) acc[0][mt][c] = fmaf(s.sc[WIDE ? 0 : j][2 * mt + (c >> 1)], part[0][mt][c], acc[0][mt][c]);
          if (two) {
#pragma unroll
            for (int mt = 0; mt < 2; ++mt)
#pragma unroll
              for (int c = 0; c < 4; ++c)
                acc[1][mt][c] = fmaf(s.sc[WIDE ? 0 : j][2 * mt + (c >> 1)], part[1][mt][c], acc[1][mt][c]);
          }
        }
      }
    }

    // the warps' sums, joined in warp order
    if (sub < active) {
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        if (n == 1 && !two) break;
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
          for (int c = 0; c < 4; ++c) red[warp][n * 8 + t * 2 + (c & 1)][mt * 16 + (c >> 1) * 8 + g] = acc[n][mt][c];
      }
    }
    asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "r"(a.split * 32) : "memory");
    const int w0 = team * a.split;
    auto sum = [&](int tok, int row) {
      float v = 0.f;
      for (int w = 0; w < active; ++w) {
#pragma unroll
        for (int p = 0; p < kPlanes; ++p) v += red[w0 + w][tok * kPlanes + p][row];
      }
      return v * 4.f;
    };
    for (int o = sub * 32 + lane; o < un.m * kOut; o += a.split * 32) {
      const int tok = o / kOut, out = o % kOut;
      if (un.row0 + out >= outs) continue;
      const float v = sum(tok, out);
      if (SWIGLU) {
        const float up = sum(tok, 16 + out);
        const float act = v / (1.f + expf(-v)) * up;
        const __nv_bfloat16 hi = __float2bfloat16_rn(act);
        // an infinite or NaN value is its own high term alone
        const __nv_bfloat16 lo = __float2bfloat16_rn(fabsf(act) < INFINITY ? act - __bfloat162float(hi) : 0.f);
        __nv_bfloat16* y = static_cast<__nv_bfloat16*>(a.y) + static_cast<size_t>(un.first + tok) * 2 * outs + paired_place(un.row0 + out);
        y[0] = hi;
        y[outs] = lo;
      } else {
        const size_t at = static_cast<size_t>(un.first + tok) * outs + un.row0 + out;
        if (a.y_f32)
          static_cast<float*>(a.y)[at] = v;
        else
          static_cast<__nv_bfloat16*>(a.y)[at] = __float2bfloat16_rn(v);
      }
    }
    asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "r"(a.split * 32) : "memory");  // red is free again
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
bool units_fit(int n_rows, int E, int outs, int unit_outs, int unit_tokens) {
  const long long units = (static_cast<long long>(n_rows) / unit_tokens + E) * ((outs + unit_outs - 1) / unit_outs);
  return units < (1LL << 31) - 65536;
}

int check_w4_pointers(const afd_ffn_w4* w) {
  // scales and zero points are fetched in 4-byte words
  const uintptr_t mis = (reinterpret_cast<uintptr_t>(w->scale) | reinterpret_cast<uintptr_t>(w->zero)) & 3u;
  if (!w->codes || !w->scale || !aligned16(w->codes) || mis) return AFD_ERR_INVALID_ARG;
  return AFD_OK;
}

constexpr int kMaxSlotBytes = kTileBytes + 32 * 4 * (4 + 2);
constexpr int kMaxDevices = 64;

// Warps that share a unit.  A step takes a warp the same time whatever the split; a unit costs its
// team ceil(K / 128 / split) steps and about one more for the join, and the teams take
// ceil(units / teams) units one after another.  The smallest such product wins; experts that rows
// reach are taken as min(E, n_rows).
int choose_split(int n_rows, int E, int blocks, int K, int ctas) {
  const long long units = static_cast<long long>(std::min(E, n_rows)) * blocks;
  int best = 8;
  long long least = -1;
  for (int split = 8; split >= 1; split /= 2) {
    const long long teams = static_cast<long long>(ctas) * (kWarps / split);
    const long long cost = ((units + teams - 1) / teams) * ((K + kSliceK * split - 1) / (kSliceK * split) + 1);
    if (least < 0 || cost < least) {
      least = cost;
      best = split;
    }
  }
  return best;
}

template <int MODE, bool WIDE, bool ZERO>
cudaError_t launch_w4_kernel(W4Args& a, cudaStream_t s) {
  auto kernel = w4_rows_kernel<MODE, WIDE, ZERO>;
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
  constexpr int kOut = MODE == kGateUp ? kUnitRows / 2 : kUnitRows;
  const int outs = MODE == kGateUp ? a.N / 2 : a.N;
  a.split = choose_split(a.n_rows, a.E, (outs + kOut - 1) / kOut, a.K, 2 * sms);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(2 * sms);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kWarps * kStages * a.slot_bytes;
  cfg.stream = s;
  // The down product starts on its weights while the gate/up product drains.
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = MODE == kDown ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <int MODE>
cudaError_t launch_w4(const afd_ffn_w4& w, int E, const void* x, const int32_t* counts, int n_rows, void* y, int y_f32,
                      int* err, cudaStream_t s) {
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
  // groups that 128 inputs can reach, in 4-byte words that may start inside one
  const bool wide = w.group % kSliceK == 0;
  const int reach = wide ? 1 : w.group == 32 ? 4 : 2;
  a.scale_words = a.scale_f32 ? reach : reach / 2 + 1;
  a.zero_words = w.zero ? (reach == 1 ? 1 : 2) : 0;
  a.slot_bytes = kTileBytes + 32 * 4 * (a.scale_words + a.zero_words);
  const unsigned q = w.group / 32;
  a.group_inv = ((1ull << 32) + q - 1) / q;
  a.err = err;
  if (wide) return w.zero ? launch_w4_kernel<MODE, true, true>(a, s) : launch_w4_kernel<MODE, true, false>(a, s);
  return w.zero ? launch_w4_kernel<MODE, false, true>(a, s) : launch_w4_kernel<MODE, false, false>(a, s);
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
  if (n_rows > kW4MaxRows || !units_fit(n_rows, E, w->N, kUnitRows, kCols)) return AFD_ERR_UNSUPPORTED;
  if (n_rows == 0) return AFD_OK;
  if ((st = check_w4_pointers(w)) != AFD_OK) return st;
  if (!x || !y || !aligned16(x) || !aligned16(y)) return AFD_ERR_INVALID_ARG;
  int* err = nullptr;
  if ((st = rows_err_word(&err)) != AFD_OK) return st;
  const cudaError_t e = launch_w4<kRows>(*w, E, x, counts, n_rows, y, y_dtype == AFD_DT_F32, err,
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
  if (n_rows > kW4MaxRows || !units_fit(n_rows, E, w2->K, kUnitRows / 2, kCols) || !units_fit(n_rows, E, w2->N, kUnitRows, kCols / 2))
    return AFD_ERR_UNSUPPORTED;
  if (n_rows == 0) return AFD_OK;
  if ((st = check_w4_pointers(w13)) != AFD_OK || (st = check_w4_pointers(w2)) != AFD_OK) return st;
  if (!rows || !Y || !scratch || !aligned16(rows) || !aligned16(Y) || !aligned16(scratch)) return AFD_ERR_INVALID_ARG;
  int* err = nullptr;
  if ((st = rows_err_word(&err)) != AFD_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = launch_w4<kGateUp>(*w13, E, rows, counts, n_rows, scratch, 0, err, s);
  if (e == cudaSuccess) e = launch_w4<kDown>(*w2, E, scratch, counts, n_rows, Y, y_dtype == AFD_DT_F32, err, s);
  return e == cudaSuccess ? AFD_OK : rows_cuda_fail(e);
}
