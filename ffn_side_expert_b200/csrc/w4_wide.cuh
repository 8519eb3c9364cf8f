// w4_wide.cuh -- 4-bit products of the experts with more columns (tokens, or planes of tokens) than
// w4_narrow.cuh takes, on the 5th-generation tensor cores.
//
// A unit is 128 weight rows (SwiGLU: 64 gate rows and their 64 up rows) and up to 64 columns (tokens,
// or planes of tokens).  A warpgroup's thread owns a weight row, that is a TMEM lane: it unpacks the
// row's codes of a slice of 128 inputs to bf16 (q - z) / 4 and stores them to TMEM, where they are
// the A operand (tcgen05.mma with A in TMEM), so unpacked weights cost no shared-memory traffic.
// The tokens' slice goes to shared memory, in the order in which unpack_word pairs the codes.
// One accumulator per group of inputs; the thread adds it, times the group's scale, to its row's
// sums in registers: fp32 throughout, and (q - z) / 4 is exact.
//
// What bounds it: unpacking (w4.cu), once per 64 columns.  Four warpgroups work on their
// own slices or units, so one's unpacking covers the others' MMA and TMEM round trips.  Codes come by
// TMA, a ring of three slices per warpgroup.
#pragma once

#include <cuda.h>

namespace afd {

constexpr int kWgs = 4, kWideThreads = kWgs * 128;
constexpr int kWideRows = 128, kWideCols = 64;
constexpr int kWideStages = 3;
constexpr int kCodeBytes = kWideRows * kSliceK / 2;            // a slice's codes
constexpr int kTokenBytes = kWideCols * kSliceK * 2;           // and tokens; the join's buffer too
constexpr int kWindowBytes = 16 + 8;                           // a thread's scales and zero points
constexpr int kWideSmem = 1024 + kWgs * (kWideStages * kCodeBytes + kTokenBytes) + kWideThreads * kWindowBytes;
static_assert(16 * kWideRows * 4 <= kTokenBytes, "the join's 16 columns of partial sums fit");

// D[tmem] (+)= A[tmem] B[smem]^T, one M128 x N x K16 instruction.
__device__ __forceinline__ void tc_mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                          uint32_t accumulate) {
  const uint32_t z = 0;
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, {%5, %6, %7, %8}, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(z), "r"(z), "r"(z), "r"(z));
}

// 32 lanes x 16 columns from registers to TMEM.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[4][4]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0][0]), "r"(r[0][1]), "r"(r[0][2]), "r"(r[0][3]), "r"(r[1][0]), "r"(r[1][1]), "r"(r[1][2]), "r"(r[1][3]),
      "r"(r[2][0]), "r"(r[2][1]), "r"(r[2][2]), "r"(r[2][3]), "r"(r[3][0]), "r"(r[3][1]), "r"(r[3][2]), "r"(r[3][3])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void group_barrier(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// Columns of a unit and warpgroups that share one, each with its own slices.
struct WideShape {
  int cols, split;
};

// The shape of the least cost: a team takes ceil(units / teams) units of ceil(slices / split) steps and about
// 1.5 more for the join; a step of 32 columns takes 1.2 and one of 64 twice the time of one of 16.
// tiles: token tiles of all experts at 16, 32 and 64 columns.
__device__ __forceinline__ WideShape choose_wide(const int (&tiles)[3], unsigned blocks, unsigned slices, unsigned ctas) {
  const int lane = threadIdx.x & 31, log = lane % 3, size = lane / 3;  // a lane for each candidate
  static_assert(kWgs == 4, "splits of 1, 2 and 4");
  unsigned cost = 0xffffffffu;
  if (lane < 9) {
    const unsigned teams = ctas * (kWgs >> log), units = (size == 0 ? tiles[0] : size == 1 ? tiles[1] : tiles[2]) * blocks;
    const float step = size == 0 ? 10.f : size == 1 ? 12.f : 20.f;
    const float c = static_cast<float>((units + teams - 1) / teams) *
                    (static_cast<float>((slices + (1u << log) - 1) >> log) * step + 15.f);
    cost = (__float_as_uint(c) & ~31u) | lane;
  }
  const int best = __reduce_min_sync(0xffffffffu, cost) & 31;
  return WideShape{16 << best / 3, 1 << best % 3};
}

struct WideUnit {
  int e, first, m, row0;  // expert, first token row, tokens, first output
};

template <int MODE>
__device__ __forceinline__ WideUnit wide_unit_at(int u, int* e, int tokens, const UnitTables& tb) {
  while (u >= tb.unit_base[*e + 1]) ++*e;
  WideUnit r;
  r.e = *e;
  const int rows = tb.rows[r.e], tiles = (rows + tokens - 1) / tokens;
  const int at = u - tb.unit_base[r.e], block = at / tiles, tile = at - block * tiles;
  r.first = tb.first[r.e] + tile * tokens;
  r.m = min(tokens, rows - tile * tokens);
  r.row0 = block * (MODE == kGateUp ? kWideRows / 2 : kWideRows);
  return r;
}

// PARTS: groups of a slice with a scale each (1, 2 or 4).
template <int MODE, int PARTS>
__global__ void __launch_bounds__(kWideThreads, 1)
w4_wide_kernel(const __grid_constant__ CUtensorMap codes, const W4Args a) {
  constexpr int kPlanes = MODE == kDown ? 2 : 1;
  constexpr int kOut = MODE == kGateUp ? kWideRows / 2 : kWideRows;
  extern __shared__ uint8_t smem_raw[];
  __shared__ UnitTables tb;
  __shared__ __align__(8) uint64_t bars[kWgs * (kWideStages + 1)];
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  // uniform over a warp, for the compiler too: an MMA with operands that it takes for per-thread values
  // is issued every 85 clocks, one with uniform operands every 15 (N = 16)
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const bool leader = elect_one();  // of its warp
  const int wg = warp >> 2, r = tid & 127;  // warpgroup; row of the unit, which is the TMEM lane
  volatile int* abort = &abort_flag;

  // what needs no input: barriers and TMEM
  if (tid < kWgs * (kWideStages + 1)) {
    mbar_init(smem_u32(&bars[tid]), 1);
    fence_barrier_init();
  }
  if (tid == 0) abort_flag = 0;
  if (warp == 1) {
    tmem_alloc(smem_u32(&tmem_slot), 512);
    tmem_relinquish();
  }
  if (a.first) wait_dependency();  // else the call's first kernel has, before this one could start (W4Args::first)
  const int outs = MODE == kGateUp ? a.N / 2 : a.N;
  const int blocks = (outs + kOut - 1) / kOut;
  const int slices = (a.K + kSliceK - 1) / kSliceK;
  int tiles[3];
  auto cols_of = [&](int rows) { return rows > a.above / kPlanes ? rows * kPlanes : 0; };
  count_rows<1>(a, cols_of, tb, tiles);
  const WideShape shape = choose_wide(tiles, blocks, slices, gridDim.x);
  const int tile = shape.cols / kPlanes;
  const int total = (shape.cols == 16 ? tiles[0] : shape.cols == 32 ? tiles[1] : tiles[2]) * blocks;
  if (warp == 0)
    base_units(a, [&](int rows) { return (cols_of(rows) + shape.cols - 1) / shape.cols * blocks; }, tb);
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* const gbase = smem_raw + (base - smem_u32(smem_raw));
  const uint32_t tokens = base + wg * kTokenBytes;                                             // this group's tokens
  uint8_t* const tokens_at = gbase + wg * kTokenBytes;
  const int ring_off = kWgs * kTokenBytes + wg * kWideStages * kCodeBytes;                     // and ring
  constexpr int kWindowOff = kWgs * (kTokenBytes + kWideStages * kCodeBytes);
  const uint32_t full = smem_u32(&bars[wg * (kWideStages + 1)]), mma_bar = full + 8 * kWideStages;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  launch_dependents();  // behind the wait above, and what follows allocates TMEM after this: as in w4_narrow.cuh
  const uint32_t tmem = tmem_slot;
  if (total == 0) {
    wait_dependency();  // what follows may rely on the kernel before this one
    if (warp == 1) tmem_dealloc(tmem, 512);
    return;
  }
  const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;  // the warp's lane quarter
  const uint64_t desc0 = sw128_desc(tokens);
  const uint32_t tm_a = tmem + wg * 64, tm_d = tmem + 256 + wg * 64;

  const int KG = a.KG, cps = a.scale_f32 ? 4 : 2;
  const int split = shape.split;
  const int sub = wg & (split - 1), team = wg / split;
  const int per = (slices + split - 1) / split;  // a group's consecutive slices
  const int steps = max(0, min(per, slices - sub * per));
  const int active = (slices + per - 1) / per;   // groups of a team with a slice
  const int teams = gridDim.x * (kWgs / split);
  const int u0 = team * gridDim.x + blockIdx.x;
  constexpr int kPartK = kSliceK / PARTS;

  auto wait = [&](uint32_t bar, uint32_t parity) {
    if (!mbar_wait(bar, parity, abort)) {
      *abort = 1;
      atomicOr(a.err, kErrTimeout);
    }
  };

  // ---- loads, by a lane of the group's second warp; one of the first issues the MMAs
  int lu = steps > 0 ? u0 : total, ls = 0, le = 0, lx = 0, lrow = 0, issued = 0;
  auto load_step = [&]() {
    if (lu >= total || *abort) return;
    if (ls == 0) {
      const WideUnit un = wide_unit_at<MODE>(lu, &le, tile, tb);
      lrow = un.e * a.N + un.row0;
      lx = sub * per * (kSliceK / 2);
    }
    const int slot = issued % kWideStages;
    const uint32_t bar = full + 8 * slot, dst = base + ring_off + slot * kCodeBytes;
    mbar_arrive_expect_tx(bar, kCodeBytes);
    tma_load_2d(dst, &codes, bar, lx, lrow, kEvictNormal);
    tma_load_2d(dst + kCodeBytes / 2, &codes, bar, lx, lrow + (MODE == kGateUp ? outs : 64), kEvictNormal);
    ++issued;
    lx += kSliceK / 2;
    if (++ls == steps) {
      ls = 0;
      lu += teams;
    }
  };
  if ((warp & 3) == 1 && leader)
    for (int i = 0; i < kWideStages; ++i) load_step();
  __syncwarp();

  // Row of the weights whose scales this thread applies, as the place of its first group; rows past
  // the end repeat the last one.
  auto scale_row = [&](const WideUnit& un) {
    const int row = MODE == kGateUp ? (r < 64 ? 0 : outs) + min(un.row0 + (r & 63), outs - 1) : min(un.row0 + r, outs - 1);
    return (static_cast<size_t>(un.e) * a.N + row) * KG;
  };
  // a unit's scales and zero points, into L2 a unit ahead
  int pe = 0;
  auto prefetch_scales = [&](int u) {
    if (u >= total) return;
    const size_t at = scale_row(wide_unit_at<MODE>(u, &pe, tile, tb));
    const uint8_t* sp = static_cast<const uint8_t*>(a.scale) + at * cps;
    for (int o = sub * 32; o < KG * cps; o += split * 32) prefetch_l2(sp + o);
    if (a.zero)
      for (int o = sub * 32; o < KG; o += split * 32) prefetch_l2(a.zero + at + o);
  };
  if (MODE == kDown) wait_dependency();

  int it = 0, ce = 0;
  uint32_t mma_phase = 0;
  for (int u = u0; u < total; u += teams) {
    const WideUnit un = wide_unit_at<MODE>(u, &ce, tile, tb);
    const int cols = un.m * kPlanes;
    const size_t srow = scale_row(un);
    prefetch_scales(u + teams);

    auto unit = [&](auto tiles) {
      constexpr int NT = decltype(tiles)::value, N = NT * 16;
      constexpr uint32_t idesc = idesc_mn(128, N, false);
      constexpr int kAtOnce = PARTS < kWideCols / N ? PARTS : kWideCols / N;  // parts whose accumulators fit side by side
      constexpr int kPer = 8 / PARTS;                                         // K16 steps of a part
      float acc[N];
#pragma unroll
      for (int i = 0; i < N; ++i) acc[i] = 0.f;
      // tokens: this thread moves 8 inputs (chunk kc of a slice) of columns r / 16 + 8 i
      const int kc = r & 15;
      const __nv_bfloat16* xb = a.x + static_cast<size_t>(un.first) * kPlanes * a.K + kc * 8;

      // Tokens: a thread moves its chunk of 8 inputs of columns r / 16 + 8 i.  The SwiGLU rows are in the
      // codes' order already, and 64 columns are multiplied in their own order, with codes unpacked
      // to it: those go by cp.async, as soon as the MMAs have read the slice before.  Fewer columns
      // go through registers, which put inputs i and i + 4 side by side.
      constexpr bool kOwnOrder = MODE != kDown && NT == 4, kAsync = MODE == kDown || kOwnOrder;
      uint4 v[kAsync ? 1 : NT * 2];
      auto load_tokens = [&](int k) {
        const bool in = k + kc * 8 < a.K;
#pragma unroll
        for (int i = 0; i < NT * 2; ++i) {
          const int n = i * 8 + (r >> 4);
          const __nv_bfloat16* src = xb + min(n, cols - 1) * a.K + k;
          if constexpr (kAsync)
            cp_async16(tokens + (kc >> 3) * (N * 128) + n * 128 + (((kc & 7) ^ (n & 7)) * 16), in ? src : a.x, in);
          else
            v[i] = in ? __ldcg(reinterpret_cast<const uint4*>(src)) : make_uint4(0u, 0u, 0u, 0u);
        }
        if constexpr (kAsync) cp_async_commit();
      };
      auto store_tokens = [&]() {
        if constexpr (!kAsync) {
#pragma unroll
          for (int i = 0; i < NT * 2; ++i) {
            const int n = i * 8 + (r >> 4);
            *reinterpret_cast<uint4*>(tokens_at + (kc >> 3) * (N * 128) + n * 128 + (((kc & 7) ^ (n & 7)) * 16)) =
                make_uint4(__byte_perm(v[i].x, v[i].z, 0x5410), __byte_perm(v[i].x, v[i].z, 0x7632),
                           __byte_perm(v[i].y, v[i].w, 0x5410), __byte_perm(v[i].y, v[i].w, 0x7632));
          }
        }
      };
      // Scales and zero points come in windows of 16 bytes of scales, by cp.async to a place of the
      // thread's own; a thread per row is 32 lines a load, so one load for eight groups matters.
      // Rows of an odd length or start are read group by group.
      const uint32_t wsc = base + kWindowOff + tid * 16, wz = base + kWindowOff + kWideThreads * 16 + tid * 8;
      const uint8_t* wat = gbase + kWindowOff + tid * 16;
      const uint8_t* zat = gbase + kWindowOff + kWideThreads * 16 + tid * 8;
      const int wlog = a.scale_f32 ? 2 : 3;
      int window = -1;
      uint32_t next_sc[PARTS], next_z[PARTS];  // as they are in memory
      auto load_scales = [&](int k) {
        if (a.windows) {
          const int w = group_of(a, k / 32) >> wlog;
          if (w != window) {
            window = w;
            const size_t at = srow + (static_cast<size_t>(w) << wlog);
            cp_async16(wsc, static_cast<const uint8_t*>(a.scale) + at * cps);
            if (a.zero) {
              if (wlog == 3) cp_async8(wz, a.zero + at);
              else cp_async4(wz, a.zero + at);
            }
            cp_async_commit();
          }
        } else {
#pragma unroll
          for (int p = 0; p < PARTS; ++p) {
            const size_t at = srow + group_of(a, min(k + p * kPartK, a.K - 32) / 32);
            if (a.scale_f32) next_sc[p] = __ldg(static_cast<const unsigned*>(a.scale) + at);
            else next_sc[p] = __ldg(static_cast<const unsigned short*>(a.scale) + at);
            next_z[p] = 8u;
            if (a.zero) next_z[p] = __ldg(a.zero + at);
          }
        }
      };
      const int k0 = sub * per * kSliceK;
      if (steps > 0) {
        load_tokens(k0);
        load_scales(k0);
      }

#pragma unroll 1
      for (int s = 0; s < steps; ++s, ++it) {
        const int k = k0 + s * kSliceK;
        float sc[PARTS];
        uint32_t z[PARTS];
        if (kAsync || a.windows) cp_async_wait<0>();
        if (a.windows) {
          const int at = group_of(a, k / 32) & ((1 << wlog) - 1);  // the parts' groups follow one another in it
#pragma unroll
          for (int p = 0; p < PARTS; ++p) {
            sc[p] = a.scale_f32 ? reinterpret_cast<const float*>(wat)[at + p]
                                : __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const unsigned short*>(wat)[at + p]) << 16);
            z[p] = a.zero ? zat[at + p] : 8u;
          }
        } else {
#pragma unroll
          for (int p = 0; p < PARTS; ++p) {
            sc[p] = __uint_as_float(a.scale_f32 ? next_sc[p] : next_sc[p] << 16);
            z[p] = next_z[p];
          }
        }
        wait(full + 8 * (it % kWideStages), (it / kWideStages) & 1);
        const uint8_t* row = gbase + ring_off + (it % kWideStages) * kCodeBytes + r * 64;
        uint32_t c0 = 0, c1 = 0;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint4 w = *reinterpret_cast<const uint4*>(row + ((c ^ ((r >> 1) & 3)) * 16));
          if (c % (4 / PARTS) == 0) {
            const uint32_t q = ((z[c * PARTS / 4] & 15u) | 0x4300u) * 0x10001u;  // 128 + z
            c0 = fma_bf16x2(q, 0xBE80BE80u, 0x80008000u);                        // -(128 + z) / 4
            c1 = fma_bf16x2(q, 0xBE80BE80u, 0x42004200u);                        // -z / 4
          }
          uint32_t p[4][4];
          unpack_word<kOwnOrder>(w.x, c0, c1, p[0]);
          unpack_word<kOwnOrder>(w.y, c0, c1, p[1]);
          unpack_word<kOwnOrder>(w.z, c0, c1, p[2]);
          unpack_word<kOwnOrder>(w.w, c0, c1, p[3]);
          tmem_st16(tm_a + lanes + c * 16, p);
        }
        store_tokens();
        tmem_st_wait();
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
#pragma unroll
        for (int p0 = 0; p0 < PARTS; p0 += kAtOnce) {
          // the slice is in place, or the accumulators of the parts before are read
          tc_fence_before();
          group_barrier(1 + wg, 128);
          if ((warp & 3) == 0 && leader) {
            tc_fence_after();
#pragma unroll
            for (int i = 0; i < kAtOnce * kPer; ++i) {
              const int ks = p0 * kPer + i;
              tc_mma_ts(tm_d + i / kPer * N, tm_a + ks * 8, desc0 + (((ks >> 2) * (N * 128) + (ks & 3) * 32) >> 4), idesc,
                        i % kPer > 0);
            }
            tc_commit(mma_bar);
          }
          if (p0 == 0 && (warp & 3) == 1 && leader) load_step();  // the ring's slot is read
          __syncwarp();
          const bool ahead = s + 1 < steps;
          if (p0 == 0 && ahead) {
            load_scales(k + kSliceK);
            if (!kAsync) load_tokens(k + kSliceK);
          }
          wait(mma_bar, mma_phase);
          mma_phase ^= 1;
          tc_fence_after();
          if (kAsync && p0 + kAtOnce == PARTS && ahead) load_tokens(k + kSliceK);
#pragma unroll
          for (int p = 0; p < kAtOnce; ++p) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              uint32_t d[16];
              tmem_ld16(tm_d + lanes + p * N + n * 16, d);
              tmem_ld_wait(d);
#pragma unroll
              for (int c = 0; c < 16; ++c) acc[n * 16 + c] = fmaf(sc[p0 + p], __uint_as_float(d[c]), acc[n * 16 + c]);
            }
          }
        }
      }

      // ---- results, sixteen columns at a time
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        if (n * 16 >= cols) break;
        if (split == 1 && MODE != kGateUp) {
          if (un.row0 + r < outs) {
#pragma unroll
            for (int c = 0; c < 16; c += kPlanes) {
              const int tok = (n * 16 + c) / kPlanes;
              const float v = kPlanes == 2 ? acc[n * 16 + c] + acc[n * 16 + c + 1] : acc[n * 16 + c];
              if (tok < un.m) store_out<MODE>(a, un.first + tok, un.row0 + r, outs, v * 4.f, 0.f);
            }
          }
          continue;
        }
        // partial sums to the group's token buffer, which its MMAs have read; joined in group order
        float* mine = reinterpret_cast<float*>(tokens_at);
#pragma unroll
        for (int c = 0; c < 16; ++c) mine[c * kWideRows + r] = acc[n * 16 + c];
        group_barrier(1 + kWgs + team, split * 128);
        const float* part = reinterpret_cast<const float*>(gbase + team * split * kTokenBytes);
        auto sum = [&](int c, int row) {
          float v = 0.f;
          for (int w = 0; w < active; ++w)
#pragma unroll
            for (int p = 0; p < kPlanes; ++p) v += part[w * (kTokenBytes / 4) + (c * kPlanes + p) * kWideRows + row];
          return v * 4.f;
        };
        constexpr int kShare = kWideRows / kOut;  // threads of a group per output
        for (int c = sub * kShare + r / kOut; c < 16 / kPlanes; c += split * kShare) {
          const int tok = n * (16 / kPlanes) + c, out = r % kOut;
          if (tok < un.m && un.row0 + out < outs)
            store_out<MODE>(a, un.first + tok, un.row0 + out, outs, sum(c, out), MODE == kGateUp ? sum(c, 64 + out) : 0.f);
        }
        group_barrier(1 + kWgs + team, split * 128);
      }
    };
    if (cols <= 16) unit(std::integral_constant<int, 1>());
    else if (cols <= 32) unit(std::integral_constant<int, 2>());
    else unit(std::integral_constant<int, 4>());
  }

  // After a wait that gave up: the group's own copies in flight, with a limit, before shared memory goes.
  if ((warp & 3) == 1 && leader && *abort) {
    int none = 0;
    for (; it < issued; ++it) mbar_wait(full + 8 * (it % kWideStages), (it / kWideStages) & 1, &none);
  }
  if (MODE != kDown) wait_dependency();  // what follows may rely on the kernel before this one
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace afd
