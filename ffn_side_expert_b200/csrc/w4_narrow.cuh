// w4_narrow.cuh -- 4-bit products of the experts with few columns (tokens, or planes of tokens), on
// the 5th-generation tensor cores, as in w4_wide.cuh: codes unpacked into TMEM as the A operand.
//
// A step of a warpgroup is 128 TMEM lanes of S inputs each against a tile of 16 columns: S = 256, or 128
// where groups are shorter than that.  With R = 128 the lanes are 128 weight rows of one slice of K, and
// the tile is 16 columns.  With R = 64 or 32 they are 128 / R slices of R rows, the tile holds R / 8
// columns of each slice, and a lane reads those of its own slice: what a wider MMA computes beside them
// costs nothing, and units of fewer rows spread few experts over the SMs.
//
// What bounds it: the chain of a step, at the 12 or 16 warps an SM that TMEM leaves room for, and whole units in
// rounds (one token's eight experts of H = 7168, I = 2048: 20 and 12 steps, where 16.1 and 8.1 would do if all
// groups got the same; 59 us for 28 of bytes).  At the HBM rate an SM gets 46 codes a clock, and unpacking
// alone takes 1.1 instructions a code; what a step takes besides (waits, barrier, scales, MMA issue,
// accumulators) is as much again for 128 inputs, which is why a step takes 256 where TMEM has room.  Issue
// is at half.  The accumulators of a step are read only when the next step's codes are there, so the MMAs
// run meanwhile.
#pragma once

namespace afd {

constexpr int kNarrowN = 16;                                    // columns of an MMA
constexpr int kNarrowMost = 64;                                 // columns of an expert, in tiles

// S: inputs of a step.  Warpgroups, TMEM columns of a warpgroup's accumulators, ring stages, shared memory.
template <int S>
struct Narrow {
  static constexpr int kWgs = S == 256 ? 3 : 4, kThreads = kWgs * 128;
  static constexpr int kAccs = S == 256 ? 32 : 64;
  static constexpr int kStages = S == 256 ? 3 : 4;
  static constexpr int kACols = S / 2;                          // TMEM columns of the A operand
  static constexpr int kStep = 128 * S / 2;                     // bytes of a step's codes
  static constexpr int kTile = kNarrowN * S * 2;                // of its tokens
  static constexpr int kTokens = 2 * kTile;                     // two tiles; the join's buffer too
  static constexpr int kSmem = 1024 + kWgs * (kStages * kStep + kTokens) + 2 * kThreads * kWindowBytes;
  static_assert(kNarrowN * 128 * 4 <= kTokens, "the join's partial sums fit");
  static_assert(kWgs * (kACols + kAccs) <= 512, "TMEM has 512 columns");
};

// The codes as boxes of S / 2 bytes of 64, 32 and 16 rows: half the rows of a unit.
struct NarrowMaps {
  CUtensorMap map[3];
};

// Rows of a unit and warpgroups that share one (all or one).
struct NarrowShape {
  int log_rows, split;
};

// The shape of the least cost: a team takes ceil(units / teams) units of ceil(steps / split) steps and
// about one more for its first loads and the join.  Fewer rows are more scales, tokens and TMA boxes a step: counted
// as equal, 18 experts of 3840 x 1024 took units of 64 rows and 59 us, where 128 rows take 50.  R rows leave R / 8 columns; tiles: token tiles of all experts at 16,
// 8 and 4 columns.  A lane works out each candidate: one after another the divisions took 2 us of a kernel's
// start.
__device__ __forceinline__ NarrowShape choose_narrow(const int (&tiles)[3], int outs, int log_pair, int slices, int ctas, int wgs) {
  const int lane = threadIdx.x & 31, lr = 7 - (lane >> 1), split = lane & 1 ? wgs : 1;
  unsigned cost = 0xffffffffu;
  if (lane < 6) {
    const unsigned units = (lane < 2 ? tiles[0] : lane < 4 ? tiles[1] : tiles[2]) * (static_cast<unsigned>(outs + (1 << (lr - log_pair)) - 1) >> (lr - log_pair));
    const unsigned steps = static_cast<unsigned>(slices + (128 >> lr) - 1) >> (7 - lr);
    const unsigned teams = ctas * (split == 1 ? wgs : 1);
    // up to 2^24 in floats, which is enough for a choice, with room for the candidate below it
    const float step = lane < 2 ? 10.f : lane < 4 ? 14.f : 18.f;
    const float c = static_cast<float>((units + teams - 1) / teams) *
                    (static_cast<float>(split == 1 ? steps : (steps + wgs - 1) / static_cast<unsigned>(wgs)) * step + 8.f);
    cost = (__float_as_uint(c) & ~31u) | lane;
  }
  const int best = __reduce_min_sync(0xffffffffu, cost) & 31;
  return NarrowShape{7 - (best >> 1), best & 1 ? wgs : 1};
}

// 32 lanes x C columns, waited for.
template <int C>
__device__ __forceinline__ void tmem_read(uint32_t taddr, uint32_t (&r)[C]) {
  static_assert(C == 4 || C == 8 || C == 16, "columns");
  if constexpr (C == 16) {
    tmem_ld16(taddr, r);
    tmem_ld_wait(r);
  } else if constexpr (C == 8) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n\ttcgen05.wait::ld.sync.aligned;"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr)
                 : "memory");
  } else {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];\n\ttcgen05.wait::ld.sync.aligned;"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(taddr)
                 : "memory");
  }
}

// mbar_wait, recorded where it gives up; out of line, since most waits end at the first try.
__device__ __noinline__ void wait_longer(uint32_t bar, uint32_t parity, volatile int* abort, int* err) {
  if (!mbar_wait(bar, parity, abort)) {
    *abort = 1;
    atomicOr(err, kErrTimeout);
  }
}

// PARTS: groups of a slice of S inputs with a scale each (1, 2 or 4).
template <int MODE, int PARTS, int S>
__global__ void __launch_bounds__(Narrow<S>::kThreads, 1)
w4_narrow_kernel(const __grid_constant__ NarrowMaps codes, const W4Args a) {
  constexpr int kPlanes = MODE == kDown ? 2 : 1;
  constexpr int kLogPair = MODE == kGateUp ? 1 : 0;  // weight rows per output, as a power of two
  using L = Narrow<S>;
  constexpr int kWgs = L::kWgs, kThreads = L::kThreads, kStages = L::kStages, N = kNarrowN;
  constexpr int kPartK = S / PARTS, kPer = S / 16 / PARTS;  // inputs and K16 steps of a part
  static_assert(PARTS * N <= L::kAccs, "every part has an accumulator");
  extern __shared__ uint8_t smem_raw[];
  __shared__ UnitTables tb;                          // unit_base: token tiles of the experts before
  // of a token tile: its expert, and its number there * 256.  At most four tiles an expert with 16 columns, or
  // kNarrowMost columns in all, and one more an expert.
  __shared__ uint16_t tile_of[4 * kW4MaxExperts];
  __shared__ __align__(8) uint64_t bars[kWgs * (kStages + 1)];
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  // uniform over a warp, for the compiler too: an MMA with operands that it takes for per-thread values
  // is issued every 85 clocks, one with uniform operands every 15
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const bool leader = elect_one();                   // of its warp
  const int wg = warp >> 2, r = tid & 127;           // warpgroup; TMEM lane
  volatile int* abort = &abort_flag;

  // what needs no input: barriers and TMEM
  if (tid < kWgs * (kStages + 1)) {
    mbar_init(smem_u32(&bars[tid]), 1);
    fence_barrier_init();
  }
  if (tid == 0) abort_flag = 0;
  if (warp == 1) {
    tmem_alloc(smem_u32(&tmem_slot), 512);
    tmem_relinquish();
  }
  if (a.first) wait_dependency();  // else the call's first kernel has, before this one could start (W4Args::first)
  const int outs = MODE == kGateUp ? a.N / 2 : a.N, lane = tid & 31;
  const int slices = (a.K + S - 1) / S;
  int tiles[3];
  auto cols_of = [&](int rows) { return rows > a.most / kPlanes ? 0 : rows * kPlanes; };
  count_rows<-1>(a, cols_of, tb, tiles);
  const NarrowShape shape = choose_narrow(tiles, outs, kLogPair, slices, gridDim.x, kWgs);
  const int n_tiles = shape.log_rows == 7 ? tiles[0] : shape.log_rows == 6 ? tiles[1] : tiles[2];
  if (warp == 0) {
    auto tiles_of = [&](int rows) { return (cols_of(rows) + (1 << shape.log_rows) / 8 - 1) >> (shape.log_rows - 3); };
    base_units(a, tiles_of, tb);
    __syncwarp();
    for (int e = lane; e < a.E; e += 32)
      for (int at = tb.unit_base[e], t = 0; at < tb.unit_base[e + 1]; ++at, ++t) tile_of[at] = static_cast<uint16_t>(e | t << 8);
  }
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* const gbase = smem_raw + (base - smem_u32(smem_raw));
  constexpr int kRingOff = kWgs * L::kTokens, kWindowOff = kRingOff + kWgs * kStages * L::kStep;
  const uint32_t tokens = base + wg * L::kTokens;
  uint8_t* const tokens_at = gbase + wg * L::kTokens;
  const int ring_off = kRingOff + wg * kStages * L::kStep;
  const uint32_t full = smem_u32(&bars[wg * (kStages + 1)]), mma_bar = full + 8 * kStages;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // What follows allocates TMEM after this.  It must stay behind the wait above: a call's next kernel reads counts,
  // and rows, as soon as it starts, on the strength of that wait.
  launch_dependents();
  const uint32_t tmem = tmem_slot;
  if (n_tiles == 0) {
    wait_dependency();  // what follows may rely on the kernel before this one
    if (warp == 1) tmem_dealloc(tmem, 512);
    return;
  }
  const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;  // the warp's lane quarter
  const uint32_t tm_a = tmem + wg * L::kACols, tm_d = tmem + kWgs * L::kACols + wg * L::kAccs;
  const uint64_t desc0 = sw128_desc(tokens);
  constexpr uint32_t idesc = idesc_mn(128, N, false);

  const int KG = a.KG, cps = a.scale_f32 ? 4 : 2;
  const int split = shape.split;
  int it = 0, issued = 0;                            // steps of this group: taken, and under way

  auto wait = [&](uint32_t bar, uint32_t parity) {
    if (!mbar_try_wait(bar, parity)) wait_longer(bar, parity, abort, a.err);
  };

  auto run = [&](auto log_rows) {
    constexpr int LR = decltype(log_rows)::value, R = 1 << LR, C = R / 8;
    constexpr int kStack = 128 >> LR;                  // slices of a step
    constexpr int kOutRows = R >> kLogPair;            // outputs of a unit
    const int blocks = (outs + kOutRows - 1) / kOutRows;
    const int total = n_tiles * blocks;
    const int ksteps = (slices + kStack - 1) / kStack, per = split == 1 ? ksteps : (ksteps + kWgs - 1) / kWgs;
    const int sub = split == 1 ? 0 : wg, team = split == 1 ? wg : 0;
    const int steps = max(0, min(per, ksteps - sub * per));
    const int active = split == 1 ? 1 : (ksteps + per - 1) / per;  // groups of a team with a step
    const int teams = gridDim.x * (split == 1 ? kWgs : 1);
    const int u0 = team * gridDim.x + blockIdx.x;
    const int row = r & (R - 1), q = ((warp & 3) * 32) >> LR;  // row of the unit, slice of the step

    struct At {
      int e, first, m, row0;  // expert, first token row, tokens, first output
    };
    auto unit_of = [&](int u) {
      const int at = u / blocks, tile = tile_of[at];
      At t;
      t.e = tile & 255;
      t.first = tb.first[t.e] + (tile >> 8) * (C / kPlanes);
      t.m = min(C / kPlanes, tb.rows[t.e] - (tile >> 8) * (C / kPlanes));
      t.row0 = (u - at * blocks) * kOutRows;
      return t;
    };

    // ---- loads, by a lane of the group's second warp; one of the first issues the MMAs
    int lu = steps > 0 ? u0 : total, ls = 0, lrow = 0, lx = 0, lslot = 0;
    auto load_step = [&]() {
      if (lu >= total || *abort) return;
      if (ls == 0) {
        const At un = unit_of(lu);
        lrow = un.e * a.N + un.row0;
        lx = sub * per * kStack * (S / 2);
      }
      const uint32_t bar = full + 8 * lslot, dst = base + ring_off + lslot * L::kStep;
      mbar_arrive_expect_tx(bar, L::kStep);
#pragma unroll
      for (int i = 0; i < 2 * kStack; ++i)
        tma_load_2d(dst + i * (R / 2 * (S / 2)), &codes.map[7 - LR], bar, lx + (i >> 1) * (S / 2),
                    lrow + (i & 1) * (MODE == kGateUp ? outs : R / 2), kEvictNormal);
      lx += kStack * (S / 2);
      lslot = lslot + 1 == kStages ? 0 : lslot + 1;
      ++issued;
      if (++ls == steps) {
        ls = 0;
        lu += teams;
      }
    };
    if ((warp & 3) == 1 && leader)
      for (int i = 0; i < kStages; ++i) load_step();
    __syncwarp();

    // Row of the weights whose scales this thread applies, as the place of its first group; rows past
    // the end repeat the last one.
    auto scale_row = [&](const At& un) {
      int y = min(un.row0 + row, outs - 1);
      if (MODE == kGateUp) y = (row < kOutRows ? 0 : outs) + min(un.row0 + (row & (kOutRows - 1)), outs - 1);
      return (static_cast<size_t>(un.e) * a.N + y) * KG;
    };
    // a unit's scales and zero points, into L2 a unit ahead
    auto prefetch_scales = [&](int u) {
      if (u >= total) return;
      const size_t at = scale_row(unit_of(u));
      const uint8_t* sp = static_cast<const uint8_t*>(a.scale) + at * cps;
      for (int o = (sub * kStack + q) * 32; o < KG * cps; o += split * kStack * 32) prefetch_l2(sp + o);
      if (a.zero)
        for (int o = (sub * kStack + q) * 32; o < KG; o += split * kStack * 32) prefetch_l2(a.zero + at + o);
    };
    if (MODE == kDown) wait_dependency();

    // Tokens: a thread moves its piece of 8 inputs (kc) of rows n0 + kRows i of the tile, which are column
    // n % C of slice n / C; rows of columns that the unit has not are left as they are.  The SwiGLU rows are
    // in the codes' order already and go by cp.async; others go through registers, which put inputs i and
    // i + 4 side by side.
    constexpr bool kAsync = MODE == kDown;
    constexpr int kPieces = S / 8, kRows = 128 / kPieces, kMoves = N / kRows;
    const int kc = r & (kPieces - 1), n0 = r / kPieces;
    auto place_of = [&](int i) {
      const int n = n0 + i * kRows;
      return (kc >> 3) * (N * 128) + n * 128 + (((kc & 7) ^ (n & 7)) * 16);
    };
    // Scales and zero points come in windows of 16 bytes of scales, by cp.async to a place of the
    // thread's own; a thread per row is 32 lines a load, so one load for eight groups matters.
    // Rows of an odd length or start are read group by group.
    // Two windows of a thread: one in use, one on its way, asked for two steps ahead.  A commit group goes with
    // each step all the same, so that the waits count groups alike; a unit's last steps have empty ones.
    constexpr int kWindows = kThreads * 16, kZeros = 2 * kWindows, kZeroWindows = kThreads * 8;
    const uint32_t wsc = base + kWindowOff + tid * 16, wz = base + kWindowOff + kZeros + tid * 8;
    const uint8_t* const wat = gbase + kWindowOff + tid * 16;
    const uint8_t* const zat = gbase + kWindowOff + kZeros + tid * 8;
    const int wlog = a.scale_f32 ? 2 : 3, wmask = (1 << wlog) - 1;

    // this lane's row of a slot, at the place of its first piece; piece c is at ^ (c * 16)
    const uint32_t codes_at = base + ring_off + r * (S / 2) + (S == 256 ? r & 7 : (r >> 1) & 3) * 16;
    int slot = 0;
    uint32_t full_phase = 0, mma_phase = 0, buf = 0;
    for (int u = u0; u < total; u += teams) {
      const At un = unit_of(u);
      const int cols = un.m * kPlanes;
      const size_t srow = scale_row(un);
      float acc[C];
#pragma unroll
      for (int i = 0; i < C; ++i) acc[i] = 0.f;

      const __nv_bfloat16* src = a.x + static_cast<size_t>(un.first) * kPlanes * a.K + sub * per * kStack * S + kc * 8;
      int left = a.K - (sub * per * kStack * S + kc * 8);  // inputs from the piece of slice 0 to the end of its row
      [[maybe_unused]] uint4 v[kAsync ? 1 : kMoves];
      auto load_tokens = [&](uint32_t to) {
#pragma unroll
        for (int i = 0; i < kMoves; ++i) {
          const int n = n0 + i * kRows, c = n & (C - 1), off = (n / C) * S;
          if (c < cols) {
            const __nv_bfloat16* from = src + c * a.K + off;
            if constexpr (kAsync)
              cp_async16(tokens + to + place_of(i), left > off ? from : a.x, left > off);
            else
              v[i] = left > off ? __ldcg(reinterpret_cast<const uint4*>(from)) : make_uint4(0u, 0u, 0u, 0u);
          }
        }
        src += kStack * S;
        left -= kStack * S;
        if constexpr (kAsync) cp_async_commit();
      };
      int window = -1, which = 0;               // the window asked for last, and its place
      int place = 0, place_next = 0;            // of this step's window and the next one's
      int sk = (sub * per * kStack + q) * S;  // first input of the lane's slice
      // mine: a step of this group's share.  A window of the step after it would be in flight, with nothing that
      // waits for it, when the next unit's first one goes to the same place.
      auto load_window = [&](int k, bool mine) {
        if (mine && a.windows) {
          const int w = k >> (a.glog + wlog);
          if (w != window && k < a.K) {
            window = w;
            which ^= 1;
            const size_t at = srow + (static_cast<size_t>(w) << wlog);
            cp_async16(wsc + which * kWindows, static_cast<const uint8_t*>(a.scale) + at * cps);
            if (a.zero) {
              if (wlog == 3) cp_async8(wz + which * kZeroWindows, a.zero + at);
              else cp_async4(wz + which * kZeroWindows, a.zero + at);
            }
          }
        }
        cp_async_commit();
      };
      uint32_t next_sc[PARTS], next_z[PARTS];  // as they are in memory
      auto load_scales = [&](int k) {
        if (a.windows) return;
#pragma unroll
        for (int p = 0; p < PARTS; ++p) {
          const size_t at = srow + group_of(a, min(k + p * kPartK, a.K - 32) / 32);
          if (a.scale_f32) next_sc[p] = __ldg(static_cast<const unsigned*>(a.scale) + at);
          else next_sc[p] = __ldg(static_cast<const unsigned short*>(a.scale) + at);
          next_z[p] = 8u;
          if (a.zero) next_z[p] = __ldg(a.zero + at);
        }
      };
      float sc[PARTS], sc_before[PARTS];
      // the accumulators, once the step's MMAs are done
      auto collect = [&](const float (&scale)[PARTS]) {
        wait(mma_bar, mma_phase);
        mma_phase ^= 1;
        tc_fence_after();
        auto read = [&](auto columns) {
          constexpr int D = decltype(columns)::value;
#pragma unroll
          for (int p = 0; p < PARTS; ++p) {
            uint32_t d[D];
            tmem_read<D>(tm_d + lanes + p * N + q * C, d);
#pragma unroll
            for (int c = 0; c < D; ++c) acc[c] = fmaf(scale[p], __uint_as_float(d[c]), acc[c]);
          }
        };
        if (C > 4 && cols <= 4) read(std::integral_constant<int, 4>());
        else read(std::integral_constant<int, C>());
      };
      auto start = [&]() {
        tc_fence_before();
        group_barrier(1 + wg, 128);
        if ((warp & 3) == 0 && leader) {
          tc_fence_after();
          const uint64_t desc = desc0 + buf * (L::kTile >> 4);
#pragma unroll
          for (int ks = 0; ks < S / 16; ++ks)
            tc_mma_ts(tm_d + ks / kPer * N, tm_a + ks * 8, desc + (ks >> 2) * (N * 8) + (ks & 3) * 2, idesc, ks % kPer > 0);
          tc_commit(mma_bar);
        }
      };

      if (steps > 0) {
        load_window(sk, true);
        place = which;
        load_tokens(buf * L::kTile);
        load_scales(sk);
        load_window(sk + kStack * S, steps > 1);
        place_next = which;
      }
      prefetch_scales(u + teams);
#pragma unroll 1
      for (int s = 0; s < steps; ++s, ++it, sk += kStack * S) {
        // under way, the youngest last: (tokens of this step,) the next step's window
        cp_async_wait<kAsync ? 2 : 1>();
        uint32_t z[PARTS];
        if (a.windows) {
          const int at = (sk >> a.glog) & wmask;  // the parts' groups follow one another in it; a slice is inside or past the end as a whole
#pragma unroll
          for (int p = 0; p < PARTS; ++p) {
            sc[p] = a.scale_f32 ? reinterpret_cast<const float*>(wat + place * kWindows)[at + p]
                                : __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const unsigned short*>(wat + place * kWindows)[at + p]) << 16);
            z[p] = a.zero ? zat[place * kZeroWindows + at + p] : 8u;
            if (kStack > 1 && sk >= a.K) sc[p] = 0.f;
          }
        } else {
#pragma unroll
          for (int p = 0; p < PARTS; ++p) {
            sc[p] = __uint_as_float(a.scale_f32 ? next_sc[p] : next_sc[p] << 16);
            z[p] = next_z[p];
          }
        }
        wait(full + 8 * slot, full_phase);
        const uint32_t at = codes_at + slot * L::kStep;
        if (++slot == kStages) {
          slot = 0;
          full_phase ^= 1;
        }
        if (s > 0) collect(sc_before);  // the A operand is free again
        uint32_t c0 = 0, c1 = 0;
#pragma unroll
        for (int c = 0; c < S / 32; ++c) {
          const uint4 w = lds128(at ^ (c * 16));
          if (c % (S / 32 / PARTS) == 0) {
            const uint32_t b = ((z[c * PARTS / (S / 32)] & 15u) | 0x4300u) * 0x10001u;  // 128 + z
            c0 = fma_bf16x2(b, 0xBE80BE80u, 0x80008000u);                        // -(128 + z) / 4
            c1 = fma_bf16x2(b, 0xBE80BE80u, 0x42004200u);                        // -z / 4
          }
          uint32_t p[4][4];
          unpack_word(w.x, c0, c1, p[0]);
          unpack_word(w.y, c0, c1, p[1]);
          unpack_word(w.z, c0, c1, p[2]);
          unpack_word(w.w, c0, c1, p[3]);
          tmem_st16(tm_a + lanes + c * 16, p);
        }
        if constexpr (!kAsync) {
#pragma unroll
          for (int i = 0; i < kMoves; ++i)
            if (((n0 + i * kRows) & (C - 1)) < cols)
              *reinterpret_cast<uint4*>(tokens_at + buf * L::kTile + place_of(i)) =
                  make_uint4(__byte_perm(v[i].x, v[i].z, 0x5410), __byte_perm(v[i].x, v[i].z, 0x7632),
                             __byte_perm(v[i].y, v[i].w, 0x5410), __byte_perm(v[i].y, v[i].w, 0x7632));
        }
        if constexpr (kAsync) cp_async_wait<1>();
        tmem_st_wait();
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        start();
        if ((warp & 3) == 1 && leader) load_step();  // the ring's slot is read
        __syncwarp();
        if (s + 1 < steps) {
          load_scales(sk + kStack * S);
          load_tokens((buf ^ 1) * L::kTile);
          load_window(sk + 2 * kStack * S, s + 2 < steps);
          place = place_next;
          place_next = which;
        }
        buf ^= 1;
#pragma unroll
        for (int p = 0; p < PARTS; ++p) sc_before[p] = sc[p];
      }
      if (steps > 0) collect(sc_before);

      // ---- results
      if (split == 1 && kStack == 1 && MODE != kGateUp) {
        if (un.row0 + r < outs) {
#pragma unroll
          for (int c = 0; c < C; c += kPlanes) {
            const float sum = kPlanes == 2 ? acc[c] + acc[c + 1] : acc[c];
            if (c / kPlanes < un.m) store_out<MODE>(a, un.first + c / kPlanes, un.row0 + r, outs, sum * 4.f, 0.f);
          }
        }
        continue;
      }
      // partial sums to the group's token buffer, which its MMAs have read; joined in order of groups and slices
      float* to = reinterpret_cast<float*>(tokens_at);
#pragma unroll
      for (int c = 0; c < C; ++c)
        if (c < cols) to[c * 128 + r] = acc[c];
      group_barrier(1 + kWgs + team, split * 128);
      const float* part = reinterpret_cast<const float*>(gbase + (split == 1 ? wg : 0) * L::kTokens);
      auto sum = [&](int c, int y) {
        float t = 0.f;
#pragma unroll
        for (int w = 0; w < kWgs; ++w)
          if (w < active) {
#pragma unroll
            for (int l = 0; l < 128; l += R)
#pragma unroll
              for (int p = 0; p < kPlanes; ++p) t += part[w * (L::kTokens / 4) + (c * kPlanes + p) * 128 + l + y];
          }
        return t * 4.f;
      };
      for (int i = sub * 128 + r; i < un.m * kOutRows; i += split * 128) {
        const int tok = i / kOutRows, out = i & (kOutRows - 1);
        if (un.row0 + out < outs)
          store_out<MODE>(a, un.first + tok, un.row0 + out, outs, sum(tok, out), MODE == kGateUp ? sum(tok, kOutRows + out) : 0.f);
      }
      group_barrier(1 + kWgs + team, split * 128);
    }
  };
  if (shape.log_rows == 7) run(std::integral_constant<int, 7>());
  else if (shape.log_rows == 6) run(std::integral_constant<int, 6>());
  else run(std::integral_constant<int, 5>());

  // After a wait that gave up: the group's own copies in flight, with a limit, before shared memory goes.
  if ((warp & 3) == 1 && leader && *abort) {
    int none = 0;
    for (; it < issued; ++it) mbar_wait(full + 8 * (it % kStages), (it / kStages) & 1, &none);
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
