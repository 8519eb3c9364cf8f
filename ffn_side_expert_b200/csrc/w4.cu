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
// Both products run on the 5th-generation tensor cores with the unpacked weights as the A operand in TMEM:
// experts with few columns (tokens, or planes of tokens) in w4_narrow.cuh, the others in
// w4_wide.cuh.  A warp's mma.sync on codes unpacked in registers, tried first, was bound by the same
// unpacking with more instructions around it (one token's eight experts of H = 7168, I = 2048: 66 us
// against 60; 128 rows on 64 experts of 4096 x 1024: 143 against 101).
//
// At the HBM rate an SM gets 46 codes a clock, and its integer pipe does 64 lane operations; so the unpacking
// has to be short (what bounds each kernel stands there).  A word of eight codes takes nine instructions, five of
// them integer: one shift, four masks and four bf16x2 FMAs that take the zero point off
// (unpack_word).
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
constexpr int kSliceK = 128;       // inputs of a slice of K

struct W4Args {
  const void* scale;
  const uint8_t* zero;
  const __nv_bfloat16* x;   // [n_rows * planes][K]
  const int32_t* counts;    // [E], or nullptr: one expert, every row
  void* y;
  int E, N, K, G, KG, n_rows, scale_f32, y_f32;  // KG = K / G
  unsigned group_inv;       // ceil(2^32 / (G / 32)), 0 for groups of 32
  int glog;                 // log2 G, where windows says so
  int windows;              // groups of 2^i, rows of scales (and zero points) that whole 16-byte pieces cover
  // The call's first kernel waits for the stream's kernel before it and only then lets the next one start.  So a
  // later kernel of the call may read counts, and all but the down products the rows, and write results and
  // scratch, before its own wait; that one (at the start of kDown, else at the end) is for the kernel just before.
  int first;
  int most, above;          // w4_narrow.cuh: the experts with at most so many columns; w4_wide.cuh: with more than
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
// For shared memory that other proxies and warps write: not moved over barriers.
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}

// a & b | c
__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
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
    p[0] = fma_bf16x2(and_or(__byte_perm(w, 0, 0x4040), 0x00f0000fu, 0x00004300u), 0x7F003E80u, c);
    p[1] = fma_bf16x2(and_or(__byte_perm(w, 0, 0x4141), 0x00f0000fu, 0x00004300u), 0x7F003E80u, c);
    p[2] = fma_bf16x2(and_or(__byte_perm(w, 0, 0x4242), 0x00f0000fu, 0x00004300u), 0x7F003E80u, c);
    p[3] = fma_bf16x2(and_or(__byte_perm(w, 0, 0x4343), 0x00f0000fu, 0x00004300u), 0x7F003E80u, c);
  } else {
    const uint32_t s = w >> 8;
    p[0] = fma_bf16x2(and_or(w, 0x000f000fu, 0x43004300u), kQuarter, c0);
    p[1] = fma_bf16x2(w & 0x00f000f0u, k2to127, c1);
    p[2] = fma_bf16x2(and_or(s, 0x000f000fu, 0x43004300u), kQuarter, c0);
    p[3] = fma_bf16x2(s & 0x00f000f0u, k2to127, c1);
  }
}

// ---------------------------------------------------------------------- the product
struct UnitTables {
  int first[kW4MaxExperts], rows[kW4MaxExperts], unit_base[kW4MaxExperts + 1];
};

// Rows of every expert from counts, by every warp for itself, a lane for an expert; the first warp writes them down.
// Negative counts are flagged and taken as 0, rows past n_rows are flagged and cut off.  tiles: the token
// tiles of all experts with cols_of(rows) columns, at 16, 32 and 64 columns (STEP 1) or at 16, 8 and 4 (STEP -1).
// (Experts spread over the block, with its barriers, took a microsecond more of a kernel's start.  The code runs
// once, so its length counts too.)
template <int STEP, typename F>
__device__ __forceinline__ void count_rows(const W4Args& a, F cols_of, UnitTables& tb, int (&tiles)[3]) {
  const int lane = threadIdx.x & 31;
  int before = 0, n[3] = {0, 0, 0};
#pragma unroll 1
  for (int e0 = 0; e0 < a.E; e0 += 32) {
    const int e = e0 + lane;
    int c = e < a.E ? (a.counts ? a.counts[e] : a.n_rows) : 0;
    bool bad = c < 0 || c > a.n_rows;
    c = min(max(c, 0), a.n_rows);
    const int end = before + warp_incl_scan(c, lane);  // at most 256 * 2^22
    bad |= end > a.n_rows;
    const int first = min(end - c, a.n_rows), rows = min(c, a.n_rows - first);
    before = __shfl_sync(0xffffffffu, end, 31);
#pragma unroll
    for (int j = 0; j < 3; ++j) n[j] += (cols_of(rows) + (1 << (4 + j * STEP)) - 1) >> (4 + j * STEP);
    if (threadIdx.x < 32) {
      tb.first[e] = first;
      tb.rows[e] = rows;
      if (bad && blockIdx.x == 0) atomicOr(a.err, kErrBadOffsets);
    }
  }
#pragma unroll
  for (int j = 0; j < 3; ++j) tiles[j] = __reduce_add_sync(0xffffffffu, n[j]);
}

// Unit bases of every expert, by the first warp: units_of(rows) of an expert.
template <typename F>
__device__ __forceinline__ void base_units(const W4Args& a, F units_of, UnitTables& tb) {
  const int lane = threadIdx.x;
  __syncwarp();
  int before = 0;
  if (lane == 0) tb.unit_base[0] = 0;
#pragma unroll 1
  for (int e0 = 0; e0 < a.E; e0 += 32) {
    const int e = e0 + lane, units = units_of(tb.rows[e]);
    const int end = before + warp_incl_scan(units, lane);
    tb.unit_base[e + 1] = end;
    before = __shfl_sync(0xffffffffu, end, 31);
  }
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
    // a number that would round to an infinite high term is cut off to the last bf16: its low term has the rest
    const __nv_bfloat16 hi = fabsf(act) < 0x1.FFp127f ? __float2bfloat16_rn(act) : __float2bfloat16_rz(act);
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
#include "w4_narrow.cuh"

namespace afd {
namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int check_w4(const afd_ffn_w4* w, int32_t E) {
  if (!w || E < 1 || w->N < 1 || w->K < 32 || w->K % 32 != 0 || w->group < 32 || w->group % 32 != 0 ||
      w->K % w->group != 0)
    return AFD_ERR_INVALID_ARG;
  if (w->scale_dtype != AFD_DT_BF16 && w->scale_dtype != AFD_DT_F32) return AFD_ERR_INVALID_ARG;
  if (E > kW4MaxExperts || static_cast<long long>(E) * w->N > (1LL << 30) || w->K > (1 << 20)) return AFD_ERR_UNSUPPORTED;
  return AFD_OK;
}

// Units are counted in 32 bits.  w4_narrow.cuh: blocks of at least 16 outputs, for token tiles of at least 4
// columns: four of each expert with up to 16 columns, or of a call with up to 64 columns a full tile for each 4
// and one more an expert.  w4_wide.cuh: tiles of at least 8 tokens by 64 outputs.
bool units_fit(int n_rows, int E, int outs) {
  const long long narrow = std::max(4LL * E, 16LL + E) * (outs / 16 + 1);
  const long long wide = (static_cast<long long>(n_rows) / 8 + E) * (outs / 64 + 1);
  return narrow < (1LL << 31) - 65536 && wide < (1LL << 31) - 65536;
}

int check_w4_pointers(const afd_ffn_w4* w) {
  // scales and zero points are fetched in 4-byte words
  const uintptr_t mis = (reinterpret_cast<uintptr_t>(w->scale) | reinterpret_cast<uintptr_t>(w->zero)) & 3u;
  if (!w->codes || !w->scale || !aligned16(w->codes) || mis) return AFD_ERR_INVALID_ARG;
  return AFD_OK;
}

constexpr int kMaxDevices = 64;

// A kernel's launch on the current device, as the dependent of the stream's last one.
template <typename... Args>
cudaError_t launch_on_device(void (*kernel)(Args...), std::atomic<int>* sm_count, int threads, int smem, cudaStream_t s,
                             const Args&... args) {
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
  return launch_dependent(kernel, sms, threads, smem, s, args...);
}

template <int MODE, int PARTS>
cudaError_t launch_wide(const CUtensorMap& codes, const W4Args& a, cudaStream_t s) {
  static std::atomic<int> sm_count[kMaxDevices];
  return launch_on_device(w4_wide_kernel<MODE, PARTS>, sm_count, kWideThreads, kWideSmem, s, codes, a);
}

template <int MODE, int PARTS, int S>
cudaError_t launch_narrow(const NarrowMaps& codes, const W4Args& a, cudaStream_t s) {
  static std::atomic<int> sm_count[kMaxDevices];
  return launch_on_device(w4_narrow_kernel<MODE, PARTS, S>, sm_count, Narrow<S>::kThreads, Narrow<S>::kSmem, s, codes, a);
}

// One product: the experts with few rows, then those with more.  Only a call that can have such
// rows launches a kernel for them.  after: the product reads what the stream's last kernel writes.
template <int MODE>
int launch_w4(const afd_ffn_w4& w, int E, const void* x, const int32_t* counts, int n_rows, void* y, int y_f32, int* err,
              bool after, cudaStream_t s) {
  constexpr int kPlanes = MODE == kDown ? 2 : 1;
  W4Args a{};
  a.scale = w.scale;
  a.zero = w.zero;
  a.x = static_cast<const __nv_bfloat16*>(x);
  a.counts = counts;
  a.y = y;
  a.E = E; a.N = w.N; a.K = w.K; a.G = w.group; a.KG = w.K / w.group; a.n_rows = n_rows;
  a.scale_f32 = w.scale_dtype == AFD_DT_F32;
  a.y_f32 = y_f32;
  const unsigned q = w.group / 32;
  a.group_inv = q == 1 ? 0u : static_cast<unsigned>(((1ull << 32) + q - 1) / q);
  // groups that 16 bytes of scales hold; a slice's groups lie in one such piece where slices and groups nest
  const int piece = a.scale_f32 ? 4 : 8;
  a.windows = a.K / a.G % piece == 0 && (w.group & (w.group - 1)) == 0 && aligned16(w.scale) &&
              (reinterpret_cast<uintptr_t>(w.zero) & (piece - 1)) == 0;
  while (a.glog < 31 && 1 << (a.glog + 1) <= w.group) ++a.glog;
  a.err = err;
  a.first = !after;
  // One kernel or two.  Up to 16 columns are one tile of w4_narrow.cuh.  A second kernel takes 4 to 5 us to
  // start, in which 32 MB of codes stream.  So a few more columns, spread over several experts, go there as
  // further tiles (12 rows on 32 experts of 1664 x 512: 13.6 us, 15.5 us with a second kernel; 32 rows on 8
  // experts of 2048 x 1024: 15.4 and 18.8 us evenly, 15.6 and 18.2 us all on one).  Small weights go to
  // w4_wide.cuh alone (16 rows on 2 experts of 2048 x 1024, the product of K 1024 there: 13.6 us, 16.0 us as
  // tiles), unless K is long, which units of few rows split better (16 rows on each of 8 experts of 256 x 512:
  // 26 us with two a product, 17 us with one).
  const long long columns = static_cast<long long>(n_rows) * kPlanes;
  const bool light = static_cast<long long>(E) * w.N * (w.K / 2) <= 32 << 20 && w.K <= 1024;
  const bool more = columns > (!counts || (light && E < 4) ? kNarrowN : E < 4 ? 2 * kNarrowN : kNarrowMost);
  const bool small = more && light;
  a.most = more ? kNarrowN : kNarrowMost;
  a.above = small ? 0 : kNarrowN;
  const uint64_t row_bytes = w.K / 2, rows = static_cast<uint64_t>(E) * w.N;
  cudaError_t e = cudaSuccess;
  if (!more || (counts && !small)) {
    const bool wide = w.group % 128 == 0;  // steps of 256 inputs
    NarrowMaps maps;
    for (int i = 0; i < 3; ++i)
      if (!encode_byte_rows(&maps.map[i], w.codes, row_bytes, rows, wide ? 128 : 64, 64 >> i)) return AFD_ERR_NO_DEVICE;
    e = w.group % 256 == 0  ? launch_narrow<MODE, 1, 256>(maps, a, s)
        : wide              ? launch_narrow<MODE, 2, 256>(maps, a, s)
        : w.group % 64 == 0 ? launch_narrow<MODE, 2, 128>(maps, a, s)
                            : launch_narrow<MODE, 4, 128>(maps, a, s);
    a.first = 0;
  }
  if (more && e == cudaSuccess) {
    CUtensorMap map;
    if (!encode_byte_rows(&map, w.codes, row_bytes, rows, kSliceK / 2, kWideRows / 2)) return AFD_ERR_NO_DEVICE;
    e = w.group % 128 == 0  ? launch_wide<MODE, 1>(map, a, s)
        : w.group % 64 == 0 ? launch_wide<MODE, 2>(map, a, s)
                            : launch_wide<MODE, 4>(map, a, s);
  }
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
