// mx_attention_tile.cu -- attention over the FP4 cache for many query rows (prompt chunks, trees of
// drafted tokens) on the fifth-generation tensor cores.
//
// The formulas are those of mx_cache_attention.cu.  With 128 query rows and more per key/value head the
// products dominate: 4 D multiply-adds per row and position against 1 + 2 / N bytes per position and
// dimension.  So K and V are dequantized once per chunk of 128 positions into shared memory (f16,
// exact) and serve TILES x 128 rows; scores and outputs stay in tensor memory.
//
// One thread block per SM, whose warps have one job each:
//   * 4 warps per 128-row tile: load and scale the queries (f16, 128-byte-swizzled shared memory);
//     then per chunk, one row per thread: read the scores from tensor memory, mask, weights
//     p = 2^(s c - m c + 7), running sum, write p as f16 over the scores; scale the outputs when the
//     maximum moves (by more than 2^8: weights may be up to 2^15); at the end read the outputs;
//   * 1 warp: brings codes and scales into a ring in shared memory (16-byte asynchronous copies; bulk
//     copies of the 64- to 1024-byte runs that a page holds took 1.4 times as long without the other
//     warps' work);
//   * 2 warps: a chunk's keys, one position per thread, into the K-major B operand of q K^T;
//   * 4 warps: its values (two of them every other half), 8 positions x D / 8 values per thread,
//     transposed into the K-major (along the positions) B operand of p V: two positions' codes are
//     interleaved as nibbles, so that a conversion gives f16 pairs along the positions and no data moves
//     between threads;
//   * 1 warp, one thread: issues the products.  Two tiles take turns: while one tile's weights are
//     computed, the tensor cores work on the other's.  p comes from tensor memory (A operand), half a
//     chunk at a time.
// Keys, values and codes move in halves of a chunk.  Tensor memory per tile: 128 columns of scores
// (weights overlay them), D columns of outputs.  (Two buffers of 64 columns would let a tile's scores run
// ahead of its weights, but products 64 columns wide take as long as those 128 wide: for the case below
// 1164 us when 128 columns took 1067.)
//
// What bounds it: 2048 prompt tokens over 16384 positions, 64 heads on 8 of 128, take 964 us at 1965 MHz,
// 1.07 PFLOP/s or 0.64 of the measured bf16 burst peak (1040 us at the 1825 MHz that the power cap leaves
// of it after a second, 0.69 of the peak measured that way); the tensor pipes, the exponentials' unit and
// the issue slots are busy half of it each.  Many rows over short sequences are bound by what
// a piece costs besides its chunks (queries in, outputs out, the first scores and the last outputs alone):
// 383 tokens of 4 sequences of up to 498 positions, 128 heads on 8, take 99 us; their bytes, 16.
//
// Every wait is bounded (mbar_wait below): a block that gives up says so in a device counter
// (mx_matmul_gave_up), lets its issued products finish, frees its tensor memory and returns; blocks do
// not wait for one another.
#include <atomic>

#include "mx_attention.cuh"
#include "mx_launch.h"
#include "mx_tc.cuh"

namespace mxk {
namespace attn {

__device__ unsigned int g_tile_gave_up;

namespace {

constexpr int kChunk = 128, kHalf = 64;  // positions per chunk, and per step of its loads
constexpr int kKeyWarps = 2, kValueWarps = 4;
constexpr uint32_t kPolls = 1u << 20;

template <int D, int TILES>
struct Tile {
  static constexpr int kRows = 128 * TILES;
  // Cut::start, in chunks (383 tokens of 4 sequences of up to 498 positions, 128 heads on 8 of 128: with 1,
  // 2, 3, 5 chunks 122, 109, 99, 101 us; a chunk of head_dim 256 takes longer, 914 tokens of 3 sequences,
  // 64 heads on 8: 304, 298, 315, 321 us)
  static constexpr int kStart = D == 256 ? 2 : 3;
  static constexpr int kStages = D == 256 ? 2 : 4;       // of half a chunk
  static constexpr int kQ = 128 * D * 2;                // bytes of one tile's queries
  static constexpr int kK = kHalf * D * 2;              // bytes of half a chunk's keys (and values)
  // ring of codes and scales: keys, values (8 positions at a time, 16 bytes apart, so that the threads
  // of 8 runs of 8 positions read different banks), their scales (at most one per 16 values)
  static constexpr int kRing = D == 256 ? 1 : 3;
  static constexpr int kOctet = 8 * (D / 2) + 16;
  static constexpr int kRawV = kHalf * (D / 2), kRawKS = kRawV + kHalf / 8 * kOctet,
                       kRawVS = kRawKS + kHalf * (D / 16), kRaw = kRawVS + kHalf * (D / 16);
  static constexpr int kSmem = TILES * kQ + 2 * kStages * kK + kRing * kRaw + 1024;
  static_assert(kSmem <= 230000, "shared memory");
  static constexpr int kThreads = 128 * (TILES + 2);
  static constexpr uint32_t kScoreCol = 0, kOutCol = kChunk * TILES;
  static_assert(kOutCol + TILES * D <= 512, "tensor memory");
  // Instruction descriptors of kind::f16: float32 accumulator (bits 4..5 = 1), A and B f16, K-major,
  // N / 8 in bits 17..22, M / 16 in bits 24..28.
  static constexpr uint32_t kIdescS = (1u << 4) | ((uint32_t)(kChunk >> 3) << 17) | (8u << 24);
  static constexpr uint32_t kIdescO = (1u << 4) | ((uint32_t)(D >> 3) << 17) | (8u << 24);
};

// True once the barrier's phase with this parity has completed; false after kPolls polls, or once
// another warp of the block has given up.  SLEEP_NS: between polls of waits that are not urgent.
template <int SLEEP_NS = 0>
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, volatile int* gave_up) {
#pragma unroll 1
  for (uint32_t i = 0; i < kPolls; ++i) {
    if (SLEEP_NS > 0 && i > 0) __nanosleep(SLEEP_NS);
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    if (ok) return true;
    if ((i & 255u) == 255u && *gave_up) return false;
  }
  *gave_up = 1;
  return false;
}

// True in one lane of the warp, which is converged.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

// Shared-memory operands are named by the low word of their descriptor (desc_sw128): the high word is
// the same for all of them, and the fewer registers an issue has to move, the faster it is.
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_low(uint32_t addr) { return (addr >> 4) | (1u << 16); }
// d (+)= a b with a in shared memory, or in tensor memory (f16 pairs).
template <bool ADD>
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
      "mov.b64 da, {%1, %4};\n\tmov.b64 db, {%2, %4};\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "n"(kDescHigh), "n"(ADD ? 1 : 0)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 db;\n\t"
      "mov.b64 db, {%2, %4};\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "n"(kDescHigh), "r"((uint32_t)add)
      : "memory");
}
__device__ __forceinline__ void tc_load16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15}, [%16];\n\ttcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tc_store16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// 32 columns of this warp's lanes, complete only after tc_wait_load.
__device__ __forceinline__ void tc_load32_async(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, "
      "%30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
// (the registers pass through, so that no use of them moves in front of the wait)
template <int N>
__device__ __forceinline__ void tc_wait_load(uint32_t (&r)[N]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}
__device__ __forceinline__ void tc_wait_store() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// Two scale codes x, y -> f16 pair (x, y) 2^-kScaleShift.  E4M3 by the hardware's conversion; UE5M3 by
// value (two scales serve 32 or more codes here).
template <int FMT>
__device__ __forceinline__ uint32_t scale_pair(uint32_t x, uint32_t y) {
  if constexpr (FMT == kE4M3) {
    uint32_t d;
    asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}"
        : "=r"(d) : "r"(__byte_perm(x, y, 0x0040)));
    return d;
  } else {
    return pack_f16x2(scale_value((int)x, FMT) * 0x1p-4f, scale_value((int)y, FMT) * 0x1p-4f);
  }
}

// What the warps need of the piece that a walk is at.
struct PieceOf {
  int64_t b;
  int h, rt, c0, chunks, end;
  __device__ __forceinline__ PieceOf() {}
  __device__ __forceinline__ explicit PieceOf(const Walk& w)
      : b(w.b), h(w.h), rt(w.rt), c0(w.c0), chunks(w.c1 - w.c0), end(w.end) {}
};

template <int D, int TILES, int FMT>
__global__ void __launch_bounds__(Tile<D, TILES>::kThreads, 1)
    k_attention_tile(const __grid_constant__ AttnArgs a) {
  using T = Tile<D, TILES>;
  constexpr int S = T::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const uint32_t s_q = smem_u32(smem), s_k = s_q + TILES * T::kQ, s_v = s_k + S * T::kK,
                 s_raw = s_v + S * T::kK;
  constexpr int R = T::kRing;
  __shared__ uint64_t bars[10 + 4 * S + 2 * R + 1];
  __shared__ uint32_t tmem_slot;
  __shared__ int s_gave_up;
  __shared__ int64_t s_scan[T::kThreads / 32];
  __shared__ Share s_share;
  __shared__ Walk s_walk[T::kThreads / 32];
  volatile int* gave_up = &s_gave_up;
  auto bar = [&](int i) { return smem_u32(bars + i); };
  // barriers: per tile, queries in place, scores done, weights in place (by halves), outputs done; per
  // stage (a chunk), keys in place, keys and values read, per half of it, values in place; per place of
  // the ring, codes in place and read.  (A wait by parity is sound where the phase before the awaited one
  // is known to be over, and the one behind it cannot end before the wait does.)
  auto q_full = [&](int t) { return bar(t); };
  auto o_full = [&](int t) { return bar(2 + t); };
  auto s_full = [&](int t) { return bar(4 + t); };
  auto p_full = [&](int t, int half) { return bar(6 + 2 * t + half); };
  auto k_full = [&](int s) { return bar(10 + s); };
  auto k_empty = [&](int s) { return bar(10 + S + s); };
  auto v_empty = [&](int s) { return bar(10 + 2 * S + s); };
  auto v_full = [&](int half) { return bar(10 + 3 * S + half); };
  auto raw_full = [&](int r) { return bar(10 + 4 * S + r); };
  auto raw_empty = [&](int r) { return bar(10 + 4 * S + R + r); };
  const uint32_t done = bar(10 + 4 * S + 2 * R);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int group = a.heads / a.c.kv_heads, ctas = gridDim.x, cta = blockIdx.x;
  if (threadIdx.x == 0) {
    for (int t = 0; t < 2; ++t) {
      mbar_init(q_full(t), 4);
      mbar_init(o_full(t), 1);
      mbar_init(s_full(t), 1);
      for (int half = 0; half < 2; ++half) mbar_init(p_full(t, half), 4);
    }
    for (int s = 0; s < S; ++s) {
      mbar_init(k_full(s), 2 * kKeyWarps);  // (by halves)
      mbar_init(k_empty(s), 1);
      mbar_init(v_full(s), kValueWarps / 2);
      mbar_init(v_empty(s), 1);
    }
    for (int r = 0; r < R; ++r) {
      mbar_init(raw_full(r), 32);
      mbar_init(raw_empty(r), kKeyWarps + kValueWarps);
    }
    mbar_init(done, 1);
    s_gave_up = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&tmem_slot)),
                 "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  griddep_wait();
  griddep_launch_next();
  const Cut cut{T::kRows, group, kChunk, T::kStart};
  find_share<T::kThreads>(a, cut, cta, ctas, s_scan, &s_share);
  // The warp's walk is kept in shared memory (registers are short) and moved on by one lane.
  Walk& walk = s_walk[warp];
  auto first_piece = [&] {
    int any = 0;
    if (lane == 0) any = walk.begin(a, cut, s_share);
    __syncwarp();
    any = __shfl_sync(0xffffffffu, any, 0);
    return any != 0;
  };
  auto next_piece = [&] {
    int any = 0;
    __syncwarp();
    if (lane == 0) any = walk.next(a, cut);
    __syncwarp();
    any = __shfl_sync(0xffffffffu, any, 0);
    return any != 0;
  };
  bool more = first_piece();
  int n = 0, piece = 0;  // chunks and pieces so far

  if (warp < 4 * TILES) {
    // ---------------- softmax: one query row per thread ----------------
    const int tile = warp >> 2, r = 32 * (warp & 3) + lane;
    const uint32_t t_lane = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t t_s = tmem + T::kScoreCol + kChunk * tile + t_lane;
    const uint32_t t_o = tmem + T::kOutCol + D * tile + t_lane;
    const float gv = fp16_bits_to_float(a.c.g_bits[1]) * (float)(1 << kScaleShift<FMT>);
    // The warp's 32 rows in the queries' place, 2 D bytes each: 16-byte piece i of row rr.  kLanes lanes
    // move a row to or from global memory, kTogether rows at a time.
    constexpr int kLanes = D / 8, kTogether = 32 / kLanes;
    const int piece_of = lane % kLanes;
    const uint32_t q_rows = s_q + tile * T::kQ + (uint32_t)(warp & 3) * 4096u;
    auto own_rows = [&](int rr, int i) {
      return q_rows + (uint32_t)(i >> 3) * 16384u + (uint32_t)rr * 128u + (uint32_t)((i ^ rr) & 7) * 16u;
    };
    if (threadIdx.x == 0) reinterpret_cast<Record*>(a.workspace)[cta].last = -1;
    while (more) {
      const PieceOf k(walk);
      const Seq seq = walk.seq;
      const int rows = seq.count * group, row = k.rt * T::kRows + 128 * tile + r;
      if (TILES > 1 && rows - k.rt * T::kRows <= 128 * tile) {  // no rows here (tile 0 always has some)
        more = next_piece();
        continue;
      }
      const bool in = row < rows;
      const int t = in ? row / group : 0, head = k.h * group + (in ? row % group : 0);
      float mult;
      {
        // the row times a power of two that brings its largest magnitude to [2^14, 2^15), as f16.  D / 8
        // lanes copy a row together into its place, where the lane whose row it is scales it.  (Rolled
        // up, like all that runs once a piece: what has to come into the instruction caches costs more
        // than it does.)
        const int64_t off = row_offset(a.q, k.b, t, head);
#pragma unroll 2
        for (int x = 0; x < kLanes; ++x) {
          const int rr = x * kTogether + lane / kLanes;
          const int64_t at = __shfl_sync(0xffffffffu, off, rr);
          const bool there = row - lane + rr < rows && a.scale != 0.0f;
          cp_async16(own_rows(rr, piece_of), static_cast<const uint16_t*>(a.q.p) + (there ? at + 8 * piece_of : 0),
                     there ? 16 : 0);
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncwarp();
        uint32_t mx = 0;
#pragma unroll 4
        for (int i = 0; i < D / 8; ++i) {
          uint32_t v[4];
          lds<16>(own_rows(lane, i), v);
#pragma unroll
          for (int e = 0; e < 4; ++e) mx = max(mx, max(v[e] & 0x7FFFu, (v[e] >> 16) & 0x7FFFu));
        }
        const int f = mx == 0 || mx >= 0x7F80u ? 0 : 141 - max((int)(mx >> 7), 1);
        const int f1 = f / 2, f2 = f - f1;  // |f| may be 140: two steps
        const float s1 = __uint_as_float((uint32_t)(127 + f1) << 23);
        const float s2 = __uint_as_float((uint32_t)(127 + f2) << 23);
        const uint32_t flip = a.scale < 0.0f ? 0x80008000u : 0u;
#pragma unroll 2
        for (int i = 0; i < D / 8; ++i) {
          uint32_t v[4];
          lds<16>(own_rows(lane, i), v);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            v[e] = pack_f16x2(bf16lo(v[e]) * s1 * s2, bf16hi(v[e]) * s1 * s2) ^ flip;
          st_shared16(own_rows(lane, i), v[0], v[1], v[2], v[3]);
        }
        const float gk = fp16_bits_to_float(a.c.g_bits[0]) * (float)(1 << kScaleShift<FMT>);
        mult = (a.scale == 0.0f ? 1.0f : fabsf(a.scale) * gk * 1.4426950408889634f) *
               __uint_as_float((uint32_t)(127 - f1) << 23) * __uint_as_float((uint32_t)(127 - f2) << 23);
        mult = fminf(fmaxf(mult, 0x1p-126f), 0x1p126f);
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full(tile));

      const uint64_t word = in && a.tree ? a.tree[k.b * a.tokens + t] : 0;
      const int plain_end = min(k.end, seen_by_all(a, seq, (row - lane) / group));
      const int chunks = k.chunks;
      Maximum top;
      top.reset();
      float2 l = make_float2(0.0f, 0.0f);
      bool ok = true;
      // whether any position of the piece has no page (then its chunks look them up again, below)
      bool holes = false;
      {
        const int shift = a.c.page_shift;
        const int32_t* ids = a.table.pages + k.b * a.table.stride;
        const int stop = min(k.end, (k.c0 + chunks) * kChunk);
        for (int g = ((k.c0 * kChunk) >> shift) + lane; g << shift < stop; g += 32) {
          const int id = __ldg(ids + g);
          holes |= id < 0 || id >= a.c.pages;
        }
        holes = __any_sync(0xffffffffu, holes);
      }
      // chunks before this one need no mask
      const int plain = holes ? 0 : plain_end / kChunk - k.c0;
#pragma unroll 1
      for (int j = 0; j < chunks; ++j) {
        ok = mbar_wait(s_full(tile), (n + j) & 1, gave_up);
        if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
        tc_fence_after();
        if (j >= plain) {
          const int p = (k.c0 + j) * kChunk;
          // which 16-position groups of the chunk have a page
          bool page = true;
          if (holes && lane < kChunk / 16 && p + 16 * lane < k.end)
            page = a.table.slot(a.c, k.b, p + 16 * lane) >= 0;
          const uint32_t pages = __ballot_sync(0xffffffffu, page);
          // bit i of seen(c): whether this row sees position p + 32 c + i
          auto seen = [&](int c) -> uint32_t {
            const int first = p + 32 * c;
            auto below = [](int x) { return x >= 32 ? ~0u : x <= 0 ? 0u : (1u << x) - 1u; };
            uint32_t w = below(k.end - first);
            if (a.tree) {
              const int j0 = first - seq.base;  // the group's first position among the new tokens
              const uint64_t have = seq.count >= 64 ? ~0ull : (1ull << seq.count) - 1ull;
              const uint64_t v = word & have;
              w &= j0 >= 64 ? 0u : j0 >= 0 ? (uint32_t)(v >> j0)
                   : j0 <= -32 ? ~0u : ((uint32_t)(v << -j0) | below(-j0));
            } else {
              w &= below(seq.base + t + 1 - first);
            }
            return w & (((pages >> (2 * c)) & 1 ? 0xFFFFu : 0u) |
                        ((pages >> (2 * c + 1)) & 1 ? 0xFFFF0000u : 0u));
          };
          // boundary chunks (few): the scores that this row does not see become -infinity in place
#pragma unroll 1
          for (int c = 0; c < kChunk / 16; ++c) {
            uint32_t x[16];
            tc_load16(t_s + 16 * c, x);
            const uint32_t w = seen(c >> 1) >> (16 * (c & 1));
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (!((w >> i) & 1)) x[i] = 0xFF800000u;
            __syncwarp();
            tc_store16(t_s + 16 * c, x);
          }
          tc_wait_store();
        }
        // ---- the chunk's maximum
        float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          uint32_t v[64];
          tc_load32_async(t_s + 64 * h, v);
          tc_load32_async(t_s + 64 * h + 32, v + 32);
          tc_wait_load(v);
#pragma unroll
          for (int i = 0; i < 64; i += 8)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              mx4[e] =
                  fmaxf(fmaxf(mx4[e], __uint_as_float(v[i + 2 * e])), __uint_as_float(v[i + 2 * e + 1]));
        }
        const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
        const bool grew = mx > top.lim;
        if (__any_sync(0xffffffffu, grew)) {
          float alpha = 1.0f;
          if (grew) {
            const float m = fmaxf(mx, top.m);
            alpha = top.m == -INFINITY ? 0.0f : ex2((top.m - m) * mult);
            top.set(m, mult);
            l.x *= alpha;
            l.y *= alpha;
          }
          __syncwarp();
          // The outputs so far times alpha (the scores are done, so the products into the outputs issued
          // before them are too); in front of them, if there are far rows, the scores less the maximum.
          const bool far = top.far(mult);
          const float sub = far ? top.m : 0.0f;
          const bool scores = __any_sync(0xffffffffu, far);
#pragma unroll 1
          for (int c = scores ? -kChunk / 16 : 0; c < (j > 0 ? D / 16 : 0); ++c) {
            const uint32_t at = c < 0 ? t_s + kChunk + 16 * c : t_o + 16 * c;
            const float f = c < 0 ? 1.0f : alpha, less = c < 0 ? sub : 0.0f;
            uint32_t x[16];
            tc_load16(at, x);
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] = __float_as_uint(fmaf(__uint_as_float(x[i]), f, -less));
            tc_store16(at, x);
          }
          tc_wait_store();
        }
        __syncwarp();
        // ---- weights: f16 pairs over the scores.  (Rolled up: unrolled, the warps' different code keeps
        // missing the instruction caches.)
        auto weights = [&](int c, const uint32_t* x) {
          uint32_t w[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float2 e = __ffma2_rn(make_float2(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1])),
                                  make_float2(mult, mult), make_float2(-top.mu, -top.mu));
            e = make_float2(ex2(e.x), ex2(e.y));
            l = __fadd2_rn(l, e);
            w[i] = pack_f16x2(e.x, e.y);
          }
          tc_store16(t_s + 16 * c, w);
        };
        uint32_t v[32], u[32];
        tc_load32_async(t_s, v);
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          tc_wait_load(v);
          tc_load32_async(t_s + 64 * half + 32, u);
          weights(2 * half, v);
          tc_wait_load(u);
          if (half == 0) tc_load32_async(t_s + 64, v);
          weights(2 * half + 1, u);
          tc_wait_store();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(p_full(tile, half));
        }
      }
      if (!ok) break;
      ok = mbar_wait(o_full(tile), piece & 1, gave_up);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after();
      const float sum = l.x + l.y;
      const bool whole = walk.whole();
      float* part = partial(a, ctas, T::kRows, D, 2 * cta + (k.c0 == 0));
      const float f = whole ? (sum == 0.0f ? 0.0f : gv / sum) : 1.0f;
      const int pr = 128 * tile + r;
      // The outputs (bf16), or D / 2 of a piece's (float32) at a time, go through the place of the
      // queries, which the products have read, so that rows leave as a whole.
      const int64_t off = row_offset(a.out, k.b, t, head);
#pragma unroll 1
      for (int pass = 0; pass < (whole ? 1 : 2); ++pass) {
#pragma unroll 1
        for (int c = 0; c < D / 16; c += whole ? 1 : 2) {
          uint32_t x[16];
          tc_load16(t_o + 16 * (whole ? c : (D / 32) * pass + (c >> 1)), x);
          if (whole) {
            uint32_t y[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
              y[i] = pack_bf16x2(__uint_as_float(x[2 * i]) * f, __uint_as_float(x[2 * i + 1]) * f);
            st_shared16(own_rows(lane, 2 * c), y[0], y[1], y[2], y[3]);
            st_shared16(own_rows(lane, 2 * c + 1), y[4], y[5], y[6], y[7]);
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              st_shared16(own_rows(lane, 2 * c + i), x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
          }
        }
        __syncwarp();
#pragma unroll 4
        for (int x = 0; x < kLanes; ++x) {
          const int rr = x * kTogether + lane / kLanes;
          const int64_t at = __shfl_sync(0xffffffffu, off, rr);
          uint32_t v[4];
          lds<16>(own_rows(rr, piece_of), v);
          if (row - lane + rr < rows) {
            char* dst = whole ? static_cast<char*>(a.out.p) + 2 * at
                              : reinterpret_cast<char*>(part + 2 * T::kRows +
                                                        (size_t)(pr - lane + rr) * D + (D / 2) * pass);
            reinterpret_cast<uint4*>(dst)[piece_of] = make_uint4(v[0], v[1], v[2], v[3]);
          }
        }
        __syncwarp();
      }
      if (in) {
        if (whole) {
          if (a.lse) a.lse[(k.b * a.tokens + t) * a.heads + head] = log_sum(top.log2(mult), sum);
        } else {
          part[pr] = top.log2(mult);
          part[T::kRows + pr] = sum;
        }
      }
      if (threadIdx.x == 0 && k.c0 == 0 && !whole)
        reinterpret_cast<Record*>(a.workspace)[cta] = {
            k.b, k.h, k.rt, block_of(walk.u0 + walk.n + T::kStart - 1, s_share),
            min(T::kRows, rows - k.rt * T::kRows)};
      tc_fence_before();
      n += chunks;
      ++piece;
      more = next_piece();
    }
  } else {
    const int log_block = a.c.log_block, log_sb = log2_of(D) - log_block;
    PieceOf k;
    if (warp < 4 * TILES + kValueWarps) {
    // ---------------- values: 8 positions x D / 8 values per thread ----------------
    const int w4 = warp - 4 * TILES;
    const int turn = w4 >> 1;                            // these two warps take every other half
    const int oct = lane & 7;                            // positions 8 oct ..
    const int run = (lane >> 3) + 4 * (w4 & 1);          // values (D / 8) run ..
    constexpr int W = D / 64;                            // code words per position
    const uint32_t src = s_raw + T::kRawV + oct * T::kOctet + (D / 16) * run;
    const uint32_t src_s = s_raw + T::kRawVS + ((8 * oct) << log_sb) + (((D / 8) * run) >> log_block);
    while (more) {
      k = PieceOf(walk);
      const int halves = 2 * k.chunks;
      bool ok = true;
#pragma unroll 1
      for (int j = 0; j < halves; ++j) {
        // every half's codes are waited for, also the other warps': a place of the ring that came round
        // twice unseen could not be told from one that did not
        const int i = n + j, s = i % S, r = i % R;
        const bool ours = (i & 1) == turn;
        ok = mbar_wait<20>(raw_full(r), (i / R) & 1, gave_up);
        if (ok && ours && i >= S) ok = mbar_wait<20>(v_empty(s >> 1), ((i / S) + 1) & 1, gave_up);
        if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
        if (!ours) {
          if (lane == 0) mbar_arrive(raw_empty(r));
          continue;
        }
        uint32_t code[8][W], sc[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          lds<4 * W>(src + r * T::kRaw + e * (D / 2), code[e]);
          const uint32_t at = src_s + r * T::kRaw + (e << log_sb);
          sc[e] = W == 4 && log_block == 4 ? lds_u16(at) : lds_u8(at) * (W == 4 ? 0x101u : 1u);
        }
        // row d of the transposed tile: 128 bytes = 64 positions
        const uint32_t dst = s_v + s * T::kK;
#pragma unroll
        for (int e = 0; e < W; ++e) {
          uint32_t ev[4][4], od[4][4];  // [pair of positions][even / odd values 2 i, 2 i + 1]
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const uint32_t x = code[2 * q][e], y = code[2 * q + 1][e];
            const uint32_t f =
                W == 4 ? scale_pair<FMT>((sc[2 * q] >> (8 * (e >> 1))) & 0xFFu,
                                         (sc[2 * q + 1] >> (8 * (e >> 1))) & 0xFFu)
                       : scale_pair<FMT>(sc[2 * q], sc[2 * q + 1]);
            e2m1x8_to_f16((x & 0x0F0F0F0Fu) | ((y << 4) & 0xF0F0F0F0u), ev[q]);
            e2m1x8_to_f16(((x >> 4) & 0x0F0F0F0Fu) | (y & 0xF0F0F0F0u), od[q]);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              ev[q][u] = mul_f16x2(ev[q][u], f);
              od[q][u] = mul_f16x2(od[q][u], f);
            }
          }
          const uint32_t at = dst + (uint32_t)(W * run + e) * 1024u;
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            st_shared16(at + (2 * u) * 128u + (((uint32_t)oct ^ (2 * u)) << 4), ev[0][u], ev[1][u],
                        ev[2][u], ev[3][u]);
            st_shared16(at + (2 * u + 1) * 128u + (((uint32_t)oct ^ (2 * u + 1)) << 4), od[0][u],
                        od[1][u], od[2][u], od[3][u]);
          }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(v_full(s));
          mbar_arrive(raw_empty(r));  // (every lane has used what it read)
        }
      }
      if (!ok) break;
      n += halves;
      more = next_piece();
    }
    } else if (warp < 4 * TILES + kValueWarps + kKeyWarps) {
    // ---------------- keys: one position per thread ----------------
    const int pos = 32 * (warp - 4 * TILES - kValueWarps) + lane;
    const uint32_t src = s_raw + pos * (D / 2), src_s = s_raw + T::kRawKS + (pos << log_sb);
    const uint32_t dst = s_k + (uint32_t)(pos >> 3) * 1024u + (uint32_t)(pos & 7) * 128u;
    while (more) {
      k = PieceOf(walk);
      const int halves = 2 * k.chunks;
      bool ok = true;
#pragma unroll 1
      for (int j = 0; j < halves; ++j) {
        const int i = n + j, s = i % S, r = i % R;
        ok = mbar_wait<20>(raw_full(r), (i / R) & 1, gave_up);
        if (ok && i >= S) ok = mbar_wait<20>(k_empty(s >> 1), ((i / S) + 1) & 1, gave_up);
        if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
        // runs of 32 values; lanes start at different ones, so that they read different banks
        uint32_t w[D / 32][4], sc[D / 32];
#pragma unroll
        for (int q = 0; q < D / 32; ++q) {
          const uint32_t run = (q + (lane >> 1)) & (D / 32 - 1);
          lds<16>(src + r * T::kRaw + 16 * run, w[q]);
          const uint32_t at = src_s + r * T::kRaw + ((32 * run) >> log_block);
          sc[q] = log_block == 4 ? lds_u16(at) : lds_u8(at) * 0x101u;
        }
#pragma unroll
        for (int q = 0; q < D / 32; ++q) {
          const uint32_t run = (q + (lane >> 1)) & (D / 32 - 1);
          const uint32_t f2 = scale_pair<FMT>(sc[q] & 0xFFu, sc[q] >> 8);
          const uint32_t f[2] = {__byte_perm(f2, f2, 0x1010), __byte_perm(f2, f2, 0x3232)};
          const uint32_t to = dst + (s >> 1) * (2 * T::kK) + (s & 1) * (kHalf * 128u) +
                              (run >> 1) * (kChunk * 128u);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint32_t h[4];
            e2m1x8_to_f16(w[q][e], h);
            st_shared16(to + (((4 * (run & 1) + e) ^ (pos & 7u)) << 4), mul_f16x2(h[0], f[e >> 1]),
                        mul_f16x2(h[1], f[e >> 1]), mul_f16x2(h[2], f[e >> 1]),
                        mul_f16x2(h[3], f[e >> 1]));
          }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(k_full(s >> 1));
          mbar_arrive(raw_empty(r));
        }
      }
      if (!ok) break;
      n += halves;
      more = next_piece();
    }
    } else if (warp < 4 * TILES + kValueWarps + kKeyWarps + 1) {
    // ---------------- copies of codes and scales ----------------
    // Positions behind the end, or without a page, become zeros: a zero scale makes zeros of any codes,
    // while what lies there may be NaN.
    constexpr int CH = D / 32, PER = D / 64;  // 16-byte pieces of a position's codes; of 16, per lane
    const int i0 = lane / CH, piece = lane % CH;
    const uint32_t put_k = s_raw + i0 * (D / 2) + 16 * piece;
    const uint32_t put_v = s_raw + T::kRawV + (i0 >> 3) * T::kOctet + (i0 & 7) * (D / 2) + 16 * piece;
    const uint8_t* src_k = a.c.codes[0] + i0 * (D / 2) + 16 * piece;
    const uint8_t* src_v = a.c.codes[1] + i0 * (D / 2) + 16 * piece;
    const int sgr = lane >> log_sb, sfirst = (lane & ((1 << log_sb) - 1)) << (4 - log_sb);
    // Lane i < 4 gets the place of the half's positions 16 i ..: the row of the cache (slots of one head)
    // divided by 16, or -1.
    auto place = [&](int half) {
      const int p = half * kHalf + 16 * lane;
      int row = -1;
      if (lane < 4 && p < k.end) {
        const int64_t slot = a.table.slot(a.c, k.b, p);
        if (slot >= 0) row = (int)((slot + ((int64_t)k.h << a.c.page_shift)) >> 4);
      }
      return row;
    };
    while (more) {
      k = PieceOf(walk);
      const int halves = 2 * k.chunks, h0 = 2 * k.c0;
      bool ok = true;
      int next = place(h0);
#pragma unroll 1
      for (int j = 0; j < halves; ++j) {
        const int i = n + j, r = i % R, p = (h0 + j) * kHalf;
        const int rows = next;
        next = place(h0 + j + 1);
        if (i >= R) ok = mbar_wait<20>(raw_empty(r), ((i / R) + 1) & 1, gave_up);
        if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
        const uint32_t at = r * T::kRaw;
#pragma unroll
        for (int gr = 0; gr < 4; ++gr) {
          const int row = __shfl_sync(0xffffffffu, rows, gr);
          const int left = row >= 0 ? k.end - (p + 16 * gr) : 0;  // positions that are there
          const uint64_t from = (uint64_t)(uint32_t)max(row, 0) * (16 * (D / 2));
#pragma unroll
          for (int e = 0; e < PER; ++e) {
            // positions i0 + e (32 / CH) of the 16
            const int size = i0 + e * (32 / CH) < left ? 16 : 0;
            const int pos = 16 * gr + e * (32 / CH);
            cp_async16(put_k + at + pos * (D / 2), src_k + from + 512 * e, size);
            cp_async16(put_v + at + (pos >> 3) * T::kOctet + (pos & 7) * (D / 2), src_v + from + 512 * e,
                       size);
          }
        }
        // scales: a piece of 16 bytes is those of 16 >> log_sb positions; 64 positions have at most 64
        // pieces (32 and fewer but for head_dim 256 in blocks of 16)
#pragma unroll
        for (int e = 0; e < (D == 256 ? 2 : 1); ++e) {
          const int gr = sgr + e * (32 >> log_sb);
          const int row = __shfl_sync(0xffffffffu, rows, gr & 3);
          if (gr < 4) {
            const int left = row >= 0 ? k.end - (p + 16 * gr) - sfirst : 0;
            const int size = min(max(left, 0), 16 >> log_sb) << log_sb;
            const uint64_t from = ((uint64_t)(uint32_t)max(row, 0) << (4 + log_sb)) + (sfirst << log_sb);
            const uint32_t to = s_raw + at + ((16 * gr + sfirst) << log_sb);
            cp_async16(to + T::kRawKS, a.c.scales[0] + (size ? from : 0), size);
            cp_async16(to + T::kRawVS, a.c.scales[1] + (size ? from : 0), size);
          }
        }
        // this lane's arrival comes when its copies are there
        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(raw_full(r))
                     : "memory");
      }
      if (!ok) break;
      n += halves;
      more = next_piece();
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncwarp();
    } else {
    // ---------------- products (one elected thread) ----------------
    if (elect_one()) {
      constexpr int P = S / 2;                   // stages of whole chunks
      int tiles = TILES;                         // with rows, of the piece
      int seen[2] = {0, 0}, pieces[2] = {0, 0};  // chunks and pieces so far, by tile
      auto scores = [&](int t, int s) {
        const uint32_t qd = desc_low(s_q + t * T::kQ), kd = desc_low(s_k + s * (2 * T::kK));
        const uint32_t d = tmem + T::kScoreCol + kChunk * t;
        // 16 values of the head a step: 32 bytes on, after 64 the next 128-byte-wide block
        mma_ss<false>(d, qd, kd, T::kIdescS);
#pragma unroll
        for (int x = 1; x < D / 16; ++x) {
          const uint32_t on = (x >> 2) * ((128 * 128) >> 4) + 2 * (x & 3);
          mma_ss<true>(d, qd + on, kd + on, T::kIdescS);
        }
        tc_commit(s_full(t));
        if (t == tiles - 1) tc_commit(k_empty(s));
      };
      auto outputs = [&](int t, int s, int half, bool add) {
        const uint32_t vd = desc_low(s_v + (2 * s + half) * T::kK);
        const uint32_t pa = tmem + T::kScoreCol + kChunk * t + 32 * half;
        mma_ts(tmem + T::kOutCol + D * t, pa, vd, T::kIdescO, add);
#pragma unroll
        for (int x = 1; x < kHalf / 16; ++x)
          mma_ts(tmem + T::kOutCol + D * t, pa + 8 * x, vd + 2 * x, T::kIdescO, true);
      };
      bool ok = true;
      while (more && ok) {
        const int chunks = walk.c1 - walk.c0, stop = n + chunks;
        if constexpr (TILES > 1) {
          tiles = walk.seq.count * group - walk.rt * T::kRows > 128 ? 2 : 1;
        }
#pragma unroll
        for (int t = 0; t < TILES; ++t)
          if (ok && t < tiles) ok = mbar_wait(q_full(t), pieces[t]++ & 1, gave_up);
        ok = ok && mbar_wait(k_full(n % P), (n / P) & 1, gave_up);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int t = 0; t < TILES; ++t)
          if (t < tiles) scores(t, n % P);
#pragma unroll 1
        for (int c = n; c < stop; ++c) {
          const int s = c % P, s1 = (c + 1) % P;
          const bool go = c + 1 < stop;
#pragma unroll
          for (int t = 0; t < TILES; ++t) {
            if (t >= tiles || !ok) continue;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              if (t == 0) ok = ok && mbar_wait(v_full(2 * s + half), (c / P) & 1, gave_up);
              ok = ok && mbar_wait(p_full(t, half), seen[t] & 1, gave_up);
              tc_fence_after();
              if (ok) outputs(t, s, half, c > stop - chunks || half > 0);
            }
            if (t == tiles - 1) tc_commit(v_empty(s));
            ++seen[t];
            if (go) {
              // (in order behind the outputs, which have read the weights there)
              if (t == 0) ok = ok && mbar_wait(k_full(s1), ((c + 1) / P) & 1, gave_up);
              tc_fence_after();
              if (ok) scores(t, s1);
            } else {
              tc_commit(o_full(t));
            }
          }
          if (!ok) break;
        }
        n = stop;
        more = walk.next(a, cut);
      }
      tc_commit(done);  // also after giving up: every issued product
    }
    __syncwarp();
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    int unused = 0;
    if (lane == 0) mbar_wait(done, 0, &unused);
    __syncwarp();
    if (lane == 0 && *gave_up) atomicAdd(&g_tile_gave_up, 1u);
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u)
                 : "memory");
  }
}

template <int D, int TILES, int FMT>
cudaError_t launch_tile(const AttnArgs& a, cudaStream_t stream, int* launches) {
  using T = Tile<D, TILES>;
  static std::atomic<bool> attr[kMaxDevices];
  auto* kern = k_attention_tile<D, TILES, FMT>;
  cudaError_t e = allow_dynamic_smem(attr, kern, T::kSmem);
  if (e != cudaSuccess) return e;
  int dev = 0, sms = 148;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  const int ctas = sms < kMaxTileCtas ? sms : kMaxTileCtas;
  e = launch_pdl_smem(kern, ctas, T::kThreads, T::kSmem, stream, a);
  if (e != cudaSuccess) return e;
  ++*launches;
  return launch_join<D, T::kRows, kMaxTileCtas>(a, ctas, sms, kScaleShift<FMT>, stream, launches);
}

template <int D, int TILES>
cudaError_t dispatch(const AttnArgs& a, cudaStream_t stream, int* launches) {
  return a.c.fmt == kUE5M3 ? launch_tile<D, TILES, kUE5M3>(a, stream, launches)
                           : launch_tile<D, TILES, kE4M3>(a, stream, launches);
}

}  // namespace

cudaError_t run_tile(const AttnArgs& a, cudaStream_t stream, int* launches) {
  const bool two = tile_rows(a.tokens * (a.heads / a.c.kv_heads), a.c.head_dim) == 256;
  switch (a.c.head_dim) {
    case 64: return two ? dispatch<64, 2>(a, stream, launches) : dispatch<64, 1>(a, stream, launches);
    case 128: return two ? dispatch<128, 2>(a, stream, launches) : dispatch<128, 1>(a, stream, launches);
    default: return dispatch<256, 1>(a, stream, launches);
  }
}

}  // namespace attn

cudaError_t attention_gave_up(unsigned int* count) {
  static std::atomic<unsigned int> seen[kMaxDevices];
  return counted_since(attn::g_tile_gave_up, seen, count);
}

}  // namespace mxk
