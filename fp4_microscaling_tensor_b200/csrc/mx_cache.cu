// mx_cache.cu -- a paged FP4 key/value cache: quantizing keys and values as they are written, and
// reading them back.
//
// Method: the microscaling article (hotelren.com/news/2192771) §3.1 items 1-3 on every key and
// value vector: blocks of N consecutive values of a head share one FP8 scale S = Q_fp8(absmax /
// (6 g)), each value becomes Q_fp4(x / (S g)); two codes per byte (4-bit float article,
// gtnt.cn/news/16247, §4.3).  The arithmetic is that of mx_quantize / mx_dequantize
// (mx_device.cuh), so the codes, scales and values are theirs bit for bit; what differs is where
// they go: position p of sequence b lives in slot p % P of page table[b][p / P], so tokens enter
// and leave a sequence without moving the others.
//
// Both kernels stream: per value they move e + 1/2 + 1/N bytes (e = 2 or 4, the width of the
// outside values) and hold nothing.  A thread owns 16 consecutive values of a head (an item: two
// 16-byte accesses outside for bf16, 8 bytes of codes), of the keys and of the values, so both
// streams are in flight at once.  Items run along the head, then along the tokens, then across the
// heads: consecutive lanes touch whole 256-byte rows outside (bf16, head_dim 128) and adjacent
// slots of one head -- contiguous memory -- in the cache.  Measured, 8 heads of 128, blocks of 32, against
// the bytes at the measured copy peak: 24862 tokens of 4 sequences of up to 8192 in, bf16 26 us (0.77), fp32
// 56 us (0.64); 106205 of 8 of up to 16000 out, bf16 111 us (0.77), fp32 298 us (0.51).
#include <string.h>

#include <type_traits>

#include "mx_cache.h"
#include "mx_device.cuh"
#include "mx_launch.h"

namespace mxk {
namespace {

struct MoveArgs {
  CacheArgs c;
  PageTable table;
  Rows x[2];  // keys, values
  int64_t tokens;
  const int32_t* start;
  const int32_t* count;
  int tile_shift;  // log2 of the tokens per CTA
  int tiles;       // CTAs per sequence
};

// Item i of a CTA's tile: head i / (tokens x items per head), token, 16-element chunk.
struct Item {
  int h, t, chunk;
  __device__ __forceinline__ Item(int i, int log_chunks, int tile_shift)
      : h(i >> (log_chunks + tile_shift)),
        t((i >> log_chunks) & ((1 << tile_shift) - 1)),
        chunk(i & ((1 << log_chunks) - 1)) {}
};

// A block's scale code from its largest magnitude a, and the divisor S g of its elements.
template <int FMT>
__device__ __forceinline__ float divisor(uint32_t code, float g) {
  return __fmul_rn(scale_value((int)code, FMT), g);  // exact (<= 15 significant bits)
}

// The largest of m over the lanes that share a block of N (adjacent lanes, 16 elements each).
template <typename T>
__device__ __forceinline__ T block_max(T m, int lanes) {
  for (int off = 1; off < lanes; off <<= 1) {
    const T o = __shfl_xor_sync(0xffffffffu, m, off);
    m = o > m ? o : m;
  }
  return m;
}

// 16 bf16 values (8 words) -> two words of codes and the block's scale code.  Infinities saturate and
// NaNs do not count for the scale (the maximum drops them beside other values, the comparison where there
// are none), so that no NaN scale is ever stored; a NaN itself becomes code 6.
template <int FMT>
__device__ __forceinline__ uint32_t quantize16(const uint32_t (&w)[8], int lanes, float g, float r6,
                                               uint2& codes) {
  uint32_t t = w[0];
#pragma unroll
  for (int k = 1; k < 8; ++k) t = bf16x2_absmax(t, w[k]);
  t &= 0x7FFF7FFFu;
  const uint32_t lo = t & 0xFFFFu, hi = t >> 16;
  const uint32_t m = block_max(max(lo > 0x7F80u ? 0u : lo, hi > 0x7F80u ? 0u : hi), lanes);
  const uint32_t sc = encode_scale<FMT>(snap21(__fmul_rn(__uint_as_float(m << 16), r6)));
  const float D = divisor<FMT>(sc, g);
  const float r = D > 0.0f ? __frcp_rn(D) : 0.0f;  // zero scale: every code is +-0
  float q[16];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float2 v = snap_quotient2(w[k] << 16, w[k] & 0xFFFF0000u, r);
    q[2 * k] = v.x;
    q[2 * k + 1] = v.y;
  }
  codes.x = cvt_e2m1x8(q[0], q[1], q[2], q[3], q[4], q[5], q[6], q[7]);
  codes.y = cvt_e2m1x8(q[8], q[9], q[10], q[11], q[12], q[13], q[14], q[15]);
  return sc;
}

// The same of 16 fp32 values, by division (mx_device.cuh: 24-bit inputs leave no room for the
// reciprocal).
template <int FMT>
__device__ __forceinline__ uint32_t quantize16(const float (&x)[16], int lanes, float g, float g6,
                                               uint2& codes) {
  float a = 0.0f;
#pragma unroll
  for (int k = 0; k < 16; ++k) a = fmaxf(a, fabsf(x[k]));
  a = block_max(a, lanes);
  const uint32_t sc = encode_scale<FMT>(__fdiv_rn(a, g6));
  const float D = divisor<FMT>(sc, g);
  float q[16];
#pragma unroll
  for (int k = 0; k < 16; ++k) q[k] = D > 0.0f ? __fdiv_rn(x[k], D) : x[k] * 0.0f;  // (signed zeros)
  codes.x = cvt_e2m1x8(q[0], q[1], q[2], q[3], q[4], q[5], q[6], q[7]);
  codes.y = cvt_e2m1x8(q[8], q[9], q[10], q[11], q[12], q[13], q[14], q[15]);
  return sc;
}

template <int FMT, bool BF16>
__global__ void __launch_bounds__(kThreads) k_cache_append(const __grid_constant__ MoveArgs a) {
  using T = typename std::conditional<BF16, uint32_t, float>::type;  // bf16: pairs
  constexpr int kW = BF16 ? 2 : 4;                                   // 16-byte loads of an item
  const CacheArgs& c = a.c;
  const int64_t b = blockIdx.x / (unsigned)a.tiles;
  const int64_t t0 = (int64_t)(blockIdx.x % (unsigned)a.tiles) << a.tile_shift;
  const float g[2] = {fp16_bits_to_float(c.g_bits[0]), fp16_bits_to_float(c.g_bits[1])};
  float c6[2];  // 1 / (6 g) for bf16, 6 g for fp32
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    c6[s] = __fmul_rn(6.0f, g[s]);
    if (BF16) c6[s] = __frcp_rn(c6[s]);
  }
  const int log_chunks = __ffs(c.head_dim) - 5;  // 16-element chunks of a head
  const int n = c.kv_heads << (a.tile_shift + log_chunks);
  const int lanes = c.block >> 4;
  griddep_wait();  // inputs may come from the previous kernel in the stream
  griddep_launch_next();
  const int64_t first = a.start[b];
  const int64_t count = a.count ? min((int64_t)a.count[b], a.tokens) : a.tokens;
  if (t0 >= count) return;

  for (int i0 = 0; i0 < n; i0 += blockDim.x) {
    const Item it(i0 + (int)threadIdx.x, log_chunks, a.tile_shift);
    const bool in = it.h < c.kv_heads && t0 + it.t < count;
    const int64_t slot = in ? a.table.slot(c, b, first + t0 + it.t) : -1;
    const bool ok = slot >= 0;
    const int64_t row = slot + ((int64_t)it.h << c.page_shift);
    if (!__any_sync(0xffffffffu, ok)) continue;  // (fp32 divisions of zeros are slow)
    T x[2][4 * kW];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const uint4* src = reinterpret_cast<const uint4*>(
          static_cast<const char*>(a.x[s].p) +
          (b * a.x[s].sb + (t0 + it.t) * a.x[s].st + it.h * a.x[s].sh + 16 * it.chunk) *
              (BF16 ? 2 : 4));
#pragma unroll
      for (int k = 0; k < kW; ++k) {
        const uint4 v = ok ? ld_stream16(src + k) : make_uint4(0, 0, 0, 0);
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) memcpy(&x[s][4 * k + e], &u[e], 4);
      }
    }
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      uint2 codes;
      const uint32_t sc = quantize16<FMT>(x[s], lanes, g[s], c6[s], codes);
      if (!ok) continue;
      *reinterpret_cast<uint2*>(c.codes[s] + row * (c.head_dim >> 1) + 8 * it.chunk) = codes;
      if ((it.chunk & (lanes - 1)) == 0)
        c.scales[s][row * (c.head_dim >> c.log_block) + ((16 * it.chunk) >> c.log_block)] = (uint8_t)sc;
    }
  }
}

template <int FMT, bool BF16>
__global__ void __launch_bounds__(kThreads) k_cache_read(const __grid_constant__ MoveArgs a) {
  const CacheArgs& c = a.c;
  const int64_t b = blockIdx.x / (unsigned)a.tiles;
  const int64_t t0 = (int64_t)(blockIdx.x % (unsigned)a.tiles) << a.tile_shift;
  const float g[2] = {fp16_bits_to_float(c.g_bits[0]), fp16_bits_to_float(c.g_bits[1])};
  const int log_chunks = __ffs(c.head_dim) - 5;
  const int n = c.kv_heads << (a.tile_shift + log_chunks);
  griddep_wait();
  griddep_launch_next();
  const int64_t first = a.start[b];
  const int64_t count = a.count ? min((int64_t)a.count[b], a.tokens) : a.tokens;
  if (t0 >= count) return;

  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    const Item it(i, log_chunks, a.tile_shift);
    if (t0 + it.t >= count) continue;
    const int64_t slot = a.table.slot(c, b, first + t0 + it.t);
    const int64_t row = slot + ((int64_t)it.h << c.page_shift);
    uint2 codes[2];
    uint32_t sc[2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      codes[s] = make_uint2(0, 0);  // a position without a page reads as zeros
      sc[s] = 0;
      if (slot >= 0) {
        codes[s] = __ldg(reinterpret_cast<const uint2*>(c.codes[s] + row * (c.head_dim >> 1) +
                                                        8 * it.chunk));
        sc[s] = __ldg(c.scales[s] + row * (c.head_dim >> c.log_block) +
                      ((16 * it.chunk) >> c.log_block));
      }
    }
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const float D = __fmul_rn(scale_value((int)sc[s], FMT), g[s]);  // exact
      const uint32_t cw[2] = {codes[s].x, codes[s].y};
      uint32_t h[2][4];
#pragma unroll
      for (int k = 0; k < 2; ++k) e2m1x8_to_f16(cw[k], h[k]);
      float y[16];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float2 v = __fmul2_rn(__half22float2(*reinterpret_cast<const __half2*>(&h[k >> 2][k & 3])),
                                    make_float2(D, D));  // exact
        y[2 * k] = v.x;
        y[2 * k + 1] = v.y;
      }
      const int64_t at = b * a.x[s].sb + (t0 + it.t) * a.x[s].st + it.h * a.x[s].sh + 16 * it.chunk;
      if constexpr (BF16) {
        uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.x[s].p) + at);
#pragma unroll
        for (int k = 0; k < 2; ++k)
          __stcs(dst + k, make_uint4(pack_bf16x2(y[8 * k], y[8 * k + 1]),
                                     pack_bf16x2(y[8 * k + 2], y[8 * k + 3]),
                                     pack_bf16x2(y[8 * k + 4], y[8 * k + 5]),
                                     pack_bf16x2(y[8 * k + 6], y[8 * k + 7])));
      } else {
        float4* dst = reinterpret_cast<float4*>(static_cast<float*>(a.x[s].p) + at);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          __stcs(dst + k, make_float4(y[4 * k], y[4 * k + 1], y[4 * k + 2], y[4 * k + 3]));
      }
    }
  }
}

// The items of a CTA's tile.
int tile_items(const CacheArgs& c, int tile_shift) {
  return c.kv_heads * (c.head_dim / 16) << tile_shift;
}

// Tokens per CTA: 16 (8 sequences of 16000 tokens of 8 heads of 128 read to bf16: 109 us, with 4 and 32
// 112), halved while there would be less than four CTAs per SM and two warps keep their items: a small
// call is one thread's chain of loads, so it goes wide (100 tokens of 4 heads of 256 values read to fp32:
// 2.2 us; 3.0 if no CTA may have less than 256 items, 4.2 with 512).
MoveArgs move_args(const CacheArgs& c, const PageTable& table, const Rows& k, const Rows& v,
                   int64_t batch, int64_t tokens, const int32_t* start, const int32_t* count) {
  MoveArgs a{c, table, {k, v}, tokens, start, count, 4, 0};
  while (a.tile_shift > 0 && tile_items(c, a.tile_shift) > 64 &&
         batch * ((tokens + (1 << a.tile_shift) - 1) >> a.tile_shift) < 4 * 148)
    --a.tile_shift;
  return a;
}

template <typename K>
cudaError_t launch_move(K* kern, MoveArgs& a, int64_t batch, cudaStream_t stream, int* launches) {
  const int64_t tiles = (a.tokens + (int64_t(1) << a.tile_shift) - 1) >> a.tile_shift;
  if (tiles >= (int64_t(1) << 31) || batch * tiles >= (int64_t(1) << 31))
    return cudaErrorInvalidConfiguration;
  a.tiles = (int)tiles;
  const int items = tile_items(a.c, a.tile_shift);
  const int threads = items < kThreads ? (items + 31) / 32 * 32 : kThreads;
  const cudaError_t e = launch_pdl(kern, (int)(batch * tiles), threads, stream, a);
  if (e == cudaSuccess) ++*launches;
  return e;
}

}  // namespace

cudaError_t run_cache_append(const CacheArgs& c, const PageTable& table, const Rows& k,
                             const Rows& v, bool bf16, int64_t batch, int64_t tokens,
                             const int32_t* start, const int32_t* count, cudaStream_t stream,
                             int* launches) {
  MoveArgs a = move_args(c, table, k, v, batch, tokens, start, count);
  if (bf16)
    return c.fmt == kUE5M3 ? launch_move(k_cache_append<kUE5M3, true>, a, batch, stream, launches)
                           : launch_move(k_cache_append<kE4M3, true>, a, batch, stream, launches);
  return c.fmt == kUE5M3 ? launch_move(k_cache_append<kUE5M3, false>, a, batch, stream, launches)
                         : launch_move(k_cache_append<kE4M3, false>, a, batch, stream, launches);
}

cudaError_t run_cache_read(const CacheArgs& c, const PageTable& table, const Rows& k,
                           const Rows& v, bool bf16, int64_t batch, int64_t tokens,
                           const int32_t* start, const int32_t* count, cudaStream_t stream,
                           int* launches) {
  MoveArgs a = move_args(c, table, k, v, batch, tokens, start, count);
  if (bf16)
    return c.fmt == kUE5M3 ? launch_move(k_cache_read<kUE5M3, true>, a, batch, stream, launches)
                           : launch_move(k_cache_read<kE4M3, true>, a, batch, stream, launches);
  return c.fmt == kUE5M3 ? launch_move(k_cache_read<kUE5M3, false>, a, batch, stream, launches)
                         : launch_move(k_cache_read<kE4M3, false>, a, batch, stream, launches);
}

}  // namespace mxk
