// mx_attention.cuh -- what the attention kernels over the FP4 cache share: how the work is cut, the
// partial results of pieces, and small device helpers.
//
// The work of a call is a list of units, the chunks of 64 or 128 positions of every segment, a segment being
// (sequence, key/value head, tile of query rows).  The query rows of a key/value head are its
// heads / kv_heads query heads of every token, row r = token r / G, head r % G.  How long the
// sequences are is known on the device only, so every thread block adds the units up itself and
// takes an equal share of the list: [W c / n, W (c + 1) / n) for block c of n, whatever the lengths
// are (with fewer units than blocks the first blocks get one each).  A share covers segments whole, or
// pieces of at most two (its first and its last one); the pieces of a segment leave their running
// maximum, sum and unnormalised output in the workspace, and k_attention_join adds them up in the order
// of the list, so results do not depend on timing.
#pragma once

#include <float.h>
#include <math.h>

#include "mx_cache.h"
#include "mx_device.cuh"

namespace mxk {
namespace attn {

// How a kernel cuts the work: query rows per tile, query heads per key/value head, positions per unit,
// and what starting a piece costs a block (loading queries, filling its pipeline, joining), in units:
// every segment counts that many units more than it has, in front; a share that would begin or end
// within them begins or ends at the segment instead.
struct Cut {
  int rows, group, unit, start;
};

// a / b for a >= 0, b > 0 (the 64-bit division is an order of magnitude slower).
__device__ __forceinline__ int64_t divide(int64_t a, int64_t b) {
  if (((a | b) >> 32) == 0) return (uint32_t)a / (uint32_t)b;
  return a / b;
}

// A sequence's numbers, cut to what is there: len positions, of which the newest `count` are this
// call's tokens, from position base on (negative where the sequence is shorter than its count).
struct Seq {
  int len, count, base;
  Seq() = default;
  __device__ __forceinline__ Seq(const AttnArgs& a, int64_t b) {
    const int64_t reach = a.table.width << a.c.page_shift;  // at most 2^30
    len = (int)min((int64_t)max(a.length[b], 0), reach);
    count = a.count ? (int)min((int64_t)max(a.count[b], 0), a.tokens) : (int)a.tokens;
    base = len - count;
  }
  // Tiles of `rows` query rows, and the positions that the rows of tile rt see at most.
  __device__ __forceinline__ int tiles(const Cut& c) const {
    return (int)(((int64_t)count * c.group + c.rows - 1) / c.rows);
  }
  __device__ __forceinline__ int end(const AttnArgs& a, const Cut& c, int rt) const {
    if (a.tree) return len;
    const int64_t last = divide((int64_t)(rt + 1) * c.rows - 1, c.group);  // the tile's last token
    return max(0, (int)min((int64_t)len, base + min((int64_t)count - 1, last) + 1));
  }
};

__device__ __forceinline__ int units_of(const Cut& c, int end) {
  return c.start + max(1, (end + c.unit - 1) / c.unit);
}

// Units of one key/value head of a sequence: the part that lane `sub` of `lanes` adds up.
__device__ __forceinline__ int64_t head_units(const AttnArgs& a, const Seq& s, const Cut& c, int sub,
                                              int lanes) {
  const int tiles = s.tiles(c);
  if (a.tree || tiles <= 1)
    return tiles && sub == 0 ? (int64_t)tiles * units_of(c, s.end(a, c, 0)) : 0;
  int64_t n = 0;
  for (int rt = sub; rt < tiles; rt += lanes) n += units_of(c, s.end(a, c, rt));
  return n;
}

// Where a thread block's share of the list begins, and how long the list is.
struct Share {
  int64_t b;          // the segment of the share's first unit,
  int h, rt;
  int at;             // and the unit's place in it
  int blocks;         // how many blocks have a share that is not empty: the first ones
  int64_t lo, hi, total;
};

// All THREADS threads; scratch: THREADS / 32 values.  A group of threads (32, fewer for many sequences,
// then one for a run of them) adds up the tiles of a sequence; the warp in whose run the share's first
// unit is looks the tile up, 32 at a time.
template <int THREADS>
__device__ __forceinline__ void find_share(const AttnArgs& a, const Cut& c, int cta, int ctas,
                                           int64_t* scratch, Share* out) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int lanes = 32;
  while (lanes > 1 && a.batch * lanes > THREADS) lanes >>= 1;
  const int sub = tid & (lanes - 1), gid = tid / lanes;
  const int64_t per = divide(a.batch + THREADS / lanes - 1, THREADS / lanes);  // 1 if lanes > 1
  const int64_t b0 = min(a.batch, gid * per), b1 = min(a.batch, b0 + per);
  int64_t sum = 0;
  for (int64_t b = b0; b < b1; ++b) sum += head_units(a, Seq(a, b), c, sub, lanes);
  for (int o = 1; o < lanes; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  int64_t units = sum;  // of a key/value head, in all the sequences of the run
  sum *= a.c.kv_heads;
  int64_t incl = sub == 0 ? sum : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) scratch[warp] = incl;
  __syncthreads();
  int64_t before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w < warp) before += scratch[w];
    total += scratch[w];
  }
  // (a list of 2^52 units, where the product would not fit, would take years)
  const int n = (int)min((int64_t)ctas, total);
  const int64_t lo = cta < n ? divide(total * cta, n) : total;
  const int64_t hi = cta < n ? divide(total * (cta + 1), n) : total;
  const int64_t first = before + incl - sum;
  const uint32_t who = __ballot_sync(0xffffffffu, lo < hi && lo >= first && lo < first + sum);
  if (who) {
    int64_t at = lo - first, b = b0;
    if (lanes == 1 && (who >> lane & 1)) {
      for (;; ++b) {
        units = head_units(a, Seq(a, b), c, 0, 1);
        if (at < units * a.c.kv_heads) break;
        at -= units * a.c.kv_heads;
      }
    }
    const int src = __ffs(who) - 1;
    at = __shfl_sync(0xffffffffu, at, src);
    b = __shfl_sync(0xffffffffu, b, src);
    units = __shfl_sync(0xffffffffu, units, src);
    const int h = (int)divide(at, units);
    at -= h * units;
    const Seq s(a, b);
    const int tiles = s.tiles(c);
    for (int rt0 = 0; rt0 < tiles; rt0 += 32) {
      const int mine = rt0 + lane < tiles ? units_of(c, s.end(a, c, rt0 + lane)) : 0;
      int upto = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += v;
      }
      const uint32_t past = __ballot_sync(0xffffffffu, upto > at);
      if (past) {
        if (lane == __ffs(past) - 1)
          *out = {b, h, rt0 + lane, (int)at - (upto - mine), n, lo, hi, total};
        break;
      }
      at -= __shfl_sync(0xffffffffu, upto, 31);
    }
  }
  if (tid == 0 && lo >= hi) *out = {0, 0, 0, 0, n, 0, 0, total};  // an empty share
  __syncthreads();
}

// The block whose share unit u is in (the inverse of find_share's split).
__device__ __forceinline__ int block_of(int64_t u, const Share& sh) {
  return (int)divide((u + 1) * sh.blocks - 1, sh.total);
}

// A walk over the pieces of a share: segment (b, h, rt), its chunks (of Cut::unit positions) c0 .. c1 - 1 of `n`.
struct Walk {
  int64_t b;
  int h, rt;
  int c0, c1, n;
  int end;             // positions the tile's rows see at most
  int64_t left;        // units of the share behind this piece
  int64_t u0;          // the list's place of the segment's first unit
  Seq seq;
  __device__ __forceinline__ void set(const AttnArgs& a, const Cut& c, int at) {
    end = seq.end(a, c, rt);
    const int units = units_of(c, end);
    const int take = (int)min((int64_t)(units - at), left);
    n = units - c.start;
    c0 = max(0, at - c.start);
    c1 = at + take - c.start;
    left -= take;
  }
  // The share's first piece; false if there is none.
  __device__ __forceinline__ bool begin(const AttnArgs& a, const Cut& c, const Share& sh) {
    if (sh.lo >= sh.hi) return false;
    b = sh.b;
    h = sh.h;
    rt = sh.rt;
    seq = Seq(a, b);
    int at = sh.at;
    u0 = sh.lo - at;
    if (at <= c.start) at = 0;
    left = sh.hi - (u0 + at);
    if (left <= c.start && at == 0) return false;
    set(a, c, at);
    return true;
  }
  // The next piece; false if there is none.
  __device__ __forceinline__ bool next(const AttnArgs& a, const Cut& c) {
    if (left <= c.start) return false;
    u0 += n + c.start;
    if (++rt >= seq.tiles(c)) {
      rt = 0;
      if (++h >= a.c.kv_heads) {
        h = 0;
        do seq = Seq(a, ++b);
        while (seq.tiles(c) == 0);
      }
    }
    set(a, c, 0);
    return true;
  }
  __device__ __forceinline__ bool whole() const { return c0 == 0 && c1 == n; }
};

// ---- the kernel for many query rows (mx_attention_tile.cu) -----------------------------------------

constexpr int kMaxTileCtas = 160;
// Query rows per tile: two 128-row tiles take turns on the tensor cores where there are rows for both
// (and tensor memory: not with head_dim 256).
inline int tile_rows(int64_t rows, int dim) { return rows > 128 && dim < 256 ? 256 : 128; }
cudaError_t run_tile(const AttnArgs& a, cudaStream_t stream, int* launches);

// ---- workspace: one record per thread block, then two partial results per thread block ------------

// Written by the block that holds a split segment's first units: the segment, the last of the blocks
// that hold its pieces, and its query rows; last < 0: nothing to join.
struct Record {
  int64_t b;
  int h, rt, last, rows;
};
static_assert(sizeof(Record) == 24, "record layout");

// A partial result of up to R rows: R maxima (log2 domain), R sums, R x D outputs in float32.
__host__ __device__ inline size_t partial_floats(int rows, int dim) {
  return (size_t)rows * (dim + 2);
}
__host__ __device__ inline size_t records_bytes(int ctas) {
  return ((size_t)ctas * sizeof(Record) + 255) / 256 * 256;
}
// Place 2 c holds block c's piece that begins inside a segment, place 2 c + 1 the one that begins
// with a segment and does not end it.
__device__ __forceinline__ float* partial(const AttnArgs& a, int ctas, int rows, int dim, int place) {
  return reinterpret_cast<float*>(static_cast<char*>(a.workspace) + records_bytes(ctas)) +
         (size_t)place * partial_floats(rows, dim);
}

// log2 of a power of two.
__host__ __device__ constexpr int log2_of(int n) { return n <= 1 ? 0 : 1 + log2_of(n / 2); }

// ---- small helpers ---------------------------------------------------------------------------------

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 16 bytes into shared memory; of the form with a size, the rest are zeros.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
template <int BYTES>
__device__ __forceinline__ void lds(uint32_t addr, uint32_t* v) {
  if constexpr (BYTES == 16)
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(addr));
  else if constexpr (BYTES == 8)
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v[0]), "=r"(v[1]) : "r"(addr));
  else
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v[0]) : "r"(addr));
}
__device__ __forceinline__ uint32_t lds_u8(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint32_t lds_u16(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

// Scales enter the products as f16 values S 2^-kScaleShift: with E4M3, E2M1 x S has at most 6
// significant bits and lies in [2^-10, 2688]; with UE5M3, E2M1 x S 2^-4 in [2^-22, 46080], a multiple
// of 2^-22.  Both are exact in f16 (subnormals included), so K and V enter the products exactly.
template <int FMT>
constexpr int kScaleShift = FMT == kUE5M3 ? 4 : 0;

// f16 bits of a scale code, in both halves.
template <int FMT>
__device__ __forceinline__ uint32_t scale_f16x2(int code) {
  const float v = scale_value(code, FMT) * (FMT == kUE5M3 ? 0x1p-4f : 1.0f);
  return pack_f16x2(v, v);
}

__device__ __forceinline__ int64_t row_offset(const Rows& x, int64_t b, int t, int head) {
  return b * x.sb + (int64_t)t * x.st + (int64_t)head * x.sh;
}

// Whether the new token t (its tree word w) sees position pos < end.
__device__ __forceinline__ bool sees(const AttnArgs& a, const Seq& s, int t, uint64_t w, int pos) {
  const int j = pos - s.base;
  return j < 0 || (a.tree ? j < s.count && ((w >> j) & 1) : j <= t);
}

// Every row from new token t on sees the positions before this one: the old ones and, in a chain, the
// tokens up to t.  (A tree's words need not name token 0.)
__device__ __forceinline__ int seen_by_all(const AttnArgs& a, const Seq& s, int t) {
  return s.base + (a.tree ? 0 : t + 1);
}

// The softmax's maximum in use and the weights 2^(s mult - mu) of raw scores s.  The maximum moves only
// when a score exceeds it by kSlack (in log2), and weights are kLift above what that makes them: binary16
// holds up to 2^16, and the step of the small ones, 2^-24, is 2^-31 of the weight at the maximum then.
// mu = m mult - kLift is rounded; the weights of a row share the factor that this makes, 2^(2^-24 |mu|) at
// most, and dividing by their sum takes it out again.  But binary16 has little room for it, so from
// |m mult| = 2^21 on (`far`) the maximum is taken from the scores before they are multiplied:
// 2^((s - m) mult + kLift).  That happens where the maximum is looked at, so any score of such a row counts
// as one that may move it.
constexpr float kSlack = 8.0f, kLift = 7.0f, kFar = 0x1p21f;
static_assert(kLift == 7.0f, "log_sum takes 2^7 out of the weights' sum");
struct Maximum {
  float m, mu, lim;  // raw, what scaled scores are relative to, the score that moves it
  __device__ __forceinline__ void reset() { m = lim = -INFINITY, mu = 0.0f; }
  __device__ __forceinline__ bool far(float mult) const {
    return m > -INFINITY && fabsf(m * mult) >= kFar;
  }
  // mn: a raw score, or -infinity if there is none yet.
  __device__ __forceinline__ void set(float mn, float mult) {
    m = mn;
    const bool f = mn == -INFINITY || far(mult);
    mu = f ? -kLift : fmaf(mn, mult, -kLift);
    lim = f ? -INFINITY : mn + kSlack / mult;
  }
  // What the weights are relative to, in log2, for a join: -infinity if there is no score, finite
  // otherwise (differences are taken of it).
  __device__ __forceinline__ float log2(float mult) const {
    return m == -INFINITY ? m : fminf(fmaxf(fmaf(m, mult, -kLift), -FLT_MAX), FLT_MAX);
  }
};

// The natural logarithm of the sum of the exponentials, from the sum l of weights relative to mu.
__device__ __forceinline__ float log_sum(float mu, float l) {
  return l == 0.0f ? -INFINITY
                   : ((mu + kLift) + log2f(l * 0x1p-7f)) * 0.6931471805599453f;
}

// ---- joining pieces --------------------------------------------------------------------------------

namespace {

constexpr int kJoinThreads = 256, kMostRuns = 16;

// How many threads share the pieces of an output, four pieces each (a power of two).
__device__ __forceinline__ int log_runs(int pieces) {
  int k = 0;
  while ((4 << k) < pieces && (1 << k) < kMostRuns) ++k;
  return k;
}

// Joins the pieces of the segments that are split: that of record c is in blocks c .. last, one piece
// each.  The work is a list of steps of kJoinThreads threads, over all records; every block adds their
// numbers up and takes every gridDim.x-th.  A thread holds four outputs of a row and a run of pieces;
// the runs are added up in order.  (With a block for each record and quarter of the head dimension, 101
// rows of one head over two sequences of up to 7681 positions took 82 us instead of 20.)
template <int D, int R, int MAX_CTAS>
__global__ void __launch_bounds__(kJoinThreads) k_attention_join(const __grid_constant__ AttnArgs a,
                                                                 int ctas, float gv) {
  constexpr int kPer = (MAX_CTAS + kJoinThreads - 1) / kJoinThreads;  // records per thread
  __shared__ int s_warp[kJoinThreads / 32];
  __shared__ Record s_rec;
  __shared__ int s_first, s_step;  // the block that began the segment; the step's place among its steps
  __shared__ float4 s_o[kJoinThreads];
  __shared__ float s_m[kJoinThreads], s_l[kJoinThreads];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // (The next kernel is not launched early.  Blocks of a next call's stream kernel that come while this
  // kernel's blocks leave spread unevenly over the SMs: calls in a row, 16 sequences of up to 4000
  // positions, head_dim 64, took 59 us each instead of 43.)
  griddep_wait();
  Record recs[kPer];
  int steps[kPer], sum = 0;
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int c = tid + k * kJoinThreads;
    steps[k] = 0;
    if (c < ctas) {
      recs[k] = reinterpret_cast<const Record*>(a.workspace)[c];
      if (recs[k].last >= 0)
        steps[k] = ((recs[k].rows * (D / 4) << log_runs(recs[k].last - c + 1)) + kJoinThreads - 1) /
                   kJoinThreads;
    }
    sum += steps[k];
  }
  int incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) s_warp[warp] = incl;
  __syncthreads();
  int total = 0;
#pragma unroll
  for (int w = 0; w < kJoinThreads / 32; ++w) {
    if (w < warp) incl += s_warp[w];
    total += s_warp[w];
  }

  const int group = a.heads / a.c.kv_heads;
  for (int u = blockIdx.x; u < total; u += gridDim.x) {
    int at = u - (incl - sum);
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      if (at >= 0 && at < steps[k]) s_rec = recs[k], s_first = tid + k * kJoinThreads, s_step = at;
      at -= steps[k];
    }
    __syncthreads();
    const Record rec = s_rec;
    const int c = s_first, n = rec.last - c + 1, lk = log_runs(n), items = kJoinThreads >> lk;
    const int i = s_step * items + (tid & (items - 1)), run = tid / items;
    const int r = i / (D / 4), d = 4 * (i % (D / 4));
    float mx = -INFINITY, l = 0.0f;
    float4 y = make_float4(0, 0, 0, 0);
    if (r < rec.rows) {
      // pieces run * per .. : an order that depends on their number only
      const int per = (n + (1 << lk) - 1) >> lk, x1 = min(n, (run + 1) * per);
      for (int x0 = run * per; x0 < x1; x0 += 4) {
        float pm[4], pl[4];
        float4 po[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          pm[e] = -INFINITY, pl[e] = 0.0f, po[e] = make_float4(0, 0, 0, 0);
          if (x0 + e < x1) {
            const float* p = partial(a, ctas, R, D, 2 * (c + x0 + e) + (x0 + e == 0));
            pm[e] = p[r], pl[e] = p[R + r];
            po[e] = *reinterpret_cast<const float4*>(p + 2 * R + r * D + d);
          }
        }
        const float mn = fmaxf(fmaxf(fmaxf(pm[0], pm[1]), fmaxf(pm[2], pm[3])), mx);
        const float mu = mn == -INFINITY ? 0.0f : mn, f = ex2(mx - mu);
        l *= f, y.x *= f, y.y *= f, y.z *= f, y.w *= f;
        mx = mn;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float w = ex2(pm[e] - mu);
          l += pl[e] * w;
          y.x += po[e].x * w, y.y += po[e].y * w, y.z += po[e].z * w, y.w += po[e].w * w;
        }
      }
    }
    if (lk > 0) {
      s_m[tid] = mx, s_l[tid] = l, s_o[tid] = y;
      __syncthreads();
      if (run == 0) {
        float mn = mx;
        for (int x = 1; x < 1 << lk; ++x) mn = fmaxf(mn, s_m[x * items + tid]);
        const float mu = mn == -INFINITY ? 0.0f : mn;
        l = 0.0f, y = make_float4(0, 0, 0, 0);
        for (int x = 0; x < 1 << lk; ++x) {
          const float w = ex2(s_m[x * items + tid] - mu);
          const float4 v = s_o[x * items + tid];
          l += s_l[x * items + tid] * w;
          y.x += v.x * w, y.y += v.y * w, y.z += v.z * w, y.w += v.w * w;
        }
        mx = mn;
      }
    }
    if (r < rec.rows && run == 0) {
      const int64_t row = (int64_t)rec.rt * R + r;
      const int t = (int)divide(row, group), head = rec.h * group + (int)(row - (int64_t)t * group);
      const float f = l == 0.0f ? 0.0f : gv / l;
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out.p) + row_offset(a.out, rec.b, t, head) +
                                d) =
          make_uint2(pack_bf16x2(y.x * f, y.y * f), pack_bf16x2(y.z * f, y.w * f));
      if (a.lse && d == 0)
        a.lse[(rec.b * a.tokens + t) * a.heads + head] = log_sum(mx, l);
    }
    __syncthreads();
  }
}

// Launches the join behind a kernel of `ctas` blocks (whose blocks only read the records where nothing
// was split).
template <int D, int R, int MAX_CTAS>
cudaError_t launch_join(const AttnArgs& a, int ctas, int sms, int scale_shift, cudaStream_t stream,
                        int* launches) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(4 * (ctas < sms ? ctas : sms)));
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = stream;
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = pdl;
  cfg.numAttrs = 1;
  const uint32_t g = a.c.g_bits[1];
  const float gv = ldexpf(g >> 10 ? (float)(1024 + (g & 1023)) : (float)g,
                          (g >> 10 ? (int)(g >> 10) - 25 : -24) + scale_shift);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, k_attention_join<D, R, MAX_CTAS>, a, ctas, gv);
  if (e == cudaSuccess) ++*launches;
  return e;
}

}  // namespace
}  // namespace attn
}  // namespace mxk
