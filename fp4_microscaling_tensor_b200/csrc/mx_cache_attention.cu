// mx_cache_attention.cu -- attention over a paged FP4 key/value cache.
//
// out = softmax(scale q K^T) V with K = E2M1 S g as the cache stores them (microscaling article,
// hotelren.com/news/2192771, §1 and §3.1 item 3), one pass over K and V with the running maximum m
// and sum l of the softmax: for every chunk of positions, scores s = q K^T, m' = max(m, max s),
// weights p = 2^((s - m') c), l = l 2^((m - m') c) + sum p, o = o 2^((m - m') c) + p V.
//
// k_attention_stream, for few query rows per key/value head (a decoder's steps, chains and small
// trees of drafted tokens): it has to read the cache, 1 + 2 / N bytes per position and head dimension,
// and turn codes into f16 (about 2 instructions per pair of codes); the layout is made for both:
//   * mma.sync m16n8k16 with the positions (scores) or the head dimension (outputs) as its 16 rows
//     and the query rows as its 8 columns: 8 query rows -- 8 query heads that share a key/value head
//     -- fill it.  The 128 lanes-deep tcgen05 tile would be 6 % full; the tensor pipe is not what
//     bounds this.
//   * the contraction index of a product may be permuted if both operands agree.  So a thread's part
//     of the A operand of q K^T is a run of D / 4 consecutive codes of one position (16 bytes for D =
//     128: one load, 1 or 2 scales), and its part of V^T is D / 8 consecutive codes of four positions.
//     Two positions' codes are interleaved as nibbles (4 instructions per 16 codes) before they
//     become f16 pairs along the positions, the layout the A operand of V^T p needs.
//   * scores come out with positions in rows; movmatrix turns a pair of 8 x 8 weights tiles into the
//     B operand of V^T p.  Nothing but codes and scales goes through shared memory.
//   * every warp works for itself: cp.async brings its next tiles (64 positions, keys and values, 8 KB
//     + scales for D = 128) into a ring of its own while it computes; 12 warps per SM keep about 100
//     KB in flight.  Bytes behind the end of the sequence, or of no page, arrive as zeros (a zero
//     scale makes what the codes say harmless).
// The warps of a block share its piece's positions evenly and join their results in shared memory at
// the piece's end.
//
// Measured: one token for each of 64 sequences of 819 to 8191 positions, 64 heads on 8 of 128, 78 us at 1965
// MHz, 0.67 of the measured copy peak (83 us at the 1840 MHz that the power cap leaves of it after a
// second).  Neither memory nor the issue slots (57 % in use, ALU and FMA pipes 51 and 32 %) bound it then:
// with 2.8 warps per scheduler the fixed latencies of dependent instructions are the largest stall.
#include <math.h>

#include "mx_attention.cuh"
#include "mx_launch.h"

namespace mxk {
namespace attn {
namespace {

// Position (0..15 of a tile's 16) that row i of an MMA stands for: rows 2 and 3, 6 and 7, ... change
// places, so that the four lanes that read V at 2 t and 2 t + 1 hit both halves of 128 bytes.
__device__ __forceinline__ int perm(int i) { return i ^ ((i >> 1) & 1); }

constexpr int kWarps = 4;
constexpr int kStreamThreads = 32 * kWarps;

constexpr int kUnit = 64, kStart = 8;  // of the stream kernel's Cut (start: 0 88, 4 83, 8 79, 16 82 us for 64
                                      // sequences of 819 to 8191 positions)
constexpr int kPart = 32;  // positions computed at a time (more outgrow the instruction cache)

template <int D, int NT>
struct Geometry {
  static constexpr int kTile = D == 256 ? 32 : 64;         // positions per tile of the ring
  static constexpr int kRow = D / 2;                       // code bytes of a position
  static constexpr int kCodes = kTile * kRow;              // bytes of a tile's key (value) codes
  static constexpr int kScales = kTile * (D / 16);         // most scale bytes of a tile's keys
  static constexpr int kStage = 2 * (kCodes + kScales);
  // blocks per SM: what the registers allow (D NT / 4 accumulators, D NT / 8 words of queries); the
  // shared memory is split evenly
  static constexpr int kBlocks = D * NT <= 128 ? 3 : 2;
  static constexpr int kWarpBytes = kBlocks == 3 ? 18432 : 27648;
  static constexpr int kStages = kWarpBytes / kStage;
  // When the warps join, each one's outputs take the last kJoin slots of its ring; the first kEarly
  // are being filled for the next piece meanwhile.
  static constexpr int kJoinPitch = D + 4;                 // floats per row
  static constexpr int kJoin = (8 * NT * kJoinPitch * 4 + kStage - 1) / kStage;
  static constexpr int kEarly = kJoin == 1 ? kStages - 1 : kStages - kJoin;
  static constexpr int kJoinAt = (kStages - kJoin) * kStage;
  static_assert(kEarly >= 1 && kEarly < kStages, "ring slots");
};

__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint32_t smem_addr(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, "
      "%9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma16816_zero(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                              uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, "
      "%9}, {%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
}
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t v) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(v));
  return d;
}

// Scale codes -> f16, times 2^-kScaleShift: E4M3 by the hardware's conversion, UE5M3 (for which there
// is none) by a table of all codes in shared memory.  pair: (x, y); both: x in both halves.
template <int FMT>
__device__ __forceinline__ uint32_t scale_pair(uint32_t x, uint32_t y, uint32_t table) {
  uint32_t d;
  if constexpr (FMT == kE4M3) {
    asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}"
        : "=r"(d) : "r"(__byte_perm(x, y, 0x0040)));
  } else {
    uint32_t v[2];
    lds<4>(table + 4 * x, &v[0]);
    lds<4>(table + 4 * y, &v[1]);
    d = __byte_perm(v[0], v[1], 0x5410);
  }
  return d;
}
template <int FMT>
__device__ __forceinline__ uint32_t scale_both(uint32_t x, uint32_t table) {
  uint32_t d;
  if constexpr (FMT == kE4M3) {
    asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}"
        : "=r"(d) : "r"(x * 0x101u));
  } else {
    lds<4>(table + 4 * x, &d);
  }
  return d;
}

// One warp's tile ring, accumulators and softmax state for NT groups of 8 query rows.
template <int D, int NT, int FMT, bool N16>
struct Stream {
  using G = Geometry<D, NT>;
  static constexpr int KS = D / 16;               // k steps of q K^T
  static constexpr int KB = D / 8;                // code bytes of a lane's run of a key
  static constexpr int VB = D / 16;               // code bytes of a lane's run of a value
  static constexpr int MT = D / 16;               // 16-row tiles of the outputs

  const AttnArgs& a;
  const int lane, g, t4;
  const uint32_t ring, table;                     // shared addresses: the warp's ring, the scales
  const int log_sb;                               // log2 of the scale bytes of a position
  // this lane's places in a tile: where its copies of keys and values go, its part of the keys of
  // MMA row g, of the values of MMA columns 2 t4 and 2 t4 + 1, and their scales
  uint32_t put_k, put_v, put_s, get_k[2], get_v[2], get_ks[2], get_vs[2];
  const uint8_t *src[2], *src_s[2];               // where its copies come from, in the cache's row 0

  uint32_t q[NT][KS][2];                          // B operand of q K^T (f16 pairs)
  float mult[NT][2];                              // log2 weight per unit of raw score, this lane's
                                                  // two columns (query rows 8 nt + 2 t4, + 1)
  Maximum mx[NT][2];
  float l[NT][2];                                 // partial sum
  float o[NT][MT][4];

  // segment
  int64_t b;
  int h, group, row0;
  int end;                                        // this warp's positions of the piece (exclusive)
  int plain_end;                                  // up to here every row sees every position
  bool holes;                                     // a position in between has no page
  Seq seq;
  int tok[NT][2];                                 // this lane's columns: token, and its tree word
  uint64_t word[NT][2];

  __device__ __forceinline__ Stream(const AttnArgs& args, uint32_t ring_addr, uint32_t table_addr)
      : a(args), lane(threadIdx.x & 31), g(lane >> 2), t4(lane & 3), ring(ring_addr),
        table(table_addr),
        log_sb(N16 ? log2_of(D / 16) : log2_of(D) - args.c.log_block), seq(args, 0) {
    constexpr int CH = D / 32;
    const int i = lane / CH, piece = lane % CH, log_block = log2_of(D) - log_sb;
    // Swizzles (of 16-byte pieces by position) that keep the loads below free of bank conflicts
    if constexpr (D == 64) {
      put_k = 32 * i + 16 * piece;
      put_v = 32 * (i ^ ((i >> 2) & 1)) + 16 * piece;
    } else if constexpr (D == 128) {
      put_k = 64 * i + 16 * piece;
      put_v = 64 * i + 16 * (piece ^ ((i >> 1) & 3));
    } else {
      put_k = 128 * i + 16 * (piece ^ ((i & 1) << 2));
      put_v = 128 * i + 16 * (piece ^ (((i >> 1) & 3) << 1));
    }
    put_v += G::kCodes;
    put_s = 2 * G::kCodes + 16 * lane;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      src[e] = args.c.codes[e] + i * G::kRow + 16 * piece;
      src_s[e] = args.c.scales[e] + 16 * (lane & ((1 << log_sb) - 1));
    }
    const int k = perm(g);
#pragma unroll
    for (int run = 0; run < 2; ++run) {  // runs of 32 (D = 64: 16) codes; D <= 128 has one
      get_k[run] = D == 256 ? k * G::kRow + 16 * ((t4 + 4 * run) ^ ((k & 1) << 2))
                            : k * G::kRow + t4 * KB;
      const int d = D == 256 ? 128 * run + 32 * t4 : (D / 4) * t4;
      get_ks[run] = 2 * G::kCodes + (k << log_sb) + (d >> log_block);
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int v = perm(2 * t4 + e);
      if constexpr (D == 64) get_v[e] = 32 * (v ^ ((v >> 2) & 1)) + 4 * g;
      else if constexpr (D == 128) get_v[e] = 64 * v + 16 * ((g >> 1) ^ ((v >> 1) & 3)) + 8 * (g & 1);
      else get_v[e] = 128 * v + 16 * (g ^ (((v >> 1) & 3) << 1));
      get_v[e] += G::kCodes;
      get_vs[e] = 2 * G::kCodes + G::kScales + (v << log_sb) + ((g * (D / 8)) >> log_block);
    }
  }

  // Query rows row0 .. row0 + 8 NT - 1 of the segment: f16, each row scaled by the power of two that
  // brings its largest magnitude to [2^14, 2^15) (exact for all values within 2^-28 of it; what is
  // lost of smaller ones is below 2^-39 of it).
  __device__ __forceinline__ void load_queries() {
    const int rows = seq.count * group;
    const float gk = fp16_bits_to_float(a.c.g_bits[0]) * (float)(1 << kScaleShift<FMT>);
    const float base = a.scale == 0.0f ? 1.0f : fabsf(a.scale) * gk * 1.4426950408889634f;
    const uint32_t flip = a.scale < 0.0f ? 0x80008000u : 0u;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = row0 + 8 * nt + g;
      uint32_t w[2 * KS];  // bf16 pairs
      const bool in = r < rows && a.scale != 0.0f;
      const int64_t at = in ? row_offset(a.q, b, r / group, h * group + r % group) : 0;
#pragma unroll
      for (int i = 0; i < KS / 2; ++i) {
        // run i of 16 bytes: values D <= 128: (D / 4) t4 + 8 i; D = 256: two runs of 32, 128 apart
        const int d = D == 256 ? 128 * (i >> 2) + 32 * t4 + 8 * (i & 3) : (D / 4) * t4 + 8 * i;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (in) v = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q.p) + at + d));
        w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
      }
      uint32_t mx = 0;
#pragma unroll
      for (int i = 0; i < 2 * KS; ++i) mx = max(mx, max(w[i] & 0x7FFFu, (w[i] >> 16) & 0x7FFFu));
      mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      // 2^f; an all-zero row and one with infinities or NaN stay as they are
      const int f = mx == 0 || mx >= 0x7F80u ? 0 : 141 - max((int)(mx >> 7), 1);
      const int f1 = f / 2, f2 = f - f1;  // |f| may be 140: two steps
      const float s1 = __uint_as_float((uint32_t)(127 + f1) << 23);
      const float s2 = __uint_as_float((uint32_t)(127 + f2) << 23);
#pragma unroll
      for (int i = 0; i < 2 * KS; ++i)
        q[nt][i >> 1][i & 1] =
            pack_f16x2(bf16lo(w[i]) * s1 * s2, bf16hi(w[i]) * s1 * s2) ^ (in ? flip : 0u);
      const float mine = base * __uint_as_float((uint32_t)(127 - f1) << 23) *
                         __uint_as_float((uint32_t)(127 - f2) << 23);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        // kept normal: a masked score times it stays -infinity
        mult[nt][e] =
            fminf(fmaxf(__shfl_sync(0xffffffffu, mine, 4 * (2 * t4 + e)), 0x1p-126f), 0x1p126f);
        const int c = row0 + 8 * nt + 2 * t4 + e;
        tok[nt][e] = c < rows ? c / group : 0;
        word[nt][e] = c < rows && a.tree ? a.tree[b * a.tokens + tok[nt][e]] : 0;
      }
    }
  }

  __device__ __forceinline__ void reset() {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int e = 0; e < 2; ++e) mx[nt][e].reset(), l[nt][e] = 0.0f;
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[nt][i][e] = 0.0f;
    }
  }

  // Lane i gets the place of the 16 positions from p + 16 i on: the row of the cache (slots of one
  // head) divided by 16, or -1.  (Pages are whole multiples of 16 slots.)
  __device__ __forceinline__ int page_rows(int p) const {
    const int pos = p + 16 * lane;
    int row = -1;
    if (pos < end) {
      const int64_t slot = a.table.slot(a.c, b, pos);
      if (slot >= 0) row = (int)((slot + ((int64_t)h << a.c.page_shift)) >> 4);
    }
    return row;
  }

  // Copies the tile from position p on to st in the ring; lanes from on hold its page_rows.
  // Bytes of positions behind the end, or without a page, arrive as zeros.
  __device__ __forceinline__ void issue(int p, int rows, int from, uint32_t st) {
    constexpr int PER = D / 64;         // 16-byte pieces per lane of 16 positions' codes
    constexpr int GR = G::kTile / 16;
    int row[GR], all = 0;
#pragma unroll
    for (int gr = 0; gr < GR; ++gr) {
      row[gr] = __shfl_sync(0xffffffffu, rows, from + gr);
      all |= row[gr];
    }
    const int sgr = lane >> log_sb;     // the 16 positions whose scales this lane copies
    const int srow = __shfl_sync(0xffffffffu, rows, from + (sgr & (GR - 1)));
    if (p + G::kTile <= end && all >= 0) {
#pragma unroll
      for (int gr = 0; gr < GR; ++gr) {
        const uint64_t at = (uint64_t)(uint32_t)row[gr] * (16 * G::kRow);
        const uint8_t *ks = src[0] + at, *vs = src[1] + at;
        const uint32_t kd = st + put_k, vd = st + put_v;
#pragma unroll
        for (int k = 0; k < PER; ++k) {
          const int to = gr * 16 * G::kRow + 512 * k;
          cp_async16(kd + to, ks + 512 * k);
          cp_async16(((D == 256 && (k & 1)) ? vd ^ 64u : vd) + to, vs + 512 * k);
        }
      }
      if (sgr < GR) {
        const uint64_t at = (uint64_t)(uint32_t)srow << (4 + log_sb);
        cp_async16(st + put_s, src_s[0] + at);
        cp_async16(st + put_s + G::kScales, src_s[1] + at);
      }
      return;
    }
#pragma unroll 1
    for (int gr = 0; gr < GR; ++gr) {
      const int r = __shfl_sync(0xffffffffu, rows, from + gr), left = end - (p + 16 * gr);
      if (r < 0 && left > 0) holes = true;
#pragma unroll
      for (int k = 0; k < PER; ++k) {
        const bool ok = r >= 0 && lane / (D / 32) + k * (1024 / D) < left;
        const uint64_t at = ok ? (uint64_t)r * (16 * G::kRow) + 512 * k : 0;
        const int to = gr * 16 * G::kRow + 512 * k;
        cp_async16(st + put_k + to, src[0] + at, ok ? 16 : 0);
        cp_async16(st + ((D == 256 && (k & 1)) ? put_v ^ 64u : put_v) + to, src[1] + at, ok ? 16 : 0);
      }
      if (sgr == gr) {
        // a piece of 16 bytes is the scales of 16 >> log_sb positions
        const int first = (lane & ((1 << log_sb) - 1)) << (4 - log_sb);
        const int n = r >= 0 ? min(max(left - first, 0), 16 >> log_sb) << log_sb : 0;
        const uint64_t at = n ? (uint64_t)r << (4 + log_sb) : 0;
        cp_async16(st + put_s, src_s[0] + at, n);
        cp_async16(st + put_s + G::kScales, src_s[1] + at, n);
      }
    }
  }

  // The kPart positions from p on, their codes at st and their scales at st_s (offset by the codes).
  __device__ __forceinline__ void compute(int p, uint32_t st, uint32_t st_s) {
    constexpr int T = kPart / 16;
    float s[NT][T][4];
    // ---- scores
#pragma unroll
    for (int mt = 0; mt < T; ++mt) {
      constexpr int RUNS = D == 256 ? 2 : 1;
      constexpr int RB = KB / RUNS;                // bytes of a run
      constexpr bool kTwo = N16 && RB == 16;       // two scales in a run
#pragma unroll
      for (int run = 0; run < RUNS; ++run) {
        uint32_t c[2][RB / 4], sc[2][2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int i = 16 * mt + 8 * e;           // and perm(g)
          lds<RB>(st + get_k[run] + i * G::kRow, c[e]);
          const uint32_t sa = st_s + get_ks[run] + (i << log_sb);
          if constexpr (kTwo) {
            const uint32_t w = lds_u16(sa);
            if constexpr (FMT == kE4M3) {
              const uint32_t f = scale_pair<FMT>(w, w >> 8, table);
              sc[e][0] = __byte_perm(f, f, 0x1010);
              sc[e][1] = __byte_perm(f, f, 0x3232);
            } else {
              sc[e][0] = scale_both<FMT>(w & 0xFFu, table);
              sc[e][1] = scale_both<FMT>(w >> 8, table);
            }
          } else {
            sc[e][0] = sc[e][1] = scale_both<FMT>(lds_u8(sa), table);
          }
        }
#pragma unroll
        for (int wd = 0; wd < RB / 4; ++wd) {
          uint32_t ha[4], hb[4];
          e2m1x8_to_f16(c[0][wd], ha);
          e2m1x8_to_f16(c[1][wd], hb);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            ha[i] = mul_f16x2(ha[i], sc[0][kTwo ? wd >> 1 : 0]);
            hb[i] = mul_f16x2(hb[i], sc[1][kTwo ? wd >> 1 : 0]);
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint32_t f[4] = {ha[2 * e], hb[2 * e], ha[2 * e + 1], hb[2 * e + 1]};
            const int k = (RB / 2) * run + 2 * wd + e;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              if (k == 0) mma16816_zero(s[nt][mt], f, q[nt][k][0], q[nt][k][1]);
              else mma16816(s[nt][mt], f, q[nt][k][0], q[nt][k][1]);
            }
          }
        }
      }
    }
    // ---- masks: only tiles with new tokens, the end, or positions without a page
    if (p + kPart > plain_end || holes) {
#pragma unroll
      for (int mt = 0; mt < T; ++mt)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int pos = p + 16 * mt + 8 * half + perm(g);
          const bool in = pos < end && (!holes || a.table.slot(a.c, b, pos) >= 0);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              if (!in || !sees(a, seq, tok[nt][e], word[nt][e], pos))
                s[nt][mt][2 * half + e] = -INFINITY;
        }
    }
    // ---- weights, relative to a maximum that follows the scores with a delay, so most tiles need no
    // exchange between lanes and leave the outputs as they are
    uint32_t pb[NT][T][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float top[2];
      bool grew = false;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        top[e] = fmaxf(s[nt][0][e], s[nt][0][2 + e]);
#pragma unroll
        for (int mt = 1; mt < T; ++mt) top[e] = fmaxf(top[e], fmaxf(s[nt][mt][e], s[nt][mt][2 + e]));
        grew |= top[e] > mx[nt][e].lim;
      }
      if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float m = mx[nt][e].m;
          float mn = fmaxf(top[e], m);
#pragma unroll
          for (int off = 4; off < 32; off <<= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, off));
          // (no score yet: nothing to scale)
          const float alpha = m == -INFINITY ? (mn == -INFINITY ? 1.0f : 0.0f)
                                             : ex2((m - mn) * mult[nt][e]);
          mx[nt][e].set(mn, mult[nt][e]);
          const float sub = mx[nt][e].far(mult[nt][e]) ? mn : 0.0f;
#pragma unroll
          for (int mt = 0; mt < T; ++mt) s[nt][mt][e] -= sub, s[nt][mt][2 + e] -= sub;
          l[nt][e] *= alpha;
#pragma unroll
          for (int i = 0; i < MT; ++i) o[nt][i][e] *= alpha, o[nt][i][2 + e] *= alpha;
        }
      }
#pragma unroll
      for (int mt = 0; mt < T; ++mt) {
        float w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          w[e] = ex2(fmaf(s[nt][mt][e], mult[nt][e & 1], -mx[nt][e & 1].mu));
          l[nt][e & 1] += w[e];
        }
        // binary16 weights: 2^-11 each, and 2^-32 of the maximum's below the normal range
        pb[nt][mt][0] = movmatrix_trans(pack_f16x2(w[0], w[1]));
        pb[nt][mt][1] = movmatrix_trans(pack_f16x2(w[2], w[3]));
      }
    }
    // ---- outputs: V^T p
#pragma unroll
    for (int kt = 0; kt < T; ++kt) {
      uint32_t c[4][VB / 4 > 0 ? VB / 4 : 1];
      uint32_t sc[2][2];  // [position pair][half of the lane's run]
      uint32_t sw[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int i = 16 * kt + 8 * (e >> 1);      // and perm(2 t4 + (e & 1))
        lds<VB>(st + get_v[e & 1] + i * G::kRow, c[e]);
        const uint32_t sa = st_s + get_vs[e & 1] + (i << log_sb);
        sw[e] = (N16 && D == 256) ? lds_u16(sa) : lds_u8(sa);
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        if constexpr (N16 && D == 256) {  // two scales in a run
          sc[e][0] = scale_pair<FMT>(sw[2 * e] & 0xFFu, sw[2 * e + 1] & 0xFFu, table);
          sc[e][1] = scale_pair<FMT>(sw[2 * e] >> 8, sw[2 * e + 1] >> 8, table);
        } else {
          sc[e][0] = sc[e][1] = scale_pair<FMT>(sw[2 * e], sw[2 * e + 1], table);
        }
      }
#pragma unroll
      for (int wd = 0; wd < VB / 4; ++wd) {
        uint32_t ev[2][4], od[2][4];  // even and odd codes of the word: pairs of positions
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t x = c[2 * e][wd], y = c[2 * e + 1][wd];
          e2m1x8_to_f16((x & 0x0F0F0F0Fu) | ((y << 4) & 0xF0F0F0F0u), ev[e]);
          e2m1x8_to_f16(((x >> 4) & 0x0F0F0F0Fu) | (y & 0xF0F0F0F0u), od[e]);
          const uint32_t f = sc[e][VB / 4 == 4 ? wd >> 1 : 0];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            ev[e][i] = mul_f16x2(ev[e][i], f);
            od[e][i] = mul_f16x2(od[e][i], f);
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t f[4] = {ev[0][i], od[0][i], ev[1][i], od[1][i]};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma16816(o[nt][4 * wd + i], f, pb[nt][kt][0], pb[nt][kt][1]);
        }
      }
    }
  }

  // What the copies are at: the next position to copy, the places of the 512 positions around it and
  // of those behind them, its place in `rows`, and where it goes.
  int ahead, rows, rows_next, from;
  uint32_t to;

  __device__ __forceinline__ void copy() {
    if (ahead < end) {
      issue(ahead, rows, from, to);
      from += G::kTile / 16;
      if (from == 32) {
        from = 0;
        rows = rows_next;
        rows_next = page_rows(ahead + G::kTile + 512);
      }
    }
    cp_commit();
    ahead += G::kTile;
    to = to == ring + (G::kStages - 1) * G::kStage ? ring : to + G::kStage;
  }

  // A piece: this warp's positions [p0, p1) (p0 a multiple of 16) of segment (b_, h_, row0_ ..).
  // Starts the first copies, and loads the queries while they are on their way.
  __device__ __forceinline__ void begin(int64_t b_, int h_, int row0_, int p0, int p1) {
    b = b_;
    h = h_;
    row0 = row0_;
    seq = Seq(a, b);
    end = p1;
    holes = false;
    plain_end = min(end, seen_by_all(a, seq, row0 / group));
    ahead = p0;
    rows = page_rows(p0);
    rows_next = page_rows(p0 + 512);
    from = 0;
    to = ring;
#pragma unroll 1
    for (int s = 0; s < G::kEarly; ++s) copy();
    load_queries();
  }

  // The rest of it.
  __device__ __forceinline__ void run(int p0) {
    reset();
#pragma unroll 1
    for (int s = G::kEarly; s < G::kStages - 1; ++s) copy();
    uint32_t st = ring;
#pragma unroll 1
    for (int p = p0; p < end; p += G::kTile) {
      copy();
      cp_wait<G::kStages - 1>();
      __syncwarp();
#pragma unroll 1
      for (int part = 0; part < G::kTile && p + part < end; part += kPart)
        compute(p + part, st + part * G::kRow, st + (part << log_sb));
      __syncwarp();
      st = st == ring + (G::kStages - 1) * G::kStage ? ring : st + G::kStage;
    }
    cp_wait<0>();
    __syncwarp();
  }
};

// Result of a piece: rows x D outputs (unnormalised, relative to the maximum), joined over the
// block's warps.  out/lse, or a partial result.
template <int D, int NT, int FMT, bool N16>
__global__ void __launch_bounds__(kStreamThreads, Geometry<D, NT>::kBlocks)
    k_attention_stream(const __grid_constant__ AttnArgs a) {
  using G = Geometry<D, NT>;
  constexpr int R = 8 * NT;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int64_t s_scan[kWarps];
  __shared__ Share s_share;
  __shared__ float s_m[kWarps][R], s_l[kWarps][R];
  __shared__ uint32_t s_table[FMT == kUE5M3 ? 256 : 1];
  if constexpr (FMT == kUE5M3)
    for (int i = threadIdx.x; i < 256; i += kStreamThreads) s_table[i] = scale_f16x2<FMT>(i);
  const int warp = threadIdx.x >> 5;
  const int group = a.heads / a.c.kv_heads, ctas = gridDim.x, cta = blockIdx.x;
  griddep_wait();
  griddep_launch_next();
  const Cut cut{R, group, kUnit, kStart};
  find_share<kStreamThreads>(a, cut, cta, ctas, s_scan, &s_share);
  const Share sh = s_share;
  Record* rec = reinterpret_cast<Record*>(a.workspace) + cta;
  Record mine{0, 0, 0, -1, 0};
  const float gv = fp16_bits_to_float(a.c.g_bits[1]) * (float)(1 << kScaleShift<FMT>);

  Walk k;
  if (k.begin(a, cut, sh)) {
    Stream<D, NT, FMT, N16> w(a, smem_addr(smem) + warp * G::kWarpBytes, smem_addr(s_table));
    w.group = group;
    int p0;
    auto begin = [&] {
      // an equal run of 16-position groups for each warp
      const int first = k.c0 * kUnit, last = min(k.end, k.c1 * kUnit), groups = (last - first + 15) / 16;
      p0 = first + 16 * (groups * warp / kWarps);
      w.begin(k.b, k.h, k.rt * R, p0, min(last, first + 16 * (groups * (warp + 1) / kWarps)));
    };
    begin();
    while (true) {
      w.run(p0);

      // this warp's maxima, sums and outputs
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float l = w.l[nt][e];
#pragma unroll
          for (int off = 4; off < 32; off <<= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
          if (w.g == 0) {
            const int r = 8 * nt + 2 * w.t4 + e;
            s_m[warp][r] = w.mx[nt][e].log2(w.mult[nt][e]);
            s_l[warp][r] = l;
          }
        }
      float* mine_o = reinterpret_cast<float*>(smem + warp * G::kWarpBytes + G::kJoinAt);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            *reinterpret_cast<float2*>(mine_o + (8 * nt + 2 * w.t4 + e) * G::kJoinPitch +
                                       (D / 8) * w.g + 2 * i) =
                make_float2(w.o[nt][i][e], w.o[nt][i][2 + e]);

      // the next piece's first copies before this one's join
      const int64_t b = k.b;
      const int h = k.h, row0 = k.rt * R, rows = min(R, w.seq.count * group - row0);
      const bool whole = k.whole();
      float* part = partial(a, ctas, R, D, 2 * cta + (k.c0 == 0));
      if (k.c0 == 0 && !whole)
        mine = {b, h, k.rt, block_of(k.u0 + k.n + kStart - 1, sh), rows};
      const bool more = k.next(a, cut);
      if (more) begin();
      __syncthreads();

      for (int i = threadIdx.x; i < R * (D / 8); i += kStreamThreads) {
        const int r = i / (D / 8), d = 8 * (i % (D / 8));
        if (r >= rows) break;
        float mx = s_m[0][r];
#pragma unroll
        for (int x = 1; x < kWarps; ++x) mx = fmaxf(mx, s_m[x][r]);
        const float mu = mx == -INFINITY ? 0.0f : mx;
        float l = 0.0f, y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = 0.0f;
#pragma unroll
        for (int x = 0; x < kWarps; ++x) {
          const float f = ex2(s_m[x][r] - mu);
          l += s_l[x][r] * f;
          const float4* src = reinterpret_cast<const float4*>(
              smem + x * G::kWarpBytes + G::kJoinAt + (r * G::kJoinPitch + d) * 4);
          const float4 v0 = src[0], v1 = src[1];
          y[0] += v0.x * f, y[1] += v0.y * f, y[2] += v0.z * f, y[3] += v0.w * f;
          y[4] += v1.x * f, y[5] += v1.y * f, y[6] += v1.z * f, y[7] += v1.w * f;
        }
        if (whole) {
          const int row = row0 + r, t = row / group, head = h * group + row % group;
          const float f = l == 0.0f ? 0.0f : gv / l;
          const uint4 v = make_uint4(pack_bf16x2(y[0] * f, y[1] * f), pack_bf16x2(y[2] * f, y[3] * f),
                                     pack_bf16x2(y[4] * f, y[5] * f), pack_bf16x2(y[6] * f, y[7] * f));
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out.p) + row_offset(a.out, b, t, head) +
                                    d) = v;
          if (a.lse && d == 0)
            a.lse[(b * a.tokens + t) * a.heads + head] = log_sum(mu, l);
        } else {
          float4* dst = reinterpret_cast<float4*>(part + 2 * R + r * D + d);
          dst[0] = make_float4(y[0], y[1], y[2], y[3]);
          dst[1] = make_float4(y[4], y[5], y[6], y[7]);
          if (d == 0) part[r] = mx, part[R + r] = l;
        }
      }
      __syncthreads();
      if (!more) break;
    }
  }
  if (threadIdx.x == 0) *rec = mine;
}

// Query rows per tile: 8, 16 or 32, as many as there are (a tile's rows share one pass over the cache);
// 16 at most for head_dim 128 and 256, where the accumulators of 32 spill (16 sequences of up to 8000
// positions, 32 rows per key/value head, head_dim 128: two passes of 16 rows 85 us, one of 32 146 us;
// head_dim 64: one pass 56 us).
int row_groups(int64_t rows, int dim) {
  const int most = dim == 64 ? 4 : 2;
  const int nt = rows <= 8 ? 1 : rows <= 16 ? 2 : 4;
  return nt < most ? nt : most;
}

constexpr int kMaxStreamCtas = 3 * 160;  // thread blocks at most: 3 per SM

template <int D, int NT, int FMT, bool N16>
cudaError_t launch_stream(const AttnArgs& a, cudaStream_t stream, int* launches) {
  static std::atomic<bool> attr[kMaxDevices];
  constexpr int smem = kWarps * Geometry<D, NT>::kWarpBytes;
  auto* kern = k_attention_stream<D, NT, FMT, N16>;
  cudaError_t e = allow_dynamic_smem(attr, kern, smem);
  if (e != cudaSuccess) return e;
  int dev = 0, sms = 148;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  const int per_sm = Geometry<D, NT>::kBlocks;
  // never more blocks than units that the table could hold
  const int group = a.heads / a.c.kv_heads;
  const int64_t tiles = (a.tokens * group + 8 * NT - 1) / (8 * NT);
  const int64_t reach = (a.table.width << a.c.page_shift) / kUnit + 1 + kStart;
  int64_t grid = (int64_t)per_sm * (sms < 160 ? sms : 160);
  const double most = (double)a.batch * a.c.kv_heads * tiles * reach;
  if (most < (double)grid) grid = (int64_t)most;
  const int ctas = (int)(grid < 1 ? 1 : grid);
  e = launch_pdl_smem(kern, ctas, kStreamThreads, smem, stream, a);
  if (e != cudaSuccess) return e;
  ++*launches;
  return launch_join<D, 8 * NT, kMaxStreamCtas>(a, ctas, sms, kScaleShift<FMT>, stream, launches);
}

template <int D, int NT>
cudaError_t dispatch_format(const AttnArgs& a, cudaStream_t stream, int* launches) {
  if (a.c.fmt == kUE5M3)
    return a.c.block == 16 ? launch_stream<D, NT, kUE5M3, true>(a, stream, launches)
                           : launch_stream<D, NT, kUE5M3, false>(a, stream, launches);
  return a.c.block == 16 ? launch_stream<D, NT, kE4M3, true>(a, stream, launches)
                         : launch_stream<D, NT, kE4M3, false>(a, stream, launches);
}

template <int D>
cudaError_t dispatch_rows(const AttnArgs& a, cudaStream_t stream, int* launches) {
  const int nt = row_groups(a.tokens * (a.heads / a.c.kv_heads), D);
  if (nt == 1) return dispatch_format<D, 1>(a, stream, launches);
  if constexpr (D == 64) {
    if (nt == 4) return dispatch_format<D, 4>(a, stream, launches);
  }
  return dispatch_format<D, 2>(a, stream, launches);
}

}  // namespace
}  // namespace attn

// Above this many query rows per key/value head the tile kernel takes over, whose time hardly depends on
// the rows up to 128.  32 rows there and here (16 sequences of up to 8000 positions): head_dim 64 100 and
// 56 us, 128 120 and 86, 256 305 and 197; of up to 600: 27 and 24, 34 and 26, 54 and 44.  64 rows: 120
// there, 250 here (head_dim 128).
static constexpr int kStreamRows = 32;

size_t attention_workspace_bytes(int64_t batch, int64_t tokens, int heads, int kv_heads,
                                 int head_dim) {
  if (batch == 0 || tokens == 0) return 16;
  const int64_t all = tokens * (heads / kv_heads);
  const bool tile = all > kStreamRows;
  const int rows = tile ? attn::tile_rows(all, head_dim) : 8 * attn::row_groups(all, head_dim);
  const int ctas = tile ? attn::kMaxTileCtas : attn::kMaxStreamCtas;
  return attn::records_bytes(ctas) + 2 * (size_t)ctas * attn::partial_floats(rows, head_dim) * 4;
}

cudaError_t run_cache_attention(const AttnArgs& a, cudaStream_t stream, int* launches) {
  if (a.tokens * (a.heads / a.c.kv_heads) > kStreamRows) return attn::run_tile(a, stream, launches);
  switch (a.c.head_dim) {
    case 64: return attn::dispatch_rows<64>(a, stream, launches);
    case 128: return attn::dispatch_rows<128>(a, stream, launches);
    default: return attn::dispatch_rows<256>(a, stream, launches);
  }
}

}  // namespace mxk
