// mx_cache_attention.cu -- attention over a paged FP4 key/value cache.
//
// One warp per query row (sequence, token, head): 32 positions at a time, one per lane for the
// scores, running maximum and sum of the softmax in fp32, head_dim / 32 output values per lane.
#include "mx_cache.h"
#include "mx_device.cuh"
#include "mx_launch.h"

namespace mxk {
namespace {

constexpr int kWarps = 4;

template <int D, int FMT>
__global__ void __launch_bounds__(32 * kWarps) k_cache_attention(const __grid_constant__ AttnArgs a) {
  __shared__ float s_q[kWarps][D];
  const CacheArgs& c = a.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t r = (int64_t)blockIdx.x * kWarps + warp;
  griddep_wait();
  griddep_launch_next();
  const int h = (int)(r % a.heads);
  const int64_t bt = r / a.heads, b = bt / a.tokens, t = bt % a.tokens;
  if (b >= a.batch) return;
  const int64_t cnt = a.count ? min((int64_t)max(a.count[b], 0), a.tokens) : a.tokens;
  if (t >= cnt) return;
  const int64_t len = min((int64_t)max(a.length[b], 0), a.table.width << c.page_shift);
  const int64_t base = len - cnt;
  const uint16_t* q = static_cast<const uint16_t*>(a.q.p) + b * a.q.sb + t * a.q.st + h * a.q.sh;
  for (int i = lane; i < D; i += 32) s_q[warp][i] = __uint_as_float((uint32_t)q[i] << 16);
  __syncwarp();
  const uint64_t word = a.tree ? a.tree[b * a.tokens + t] : 0;
  const int kvh = h / (a.heads / c.kv_heads);
  const float kscale = a.scale * fp16_bits_to_float(c.g_bits[0]);
  const int64_t end = a.tree ? len : min(len, base + t + 1);
  float m = -INFINITY, l = 0.0f, acc[D / 32];
  for (int i = 0; i < D / 32; ++i) acc[i] = 0.0f;
  for (int64_t p0 = 0; p0 < end; p0 += 32) {
    const int64_t p = p0 + lane;
    const int64_t j = p - base;
    const bool seen = p < end && (!a.tree || j < 0 || ((word >> j) & 1));
    int64_t row = p < end ? a.table.slot(c, b, p) : -1;
    if (row >= 0) row += (int64_t)kvh << c.page_shift;
    float s = -INFINITY;
    if (seen && row >= 0) {
      s = 0.0f;
      for (int i = 0; i < D; i += 2) {
        const uint32_t cw = c.codes[0][row * (D / 2) + i / 2];
        const float S = scale_value(c.scales[0][row * (D / c.block) + i / c.block], FMT);
        s += (e2m1_to_float(cw & 15u) * s_q[warp][i] + e2m1_to_float(cw >> 4) * s_q[warp][i + 1]) * S;
      }
      s *= kscale;
    }
    float mx = s;
    for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    const float mn = fmaxf(m, mx);
    const float mu = mn == -INFINITY ? 0.0f : mn;  // nothing seen yet (or only NaN scores)
    const float w = expf(s - mu), f = expf(m - mu);
    float sum = w;
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    l = l * f + sum;
    m = mn;
    for (int i = 0; i < D / 32; ++i) acc[i] *= f;
    for (int k = 0; k < 32; ++k) {
      const float wk = __shfl_sync(0xffffffffu, w, k);
      const int64_t rk = __shfl_sync(0xffffffffu, row, k);
      if (wk == 0.0f || rk < 0) continue;
      for (int i = 0; i < D / 32; ++i) {
        const int d = lane + 32 * i;
        const uint32_t cw = c.codes[1][rk * (D / 2) + d / 2];
        const float S = scale_value(c.scales[1][rk * (D / c.block) + d / c.block], FMT);
        acc[i] += wk * (e2m1_to_float((cw >> (4 * (d & 1))) & 15u) * S);
      }
    }
  }
  const float f = l == 0.0f ? 0.0f : fp16_bits_to_float(c.g_bits[1]) / l;
  __nv_bfloat16* out =
      static_cast<__nv_bfloat16*>(a.out.p) + b * a.out.sb + t * a.out.st + h * a.out.sh;
  for (int i = 0; i < D / 32; ++i) out[lane + 32 * i] = __float2bfloat16_rn(acc[i] * f);
  if (a.lse && lane == 0) a.lse[bt * a.heads + h] = l == 0.0f ? -INFINITY : (m == -INFINITY ? 0.0f : m) + logf(l);
}

template <int D>
cudaError_t launch(const AttnArgs& a, cudaStream_t stream) {
  const int64_t grid = (a.batch * a.tokens * a.heads + kWarps - 1) / kWarps;
  if (grid >= (int64_t(1) << 31)) return cudaErrorInvalidConfiguration;
  return a.c.fmt == kUE5M3
             ? launch_pdl(k_cache_attention<D, kUE5M3>, (int)grid, 32 * kWarps, stream, a)
             : launch_pdl(k_cache_attention<D, kE4M3>, (int)grid, 32 * kWarps, stream, a);
}

}  // namespace

size_t attention_workspace_bytes(int64_t, int64_t, int, int, int) { return 16; }

cudaError_t run_cache_attention(const AttnArgs& a, cudaStream_t stream, int* launches) {
  const cudaError_t e = a.c.head_dim == 64    ? launch<64>(a, stream)
                        : a.c.head_dim == 128 ? launch<128>(a, stream)
                                              : launch<256>(a, stream);
  if (e == cudaSuccess) ++*launches;
  return e;
}

}  // namespace mxk
