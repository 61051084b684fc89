// mx_cache.h -- kernel parameters and internal entry points of the paged FP4 key/value cache.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace mxk {

// One layer's cache (see mx_cache_t in include/mx.h): position p of a sequence is slot
// p % page_size of its page number p / page_size; a slot holds, per key/value head, head_dim / 2
// code bytes and head_dim / block scale bytes, head-major within a page.
struct CacheArgs {
  uint8_t* codes[2];   // keys, values: [pages][kv_heads][page_size][head_dim / 2]
  uint8_t* scales[2];  //               [pages][kv_heads][page_size][head_dim / block]
  int64_t pages;
  int kv_heads, head_dim, block, fmt;
  int page_shift;      // log2(page_size)
  int log_block;       // log2(block)
  uint16_t g_bits[2];
};

// The sequences' pages: row b of the table holds the page numbers of sequence b.
struct PageTable {
  const int32_t* pages;
  int64_t stride;   // entries from one row to the next
  int64_t width;    // entries of a row
#ifdef __CUDACC__
  // Index of the (page, slot) row of position pos of sequence b in units of slots of one head
  // (page * kv_heads * page_size + slot), or -1 where the table does not reach or names no page of
  // the cache.
  __device__ __forceinline__ int64_t slot(const CacheArgs& c, int64_t b, int64_t pos) const {
    const int64_t pg = pos >> c.page_shift;
    if (pos < 0 || pg >= width) return -1;
    const int32_t id = __ldg(pages + b * stride + pg);
    if (id < 0 || id >= c.pages) return -1;
    return (((int64_t)id * c.kv_heads) << c.page_shift) + (pos & ((1 << c.page_shift) - 1));
  }
#endif
};

// Keys or values outside the cache: element (b, t, h, i) at p[b * sb + t * st + h * sh + i].
struct Rows {
  void* p;
  int64_t sb, st, sh;
};

// Quantizes k and v [batch, tokens, kv_heads, head_dim] (bf16 or fp32) into positions start[b] + t,
// t < count[b] (all tokens when count is null).
cudaError_t run_cache_append(const CacheArgs& c, const PageTable& table, const Rows& k,
                             const Rows& v, bool bf16, int64_t batch, int64_t tokens,
                             const int32_t* start, const int32_t* count, cudaStream_t stream,
                             int* launches);
// Dequantizes positions start[b] + t, t < count[b], into k and v.
cudaError_t run_cache_read(const CacheArgs& c, const PageTable& table, const Rows& k,
                           const Rows& v, bool bf16, int64_t batch, int64_t tokens,
                           const int32_t* start, const int32_t* count, cudaStream_t stream,
                           int* launches);

// Attention of q [batch, tokens, heads, head_dim] over the cache (mx_cache_attention).
struct AttnArgs {
  CacheArgs c;
  PageTable table;
  Rows q, out;
  int64_t batch, tokens;
  int heads;
  const int32_t* length;
  const int32_t* count;   // null: tokens for every sequence
  const uint64_t* tree;   // null: a chain (token t sees tokens 0 .. t)
  float scale;            // of the scores (before the cache's factors)
  float* lse;             // null: not written
  void* workspace;
};
size_t attention_workspace_bytes(int64_t batch, int64_t tokens, int heads, int kv_heads,
                                 int head_dim);
cudaError_t run_cache_attention(const AttnArgs& a, cudaStream_t stream, int* launches);
// The count of attention thread blocks whose bounded waits have run out since the last call.
cudaError_t attention_gave_up(unsigned int* count);

}  // namespace mxk
