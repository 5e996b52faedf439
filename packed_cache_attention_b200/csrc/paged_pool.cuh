// What the kernels on a paged pool share: its description, the check of its header, and the small
// scans that share out a ragged batch.
#pragma once

#include "common.cuh"
#include "paged_split.h"

namespace kvq {

constexpr uint32_t kPagedMagic = 0x5051564Bu;    // "KVQP"
constexpr int kPagedMaxBatch = 1024;

// A pool and the batch's pages in it.
struct PagedArgs {
  const int32_t* block_table;
  const int32_t* seq_lens;
  int64_t table_stride;
  int batch, max_pages;
  int n_pages, page_tiles, n_kv_heads;
  int bits_k, bits_v, rec_bytes, hdr_bytes;
};

// 0 if the pool's header fields name this layout, these shapes and widths and carry no status;
// else the status a call on the pool reports. Digests are compared by the caller. Every
// field is loaded before any is compared, so the loads overlap. An append passes over a
// KVQ_ERR_RANGE: a CTA of its own grid may have just recorded it, and which of the call's
// other tiles are written must not depend on when a CTA starts.
template <bool kAppend = false>
__device__ __forceinline__ unsigned paged_header_code(const uint8_t* pool, const PagedArgs& a) {
  const uint4 h0 = __ldcg(reinterpret_cast<const uint4*>(pool)), h1 = __ldcg(reinterpret_cast<const uint4*>(pool + 16));
  const uint32_t want2 = static_cast<uint32_t>(a.bits_k) | (static_cast<uint32_t>(a.bits_v) << 8);
  if (h0.w != 0 && !(kAppend && h0.w == KVQ_ERR_RANGE)) return h0.w;
  const bool ok = (h0.x == kPagedMagic) & (h0.y == (1u | (kD << 16))) & ((h0.z & 0xffffu) == want2) &
                  (static_cast<int>(h1.x) == a.n_pages) & (static_cast<int>(h1.y) == a.n_kv_heads) &
                  (static_cast<int>(h1.z) == a.page_tiles * kTile) & (static_cast<int>(h1.w) == a.rec_bytes);
  return ok ? 0u : static_cast<unsigned>(KVQ_ERR_MISMATCH);
}
__device__ __forceinline__ uint64_t paged_digest(const uint8_t* pool, int h) {
  return __ldcg(reinterpret_cast<const unsigned long long*>(pool + sizeof(kvq_packed_header)) + h);
}

// Exclusive sum of v over the CTA's threads in order (n_warps warps); `total` is the whole sum.
// `part` holds n_warps ints of shared memory. Two barriers.
__device__ __forceinline__ int block_exclusive(int v, int* part, int n_warps, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += x;
  }
  if (lane == 31) part[warp] = inc;
  __syncthreads();
  int before = 0;
  total = 0;
  for (int w = 0; w < n_warps; ++w) {
    if (w < warp) before += part[w];
    total += part[w];
  }
  __syncthreads();
  return before + inc - v;
}

}  // namespace kvq
