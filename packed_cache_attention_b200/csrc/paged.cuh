// Paged packed cache: the pool's header, and the append that rotates, quantizes and packs a
// ragged batch's new tokens into its pages.
//
// A pool is a header (kvq_packed_header with magic "KVQP", then one allocation digest per KV
// head) and n_pages pages; a page is, per KV head, page_tokens / 32 of the tile records that
// the quantizer writes (quantize.cuh). The quantizer's arithmetic is used as it is, so a
// paged cache holds the bytes that a contiguous one would.
#pragma once

#include "common.cuh"
#include "paged_pool.cuh"
#include "quantize.cuh"
#include "rope.cuh"

namespace kvq {

// One CTA writes the header.
__global__ void kvq_paged_header(uint8_t* pool, PagedArgs a, const kvq_head_alloc* alloc) {
  grid_dependency_wait();
  uint32_t* w = reinterpret_cast<uint32_t*>(pool);
  for (int i = threadIdx.x; i < a.hdr_bytes / 4; i += blockDim.x) {
    uint32_t v = 0u;
    if (i == 0) v = kPagedMagic;
    else if (i == 1) v = 1u | (static_cast<uint32_t>(kD) << 16);           // layout 1, head_dim
    else if (i == 2) v = static_cast<uint32_t>(a.bits_k) | (static_cast<uint32_t>(a.bits_v) << 8) |
                         (static_cast<uint32_t>(alloc->w_max & 0xff) << 16) |
                         (static_cast<uint32_t>(alloc->mode & 0xff) << 24);
    else if (i == 4) v = static_cast<uint32_t>(a.n_pages);
    else if (i == 5) v = static_cast<uint32_t>(a.n_kv_heads);
    else if (i == 6) v = static_cast<uint32_t>(a.page_tiles * kTile);
    else if (i == 7) v = static_cast<uint32_t>(a.rec_bytes);
    else if (i >= 16 && i < 16 + 2 * a.n_kv_heads) {
      const uint64_t d = alloc[(i - 16) >> 1].digest;
      v = static_cast<uint32_t>((i & 1) ? (d >> 32) : d);
    }
    w[i] = v;
  }
}

struct PagedQuant {
  const uint8_t* K;
  const uint8_t* V;
  int64_t ksh, kst, vsh, vst;        // strides in elements
  int n_tokens;
  const int32_t* cu;
  const kvq_head_alloc* alloc;
  uint8_t* pool;
};

// Rotates rows r_lo .. r_hi - 1 of a staged K tile in place, rounding to the tile's type. Lane l
// owns blocks 2l and 2l + 1 of every row; row r_lo is token tok0 of the call.
template <int DT>
__device__ __forceinline__ bool rotate_tile(uint32_t* tile, const RopeArgs& r, int64_t tok0, int r_lo, int r_hi, int lane) {
  using Q = QTile<DT>;
  const int32_t* p0 = r.positions + r.axis[2 * lane] * r.axis_stride + tok0 - r_lo;
  const int32_t* p1 = r.positions + r.axis[2 * lane + 1] * r.axis_stride + tok0 - r_lo;
  bool bad = false;
  constexpr int kAhead = 4;                                // rows whose angles are loaded together
  for (int row = r_lo; row < r_hi; row += kAhead) {
    float2 c0[kAhead], c1[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int i = min(row + u, r_hi - 1);
      const int a = __ldg(p0 + i), b = __ldg(p1 + i);
      bad |= (static_cast<unsigned>(a) >= static_cast<unsigned>(r.n_positions)) |
             (static_cast<unsigned>(b) >= static_cast<unsigned>(r.n_positions));
      c0[u] = rope_cs(r, a, 2 * lane);
      c1[u] = rope_cs(r, b, 2 * lane + 1);
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (row + u >= r_hi) break;
      uint32_t* x = tile + (row + u) * Q::kPitch;
      float a1, a2, b1, b2;
      if constexpr (DT == KVQ_F32) {
        float2* lo = reinterpret_cast<float2*>(x) + lane;
        float2* hi = lo + kH / 2;
        const float2 v1 = *lo, v2 = *hi;
        rotate_pair(v1.x, v2.x, c0[u], a1, a2);
        rotate_pair(v1.y, v2.y, c1[u], b1, b2);
        *lo = make_float2(a1, b1);
        *hi = make_float2(a2, b2);
      } else {
        const float2 v1 = word_to_pair<DT>(x[lane]), v2 = word_to_pair<DT>(x[lane + kH / 2]);
        rotate_pair(v1.x, v2.x, c0[u], a1, a2);
        rotate_pair(v1.y, v2.y, c1[u], b1, b2);
        x[lane] = pair_to_word<DT>(a1, b1);
        x[lane + kH / 2] = pair_to_word<DT>(a2, b2);
      }
    }
  }
  return bad;
}

// Dynamic shared memory: the quantizer's, then the scan of the batch's tiles.
inline size_t append_smem_bytes(int dtype, int batch) { return quant_smem_bytes(dtype) + 4 * (16 + batch + 1); }

// Append of a ragged batch. Persistent warps; a task is one 32-token tile of one sequence that
// gets tokens, for one KV head (heads inner, so a tile's rows and angles are read while they
// are in cache). K and V tiles are staged as in kvq_quant_pack, half a task ahead; the K
// tile is rotated in shared memory before its norms are taken.
template <int DT, int BVT>
__global__ void __launch_bounds__(QTile<DT>::kWarps * 32, 1) kvq_paged_quant(const PagedArgs a, const PagedQuant p,
                                                                             const RopeArgs rope) {
  using Q = QTile<DT>;
  using T = typename Elem<DT>::T;
  constexpr int kWarps = Q::kWarps;
  extern __shared__ __align__(16) uint8_t smem[];
  // (all of it dynamic: a static part is padded to 1 KB, which would not fit)
  int* sPart = reinterpret_cast<int*>(smem + quant_smem_bytes(DT));   // kWarps
  unsigned& sCode = *reinterpret_cast<unsigned*>(sPart + 12);
  int* sTile = sPart + 16;                           // batch + 1: tiles of the sequences before each
  uint2* sLut = reinterpret_cast<uint2*>(smem);
  for (int i = threadIdx.x; i < kLutEntries; i += blockDim.x)
    sLut[i] = make_uint2(g_quant_lut[2 * i], g_quant_lut[2 * i + 1]);
  const uint32_t lut_s = static_cast<uint32_t>(__cvta_generic_to_shared(sLut));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) sCode = 0u;
  // The table is the library's own; the caller's memory is touched only after the previous
  // kernel in the stream is done with it (programmatic dependent launch).
  grid_dependency_wait();
  uint32_t* status = reinterpret_cast<uint32_t*>(p.pool + offsetof(kvq_packed_header, status));
  __syncthreads();
  {
    unsigned code = (threadIdx.x == 0) ? paged_header_code<true>(p.pool, a) : 0u;
    for (int h = threadIdx.x; h < a.n_kv_heads; h += blockDim.x)
      if (paged_digest(p.pool, h) != p.alloc[h].digest) code = KVQ_ERR_MISMATCH;
    if (code) atomicCAS(&sCode, 0u, code);
  }
  // Tiles per sequence. A sequence whose rows or positions do not fit gets none.
  const long long room = static_cast<long long>(a.max_pages) * a.page_tiles * kTile;
  int n_total = 0;
  for (int b0 = 0; b0 < a.batch; b0 += kWarps * 32) {
    const int b = b0 + threadIdx.x;
    int n = 0;
    if (b < a.batch) {
      const int c0 = __ldg(p.cu + b), c1 = __ldg(p.cu + b + 1), len = __ldg(a.seq_lens + b);
      if (c0 < 0 || c1 < c0 || c1 > p.n_tokens || len < 0 || static_cast<long long>(len) + (c1 - c0) > room) {
        atomicCAS(status, 0u, static_cast<uint32_t>(KVQ_ERR_RANGE));
      } else if (c1 > c0) {
        n = (len + (c1 - c0) + kTile - 1) / kTile - len / kTile;
      }
    }
    int total;
    const int before = block_exclusive(n, sPart, kWarps, total);
    if (b < a.batch) sTile[b] = n_total + before;
    n_total += total;
  }
  if (threadIdx.x == 0) sTile[a.batch] = n_total;
  __syncthreads();
  if (sCode) {
    if (threadIdx.x == 0) atomicCAS(status, 0u, sCode);
    return;
  }
  const long long n_tasks = static_cast<long long>(n_total) * a.n_kv_heads;
  uint8_t* records = p.pool + a.hdr_bytes;
  const int k_words = a.bits_k * kD;
  uint8_t* wbase = smem + kLutEntries * 8 + warp * QWarpSmem<DT>::kBytes;
  uint32_t* kbuf = reinterpret_cast<uint32_t*>(wbase);
  uint32_t* vbuf = kbuf + Q::kWords;
  float2* sA2 = reinterpret_cast<float2*>(vbuf + Q::kWords);
  KEntry* sEnt = reinterpret_cast<KEntry*>(sA2 + kTile);
  uint32_t* sCls = reinterpret_cast<uint32_t*>(sEnt + kKEntries);     // width | first << 8 | blocks << 16
  const uint32_t* myv = vbuf + lane * Q::kPitch;
  int cur_h = -1, n_cls = 0;

  const long long stride = static_cast<long long>(gridDim.x) * kWarps;
  long long task = static_cast<long long>(blockIdx.x) * kWarps + warp;

  // A task's head, record, the rows of the tile it writes [r_lo, r_hi) and the call's token of r_lo.
  struct Task {
    int h, r_lo, r_hi, tok0;
    uint8_t* rec;                                    // null: the page is outside the pool
  };
  auto task_of = [&](long long tk) {
    Task t;
    const int tq = static_cast<int>(tk / a.n_kv_heads);
    t.h = static_cast<int>(tk - static_cast<long long>(tq) * a.n_kv_heads);
    const int b = find_span(sTile, a.batch, tq);
    const int len = __ldg(a.seq_lens + b), c0 = __ldg(p.cu + b), n = __ldg(p.cu + b + 1) - c0;
    const int tile = len / kTile + tq - sTile[b];
    const int t0 = tile * kTile;
    t.r_lo = max(0, len - t0);
    t.r_hi = min(kTile, len + n - t0);
    t.tok0 = c0 + t0 + t.r_lo - len;
    const int slot = tile / a.page_tiles;
    const int page = __ldg(a.block_table + b * a.table_stride + slot);
    t.rec = nullptr;
    if (static_cast<unsigned>(page) < static_cast<unsigned>(a.n_pages))
      t.rec = records + ((static_cast<size_t>(page) * a.n_kv_heads + t.h) * a.page_tiles + (tile - slot * a.page_tiles)) *
                            a.rec_bytes;
    else if (lane == 0)
      atomicCAS(status, 0u, static_cast<uint32_t>(KVQ_ERR_RANGE));
    return t;
  };
  auto load_k = [&](const Task& t) {
    tile_load_async<DT>(kbuf, reinterpret_cast<const T*>(p.K) + t.h * p.ksh + t.tok0 * p.kst, p.kst, t.r_lo, t.r_hi, lane);
  };
  auto load_v = [&](const Task& t) {
    tile_load_async<DT>(vbuf, reinterpret_cast<const T*>(p.V) + t.h * p.vsh + t.tok0 * p.vst, p.vst, t.r_lo, t.r_hi, lane);
  };

  Task cur{}, nxt{};
  if (task < n_tasks) {
    cur = task_of(task);
    load_k(cur);
    cp_async_commit();
    load_v(cur);
    cp_async_commit();
  }
  for (; task < n_tasks; task += stride) {
    const bool more = task + stride < n_tasks;
    if (more) nxt = task_of(task + stride);
    const bool mine = lane >= cur.r_lo;              // token written by this call (or past its end)
    const bool valid = mine && lane < cur.r_hi;      // token quantized by this call
    if (cur.h != cur_h) {
      const kvq_head_alloc* al = p.alloc + cur.h;
      for (int i = lane; i < kKEntries; i += 32) {
        const int blk = (i < kH) ? al->stream_block[i] : 0xff;
        KEntry e{0x1044u, 0.0f};
        if (blk < kH) {
          const float g = al->gain[blk];
          if constexpr (DT == KVQ_F32) e = KEntry{(4u * blk) << 16, g};
          else if constexpr (DT == KVQ_BF16) e = KEntry{((4u * (blk >> 1)) << 16) | ((blk & 1) ? 0x3244u : 0x1044u), g};
          else e = KEntry{((4u * (blk >> 1)) << 16) | ((blk & 1) ? 0x7632u : 0x5410u), g};
        }
        sEnt[i] = e;
      }
      n_cls = al->k_words == k_words ? min(max(al->n_classes, 0), 8) : -1;   // -1: made for another budget
      if (lane < 8)
        sCls[lane] = static_cast<uint32_t>(al->class_width[lane]) | (static_cast<uint32_t>(al->class_first[lane]) << 8) |
                     (static_cast<uint32_t>(al->class_blocks[lane]) << 16);
      __syncwarp();
      cur_h = cur.h;
    }
    const bool write = cur.rec != nullptr && n_cls >= 0;
    uint32_t* kout = reinterpret_cast<uint32_t*>(cur.rec);
    uint16_t* norms = reinterpret_cast<uint16_t*>(kout + k_words);   // 32 K norms, then 32 V norms
    uint32_t* vout = kout + k_words + kTile;

    // ---------------------------------------------------------------- K (rotation, Block-GTQ widths)
    cp_async_wait<1>();                              // this task's K rows (its V rows may be in flight)
    __syncwarp();
    if (write) {
      if (rope.n_positions > 0) {
        if (rotate_tile<DT>(kbuf, rope, cur.tok0, cur.r_lo, cur.r_hi, lane))
          atomicCAS(status, 0u, static_cast<uint32_t>(KVQ_ERR_RANGE));
        __syncwarp();
      }
      __half n16;
      float sc;
      const uint32_t* myk = kbuf + lane * Q::kPitch;
      row_norm_scale<DT>(myk, n16, sc);
      if (mine) norms[lane] = valid ? __half_as_ushort(n16) : 0;
      if (!valid) sc = __int_as_float(0x7fc00000);   // NaN: every code is 0
      const float2 aa = make_float2(sc, sc);
      const uint8_t* row = reinterpret_cast<const uint8_t*>(myk);
      KStream ks;
      ks.store = mine;
      for (int c = 0; c < n_cls; ++c) {
        const uint32_t e = sCls[c];
        const int w = e & 0xffu, first = (e >> 8) & 0xffu, nb = e >> 16;
        const KEntry* ent = sEnt + first;
        switch (w) {
          case 1: quant_k_class<DT, 1>(row, aa, ent, nb, lut_s, ks, kout, lane); break;
          case 2: quant_k_class<DT, 2>(row, aa, ent, nb, lut_s, ks, kout, lane); break;
          case 3: quant_k_class<DT, 3>(row, aa, ent, nb, lut_s, ks, kout, lane); break;
          case 4: quant_k_class<DT, 4>(row, aa, ent, nb, lut_s, ks, kout, lane); break;
          case 5: quant_k_class<DT, 5>(row, aa, ent, nb, lut_s, ks, kout, lane); break;
          case 6: quant_k_class<DT, 6>(row, aa, ent, nb, lut_s, ks, kout, lane); break;
          case 7: quant_k_class<DT, 7>(row, aa, ent, nb, lut_s, ks, kout, lane); break;
          default: quant_k_class<DT, 8>(row, aa, ent, nb, lut_s, ks, kout, lane); break;
        }
      }
    }
    __syncwarp();                                    // every lane is done with the K tile
    if (more) load_k(nxt);
    cp_async_commit();

    // ---------------------------------------------------------------- V (uniform width)
    cp_async_wait<1>();                              // this task's V rows (next K rows may be in flight)
    __syncwarp();
    if (write) {
      __half n16;
      float sc;
      row_norm_scale<DT>(myv, n16, sc);
      if (mine) norms[kTile + lane] = valid ? __half_as_ushort(n16) : 0;
      if (!valid) sc = __int_as_float(0x7fc00000);
      sA2[lane] = make_float2(sc, sc);
      __syncwarp();
      quant_v_tile<DT, BVT>(vbuf, sA2, lut_s, vout, a.bits_v * cur.r_lo, lane);
    }
    __syncwarp();                                    // every lane is done with the V tile and sA2
    if (more) load_v(nxt);
    cp_async_commit();
    cur = nxt;
  }
  allow_dependents();                                // this warp has no task left
  asm volatile("cp.async.wait_all;" ::: "memory");
}

}  // namespace kvq
