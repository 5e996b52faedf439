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

// Positions of up to 32 tokens, one lane each, for the axes of the lane's blocks 2 lane and 2 lane + 1.
struct RowPositions {
  int p[4];                                          // this lane's token, per axis
  int a0, a1;                                        // axes of the lane's blocks
  __device__ __forceinline__ void load(const RopeArgs& r, int64_t tok, bool live, int lane) {
    a0 = r.axis[2 * lane];
    a1 = r.axis[2 * lane + 1];
#pragma unroll
    for (int a = 0; a < 4; ++a) p[a] = (a < r.n_axes && live) ? __ldg(r.positions + a * r.axis_stride + tok) : 0;
  }
  // Positions of the token held by lane `src`, for the two blocks. Called by the whole warp.
  __device__ __forceinline__ int2 of(const RopeArgs& r, int src) const {
    int q0 = __shfl_sync(0xffffffffu, p[0], src), q1 = q0;
#pragma unroll
    for (int a = 1; a < 4; ++a) {
      if (a >= r.n_axes) break;
      const int q = __shfl_sync(0xffffffffu, p[a], src);
      if (a0 == a) q0 = q;
      if (a1 == a) q1 = q;
    }
    return make_int2(q0, q1);
  }
};

// One row's blocks 2 lane and 2 lane + 1 rotated in a staged row and rounded to its type.
template <int DT>
__device__ __forceinline__ void rotate_row(uint32_t* x, float2 c0, float2 c1, int lane) {
  float a1, a2, b1, b2;
  if constexpr (DT == KVQ_F32) {
    float2* lo = reinterpret_cast<float2*>(x) + lane;
    float2* hi = lo + kH / 2;
    const float2 v1 = *lo, v2 = *hi;
    rotate_pair(v1.x, v2.x, c0, a1, a2);
    rotate_pair(v1.y, v2.y, c1, b1, b2);
    *lo = make_float2(a1, b1);
    *hi = make_float2(a2, b2);
  } else {
    const float2 v1 = word_to_pair<DT>(x[lane]), v2 = word_to_pair<DT>(x[lane + kH / 2]);
    rotate_pair(v1.x, v2.x, c0, a1, a2);
    rotate_pair(v1.y, v2.y, c1, b1, b2);
    x[lane] = pair_to_word<DT>(a1, b1);
    x[lane + kH / 2] = pair_to_word<DT>(a2, b2);
  }
}

__device__ __forceinline__ bool outside(const RopeArgs& r, int2 p) {
  return (static_cast<unsigned>(p.x) >= static_cast<unsigned>(r.n_positions)) |
         (static_cast<unsigned>(p.y) >= static_cast<unsigned>(r.n_positions));
}

// Rotates rows r_lo .. r_hi - 1 of a staged K tile in place; row r_lo is token tok0 of the call. True if
// a position was outside the table. Where every lane's two blocks share an axis (one axis, or
// sections of even length) and every position is inside, a row takes one 16-byte load of angles
// per lane and no checks, 16 rows in flight; with two 8-byte loads and checks per row the rotation
// took 40 us of 131072 tokens x 2 heads, for its instructions more than its latency.
template <int DT>
__device__ __forceinline__ bool rotate_tile(uint32_t* tile, const RopeArgs& r, int64_t tok0, int r_lo, int r_hi, int lane) {
  using Q = QTile<DT>;
  RowPositions pos;
  pos.load(r, tok0 + lane - r_lo, lane >= r_lo && lane < r_hi, lane);
  bool off = false;
#pragma unroll
  for (int a = 0; a < 4; ++a) off |= a < r.n_axes && static_cast<unsigned>(pos.p[a]) >= static_cast<unsigned>(r.n_positions);
  if (__all_sync(0xffffffffu, !off && pos.a0 == pos.a1)) {
    constexpr int kAhead = 16;
    const float4* table = reinterpret_cast<const float4*>(r.table) + lane;
#pragma unroll 1
    for (int row = r_lo; row < r_hi; row += kAhead) {
      float4 c[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) c[u] = __ldg(table + static_cast<int64_t>(pos.of(r, min(row + u, r_hi - 1)).x) * (kH / 2));
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        if (row + u >= r_hi) break;
        rotate_row<DT>(tile + (row + u) * Q::kPitch, make_float2(c[u].x, c[u].y), make_float2(c[u].z, c[u].w), lane);
      }
    }
    return false;
  }
  constexpr int kAhead = 4;
#pragma unroll 1
  for (int row = r_lo; row < r_hi; row += kAhead) {
    float2 c0[kAhead], c1[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int2 q = pos.of(r, min(row + u, r_hi - 1));
      c0[u] = rope_cs(r, q.x, 2 * lane);
      c1[u] = rope_cs(r, q.y, 2 * lane + 1);
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (row + u >= r_hi) break;
      rotate_row<DT>(tile + (row + u) * Q::kPitch, c0[u], c1[u], lane);
    }
  }
  return off;
}

// ---------------------------------------------------------------- tiles that get few tokens

// A decode step brings one token per sequence. Taking it through the tile path costs what 32 cost (a lane
// per token for the keys, 32 tokens per dim for the values); for up to kFewRows tokens the warp
// instead shares out each row's dims: lane l owns blocks 2l and 2l + 1 of keys and values.
constexpr int kFewRows = 4;

// Codes of a pair for a width known at run time: quantize.cuh's table lookup.
__device__ __forceinline__ uint2 lut_code2_any(int w, float2 y, uint32_t lut_s) {
  if (w == 1) return make_uint2(y.x > 0.0f ? 1u : 0u, y.y > 0.0f ? 1u : 0u);
  switch (w) {
    case 2: return lut_code2<2>(y, lut_s);
    case 3: return lut_code2<3>(y, lut_s);
    case 4: return lut_code2<4>(y, lut_s);
    case 5: return lut_code2<5>(y, lut_s);
    case 6: return lut_code2<6>(y, lut_s);
    case 7: return lut_code2<7>(y, lut_s);
    default: return lut_code2<8>(y, lut_s);
  }
}

__device__ __forceinline__ uint32_t shl_clamp(uint32_t x, uint32_t n) {
  uint32_t y;
  asm("shl.b32 %0, %1, %2;" : "=r"(y) : "r"(x), "r"(n));   // 0 from 32 on
  return y;
}
__device__ __forceinline__ uint32_t shr_clamp(uint32_t x, uint32_t n) {
  uint32_t y;
  asm("shr.b32 %0, %1, %2;" : "=r"(y) : "r"(x), "r"(n));
  return y;
}

// fp16 norm and scale of one row whose dims 2l, 2l + 1, 64 + 2l, 65 + 2l lane l holds: the sum of
// squares in the quantizer's order (lane r of 8 sums the dims of residue r in ascending order).
__device__ __forceinline__ void spread_norm_scale(float2 lo, float2 hi, float* row, int lane, __half& n16, float& a) {
  reinterpret_cast<float2*>(row)[lane] = lo;
  reinterpret_cast<float2*>(row)[lane + 32] = hi;
  __syncwarp();
  float s = 0.0f;
  if (lane < 8) {
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const float x = row[8 * j + lane];
      s = __fadd_rn(s, __fmul_rn(x, x));
    }
  }
  s = __fadd_rn(s, __shfl_xor_sync(0xffffffffu, s, 1));
  s = __fadd_rn(s, __shfl_xor_sync(0xffffffffu, s, 2));
  s = __fadd_rn(s, __shfl_xor_sync(0xffffffffu, s, 4));
  s = __shfl_sync(0xffffffffu, s, 0);
  n16 = __float2half_rn(__fsqrt_rn(s));
  const float nf = __half2float(n16);
  a = (nf == 0.0f) ? 0.0f : __fdiv_rn(11.313708305358887f, nf);   // fp32(sqrt(128)) / norm
  __syncwarp();                                      // the row may be overwritten
}

// Dims 2l, 2l + 1 (half 0) or 64 + 2l, 65 + 2l (half 1) of a row in global memory.
template <int DT>
__device__ __forceinline__ float2 row_pair(const uint8_t* row, int half, int lane) {
  if constexpr (DT == KVQ_F32) return __ldg(reinterpret_cast<const float2*>(row) + lane + 32 * half);
  else return word_to_pair<DT>(__ldg(reinterpret_cast<const uint32_t*>(row) + lane + 32 * half));
}

// Rows r_lo .. r_hi - 1 of one tile (at most kFewRows; row r_lo at `krow`, `vrow`), stored as the
// tile path stores them. `scratch`: 128 floats, then kFewRows x 32 words. True if a position was
// outside the table.
template <int DT, int BVT>
__device__ __forceinline__ bool append_few(const uint8_t* krow, const uint8_t* vrow, int64_t kstep, int64_t vstep,
                                           const RopeArgs& rope, int64_t tok0, int r_lo, int r_hi, const kvq_head_alloc* al,
                                           uint8_t* rec, int bits_k, float* scratch, uint32_t lut_s, int lane) {
  const int n = r_hi - r_lo, n_words = 4 * bits_k;
  uint32_t* words = reinterpret_cast<uint32_t*>(scratch + kD);
  uint32_t* kout = reinterpret_cast<uint32_t*>(rec);
  uint16_t* norms = reinterpret_cast<uint16_t*>(kout + bits_k * kD);
  uint32_t* vout = kout + bits_k * kD + kTile;
  // the words of this lane's dims that the new codes share with stored ones
  const int keep = BVT * r_lo, wk = keep >> 5;
  uint2 old0 = make_uint2(0u, 0u), old1 = old0;
  if (keep & 31) {
    old0 = *reinterpret_cast<const uint2*>(vout + wk * kD + 2 * lane);
    old1 = *reinterpret_cast<const uint2*>(vout + wk * kD + kH + 2 * lane);
  }
  const int f0 = al->bit_off[2 * lane], f1 = al->bit_off[2 * lane + 1];
  // (a block that would not end inside the key stream is left out: the words are the warp's own memory)
  auto width = [&](int w, int f) { return w <= 8 && f >= 0 && f + 2 * w <= bits_k * kD ? w : 0; };
  const int w0 = width(al->width[2 * lane], f0), w1 = width(al->width[2 * lane + 1], f1);
  const float2 g = *reinterpret_cast<const float2*>(al->gain + 2 * lane);
  float2 kl[kFewRows], kh[kFewRows], vl[kFewRows], vh[kFewRows];
#pragma unroll
  for (int i = 0; i < kFewRows; ++i) {
    if (i >= n) break;
    kl[i] = row_pair<DT>(krow + i * kstep, 0, lane);
    kh[i] = row_pair<DT>(krow + i * kstep, 1, lane);
    vl[i] = row_pair<DT>(vrow + i * vstep, 0, lane);
    vh[i] = row_pair<DT>(vrow + i * vstep, 1, lane);
  }
  bool bad = false;
  RowPositions pos;
  if (rope.n_positions > 0) pos.load(rope, tok0 + lane, lane < n, lane);
  for (int i = lane; i < kFewRows * 32; i += 32) words[i] = 0u;
  uint16_t kn = 0, vn = 0;                           // of the token that this lane stores
  uint32_t v0[BVT], v1[BVT], v2[BVT], v3[BVT];
#pragma unroll
  for (int i = 0; i < BVT; ++i) v0[i] = v1[i] = v2[i] = v3[i] = 0u;
#pragma unroll
  for (int i = 0; i < kFewRows; ++i) {
    if (i >= n) break;
    __half n16;
    float a;
    // ---- key
    float2 lo = kl[i], hi = kh[i];
    if (rope.n_positions > 0) {
      const int2 q = pos.of(rope, i);
      bad |= outside(rope, q);
      const float2 c0 = rope_cs(rope, q.x, 2 * lane), c1 = rope_cs(rope, q.y, 2 * lane + 1);
      float2 nl, nh;
      rotate_pair(lo.x, hi.x, c0, nl.x, nh.x);
      rotate_pair(lo.y, hi.y, c1, nl.y, nh.y);
      lo = nl;
      hi = nh;
      if constexpr (DT != KVQ_F32) {
        lo = word_to_pair<DT>(pair_to_word<DT>(lo.x, lo.y));
        hi = word_to_pair<DT>(pair_to_word<DT>(hi.x, hi.y));
      }
    }
    spread_norm_scale(lo, hi, scratch, lane, n16, a);
    if (lane == r_lo + i) kn = __half_as_ushort(n16);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int w = u ? w1 : w0, f = u ? f1 : f0;
      if (w == 0) continue;
      const float2 x = u ? make_float2(lo.y, hi.y) : make_float2(lo.x, hi.x);
      const float gb = u ? g.y : g.x;
      const uint2 c = lut_code2_any(w, mul2(mul2(x, make_float2(a, a)), make_float2(gb, gb)), lut_s);
      const uint64_t bits = static_cast<uint64_t>(c.x | c.y << w) << (f & 31);
      atomicOr(words + 32 * i + (f >> 5), static_cast<uint32_t>(bits));
      if (bits >> 32) atomicOr(words + 32 * i + (f >> 5) + 1, static_cast<uint32_t>(bits >> 32));
    }
    // ---- value
    spread_norm_scale(vl[i], vh[i], scratch, lane, n16, a);
    if (lane == r_lo + i) vn = __half_as_ushort(n16);
    const uint2 ca = lut_code2<BVT>(mul2(vl[i], make_float2(a, a)), lut_s);
    const uint2 cb = lut_code2<BVT>(mul2(vh[i], make_float2(a, a)), lut_s);
    const int bit = BVT * (r_lo + i);
#pragma unroll
    for (int j = 0; j < BVT; ++j) {
      const int sh = bit - 32 * j;                   // from its first bit on, or what the word before left
      const uint32_t up = static_cast<uint32_t>(max(sh, 0)), down = static_cast<uint32_t>(max(-sh, 0));
      v0[j] |= shr_clamp(shl_clamp(ca.x, up), down);
      v1[j] |= shr_clamp(shl_clamp(ca.y, up), down);
      v2[j] |= shr_clamp(shl_clamp(cb.x, up), down);
      v3[j] |= shr_clamp(shl_clamp(cb.y, up), down);
    }
  }
  __syncwarp();
  const bool mine = lane >= r_lo, valid = mine && lane < r_hi;
  for (int i = 0; i < n_words; ++i) {
    const uint32_t v = valid ? words[32 * (lane - r_lo) + i] : 0u;
    if (mine) kout[i * kTile + lane] = v;
  }
  if (mine) {
    norms[lane] = kn;
    norms[kTile + lane] = vn;
  }
  const uint32_t m = (1u << (keep & 31)) - 1u;
#pragma unroll
  for (int j = 0; j < BVT; ++j) {
    if (j < wk) continue;                            // stored codes alone
    if (j == wk) {
      v0[j] |= old0.x & m;
      v1[j] |= old0.y & m;
      v2[j] |= old1.x & m;
      v3[j] |= old1.y & m;
    }
    *reinterpret_cast<uint2*>(vout + j * kD + 2 * lane) = make_uint2(v0[j], v1[j]);
    *reinterpret_cast<uint2*>(vout + j * kD + kH + 2 * lane) = make_uint2(v2[j], v3[j]);
  }
  __syncwarp();                                      // the scratch is free
  return bad;
}

// Dynamic shared memory: the quantizer's, then the scan of the batch's tiles.
inline size_t append_smem_bytes(int dtype, int batch) { return quant_smem_bytes(dtype) + 4 * (16 + batch + 1); }

// Append of a ragged batch. Persistent warps; a task is one 32-token tile of one sequence that
// gets tokens, for one KV head (heads inner, so a tile's rows and angles are read while they
// are in cache). K and V tiles are staged as in kvq_quant_pack, half a task ahead; the K
// tile is rotated in shared memory before its norms are taken. A tile that gets up to kFewRows
// tokens goes by rows instead.
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
      // (the digest does not cover the budget: a pool may have been given an allocation of another one)
      if ((paged_digest(p.pool, h) != p.alloc[h].digest) | (p.alloc[h].bits_k != a.bits_k) | (p.alloc[h].k_words != a.bits_k * kD))
        code = KVQ_ERR_MISMATCH;
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
  long long task = static_cast<long long>(warp) * gridDim.x + blockIdx.x;   // spread over the SMs first

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
  auto few = [](const Task& t) { return t.r_hi - t.r_lo <= kFewRows; };
  auto load_k = [&](const Task& t) {
    if (few(t)) return;
    tile_load_async<DT>(kbuf, reinterpret_cast<const T*>(p.K) + t.h * p.ksh + t.tok0 * p.kst, p.kst, t.r_lo, t.r_hi, lane);
  };
  auto load_v = [&](const Task& t) {
    if (few(t)) return;
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
      n_cls = min(max(al->n_classes, 0), 8);
      if (lane < 8)
        sCls[lane] = static_cast<uint32_t>(al->class_width[lane]) | (static_cast<uint32_t>(al->class_first[lane]) << 8) |
                     (static_cast<uint32_t>(al->class_blocks[lane]) << 16);
      __syncwarp();
      cur_h = cur.h;
    }
    const bool write = cur.rec != nullptr, by_rows = few(cur);
    if (by_rows && write) {
      const int64_t es = sizeof(T);
      if (append_few<DT, BVT>(p.K + es * (cur.h * p.ksh + cur.tok0 * p.kst), p.V + es * (cur.h * p.vsh + cur.tok0 * p.vst),
                              es * p.kst, es * p.vst, rope, cur.tok0, cur.r_lo, cur.r_hi, p.alloc + cur.h, cur.rec, a.bits_k,
                              reinterpret_cast<float*>(kbuf), lut_s, lane))
        atomicCAS(status, 0u, static_cast<uint32_t>(KVQ_ERR_RANGE));
    }
    uint32_t* kout = reinterpret_cast<uint32_t*>(cur.rec);
    uint16_t* norms = reinterpret_cast<uint16_t*>(kout + k_words);   // 32 K norms, then 32 V norms
    uint32_t* vout = kout + k_words + kTile;

    // ---------------------------------------------------------------- K (rotation, Block-GTQ widths)
    cp_async_wait<1>();                              // this task's K rows (its V rows may be in flight)
    __syncwarp();
    if (write && !by_rows) {
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
    if (write && !by_rows) {
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
