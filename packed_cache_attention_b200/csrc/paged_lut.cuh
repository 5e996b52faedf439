// Dequantization of tile records in the paged attention kernels: centroid lookups in shared
// memory, and the copies that bring tiles out of their pages.
//
// A lookup turns the 2w bits of two consecutive codes into one word of two fp16 centroids. For
// widths 1..4 every lane has its own copy of the table (entry i of lane l at word 32 i + l), so
// 32 lanes never share a bank; with one shared copy of width 4's 256 entries a warp's lookup
// takes 3.5 passes on average. A field is moved to bit 7 of a word by one funnel shift, masked and
// joined with the lane and the table's base by one three-input operation, and is then the
// entry's byte address: three instructions a pair. Width 5 (4 KB) has one copy, its fields at bit 2;
// widths 6..8 (the few blocks of the highest energy, or large budgets) take two single lookups.
#pragma once

#include "decode.cuh"
#include "paged_pool.cuh"

namespace kvq {

// Byte offsets of the tables (pair tables: a multiple of their size, so that OR adds them).
__host__ __device__ constexpr int plut_off(int w) {
  return w == 4 ? 0 : w == 3 ? 32768 : w == 2 ? 40960 : w == 1 ? 43008 : w == 6 ? 43520 : w == 7 ? 43648 : w == 8 ? 44032 : 45056;
}
constexpr int kPlutBytes = 49152;
__host__ __device__ constexpr int plut_pos(int w) { return w <= 4 ? 7 : 2; }   // bit position of a field

// Host: the image from the fp16 centroid table (width w at c16 + 2^w - 2).
inline void paged_lut_image(const uint16_t* c16, uint8_t* img) {
  std::memset(img, 0, kPlutBytes);
  for (int w = 1; w <= 8; ++w) {
    const uint16_t* c = c16 + (1 << w) - 2;
    if (w > 5) {
      std::memcpy(img + plut_off(w), c, 2u << w);
      continue;
    }
    uint32_t* t = reinterpret_cast<uint32_t*>(img + plut_off(w));
    const int copies = w <= 4 ? 32 : 1;
    for (int e = 0; e < (1 << (2 * w)); ++e)
      for (int l = 0; l < copies; ++l)
        t[e * copies + l] = static_cast<uint32_t>(c[e & ((1 << w) - 1)]) | (static_cast<uint32_t>(c[e >> w]) << 16);
  }
}

__device__ __align__(16) uint8_t g_paged_lut[kPlutBytes];

// ---------------------------------------------------------------- keys

// Descriptor of a plan slot (4 block pairs of one width), read by every lane:
//   x  byte offset of the first stream word of the lane's token (-128 when the field's place
//      reaches back before the stream: what is read there is masked out)
//   y  shift that brings the first code to its place, then 2w, 4w, 6w, one per byte
//   z  mask of a pair in its place (0: a wide slot)
//   w  table base, bit 31 set when the table has a copy per lane; a wide slot: its width
__device__ __forceinline__ uint4 k_slot_desc(uint32_t e, int stream_bits, bool& bad) {
  uint32_t w = e & 15u, off = e >> 8;
  bad = w > 8 || (w > 0 && off >= static_cast<uint32_t>(stream_bits));
  if (bad || w == 0) { w = 1; off = 0; }               // an empty slot: finite values against zero rows of Q'
  const int pos = w <= 5 ? plut_pos(static_cast<int>(w)) : 0;
  const int at = static_cast<int>(off) - pos;
  uint4 d;
  d.x = static_cast<uint32_t>((at >> 5) * 128);
  d.y = (static_cast<uint32_t>(at) & 31u) | (2 * w) << 8 | (4 * w) << 16 | (6 * w) << 24;
  d.z = w <= 5 ? ((1u << (2 * w)) - 1u) << pos : 0u;
  d.w = w <= 5 ? static_cast<uint32_t>(plut_off(static_cast<int>(w))) | (w <= 4 ? 0x80000000u : 0u) : w;
  return d;
}

// One wide slot (widths 6..8) from its two aligned stream words.
__device__ __forceinline__ void k_wide_vals(uint32_t w, uint32_t r0, uint32_t r1, const uint8_t* lut, uint32_t* v) {
  const uint8_t* t = lut + (w == 6 ? plut_off(6) : w == 7 ? plut_off(7) : plut_off(8));
  const uint32_t m = (2u << w) - 2u;                   // a code, doubled
  uint64_t r = (static_cast<uint64_t>(r1) << 32 | r0) << 1;
  const uint32_t top = r1 >> 31;                       // the bit that the doubling pushed out
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t a = static_cast<uint32_t>(r) & m;
    r >>= w;
    if (k == 0) r |= static_cast<uint64_t>(top) << (64 - w);
    const uint32_t b = static_cast<uint32_t>(r) & m;
    r >>= w;
    v[k] = static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(t + a)) |
           static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(t + b)) << 16;
  }
}

// 16 K-hat columns (4 plan slots) of this lane's token; kw points at word 0 of the token (word i
// at byte 128 i). kWide: some slot of the four is wider than 5.
template <bool kWide>
__device__ __forceinline__ void k_vals(const uint8_t* kw, const uint4* desc, const uint8_t* lut, uint32_t lane4,
                                       uint32_t (&v)[16]) {
  uint4 d[4];
  uint32_t r0[4], r1[4], lb[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    d[i] = desc[i];
    const uint32_t* p = reinterpret_cast<const uint32_t*>(kw + static_cast<int>(d[i].x));
    const uint32_t x0 = p[0], x1 = p[32], x2 = p[64];
    r0[i] = __funnelshift_r(x0, x1, d[i].y);
    r1[i] = __funnelshift_r(x1, x2, d[i].y);
    lb[i] = (d[i].w & 0xffffu) | (static_cast<int>(d[i].w) < 0 ? lane4 : 0u);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (kWide && d[i].z == 0u) {
      k_wide_vals(d[i].w, r0[i], r1[i], lut, v + 4 * i);
      continue;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t t = (k == 0) ? r0[i] : __funnelshift_r(r0[i], r1[i], d[i].y >> (8 * k));
      v[4 * i + k] = *reinterpret_cast<const uint32_t*>(lut + ((t & d[i].z) | lb[i]));
    }
  }
}

// ---------------------------------------------------------------- values

template <int W>
__device__ __forceinline__ uint32_t pair_of(uint32_t lo, uint32_t hi, int p, const uint8_t* lut, uint32_t lane4) {
  if constexpr (W <= 4) {
    return *reinterpret_cast<const uint32_t*>(lut + plut_off(W) + (field_at(lo, hi, p, 2 * W, 7) | lane4));
  } else if constexpr (W == 5) {
    return *reinterpret_cast<const uint32_t*>(lut + plut_off(W) + field_at(lo, hi, p, 2 * W, 2));
  } else {
    const uint8_t* t = lut + plut_off(W);
    return static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(t + field_at(lo, hi, p, W, 1))) |
           (static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(t + field_at(lo, hi, p + W, W, 1))) << 16);
  }
}

// V-hat of one dim for the 32 tokens of a tile: 16 token pairs (2u, 2u + 1). vw: word 0 of the dim.
template <int BV>
__device__ __forceinline__ void v_vals(const uint32_t* vw, const uint8_t* lut, uint32_t lane4, uint32_t (&v)[16]) {
  uint32_t x[BV + 1];
#pragma unroll
  for (int i = 0; i < BV; ++i) x[i] = vw[i * kD];
  x[BV] = 0u;
#pragma unroll
  for (int u = 0; u < 16; ++u) {
    const int p = 2 * BV * u;
    v[u] = pair_of<BV>(x[p >> 5], x[(p >> 5) + 1], p & 31, lut, lane4);
  }
}

// ---------------------------------------------------------------- pages

// Record of tile `tile` of a paged sequence for one head; a page outside the pool gives page 0's
// and sets `bad`.
__device__ __forceinline__ const uint8_t* paged_record(const uint8_t* pool, const PagedArgs& a, const int32_t* pages,
                                                       int tile, int hkv, bool& bad) {
  const int slot = tile / a.page_tiles, in = tile - slot * a.page_tiles;
  int page = __ldg(pages + slot);
  if (static_cast<unsigned>(page) >= static_cast<unsigned>(a.n_pages)) {
    bad = true;
    page = 0;
  }
  return pool + a.hdr_bytes + ((static_cast<size_t>(page) * a.n_kv_heads + hkv) * a.page_tiles + in) * a.rec_bytes;
}

// Element i of an output of run-time dtype.
__device__ __forceinline__ void store_f32(void* p, int dtype, int64_t i, float v) {
  if (dtype == KVQ_F32) static_cast<float*>(p)[i] = v;
  else if (dtype == KVQ_F16) static_cast<__half*>(p)[i] = __float2half_rn(v);
  else static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
}

// Running maxima move when a logit exceeds them by more than 2^6 (log2 units); P' is stored
// times 2^-3, at most 2^3 * 65504 / sqrt(128), inside fp16, and its low parts end 2^-22 below the
// largest share.
constexpr int kPgThr = 6;
constexpr float kPgScale = 0.125f;

}  // namespace kvq
