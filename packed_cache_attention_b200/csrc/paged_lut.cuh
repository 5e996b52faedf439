// Dequantization of tile records in the paged attention kernels: centroid lookups in shared
// memory, and the copies that bring tiles out of their pages.
//
// A lookup turns the 2w bits of two consecutive codes into one word of two fp16 centroids. For
// widths 1..4 every lane has its own copy of the table (entry i of lane l at word 32 i + l), so
// 32 lanes never share a bank; with one shared copy of width 4's 256 entries a warp's lookup
// takes 3.5 passes on average. A field is moved to bit 7 of a word by one shift, masked and joined
// with the lane by one three-input operation, and is then the entry's byte offset: three
// instructions a pair, two of them on the half-rate integer pipe. Width 5 (4 KB) has one copy, its fields at bit 2;
// widths 6..8 (the few blocks of the highest energy, or large budgets) take two single lookups.
#pragma once

#include <type_traits>

#include "decode.cuh"
#include "paged_pool.cuh"
#include "quantize.cuh"

namespace kvq {

// Byte offsets of the tables, each a multiple of its size. The image sits at a shared-memory
// address that is a multiple of 32 KB (kPlutAddr), so that a field, the lane and a table's
// address have no bits in common.
__host__ __device__ constexpr int plut_off(int w) {
  return w == 4 ? 0 : w == 3 ? 32768 : w == 2 ? 40960 : w == 1 ? 43008 : w == 8 ? 43520 : w == 7 ? 44032 : w == 6 ? 44288 : 45056;
}
constexpr int kPlutBytes = 49152;

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

// Dynamic shared memory of a kernel without static variables begins behind the 1 KB that the system
// keeps (the host checks that, the kernels too); the image begins 32 KB into the window.
constexpr uint32_t kSmemBase = 1024, kPlutAddr = 32768;
constexpr int kPlutAt = kPlutAddr - kSmemBase, kPlutEnd = kPlutAt + kPlutBytes;   // from the start of dynamic shared memory

__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t v;
  asm("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t addr) {
  uint16_t v;
  asm("ld.shared.b16 %0, [%1];" : "=h"(v) : "r"(addr));
  return v;
}
// Address of width w's table as this lane uses it.
__device__ __forceinline__ uint32_t plut_lane(int w, uint32_t lane) {
  return kPlutAddr + static_cast<uint32_t>(plut_off(w)) + (w <= 4 ? 4u * lane : 0u);
}

// ---------------------------------------------------------------- keys

// Descriptor of a plan slot (4 block pairs of one width), read by every lane. A narrow slot
// (width <= 5): `a` = byte offset of the stream word where the first field's place starts (-128 when
// it reaches back before the stream: what is read there is masked out), shift that brings the
// field to its place, 2w, mask of a field in its place; `b` = table base, lane bits of an address.
// A wide slot: offset, shift and width of the first code.
struct KSlots {
  alignas(16) uint4 a[kPlanSlots];
  alignas(8) uint2 b[kPlanSlots];
  int n_wide, n;                          // widths descend: slots 0 .. n_wide - 1 are wide
};

// Builds the descriptors of `n_cols` columns (a multiple of 8; slots past the plan's last are empty:
// finite values against zero rows of Q'). False for a slot that starts past the stream or a
// wide one behind a narrow one. A whole warp, lane = slot.
__device__ __forceinline__ bool k_slots(const uint32_t* slots, int n_cols, int stream_bits, KSlots& S) {
  const int s = threadIdx.x & 31, n = n_cols / 4;
  const uint32_t in = s < kPlanSlots ? slots[s] : 0u;       // (loaded beside n_cols, not after it)
  const uint32_t e = s < n ? in : 0u;
  uint32_t w = e & 15u, off = e >> 8;
  bool ok = w <= 8 && (w == 0 || off < static_cast<uint32_t>(stream_bits));
  if (!ok || w == 0) { w = 1; off = 0; }
  const uint32_t wide = __ballot_sync(0xffffffffu, w > 5);
  const int n_wide = __popc(wide);
  ok = ok && wide == (1u << n_wide) - 1u;
  const int at = static_cast<int>(off) - (w <= 4 ? 7 : w == 5 ? 2 : 0);
  if (s < n) {
    S.a[s] = make_uint4(static_cast<uint32_t>((at >> 5) * 128), static_cast<uint32_t>(at) & 31u, w <= 5 ? 2 * w : w,
                        w <= 5 ? ((1u << (2 * w)) - 1u) << (w <= 4 ? 7 : 2) : 0u);
    S.b[s] = make_uint2(kPlutAddr + static_cast<uint32_t>(plut_off(static_cast<int>(w))), w <= 4 ? 0x7cu : 0u);
  }
  if (s == 0) {
    S.n_wide = n_wide;
    S.n = n;
  }
  return __all_sync(0xffffffffu, ok);
}

// ---------------------------------------------------------------- values

// Two consecutive codes of width W at bit p of hi:lo; `tab` = plut_lane(W, lane).
template <int W>
__device__ __forceinline__ uint32_t pair_of(uint32_t lo, uint32_t hi, int p, uint32_t tab) {
  if constexpr (W <= 4) return lds32(field_at(lo, hi, p, 2 * W, 7) | tab);
  else if constexpr (W == 5) return lds32(field_at(lo, hi, p, 2 * W, 2) | tab);
  else return lds16(field_at(lo, hi, p, W, 1) | tab) | lds16(field_at(lo, hi, p + W, W, 1) | tab) << 16;
}

// V-hat of one dim for the 32 tokens of a tile: 16 token pairs (2u, 2u + 1). vw: word 0 of the
// dim, tab: plut_lane(BV, lane).
template <int BV>
__device__ __forceinline__ void v_vals(const uint32_t* vw, uint32_t tab, uint32_t (&v)[16]) {
  uint32_t x[BV + 1];
#pragma unroll
  for (int i = 0; i < BV; ++i) x[i] = vw[i * kD];
  x[BV] = 0u;
#pragma unroll
  for (int u = 0; u < 16; ++u) {
    const int p = 2 * BV * u;
    v[u] = pair_of<BV>(x[p >> 5], x[(p >> 5) + 1], p & 31, tab);
  }
}

// The 4 words of one wide slot from its two aligned stream words.
template <int W>
__device__ __forceinline__ void k_wide_vals(uint32_t r0, uint32_t r1, uint32_t (&v)[4]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int p = 2 * W * k;
    v[k] = p < 32 ? pair_of<W>(r0, r1, p, kPlutAddr + plut_off(W)) : pair_of<W>(r1, 0u, p - 32, kPlutAddr + plut_off(W));
  }
}

// K-hat columns of slots first, first + step, .. below end (at most S.n) of the lane's token; kw: its
// word 0 (word i at byte 128 i). put(slot, v) takes a slot's 4 columns. Narrow slots of every width go through one
// sequence of instructions, kAtOnce at a time. Words past the stream are read inside the stage and not
// used.
template <int kAtOnce, typename Put>
__device__ __forceinline__ void k_lookup(const uint8_t* kw, const KSlots& S, int first, int end, int step,
                                         uint32_t lane4, Put put) {
  end = min(end, S.n);
  const int wide_end = min(end, S.n_wide);
  int s = first;
#pragma unroll 1
  for (; s < wide_end; s += step) {
    const uint4 d = S.a[s];
    const uint32_t* p = reinterpret_cast<const uint32_t*>(kw + static_cast<int>(d.x));
    const uint32_t x0 = p[0], x1 = p[32], x2 = p[64];
    const uint32_t r0 = __funnelshift_r(x0, x1, d.y), r1 = __funnelshift_r(x1, x2, d.y);
    uint32_t v[4];
    if (d.z == 6) k_wide_vals<6>(r0, r1, v);
    else if (d.z == 7) k_wide_vals<7>(r0, r1, v);
    else k_wide_vals<8>(r0, r1, v);
    put(s, v);
  }
#pragma unroll 1
  for (; s < end; s += kAtOnce * step) {
    // (past the last slot it is looked up again)
    int at[kAtOnce];
    uint4 d[kAtOnce];
    uint32_t lb[kAtOnce], r0[kAtOnce], r1[kAtOnce];
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      at[u] = (u == 0 || s + u * step < end) ? s + u * step : at[u - 1];
      d[u] = S.a[at[u]];
      const uint2 b = S.b[at[u]];
      lb[u] = b.x | (lane4 & b.y);
    }
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      const uint32_t* p = reinterpret_cast<const uint32_t*>(kw + static_cast<int>(d[u].x));
      const uint32_t x0 = p[0], x1 = p[32], x2 = p[64];
      r0[u] = __funnelshift_r(x0, x1, d[u].y);
      r1[u] = __funnelshift_r(x1, x2, d[u].y);
    }
    uint32_t v[kAtOnce][4];
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t f = (k == 0) ? r0[u] : __funnelshift_r(r0[u], r1[u], d[u].z * k);
        v[u][k] = lds32((f & d[u].w) | lb[u]);
      }
    }
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) put(at[u], v[u]);
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

// Scale of a row of Q' from the largest bits of its |values|: its largest value comes to [2^13, 2^14), so that
// the low parts of its fp16 pairs end at 2^-38 of it (scaled to [0.5, 1) they ended at 2^-25, and a logit
// had 22 bits). A block without key bits counts as 0 there, as its keys do. `back` undoes the scale; it is
// NaN, and with it the row's logits, if a query value is not finite, in a block without key bits too
// (inf * 0). Exponents stay where both scales are normal numbers.
__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }
__device__ __forceinline__ float query_scale(uint32_t max_bits, float& back) {
  const bool finite = max_bits < 0x7f800000u;
  int e = 0;
  if (finite && max_bits > 0) frexpf(__uint_as_float(max_bits), &e);
  e = max(e, -111) - 14;
  back = finite ? ldexpf(1.0f, e) : __int_as_float(0x7fc00000);
  return ldexpf(1.0f, -e);
}

// Elements i .. i + 3 of a row of 16-bit or fp32 values (i a multiple of 4, rows 16-byte aligned).
template <int DT>
__device__ __forceinline__ float4 load4(const void* p, int64_t i) {
  if constexpr (DT == KVQ_F32) {
    return *reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
  } else {
    const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + i);
    const float2 a = unpack_pair<DT>(u.x), b = unpack_pair<DT>(u.y);
    return make_float4(a.x, a.y, b.x, b.y);
  }
}
// f(type) with the run-time dtype as a constant: loads inside one call of f are in flight together
// (a branch on the type at every element makes each wait for the one before).
template <typename F>
__device__ __forceinline__ void by_dtype(int dtype, F f) {
  if (dtype == KVQ_F32) f(std::integral_constant<int, KVQ_F32>{});
  else if (dtype == KVQ_F16) f(std::integral_constant<int, KVQ_F16>{});
  else f(std::integral_constant<int, KVQ_BF16>{});
}

// Element i of an output of run-time dtype.
__device__ __forceinline__ void store_f32(void* p, int dtype, int64_t i, float v) {
  if (dtype == KVQ_F32) static_cast<float*>(p)[i] = v;
  else if (dtype == KVQ_F16) static_cast<__half*>(p)[i] = __float2half_rn(v);
  else static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
}

// Shares P' = 2^(logit - M) * |value| / sqrt(128) * scale as fp16 pairs. M is a row's running maximum not
// of its logits but of logit + log2(|value| / sqrt(128)): the largest share is in [scale, 2^thr scale]
// whatever the values' norms are, and the row sum, with the same M, is fp32. M moves when it is
// exceeded by more than `thr` (log2 units); 2^thr * scale = 2^15 stays inside fp16. A pair is good to
// 2^-22 of its share down to fp16's smallest normal number in the high part, and below that to an
// absolute error: 2^-36 where low parts have rows of their own in the product and are stored times
// 2^11 (decode), 2^-25 where they join the high parts' sums (prefix); that is 2^-45 and 2^-38 of the
// row's largest share. (M of the logits alone and a fixed scale lost the shares of small values:
// over 4096 tokens of a prefix 2e-3 of the output at |v| = 1e-3, 0.2 at 1e-5. The maxima of the prefix move sooner, which a chunk's
// time does not show; for decode the same costs 3 %.)
constexpr int kPgThr = 6, kPreThr = 2;
constexpr float kPgScale = 512.0f, kPreScale = 8192.0f, kPgLow = 2048.0f;

// log2 of a value's norm / sqrt(128) for M. Stored norms are 0 or 2^-24 .. 65504. A value of norm 0 counts
// as 2^-60: shares of other values stay exact when all of them together are 2^-60 of such a token's
// softmax weight, and row sums stay below 2^97. An infinite or NaN norm (its share is not finite
// anyway) counts as one inside the range.
__device__ __forceinline__ float share_log2(float vn) { return fminf(fmaxf(__log2f(vn), -60.0f), 13.0f); }

}  // namespace kvq
