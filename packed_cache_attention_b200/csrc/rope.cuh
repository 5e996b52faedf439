// Rotary positions with one or several axes.
//
// Block b is the pair (x_b, x_b+64), turned by the angle whose cosine and sine the caller's
// table holds for position positions[axis[b]][token]:
//   out_b = fl(fl(x_b c) - fl(x_b+64 s)),  out_b+64 = fl(fl(x_b+64 c) + fl(x_b s))
// Products and sums are rounded one by one (no fused multiply-add), so a key rotated here and
// one rotated inside an append are the same bits.
//
// kvq_rope_rows is bound by memory: a row is read and written once, a token's 512 table bytes
// are read once per group of heads. A thread owns 16 bytes of both halves of a row, loads
// their cosines and sines once and walks the heads of its group, four rows in flight.
#pragma once

#include "common.cuh"

namespace kvq {

struct RopeArgs {
  const float2* table;               // [n_positions][64]: cos, sin
  const int32_t* positions;          // [n_axes][tokens], axis stride in elements
  int64_t axis_stride;
  int n_positions;                   // 0: no rotation (append)
  int n_axes;
  uint8_t axis[kH];
};

// Rotation of one pair, every operation rounded.
__device__ __forceinline__ void rotate_pair(float x1, float x2, float2 cs, float& o1, float& o2) {
  o1 = __fsub_rn(__fmul_rn(x1, cs.x), __fmul_rn(x2, cs.y));
  o2 = __fadd_rn(__fmul_rn(x2, cs.x), __fmul_rn(x1, cs.y));
}

// Cosine and sine of block b at a position; NaN outside the table.
__device__ __forceinline__ float2 rope_cs(const RopeArgs& r, int pos, int b) {
  if (static_cast<unsigned>(pos) >= static_cast<unsigned>(r.n_positions)) {
    const float nan = __int_as_float(0x7fc00000);
    return make_float2(nan, nan);
  }
  return __ldg(r.table + static_cast<int64_t>(pos) * kH + b);
}

// Two consecutive values of a 16-bit type from and to one 32-bit word.
template <int DT>
__device__ __forceinline__ float2 word_to_pair(uint32_t w) {
  if constexpr (DT == KVQ_BF16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  else return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
template <int DT>
__device__ __forceinline__ uint32_t pair_to_word(float a, float b) {
  if constexpr (DT == KVQ_BF16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  } else {
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
}

struct RopeRows {
  const uint8_t* x;
  uint8_t* out;
  int64_t xsb, xsh, xst, osb, osh, ost;   // strides in elements
  int64_t n_tokens;
  int seq_len, n_heads, heads_per_cta;
};

constexpr int kRopeThreads = 256;
constexpr int kRopeBatch = 4;             // rows in flight per thread

// Tokens a CTA covers: a row takes 8 threads (16-bit types) or 16 (fp32).
__host__ __device__ constexpr int rope_cta_tokens(int dt) { return kRopeThreads / (dt == KVQ_F32 ? 16 : 8); }

template <int DT>
__global__ void __launch_bounds__(kRopeThreads) kvq_rope_rows(const RopeRows a, const RopeArgs r) {
  constexpr int ES = DT == KVQ_F32 ? 4 : 2;
  constexpr int V = 16 / ES;                               // blocks a thread owns
  constexpr int LPR = kH / V;                              // threads of a row
  grid_dependency_wait();
  const int64_t tok = static_cast<int64_t>(blockIdx.x) * (kRopeThreads / LPR) + threadIdx.x / LPR;
  if (tok < a.n_tokens) {
    const int b0 = V * (threadIdx.x % LPR);
    const int64_t b = tok / a.seq_len, t = tok % a.seq_len;
    const int h0 = blockIdx.y * a.heads_per_cta, h1 = min(a.n_heads, h0 + a.heads_per_cta);
    const uint8_t* xp = a.x + ES * (b * a.xsb + t * a.xst + b0);
    uint8_t* op = a.out + ES * (b * a.osb + t * a.ost + b0);
    // the first rows are on their way before the positions are looked at
    uint4 lo[kRopeBatch], hi[kRopeBatch];
    auto load = [&](int h) {
#pragma unroll
      for (int u = 0; u < kRopeBatch; ++u) {
        if (h + u < h1) {
          const uint8_t* p = xp + ES * (h + u) * a.xsh;
          lo[u] = *reinterpret_cast<const uint4*>(p);
          hi[u] = *reinterpret_cast<const uint4*>(p + ES * kH);
        }
      }
    };
    load(h0);
    float2 cs[V];
#pragma unroll
    for (int i = 0; i < V; ++i) cs[i] = rope_cs(r, r.positions[r.axis[b0 + i] * r.axis_stride + tok], b0 + i);
    for (int h = h0; h < h1; h += kRopeBatch) {
#pragma unroll
      for (int u = 0; u < kRopeBatch; ++u) {
        if (h + u >= h1) break;
        uint32_t l[4] = {lo[u].x, lo[u].y, lo[u].z, lo[u].w}, g[4] = {hi[u].x, hi[u].y, hi[u].z, hi[u].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if constexpr (DT == KVQ_F32) {
            float o1, o2;
            rotate_pair(__uint_as_float(l[i]), __uint_as_float(g[i]), cs[i], o1, o2);
            l[i] = __float_as_uint(o1);
            g[i] = __float_as_uint(o2);
          } else {
            const float2 x1 = word_to_pair<DT>(l[i]), x2 = word_to_pair<DT>(g[i]);
            float a1, a2, c1, c2;
            rotate_pair(x1.x, x2.x, cs[2 * i], a1, a2);
            rotate_pair(x1.y, x2.y, cs[2 * i + 1], c1, c2);
            l[i] = pair_to_word<DT>(a1, c1);
            g[i] = pair_to_word<DT>(a2, c2);
          }
        }
        uint8_t* p = op + ES * (h + u) * a.osh;
        *reinterpret_cast<uint4*>(p) = make_uint4(l[0], l[1], l[2], l[3]);
        *reinterpret_cast<uint4*>(p + ES * kH) = make_uint4(g[0], g[1], g[2], g[3]);
      }
      if (h + kRopeBatch < h1) load(h + kRopeBatch);
    }
  }
  allow_dependents();
}

}  // namespace kvq
