// Attention of a whole batch over one shared prefix in a paged pool.
//
// For one KV head all query rows of the batch (row = sequence * group + head of the group) meet
// the same keys and values, so a chunk of 128 tokens is dequantized once for up to 128 rows:
//   S[128 rows][128 tokens] = Q' x Khat^T,   O[128 rows][128 dims] += P' x Vhat
// with tcgen05.mma (M 128, N 128). lane = row in the softmax: a row's maximum and sum are a
// thread's own values. Two warpgroups look Khat and Vhat up (shared-memory loads and integer
// operations), two run the softmax (exponentials, fp32), 64 tokens each of the same rows.
//
// Precision: Q' and P' are fp16 high + low parts (Khat and Vhat are fp16 centroids, exact), so every
// product runs twice; the norms of keys and values multiply the fp32 logits and shares. A
// single fp16 Q' would move a logit of 100 by 2^-5. The output's type makes no difference up to its
// rounding.
//
// Layout. Tensor memory: Q' high (A operand, 96 columns), two buffers of 128 columns for S, O. A
// warpgroup writes its P' over the S columns that it has read (16 columns high parts, 16 low).
// Shared memory: Q' low (A operand), Khat and Vhat (B operands), all K-major without swizzle: 8
// rows x 16 bytes contiguous, 2048 bytes per 8 K elements, so a lookup's 4 words (8 elements
// of a token's key, or 8 tokens of a dim) are one 16-byte store next to its neighbour lane's.
//
// Order: the producers write Khat(j + 1) once S(j) is done and Vhat(j) once O(j - 1) is; S(j + 1) is
// issued before O(j), into the other buffer, so it runs under the softmax of chunk j. A chunk takes
// 5.6k cycles (3.2 us; K3V3, 128 rows), 0.3k of them for the low parts of P' and the values' part of M;
// with tokens as lanes, whose row maxima need a warp reduction per row, it took 12.9k.
//
// Every wait is bounded, as in kvq_decode_gtq; a CTA that gave up, or met a bad header or page,
// leaves NaN maxima, at which the merge leaves the rows as they are.
#pragma once

#include "paged_attn.cuh"

namespace kvq {

constexpr int kPreThreads = 17 * 32;       // 16 compute warps and the issuing one

struct PrefixArgs {
  const void* q;
  int64_t qsb, qsh;
  int q_dtype;
  int n_rows, group;                      // query rows per KV head, rows per sequence
  const uint8_t* pool;
  const kvq_head_alloc* alloc;
  PagedArgs pg;
  const int32_t* pages;                   // the prefix's pages
  int len, per, row_groups, n_stages;     // per: chunks of a split
  float* part_m;                          // [CTA][kPreRows]
  float* part_l;
  float* part_o;                          // [CTA][kPreRows][128]
  unsigned* status;
  uint32_t wait_limit;
  int debug_no_loads;
};

struct PreHeader {
  uint64_t fullk[kPgStagesMax], fullv[kPgStagesMax];
  uint64_t kready, ofull, drain, setup;
  uint64_t sfull[2], vready[2];                 // by chunk parity: see the consumers
  uint32_t tmem_base;
  int bad, bad_page, abort;
  int k_cols;
  KSlots slots;
  alignas(16) float dequant[kH];
  int8_t col_block[96];
  alignas(16) float norm[4][3][kChunkTokens];   // [chunk mod 4][key, value / sqrt(d), its log2 for M][token]
  float xch[2][2][kPreRows];                    // [chunk parity][softmax warpgroup][row]: maximum; sums at the end
};

// Shared memory: header, Q' low of the first kPreQCut K steps; lookup tables (at their address); Q'
// low of the other steps, Khat, Vhat, stages.
constexpr int kPreHdrOff = 0, kPreQCut = 5;
constexpr int kPreQ0 = kPreHdrOff + (static_cast<int>(sizeof(PreHeader)) + 127) / 128 * 128;
static_assert(kPreQ0 + kPreQCut * 4096 <= kPlutAt, "before the lookup tables");
constexpr int kPreQ1 = kPlutEnd;
constexpr int kPreKOff = kPreQ1 + (12 - kPreQCut) * 4096;
constexpr int kPreVOff = kPreKOff + 192 * kChunkTokens * 2;
constexpr int kPreStageOff = kPreVOff + kD * kChunkTokens * 2;
__device__ __forceinline__ int pre_q_step(int ks) { return ks < kPreQCut ? kPreQ0 + 4096 * ks : kPreQ1 + 4096 * (ks - kPreQCut); }
constexpr int kPreQPitch = kD + 1;                   // staged fp32 queries, over Khat and Vhat before the first chunk
static_assert(kPreRows * kPreQPitch * 4 <= kPreStageOff - kPreKOff, "staged queries");
constexpr uint32_t kPreS = 96, kPreO = 352;          // tensor-memory columns (Q' high at 0)

// V-hat values of one tile for a run-time width.
__device__ __forceinline__ void v_vals_any(int bv, const uint32_t* vw, uint32_t tab, uint32_t (&v)[16]) {
  switch (bv) {
    case 1: v_vals<1>(vw, tab, v); break;
    case 2: v_vals<2>(vw, tab, v); break;
    case 3: v_vals<3>(vw, tab, v); break;
    case 4: v_vals<4>(vw, tab, v); break;
    case 5: v_vals<5>(vw, tab, v); break;
    case 6: v_vals<6>(vw, tab, v); break;
    case 7: v_vals<7>(vw, tab, v); break;
    default: v_vals<8>(vw, tab, v); break;
  }
}

__global__ void __launch_bounds__(kPreThreads, 1) kvq_prefix_gtq(const PrefixArgs a) {
  extern __shared__ __align__(1024) uint8_t sm[];
  PreHeader& S = *reinterpret_cast<PreHeader*>(sm + kPreHdrOff);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int hkv = blockIdx.x % a.pg.n_kv_heads;
  const int rg = blockIdx.x / a.pg.n_kv_heads % a.row_groups;
  const int split = blockIdx.x / (a.pg.n_kv_heads * a.row_groups);
  const kvq_head_alloc* al = a.alloc + hkv;
  const int kbytes = 4 * kD * a.pg.bits_k + 4 * kTile, vbytes = 4 * kD * a.pg.bits_v;   // of a record: K words, norms; V words
  const int cbytes = kChunkTiles * (kbytes + vbytes);
  const int NS = a.n_stages;
  const float inv_sqrt_d = 0.08838834764831845f;
  const uint32_t WL = a.wait_limit;
  const bool is_issuer = warp == 16;
  const int wg = warp >> 2, q = warp & 3;
  uint8_t* stages = sm + kPreStageOff;
  volatile int* abort_flag = &S.abort;

  if (tid == 0) {
    for (int s = 0; s < kPgStagesMax; ++s) {
      tc::mbar_init(&S.fullk[s], 1);
      tc::mbar_init(&S.fullv[s], 1);
    }
    tc::mbar_init(&S.kready, 8);
    tc::mbar_init(&S.sfull[0], 2);
    tc::mbar_init(&S.sfull[1], 2);
    tc::mbar_init(&S.vready[0], 16);
    tc::mbar_init(&S.vready[1], 16);
    tc::mbar_init(&S.ofull, 1);
    tc::mbar_init(&S.drain, 2);
    tc::mbar_init(&S.setup, 1);
    S.bad = tc::smem_u32(sm) != kSmemBase;                  // the tables would not be at their address
    if (S.bad) record_status(a.status, KVQ_ERR_UNSUPPORTED);
    S.bad_page = 0;
    S.abort = 0;
    tc::mbar_fence_init();
    tc::mbar_arrive_expect_tx(&S.setup, kPlutBytes);
    tc::bulk_g2s(sm + kPlutAt, g_paged_lut, kPlutBytes, &S.setup);
  }
  if (is_issuer) tc::tmem_alloc(&S.tmem_base, kTmemCols);
  __syncthreads();
  grid_dependency_wait();
  allow_dependents();                                       // the call's own-pages kernel may fill the other SMs
  if (warp == 0) {
    const int k_cols = min(max(al->plan_k_cols, 8), 96) & ~7;
    const bool ok = k_slots(al->plan_slot, k_cols, kD * a.pg.bits_k, S.slots);
    if (lane == 0) {
      S.k_cols = k_cols;
      if (!ok) {
        S.bad = 1;
        record_status(a.status, KVQ_ERR_MISMATCH);
      }
    }
  } else if (tid >= 64 && tid < 64 + 96) {
    const int blk = al->plan_col_block[tid - 64];
    S.col_block[tid - 64] = static_cast<int8_t>(blk < kH ? blk : -1);
  } else if (tid >= 192 && tid < 192 + kH) {
    S.dequant[tid - 192] = al->width[tid - 192] ? al->dequant[tid - 192] * (inv_sqrt_d * kLog2e) : 0.0f;
  } else if (tid == 256) {
    // (asked for before the header's fields are looked at, so one round trip brings everything)
    const uint64_t dg = paged_digest(a.pool, hkv), ad = __ldcg(reinterpret_cast<const unsigned long long*>(&al->digest));
    const int abk = __ldcg(&al->bits_k), akw = __ldcg(&al->k_words), apk = __ldcg(&al->plan_k_cols), aps = __ldcg(&al->plan_n_slots);
    unsigned code = paged_header_code(a.pool, a.pg);
    if (!code && !((dg == ad) & (abk == a.pg.bits_k) & (akw == a.pg.bits_k * kD) & (apk <= 96) & (apk >= 8) & (aps >= 1) &
                   (aps <= kPlanSlots)))
      code = KVQ_ERR_MISMATCH;
    if (code) {
      S.bad = 1;
      record_status(a.status, code);
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const bool bad = S.bad != 0;
  const uint32_t tb = S.tmem_base;
  const int k_steps = S.k_cols >> 3;

  const int n_tiles = (a.len + kTile - 1) / kTile;
  const int n_chunks_all = (n_tiles + kChunkTiles - 1) / kChunkTiles;
  const int c_begin = split * a.per;
  const int n = min(a.per, n_chunks_all - c_begin);         // at least 1: the host leaves no split empty
  const int rows = min(kPreRows, a.n_rows - rg * kPreRows);

  float M = -INFINITY, L = 0.0f;                            // row 32 q + lane (see kPreThr); this warpgroup's tokens

  if (bad) {
  } else if (is_issuer) {
    // ------------------------------------------------------------------ issuing warp
    // One lane issues the products. Elected for the logits, which the consumers wait for (2.96 -> 2.79 us
    // a chunk, with high parts of P' alone), lane 0 for O's: those issued as fast held up the warps' own
    // tensor memory accesses (3.2 us). Lanes 0..3 each copy one tile of a chunk.
    int nk = 0, nv = 0;                                     // chunks whose K (V) copies are started
    Ring rk, rv;
    auto copy_part = [&](int& i, Ring& r, uint64_t* bars, int skip, int bytes, int at) {
      const int s = r.s, tile0 = (c_begin + i) * kChunkTiles;
      const int nt = min(kChunkTiles, n_tiles - tile0);
      bool off = false;
      const uint8_t* rec = nullptr;
      if (lane < nt) rec = paged_record(a.pool, a.pg, a.pages, tile0 + lane, hkv, off);
      if (off) {
        S.bad_page = 1;
        record_status(a.status, KVQ_ERR_RANGE);
      }
      if (lane == 0) tc::mbar_arrive_expect_tx(&bars[s], static_cast<uint32_t>(nt * bytes));
      __syncwarp();
      if (lane < nt)
        tc::bulk_g2s(stages + static_cast<size_t>(s) * cbytes + at + lane * bytes, rec + skip, bytes, &bars[s]);
      ++i;
      r.next(NS);
    };
    auto copy_k = [&]() { copy_part(nk, rk, S.fullk, 0, kbytes, 0); };
    auto copy_v = [&]() { copy_part(nv, rv, S.fullv, kbytes, vbytes, kChunkTiles * kbytes); };
    const bool loads = !a.debug_no_loads;
    if (loads)
      while (nv < min(NS, n)) {
        copy_k();
        copy_v();
      }
    auto wait_warp = [&](uint64_t* bar, uint32_t parity) {  // lane 0 waits for the warp
      int r = 1;
      if (lane == 0) r = tc::mbar_wait(bar, parity, WL);
      r = __shfl_sync(0xffffffffu, r, 0);
      __syncwarp();
      return r != 0;
    };
    const uint32_t id = tc::idesc_f16(128, 128, false);
    const uint32_t smb = tc::smem_u32(sm), bk = tc::smem_u32(sm + kPreKOff), bv = tc::smem_u32(sm + kPreVOff);
    auto logits = [&](int j) {                              // S(j), once Khat(j) is there
      if (!wait_warp(&S.kready, j & 1)) return false;
      if (j >= 2 && !wait_warp(&S.ofull, j & 1)) return false;        // P'(j - 2) in its buffer is read
      tc::fence_after_sync();
      if (tc::elect_one()) {
        const uint32_t d = tb + kPreS + 128u * (j & 1);
        // The products' sums are cut off at 24 bits after every step: the small terms first (low parts, and
        // from the narrow blocks to the wide ones). High and low step by step from the wide end was up to
        // twice as far from the exact output.
        for (int ks = k_steps - 1; ks >= 0; --ks)
          tc::mma_ss(d, tc::sdesc(smb + pre_q_step(ks), 2048, 128), tc::sdesc(bk + 4096 * ks, 2048, 128), id, ks < k_steps - 1 ? 1u : 0u);
        for (int ks = k_steps - 1; ks >= 0; --ks) tc::mma_ts(d, tb + 8 * ks, tc::sdesc(bk + 4096 * ks, 2048, 128), id, 1u);
        tc::mma_commit(&S.sfull[j & 1]);
        tc::mbar_arrive(&S.sfull[j & 1]);                   // (passes on the producers' norms)
      }
      __syncwarp();
      if (nk < n && loads) copy_k();
      return true;
    };
    bool ok = logits(0);
    for (int j = 0; j < n && ok; ++j) {
      if (j + 1 < n && !logits(j + 1)) { ok = false; break; }
      if (!wait_warp(&S.vready[j & 1], (j >> 1) & 1)) { ok = false; break; }
      tc::fence_after_sync();
      if (lane == 0) {
        const uint32_t p = tb + kPreS + 128u * (j & 1);
#pragma unroll
        for (int ks = 0; ks < 2 * (kChunkTokens / 16); ++ks) {
          const int kk = ks % (kChunkTokens / 16);          // high parts, then low parts
          tc::mma_ts(tb + kPreO, p + 32 * (kk >> 1) + 8 * (kk & 1) + (ks >= kChunkTokens / 16 ? 16 : 0),
                     tc::sdesc(bv + 4096 * kk, 2048, 128), id, (j > 0 || ks > 0) ? 1u : 0u);
        }
        tc::mma_commit(&S.ofull);
      }
      __syncwarp();
      if (nv < n && loads) copy_v();
    }
    if (!ok) *abort_flag = 1;
    // products committed and copies started end before the CTA frees what they use
    if (tc::elect_one()) tc::mma_commit(&S.drain);          // the logits' products
    if (lane == 0) {
      tc::mma_commit(&S.drain);                             // O's
      tc::mbar_wait(&S.drain, 0, WL);
      for (int s = 0; s < NS; ++s) {
        if (nk > s) tc::mbar_wait(&S.fullk[s], ((nk - 1 - s) / NS) & 1, WL);
        if (nv > s) tc::mbar_wait(&S.fullv[s], ((nv - 1 - s) / NS) & 1, WL);
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------------ compute warps
    const uint32_t lane_base = static_cast<uint32_t>(32 * q) << 16;
    const uint32_t lane4 = static_cast<uint32_t>(lane) << 2, tab = plut_lane(a.pg.bits_v, lane);
    const int t = 32 * q + lane;                            // row of S and O, token of Khat, dim of Vhat
    const bool live = 32 * q < rows;                        // some row of the warp is a query
    // -------------------------------------------------------------- Q'
    // Row r: q * f_b * log2(e) / sqrt(d) by a power of two (query_scale). The rows are staged in fp32 and
    // taken up by row: columns 24 wg .. 24 wg + 23 of row t.
    float* stg = reinterpret_cast<float*>(sm + kPreKOff);
    by_dtype(a.q_dtype, [&](auto dt) {
      float4 v[kPreRows / 16];                              // (all rows' loads are in flight together)
      const float per = 1.0f / static_cast<float>(a.group);
#pragma unroll
      for (int i = 0; i < kPreRows / 16; ++i) {
        const int r = warp + 16 * i, row = rg * kPreRows + r;
        const int b = static_cast<int>((static_cast<float>(row) + 0.5f) * per);   // row / group: rows are below 2^13
        v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r < rows)
          v[i] = load4<dt.value>(a.q, b * a.qsb + (static_cast<int64_t>(hkv) * a.group + (row - b * a.group)) * a.qsh + 4 * lane);
      }
      const float4 f = *reinterpret_cast<const float4*>(S.dequant + (4 * lane) % kH);
#pragma unroll
      for (int i = 0; i < kPreRows / 16; ++i) {
        if (16 * i >= ((rows + 31) & ~31)) break;
        float* x = stg + (warp + 16 * i) * kPreQPitch + 4 * lane;
        x[0] = v[i].x * f.x;
        x[1] = v[i].y * f.y;
        x[2] = v[i].z * f.z;
        x[3] = v[i].w * f.w;
      }
    });
    named_sync(1, 512);
    // (rows past the batch come up to the warp's end as zeros; a warp of such rows alone takes no part: what its
    // rows of Q', S and O hold concerns no other row)
    uint32_t mx = 0u;
    if (live) {
#pragma unroll 8
      for (int i = 0; i < 32; ++i) mx = max(mx, abs_bits(stg[t * kPreQPitch + 32 * wg + i]));
    }
    S.xch[wg >> 1][wg & 1][t] = __uint_as_float(mx);
    named_sync(1, 512);
    mx = max(max(abs_bits(S.xch[0][0][t]), abs_bits(S.xch[0][1][t])), max(abs_bits(S.xch[1][0][t]), abs_bits(S.xch[1][1][t])));
    float qs;
    const float sc = query_scale(mx, qs);
#pragma unroll
    for (int c8 = 0; c8 < 24; c8 += 8) {
      if (!live) break;
      uint32_t hi[8], lo[8];
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const int blk = S.col_block[24 * wg + c8 + c];
        uint32_t h0 = 0u, l0 = 0u, h1 = 0u, l1 = 0u;
        if (blk >= 0) {
          split16<false>(stg[t * kPreQPitch + blk] * sc, h0, l0);
          split16<false>(stg[t * kPreQPitch + kH + blk] * sc, h1, l1);
        }
        hi[c] = h0 | (h1 << 16);
        lo[c] = l0 | (l1 << 16);
      }
      tc::tmem_st<8>(tb + lane_base + 24 * wg + c8, hi);
      uint8_t* p = sm + pre_q_step((24 * wg + c8) / 8) + t * 16;
      *reinterpret_cast<uint4*>(p) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
      *reinterpret_cast<uint4*>(p + 2048) = make_uint4(lo[4], lo[5], lo[6], lo[7]);
    }
    tc::wait_st();
    tc::fence_proxy_async_smem();                           // Q' low, before anyone's kready
    tc::fence_before_sync();
    named_sync(1, 512);                                     // the staged rows are read
    if (!tc::mbar_wait(&S.setup, 0, WL)) *abort_flag = 1;

    if (wg < 2) {
      // ---------------------------------------------------------------- producers: Khat and Vhat
      Ring rk, rv;
      // Khat(j) and the norms of its tokens (lane = token; a warpgroup takes every second slot)
      auto keys = [&](int j) {
        const int s = rk.s;
        if (!tc::mbar_wait(&S.fullk[s], rk.parity, WL)) *abort_flag = 1;
        rk.next(NS);
        const uint8_t* rec = stages + static_cast<size_t>(s) * cbytes + q * kbytes;
        k_lookup<4>(rec + lane4, S.slots, wg, kPlanSlots, 2, lane4, [&](int slot, const uint32_t (&v)[4]) {
          *reinterpret_cast<uint4*>(sm + kPreKOff + slot * 2048 + t * 16) = make_uint4(v[0], v[1], v[2], v[3]);
        });
        if (wg == (j & 1)) {
          const bool valid = (c_begin + j) * kChunkTokens + t < a.len;
          const uint16_t* nrm = reinterpret_cast<const uint16_t*>(rec + 4 * kD * a.pg.bits_k) + lane;
          S.norm[j & 3][0][t] = valid ? __half2float(__ushort_as_half(nrm[0])) : 0.0f;
          const float vn = valid ? __half2float(__ushort_as_half(nrm[kTile])) * inv_sqrt_d : 0.0f;
          S.norm[j & 3][1][t] = vn * kPreScale;
          S.norm[j & 3][2][t] = share_log2(vn);
        }
        tc::fence_proxy_async_smem();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&S.kready);
      };
      keys(0);
      for (int j = 0; j < n && *abort_flag == 0; ++j) {
        if (j + 1 < n) {
          if (!tc::mbar_wait(&S.sfull[j & 1], (j >> 1) & 1, WL)) *abort_flag = 1;   // Khat(j) is read
          keys(j + 1);
        }
        // Vhat(j) (lane = dim; a warpgroup takes two tiles)
        if (!tc::mbar_wait(&S.fullv[rv.s], rv.parity, WL)) *abort_flag = 1;
        const uint8_t* sv = stages + static_cast<size_t>(rv.s) * cbytes + kChunkTiles * kbytes;
        rv.next(NS);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          uint32_t v16[16];
          v_vals_any(a.pg.bits_v, reinterpret_cast<const uint32_t*>(sv + (wg + 2 * u) * vbytes) + t, tab, v16);
          if (u == 0 && j > 0 && !tc::mbar_wait(&S.ofull, (j - 1) & 1, WL)) *abort_flag = 1;   // Vhat(j - 1) is read
#pragma unroll
          for (int i = 0; i < 4; ++i)
            *reinterpret_cast<uint4*>(sm + kPreVOff + (4 * (wg + 2 * u) + i) * 2048 + t * 16) =
                make_uint4(v16[4 * i], v16[4 * i + 1], v16[4 * i + 2], v16[4 * i + 3]);
        }
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&S.vready[j & 1]);
      }
    } else {
      // ---------------------------------------------------------------- consumers: softmax (lane = row)
      const int cw = wg - 2;                                // tokens 64 cw .. 64 cw + 63
      const uint32_t tO = tb + kPreO + lane_base + 64 * cw;
      bool stopped = false;
      for (int j = 0; j < n; ++j) {
        // S(j + 1) may be done before a warp that lags gets here, S(j + 2) not (it needs O(j)): two
        // barriers tell their phases apart. For the same reason P'(j + 1) may be ready (its rows are few,
        // or the warp has none) before the last producer has Vhat(j): on one barrier that arrival
        // would stand in for the producer's, and O(j) would read a Vhat that is not there yet.
        if (!tc::mbar_wait(&S.sfull[j & 1], (j >> 1) & 1, WL)) *abort_flag = 1;
        tc::fence_after_sync();
        const uint32_t tS = tb + kPreS + 128u * (j & 1) + lane_base + 64 * cw;
        const float4* kn = reinterpret_cast<const float4*>(S.norm[j & 3][0] + 64 * cw);
        const float4* vn = reinterpret_cast<const float4*>(S.norm[j & 3][1] + 64 * cw);
        const float4* lv = reinterpret_cast<const float4*>(S.norm[j & 3][2] + 64 * cw);
        const float2 qs2 = make_float2(qs, qs);
        const int left = a.len - (c_begin + j) * kChunkTokens - 64 * cw;   // tokens of the prefix from the first one on
        // logits over 2^e of 32 tokens: S times the keys' norms, -inf past the prefix
        auto logits = [&](int c0, float2 (&x)[16]) {
          uint32_t s0[16], s1[16];
          tc::tmem_ld<16>(tS + c0, s0);
          tc::tmem_ld<16>(tS + c0 + 16, s1);
          tc::wait_ld();
#pragma unroll
          for (int i = 0; i < 16; i += 2) {
            const float4 f = kn[(c0 >> 2) + (i >> 1)];
            const uint32_t* r = i < 8 ? s0 + 2 * i : s1 + 2 * i - 16;
            x[i] = mul2(make_float2(__uint_as_float(r[0]), __uint_as_float(r[1])), make_float2(f.x, f.y));
            x[i + 1] = mul2(make_float2(__uint_as_float(r[2]), __uint_as_float(r[3])), make_float2(f.z, f.w));
          }
          if (left < 64) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              x[i].x = c0 + 2 * i < left ? x[i].x : -INFINITY;
              x[i].y = c0 + 2 * i + 1 < left ? x[i].y : -INFINITY;
            }
          }
        };
        float top = -INFINITY;
        if (live) {
          float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int c0 = 0; c0 < 64; c0 += 32) {
            float2 x[16];
            logits(c0, x);
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
              const float4 f = lv[(c0 >> 2) + (i >> 1)];
              const float2 y0 = fma2(x[i], qs2, make_float2(f.x, f.y)), y1 = fma2(x[i + 1], qs2, make_float2(f.z, f.w));
              m4[i & 2] = fmaxf(m4[i & 2], fmaxf(y0.x, y0.y));
              m4[(i & 2) + 1] = fmaxf(m4[(i & 2) + 1], fmaxf(y1.x, y1.y));
            }
          }
          top = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
        }
        S.xch[j & 1][cw][t] = top;
        // a wait that gave up joins the barrier's vote, so that the warps stop as one
        if (named_sync_or(2, 256, *abort_flag != 0)) {
          stopped = true;
          break;
        }
        if (live) {
          const float cm = fmaxf(S.xch[j & 1][0][t], S.xch[j & 1][1][t]);
          const bool up = cm > M + static_cast<float>(kPreThr);
          if (__any_sync(0xffffffffu, up)) {
            const float mn = up ? cm : M;
            const float alpha = (M == -INFINITY) ? 0.0f : fast_exp2(M - mn);
            M = mn;
            L *= alpha;
            if (j > 0) {                                    // O holds earlier chunks
              if (!tc::mbar_wait(&S.ofull, (j - 1) & 1, WL)) *abort_flag = 1;
              tc::fence_after_sync();
              const float2 al2 = make_float2(alpha, alpha);
#pragma unroll
              for (int c0 = 0; c0 < 64; c0 += 32) {
                uint32_t o[2][16];
                tc::tmem_ld<16>(tO + c0, o[0]);
                tc::tmem_ld<16>(tO + c0 + 16, o[1]);
                tc::wait_ld();
#pragma unroll
                for (int c = 0; c < 32; c += 2) {
                  uint32_t* y = &o[c >> 4][c & 15];
                  const float2 z = mul2(make_float2(__uint_as_float(y[0]), __uint_as_float(y[1])), al2);
                  y[0] = __float_as_uint(z.x);
                  y[1] = __float_as_uint(z.y);
                }
                tc::tmem_st<16>(tO + c0, o[0]);
                tc::tmem_st<16>(tO + c0 + 16, o[1]);
              }
            }
          }
          // P' of 32 tokens at a time, over the S columns just read
          const float2 nM = make_float2(-M, -M);
          float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
          for (int g0 = 0; g0 < 64; g0 += 32) {
            float2 x[16];
            logits(g0, x);
            uint32_t hi[16];
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
              const float4 f = vn[(g0 >> 2) + (i >> 1)];
#pragma unroll
              for (int k = i; k < i + 2; ++k) {
                const float2 z = fma2(x[k], qs2, nM);
                const float2 p = make_float2(fast_exp2(z.x), fast_exp2(z.y));
                sum = add2(sum, p);
                x[k] = mul2(p, k == i ? make_float2(f.x, f.y) : make_float2(f.z, f.w));
                const __half2 yh = __floats2half2_rn(x[k].x, x[k].y);
                hi[k] = *reinterpret_cast<const uint32_t*>(&yh);
              }
            }
            tc::tmem_st<16>(tS + g0, hi);
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              const float2 r = fma2(__half22float2(*reinterpret_cast<const __half2*>(&hi[k])), make_float2(-1.0f, -1.0f), x[k]);
              const __half2 yl = __floats2half2_rn(r.x, r.y);
              hi[k] = *reinterpret_cast<const uint32_t*>(&yl);
            }
            tc::tmem_st<16>(tS + g0 + 16, hi);
          }
          L += sum.x + sum.y;
        }
        tc::wait_st();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&S.vready[j & 1]);
      }
      if (!stopped) {
        if (!tc::mbar_wait(&S.ofull, (n - 1) & 1, WL)) *abort_flag = 1;
        tc::fence_after_sync();
        S.xch[n & 1][cw][t] = L;
      }
    }
  }
  __syncthreads();
  tc::fence_after_sync();
  const bool aborted = bad || S.bad_page != 0 || S.abort != 0;
  if (tid == 0) {
    // (the table's copy lands before the CTA leaves, used or not)
    if (!tc::mbar_wait(&S.setup, 0, WL) || S.abort != 0) record_status(a.status, KVQ_ERR_TIMEOUT);
  }
  // ------------------------------------------------------------------ the CTA's (m, l, O)
  if (!is_issuer) {
    const int t = 32 * q + lane;
    const size_t i = static_cast<size_t>(blockIdx.x) * kPreRows + t;
    if (wg == 2 && t < rows) {
      const float (*xc)[kPreRows] = S.xch[n & 1];
      a.part_m[i] = aborted ? __int_as_float(0x7fc00000) : M;
      a.part_l[i] = aborted ? 0.0f : xc[0][t] + xc[1][t];
    }
    if (!aborted && 32 * q < rows) {
      float4* po = reinterpret_cast<float4*>(a.part_o + i * kD + 32 * wg);
#pragma unroll
      for (int c0 = 0; c0 < 32; c0 += 16) {
        uint32_t o[16];
        tc::tmem_ld<16>(tb + kPreO + (static_cast<uint32_t>(32 * q) << 16) + 32 * wg + c0, o);
        tc::wait_ld();
        if (t < rows) {
#pragma unroll
          for (int c = 0; c < 16; c += 4)
            po[(c0 + c) >> 2] = make_float4(__uint_as_float(o[c]) * (1.0f / kPreScale), __uint_as_float(o[c + 1]) * (1.0f / kPreScale),
                                            __uint_as_float(o[c + 2]) * (1.0f / kPreScale), __uint_as_float(o[c + 3]) * (1.0f / kPreScale));
        }
      }
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (is_issuer) tc::tmem_dealloc(tb, kTmemCols);
}

}  // namespace kvq
