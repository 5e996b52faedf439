// Attention of a whole batch over one shared prefix in a paged pool, and the merge that joins
// it to every sequence's own pages.
//
// For one KV head all query rows of the batch (row = sequence * group + head of the group) meet
// the same keys and values, so each chunk of 128 tokens is dequantized once for up to R rows:
//   S^T[128 tokens][R]  = Khat x Q'^T        (tcgen05.mma, M 128, N R; fp16 high, then low parts)
//   O^T[128 dims][R]   += Vhat^T x P'^T      (the same, P' high then low parts)
// Khat and Vhat^T are written to tensor memory as in kvq_decode_gtq (decode.cuh), with Q' and
// P' in shared memory as its B operands; lane = token in the softmax, so a row's statistics
// are one value for a whole column: the running maximum sits in shared memory and moves only
// when a logit exceeds it by more than 2^3 (one vote per chunk), the row sums are per-lane
// registers until the end.
//
// A CTA owns a range of chunks for one KV head and one group of R rows and runs kPipes
// pipelines over it, each of 4 / kPipes warpgroups and one issuing warp: the warpgroups of
// a pipeline share out a chunk's K columns and V tiles, then its rows. While one pipeline waits
// for its products another computes; with R = 128 tensor memory holds only one pipeline, whose V
// buffer is then apart from its K buffer, so O's products run under the next chunk's lookups.
// Each pipeline leaves (m, l, O) of its R rows to the merge.
//
// Every wait is bounded, as in kvq_decode_gtq; a CTA that gave up, or met a bad header or page,
// leaves NaN maxima, at which the merge leaves the rows as they are.
#pragma once

#include "decode.cuh"
#include "quantize.cuh"

namespace kvq {

constexpr int kPreThr = 3;                // lazy rescale threshold (log2 units), as in the paged decode

struct PrefixArgs {
  const void* q;
  int64_t qsb, qsh;
  int q_dtype;
  int n_rows, group;                      // query rows per KV head, rows per sequence
  const uint8_t* pool;
  const kvq_head_alloc* alloc;
  PagedArgs pg;
  const int32_t* pages;                   // the prefix's pages
  int len, splits, row_groups, n_stages;
  float* part_m;                          // [entry][R], entry = CTA * kPipes + pipeline
  float* part_l;
  float* part_o;                          // [entry][R][128]
  unsigned* status;
  uint32_t wait_limit;
  int debug_no_loads;
};

template <int R, int kPipes>
struct PrefixCfg {
  static constexpr int kWgs = 4 / kPipes;                    // warpgroups of a pipeline
  static constexpr int kCols = R / kWgs;                     // rows a warpgroup's softmax takes
  static constexpr int kThreads = (16 + kPipes) * 32;
  static constexpr bool kShareKV = kPipes > 1;               // one buffer for K-hat, then V-hat^T
  static constexpr int kVCol = kShareKV ? 0 : 96;
  static constexpr int kSCol = kShareKV ? 96 : 160;
  static constexpr int kOCol = kSCol + R;
  static constexpr int kPipeCols = kOCol + R;
  static_assert(kPipes * kPipeCols <= static_cast<int>(kTmemCols), "tensor memory");
  static_assert(kCols % 16 == 0 && R % 16 == 0, "columns in batches of 16");
  // shared memory: lookup tables, allocation, Q' high and low, P' high and low, header, stages
  static constexpr int kQBytes = 192 * R * 2;
  static constexpr int kPBytes = kChunkTokens * R * 2;
  static constexpr int kQOff = kBQOff;
  static constexpr int kPOff = kQOff + 2 * kQBytes;
  static constexpr int kHdr = kPOff + kPipes * 2 * kPBytes;
};

template <int R, int kPipes>
struct PrefixHeader {
  uint64_t full[kPipes][kStagesMax];
  uint64_t kready[kPipes], sfull[kPipes], vready[kPipes], ofull[kPipes], drain[kPipes];
  uint64_t setup;
  uint32_t tmem_base;
  int bad, bad_page;
  int pipe_abort[kPipes];
  int wg_stop[4];                          // the warpgroup leaves its loop (read between two of its barriers)
  uint4 kdesc[kPlanSlots];
  uint32_t kbase[kPlanSlots];
  int bkind[kPlanSlots / 4];
  int8_t col_of[kH];                       // column of a block (-1: width 0)
  alignas(16) float qscale[R];             // 2^e of row r
  alignas(16) float neg_m[kPipes][R];      // minus the running maximum
  alignas(16) float limit[kPipes][R];      // (maximum + 2^3's exponent) / 2^e: S * norm above it moves the maximum
  alignas(16) float alpha[kPipes][R];
  float xch[4][4][PrefixCfg<R, kPipes>::kCols];
  float lred[4][4][PrefixCfg<R, kPipes>::kCols];
};

template <int R, int kPipes>
__host__ __device__ constexpr int prefix_stage_off() {
  return PrefixCfg<R, kPipes>::kHdr + (static_cast<int>(sizeof(PrefixHeader<R, kPipes>)) + 127) / 128 * 128;
}

// V-hat^T values of one tile for a run-time width.
__device__ __forceinline__ void v_vals_any(int bv, const uint32_t* vw, const uint8_t* sm, uint32_t lane4, uint32_t (&v)[16]) {
  switch (bv) {
    case 1: v_vals<1>(vw, sm, lane4, v); break;
    case 2: v_vals<2>(vw, sm, lane4, v); break;
    case 3: v_vals<3>(vw, sm, lane4, v); break;
    case 4: v_vals<4>(vw, sm, lane4, v); break;
    case 5: v_vals<5>(vw, sm, lane4, v); break;
    case 6: v_vals<6>(vw, sm, lane4, v); break;
    case 7: v_vals<7>(vw, sm, lane4, v); break;
    default: v_vals<8>(vw, sm, lane4, v); break;
  }
}

template <int R, int kPipes>
__global__ void __launch_bounds__(PrefixCfg<R, kPipes>::kThreads, 1) kvq_prefix_gtq(const PrefixArgs a) {
  using C = PrefixCfg<R, kPipes>;
  constexpr int kWgs = C::kWgs, kCols = C::kCols;
  extern __shared__ __align__(1024) uint8_t sm[];
  PrefixHeader<R, kPipes>& S = *reinterpret_cast<PrefixHeader<R, kPipes>*>(sm + C::kHdr);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int hkv = blockIdx.x % a.pg.n_kv_heads;
  const int rg = blockIdx.x / a.pg.n_kv_heads % a.row_groups;
  const int split = blockIdx.x / (a.pg.n_kv_heads * a.row_groups);
  const kvq_head_alloc* al = a.alloc + hkv;
  const int rec_bytes = a.pg.rec_bytes, cbytes = kChunkTiles * rec_bytes, kbytes = 4 * kD * a.pg.bits_k;
  const int NS = a.n_stages;
  const float inv_sqrt_d = 0.08838834764831845f;
  const uint32_t WL = a.wait_limit;
  const bool is_issuer = warp >= 16;
  const int pipe = is_issuer ? warp - 16 : warp / (4 * kWgs);
  const int wg = (warp >> 2) % kWgs;                        // warpgroup inside its pipeline
  const int q = warp & 3;                                   // tensor-memory quarter
  const bool issuer = is_issuer && lane == 0;
  uint8_t* my_stages = sm + prefix_stage_off<R, kPipes>() + static_cast<size_t>(pipe) * NS * cbytes;

  if (tid == 0) {
    for (int i = 0; i < 4; ++i) S.wg_stop[i] = 0;
    for (int p = 0; p < kPipes; ++p) {
      for (int i = 0; i < kStagesMax; ++i) tc::mbar_init(&S.full[p][i], 1);
      tc::mbar_init(&S.kready[p], 4 * kWgs);
      tc::mbar_init(&S.sfull[p], 1);
      tc::mbar_init(&S.vready[p], 4 * kWgs);
      tc::mbar_init(&S.ofull[p], 1);
      tc::mbar_init(&S.drain[p], 1);
      S.pipe_abort[p] = 0;
    }
    tc::mbar_init(&S.setup, 1);
    S.bad = 0;
    S.bad_page = 0;
    tc::mbar_fence_init();
    tc::mbar_arrive_expect_tx(&S.setup, kLutBytes + static_cast<uint32_t>(sizeof(kvq_head_alloc)));
    tc::bulk_g2s(sm, g_dec_lut, kLutBytes, &S.setup);
  }
  if (warp == 16) tc::tmem_alloc(&S.tmem_base, kTmemCols);
  for (int i = tid; i < 2 * C::kQBytes / 16; i += C::kThreads)
    reinterpret_cast<uint4*>(sm + C::kQOff)[i] = make_uint4(0u, 0u, 0u, 0u);
  if (tid < kPipes * R) {
    (&S.neg_m[0][0])[tid] = INFINITY;
    (&S.limit[0][0])[tid] = -INFINITY;
  }
  if (tid < kH) S.col_of[tid] = -1;
  grid_dependency_wait();
  if (tid == 0) tc::bulk_g2s(sm + kAllocOff, al, sizeof(kvq_head_alloc), &S.setup);
  if (tid == 32) {
    unsigned code = paged_header_code(a.pool, a.pg);
    const uint64_t dg = paged_digest(a.pool, hkv), ad = al->digest;
    const int abk = al->bits_k, akw = al->k_words, apk = al->plan_k_cols, aps = al->plan_n_slots;
    if (!code && !((dg == ad) & (abk == a.pg.bits_k) & (akw == a.pg.bits_k * kD) & (apk <= 96) & (apk >= 8) &
                   (aps >= 1) & (aps <= kPlanSlots)))
      code = KVQ_ERR_MISMATCH;
    if (code) {
      S.bad = 1;
      record_status(a.status, code);
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tbase = S.tmem_base + static_cast<uint32_t>(pipe) * C::kPipeCols;

  const int n_tiles = (a.len + kTile - 1) / kTile;
  const int n_chunks_all = (n_tiles + kChunkTiles - 1) / kChunkTiles;
  const int c_begin = static_cast<int>((static_cast<long long>(split) * n_chunks_all) / a.splits);
  const int c_end = static_cast<int>((static_cast<long long>(split + 1) * n_chunks_all) / a.splits);
  const int n_chunks = c_end - c_begin;
  const int nj = (n_chunks > pipe) ? (n_chunks - pipe + kPipes - 1) / kPipes : 0;   // this pipeline's chunks

  int issued = 0;
  auto issue_chunk = [&](int j) {                           // issuer only
    const int tile0 = (c_begin + pipe + kPipes * j) * kChunkTiles;
    const int nt = min(kChunkTiles, n_tiles - tile0);
    const int s = j % NS;
    tc::mbar_arrive_expect_tx(&S.full[pipe][s], static_cast<uint32_t>(nt * rec_bytes));
    paged_copy_tiles(my_stages + static_cast<size_t>(s) * cbytes, a.pool, a.pg, a.pages, tile0, nt, hkv,
                     &S.full[pipe][s], &S.bad_page, a.status);
  };
  if (issuer && !S.bad && !a.debug_no_loads) {
    for (; issued < min(NS, nj); ++issued) issue_chunk(issued);
  }
  if (!tc::mbar_wait(&S.setup, 0, WL)) {
    S.bad = 1;
    record_status(a.status, KVQ_ERR_TIMEOUT);
  }
  __syncthreads();
  const kvq_head_alloc& A = *reinterpret_cast<const kvq_head_alloc*>(sm + kAllocOff);
  // ------------------------------------------------------------------ slot descriptors, columns
  if (tid < kPlanSlots) {
    const uint32_t e = A.plan_slot[tid];
    uint32_t w = e & 15u, off = e >> 8;
    if (w > 8 || (w > 0 && off >= static_cast<uint32_t>(kD * a.pg.bits_k))) {
      S.bad = 1;
      record_status(a.status, KVQ_ERR_MISMATCH);
    }
    if (w == 0 || w > 5 || off >= static_cast<uint32_t>(kD * a.pg.bits_k)) { w = 1; off = 0; }
    S.kdesc[tid] = make_uint4((off >> 5) * 128u, (off & 31u) | (2 * w) << 8 | (4 * w) << 16 | (6 * w) << 24,
                              (1u << (2 * w)) - 1u, w <= 3 ? 128u : 4u);
    S.kbase[tid] = static_cast<uint32_t>(pair_off(static_cast<int>(w)));
  } else if (tid >= 32 && tid < 32 + kPlanSlots / 4) {
    uint32_t wmax = 0;
    for (int i = 0; i < 4; ++i) wmax = max(wmax, A.plan_slot[4 * (tid - 32) + i] & 15u);
    S.bkind[tid - 32] = wmax <= 5 ? 0 : 1;
  } else if (tid >= 64 && tid < 64 + 96) {
    const int blk = A.plan_col_block[tid - 64];
    if (blk >= 0 && blk < kH && tid - 64 < A.plan_k_cols) S.col_of[blk] = static_cast<int8_t>(tid - 64);
  }
  __syncthreads();
  // ------------------------------------------------------------------ Q' (a warp per row)
  // Row r: q * f_b * log2(e) / sqrt(d), scaled by 2^-e so its largest |value| is in [0.5, 1); the
  // B operand of S, K-major, no swizzle: element (n, k) at (k / 8) * 16 R + (n / 8) * 128 +
  // (n % 8) * 16 + (k % 8) * 2, k = 2 * column + half. Rows past the batch stay zero.
  for (int r = warp; r < R; r += 16 + kPipes) {
    const int row = rg * R + r;
    float x[4] = {0.f, 0.f, 0.f, 0.f};                      // dims 2l, 2l + 1, 64 + 2l, 65 + 2l
    if (row < a.n_rows) {
      const int b = row / a.group;
      const int64_t qi = b * a.qsb + (static_cast<int64_t>(hkv) * a.group + (row - b * a.group)) * a.qsh + 2 * lane;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        x[i] = load_f32(a.q, a.q_dtype, qi + (i >> 1) * kH + (i & 1)) * (A.dequant[2 * lane + (i & 1)] * (inv_sqrt_d * kLog2e));
    }
    float mx = fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3])));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    int e = 0;
    if (mx > 0.0f) frexpf(mx, &e);
    e = max(e, -126);                                       // 2^-e stays finite
    const float sc = ldexpf(1.0f, -e);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int c = S.col_of[2 * lane + i];
      if (c < 0) continue;
      uint32_t h0, l0, h1, l1;
      split16<false>(x[i] * sc, h0, l0);
      split16<false>(x[2 + i] * sc, h1, l1);
      uint8_t* p = sm + C::kQOff + (c >> 2) * (16 * R) + (r >> 3) * 128 + (r & 7) * 16 + (c & 3) * 4;
      *reinterpret_cast<uint32_t*>(p) = h0 | (h1 << 16);
      *reinterpret_cast<uint32_t*>(p + C::kQBytes) = l0 | (l1 << 16);
    }
    if (lane == 0) S.qscale[r] = ldexpf(1.0f, e);
  }
  tc::fence_proxy_async_smem();
  __syncthreads();
  const bool bad = S.bad != 0;
  volatile int* abort_flag = &S.pipe_abort[pipe];

  float L[kCols];                                           // this lane's share of the row sums
#pragma unroll
  for (int c = 0; c < kCols; ++c) L[c] = 0.0f;

  if (!bad && is_issuer) {
    if (issuer) {
      const uint32_t id_s = tc::idesc_f16(128, R, false), id_o = tc::idesc_f16(128, R, true);
      const uint32_t bq = tc::smem_u32(sm + C::kQOff), bp = tc::smem_u32(sm + C::kPOff + pipe * 2 * C::kPBytes);
      const int k_steps = A.plan_k_cols >> 3;
      bool ok = true;
      for (int j = 0; j < nj; ++j) {
        if (!tc::mbar_wait(&S.kready[pipe], j & 1, WL)) { ok = false; break; }
        tc::fence_after_sync();
        for (int ks = 0; ks < k_steps; ++ks)
          tc::mma_ts(tbase + C::kSCol, tbase + 8 * ks, tc::sdesc(bq + 32 * R * ks, 16 * R, 128), id_s, ks > 0 ? 1u : 0u);
        for (int ks = 0; ks < k_steps; ++ks)
          tc::mma_ts(tbase + C::kSCol, tbase + 8 * ks, tc::sdesc(bq + C::kQBytes + 32 * R * ks, 16 * R, 128), id_s, 1u);
        tc::mma_commit(&S.sfull[pipe]);
        if (!tc::mbar_wait(&S.vready[pipe], j & 1, WL)) { ok = false; break; }
        tc::fence_after_sync();
#pragma unroll
        for (int ks = 0; ks < 2 * (kChunkTokens / 16); ++ks) {
          const int kk = ks % (kChunkTokens / 16);          // high parts, then low parts
          tc::mma_ts(tbase + C::kOCol, tbase + C::kVCol + 8 * kk,
                     tc::sdesc(bp + (ks >= kChunkTokens / 16 ? C::kPBytes : 0) + 32 * R * kk, 16 * R, 128), id_o,
                     (j > 0 || ks > 0) ? 1u : 0u);
        }
        tc::mma_commit(&S.ofull[pipe]);
        if (issued < nj && !a.debug_no_loads) issue_chunk(issued++);   // the stage is consumed: refill it
      }
      if (!ok) *abort_flag = 1;
      tc::mma_commit(&S.drain[pipe]);
      tc::mbar_wait(&S.drain[pipe], 0, WL);
      for (int s = 0; s < NS; ++s) {
        int last = -1;
        for (int j = s; j < issued; j += NS) last = j;
        if (last >= 0) tc::mbar_wait(&S.full[pipe][s], (last / NS) & 1, WL);
      }
    }
    __syncwarp();
  } else if (!bad) {
    // ------------------------------------------------------------------ compute warps
    const uint32_t lane_base = static_cast<uint32_t>(32 * q) << 16;
    const uint32_t lane4 = static_cast<uint32_t>(lane) << 2;
    const uint32_t tS = tbase + C::kSCol + lane_base + wg * kCols, tO = tbase + C::kOCol + lane_base + wg * kCols;
    const int nb = (min(A.plan_n_slots, kPlanSlots) + 3) >> 2;
    const int bar_id = 1 + pipe * kWgs + wg;
    const int t = 32 * q + lane;                            // token of the chunk
    uint8_t* pb = sm + C::kPOff + pipe * 2 * C::kPBytes + (t >> 3) * (16 * R) + (t & 7) * 16 + wg * (kCols / 8) * 128;
    const uint4* slots4 = reinterpret_cast<const uint4*>(A.plan_slot);
    const float* qs = S.qscale + wg * kCols;
    float* nm = S.neg_m[pipe] + wg * kCols;
    float* lim = S.limit[pipe] + wg * kCols;
    float* alp = S.alpha[pipe] + wg * kCols;
    float (*xch)[kCols] = S.xch[pipe * kWgs + wg];
    int done = 0;

    for (int j = 0; j < nj; ++j) {
      const int ci = c_begin + pipe + kPipes * j;
      const int s = j % NS;
      const uint8_t* st = my_stages + static_cast<size_t>(s) * cbytes;
      if (!tc::mbar_wait(&S.full[pipe][s], (j / NS) & 1, WL)) *abort_flag = 1;
      // -------------------------------------------------------------- keys (lane = token)
      const uint8_t* tq = st + q * rec_bytes;
      const uint32_t* kw = reinterpret_cast<const uint32_t*>(tq) + lane;
      bool free_waited = !C::kShareKV || j == 0;            // V-hat^T of the last chunk is read
      for (int bt = wg; bt < nb; bt += kWgs) {
        uint32_t v16[16];
        if (S.bkind[bt] == 0) k_batch_gen(kw, S.kdesc + 4 * bt, S.kbase + 4 * bt, sm, lane4, v16);
        else k_batch(kw, slots4[bt], sm, lane4, v16);
        if (!free_waited) {
          if (!tc::mbar_wait(&S.ofull[pipe], (j - 1) & 1, WL)) *abort_flag = 1;
          tc::fence_after_sync();
          free_waited = true;
        }
        tc::tmem_st<16>(tbase + lane_base + 16 * bt, v16);
      }
      tc::wait_st();
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&S.kready[pipe]);
      const bool valid = ci * kChunkTokens + t < a.len;
      const float kn = valid ? __half2float(__ushort_as_half(reinterpret_cast<const uint16_t*>(tq + kbytes)[lane])) : 0.0f;
      const float vs = valid ? __half2float(__ushort_as_half(reinterpret_cast<const uint16_t*>(tq + kbytes + 2 * kTile)[lane])) *
                                   inv_sqrt_d : 0.0f;
      // -------------------------------------------------------------- values (lane = dim)
      uint32_t vv[kChunkTiles / kWgs][16];
#pragma unroll
      for (int i = 0; i < kChunkTiles / kWgs; ++i) {
        const int u = wg + kWgs * i;
        const uint32_t* vw = reinterpret_cast<const uint32_t*>(st + u * rec_bytes + kbytes + 4 * kTile) + t;
        v_vals_any(a.pg.bits_v, vw, sm, lane4, vv[i]);
      }
      // V-hat^T's columns and P' are free once the previous chunk's O products are complete, and
      // a shared buffer once this chunk's S products are
      if (j > 0 && !tc::mbar_wait(&S.ofull[pipe], (j - 1) & 1, WL)) *abort_flag = 1;
      if (!tc::mbar_wait(&S.sfull[pipe], j & 1, WL)) *abort_flag = 1;
      tc::fence_after_sync();
#pragma unroll
      for (int i = 0; i < kChunkTiles / kWgs; ++i)
        tc::tmem_st<16>(tbase + C::kVCol + lane_base + 16 * (wg + kWgs * i), vv[i]);
      // -------------------------------------------------------------- does a maximum move?
      const float2 kn2 = make_float2(kn, kn);
      bool over = false;
#pragma unroll
      for (int c0 = 0; c0 < kCols; c0 += 16) {
        uint32_t sr[16];
        tc::tmem_ld<16>(tS + c0, sr);
        tc::wait_ld();
#pragma unroll
        for (int c = 0; c < 16; c += 4) {
          const float4 l4 = *reinterpret_cast<const float4*>(lim + c0 + c);
          const float2 x = mul2(make_float2(__uint_as_float(sr[c]), __uint_as_float(sr[c + 1])), kn2);
          const float2 y = mul2(make_float2(__uint_as_float(sr[c + 2]), __uint_as_float(sr[c + 3])), kn2);
          over |= (x.x > l4.x) | (x.y > l4.y) | (y.x > l4.z) | (y.y > l4.w);
        }
      }
      // a wait that gave up joins the vote, so that the warpgroup stops as one
      const bool stop = *abort_flag != 0;
      const bool any_over = named_sync_or(bar_id, 128, (over && valid) || stop);
      if (any_over) {
        if (stop) S.wg_stop[pipe * kWgs + wg] = 1;
#pragma unroll
        for (int c0 = 0; c0 < kCols; c0 += 16) {
          uint32_t sr[16];
          tc::tmem_ld<16>(tS + c0, sr);
          tc::wait_ld();
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            const float x = valid ? __uint_as_float(sr[c]) * kn * qs[c0 + c] : -INFINITY;
            const int m = __reduce_max_sync(0xffffffffu, ordered(x));
            if (lane == 0) xch[q][c0 + c] = from_ordered(m);
          }
        }
        named_sync(bar_id, 128);
        if (*reinterpret_cast<volatile int*>(&S.wg_stop[pipe * kWgs + wg])) break;
        if (q == 0 && lane < kCols) {
          const float old = -nm[lane];
          const float mn = fmaxf(old, fmaxf(fmaxf(xch[0][lane], xch[1][lane]), fmaxf(xch[2][lane], xch[3][lane])));
          alp[lane] = (old == -INFINITY) ? 0.0f : fast_exp2(old - mn);
          nm[lane] = -mn;
          lim[lane] = (mn + static_cast<float>(kPreThr)) / qs[lane];
        }
        named_sync(bar_id, 128);
#pragma unroll
        for (int c = 0; c < kCols; ++c) L[c] *= alp[c];
        if (j > 0) {                                        // O holds earlier chunks (lane = dim)
#pragma unroll
          for (int c0 = 0; c0 < kCols; c0 += 16) {
            uint32_t o[16];
            tc::tmem_ld<16>(tO + c0, o);
            tc::wait_ld();
#pragma unroll
            for (int c = 0; c < 16; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * alp[c0 + c]);
            tc::tmem_st<16>(tO + c0, o);
          }
        }
      }
      // -------------------------------------------------------------- P' (lane = token)
      const float2 vs2 = make_float2(vs, vs);
      const float gone = valid ? 0.0f : -INFINITY;
#pragma unroll
      for (int c0 = 0; c0 < kCols; c0 += 16) {
        uint32_t sr[16];
        tc::tmem_ld<16>(tS + c0, sr);
        tc::wait_ld();
#pragma unroll
        for (int c8 = 0; c8 < 16; c8 += 8) {
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int c = 0; c < 8; c += 2) {
            const int cc = c8 + c;
            const float2 qv = *reinterpret_cast<const float2*>(qs + c0 + cc);
            const float2 mv = *reinterpret_cast<const float2*>(nm + c0 + cc);
            const float2 x = mul2(make_float2(__uint_as_float(sr[cc]), __uint_as_float(sr[cc + 1])), kn2);
            const float2 z = fma2(x, qv, add2(mv, make_float2(gone, gone)));
            const float2 p = make_float2(fast_exp2(z.x), fast_exp2(z.y));
            L[c0 + cc] += p.x;
            L[c0 + cc + 1] += p.y;
            const float2 y = mul2(p, vs2);
            const __half2 h = __floats2half2_rn(y.x, y.y);
            const float2 hf = __half22float2(h);
            const __half2 l = __floats2half2_rn(y.x - hf.x, y.y - hf.y);
            hi[c >> 1] = *reinterpret_cast<const uint32_t*>(&h);
            lo[c >> 1] = *reinterpret_cast<const uint32_t*>(&l);
          }
          uint8_t* p8 = pb + ((c0 + c8) >> 3) * 128;
          *reinterpret_cast<uint4*>(p8) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          *reinterpret_cast<uint4*>(p8 + C::kPBytes) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
      }
      tc::fence_proxy_async_smem();
      tc::wait_st();
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&S.vready[pipe]);
      done = j + 1;
    }
    if (done > 0 && !*abort_flag && !tc::mbar_wait(&S.ofull[pipe], (done - 1) & 1, WL)) *abort_flag = 1;
    tc::fence_after_sync();
#pragma unroll
    for (int c = 0; c < kCols; ++c) {
      float l = L[c];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
      if (lane == 0) S.lred[pipe * kWgs + wg][q][c] = l;
    }
  } else if (issuer) {
    for (int s = 0; s < NS; ++s) {
      int last = -1;
      for (int j = s; j < issued; j += NS) last = j;
      if (last >= 0) tc::mbar_wait(&S.full[pipe][s], (last / NS) & 1, WL);
    }
  }
  __syncthreads();
  allow_dependents();
  bool aborted = bad || S.bad_page != 0;
#pragma unroll
  for (int p = 0; p < kPipes; ++p) aborted |= S.pipe_abort[p] != 0;
  if (aborted && tid == 0) record_status(a.status, KVQ_ERR_TIMEOUT);    // keeps an earlier status
  // ------------------------------------------------------------------ the pipeline's (m, l, O)
  if (!is_issuer) {
    const size_t e = static_cast<size_t>(blockIdx.x) * kPipes + pipe;
    const int c_first = wg * kCols;
    if (q == 0 && lane < kCols) {
      const float (*lr)[kCols] = S.lred[pipe * kWgs + wg];
      const size_t i = e * R + c_first + lane;
      a.part_m[i] = aborted ? __int_as_float(0x7fc00000) : (nj > 0 ? -S.neg_m[pipe][c_first + lane] : -INFINITY);
      a.part_l[i] = (!aborted && nj > 0) ? lr[0][lane] + lr[1][lane] + lr[2][lane] + lr[3][lane] : 0.0f;
    }
    if (!aborted && nj > 0) {
      const int live = min(kCols, a.n_rows - rg * R - c_first);          // rows of the batch
      float* po = a.part_o + (e * R + c_first) * kD + 32 * q + lane;
#pragma unroll
      for (int c0 = 0; c0 < kCols; c0 += 16) {
        uint32_t o[16];
        tc::tmem_ld<16>(tbase + C::kOCol + (static_cast<uint32_t>(32 * q) << 16) + c_first + c0, o);
        tc::wait_ld();
#pragma unroll
        for (int c = 0; c < 16; ++c)
          if (c0 + c < live) po[(c0 + c) * kD] = __uint_as_float(o[c]);
      }
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == 16) tc::tmem_dealloc(S.tmem_base, kTmemCols);
}

// ---------------------------------------------------------------- merge

struct MergeArgs {
  void* out;
  int out_dtype, n_q_heads, n_kv_heads, group;
  const int32_t* seq_lens;
  const int2* plan;
  int direct;
  const float *own_m, *own_l, *own_o;      // [slot * n_kv_heads + head][8], ...
  int prefix_len, pre_rows, pre_groups, pre_splits, pre_pipes;
  const float *pre_m, *pre_l, *pre_o;      // [CTA * pipes + pipe][pre_rows], ...
};

constexpr int kMergeWarps = 8;

// One CTA joins the shares of one (sequence, query head): the prefix's splits, then the
// sequence's own. Warp w folds shares w, w + 8, .. with its own running maximum (lane = 4 dims,
// the loads of four shares in flight), then the warps meet in shared memory. The order of the sums is
// fixed. A NaN maximum marks a missing share: the row is left as it is.
__global__ void __launch_bounds__(kMergeWarps * 32) kvq_paged_merge(const MergeArgs a) {
  __shared__ float sm_m[kMergeWarps], sm_l[kMergeWarps];
  __shared__ float4 sm_o[kMergeWarps][32];
  const int hq = blockIdx.x % a.n_q_heads, b = blockIdx.x / a.n_q_heads;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int hkv = hq / a.group, h = hq - hkv * a.group;
  grid_dependency_wait();
  const int2 plan = __ldcg(a.plan + b);
  if (plan.y < 0 || (a.direct && plan.y == 1)) return;       // refused, or written already
  const int n_pre = a.prefix_len > 0 ? a.pre_splits * a.pre_pipes : 0;
  const int n = n_pre + plan.y;
  const int row = b * a.group + h;
  const int rg = a.prefix_len > 0 ? row / a.pre_rows : 0, r = row - rg * a.pre_rows;
  auto entry = [&](int i, const float*& m, const float*& l, const float*& o) {
    if (i < n_pre) {
      const int split = i / a.pre_pipes, pipe = i - split * a.pre_pipes;
      const size_t e = ((static_cast<size_t>(split) * a.pre_groups + rg) * a.n_kv_heads + hkv) * a.pre_pipes + pipe;
      m = a.pre_m + e * a.pre_rows + r;
      l = a.pre_l + e * a.pre_rows + r;
      o = a.pre_o + (e * a.pre_rows + r) * kD;
    } else {
      const size_t e = (static_cast<size_t>(plan.x + i - n_pre) * a.n_kv_heads + hkv) * 8 + h;
      m = a.own_m + e;
      l = a.own_l + e;
      o = a.own_o + e * kD;
    }
  };
  float M = -INFINITY, L = 0.0f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  bool missing = false;
  constexpr int kBatch = 4;
  for (int i0 = warp; i0 < n; i0 += kMergeWarps * kBatch) {
    float mv[kBatch], lv[kBatch];
    float4 ov[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int i = i0 + kMergeWarps * u;
      mv[u] = -INFINITY;
      lv[u] = 0.0f;
      ov[u] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i < n) {
        const float *pm, *pl, *po;
        entry(i, pm, pl, po);
        mv[u] = __ldcg(pm);
        lv[u] = __ldcg(pl);
        ov[u] = __ldcg(reinterpret_cast<const float4*>(po) + lane);
      }
    }
    float mx = M;
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      missing |= mv[u] != mv[u];
      mx = fmaxf(mx, mv[u]);
    }
    const float sc = (M == -INFINITY) ? 0.0f : fast_exp2(M - mx);
    L *= sc;
    o.x *= sc; o.y *= sc; o.z *= sc; o.w *= sc;
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (mv[u] == -INFINITY) {                              // no share, or one of NaN logits alone
        if (lv[u] != lv[u]) L = lv[u];
        continue;
      }
      const float wt = fast_exp2(mv[u] - mx);
      L += lv[u] * wt;
      o.x += ov[u].x * wt; o.y += ov[u].y * wt; o.z += ov[u].z * wt; o.w += ov[u].w * wt;
    }
    M = mx;
  }
  if (lane == 0) {
    sm_m[warp] = M;
    sm_l[warp] = L;
  }
  sm_o[warp][lane] = o;
  if (__syncthreads_or(missing)) return;
  if (threadIdx.x >= kD) return;
  const int d = threadIdx.x;
  float mx = -INFINITY, Ls = 0.0f, Os = 0.0f;
#pragma unroll
  for (int w = 0; w < kMergeWarps; ++w) mx = fmaxf(mx, sm_m[w]);
#pragma unroll
  for (int w = 0; w < kMergeWarps; ++w) {
    if (sm_m[w] == -INFINITY) {
      if (sm_l[w] != sm_l[w]) Ls = sm_l[w];
      continue;
    }
    const float wt = fast_exp2(sm_m[w] - mx);
    Ls += wt * sm_l[w];
    Os += wt * reinterpret_cast<const float*>(&sm_o[w][0])[d];
  }
  const bool nothing = a.prefix_len == 0 && plan.y == 0;
  store_f32(a.out, a.out_dtype, (static_cast<int64_t>(b) * a.n_q_heads + hq) * kD + d, nothing ? 0.0f : Os / Ls);
}

}  // namespace kvq
