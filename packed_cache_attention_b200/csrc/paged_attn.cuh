// Decode attention over a paged packed cache: every sequence of a ragged batch attends over its
// own pages.
//
// The arithmetic is kvq_decode_gtq's (decode.cuh): per chunk of 128 tokens
//   S^T[128 tokens][16] = Khat x Q'^T,  O^T[128 dims][16] += Vhat^T x P'^T
// with tcgen05.mma (M 128, N 16: 8 rows' high parts, then their low parts), Khat and Vhat^T looked
// up into tensor memory, an online softmax with lane = token between them.
//
// Work split. A batch's sequences differ in length by orders of magnitude, so the unit is not a
// sequence but a chunk: per KV head, all chunks of the batch form one list, cut into equal
// contiguous ranges, one per warpgroup (4 per CTA, one CTA per SM). A warpgroup walks the
// sequences of its range, building Q' anew for each, and leaves one (m, l, O) per sequence it
// met (paged_split.h). The fewest warpgroups that keep the longest range are used, spread over
// the SMs; those of a CTA that all lie in one sequence join their results first. One CTA per
// (sequence, head) instead took 217 us on 32 sequences of 64 to 16384 tokens, where the longest
// sequence set the time; this split takes 92 us.
//
// Inside a warpgroup: 64 of K-hat's 96 columns of tensor memory hold V-hat^T next (128 columns per
// warpgroup in all); the next chunk's first 32 columns are looked up while O's products run. The issuing warp copies a chunk's keys and values separately, so the keys of
// the next chunk arrive while the values of this one are used, even with a single buffer of each.
// Every wait is bounded; a warpgroup that gave up, and a segment with a page outside the pool,
// leave NaN maxima, at which the merge leaves the rows as they are.
#pragma once

#include "paged_lut.cuh"
#include "quantize.cuh"

namespace kvq {

constexpr int kPgStagesMax = 4;
constexpr int kPgVCol = 32;               // first of V-hat^T's 64 columns; K-hat has columns 0..95

struct PagedAttn {
  const void* q;
  int64_t qsb, qsh;
  int q_dtype, group;
  const uint8_t* pool;
  const kvq_head_alloc* alloc;
  PagedArgs pg;
  int ctas;                               // CTAs per KV head
  int entries;                            // per KV head: 4 * ctas + batch
  int n_stages;
  float* part_m;                          // [head][entry][8]
  float* part_l;                          // [head][entry][4 quarters][8]
  float* part_o;                          // [head][entry][8][128]
  int2* plan;                             // [batch + 1]: first chunk and chunks of a sequence (-1: not decoded);
                                          // then all chunks
  int* refused;                           // [head]: its header or allocation does not fit, its rows stay as they are
  unsigned* status;
  uint32_t wait_limit;
  int debug_no_loads;
  int after_prefix;                       // the previous grid is the same call's prefix kernel: see the kernel
};

struct PgHeader {
  uint64_t fullk[4][kPgStagesMax], fullv[4][kPgStagesMax];
  uint64_t kready[4], sfull[4], vready[4], ofull[4], drain[4];
  uint64_t setup;
  uint32_t tmem_base;
  int bad;
  int wg_abort[4], wg_stop[4];
  int stage_bad[4][kPgStagesMax];          // the chunk of this stage lies in a page outside the pool
  int k_cols;
  alignas(16) float qscale[4][8];
  float xch[4][4][8];
  float join_m[4][8], join_l[4][4][8];     // shares of one sequence: [warpgroup][row], [warpgroup][quarter][row]
  int scan[kDecThreads / 32];
  KSlots slots;
  alignas(16) float dequant[kH];
  alignas(4) int8_t col_of[kH];            // column of a block (-1: width 0)
};

// Shared memory: Q' of each warpgroup, header, chunk offsets; lookup tables (at their address);
// P', stages.
constexpr int kPgQBytes = 6144;            // 192 K elements x 16 rows
constexpr int kPgPBytes = 4096;            // 128 tokens x 16 rows
constexpr int kPgQOff = 0;
constexpr int kPgHdrOff = kPgQOff + 4 * kPgQBytes;
constexpr int kPgScanOff = kPgHdrOff + (static_cast<int>(sizeof(PgHeader)) + 15) / 16 * 16;
static_assert(kPgScanOff + 4 * (kPagedMaxBatch + 1) <= kPlutAt, "before the lookup tables");
constexpr int kPgPOff = kPlutEnd;
constexpr int kPgStageOff = kPgPOff + 4 * kPgPBytes;

// Place in a ring of stages and the parity of its phase.
struct Ring {
  int s = 0;
  uint32_t parity = 0;
  __device__ __forceinline__ void next(int n) {
    if (++s == n) {
      s = 0;
      parity ^= 1u;
    }
  }
};

// Shares the batch out: chunk offsets of the sequences to `cs` (batch + 1 entries); `len` is that of
// sequence threadIdx.x (of the lane's for up to 32 sequences), loaded ahead. A length that is negative or past the table counts as none
// and is recorded.
struct PgScan {
  int at, n;                              // of sequence threadIdx.x: first chunk, chunks (-1: refused)
};
__device__ __forceinline__ int pg_scan(const PagedAttn& a, PgHeader& S, int* cs, int len, PgScan& mine) {
  const int n = a.pg.batch;
  const long long room = static_cast<long long>(a.pg.max_pages) * a.pg.page_tiles * kTile;
  if (n <= 32) {                          // a warp's scan, which every warp makes for itself
    const int lane = threadIdx.x & 31;
    const bool ok = len >= 0 && len <= room;
    const int c = ok ? len / kChunkTokens + (len % kChunkTokens != 0) : 0;
    int inc = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += x;
    }
    const int sum = __shfl_sync(0xffffffffu, inc, 31);
    if (threadIdx.x < n) {
      if (!ok) record_status(a.status, KVQ_ERR_RANGE);
      cs[lane] = inc - c;
    }
    mine = PgScan{inc - c, ok ? c : -1};
    if (threadIdx.x == 0) {
      cs[n] = sum;
      if (blockIdx.x == 0) a.plan[n] = make_int2(sum, 0);
    }
    return sum;
  }
  int sum = 0;
  for (int b0 = 0; b0 < n; b0 += kDecThreads) {
    const int b = b0 + threadIdx.x;
    int c = 0;
    bool ok = true;
    if (b < n) {
      if (b0 > 0) len = __ldg(a.pg.seq_lens + b);
      ok = len >= 0 && len <= room;
      if (ok) c = len / kChunkTokens + (len % kChunkTokens != 0);
      else record_status(a.status, KVQ_ERR_RANGE);
    }
    int total;
    const int at = sum + block_exclusive(c, S.scan, kDecThreads / 32, total);
    if (b < n) cs[b] = at;
    if (b0 == 0) mine = PgScan{at, ok ? c : -1};
    else if (b < n && blockIdx.x == 0) a.plan[b] = make_int2(at, ok ? c : -1);
    sum += total;
  }
  if (threadIdx.x == 0) {
    cs[n] = sum;
    if (blockIdx.x == 0) a.plan[n] = make_int2(sum, 0);
  }
  return sum;
}

// kRows: query rows computed, 4 or 8 (the group is at most that many).
template <int VM, int kRows>
__global__ void __launch_bounds__(kDecThreads, 1) kvq_paged_gtq(const PagedAttn a) {
  extern __shared__ __align__(1024) uint8_t sm[];
  PgHeader& S = *reinterpret_cast<PgHeader*>(sm + kPgHdrOff);
  int* cs = reinterpret_cast<int*>(sm + kPgScanOff);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int hkv = blockIdx.x % a.pg.n_kv_heads, cta = blockIdx.x / a.pg.n_kv_heads;
  const kvq_head_alloc* al = a.alloc + hkv;
  const int kbytes = 4 * kD * a.pg.bits_k, vbytes = 4 * kTile + 4 * kD * VM;   // of a record: K words; norms, V words
  const int cbytes = kChunkTiles * (kbytes + vbytes);
  const int NS = a.n_stages;
  const float inv_sqrt_d = 0.08838834764831845f;
  const uint32_t WL = a.wait_limit;
  const bool is_issuer = warp >= kDecIssuerWarp0;
  const int g = is_issuer ? warp - kDecIssuerWarp0 : warp >> 2;
  const int q = warp & 3;
  uint8_t* my_stages = sm + kPgStageOff + static_cast<size_t>(g) * NS * cbytes;   // K of a chunk, then V

  if (tid == 0) {
    for (int i = 0; i < 4; ++i) {
      for (int s = 0; s < kPgStagesMax; ++s) {
        tc::mbar_init(&S.fullk[i][s], 1);
        tc::mbar_init(&S.fullv[i][s], 1);
      }
      tc::mbar_init(&S.kready[i], 4);
      tc::mbar_init(&S.sfull[i], 1);
      tc::mbar_init(&S.vready[i], 4);
      tc::mbar_init(&S.ofull[i], 1);
      tc::mbar_init(&S.drain[i], 1);
      S.wg_abort[i] = 0;
      S.wg_stop[i] = 0;
    }
    tc::mbar_init(&S.setup, 1);
    S.bad = tc::smem_u32(sm) != kSmemBase;                  // the tables would not be at their address
    if (S.bad) record_status(a.status, KVQ_ERR_UNSUPPORTED);
    tc::mbar_fence_init();
    tc::mbar_arrive_expect_tx(&S.setup, kPlutBytes);
    tc::bulk_g2s(sm + kPlutAt, g_paged_lut, kPlutBytes, &S.setup);
  }
  if (warp == kDecIssuerWarp0) tc::tmem_alloc(&S.tmem_base, kTmemCols);
  for (int i = tid; i < 4 * kPgQBytes / 16; i += kDecThreads)
    reinterpret_cast<uint4*>(sm + kPgQOff)[i] = make_uint4(0u, 0u, 0u, 0u);
  if (tid < kH) S.col_of[tid] = -1;
  __syncthreads();
  // Behind the same call's prefix kernel this grid starts as soon as that one's CTAs run: they have
  // waited for everything before the call, and nothing here depends on the prefix. The merge does, and
  // waits for this grid alone, so this one waits for the prefix kernel before it ends.
  if (!a.after_prefix) grid_dependency_wait();
  // ------------------------------------------------------------------ header, slots, the batch
  const int scan_i = a.pg.batch <= 32 ? lane : tid;
  const int len0 = scan_i < a.pg.batch ? __ldg(a.pg.seq_lens + scan_i) : 0;
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
    const int c = tid - 64, blk = al->plan_col_block[c];
    if (blk >= 0 && blk < kH && c < al->plan_k_cols) S.col_of[blk] = static_cast<int8_t>(c);
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
  PgScan mine;
  const int chunks = pg_scan(a, S, cs, len0, mine);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const bool bad = S.bad != 0;
  if (blockIdx.x == 0 && tid < a.pg.batch) a.plan[tid] = make_int2(mine.at, mine.n);
  if (cta == 0 && tid == 0) a.refused[hkv] = bad;
  const uint32_t tbase = S.tmem_base + 128u * g;            // K-hat 96 (V-hat^T in 64 of them), S 16, O 16
  const uint32_t tS = tbase + 96, tO = tbase + 112;
  const Shares sh(chunks, a.ctas);
  const CtaShare mine_cta(sh, cs, a.pg.batch, cta);         // this CTA's workers
  const int w_cta = mine_cta.w, w_end = mine_cta.w_end, b_cta = mine_cta.b;
  const bool joint = mine_cta.joint;
  const int w = g < sh.per_cta ? w_cta + g : sh.workers;
  const int x0 = w < sh.workers ? sh.first(w) : 0, x1 = w < sh.workers ? sh.first(w + 1) : 0;
  const int b0 = x1 > x0 ? find_span(cs, a.pg.batch, x0) : 0;
  volatile int* abort_flag = &S.wg_abort[g];
  const size_t e0 = static_cast<size_t>(hkv) * a.entries + w;   // entry of sequence b: e0 + b

  if (bad) {
    // no share of this head is usable
    if (!is_issuer && q == 0 && lane < 8)
      for (int x = x0, b = b0; x < x1; ++b)
        if (cs[b + 1] > x) {
          a.part_m[(e0 + b) * 8 + lane] = __int_as_float(0x7fc00000);
          x = cs[b + 1];
        }
  } else if (is_issuer) {
    // ------------------------------------------------------------------ issuing warp
    // One lane, elected rather than lane 0, issues the products (4.5 -> 4.3 us per 4 chunks of an SM);
    // lanes 0..3 each copy one tile of a chunk.
    struct Cursor {
      int b, c, nt;                                         // sequence, chunk of it, its tiles
    };
    auto tiles_of = [&](int b) { return (__ldg(a.pg.seq_lens + b) + kTile - 1) / kTile; };
    auto advance = [&](Cursor& u) {                         // to the next chunk of the list
      if ((u.c + 1) * kChunkTiles < u.nt) {
        ++u.c;
      } else {
        u.c = 0;
        do ++u.b; while (u.b + 1 < a.pg.batch && cs[u.b + 1] == cs[u.b]);
        u.nt = u.b < a.pg.batch ? tiles_of(u.b) : 0;
      }
    };
    const int total = x1 - x0;
    Cursor ck{b0, 0, 0}, cv{b0, 0, 0};
    if (total > 0) {
      ck.c = cv.c = x0 - cs[b0];
      ck.nt = cv.nt = tiles_of(b0);
    }
    int nk = 0, nv = 0;                                     // chunks whose K (V) copies are started
    Ring rk, rv;
    auto copy_k = [&]() {
      const int tile = ck.c * kChunkTiles + lane;
      const int nt = min(kChunkTiles, ck.nt - ck.c * kChunkTiles), s = rk.s;
      bool off = false;
      const uint8_t* rec = nullptr;
      if (lane < nt) rec = paged_record(a.pool, a.pg, a.pg.block_table + ck.b * a.pg.table_stride, tile, hkv, off);
      const bool any_off = __any_sync(0xffffffffu, off);
      if (lane == 0) {
        if (any_off) record_status(a.status, KVQ_ERR_RANGE);
        *reinterpret_cast<volatile int*>(&S.stage_bad[g][s]) = any_off;
        tc::mbar_arrive_expect_tx(&S.fullk[g][s], static_cast<uint32_t>(nt * kbytes));
      }
      __syncwarp();
      if (lane < nt) tc::bulk_g2s(my_stages + static_cast<size_t>(s) * cbytes + lane * kbytes, rec, kbytes, &S.fullk[g][s]);
      ++nk;
      rk.next(NS);
      if (nk < total) advance(ck);
    };
    auto copy_v = [&]() {
      const int tile = cv.c * kChunkTiles + lane;
      const int nt = min(kChunkTiles, cv.nt - cv.c * kChunkTiles), s = rv.s;
      bool off = false;
      const uint8_t* rec = nullptr;
      if (lane < nt) rec = paged_record(a.pool, a.pg, a.pg.block_table + cv.b * a.pg.table_stride, tile, hkv, off);
      if (lane == 0) tc::mbar_arrive_expect_tx(&S.fullv[g][s], static_cast<uint32_t>(nt * vbytes));
      __syncwarp();
      if (lane < nt)
        tc::bulk_g2s(my_stages + static_cast<size_t>(s) * cbytes + kChunkTiles * kbytes + lane * vbytes, rec + kbytes, vbytes,
                     &S.fullv[g][s]);
      ++nv;
      rv.next(NS);
      if (nv < total) advance(cv);
    };
    const bool loads = !a.debug_no_loads;
    if (loads)
      while (nv < min(NS, total)) {
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
    const uint32_t id_s = tc::idesc_f16(128, 16, false), id_o = tc::idesc_f16(128, 16, true);
    const uint32_t bq = tc::smem_u32(sm + kPgQOff + g * kPgQBytes), bp = tc::smem_u32(sm + kPgPOff + g * kPgPBytes);
    const int k_steps = S.k_cols >> 3;
    bool ok = true;
    int seg_end = total > 0 ? cs[b0 + 1] : 0, seg_b = b0;   // end of the current sequence in the list
    bool fresh = true;                                      // the next chunk is the first of its segment
    for (int j = 0; j < total; ++j) {
      if (x0 + j == seg_end) {
        do ++seg_b; while (cs[seg_b + 1] == seg_end);
        seg_end = cs[seg_b + 1];
        fresh = true;
      }
      if (!wait_warp(&S.kready[g], j & 1)) { ok = false; break; }
      tc::fence_after_sync();
      if (tc::elect_one()) {
        // (from the narrow blocks to the wide ones: sums are cut off at 24 bits after every step)
        for (int ks = k_steps - 1; ks >= 0; --ks)
          tc::mma_ts(tS, tbase + 8 * ks, tc::sdesc(bq + 512 * ks, 256, 128), id_s, ks < k_steps - 1 ? 1u : 0u);
        tc::mma_commit(&S.sfull[g]);
      }
      __syncwarp();
      if (nk < total && loads) copy_k();                    // the chunk's keys are read: the next ones
      if (!wait_warp(&S.vready[g], j & 1)) { ok = false; break; }
      tc::fence_after_sync();
      if (tc::elect_one()) {
#pragma unroll
        for (int ks = 0; ks < kChunkTokens / 16; ++ks)
          tc::mma_ts(tO, tbase + kPgVCol + 8 * ks, tc::sdesc(bp + 512 * ks, 256, 128), id_o, (!fresh || ks > 0) ? 1u : 0u);
        tc::mma_commit(&S.ofull[g]);
      }
      __syncwarp();
      fresh = false;
      if (nv < total && loads) copy_v();
    }
    if (!ok) *abort_flag = 1;
    // products committed and copies started end before the CTA frees what they use
    if (tc::elect_one()) tc::mma_commit(&S.drain[g]);
    if (lane == 0) {
      tc::mbar_wait(&S.drain[g], 0, WL);
      for (int s = 0; s < NS; ++s) {
        if (nk > s) tc::mbar_wait(&S.fullk[g][s], ((nk - 1 - s) / NS) & 1, WL);
        if (nv > s) tc::mbar_wait(&S.fullv[g][s], ((nv - 1 - s) / NS) & 1, WL);
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------------ compute warps
    const uint32_t lane_base = static_cast<uint32_t>(32 * q) << 16;
    const uint32_t lane4 = static_cast<uint32_t>(lane) << 2, tab = plut_lane(VM, lane);
    const int t = 32 * q + lane;                            // token of a chunk, dim of a value, thread of the warpgroup
    uint8_t* pb = sm + kPgPOff + g * kPgPBytes + (t >> 3) * 256 + (t & 7) * 16;
    uint8_t* qb = sm + kPgQOff + g * kPgQBytes;
    const float* qs = S.qscale[g];
    if (x1 > x0 && !tc::mbar_wait(&S.setup, 0, WL)) *abort_flag = 1;

    int j = 0;                                              // chunks done
    Ring ring;
    int x = x0, b = b0;
    bool stopped = false;
    while (x < x1) {
      const int nseg = min(x1, cs[b + 1]) - x;
      const int len = __ldg(a.pg.seq_lens + b);
      const int c_first = x - cs[b];
      // -------------------------------------------------------------- Q' (16 threads a row)
      // Row h: q * f_b * log2(e) / sqrt(d) by a power of two (query_scale); B operand of S, K-major: element (n, k) at (k / 8) * 256 + (n / 8) * 128 + (n % 8) * 16 + (k % 8) * 2, k = 2 * column
      // + half; n < 8 high parts, n >= 8 low parts. The last chunk's products have read the old one.
      {
        const int h = t >> 4, i4 = 4 * (t & 15);
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 0.0f;
        if (h < a.group) {
          const int64_t qi = b * a.qsb + (static_cast<int64_t>(hkv) * a.group + h) * a.qsh + i4;
          const float4 f = *reinterpret_cast<const float4*>(S.dequant + i4);
          by_dtype(a.q_dtype, [&](auto dt) {
            const float4 lo = load4<dt.value>(a.q, qi), hi = load4<dt.value>(a.q, qi + kH);
            v[0] = lo.x * f.x; v[1] = lo.y * f.y; v[2] = lo.z * f.z; v[3] = lo.w * f.w;
            v[4] = hi.x * f.x; v[5] = hi.y * f.y; v[6] = hi.z * f.z; v[7] = hi.w * f.w;
          });
        }
        uint32_t mx = 0u;
#pragma unroll
        for (int i = 0; i < 8; ++i) mx = max(mx, abs_bits(v[i]));
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        float back;
        const float sc = query_scale(mx, back);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int c = S.col_of[i4 + i];
          if (c < 0) continue;
          uint32_t h0, l0, h1, l1;
          split16<false>(v[i] * sc, h0, l0);
          split16<false>(v[4 + i] * sc, h1, l1);
          uint8_t* p = qb + (c >> 2) * 256 + h * 16 + (c & 3) * 4;
          *reinterpret_cast<uint32_t*>(p) = h0 | (h1 << 16);
          *reinterpret_cast<uint32_t*>(p + 128) = l0 | (l1 << 16);
        }
        if ((t & 15) == 0) S.qscale[g][h] = back;
        tc::fence_proxy_async_smem();
        named_sync(1 + g, 128);
      }
      float2 nM[kRows / 2], L[kRows / 2];                   // minus the running maxima (-M); this lane's row sums
#pragma unroll
      for (int h = 0; h < kRows / 2; ++h) {
        nM[h] = make_float2(INFINITY, INFINITY);
        L[h] = make_float2(0.0f, 0.0f);
      }
      int seg_bad = 0;
      for (int i = 0; i < nseg; ++i, ++j) {
        const int s = ring.s;
        const uint8_t* st = my_stages + static_cast<size_t>(s) * cbytes;
        // ------------------------------------------------------------ keys (lane = token)
        if (!tc::mbar_wait(&S.fullk[g][s], ring.parity, WL)) *abort_flag = 1;
        seg_bad |= *reinterpret_cast<volatile int*>(&S.stage_bad[g][s]);
        const uint8_t* kw = st + q * kbytes + lane4;
        auto put = [&](int slot, const uint32_t (&v)[4]) { tc::tmem_st<4>(tbase + lane_base + 4 * slot, v); };
        // the first columns are free already, the others held the last chunk's V-hat^T
        k_lookup<2>(kw, S.slots, 0, kPgVCol / 4, 1, lane4, put);
        if (j > 0 && !tc::mbar_wait(&S.ofull[g], (j - 1) & 1, WL)) *abort_flag = 1;
        tc::fence_after_sync();
        k_lookup<2>(kw, S.slots, kPgVCol / 4, kPlanSlots, 1, lane4, put);
        tc::wait_st();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&S.kready[g]);
        // ------------------------------------------------------------ values (lane = dim)
        const uint8_t* sv = st + kChunkTiles * kbytes;
        if (!tc::mbar_wait(&S.fullv[g][s], ring.parity, WL)) *abort_flag = 1;
        ring.next(NS);
        const bool valid = (c_first + i) * kChunkTokens + t < len;
        const uint16_t* nrm = reinterpret_cast<const uint16_t*>(sv + q * vbytes) + lane;
        const float kn = valid ? __half2float(__ushort_as_half(nrm[0])) : 0.0f;
        const float vn = valid ? __half2float(__ushort_as_half(nrm[kTile])) * inv_sqrt_d : 0.0f;
        const float vs = vn * kPgScale, lv = share_log2(vn);
        {
          uint32_t v16[16];
          const uint32_t* vw = reinterpret_cast<const uint32_t*>(sv + 4 * kTile) + t;
          v_vals<VM>(vw, tab, v16);
          if (!tc::mbar_wait(&S.sfull[g], j & 1, WL)) *abort_flag = 1;   // K-hat is read
          tc::fence_after_sync();
          tc::tmem_st<16>(tbase + kPgVCol + lane_base, v16);
#pragma unroll
          for (int u = 1; u < kChunkTiles; ++u) {
            vw = reinterpret_cast<const uint32_t*>(sv + u * vbytes + 4 * kTile) + t;
            v_vals<VM>(vw, tab, v16);
            tc::tmem_st<16>(tbase + kPgVCol + lane_base + 16 * u, v16);
          }
        }
        // ------------------------------------------------------------ logits minus M (see kPgThr)
        float2 xv[kRows / 2], z[kRows / 2];
        {
          uint32_t sr[16];
          tc::tmem_ld<16>(tS + lane_base, sr);
          tc::wait_ld();
          const float gone = valid ? 0.0f : -INFINITY;
#pragma unroll
          for (int h = 0; h < kRows / 2; ++h) {
            const float2 kq = mul2(make_float2(kn, kn), *reinterpret_cast<const float2*>(qs + 2 * h));
            const float2 sum = add2(make_float2(__uint_as_float(sr[2 * h]), __uint_as_float(sr[2 * h + 1])),
                                    make_float2(__uint_as_float(sr[8 + 2 * h]), __uint_as_float(sr[9 + 2 * h])));
            xv[h] = fma2(sum, kq, make_float2(gone, gone));
            z[h] = add2(xv[h], nM[h]);
          }
        }
        bool over = false;
#pragma unroll
        for (int h = 0; h < kRows / 2; ++h)
          over |= (z[h].x > static_cast<float>(kPgThr) - lv) | (z[h].y > static_cast<float>(kPgThr) - lv);
        // a wait that gave up joins the vote, so that the four warps stop as one
        const bool stop = *abort_flag != 0;
        if (named_sync_or(1 + g, 128, over || stop)) {
          if (stop) S.wg_stop[g] = 1;
#pragma unroll
          for (int h = 0; h < kRows; ++h) {
            const int m = __reduce_max_sync(0xffffffffu, ordered(((h & 1) ? xv[h >> 1].y : xv[h >> 1].x) + lv));
            if (lane == 0) S.xch[g][q][h] = from_ordered(m);
          }
          named_sync(1 + g, 128);
          if (*reinterpret_cast<volatile int*>(&S.wg_stop[g])) {
            stopped = true;
            break;
          }
          float alpha[kRows];
#pragma unroll
          for (int h = 0; h < kRows; ++h) {
            const float cm = fmaxf(fmaxf(S.xch[g][0][h], S.xch[g][1][h]), fmaxf(S.xch[g][2][h], S.xch[g][3][h]));
            float& nm = (h & 1) ? nM[h >> 1].y : nM[h >> 1].x;
            float& l = (h & 1) ? L[h >> 1].y : L[h >> 1].x;
            const float mn = fmaxf(-nm, cm);
            alpha[h] = (nm == INFINITY) ? 0.0f : fast_exp2(-nm - mn);
            nm = -mn;
            l *= alpha[h];
          }
          if (i > 0) {                                      // O holds earlier chunks (lane = dim)
            uint32_t o[16];
            tc::tmem_ld<16>(tO + lane_base, o);
            tc::wait_ld();
#pragma unroll
            for (int c = 0; c < 16; ++c)
              if ((c & 7) < kRows) o[c] = __float_as_uint(__uint_as_float(o[c]) * alpha[c & (kRows - 1)]);
            tc::tmem_st<16>(tO + lane_base, o);
          }
#pragma unroll
          for (int h = 0; h < kRows / 2; ++h) z[h] = add2(xv[h], nM[h]);
        }
        // ------------------------------------------------------------ P' (lane = token)
        {
          const float2 vs2 = make_float2(vs, vs), minus1 = make_float2(-1.0f, -1.0f), low_up = make_float2(kPgLow, kPgLow);
          uint32_t hi[4] = {0u, 0u, 0u, 0u}, lo[4] = {0u, 0u, 0u, 0u};
#pragma unroll
          for (int h = 0; h < kRows / 2; ++h) {
            const float2 p = make_float2(fast_exp2(z[h].x), fast_exp2(z[h].y));
            L[h] = add2(L[h], p);
            const float2 y = mul2(p, vs2);
            const __half2 yh = __floats2half2_rn(y.x, y.y);
            const float2 r = mul2(fma2(__half22float2(yh), minus1, y), low_up);
            const __half2 yl = __floats2half2_rn(r.x, r.y);
            hi[h] = *reinterpret_cast<const uint32_t*>(&yh);
            lo[h] = *reinterpret_cast<const uint32_t*>(&yl);
          }
          *reinterpret_cast<uint4*>(pb) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          *reinterpret_cast<uint4*>(pb + 128) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
        tc::fence_proxy_async_smem();
        tc::wait_st();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&S.vready[g]);
      }
      if (stopped) break;
      // -------------------------------------------------------------- the segment's (m, l, O)
      if (!tc::mbar_wait(&S.ofull[g], (j - 1) & 1, WL)) seg_bad = 1, *abort_flag = 1;
      tc::fence_after_sync();
      {
        uint32_t o[16];
        tc::tmem_ld<16>(tO + lane_base, o);
        tc::wait_ld();
        // Row sums over the warp: at each step a lane keeps half of its rows and passes on the others;
        // lane l ends with row l / (32 / kRows).
        float l[kRows];
#pragma unroll
        for (int h = 0; h < kRows; ++h) l[h] = (h & 1) ? L[h >> 1].y : L[h >> 1].x;
#pragma unroll
        for (int k = 16, nr = kRows / 2; k > 0; k >>= 1, nr >>= 1) {
          if (nr > 0) {
            const bool up = (lane & k) != 0;
#pragma unroll
            for (int h = 0; h < nr; ++h) {
              const float give = up ? l[h] : l[h + nr], keep = up ? l[h + nr] : l[h];
              l[h] = keep + __shfl_xor_sync(0xffffffffu, give, k);
            }
          } else {
            l[0] += __shfl_xor_sync(0xffffffffu, l[0], k);
          }
        }
        constexpr int kPer = 32 / kRows;
        const int lr = lane / kPer;                         // the row whose sum this lane has
        const float gone = __int_as_float(0x7fc00000);
        if (joint) {
          // the stages are free now: every copy of this warpgroup has been read
          float* po = reinterpret_cast<float*>(my_stages) + t;
#pragma unroll
          for (int h = 0; h < kRows; ++h) {
            po[h * kD] = __uint_as_float(o[h]) + __uint_as_float(o[8 + h]) * (1.0f / kPgLow);
            if (lane == 0 && q == 0) S.join_m[g][h] = seg_bad ? gone : -((h & 1) ? nM[h >> 1].y : nM[h >> 1].x);
          }
          if (lane % kPer == 0) S.join_l[g][q][lr] = l[0];
        } else {
          const size_t e = e0 + b;
          float* po = a.part_o + e * 8 * kD + t;
#pragma unroll
          for (int h = 0; h < kRows; ++h) {
            if (h < a.group) po[h * kD] = (__uint_as_float(o[h]) + __uint_as_float(o[8 + h]) * (1.0f / kPgLow)) * (1.0f / kPgScale);
            if (lane == 0 && q == 0) a.part_m[e * 8 + h] = seg_bad ? gone : -((h & 1) ? nM[h >> 1].y : nM[h >> 1].x);
          }
          if (lane % kPer == 0) a.part_l[(e * 4 + q) * 8 + lr] = l[0];
        }
      }
      x += nseg;
      if (x < x1) {
        do ++b; while (cs[b + 1] == x);
      }
    }
    if (stopped) {                                          // the segments left have no result
      if (lane == 0 && q == 0) record_status(a.status, KVQ_ERR_TIMEOUT);
      if (q == 0 && lane < 8) {
        if (joint) S.join_m[g][lane] = __int_as_float(0x7fc00000);
        else
          for (; x < x1; ++b)
            if (cs[b + 1] > x) {
              a.part_m[(e0 + b) * 8 + lane] = __int_as_float(0x7fc00000);
              x = cs[b + 1];
            }
      }
    }
  }
  __syncthreads();
  allow_dependents();
  if (tid == 0) {
    // (the table's copy lands before the CTA leaves, used or not)
    const bool landed = tc::mbar_wait(&S.setup, 0, WL);
    if (!landed || S.wg_abort[0] | S.wg_abort[1] | S.wg_abort[2] | S.wg_abort[3]) record_status(a.status, KVQ_ERR_TIMEOUT);
  }
  if (joint && !bad) {
    // The warpgroups' shares of one sequence meet at a common maximum. A NaN maximum (a missing
    // share) stays one.
    const int nw = w_end - w_cta;
    const size_t e_first = static_cast<size_t>(hkv) * a.entries + w_cta + b_cta;
    const float* share = reinterpret_cast<const float*>(sm + kPgStageOff);
    const int pitch = NS * cbytes / 4;
    for (int i = tid; i < a.group * kD; i += kDecThreads) {
      const int h = i >> 7, d = i & (kD - 1);
      float mx = -INFINITY;
      bool missing = false;
      for (int k = 0; k < nw; ++k) {
        missing |= S.join_m[k][h] != S.join_m[k][h];
        mx = fmaxf(mx, S.join_m[k][h]);
      }
      float os = 0.0f, ls[4] = {0.f, 0.f, 0.f, 0.f};
      for (int k = 0; k < nw; ++k) {
        // (a share of NaN logits alone has maximum -inf and a NaN sum)
        const float wt = S.join_m[k][h] == -INFINITY ? (S.join_l[k][0][h] == 0.0f ? 0.0f : S.join_l[k][0][h]) : fast_exp2(S.join_m[k][h] - mx);
        os += wt * share[k * pitch + h * kD + d];
#pragma unroll
        for (int r = 0; r < 4; ++r) ls[r] += wt * S.join_l[k][r][h];
      }
      a.part_o[(e_first * 8 + h) * kD + d] = os * (1.0f / kPgScale);
      if (d < 4) a.part_l[(e_first * 4 + d) * 8 + h] = d == 0 ? ls[0] : d == 1 ? ls[1] : d == 2 ? ls[2] : ls[3];
      if (d == 0) a.part_m[e_first * 8 + h] = missing ? __int_as_float(0x7fc00000) : mx;
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == kDecIssuerWarp0) tc::tmem_dealloc(S.tmem_base, kTmemCols);
  if (a.after_prefix) grid_dependency_wait();
}

// ---------------------------------------------------------------- merge

struct MergeArgs {
  void* out;
  int out_dtype, n_q_heads, n_kv_heads, group, batch;
  const int2* plan;
  const int* refused;
  int entries, ctas;
  const float *own_m, *own_l, *own_o;      // as PagedAttn's part_*
  int prefix_len, pre_groups, pre_splits;
  const float *pre_m, *pre_l, *pre_o;      // [CTA][kPreRows], ..., CTA = (split * groups + group) * heads + head
};

constexpr int kPreRows = 128;              // query rows of a CTA on the prefix

constexpr int kMergeWarps = 16;            // at most

// One CTA joins the shares of one (sequence, query head): the prefix's splits, then the
// sequence's own. Warp w of n folds shares w, w + n, .. with its own running maximum (lane = 4 dims,
// the loads of eight shares in flight), then the warps meet in shared memory. The order of the
// sums is fixed. A NaN maximum marks a missing share: the row is left as it is.
// The host gives few rows 16 warps each and many rows 4.
__global__ void __launch_bounds__(kMergeWarps * 32) kvq_paged_merge(const MergeArgs a) {
  __shared__ float sm_m[kMergeWarps], sm_l[kMergeWarps];
  __shared__ float4 sm_o[kMergeWarps][32];
  const int hq = blockIdx.x % a.n_q_heads, b = blockIdx.x / a.n_q_heads;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n_warps = blockDim.x >> 5;
  const int hkv = hq / a.group, h = hq - hkv * a.group;
  grid_dependency_wait();
  const int2 plan = __ldcg(a.plan + b), all = __ldcg(a.plan + a.batch);
  const int refused = __ldcg(a.refused + hkv);
  if (plan.y < 0 || refused) return;
  const OwnShares own(Shares(all.x, a.ctas), plan.x, plan.y);
  const int n_pre = a.prefix_len > 0 ? a.pre_splits : 0;
  const int n = n_pre + own.n;
  const int row = b * a.group + h, rg = row / kPreRows, r = row - rg * kPreRows;
  float M = -INFINITY, L = 0.0f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  bool missing = false;
  constexpr int kBatch = 8;
  for (int i0 = warp; i0 < n; i0 += n_warps * kBatch) {
    float mv[kBatch], lv[kBatch];
    float4 ov[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int i = i0 + n_warps * u;
      mv[u] = -INFINITY;
      lv[u] = 0.0f;
      ov[u] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i < n_pre) {
        const size_t e = ((static_cast<size_t>(i) * a.pre_groups + rg) * a.n_kv_heads + hkv) * kPreRows + r;
        mv[u] = __ldcg(a.pre_m + e);
        lv[u] = __ldcg(a.pre_l + e);
        ov[u] = __ldcg(reinterpret_cast<const float4*>(a.pre_o + e * kD) + lane);
      } else if (i < n) {
        const size_t e = static_cast<size_t>(hkv) * a.entries + own.worker(i - n_pre) + b;
        mv[u] = __ldcg(a.own_m + e * 8 + h);
        const float* l = a.own_l + e * 32 + h;
        lv[u] = (__ldcg(l) + __ldcg(l + 8)) + (__ldcg(l + 16) + __ldcg(l + 24));
        ov[u] = __ldcg(reinterpret_cast<const float4*>(a.own_o + (e * 8 + h) * kD) + lane);
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
  for (int w = 0; w < n_warps; ++w) mx = fmaxf(mx, sm_m[w]);
  for (int w = 0; w < n_warps; ++w) {
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
