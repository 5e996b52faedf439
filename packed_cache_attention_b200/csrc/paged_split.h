// How a ragged batch's chunks are shared out over a head's warpgroups (paged decode), and which shares
// belong to a sequence (merge). Plain C++ for host and device: the decode and the merge, which must
// agree entry by entry, call the same functions, and a test runs them on the CPU.
#pragma once

#ifdef __CUDACC__
#define KVQ_HD __host__ __device__ __forceinline__
#else
#define KVQ_HD inline
#endif

namespace kvq {

KVQ_HD int min_of(int a, int b) { return a < b ? a : b; }
KVQ_HD int max_of(int a, int b) { return a < b ? b : a; }

// Largest i with start[i] <= x, start ascending over n + 1 entries, start[0] <= x < start[n].
KVQ_HD int find_span(const int* start, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (start[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

// The 4 * ctas warpgroups of a head share `chunks` chunks, `per` each (the last one what is left):
// as few as keep the longest range. (32-bit divisions: 64-bit ones took 1 us of a call.)
struct Shares {
  int per, workers, per_cta, chunks;        // chunks of a worker, workers, workers of a CTA (consecutive ranges)
  KVQ_HD Shares(int chunks, int ctas) : chunks(chunks) {
    per = max_of(1, (chunks + 4 * ctas - 1) / (4 * ctas));
    workers = (chunks + per - 1) / per;
    per_cta = max_of(1, (workers + ctas - 1) / ctas);
  }
  KVQ_HD int first(int w) const { return min_of(w * per, chunks); }   // first chunk of worker w
  KVQ_HD int of(int x) const { return x / per; }                      // worker of chunk x
};

// The workers w .. w_end - 1 of one CTA. Where several all lie in one sequence (`joint`) they leave one share
// of that sequence, b, as the first of them; otherwise worker w leaves one of each sequence it meets.
// Worker w's share of sequence b has the entry w + b: along the list either w or b grows, so no two meet.
struct CtaShare {
  int w, w_end, b;
  bool joint;
  KVQ_HD CtaShare(const Shares& sh, const int* cs, int batch, int cta) {
    w = cta * sh.per_cta;
    w_end = min_of(w + sh.per_cta, sh.workers);
    b = w + 1 < w_end ? find_span(cs, batch, sh.first(w)) : 0;
    joint = w + 1 < w_end && sh.first(w_end) <= cs[b + 1];
  }
};

// The shares of a sequence with chunks at .. at + n - 1 of the list: workers one by one up to the first CTA
// that lies in the sequence as a whole, such CTAs by their first worker, the rest one by one.
struct OwnShares {
  int n, lo, mid, w0, w_mid, per_cta;       // shares in all, before and of whole CTAs; first worker, first of them
  KVQ_HD OwnShares(const Shares& sh, int at, int chunks) : n(0), lo(0), mid(0), w0(0), w_mid(0), per_cta(sh.per_cta) {
    if (chunks <= 0) return;
    w0 = sh.of(at);
    const int w_end = sh.of(at + chunks - 1) + 1;
    int c_lo = w0 / per_cta, c_hi = (w_end + per_cta - 1) / per_cta;
    if (sh.first(c_lo * per_cta) < at) ++c_lo;
    if (sh.first(min_of(c_hi * per_cta, sh.workers)) > at + chunks) --c_hi;
    mid = max_of(0, c_hi - c_lo);
    if (mid > 0) {
      w_mid = c_lo * per_cta;
      lo = w_mid - w0;
      n = lo + mid + max_of(0, w_end - c_hi * per_cta);
    } else {
      lo = n = w_end - w0;
    }
  }
  // Worker whose entry holds share k.
  KVQ_HD int worker(int k) const {
    return k < lo ? w0 + k : k < lo + mid ? w_mid + (k - lo) * per_cta : w_mid + mid * per_cta + (k - lo - mid);
  }
};

}  // namespace kvq
