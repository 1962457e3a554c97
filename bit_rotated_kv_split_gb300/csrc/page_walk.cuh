// How the decodes over paged layers divide their work: the pages of all
// (request, set of heads) runs stand in one row, and each CTA takes an equal
// share of it, which it walks through run by run.
#pragma once

#include <cstdint>

#include "int4.h"
#include "oscar.h"

namespace oscar {

// The tokens of a request that its query sees, and their pages.
struct Span {
  int len, first;
  __device__ __forceinline__ int page0() const { return first / kPageTokens; }
  __device__ __forceinline__ int pages() const { return (len + kPageTokens - 1) / kPageTokens - page0(); }
};
// Params: a kernel's, with the cache as `c` and the score's form as `s`.
template <class Params>
__device__ __forceinline__ Span span_of(const Params& p, int b, bool report) {
  int len = p.c.seq_len[b];
  if (len < 0 || len > p.c.max_len) {
    if (report && p.c.dev_status) atomicOr(p.c.dev_status, OSCAR_DEV_LENGTH);
    len = min(max(len, 0), p.c.max_len);
  }
  return {len, p.s.window ? max(0, len - p.s.window) : 0};
}

// A run's pages, or the part of them in this CTA's share: pages lo .. hi - 1 of
// request b, head set h; `off` pages of the run lie before it, `pages` in all; it
// begins at place `at` of the row.
struct Segment {
  int b, h, lo, hi, off, pages, len, first, at;
};

// Walks through a share, run by run.  A run takes up kRunCost more places in the
// row than its pages; one of at most kWhole pages goes whole to the CTA whose
// share holds its first page.
template <int kRunCost, int kWhole>
struct PageWalk {
  int b, h, off;        // where the next segment begins: `off` pages into the run
  int at, end;          // its place, and the share's end
  Span span;            // of request b
  template <class Params>
  __device__ __forceinline__ bool next(const Params& p, int sets, Segment* s) {
    int pages = span.pages();
    // the share begins behind a run's pages, or within a run that is another's whole
    if (at < end && off > 0 && (off >= pages || pages <= kWhole)) step(p, sets), pages = span.pages();
    if (at >= end) return false;
    const int n = pages <= kWhole ? pages : min(pages - off, end - at), lo = span.page0() + off;
    *s = {b, h, lo, lo + n, off, pages, span.len, span.first, at};
    off += n;
    at += n;
    if (off == pages) step(p, sets);
    return true;
  }
  template <class Params>
  __device__ __forceinline__ void step(const Params& p, int sets) {   // to the next run's first page
    at += span.pages() + kRunCost - off;
    off = 0;
    if (++h < sets) return;
    h = 0;
    while (at < end && ++b < p.c.batch) {
      span = span_of(p, b, false);
      if (span.pages() > 0) return;
    }
    at = end;
  }
};

// This CTA's share of the row, at least min_share places: a prefix sum over the
// places of the requests' runs, a thread taking batch / kThreads of them.  The
// whole CTA; false if the share is empty, else *walk (shared memory) begins it
// and may be read after the next barrier.  *share: places of every CTA's.
template <int kThreads, int kRunCost, int kWhole, class Params>
__device__ __forceinline__ bool begin_share(const Params& p, int sets, int min_share, int* sm_scan,
                                            PageWalk<kRunCost, kWhole>* walk, int* share) {
  constexpr int kWarps = kThreads / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, batch = p.c.batch;
  const int per = (batch + kThreads - 1) / kThreads, b0 = min(batch, int(threadIdx.x) * per), b1 = min(batch, b0 + per);
  int mine = 0;
#pragma unroll 1
  for (int b = b0; b < b1; ++b) {
    const int n = span_of(p, b, blockIdx.x == 0).pages();
    mine += n ? (n + kRunCost) * sets : 0;
  }
  int before = mine;
#pragma unroll
  for (int x = 1; x < 32; x <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, before, x);
    if (lane >= x) before += v;
  }
  if (lane == 31) sm_scan[warp] = before;
  __syncthreads();
  int total = 0;
  before -= mine;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += sm_scan[w];
    total += sm_scan[w];
  }
  *share = max(min_share, int((unsigned(total) + gridDim.x - 1) / gridDim.x));
  const int64_t start = int64_t(*share) * blockIdx.x;
  const bool any = start < total;
  if (any && start >= before && start - before < mine) {
    int b = b0, at = int(start) - before;
    Span s = span_of(p, b, false);
#pragma unroll 1
    while (s.pages() == 0 || at >= (s.pages() + kRunCost) * sets) {
      at -= s.pages() ? (s.pages() + kRunCost) * sets : 0;
      s = span_of(p, ++b, false);
    }
    const int run = s.pages() + kRunCost;
    *walk = {b, at / run, at % run, int(start), int(min(int64_t(total), start + *share)), s};
  }
  return any;
}

}  // namespace oscar
