// query_steps.cuh — the query steps of a key tile, in the order the key-major
// kernels (dK/dV, key weights) visit them.
#pragma once

#include "internal.h"

namespace cpattn {

// Walks the query steps of a key tile: for every query head of the GQA
// group, every query run of the plan, cut into BNQ-row tiles.
template <int BNQ>
struct StepCursor {
  const RangeDesc* r;
  int count, G, kvh, hkv, inter;
  int g, ri, off;
  RangeDesc cur;
  __device__ void init(const RangeDesc* ranges, int begin, int cnt, int G_, int kvh_, int hkv_, int inter_) {
    r = ranges + begin;
    count = cnt;
    G = G_;
    kvh = kvh_;
    hkv = hkv_;
    inter = inter_;
    g = 0;
    ri = 0;
    off = 0;
    if (count > 0) cur = r[0];
  }
  __device__ int head() const { return inter ? g * hkv + kvh : kvh * G + g; }
  // a gathered query tile (packed()) has its pieces from entry row0
  __device__ bool packed() const { return (cur.flags & kRangePacked) != 0; }
  __device__ int row() const { return cur.row0 + off; }
  __device__ int n() const { return min(BNQ, cur.nrows - off); }
  __device__ int pos() const { return cur.pos0 + off; }
  __device__ void next() {
    off += BNQ;
    if (off >= cur.nrows) {
      off = 0;
      if (++ri >= count) {
        ri = 0;
        ++g;
      }
      if (count > 0) cur = r[ri];
    }
  }
};

}  // namespace cpattn
