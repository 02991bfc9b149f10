// What the attention kernels share: where a sequence lies on a packed token
// axis, and which keys a query sees.
#pragma once

#include "internal.h"

namespace muon {

struct Span {
  int start, len;
};

// Sequence i of a packed axis of `total` tokens.  Offsets come from device
// memory and are not trusted: what lies outside the axis, or runs backwards,
// is cut to a valid (possibly empty) range.
__device__ __forceinline__ Span span_of(const int* cu, int i, int total) {
  const int a = min(max(cu[i], 0), total);
  const int b = min(max(cu[i + 1], a), total);
  return Span{a, b - a};
}

struct Keys {
  int first, end;
};

// The keys [first, end) that query i of a sequence with nq queries and nk
// keys sees; empty when end <= first.
__device__ __forceinline__ Keys keys_of(const AttnParams& p, int i, int nq, int nk) {
  if (!p.causal) return Keys{0, nk};
  const int place = i + nk - nq;
  return Keys{p.window > 0 ? max(place - p.window + 1, 0) : 0, min(place + 1, nk)};
}

}  // namespace muon
