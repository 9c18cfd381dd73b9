// The keys that a row's queries see with a sliding window and first tokens that
// stay visible, as pages: shared by the kernels of the attention with a window.
#pragma once

#include "common.cuh"

namespace pa {

// Queries at positions L - n .. L - 1 see together [0, min(S, L)) and [lo, L), lo =
// the first one's position - W + 1: leading pages 0 .. lead - 1, then first .. end - 1.
// The pages of a row are counted through (v = 0 .. count - 1), the gap left out.
struct Seen {
  int lead, first, end;
  __host__ __device__ __forceinline__ int count() const { return lead + end - first; }
  __host__ __device__ __forceinline__ int page(int v) const { return v < lead ? v : v + first - lead; }
};
__host__ __device__ __forceinline__ Seen seen_pages(int L, int n, int window, int sinks) {
  Seen s;
  s.end = (L + kPage - 1) / kPage;
  const int lead = sinks / kPage + (sinks % kPage != 0);
  s.lead = lead < s.end ? lead : s.end;
  const int low = L - n - window + 1;  // (window >= 1, L - n >= 0: no overflow)
  s.first = low > 0 ? low / kPage : 0;
  s.first = s.first > s.lead ? s.first : s.lead;
  return s;
}

}  // namespace pa
