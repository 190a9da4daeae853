// Which rows of a slot a part of a split contraction takes: plain C++ for the
// device and for host-side checks (the including file provides the __host__ /
// __device__ / __forceinline__ qualifiers).
#pragma once

namespace moe {

// Part `split` of `splits` of a slot's rows [lo, hi): whole slices, the same
// number for each part, as long as there are any. Parts behind the last row get
// none, at hi. Nothing passes 31 bits where hi is under 2^31 - 1024, slices have
// at most 128 rows and there are at most 16 parts: the parts before reach at most
// 15 slices behind the last row, so they are cut there before lo is added.
__host__ __device__ __forceinline__ void split_rows(int lo, int hi, int slice, int splits, int split,
                                                    int* row0, int* rows) {
  const int all = hi - lo, whole = (all + slice - 1) / slice;
  const int each = (whole + splits - 1) / splits * slice;
  const int before = split * each < all ? split * each : all;
  *row0 = lo + before;
  *rows = all - before < each ? all - before : each;
}

}  // namespace moe
