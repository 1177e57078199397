// Sums of token counts in the plan of the batched adapters.
#pragma once

namespace qlk {

// a + b cut at M, for a and b in [0, M]: with M up to 2^30 the plain sum can be
// 2^31, so it is compared before it is formed.  Cutting the sum of non-negative
// numbers is associative, so any order of a prefix sum gives the same.
constexpr int cut_sum(int a, int b, int M) { return b < M - a ? a + b : M; }

}  // namespace qlk
