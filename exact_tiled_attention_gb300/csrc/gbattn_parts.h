// gbattn_parts.h -- what a second kernel may believe of the words that the first one
// left in the caller's workspace.  Plain C++, for kernels and for a test without a GPU.
#pragma once

namespace gbattn {

// Whether a unit was split into n >= 2 parts whose states the CTAs [first, first + n)
// of a grid of `ctas` left.  Also false for what a workspace held before the call: a CTA
// that gave up a wait, which the status tells, leaves a unit's entry as it was.
constexpr bool split_parts(int first, int n, int ctas) { return n >= 2 && first >= 0 && first < ctas && n <= ctas - first; }

}  // namespace gbattn
