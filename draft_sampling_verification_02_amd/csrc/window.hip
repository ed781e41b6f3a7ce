// window.hip -- attention over a paged key-value cache through a sliding window,
// with a few first tokens (sinks) that stay visible.
//
// For row i of request b (position p = start_b + i) and head h:
//   s_t = scale q . k_t over t <= p with p - t < window or t < sinks,
//   out = sum_t exp(s_t - lse) v_t,  lse = log sum_t exp(s_t).
// Few rows a request go through the kernel of paged attention (paged.hpp), whose
// walk leaves out the tokens between the sinks and the first row's window: what
// no row sees is not read, and its pages may be gone.
#include "paged.hpp"

namespace dspark {

hipError_t launch_window_rows(const PagedArgs &a, const PagedPlan &plan, const PagedWork &w, hipStream_t s) {
    return launch_paged_any<true>(a, plan, w, s);
}

}  // namespace dspark
