// window_rows.hip -- windowed attention of few rows a request (window.hip has the
// mathematics): the walk of paged attention without the tokens between the sinks
// and the first row's window.
#include "paged.hpp"

namespace dspark {

hipError_t launch_window_rows(const PagedArgs &a, const PagedPlan &plan, const PagedWork &w, hipStream_t s) {
    return launch_paged_any<true>(a, plan, w, s);
}

}  // namespace dspark
