// The paged attention for callers that bring a table of their own for every kv head.
#pragma once
#include <functional>

#include "../../include/mk.h"

namespace mk {

// mk_paged_attention's checks and launches; between them `before` (a launch that fills what the
// attention reads).  head_stride: entries from one kv head's table row to the next's, 0 where the
// heads share one.
mk_status attend_pages(const mk_attend_args& args, const mk_page_view& cache, long long head_stride, int32_t* status,
                       void* stream, const std::function<mk_status()>& before);

}  // namespace mk
