// What the norms' workspace is sized by.
#pragma once

#include <cstdint>

namespace moe {

// Rows of up to three partial column sums that the backward leaves.
int64_t norm_partial_rows(int64_t T, int64_t d);

}  // namespace moe
