// Row numbers of the expert sort. A sorted buffer may have any number of rows below 2^31, so a
// count or row may be that close to the end of 32 bits: nothing here goes past its own result.
// constexpr, so that the same code runs in kernels and on the host.
#pragma once

#include <stdint.h>

namespace fp8lin {

// n >= 0 rounded up to a multiple of `multiple` >= 1, where that is below 2^31.
constexpr int32_t padded_count(int32_t n, int32_t multiple) {
  const int32_t over = n % multiple;
  return over == 0 ? n : n - over + multiple;
}

// f(row) for the rows [from, to) that fall to one of 16 lanes, from the last one down: a step
// past the first row is above -16, where a step past the last could pass 2^31.
template <typename F>
constexpr void each_padding_row(int32_t from, int32_t to, int32_t lane, F&& f) {
  for (int32_t r = to - 1 - lane; r >= from; r -= 16) f(r);
}

}  // namespace fp8lin
