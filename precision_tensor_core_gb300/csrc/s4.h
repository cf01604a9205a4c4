// s4.h -- host-side declarations of the products with grouped 4-bit integer weights
// (s4_tokens.cu, s4_experts.cu).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace ptc {

struct S4Weights;
// The argument checks of a weight matrix.
int check_s4(const S4Weights &w);
// The experts' error word, read and cleared.
cudaError_t read_and_clear_moe_error_word(uint32_t *out);
// The keys "s4_tokens_rows", "s4_tokens_split" and "s4_tokens_tiles" of
// ptc_set_tuning; false for another key or a value out of range.
bool set_s4_tuning(const char *key, int64_t value);

}  // namespace ptc
