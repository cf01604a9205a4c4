// s4.h -- host-side declarations of the products with grouped 4-bit integer weights
// (s4_tokens.cu, s4_experts.cu).
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace ptc {

struct S4Weights;
// Codes of `experts` matrices of `rows` rows of row_bytes, `pitch` and `expert` bytes
// apart: boxes of 128 bytes x box_rows rows in the 128-byte swizzle, zeros outside.
int encode_tmap_codes(CUtensorMap *map, const void *base, uint64_t row_bytes, uint64_t rows, uint64_t experts, uint64_t pitch,
                      uint64_t expert, uint32_t box_rows);
// The argument checks of a weight matrix.
int check_s4(const S4Weights &w);
// The products' error words, read and cleared.
cudaError_t read_and_clear_s4_error_word(uint32_t *out);
cudaError_t read_and_clear_moe_error_word(uint32_t *out);
// The keys "s4_tokens_rows", "s4_tokens_split" and "s4_tokens_tiles" of
// ptc_set_tuning; false for another key or a value out of range.
bool set_s4_tuning(const char *key, int64_t value);

}  // namespace ptc
