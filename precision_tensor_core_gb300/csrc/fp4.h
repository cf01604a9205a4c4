// fp4.h -- host-side declarations of the 4-bit operators (fp4_quant.cu,
// fp4_gemm.cu, fp4_tokens.cu) and of what api.cu lends them.  The integer and FP16
// kernels do not include it, so that their recorded profiles stay those of their
// sources when it changes.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace ptc {

// Tiled block scales (tiles of 512 bytes, ktiles per 128 rows, rtiles x 128
// rows): boxes of box_k x box_r tiles, of the first dimension box_words 32-bit
// words, zero fill outside.
int encode_tmap_scales(CUtensorMap *map, const void *base, uint64_t ktiles, uint64_t rtiles, uint32_t box_k,
                       uint32_t box_r, uint32_t box_words = 128);

// Host helpers of the entry points (api.cu): a status with its text, a failed
// CUDA call, the current device's SM count (PTC_ERR_DEVICE when it is not
// usable), the process-wide knobs.
int fail_status(int code, const char *text);
int fail_launch(cudaError_t e, const char *what);
int usable_device(int *sms);
bool pdl_enabled();
uint64_t wait_limit_ns();
int take_stall_tile();
// Bytes spanned by `rows` rows of `cols` elements of `esize` bytes, `ld`
// elements apart (saturating), and whether two byte ranges intersect.
uint64_t span_of(int64_t rows, int64_t cols, int64_t ld, int esize);
bool ranges_overlap(const void *a, uint64_t alen, const void *b, uint64_t blen);

// 4-bit matrices (fp4_quant.cu): bytes of the tiled scales and of the codes
// of `rows` rows of `cols` values, and the argument checks of one.
uint64_t fp4_scale_bytes(int64_t rows, int64_t cols, bool nv);
uint64_t fp4_code_span(int64_t rows, int64_t cols, int64_t pitch);
int check_fp4(const void *codes, int64_t pitch, const void *scales, const void *g, int64_t rows, int64_t cols, bool nv);

// The 4-bit products' error words (fp4_gemm.cu, fp4_tokens.cu), read and cleared.
cudaError_t read_and_clear_fp4_error_word(uint32_t *out);
cudaError_t read_and_clear_tokens_error_word(uint32_t *out);
// The keys "fp4_tile", "fp4_ksplit" and "fp4_group_m" of ptc_set_tuning;
// false for another key or a value out of range.
bool set_fp4_tuning(const char *key, int64_t value);

}  // namespace ptc
