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
// Rows of `width` bytes, `pitch` bytes apart; what each argument of a call reads or
// writes.  Two of them with one pitch that lie side by side in one buffer share no
// byte although their spans intersect.
struct ByteRows {
    const void *p;  // NULL: none
    int64_t rows;
    uint64_t width, pitch;
};
// Whether they share a byte (for different pitches: whether their spans intersect).
bool rows_overlap(const ByteRows &a, const ByteRows &b);

// `rows` rows of `cols` elements of `esize` bytes, `ld` elements apart.
inline ByteRows elem_rows(const void *p, int64_t rows, int64_t cols, int64_t ld, int esize) {
    return {p, rows, uint64_t(cols) * uint64_t(esize), uint64_t(ld) * uint64_t(esize)};
}
inline ByteRows flat_bytes(const void *p, uint64_t n) { return {p, 1, n, n}; }

// 4-bit matrices of `rows` rows of `cols` values (fp4_quant.cu): the bytes of the
// codes and of the tiled scales, and the argument checks of one.
ByteRows fp4_code_rows(const void *codes, int64_t rows, int64_t cols, int64_t pitch);
ByteRows fp4_scale_rows(const void *scales, int64_t rows, int64_t cols, bool nv);
int check_fp4(const void *codes, int64_t pitch, const void *scales, const void *g, int64_t cols, bool nv);

// The 4-bit products' error words (fp4_gemm.cu, fp4_tokens.cu), read and cleared.
cudaError_t read_and_clear_fp4_error_word(uint32_t *out);
cudaError_t read_and_clear_tokens_error_word(uint32_t *out);
// The keys "fp4_tile", "fp4_ksplit" and "fp4_group_m", "fp4_tokens_rows" and
// "fp4_tokens_split" of ptc_set_tuning; false for another key or a value out of range.
bool set_fp4_tuning(const char *key, int64_t value);
bool set_tokens_tuning(const char *key, int64_t value);
// What ptc_last_fp4_launch reports (api.cu).
void note_fp4_launch(int64_t grid, int cluster, int ksplit, int tile);

}  // namespace ptc
