// What the library's translation units share on the host: the error state,
// the mask and score programs in the form the kernels take, and per-device
// facts. bsmt.cu defines these functions.
#pragma once
#include <cstdint>

#include <cuda.h>

#include "bsmt.h"
#include "mask_dnf.cuh"

namespace bsmt_host {

// Sets the thread's error message (printf form) and returns `code`.
bsmt_status fail(bsmt_status code, const char* fmt, ...);
// Clears it and returns BSMT_OK.
bsmt_status ok();

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

constexpr int64_t kMaxLen = (int64_t(1) << 31) - 256;

// Score mods -> mode (kScore* of the attention kernels), the soft-cap and the
// ALiBi slopes (explicit, or the default ones of heads h0 .. h0 + Hq - 1 of a
// model of `heads` heads).
struct ScoreArgs {
    int mode = 0;
    float cap = 1.f;
    const float* slopes = nullptr;
    int32_t alibi_h0 = 0, alibi_heads = 1;
};

bsmt_status build_dnf(const bsmt_mask_spec* spec, int64_t B, bsmt::MaskDnf* out);
bsmt_status score_args(const bsmt_score_spec* score, int64_t Hq, ScoreArgs* out);
// The current device (checked to be sm_100) and its SM count.
bsmt_status sm_count(int* dev, int* n);
// Device address of the current device's status word.
bsmt_status status_word(int dev, int** addr);

// Tensor map of `rows` rows of `row_bytes` (64 or 128) bytes, copied `box` rows at a
// time with the swizzle of their length. `base` 16-byte aligned.
bsmt_status encode_rows(CUtensorMap* map, void* base, int64_t rows, int row_bytes, int box);

}  // namespace bsmt_host
