// cache4_internal.h -- what the plan, the append, the reading back and the
// attention of the paged 4-bit K/V cache share. Not part of the public ABI.
#pragma once
#include "ops_internal.h"

namespace gsdpa {

constexpr int kPage = 64;        // tokens of a page
constexpr int kGroup = 16;       // columns of a token that share a scale
constexpr int kMaxExp = 64;      // of k_exp and v_exp

// Offsets in the 72 d bytes that a page has of one head: key codes, key scales,
// value codes, value scales.
constexpr int page_bytes(int d) { return 72 * d; }
constexpr int key_scales_at(int d) { return 32 * d; }
constexpr int value_codes_at(int d) { return 36 * d; }
constexpr int value_scales_at(int d) { return 68 * d; }

// Host-side checks of the cache's description (cache4_rows_sm103.cu).
int validate_cache4(const gsdpa_cache4* c);
int validate_cache4_pointers(const gsdpa_cache4* c);

}  // namespace gsdpa
