// cache8_internal.h -- what the append and the attention of the 8-bit K/V
// cache share. Not part of the public ABI.
#pragma once
#include "ops_internal.h"

namespace gsdpa {

constexpr int kCacheBlock = 64;   // tokens that share a scale

// A sequence's tokens before (len) and of this step (n), as the kernels take
// them: numbers out of range make the sequence empty (ok = false), so that no
// read or write can leave the cache.
struct SeqRange {
    int len, n;
    bool ok;
};
__device__ __forceinline__ SeqRange seq_range(const int* lens, const int* n_new, int b, int L, int capacity) {
    SeqRange r;
    r.len = lens[b];
    r.n = n_new ? n_new[b] : L;
    r.ok = r.len >= 0 && r.n >= 0 && r.n <= L && r.len <= capacity && r.n <= capacity - r.len;
    if (!r.ok) r.len = r.n = 0;
    return r;
}

// Host-side checks of the cache's description (cache8_append_sm103.cu).
int validate_cache8(const gsdpa_cache8* c);
int validate_cache8_pointers(const gsdpa_cache8* c);

}  // namespace gsdpa
