// landing.cuh -- the end of a CTA one of whose bounded waits ran out: what is still
// under way (copies into its shared memory, MMAs) lands before its memory goes.
#pragma once
#include "sm103_ptx.cuh"

namespace gsdpa {

// The limit of a wait for what is already under way (copies, MMAs) before a CTA that
// gave up ends: a second at least, however short the caller's limit is.
static __device__ __forceinline__ WaitCtl landing_limit(WaitCtl ctl) {
    if (ctl.limit_ns < 1000000000ull) ctl.limit_ns = 1000000000ull;
    return ctl;
}

// The end of a CTA one of whose waits may have run out: copies into its shared memory
// and MMAs that another of its threads, or the other CTA of a pair, had issued before
// that may still be under way, and no one waits for them any more. 200 us are far more
// than a ring of copies takes; a CTA that did not give up reads one word.
static __device__ __forceinline__ void let_land_after_abort(const volatile int* abort_flag) {
    if (*abort_flag == 0) return;
    const unsigned long long t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 200000ull) {
    }
}

}  // namespace gsdpa
