// ops_internal.h -- what the operators around the attention (norm with rotary
// positions, 8-bit cache) share with each other and with the host API. Not part
// of the public ABI.
#pragma once
#include "gsdpa.h"
#include "gsdpa_internal.h"
#include "sm103_ptx.cuh"

namespace gsdpa {

// Beside ERR_WAIT_TIMEOUT in the error word: a sequence's length or token count,
// read on the device, lies outside its cache.
constexpr uint32_t ERR_CACHE_RANGE = 2u;

// The gate-logit pre-pass over few rows (decode): rows, columns and K splits,
// enough of them to spread the read of W_g over the SMs (gsdpa_api.cu).
void plan_gate_rows(const Problem& p, int num_sms, WorkspacePlan* w);

// Untiled copy of `bytes` contiguous bytes (addresses and size multiples of 16).
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     smem_u32(dst)),
                 "l"(src), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}

}  // namespace gsdpa
