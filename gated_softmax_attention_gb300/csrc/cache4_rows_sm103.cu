// cache4_rows_sm103.cu -- the paged 4-bit K/V cache, token by token: the append (bf16
// keys and values to codes and scales at their slots) and the reading back.
//
// Per 16 columns x of a token: scale s = e4m3(max |x| 2^-exp / top), codes
// round(x 2^-exp / s). x has 8 significant bits and s 4: their quotient is either on a
// border between two codes, and then a float32 number, or 2^-13 of itself away from it.
// So one step of correction of the product with the rounded reciprocal gives the code of
// the exact quotient, ties among it (without the step one code in 500 was not: 1/13 is off by
// up to half a place, and so are ties).
//
// Bound by HBM for prompts (4 d bytes in, 1.125 d out per token and head), by latency
// for a decoding step. A block has 32 rows of one head: it reads them whole,
// leaves codes and scales in shared memory token by token, and writes what
// the pages want: a key is 8 d bits of contiguous page, but a value's codes go one
// byte to each of d / 2 words, whose other bytes are other tokens'. Where the block
// has all four tokens of a word it writes the word, else bytes, so that tokens next
// to each other can be written by different blocks and calls.
#include "cache4_internal.h"

#include <cuda_fp16.h>
#include <cuda_fp8.h>

namespace gsdpa {
namespace {

constexpr int kRows = 32;        // rows of a block: one warp of them
constexpr int kThreads = 256;

struct RowsArgs {
    const __nv_bfloat16 *K, *V;  // the append's
    __nv_bfloat16 *Ko, *Vo;      // the reading's
    long long ld_k, ld_v;
    const long long* slots;
    uint8_t* pool;
    int n_rows, Hkv, n_pages;
    float k_down, v_down;        // 2^-exp (append), 2^exp (reading)
    uint32_t* err;
};

// |x| of two bf16 numbers, larger of each half; NaN wins.
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Two numbers -> their e2m1 codes, the first in the low 4 bits.
__device__ __forceinline__ uint32_t to_e2m1x2(float lo, float hi) {
    uint32_t r;
    asm("{\n\t.reg .b8 t;\n\tcvt.rn.satfinite.e2m1x2.f32 t, %2, %1;\n\tcvt.u32.u8 %0, t;\n\t}" : "=r"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ uint32_t to_int4(float y) {
    return (uint32_t)(min(max(__float2int_rn(y), -7), 7) + 8);
}

// Eight columns, half of a group (the other half is the neighbouring lane's) -> eight
// codes, 4 bits each, and the group's scale.
template <bool E2M1>
__device__ __forceinline__ uint32_t quantise(const uint4& x, float down, uint32_t& scale) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t top = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) top = max_bf16x2(top, w[k] & 0x7fff7fffu);
    top = max_bf16x2(top, __shfl_xor_sync(0xffffffffu, top, 1));
    const float amax = fmaxf(__uint_as_float(top << 16), __uint_as_float(top & 0xffff0000u));
    const bool number = (top & 0x7fff) < 0x7f80 && (top >> 16) < 0x7f80;   // (no NaN, no infinity)
    const __nv_fp8_storage_t byte = __nv_cvt_float_to_fp8(amax * down * (1.f / (E2M1 ? 6.f : 7.f)), __NV_SATFINITE, __NV_E4M3);
    scale = number ? byte : 0x7fu;
    const float s = __half2float(__half(__nv_cvt_fp8_to_halfraw(byte, __NV_E4M3)));
    if (!number || byte == 0) return E2M1 ? 0u : 0x88888888u;
    const float inv = __frcp_rn(s);
    // (an infinite quotient, of a scale cut off at 448, has no correction)
    const auto over = [&](uint32_t bits) {
        const float v = __uint_as_float(bits) * down, y = v * inv;
        return fabsf(y) <= 16.f ? fmaf(fmaf(-y, s, v), inv, y) : y;
    };
    uint32_t codes = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float lo = over(w[k] << 16), hi = over(w[k] & 0xffff0000u);
        codes |= (E2M1 ? to_e2m1x2(lo, hi) : to_int4(lo) | to_int4(hi) << 4) << (8 * k);
    }
    return codes;
}

// Where code c (0 .. 7) of columns 8 half .. of group j goes: byte of a token's key
// row, and which 4 bits.
template <int D, bool E2M1>
__device__ __forceinline__ void key_place(int j, int half, int c, int& byte, int& high) {
    const int r = 8 * half + c, t = r / 4, pair = r / 2 % 2, side = r % 2;
    if (E2M1) {
        byte = t * (D / 8) + 2 * j + pair;
        high = side;
    } else {
        byte = t * (D / 8) + 4 * (j / 2) + 2 * side + j % 2;
        high = pair;
    }
}

// 4-bit places 0 .. 7 of a word in another order.
__device__ __forceinline__ uint32_t nibble(uint32_t codes, int k) { return codes >> (4 * k) & 15u; }

// Rows of one block: the slot of each, and the runs of rows that lie in one tile of
// 16 tokens (a run begins where the tile changes).
struct Runs {
    long long slot[kRows];       // -1: none
    int lead[kRows];             // row at which this row's run begins
    signed char at[kRows][16];   // by leading row: the run's row at each place of the tile, or -1
};

__device__ __forceinline__ void find_runs(const RowsArgs& a, long long first, Runs& s) {
    const int tid = threadIdx.x;
    for (int k = tid; k < kRows * 4; k += kThreads) reinterpret_cast<uint32_t*>(s.at)[k] = 0xffffffffu;
    __syncthreads();
    if (tid < 32) {
        const long long row = first + tid;
        long long slot = row < a.n_rows ? a.slots[row] : -1;
        if (slot >= (long long)a.n_pages * kPage) {
            slot = -1;
            atomicOr(a.err, ERR_CACHE_RANGE);
        }
        if (slot < 0) slot = -1;
        const long long before = __shfl_up_sync(0xffffffffu, slot, 1);
        const uint32_t leads = __ballot_sync(0xffffffffu, tid == 0 || (slot >> 4) != (before >> 4));
        const int lead = 31 - __clz(leads & (0xffffffffu >> (31 - tid)));
        s.slot[tid] = slot;
        s.lead[tid] = lead;
        if (slot >= 0) s.at[lead][slot & 15] = (signed char)tid;
    }
    __syncthreads();
}

template <int D, bool E2M1>
__global__ void __launch_bounds__(kThreads) cache4_append_kernel(const __grid_constant__ RowsArgs a) {
    __shared__ Runs runs;
    __shared__ __align__(16) uint8_t s_key[kRows][D / 2], s_value[kRows][D / 2];   // value: [quad][g][j % 4]
    __shared__ __align__(16) uint8_t s_kscale[kRows][D / 16], s_vscale[kRows][D / 16];
    pdl_trigger();
    pdl_wait();
    const int tid = threadIdx.x, h = blockIdx.y;
    const long long first = (long long)blockIdx.x * kRows;
    find_runs(a, first, runs);

    // ---- codes and scales, a lane to eight columns
    for (int k = tid; k < 2 * kRows * (D / 8); k += kThreads) {
        const bool value = k >= kRows * (D / 8);
        const int i = k % (kRows * (D / 8)), r = i / (D / 8), j = i % (D / 8) / 2, half = i % 2;
        uint4 x = make_uint4(0, 0, 0, 0);
        if (runs.slot[r] >= 0)
            x = *reinterpret_cast<const uint4*>((value ? a.V + (first + r) * a.ld_v : a.K + (first + r) * a.ld_k) +
                                                (long long)h * D + 16 * j + 8 * half);
        uint32_t scale;
        const uint32_t codes = quantise<E2M1>(x, value ? a.v_down : a.k_down, scale);
        if (half == 0) (value ? s_vscale : s_kscale)[r][j] = (uint8_t)scale;
        if (!value) {
            // e2m1: pairs of columns are pairs of bytes; int4: the sides of a pair are 2 bytes apart
#pragma unroll
            for (int c = 0; c < 8; c += 4) {
                const int t = 2 * half + c / 4;
                if (E2M1) {
                    *reinterpret_cast<uint16_t*>(&s_key[r][t * (D / 8) + 2 * j]) = (uint16_t)(codes >> (4 * c));
                } else {
                    uint8_t* to = &s_key[r][t * (D / 8) + 4 * (j / 2) + j % 2];
                    to[0] = (uint8_t)(nibble(codes, c) | nibble(codes, c + 2) << 4);
                    to[2] = (uint8_t)(nibble(codes, c + 1) | nibble(codes, c + 3) << 4);
                }
            }
        } else {
            // a byte holds columns g and 8 + g: the two halves' codes
            const uint32_t other = __shfl_xor_sync(0xffffffffu, codes, 1);
            const uint32_t lo = half ? other : codes, hi = half ? codes : other;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int g = 4 * half + c;
                s_value[r][j / 4 * 32 + g * 4 + j % 4] = (uint8_t)(nibble(lo, g) | nibble(hi, g) << 4);
            }
        }
    }
    __syncthreads();

    // ---- keys: rows of D / 2 bytes, and their scales
    const auto page_of = [&](long long slot) { return a.pool + ((slot / kPage) * a.Hkv + h) * page_bytes(D); };
    for (int k = tid; k < kRows * (D / 32); k += kThreads) {
        const int r = k / (D / 32), c = k % (D / 32);
        const long long slot = runs.slot[r];
        if (slot >= 0)
            *reinterpret_cast<uint4*>(page_of(slot) + (slot % kPage) * (D / 2) + 16 * c) =
                *reinterpret_cast<const uint4*>(&s_key[r][16 * c]);
    }
    for (int k = tid; k < kRows * (D / 64); k += kThreads) {
        const int r = k / (D / 64), c = k % (D / 64);
        const long long slot = runs.slot[r];
        if (slot >= 0)
            *reinterpret_cast<uint32_t*>(page_of(slot) + key_scales_at(D) + (slot % kPage) * (D / 16) + 4 * c) =
                *reinterpret_cast<const uint32_t*>(&s_kscale[r][4 * c]);
    }

    // ---- values: words of four tokens, run by run
    constexpr int WORDS = 2 * D, SCALES = D / 4;   // of a tile
    for (int k = tid; k < kRows * (WORDS + SCALES); k += kThreads) {
        const int r = k / (WORDS + SCALES), w = k % (WORDS + SCALES);
        if (runs.lead[r] != r || runs.slot[r] < 0) continue;
        const bool scales = w >= WORDS;
        int t, from;   // lane of the tile's operand, byte of a token
        if (scales) {
            t = (w - WORDS) / (D / 16);
            from = (w - WORDS) % (D / 16);
        } else {
            t = w / 4 % 4;
            from = w / 128 * 32 + w % 128 / 16 * 4 + w % 4;
        }
        const int places[4] = {2 * t, 2 * t + 1, 2 * t + 8, 2 * t + 9};
        uint32_t word = 0;
        int have = 0;
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const int row = runs.at[r][places[b]];
            const int byte = scales || E2M1 ? b : (b == 1 ? 2 : (b == 2 ? 1 : b));
            if (row >= 0) {
                have |= 1 << byte;
                word |= (uint32_t)(scales ? s_vscale[row][from] : s_value[row][from]) << (8 * byte);
            }
        }
        const long long slot = runs.slot[r];
        const int tile = (int)(slot % kPage) / 16;
        uint8_t* to = page_of(slot) + (scales ? value_scales_at(D) + 4 * (tile * SCALES + w - WORDS)
                                              : value_codes_at(D) + 4 * (tile * WORDS + w));
        if (have == 15) {
            *reinterpret_cast<uint32_t*>(to) = word;
        } else {
#pragma unroll
            for (int b = 0; b < 4; ++b)
                if (have & (1 << b)) to[b] = (uint8_t)(word >> (8 * b));
        }
    }
}

// A code of 4 bits as the number it stands for.
template <bool E2M1>
__device__ __forceinline__ float code_value(uint32_t c) {
    if (!E2M1) return (float)((int)c - 8);
    const uint32_t m = c & 7u;
    // exponent 1 + m / 2 of a number whose exponents start at 2^-1, or the subnormal 0 and 0.5
    const float v = m < 2 ? 0.5f * m : __uint_as_float((126u + m / 2) << 23 | (m & 1u) << 22);
    return c & 8u ? -v : v;
}

__device__ __forceinline__ float scale_value(uint32_t byte) {
    return __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)byte, __NV_E4M3)));
}

template <int D, bool E2M1>
__global__ void __launch_bounds__(kThreads) cache4_read_kernel(const __grid_constant__ RowsArgs a) {
    pdl_trigger();
    pdl_wait();
    const int h = blockIdx.y;
    const long long first = (long long)blockIdx.x * kRows;
    for (int k = threadIdx.x; k < 2 * kRows * (D / 8); k += kThreads) {
        const bool value = k >= kRows * (D / 8);
        const int i = k % (kRows * (D / 8)), r = i / (D / 8), j = i % (D / 8) / 2, half = i % 2;
        if (first + r >= a.n_rows) continue;
        const long long slot = a.slots[first + r];
        uint32_t out[4] = {0, 0, 0, 0};
        if (slot >= (long long)a.n_pages * kPage) {
            atomicOr(a.err, ERR_CACHE_RANGE);
        } else if (slot >= 0) {
            const uint8_t* page = a.pool + ((slot / kPage) * a.Hkv + h) * page_bytes(D);
            const int n = (int)(slot % kPage), t = n % 8 / 2, y = n % 16 / 8, z = n % 2;
            float s, x[8];
            if (!value) {
                s = scale_value(page[key_scales_at(D) + n * (D / 16) + j]) * a.k_down;
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    int byte, high;
                    key_place<D, E2M1>(j, half, c, byte, high);
                    x[c] = code_value<E2M1>(page[n * (D / 2) + byte] >> (4 * high) & 15u) * s;
                }
            } else {
                s = scale_value(page[value_scales_at(D) + 4 * ((n / 16 * 4 + t) * (D / 16) + j) + 2 * y + z]) * a.v_down;
                const int byte = E2M1 ? 2 * y + z : 2 * z + y;
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    const int word = ((n / 16 * (D / 64) + j / 4) * 32 + 4 * c + t) * 4 + j % 4;
                    x[c] = code_value<E2M1>(page[value_codes_at(D) + 4 * word + byte] >> (4 * half) & 15u) * s;
                }
            }
#pragma unroll
            for (int c = 0; c < 4; ++c) out[c] = pack_bf16x2(x[2 * c], x[2 * c + 1]);
        }
        __nv_bfloat16* to = value ? a.Vo + (first + r) * a.ld_v : a.Ko + (first + r) * a.ld_k;
        *reinterpret_cast<uint4*>(to + (long long)h * D + 16 * j + 8 * half) = make_uint4(out[0], out[1], out[2], out[3]);
    }
}

bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

// What the append and the reading refuse; GSDPA_OK with *any false: nothing to do.
int check_rows(const gsdpa_cache4* c, const void* K, const void* V, long long ld_k, long long ld_v,
               const long long* slots, int n_rows, bool* any) {
    *any = false;
    int st = validate_cache4(c);
    if (st != GSDPA_OK) return st;
    if (n_rows < 0) return GSDPA_ERR_INVALID_ARG;
    if (n_rows == 0) return GSDPA_OK;
    if ((st = validate_cache4_pointers(c)) != GSDPA_OK) return st;
    if (!K || !V || !slots) return GSDPA_ERR_INVALID_ARG;
    const long long row = (long long)c->H_kv * c->d_k;
    if (ld_k < row || ld_v < row) return GSDPA_ERR_INVALID_ARG;
    if (!aligned(K, 16) || !aligned(V, 16) || ld_k % 8 != 0 || ld_v % 8 != 0 || !aligned(slots, 8))
        return GSDPA_ERR_ALIGNMENT;
    if (c->H_kv > 65535) return GSDPA_ERR_UNSUPPORTED;   // (heads are the grid's second axis)
    *any = true;
    return GSDPA_OK;
}

template <typename F>
int launch_rows(const gsdpa_cache4* c, RowsArgs& a, F launch) {
    Runtime rt;
    int major = 0, minor = 0;
    if (!current_runtime(&rt, &major, &minor)) return GSDPA_ERR_LAUNCH;
    if (!(major == 10 && minor == 3)) return GSDPA_ERR_UNSUPPORTED;
    a.pool = static_cast<uint8_t*>(c->pool);
    a.Hkv = c->H_kv;
    a.n_pages = c->n_pages;
    a.err = rt.err;
    return launch(dim3((unsigned)((a.n_rows + (long long)kRows - 1) / kRows), (unsigned)c->H_kv)) == cudaSuccess
               ? GSDPA_OK : GSDPA_ERR_LAUNCH;
}

}  // namespace

int validate_cache4(const gsdpa_cache4* c) {
    if (!c) return GSDPA_ERR_INVALID_ARG;
    if (c->kind != GSDPA_CACHE_INT4 && c->kind != GSDPA_CACHE_E2M1) return GSDPA_ERR_INVALID_ARG;
    if (c->n_pages < 1 || c->H_kv < 1) return GSDPA_ERR_INVALID_ARG;
    if (c->k_exp < -kMaxExp || c->k_exp > kMaxExp || c->v_exp < -kMaxExp || c->v_exp > kMaxExp) return GSDPA_ERR_INVALID_ARG;
    if (c->d_k != 64 && c->d_k != 128) return GSDPA_ERR_UNSUPPORTED;
    return GSDPA_OK;
}

int validate_cache4_pointers(const gsdpa_cache4* c) {
    if (!c->pool) return GSDPA_ERR_INVALID_ARG;
    return aligned(c->pool, 16) ? GSDPA_OK : GSDPA_ERR_ALIGNMENT;
}

}  // namespace gsdpa

using namespace gsdpa;

extern "C" {

int gsdpa_cache4_append(const gsdpa_cache4* cache, const void* K, const void* V, long long ld_k, long long ld_v,
                        const long long* slots, int n_rows, void* stream) {
    bool any;
    const int st = check_rows(cache, K, V, ld_k, ld_v, slots, n_rows, &any);
    if (st != GSDPA_OK || !any) return st;
    RowsArgs a{static_cast<const __nv_bfloat16*>(K), static_cast<const __nv_bfloat16*>(V), nullptr, nullptr, ld_k, ld_v,
               slots, nullptr, n_rows, 0, 0, ldexpf(1.f, -cache->k_exp), ldexpf(1.f, -cache->v_exp), nullptr};
    return launch_rows(cache, a, [&](dim3 grid) {
        const bool e2m1 = cache->kind == GSDPA_CACHE_E2M1;
        const auto k = cache->d_k == 128 ? (e2m1 ? cache4_append_kernel<128, true> : cache4_append_kernel<128, false>)
                                         : (e2m1 ? cache4_append_kernel<64, true> : cache4_append_kernel<64, false>);
        return launch_dependent(k, grid, dim3(kThreads), 0, static_cast<cudaStream_t>(stream), a);
    });
}

int gsdpa_cache4_read(const gsdpa_cache4* cache, const long long* slots, void* K, void* V, long long ld_k,
                      long long ld_v, int n_rows, void* stream) {
    bool any;
    const int st = check_rows(cache, K, V, ld_k, ld_v, slots, n_rows, &any);
    if (st != GSDPA_OK || !any) return st;
    RowsArgs a{nullptr, nullptr, static_cast<__nv_bfloat16*>(K), static_cast<__nv_bfloat16*>(V), ld_k, ld_v,
               slots, nullptr, n_rows, 0, 0, ldexpf(1.f, cache->k_exp), ldexpf(1.f, cache->v_exp), nullptr};
    return launch_rows(cache, a, [&](dim3 grid) {
        const bool e2m1 = cache->kind == GSDPA_CACHE_E2M1;
        const auto k = cache->d_k == 128 ? (e2m1 ? cache4_read_kernel<128, true> : cache4_read_kernel<128, false>)
                                         : (e2m1 ? cache4_read_kernel<64, true> : cache4_read_kernel<64, false>);
        return launch_dependent(k, grid, dim3(kThreads), 0, static_cast<cudaStream_t>(stream), a);
    });
}

}  // extern "C"
