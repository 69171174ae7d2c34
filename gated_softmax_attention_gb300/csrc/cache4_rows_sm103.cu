// cache4_rows_sm103.cu -- the paged 4-bit K/V cache, token by token: the append (bf16
// keys and values to codes and scales at their slots) and the reading back.
//
// Per 16 columns x of a token: scale s = e4m3(max |x| 2^-exp / top), codes
// round(x 2^-exp / s). x has 8 significant bits, s 4 and a border b between two codes 4, so
// that x and b s are whole numbers below 2^8 times powers of two: the quotient is on the border or
// 2^-8 of it away. The product with the rounded reciprocal is off by 2^-21 of itself at most; rounded
// to a multiple of 2^-15, as one fused multiply-add with 384 does, it is on a border where the
// quotient is and on its side elsewhere, so ties go as they should (plain products gave one code in 500
// another).
//
// Bound by HBM for prompts (4 d bytes in, 1.125 d out per token and head), by latency
// for a decoding step. A block has some rows of one head: it reads them whole, leaves codes
// and scales in shared memory token by token, and writes what the pages want: a
// key is d / 2 bytes in a row, but a value's go one to each of d / 2 words, whose other
// bytes are other tokens'. A thread has four words next to each other, 16 bytes, for
// which it turns four tokens' words around; where the block has all four tokens it
// writes them at once, else their bytes one by one, so that tokens next to each other can be
// written by different blocks and calls. The reading goes the same way back.
// Measured: prompts of 4 x 8190 tokens, 8 heads of 128 (172 MB), e2m1 33.5 us, 5.1 TB/s, int4 34.9 us, 4.9 TB/s, the
// issue slots three quarters busy with unpacking, codes and exchanges; heads of 64 18.8 us int4; 64 single tokens 3.0 us;
// reading 98k tokens, 2 heads of 128 (110 MB) 23 us, 4.8 TB/s.
#include "cache4_internal.h"

#include <cuda_fp16.h>
#include <cuda_fp8.h>

namespace gsdpa {
namespace {

// Threads of a block of 32 rows. (64 and 256 took 13 and 4 % longer for prompts of 4 x 8190 tokens, 3 and 9 % for
// reading 98k.)
constexpr int kMany = 128;

struct RowsArgs {
    const __nv_bfloat16 *K, *V;  // the append's
    __nv_bfloat16 *Ko, *Vo;      // the reading's
    long long ld_k, ld_v;
    const long long* slots;
    uint8_t* pool;
    int n_rows, Hkv, n_pages;
    float k_unit, v_unit;        // 2^exp
    uint32_t* err;
};

// Of two pairs of bf16 numbers the larger magnitudes, with some sign; NaN wins.
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Eight quotients -> their e2m1 codes, the first in the low 4 bits.
__device__ __forceinline__ uint32_t to_e2m1x8(const float (&y)[8]) {
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(r)
        : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
    return r;
}
using Pair = unsigned long long;   // two float32 numbers
__device__ __forceinline__ Pair pair_of(float lo, float hi) {
    Pair r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
    Pair r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

__device__ __forceinline__ Pair add2(Pair a, Pair b) {
    Pair r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ void unpair(Pair x, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(x));
}

// The 16 columns of a group -> their codes, 4 bits each, and the scale.
template <bool E2M1>
__device__ __forceinline__ void quantise(const uint4 (&x)[2], float unit, uint32_t (&codes)[2], uint32_t& scale) {
    const uint32_t w[8] = {x[0].x, x[0].y, x[0].z, x[0].w, x[1].x, x[1].y, x[1].z, x[1].w};
    uint32_t top = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) top = max_bf16x2(top, w[k]);
    top &= 0x7fff7fffu;
    const uint32_t most = max(top & 0xffffu, top >> 16);   // (a NaN is above all)
    const bool number = most < 0x7f80u;                    // (no NaN, no infinity)
    const float amax = __uint_as_float(most << 16);
    const float down = __uint_as_float(0x7f000000u - __float_as_uint(unit));   // 1 / unit
    const __nv_fp8_storage_t byte = __nv_cvt_float_to_fp8(amax * down * (1.f / (E2M1 ? 6.f : 7.f)), __NV_SATFINITE, __NV_E4M3);
    scale = number ? byte : 0x7fu;
    codes[0] = codes[1] = E2M1 ? 0u : 0x88888888u;
    if (!number || byte == 0) return;
    const float s = __half2float(__half(__nv_cvt_fp8_to_halfraw(byte, __NV_E4M3)));
    const float inv = __fdividef(1.f, s) * down;   // (the power of two: exact)
    const Pair inv2 = pair_of(inv, inv), up = pair_of(384.f, 384.f);
    // The largest quotient is at most 7 / (1 - 1 / 17) < 7.5, unless the scale is cut off at 448 or one of the least.
    const bool over = !E2M1 && amax * inv > 7.45f;
    Pair y[8];
#pragma unroll
    for (int k = 0; k < 8; ++k)
        y[k] = fma2(pair_of(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xffff0000u)), inv2, up);
    if (over) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            float a, b;
            unpair(y[k], a, b);
            y[k] = pair_of(fminf(fmaxf(a, 377.f), 391.f), fminf(fmaxf(b, 377.f), 391.f));
        }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float q[8];
        // e2m1: the 384 off again. int4: added to 1.5 2^23 + 8 (less the 384) a number is rounded to even and
        // stands in the low bits.
#pragma unroll
        for (int k = 0; k < 4; ++k)
            unpair(add2(y[4 * h + k], E2M1 ? pair_of(-384.f, -384.f) : pair_of(12582536.f, 12582536.f)), q[2 * k], q[2 * k + 1]);
        if constexpr (E2M1) {
            // (a number that is rounded to 384 has lost its sign, which the code of zero has too: bit 7 of every other byte)
            const uint32_t a = __byte_perm(w[4 * h], w[4 * h + 1], 0x7351), b = __byte_perm(w[4 * h + 2], w[4 * h + 3], 0x7351);
            codes[h] = to_e2m1x8(q) | (__byte_perm(a, b, 0x5410) >> 4 & 0x08080808u) | (__byte_perm(a, b, 0x7632) & 0x80808080u);
        } else {
            uint32_t r = 0;
#pragma unroll
            for (int k = 7; k >= 0; --k) r = r * 16 + __float_as_uint(q[k]);
            codes[h] = r - 0x4b400000u * 0x11111111u;
        }
    }
}

// Byte b of words 0 .. 3 -> byte 0 .. 3 of word b.
__device__ __forceinline__ void turn_bytes(uint32_t (&w)[4]) {
    const uint32_t a = __byte_perm(w[0], w[1], 0x5140), b = __byte_perm(w[2], w[3], 0x5140);
    const uint32_t c = __byte_perm(w[0], w[1], 0x7362), d = __byte_perm(w[2], w[3], 0x7362);
    w[0] = __byte_perm(a, b, 0x5410);
    w[1] = __byte_perm(a, b, 0x7632);
    w[2] = __byte_perm(c, d, 0x5410);
    w[3] = __byte_perm(c, d, 0x7632);
}

// The rows of one block: the slot of each, and the runs of rows that lie in one tile of
// 16 tokens (a run begins where the tile changes).
template <int R, int THREADS>
struct Runs {
    long long slot[R];        // -1: none
    long long tile[R];        // by run: slot / 16
    int run[R];               // by row
    signed char at[R][16];    // by run: its row at each place of the tile, or -1
    int n;                    // runs
    __device__ __forceinline__ void find(const RowsArgs& a, long long first) {
        const int tid = threadIdx.x;
        for (int k = tid; k < R * 4; k += THREADS) reinterpret_cast<uint32_t*>(at)[k] = 0xffffffffu;
        __syncthreads();
        if (tid < 32) {
            const long long row = first + tid;
            long long s = tid < R && row < a.n_rows ? a.slots[row] : -1;
            if (s >= (long long)a.n_pages * kPage) {
                s = -1;
                atomicOr(a.err, ERR_CACHE_RANGE);
            }
            if (s < 0) s = -1;
            const long long before = __shfl_up_sync(0xffffffffu, s, 1);
            const bool lead = s >= 0 && (tid == 0 || (s >> 4) != (before >> 4));
            const uint32_t leads = __ballot_sync(0xffffffffu, lead);
            const int run_of = __popc(leads & (0xffffffffu >> (31 - tid))) - 1;
            if (tid < R) {
                slot[tid] = s;
                run[tid] = run_of;
            }
            if (lead) tile[run_of] = s >> 4;
            if (s >= 0) at[run_of][s & 15] = (signed char)tid;
            if (tid == 0) n = __popc(leads);
        }
        __syncthreads();
    }
};

// A block's tokens as bytes: keys as the pages have them, values [quad][g][j % 4], whose rows lie
// so that four tokens' words 2 t are in different banks.
template <int D, int R>
struct Tokens {
    static constexpr int LDV = D == 128 ? 80 : 48;
    __align__(16) uint8_t key[R][D / 2];
    __align__(16) uint8_t value[R][LDV];
    __align__(16) uint8_t kscale[R][D / 16], vscale[R][D / 16];
};

// The 16-byte pieces of a tile's value codes (quad, g, t) and, behind them, of its scales (t, 4 groups).
template <int D>
struct Pieces {
    static constexpr int CODES = D / 2, ALL = D / 2 + D / 16;
    int t, from, to;   // lane; first byte of a token's; byte of the page's tile
    bool scales;
    __device__ __forceinline__ explicit Pieces(int w) {
        scales = w >= CODES;
        if (scales) {
            t = (w - CODES) / (D / 64);
            from = 4 * ((w - CODES) % (D / 64));
        } else {
            t = w % 4;
            from = 4 * (w / 4);
        }
        to = 16 * (scales ? w - CODES : w);
    }
    __device__ __forceinline__ uint8_t* at(uint8_t* page, int tile) const {
        return page + (scales ? value_scales_at(D) + D * tile : value_codes_at(D) + 8 * D * tile) + to;
    }
    // place of the token that has byte b of a word
    template <bool E2M1>
    __device__ __forceinline__ int place(int b) const {
        if (E2M1 || b == 0 || b == 3) return 2 * t + (b & 1) + 8 * (b >> 1);
        return 2 * t + (scales == (b == 1) ? 1 : 8);
    }
};

template <int D, bool E2M1, int R, int THREADS>
__global__ void __launch_bounds__(THREADS) cache4_append_kernel(const __grid_constant__ RowsArgs a) {
    __shared__ Runs<R, THREADS> runs;
    __shared__ Tokens<D, R> tok;
    pdl_trigger();
    pdl_wait();
    const int tid = threadIdx.x, h = blockIdx.y;
    const long long first = (long long)blockIdx.x * R;
    // ---- a lane has a group's 16 columns; lanes next to each other the groups of one token. All is loaded at once,
    // before the slots are known.
    constexpr int GROUPS = 2 * R * (D / 16), EACH = (GROUPS + THREADS - 1) / THREADS;
    static_assert(GROUPS % THREADS == 0 || GROUPS < THREADS, "whole warps");
    uint4 x[EACH][2];
#pragma unroll
    for (int n = 0; n < EACH; ++n) {
        const int k = n * THREADS + tid;
        const bool value = k >= R * (D / 16);
        const int i = k % (R * (D / 16)), r = i / (D / 16), j = i % (D / 16);
        x[n][0] = x[n][1] = make_uint4(0, 0, 0, 0);
        if (k < GROUPS && first + r < a.n_rows) {
            const uint4* from = reinterpret_cast<const uint4*>((value ? a.V + (first + r) * a.ld_v : a.K + (first + r) * a.ld_k) +
                                                               (long long)h * D + 16 * j);
            x[n][0] = from[0];
            x[n][1] = from[1];
        }
    }
    runs.find(a, first);

    // ---- codes and scales
#pragma unroll
    for (int n = 0; n < EACH; ++n) {
        const int k = n * THREADS + tid;
        if (k >= GROUPS) break;
        const bool value = k >= R * (D / 16);
        const int i = k % (R * (D / 16)), r = i / (D / 16), j = i % (D / 16);
        uint32_t codes[2], scale;
        quantise<E2M1>(x[n], value ? a.v_unit : a.k_unit, codes, scale);
        (value ? tok.vscale : tok.kscale)[r][j] = (uint8_t)scale;
        if (!value) {
            if (E2M1) {   // two bytes of each t
#pragma unroll
                for (int t = 0; t < 4; ++t)
                    *reinterpret_cast<uint16_t*>(&tok.key[r][t * (D / 8) + 2 * j]) = (uint16_t)(codes[t / 2] >> (16 * (t % 2)));
            } else {
                // a word of each t: of this group and its neighbour columns 0 | 2, 0 | 2, 1 | 3, 1 | 3. Lanes
                // of even groups take those of t = 0, 1.
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const uint32_t d = (codes[c] ^ (codes[c] >> 4)) & 0x00f000f0u;
                    codes[c] ^= d ^ (d << 4);
                }
                const uint32_t other = __shfl_xor_sync(0xffffffffu, j % 2 ? codes[0] : codes[1], 1);
                const uint32_t even = j % 2 ? other : codes[0], odd = j % 2 ? codes[1] : other;
                uint8_t* to = &tok.key[r][2 * (j % 2) * (D / 8) + 4 * (j / 2)];
                *reinterpret_cast<uint32_t*>(to) = __byte_perm(even, odd, 0x5140);
                *reinterpret_cast<uint32_t*>(to + D / 8) = __byte_perm(even, odd, 0x7362);
            }
        } else {
            // bytes of columns g and 8 + g, the even and the odd g; four groups' of one g are a word: lane j % 4 ends
            // with those of two of the eight
            uint32_t mine = (codes[0] & 0x0f0f0f0fu) | (codes[1] << 4 & 0xf0f0f0f0u);
            uint32_t give = (codes[0] >> 4 & 0x0f0f0f0fu) | (codes[1] & 0xf0f0f0f0u);
            if (j & 1) {
                const uint32_t x = mine;
                mine = give;
                give = x;
            }
            uint32_t got = __shfl_xor_sync(0xffffffffu, give, 1);
            const uint32_t lo = j & 1 ? got : mine, hi = j & 1 ? mine : got;
            mine = __byte_perm(lo, hi, 0x5140);   // two of this lane's g (the first two of its four)
            give = __byte_perm(lo, hi, 0x7362);
            if (j & 2) {
                const uint32_t x = mine;
                mine = give;
                give = x;
            }
            got = __shfl_xor_sync(0xffffffffu, give, 2);
            const uint32_t first_two = j & 2 ? got : mine, last_two = j & 2 ? mine : got;
            uint32_t* to = reinterpret_cast<uint32_t*>(&tok.value[r][j / 4 * 32]) + (j & 1) + 2 * (j & 2);
            to[0] = __byte_perm(first_two, last_two, 0x5410);
            to[2] = __byte_perm(first_two, last_two, 0x7632);
        }
    }
    __syncthreads();

    // ---- keys: rows of D / 2 bytes, and their scales
    const auto page_of = [&](long long slot) { return a.pool + ((slot / kPage) * a.Hkv + h) * page_bytes(D); };
    for (int k = tid; k < R * (D / 32); k += THREADS) {
        const int r = k / (D / 32), c = k % (D / 32);
        const long long slot = runs.slot[r];
        if (slot >= 0)
            *reinterpret_cast<uint4*>(page_of(slot) + (slot % kPage) * (D / 2) + 16 * c) =
                *reinterpret_cast<const uint4*>(&tok.key[r][16 * c]);
    }
    for (int k = tid; k < R * (D / 64); k += THREADS) {
        const int r = k / (D / 64), c = k % (D / 64);
        const long long slot = runs.slot[r];
        if (slot >= 0)
            *reinterpret_cast<uint32_t*>(page_of(slot) + key_scales_at(D) + (slot % kPage) * (D / 16) + 4 * c) =
                *reinterpret_cast<const uint32_t*>(&tok.kscale[r][4 * c]);
    }

    // ---- values: four words of four tokens, run by run
    using P = Pieces<D>;
    for (int k = tid; k < runs.n * P::ALL; k += THREADS) {
        const int run = k / P::ALL;
        const P p(k % P::ALL);
        uint32_t w[4];
        int have = 0;
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const int row = runs.at[run][p.template place<E2M1>(b)];
            w[b] = 0;
            if (row >= 0) {
                have |= 1 << b;
                w[b] = *reinterpret_cast<const uint32_t*>(p.scales ? &tok.vscale[row][p.from] : &tok.value[row][p.from]);
            }
        }
        turn_bytes(w);
        if (have == 0) continue;
        uint8_t* to = p.at(page_of(runs.tile[run] * 16), (int)(runs.tile[run] % 4));
        if (have == 15) {
            *reinterpret_cast<uint4*>(to) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
#pragma unroll
            for (int b = 0; b < 4; ++b)
                if (have & (1 << b))
#pragma unroll
                    for (int c = 0; c < 4; ++c) to[4 * c + b] = (uint8_t)(w[c] >> (8 * b));
        }
    }
}

__device__ __forceinline__ float scale_value(uint32_t byte) {
    return __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)byte, __NV_E4M3)));
}
// The two codes of a byte as the numbers they stand for.
template <bool E2M1>
__device__ __forceinline__ float2 code_values(uint32_t byte) {
    if constexpr (E2M1) {
        uint32_t h;
        asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, a;\n\t}" : "=r"(h) : "r"(byte));
        return __half22float2(*reinterpret_cast<const __half2*>(&h));
    } else {
        return make_float2((float)((int)(byte & 15u) - 8), (float)((int)(byte >> 4 & 15u) - 8));
    }
}

template <int D, bool E2M1, int R, int THREADS>
__global__ void __launch_bounds__(THREADS) cache4_read_kernel(const __grid_constant__ RowsArgs a) {
    __shared__ Runs<R, THREADS> runs;
    __shared__ Tokens<D, R> tok;
    pdl_trigger();
    pdl_wait();
    const int tid = threadIdx.x, h = blockIdx.y;
    const long long first = (long long)blockIdx.x * R;
    runs.find(a, first);
    const auto page_of = [&](long long slot) { return a.pool + ((slot / kPage) * a.Hkv + h) * page_bytes(D); };
    for (int k = tid; k < R * (D / 32); k += THREADS) {
        const int r = k / (D / 32), c = k % (D / 32);
        const long long slot = runs.slot[r];
        if (slot >= 0)
            *reinterpret_cast<uint4*>(&tok.key[r][16 * c]) =
                *reinterpret_cast<const uint4*>(page_of(slot) + (slot % kPage) * (D / 2) + 16 * c);
    }
    for (int k = tid; k < R * (D / 64); k += THREADS) {
        const int r = k / (D / 64), c = k % (D / 64);
        const long long slot = runs.slot[r];
        if (slot >= 0)
            *reinterpret_cast<uint32_t*>(&tok.kscale[r][4 * c]) =
                *reinterpret_cast<const uint32_t*>(page_of(slot) + key_scales_at(D) + (slot % kPage) * (D / 16) + 4 * c);
    }
    using P = Pieces<D>;
    for (int k = tid; k < runs.n * P::ALL; k += THREADS) {
        const int run = k / P::ALL;
        const P p(k % P::ALL);
        const uint4 x = *reinterpret_cast<const uint4*>(p.at(page_of(runs.tile[run] * 16), (int)(runs.tile[run] % 4)));
        uint32_t w[4] = {x.x, x.y, x.z, x.w};
        turn_bytes(w);
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const int row = runs.at[run][p.template place<E2M1>(b)];
            if (row >= 0)
                *reinterpret_cast<uint32_t*>(p.scales ? &tok.vscale[row][p.from] : &tok.value[row][p.from]) = w[b];
        }
    }
    __syncthreads();

    // ---- a thread to a group's 16 columns
    for (int k = tid; k < 2 * R * (D / 16); k += THREADS) {
        const bool value = k >= R * (D / 16);
        const int i = k % (R * (D / 16)), r = i / (D / 16), j = i % (D / 16);
        if (first + r >= a.n_rows) continue;
        uint32_t out[8] = {};
        if (runs.slot[r] >= 0) {
            // (of rows with the same slot the values' bytes are one row's)
            const int from_row = value ? runs.at[runs.run[r]][runs.slot[r] & 15] : r;
            const float s = scale_value((value ? tok.vscale : tok.kscale)[from_row][j]) * (value ? a.v_unit : a.k_unit);
            if (value) {
                float2 x[8];   // columns g and 8 + g
#pragma unroll
                for (int g = 0; g < 8; ++g) x[g] = code_values<E2M1>(tok.value[from_row][j / 4 * 32 + g * 4 + j % 4]);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    out[c] = pack_bf16x2(x[2 * c].x * s, x[2 * c + 1].x * s);
                    out[4 + c] = pack_bf16x2(x[2 * c].y * s, x[2 * c + 1].y * s);
                }
            } else {
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    const uint8_t* from = &tok.key[r][t * (D / 8) + (E2M1 ? 2 * j : 4 * (j / 2) + j % 2)];
                    const float2 x = code_values<E2M1>(from[0]), y = code_values<E2M1>(from[E2M1 ? 1 : 2]);
                    // e2m1: columns 0, 1 and 2, 3 of the lane's four; int4: 0, 2 and 1, 3
                    out[2 * t] = E2M1 ? pack_bf16x2(x.x * s, x.y * s) : pack_bf16x2(x.x * s, y.x * s);
                    out[2 * t + 1] = E2M1 ? pack_bf16x2(y.x * s, y.y * s) : pack_bf16x2(x.y * s, y.y * s);
                }
            }
        }
        uint4* to = reinterpret_cast<uint4*>((value ? a.Vo + (first + r) * a.ld_v : a.Ko + (first + r) * a.ld_k) +
                                             (long long)h * D + 16 * j);
        to[0] = make_uint4(out[0], out[1], out[2], out[3]);
        to[1] = make_uint4(out[4], out[5], out[6], out[7]);
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

template <bool READ, int D, bool E2M1>
cudaError_t launch(const RowsArgs& a, int sms, cudaStream_t s) {
    const auto go = [&](auto kernel, int rows, int threads) {
        const dim3 grid((unsigned)((a.n_rows + (long long)rows - 1) / rows), (unsigned)a.Hkv);
        return launch_dependent(kernel, grid, dim3(threads), 0, s, a);
    };
    // Blocks of few rows, with more threads to a row, until there are two of the others for every SM (2849 tokens, 5 heads of
    // 64: 450 of the others, 3.6 us, of these 4.4; one token of 64 sequences, 8 heads of 128: 3.1 and 3.0).
    constexpr int FEW = 2 * D;
    if ((a.n_rows + 31LL) / 32 * a.Hkv < 2LL * sms) {
        if constexpr (READ) return go(cache4_read_kernel<D, E2M1, 8, FEW>, 8, FEW);
        else return go(cache4_append_kernel<D, E2M1, 8, FEW>, 8, FEW);
    }
    if constexpr (READ) return go(cache4_read_kernel<D, E2M1, 32, kMany>, 32, kMany);
    else return go(cache4_append_kernel<D, E2M1, 32, kMany>, 32, kMany);
}

template <bool READ>
int launch_rows(const gsdpa_cache4* c, RowsArgs& a, void* stream) {
    Runtime rt;
    int major = 0, minor = 0;
    if (!current_runtime(&rt, &major, &minor)) return GSDPA_ERR_LAUNCH;
    if (!(major == 10 && minor == 3)) return GSDPA_ERR_UNSUPPORTED;
    a.pool = static_cast<uint8_t*>(c->pool);
    a.Hkv = c->H_kv;
    a.n_pages = c->n_pages;
    a.k_unit = ldexpf(1.f, c->k_exp);
    a.v_unit = ldexpf(1.f, c->v_exp);
    a.err = rt.err;
    const bool e2m1 = c->kind == GSDPA_CACHE_E2M1;
    const auto s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = c->d_k == 128 ? (e2m1 ? launch<READ, 128, true>(a, rt.num_sms, s) : launch<READ, 128, false>(a, rt.num_sms, s))
                                        : (e2m1 ? launch<READ, 64, true>(a, rt.num_sms, s) : launch<READ, 64, false>(a, rt.num_sms, s));
    return e == cudaSuccess ? GSDPA_OK : GSDPA_ERR_LAUNCH;
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
    RowsArgs a{};
    a.K = static_cast<const __nv_bfloat16*>(K);
    a.V = static_cast<const __nv_bfloat16*>(V);
    a.ld_k = ld_k;
    a.ld_v = ld_v;
    a.slots = slots;
    a.n_rows = n_rows;
    return launch_rows<false>(cache, a, stream);
}

int gsdpa_cache4_read(const gsdpa_cache4* cache, const long long* slots, void* K, void* V, long long ld_k,
                      long long ld_v, int n_rows, void* stream) {
    bool any;
    const int st = check_rows(cache, K, V, ld_k, ld_v, slots, n_rows, &any);
    if (st != GSDPA_OK || !any) return st;
    RowsArgs a{};
    a.Ko = static_cast<__nv_bfloat16*>(K);
    a.Vo = static_cast<__nv_bfloat16*>(V);
    a.ld_k = ld_k;
    a.ld_v = ld_v;
    a.slots = slots;
    a.n_rows = n_rows;
    return launch_rows<true>(cache, a, stream);
}

}  // extern "C"
