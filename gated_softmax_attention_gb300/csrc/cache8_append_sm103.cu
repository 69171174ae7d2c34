// cache8_append_sm103.cu -- new keys and values into the K/V cache held in 8
// bits with one scale per block of 64 tokens and head.
//
// A block is written in 8 bits once, when its 64 tokens are known; until then
// they wait as bf16 in one of two open-block buffers (even and odd blocks). So
// every element is rounded once, and the cache's contents do not depend on how
// the tokens were split over calls. With amax the largest |x| of the block:
//   int8: s = fl32(amax fl32(1 / 127)), code = x / s rounded to nearest even;
//   e4m3: s = 2^e with the least e >= -126 that keeps amax <= 448 s (a power
//         of two costs a floating-point code nothing but range and makes x / s
//         exact), code = x / s rounded to nearest even.
// The int8 quotient is decided exactly: q0 = x * (1/s) rounded is off by one at
// most, and the remainder x - q0 s, exact in one fused multiply-add (x has 8
// significant bits, and where q0 is not zero its last bit is not below s's),
// says whether it is (hardly ever: four elements share the question).
//
// Bound by HBM for prompts (2 bytes in, 1 out for each element) and by latency
// for single tokens. One CTA per (sequence, head, touched block) handles keys
// and values, so a prompt fills the GPU and the tile stays in registers between
// the maximum and the rounding. Values are stored transposed ([d_k][64]: the
// product with the weights sums over tokens); a thread holds 4 tokens x 8
// columns of them, so that the 4 tokens of a column make one 32-bit store.
// The first block's CTA also writes the open block: it alone reads the old
// open tokens, and writes after it has read.
//
// Measured, 8 heads of 128: 4 x 8190 tokens 34 us in e4m3 (5.9 TB/s, 87 % of a plain
// copy), 37.5 us in int8; one token of 64 sequences 5.1 us.
#include "cache8_internal.h"

namespace gsdpa {
namespace {

constexpr int kThreads = 256;

struct AppendArgs {
    const __nv_bfloat16 *K, *V;   // [B, L] rows of H_kv * d_k
    long long ld_k, ld_v;
    const int *lens, *n_new;
    uint8_t *k8, *v8;
    float *k_scale, *v_scale;
    __nv_bfloat16 *k_tail, *v_tail;
    int L, Hkv, blocks, capacity, touched;
    uint32_t* err;
};

__device__ __forceinline__ void unpack_bf16x8(const uint4& w, float (&f)[8]) {
    const uint32_t r[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        f[2 * k] = __uint_as_float(r[k] << 16);
        f[2 * k + 1] = __uint_as_float(r[k] & 0xffff0000u);
    }
}

// The largest |x| of two bf16 pairs each, as bits (ordered like the values, NaN above infinity).
__device__ __forceinline__ uint32_t abs_max2(uint32_t m, uint32_t pair) { return __vmaxu2(m, pair & 0x7fff7fffu); }

// A block's scale and how its elements are rounded.
template <bool E4M3>
struct Quantiser {
    float scale;   // stored
    float s, inv, lift;
    __device__ __forceinline__ explicit Quantiser(uint32_t amax_bits) {
        const float amax = __uint_as_float(amax_bits);
        lift = 1.f;
        if (amax_bits >= 0x7f800000u) {   // an infinity or NaN: the scale says so, the codes are zero
            scale = __uint_as_float(0x7fc00000u);
            s = 1.f;
            inv = lift = 0.f;
        } else if (amax_bits == 0) {
            scale = 0.f;
            s = 1.f;
            inv = lift = 0.f;
        } else if constexpr (E4M3) {
            const int k = (int)(amax_bits >> 23) - 127;   // (a subnormal amax: k = -127, e = -126 below)
            int e = (amax_bits & 0x7fffffu) <= 0x600000u ? k - 8 : k - 7;
            e = e < -126 ? -126 : e;
            scale = s = __uint_as_float((uint32_t)(e + 127) << 23);
            inv = __uint_as_float((uint32_t)(127 - e) << 23);
        } else {
            scale = s = __fmul_rn(amax, 1.f / 127.f);
            if (s < 8.6736174e-19f) {   // 2^-60: lifted by 2^60 so that 1/s and the remainders stay normal
                lift = 1.152921504606847e18f;
                s *= lift;
            }
            inv = __fdiv_rn(1.f, s);
        }
    }
    // one code, exactly
    __device__ __forceinline__ uint32_t exact(float x) const {
        const float y = x * lift;
        float q = rintf(y * inv);
        const float r = fmaf(-q, s, y), h = 0.5f * s;
        if (fabsf(r) > h || (fabsf(r) == h && ((int)q & 1))) q += r > 0.f ? 1.f : -1.f;
        q = fminf(fmaxf(q, -127.f), 127.f);
        return (uint32_t)(int)q & 255u;
    }
    // 4 codes as one word, the first in the lowest byte
    __device__ __forceinline__ uint32_t word(float a, float b, float c, float d) const {
        if (lift == 0.f) return 0;
        if constexpr (E4M3) {
            uint16_t lo, hi;
            asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b * inv), "f"(a * inv));
            asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d * inv), "f"(c * inv));
            return (uint32_t)lo | ((uint32_t)hi << 16);
        } else {
            // x inv + 1.5 2^23 has the quotient, rounded to nearest even, in its low bits
            constexpr float kRound = 12582912.f;
            const float2 x[2] = {make_float2(a, b), make_float2(c, d)};
            float2 t[2];
            float off = 0.f;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                t[k] = __ffma2_rn(x[k], make_float2(inv, inv), make_float2(kRound, kRound));
                const float2 q = __fadd2_rn(t[k], make_float2(-kRound, -kRound));
                const float2 r = __ffma2_rn(q, make_float2(-s, -s), x[k]);
                off = fmaxf(off, fmaxf(fabsf(r.x), fabsf(r.y)));
            }
            if (lift == 1.f && off < 0.5f * s) {   // every remainder is below half a step
                const uint32_t lo = __byte_perm(__float_as_uint(t[0].x), __float_as_uint(t[0].y), 0x0040);
                const uint32_t hi = __byte_perm(__float_as_uint(t[1].x), __float_as_uint(t[1].y), 0x0040);
                return __byte_perm(lo, hi, 0x5410);
            }
            return exact(a) | (exact(b) << 8) | (exact(c) << 16) | (exact(d) << 24);
        }
    }
};

// CTAS: of an SM. Prompts gain by the fifth (4 x 8190 tokens 35.1 -> 34.2 us), whose
// fewer registers cost a step or a short prompt (one token of 64 sequences 5.1 ->
// 5.9 us, 4 x 1000 tokens 9.5 -> 10.3).
template <int D, bool E4M3, int CTAS>
__global__ void __launch_bounds__(kThreads, CTAS) cache8_append_kernel(const AppendArgs a) {
    constexpr int CH = D / 8;                              // 16-byte pieces of a row
    constexpr int KP = kCacheBlock * CH / kThreads;        // ... of the key tile per thread
    __shared__ uint32_t red[2][kThreads / 32];
    const int tid = threadIdx.x;
    // (heads first: CTAs that run together read whole token rows; one head's blocks after the other 36.7 instead of 35.1 us)
    const int h = blockIdx.x % a.Hkv, x = blockIdx.x / a.Hkv % a.touched, b = blockIdx.x / a.Hkv / a.touched;
    const int unit = b * a.Hkv + h;
    pdl_wait();   // the new rows and lengths may be the previous kernel's outputs
    pdl_trigger();
    const SeqRange q = seq_range(a.lens, a.n_new, b, a.L, a.capacity);
    if (!q.ok && x == 0 && h == 0 && tid == 0) atomicOr(a.err, ERR_CACHE_RANGE);
    if (q.n == 0) return;
    const int end = q.len + q.n;
    const int first = q.len / kCacheBlock, last = (end - 1) / kCacheBlock;
    const int j = first + x;
    if (j > last) return;
    const __nv_bfloat16* newK = a.K + (long long)b * a.L * a.ld_k + (long long)h * D;
    const __nv_bfloat16* newV = a.V + (long long)b * a.L * a.ld_v + (long long)h * D;
    __nv_bfloat16* tailK = a.k_tail + (long long)unit * 2 * kCacheBlock * D;   // [2][64][D]
    __nv_bfloat16* tailV = a.v_tail + (long long)unit * 2 * kCacheBlock * D;   // [2][D][64]
    // values: tokens 4 vq .. 4 vq + 3, columns 8 vc .. 8 vc + 7
    const int vq = tid % 16, vc = tid / 16;
    const bool has_v = vc < CH;
    const int p0 = j * kCacheBlock;

    // The new tokens of the last two touched blocks also go to the open-block
    // buffers: the last one may still be open, and the one before keeps the
    // step reversible (a length taken back by up to 64 tokens finds its open
    // block's tokens there).
    const auto keep_open = [&]() {
        for (int t = max(first, last - 1); t <= last; ++t) {
            const int lo = max(q.len, t * kCacheBlock), hi = min(end, (t + 1) * kCacheBlock);
            __nv_bfloat16* toK = tailK + (long long)(t & 1) * kCacheBlock * D;
            __nv_bfloat16* toV = tailV + (long long)(t & 1) * kCacheBlock * D;
            for (int i = tid; i < (hi - lo) * CH; i += kThreads) {
                const int p = lo + i / CH, c = i % CH;
                *reinterpret_cast<uint4*>(toK + (p - t * kCacheBlock) * D + 8 * c) =
                    *reinterpret_cast<const uint4*>(newK + (long long)(p - q.len) * a.ld_k + 8 * c);
            }
            if (!has_v) continue;
            const int pv = t * kCacheBlock + 4 * vq;
            if (pv + 3 < lo || pv >= hi) continue;
            uint32_t w[4][4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                uint4 r = make_uint4(0, 0, 0, 0);
                if (pv + k >= lo && pv + k < hi)
                    r = *reinterpret_cast<const uint4*>(newV + (long long)(pv + k - q.len) * a.ld_v + 8 * vc);
                w[k][0] = r.x;
                w[k][1] = r.y;
                w[k][2] = r.z;
                w[k][3] = r.w;
            }
            const bool whole = pv >= lo && pv + 3 < hi;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint32_t sel = (e & 1) ? 0x7632u : 0x5410u;
                const uint32_t ab = __byte_perm(w[0][e / 2], w[1][e / 2], sel);
                const uint32_t cd = __byte_perm(w[2][e / 2], w[3][e / 2], sel);
                uint16_t* to = reinterpret_cast<uint16_t*>(toV) + (8 * vc + e) * kCacheBlock + 4 * vq;
                if (whole) {
                    *reinterpret_cast<uint2*>(to) = make_uint2(ab, cd);
                } else {
                    if (pv >= lo && pv < hi) to[0] = (uint16_t)ab;
                    if (pv + 1 >= lo && pv + 1 < hi) to[1] = (uint16_t)(ab >> 16);
                    if (pv + 2 >= lo && pv + 2 < hi) to[2] = (uint16_t)cd;
                    if (pv + 3 >= lo && pv + 3 < hi) to[3] = (uint16_t)(cd >> 16);
                }
            }
        }
    };
    // With one or two touched blocks no new token takes the place of an old one
    // that the first block still needs, so there is nothing to wait for.
    const bool early = last - first < 2;
    if (x == 0 && early) keep_open();

    if (p0 + kCacheBlock <= end) {
        uint4 kw[KP], vw[4];
#pragma unroll
        for (int i = 0; i < KP; ++i) {
            const int row = (i * kThreads + tid) / CH, c = (i * kThreads + tid) % CH;
            const int p = p0 + row;
            const __nv_bfloat16* src = p < q.len ? tailK + ((long long)(j & 1) * kCacheBlock + row) * D
                                                 : newK + (long long)(p - q.len) * a.ld_k;
            kw[i] = *reinterpret_cast<const uint4*>(src + 8 * c);
        }
        const int pv = p0 + 4 * vq;
        const int n_old = q.len - pv;   // of the thread's 4 tokens, how many are in the open block
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            vw[k] = make_uint4(0, 0, 0, 0);
            if (has_v && k >= n_old)
                vw[k] = *reinterpret_cast<const uint4*>(newV + (long long)(pv + k - q.len) * a.ld_v + 8 * vc);
        }
        if (has_v && n_old > 0) {   // (the first block only: 4 tokens of a column are 8 bytes there)
            uint2 old[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                old[e] = *reinterpret_cast<const uint2*>(tailV + ((long long)(j & 1) * D + 8 * vc + e) * kCacheBlock + 4 * vq);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t sel = (k & 1) ? 0x7632u : 0x5410u;
                if (k < n_old)
                    vw[k] = k < 2 ? make_uint4(__byte_perm(old[0].x, old[1].x, sel), __byte_perm(old[2].x, old[3].x, sel),
                                               __byte_perm(old[4].x, old[5].x, sel), __byte_perm(old[6].x, old[7].x, sel))
                                  : make_uint4(__byte_perm(old[0].y, old[1].y, sel), __byte_perm(old[2].y, old[3].y, sel),
                                               __byte_perm(old[4].y, old[5].y, sel), __byte_perm(old[6].y, old[7].y, sel));
            }
        }
        uint32_t mk = 0, mv = 0;
#pragma unroll
        for (int i = 0; i < KP; ++i)
            mk = abs_max2(abs_max2(abs_max2(abs_max2(mk, kw[i].x), kw[i].y), kw[i].z), kw[i].w);
#pragma unroll
        for (int k = 0; k < 4; ++k)
            mv = abs_max2(abs_max2(abs_max2(abs_max2(mv, vw[k].x), vw[k].y), vw[k].z), vw[k].w);
        mk = __reduce_max_sync(0xffffffffu, max(mk & 0xffffu, mk >> 16));
        mv = __reduce_max_sync(0xffffffffu, max(mv & 0xffffu, mv >> 16));
        if ((tid & 31) == 0) {
            red[0][tid / 32] = mk;
            red[1][tid / 32] = mv;
        }
        __syncthreads();   // (the old open tokens have been read by every thread: they are in the maxima)
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) {
            mk = max(mk, red[0][w]);
            mv = max(mv, red[1][w]);
        }
        const long long tile = (long long)unit * a.blocks + j;
        const Quantiser<E4M3> qk(mk << 16), qv(mv << 16);
        if (tid == 0) {
            a.k_scale[tile] = qk.scale;
            a.v_scale[tile] = qv.scale;
        }
        uint8_t* k8 = a.k8 + tile * kCacheBlock * D;
        uint8_t* v8 = a.v8 + tile * kCacheBlock * D;
#pragma unroll
        for (int i = 0; i < KP; ++i) {
            const int row = (i * kThreads + tid) / CH, c = (i * kThreads + tid) % CH;
            float f[8];
            unpack_bf16x8(kw[i], f);
            *reinterpret_cast<uint2*>(k8 + row * D + 8 * c) =
                make_uint2(qk.word(f[0], f[1], f[2], f[3]), qk.word(f[4], f[5], f[6], f[7]));
        }
        if (has_v) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float f[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t r = e < 2 ? vw[k].x : (e < 4 ? vw[k].y : (e < 6 ? vw[k].z : vw[k].w));
                    f[k] = __uint_as_float((e & 1) ? r & 0xffff0000u : r << 16);
                }
                *reinterpret_cast<uint32_t*>(v8 + (8 * vc + e) * kCacheBlock + 4 * vq) = qv.word(f[0], f[1], f[2], f[3]);
            }
        }
    }
    if (x == 0 && !early) keep_open();
}

template <int D, bool E4M3>
cudaError_t launch(const AppendArgs& a, bool many, unsigned grid, cudaStream_t s) {
    return many ? launch_dependent(cache8_append_kernel<D, E4M3, 5>, dim3(grid), dim3(kThreads), 0, s, a)
                : launch_dependent(cache8_append_kernel<D, E4M3, 4>, dim3(grid), dim3(kThreads), 0, s, a);
}

bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

}  // namespace

int validate_cache8(const gsdpa_cache8* c) {
    if (!c) return GSDPA_ERR_INVALID_ARG;
    if (c->kind != GSDPA_CACHE_INT8 && c->kind != GSDPA_CACHE_E4M3) return GSDPA_ERR_INVALID_ARG;
    if (c->B < 0 || c->H_kv < 1) return GSDPA_ERR_INVALID_ARG;
    if (c->capacity < kCacheBlock || c->capacity % kCacheBlock != 0) return GSDPA_ERR_INVALID_ARG;
    if (c->d_k != 64 && c->d_k != 128) return GSDPA_ERR_UNSUPPORTED;
    // (units and tiles are counted in 32 and 64 bits)
    if ((long long)c->B * c->H_kv > 0x7fffffffLL) return GSDPA_ERR_UNSUPPORTED;
    return GSDPA_OK;
}

int validate_cache8_pointers(const gsdpa_cache8* c) {
    if (!c->k8 || !c->v8 || !c->k_scale || !c->v_scale || !c->k_tail || !c->v_tail) return GSDPA_ERR_INVALID_ARG;
    if (!aligned(c->k8, 16) || !aligned(c->v8, 16) || !aligned(c->k_tail, 16) || !aligned(c->v_tail, 16))
        return GSDPA_ERR_ALIGNMENT;
    if (!aligned(c->k_scale, 4) || !aligned(c->v_scale, 4)) return GSDPA_ERR_ALIGNMENT;
    return GSDPA_OK;
}

}  // namespace gsdpa

using namespace gsdpa;

extern "C" int gsdpa_cache8_append(const gsdpa_cache8* cache, const void* K, const void* V, long long ld_k,
                                   long long ld_v, const int* lens, const int* n_new, int L, void* stream) {
    int st = validate_cache8(cache);
    if (st != GSDPA_OK) return st;
    if (L < 0) return GSDPA_ERR_INVALID_ARG;
    if (cache->B == 0 || L == 0) return GSDPA_OK;
    if ((st = validate_cache8_pointers(cache)) != GSDPA_OK) return st;
    if (!K || !V || !lens) return GSDPA_ERR_INVALID_ARG;
    const long long row = (long long)cache->H_kv * cache->d_k;
    if (ld_k < row || ld_v < row) return GSDPA_ERR_INVALID_ARG;
    if (!aligned(K, 16) || !aligned(V, 16) || ld_k % 8 != 0 || ld_v % 8 != 0) return GSDPA_ERR_ALIGNMENT;
    if (!aligned(lens, 4) || !aligned(n_new, 4)) return GSDPA_ERR_ALIGNMENT;
    // blocks a sequence's new tokens can touch; no more than the cache has
    long long touched = ((long long)L + kCacheBlock - 2) / kCacheBlock + 1;
    const int blocks = cache->capacity / kCacheBlock;
    if (touched > blocks) touched = blocks;
    const long long grid = (long long)cache->B * cache->H_kv * touched;
    if (grid > 0x7fffffffLL) return GSDPA_ERR_UNSUPPORTED;
    Runtime rt;
    int major = 0, minor = 0;
    if (!current_runtime(&rt, &major, &minor)) return GSDPA_ERR_LAUNCH;
    if (!(major == 10 && minor == 3)) return GSDPA_ERR_UNSUPPORTED;
    AppendArgs a;
    a.K = static_cast<const __nv_bfloat16*>(K);
    a.V = static_cast<const __nv_bfloat16*>(V);
    a.ld_k = ld_k;
    a.ld_v = ld_v;
    a.lens = lens;
    a.n_new = n_new;
    a.k8 = static_cast<uint8_t*>(cache->k8);
    a.v8 = static_cast<uint8_t*>(cache->v8);
    a.k_scale = cache->k_scale;
    a.v_scale = cache->v_scale;
    a.k_tail = static_cast<__nv_bfloat16*>(cache->k_tail);
    a.v_tail = static_cast<__nv_bfloat16*>(cache->v_tail);
    a.L = L;
    a.Hkv = cache->H_kv;
    a.blocks = blocks;
    a.capacity = cache->capacity;
    a.touched = (int)touched;
    a.err = rt.err;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    const bool e4m3 = cache->kind == GSDPA_CACHE_E4M3, many = touched > 2 && grid > 4LL * rt.num_sms;
    if (cache->d_k == 128)
        e = e4m3 ? launch<128, true>(a, many, (unsigned)grid, s) : launch<128, false>(a, many, (unsigned)grid, s);
    else
        e = e4m3 ? launch<64, true>(a, many, (unsigned)grid, s) : launch<64, false>(a, many, (unsigned)grid, s);
    return e == cudaSuccess ? GSDPA_OK : GSDPA_ERR_LAUNCH;
}
