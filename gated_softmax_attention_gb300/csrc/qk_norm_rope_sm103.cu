// qk_norm_rope_sm103.cu -- the per-head RMS norm of queries and keys with the
// rotary positions in the same pass, forward and backward.
//
// For one head's row x [d_k] at position p (gamma = 1 when absent, y = x
// without the norm):
//     r = 1 / sqrt(mean_c x_c^2 + eps),          y_c = x_c r gamma_c
//     a = p w_i,  (y_a, y_b) -> t (y_a cos a - y_b sin a, y_b cos a + y_a sin a)
// for the rotary pairs i (columns (i, i + rd/2) or (2i, 2i + 1)); the columns
// past rd pass through. With A_c = gamma_c t cos a and B_c = -+ gamma_c' t sin a
// (c' the pair's other column) a row is z_c = r (x_c A_c + x_c' B_c), and A, B
// are the same for every head of a token. The backward, with dy the inverse
// rotation of dz, h = dy gamma and s = sum_c h_c x_c:
//     dx = r h - x (r^3 s / d_k),      dgamma_c = sum over rows of dy_c x_c r
//
// Bound by HBM: every element is read once and written once (the backward
// reads two), about 10 operations each. A warp takes a part of a token's heads,
// all of one tensor: it starts their loads, turns the position into its lanes'
// cosines and sines meanwhile, and finishes the rows from registers; nothing is
// shared between warps. d_k / 8 lanes have a row, each 4 columns and the 4 that they are
// rotated with (half layout: two 8-byte pieces of a bf16 row, rotary_dim / 2
// columns apart; else 16 bytes in one), so the rotation needs no exchange
// between lanes, only the norm's sums do.
//
// Angles: a position times a frequency in float32 is off by 0.06 rad at
// position 10^6, and FP64 arithmetic is slow here. The frequency is kept as a
// 64-bit fraction of a whole turn per position instead; the low 64 bits of
// position * fraction are the angle modulo one turn, exact but for the
// fraction's own rounding (position * 2^-63 turns), and its upper 32 bits go
// to sincospif for float32, to the hardware's sine and cosine (2^-20.9
// absolute) for bf16, which rounds at 2^-9. Everything after that is float32, rounded
// once at the store.
//
// Measured: 32/4 heads of 128, 4096 tokens 12.6 us (6.0 TB/s, 88 % of a plain copy),
// one token of 64 sequences 1.9 us; backward, 16/2 heads, 32768 tokens 74 us (6.1
// TB/s), 16/16 heads, 2 x 2048 tokens 22 us.
#include "landing.cuh"
#include "ops_internal.h"

#include <cmath>
#include <type_traits>

namespace gsdpa {
namespace {

constexpr int kThreads = 128;     // (256: 32/4 heads L4096 14.6 instead of 13.5 us)
constexpr int kWarps = kThreads / 32;
constexpr int kSumThreads = 256, kSumBatch = 20;
constexpr int kMaxPairs = 64;
constexpr int kRing = 3;          // backward: tasks whose rows a warp has in shared memory or on the way
constexpr int kBwdCtasPerSm = 4;  // ... 4 CTAs of 48 KB

struct RopeArgs {
    const void *Q, *K;            // forward: inputs; backward: the forward's inputs (null without the norm)
    const void *dQ, *dK;          // backward: gradients of the outputs
    void *Qo, *Ko;                // forward: outputs; backward: gradients of the inputs
    const void *gamma_q, *gamma_k;
    const int* positions;         // [B, L] or null: 0 .. L - 1
    float* part;                  // backward: [CTAs][2][d_k] shares of dgamma
    long long ld_q, ld_k, ld_dq, ld_dk, ld_qo, ld_ko;
    int L, Hq, Hkv;
    int q_parts, k_parts;         // parts of a token's heads
    unsigned tokens, tasks;       // B * L; tokens * (q_parts + k_parts)
    int lg_split;                 // backward: warps that share a token's parts, 2^lg_split
    float eps;
    int rd;                       // rotated columns (0: none)
    float attn_scale;
    WaitCtl ctl;
    alignas(16) unsigned long long turn[kMaxPairs];
};

// 8 elements of a row in one lane: 4 at p and 4 at q.
template <typename T, bool HALF>
struct Raw;
template <bool HALF>
struct Raw<__nv_bfloat16, HALF> {
    uint4 v;
    __device__ __forceinline__ void load(const __nv_bfloat16* p, const __nv_bfloat16* q) {
        if constexpr (HALF) {
            const uint2 a = *reinterpret_cast<const uint2*>(p), b = *reinterpret_cast<const uint2*>(q);
            v = make_uint4(a.x, a.y, b.x, b.y);
        } else {
            v = *reinterpret_cast<const uint4*>(p);
        }
    }
    __device__ __forceinline__ void zero() { v = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void unpack(float2 (&f)[4]) const {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int k = 0; k < 4; ++k)
            f[k] = make_float2(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xffff0000u));
    }
    static __device__ __forceinline__ void store(__nv_bfloat16* p, __nv_bfloat16* q, const float2 (&f)[4]) {
        const uint2 a = make_uint2(pack_bf16x2(f[0].x, f[0].y), pack_bf16x2(f[1].x, f[1].y));
        const uint2 b = make_uint2(pack_bf16x2(f[2].x, f[2].y), pack_bf16x2(f[3].x, f[3].y));
        if constexpr (HALF) {
            *reinterpret_cast<uint2*>(p) = a;
            *reinterpret_cast<uint2*>(q) = b;
        } else {
            *reinterpret_cast<uint4*>(p) = make_uint4(a.x, a.y, b.x, b.y);
        }
    }
};
template <bool HALF>
struct Raw<float, HALF> {
    float4 a, b;
    __device__ __forceinline__ void load(const float* p, const float* q) {
        a = *reinterpret_cast<const float4*>(p);
        b = *reinterpret_cast<const float4*>(q);
    }
    __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ void unpack(float2 (&f)[4]) const {
        f[0] = make_float2(a.x, a.y);
        f[1] = make_float2(a.z, a.w);
        f[2] = make_float2(b.x, b.y);
        f[3] = make_float2(b.z, b.w);
    }
    static __device__ __forceinline__ void store(float* p, float* q, const float2 (&f)[4]) {
        *reinterpret_cast<float4*>(p) = make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
        *reinterpret_cast<float4*>(q) = make_float4(f[2].x, f[2].y, f[3].x, f[3].y);
    }
};

// The sums over a row's lanes of N values (1, 2 or 4) at once, every lane's v
// becoming the totals through f: lanes exchange halves of the values while there
// are some to give away, so that each ends with one total, applies f to it, and
// hands it round (for 4 values and 16 lanes 9 shuffles instead of 16, and f once).
template <int LANES, int N, typename F>
__device__ __forceinline__ void row_sums(float (&v)[N], int lane, F f) {
    float t[N];
#pragma unroll
    for (int k = 0; k < N; ++k) t[k] = v[k];
    int sh = LANES / 2;
#pragma unroll
    for (int n = N; n > 1; n >>= 1, sh >>= 1) {
        const bool upper = lane & sh;
#pragma unroll
        for (int k = 0; k < n / 2; ++k) {
            const float keep = upper ? t[k + n / 2] : t[k], give = upper ? t[k] : t[k + n / 2];
            t[k] = keep + __shfl_xor_sync(0xffffffffu, give, sh);
        }
    }
#pragma unroll
    for (; sh > 0; sh >>= 1) t[0] += __shfl_xor_sync(0xffffffffu, t[0], sh);
    const float mine = f(t[0]);
    if constexpr (N == 1) {
        v[0] = mine;
    } else {
        // value k's total is in the lanes whose upper bits spell k
        const int base = lane & ~(LANES - 1);
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] = __shfl_sync(0xffffffffu, mine, base + k * (LANES / N));
    }
}

__device__ __forceinline__ float dot2(const float2 (&a)[4], const float2 (&b)[4]) {
    float2 s = __fmul2_rn(a[0], b[0]);
#pragma unroll
    for (int k = 1; k < 4; ++k) s = __ffma2_rn(a[k], b[k], s);
    return s.x + s.y;
}

// Scaled cosines and sines of a lane's four pairs.
struct Trig {
    float c[4], s[4];
};
template <typename T>
__device__ __forceinline__ void angles(Trig& t, const RopeArgs& a, long long pos, int first_pair, bool rotated) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        t.c[k] = 1.f;
        t.s[k] = 0.f;
    }
    if (!rotated) return;
    // (a load from the parameters' generic address: indexed by the lane, constant memory would answer
    // one lane after another)
    unsigned long long turn[4];
#pragma unroll
    for (int k = 0; k < 4; k += 2)
        asm("ld.v2.u64 {%0, %1}, [%2];" : "=l"(turn[k]), "=l"(turn[k + 1]) : "l"(a.turn + first_pair + k));
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const unsigned long long at = (unsigned long long)pos * turn[k];
        const float x = (float)(int)(at >> 32);   // 2^-32 turns, within half a turn
        float sn, cs;
        if constexpr (std::is_same<T, float>::value) {
            sincospif(x * 4.656612873077393e-10f, &sn, &cs);
        } else {
            const float w = x * 1.4629180792671596e-09f;   // 2 pi 2^-32
            sn = __sinf(w);
            cs = __cosf(w);
        }
        t.c[k] = cs * a.attn_scale;
        t.s[k] = sn * a.attn_scale;
    }
}

// The pairs (y_a, y_b) of a lane turned: forward by the angle, back by its
// negative. Half layout: pair k is elements k and 4 + k; else 2 k and 2 k + 1.
template <bool HALF, bool BACK>
__device__ __forceinline__ void turn_pairs(float2 (&y)[4], const Trig& t) {
    float s[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) s[k] = BACK ? -t.s[k] : t.s[k];
    if constexpr (HALF) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const float2 u = y[k], v = y[2 + k];
            const float2 c2 = make_float2(t.c[2 * k], t.c[2 * k + 1]), s2 = make_float2(s[2 * k], s[2 * k + 1]);
            const float2 n2 = make_float2(-s2.x, -s2.y);
            y[k] = __ffma2_rn(v, n2, __fmul2_rn(u, c2));
            y[2 + k] = __ffma2_rn(u, s2, __fmul2_rn(v, c2));
        }
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float2 u = y[k];
            y[k] = make_float2(fmaf(-u.y, s[k], u.x * t.c[k]), fmaf(u.x, s[k], u.y * t.c[k]));
        }
    }
}

// Steps of ROWS rows to a part, all under way at once: 2 KB of rows.
template <typename T>
__host__ __device__ constexpr int part_steps() {
    return sizeof(T) == 2 ? 4 : 2;
}
constexpr int kPartBytes = 2048;

// A warp's task: a token and a part of its Q or K heads.
struct Task {
    unsigned tok;
    bool is_q;
    int h0, rows;       // first head, heads (at most part_steps * ROWS)
    long long at;       // of the first head in the token's row
    template <int ROWS, int D>
    __device__ __forceinline__ void set(const RopeArgs& a, unsigned task, int steps) {
        const unsigned parts = a.q_parts + a.k_parts;
        tok = task / parts;
        const int part = (int)(task - tok * parts);
        is_q = part < a.q_parts;
        h0 = (is_q ? part : part - a.q_parts) * steps * ROWS;
        rows = min(steps * ROWS, (is_q ? a.Hq : a.Hkv) - h0);
        at = (long long)h0 * D;
    }
};

__device__ __forceinline__ long long position(const RopeArgs& a, unsigned tok) {
    return a.positions ? (long long)a.positions[tok] : (long long)(tok % (unsigned)a.L);
}

// The lane's columns of a row, and what it multiplies them by.
template <typename T, int D, bool HALF>
struct Lane {
    int lane, j, slot, col0, col1;
    bool rotated;
    __device__ __forceinline__ explicit Lane(const RopeArgs& a) {
        lane = threadIdx.x % 32;
        j = lane % (D / 8);
        slot = lane / (D / 8);
        rotated = 8 * j < a.rd;
        col0 = HALF && rotated ? 4 * j : 8 * j;
        col1 = HALF && rotated ? (a.rd >> 1) + 4 * j : 8 * j + 4;
    }
    __device__ __forceinline__ void gamma(const void* p, float2 (&g)[4]) const {
        if (p) {
            Raw<T, HALF> r;
            r.load(static_cast<const T*>(p) + col0, static_cast<const T*>(p) + col1);
            r.unpack(g);
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) g[k] = make_float2(1.f, 1.f);
        }
    }
};

// The forward: short warps, a task each, that hide one another's loads.
template <typename T, int D, bool NORM, bool HALF>
__global__ void __launch_bounds__(kThreads) qk_norm_rope_kernel(const __grid_constant__ RopeArgs a) {
    constexpr int LANES = D / 8, ROWS = 32 / LANES, U = part_steps<T>();
    const unsigned task = blockIdx.x * kWarps + threadIdx.x / 32;
    const Lane<T, D, HALF> ln(a);
    pdl_wait();   // the inputs may be the previous kernel's outputs
    pdl_trigger();
    if (task >= a.tasks) return;
    Task w = {};
    w.set<ROWS, D>(a, task, U);
    const T* x = static_cast<const T*>(w.is_q ? a.Q : a.K) + w.tok * (w.is_q ? a.ld_q : a.ld_k) + w.at + ln.slot * D;
    T* o = static_cast<T*>(w.is_q ? a.Qo : a.Ko) + w.tok * (w.is_q ? a.ld_qo : a.ld_ko) + w.at + ln.slot * D;
    Raw<T, HALF> rx[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        rx[u].zero();
        if (u * ROWS + ln.slot < w.rows) rx[u].load(x + u * ROWS * D + ln.col0, x + u * ROWS * D + ln.col1);
    }
    float2 g[4];
    if constexpr (NORM) ln.gamma(w.is_q ? a.gamma_q : a.gamma_k, g);
    Trig t;
    angles<T>(t, a, position(a, w.tok), 4 * ln.j, ln.rotated);
    float r[U];
    if constexpr (NORM) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float2 v[4];
            rx[u].unpack(v);
            r[u] = dot2(v, v);
        }
        row_sums<LANES, U>(r, ln.lane, [&](float ss) { return rsqrtf(ss * (1.f / D) + a.eps); });
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (u * ROWS >= w.rows) break;   // (the whole warp)
        float2 y[4];
        rx[u].unpack(y);
        if constexpr (NORM) {
            const float2 r2 = make_float2(r[u], r[u]);
#pragma unroll
            for (int k = 0; k < 4; ++k) y[k] = __fmul2_rn(__fmul2_rn(y[k], r2), g[k]);
        }
        turn_pairs<HALF, false>(y, t);
        if (u * ROWS + ln.slot < w.rows)
            Raw<T, HALF>::store(o + u * ROWS * D + ln.col0, o + u * ROWS * D + ln.col1, y);
    }
}

// The backward: warps that stay (each CTA leaves a share of dgamma) and walk over
// tokens, part by part, every warp with a ring of its own that asynchronous copies
// keep filled with the rows of its next parts. It is bound by the instructions it issues,
// so what does not change with the row is done once for the token.
template <typename T, int D, bool NORM, bool HALF>
__global__ void __launch_bounds__(kThreads, 4) qk_norm_rope_bwd_kernel(const __grid_constant__ RopeArgs a) {
    constexpr int LANES = D / 8, ROWS = 32 / LANES, U = part_steps<T>();
    constexpr int SLOT = (NORM ? 2 : 1) * kPartBytes;   // dz, and x with the norm
    static_assert(U * ROWS * D * sizeof(T) == kPartBytes, "a part fills its half of a slot");
    extern __shared__ __align__(128) uint8_t smem[];   // [warps][kRing][SLOT]
    __shared__ uint64_t full[kWarps][kRing];
    __shared__ int abort_flags[kWarps];
    __shared__ float2 share[NORM ? kWarps : 1][2][D / 2];
    const int warp = threadIdx.x / 32;
    const Lane<T, D, HALF> ln(a);
    uint8_t* ring = smem + warp * kRing * SLOT;
    if (ln.lane == 0) {
        for (int k = 0; k < kRing; ++k) mbar_init(&full[warp][k], 1);
        abort_flags[warp] = 0;
        mbar_fence_init();
    }
    __syncwarp();
    pdl_wait();   // the inputs may be the previous kernel's outputs
    pdl_trigger();

    // the warp's tokens and, of each, its parts: every a.split-th
    const unsigned gw = blockIdx.x * kWarps + warp, stride = (gridDim.x * kWarps) >> a.lg_split;
    const unsigned tok0 = gw >> a.lg_split;
    const int part0 = gw & ((1 << a.lg_split) - 1), step = 1 << a.lg_split, parts = a.q_parts + a.k_parts;
    // the next part's copies (lane 0), and the place after it
    unsigned next_tok = tok0;
    int next_part = part0;
    uint32_t fetched[kRing] = {};   // how often each slot was filled
    const auto fetch = [&](int slot) {
#pragma unroll
        for (int k = 0; k < kRing; ++k) fetched[k] += k == slot ? 1 : 0;
        const bool is_q = next_part < a.q_parts;
        const int h0 = (is_q ? next_part : next_part - a.q_parts) * U * ROWS;
        const uint32_t bytes = min(U * ROWS, (is_q ? a.Hq : a.Hkv) - h0) * D * sizeof(T);
        const long long at = (long long)h0 * D;
        uint8_t* to = ring + slot * SLOT;
        mbar_arrive_expect_tx(&full[warp][slot], NORM ? 2 * bytes : bytes);
        bulk_load(to, static_cast<const T*>(is_q ? a.dQ : a.dK) + next_tok * (is_q ? a.ld_dq : a.ld_dk) + at, bytes,
                  &full[warp][slot]);
        if constexpr (NORM)
            bulk_load(to + kPartBytes, static_cast<const T*>(is_q ? a.Q : a.K) + next_tok * (is_q ? a.ld_q : a.ld_k) + at,
                      bytes, &full[warp][slot]);
        next_part += step;
        if (next_part >= parts) {
            next_part = part0;
            next_tok += stride;   // (no overflow: tokens and warps are below 2^30)
        }
    };
    if (ln.lane == 0)
        for (int k = 0; k < kRing; ++k)
            if (next_tok < a.tokens) fetch(k);
    float2 gq[4], gk[4], dgq[4], dgk[4];
    if constexpr (NORM) {
        ln.gamma(a.gamma_q, gq);
        ln.gamma(a.gamma_k, gk);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) dgq[k] = dgk[k] = make_float2(0.f, 0.f);
    int slot = 0;
    uint32_t phase = 0;
    bool ok = true;
    Trig t;
    // a part's rows from the slot, and their gradients to o
    const auto part_rows = [&](const float2 (&g)[4], float2 (&dg)[4], T* o, int rows) {
        const T* z = reinterpret_cast<const T*>(ring + slot * SLOT) + ln.slot * D;
        const T* x = z + kPartBytes / sizeof(T);
#pragma unroll
        for (int u0 = 0; u0 < U; u0 += 2) {   // two steps' sums at once
            if (u0 * ROWS >= rows) break;     // (the whole warp)
            float2 dy[2][4], xs[2][4];
            float v[4];                       // sums of x^2 and of h x, of each step
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const bool in = (u0 + k) * ROWS + ln.slot < rows;
                const int off = (u0 + k) * ROWS * D;
                Raw<T, HALF> r;
                r.zero();   // (a slot's bytes past the part's rows are an earlier part's)
                if (in) r.load(z + off + ln.col0, z + off + ln.col1);
                r.unpack(dy[k]);
                turn_pairs<HALF, true>(dy[k], t);
                if constexpr (NORM) {
                    r.zero();
                    if (in) r.load(x + off + ln.col0, x + off + ln.col1);
                    r.unpack(xs[k]);
                    float2 hh[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) hh[e] = __fmul2_rn(dy[k][e], g[e]);
                    v[2 * k] = dot2(xs[k], xs[k]);
                    v[2 * k + 1] = dot2(hh, xs[k]);
                }
            }
            if constexpr (NORM) row_sums<LANES, 4>(v, ln.lane, [](float s) { return s * (1.f / D); });
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const bool in = (u0 + k) * ROWS + ln.slot < rows;
                if constexpr (NORM) {
                    // r (h - xh mean(h xh)), xh = x r (rows past the last head are all zeros: r = 0 for eps = 0)
                    const float r = in ? rsqrtf(v[2 * k] + a.eps) : 0.f;
                    const float m = -(v[2 * k + 1] * r);
                    const float2 r2 = make_float2(r, r), m2 = make_float2(m, m);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 xh = __fmul2_rn(xs[k][e], r2);
                        dg[e] = __ffma2_rn(dy[k][e], xh, dg[e]);
                        dy[k][e] = __fmul2_rn(__ffma2_rn(xh, m2, __fmul2_rn(dy[k][e], g[e])), r2);
                    }
                }
                if (in) {
                    T* to = o + (u0 + k) * ROWS * D;
                    Raw<T, HALF>::store(to + ln.col0, to + ln.col1, dy[k]);
                }
            }
        }
    };
    long long pos = tok0 < a.tokens ? position(a, tok0) : 0;
    for (unsigned tok = tok0; ok && tok < a.tokens && part0 < parts; tok += stride) {
        angles<T>(t, a, pos, 4 * ln.j, ln.rotated);
        if (tok + stride < a.tokens) pos = position(a, tok + stride);
        for (int part = part0; part < parts; part += step) {
            ok = __all_sync(0xffffffffu, mbar_wait(&full[warp][slot], phase, &abort_flags[warp], a.ctl));
            if (!ok) break;
            if (part < a.q_parts) {
                const int h0 = part * U * ROWS;
                part_rows(gq, dgq, static_cast<T*>(a.Qo) + tok * a.ld_qo + (h0 + ln.slot) * D, a.Hq - h0);
            } else {
                const int h0 = (part - a.q_parts) * U * ROWS;
                part_rows(gk, dgk, static_cast<T*>(a.Ko) + tok * a.ld_ko + (h0 + ln.slot) * D, a.Hkv - h0);
            }
            __syncwarp();   // every lane has read the slot
            if (ln.lane == 0 && next_tok < a.tokens) fetch(slot);
            if (++slot == kRing) {
                slot = 0;
                phase ^= 1u;
            }
        }
    }
    if (!ok && ln.lane == 0) {
        // let copies in flight land before the CTA exits
        volatile int never = 0;
        const WaitCtl c2 = landing_limit(a.ctl);
#pragma unroll
        for (int k = 0; k < kRing; ++k)
            if (fetched[k] > 0) mbar_wait(&full[warp][k], (fetched[k] - 1) & 1u, &never, c2);
    }
    __syncwarp();
    if constexpr (NORM) {
        // the CTA's share of dgamma: a warp's rows, then the warps, in a fixed order
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            float2(&dg)[4] = q == 0 ? dgq : dgk;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
#pragma unroll
                for (int sh = 16; sh >= LANES; sh >>= 1) {
                    dg[k].x += __shfl_xor_sync(0xffffffffu, dg[k].x, sh);
                    dg[k].y += __shfl_xor_sync(0xffffffffu, dg[k].y, sh);
                }
            }
            if (ln.slot == 0) {
                share[warp][q][ln.col0 / 2] = dg[0];
                share[warp][q][ln.col0 / 2 + 1] = dg[1];
                share[warp][q][ln.col1 / 2] = dg[2];
                share[warp][q][ln.col1 / 2 + 1] = dg[3];
            }
        }
        __syncthreads();
        const float* flat = reinterpret_cast<const float*>(share);
        for (int i = threadIdx.x; i < 2 * D; i += kThreads) {
            float s = 0.f;
#pragma unroll
            for (int k = 0; k < kWarps; ++k) s += flat[k * 2 * D + i];
            a.part[(long long)blockIdx.x * 2 * D + i] = s;
        }
    }
}

// dgamma[c] = the CTAs' shares added up, always in the same order: 8 columns
// to a CTA, 32 threads to a column, whose loads are under way together (one after
// the other 16/16 heads L2048 took 2 us more).
template <typename T>
__global__ void __launch_bounds__(kSumThreads) dgamma_kernel(const float* __restrict__ part, int parts, int d, T* dgq,
                                                          T* dgk) {
    __shared__ float red[32][8];
    pdl_wait();
    pdl_trigger();
    const int col = blockIdx.x * 8 + (threadIdx.x & 7), row = threadIdx.x >> 3;
    float t = 0.f;
    for (int i = row; i < parts; i += 32 * kSumBatch) {
        float v[kSumBatch];
#pragma unroll
        for (int k = 0; k < kSumBatch; ++k) v[k] = i + 32 * k < parts ? part[(long long)(i + 32 * k) * 2 * d + col] : 0.f;
#pragma unroll
        for (int k = 0; k < kSumBatch; ++k) t += v[k];
    }
    red[row][threadIdx.x & 7] = t;
    __syncthreads();
    if (threadIdx.x < 8) {
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < 32; ++i) sum += red[i][threadIdx.x];
        T* to = col < d ? dgq : dgk;   // (a CTA's 8 columns are of one tensor: d is a multiple of 8)
        if (to) {
            if constexpr (std::is_same<T, float>::value) to[col % d] = sum;
            else to[col % d] = __float2bfloat16_rn(sum);
        }
    }
}

// CTAs of the backward: each leaves one share of dgamma, so they stay for
// several tasks, as many CTAs as fit on the SMs at once.
long long bwd_ctas(long long tasks, int sms) {
    const long long need = (tasks + kWarps - 1) / kWarps, most = kBwdCtasPerSm * (sms < plan_sms() ? sms : plan_sms());
    return need < most ? need : most;
}

bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

// The checks that forward and backward share.
int validate(int B, int L, int Hq, int Hkv, int dk, int norm, float eps, const gsdpa_rope* rope, int dtype,
             const void* gamma_q, const void* gamma_k, const int* positions) {
    if (B < 0 || L < 0 || Hq < 1 || Hkv < 1) return GSDPA_ERR_INVALID_ARG;
    if (dtype != GSDPA_F32 && dtype != GSDPA_BF16) return GSDPA_ERR_INVALID_ARG;
    if (norm != 0 && norm != 1) return GSDPA_ERR_INVALID_ARG;
    if (norm && !(eps >= 0.f && eps < INFINITY)) return GSDPA_ERR_INVALID_ARG;
    if (!norm && (gamma_q || gamma_k)) return GSDPA_ERR_INVALID_ARG;
    if (dk != 64 && dk != 128) return GSDPA_ERR_UNSUPPORTED;
    if (rope) {
        if (rope->rotary_dim < 16 || rope->rotary_dim % 16 != 0 || rope->rotary_dim > dk) return GSDPA_ERR_INVALID_ARG;
        if (rope->layout != GSDPA_ROPE_HALF && rope->layout != GSDPA_ROPE_INTERLEAVED) return GSDPA_ERR_INVALID_ARG;
        if (!std::isfinite(rope->attn_scale)) return GSDPA_ERR_INVALID_ARG;
    }
    if (!aligned(gamma_q, 16) || !aligned(gamma_k, 16) || !aligned(positions, 4)) return GSDPA_ERR_ALIGNMENT;
    if ((long long)B * L > 0x7fffffffLL || (long long)Hq * dk > 0x7fffffffLL || (long long)Hkv * dk > 0x7fffffffLL)
        return GSDPA_ERR_UNSUPPORTED;
    return GSDPA_OK;
}

// One strided tensor [tokens] x [H * d_k]: rows that do not overlap and start on 16 bytes.
int check_rows(const void* p, long long ld, int H, int dk, int dtype) {
    if (!p) return GSDPA_ERR_INVALID_ARG;
    if (ld < (long long)H * dk) return GSDPA_ERR_INVALID_ARG;
    if (!aligned(p, 16) || ld % (dtype == GSDPA_BF16 ? 8 : 4) != 0) return GSDPA_ERR_ALIGNMENT;
    return GSDPA_OK;
}

// What forward and backward share of the launch.
int set_problem(RopeArgs& a, int steps, int B, int L, int Hq, int Hkv, int dk, float eps, const gsdpa_rope* rope,
                const int* positions, const void* gamma_q, const void* gamma_k) {
    a.positions = positions;
    a.gamma_q = gamma_q;
    a.gamma_k = gamma_k;
    a.L = L;
    a.Hq = Hq;
    a.Hkv = Hkv;
    const int rows = 32 / (dk / 8) * steps;
    a.q_parts = (Hq + rows - 1) / rows;
    a.k_parts = (Hkv + rows - 1) / rows;
    const long long tasks = (long long)B * L * (a.q_parts + a.k_parts);
    if (tasks > 0x7fffffffLL || (long long)B * L >= 1 << 30) return GSDPA_ERR_UNSUPPORTED;
    a.tokens = (unsigned)(B * L);
    a.tasks = (unsigned)tasks;
    // (backward) a warp to a token, or up to four while the warps would have less than two
    // tokens each (16/16 heads: 2 x 2048 tokens 23.7 -> 21.8 us; four tokens each 22.9)
    while (a.lg_split < 2 && (2 << a.lg_split) <= a.q_parts + a.k_parts &&
           ((long long)a.tokens << a.lg_split) < 2LL * kWarps * kBwdCtasPerSm * plan_sms())
        ++a.lg_split;
    a.eps = eps;
    a.attn_scale = 1.f;
    if (!rope) return GSDPA_OK;
    a.rd = rope->rotary_dim;
    a.attn_scale = rope->attn_scale;
    for (int i = 0; i < a.rd / 2; ++i) a.turn[i] = rope->turn[i];
    return GSDPA_OK;
}

template <typename T, int D, bool NORM, bool HALF>
cudaError_t launch_n(const RopeArgs& a, bool bwd, unsigned grid, cudaStream_t s) {
    if (!bwd) return launch_dependent(qk_norm_rope_kernel<T, D, NORM, HALF>, dim3(grid), dim3(kThreads), 0, s, a);
    constexpr int bytes = kWarps * kRing * (NORM ? 2 : 1) * kPartBytes;
    static PerDeviceSetup setup;
    const cudaError_t e = setup_once_per_device(setup, [](int&) {
        return cudaFuncSetAttribute(qk_norm_rope_bwd_kernel<T, D, NORM, HALF>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    bytes);
    });
    if (e != cudaSuccess) return e;
    return launch_dependent(qk_norm_rope_bwd_kernel<T, D, NORM, HALF>, dim3(grid), dim3(kThreads), bytes, s, a);
}
template <typename T, int D>
cudaError_t launch_t(const RopeArgs& a, bool bwd, bool norm, bool half, unsigned grid, cudaStream_t s) {
    if (norm) return half ? launch_n<T, D, true, true>(a, bwd, grid, s) : launch_n<T, D, true, false>(a, bwd, grid, s);
    return half ? launch_n<T, D, false, true>(a, bwd, grid, s) : launch_n<T, D, false, false>(a, bwd, grid, s);
}
cudaError_t launch(const RopeArgs& a, bool bwd, bool norm, const gsdpa_rope* rope, int dk, int dtype, unsigned grid,
                   cudaStream_t s) {
    const bool half = rope && rope->layout == GSDPA_ROPE_HALF;   // (no rotation: the columns in order)
    if (dtype == GSDPA_BF16)
        return dk == 128 ? launch_t<__nv_bfloat16, 128>(a, bwd, norm, half, grid, s)
                         : launch_t<__nv_bfloat16, 64>(a, bwd, norm, half, grid, s);
    return dk == 128 ? launch_t<float, 128>(a, bwd, norm, half, grid, s) : launch_t<float, 64>(a, bwd, norm, half, grid, s);
}
template <typename T>
cudaError_t launch_dgamma(const float* part, int parts, int dk, void* dgq, void* dgk, cudaStream_t s) {
    return launch_dependent(dgamma_kernel<T>, dim3(2 * dk / 8), dim3(kSumThreads), 0, s, part, parts, dk, static_cast<T*>(dgq),
                            static_cast<T*>(dgk));
}

constexpr double kTwoPi = 6.283185307179586, kTwoPiRest = 2.4492935982947064e-16;

// Turns modulo one, times 2^64: positions are whole numbers, so whole turns drop out.
unsigned long long part_of_turn(double turns) {
    const double scaled = std::ldexp(turns - std::rint(turns), 64);   // (the difference is exact)
    return scaled >= 9223372036854775808.0 ? 1ull << 63 : (unsigned long long)(long long)std::rint(scaled);
}

}  // namespace
}  // namespace gsdpa

using namespace gsdpa;

extern "C" {

int gsdpa_rope_init_freqs(gsdpa_rope* rope, int rotary_dim, int layout, const double* inv_freq, double attn_scale) {
    if (!rope || !inv_freq) return GSDPA_ERR_INVALID_ARG;
    if (rotary_dim < 16 || rotary_dim > 2 * kMaxPairs || rotary_dim % 16 != 0) return GSDPA_ERR_INVALID_ARG;
    if (layout != GSDPA_ROPE_HALF && layout != GSDPA_ROPE_INTERLEAVED) return GSDPA_ERR_INVALID_ARG;
    if (!std::isfinite(attn_scale)) return GSDPA_ERR_INVALID_ARG;
    for (int i = 0; i < rotary_dim / 2; ++i)
        if (!std::isfinite(inv_freq[i])) return GSDPA_ERR_INVALID_ARG;
    rope->rotary_dim = rotary_dim;
    rope->layout = layout;
    rope->attn_scale = (float)attn_scale;
    rope->reserved = 0;
    for (int i = 0; i < kMaxPairs; ++i) rope->turn[i] = 0;
    for (int i = 0; i < rotary_dim / 2; ++i) {
        // turns per position, as a double and the rest of the quotient (2 pi in two doubles)
        const double q = inv_freq[i] / kTwoPi, rest = (std::fma(-q, kTwoPi, inv_freq[i]) - q * kTwoPiRest) / kTwoPi;
        rope->turn[i] = part_of_turn(q) + part_of_turn(rest);
    }
    return GSDPA_OK;
}

int gsdpa_rope_init(gsdpa_rope* rope, int rotary_dim, int layout, double theta, int scaling, double factor,
                    double orig_len, double beta_fast, double beta_slow, double attn_scale) {
    if (rotary_dim < 16 || rotary_dim > 2 * kMaxPairs || rotary_dim % 16 != 0) return GSDPA_ERR_INVALID_ARG;
    if (!(theta > 1.0) || !std::isfinite(theta) || !std::isfinite(attn_scale)) return GSDPA_ERR_INVALID_ARG;
    if (scaling < GSDPA_ROPE_PLAIN || scaling > GSDPA_ROPE_PARTS) return GSDPA_ERR_INVALID_ARG;
    if (scaling != GSDPA_ROPE_PLAIN && !(factor >= 1.0 && std::isfinite(factor))) return GSDPA_ERR_INVALID_ARG;
    const double rd = rotary_dim;
    double lo = 0.0, hi = 0.0;
    if (scaling == GSDPA_ROPE_PARTS) {
        if (!(orig_len >= 1.0 && std::isfinite(orig_len))) return GSDPA_ERR_INVALID_ARG;
        if (!(beta_slow > 0.0 && beta_fast >= beta_slow && std::isfinite(beta_fast))) return GSDPA_ERR_INVALID_ARG;
        const double k = 2.0 * std::log(theta);
        lo = std::floor(rd * std::log(orig_len / (beta_fast * kTwoPi)) / k);
        hi = std::ceil(rd * std::log(orig_len / (beta_slow * kTwoPi)) / k);
        lo = lo < 0.0 ? 0.0 : lo;
        hi = hi > rd - 1.0 ? rd - 1.0 : hi;
    }
    double w[kMaxPairs];
    for (int i = 0; i < rotary_dim / 2; ++i) {
        double base = theta;
        if (scaling == GSDPA_ROPE_BASE) base = theta * std::pow(factor, rd / (rd - 2.0));
        w[i] = std::pow(base, -2.0 * i / rd);
        if (scaling == GSDPA_ROPE_LINEAR) w[i] /= factor;
        if (scaling == GSDPA_ROPE_PARTS) {
            const double span = hi - lo > 1e-3 ? hi - lo : 1e-3;
            double u = (i - lo) / span;
            u = u < 0.0 ? 0.0 : (u > 1.0 ? 1.0 : u);
            w[i] = w[i] / factor * u + w[i] * (1.0 - u);
        }
    }
    double t = attn_scale;
    if (t == 0.0) t = scaling == GSDPA_ROPE_PARTS ? 0.1 * std::log(factor) + 1.0 : 1.0;
    return gsdpa_rope_init_freqs(rope, rotary_dim, layout, w, t);
}

int gsdpa_qk_norm_rope(const void* Q, const void* K, const void* gamma_q, const void* gamma_k, const int* positions,
                       void* Qo, void* Ko, long long ld_q, long long ld_k, long long ld_qo, long long ld_ko, int B,
                       int L, int H_q, int H_kv, int d_k, int norm, float eps, const gsdpa_rope* rope, int dtype,
                       void* stream) {
    int st = validate(B, L, H_q, H_kv, d_k, norm, eps, rope, dtype, gamma_q, gamma_k, positions);
    if (st != GSDPA_OK) return st;
    if (B == 0 || L == 0) return GSDPA_OK;
    if ((st = check_rows(Q, ld_q, H_q, d_k, dtype)) != GSDPA_OK) return st;
    if ((st = check_rows(K, ld_k, H_kv, d_k, dtype)) != GSDPA_OK) return st;
    if ((st = check_rows(Qo, ld_qo, H_q, d_k, dtype)) != GSDPA_OK) return st;
    if ((st = check_rows(Ko, ld_ko, H_kv, d_k, dtype)) != GSDPA_OK) return st;
    if ((Qo == Q && ld_qo != ld_q) || (Ko == K && ld_ko != ld_k)) return GSDPA_ERR_INVALID_ARG;   // in place
    Runtime rt;
    int major = 0, minor = 0;
    if (!current_runtime(&rt, &major, &minor)) return GSDPA_ERR_LAUNCH;
    if (!(major == 10 && minor == 3)) return GSDPA_ERR_UNSUPPORTED;
    RopeArgs a = {};
    a.Q = Q;
    a.K = K;
    a.Qo = Qo;
    a.Ko = Ko;
    a.ld_q = ld_q;
    a.ld_k = ld_k;
    a.ld_qo = ld_qo;
    a.ld_ko = ld_ko;
    st = set_problem(a, dtype == GSDPA_BF16 ? part_steps<__nv_bfloat16>() : part_steps<float>(), B, L, H_q, H_kv,
                     d_k, eps, rope, positions, gamma_q, gamma_k);
    if (st != GSDPA_OK) return st;
    const cudaError_t e = launch(a, false, norm != 0, rope, d_k, dtype, (a.tasks + kWarps - 1) / kWarps,
                                        static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? GSDPA_OK : GSDPA_ERR_LAUNCH;
}

size_t gsdpa_qk_norm_rope_bwd_workspace_bytes(int B, int L, int d_k, int norm) {
    if (B < 0 || L < 0 || (d_k != 64 && d_k != 128) || (norm != 0 && norm != 1) || (long long)B * L > 0x7fffffffLL)
        return (size_t)-1;
    if (!norm || B == 0 || L == 0) return 0;
    return (size_t)kBwdCtasPerSm * plan_sms() * 2 * d_k * sizeof(float);   // (the most CTAs there are)
}

int gsdpa_qk_norm_rope_bwd(const void* Q, const void* K, const void* gamma_q, const void* gamma_k,
                           const int* positions, const void* dQo, const void* dKo, void* dQ, void* dK, void* dgamma_q,
                           void* dgamma_k, long long ld_q, long long ld_k, long long ld_dqo, long long ld_dko,
                           long long ld_dq, long long ld_dk, int B, int L, int H_q, int H_kv, int d_k, int norm,
                           float eps, const gsdpa_rope* rope, int dtype, void* workspace, size_t workspace_bytes,
                           void* stream) {
    int st = validate(B, L, H_q, H_kv, d_k, norm, eps, rope, dtype, gamma_q, gamma_k, positions);
    if (st != GSDPA_OK) return st;
    if (!norm && (dgamma_q || dgamma_k)) return GSDPA_ERR_INVALID_ARG;
    if (!aligned(dgamma_q, 16) || !aligned(dgamma_k, 16)) return GSDPA_ERR_ALIGNMENT;
    if (B == 0 || L == 0) return GSDPA_OK;
    if (norm) {
        if ((st = check_rows(Q, ld_q, H_q, d_k, dtype)) != GSDPA_OK) return st;
        if ((st = check_rows(K, ld_k, H_kv, d_k, dtype)) != GSDPA_OK) return st;
    }
    if ((st = check_rows(dQo, ld_dqo, H_q, d_k, dtype)) != GSDPA_OK) return st;
    if ((st = check_rows(dKo, ld_dko, H_kv, d_k, dtype)) != GSDPA_OK) return st;
    if ((st = check_rows(dQ, ld_dq, H_q, d_k, dtype)) != GSDPA_OK) return st;
    if ((st = check_rows(dK, ld_dk, H_kv, d_k, dtype)) != GSDPA_OK) return st;
    if ((dQ == dQo && ld_dq != ld_dqo) || (dK == dKo && ld_dk != ld_dko)) return GSDPA_ERR_INVALID_ARG;
    Runtime rt;
    int major = 0, minor = 0;
    if (!current_runtime(&rt, &major, &minor)) return GSDPA_ERR_LAUNCH;
    if (!(major == 10 && minor == 3)) return GSDPA_ERR_UNSUPPORTED;
    const size_t need = gsdpa_qk_norm_rope_bwd_workspace_bytes(B, L, d_k, norm);
    if (need > 0) {
        if (!workspace || workspace_bytes < need) return GSDPA_ERR_WORKSPACE;
        if (!aligned(workspace, 256)) return GSDPA_ERR_ALIGNMENT;
    }
    RopeArgs a = {};
    a.Q = Q;
    a.K = K;
    a.dQ = dQo;
    a.dK = dKo;
    a.Qo = dQ;
    a.Ko = dK;
    a.part = static_cast<float*>(workspace);
    a.ld_q = ld_q;
    a.ld_k = ld_k;
    a.ld_dq = ld_dqo;
    a.ld_dk = ld_dko;
    a.ld_qo = ld_dq;
    a.ld_ko = ld_dk;
    st = set_problem(a, dtype == GSDPA_BF16 ? part_steps<__nv_bfloat16>() : part_steps<float>(), B, L, H_q, H_kv,
                     d_k, eps, rope, positions, gamma_q, gamma_k);
    if (st != GSDPA_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    a.ctl.err = rt.err;
    a.ctl.limit_ns = rt.limit_ns;
    const int ctas = (int)bwd_ctas(a.tasks, rt.num_sms);
    cudaError_t e = launch(a, true, norm != 0, rope, d_k, dtype, (unsigned)ctas, s);
    if (e == cudaSuccess && (dgamma_q || dgamma_k))
        e = dtype == GSDPA_BF16 ? launch_dgamma<__nv_bfloat16>(a.part, ctas, d_k, dgamma_q, dgamma_k, s)
                                : launch_dgamma<float>(a.part, ctas, d_k, dgamma_q, dgamma_k, s);
    return e == cudaSuccess ? GSDPA_OK : GSDPA_ERR_LAUNCH;
}

}  // extern "C"
