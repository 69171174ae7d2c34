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
// reads two), about 10 operations each. A warp takes one token: it turns the
// position into the token's cosines and sines once, in shared memory, keeps
// A, B in registers and walks over the token's heads, d_k / 8 lanes to a row,
// 8 elements (one 16-byte load in bf16) to a lane, the pair's other column
// from a shuffle.
//
// Angles: a position times a frequency in float32 is off by 0.06 rad at
// position 10^6, and FP64 arithmetic is slow here. The frequency is kept as a
// 64-bit fraction of a whole turn per position instead; the low 64 bits of
// position * fraction are the angle modulo one turn, exact but for the
// fraction's own rounding (position * 2^-54 turns), and its upper 32 bits go
// to sincospif. Everything after that is float32, rounded once at the store.
#include "gsdpa.h"
#include "gsdpa_internal.h"
#include "sm103_ptx.cuh"

#include <cmath>
#include <type_traits>

namespace gsdpa {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxPairs = 64;

struct RopeArgs {
    const void *Q, *K;            // forward: inputs; backward: the forward's inputs (null without the norm)
    const void *dQ, *dK;          // backward: gradients of the outputs
    void *Qo, *Ko;                // forward: outputs; backward: gradients of the inputs
    const void *gamma_q, *gamma_k;
    const int* positions;         // [B, L] or null: 0 .. L - 1
    float* part;                  // backward: [CTAs][2][d_k] shares of dgamma
    long long ld_q, ld_k, ld_dq, ld_dk, ld_qo, ld_ko;
    long long tokens;             // B * L
    int L, Hq, Hkv;
    int wpt;                      // warps per token (1, 2, 4 or 8)
    float eps;
    int rd;                       // rotated columns (0: none)
    int interleaved;
    float attn_scale;
    unsigned long long turn[kMaxPairs];
};

// 8 elements of a row in one lane
template <typename T>
struct Raw;
template <>
struct Raw<__nv_bfloat16> {
    uint4 v;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ void zero() { v = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void unpack(float2 (&f)[4]) const {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int k = 0; k < 4; ++k)
            f[k] = make_float2(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xffff0000u));
    }
    __device__ __forceinline__ Raw from_lane(int src) const {
        Raw o;
        o.v.x = __shfl_sync(0xffffffffu, v.x, src);
        o.v.y = __shfl_sync(0xffffffffu, v.y, src);
        o.v.z = __shfl_sync(0xffffffffu, v.z, src);
        o.v.w = __shfl_sync(0xffffffffu, v.w, src);
        return o;
    }
    static __device__ __forceinline__ void store(__nv_bfloat16* p, const float2 (&f)[4]) {
        *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(f[0].x, f[0].y), pack_bf16x2(f[1].x, f[1].y),
                                                  pack_bf16x2(f[2].x, f[2].y), pack_bf16x2(f[3].x, f[3].y));
    }
};
template <>
struct Raw<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float* p) {
        a = *reinterpret_cast<const float4*>(p);
        b = *reinterpret_cast<const float4*>(p + 4);
    }
    __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ void unpack(float2 (&f)[4]) const {
        f[0] = make_float2(a.x, a.y);
        f[1] = make_float2(a.z, a.w);
        f[2] = make_float2(b.x, b.y);
        f[3] = make_float2(b.z, b.w);
    }
    __device__ __forceinline__ Raw from_lane(int src) const {
        Raw o;
        o.a.x = __shfl_sync(0xffffffffu, a.x, src);
        o.a.y = __shfl_sync(0xffffffffu, a.y, src);
        o.a.z = __shfl_sync(0xffffffffu, a.z, src);
        o.a.w = __shfl_sync(0xffffffffu, a.w, src);
        o.b.x = __shfl_sync(0xffffffffu, b.x, src);
        o.b.y = __shfl_sync(0xffffffffu, b.y, src);
        o.b.z = __shfl_sync(0xffffffffu, b.z, src);
        o.b.w = __shfl_sync(0xffffffffu, b.w, src);
        return o;
    }
    static __device__ __forceinline__ void store(float* p, const float2 (&f)[4]) {
        *reinterpret_cast<float4*>(p) = make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
        *reinterpret_cast<float4*>(p + 4) = make_float4(f[2].x, f[2].y, f[3].x, f[3].y);
    }
};

template <int LANES>
__device__ __forceinline__ float row_sum(float s) {
#pragma unroll
    for (int sh = LANES / 2; sh > 0; sh >>= 1) s += __shfl_xor_sync(0xffffffffu, s, sh);
    return s;
}

__device__ __forceinline__ float dot2(const float2 (&a)[4], const float2 (&b)[4]) {
    float2 s = __fmul2_rn(a[0], b[0]);
#pragma unroll
    for (int k = 1; k < 4; ++k) s = __ffma2_rn(a[k], b[k], s);
    return s.x + s.y;
}

// What a lane needs of its row's geometry.
struct LanePlan {
    int lane, j, slot, partner;   // j: 8-column chunk; slot: which of the warp's rows; partner: lane of the pair
    bool rotated;                 // the chunk lies in the rotated columns
    float sign;                   // half layout: -1 for the first member's chunk, +1 for the second's
    int i0;                       // first pair of the chunk (half: pair of column 8 j; interleaved: of 8 j, 8 j + 1)
};
template <int LANES>
__device__ __forceinline__ LanePlan lane_plan(const RopeArgs& a) {
    LanePlan p;
    p.lane = threadIdx.x & 31;
    p.j = p.lane % LANES;
    p.slot = p.lane / LANES;
    p.partner = p.lane;
    const int half = a.rd >> 1;
    p.rotated = 8 * p.j < a.rd;
    p.sign = 1.f;
    p.i0 = 4 * p.j;
    if (!a.interleaved) {
        const bool first = 8 * p.j < half;
        p.sign = first ? -1.f : 1.f;
        p.i0 = first ? 8 * p.j : 8 * p.j - half;
        if (p.rotated) p.partner = p.lane + (first ? half / 8 : -(half / 8));
    }
    return p;
}

// The token's scaled cosines and sines into the warp's table (all lanes call it).
__device__ __forceinline__ void fill_table(float2* tab, const RopeArgs& a, long long tok, int lane) {
    const int pairs = a.rd >> 1;
    if (pairs == 0) return;
    const long long pos = a.positions ? (long long)a.positions[tok] : tok % a.L;
    for (int i = lane; i < pairs; i += 32) {
        const unsigned long long at = (unsigned long long)pos * a.turn[i];
        float s, c;
        sincospif((float)(int)(at >> 32) * 4.656612873077393e-10f, &s, &c);   // 2^-31: half turns
        tab[i] = make_float2(c * a.attn_scale, s * a.attn_scale);
    }
    __syncwarp();
}

// cos and sin of the lane's 8 columns (cos 1, sin 0 outside the rotated part);
// sin with the sign of the forward's second term.
__device__ __forceinline__ void lane_trig(const float2* tab, const RopeArgs& a, const LanePlan& p, float2 (&c)[4],
                                          float2 (&s)[4]) {
    if (!p.rotated) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            c[k] = make_float2(1.f, 1.f);
            s[k] = make_float2(0.f, 0.f);
        }
    } else if (a.interleaved) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float2 t = tab[p.i0 + k];
            c[k] = make_float2(t.x, t.x);
            s[k] = make_float2(-t.y, t.y);
        }
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float2 t = tab[p.i0 + 2 * k], u = tab[p.i0 + 2 * k + 1];
            c[k] = make_float2(t.x, u.x);
            s[k] = make_float2(p.sign * t.y, p.sign * u.y);
        }
    }
}

// x_c' for each column c of the lane
template <typename T>
__device__ __forceinline__ void pair_of(const Raw<T>& raw, const float2 (&x)[4], const RopeArgs& a, const LanePlan& p,
                                        float2 (&xp)[4]) {
    if (a.interleaved) {
#pragma unroll
        for (int k = 0; k < 4; ++k) xp[k] = make_float2(x[k].y, x[k].x);
    } else {
        raw.from_lane(p.partner).unpack(xp);
    }
}

template <typename T>
__device__ __forceinline__ void load_gamma(const void* gamma, int j, float2 (&g)[4]) {
    if (gamma) {
        Raw<T> r;
        r.load(static_cast<const T*>(gamma) + 8 * j);
        r.unpack(g);
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) g[k] = make_float2(1.f, 1.f);
    }
}

// ---------------------------------------------------------------- forward
template <typename T, int D, bool NORM, int U>
__device__ __forceinline__ void forward_rows(const T* src, T* dst, int H, int wi, int wpt, const void* gamma,
                                             const float2 (&c)[4], const float2 (&s)[4], const RopeArgs& a,
                                             const LanePlan& p) {
    constexpr int LANES = D / 8, ROWS = 32 / LANES;
    float2 A[4], B[4];
    bool ready = false;
    for (int hb = wi * ROWS; hb < H; hb += U * wpt * ROWS) {
        Raw<T> raw[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int h = hb + u * wpt * ROWS + p.slot;
            if (h < H) raw[u].load(src + (long long)h * D + 8 * p.j);
            else raw[u].zero();
        }
        if (!ready) {
            ready = true;
            float2 g[4], gp[4];
            if constexpr (NORM) {
                load_gamma<T>(gamma, p.j, g);
                if (a.interleaved) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) gp[k] = make_float2(g[k].y, g[k].x);
                } else {
                    load_gamma<T>(gamma, p.partner % LANES, gp);
                }
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k) g[k] = gp[k] = make_float2(1.f, 1.f);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                A[k] = __fmul2_rn(c[k], g[k]);
                B[k] = __fmul2_rn(s[k], gp[k]);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int h = hb + u * wpt * ROWS + p.slot;
            float2 x[4], xp[4], z[4];
            raw[u].unpack(x);
            pair_of<T>(raw[u], x, a, p, xp);
#pragma unroll
            for (int k = 0; k < 4; ++k) z[k] = __ffma2_rn(xp[k], B[k], __fmul2_rn(x[k], A[k]));
            if constexpr (NORM) {
                const float r = rsqrtf(row_sum<LANES>(dot2(x, x)) * (1.f / D) + a.eps);
                const float2 r2 = make_float2(r, r);
#pragma unroll
                for (int k = 0; k < 4; ++k) z[k] = __fmul2_rn(z[k], r2);
            }
            if (h < H) Raw<T>::store(dst + (long long)h * D + 8 * p.j, z);
        }
    }
}

template <typename T, int D, bool NORM>
__global__ void __launch_bounds__(kThreads) qk_norm_rope_kernel(const __grid_constant__ RopeArgs a) {
    __shared__ float2 table[kWarps][kMaxPairs];
    const LanePlan p = lane_plan<D / 8>(a);
    const int warp = threadIdx.x / 32;
    const int per_cta = kWarps / a.wpt;
    const long long tok = (long long)blockIdx.x * per_cta + warp / a.wpt;
    const int wi = warp % a.wpt;
    pdl_wait();   // the inputs may be the previous kernel's outputs
    pdl_trigger();
    if (tok >= a.tokens) return;
    fill_table(table[warp], a, tok, p.lane);
    float2 c[4], s[4];
    lane_trig(table[warp], a, p, c, s);
    constexpr int U = 4;
    forward_rows<T, D, NORM, U>(static_cast<const T*>(a.Q) + tok * a.ld_q, static_cast<T*>(a.Qo) + tok * a.ld_qo,
                                a.Hq, wi, a.wpt, a.gamma_q, c, s, a, p);
    forward_rows<T, D, NORM, U>(static_cast<const T*>(a.K) + tok * a.ld_k, static_cast<T*>(a.Ko) + tok * a.ld_ko,
                                a.Hkv, wi, a.wpt, a.gamma_k, c, s, a, p);
}

// ---------------------------------------------------------------- backward
template <typename T, int D, bool NORM, int U>
__device__ __forceinline__ void backward_rows(const T* xsrc, const T* zsrc, T* dst, int H, int wi, int wpt,
                                              const float2 (&g)[4], const float2 (&c)[4], const float2 (&s)[4],
                                              const RopeArgs& a, const LanePlan& p, float2 (&dg)[4]) {
    constexpr int LANES = D / 8, ROWS = 32 / LANES;
    for (int hb = wi * ROWS; hb < H; hb += U * wpt * ROWS) {
        Raw<T> rx[U], rz[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int h = hb + u * wpt * ROWS + p.slot;
            rz[u].zero();
            if constexpr (NORM) rx[u].zero();
            if (h < H) {
                rz[u].load(zsrc + (long long)h * D + 8 * p.j);
                if constexpr (NORM) rx[u].load(xsrc + (long long)h * D + 8 * p.j);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int h = hb + u * wpt * ROWS + p.slot;
            float2 z[4], zp[4], dy[4];
            rz[u].unpack(z);
            pair_of<T>(rz[u], z, a, p, zp);
            // the inverse rotation: the forward's, with the sine's sign turned
#pragma unroll
            for (int k = 0; k < 4; ++k)
                dy[k] = __ffma2_rn(zp[k], make_float2(-s[k].x, -s[k].y), __fmul2_rn(z[k], c[k]));
            if constexpr (NORM) {
                float2 x[4], hh[4];
                rx[u].unpack(x);
#pragma unroll
                for (int k = 0; k < 4; ++k) hh[k] = __fmul2_rn(dy[k], g[k]);
                float ss = dot2(x, x), hx = dot2(hh, x);
                ss = row_sum<LANES>(ss);
                hx = row_sum<LANES>(hx);
                // (a row past the last head is all zeros: with eps = 0 its r would be infinite)
                const float r = h < H ? rsqrtf(ss * (1.f / D) + a.eps) : 0.f;
                const float2 r2 = make_float2(r, r);
                // r^3 s / d_k, grouped so that no factor leaves the range before the others bring it back
                const float m = -(r * hx) * (1.f / D) * r;
                const float2 m2 = make_float2(m, m);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float2 xh = __fmul2_rn(x[k], r2);
                    dg[k] = __ffma2_rn(dy[k], xh, dg[k]);
                    dy[k] = __ffma2_rn(xh, m2, __fmul2_rn(hh[k], r2));
                }
            }
            if (h < H) Raw<T>::store(dst + (long long)h * D + 8 * p.j, dy);
        }
    }
}

template <typename T, int D, bool NORM>
__global__ void __launch_bounds__(kThreads) qk_norm_rope_bwd_kernel(const __grid_constant__ RopeArgs a) {
    __shared__ float2 table[kWarps][kMaxPairs];
    __shared__ float2 share[kWarps][2][D / 2];
    constexpr int LANES = D / 8;
    const LanePlan p = lane_plan<LANES>(a);
    const int warp = threadIdx.x / 32;
    const int per_cta = kWarps / a.wpt;
    const int wi = warp % a.wpt;
    pdl_wait();
    pdl_trigger();
    float2 gq[4], gk[4], dgq[4], dgk[4];
    load_gamma<T>(NORM ? a.gamma_q : nullptr, p.j, gq);
    load_gamma<T>(NORM ? a.gamma_k : nullptr, p.j, gk);
#pragma unroll
    for (int k = 0; k < 4; ++k) dgq[k] = dgk[k] = make_float2(0.f, 0.f);
    constexpr int U = sizeof(T) == 2 ? 2 : 1;
    for (long long tok = (long long)blockIdx.x * per_cta + warp / a.wpt; tok < a.tokens;
         tok += (long long)gridDim.x * per_cta) {
        __syncwarp();   // the table's readers of the previous token are done
        fill_table(table[warp], a, tok, p.lane);
        float2 c[4], s[4];
        lane_trig(table[warp], a, p, c, s);
        backward_rows<T, D, NORM, U>(static_cast<const T*>(a.Q) + tok * a.ld_q,
                                     static_cast<const T*>(a.dQ) + tok * a.ld_dq,
                                     static_cast<T*>(a.Qo) + tok * a.ld_qo, a.Hq, wi, a.wpt, gq, c, s, a, p, dgq);
        backward_rows<T, D, NORM, U>(static_cast<const T*>(a.K) + tok * a.ld_k,
                                     static_cast<const T*>(a.dK) + tok * a.ld_dk,
                                     static_cast<T*>(a.Ko) + tok * a.ld_ko, a.Hkv, wi, a.wpt, gk, c, s, a, p, dgk);
    }
    if constexpr (NORM) {
        // the CTA's share of dgamma: its rows, then its warps, in a fixed order
#pragma unroll
        for (int k = 0; k < 4; ++k) {
#pragma unroll
            for (int sh = 16; sh >= LANES; sh >>= 1) {
                dgq[k].x += __shfl_xor_sync(0xffffffffu, dgq[k].x, sh);
                dgq[k].y += __shfl_xor_sync(0xffffffffu, dgq[k].y, sh);
                dgk[k].x += __shfl_xor_sync(0xffffffffu, dgk[k].x, sh);
                dgk[k].y += __shfl_xor_sync(0xffffffffu, dgk[k].y, sh);
            }
            if (p.slot == 0) {
                share[warp][0][4 * p.j + k] = dgq[k];
                share[warp][1][4 * p.j + k] = dgk[k];
            }
        }
        __syncthreads();
        const float* flat = reinterpret_cast<const float*>(share);
        for (int i = threadIdx.x; i < 2 * D; i += kThreads) {
            float t = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) t += flat[w * 2 * D + i];
            a.part[(long long)blockIdx.x * 2 * D + i] = t;
        }
    }
}

// dgamma[c] = the CTAs' shares added up, always in the same order: 8 columns
// to a CTA, 32 threads to a column.
template <typename T>
__global__ void __launch_bounds__(kThreads) dgamma_kernel(const float* __restrict__ part, int parts, int d, T* dgq,
                                                          T* dgk) {
    __shared__ float red[32][8];
    pdl_wait();
    pdl_trigger();
    const int col = blockIdx.x * 8 + (threadIdx.x & 7), row = threadIdx.x >> 3;
    float t = 0.f;
    for (int i = row; i < parts; i += 32) t += part[(long long)i * 2 * d + col];
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

// Warps per token: one, as long as that gives every SM 16 warps; fewer tokens
// are spread over up to 8 warps each, down to one row to a warp.
int warps_per_token(long long tokens) {
    const long long want = 16LL * plan_sms();
    int w = 1;
    while (w < kWarps && tokens * w < want) w *= 2;
    return w;
}

// CTAs of the backward: each leaves one share of dgamma, so no more than two to an SM.
long long bwd_ctas(long long tokens) {
    const long long per_cta = kWarps / warps_per_token(tokens);
    const long long need = (tokens + per_cta - 1) / per_cta;
    const long long most = 2LL * plan_sms();
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
    if ((long long)B * L > 0x7fffffffLL) return GSDPA_ERR_UNSUPPORTED;
    return GSDPA_OK;
}

// One strided tensor [tokens] x [H * d_k]: rows that do not overlap and start on 16 bytes.
int check_rows(const void* p, long long ld, int H, int dk, int dtype) {
    if (!p) return GSDPA_ERR_INVALID_ARG;
    if (ld < (long long)H * dk) return GSDPA_ERR_INVALID_ARG;
    if (!aligned(p, 16) || ld % (dtype == GSDPA_BF16 ? 8 : 4) != 0) return GSDPA_ERR_ALIGNMENT;
    return GSDPA_OK;
}

void set_rope(RopeArgs& a, const gsdpa_rope* rope) {
    a.rd = 0;
    a.interleaved = 0;
    a.attn_scale = 1.f;
    for (int i = 0; i < kMaxPairs; ++i) a.turn[i] = 0;
    if (!rope) return;
    a.rd = rope->rotary_dim;
    a.interleaved = rope->layout == GSDPA_ROPE_INTERLEAVED;
    a.attn_scale = rope->attn_scale;
    for (int i = 0; i < a.rd / 2; ++i) a.turn[i] = rope->turn[i];
}

template <typename T, int D>
cudaError_t launch_fwd(const RopeArgs& a, bool norm, cudaStream_t s) {
    const long long per_cta = kWarps / a.wpt;
    const dim3 grid((unsigned)((a.tokens + per_cta - 1) / per_cta));
    return norm ? launch_dependent(qk_norm_rope_kernel<T, D, true>, grid, dim3(kThreads), 0, s, a)
                : launch_dependent(qk_norm_rope_kernel<T, D, false>, grid, dim3(kThreads), 0, s, a);
}

template <typename T, int D>
cudaError_t launch_bwd(const RopeArgs& a, bool norm, void* dgq, void* dgk, cudaStream_t s) {
    const dim3 grid((unsigned)bwd_ctas(a.tokens));
    if (!norm) return launch_dependent(qk_norm_rope_bwd_kernel<T, D, false>, grid, dim3(kThreads), 0, s, a);
    cudaError_t e = launch_dependent(qk_norm_rope_bwd_kernel<T, D, true>, grid, dim3(kThreads), 0, s, a);
    if (e != cudaSuccess || (!dgq && !dgk)) return e;
    return launch_dependent(dgamma_kernel<T>, dim3(2 * D / 8), dim3(kThreads), 0, s, (const float*)a.part,
                            (int)grid.x, D, static_cast<T*>(dgq), static_cast<T*>(dgk));
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
        // turns per position; positions are whole numbers, so whole turns drop out
        double t = inv_freq[i] / 6.283185307179586;
        t -= std::floor(t);
        const double scaled = std::floor(std::ldexp(t, 64) + 0.5);
        rope->turn[i] = scaled >= 18446744073709551616.0 ? 0ull : (unsigned long long)scaled;
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
        const double turn = 6.283185307179586, k = 2.0 * std::log(theta);
        lo = std::floor(rd * std::log(orig_len / (beta_fast * turn)) / k);
        hi = std::ceil(rd * std::log(orig_len / (beta_slow * turn)) / k);
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
    a.gamma_q = gamma_q;
    a.gamma_k = gamma_k;
    a.positions = positions;
    a.ld_q = ld_q;
    a.ld_k = ld_k;
    a.ld_qo = ld_qo;
    a.ld_ko = ld_ko;
    a.tokens = (long long)B * L;
    a.L = L;
    a.Hq = H_q;
    a.Hkv = H_kv;
    a.wpt = warps_per_token(a.tokens);
    a.eps = eps;
    set_rope(a, rope);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (dtype == GSDPA_BF16)
        e = d_k == 128 ? launch_fwd<__nv_bfloat16, 128>(a, norm != 0, s) : launch_fwd<__nv_bfloat16, 64>(a, norm != 0, s);
    else
        e = d_k == 128 ? launch_fwd<float, 128>(a, norm != 0, s) : launch_fwd<float, 64>(a, norm != 0, s);
    return e == cudaSuccess ? GSDPA_OK : GSDPA_ERR_LAUNCH;
}

size_t gsdpa_qk_norm_rope_bwd_workspace_bytes(int B, int L, int d_k, int norm) {
    if (B < 0 || L < 0 || (d_k != 64 && d_k != 128) || (norm != 0 && norm != 1) || (long long)B * L > 0x7fffffffLL)
        return (size_t)-1;
    if (!norm || B == 0 || L == 0) return 0;
    return (size_t)bwd_ctas((long long)B * L) * 2 * d_k * sizeof(float);
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
    a.gamma_q = gamma_q;
    a.gamma_k = gamma_k;
    a.positions = positions;
    a.part = static_cast<float*>(workspace);
    a.ld_q = ld_q;
    a.ld_k = ld_k;
    a.ld_dq = ld_dqo;
    a.ld_dk = ld_dko;
    a.ld_qo = ld_dq;
    a.ld_ko = ld_dk;
    a.tokens = (long long)B * L;
    a.L = L;
    a.Hq = H_q;
    a.Hkv = H_kv;
    a.wpt = warps_per_token(a.tokens);
    a.eps = eps;
    set_rope(a, rope);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (dtype == GSDPA_BF16)
        e = d_k == 128 ? launch_bwd<__nv_bfloat16, 128>(a, norm != 0, dgamma_q, dgamma_k, s)
                       : launch_bwd<__nv_bfloat16, 64>(a, norm != 0, dgamma_q, dgamma_k, s);
    else
        e = d_k == 128 ? launch_bwd<float, 128>(a, norm != 0, dgamma_q, dgamma_k, s)
                       : launch_bwd<float, 64>(a, norm != 0, dgamma_q, dgamma_k, s);
    return e == cudaSuccess ? GSDPA_OK : GSDPA_ERR_LAUNCH;
}

}  // extern "C"
