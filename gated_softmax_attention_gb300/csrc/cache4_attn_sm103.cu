// cache4_attn_sm103.cu -- gated attention of a step's new tokens against the paged
// K/V cache held in 4 bits (a scale per token and 16 columns), through a block table.
//
// For request b with T = len + n tokens, query row i < n of head h:
//     s_j = q . k_j / sqrt(d_k), j <= len + i;   O = softmax(s) V (.) sigma(gl)
// with k_j[c] = 2^ke ks(j, c / 16) K4[j, c], v_j[c] = 2^ve vs(j, c / 16) V4[j, c].
//
// Bound by HBM: the cache is read once for all the query heads that share it, 1.125
// d_k bytes a token and K/V head. In the time that a 4-bit code takes to arrive an SM
// has 8 half-rate (integer and conversion) instructions for 64 codes, so both products
// run on the tensor cores with mma.sync (16 tokens, then 16 value columns, on the
// wide side, 8 query rows on the narrow one; tcgen05 wants 64 or 128 rows and its
// operands in shared memory in a type of its own), and a page's bytes lie so
// that what a lane loads becomes its operand with as few of these as possible:
//   e2m1  a byte is two codes, one conversion to fp16 each. For keys these are
//         neighbouring columns, the contraction's axis, and done; for values the axis is the
//         tokens, and so that a token has whole bytes (the append writes them alone)
//         the two tokens' halves of two bytes change places first, four operations a word.
//   int4  code + 8 as the low bits of the fp16 number 1024 or, the next 4 bits, 16 (code + 8): one LOP3 each and a
//         shift for every two, then 1032 or 72 taken off by a multiply-add on a pipe that has room, exact. (As subnormal
//         numbers, without the second step and with the 8 taken off in the sums by one more product, the sums were
//         not float32's: products are lined up by the exponent that an operand has in name, and beside one of a subnormal 8,
//         which a code of zero was too, all under 2^-18 of it was lost; measured, with ordinary operands 2^-23.)
// A key's scale multiplies the sum over its 16 columns in float32, one product's
// depth. A value's multiplies the weights, in fp16, whose pairs are the same for all 16
// columns: 2 instructions for 256 codes instead of 8.
//
// q, a bf16 row scaled by a power of two to below 2^15, is exact in fp16 (elements
// under 2^-31 of the row's largest lose bits that weigh less than 2^-39 of it). The
// weights p 2^-m are rounded to fp16, and again where they take the value scale. fp16's
// range is short, so they use all of it: m follows the row's largest score plus ev, ev
// the exponent of the page's largest value scale where that is above 1 (0 .. 9), and stands
// 2^13 below, so that neither p nor p vs exceeds 2^15. It moves when a tile exceeds it by 2^2.
//
// Tile = one page: keys with their scales, then values with theirs, 72 d_k contiguous
// bytes, brought by one cp.async.bulk from where the table says. The tiles of all
// requests and K/V heads are dealt evenly to teams of warps and the heads that they cut
// merged by a second kernel, as for the 8-bit cache (cache_attn.cuh).
//
// Measured (32 query heads, 8 K/V heads of 128, 64 x 8192 tokens, 604 MB, no gate): e2m1 118 us, 5.1 TB/s, int4
// 117 us, heads of 64 71 and 70 us. Of the 118 the copies alone take 102 and the products
// alone 102 (integer pipe 65 to 66 % busy, issue slots 59 %): neither hides behind the other wholly. What
// brought it there: up to 8 rows every warp is a team of its own and copies for itself, a
// page at a time, into one buffer, where the one before has just been used (the other 15 warps are work enough
// meanwhile; keys' and values' halves in a ring of three 121 us, in two buffers of their own 119), in heads of 64 three
// pages ahead (by halves 81 us; a copying warp and eight teams of two warps 133,
// 95 in heads of 64); up to 4 rows both halves of the narrow side are in use (HALF: 127 without).
// Beyond 8 rows the codes are converted again for every 16: 16 x 8000 tokens, 22 us of bytes, 16, 32 and 64 rows
// 55, 90 and 161 us (58, 96, 173 by halves of a page; a page converted once for its team, in shared memory, with rows on the
// side of 16 and scales in the operands 71, 120, 198: eight warps that meet at two barriers a page leave the SM idle
// more than the second conversion costs).
#include "cache4_internal.h"
#include "cache_attn.cuh"
#include "landing.cuh"

namespace gsdpa {
namespace {

constexpr int kMaxStages = 16;       // ring stages per team
constexpr int kBars = 96;            // ring stages of all teams
constexpr uint32_t kSmemMax = 232448 - 4608;   // dynamic: what a CTA may have, less barriers, parts and a few words
// Most tiles of a head for each team of a CTA that takes it alone.
constexpr int kWholeTiles = 4;
constexpr int kRegs = 232, kCopyRegs = 40;       // of a thread where a warp copies for the others: see Config
constexpr float kUp = 13.0f, kMove = 2.0f;     // where m stands, and how far a tile may exceed it: see above

// The largest factor from a row's sums to its scores. A row's scaled elements are below 2^15, so its sums are below
// 2^33.6: times this factor they are numbers. Two sums that differ do so by 2^-34 at least, which is 2^59
// in scores: under a larger factor, too, the largest has all the weight.
constexpr float kMostFactor = 0x1p93f;

struct PagedSeq;
struct Cache4Args {
    using Seq = PagedSeq;
    static constexpr bool kJoins = true;   // a CTA whose share is one head's leaves one part
    static constexpr int kSwitch = 1;
    __device__ __forceinline__ long long token(int b, int i) const { return (long long)cu[b] + i; }
    __device__ __forceinline__ long long tokens() const { return N; }
    // A CTA to each head, no merge, but the others idle: where the longest head gives its teams at most
    // 2 tiles more than an even share. (4 rows, heads of 128: 8 of them of 1000, 2000, 3000 tokens 12.0, 15.3,
    // 18.6 us so, cut 14.5, 15.9, 14.0; 32 heads 12.4, 15.8, 19.2 and 14.2, 14.7, 15.5; 128 heads of 2000, 4000,
    // 6000 17.1, 24.4, 34.1 and 19.4, 28.4, 35.3. Heads of 64: 10.2, 12.1, 13.8 and 12.0, 13.2, 11.7; 10.6, 12.4,
    // 14.5 and 11.8, 12.2, 12.0; 13.4, 17.9, 21.9 and 15.1, 20.5, 22.4. 16 rows, of which a team has its own ring, heads
    // of 128: 16.1, 21.2, 25.9 and 15.5, 15.9, 15.9; 128 heads 22.1, 32.5, 46.8 and 25.3, 33.9, 47.8; of 64: 11.0, 13.8,
    // 16.7 and 11.6, 11.4, 11.6; 15.3, 21.0, 27.1 and 17.5, 22.4, 27.1. One rule for all: at worst 3 us off the better;
    // where the table's width leaves few CTAs 4.5: 8 heads of 3000 tokens in 47 pages 18.5 so, cut 14.0 in a wider table.)
    __device__ __forceinline__ bool by_head(int longest, int N) const {
        const int each = (longest + (1 << lg_teams) - 1) >> lg_teams;
        return each <= kWholeTiles && each * ctas - (N >> lg_teams) <= 2 * ctas;
    }
    const __nv_bfloat16* Q;          // [N, Hq, D]
    __nv_bfloat16* O;
    const int *table, *lens, *cu, *n_new;
    const uint8_t* pool;             // [n_pages, Hkv, 72 D]
    int B, N, max_new, Hq, Hkv, G;   // G = Hq / Hkv
    int g_inverse;                   // 65536 / G, rounded up: row / G is row * g_inverse >> 16 for the rows there are
    int rows;                        // G * max_new
    int width, n_pages;              // pages of a request's row of the table; of the pool
    int lg_teams;                    // teams of a CTA, 2^lg_teams: 16, or 8 / R
    int R, stages;                   // groups of query rows (of 8 NT) to a team; ring stages per team
    float k_up;                      // 2^k_exp
    float v_exp;
    const float* gate_part;          // [gate_splits, N, gate_cols] or null
    int gate_splits, gate_cols, gate_mode;
    float* part;                     // [CTAs][teams][2][rows][D + 4]: a team's first and last head, where cut
    int ctas;                        // of the attention kernel
    int whole;                       // a CTA to each head, known from the table's width
    int wait_first;                  // no gate kernel: everything before this kernel is waited for at once
    WaitCtl ctl;
};

// A request's tokens before (len) and of this step (n), as the kernels take them:
// numbers out of range make it empty (ok = false), so that no read or write can leave
// the table, the queries or the outputs.
struct PagedSeq {
    int len, n, T, tiles;
    bool ok;
    __device__ __forceinline__ PagedSeq(const Cache4Args& a, int b) {
        const int c0 = a.cu[b], c1 = a.cu[b + 1];
        len = a.lens[b];
        const int brought = c0 >= 0 && c1 >= c0 && c1 <= a.N ? c1 - c0 : -1;
        n = a.n_new ? a.n_new[b] : brought;
        ok = brought >= 0 && brought <= a.max_new && n >= 0 && n <= brought && len >= 0 && len <= a.width * kPage - n;
        if (!ok) len = n = 0;
        T = n > 0 ? len + n : 0;   // (a request without new tokens has no rows to compute)
        tiles = (T + kPage - 1) / kPage;
    }
    __device__ __forceinline__ int span() const { return span_of<Cache4Args>(tiles); }
};

// A word of eight codes -> four fp16 pairs: pair p from bits 4 p .. and 16 + 4 p .. (int4), or from byte p (e2m1).
template <bool E2M1>
__device__ __forceinline__ void codes_to_f16(uint32_t w, uint32_t (&x)[4]) {
    if constexpr (E2M1) {
        asm("{\n\t.reg .b8 a, b, c, d;\n\t"
            "mov.b32 {a, b, c, d}, %4;\n\t"
            "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
            "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
            "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
            "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
            : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
            : "r"(w));
    } else {
        const __half2 off = __half2half2(__ushort_as_half(0x6408));                                        // 1032
        const __half2 down = __half2half2(__ushort_as_half(0x2c00)), low = __half2half2(__ushort_as_half(0xd480));   // 1/16, -72
        const uint32_t v = w >> 8;
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            uint32_t a;   // 1024 | the codes: 1024 + code + 8, or 1024 + 16 (code + 8)
            asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(a) : "r"(p < 2 ? w : v), "r"(p % 2 ? 0x00f000f0u : 0x000f000fu), "r"(0x64006400u));
            const __half2 h = *reinterpret_cast<const __half2*>(&a), c = p % 2 ? __hfma2(h, down, low) : __hsub2(h, off);
            x[p] = *reinterpret_cast<const uint32_t*>(&c);
        }
    }
}

// A word of values -> the wide operand of its 16 tokens and 16 columns. e2m1: a byte has a
// column 16 j + g and one 8 further of one token, a pair wants two tokens of one column.
template <bool E2M1>
__device__ __forceinline__ void values_to_f16(uint32_t w, uint32_t (&x)[4]) {
    if constexpr (E2M1) {
        const uint32_t low = (w & 0x0f0f0f0fu) | (w >> 4 & 0xf0f0f0f0u);    // bytes 0, 2: the columns' low halves
        const uint32_t high = (w & 0xf0f0f0f0u) | (w << 4 & 0x0f0f0f0fu);   // bytes 1, 3: the high ones
        asm("{\n\t.reg .b8 a, b, c, d;\n\t"
            "mov.b32 {a, b, c, d}, %2;\n\t"
            "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
            "cvt.rn.f16x2.e2m1x2 %1, c;\n\t}"
            : "=r"(x[0]), "=r"(x[2])
            : "r"(low));
        asm("{\n\t.reg .b8 a, b, c, d;\n\t"
            "mov.b32 {a, b, c, d}, %2;\n\t"
            "cvt.rn.f16x2.e2m1x2 %0, b;\n\t"
            "cvt.rn.f16x2.e2m1x2 %1, d;\n\t}"
            : "=r"(x[1]), "=r"(x[3])
            : "r"(high));
    } else {
        codes_to_f16<false>(w, x);
    }
}

// r = operands' product + c.
__device__ __forceinline__ void mma_f16_from(float (&r)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, float c) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
                 : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c));
}

// Four scales -> two fp16 pairs.
__device__ __forceinline__ void scales_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 a, b;\n\t"
        "mov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ float2 floats(uint32_t h) { return __half22float2(*reinterpret_cast<const __half2*>(&h)); }
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Words of a token's or lane's share, in as wide loads as they allow.
template <int N>
__device__ __forceinline__ void load_words(const uint8_t* from, uint32_t (&w)[N]) {
    if constexpr (N % 4 == 0) {
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            const uint4 v = reinterpret_cast<const uint4*>(from)[i];
            w[4 * i] = v.x;
            w[4 * i + 1] = v.y;
            w[4 * i + 2] = v.z;
            w[4 * i + 3] = v.w;
        }
    } else if constexpr (N == 2) {
        const uint2 v = *reinterpret_cast<const uint2*>(from);
        w[0] = v.x;
        w[1] = v.y;
    } else {
        w[0] = *reinterpret_cast<const uint32_t*>(from);
    }
}

// Which of a word's four tokens (2 t, 2 t + 1, 2 t + 8, 2 t + 9 of 16) are among the
// first `left` of the 16, as bytes.
__device__ __forceinline__ uint32_t keep_tokens(int left, int t) {
    const int over = left - 2 * t;
    return (over > 0 ? 0xffu : 0u) | (over > 1 ? 0xff00u : 0u) | (over > 8 ? 0xff0000u : 0u) | (over > 9 ? 0xff000000u : 0u);
}

// The exponent ev >= 0 of the largest of the value scales of 16 MT tokens: all are below 2^ev or
// at most 1.
template <int D, int MT>
__device__ __forceinline__ float scale_exponent(const uint8_t* scales, int lane) {
    constexpr int W = MT * D / 128;   // words of a lane
    uint32_t w[W], top = 0;
    load_words(scales + 4 * W * lane, w);
#pragma unroll
    for (int k = 0; k < W; ++k) {
        const uint32_t x = w[k] & 0x7f7f7f7fu;
        top = max_u16x2(top, max_u16x2(x, x << 8));
    }
    const uint32_t byte = __reduce_max_sync(0xffffffffu, max(top >> 24, top >> 8 & 0xffu));
    return (float)max((int)(byte >> 3) - 6, 0);
}

// Value scales of the tokens past the page's first `left`: zero, not what was there before (NaN,
// maybe). In shared memory, by a warp.
template <int D>
__device__ __forceinline__ void clear_scales(uint8_t* scales, int lane, int left) {
#pragma unroll
    for (int k = 0; k < D / 32; ++k) {
        const int word = 32 * k + lane;
        reinterpret_cast<uint32_t*>(scales)[word] &= keep_tokens(left - 16 * (word / (D / 4)), word % (D / 4) / (D / 16));
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // (before the stage's next copy)
    __syncwarp();
}

using Pair = unsigned long long;   // two float32 numbers
__device__ __forceinline__ Pair pair_of(float lo, float hi) {
    Pair r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpair(Pair x, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(x));
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
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// The products of 16 MT tokens become weights: element 2 x + e of s[n][i] is token
// at + 16 i + 8 x and row 8 n + 2 t + e (EL = 2: row 2 (t % 2) + e), seen up to token lim; times f it is the score
// (log2 units). On return s holds p 2^-m, and l and m are up to date. m is compared with
// the lane's own largest score only; the row's is found when one of them has to move.
// No weight times 2^ev exceeds 2^(kUp + kMove + 1 / 16): sums with m are rounded towards larger m,
// and where m is so large that its own last place counts (far), so is every score.
template <int D, int NT, int MT, int EL, bool MASK>
__device__ __forceinline__ void soften(float (&s)[NT][MT][EL], const float (&f)[NT][2], int at, const int (&lim)[NT][2],
                                       float ev, RowState<D, NT>& st, bool& far) {
    float top[NT][2];
    bool need = false;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int e = 0; e < EL; ++e)
                if (MASK && at + 16 * i + 8 * (e >> 1) > lim[n][e & 1]) s[n][i][e] = -INFINITY;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            // (a score that is no number is not above anything: the weights show it)
            static_assert(MT == 4, "four groups of 16 tokens");
            float x = max3(s[n][0][e], s[n][1][e], s[n][2][e]);
            if constexpr (EL == 4) {
                x = max3(x, s[n][3][e], s[n][0][2 + e]);
                x = fmaxf(max3(x, s[n][1][2 + e], s[n][2][2 + e]), s[n][3][2 + e]);
            } else {
                x = fmaxf(x, s[n][3][e]);
            }
            top[n][e] = MASK && x == -INFINITY ? x : x * f[n][e];
            need = need || __fadd_ru(top[n][e], ev - (kUp + kMove)) > st.m[n][e];
        }
    }
    if (__any_sync(0xffffffffu, need)) {
        bool large = false;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float fo[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float x = top[n][e];
#pragma unroll
                for (int sh = EL == 4 ? 4 : 2; sh < 32; sh <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, sh));
                const float m = fmaxf(st.m[n][e], __fadd_ru(x, ev - kUp));
                fo[e] = st.m[n][e] == -INFINITY ? 0.f : ex2_approx(st.m[n][e] - m);
                st.l[n][e] *= fo[e];
                st.m[n][e] = m;
                large = large || (fabsf(m) > 1048576.f && m != -INFINITY);
            }
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) st.o[n][i][e] *= fo[e & 1];
        }
        far = __any_sync(0xffffffffu, large);
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        float m[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) m[e] = st.m[n][e] == -INFINITY ? 0.f : st.m[n][e];   // (no token seen yet)
        const Pair minus = pair_of(-m[0], -m[1]), scale = pair_of(f[n][0], f[n][1]);
        Pair l = pair_of(st.l[n][0], st.l[n][1]);
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int x = 0; x < EL / 2; ++x) {
                float p[2];
                if (far) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) p[e] = __fsub_rn(__fmul_rn(s[n][i][2 * x + e], f[n][e]), m[e]);
                } else {
                    unpair(fma2(pair_of(s[n][i][2 * x], s[n][i][2 * x + 1]), scale, minus), p[0], p[1]);
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    p[e] = ex2_approx(p[e]);
                    // masked: nothing, whatever the factors are (0 * -inf among them)
                    if (MASK && at + 16 * i + 8 * x > lim[n][e]) p[e] = 0.f;
                    s[n][i][2 * x + e] = p[e];
                }
                l = add2(l, pair_of(p[0], p[1]));
            }
        unpair(l, st.l[n][0], st.l[n][1]);
    }
}

// A query row as the first product's narrow operand: product j of lane t covers
// columns 16 j + 4 t .. + 3. HALF: of the even or the odd products only, the others zero.
template <int D, bool HALF>
__device__ __forceinline__ void load_row(const __nv_bfloat16* src, int t, int odd, uint32_t (&w)[D / 16][2]) {
#pragma unroll
    for (int j = 0; j < D / 16; ++j) {
        uint2 v = make_uint2(0, 0);
        if (src && (!HALF || j % 2 == odd)) v = *reinterpret_cast<const uint2*>(src + 16 * j + 4 * t);
        w[j][0] = v.x;
        w[j][1] = v.y;
    }
}

// A bf16 row -> fp16 scaled by a power of two to below 2^15; returns the factor that undoes the scale.
template <int D, bool HALF>
__device__ __forceinline__ float row_to_f16(uint32_t (&w)[D / 16][2]) {
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < D / 16; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h) top = max(top, max(w[j][h] & 0x7fffu, (w[j][h] >> 16) & 0x7fffu));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    if (HALF) top = max(top, __shfl_xor_sync(0xffffffffu, top, 16));   // (the row's other products)
    // The largest element's exponent field; not below 15, so that the factor which undoes the scale is a number. (Up to
    // 254, bf16's largest, and 255, infinity and NaN, which stay what they are, both factors are.)
    const uint32_t e = max(top >> 7, 15u);
    const float scale = __uint_as_float((268u - e) << 23);
#pragma unroll
    for (int j = 0; j < D / 16; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h)
            w[j][h] = pack_f16x2(__uint_as_float(w[j][h] << 16) * scale, __uint_as_float(w[j][h] & 0xffff0000u) * scale);
    return __uint_as_float((e - 14u) << 23);
}

// The finished rows of a head that a warp has alone: element 2 x + e of o[i] is column
// 16 i + 8 x + g of row 2 t + e. Turned around by shuffles, so that a lane has columns 2 t, 2 t + 1
// of row g, times the gate, stored.
template <int D>
__device__ __forceinline__ void finish_warp(const Cache4Args& a, int b, int kvh, int n, int lane,
                                            const float (&o)[D / 16][4]) {
    const int row = lane >> 2, t = lane & 3, i = row * a.g_inverse >> 16;
    const bool live = row < a.rows && i < n;
    const int h = live ? (kvh - i) * a.G + row : 0;   // kvh G + row % G
    const long long token = live ? a.token(b, i) : 0;
    const bool gated = a.gate_mode != GSDPA_GATE_NONE, per_col = a.gate_mode == GSDPA_GATE_ELEMENTWISE;
    const long long step = a.tokens() * a.gate_cols;
    const float* gp = gated ? a.gate_part + token * a.gate_cols + (per_col ? (long long)h * D + 2 * t : h) : nullptr;
    float2 gate = make_float2(1.f, 1.f);
    if (gated) pdl_wait();   // the gate logits
    if (gated && !per_col && live) {
        float gl = 0.f;
        for (int sp = 0; sp < a.gate_splits; ++sp) gl += gp[sp * step];
        gate.x = gate.y = sigmoid(gl);
    }
    __nv_bfloat16* to = a.O + (token * a.Hq + h) * D + 2 * t;
    const int from = 8 * t + (row >> 1);   // the lane that has column 2 t of the eight; column 2 t + 1: 4 further
#pragma unroll
    for (int c = 0; c < D / 8; ++c) {   // eight columns
        const float x = o[c / 2][2 * (c % 2)], y = o[c / 2][2 * (c % 2) + 1];
        const float x0 = __shfl_sync(0xffffffffu, x, from), y0 = __shfl_sync(0xffffffffu, y, from);
        const float x1 = __shfl_sync(0xffffffffu, x, from + 4), y1 = __shfl_sync(0xffffffffu, y, from + 4);
        if (!live) continue;
        if (per_col) {
            float2 gl = make_float2(0.f, 0.f);
#pragma unroll 4
            for (int sp = 0; sp < a.gate_splits; ++sp) {
                const float2 v = *reinterpret_cast<const float2*>(gp + sp * step + 8 * c);
                gl.x += v.x;
                gl.y += v.y;
            }
            gate = make_float2(sigmoid(gl.x), sigmoid(gl.y));
        }
        *reinterpret_cast<uint32_t*>(to + 8 * c) = pack_bf16x2((row & 1 ? y0 : x0) * gate.x, (row & 1 ? y1 : x1) * gate.y);
    }
}

// Up to 8 query rows, a team is one warp and copies for itself; beyond, a team's warps
// share its tiles and one more warp issues all copies, in a group of four of its own: its registers
// go to the others (at launch 384 threads have 168 each: 64512 in all, which is 256 x 232 + 128 x 40).
template <int D, int NT>
struct Config {
    static constexpr bool ALONE = NT == 1;
    static constexpr int WARPS = ALONE ? 16 : 8;        // that compute
    static constexpr int CONSUMERS = WARPS * 32;
    static constexpr int THREADS = CONSUMERS + (ALONE ? 0 : 128);
    static constexpr int STRIDE = D + 4;                // floats of a row's part: D columns, then m, l, M
    static constexpr uint32_t STAGE = page_bytes(D);    // bytes: a page
    static constexpr int STAGES = kSmemMax / (WARPS * STAGE);   // of a lone warp: 1 (d_k 128), 3
};

// What is copied next for a team: the tiles of its share.
template <int D>
struct Feed {
    Cursor next;
    const int* row;     // of the table
    int page, after;    // of the tile at `next` and of the one after it
    __device__ __forceinline__ void enter(const Cache4Args& a) {
        row = a.table + (long long)next.b * a.width;
        page = row[next.j];
        after = next.j + 1 < next.tiles ? row[next.j + 1] : 0;
    }
    __device__ __forceinline__ void start(const Cache4Args& a, const Cursor& at) {
        next = at;
        row = a.table;
        page = after = 0;
        if (next.left > 0) enter(a);
    }
    __device__ __forceinline__ bool more() const { return next.left > 0; }
    // The next stage, to `to`; `go` in the thread that issues it. (No branch for one thread of a warp: two such a
    // page were a tenth of its time.)
    __device__ __forceinline__ void issue(const Cache4Args& a, uint8_t* to, uint64_t* full, bool go) {
        constexpr uint32_t STAGE = page_bytes(D);
        if (page >= 0 && page < a.n_pages) {
            const uint8_t* from = a.pool + ((long long)page * a.Hkv + next.kvh) * STAGE;
            asm volatile(
                "{\n\t.reg .pred p;\n\t"
                "setp.ne.u32 p, %4, 0;\n\t"
                "@p mbarrier.arrive.expect_tx.shared::cta.b64 _, [%2], %3;\n\t"
                "@p cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %3, [%2];\n\t}" ::"r"(smem_u32(to)),
                "l"(from), "r"(smem_u32(full)), "r"(STAGE), "r"((uint32_t)go)
                : "memory");
        } else if (go) {
            // no page of the pool: keys whose scales are NaN (who sees them is NaN), values of scale 0
            const uint32_t x = 0x7f7f7f7fu;
            for (int k = 0; k < 4 * D / 16; ++k) {
                reinterpret_cast<uint4*>(to + key_scales_at(D))[k] = make_uint4(x, x, x, x);
                reinterpret_cast<uint4*>(to + value_scales_at(D))[k] = make_uint4(0, 0, 0, 0);
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // (before the stage's next copy)
            mbar_arrive(full);
            atomicOr(a.ctl.err, ERR_CACHE_RANGE);
        }
        if (next.j + 1 < next.tiles) {
            ++next.j;
            --next.left;
            page = after;
            if (next.j + 1 < next.tiles) after = row[next.j + 1];
        } else {
            next.next_head(a);
            if (next.left > 0) enter(a);
        }
    }
};

template <int D, bool E2M1, int NT, bool HALF>
__global__ void __launch_bounds__(Config<D, NT>::THREADS, 1) cache4_attn_kernel(const __grid_constant__ Cache4Args a) {
    using C = Config<D, NT>;
    constexpr uint32_t STAGE = C::STAGE;
    constexpr int kConsumers = C::CONSUMERS, MT = 4, STRIDE = C::STRIDE;   // (MT: groups of 16 tokens of a tile)
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint64_t s_full[kBars], s_empty[C::ALONE ? 1 : kBars];
    __shared__ int s_place[kScan + 1], s_scan[2 * kScan / 32];
    __shared__ float s_weight[kSlots * 16], s_l[C::ALONE ? 8 : kMaxRows], s_m[C::ALONE ? 8 : kMaxRows];   // [part][row]; by row
    __shared__ Cursor s_start[2 * kSlots];
    __shared__ JoinedHead s_head;
    __shared__ int s_abort;
    volatile int* abort_flag = &s_abort;

    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int g = lane >> 2, t = lane & 3;
    const int team_warps = C::ALONE ? 1 : a.R, teams = 1 << a.lg_teams;
    const int team = warp / team_warps, rt = warp % team_warps;   // (rt: the warp's query rows; the copying warp: neither)
    // Where a team leaves its rows: a lone warp in its ring, when that is empty.
    const auto slot_of = [&](int k) {
        return reinterpret_cast<float*>(smem + (C::ALONE ? (size_t)k * a.stages * STAGE
                                                          : (size_t)teams * a.stages * STAGE + (size_t)k * a.rows * STRIDE * 4));
    };
    if (tid < teams * a.stages) {
        mbar_init(&s_full[tid], 1);
        if (!C::ALONE) mbar_init(&s_empty[tid], team_warps);
    }
    mbar_fence_init();
    if (tid == 0) s_abort = 0;
    if (a.wait_first) pdl_wait();
    pdl_trigger();   // the next kernel may be set up; it waits for this grid before it touches memory

    // ---- the teams' shares of all tiles, or of the CTA's own head
    if (a.whole) __syncthreads();   // (the barriers; else the layout's)
    const Layout all = a.whole ? Layout(s_place) : Layout(a, s_place, s_scan, tid);
    const int me = blockIdx.x, N = all.N, ctas = all.ctas;
    const bool by_head = all.by_head;
    const Deal deal(N, ctas * teams);
    const int whole_head = by_head && me < a.B * a.Hkv ? PagedSeq(a, me / a.Hkv).tiles : 0;   // the CTA's own head
    const auto team_lo = [&](int k) {
        return by_head ? Deal(whole_head, teams).from(k) : (me < ctas ? deal.from(me * teams + k) : N);
    };
    const auto start_of = [&](int k) {
        Cursor c;
        const int from = team_lo(k);
        c.left = team_lo(k + 1) - from;
        c.b = c.kvh = c.j = c.tiles = 0;
        if (c.left > 0) {
            if (by_head) {
                c.b = me / a.Hkv;
                c.tiles = whole_head;
                c.kvh = me % a.Hkv;
                c.j = from;
                return c;
            }
            int rem;
            all.find(a, from, c.b, rem);
            c.tiles = PagedSeq(a, c.b).tiles;
            if (c.tiles == 0) {
                c.left = 0;
            } else {
                const int span = span_of<Cache4Args>(c.tiles);
                c.kvh = rem / span;
                c.j = rem % span;
                if (c.j >= c.tiles) c.next_head(a);
            }
        }
        return c;
    };
    if (warp == 0 && lane < teams) s_start[lane] = start_of(lane);
    // All tiles of the CTA's share are one head's: its teams' parts are joined here, and one is left.
    if (tid == 32) {
        JoinedHead head{-1, 0};
        if (!by_head && me < ctas) head = joined_head(a, deal, me, [&](int x, int& b, int& rem) { all.find(a, x, b, rem); });
        s_head = head;
    }
    __syncthreads();
    const bool joined = s_head.first >= 0;
    const int head_place = s_head.first, head_tiles = s_head.tiles;   // of its first tile; its tiles
    if constexpr (!C::ALONE) {
        if (warp >= C::WARPS) {
            asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kCopyRegs));
            if (warp > C::WARPS) return;
            // ---- copies: lane k serves team k, in the order the team consumes them
            Cursor none;
            none.left = none.b = none.kvh = none.j = none.tiles = 0;
            Feed<D> feed;
            feed.start(a, lane < teams ? s_start[lane] : none);
            uint8_t* ring = smem + (size_t)lane * a.stages * STAGE;
            uint64_t *full = s_full + lane * a.stages, *empty = s_empty + lane * a.stages;
            uint32_t stage = 0, phase = 0, armed = 0, armed_phase = 0;
            unsigned long long idle_since = 0;
            while (__any_sync(0xffffffffu, feed.more())) {
                bool did = false;
                if (feed.more() && mbar_test(&empty[stage], phase ^ 1u)) {
                    did = true;
                    armed |= 1u << stage;
                    armed_phase = (armed_phase & ~(1u << stage)) | (phase << stage);
                    feed.issue(a, ring + stage * STAGE, &full[stage], true);
                    if (++stage == (uint32_t)a.stages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                if (__any_sync(0xffffffffu, did)) {
                    idle_since = 0;
                    continue;
                }
                // every team's ring is full: look again shortly, but not for ever
                if (__any_sync(0xffffffffu, *abort_flag != 0)) break;
                const unsigned long long now = globaltimer_ns();
                if (idle_since == 0) idle_since = now;
                if (__any_sync(0xffffffffu, now - idle_since > a.ctl.limit_ns)) {
                    if (lane == 0) {
                        atomicOr(a.ctl.err, ERR_WAIT_TIMEOUT);
                        *abort_flag = 1;
                    }
                    break;
                }
                __nanosleep(40);
            }
            // The CTA keeps its shared memory until this warp is done: it stays until what it
            // has issued is there, whoever gave up. (A share that is no longer than its ring is
            // issued at once, and its consumers may still give up; where they wait for the same
            // copies this costs nothing.)
            volatile int never = 0;
            const WaitCtl c2 = landing_limit(a.ctl);
            for (int k = 0; k < a.stages; ++k)
                if (armed & (1u << k)) mbar_wait(&full[k], (armed_phase >> k) & 1u, &never, c2);
            return;
        }
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
    }
    bool ok = true;
    {
        // ---- the team's tiles
        const uint8_t* ring = smem + (size_t)team * a.stages * STAGE;
        uint64_t *full = s_full + team * a.stages, *empty = C::ALONE ? s_empty : s_empty + team * a.stages;
        const int team_threads = 32 * team_warps, team_tid = 32 * rt + lane;
        float* slot = slot_of(team);
        const int stages = C::ALONE ? C::STAGES : a.stages;
        uint32_t stage = 0, phase = 0;   // the oldest stage that is not released
        int ahead = 0;                   // ALONE: stages that are issued and not released
        Cursor at = s_start[team];
        const int share_end = team_lo(team + 1);
        // The first head's queries are asked for before the copies: behind 30 MB of these they took 4 us more.
        uint32_t qf[NT][D / 16][2];
        const auto load_queries = [&](const PagedSeq& q) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const int row = HALF ? g & 3 : 8 * (NT * rt + n) + g, i = row * a.g_inverse >> 16;
                load_row<D, HALF>(row < a.rows && i < q.n
                                      ? a.Q + (a.token(at.b, i) * a.Hq + (at.kvh - i) * a.G + row) * D : nullptr,
                                  t, g >> 2, qf[n]);
            }
        };
        if (at.left > 0) load_queries(PagedSeq(a, at.b));
        Feed<D> feed;
        if constexpr (C::ALONE) {
            feed.start(a, at);
            for (; ahead < stages && feed.more(); ++ahead)
                feed.issue(a, smem + ((size_t)team * stages + ahead) * STAGE, &full[ahead], lane == 0);
        }
        const auto wait_full = [&]() -> const uint8_t* {
            if (!__all_sync(0xffffffffu, mbar_wait(&full[stage], phase, abort_flag, a.ctl))) {
                ok = false;
                return nullptr;
            }
            return ring + stage * STAGE;
        };
        const auto release = [&]() {
            __syncwarp();
            if constexpr (C::ALONE) {
                --ahead;
                if (feed.more()) {
                    feed.issue(a, const_cast<uint8_t*>(ring) + stage * STAGE, &full[stage], lane == 0);
                    ++ahead;
                }
            } else {
                if (lane == 0) mbar_arrive(&empty[stage]);
            }
            if (++stage == (uint32_t)stages) {
                stage = 0;
                phase ^= 1u;
            }
        };
        const auto team_and = [&](bool x) {
            if constexpr (C::ALONE) {
                x = __all_sync(0xffffffffu, x);
                __syncwarp();
                return x;
            } else {
                return named_bar_and(1 + team, team_threads, x);
            }
        };
        // rows that count for no request are zero
        const auto clear_rows = [&](int from, int to) {
            const long long words = (long long)a.Hq * D / 8;
            for (long long i = from * words + tid; i < to * words; i += kConsumers)
                reinterpret_cast<uint4*>(a.O)[i] = make_uint4(0, 0, 0, 0);
        };
        const auto row_at = [&](int b) { return min(max(a.cu[b], 0), a.N); };
        for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
            const PagedSeq r(a, b);
            if (!r.ok && tid == 0) atomicOr(a.ctl.err, ERR_CACHE_RANGE);
            clear_rows(row_at(b) + r.n, row_at(b + 1));
        }
        if (blockIdx.x == 0) clear_rows(0, row_at(0));
        if (blockIdx.x == gridDim.x - 1) clear_rows(row_at(a.B), a.N);
        RowState<D, NT> st;
        const float unscaled = kLog2e * rsqrtf((float)D) * a.k_up;
        while (at.left > 0) {
            const PagedSeq q(a, at.b);
            const int j1 = min(at.tiles, at.j + at.left);   // segment: tiles [at.j, j1) of the head
            float f[NT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const float back = fminf(row_to_f16<D, HALF>(qf[n]) * unscaled, kMostFactor);
#pragma unroll
                for (int e = 0; e < 2; ++e) f[n][e] = __shfl_sync(0xffffffffu, back, 4 * (2 * (HALF ? t & 1 : t) + e));
            }
            st.clear();
            bool far = false;   // (scores so large that their own last place counts: see soften)
            for (int j = at.j; ok && j < j1; ++j) {
                constexpr int EL = HALF ? 2 : 4;
                float s[NT][MT][EL];
                const uint8_t* kt = wait_full();
                if (!kt) break;
                const uint8_t* vt = kt + value_codes_at(D);
                // (the first query row sees tokens up to len: tiles before need no mask)
                const int base = j * kPage;
                const bool masked = base + kPage - 1 > q.len;
                const uint8_t* scales = kt + value_scales_at(D);
                if (masked && q.T < base + kPage) clear_scales<D>(const_cast<uint8_t*>(scales), lane, q.T - base);
                const float ev = scale_exponent<D, MT>(scales, lane);
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    const int n0 = 16 * i + g;   // and n0 + 8
                    uint32_t x[D / 32], y[D / 32], xs[D / 64], ys[D / 64];
                    load_words(kt + n0 * (D / 2) + t * (D / 8), x);
                    load_words(kt + (n0 + 8) * (D / 2) + t * (D / 8), y);
                    load_words(kt + key_scales_at(D) + n0 * (D / 16), xs);
                    load_words(kt + key_scales_at(D) + (n0 + 8) * (D / 16), ys);
                    float sum[NT][4];
                    const auto add = [&](int n, const float (&r)[4], float kx, float ky, bool first) {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            sum[n][e] = first ? r[e] * (e < 2 ? kx : ky) : fmaf(r[e], e < 2 ? kx : ky, sum[n][e]);
                    };
                    if constexpr (HALF) {
                        // lanes t < 2 have the even groups' sums of rows 0 .. 3, the others the odd groups'
                        float2 fx[D / 64], fy[D / 64];
#pragma unroll
                        for (int w = 0; w < D / 64; ++w) {
                            const uint32_t pick = t & 2 ? 0x4431u : 0x4420u;
                            uint32_t hx, hy, none;
                            scales_to_f16(__byte_perm(xs[w], 0, pick), hx, none);
                            scales_to_f16(__byte_perm(ys[w], 0, pick), hy, none);
                            fx[w] = floats(hx);
                            fy[w] = floats(hy);
                        }
#pragma unroll
                        for (int w = 0; w < D / 32; ++w) {   // two groups of columns
                            uint32_t xc[4], yc[4];
                            codes_to_f16<E2M1>(x[w], xc);
                            codes_to_f16<E2M1>(y[w], yc);
                            const uint32_t even[4] = {xc[0], yc[0], xc[1], yc[1]}, odd[4] = {xc[2], yc[2], xc[3], yc[3]};
#pragma unroll
                            for (int n = 0; n < NT; ++n) {
                                float r[4];
                                mma_f16_from(r, even, qf[n][2 * w][0], qf[n][2 * w][1], 0.f);
                                mma_f16(r, odd, qf[n][2 * w + 1][0], qf[n][2 * w + 1][1]);
                                add(n, r, w % 2 ? fx[w / 2].y : fx[w / 2].x, w % 2 ? fy[w / 2].y : fy[w / 2].x, w == 0);
                            }
                        }
                        // both added up: token n0 in lanes t < 2, n0 + 8 in the others
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int e = 0; e < 2; ++e)
                                s[n][i][e] = (t & 2 ? sum[n][2 + e] : sum[n][e]) +
                                             __shfl_xor_sync(0xffffffffu, t & 2 ? sum[n][e] : sum[n][2 + e], 2);
                    } else {
                        uint32_t hx[D / 32], hy[D / 32];
#pragma unroll
                        for (int w = 0; w < D / 64; ++w) {
                            scales_to_f16(xs[w], hx[2 * w], hx[2 * w + 1]);
                            scales_to_f16(ys[w], hy[2 * w], hy[2 * w + 1]);
                        }
#pragma unroll
                        for (int w = 0; w < D / 32; ++w) {   // two groups of columns
                            uint32_t xc[4], yc[4];
                            codes_to_f16<E2M1>(x[w], xc);
                            codes_to_f16<E2M1>(y[w], yc);
                            const float2 fx = floats(hx[w]), fy = floats(hy[w]);
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                const uint32_t op[4] = {xc[2 * k], yc[2 * k], xc[2 * k + 1], yc[2 * k + 1]};
#pragma unroll
                                for (int n = 0; n < NT; ++n) {
                                    const int c = 2 * w + k;
                                    float r[4];
                                    mma_f16_from(r, op, qf[n][c][0], qf[n][c][1], 0.f);
                                    add(n, r, k ? fx.y : fx.x, k ? fy.y : fy.x, c == 0);
                                }
                            }
                        }
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int e = 0; e < EL; ++e) s[n][i][e] = sum[n][e];
                    }
                }
                int lim[NT][2] = {};
                const int at0 = base + g + (HALF ? 4 * (t & 2) : 0);   // the lane's first token
                if (masked) {
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {   // the last token that each of the lane's rows sees
                            const int row = 8 * (NT * rt + n) + 2 * (HALF ? t & 1 : t) + e, i = row * a.g_inverse >> 16;
                            lim[n][e] = row < a.rows && i < q.n ? q.len + i : -1;
                        }
                    soften<D, NT, MT, EL, true>(s, f, at0, lim, ev, st, far);
                } else {
                    soften<D, NT, MT, EL, false>(s, f, at0, lim, ev, st, far);
                }
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    uint32_t pf[NT][2], sw[D / 16];
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int x = 0; x < EL / 2; ++x)
                            pf[n][x] = transpose8(pack_f16x2(s[n][i][2 * x], s[n][i][2 * x + 1]));
                    if constexpr (HALF) {   // (tokens 8 .. 15 came out in lanes g >= 4)
#pragma unroll
                        for (int n = 0; n < NT; ++n) pf[n][1] = __shfl_xor_sync(0xffffffffu, pf[n][0], 16);
                    }
                    load_words(scales + i * D + t * (D / 4), sw);
#pragma unroll
                    for (int quad = 0; quad < D / 64; ++quad) {
                        uint32_t w[4];
                        load_words(vt + ((i * (D / 64) + quad) * 32 + lane) * 16, w);
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int c = 4 * quad + k;
                            uint32_t op[4], sc[2];
                            values_to_f16<E2M1>(w[k], op);
                            scales_to_f16(sw[c], sc[0], sc[1]);
#pragma unroll
                            for (int n = 0; n < NT; ++n) {
                                const uint32_t b0 = mul_f16x2(pf[n][0], sc[0]), b1 = mul_f16x2(pf[n][1], sc[1]);
                                mma_f16(st.o[n][c], op, b0, b1);
                            }
                        }
                    }
                }
                release();
            }

            // ---- the segment's rows: sums over the lanes, and the values' unit into the outputs
            const bool whole = at.j == 0 && j1 == at.tiles && !joined, final = at.left <= span_of<Cache4Args>(at.tiles) - at.j;
            const float unit = exp2f(a.v_exp);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float k[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    st.M[n][e] = st.m[n][e];
#pragma unroll
                    for (int sh = HALF ? 2 : 4; sh < 32; sh <<= 1)
                        st.l[n][e] += __shfl_xor_sync(0xffffffffu, st.l[n][e], sh);
                    k[e] = unit;
                    // (a row that saw nothing is zero)
                    if (C::ALONE && whole) k[e] = st.l[n][e] > 0.f || st.l[n][e] != st.l[n][e] ? unit / st.l[n][e] : 0.f;
                }
#pragma unroll
                for (int i = 0; i < D / 16; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) st.o[n][i][e] *= k[e & 1];
            }
            const auto put = [&](float* base) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int row = 8 * (NT * rt + n) + 2 * t + e;
                        if (row >= a.rows) continue;
                        float* to = base + row * STRIDE;
#pragma unroll
                        for (int i = 0; i < D / 16; ++i) {
                            to[16 * i + g] = st.o[n][i][e];
                            to[16 * i + 8 + g] = st.o[n][i][2 + e];
                        }
                        if (g == 0)
                            *reinterpret_cast<float4*>(to + D) = make_float4(st.m[n][e], st.l[n][e], st.M[n][e], 0.f);
                    }
            };
            // A head of the team's alone is finished; else its part is left in global memory
            // for the merge kernel, or in shared memory where the CTA's teams have one head.
            if (C::ALONE && whole) {
                if constexpr (C::ALONE) finish_warp<D>(a, at.b, at.kvh, q.n, lane, st.o[0]);
                ok = team_and(ok && !*abort_flag);
                if (!ok) break;
            } else {
                put(whole || by_head || joined ? slot
                                               : part_of<D>(a, deal, me * teams + team, share_end - at.left - at.j));
                ok = team_and(ok && !*abort_flag);
                if (!ok) break;
                if (whole) {
                    if (a.gate_mode != GSDPA_GATE_NONE) pdl_wait();   // the gate logits
                    for (int idx = team_tid; idx < a.rows * (D / 4); idx += team_threads) {
                        const int row = idx / (D / 4), col = 4 * (idx % (D / 4));
                        const float* from = slot + row * STRIDE;
                        const float4 x = *reinterpret_cast<const float4*>(from + D);
                        finish<D>(a, at.b, at.kvh, q.n, row, col, out_scale(x.x, x.y, x.z),
                                  *reinterpret_cast<const float4*>(from + col), gate_of<D>(a, at.b, at.kvh, q.n, row, col));
                    }
                    if (!final) team_and(true);   // (the slot may be written again)
                }
            }
            at.next_head(a);
            if (at.left > 0) load_queries(PagedSeq(a, at.b));
        }
        if constexpr (C::ALONE) {
            // (a warp that gave up stays until its copies have landed: the CTA keeps its shared memory that long)
            volatile int never = 0;
            const WaitCtl c2 = landing_limit(a.ctl);
            for (; ahead > 0; --ahead) {
                mbar_wait(&full[stage], phase, &never, c2);
                if (++stage == (uint32_t)stages) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        }
    }

    pdl_wait();   // the gate logits; and what follows on the stream may rely on the gate kernel having ended
    // Parts in shared memory: of the CTA's own head (more than one, or it is done), or of a piece of a head.
    int parts = 0;
    if (by_head) parts = min(whole_head, teams);
    else if (joined) parts = min(teams, deal.taker(head_place + head_tiles - 1) - me * teams + 1);
    if ((by_head || joined) && named_bar_and(kSlots + 1, kConsumers, ok && !*abort_flag) && (joined || parts > 1)) {
        const int b = by_head ? me / a.Hkv : 0, n = by_head ? PagedSeq(a, b).n : 0;
        // each part's weight in each row, and the rows' sums: a row's parts in lanes next to each other
        if (tid < ((a.rows * teams + 31) & ~31)) {
            const int row = tid >> a.lg_teams, part = tid & (teams - 1);
            float m = -INFINITY, l = 0.f;
            if (row < a.rows && part < parts) {
                const float2 x = *reinterpret_cast<const float2*>(slot_of(part) + row * STRIDE + D);
                m = x.x;
                l = x.y;
            }
            float top = m;
            for (int sh = 1; sh < teams; sh <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, sh));
            const float w = part_weight(m, top);
            l *= w;
            for (int sh = 1; sh < teams; sh <<= 1) l += __shfl_xor_sync(0xffffffffu, l, sh);
            if (row < a.rows) {
                s_weight[part * a.rows + row] = w;
                s_l[row] = l;
                s_m[row] = top;
            }
        }
        named_bar_sync(kSlots + 1, kConsumers);
        for (int idx = tid; idx < a.rows * (D / 4); idx += kConsumers) {
            const int row = idx / (D / 4), col = 4 * (idx % (D / 4));
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
            for (int i = 0; i < parts; ++i) {
                const float w = s_weight[i * a.rows + row];
                const float4 x = *reinterpret_cast<const float4*>(slot_of(i) + row * STRIDE + col);
                o.x = fmaf(w, x.x, o.x);
                o.y = fmaf(w, x.y, o.y);
                o.z = fmaf(w, x.z, o.z);
                o.w = fmaf(w, x.w, o.w);
            }
            if (by_head) {
                finish<D>(a, b, me % a.Hkv, n, row, col, out_scale(s_m[row], s_l[row], s_m[row]), o,
                          gate_of<D>(a, b, me % a.Hkv, n, row, col));
            } else {
                float* to = part_of<D>(a, deal, me * teams, head_place) + row * STRIDE;
                *reinterpret_cast<float4*>(to + col) = o;
                if (col == 0) *reinterpret_cast<float4*>(to + D) = make_float4(s_m[row], s_l[row], s_m[row], 0.f);
            }
        }
    }
}

// Shared memory and ring of one problem.
struct Shape {
    int NT, R, teams, stages;
    uint32_t smem;
};
Shape shape_of(int rows, int D) {
    Shape s;
    s.NT = rows <= 8 ? 1 : 2;
    s.R = rows <= 16 ? 1 : (rows <= 32 ? 2 : (rows <= 64 ? 4 : 8));
    s.teams = (s.NT == 1 ? 2 * kSlots : kSlots) / s.R;
    const uint32_t merge = s.NT == 1 ? 0 : (uint32_t)(s.teams * rows * (D + 4)) * 4;
    const uint32_t per_stage = (uint32_t)s.teams * page_bytes(D);
    // as many copies in flight as fit
    s.stages = (int)((kSmemMax - merge) / per_stage);
    if (s.stages > kMaxStages) s.stages = kMaxStages;
    if (s.stages > kBars / s.teams) s.stages = kBars / s.teams;
    s.smem = (uint32_t)s.stages * per_stage + merge;
    return s;
}

struct Cache4Plan {
    Problem p{};
    WorkspacePlan w;   // the gate kernel's part
    size_t part = 0, total = 0;
};

int plan_cache4(const gsdpa_cache4* c, int B, int max_pages, int n_rows, int max_new, int d_model, int Hq, int gate_mode,
                Cache4Plan* out) {
    const int st = validate_cache4(c);
    if (st != GSDPA_OK) return st;
    if (B < 0 || max_pages < 1 || n_rows < 0 || max_new < 1 || Hq < 1 || Hq % c->H_kv != 0) return GSDPA_ERR_INVALID_ARG;
    if (gate_mode < GSDPA_GATE_NONE || gate_mode > GSDPA_GATE_ELEMENTWISE) return GSDPA_ERR_INVALID_ARG;
    if (gate_mode != GSDPA_GATE_NONE && d_model < 1) return GSDPA_ERR_INVALID_ARG;
    if (gate_mode != GSDPA_GATE_NONE && d_model % 8 != 0) return GSDPA_ERR_UNSUPPORTED;
    if (gate_mode == GSDPA_GATE_HEADWISE && Hq % 8 != 0) return GSDPA_ERR_UNSUPPORTED;
    const long long rows = (long long)(Hq / c->H_kv) * max_new;
    if (rows > kMaxRows) return GSDPA_ERR_UNSUPPORTED;
    // (places are counted in 32 bits, and so are a request's tokens)
    if (max_pages > 0x7fffffff / kPage - 1) return GSDPA_ERR_UNSUPPORTED;
    const long long heads = (long long)B * c->H_kv;
    if (heads > 0x7fffffffLL - 2 * kMaxCtas || heads * (max_pages + Cache4Args::kSwitch) > 0x7fffffffLL) return GSDPA_ERR_UNSUPPORTED;
    if (n_rows > 0x7fffffff / 8) return GSDPA_ERR_UNSUPPORTED;
    if (B == 0 || n_rows == 0) return GSDPA_OK;   // an empty problem: nothing to plan
    Cache4Plan& o = *out;
    Problem& p = o.p;
    p.B = 1;
    p.Lq = n_rows;
    p.d_model = d_model;
    p.Hq = Hq;
    p.Hkv = c->H_kv;
    p.dk = c->d_k;
    p.gate_mode = gate_mode;
    p.causal = 1;
    p.dtype = GSDPA_BF16;
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off = (off + bytes + 255) & ~size_t(255);
        return at;
    };
    if (gate_mode != GSDPA_GATE_NONE) plan_gate_rows(p, plan_sms(), &o.w);
    o.w.gate_part = take(sizeof(float) * (size_t)o.w.gate_splits * o.w.gate_rows * o.w.gate_cols);
    const size_t part = sizeof(float) * (size_t)rows * (c->d_k + 4);
    o.part = take(part * plan_sms() * 2 * shape_of((int)rows, c->d_k).teams);
    o.total = off;
    return GSDPA_OK;
}

template <int D, bool E2M1, int NT, bool HALF>
cudaError_t launch(const Cache4Args& a, const Shape& sh, unsigned grid, cudaStream_t s) {
    static PerDeviceSetup setup;
    const cudaError_t e = setup_once_per_device(setup, [](int&) {
        return cudaFuncSetAttribute(cache4_attn_kernel<D, E2M1, NT, HALF>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    (int)kSmemMax);
    });
    if (e != cudaSuccess) return e;
    return launch_dependent(cache4_attn_kernel<D, E2M1, NT, HALF>, dim3(grid), dim3(Config<D, NT>::THREADS), sh.smem, s,
                            a);
}
template <int D, bool E2M1>
cudaError_t launch(const Cache4Args& a, const Shape& sh, unsigned grid, cudaStream_t s) {
    if (sh.NT == 2) return launch<D, E2M1, 2, false>(a, sh, grid, s);
    return a.rows <= 4 ? launch<D, E2M1, 1, true>(a, sh, grid, s) : launch<D, E2M1, 1, false>(a, sh, grid, s);
}

}  // namespace
}  // namespace gsdpa

using namespace gsdpa;

extern "C" {

size_t gsdpa_cache4_workspace_bytes(const gsdpa_cache4* cache, int B, int max_pages, int n_rows, int max_new,
                                    int d_model, int H_q, int gate_mode) {
    Cache4Plan pl;
    if (plan_cache4(cache, B, max_pages, n_rows, max_new, d_model, H_q, gate_mode, &pl) != GSDPA_OK) return (size_t)-1;
    return pl.total;
}

int gated_sdpa_cache4(const void* X, const void* Q, const gsdpa_cache4* cache, const int* table, const int* lens,
                      const int* cu, const int* n_new, const void* W_g, void* O, int B, int max_pages, int n_rows,
                      int max_new, int d_model, int H_q, int gate_mode, void* workspace, size_t workspace_bytes,
                      void* stream) {
    Cache4Plan pl;
    int st = plan_cache4(cache, B, max_pages, n_rows, max_new, d_model, H_q, gate_mode, &pl);
    if (st != GSDPA_OK) return st;
    if (n_rows == 0) return GSDPA_OK;
    if ((st = validate_cache4_pointers(cache)) != GSDPA_OK) return st;
    const bool gated = gate_mode != GSDPA_GATE_NONE;
    if (!Q || !O || (B > 0 && (!table || !lens || !cu)) || (gated && (!X || !W_g))) return GSDPA_ERR_INVALID_ARG;
    const auto off = [](const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; };
    if (off(Q, 16) || off(O, 16) || (gated && (off(X, 16) || off(W_g, 16)))) return GSDPA_ERR_ALIGNMENT;
    if (off(table, 4) || off(lens, 4) || off(cu, 4) || off(n_new, 4)) return GSDPA_ERR_ALIGNMENT;
    Runtime rt;
    int major = 0, minor = 0;
    if (!current_runtime(&rt, &major, &minor)) return GSDPA_ERR_LAUNCH;
    if (!(major == 10 && minor == 3) || !encode_tiled_fn()) return GSDPA_ERR_UNSUPPORTED;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (B == 0)   // rows of no request
        return cudaMemsetAsync(O, 0, (size_t)n_rows * H_q * cache->d_k * 2, s) == cudaSuccess ? GSDPA_OK : GSDPA_ERR_LAUNCH;
    if (!workspace || workspace_bytes < pl.total) return GSDPA_ERR_WORKSPACE;
    if (off(workspace, 256)) return GSDPA_ERR_ALIGNMENT;
    char* ws = static_cast<char*>(workspace);
    pl.p.X = X;
    pl.p.Wg = W_g;

    // The gate logits' kernel first: it waits for the kernels before it and then lets
    // the attention, its programmatic dependent, start: that finds the cache and the
    // queries written and waits for the logits where it reads them.
    const int sms = rt.num_sms < kMaxCtas ? rt.num_sms : kMaxCtas;
    bool launched = false;
    cudaError_t e = launch_gate_logits_bf16(pl.p, pl.w, ws, rt, s, &launched, ZeroJob());
    if (e == cudaErrorInvalidValue) return GSDPA_ERR_INVALID_ARG;
    if (e != cudaSuccess) return GSDPA_ERR_LAUNCH;

    Cache4Args a;
    a.Q = static_cast<const __nv_bfloat16*>(Q);
    a.O = static_cast<__nv_bfloat16*>(O);
    a.table = table;
    a.lens = lens;
    a.cu = cu;
    a.n_new = n_new;
    a.pool = static_cast<const uint8_t*>(cache->pool);
    a.B = B;
    a.N = n_rows;
    a.max_new = max_new;
    a.Hq = H_q;
    a.Hkv = cache->H_kv;
    a.G = H_q / cache->H_kv;
    a.g_inverse = (65536 + a.G - 1) / a.G;
    a.rows = a.G * max_new;
    a.width = max_pages;
    a.n_pages = cache->n_pages;
    const Shape sh = shape_of(a.rows, cache->d_k);
    a.R = sh.R;
    a.lg_teams = 0;
    while (1 << a.lg_teams < sh.teams) ++a.lg_teams;
    a.stages = sh.stages;
    a.k_up = ldexpf(1.f, cache->k_exp);
    a.v_exp = (float)cache->v_exp;
    a.gate_part = gated ? reinterpret_cast<const float*>(ws + pl.w.gate_part) : nullptr;
    a.gate_splits = pl.w.gate_splits;
    a.gate_cols = pl.w.gate_cols;
    a.gate_mode = gate_mode;
    a.part = reinterpret_cast<float*>(ws + pl.part);
    a.wait_first = launched ? 0 : 1;
    a.ctl.err = rt.err;
    a.ctl.limit_ns = rt.limit_ns;
    // one CTA per SM, fewer where full tables would not give each its tiles
    const long long most = (long long)B * a.Hkv * ((max_pages + sh.teams - 1) / sh.teams);
    long long grid = sms;   // (no fewer than the heads, where those fit)
    if (grid > most) grid = most;
    a.ctas = (int)grid;
    // By the table's width, which saves the lengths' lookup and the merge kernel: the same with 2 tiles (4 rows, heads of
    // 128: 8 heads of 1000, 2000 tokens 9.9, 13.8 us, 32 heads 10.4, 14.0, 128 heads of 2000, 4000 14.9, 22.2; of 64: 8.1, 10.6,
    // 8.5, 10.8 and 11.4, 16.1).
    const long long heads = (long long)B * a.Hkv, each = (max_pages + sh.teams - 1) / sh.teams;
    const bool whole = heads <= grid && each <= kWholeTiles && each * (sms - heads) <= 2 * sms;
    a.whole = whole;
    const bool e2m1 = cache->kind == GSDPA_CACHE_E2M1;
    if (cache->d_k == 128)
        e = e2m1 ? launch<128, true>(a, sh, (unsigned)grid, s) : launch<128, false>(a, sh, (unsigned)grid, s);
    else
        e = e2m1 ? launch<64, true>(a, sh, (unsigned)grid, s) : launch<64, false>(a, sh, (unsigned)grid, s);
    // (Not a CTA for every SM: the SMs that are done first take them all, and they are
    // set up when the last are done.)
    if (e == cudaSuccess && !whole)
        e = launch_dependent(cache->d_k == 128 ? cache_merge_kernel<128, Cache4Args> : cache_merge_kernel<64, Cache4Args>,
                             dim3((unsigned)(sms - sms / 8)), dim3(kMergeThreads), 0, s, a);
    return e == cudaSuccess ? GSDPA_OK : GSDPA_ERR_LAUNCH;
}

}  // extern "C"
