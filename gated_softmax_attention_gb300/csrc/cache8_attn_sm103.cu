// cache8_attn_sm103.cu -- gated attention of a step's new tokens against the
// K/V cache held in 8 bits (one scale per block of 64 tokens and head).
//
// For sequence b with T = len + n tokens, query row i < n of head h:
//     s_j = q . k_j / sqrt(d_k), j <= len + i;   O = softmax(s) V (.) sigma(gl)
// with k_j = ks(j / 64) K8[j], v_j = vs(j / 64) V8[j], and the open block's
// tokens taken as the bf16 values they still are.
//
// Bound by HBM: the cache is read once for all the query heads that share it,
// 2 d_k bytes a token and K/V head. 8-bit elements arrive twice as fast as
// 16-bit ones, and four or eight query heads' products per element are then
// more than the CUDA cores do in that time, so both products run on the tensor
// cores with mma.sync, fp16 operands and fp32 sums: 16 tokens (then 16 value
// columns) on the wide side, 8 query rows (heads of the group x new tokens) on
// the narrow one. (tcgen05 wants 64 or 128 rows, operands in shared memory in
// one of its own types, and leaves the scores in tensor memory; here the 8-bit
// codes have to pass through registers anyway, to become fp16.) What is left
// to the ordinary pipes is turning codes into fp16, 5 instructions for 4 int8
// codes, and it sets the shape: a code is converted once for up to 16 query
// rows, and with 16 x 8 products the unused part of the narrow side is small
// for a decoding step (the first build put the query rows on the side of 16: twice the
// products, sums and registers, 2010 instructions a tile, and 64 sequences of
// 2048 tokens took 88 us instead of the 40 us of their bytes).
//
// int8 and e4m3 codes are exact in fp16; q, a bf16 row scaled by a power of two
// to below 1, too (elements under 2^-14 of the row's largest lose bits that
// weigh less than 2^-24 of it). The weights, times their block's value scale, are
// rounded to fp16 for the second product. fp16's own range is short, so they use
// all of it: the largest stand for 2^12 to 2^15, those down to 2^-26 of them keep 11
// bits, smaller ones lose bits and from 2^-37 on vanish (with the largest at 2^-1,
// 8192 tokens beside one of zero values that had 99.9 % of the weight came out 10 %
// off). The open block's, whose values may exceed fp16's range, become two bf16
// parts (16 bits).
//
// Two running references, both only for range: m for the sum of weights, and
// M for the outputs, which carry the value scales: a block adds
// (p c) V8 with c = vs 2^(m - M), so that a block of large values that the
// query hardly looks at cannot push the others' products out of fp16's range.
// They move when a tile exceeds them by 2^8 and 2^2 (rarely after the first tile). M also
// follows m from kApart below: where the row's weight went to a block whose
// values are zero or next to it, c would exceed float32 for the blocks whose weights
// vanish beside it (less than 2^-126 of the row's largest weight is nothing).
//
// Tile = one block: K8 [64][d_k] and V8 [d_k][64], each 64 d_k contiguous bytes,
// brought by cp.async.bulk. The tiles of all sequences and K/V heads form one
// sequence of tiles that is cut evenly over the CTAs, and a CTA's share again
// over its teams of warps (lengths are read on the device: no length, however
// uneven, leaves SMs idle): up to 8 query rows, 8 teams of two warps that have
// 32 of a tile's tokens each; beyond, teams of one, two, four or eight warps
// with 16 query rows each. A team streams its tiles through a ring of its own
// (one warp issues all copies) and needs no other team until its share is done: a
// K/V head that lies within the share is finished by the team, of the two heads
// that its ends cut it leaves parts (outputs, m, l, M) in global memory, and a
// second kernel merges these in a fixed order. No CTA waits for another.
// (With the tiles dealt to the teams in turn, and all warps merging at the end of
// every head, the same 64 sequences took 90 us. Dealing out the last fifth of
// the tiles in small chunks to the teams that were done first made all SMs end
// at the same time, with even shares they do between 140 and 170 us for 64
// sequences of 8192 tokens, but none earlier: the memory is busy to the end.)
//
// The order of the tokens inside a tile's products is chosen so that 16
// consecutive bytes of a value column are one lane's share of the second
// product's wide operand; the weights reach their place in its narrow operand
// by one 8 x 8 transposition (movmatrix) for each 8 tokens.
//
// Measured, heads of 128, without a gate: 64 sequences of 8192 tokens, 32/8 heads
// 171 us (6.3 TB/s, 93 % of a plain copy); one of 131072 tokens, 16/2 heads 23 us;
// 24 of up to 32767 tokens, 16/2 heads 48.5 us; one of 1000 tokens 11.5 us.
#include "cache8_internal.h"
#include "cache_attn.cuh"
#include "landing.cuh"

namespace gsdpa {
namespace {

constexpr int kMaxStages = 16;       // ring stages per team
// A head is one CTA's where all have at most this many tiles for each team of it and
// there are CTAs for all: the teams then merge in shared memory. If the capacity says
// so already, the merge kernel is not launched (1000 tokens, 8 teams: 11.5 us and 2.5
// us less of the host's time, cut up 10.3 us); if only the lengths do, it is, for
// nothing (60 tokens: 6.9 us, cut up 10.1; 500 tokens 10.1 and 10.1; 1000 tokens 12.1
// and 10.3). (128 query rows are one team's: 1000 tokens by a CTA 47.7 us, cut up 14.3.)
constexpr int kWholeTiles = 3, kFewTiles = 1;
constexpr int kBars = 48;            // ring stages of all teams
constexpr uint32_t kSmemMax = 232448 - 1984;   // dynamic: what a CTA may have, less barriers, parts and a few words
constexpr float kMove = 8.0f, kMoveOut = 2.0f;   // how far a tile may exceed m, and M, in log2 units
constexpr float kUp = 13.0f;         // M stands 2^kUp below the largest product: 2^(kUp + kMoveOut) is in fp16's range
constexpr float kApart = 100.0f;

struct SeqTiles;
struct Cache8Args {
    using Seq = SeqTiles;
    static constexpr bool kJoins = false;   // (a head's parts are its teams')
    static constexpr int kSwitch = 4;
    __device__ __forceinline__ long long token(int b, int i) const { return (long long)b * Lq + i; }
    __device__ __forceinline__ long long tokens() const { return (long long)B * Lq; }
    __device__ __forceinline__ bool by_head(int longest, int) const { return longest <= whole_tiles; }
    const __nv_bfloat16* Q;          // [B, Lq, Hq, D]
    __nv_bfloat16* O;
    const int *lens, *n_new;
    const uint8_t *k8, *v8;
    const float *k_scale, *v_scale;
    const __nv_bfloat16 *k_tail, *v_tail;
    int B, Lq, Hq, Hkv, G;           // G = Hq / Hkv
    int g_inverse;                   // 65536 / G, rounded up: row / G is row * g_inverse >> 16 for the rows there are
    int rows;                        // G * Lq
    int blocks, capacity;
    int lg_teams;                    // teams of a CTA, 2^lg_teams = 8 / R
    int R, stages;                   // groups of query rows (of 8 NT) to a team; ring stages per team
    const float* gate_part;          // [gate_splits, B * Lq, gate_cols] or null
    int gate_splits, gate_cols, gate_mode;
    float* part;                     // [CTAs][teams][2][rows][D + 4]: a team's first and last head, where cut
    int ctas;                        // of the attention kernel
    int whole_tiles;                 // most tiles of a head for one CTA to take it alone
    int wait_first;                  // no gate kernel: everything before this kernel is waited for at once
    WaitCtl ctl;
};

__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// 4 codes -> two fp16 pairs, exactly: int8 codes 0, 2 and 1, 3; e4m3 codes 0, 1
// and 2, 3. pair_first() and pair_step() say which: code k of pair h is the
// word's code h * pair_first + k * pair_step.
template <bool E4M3>
__device__ __forceinline__ void codes_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
    if constexpr (E4M3) {
        asm("{\n\t.reg .b16 a, b;\n\t"
            "mov.b32 {a, b}, %2;\n\t"
            "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
            "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
            : "=r"(lo), "=r"(hi)
            : "r"(w));
    } else {
        // code + 128 in the low bits of the fp16 number 1024, then 1152 taken off
        const __half2 off = __half2half2(__ushort_as_half(0x6480));   // 1152
        // (as one three-input operation: left to itself the compiler makes two of it, and the integer pipe
        // is what the conversion is bound by)
        uint32_t a, b;
        asm("lop3.b32 %0, %1, %2, %3, 0x6a;" : "=r"(a) : "r"(w), "r"(0x00ff00ffu), "r"(0x64806480u));
        asm("lop3.b32 %0, %1, %2, %3, 0x6a;" : "=r"(b) : "r"(w >> 8), "r"(0x00ff00ffu), "r"(0x64806480u));
        const __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&a), off);
        const __half2 y = __hsub2(*reinterpret_cast<const __half2*>(&b), off);
        lo = *reinterpret_cast<const uint32_t*>(&x);
        hi = *reinterpret_cast<const uint32_t*>(&y);
    }
}
template <bool E4M3>
__device__ constexpr int pair_first() { return E4M3 ? 2 : 1; }
template <bool E4M3>
__device__ constexpr int pair_step() { return E4M3 ? 1 : 2; }
// the same order for 4 16-bit elements in two words
template <bool E4M3>
__device__ __forceinline__ void pair_up(uint32_t& a, uint32_t& b) {
    if constexpr (!E4M3) {
        const uint32_t lo = __byte_perm(a, b, 0x5410), hi = __byte_perm(a, b, 0x7632);
        a = lo;
        b = hi;
    }
}

struct SeqTiles {
    int len, n, T, tiles;
    __device__ __forceinline__ SeqTiles(const Cache8Args& a, int b) {
        const SeqRange r = seq_range(a.lens, a.n_new, b, a.Lq, a.capacity);
        len = r.len;
        n = r.n;
        T = r.n > 0 ? r.len + r.n : 0;   // (a sequence without new tokens has no rows to compute)
        tiles = (T + kCacheBlock - 1) / kCacheBlock;
    }
    __device__ __forceinline__ bool open(int j) const { return (j + 1) * kCacheBlock > T; }
    __device__ __forceinline__ int span() const { return span_of<Cache8Args>(tiles); }
};

// A value scale as frac 2^ev, frac in [1, 2) (0, NaN and infinity stay what they are).
__device__ __forceinline__ void split_scale(float vs, float& frac, float& ev) {
    frac = vs;
    ev = 0.f;
    if (vs < 8.6736174e-19f) {   // 2^-60: out of the subnormal numbers
        frac *= 1.152921504606847e18f;
        ev = -60.f;
    }
    const uint32_t bits = __float_as_uint(frac);
    if (vs > 0.f && (bits >> 23) < 255u) {
        ev += (float)((int)(bits >> 23) - 127);
        frac = __uint_as_float((bits & 0x7fffffu) | 0x3f800000u);
    } else {
        ev = -INFINITY;   // (nothing that M should follow)
    }
}

// The products of a warp's 16 MT tokens of a tile become weights: element
// 2 x + e of s[n][i] is token at + 4 i + x * pair_first and row 8 n + 2 t + e,
// seen up to token lim. f ks turns products into scores (log2 units), frac 2^ev
// is the tile's value scale. On return s holds p c, and l and the references
// are up to date. The references are compared with the lane's own largest score
// only; the row's is found when one of them has to move.
template <int D, int NT, int MT, bool E4M3, bool MASK>
__device__ __forceinline__ void soften(float (&s)[NT][MT][4], const float (&f)[NT][2], float ks, int at,
                                       const int (&lim)[NT][2], float frac, float ev, RowState<D, NT>& st) {
    float k[NT][2], top[NT][2];
    bool need = false;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        top[n][0] = top[n][1] = -INFINITY;
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (MASK && at + 4 * i + (e >> 1) * pair_first<E4M3>() > lim[n][e & 1]) s[n][i][e] = -INFINITY;
                top[n][e & 1] = fmaxf(top[n][e & 1], s[n][i][e]);
            }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            k[n][e] = f[n][e] * ks;
            // (a score that is no number is not above anything: the weights show it)
            top[n][e] = top[n][e] == -INFINITY ? -INFINITY : top[n][e] * k[n][e];
            need = need || top[n][e] > st.m[n][e] + kMove ||
                   fmaxf(top[n][e], st.m[n][e] - kApart) + ev + 1.f - kUp > st.M[n][e] + kMoveOut;
        }
    }
    if (__any_sync(0xffffffffu, need)) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float fo[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float x = top[n][e];
#pragma unroll
                for (int sh = 4; sh < 32; sh <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, sh));
                const float m = fmaxf(st.m[n][e], x), M = fmaxf(st.M[n][e], fmaxf(x, m - kApart) + ev + 1.f - kUp);
                st.l[n][e] *= st.m[n][e] == -INFINITY ? 0.f : ex2_approx(st.m[n][e] - m);
                fo[e] = st.M[n][e] == -INFINITY ? 0.f : ex2_approx(st.M[n][e] - M);
                st.m[n][e] = m;
                st.M[n][e] = M;
            }
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) st.o[n][i][e] *= fo[e & 1];
        }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        float c[2], m[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            // (a row that has seen no token yet has no reference; a scale of zero adds nothing)
            m[e] = st.m[n][e] == -INFINITY ? 0.f : st.m[n][e];
            c[e] = ev == -INFINITY || st.M[n][e] == -INFINITY ? frac : frac * ex2_approx(m[e] + ev - st.M[n][e]);
        }
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float p = ex2_approx(fmaf(s[n][i][e], k[n][e & 1], -m[e & 1]));
                // masked: nothing, whatever the scales are (0 * -inf and NaN scales among them)
                if (MASK && at + 4 * i + (e >> 1) * pair_first<E4M3>() > lim[n][e & 1]) {
                    s[n][i][e] = 0.f;
                } else {
                    st.l[n][e & 1] += p;
                    s[n][i][e] = p * c[e & 1];
                }
            }
    }
}

// A query row as the first product's narrow operand: k step 4 c + q of lane t
// covers columns 16 (t + 4 c) + 4 q .. + 3.
template <int D>
__device__ __forceinline__ void load_row(const __nv_bfloat16* src, int t, uint32_t (&w)[D / 16][2]) {
#pragma unroll
    for (int c = 0; c < D / 64; ++c)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            uint4 v = make_uint4(0, 0, 0, 0);
            if (src) v = *reinterpret_cast<const uint4*>(src + 16 * (t + 4 * c) + 8 * half);
            w[4 * c + 2 * half][0] = v.x;
            w[4 * c + 2 * half][1] = v.y;
            w[4 * c + 2 * half + 1][0] = v.z;
            w[4 * c + 2 * half + 1][1] = v.w;
        }
}

// A bf16 row -> fp16 scaled by a power of two to below 1, its pairs in the order
// of the codes'; returns the factor that undoes the scale.
template <int D, bool E4M3>
__device__ __forceinline__ float row_to_f16(uint32_t (&w)[D / 16][2]) {
    uint32_t top = 0;
#pragma unroll
    for (int k = 0; k < D / 16; ++k)
#pragma unroll
        for (int h = 0; h < 2; ++h) top = max(top, max(w[k][h] & 0x7fffu, (w[k][h] >> 16) & 0x7fffu));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const uint32_t e = min(max(top >> 7, 1u), 252u);   // the largest element's exponent field
    const float scale = __uint_as_float((253u - e) << 23);
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t v = w[k][h];
            w[k][h] = pack_f16x2(__uint_as_float(v << 16) * scale, __uint_as_float(v & 0xffff0000u) * scale);
        }
        pair_up<E4M3>(w[k][0], w[k][1]);
    }
    return __uint_as_float((e + 1u) << 23);
}

template <int D, bool E4M3, int NT>
struct Config {
    static constexpr int KS = NT == 1 ? 2 : 1;          // warps that share a tile's tokens
    static constexpr int WARPS = kSlots * KS;           // ... that compute
    static constexpr int CONSUMERS = WARPS * 32;
    static constexpr int THREADS = CONSUMERS + 128;     // one more warp issues the copies, in a group of four of its own:
    // its registers go to the others (at launch 640 threads have 96 each, 384 have 168: 61440 and 64512 in
    // all, which is 512 x 112 + 128 x 32 and 256 x 232 + 128 x 40)
    static constexpr int REGS = NT == 1 ? 112 : 232, COPY_REGS = NT == 1 ? 32 : 40;
    static constexpr int MT = 4 / KS;                   // groups of 16 tokens to a warp
    static constexpr int STRIDE = D + 4;                // floats of a row's part: D columns, then m, l, M
    static constexpr uint32_t STAGE = kCacheBlock * D;  // bytes: an 8-bit tile's K or V, or half the open block's
};

template <int D, bool E4M3, int NT>
__global__ void __launch_bounds__(Config<D, E4M3, NT>::THREADS, 1)
cache8_attn_kernel(const __grid_constant__ Cache8Args a) {
    using C = Config<D, E4M3, NT>;
    constexpr uint32_t STAGE = C::STAGE;
    constexpr int kConsumers = C::CONSUMERS, MT = C::MT, STRIDE = C::STRIDE;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint64_t s_full[kBars], s_empty[kBars];
    __shared__ int s_place[kScan + 1], s_scan[2 * kScan / 32];
    __shared__ int s_abort;
    volatile int* abort_flag = &s_abort;

    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int g = lane >> 2, t = lane & 3;
    const int team_warps = C::KS * a.R, teams = 1 << a.lg_teams;
    const int team = warp / team_warps, in_team = warp % team_warps;   // (the copying warp: neither)
    float* slots = reinterpret_cast<float*>(smem + (size_t)teams * a.stages * STAGE);   // [teams][rows][STRIDE]
    if (tid < teams * a.stages) {
        mbar_init(&s_full[tid], 1);
        mbar_init(&s_empty[tid], team_warps);
    }
    mbar_fence_init();
    if (tid == 0) s_abort = 0;
    if (a.wait_first) pdl_wait();
    pdl_trigger();   // the next kernel may be set up; it waits for this grid before it touches memory

    // ---- the teams' shares of all tiles, or of the CTA's own head
    const Layout all(a, s_place, s_scan, tid);
    const int me = blockIdx.x, N = all.N, ctas = all.ctas;
    const bool by_head = all.by_head;
    const Deal deal(N, ctas * teams);
    const int whole_head = by_head && me < a.B * a.Hkv ? SeqTiles(a, me / a.Hkv).tiles : 0;   // the CTA's own head
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
            c.tiles = SeqTiles(a, c.b).tiles;
            if (c.tiles == 0) {
                c.left = 0;
            } else {
                const int span = span_of<Cache8Args>(c.tiles);
                c.kvh = rem / span;
                c.j = rem % span;
                if (c.j >= c.tiles) c.next_head(a);
            }
        }
        return c;
    };
    if (warp >= C::WARPS) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::COPY_REGS));
        if (warp > C::WARPS) return;
        // ---- copies: lane k serves team k, in the order the team consumes them
        Cursor next;
        next.left = 0;
        if (lane < teams) next = start_of(lane);
        uint8_t* ring = smem + (size_t)lane * a.stages * STAGE;
        uint64_t *full = s_full + lane * a.stages, *empty = s_empty + lane * a.stages;
        uint32_t stage = 0, phase = 0, armed = 0, armed_phase = 0;
        int part = 0;   // copy of the tile at `next`: 8 bits K, V; open block K, K, V, V
        long long unit = 0;
        int T = 0;
        const auto enter = [&]() {
            unit = (long long)next.b * a.Hkv + next.kvh;
            T = SeqTiles(a, next.b).T;
        };
        if (next.left > 0) enter();
        unsigned long long idle_since = 0;
        while (__any_sync(0xffffffffu, next.left > 0)) {
            bool did = false;
            if (next.left > 0 && mbar_test(&empty[stage], phase ^ 1u)) {
                did = true;
                mbar_arrive_expect_tx(&full[stage], STAGE);
                armed |= 1u << stage;
                armed_phase = (armed_phase & ~(1u << stage)) | (phase << stage);
                const bool open = (next.j + 1) * kCacheBlock > T;
                const uint8_t* src;
                if (!open) {
                    src = (part == 0 ? a.k8 : a.v8) + (unit * a.blocks + next.j) * STAGE;
                } else {
                    const __nv_bfloat16* tail = part < 2 ? a.k_tail : a.v_tail;
                    src = reinterpret_cast<const uint8_t*>(tail) +
                          ((unit * 2 + (next.j & 1)) * 2 + (part & 1)) * STAGE;
                }
                bulk_load(ring + stage * STAGE, src, STAGE, &full[stage]);
                if (++part == (open ? 4 : 2)) {
                    part = 0;
                    if (next.j + 1 < next.tiles) {
                        ++next.j;
                        --next.left;
                    } else {
                        next.next_head(a);
                        if (next.left > 0) enter();
                    }
                }
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
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::REGS));
    bool ok = true;
    {
        // ---- the team's tiles
        const uint8_t* ring = smem + (size_t)team * a.stages * STAGE;
        uint64_t *full = s_full + team * a.stages, *empty = s_empty + team * a.stages;
        const int rt = in_team / C::KS, kh = in_team % C::KS;   // the warp's query rows and part of a tile's tokens
        const int team_threads = 32 * team_warps, team_tid = 32 * in_team + lane;
        float* slot = slots + (size_t)team * a.rows * STRIDE;
        uint32_t stage = 0, phase = 0;   // the oldest stage that is not released
        const auto wait_full = [&](uint32_t ahead = 0) -> const uint8_t* {   // that stage, or the next
            uint32_t k = stage + ahead, ph = phase;
            if (k >= (uint32_t)a.stages) {
                k -= a.stages;
                ph ^= 1u;
            }
            if (!__all_sync(0xffffffffu, mbar_wait(&full[k], ph, abort_flag, a.ctl))) {
                ok = false;
                return nullptr;
            }
            return ring + k * STAGE;
        };
        const auto release = [&]() {
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[stage]);
            if (++stage == (uint32_t)a.stages) {
                stage = 0;
                phase ^= 1u;
            }
        };
        RowState<D, NT> st;
        // (the lane's tokens of a tile's first 16: see soften)
        const int key0 = 16 * (g >> 1) + 4 * MT * kh + (g & 1) * pair_step<E4M3>();
        const float unscaled = kLog2e * rsqrtf((float)D);
        Cursor at = start_of(team);
        const int share_end = team_lo(team + 1);
        while (at.left > 0) {
            const SeqTiles q(a, at.b);
            const long long unit = (long long)at.b * a.Hkv + at.kvh;
            const int j1 = min(at.tiles, at.j + at.left);   // segment: tiles [at.j, j1) of the head
            uint32_t qf[NT][D / 16][2];
            float f[NT][2];
            const auto row_of = [&](int n) -> const __nv_bfloat16* {
                const int row = 8 * (NT * rt + n) + g, i = row * a.g_inverse >> 16;
                return row < a.rows && i < q.n
                           ? a.Q + (((long long)at.b * a.Lq + i) * a.Hq + (at.kvh - i) * a.G + row) * D : nullptr;
            };
            const auto limits = [&](int (&lim)[NT][2]) {   // the last token that each of the lane's rows sees
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int row = 8 * (NT * rt + n) + 2 * t + e, i = row * a.g_inverse >> 16;
                        lim[n][e] = row < a.rows && i < q.n ? q.len + i : -1;
                    }
            };
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                load_row<D>(row_of(n), t, qf[n]);
                const float back = row_to_f16<D, E4M3>(qf[n]) * unscaled;
#pragma unroll
                for (int e = 0; e < 2; ++e) f[n][e] = __shfl_sync(0xffffffffu, back, 4 * (2 * t + e));
            }
            st.clear();
            // the segment's scales, 16 tiles at a time, one batch ahead: the keys' in lanes
            // 0 .. 15, the values' (split) in lanes 16 .. 31
            const float* scales = (lane < 16 ? a.k_scale : a.v_scale) + unit * a.blocks;
            const auto scale_of = [&](int from) {
                const int k = from + (lane & 15);
                return k < j1 && !q.open(k) ? scales[k] : 0.f;
            };
            float sc_next = scale_of(at.j + 16), sc = scale_of(at.j), ev_of;
            {
                float frac;
                split_scale(sc, frac, ev_of);
                if (lane >= 16) sc = frac;
            }
            const int full_end = min(j1, q.T / kCacheBlock);   // (the open block, if any, is the head's last)
            for (int j = at.j, it = 0; ok && j < full_end; ++j, ++it) {
                if (it == 16) {
                    it = 0;
                    sc = sc_next;
                    float frac;
                    split_scale(sc, frac, ev_of);
                    if (lane >= 16) sc = frac;
                    sc_next = scale_of(j + 16);
                }
                const int base = j * kCacheBlock;
                float s[NT][MT][4];
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < MT; ++i)
#pragma unroll
                        for (int e = 0; e < 4; ++e) s[n][i][e] = 0.f;
                const float ks = __shfl_sync(0xffffffffu, sc, it);
                const float frac = __shfl_sync(0xffffffffu, sc, 16 + it), ev = __shfl_sync(0xffffffffu, ev_of, 16 + it);
                const uint8_t* kt = wait_full();
                if (!kt) break;
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    const uint8_t* r0 = kt + (key0 + 4 * i) * D + 16 * t;
                    const uint8_t* r1 = r0 + pair_first<E4M3>() * D;
#pragma unroll
                    for (int c = 0; c < D / 64; ++c) {
                        const uint4 x = *reinterpret_cast<const uint4*>(r0 + 64 * c);
                        const uint4 y = *reinterpret_cast<const uint4*>(r1 + 64 * c);
                        const uint32_t x4[4] = {x.x, x.y, x.z, x.w}, y4[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            uint32_t w[4];
                            codes_to_f16<E4M3>(x4[k], w[0], w[2]);
                            codes_to_f16<E4M3>(y4[k], w[1], w[3]);
#pragma unroll
                            for (int n = 0; n < NT; ++n)
                                mma_f16(s[n][i], w, qf[n][4 * c + k][0], qf[n][4 * c + k][1]);
                        }
                    }
                }
                release();
                // (the first query row sees tokens up to len: tiles before need no mask)
                int lim[NT][2] = {};
                if (base + kCacheBlock - 1 > q.len) {
                    limits(lim);
                    soften<D, NT, MT, E4M3, true>(s, f, ks, base + key0, lim, frac, ev, st);
                } else {
                    soften<D, NT, MT, E4M3, false>(s, f, ks, base + key0, lim, frac, ev, st);
                }
                uint32_t pf[NT][MT][2];
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < MT; ++i)
#pragma unroll
                        for (int x = 0; x < 2; ++x)
                            pf[n][i][x] = transpose8(pack_f16x2(s[n][i][2 * x], s[n][i][2 * x + 1]));
                const uint8_t* vt = wait_full();
                if (!vt) break;
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    const uint8_t* r = vt + (16 * i + g) * kCacheBlock + 16 * t + 4 * MT * kh;
                    uint32_t x4[MT], y4[MT];
                    if constexpr (MT == 4) {
                        *reinterpret_cast<uint4*>(x4) = *reinterpret_cast<const uint4*>(r);
                        *reinterpret_cast<uint4*>(y4) = *reinterpret_cast<const uint4*>(r + 8 * kCacheBlock);
                    } else {
                        *reinterpret_cast<uint2*>(x4) = *reinterpret_cast<const uint2*>(r);
                        *reinterpret_cast<uint2*>(y4) = *reinterpret_cast<const uint2*>(r + 8 * kCacheBlock);
                    }
#pragma unroll
                    for (int k = 0; k < MT; ++k) {
                        uint32_t w[4];
                        codes_to_f16<E4M3>(x4[k], w[0], w[2]);
                        codes_to_f16<E4M3>(y4[k], w[1], w[3]);
#pragma unroll
                        for (int n = 0; n < NT; ++n) mma_f16(st.o[n][i], w, pf[n][k][0], pf[n][k][1]);
                    }
                }
                release();
            }
            while (ok && j1 > full_end) {   // (once: `break` where a wait ran out)
                const int base = full_end * kCacheBlock;
                float s[NT][MT][4];
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < MT; ++i)
#pragma unroll
                        for (int e = 0; e < 4; ++e) s[n][i][e] = 0.f;
                // the open block, in bf16: keys [64][D], values [D][64], each in two stages
                uint32_t qb[NT][D / 16][2];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    load_row<D>(row_of(n), t, qb[n]);
                }
                const uint8_t* k0 = wait_full();
                if (!k0) break;
                const uint8_t* k1 = wait_full(1);
                if (!k1) break;
                const uint8_t* half = g < 4 ? k0 : k1 - 32 * D * 2;   // tokens 16 (g / 2) ..: first or second 32
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    const uint8_t* r0 = half + (key0 + 4 * i) * D * 2 + 32 * t;
                    const uint8_t* r1 = r0 + pair_first<E4M3>() * D * 2;
#pragma unroll
                    for (int c = 0; c < D / 64; ++c)
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const uint4 x = *reinterpret_cast<const uint4*>(r0 + 128 * c + 16 * k);
                            const uint4 y = *reinterpret_cast<const uint4*>(r1 + 128 * c + 16 * k);
                            const uint32_t w0[4] = {x.x, y.x, x.y, y.y}, w1[4] = {x.z, y.z, x.w, y.w};
#pragma unroll
                            for (int n = 0; n < NT; ++n) {
                                const int ko = 4 * c + 2 * k;
                                mma_bf16(s[n][i], w0, qb[n][ko][0], qb[n][ko][1]);
                                mma_bf16(s[n][i], w1, qb[n][ko + 1][0], qb[n][ko + 1][1]);
                            }
                        }
                }
                release();
                release();
                float fo[NT][2];
#pragma unroll
                for (int n = 0; n < NT; ++n) fo[n][0] = fo[n][1] = unscaled;
                int lim[NT][2];
                limits(lim);
                soften<D, NT, MT, E4M3, true>(s, fo, 1.f, base + key0, lim, 1.f, 0.f, st);
                // each weight as two bf16 parts
                uint32_t wh[NT][MT][2], wl[NT][MT][2];
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < MT; ++i)
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            const float p0 = s[n][i][2 * x], p1 = s[n][i][2 * x + 1];
                            const uint32_t h = pack_bf16x2(p0, p1);
                            wh[n][i][x] = transpose8(h);
                            wl[n][i][x] = transpose8(pack_bf16x2(p0 - __uint_as_float(h << 16),
                                                                 p1 - __uint_as_float(h & 0xffff0000u)));
                        }
                // slots past the sequence's end hold whatever was there before: zero, not 0 * NaN
                uint32_t keep[2 * MT];
#pragma unroll
                for (int k = 0; k < 2 * MT; ++k) {
                    const int over = q.T - (base + 16 * t + 4 * MT * kh + 2 * k);
                    keep[k] = over > 1 ? 0xffffffffu : (over == 1 ? 0x0000ffffu : 0u);
                }
                const uint8_t* v0 = wait_full();
                if (!v0) break;
                const uint8_t* v1 = wait_full(1);
                if (!v1) break;
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    const uint8_t* r = (i < D / 32 ? v0 : v1) + (16 * (i % (D / 32)) + g) * kCacheBlock * 2 +
                                       32 * t + 8 * MT * kh;
#pragma unroll
                    for (int k = 0; k < MT / 2; ++k) {
                        uint4 x = *reinterpret_cast<const uint4*>(r + 16 * k);
                        uint4 y = *reinterpret_cast<const uint4*>(r + 8 * kCacheBlock * 2 + 16 * k);
                        x.x &= keep[4 * k];
                        x.y &= keep[4 * k + 1];
                        x.z &= keep[4 * k + 2];
                        x.w &= keep[4 * k + 3];
                        y.x &= keep[4 * k];
                        y.y &= keep[4 * k + 1];
                        y.z &= keep[4 * k + 2];
                        y.w &= keep[4 * k + 3];
                        pair_up<E4M3>(x.x, x.y);
                        pair_up<E4M3>(x.z, x.w);
                        pair_up<E4M3>(y.x, y.y);
                        pair_up<E4M3>(y.z, y.w);
                        const uint32_t w0[4] = {x.x, y.x, x.y, y.y}, w1[4] = {x.z, y.z, x.w, y.w};
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            mma_bf16(st.o[n][i], w0, wh[n][2 * k][0], wh[n][2 * k][1]);
                            mma_bf16(st.o[n][i], w0, wl[n][2 * k][0], wl[n][2 * k][1]);
                            mma_bf16(st.o[n][i], w1, wh[n][2 * k + 1][0], wh[n][2 * k + 1][1]);
                            mma_bf16(st.o[n][i], w1, wl[n][2 * k + 1][0], wl[n][2 * k + 1][1]);
                        }
                    }
                }
                release();
                release();
                break;
            }

            // ---- the segment's rows, merged where two warps shared the tokens
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int sh = 4; sh < 32; sh <<= 1)
                        st.l[n][e] += __shfl_xor_sync(0xffffffffu, st.l[n][e], sh);
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
            // A head of the team's alone is finished; else its part is left in global
            // memory for the merge kernel, or, of the CTA's own head, in shared memory:
            // the first warp's rows in the slot, the second's in the ring, which is empty.
            const bool whole = at.j == 0 && j1 == at.tiles, final = at.left <= span_of<Cache8Args>(at.tiles) - at.j;
            const bool apart = C::KS == 2 && by_head && !whole;
            float* to = whole || by_head
                            ? slot : part_of<D>(a, deal, me * teams + team, share_end - at.left - at.j);
            if (C::KS == 2 && !apart && kh == 1) put(slot);
            if (C::KS == 1 || (apart && kh == 0)) put(to);
            ok = named_bar_and(1 + team, team_threads, ok && !*abort_flag);
            if (!ok) break;
            if (apart) {
                if (kh == 1) put(reinterpret_cast<float*>(smem + (size_t)team * a.stages * STAGE));
            } else if constexpr (C::KS == 2) {
                if (kh == 0) {
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int row = 8 * (NT * rt + n) + 2 * t + e;
                            if (row >= a.rows) continue;
                            const float* from = slot + row * STRIDE;
                            const float4 x = *reinterpret_cast<const float4*>(from + D);
                            const float m = fmaxf(st.m[n][e], x.x), M = fmaxf(st.M[n][e], x.z);
                            const float oa = part_weight(st.M[n][e], M), ob = part_weight(x.z, M);
                            st.l[n][e] = st.l[n][e] * part_weight(st.m[n][e], m) + x.y * part_weight(x.x, m);
                            st.m[n][e] = m;
                            st.M[n][e] = M;
#pragma unroll
                            for (int i = 0; i < D / 16; ++i) {
                                st.o[n][i][e] = st.o[n][i][e] * oa + from[16 * i + g] * ob;
                                st.o[n][i][2 + e] = st.o[n][i][2 + e] * oa + from[16 * i + 8 + g] * ob;
                            }
                        }
                    __syncwarp();
                    put(to);
                }
                if (whole || !final) named_bar_sync(1 + team, team_threads);   // (the slot may be written again)
            }
            if (whole) {
                if (a.gate_mode != GSDPA_GATE_NONE) pdl_wait();   // the gate logits
                for (int idx = team_tid; idx < a.rows * (D / 4); idx += team_threads) {
                    const int row = idx / (D / 4), col = 4 * (idx % (D / 4));
                    const float* from = slot + row * STRIDE;
                    const float4 x = *reinterpret_cast<const float4*>(from + D);
                    finish<D>(a, at.b, at.kvh, q.n, row, col, out_scale(x.x, x.y, x.z),
                              *reinterpret_cast<const float4*>(from + col), gate_of<D>(a, at.b, at.kvh, q.n, row, col));
                }
                if (!final) named_bar_sync(1 + team, team_threads);
            }
            at.next_head(a);
        }
    }

    pdl_wait();   // the gate logits; and what follows on the stream may rely on the gate kernel having ended
    const int parts = min(whole_head, teams);   // (of the CTA's own head: more than one, or it is done)
    if (by_head && named_bar_and(kSlots + 1, kConsumers, ok && !*abort_flag) && parts > 1) {
        const int items = a.rows * (D / 4), b = me / a.Hkv, n = SeqTiles(a, b).n;
        // A thread has four columns of a row; its parts are split over lanes that
        // would be idle (whole warps: items come in sixteens).
        int lg = 0;
        while (lg < 3 && (items << (lg + 1)) <= kConsumers) ++lg;
        for (int idx = tid; idx < items << lg; idx += kConsumers) {
            const int item = idx >> lg, row = item / (D / 4), col = 4 * (item % (D / 4));
            const float4 gate = gate_of<D>(a, b, me % a.Hkv, n, row, col);
            Sums r;
            r.add(idx & ((1 << lg) - 1), parts * C::KS, 1 << lg, D, col, [&](int i) {
                return (i < parts ? slots + (size_t)i * a.rows * STRIDE
                                  : reinterpret_cast<const float*>(smem + (size_t)(i - parts) * a.stages * STAGE)) +
                       row * STRIDE;
            });
            for (int sh = 1; sh < 1 << lg; sh <<= 1) r.join_lane(sh);
            if ((idx & ((1 << lg) - 1)) == 0)
                finish<D>(a, b, me % a.Hkv, n, row, col, out_scale(r.m, r.l, r.M), r.o, gate);
        }
    }

    // rows that no sequence has a token for are zero
    for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
        const SeqRange r = seq_range(a.lens, a.n_new, b, a.Lq, a.capacity);
        if (!r.ok && tid == 0) atomicOr(a.ctl.err, ERR_CACHE_RANGE);
        const long long from = ((long long)b * a.Lq + r.n) * a.Hq * D / 8, to = ((long long)b + 1) * a.Lq * a.Hq * D / 8;
        for (long long i = from + tid; i < to; i += kConsumers)
            reinterpret_cast<uint4*>(a.O)[i] = make_uint4(0, 0, 0, 0);
    }
}

// Shared memory and ring of one problem.
struct Shape {
    int NT, R, stages;
    uint32_t smem;
};
Shape shape_of(int rows, int D) {
    Shape s;
    s.NT = rows <= 8 ? 1 : 2;
    s.R = rows <= 16 ? 1 : (rows <= 32 ? 2 : (rows <= 64 ? 4 : 8));
    const uint32_t merge = (uint32_t)(kSlots / s.R * rows * (D + 4)) * 4;
    const uint32_t per_stage = (uint32_t)(kSlots / s.R) * kCacheBlock * D;
    // as many copies in flight as fit, up to 192 KB (an open block holds two stages at once)
    s.stages = (int)((kSmemMax - merge) / per_stage);
    const int most = (int)(196608 / per_stage);
    if (s.stages > most) s.stages = most;
    if (s.stages > kMaxStages) s.stages = kMaxStages;
    if (s.stages > kBars * s.R / kSlots) s.stages = kBars * s.R / kSlots;
    s.smem = (uint32_t)s.stages * per_stage + merge;
    return s;
}

struct Cache8Plan {
    Problem p{};
    WorkspacePlan w;   // the gate kernel's part
    size_t part = 0, total = 0;
};

int plan_cache8(const gsdpa_cache8* c, int Lq, int d_model, int Hq, int gate_mode, Cache8Plan* out) {
    int st = validate_cache8(c);
    if (st != GSDPA_OK) return st;
    if (Lq < 0 || Hq < 1 || Hq % c->H_kv != 0) return GSDPA_ERR_INVALID_ARG;
    if (gate_mode < GSDPA_GATE_NONE || gate_mode > GSDPA_GATE_ELEMENTWISE) return GSDPA_ERR_INVALID_ARG;
    if (gate_mode != GSDPA_GATE_NONE && d_model < 1) return GSDPA_ERR_INVALID_ARG;
    if (gate_mode != GSDPA_GATE_NONE && d_model % 8 != 0) return GSDPA_ERR_UNSUPPORTED;
    if (gate_mode == GSDPA_GATE_HEADWISE && Hq % 8 != 0) return GSDPA_ERR_UNSUPPORTED;
    const long long rows = (long long)(Hq / c->H_kv) * Lq;
    if (rows > kMaxRows) return GSDPA_ERR_UNSUPPORTED;
    // (places are counted in 32 bits)
    if ((long long)c->B * c->H_kv * (c->capacity / kCacheBlock + Cache8Args::kSwitch) > 0x7fffffffLL) return GSDPA_ERR_UNSUPPORTED;
    if ((long long)c->B * Lq > 0x7fffffffLL / 8 || (long long)c->B * c->H_kv > 0x7fffffffLL - 2 * kMaxCtas)
        return GSDPA_ERR_UNSUPPORTED;
    if (c->B == 0 || Lq == 0) return GSDPA_OK;   // an empty problem: nothing to plan
    Cache8Plan& o = *out;
    Problem& p = o.p;
    p.B = c->B;
    p.Lq = Lq;
    p.Lk = c->capacity;
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
    o.part = take(part * plan_sms() * 2 * (kSlots / shape_of((int)rows, c->d_k).R));
    o.total = off;
    return GSDPA_OK;
}

template <int D, bool E4M3, int NT>
cudaError_t launch(const Cache8Args& a, const Shape& sh, unsigned grid, cudaStream_t s) {
    static PerDeviceSetup setup;
    const cudaError_t e = setup_once_per_device(setup, [](int&) {
        return cudaFuncSetAttribute(cache8_attn_kernel<D, E4M3, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    (int)kSmemMax);
    });
    if (e != cudaSuccess) return e;
    return launch_dependent(cache8_attn_kernel<D, E4M3, NT>, dim3(grid), dim3(Config<D, E4M3, NT>::THREADS), sh.smem, s,
                            a);
}
template <int D, bool E4M3>
cudaError_t launch(const Cache8Args& a, const Shape& sh, unsigned grid, cudaStream_t s) {
    return sh.NT == 1 ? launch<D, E4M3, 1>(a, sh, grid, s) : launch<D, E4M3, 2>(a, sh, grid, s);
}

}  // namespace
}  // namespace gsdpa

using namespace gsdpa;

extern "C" {

size_t gsdpa_cache8_workspace_bytes(const gsdpa_cache8* cache, int L_q, int d_model, int H_q, int gate_mode) {
    Cache8Plan pl;
    if (plan_cache8(cache, L_q, d_model, H_q, gate_mode, &pl) != GSDPA_OK) return (size_t)-1;
    if (cache->B == 0 || L_q == 0) return 0;
    return pl.total;
}

int gated_sdpa_cache8(const void* X, const void* Q, const gsdpa_cache8* cache, const int* lens, const int* n_new,
                      const void* W_g, void* O, int L_q, int d_model, int H_q, int gate_mode, void* workspace,
                      size_t workspace_bytes, void* stream) {
    Cache8Plan pl;
    int st = plan_cache8(cache, L_q, d_model, H_q, gate_mode, &pl);
    if (st != GSDPA_OK) return st;
    if (cache->B == 0 || L_q == 0) return GSDPA_OK;
    if ((st = validate_cache8_pointers(cache)) != GSDPA_OK) return st;
    const bool gated = gate_mode != GSDPA_GATE_NONE;
    if (!Q || !O || !lens || (gated && (!X || !W_g))) return GSDPA_ERR_INVALID_ARG;
    const auto off16 = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; };
    if (off16(Q) || off16(O) || (gated && (off16(X) || off16(W_g)))) return GSDPA_ERR_ALIGNMENT;
    if ((reinterpret_cast<uintptr_t>(lens) & 3u) || (reinterpret_cast<uintptr_t>(n_new) & 3u))
        return GSDPA_ERR_ALIGNMENT;
    Runtime rt;
    int major = 0, minor = 0;
    if (!current_runtime(&rt, &major, &minor)) return GSDPA_ERR_LAUNCH;
    if (!(major == 10 && minor == 3) || !encode_tiled_fn()) return GSDPA_ERR_UNSUPPORTED;
    if (!workspace || workspace_bytes < pl.total) return GSDPA_ERR_WORKSPACE;
    if (reinterpret_cast<uintptr_t>(workspace) & 255u) return GSDPA_ERR_ALIGNMENT;
    char* ws = static_cast<char*>(workspace);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
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

    Cache8Args a;
    a.Q = static_cast<const __nv_bfloat16*>(Q);
    a.O = static_cast<__nv_bfloat16*>(O);
    a.lens = lens;
    a.n_new = n_new;
    a.k8 = static_cast<const uint8_t*>(cache->k8);
    a.v8 = static_cast<const uint8_t*>(cache->v8);
    a.k_scale = cache->k_scale;
    a.v_scale = cache->v_scale;
    a.k_tail = static_cast<const __nv_bfloat16*>(cache->k_tail);
    a.v_tail = static_cast<const __nv_bfloat16*>(cache->v_tail);
    a.B = cache->B;
    a.Lq = L_q;
    a.Hq = H_q;
    a.Hkv = cache->H_kv;
    a.G = H_q / cache->H_kv;
    a.g_inverse = (65536 + a.G - 1) / a.G;
    a.rows = a.G * L_q;
    a.blocks = cache->capacity / kCacheBlock;
    a.capacity = cache->capacity;
    const Shape sh = shape_of(a.rows, cache->d_k);
    a.R = sh.R;
    a.lg_teams = sh.R == 1 ? 3 : (sh.R == 2 ? 2 : (sh.R == 4 ? 1 : 0));
    a.stages = sh.stages;
    a.gate_part = gated ? reinterpret_cast<const float*>(ws + pl.w.gate_part) : nullptr;
    a.gate_splits = pl.w.gate_splits;
    a.gate_cols = pl.w.gate_cols;
    a.gate_mode = gate_mode;
    a.part = reinterpret_cast<float*>(ws + pl.part);
    a.wait_first = launched ? 0 : 1;
    a.ctl.err = rt.err;
    a.ctl.limit_ns = rt.limit_ns;
    // one CTA per SM, fewer where a full cache would not give each its tiles
    const long long most = (long long)a.B * a.Hkv * ((a.blocks + kSlots / a.R - 1) / (kSlots / a.R));
    long long grid = sms;   // (no fewer than the heads, where those fit)
    if (grid > most) grid = most;
    a.ctas = (int)grid;
    const bool whole = a.blocks <= kWholeTiles << a.lg_teams && (long long)a.B * a.Hkv <= grid;
    a.whole_tiles = (whole ? kWholeTiles : kFewTiles) << a.lg_teams;
    const bool e4m3 = cache->kind == GSDPA_CACHE_E4M3;
    if (cache->d_k == 128)
        e = e4m3 ? launch<128, true>(a, sh, (unsigned)grid, s) : launch<128, false>(a, sh, (unsigned)grid, s);
    else
        e = e4m3 ? launch<64, true>(a, sh, (unsigned)grid, s) : launch<64, false>(a, sh, (unsigned)grid, s);
    // (Not a CTA for every SM: the SMs that are done first take them all, and they are
    // set up when the last are done.)
    if (e == cudaSuccess && !whole)
        e = launch_dependent(cache->d_k == 128 ? cache_merge_kernel<128, Cache8Args> : cache_merge_kernel<64, Cache8Args>, dim3((unsigned)(sms - sms / 8)),
                             dim3(kMergeThreads), 0, s, a);
    return e == cudaSuccess ? GSDPA_OK : GSDPA_ERR_LAUNCH;
}

}  // extern "C"
