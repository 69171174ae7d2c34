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
// cores with mma.sync: 16 query rows (heads of the group x new tokens) against
// 8 tokens or columns, fp16 operands, fp32 sums. (tcgen05 needs 64 or 128
// rows on one side, operands in shared memory in one of its own types, and
// leaves the scores in tensor memory; here the rows are few and the 8-bit codes
// have to pass through registers anyway, to become fp16.) int8 and e4m3 codes
// are exact in fp16; q, a bf16 row scaled by a power of two to below 1, too
// (elements under 2^-14 of the row's largest lose bits that weigh less than
// 2^-24 of it). The weights are rounded to fp16 (11 bits) for the second product, to
// bf16 for the open block's, whose values may exceed fp16's range.
//
// Two running references, both only for range: m for the sum of weights, and
// M for the outputs, which carry the value scales: a block adds
// (p c) V8 with c = vs 2^(m - M), so that a block of large values that the
// query hardly looks at cannot push the others' products out of fp16's range.
// They move when a tile exceeds them by 2^8 (rarely after the first tile).
//
// Tile = one block: K8 [64][d_k] and V8 [d_k][64], each 64 d_k contiguous bytes,
// brought by cp.async.bulk. The tiles of all sequences and K/V heads form one
// sequence of tiles that is cut evenly over the CTAs (lengths are read on the
// device: no length, however uneven, leaves SMs idle). In a CTA, 8 warps work on 8 / R tiles at a
// time, R warps to a tile (R = 1 up to 16 query rows, then 2, 4, 8); each such
// team streams its own tiles through a ring of its own. At the end of a K/V
// head's tiles the warps merge in shared memory; a head whose tiles are split
// over CTAs is merged by the CTA that arrives last (an atomic counter; the
// partial results are added in a fixed order). No CTA waits for another.
//
// The order of the tokens inside a tile's products is chosen so that no
// element moves between lanes: lane (g, t) of a warp holds, after the first
// product, the scores of tokens 16 t .. 16 t + 15, which is what it needs as
// the second product's weights, and 16 consecutive bytes of a value column are
// its share of that product's other operand.
#include "cache8_internal.h"

#include <cuda_fp16.h>

namespace gsdpa {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxRows = 128;        // query rows (heads of a group x new tokens) per K/V head
constexpr int kMaxStages = 16;       // ring stages per team
constexpr int kMinTiles = 8;         // fewest tiles worth a CTA
constexpr int kBars = 64;            // ring stages of all teams
constexpr uint32_t kSmemMax = 232448 - 1536;   // dynamic: what a CTA may have, less barriers and a few words
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kMove = 8.0f;

struct Cache8Args {
    const __nv_bfloat16* Q;          // [B, Lq, Hq, D]
    __nv_bfloat16* O;
    const int *lens, *n_new;
    const uint8_t *k8, *v8;
    const float *k_scale, *v_scale;
    const __nv_bfloat16 *k_tail, *v_tail;
    int B, Lq, Hq, Hkv, G;           // G = Hq / Hkv
    int rows;                        // G * Lq
    int blocks, capacity;
    int R, stages;                   // warps to a tile; ring stages per team
    int merge_rows;                  // rows of a warp's part of the merge buffer
    const float* gate_part;          // [gate_splits, B * Lq, gate_cols] or null
    int gate_splits, gate_cols, gate_mode;
    float* part_o;                   // [CTAs][2][rows][D]
    float* part_s;                   // [CTAs][2][rows][4]: m, l, M
    int* counters;                   // [B * Hkv]
    WaitCtl ctl;
};

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     smem_u32(dst)),
                 "l"(src), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// 4 codes -> two fp16 pairs (codes 0, 1 and codes 2, 3), exactly.
template <bool E4M3>
__device__ __forceinline__ void codes_to_f16(uint32_t w, uint32_t& p01, uint32_t& p23) {
    if constexpr (E4M3) {
        asm("{\n\t.reg .b16 lo, hi;\n\t"
            "mov.b32 {lo, hi}, %2;\n\t"
            "cvt.rn.f16x2.e4m3x2 %0, lo;\n\t"
            "cvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
            : "=r"(p01), "=r"(p23)
            : "r"(w));
    } else {
        // code + 128 in the low bits of the fp16 number 1024, then 1152 taken off
        const uint32_t u = w ^ 0x80808080u;
        const __half2 off = __half2half2(__ushort_as_half(0x6480));   // 1152
        uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
        __half2 x = __hsub2(*reinterpret_cast<__half2*>(&a), off), y = __hsub2(*reinterpret_cast<__half2*>(&b), off);
        p01 = *reinterpret_cast<uint32_t*>(&x);
        p23 = *reinterpret_cast<uint32_t*>(&y);
    }
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// 1 / (1 + e^-x), accurate to a few units of float32's last place.
__device__ __forceinline__ float sigmoid(float x) { return __fdividef(1.f, 1.f + __expf(-x)); }

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
};

// A place in the sequence of all tiles. (Where tiles are left a sequence with
// tiles follows; lengths that change during the call, which they must not, end
// the walk instead of leading it out of the batch.)
struct Cursor {
    int b, kvh, j, tiles;
    long long left;   // tiles of the CTA's range from here on
    __device__ __forceinline__ void skip(const Cache8Args& a, long long n) {
        left -= n;
        if (left <= 0) return;
        long long at = j + n;
        while (at >= tiles) {
            at -= tiles;
            if (++kvh == a.Hkv) {
                kvh = 0;
                do {
                    if (++b >= a.B) {
                        left = 0;
                        return;
                    }
                    tiles = SeqTiles(a, b).tiles;
                } while (tiles == 0);
            }
        }
        j = (int)at;
    }
};

// What a warp keeps of its 16 query rows; lane (g, t) has rows g and g + 8.
template <int D>
struct RowState {
    float o[D / 8][4];   // columns 8 i + 2 t, + 1 of rows g, g + 8
    float m[2], l[2], M[2];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            m[r] = M[r] = -INFINITY;
            l[r] = 0.f;
        }
    }
};

// The scores of a tile (log2 units, tokens masked past lim) become weights:
// s holds p c on return, l and the references are brought up to date. vs is
// the tile's value scale.
template <int D>
__device__ __forceinline__ void soften(float (&s)[8][4], const float (&f)[2], bool mask, int base, const int (&lim)[2],
                                       float vs, int t, RowState<D>& st) {
    float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            s[i][e] *= f[e >> 1];
            if (mask && base + 16 * t + 2 * i + (e & 1) > lim[e >> 1]) s[i][e] = -INFINITY;
            top[e >> 1] = fmaxf(top[e >> 1], s[i][e]);
        }
    // vs = frac 2^e
    float frac = vs, ev = 0.f;
    if (vs < 8.6736174e-19f) {   // 2^-60: out of the subnormal numbers
        frac *= 1.152921504606847e18f;
        ev = -60.f;
    }
    const uint32_t bits = __float_as_uint(frac);
    if (vs > 0.f && (bits >> 23) < 255u) {
        ev += (float)((int)(bits >> 23) - 127);
        frac = __uint_as_float((bits & 0x7fffffu) | 0x3f800000u);
    }
    bool need = false;
    float tv[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 1));
        top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 2));
        tv[r] = vs > 0.f ? top[r] + ev + 1.f : -INFINITY;
        need = need || top[r] > st.m[r] + kMove || tv[r] > st.M[r] + kMove;
    }
    if (__any_sync(0xffffffffu, need)) {
        float fo[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const float m = fmaxf(st.m[r], top[r]), M = fmaxf(st.M[r], tv[r]);
            st.l[r] *= st.m[r] == -INFINITY ? 0.f : ex2_approx(st.m[r] - m);
            fo[r] = st.M[r] == -INFINITY ? 0.f : ex2_approx(st.M[r] - M);
            st.m[r] = m;
            st.M[r] = M;
        }
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) st.o[i][e] *= fo[e >> 1];
    }
    float c[2], m[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        // (a row that has seen no token yet has no reference; a scale of zero adds nothing)
        m[r] = st.m[r] == -INFINITY ? 0.f : st.m[r];
        c[r] = vs == 0.f ? 0.f : frac * (st.M[r] == -INFINITY ? 1.f : ex2_approx(m[r] + ev - st.M[r]));
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float p = ex2_approx(s[i][e] - m[e >> 1]);
            st.l[e >> 1] += p;
            s[i][e] = p * c[e >> 1];
        }
    if (mask) {   // a block with a NaN scale must not reach the rows that see none of it
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (base + 16 * t + 2 * i + (e & 1) > lim[e >> 1]) s[i][e] = 0.f;
    }
}

// Query rows as the first product's operand: k step (c, q) of lane t covers
// columns 16 c + 4 q .. + 3 of its piece c (t, then t + 4 when d_k = 128).
template <int D>
__device__ __forceinline__ void load_rows(const __nv_bfloat16* const (&src)[2], int t, uint32_t (&w)[D / 16][4]) {
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int c = 0; c < D / 64; ++c)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                uint4 v = make_uint4(0, 0, 0, 0);
                if (src[r]) v = *reinterpret_cast<const uint4*>(src[r] + 16 * (t + 4 * c) + 8 * half);
                w[4 * c + 2 * half][r] = v.x;
                w[4 * c + 2 * half][2 + r] = v.y;
                w[4 * c + 2 * half + 1][r] = v.z;
                w[4 * c + 2 * half + 1][2 + r] = v.w;
            }
}

// bf16 rows -> fp16 rows scaled by a power of two to below 1; back[r] undoes it.
template <int D>
__device__ __forceinline__ void rows_to_f16(uint32_t (&w)[D / 16][4], float (&back)[2]) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        uint32_t top = 0;
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t v = w[k][2 * h + r];
                top = max(top, max(v & 0x7fffu, (v >> 16) & 0x7fffu));
            }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const uint32_t e = min(max(top >> 7, 1u), 252u);   // the largest element's exponent field
        const float scale = __uint_as_float((253u - e) << 23);
        back[r] = __uint_as_float((e + 1u) << 23);
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t v = w[k][2 * h + r];
                w[k][2 * h + r] = pack_f16x2(__uint_as_float(v << 16) * scale, __uint_as_float(v & 0xffff0000u) * scale);
            }
    }
}

// Output columns [col, col + 4) of query row `row`: the sums become the
// attention's output, gated and stored.
template <int D>
__device__ __forceinline__ void finish(const Cache8Args& a, int b, int kvh, int n, int row, int col, float m, float l,
                                       float M, const float4& o) {
    const int i = row / a.G;
    if (i >= n) return;
    const int h = kvh * a.G + row % a.G;
    // (a row whose weights leave nothing is zero)
    const float k = l > 0.f || l != l ? (M == -INFINITY ? 0.f : ex2_approx(M - m)) / l : 0.f;
    float y[4] = {o.x * k, o.y * k, o.z * k, o.w * k};
    const long long token = (long long)b * a.Lq + i;
    if (a.gate_mode != GSDPA_GATE_NONE) {
        const bool per_col = a.gate_mode == GSDPA_GATE_ELEMENTWISE;
        const float* gp = a.gate_part + token * a.gate_cols + (per_col ? (long long)h * D + col : h);
        const long long step = (long long)a.B * a.Lq * a.gate_cols;
        float gl[4] = {0.f, 0.f, 0.f, 0.f};
        for (int sp = 0; sp < a.gate_splits; ++sp) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (per_col || e == 0) gl[e] += gp[sp * step + e];
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] *= sigmoid(per_col ? gl[e] : gl[0]);
    }
    *reinterpret_cast<uint2*>(a.O + (token * a.Hq + h) * D + col) =
        make_uint2(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]));
}

// One more (m, l, M, o) into a running merge.
__device__ __forceinline__ void merge(float& m, float& l, float& M, float4& o, float m2, float l2, float M2,
                                      const float4& o2) {
    const float mn = fmaxf(m, m2), Mn = fmaxf(M, M2);
    const float a = m == -INFINITY ? 0.f : ex2_approx(m - mn), b = m2 == -INFINITY ? 0.f : ex2_approx(m2 - mn);
    const float c = M == -INFINITY ? 0.f : ex2_approx(M - Mn), d = M2 == -INFINITY ? 0.f : ex2_approx(M2 - Mn);
    l = l * a + l2 * b;
    o.x = o.x * c + o2.x * d;
    o.y = o.y * c + o2.y * d;
    o.z = o.z * c + o2.z * d;
    o.w = o.w * c + o2.w * d;
    m = mn;
    M = Mn;
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(kThreads, 1) cache8_attn_kernel(const Cache8Args a) {
    constexpr uint32_t STAGE = kCacheBlock * D;   // bytes: an 8-bit tile's K or V, or half the open block's
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint64_t s_full[kBars], s_empty[kBars];
    __shared__ long long s_scan[kWarps];
    __shared__ int s_b, s_rem, s_last;
    __shared__ int s_abort;
    volatile int* abort_flag = &s_abort;

    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int g = lane >> 2, t = lane & 3;
    const int teams = kWarps / a.R, team = warp / a.R, rt = warp % a.R;
    const bool leader = rt == 0 && lane == 0;
    uint8_t* ring = smem + (size_t)team * a.stages * STAGE;
    float* red_o = reinterpret_cast<float*>(smem + (size_t)teams * a.stages * STAGE);   // [8 warps][merge_rows][D]
    float* red_s = red_o + kWarps * a.merge_rows * D;                                   // [8 warps][merge_rows][4]
    uint64_t* full = s_full + team * a.stages;
    uint64_t* empty = s_empty + team * a.stages;
    if (leader) {
        for (int k = 0; k < a.stages; ++k) {
            mbar_init(&full[k], 1);
            mbar_init(&empty[k], a.R);
        }
        mbar_fence_init();
    }
    if (tid == 0) s_abort = 0;

    // ---- the CTA's share of all tiles: [lo, hi) of N
    const int per = (a.B + kThreads - 1) / kThreads;
    long long mine = 0;
    for (int b = tid * per; b < min(a.B, (tid + 1) * per); ++b) mine += SeqTiles(a, b).tiles;
    mine *= a.Hkv;
    long long scan = mine;
#pragma unroll
    for (int sh = 1; sh < 32; sh <<= 1) {
        const long long up = __shfl_up_sync(0xffffffffu, scan, sh);
        if (lane >= sh) scan += up;
    }
    if (lane == 31) s_scan[warp] = scan;
    __syncthreads();
    long long N = 0, before = scan - mine;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += s_scan[w];
        N += s_scan[w];
    }
    long long ctas = (N + kMinTiles - 1) / kMinTiles;
    ctas = ctas < 1 ? 1 : (ctas > (long long)gridDim.x ? (long long)gridDim.x : ctas);
    const long long me = blockIdx.x;
    const long long lo = me < ctas ? N * me / ctas : N, hi = me < ctas ? N * (me + 1) / ctas : N;
    if (lo < hi && lo >= before && lo < before + mine) {
        long long at = lo - before;
        int b = tid * per;
        long long in_seq = (long long)SeqTiles(a, b).tiles * a.Hkv;
        while (at >= in_seq && b + 1 < a.B) {
            at -= in_seq;
            in_seq = (long long)SeqTiles(a, ++b).tiles * a.Hkv;
        }
        s_b = b;
        s_rem = (int)at;   // (below H_kv * capacity / 64, checked on the host)
    }
    // rows that no sequence has a token for are zero
    for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
        const SeqRange r = seq_range(a.lens, a.n_new, b, a.Lq, a.capacity);
        if (!r.ok && tid == 0) atomicOr(a.ctl.err, ERR_CACHE_RANGE);
        const long long from = ((long long)b * a.Lq + r.n) * a.Hq * D / 8, to = ((long long)b + 1) * a.Lq * a.Hq * D / 8;
        for (long long i = from + tid; i < to; i += kThreads)
            reinterpret_cast<uint4*>(a.O)[i] = make_uint4(0, 0, 0, 0);
    }
    __syncthreads();
    Cursor at;   // the CTA's place: start of the current segment
    at.b = lo < hi ? s_b : 0;
    at.tiles = SeqTiles(a, at.b).tiles;
    if (lo >= hi || at.tiles == 0) {
        pdl_wait();
        return;
    }
    at.kvh = s_rem / at.tiles;
    at.j = s_rem % at.tiles;
    at.left = hi - lo;

    // ---- producer (the team's leader): copies in the order the team consumes them
    Cursor next = at;
    int part = 0;               // copy of the tile at `next`: 8 bits K, V; open block K, K, V, V
    bool more = leader && team < next.left;
    if (more) next.skip(a, team);
    uint32_t p_stage = 0, p_phase = 0, armed = 0, armed_phase = 0;
    auto produce = [&]() -> bool {
        if (!mbar_wait(&empty[p_stage], p_phase ^ 1u, abort_flag, a.ctl)) return false;
        mbar_arrive_expect_tx(&full[p_stage], STAGE);
        armed |= 1u << p_stage;
        armed_phase = (armed_phase & ~(1u << p_stage)) | (p_phase << p_stage);
        const long long unit = (long long)next.b * a.Hkv + next.kvh;
        const bool open = SeqTiles(a, next.b).open(next.j);
        const uint8_t* src;
        if (!open) {
            src = (part == 0 ? a.k8 : a.v8) + (unit * a.blocks + next.j) * STAGE;
        } else {
            const __nv_bfloat16* tail = part < 2 ? a.k_tail : a.v_tail;
            src = reinterpret_cast<const uint8_t*>(tail) + ((unit * 2 + (next.j & 1)) * 2 + (part & 1)) * STAGE;
        }
        bulk_load(ring + p_stage * STAGE, src, STAGE, &full[p_stage]);
        if (++part == (open ? 4 : 2)) {
            part = 0;
            more = teams < next.left;
            next.skip(a, teams);
        }
        if (++p_stage == (uint32_t)a.stages) {
            p_stage = 0;
            p_phase ^= 1u;
        }
        return true;
    };
    bool ok = true;
    if (leader)
        for (int k = 0; k < a.stages && more && ok; ++k) ok = produce();
    ok = __all_sync(0xffffffffu, ok);

    // ---- consumer
    uint32_t c_stage = 0, c_phase = 0;
    auto wait_full = [&]() -> const uint8_t* {
        if (!__all_sync(0xffffffffu, mbar_wait(&full[c_stage], c_phase, abort_flag, a.ctl))) {
            ok = false;
            return nullptr;
        }
        const uint8_t* p = ring + c_stage * STAGE;
        if (++c_stage == (uint32_t)a.stages) {
            c_stage = 0;
            c_phase ^= 1u;
        }
        return p;
    };
    uint32_t r_stage = 0;
    auto release = [&]() {   // the oldest stage that is still held
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[r_stage]);
        if (++r_stage == (uint32_t)a.stages) r_stage = 0;
        if (leader && more && !produce()) *abort_flag = 1;
        __syncwarp();
    };

    RowState<D> st;
    long long done = 0;   // tiles of the CTA's range before the current segment
    while (at.left > 0) {
        const SeqTiles q(a, at.b);
        const long long unit = (long long)at.b * a.Hkv + at.kvh;
        const int j1 = (int)min((long long)at.tiles, at.j + at.left);   // segment: tiles [at.j, j1) of the unit
        const __nv_bfloat16* src[2];
        int lim[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int row = 16 * rt + g + 8 * r, i = row / a.G;
            const bool real = row < a.rows && i < q.n;
            src[r] = real ? a.Q + (((long long)at.b * a.Lq + i) * a.Hq + at.kvh * a.G + row % a.G) * D : nullptr;
            lim[r] = real ? q.len + i : -1;
        }
        uint32_t qf[D / 16][4];
        float f[2];
        load_rows<D>(src, t, qf);
        rows_to_f16<D>(qf, f);
        const float unscaled = kLog2e * rsqrtf((float)D);
        f[0] *= unscaled;
        f[1] *= unscaled;
        st.clear();
        // the team's tiles of the segment: every teams-th of the CTA's range; their
        // scales come 32 tiles at a time, one batch ahead
        int j = at.j + (int)((team - done % teams + teams) % teams);
        const float *ksp = a.k_scale + unit * a.blocks, *vsp = a.v_scale + unit * a.blocks;
        auto scale_of = [&](const float* p, int from) {
            const int k = from + lane * teams;
            return k < j1 && !q.open(k) ? p[k] : 0.f;
        };
        float ks_now = scale_of(ksp, j), vs_now = scale_of(vsp, j);
        float ks_next = scale_of(ksp, j + 32 * teams), vs_next = scale_of(vsp, j + 32 * teams);
        for (int it = 0; ok && j < j1; j += teams, ++it) {
            if (it == 32) {
                it = 0;
                ks_now = ks_next;
                vs_now = vs_next;
                ks_next = scale_of(ksp, j + 32 * teams);
                vs_next = scale_of(vsp, j + 32 * teams);
            }
            const int base = j * kCacheBlock;
            const bool mask = base + kCacheBlock - 1 > q.len;   // (the first query row sees tokens up to len)
            float s[8][4];
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[i][e] = 0.f;
            // tokens of the first product's columns: column n of step i is token 16 (n / 2) + 2 i + n % 2
            if (!q.open(j)) {
                const float ks = __shfl_sync(0xffffffffu, ks_now, it), vs = __shfl_sync(0xffffffffu, vs_now, it);
                const uint8_t* kt = wait_full();
                if (!kt) break;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint8_t* row = kt + (16 * (g >> 1) + 2 * i + (g & 1)) * D + 16 * t;
#pragma unroll
                    for (int c = 0; c < D / 64; ++c) {
                        const uint4 w = *reinterpret_cast<const uint4*>(row + 64 * c);
                        const uint32_t w4[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            uint32_t b0, b1;
                            codes_to_f16<E4M3>(w4[k], b0, b1);
                            mma_f16(s[i], qf[4 * c + k], b0, b1);
                        }
                    }
                }
                release();
                const float fk[2] = {f[0] * ks, f[1] * ks};
                soften<D>(s, fk, mask, base, lim, vs, t, st);
                uint32_t pf[4][4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    pf[k][0] = pack_f16x2(s[2 * k][0], s[2 * k][1]);
                    pf[k][1] = pack_f16x2(s[2 * k][2], s[2 * k][3]);
                    pf[k][2] = pack_f16x2(s[2 * k + 1][0], s[2 * k + 1][1]);
                    pf[k][3] = pack_f16x2(s[2 * k + 1][2], s[2 * k + 1][3]);
                }
                const uint8_t* vt = wait_full();
                if (!vt) break;
#pragma unroll
                for (int i = 0; i < D / 8; ++i) {
                    const uint4 w = *reinterpret_cast<const uint4*>(vt + (8 * i + g) * kCacheBlock + 16 * t);
                    const uint32_t w4[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        uint32_t b0, b1;
                        codes_to_f16<E4M3>(w4[k], b0, b1);
                        mma_f16(st.o[i], pf[k], b0, b1);
                    }
                }
                release();
            } else {
                // the open block, in bf16: keys [64][D], values [D][64], each in two stages
                uint32_t qb[D / 16][4];
                load_rows<D>(src, t, qb);
                const uint8_t* k0 = wait_full();
                if (!k0) break;
                const uint8_t* k1 = wait_full();
                if (!k1) break;
                const uint8_t* half = g < 4 ? k0 : k1;   // tokens 16 (g / 2) ..: the first or second 32
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint8_t* row = half + (16 * ((g >> 1) & 1) + 2 * i + (g & 1)) * D * 2 + 32 * t;
#pragma unroll
                    for (int c = 0; c < D / 64; ++c)
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const uint4 w = *reinterpret_cast<const uint4*>(row + 128 * c + 16 * k);
                            mma_bf16(s[i], qb[4 * c + 2 * k], w.x, w.y);
                            mma_bf16(s[i], qb[4 * c + 2 * k + 1], w.z, w.w);
                        }
                }
                release();
                release();
                const float fk[2] = {unscaled, unscaled};
                soften<D>(s, fk, true, base, lim, 1.f, t, st);
                uint32_t pf[4][4], keep[8];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    pf[k][0] = pack_bf16x2(s[2 * k][0], s[2 * k][1]);
                    pf[k][1] = pack_bf16x2(s[2 * k][2], s[2 * k][3]);
                    pf[k][2] = pack_bf16x2(s[2 * k + 1][0], s[2 * k + 1][1]);
                    pf[k][3] = pack_bf16x2(s[2 * k + 1][2], s[2 * k + 1][3]);
                }
                // slots past the sequence's end hold whatever was there before: zero, not 0 * NaN
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int over = q.T - (base + 16 * t + 2 * k);
                    keep[k] = over > 1 ? 0xffffffffu : (over == 1 ? 0x0000ffffu : 0u);
                }
                const uint8_t* v0 = wait_full();
                if (!v0) break;
                const uint8_t* v1 = wait_full();
                if (!v1) break;
#pragma unroll
                for (int i = 0; i < D / 8; ++i) {
                    const uint8_t* row = (i < D / 16 ? v0 : v1) + (8 * (i % (D / 16)) + g) * kCacheBlock * 2 + 32 * t;
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const uint4 w = *reinterpret_cast<const uint4*>(row + 16 * k);
                        mma_bf16(st.o[i], pf[2 * k], w.x & keep[4 * k], w.y & keep[4 * k + 1]);
                        mma_bf16(st.o[i], pf[2 * k + 1], w.z & keep[4 * k + 2], w.w & keep[4 * k + 3]);
                    }
                }
                release();
                release();
            }
        }

        // ---- merge the teams
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            st.l[r] += __shfl_xor_sync(0xffffffffu, st.l[r], 1);
            st.l[r] += __shfl_xor_sync(0xffffffffu, st.l[r], 2);
            const int row = g + 8 * r;
            if (16 * rt + row < a.rows) {
                float* to = red_o + ((long long)warp * a.merge_rows + row) * D + 2 * t;
#pragma unroll
                for (int i = 0; i < D / 8; ++i)
                    *reinterpret_cast<float2*>(to + 8 * i) = make_float2(st.o[i][2 * r], st.o[i][2 * r + 1]);
                if (t == 0)
                    *reinterpret_cast<float4*>(red_s + (warp * a.merge_rows + row) * 4) =
                        make_float4(st.m[r], st.l[r], st.M[r], 0.f);
            }
        }
        if (!__syncthreads_and(ok && !*abort_flag)) {
            ok = false;
            break;
        }
        const bool whole = at.j == 0 && j1 == at.tiles;
        // the unit's place in the sequence of all tiles, and the CTAs it is split over
        const long long u0 = lo + done - at.j, u1 = u0 + at.tiles - 1;
        long long c0 = u0 * ctas / N, c1 = u1 * ctas / N;
        while (N * (c0 + 1) / ctas <= u0) ++c0;
        while (N * (c1 + 1) / ctas <= u1) ++c1;
        const auto slot = [&](long long c) { return 2 * c + (c > c0 || u0 == N * c0 / ctas ? 0 : 1); };
        if (whole && a.gate_mode != GSDPA_GATE_NONE) pdl_wait();   // the gate logits
        for (int idx = tid; idx < a.rows * (D / 4); idx += kThreads) {
            const int row = idx / (D / 4), col = 4 * (idx % (D / 4));
            float m = -INFINITY, l = 0.f, M = -INFINITY;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int w = row / 16; w < kWarps; w += a.R) {
                const float4 x = *reinterpret_cast<const float4*>(red_s + (w * a.merge_rows + row % 16) * 4);
                merge(m, l, M, o, x.x, x.y, x.z,
                      *reinterpret_cast<const float4*>(red_o + ((long long)w * a.merge_rows + row % 16) * D + col));
            }
            if (whole) {
                finish<D>(a, at.b, at.kvh, q.n, row, col, m, l, M, o);
            } else {
                const long long to = slot(me) * a.rows + row;
                *reinterpret_cast<float4*>(a.part_o + to * D + col) = o;
                if (col == 0) *reinterpret_cast<float4*>(a.part_s + to * 4) = make_float4(m, l, M, 0.f);
            }
        }
        if (!whole) {
            __threadfence();
            __syncthreads();
            if (tid == 0) s_last = atomicAdd(a.counters + unit, 1) == (int)(c1 - c0);
            __syncthreads();
            if (s_last) {
                __threadfence();
                if (a.gate_mode != GSDPA_GATE_NONE) pdl_wait();
                for (int idx = tid; idx < a.rows * (D / 4); idx += kThreads) {
                    const int row = idx / (D / 4), col = 4 * (idx % (D / 4));
                    float m = -INFINITY, l = 0.f, M = -INFINITY;
                    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
                    for (long long c = c0; c <= c1; ++c) {
                        const long long from = slot(c) * a.rows + row;
                        const float4 x = __ldcg(reinterpret_cast<const float4*>(a.part_s + from * 4));
                        merge(m, l, M, o, x.x, x.y, x.z, __ldcg(reinterpret_cast<const float4*>(a.part_o + from * D + col)));
                    }
                    finish<D>(a, at.b, at.kvh, q.n, row, col, m, l, M, o);
                }
            }
        }
        __syncthreads();   // the merge buffer may be written again
        const int took = j1 - at.j;
        done += took;
        at.skip(a, took);
    }
    pdl_wait();   // (the next kernel on the stream may rely on the gate kernel having ended too)
    if (!ok && leader) {
        // let copies in flight land before the CTA exits
        volatile int never = 0;
        WaitCtl c2 = a.ctl;
        if (c2.limit_ns < 1000000000ull) c2.limit_ns = 1000000000ull;
        for (int k = 0; k < a.stages; ++k)
            if (armed & (1u << k)) mbar_wait(&full[k], (armed_phase >> k) & 1u, &never, c2);
    }
}

// Shared memory and ring of one problem.
struct Shape {
    int R, stages, merge_rows;
    uint32_t smem;
};
Shape shape_of(int rows, int D) {
    Shape s;
    s.R = rows <= 16 ? 1 : (rows <= 32 ? 2 : (rows <= 64 ? 4 : 8));
    s.merge_rows = rows < 16 ? rows : 16;
    const uint32_t merge = kWarps * (uint32_t)(s.merge_rows * (D + 4)) * 4;
    const uint32_t per_stage = (uint32_t)(kWarps / s.R) * kCacheBlock * D;
    // as many copies in flight as fit, up to 192 KB (an open block holds two stages at once)
    s.stages = (int)((kSmemMax - merge) / per_stage);
    const int most = (int)(196608 / per_stage);
    if (s.stages > most) s.stages = most;
    if (s.stages > kMaxStages) s.stages = kMaxStages;
    if (s.stages > kBars * s.R / kWarps) s.stages = kBars * s.R / kWarps;
    s.smem = (uint32_t)s.stages * per_stage + merge;
    return s;
}

struct Cache8Plan {
    Problem p{};
    WorkspacePlan w;   // the gate kernel's part
    size_t part_o = 0, part_s = 0, counters = 0, total = 0;
    int n_counters = 0;
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
    if ((long long)c->H_kv * (c->capacity / kCacheBlock) > 0x7fffffffLL) return GSDPA_ERR_UNSUPPORTED;
    if ((long long)c->B * Lq > 0x7fffffffLL / 8) return GSDPA_ERR_UNSUPPORTED;
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
    o.part_o = take(sizeof(float) * 2 * plan_sms() * (size_t)rows * c->d_k);
    o.part_s = take(sizeof(float) * 2 * plan_sms() * (size_t)rows * 4);
    o.n_counters = c->B * c->H_kv;
    o.counters = take(sizeof(int) * (size_t)o.n_counters);
    o.total = off;
    return GSDPA_OK;
}

template <int D, bool E4M3>
cudaError_t launch(const Cache8Args& a, const Shape& sh, unsigned grid, cudaStream_t s) {
    static PerDeviceSetup setup;
    const cudaError_t e = setup_once_per_device(setup, [](int&) {
        return cudaFuncSetAttribute(cache8_attn_kernel<D, E4M3>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    (int)kSmemMax);
    });
    if (e != cudaSuccess) return e;
    return launch_dependent(cache8_attn_kernel<D, E4M3>, dim3(grid), dim3(kThreads), sh.smem, s, a);
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

    // The arrival counters are zeroed by the kernel that runs first: the gate
    // logits' or, without a gate, state_zero_kernel. Both wait for the kernels
    // before them, so the attention, their programmatic dependent, finds the
    // cache and the queries written; it waits for the logits where it reads them.
    ZeroJob zero;
    zero.p = reinterpret_cast<int*>(ws + pl.counters);
    zero.n = pl.n_counters;
    bool launched = false;
    cudaError_t e = launch_gate_logits_bf16(pl.p, pl.w, ws, rt, s, &launched, zero);
    if (e == cudaSuccess && !launched) e = launch_state_zero(zero, s);
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
    a.rows = a.G * L_q;
    a.blocks = cache->capacity / kCacheBlock;
    a.capacity = cache->capacity;
    const Shape sh = shape_of(a.rows, cache->d_k);
    a.R = sh.R;
    a.stages = sh.stages;
    a.merge_rows = sh.merge_rows;
    a.gate_part = gated ? reinterpret_cast<const float*>(ws + pl.w.gate_part) : nullptr;
    a.gate_splits = pl.w.gate_splits;
    a.gate_cols = pl.w.gate_cols;
    a.gate_mode = gate_mode;
    a.part_o = reinterpret_cast<float*>(ws + pl.part_o);
    a.part_s = reinterpret_cast<float*>(ws + pl.part_s);
    a.counters = zero.p;
    a.ctl.err = rt.err;
    a.ctl.limit_ns = rt.limit_ns;
    // one CTA per SM, fewer where a full cache would not give each its tiles
    const long long most = ((long long)a.B * a.Hkv * a.blocks + kMinTiles - 1) / kMinTiles;
    long long grid = rt.num_sms < plan_sms() ? rt.num_sms : plan_sms();
    if (grid > most) grid = most;
    const bool e4m3 = cache->kind == GSDPA_CACHE_E4M3;
    if (cache->d_k == 128)
        e = e4m3 ? launch<128, true>(a, sh, (unsigned)grid, s) : launch<128, false>(a, sh, (unsigned)grid, s);
    else
        e = e4m3 ? launch<64, true>(a, sh, (unsigned)grid, s) : launch<64, false>(a, sh, (unsigned)grid, s);
    return e == cudaSuccess ? GSDPA_OK : GSDPA_ERR_LAUNCH;
}

}  // extern "C"
