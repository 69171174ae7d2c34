// cache_attn.cuh -- what the attention kernels over a cache of few bits (8 bits,
// one piece per sequence; 4 bits, in pages) have in common: the walk of a team through
// its tiles, how the parts of a head that several teams share are merged, and the gate at
// the end. (How tiles are dealt: cache_deal.h.) Not part of the public ABI.
//
// A kernel's arguments A have the members used here and
//   A::Seq(a, b)   sequence b: n (new tokens), T (tokens in all, 0 without new ones), tiles, span()
//   by_head(longest, N)   whether heads of at most so many tiles, N places in all, are better one CTA's each
//   token(b, i)    the row of Q, X and O that holds new token i of sequence b
//   tokens()       all rows
#pragma once
#include "cache_deal.h"
#include "ops_internal.h"

#include <cuda_fp16.h>

namespace gsdpa {

constexpr int kSlots = 8;            // most teams that a copying warp serves (twice as many where each warp copies for itself)
constexpr int kMaxRows = 128;        // query rows (heads of a group x new tokens) per K/V head
constexpr int kMaxCtas = 160;        // most CTAs (plan_sms)
constexpr int kMergeThreads = 512;
constexpr int kBatch = 6;            // parts that a thread of a merge has under way
constexpr int kScan = 128;           // places in the sequence of all tiles that are looked up
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// An 8 x 8 matrix of 16-bit elements, row g columns 2 t, 2 t + 1 in lane (g, t), transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// 1 / (1 + e^-x), accurate to a few units of float32's last place.
__device__ __forceinline__ float sigmoid(float x) { return __fdividef(1.f, 1.f + __expf(-x)); }

// A place in the sequence of all tiles. (Where places are left a sequence with
// tiles follows; lengths that change during the call, which they must not, end
// the walk instead of leading it out of the batch.)
struct Cursor {
    int b, kvh, j, tiles;
    int left;   // places of the share from here on
    template <class A>
    __device__ __forceinline__ void next_head(const A& a) {
        left -= span_of<A>(tiles) - j;
        j = 0;
        if (left <= 0) return;
        if (++kvh == a.Hkv) {
            kvh = 0;
            do {
                if (++b >= a.B) {
                    left = 0;
                    return;
                }
                tiles = typename A::Seq(a, b).tiles;
            } while (tiles == 0);
        }
    }
};

// What a warp keeps of its 8 NT query rows; lane (g, t) has rows 8 n + 2 t + e.
template <int D, int NT>
struct RowState {
    float o[NT][D / 16][4];   // element 2 x + e: column 16 i + 8 x + g of row 8 n + 2 t + e
    float m[NT][2], l[NT][2], M[NT][2];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[n][i][e] = 0.f;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                m[n][e] = M[n][e] = -INFINITY;
                l[n][e] = 0.f;
            }
        }
    }
};

// What turns a row's summed outputs into the attention's (a row whose weights
// leave nothing is zero): two factors, because 2^(M - m) alone may leave float32's
// range where the output does not.
__device__ __forceinline__ float2 out_scale(float m, float l, float M) {
    const float half = M == -INFINITY ? 0.f : ex2_approx(0.5f * (M - m));
    return make_float2(half, l > 0.f || l != l ? half / l : 0.f);
}

// The gate's values for columns [col, col + 4) of query row `row`: of all K splits of
// the logits a batch of loads is under way at a time.
template <int D, class A>
__device__ __forceinline__ float4 gate_of(const A& a, int b, int kvh, int n, int row, int col) {
    const int i = row * a.g_inverse >> 16;
    if (a.gate_mode == GSDPA_GATE_NONE || i >= n) return make_float4(1.f, 1.f, 1.f, 1.f);
    const int h = (kvh - i) * a.G + row;   // kvh G + row % G
    const long long token = a.token(b, i), step = a.tokens() * a.gate_cols;
    const bool per_col = a.gate_mode == GSDPA_GATE_ELEMENTWISE;
    const float* gp = a.gate_part + token * a.gate_cols + (per_col ? (long long)h * D + col : h);
    float4 gl = make_float4(0.f, 0.f, 0.f, 0.f);
    constexpr int BATCH = 8;
    for (int sp = 0; sp < a.gate_splits; sp += BATCH) {
        float4 v[BATCH];
#pragma unroll
        for (int k = 0; k < BATCH; ++k) {
            v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (sp + k >= a.gate_splits) continue;
            if (per_col) v[k] = *reinterpret_cast<const float4*>(gp + (sp + k) * step);
            else v[k].x = gp[(sp + k) * step];
        }
#pragma unroll
        for (int k = 0; k < BATCH; ++k) {
            gl.x += v[k].x;
            gl.y += v[k].y;
            gl.z += v[k].z;
            gl.w += v[k].w;
        }
    }
    if (!per_col) gl.y = gl.z = gl.w = gl.x;
    return make_float4(sigmoid(gl.x), sigmoid(gl.y), sigmoid(gl.z), sigmoid(gl.w));
}

// Output columns [col, col + 4) of query row `row`: the sums o, scaled by both of k,
// times the gate, stored.
template <int D, class A>
__device__ __forceinline__ void finish(const A& a, int b, int kvh, int n, int row, int col, const float2& k,
                                       const float4& o, const float4& gate) {
    const int i = row * a.g_inverse >> 16;
    if (i >= n) return;
    const int h = (kvh - i) * a.G + row;
    *reinterpret_cast<uint2*>(a.O + (a.token(b, i) * a.Hq + h) * D + col) =
        make_uint2(pack_bf16x2(o.x * k.x * k.y * gate.x, o.y * k.x * k.y * gate.y),
                   pack_bf16x2(o.z * k.x * k.y * gate.z, o.w * k.x * k.y * gate.w));
}

// 2^(x - top), 0 for a part that saw nothing.
__device__ __forceinline__ float part_weight(float x, float top) { return x == -INFINITY ? 0.f : ex2_approx(x - top); }

__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}

// Four columns of a row, merged from several parts.
struct Sums {
    float m = -INFINITY, l = 0.f, M = -INFINITY;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    // parts i, i + step, .. below end; where(i) points to part i's row: its columns, then its m, l, M at `state`
    template <typename F>
    __device__ __forceinline__ void add(int i, int end, int step, int state, int col, F where) {
        for (; i < end; i += kBatch * step) {   // a batch of loads under way
            float4 x[kBatch], v[kBatch];
            float mn = m, Mn = M;
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                x[k] = make_float4(-INFINITY, 0.f, -INFINITY, 0.f);
                v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (i + k * step < end) {
                    const float* from = where(i + k * step);
                    x[k] = *reinterpret_cast<const float4*>(from + state);
                    v[k] = *reinterpret_cast<const float4*>(from + col);
                }
            }
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                mn = fmaxf(mn, x[k].x);
                Mn = fmaxf(Mn, x[k].z);
            }
            const float w0 = part_weight(M, Mn);
            l *= part_weight(m, mn);
            o.x *= w0;
            o.y *= w0;
            o.z *= w0;
            o.w *= w0;
            m = mn;
            M = Mn;
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const float w = part_weight(x[k].z, M);
                l += x[k].y * part_weight(x[k].x, m);
                o.x += v[k].x * w;
                o.y += v[k].y * w;
                o.z += v[k].z * w;
                o.w += v[k].w * w;
            }
        }
    }
    __device__ __forceinline__ void join(float m2, float l2, float M2, const float4& o2) {
        const float mn = fmaxf(m, m2), Mn = fmaxf(M, M2);
        const float wa = part_weight(M, Mn), wb = part_weight(M2, Mn);
        l = l * part_weight(m, mn) + l2 * part_weight(m2, mn);
        o.x = o.x * wa + o2.x * wb;
        o.y = o.y * wa + o2.y * wb;
        o.z = o.z * wa + o2.z * wb;
        o.w = o.w * wa + o2.w * wb;
        m = mn;
        M = Mn;
    }
    __device__ __forceinline__ void join_lane(int sh) {
        const float m2 = __shfl_xor_sync(0xffffffffu, m, sh), l2 = __shfl_xor_sync(0xffffffffu, l, sh);
        const float M2 = __shfl_xor_sync(0xffffffffu, M, sh);
        join(m2, l2, M2, make_float4(__shfl_xor_sync(0xffffffffu, o.x, sh), __shfl_xor_sync(0xffffffffu, o.y, sh),
                                     __shfl_xor_sync(0xffffffffu, o.z, sh), __shfl_xor_sync(0xffffffffu, o.w, sh)));
    }
};

// Where team n leaves its rows of the cut head whose first tile is u0.
template <int D, class A>
__device__ __forceinline__ float* part_of(const A& a, const Deal& deal, int n, int u0) {
    return a.part + (long long)part_index(deal, n, u0) * a.rows * (D + 4);
}

// The sequence of all tiles: sequence after sequence, in each one K/V head after
// the other. (Its scan in four warps: in all twenty of a block it took 0.6 us more.)
struct Layout {
    int per;            // sequences to a place
    int N, longest;     // all places; most tiles of a head
    int ctas;           // that have any
    bool by_head;
    const int* place;   // [kScan + 1], in shared memory: the places before sequence per * k
    // a CTA to each head, whatever the lengths (nothing is looked up)
    __device__ __forceinline__ explicit Layout(const int* s_place)
        : per(1), N(0), longest(0), ctas(1), by_head(true), place(s_place) {}
    // by all threads of a block of kScan or more
    template <class A>
    __device__ __forceinline__ Layout(const A& a, int* s_place, int* s_scan, int tid) : place(s_place) {
        const int warp = tid / 32, lane = tid % 32;
        constexpr int W = kScan / 32;
        per = (a.B + kScan - 1) / kScan;
        int mine = 0, scan = 0;
        if (warp < W) {
            longest = 0;
            for (int b = tid * per; b < min(a.B, (tid + 1) * per); ++b) {
                const typename A::Seq q(a, b);
                mine += q.span();
                longest = max(longest, q.tiles);
            }
            mine *= a.Hkv;
            scan = mine;
#pragma unroll
            for (int sh = 1; sh < 32; sh <<= 1) {
                const int up = __shfl_up_sync(0xffffffffu, scan, sh);
                if (lane >= sh) scan += up;
            }
            longest = __reduce_max_sync(0xffffffffu, longest);
            if (lane == 31) s_scan[warp] = scan;
            if (lane == 0) s_scan[W + warp] = longest;
        }
        __syncthreads();
        N = longest = 0;   // (fits: the host checks the number of places)
        int before = scan - mine;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            if (w < warp) before += s_scan[w];
            N += s_scan[w];
            longest = max(longest, s_scan[W + w]);
        }
        if (warp < W) s_place[tid] = before;
        if (tid == 0) s_place[kScan] = N;
        __syncthreads();
        ctas = max(1, min(a.ctas, N >> a.lg_teams));   // every team has a place (or there is one CTA)
        // Short sequences, a CTA for each head: no head is cut between CTAs, whose
        // merge would take longer than the tiles.
        by_head = a.B * (long long)a.Hkv <= a.ctas && a.by_head(longest, N);
    }
    // place x < N is place `rem` of sequence b
    template <class A>
    __device__ __forceinline__ void find(const A& a, int x, int& b, int& rem) const {
        int k = 0;
#pragma unroll
        for (int step = kScan / 2; step > 0; step >>= 1)
            if (place[k + step] <= x) k += step;
        b = k * per;
        rem = x - place[k];
        if (per > 1) {
            int in_seq = typename A::Seq(a, b).span() * a.Hkv;
            while (rem >= in_seq && b + 1 < a.B) {
                rem -= in_seq;
                in_seq = typename A::Seq(a, ++b).span() * a.Hkv;
            }
        }
    }
    // places before sequence b
    template <class A>
    __device__ __forceinline__ int before(const A& a, int b) const {
        int at = place[b / per];
        for (int k = b / per * per; k < b; ++k) at += typename A::Seq(a, k).span() * a.Hkv;
        return at;
    }
};

// The heads that were cut between teams, from the teams' parts. Four lanes have
// 16 columns of a row; a head's parts are split over as many such groups as give
// every thread of the grid work, down to four parts each (one sequence of 131072
// tokens leaves 608 parts of each head), and joined by shuffles and through
// shared memory. Its own kernel, because the end of the attention kernel is the
// one point at which all parts are known to be there without atomics: a launch
// that was set up early costs less than a chain of counters (one sequence of
// 131072 tokens: merged in the attention kernel, by the CTAs that arrive last at
// two levels of counters, 26.7 us in all, so 23.1; two blocks to an SM with half
// the registers and batches of four: 25.7).
template <int D, class A>
__global__ void __launch_bounds__(kMergeThreads) cache_merge_kernel(const __grid_constant__ A a) {
    constexpr int kWarps = kMergeThreads / 32;
    __shared__ int s_place[kScan + 1], s_scan[2 * kScan / 32];
    __shared__ float4 s_o[kWarps][4], s_x[kWarps][4];
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    pdl_trigger();
    // (the attention kernel started after everything before this call had ended: the lengths may be read)
    const Layout all(a, s_place, s_scan, tid);
    const Deal deal(all.N, all.ctas << a.lg_teams);
    const int items = a.rows * (D / 4), takers = all.ctas << a.lg_teams, threads = gridDim.x * kMergeThreads;
    // A unit of the work is a head, or where there are more heads than places at which
    // shares begin, such a place, for the head that it is the first to cut.
    const long long heads = (long long)a.B * a.Hkv;
    const bool by_place = heads >= takers;
    const int units = all.by_head ? 0 : (by_place ? takers - 1 : (int)heads);
    int most = deal.each > 0 ? all.longest / deal.each + 2 : 1;   // parts of a head
    if (A::kJoins && all.N > 0)   // CTAs that a head lies across, and the teams of the two at its ends
        most = min(most, (int)((long long)all.longest * all.ctas / all.N) + (1 << a.lg_teams));
    int lg = 0;
    while ((8 << lg) <= kMergeThreads && ((units * items) << (lg + 1)) <= threads && (4 << lg) < most) ++lg;
    const int total = (units * items) << lg;   // (below 2560 x 4096, or the grid's threads)
    bool waited = false;
    for (int base = blockIdx.x * kMergeThreads; base < total; base += threads) {
        const int idx = base + tid, unit = idx / (items << lg);
        const int x = idx - unit * (items << lg), item = (x >> (lg + 2) << 2) + (x & 3), sub = (x >> 2) & ((1 << lg) - 1);
        const int row = item / (D / 4), col = 4 * (item % (D / 4));
        int b = 0, kvh = 0, u0 = 0, n0 = 0, n1 = 0, span = 0;
        if (by_place) {
            const int from = idx < total ? deal.from(unit + 1) : all.N;
            if (from < all.N) {
                all.find(a, from, b, u0);
                const int tiles = typename A::Seq(a, b).tiles;
                span = span_of<A>(tiles);
                const int at = u0 % max(span, 1);
                kvh = u0 / max(span, 1);
                u0 = from - at;
                if (at > 0 && at < tiles && deal.taker(u0) == unit) {
                    n0 = unit;
                    n1 = deal.taker(u0 + tiles - 1);
                }
            }
        } else if (idx < total) {
            b = unit / a.Hkv;
            kvh = unit % a.Hkv;
            const int tiles = typename A::Seq(a, b).tiles;
            span = span_of<A>(tiles);
            u0 = all.before(a, b) + kvh * span;
            if (tiles > 0) {
                n0 = deal.taker(u0);
                n1 = deal.taker(u0 + tiles - 1);
            }
        }
        if (!waited) pdl_wait();
        waited = true;
        const bool cut = n1 > n0;
        const Parts<A> parts(a, deal, n0, n1, u0, span);
        const int n = cut ? typename A::Seq(a, b).n : 0;
        float4 gate = make_float4(1.f, 1.f, 1.f, 1.f);
        if (cut && sub == 0) gate = gate_of<D>(a, b, kvh, n, row, col);
        Sums r;
        if (cut)
            r.add(sub, parts.n, 1 << lg, D, col,
                  [&](int k) { return part_of<D>(a, deal, parts.team(k), u0) + row * (D + 4); });
        for (int k = 0; k < min(lg, 3); ++k) r.join_lane(4 << k);
        if (lg > 3) {   // warps that share items
            const int share = 1 << (lg - 3);
            if (lane < 4) {
                s_o[warp][lane] = r.o;
                s_x[warp][lane] = make_float4(r.m, r.l, r.M, 0.f);
            }
            __syncthreads();
            if (warp % share == 0) {
                r = Sums();
                for (int k = lane >> 2; k < share; k += 8) {
                    const float4 y = s_x[warp + k][lane & 3];
                    r.join(y.x, y.y, y.z, s_o[warp + k][lane & 3]);
                }
                for (int k = 0; k < 3; ++k) r.join_lane(4 << k);
            }
            __syncthreads();
        }
        if (cut && sub == 0) finish<D>(a, b, kvh, n, row, col, out_scale(r.m, r.l, r.M), r.o, gate);
    }
    if (!waited) pdl_wait();   // the next kernel on the stream relies on the attention kernel having ended
}

}  // namespace gsdpa
