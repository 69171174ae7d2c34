// pages_step_sm103.cu -- the plan of a step over a paged K/V cache: which pages the
// requests give back and take, the block table, and each token's slot and position.
//
// With p(x) = ceil(x / 64), request b gives back F_b = p(lens) - p(keep) pages and
// needs P_b = p(keep + n) - p(keep). The pages given back are pushed on the free
// stack in the order of the requests, then the needs are served from its top in the
// same order: all that is needed is the running sums of n, F and P over the requests.
// No atomics decide an order, so a plan repeats bit for bit.
//
// Bound by latency: 64 requests are 1 KB in and 1 KB out. One block does the sums
// (three scans of up to 8 requests a thread) and moves page numbers, whose owners it finds by
// bisection of the sums in shared memory; the tokens of a decoding step are filled
// in by the same block, a prompt's by a second kernel that is set up while the first
// runs. Measured: 64 requests of one token 4.0 us, 256 with eight prompts of 1023 tokens 7.1 us, 1000 of one
// token 5.9 us, 8000 28 us.
#include "cache4_internal.h"

namespace gsdpa {
namespace {

constexpr int kMaxRequests = 8192;
constexpr int kPlanThreads = 1024, kFillThreads = 256;
constexpr int kEach = kMaxRequests / kPlanThreads;
// Rows to a thread that the planning block fills in itself (64 requests, 256 threads, 64, 1024, 2048 rows: 4.2, 6.5,
// 8.8 us so, 5.9, 5.6, 5.6 with the second kernel, which also costs the host 2.5 us).
constexpr int kFewRows = 2;

struct PagesArgs {
    const int *lens, *keep, *n_new;
    int *table, *free_pages;
    const int* n_free;
    int *n_free_out, *cu, *granted;
    long long* slots;
    int* positions;
    int B, width, n_pages, n_rows;
    uint32_t* err;
};

__device__ __forceinline__ int pages_of(int tokens) { return (tokens + kPage - 1) / kPage; }   // (tokens <= 2^31 - 64)

// A request's tokens held, kept and brought; ok: within what its row of the table can hold.
struct Request {
    int held, kept, n;
    bool ok;
    __device__ __forceinline__ Request(const PagesArgs& a, int b) {
        held = a.lens[b];
        kept = a.keep ? a.keep[b] : held;
        n = a.n_new[b];
        const int most = a.width * kPage;
        ok = held >= 0 && held <= most && kept >= 0 && kept <= held && n >= 0 && n <= most - kept;
    }
};

// The last of sums[0 .. n] (ascending, sums[0] <= x) that is not above x.
__device__ __forceinline__ int owner(const int* sums, int n, int x) {
    int lo = 0, hi = n;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (sums[mid] <= x) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// Slot and position of row i, a token of the step.
__device__ __forceinline__ void fill_row(const PagesArgs& a, const int* cu, int i) {
    long long slot = -1;
    int position = 0;
    if (i < cu[a.B]) {
        const int b = owner(cu, a.B, i);
        const Request r(a, b);
        if (r.ok) {
            position = r.kept + (i - cu[b]);
            if (a.granted[b] > 0) {
                const int page = a.table[(long long)b * a.width + position / kPage];
                if (page >= 0 && page < a.n_pages) slot = (long long)page * kPage + position % kPage;
                else atomicOr(a.err, ERR_CACHE_RANGE);
            }
        }
    }
    a.slots[i] = slot;
    if (a.positions) a.positions[i] = position;
}

// Sum of v over the threads before this one; total over all.
template <int THREADS>
__device__ __forceinline__ long long scan(long long v, long long* s_warp, long long& total) {
    constexpr int W = THREADS / 32;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    long long sum = v;
#pragma unroll
    for (int sh = 1; sh < 32; sh <<= 1) {
        const long long up = __shfl_up_sync(0xffffffffu, sum, sh);
        if (lane >= sh) sum += up;
    }
    __syncthreads();   // (s_warp may still be read)
    if (lane == 31) s_warp[warp] = sum;
    __syncthreads();
    long long mine = lane < W ? s_warp[lane] : 0, all = mine;
#pragma unroll
    for (int sh = 1; sh < 32; sh <<= 1) {
        const long long up = __shfl_up_sync(0xffffffffu, all, sh);
        if (lane >= sh) all += up;
    }
    total = __shfl_sync(0xffffffffu, all, 31);
    return sum - v + __shfl_sync(0xffffffffu, all - mine, warp);
}

__device__ __forceinline__ int clamp_int(long long v) { return (int)(v < 0x7fffffffLL ? v : 0x7fffffffLL); }

// s_sums: [3][B + 1], the requests' running sums of rows, pages given back and pages needed.
template <int THREADS, int EACH>
__global__ void __launch_bounds__(THREADS) pages_plan_kernel(const __grid_constant__ PagesArgs a, int fill) {
    extern __shared__ int s_sums[];
    __shared__ long long s_warp[32];
    __shared__ int s_taken;
    const int tid = threadIdx.x, B = a.B;
    int *s_cu = s_sums, *s_free = s_sums + B + 1, *s_need = s_sums + 2 * (B + 1);
    if (tid == 0) s_taken = 0;
    pdl_wait();
    pdl_trigger();

    const int first = tid * EACH;
    long long rows = 0, freed = 0, need = 0, total;
    bool bad = false;
#pragma unroll
    for (int k = 0; k < EACH; ++k)
        if (first + k < B) rows += max(a.n_new[first + k], 0);
    long long row = scan<THREADS>(rows, s_warp, total);
    if (tid == 0) s_cu[B] = (int)min(total, (long long)a.n_rows);
    uint32_t ok = 0;   // bit k: request first + k can be served as far as its own numbers go
#pragma unroll
    for (int k = 0; k < EACH; ++k) {
        if (first + k >= B) continue;
        const Request r(a, first + k);
        s_cu[first + k] = (int)min(row, (long long)a.n_rows);
        row += max(r.n, 0);
        if (r.ok && row <= a.n_rows) {
            ok |= 1u << k;
            freed += pages_of(r.held) - pages_of(r.kept);
            need += pages_of(r.kept + r.n) - pages_of(r.kept);
        } else {
            bad = true;
        }
    }
    long long n_freed, n_needed;
    long long free_at = scan<THREADS>(freed, s_warp, n_freed), need_at = scan<THREADS>(need, s_warp, n_needed);
    if (tid == 0) {
        s_free[B] = clamp_int(n_freed);
        s_need[B] = clamp_int(n_needed);
    }
#pragma unroll
    for (int k = 0; k < EACH; ++k) {
        if (first + k >= B) continue;
        s_free[first + k] = clamp_int(free_at);
        s_need[first + k] = clamp_int(need_at);
        if (ok & (1u << k)) {
            const Request r(a, first + k);
            free_at += pages_of(r.held) - pages_of(r.kept);
            need_at += pages_of(r.kept + r.n) - pages_of(r.kept);
        }
    }
    int held = *a.n_free;
    if (held < 0 || held > a.n_pages) {
        bad = true;
        held = 0;   // (a count that is none: nothing to take)
    }
    __syncthreads();

    // ---- pages given back, on top of the free ones
    const int back = min(s_free[B], a.n_pages - held);   // (more than the pool has: lengths that are none)
    bad = bad || back < s_free[B];
    for (int k = tid; k < back; k += THREADS) {
        const int b = owner(s_free, B - 1, k);   // (requests that give back none share their sum with the next)
        const Request r(a, b);
        const int page = a.table[(long long)b * a.width + pages_of(r.kept) + (k - s_free[b])];
        bad = bad || page < 0 || page >= a.n_pages;
        a.free_pages[held + k] = page;
    }
    const int top = held + back;
    // ---- who gets what: the needs are served in order as long as they fit
#pragma unroll
    for (int k = 0; k < EACH; ++k) {
        const int b = first + k;
        if (b >= B) continue;
        a.cu[b] = s_cu[b];
        int n = 0;
        if (ok & (1u << k)) {
            const Request r(a, b);
            const int p = pages_of(r.kept + r.n) - pages_of(r.kept);
            const long long upto = (long long)s_need[b] + p;
            if (p == 0 || upto <= top) n = r.n;
            if (p > 0 && upto <= top) atomicMax(&s_taken, (int)upto);
        }
        a.granted[b] = n;
    }
    if (tid == 0) a.cu[B] = s_cu[B];
    __syncthreads();
    const int taken = s_taken;
    for (int k = tid; k < taken; k += THREADS) {
        const int b = owner(s_need, B - 1, k);
        const Request r(a, b);
        const int page = a.free_pages[top - 1 - k];
        bad = bad || page < 0 || page >= a.n_pages;
        a.table[(long long)b * a.width + pages_of(r.kept) + (k - s_need[b])] = page;
    }
    if (tid == 0) *a.n_free_out = top - taken;
    if (bad) atomicOr(a.err, ERR_CACHE_RANGE);
    if (fill) {
        __syncthreads();
        for (int i = tid; i < a.n_rows; i += THREADS) fill_row(a, s_cu, i);
    }
}

__global__ void __launch_bounds__(kFillThreads) pages_fill_kernel(const __grid_constant__ PagesArgs a) {
    pdl_trigger();
    pdl_wait();
    const int i = blockIdx.x * kFillThreads + threadIdx.x;
    if (i < a.n_rows) fill_row(a, a.cu, i);
}

bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

}  // namespace
}  // namespace gsdpa

using namespace gsdpa;

extern "C" int gsdpa_pages_step(const int* lens, const int* keep, const int* n_new, int* table, int* free_pages,
                                const int* n_free, int* n_free_out, int* cu, int* granted, long long* slots,
                                int* positions, int B, int max_pages, int n_pages, int n_rows, void* stream) {
    if (B < 0 || max_pages < 1 || n_pages < 1 || n_rows < 0) return GSDPA_ERR_INVALID_ARG;
    // (a request's tokens, and rows past the last block, are counted in 32 bits)
    if (B > kMaxRequests || max_pages > 0x7fffffff / kPage - 1 || n_rows > 0x7fffffff - kFillThreads)
        return GSDPA_ERR_UNSUPPORTED;
    if (!free_pages || !n_free || !n_free_out || !cu || (B > 0 && (!lens || !n_new || !table || !granted)) ||
        (n_rows > 0 && !slots))
        return GSDPA_ERR_INVALID_ARG;
    for (const void* p : {(const void*)lens, (const void*)keep, (const void*)n_new, (const void*)table,
                          (const void*)free_pages, (const void*)n_free, (const void*)n_free_out, (const void*)cu,
                          (const void*)granted, (const void*)positions})
        if (!aligned(p, 4)) return GSDPA_ERR_ALIGNMENT;
    if (!aligned(slots, 8)) return GSDPA_ERR_ALIGNMENT;
    Runtime rt;
    int major = 0, minor = 0;
    if (!current_runtime(&rt, &major, &minor)) return GSDPA_ERR_LAUNCH;
    if (!(major == 10 && minor == 3)) return GSDPA_ERR_UNSUPPORTED;
    const PagesArgs a{lens, keep, n_new, table, free_pages, n_free, n_free_out, cu, granted, slots, positions,
                      B, max_pages, n_pages, n_rows, rt.err};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int fill = n_rows <= kFewRows * (B <= 256 ? 256 : kPlanThreads);
    const size_t smem = 3 * sizeof(int) * ((size_t)B + 1);
    cudaError_t e;
    if (B <= 256) {
        e = launch_dependent(pages_plan_kernel<256, 1>, dim3(1), dim3(256), smem, s, a, fill);
    } else if (B <= kPlanThreads) {
        e = launch_dependent(pages_plan_kernel<kPlanThreads, 1>, dim3(1), dim3(kPlanThreads), smem, s, a, fill);
    } else {
        static PerDeviceSetup setup;
        e = setup_once_per_device(setup, [](int&) {
            return cudaFuncSetAttribute(pages_plan_kernel<kPlanThreads, kEach>,
                                        cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        (int)(3 * sizeof(int) * (kMaxRequests + 1)));
        });
        if (e == cudaSuccess)
            e = launch_dependent(pages_plan_kernel<kPlanThreads, kEach>, dim3(1), dim3(kPlanThreads), smem, s, a, fill);
    }
    if (e == cudaSuccess && !fill)
        e = launch_dependent(pages_fill_kernel, dim3((unsigned)((n_rows + kFillThreads - 1) / kFillThreads)),
                             dim3(kFillThreads), 0, s, a);
    return e == cudaSuccess ? GSDPA_OK : GSDPA_ERR_LAUNCH;
}
