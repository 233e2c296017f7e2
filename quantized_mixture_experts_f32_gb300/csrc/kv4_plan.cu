// kv4_plan.cu -- block tables and slot maps of one serving step, built on the GPU
// from the requests' lengths.
//
// Per request s (L cached positions, N arriving, page size P):
//   add = max(N, 0); have = ceil(L/P); need = N < 0 ? 0 : ceil((L+add)/P) - have
//   back = N < 0 ? have : 0          pages a finished request returns
// With R the returned pages in the order of requests and columns (r of them) and f
// free pages, the k-th page taken is the k-th from the top of free[0..f) ++ R, so a
// step takes returned pages first.  Token t of request s has position
// L + t - cu[s], cu the exclusive prefix sum of add.
//
// One launch.  Every CTA scans all lengths into shared memory (at most 4096
// requests, 8 a thread: 32 KB from L2, cheaper than a second launch or a wait
// between CTAs), then the grid shares the tokens, the new table entries and the
// pushed pages; each finds its request by a binary search in shared memory, and no
// item reads what another one writes.  Lengths and n_free may be updated in place,
// so the last CTA to arrive writes them, after every CTA has read them.
//
// Bound by latency: the lengths' load, the scan, the search, the free page, the store,
// each waiting for the one before.  8 requests of one token 3.2 us (one CTA, which needs
// no arrival), 2048 requests with up to 200 tokens each 9.5 us, of which 2.2 MB take 0.3.
// Two and three CTAs a multiprocessor took 11.4 and 14.9 us there, more scanning than they
// saved.
#include "kv4.cuh"
#include "ptx_sync.cuh"

namespace qmoe {

namespace {

constexpr int PL_THREADS = 512;
constexpr int PL_MAX = 8 * PL_THREADS;          // requests

struct Sum3 {
    long long tok, need, back;
};

__device__ __forceinline__ Sum3 operator+(const Sum3& a, const Sum3& b) {
    return {a.tok + b.tok, a.need + b.need, a.back + b.back};
}

__device__ __forceinline__ Sum3 shfl_up3(const Sum3& v, int d) {
    return {__shfl_up_sync(0xffffffffu, v.tok, d), __shfl_up_sync(0xffffffffu, v.need, d),
            __shfl_up_sync(0xffffffffu, v.back, d)};
}

// the last s in [0, n) with pre[s] <= x (pre ascending, pre[0] = 0)
__device__ __forceinline__ int find_owner(const int* pre, int n, int x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (pre[mid] <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

// PER: requests a thread scans, no more than there have to be: a small step is latency
// alone, and the code of eight takes longer to fetch than to run (8 requests, 5.6 us with
// PER 8 and 3.3 with 1).
template <int PER>
__global__ void __launch_bounds__(PL_THREADS) kv4_plan_kernel(const Kv4PlanArgs a) {
    extern __shared__ int sm[];
    int* s_len = sm;                            // [n]
    int* p_tok = s_len + a.n;                   // [n] exclusive prefix sums
    int* p_need = p_tok + a.n;
    int* p_back = p_need + a.n;
    __shared__ Sum3 warp_sum3[PL_THREADS / 32];
    __shared__ int why;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) why = 0;
    pdl_wait();
    pdl_launch_dependents();
    const int f = *a.n_free;
    __syncthreads();

    Sum3 mine[PER], run{0, 0, 0};
    int bad = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int s = tid * PER + i;
        mine[i] = run;
        if (s < a.n) {
            const int L = a.seq_len[s], N = a.new_len[s];
            s_len[s] = N < 0 ? ~L : L;                 // the sign tells finished requests apart
            if (L < 0 || (long long)L > (long long)a.width * a.page) {
                bad = max(bad, ST_DEVICE_CHECK);
            } else {
                const long long end = (long long)L + (N > 0 ? N : 0);
                const long long have = (L + a.page - 1) / a.page, all = (end + a.page - 1) / a.page;
                if (all > a.width) bad = max(bad, 4);
                run = run + Sum3{N > 0 ? N : 0, N < 0 ? 0 : all - have, N < 0 ? have : 0};
            }
        }
    }
    if (bad) atomicMax(&why, bad);
    Sum3 inc = run;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const Sum3 o = shfl_up3(inc, d);
        if (lane >= d) inc = inc + o;
    }
    if (lane == 31) warp_sum3[warp] = inc;
    __syncthreads();
    Sum3 before{0, 0, 0}, total{0, 0, 0};
#pragma unroll
    for (int w = 0; w < PL_THREADS / 32; ++w) {
        if (w < warp) before = before + warp_sum3[w];
        total = total + warp_sum3[w];
    }
    const Sum3 base = {before.tok + inc.tok - run.tok, before.need + inc.need - run.need,
                       before.back + inc.back - run.back};
    // the step is served as a whole or not at all
    int st = why;
    if (st == 0 || st == 4) {
        const long long left = (long long)f + total.back - total.need;
        if (f < 0 || f > a.n_pages || left > a.n_pages) st = ST_DEVICE_CHECK;
        else if (st == 0 && total.tok > a.cap) st = 4;
        else if (st == 0 && left < 0) st = 5;
    }
    const bool ok = st == 0;
    const int n_tok = ok ? (int)total.tok : 0, n_need = ok ? (int)total.need : 0, n_back = ok ? (int)total.back : 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int s = tid * PER + i;
        if (s < a.n) {
            const Sum3 p = base + mine[i];
            p_tok[s] = ok ? (int)p.tok : 0;
            p_need[s] = ok ? (int)p.need : 0;
            p_back[s] = ok ? (int)p.back : 0;
        }
    }
    __syncthreads();

    const int gtid = blockIdx.x * PL_THREADS + tid, gn = gridDim.x * PL_THREADS;
    // the i-th returned page, the k-th page taken, the page of column c of request s
    auto returned = [&](int i) {
        const int s = find_owner(p_back, a.n, i);
        return a.table[(size_t)s * a.width + (i - p_back[s])];
    };
    auto taken = [&](int k) { return k < n_back ? returned(n_back - 1 - k) : a.free_pages[f - 1 - (k - n_back)]; };
    auto len_of = [&](int s) { return s_len[s] < 0 ? ~s_len[s] : s_len[s]; };
    auto have_of = [&](int s) { return (len_of(s) + a.page - 1) / a.page; };
    // Page ids are handed on as they are; one that is no page's is reported, and its tokens go nowhere.  Every
    // page that is taken has a token.
    auto is_page = [&](int pg) {
        const bool good = (unsigned)pg < (unsigned)a.n_pages;
        if (!good) atomicExch(a.status, ST_DEVICE_CHECK);
        return good;
    };

    for (int t = gtid; t < a.cap; t += gn) {
        int pos = -1;
        int64_t slot = -1;
        if (t < n_tok) {
            const int s = find_owner(p_tok, a.n, t);
            pos = len_of(s) + (t - p_tok[s]);
            const int c = pos / a.page, h = have_of(s);
            const int pg = c < h ? a.table[(size_t)s * a.width + c] : taken(p_need[s] + c - h);
            if (is_page(pg)) slot = (int64_t)pg * a.page + (pos - c * a.page);
        }
        a.positions[t] = pos;
        a.slots[t] = slot;
    }
    for (int k = gtid; k < n_need; k += gn) {
        const int s = find_owner(p_need, a.n, k);
        a.table[(size_t)s * a.width + have_of(s) + (k - p_need[s])] = taken(k);
    }
    for (int i = gtid; i < n_back - n_need; i += gn) {
        const int pg = returned(i);
        is_page(pg);
        a.free_pages[f + i] = pg;
    }
    for (int s = gtid; s <= a.n; s += gn) a.cu[s] = s < a.n ? p_tok[s] : n_tok;

    // last CTA out: every CTA has read the lengths and n_free
    if (gridDim.x > 1) {
        __shared__ int last;
        __syncthreads();
        if (tid == 0) {
            __threadfence();
            last = atomicAdd(a.arrive, 1u) == gridDim.x - 1;
        }
        __syncthreads();
        if (!last) return;
        if (tid == 0) *a.arrive = 0u;
    } else {
        __syncthreads();
    }
    for (int s = tid; s < a.n; s += PL_THREADS) {
        const int add = (s + 1 < a.n ? p_tok[s + 1] : n_tok) - p_tok[s];
        a.seq_len_out[s] = !ok ? a.seq_len[s] : s_len[s] < 0 ? 0 : s_len[s] + add;
    }
    if (tid == 0) {
        *a.n_free_out = f + n_back - n_need;
        if (!ok) atomicExch(a.status, st);
    }
}

}  // namespace

cudaError_t kv4_plan_prepare() {
    static_assert(sizeof(int) * 4 * PL_MAX <= 64 * 1024, "the scan's shared memory");
    return cudaFuncSetAttribute(kv4_plan_kernel<8>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)(sizeof(int) * 4 * PL_MAX));
}

cudaError_t launch_kv4_plan(const Kv4PlanArgs& a, int num_sms, cudaStream_t st) {
    const int items = a.cap > a.n ? a.cap : a.n;
    int grid = (items + PL_THREADS - 1) / PL_THREADS;
    if (grid > num_sms) grid = num_sms;
    const size_t smem = sizeof(int) * 4 * (size_t)a.n;
    const int per = (a.n + PL_THREADS - 1) / PL_THREADS;
    return launch_pdl(per <= 1 ? kv4_plan_kernel<1> : per <= 2 ? kv4_plan_kernel<2> : per <= 4 ? kv4_plan_kernel<4>
                                                                                       : kv4_plan_kernel<8>,
                      dim3(grid), dim3(PL_THREADS), smem, st, a);
}

}  // namespace qmoe
