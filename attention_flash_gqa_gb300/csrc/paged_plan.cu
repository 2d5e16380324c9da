// The plan of one step over a paged cache, made on the GPU from the requests' lengths: which pages each
// request takes, and for every new token its position, its cache slot and its row.
//
// With kv_b cached tokens, n_b new ones and held_b pages in the block table, request b needs
//     need_b = max(0, ceil((kv_b + n_b) / 16) - held_b)
// more pages. Requests are admitted in order up to the first one whose tokens would pass the T rows or
// whose pages would pass the F free ones; from there on nothing is taken (n_b = need_b = 0). Then
//     cu_q = exclusive prefix sum of n,   off = exclusive prefix sum of need,
//     table[b, held_b + i] = free[used + off_b + i]           for i < need_b,
//     row cu_q[b] + i: position kv_b + i, slot = table[b, position / 16] * 16 + position % 16.
//
// There is next to nothing to move (24 bytes a request, 8 a token, 8 a page taken), so the call is bound
// by latency: one launch, and no value passes from one CTA to another. Every CTA scans all requests
// itself into shared memory (R <= 16384: two prefix sums of 64 KB) and then fills its share of the rows
// and pages. Where there are more rows than threads, a thread takes four consecutive ones, or eight if there
// are more than four a thread: it finds the request of the first by bisection of the prefix sums, steps on
// from there, reads a page id once for rows of one page, and stores 16 bytes at a time where the outputs are
// aligned (1000 requests, 500 thousand rows: 6.5 us by eights, 7.1 by fours, 9.4 a row at a time). Otherwise
// it takes one (64 requests of one row each: 2.9 us against 4.2 by fours, whose rows read the state of four
// requests one after the other). A new
// page's id is read from the free list, not from the table, so no row waits for another thread's table
// entry.
//
// The lengths, held pages and the free list's cursor may be updated in place: the CTAs are then one
// cluster, and all of them have read the old state before the first writes the new (a cluster barrier): eight
// SMs at most, so a long step takes longer (the 500 thousand rows 38 us; 64 requests of one row 3.4).
// Otherwise the grid is as wide as the rows need. Programmatic serialisation hides the launch behind the
// end of the kernel in front (1000 requests, call after call: 10.2 -> 7.5 us).
#include <cuda_runtime.h>

#include "attn_internal.h"
#include "ptx.cuh"

namespace attn {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kCluster = 8;
constexpr int kPage = 16;
constexpr int kMaxReqs = 16384;
constexpr size_t prefix_bytes(int R) { return (size_t)(R + 1) * 2 * sizeof(int); }

// What request b asks for; an inconsistent one asks for nothing.
struct Ask {
    int n, need;
    bool bad;
};
__device__ __forceinline__ Ask ask_of(const PlanLaunch& a, int b) {
    const int kv = a.kv_lens[b], n = a.new_lens[b], held = a.held[b];
    const long long cap = (long long)a.max_pages * kPage;
    if (kv < 0 || n < 0 || held < 0 || held > a.max_pages || kv > (long long)held * kPage || (long long)kv + n > cap)
        return {0, 0, true};
    const int pages = (int)(((long long)kv + n + kPage - 1) / kPage);
    return {n, pages > held ? pages - held : 0, false};
}

// Largest b with first[b] <= x, over first[0 .. count).
__device__ __forceinline__ int owner(const int* first, int count, int x) {
    int lo = 0, hi = count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (first[mid] <= x) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

template <bool IN_PLACE, int PER>  // PER: rows a thread takes at a time
__global__ void __launch_bounds__(kThreads) paged_plan_kernel(const __grid_constant__ PlanLaunch a) {
    extern __shared__ int prefix[];
    const int R = a.R;
    int* cu = prefix;           // [R + 1] tokens before request b
    int* off = prefix + R + 1;  // [R + 1] pages taken before request b
    __shared__ long long warp_n[kWarps], warp_p[kWarps];
    __shared__ int first_out;  // first request that is not admitted
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    griddep_wait();
    const int used = *a.used;
    const bool used_ok = used >= 0 && used <= a.F;
    const long long room = used_ok ? a.F - used : 0;
    if (tid == 0) first_out = R;

    // each thread's run of requests, then the scan of the threads' sums (64 bits: lengths are not trusted)
    const int per = (R + kThreads - 1) / kThreads;
    const int b0 = min(tid * per, R), b1 = min(b0 + per, R);
    long long sn = 0, sp = 0;
    bool bad = !used_ok;
    for (int b = b0; b < b1; ++b) {
        const Ask k = ask_of(a, b);
        sn += k.n, sp += k.need;
        bad |= k.bad;
    }
    long long xn = sn, xp = sp;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long yn = __shfl_up_sync(0xffffffffu, xn, d), yp = __shfl_up_sync(0xffffffffu, xp, d);
        if (lane >= d) xn += yn, xp += yp;
    }
    if (lane == 31) warp_n[warp] = xn, warp_p[warp] = xp;
    __syncthreads();
    xn -= sn, xp -= sp;
    for (int w = 0; w < warp; ++w) xn += warp_n[w], xp += warp_p[w];
    const int big = 0x7fffffff;
    for (int b = b0; b < b1; ++b) {
        const Ask k = ask_of(a, b);
        cu[b] = (int)min(xn, (long long)big), off[b] = (int)min(xp, (long long)big);
        xn += k.n, xp += k.need;
        if (xn > a.T || xp > room) {
            atomicMin(&first_out, b);
            bad = true;
            // the sums only grow: the rest of this run is not admitted either
            for (int i = b + 1; i < b1; ++i) cu[i] = off[i] = big;
            break;
        }
    }
    if (tid == kThreads - 1) cu[R] = (int)min(xn, (long long)big), off[R] = (int)min(xp, (long long)big);
    if (bad) atomicOr(a.status, DEVSTAT_BOUNDS);
    __syncthreads();
    const int adm = first_out;  // requests 0 .. adm - 1 are served
    const int tokens = cu[adm], pages = off[adm];

    const int gtid = blockIdx.x * kThreads + tid, gsize = gridDim.x * kThreads;
    auto checked = [&](int page) -> int {
        if (page >= 0 && page < a.num_pages) return page;
        atomicOr(a.status, DEVSTAT_BOUNDS);
        return -1;
    };
    // pages taken -> block table
    for (int i = gtid; i < pages; i += gsize) {
        const int b = owner(off, adm, i);
        a.table[(size_t)b * a.max_pages + a.held[b] + (i - off[b])] = checked(a.free_pages[used + i]);
    }
    // rows
    const bool wide = PER >= 4 && ((reinterpret_cast<uintptr_t>(a.positions) | reinterpret_cast<uintptr_t>(a.slots)) & 15u) == 0;
    const int groups = a.T / PER + (a.T % PER != 0);
    for (int g = gtid; g < groups; g += gsize) {
        const int t0 = PER * g;
        int pos[PER], slot[PER];
        int b = t0 < tokens ? owner(cu, adm, t0) : 0, at = -1, page = -1;  // page: of block-table entry `at`
        int kv = 0, held = 0, row = -1;                                    // of request `row`
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int t = t0 + i;
            pos[i] = 0, slot[i] = -1;
            if (t < tokens) {
                while (t >= cu[b + 1]) ++b;
                if (b != row) row = b, at = -1, kv = a.kv_lens[b], held = a.held[b];
                pos[i] = kv + (t - cu[b]);
                const int p = pos[i] / kPage;
                if (p != at) {
                    at = p;
                    page = checked(p < held ? a.table[(size_t)b * a.max_pages + p] : a.free_pages[used + off[b] + p - held]);
                }
                if (page >= 0) slot[i] = page * kPage + pos[i] % kPage;
            }
        }
        if (wide && t0 + PER <= a.T) {
#pragma unroll
            for (int i = 0; i + 3 < PER; i += 4) {
                *reinterpret_cast<int4*>(a.positions + t0 + i) = make_int4(pos[i], pos[i + 1], pos[i + 2], pos[i + 3]);
                *reinterpret_cast<int4*>(a.slots + t0 + i) = make_int4(slot[i], slot[i + 1], slot[i + 2], slot[i + 3]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < PER; ++i)
                if (t0 + i < a.T) a.positions[t0 + i] = pos[i], a.slots[t0 + i] = slot[i];
        }
    }
    // the new state
    if (IN_PLACE) cluster_sync_all();  // every CTA of the grid has read the old one
    for (int b = gtid; b < R; b += gsize) {
        const bool in = b < adm;
        // in place, another thread of the grid never writes request b: its old state is still there
        const int kv = a.kv_lens[b], held = a.held[b];
        a.cu_q[b] = in ? cu[b] : tokens;
        a.seq_lens[b] = in ? kv + (cu[b + 1] - cu[b]) : kv;
        a.held_out[b] = in ? held + (off[b + 1] - off[b]) : held;
    }
    if (gtid == 0) {
        a.cu_q[R] = tokens;
        *a.used_out = used + pages;
        *a.admitted = adm;
    }
}

template <bool IN_PLACE, int PER>
cudaError_t launch_t(const PlanLaunch& L, cudaStream_t stream) {
    const size_t smem = prefix_bytes(L.R);
    cudaError_t e = cudaSuccess;
    // Beyond what a kernel may use unasked (static shared memory counts). The limit belongs to the kernel, not to the
    // call: every call sets the same, so that none lowers it between another thread's setting and its launch.
    if (smem > 48 * 1024 - 512)
        e = cudaFuncSetAttribute(paged_plan_kernel<IN_PLACE, PER>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)prefix_bytes(kMaxReqs));
    if (e != cudaSuccess) return e;
    const long long rows = ((long long)L.T + PER - 1) / PER, items = rows > L.R ? rows : L.R;
    const long long want = items > kThreads ? (items + kThreads - 1) / kThreads : 1, most = IN_PLACE ? kCluster : L.sms;
    const int grid = (int)(want < most ? want : most);
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = grid;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = IN_PLACE ? 2 : 1;
    const ProfMark m = prof_begin(stream, "paged_plan");
    e = cudaLaunchKernelEx(&cfg, paged_plan_kernel<IN_PLACE, PER>, L);
    prof_end(stream, m);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_plan(const PlanLaunch& L, cudaStream_t stream) {
    if (L.R > kMaxReqs) return cudaErrorInvalidValue;
    const int threads = (L.in_place ? kCluster : L.sms) * kThreads;
    if (L.T / 4 > threads) return L.in_place ? launch_t<true, 8>(L, stream) : launch_t<false, 8>(L, stream);
    if (L.T > threads) return L.in_place ? launch_t<true, 4>(L, stream) : launch_t<false, 4>(L, stream);
    return L.in_place ? launch_t<true, 1>(L, stream) : launch_t<false, 1>(L, stream);
}

}  // namespace attn
