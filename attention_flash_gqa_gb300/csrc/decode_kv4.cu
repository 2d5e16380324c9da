// Single-token decode over the 4-bit paged cache (kv4.cuh has the format), optionally over a sliding window with sinks.
//
// Definition: attn_decode_paged over the values that the cache stands for. Every visible byte of the cache is read once;
// at 18 D bytes a page and KV head against 64 D in bf16 the arithmetic is no longer free. Measured, call after call: 12 contexts of 5 to
// 60 thousand keys, 8 heads of 128: 104 us for 498 MB, 0.70 of the copy rate (in bf16 its 1.77 GB alone would take 261); 64 requests of 256
// to 1024: 20.0 us for 46 MB; 33 requests, 16 heads of 256, window 1024, 4 sinks: 40.0 us for 150 MB. What bounds it: the same rings
// without arithmetic take 82 us over the long contexts. A unit at D = 128 is 360 instructions of a warp, 162 of them shifts and masks, whose
// pipe is half as wide, and 63 % of the issue slots are used: K's part alone takes 89 us, V's alone 100. The batch pays 5 us of layout and
// first records, and 2 of the join's launch.
//
//  * A unit is one page of one KV head: a record, contiguous. The units of a call lie in the order (request, head, page), and
//    every warp of the grid takes an equal stretch of them. It fetches them itself, one bulk copy a unit, through a ring of its
//    own, two units a barrier, four ahead (eight at D = 64): warps never wait for each other. 32 units' page ids and masks are worked out at a time,
//    one a lane, 32 units before they are needed.
//  * A unit is two chains of warp MMAs with the tokens, then the dims, as the 16 rows and the group's query heads as the 8
//    columns: S^T = K Q^T, O^T += V^T P^T. (With the heads as rows, as the bf16 decode has them, at least half of
//    each product would be rows of zeros.) Codes become bf16 operands in registers:
//      K: by masking alone. Bits 4 .. 7 of a bf16 pattern whose other bits are zero are the number code * 2^-129 (below the
//         smallest exponent and in the one after it the spacing is the same), bits 0 .. 3 are code * 2^-133. The missing powers
//         of two sit in q, whose rows are brought to 2^120 at the start of a segment, and in the factor of the scores. The
//         scale of a group of 32 dims is applied to its part of the score in fp32, and 8 sum(q) s taken away for all groups by one
//         more MMA;
//      V: by masking too, and one fused multiply-add for two tokens: (code 2^-129) (s 2^(129 - down)) - 8 s 2^-down, exact (at
//         least for s above 2^(down - 126)). `down`, 6 at first, follows the largest scale that a lane's dims have met, as the
//         softmax's maximum does, so that the factor stays finite. Masks and shifts share a pipe that is half as wide as the
//         instruction rate, multiplications have another one.
//         P is rounded to bf16, as everywhere in this library; turned from columns to rows by movmatrix.
//    The softmax stays in registers (running maximum that moves only past 2^8, as in the bf16 decode).
//  * A stretch may hold several (request, head) segments and begin and end inside one. What a warp finishes alone it writes
//    out. The other pieces (o, m, l) meet in shared memory at the end of the block; those that begin or end
//    outside it go to the workspace, at most two a block, and a second kernel joins them.
#include <cuda_runtime.h>

#include <algorithm>

#include "attn_internal.h"
#include "kv4.cuh"
#include "ptx.cuh"

namespace attn {
namespace {

constexpr int kPage = 16;
constexpr int kMaxB = 4096;
constexpr uint32_t kSmemLimit = 232448;
constexpr int kMaxG = 8;  // query heads of a KV head: the columns of an MMA

template <int D>
struct Cfg {
    static constexpr int kWarps = D == 256 ? 8 : 16;
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int kStages = D == 64 ? 4 : 2;  // of each warp's ring: two units each
    static constexpr int kRow = D + 4;                             // floats of a piece's row: o, m, l, padding
    static constexpr uint32_t kOffBar = kWarps * kStages * 2 * kv4_record_bytes(D);  // [warp][stage]
    static constexpr uint32_t kOffMeta = kOffBar + kWarps * kStages * 8;         // abort flag, sums, segments of pieces
    static constexpr uint32_t kOffHead = kOffMeta + (4 * (4 + 3 * kWarps) + 15) / 16 * 16;  // [warp][G][kRow]: first pieces
    // behind it [B + 1] pages before a request, and [B] their lengths where there is room
    static uint32_t smem_bytes(int B, int G, bool lens) { return kOffHead + kWarps * G * kRow * 4 + (B + 1) * 4 + (lens ? B * 4 : 0) + 128; }
    static_assert(kOffHead + kWarps * kMaxG * kRow * 4 + (kMaxB + 1) * 4 + 128 <= kSmemLimit, "shared memory");
    // a warp's last piece is put where its own ring was
    static_assert(kMaxG * kRow * 4 <= kStages * 2 * kv4_record_bytes(D), "ring");
};

struct Args {
    const uint16_t* q;
    const uint8_t* cache;
    const int32_t *block_table, *seq_lens;
    uint16_t* o;
    float* lse;
    float* part;     // [block][2][G][kRow]
    int32_t* starts;  // [B + 1] pages before a request, for the join of many requests; null: it sums the lengths itself
    unsigned* status;
    int B, Hq, Hkv, G, max_pages, num_pages, window, sink;
    bool lens_here;  // the lengths are kept in shared memory
    float scale_log2;
};

// mma_16x8x16_bf16 from zero: d = a b.
__device__ __forceinline__ void mma0(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void lds64(uint32_t addr, uint32_t& a, uint32_t& b) {
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(a), "=r"(b) : "r"(addr) : "memory");
}
__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
    uint32_t a;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(a) : "r"(addr) : "memory");
    return a;
}

// First token of the window of a request's query.
__device__ __forceinline__ int first_token(const Args& a, int L) { return a.window > 0 && L > a.window ? L - a.window : 0; }
// Pages of sinks in front of the window's first page.
__device__ __forceinline__ int sink_pages(const Args& a, int L) { return min((a.sink + kPage - 1) / kPage, first_token(a, L) / kPage); }
__device__ __forceinline__ int seen_pages(const Args& a, int L) {
    return L > 0 ? (L - 1) / kPage - first_token(a, L) / kPage + 1 + sink_pages(a, L) : 0;
}
// A value that another kernel may be writing: read from L2, and again at every call.
__device__ __forceinline__ int32_t load_l2(const int32_t* p) {
    int32_t v;
    asm volatile("ld.global.cg.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}
// Length of request b within its block-table row.
__device__ __forceinline__ int req_len(const Args& a, int b, bool record) {
    const int L = load_l2(a.seq_lens + b);
    const long long cap = (long long)a.max_pages * kPage;
    if (L >= 0 && L <= cap) return L;
    if (record) atomicOr(a.status, DEVSTAT_BOUNDS);
    return L < 0 ? 0 : (int)cap;
}

constexpr uint32_t kLowNibbles = 0x000f000fu, kHighNibbles = 0x00f000f0u;
// Least and largest exponent by which O's sums are kept down. Scales up to 2^(down - 6) times 16 times 2^(129 - down) are finite.
constexpr int kDownMin = 6, kDownMax = 129;
static_assert(kDownMin + 121 >= 127, "scales below 2 need no look");

// A unit as its warp needs it.
struct Unit {
    const uint8_t* record;  // null: its page id is outside the pool (reported, its tokens are not seen)
    int segment;            // request * Hkv + head
    uint32_t see;           // bits 0 .. 15: visible tokens; 16: first of its segment; 17: last
};

// `units` are shared out over `blocks`, the first units % blocks of which have one more.
struct Share {
    int each, more;
    __device__ Share(int units, int blocks) : each(units / blocks), more(units - each * blocks) {}
    __device__ int first(int k) const { return k * each + min(k, more); }
    __device__ int owner(int u) const {  // the block that unit u is in
        const int at = u - more * (each + 1);
        return at < 0 ? u / (each + 1) : more + at / each;
    }
};

__device__ __forceinline__ float log_sum(float M, float L) { return L == 0.f ? -INFINITY : (M + __log2f(L)) * 0.69314718055994531f; }

template <int D>
__global__ void __launch_bounds__(Cfg<D>::kThreads, 1) decode_kv4_kernel(Args a) {
    using C = Cfg<D>;
    using F = Kv4<D>;
    constexpr int kGroups = F::kGroups, kBlocks = D / F::W, kTiles = F::W / 16;  // tiles of 16 dims in a block
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));
    float* head_piece = reinterpret_cast<float*>(smem + C::kOffHead);
    int32_t* start = reinterpret_cast<int32_t*>(head_piece + C::kWarps * a.G * C::kRow);
    int32_t* lens = a.lens_here ? start + a.B + 1 : nullptr;
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMeta);
    int* warp_sum = reinterpret_cast<int*>(smem + C::kOffMeta) + 4;
    // a warp's first piece and its last one: segment << 2 | whether it ends in the warp's stretch | whether it began there; -1: none
    int* head_piece_of = warp_sum + C::kWarps;
    int* tail_piece = head_piece_of + C::kWarps;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, c = lane & 3;
    uint8_t* ring = smem + warp * (2 * C::kStages * F::kRecord);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kOffBar) + warp * C::kStages;
    if (tid == 0) *abort_flag = 0;
    if (lane == 0) {
        for (int s = 0; s < C::kStages; ++s) mbar_init(smem_u32(&full[s]), 2);
        head_piece_of[warp] = tail_piece[warp] = -1;
        fence_mbar_init();
    }
    const uint64_t policy = l2_policy_evict_first();  // every byte is read once
    int u0 = 0, u1 = 0, n = 0;  // the warp's stretch
    const int32_t* entry = nullptr;  // of the last unit worked out: its block-table entry and what it held
    int entry_page = -1;
    auto unit_at = [&](uint32_t at, bool record) -> Unit {
        Unit r = {nullptr, -1, 0u};
        entry = nullptr;
        if (at >= (uint32_t)u1) return r;  // (past the last unit it may be above 2^31)
        const int u = (int)at;
        int lo = 0, hi = a.B - 1;  // the last request that starts at or before u: it has pages
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (start[mid] * a.Hkv <= u) lo = mid;
            else hi = mid - 1;
        }
        const int np = start[lo + 1] - start[lo], rem = u - start[lo] * a.Hkv;
        const int h = rem / np, i = rem - h * np;
        const int L = lens ? lens[lo] : req_len(a, lo, false);
        const int first = first_token(a, L), early = sink_pages(a, L);
        const int p = i < early ? i : first / kPage + i - early;
        const int end = min(kPage, (i < early ? a.sink : L) - p * kPage);
        uint32_t see = low_bits(end);
        // the window's first page: tokens before the window are seen only if they are sinks
        if (i == early) see &= ~low_bits(first % kPage) | low_bits(a.sink - p * kPage);
        entry = a.block_table + (size_t)lo * a.max_pages + p, entry_page = load_l2(entry);
        if (entry_page >= 0 && entry_page < a.num_pages) {
            r.record = a.cache + ((size_t)entry_page * a.Hkv + h) * F::kRecord;
        } else {
            if (record) atomicOr(a.status, DEVSTAT_BOUNDS);
            see = 0u;
        }
        r.segment = lo * a.Hkv + h;
        r.see = see | (i == 0 ? 1u << 16 : 0u) | (i == np - 1 ? 1u << 17 : 0u);
        return r;
    };
    // Units first .. first + count - 1 (pairs of them), those from n on being none: by the lanes that have them.
    auto issue = [&](int first, int count, const uint8_t* record) {
        const int x = (lane - first) & 31;
        if (x < count) {
            const uint32_t u = first + x, slot = u % (2 * C::kStages), bar = smem_u32(&full[slot / 2]);
            if ((int)u < n && record) {
                mbar_expect_tx(bar, F::kRecord);
                bulk_load_hint(smem_u32(ring + slot * F::kRecord), record, F::kRecord, bar, policy);
            } else {
                mbar_arrive(bar);
            }
        }
    };

    // ---- the layout: pages before every request, the warp's stretch and its first units -----------------
    // Launched with programmatic serialisation the block may be here before the kernel in front ends. Lengths, block table and
    // cache may be what that one writes, so what counts is read after griddep_wait; but with up to a request a thread the
    // layout is made before it, on a guess, from lengths and page ids as they are in L2, and the first records asked for
    // there. After the wait the first copies start by that layout, and while they are on their way what it was made
    // from is read again; if anything differs the copies are waited for and all of it is done anew.
    const bool guess = lens && a.B <= C::kThreads;
    Unit nxt = {};
    uint32_t flip = 0;  // 1: the barriers are a phase ahead
    for (bool sure = !guess;;) {
        if (!guess) griddep_wait();
        const int per = (a.B + C::kThreads - 1) / C::kThreads, b0 = tid * per;
        int mine = 0;
        for (int b = b0; b < min(a.B, b0 + per); ++b) {
            const int L = req_len(a, b, sure && blockIdx.x == 0);
            if (lens) lens[b] = L;
            mine += seen_pages(a, L);
        }
        int v = mine;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, v, off);
            if (lane >= off) v += y;
        }
        if (lane == 31) warp_sum[warp] = v;
        __syncthreads();
        int at = v - mine;
        for (int w = 0; w < warp; ++w) at += warp_sum[w];
        for (int b = b0; b < min(a.B, b0 + per); ++b) {
            start[b] = at;
            at += per == 1 ? mine : seen_pages(a, lens ? lens[b] : req_len(a, b, false));
        }
        if (b0 < a.B && b0 + per >= a.B) start[a.B] = at;
        __syncthreads();
        const int units = start[a.B] * a.Hkv;
        const int blocks = min((int)gridDim.x, units);  // every one that takes part has a unit
        u0 = u1 = n = 0;
        if ((int)blockIdx.x < blocks) {
            const Share share(units, blocks);
            const int first = share.first(blockIdx.x), many = share.first(blockIdx.x + 1) - first;
            // (a block's units times its warps stay within 32 bits: 2^31 units are at least 152 blocks')
            u0 = first + (int)((uint32_t)many * warp / C::kWarps), u1 = first + (int)((uint32_t)many * (warp + 1) / C::kWarps);
            n = u1 - u0;
        }
        nxt = unit_at((uint32_t)u0 + lane, sure);
        if (!sure) {
            if (lane < min(n, 2 * C::kStages) && nxt.record) prefetch_bulk(nxt.record, F::kRecord);
            griddep_wait();
        }
        issue(0, 2 * C::kStages, nxt.record);
        if (sure) break;
        bool same = true, bad = false;
        if (tid < a.B) {
            const int L = load_l2(a.seq_lens + tid);
            const bool within = L >= 0 && L <= (long long)a.max_pages * kPage;
            same = lens[tid] == (within ? L : L < 0 ? 0 : a.max_pages * kPage), bad = !within;
        }
        if (entry) same &= load_l2(entry) == entry_page, bad |= !nxt.record;
        same = __syncthreads_and(same);
        if (same && bad) atomicOr(a.status, DEVSTAT_BOUNDS);
        if (same) break;
        if (lane == 0)
            for (int s = 0; s < C::kStages; ++s) mbar_drain(smem_u32(&full[s]), 0, a.status, 0x63);
        __syncwarp();
        flip = 1, sure = true;
    }
    if (a.starts && blockIdx.x == 0)
        for (int b = tid; b <= a.B; b += C::kThreads) a.starts[b] = start[b];
    // the second kernel may be placed from here on; it waits for this one's end
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    uint32_t qf[kGroups][4];  // lane (g, c): head g, dims 8c .. 8c+7 of a group, scaled
    uint32_t eight[3];        // operand (b0, b1, and b0 of a second step) of the product that takes the codes' 8 away
    float factor[2];          // of a product of heads 2c and 2c+1: softmax scale and the powers of two, in log2 units
    // tile t: dims 128 block + (W/8) g + 2 t, + 1 of heads 2c, 2c+1: {(d, h), (d, h+1), (d+1, h), (d+1, h+1)}, times 2^-down
    float o[kBlocks][kTiles][4] = {};
    int down[kBlocks];
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};  // heads 2c, 2c+1 (l: this lane's share)
    float m_use[2] = {0.f, 0.f};                             // m, but 0 where nothing was seen yet
    int segment = 0;
    bool began = false;  // the segment began in this stretch
    bool ok = true;
    Unit cur = nxt;
    int described = 1;  // batches of 32 units

    // this lane's values of head 2c + e, dims of block bl in order
    auto out_value = [&](int bl, int e, int d) -> float { return o[bl][d >> 1][(d & 1) * 2 + e]; };
    auto write_piece = [&](float* rows) {  // [head][kRow]
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            if (2 * c + e >= a.G) continue;
            float* row = rows + (2 * c + e) * C::kRow;
#pragma unroll
            for (int bl = 0; bl < kBlocks; ++bl)
#pragma unroll
                for (int d = 0; d < 2 * kTiles; d += 4)
                    *reinterpret_cast<float4*>(row + bl * F::W + 2 * kTiles * g + d) =
                        make_float4(out_value(bl, e, d), out_value(bl, e, d + 1), out_value(bl, e, d + 2), out_value(bl, e, d + 3));
            if (g == 0) row[D] = l[e] == l[e] ? m[e] : INFINITY, row[D + 1] = l[e];  // (NaN: whatever it is joined with)
        }
    };
    auto write_result = [&]() {
        const size_t row0 = (size_t)segment * a.G;  // query head h G of request b: b Hq + h G
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            if (2 * c + e >= a.G) continue;
            const float inv = l[e] == 0.f ? 0.f : 1.f / l[e];
            uint16_t* row = a.o + (row0 + 2 * c + e) * D;
#pragma unroll
            for (int bl = 0; bl < kBlocks; ++bl)
#pragma unroll
                for (int d = 0; d < 2 * kTiles; d += 8) {
                    uint32_t w[4];
#pragma unroll
                    for (int x = 0; x < 4; ++x) w[x] = pack_bf16x2(out_value(bl, e, d + 2 * x) * inv, out_value(bl, e, d + 2 * x + 1) * inv);
                    *reinterpret_cast<uint4*>(row + bl * F::W + 2 * kTiles * g + d) = make_uint4(w[0], w[1], w[2], w[3]);
                }
            if (g == 0) a.lse[row0 + 2 * c + e] = log_sum(m[e], l[e]);
        }
    };

    // Two units at a time, whatever their segments: one wait and one refill for both.
    for (int i = 0; i < n; i += 2) {
        if (32 * described <= i + 16) {  // a batch is worked out half a batch ahead
            nxt = unit_at((uint32_t)u0 + 32u * described + lane, true);
            ++described;
        }
        if ((i & 31) == 0) cur = nxt;
        const uint32_t stage = (uint32_t)i / 2 % C::kStages, phase = ((uint32_t)i / 2 / C::kStages & 1) ^ flip;
        if (ok) {
            ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&full[stage]), phase, abort_flag, a.status, 0x61));
            if (!ok && lane == 0) ring_drain(full, stage, (int)phase, C::kStages, (n - i + 1) / 2, a.status, 0x62);
            __syncwarp();
        }
        uint32_t rec = smem_u32(ring + stage * (2 * F::kRecord));
#pragma unroll 1
        for (int x = i; x < min(i + 2, n); ++x, rec += F::kRecord) {
            const uint32_t see = __shfl_sync(0xffffffffu, cur.see, x & 31);
            if (x == 0 || (see & (1u << 16))) {
                // ---- a new segment ----
                began = (see & (1u << 16)) != 0;
                segment = __shfl_sync(0xffffffffu, cur.segment, x & 31);
                const uint16_t* row = a.q + ((size_t)segment * a.G + g) * D + 8 * c;
#pragma unroll
                for (int gr = 0; gr < kGroups; ++gr) {
                    const uint4 w = g < a.G ? *reinterpret_cast<const uint4*>(row + 32 * gr) : make_uint4(0, 0, 0, 0);
                    qf[gr][0] = w.x, qf[gr][1] = w.y, qf[gr][2] = w.z, qf[gr][3] = w.w;
                }
                // The row's largest exponent goes to 120 (by 2^123 at most): then a product with a code, some 2^-129 of it, is a
                // normal number. Words that meet low nibbles get 2^4 more.
                uint32_t top = 0;
#pragma unroll
                for (int gr = 0; gr < kGroups; ++gr)
#pragma unroll
                    for (int x = 0; x < 4; ++x) top = max(top, max(qf[gr][x] & 0x7f80u, qf[gr][x] >> 16 & 0x7f80u));
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
                const int up = min(247 - (int)(top >> 7), 123);
                const uint32_t by = (uint32_t)(up + 127) * 0x00800080u, by16 = by + 4 * 0x00800080u;
                float minus[kGroups];  // -8 sum of q over a group, head g, in the units of the products
#pragma unroll
                for (int gr = 0; gr < kGroups; ++gr) {
#pragma unroll
                    for (int x = 0; x < 4; ++x) qf[gr][x] = bf16x2_mul(qf[gr][x], x & 1 ? by : by16);
                    float d[4] = {0.f, 0.f, 0.f, 0.f};
                    constexpr uint32_t kLow = 0x80088008u, kHigh = 0x80808080u;  // -8 * 2^-133, -8 * 2^-129
                    mma_16x8x16_bf16(d, kLow, kLow, kHigh, kHigh, qf[gr][0], qf[gr][1]);
                    mma_16x8x16_bf16(d, kLow, kLow, kHigh, kHigh, qf[gr][2], qf[gr][3]);
                    const float even = __shfl_sync(0xffffffffu, d[0], g >> 1), odd = __shfl_sync(0xffffffffu, d[1], g >> 1);
                    minus[gr] = g & 1 ? odd : even;
                }
                {
                    // Taken away through an MMA whose columns are groups: scales (exact) times these sums in three bf16 parts, which
                        // hold all 24 bits. Columns 2c, 2c + 1 of a step: a pair of groups of one part, as many parts a step as there is room for.
                        float x0 = minus[0], x1 = minus[1];
#pragma unroll
                    for (int w = 1; w < kGroups / 2; ++w)
                        if (c % (kGroups / 2) == w) x0 = minus[2 * w], x1 = minus[2 * w + 1];
                    uint32_t part[3];
#pragma unroll
                    for (int x = 0; x < 3; ++x) {
                        part[x] = pack_bf16x2(x0, x1);
                        x0 -= __uint_as_float(part[x] << 16), x1 -= __uint_as_float(part[x] & 0xffff0000u);
                    }
                    if (kGroups == 8) eight[0] = part[0], eight[1] = part[1], eight[2] = part[2];
                    else if (kGroups == 4) eight[0] = c < 2 ? part[0] : part[1], eight[1] = c < 2 ? part[2] : 0u;
                    else eight[0] = c == 0 ? part[0] : c == 1 ? part[1] : c == 2 ? part[2] : 0u, eight[1] = 0u;
                }
                const float fac = fminf(ldexpf(a.scale_log2, 129 - up), 3e38f);
                factor[0] = __shfl_sync(0xffffffffu, fac, 8 * c), factor[1] = __shfl_sync(0xffffffffu, fac, 8 * c + 4);
#pragma unroll
                for (int bl = 0; bl < kBlocks; ++bl) {
                    down[bl] = kDownMin;
#pragma unroll
                    for (int t = 0; t < kTiles; ++t)
#pragma unroll
                        for (int e = 0; e < 4; ++e) o[bl][t][e] = 0.f;
                }
                m[0] = m[1] = -INFINITY, m_use[0] = m_use[1] = l[0] = l[1] = 0.f;
            }
            if (!ok) {  // given up: the rows of this unit and of those behind it in the stretch are NaN
                m[0] = m[1] = INFINITY, l[0] = l[1] = __int_as_float(0x7fc00000);
            } else if (see & 0xffffu) {
                // ---- S^T: tokens g and g + 8, heads 2c and 2c + 1 ----
                float s[4];
                {
                    const int w = 2 * (c % (kGroups / 2));
                    const uint32_t a0 = lds32(rec + F::key_scale(g, w)), a1 = lds32(rec + F::key_scale(g + 8, w));
                    mma0(s, a0, a1, a0, a1, eight[0], eight[1]);
                    if (kGroups == 8) mma_16x8x16_bf16(s, a0, a1, a0, a1, eight[2], 0u);
                }
                uint32_t sw[2][kGroups / 2];  // scales of tokens g, g + 8: two groups a word
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const uint32_t at = rec + F::key_scale(g + 8 * r, 0);
                    if constexpr (kGroups == 8) ld_shared_v4(at, sw[r][0], sw[r][1], sw[r][2], sw[r][3]);
                    else if constexpr (kGroups == 4) lds64(at, sw[r][0], sw[r][1]);
                    else sw[r][0] = lds32(at);
                }
#pragma unroll
                for (int bl = 0; bl < kBlocks; ++bl) {
                    uint32_t kw[2][F::kBlockGroups];
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const uint32_t at = rec + F::key_strip(bl, g + 8 * r, c);
                        if constexpr (F::kBlockGroups == 4) ld_shared_v4(at, kw[r][0], kw[r][1], kw[r][2], kw[r][3]);
                        else lds64(at, kw[r][0], kw[r][1]);
                    }
#pragma unroll
                    for (int x = 0; x < F::kBlockGroups; ++x) {
                        const int gr = bl * F::kBlockGroups + x;
                        float d[4];
                        const uint32_t w0 = kw[0][x], w1 = kw[1][x], y0 = w0 >> 8, y1 = w1 >> 8;
                        mma0(d, w0 & kLowNibbles, w1 & kLowNibbles, w0 & kHighNibbles, w1 & kHighNibbles, qf[gr][0], qf[gr][1]);
                        mma_16x8x16_bf16(d, y0 & kLowNibbles, y1 & kLowNibbles, y0 & kHighNibbles, y1 & kHighNibbles, qf[gr][2], qf[gr][3]);
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            const float sc = __uint_as_float(gr & 1 ? sw[r][gr / 2] & 0xffff0000u : sw[r][gr / 2] << 16);
                            s[2 * r] = fmaf(sc, d[2 * r], s[2 * r]), s[2 * r + 1] = fmaf(sc, d[2 * r + 1], s[2 * r + 1]);
                        }
                    }
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) s[e] *= factor[e & 1];
                const bool whole = (see & 0xffffu) == 0xffffu;
                if (!whole) {
                    if (!(see >> g & 1u)) s[0] = s[1] = -INFINITY;
                    if (!(see >> (g + 8) & 1u)) s[2] = s[3] = -INFINITY;
                }
                // ---- softmax: the maximum moves only when a score is past it by more than 8 (p <= 2^8) ----
                const float top0 = fmaxf(s[0], s[2]), top1 = fmaxf(s[1], s[3]);
                if (__any_sync(0xffffffffu, top0 > m[0] + 8.f || top1 > m[1] + 8.f)) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float mx = e ? top1 : top0;
#pragma unroll 1
                        for (int off = 4; off < 32; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
                        const float to = mx > m[e] + 8.f ? mx : m[e];
                        const float f = m[e] == -INFINITY ? 0.f : fast_exp2(m[e] - to);
                        m[e] = to, l[e] *= f, m_use[e] = to == -INFINITY ? 0.f : to;
#pragma unroll
                        for (int bl = 0; bl < kBlocks; ++bl)
#pragma unroll
                            for (int t = 0; t < kTiles; ++t) o[bl][t][e] *= f, o[bl][t][e + 2] *= f;
                    }
                }
                float p[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    p[e] = fast_exp2(s[e] - m_use[e & 1]);  // (0 for -inf)
                    l[e & 1] += p[e];
                }
                // ---- O^T += V^T P^T ----
                const uint32_t b0 = transpose8(pack_bf16x2(p[0], p[1])), b1 = transpose8(pack_bf16x2(p[2], p[3]));
                uint32_t hide0 = 0xffffffffu, hide1 = 0xffffffffu;  // tokens that are not seen may hold anything: scale 0
                if (!whole) {
                    hide0 = (see >> (2 * c) & 1u ? 0xffffu : 0u) | (see >> (2 * c + 1) & 1u ? 0xffff0000u : 0u);
                    hide1 = (see >> (2 * c + 8) & 1u ? 0xffffu : 0u) | (see >> (2 * c + 9) & 1u ? 0xffff0000u : 0u);
                }
#pragma unroll
                for (int bl = 0; bl < kBlocks; ++bl) {
                    // words[pair][token of the pair][8 dims]
                    constexpr int kWords = F::W / 64;
                    uint32_t vw[2][2][kWords];
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const uint32_t at = rec + F::value_chunk(bl, c + 4 * r, g);
                        if constexpr (kWords == 2) ld_shared_v4(at, vw[r][0][0], vw[r][0][1], vw[r][1][0], vw[r][1][1]);
                        else lds64(at, vw[r][0][0], vw[r][1][0]);
                    }
                    const int gr = bl * F::kBlockGroups + g / (8 / F::kBlockGroups);
                    const uint32_t s0 = lds32(rec + F::value_scale(gr, 2 * c)) & hide0;
                    const uint32_t s1 = lds32(rec + F::value_scale(gr, 2 * c + 8)) & hide1;
                    // Every `down` allows scales below 2: bit 14 of a half says whether there is a larger one, and only then it is looked at
                    // closer, whether its exponent is above what `down` allows (bit 15 of a sum).
                    const uint32_t past = (0x8000u - ((uint32_t)(down[bl] + 122) << 7)) * 0x10001u;
                    if (__any_sync(0xffffffffu, (s0 | s1) & 0x40004000u) &&
                        __any_sync(0xffffffffu, (((s0 & 0x7fff7fffu) + past) | ((s1 & 0x7fff7fffu) + past)) & 0x80008000u)) {
                        uint32_t e = max(max(s0 & 0x7f80u, s0 >> 16 & 0x7f80u), max(s1 & 0x7f80u, s1 >> 16 & 0x7f80u)) >> 7;
                        e = max(e, __shfl_xor_sync(0xffffffffu, e, 1));  // the four lanes of a row
                        e = max(e, __shfl_xor_sync(0xffffffffu, e, 2));
                        const int to = (int)e > down[bl] + 121 ? min((int)e - 121 + 8, kDownMax) : down[bl];
                        const float f = to - down[bl] > 126 ? 0.f : __int_as_float((127 - (to - down[bl])) << 23);
                        down[bl] = to;
#pragma unroll
                        for (int t = 0; t < kTiles; ++t)
#pragma unroll
                            for (int x = 0; x < 4; ++x) o[bl][t][x] *= f;
                    }
                    const uint32_t up_high = (uint32_t)(256 - down[bl]) * 0x00800080u;  // 2^(129 - down)
                    const uint32_t fh0 = bf16x2_mul(s0, up_high), fh1 = bf16x2_mul(s1, up_high);
                    const uint32_t up_low = up_high + 4 * 0x00800080u;
                    const uint32_t minus8 = (up_high - 126 * 0x00800080u) | 0x80008000u;  // -8 * 2^-down
                    const uint32_t fl0 = bf16x2_mul(s0, up_low), fl1 = bf16x2_mul(s1, up_low);
                    const uint32_t c0 = bf16x2_mul(s0, minus8), c1 = bf16x2_mul(s1, minus8);
#pragma unroll
                    for (int half = 0; half < 2 * kWords; ++half) {  // 4 dims of both tokens side by side
                        const uint32_t sel = half & 1 ? 0x7632u : 0x5410u;
                        const uint32_t x0 = __byte_perm(vw[0][0][half / 2], vw[0][1][half / 2], sel);
                        const uint32_t x1 = __byte_perm(vw[1][0][half / 2], vw[1][1][half / 2], sel);
#pragma unroll
                        for (int d = 0; d < 4; d += 2) {
                            const uint32_t y0 = x0 >> (4 * d), y1 = x1 >> (4 * d);
                            mma_16x8x16_bf16(o[bl][half * 2 + d / 2], bf16x2_fma(y0 & kLowNibbles, fl0, c0), bf16x2_fma(y0 & kHighNibbles, fh0, c0),
                                bf16x2_fma(y1 & kLowNibbles, fl1, c1), bf16x2_fma(y1 & kHighNibbles, fh1, c1), b0, b1);
                        }
                    }
                }
            }
            const bool ends = (see & (1u << 17)) != 0, last = x + 1 == n;
            if (ends || last) {
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll 1
                    for (int off = 4; off < 32; off <<= 1) l[e] += __shfl_xor_sync(0xffffffffu, l[e], off);
#pragma unroll
                for (int bl = 0; bl < kBlocks; ++bl) {
                    const float f = __int_as_float((127 + down[bl] / 2) << 23), f2 = __int_as_float((127 + down[bl] - down[bl] / 2) << 23);
#pragma unroll
                    for (int t = 0; t < kTiles; ++t)
#pragma unroll
                        for (int x = 0; x < 4; ++x) o[bl][t][x] = o[bl][t][x] * f * f2;
                }
                if (began && ends) {
                    write_result();
                } else {  // its first piece, of a segment that began in an earlier stretch; or what is left at the end
                    write_piece(last ? reinterpret_cast<float*>(ring) : head_piece + warp * a.G * C::kRow);
                    if (lane == 0) (last ? tail_piece : head_piece_of)[warp] = segment << 2 | (ends ? 2 : 0) | (began ? 1 : 0);
                }
            }
        }
        __syncwarp();  // the records have been read
        if (ok && i + 2 * C::kStages < n) issue(i + 2 * C::kStages, 2, lane >= (i & 31) ? cur.record : nxt.record);
    }
    __syncthreads();
    // ---- pieces of a segment that lie in this block: joined by the warp that has the first ------------
    // Pieces: lanes 0 .. 15 have the warps' last ones, lanes 16 .. 31 their first ones. Those of one segment are the last pieces of
    // warps that it fills or opens in, and the first piece of the warp that it ends in; the warps share out the heads of all segments.
    const int piece = (lane & 15) < C::kWarps ? (lane < 16 ? tail_piece[lane] : head_piece_of[lane - 16]) : -1;
    const uint32_t alike = __match_any_sync(0xffffffffu, piece >> 2);
    uint32_t leads = __ballot_sync(0xffffffffu, piece >= 0 && __ffs(alike) - 1 == lane);  // one lane for each segment
    const float* rows = lane < 16 ? reinterpret_cast<const float*>(smem + lane * (2 * C::kStages * F::kRecord))
                                  : head_piece + (lane - 16) * a.G * C::kRow;
    const int tasks = __popc(leads) * a.G;
    for (int task = warp, at = 0; task < tasks; task += C::kWarps) {
        for (; at < task / a.G; ++at) leads &= leads - 1;  // the segment of this task
        const int hh = task % a.G, seg = __shfl_sync(0xffffffffu, piece, __ffs(leads) - 1) >> 2;
        const bool mine = piece >> 2 == seg;
        uint32_t members = __ballot_sync(0xffffffffu, mine);
        const bool begins = __any_sync(0xffffffffu, mine && (piece & 1)), ends = __any_sync(0xffffffffu, mine && (piece & 2));
        constexpr int N = D / 32;
        const float pm = mine ? rows[hh * C::kRow + D] : -INFINITY, pl = mine ? rows[hh * C::kRow + D + 1] : 0.f;
        float M = pm;
#pragma unroll
        for (int off = 16; off; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
        const float weight = pm == -INFINITY ? 0.f : fast_exp2(pm - M);
        float L = weight * pl, O[N] = {};
#pragma unroll
        for (int off = 16; off; off >>= 1) L += __shfl_xor_sync(0xffffffffu, L, off);
        while (members) {  // four pieces at a time (the last one again, with weight 0, where there are fewer)
            float w[4], x[4][N];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int from = members ? __ffs(members) - 1 : 0;
                const float there = __shfl_sync(0xffffffffu, weight, from);
                w[k] = members ? there : 0.f;
                const float* row = (from < 16 ? reinterpret_cast<const float*>(smem + from * (2 * C::kStages * F::kRecord))
                                              : head_piece + (from - 16) * a.G * C::kRow) + hh * C::kRow + N * lane;
#pragma unroll
                for (int e = 0; e < N; e += 2) {
                    const float2 y = members ? *reinterpret_cast<const float2*>(row + e) : make_float2(0.f, 0.f);
                    x[k][e] = y.x, x[k][e + 1] = y.y;
                }
                members &= members - 1;
            }
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int e = 0; e < N; ++e) O[e] = fmaf(w[k], x[k][e], O[e]);
        }
        const size_t out = (size_t)seg * a.G + hh;
        if (begins && ends) {
            const float inv = L == 0.f ? 0.f : 1.f / L;
#pragma unroll
            for (int e = 0; e < N; e += 2) *reinterpret_cast<uint32_t*>(a.o + out * D + N * lane + e) = pack_bf16x2(O[e] * inv, O[e + 1] * inv);
            if (lane == 0) a.lse[out] = log_sum(M, L);
        } else {
            // at most two segments of a block reach past it: slot 0 the one that began before it
            float* row = a.part + (((size_t)blockIdx.x * 2 + (begins ? 1 : 0)) * a.G + hh) * C::kRow;
#pragma unroll
            for (int e = 0; e < N; e += 2) *reinterpret_cast<float2*>(row + N * lane + e) = make_float2(O[e], O[e + 1]);
            if (lane == 0) row[D] = L == L ? M : INFINITY, row[D + 1] = L;
        }
    }
}

// ---- the second kernel ----------------------------------------------------------------------------
// Joins the pieces of the segments that several blocks of the decode kernel shared; the others are done, but for the rows of requests
// without a key, which come out as o = 0, lse = -inf.
constexpr int kJoinThreads = 128;

// Where the pieces of a segment of `np` units, the first of them `s0`, are: blocks kf .. kl, of kf in its slot `opens` (a block's first
// slot holds what began before it).
struct Pieces {
    int kf, kl, opens;
    __device__ Pieces(const Share& share, int s0, int np) : kf(share.owner(s0)), kl(share.owner(max(s0 + np - 1, s0))), opens(s0 < share.first(kf) ? 0 : 1) {}
};

// A thread has 4 dims of a head; 8 pieces are on their way at once.
template <int D>
__device__ __forceinline__ void join_segment(const Args& a, int segment, int np, const Pieces& at) {
    using C = Cfg<D>;
    const int items = a.G * (D / 4);
    const size_t row0 = (size_t)segment * a.G;
    if (np == 0) {
        for (int it = threadIdx.x; it < items; it += kJoinThreads) {
            *reinterpret_cast<uint2*>(a.o + row0 * D + 4 * it) = make_uint2(0, 0);
            if (it % (D / 4) == 0) a.lse[row0 + it / (D / 4)] = -INFINITY;
        }
        return;
    }
    if (at.kf == at.kl) return;
    for (int it = threadIdx.x; it < items; it += kJoinThreads) {
        const int hh = it / (D / 4), d = 4 * (it % (D / 4));
        float O[4] = {}, M = -INFINITY, L = 0.f;
        for (int k0 = at.kf; k0 <= at.kl; k0 += 8) {
            float4 x[8];
            float2 ml[8];
            float top = M;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                x[j] = make_float4(0.f, 0.f, 0.f, 0.f), ml[j] = make_float2(-INFINITY, 0.f);
                const int k = k0 + j;
                if (k <= at.kl) {
                    const float* row = a.part + (((size_t)k * 2 + (k == at.kf ? at.opens : 0)) * a.G + hh) * C::kRow;
                    x[j] = __ldcg(reinterpret_cast<const float4*>(row + d));
                    ml[j] = __ldcg(reinterpret_cast<const float2*>(row + D));
                }
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) top = fmaxf(top, ml[j].x);
            const float keep = M == -INFINITY ? 0.f : fast_exp2(M - top);
            O[0] *= keep, O[1] *= keep, O[2] *= keep, O[3] *= keep, L *= keep, M = top;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float w = ml[j].x == -INFINITY ? 0.f : fast_exp2(ml[j].x - top);
                O[0] = fmaf(w, x[j].x, O[0]), O[1] = fmaf(w, x[j].y, O[1]), O[2] = fmaf(w, x[j].z, O[2]), O[3] = fmaf(w, x[j].w, O[3]);
                L = fmaf(w, ml[j].y, L);
            }
        }
        const float inv = L == 0.f ? 0.f : 1.f / L;
        *reinterpret_cast<uint2*>(a.o + (row0 + hh) * D + d) = make_uint2(pack_bf16x2(O[0] * inv, O[1] * inv), pack_bf16x2(O[2] * inv, O[3] * inv));
        if (d == 0) a.lse[row0 + hh] = log_sum(M, L);
    }
}

// Up to kSumRequests requests: a block for each segment. Which pieces there are follows from the lengths
// alone, inputs of the call, so that it is known before the decode kernel ends. (It adds 2 us. Registers that let its warps be placed beside the
// decode kernel's blocks, 32 a thread here and 120 there, would gain 0.1 of 20.7 in a batch of 64 and lose 5 of 106 over long contexts; a block
// for each border between blocks instead of each segment loses 1 in the batch.)
template <int D>
__global__ void __launch_bounds__(kJoinThreads) decode_kv4_join_kernel(Args a, int grid) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int segment = blockIdx.x, b = segment / a.Hkv, h = segment - b * a.Hkv, lane = threadIdx.x & 31;
    int first = 0, units = 0;
    for (int i = lane; i < a.B; i += 32) {
        const int np = seen_pages(a, req_len(a, i, false));
        units += np;
        if (i < b) first += np;
    }
#pragma unroll
    for (int off = 16; off; off >>= 1) {
        first += __shfl_xor_sync(0xffffffffu, first, off);
        units += __shfl_xor_sync(0xffffffffu, units, off);
    }
    units *= a.Hkv;
    const int np = seen_pages(a, req_len(a, b, false));
    const Share share(max(units, 1), max(min(grid, units), 1));
    const Pieces at(share, first * a.Hkv + h * np, np);
    griddep_wait();
    join_segment<D>(a, segment, np, at);
}

// More requests: each block looks at `per` segments, one a thread, by the pages that the decode kernel counted, and joins those that need it
// (every block summing all lengths took B^2 Hkv reads).
template <int D>
__global__ void __launch_bounds__(kJoinThreads) decode_kv4_join_many_kernel(Args a, int grid, int per) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    griddep_wait();
    __shared__ uint32_t todo[kJoinThreads / 32];
    const int first = blockIdx.x * per, units = __ldcg(a.starts + a.B) * a.Hkv;
    const Share share(max(units, 1), max(min(grid, units), 1));
    auto pages = [&](int segment, int& s0) -> int {
        const int b = segment / a.Hkv, at = __ldcg(a.starts + b), np = __ldcg(a.starts + b + 1) - at;
        s0 = at * a.Hkv + (segment - b * a.Hkv) * np;
        return np;
    };
    bool mine = false;
    if ((int)threadIdx.x < per && first + (int)threadIdx.x < a.B * a.Hkv) {
        int s0;
        const int np = pages(first + threadIdx.x, s0);
        const Pieces at(share, s0, np);
        mine = np == 0 || at.kf != at.kl;
    }
    const uint32_t vote = __ballot_sync(0xffffffffu, mine);
    if ((threadIdx.x & 31) == 0) todo[threadIdx.x >> 5] = vote;
    __syncthreads();
    for (int w = 0; w < kJoinThreads / 32; ++w) {
        for (uint32_t left = todo[w]; left; left &= left - 1) {
            const int segment = first + 32 * w + __ffs(left) - 1;
            int s0;
            const int np = pages(segment, s0);
            join_segment<D>(a, segment, np, Pieces(share, s0, np));
        }
    }
}

// Requests up to which the join's blocks sum the lengths, which they do while the decode kernel runs. (The whole call, us, this way and by counted
// pages, 8 heads of 128: 64 requests of 512 27 and 28, 128 of 300 28.0 and 29.5, 200 of 300 40 and 37, 1024 of 100 101 and 55, 4096 of 100 849 and
// 152, of 17 779 and 80; 2 heads, 128 of 300 19.2 and 20.3.)
constexpr int kSumRequests = 128;

size_t part_bytes(int G, int D, int grid) { return (size_t)grid * 2 * G * (D + 4) * 4; }

template <int D>
cudaError_t launch_t(const DecodeKv4Launch& L, cudaStream_t stream) {
    using C = Cfg<D>;
    Args a = {};
    a.q = L.q, a.cache = L.cache, a.block_table = L.block_table, a.seq_lens = L.seq_lens, a.o = L.o, a.lse = L.lse;
    a.part = static_cast<float*>(L.workspace);
    a.status = L.status, a.B = L.B, a.Hq = L.Hq, a.Hkv = L.Hkv, a.G = L.Hq / L.Hkv;
    a.starts = L.B > kSumRequests ? reinterpret_cast<int32_t*>(static_cast<uint8_t*>(L.workspace) + part_bytes(a.G, D, L.max_grid)) : nullptr;
    a.max_pages = L.max_pages, a.num_pages = L.num_pages, a.window = L.window, a.sink = L.window > 0 ? L.sink : 0;
    a.scale_log2 = L.scale * 1.4426950408889634f;
    a.lens_here = C::smem_bytes(L.B, a.G, true) <= kSmemLimit;
    // (the limit belongs to the kernel: the same in every call, whatever other threads call it with)
    cudaError_t e = cudaFuncSetAttribute(decode_kv4_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemLimit);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(L.grid);
    cfg.blockDim = dim3(C::kThreads);
    cfg.dynamicSmemBytes = C::smem_bytes(L.B, a.G, a.lens_here);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    ProfMark mark = prof_begin(stream, "decode_kv4");
    e = cudaLaunchKernelEx(&cfg, decode_kv4_kernel<D>, a);
    prof_end(stream, mark);
    if (e != cudaSuccess || (e = cudaGetLastError()) != cudaSuccess) return e;
    const int segments = L.B * L.Hkv;
    cfg.blockDim = dim3(kJoinThreads);
    cfg.dynamicSmemBytes = 0;
    mark = prof_begin(stream, "decode_kv4_join");
    if (a.starts) {
        const int per = std::min((segments + 8 * L.grid - 1) / (8 * L.grid), kJoinThreads);  // 8 blocks an SM, where that is enough
        cfg.gridDim = dim3((segments + per - 1) / per);
        e = cudaLaunchKernelEx(&cfg, decode_kv4_join_many_kernel<D>, a, L.grid, per);
    } else {
        cfg.gridDim = dim3(segments);
        e = cudaLaunchKernelEx(&cfg, decode_kv4_join_kernel<D>, a, L.grid);
    }
    prof_end(stream, mark);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

size_t decode_kv4_workspace_bytes(int B, int G, int D, int max_grid) {
    return part_bytes(G, D, max_grid) + (B > kSumRequests ? (size_t)(B + 1) * 4 : 0);
}

cudaError_t launch_decode_kv4(const DecodeKv4Launch& L, cudaStream_t stream) {
    if (L.D == 64) return launch_t<64>(L, stream);
    if (L.D == 128) return launch_t<128>(L, stream);
    if (L.D == 256) return launch_t<256>(L, stream);
    return cudaErrorInvalidValue;
}

}  // namespace attn
