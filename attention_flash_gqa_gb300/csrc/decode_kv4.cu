// Single-token decode over the 4-bit paged cache (kv4.cuh has the format), optionally over a sliding window with sinks.
//
// Definition: attn_decode_paged over the values that the cache stands for. Every visible byte of the cache is read once;
// at 18 D bytes a page and KV head against 64 D in bf16 the arithmetic is no longer free: see the count below.
//
//  * A unit is one page of one KV head: a record, contiguous. The units of a call lie in the order (request, head, page), and
//    every warp of the grid takes an equal stretch of them. It fetches them itself, one bulk copy a unit, through a ring of its
//    own, several units ahead: warps never wait for each other. 32 units' page ids and masks are worked out at a time,
//    one a lane, 32 units before they are needed.
//  * A unit is two chains of warp MMAs with the tokens, then the dims, as the 16 rows and the group's query heads as the 8
//    columns: S^T = K Q^T, O^T += V^T P^T. (With the heads as rows, as the bf16 decode has them, at least half of
//    each product would be rows of zeros.) Codes become bf16 operands in registers:
//      K: by masking alone. Bits 4 .. 7 of a bf16 pattern whose other bits are zero are the number code * 2^-129 (below the
//         smallest exponent and in the one after it the spacing is the same), bits 0 .. 3 are code * 2^-133. The missing powers
//         of two sit in q, whose rows are brought to 2^120 at the start of a segment, and in the factor of the scores. The
//         products of a group of 32 dims start from those of q with code 8, so that they are sums of q (code - 8),
//         and the group's scale is applied to the score in fp32;
//      V: low nibbles as 128 + code by mask and magic bits, from which 136 is taken before s is multiplied in, high nibbles
//         masked, times 2^127 and (code / 4) 4 s - 8 s in one fused multiply-add; every step exact. Masks and shifts share a pipe
//         that is half as wide as the instruction rate, multiplications have another one: so no shift but the one by 8.
//         P is rounded to bf16, as everywhere in this library; turned from columns to rows by movmatrix.
//    The softmax stays in registers (running maximum that moves only past 2^8, as in the bf16 decode).
//  * A stretch may hold several (request, head) segments and begin and end inside one. What a warp finishes alone it writes
//    out. The other pieces (o, m, l) meet in shared memory at the end of the block; those that begin or end
//    outside it go to the workspace, at most two a block, and a second kernel joins them.
#include <cuda_runtime.h>

#include "attn_internal.h"
#include "kv4.cuh"
#include "ptx.cuh"

namespace attn {
namespace {

constexpr int kPage = 16;
constexpr int kMaxB = 4096;
constexpr int kMaxG = 8;  // query heads of a KV head: the columns of an MMA

template <int D>
struct Cfg {
    static constexpr int kWarps = D == 256 ? 8 : D == 128 ? 16 : 16;
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int kStages = D == 64 ? 8 : D == 128 ? 4 : 3;  // units on their way in each warp's ring
    static constexpr int kRow = D + 4;                             // floats of a piece's row: o, m, l, padding
    static constexpr uint32_t kOffHead = kWarps * kStages * kv4_record_bytes(D);     // [warp][head][kRow]: first pieces
    static constexpr uint32_t kOffStart = kOffHead + kWarps * kMaxG * kRow * 4;      // [kMaxB + 1] pages before a request
    static constexpr uint32_t kOffBar = kOffStart + (kMaxB + 8) * 4;                 // [warp][stage]
    static constexpr uint32_t kOffMeta = kOffBar + kWarps * kStages * 8;             // abort flag, sums, segments of pieces
    static constexpr uint32_t kSmem = kOffMeta + 4 * (4 + 3 * kWarps) + 128;         // + slack for the alignment
    static_assert(kSmem <= 232448, "shared memory");
    // a warp's last piece is put where its own ring was
    static_assert(kMaxG * kRow * 4 <= kStages * kv4_record_bytes(D), "ring");
};

struct Args {
    const uint16_t* q;
    const uint8_t* cache;
    const int32_t *block_table, *seq_lens;
    uint16_t* o;
    float* lse;
    int32_t* start;  // [B + 1], for the second kernel
    float* part;     // [block][2][G][kRow]
    unsigned* status;
    int B, Hq, Hkv, G, max_pages, num_pages, window, sink;
    float scale_log2;
};

// d += a b on one warp: a 16 x 16 (row-major), b 16 x 8 (column-major), bf16 in, fp32 out.
// Fragments: g = lane / 4, c = lane % 4; a = {(g, 2c..2c+1), (g+8, 2c..), (g, 2c+8..2c+9), (g+8, 2c+8..)},
// b = {(2c..2c+1, g), (2c+8.., g)}, d = {(g, 2c), (g, 2c+1), (g+8, 2c), (g+8, 2c+1)}.
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// An 8 x 8 matrix of 16-bit values, lane (g, c) holding columns 2c, 2c+1 of row g, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
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
// Length of request b within its block-table row.
__device__ __forceinline__ int req_len(const Args& a, int b, bool record) {
    const int L = a.seq_lens[b];
    const long long cap = (long long)a.max_pages * kPage;
    if (L >= 0 && L <= cap) return L;
    if (record) atomicOr(a.status, DEVSTAT_BOUNDS);
    return L < 0 ? 0 : (int)cap;
}

constexpr uint32_t kLowNibbles = 0x000f000fu, kHighNibbles = 0x00f000f0u;
// two bf16 numbers each
constexpr uint32_t k4 = 0x40804080u, k128 = 0x43004300u, k2to127 = 0x7f007f00u, kMinus8 = 0xc100c100u, kMinus136 = 0xc308c308u;

// A unit as its warp needs it.
struct Unit {
    int page;      // -1: outside the pool (reported, its tokens are not seen)
    int segment;   // request * Hkv + head
    uint32_t see;  // bits 0 .. 15: visible tokens; 16: first of its segment; 17: last; 18 ..: KV head
};

// Folds a piece (o, m, l) into (O, M, L): both are weighed by the larger maximum.
template <int N>
__device__ __forceinline__ void fold(float (&O)[N], float& M, float& L, const float* o, float m, float l) {
    const float top = fmaxf(M, m);
    const float wa = M == -INFINITY ? 0.f : fast_exp2(M - top), wb = m == -INFINITY ? 0.f : fast_exp2(m - top);
#pragma unroll
    for (int e = 0; e < N; ++e) O[e] = O[e] * wa + o[e] * wb;
    L = L * wa + l * wb, M = top;
}

__device__ __forceinline__ float log_sum(float M, float L) { return L == 0.f ? -INFINITY : (M + __log2f(L)) * 0.69314718055994531f; }

template <int D>
__global__ void __launch_bounds__(Cfg<D>::kThreads, 1) decode_kv4_kernel(Args a) {
    using C = Cfg<D>;
    using F = Kv4<D>;
    constexpr int kGroups = F::kGroups, kBlocks = D / F::W, kTiles = F::W / 16;  // tiles of 16 dims in a block
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));
    float* head_piece = reinterpret_cast<float*>(smem + C::kOffHead);
    int32_t* start = reinterpret_cast<int32_t*>(smem + C::kOffStart);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMeta);
    int* warp_sum = reinterpret_cast<int*>(smem + C::kOffMeta) + 4;
    int* head_seg = warp_sum + C::kWarps;  // segment of a warp's first piece, -1: none
    int* tail_seg = head_seg + C::kWarps;  // of its last
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, c = lane & 3;
    uint8_t* ring = smem + warp * (C::kStages * F::kRecord);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kOffBar) + warp * C::kStages;
    if (tid == 0) *abort_flag = 0;
    if (lane == 0) {
        for (int s = 0; s < C::kStages; ++s) mbar_init(smem_u32(&full[s]), 1);
        head_seg[warp] = tail_seg[warp] = -1;
        fence_mbar_init();
    }
    griddep_wait();
    // the second kernel may be placed from here on; it waits for this one's end
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    // ---- pages before every request -------------------------------------------------------------
    {
        const int per = (a.B + C::kThreads - 1) / C::kThreads, b0 = tid * per;
        int mine = 0;
        for (int b = b0; b < min(a.B, b0 + per); ++b) mine += seen_pages(a, req_len(a, b, blockIdx.x == 0));
        int v = mine;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int n = __shfl_up_sync(0xffffffffu, v, off);
            if (lane >= off) v += n;
        }
        if (lane == 31) warp_sum[warp] = v;
        __syncthreads();
        int at = v - mine;
        for (int w = 0; w < warp; ++w) at += warp_sum[w];
        for (int b = b0; b < min(a.B, b0 + per); ++b) {
            start[b] = at;
            at += seen_pages(a, req_len(a, b, false));
        }
        if (b0 < a.B && b0 + per >= a.B) start[a.B] = at;
        __syncthreads();
        if (blockIdx.x == 0)
            for (int b = tid; b <= a.B; b += C::kThreads) a.start[b] = start[b];
    }
    // ---- this block's and this warp's stretch -----------------------------------------------------
    const int units = start[a.B] * a.Hkv;
    const int blocks = min((int)gridDim.x, units);  // every one that takes part has a unit
    if ((int)blockIdx.x >= blocks) return;
    const long long all = (long long)blocks * C::kWarps;
    const long long mine = (long long)blockIdx.x * C::kWarps + warp;
    const int u0 = (int)(mine * units / all), u1 = (int)((mine + 1) * units / all), n = u1 - u0;

    auto unit_at = [&](int u) -> Unit {
        Unit r = {-1, -1, 0u};
        if (u >= u1) return r;
        int lo = 0, hi = a.B - 1;  // the last request that starts at or before u: it has pages
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (start[mid] * a.Hkv <= u) lo = mid;
            else hi = mid - 1;
        }
        const int np = start[lo + 1] - start[lo], rem = u - start[lo] * a.Hkv;
        const int h = rem / np, i = rem - h * np;
        const int L = req_len(a, lo, false);
        const int first = first_token(a, L), early = sink_pages(a, L);
        const int p = i < early ? i : first / kPage + i - early;
        const int end = min(kPage, (i < early ? a.sink : L) - p * kPage);
        uint32_t see = (1u << end) - 1u;
        if (i == early) {  // the window's first page: tokens before the window are seen only if they are sinks
            const int keep = max(0, min(kPage, a.sink - p * kPage));
            see &= ~((1u << (first % kPage)) - 1u) | ((1u << (a.window > 0 ? keep : 0)) - 1u);
        }
        r.page = a.block_table[(size_t)lo * a.max_pages + p];
        if (r.page < 0 || r.page >= a.num_pages) {
            if (h == 0) atomicOr(a.status, DEVSTAT_BOUNDS);
            r.page = -1, see = 0u;
        }
        r.segment = lo * a.Hkv + h;
        r.see = see | (i == 0 ? 1u << 16 : 0u) | (i == np - 1 ? 1u << 17 : 0u) | ((uint32_t)h << 18);
        return r;
    };
    const uint64_t policy = l2_policy_evict_first();  // every byte is read once
    auto issue = [&](int i, int s, const Unit& of) {  // unit i into stage s; `of`: the batch of 32 that it is in
        if (lane == (i & 31)) {  // the lane that has it
            const uint32_t bar = smem_u32(&full[s]);
            if (of.page >= 0) {
                mbar_expect_tx(bar, F::kRecord);
                bulk_load_hint(smem_u32(ring + s * F::kRecord), a.cache + ((size_t)of.page * a.Hkv + (of.see >> 18)) * F::kRecord,
                               F::kRecord, bar, policy);
            } else {
                mbar_arrive(bar);
            }
        }
    };

    Unit cur = unit_at(u0 + lane), nxt = unit_at(u0 + 32 + lane);
    for (int i = 0; i < C::kStages && i < n; ++i) issue(i, i, cur);

    uint32_t qf[kGroups][4];  // lane (g, c): head g, dims 8c .. 8c+7 of a group, scaled
    float cq[kGroups][2];     // what a group's products start from, heads 2c and 2c+1
    float factor[2];          // of a product of heads 2c and 2c+1: softmax scale and the powers of two, in log2 units
    float o[kBlocks][kTiles][4] = {};  // tile t: dims 128 block + (W/8) g + 2 t, + 1 of heads 2c, 2c+1: {(d, h), (d, h+1), (d+1, h), (d+1, h+1)}
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};  // heads 2c, 2c+1 (l: this lane's share)
    float m_use[2] = {0.f, 0.f};                             // m, but 0 where nothing was seen yet
    int segment = 0;
    bool began = false;  // the segment began in this stretch
    bool ok = true;
    int stage = 0;
    uint32_t phase = 0;

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
    auto write_result = [&](int segment) {
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

    for (int i = 0; i < n; ++i) {
        if (i > 0 && (i & 31) == 0) cur = nxt, nxt = unit_at(u0 + i + 32 + lane);
        const uint32_t see = __shfl_sync(0xffffffffu, cur.see, i & 31);
        if (i == 0 || (see & (1u << 16))) {
            // ---- a new segment ----
            began = (see & (1u << 16)) != 0;
            segment = __shfl_sync(0xffffffffu, cur.segment, i & 31);
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
#pragma unroll
            for (int gr = 0; gr < kGroups; ++gr) {
#pragma unroll
                for (int x = 0; x < 4; ++x) qf[gr][x] = bf16x2_mul(qf[gr][x], x & 1 ? by : by16);
                float d[4] = {0.f, 0.f, 0.f, 0.f};
                constexpr uint32_t kLow = 0x80088008u, kHigh = 0x80808080u;  // -8 * 2^-133, -8 * 2^-129
                mma(d, kLow, kLow, kHigh, kHigh, qf[gr][0], qf[gr][1]);
                mma(d, kLow, kLow, kHigh, kHigh, qf[gr][2], qf[gr][3]);
                cq[gr][0] = d[0], cq[gr][1] = d[1];
            }
            const float fac = fminf(ldexpf(a.scale_log2, 129 - up), 3e38f);
            factor[0] = __shfl_sync(0xffffffffu, fac, 8 * c), factor[1] = __shfl_sync(0xffffffffu, fac, 8 * c + 4);
#pragma unroll
            for (int bl = 0; bl < kBlocks; ++bl)
#pragma unroll
                for (int t = 0; t < kTiles; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[bl][t][e] = 0.f;
            m[0] = m[1] = -INFINITY, m_use[0] = m_use[1] = l[0] = l[1] = 0.f;
        }
        if (ok) {
            ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&full[stage]), phase, abort_flag, a.status, 0x61));
            if (!ok && lane == 0) ring_drain(full, stage, (int)phase, C::kStages, n - i, a.status, 0x62);
            __syncwarp();
        }
        if (!ok) {  // given up: the rows of this unit and of those behind it in the stretch are NaN
            m[0] = m[1] = INFINITY, l[0] = l[1] = __int_as_float(0x7fc00000);
        } else if (see & 0xffffu) {
            const uint32_t rec = smem_u32(ring + stage * F::kRecord);
            // ---- S^T: tokens g and g + 8, heads 2c and 2c + 1 ----
            float s[4] = {0.f, 0.f, 0.f, 0.f};
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
                    float d[4] = {cq[gr][0], cq[gr][1], cq[gr][0], cq[gr][1]};
                    const uint32_t w0 = kw[0][x], w1 = kw[1][x], u0 = w0 >> 8, u1 = w1 >> 8;
                    mma(d, w0 & kLowNibbles, w1 & kLowNibbles, w0 & kHighNibbles, w1 & kHighNibbles, qf[gr][0], qf[gr][1]);
                    mma(d, u0 & kLowNibbles, u1 & kLowNibbles, u0 & kHighNibbles, u1 & kHighNibbles, qf[gr][2], qf[gr][3]);
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
            const bool over = fmaxf(s[0], s[2]) > m[0] + 8.f || fmaxf(s[1], s[3]) > m[1] + 8.f;
            if (__any_sync(0xffffffffu, over)) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float mx = fmaxf(s[e], s[e + 2]);
#pragma unroll
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
                const uint32_t s0 = lds32(rec + F::value_scale(gr, 2 * c)) & hide0, s1 = lds32(rec + F::value_scale(gr, 2 * c + 8)) & hide1;
                const uint32_t f0 = bf16x2_mul(s0, k4), f1 = bf16x2_mul(s1, k4), c0 = bf16x2_mul(s0, kMinus8), c1 = bf16x2_mul(s1, kMinus8);
                auto low = [](uint32_t x, uint32_t s) { return bf16x2_mul(bf16x2_add((x & kLowNibbles) | k128, kMinus136), s); };
                auto high = [](uint32_t x, uint32_t f, uint32_t c) { return bf16x2_fma(bf16x2_mul(x & kHighNibbles, k2to127), f, c); };
#pragma unroll
                for (int half = 0; half < 2 * kWords; ++half) {  // 4 dims of both tokens side by side
                    const uint32_t sel = half & 1 ? 0x7632u : 0x5410u;
                    const uint32_t x0 = __byte_perm(vw[0][0][half / 2], vw[0][1][half / 2], sel);
                    const uint32_t x1 = __byte_perm(vw[1][0][half / 2], vw[1][1][half / 2], sel);
#pragma unroll
                    for (int d = 0; d < 4; d += 2) {
                        const uint32_t y0 = x0 >> (4 * d), y1 = x1 >> (4 * d);
                        mma(o[bl][half * 2 + d / 2], low(y0, s0), high(y0, f0, c0), low(y1, s1), high(y1, f1, c1), b0, b1);
                    }
                }
            }
        }
        __syncwarp();  // the record has been read
        if (ok && i + C::kStages < n) {
            const int j = i + C::kStages;
            if ((j ^ i) < 32) issue(j, stage, cur);
            else issue(j, stage, nxt);
        }
        if (++stage == C::kStages) stage = 0, phase ^= 1u;
        const bool ends = (see & (1u << 17)) != 0, last = i + 1 == n;
        if (ends || last) {
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) l[e] += __shfl_xor_sync(0xffffffffu, l[e], off);
            if (began && ends) {
                write_result(segment);
            } else if (!last) {  // it began in an earlier stretch
                write_piece(head_piece + warp * kMaxG * C::kRow);
                if (lane == 0) head_seg[warp] = segment;
            } else {
                write_piece(reinterpret_cast<float*>(ring));
                if (lane == 0) tail_seg[warp] = segment;
            }
        }
    }
    __syncthreads();
    // ---- pieces of a segment that lie in this block: joined by the warp that has the first ------------
    const int first_unit = (int)((long long)blockIdx.x * units / blocks), end_unit = (int)((long long)(blockIdx.x + 1) * units / blocks);
    auto finish = [&](int w, bool head) {  // from warp w's piece on, in the order of the warps
        const int segment = head ? head_seg[w] : tail_seg[w];
        int more = 0;  // pieces behind the first: last pieces of warps that the segment fills, then a first piece
        const int b = segment / a.Hkv, h = segment - b * a.Hkv, np = start[b + 1] - start[b];
        const int s0 = start[b] * a.Hkv + h * np, s1 = s0 + np;
        if (!head) more = C::kWarps - 1 - w;
        const bool whole = s0 >= first_unit && s1 <= end_unit;
        float* slot = a.part + ((size_t)blockIdx.x * 2 + (s0 < first_unit ? 0 : 1)) * a.G * C::kRow;
        constexpr int N = D / 32;
        for (int hh = 0; hh < a.G; ++hh) {
            float O[N] = {}, M = -INFINITY, L = 0.f;
            auto take = [&](const float* rows) {
                const float* row = rows + hh * C::kRow;
                float x[N];
#pragma unroll
                for (int e = 0; e < N; e += 2) *reinterpret_cast<float2*>(x + e) = *reinterpret_cast<const float2*>(row + N * lane + e);
                fold<N>(O, M, L, x, row[D], row[D + 1]);
            };
            take(head ? head_piece + w * kMaxG * C::kRow : reinterpret_cast<const float*>(smem + w * (C::kStages * F::kRecord)));
            for (int x = w + 1; x <= w + more; ++x) {
                if (head_seg[x] == segment) {
                    take(head_piece + x * kMaxG * C::kRow);
                    break;
                }
                if (tail_seg[x] == segment) take(reinterpret_cast<const float*>(smem + x * (C::kStages * F::kRecord)));
            }
            const size_t at = (size_t)segment * a.G + hh;
            if (whole) {
                const float inv = L == 0.f ? 0.f : 1.f / L;
#pragma unroll
                for (int e = 0; e < N; e += 2) *reinterpret_cast<uint32_t*>(a.o + at * D + N * lane + e) = pack_bf16x2(O[e] * inv, O[e + 1] * inv);
                if (lane == 0) a.lse[at] = log_sum(M, L);
            } else {
                float* row = slot + hh * C::kRow;
#pragma unroll
                for (int e = 0; e < N; e += 2) *reinterpret_cast<float2*>(row + N * lane + e) = make_float2(O[e], O[e + 1]);
                if (lane == 0) row[D] = L == L ? M : INFINITY, row[D + 1] = L;
            }
        }
    };
    if (head_seg[warp] >= 0) {
        // a first piece stands alone if no earlier warp of the block has one of its segment
        bool alone = true;
        for (int w = 0; w < warp; ++w) alone &= tail_seg[w] != head_seg[warp];
        if (alone) finish(warp, true);
    }
    if (tail_seg[warp] >= 0) {
        bool opens = true;
        for (int w = 0; w < warp; ++w) opens &= tail_seg[w] != tail_seg[warp];
        if (opens) finish(warp, false);
    }
}

struct JoinArgs {
    const float* part;
    const int32_t* start;
    uint16_t* o;
    float* lse;
    int B, Hkv, G, grid;
};

// Joins the pieces of the segments that several blocks of the decode kernel shared, a block for each segment; the others are done,
// but for the rows of requests without a key, which come out as o = 0, lse = -inf. A thread has 4 dims of a head and folds up to 8 pieces
// with all their loads on the way at once.
template <int D>
__global__ void __launch_bounds__(128) decode_kv4_join_kernel(JoinArgs a) {
    using C = Cfg<D>;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    griddep_wait();
    const int segment = blockIdx.x, b = segment / a.Hkv, h = segment - b * a.Hkv;
    const int first = a.start[b], np = a.start[b + 1] - first, units = a.start[a.B] * a.Hkv;
    const int items = a.G * (D / 4);
    const size_t row0 = (size_t)segment * a.G;
    if (np == 0) {
        for (int it = threadIdx.x; it < items; it += 128) {
            *reinterpret_cast<uint2*>(a.o + row0 * D + 4 * it) = make_uint2(0, 0);
            if (it % (D / 4) == 0) a.lse[row0 + it / (D / 4)] = -INFINITY;
        }
        return;
    }
    const int s0 = first * a.Hkv + h * np, s1 = s0 + np;
    const long long blocks = min(a.grid, units);
    // the block that unit u belongs to: block k has units floor(k units / blocks) ..
    const int kf = (int)(((s0 + 1) * blocks - 1) / units), kl = (int)((s1 * blocks - 1) / units);
    if (kf == kl) return;
    for (int it = threadIdx.x; it < items; it += 128) {
        const int hh = it / (D / 4), d = 4 * (it % (D / 4));
        float O[4] = {}, M = -INFINITY, L = 0.f;
        for (int k0 = kf; k0 <= kl; k0 += 8) {
            float4 x[8];
            float2 ml[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                x[j] = make_float4(0.f, 0.f, 0.f, 0.f), ml[j] = make_float2(-INFINITY, 0.f);
                const int k = k0 + j;
                if (k <= kl) {
                    // a block's first slot holds what began before it
                    const int which = s0 < (int)(k * (long long)units / blocks) ? 0 : 1;
                    const float* row = a.part + (((size_t)k * 2 + which) * a.G + hh) * C::kRow;
                    x[j] = __ldcg(reinterpret_cast<const float4*>(row + d));
                    ml[j] = __ldcg(reinterpret_cast<const float2*>(row + D));
                }
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float y[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
                fold<4>(O, M, L, y, ml[j].x, ml[j].y);
            }
        }
        const float inv = L == 0.f ? 0.f : 1.f / L;
        *reinterpret_cast<uint2*>(a.o + (row0 + hh) * D + d) = make_uint2(pack_bf16x2(O[0] * inv, O[1] * inv), pack_bf16x2(O[2] * inv, O[3] * inv));
        if (d == 0) a.lse[row0 + hh] = log_sum(M, L);
    }
}

size_t start_bytes(int B) { return ((size_t)(B + 1) * 4 + 255) & ~size_t(255); }

template <int D>
cudaError_t launch_t(const DecodeKv4Launch& L, cudaStream_t stream) {
    using C = Cfg<D>;
    Args a;
    a.q = L.q, a.cache = L.cache, a.block_table = L.block_table, a.seq_lens = L.seq_lens, a.o = L.o, a.lse = L.lse;
    a.start = static_cast<int32_t*>(L.workspace);
    a.part = reinterpret_cast<float*>(static_cast<uint8_t*>(L.workspace) + start_bytes(L.B));
    a.status = L.status, a.B = L.B, a.Hq = L.Hq, a.Hkv = L.Hkv, a.G = L.Hq / L.Hkv;
    a.max_pages = L.max_pages, a.num_pages = L.num_pages, a.window = L.window, a.sink = L.window > 0 ? L.sink : 0;
    a.scale_log2 = L.scale * 1.4426950408889634f;
    cudaError_t e = cudaFuncSetAttribute(decode_kv4_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(L.grid);
    cfg.blockDim = dim3(C::kThreads);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    ProfMark mark = prof_begin(stream, "decode_kv4");
    e = cudaLaunchKernelEx(&cfg, decode_kv4_kernel<D>, a);
    prof_end(stream, mark);
    if (e != cudaSuccess || (e = cudaGetLastError()) != cudaSuccess) return e;
    JoinArgs ja;
    ja.part = a.part, ja.start = a.start, ja.o = L.o, ja.lse = L.lse, ja.B = L.B, ja.Hkv = L.Hkv, ja.G = a.G, ja.grid = L.grid;
    cfg.gridDim = dim3(L.B * L.Hkv);
    cfg.blockDim = dim3(128);
    cfg.dynamicSmemBytes = 0;
    mark = prof_begin(stream, "decode_kv4_join");
    e = cudaLaunchKernelEx(&cfg, decode_kv4_join_kernel<D>, ja);
    prof_end(stream, mark);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

size_t decode_kv4_workspace_bytes(int B, int G, int D, int grid) { return start_bytes(B) + (size_t)grid * 2 * G * (D + 4) * 4; }

cudaError_t launch_decode_kv4(const DecodeKv4Launch& L, cudaStream_t stream) {
    if (L.D == 64) return launch_t<64>(L, stream);
    if (L.D == 128) return launch_t<128>(L, stream);
    if (L.D == 256) return launch_t<256>(L, stream);
    return cudaErrorInvalidValue;
}

}  // namespace attn
