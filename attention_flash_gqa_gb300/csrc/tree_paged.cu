// Attention of drafted token trees over a paged cache: the verification step of speculative decoding.
//
// Row i of a request with n drafted tokens behind c = L - n cached ones sees the context keys
// j < c (with a window only those with p_i - j < W, p_i = max(position, c)) and the drafted tokens
// d whose bit is set in its mask row:
//     s_ij = scale q_i . k_j,   o_i = sum_j softmax_j(s_ij | visible) v_j,   lse_i = ln sum_j exp(s_ij)
// A row that sees nothing gets o = 0 and lse = -inf.
//
// Few rows over many keys: K and V must be read once for all rows that share them, and one request's
// keys spread over the whole GPU.
//  * A row tile packs the drafted tokens and the G query heads of one KV head into the 128 rows of
//    an MMA (row = token * G + head, 128 / G tokens a tile), so a KV head's keys serve all of them.
//  * A unit of work is one page (16 keys) of one segment = (request, KV head, 256-column half of O at
//    D = 512, row tile). All units are laid end to end and CTA k takes the k-th equal share: it may
//    finish one segment, run through some and start another. A segment that one CTA covers is
//    written out by it; of a shared one every CTA leaves (O, m, l) unnormalised in the workspace and
//    tree_merge_kernel combines them (launched with programmatic serialisation behind this grid).
//  * Inside a CTA the pages are taken in tiles of up to eight (128 keys) through the pipeline of the
//    prefill forward, and the pipeline runs on across segments. Tensor memory: O (fp32, up to 256
//    columns) and 3 (D <= 128) or 2 score buffers of 128 columns, P (bf16) over the scores. Only
//    the pages of a tile that exist are loaded and multiplied (N of Q K^T and K of P V follow them,
//    a page being one K step of 16), so only the last page's slots past L need care: the issuer's
//    warp zeroes those V rows before their P V (P is 0 there, but 0 * NaN is not).
//
// Warp roles (320 threads): 0 TMA producer (lanes 0-7: a page each), 1 MMA issuer, 2-9 softmax
// (warps w and w + 4 share TMEM lane quarter w & 3, each on 64 of a tile's 128 keys). Quarters
// without rows only keep the barriers going.
#include <cuda_runtime.h>

#include "attn_internal.h"
#include "ptx.cuh"

namespace attn {
namespace {

constexpr int kPage = 16;
constexpr int kTilePages = 8;
constexpr int kThreads = 320;
constexpr int kWarps = kThreads / 32;
constexpr int kSoftmaxWarps = 8;
constexpr uint32_t kSubBytes = 16384;  // 128 rows x 64 bf16
constexpr float kRescaleLog2 = 8.0f;
constexpr int kMinPages = 8;   // a CTA's share at least: one tile
constexpr int kMaxGrid = 192;  // sizes the workspace

template <int D>
struct TreeCfg {
    static constexpr int kDV = D < 256 ? D : 256;      // O columns per segment
    static constexpr int kSplit = D / kDV;
    static constexpr int kSBuf = kDV <= 128 ? 3 : 2;   // score buffers in tensor memory
    static constexpr int kSubs = D >= 128 ? 2 : 1;     // 64-column sub-tiles per slot
    static constexpr int kSlotCols = 64 * kSubs;
    static constexpr uint32_t kSlotBytes = kSubs * kSubBytes;
    static constexpr int kKC = D / kSlotCols;          // slots per K tile
    static constexpr int kVC = kDV / kSlotCols;        // slots per V tile
    static constexpr int kQBufs = D == 64 ? 2 : 1;
    static constexpr int kStages = D == 512 ? 3 : D == 256 ? 5 : D == 128 ? 6 : 12;
    static constexpr uint32_t kQBytes = D * 256;       // 128 rows
    static constexpr uint32_t kPageBytes = 2048 * kSubs;     // one page's rows in a slot
    static constexpr uint32_t kGroupStride = 1024 * kSubs;   // 8 rows of both sub-tiles
    static constexpr uint32_t kOffSlots = kQBufs * kQBytes;
    static constexpr uint32_t kOffXch = kOffSlots + kStages * kSlotBytes;  // [2][128] fp32
    static constexpr uint32_t kOffBar = kOffXch + 1024;
    static constexpr uint32_t kOffScan = kOffBar + 512;
    static constexpr uint32_t kSmem = kOffScan + 256 + 1024;
    static constexpr int kRowF = kDV + 4;              // partial row: O, m, l, 2 pad
    static_assert(kSmem <= 232448, "shared memory");
    static_assert(kQBufs == 1 || kQBufs == 2, "Q buffers");
};

// What the merge of a segment needs; one per CTA, for the segment that starts in it and ends elsewhere.
struct TreeSpan {
    int ctas;   // CTAs that share the segment (0: none)
    int row0;   // first token row of the tile
    int rows;   // rows of the tile (tokens * G)
    int head0;  // first query head
    int col0;   // first O column
    int pad[3];
};

struct TreeArgs {
    const int32_t *block_table, *seq_lens, *cu_q, *mask, *positions;
    uint16_t* o;
    float* lse;
    unsigned* status;
    float* part;      // [2 * grid][rows_cap][kRowF]
    TreeSpan* span;   // [grid]
    int R, T, max_q, words, Hq, Hkv, G, tokens_tile, rows_cap, max_pages, num_pages, window;
    float scale_log2;
};

// A request as the walk sees it; no units if it is empty or inconsistent.
struct Req {
    int start, n, L, pg0, npg, tiles;
    bool bad;
};
__device__ __forceinline__ Req load_req(const TreeArgs& a, int b) {
    Req r;
    r.start = a.cu_q[b];
    r.n = a.cu_q[b + 1] - r.start;
    r.L = a.seq_lens[b];
    r.bad = r.start < 0 || r.n < 0 || r.n > a.max_q || r.start > a.T - r.n || r.n > r.L ||
            (long long)r.L > (long long)a.max_pages * kPage;
    if (r.bad || r.n == 0) {
        r.n = r.npg = r.pg0 = r.tiles = 0;
        return r;
    }
    const int c = r.L - r.n;
    r.pg0 = a.window > 0 && c >= a.window ? (c - a.window + 1) / kPage : 0;  // no row sees an earlier key
    r.npg = (r.L + kPage - 1) / kPage - r.pg0;
    r.tiles = (r.n + a.tokens_tile - 1) / a.tokens_tile;
    return r;
}
template <int D>
__device__ __forceinline__ long long req_units(const TreeArgs& a, const Req& r) {
    return (long long)r.npg * r.tiles * a.Hkv * TreeCfg<D>::kSplit;
}

// Walks the tiles of a CTA's share.
template <int D>
struct Walk {
    Req r;
    int b, seg, pg, np;  // request, segment in it, first page (from pg0) and pages of the tile
    long long left;      // pages of the share from here on
    bool begins;         // first tile of a piece (a segment's pages in this CTA)

    __device__ __forceinline__ void start(const TreeArgs& a, int b_, long long off, long long units) {
        b = b_;
        r = load_req(a, b);
        seg = (int)(off / r.npg);
        pg = (int)(off - (long long)seg * r.npg);
        left = units;
        begins = true;
        size();
    }
    __device__ __forceinline__ void size() {
        np = min(kTilePages, r.npg - pg);
        if (left < np) np = (int)left;
    }
    __device__ __forceinline__ bool more() const { return left > 0; }
    __device__ __forceinline__ bool ends() const { return pg + np == r.npg || left == np; }
    __device__ __forceinline__ void next(const TreeArgs& a) {
        pg += np, left -= np;
        begins = false;
        if (left <= 0) return;
        if (pg == r.npg) {
            pg = 0, begins = true;
            if (++seg == r.tiles * a.Hkv * TreeCfg<D>::kSplit) {
                seg = 0;
                do r = load_req(a, ++b);  // the share holds more units: there is another request
                while (r.npg == 0);
            }
        }
        size();
    }
    __device__ __forceinline__ int tile() const { return seg % r.tiles; }
    __device__ __forceinline__ int split() const { return seg / r.tiles % TreeCfg<D>::kSplit; }
    __device__ __forceinline__ int head() const { return seg / (r.tiles * TreeCfg<D>::kSplit); }
    // the tile holds the request's last page, and slots of it lie past L
    __device__ __forceinline__ bool tail() const { return pg + np == r.npg && r.L % kPage != 0; }
};

__device__ __forceinline__ uint64_t low_bits(int n) { return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1; }

// CTA that owns unit u when P units are split evenly over G CTAs.
__device__ __forceinline__ int owner_of(long long u, long long P, int G) {
    return (int)(((u + 1) * (long long)G - 1) / P);
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    tree_paged_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                      const __grid_constant__ CUtensorMap tv, TreeArgs a) {
    using C = TreeCfg<D>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    const uint32_t sQ = sbase, sSlots = sbase + C::kOffSlots;
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
    uint64_t* full = bars;                   // [kStages]
    uint64_t* empty = full + C::kStages;     // [kStages]
    uint64_t* q_full = empty + C::kStages;   // [2]
    uint64_t* q_free = q_full + 2;           // [2]
    // per score buffer (step j uses j % kSBuf): at most one pending phase each, as in the prefill forward
    uint64_t* s_full = q_free + 2;           // [3]
    uint64_t* p_full = s_full + 3;           // [3]
    uint64_t* pv_done = p_full + 3;          // [3]
    uint64_t* o_free = pv_done + 3;          // the epilogue has read O
    uint64_t* mma_idle = o_free + 1;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_idle + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    long long* scan = reinterpret_cast<long long*>(smem + C::kOffScan);  // [kWarps], then the share's start
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int k = blockIdx.x;

    if (tid == 0) {
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(smem_u32(&full[s]), 1);
            mbar_init(smem_u32(&empty[s]), 1);
        }
        for (int i = 0; i < 2; ++i) mbar_init(smem_u32(&q_full[i]), 1), mbar_init(smem_u32(&q_free[i]), 1);
        for (int i = 0; i < 3; ++i) {
            mbar_init(smem_u32(&s_full[i]), 1);
            mbar_init(smem_u32(&p_full[i]), kSoftmaxWarps);
            mbar_init(smem_u32(&pv_done[i]), 1);
        }
        mbar_init(smem_u32(o_free), kSoftmaxWarps);
        mbar_init(smem_u32(mma_idle), 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(tmem_slot), 512);
        tmem_relinquish();
    }
    // Launched with programmatic serialisation: nothing is read before the kernel in front has
    // finished. The merge kernel may be scheduled from here on (it waits for this grid).
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    // ---- the CTA's share: units before each thread's run of requests ---------------------------
    const int per = (a.R + kThreads - 1) / kThreads;
    const int b0 = min(tid * per, a.R), b1 = min(b0 + per, a.R);
    long long sum = 0;
    for (int b = b0; b < b1; ++b) {
        const Req r = load_req(a, b);
        if (r.bad && k == 0) atomicOr(a.status, DEVSTAT_BOUNDS);
        sum += req_units<D>(a, r);
    }
    long long x = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
    }
    if (lane == 31) scan[warp] = x;
    __syncthreads();
    long long P = 0;
    x -= sum;
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) x += scan[w];
        P += scan[w];
    }
    const long long want = (P + kMinPages - 1) / kMinPages;
    const int Gc = (int)(want < (long long)gridDim.x ? want : (long long)gridDim.x);
    const bool works = k < Gc;  // uniform
    const long long u0 = works ? (long long)k * P / Gc : 0, u1 = works ? (long long)(k + 1) * P / Gc : 0;
    if (works && x <= u0 && u0 < x + sum) {
        for (int b = b0; b < b1; ++b) {
            const long long n = req_units<D>(a, load_req(a, b));
            if (u0 < x + n) {
                scan[kWarps] = b, scan[kWarps + 1] = u0 - x;
                break;
            }
            x += n;
        }
    }
    if (tid == 0) a.span[k].ctas = 0;  // until the share's last piece says otherwise
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = *tmem_slot;
    const uint32_t tO = tbase, tS0 = tbase + 512 - C::kSBuf * 128;
    const int first_b = (int)scan[kWarps];
    const long long first_off = scan[kWarps + 1];

    if (!works) {
        // no units left for this CTA
    } else if (warp == 0) {
        // ------------------------------- TMA producer ----------------------------------------
        if (lane == 0) prefetch_tmap(&tq), prefetch_tmap(&tk), prefetch_tmap(&tv);
        int slot = 0, round = 0;
        bool ok = true;
        auto page_id = [&](const Walk<D>& w) -> int {  // lane i: id of the tile's page i
            if (lane >= w.np) return 0;
            int id = a.block_table[(size_t)w.b * a.max_pages + w.r.pg0 + w.pg + lane];
            if (id < 0 || id >= a.num_pages) {
                atomicOr(a.status, DEVSTAT_BOUNDS);
                id = 0;
            }
            return id;
        };
        // one slot: np pages, lane i loads page i's 16 rows x kSlotCols columns
        auto load_slot = [&](const CUtensorMap* map, int chunk, int np, int id) -> bool {
            if (round > 0 && !__all_sync(0xffffffffu, mbar_wait(smem_u32(&empty[slot]), (round - 1) & 1, abort_flag, a.status, 0x41)))
                return false;
            const uint32_t fb = smem_u32(&full[slot]);
            if (lane == 0) mbar_expect_tx(fb, np * C::kPageBytes);
            __syncwarp();
            if (lane < np) tma_load_5d(sSlots + slot * C::kSlotBytes + lane * C::kPageBytes, map, fb, 0, 0, chunk, 0, id);
            if (++slot == C::kStages) slot = 0, ++round;
            return true;
        };
        Walk<D> wk, wv;
        wk.start(a, first_b, first_off, u1 - u0);
        wv = wk;
        int idk = page_id(wk), idv = idk, pieces = 0;
        auto load_k = [&]() -> bool {
            if (wk.begins) {
                const int qb = pieces % C::kQBufs;
                if (pieces >= C::kQBufs &&
                    !__all_sync(0xffffffffu, mbar_wait(smem_u32(&q_free[qb]), (pieces / C::kQBufs - 1) & 1, abort_flag, a.status, 0x42)))
                    return false;
                if (lane == 0) {
                    const uint32_t fb = smem_u32(&q_full[qb]);
                    mbar_expect_tx(fb, (uint32_t)(D / 64) * a.G * a.tokens_tile * 128);
                    for (int c = 0; c < D / 64; ++c)
                        tma_load_4d(sQ + qb * C::kQBytes + c * kSubBytes, &tq, fb, c * 64, wk.head() * a.G,
                                    wk.r.start + wk.tile() * a.tokens_tile, 0);
                }
                __syncwarp();
                ++pieces;
            }
            for (int c = 0; c < C::kKC; ++c)
                if (!load_slot(&tk, wk.head() * (D / 64) + c * C::kSubs, wk.np, idk)) return false;
            wk.next(a);
            if (wk.more()) idk = page_id(wk);
            return true;
        };
        auto load_v = [&]() -> bool {
            for (int c = 0; c < C::kVC; ++c)
                if (!load_slot(&tv, wv.head() * (D / 64) + wv.split() * (C::kDV / 64) + c * C::kSubs, wv.np, idv)) return false;
            wv.next(a);
            if (wv.more()) idv = page_id(wv);
            return true;
        };
        // the issuer's order: K(0) .. K(kSBuf - 1), then V(j), K(j + kSBuf)
        for (int i = 0; ok && i < C::kSBuf && wk.more(); ++i) ok = load_k();
        while (ok && wv.more()) {
            ok = load_v();
            if (ok && wk.more()) ok = load_k();
        }
        // every issued copy has landed before the CTA may leave
        if (lane == 0) {
            const int issued = round * C::kStages + slot;
            for (int s = 0; s < C::kStages && s < issued; ++s) {
                const int last = s + ((issued - 1 - s) / C::kStages) * C::kStages;
                mbar_drain(smem_u32(&full[s]), (last / C::kStages) & 1, a.status, 0x43);
            }
            for (int i = 0; i < C::kQBufs && i < pieces; ++i) {
                const int last = i + ((pieces - 1 - i) / C::kQBufs) * C::kQBufs;
                mbar_drain(smem_u32(&q_full[i]), (last / C::kQBufs) & 1, a.status, 0x44);
            }
        }
    } else if (warp == 1) {
        // ------------------------------- MMA issuer -------------------------------------------
        // lane 0 issues; the other lanes follow it to zero V rows
        constexpr uint32_t idO = idesc_bf16_f32(128, C::kSlotCols, false, true);  // V is N-major
        int slot = 0, round = 0, pieces_s = 0, pieces_o = 0, js = 0, jp = 0;
        bool ok = true;
        auto wait = [&](uint64_t* bar, int phase, unsigned site) -> bool {
            if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(bar), phase & 1, abort_flag, a.status, site))) return false;
            tc_fence_after();
            return true;
        };
        auto release_slot = [&]() {
            if (elect_one()) umma_commit(smem_u32(&empty[slot]));
            if (++slot == C::kStages) slot = 0, ++round;
        };
        Walk<D> ws, wp;
        ws.start(a, first_b, first_off, u1 - u0);
        wp = ws;
        auto issue_s = [&]() -> bool {
            if (ws.begins) {
                if (!wait(&q_full[pieces_s % C::kQBufs], pieces_s / C::kQBufs, 0x45)) return false;
                ++pieces_s;
            }
            const int qb = (pieces_s - 1) % C::kQBufs;
            const uint32_t dst = tS0 + (js % C::kSBuf) * 128;
            const uint32_t idS = idesc_bf16_f32(128, ws.np * kPage, false, false);
            const uint64_t dq0 = sdesc_sw128(sQ + qb * C::kQBytes, 16, 1024);
            for (int c = 0; c < C::kKC; ++c) {
                if (!wait(&full[slot], round, 0x46)) return false;
                const uint64_t dk = sdesc_sw128(sSlots + slot * C::kSlotBytes, 16, C::kGroupStride);
                const uint64_t dq = sdesc_at(dq0, C::kSubs * c * kSubBytes);
                if (elect_one()) {
#pragma unroll
                    for (int sub = 0; sub < C::kSubs; ++sub)
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            umma_bf16_ss(dst, sdesc_at(dq, sub * kSubBytes + kk * 32), sdesc_at(dk, sub * 1024 + kk * 32), idS,
                                         (c | sub | kk) ? 1u : 0u);
                }
                release_slot();
            }
            if (elect_one()) {
                umma_commit(smem_u32(&s_full[js % C::kSBuf]));
                if (ws.ends()) umma_commit(smem_u32(&q_free[qb]));
            }
            ++js;
            ws.next(a);
            return true;
        };
        auto issue_pv = [&]() -> bool {
            const int buf = jp % C::kSBuf;
            if (!wait(&p_full[buf], jp / C::kSBuf, 0x47)) return false;
            if (wp.begins) {
                // the piece before has been read out of O
                if (pieces_o > 0 && !wait(o_free, pieces_o - 1, 0x48)) return false;
                ++pieces_o;
            }
            const uint32_t tP = tS0 + buf * 128;
            for (int c = 0; c < C::kVC; ++c) {
                if (!wait(&full[slot], round, 0x49)) return false;
                const uint32_t vslot = sSlots + slot * C::kSlotBytes;
                if (wp.tail()) {  // zero the last page's rows past L
                    const int r0 = wp.r.L % kPage;
                    const uint32_t base = vslot + (wp.np - 1) * C::kPageBytes;
                    for (int e = lane; e < (kPage - r0) * 8 * C::kSubs; e += 32) {  // 16-byte pieces
                        const int row = r0 + e / (8 * C::kSubs), sub = (e >> 3) % C::kSubs;
                        st_shared_v4(base + (row >> 3) * C::kGroupStride + sub * 1024 + (row & 7) * 128 + (e & 7) * 16, 0u, 0u, 0u, 0u);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                }
                if (elect_one()) {
                    const uint64_t dv = sdesc_sw128(vslot, 1024, C::kGroupStride);
                    for (int kk = 0; kk < wp.np; ++kk)  // a page of 16 keys per step
                        umma_bf16_ts(tO + c * C::kSlotCols, tP + (kk >> 2) * 64 + (kk & 3) * 8, sdesc_at(dv, kk * C::kPageBytes), idO,
                                     (!wp.begins || kk > 0) ? 1u : 0u);
                }
                release_slot();
            }
            if (elect_one()) umma_commit(smem_u32(&pv_done[buf]));
            ++jp;
            wp.next(a);
            return true;
        };
        for (int i = 0; ok && i < C::kSBuf && ws.more(); ++i) ok = issue_s();
        while (ok && wp.more()) {
            ok = issue_pv();
            // S(j + kSBuf) over the buffer that P(j) came from: the pipe runs in order
            if (ok && ws.more()) ok = issue_s();
        }
        if (elect_one()) {
            umma_commit(smem_u32(mma_idle));
            mbar_drain(smem_u32(mma_idle), 0, a.status, 0x4a);
        }
        __syncwarp();
    } else {
        // --------------------------------- softmax ----------------------------------------------
        const int quad = warp & 3, hf = (warp - 2) >> 2;
        const int row = quad * 32 + lane;  // row of the tile = TMEM lane
        const uint32_t lane_base = (uint32_t)(quad * 32) << 16;
        const uint32_t pair_bar = 1 + quad;
        float* xch = reinterpret_cast<float*>(smem + C::kOffXch);
        float m_ref = -INFINITY, l = 0.f;
        int first_key = 0, token = 0, pg_begin = 0, tok0 = 0, rows = 0, ctx = 0;
        bool busy = false;
        bool ok = true;
        Walk<D> w;
        w.start(a, first_b, first_off, u1 - u0);
        for (int j = 0; ok && w.more(); ++j, w.next(a)) {
            const int buf = j % C::kSBuf;
            if (w.begins) {
                ctx = w.r.L - w.r.n;
                tok0 = w.tile() * a.tokens_tile;  // of the request
                rows = min(a.tokens_tile, w.r.n - tok0) * a.G;
                busy = quad * 32 < rows;          // the quarter has rows (uniform over the pair)
                m_ref = -INFINITY, l = 0.f;
                pg_begin = w.pg;
                token = w.r.start + min(tok0 + row / a.G, w.r.n - 1);
                first_key = a.window > 0 ? max(0, min(ctx, max(a.positions[token], ctx) - a.window + 1)) : 0;
            }
            ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&s_full[buf]), (j / C::kSBuf) & 1, abort_flag, a.status, 0x4c));
            if (busy) {
                float s[64];
                float mx = -INFINITY;
                if (ok) {
                    tc_fence_after();
                    {
                        uint32_t raw[2][32];
#pragma unroll
                        for (int c = 0; c < 2; ++c) tmem_ld32(tS0 + buf * 128 + 64 * hf + c * 32 + lane_base, raw[c]);
                        tmem_ld_wait();
#pragma unroll
                        for (int c = 0; c < 2; ++c)
#pragma unroll
                            for (int e = 0; e < 32; ++e) s[c * 32 + e] = __uint_as_float(raw[c][e]);
                    }
                    const int key0 = (w.r.pg0 + w.pg) * kPage + 64 * hf;
                    const int cols = w.np * kPage - 64 * hf;  // loaded keys of this half
                    if (__any_sync(0xffffffffu, key0 + 63 >= ctx || cols < 64 || key0 < first_key)) {
                        uint64_t vis = low_bits(cols) & ~low_bits(first_key - key0);
                        const int dc = ctx - key0;  // column of the first drafted token
                        if (dc < 64) {
                            const int d0 = max(0, -dc), wi = d0 >> 5, sh = d0 & 31;
                            const int32_t* mw = a.mask + (size_t)token * a.words;
                            auto word = [&](int i) -> uint64_t { return i < a.words ? (uint64_t)(uint32_t)mw[i] : 0ull; };
                            uint64_t bits = (word(wi) | word(wi + 1) << 32) >> sh;
                            if (sh) bits |= word(wi + 2) << (64 - sh);
                            bits &= low_bits(w.r.n - d0);
                            vis &= low_bits(dc) | bits << max(dc, 0);
                        }
                        const uint32_t v0 = (uint32_t)vis, v1 = (uint32_t)(vis >> 32);
#pragma unroll
                        for (int c = 0; c < 32; ++c) {
                            if (!(v0 >> c & 1u)) s[c] = -INFINITY;
                            if (!(v1 >> c & 1u)) s[32 + c] = -INFINITY;
                        }
                    }
                    float m8[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) m8[i] = s[i];
#pragma unroll
                    for (int c = 8; c < 64; c += 8)
#pragma unroll
                        for (int i = 0; i < 8; ++i) m8[i] = fmaxf(m8[i], s[c + i]);
                    mx = fmaxf(fmaxf(fmaxf(m8[0], m8[1]), fmaxf(m8[2], m8[3])), fmaxf(fmaxf(m8[4], m8[5]), fmaxf(m8[6], m8[7])));
                    xch[hf * 128 + row] = mx;
                }
                ok = named_bar_and(pair_bar, 64, ok);
                if (!ok) break;
                mx = fmaxf(mx, xch[(1 - hf) * 128 + row]);
                named_bar_sync(pair_bar, 64);  // both read before the buffer is reused
                const float m_tile = mx * a.scale_log2;
                float alpha = 1.f;
                const bool moved = m_tile > m_ref + kRescaleLog2;  // lazy: p stays below 2^8
                if (moved) {
                    alpha = m_ref == -INFINITY ? 0.f : fast_exp2(m_ref - m_tile);
                    m_ref = m_tile;
                }
                const float m_use = m_ref == -INFINITY ? 0.f : m_ref;
                float rs[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
                uint32_t pk[32];
                // l sums p in fp32; the P of the product is rounded to bf16 (an MMA takes both operands
                // in V's type), half a step of 2^-8 that averages out over the keys
#pragma unroll
                for (int c = 0; c < 64; c += 2) {
                    const float p0 = fast_exp2(fmaf(s[c], a.scale_log2, -m_use));
                    const float p1 = fast_exp2(fmaf(s[c + 1], a.scale_log2, -m_use));
                    rs[(c >> 1) & 7] += p0 + p1;
                    pk[c >> 1] = pack_bf16x2(p0, p1);
                }
                l = l * alpha + (((rs[0] + rs[1]) + (rs[2] + rs[3])) + ((rs[4] + rs[5]) + (rs[6] + rs[7])));
                if (!w.begins && __any_sync(0xffffffffu, moved)) {  // the same for the pair
                    const int jp = j - 1;
                    const bool okw = __all_sync(0xffffffffu, mbar_wait(smem_u32(&pv_done[jp % C::kSBuf]), (jp / C::kSBuf) & 1,
                                                                       abort_flag, a.status, 0x4d));
                    ok = named_bar_and(pair_bar, 64, okw);
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll 1
                    for (int c = hf * (C::kDV / 64); c < (hf + 1) * (C::kDV / 64); ++c) {
                        uint32_t raw[32];
                        tmem_ld32(tO + c * 32 + lane_base, raw);
                        tmem_ld_wait();
#pragma unroll
                        for (int e = 0; e < 32; ++e) raw[e] = __float_as_uint(__uint_as_float(raw[e]) * alpha);
                        tmem_st32(tO + c * 32 + lane_base, raw);
                    }
                }
                tmem_st32(tS0 + buf * 128 + 64 * hf + lane_base, pk);
                tmem_st_wait();
                tc_fence_before();
            }
            if (!ok) break;
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&p_full[buf]));
            if (!w.ends()) continue;

            // ---- the piece is done: results, or this CTA's partials --------------------------------
            // (a quarter without rows waits as well: its arrival on o_free must not run a piece ahead)
            const bool okw = __all_sync(0xffffffffu, mbar_wait(smem_u32(&pv_done[buf]), (j / C::kSBuf) & 1, abort_flag, a.status, 0x4e));
            if (!busy) ok = okw;
            if (busy) {
                xch[hf * 128 + row] = l;
                ok = named_bar_and(pair_bar, 64, okw);
                if (!ok) break;
                tc_fence_after();
                l += xch[(1 - hf) * 128 + row];
                named_bar_sync(pair_bar, 64);
                const bool from = pg_begin == 0, to = w.pg + w.np == w.r.npg;
                const bool row_ok = row < rows;
                const int head = w.head() * a.G + row % a.G, col0 = w.split() * C::kDV;
                const float inv = l > 0.f ? 1.f / l : 0.f;
                uint16_t* orow = a.o + ((size_t)token * a.Hq + head) * D + col0;
                float* prow = a.part + ((size_t)(2 * k + (from ? 1 : 0)) * a.rows_cap + row) * C::kRowF;
#pragma unroll 1
                for (int c = hf * (C::kDV / 64); c < (hf + 1) * (C::kDV / 64); ++c) {
                    uint32_t raw[32];
                    tmem_ld32(tO + c * 32 + lane_base, raw);
                    tmem_ld_wait();
                    if (!row_ok) continue;
                    if (from && to) {
#pragma unroll
                        for (int e = 0; e < 32; e += 8) {
                            uint4 x4;
                            x4.x = pack_bf16x2(__uint_as_float(raw[e]) * inv, __uint_as_float(raw[e + 1]) * inv);
                            x4.y = pack_bf16x2(__uint_as_float(raw[e + 2]) * inv, __uint_as_float(raw[e + 3]) * inv);
                            x4.z = pack_bf16x2(__uint_as_float(raw[e + 4]) * inv, __uint_as_float(raw[e + 5]) * inv);
                            x4.w = pack_bf16x2(__uint_as_float(raw[e + 6]) * inv, __uint_as_float(raw[e + 7]) * inv);
                            *reinterpret_cast<uint4*>(orow + c * 32 + e) = x4;
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; e += 4)
                            *reinterpret_cast<uint4*>(prow + c * 32 + e) = make_uint4(raw[e], raw[e + 1], raw[e + 2], raw[e + 3]);
                    }
                }
                if (row_ok && hf == 0) {
                    if (!(from && to)) prow[C::kDV] = m_ref, prow[C::kDV + 1] = l;
                    else if (col0 == 0)
                        a.lse[(size_t)head * a.T + token] = l > 0.f ? (m_ref + __log2f(l)) * 0.69314718055994531f : -INFINITY;
                }
            }
            if (!ok) break;
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(o_free));
            if (warp == 2 && lane == 0 && w.left == w.np) {  // the share's last piece
                TreeSpan sp = {};
                if (pg_begin == 0 && w.pg + w.np < w.r.npg) {
                    const long long last = u1 - 1 + (w.r.npg - (w.pg + w.np));  // the segment's last unit
                    sp.ctas = owner_of(last, P, Gc) - k + 1;
                    sp.row0 = w.r.start + tok0, sp.rows = rows, sp.head0 = w.head() * a.G, sp.col0 = w.split() * C::kDV;
                }
                a.span[k] = sp;
            }
        }
    }
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tbase, 512);
    }
}

// Combines the partials of the segment that starts in CTA blockIdx.x of the grid above and ends in a later
// one: its own tail slot, then the head slots of the CTAs behind it. A thread owns 8 columns of a row and
// folds kFold slots at a time, their loads in flight together.
constexpr int kMergeThreads = 128;
constexpr int kMergeY = 16;
constexpr int kFold = 4;

template <int D>
__global__ void __launch_bounds__(kMergeThreads) tree_merge_kernel(TreeArgs a) {
    using C = TreeCfg<D>;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const TreeSpan sp = a.span[blockIdx.x];
    if (sp.ctas == 0) return;
    constexpr int VPR = C::kDV / 8;
    for (int it = blockIdx.y * kMergeThreads + threadIdx.x; it < sp.rows * VPR; it += kMergeY * kMergeThreads) {
        const int row = it / VPR, col = it % VPR * 8;
        float M = -INFINITY, l = 0.f, O[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        for (int q0 = 0; q0 < sp.ctas; q0 += kFold) {
            float2 ml[kFold];
            float4 v[kFold][2];
#pragma unroll
            for (int i = 0; i < kFold; ++i) {
                ml[i] = make_float2(-INFINITY, 0.f);
                v[i][0] = v[i][1] = make_float4(0.f, 0.f, 0.f, 0.f);
                const int q = q0 + i;
                if (q < sp.ctas) {
                    const float* p = a.part + ((size_t)(2 * (blockIdx.x + q) + (q == 0 ? 1 : 0)) * a.rows_cap + row) * C::kRowF;
                    ml[i] = __ldcg(reinterpret_cast<const float2*>(p + C::kDV));
                    v[i][0] = __ldcg(reinterpret_cast<const float4*>(p + col));
                    v[i][1] = __ldcg(reinterpret_cast<const float4*>(p + col) + 1);
                }
            }
            float Mn = M;
#pragma unroll
            for (int i = 0; i < kFold; ++i) Mn = fmaxf(Mn, ml[i].x);
            if (Mn == -INFINITY) continue;
            const float f = M == -INFINITY ? 0.f : fast_exp2(M - Mn);
            l *= f;
#pragma unroll
            for (int e = 0; e < 8; ++e) O[e] *= f;
#pragma unroll
            for (int i = 0; i < kFold; ++i) {
                const float wt = ml[i].x == -INFINITY ? 0.f : fast_exp2(ml[i].x - Mn);
                l += wt * ml[i].y;
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    O[4 * c] += wt * v[i][c].x, O[4 * c + 1] += wt * v[i][c].y;
                    O[4 * c + 2] += wt * v[i][c].z, O[4 * c + 3] += wt * v[i][c].w;
                }
            }
            M = Mn;
        }
        const float inv = l > 0.f ? 1.f / l : 0.f;
        const int token = sp.row0 + row / a.G, head = sp.head0 + row % a.G;
        uint4 x;
        x.x = pack_bf16x2(O[0] * inv, O[1] * inv), x.y = pack_bf16x2(O[2] * inv, O[3] * inv);
        x.z = pack_bf16x2(O[4] * inv, O[5] * inv), x.w = pack_bf16x2(O[6] * inv, O[7] * inv);
        *reinterpret_cast<uint4*>(a.o + ((size_t)token * a.Hq + head) * D + sp.col0 + col) = x;
        if (col == 0 && sp.col0 == 0)
            a.lse[(size_t)head * a.T + token] = l > 0.f ? (M + __log2f(l)) * 0.69314718055994531f : -INFINITY;
    }
}

template <int D>
cudaError_t launch_t(const TreeLaunch& L, TreeArgs a, cudaStream_t stream) {
    using C = TreeCfg<D>;
    cudaError_t e = cudaFuncSetAttribute(tree_paged_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem);
    if (e != cudaSuccess) return e;
    // at most one CTA per tile of the longest step that fits the arguments
    const long long tiles = (L.max_q + a.tokens_tile - 1) / a.tokens_tile;
    const long long most = ((long long)L.max_pages * L.R * tiles * L.Hkv * C::kSplit + kMinPages - 1) / kMinPages;
    int grid = L.sms < kMaxGrid ? L.sms : kMaxGrid;
    if (most < grid) grid = (int)most;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    static const char* const kNames[4] = {"tree_paged_d64", "tree_paged_d128", "tree_paged_d256", "tree_paged_d512"};
    ProfMark m = prof_begin(stream, kNames[D == 64 ? 0 : D == 128 ? 1 : D == 256 ? 2 : 3]);
    e = cudaLaunchKernelEx(&cfg, tree_paged_kernel<D>, L.tq, L.tk, L.tv, a);
    prof_end(stream, m);
    if (e != cudaSuccess || (e = cudaGetLastError()) != cudaSuccess) return e;
    cfg.gridDim = dim3(grid, kMergeY);
    cfg.blockDim = dim3(kMergeThreads);
    cfg.dynamicSmemBytes = 0;
    m = prof_begin(stream, "tree_merge");
    e = cudaLaunchKernelEx(&cfg, tree_merge_kernel<D>, a);
    prof_end(stream, m);
    return e != cudaSuccess ? e : cudaGetLastError();
}

int rows_cap(int G, int max_q) {
    const int tokens = 128 / G;
    return (max_q < tokens ? max_q : tokens) * G;
}
constexpr size_t kSpanBytes = (kMaxGrid * sizeof(TreeSpan) + 255) & ~size_t(255);

}  // namespace

int tree_tokens_per_tile(int G) { return 128 / G; }

size_t tree_workspace_bytes(int G, int max_q, int D) {
    const int dv = D < 256 ? D : 256;
    return kSpanBytes + (size_t)2 * kMaxGrid * rows_cap(G, max_q) * (dv + 4) * 4;
}

cudaError_t launch_tree_paged(const TreeLaunch& L, cudaStream_t stream) {
    TreeArgs a;
    a.block_table = L.block_table, a.seq_lens = L.seq_lens, a.cu_q = L.cu_q, a.mask = L.mask, a.positions = L.positions;
    a.o = L.o, a.lse = L.lse, a.status = L.status;
    a.span = static_cast<TreeSpan*>(L.workspace);
    a.part = reinterpret_cast<float*>(static_cast<uint8_t*>(L.workspace) + kSpanBytes);
    a.R = L.R, a.T = L.T, a.max_q = L.max_q, a.words = L.words, a.Hq = L.Hq, a.Hkv = L.Hkv, a.G = L.Hq / L.Hkv;
    a.tokens_tile = tree_tokens_per_tile(a.G), a.rows_cap = rows_cap(a.G, L.max_q);
    a.max_pages = L.max_pages, a.num_pages = L.num_pages, a.window = L.window;
    a.scale_log2 = L.scale * 1.4426950408889634f;
    switch (L.D) {
        case 64: return launch_t<64>(L, a, stream);
        case 128: return launch_t<128>(L, a, stream);
        case 256: return launch_t<256>(L, a, stream);
        case 512: return launch_t<512>(L, a, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace attn
