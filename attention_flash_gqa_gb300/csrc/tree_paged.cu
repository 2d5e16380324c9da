// Attention of drafted token trees over a paged cache: the verification step of speculative decoding.
//
// Row i of a request with n drafted tokens behind c = L - n cached ones sees the context keys
// j < c (with a window only those with p_i - j < W, p_i = max(position, c)) and the drafted tokens
// d whose bit is set in its mask row:
//     s_ij = scale q_i . k_j,   o_i = sum_j softmax_j(s_ij | visible) v_j,   lse_i = ln sum_j exp(s_ij)
// A row that sees nothing gets o = 0 and lse = -inf.
//
// Few rows over many keys: K and V must be read once for all rows that share them, and one request's
// keys spread over the whole GPU. The floor is the bytes of K and V: a byte serves one FLOP for each row
// of its KV head, and the tensor cores could do some 280 in the time it takes to arrive.
//  * A row tile packs the drafted tokens and the G query heads of one KV head into the 128 rows of
//    an MMA (row = token * G + head, 128 / G tokens a tile), so a KV head's keys serve all of them.
//  * At D <= 128 tensor memory holds two O accumulators, so a CTA has two sets of softmax warps, each
//    with its own O, Q tile, running state, score buffers and MMA issuer. Where a request has more rows
//    than one tile, two row tiles go through together, one per set, and share every key tile (12 requests
//    of 5 to 24 thousand keys and 33 to 64 drafts, Hq 32, Hkv 8, D 128: 193 us, against 299 when each of
//    the two row tiles read all of K and V for itself; 167 with the later steps). Otherwise consecutive
//    segments alternate between the sets: one set's epilogue runs beside the other's first tiles. (Key
//    tiles of one segment in turn to both sets, whose results the epilogue then adds: 45 us against 39
//    for a batch of 64.)
//  * At D = 512 a CTA computes one 256-column half of O; the two CTAs of a key range run side by side
//    (CTAs 2 i and 2 i + 1), so the second copy of K, for the scores, comes from L2.
//  * A unit of work is one key tile, up to eight pages (128 keys), of one segment = (request, KV head,
//    row tile or pair of them). All units are laid end to end and CTA k takes the k-th equal share: it
//    may finish one segment, run through some and start another. (Pages as units: 46.6 us against 43.6
//    for a batch of 64. Some CTAs then had a third more tiles than others, and a tile costs the softmax
//    the same however few pages it has.) A segment that one CTA covers is written out by it; of a shared
//    one every CTA leaves (O, m, l) unnormalised in the workspace and tree_merge_kernel, launched with
//    programmatic serialisation, combines them.
//  * The tiles go through an mbarrier ring, and the pipeline runs on across segments. Tensor memory: O
//    (fp32, up to 256 columns in all) and 256 columns of scores, P (bf16) over them. One set: two buffers
//    of a key tile each. Two sets: two buffers of half a key tile for each, so that a set's softmax of one
//    half runs beside the MMAs of its other half (one buffer of a whole tile per set: 169 us for the 12 long
//    contexts, 54 for 32 requests of 1 to 4 thousand keys at D = 64, against 167 and 51; with P in shared
//    memory instead, which leaves three slots of the ring, 260 for the long ones).
//    Only the pages of a tile that exist are loaded and multiplied (N of Q K^T and K of P V follow them,
//    a page being one K step of 16), so only the last page's slots past L need care: a fixer warp zeroes
//    those V rows before their P V (P is 0 there, but 0 * NaN is not).
//
// What bounds it, 152 SMs: at D = 256 the memory (64 requests of 1 to 4 thousand keys, window 1024:
// 185 us, 6.0 TB/s of K and V). At D = 128 and up to 128 rows a request (64 requests of 256 to 1024 keys
// and 5 to 16 drafts: 40 us, 4.3 TB/s) the memory too, once it runs (1.45 us a key tile and SM): 3 us pass
// before the first load, 3 until it arrives, and 8 from the first CTA's end to the merge's. With two row
// tiles (167 us, 5.0 TB/s; 180 once the clock has come down under load) the softmax: the two sets' warps
// of a quarter share a scheduler, and half a tile takes both some 1700 cycles, of which 530 are the
// exponential unit's. At D = 64 (51 us, 3.3 TB/s) the softmax of one set, some 1000 cycles for half a tile.
//
// Warp roles: four softmax warps a set (0-3, and 4-7 at two sets), one TMEM lane quarter each and one
// thread a row, so nothing of a row is exchanged; then set 0's MMA issuer (idle at one set), the fixer, the
// TMA producer (lanes 0-7: a page each) and the other MMA issuer. The last two sit on the schedulers of
// quarters 2 and 3, which have no rows where a tile has 64 or fewer. Quarters without rows only keep the
// barriers going. An issuer is one thread that reads what to do from a word the producer leaves with every
// copy: walking the work itself took it longer than the MMAs (per 128-key tile 1.4 us, of which 0.56 us of
// MMAs). One issuer for both sets' half tiles took 2.9 us a tile (244 us for the 12 long contexts).
#include <cuda_runtime.h>

#include "attn_internal.h"
#include "ptx.cuh"

namespace attn {
namespace {

constexpr int kPage = 16;
constexpr int kTilePages = 8;
constexpr int kSetWarps = 4;
constexpr uint32_t kSubBytes = 16384;  // 128 rows x 64 bf16
constexpr float kRescaleLog2 = 8.0f;
constexpr int kFewUnits = 1 << 14;  // beyond that many units equal shares are long enough
constexpr int kMaxGrid = 192;  // sizes the workspace

__host__ __device__ constexpr int tree_sets(int D) { return D <= 128 ? 2 : 1; }

template <int D>
struct TreeCfg {
    static constexpr int kDV = D < 256 ? D : 256;      // O columns per segment
    static constexpr int kSplit = D / kDV;
    static constexpr int kSets = tree_sets(D);
    // kIssuer0 is set 0's at two sets, and idle at one
    static constexpr int kIssuer0 = kSets * kSetWarps, kFixer = kIssuer0 + 1, kProducer = kFixer + 1, kIssuer = kProducer + 1;
    static constexpr int kWarps = kIssuer + 1;
    static constexpr int kThreads = kWarps * 32;
    static constexpr int kSubs = D >= 128 ? 2 : 1;     // 64-column sub-tiles per slot
    static constexpr int kSlotCols = 64 * kSubs;
    static constexpr uint32_t kSlotBytes = kSubs * kSubBytes;
    static constexpr int kKC = D / kSlotCols;          // slots per K tile
    static constexpr int kVC = kDV / kSlotCols;        // slots per V tile
    // The Q tiles and the ring share kPool bytes. Q holds the rows that a step's largest tile has (a multiple
    // of 8); the MMAs read 128 all the same, past its end whatever follows, for rows of the product that
    // nobody uses. The ring takes what is left, up to kMaxStages slots: at D = 512 three with 128 rows, six
    // with 32.
    static constexpr uint32_t kPool = 229376;
    static constexpr int kMaxStages = D == 64 ? 12 : 6;
    static constexpr uint32_t kPageBytes = 2048 * kSubs;     // one page's rows in a slot
    static constexpr uint32_t kGroupStride = 1024 * kSubs;   // 8 rows of both sub-tiles
    static constexpr uint32_t kOffBar = kPool;
    static constexpr uint32_t kOffScan = kOffBar + 512;
    static constexpr uint32_t kSmem = kOffScan + 192 + 1024;
    static constexpr int kRowF = kDV + 4;              // partial row: O, m, l, 2 pad
    // tensor memory: O of set i at 0 + i * kDV, score buffers at the top
    static_assert(kSets * kDV + 256 <= 512, "tensor memory");
    static_assert(kSmem <= 232448, "shared memory");
    static_assert(kSets == 1 || (kKC == 1 && kVC == 1), "two sets: one slot a tile, K and V in turn");
    static_assert((kPool - kSets * D * 256) / kSlotBytes >= (kSets == 2 ? 4 : 3), "the ring's depth with 128 rows");
};

// What the merge of a segment needs; one per CTA, for the segment that starts in it and ends elsewhere.
struct TreeSpan {
    int ctas;     // shares of the units that hold part of it (0: just this one)
    int row0;     // its first token row
    int rows[2];  // rows (tokens * G) of its row tiles
    int head0;    // first query head
    int col0;     // first O column
    int pad[2];
};

struct TreeArgs {
    const int32_t *block_table, *seq_lens, *cu_q, *mask, *positions;
    uint16_t* o;
    float* lse;
    unsigned* status;
    float* part;      // [2 * grid][rows_cap][kRowF]
    TreeSpan* span;   // [grid]
    int R, T, max_q, words, Hq, Hkv, G, tokens_tile, rows_cap, max_pages, num_pages, window;
    int part_cost, min_share;      // see launch_t
    int q_tokens, q_rows, stages;  // tokens of a copy of Q, rows of a Q tile in shared memory, slots of the ring
    float scale_log2;
};

// A request as the walk sees it; no units if it is empty or inconsistent.
struct Req {
    int start, n, L, pg0, npg, tiles, groups;  // tiles: key tiles; groups: row tiles, or pairs of them
    bool bad;
};
template <int D>
__device__ __forceinline__ Req load_req(const TreeArgs& a, int b) {
    Req r;
    r.start = a.cu_q[b];
    r.n = a.cu_q[b + 1] - r.start;
    r.L = a.seq_lens[b];
    r.bad = r.start < 0 || r.n < 0 || r.n > a.max_q || r.start > a.T - r.n || r.n > r.L ||
            (long long)r.L > (long long)a.max_pages * kPage;
    if (r.bad || r.n == 0) {
        r.n = r.npg = r.pg0 = r.tiles = r.groups = 0;
        return r;
    }
    const int c = r.L - r.n;
    r.pg0 = a.window > 0 && c >= a.window ? (c - a.window + 1) / kPage : 0;  // no row sees an earlier key
    r.npg = (r.L + kPage - 1) / kPage - r.pg0;
    r.tiles = (r.npg + kTilePages - 1) / kTilePages;
    const int tokens = a.tokens_tile * TreeCfg<D>::kSets;
    r.groups = (r.n + tokens - 1) / tokens;
    return r;
}
template <int D>
__device__ __forceinline__ long long req_units(const TreeArgs& a, const Req& r) {
    return (long long)r.tiles * r.groups * a.Hkv;
}

// A copy's word: pages of the tile in bits 0-3, rows of its last page to keep in bits 4-7 (0: all), and flags.
enum : uint32_t {
    kBegins = 1u << 8,    // first tile of a piece
    kEnds = 1u << 9,      // last tile of a piece
    kDual = 1u << 10,     // both sets work on it
    kSet1 = 1u << 11,     // otherwise: set 1 does
    kLast = 1u << 12,     // last tile of the share
    kIsV = 1u << 13,      // a copy of V
    kChunkEnd = 1u << 14  // the tile's last copy
};

// Walks the tiles of a CTA's share; the producer and the softmax warps follow the same walk.
template <int D>
struct Walk {
    using C = TreeCfg<D>;
    Req r;
    int b, seg, pg, np;     // request, segment in it, first page (from pg0) and pages of the tile
    int head, tok0;         // of the segment; tok0: first drafted token of its rows
    int left;               // tiles of the share from here on
    bool begins, ends;      // first / last tile of a piece (a segment's pages in this CTA)
    bool dual;              // two row tiles: one for each set
    int set;                // the set that takes the piece (dual: both)
    int turn;               // the next single piece's set

    __device__ __forceinline__ void start(const TreeArgs& a, int b_, const Req& r_, int off, int units) {
        b = b_;
        r = a.R <= 32 ? r_ : load_req<D>(a, b);
        seg = off / r.tiles;
        pg = (off - seg * r.tiles) * kTilePages;
        left = units;
        turn = 0;
        piece(a);
        size();
    }
    __device__ __forceinline__ void piece(const TreeArgs& a) {
        begins = true;
        const int group = seg % r.groups;
        head = seg / r.groups;
        tok0 = group * a.tokens_tile * C::kSets;
        dual = C::kSets == 2 && tok0 + a.tokens_tile < r.n;
        set = 0;
        if (C::kSets == 2 && !dual) set = turn, turn ^= 1;
    }
    __device__ __forceinline__ void size() {
        np = min(kTilePages, r.npg - pg);
        ends = pg + np == r.npg || left == 1;
    }
    __device__ __forceinline__ bool more() const { return left > 0; }
    __device__ __forceinline__ void next(const TreeArgs& a) {
        pg += np, --left;
        begins = false;
        if (ends) {
            if (left == 0) return;
            pg = 0;  // a piece ends before the share does only with its segment
            if (++seg == r.groups * a.Hkv) {
                seg = 0;
                do r = load_req<D>(a, ++b);  // the share holds more units: there is another request
                while (r.npg == 0);
            }
            piece(a);
        }
        size();
    }
    // what the issuer and the fixer need of the tile
    __device__ __forceinline__ uint32_t word() const {
        const int tail = pg + np == r.npg ? r.L % kPage : 0;  // rows of its last page, if slots of it lie past L
        return (uint32_t)np | (uint32_t)tail << 4 | (begins ? kBegins : 0u) | (ends ? kEnds : 0u) | (dual ? kDual : 0u) |
               (set ? kSet1 : 0u) | (left == 1 ? kLast : 0u);
    }
    // whether set s works on the piece
    __device__ __forceinline__ bool mine(int s) const { return dual || set == s; }
};

__device__ __forceinline__ uint64_t low_bits(int n) { return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1; }

// ceil(x / y) for 0 <= x, 1 <= y, x + y < kCeilDivSum. The numerator x + y - 1/2 is exact, and the exact quotient lies
// 1 / (2 y) or more from an integer; __fdividef is off by 2 ulp at most, less than (x + y) / y * 2^-22, which is less
// than 1 / (2 y) while x + y < 2^21. Calls here have x below kFewUnits (units, tiles, shares) and y below it too.
constexpr int kCeilDivSum = 1 << 21;
static_assert(2 * kFewUnits <= kCeilDivSum, "ceil_div's range");
__device__ __forceinline__ int ceil_div(int x, int y) { return __float2int_rd(__fdividef((float)(x + y) - 0.5f, (float)y)); }

// P units over G CTAs: the first P % G of them take one more than the others.
__device__ __forceinline__ int share_start(int k, int q, int rem) { return k * q + min(k, rem); }
__device__ __forceinline__ int owner_of(int u, int q, int rem) {
    const int big = rem * (q + 1);
    return u < big ? u / (q + 1) : rem + (u - big) / q;
}

template <int D>
__global__ void __launch_bounds__(TreeCfg<D>::kThreads, 1)
    tree_paged_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                      const __grid_constant__ CUtensorMap tv, const __grid_constant__ TreeArgs a) {
    using C = TreeCfg<D>;
    constexpr bool kHalf = C::kSets == 2;  // steps of half a key tile
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    const int stages = a.stages;
    const uint32_t q_sub = a.q_rows * 128, q_bytes = q_sub * (D / 64);  // a 64-column sub-tile of Q, all of it
    const uint32_t sQ = sbase, sSlots = sbase + C::kSets * q_bytes;
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
    uint64_t* full = bars;                      // [kMaxStages]
    uint64_t* empty = full + C::kMaxStages;     // [kMaxStages]
    // per set: its Q tile is loaded / was last read, its O was read out
    uint64_t* q_full = empty + C::kMaxStages;   // [2]
    uint64_t* q_free = q_full + 2;           // [2]
    uint64_t* o_free = q_free + 2;           // [2]
    // per set and score buffer (index 2 set + buffer): at most one pending phase each, and only the set's
    // own steps, so that it sees every phase
    uint64_t* s_full = o_free + 2;           // [4]
    uint64_t* p_full = s_full + 4;           // [4]
    uint64_t* pv_done = p_full + 4;          // [4]
    uint64_t* vfix = pv_done + 4;            // [kMaxStages] the last page's V rows past L are zeroed
    uint64_t* mma_idle = vfix + C::kMaxStages;
    uint32_t* words = reinterpret_cast<uint32_t*>(mma_idle + 1);  // [kMaxStages] the copies' words
    uint32_t* tmem_slot = words + C::kMaxStages;
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    long long* scan = reinterpret_cast<long long*>(smem + C::kOffScan);  // [kWarps]
    int* first = reinterpret_cast<int*>(scan + C::kWarps);               // where the share starts
    static_assert((3 * C::kMaxStages + 19) * 8 + C::kMaxStages * 4 + 8 <= 512 && (C::kWarps + 1) * 8 <= 192, "barrier area");
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int k = blockIdx.x;
    const int part = k / C::kSplit, split = k % C::kSplit;  // its share of the units, and of O's columns

    if (tid == 0) {
        for (int s = 0; s < C::kMaxStages; ++s) {
            mbar_init(smem_u32(&full[s]), 1);
            mbar_init(smem_u32(&empty[s]), C::kSets + 1);  // each issuer's MMAs that read it, and the fixer
            mbar_init(smem_u32(&vfix[s]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&q_full[i]), 1);
            mbar_init(smem_u32(&q_free[i]), 1);
            mbar_init(smem_u32(&o_free[i]), kSetWarps);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(smem_u32(&s_full[i]), 1);
            mbar_init(smem_u32(&p_full[i]), kSetWarps);
            mbar_init(smem_u32(&pv_done[i]), 1);
        }
        mbar_init(smem_u32(mma_idle), C::kSets);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (tid == C::kProducer * 32) prefetch_tmap(&tq), prefetch_tmap(&tk), prefetch_tmap(&tv);
    if (warp == C::kIssuer) {
        tmem_alloc(smem_u32(tmem_slot), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = *tmem_slot;
    const uint32_t tO = tbase, tS0 = tbase + 256;
    // Launched with programmatic serialisation: nothing is read before the kernel in front has
    // finished. The merge kernel may be scheduled from here on (it waits for this grid).
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    // ---- the CTA's share -----------------------------------------------------------------------
    long long P = 0;  // units of the step
    int q = 0, rem = 0, u0 = 0, share = 0, first_b = 0, first_off = 0;
    int chunks = 0;  // shares that a segment is cut into, if each lies in one segment
    Req first_req = {};
    // (a step of 2^31 tiles or more, far beyond what a cache can hold, is reported and left alone)
    auto shares = [&]() -> bool {  // whether the CTA has one
        if (P > 0x7fffffffll) {
            if (tid == 0 && k == 0) atomicOr(a.status, DEVSTAT_BOUNDS);
            return false;
        }
        const int units = (int)P, Gc = min(units, (int)gridDim.x / C::kSplit);
        if (part >= Gc) return false;
        q = units / Gc, rem = units - q * Gc;
        u0 = share_start(part, q, rem), share = q + (part < rem);
        return true;
    };
    bool works;  // uniform
    if (a.R <= 32) {
        // Every warp looks through all requests, a lane each, and nobody waits for another (one request of 8 drafts
        // and 950 keys, D 128: 10.4 us against 11.2 the other way).
        Req r = {};
        if (lane < a.R) r = load_req<D>(a, lane);
        if (r.bad && k == 0 && warp == 0) atomicOr(a.status, DEVSTAT_BOUNDS);
        const long long n = req_units<D>(a, r);
        long long x = n;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, x, d);
            if (lane >= d) x += y;
        }
        P = __shfl_sync(0xffffffffu, x, 31);
        // Shares that lie in one segment each, where those are not much longer than equal shares of the whole: a CTA
        // then leaves one partial result instead of two (3 requests, window 1024, up to 37 drafts, 30 heads over 5, D
        // 256: 22.0 us against 28.3; 4 requests of 700 to 2162 keys, 33 to 41 drafts, 12 heads over 3, D 128: 19.0
        // against 24.5; the search costs calls that do not end up so 0.1 to 0.4 us).
        const int G = gridDim.x / C::kSplit;
        unsigned at = 0u;
        bool aligned = false;
        if (__builtin_expect((P > G || a.min_share > 1) && P < kFewUnits, 0)) {
            const int segs = r.groups * a.Hkv;
            int most = max(ceil_div((int)P, G), a.min_share), c, total;  // tiles of a share, shares of a segment, of all
            const int end = max(most, (4 * (int)P + G * a.part_cost / 2) / (4 * G));
            do {
                c = ceil_div(r.tiles, most);
                total = (int)__reduce_add_sync(0xffffffffu, (unsigned)(segs * c));
            } while (total > G && ++most <= end);
            if (total <= G) {
                aligned = true;
                works = part < total;
                int y = segs * c;
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const int z = __shfl_up_sync(0xffffffffu, y, d);
                    if (lane >= d) y += z;
                }
                const int off = part - (y - segs * c);
                at = __ballot_sync(0xffffffffu, off >= 0 && part < y);
                if (off >= 0 && part < y) {
                    const int each = ceil_div(r.tiles, c), seg_ = ceil_div(off + 1, c) - 1, chunk = off - seg_ * c;
                    first_off = seg_ * r.tiles + chunk * each;
                    share = min(each, r.tiles - chunk * each);
                    chunks = c;
                }
            }
        }
        if (!aligned) {
            works = shares();
            at = __ballot_sync(0xffffffffu, works && x - n <= u0 && u0 < x);
            first_off = u0 - (int)(x - n);
        }
        if (at) {
            first_b = __ffs(at) - 1;
            first_off = __shfl_sync(0xffffffffu, first_off, first_b);
            share = __shfl_sync(0xffffffffu, share, first_b);
            chunks = __shfl_sync(0xffffffffu, chunks, first_b);
            first_req.start = __shfl_sync(0xffffffffu, r.start, first_b);
            first_req.n = __shfl_sync(0xffffffffu, r.n, first_b);
            first_req.L = __shfl_sync(0xffffffffu, r.L, first_b);
            first_req.pg0 = __shfl_sync(0xffffffffu, r.pg0, first_b);
            first_req.npg = __shfl_sync(0xffffffffu, r.npg, first_b);
            first_req.tiles = __shfl_sync(0xffffffffu, r.tiles, first_b);
            first_req.groups = __shfl_sync(0xffffffffu, r.groups, first_b);
        }
    } else {
        // units before each thread's run of requests
        const int per = (a.R + C::kThreads - 1) / C::kThreads;
        const int b0 = min(tid * per, a.R), b1 = min(b0 + per, a.R);
        long long sum = 0;
        for (int b = b0; b < b1; ++b) {
            const Req r = load_req<D>(a, b);
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
        x -= sum;
        for (int w = 0; w < C::kWarps; ++w) {
            if (w < warp) x += scan[w];
            P += scan[w];
        }
        works = shares();
        if (works && x <= u0 && u0 < x + sum) {
            Req r;
            int b = b0, off = 0;
            for (;; ++b) {
                r = load_req<D>(a, b);
                const long long n = req_units<D>(a, r);
                off = u0 - (int)x;
                if (off < n) break;
                x += n;
            }
            first[0] = b, first[1] = off;
            // the producer's first page ids, on their way while the CTA meets
            asm volatile("prefetch.global.L2 [%0];" ::"l"(a.block_table + (size_t)b * a.max_pages + r.pg0 + off % r.tiles * kTilePages));
        }
        __syncthreads();
        first_b = first[0], first_off = first[1];
    }
    if (tid == 0 && !works) a.span[k].ctas = 0;  // (else the share's last piece writes it)
    // The ring's slots go round in the order of the copies. One set: K and V slots in the issuer's order, K(0)
    // K(1) V(0) K(2) V(1) .. (a K tile of D = 512 is longer than the ring). Two sets: K(0) V(0) K(1) V(1) ..,
    // each issuer following all of them: tile i's K is copy 2 i, its V copy 2 i + 1.

    if (!works) {
        // no units left for this CTA
    } else if (warp < C::kSets * kSetWarps) {
        // --------------------------------- softmax ----------------------------------------------
        const int set = warp / kSetWarps, quad = warp & 3;
        const int row = quad * 32 + lane;  // row of the tile = TMEM lane
        const uint32_t lane_base = (uint32_t)(quad * 32) << 16;
        const uint32_t tOset = tO + set * C::kDV + lane_base;
        float m_ref = -INFINITY, l = 0.f;
        int first_key = 0, token = 0, pg_begin = 0, rows = 0, ctx = 0;
        uint64_t bits0 = 0;
        int step = 0;                       // tile of the share
        uint32_t phases = 0u;               // of the set's two buffers
        int prev = 0;                       // the set's step before: buffer, and its phase
        uint32_t prev_phase = 0u;
        bool busy = false, ok = true;
        Walk<D> w;
        w.start(a, first_b, first_req, first_off, share);
        for (; ok && w.more(); ++step, w.next(a)) {
            if (!w.mine(set)) continue;
            if (w.begins) {
                const int tok = w.tok0 + (w.dual && set ? a.tokens_tile : 0);  // of the request
                ctx = w.r.L - w.r.n;
                rows = min(a.tokens_tile, w.r.n - tok) * a.G;
                busy = quad * 32 < rows;  // the quarter has rows
                m_ref = -INFINITY, l = 0.f;
                pg_begin = w.pg;
                token = w.r.start + min(tok + row / a.G, w.r.n - 1);
                // the row's first 64 mask bits, on their way while the scores are made
                const int32_t* mw = a.mask + (size_t)token * a.words;
                bits0 = (uint64_t)(uint32_t)mw[0] | (a.words > 1 ? (uint64_t)(uint32_t)mw[1] << 32 : 0ull);
                first_key = a.window > 0 ? max(0, min(ctx, max(a.positions[token], ctx) - a.window + 1)) : 0;
            }
            const int steps = kHalf && w.np > kTilePages / 2 ? 2 : 1;
#pragma unroll 1
            for (int h = 0; h < steps; ++h) {
                const int buf = kHalf ? h : step & 1;
                const uint32_t phase = phases >> buf & 1u;
                phases ^= 1u << buf;
                const uint32_t tS = tS0 + (kHalf ? (2 * set + h) * 64 : buf * 128) + lane_base;
                ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&s_full[2 * set + buf]), phase, abort_flag, a.status, 0x4c));
                if (busy && ok) {
                    const int key0 = (w.r.pg0 + w.pg) * kPage;
                    const bool edge = __any_sync(0xffffffffu, key0 + 127 >= ctx || w.np < kTilePages || key0 < first_key);
                    auto visible = [&](int half) -> uint64_t {  // the row's visible keys of 64 half .. of the tile
                        const int k0 = key0 + 64 * half;
                        uint64_t vis = low_bits(w.np * kPage - 64 * half) & ~low_bits(first_key - k0);
                        const int dc = ctx - k0;  // column of the first drafted token
                        if (dc < 64) {
                            const int d0 = max(0, -dc);
                            uint64_t bits;
                            if (d0 == 0 || a.words <= 2) {
                                bits = d0 < 64 ? bits0 >> d0 : 0ull;
                            } else {
                                const int wi = d0 >> 5, sh = d0 & 31;
                                const int32_t* mw = a.mask + (size_t)token * a.words;
                                auto word = [&](int i) -> uint64_t { return i < a.words ? (uint64_t)(uint32_t)mw[i] : 0ull; };
                                bits = (word(wi) | word(wi + 1) << 32) >> sh;
                                if (sh) bits |= word(wi + 2) << (64 - sh);
                            }
                            bits &= low_bits(w.r.n - d0);
                            vis &= low_bits(dc) | bits << max(dc, 0);
                        }
                        return vis;
                    };
                    // The running maximum is lazy: it moves only when a row's tile maximum exceeds it by more than
                    // 2^8, so p stays below that and most tiles need no rescale.
                    auto move_max = [&](float mx) -> bool {
                        const float m_tile = mx * a.scale_log2;
                        const bool moved = m_tile > m_ref + kRescaleLog2;
                        if (!__any_sync(0xffffffffu, moved)) return true;
                        const float alpha = !moved ? 1.f : m_ref == -INFINITY ? 0.f : fast_exp2(m_ref - m_tile);
                        if (moved) m_ref = m_tile;
                        l *= alpha;
                        if (w.begins && h == 0) return true;
                        // P V of the set's step before, and so every earlier one, is complete
                        ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&pv_done[2 * set + prev]), prev_phase, abort_flag, a.status, 0x4d));
                        if (!ok) return false;
                        tc_fence_after();
#pragma unroll 1
                        for (int c = 0; c < C::kDV / 16; ++c) {
                            uint32_t raw[16];
                            tmem_ld16(tOset + c * 16, raw);
                            tmem_ld_wait();
#pragma unroll
                            for (int e = 0; e < 16; ++e) raw[e] = __float_as_uint(__uint_as_float(raw[e]) * alpha);
                            tmem_st16(tOset + c * 16, raw);
                        }
                        return true;
                    };
                    float2 rs[2] = {{0.f, 0.f}, {0.f, 0.f}};
                    const float2 sc = make_float2(a.scale_log2, a.scale_log2);
                    tc_fence_after();
                    // l sums p in fp32; the P of the product is rounded to bf16, since an MMA takes both operands in V's
                    // type, as in the other attention kernels here: o is then off by 0.0023 of its size against 64
                    // bits, 0.0017 of it the rounding of o itself. A second product, with what the rounding leaves of P,
                    // takes the rest away and was measured: batch of 64 at D 128 46.4 us against 40.1, 12 long contexts
                    // 213 against 166, D 64 59.8 against 51.4, windowed D 256 188.8 against 185.8, D 512 39.5 against 38.0.
                    // Two sets: the half tile's 64 scores in registers. One set: two passes over the tile, 64 scores at a
                    // time: the maximum of the lower and the upper half, then the exponentials of the upper half, still
                    // in registers, and of the lower one, read again. One loop, so that each part's code is there once:
                    // a CTA of a short call runs some twenty tiles, and the instruction fetches of a longer body cost
                    // more than they save (64 requests, window 1024, D 256: 192 us against 202 unrolled).
                    if constexpr (kHalf) {
                        float s[64];
                        {
                            uint32_t raw[2][32];
#pragma unroll
                            for (int c = 0; c < 2; ++c) tmem_ld32(tS + c * 32, raw[c]);
                            tmem_ld_wait();
#pragma unroll
                            for (int c = 0; c < 2; ++c)
#pragma unroll
                                for (int e = 0; e < 32; ++e) s[c * 32 + e] = __uint_as_float(raw[c][e]);
                        }
                        if (edge) {  // hidden keys to -inf
                            const uint64_t vis = visible(h);
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
                        const float mx = fmaxf(fmaxf(fmaxf(m8[0], m8[1]), fmaxf(m8[2], m8[3])), fmaxf(fmaxf(m8[4], m8[5]), fmaxf(m8[6], m8[7])));
                        if (!move_max(mx)) break;
                        const float m_use = m_ref == -INFINITY ? 0.f : -m_ref;
                        const float2 mm = make_float2(m_use, m_use);
                        uint32_t pk[32];
#pragma unroll
                        for (int e = 0; e < 64; e += 2) {
                            const float2 x2 = __ffma2_rn(make_float2(s[e], s[e + 1]), sc, mm);
                            const float2 p2 = make_float2(fast_exp2(x2.x), fast_exp2(x2.y));
                            rs[(e >> 1) & 1] = __fadd2_rn(rs[(e >> 1) & 1], p2);
                            pk[e >> 1] = pack_bf16x2(p2.x, p2.y);
                        }
                        tmem_st32(tS, pk);
                    } else {
                        float s[64];
                        float mx = -INFINITY;
                        float2 mm = {0.f, 0.f};
#pragma unroll 1
                        for (int pass = 0; pass < 4; ++pass) {
                            const int half = pass == 1 || pass == 2;
                            if (pass != 2) {  // scores of keys 64 half .. of the tile, hidden ones at -inf
                                uint32_t raw[2][32];
#pragma unroll
                                for (int c = 0; c < 2; ++c) tmem_ld32(tS + 64 * half + c * 32, raw[c]);
                                tmem_ld_wait();
#pragma unroll
                                for (int c = 0; c < 2; ++c)
#pragma unroll
                                    for (int e = 0; e < 32; ++e) s[c * 32 + e] = __uint_as_float(raw[c][e]);
                                if (edge) {
                                    const uint64_t vis = visible(half);
                                    const uint32_t v0 = (uint32_t)vis, v1 = (uint32_t)(vis >> 32);
#pragma unroll
                                    for (int c = 0; c < 32; ++c) {
                                        if (!(v0 >> c & 1u)) s[c] = -INFINITY;
                                        if (!(v1 >> c & 1u)) s[32 + c] = -INFINITY;
                                    }
                                }
                            }
                            if (pass < 2) {
                                float m8[8];
#pragma unroll
                                for (int i = 0; i < 8; ++i) m8[i] = s[i];
#pragma unroll
                                for (int c = 8; c < 64; c += 8)
#pragma unroll
                                    for (int i = 0; i < 8; ++i) m8[i] = fmaxf(m8[i], s[c + i]);
                                mx = fmaxf(mx, fmaxf(fmaxf(fmaxf(m8[0], m8[1]), fmaxf(m8[2], m8[3])), fmaxf(fmaxf(m8[4], m8[5]), fmaxf(m8[6], m8[7]))));
                                if (pass == 0) continue;
                                if (!move_max(mx)) break;
                                mm.x = mm.y = m_ref == -INFINITY ? 0.f : -m_ref;
                            } else {
                                uint32_t pk[32];
#pragma unroll
                                for (int e = 0; e < 64; e += 2) {
                                    const float2 x2 = __ffma2_rn(make_float2(s[e], s[e + 1]), sc, mm);
                                    const float2 p2 = make_float2(fast_exp2(x2.x), fast_exp2(x2.y));
                                    rs[(e >> 1) & 1] = __fadd2_rn(rs[(e >> 1) & 1], p2);
                                    pk[e >> 1] = pack_bf16x2(p2.x, p2.y);
                                }
                                tmem_st32(tS + 64 * half, pk);
                            }
                        }
                    }
                    l += (rs[0].x + rs[0].y) + (rs[1].x + rs[1].y);
                    tmem_st_wait();
                    tc_fence_before();
                }
                if (!ok) break;
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&p_full[2 * set + buf]));
                prev = buf, prev_phase = phase;
            }
            if (!ok) break;
            if (!w.ends) continue;

            // ---- the piece is done: results, or this CTA's partials --------------------------------
            // (a quarter without rows waits as well: its arrival on o_free must not run a piece ahead)
            ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&pv_done[2 * set + prev]), prev_phase, abort_flag, a.status, 0x4e));
            if (!ok) break;
            tc_fence_after();
            if (busy) {
                const bool from = pg_begin == 0, to = w.pg + w.np == w.r.npg;
                const bool row_ok = row < rows;
                const int head = w.head * a.G + row % a.G, col0 = split * C::kDV;
                const float inv = l == 0.f ? 0.f : 1.f / l;  // (l of a row with NaN scores is NaN, and so are o and lse)
                uint16_t* orow = a.o + ((size_t)token * a.Hq + head) * D + col0;
                float* prow = a.part + ((size_t)(2 * k + (from ? 1 : 0)) * a.rows_cap + (w.dual && set ? 128 : 0) + row) * C::kRowF;
#pragma unroll 1
                for (int c = 0; c < C::kDV / 32; ++c) {
                    uint32_t raw[32];
                    tmem_ld32(tOset + c * 32, raw);
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
                if (row_ok) {
                    // NaN scores move no maximum: a partial with some has m = inf, so that the merge, which passes over
                    // those with m = -inf, makes the row NaN whatever its other partials hold
                    if (!(from && to)) prow[C::kDV] = l == l ? m_ref : INFINITY, prow[C::kDV + 1] = l;
                    else if (col0 == 0)
                        a.lse[(size_t)head * a.T + token] = l == 0.f ? -INFINITY : (m_ref + __log2f(l)) * 0.69314718055994531f;
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&o_free[set]));
            // the share's last piece: does its segment go on elsewhere?
            if (quad == 0 && lane == 0 && w.left == 1 && (!w.dual || set == 0)) {
                TreeSpan sp = {};
                if (pg_begin == 0 && w.pg + w.np < w.r.npg) {
                    // (else the CTA that holds the segment's last unit)
                    sp.ctas = chunks > 0 ? chunks
                                         : owner_of(u0 + share - 1 + (w.r.npg - (w.pg + w.np) + kTilePages - 1) / kTilePages, q, rem) - part + 1;
                    sp.row0 = w.r.start + w.tok0, sp.head0 = w.head * a.G, sp.col0 = split * C::kDV;
                    sp.rows[0] = rows;
                    sp.rows[1] = w.dual ? min(a.tokens_tile, w.r.n - w.tok0 - a.tokens_tile) * a.G : 0;
                }
                a.span[k] = sp;
            }
        }
    }
    if (!works || warp < C::kSets * kSetWarps) {
    } else if (warp == C::kProducer) {
        // ------------------------------- TMA producer ----------------------------------------
        // what a step reads once goes through L2 as the first to be evicted
        const uint64_t policy = l2_policy_evict_first();
        int slot = 0, round = 0;
        bool ok = true;
        int q_uses[2] = {0, 0};
        auto page_id = [&](const Walk<D>& w) -> int {  // lane i: id of the tile's page i (checked at its use)
            return lane < w.np ? a.block_table[(size_t)w.b * a.max_pages + w.r.pg0 + w.pg + lane] : 0;
        };
        // one slot: np pages, lane i loads page i's 16 rows x kSlotCols columns
        auto load_slot = [&](const CUtensorMap* map, int chunk, int np, int id, uint32_t word, bool once) -> bool {
            if (id < 0 || id >= a.num_pages) {
                atomicOr(a.status, DEVSTAT_BOUNDS);
                id = 0;
            }
            if (round > 0 && !__all_sync(0xffffffffu, mbar_wait(smem_u32(&empty[slot]), (round - 1) & 1, abort_flag, a.status, 0x41)))
                return false;
            const uint32_t fb = smem_u32(&full[slot]);
            if (lane == 0) {
                words[slot] = word;
                mbar_expect_tx(fb, np * C::kPageBytes);
            }
            __syncwarp();
            if (lane < np) {
                const uint32_t dst = sSlots + slot * C::kSlotBytes + lane * C::kPageBytes;
                if (once) tma_load_5d_hint(dst, map, fb, 0, 0, chunk, 0, id, policy);
                else tma_load_5d(dst, map, fb, 0, 0, chunk, 0, id);
            }
            if (++slot == stages) slot = 0, ++round;
            return true;
        };
        auto load_q = [&](const Walk<D>& w, int s, int tok) -> bool {  // rows of drafted tokens tok .. of the piece
            const int uses = s ? q_uses[1] : q_uses[0];
            if (uses > 0 && !__all_sync(0xffffffffu, mbar_wait(smem_u32(&q_free[s]), (uses - 1) & 1, abort_flag, a.status, 0x42)))
                return false;
            if (lane == 0) {
                const uint32_t fb = smem_u32(&q_full[s]);
                mbar_expect_tx(fb, (uint32_t)(D / 64) * a.G * a.q_tokens * 128);
                for (int c = 0; c < D / 64; ++c)
                    tma_load_4d(sQ + s * q_bytes + c * q_sub, &tq, fb, c * 64, w.head * a.G, w.r.start + tok, 0);
            }
            __syncwarp();
            if (s) ++q_uses[1];
            else ++q_uses[0];
            return true;
        };
        Walk<D> wk, wv;
        wk.start(a, first_b, first_req, first_off, share);
        wv = wk;
        int idk = page_id(wk), idv = idk;
        auto load_k = [&]() -> bool {
            if (wk.begins) {
                if (!load_q(wk, wk.set, wk.tok0)) return false;
                if (wk.dual && !load_q(wk, 1, wk.tok0 + a.tokens_tile)) return false;
            }
            for (int c = 0; c < C::kKC; ++c)
                if (!load_slot(&tk, wk.head * (D / 64) + c * C::kSubs, wk.np, idk, wk.word(), C::kSplit == 1 && wk.r.groups == 1)) return false;
            if (C::kSets == 2) idv = idk, wv = wk;
            wk.next(a);
            if (wk.more()) idk = page_id(wk);
            return true;
        };
        auto load_v = [&]() -> bool {
            for (int c = 0; c < C::kVC; ++c)
                if (!load_slot(&tv, wv.head * (D / 64) + split * (C::kDV / 64) + c * C::kSubs, wv.np, idv,
                               wv.word() | kIsV | (c == C::kVC - 1 ? kChunkEnd : 0u), wv.r.groups == 1))
                    return false;
            if (C::kSets == 1) {
                wv.next(a);
                if (wv.more()) idv = page_id(wv);
            }
            return true;
        };
        if constexpr (C::kSets == 2) {
            while (ok && wk.more()) ok = load_k() && load_v();
        } else {
            for (int i = 0; ok && i < 2 && wk.more(); ++i) ok = load_k();
            while (ok && wv.more()) {
                ok = load_v();
                if (ok && wk.more()) ok = load_k();
            }
        }
        // every issued copy has landed before the CTA may leave
        if (lane == 0) {
            const int issued = round * stages + slot;
            for (int s = 0; s < stages && s < issued; ++s) {
                const int last = s + ((issued - 1 - s) / stages) * stages;
                mbar_drain(smem_u32(&full[s]), (last / stages) & 1, a.status, 0x43);
            }
            if (q_uses[0] > 0) mbar_drain(smem_u32(&q_full[0]), (q_uses[0] - 1) & 1, a.status, 0x44);
            if (q_uses[1] > 0) mbar_drain(smem_u32(&q_full[1]), (q_uses[1] - 1) & 1, a.status, 0x44);
        }
    } else if (warp == C::kFixer) {
        // ---------- follows every copy; zeroes V rows past L in a request's last page ---------------
        int slot = 0, phase = 0;
        while (true) {
            if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&full[slot]), phase, abort_flag, a.status, 0x4b))) break;
            const uint32_t word = words[slot];
            const int keep = word >> 4 & 15;
            if ((word & kIsV) && keep) {
                const uint32_t base = sSlots + slot * C::kSlotBytes + ((word & 15) - 1) * C::kPageBytes;
                for (int e = lane; e < (kPage - keep) * 8 * C::kSubs; e += 32) {  // 16-byte pieces
                    const int row = keep + e / (8 * C::kSubs), sub = (e >> 3) % C::kSubs;
                    st_shared_v4(base + (row >> 3) * C::kGroupStride + sub * 1024 + (row & 7) * 128 + (e & 7) * 16, 0u, 0u, 0u, 0u);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&vfix[slot]));
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&empty[slot]));
            if ((word & kLast) && (word & kChunkEnd)) break;
            if (++slot == stages) slot = 0, phase ^= 1;
        }
    } else if (C::kSets == 2 && (warp == C::kIssuer || warp == C::kIssuer0)) {
        // ------------------------------- MMA issuers at two sets, one for each -----------------
        // A step is half a key tile: scores of (set, half) go to that pair's buffer of 64 columns, after the P V
        // that last read it (the pipe runs in order). Beside P V of tile i - 1 come the scores of tile i.
        if (elect_one()) {
            constexpr uint32_t idO = idesc_bf16_f32(128, C::kSlotCols, false, true);  // V is N-major
            const uint32_t set = warp == C::kIssuer ? 1u : 0u;
            auto wait = [&](uint64_t* bar, uint32_t phase, unsigned site) -> bool {
                return mbar_wait(smem_u32(bar), phase, abort_flag, a.status, site);
            };
            auto mine = [&](uint32_t word) -> bool { return (word & kDual) || ((word & kSet1) ? 1u : 0u) == set; };
            const uint64_t dq = sdesc_sw128(sQ + set * q_bytes, 16, 1024);
            const uint32_t tD = tO + set * C::kDV, tB = tS0 + set * 128;
            int ks = 0, vs = 1;                                   // slots of K and V
            uint32_t k_phase = 0u, v_phase = 0u, fix_phase = 0u;  // fix_phase: bits by slot
            uint32_t q_phase = 0u, o_phase = 0u, p_phase = 0u;    // p_phase: bits by half
            bool o_used = false, ok = true, more_s = true, before = false;
            uint32_t ws = 0u, wp = 0u;  // the words of tiles i and i - 1
            do {
                if (before) {
                    if (!(ok = wait(&full[vs], v_phase, 0x49))) break;
                    if (wp >> 4 & 15u) {
                        if (mine(wp) && !(ok = wait(&vfix[vs], fix_phase >> vs & 1u, 0x4f))) break;
                        fix_phase ^= 1u << vs;
                    }
                }
                const bool does_p = before && mine(wp);
                bool does_s = false;
#pragma unroll
                for (uint32_t h = 0; h < 2u; ++h) {
                    const int np = min((int)(wp & 15u) - 4 * (int)h, 4);
                    if (does_p && np > 0) {
                        const bool fresh = (wp & kBegins) && h == 0u;
                        if (fresh) {  // the set's piece before has been read out of O
                            if (o_used && !(ok = wait(&o_free[set], o_phase, 0x48))) break;
                            if (o_used) o_phase ^= 1u;
                            o_used = true;
                        }
                        if (!(ok = wait(&p_full[2 * set + h], p_phase >> h & 1u, 0x47))) break;
                        p_phase ^= 1u << h;
                        tc_fence_after();
                        const uint64_t dv = sdesc_sw128(sSlots + vs * C::kSlotBytes + h * 4 * C::kPageBytes, 1024, C::kGroupStride);
                        const uint32_t tP = tB + h * 64;
                        umma_bf16_ts(tD, tP, dv, idO, fresh ? 0u : 1u);
#pragma unroll
                        for (int kk = 1; kk < 4; ++kk)
                            if (kk < np) umma_bf16_ts(tD, tP + kk * 8, sdesc_at(dv, kk * C::kPageBytes), idO, 1u);
                        umma_commit(smem_u32(&pv_done[2 * set + h]));
                    }
                    if (h == 0u && more_s) {
                        if (!(ok = wait(&full[ks], k_phase, 0x46))) break;
                        ws = words[ks];
                        does_s = mine(ws);
                        if (does_s && (ws & kBegins)) {
                            if (!(ok = wait(&q_full[set], q_phase, 0x45))) break;
                            q_phase ^= 1u;
                        }
                        tc_fence_after();
                    }
                    const int keys = min((int)(ws & 15u) * kPage - 64 * (int)h, 64);
                    if (does_s && keys > 0) {
                        const uint32_t idS = idesc_bf16_f32(128, keys, false, false);
                        const uint64_t dk = sdesc_sw128(sSlots + ks * C::kSlotBytes + h * 8 * C::kGroupStride, 16, C::kGroupStride);
#pragma unroll
                        for (int i = 0; i < 4 * C::kSubs; ++i)
                            umma_bf16_ss(tB + h * 64, sdesc_at(dq, (i >> 2) * q_sub + (i & 3) * 32), sdesc_at(dk, (i >> 2) * 1024 + (i & 3) * 32),
                                         idS, i ? 1u : 0u);
                        umma_commit(smem_u32(&s_full[2 * set + h]));
                    }
                }
                if (!ok) break;
                if (before) {  // done with the V slot
                    if (does_p) umma_commit(smem_u32(&empty[vs]));
                    else mbar_arrive(smem_u32(&empty[vs]));
                    vs += 2;
                    if (vs >= stages) vs -= stages, v_phase ^= 1u;
                    if (wp & kLast) break;
                }
                if (more_s) {  // and with the K slot
                    if (does_s) {
                        umma_commit(smem_u32(&empty[ks]));
                        if (ws & kEnds) umma_commit(smem_u32(&q_free[set]));
                    } else {
                        mbar_arrive(smem_u32(&empty[ks]));
                    }
                    ks += 2;
                    if (ks >= stages) ks -= stages, k_phase ^= 1u;
                    wp = ws, before = true;
                    if (ws & kLast) more_s = false;
                }
            } while (true);
            umma_commit(smem_u32(mma_idle));
            mbar_drain(smem_u32(mma_idle), 0, a.status, 0x4a);
        }
        __syncwarp();
    } else if (C::kSets == 1 && warp == C::kIssuer) {
        // ------------------------------- MMA issuer at one set --------------------------------
        // A step is a key tile; step j uses score buffer j % 2, and S(j + 2) follows P V(j), which has read P
        // from that buffer (the pipe runs in order).
        if (elect_one()) {
            constexpr uint32_t idO = idesc_bf16_f32(128, C::kSlotCols, false, true);  // V is N-major
            auto wait = [&](uint64_t* bar, uint32_t phase, unsigned site) -> bool {
                return mbar_wait(smem_u32(bar), phase, abort_flag, a.status, site);
            };
            int slot = 0;  // of the ring, and its phase
            uint32_t phase = 0u;
            auto advance = [&]() {
                if (++slot == stages) slot = 0, phase ^= 1u;
            };
            uint32_t ws = 0u, wp = 0u;                        // the tiles' words
            uint32_t buf_s = 0u, buf_p = 0u, fix_phase = 0u;  // fix_phase: bits by slot
            uint32_t q_phase = 0u, o_phase = 0u, p_phase = 0u;  // p_phase: bits by buffer
            bool more_s = true, more_p = true, ok = true, o_used = false;
            auto issue_s = [&]() -> bool {
#pragma unroll 1
                for (int c = 0; c < C::kKC; ++c) {
                    if (!wait(&full[slot], phase, 0x46)) return false;
                    ws = words[slot];
                    if (c == 0 && (ws & kBegins)) {
                        if (!wait(&q_full[0], q_phase, 0x45)) return false;
                        q_phase ^= 1u;
                    }
                    tc_fence_after();
                    const uint32_t dst = tS0 + buf_s * 128, idS = idesc_bf16_f32(128, (ws & 15u) * kPage, false, false);
                    const uint64_t dk = sdesc_sw128(sSlots + slot * C::kSlotBytes, 16, C::kGroupStride);
                    const uint64_t dq = sdesc_sw128(sQ + C::kSubs * c * q_sub, 16, 1024);
#pragma unroll
                    for (int i = 0; i < 4 * C::kSubs; ++i)
                        umma_bf16_ss(dst, sdesc_at(dq, (i >> 2) * q_sub + (i & 3) * 32), sdesc_at(dk, (i >> 2) * 1024 + (i & 3) * 32), idS,
                                     (c | i) ? 1u : 0u);
                    umma_commit(smem_u32(&empty[slot]));
                    advance();
                }
                umma_commit(smem_u32(&s_full[buf_s]));
                if (ws & kEnds) umma_commit(smem_u32(&q_free[0]));
                buf_s ^= 1u;
                if (ws & kLast) more_s = false;
                return true;
            };
            auto issue_pv = [&]() -> bool {
#pragma unroll 1
                for (int c = 0; c < C::kVC; ++c) {
                    if (!wait(&full[slot], phase, 0x49)) return false;
                    wp = words[slot];
                    if (wp >> 4 & 15u) {
                        if (!wait(&vfix[slot], fix_phase >> slot & 1u, 0x4f)) return false;
                        fix_phase ^= 1u << slot;
                    }
                    if (c == 0) {
                        if (wp & kBegins) {  // the piece before has been read out of O
                            if (o_used && !wait(&o_free[0], o_phase, 0x48)) return false;
                            if (o_used) o_phase ^= 1u;
                            o_used = true;
                        }
                        if (!wait(&p_full[buf_p], p_phase >> buf_p & 1u, 0x47)) return false;
                        p_phase ^= 1u << buf_p;
                    }
                    tc_fence_after();
                    const uint64_t dv = sdesc_sw128(sSlots + slot * C::kSlotBytes, 1024, C::kGroupStride);
                    const uint32_t tP = tS0 + buf_p * 128, tD = tO + c * C::kSlotCols;
                    const int np = wp & 15u;
                    // a page of 16 keys per MMA; keys 64 h .. of P at columns 64 h ..
                    umma_bf16_ts(tD, tP, dv, idO, (wp & kBegins) ? 0u : 1u);
                    if (np == kTilePages) {
#pragma unroll
                        for (int kk = 1; kk < kTilePages; ++kk)
                            umma_bf16_ts(tD, tP + (kk >> 2) * 64 + (kk & 3) * 8, sdesc_at(dv, kk * C::kPageBytes), idO, 1u);
                    } else {
#pragma unroll 1
                        for (int kk = 1; kk < np; ++kk)
                            umma_bf16_ts(tD, tP + (kk >> 2) * 64 + (kk & 3) * 8, sdesc_at(dv, kk * C::kPageBytes), idO, 1u);
                    }
                    umma_commit(smem_u32(&empty[slot]));
                    advance();
                }
                umma_commit(smem_u32(&pv_done[buf_p]));
                buf_p ^= 1u;
                if (wp & kLast) more_p = false;
                return true;
            };
            for (int step = 0; ok && more_p; ++step) {
                if (step >= 2) ok = issue_pv();
                if (ok && more_s) ok = issue_s();
            }
            umma_commit(smem_u32(mma_idle));
            mbar_drain(smem_u32(mma_idle), 0, a.status, 0x4a);
        }
        __syncwarp();
    }
    __syncthreads();
    if (tid == 0 && works && *abort_flag) a.span[k].ctas = 0;  // a wait was given up: nothing to merge
    if (warp == C::kIssuer) {
        tc_fence_after();
        tmem_dealloc(tbase, 512);
    }
}

// Combines the partials of the segment that starts in CTA blockIdx.x of the grid above and ends in a later
// one: its own tail slot, then the head slots of the CTAs behind it. A thread owns 8 columns of a row and
// folds kFold slots at a time, their loads in flight together. (With eight at a time the registers cost more
// than the loads gain: 40.9 us against 40.2 for a batch of 64, 23.8 against 24.0 for one context of 16
// thousand keys, whose segments have 19 slots.)
constexpr int kMergeThreads = 128;
constexpr int kMergeY = 16;  // blocks of a segment, at most
constexpr int kFold = 4;

template <int D>
__global__ void __launch_bounds__(kMergeThreads) tree_merge_kernel(const __grid_constant__ TreeArgs a) {
    using C = TreeCfg<D>;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const TreeSpan sp = a.span[blockIdx.x];
    if (sp.ctas == 0) return;
    constexpr int VPR = C::kDV / 8;
    for (int it = blockIdx.y * kMergeThreads + threadIdx.x; it < (sp.rows[0] + sp.rows[1]) * VPR; it += gridDim.y * kMergeThreads) {
        const int r = it / VPR, col = it % VPR * 8;
        const int second = r >= sp.rows[0], tile_row = second ? r - sp.rows[0] : r;
        const int row = second * 128 + tile_row;  // of the partials
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
                    const float* p = a.part + ((size_t)(2 * (blockIdx.x + q * C::kSplit) + (q == 0 ? 1 : 0)) * a.rows_cap + row) * C::kRowF;
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
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const int token = sp.row0 + second * a.tokens_tile + tile_row / a.G, head = sp.head0 + tile_row % a.G;
        uint4 x;
        x.x = pack_bf16x2(O[0] * inv, O[1] * inv), x.y = pack_bf16x2(O[2] * inv, O[3] * inv);
        x.z = pack_bf16x2(O[4] * inv, O[5] * inv), x.w = pack_bf16x2(O[6] * inv, O[7] * inv);
        *reinterpret_cast<uint4*>(a.o + ((size_t)token * a.Hq + head) * D + sp.col0 + col) = x;
        if (col == 0 && sp.col0 == 0)
            a.lse[(size_t)head * a.T + token] = l == 0.f ? -INFINITY : (M + __log2f(l)) * 0.69314718055994531f;
    }
}

template <int D>
cudaError_t launch_t(const TreeLaunch& L, TreeArgs a, cudaStream_t stream) {
    using C = TreeCfg<D>;
    const int fit = (int)((C::kPool - C::kSets * a.q_rows * D * 2) / C::kSlotBytes);
    a.stages = fit < C::kMaxStages ? fit : C::kMaxStages;
    cudaError_t e = cudaFuncSetAttribute(tree_paged_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem);
    if (e != cudaSuccess) return e;
    // Bytes that a piece's partial result costs, written and read, in quarters of a key tile's; shares shorter than
    // that cost more than they gain (4 requests, window 1024, 12 to 14 drafts, 14 heads over 2, D 256: 17.5 us, and
    // 19.0 with shares of one tile).
    a.part_cost = a.rows_cap * C::kDV / (8 * (D + C::kDV));
    a.min_share = a.part_cost < 6 ? 1 : (a.part_cost + 2) / 4;
    // at most one CTA per tile of the longest step that fits the arguments
    const int tokens = a.tokens_tile * C::kSets;
    const long long groups = (L.max_q + tokens - 1) / tokens;
    const long long most = ((long long)L.max_pages + kTilePages) / kTilePages * L.R * groups * L.Hkv;
    int grid = (L.sms < kMaxGrid ? L.sms : kMaxGrid) / C::kSplit;
    if (most < grid) grid = (int)most;
    grid *= C::kSplit;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(C::kThreads);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    static const char* const kNames[4] = {"tree_paged_d64", "tree_paged_d128", "tree_paged_d256", "tree_paged_d512"};
    ProfMark m = prof_begin(stream, kNames[D == 64 ? 0 : D == 128 ? 1 : D == 256 ? 2 : 3]);
    e = cudaLaunchKernelEx(&cfg, tree_paged_kernel<D>, L.tq, L.tk, L.tv, a);
    prof_end(stream, m);
    if (e != cudaSuccess || (e = cudaGetLastError()) != cudaSuccess) return e;
    const int merge_y = (a.rows_cap * (C::kDV / 8) + kMergeThreads - 1) / kMergeThreads;
    cfg.gridDim = dim3(grid, merge_y < kMergeY ? merge_y : kMergeY);
    cfg.blockDim = dim3(kMergeThreads);
    cfg.dynamicSmemBytes = 0;
    m = prof_begin(stream, "tree_merge");
    e = cudaLaunchKernelEx(&cfg, tree_merge_kernel<D>, a);
    prof_end(stream, m);
    return e != cudaSuccess ? e : cudaGetLastError();
}

// Rows of a partial: those of one row tile, or two tiles of 128.
int rows_cap(int G, int max_q, int D) {
    const int tokens = 128 / G;
    return max_q <= tokens ? max_q * G : tree_sets(D) * 128;
}
constexpr size_t kSpanBytes = (kMaxGrid * sizeof(TreeSpan) + 255) & ~size_t(255);

}  // namespace

int tree_tokens_per_copy(int G, int max_q) { return max_q < 128 / G ? max_q : 128 / G; }

size_t tree_workspace_bytes(int G, int max_q, int D) {
    const int dv = D < 256 ? D : 256;
    return kSpanBytes + (size_t)2 * kMaxGrid * rows_cap(G, max_q, D) * (dv + 4) * 4;
}

cudaError_t launch_tree_paged(const TreeLaunch& L, cudaStream_t stream) {
    TreeArgs a;
    a.block_table = L.block_table, a.seq_lens = L.seq_lens, a.cu_q = L.cu_q, a.mask = L.mask, a.positions = L.positions;
    a.o = L.o, a.lse = L.lse, a.status = L.status;
    a.span = static_cast<TreeSpan*>(L.workspace);
    a.part = reinterpret_cast<float*>(static_cast<uint8_t*>(L.workspace) + kSpanBytes);
    a.R = L.R, a.T = L.T, a.max_q = L.max_q, a.words = L.words, a.Hq = L.Hq, a.Hkv = L.Hkv, a.G = L.Hq / L.Hkv;
    a.tokens_tile = 128 / a.G, a.rows_cap = rows_cap(a.G, L.max_q, L.D);
    a.max_pages = L.max_pages, a.num_pages = L.num_pages, a.window = L.window;
    a.scale_log2 = L.scale * 1.4426950408889634f;
    a.q_tokens = tree_tokens_per_copy(a.G, L.max_q);
    a.q_rows = (a.G * a.q_tokens + 7) / 8 * 8;
    switch (L.D) {
        case 64: return launch_t<64>(L, a, stream);
        case 128: return launch_t<128>(L, a, stream);
        case 256: return launch_t<256>(L, a, stream);
        case 512: return launch_t<512>(L, a, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace attn
