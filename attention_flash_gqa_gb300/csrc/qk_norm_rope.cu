// RMS norm of every query and key head with the rotary position encoding in the same pass: the
// step between the projections and the attention kernels, forward, gradient, and the serving form
// that writes K and V straight into the paged cache.
//
// Per row x (one head of one token, D values) with weight v = offset + w, r = rsqrt(mean(x^2) + eps):
//     xh = r x,   n = v xh,   y = R n
// R turns the pairs of the first `rot` dims by the token's angles (cos and sin from a table of the
// caller's): (a, b) -> (a cos - b sin, b cos + a sin), pairs (i, i + rot/2) or, interleaved,
// (2i, 2i + 1). The gradient, for dy:
//     dn = R^T dy,   dw = sum over rows of dn xh,   g = v dn,   dx = r (g - xh mean(g xh))
// All of it is evaluated in fp32 from the bf16 inputs; the results round once to bf16 (dw stays fp32).
//
// Memory bound: a row is read once and written once (gradient: x and dy in, dx out). A thread owns
// 16 dims of a row as two 16-byte chunks chosen so that both members of every rotated pair are its
// own: chunks (j, j + rot/16) for j < rot/16, else (2j, 2j + 1); interleaved, always (2j, 2j + 1).
// Either way its angles are 8j .. 8j + 7. D / 16 lanes share a row, so a warp takes 512 / D rows at a
// time and the only exchange is the butterfly sum of a row's lanes. A task is one token's block of
// kU such passes, all queries or all keys; a warp keeps its block and walks the tokens, so the norm
// weights (and, in the gradient, their sums) stay in registers and a token's angles are loaded once
// for kU passes. All loads of a task are issued before the first is used; in the gradient, and in long calls
// of the paged form, they come through rings in shared memory (see there).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "attn_internal.h"
#include "ptx.cuh"

namespace attn {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kUF = 4;  // passes per task, forward (1 where heads are few: see launch_fwd_d)
constexpr int kUB = 4;  // passes per task, gradient
constexpr int kMaxCtas = 1024;  // sizes the gradient's workspace

__device__ __forceinline__ void unpack8(const uint4& w, float (&x)[16], int at) {
    const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        x[at + 2 * e] = __uint_as_float(v[e] << 16);
        x[at + 2 * e + 1] = __uint_as_float(v[e] & 0xffff0000u);
    }
}
__device__ __forceinline__ uint4 pack8(const float (&x)[16], int at) {
    uint4 w;
    w.x = pack_bf16x2(x[at], x[at + 1]), w.y = pack_bf16x2(x[at + 2], x[at + 3]);
    w.z = pack_bf16x2(x[at + 4], x[at + 5]), w.w = pack_bf16x2(x[at + 6], x[at + 7]);
    return w;
}

// The LPR lanes that share row group `sub`, and a sum over them.
template <int LPR>
__device__ __forceinline__ unsigned row_peers(int sub) {
    return LPR == 32 ? 0xffffffffu : ((1u << (LPR & 31)) - 1u) << (sub * LPR & 31);
}
template <int LPR>
__device__ __forceinline__ float row_sum(float v, unsigned peers = 0xffffffffu) {
#pragma unroll
    for (int off = LPR / 2; off; off >>= 1) v += __shfl_xor_sync(peers, v, off);
    return v;
}

// The rotation of a thread's 16 dims (sin negated: its transpose).
__device__ __forceinline__ void turn(float (&x)[16], const float (&c)[8], const float (&s)[8], bool inter) {
    if (inter) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float a = x[2 * e], b = x[2 * e + 1];
            x[2 * e] = a * c[e] - b * s[e], x[2 * e + 1] = b * c[e] + a * s[e];
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float a = x[e], b = x[8 + e];
            x[e] = a * c[e] - b * s[e], x[8 + e] = b * c[e] + a * s[e];
        }
    }
}

// What a warp works on: block `blk` of every token it walks.
struct Block {
    int kind;   // 0: queries, 1: keys, 2: values (paged form)
    int head0;  // first head
    int heads;  // heads of that kind
    int rows;   // heads of the block
};
// RPT: rows (heads) per task, at most. EVEN: the blocks of a kind get the same number of heads, to one, instead of
// a last one with what is left (gradient, 6666 tokens, 24 + 4 heads of 128: 31.5 us against 35.9; 5664 tokens, 5 +
// 5 heads of 512: 39.5 against 43.8; the forward, whose loads go to registers, gains nothing by it).
template <int RPT, bool EVEN = false>
__device__ __forceinline__ Block block_of(int blk, int Hq, int Hkv) {
    const int nq = (Hq + RPT - 1) / RPT, nk = (Hkv + RPT - 1) / RPT;
    const int rq = EVEN ? (Hq + nq - 1) / nq : RPT, rk = EVEN ? (Hkv + nk - 1) / nk : RPT;
    if (blk < nq) return {0, blk * rq, Hq, min(rq, Hq - blk * rq)};
    if (blk < nq + nk) return {1, (blk - nq) * rk, Hkv, min(rk, Hkv - (blk - nq) * rk)};
    return {2, (blk - nq - nk) * rk, Hkv, min(rk, Hkv - (blk - nq - nk) * rk)};
}

// A thread's 16 effective weights, offset + w (1 without weights).
__device__ __forceinline__ void load_weights(const NormRopeLaunch& a, const void* w, int c0, int c1, float (&v)[16]) {
#pragma unroll
    for (int e = 0; e < 16; ++e) {
        const int d = (e < 8 ? 8 * c0 : 8 * c1) + (e & 7);
        if (!w) v[e] = 1.f;
        else if (a.weight_fp32) v[e] = a.weight_offset + static_cast<const float*>(w)[d];
        else v[e] = a.weight_offset + __uint_as_float((uint32_t) static_cast<const uint16_t*>(w)[d] << 16);
    }
}

__device__ __forceinline__ void load_angles(const NormRopeLaunch& a, int pos, int j, float (&c)[8], float (&s)[8]) {
    const float* row = a.cos_sin + (size_t)pos * a.rot + 8 * j;
#pragma unroll
    for (int e = 0; e < 8; e += 4) {
        const float4 x = __ldg(reinterpret_cast<const float4*>(row + e));
        const float4 y = __ldg(reinterpret_cast<const float4*>(row + a.rot / 2 + e));
        c[e] = x.x, c[e + 1] = x.y, c[e + 2] = x.z, c[e + 3] = x.w;
        s[e] = y.x, s[e + 1] = y.y, s[e + 2] = y.z, s[e + 3] = y.w;
    }
}

template <int D, bool PAGED, int U>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(const __grid_constant__ NormRopeLaunch a) {
    constexpr int LPR = D / 16, RPW = 32 / LPR, RPT = RPW * U;
    griddep_wait();
    const int lane = threadIdx.x & 31, j = lane % LPR, sub = lane / LPR;
    const int nblk = (a.Hq + RPT - 1) / RPT + (PAGED ? 2 : 1) * ((a.Hkv + RPT - 1) / RPT);
    const int warp = blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int lanes = gridDim.x * kWarps / nblk;  // token lanes: a warp takes tokens warp / nblk + i * lanes
    if (warp >= lanes * nblk) return;
    const Block b = block_of<RPT>(warp % nblk, a.Hq, a.Hkv);
    const int rc = a.rot / 16;  // lanes whose dims are rotated
    const bool rotated = j < rc;
    const int c0 = rotated && !a.interleaved ? j : 2 * j, c1 = rotated && !a.interleaved ? j + rc : 2 * j + 1;
    float v[16];
    if (b.kind < 2) load_weights(a, b.kind == 0 ? a.q_weight : a.k_weight, c0, c1, v);
    const uint16_t* src = b.kind == 0 ? a.q : b.kind == 1 ? a.k : a.v;
    const long long stride = b.kind == 0 ? a.q_stride : b.kind == 1 ? a.k_stride : a.v_stride;
    uint16_t* dst = b.kind == 0 ? a.q_out : b.kind == 1 ? a.k_out : a.v_out;

    for (int t = warp / nblk; t < a.T; t += lanes) {
        long long orow = t;  // output row: the token, or its cache slot
        if (PAGED) {
            const int slot = a.slots[t];
            if (slot == -1) continue;  // a padding row
            if (slot < 0 || slot >= a.num_slots) {
                if (lane == 0) atomicOr(a.status, DEVSTAT_BOUNDS);
                continue;
            }
            if (b.kind) orow = slot;
        }
        uint4 raw[U][2];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int h = b.head0 + u * RPW + sub;
            if (h < b.heads) {
                const uint16_t* row = src + (size_t)t * stride + (size_t)h * D;
                raw[u][0] = *reinterpret_cast<const uint4*>(row + 8 * c0);
                raw[u][1] = *reinterpret_cast<const uint4*>(row + 8 * c1);
            } else {
                raw[u][0] = raw[u][1] = make_uint4(0u, 0u, 0u, 0u);
            }
        }
        float c[8], s[8];
        if (a.rot > 0) {
            const int pos = a.positions[t];
            if (pos < 0 || pos >= a.max_pos) {
                if (lane == 0) atomicOr(a.status, DEVSTAT_BOUNDS);
                continue;
            }
            if (rotated && b.kind < 2) load_angles(a, pos, j, c, s);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int h = b.head0 + u * RPW + sub;
            if (b.kind < 2) {
                float x[16];
                unpack8(raw[u][0], x, 0);
                unpack8(raw[u][1], x, 8);
                float ss = 0.f;
#pragma unroll
                for (int e = 0; e < 16; ++e) ss = fmaf(x[e], x[e], ss);
                const float r = rsqrtf(row_sum<LPR>(ss) * (1.f / D) + a.eps);
#pragma unroll
                for (int e = 0; e < 16; ++e) x[e] = x[e] * r * v[e];
                if (rotated) turn(x, c, s, a.interleaved);
                raw[u][0] = pack8(x, 0);
                raw[u][1] = pack8(x, 8);
            }
            if (h < b.heads) {
                uint16_t* row = dst + ((size_t)orow * b.heads + h) * D;
                *reinterpret_cast<uint4*>(row + 8 * c0) = raw[u][0];
                *reinterpret_cast<uint4*>(row + 8 * c1) = raw[u][1];
            }
        }
    }
}

// The gradient. The rows of a task come into shared memory by bulk copies, 4 KB of x and 4 KB of dy, into a
// ring of kRing stages that each warp has for itself: its lane 0 refills a stage as soon as the warp has
// read it, so 12 warps an SM keep up to 192 KB on their way (with loads into registers, 163 of them and
// 48 KB on their way, 18001 tokens of 36 heads of 512 took 487 us, 4.1 TB/s; now 294 us, 6.8 TB/s). At D = 512
// tasks of fewer rows get more, smaller stages (5664 tokens, 5 + 5 heads: 38.5 us against 39.6, and the loop with
// a variable depth is compiled to 167 registers instead of 128: 294 us against 312 for the 36 heads); at D <= 256
// deeper rings cost up to 8 %. Each CTA leaves its sums of dn xh in part[CTA][query | key][D], in an order of its
// own that depends on the launch alone; norm_rope_dw_kernel adds them up.
constexpr int kRing = 2;
constexpr int kStageBytes = 8192;
constexpr int kMaxRing = 8;  // D = 512
constexpr int kBwdSmem = kWarps * kRing * kStageBytes + kWarps * kMaxRing * 8 + 64;

template <int D>
__global__ void __launch_bounds__(kThreads) norm_rope_bwd_kernel(const __grid_constant__ NormRopeLaunch a) {
    constexpr int LPR = D / 16, RPW = 32 / LPR, RPT = RPW * kUB;
    static_assert(RPT * D * 4 == kStageBytes, "a stage holds a task's x and dy");
    extern __shared__ __align__(128) uint8_t ring[];
    uint64_t* bars = reinterpret_cast<uint64_t*>(ring + kWarps * kRing * kStageBytes);  // [kWarps][kMaxRing]
    volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + kWarps * kMaxRing);
    const int lane = threadIdx.x & 31, j = lane % LPR, sub = lane / LPR, wid = threadIdx.x >> 5;
    const int nblk = (a.Hq + RPT - 1) / RPT + (a.Hkv + RPT - 1) / RPT;
    const int warp = blockIdx.x * kWarps + wid;
    const int lanes = gridDim.x * kWarps / nblk;
    const bool works = warp < lanes * nblk;
    const Block b = block_of<RPT, true>(warp % nblk, a.Hq, a.Hkv);
    const int rc = a.rot / 16;
    const bool rotated = j < rc;
    const int c0 = rotated && !a.interleaved ? j : 2 * j, c1 = rotated && !a.interleaved ? j + rc : 2 * j + 1;
    griddep_wait();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // norm_rope_dw_kernel waits for this grid
    const uint16_t* src = (b.kind == 0 ? a.q : a.k) + (size_t)b.head0 * D;
    const uint16_t* gsrc = (b.kind == 0 ? a.dq_out : a.dk_out) + (size_t)b.head0 * D;
    const long long stride = b.kind == 0 ? a.q_stride : a.k_stride;
    const long long ostride = b.kind == 0 ? a.dq_stride : a.dk_stride;
    uint16_t* dst = (b.kind == 0 ? a.dq : a.dk) + (size_t)b.head0 * D;
    const int rows = b.rows;
    uint8_t* mine = ring + wid * kRing * kStageBytes;
    uint64_t* full = bars + wid * kMaxRing;
    const uint32_t bytes = rows * D * 2;  // of x, and of dy; a stage holds both
    const int depth = D == 512 ? min(kMaxRing, (int)(kRing * kStageBytes / (2 * bytes))) : kRing;
    if (threadIdx.x == 0) *abort_flag = 0;
    if (lane == 0)
        for (int s = 0; s < kMaxRing; ++s) mbar_init(smem_u32(&full[s]), 1);
    fence_mbar_init();
    __syncthreads();
    auto fetch = [&](int t, int s) {  // lane 0
        const uint32_t bar = smem_u32(&full[s]), at = smem_u32(mine + s * 2 * bytes);
        mbar_expect_tx(bar, 2 * bytes);
        bulk_load(at, src + (size_t)t * stride, bytes, bar);
        bulk_load(at + bytes, gsrc + (size_t)t * b.heads * D, bytes, bar);
    };
    const int t0 = warp / nblk;
    if (works && lane == 0)
        for (int s = 0; s < depth; ++s)
            if (t0 + (long long)s * lanes < a.T) fetch(t0 + s * lanes, s);
    float v[16], dw[16];
    load_weights(a, b.kind == 0 ? a.q_weight : a.k_weight, c0, c1, v);
#pragma unroll
    for (int e = 0; e < 16; ++e) dw[e] = 0.f;

    int stage = 0, phase = 0;
    for (int t = t0; works && t < a.T; t += lanes) {
        bool skip = false;
        float c[8], s[8];
        if (a.rot > 0) {
            const int pos = a.positions[t];
            skip = pos < 0 || pos >= a.max_pos;
            if (skip) {
                if (lane == 0) atomicOr(a.status, DEVSTAT_BOUNDS);
            } else if (rotated) {
                load_angles(a, pos, j, c, s);
#pragma unroll
                for (int e = 0; e < 8; ++e) s[e] = -s[e];  // the transpose
            }
        }
        if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&full[stage]), phase, abort_flag, a.status, 0x51))) {
            // given up: the CTA outlasts the copies that this warp has on their way
            if (lane == 0) ring_drain(full, stage, phase, depth, ((long long)a.T - t + lanes - 1) / lanes, a.status, 0x53);
            __syncwarp();
            break;
        }
        const uint8_t* xs = mine + stage * 2 * bytes;
#pragma unroll
        for (int u = 0; u < kUB; ++u) {
            const int r = u * RPW + sub;
            if (skip || r >= rows) continue;  // a row's lanes agree
            float x[16], g[16];
            const uint8_t* xrow = xs + r * D * 2;
            unpack8(*reinterpret_cast<const uint4*>(xrow + 16 * c0), x, 0);
            unpack8(*reinterpret_cast<const uint4*>(xrow + 16 * c1), x, 8);
            unpack8(*reinterpret_cast<const uint4*>(xrow + bytes + 16 * c0), g, 0);
            unpack8(*reinterpret_cast<const uint4*>(xrow + bytes + 16 * c1), g, 8);
            if (rotated) turn(g, c, s, a.interleaved);  // dn
            float ss = 0.f, sg = 0.f;
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                ss = fmaf(x[e], x[e], ss);
                sg = fmaf(g[e] * v[e], x[e], sg);
            }
            const unsigned peers = row_peers<LPR>(sub);
            const float rr = rsqrtf(row_sum<LPR>(ss, peers) * (1.f / D) + a.eps);
            const float m = row_sum<LPR>(sg, peers) * (1.f / D) * rr;  // mean(g xh)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const float xh = x[e] * rr;
                dw[e] = fmaf(g[e], xh, dw[e]);
                x[e] = rr * (g[e] * v[e] - xh * m);
            }
            uint16_t* row = dst + (size_t)t * ostride + (size_t)r * D;
            *reinterpret_cast<uint4*>(row + 8 * c0) = pack8(x, 0);
            *reinterpret_cast<uint4*>(row + 8 * c1) = pack8(x, 8);
        }
        __syncwarp();  // the stage has been read
        if (lane == 0 && t + (long long)depth * lanes < a.T) fetch(t + depth * lanes, stage);
        if (++stage == depth) stage = 0, phase ^= 1;
    }
    // the warp's row groups, then the CTA's warps, in order
    __shared__ float sums[kWarps][D];
    __shared__ int kinds[kWarps];
#pragma unroll
    for (int e = 0; e < 16; ++e)
#pragma unroll
        for (int off = LPR; off < 32; off <<= 1) dw[e] += __shfl_xor_sync(0xffffffffu, dw[e], off);
    if (sub == 0) {
#pragma unroll
        for (int e = 0; e < 16; ++e) sums[wid][(e < 8 ? 8 * c0 : 8 * c1) + (e & 7)] = dw[e];
    }
    if (lane == 0) kinds[wid] = works ? b.kind : -1;
    __syncthreads();
    float* part = a.part + (size_t)blockIdx.x * 2 * D;
    for (int i = threadIdx.x; i < 2 * D; i += kThreads) {
        float acc = *abort_flag ? NAN : 0.f;  // a wait was given up: the sums lack rows, and say so
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
            if (kinds[w] == i / D) acc += sums[w][i % D];
        part[i] = acc;
    }
}

// dw[i] = sum over the CTAs of part[CTA][i]: 32 columns a CTA, its warps take every kDwWarps-th partial.
constexpr int kDwWarps = 16;
__global__ void __launch_bounds__(kDwWarps * 32) norm_rope_dw_kernel(const float* part, float* dqw, float* dkw, int D, int n) {
    __shared__ float acc[kDwWarps][32];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, col = blockIdx.x * 32 + lane;
    griddep_wait();  // launched while the gradient kernel runs
    float x = 0.f;
    for (int i = w; i < n; i += kDwWarps) x += part[(size_t)i * 2 * D + col];
    acc[w][lane] = x;
    __syncthreads();
    if (w == 0) {
        x = 0.f;
#pragma unroll
        for (int i = 0; i < kDwWarps; ++i) x += acc[i][lane];
        float* out = col < D ? dqw : dkw;
        if (out) out[col < D ? col : col - D] = x;
    }
}

// The paged form of long calls, with its rows in rings like the gradient's: 4 KB a stage, two stages a warp, five
// CTAs an SM (8468 tokens, 10 + 2 + 2 heads of 512: 41.4 us against 53.9 with loads into registers; 12590 tokens,
// 30 + 15 + 15 of 64: 34.9 against 43.7; 4096 tokens, 32 + 4 + 4 of 512: 55.4 against 57.7). The form that is not
// paged has none, and is better off without for long calls alone: 16384 tokens, 32 + 16 heads of 256, 125 us against
// 138 to 142 with rings. Of the calls of 10 to 80 us most would gain a little (5749 tokens, 32 + 8 heads of 128: 24.6 us,
// 22.4 with rings of two stages and four CTAs an SM; 2637, 50 + 10 of 64: 11.3, 10.6; 1197, 30 + 10 of 512: 21.5, 20.4;
// 2470, 80 + 16 of 512: 78.9, 76.6; 421, 45 + 15 of 512: 12.5, 12.5), short ones lose up to 8 %. What makes the first
// one lose is not known, so there is no rule to choose by yet.
constexpr int kFwdRing = 2;
constexpr int kFwdStage = 4096;
constexpr int kFwdSmem = kWarps * kFwdRing * kFwdStage + kWarps * kFwdRing * 8 + 64;

template <int D>
__global__ void __launch_bounds__(kThreads) norm_rope_ring_kernel(const __grid_constant__ NormRopeLaunch a) {
    constexpr int LPR = D / 16, RPW = 32 / LPR, RPT = RPW * kUF;
    static_assert(RPT * D * 2 == kFwdStage, "a stage holds a task's rows");
    extern __shared__ __align__(128) uint8_t ring[];
    uint64_t* bars = reinterpret_cast<uint64_t*>(ring + kWarps * kFwdRing * kFwdStage);  // [kWarps][kFwdRing]
    volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + kWarps * kFwdRing);
    griddep_wait();
    const int lane = threadIdx.x & 31, j = lane % LPR, sub = lane / LPR, wid = threadIdx.x >> 5;
    const int nblk = (a.Hq + RPT - 1) / RPT + 2 * ((a.Hkv + RPT - 1) / RPT);
    const int warp = blockIdx.x * kWarps + wid;
    const int lanes = gridDim.x * kWarps / nblk;
    const bool works = warp < lanes * nblk;
    const Block b = block_of<RPT, true>(warp % nblk, a.Hq, a.Hkv);
    const int rc = a.rot / 16;
    const bool rotated = j < rc;
    const int c0 = rotated && !a.interleaved ? j : 2 * j, c1 = rotated && !a.interleaved ? j + rc : 2 * j + 1;
    const uint16_t* src = (b.kind == 0 ? a.q : b.kind == 1 ? a.k : a.v) + (size_t)b.head0 * D;
    const long long stride = b.kind == 0 ? a.q_stride : b.kind == 1 ? a.k_stride : a.v_stride;
    uint16_t* dst = (b.kind == 0 ? a.q_out : b.kind == 1 ? a.k_out : a.v_out) + (size_t)b.head0 * D;
    uint8_t* mine = ring + wid * kFwdRing * kFwdStage;
    uint64_t* full = bars + wid * kFwdRing;
    const uint32_t bytes = b.rows * D * 2;
    if (threadIdx.x == 0) *abort_flag = 0;
    if (lane == 0)
        for (int s = 0; s < kFwdRing; ++s) mbar_init(smem_u32(&full[s]), 1);
    fence_mbar_init();
    __syncthreads();
    if (!works) return;
    auto fetch = [&](int t, int s) {  // lane 0
        const uint32_t bar = smem_u32(&full[s]);
        mbar_expect_tx(bar, bytes);
        bulk_load(smem_u32(mine + s * kFwdStage), src + (size_t)t * stride, bytes, bar);
    };
    const int t0 = warp / nblk;
    if (lane == 0)
        for (int s = 0; s < kFwdRing; ++s)
            if (t0 + (long long)s * lanes < a.T) fetch(t0 + s * lanes, s);
    float v[16];
    if (b.kind < 2) load_weights(a, b.kind == 0 ? a.q_weight : a.k_weight, c0, c1, v);
    int stage = 0, phase = 0;
    for (int t = t0; t < a.T; t += lanes) {
        const int slot = a.slots[t];
        const size_t orow = b.kind ? slot : t;  // output row: the token, or its cache slot
        bool skip = slot == -1;                 // a padding row
        bool bad = !skip && (slot < 0 || slot >= a.num_slots);
        float c[8], s[8];
        if (a.rot > 0) {
            const int pos = a.positions[t];
            if (!skip) bad |= pos < 0 || pos >= a.max_pos;
            if (!skip && !bad && rotated && b.kind < 2) load_angles(a, pos, j, c, s);
        }
        if (bad) {
            skip = true;
            if (lane == 0) atomicOr(a.status, DEVSTAT_BOUNDS);
        }
        if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&full[stage]), phase, abort_flag, a.status, 0x52))) {
            // given up: the CTA outlasts the copies that this warp has on their way
            if (lane == 0) ring_drain(full, stage, phase, kFwdRing, ((long long)a.T - t + lanes - 1) / lanes, a.status, 0x54);
            __syncwarp();
            break;
        }
        const uint8_t* xs = mine + stage * kFwdStage;
#pragma unroll
        for (int u = 0; u < kUF; ++u) {
            const int r = u * RPW + sub;
            if (skip || r >= b.rows) continue;  // a row's lanes agree
            uint4 lo = *reinterpret_cast<const uint4*>(xs + r * D * 2 + 16 * c0), hi = *reinterpret_cast<const uint4*>(xs + r * D * 2 + 16 * c1);
            if (b.kind < 2) {
                float x[16];
                unpack8(lo, x, 0);
                unpack8(hi, x, 8);
                float ss = 0.f;
#pragma unroll
                for (int e = 0; e < 16; ++e) ss = fmaf(x[e], x[e], ss);
                const float rr = rsqrtf(row_sum<LPR>(ss, row_peers<LPR>(sub)) * (1.f / D) + a.eps);
#pragma unroll
                for (int e = 0; e < 16; ++e) x[e] = x[e] * rr * v[e];
                if (rotated) turn(x, c, s, a.interleaved);
                lo = pack8(x, 0);
                hi = pack8(x, 8);
            }
            uint16_t* row = dst + (orow * b.heads + r) * D;
            *reinterpret_cast<uint4*>(row + 8 * c0) = lo;
            *reinterpret_cast<uint4*>(row + 8 * c1) = hi;
        }
        __syncwarp();  // the stage has been read
        if (lane == 0 && t + (long long)kFwdRing * lanes < a.T) fetch(t + kFwdRing * lanes, stage);
        if (++stage == kFwdRing) stage = 0, phase ^= 1;
    }
}

// CTAs for `tasks` warp tasks: enough for all of them at once, at most `per_sm` per SM, and at least one
// warp for each block of a token.
int norm_grid(long long T, int nblk, int sms, int per_sm) {
    const long long want = (T * nblk + kWarps - 1) / kWarps, least = (nblk + kWarps - 1) / kWarps;
    long long g = (long long)sms * per_sm;
    if (want < g) g = want;
    if (g < least) g = least;  // at most 2048 heads of each kind: 4096 / kWarps
    return (int)g;
}

constexpr int kRingPerSm = 5;
constexpr int kFwdPerSm = 4, kFewPerSm = 12, kBwdPerSm = 3;
constexpr int kMaxSms = kMaxCtas / kBwdPerSm;  // more of them are not used by the gradient

// A launch with programmatic serialisation: its CTAs may start while the kernel in front ends, and wait for it
// (griddep_wait) before they read or write anything.
template <class... Params, class... Args>
cudaError_t launch_early(void (*kernel)(Params...), int grid, int threads, int smem, cudaStream_t stream, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, Params(args)...);
}

template <int D, bool PAGED, int U>
cudaError_t launch_fwd_u(const NormRopeLaunch& L, int per_sm, cudaStream_t stream) {
    constexpr int RPT = 512 / D * U;
    const int nblk = (L.Hq + RPT - 1) / RPT + (PAGED ? 2 : 1) * ((L.Hkv + RPT - 1) / RPT);
    const ProfMark m = prof_begin(stream, PAGED ? "qk_norm_rope_paged" : "qk_norm_rope");
    const cudaError_t e = launch_early(norm_rope_kernel<D, PAGED, U>, norm_grid(L.T, nblk, L.sms, per_sm), kThreads, 0, stream, L);
    prof_end(stream, m);
    return e != cudaSuccess ? e : cudaGetLastError();
}

// A task has four passes and an SM four CTAs, whose loads are all in flight; but where the heads leave most of a
// task's rows empty, tasks of one pass, and twelve CTAs an SM, have more of them on their way (17030 tokens, 3 + 3
// heads of 64: 11.6 us against 28.3; 36190 tokens, 8 + 2 + 2 heads of 128 into the cache: 57 against 98; 333 tokens, 12
// + 3 heads of 64: 2.6 against 3.3). Where more than half of the rows are there it is the other way round (11076
// tokens, 10 + 5 + 5 heads of 256: 60 against 53; 16384 tokens, 32 + 16 heads of 256: 158 against 125), and where the
// tasks of four passes come to about one a warp (921 tokens, 15 + 15 + 15 heads of 64: 6.0 against 5.2).
template <int D, bool PAGED>
cudaError_t launch_fwd_d(const NormRopeLaunch& L, cudaStream_t stream) {
    constexpr int RPW = 512 / D, RPT = RPW * kUF, kinds = PAGED ? 2 : 1;
    const int nblk = (L.Hq + RPT - 1) / RPT + kinds * ((L.Hkv + RPT - 1) / RPT);
    const long long tasks = (long long)L.T * nblk, warps = (long long)L.sms * kFwdPerSm * kWarps;
    if (L.Hq + kinds * L.Hkv <= nblk * RPT / 2 && (tasks <= warps / 2 || tasks > 2 * warps))
        return launch_fwd_u<D, PAGED, 1>(L, kFewPerSm, stream);
    if constexpr (PAGED) {
        if (tasks > 3 * warps) {  // (418 tokens, 96 + 16 + 16 heads of 256, 2.8 tasks a warp: 14.3 us in rings, 13.0 not)
            cudaError_t e = cudaFuncSetAttribute(norm_rope_ring_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, kFwdSmem);
            if (e != cudaSuccess) return e;
            const ProfMark m = prof_begin(stream, "qk_norm_rope_paged");
            e = launch_early(norm_rope_ring_kernel<D>, norm_grid(L.T, nblk, L.sms, kRingPerSm), kThreads, kFwdSmem, stream, L);
            prof_end(stream, m);
            return e != cudaSuccess ? e : cudaGetLastError();
        }
    }
    return launch_fwd_u<D, PAGED, kUF>(L, kFwdPerSm, stream);
}

template <int D>
cudaError_t launch_bwd_d(const NormRopeLaunch& L, cudaStream_t stream) {
    constexpr int RPT = 512 / D * kUB;
    const int nblk = (L.Hq + RPT - 1) / RPT + (L.Hkv + RPT - 1) / RPT;
    const int grid = norm_grid(L.T, nblk, L.sms < kMaxSms ? L.sms : kMaxSms, kBwdPerSm);
    cudaError_t e = cudaFuncSetAttribute(norm_rope_bwd_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, kBwdSmem);
    if (e != cudaSuccess) return e;
    ProfMark m = prof_begin(stream, "qk_norm_rope_bwd");
    e = launch_early(norm_rope_bwd_kernel<D>, grid, kThreads, kBwdSmem, stream, L);
    prof_end(stream, m);
    if (e != cudaSuccess || (e = cudaGetLastError()) != cudaSuccess) return e;
    m = prof_begin(stream, "qk_norm_rope_dw");
    e = launch_early(norm_rope_dw_kernel, 2 * D / 32, kDwWarps * 32, 0, stream, (const float*)L.part, L.dq_weight, L.dk_weight, D, grid);
    prof_end(stream, m);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

int norm_rope_bwd_max_ctas() { return kMaxCtas; }

cudaError_t launch_norm_rope(const NormRopeLaunch& L, cudaStream_t stream) {
    switch (L.D) {
        case 64: return launch_fwd_d<64, false>(L, stream);
        case 128: return launch_fwd_d<128, false>(L, stream);
        case 256: return launch_fwd_d<256, false>(L, stream);
        case 512: return launch_fwd_d<512, false>(L, stream);
        default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_norm_rope_paged(const NormRopeLaunch& L, cudaStream_t stream) {
    switch (L.D) {
        case 64: return launch_fwd_d<64, true>(L, stream);
        case 128: return launch_fwd_d<128, true>(L, stream);
        case 256: return launch_fwd_d<256, true>(L, stream);
        case 512: return launch_fwd_d<512, true>(L, stream);
        default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_norm_rope_bwd(const NormRopeLaunch& L, cudaStream_t stream) {
    switch (L.D) {
        case 64: return launch_bwd_d<64>(L, stream);
        case 128: return launch_bwd_d<128>(L, stream);
        case 256: return launch_bwd_d<256>(L, stream);
        case 512: return launch_bwd_d<512>(L, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace attn
