// Sinks in the backward (attn_internal.h, SinkSplit): the far queries' share where the sinks are few, and the sum of all parts.
#include <cuda_runtime.h>

#include "attn_internal.h"
#include "ptx.cuh"

namespace attn {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

// bwd_far_sink_kernel: a far query sees of key tile 0 its sinks alone, at most 16 of the tile's 128 keys. As a step of the main
// kernel that is five products of 128 x 128 x D for an eighth or less of their use (and 16384 fp32 reductions into dQ a step); here
// it rides on the pass that makes Delta anyway. That pass reads o and dO; with q besides it has all that the sinks' terms
// take, and instead of zeros it leaves their dQ in the accumulator:
//   S^T = K Q^T, dP^T = V dO^T (16 keys x 16 rows a warp, by k = D), Delta = rowsum(dO o), P^T = exp2(S^T - lse),
//   dS^T = P^T (dP^T - Delta), dQ = dS K to the accumulator, dV += P^T dO, dK += dS^T Q.
// So it is bound by memory: 6 bytes read and 4 written an element of q (the pass without q and sums: 4 and 4). At B = 2, S = 8192, 32 heads of
// 256, window 1024: 203 us for 1.15 GB, 0.83 of the copy rate, where the slices in the main kernel take 260 and the pass 128 more.
// A block has a slice of queries and the query heads of one KV head or a share of them, 64 rows a step, copied to shared memory by cp.async (chunks of
// 16 bytes at chunk ^ row % 8, so that the matrix loads touch every bank once). A warp has 16 of the rows for S, dP and dQ,
// then all 64 rows and a quarter of the dims for dV and dK, which stay in registers over the slice. P and dS are rounded to bf16 for their
// products, as in the main kernel (dS from P in fp32).
constexpr int kRows = 64, kWarps = 4, kThreads = 32 * kWarps;

template <int D>
struct FarCfg {
    static constexpr int kRowBytes = 2 * D;
    static constexpr int kTile = kRows * kRowBytes;
    static constexpr int kKeys = kFewSinks * kRowBytes;
    static constexpr int kStages = D == 256 ? 1 : 2;  // of q and dO: at head_dim 256 a second one would leave room for one block an SM
    static constexpr int kOffDO = kTile, kOffK = kStages * 2 * kTile, kOffV = kOffK + kKeys, kOffP = kOffV + kKeys;
    static constexpr int kOffDS = kOffP + kWarps * 512;  // A operands of a k-step, 16 bytes a lane
    static constexpr int kSmem = kOffDS + kWarps * 512;
    // blocks of an SM: as many as shared memory holds, up to 4 (128 registers a thread)
    static constexpr int kResident = 232448 / (kSmem + 1024) < 4 ? 232448 / (kSmem + 1024) : 4;
};

struct FarArgs {
    const uint16_t *q, *k, *v, *o, *dO;
    const float* lse;
    float *delta, *dq_acc;
    const int32_t* cu;
    int Hq, Hkv, S, T, window;
    float scale, scale_log2;
    SinkSplit sink;
};

// 16 bytes to shared memory, or zeros.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {  // all but the last N groups
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <int D>
__global__ void __launch_bounds__(kThreads, FarCfg<D>::kResident) bwd_far_sink_kernel(FarArgs a) {
    using C = FarCfg<D>;
    constexpr int kChunks = D / 8, kMine = D / kWarps / 8;  // chunks of 16 bytes of a row; n-tiles of 8 dims of a warp's quarter
    griddep_wait();
    extern __shared__ __align__(1024) uint8_t smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
    const int hk = blockIdx.y, seq = blockIdx.z;
    int start = seq * a.S, L = a.S;
    if (a.cu) {
        start = a.cu[seq], L = a.cu[seq + 1] - start;
        if (!varlen_seq_ok(start, L, a.T, a.S)) return;  // (reported by the main kernel)
    }
    const int slice = blockIdx.x / a.sink.shares, share = blockIdx.x - slice * a.sink.shares;
    const int r_begin = far_from(L, a.window) + slice * a.sink.rows, r_end = min(r_begin + a.sink.rows, L);
    if (r_begin >= L) return;
    // query heads of this block
    const int h0 = hk * (a.Hq / a.Hkv) + a.Hq / a.Hkv * share / a.sink.shares, heads = hk * (a.Hq / a.Hkv) + a.Hq / a.Hkv * (share + 1) / a.sink.shares - h0;
    const uint32_t sTiles = smem_u32(smem), sK = sTiles + C::kOffK, sV = sTiles + C::kOffV;
    uint4* pf = reinterpret_cast<uint4*>(smem + C::kOffP);
    uint4* df = reinterpret_cast<uint4*>(smem + C::kOffDS);
    // chunk `ch` of row r
    auto at = [](uint32_t base, int r, int ch) { return base + r * C::kRowBytes + ((ch ^ (r & 7)) << 4); };
    for (int x = tid; x < kFewSinks * kChunks; x += kThreads) {
        const int j = x / kChunks, ch = x % kChunks;
        const size_t src = ((size_t)(start + j) * a.Hkv + hk) * D + 8 * ch;  // (far queries: the sequence has more than 128 keys)
        copy16(at(sK, j, ch), a.k + src, j < a.sink.sink);
        copy16(at(sV, j, ch), a.v + src, j < a.sink.sink);
    }
    float dv[kMine][4] = {}, dk[kMine][4] = {};
    // matrix loads of a 16 x 16 block: lane's row within it and chunk of its two
    const int mr = lane & 15, mc = lane >> 4;
    // steps: query heads, and of each the slice's rows 64 at a time
    const int nr = (r_end - r_begin + kRows - 1) / kRows, n = heads * nr;
    const size_t pitch = (size_t)a.Hq * D;
    auto row_of = [&](int step) { return r_begin + step % nr * kRows; };
    auto base_of = [&](int step) { return ((size_t)(start + row_of(step)) * a.Hq + h0 + step / nr) * D; };
    auto load = [&](int step) {
        const int rows = r_end - row_of(step);
        const size_t base = base_of(step);
        const uint32_t dst = sTiles + step % C::kStages * (2 * C::kTile);
#pragma unroll 4
        for (int x = tid; x < kRows * kChunks; x += kThreads) {
            const int r = x / kChunks, ch = x % kChunks;
            const size_t src = base + (r < rows ? r : 0) * pitch + 8 * ch;
            copy16(at(dst, r, ch), a.q + src, r < rows);
            copy16(at(dst + C::kOffDO, r, ch), a.dO + src, r < rows);
        }
    };
    uint4 o[2][kChunks / 4];  // of rows 16 warp + 8 t + g: chunks 4 i + c
    float lse2[2][2];         // of rows 16 warp + 8 t + 2 c + e, in log2 units; +inf (P = 0) past the end
    auto lse_at = [&](int step) {
        const int h = h0 + step / nr;
        return (a.cu ? (size_t)h * a.T + start : ((size_t)seq * a.Hq + h) * a.S) + row_of(step);
    };
    auto load_rows = [&](int step) {
        const int rows = r_end - row_of(step);
        const uint16_t* src = a.o + base_of(step);
        const float* lse = a.lse + lse_at(step);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const int r = 16 * warp + 8 * t + g;
#pragma unroll
            for (int i = 0; i < kChunks / 4; ++i)
                o[t][i] = r < rows ? *reinterpret_cast<const uint4*>(src + r * pitch + 8 * (4 * i + c)) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int rr = 16 * warp + 8 * t + 2 * c + e;
                lse2[t][e] = rr < rows ? lse[rr] * kLog2e : INFINITY;
            }
        }
    };
    if (C::kStages == 2) {
        load(0);
        load_rows(0);
    }
    copies_commit();
    for (int step = 0; step < n; ++step) {
        const int rows = min(kRows, r_end - row_of(step));
        const size_t base = base_of(step), lbase = lse_at(step);
        const uint32_t sQ = sTiles + step % C::kStages * (2 * C::kTile), sDO = sQ + C::kOffDO;
        if (C::kStages == 2) {
            if (step + 1 < n) load(step + 1);
            copies_commit();
            copies_wait<1>();
        } else {
            load(step);
            copies_commit();
            load_rows(step);
            const int rn = step + 1 < n ? row_of(step + 1) + (tid & 63) : r_end;  // the step behind this one: into L2
            if (rn < r_end) {
                const size_t src = base_of(step + 1) + (tid & 63) * pitch;
                prefetch_bulk((tid < 64 ? a.q : a.dO) + src, C::kRowBytes);
                if (tid < 64) prefetch_bulk(a.o + src, C::kRowBytes);
            }
            copies_wait<0>();
        }
        __syncthreads();
        float delta[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const int r = 16 * warp + 8 * t + g;
            float acc = 0.f;
            auto dot2 = [](uint32_t x, uint32_t y) {
                return __uint_as_float(x << 16) * __uint_as_float(y << 16) +
                       __uint_as_float(x & 0xffff0000u) * __uint_as_float(y & 0xffff0000u);
            };
#pragma unroll
            for (int i = 0; i < kChunks / 4; ++i) {
                uint32_t w[4];
                ld_shared_v4(at(sDO, r, 4 * i + c), w[0], w[1], w[2], w[3]);
                acc += dot2(o[t][i].x, w[0]) + dot2(o[t][i].y, w[1]) + dot2(o[t][i].z, w[2]) + dot2(o[t][i].w, w[3]);
            }
            acc += __shfl_xor_sync(0xffffffffu, acc, 1);
            acc += __shfl_xor_sync(0xffffffffu, acc, 2);
            delta[t] = acc;
            if (c == 0 && r < rows) a.delta[lbase + r] = acc;
        }
        // S^T and dP^T: keys g, g + 8; rows 8 t + 2c, + 1
        float s[2][4] = {}, dp[2][4] = {};
#pragma unroll 4
        for (int ks = 0; ks < D / 16; ++ks) {
            uint32_t x0, x1, x2, x3, y0, y1, y2, y3;
            ldsm_x4(at(sK, mr, 2 * ks + mc), x0, x1, x2, x3);
            ldsm_x4(at(sQ, 16 * warp + mr, 2 * ks + mc), y0, y1, y2, y3);
            mma_16x8x16_bf16(s[0], x0, x1, x2, x3, y0, y2);
            mma_16x8x16_bf16(s[1], x0, x1, x2, x3, y1, y3);
            ldsm_x4(at(sV, mr, 2 * ks + mc), x0, x1, x2, x3);
            ldsm_x4(at(sDO, 16 * warp + mr, 2 * ks + mc), y0, y1, y2, y3);
            mma_16x8x16_bf16(dp[0], x0, x1, x2, x3, y0, y2);
            mma_16x8x16_bf16(dp[1], x0, x1, x2, x3, y1, y3);
        }
        uint32_t pw[2][2], dw[2][2];  // [t][key half]: rows 8 t + 2c, + 1
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const float d0 = __shfl_sync(0xffffffffu, delta[t], 8 * c), d1 = __shfl_sync(0xffffffffu, delta[t], 8 * c + 4);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const bool seen = g + 8 * half < a.sink.sink;
                const float p0 = seen ? fast_exp2(fmaf(s[t][2 * half], a.scale_log2, -lse2[t][0])) : 0.f;
                const float p1 = seen ? fast_exp2(fmaf(s[t][2 * half + 1], a.scale_log2, -lse2[t][1])) : 0.f;
                pw[t][half] = pack_bf16x2(p0, p1);
                dw[t][half] = pack_bf16x2(p0 * (dp[t][2 * half] - d0), p1 * (dp[t][2 * half + 1] - d1));
            }
        }
        if (C::kStages == 2 && step + 1 < n) load_rows(step + 1);
        pf[warp * 32 + lane] = make_uint4(pw[0][0], pw[0][1], pw[1][0], pw[1][1]);
        df[warp * 32 + lane] = make_uint4(dw[0][0], dw[0][1], dw[1][0], dw[1][1]);
        // dQ: rows g, g + 8, dims 8 n + 2c, + 1
        {
            const uint32_t a0 = transpose8(dw[0][0]), a1 = transpose8(dw[1][0]), a2 = transpose8(dw[0][1]), a3 = transpose8(dw[1][1]);
            const int r = 16 * warp + g;
            float* row = a.dq_acc + base + r * pitch + 2 * c;
#pragma unroll 4
            for (int x = 0; x < kChunks; x += 2) {
                uint32_t x0, x1, x2, x3;
                ldsm_x4_trans(at(sK, mr, x + mc), x0, x1, x2, x3);
                float d0[4] = {}, d1[4] = {};
                mma_16x8x16_bf16(d0, a0, a1, a2, a3, x0, x1);
                mma_16x8x16_bf16(d1, a0, a1, a2, a3, x2, x3);
                if (r < rows) {
                    *reinterpret_cast<float2*>(row + 8 * x) = make_float2(d0[0] * a.scale, d0[1] * a.scale);
                    *reinterpret_cast<float2*>(row + 8 * x + 8) = make_float2(d1[0] * a.scale, d1[1] * a.scale);
                }
                if (r + 8 < rows) {
                    *reinterpret_cast<float2*>(row + 8 * pitch + 8 * x) = make_float2(d0[2] * a.scale, d0[3] * a.scale);
                    *reinterpret_cast<float2*>(row + 8 * pitch + 8 * x + 8) = make_float2(d1[2] * a.scale, d1[3] * a.scale);
                }
            }
        }
        __syncthreads();
        // dV and dK: keys g, g + 8, dims of the warp's quarter
#pragma unroll
        for (int ks = 0; ks < kWarps; ++ks) {
            const uint4 p = pf[ks * 32 + lane], d = df[ks * 32 + lane];
#pragma unroll
            for (int n = 0; n < kMine; n += 2) {
                uint32_t x0, x1, x2, x3;
                ldsm_x4_trans(at(sDO, 16 * ks + mr, warp * kMine + n + mc), x0, x1, x2, x3);
                mma_16x8x16_bf16(dv[n], p.x, p.y, p.z, p.w, x0, x1);
                mma_16x8x16_bf16(dv[n + 1], p.x, p.y, p.z, p.w, x2, x3);
                ldsm_x4_trans(at(sQ, 16 * ks + mr, warp * kMine + n + mc), x0, x1, x2, x3);
                mma_16x8x16_bf16(dk[n], d.x, d.y, d.z, d.w, x0, x1);
                mma_16x8x16_bf16(dk[n + 1], d.x, d.y, d.z, d.w, x2, x3);
            }
        }
        __syncthreads();
    }
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        const int j = g + 8 * half;
        if (j >= a.sink.sink) continue;
        float* pv = a.sink.row(seq, start, 1 + blockIdx.x, hk, a.Hkv, j, D) + warp * (D / kWarps) + 2 * c;
        float* pk = pv + (size_t)a.sink.sink * D;
#pragma unroll
        for (int n = 0; n < kMine; ++n) {
            *reinterpret_cast<float2*>(pv + 8 * n) = make_float2(dv[n][2 * half], dv[n][2 * half + 1]);
            *reinterpret_cast<float2*>(pk + 8 * n) = make_float2(dk[n][2 * half] * a.scale, dk[n][2 * half + 1] * a.scale);
        }
    }
}

// dK and dV of the sinks of the sequences whose far queries were shared out: the sum of the near part and the slices',
// in one order, whatever order they were computed in. A block owns one (sequence, KV head, sink) of dV or dK; D / 4 threads read a part,
// 4 dims each, the block's several groups of them a stretch of the parts each, 8 of them at once, and the groups' sums are added in
// shared memory.
constexpr int kSumThreads = 512;

__global__ void __launch_bounds__(kSumThreads) bwd_sink_sum_kernel(SinkSplit sk, uint16_t* __restrict__ dK, uint16_t* __restrict__ dV,
                                                                   const int32_t* __restrict__ cu, int S, int T, int Hkv, int D, int window) {
    griddep_wait();
    __shared__ float4 sums[kSumThreads];
    const int j = blockIdx.x >> 1, g = blockIdx.y, seq = blockIdx.z, per = D / 4, group = threadIdx.x / per, d = 4 * (threadIdx.x % per);
    int start = seq * S, L = S;
    if (cu) {
        start = cu[seq], L = cu[seq + 1] - start;
        if (!varlen_seq_ok(start, L, T, S)) return;
    }
    const int far = far_from(L, window);
    if (far >= L) return;  // the main kernel wrote them
    const int parts = 1 + (L - far + sk.rows - 1) / sk.rows * sk.shares, groups = kSumThreads / per;
    const int p0 = (int)((long long)parts * group / groups), p1 = (int)((long long)parts * (group + 1) / groups);
    const float* part = sk.row(seq, start, 0, g, Hkv, j, D) + (blockIdx.x & 1) * (size_t)sk.sink * D + d;
    const size_t pitch = sk.row(seq, start, 1, g, Hkv, j, D) - sk.row(seq, start, 0, g, Hkv, j, D);
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int p = p0; p < p1; ++p) {
        const float4 x = *reinterpret_cast<const float4*>(part + p * pitch);
        s.x += x.x, s.y += x.y, s.z += x.z, s.w += x.w;
    }
    sums[threadIdx.x] = s;
    __syncthreads();
    if (group) return;
    for (int n = 1; n < groups; ++n) {
        const float4 x = sums[n * per + threadIdx.x];
        s.x += x.x, s.y += x.y, s.z += x.z, s.w += x.w;
    }
    *reinterpret_cast<uint2*>((blockIdx.x & 1 ? dK : dV) + ((size_t)(start + j) * Hkv + g) * D + d) =
        make_uint2(pack_bf16x2(s.x, s.y), pack_bf16x2(s.z, s.w));
}

template <int D>
cudaError_t launch_far(const BwdLaunch& L, cudaStream_t stream) {
    FarArgs a;
    a.q = L.q, a.k = L.k, a.v = L.v, a.o = L.o, a.dO = L.dO, a.lse = L.lse, a.delta = L.delta, a.dq_acc = L.dq_acc;
    a.cu = L.cu_seqlens, a.Hq = L.Hq, a.Hkv = L.Hkv, a.S = L.S, a.T = L.total_rows, a.window = L.window;
    a.scale = L.scale, a.scale_log2 = L.scale * kLog2e, a.sink = L.sink;
    constexpr int kSmem = FarCfg<D>::kSmem;
    cudaError_t e = cudaFuncSetAttribute(bwd_far_sink_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    const ProfMark m = prof_begin(stream, "bwd_far_sink");
    e = launch_behind(bwd_far_sink_kernel<D>, dim3(L.sink.slices * L.sink.shares, L.Hkv, L.nseq), dim3(kThreads), kSmem, stream, a);
    prof_end(stream, m);
    return e;
}

}  // namespace

cudaError_t launch_bwd_far_sinks(const BwdLaunch& L, cudaStream_t stream) {
    if (L.D == 64) return launch_far<64>(L, stream);
    if (L.D == 128) return launch_far<128>(L, stream);
    if (L.D == 256) return launch_far<256>(L, stream);
    return cudaErrorInvalidValue;
}

cudaError_t launch_bwd_sink_sum(const BwdLaunch& L, cudaStream_t stream) {
    const ProfMark m = prof_begin(stream, "bwd_sink_sum");
    const cudaError_t e = launch_behind(bwd_sink_sum_kernel, dim3(2 * L.sink.sink, L.Hkv, L.nseq), dim3(kSumThreads), 0, stream, L.sink, L.dK,
                                        L.dV, L.cu_seqlens, L.S, L.total_rows, L.Hkv, L.D, L.window);
    prof_end(stream, m);
    return e;
}

}  // namespace attn
