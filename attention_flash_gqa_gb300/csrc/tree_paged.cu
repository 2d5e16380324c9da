// Attention of drafted token trees over a paged cache: the verification step of speculative decoding.
//
// Row i of a request with n drafted tokens behind c = L - n cached ones sees the context keys
// j < c (with a window only those with p_i - j < W, p_i = max(position, c)) and the drafted tokens
// d whose bit is set in its mask row:
//     s_ij = scale q_i . k_j,   o_i = sum_j softmax_j(s_ij | visible) v_j,   lse_i = ln sum_j exp(s_ij)
// A row that sees nothing gets o = 0 and lse = -inf.
//
// One warp per (row, query head): the lanes split the dims, keys are taken one at a time with a running
// maximum and sum in the log2 domain.
#include <cuda_runtime.h>

#include "attn_internal.h"
#include "ptx.cuh"

namespace attn {
namespace {

constexpr int kPage = 16;
constexpr int kWarps = 4;

template <int D>
__global__ void __launch_bounds__(kWarps * 32) tree_paged_kernel(const __grid_constant__ TreeLaunch a) {
    constexpr int DL = D / 32;  // dims per lane
    const int lane = threadIdx.x & 31, h = blockIdx.y, b = blockIdx.z;
    const int start = a.cu_q[b], n = a.cu_q[b + 1] - start, L = a.seq_lens[b];
    if (start < 0 || n < 0 || n > a.max_q || start > a.T - n || n > L || (long long)L > (long long)a.max_pages * kPage) {
        if (threadIdx.x == 0 && blockIdx.x == 0 && h == 0) atomicOr(a.status, DEVSTAT_BOUNDS);
        return;
    }
    const int i = blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (i >= n) return;
    const int c = L - n, row = start + i, g = h / (a.Hq / a.Hkv);
    int lo = 0;
    if (a.window > 0) lo = max(0, min(c, max(a.positions[row], c) - a.window + 1));
    float q[DL], o[DL], m = -INFINITY, l = 0.f;
    const float scale_log2 = a.scale * 1.4426950408889634f;
#pragma unroll
    for (int e = 0; e < DL; ++e) {
        q[e] = __uint_as_float((uint32_t)a.q[((size_t)row * a.Hq + h) * D + 32 * e + lane] << 16) * scale_log2;
        o[e] = 0.f;
    }
    for (int j = lo; j < L; ++j) {
        if (j >= c && !(a.mask[(size_t)row * a.words + ((j - c) >> 5)] >> ((j - c) & 31) & 1)) continue;
        int page = a.block_table[(size_t)b * a.max_pages + j / kPage];
        if (page < 0 || page >= a.num_pages) {
            if (lane == 0) atomicOr(a.status, DEVSTAT_BOUNDS);
            page = 0;
        }
        const size_t at = (((size_t)page * kPage + j % kPage) * a.Hkv + g) * D;
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < DL; ++e) s = fmaf(q[e], __uint_as_float((uint32_t)a.k_cache[at + 32 * e + lane] << 16), s);
#pragma unroll
        for (int off = 16; off; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
        const float mn = fmaxf(m, s), al = exp2f(m - mn), p = exp2f(s - mn);
        l = l * al + p, m = mn;
#pragma unroll
        for (int e = 0; e < DL; ++e) o[e] = fmaf(p, __uint_as_float((uint32_t)a.v_cache[at + 32 * e + lane] << 16), o[e] * al);
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
    for (int e = 0; e < DL; ++e) {
        const uint32_t w = pack_bf16x2(o[e] * inv, 0.f);
        a.o[((size_t)row * a.Hq + h) * D + 32 * e + lane] = (uint16_t)(w & 0xffffu);
    }
    if (lane == 0) a.lse[(size_t)h * a.T + row] = l > 0.f ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
}

}  // namespace

cudaError_t launch_tree_paged(const TreeLaunch& L, cudaStream_t stream) {
    const dim3 grid((L.max_q + kWarps - 1) / kWarps, L.Hq, L.R);
    const ProfMark m = prof_begin(stream, "tree_paged");
    switch (L.D) {
        case 64: tree_paged_kernel<64><<<grid, kWarps * 32, 0, stream>>>(L); break;
        case 128: tree_paged_kernel<128><<<grid, kWarps * 32, 0, stream>>>(L); break;
        case 256: tree_paged_kernel<256><<<grid, kWarps * 32, 0, stream>>>(L); break;
        case 512: tree_paged_kernel<512><<<grid, kWarps * 32, 0, stream>>>(L); break;
        default: return cudaErrorInvalidValue;
    }
    prof_end(stream, m);
    return cudaGetLastError();
}

}  // namespace attn
