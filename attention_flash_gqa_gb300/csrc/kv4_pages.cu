// Writing and reading back the 4-bit paged cache (kv4.cuh has the format).
//
// append: rows of K and V, in bf16, become records' tokens at their slots. A group of 32 values x gets
//   s = -(its value of largest magnitude) / 8 rounded to 5 significant bits, n = x / s rounded to the nearest whole number
// so that value is n = -8, the one level that has no counterpart, and a step is an eighth of it instead of a seventh. A thread
// has 8 dims of one token and head, K and V, and four neighbours share a group: two exchanges give them its largest and
// smallest value. Nothing is read of the record, and no byte holds two tokens: tokens of a call may be any.
// unpack: pages back as bf16 pages, exactly. A thread has 8 dims of two neighbouring tokens (which share the V sectors).
// Both are bound by memory: see the table of measured cases.
#include <cuda_runtime.h>

#include "attn_internal.h"
#include "kv4.cuh"
#include "ptx.cuh"

namespace attn {
namespace {

constexpr int kThreads = 256;

struct AppendArgs {
    const uint16_t *k, *v;
    const int32_t* slots;
    uint8_t* cache;
    unsigned* status;
    long long k_stride, v_stride;
    int T, Hkv, num_slots;
};

// 8 values of a group, two to a word -> their codes, 0 .. 15; s: the group's scale as bf16 bits.
__device__ __forceinline__ void quantise(const uint4 in, uint32_t (&code)[8], uint32_t& s) {
    const uint32_t w[4] = {in.x, in.y, in.z, in.w};
    float x[8];
    bool bad = false;  // an infinity or a NaN
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        x[2 * e] = __uint_as_float(w[e] << 16), x[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
        bad |= (w[e] & 0x7f80u) == 0x7f80u || (w[e] & 0x7f800000u) == 0x7f800000u;
    }
    float hi = x[0], lo = x[0];
#pragma unroll
    for (int e = 1; e < 8; ++e) hi = fmaxf(hi, x[e]), lo = fminf(lo, x[e]);
#pragma unroll
    for (int off = 1; off < 4; off <<= 1) {
        hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, off));
        lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, off));
    }
    const unsigned votes = __ballot_sync(0xffffffffu, bad) >> (threadIdx.x & 28);
    bad = (votes & 15u) != 0;
    // An eighth of the magnitude (a bf16 number: three off the exponent, which may leave the pattern below that of 2^-126,
    // where the exponent still counts on), to 5 significant bits, ties to even.
    const bool pos = hi > -lo;
    const int m = (int)(__float_as_uint(pos ? hi : lo) >> 16 & 0x7fffu) - (3 << 7);
    int r = (m + 3 + ((m >> 3) & 1)) & ~7;
    if (m < 0 || r < 0x80) r = 0;
    r = min(r, 0x7cf8);  // 31 * 2^118: 24 s stays finite
    s = bad ? 0x7fc0u : (uint32_t)r | (pos && r ? 0x8000u : 0u);
    // x / s is at least 2^-10 from half of an odd number unless it is one (x has 8 bits, s has 5), and x * (1 / s) is off
    // by 2^-19 at most: rounded to whole multiples of 2^-12 first, it ties where x / s does and nowhere else.
    const float inv = bad || r == 0 ? 0.f : __frcp_rn(__uint_as_float(s << 16));
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float q = __fadd_rn(__fadd_rn(bad ? 0.f : x[e] * inv, 3072.f), -3072.f);
        code[e] = (uint32_t)(min(max(__float2int_rn(q), -8), 7) + 8);
    }
}

template <int D>
__global__ void __launch_bounds__(kThreads) kv4_append_kernel(AppendArgs a) {
    using F = Kv4<D>;
    griddep_wait();
    constexpr int kPerRow = D / 8;
    const long long row = (long long)blockIdx.x * (kThreads / kPerRow) + threadIdx.x / kPerRow;
    const bool there = row < (long long)a.T * a.Hkv;
    const int t = there ? (int)((uint32_t)row / (uint32_t)a.Hkv) : 0, h = there ? (int)row - t * a.Hkv : 0;
    const int d = 8 * (threadIdx.x % kPerRow);
    const int slot = there ? a.slots[t] : -1;
    const bool live = slot >= 0 && slot < a.num_slots;
    if (slot != -1 && !live && h == 0 && d == 0) atomicOr(a.status, DEVSTAT_BOUNDS);
    if (!__any_sync(0xffffffffu, live)) return;
    uint4 kx = make_uint4(0, 0, 0, 0), vx = kx;
    if (live) {
        kx = *reinterpret_cast<const uint4*>(a.k + t * a.k_stride + (size_t)h * D + d);
        vx = *reinterpret_cast<const uint4*>(a.v + t * a.v_stride + (size_t)h * D + d);
    }
    uint32_t kc[8], vc[8], ks, vs;
    quantise(kx, kc, ks);
    quantise(vx, vc, vs);
    if (!live) return;
    uint8_t* rec = a.cache + ((size_t)(slot >> 4) * a.Hkv + h) * F::kRecord;
    const int tok = slot & 15, block = d / F::W, e = d % F::W, group = e / 32;
    uint32_t kw = 0, vw = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        kw |= kc[i] << (4 * (i / 2 + 4 * (i & 1)));
        vw |= vc[i] << (4 * i);
    }
    *reinterpret_cast<uint32_t*>(rec + F::key_strip(block, tok, (e % 32) / 8) + 4 * group) = kw;
    constexpr int kChunk = F::W / 8;  // dims
    *reinterpret_cast<uint32_t*>(rec + F::value_chunk(block, tok >> 1, e / kChunk) + (tok & 1) * (kChunk / 2) + (e % kChunk) / 2) = vw;
    if (d % 32 == 0) {
        *reinterpret_cast<uint16_t*>(rec + F::key_scale(tok, d / 32)) = (uint16_t)ks;
        *reinterpret_cast<uint16_t*>(rec + F::value_scale(d / 32, tok)) = (uint16_t)vs;
    }
}

struct UnpackArgs {
    const uint8_t* cache;
    const int32_t* pages;
    uint16_t *k, *v;
    unsigned* status;
    int n, Hkv, num_pages;
};

template <int D>
__global__ void __launch_bounds__(kThreads) kv4_unpack_kernel(UnpackArgs a) {
    using F = Kv4<D>;
    griddep_wait();
    constexpr int kPerRow = D / 8;
    // rows in the order of the result: page, token pair, head
    const long long row = (long long)blockIdx.x * (kThreads / kPerRow) + threadIdx.x / kPerRow;
    if (row >= (long long)a.n * 8 * a.Hkv) return;
    const int pp = (int)((uint32_t)row / (uint32_t)a.Hkv), h = (int)row - pp * a.Hkv;
    const int pair = pp & 7, d = 8 * (threadIdx.x % kPerRow);
    const int page = a.pages[pp >> 3];
    if (page < 0 || page >= a.num_pages) {
        if (page != -1 && h == 0 && d == 0 && pair == 0) atomicOr(a.status, DEVSTAT_BOUNDS);
        return;
    }
    const uint8_t* rec = a.cache + ((size_t)page * a.Hkv + h) * F::kRecord;
    const int block = d / F::W, e = d % F::W, group = e / 32;
    constexpr int kChunk = F::W / 8;
    const uint8_t* chunk = rec + F::value_chunk(block, pair, e / kChunk) + (e % kChunk) / 2;
    uint32_t kw[2], vw[2], ks[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        kw[i] = *reinterpret_cast<const uint32_t*>(rec + F::key_strip(block, 2 * pair + i, (e % 32) / 8) + 4 * group);
        vw[i] = *reinterpret_cast<const uint32_t*>(chunk + i * (kChunk / 2));
        ks[i] = *reinterpret_cast<const uint16_t*>(rec + F::key_scale(2 * pair + i, d / 32));
    }
    const uint32_t vs2 = *reinterpret_cast<const uint32_t*>(rec + F::value_scale(d / 32, 2 * pair));
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t sk = ks[i] * 0x10001u, sv = (i ? vs2 >> 16 : vs2 & 0xffffu) * 0x10001u;
        const uint32_t ck = bf16x2_mul(sk, kMinus24), cv = bf16x2_mul(sv, kMinus24);
        uint32_t ko[4], vo[4];
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            ko[p] = bf16x2_fma(kv4_pair(kw[i], p), sk, ck);
            // V's dims 2 p and 2 p + 1 are neighbouring nibbles: moved to the halves of a word
            const uint32_t two = vw[i] >> (8 * p);
            vo[p] = bf16x2_fma(kv4_pair((two & 15u) | ((two & 0xf0u) << 12), 0), sv, cv);
        }
        const size_t at = (((size_t)(pp >> 3) * 16 + 2 * pair + i) * a.Hkv + h) * D + d;
        *reinterpret_cast<uint4*>(a.k + at) = make_uint4(ko[0], ko[1], ko[2], ko[3]);
        *reinterpret_cast<uint4*>(a.v + at) = make_uint4(vo[0], vo[1], vo[2], vo[3]);
    }
}

template <class Kernel, class Args>
cudaError_t launch(Kernel kern, const Args& a, long long rows, int D, const char* name, cudaStream_t stream) {
    const int per_block = kThreads / (D / 8);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((rows + per_block - 1) / per_block));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const ProfMark m = prof_begin(stream, name);
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, a);
    prof_end(stream, m);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv4_append(const Kv4Launch& L, cudaStream_t stream) {
    AppendArgs a;
    a.k = L.k, a.v = L.v, a.slots = L.slots, a.cache = L.cache, a.status = L.status;
    a.k_stride = L.k_stride, a.v_stride = L.v_stride, a.T = L.n, a.Hkv = L.Hkv, a.num_slots = L.num_pages * 16;
    const long long rows = (long long)L.n * L.Hkv;
    if (L.D == 64) return launch(kv4_append_kernel<64>, a, rows, 64, "kv4_append", stream);
    if (L.D == 128) return launch(kv4_append_kernel<128>, a, rows, 128, "kv4_append", stream);
    if (L.D == 256) return launch(kv4_append_kernel<256>, a, rows, 256, "kv4_append", stream);
    return cudaErrorInvalidValue;
}

cudaError_t launch_kv4_unpack(const Kv4Launch& L, cudaStream_t stream) {
    UnpackArgs a;
    a.cache = L.cache, a.pages = L.pages, a.k = L.k_out, a.v = L.v_out, a.status = L.status;
    a.n = L.n, a.Hkv = L.Hkv, a.num_pages = L.num_pages;
    const long long rows = (long long)L.n * 8 * L.Hkv;
    if (L.D == 64) return launch(kv4_unpack_kernel<64>, a, rows, 64, "kv4_unpack", stream);
    if (L.D == 128) return launch(kv4_unpack_kernel<128>, a, rows, 128, "kv4_unpack", stream);
    if (L.D == 256) return launch(kv4_unpack_kernel<256>, a, rows, 256, "kv4_unpack", stream);
    return cudaErrorInvalidValue;
}

}  // namespace attn
