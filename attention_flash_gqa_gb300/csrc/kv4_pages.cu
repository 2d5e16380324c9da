// Writing and reading back the 4-bit paged cache (kv4.cuh has the format).
//
// append: rows of K and V, in bf16, become records' tokens at their slots. A group of 32 values x gets
//   s = -(its value of largest magnitude) / 8 rounded to 5 significant bits, n = x / s rounded to the nearest whole number
// so that value is n = -8, the one level that has no counterpart, and a step is an eighth of it instead of a seventh. Nothing is read
// of the record, and no byte holds two tokens: tokens of a call may be any.
// unpack: pages back as bf16 pages, exactly. A thread has 8 dims of two neighbouring tokens (which share the V sectors).
// 8192 tokens, 16 heads of 256: append 31 us (172 MB, 0.81 of the copy rate; behind other work 36, 0.70 of its issue slots used: its
// arithmetic is kept on the pipe of the multiplications as far as that goes, before which it took 66), unpack 28.5 (0.89). A
// decode step's few rows are launch and latency: 2.9 and 6 us, the latter the host's (two outputs to allocate).
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

// The larger / smaller of two bf16 numbers each, NaN where one is.
__device__ __forceinline__ uint32_t bf16x2_max(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t bf16x2_min(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

__device__ __forceinline__ float reciprocal(float x) {  // within an ulp
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// a b + c, where a shift would be meant: the pipe of the multiplications has room, that of shifts and comparisons has none.
__device__ __forceinline__ uint32_t mad(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("mad.lo.u32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}

// The largest of 8 values and the negative of the smallest, as the halves of a word (NaN if one is).
__device__ __forceinline__ uint32_t ends_of(const uint32_t* w) {
    const uint32_t mx = bf16x2_max(bf16x2_max(w[0], w[1]), bf16x2_max(w[2], w[3]));
    const uint32_t mn = bf16x2_min(bf16x2_min(w[0], w[1]), bf16x2_min(w[2], w[3])) ^ 0x80008000u;
    return bf16x2_max(__byte_perm(mx, mn, 0x5410), __byte_perm(mx, mn, 0x7632));
}

constexpr uint32_t kMaxScale = 0x7cf8;  // 31 * 2^118: 24 s stays finite

// The scale of a group with these ends, as bf16 bits: an eighth of the larger magnitude (a bf16 number: three off the exponent, which
// may leave the pattern below that of 2^-126, where the exponent still counts on), to 5 significant bits, ties to even.
__device__ __forceinline__ uint32_t scale_of(uint32_t ends) {
    const uint32_t hi = ends & 0x7fffu, lo = ends >> 16 & 0x7fffu;
    // (the half of larger magnitude is not negative: the ends are a maximum and minus a minimum)
    const bool pos = __uint_as_float(ends << 16) > __uint_as_float(ends & 0xffff0000u);
    const int m = (int)(pos ? hi : lo) - (3 << 7);
    const int r = (m + 3 + ((m >> 3) & 1)) & ~7;
    const uint32_t s = r < 0x80 ? 0u : min((uint32_t)r, kMaxScale);  // (m is negative where r is, or r is 0)
    return max(hi, lo) >= 0x7f80u ? 0x7fc0u : s | (pos && s ? 0x8000u : 0u);  // an infinity or a NaN: NaN
}

// Codes of 8 values with the group's scale, that of value i in nibble (kSplit: i / 2 + 4 (i % 2), else i) of the word.
// x / s is at least 2^-10 from half of an odd number unless it is one (x has 8 bits, s has 5), and x (1 / s) is off by 2^-19 at
// most: rounded to multiples of 2^-12 first, it ties where x / s does and nowhere else. So, in the pipe of the multiplications
// alone: (x / s + 9) / 16 cut to 1 from above (7; below -8.25 it does not get), times 16 + 1.5 * 2^11, whose last place is 2^-12, and the
// sum with 1.5 * 2^23 that leaves code + 0x4b400000 as its bits; the upper parts drop out of the word by one subtraction.
template <bool kSplit>
__device__ __forceinline__ uint32_t codes_of(uint32_t* w, uint32_t s) {
    if ((s & 0x7fffu) >= kMaxScale) {  // (or NaN)
        if ((s & 0x7fffu) > kMaxScale) return 0x88888888u;
        const uint32_t most = (kMaxScale + (3u << 7)) * 0x10001u;  // values beyond 8 s count as 8 s
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = bf16x2_max(bf16x2_min(w[e], most), most ^ 0x80008000u);
    }
    const float inv = (s & 0x7fffu) == 0 ? 0.f : 0.0625f * reciprocal(__uint_as_float(s << 16));
    uint32_t word = 0u - 0x4b400000u * 0x11111111u;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float x = __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : mad(w[i / 2], 1u << 16, 0u));
        float y;
        asm("fma.rn.sat.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(x), "f"(inv), "f"(0.5625f));
        constexpr float kTies = 1.5f * 2048.f;
        const float z = __fadd_rn(__fmaf_rn(y, 16.f, kTies - 1.f), 12582912.f - kTies);
        word = mad(__float_as_uint(z), 1u << (4 * (kSplit ? i / 2 + 4 * (i & 1) : i)), word);
    }
    return word;
}

// row / Hkv for rows below 2^31: high word of a product, Hkv's multiplier being ceil(2^(31 + bits) / Hkv), 2^bits the power of two
// at or above Hkv. (It is above 2^(31 + bits) / Hkv by less than 1, so the quotient by less than row / 2^(31 + bits) <= 1 / Hkv.)
struct HeadDivision {
    uint32_t by;
    int shift;
    explicit HeadDivision(int heads) {
        int bits = 0;
        while ((1 << bits) < heads) ++bits;
        by = (uint32_t)(((1ull << (31 + bits)) + heads - 1) / heads), shift = bits - 1;
    }
    __device__ __forceinline__ int operator()(int row) const { return shift < 0 ? row : (int)(__umulhi((uint32_t)row, by) >> shift); }
};

// A thread has 16 dims of K and of V of a (token, head) row, half a group: one of the two that share it works out K's scale, the
// other V's.
template <int D>
__global__ void __launch_bounds__(kThreads) kv4_append_kernel(AppendArgs a, HeadDivision token_of) {
    using F = Kv4<D>;
    constexpr int kPerRow = D / 16;
    const int d = 16 * (threadIdx.x % kPerRow), block = d / F::W, e = d % F::W, group = e / 32, strip = (e % 32) / 8;
    const uint32_t row = blockIdx.x * (uint32_t)(kThreads / kPerRow) + threadIdx.x / kPerRow;
    griddep_wait();
    const bool there = row < (uint32_t)(a.T * a.Hkv);
    const int t = there ? token_of((int)row) : 0, head = (int)row - t * a.Hkv;
    uint32_t kx[8] = {}, vx[8] = {};
    int slot = -1;
    if (there) {  // (padding's too: its slot is not waited for before the values are asked for)
        slot = a.slots[t];
        const uint4* k = reinterpret_cast<const uint4*>(a.k + t * a.k_stride + head * D + d);
        const uint4* v = reinterpret_cast<const uint4*>(a.v + t * a.v_stride + head * D + d);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const uint4 y = k[x], z = v[x];
            kx[4 * x] = y.x, kx[4 * x + 1] = y.y, kx[4 * x + 2] = y.z, kx[4 * x + 3] = y.w;
            vx[4 * x] = z.x, vx[4 * x + 1] = z.y, vx[4 * x + 2] = z.z, vx[4 * x + 3] = z.w;
        }
    }
    const bool live = (uint32_t)slot < (uint32_t)a.num_slots;
    if (!live && slot != -1 && head == 0 && d == 0) atomicOr(a.status, DEVSTAT_BOUNDS);
    const bool odd = threadIdx.x & 1;
    const uint32_t ke = bf16x2_max(ends_of(kx), ends_of(kx + 4)), ve = bf16x2_max(ends_of(vx), ends_of(vx + 4));
    const uint32_t mine = scale_of(bf16x2_max(odd ? ve : ke, __shfl_xor_sync(0xffffffffu, odd ? ke : ve, 1)));
    const uint32_t other = __shfl_xor_sync(0xffffffffu, mine, 1);
    const uint32_t ks = odd ? other : mine, vs = odd ? mine : other;
    if (!live) return;
    uint8_t* rec = a.cache + ((size_t)(slot >> 4) * a.Hkv + head) * F::kRecord;
    const int tok = slot & 15;
    uint32_t vw[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        *reinterpret_cast<uint32_t*>(rec + F::key_strip(block, tok, strip + x) + 4 * group) = codes_of<true>(kx + 4 * x, ks);
        vw[x] = codes_of<false>(vx + 4 * x, vs);
    }
    if constexpr (F::W == 128) {
        *reinterpret_cast<uint2*>(rec + F::value_chunk(block, tok >> 1, e / 16) + (tok & 1) * 8) = make_uint2(vw[0], vw[1]);
    } else {
#pragma unroll
        for (int x = 0; x < 2; ++x) *reinterpret_cast<uint32_t*>(rec + F::value_chunk(0, tok >> 1, e / 8 + x) + (tok & 1) * 4) = vw[x];
    }
    if (odd) *reinterpret_cast<uint16_t*>(rec + F::value_scale(d / 32, tok)) = (uint16_t)vs;
    else *reinterpret_cast<uint16_t*>(rec + F::key_scale(tok, d / 32)) = (uint16_t)ks;
}

struct UnpackArgs {
    const uint8_t* cache;
    const int32_t* pages;
    uint16_t *k, *v;
    unsigned* status;
    int n, Hkv, num_pages;
};

template <int D>
__global__ void __launch_bounds__(kThreads) kv4_unpack_kernel(UnpackArgs a, HeadDivision page_pair_of) {
    using F = Kv4<D>;
    griddep_wait();
    constexpr int kPerRow = D / 8;
    // rows in the order of the result: page, token pair, head
    const long long row = (long long)blockIdx.x * (kThreads / kPerRow) + threadIdx.x / kPerRow;
    if (row >= (long long)a.n * 8 * a.Hkv) return;
    const int pp = page_pair_of((int)row), h = (int)row - pp * a.Hkv;
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

template <class... Params, class... Args>
cudaError_t launch(void (*kern)(Params...), long long rows, int per_block, const char* name, cudaStream_t stream, const Args&... args) {
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
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
    prof_end(stream, m);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv4_append(const Kv4Launch& L, cudaStream_t stream) {
    AppendArgs a;
    a.k = L.k, a.v = L.v, a.slots = L.slots, a.cache = L.cache, a.status = L.status;
    a.k_stride = L.k_stride, a.v_stride = L.v_stride, a.T = L.n, a.Hkv = L.Hkv, a.num_slots = L.num_pages * 16;
    const long long rows = (long long)L.n * L.Hkv;
    if (L.D == 64) return launch(kv4_append_kernel<64>, rows, kThreads * 16 / 64, "kv4_append", stream, a, HeadDivision(L.Hkv));
    if (L.D == 128) return launch(kv4_append_kernel<128>, rows, kThreads * 16 / 128, "kv4_append", stream, a, HeadDivision(L.Hkv));
    if (L.D == 256) return launch(kv4_append_kernel<256>, rows, kThreads * 16 / 256, "kv4_append", stream, a, HeadDivision(L.Hkv));
    return cudaErrorInvalidValue;
}

cudaError_t launch_kv4_unpack(const Kv4Launch& L, cudaStream_t stream) {
    UnpackArgs a;
    a.cache = L.cache, a.pages = L.pages, a.k = L.k_out, a.v = L.v_out, a.status = L.status;
    a.n = L.n, a.Hkv = L.Hkv, a.num_pages = L.num_pages;
    const long long rows = (long long)L.n * 8 * L.Hkv;
    if (L.D == 64) return launch(kv4_unpack_kernel<64>, rows, kThreads * 8 / 64, "kv4_unpack", stream, a, HeadDivision(L.Hkv));
    if (L.D == 128) return launch(kv4_unpack_kernel<128>, rows, kThreads * 8 / 128, "kv4_unpack", stream, a, HeadDivision(L.Hkv));
    if (L.D == 256) return launch(kv4_unpack_kernel<256>, rows, kThreads * 8 / 256, "kv4_unpack", stream, a, HeadDivision(L.Hkv));
    return cudaErrorInvalidValue;
}

}  // namespace attn
