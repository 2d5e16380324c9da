// The 4-bit paged cache: what a record holds and where. Used by the kernels that write it and read it.
//
// A record holds the 16 tokens of one page and KV head, 18 D bytes: codes of K (8 D), codes of V (8 D), scales of
// K (D), scales of V (D). 32 consecutive dims of a token are a group; its values are n * s with n = -8 .. 7, held as the
// code n + 8 in 4 bits, and s a bf16 number of 5 significant bits. So n * s is a bf16 number (3 + 5 bits), and so is
// 24 s, which lets one fused multiply-add in bf16 turn the bit pattern of 16 + code into n * s exactly:
// (16 + code) s - 24 s = (code - 8) s. (16 + code is the code put in the upper bits of the mantissa of 16. In the lower ones
// it would be 128 + code and save one shift in eight, but sums of products with it lose three more bits.)
//
// The order of the codes is that of the fragments of a 16 x 16 warp MMA operand, so that a decode warp loads them with
// 16-byte loads that touch every bank once, and unpacks a word by shifting and masking alone:
//  * K, the A operand of S^T = K Q^T (rows tokens, columns dims): [block of 128 dims][token][strip c of 4][group], a
//    4-byte word each. Lane (g, c) reads strip c of tokens g and g + 8. A word holds dims 8 c .. 8 c + 7 of its
//    group, the even ones in nibbles 0 .. 3 and the odd ones in nibbles 4 .. 7: word >> 4 i has dims 8 c + 2 i and
//    8 c + 2 i + 1 in the low nibbles of its halves.
//  * V, the A operand of O^T = V^T P^T (rows dims, columns tokens): [block of 128 dims][token pair][chunk of 16 dims][token
//    of the pair], 8 bytes each, the dims in order. Lane (g, c) reads chunk g of pairs c and c + 4; half words of the two
//    tokens side by side then have a dim of both in the low nibbles of their halves. Chunks of a pair are
//    exchanged by its number (chunk ^ 2 (pair % 4)), which puts the eight lanes of a 16-byte access in eight bank groups.
//  * D = 64 has one block of 64 dims: two groups, chunks of 8 dims (4 bytes), two pairs in 128 bytes.
//  * Scales: K [token][group], V [group][token] (so that a lane reads those of two tokens as one word).
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

namespace attn {

constexpr int kv4_record_bytes(int D) { return 18 * D; }

// Byte offsets within a record.
template <int D>
struct Kv4 {
    static constexpr int W = D < 128 ? D : 128;  // dims of a block
    static constexpr int kGroups = D / 32;
    static constexpr int kBlockGroups = W / 32;
    static constexpr int kV = 8 * D, kScaleK = 16 * D, kScaleV = 17 * D;
    static constexpr int kRecord = 18 * D;

    // word of strip c, token t, group 0 of a block (the block's other groups follow)
    __host__ __device__ static int key_strip(int block, int t, int c) { return block * 8 * W + t * (W / 2) + c * (4 * kBlockGroups); }
    // chunk g of a token pair (its even token; the odd one follows after W / 16 bytes)
    __host__ __device__ static int value_chunk(int block, int pair, int g) {
        if (W == 128) return kV + block * 8 * W + pair * 128 + ((g ^ (2 * (pair & 3))) << 4);
        return kV + (pair >> 1) * 128 + ((((pair & 1) * 8 + g) ^ (4 * ((pair >> 1) & 1))) << 3);
    }
    __host__ __device__ static int key_scale(int t, int group) { return kScaleK + 2 * (t * kGroups + group); }
    __host__ __device__ static int value_scale(int group, int t) { return kScaleV + 2 * (group * 16 + t); }
};

// Codes i and i + 4 of a word as bf16 numbers 16 + code, i = 0 .. 3.
__device__ __forceinline__ uint32_t kv4_pair(uint32_t w, int i) {
    return ((i == 0 ? w << 3 : w >> (4 * i - 3)) & 0x00780078u) | 0x41804180u;
}

constexpr uint32_t kMinus24 = 0xc1c0c1c0u;  // two bf16 numbers -24

__device__ __forceinline__ uint32_t bf16x2_mul(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t bf16x2_fma(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}

}  // namespace attn
