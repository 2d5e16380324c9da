// Internal launch interfaces between the host API (api.cu) and the kernel files.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace attn {

// ---- launch accounting (api.cu) ------------------------------------------------------------
// Every kernel launch of the library goes through these: a process-wide launch counter and,
// when profiling is on, a CUDA event pair on the launching stream.
struct ProfMark {
    int slot = -1;
};
ProfMark prof_begin(cudaStream_t stream, const char* kernel);
void prof_end(cudaStream_t stream, ProfMark m);

// A launch with programmatic stream serialisation: the kernel may be placed while the one in front ends, so it has to wait
// (griddepcontrol.wait, every thread of every block, also of blocks that have nothing to do) before it reads or writes anything of the call's.
template <class... Params, class... Args>
cudaError_t launch_behind(void (*kern)(Params...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream, const Args&... args) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid, cfg.blockDim = block, cfg.dynamicSmemBytes = smem, cfg.stream = stream;
    cfg.attrs = attr, cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
    return e != cudaSuccess ? e : cudaGetLastError();
}

// ---- paged decode -----------------------------------------------------------------------
// tk / tv: 3-D maps over the caches (D, Hkv, num_pages * 16) with a D x hb x 16 box, no swizzle;
// used only when the KV heads are split into several blocks (hb < Hkv).
struct DecodeLaunch {
    CUtensorMap tk, tv;
    const uint16_t *q, *k_cache, *v_cache;
    const int32_t *block_table, *seq_lens;
    uint16_t* o;
    float* lse;
    float* part;
    unsigned* status;
    int B, Hq, Hkv, D, max_pages, num_pages, grid, window, sink;
    float scale;
};
size_t decode_smem_bytes(int hb, int D);
int decode_max_grid();
int decode_row_floats(int D);              // floats per (slot, head) partial row
int decode_heads_per_unit(int Hkv, int D, int G);  // hb: KV heads per unit (divides Hkv)
bool decode_packed_layout(int G, int D);  // K, V copied as [64-dim half][head][token][64], 128-byte swizzled
cudaError_t launch_decode_paged(const DecodeLaunch& L, cudaStream_t stream);

// ---- prefill forward ---------------------------------------------------------------------
// q/k/v tensor maps are 4-D over [D, H, S, B] (varlen: B = 1, S = total tokens) with a
// 64 x 1 x 128 x 1 box and 128-byte swizzle. Paged prefill: q as varlen over the packed new
// tokens; k/v over the caches as 5-D (64, 8, Hkv*D/64, 2, num_pages) with a 64 x 8 x 2 x 2 x 1
// box (16 rows x 128 dims of one head of one page).
struct FwdLaunch {
    CUtensorMap tq, tk, tv;
    CUtensorMap tk_half;        // k with a 64 x 1 x 64 x 1 box (CTA-pair forward: half a key tile per CTA)
    bool pair_ok = false;       // tk_half is valid: the CTA-pair forward may be used
    uint16_t* o;
    float* lse;
    const int32_t* cu_seqlens;  // null: dense (or paged)
    unsigned* status;
    int nseq;                   // B (dense), num_seqs (varlen) or num_reqs (paged)
    int Hq, Hkv, S, D;          // S: dense sequence length, max_seqlen (varlen) or max new tokens (paged)
    int total_rows;             // B*S (dense), total tokens (varlen) or total new tokens (paged)
    int window;
    float scale;
    // paged prefill (block_table non-null): request b's n_b = cu_q[b+1] - cu_q[b] new tokens
    // are the last n_b of its seq_lens[b] cached tokens
    const int32_t* block_table = nullptr;  // [num_reqs, max_pages]
    const int32_t* seq_lens = nullptr;
    const int32_t* cu_q = nullptr;
    int max_pages = 0, num_pages = 0;
    int sink = 0;  // first keys that stay visible past the window (0 .. 128)
    int sms = 0;
};
// Query heads that a block of the forward without pages takes at head_dim <= 256, one after the other (1, 2 or 4, Hq at most).
//  * Two where every SM has 12 query tiles for certain, four from 24 on (attn_fwd.cu, MULTI, has both sides). Dense calls know their tiles; of
//    packed ones the host knows only that no tile holds more than 128 rows, and none more than max_seqlen.
//  * Also where the grid has so many blocks that the empty ones count: of packed sequences far shorter than max_seqlen most blocks find no rows, 0.9 us
//    each on its SM. A further head costs at most the longest tile's time, about 2 us a key tile and 6. (Heads of 128, us with 1 and 4 heads a
//    block: one sequence of 4096 and 300 of 16, 8 heads, 77 thousand blocks 457 and 183; 4096 and 63 of 16, 16 thousand 132 and
//    162; one of 1000 where max_seqlen is 32768, 16 heads, 4 thousand 35 and 56.)
inline int fwd_heads(int Hq, int nseq, int S, int rows, bool packed, int window, int sms) {
    if (S < 1) return 1;  // (nothing to launch)
    const long long blocks = (long long)Hq * nseq * ((S + 127) / 128);
    const int tile = S < 128 ? S : 128, longest = S < rows ? S : rows;
    const long long tiles = packed ? (long long)Hq * ((rows + (long long)tile - 1) / tile) : blocks;
    long long keys = (longest + 127) / 128;  // key tiles of the longest query tile
    if (window > 0 && (window + 254ll) / 128 + 1 < keys) keys = (window + 254ll) / 128 + 1;
    for (int heads = 4; heads > 1; heads /= 2)
        if (heads <= Hq && (tiles >= 6ll * heads * sms || blocks >= heads * sms * (2 * keys + 7))) return heads;
    return 1;
}
cudaError_t launch_fwd(const FwdLaunch& L, cudaStream_t stream);

// ---- backward ---------------------------------------------------------------------------
// Sinks in the backward: the first `sink` keys of a sequence are seen by its every query, the other keys of their tile
// by those of the window alone. The near queries, those of the tile's windows, belong to the tile's own block; the far ones
// are shared out in slices of `rows` queries: to a kernel of their own where the sinks are few enough for its warp MMAs, else to
// blocks of the main kernel, so that none has much more to do than one of the window's. The near block and each slice
// (in its kernel: each share of a slice) leave dV and dK of the sinks as parts in fp32, [part][Hkv][2][sink][D], and a small kernel
// adds them up. Parts of a sequence start at (floor(first row / rows of a slice) + 2 m) x shares, m being the smaller of its number and
// floor(first row / reach): it has at most (floor(length / rows of a slice) + 1) x shares + 1 of them, and a sequence with far queries has more than
// `reach` rows, so that m rises by one at least from one of those to the next. So none overlap, nobody has to count those of the others, and short sequences need no room.
struct SinkSplit {
    float* part;
    int sink;    // 0: none
    int slices;   // far slices of the longest sequence that there may be; 0: no query is far
    int rows;     // queries of a slice
    int shares;   // of the heads of a group, each a block and a part of its own
    int in_main;  // far slices that are blocks of the main kernel: all of them, or none where a kernel of their own has them
    int reach;    // window + 127: a sequence with far queries is longer
    // Bound on the parts of all sequences with far queries.
    __host__ __device__ long long parts(long long total_rows, long long nseq) const {
        const long long m = total_rows / reach;
        return (total_rows / rows + 2 * (m < nseq ? m : nseq)) * shares;
    }
    __host__ __device__ long long first_part(int seq, int start) const {
        const int m = start / reach;
        return (long long)(start / rows + 2 * (m < seq ? m : seq)) * shares;
    }
    __host__ __device__ float* row(int seq, int start, int p, int g, int Hkv, int j, int D) const {
        const size_t at = (size_t)(first_part(seq, start) + p) * Hkv + g;
        return part + (at * 2 * sink + j) * D;
    }
};

struct BwdLaunch {
    CUtensorMap tq, tk, tv, tdo;
    CUtensorMap tqh, tdoh;  // q / dO with a 64 x 1 x (256*128/D) x 1 box: one cluster CTA's query share
    CUtensorMap tdq;  // fp32 dQ accumulator, 4-D [D, Hq, S, B], box 32 x 1 x 128 x 1, 128-byte swizzle
    const uint16_t *q, *k, *v, *o, *dO;
    const float* lse;
    uint16_t *dQ, *dK, *dV;
    float* dq_acc;  // [rows, Hq, D] fp32
    float* delta;   // same layout as lse
    const int32_t* cu_seqlens;
    unsigned* status;
    int nseq, Hq, Hkv, S, D, total_rows, window;
    float scale;
    SinkSplit sink;
};
cudaError_t launch_bwd(const BwdLaunch& L, cudaStream_t stream);
constexpr int kFewSinks = 16;  // sinks that launch_bwd_far_sinks takes at most (and head_dim 256 at most)
cudaError_t launch_bwd_far_sinks(const BwdLaunch& L, cudaStream_t stream);
cudaError_t launch_bwd_sink_sum(const BwdLaunch& L, cudaStream_t stream);
// First far query of a sequence of L tokens (a multiple of 128; L or more: there are none).
__host__ __device__ __forceinline__ int far_from(int L, int window) { return ((127 + window < L ? 127 + window : L) + 127) / 128 * 128; }
// main kernel of the backward at D = 64 / 128 (one CTA per key tile; attn_bwd_small.cu)
template <int D>
cudaError_t launch_bwd_small_main(const BwdLaunch& L, cudaStream_t stream);

// ---- merge of attention results over disjoint key sets -----------------------------------
struct MergeLaunch {
    const uint16_t* o_parts;  // [P, B, S, H, D] bf16
    const float* lse_parts;   // [P, B, H, S]
    uint16_t* o;              // [B, S, H, D]
    float* lse;               // [B, H, S]
    int P, B, S, H, D;        // D in {64, 128, 256, 512}
    int sms;
};
cudaError_t launch_merge_lse(const MergeLaunch& L, cudaStream_t stream);

// ---- plan of a step over a paged cache ------------------------------------------------------
struct PlanLaunch {
    const int32_t *kv_lens, *new_lens, *held, *free_pages, *used;  // used: one value
    int32_t *table;                                                // [R, max_pages]
    int32_t *seq_lens, *cu_q, *positions, *slots, *held_out, *used_out, *admitted;
    unsigned* status;
    int R, T, F, max_pages, num_pages, sms;
    bool in_place;  // seq_lens / held_out / used_out is kv_lens / held / used
};
cudaError_t launch_paged_plan(const PlanLaunch& L, cudaStream_t stream);

// ---- head norm with rotary position encoding -------------------------------------------------
struct NormRopeLaunch {
    const uint16_t *q, *k, *v;          // rows [T] of H x D, token strides below
    const uint16_t *dq_out, *dk_out;    // gradient: of the results, contiguous
    uint16_t *q_out, *k_out, *v_out;    // contiguous; paged: k_out / v_out are the caches
    uint16_t *dq, *dk;                  // gradient: token strides below
    const void *q_weight, *k_weight;    // [D] bf16 or fp32, or null
    float *dq_weight, *dk_weight;       // [D] fp32
    float* part;                        // gradient: [CTAs][2][D]
    const int32_t *positions, *slots;   // slots: paged only
    const float* cos_sin;               // [max_pos, rot]: cos | sin
    unsigned* status;
    long long q_stride, k_stride, v_stride, dq_stride, dk_stride;  // elements
    int T, Hq, Hkv, D, rot, max_pos, num_slots, sms;
    float eps, weight_offset;
    bool weight_fp32, interleaved;
};
int norm_rope_bwd_max_ctas();  // CTAs of the gradient kernel at most
cudaError_t launch_norm_rope(const NormRopeLaunch& L, cudaStream_t stream);
cudaError_t launch_norm_rope_paged(const NormRopeLaunch& L, cudaStream_t stream);
cudaError_t launch_norm_rope_bwd(const NormRopeLaunch& L, cudaStream_t stream);

// ---- attention of drafted token trees over a paged cache --------------------------------------
// tq: 4-D over q [D, Hq, T, 1], box 64 x G x tree_tokens_per_copy x 1; tk / tv as in the paged prefill
struct TreeLaunch {
    CUtensorMap tq, tk, tv;
    const int32_t *block_table, *seq_lens, *cu_q, *mask, *positions;
    uint16_t* o;
    float* lse;
    unsigned* status;
    void* workspace;
    int R, T, max_q, words, Hq, Hkv, D, max_pages, num_pages, window, sms;
    float scale;
};
int tree_tokens_per_copy(int G, int max_q);  // drafted tokens of a copy of Q: those of a 128-row tile, or fewer
size_t tree_workspace_bytes(int G, int max_q, int D);
cudaError_t launch_tree_paged(const TreeLaunch& L, cudaStream_t stream);

// ---- 4-bit paged cache (kv4.cuh): rows in by slot, pages out as bf16 ----------------------------
struct Kv4Launch {
    const uint16_t *k, *v;   // append: rows [n] of Hkv x D, token strides below
    const int32_t* slots;    // append: [n]
    const int32_t* pages;    // unpack: [n]
    uint16_t *k_out, *v_out;  // unpack: [n, 16, Hkv, D]
    uint8_t* cache;          // [num_pages, Hkv, 18 D]
    unsigned* status;
    long long k_stride, v_stride;  // elements
    int n, Hkv, D, num_pages;
};
cudaError_t launch_kv4_append(const Kv4Launch& L, cudaStream_t stream);
cudaError_t launch_kv4_unpack(const Kv4Launch& L, cudaStream_t stream);

struct DecodeKv4Launch {
    const uint16_t* q;
    const uint8_t* cache;
    const int32_t *block_table, *seq_lens;
    uint16_t* o;
    float* lse;
    unsigned* status;
    void* workspace;
    int B, Hq, Hkv, D, max_pages, num_pages, window, sink, grid;
    int max_grid;  // that the workspace is made for
    float scale;
};
size_t decode_kv4_workspace_bytes(int B, int G, int D, int max_grid);
cudaError_t launch_decode_kv4(const DecodeKv4Launch& L, cudaStream_t stream);

}  // namespace attn
