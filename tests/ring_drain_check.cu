// One warp walks `tokens` copies of `bytes` each through a ring of `depth` stages, as the head norm's kernels do, and
// leaves the loop before copy `stop` as they do when a wait is given up: without having waited for it. What ring_drain
// is meant to wait for is then read out of the ring at once. out [tokens][bytes]: everything that was read.
#include "ptx.cuh"

namespace {

__global__ void ring_drain_kernel(const uint8_t* src, uint8_t* out, unsigned* status, int tokens, int bytes, int depth, int stop) {
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ uint64_t full[8];
    __shared__ int aborted;
    const int lane = threadIdx.x;
    for (int i = lane; i < depth * bytes; i += 32) ring[i] = 0xff;
    if (lane == 0) {
        aborted = 0;
        for (int s = 0; s < 8; ++s) attn::mbar_init(attn::smem_u32(&full[s]), 1);
        attn::fence_mbar_init();
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    __syncwarp();
    auto fetch = [&](int t, int s) {
        attn::mbar_expect_tx(attn::smem_u32(&full[s]), bytes);
        attn::bulk_load(attn::smem_u32(ring + s * bytes), src + (size_t)t * bytes, bytes, attn::smem_u32(&full[s]));
    };
    if (lane == 0)
        for (int s = 0; s < depth && s < tokens; ++s) fetch(s, s);
    auto read = [&](int t, int s) {
        for (int i = lane; i < bytes; i += 32) out[(size_t)t * bytes + i] = reinterpret_cast<volatile uint8_t*>(ring)[s * bytes + i];
    };
    int stage = 0, phase = 0, t = 0;
    for (; t < tokens && t < stop; ++t) {
        if (!__all_sync(0xffffffffu, attn::mbar_wait(attn::smem_u32(&full[stage]), phase, &aborted, status, 1))) return;
        read(t, stage);
        __syncwarp();
        if (lane == 0 && t + depth < tokens) fetch(t + depth, stage);
        if (++stage == depth) stage = 0, phase ^= 1;
    }
    if (lane == 0) attn::ring_drain(full, stage, phase, depth, tokens - t, status, 2);
    __syncwarp();
    for (int n = 0; n < depth && t + n < tokens; ++n) read(t + n, (stage + n) % depth);
}

}  // namespace

extern "C" int ring_drain_check(const void* src, void* out, unsigned* status, int tokens, int bytes, int depth, int stop) {
    if (depth < 1 || depth > 8 || bytes < 16 || bytes % 16 || depth * bytes > 160 * 1024) return -1;
    cudaError_t e = cudaFuncSetAttribute(ring_drain_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, depth * bytes);
    if (e != cudaSuccess) return (int)e;
    ring_drain_kernel<<<1, 32, depth * bytes>>>(static_cast<const uint8_t*>(src), static_cast<uint8_t*>(out), status, tokens, bytes,
                                                depth, stop);
    return (int)cudaGetLastError();
}
