// tree_accept.cuh -- after a draft tree has been verified: the accepted
// nodes' blocks move to the front of the drafted region, in the caches of
// every layer, and the new lengths are counted.
//
//   new block[ctx_b + i] = old block[ctx_b + path_b[i]],  i < n_accept_b
//   new_len_b = ctx_b + n_accept_b
//
// Blocks are moved as bytes.  A key keeps the rotary position it was encoded
// with, which for a path node is ctx_b + its depth: its new slot.
#pragma once
#include "common.cuh"

namespace tbq4 {

constexpr int kAcceptLayers = 64;                // layers per launch (pointers in the parameters)
constexpr int kMaxAcceptLayers = 1024;          // layers per call
constexpr int kMaxPath = 64;
constexpr int kAcceptWarps = 8;

struct AcceptParams {
    uint8_t *cache[2 * kAcceptLayers];           // K and V of each layer
    int n_caches, B, Hkv, max_path;
    int64_t capacity;
    const int32_t *ctx_lens, *path, *n_accept;
    const int32_t *table;                        // nullptr: contiguous caches
    int max_pages, page_size;
    int64_t n_pages;
    int32_t *new_lens;                           // nullptr: not wanted (or not this launch's)
    int64_t cache_bytes;                         // extent, for the debug build's bounds checks
};

// One warp per (cache, sequence, KV head).  The warp reads every block it
// moves into shared memory before it writes the first, so the path may be any
// list of nodes (sources and destinations overlap).  Latency is all there is
// to it: a few blocks of 66 bytes per warp.
__global__ void __launch_bounds__(kAcceptWarps * 32)
tree_accept_kernel(const __grid_constant__ AcceptParams p) {
    constexpr int kPieces = kBlockBytes / 2;     // 16-bit pieces per block
    __shared__ uint16_t stage[kAcceptWarps][kMaxPath * kPieces];
    __shared__ int64_t offs[kAcceptWarps][2 * kMaxPath];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t item = (int64_t)blockIdx.x * kAcceptWarps + warp;
    if (item >= (int64_t)p.n_caches * p.B * p.Hkv) return;
    const int h = (int)(item % p.Hkv), b = (int)(item / p.Hkv % p.B);
    const int c = (int)(item / p.Hkv / p.B);
    const int32_t ctx = __ldg(p.ctx_lens + b);
    int n = __ldg(p.n_accept + b);
    if (n < 0 || n > p.max_path || ctx < 0 || (int64_t)ctx + n > p.capacity) {
        if (lane == 0) record_status(4u /* TBQ4_ERR_CAPACITY */);
        n = 0;                                   // nothing moves
    }
    if (p.new_lens && c == 0 && h == 0 && lane == 0) p.new_lens[b] = ctx + n;
    uint8_t *cache = p.cache[c];
    // byte offset of a slot's block, -1 where there is none
    auto block_at = [&](int64_t slot) -> int64_t {
        if (slot < 0 || slot >= p.capacity) return -1;
        int64_t off;
        if (p.table) {
            const int32_t pid = __ldg(p.table + (int64_t)b * p.max_pages + slot / p.page_size);
            if (pid < 0 || (int64_t)pid >= p.n_pages) return -1;
            off = (((int64_t)pid * p.Hkv + h) * p.page_size + slot % p.page_size) * kBlockBytes;
        } else {
            off = (((int64_t)b * p.Hkv + h) * p.capacity + slot) * kBlockBytes;
        }
        return in_extent(off, kBlockBytes, p.cache_bytes) ? off : -1;
    };
    for (int i = lane; i < n; i += 32) {
        const int32_t node = __ldg(p.path + (int64_t)b * p.max_path + i);
        int64_t src = node < 0 ? -1 : block_at((int64_t)ctx + node), dst = block_at((int64_t)ctx + i);
        if (src < 0 || dst < 0) {
            record_status(4u /* TBQ4_ERR_CAPACITY */);
            src = dst = -1;
        }
        offs[warp][2 * i] = src;
        offs[warp][2 * i + 1] = dst;
    }
    __syncwarp();
    for (int e = lane; e < n * kPieces; e += 32) {
        const int64_t src = offs[warp][2 * (e / kPieces)];
        if (src >= 0)
            stage[warp][e] = *reinterpret_cast<const uint16_t *>(cache + src + 2 * (e % kPieces));
    }
    __syncwarp();
    for (int e = lane; e < n * kPieces; e += 32) {
        const int64_t dst = offs[warp][2 * (e / kPieces) + 1];
        if (dst >= 0)
            *reinterpret_cast<uint16_t *>(cache + dst + 2 * (e % kPieces)) = stage[warp][e];
    }
}

}  // namespace tbq4
