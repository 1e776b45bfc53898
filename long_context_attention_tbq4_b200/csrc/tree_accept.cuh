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

// Shared bytes of one warp: the staged blocks, and source and destination
// offsets of each.
__host__ __device__ constexpr int accept_warp_bytes(int max_path) {
    return max_path * 16 + (max_path * kBlockBytes + 15) / 16 * 16;
}

// One warp per (cache, sequence, KV head).  The warp reads every block it
// moves into shared memory before it writes the first, so the path may be any
// list of nodes (sources and destinations overlap).  A few blocks of 66 bytes
// per warp: latency is all there is to it, four dependent loads (length and
// path, page, block, store), so shared memory is sized by max_path to keep
// the SM full of warps: 28 layers x 64 sequences x 4 heads with paths of up
// to 9 take 16.8 us, 22.2 with room for 64 blocks in every warp (42 KB per
// block of eight) and the path read after the counts.
__global__ void __launch_bounds__(kAcceptWarps * 32)
tree_accept_kernel(const __grid_constant__ AcceptParams p) {
    constexpr int kPieces = kBlockBytes / 2;     // 16-bit pieces per block
    extern __shared__ __align__(16) uint8_t accept_smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t *offs = reinterpret_cast<int64_t *>(accept_smem + warp * accept_warp_bytes(p.max_path));
    uint16_t *stage = reinterpret_cast<uint16_t *>(offs + 2 * p.max_path);
    const int64_t item = (int64_t)blockIdx.x * kAcceptWarps + warp;
    if (item >= (int64_t)p.n_caches * p.B * p.Hkv) return;
    const int c = (int)(item / ((int64_t)p.B * p.Hkv)), rest = (int)(item - (int64_t)c * p.B * p.Hkv);
    const int b = rest / p.Hkv, h = rest - b * p.Hkv;
    const int32_t ctx = __ldg(p.ctx_lens + b);
    int n = __ldg(p.n_accept + b);
    int32_t nodes[2];                            // this lane's entries of the path
#pragma unroll
    for (int k = 0; k < 2; ++k)
        nodes[k] = lane + 32 * k < p.max_path ? __ldg(p.path + (int64_t)b * p.max_path + lane + 32 * k) : 0;
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
            const int32_t pid = __ldg(p.table + (int64_t)b * p.max_pages + (int32_t)slot / p.page_size);
            if (pid < 0 || (int64_t)pid >= p.n_pages) return -1;
            off = (((int64_t)pid * p.Hkv + h) * p.page_size + (int32_t)slot % p.page_size) * kBlockBytes;
        } else {
            off = (((int64_t)b * p.Hkv + h) * p.capacity + slot) * kBlockBytes;
        }
        return in_extent(off, kBlockBytes, p.cache_bytes) ? off : -1;
    };
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int i = lane + 32 * k;
        if (i >= n) continue;
        int64_t src = nodes[k] < 0 ? -1 : block_at((int64_t)ctx + nodes[k]), dst = block_at((int64_t)ctx + i);
        if (src < 0 || dst < 0) {
            record_status(4u /* TBQ4_ERR_CAPACITY */);
            src = dst = -1;
        }
        offs[2 * i] = src;
        offs[2 * i + 1] = dst;
    }
    __syncwarp();
#pragma unroll 4
    for (int e = lane; e < n * kPieces; e += 32) {
        const int64_t src = offs[2 * (e / kPieces)];
        if (src >= 0) stage[e] = *reinterpret_cast<const uint16_t *>(cache + src + 2 * (e % kPieces));
    }
    __syncwarp();
#pragma unroll 4
    for (int e = lane; e < n * kPieces; e += 32) {
        const int64_t dst = offs[2 * (e / kPieces) + 1];
        if (dst >= 0) *reinterpret_cast<uint16_t *>(cache + dst + 2 * (e % kPieces)) = stage[e];
    }
}

}  // namespace tbq4
