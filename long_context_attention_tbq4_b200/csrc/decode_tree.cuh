// decode_tree.cuh -- attention of a tree of drafted tokens over TBQ4 caches:
// parameters, work schedule and the join of split rows.
//
// Sequence b holds ctx_b cached tokens and, in the slots right behind them,
// the n_b nodes of a draft tree.  Node i sees every cached token and the
// nodes whose bits are set in its mask:
//
//   O_i = sum_t p_it v_t / sum_t p_it,  p_it = exp(scale q_i . k_t),
//   t in [0, ctx_b) and ctx_b + {j < n_b : bit j of mask_bi}
//
// over the raw blocks, in the rotated domain (trefon.com, "Kontekst 262K na
// jednej RTX 4090", section "Od czego zaczalem"; drafted tokens: section
// "Konfiguracja").  A row that sees nothing is 0.
//
// Work.  The G heads of a KV head and the nodes make n_b G query rows that
// read the same keys; they go in blocks of up to kRows rows (row c of the
// sequence's rows = node c / G, head c % G).  A work is one (sequence, KV
// head, row block) over all of its 128-token tiles.  The tiles of all works
// are numbered through, and the grid's CTAs (one per SM) take equal
// consecutive shares, so ragged batches balance whatever the lengths on the
// device are, and one captured launch serves any lengths.  A CTA that holds
// a whole work writes its rows; a work that crosses CTAs leaves one partial
// (O_rot, m, l) per CTA, which tree_combine_kernel joins by log-sum-exp.
#pragma once
#include "common.cuh"
#include "decode.cuh"
#include "rope_append.cuh"

namespace tbq4 {
namespace tree {

constexpr int kTileT = 128;                 // tokens per tile
constexpr int kMaxNodes = 64;
constexpr int kMaxBatch = 1024;             // prefix sums in shared memory

struct TreeParams {
    const void *q;                          // [B][T][Hq][128]
    int q_type;                             // ElemType
    const uint8_t *k, *v;                   // caches or pools
    int64_t capacity;                       // tokens a sequence can hold
    int64_t seq_stride, head_stride;        // bytes (contiguous caches)
    const int32_t *table;                   // nullptr: contiguous
    int max_pages, page_size;
    int64_t n_pages;
    const int32_t *ctx_lens, *n_nodes;      // n_nodes may be nullptr: T
    const unsigned long long *mask;         // [B][T], or [T] with mask_stride 0
    int64_t mask_stride;
    int B, T, Hq, Hkv, G;
    int rows;                               // rows per block
    float scale;
    uint64_t sign_lo, sign_hi;
    float *part_o;                          // [2 n_ctas][rows][128]
    float2 *part_ml;                        // [2 n_ctas][rows]: max (log2 units), sum
    int n_ctas;
    int join_starts;                        // how tree_combine_kernel finds the split works
    void *out;                              // [B][T][Hq][128]
    int out_type;
    int64_t cache_bytes, out_elems;         // extents, for the debug build's bounds checks
};

// Tokens and nodes of sequence b, clamped to what its cache can hold.
__device__ __forceinline__ void seq_extent(const TreeParams &p, int b, int &ctx, int &n) {
    ctx = __ldg(p.ctx_lens + b);
    n = p.n_nodes ? __ldg(p.n_nodes + b) : p.T;
    bool bad = n < 0 || n > p.T || ctx < 0;
    n = min(max(n, 0), p.T);
    ctx = max(ctx, 0);
    if ((int64_t)ctx + n > p.capacity) {
        bad = true;
        n = (int)min((int64_t)n, p.capacity);
        ctx = (int)min((int64_t)ctx, p.capacity - n);
    }
    if (bad) record_status(4u /* TBQ4_ERR_CAPACITY */);
}

// Tiles and row blocks of a sequence with ctx cached tokens and n nodes.
__device__ __forceinline__ int seq_tiles(int ctx, int n) {
    return n > 0 ? (int)(((int64_t)ctx + n + kTileT - 1) / kTileT) : 0;
}
__device__ __forceinline__ int seq_blocks(const TreeParams &p, int n) {
    return (n * p.G + p.rows - 1) / p.rows;
}

// prefix[b] = units (tiles of all works) of the sequences before b, b <= B,
// every thread of the CTA calls it, and warp 0 `then` once they are there.
// The host bounds the total below 2^31.
template <class F>
__device__ __forceinline__ void build_prefix(const TreeParams &p, int *prefix, F then) {
    for (int b = threadIdx.x; b < p.B; b += blockDim.x) {
        int ctx, n;
        seq_extent(p, b, ctx, n);
        prefix[b + 1] = seq_tiles(ctx, n) * seq_blocks(p, n) * p.Hkv;
    }
    if (threadIdx.x == 0) prefix[0] = 0;
    __syncthreads();
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x, per = (p.B + 31) / 32;
        const int b0 = min(lane * per, p.B), b1 = min(b0 + per, p.B);
        int sum = 0;
        for (int b = b0; b < b1; ++b) sum += prefix[b + 1];
        int base = sum;
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const int o = __shfl_up_sync(kFull, base, m);
            if (lane >= m) base += o;
        }
        base -= sum;
        for (int b = b0; b < b1; ++b) {
            base += prefix[b + 1];
            prefix[b + 1] = base;
        }
        __syncwarp();
        then();
    }
    __syncthreads();
}

// CTAs that get a share (each of at least one unit), the first unit of share
// c, and the share that holds unit u.
__device__ __forceinline__ int n_shares(const TreeParams &p, int units) { return min(p.n_ctas, units); }
__device__ __forceinline__ int share_begin(int units, int c, int shares) {
    // units c / shares; the remainder's product is small (shares^2)
    const int each = units / shares, rest = units - each * shares;
    return each * c + rest * c / shares;
}
__device__ __forceinline__ int share_of(int units, int u, int shares) {
    return (int)((((int64_t)u + 1) * shares - 1) / units);
}

// One CTA's run of tiles inside one work.
struct Segment {
    int b, g, blk;                          // sequence, KV head, row block
    int ctx, n;                             // its cached tokens and nodes
    int tile0, tiles;                       // tiles of this run
    int row0, rows;                         // rows of the block
    int begin, work_tiles;                  // the work's first unit, and its units
};

// The segment that starts at unit u and ends at the work's end or at `end`.
__device__ __forceinline__ Segment segment_at(const TreeParams &p, const int *prefix, int u, int end) {
    int lo = 0, hi = p.B - 1;               // the last b with prefix[b] <= u
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (prefix[mid] <= u) lo = mid; else hi = mid - 1;
    }
    Segment s;
    s.b = lo;
    seq_extent(p, s.b, s.ctx, s.n);
    s.work_tiles = seq_tiles(s.ctx, s.n);
    const int blocks = seq_blocks(p, s.n), local = u - prefix[s.b];
    const int w = local / s.work_tiles;
    s.tile0 = local - w * s.work_tiles;
    s.begin = prefix[s.b] + w * s.work_tiles;
    s.tiles = min(s.work_tiles - s.tile0, end - u);
    s.g = w / blocks;
    s.blk = w - s.g * blocks;
    // rows spread evenly over the blocks, in whole eights
    const int all = s.n * p.G, per = ((all + blocks - 1) / blocks + 7) & ~7;
    s.row0 = s.blk * per;
    s.rows = max(0, min(per, all - s.row0));
    return s;
}
// Where a partial of CTA c goes: its first run when that starts inside a
// work, its last when that ends inside one.
__device__ __forceinline__ int part_slot(const Segment &s, int c) { return 2 * c + (s.tile0 == 0); }

// o = D H o_rot / sqrt(128) of one normalised row held four values per lane,
// rounded to the output's type and stored (row c of the work's sequence).
__device__ __forceinline__ void store_out(const TreeParams &p, int b, int g, int c, float (&v)[4],
                                          int lane) {
    warp_fwht128(v, lane);
    const uint32_t sbits = lane_sign_bits(p.sign_lo, p.sign_hi, lane);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        v[k] *= rot_c();
        if ((sbits >> k) & 1u) v[k] = -v[k];
    }
    const int i = c / p.G, h = g * p.G + (c - i * p.G);
    const int64_t oi = (((int64_t)b * p.T + i) * p.Hq + h) * kD + 4 * lane;
    if (in_extent(oi, 4, p.out_elems)) store4(p.out, p.out_type, oi, v);
}

// Joins the works that cross CTAs.  Few works: grid.x numbers them (sequence,
// KV head, row block).  More works than shares (p.join_starts): grid.x walks
// the starts of shares 1 .. instead; a start that lies inside a work, and is
// the first such start, owns the work.  Either way at most one CTA column per
// split work does anything (walking the starts of 148 shares for the four
// works of one sequence took 17 to 39 us, mostly CTAs that found nothing).
// A CTA's warps share the work's partials: four warps per row where it has
// more than kJoinMany, else one, and rows in turn.  A warp takes its partials'
// maxima and sums first, a lane each, then the rows, kJoinBatch in flight; the
// warps of a row meet in shared memory.  (kJoinMany 64, so that hardly any row
// has four: 16 nodes at 262K 87.2 us instead of 83.8, 1 node at 32K 20.0 instead
// of 18.4; 8: 64 nodes 252.9 instead of 244.3; 4: also 8 trees of 25 nodes 238.6
// instead of 226.0; 32 is as good as 16.  A running maximum over partials read
// one by one cost 10 us more on the long sequences.)
constexpr int kJoinWarps = 16, kJoinMany = 16, kJoinBatch = 8;

__global__ void __launch_bounds__(kJoinWarps * 32)
tree_combine_kernel(const __grid_constant__ TreeParams p) {
    __shared__ int prefix[kMaxBatch + 1];
    __shared__ float4 o_s[kJoinWarps][32];
    __shared__ float2 ml_s[kJoinWarps];
    // the schedule follows from the lengths: inputs, not results of the kernel
    // before, so it is worked out while that one still runs
    build_prefix(p, prefix, [] {});
    const int units = prefix[p.B], shares = n_shares(p, units);
    int u = -1;                             // a unit of the work
    if (p.join_starts) {
        if ((int)blockIdx.x + 1 < shares) u = share_begin(units, blockIdx.x + 1, shares);
    } else {
        const int most = (p.T * p.G + p.rows - 1) / p.rows;        // blocks of a sequence, at most
        const int blk = blockIdx.x % most, bg = blockIdx.x / most;
        const int b = bg / p.Hkv, g = bg - b * p.Hkv;
        int ctx, n;
        seq_extent(p, b, ctx, n);
        const int blocks = seq_blocks(p, n);
        if (blk < blocks) u = prefix[b] + (g * blocks + blk) * seq_tiles(ctx, n);
    }
    Segment s = {};
    int first = 0, last = 0;
    if (u >= 0) {
        s = segment_at(p, prefix, u, units);
        first = share_of(units, s.begin, shares);
        last = share_of(units, s.begin + s.work_tiles - 1, shares);
    }
    // every CTA waits, also one that then has nothing to do: a kernel after
    // this one may start once this grid has ended
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (first == last) return;              // none, or whole: its CTA wrote the rows
    if (p.join_starts && (u == s.begin || first != (int)blockIdx.x)) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int per = last - first >= kJoinMany ? 4 : 1;              // warps per row
    const int sub = warp & (per - 1), step = kJoinWarps / per;
    for (int r0 = blockIdx.y * step; r0 < s.rows; r0 += gridDim.y * step) {
        const int r = r0 + warp / per;
        float M = -INFINITY, L = 0.f;
        float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r < s.rows) {
            // this warp's partials are k = 0 .. n - 1; lane l holds (m, l) of l and l + 32
            const int c0 = first + sub, n = c0 <= last ? (last - c0) / per + 1 : 0;
            auto row_of = [&](int k) {
                const int c = c0 + per * k;
                return (int64_t)(2 * c + (c == first)) * p.rows + r;
            };
            float2 ml[2];
#pragma unroll
            for (int h = 0; h < 2; ++h)
                ml[h] = lane + 32 * h < n ? __ldcg(p.part_ml + row_of(lane + 32 * h)) : make_float2(0.f, 0.f);
            float w[2] = {};
#pragma unroll 1
            for (int k0 = 0; k0 < n; k0 += kJoinBatch) {
                float4 o[kJoinBatch];
#pragma unroll
                for (int k = 0; k < kJoinBatch; ++k)
                    if (k0 + k < n)
                        o[k] = __ldcg(reinterpret_cast<const float4 *>(p.part_o + row_of(k0 + k) * kD) + lane);
                if (k0 == 0) {              // a sum of 0: the run's tokens are all invisible to this row
                    M = warp_max(fmaxf(ml[0].y == 0.f ? -INFINITY : ml[0].x,
                                       ml[1].y == 0.f ? -INFINITY : ml[1].x));
#pragma unroll
                    for (int h = 0; h < 2; ++h) w[h] = ml[h].y == 0.f ? 0.f : exp2f(ml[h].x - M);
                    L = warp_sum(w[0] * ml[0].y + w[1] * ml[1].y);
                }
#pragma unroll
                for (int k = 0; k < kJoinBatch; ++k) {
                    const float f = __shfl_sync(kFull, k0 + k < 32 ? w[0] : w[1], (k0 + k) & 31);
                    if (k0 + k >= n) break;
                    O.x += f * o[k].x;
                    O.y += f * o[k].y;
                    O.z += f * o[k].z;
                    O.w += f * o[k].w;
                }
            }
        }
        float v[4] = {O.x, O.y, O.z, O.w};
        if (per > 1) {
            o_s[warp][lane] = O;
            if (lane == 0) ml_s[warp] = make_float2(M, L);
            __syncthreads();
            if (sub == 0) {
                float Mt = M, f[4];
#pragma unroll
                for (int w = 1; w < 4; ++w) Mt = fmaxf(Mt, ml_s[warp + w].x);
                L = v[0] = v[1] = v[2] = v[3] = 0.f;
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const float2 ml = ml_s[warp + w];
                    const float4 o = o_s[warp + w][lane];
                    f[w] = ml.y == 0.f ? 0.f : exp2f(ml.x - Mt);
                    v[0] += f[w] * o.x;
                    v[1] += f[w] * o.y;
                    v[2] += f[w] * o.z;
                    v[3] += f[w] * o.w;
                    L += f[w] * ml.y;
                }
            }
            __syncthreads();                // o_s is free for the next rows
        }
        if (sub != 0 || r >= s.rows) continue;
        const float inv = L == 0.f ? 0.f : 1.0f / L;
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] *= inv;
        store_out(p, s.b, s.g, s.row0 + r, v, lane);
    }
}

// Byte offset of 32-token piece `t` (a multiple of 32) of (b, g) in either
// cache.  A page id outside the pool reads page 0 and is flagged.
__device__ __forceinline__ int64_t piece_offset(const TreeParams &p, int b, int g, int32_t t) {
    if (!p.table) return b * p.seq_stride + g * p.head_stride + (int64_t)t * kBlockBytes;
    int32_t pid = __ldg(p.table + (int64_t)b * p.max_pages + t / p.page_size);
    if (pid < 0 || (int64_t)pid >= p.n_pages) {
        record_status(4u /* TBQ4_ERR_CAPACITY */);
        pid = 0;
    }
    return (((int64_t)pid * p.Hkv + g) * p.page_size + t % p.page_size) * kBlockBytes;
}

}  // namespace tree
}  // namespace tbq4
