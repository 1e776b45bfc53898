// decode_tree_tc.cuh -- tree attention over TBQ4 caches on the tensor cores
// (tcgen05); the operator, its work schedule and its join are in
// decode_tree.cuh.
//
// Per tile of 128 tokens and a block of N query rows (N <= 128):
//
//   S^T (128 tokens x N) = K (128 x 128, fp16 levels, tensor memory) . Q^T
//   O^T (128 dims x N)  += V^T (128 dims x 128 tokens, fp16 levels) . P'^T
//
// Tokens are the rows of S^T and dimensions the rows of O^T, so the width of
// both products is the number of query rows: a small tree pays for its own
// rows only.  Operands:
//   K     levels (2n - 15) 2^-11, exact in fp16 (nibbles masked into
//         subnormals, one HFMA2); the block scales stay out of the products.
//         A word of nibbles gives eight levels in the order 0 4 1 5 2 6 3 7,
//         which is the order of the dimensions in every operand here.  K goes
//         from registers to tensor memory, thread = token = lane.
//   V     levels times the power of two of their block's scale, S_v = m 2^e
//         with m in [1, 2): (2n - 15) 2^(e-7), exact in fp16 for every e (-14
//         .. 15; smaller scales are subnormal and keep e = -14, m < 1).  V goes
//         to shared memory as it lies, token by token, and enters as the
//         MN-major operand (no transposition anywhere).
//   Q     q_rot times a power of two that brings the block's largest finite
//         channel below 2^15.  kTerms = 2 adds the remainder as a second fp16
//         term.  Where a row's largest channel lies more than 2^14 below the
//         block's (a row may hold anything in a padded tree), each row takes a
//         power of two of its own, and the softmax puts it back into S: a row's
//         channels are rounded by 2^-25 of its own largest at worst, 2^-11 (or
//         2^-22) relative above that.
//   P'    p m 2^8 <= 2^15 (p <= 2^6), thread = token writes eight rows per
//         16-byte store (MN-major).  The scale's power of two lies in V's
//         levels, so what a weight is rounded to depends on its own row and
//         token only: 2^-11 relative, or 2^-25 where P' is subnormal.  A row's
//         largest weight is at least 2^-4 (kHeadroom), so that is 2^-29 of the
//         row's largest weight (times S_v, or 2^-14 if that is more).  (One
//         power of two for all tokens, from the largest V scale among them, had
//         rows lose bits to tokens that their mask hid.)  kTerms = 2 adds the
//         remainder as a second term, times 2^11 and with an accumulator of its
//         own: 2^-22 relative, or 2^-40 of the row's largest weight.  (Added to
//         O itself, the remainder is subnormal where P' < 2^-3: 32,767 tokens
//         20 below a token without V, which make the row, were 6 % off.)
// One term rounds a query or a weight by up to 2^-11 relative: an eighth of what
// a bf16 query and a bf16 output are rounded by themselves.  It is taken where
// both are bf16 (rel-L2 against 64 bits 1.69e-3 to 1.79e-3 where an fp32
// computation rounded to bf16 has 1.64e-3 to 1.67e-3, most of it the queries').
// Everything else takes two terms (22 bits), in blocks of 64 rows in the same
// shared memory: sharp rows of fp32 queries lose more to an 11-bit query than to
// a bf16 output.  Two terms throughout, bf16 at 262K in a graph: 5 nodes 76 us
// instead of 68, 16 nodes 156 instead of 84, 64 nodes 434 instead of 242.
//
// Softmax.  thread = token, so its S_k and S_v are scalars and a row's
// running maximum is one number for all threads (shared memory).  The
// maximum moves only when a logit exceeds it by 6 in log2 units: one
// barrier-with-vote per warpgroup and tile decides that, and the rare path
// takes the tile's maxima and rescales O (see soft_tile).  Sums stay in
// registers until the end.  Tiles that hold drafted nodes or the end of the
// sequence apply masks by select, to logits and to weights (a hidden block may
// hold anything).
//
// Warps (28): 0 producer (cp.async.bulk, 32-token pieces), 1 tensor-memory
// allocation and every tcgen05.mma, 2 block scales, 3 masks, 4-7 and 8-11
// levels (K and V of the even and of the odd tiles), 12-27 softmax (four
// warpgroups of 32 rows each; those without rows sleep until the block is
// done).  Every role is bound by latency rather than by a unit, hence that many
// warps and the two level groups.
// The softmax waits for one barrier per tile: QK(j) is issued once levels and
// scales of tile j are there, and its commit covers PV(j - 2), which read the
// P' buffer that the softmax will write.
// Hand-offs are mbarriers with bounded waits; a warp whose wait runs out
// records the error and goes on without waiting, so the named barriers of
// its warpgroup and of the CTA always fill.
#pragma once
#include "decode_mq.cuh"
#include "decode_tree.cuh"
#include "tcgen05.cuh"

namespace tbq4 {
namespace tree {

constexpr int kTcThreads = 896;
constexpr int kSoftWarp0 = 12, kSoftWarps = 16;
constexpr int kRaw = 3;                                 // raw tiles in flight, K and V each
constexpr int kRawTile = kTileT * kBlockBytes;          // 8448
constexpr int kRawStride = kRawTile + 16;
constexpr int kSig = 4;                                 // tiles whose scales are kept
constexpr uint32_t kSpinTree = 1u << 22;
// Growth that a row's maximum is left behind by (log2 units), and the power of
// two of P': 2^(kGrow + 1 + kPShift) is in fp16's range.  8 and 6 take 1 % less
// time at 64 nodes, 4 and 10 take 1 % more; a weight's floor moves with kPShift.
constexpr float kGrow = 6.0f;
constexpr int kPShift = 8;
constexpr float kLowest = -3e38f;                       // running maximum before any token
// Room left above a maximum when it is moved (log2 units): the next keys are
// often a little larger, and moving costs a tile's time.
constexpr float kHeadroom = 4.0f;
// registers per thread by warpgroup: control, levels (2), softmax (4)
// (setmaxnreg draws on what the block was launched with: the host refuses to
// launch a build that compiled to fewer than kLaunchRegs)
constexpr uint32_t kRegCtl = 40, kRegLev = 40, kRegSoft = 96;
constexpr int kLaunchRegs = 72;
static_assert(4 * kRegCtl + 8 * kRegLev + 16 * kRegSoft <= 28 * kLaunchRegs, "register split");

constexpr int kOffQ = 0;                                // 32 KB: kTerms x rows x 256 B
constexpr int kOffP = 32768;                            // 2 x 32 KB: kTerms x rows/64 x 16 KB
constexpr int kOffV = kOffP + 2 * 32768;                // 2 x 32 KB
constexpr int kOffRawK = kOffV + 2 * 32768;
constexpr int kOffRawV = kOffRawK + kRaw * kRawStride;
constexpr int kOffSig = kOffRawV + kRaw * kRawStride;   // S_k, m 2^kPShift: [2][4][128] floats
constexpr int kOffNegM = kOffSig + 2 * kSig * kTileT * 4;  // minus the running maxima [128]
constexpr int kOffXch = kOffNegM + 128 * 4;             // [4][128] floats
constexpr int kOffLinv = kOffXch + 4 * 128 * 4;         // [128] floats
constexpr int kOffFactor = kOffLinv;                    // [128] floats, before those
constexpr int kOffRow = kOffLinv + 128 * 4;             // [128]: a row's largest |q_rot|, then its power of two
constexpr int kOffVis = kOffRow + 128 * 4;              // [64 nodes][4] words: rows that see it
constexpr int kOffSegment = kOffVis + kMaxNodes * 16;   // the first Segment, the CTA's units
constexpr int kOffQMax = kOffSegment + 56;              // bits of the largest |q_rot|, of the least row's
constexpr int kOffTmem = kOffQMax + 8;
constexpr int kOffBars = kOffTmem + 8;
constexpr int kTreeBars = 2 * kRaw + 10 + 1;
constexpr int kOffPrefix = kOffBars + kTreeBars * 8;
constexpr int kTcSmem = kOffPrefix + (kMaxBatch + 1) * 4 + 1024;   // + alignment slack
static_assert(kOffRawK % 16 == 0 && kRawStride % 16 == 0 && kOffBars % 8 == 0 && kOffVis % 16 == 0,
              "alignment");
static_assert(kTcSmem <= 232448 && sizeof(Segment) + 8 <= 56, "shared memory");

// tensor memory columns: S (two buffers of 128), O, K levels (two of 64)
// (kTerms = 2: S takes 64 columns, and the remainders' O those behind it)
constexpr uint32_t kColS = 0, kColO = 256, kColK = 384, kColO2 = 64;
constexpr float kLowTerm = 2048.0f;

__device__ __forceinline__ void named_sync(int id, int threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ bool named_or(int id, int threads, bool x) {
    uint32_t r;
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.u32 p, %3, 0;\n bar.red.or.pred q, %1, %2, p;\n"
        " selp.u32 %0, 1, 0, q;\n}\n"
        : "=r"(r)
        : "r"(id), "r"(threads), "r"((uint32_t)x)
        : "memory");
    return r != 0;
}
__device__ __forceinline__ float warp_redux_max(float x) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ uint32_t half2_bits(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// Eight levels (2n - 15) 2^-11 of a word of nibbles, as four fp16 pairs: the
// nibbles 0 4 1 5 2 6 3 7 (dmq::vlo, dmq::vhi).
__device__ __forceinline__ void word_levels(uint32_t w, uint32_t (&o)[4]) {
    o[0] = dmq::vlo(w);
    o[1] = dmq::vhi(w);
    o[2] = dmq::vlo(w >> 8);
    o[3] = dmq::vhi(w >> 8);
}
// The same nibbles as (2n - 15) 2^(e-7) for a block scale's power of two 2^e,
// given as its fp16 bits twice: with n moved into the mantissa of 1 + n / 64,
// that is 2^e (1 + n / 64) - 143 2^(e-7), one HFMA2 with exact operands.
__device__ __forceinline__ void word_levels_scaled(uint32_t w, uint32_t pow2, uint32_t (&o)[4]) {
    const uint32_t less = pow2 | 0x80788078u;             // -143 2^(e-7)
    auto level = [&](uint32_t x) { return dmq::hfma2u((x & 0x00F000F0u) | 0x3C003C00u, pow2, less); };
    o[0] = level(w << 4);
    o[1] = level(w);
    o[2] = level(w >> 4);
    o[3] = level(w >> 8);
}
// Exponent field of a block scale's power of two: at least that of 2^-14, and
// finite also where the scale is not.
__device__ __forceinline__ uint32_t scale_field(uint32_t half_bits) {
    return min(max((half_bits >> 10) & 31u, 1u), 30u);
}
// Dimension at position `pos` of an operand: the order above, by eights.
__device__ __forceinline__ int dim_at(int pos) {
    return (pos & ~7) | ((pos & 1) << 2) | ((pos & 7) >> 1);
}

// Sum over the warp of 32 values per lane: lane l gets the sum of v[l].
__device__ __forceinline__ float transpose_sum(float (&v)[32], int lane) {
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) {
        const bool up = (lane & m) != 0;
#pragma unroll
        for (int k = 0; k < m; ++k) {
            const float give = up ? v[k] : v[k + m], keep = up ? v[k + m] : v[k];
            v[k] = keep + __shfl_xor_sync(kFull, give, m);
        }
    }
    return v[0];
}

__device__ __forceinline__ float4 lds128f(uint32_t a) {
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ float ldsf(uint32_t a) { return __uint_as_float(dmq::lds32(a)); }
__device__ __forceinline__ void stsf(uint32_t a, float x) {
    asm volatile("st.shared.f32 [%0], %1;" ::"r"(a), "f"(x) : "memory");
}

// Arrivals that complete a P' tile: each of the 4 n warps of the n
// warpgroups with rows counts 12 / n.
constexpr uint32_t kPArrivals = 48;
__device__ __forceinline__ void mbar_arrive_n(uint32_t bar, uint32_t count) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}

// Bounded wait of one warp: false once one has run out, and from then on at
// once (the error is recorded the first time).  Each poll suspends the warp
// for up to kPollNs, or returns when the phase completes.
constexpr uint32_t kPolls = 1u << 20, kPollNs = 2000;
__device__ __forceinline__ void wait_or_fail(bool &ok, uint32_t bar, uint32_t parity) {
    if (!ok || __all_sync(kFull, mbar_test(bar, parity))) return;
    uint32_t left;
    asm volatile(
        "{\n .reg .pred p;\n mov.u32 %0, %3;\n"
        "WAIT:\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %4;\n"
        " @p bra DONE;\n sub.u32 %0, %0, 1;\n setp.ne.u32 p, %0, 0;\n @p bra WAIT;\n"
        "DONE:\n}\n"
        : "=&r"(left)
        : "r"(bar), "r"(parity), "n"(kPolls), "r"(kPollNs)
        : "memory");
    if (!__all_sync(kFull, left != 0)) {
        ok = false;
        record_status(7u /* TBQ4_ERR_DEVICE_TIMEOUT */);
    }
}

// What a softmax thread keeps across the tiles of a segment.
struct Soft {
    uint32_t sbase, tmem, bx;               // shared memory, tensor memory, first hand-off barrier
    int t, lane, wg;                        // token of the tile, lane, warpgroup
    uint32_t weight;                        // what its arrival counts (kPArrivals)
    float c2;                               // log2 logit = S S_k c2
    bool spread;                            // S is yet to be multiplied by its rows' powers of two
};

// S of a tile by its rows' powers of two, in place.
template <int kN>
__device__ __forceinline__ void spread_rows(const Soft &c, int it, bool &ok) {
    const int b = it & 1;
    wait_or_fail(ok, c.bx + 8 * (2 + b), (it >> 1) & 1);
    tc::fence_after_sync();
#pragma unroll 1
    for (int i = 0; i < kN; ++i) {
        const uint32_t col = c.tmem + ((uint32_t)(c.t & ~31) << 16) + kColS + 128 * b + 32 * c.wg + 8 * i;
        uint32_t r[8];
        tc::tmem_ld8(col, r);
        tc::tmem_wait_ld();
#pragma unroll
        for (int k = 0; k < 8; ++k)
            r[k] = __float_as_uint(__uint_as_float(r[k]) *
                                   ldsf(c.sbase + kOffRow + 128 * c.wg + 32 * i + 4 * k));
        tc::tmem_st8(col, r);
    }
    tc::tmem_wait_st();
}

// One tile for kN chunks of 8 rows (rows 32 wg + 8 i ..).  The weights are
// taken with the running maxima as they are, stored, and only then does the
// warpgroup vote on whether a logit exceeded its maximum by more than kGrow
// (a weight above 2^6, which fp16 may not hold): the rare tile that did is
// stored again with the new maxima.  The sums take that without a second
// pass: fp32 holds weights of up to 2^127, so they are scaled afterwards, and
// where a maximum rose by more than 64 the old sum no longer counts.  (Voting
// first kept 32 logits a thread in registers across the barrier and spilled.)
// kMasked: the tile holds drafted nodes or ends the sequence; `node` is then
// this token's node (below 0: context).
template <int kTerms, int kN, bool kMasked>
__device__ __forceinline__ void soft_tile(const Soft &c, int it, bool first, int node, int n_nodes,
                                          float (&lp)[8 * kN], bool &ok) {
    const int b = it & 1, sg = it & (kSig - 1);
    wait_or_fail(ok, c.bx + 8 * (2 + b), (it >> 1) & 1);           // S, and the scales with it
    tc::fence_after_sync();
    const uint32_t q_lane = (uint32_t)(c.t & ~31) << 16;
    const uint32_t s_col = c.tmem + q_lane + kColS + 128 * b + 32 * c.wg;
    const float skc = ldsf(c.sbase + kOffSig + (kTileT * sg + c.t) * 4) * c.c2;
    const float m8 = ldsf(c.sbase + kOffSig + (kTileT * (kSig + sg) + c.t) * 4);
    uint32_t see = 0xFFFFFFFFu;                                    // rows that see this token
    if (kMasked && node >= 0)
        see = node < n_nodes ? dmq::lds32(c.sbase + kOffVis + 16 * node + 4 * c.wg) : 0u;
    auto sees = [&](int i, int k) -> bool { return !kMasked || ((see >> (8 * i + k)) & 1u); };
    // 16-byte chunk x of a P' row lies at x ^ (t % 8); this warpgroup's are
    // 4 (wg % 2) + i of the 64-row atom wg / 2
    const uint32_t pt = c.sbase + kOffP + 32768 * b + (c.wg >> 1) * 16384 + c.t * 128 +
                        ((((c.wg & 1) << 2) ^ (c.t & 7)) << 4);
    // P' = p m 2^8 of chunk i
    auto store = [&](int i, const float (&pr)[8]) {
        float y[8];
#pragma unroll
        for (int k = 0; k < 8; k += 2) {
            unpack2(mul2(pack2(pr[k], pr[k + 1]), pack2(m8, m8)), y[k], y[k + 1]);
            if constexpr (kMasked) {                               // a hidden block may hold anything
                if (!sees(i, k)) y[k] = 0.f;
                if (!sees(i, k + 1)) y[k + 1] = 0.f;
            }
        }
        const uint32_t at = pt ^ (i << 4);
        uint32_t h[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) h[k] = half2_bits(y[2 * k], y[2 * k + 1]);
        dmq::sts128(at, h[0], h[1], h[2], h[3]);
        if constexpr (kTerms == 2) {
            uint32_t lo[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h[k]));
                lo[k] = half2_bits((y[2 * k] - f.x) * kLowTerm, (y[2 * k + 1] - f.y) * kLowTerm);
            }
            dmq::sts128(at + 16384, lo[0], lo[1], lo[2], lo[3]);
        }
    };
    // the first tile has no maxima to go by: it takes the rare path at once
    float top = first ? INFINITY : -INFINITY;
    if (!first) {
#pragma unroll
        for (int i0 = 0; i0 < kN; i0 += 2) {
            float r[16];
            tc::tmem_ld16(s_col + 8 * i0, r);
            tc::tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int i = i0 + e;
                const uint32_t nega = c.sbase + kOffNegM + 128 * c.wg + 32 * i;
                const float4 n0 = lds128f(nega), n1 = lds128f(nega + 16);
                const float nm[8] = {n0.x, n0.y, n0.z, n0.w, n1.x, n1.y, n1.z, n1.w};
                float x[8];                                            // log2 p: S skc - m, hidden ones -inf
#pragma unroll
                for (int k = 0; k < 8; k += 2) {
                    unpack2(fma2(pack2(r[8 * e + k], r[8 * e + k + 1]), pack2(skc, skc),
                                 pack2(nm[k], nm[k + 1])), x[k], x[k + 1]);
                    if (!sees(i, k)) x[k] = -INFINITY;
                    if (!sees(i, k + 1)) x[k + 1] = -INFINITY;
                }
#pragma unroll
                for (int k = 0; k < 8; ++k) top = fmaxf(top, x[k]);
#pragma unroll
                for (int k = 0; k < 8; ++k) x[k] = tc::ex2(x[k]);
#pragma unroll
                for (int k = 0; k < 8; k += 2)
                    unpack2(add2(pack2(lp[8 * i + k], lp[8 * i + k + 1]), pack2(x[k], x[k + 1])),
                            lp[8 * i + k], lp[8 * i + k + 1]);
                store(i, x);
            }
        }
    }
    if (__builtin_expect(named_or(4 + c.wg, 128, top > kGrow), 0)) {
        // move the maxima to the tile's; lane 8 i + k stands for row k of chunk i
        float keep = kLowest;
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            uint32_t r[8];
            tc::tmem_ld8(s_col + 8 * i, r);
            tc::tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float m = warp_redux_max(sees(i, k) ? __fmul_rn(__uint_as_float(r[k]), skc) : -INFINITY);
                if (c.lane == 8 * i + k) keep = m;
            }
        }
        const uint32_t row = 32 * c.wg + c.lane;
        const bool mine = c.lane < 8 * kN;
        const uint32_t xch = c.sbase + kOffXch + 4 * row, neg = c.sbase + kOffNegM + 4 * row;
        if (mine) stsf(xch + 512 * (c.t >> 5), keep);
        named_sync(4 + c.wg, 128);
        float f_mine = 1.f, nmx = 0.f;
        if (mine) {
            const float old = -ldsf(neg);
            const float tm = fmaxf(fmaxf(ldsf(xch), ldsf(xch + 512)),
                                   fmaxf(ldsf(xch + 1024), ldsf(xch + 1536)));
            nmx = tm > old ? tm + kHeadroom : old;
            f_mine = nmx - old > 64.0f ? 0.f : tc::ex2(old - nmx);
        }
        named_sync(4 + c.wg, 128);
        if (mine && c.t < 32) {
            stsf(neg, -nmx);
            stsf(c.sbase + kOffFactor + 4 * row, f_mine);
        }
        named_sync(4 + c.wg, 128);
        if (!first) wait_or_fail(ok, c.bx + 8 * (8 + ((it - 1) & 1)), ((it - 1) >> 1) & 1);
        tc::fence_after_sync();
        // this token's weights once more, the sums and O by 2^-rise
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            uint32_t r[8], o[8] = {};
            const uint32_t col = c.tmem + q_lane + kColO + 32 * c.wg + 8 * i;
            tc::tmem_ld8(s_col + 8 * i, r);
            if (!first) tc::tmem_ld8(col, o);
            const uint32_t at = 128 * c.wg + 32 * i;
            const float4 n0 = lds128f(c.sbase + kOffNegM + at), n1 = lds128f(c.sbase + kOffNegM + at + 16);
            const float4 f0 = lds128f(c.sbase + kOffFactor + at), f1 = lds128f(c.sbase + kOffFactor + at + 16);
            const float nm[8] = {n0.x, n0.y, n0.z, n0.w, n1.x, n1.y, n1.z, n1.w};
            const float f[8] = {f0.x, f0.y, f0.z, f0.w, f1.x, f1.y, f1.z, f1.w};
            tc::tmem_wait_ld();
            float x[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                // the rounded product, as the maximum was taken from: unrounded, it
                // exceeds a large maximum by more than fp16 weights allow
                x[k] = sees(i, k) ? tc::ex2(__fadd_rn(__fmul_rn(__uint_as_float(r[k]), skc), nm[k])) : 0.f;
                lp[8 * i + k] = f[k] == 0.f ? x[k] : lp[8 * i + k] * f[k];
                o[k] = __float_as_uint(__uint_as_float(o[k]) * f[k]);
            }
            if (!first) tc::tmem_st8(col, o);
            store(i, x);
        }
        if constexpr (kTerms == 2) {
            if (!first) {
                // a rolled loop of its own: inside the one above, the spills that it
                // brings reach the frequent path (5 nodes at 262K 153 us instead of 76)
#pragma unroll 1
                for (int i = 0; i < kN; ++i) {
                    uint32_t o[8];
                    const uint32_t col = c.tmem + q_lane + kColO2 + 32 * c.wg + 8 * i;
                    tc::tmem_ld8(col, o);
                    tc::tmem_wait_ld();
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        o[k] = __float_as_uint(__uint_as_float(o[k]) *
                                               ldsf(c.sbase + kOffFactor + 128 * c.wg + 32 * i + 4 * k));
                    tc::tmem_st8(col, o);
                }
            }
        }
        tc::tmem_wait_st();
    }
    fence_proxy_async();                                           // read by the tensor core
    tc::fence_before_sync();
    __syncwarp();
    if (c.lane == 0) mbar_arrive_n(c.bx + 8 * (4 + b), c.weight);
}

// The tiles of a segment, and each row's sum into xch[quarter][row].  A
// loop for the tiles that every row sees in full and one for the last one or
// two, so that the frequent one is short straight code.  Rows with powers of
// two of their own are rare and take the second throughout.  (A test in every
// tile took 4 % at 5 nodes, products in both loops 3 %: registers.)
template <int kTerms, int kN>
__device__ __forceinline__ void soft_segment(const Soft &c, int it, int tiles, int t0, int ctx,
                                             int n_nodes, bool &ok) {
    float lp[8 * kN];
#pragma unroll
    for (int k = 0; k < 8 * kN; ++k) lp[k] = 0.f;
    const int full = c.spread ? 0 : min(tiles, max(0, (ctx - t0) / kTileT));
    int j = 0;
#pragma unroll 1
    for (; j < full; ++j) soft_tile<kTerms, kN, false>(c, it + j, j == 0, 0, 0, lp, ok);
#pragma unroll 1
    for (; j < tiles; ++j) {
        if (c.spread) spread_rows<kN>(c, it + j, ok);
        soft_tile<kTerms, kN, true>(c, it + j, j == 0, t0 + j * kTileT + c.t - ctx, n_nodes, lp, ok);
    }
    float v[32];
#pragma unroll
    for (int k = 0; k < 32; ++k) v[k] = k < 8 * kN ? lp[k < 8 * kN ? k : 0] : 0.f;
    const float sum = transpose_sum(v, c.lane);
    if (c.lane < 8 * kN)
        stsf(c.sbase + kOffXch + 512 * (c.t >> 5) + 4 * (32 * c.wg + c.lane), sum);
}

template <int kTerms>
__global__ void __launch_bounds__(kTcThreads, 1)
tree_tc_kernel(const __grid_constant__ TreeParams p) {
    constexpr int kRows = 128 / kTerms;                 // rows per block, at most
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    const uint32_t sbase = smem_u32(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    const uint32_t bar0 = sbase + kOffBars;
    auto raw_full = [&](int s) { return bar0 + 8 * s; };
    auto raw_empty = [&](int s) { return bar0 + 8 * (kRaw + s); };
    const uint32_t bx = bar0 + 8 * 2 * kRaw;
    auto k_full = [&](int b) { return bx + 8 * b; };            // K levels, scales -> MMA
    auto s_full = [&](int b) { return bx + 8 * (2 + b); };      // S ready (K levels read)
    auto v_full = [&](int b) { return bx + 8 * (6 + b); };      // V levels -> MMA
    auto p_full = [&](int b) { return bx + 8 * (4 + b); };      // P' -> MMA; S and the scales read
    auto pv_done = [&](int b) { return bx + 8 * (8 + b); };     // V levels and P' read
    const uint32_t drained = bx + 8 * 10;
    uint32_t *tmem_ptr = reinterpret_cast<uint32_t *>(smem + kOffTmem);
    float *sig_k = reinterpret_cast<float *>(smem + kOffSig);       // [4][128]
    float *sig_v = sig_k + kSig * kTileT;                           // [4][128]
    float *negm = reinterpret_cast<float *>(smem + kOffNegM);
    float *xch = reinterpret_cast<float *>(smem + kOffXch);
    float *linv = reinterpret_cast<float *>(smem + kOffLinv);
    float *row_pow2 = reinterpret_cast<float *>(smem + kOffRow);
    uint32_t *vis = reinterpret_cast<uint32_t *>(smem + kOffVis);
    uint32_t *qmax = reinterpret_cast<uint32_t *>(smem + kOffQMax);

    // The allocation takes its time while the schedule is worked out.  Twenty
    // warps that each worked out the first segment spent 3,000 cycles on it, so
    // one does; every role finds later ones by itself, as it gets there.
    if (threadIdx.x == 64) {
        for (int s = 0; s < kRaw; ++s) {
            mbar_init(raw_full(s), 1);
            mbar_init(raw_empty(s), 5);                 // the tile's level warps, the scales
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(k_full(b), 5);                    // four warps' levels, the scales
            mbar_init(s_full(b), 1);
            mbar_init(v_full(b), 4);
            mbar_init(p_full(b), kPArrivals);
            mbar_init(pv_done(b), 1);
        }
        mbar_init(drained, 1);
        qmax[0] = 0u;
        qmax[1] = 0x7F800000u;
        fence_barrier_init();
    }
    if (warp == 1) {
        tc::tmem_alloc(smem_u32(tmem_ptr), 512);
        tc::tmem_relinquish();
    }
    tc::fence_before_sync();
    int *prefix = reinterpret_cast<int *>(smem + kOffPrefix);
    Segment *first = reinterpret_cast<Segment *>(smem + kOffSegment);
    int *range = reinterpret_cast<int *>(first + 1);    // first and last unit + 1
    const int cta = blockIdx.x;
    build_prefix(p, prefix, [&] {
        const int units = prefix[p.B], shares = n_shares(p, units);
        Segment s = {};
        int u0 = 0, u1 = 0;
        if (cta < shares) {
            u0 = share_begin(units, cta, shares);
            u1 = share_begin(units, cta + 1, shares);
            s = segment_at(p, prefix, u0, u1);
        }
        if (lane == 0) {
            *first = s;
            range[0] = u0;
            range[1] = u1;
        }
    });
    tc::fence_after_sync();
    const uint32_t tmem = *tmem_ptr;
    const int u0 = range[0], u1 = range[1];
    if (u0 == u1) {                                     // more CTAs than units
        if (warp == 1) tc::tmem_dealloc(tmem, 512);
        return;
    }
    auto segment = [&](int u) { return u == u0 ? *first : segment_at(p, prefix, u, u1); };

    bool ok = true;                                     // this warp's waits have all come through
    auto wait = [&](uint32_t bar, uint32_t parity) { wait_or_fail(ok, bar, parity); };
    // Where a segment begins, the softmax warps agree among themselves, then
    // warps 1 and 3 join them (Q and the masks are there), and again once the
    // segment's rows are out (tensor memory and masks are free).  The other
    // warps know tiles only, and run ahead across segments.
    auto soft_sync = [&]() { named_sync(1, kSoftWarps * 32); };
    auto ready_sync = [&]() { named_sync(2, (kSoftWarps + 2) * 32); };
    auto done_sync = [&]() { named_sync(8, (kSoftWarps + 2) * 32); };

    if (warp < 4) {
        tc::regs_dec<kRegCtl>();
        if (warp == 0) {
            // ======================= producer ================================
            int it = 0;
            for (int u = u0; u < u1 && ok;) {
                const Segment s = segment(u);
                u += s.tiles;
                const int stop = s.ctx + s.n;
                for (int j = 0; j < s.tiles; ++j, ++it) {
                    const int st = it % kRaw;
                    if (it >= kRaw) {
                        wait(raw_empty(st), ((it / kRaw) - 1) & 1);
                        if (!ok) break;
                    }
                    const int t = (s.tile0 + j) * kTileT;
                    // whole 8-row groups: capacity and page size are multiples of 8
                    const int rows = (min(kTileT, stop - t) + 7) & ~7;
                    if (lane == 0) {
                        fence_proxy_async();
                        mbar_expect_tx(raw_full(st), 2u * (uint32_t)rows * kBlockBytes);
                    }
                    __syncwarp();
                    const int r0 = (lane >> 1) * 32;
                    if (lane < 8 && r0 < rows) {
                        const uint32_t nb = (uint32_t)min(32, rows - r0) * kBlockBytes;
                        int64_t off = piece_offset(p, s.b, s.g, t + r0);
                        if constexpr (kDebugBounds) off = checked_off(off, nb, p.cache_bytes);
                        const uint32_t to = sbase + st * kRawStride + r0 * kBlockBytes;
                        bulk_g2s(to + ((lane & 1) ? kOffRawV : kOffRawK), ((lane & 1) ? p.v : p.k) + off,
                                 nb, raw_full(st));
                    }
                }
            }
            // after a lost hand-off: the copies still in flight land before the
            // shared memory goes away
            for (int i = max(0, it - kRaw); i < it; ++i)
                mbar_wait_bounded(raw_full(i % kRaw), (i / kRaw) & 1, kSpinTree);
        } else if (warp == 1) {
            // ======================= MMA issuer ==============================
            int it0 = 0;
            for (int u = u0; u < u1;) {
                const Segment s = segment(u);
                u += s.tiles;
                const int N = (s.rows + 15) & ~15;
                const uint32_t idesc_qk = tc::idesc_f16(128, N, false);
                const uint32_t idesc_pv = tc::idesc_f16(128, N, true);
                ready_sync();                           // Q is there
                tc::fence_after_sync();
                // the whole warp runs the loop, one elected lane issues
                const bool leader = tc::elect_one();
                const uint64_t q_desc = tc::desc_sw128(sbase + kOffQ);
                const uint64_t v_desc = tc::desc_mn_sw128(sbase + kOffV, 16384);
                const uint64_t p_desc = tc::desc_mn_sw128(sbase + kOffP, 16384);
                // QK two tiles ahead: S of tile j - 2 and its scales are read once
                // its P' is there
#pragma unroll 1
                for (int j = 0; j < s.tiles + 2; ++j) {
                    const int it = it0 + j, b = it & 1;
                    const uint32_t par = (it >> 1) & 1;
                    if (j >= 2) {
                        wait(v_full(b), par ^ 1);
                        wait(p_full(b), par ^ 1);
                        tc::fence_after_sync();
                        if (leader) {
                            const uint64_t va = v_desc + 2048 * b, pb = p_desc + 2048 * b;
#pragma unroll
                            for (int e = 0; e < kTerms; ++e) {           // descriptors count 16 bytes
                                const uint32_t d = tmem + (e ? kColO2 : kColO);
                                if (j > 2)
                                    tc::mma_ss_c<true>(d, va, pb + 1024 * e, idesc_pv);
                                else
                                    tc::mma_ss_c<false>(d, va, pb + 1024 * e, idesc_pv);
#pragma unroll
                                for (int i = 1; i < 8; ++i)
                                    tc::mma_ss_c<true>(d, va + 128 * i, pb + 1024 * e + 128 * i, idesc_pv);
                            }
                            tc::mma_commit(pv_done(b));
                        }
                        __syncwarp();
                    }
                    if (j < s.tiles) {
                        wait(k_full(b), par);
                        tc::fence_after_sync();
                        if (leader) {
                            const uint32_t d = tmem + kColS + 128 * b, ka = tmem + kColK + 64 * b;
                            tc::mma_ts_c<false>(d, ka, q_desc, idesc_qk);
#pragma unroll
                            for (int i = 1; i < 8 * kTerms; ++i)
                                tc::mma_ts_c<true>(d, ka + 8 * (i & 7),
                                                   q_desc + (i >> 3) * (kRows * 16) +
                                                       ((i & 7) >> 2) * (kRows * 8) + (i & 3) * 2,
                                                   idesc_qk);
                            tc::mma_commit(s_full(b));
                        }
                        __syncwarp();
                    }
                }
                it0 += s.tiles;
                done_sync();
            }
            if (tc::elect_one()) tc::mma_commit(drained);    // every product issued has ended
            __syncwarp();
            mbar_wait_bounded(drained, 0, kSpinTree);
            tc::fence_after_sync();
            tc::tmem_dealloc(tmem, 512);
        } else if (warp == 2) {
            // ======================= block scales ============================
            int it = 0;
            for (int u = u0; u < u1;) {
                const Segment s = segment(u);
                u += s.tiles;
#pragma unroll 1
                for (int j = 0; j < s.tiles; ++j, ++it) {
                    const int st = it % kRaw, b = it & 1, sg = it & (kSig - 1);
                    wait(raw_full(st), (it / kRaw) & 1);
                    const uint32_t row = sbase + kOffRawK + st * kRawStride + lane * kBlockBytes;
                    float sk[4], m8[4];                 // S_k, and m 2^8 of S_v = m 2^e
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t at = row + 32 * i * kBlockBytes;
                        sk[i] = half_bits_to_float((uint16_t)dmq::lds16(at));
                        const uint32_t sv = dmq::lds16(at + kOffRawV - kOffRawK);
                        m8[i] = half_bits_to_float((uint16_t)sv) *
                                __uint_as_float((142u + kPShift - scale_field(sv)) << 23);
                    }
                    // QK(it - 2) was issued after the softmax had read tile it - 4's
                    if (it >= 2) wait(s_full(b), ((it >> 1) - 1) & 1);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        sig_k[kTileT * sg + 32 * i + lane] = sk[i];
                        sig_v[kTileT * sg + 32 * i + lane] = m8[i];
                    }
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(k_full(b));
                        mbar_arrive(raw_empty(st));
                    }
                }
            }
        } else {
            // ======================= masks ===================================
            // rows of the block that see node j, one bit each: 32 rows' masks (lane =
            // row) transposed, 32 nodes at a time
            for (int u = u0; u < u1;) {
                const Segment s = segment(u);
                u += s.tiles;
#pragma unroll 1
                for (int w = 0; 32 * w < s.rows; ++w) {
                    const int c = 32 * w + lane;
                    unsigned long long m = 0ull;
                    if (c < s.rows) m = __ldg(p.mask + s.b * p.mask_stride + (s.row0 + c) / p.G);
#pragma unroll
                    for (int jh = 0; jh < 2; ++jh) {
                        uint32_t x = (uint32_t)(m >> (32 * jh)), low = 0x0000FFFFu;
#pragma unroll
                        for (int k = 16; k > 0; k >>= 1) {
                            const uint32_t y = __shfl_xor_sync(kFull, x, k);
                            x = (lane & k) ? (x & ~low) | ((y >> k) & low) : (x & low) | ((y & low) << k);
                            low ^= low << (k >> 1);
                        }
                        vis[4 * (32 * jh + lane) + w] = x;
                    }
                }
                ready_sync();
                done_sync();
            }
        }
    } else if (warp < kSoftWarp0) {
        // ======================= levels ======================================
        tc::regs_dec<kRegLev>();
        const int half = (warp >> 2) - 1;               // 0: even tiles, 1: odd ones
        const int t = threadIdx.x & 127;                // token of the tile = tensor-memory lane
        const uint32_t k_col = tmem + ((uint32_t)(t & ~31) << 16) + kColK + 64 * half;
        // 16-byte chunk c of V's row t lies at c ^ (t % 8)
        const uint32_t v_row = sbase + kOffV + 32768 * half + t * 128 + ((t & 7) << 4);
#pragma unroll 1
        for (int it = half; it < u1 - u0; it += 2) {     // a unit is a tile
            const int st = it % kRaw;
            const uint32_t before = ((it >> 1) - 1) & 1;
            wait(raw_full(st), (it / kRaw) & 1);
            // the row's nibbles start 2 bytes behind a word boundary (even
            // tokens) or 4 (odd ones): read from there, 32 lanes hit 32 banks
            const uint32_t a0 = (sbase + kOffRawK + st * kRawStride + t * kBlockBytes) & ~3u;
            const uint32_t sh = (t & 1) ? 32u : 16u;
            if (it >= 2) wait(s_full(half), before);            // QK(it - 2) has read this buffer
            tc::fence_after_sync();
            // four words at a time: 32 levels, 16 columns; the next four are on
            // their way meanwhile (reads past the row stay inside the stage)
            const uint32_t v0 = a0 + kOffRawV - kOffRawK;
            uint32_t w[5];
#pragma unroll
            for (int i = 0; i < 5; ++i) w[i] = dmq::lds32(a0 + 4 * i);
            uint32_t ka = a0;
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
                uint32_t o[16], nx[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) nx[i] = dmq::lds32(ka + 20 + 4 * i);
                ka += 16;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t l[4];
                    word_levels(__funnelshift_rc(w[i], w[i + 1], sh), l);
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[4 * i + e] = l[e];
                }
                tc::tmem_st16(k_col + 16 * c, o);
                w[0] = w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) w[i + 1] = nx[i];
            }
#pragma unroll
            for (int i = 0; i < 5; ++i) w[i] = dmq::lds32(v0 + 4 * i);
            tc::tmem_wait_st();
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(k_full(half));
            if (it >= 2) wait(pv_done(half), before);
            // the scale lies in front of the first nibbles, in the word's other half
            uint32_t va = v0;
            const uint32_t pow2 = scale_field(w[0] >> (sh - 16)) * 0x04000400u;
#pragma unroll 1
            for (int c = 0; c < 16; c += 4, va += 16) {       // a word: eight levels, 16 bytes
                uint32_t nx[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) nx[i] = dmq::lds32(va + 20 + 4 * i);
                const uint32_t to = (v_row ^ ((c & 4) << 4)) + (c >> 3) * 16384;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t l[4];
                    word_levels_scaled(__funnelshift_rc(w[i], w[i + 1], sh), pow2, l);
                    dmq::sts128(to ^ (i << 4), l[0], l[1], l[2], l[3]);
                }
                w[0] = w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) w[i + 1] = nx[i];
            }
            fence_proxy_async();                    // read by the tensor core
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(v_full(half));
                mbar_arrive(raw_empty(st));
            }
        }
    } else {
        // ======================= softmax =====================================
        tc::regs_inc<kRegSoft>();
        const int ws = warp - kSoftWarp0, wg = ws >> 2, q4 = warp & 3;
        const int t = 32 * q4 + lane;                   // token, at the end position of a dimension
        const uint32_t t_lane = tmem + ((uint32_t)(32 * q4) << 16);
        const int wg_bar = 4 + wg;
        int it = 0;
        for (int u = u0; u < u1;) {
            const Segment s = segment(u);
            const bool whole = s.tiles == s.work_tiles;
            u += s.tiles;
            const int N = (s.rows + 15) & ~15, nch = N >> 3;
            // ---- queries: rotate, agree on the power of two, store -----------
            // Eight lanes per row: lane j holds channels 4 j .. 4 j + 3 of each
            // quarter, so that only strides 4, 8 and 16 of the transform are
            // shuffles.  (Rolled loops through shared memory: straight-line code
            // that runs once per segment costs its instruction fetches.)
            float *stage = reinterpret_cast<float *>(smem + kOffP);   // [rows][128], no P' in it yet
            const int j = lane & 7;
            float mx = 0.f, mn = INFINITY;
#pragma unroll 1
            for (int r = 4 * ws + (lane >> 3); r - (lane >> 3) < s.rows; r += 4 * kSoftWarps) {
                const int c = s.row0 + min(r, s.rows - 1);
                const int i = c / p.G, h = s.g * p.G + (c - i * p.G);
                const int64_t at = (((int64_t)s.b * p.T + i) * p.Hq + h) * kD + 4 * j;
                uint64_t v[8];                          // channels (0, 1), (2, 3) of quarter k: 2 k, 2 k + 1
                float x[4][4];
#pragma unroll
                for (int k = 0; k < 4; ++k) load4(p.q, p.q_type, at + 32 * k, x[k]);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t sb = lane_sign_bits(p.sign_lo, p.sign_hi, j + 8 * k);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if ((sb >> e) & 1u) x[k][e] = -x[k][e];
                    v[2 * k] = pack2(x[k][0] + x[k][1], x[k][0] - x[k][1]);
                    v[2 * k + 1] = pack2(x[k][2] + x[k][3], x[k][2] - x[k][3]);
                }
                const uint64_t minus = pack2(-1.f, -1.f);
                auto butterfly = [&](uint64_t &x, uint64_t &y) {
                    const uint64_t sum = add2(x, y);
                    y = fma2(y, minus, x);
                    x = sum;
                };
#pragma unroll
                for (int k = 0; k < 8; k += 2) butterfly(v[k], v[k + 1]);               // stride 2
#pragma unroll
                for (int m = 1; m < 8; m <<= 1) {                                       // 4, 8, 16
                    const float neg = (j & m) ? -1.f : 1.f;
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        float lo, hi;
                        unpack2(v[k], lo, hi);
                        v[k] = fma2(v[k], pack2(neg, neg), pack2(__shfl_xor_sync(kFull, lo, m),
                                                                 __shfl_xor_sync(kFull, hi, m)));
                    }
                }
#pragma unroll
                for (int k = 0; k < 8; ++k)                                             // 32, 64
                    if (!(k & 2)) butterfly(v[k], v[k + 2]);
#pragma unroll
                for (int k = 0; k < 4; ++k) butterfly(v[k], v[k + 4]);
                float of_row = 0.f;                     // its largest finite channel
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    float4 y;
                    unpack2(mul2(v[2 * k], pack2(rot_c(), rot_c())), y.x, y.y);
                    unpack2(mul2(v[2 * k + 1], pack2(rot_c(), rot_c())), y.z, y.w);
                    const float top = fmaxf(fmaxf(fabsf(y.x), fabsf(y.y)), fmaxf(fabsf(y.z), fabsf(y.w)));
                    if (isfinite(y.x) && isfinite(y.y) && isfinite(y.z) && isfinite(y.w)) of_row = fmaxf(of_row, top);
                    if (r < s.rows) *reinterpret_cast<float4 *>(stage + r * kD + 4 * j + 32 * k) = y;
                }
#pragma unroll
                for (int m = 1; m < 8; m <<= 1) of_row = fmaxf(of_row, __shfl_xor_sync(kFull, of_row, m));
                if (j == 0 && r < s.rows) row_pow2[r] = of_row;
                mx = fmaxf(mx, of_row);
                if (of_row > 0.f) mn = fminf(mn, of_row);
            }
            mx = warp_max(mx);
            mn = -warp_max(-mn);
            if (lane == 0 && mx > 0.f) {
                atomicMax(qmax, __float_as_uint(mx));
                atomicMin(qmax + 1, __float_as_uint(mn));
            }
            for (int r = ws * 32 + lane; r < kRows; r += 32 * kSoftWarps) negm[r] = -kLowest;
            soft_sync();
            // x < 2^exponent(x); 2^(15 - exponent(x)) brings it below 2^15
            auto exponent = [](float x) { return max((int)(__float_as_uint(x) >> 23) - 126, -100); };
            auto pow2 = [](int e) { return __uint_as_float((uint32_t)(127 + e) << 23); };
            const float big = __uint_as_float(qmax[0]);
            const bool spread = __uint_as_float(qmax[1]) < big * 0x1p-14f;
            const int e2 = exponent(big);
            // log2 logit = S skc with skc = S_k c (levels are (2n - 15) 2^-11)
            const float c2 = p.scale * (1.4426950408889634f * 2048.0f / 15.0f) *
                             (spread ? 1.0f : pow2(e2 - 15));
            // 16 lanes per row, eight dimensions each
#pragma unroll 1
            for (int r = 2 * ws + (lane >> 4); r < N; r += 2 * kSoftWarps) {
                const int ch = lane & 15;
                int er = e2;
                if (spread) {
                    if (r < s.rows) er = exponent(row_pow2[r]);
                    __syncwarp();                       // both rows' lanes have read
                    if (ch == 0) row_pow2[r] = pow2(er - 15);
                }
                const float up = pow2(15 - er);
                float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
                if (r < s.rows) {
                    a = *reinterpret_cast<const float4 *>(stage + r * kD + 8 * ch);
                    b = *reinterpret_cast<const float4 *>(stage + r * kD + 8 * ch + 4);
                }
                const float x[8] = {a.x * up, b.x * up, a.y * up, b.y * up,     // the operands' order
                                    a.z * up, b.z * up, a.w * up, b.w * up};
                const uint32_t at = sbase + kOffQ + (ch >> 3) * (kRows * 128) + (r >> 3) * 1024 +
                                    (r & 7) * 128 + (((ch & 7) ^ (r & 7)) << 4);
                uint32_t h[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) h[k] = half2_bits(x[2 * k], x[2 * k + 1]);
                dmq::sts128(at, h[0], h[1], h[2], h[3]);
                if constexpr (kTerms == 2) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h[k]));
                        h[k] = half2_bits(x[2 * k] - f.x, x[2 * k + 1] - f.y);
                    }
                    dmq::sts128(at + kRows * 256, h[0], h[1], h[2], h[3]);
                }
            }
            fence_proxy_async();                        // read by the tensor core
            ready_sync();
            if (ws == 0 && lane == 0) {                 // for the next segment (read before the barrier)
                qmax[0] = 0u;
                qmax[1] = 0x7F800000u;
            }

            const Soft sc = {sbase, tmem, bx, t, lane, wg, kPArrivals / 4 / ((nch + 3) >> 2), c2, spread};
            const int t0 = s.tile0 * kTileT;
            const int mine = min(4, nch - 4 * wg);      // chunks of this warpgroup
            if (mine == 4)
                soft_segment<kTerms, 4>(sc, it, s.tiles, t0, s.ctx, s.n, ok);
            else if (mine == 2)
                soft_segment<kTerms, 2>(sc, it, s.tiles, t0, s.ctx, s.n, ok);
            it += s.tiles;

            // ---- the block's rows: thread = position of a dimension ----------
            const int last = it - 1;
            wait(pv_done(last & 1), (last >> 1) & 1);
            tc::fence_after_sync();
            // sum_t p m 2^8 (2n - 15) 2^(e-7) -> sum_t p S_v (2n - 15) / 15
            constexpr float back = 128.0f / (15 << kPShift);
            named_sync(wg_bar, 128);
            const int row = 32 * wg + t;
            if (t < 32 && row < s.rows) {
                const float L = (xch[row] + xch[128 + row]) + (xch[256 + row] + xch[384 + row]);
                if (whole)
                    linv[row] = L == 0.f ? 0.f : 1.0f / L;
                else
                    p.part_ml[(int64_t)part_slot(s, cta) * p.rows + row] = make_float2(-negm[row], L);
            }
            const int d = dim_at(t);
            float *po = p.part_o + (int64_t)part_slot(s, cta) * p.rows * kD;
#pragma unroll 1
            for (int c = 4 * wg; c < min(nch, 4 * wg + 4); ++c) {   // (P' is done with its buffers)
                uint32_t o[8];
                tc::tmem_ld8(t_lane + kColO + 8 * c, o);
                tc::tmem_wait_ld();
                if constexpr (kTerms == 2) {
                    uint32_t lo[8];
                    tc::tmem_ld8(t_lane + kColO2 + 8 * c, lo);
                    tc::tmem_wait_ld();
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        o[k] = __float_as_uint(__uint_as_float(o[k]) + __uint_as_float(lo[k]) * (1.0f / kLowTerm));
                }
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int row = 8 * c + k;
                    if (row < s.rows) (whole ? stage : po)[row * kD + d] = __uint_as_float(o[k]) * back;
                }
            }
            tc::fence_before_sync();
            if (whole) {
                named_sync(3, kSoftWarps * 32);
                for (int r = ws; r < s.rows; r += kSoftWarps) {
                    const float4 o = *reinterpret_cast<const float4 *>(stage + r * kD + 4 * lane);
                    const float inv = linv[r];
                    float v[4] = {o.x * inv, o.y * inv, o.z * inv, o.w * inv};
                    store_out(p, s.b, s.g, s.row0 + r, v, lane);
                }
            }
            done_sync();
        }
    }
}

}  // namespace tree
}  // namespace tbq4
