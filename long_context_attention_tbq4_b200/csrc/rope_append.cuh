// rope_append.cuh -- one launch between a layer's projections and its
// attention: rotary position embedding of the new tokens' queries and keys,
// TBQ4 encoding of keys and values, and their store into the caches.
//
// Rotary embedding.  theta_i = fl64(pos * inv_freq_i); c_i, s_i = cos and sin
// of theta_i in binary64, rounded once to binary32; for the pair (x1, x2)
//   y1 = fl32(fl32(x1 c) - fl32(x2 s)),  y2 = fl32(fl32(x2 c) + fl32(x1 s)),
// every operation rounded to binary32 by itself, so that the bytes that the
// encoder (encode_row: the codebook of include/tbq4.h) makes of y are defined
// bit for bit.  A key goes from y to the encoder in binary32, without a
// rounding to the input's type in between; a query is rounded once, to its
// own type.
#pragma once
#include "common.cuh"
#include "quantize.cuh"

namespace tbq4 {

enum ElemType { kElemF32 = 0, kElemF16 = 1, kElemBF16 = 2 };

// Four consecutive elements of a row, element index idx (a multiple of 4).
__device__ __forceinline__ void load4(const void *p, int type, int64_t idx, float (&v)[4]) {
    if (type == kElemF32) {
        const float4 x = *reinterpret_cast<const float4 *>(static_cast<const float *>(p) + idx);
        v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
        return;
    }
    const uint2 r = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(p) + idx);
    if (type == kElemBF16) {
        v[0] = __uint_as_float(r.x << 16);
        v[1] = __uint_as_float(r.x & 0xFFFF0000u);
        v[2] = __uint_as_float(r.y << 16);
        v[3] = __uint_as_float(r.y & 0xFFFF0000u);
    } else {
        const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&r.x));
        const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&r.y));
        v[0] = a.x; v[1] = a.y; v[2] = b.x; v[3] = b.y;
    }
}

// Four consecutive elements, rounded to nearest even.
__device__ __forceinline__ void store4(void *p, int type, int64_t idx, const float (&v)[4]) {
    if (type == kElemF32) {
        *reinterpret_cast<float4 *>(static_cast<float *>(p) + idx) =
            make_float4(v[0], v[1], v[2], v[3]);
        return;
    }
    uint2 r;
    if (type == kElemBF16) {
        __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
        r.x = *reinterpret_cast<uint32_t *>(&a);
        r.y = *reinterpret_cast<uint32_t *>(&b);
    } else {
        __half2 a = __floats2half2_rn(v[0], v[1]), b = __floats2half2_rn(v[2], v[3]);
        r.x = *reinterpret_cast<uint32_t *>(&a);
        r.y = *reinterpret_cast<uint32_t *>(&b);
    }
    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p) + idx) = r;
}

struct RopeParams {
    const void *q, *k, *v;             // rows of 128, strides in elements
    int64_t q_tok, q_head, k_tok, k_head, v_tok, v_head;
    int n_tokens, Hq, Hkv, B;
    int per_seq;                       // seq_ids == nullptr: token i is of sequence i / per_seq
    const int32_t *seq_ids, *slots, *positions;   // positions may be nullptr: the slots
    const double *inv_freq;            // [rot / 2]
    int rot;
    int64_t capacity;
    uint64_t sign_lo, sign_hi;
    PageMap pm;                        // table == nullptr: contiguous caches
    uint8_t *kc, *vc;
    void *q_out;                       // [n_tokens][Hq][128]
    int64_t q_out_elems;               // extent, for the debug build's bounds checks
};

// cos and sin of fl64(pos * inv_freq), rounded to binary32.  theta / pi is
// formed as a product with 1/pi carried to twice the precision (the error of
// the leading product by FMA, after Dekker), whole turns are removed exactly,
// and sincospi takes the rest: about 2^-52 of error at any 32-bit position.
__device__ __forceinline__ float2 rope_cos_sin(int32_t pos, double inv_freq) {
    constexpr double kInvPiHi = 0.31830988618379069, kInvPiLo = -1.9678676675182486e-17;
    const double theta = __dmul_rn((double)pos, inv_freq);
    const double h = __dmul_rn(theta, kInvPiHi);
    const double e = fma(theta, kInvPiLo, fma(theta, kInvPiHi, -h));
    const double r = h - 2.0 * rint(0.5 * h);          // exact
    double s, c;
    sincospi(r + e, &s, &c);
    return make_float2((float)c, (float)s);
}

// A row of 128 by 16 lanes, two rows per warp: lane j of a half-warp holds
// channels 4 j .. 4 j + 3 (chunk a) and 64 + 4 j .. 67 + 4 j (chunk b).  The
// transform's strides 1 and 2 then lie inside a chunk, 4 to 32 between lanes
// (16 shuffles per row) and 64 between the lane's two chunks; with all 128
// channels rotated by halves a pair is the lane's own as well.
struct LaneRow {
    float a[4], b[4];
};

// How a call's heads are rotated: not, pairs (2i, 2i + 1), all 128 channels by
// halves, or some by halves.
enum RopeMode { kRopeNone, kRopeInterleaved, kRopeAll, kRopePart };

// Row encoder: the codebook's steps in the order of encode_row (same bytes),
// on LaneRow's layout.  Division by the scale and rounding as in
// quantize_rows_kernel.  Returns the two 16-bit index pieces.
__device__ __forceinline__ void encode_lane_row(const LaneRow &r, const float (&sg)[8], int j,
                                                uint16_t &scale, uint16_t &pa, uint16_t &pb) {
    // stride 1 inside the pairs (0 1), (2 3), (4 5), (6 7); from there on the
    // pairs move together
    uint64_t v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float x0 = e < 2 ? r.a[2 * e] : r.b[2 * e - 4], x1 = e < 2 ? r.a[2 * e + 1] : r.b[2 * e - 3];
        const float y0 = __fmul_rn(x0, sg[2 * e]), y1 = __fmul_rn(x1, sg[2 * e + 1]);
        v[e] = pack2(__fadd_rn(y0, y1), __fsub_rn(y0, y1));
    }
    const uint64_t minus = pack2(-1.0f, -1.0f);
    auto butterfly = [&](uint64_t &x, uint64_t &y) {   // x + y, x - y
        const uint64_t s = add2(x, y);
        y = fma2(y, minus, x);
        x = s;
    };
    butterfly(v[0], v[1]);                          // stride 2
    butterfly(v[2], v[3]);
#pragma unroll
    for (int m = 1; m < 16; m <<= 1) {              // strides 4 .. 32
        const float neg = (j & m) ? -1.0f : 1.0f;   // upper: partner - own, as one FMA
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float x, y;
            unpack2(v[e], x, y);
            x = __shfl_xor_sync(kFull, x, m);
            y = __shfl_xor_sync(kFull, y, m);
            v[e] = fma2(v[e], pack2(neg, neg), pack2(x, y));
        }
    }
    butterfly(v[0], v[2]);                          // stride 64
    butterfly(v[1], v[3]);
    float f[8], m = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        v[e] = mul2(v[e], pack2(rot_c(), rot_c()));
        unpack2(v[e], f[2 * e], f[2 * e + 1]);
        m = fmaxf(m, fmaxf(fabsf(f[2 * e]), fabsf(f[2 * e + 1])));
    }
#pragma unroll
    for (int x = 1; x < 16; x <<= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, x));
    uint16_t sb = __half_as_ushort(__float2half_rn(m));
    if ((sb & 0x7FFFu) == 0x7C00u) sb = 0x7BFFu;    // saturate at 65504
    scale = sb;
    const float S = half_bits_to_float(sb);
    const uint32_t sabs = sb & 0x7FFFu;
    // a normal, unsaturated scale needs no clamp (see quantize_rows_kernel)
    if (sabs < 0x0400u || sabs >= 0x7BFFu) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            v[e] = pack2(fminf(fmaxf(f[2 * e], -S), S), fminf(fmaxf(f[2 * e + 1], -S), S));
    }
    const float Sd = S == 0.0f ? 1.0f : S, rs = __frcp_rn(Sd);
    uint32_t idx[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const uint64_t q0 = mul2(v[e], pack2(rs, rs));
        const uint64_t q = fma2(fma2(q0, pack2(-Sd, -Sd), v[e]), pack2(rs, rs), q0);
        float x, y;
        unpack2(q, x, y);
        // a scalar product: packed, it would be fused with the sum behind it
        const uint64_t u = add2(pack2(__fmul_rn(x, 7.5f), __fmul_rn(y, 7.5f)), pack2(7.5f, 7.5f));
        unpack2(add2(u, pack2(12582912.0f, 12582912.0f)), x, y);
        idx[2 * e] = __float_as_uint(x) & 0xFu;
        idx[2 * e + 1] = __float_as_uint(y) & 0xFu;
    }
    pa = (uint16_t)(idx[0] | (idx[1] << 4) | (idx[2] << 8) | (idx[3] << 12));
    pb = (uint16_t)(idx[4] | (idx[5] << 4) | (idx[6] << 8) | (idx[7] << 12));
}

// A warp takes a token, or, where there are few, every `parts`-th pair of
// rows of one: its cosines and sines into shared memory (32 lanes, up to two
// each), then pair after pair of its Hq + 2 Hkv rows.  Bound by issue and by
// the latency of its loads: 16,384 tokens of 24/4 heads in bf16 take 62.6 us
// (3.9 TB/s; the copy rate would allow 37 us), 117 us with one row per warp
// and the token's angles behind a block barrier.  Seven blocks of four warps
// per SM: eight spill, six hide less (82 us with four pairs in flight).
// Fetching queries ahead of the angles cost registers and 8 us.
constexpr int kRopeWarps = 4;

// A row at p as this lane's two chunks (p points at chunk a).
template <int kType>
__device__ __forceinline__ LaneRow load_row(const uint8_t *p) {
    LaneRow r;
    load4(p, kType, 0, r.a);
    load4(p, kType, 64, r.b);
    return r;
}

template <int kType, int kMode>
__global__ void __launch_bounds__(kRopeWarps * 32, 7)
rope_append_kernel(const __grid_constant__ RopeParams p, int parts) {
    constexpr int kSize = kType == kElemF32 ? 4 : 2;
    __shared__ float2 cs_all[kRopeWarps][kD / 2];
    const int lane = threadIdx.x & 31, j = lane & 15, side = lane >> 4;
    float2 *cs = cs_all[threadIdx.x >> 5];
    const int64_t item = (int64_t)blockIdx.x * kRopeWarps + (threadIdx.x >> 5);
    const int t = (int)(item / parts), part = (int)(item - (int64_t)t * parts);
    if (t >= p.n_tokens) return;
    const int b = p.seq_ids ? __ldg(p.seq_ids + t) : t / p.per_seq;
    if (b < 0) return;                                 // padding: nothing of it is written
    if (b >= p.B) {
        if (lane == 0) record_status(4u /* TBQ4_ERR_CAPACITY */);
        return;
    }
    const int32_t slot = __ldg(p.slots + t);
    const int half = p.rot >> 1;
    if constexpr (kMode != kRopeNone) {
        const int32_t pos = p.positions ? __ldg(p.positions + t) : slot;
        for (int i = lane; i < half; i += 32) cs[i] = rope_cos_sin(pos, __ldg(p.inv_freq + i));
        __syncwarp();
    }
    const int ca = 4 * j, cb = 64 + 4 * j;             // first channels of the two chunks
    // rotated whole or not at all (rot % 8 == 0)
    const bool ta = kMode == kRopeAll || ca < p.rot, tb = kMode == kRopeAll || cb < p.rot;
    const bool fa = kMode == kRopeAll || ca < half, fb = kMode != kRopeAll && cb < half;   // first of the pair
    // y = x c + partner s, with the sign of s that the pair's formula asks for
    // (negation is exact, so this is the documented sequence of roundings); the
    // same for every head
    float cos_a[4], sin_a[4], cos_b[4], sin_b[4];
    if constexpr (kMode != kRopeNone) {
#pragma unroll
        for (int e = 0; e < 4; e += 2) {
            float2 x0, x1, y0, y1;
            if constexpr (kMode == kRopeInterleaved) {
                x0 = x1 = cs[ta ? (ca + e) >> 1 : 0];
                y0 = y1 = cs[tb ? (cb + e) >> 1 : 0];
                sin_a[e] = -x0.y;
                sin_a[e + 1] = x0.y;
                sin_b[e] = -y0.y;
                sin_b[e + 1] = y0.y;
            } else {
                const int ia = ta ? ca + e - (fa ? 0 : half) : 0, ib = tb ? cb + e - (fb ? 0 : half) : 0;
                x0 = cs[ia];
                x1 = cs[ia + 1];
                y0 = cs[ib];
                y1 = cs[ib + 1];
                sin_a[e] = fa ? -x0.y : x0.y;
                sin_a[e + 1] = fa ? -x1.y : x1.y;
                sin_b[e] = fb ? -y0.y : y0.y;
                sin_b[e + 1] = fb ? -y1.y : y1.y;
            }
            cos_a[e] = x0.x;
            cos_a[e + 1] = x1.x;
            cos_b[e] = y0.x;
            cos_b[e + 1] = y1.x;
        }
    }
    // the chunks that pair with this lane's (kRopePart: read again, from cache)
    const int qa = !ta ? 0 : fa ? half : -half, qb = !tb ? 0 : fb ? half : -half;
    auto rotate = [&](LaneRow &r, const uint8_t *row) {
        if constexpr (kMode == kRopeNone) return;
        LaneRow o = {{r.b[0], r.b[1], r.b[2], r.b[3]}, {r.a[0], r.a[1], r.a[2], r.a[3]}};
        if constexpr (kMode == kRopeInterleaved)
            o = {{r.a[1], r.a[0], r.a[3], r.a[2]}, {r.b[1], r.b[0], r.b[3], r.b[2]}};
        if constexpr (kMode == kRopePart) {
            load4(row + qa * kSize, kType, 0, o.a);
            load4(row + qb * kSize, kType, 64, o.b);
            __syncwarp();                              // before any lane stores over the row
        }
#pragma unroll
        for (int e = 0; e < 4; e += 2) {
            // scalar products: a packed product and a packed sum end up fused
            float x, y;
            unpack2(add2(pack2(__fmul_rn(r.a[e], cos_a[e]), __fmul_rn(r.a[e + 1], cos_a[e + 1])),
                         pack2(__fmul_rn(o.a[e], sin_a[e]), __fmul_rn(o.a[e + 1], sin_a[e + 1]))), x, y);
            if (ta) { r.a[e] = x; r.a[e + 1] = y; }
            unpack2(add2(pack2(__fmul_rn(r.b[e], cos_b[e]), __fmul_rn(r.b[e + 1], cos_b[e + 1])),
                         pack2(__fmul_rn(o.b[e], sin_b[e]), __fmul_rn(o.b[e + 1], sin_b[e + 1]))), x, y);
            if (tb) { r.b[e] = x; r.b[e + 1] = y; }
        }
    };

    // ---- queries: kBatch pairs of rows in flight.  Both halves of the warp
    // walk heads 2 i + side; the odd one out of an odd count repeats its
    // neighbour and stores nothing.
    constexpr int kBatch = 2;
    const int q_pairs = (p.Hq + 1) >> 1, kv_pairs = (p.Hkv + 1) >> 1;
    {
        const uint8_t *src = static_cast<const uint8_t *>(p.q) +
                             ((int64_t)t * p.q_tok + (int64_t)(2 * part) * p.q_head + ca) * kSize;
        const int64_t step = 2 * (int64_t)parts * p.q_head * kSize, beside = side * p.q_head * kSize;
        uint8_t *dst = static_cast<uint8_t *>(p.q_out) +
                       (((int64_t)t * p.Hq + 2 * part + side) * kD + ca) * kSize;
        for (int i = part; i < q_pairs; i += kBatch * parts) {
            LaneRow r[kBatch];
            const uint8_t *row[kBatch];
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const int h = 2 * (i + k * parts);
                row[k] = src + (h + 1 < p.Hq ? beside : 0);
                if (h < p.Hq) r[k] = load_row<kType>(row[k]);
                src += step;
            }
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const int h = 2 * (i + k * parts);
                if (h >= p.Hq) break;
                rotate(r[k], row[k]);
                if (h + side < p.Hq && in_extent(((int64_t)t * p.Hq + h + side) * kD, kD, p.q_out_elems)) {
                    store4(dst, kType, 0, r[k].a);
                    store4(dst, kType, 64, r[k].b);
                }
                dst += 2 * parts * kD * kSize;
            }
        }
    }

    // ---- keys, then values (pairs are numbered on from the queries')
    // where this token's blocks go: KV head h at off + h * head_bytes
    int64_t off = -1, head_bytes = 0;
    if (slot >= 0 && slot < p.capacity) {
        if (p.pm.table) {
            const int32_t pid = __ldg(p.pm.table + (int64_t)b * p.pm.max_pages + slot / p.pm.page_size);
            head_bytes = (int64_t)p.pm.page_size * kBlockBytes;
            if (pid >= 0 && (int64_t)pid < p.pm.n_pages)
                off = (int64_t)pid * p.Hkv * head_bytes + (int64_t)(slot % p.pm.page_size) * kBlockBytes;
        } else {
            head_bytes = p.capacity * kBlockBytes;
            off = (int64_t)b * p.Hkv * head_bytes + (int64_t)slot * kBlockBytes;
        }
        if (off >= 0 && !in_extent(off, (p.Hkv - 1) * head_bytes + kBlockBytes, p.pm.cache_bytes)) off = -1;
    }
    if (off < 0) {
        if (lane == 0) record_status(4u /* TBQ4_ERR_CAPACITY */);
        return;
    }
    float sg[8];
    {
        const uint32_t sa = lane_sign_bits(p.sign_lo, p.sign_hi, j), sb = lane_sign_bits(p.sign_lo, p.sign_hi, 16 + j);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            sg[e] = ((sa >> e) & 1u) ? -1.0f : 1.0f;
            sg[4 + e] = ((sb >> e) & 1u) ? -1.0f : 1.0f;
        }
    }
    const int first = (part - q_pairs % parts + parts) % parts;
    auto row_of = [&](int i) -> const uint8_t * {
        const bool is_v = i >= kv_pairs;
        const int h = min(2 * (is_v ? i - kv_pairs : i) + side, p.Hkv - 1);
        return static_cast<const uint8_t *>(is_v ? p.v : p.k) +
               ((int64_t)t * (is_v ? p.v_tok : p.k_tok) + h * (is_v ? p.v_head : p.k_head) + ca) * kSize;
    };
    const uint8_t *row = row_of(min(first, 2 * kv_pairs - 1));
    LaneRow ahead = load_row<kType>(row);
#pragma unroll 1
    for (int i = first; i < 2 * kv_pairs; i += parts) {
        LaneRow r = ahead;
        const uint8_t *now = row;
        row = row_of(min(i + parts, 2 * kv_pairs - 1));
        ahead = load_row<kType>(row);
        const bool is_v = i >= kv_pairs;
        const int h = 2 * (is_v ? i - kv_pairs : i) + side;
        if (!is_v) rotate(r, now);
        uint16_t scale, pa, pb;
        encode_lane_row(r, sg, j, scale, pa, pb);
        if (h < p.Hkv) {
            uint16_t *dst = reinterpret_cast<uint16_t *>((is_v ? p.vc : p.kc) + off + h * head_bytes);
            dst[1 + j] = pa;
            dst[17 + j] = pb;
            if (j == 0) dst[0] = scale;
        }
    }
}

}  // namespace tbq4
