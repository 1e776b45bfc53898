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
    int type;                          // ElemType of q, k, v and q_out
    int n_tokens, Hq, Hkv, B;
    int per_seq;                       // seq_ids == nullptr: token i is of sequence i / per_seq
    const int32_t *seq_ids, *slots, *positions;   // positions may be nullptr: the slots
    const double *inv_freq;            // [rot / 2]
    int rot, interleaved;
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

// One CTA per token (strided): the token's cosines and sines into shared
// memory, then one warp per row (4 values per lane) of its Hq + 2 Hkv rows.
constexpr int kRopeWarps = 8;

__global__ void __launch_bounds__(kRopeWarps * 32)
rope_append_kernel(const RopeParams p) {
    __shared__ float2 cs[kD / 2];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t sbits = lane_sign_bits(p.sign_lo, p.sign_hi, lane);
    const int half = p.rot >> 1;
    for (int t = blockIdx.x; t < p.n_tokens; t += gridDim.x) {
        const int b = p.seq_ids ? __ldg(p.seq_ids + t) : t / p.per_seq;
        if (b < 0) continue;                           // padding: nothing of it is written
        if (b >= p.B) {
            if (threadIdx.x == 0) record_status(4u /* TBQ4_ERR_CAPACITY */);
            continue;
        }
        const int32_t slot = __ldg(p.slots + t);
        const int32_t pos = p.positions ? __ldg(p.positions + t) : slot;
        if (threadIdx.x < half) cs[threadIdx.x] = rope_cos_sin(pos, p.inv_freq[threadIdx.x]);
        __syncthreads();
        for (int r = warp; r < p.Hq + 2 * p.Hkv; r += kRopeWarps) {
            const bool is_q = r < p.Hq, is_v = r >= p.Hq + p.Hkv;
            const int h = is_q ? r : is_v ? r - p.Hq - p.Hkv : r - p.Hq;
            float v[4];
            load4(is_q ? p.q : is_v ? p.v : p.k, p.type,
                  (int64_t)t * (is_q ? p.q_tok : is_v ? p.v_tok : p.k_tok) +
                      (int64_t)h * (is_q ? p.q_head : is_v ? p.v_head : p.k_head) + 4 * lane, v);
            if (!is_v) {
                if (p.interleaved) {                   // pairs (2 i, 2 i + 1)
                    if (4 * lane < p.rot) {
#pragma unroll
                        for (int e = 0; e < 4; e += 2) {
                            const float2 a = cs[2 * lane + (e >> 1)];
                            const float x1 = v[e], x2 = v[e + 1];
                            v[e] = __fsub_rn(__fmul_rn(x1, a.x), __fmul_rn(x2, a.y));
                            v[e + 1] = __fadd_rn(__fmul_rn(x2, a.x), __fmul_rn(x1, a.y));
                        }
                    }
                } else {                               // pairs (i, i + rot / 2)
                    const int hl = p.rot >> 3;         // lanes of each half
                    const bool low = lane < hl, in = lane < 2 * hl;
                    const int other = low ? lane + hl : in ? lane - hl : lane;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float x = __shfl_sync(kFull, v[e], other);
                        if (in) {
                            const float2 a = cs[4 * (low ? lane : other) + e];
                            const float own = __fmul_rn(v[e], a.x), oth = __fmul_rn(x, a.y);
                            v[e] = low ? __fsub_rn(own, oth) : __fadd_rn(own, oth);
                        }
                    }
                }
            }
            if (is_q) {
                const int64_t oi = ((int64_t)t * p.Hq + h) * kD + 4 * lane;
                if (in_extent(oi, 4, p.q_out_elems)) store4(p.q_out, p.type, oi, v);
                continue;
            }
            uint16_t sb;
            const uint32_t packed = encode_row(v, sbits, lane, &sb);
            int64_t off = -1;
            if (slot >= 0 && slot < p.capacity) {
                if (p.pm.table) {
                    const int32_t pid =
                        __ldg(p.pm.table + (int64_t)b * p.pm.max_pages + slot / p.pm.page_size);
                    if (pid >= 0 && (int64_t)pid < p.pm.n_pages)
                        off = (((int64_t)pid * p.Hkv + h) * p.pm.page_size + slot % p.pm.page_size) *
                              kBlockBytes;
                } else {
                    off = (((int64_t)b * p.Hkv + h) * p.capacity + slot) * kBlockBytes;
                }
                if (off >= 0 && !in_extent(off, kBlockBytes, p.pm.cache_bytes)) off = -1;
            }
            if (off < 0) {
                if (lane == 0) record_status(4u /* TBQ4_ERR_CAPACITY */);
                continue;
            }
            uint8_t *dst = (is_v ? p.vc : p.kc) + off;
            reinterpret_cast<uint16_t *>(dst + 2)[lane] = (uint16_t)packed;
            if (lane == 0) *reinterpret_cast<uint16_t *>(dst) = sb;
        }
        __syncthreads();
    }
}

}  // namespace tbq4
