// q4_rows.cuh -- the row set of one sequence of the 4-bit attention, in units of 64 rows, and
// the parameters shared by its kernels.
#pragma once
#include "q4.cuh"

namespace lsa {
namespace q4 {

struct DecodeParams {
    const void *q;                  // [B, Hq, dqk] bf16 or f16
    const uint8_t *k_pool, *v_pool; // v_pool null: latent rows
    const int32_t *table, *topk_idx, *topk_count, *window_start, *window_len;
    void *out;                      // [B, Hq, dv] of out_dtype
    float *lse;                     // [B, Hq] or null
    // Latent: [B, splits, Hq, dv] and [B, splits, Hq].  Separate: two parts a CTA, [CTAs, 2, heads of a CTA, dv],
    // and the first and last CTA of every segment.
    float *o_part, *m_part, *l_part;
    int2 *seg_range;
    int32_t *status;
    int64_t n_slots;
    int table_stride, k, Hq, heads, n_splits;   // n_splits: CTA pairs a sequence (latent), CTAs in all (separate)
    float scale_log2, v_scale;      // scale_log2: scale * k_scale * log2(e)
    int q_f16, out_dtype;
};

// Window rows that a table row can hold: positions behind its last chunk have no slot, so a longer window is cut here
// (and flagged) instead of being walked.
__device__ __forceinline__ int window_rows(const DecodeParams &p, int start, int len) {
    if (start < 0) return 0;
    const int64_t end = lsa_min64((int64_t)p.table_stride * LSA_CHUNK, INT32_MAX - 63);
    return (int)lsa_min64(max(len, 0), lsa_max64(end - start, 0));
}

// Units of one sequence: ceil(tk / 64) units of 64 top-k rows, then the window chunk by chunk
// (its first and last chunk may be partly outside the window).
struct Units {
    int tk, wstart, wlen, t_topk, first_chunk, total;
    __device__ Units(const DecodeParams &p, int b) {
        tk = p.k > 0 ? min(max(p.topk_count[b], 0), p.k) : 0;
        wstart = p.window_start[b];
        const int len = p.window_len[b];
        wlen = window_rows(p, wstart, len);
        if (len > wlen && threadIdx.x == 0) flag(p.status, wstart < 0 ? LSA_DEV_INDEX : LSA_DEV_TABLE);
        wstart = max(wstart, 0);     // a window before position 0 does not exist
        t_topk = (tk + LSA_CHUNK - 1) / LSA_CHUNK;
        first_chunk = wstart / LSA_CHUNK;
        total = t_topk + (wlen > 0 ? (wstart + wlen - 1) / LSA_CHUNK - first_chunk + 1 : 0);
    }
    // Pool slot of window unit u, or -1.
    __device__ int window_slot(const DecodeParams &p, int b, int u) const {
        const int chunk = first_chunk + (u - t_topk);
        const int slot = chunk < p.table_stride ? __ldg(p.table + (size_t)b * p.table_stride + chunk) : -1;
        if (slot >= 0 && slot < p.n_slots) return slot;
        flag(p.status, LSA_DEV_TABLE);
        return -1;
    }
    // Is row i of window unit u inside the window?
    __device__ bool in_window(int u, int i) const {
        const int pos = (first_chunk + (u - t_topk)) * LSA_CHUNK + i;
        return pos >= wstart && pos - wstart < wlen;
    }
    // Pool row (slot * 64 + row) of row i of top-k unit u, or -1.
    __device__ int64_t topk_row(const DecodeParams &p, int b, int u, int i) const {
        const int r = u * LSA_CHUNK + i;
        if (r >= tk) return -1;
        const int pos = __ldg(p.topk_idx + (size_t)b * p.k + r);
        if (pos < 0) { flag(p.status, LSA_DEV_INDEX); return -1; }
        const int chunk = pos / LSA_CHUNK;
        const int slot = chunk < p.table_stride ? __ldg(p.table + (size_t)b * p.table_stride + chunk) : -1;
        if (slot >= 0 && slot < p.n_slots) return (int64_t)slot * LSA_CHUNK + (pos % LSA_CHUNK);
        flag(p.status, LSA_DEV_TABLE);
        return -1;
    }
};

// Softmax weights enter P V as f16: exp2(s - m_ref + P_SHIFT), where the reference m_ref follows
// the row maximum only when that has grown by more than 2^RESCALE (so O is rarely rescaled).
// The largest weight is 2^(P_SHIFT + RESCALE) = 2^14 < 65504; a weight stays a normal f16
// number, 11 significant bits, down to 2^-20 of the largest.  Rounding it so leaves a relative
// error of 2^-12 on each weight, an eighth of what rounding a bf16 result leaves, so one part
// serves bf16 outputs.  For f16 and fp32 outputs it would be the largest error of all; there a weight has two
// parts, its f16 rounding and the f16 rounding of the rest, 22 significant bits, and the value product is done
// for both.  Measured, two parts and one: 512K rows whole 71.0 and 64.4 us, 16 ragged sequences 20.2 and 18.9,
// latent rows 49.5 and 38.8 (8 x 10K rows, 128 heads), 169 and 122.6 (32 x 10K, 64 heads); the error of an f16 result
// against 64 bits is 1.0 and 1.4 times that of its rounding alone.
constexpr float RESCALE = 8.f, P_SHIFT = 6.f;
inline bool two_parts(int out_dtype) { return out_dtype != LSA_DTYPE_BF16; }

// What an f16 pair of weights leaves of them.
__device__ __forceinline__ uint32_t rest_f16x2(float lo, float hi, uint32_t rounded) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&rounded));
    return pack_f16x2(lo - f.x, hi - f.y);
}

// Queries enter Q K^T as f16 after a multiplication by a power of two that brings the largest entry of the row into
// [2^15, 2^16), the top of f16's range: f16 queries lose nothing, bf16 ones, which have fewer significant bits, are
// exact down to 2^-32 of the largest, and what is smaller is off by at most 2^-40 of it.
// Products of up to 2^16 * 2688 and their sums are fp32.  Rows below 2^-111 are brought as far up as fp32 factors go.
__device__ __forceinline__ float row_exponent(float amax, float &inv) {
    const uint32_t e = max((__float_as_uint(amax) >> 23) & 255u, 16u);     // 255, infinite or NaN: stays so
    inv = __uint_as_float((269u - e) << 23);
    return __uint_as_float((e - 15u) << 23);
}

// Factor from raw products to scores in base 2.  Positive, so that it keeps the order, and finite: 0 * inf is NaN.
// References are raw products and weights exp2((s - m_ref) * factor + P_SHIFT): the difference is 0 at the
// reference however large the scores are.  With the factor applied first, the roundings of two products of 2^29
// (half a step is 16 there) would push the largest weight out of f16's range, or to zero.
__device__ __forceinline__ float score_factor(float e, float scale_log2) { return fminf(fmaxf(e * scale_log2, 1.2e-38f), 3e38f); }

}  // namespace q4

namespace q4mla {
int launch(const q4::DecodeParams &p, int B, cudaStream_t stream);
int splits(int B, int max_units);
}  // namespace q4mla

}  // namespace lsa
