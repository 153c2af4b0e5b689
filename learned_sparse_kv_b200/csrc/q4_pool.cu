// q4_pool.cu -- rows in and out of the 4-bit chunk pools: quantised writes through a slot map
// (prefill and decode batches) or to the end of the recent window (one decoded token per
// sequence), and the read back.
//
// One thread owns one group of 16 values: its maximum, its scale, its 8 code bytes and its
// scale byte need no other thread, and consecutive threads touch consecutive memory.  Bound
// by memory: 2 + 0.5625 bytes a bf16 value.
#include "nvtx_range.cuh"
#include "q4.cuh"

namespace lsa {

// One side (K or V) of a write: rows x[t, h, 0..W) at x + t * token_stride + h * head_stride.
struct Q4Side {
    const void *x;
    uint8_t *pool;
    int64_t token_stride, head_stride;
    int W;
    float g, g6;
};

// Quantises group `grp` of row (t, h) into pool row `slot` (slot * 64 + row in the chunk).
template <class T>
__device__ __forceinline__ void write_group(const Q4Side &s, int heads, int64_t t, int h, int grp, int64_t slot) {
    const T *src = static_cast<const T *>(s.x) + t * s.token_stride + h * s.head_stride + grp * q4::GROUP;
    float x[16];
    constexpr int PER = 16 / sizeof(T);
#pragma unroll
    for (int i = 0; i < 16 / PER; ++i) {
        const Vec<T, PER> v = *reinterpret_cast<const Vec<T, PER> *>(src + i * PER);
#pragma unroll
        for (int j = 0; j < PER; ++j) x[i * PER + j] = to_f32(v.v[j]);
    }
    uint32_t sb;
    const uint2 codes = q4::quantise_group(x, s.g, s.g6, sb);
    uint8_t *chunk = s.pool + ((slot / LSA_CHUNK) * heads + h) * q4::chunk_bytes(s.W);
    const int r = (int)(slot % LSA_CHUNK);
    *reinterpret_cast<uint2 *>(chunk + r * q4::code_row(s.W) + grp * 8) = codes;
    chunk[q4::scale_base(s.W) + r * q4::scale_row(s.W) + grp] = (uint8_t)sb;
}

// grid-stride over (token, side, head, group); `per` groups a token over both sides.
template <class T>
__global__ void __launch_bounds__(256) q4_write_kernel(const Q4Side a, const Q4Side b, int heads, int64_t n, int per,
                                                       int per_a, int64_t n_rows, const int64_t *__restrict__ slot_map,
                                                       int32_t *status) {
    for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < n; i += gridDim.x * 256ll) {
        const int64_t t = i / per;
        int u = (int)(i - t * per);
        const int64_t slot = slot_map[t];
        if (slot < 0 || slot >= n_rows) {
            if (slot != -1) flag(status, LSA_DEV_INDEX);
            continue;
        }
        const bool first = u < per_a;
        if (!first) u -= per_a;
        const Q4Side &s = first ? a : b;
        const int groups = s.W / q4::GROUP, h = u / groups;
        write_group<T>(s, heads, t, h, u - h * groups, slot);
    }
}

// One CTA per sequence: the rows of the token at window_start + window_len, then window_len + 1.
template <class T>
__global__ void __launch_bounds__(256) q4_append_kernel(const Q4Side a, const Q4Side b, int heads, int per, int per_a,
                                                        const uint16_t *__restrict__ new_li,
                                                        uint16_t *__restrict__ li_pool, int dl, int64_t n_slots,
                                                        const int32_t *__restrict__ table, int table_stride,
                                                        const int32_t *__restrict__ window_start,
                                                        int32_t *__restrict__ window_len, int32_t *status) {
    __shared__ int64_t s_row;
    const int seq = blockIdx.x;
    if (threadIdx.x == 0) {
        const int64_t pos = (int64_t)window_start[seq] + window_len[seq];
        const int64_t chunk = pos / LSA_CHUNK;
        const int slot = (pos >= 0 && chunk < table_stride) ? table[(size_t)seq * table_stride + chunk] : -1;
        s_row = (slot >= 0 && slot < n_slots) ? (int64_t)slot * LSA_CHUNK + pos % LSA_CHUNK : -1;
        if (s_row < 0) flag(status, LSA_DEV_TABLE);
    }
    __syncthreads();
    const int64_t row = s_row;
    if (row < 0) return;
    for (int i = threadIdx.x; i < per; i += 256) {
        const bool first = i < per_a;
        const Q4Side &s = first ? a : b;
        const int u = first ? i : i - per_a, groups = s.W / q4::GROUP, h = u / groups;
        write_group<T>(s, heads, seq, h, u - h * groups, row);
    }
    if (li_pool)
        for (int c = threadIdx.x; c < dl / 8; c += 256)
            reinterpret_cast<uint4 *>(li_pool + row * dl)[c] = reinterpret_cast<const uint4 *>(new_li + (size_t)seq * dl)[c];
    if (threadIdx.x == 0) window_len[seq] += 1;   // after the barrier above: every thread has its row
}

template <class T>
__global__ void __launch_bounds__(256) q4_read_kernel(const uint8_t *__restrict__ pool, int heads, int W, int64_t n_rows,
                                                      const int64_t *__restrict__ slot_map, int64_t n, float g,
                                                      T *__restrict__ out, int32_t *status) {
    const int groups = W / q4::GROUP, per = heads * groups;
    for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < n; i += gridDim.x * 256ll) {
        const int64_t t = i / per;
        const int u = (int)(i - t * per), h = u / groups, grp = u - h * groups;
        const int64_t slot = slot_map[t];
        const bool there = slot >= 0 && slot < n_rows;
        uint2 codes = make_uint2(0u, 0u);
        float s = 0.f;
        if (there) {
            const uint8_t *chunk = pool + ((slot / LSA_CHUNK) * heads + h) * q4::chunk_bytes(W);
            const int r = (int)(slot % LSA_CHUNK);
            codes = *reinterpret_cast<const uint2 *>(chunk + r * q4::code_row(W) + grp * 8);
            const uint32_t sh = q4::e4m3x2_to_f16(chunk[q4::scale_base(W) + r * q4::scale_row(W) + grp]);
            s = __half2float(__ushort_as_half((uint16_t)sh));
        } else if (slot != -1) {
            flag(status, LSA_DEV_INDEX);
        }
        float x[16];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            uint32_t p[4];
            q4::e2m1x8_to_f16(j ? codes.y : codes.x, p);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&p[k]));
                x[8 * j + 2 * k] = f.x * s * g;        // e2m1 * e4m3 is exact: one rounding, with g
                x[8 * j + 2 * k + 1] = f.y * s * g;
            }
        }
        constexpr int PER = 16 / sizeof(T);
        T *dst = out + i * q4::GROUP;
#pragma unroll
        for (int k = 0; k < 16 / PER; ++k) {
            Vec<T, PER> v;
#pragma unroll
            for (int j = 0; j < PER; ++j) v.v[j] = from_f32<T>(x[k * PER + j]);
            *reinterpret_cast<Vec<T, PER> *>(dst + k * PER) = v;
        }
    }
}

static int q4_blocks(int64_t n) { return (int)lsa_min64((n + 255) / 256, (int64_t)sm_count() * 16); }

static bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Checks one side (`rows`: there are rows to read); returns LSA_OK or the error.
static int check_side(const char *who, const char *name, const Q4Side &s, int dtype, bool rows) {
    const int per = 16 / dtype_size(dtype);
    LSA_REQUIRE((s.x || !rows) && s.pool, LSA_ERR_INVALID_ARG, "%s: null pointer (%s)", who, name);
    LSA_REQUIRE(s.W >= 16 && s.W % 16 == 0 && s.W <= 4096, LSA_ERR_SHAPE,
                "%s: unsupported %s width %d (a multiple of 16 up to 4096)", who, name, s.W);
    LSA_REQUIRE(s.token_stride % per == 0 && s.head_stride % per == 0 && aligned16(s.x) && aligned16(s.pool),
                LSA_ERR_INVALID_ARG, "%s: %s rows and pool must be 16-byte aligned, row strides too", who, name);
    LSA_REQUIRE(s.g > 0.f && s.g <= 1e30f && s.g >= 1e-30f, LSA_ERR_INVALID_ARG,
                "%s: the %s pool scale must be positive and between 1e-30 and 1e30", who, name);
    return LSA_OK;
}

}  // namespace lsa

using namespace lsa;

extern "C" int64_t lsa_q4_chunk_bytes(int width) {
    return width >= 16 && width % 16 == 0 && width <= 4096 ? q4::chunk_bytes(width) : 0;
}

extern "C" int lsa_write_q4(int dtype, int64_t T, int heads, const void *k, int64_t k_token_stride,
                            int64_t k_head_stride, int k_width, uint8_t *k_pool, float k_scale, const void *v,
                            int64_t v_token_stride, int64_t v_head_stride, int v_width, uint8_t *v_pool, float v_scale,
                            int64_t n_slots, const int64_t *slot_map, int32_t *dev_status, lsa_stream_t stream) {
    LSA_ABI_RANGE();
    LSA_REQUIRE(dtype_known(dtype), LSA_ERR_INVALID_ARG, "lsa_write_q4: unknown dtype %d", dtype);
    LSA_REQUIRE(T >= 0 && T < (1ll << 31) && heads >= 1 && heads <= 1024 && n_slots >= 1 && n_slots < (1ll << 31),
                LSA_ERR_INVALID_ARG, "lsa_write_q4: bad sizes (T=%lld heads=%d n_slots=%lld)", (long long)T, heads,
                (long long)n_slots);
    Q4Side a = {k, k_pool, k_token_stride, k_head_stride, k_width, k_scale, q4::E2M1_MAX * k_scale};
    Q4Side b = {v, v_pool, v_token_stride, v_head_stride, v_width, v_scale, q4::E2M1_MAX * v_scale};
    if (int rc = check_side("lsa_write_q4", "k", a, dtype, T > 0)) return rc;
    const bool two = v_pool != nullptr;
    if (two)
        if (int rc = check_side("lsa_write_q4", "v", b, dtype, T > 0)) return rc;
    LSA_REQUIRE(two || !v, LSA_ERR_INVALID_ARG, "lsa_write_q4: v without a v_pool");
    LSA_REQUIRE(slot_map || T == 0, LSA_ERR_INVALID_ARG, "lsa_write_q4: null pointer (slot_map)");
    if (T == 0) return LSA_OK;
    const int per_a = heads * (a.W / 16), per = per_a + (two ? heads * (b.W / 16) : 0);
    const int64_t n = T * per, rows = n_slots * LSA_CHUNK;
    const int blocks = q4_blocks(n);
    if (dtype == LSA_DTYPE_BF16)
        q4_write_kernel<__nv_bfloat16><<<blocks, 256, 0, stream>>>(a, b, heads, n, per, per_a, rows, slot_map, dev_status);
    else if (dtype == LSA_DTYPE_F16)
        q4_write_kernel<__half><<<blocks, 256, 0, stream>>>(a, b, heads, n, per, per_a, rows, slot_map, dev_status);
    else
        q4_write_kernel<float><<<blocks, 256, 0, stream>>>(a, b, heads, n, per, per_a, rows, slot_map, dev_status);
    return check_launch("q4_write_kernel");
}

extern "C" int lsa_append_token_q4(int dtype, int heads, const void *new_k, int k_width, uint8_t *k_pool, float k_scale,
                                   const void *new_v, int v_width, uint8_t *v_pool, float v_scale,
                                   const lsa_bf16 *new_li, lsa_bf16 *li_pool, int dl, int64_t n_slots,
                                   const int32_t *chunk_table, int table_stride, const int32_t *window_start,
                                   int32_t *window_len, int B, int32_t *dev_status, lsa_stream_t stream) {
    LSA_ABI_RANGE();
    LSA_REQUIRE(dtype_known(dtype), LSA_ERR_INVALID_ARG, "lsa_append_token_q4: unknown dtype %d", dtype);
    LSA_REQUIRE(B > 0 && heads >= 1 && heads <= 1024 && n_slots >= 1 && n_slots < (1ll << 31) && table_stride >= 1,
                LSA_ERR_INVALID_ARG, "lsa_append_token_q4: bad sizes (B=%d heads=%d n_slots=%lld table_stride=%d)", B,
                heads, (long long)n_slots, table_stride);
    LSA_REQUIRE(chunk_table && window_start && window_len, LSA_ERR_INVALID_ARG, "lsa_append_token_q4: null pointer");
    Q4Side a = {new_k, k_pool, (int64_t)heads * k_width, k_width, k_width, k_scale, q4::E2M1_MAX * k_scale};
    Q4Side b = {new_v, v_pool, (int64_t)heads * v_width, v_width, v_width, v_scale, q4::E2M1_MAX * v_scale};
    if (int rc = check_side("lsa_append_token_q4", "k", a, dtype, true)) return rc;
    const bool two = v_pool != nullptr;
    if (two)
        if (int rc = check_side("lsa_append_token_q4", "v", b, dtype, true)) return rc;
    LSA_REQUIRE(two || !new_v, LSA_ERR_INVALID_ARG, "lsa_append_token_q4: new_v without a v_pool");
    LSA_REQUIRE((li_pool != nullptr) == (new_li != nullptr) &&
                    (!li_pool || (dl >= 8 && dl % 8 == 0 && aligned16(new_li) && aligned16(li_pool))),
                LSA_ERR_INVALID_ARG,
                "lsa_append_token_q4: new_li and li_pool come together, 16-byte aligned, dl a multiple of 8");
    const int per_a = heads * (a.W / 16), per = per_a + (two ? heads * (b.W / 16) : 0);
    if (dtype == LSA_DTYPE_BF16)
        q4_append_kernel<__nv_bfloat16><<<B, 256, 0, stream>>>(a, b, heads, per, per_a, new_li, li_pool, dl, n_slots, chunk_table, table_stride, window_start, window_len, dev_status);
    else if (dtype == LSA_DTYPE_F16)
        q4_append_kernel<__half><<<B, 256, 0, stream>>>(a, b, heads, per, per_a, new_li, li_pool, dl, n_slots, chunk_table, table_stride, window_start, window_len, dev_status);
    else
        q4_append_kernel<float><<<B, 256, 0, stream>>>(a, b, heads, per, per_a, new_li, li_pool, dl, n_slots, chunk_table, table_stride, window_start, window_len, dev_status);
    return check_launch("q4_append_kernel");
}

extern "C" int lsa_read_q4(const uint8_t *pool, int64_t n_slots, int heads, int width, float scale,
                           const int64_t *slot_map, int64_t T, int out_dtype, void *out, int32_t *dev_status,
                           lsa_stream_t stream) {
    LSA_ABI_RANGE();
    LSA_REQUIRE(dtype_known(out_dtype), LSA_ERR_INVALID_ARG, "lsa_read_q4: unknown dtype %d", out_dtype);
    LSA_REQUIRE(T >= 0 && T < (1ll << 31) && heads >= 1 && heads <= 1024 && n_slots >= 1 && n_slots < (1ll << 31),
                LSA_ERR_INVALID_ARG, "lsa_read_q4: bad sizes (T=%lld heads=%d n_slots=%lld)", (long long)T, heads,
                (long long)n_slots);
    LSA_REQUIRE(width >= 16 && width % 16 == 0 && width <= 4096, LSA_ERR_SHAPE,
                "lsa_read_q4: unsupported width %d (a multiple of 16 up to 4096)", width);
    LSA_REQUIRE(pool && (T == 0 || (slot_map && out)), LSA_ERR_INVALID_ARG, "lsa_read_q4: null pointer");
    LSA_REQUIRE(aligned16(pool) && aligned16(out), LSA_ERR_INVALID_ARG, "lsa_read_q4: pool and out must be 16-byte aligned");
    LSA_REQUIRE(scale > 0.f && scale <= 1e30f && scale >= 1e-30f, LSA_ERR_INVALID_ARG,
                "lsa_read_q4: the pool scale must be positive and between 1e-30 and 1e30");
    if (T == 0) return LSA_OK;
    const int64_t n = T * heads * (width / 16), rows = n_slots * LSA_CHUNK;
    const int blocks = q4_blocks(n);
    if (out_dtype == LSA_DTYPE_BF16)
        q4_read_kernel<<<blocks, 256, 0, stream>>>(pool, heads, width, rows, slot_map, n, scale, static_cast<__nv_bfloat16 *>(out), dev_status);
    else if (out_dtype == LSA_DTYPE_F16)
        q4_read_kernel<<<blocks, 256, 0, stream>>>(pool, heads, width, rows, slot_map, n, scale, static_cast<__half *>(out), dev_status);
    else
        q4_read_kernel<<<blocks, 256, 0, stream>>>(pool, heads, width, rows, slot_map, n, scale, static_cast<float *>(out), dev_status);
    return check_launch("q4_read_kernel");
}
