// norm_rope.cu -- RMS norm of queries and keys for each head and the position rotation, in
// one pass over the rows.
//
//   y = x / sqrt(mean(x[0..nw)^2) + eps) * w      on columns < nw (the norm width, 0: none)
//   columns [ro, ro + rd) are turned by the angles position * inv_freq[i], i < rd / 2, in pairs
//   (u, v) = (ro + i, ro + rd / 2 + i), or interleaved (ro + 2i, ro + 2i + 1):
//     (u, v) <- (u cos - v sin, v cos + u sin)
// Rows are q [T, Hq, D] and k [T, Hk, D]; the same angles serve every head of a token.
//
// A row is read once into registers, by a group of LPR lanes.  A lane takes "items": both
// vectors of a rotated pair (so the partner is always its own), or one vector outside the
// rotation; an interleaved pair lies inside one vector.  The angle is taken in 64 bits: at
// position 5e5 the product has 20 bits before the point, and fp32 would leave it an error of
// 0.03 rad; turns = position * inv_freq / 2 pi, minus its nearest integer, then sincospi in fp32.
// A CTA computes its tokens' cosines and sines once, into shared memory.
#include "nvtx_range.cuh"
#include "q4.cuh"

namespace lsa {
namespace rope {

constexpr int THREADS = 256;
constexpr int MAX_ANGLES = 1024;   // (cos, sin) pairs a CTA holds: tokens x rot / 2

struct Side {
    const void *x;
    void *out;
    const void *w;
    int64_t token_stride, head_stride, out_token_stride, out_head_stride;
    int heads, norm_width;
};

struct Params {
    Side q, k;
    const int32_t *position;
    const float *inv_freq;
    int64_t T;
    int D, ro, rd;
    int tokens;       // tokens a CTA takes
    int row_blocks;   // CTAs that share those tokens' rows (grid.y)
    float eps;
};

// V: elements of a vector; LPR: lanes of a row; ITEMS: items of a lane.
// SCALAR: rows whose addresses allow no vector access are moved element by element.
template <class T, int V, bool SCALAR>
__device__ __forceinline__ Vec<T, V> load_vec(const T *src) {
    if constexpr (!SCALAR) return *reinterpret_cast<const Vec<T, V> *>(src);
    Vec<T, V> v;
#pragma unroll
    for (int j = 0; j < V; ++j) v.v[j] = src[j];
    return v;
}
template <class T, int V, bool SCALAR>
__device__ __forceinline__ void store_vec(T *dst, const Vec<T, V> &v) {
    if constexpr (!SCALAR) {
        *reinterpret_cast<Vec<T, V> *>(dst) = v;
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) dst[j] = v.v[j];
    }
}

template <class T, int V, int LPR, int ITEMS, bool INTER>
__global__ void __launch_bounds__(THREADS) norm_rope_kernel(const Params p) {
    constexpr bool SCALAR = V <= 2;
    __shared__ float2 cs[MAX_ANGLES];
    const int half = p.rd / 2;
    const int64_t t0 = blockIdx.x * (int64_t)p.tokens;
    const int nt = (int)min((int64_t)p.tokens, p.T - t0);
    for (int i = threadIdx.x; i < nt * half; i += THREADS) {
        const int t = i / half;
        const double turns = (double)p.position[t0 + t] * (double)p.inv_freq[i - t * half] * 0.15915494309189533577;
        float s, c;
        sincospif((float)(2.0 * (turns - rint(turns))), &s, &c);
        cs[i] = make_float2(c, s);
    }
    __syncthreads();

    const int sub = threadIdx.x % LPR, grp = threadIdx.x / LPR;
    constexpr int GROUPS = THREADS / LPR;
    const int heads = p.q.heads + p.k.heads, rows = nt * heads;
    // items: the rotated pairs first (half / V of them, or rd / V interleaved vectors), then the rest
    const int pairs = INTER ? 0 : half / V, n_items = p.D / V - pairs;
    for (int r0 = blockIdx.y * GROUPS; r0 < rows; r0 += p.row_blocks * GROUPS) {
        const int r = r0 + grp;
        // every lane of the warp takes part in the shuffles below
        const bool live = r < rows;
        const int t = live ? r / heads : 0, hh = live ? r - t * heads : 0;
        const bool is_q = hh < p.q.heads;
        const Side &s = is_q ? p.q : p.k;
        const int h = is_q ? hh : hh - p.q.heads;
        const bool skip = !live || p.position[t0 + t] < 0;     // padding: the output row stays as it is
        const T *src = static_cast<const T *>(s.x) + (t0 + t) * s.token_stride + h * s.head_stride;
        T *dst = static_cast<T *>(s.out) + (t0 + t) * s.out_token_stride + h * s.out_head_stride;
        float a[ITEMS][V], b[INTER ? 1 : ITEMS][V];
        float sum = 0.f;
        auto first_col = [&](int item) { return item < pairs ? p.ro + item * V : (item - pairs) * V; };
        // outside the rotated columns: vectors are numbered over the whole row, skipping the rotation's
        auto plain_col = [&](int item) {
            const int c = (item - pairs) * V;
            return INTER || c < p.ro ? c : c + p.rd;
        };
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const int item = sub + i * LPR;
            if (skip || item >= n_items) continue;
            const bool pair = !INTER && item < pairs;
            const int c = pair ? first_col(item) : plain_col(item);
            const Vec<T, V> x = load_vec<T, V, SCALAR>(src + c);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                a[i][j] = to_f32(x.v[j]);
                if (c + j < s.norm_width) sum += a[i][j] * a[i][j];
            }
            if constexpr (!INTER) {
                if (pair) {
                    const Vec<T, V> y = load_vec<T, V, SCALAR>(src + c + half);
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        b[i][j] = to_f32(y.v[j]);
                        if (c + half + j < s.norm_width) sum += b[i][j] * b[i][j];
                    }
                }
            }
        }
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (skip) continue;
        const float rms = s.norm_width > 0 ? 1.f / sqrtf(sum / s.norm_width + p.eps) : 1.f;
        const T *w = static_cast<const T *>(s.w);
        auto normed = [&](float x, int c) {
            if (c >= s.norm_width) return x;
            return w ? x * rms * to_f32(w[c]) : x * rms;
        };
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const int item = sub + i * LPR;
            if (item >= n_items) continue;
            const bool pair = !INTER && item < pairs;
            const int c = pair ? first_col(item) : plain_col(item);
#pragma unroll
            for (int j = 0; j < V; ++j) a[i][j] = normed(a[i][j], c + j);
            Vec<T, V> o;
            if constexpr (INTER) {
                if (c >= p.ro && c < p.ro + p.rd) {
#pragma unroll
                    for (int j = 0; j + 1 < V; j += 2) {
                        const float2 f = cs[t * half + (c - p.ro + j) / 2];
                        const float u = a[i][j], v = a[i][j + 1];
                        a[i][j] = u * f.x - v * f.y;
                        a[i][j + 1] = v * f.x + u * f.y;
                    }
                }
            } else if (pair) {
                Vec<T, V> o2;
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float2 f = cs[t * half + item * V + j];
                    const float u = a[i][j], v = normed(b[i][j], c + half + j);
                    a[i][j] = u * f.x - v * f.y;
                    o2.v[j] = from_f32<T>(v * f.x + u * f.y);
                }
                store_vec<T, V, SCALAR>(dst + c + half, o2);
            }
#pragma unroll
            for (int j = 0; j < V; ++j) o.v[j] = from_f32<T>(a[i][j]);
            store_vec<T, V, SCALAR>(dst + c, o);
        }
    }
}

template <class T, int V, bool INTER>
static int launch(Params &p, cudaStream_t stream) {
    const int n_items = p.D / V - (INTER ? 0 : p.rd / 2 / V);
    // as few lanes a row as hold it with one item each, up to a warp
    int lpr = 4;
    while (lpr < 32 && lpr < n_items) lpr *= 2;
    const int items = (n_items + lpr - 1) / lpr;
    const int heads = p.q.heads + p.k.heads, groups = THREADS / lpr, half = p.rd / 2;
    // A CTA takes enough tokens to fill its threads with angles, fewer where that leaves the GPU
    // empty; a single token's rows are dealt over several CTAs when tokens are few.
    const int ctas = 4 * sm_count();
    int tokens = max(1, min(half > 0 ? THREADS / half : 8, MAX_ANGLES / max(half, 1)));
    while (tokens > 1 && (p.T + tokens - 1) / tokens < ctas) tokens /= 2;
    const int64_t blocks = (p.T + tokens - 1) / tokens;
    const int passes = (tokens * heads + groups - 1) / groups;
    p.tokens = tokens;
    p.row_blocks = (int)max((int64_t)1, min((int64_t)passes, ctas / blocks));
    const dim3 grid((unsigned)blocks, p.row_blocks);
#define LSA_ROPE(L, I) norm_rope_kernel<T, V, L, I, INTER><<<grid, THREADS, 0, stream>>>(p)
    constexpr int MOST = 1024 / V / 32;   // items a lane of the widest row can have
    if (items == 1) {
        if (lpr == 4) LSA_ROPE(4, 1);
        else if (lpr == 8) LSA_ROPE(8, 1);
        else if (lpr == 16) LSA_ROPE(16, 1);
        else LSA_ROPE(32, 1);
    } else if (items == 2) LSA_ROPE(32, 2);
    else if (MOST <= 4 || items <= 4) LSA_ROPE(32, 4);
    else LSA_ROPE(32, (MOST <= 4 ? 4 : MOST));
#undef LSA_ROPE
    return check_launch("norm_rope_kernel");
}

template <class T>
static int dispatch(Params &p, bool inter, int vec, cudaStream_t stream) {
    constexpr int FULL = 16 / sizeof(T);
    if (inter) {
        if (vec == FULL) return launch<T, FULL, true>(p, stream);
        if (vec >= 4) return launch<T, 4, true>(p, stream);
        return launch<T, 2, true>(p, stream);
    }
    if (vec == FULL) return launch<T, FULL, false>(p, stream);
    if (vec >= 4) return launch<T, 4, false>(p, stream);
    return launch<T, 1, false>(p, stream);
}

}  // namespace rope
}  // namespace lsa

using namespace lsa;

extern "C" int lsa_qk_norm_rope(int dtype, int64_t T, int head_dim, const void *q, int64_t q_token_stride,
                                int64_t q_head_stride, int Hq, const void *q_weight, int q_norm_width, void *q_out,
                                int64_t q_out_token_stride, int64_t q_out_head_stride, const void *k,
                                int64_t k_token_stride, int64_t k_head_stride, int Hk, const void *k_weight,
                                int k_norm_width, void *k_out, int64_t k_out_token_stride, int64_t k_out_head_stride,
                                float eps, const int32_t *position, const float *inv_freq, int rot_offset, int rot_dim,
                                int interleaved, lsa_stream_t stream) {
    LSA_ABI_RANGE();
    LSA_REQUIRE(dtype_known(dtype), LSA_ERR_INVALID_ARG, "lsa_qk_norm_rope: unknown dtype %d", dtype);
    LSA_REQUIRE(T >= 0 && T < (1ll << 31) && Hq >= 0 && Hk >= 0 && Hq + Hk >= 1 && Hq <= 1024 && Hk <= 1024,
                LSA_ERR_INVALID_ARG, "lsa_qk_norm_rope: bad sizes (T=%lld Hq=%d Hk=%d)", (long long)T, Hq, Hk);
    LSA_REQUIRE(head_dim >= 2 && head_dim % 2 == 0 && head_dim <= 1024 && rot_dim >= 0 && rot_dim % 2 == 0 &&
                    rot_offset >= 0 && rot_offset % 2 == 0 && rot_offset + rot_dim <= head_dim,
                LSA_ERR_SHAPE,
                "lsa_qk_norm_rope: unsupported head_dim=%d rot_offset=%d rot_dim=%d (even, head_dim up to 1024, the "
                "rotation inside the row)",
                head_dim, rot_offset, rot_dim);
    LSA_REQUIRE(q_norm_width >= 0 && q_norm_width <= head_dim && k_norm_width >= 0 && k_norm_width <= head_dim,
                LSA_ERR_INVALID_ARG, "lsa_qk_norm_rope: norm widths (%d, %d) outside [0, %d]", q_norm_width,
                k_norm_width, head_dim);
    LSA_REQUIRE(eps >= 0.f, LSA_ERR_INVALID_ARG, "lsa_qk_norm_rope: eps must not be negative");
    LSA_REQUIRE(T == 0 || ((Hq == 0 || (q && q_out)) && (Hk == 0 || (k && k_out)) && position && (rot_dim == 0 || inv_freq)),
                LSA_ERR_INVALID_ARG, "lsa_qk_norm_rope: null pointer");
    const int64_t size = dtype_size(dtype);
    auto natural = [&](const void *ptr) { return reinterpret_cast<uintptr_t>(ptr) % size == 0; };
    LSA_REQUIRE(natural(q) && natural(k) && natural(q_out) && natural(k_out) && natural(q_weight) && natural(k_weight),
                LSA_ERR_INVALID_ARG, "lsa_qk_norm_rope: a pointer is not aligned to its element type");
    if (T == 0) return LSA_OK;
    rope::Params p = {};
    p.q = {q, q_out, q_weight, q_token_stride, q_head_stride, q_out_token_stride, q_out_head_stride, Hq, q_norm_width};
    p.k = {k, k_out, k_weight, k_token_stride, k_head_stride, k_out_token_stride, k_out_head_stride, Hk, k_norm_width};
    p.position = position; p.inv_freq = inv_freq; p.T = T; p.D = head_dim; p.ro = rot_offset; p.rd = rot_dim; p.eps = eps;
    // The widest vector (up to 16 bytes) that divides the row, the rotation's bounds, and every
    // row's address.
    const int64_t full = 16 / size, unit = interleaved ? 1 : rot_dim / 2;
    int64_t bits = head_dim | rot_offset | (interleaved ? rot_dim : unit);
    for (const rope::Side *s : {&p.q, &p.k})
        if (s->heads)
            bits |= s->token_stride | s->head_stride | s->out_token_stride | s->out_head_stride |
                    (int64_t)(reinterpret_cast<uintptr_t>(s->x) / size) | (int64_t)(reinterpret_cast<uintptr_t>(s->out) / size);
    int64_t vec = full;
    while (vec > 1 && bits % vec) vec /= 2;
    if (dtype == LSA_DTYPE_BF16) return rope::dispatch<__nv_bfloat16>(p, interleaved != 0, (int)vec, stream);
    if (dtype == LSA_DTYPE_F16) return rope::dispatch<__half>(p, interleaved != 0, (int)vec, stream);
    return rope::dispatch<float>(p, interleaved != 0, (int)vec, stream);
}
