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
// rotation; an interleaved pair lies inside one vector.  A group keeps to one token and walks its
// heads; the next head's vectors are loaded while this one's are worked on.
// Norm weight, cosine and sine are folded once per token into two coefficients a value: with
// n = x / rms,  out = n P + n_partner Q,  P = w cos, Q = -+ w_partner sin (w and 0 outside the rotation).
// That leaves about 150 instructions for the 16 values a lane has of a row; with weights converted
// and three products a value for every head it was 520, and the issue slots were the bound (65 us for
// 8192 tokens of 40 rows of 128, now 36.5; several heads in flight at fewer warps: 110 us).
// The angle is taken in 64 bits: at position 5e5 the product has 20 bits before the point, and
// fp32 would leave it an error of 0.03 rad; turns = position * inv_freq / 2 pi, minus its nearest
// integer, then sincospi in fp32.  A CTA computes its tokens' cosines and sines once, into shared
// memory, laid out so that neighbouring lanes read neighbouring words.
// Bound by memory: 4 bytes a bf16 value.
#include "nvtx_range.cuh"
#include "q4.cuh"

namespace lsa {
namespace rope {

constexpr int THREADS = 128;
constexpr int MAX_ANGLES = 1024;   // (cos, sin) pairs a CTA holds: tokens x rot / 2

struct Side {
    const void *x;
    void *out;
    const void *w;
    int64_t token_stride, head_stride, out_token_stride, out_head_stride;
    int heads, norm_width;
    float inv_width;  // 1 / norm_width
};

struct Params {
    Side q, k;
    const int32_t *position;
    const float *inv_freq;
    int64_t T;
    int D, ro, rd;
    int tokens;       // tokens a CTA takes
    int per_token;    // lane groups of a CTA that share a token's heads: tokens * per_token = THREADS / LPR
    float eps;
};

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

// V: elements of a vector; LPR: lanes of a row; ITEMS: items of a lane.  V > 2 divides every bound of the row
// (rotation, norm widths); V <= 2 moves and checks element by element.
template <class T, int V, int LPR, int ITEMS, bool INTER>
__global__ void __launch_bounds__(THREADS, ITEMS == 1 ? 5 : 1) norm_rope_kernel(const Params p) {
    constexpr bool SCALAR = V <= 2;
    constexpr int NA = INTER ? (V + 1) / 2 : V;      // angles of an item
    constexpr int IB = INTER ? 1 : ITEMS;            // second vectors of items
    __shared__ float2 cs[MAX_ANGLES];
    const int half = p.rd / 2;
    const int slots = half / NA;                     // rotated items of a row
    const int64_t t0 = blockIdx.x * (int64_t)p.tokens;
    const int nt = (int)min((int64_t)p.tokens, p.T - t0);
    const int sub = threadIdx.x % LPR, grp = threadIdx.x / LPR;
    const int t = grp / p.per_token, g = grp - t * p.per_token;
    // padding: the output rows stay as they are
    const bool live = t < nt && p.position[t0 + min(t, nt - 1)] >= 0;

    // items: the rotated pairs first (or, interleaved, every vector in order), then the rest
    const int pairs = INTER ? 0 : half / V, n_items = p.D / V - pairs;
    int col[ITEMS];
    bool turn[ITEMS], have[ITEMS];
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
        const int item = sub + i * LPR;
        have[i] = live && item < n_items;
        const int rest = (item - pairs) * V;
        col[i] = item < pairs ? p.ro + item * V : (INTER || rest < p.ro ? rest : rest + p.rd);
        turn[i] = have[i] && (INTER ? col[i] >= p.ro && col[i] < p.ro + p.rd : item < pairs);
    }
    // The groups of a warp take the same turns, so that the shuffles need no masks of their own: shuffles under
    // masks that differ from lane to lane are serialised.
    const int first = blockIdx.y * p.per_token, step = gridDim.y * p.per_token;
    Vec<T, V> xa[ITEMS], xb[IB];
    auto fetch = [&](const Side &s, int h) {
        if (h >= s.heads) return;
        const T *src = static_cast<const T *>(s.x) + (t0 + t) * s.token_stride + h * s.head_stride;
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            if (have[i]) xa[i] = load_vec<T, V, SCALAR>(src + col[i]);
            if constexpr (!INTER)
                if (turn[i]) xb[i] = load_vec<T, V, SCALAR>(src + col[i] + half);
        }
    };
    fetch(p.q, first + g);     // on its way while the angles are computed

    // angle i = slot * NA + j of token t sits at (t * NA + j) * slots + slot
    for (int i = threadIdx.x; i < nt * half; i += THREADS) {
        const int t = i / half, a = i - t * half, slot = a / NA, j = a - slot * NA;
        const double turns = (double)p.position[t0 + t] * (double)p.inv_freq[a] * 0.15915494309189533577;
        float s, c;
        sincospif((float)(2.0 * (turns - rint(turns))), &s, &c);
        cs[(t * NA + j) * slots + slot] = make_float2(c, s);
    }
    __syncthreads();

    auto walk = [&](const Side &s, bool fetched) {
        if (first >= s.heads) return;
        if (!fetched) fetch(s, first + g);
        const int nw = s.norm_width;
        // column c takes part in the norm; a vector does as a whole where V > 2
        auto normed = [&](int c) { return c < nw; };
        float Pa[ITEMS][V], Qa[ITEMS][V], Pb[IB][V], Qb[IB][V];
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const T *w = static_cast<const T *>(s.w);
            float wa[V], wb[V];
#pragma unroll
            for (int j = 0; j < V; ++j) wa[j] = wb[j] = 1.f;
            if constexpr (SCALAR) {
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    if (w && have[i] && normed(col[i] + j)) wa[j] = to_f32(w[col[i] + j]);
                    if (!INTER && w && turn[i] && normed(col[i] + half + j)) wb[j] = to_f32(w[col[i] + half + j]);
                }
            } else {
                if (w && have[i] && normed(col[i])) widen(load_vec<T, V, false>(w + col[i]), wa);
                if (!INTER && w && turn[i] && normed(col[i] + half)) widen(load_vec<T, V, false>(w + col[i] + half), wb);
            }
            const int slot = INTER ? (col[i] - p.ro) / V : sub + i * LPR;
#pragma unroll
            for (int j = 0; j < NA; ++j) {
                const float2 f = turn[i] ? cs[(t * NA + j) * slots + slot] : make_float2(1.f, 0.f);
                if constexpr (INTER) {
                    Pa[i][2 * j] = wa[2 * j] * f.x;
                    Qa[i][2 * j] = -wa[2 * j + 1] * f.y;
                    Pa[i][2 * j + 1] = wa[2 * j + 1] * f.x;
                    Qa[i][2 * j + 1] = wa[2 * j] * f.y;
                } else {
                    Pa[i][j] = wa[j] * f.x;
                    Qa[i][j] = -wb[j] * f.y;
                    Pb[i][j] = wb[j] * f.x;
                    Qb[i][j] = wa[j] * f.y;
                }
            }
        }
        T *dst = static_cast<T *>(s.out) + (t0 + t) * s.out_token_stride + (first + g) * s.out_head_stride;
#pragma unroll 1
        for (int h0 = first; h0 < s.heads; h0 += step, dst += step * s.out_head_stride) {
            float a[ITEMS][V], b[IB][V];
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < ITEMS; ++i) {
                widen(xa[i], a[i]);
                if constexpr (!INTER) widen(xb[i], b[i]);
                if (have[i] && (SCALAR || normed(col[i])))
#pragma unroll
                    for (int j = 0; j < V; ++j)
                        if (!SCALAR || normed(col[i] + j)) sum += a[i][j] * a[i][j];
                if constexpr (!INTER)
                    if (turn[i] && (SCALAR || normed(col[i] + half)))
#pragma unroll
                        for (int j = 0; j < V; ++j)
                            if (!SCALAR || normed(col[i] + half + j)) sum += b[i][j] * b[i][j];
            }
            fetch(s, h0 + step + g);
            float rms = 1.f;
            if (nw > 0) {
#pragma unroll
                for (int o = LPR / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                rms = rsqrtf(sum * s.inv_width + p.eps);
            }
            if (h0 + g >= s.heads) continue;
#pragma unroll
            for (int i = 0; i < ITEMS; ++i) {
                if (!have[i]) continue;
                const float ra = normed(col[i]) ? rms : 1.f, rb = normed(col[i] + half) ? rms : 1.f;
                float oa[V];
#pragma unroll
                for (int j = 0; j < V; ++j) a[i][j] *= SCALAR && !normed(col[i] + j) ? 1.f : SCALAR ? rms : ra;
                if constexpr (INTER) {
#pragma unroll
                    for (int j = 0; j < V; ++j) oa[j] = turn[i] ? fmaf(a[i][j ^ 1], Qa[i][j], a[i][j] * Pa[i][j]) : a[i][j] * Pa[i][j];
                } else if (turn[i]) {
                    float ob[V];
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        b[i][j] *= SCALAR && !normed(col[i] + half + j) ? 1.f : SCALAR ? rms : rb;
                        oa[j] = fmaf(b[i][j], Qa[i][j], a[i][j] * Pa[i][j]);
                        ob[j] = fmaf(a[i][j], Qb[i][j], b[i][j] * Pb[i][j]);
                    }
                    store_vec<T, V, SCALAR>(dst + col[i] + half, narrow<T, V>(ob));
                } else {
#pragma unroll
                    for (int j = 0; j < V; ++j) oa[j] = a[i][j] * Pa[i][j];
                }
                store_vec<T, V, SCALAR>(dst + col[i], narrow<T, V>(oa));
            }
        }
    };
    walk(p.q, true);
    walk(p.k, false);
}

template <class T, int V, bool INTER>
static int launch(Params &p, cudaStream_t stream) {
    const int n_items = p.D / V - (INTER ? 0 : p.rd / 2 / V);
    // as few lanes a row as hold it with one item each, up to a warp
    int lpr = 4;
    while (lpr < 32 && lpr < n_items) lpr *= 2;
    const int items = (n_items + lpr - 1) / lpr;
    const int heads = max(p.q.heads, p.k.heads), groups = THREADS / lpr, half = p.rd / 2;
    // Lane groups that fill the GPU (2048 threads a multiprocessor), dealt to the tokens: with many tokens a group
    // takes many heads of its token, with few the heads are spread over groups and CTAs.  (8192 tokens of 40
    // rows: 36.5 us; groups for 4096 or 1024 threads: 46 and 48; CTAs of 256: 39; 7 or 8 CTAs a
    // multiprocessor, which spill: 39 and 43.)
    const int64_t all = (int64_t)sm_count() * 2048 / lpr;
    int64_t want = lsa_max64(1, lsa_min64(heads, all / lsa_max64(p.T, 1)));
    int per_token = 1;
    while (per_token < groups && per_token < want) per_token *= 2;
    while (half > 0 && groups / per_token * half > MAX_ANGLES && per_token < groups) per_token *= 2;
    p.per_token = per_token;
    p.tokens = groups / per_token;
    const dim3 grid((unsigned)((p.T + p.tokens - 1) / p.tokens), (unsigned)((want + per_token - 1) / per_token));
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
    // rows nearer to each other than their length overlap, as the rows of an expanded tensor do
    auto apart = [&](int64_t stride, int64_t n) { return n <= 1 || stride >= head_dim || stride <= -head_dim; };
    LSA_REQUIRE((Hq == 0 || (apart(q_out_token_stride, T) && apart(q_out_head_stride, Hq))) &&
                    (Hk == 0 || (apart(k_out_token_stride, T) && apart(k_out_head_stride, Hk))),
                LSA_ERR_INVALID_ARG, "lsa_qk_norm_rope: output rows overlap");
    if (T == 0) return LSA_OK;
    rope::Params p = {};
    p.q = {q, q_out, q_weight, q_token_stride, q_head_stride, q_out_token_stride, q_out_head_stride, Hq, q_norm_width, q_norm_width ? 1.f / q_norm_width : 0.f};
    p.k = {k, k_out, k_weight, k_token_stride, k_head_stride, k_out_token_stride, k_out_head_stride, Hk, k_norm_width, k_norm_width ? 1.f / k_norm_width : 0.f};
    p.position = position; p.inv_freq = inv_freq; p.T = T; p.D = head_dim; p.ro = rot_offset; p.rd = rot_dim; p.eps = eps;
    // The widest vector (up to 16 bytes) that divides the row, the rotation's and norms' bounds, and
    // every row's address.
    const int64_t full = 16 / size, unit = interleaved ? 1 : rot_dim / 2;
    int64_t bits = head_dim | rot_offset | (interleaved ? rot_dim : unit);
    for (const rope::Side *s : {&p.q, &p.k})
        if (s->heads)
            bits |= s->norm_width | (int64_t)(reinterpret_cast<uintptr_t>(s->w) / size) | s->token_stride | s->head_stride | s->out_token_stride | s->out_head_stride |
                    (int64_t)(reinterpret_cast<uintptr_t>(s->x) / size) | (int64_t)(reinterpret_cast<uintptr_t>(s->out) / size);
    int64_t vec = full;
    while (vec > 1 && bits % vec) vec /= 2;
    if (dtype == LSA_DTYPE_BF16) return rope::dispatch<__nv_bfloat16>(p, interleaved != 0, (int)vec, stream);
    if (dtype == LSA_DTYPE_F16) return rope::dispatch<__half>(p, interleaved != 0, (int)vec, stream);
    return rope::dispatch<float>(p, interleaved != 0, (int)vec, stream);
}
