// q4_decode.cu -- decode attention over 4-bit pools: the entry point, the kernel for separate
// K and V pools (grouped heads), and the merge of the splits.  (Latent rows: q4_decode_sm100.cu.)
//
//   o[h] = sum_j softmax_j(scale q_h . K_j) V_j over the top-k rows and the window
//
// A row of one K/V head is 0.5625 byte a value, and G = Hq / Hkv query heads share it: 3.6 G
// flops a byte, so for the usual G the pool's bytes bound it.  Design:
//  - A warp owns units of 64 rows by itself (a window chunk, or 64 gathered top-k rows): it
//    copies codes and scales with cp.async into its own ring of shared-memory stages and waits
//    for its own copies only, so the loop has no block barrier.
//  - The matrix products are transposed, S^T = K Q^T and O^T = V^T P^T, on m16n8k16: rows of K
//    are the M side and 8 query heads the N side, which wastes nothing for up to 8 heads a K/V
//    head, and the dequantised codes are the A operand straight from registers.
//  - The contraction index of a product may be permuted freely.  For S^T lane t of a row's four
//    lanes takes columns D/4 t .. D/4 t + D/4 - 1, contiguous codes: one 16-byte shared load; for
//    O^T lane group g takes value columns D/8 g .. , contiguous again.  There a register holds two
//    tokens of one column: the nibbles of two tokens' words are interleaved before the conversion (four
//    operations for 16 values), and their scales are a pair likewise.
//  - P^T goes from the accumulator layout to the operand layout with movmatrix, no memory.
// The grid is one wave of CTAs.  All units of all (sequence, K/V head, group of query heads) segments are
// counted on the device and dealt to the CTAs in equal contiguous ranges, so ragged lengths cost
// nothing: a CTA walks the segments of its range, its warps take a segment's units in turn and merge
// through shared memory.  A segment counts SETUP units more than it has, which is what its start
// and its merge take: otherwise one CTA could be dealt all of the shortest sequences (16 sequences of 1 to
// 16K tokens, 8 K/V heads: 41.6 us without).  A segment that lies inside one range is finished there; the at most two
// that a CTA shares with others leave partials for a second kernel.
// Measured on the device, both kernels, bf16 and f16 results (the second with weights in two parts): one sequence of
// 524,288 tokens, 32 heads over 4: 64.4 and 70.7 us for 302 MB, 4.7 and 4.3 of 6.55 TB/s (conversions, mma.sync and copies
// share the issue slots); 16 sequences of 1 to 16K tokens, 8 K/V heads: 19.0 and 20.2 us for 37 MB (rows of 64: 16.1 for
// half the bytes); 4 of 32K, 16 and 32 heads on one: 17.1 and 22.6 us, since more than 16 heads read the pool again;
// one sequence of 8,512 rows, 16 heads on one: 12.8 us, all of it latency (lengths, positions, slots, rows,
// the merge: loads that wait for each other).
#include "block_scan.cuh"
#include "nvtx_range.cuh"
#include "q4_rows.cuh"

namespace lsa {
namespace q4 {

constexpr int WARPS = 4;
constexpr int SETUP = 8;

template <int D_, int NH_>
struct Cfg {
    static constexpr int D = D_, NH = NH_;          // head width; tiles of 8 query heads
    static constexpr int CTAS = NH == 1 ? 3 : 2;    // a multiprocessor: registers
    static constexpr int STAGES = NH == 1 ? 2 : 3;
    static constexpr int CODE = D / 2, SCALES = D / 16;   // bytes of a row
    static constexpr int HALF = 64 * (CODE + SCALES);     // one side of one unit: 36 D
    static constexpr int STAGE = 2 * HALF;
    static constexpr int OBUF = 8 * NH * D * 4;     // one warp's O, fp32
    static constexpr int RING = WARPS * STAGES * STAGE;
    static constexpr int SMEM = RING > WARPS * OBUF ? RING : WARPS * OBUF;
    static constexpr int KS = D / 16;               // k16 steps of S^T, m16 tiles of O^T
    static constexpr int HPC = 8 * NH;              // query heads of a CTA
};

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Bits of a where the mask is set, of b elsewhere.
__device__ __forceinline__ uint32_t select_bits(uint32_t mask, uint32_t a, uint32_t b) { return (a & mask) | (b & ~mask); }

__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(d) : "r"(v));
    return d;
}

// cp.async of N = 4, 8 or 16 bytes; src_bytes = 0 writes zeros and reads nothing.
template <int N>
__device__ __forceinline__ void copy_async(uint32_t dst, const void *src, int src_bytes) {
    if constexpr (N == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src), "r"(src_bytes) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;\n" ::"r"(dst), "l"(src), "n"(N), "r"(src_bytes)
                     : "memory");
}

// V rows of a 16-row block are stored in another order (row 8a + 2t + c at 8a + 4c + t) and, for
// 64-byte rows, with the 16-byte pieces of every second pair of rows exchanged, so that the
// four token lanes of a shared load touch different banks.
__device__ __forceinline__ int v_row(int r) { return (r & ~7) | ((r & 1) << 2) | ((r >> 1) & 3); }
template <int D>
__device__ __forceinline__ int v_piece(int row, int piece) {
    return D == 128 ? piece ^ (((row >> 1) & 1) << 1) : piece;
}

template <class T> __device__ __forceinline__ T ld_shared(uint32_t addr);
template <> __device__ __forceinline__ uint32_t ld_shared<uint32_t>(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
}
template <> __device__ __forceinline__ uint2 ld_shared<uint2>(uint32_t addr) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
    return v;
}
template <> __device__ __forceinline__ uint4 ld_shared<uint4>(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
    return v;
}
__device__ __forceinline__ uint32_t ld_shared_u16(uint32_t addr) {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr));
    return v;
}
__device__ __forceinline__ uint32_t ld_shared_u8(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
}

// Number of units of sequence b (as Units counts them).
__device__ __forceinline__ int count_units(const DecodeParams &p, int b) {
    const int tk = p.k > 0 ? min(max(__ldg(p.topk_count + b), 0), p.k) : 0;
    const int start = __ldg(p.window_start + b);
    const int len = window_rows(p, start, __ldg(p.window_len + b));
    return (tk + LSA_CHUNK - 1) / LSA_CHUNK + (len > 0 ? (start + len - 1) / LSA_CHUNK - start / LSA_CHUNK + 1 : 0);
}

template <class T>
__device__ __forceinline__ void store_out4(void *out, size_t at, const float4 &v) {
    Vec<T, 4> o;
    o.v[0] = from_f32<T>(v.x); o.v[1] = from_f32<T>(v.y); o.v[2] = from_f32<T>(v.z); o.v[3] = from_f32<T>(v.w);
    *reinterpret_cast<Vec<T, 4> *>(static_cast<T *>(out) + at) = o;
}
// Four output values at element `at` (a multiple of 4) of out, in its type.
__device__ __forceinline__ void store_out(const DecodeParams &p, size_t at, const float4 &v) {
    if (p.out_dtype == LSA_DTYPE_BF16) store_out4<__nv_bfloat16>(p.out, at, v);
    else if (p.out_dtype == LSA_DTYPE_F16) store_out4<__half>(p.out, at, v);
    else store_out4<float>(p.out, at, v);
}
__device__ __forceinline__ float lse_of(float M, float L) {
    return L == 0.f ? -INFINITY : (M + log2f(L)) * 0.69314718055994530942f;
}

template <class C, bool TWO>
__global__ void __launch_bounds__(WARPS * 32, C::CTAS) q4_decode_kernel(const DecodeParams p, int B) {
    constexpr int D = C::D, NH = C::NH, NT = WARPS * 32;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int warp_tot[NT / 32 + 1];
    __shared__ int64_t s_sum[WARPS];
    __shared__ int s_first_b;
    __shared__ int64_t s_first_off;
    __shared__ float sm_m[WARPS][C::HPC], sm_l[WARPS][C::HPC];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int G = p.Hq / p.heads, groups = (G + C::HPC - 1) / C::HPC, per_seq = p.heads * groups;

    // ---- this CTA's range [lo, hi) of the units of all segments, and the sequence where it begins
    int64_t total = 0;
    for (int b = threadIdx.x; b < B; b += NT) {
        const int n = count_units(p, b);
        total += n > 0 ? n + SETUP : 0;
        if (blockIdx.x == 0 && p.window_len[b] > window_rows(p, p.window_start[b], p.window_len[b]))
            flag(p.status, p.window_start[b] < 0 ? LSA_DEV_INDEX : LSA_DEV_TABLE);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    if (lane == 0) s_sum[warp] = total;
    __syncthreads();
    total = 0;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) total += s_sum[w];
    total *= per_seq;
    // no more CTAs than give every warp a unit; then no range is empty
    const int64_t ctas = lsa_min64(gridDim.x, (total + WARPS - 1) / WARPS);
    if (blockIdx.x >= ctas) return;
    const int64_t lo = total * blockIdx.x / ctas, hi = total * (blockIdx.x + 1) / ctas;
    int64_t before = 0;          // units of the sequences before b0
    for (int b0 = 0; b0 < B; b0 += NT) {
        const int b = b0 + threadIdx.x;
        int n = b < B ? count_units(p, b) : 0;
        if (n > 0) n += SETUP;
        int tot;
        const int64_t at = (before + block_exclusive_scan<NT>(n, warp_tot, &tot)) * per_seq;
        if (n > 0 && at <= lo && lo < at + (int64_t)n * per_seq) { s_first_b = b; s_first_off = at; }
        before += tot;
        if (before * per_seq > lo) break;      // uniform
    }
    __syncthreads();
    int b = s_first_b;
    int64_t seq_at = s_first_off;              // units before sequence b

    const uint32_t ring = smem_addr(smem) + warp * C::STAGES * C::STAGE;
    const int64_t slot_stride = p.heads * chunk_bytes(D);

    for (int64_t pos = lo; pos < hi;) {
    const Units un(p, b);
    if (un.total == 0) { ++b; continue; }
    const int cost = un.total + SETUP;
    const int seg = (int)((pos - seq_at) / cost);                      // K/V head and group
    const int64_t seg_at = seq_at + (int64_t)seg * cost, seg_end = seg_at + cost;
    const int kvh = seg / groups, h0 = (seg - kvh * groups) * C::HPC;  // first query head of the group
    const int nh = min(C::HPC, G - h0);                                // query heads here
    const size_t qrow0 = (size_t)b * p.Hq + (size_t)kvh * G + h0;
    const int unit0 = max((int)(pos - seg_at) - SETUP, 0), unit1 = (int)(lsa_min64(seg_end, hi) - seg_at) - SETUP;
    const bool next_seq = seg == per_seq - 1;
    pos = lsa_min64(seg_end, hi);
    if (unit1 <= 0) continue;                // the range ends before the segment's first unit
    const uint8_t *kb = p.k_pool + kvh * chunk_bytes(D), *vb = p.v_pool + kvh * chunk_bytes(D);
    const int u_first = unit0 + warp, u_step = WARPS;
    const int n_mine = u_first < unit1 ? (unit1 - 1 - u_first) / u_step + 1 : 0;

    // ---- copies of one unit into a stage; returns this lane's rows (lane, lane + 32) as present
    auto issue = [&](int i) -> uint32_t {
        uint32_t have = 0;
        if (i < n_mine) {
            const int u = u_first + i * u_step;
            const uint32_t ks = ring + (i % C::STAGES) * C::STAGE, vs = ks + C::HALF;
            if (u >= un.t_topk) {
                const int slot = un.window_slot(p, b, u);
                if (slot >= 0) {
                    const uint8_t *kc = kb + slot * slot_stride, *vc = vb + slot * slot_stride;
                    constexpr int PPR = C::CODE / 16, CODES = 64 * PPR;
#pragma unroll
                    for (int n = 0; n < CODES / 32; ++n) {
                        const int q = lane + 32 * n, r = q / PPR, c = q % PPR, vr = v_row(r);
                        copy_async<16>(ks + q * 16, kc + q * 16, 16);
                        copy_async<16>(vs + vr * C::CODE + v_piece<D>(vr, c) * 16, vc + q * 16, 16);
                    }
                    if (D == 128 || lane < 16) {
                        copy_async<16>(ks + 64 * C::CODE + lane * 16, kc + 64 * C::CODE + lane * 16, 16);
                        copy_async<16>(vs + 64 * C::CODE + lane * 16, vc + 64 * C::CODE + lane * 16, 16);
                    }
                    have = (un.in_window(u, lane) ? 1u : 0u) | (un.in_window(u, lane + 32) ? 2u : 0u);
                }
            } else {
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    const int r = lane + 32 * n, vr = v_row(r);
                    const int64_t row = un.topk_row(p, b, u, r);
                    if (row < 0) continue;
                    have |= 1u << n;
                    const int64_t at = (row / LSA_CHUNK) * slot_stride;
                    const int in = (int)(row % LSA_CHUNK);
                    const uint8_t *kr = kb + at + in * C::CODE, *vr_ = vb + at + in * C::CODE;
#pragma unroll
                    for (int c = 0; c < C::CODE / 16; ++c) {
                        copy_async<16>(ks + r * C::CODE + c * 16, kr + c * 16, 16);
                        copy_async<16>(vs + vr * C::CODE + v_piece<D>(vr, c) * 16, vr_ + c * 16, 16);
                    }
                    copy_async<C::SCALES>(ks + 64 * C::CODE + r * C::SCALES, kb + at + 64 * C::CODE + in * C::SCALES, C::SCALES);
                    copy_async<C::SCALES>(vs + 64 * C::CODE + r * C::SCALES, vb + at + 64 * C::CODE + in * C::SCALES, C::SCALES);
                }
            }
        }
        cp_async_commit();
        return have;
    };

    uint32_t have[C::STAGES];
#pragma unroll
    for (int s = 0; s < C::STAGES - 1; ++s) have[s] = issue(s);

    // ---- queries of the group, B operand of S^T: lane (g, t) holds head g's columns D/4 t ..
    uint32_t qf[NH][C::KS][2];
    float smul[NH][2];
#pragma unroll
    for (int n = 0; n < NH; ++n) {
        float x[D / 4];
        const int h = 8 * n + g;
        const bool live = h < nh;
        const uint16_t *src = static_cast<const uint16_t *>(p.q) + (qrow0 + (live ? h : 0)) * D + t * (D / 4);
        float amax = 0.f;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
            const uint4 w = live ? __ldg(reinterpret_cast<const uint4 *>(src) + c) : make_uint4(0, 0, 0, 0);
            const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float lo, hi;
                if (p.q_f16) {
                    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&ww[j]));
                    lo = f.x; hi = f.y;
                } else {
                    lo = __uint_as_float(ww[j] << 16);
                    hi = __uint_as_float(ww[j] & 0xffff0000u);
                }
                x[8 * c + 2 * j] = lo;
                x[8 * c + 2 * j + 1] = hi;
                amax = fmaxf(amax, fmaxf(fabsf(lo), fabsf(hi)));
            }
        }
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        float inv;
        const float e = score_factor(row_exponent(amax, inv), p.scale_log2);
        smul[n][0] = __shfl_sync(0xffffffffu, e, 8 * t);        // head 2t: lane (2t, 0)
        smul[n][1] = __shfl_sync(0xffffffffu, e, 8 * t + 4);
#pragma unroll
        for (int j = 0; j < C::KS; ++j) {
            qf[n][j][0] = pack_f16x2(x[4 * j] * inv, x[4 * j + 1] * inv);
            qf[n][j][1] = pack_f16x2(x[4 * j + 2] * inv, x[4 * j + 3] * inv);
        }
    }

    float o[C::KS][NH][4];
    float m_ref[NH][2], l[NH][2];
#pragma unroll
    for (int i = 0; i < C::KS; ++i)
#pragma unroll
        for (int n = 0; n < NH; ++n) o[i][n][0] = o[i][n][1] = o[i][n][2] = o[i][n][3] = 0.f;
#pragma unroll
    for (int n = 0; n < NH; ++n) m_ref[n][0] = m_ref[n][1] = -INFINITY, l[n][0] = l[n][1] = 0.f;

    for (int i = 0; i < n_mine; ++i) {
        const uint32_t have_new = issue(i + C::STAGES - 1);
        cp_async_wait<C::STAGES - 1>();
        __syncwarp();
        uint32_t h_now = have[0];
#pragma unroll
        for (int s = 0; s < C::STAGES - 2; ++s) have[s] = have[s + 1];
        have[C::STAGES - 2] = have_new;
        const uint32_t lo = __ballot_sync(0xffffffffu, h_now & 1u), hi = __ballot_sync(0xffffffffu, h_now & 2u);
        if ((lo | hi) == 0u) {
            __syncwarp();
            continue;
        }
        const uint32_t ks = ring + (i % C::STAGES) * C::STAGE, vs = ks + C::HALF;
        const bool full = (lo & hi) == 0xffffffffu;
        if (!full) {
            // rows outside the set may hold anything, NaN scales too: their V scales become 0 (and their scores,
            // below, -inf)
#pragma unroll
            for (int n = 0; n < 2; ++n)
                if (!((n ? hi : lo) >> lane & 1u)) {
                    const uint32_t at = vs + 64 * C::CODE + (lane + 32 * n) * C::SCALES;
                    asm volatile("st.shared.u32 [%0], %1;" ::"r"(at), "r"(0) : "memory");
                    if constexpr (D == 128) asm volatile("st.shared.u32 [%0], %1;" ::"r"(at + 4), "r"(0) : "memory");
                }
            __syncwarp();
        }

        // ---- S^T = K Q^T: four tiles of 16 rows
        float s[4][NH][4];
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) {
#pragma unroll
            for (int n = 0; n < NH; ++n) s[mt][n][0] = s[mt][n][1] = s[mt][n][2] = s[mt][n][3] = 0.f;
            const int r0 = 16 * mt + g, r1 = r0 + 8;
            uint32_t c0[D / 32], c1[D / 32], f0, f1;   // codes and scales (f16 pairs) of rows r0, r1
            if constexpr (D == 128) {
                const uint4 w0 = ld_shared<uint4>(ks + r0 * 64 + t * 16), w1 = ld_shared<uint4>(ks + r1 * 64 + t * 16);
                c0[0] = w0.x; c0[1] = w0.y; c0[2] = w0.z; c0[3] = w0.w;
                c1[0] = w1.x; c1[1] = w1.y; c1[2] = w1.z; c1[3] = w1.w;
                f0 = e4m3x2_to_f16(ld_shared_u16(ks + 64 * C::CODE + r0 * 8 + 2 * t));
                f1 = e4m3x2_to_f16(ld_shared_u16(ks + 64 * C::CODE + r1 * 8 + 2 * t));
            } else {
                const uint2 w0 = ld_shared<uint2>(ks + r0 * 32 + t * 8), w1 = ld_shared<uint2>(ks + r1 * 32 + t * 8);
                c0[0] = w0.x; c0[1] = w0.y;
                c1[0] = w1.x; c1[1] = w1.y;
                f0 = e4m3x2_to_f16(ld_shared_u8(ks + 64 * C::CODE + r0 * 4 + t));
                f1 = e4m3x2_to_f16(ld_shared_u8(ks + 64 * C::CODE + r1 * 4 + t));
            }
#pragma unroll
            for (int w = 0; w < D / 32; ++w) {     // 8 columns of each row: two k16 steps
                uint32_t a0[4], a1[4];
                e2m1x8_to_f16(c0[w], a0);
                e2m1x8_to_f16(c1[w], a1);
                const uint32_t s0 = w < D / 64 || D == 64 ? dup_lo(f0) : dup_hi(f0);
                const uint32_t s1 = w < D / 64 || D == 64 ? dup_lo(f1) : dup_hi(f1);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    a0[q] = hmul2(a0[q], s0);
                    a1[q] = hmul2(a1[q], s1);
                }
#pragma unroll
                for (int q = 0; q < 2; ++q)
#pragma unroll
                    for (int n = 0; n < NH; ++n)
                        mma_f16(s[mt][n], a0[2 * q], a1[2 * q], a0[2 * q + 1], a1[2 * q + 1], qf[n][2 * w + q][0],
                                qf[n][2 * w + q][1]);
            }
        }

        // ---- softmax over the unit's rows; a head's column lives in the 8 lanes of equal t
        uint32_t pt[4][NH][2], pl[4][NH][TWO ? 2 : 1];
#pragma unroll
        for (int n = 0; n < NH; ++n) {
            if (!full) {
#pragma unroll
                for (int mt = 0; mt < 4; ++mt) {
                    const uint32_t half = mt < 2 ? lo : hi;
                    if (!((half >> (16 * (mt & 1) + g)) & 1u)) s[mt][n][0] = s[mt][n][1] = -INFINITY;
                    if (!((half >> (16 * (mt & 1) + g + 8)) & 1u)) s[mt][n][2] = s[mt][n][3] = -INFINITY;
                }
            }
            // the factor is positive: the maximum of the raw products is the scores', and the reference is kept
            // as a raw product (see score_factor)
            float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) {
                mx0 = fmaxf(mx0, fmaxf(s[mt][n][0], s[mt][n][2]));
                mx1 = fmaxf(mx1, fmaxf(s[mt][n][1], s[mt][n][3]));
            }
#pragma unroll
            for (int q = 4; q < 32; q *= 2) {
                mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, q));
                mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, q));
            }
            const bool move0 = (mx0 - m_ref[n][0]) * smul[n][0] > RESCALE, move1 = (mx1 - m_ref[n][1]) * smul[n][1] > RESCALE;
            if (__any_sync(0xffffffffu, move0 || move1)) {
                const float a0 = move0 ? ex2((m_ref[n][0] - mx0) * smul[n][0]) : 1.f;
                const float a1 = move1 ? ex2((m_ref[n][1] - mx1) * smul[n][1]) : 1.f;
                if (move0) m_ref[n][0] = mx0;
                if (move1) m_ref[n][1] = mx1;
                l[n][0] *= a0;
                l[n][1] *= a1;
#pragma unroll
                for (int j = 0; j < C::KS; ++j) {
                    o[j][n][0] *= a0; o[j][n][1] *= a1;
                    o[j][n][2] *= a0; o[j][n][3] *= a1;
                }
            }
            const float r0 = m_ref[n][0] == -INFINITY ? 0.f : m_ref[n][0];
            const float r1 = m_ref[n][1] == -INFINITY ? 0.f : m_ref[n][1];
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) {
                const float p0 = ex2(fmaf(s[mt][n][0] - r0, smul[n][0], P_SHIFT)), p1 = ex2(fmaf(s[mt][n][1] - r1, smul[n][1], P_SHIFT));
                const float p2 = ex2(fmaf(s[mt][n][2] - r0, smul[n][0], P_SHIFT)), p3 = ex2(fmaf(s[mt][n][3] - r1, smul[n][1], P_SHIFT));
                l[n][0] += p0 + p2;
                l[n][1] += p1 + p3;
                const uint32_t h0 = pack_f16x2(p0, p1), h1 = pack_f16x2(p2, p3);
                pt[mt][n][0] = transpose8x8(h0);
                pt[mt][n][1] = transpose8x8(h1);
                if constexpr (TWO) {
                    pl[mt][n][0] = transpose8x8(rest_f16x2(p0, p1, h0));
                    pl[mt][n][1] = transpose8x8(rest_f16x2(p2, p3, h1));
                }
            }
        }

        // ---- O^T += V^T P^T: four blocks of 16 rows as the contraction
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) {
            // the lane's four rows: 2t, 2t + 1, 2t + 8, 2t + 9 of the block
            uint32_t code[4][D / 64], byte[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int in = 2 * t + (q & 1) + 8 * (q >> 1), r = 16 * mt + in, vr = v_row(r);
                if constexpr (D == 128) {
                    const uint2 w = ld_shared<uint2>(vs + vr * 64 + v_piece<D>(vr, g >> 1) * 16 + (g & 1) * 8);
                    code[q][0] = w.x;
                    code[q][1] = w.y;
                } else {
                    code[q][0] = ld_shared<uint32_t>(vs + vr * 32 + g * 4);
                }
                byte[q] = ld_shared_u8(vs + 64 * C::CODE + r * C::SCALES + (D == 128 ? g : g >> 1));
            }
            const uint32_t s01 = e4m3x2_to_f16(byte[0] | byte[1] << 8), s23 = e4m3x2_to_f16(byte[2] | byte[3] << 8);
#pragma unroll
            for (int w = 0; w < D / 64; ++w) {
                // even and odd columns of the word, two rows a byte
                uint32_t e01[4], o01[4], e23[4], o23[4];
                e2m1x8_to_f16(select_bits(0x0f0f0f0fu, code[0][w], code[1][w] << 4), e01);
                e2m1x8_to_f16(select_bits(0x0f0f0f0fu, code[0][w] >> 4, code[1][w]), o01);
                e2m1x8_to_f16(select_bits(0x0f0f0f0fu, code[2][w], code[3][w] << 4), e23);
                e2m1x8_to_f16(select_bits(0x0f0f0f0fu, code[2][w] >> 4, code[3][w]), o23);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    // columns 2 (4w + j) and + 1 of the lane group's D / 8
                    const uint32_t a0 = hmul2(e01[j], s01), a1 = hmul2(o01[j], s01);
                    const uint32_t a2 = hmul2(e23[j], s23), a3 = hmul2(o23[j], s23);
#pragma unroll
                    for (int n = 0; n < NH; ++n) {
                        mma_f16(o[4 * w + j][n], a0, a1, a2, a3, pt[mt][n][0], pt[mt][n][1]);
                        if constexpr (TWO) mma_f16(o[4 * w + j][n], a0, a1, a2, a3, pl[mt][n][0], pl[mt][n][1]);
                    }
                }
            }
        }
        __syncwarp();      // the stage may be refilled
    }
    cp_async_wait<0>();

    // ---- the CTA's warps: M and sum per head, then O through shared memory
    __syncthreads();       // every warp is done with its ring
#pragma unroll
    for (int n = 0; n < NH; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            float x = l[n][c];
#pragma unroll
            for (int q = 4; q < 32; q *= 2) x += __shfl_xor_sync(0xffffffffu, x, q);
            if (g == 0) {
                sm_m[warp][8 * n + 2 * t + c] = fmaf(m_ref[n][c], smul[n][c], -P_SHIFT);
                sm_l[warp][8 * n + 2 * t + c] = x;
            }
        }
    float *obuf = reinterpret_cast<float *>(smem) + warp * C::HPC * D;
#pragma unroll
    for (int j = 0; j < C::KS; ++j)
#pragma unroll
        for (int n = 0; n < NH; ++n) {
            const int col = g * (D / 8) + 2 * j, h = 8 * n + 2 * t;
            *reinterpret_cast<float2 *>(obuf + h * D + col) = make_float2(o[j][n][0], o[j][n][2]);
            *reinterpret_cast<float2 *>(obuf + (h + 1) * D + col) = make_float2(o[j][n][1], o[j][n][3]);
        }
    __syncthreads();
    const bool whole = unit0 == 0 && unit1 == un.total;
    // partials: slot 2c + 1 of CTA c for the segment that begins in its range, slot 2c for one begun before
    const size_t part0 = (2 * (size_t)blockIdx.x + (unit0 == 0 ? 1 : 0)) * C::HPC;
    for (int i = threadIdx.x; i < nh * (D / 4); i += NT) {
        const int h = i / (D / 4), c = i % (D / 4);
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) M = fmaxf(M, sm_m[w][h]);
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
        float L = 0.f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
            const float f = sm_m[w][h] == -INFINITY ? 0.f : exp2f(sm_m[w][h] - M);
            const float4 v = reinterpret_cast<const float4 *>(smem)[(w * C::HPC + h) * (D / 4) + c];
            L += f * sm_l[w][h];
            a.x += f * v.x; a.y += f * v.y; a.z += f * v.z; a.w += f * v.w;
        }
        if (whole) {
            const float inv = L == 0.f ? 0.f : p.v_scale / L;
            store_out(p, (qrow0 + h) * D + 4 * c, make_float4(a.x * inv, a.y * inv, a.z * inv, a.w * inv));
            if (p.lse && c == 0) p.lse[qrow0 + h] = lse_of(M, L);
        } else {
            reinterpret_cast<float4 *>(p.o_part + (part0 + h) * D)[c] = a;
            if (c == 0) {
                p.m_part[part0 + h] = M;
                p.l_part[part0 + h] = L;
            }
        }
    }
    // the CTA where a segment begins notes which CTAs hold its parts
    if (unit0 == 0 && threadIdx.x == 0) {
        // the last CTA whose range begins before the segment's end
        const int64_t end = seg_end;
        int last = (int)(((end - 1) * ctas) / total);
        while (total * (last + 1) / ctas < end) ++last;
        while (last > 0 && total * last / ctas >= end) --last;
        p.seg_range[(size_t)b * per_seq + seg] = make_int2(blockIdx.x, last);
    }
    __syncthreads();       // O in shared memory is read before the next segment's copies
    if (pos == seg_end && next_seq) { seq_at = seg_end; ++b; }
    }
}

// One CTA per (sequence, query head) merges the parts of a segment that several CTAs share: the
// weights of up to MERGE parts at a time, then D / 4 columns x ROWS parts in flight.  It also answers for
// sequences without rows (o = 0, lse = -inf).  Nothing but latency: the range is read beside the lengths, and a
// thread's first FLIGHT parts beside the maxima.
constexpr int MERGE = 256;
template <int D, int HPC>
__global__ void __launch_bounds__(MERGE) q4_merge_split_kernel(const DecodeParams p) {
    constexpr int COLS = D / 4, ROWS = MERGE / COLS, FLIGHT = 16;
    __shared__ float4 red[ROWS][COLS];
    __shared__ float wmax[MERGE / 32], wsum[MERGE / 32], w_of[MERGE];
    const int b = blockIdx.y, head = blockIdx.x, G = p.Hq / p.heads, groups = (G + HPC - 1) / HPC;
    const int kvh = head / G, gh = head - kvh * G, grp = gh / HPC, h = gh - grp * HPC;
    const size_t row = (size_t)b * p.Hq + head;
    const int col = threadIdx.x % COLS, r = threadIdx.x / COLS;
    const int2 range = p.seg_range[((size_t)b * p.heads + kvh) * groups + grp];     // anything if there are no units
    if (count_units(p, b) == 0) {
        if (r == 0) store_out(p, row * D + 4 * col, make_float4(0.f, 0.f, 0.f, 0.f));
        if (p.lse && threadIdx.x == 0) p.lse[row] = -INFINITY;
        return;
    }
    if (range.x == range.y) return;            // finished by its CTA
    const int n = range.y - range.x + 1;
    auto part = [&](int i) { return (2 * (size_t)(range.x + i) + (i == 0 ? 1 : 0)) * HPC + h; };
    float4 v[FLIGHT];
#pragma unroll
    for (int j = 0; j < FLIGHT; ++j)
        if (r + j * ROWS < n) v[j] = __ldcs(reinterpret_cast<const float4 *>(p.o_part + part(r + j * ROWS) * D) + col);
    float m0 = -INFINITY, l0 = 0.f;            // of this thread's first part
    if (threadIdx.x < n) {
        m0 = p.m_part[part(threadIdx.x)];
        l0 = p.l_part[part(threadIdx.x)];
    }
    float M = m0;
    for (int i = threadIdx.x + MERGE; i < n; i += MERGE) M = fmaxf(M, p.m_part[part(i)]);
    M = warp_max(M);
    if ((threadIdx.x & 31) == 0) wmax[threadIdx.x >> 5] = M;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < MERGE / 32; ++w) M = fmaxf(M, wmax[w]);
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    float L = 0.f;
    for (int i0 = 0; i0 < n; i0 += MERGE) {
        const int i = i0 + threadIdx.x;
        float f = 0.f;
        if (i < n) {
            const float m = i0 == 0 ? m0 : p.m_part[part(i)], l = i0 == 0 ? l0 : p.l_part[part(i)];
            f = m == -INFINITY ? 0.f : exp2f(m - M);
            L += f * l;
        }
        w_of[threadIdx.x] = f;
        __syncthreads();
        const int here = min(MERGE, n - i0);
        for (int j0 = r; j0 < here; j0 += FLIGHT * ROWS) {
            if (i0 + j0 != r) {
#pragma unroll
                for (int j = 0; j < FLIGHT; ++j)
                    if (j0 + j * ROWS < here)
                        v[j] = __ldcs(reinterpret_cast<const float4 *>(p.o_part + part(i0 + j0 + j * ROWS) * D) + col);
            }
#pragma unroll
            for (int j = 0; j < FLIGHT; ++j)
                if (j0 + j * ROWS < here) {
                    const float wgt = w_of[j0 + j * ROWS];
                    a.x += wgt * v[j].x; a.y += wgt * v[j].y; a.z += wgt * v[j].z; a.w += wgt * v[j].w;
                }
        }
        __syncthreads();
    }
    L = warp_sum(L);
    if ((threadIdx.x & 31) == 0) wsum[threadIdx.x >> 5] = L;
    red[r][col] = a;
    __syncthreads();
    L = 0.f;
#pragma unroll
    for (int w = 0; w < MERGE / 32; ++w) L += wsum[w];
    if (r == 0) {
#pragma unroll
        for (int j = 1; j < ROWS; ++j) {
            const float4 v = red[j][col];
            a.x += v.x; a.y += v.y; a.z += v.z; a.w += v.w;
        }
        const float inv = L == 0.f ? 0.f : p.v_scale / L;
        store_out(p, row * D + 4 * col, make_float4(a.x * inv, a.y * inv, a.z * inv, a.w * inv));
        if (p.lse && col == 0) p.lse[row] = lse_of(M, L);
    }
}

// Latent rows: one CTA of dv / 4 threads per (sequence, head).  The loads of a group of splits are issued
// before any arithmetic.
__global__ void __launch_bounds__(128) q4_merge_kernel(const DecodeParams p, int dv) {
    constexpr int GROUP = 10;
    const int h = blockIdx.x, b = blockIdx.y, c = threadIdx.x;
    const size_t row0 = (size_t)b * p.n_splits * p.Hq + h;
    float M = -INFINITY, L = 0.f;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s0 = 0; s0 < p.n_splits; s0 += GROUP) {
        float4 v[GROUP];
        float m[GROUP], l[GROUP];
#pragma unroll
        for (int j = 0; j < GROUP; ++j) {
            m[j] = -INFINITY;
            l[j] = 0.f;
            v[j] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (s0 + j < p.n_splits) {
                const size_t r = row0 + (size_t)(s0 + j) * p.Hq;
                v[j] = __ldcs(reinterpret_cast<const float4 *>(p.o_part + r * dv) + c);
                m[j] = __ldg(p.m_part + r);
                l[j] = __ldg(p.l_part + r);
            }
        }
        float Mn = M;
#pragma unroll
        for (int j = 0; j < GROUP; ++j) Mn = fmaxf(Mn, m[j]);
        const float r = M == -INFINITY ? 0.f : exp2f(M - Mn);
        L *= r;
        a.x *= r; a.y *= r; a.z *= r; a.w *= r;
#pragma unroll
        for (int j = 0; j < GROUP; ++j) {
            const float f = m[j] == -INFINITY ? 0.f : exp2f(m[j] - Mn);
            L += f * l[j];
            a.x += f * v[j].x; a.y += f * v[j].y; a.z += f * v[j].z; a.w += f * v[j].w;
        }
        M = Mn;
    }
    // no rows at all: o = 0, lse = -inf.  A NaN sum (a NaN row in the set) stays NaN.
    const float inv = L == 0.f ? 0.f : p.v_scale / L;
    store_out(p, ((size_t)b * p.Hq + h) * dv + 4 * c, make_float4(a.x * inv, a.y * inv, a.z * inv, a.w * inv));
    if (p.lse && c == 0) p.lse[(size_t)b * p.Hq + h] = lse_of(M, L);
}

static int max_units(int k, int max_window_len) { return (k + 63) / 64 + (max_window_len + 63) / 64 + 1; }

// CTAs of the separate K/V kernel: one wave (3 or 2 a multiprocessor), fewer where there would be less than a
// unit for each warp even if every sequence had its longest row set.
static int separate_ctas(int B, int heads, int G, int units) {
    const int hpc = G <= 8 ? 8 : 16, groups = (G + hpc - 1) / hpc;
    const int64_t most = ((int64_t)B * heads * groups * (units + SETUP) + WARPS - 1) / WARPS;
    return (int)lsa_max64(1, lsa_min64(sm_count() * (G <= 8 ? 3 : 2), most));
}

template <class C, bool TWO>
static int launch_separate(const DecodeParams &p, int B, cudaStream_t stream) {
    static std::atomic<uint64_t> done{0};
    if (int rc = allow_shared(q4_decode_kernel<C, TWO>, C::SMEM, done)) return rc;
    q4_decode_kernel<C, TWO><<<p.n_splits, WARPS * 32, C::SMEM, stream>>>(p, B);
    if (int rc = check_launch("q4_decode_kernel")) return rc;
    q4_merge_split_kernel<C::D, C::HPC><<<dim3(p.Hq, B), MERGE, 0, stream>>>(p);
    return check_launch("q4_merge_split_kernel");
}

static bool supported(int Hq, int heads, int dqk, int dv, bool latent) {
    if (Hq < 1 || heads < 1 || Hq % heads) return false;
    if (latent) return heads == 1 && dqk == 576 && dv == 512 && Hq <= 128;
    return dqk == dv && (dqk == 64 || dqk == 128) && Hq <= 1024;
}

static int splits_for(int B, int Hq, int heads, bool latent, int k, int max_window_len) {
    const int units = max_units(k, max_window_len);
    return latent ? q4mla::splits(B, units) : separate_ctas(B, heads, Hq / heads, units);
}

// Carves the workspace: partials of every split (latent), or two a CTA and the segments' ranges.
static size_t carve(Carver &c, DecodeParams &p, int B, int dv, bool latent) {
    const int G = p.Hq / p.heads, hpc = G <= 8 ? 8 : 16;
    const size_t rows = latent ? (size_t)B * p.n_splits * p.Hq : (size_t)p.n_splits * 2 * hpc;
    p.o_part = c.take<float>(rows * dv);
    p.m_part = c.take<float>(rows);
    p.l_part = c.take<float>(rows);
    p.seg_range = c.take<int2>(latent ? 0 : (size_t)B * p.heads * ((G + hpc - 1) / hpc));
    return align_up(c.used, 256);
}

}  // namespace q4
}  // namespace lsa

using namespace lsa;

extern "C" size_t lsa_sparse_decode_q4_workspace_size(int B, int Hq, int heads, int dqk, int dv, int k,
                                                      int max_window_len) {
    const bool latent = dqk != dv;
    if (!q4::supported(Hq, heads, dqk, dv, latent) || B < 1 || B > 65535 || k < 0 || max_window_len < 0) return 0;
    q4::DecodeParams p = {};
    p.Hq = Hq; p.heads = heads;
    p.n_splits = q4::splits_for(B, Hq, heads, latent, k, max_window_len);
    Carver c(nullptr);
    return q4::carve(c, p, B, dv, latent);
}

extern "C" int lsa_sparse_decode_q4(int q_dtype, const void *q, const uint8_t *k_pool, float k_scale,
                                    const uint8_t *v_pool, float v_scale, int64_t n_slots, int heads,
                                    const int32_t *chunk_table, int table_stride, const int32_t *topk_idx,
                                    const int32_t *topk_count, int k, const int32_t *window_start,
                                    const int32_t *window_len, int max_window_len, int B, int Hq, int dqk, int dv,
                                    float scale, int out_dtype, void *out, float *lse, int32_t *dev_status, void *ws,
                                    size_t ws_bytes, lsa_stream_t stream) {
    LSA_ABI_RANGE();
    LSA_REQUIRE(B > 0 && B <= 65535 && n_slots > 0 && n_slots < (1ll << 31) && table_stride > 0 && k >= 0 &&
                    k <= (1 << 30) && max_window_len >= 0 && max_window_len <= (1 << 30),
                LSA_ERR_INVALID_ARG, "lsa_sparse_decode_q4: bad sizes (B=%d n_slots=%lld table_stride=%d k=%d max_window_len=%d)",
                B, (long long)n_slots, table_stride, k, max_window_len);
    LSA_REQUIRE(q_dtype == LSA_DTYPE_BF16 || q_dtype == LSA_DTYPE_F16, LSA_ERR_INVALID_ARG,
                "lsa_sparse_decode_q4: q must be bf16 or f16 (dtype %d)", q_dtype);
    LSA_REQUIRE(dtype_known(out_dtype), LSA_ERR_INVALID_ARG, "lsa_sparse_decode_q4: unknown output dtype %d", out_dtype);
    LSA_REQUIRE(q && k_pool && chunk_table && window_start && window_len && out && (k == 0 || (topk_idx && topk_count)),
                LSA_ERR_INVALID_ARG, "lsa_sparse_decode_q4: null pointer");
    const bool latent = v_pool == nullptr;
    LSA_REQUIRE(q4::supported(Hq, heads, dqk, dv, latent) && latent == (dqk != dv), LSA_ERR_SHAPE,
                "lsa_sparse_decode_q4: unsupported (Hq=%d, heads=%d, dqk=%d, dv=%d, %s); supported: Hq a multiple of "
                "heads with (64,64) or (128,128) separate K/V, and up to 128 query heads over one (576,512) latent row",
                Hq, heads, dqk, dv, latent ? "latent" : "separate K/V");
    auto al = [](const void *x) { return (reinterpret_cast<uintptr_t>(x) & 15) == 0; };
    LSA_REQUIRE(al(q) && al(k_pool) && al(v_pool) && al(out), LSA_ERR_INVALID_ARG,
                "lsa_sparse_decode_q4: q, pools and out must be 16-byte aligned");
    LSA_REQUIRE(scale > 0.f && scale <= 1e30f && k_scale > 0.f && k_scale <= 1e30f && v_scale > 0.f && v_scale <= 1e30f,
                LSA_ERR_INVALID_ARG, "lsa_sparse_decode_q4: scales must be positive and at most 1e30");
    q4::DecodeParams p = {};
    p.Hq = Hq; p.heads = heads;
    p.n_splits = q4::splits_for(B, Hq, heads, latent, k, max_window_len);
    Carver c(ws);
    const size_t need = q4::carve(c, p, B, dv, latent);
    LSA_REQUIRE(ws && ws_bytes >= need, LSA_ERR_WORKSPACE, "lsa_sparse_decode_q4: workspace of %zu bytes, %zu needed",
                ws_bytes, need);
    LSA_REQUIRE(al(ws), LSA_ERR_WORKSPACE, "lsa_sparse_decode_q4: workspace not 16-byte aligned");
    p.q = q; p.k_pool = k_pool; p.v_pool = v_pool; p.table = chunk_table; p.topk_idx = topk_idx;
    p.topk_count = topk_count; p.window_start = window_start; p.window_len = window_len; p.status = dev_status;
    p.n_slots = n_slots; p.table_stride = table_stride; p.k = k;
    p.scale_log2 = scale * k_scale * 1.4426950408889634f;
    p.v_scale = latent ? k_scale : v_scale;
    p.q_f16 = q_dtype == LSA_DTYPE_F16;
    p.out = out; p.lse = lse; p.out_dtype = out_dtype;
    const int G = Hq / heads;
    if (latent) {
        if (int rc = q4mla::launch(p, B, stream)) return rc;
        q4::q4_merge_kernel<<<dim3(Hq, B), dv / 4, 0, stream>>>(p, dv);
        return check_launch("q4_merge_kernel");
    }
    const bool two = q4::two_parts(out_dtype);
#define LSA_SEPARATE(D, NH) (two ? q4::launch_separate<q4::Cfg<D, NH>, true>(p, B, stream) : q4::launch_separate<q4::Cfg<D, NH>, false>(p, B, stream))
    if (dqk == 128) return G <= 8 ? LSA_SEPARATE(128, 1) : LSA_SEPARATE(128, 2);
    return G <= 8 ? LSA_SEPARATE(64, 1) : LSA_SEPARATE(64, 2);
#undef LSA_SEPARATE
}
