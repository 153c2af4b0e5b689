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
//    O^T lane group g takes value columns D/8 g .. , contiguous again, and the tokens pair up by
//    byte permutes of two tokens' f16 pairs.
//  - P^T goes from the accumulator layout to the operand layout with movmatrix, no memory.
// A CTA's warps merge through shared memory; CTAs of one (sequence, K/V head) split its units
// and their partials are merged by a second kernel.
#include "nvtx_range.cuh"
#include "q4_rows.cuh"

namespace lsa {
namespace q4 {

constexpr int WARPS = 4;

template <int D_, int NH_>
struct Cfg {
    static constexpr int D = D_, NH = NH_;          // head width; tiles of 8 query heads
    static constexpr int STAGES = 3;
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

template <class C>
__global__ void __launch_bounds__(WARPS * 32, C::NH == 1 ? 3 : 2) q4_decode_kernel(const DecodeParams p) {
    constexpr int D = C::D, NH = C::NH;
    extern __shared__ __align__(128) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int b = blockIdx.z, split = blockIdx.x;
    const int G = p.Hq / p.heads, groups = (G + C::HPC - 1) / C::HPC;
    const int kvh = blockIdx.y / groups, h0 = (blockIdx.y - kvh * groups) * C::HPC;   // first query head of the group
    const int nh = min(C::HPC, G - h0);                                               // query heads here
    const size_t qrow0 = (size_t)b * p.Hq + (size_t)kvh * G + h0;
    const Units un(p, b);

    const uint32_t ring = smem_addr(smem) + warp * C::STAGES * C::STAGE;
    const int64_t slot_stride = p.heads * chunk_bytes(D);
    const uint8_t *kb = p.k_pool + kvh * chunk_bytes(D), *vb = p.v_pool + kvh * chunk_bytes(D);
    const int u_first = split * WARPS + warp, u_step = p.n_splits * WARPS;
    const int n_mine = u_first < un.total ? (un.total - 1 - u_first) / u_step + 1 : 0;

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
        const float e = row_exponent(amax, inv) * p.scale_log2;
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
        uint32_t pt[4][NH][2];
#pragma unroll
        for (int n = 0; n < NH; ++n) {
            float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) {
                const uint32_t half = mt < 2 ? lo : hi;
                const bool v0 = (half >> (16 * (mt & 1) + g)) & 1u, v1 = (half >> (16 * (mt & 1) + g + 8)) & 1u;
                s[mt][n][0] = v0 ? s[mt][n][0] * smul[n][0] : -INFINITY;
                s[mt][n][1] = v0 ? s[mt][n][1] * smul[n][1] : -INFINITY;
                s[mt][n][2] = v1 ? s[mt][n][2] * smul[n][0] : -INFINITY;
                s[mt][n][3] = v1 ? s[mt][n][3] * smul[n][1] : -INFINITY;
                mx0 = fmaxf(mx0, fmaxf(s[mt][n][0], s[mt][n][2]));
                mx1 = fmaxf(mx1, fmaxf(s[mt][n][1], s[mt][n][3]));
            }
#pragma unroll
            for (int q = 4; q < 32; q *= 2) {
                mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, q));
                mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, q));
            }
            const bool move0 = mx0 > m_ref[n][0] + RESCALE, move1 = mx1 > m_ref[n][1] + RESCALE;
            if (__any_sync(0xffffffffu, move0 || move1)) {
                const float a0 = move0 ? exp2f(m_ref[n][0] - mx0) : 1.f, a1 = move1 ? exp2f(m_ref[n][1] - mx1) : 1.f;
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
            const float r0 = m_ref[n][0] == -INFINITY ? 0.f : m_ref[n][0] - P_SHIFT;
            const float r1 = m_ref[n][1] == -INFINITY ? 0.f : m_ref[n][1] - P_SHIFT;
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) {
                const float p0 = exp2f(s[mt][n][0] - r0), p1 = exp2f(s[mt][n][1] - r1);
                const float p2 = exp2f(s[mt][n][2] - r0), p3 = exp2f(s[mt][n][3] - r1);
                l[n][0] += p0 + p2;
                l[n][1] += p1 + p3;
                pt[mt][n][0] = transpose8x8(pack_f16x2(p0, p1));
                pt[mt][n][1] = transpose8x8(pack_f16x2(p2, p3));
            }
        }

        // ---- O^T += V^T P^T: four blocks of 16 rows as the contraction
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) {
            const uint32_t half = mt < 2 ? lo : hi;
            // the lane's four rows: 2t, 2t + 1, 2t + 8, 2t + 9 of the block
            uint32_t code[4][D / 64], sc[4];
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
                // a row outside the set may hold anything, a NaN scale too: its scale becomes 0
                const uint32_t sb = ld_shared_u8(vs + 64 * C::CODE + r * C::SCALES + (D == 128 ? g : g >> 1));
                const bool there = (half >> (16 * (mt & 1) + in)) & 1u;
                sc[q] = dup_lo(e4m3x2_to_f16(there ? sb : 0u));
            }
#pragma unroll
            for (int w = 0; w < D / 64; ++w) {
                uint32_t v[4][4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    e2m1x8_to_f16(code[q][w], v[q]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) v[q][j] = hmul2(v[q][j], sc[q]);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    // columns 2 (4w + j) and + 1 of the lane group's D / 8, tokens paired
                    const uint32_t a0 = __byte_perm(v[0][j], v[1][j], 0x5410), a1 = __byte_perm(v[0][j], v[1][j], 0x7632);
                    const uint32_t a2 = __byte_perm(v[2][j], v[3][j], 0x5410), a3 = __byte_perm(v[2][j], v[3][j], 0x7632);
#pragma unroll
                    for (int n = 0; n < NH; ++n) mma_f16(o[4 * w + j][n], a0, a1, a2, a3, pt[mt][n][0], pt[mt][n][1]);
                }
            }
        }
        __syncwarp();      // the stage may be refilled
    }
    cp_async_wait<0>();

    // ---- the CTA's warps: M and sum per head, then O through shared memory
    __shared__ float sm_m[WARPS][C::HPC], sm_l[WARPS][C::HPC];
    __syncthreads();       // every warp is done with its ring
#pragma unroll
    for (int n = 0; n < NH; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            float x = l[n][c];
#pragma unroll
            for (int q = 4; q < 32; q *= 2) x += __shfl_xor_sync(0xffffffffu, x, q);
            if (g == 0) {
                sm_m[warp][8 * n + 2 * t + c] = m_ref[n][c] - P_SHIFT;
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
    const size_t part0 = ((size_t)b * p.n_splits + split) * p.Hq + (size_t)kvh * G + h0;
    for (int i = threadIdx.x; i < nh * (D / 4); i += WARPS * 32) {
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
        reinterpret_cast<float4 *>(p.o_part + (part0 + h) * D)[c] = a;
        if (c == 0) {
            p.m_part[part0 + h] = M;
            p.l_part[part0 + h] = L;
        }
    }
}

// One CTA of dv / 4 threads per (sequence, head): the weight of each split, then its columns.
template <class T>
__global__ void __launch_bounds__(128) q4_merge_kernel(const DecodeParams p, int dv, T *__restrict__ out,
                                                       float *__restrict__ lse) {
    const int h = blockIdx.x, b = blockIdx.y, c = threadIdx.x;
    const size_t row0 = (size_t)b * p.n_splits * p.Hq + h;
    float M = -INFINITY;
    for (int s = 0; s < p.n_splits; ++s) M = fmaxf(M, p.m_part[row0 + (size_t)s * p.Hq]);
    float L = 0.f;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int s = 0; s < p.n_splits; ++s) {
        const size_t r = row0 + (size_t)s * p.Hq;
        const float m = p.m_part[r], f = m == -INFINITY ? 0.f : exp2f(m - M);
        const float4 v = __ldcs(reinterpret_cast<const float4 *>(p.o_part + r * dv) + c);
        L += f * p.l_part[r];
        a.x += f * v.x; a.y += f * v.y; a.z += f * v.z; a.w += f * v.w;
    }
    // no rows at all: o = 0, lse = -inf.  A NaN sum (a NaN row in the set) stays NaN.
    const float inv = L == 0.f ? 0.f : p.v_scale / L;
    Vec<T, 4> o;
    o.v[0] = from_f32<T>(a.x * inv); o.v[1] = from_f32<T>(a.y * inv);
    o.v[2] = from_f32<T>(a.z * inv); o.v[3] = from_f32<T>(a.w * inv);
    *reinterpret_cast<Vec<T, 4> *>(out + ((size_t)b * p.Hq + h) * dv + 4 * c) = o;
    if (lse && c == 0) lse[(size_t)b * p.Hq + h] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.69314718055994530942f;
}

int launch_merge(const DecodeParams &p, int B, int dv, int out_dtype, void *out, float *lse, cudaStream_t stream) {
    const dim3 grid(p.Hq, B);
    if (out_dtype == LSA_DTYPE_BF16)
        q4_merge_kernel<<<grid, dv / 4, 0, stream>>>(p, dv, static_cast<__nv_bfloat16 *>(out), lse);
    else if (out_dtype == LSA_DTYPE_F16)
        q4_merge_kernel<<<grid, dv / 4, 0, stream>>>(p, dv, static_cast<__half *>(out), lse);
    else
        q4_merge_kernel<<<grid, dv / 4, 0, stream>>>(p, dv, static_cast<float *>(out), lse);
    return check_launch("q4_merge_kernel");
}

static int max_units(int k, int max_window_len) { return (k + 63) / 64 + (max_window_len + 63) / 64 + 1; }

// Splits of one (sequence, K/V head, head group): enough CTAs for two a multiprocessor, each
// warp at least one unit.
static int separate_splits(int B, int heads, int G, int units) {
    const int hpc = G <= 8 ? 8 : 16, groups = (G + hpc - 1) / hpc;
    const int64_t per = (int64_t)B * heads * groups;
    const int64_t want = (2 * sm_count() + per - 1) / per;
    return (int)lsa_max64(1, lsa_min64(want, (units + WARPS - 1) / WARPS));
}

template <class C>
static int launch_separate(const DecodeParams &p, int B, int G, cudaStream_t stream) {
    const int groups = (G + C::HPC - 1) / C::HPC;
    LSA_CUDA(cudaFuncSetAttribute(q4_decode_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM));
    q4_decode_kernel<C><<<dim3(p.n_splits, p.heads * groups, B), WARPS * 32, C::SMEM, stream>>>(p);
    return check_launch("q4_decode_kernel");
}

static bool supported(int Hq, int heads, int dqk, int dv, bool latent) {
    if (Hq < 1 || heads < 1 || Hq % heads) return false;
    if (latent) return heads == 1 && dqk == 576 && dv == 512 && Hq <= 128;
    return dqk == dv && (dqk == 64 || dqk == 128) && Hq <= 1024;
}

static int splits_for(int B, int Hq, int heads, bool latent, int k, int max_window_len) {
    const int units = max_units(k, max_window_len);
    return latent ? q4mla::splits(B, units) : separate_splits(B, heads, Hq / heads, units);
}

}  // namespace q4
}  // namespace lsa

using namespace lsa;

extern "C" size_t lsa_sparse_decode_q4_workspace_size(int B, int Hq, int heads, int dqk, int dv, int k,
                                                      int max_window_len) {
    const bool latent = dqk != dv;
    if (!q4::supported(Hq, heads, dqk, dv, latent) || B < 1 || B > 65535 || k < 0 || max_window_len < 0) return 0;
    const int ns = q4::splits_for(B, Hq, heads, latent, k, max_window_len);
    Carver c(nullptr);
    c.take<float>((size_t)B * ns * Hq * dv);
    c.take<float>((size_t)B * ns * Hq);
    c.take<float>((size_t)B * ns * Hq);
    return align_up(c.used, 256);
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
    const size_t need = lsa_sparse_decode_q4_workspace_size(B, Hq, heads, dqk, dv, k, max_window_len);
    LSA_REQUIRE(ws && ws_bytes >= need, LSA_ERR_WORKSPACE, "lsa_sparse_decode_q4: workspace of %zu bytes, %zu needed",
                ws_bytes, need);
    q4::DecodeParams p = {};
    p.n_splits = q4::splits_for(B, Hq, heads, latent, k, max_window_len);
    Carver c(ws);
    p.o_part = c.take<float>((size_t)B * p.n_splits * Hq * dv);
    p.m_part = c.take<float>((size_t)B * p.n_splits * Hq);
    p.l_part = c.take<float>((size_t)B * p.n_splits * Hq);
    p.q = q; p.k_pool = k_pool; p.v_pool = v_pool; p.table = chunk_table; p.topk_idx = topk_idx;
    p.topk_count = topk_count; p.window_start = window_start; p.window_len = window_len; p.status = dev_status;
    p.n_slots = n_slots; p.table_stride = table_stride; p.k = k; p.Hq = Hq; p.heads = heads;
    p.scale_log2 = scale * k_scale * 1.4426950408889634f;
    p.v_scale = latent ? k_scale : v_scale;
    p.q_f16 = q_dtype == LSA_DTYPE_F16;
    const int G = Hq / heads;
    int rc;
    if (latent) rc = q4mla::launch(p, B, stream);
    else if (dqk == 128) rc = G <= 8 ? q4::launch_separate<q4::Cfg<128, 1>>(p, B, G, stream) : q4::launch_separate<q4::Cfg<128, 2>>(p, B, G, stream);
    else rc = G <= 8 ? q4::launch_separate<q4::Cfg<64, 1>>(p, B, G, stream) : q4::launch_separate<q4::Cfg<64, 2>>(p, B, G, stream);
    if (rc) return rc;
    return q4::launch_merge(p, B, dv, out_dtype, out, lse, stream);
}
