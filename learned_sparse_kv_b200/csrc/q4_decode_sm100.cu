// q4_decode_sm100.cu -- decode attention over 4-bit latent rows (576-wide keys, the first 512
// columns are the values, up to 128 query heads) on 5th-generation tensor cores.
//
// 278,528 flops for the 324 bytes of a row at 128 heads: bound by the tensor cores, so the
// codes are dequantised once per CTA into the f16 operand layout and everything else runs
// beside the products.
//
// A cluster of two CTAs owns one (sequence, split); tiles of 128 rows = two units of 64 (a window
// chunk, or 64 gathered top-k rows).  Every MMA is a cta_group::2 tcgen05.mma with M = 128 heads
// (CTA r holds heads 64r..64r+63 of Q and P; missing heads are zero rows), kind::f16, both
// operands f16:
//   S = Q K^T   N = 128 rows: CTA r dequantises unit r of the tile, all 576 columns (72 KB)
//   O += P V    N = 256 value columns: CTA r dequantises all 128 rows of its value columns
//               128r..128r+127 and 256+128r.. (64 KB)
// N = 128 because a pair MMA costs the same 45 cycles at N = 64 and at N = 128.  With Q (72 KB) and P
// (16 KB) that is all of shared memory, so K and V have one stage each: K of the next tile is
// written while P V runs, V of the next one while Q K^T runs.  The codes of the next tile
// are already in registers by then, and the slots of the one after are being looked up.
// TMEM per CTA: two S buffers of 64 columns and O = 64 heads x 512 values in 256 columns.
// Warp roles:
//   0      S = Q K^T issuer (even CTA)     1   O += P V issuer (even CTA)
//   2      TMEM allocator
//   4..7   softmax, O rescale, epilogue (one thread per TMEM lane: head x unit of the tile)
//   8..11  dequantise K                    12..15  dequantise V, row masks
// Every mbarrier wait is bounded: on timeout the kernel sets LSA_DEV_TIMEOUT and the abort flag of
// both CTAs, the other waits return, the MMAs issued so far complete, and the pair exits.  No
// copy is asynchronous (codes come through registers), so nothing else is in flight.
#include "q4_rows.cuh"
#include "sm100.cuh"

namespace lsa {
namespace q4mla {

using namespace sm100;
using q4::DecodeParams;
using q4::Units;

constexpr int HPC = 64, HQ = 128;       // heads per CTA, per cluster
constexpr int DQK = 576, DV = 512;
constexpr int KCH = DQK / 64;           // 9 column chunks of 64
constexpr int TILE = 128;
constexpr int INFO = 4;                 // row-mask ring
constexpr int THREADS = 512;
constexpr int ROW_CODE = DQK / 2, ROW_SCALE = DQK / 16;      // 288, 36 bytes

constexpr uint32_t TM_S = 0;            // S buffers at 0 and 64
constexpr uint32_t TM_O = 128;          // O at 128..383
constexpr uint32_t TM_COLS = 512;

struct __align__(1024) Smem {
    uint8_t q[KCH][HPC * 128];          // 9 x [64 heads][128 B], 128B-swizzled, K-major
    uint8_t k[KCH][64 * 128];           // [chunk][64 rows][64 columns], K-major
    uint8_t v[2][2][TILE * 128];        // [value block j][atom][128 rows][64 columns], MN-major
    uint8_t p[2][HPC * 128];            // [unit][64 heads][64 rows], K-major
    uint64_t k_full, v_full, p_full;    // the even CTA's: 8, 8 and 2 arrivals
    uint64_t s_full[2], s_empty[2];     // s_full[u & 1]: Q K^T of tile u done (K may be rewritten)
    uint64_t pv_done[2];                // pv_done[u & 1]: P V of tile u done (V and P may be rewritten)
    uint64_t info_full[INFO];
    uint64_t mma_done;
    uint64_t never;                     // no arrival ever: the failure-path test's wait
    uint32_t mask[INFO][4];             // present rows of a tile
    float qmul[HPC];                    // per head: score factor, scale * log2(e) * k_scale * 2^e
    float red[128];
    uint32_t tmem_base;
    int abort_flag;
};
static_assert(sizeof(Smem) + 1024 <= 232448, "shared memory of one CTA");

__device__ __noinline__ void set_abort(Smem &sm, int32_t *status) {
    sm.abort_flag = 1;
    asm volatile("st.shared::cluster.s32 [%0], %1;\n" ::"r"(map_to_rank(&sm.abort_flag, cluster_rank() ^ 1u)), "r"(1)
                 : "memory");
    flag(status, LSA_DEV_TIMEOUT);
}

// Warp-uniform bounded wait (lane 0 polls, result broadcast).
template <bool CLUSTER>
__device__ __forceinline__ bool warp_wait(Smem &sm, const uint64_t *bar, uint32_t parity, int32_t *status,
                                          uint64_t limit = WAIT_NS) {
    bool ok = true;
    if ((threadIdx.x & 31) == 0) {
        volatile int *abort = &sm.abort_flag;
        ok = *abort == 0 && (CLUSTER ? mbar_wait_cluster(bar, parity, limit, abort) : mbar_wait(bar, parity, limit, abort));
        if (!ok && *abort == 0) set_abort(sm, status);
    }
    return __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
}

__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N, bool b_mn_major) {
    return (1u << 4) /* D: f32; A and B: f16 = 0 */ | (uint32_t(b_mn_major) << 16) | (uint32_t(N >> 3) << 17) |
           (uint32_t(M >> 4) << 24);
}

// 32 codes (two groups) with their two scale bytes -> four 16-byte units of eight f16 values at
// units first .. first + 3 of a 128-byte swizzled row.
__device__ __forceinline__ void store_piece(uint32_t row_addr, int row, int first, const uint4 &c, uint32_t scales) {
    const uint32_t f = q4::e4m3x2_to_f16(scales), s[2] = {q4::dup_lo(f), q4::dup_hi(f)};
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t h[4];
        q4::e2m1x8_to_f16(w[i], h);
#pragma unroll
        for (int j = 0; j < 4; ++j) h[j] = q4::hmul2(h[j], s[i >> 1]);
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(row_addr + (((first + i) ^ (row & 7)) << 4)),
                     "r"(h[0]), "r"(h[1]), "r"(h[2]), "r"(h[3])
                     : "memory");
    }
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Pool row of row i of unit u, -1 if absent (past the set, or without a slot).
__device__ __forceinline__ int64_t unit_row(const Units &un, const DecodeParams &p, int b, int u, int i) {
    if (u >= un.total) return -1;
    if (u < un.t_topk) return un.topk_row(p, b, u, i);
    if (!un.in_window(u, i)) return -1;
    const int slot = un.window_slot(p, b, u);
    return slot < 0 ? -1 : (int64_t)slot * LSA_CHUNK + i;
}

// Reads piece `piece` (32 codes) of a row and its two scales.
__device__ __forceinline__ void load_piece(const uint8_t *pool, int64_t row, int piece, uint4 &c, uint32_t &s) {
    c = make_uint4(0, 0, 0, 0);
    s = 0;
    if (row >= 0) {
        const uint8_t *chunk = pool + (row >> 6) * q4::chunk_bytes(DQK);
        const int r = (int)(row & 63);
        c = __ldg(reinterpret_cast<const uint4 *>(chunk + r * ROW_CODE + piece * 16));
        s = __ldg(reinterpret_cast<const uint16_t *>(chunk + LSA_CHUNK * ROW_CODE + r * ROW_SCALE + piece * 2));
    }
}

__global__ void __launch_bounds__(THREADS, 1) q4_mla_kernel(const DecodeParams p, int stall) {
    extern __shared__ uint8_t smem_raw[];
    Smem &sm = *reinterpret_cast<Smem *>(smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const int split = blockIdx.x >> 1, b = blockIdx.y;
    const Units un(p, b);
    const int tiles = (un.total + 1) / 2;
    const int n_tiles = split < tiles ? (tiles - 1 - split) / p.n_splits + 1 : 0;   // dealt round-robin
    auto tile_of = [&](int u) { return split + u * p.n_splits; };

    if (threadIdx.x == 0) {
        mbar_init(&sm.k_full, 8);
        mbar_init(&sm.v_full, 8);
        mbar_init(&sm.p_full, 2);
        for (int i = 0; i < 2; ++i) { mbar_init(&sm.s_full[i], 1); mbar_init(&sm.s_empty[i], 2); mbar_init(&sm.pv_done[i], 1); }
        for (int i = 0; i < INFO; ++i) mbar_init(&sm.info_full[i], 4);
        mbar_init(&sm.mma_done, 2);   // one commit from each MMA issuer
        mbar_init(&sm.never, 1);
        sm.abort_flag = 0;
        fence_mbar_init_cluster();
    }
    if (warp == 2) tmem_alloc_pair(&sm.tmem_base, TM_COLS);
    if (n_tiles > 0) {
        // queries as f16 over a power of two, straight into the operand layout
        const uint32_t qb = smem_addr(sm.q);
        for (int h = warp; h < HPC; h += THREADS / 32) {
            const int head = HPC * (int)rank + h;
            const bool live = head < p.Hq;
            const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.q) +
                                                               ((size_t)b * p.Hq + (live ? head : 0)) * DQK);
            float x[3][8];
            float amax = 0.f;
#pragma unroll
            for (int i = 0; i < 3; ++i) {
                const int piece = lane + 32 * i;
                const uint4 w = live && piece < DQK / 8 ? __ldg(src + piece) : make_uint4(0, 0, 0, 0);
                const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (p.q_f16) {
                        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&ww[j]));
                        x[i][2 * j] = f.x; x[i][2 * j + 1] = f.y;
                    } else {
                        x[i][2 * j] = __uint_as_float(ww[j] << 16);
                        x[i][2 * j + 1] = __uint_as_float(ww[j] & 0xffff0000u);
                    }
                    amax = fmaxf(amax, fmaxf(fabsf(x[i][2 * j]), fabsf(x[i][2 * j + 1])));
                }
            }
            amax = warp_max(amax);
            float inv;
            const float e = q4::row_exponent(amax, inv);
            if (lane == 0) sm.qmul[h] = e * p.scale_log2;
#pragma unroll
            for (int i = 0; i < 3; ++i) {
                const int piece = lane + 32 * i;
                if (piece < DQK / 8)
                    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                                     qb + (piece >> 3) * (HPC * 128) + h * 128 + (((piece & 7) ^ (h & 7)) << 4)),
                                 "r"(q4::pack_f16x2(x[i][0] * inv, x[i][1] * inv)), "r"(q4::pack_f16x2(x[i][2] * inv, x[i][3] * inv)),
                                 "r"(q4::pack_f16x2(x[i][4] * inv, x[i][5] * inv)), "r"(q4::pack_f16x2(x[i][6] * inv, x[i][7] * inv))
                                 : "memory");
            }
        }
        fence_proxy_async_smem();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    cluster_sync();
    const uint32_t tmem = sm.tmem_base;

    if (warp == 0 && rank == 0 && n_tiles > 0) {
        // ------------------------------------------------ S = Q K^T issuer
        constexpr uint32_t IDESC = idesc_f16_f32(HQ, TILE, false);
        constexpr uint64_t CHUNK = (64 * 128) >> 4, K16 = 32 >> 4;
        const uint64_t qd = smem_desc_sw128(smem_addr(sm.q), 16, 1024), kd = smem_desc_sw128(smem_addr(sm.k), 16, 1024);
        bool ok = true;
        if (stall) ok = warp_wait<false>(sm, &sm.never, 0, p.status, TEST_STALL_NS);
        for (int u = 0; u < n_tiles && ok; ++u) {
            const int sb = u & 1;
            ok = warp_wait<true>(sm, &sm.s_empty[sb], ((u >> 1) + 1) & 1, p.status) &&
                 warp_wait<true>(sm, &sm.k_full, u & 1, p.status);
            if (!ok) break;
            tc_fence_after();
            if (lane == 0) {
#pragma unroll
                for (int c = 0; c < KCH; ++c)
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        umma_pair_ss(tmem + TM_S + 64 * sb, qd + CHUNK * c + K16 * kk, kd + CHUNK * c + K16 * kk, IDESC,
                                     (c | kk) != 0);
                umma_commit_pair(&sm.s_full[sb], 0x3);
            }
            __syncwarp();
        }
        if (lane == 0) umma_commit_pair(&sm.mma_done, 0x3);
        __syncwarp();
    } else if (warp == 1 && rank == 0 && n_tiles > 0) {
        // ------------------------------------------------ O += P V issuer
        constexpr uint32_t IDESC = idesc_f16_f32(HQ, 256, true);
        constexpr uint64_t P_ATOM = (HPC * 128) >> 4, V_J = (2 * TILE * 128) >> 4, V16 = (16 * 128) >> 4, K16 = 32 >> 4;
        const uint64_t pd = smem_desc_sw128(smem_addr(sm.p), 16, 1024);
        const uint64_t vd = smem_desc_sw128(smem_addr(sm.v), TILE * 128, 1024);
        bool ok = true;
        for (int u = 0; u < n_tiles && ok; ++u) {
            ok = warp_wait<true>(sm, &sm.p_full, u & 1, p.status) && warp_wait<true>(sm, &sm.v_full, u & 1, p.status);
            if (!ok) break;
            tc_fence_after();
            if (lane == 0) {
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)
                        umma_pair_ss(tmem + TM_O + 128 * j, pd + P_ATOM * (kk >> 2) + K16 * (kk & 3), vd + V_J * j + V16 * kk,
                                     IDESC, u > 0 || kk > 0);
                umma_commit_pair(&sm.pv_done[u & 1], 0x3);
            }
            __syncwarp();
        }
        if (lane == 0) umma_commit_pair(&sm.mma_done, 0x3);
        __syncwarp();
    } else if (warp >= 8 && warp < 12 && n_tiles > 0) {
        // ------------------------------------------------ K: unit `rank` of each tile, 16 rows a warp
        const int w = warp - 8, row = 16 * w + (lane >> 1), hf = lane & 1;
        const uint32_t dst = smem_addr(sm.k) + row * 128, full = map_to_rank(&sm.k_full, 0);
        auto resolve = [&](int u) -> int64_t {
            return u < n_tiles ? unit_row(un, p, b, 2 * tile_of(u) + (int)rank, row) : -1;
        };
        uint4 c[KCH];
        uint32_t s[KCH];
        int64_t r = resolve(0);
#pragma unroll
        for (int i = 0; i < KCH; ++i) load_piece(p.k_pool, r, 2 * i + hf, c[i], s[i]);
        r = resolve(1);
        for (int u = 0; u < n_tiles; ++u) {
            if (u > 0 && !warp_wait<false>(sm, &sm.s_full[(u - 1) & 1], ((u - 1) >> 1) & 1, p.status)) break;
#pragma unroll
            for (int i = 0; i < KCH; ++i) store_piece(dst + i * (64 * 128), row, 4 * hf, c[i], s[i]);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive_release_cluster(full);
#pragma unroll
            for (int i = 0; i < KCH; ++i) load_piece(p.k_pool, r, 2 * i + hf, c[i], s[i]);
            r = resolve(u + 2);
        }
    } else if (warp >= 12 && n_tiles > 0) {
        // ------------------------------------------------ V: all rows of the tile, this CTA's columns, 32 rows a warp
        const int w = warp - 12, hf = lane & 1;
        const uint32_t vb = smem_addr(sm.v), full = map_to_rank(&sm.v_full, 0);
        // lane i looks up row 32 w + i of the tile, whose presence the softmax needs
        auto resolve = [&](int u) -> int64_t {
            if (u >= n_tiles) return -1;
            const int i = 32 * w + lane;
            const int64_t r = unit_row(un, p, b, 2 * tile_of(u) + (i >> 6), i & 63);
            const uint32_t m = __ballot_sync(0xffffffffu, r >= 0);
            // The ring slot was last read for tile u - 4; P V of tile u - 3 was done before
            // this warp wrote V of tile u - 2, so that read is long past.
            if (lane == 0) {
                sm.mask[u % INFO][w] = m;
                asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];\n" ::"r"(smem_addr(&sm.info_full[u % INFO])) : "memory");
            }
            __syncwarp();
            return r;
        };
        uint4 c[8];
        uint32_t s[8];
        auto load = [&](int64_t r) {
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int64_t rr = __shfl_sync(0xffffffffu, r, 16 * q + (lane >> 1));
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    load_piece(p.k_pool, rr, 2 * (4 * (i >> 1) + 2 * (int)rank + (i & 1)) + hf, c[4 * q + i], s[4 * q + i]);
            }
        };
        int64_t r = resolve(0);
        load(r);
        r = resolve(1);
        for (int u = 0; u < n_tiles; ++u) {
            if (u > 0 && !warp_wait<false>(sm, &sm.pv_done[(u - 1) & 1], ((u - 1) >> 1) & 1, p.status)) break;
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int row = 32 * w + 16 * q + (lane >> 1);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    store_piece(vb + i * (TILE * 128) + row * 128, row, 4 * hf, c[4 * q + i], s[4 * q + i]);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive_release_cluster(full);
            load(r);
            r = resolve(u + 2);
        }
    } else if (warp >= 4 && warp < 8) {
        // ------------------------------------------------ softmax + epilogue
        const int L = threadIdx.x - 128;         // TMEM lane of this thread
        const int h = L & 63, half = L >> 6;     // head within the CTA, unit of the tile
        const uint32_t lane_base = (uint32_t)(32 * (warp & 3)) << 16;
        const float mul = n_tiles > 0 ? sm.qmul[h] : 0.f;
        float m_ref = -INFINITY, l = 0.f;
        bool ok = true;
        for (int u = 0; u < n_tiles; ++u) {
            const int s = u & 1;
            ok = ok && *(volatile int *)&sm.abort_flag == 0;
            if (ok) ok = mbar_wait(&sm.info_full[u % INFO], (u / INFO) & 1, WAIT_NS, &sm.abort_flag);
            uint32_t vm[2] = {0u, 0u};
            if (ok) { vm[0] = sm.mask[u % INFO][2 * half]; vm[1] = sm.mask[u % INFO][2 * half + 1]; }
            if (ok) ok = mbar_wait(&sm.s_full[s], (u >> 1) & 1, WAIT_NS, &sm.abort_flag);
            if (!ok && *(volatile int *)&sm.abort_flag == 0) set_abort(sm, p.status);
            tc_fence_after();
            uint32_t raw[2][32];
            tmem_ld32(tmem + lane_base + TM_S + 64 * s, raw[0]);
            tmem_ld32(tmem + lane_base + TM_S + 64 * s + 32, raw[1]);
            tmem_wait_ld();
            tc_fence_before();
            float mx = -INFINITY;
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    const float x = (vm[q] >> i) & 1u ? __uint_as_float(raw[q][i]) * mul : -INFINITY;
                    raw[q][i] = __float_as_uint(x);
                    mx = fmaxf(mx, x);
                }
            sm.red[L] = mx;
            named_barrier(1, 128);
            if (L == 0) mbar_arrive_release_cluster(map_to_rank(&sm.s_empty[s], 0));
            mx = fmaxf(mx, sm.red[L ^ 64]);
            const bool move = mx > m_ref + q4::RESCALE;
            const float alpha = move ? ex2(m_ref - mx) : 1.f;      // 0 the first time (m_ref = -inf)
            if (move) {
                l *= alpha;
                m_ref = mx;
            }
            const float ref = m_ref == -INFINITY ? 0.f : m_ref - q4::P_SHIFT;
            float psum = 0.f;
            uint32_t pk[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                const float p0 = ex2(__uint_as_float(raw[i >> 4][2 * (i & 15)]) - ref);
                const float p1 = ex2(__uint_as_float(raw[i >> 4][2 * (i & 15) + 1]) - ref);
                psum += p0 + p1;
                pk[i] = q4::pack_f16x2(p0, p1);
            }
            l += psum;
            // P is rewritten and O may be rescaled: P V of tile u - 1 must be done
            if (u > 0 && ok) {
                ok = mbar_wait(&sm.pv_done[(u - 1) & 1], ((u - 1) >> 1) & 1, WAIT_NS, &sm.abort_flag);
                if (!ok && *(volatile int *)&sm.abort_flag == 0) set_abort(sm, p.status);
            }
            // tcgen05.ld / st are warp-collective: the whole warp rescales when any row moves
            if (__any_sync(0xffffffffu, move) && u > 0) {
                tc_fence_after();
#pragma unroll 1
                for (int q = 0; q < 8; ++q) {
                    uint32_t o[32];
                    tmem_ld32(tmem + lane_base + TM_O + 32 * q, o);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
                    tmem_st32(tmem + lane_base + TM_O + 32 * q, o);
                }
                tmem_wait_st();
            }
            uint8_t *prow = sm.p[half] + h * 128;
#pragma unroll
            for (int c = 0; c < 8; ++c)
                *reinterpret_cast<uint4 *>(prow + ((c ^ (h & 7)) << 4)) =
                    make_uint4(pk[4 * c], pk[4 * c + 1], pk[4 * c + 2], pk[4 * c + 3]);
            fence_proxy_async_smem();
            tc_fence_before();
            named_barrier(1, 128);
            if (L == 0) mbar_arrive_release_cluster(map_to_rank(&sm.p_full, 0));
        }
        // ---- epilogue: wait for the last P V, then write the partial
        if (n_tiles > 0 && ok) {
            ok = mbar_wait(&sm.pv_done[(n_tiles - 1) & 1], ((n_tiles - 1) >> 1) & 1, WAIT_NS, &sm.abort_flag);
            if (!ok && *(volatile int *)&sm.abort_flag == 0) set_abort(sm, p.status);
        }
        tc_fence_after();
        named_barrier(1, 128);
        sm.red[L] = l;
        named_barrier(1, 128);
        const float l_tot = l + sm.red[L ^ 64];
        const int head = HPC * (int)rank + h;
        const size_t part0 = ((size_t)b * p.n_splits + split) * p.Hq;
        if (half == 0 && head < p.Hq) {
            p.m_part[part0 + head] = m_ref - q4::P_SHIFT;
            p.l_part[part0 + head] = l_tot;
        }
        // O leaves tensor memory 32 columns at a time and passes through shared memory (the P
        // buffers), so that every store instruction writes whole 128-byte row pieces.
        float *xbuf = reinterpret_cast<float *>(sm.p[0]) + (warp & 3) * 1024;
        const int head0 = HPC * (int)rank + (32 * (warp & 3) & 63);
#pragma unroll 1
        for (int q = 0; q < 8; ++q) {
            uint32_t o[32];
            if (n_tiles > 0) {
                tmem_ld32(tmem + lane_base + TM_O + 32 * q, o);
                tmem_wait_ld();
            } else {
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] = 0u;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
                *reinterpret_cast<uint4 *>(xbuf + lane * 32 + 4 * ((i ^ lane) & 7)) =
                    make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
            __syncwarp();
            // O columns 0..127 hold values 0..255 split by lane half; 128..255 hold 256..511
            const int col = 256 * (q >> 2) + 128 * half + (q & 3) * 32 + 4 * (lane & 7);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int r = 4 * k + (lane >> 3);
                const float4 v = *reinterpret_cast<const float4 *>(xbuf + r * 32 + 4 * (((lane & 7) ^ r) & 7));
                if (head0 + r < p.Hq) *reinterpret_cast<float4 *>(p.o_part + (part0 + head0 + r) * DV + col) = v;
            }
            __syncwarp();
        }
        tc_fence_before();
    }

    // ---- teardown: every MMA finished before TMEM is released and before either CTA leaves
    if (warp == 2 && n_tiles > 0) {
        if (lane == 0 && !mbar_wait(&sm.mma_done, 0, WAIT_NS)) set_abort(sm, p.status);
        __syncwarp();
    }
    __syncthreads();
    cluster_sync();
    if (warp == 2) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, TM_COLS);
        tmem_relinquish_pair();
    }
}

// Splits per sequence: one CTA pair each, all co-resident; a single sequence takes half the pairs.
int splits(int B, int max_units) {
    const int clusters = sm_count() / 2, tiles = (max_units + 1) / 2;
    return max(1, min(min(clusters / max(B, 1), clusters / 2), tiles));
}

int launch(const DecodeParams &p, int B, cudaStream_t stream) {
    const size_t smem = sizeof(Smem) + 1024;
    LSA_CUDA(cudaFuncSetAttribute(q4_mla_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * p.n_splits, B, 1);
    cfg.blockDim = dim3(THREADS, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    LSA_CUDA(cudaLaunchKernelEx(&cfg, q4_mla_kernel, p, take_test_stall(LSA_TEST_STALL_ATTENTION_Q4)));
    return LSA_OK;
}

}  // namespace q4mla
}  // namespace lsa
