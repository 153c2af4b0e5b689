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
// (16 KB) that is all of shared memory, so K and V have one stage each, handed over in parts: K
// in groups of 256, 256 and 64 columns, V and P unit by unit.  A part of the next tile is written
// as soon as the MMAs that read it are done, while the MMAs of the other parts run.  The
// codes of the next tile are in registers by then, the slots of the one after are being loaded.
// TMEM per CTA: two S buffers of 64 columns and O = 64 heads x 512 values in 256 columns.
// Warp roles:
//   0      MMA issuer (even CTA)            2   TMEM allocator
//   4..7   softmax, O rescale (one thread per TMEM lane: head x unit of the tile)
//   8..15  dequantise K                    16..23  dequantise V, row masks; both write O at the end
// (Eight warps each: with four the conversion, a chain of dependent instructions, took 3000
// cycles a tile and paced the pipeline while the issue slots were 25 % used.)
// Measured on the device, merge included: 8 sequences of 10,048 rows, 128 heads: 38.8 us (577 TFLOP/s), with weights in
// two parts 49.2; 32 such sequences, 64 heads: 122.5 and 168 us.  A tile takes 4,400 cycles for 2,640 of MMAs timed
// alone: operand reads (240 KB a tile and CTA) and the conversion's stores (152 KB) share the shared-memory pipe, 128
// bytes a cycle, which is 3,060 of them, and while the conversion stores an MMA of Q K^T takes 72 cycles instead of
// 45.  What shortens other chains did not help: eight softmax warps of 32 columns a thread 41.2 us, rows looked up by one warp for
// all 40.0, loads of a row by 12 neighbouring lanes 42.9.  A launch spends 9,000 cycles on its prologue
// (lengths, positions, slots, codes: loads that wait for each other).
// Every mbarrier wait is bounded, each by itself and never the launch as a whole: on timeout the kernel sets
// LSA_DEV_TIMEOUT and the abort flag of both CTAs, the other waits return, the MMAs issued so far complete (a wait
// that starts when all roles have ended and that the abort flag does not cut short), and the pair exits.  No
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
constexpr int KG = 3;                   // K in groups of 256, 256 and 64 columns
constexpr int INFO = 4;                 // row-mask ring
constexpr int THREADS = 768, DEQ = 8;    // DEQ: warps of each dequantising group
constexpr int ROW_CODE = DQK / 2, ROW_SCALE = DQK / 16;      // 288, 36 bytes

constexpr uint32_t TM_S = 0;            // S buffers at 0 and 64
constexpr uint32_t TM_O = 128;          // O at 128..383
constexpr uint32_t TM_COLS = 512;

struct __align__(1024) Smem {
    uint8_t q[KCH][HPC * 128];          // 9 x [64 heads][128 B], 128B-swizzled, K-major
    uint8_t k[KCH][64 * 128];           // [chunk][64 rows][64 columns], K-major
    uint8_t v[2][2][TILE * 128];        // [value block j][atom][128 rows][64 columns], MN-major
    uint8_t p[2][HPC * 128];            // [unit][64 heads][64 rows], K-major
    uint64_t k_full;                    // the even CTA's, 16 arrivals (one a warp): K is written
    uint64_t k_empty[KG];               // the MMAs that read that part of K are done
    uint64_t pv_full[2];                // the even CTA's, 16 arrivals: V and P of unit a of the tile are written
    uint64_t pv_done[2];                // P V over unit a is done: its V and P may be rewritten
    uint64_t first_done[2];             // two-part weights: the product with the first part is done, P may be rewritten
    uint64_t rest_full[2];              // the even CTA's, 4 arrivals: the second part of P of unit a is written
    uint64_t s_full[2];                 // S buffers
    uint64_t info_full[INFO];
    uint64_t mma_done;                  // all MMAs are done
    uint64_t never;                     // no arrival ever: the failure-path test's wait
    alignas(16) uint16_t mask[INFO][DEQ];           // present rows of a tile, 16 a word
    float qmul[HPC];                    // per head: score factor, scale * log2(e) * k_scale * 2^e
    float red[2][128];                  // row maxima of the two units, by u & 1
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

// Bounded wait on the SM's own clock: reading the global timer between two tries takes longer than most
// of these waits last.  The limit is some two seconds of cycles; the abort flag, if given, is looked at after 2^18.
constexpr long long WAIT_CYCLES = 1ll << 32, STALL_CYCLES = 1ll << 22, ABORT_CYCLES = 1ll << 18;
__device__ __noinline__ bool wait_longer(uint32_t a, uint32_t parity, const volatile int *abort, long long limit) {
    const long long t0 = clock64();
    for (;;) {
        if (mbar_try_wait(a, parity)) return true;
        const long long dt = clock64() - t0;
        if (dt > limit || (abort && dt > ABORT_CYCLES && *abort)) return false;
    }
}
__device__ __forceinline__ bool wait_for(const uint64_t *bar, uint32_t parity, const volatile int *abort,
                                         long long limit = WAIT_CYCLES) {
    const uint32_t a = smem_addr(bar);
    return mbar_try_wait(a, parity) || wait_longer(a, parity, abort, limit);
}

// Bounded wait of a whole warp (every lane polls the same word, so that the usual case, a phase that is
// complete already, is one shared-memory access and no exchange).  Operands in shared memory are
// written by generic stores, each writer's followed by its own fence.proxy.async before the arrive.
__device__ __forceinline__ bool warp_wait(Smem &sm, const uint64_t *bar, uint32_t parity, int32_t *status,
                                          long long limit = WAIT_CYCLES) {
    volatile int *abort = &sm.abort_flag;
    const bool ok = __all_sync(0xffffffffu, wait_for(bar, parity, abort, limit));
    if (!ok && *abort == 0) set_abort(sm, status);
    return ok;
}

// One lane of a converged warp (always the same one), by the instruction that says so: the compiler then
// knows that the branch is taken by one lane and keeps the MMA descriptors in uniform registers.
__device__ __forceinline__ bool elect_one() {
    uint32_t pred;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(pred));
    return pred != 0;
}

__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N, bool b_mn_major) {
    return (1u << 4) /* D: f32; A and B: f16 = 0 */ | (uint32_t(b_mn_major) << 16) | (uint32_t(N >> 3) << 17) |
           (uint32_t(M >> 4) << 24);
}

// Eight codes times a scale -> one 16-byte unit of f16 values.
__device__ __forceinline__ void store_unit(uint32_t at, uint32_t codes, uint32_t scale2) {
    uint32_t h[4];
    q4::e2m1x8_to_f16(codes, h);
#pragma unroll
    for (int j = 0; j < 4; ++j) h[j] = q4::hmul2(h[j], scale2);
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(h[0]), "r"(h[1]), "r"(h[2]), "r"(h[3]) : "memory");
}

// 32 columns of a row, a half of a 64-column chunk: four units at `at` ^ 16 i.  Lanes of odd chunks (`odd`) hand in
// the address of their third unit and take the second group first, so that eight neighbouring lanes (two
// rows of 128 columns) store to all banks.
__device__ __forceinline__ void store_half(uint32_t at, bool odd, const uint4 &c, uint32_t scales) {
    const uint32_t s = q4::e4m3x2_to_f16(scales);
    const uint32_t s0 = __byte_perm(s, 0, odd ? 0x3232 : 0x1010), s1 = __byte_perm(s, 0, odd ? 0x1010 : 0x3232);
    store_unit(at, odd ? c.z : c.x, s0);
    store_unit(at ^ 16, odd ? c.w : c.y, s0);
    store_unit(at ^ 32, odd ? c.x : c.z, s1);
    store_unit(at ^ 48, odd ? c.y : c.w, s1);
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The row lookup is two dependent loads (position, slot), each issued a tile ahead of its use and
// checked only then, so that no warp stands still for it.
// Position of row i of unit u; ABSENT past the set.
constexpr int ABSENT = INT32_MIN;
__device__ __forceinline__ int row_position(const Units &un, const DecodeParams &p, int b, int u, int i) {
    if (u >= un.total) return ABSENT;
    if (u < un.t_topk) {
        const int r = u * LSA_CHUNK + i;
        return r < un.tk ? __ldg(p.topk_idx + (size_t)b * p.k + r) : ABSENT;
    }
    return un.in_window(u, i) ? (un.first_chunk + (u - un.t_topk)) * LSA_CHUNK + i : ABSENT;
}
// Table entry of a position, -1 if it has none.
__device__ __forceinline__ int row_slot(const DecodeParams &p, int b, int pos) {
    return pos >= 0 && pos / LSA_CHUNK < p.table_stride ? __ldg(p.table + (size_t)b * p.table_stride + pos / LSA_CHUNK) : -1;
}
// Pool row from both, -1 if the row takes no part (flagged unless it is past the set, which is asked of the set
// itself: ABSENT can be an index, too).
__device__ __forceinline__ int64_t pool_row(const Units &un, const DecodeParams &p, int pos, int slot, int u, int i) {
    if (slot >= 0 && slot < p.n_slots) return (int64_t)slot * LSA_CHUNK + (pos & (LSA_CHUNK - 1));
    if (u < un.total && (u < un.t_topk ? u * LSA_CHUNK + i < un.tk : un.in_window(u, i)))
        flag(p.status, pos < 0 ? LSA_DEV_INDEX : LSA_DEV_TABLE);
    return -1;
}

// A pool row.  Four lanes share it, lane `quarter` takes 32 of every 128 columns, and 16 of the last 64 of a key.
// An absent row reads the pool's first row and gets zero scales, which make it zeros whatever it holds.
struct RowPtr {
    const uint8_t *code, *scale;
    bool there;
    __device__ RowPtr(const uint8_t *pool, int64_t row) {
        there = row >= 0;
        const uint8_t *chunk = pool + (there ? row >> 6 : 0) * q4::chunk_bytes(DQK);
        const int r = there ? (int)(row & 63) : 0;
        code = chunk + r * ROW_CODE;
        scale = chunk + LSA_CHUNK * ROW_CODE + r * ROW_SCALE;
    }
    __device__ __forceinline__ void load(int block, int quarter, uint4 &c, uint32_t &s) const {
        c = __ldg(reinterpret_cast<const uint4 *>(code + 64 * block + 16 * quarter));
        s = there ? (uint32_t)__ldg(reinterpret_cast<const uint16_t *>(scale + 8 * block + 2 * quarter)) : 0u;
    }
    __device__ __forceinline__ void load_last(int quarter, uint2 &c, uint32_t &s) const {
        c = __ldg(reinterpret_cast<const uint2 *>(code + 256 + 8 * quarter));
        s = there ? (uint32_t)__ldg(scale + 32 + quarter) : 0u;
    }
};

// TWO: weights in two parts (q4::two_parts).  The second goes through the same P buffer once the first has been
// multiplied, so a tile's products take 1300 cycles more.
template <bool TWO>
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
        mbar_init(&sm.k_full, 2 * DEQ);
        for (int i = 0; i < KG; ++i) mbar_init(&sm.k_empty[i], 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.pv_full[i], DEQ + 8);
            mbar_init(&sm.pv_done[i], 1);
            mbar_init(&sm.first_done[i], 1);
            mbar_init(&sm.rest_full[i], 4);
            mbar_init(&sm.s_full[i], 1);
        }
        for (int i = 0; i < INFO; ++i) mbar_init(&sm.info_full[i], DEQ);
        mbar_init(&sm.mma_done, 1);
        mbar_init(&sm.never, 1);
        sm.abort_flag = 0;
        fence_mbar_init_cluster();
    }
    if (warp == 2) tmem_alloc_pair(&sm.tmem_base, TM_COLS);
    // ---- the dequantising warps look up and load their part of the first tile
    // K: unit `rank` of each tile, 8 rows a warp, all columns.  V: all rows of the tile, 16 a warp in
    // two passes of 8, this CTA's two blocks of 128 columns.  Lane i looks up row i of the warp's.
    const bool kwarp = warp >= 8 && warp < 16, vwarp = warp >= 16;
    const int w = warp & 7, quarter = lane & 3;
    const int unit_in_tile = kwarp ? (int)rank : w >> 2, first_row = kwarp ? 8 * w : 16 * (w & 3);   // in that unit
    const int my_row = first_row + (lane & (kwarp ? 7 : 15));
    auto position = [&](int u) -> int {
        return u < n_tiles ? row_position(un, p, b, 2 * tile_of(u) + unit_in_tile, my_row) : ABSENT;
    };
    auto pool_row_of = [&](int u, int pos, int slot) { return pool_row(un, p, pos, slot, 2 * tile_of(u) + unit_in_tile, my_row); };
    uint4 c[4];          // K: the four blocks of 128 columns; V: block i >> 1, row pass i & 1
    uint2 c_last;        // K: columns 512..575
    uint32_t sc[5];
    int pos1 = ABSENT, pos2 = ABSENT, slot1 = -1;     // of tiles u + 1 and u + 2 in the loops below
    auto load = [&](int64_t r) {
        if (kwarp) {
            const RowPtr row(p.k_pool, __shfl_sync(0xffffffffu, r, lane >> 2));
#pragma unroll
            for (int i = 0; i < 4; ++i) row.load(i, quarter, c[i], sc[i]);
            row.load_last(quarter, c_last, sc[4]);
        } else {
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const RowPtr row(p.k_pool, __shfl_sync(0xffffffffu, r, 8 * q + (lane >> 2)));
#pragma unroll
                for (int j = 0; j < 2; ++j) row.load(2 * j + (int)rank, quarter, c[2 * j + q], sc[2 * j + q]);
            }
        }
    };
    // Row presence of tile u for the softmax, posted before this warp writes V of tile u - 1.  The ring slot
    // was last read for tile u - 4, by softmax warps of the same unit, whose P V was done before this warp
    // wrote V of tile u - 3.
    auto post_mask = [&](int u, int64_t r) {
        const uint32_t m = __ballot_sync(0xffffffffu, r >= 0);
        if (lane == 0) {
            sm.mask[u % INFO][w] = (uint16_t)m;
            asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];\n" ::"r"(smem_addr(&sm.info_full[u % INFO])) : "memory");
        }
        __syncwarp();
    };
    int64_t row0 = -1;
    if (warp >= 8 && n_tiles > 0) {
        const int pos0 = position(0);
        pos1 = position(1);
        pos2 = position(2);
        const int slot0 = row_slot(p, b, pos0);
        slot1 = row_slot(p, b, pos1);
        row0 = pool_row_of(0, pos0, slot0);
        load(row0);
    }
    if (n_tiles > 0) {
        // ---- queries as f16 over a power of two, straight into the operand layout: four heads each by warps 0..7,
        // two by the others, whose codes are under way
        const uint32_t qb = smem_addr(sm.q);
#pragma unroll 1
        for (int h0 = warp < 8 ? 4 * warp : 16 + 2 * warp, h1 = h0 + (warp < 8 ? 4 : 2); h0 < h1; h0 += 2) {
        uint4 held[2][3];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            const int head = HPC * (int)rank + h0 + n;
            const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.q) + ((size_t)b * p.Hq + head) * DQK);
#pragma unroll
            for (int i = 0; i < 3; ++i)
                held[n][i] = head < p.Hq && lane + 32 * i < DQK / 8 ? __ldg(src + lane + 32 * i) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            const int h = h0 + n;
            const uint4 (&raw)[3] = held[n];
            float x[3][8];
            float amax = 0.f;
#pragma unroll
            for (int i = 0; i < 3; ++i) {
                const uint32_t ww[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
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
            if (lane == 0) sm.qmul[h] = q4::score_factor(e, p.scale_log2);
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
        }
        fence_proxy_async_smem();
    }
    __syncwarp();          // the barriers take converged warps
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    cluster_sync();
    const uint32_t tmem = sm.tmem_base;

    if (warp == 0 && rank == 0 && n_tiles > 0) {
        // ------------------------------------------------ MMA issuer: S(0), then S(u + 1) and O += P V(u) in turn
        constexpr uint32_t IDESC_QK = idesc_f16_f32(HQ, TILE, false), IDESC_PV = idesc_f16_f32(HQ, 256, true);
        constexpr uint64_t CHUNK = (64 * 128) >> 4, K16 = 32 >> 4;
        constexpr uint64_t P_ATOM = (HPC * 128) >> 4, V_J = (2 * TILE * 128) >> 4, V16 = (16 * 128) >> 4;
        const uint64_t qd = smem_desc_sw128(smem_addr(sm.q), 16, 1024), kd = smem_desc_sw128(smem_addr(sm.k), 16, 1024);
        const uint64_t pd = smem_desc_sw128(smem_addr(sm.p), 16, 1024), vd = smem_desc_sw128(smem_addr(sm.v), TILE * 128, 1024);
        bool ok = true;
        if (stall) ok = warp_wait(sm, &sm.never, 0, p.status, STALL_CYCLES);
#pragma unroll 1
        for (int u = -1; u < n_tiles && ok; ++u) {
            // The S buffer of tile u + 1 was read before P of tile u - 1 (all of its parts) was written, which
            // P V(u - 1) waited for.
            const int n = u + 1, sb = n & 1;
            if (n < n_tiles) {
                ok = warp_wait(sm, &sm.k_full, n & 1, p.status);
                if (!ok) break;
                tc_fence_after();
                if (elect_one()) {
#pragma unroll 1
                    for (int g = 0; g < KG; ++g) {
#pragma unroll 1
                        for (int c = 4 * g; c < min(4 * (g + 1), KCH); ++c) {
                            const uint64_t at = CHUNK * c;
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk)
                                umma_pair_ss(tmem + TM_S + 64 * sb, qd + at + K16 * kk, kd + at + K16 * kk, IDESC_QK, (c | kk) != 0);
                        }
                        umma_commit_pair(&sm.k_empty[g], 0x3);
                    }
                    umma_commit_pair(&sm.s_full[sb], 0x3);
                }
                __syncwarp();
            }
#pragma unroll 1
            for (int i = 0; i < (TWO ? 4 : 2) && u >= 0; ++i) {
                const int a = i & 1;
                ok = warp_wait(sm, i < 2 ? &sm.pv_full[a] : &sm.rest_full[a], u & 1, p.status);
                if (!ok) break;
                tc_fence_after();
                if (elect_one()) {
#pragma unroll 1
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            umma_pair_ss(tmem + TM_O + 128 * j, pd + P_ATOM * a + K16 * kk, vd + V_J * j + V16 * (4 * a + kk), IDESC_PV,
                                         (u | i | kk) != 0);
                    umma_commit_pair(!TWO || i >= 2 ? &sm.pv_done[a] : &sm.first_done[a], 0x3);
                }
                __syncwarp();
            }
        }
        if (elect_one()) umma_commit_pair(&sm.mma_done, 0x3);
        __syncwarp();
    } else if (kwarp && n_tiles > 0) {
        // ------------------------------------------------ dequantise K
        const int row = first_row + (lane >> 2);
        const bool odd = quarter >> 1;
        const uint32_t rows = smem_addr(sm.k) + row * 128, full = map_to_rank(&sm.k_full, 0);
        const uint32_t at = rows + odd * (64 * 128) + (((4 * (quarter & 1) + 2 * odd) ^ (row & 7)) << 4);
        const uint32_t at_last = rows + 8 * (64 * 128) + (((2 * quarter) ^ (row & 7)) << 4);
        bool ok = true;
        for (int u = 0; u < n_tiles && ok; ++u) {
#pragma unroll
            for (int g = 0; g < KG; ++g) {
                if (u > 0) ok = ok && warp_wait(sm, &sm.k_empty[g], (u - 1) & 1, p.status);
                if (!ok) break;
                if (g < 2) {
                    store_half(at + 4 * g * (64 * 128), odd, c[2 * g], sc[2 * g]);
                    store_half(at + (4 * g + 2) * (64 * 128), odd, c[2 * g + 1], sc[2 * g + 1]);
                } else {
                    const uint32_t s2 = q4::dup_lo(q4::e4m3x2_to_f16(sc[4]));
                    store_unit(at_last, c_last.x, s2);
                    store_unit(at_last ^ 16, c_last.y, s2);
                }
            }
            if (!ok) break;
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(full);
            load(pool_row_of(u + 1, pos1, slot1));
            slot1 = row_slot(p, b, pos2);
            pos1 = pos2;
            pos2 = position(u + 3);
        }
    } else if (vwarp && n_tiles > 0) {
        // ------------------------------------------------ dequantise V, post the row masks
        const int row = 16 * w + (lane >> 2);
        const bool odd = quarter >> 1;
        const uint32_t full = map_to_rank(&sm.pv_full[w >> 2], 0);
        const uint32_t at = smem_addr(sm.v) + row * 128 + odd * (TILE * 128) + (((4 * (quarter & 1) + 2 * odd) ^ (row & 7)) << 4);
        bool ok = true;
        post_mask(0, row0);
        for (int u = 0; u < n_tiles && ok; ++u) {
            const int64_t next = pool_row_of(u + 1, pos1, slot1);
            if (u + 1 < n_tiles) post_mask(u + 1, next);
            if (u > 0) ok = warp_wait(sm, &sm.pv_done[w >> 2], (u - 1) & 1, p.status);
            if (!ok) break;
#pragma unroll
            for (int i = 0; i < 4; ++i)       // rows row and row + 8
                store_half(at + (i >> 1) * (2 * TILE * 128) + (i & 1) * 1024, odd, c[i], sc[i]);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(full);
            load(next);
            slot1 = row_slot(p, b, pos2);
            pos1 = pos2;
            pos2 = position(u + 3);
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
            if (ok) ok = wait_for(&sm.info_full[u % INFO], (u / INFO) & 1, &sm.abort_flag);
            uint32_t vm[2] = {0u, 0u};
            if (ok) {
                const uint32_t *m = reinterpret_cast<const uint32_t *>(&sm.mask[u % INFO][4 * half]);
                vm[0] = m[0];
                vm[1] = m[1];
            }
            if (ok) ok = wait_for(&sm.s_full[s], (u >> 1) & 1, &sm.abort_flag);
            if (!ok && *(volatile int *)&sm.abort_flag == 0) set_abort(sm, p.status);
            __syncwarp();
            tc_fence_after();
            // Two passes over S (maximum, then weights), 32 columns at a time: 64 scores at once
            // would not fit the registers of 24 warps.  The factor is positive, so the
            // maximum of the raw products is the scores', and m_ref is a raw product (see score_factor).
            uint32_t raw[32];
            auto fetch = [&](int q) {
                tmem_ld32(tmem + lane_base + TM_S + 64 * s + 32 * q, raw);
                tmem_wait_ld();
                if (vm[q] != 0xffffffffu) {      // uniform over the warp: absent rows in this unit
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (!((vm[q] >> i) & 1u)) raw[i] = 0xff800000u;
                }
            };
            float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
            for (int q = 0; q < 2; ++q) {
                fetch(q);
#pragma unroll
                for (int i = 0; i < 32; ++i) mx4[i & 3] = fmaxf(mx4[i & 3], __uint_as_float(raw[i]));
            }
            float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
            sm.red[u & 1][L] = mx;
            __syncwarp();
            named_barrier(1, 128);
            mx = fmaxf(mx, sm.red[u & 1][L ^ 64]);
            const bool move = (mx - m_ref) * mul > q4::RESCALE;
            const float alpha = move ? ex2((m_ref - mx) * mul) : 1.f;      // 0 the first time (m_ref = -inf)
            if (move) {
                l *= alpha;
                m_ref = mx;
            }
            // O may only be rescaled once both units' P V of tile u - 1 are done.  tcgen05.ld / st are
            // warp-collective: the whole warp rescales when any of its rows moves.
            if (__any_sync(0xffffffffu, move) && u > 0) {
#pragma unroll 1
                for (int a = 0; a < 2; ++a) {
                    ok = ok && wait_for(&sm.pv_done[a], (u - 1) & 1, &sm.abort_flag);
                    if (!ok && *(volatile int *)&sm.abort_flag == 0) set_abort(sm, p.status);
                }
                __syncwarp();          // lanes wait for themselves; what follows takes converged warps
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
                tc_fence_before();
            }
            const float ref = m_ref == -INFINITY ? 0.f : m_ref;
            // P V of tile u over the other unit needs this warp's lanes of O rescaled, though not its P, so
            // the warp arrives for that unit too -- once P V of tile u - 1 over it is done: only then has the
            // barrier's phase of tile u begun (the peer CTA may be a tile behind).
            auto done = [&](int a) {
                if (ok) ok = wait_for(&sm.pv_done[a], (u - 1) & 1, &sm.abort_flag);
                if (!ok && *(volatile int *)&sm.abort_flag == 0) set_abort(sm, p.status);
                __syncwarp();          // the next columns are fetched by a converged warp
            };
            auto turn = [&](int a) {
                if (u > 0) done(a);
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(map_to_rank(&sm.pv_full[a], 0));
            };
            float psum[4] = {0.f, 0.f, 0.f, 0.f};
            uint8_t *prow = sm.p[half] + h * 128;
#pragma unroll 1
            for (int q = 0; q < 2; ++q) {
                fetch(q);
                uint32_t pk[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float p0 = ex2(fmaf(__uint_as_float(raw[2 * i]) - ref, mul, q4::P_SHIFT));
                    const float p1 = ex2(fmaf(__uint_as_float(raw[2 * i + 1]) - ref, mul, q4::P_SHIFT));
                    psum[i & 3] += p0 + p1;
                    pk[i] = q4::pack_f16x2(p0, p1);
                }
                if (q == 0) {
                    if (half == 1) turn(0);
                    if (u > 0) done(half);         // P of this unit is rewritten
                }
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    *reinterpret_cast<uint4 *>(prow + (((4 * q + c) ^ (h & 7)) << 4)) =
                        make_uint4(pk[4 * c], pk[4 * c + 1], pk[4 * c + 2], pk[4 * c + 3]);
            }
            l += (psum[0] + psum[1]) + (psum[2] + psum[3]);
            tc_fence_before();
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(map_to_rank(&sm.pv_full[half], 0));
            if (half == 0) turn(1);
            if constexpr (TWO) {
                // the second part, from the same S (its buffer is written again after P V of this tile)
#pragma unroll 1
                for (int q = 0; q < 2; ++q) {
                    fetch(q);
                    uint32_t pk[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float p0 = ex2(fmaf(__uint_as_float(raw[2 * i]) - ref, mul, q4::P_SHIFT));
                        const float p1 = ex2(fmaf(__uint_as_float(raw[2 * i + 1]) - ref, mul, q4::P_SHIFT));
                        pk[i] = q4::rest_f16x2(p0, p1, q4::pack_f16x2(p0, p1));
                    }
                    if (q == 0) {
                        if (ok) ok = wait_for(&sm.first_done[half], u & 1, &sm.abort_flag);
                        if (!ok && *(volatile int *)&sm.abort_flag == 0) set_abort(sm, p.status);
                        __syncwarp();
                    }
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        *reinterpret_cast<uint4 *>(prow + (((4 * q + c) ^ (h & 7)) << 4)) =
                            make_uint4(pk[4 * c], pk[4 * c + 1], pk[4 * c + 2], pk[4 * c + 3]);
                }
                tc_fence_before();
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(map_to_rank(&sm.rest_full[half], 0));
            }
        }
        // ---- epilogue: wait for the last P V, then write the partial
#pragma unroll 1
        for (int a = 0; a < 2 && n_tiles > 0 && ok; ++a) {
            ok = wait_for(&sm.pv_done[a], (n_tiles - 1) & 1, &sm.abort_flag);
            if (!ok && *(volatile int *)&sm.abort_flag == 0) set_abort(sm, p.status);
        }
        __syncwarp();
        tc_fence_after();
        named_barrier(1, 128);
        sm.red[0][L] = l;
        __syncwarp();
        named_barrier(1, 128);
        const float l_tot = l + sm.red[0][L ^ 64];
        const int head = HPC * (int)rank + h;
        const size_t part0 = ((size_t)b * p.n_splits + split) * p.Hq;
        if (half == 0 && head < p.Hq) {
            p.m_part[part0 + head] = n_tiles > 0 ? fmaf(m_ref, mul, -q4::P_SHIFT) : -INFINITY;
            p.l_part[part0 + head] = l_tot;
        }
    }

    // ---- epilogue of O, by the 16 warps that dequantised (four column blocks at a time)
    if (warp >= 8) {
        // Not pv_done: these warps do not wait for it tile by tile (K's never, V's only for their own unit), and a
        // parity that is asked for once the next phase is over as well reads as not yet done.
        if (n_tiles > 0) warp_wait(sm, &sm.mma_done, 0, p.status);
        tc_fence_after();
        // O leaves tensor memory 32 columns at a time and passes through shared memory (the K buffer, free now),
        // so that every store instruction writes whole 128-byte row pieces.
        float *xbuf = reinterpret_cast<float *>(sm.k) + (warp - 8) * 1024;
        const uint32_t lane_base = (uint32_t)(32 * (warp & 3)) << 16;
        const int half = (warp & 3) >> 1;                      // lanes 64..127 hold the second half of the columns
        const int head0 = HPC * (int)rank + (32 * (warp & 3) & 63);
        const size_t part0 = ((size_t)b * p.n_splits + split) * p.Hq;
#pragma unroll 1
        for (int q = (warp - 8) >> 2; q < 8; q += 4) {
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
    __syncwarp();
    __syncthreads();
    if (warp == 2 && n_tiles > 0) {
        if (lane == 0 && !wait_for(&sm.mma_done, 0, nullptr)) set_abort(sm, p.status);
        __syncwarp();
    }
    cluster_sync();
    if (warp == 2) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, TM_COLS);
        tmem_relinquish_pair();
    }
}

// Splits per sequence: one CTA pair each, all co-resident; a single sequence takes half the pairs.  Both sides of
// that, one sequence of 128 heads, half and all: 10K rows 23.9 and 24.6 us, 32K 34.1 and 31.0, 128K 84.9 and 56.2.
int splits(int B, int max_units) {
    const int clusters = sm_count() / 2, tiles = (max_units + 1) / 2;
    return max(1, min(min(clusters / max(B, 1), clusters / 2), tiles));
}

template <bool TWO>
static int launch_parts(const DecodeParams &p, int B, cudaStream_t stream) {
    const size_t smem = sizeof(Smem) + 1024;
    static std::atomic<uint64_t> done{0};
    if (int rc = allow_shared(q4_mla_kernel<TWO>, (int)smem, done)) return rc;
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
    LSA_CUDA(cudaLaunchKernelEx(&cfg, q4_mla_kernel<TWO>, p, take_test_stall(LSA_TEST_STALL_ATTENTION_Q4)));
    return LSA_OK;
}
int launch(const DecodeParams &p, int B, cudaStream_t stream) {
    return q4::two_parts(p.out_dtype) ? launch_parts<true>(p, B, stream) : launch_parts<false>(p, B, stream);
}

}  // namespace q4mla
}  // namespace lsa
