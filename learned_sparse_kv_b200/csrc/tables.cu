// tables.cu -- chunk tables, slot maps and positions from request lengths, on the device.
//
// Request b has cached_len[b] tokens in the pool and brings new_len[b] more:
//   have = ceil(cached / 64), need = ceil((cached + new) / 64)
//   chunks c < have keep their slot, have <= c < need take the free slots (those that no kept
//   entry names) in ascending (b, c) and slot order, every other entry becomes -1, so the
//   slots of finished requests and of chunks past the length are free again.
// Token i of request b sits at position cached + i, in pool row slot * 64 + position % 64.
//
// The work is small (4 bytes a table entry); dependent lookups and launches are what it costs.  Up to 2M table
// entries and 2048 requests one cluster of 16 CTAs does everything in one launch, its phases
// separated by cluster barriers: clear the bitmap of used slots | mark the kept ones and copy their
// entries | count the free ones | give as many as are needed to the new chunks | write the maps.
// Larger problems use all multiprocessors: five launches (clear, mark, scan by one CTA, tables,
// maps).  32 requests of 16K to 512K tokens (1 MB of tables, 73K kept chunks): 14.4 to 15.2 us on the device
// (five launches: 14.5), of which the marks, one atomic a chunk on a bitmap in L2, take 5; 4096 requests, 1.05M
// kept chunks, five launches: 56 us.
#include <limits.h>

#include "block_scan.cuh"
#include "common.cuh"
#include "nvtx_range.cuh"

namespace lsa {
namespace tables {

constexpr int SCAN = 1024;

struct Params {
    const int32_t *table, *cached, *fresh;
    int32_t *next;
    int64_t *slot_map;
    int32_t *position, *offset, *n_free;
    int32_t *status;
    uint32_t *used;        // [words()]
    int32_t *chunk_base;   // [B + 1]: new chunks before request b
    int32_t *free_list;    // [min(n_slots, B * stride)]
    int B, stride, n_slots, max_new;
    __host__ __device__ int words() const { return (int)(((int64_t)n_slots + 31) / 32); }     // of the bitmap
};

// Lengths of request b, cut to the table: chunks to keep, chunks in all, cached and new tokens.
struct Lengths {
    int have, need, cached, fresh;
    bool bad, long_;
    __device__ Lengths(const Params &p, int b) {
        const int c = p.cached[b], f = p.fresh[b];
        const int64_t cap = (int64_t)p.stride * LSA_CHUNK;
        bad = c < 0 || f < 0;
        cached = max(c, 0);
        fresh = max(f, 0);
        long_ = (int64_t)cached + fresh > cap;
        fresh = min(fresh, INT_MAX - cached);   // positions stay below 2^31
        have = (int)lsa_min64((cached + (int64_t)LSA_CHUNK - 1) / LSA_CHUNK, p.stride);
        need = (int)lsa_min64(((int64_t)cached + fresh + LSA_CHUNK - 1) / LSA_CHUNK, p.stride);
    }
};

__global__ void __launch_bounds__(256) mark_kernel(const Params p) {
    const int b = blockIdx.y, c = blockIdx.x * 256 + threadIdx.x;
    if (c >= Lengths(p, b).have) return;
    const int s = p.table[(size_t)b * p.stride + c];
    if (s >= 0 && s < p.n_slots) atomicOr(&p.used[s >> 5], 1u << (s & 31));
    else flag(p.status, LSA_DEV_TABLE);
}

__global__ void __launch_bounds__(SCAN) scan_kernel(const Params p) {
    __shared__ int warp_tot[SCAN / 32 + 1];
    const int t = threadIdx.x;
    int chunks = 0;
    int64_t tokens = 0;
    for (int b0 = 0; b0 < p.B; b0 += SCAN) {
        const int b = b0 + t;
        int nc = 0;
        int64_t nt = 0;
        if (b < p.B) {
            const Lengths len(p, b);
            nc = len.need - len.have;
            nt = len.fresh;
            if (len.bad) flag(p.status, LSA_DEV_INDEX);
            if (len.long_) flag(p.status, LSA_DEV_CAPACITY);
        }
        int tot;
        const int rc = block_exclusive_scan<SCAN>(nc, warp_tot, &tot);
        if (b < p.B) p.chunk_base[b] = chunks + rc;
        chunks += tot;
        // token counts in two halves, so that no sum of up to 1024 counts passes 32 bits
        int tot_hi;
        const int64_t rt = block_exclusive_scan<SCAN>((int)(nt & 0xffff), warp_tot, &tot) +
                           ((int64_t)block_exclusive_scan<SCAN>((int)(nt >> 16), warp_tot, &tot_hi) << 16);
        if (b < p.B) p.offset[b] = (int)lsa_min64(tokens + rt, INT_MAX);
        tokens += tot + ((int64_t)tot_hi << 16);
    }
    if (t == 0) {
        p.chunk_base[p.B] = chunks;
        p.offset[p.B] = (int)lsa_min64(tokens, INT_MAX);
        if (tokens > p.max_new) flag(p.status, LSA_DEV_CAPACITY);
    }
    int free_ = 0;
    const int words = p.words();
    for (int w0 = 0; w0 < words; w0 += SCAN) {
        const int w = w0 + t;
        uint32_t bits = 0;
        if (w < words) {
            bits = ~p.used[w];
            if (w == words - 1 && (p.n_slots & 31)) bits &= (1u << (p.n_slots & 31)) - 1u;
        }
        int tot;
        int r = free_ + block_exclusive_scan<SCAN>(__popc(bits), warp_tot, &tot);
        while (bits && r < chunks) {
            p.free_list[r++] = 32 * w + __ffs(bits) - 1;
            bits &= bits - 1;
        }
        free_ += tot;
    }
    if (t == 0) {
        p.n_free[0] = max(free_ - chunks, 0);
        p.chunk_base[p.B + 1] = free_;
        if (free_ < chunks) flag(p.status, LSA_DEV_CAPACITY);
    }
}

// Slot of chunk c of request b in the next table.
__device__ __forceinline__ int slot_of(const Params &p, int b, int c, int have, int need, int n_free) {
    if (c < have) {
        const int s = p.table[(size_t)b * p.stride + c];
        return s >= 0 && s < p.n_slots ? s : -1;
    }
    if (c >= need) return -1;
    const int r = p.chunk_base[b] + c - have;
    return r < n_free ? p.free_list[r] : -1;
}

__global__ void __launch_bounds__(256) table_kernel(const Params p) {
    const int b = blockIdx.y, c = blockIdx.x * 256 + threadIdx.x;
    if (c >= p.stride) return;
    const Lengths len(p, b);
    p.next[(size_t)b * p.stride + c] = slot_of(p, b, c, len.have, len.need, p.chunk_base[p.B + 1]);
}

__global__ void __launch_bounds__(256) map_kernel(const Params p) {
    const int total = p.offset[p.B];
    for (int i = blockIdx.x * 256 + threadIdx.x; i < p.max_new; i += gridDim.x * 256) {
        int64_t slot = -1;
        int pos = -1;
        if (i < total) {
            int lo = 0, hi = p.B - 1;      // the last request whose offset is <= i
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (p.offset[mid] <= i) lo = mid;
                else hi = mid - 1;
            }
            const Lengths len(p, lo);
            pos = len.cached + (i - p.offset[lo]);
            const int s = slot_of(p, lo, pos / LSA_CHUNK, len.have, len.need, p.chunk_base[p.B + 1]);
            if (s >= 0) slot = (int64_t)s * LSA_CHUNK + pos % LSA_CHUNK;
        }
        p.slot_map[i] = slot;
        p.position[i] = pos;
    }
}

// ---- one cluster

constexpr int CL = 16, CL_THREADS = 1024, CL_REQUESTS = 2048, CL_ENTRIES = 1 << 21;
constexpr int ROW = 256;       // table entries of one warp's turn

__device__ __forceinline__ void cluster_barrier() {
    __syncwarp();           // the instructions take whole warps
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}
__device__ __forceinline__ uint32_t cta_of_cluster() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;\n" : "=r"(r));
    return r;
}
// Plain load from L2: the bitmap and the free list are written by other CTAs of the cluster.
__device__ __forceinline__ uint32_t load_l2(const uint32_t *p) { return __ldcg(p); }

__global__ void __launch_bounds__(CL_THREADS, 1) cluster_kernel(const Params p) {
    __shared__ int warp_tot[CL_THREADS / 32 + 1];
    __shared__ int free_of[CL];
    // of each request: new chunks and new tokens before it, chunks it keeps, tokens it has
    __shared__ int base[CL_REQUESTS + 1], first_token[CL_REQUESTS + 1], have[CL_REQUESTS], cached[CL_REQUESTS];
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const int rank = (int)cta_of_cluster(), gt = rank * CL_THREADS + t;
    constexpr int ALL = CL * CL_THREADS, WARPS = ALL / 32;
    const int gw = warp * CL + rank;      // neighbouring turns go to different CTAs
    const int words = p.words();
    for (int w = gt; w < words; w += ALL) p.used[w] = 0u;
    // every CTA scans the requests for itself
    int chunks = 0;
    int64_t tokens = 0;
    for (int b0 = 0; b0 < p.B; b0 += CL_THREADS) {
        const int b = b0 + t;
        int nc = 0;
        int64_t nt = 0;
        if (b < p.B) {
            const Lengths len(p, b);
            nc = len.need - len.have;
            nt = len.fresh;
            have[b] = len.have;
            cached[b] = len.cached;
            if (rank == 0 && len.bad) flag(p.status, LSA_DEV_INDEX);
            if (rank == 0 && len.long_) flag(p.status, LSA_DEV_CAPACITY);
        }
        int tot, tot_hi;
        const int rc = block_exclusive_scan<CL_THREADS>(nc, warp_tot, &tot);
        if (b < p.B) base[b] = chunks + rc;
        chunks += tot;
        const int lo = block_exclusive_scan<CL_THREADS>((int)(nt & 0xffff), warp_tot, &tot);
        const int hi = block_exclusive_scan<CL_THREADS>((int)(nt >> 16), warp_tot, &tot_hi);
        if (b < p.B) first_token[b] = (int)lsa_min64(tokens + lo + ((int64_t)hi << 16), INT_MAX);
        tokens += tot + ((int64_t)tot_hi << 16);
    }
    if (t == 0) {
        base[p.B] = chunks;
        first_token[p.B] = (int)lsa_min64(tokens, INT_MAX);
    }
    cluster_barrier();      // the bitmap is clear

    // Kept chunks: mark their slots and copy them; chunks past the need: -1.  (New ones follow.)
    const int turns = (p.stride + ROW - 1) / ROW;      // of a warp along one table row
    for (int item = gw; item < p.B * turns; item += WARPS) {
        const int b = item / turns, c0 = (item - b * turns) * ROW + lane;
        const int keep = have[b], need = keep + base[b + 1] - base[b];
        const int32_t *row = p.table + (size_t)b * p.stride;
        int32_t *next = p.next + (size_t)b * p.stride;
        int s[ROW / 32];
#pragma unroll
        for (int i = 0; i < ROW / 32; ++i) s[i] = c0 + 32 * i < keep ? __ldg(row + c0 + 32 * i) : -1;
#pragma unroll
        for (int i = 0; i < ROW / 32; ++i) {
            const int c = c0 + 32 * i;
            if (c >= p.stride || (c >= keep && c < need)) continue;
            if (s[i] >= 0 && s[i] < p.n_slots) {
                atomicOr(&p.used[s[i] >> 5], 1u << (s[i] & 31));
            } else {
                if (c < keep) flag(p.status, LSA_DEV_TABLE);
                s[i] = -1;
            }
            next[c] = s[i];
        }
    }
    cluster_barrier();      // every kept slot is marked

    // Free slots: each CTA counts its part of the bitmap, then gives those whose rank is needed to the new chunks.
    const int per_cta = (words + CL - 1) / CL, w_lo = min(rank * per_cta, words), w_hi = min(w_lo + per_cta, words);
    auto free_bits = [&](int w) -> uint32_t {
        uint32_t bits = ~load_l2(p.used + w);
        if (w == words - 1 && (p.n_slots & 31)) bits &= (1u << (p.n_slots & 31)) - 1u;
        return bits;
    };
    int mine = 0;
    for (int w = w_lo + t; w < w_hi; w += CL_THREADS) mine += __popc(free_bits(w));
    int cta_free;
    block_exclusive_scan<CL_THREADS>(mine, warp_tot, &cta_free);
    if (t < CL) {
        uint32_t remote;
        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(remote) : "r"(smem_addr(&free_of[rank])), "r"(t));
        asm volatile("st.shared::cluster.s32 [%0], %1;\n" ::"r"(remote), "r"(cta_free) : "memory");
    }
    cluster_barrier();      // the counts are everywhere
    int before = 0, n_free = 0;
#pragma unroll
    for (int r = 0; r < CL; ++r) {
        if (r < rank) before += free_of[r];
        n_free += free_of[r];
    }
    // the last request whose first item is <= i, of B + 1 ascending entries
    auto find = [&](const int *first, int i) {
        int lo = 0, hi = p.B - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (first[mid] <= i) lo = mid;
            else hi = mid - 1;
        }
        return lo;
    };
    auto give = [&](int r, int slot) {      // new chunk of rank r
        const int b = find(base, r);
        p.next[(size_t)b * p.stride + have[b] + r - base[b]] = slot;
    };
    // eight slots a thread: few enough that no thread gives many in a row
    for (int u0 = 4 * w_lo; u0 < 4 * w_hi && before < chunks; u0 += CL_THREADS) {
        const int u = u0 + t;
        uint32_t bits = u < 4 * w_hi ? (free_bits(u >> 2) >> (8 * (u & 3))) & 0xffu : 0u;
        int tot;
        int r = before + block_exclusive_scan<CL_THREADS>(__popc(bits), warp_tot, &tot);
        while (bits && r < chunks) {
            give(r++, 8 * u + __ffs(bits) - 1);
            bits &= bits - 1;
        }
        before += tot;
    }
    for (int64_t r = (int64_t)n_free + gt; r < chunks; r += ALL) give((int)r, -1);      // past 2^31 at the largest pools
    if (gt == 0) {
        p.n_free[0] = max(n_free - chunks, 0);
        if (n_free < chunks || tokens > p.max_new) flag(p.status, LSA_DEV_CAPACITY);
    }
    for (int b = gt; b <= p.B; b += ALL) p.offset[b] = first_token[b];
    if (p.max_new == 0) return;             // uniform
    cluster_barrier();      // the next tables are written

    const int total = first_token[p.B];
    for (int i0 = gt; i0 < p.max_new; i0 += 4 * ALL) {
        int pos[4], s[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int i = i0 + j * ALL;
            pos[j] = s[j] = -1;
            if (i < total && i < p.max_new) {
                const int b = find(first_token, i);
                pos[j] = cached[b] + (i - first_token[b]);
                if (pos[j] / LSA_CHUNK < p.stride) s[j] = __ldcg(p.next + (size_t)b * p.stride + pos[j] / LSA_CHUNK);
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int i = i0 + j * ALL;
            if (i >= p.max_new) break;
            p.slot_map[i] = s[j] >= 0 ? (int64_t)s[j] * LSA_CHUNK + pos[j] % LSA_CHUNK : -1;
            p.position[i] = pos[j];
        }
    }
}

static int launch_cluster(const Params &p, cudaStream_t stream) {
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    LSA_CUDA(cudaGetDevice(&dev));
    if (!(done.load(std::memory_order_relaxed) >> (dev & 63) & 1)) {     // 16 CTAs: more than the portable size
        LSA_CUDA(cudaFuncSetAttribute(cluster_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1));
        done.fetch_or(1ull << (dev & 63), std::memory_order_relaxed);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(CL, 1, 1);
    cfg.blockDim = dim3(CL_THREADS, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = CL;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    LSA_CUDA(cudaLaunchKernelEx(&cfg, cluster_kernel, p));
    return LSA_OK;
}

static size_t carve(Carver &c, Params &p) {
    p.used = c.take<uint32_t>(p.words());
    p.chunk_base = c.take<int32_t>(p.B + 2);
    p.free_list = c.take<int32_t>(lsa_min64(p.n_slots, (int64_t)p.B * p.stride));
    return align_up(c.used, 256);
}

}  // namespace tables
}  // namespace lsa

using namespace lsa;

extern "C" size_t lsa_build_tables_workspace_size(int B, int table_stride, int64_t n_slots) {
    if (B < 1 || table_stride < 1 || n_slots < 1 || n_slots >= (1ll << 31)) return 0;
    tables::Params p = {};
    p.B = B; p.stride = table_stride; p.n_slots = (int)n_slots;
    Carver c(nullptr);
    return tables::carve(c, p);
}

extern "C" int lsa_build_tables(const int32_t *table, int table_stride, const int32_t *cached_len,
                                const int32_t *new_len, int B, int64_t n_slots, int max_new, int32_t *table_next,
                                int64_t *slot_map, int32_t *position, int32_t *new_offset, int32_t *n_free,
                                int32_t *dev_status, void *ws, size_t ws_bytes, lsa_stream_t stream) {
    LSA_ABI_RANGE();
    LSA_REQUIRE(B >= 1 && B <= 65535 && table_stride >= 1 && table_stride < (1 << 25) && n_slots >= 1 &&
                    n_slots < (1ll << 31) && max_new >= 0 && max_new < (1 << 30),
                LSA_ERR_INVALID_ARG, "lsa_build_tables: bad sizes (B=%d table_stride=%d n_slots=%lld max_new=%d)", B,
                table_stride, (long long)n_slots, max_new);
    LSA_REQUIRE(table && cached_len && new_len && table_next && new_offset && n_free &&
                    (max_new == 0 || (slot_map && position)),
                LSA_ERR_INVALID_ARG, "lsa_build_tables: null pointer");
    LSA_REQUIRE((int64_t)B * table_stride < (1ll << 31), LSA_ERR_INVALID_ARG,
                "lsa_build_tables: a table of %lld entries (less than 2^31)", (long long)B * table_stride);
    LSA_REQUIRE(table + (size_t)B * table_stride <= table_next || table_next + (size_t)B * table_stride <= table,
                LSA_ERR_INVALID_ARG, "lsa_build_tables: table_next must not be table or overlap it");
    const size_t need = lsa_build_tables_workspace_size(B, table_stride, n_slots);
    LSA_REQUIRE(ws && ws_bytes >= need, LSA_ERR_WORKSPACE, "lsa_build_tables: workspace of %zu bytes, %zu needed",
                ws_bytes, need);
    LSA_REQUIRE((reinterpret_cast<uintptr_t>(ws) & 15) == 0, LSA_ERR_WORKSPACE, "lsa_build_tables: workspace not 16-byte aligned");
    tables::Params p = {};
    p.table = table; p.cached = cached_len; p.fresh = new_len; p.next = table_next; p.slot_map = slot_map;
    p.position = position; p.offset = new_offset; p.n_free = n_free; p.status = dev_status;
    p.B = B; p.stride = table_stride; p.n_slots = (int)n_slots; p.max_new = max_new;
    Carver c(ws);
    tables::carve(c, p);
    if (B <= tables::CL_REQUESTS && (int64_t)B * table_stride <= tables::CL_ENTRIES) {
        return tables::launch_cluster(p, stream);
    }
    LSA_CUDA(cudaMemsetAsync(p.used, 0, (size_t)p.words() * 4, stream));
    const dim3 grid((table_stride + 255) / 256, B);
    tables::mark_kernel<<<grid, 256, 0, stream>>>(p);
    tables::scan_kernel<<<1, tables::SCAN, 0, stream>>>(p);
    tables::table_kernel<<<grid, 256, 0, stream>>>(p);
    if (max_new > 0) tables::map_kernel<<<min((max_new + 255) / 256, 8 * sm_count()), 256, 0, stream>>>(p);
    return check_launch("lsa_build_tables kernels");
}
