// tables.cu -- chunk tables, slot maps and positions from request lengths, on the device.
//
// Request b has cached_len[b] tokens in the pool and brings new_len[b] more:
//   have = ceil(cached / 64), need = ceil((cached + new) / 64)
//   chunks c < have keep their slot, have <= c < need take the free slots (those that no kept
//   entry names) in ascending (b, c) and slot order, every other entry becomes -1, so the
//   slots of finished requests and of chunks past the length are free again.
// Token i of request b sits at position cached + i, in pool row slot * 64 + position % 64.
//
// Three launches: mark the kept slots in a bitmap; one CTA scans the requests' chunk and token
// counts and lists the free slots; every table entry and every new token then finds its own
// value.  The work is small (4 bytes a table entry): the launches and their dependent
// lookups are what it costs.
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
    uint32_t *used;        // [ceil(n_slots / 32)]
    int32_t *chunk_base;   // [B + 1]: new chunks before request b
    int32_t *free_list;    // [min(n_slots, B * stride)]
    int B, stride, n_slots, max_new;
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
    const int words = (p.n_slots + 31) / 32;
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

static size_t carve(Carver &c, Params &p) {
    p.used = c.take<uint32_t>((p.n_slots + 31) / 32);
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
    LSA_REQUIRE(table != table_next, LSA_ERR_INVALID_ARG, "lsa_build_tables: table_next must not be table");
    const size_t need = lsa_build_tables_workspace_size(B, table_stride, n_slots);
    LSA_REQUIRE(ws && ws_bytes >= need, LSA_ERR_WORKSPACE, "lsa_build_tables: workspace of %zu bytes, %zu needed",
                ws_bytes, need);
    tables::Params p = {};
    p.table = table; p.cached = cached_len; p.fresh = new_len; p.next = table_next; p.slot_map = slot_map;
    p.position = position; p.offset = new_offset; p.n_free = n_free; p.status = dev_status;
    p.B = B; p.stride = table_stride; p.n_slots = (int)n_slots; p.max_new = max_new;
    Carver c(ws);
    tables::carve(c, p);
    LSA_CUDA(cudaMemsetAsync(p.used, 0, (size_t)(p.n_slots + 31) / 32 * 4, stream));
    const dim3 grid((table_stride + 255) / 256, B);
    tables::mark_kernel<<<grid, 256, 0, stream>>>(p);
    tables::scan_kernel<<<1, tables::SCAN, 0, stream>>>(p);
    tables::table_kernel<<<grid, 256, 0, stream>>>(p);
    if (max_new > 0) tables::map_kernel<<<min((max_new + 255) / 256, 8 * sm_count()), 256, 0, stream>>>(p);
    return check_launch("lsa_build_tables kernels");
}
