// kv_pages.hip -- block tables, slots and positions of a step, for gfx950.
//
// Three running sums over the sequences carry the whole step: of rows appended
// (q_start), of pages taken, of pages given back. With them every output is a
// function of its own index: row r belongs to the sequence that a binary search
// over the first finds, the n-th page taken to the one that a search over the
// second finds, and the page it gets is the n-th given back (a search over the
// third) or an entry of the list. So one launch does it, without an order between
// workgroups: each one computes the sums for itself, in LDS (2 KB of lengths
// for 128 sequences, from L2), and then its share of the rows and pages.
//
// In place, without a race: what a call writes (table entries past the held ones of
// growing sequences, list entries at and past the count) no workgroup of it
// reads; what all of them read (lens, held, the count) is written by the last
// workgroup to finish, which an arrival counter beside the count names.
//
// Bound by latency: two launches' worth of dependent loads (lengths, then table).
#include <hip/hip_runtime.h>

#include <algorithm>

#include "bitmap_spmm.h"
#include "device_common.h"

namespace {

#define PG_BLOCK 256
#define PG_WAVES (PG_BLOCK / BSP_WAVE)
#define PG_ROWS 4            // rows a thread, so that long calls reach few workgroups
#define PG_MAX_GRID 512

struct PgArgs {
    int32_t *table, *lens, *held, *free_pages;
    const int32_t *keep, *more;
    const uint64_t *mask;
    int64_t *slots;
    int32_t *positions, *sequences, *q_start, *kv_lens;
    int32_t n, width, shift, pool, rows;
};

// What a sequence asks for: its kept and new tokens, and the pages it holds, takes and gives back.
struct PgSeq {
    uint32_t kept, more, held;      // more: at most rows + 1
    uint32_t grow, shrink;
    bool fits;                      // its rows and its row of the table
};

// end: new tokens up to and with this sequence, at most rows + 1
__device__ __forceinline__ PgSeq pg_seq(const PgArgs &a, int b, uint32_t end) {
    PgSeq s;
    const uint32_t len = (uint32_t)min(max(a.lens[b], 0), a.width << a.shift);
    s.kept = a.keep == nullptr ? len : min((uint32_t)max(a.keep[b], 0), len);
    s.more = (uint32_t)min(max(a.more[b], 0), a.rows + 1);
    s.held = (uint32_t)min(max(a.held[b], 0), a.width);
    const uint32_t want = (s.kept + s.more + (1u << a.shift) - 1) >> a.shift;
    s.fits = s.more == 0 || (end <= (uint32_t)a.rows && want <= (uint32_t)a.width);
    s.grow = s.fits && want > s.held ? want - s.held : 0;
    s.shrink = s.fits && want < s.held ? s.held - want : 0;
    return s;
}

// Inclusive running sums of v over the workgroup, from `carry` on, at most `most`
// (a sum cut off there is associative for values that are not negative).
__device__ __forceinline__ uint32_t pg_scan(uint32_t v, uint32_t carry, uint32_t most, uint32_t *sums) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const uint32_t o = (uint32_t)__shfl_up((int)v, d, 64);
        if (lane >= d) v = min(v + o, most);
    }
    if (lane == 63) sums[wave] = v;
    __syncthreads();
    uint32_t before = carry;
#pragma unroll
    for (int w = 0; w < PG_WAVES; ++w)
        if (w < wave) before = min(before + sums[w], most);
    __syncthreads();
    return min(v + before, most);
}

// The first b with end[b] > x (n when there is none).
__device__ __forceinline__ int pg_upper(const uint32_t *end, int n, uint32_t x) {
    int lo = 0, hi = n;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (end[mid] > x)
            hi = mid;
        else
            lo = mid + 1;
    }
    return lo;
}

__global__ __launch_bounds__(PG_BLOCK) void k_pages_step(const PgArgs a) {
    extern __shared__ uint32_t pg_lds[];
    __shared__ uint32_t sums[PG_WAVES];
    __shared__ int last;
    uint32_t *rows_end = pg_lds, *take_end = rows_end + a.n, *give_end = take_end + a.n;
    const int tid = threadIdx.x;
    uint32_t rows_sum = 0, take_sum = 0, give_sum = 0;
    for (int b0 = 0; b0 < a.n; b0 += PG_BLOCK) {
        const int b = b0 + tid;
        const bool in = b < a.n;
        const uint32_t more = in ? (uint32_t)min(max(a.more[b], 0), a.rows + 1) : 0;
        const uint32_t end = pg_scan(more, rows_sum, (uint32_t)a.rows + 1, sums);
        uint32_t grow = 0, shrink = 0;
        if (in) {
            const PgSeq s = pg_seq(a, b, end);
            grow = s.grow, shrink = s.shrink;
        }
        const uint32_t take = pg_scan(grow, take_sum, 0x7FFFFFFFu, sums);
        const uint32_t give = pg_scan(shrink, give_sum, 0x7FFFFFFFu, sums);
        if (in) rows_end[b] = end, take_end[b] = take, give_end[b] = give;
        __syncthreads();
        const int top = min(b0 + PG_BLOCK, a.n) - 1;
        rows_sum = rows_end[top], take_sum = take_end[top], give_sum = give_end[top];
    }
    const uint32_t count = (uint32_t)min(max(a.free_pages[0], 0), a.pool);
    int32_t *list = a.free_pages + 2;
    // pages taken by the sequences that need not wait: the running sum up to the first one that does
    const uint32_t have = count + give_sum;
    const int wait = pg_upper(take_end, a.n, have);
    const uint32_t taken = wait > 0 ? take_end[wait - 1] : 0;

    auto given = [&](uint32_t n) {      // the n-th page given back
        const int b = pg_upper(give_end, a.n, n);
        const PgSeq s = pg_seq(a, b, rows_end[b]);
        return a.table[(int64_t)b * a.width + (s.held - s.shrink) + (n - (give_end[b] - s.shrink))];
    };
    auto page_taken = [&](uint32_t n) { return n < give_sum ? given(n) : list[count - 1 - (n - give_sum)]; };

    const uint32_t me = blockIdx.x * PG_BLOCK + tid, all = gridDim.x * PG_BLOCK;
    for (uint32_t r = me; r < (uint32_t)a.rows; r += all) {
        const int b = pg_upper(rows_end, a.n, r);
        int64_t slot = -1;
        int32_t position = 0;
        if (b < a.n) {
            const PgSeq s = pg_seq(a, b, rows_end[b]);
            const uint32_t i = r - (b > 0 ? rows_end[b - 1] : 0), t = s.kept + i, p = t >> a.shift;
            if (s.fits && (s.grow == 0 || take_end[b] <= have)) {
                const int32_t page = p < s.held ? a.table[(int64_t)b * a.width + p]
                                                : page_taken(take_end[b] - s.grow + (p - s.held));
                slot = ((int64_t)page << a.shift) + (t & ((1u << a.shift) - 1));
            }
            position = (int32_t)t;
            if (a.mask != nullptr && a.more[b] <= BSP_TREE_MAX)
                position = (int32_t)s.kept + __popcll(a.mask[r] & ((UINT64_C(1) << i) - 1));
        }
        a.slots[r] = slot;
        a.positions[r] = position;
        a.sequences[r] = b < a.n ? b : -1;
    }
    for (uint32_t n = me; n < max(taken, give_sum); n += all) {
        if (n < taken) {
            const int b = pg_upper(take_end, a.n, n);
            const PgSeq s = pg_seq(a, b, rows_end[b]);
            a.table[(int64_t)b * a.width + s.held + (n - (take_end[b] - s.grow))] = page_taken(n);
        } else {
            const uint32_t at = have - 1 - n;
            if (at < (uint32_t)a.pool) list[at] = given(n);
        }
    }
    for (uint32_t b = me; b <= (uint32_t)a.n; b += all) {
        a.q_start[b] = (int32_t)min(b > 0 ? rows_end[b - 1] : 0, (uint32_t)a.rows);
        if (b < (uint32_t)a.n) {
            const PgSeq s = pg_seq(a, (int)b, rows_end[b]);
            const bool ok = s.fits && (s.grow == 0 || take_end[b] <= have);
            a.kv_lens[b] = ok ? (int32_t)(s.kept + s.more) : 0;
        }
    }
    // the last workgroup: every other has read all it needs
    __syncthreads();
    if (tid == 0) {
        __threadfence();
        last = atomicAdd(&a.free_pages[1], 1) == (int)gridDim.x - 1;
    }
    __syncthreads();
    if (!last) return;
    __threadfence();
    for (int b = tid; b < a.n; b += PG_BLOCK) {
        const PgSeq s = pg_seq(a, b, rows_end[b]);
        const bool ok = s.fits && (s.grow == 0 || take_end[b] <= have);
        a.lens[b] = (int32_t)(ok ? s.kept + s.more : s.kept);
        a.held[b] = (int32_t)(ok ? s.held + s.grow - s.shrink : s.held);
    }
    if (tid == 0) {
        a.free_pages[0] = (int32_t)min(have - taken, (uint32_t)a.pool);
        a.free_pages[1] = 0;
    }
}

}  // namespace

extern "C" int kv_pages_step(const bsp_kv_pages *pages, const int32_t *keep, const int32_t *new_tokens,
                             const uint64_t *tree_mask, int64_t rows, int64_t *slots, int32_t *positions,
                             int32_t *sequences, int32_t *q_start, int32_t *kv_lens, hipStream_t stream) {
    const bsp_kv_pages *p = pages;
    if (p == nullptr) return BSP_E_ARG;
    if (p->sequences < 0 || p->table_width < 0 || p->pool < 0 || rows < 0) return BSP_E_ARG;
    if (p->page_size < 16 || p->page_size > 4096 || (p->page_size & (p->page_size - 1)) != 0) return BSP_E_ARG;
    if (p->sequences > BSP_PAGES_MAX_SEQUENCES) return BSP_E_UNSUPPORTED;
    if (rows >= INT64_C(1) << 28) return BSP_E_OVERFLOW;
    if (p->table_width >= (INT32_MAX - 4095) / p->page_size) return BSP_E_OVERFLOW;
    if (p->pool > INT32_MAX || p->sequences * p->table_width + p->pool > INT32_MAX) return BSP_E_OVERFLOW;
    if (q_start == nullptr || p->free_pages == nullptr) return BSP_E_ARG;
    if (p->sequences > 0) {
        if (p->lens == nullptr || p->held == nullptr || new_tokens == nullptr || kv_lens == nullptr) return BSP_E_ARG;
        if (p->table_width > 0 && p->block_table == nullptr) return BSP_E_ARG;
    }
    if (rows > 0 && (slots == nullptr || positions == nullptr || sequences == nullptr)) return BSP_E_ARG;
    if ((((uintptr_t)p->block_table | (uintptr_t)p->lens | (uintptr_t)p->held | (uintptr_t)p->free_pages |
          (uintptr_t)keep | (uintptr_t)new_tokens | (uintptr_t)positions | (uintptr_t)sequences |
          (uintptr_t)q_start | (uintptr_t)kv_lens) & 3u) != 0)
        return BSP_E_ARG;
    if ((((uintptr_t)slots | (uintptr_t)tree_mask) & 7u) != 0) return BSP_E_ARG;
    PgArgs a{};
    a.table = p->block_table, a.lens = p->lens, a.held = p->held, a.free_pages = p->free_pages;
    a.keep = keep, a.more = new_tokens, a.mask = tree_mask;
    a.slots = slots, a.positions = positions, a.sequences = sequences, a.q_start = q_start, a.kv_lens = kv_lens;
    a.n = (int32_t)p->sequences, a.width = (int32_t)p->table_width, a.pool = (int32_t)p->pool, a.rows = (int32_t)rows;
    a.shift = __builtin_ctzll((unsigned long long)p->page_size);
    const int64_t work = std::max<int64_t>(rows, p->sequences);
    const unsigned grid = (unsigned)std::min<int64_t>(std::max<int64_t>((work + PG_BLOCK * PG_ROWS - 1) /
                                                                        (PG_BLOCK * PG_ROWS), 1), PG_MAX_GRID);
    hipLaunchKernelGGL(k_pages_step, dim3(grid), dim3(PG_BLOCK), (unsigned)(3 * 4 * p->sequences), stream, a);
    return hipGetLastError() == hipSuccess ? BSP_OK : BSP_E_HIP;
}
