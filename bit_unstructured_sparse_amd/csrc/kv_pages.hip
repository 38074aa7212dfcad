// kv_pages.hip -- block tables, slots and positions of a step, for gfx950.
//
// Three running sums over the sequences carry the whole step: of rows appended
// (q_start), of pages taken, of pages given back. With them every output is a
// function of its own index: row r belongs to the sequence that a binary search
// over the first finds, the n-th page taken to the one that a search over the
// second finds, and the page it gets is the n-th given back (a search over the
// third) or an entry of the list. So one launch does it, without an order between
// workgroups: each one computes the sums for itself, into LDS (20 bytes a sequence),
// and then its share of the rows and pages.
//
// In place, without a race: what a call writes (table entries past the held ones of
// growing sequences, list entries at and past the count) no workgroup of it
// reads; what all of them read (lens, held, the count) is written by the last
// workgroup to finish, which an arrival counter beside the count names.
//
// Short calls are bound by latency: dependent trips to memory (lengths; a row's page; the state) beside an empty launch's
// 1.8 us. 32 sequences of one token 3.3 us (3.7 in a graph), in one workgroup. Several workgroups have the arrivals at
// one counter besides, and each computes the sums for itself: 256 with trees (7,700 rows) 5.1 us, 512 with prompts (62,000
// rows) 9.6, of which the rows' bytes are 0.3 (at most 256 workgroups: with 64 12.5, with 1024 11.2; with a fence before
// the arrival 16). Sequences are summed 256 at a time, about 1.5 us a time: one token each for 512 of them 6.3 us, for
// 1,024 9.3, for 4,096 26.6.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "bitmap_spmm.h"
#include "device_common.h"

namespace {

#define PG_BLOCK 256
#define PG_WAVES (PG_BLOCK / BSP_WAVE)
#define PG_MAX_GRID 256
#define PG_WAITS 0x80000000u      // beside a sequence's kept tokens: its rows or its row of the table do not fit

struct PgArgs {
    int32_t *table, *lens, *held, *free_pages;
    const int32_t *keep, *more;
    const uint64_t *mask;
    int64_t *slots;
    int32_t *positions, *sequences, *q_start, *kv_lens;
    int32_t n, width, shift, pool, rows;
};

// Inclusive running sums over the wavefront, cut off at `most` (sums of values that are not negative, cut off
// there, are associative). Lanes 1, 2, 4, 8 below in a row of 16, then the last lane of the rows below.
__device__ __forceinline__ uint32_t pg_wave_scan(uint32_t v, uint32_t most) {
#define PG_STEP(ctrl, rows) \
    v = min(v + (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, ctrl, rows, 0xF, false), most);
    PG_STEP(0x111, 0xF) PG_STEP(0x112, 0xF) PG_STEP(0x114, 0xF) PG_STEP(0x118, 0xF) PG_STEP(0x142, 0xA) PG_STEP(0x143, 0xC)
#undef PG_STEP
    return v;
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
    // of each sequence: the running sums of rows (cut off at rows + 1), pages taken and pages given back, with its
    // own; its kept tokens (and PG_WAITS); the pages it holds
    extern __shared__ uint32_t pg_lds[];
    __shared__ uint32_t row_sums[PG_WAVES], take_sums[PG_WAVES], give_sums[PG_WAVES];
    __shared__ int last;
    uint32_t *rows_end = pg_lds, *take_end = rows_end + a.n, *give_end = take_end + a.n, *kept_of = give_end + a.n,
             *held_of = kept_of + a.n;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const uint32_t count = (uint32_t)min(max(a.free_pages[0], 0), a.pool), most = (uint32_t)a.rows + 1;
    uint32_t rows_sum = 0, take_sum = 0, give_sum = 0;
    for (int b0 = 0; b0 < a.n; b0 += PG_BLOCK) {
        const int b = b0 + tid;
        uint32_t kept = 0, more = 0, held = 0;
        if (b < a.n) {
            const uint32_t len = (uint32_t)min(max(a.lens[b], 0), a.width << a.shift);
            kept = a.keep == nullptr ? len : min((uint32_t)max(a.keep[b], 0), len);
            more = min((uint32_t)max(a.more[b], 0), most);
            held = (uint32_t)min(max(a.held[b], 0), a.width);
        }
        uint32_t end = pg_wave_scan(more, most);
        if (lane == 63) row_sums[wave] = end;
        __syncthreads();
        for (int w = 0; w < PG_WAVES; ++w) {
            if (w < wave) end = min(end + row_sums[w], most);
        }
        end = min(end + rows_sum, most);
        const uint32_t want = (kept + more + (1u << a.shift) - 1) >> a.shift;
        const bool fits = more == 0 || (end <= (uint32_t)a.rows && want <= (uint32_t)a.width);
        uint32_t take = pg_wave_scan(fits && want > held ? want - held : 0, 0x7FFFFFFFu);
        uint32_t give = pg_wave_scan(fits && want < held ? held - want : 0, 0x7FFFFFFFu);
        if (lane == 63) take_sums[wave] = take, give_sums[wave] = give;
        __syncthreads();
        for (int w = 0; w < PG_WAVES; ++w) {
            if (w < wave) take += take_sums[w], give += give_sums[w];
            rows_sum = min(rows_sum + row_sums[w], most);
        }
        if (b < a.n) {
            rows_end[b] = end, take_end[b] = take_sum + take, give_end[b] = give_sum + give;
            kept_of[b] = fits ? kept : kept | PG_WAITS, held_of[b] = held;
        }
        for (int w = 0; w < PG_WAVES; ++w) take_sum += take_sums[w], give_sum += give_sums[w];
        __syncthreads();
    }
    int32_t *list = a.free_pages + 2;
    // pages taken: all that are asked for, or those up to the first sequence that takes more than there are
    const uint32_t have = count + give_sum;
    uint32_t taken = take_sum;
    if (taken > have) {
        const int wait = pg_upper(take_end, a.n, have);
        taken = wait > 0 ? take_end[wait - 1] : 0;
    }
    auto before = [](const uint32_t *end, int b) { return b > 0 ? end[b - 1] : 0u; };
    auto goes = [&](int b) {      // whether the sequence need not wait
        return (kept_of[b] & PG_WAITS) == 0 && (take_end[b] <= have || take_end[b] == before(take_end, b));
    };
    auto given = [&](uint32_t n) {      // the n-th page given back
        const int b = pg_upper(give_end, a.n, n);
        return a.table[(int64_t)b * a.width + held_of[b] - (give_end[b] - n)];
    };
    auto page_taken = [&](uint32_t n) { return n < give_sum ? given(n) : list[count - 1 - (n - give_sum)]; };

    const uint32_t me = blockIdx.x * PG_BLOCK + tid, all = gridDim.x * PG_BLOCK;
    for (uint32_t r = me; r < (uint32_t)a.rows; r += all) {
        const int b = pg_upper(rows_end, a.n, r);
        int64_t slot = -1;
        int32_t position = 0;
        if (b < a.n) {
            const uint32_t kept = kept_of[b] & ~PG_WAITS, i = r - before(rows_end, b), t = kept + i, p = t >> a.shift;
            position = (int32_t)t;
            if (a.mask != nullptr && a.more[b] <= BSP_TREE_MAX)
                position = (int32_t)kept + __popcll(a.mask[r] & ((UINT64_C(1) << i) - 1));
            if (goes(b)) {
                const int32_t page = p < held_of[b] ? a.table[(int64_t)b * a.width + p]
                                                    : page_taken(before(take_end, b) + (p - held_of[b]));
                slot = ((int64_t)page << a.shift) + (t & ((1u << a.shift) - 1));
            }
        }
        a.slots[r] = slot;
        a.positions[r] = position;
        a.sequences[r] = b < a.n ? b : -1;
    }
    // pages, from the last thread down: short calls have them beside the rows
    for (uint32_t n = all - 1 - me; n < max(taken, give_sum); n += all) {
        if (n < taken) {
            const int b = pg_upper(take_end, a.n, n);
            a.table[(int64_t)b * a.width + held_of[b] + (n - before(take_end, b))] = page_taken(n);
        } else {
            const uint32_t at = have - 1 - n;
            if (at < (uint32_t)a.pool) list[at] = given(n);
        }
    }
    auto length = [&](int b) { return (int32_t)((kept_of[b] & ~PG_WAITS) + rows_end[b] - before(rows_end, b)); };
    for (uint32_t b = me; b <= (uint32_t)a.n; b += all) {
        a.q_start[b] = (int32_t)min(before(rows_end, (int)b), (uint32_t)a.rows);
        if (b < (uint32_t)a.n) a.kv_lens[b] = goes((int)b) ? length((int)b) : 0;
    }
    // the state, once every workgroup has read all it needs: by the last one. What was read has been used, in
    // stores or in LDS, before the barrier; nothing that another workgroup wrote is read, so no fence is needed
    __syncthreads();
    if (gridDim.x > 1) {
        if (tid == 0) last = atomicAdd(&a.free_pages[1], 1) == (int)gridDim.x - 1;
        __syncthreads();
        if (!last) return;
    }
    for (int b = tid; b < a.n; b += PG_BLOCK) {
        const bool ok = goes(b);
        a.lens[b] = ok ? length(b) : (int32_t)(kept_of[b] & ~PG_WAITS);
        a.held[b] = (int32_t)(ok ? held_of[b] + (take_end[b] - before(take_end, b)) - (give_end[b] - before(give_end, b))
                                 : held_of[b]);
    }
    if (tid == 0) {
        a.free_pages[0] = (int32_t)min(have - taken, (uint32_t)a.pool);
        a.free_pages[1] = 0;
    }
}

// Whether a result lies over an input, the state or another result: workgroups read the inputs while others write.
bool pg_overlap(const bsp_kv_pages *p, const int32_t *keep, const int32_t *more, const uint64_t *mask, int64_t rows,
                const int64_t *slots, const int32_t *positions, const int32_t *sequences, const int32_t *q_start,
                const int32_t *kv_lens) {
    struct {
        const void *at;
        int64_t bytes;
    } r[] = {{slots, rows * 8}, {positions, rows * 4}, {sequences, rows * 4}, {q_start, (p->sequences + 1) * 4},
             {kv_lens, p->sequences * 4},      // the results, then what must not be under them
             {keep, p->sequences * 4}, {more, p->sequences * 4}, {mask, rows * 8}, {p->lens, p->sequences * 4},
             {p->held, p->sequences * 4}, {p->block_table, p->sequences * p->table_width * 4},
             {p->free_pages, (p->pool + 2) * 4}};
    constexpr int ALL = sizeof r / sizeof r[0];
    for (int i = 0; i < 5; ++i)
        for (int j = i + 1; j < ALL; ++j) {
            if (r[i].at == nullptr || r[j].at == nullptr || r[i].bytes == 0 || r[j].bytes == 0) continue;
            const uintptr_t a = (uintptr_t)r[i].at, b = (uintptr_t)r[j].at;
            if (a < b + (uintptr_t)r[j].bytes && b < a + (uintptr_t)r[i].bytes) return true;
        }
    return false;
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
    if (pg_overlap(p, keep, new_tokens, tree_mask, rows, slots, positions, sequences, q_start, kv_lens)) return BSP_E_ARG;
    PgArgs a{};
    a.table = p->block_table, a.lens = p->lens, a.held = p->held, a.free_pages = p->free_pages;
    a.keep = keep, a.more = new_tokens, a.mask = tree_mask;
    a.slots = slots, a.positions = positions, a.sequences = sequences, a.q_start = q_start, a.kv_lens = kv_lens;
    a.n = (int32_t)p->sequences, a.width = (int32_t)p->table_width, a.pool = (int32_t)p->pool, a.rows = (int32_t)rows;
    a.shift = __builtin_ctzll((unsigned long long)p->page_size);
    const unsigned grid = (unsigned)std::min<int64_t>(std::max<int64_t>((rows + PG_BLOCK - 1) / PG_BLOCK, 1), PG_MAX_GRID);
    const unsigned lds = (unsigned)(5 * 4 * p->sequences);
    if (lds > 65536)
        (void)hipFuncSetAttribute((const void *)k_pages_step, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    hipLaunchKernelGGL(k_pages_step, dim3(grid), dim3(PG_BLOCK), lds, stream, a);
    return hipGetLastError() == hipSuccess ? BSP_OK : BSP_E_HIP;
}
