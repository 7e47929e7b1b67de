// ha_cache.cu -- the steps of the paged key/value cache: freeing, forking, reserving (with the copy of a shared last
// page), appending and committing (compacting) sequences.
//
// All state is in device memory (page table, lengths, pages held, reference counts), so no step waits for the host
// and all of them can be captured into a graph. A page is free when its reference count is 0; pages are taken
// lowest index first and in list order, so the same calls always give the same pages. Integer additions are the
// only atomics; their order changes nothing.
//
// What bounds these kernels: the row traffic (each row read once and written once, 16 bytes per thread) for large
// calls, launch latency and the chain of dependent loads (slot -> length -> page -> row) for small ones. All five steps for
// 64 branches of 8 prompts (drafts of up to 16, 32 layers, 8 heads, d = 128): 68 us against 38 to 41 us for the rows' bytes at
// the memory's rate; for two branches in one layer: 16.6 us, five launches.
#include "ha_common.cuh"
#include "ha_internal.h"
#include "ha_serve.cuh"

namespace ha {
namespace {

// True on every thread of the block when value v occurs in list[0 .. n).
__device__ __forceinline__ bool block_contains(const int32_t *list, int n, int32_t v) {
    bool hit = false;
    for (int j = threadIdx.x; j < n; j += blockDim.x) hit |= list[j] == v;
    return __syncthreads_or(hit);
}

// A page number out of range is reported and passed over: leaving the slot as it is would hold its other pages for good.
__global__ void __launch_bounds__(256) cache_free_kernel(const ServeCache c, const int32_t *slots, int *status) {
    grid_dependency_wait();
    const int i = blockIdx.x;
    const int32_t s = slots[i];
    const bool dup = block_contains(slots, i, s);
    if (s < 0 || s >= c.slots || dup) {
        if (threadIdx.x == 0) atomicOr(status, kStatusData);
        return;
    }
    const int held = c.held[s];
    if (held < 0 || held > c.max_pages) {
        if (threadIdx.x == 0) atomicOr(status, kStatusData);
        return;
    }
    int32_t *row = c.table + static_cast<int64_t>(s) * c.max_pages;
    for (int p = threadIdx.x; p < held; p += blockDim.x) {
        const int32_t id = row[p];
        if (id >= 0 && id < c.pages) atomicSub(c.refs + id, 1);
        else atomicOr(status, kStatusData);
        row[p] = -1;
    }
    __syncthreads();   // every thread has read held
    if (threadIdx.x == 0) {
        c.held[s] = 0;
        c.lens[s] = 0;
    }
}

// Sources are read as they were before the call: a source that is also a destination of the call is refused, and so is one whose
// row of the table names a page out of range.
__global__ void __launch_bounds__(256) cache_fork_kernel(const ServeCache c, const int32_t *src, const int32_t *dst, int n,
                                                         int *status) {
    grid_dependency_wait();
    const int i = blockIdx.x;
    const int32_t s = src[i], t = dst[i];
    bool bad = block_contains(dst, i, t);
    bad |= block_contains(dst, n, s);
    bad |= s < 0 || s >= c.slots || t < 0 || t >= c.slots;
    int len = 0, pages = 0;
    if (!bad) {
        len = c.lens[s];
        const int held = c.held[s];
        const int64_t need = (static_cast<int64_t>(len) + c.page - 1) >> c.page_shift;
        bad = len < 0 || need > held || held > c.max_pages || c.held[t] != 0 || c.lens[t] != 0;
        pages = bad ? 0 : static_cast<int>(need);
    }
    const int32_t *from = c.table + static_cast<int64_t>(s) * c.max_pages;
    for (int p = threadIdx.x; p < pages; p += blockDim.x) bad |= from[p] < 0 || from[p] >= c.pages;
    // from here on every thread has read the destination's length, which thread 0 writes
    if (__syncthreads_or(bad)) {
        if (threadIdx.x == 0) atomicOr(status, kStatusData);
        return;
    }
    int32_t *to = c.table + static_cast<int64_t>(t) * c.max_pages;
    for (int p = threadIdx.x; p < pages; p += blockDim.x) {
        const int32_t id = from[p];
        atomicAdd(c.refs + id, 1);
        to[p] = id;
    }
    if (threadIdx.x == 0) {
        c.lens[t] = len;
        c.held[t] = pages;
    }
}

// Workspace of a reserve call of n entries: per entry the running total of pages needed, the pages held before, the
// pages to copy (from, to; -1: none) and the rows to copy; then the list of free pages taken.
struct ReservePlan {
    int64_t *upto;     // pages needed by entries 0 .. i
    int32_t *last;     // page that entry i would append to (-1: none)
    int32_t *held;
    int32_t *from, *to, *rows;
    int32_t *ids;
};

__host__ __device__ inline ReservePlan reserve_plan(void *ws, int n) {
    ReservePlan p;
    p.upto = static_cast<int64_t *>(ws);
    p.last = reinterpret_cast<int32_t *>(p.upto + n);
    p.held = p.last + n;
    p.from = p.held + n;
    p.to = p.from + n;
    p.rows = p.to + n;
    p.ids = p.rows + n;
    return p;
}

constexpr int kPlanThreads = 1024;

// Inclusive sum over the block; *total gets the block's sum on every thread. scratch: 33 values.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t *scratch, int64_t *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();   // the previous call's readers are done
    if (lane == 31) scratch[warp] = x;
    __syncthreads();
    if (warp == 0) {
        int64_t w = scratch[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, w, o);
            if (lane >= o) w += y;
        }
        scratch[lane] = w;
    }
    __syncthreads();
    *total = scratch[31];
    return x + (warp ? scratch[warp - 1] : 0);
}

// The committed rows (`rows` of each head) of page `from` go to page `to`, in one layer of k or v; THREADS threads take part.
template <int THREADS>
__device__ __forceinline__ void copy_page(const ServeCache &c, int esz, char *base, int64_t layer, int from, int to, int rows) {
    const int64_t row_bytes = static_cast<int64_t>(c.d) * esz, head_bytes = row_bytes * c.page,
                  page_bytes = head_bytes * c.kv_heads;
    const char *src = base + (layer * c.pages + from) * page_bytes;
    char *dst = base + (layer * c.pages + to) * page_bytes;
    const int per_head = static_cast<int>(rows * row_bytes / 16);
    const int total = per_head * c.kv_heads;
    for (int x0 = threadIdx.x; x0 < total; x0 += THREADS * 4) {
        int4 buf[4];
        int64_t off[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int x = x0 + THREADS * u, h = x / per_head;
            off[u] = h * head_bytes + (x - h * per_head) * 16;
            if (x < total) buf[u] = *reinterpret_cast<const int4 *>(src + off[u]);
        }
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (x0 + THREADS * u < total) *reinterpret_cast<int4 *>(dst + off[u]) = buf[u];
    }
}

// One block plans the call: what each entry needs, the lowest free pages, and who gets which. One block because the
// order matters (list order, lowest page first) and the data is small: the scan of the reference counts reads 16 of
// them per thread and stops as soon as enough free pages are found.
__global__ void __launch_bounds__(kPlanThreads) cache_reserve_plan_kernel(const ServeCache c, const int32_t *slots,
                                                                          const int32_t *add, int n, int32_t *granted,
                                                                          void *ws, int esz, bool copy, int *status) {
    grid_dependency_wait();
    __shared__ int64_t scratch[33];
    __shared__ int32_t slot_of[kPlanThreads], last_of[kPlanThreads];   // of 1024 entries at a time
    const ReservePlan p = reserve_plan(ws, n);
    const int tid = threadIdx.x;
    // the first reference counts, on their way while the entries are looked over
    const bool ahead = tid * 16 + 16 <= c.pages;
    int4 first_refs[4];
    if (ahead) {
#pragma unroll
        for (int q = 0; q < 4; ++q) first_refs[q] = *reinterpret_cast<const int4 *>(c.refs + tid * 16 + 4 * q);
    }
    // 1. what each entry would append to (an entry out of range, or a slot's second one, asks for nothing), and
    // 2. the pages it needs, in list order: a shared last page is copied by every entry but the last one that holds it
    int64_t carry = 0;
    for (int base = 0; base < n; base += kPlanThreads) {
        const int i = base + tid;
        const int32_t s = i < n ? slots[i] : -1;
        const int32_t want = i < n ? add[i] : 0;
        __syncthreads();   // the 1024 entries before have been read
        slot_of[tid] = s;
        __syncthreads();
        bool ok = i < n && s >= 0 && s < c.slots && want >= 0;
        int64_t len = 0, pages = 0;
        int held = -1, last = -1, shared = 0;
        if (ok) {
            len = c.lens[s];
            held = c.held[s];
            pages = (len + want + c.page - 1) >> c.page_shift;
            ok = len >= 0 && held >= 0 && held <= c.max_pages && ((len + c.page - 1) >> c.page_shift) <= held &&
                 pages <= c.max_pages;
            if (ok && (len & (c.page - 1)) != 0 && want > 0) {
                last = c.table[s * c.max_pages + (len >> c.page_shift)];
                ok = last >= 0 && last < c.pages;
                if (ok) shared = c.refs[last];
            }
        }
        for (int j = 0; ok && j < tid; ++j) ok = slot_of[j] != s;
        for (int j = 0; ok && j < base; ++j) ok = slots[j] != s;
        if (!ok) {
            last = held = -1;
            if (i < n) atomicOr(status, kStatusData);
        }
        last_of[tid] = last;
        if (i < n) {
            p.last[i] = last;
            p.held[i] = held;
        }
        __syncthreads();
        int64_t need = 0;
        int from = -1;
        if (ok) {
            need = pages > held ? pages - held : 0;
            if (last >= 0 && shared > 1) {
                for (int j = 0; j < tid; ++j) shared -= last_of[j] == last;
                for (int j = 0; j < base; ++j) shared -= p.last[j] == last;
                if (shared > 1) from = last;
            }
            need += from >= 0;
        }
        int64_t total;
        const int64_t sum = block_scan(need, scratch, &total);
        if (i < n) {
            p.from[i] = from;
            p.to[i] = -1;
            p.rows[i] = static_cast<int32_t>(len & (c.page - 1));
            p.upto[i] = carry + sum;
        }
        carry += total;
    }
    const int64_t wanted = carry < c.pages ? carry : c.pages;
    // 3. the lowest free pages
    int64_t found = 0;
    for (int64_t base = 0; base < c.pages && found < wanted; base += kPlanThreads * 16) {
        const int64_t first = base + tid * 16;
        unsigned free = 0;
        if (first + 16 <= c.pages) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int4 r = base == 0 ? first_refs[q] : *reinterpret_cast<const int4 *>(c.refs + first + 4 * q);
                free |= static_cast<unsigned>((r.x == 0) | (r.y == 0) << 1 | (r.z == 0) << 2 | (r.w == 0) << 3) << (4 * q);
            }
        } else {
            for (int q = 0; q < 16; ++q)
                if (first + q < c.pages && c.refs[first + q] == 0) free |= 1u << q;
        }
        int64_t total;
        int64_t at = found + block_scan(__popc(free), scratch, &total) - __popc(free);
        while (free && at < wanted) {
            p.ids[at++] = static_cast<int32_t>(first + __ffs(free) - 1);
            free &= free - 1;
        }
        found += total;
    }
    if (found > wanted) found = wanted;
    __syncthreads();
    // 4. a prefix of the list is served: the entries whose running total the free pages cover
    for (int i = tid; i < n; i += kPlanThreads) {
        const bool ok = p.held[i] >= 0 && p.upto[i] <= found;
        if (granted) granted[i] = ok ? add[i] : 0;
        if (!ok) p.from[i] = -1;
        if (ok) {
            const int32_t s = slots[i];
            const int64_t pages = (static_cast<int64_t>(c.lens[s]) + add[i] + c.page - 1) >> c.page_shift;
            if (pages > p.held[i]) c.held[s] = static_cast<int32_t>(pages);
        }
    }
    __syncthreads();
    for (int64_t t = tid; t < found; t += kPlanThreads) {
        int lo = 0, hi = n - 1;   // the entry that page t goes to: the first whose running total exceeds t
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (p.upto[mid] > t) hi = mid;
            else lo = mid + 1;
        }
        const int i = lo;
        if (p.upto[i] > found) continue;   // not served
        const int64_t start = i ? p.upto[i - 1] : 0;
        const int32_t s = slots[i], id = p.ids[t];
        int64_t j = t - start;
        int32_t *row = c.table + s * c.max_pages;
        c.refs[id] = 1;
        if (p.from[i] >= 0 && j == 0) {
            row[c.lens[s] >> c.page_shift] = id;
            atomicSub(c.refs + p.from[i], 1);
            p.to[i] = id;
        } else {
            j -= p.from[i] >= 0;
            row[p.held[i] + j] = id;
        }
    }
    // 5. few copies are made here, without a second launch
    if (copy) {
        __syncthreads();
        for (int i = 0; i < n; ++i)
            if (p.from[i] >= 0 && p.to[i] >= 0)
                for (int y = 0; y < 2 * static_cast<int>(c.layers); ++y)
                    copy_page<kPlanThreads>(c, esz, static_cast<char *>((y & 1) ? c.v : c.k), y >> 1, p.from[i], p.to[i], p.rows[i]);
    }
}

// One block per (entry, layer, k or v).
__global__ void __launch_bounds__(256) cache_reserve_copy_kernel(const ServeCache c, int esz, int n, void *ws) {
    grid_dependency_wait();
    const ReservePlan p = reserve_plan(ws, n);
    const int from = p.from[blockIdx.x], to = p.to[blockIdx.x];
    if (from < 0 || to < 0) return;
    copy_page<256>(c, esz, static_cast<char *>((blockIdx.y & 1) ? c.v : c.k), blockIdx.y >> 1, from, to, p.rows[blockIdx.x]);
}

struct AppendArgs {
    const char *k, *v;
    int64_t kl, kt, kh, vl, vt, vh;   // strides in bytes: layer, token, head
    int64_t layer, layers;
};

constexpr int kAppendLayers = 8;   // layers per block (4: 1.3% slower for a whole branch step of 32 layers, 16: as 8)

// Row t of the call goes to place `at` behind the committed rows of slot s, in up to kAppendLayers layers; the whole block
// takes part. dup: the slot was named before (two entries of a slot would write the same rows).
__device__ __forceinline__ void append_row(const ServeCache &c, int esz, const AppendArgs &a, int64_t t, int32_t s, int64_t place,
                                           bool dup, int *status) {
    bool ok = !dup && s >= 0 && s < c.slots;
    int32_t id = -1;
    int64_t at = 0;
    if (ok) {
        const int64_t len = c.lens[s], held = c.held[s];
        at = len + place;
        const int64_t pi = at >> c.page_shift;
        ok = len >= 0 && pi < held && held <= c.max_pages;
        if (ok) id = c.table[s * c.max_pages + pi];
    }
    if (id < 0 || id >= c.pages || c.refs[id] != 1) {   // a page that another slot shares is not written
        if (threadIdx.x == 0) atomicOr(status, kStatusData);
        return;
    }
    const int64_t row_bytes = static_cast<int64_t>(c.d) * esz, head_bytes = row_bytes * c.page,
                  page_bytes = head_bytes * c.kv_heads;
    const int64_t l0 = static_cast<int64_t>(blockIdx.y) * kAppendLayers;
    const int nl = static_cast<int>(min(static_cast<int64_t>(kAppendLayers), a.layers - l0));
    const int rows = 2 * nl * c.kv_heads;          // of k in all layers, then of v
    // a thread has one 16-byte piece of every (256 / pieces)-th row; pieces is 8, 16 or 32
    const int shift = 31 - __clz(static_cast<int>(row_bytes / 16));
    const int piece = (threadIdx.x & ((1 << shift) - 1)) * 16, step = 256 >> shift;
    const char *const k = a.k + l0 * a.kl + t * a.kt + piece, *const v = a.v + l0 * a.vl + t * a.vt + piece;
    const int64_t layer_bytes = c.pages * page_bytes;
    const int64_t off = (a.layer + l0) * layer_bytes + id * page_bytes + (at & (c.page - 1)) * row_bytes + piece;
    for (int r0 = threadIdx.x >> shift; r0 < rows; r0 += step * 4) {
        int4 buf[4];
        char *dst[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int r = r0 + step * u;
            dst[u] = nullptr;
            if (r >= rows) continue;
            const int y = r / c.kv_heads, h = r - y * c.kv_heads;
            const bool second = y >= nl;
            const int l = second ? y - nl : y;
            buf[u] = *reinterpret_cast<const int4 *>(second ? v + l * a.vl + h * a.vh : k + l * a.kl + h * a.kh);
            dst[u] = static_cast<char *>(second ? c.v : c.k) + l * layer_bytes + h * head_bytes + off;
        }
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (dst[u]) *reinterpret_cast<int4 *>(dst[u]) = buf[u];
    }
}

// Sequences of a long list, whose blocks take kAppendEach tokens each.
constexpr int kAppendMany = 4096, kAppendEach = 8;

// One block per token and group of layers: the sequences that hold the token are looked up, then the rows are copied.
//
// A list in order (ascending rows of the call) has one such sequence, or none for rows in front of the first and behind the
// last. In a list with a fault two sequences that are both in range may share rows: each of them gets them, and those that are
// not rows of the call are left out and reported. Every block looks the whole list over, a thread per sequence. That costs
// nothing beside the copies for a few hundred sequences (256 of one token, one layer, 8 heads, d = 128: 6.2 us, 1024: 6.6) and
// is the bound for many, so a long list is looked over for its order only, once for several tokens, and bisected for each
// (16384: 134 us, and 229 us the other way).
template <bool MANY>
__global__ void __launch_bounds__(256) cache_append_kernel(const ServeCache c, int esz, const int32_t *slots,
                                                           const int32_t *cu, int n, int64_t tokens, const AppendArgs a,
                                                           int *status) {
    grid_dependency_wait();
    __shared__ int first;
    const int last = static_cast<int>(tokens);     // at most 2^30
    const bool few = !MANY && n <= 256;
    const int32_t slot = few && threadIdx.x < n ? slots[threadIdx.x] : 0;   // on its way for the search for a second entry
    bool ordered = false;
    if (MANY) {
        bool down = cu[0] < 0 || cu[n] > last;
#pragma unroll 8
        for (int i = static_cast<int>(threadIdx.x); i < n; i += 256) down |= cu[i + 1] < cu[i];
        ordered = !__syncthreads_or(down);
    }
    int t = static_cast<int>(blockIdx.x) * (MANY ? kAppendEach : 1);
    const int end = MANY ? min(last, t + kAppendEach) : t + 1;
    for (int from = 0; t < end;) {
        int at = n;                                // the first sequence from `from` on that holds t
        bool more = false;                         // others do, too
        if (MANY && ordered) {
            int lo = 0;
            while (lo < at) {
                const int mid = (lo + at) >> 1;
                if (cu[mid + 1] > t) at = mid;
                else lo = mid + 1;
            }
            if (t < cu[0]) at = n;
        } else {
            if (threadIdx.x == 0) first = n;
            __syncthreads();
            int found = 0, mine = n;
            bool bad = false;
#pragma unroll 4
            for (int i = from + static_cast<int>(threadIdx.x); i < n; i += 256) {
                const int s = cu[i], e = cu[i + 1];
                const bool ok = s >= 0 && e >= s && e <= last;
                if (ok && s <= t && t < e) {
                    mine = min(mine, i);
                    ++found;
                }
                bad |= !ok;
            }
            if (found) atomicMin(&first, mine);
            if (bad && blockIdx.x == 0 && blockIdx.y == 0) atomicOr(status, kStatusData);
            more = __syncthreads_count(found) > 1;
            if (!few) more |= __syncthreads_or(found > 1);
            at = first;
        }
        if (at < n) {
            const int32_t s = slots[at];
            const bool dup = few ? __syncthreads_or(threadIdx.x < at && slot == s) : block_contains(slots, at, s);
            append_row(c, esz, a, t, s, t - cu[at], dup, status);
        }
        if (!MANY && !more) return;
        from = more ? at + 1 : 0;
        t += !more;
        __syncthreads();   // every thread has read `first`
    }
}

// Whether entry i of a commit is valid; the whole block takes part. *len, *held, *count of the slot.
__device__ bool commit_entry(const ServeCache &c, const int32_t *slots, const int32_t *counts, const int32_t *keep,
                             int64_t max_keep, int i, int *len, int *held, int *count) {
    const int32_t s = slots[i];
    bool bad = block_contains(slots, i, s) || s < 0 || s >= c.slots;
    if (bad) return false;
    *len = c.lens[s];
    *held = c.held[s];
    *count = counts[i];
    const int64_t room = static_cast<int64_t>(*held) * c.page - *len;
    if (*len < 0 || *held < 0 || *held > c.max_pages || *count < 0 || *count > room || (keep && *count > max_keep))
        return false;
    if (keep) {
        const int32_t *mine = keep + i * max_keep;
        for (int j = threadIdx.x; j < *count; j += blockDim.x) {
            const int32_t x = mine[j];
            bad |= x < 0 || x >= room || (j > 0 && x <= mine[j - 1]);
        }
    }
    // the pages that rows are read from and written to; none that another slot shares is written
    const int32_t *row = c.table + s * c.max_pages;
    const int written = keep && *count > 0 ? (*len + *count + c.page - 1) >> c.page_shift : 0;
    for (int p = (*len >> c.page_shift) + threadIdx.x; p < *held; p += blockDim.x) {
        const int32_t id = row[p];
        const bool out = id < 0 || id >= c.pages;
        bad |= out || (p < written && c.refs[id] != 1);
    }
    return !__syncthreads_or(bad);
}

constexpr int kMoveChunk = 256;   // kept rows staged at a time

// The kept rows of a draft move to the front of it, in one layer of k and v: row len + keep[i] -> len + i. keep is ascending,
// so keep[i] >= i and a row is read before a later row is written over it; every thread moves its own 16-byte column in
// ascending order, eight rows in flight.
__device__ __forceinline__ void move_rows(const ServeCache &c, int esz, int64_t layer, const int32_t *row, int len,
                                          const int32_t *mine, int count, int64_t *from, int64_t *to) {
    const int64_t row_bytes = static_cast<int64_t>(c.d) * esz, head_bytes = row_bytes * c.page,
                  page_bytes = head_bytes * c.kv_heads;
    const int per_row = static_cast<int>(row_bytes / 16), total = per_row * c.kv_heads;
    for (int first = 0; first < count; first += kMoveChunk) {
        const int m = min(kMoveChunk, count - first);
        __syncthreads();
        for (int j = threadIdx.x; j < m; j += blockDim.x) {
            const int64_t a = static_cast<int64_t>(len) + mine[first + j], b = static_cast<int64_t>(len) + first + j;
            from[j] = row[a >> c.page_shift] * page_bytes + (a & (c.page - 1)) * row_bytes;
            to[j] = row[b >> c.page_shift] * page_bytes + (b & (c.page - 1)) * row_bytes;
        }
        __syncthreads();
        for (int y = threadIdx.x; y < 2 * total; y += blockDim.x) {
            const int x = y < total ? y : y - total;
            char *col = static_cast<char *>(y < total ? c.k : c.v) + layer * c.pages * page_bytes + (x / per_row) * head_bytes +
                        (x % per_row) * 16;
            for (int j0 = 0; j0 < m; j0 += 8) {
                int4 buf[8];
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    if (j0 + u < m && from[j0 + u] != to[j0 + u]) buf[u] = *reinterpret_cast<const int4 *>(col + from[j0 + u]);
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    if (j0 + u < m && from[j0 + u] != to[j0 + u]) *reinterpret_cast<int4 *>(col + to[j0 + u]) = buf[u];
            }
        }
    }
}

// One block per (entry, layer).
__global__ void __launch_bounds__(128) cache_commit_move_kernel(const ServeCache c, int esz, const int32_t *slots,
                                                                const int32_t *counts, const int32_t *keep,
                                                                int64_t max_keep) {
    grid_dependency_wait();
    __shared__ int64_t from[kMoveChunk], to[kMoveChunk];   // byte offsets of the rows in a layer, head 0
    int len = 0, held = 0, count = 0;
    if (!commit_entry(c, slots, counts, keep, max_keep, blockIdx.x, &len, &held, &count)) return;   // flagged below
    move_rows(c, esz, blockIdx.y, c.table + static_cast<int64_t>(slots[blockIdx.x]) * c.max_pages, len,
              keep + static_cast<int64_t>(blockIdx.x) * max_keep, count, from, to);
}

// Lengths grow by the kept rows; the pages behind the new length are released. move: the rows are moved here first.
__global__ void __launch_bounds__(128) cache_commit_kernel(const ServeCache c, int esz, const int32_t *slots,
                                                           const int32_t *counts, const int32_t *keep, int64_t max_keep,
                                                           bool move, int *status) {
    grid_dependency_wait();
    __shared__ int64_t from[kMoveChunk], to[kMoveChunk];
    int len = 0, held = 0, count = 0;
    if (!commit_entry(c, slots, counts, keep, max_keep, blockIdx.x, &len, &held, &count)) {
        if (threadIdx.x == 0) atomicOr(status, kStatusData);
        return;
    }
    const int32_t s = slots[blockIdx.x];
    int32_t *row = c.table + static_cast<int64_t>(s) * c.max_pages;
    if (move) {
        for (int y = 0; y < static_cast<int>(c.layers); ++y)
            move_rows(c, esz, y, row, len, keep + static_cast<int64_t>(blockIdx.x) * max_keep, count, from, to);
        __syncthreads();   // the table has been read
    }
    const int after = (len + count + c.page - 1) >> c.page_shift;
    for (int p = after + threadIdx.x; p < held; p += blockDim.x) {
        atomicSub(c.refs + row[p], 1);
        row[p] = -1;
    }
    if (threadIdx.x == 0) {
        c.lens[s] = len + count;
        c.held[s] = after;
    }
}

}  // namespace

size_t cache_workspace(int64_t n, int64_t pages) {
    return static_cast<size_t>(n) * (sizeof(int64_t) + 5 * sizeof(int32_t)) + static_cast<size_t>(pages) * sizeof(int32_t);
}

// All of these start behind the previous kernel of the stream without waiting for its last block to drain (they wait
// themselves): a cache step is a chain of short kernels, and this takes about a microsecond off each.

int launch_cache_free(const ServeCache &c, const int32_t *slots, int n, int *status, cudaStream_t st) {
    return launch_dependent(cache_free_kernel, dim3(n), dim3(256), 0, st, c, slots, status) ? 1 : -1;
}

int launch_cache_fork(const ServeCache &c, const int32_t *src, const int32_t *dst, int n, int *status, cudaStream_t st) {
    return launch_dependent(cache_fork_kernel, dim3(n), dim3(256), 0, st, c, src, dst, n, status) ? 1 : -1;
}

// Bytes of one row in all layers of k and v.
static int64_t row_bytes_all(const ServeCache &c, int esz) { return 2 * c.layers * c.kv_heads * c.d * esz; }

int launch_cache_reserve(const ServeCache &c, int esz, const int32_t *slots, const int32_t *add, int n, int32_t *granted,
                         void *ws, int *status, cudaStream_t st) {
    // up to about 256 KB the planning block copies as fast as a second launch starts
    const bool copy = n * c.page * row_bytes_all(c, esz) <= 256 * 1024;
    if (!launch_dependent(cache_reserve_plan_kernel, dim3(1), dim3(kPlanThreads), 0, st, c, slots, add, n, granted, ws, esz, copy,
                          status))
        return -1;
    if (copy) return 1;
    const dim3 grid(static_cast<unsigned>(n), static_cast<unsigned>(2 * c.layers));
    return launch_dependent(cache_reserve_copy_kernel, grid, dim3(256), 0, st, c, esz, n, ws) ? 2 : -1;
}

int launch_cache_append(const ServeCache &c, int esz, const int32_t *slots, const int32_t *cu, int n, int64_t tokens,
                        const void *k, const void *v, const int64_t kstr[3], const int64_t vstr[3], int64_t layer,
                        int64_t layers, int *status, cudaStream_t st) {
    AppendArgs a;
    a.k = static_cast<const char *>(k);
    a.v = static_cast<const char *>(v);
    a.kl = kstr[0] * esz; a.kt = kstr[1] * esz; a.kh = kstr[2] * esz;
    a.vl = vstr[0] * esz; a.vt = vstr[1] * esz; a.vh = vstr[2] * esz;
    a.layer = layer;
    a.layers = layers;
    const bool many = n > kAppendMany;
    const int64_t blocks = many ? (tokens + kAppendEach - 1) / kAppendEach : tokens;
    const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>((layers + kAppendLayers - 1) / kAppendLayers));
    return launch_dependent(many ? cache_append_kernel<true> : cache_append_kernel<false>, grid, dim3(256), 0, st, c, esz, slots,
                            cu, n, tokens, a, status)
               ? 1
               : -1;
}

int launch_cache_commit(const ServeCache &c, int esz, const int32_t *slots, const int32_t *counts, const int32_t *keep,
                        int64_t max_keep, int n, int *status, cudaStream_t st) {
    // small moves (a row of all layers within 16 KB) are made by the block that commits the entry
    const bool move = keep && row_bytes_all(c, esz) <= 16 * 1024;
    int launches = 0;
    if (keep && !move) {
        const dim3 grid(static_cast<unsigned>(n), static_cast<unsigned>(c.layers));
        if (!launch_dependent(cache_commit_move_kernel, grid, dim3(128), 0, st, c, esz, slots, counts, keep, max_keep)) return -1;
        ++launches;
    }
    if (!launch_dependent(cache_commit_kernel, dim3(n), dim3(128), 0, st, c, esz, slots, counts, keep, max_keep, move, status))
        return -1;
    return launches + 1;
}

}  // namespace ha
