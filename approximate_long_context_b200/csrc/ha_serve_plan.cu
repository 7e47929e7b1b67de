// ha_serve_plan.cu -- the list of work items of a prompt call with many sequences: one block sorts the items (a sequence
// and a group of its query rows) by falling position in their sequence, that is by falling cost, with a counting sort over
// positions. What bounds it is the chain offsets -> counts -> list in one block (5 to 6 us for 256 sequences); the
// attention kernels that follow take the items in turn and end together.
#include "ha_internal.h"
#include "ha_serve.cuh"

namespace ha {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanBuckets = 4096;

__global__ void __launch_bounds__(kPlanThreads) prompt_plan_kernel(const ServeArgs a, int64_t rows, bool singles_last, int capacity) {
    allow_dependents();
    grid_dependency_wait();
    __shared__ int cursor[kPlanBuckets];
    __shared__ int sums[32];
    PromptPlan *head = static_cast<PromptPlan *>(a.ws);
    int2 *list = reinterpret_cast<int2 *>(head + 1);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int levels = static_cast<int>((static_cast<int64_t>(a.max_len) * a.group + rows - 1) / rows);
    int shift = 0;
    while (((levels - 1) >> shift) + 2 > kPlanBuckets) ++shift;
    const int buckets = ((levels - 1) >> shift) + 2;   // the last one: sequences of one query tile
    // A lane reads a sequence; its entries are handled by the lane itself, or by the whole warp if there are many.
    auto visit = [&](auto entry, bool report) {
        bool ok = true;
        for (int b = warp * 32; b < a.seqs; b += kPlanThreads) {
            int start = 0, len = 0;
            if (b + lane < a.seqs) ok &= prompt_seq(a, b + lane, &start, &len);
            const int64_t mine_rows = static_cast<int64_t>(len) * a.group;
            const int pairs = static_cast<int>((mine_rows + rows - 1) / rows);
            const bool single = singles_last && len > 0 && 2 * mine_rows <= rows;
            if (singles_last) entry(single, buckets - 1, b + lane, 0);
            const unsigned big = __ballot_sync(0xffffffffu, pairs > 4);
            for (int p = 0; p < 4; ++p) {
                const bool mine = !single && p < pairs && !(big >> lane & 1u);
                if (__any_sync(0xffffffffu, mine)) entry(mine, buckets - 2 - (p >> shift), b + lane, p);
            }
            for (unsigned rest = big; rest; rest &= rest - 1) {
                const int l = __ffs(rest) - 1, n = __shfl_sync(0xffffffffu, pairs, l);
                for (int p0 = 0; p0 < n; p0 += 32) entry(p0 + lane < n, buckets - 2 - ((p0 + lane) >> shift), b + l, p0 + lane);
            }
        }
        if (report && !ok) atomicOr(a.status, kStatusData);
    };
    // the place of an entry in its bucket; the lanes of a warp that meet in one bucket take their places with one addition
    auto place = [&](bool mine, int b) -> int {
        const unsigned same = __match_any_sync(0xffffffffu, mine ? b : -1);
        const int leader = __ffs(same) - 1;
        int at = 0;
        if (mine && lane == leader) at = atomicAdd(&cursor[b], __popc(same));
        return __shfl_sync(0xffffffffu, at, leader) + __popc(same & ((1u << lane) - 1u));
    };
    for (int b = tid; b < buckets; b += kPlanThreads) cursor[b] = 0;
    __syncthreads();
    visit([&](bool mine, int b, int, int) { place(mine, b); }, true);
    __syncthreads();
    const int singles = cursor[buckets - 1];
    // exclusive sums over the buckets, highest position first: four buckets per thread
    int mine[kPlanBuckets / kPlanThreads], sum = 0;
#pragma unroll
    for (int i = 0; i < kPlanBuckets / kPlanThreads; ++i) {
        const int b = tid * (kPlanBuckets / kPlanThreads) + i;
        mine[i] = sum;
        sum += b < buckets ? cursor[b] : 0;
    }
    int x = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) sums[warp] = x;
    __syncthreads();
    if (warp == 0) {
        int w = sums[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, w, o);
            if (lane >= o) w += y;
        }
        sums[lane] = w;
    }
    __syncthreads();
    const int before = x - sum + (warp ? sums[warp - 1] : 0);
#pragma unroll
    for (int i = 0; i < kPlanBuckets / kPlanThreads; ++i) {
        const int b = tid * (kPlanBuckets / kPlanThreads) + i;
        if (b < buckets) cursor[b] = before + mine[i];
    }
    if (tid == 0) {
        head->count = min(sums[31], capacity);   // overlapping sequences (reported) could ask for more
        head->single = max(0, singles - (sums[31] - head->count));
    }
    __syncthreads();
    visit([&](bool mine, int b, int s, int p) {
        const int at = place(mine, b);
        if (mine && at < capacity) list[at] = make_int2(s, p);
    }, false);
}

}  // namespace

int64_t prompt_items(int64_t tokens, int64_t seqs, int64_t rows, int group) {
    // every sequence has at most one group of rows that is not full
    return tokens * group / rows + seqs;
}

size_t prompt_plan_bytes(int64_t items) { return sizeof(PromptPlan) + static_cast<size_t>(items) * sizeof(int2); }

bool launch_prompt_plan(const ServeArgs &a, int64_t rows, bool singles_last, int64_t items, cudaStream_t st) {
    return launch_dependent(prompt_plan_kernel, dim3(1), dim3(kPlanThreads), 0, st, a, rows, singles_last, static_cast<int>(items));
}

}  // namespace ha
