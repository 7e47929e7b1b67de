// ha_serve_tc.cu -- exact softmax attention for serving on the tensor cores (tcgen05 / TMEM / TMA), bf16 inputs: packed
// prompts (causal, grouped heads) and trees of drafted tokens over a paged cache.
//
// A query tile has 128 rows: the query tokens of one key head times the heads that share it (row = token * group + head),
// so every key tile that is loaded serves all of them. A work item has two tiles t = 0, 1, each with a softmax warpgroup of
// its own, so that the tensor core multiplies for one while the other's exponentials run:
//   PAIR: two neighbouring query tiles over the same key tiles (prompts; drafts of more than one tile);
//   ALT:  one query tile, tile t takes every other key tile; the two results are joined in the epilogue (decoding and
//         small trees, which are bound by reading the cache).
//   ALT16: ALT for d = 128 and pages of 16 rows. A load of a page brings one box of 64 columns; with 2 KB boxes the copy
//         engine and not the memory is the bound (64 users decoding: 424 us, against 330 us with larger pages and 342 us
//         here; 16 trees of 32 tokens: 100 -> 83 us). Here a box has both halves of the page's rows (4 KB). A key
//         tile then lies page by page, [half][16 rows][128 bytes], which the score product reads as two products of
//         64 keys, rows 0-7 and rows 8-15 of the eight pages; the softmax puts the keys back in order when it
//         writes P.
// Tree items come from an even cut of all key tiles over the blocks (TreeWalk); pieces of a cut segment go to the
// workspace and a second kernel joins them.
//
// Per unit (tile t, key tile): S = Q K^T (128 x 128, fp32, TMEM), P = 2^(c S - m) in bf16 over the first half of S's
// columns, O_t += P V (TMEM). A thread of the softmax owns a query row; it keeps m and l in fp32 and rescales O only when
// the maximum grows by more than 2^8 (P stays below 2^8; the sums are fp32, so the unscaled start costs no precision).
// P is rounded to bf16 because the tensor core multiplies bf16; l sums the unrounded values. The exponentials and the final
// quotient are the hardware's ex2.approx and rcp.approx: a few units in the last place of fp32, far below a weight's rounding
// to bf16. Calls that want fp32 weights take the SIMT family.
//
// Issue order: S(next unit) goes out before P V(unit) is waited for when it belongs to the other tile, so a tile's P V and
// next S run back to back while the other tile is in its softmax. A commit after S(j + 1) covers P V(j) too (same issuing
// thread): a softmax thread that sees S(j + 1) may rescale O.
//
// Values of masked keys may be infinities or NaN: 0 * inf would reach rows that do not see them. Two warps look each
// value tile over that some row does not see in full, replace what is not finite by 0 before the product and note it
// for the item; the epilogue of a noted item adds those values to the rows that do see them.
//
// Block (512 threads, one per SM, persistent): warp 0 fetches the items and loads (TMA), warp 1 issues the MMAs, warps 2
// and 3 look values over, warps 4-7 and 8-11 are the softmax of tile 0 and 1, warps 12-15 the epilogue of both (a tile's
// epilogue takes as long as one or two of its units; the softmax goes on with the next item meanwhile). Every wait is
// bounded; on expiry the status word is set, all roles stop, the loader waits for its copies and TMEM is freed.
//
// What bounds it. Prompts: per tile and unit (128 rows x 128 keys, d = 128) the softmax takes about 1900 cycles and P V
// with the next S another 1600, of which 1024 are the tensor pipe's; two tiles overlap, so tensor pipe and exponentials
// are busy 59% each, and TMEM has no room for a third tile. 32768 tokens, 8 heads on 2, d = 128: 2.00 ms back to back (1100
// TFLOP/s), 1.76 ms in a burst at full clock. 16 prompts of up to 2047 tokens, 32 heads on 8: 266 us (750 TFLOP/s), 240 in a
// burst; their items are short, and a diagonal tile costs as much as a full one. Prompts of one key tile (256 of up to 128
// tokens, 16 heads, d = 64: 53 us, 2.5 TB/s): instruction fetch, each role's code runs once per item. Decoding and small
// trees: reading the cache, 64 users and 2.2 GB: 332 to 357 us by the card (6.1 to 6.5 TB/s).
#include <cuda.h>
#include <math.h>

#include <atomic>
#include <type_traits>

#include "ha_common.cuh"
#include "ha_internal.h"
#include "ha_serve.cuh"
#include "ha_sm100.cuh"

namespace ha {
namespace {

using namespace sm100;

constexpr int kThreads = 512;
// Registers per thread of the four warpgroups after the start (512 threads start with 128 each): loads, MMAs and checks;
// softmax (two); epilogue.
constexpr int kRegsAux = 64, kRegsSoftmax = 168, kRegsOut = 112;
static_assert(kRegsAux + 2 * kRegsSoftmax + kRegsOut <= 512, "the shares add up to what the block starts with");
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kGrow = 8.0f;

enum { PROMPT = 0, TREE_PAIR = 1, TREE_ALT = 2, TREE_ALT16 = 3 };

// One work item, published by the loader.
struct Item {
    int start, tok0, tokens, len;   // first query row, first token of tile 0 and query tokens of the sequence, keys in front
    int kh, k0, n0, n1;             // key head, first key tile, key tiles of tile 0 and 1
    int masked;                     // first key tile that some row does not see in full
    int slot;                       // workspace slot of a piece, -1: the item is a whole segment
    int last;                       // no item: the end
    int odd;                        // a value that is not finite was replaced
    int64_t kv;                     // tree: row of the page table; prompt: first key row
    int k1;
    int duo;                        // two key heads kh, kh + 1 of one query tile each, with key tiles of their own
};
static_assert(sizeof(Item) == 64, "one item per 64 bytes");

constexpr int kItems = 4;

template <int D, int MODE>
struct Cfg {
    static constexpr bool ALT = MODE == TREE_ALT || MODE == TREE_ALT16, P16 = MODE == TREE_ALT16;
    static constexpr int kTile = 128 * D * 2;      // 128 rows of bf16
    static constexpr int NQ = ALT ? 1 : 2;
    static constexpr int NK = D == 64 ? (ALT ? 6 : 5) : (ALT ? 3 : 2);
    static constexpr int NV = D == 64 ? (ALT ? 6 : 4) : (ALT ? 3 : 2);
    static constexpr int kQ = 0;
    static constexpr int kK = NQ * kTile;
    static constexpr int kV = kK + NK * kTile;
    static constexpr int kOut = kV + NV * kTile;                   // PAIR: 32 rows of O in bf16 per epilogue warp
    static constexpr int kItemsAt = kOut + 4 * (ALT ? 0 : 64 * D);
    static constexpr int kStat = kItemsAt + kItems * 64;           // maximum and sum of the tiles' rows
    static constexpr int kBars = kStat + 2 * 128 * 8;
    static constexpr int bQFull = 0, bQEmpty = bQFull + 2, bKFull = bQEmpty + 2, bKEmpty = bKFull + NK,
                         bVFull = bKEmpty + NK, bVOk = bVFull + NV, bVEmpty = bVOk + NV, bItemFull = bVEmpty + NV,
                         bItemEmpty = bItemFull + kItems, bSFull = bItemEmpty + kItems, bPFull = bSFull + 2,
                         bODone = bPFull + 2, bOFree = bODone + 2, bStat = bOFree + 2, bStatFree = bStat + 2,
                         bDrain = bStatFree + 2,
                         kNumBars = bDrain + 1;
    static constexpr int kTmemSlot = kBars + kNumBars * 8;
    static constexpr int kAbort = kTmemSlot + 4;
    static constexpr int kBytes = kAbort + 4;
    static_assert(kBars % 8 == 0, "mbarriers need 8-byte alignment");
    static_assert(kBytes <= 232448, "shared memory budget");
};

struct Maps {
    CUtensorMap q, k, v;
};

struct TcArgs {
    ServeArgs a;
    int tpt;         // query tokens of a tile
    int box_rows;    // rows that a Q load brings
    int order;       // prompt: where the items come from (PromptOrder)
};

// Wait for a phase of a barrier, at most about 2 s of global time. Inlined in few instructions: under a register split no
// function can be called, and code that runs once per item is mostly waited for by instruction fetches.
__device__ __forceinline__ uint32_t timer_lo() {
    uint32_t t;
    asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(t));
    return t;
}
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, volatile int *abort, uint32_t limit_ns = 2000000000u) {
    if (__builtin_expect(mbar_try_wait(bar, parity), 1)) return true;
    const uint32_t t0 = timer_lo();
    do {
        if (mbar_try_wait(bar, parity)) return true;
    } while (*abort == 0 && timer_lo() - t0 < limit_ns);
    *abort = 1;
    return false;
}

__device__ __forceinline__ void tma_3d(uint32_t dst, const CUtensorMap *map, uint32_t bar, int x, int y, int z) {
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::
                     "r"(dst), "l"(map), "r"(bar), "r"(x), "r"(y), "r"(z)
                 : "memory");
}
__device__ __forceinline__ void tma_4d(uint32_t dst, const CUtensorMap *map, uint32_t bar, int x, int y, int z, int w) {
    asm volatile("cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], [%2];" ::
                     "r"(dst), "l"(map), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(w)
                 : "memory");
}
__device__ __forceinline__ void tma_5d(uint32_t dst, const CUtensorMap *map, uint32_t bar, int x, int y, int z, int w, int v) {
    asm volatile("cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::
                     "r"(dst), "l"(map), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(w), "r"(v)
                 : "memory");
}
__device__ __forceinline__ void prefetch_map(const CUtensorMap *map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// ---------------------------------------------------------------------------------------------- prompt items
//
// The items of a prompt call (sequence, pair of query tiles) cost as many key tiles as lie in front of them. In general a
// one-block kernel lists them by falling position, so that the persistent blocks, which take them in turn (to and fro),
// end together. No list is needed for one sequence, for fewer items than blocks (SCAN: the walk finds them in the
// offsets), nor where no sequence is longer than a pair of tiles: all items cost alike then (PAIRS), and sequences of one
// tile take two key heads at a time (SINGLES).
enum PromptOrder { SCAN = 0, LIST = 1, PAIRS = 2, SINGLES = 3 };

// The walk of one block over a prompt call's items, run by one whole warp.
struct PromptWalk {
    int64_t count;    // items
    int64_t normal;   // of them, in front: one key head each
    int64_t round;
    // One sequence, or few enough items for one round of blocks: no list.
    __device__ __forceinline__ void begin(const TcArgs &x) {
        const ServeArgs &a = x.a;
        const int lane = threadIdx.x & 31;
        round = 0;
        if (x.order >= PAIRS) {
            // the offsets are looked over here, as no list is made
            bool ok = true;
            for (int b = blockIdx.x * 32 + lane; b < a.seqs; b += gridDim.x * 32) {
                int start, len;
                ok &= prompt_seq(a, b, &start, &len);
            }
            if (!ok) atomicOr(a.status, kStatusData);
            count = static_cast<int64_t>(a.seqs) * (x.order == SINGLES ? (a.kv_heads + 1) >> 1 : a.kv_heads);
            return;
        }
        if (x.order == LIST) {
            const PromptPlan *p = static_cast<const PromptPlan *>(a.ws);
            normal = static_cast<int64_t>(p->count - p->single) * a.kv_heads;
            count = normal + static_cast<int64_t>(p->single) * ((a.kv_heads + 1) >> 1);
            return;
        }
        int64_t pairs = 0;
        bool ok = true;
        for (int b = 0; b < a.seqs; b += 32) {
            int start = 0, len = 0;
            if (b + lane < a.seqs) ok &= prompt_seq(a, b + lane, &start, &len);
            pairs += (len + 2 * x.tpt - 1) / (2 * x.tpt);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) pairs += __shfl_xor_sync(0xffffffffu, pairs, o);
        if (!ok && blockIdx.x == 0) atomicOr(a.status, kStatusData);
        normal = count = pairs * a.kv_heads;
    }
    __device__ __forceinline__ bool next(const TcArgs &x, int *seq, int *pair, int *kh, bool *single) {
        const ServeArgs &a = x.a;
        const int lane = threadIdx.x & 31;
        if (x.order >= PAIRS) {
            const int half = (a.kv_heads + 1) >> 1;
            for (;; ++round) {   // empty sequences are passed over
                const int64_t i = round * gridDim.x + blockIdx.x;
                if (i >= count) return false;
                *single = x.order == SINGLES;
                const int per = *single ? half : a.kv_heads;
                *seq = static_cast<int>(quotient(i, per));
                *kh = static_cast<int>(i - static_cast<int64_t>(*seq) * per) * (*single ? 2 : 1);
                *pair = 0;
                int start, len;
                prompt_seq(a, *seq, &start, &len);
                if (len > 0) break;
            }
            ++round;
            return true;
        }
        const int64_t turn = (round & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x;
        const int64_t i = round * gridDim.x + turn;
        ++round;
        if (i >= count) return false;   // the last round is not full
        if (x.order == LIST) {
            const int half = (a.kv_heads + 1) >> 1;
            *single = i >= normal;
            const int64_t own = *single ? i - normal : i, group = quotient(own, *single ? half : a.kv_heads);
            const int64_t at = *single ? quotient(normal, a.kv_heads) + group : group;
            *kh = static_cast<int>(own - group * (*single ? half : a.kv_heads)) * (*single ? 2 : 1);
            const int2 e = reinterpret_cast<const int2 *>(static_cast<const PromptPlan *>(a.ws) + 1)[at];
            *seq = e.x;
            *pair = e.y;
            return true;
        }
        const int64_t at = quotient(i, a.kv_heads);
        *kh = static_cast<int>(i - at * a.kv_heads);
        int64_t run = 0;
        for (int b = 0; b < a.seqs; b += 32) {
            int start = 0, len = 0;
            if (b + lane < a.seqs) prompt_seq(a, b + lane, &start, &len);
            const int64_t mine = (len + 2 * x.tpt - 1) / (2 * x.tpt);
            int64_t sum = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t z = __shfl_up_sync(0xffffffffu, sum, o);
                if (lane >= o) sum += z;
            }
            const unsigned hit = __ballot_sync(0xffffffffu, run + sum > at);
            if (hit) {
                const int l = __ffs(hit) - 1;
                *seq = b + l;
                const int64_t pairs = __shfl_sync(0xffffffffu, mine, l);
                *pair = static_cast<int>(pairs - 1 - (at - run - __shfl_sync(0xffffffffu, sum - mine, l)));
                return true;
            }
            run += __shfl_sync(0xffffffffu, sum, 31);
        }
        return false;
    }
};

// ---------------------------------------------------------------------------------------------- masks

// Which of the 32 keys from `first` on (relative to the tile's keys) a row sees.
// prompt: the keys up to `own`; tree: the committed keys and the drafted ones set in bits.
__device__ __forceinline__ uint32_t seen_causal(int own, int first) {
    const int n = own + 1 - first;
    return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u;
}
__device__ __forceinline__ uint32_t seen_tree(uint64_t bits, int len, int first) {
    const int s = first - len;   // drafted row of the first key
    if (s <= -32) return 0xffffffffu;
    if (s >= 64) return 0u;
    if (s >= 0) return static_cast<uint32_t>(bits >> s);
    return static_cast<uint32_t>(bits << -s) | ((1u << -s) - 1u);
}

__device__ __forceinline__ float rcp_approx(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

// ---------------------------------------------------------------------------------------------- the kernel

template <int D, int MODE>
__global__ void __launch_bounds__(kThreads, 1) serve_tc_kernel(const TcArgs x, const __grid_constant__ Maps maps) {
    using C = Cfg<D, MODE>;
    constexpr bool ALT = C::ALT, TREE = MODE != PROMPT, P16 = C::P16;
    const ServeArgs &a = x.a;
    extern __shared__ __align__(1024) unsigned char sm[];   // the swizzled tiles need the alignment; there is no room to pad
    const uint32_t sbase = smem_addr(sm);
    if (sbase & 1023u) {
        if (threadIdx.x == 0) atomicOr(a.status, kStatusTimeout);
        return;
    }
    auto bar = [&](int i) -> uint32_t { return sbase + C::kBars + 8u * static_cast<uint32_t>(i); };
    volatile int *abort_flag = reinterpret_cast<volatile int *>(sm + C::kAbort);
    Item *items = reinterpret_cast<Item *>(sm + C::kItemsAt);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 32) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(C::bQFull + i), 1);
            mbar_init(bar(C::bQEmpty + i), 1);
            mbar_init(bar(C::bSFull + i), 1);
            mbar_init(bar(C::bPFull + i), 4);    // one arrival per warp
            mbar_init(bar(C::bODone + i), 1);
            mbar_init(bar(C::bOFree + i), 4);
        }
        for (int i = 0; i < C::NK; ++i) {
            mbar_init(bar(C::bKFull + i), 1);
            mbar_init(bar(C::bKEmpty + i), 1);
        }
        for (int i = 0; i < C::NV; ++i) {
            mbar_init(bar(C::bVFull + i), 1);
            mbar_init(bar(C::bVOk + i), 2);
            mbar_init(bar(C::bVEmpty + i), 1);
        }
        for (int i = 0; i < kItems; ++i) {
            mbar_init(bar(C::bItemFull + i), 1);
            mbar_init(bar(C::bItemEmpty + i), 1 + 2 + 8 + 4);   // MMA issuer, looking, softmax and epilogue warps
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(C::bStat + i), 4);
            mbar_init(bar(C::bStatFree + i), 4);
        }
        mbar_init(bar(C::bDrain), 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    // Rows of the Q tiles that no load brings are zeros, so that their scores, weights and products are: multiplying what
    // happened to lie there draws power, and the clock gives way to power (64 users decoding, sustained: 365 -> 331 us).
    if (x.box_rows < 128) {
        const int rows = 128 - x.box_rows;
        for (int e = threadIdx.x; e < C::NQ * (D / 64) * rows * 8; e += kThreads) {
            const int part = e / (rows * 8), y = e - part * rows * 8;
            *reinterpret_cast<uint4 *>(sm + C::kQ + part * 16384 + (x.box_rows + (y >> 3)) * 128 + (y & 7) * 16) =
                make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();
    }
    if (warp == 0 && lane == 0) {
        prefetch_map(&maps.q);
        prefetch_map(&maps.k);
        prefetch_map(&maps.v);
    }
    if (TREE || gridDim.x < a.sms) allow_dependents();
    grid_dependency_wait();   // what was in front on the stream, the list of prompt items among it
    // TMEM only now: a block that held it while it waits could keep it from a block of what it waits for
    if (warp == 0) {
        tmem_alloc(sbase + C::kTmemSlot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(sm + C::kTmemSlot);

    // a wait of a whole warp: all of its lanes go on or none
    auto warp_wait = [&](uint32_t b, uint32_t parity) -> bool { return __all_sync(0xffffffffu, bar_wait(b, parity, abort_flag)); };
    // the item ring, read by all roles but the loader
    // one arrival for a warp whose lanes have all got here (and fenced what they wrote)
    auto warp_arrive = [&](uint32_t b) {
        __syncwarp();
        if (lane == 0) mbar_arrive(b);
    };
    auto item_bar = [&](uint32_t i) -> uint32_t { return bar(C::bItemFull + i % kItems); };

    if (warp == 0) {
        // ------------------------------------------------------------------ items and loads
        setmaxnreg_dec<kRegsAux>();
        bool ok = true;
        uint32_t ni = 0, nk = 0, nv = 0, nq[2] = {0, 0};   // items published, loads issued
        PromptWalk pw;
        TreeWalk tw;
        const int tok_tile = ALT ? x.tpt : 2 * x.tpt;
        if (TREE) {
            tw.begin(a, 128, 0, tok_tile, blockIdx.x, gridDim.x);
            if (lane == 0) tree_joins(a.ws)[blockIdx.x].pieces = 0;
        } else {
            pw.begin(x);
        }
        const int page = 1 << a.page_shift, per_tile = page >= 128 ? 1 : 128 >> a.page_shift;
        for (;;) {
            Item it{};
            TreePiece p;
            bool got;
            if (TREE) {
                got = tw.next(a, 128, 0, tok_tile, &p);
                if (got) {
                    it.start = p.x.start;
                    it.tok0 = p.tile * tok_tile;
                    it.tokens = p.x.t;
                    it.len = p.x.len;
                    it.kh = p.kh;
                    it.k0 = p.k0;
                    it.k1 = p.k1;
                    it.masked = p.x.len >> 7;
                    it.slot = p.k0 == 0 && p.k1 == p.nk ? -1 : 2 * static_cast<int>(blockIdx.x) + (p.k0 == 0);
                    it.kv = p.x.table;
                    const int n = p.k1 - p.k0;
                    it.n0 = ALT ? (n + 1) >> 1 : n;
                    it.n1 = ALT ? n >> 1 : it.tok0 + x.tpt < it.tokens ? n : 0;
                    if (p.k0 == 0 && it.slot >= 0 && lane == 0) {
                        TreeJoin j{};
                        j.pieces = tree_pieces(p, blockIdx.x);
                        j.start = it.start;
                        j.row0 = it.tok0 * a.group;
                        j.rows = min(tok_tile, it.tokens - it.tok0) * a.group;
                        j.kh = it.kh;
                        tree_joins(a.ws)[blockIdx.x] = j;
                    }
                }
            } else {
                int seq, pair, kh;
                bool single = false;
                got = pw.next(x, &seq, &pair, &kh, &single);
                if (got) {
                    prompt_seq(a, seq, &it.start, &it.tokens);
                    it.tok0 = pair * 2 * x.tpt;
                    it.kh = kh;
                    it.masked = (it.tok0 + 1) >> 7;
                    it.slot = -1;
                    it.kv = it.start;
                    it.n0 = (min(it.tokens, it.tok0 + x.tpt) + 127) >> 7;
                    it.n1 = it.tok0 + x.tpt < it.tokens ? (min(it.tokens, it.tok0 + 2 * x.tpt) + 127) >> 7 : 0;
                    if (single) {
                        it.duo = 1;
                        it.n1 = kh + 1 < a.kv_heads ? it.n0 : 0;
                    }
                    it.k1 = max(it.n0, it.n1);
                }
            }
            it.last = !got;
            const int is = ni % kItems;
            if (ni >= kItems && !warp_wait(bar(C::bItemEmpty + is), (ni / kItems - 1) & 1)) { ok = false; break; }
            if (lane == 0) {
                items[is] = it;
                mbar_arrive(bar(C::bItemFull + is));
            }
            __syncwarp();
            ++ni;
            if (!got) break;
            const int n = it.duo ? it.n0 + it.n1 : it.k1 - it.k0;
            const int keys = it.len + it.tokens;
            // page of this lane's part of key tile j (tree), -1 where the load is to bring zeros
            auto page_of = [&](int kt) -> int {
                int id = -1;
                if (TREE && lane < per_tile) {
                    const int first = page >= 128 ? kt * 128 : kt * 128 + lane * page;
                    if (first < keys) {
                        id = a.table[it.kv + (first >> a.page_shift)];
                        if (id < 0 || id >= a.pages) {
                            atomicOr(a.status, kStatusData);
                            id = -1;
                        }
                    }
                }
                return id;
            };
            auto load_tile = [&](const CUtensorMap *map, uint32_t dst, uint32_t b, int i, int id) {
                const int kt = it.k0 + (it.duo ? i >> 1 : i), kh = it.kh + (it.duo ? i & 1 : 0);
                if (lane == 0) mbar_arrive_expect_tx(b, C::kTile);
                __syncwarp();
                if (TREE) {
                    if (lane < per_tile) {
                        const int z = id < 0 ? static_cast<int>(a.pages) : id;   // past the last page: zeros
                        const int y = page > 128 ? (kt * 128) & (page - 1) : 0;
                        if (P16) {
                            tma_5d(dst + lane * 4096, map, b, 0, 0, 0, kh, z);
                        } else {
#pragma unroll
                            for (int h = 0; h < D / 64; ++h)
                                tma_4d(dst + h * 16384 + lane * (page << 7), map, b, h * 64, y, kh, z);
                        }
                    }
                } else if (lane == 0) {
#pragma unroll
                    for (int h = 0; h < D / 64; ++h) tma_3d(dst + h * 16384, map, b, h * 64, kh, static_cast<int>(it.kv) + kt * 128);
                }
            };
            auto load_k = [&](int i, int id) -> bool {
                const int s = nk % C::NK;
                if (nk >= C::NK && !warp_wait(bar(C::bKEmpty + s), (nk / C::NK - 1) & 1)) return false;
                load_tile(&maps.k, sbase + C::kK + s * C::kTile, bar(C::bKFull + s), i, id);
                ++nk;
                return true;
            };
            auto load_v = [&](int i, int id) -> bool {
                const int s = nv % C::NV;
                if (nv >= C::NV && !warp_wait(bar(C::bVEmpty + s), (nv / C::NV - 1) & 1)) return false;
                load_tile(&maps.v, sbase + C::kV + s * C::kTile, bar(C::bVFull + s), i, id);
                ++nv;
                return true;
            };
            int id = page_of(it.k0), ahead = n > 1 ? page_of(it.k0 + 1) : -1;
            ok = load_k(0, id);
            for (int t = 0; t < C::NQ && ok; ++t) {
                if (!ALT && (t == 0 ? it.n0 : it.n1) == 0) continue;
                if (nq[t] >= 1 && !warp_wait(bar(C::bQEmpty + t), (nq[t] - 1) & 1)) { ok = false; break; }
                if (lane == 0) {
                    mbar_arrive_expect_tx(bar(C::bQFull + t), x.box_rows * D * 2);
#pragma unroll
                    for (int h = 0; h < D / 64; ++h)
                        tma_3d(sbase + C::kQ + t * C::kTile + h * 16384, &maps.q, bar(C::bQFull + t), h * 64,
                               (it.kh + (it.duo ? t : 0)) * a.group, it.start + it.tok0 + (it.duo ? 0 : t * x.tpt));
                }
                __syncwarp();
                ++nq[t];
            }
            for (int j = 0; j < n && ok; ++j) {
                const int far = j + 2 < n ? page_of(it.k0 + j + 2) : -1;
                if (j + 1 < n) ok = load_k(j + 1, ahead);
                if (ok) ok = load_v(j, id);
                id = ahead;
                ahead = far;
            }
            if (!ok) break;
        }
        if (!ok) {
            if (lane == 0) atomicOr(a.status, kStatusTimeout);
            // the copies in flight land before the block ends
            volatile int no_abort = 0;
            for (uint32_t i = nk > C::NK ? nk - C::NK : 0; i < nk; ++i)
                bar_wait(bar(C::bKFull + i % C::NK), (i / C::NK) & 1, &no_abort, 200000000u);
            for (uint32_t i = nv > C::NV ? nv - C::NV : 0; i < nv; ++i)
                bar_wait(bar(C::bVFull + i % C::NV), (i / C::NV) & 1, &no_abort, 200000000u);
            for (int t = 0; t < C::NQ; ++t)
                if (nq[t]) bar_wait(bar(C::bQFull + t), (nq[t] - 1) & 1, &no_abort, 200000000u);
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------------ MMA issuer
        setmaxnreg_dec<kRegsAux>();
        // The whole warp runs the control flow and one elected lane issues: loop state stays in uniform registers, which
        // the descriptors of the MMAs have to be in. One copy of each kind of step, looped over: the warp shares its
        // scheduler's instruction cache with two softmax warps, and a straight-line version spent about 200 cycles per
        // wait on fetching itself.
        const bool leader = elect_one();
        constexpr uint32_t idesc_qk = idesc_bf16(128, P16 ? 64 : 128, false, false);
        constexpr uint32_t idesc_pv = idesc_bf16(128, D, false, true);
        const uint64_t dq0 = smem_desc(sbase + C::kQ, 16, 1024);
        const uint64_t dk0 = smem_desc(sbase + C::kK, 16, P16 ? 4096 : 1024);
        const uint64_t dv0 = smem_desc(sbase + C::kV, P16 ? 2048 : 16384, 1024);
        bool ok = true;
        uint32_t base = 0, idx = 0;          // number of the item's first key tile among the block's loads; the item
        uint32_t cq = 0, cp = 0, co = 0;     // parities, bit t: Q tiles waited for (ALT: bit 0), P tiles consumed, items begun
        uint32_t begun = 0;                  // bit t: tile t has had an item
        int n0 = 0, n1 = 0, last = 0;
        bool two = ALT;                      // the tiles take turns at the key tiles (ALT and two heads) or share them
        auto read_item = [&](uint32_t i, int *m0, int *m1, int *end, bool *turns) {
            const volatile Item &it = items[i % kItems];
            *m0 = __shfl_sync(0xffffffffu, it.n0, 0);
            *m1 = __shfl_sync(0xffffffffu, it.n1, 0);
            *end = __shfl_sync(0xffffffffu, it.last, 0);
            *turns = ALT || (!TREE && __shfl_sync(0xffffffffu, it.duo, 0) != 0);
        };
        ok = warp_wait(item_bar(0), 0);
        if (ok) read_item(0, &n0, &n1, &last, &two);
        uint32_t ahead = 0;                  // bit t: the first score product of this item's tile t is already issued
        while (ok && !last) {
            const int most = max(n0, n1);
            const uint32_t next = base + (two ? n0 + n1 : most);
            int m0 = 0, m1 = 0, end = 1;
            bool known = false, mtwo = ALT;
            uint32_t early = 0;              // as `ahead`, for the next item
#pragma unroll 1
            for (int j = -1; j < most && ok; ++j) {
                if (j == most - 1) {
                    known = __all_sync(0xffffffffu, mbar_try_wait(item_bar(idx + 1), ((idx + 1) / kItems) & 1));
                    if (known) read_item(idx + 1, &m0, &m1, &end, &mtwo);
                }
#pragma unroll 1
                for (int t = 0; t < 2; ++t) {
                    const int n = t == 0 ? n0 : n1;
                    // ---- P V of key tile j
                    if (j >= 0 && j < n) {
                        const uint32_t tile = base + (two ? 2 * j + t : j);
                        const uint32_t vs = tile % C::NV;
                        if (!warp_wait(bar(C::bVOk + vs), (tile / C::NV) & 1)) { ok = false; break; }
                        if (j == 0) {
                            if ((begun >> t & 1) && !warp_wait(bar(C::bOFree + t), co >> t & 1)) { ok = false; break; }
                            if (begun >> t & 1) co ^= 1u << t;
                            begun |= 1u << t;
                        }
                        const uint64_t dv = dv0 + static_cast<uint64_t>((vs * C::kTile) >> 4);
                        const uint32_t tO = tmem + 256 + t * D, tP = tmem + t * 128;
                        if (!warp_wait(bar(C::bPFull + t), cp >> t & 1)) { ok = false; break; }
                        cp ^= 1u << t;
                        tc_fence_after();
                        if (leader) {
#pragma unroll
                            for (int kk = 0; kk < 8; ++kk)
                                mma_ts(tO, tP + kk * 8, dv + static_cast<uint64_t>((kk * (P16 ? 4096 : 2048)) >> 4), idesc_pv,
                                       (j > 0 || kk > 0) ? 1u : 0u);
                            if (two || t == 1 || j >= n1) mma_commit(bar(C::bVEmpty + vs));
                            if (j == n - 1) mma_commit(bar(C::bODone + t));
                        }
                        __syncwarp();
                    }
                    // ---- S of this tile's next key tile, here or (if all it needs is there) in the next item
                    const bool here = j + 1 < n && !(j < 0 && (ahead >> t & 1));
                    const bool there = j == most - 1 && known && !end && (t == 0 || (early & 1) != 0) && (t == 0 ? m0 : m1) > 0;
                    if (!here && !there) continue;
                    const int k = here ? j + 1 : 0, e0 = here ? n0 : m0, e1 = here ? n1 : m1;
                    const bool turns = here ? two : mtwo;
                    const uint32_t tile = (here ? base : next) + (turns ? 2 * k + t : k);
                    const uint32_t ks = tile % C::NK, qi = ALT ? 0 : t;
                    const uint32_t kb = bar(C::bKFull + ks), kpar = (tile / C::NK) & 1;
                    const bool new_q = k == 0 && (!ALT || t == 0);
                    if (here) {
                        if (!warp_wait(kb, kpar) || (new_q && !warp_wait(bar(C::bQFull + qi), cq >> qi & 1))) { ok = false; break; }
                    } else if (!__all_sync(0xffffffffu, mbar_try_wait(kb, kpar)) ||
                               (new_q && !__all_sync(0xffffffffu, mbar_try_wait(bar(C::bQFull + qi), cq >> qi & 1)))) {
                        continue;
                    }
                    if (new_q) cq ^= 1u << qi;
                    if (!here) early |= 1u << t;
                    tc_fence_after();
                    const uint64_t dq = dq0 + static_cast<uint64_t>((qi * C::kTile) >> 4);
                    const uint64_t dk = dk0 + static_cast<uint64_t>((ks * C::kTile) >> 4);
                    const uint32_t tS = tmem + t * 128;
                    // the item's last score product with this Q
                    const bool free_q = !ALT ? k == (t == 0 ? e0 : e1) - 1 : t == 0 ? e0 == k + 1 && e1 <= k : e0 <= k + 1;
                    if (leader) {
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk) {
                            const uint64_t off = static_cast<uint64_t>(((kk >> 2) * 16384 + (kk & 3) * 32) >> 4);
                            if (P16) {
                                const uint64_t offk = static_cast<uint64_t>(((kk >> 2) * 2048 + (kk & 3) * 32) >> 4);
                                mma_ss(tS, dq + off, dk + offk, idesc_qk, kk > 0 ? 1u : 0u);
                                mma_ss(tS + 64, dq + off, dk + offk + (1024 >> 4), idesc_qk, kk > 0 ? 1u : 0u);
                            } else {
                                mma_ss(tS, dq + off, dk + off, idesc_qk, kk > 0 ? 1u : 0u);
                            }
                        }
                        mma_commit(bar(C::bSFull + t));
                        if (turns || t == 1 || k >= e1) mma_commit(bar(C::bKEmpty + ks));
                        if (free_q) mma_commit(bar(C::bQEmpty + qi));
                    }
                    __syncwarp();
                }
            }
            if (!ok) break;
            if (leader) mbar_arrive(bar(C::bItemEmpty + idx % kItems));
            ++idx;
            if (!known) {
                if (!warp_wait(item_bar(idx), (idx / kItems) & 1)) { ok = false; break; }
                read_item(idx, &m0, &m1, &end, &mtwo);
            }
            base = next;
            n0 = m0;
            n1 = m1;
            last = end;
            two = mtwo;
            ahead = early;
        }
        if (!ok && leader) atomicOr(a.status, kStatusTimeout);
        if (leader) {
            mma_commit(bar(C::bDrain));   // every MMA issued so far completes before TMEM is released
            volatile int no_abort = 0;
            bar_wait(bar(C::bDrain), 0, &no_abort, 200000000u);
        }
        __syncwarp();
    } else if (warp < 4) {
        // ------------------------------------------------------------------ values of masked keys
        setmaxnreg_dec<kRegsAux>();
        bool ok = true;
        uint32_t nv = 0;
        for (uint32_t i = 0; ok; ++i) {
            if (!warp_wait(item_bar(i), (i / kItems) & 1)) { ok = false; break; }
            Item *it = &items[i % kItems];
            if (it->last) break;
            const bool duo = !TREE && it->duo;
            const int n = duo ? it->n0 + it->n1 : it->k1 - it->k0;
            for (int j = 0; j < n; ++j, ++nv) {
                const int s = nv % C::NV;
                if (!warp_wait(bar(C::bVFull + s), (nv / C::NV) & 1)) { ok = false; break; }
                if (it->k0 + (duo ? j >> 1 : j) >= it->masked) {
                    uint4 *tile = reinterpret_cast<uint4 *>(sm + C::kV + s * C::kTile);
                    // an exponent of ones in either half carries into the bit above it
                    auto bad = [](uint32_t u) { return ((u & 0x7f807f80u) + 0x00800080u) & 0x80008000u; };
                    bool odd = false;
#pragma unroll 1
                    for (int e0 = (warp - 2) * 32 + lane; e0 < C::kTile / 16; e0 += 64 * 8) {
                        // eight loads in flight, with no store between them (256 short prompts: 55.9 -> 53.1 us, 16
                        // ragged ones: 234.6 -> 230.3 us)
                        uint32_t any = 0;
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const uint4 w = tile[e0 + e * 64];
                            any |= bad(w.x) | bad(w.y) | bad(w.z) | bad(w.w);
                        }
                        if (any) {
                            odd = true;
                            auto clean = [&](uint32_t u) {
                                const uint32_t b = bad(u);
                                return u & ~((b & 0x80000000u ? 0xffff0000u : 0u) | (b & 0x8000u ? 0xffffu : 0u));
                            };
#pragma unroll 1
                            for (int e = 0; e < 8; ++e) {
                                const uint4 w = tile[e0 + e * 64];
                                tile[e0 + e * 64] = make_uint4(clean(w.x), clean(w.y), clean(w.z), clean(w.w));
                            }
                        }
                    }
                    if (odd) it->odd = 1;
                    fence_proxy_async_smem();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(C::bVOk + s));
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(C::bItemEmpty + i % kItems));
        }
    } else if (warp < 12) {
        // ------------------------------------------------------------------ softmax
        setmaxnreg_inc<kRegsSoftmax>();
        const int t = (warp - 4) >> 2, q = warp & 3, r = q * 32 + lane;
        const uint32_t trow = tmem + (static_cast<uint32_t>(q * 32) << 16);
        const uint32_t tS = trow + t * 128, tO = trow + 256 + t * D;
        const float c = a.scale * kLog2e;
        const uint64_t c2 = f2_pack(c, c);
        const int my_tok = r / a.group;   // within the tile
        float2 *stat = reinterpret_cast<float2 *>(sm + C::kStat);
        uint32_t ns = 0, no = 0;   // score tiles read, items finished
        bool ok = true;
        for (uint32_t i = 0; ok; ++i) {
            if (!warp_wait(item_bar(i), (i / kItems) & 1)) { ok = false; break; }
            const volatile Item *it = &items[i % kItems];
            if (it->last) break;
            const int n = t == 0 ? it->n0 : it->n1;
            const bool duo = !TREE && it->duo;
            const int tok0 = it->tok0 + (ALT || duo ? 0 : t * x.tpt);
            const int rows = min(x.tpt, it->tokens - tok0) * a.group;
            const bool mine = r < rows;
            const bool active = q * 32 < rows;      // some row of the warp
            const int tok = mine ? tok0 + my_tok : tok0;
            const int k0 = it->k0, masked = TREE ? it->masked : (tok0 + 1) >> 7, len = it->len;
            const uint64_t bits = TREE ? tree_bits(a, it->start, tok, it->tokens) : 0;
            float m = -INFINITY, l = 0.f;
            for (int j = 0; j < n; ++j) {
                if (!warp_wait(bar(C::bSFull + t), ns & 1)) { ok = false; break; }
                ++ns;
                tc_fence_after();
                if (active) {
                    const int kt = k0 + (ALT ? 2 * j + t : j);
                    uint64_t sum = f2_pack(0.f, 0.f), sum2 = sum;
                    // maximum of 32 scores; 2^(c s - m) of 32 scores, to P
                    auto maximum = [&](const uint32_t (&s)[32]) -> float {
                        float u[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) u[e] = fmaxf(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1]));
#pragma unroll
                        for (int e = 8; e < 32; e += 2)
                            u[e >> 1 & 3] = fmax3(u[e >> 1 & 3], __uint_as_float(s[e]), __uint_as_float(s[e + 1]));
                        return fmaxf(fmax3(u[0], u[1], u[2]), u[3]);
                    };
                    auto exponentials = [&](int h, const uint32_t (&s)[32], uint64_t off) {
                        uint32_t pk[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const float2 y = f2_unpack(f2_fma(f2_pack(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1])), c2, off));
                            const float p0 = ex2_approx(y.x), p1 = ex2_approx(y.y);
                            if (e & 1) sum = f2_add(sum, f2_pack(p0, p1));
                            else sum2 = f2_add(sum2, f2_pack(p0, p1));
                            pk[e] = pack_bf16x2(p0, p1);
                        }
                        tmem_st16(tS + h * 16, pk);   // over scores that have been read
                    };
                    auto rescale = [&](float mx) {
                        const bool grow = mx > m + kGrow;
                        if (!__any_sync(0xffffffffu, grow)) return;
                        const float to = grow ? mx : m;
                        const float alpha = grow ? ex2_approx(m - to) : 1.0f;
                        l *= alpha;
                        m = to;
                        if (j > 0) {   // P V of the tiles before is complete: S of this one came behind it
#pragma unroll 1
                            for (int h = 0; h < D / 16; ++h) {
                                uint32_t o[16];
                                tmem_ld16(tO + h * 16, o);
                                tmem_ld_wait();
#pragma unroll
                                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                                tmem_st16(tO + h * 16, o);
                            }
                        }
                    };
                    auto seen_of = [&](int h) -> uint32_t {
                        const int first = kt * 128 + h * 32;
                        return TREE ? seen_tree(bits, len, first) : seen_causal(tok, first);
                    };
                    auto conceal = [&](uint32_t w, uint32_t (&s)[32]) {
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (!(w >> e & 1u)) s[e] = 0xff800000u;
                    };
                    // The quarters of the tile in front of `quarters` hold every key that some row of the warp sees.
                    int quarters = 4;
                    if (!ALT && kt >= masked) {
#pragma unroll
                        for (int h = 3; h >= 0; --h)
                            if (quarters == h + 1 && __all_sync(0xffffffffu, seen_of(h) == 0u)) quarters = h;
                    }
                    if (!ALT && kt < masked) {
                        // A tile that all rows see: its scores at once in registers, in one piece of straight code. Branches in it,
                        // for masks too, cost more in lost overlap than they save (2.15 against 1.83 ms for 32768 tokens with
                        // masks and skipped quarters here).
                        uint32_t s[4][32];
#pragma unroll
                        for (int h = 0; h < 4; ++h) tmem_ld32(tS + h * 32, s[h]);
                        tmem_ld_wait();
                        rescale(fmaxf(fmax3(maximum(s[0]), maximum(s[1]), maximum(s[2])), maximum(s[3])) * c);
                        const float ref = m == -INFINITY ? 0.f : m;
                        const uint64_t off = f2_pack(-ref, -ref);
#pragma unroll
                        for (int h = 0; h < 4; ++h) exponentials(h, s[h], off);
                    } else {
                        // Diagonal tiles, and ALT, which waits for memory: 32 scores at a time, twice, without the quarters that
                        // no row sees (256 short prompts: 88 -> 69 us)
                        auto read = [&](int h, uint32_t (&s)[32]) {
                            if (P16) {
                                // rows 0-7 and rows 8-15 of two pages, put in the keys' order
                                uint32_t lo[16], hi[16];
                                tmem_ld16(tS + h * 16, lo);
                                tmem_ld16(tS + 64 + h * 16, hi);
                                tmem_ld_wait();
#pragma unroll
                                for (int e = 0; e < 8; ++e) {
                                    s[e] = lo[e];
                                    s[8 + e] = hi[e];
                                    s[16 + e] = lo[8 + e];
                                    s[24 + e] = hi[8 + e];
                                }
                            } else {
                                tmem_ld32(tS + h * 32, s);
                                tmem_ld_wait();
                            }
                            if (kt >= masked) {
                                const uint32_t w = seen_of(h);
                                if (!__all_sync(0xffffffffu, w == 0xffffffffu)) conceal(w, s);
                            }
                        };
                        float top = -INFINITY;
#pragma unroll 1
                        for (int h = 0; h < quarters; ++h) {
                            uint32_t s[32];
                            read(h, s);
                            top = fmaxf(top, maximum(s));
                        }
                        rescale(top * c);
                        const float ref = m == -INFINITY ? 0.f : m;
                        const uint64_t off = f2_pack(-ref, -ref);
#pragma unroll 1
                        for (int h = 0; h < quarters; ++h) {
                            uint32_t s[32];
                            read(h, s);
                            exponentials(h, s, off);
                        }
                        if (!ALT) {
                            uint32_t zero[16];
#pragma unroll
                            for (int e = 0; e < 16; ++e) zero[e] = 0u;
#pragma unroll 1
                            for (int h = quarters; h < 4; ++h) tmem_st16(tS + h * 16, zero);
                        }
                    }
                    const float2 both = f2_unpack(f2_add(sum, sum2));
                    l += both.x + both.y;
                    tmem_st_wait();
                }
                tc_fence_before();
                warp_arrive(bar(C::bPFull + t));
            }
            if (!ok) break;
            if (n > 0) {
                // the epilogue warps take it from here, while this warp begins the next item
                if (no > 0 && !warp_wait(bar(C::bStatFree + t), (no - 1) & 1)) { ok = false; break; }
                ++no;
                stat[t * 128 + r] = make_float2(m, l);
                warp_arrive(bar(C::bStat + t));
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(C::bItemEmpty + i % kItems));
        }
        if (!ok) atomicOr(a.status, kStatusTimeout);
    } else {
        // ------------------------------------------------------------------ epilogue
        setmaxnreg_dec<kRegsOut>();
        const int q = warp & 3, r = q * 32 + lane;
        const uint32_t trow = tmem + (static_cast<uint32_t>(q * 32) << 16);
        const int my_tok = r / a.group, my_head = r - my_tok * a.group;   // within the tile
        const int64_t my_off = my_tok * a.o_tok + my_head * a.o_head;
        // the 16-byte pieces that this thread stores of the warp's 32 rows: piece lane % 8 of rows 4 e + lane / 8
        int64_t piece[ALT ? 1 : 8];
#pragma unroll
        for (int e = 0; e < 8 && !ALT; ++e) {
            const int rr = q * 32 + e * 4 + (lane >> 3), tk = rr / a.group;
            piece[ALT ? 0 : e] = tk * a.o_tok + (rr - tk * a.group) * a.o_head + (lane & 7) * 8;
        }
        const float2 *stat = reinterpret_cast<const float2 *>(sm + C::kStat);
        unsigned char *stage = sm + C::kOut + q * 64 * D;
        constexpr int kPartRows = ALT ? 128 : 256;
        uint32_t done = 0;   // parities, bit t: items of tile t
        bool ok = true;
        for (uint32_t i = 0; ok; ++i) {
            if (!warp_wait(item_bar(i), (i / kItems) & 1)) { ok = false; break; }
            Item *const at = &items[i % kItems];
            const Item &it = *at;
            if (it.last) break;
            const bool join = ALT && it.n1 > 0, duo = !TREE && it.duo;
#pragma unroll 1
            for (int t = 0; t < C::NQ; ++t) {
                if ((t == 0 ? it.n0 : it.n1) == 0) continue;
                // everything that does not depend on the result comes before the wait for it
                const int tok0 = it.tok0 + (ALT || duo ? 0 : t * x.tpt);
                const int rows = min(x.tpt, it.tokens - tok0) * a.group;
                const bool mine = r < rows, active = q * 32 < rows;
                const int tok = tok0 + my_tok;
                const int kh = it.kh + (duo ? t : 0);
                const int64_t tile_off = (static_cast<int64_t>(it.start) + tok0) * a.o_tok + static_cast<int64_t>(kh) * a.group * a.o_head;
                const uint32_t tO = trow + 256 + t * D;
                float *part = nullptr;
                if (TREE && it.slot >= 0) part = tree_slot(a.ws, gridDim.x, it.slot, kPartRows, D);
                const int prow = r + (ALT ? 0 : t * x.tpt * a.group);   // row within the segment
                if (!warp_wait(bar(C::bStat + t), done >> t & 1)) { ok = false; break; }
                const float2 st = stat[t * 128 + r];
                float m = st.x, l = st.y, w0 = 1.f, w1 = 0.f;
                warp_arrive(bar(C::bStatFree + t));
                if (join) {
                    if (!warp_wait(bar(C::bStat + 1), done >> 1 & 1)) { ok = false; break; }
                    const float2 other = stat[128 + r];
                    warp_arrive(bar(C::bStatFree + 1));
                    const float top = fmaxf(m, other.x), ref = top == -INFINITY ? 0.f : top;
                    w0 = ex2_approx(m - ref);
                    w1 = ex2_approx(other.x - ref);
                    l = w0 * l + w1 * other.y;
                    m = top;
                    if (!warp_wait(bar(C::bODone + 1), done >> 1 & 1)) { ok = false; break; }
                    done ^= 2u;
                }
                const float inv = l == 0.f ? 0.f : rcp_approx(l);
                if (!warp_wait(bar(C::bODone + t), done >> t & 1)) { ok = false; break; }
                done ^= 1u << t;
                tc_fence_after();

                // 32 columns of O (of both tiles: ALT)
                auto read = [&](int h, uint32_t (&o)[32]) {
                    __syncwarp();
                    tmem_ld32(tO + h * 32, o);
                    tmem_ld_wait();
                    if (join) {
#pragma unroll
                        for (int g = 0; g < 2; ++g) {
                            uint32_t o1[16];
                            tmem_ld16(tO + D + h * 32 + g * 16, o1);
                            tmem_ld_wait();
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                o[g * 16 + e] = __float_as_uint(w0 * __uint_as_float(o[g * 16 + e]) + w1 * __uint_as_float(o1[e]));
                        }
                    }
                    __syncwarp();
                };
                auto free_o = [&]() {
                    tc_fence_before();
                    warp_arrive(bar(C::bOFree + t));
                    if (join) warp_arrive(bar(C::bOFree + 1));
                };
                if (!active) {
                    free_o();
                } else if (!part && a.out_dtype == 0) {
                    // 64 columns of O / l at a time in bf16
                    __nv_bfloat16 *const tile_out = static_cast<__nv_bfloat16 *>(a.o) + tile_off;
#pragma unroll 1
                    for (int h = 0; h < D / 64; ++h) {
                        uint32_t w[32];
#pragma unroll
                        for (int g = 0; g < 2; ++g) {
                            uint32_t o[32];
                            read(2 * h + g, o);
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                w[g * 16 + e] = pack_bf16x2(__uint_as_float(o[2 * e]) * inv, __uint_as_float(o[2 * e + 1]) * inv);
                        }
                        if (h == D / 64 - 1) free_o();
                        if (!ALT) {
                            // through shared memory: a thread has a row, but a warp's store should cover whole 128-byte pieces
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                *reinterpret_cast<uint4 *>(stage + h * 4096 + lane * 128 + ((e ^ (lane & 7)) << 4)) =
                                    make_uint4(w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
                        } else if (mine) {
                            // few rows: straight from the threads
                            uint4 *dst = reinterpret_cast<uint4 *>(tile_out + my_off + h * 64);
#pragma unroll
                            for (int e = 0; e < 8; ++e) dst[e] = make_uint4(w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
                        }
                    }
                    // the stores come last: the next item waits for O
                    if (!ALT) {
                        __syncwarp();
#pragma unroll 1
                        for (int h = 0; h < D / 64; ++h) {
                            uint4 v[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                const int rr = e * 4 + (lane >> 3);
                                v[e] = *reinterpret_cast<const uint4 *>(stage + h * 4096 + rr * 128 + (((lane & 7) ^ (rr & 7)) << 4));
                            }
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                if (q * 32 + e * 4 + (lane >> 3) < rows)
                                    *reinterpret_cast<uint4 *>(tile_out + piece[ALT ? 0 : e] + h * 64) = v[e];
                        }
                        __syncwarp();
                    }
                } else {
                    // fp32 rows: of the output, or of a piece's numerators
                    float *dst = part ? part + static_cast<int64_t>(prow) * D : static_cast<float *>(a.o) + tile_off + my_off;
                    const float f = part ? 1.f : inv;
#pragma unroll 1
                    for (int h = 0; h < D / 32; ++h) {
                        uint32_t o[32];
                        read(h, o);
                        if (mine) {
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                reinterpret_cast<float4 *>(dst + h * 32)[e] =
                                    make_float4(__uint_as_float(o[4 * e]) * f, __uint_as_float(o[4 * e + 1]) * f,
                                                __uint_as_float(o[4 * e + 2]) * f, __uint_as_float(o[4 * e + 3]) * f);
                        }
                    }
                    __syncwarp();
                    free_o();
                }
                const int64_t out_at = tile_off + my_off;
                const bool odd = *const_cast<const volatile int *>(&at->odd) != 0;
                __syncwarp();
                if (odd && mine) {
                    // values that were replaced by 0: added to what the rows that see them have just been given
                    const uint64_t bits = TREE ? tree_bits(a, it.start, tok, it.tokens) : 0;
                    const int end = min(it.len + it.tokens, it.k1 * 128);
                    for (int key = max(it.masked, it.k0) * 128; key < end; ++key) {
                        const bool sees = TREE ? seen_tree(bits, it.len, key) & 1u : key <= tok;
                        if (!sees) continue;
                        const uint16_t *v;
                        if (TREE) {
                            const int id = a.table[it.kv + (key >> a.page_shift)];
                            if (id < 0 || id >= a.pages) continue;
                            v = static_cast<const uint16_t *>(a.vp) +
                                (((static_cast<int64_t>(id) * a.kv_heads + kh) << a.page_shift) +
                                 (key & ((1 << a.page_shift) - 1))) * D;
                        } else {
                            v = static_cast<const uint16_t *>(a.v) + (it.kv + key) * a.v_tok + kh * a.v_head;
                        }
#pragma unroll 1
                        for (int e = 0; e < D; ++e) {
                            const float f = bf16_bits_to_float(v[e]);
                            if (fabsf(f) < INFINITY) continue;
                            if (part) {
                                part[prow * D + e] += f;
                            } else if (a.out_dtype == 0) {
                                __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(a.o) + out_at + e;
                                *dst = __float2bfloat16_rn(__bfloat162float(*dst) + f);
                            } else {
                                static_cast<float *>(a.o)[out_at + e] += f;
                            }
                        }
                    }
                }
                if (mine) {
                    if (part) {
                        part[kPartRows * D + prow] = m;
                        part[kPartRows * (D + 1) + prow] = l;
                    } else if (a.lse) {
                        a.lse[(static_cast<int64_t>(kh) * a.group + my_head) * a.tokens + it.start + tok] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(C::bItemEmpty + i % kItems));
        }
        if (!ok) atomicOr(a.status, kStatusTimeout);
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ---------------------------------------------------------------------------------------------- host

using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                              const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encoder() {
    static const EncodeFn fn = []() -> EncodeFn {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &r) != cudaSuccess ||
            r != cudaDriverEntryPointSuccess)
            return nullptr;
        return reinterpret_cast<EncodeFn>(p);
    }();
    return fn;
}

// A bf16 tensor map with boxes of 64 columns (128 bytes, 128-byte swizzle). stride: elements of dimensions 1 .. rank-1.
bool make_map(CUtensorMap *map, const void *base, int rank, const int64_t *dims, const int64_t *strides, const int *box) {
    const EncodeFn fn = encoder();
    if (!fn) return false;
    cuuint64_t d[5], s[4];
    cuuint32_t b[5], e[5];
    for (int i = 0; i < rank; ++i) {
        d[i] = static_cast<cuuint64_t>(dims[i]);
        b[i] = static_cast<cuuint32_t>(box[i]);
        e[i] = 1;
        if (i) s[i - 1] = static_cast<cuuint64_t>(strides[i - 1]) * 2;
    }
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void *>(base), d, s, b, e, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool make_rows_map(CUtensorMap *map, const void *base, int d, int heads, int64_t tokens, int64_t head, int64_t token, int box_heads,
                   int box_tokens) {
    const int64_t dims[3] = {d, heads, tokens}, strides[2] = {head, token};
    const int box[3] = {64, box_heads, box_tokens};
    return make_map(map, base, 3, dims, strides, box);
}

template <int D, int MODE>
bool launch(const TcArgs &x, const Maps &maps, int blocks, cudaStream_t st) {
    using C = Cfg<D, MODE>;
    static std::atomic<uint64_t> known{0};
    if (!allow_smem(serve_tc_kernel<D, MODE>, C::kBytes, &known)) return false;
    return launch_dependent(serve_tc_kernel<D, MODE>, dim3(blocks), dim3(kThreads), C::kBytes, st, x, maps);
}

// The list costs an extra launch (about 5 us) and is made only where the order of the items matters.
int prompt_order(int64_t tokens, int64_t seqs, int64_t max_len, int kv_heads, int group, int sms) {
    const int tpt = 128 / group;
    if (seqs <= 1 || prompt_items(tokens, seqs, 2 * tpt * group, group) * kv_heads <= sms) return SCAN;
    return max_len <= tpt ? SINGLES : max_len <= 2 * tpt ? PAIRS : LIST;
}

}  // namespace

size_t prompt_tc_workspace(int64_t tokens, int64_t seqs, int64_t max_len, int kv_heads, int group, int sms) {
    if (group > 128 || prompt_order(tokens, seqs, max_len, kv_heads, group, sms) != LIST) return 0;
    return prompt_plan_bytes(prompt_items(tokens, seqs, 2 * (128 / group) * group, group));
}

int launch_prompt_tc(const ServeArgs &a, cudaStream_t st) {
    if (prompt_is_short(a)) return launch_prompt_short(a, st);
    TcArgs x{};
    x.a = a;
    x.tpt = 128 / a.group;
    const int box_tokens = static_cast<int>(a.max_len < x.tpt ? a.max_len : x.tpt);
    x.box_rows = box_tokens * a.group;
    const int64_t items = prompt_items(a.tokens, a.seqs, 2 * x.tpt * a.group, a.group);
    if (items > 0x7fffffff || a.max_len > (1 << 26)) return -2;   // an item has to end well within the limit of a wait
    x.order = prompt_order(a.tokens, a.seqs, a.max_len, a.kv_heads, a.group, a.sms);
    Maps maps;
    if (!make_rows_map(&maps.q, a.q, a.d, a.heads, a.tokens, a.q_head, a.q_tok, a.group, box_tokens) ||
        !make_rows_map(&maps.k, a.k, a.d, a.kv_heads, a.tokens, a.k_head, a.k_tok, 1, 128) ||
        !make_rows_map(&maps.v, a.v, a.d, a.kv_heads, a.tokens, a.v_head, a.v_tok, 1, 128))
        return -2;
    if (x.order == LIST) {
        if (!launch_prompt_plan(a, 2 * x.tpt * a.group, true, items, st)) return -1;
    }
    const int64_t most = items * a.kv_heads;
    const int blocks = static_cast<int>(most < a.sms ? most : a.sms);
    const bool ok = a.d == 64 ? launch<64, PROMPT>(x, maps, blocks, st) : launch<128, PROMPT>(x, maps, blocks, st);
    return ok ? 1 + (x.order == LIST) : -1;
}

int launch_tree_tc(const ServeArgs &a, cudaStream_t st) {
    TcArgs x{};
    x.a = a;
    x.tpt = 128 / a.group;
    const int box_tokens = a.max_len < x.tpt ? a.max_len : x.tpt;
    x.box_rows = box_tokens * a.group;
    const bool alt = a.max_len <= x.tpt;
    const int page = 1 << a.page_shift;
    const bool p16 = alt && a.d == 128 && page == 16;
    Maps maps;
    const int64_t dims[4] = {a.d, page, a.kv_heads, a.pages};
    const int64_t strides[3] = {a.d, static_cast<int64_t>(a.d) * page, static_cast<int64_t>(a.d) * page * a.kv_heads};
    const int box[4] = {64, page < 128 ? page : 128, 1, 1};
    const int64_t dims16[5] = {64, 16, 2, a.kv_heads, a.pages};
    const int64_t strides16[4] = {128, 64, 128 * 16, static_cast<int64_t>(128) * 16 * a.kv_heads};
    const int box16[5] = {64, 16, 2, 1, 1};
    if (!make_rows_map(&maps.q, a.q, a.d, a.heads, a.tokens, a.q_head, a.q_tok, a.group, box_tokens) ||
        !(p16 ? make_map(&maps.k, a.kp, 5, dims16, strides16, box16) : make_map(&maps.k, a.kp, 4, dims, strides, box)) ||
        !(p16 ? make_map(&maps.v, a.vp, 5, dims16, strides16, box16) : make_map(&maps.v, a.vp, 4, dims, strides, box)))
        return -2;
    bool ok;
    if (p16) ok = launch<128, TREE_ALT16>(x, maps, a.sms, st);
    else if (alt) ok = a.d == 64 ? launch<64, TREE_ALT>(x, maps, a.sms, st) : launch<128, TREE_ALT>(x, maps, a.sms, st);
    else ok = a.d == 64 ? launch<64, TREE_PAIR>(x, maps, a.sms, st) : launch<128, TREE_PAIR>(x, maps, a.sms, st);
    if (!ok) return -1;
    return launch_tree_join(a, a.sms, alt ? 128 : 256, st) ? 2 : -1;
}

}  // namespace ha
