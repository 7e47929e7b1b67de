// ha_serve.cuh -- device helpers of the serving kernels: dependent launches, the walk over packed sequences and the
// partition of the tree attention's key tiles.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "ha_internal.h"

namespace ha {

// A kernel launched with launch_dependent may start before the kernel in front of it on the stream has ended; it calls
// this before it touches memory that the other one reads or writes (returns once that kernel and its writes are done).
__device__ __forceinline__ void grid_dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// From here on the dependent kernel behind this one may take the places that this one leaves free: for kernels that leave
// many, so that the next one's launch and set-up are done when this one ends (a decode step of one user 11.3 -> 10.6 us;
// kernels that fill the device got slower by 5 to 15%, as the next one's blocks then spread unevenly).
__device__ __forceinline__ void allow_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// a / b for 0 <= a, 0 < b: 64-bit division takes some hundred cycles, and nearly all values fit in 32 bits.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
    if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
    return a / b;
}

// Launch behind the previous kernel of the stream without waiting for its last block to drain first (programmatic
// stream serialisation); the kernel must call grid_dependency_wait. True on success.
template <typename... P, typename... A>
inline bool launch_dependent(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t st, A... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...) == cudaSuccess;
}

// Lets a kernel use `bytes` of dynamic shared memory. The attribute is per device and stays: `known` has a bit for each
// device (of the first 64) on which it was set.
template <typename K>
inline bool allow_smem(K kernel, int bytes, std::atomic<uint64_t> *known) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (known->load(std::memory_order_relaxed) & bit) return true;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) return false;
    known->fetch_or(bit, std::memory_order_relaxed);
    return true;
}

// Sequence i of a prompt call: its first row and length; length 0 and a flag where the offsets are not ascending
// rows of the call or the sequence is longer than promised.
__device__ __forceinline__ bool prompt_seq(const ServeArgs &a, int i, int *start, int *len) {
    const int64_t s = a.cu[i], e = a.cu[i + 1];
    const bool ok = s >= 0 && e >= s && e <= a.tokens && e - s <= a.max_len;
    *start = ok ? static_cast<int>(s) : 0;
    *len = ok ? static_cast<int>(e - s) : 0;
    return ok;
}

// The list of a prompt call's items (sequence, index of its group of rows), in the workspace.
struct PromptPlan {
    int count;     // entries
    int single;    // of them, at the end: sequences of one query tile, whose items take two key heads at a time
    int pad[2];
};
int64_t prompt_items(int64_t tokens, int64_t seqs, int64_t rows, int group);
size_t prompt_plan_bytes(int64_t items);
// rows: query rows of an entry (token * group + head); singles_last: sequences of at most rows / 2 come last.
bool launch_prompt_plan(const ServeArgs &a, int64_t rows, bool singles_last, int64_t items, cudaStream_t st);

// Sequence i of a tree call: first query row, drafted rows t, committed rows len, its row of the page table. t = 0
// (and a flag) where something is out of range.
struct TreeSeq {
    int start, t, len;
    int64_t table;
};
__device__ __forceinline__ bool tree_seq(const ServeArgs &a, int i, TreeSeq *x) {
    const int64_t s = a.cu[i], e = a.cu[i + 1];
    const int64_t slot = a.slots ? a.slots[i] : i;
    bool ok = s >= 0 && e >= s && e <= a.tokens && e - s <= a.max_len && slot >= 0 && slot < a.max_slots;
    const int64_t in = ok ? slot : 0;   // loads without a branch: several sequences' are in flight at a time
    const int64_t len = a.lens[in], held = a.held[in];
    const int64_t t = ok ? e - s : 0;
    if (t > 0) ok = len >= 0 && held <= a.max_pages && ((len + t + (int64_t(1) << a.page_shift) - 1) >> a.page_shift) <= held;
    x->start = ok ? static_cast<int>(s) : 0;
    x->t = ok ? static_cast<int>(t) : 0;
    x->len = ok ? static_cast<int>(len) : 0;
    x->table = in * a.max_pages;
    return ok;
}

// A contiguous run of key tiles of one segment (a sequence, a key head and a tile of query rows) that one block works
// on. The segments' key tiles are numbered one segment after the other and cut into equal shares, one per block, so
// that long and short sequences keep every SM busy alike; a segment cut by a share's border is joined afterwards.
struct TreePiece {
    int seq, kh, tile;   // tile: index of the query-row tile
    TreeSeq x;
    int nk;              // key tiles of the segment
    int k0, k1;          // the piece: key tiles [k0, k1)
    int64_t total;       // key tiles of the call
    int shares;          // blocks that have some
    int64_t end;         // number behind the segment's last key tile
};

// Descriptor of a segment that starts in block c and ends in a later one: what the joining kernel needs.
struct TreeJoin {
    int pieces;          // 0: nothing to join for this block
    int start;           // first query row of the sequence
    int row0, rows;      // rows of the tile within the sequence (token * group + head), how many
    int kh;
    int pad[3];
};

// Partial results: slot 2c is the piece that block c continues, slot 2c + 1 the one it begins and does not end.
// A slot has `rows` rows of d fp32 numerators (relative to the row's maximum), then maxima (base 2), then sums; rows is
// the largest number of query rows of a segment.
__host__ __device__ inline size_t tree_slot_floats(int rows, int d) { return static_cast<size_t>(rows) * (d + 2); }

__device__ __forceinline__ TreeJoin *tree_joins(void *ws) { return static_cast<TreeJoin *>(ws); }
__device__ __forceinline__ float *tree_slot(void *ws, int blocks, int slot, int rows, int d) {
    return reinterpret_cast<float *>(static_cast<char *>(ws) + sizeof(TreeJoin) * blocks) +
           slot * tree_slot_floats(rows, d);
}

// The walk of one block over its share, run by one whole warp. rows_per_tile: tokens of a query tile times group (SIMT:
// flattened rows, tok_tile 0) or whole tokens (tok_tile tokens).
struct TreeWalk {
    int64_t total;         // key tiles of the call
    int64_t per_head;      // of one key head
    int shares;            // blocks that get some: no share is empty, so a segment's pieces are in neighbouring blocks
    int64_t at, last;      // this block's next one and the one behind its last
    int kh, seq;           // key head and sequence of `at`
    int64_t seq_first;     // number of the sequence's first key tile
    TreeSeq x;
    TreeSeq lane_seq;      // sequence `lane` where the call has at most 32: each is read once
    int nk, tiles;

    static __device__ __forceinline__ int tiles_of(const ServeArgs &a, const TreeSeq &x, int tile_rows, int tok_tile) {
        return tok_tile ? (x.t + tok_tile - 1) / tok_tile : (x.t * a.group + tile_rows - 1) / tile_rows;
    }
    // key tiles of a sequence for one key head
    static __device__ __forceinline__ int64_t cost(const ServeArgs &a, const TreeSeq &x, int key_tile, int tile_rows,
                                                   int tok_tile) {
        if (x.t == 0) return 0;
        return static_cast<int64_t>(tiles_of(a, x, tile_rows, tok_tile)) * ((x.len + x.t + key_tile - 1) / key_tile);
    }
    __device__ __forceinline__ void begin(const ServeArgs &a, int key_tile, int tile_rows, int tok_tile, int block,
                                          int blocks) {
        const int lane = threadIdx.x & 31;
        per_head = 0;
        bool ok = true;
#pragma unroll 4
        for (int b = 0; b < a.seqs; b += 32) {
            TreeSeq y;
            y.t = 0;
            if (b + lane < a.seqs) ok &= tree_seq(a, b + lane, &y);
            per_head += cost(a, y, key_tile, tile_rows, tok_tile);
            lane_seq = y;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) per_head += __shfl_xor_sync(0xffffffffu, per_head, o);
        if (!ok && block == 0) atomicOr(a.status, kStatusData);
        total = per_head * a.kv_heads;
        shares = static_cast<int>(min(total, static_cast<int64_t>(blocks)));
        at = block < shares ? quotient(total * block, shares) : 0;
        last = block < shares ? quotient(total * (block + 1), shares) : 0;
        kh = 0;
        seq = a.seqs;
        seq_first = 0;
        if (at == last) return;
        kh = static_cast<int>(quotient(at, per_head));
        const int64_t first = at - kh * per_head;
        // the sequence that holds `first`
        int64_t run = 0;
        for (int b = 0; b < a.seqs; b += 32) {
            TreeSeq y = lane_seq;
            if (a.seqs > 32) {
                y.t = 0;
                if (b + lane < a.seqs) tree_seq(a, b + lane, &y);
            }
            const int64_t mine = cost(a, y, key_tile, tile_rows, tok_tile);
            int64_t sum = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t z = __shfl_up_sync(0xffffffffu, sum, o);
                if (lane >= o) sum += z;
            }
            const unsigned hit = __ballot_sync(0xffffffffu, run + sum > first);
            if (hit) {
                const int l = __ffs(hit) - 1;
                seq = b + l;
                seq_first = kh * per_head + run + __shfl_sync(0xffffffffu, sum - mine, l);
                break;
            }
            run += __shfl_sync(0xffffffffu, sum, 31);
        }
        load(a, key_tile, tile_rows, tok_tile);
    }
    __device__ __forceinline__ void load(const ServeArgs &a, int key_tile, int tile_rows, int tok_tile) {
        if (a.seqs > 32) {
            tree_seq(a, seq, &x);
        } else {
            x.start = __shfl_sync(0xffffffffu, lane_seq.start, seq);
            x.t = __shfl_sync(0xffffffffu, lane_seq.t, seq);
            x.len = __shfl_sync(0xffffffffu, lane_seq.len, seq);
            x.table = __shfl_sync(0xffffffffu, lane_seq.table, seq);
        }
        nk = x.t ? (x.len + x.t + key_tile - 1) / key_tile : 0;
        tiles = tiles_of(a, x, tile_rows, tok_tile);
    }
    // The next piece of the share; false at its end. Key heads vary slowest: the blocks of different heads go through
    // the sequences at the same pace, so the heads' parts of a page, which lie together, are read at about the same time.
    // Row tiles of the same keys are neighbours.
    __device__ __forceinline__ bool next(const ServeArgs &a, int key_tile, int tile_rows, int tok_tile, TreePiece *p) {
        if (at >= last) return false;
        while (at - seq_first >= static_cast<int64_t>(tiles) * nk) {
            seq_first += static_cast<int64_t>(tiles) * nk;
            if (++seq >= a.seqs) {
                seq = 0;
                ++kh;
            }
            load(a, key_tile, tile_rows, tok_tile);
        }
        const int64_t off = at - seq_first;
        const int64_t segment = quotient(off, nk);
        p->seq = seq;
        p->x = x;
        p->nk = nk;
        p->tile = static_cast<int>(segment);
        p->kh = kh;
        p->k0 = static_cast<int>(off - segment * nk);
        const int64_t left = last - at;
        p->k1 = static_cast<int>(min(static_cast<int64_t>(nk), p->k0 + left));
        p->total = total;
        p->shares = shares;
        p->end = at - p->k0 + nk;
        at += p->k1 - p->k0;
        return true;
    }
};

// Blocks that share the segment of which `p` (begun and not ended by `block`) is the first piece.
__device__ __forceinline__ int tree_pieces(const TreePiece &p, int block) {
    int n = 1;   // the blocks behind it whose share begins before the segment's end
    while (block + n < p.shares && quotient(p.total * (block + n), p.shares) < p.end) ++n;
    return n;
}

// The mask of drafted rows that query token i (of t) sees, bit j for drafted row j.
__device__ __forceinline__ uint64_t tree_bits(const ServeArgs &a, int start, int i, int t) {
    const uint64_t all = t >= 64 ? ~0ull : (1ull << t) - 1;
    if (a.mask) return static_cast<uint64_t>(a.mask[start + i]) & all;
    return (i >= 63 ? ~0ull : (1ull << (i + 1)) - 1) & all;
}

}  // namespace ha
