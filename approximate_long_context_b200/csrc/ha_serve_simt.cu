// ha_serve_simt.cu -- exact softmax attention for serving in fp32 arithmetic: packed prompts (causal, grouped heads)
// and trees of drafted tokens over a paged cache. The path for fp32 tensors, and for bf16 ones when the SIMT family is
// asked for. Also the kernel that joins the tree segments cut by a block's share (both families).
//
// One block: 64 query rows (row = token * group + head within its key head) against 64 keys at a time, one online
// softmax: m' = max(m, max_j x_j), l' = l 2^(m - m') + sum_j 2^(x_j - m'), O' = O 2^(m - m') + sum_j 2^(x_j - m') v_j with
// x_j = scale log2(e) q.k_j; O = O / l, L = (m + log2 l) ln 2. 256 threads, 4 rows x 4 keys each for the scores and
// 4 rows x d/16 columns for the product with V, in packed f32x2 instructions (pairs along d for the scores, so that the
// 16-byte shared loads feed them as they are; pairs of columns for the product): 8 loads for 64 multiply-adds of 32
// lanes. Sums, maxima and numerators are fp32.
//
// A value row of a masked key can hold an infinity or NaN and must not reach the rows that do not see it (0 * inf):
// the load of a tile votes on non-finite values, and a tile with one and a mask takes the product with a select.
//
// What bounds it: shared-memory loads (81% of their rate, the FMA pipes 33% in packed instructions). 8192 tokens, 8 heads on
// 4: 36.7 TFLOP/s at d = 64, 39.2 at d = 128. Decoding over an fp32 cache (32 users x 8192 rows, d = 64) takes
// tree_few_kernel: 165 us (3.25 TB/s) against 317 us here, where 64-row tiles multiply mostly nothing.
#include <math.h>

#include <atomic>

#include "ha_common.cuh"
#include "ha_internal.h"
#include "ha_serve.cuh"

namespace ha {
namespace {

constexpr int kBM = 64, kBN = 64, kThreads = 256;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLog2e = 1.4426950408889634f;

template <typename T>
__device__ __forceinline__ float4 load4(const T *p);
template <>
__device__ __forceinline__ float4 load4<float>(const float *p) {
    return *reinterpret_cast<const float4 *>(p);
}
template <>
__device__ __forceinline__ float4 load4<uint16_t>(const uint16_t *p) {
    const uint2 r = *reinterpret_cast<const uint2 *>(p);
    return make_float4(__uint_as_float(r.x << 16), __uint_as_float(r.x & 0xffff0000u), __uint_as_float(r.y << 16),
                       __uint_as_float(r.y & 0xffff0000u));
}

__device__ __forceinline__ bool finite4(float4 v) {
    // |v| < inf is false for infinities and NaN
    return fabsf(v.x) < INFINITY && fabsf(v.y) < INFINITY && fabsf(v.z) < INFINITY && fabsf(v.w) < INFINITY;
}

__device__ __forceinline__ void copy16(float *dst, const float *src, bool ok) {
    const int n = ok ? 16 : 0;   // 0: zeros are written, nothing is read
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(n) : "memory");
}

template <int D, typename T>
struct Smem {
    // fp32 at d = 64: the next tile comes with asynchronous copies while one is worked on, with two blocks per SM still
    static constexpr bool kAsync = D == 64 && sizeof(T) == 4;
    static constexpr int LD = D + 4;      // row pitch: 16-byte aligned, eight consecutive rows on different banks
    static constexpr int LP = kBN + 4;
    static constexpr int kQ = 0;
    static constexpr int kK = kBM * LD;   // P overwrites K once the scores are done
    static constexpr int kV = kK + kBN * LD;
    static constexpr int kStage = 2 * kBN * LD;   // K and V of a tile
    static constexpr int kFloats = kK + (kAsync ? 2 : 1) * kStage;
    static constexpr int kBytes = kFloats * 4;
    static_assert(kBM * LP <= kBN * LD, "P fits in K's place");
};

// What one block works on: rows [row0, row0 + rows) of sequence rows, key head kh, key tiles [k0, k1).
struct Work {
    int start, t, len;    // first query row, query tokens, keys in front of the first query token (prompt: 0)
    int row0, rows, kh;
    int k0, k1;
    int64_t table;
};

template <int D, bool TREE, typename T>
__device__ __forceinline__ void attend(const ServeArgs &a, const Work &w, float *sm, float (&acc)[4][D / 16], float (&m)[4],
                                       float (&l)[4]) {
    using S = Smem<D, T>;
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    float *Qs = sm + S::kQ, *Ks = sm + S::kK, *Vs = sm + S::kV;
    const float c = a.scale * kLog2e;
    const T *q = static_cast<const T *>(a.q);
    const bool busy = (tid >> 5) * 8 < w.rows;   // some row of the warp
    __syncthreads();   // the previous piece's reads are done
    for (int x = tid; x < kBM * (D / 4); x += kThreads) {
        const int r = x / (D / 4), col = (x % (D / 4)) * 4;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r < w.rows) {
            const int row = w.row0 + r, tok = row / a.group, head = w.kh * a.group + row - tok * a.group;
            v = load4<T>(q + static_cast<int64_t>(w.start + tok) * a.q_tok + static_cast<int64_t>(head) * a.q_head + col);
        }
        *reinterpret_cast<float4 *>(Qs + r * S::LD + col) = v;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
#pragma unroll
        for (int j = 0; j < D / 16; ++j) acc[i][j] = 0.f;
    }
    int tok[4];
    uint64_t bits[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = min(w.rows - 1, ty * 4 + i);
        tok[i] = (w.row0 + r) / a.group;
        bits[i] = TREE ? tree_bits(a, w.start, tok[i], w.t) : 0;
    }
    const int keys = w.len + w.t;
    // the first key that some row of the tile does not see
    const int masked_from = TREE ? w.len : w.row0 / a.group + 1;
    constexpr int kPer = kThreads / (D / 4);   // rows per turn of the block
    const int col = (tid % (D / 4)) * 4;
    // where this thread's piece of a key's K and V rows lies; false: zeros
    auto place = [&](int key, int64_t *ko, int64_t *vo) -> bool {
        if (key >= keys) return false;
        if (TREE) {
            const int32_t page = a.table[w.table + (key >> a.page_shift)];
            if (page < 0 || page >= a.pages) {
                atomicOr(a.status, kStatusData);
                return false;
            }
            *ko = *vo = (((static_cast<int64_t>(page) * a.kv_heads + w.kh) << a.page_shift) +
                         (key & ((1 << a.page_shift) - 1))) * D + col;
        } else {
            const int64_t row = w.start + key;
            *ko = row * a.k_tok + w.kh * a.k_head + col;
            *vo = row * a.v_tok + w.kh * a.v_head + col;
        }
        return true;
    };
    const T *kp = static_cast<const T *>(TREE ? a.kp : a.k), *vp = static_cast<const T *>(TREE ? a.vp : a.v);
    auto copy = [&](int kt, int stage) {   // kAsync
        if (kt < w.k1) {
#pragma unroll
            for (int r = tid / (D / 4); r < kBN; r += kPer) {
                int64_t ko = 0, vo = 0;
                const bool ok = place(kt * kBN + r, &ko, &vo);
                float *to = sm + S::kK + stage * S::kStage + r * S::LD + col;
                copy16(to, reinterpret_cast<const float *>(kp) + ko, ok);
                copy16(to + kBN * S::LD, reinterpret_cast<const float *>(vp) + vo, ok);
            }
        }
        cp_async_commit();
    };
    if (S::kAsync) copy(w.k0, 0);
    for (int kt = w.k0; kt < w.k1; ++kt) {
        const int base = kt * kBN;
        bool odd = false;
        if (S::kAsync) {
            Ks = sm + S::kK + ((kt - w.k0) & 1) * S::kStage;
            Vs = Ks + kBN * S::LD;
            cp_async_wait<0>();
#pragma unroll
            for (int r = tid / (D / 4); r < kBN; r += kPer) odd |= !finite4(*reinterpret_cast<const float4 *>(Vs + r * S::LD + col));
        } else {
            __syncthreads();   // the previous tile's P and V have been read
            // some rows' pieces of K and V in flight per thread (one after the other, a tile took eight memory latencies)
            constexpr int kBatch = D == 64 ? 4 : 2;
            for (int r0 = tid / (D / 4); r0 < kBN; r0 += kPer * kBatch) {
                float4 kv[kBatch], vv[kBatch];
                int64_t ko[kBatch], vo[kBatch];
                bool ok[kBatch];
#pragma unroll
                for (int u = 0; u < kBatch; ++u) ok[u] = place(base + r0 + u * kPer, &ko[u], &vo[u]);
#pragma unroll
                for (int u = 0; u < kBatch; ++u) {
                    kv[u] = vv[u] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (ok[u]) {
                        kv[u] = load4<T>(kp + ko[u]);
                        vv[u] = load4<T>(vp + vo[u]);
                    }
                }
#pragma unroll
                for (int u = 0; u < kBatch; ++u) {
                    const int r = r0 + u * kPer;
                    odd |= !finite4(vv[u]);
                    *reinterpret_cast<float4 *>(Ks + r * S::LD + col) = kv[u];
                    *reinterpret_cast<float4 *>(Vs + r * S::LD + col) = vv[u];
                }
            }
        }
        float *Ps = Ks;
        const bool masked = base + kBN > masked_from || base + kBN > keys;
        const bool select = __syncthreads_or(odd) && masked;
        if (S::kAsync) copy(kt + 1, (kt + 1 - w.k0) & 1);   // the other stage's P and V have been read
        // two partial sums per score, over the even and the odd of the d products, in packed instructions
        uint64_t s2[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) s2[i][j] = 0;
#pragma unroll 4
        for (int k = 0; k < D && busy; k += 4) {
            ulonglong2 kf[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) kf[j] = *reinterpret_cast<const ulonglong2 *>(Ks + (tx + 16 * j) * S::LD + k);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const ulonglong2 qf = *reinterpret_cast<const ulonglong2 *>(Qs + (ty * 4 + i) * S::LD + k);
#pragma unroll
                for (int j = 0; j < 4; ++j) s2[i][j] = f2_fma(qf.y, kf[j].y, f2_fma(qf.x, kf[j].x, s2[i][j]));
            }
        }
        float s[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 v = f2_unpack(s2[i][j]);
                s[i][j] = v.x + v.y;
            }
        __syncthreads();   // K has been read: P may take its place
        if (!busy) continue;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float top = -INFINITY;
            unsigned seen = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int key = base + tx + 16 * j;
                bool see;
                if (TREE) see = key < w.len || (key < keys && (bits[i] >> (key - w.len) & 1));
                else see = key <= tok[i];
                seen |= static_cast<unsigned>(see || !masked) << j;
                s[i][j] *= c;
                if (seen >> j & 1) top = fmaxf(top, s[i][j]);
            }
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            const float mn = fmaxf(m[i], top);
            const float ref = mn == -INFINITY ? 0.f : mn;   // nothing seen so far: no -inf - -inf
            const float corr = exp2f(m[i] - ref);
            m[i] = mn;
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float p = seen >> j & 1 ? exp2f(s[i][j] - ref) : 0.f;
                sum += p;
                Ps[(ty * 4 + i) * S::LP + tx + 16 * j] = p;
            }
            l[i] = l[i] * corr + sum;
#pragma unroll
            for (int j = 0; j < D / 16; ++j) acc[i][j] *= corr;
        }
        __syncwarp();   // a row's P is written and read by the same half warp
        if (!select) {
#pragma unroll 2
            for (int k = 0; k < kBN; k += 4) {
                float4 p[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) p[i] = *reinterpret_cast<const float4 *>(Ps + (ty * 4 + i) * S::LP + k);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                    uint64_t pp[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float pk = kk == 0 ? p[i].x : kk == 1 ? p[i].y : kk == 2 ? p[i].z : p[i].w;
                        pp[i] = f2_pack(pk, pk);
                    }
#pragma unroll
                    for (int g = 0; g < D / 64; ++g) {
                        const ulonglong2 v = *reinterpret_cast<const ulonglong2 *>(Vs + (k + kk) * S::LD + g * 64 + tx * 4);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            uint64_t *o = reinterpret_cast<uint64_t *>(&acc[i][g * 4]);
                            o[0] = f2_fma(pp[i], v.x, o[0]);
                            o[1] = f2_fma(pp[i], v.y, o[1]);
                        }
                    }
                }
            }
        } else {
            for (int k = 0; k < kBN; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float pk = Ps[(ty * 4 + i) * S::LP + k];
#pragma unroll
                    for (int g = 0; g < D / 64; ++g)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float v = Vs[k * S::LD + g * 64 + tx * 4 + e];
                            if (pk != 0.f) acc[i][g * 4 + e] = fmaf(pk, v, acc[i][g * 4 + e]);
                        }
                }
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], o);
}

// O = numerator / sum; a row that sees nothing (sum 0) is 0 with L = -inf.
template <int D>
__device__ __forceinline__ void write_rows(const ServeArgs &a, const Work &w, const float (&acc)[4][D / 16],
                                           const float (&m)[4], const float (&l)[4]) {
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = ty * 4 + i;
        if (r >= w.rows) continue;
        const int row = w.row0 + r, tok = row / a.group, head = w.kh * a.group + row - tok * a.group;
        const int64_t at = static_cast<int64_t>(w.start + tok) * a.o_tok + static_cast<int64_t>(head) * a.o_head;
        const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];
#pragma unroll
        for (int g = 0; g < D / 64; ++g) {
            float o[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) o[e] = l[i] == 0.f ? 0.f : acc[i][g * 4 + e] * inv;
            const int64_t x = at + g * 64 + tx * 4;
            if (a.out_dtype == 0) {
                const __nv_bfloat162 lo = __floats2bfloat162_rn(o[0], o[1]), hi = __floats2bfloat162_rn(o[2], o[3]);
                uint2 u;
                u.x = *reinterpret_cast<const uint32_t *>(&lo);
                u.y = *reinterpret_cast<const uint32_t *>(&hi);
                *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(a.o) + x) = u;
            } else {
                *reinterpret_cast<float4 *>(static_cast<float *>(a.o) + x) = make_float4(o[0], o[1], o[2], o[3]);
            }
        }
        if (a.lse && tx == 0)
            a.lse[static_cast<int64_t>(head) * a.tokens + w.start + tok] =
                l[i] == 0.f ? -INFINITY : (m[i] + log2f(l[i])) * kLn2;
    }
}

// Block b: key head b mod kv_heads of the (b / kv_heads)-th 64-row tile. The tiles are numbered by falling position in
// their sequence (the expensive ones start first). Up to 32 sequences the block finds its tile itself: with N(p) = sum over
// the sequences of max(0, tiles - p), tile t has the position p with N(p + 1) <= t < N(p), found by bisection. Beyond that
// the tiles come from a list.
template <int D, typename T>
__global__ void __launch_bounds__(kThreads, 2) prompt_simt_kernel(const ServeArgs a, bool listed) {
    extern __shared__ __align__(16) float sm[];
    __shared__ Work shared;
    grid_dependency_wait();
    const int kh = static_cast<int>(blockIdx.x % a.kv_heads);
    const int64_t want = blockIdx.x / a.kv_heads;
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        int found = -1, p = 0;
        if (listed) {
            const PromptPlan *plan = static_cast<const PromptPlan *>(a.ws);
            if (want < plan->count) {
                const int2 e = reinterpret_cast<const int2 *>(plan + 1)[want];
                found = e.x;
                p = e.y;
            }
        } else {
            int start = 0, len = 0;
            const bool ok = lane >= a.seqs || prompt_seq(a, lane, &start, &len);
            if (!ok && blockIdx.x == 0) atomicOr(a.status, kStatusData);
            const int tiles = static_cast<int>((static_cast<int64_t>(len) * a.group + kBM - 1) / kBM);
            auto from = [&](int q) -> int64_t {   // N(q)
                int64_t n = tiles > q ? tiles - q : 0;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
                return n;
            };
            if (want < from(0)) {
                int lo = 0, hi = static_cast<int>((static_cast<int64_t>(a.max_len) * a.group + kBM - 1) / kBM);   // N(hi) = 0
                while (hi - lo > 1) {
                    const int mid = (lo + hi) >> 1;
                    if (from(mid) > want) lo = mid;
                    else hi = mid;
                }
                p = lo;
                const unsigned has = __ballot_sync(0xffffffffu, tiles > p);
                found = __fns(has, 0, static_cast<int>(want - from(p + 1)) + 1);
            }
        }
        if (lane == 0) {
            Work w{};
            w.rows = 0;
            if (found >= 0) {
                int start, len;
                prompt_seq(a, found, &start, &len);
                w.start = start;
                w.t = len;
                w.len = 0;
                w.row0 = p * kBM;
                w.rows = min(kBM, len * a.group - w.row0);
                w.kh = kh;
                w.k0 = 0;
                w.k1 = ((w.row0 + w.rows - 1) / a.group) / kBN + 1;
            }
            shared = w;
        }
    }
    __syncthreads();
    const Work w = shared;
    if (w.rows <= 0) return;
    float acc[4][D / 16], m[4], l[4];
    attend<D, false, T>(a, w, sm, acc, m, l);
    write_rows<D>(a, w, acc, m, l);
}

template <int D, typename T>
__global__ void __launch_bounds__(kThreads, 2) tree_simt_kernel(const ServeArgs a) {
    extern __shared__ __align__(16) float sm[];
    __shared__ TreePiece piece;
    __shared__ int more;
    allow_dependents();
    grid_dependency_wait();
    TreeWalk walk;
    const int warp = threadIdx.x >> 5, blocks = gridDim.x, block = blockIdx.x;
    if (warp == 0) walk.begin(a, kBN, kBM, 0, block, blocks);
    if (threadIdx.x == 0) tree_joins(a.ws)[block].pieces = 0;
    for (;;) {
        __syncthreads();
        if (warp == 0) {
            TreePiece p;
            const bool got = walk.next(a, kBN, kBM, 0, &p);
            if (threadIdx.x == 0) {
                piece = p;
                more = got;
            }
        }
        __syncthreads();
        if (!more) break;
        Work w;
        w.start = piece.x.start;
        w.t = piece.x.t;
        w.len = piece.x.len;
        w.table = piece.x.table;
        w.row0 = piece.tile * kBM;
        w.rows = min(kBM, w.t * a.group - w.row0);
        w.kh = piece.kh;
        w.k0 = piece.k0;
        w.k1 = piece.k1;
        float acc[4][D / 16], m[4], l[4];
        attend<D, true, T>(a, w, sm, acc, m, l);
        if (piece.k0 == 0 && piece.k1 == piece.nk) {
            write_rows<D>(a, w, acc, m, l);
            continue;
        }
        const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
        float *slot = tree_slot(a.ws, blocks, 2 * block + (piece.k0 == 0), kBM, D);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = ty * 4 + i;
            if (r >= w.rows) continue;
#pragma unroll
            for (int g = 0; g < D / 64; ++g)
                *reinterpret_cast<float4 *>(slot + r * D + g * 64 + tx * 4) =
                    make_float4(acc[i][g * 4], acc[i][g * 4 + 1], acc[i][g * 4 + 2], acc[i][g * 4 + 3]);
            if (tx == 0) {
                slot[kBM * D + r] = m[i];
                slot[kBM * (D + 1) + r] = l[i];
            }
        }
        if (piece.k0 == 0 && threadIdx.x == 0) {
            TreeJoin j{};
            j.pieces = tree_pieces(piece, block);
            j.start = w.start;
            j.row0 = w.row0;
            j.rows = w.rows;
            j.kh = w.kh;
            tree_joins(a.ws)[block] = j;
        }
    }
}

// ---- few rows: decoding and small trees over an fp32 cache
//
// At most 16 query rows, so reading the cache bounds it: tiles of 64 keys come with asynchronous copies, one ahead, and each
// of the eight warps takes eight keys of a tile with a softmax of its own (no exchange between warps until the piece
// ends). Scores: a lane has one row and two keys; product with V: a lane has d/32 columns of all rows.
constexpr int kFewRows = 16, kWarps = kThreads / 32, kMine = kBN / kWarps;

template <int D>
struct Few {
    static constexpr int LD = D + 4;
    static constexpr int kQ = 0;
    static constexpr int kKV = kFewRows * LD;              // two stages of K, then V
    static constexpr int kTile = kBN * LD;
    static constexpr int kP = kKV + 4 * kTile;             // [warp][key][row]
    static constexpr int kStat = kP + kWarps * kMine * 20; // [warp][row] maximum, sum
    static constexpr int kFloats = kStat + kWarps * kFewRows * 2;
    static constexpr int kBytes = kFloats * 4;
    static_assert(kWarps * kFewRows * D <= 4 * kTile, "the warps' numerators fit in the tiles' place");
};

template <int D>
__global__ void __launch_bounds__(kThreads) tree_few_kernel(const ServeArgs a) {
    using F = Few<D>;
    constexpr int C = D / 32, kPer = kThreads / (D / 4), kTurns = kBN / kPer;
    extern __shared__ __align__(16) float sm[];
    __shared__ TreePiece piece;
    __shared__ int more;
    allow_dependents();
    grid_dependency_wait();
    TreeWalk walk;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, blocks = gridDim.x, block = blockIdx.x;
    const int col = (tid % (D / 4)) * 4, row0 = tid / (D / 4);
    const float c = a.scale * kLog2e;
    float *Qs = sm + F::kQ, *Ps = sm + F::kP + warp * kMine * 20;
    float2 *stat = reinterpret_cast<float2 *>(sm + F::kStat);
    if (warp == 0) walk.begin(a, kBN, kBM, 0, block, blocks);
    if (tid == 0) tree_joins(a.ws)[block].pieces = 0;
    for (;;) {
        __syncthreads();
        if (warp == 0) {
            TreePiece p;
            const bool got = walk.next(a, kBN, kBM, 0, &p);
            if (tid == 0) {
                piece = p;
                more = got;
            }
        }
        __syncthreads();
        if (!more) break;
        const TreePiece w = piece;
        const int rows = w.x.t * a.group, keys = w.x.len + w.x.t;
        // pages of this thread's rows of a tile, and the copies of the tile into a stage
        int ids[kTurns];
        auto look = [&](int kt) {
#pragma unroll
            for (int u = 0; u < kTurns; ++u) {
                const int key = kt * kBN + row0 + u * kPer;
                ids[u] = kt < w.k1 && key < keys ? a.table[w.x.table + (key >> a.page_shift)] : -1;
            }
        };
        auto copy = [&](int kt, int stage) {
            float *Kd = sm + F::kKV + stage * 2 * F::kTile, *Vd = Kd + F::kTile;
            if (kt < w.k1) {
#pragma unroll
                for (int u = 0; u < kTurns; ++u) {
                    const int r = row0 + u * kPer, key = kt * kBN + r;
                    const bool ok = key < keys && ids[u] >= 0 && ids[u] < a.pages;
                    if (key < keys && !ok) atomicOr(a.status, kStatusData);
                    const int64_t at = ok ? (((static_cast<int64_t>(ids[u]) * a.kv_heads + w.kh) << a.page_shift) +
                                             (key & ((1 << a.page_shift) - 1))) * D + col
                                          : 0;
                    copy16(Kd + r * F::LD + col, static_cast<const float *>(a.kp) + at, ok);
                    copy16(Vd + r * F::LD + col, static_cast<const float *>(a.vp) + at, ok);
                }
            }
            cp_async_commit();
        };
        look(w.k0);
        copy(w.k0, 0);
        look(w.k0 + 1);
        for (int x = tid; x < kFewRows * (D / 4); x += kThreads) {
            const int r = x / (D / 4), cc = (x % (D / 4)) * 4;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < rows) {
                const int tok = r / a.group, head = w.kh * a.group + r - tok * a.group;
                v = load4<float>(static_cast<const float *>(a.q) + static_cast<int64_t>(w.x.start + tok) * a.q_tok +
                                 static_cast<int64_t>(head) * a.q_head + cc);
            }
            *reinterpret_cast<float4 *>(Qs + r * F::LD + cc) = v;
        }
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, acc[kFewRows][C];
        uint64_t bits[2];
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            const int r = g * 8 + (lane >> 2);
            bits[g] = tree_bits(a, w.x.start, min(r, rows - 1) / a.group, w.x.t);
        }
#pragma unroll
        for (int r = 0; r < kFewRows; ++r)
#pragma unroll
            for (int e = 0; e < C; ++e) acc[r][e] = 0.f;
        const int groups = rows > 8 ? 2 : 1;
        for (int kt = w.k0; kt < w.k1; ++kt) {
            const int stage = (kt - w.k0) & 1;
            copy(kt + 1, stage ^ 1);
            look(kt + 2);
            cp_async_wait<1>();
            __syncthreads();   // the tile is there for all warps
            const float *Ks = sm + F::kKV + stage * 2 * F::kTile + warp * kMine * F::LD, *Vs = Ks + F::kTile;
            const int first = kt * kBN + warp * kMine;
            const bool masked = first + kMine > w.x.len;
            float alpha[2] = {1.f, 1.f};
            if (first < keys) {
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    if (g >= groups) continue;
                    const int r = g * 8 + (lane >> 2), k2 = (lane & 3) * 2;
                    uint64_t s0 = 0, s1 = 0, t0 = 0, t1 = 0;
#pragma unroll 8
                    for (int d = 0; d < D; d += 4) {
                        const ulonglong2 q = *reinterpret_cast<const ulonglong2 *>(Qs + r * F::LD + d);
                        const ulonglong2 ka = *reinterpret_cast<const ulonglong2 *>(Ks + k2 * F::LD + d);
                        const ulonglong2 kb = *reinterpret_cast<const ulonglong2 *>(Ks + (k2 + 1) * F::LD + d);
                        s0 = f2_fma(q.x, ka.x, s0);
                        t0 = f2_fma(q.y, ka.y, t0);
                        s1 = f2_fma(q.x, kb.x, s1);
                        t1 = f2_fma(q.y, kb.y, t1);
                    }
                    const float2 u0 = f2_unpack(f2_add(s0, t0)), u1 = f2_unpack(f2_add(s1, t1));
                    float x0 = (u0.x + u0.y) * c, x1 = (u1.x + u1.y) * c;
                    const int key = first + k2;
                    const bool see0 = key < w.x.len || (key < keys && (bits[g] >> (key - w.x.len) & 1));
                    const bool see1 = key + 1 < w.x.len || (key + 1 < keys && (bits[g] >> (key + 1 - w.x.len) & 1));
                    float top = fmaxf(see0 ? x0 : -INFINITY, see1 ? x1 : -INFINITY);
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                    const float mn = fmaxf(m[g], top), ref = mn == -INFINITY ? 0.f : mn;
                    alpha[g] = exp2f(m[g] - ref);
                    m[g] = mn;
                    x0 = see0 ? exp2f(x0 - ref) : 0.f;
                    x1 = see1 ? exp2f(x1 - ref) : 0.f;
                    l[g] = l[g] * alpha[g] + x0 + x1;
                    Ps[k2 * 20 + r] = x0;
                    Ps[(k2 + 1) * 20 + r] = x1;
                }
                __syncwarp();
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    if (g >= groups) continue;
                    if (__any_sync(0xffffffffu, alpha[g] != 1.f)) {
#pragma unroll
                        for (int r = 0; r < 8; ++r) {
                            const float f = __shfl_sync(0xffffffffu, alpha[g], r * 4);
#pragma unroll
                            for (int e = 0; e < C; ++e) acc[g * 8 + r][e] *= f;
                        }
                    }
#pragma unroll
                    for (int k = 0; k < kMine; ++k) {
                        float v[C];
                        if (C == 4) *reinterpret_cast<float4 *>(v) = *reinterpret_cast<const float4 *>(Vs + k * F::LD + lane * 4);
                        else *reinterpret_cast<float2 *>(v) = *reinterpret_cast<const float2 *>(Vs + k * F::LD + lane * 2);
                        const float4 pa = *reinterpret_cast<const float4 *>(Ps + k * 20 + g * 8);
                        const float4 pb = *reinterpret_cast<const float4 *>(Ps + k * 20 + g * 8 + 4);
                        const float p[8] = {pa.x, pa.y, pa.z, pa.w, pb.x, pb.y, pb.z, pb.w};
#pragma unroll
                        for (int r = 0; r < 8; ++r)
#pragma unroll
                            for (int e = 0; e < C; ++e)   // a masked key's value may be no number
                                if (!masked || p[r] != 0.f) acc[g * 8 + r][e] = fmaf(p[r], v[e], acc[g * 8 + r][e]);
                    }
                }
            }
            __syncthreads();   // the stage may be filled again
        }
        // ---- the warps' results joined: numerators to the tiles' place, then one sum per row and column
        float *part = sm + F::kKV;
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            l[g] += __shfl_xor_sync(0xffffffffu, l[g], 1);
            l[g] += __shfl_xor_sync(0xffffffffu, l[g], 2);
            if ((lane & 3) == 0) stat[warp * kFewRows + g * 8 + (lane >> 2)] = make_float2(m[g], l[g]);
        }
#pragma unroll
        for (int r = 0; r < kFewRows; ++r)
            if (r < rows) {
                if (C == 4) *reinterpret_cast<float4 *>(part + (warp * kFewRows + r) * D + lane * 4) = *reinterpret_cast<float4 *>(acc[r]);
                else *reinterpret_cast<float2 *>(part + (warp * kFewRows + r) * D + lane * 2) = *reinterpret_cast<float2 *>(acc[r]);
            }
        __syncthreads();
        const bool whole = w.k0 == 0 && w.k1 == w.nk;
        float *slot = whole ? nullptr : tree_slot(a.ws, blocks, 2 * block + (w.k0 == 0), kFewRows, D);
        for (int x = tid; x < rows * (D / 4); x += kThreads) {
            const int r = x / (D / 4), cc = (x % (D / 4)) * 4;
            float mt = -INFINITY;
#pragma unroll
            for (int i = 0; i < kWarps; ++i) mt = fmaxf(mt, stat[i * kFewRows + r].x);
            const float ref = mt == -INFINITY ? 0.f : mt;
            float lt = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < kWarps; ++i) {
                const float2 st = stat[i * kFewRows + r];
                const float f = exp2f(st.x - ref);
                const float4 v = *reinterpret_cast<const float4 *>(part + (i * kFewRows + r) * D + cc);
                lt = fmaf(f, st.y, lt);
                o[0] = fmaf(f, v.x, o[0]);
                o[1] = fmaf(f, v.y, o[1]);
                o[2] = fmaf(f, v.z, o[2]);
                o[3] = fmaf(f, v.w, o[3]);
            }
            if (slot) {
                *reinterpret_cast<float4 *>(slot + r * D + cc) = make_float4(o[0], o[1], o[2], o[3]);
                if (cc == 0) {
                    slot[kFewRows * D + r] = mt;
                    slot[kFewRows * (D + 1) + r] = lt;
                }
                continue;
            }
            const int tok = r / a.group, head = w.kh * a.group + r - tok * a.group;
            const int64_t at = static_cast<int64_t>(w.x.start + tok) * a.o_tok + static_cast<int64_t>(head) * a.o_head + cc;
            const float inv = lt == 0.f ? 0.f : 1.f / lt;
#pragma unroll
            for (int e = 0; e < 4; ++e) o[e] = lt == 0.f ? 0.f : o[e] * inv;
            if (a.out_dtype == 0) {
                const __nv_bfloat162 lo = __floats2bfloat162_rn(o[0], o[1]), hi = __floats2bfloat162_rn(o[2], o[3]);
                uint2 u;
                u.x = *reinterpret_cast<const uint32_t *>(&lo);
                u.y = *reinterpret_cast<const uint32_t *>(&hi);
                *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(a.o) + at) = u;
            } else {
                *reinterpret_cast<float4 *>(static_cast<float *>(a.o) + at) = make_float4(o[0], o[1], o[2], o[3]);
            }
            if (a.lse && cc == 0)
                a.lse[static_cast<int64_t>(head) * a.tokens + w.x.start + tok] = lt == 0.f ? -INFINITY : (mt + log2f(lt)) * kLn2;
        }
        if (w.k0 == 0 && !whole && tid == 0) {
            TreeJoin j{};
            j.pieces = tree_pieces(w, block);
            j.start = w.x.start;
            j.row0 = 0;
            j.rows = rows;
            j.kh = w.kh;
            tree_joins(a.ws)[block] = j;
        }
    }
}

// Joins the pieces of the segment that block blockIdx.x begins and does not end: one warp per row, the pieces' numerators
// and sums weighted with 2^(m_piece - m). The order is fixed, so equal calls give equal bits.
constexpr int kJoinRows = 4;

template <int D>
__global__ void __launch_bounds__(32 * kJoinRows) tree_join_kernel(const ServeArgs a, int blocks, int rows) {
    allow_dependents();
    grid_dependency_wait();
    const TreeJoin j = tree_joins(a.ws)[blockIdx.x];
    const int r = blockIdx.y * kJoinRows + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (j.pieces == 0 || r >= j.rows) return;
    constexpr int C = D / 32;
    auto slot_of = [&](int i) {
        return tree_slot(a.ws, blocks, i == 0 ? 2 * blockIdx.x + 1 : 2 * (blockIdx.x + i), rows, D);
    };
    // 32 pieces at a time: lane i has the maximum and the sum of piece i, all lanes its numerators, eight pieces in flight.
    // The running result is brought to a new maximum as in the softmax itself.
    float m = -INFINITY, l = 0.f, acc[C];
#pragma unroll
    for (int e = 0; e < C; ++e) acc[e] = 0.f;
    for (int first = 0; first < j.pieces; first += 32) {
        const int n = min(32, j.pieces - first);
        float mi = -INFINITY, li = 0.f;
        if (lane < n) {
            const float *s = slot_of(first + lane);
            mi = s[rows * D + r];
            li = s[rows * (D + 1) + r];
        }
        float top = mi;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        const float mn = fmaxf(m, top), ref = mn == -INFINITY ? 0.f : mn;
        const float back = exp2f(m - ref), w = exp2f(mi - ref);
        m = mn;
        float sum = w * li;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        l = l * back + sum;
#pragma unroll
        for (int e = 0; e < C; ++e) acc[e] *= back;
        for (int b = 0; b < n; b += 8) {
            float v[8][C];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                if (b + u >= n) continue;
                const float *s = slot_of(first + b + u) + r * D;
                if (C == 4) *reinterpret_cast<float4 *>(v[u]) = *reinterpret_cast<const float4 *>(s + lane * 4);
                else *reinterpret_cast<float2 *>(v[u]) = *reinterpret_cast<const float2 *>(s + lane * 2);
            }
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const float wu = __shfl_sync(0xffffffffu, w, (b + u) & 31);
                if (b + u >= n) continue;
#pragma unroll
                for (int e = 0; e < C; ++e) acc[e] = fmaf(wu, v[u][e], acc[e]);
            }
        }
    }
    const int row = j.row0 + r, tok = row / a.group, head = j.kh * a.group + row - tok * a.group;
    const int64_t at = static_cast<int64_t>(j.start + tok) * a.o_tok + static_cast<int64_t>(head) * a.o_head + lane * C;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    if (a.out_dtype == 0) {
#pragma unroll
        for (int e = 0; e < C; e += 2)
            *reinterpret_cast<__nv_bfloat162 *>(static_cast<__nv_bfloat16 *>(a.o) + at + e) =
                __floats2bfloat162_rn(l == 0.f ? 0.f : acc[e] * inv, l == 0.f ? 0.f : acc[e + 1] * inv);
    } else {
#pragma unroll
        for (int e = 0; e < C; ++e) static_cast<float *>(a.o)[at + e] = l == 0.f ? 0.f : acc[e] * inv;
    }
    if (a.lse && lane == 0)
        a.lse[static_cast<int64_t>(head) * a.tokens + j.start + tok] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

template <int D, typename T>
int prompt_simt(const ServeArgs &a, cudaStream_t st) {
    static std::atomic<uint64_t> known{0};
    if (!allow_smem(prompt_simt_kernel<D, T>, Smem<D, T>::kBytes, &known)) return -1;
    const int64_t tiles = prompt_items(a.tokens, a.seqs, kBM, a.group);
    // blocks of a grid; row numbers within a sequence
    if (tiles * a.kv_heads > 0x7fffffff || static_cast<int64_t>(a.max_len) * a.group > 0x7fffff00) return -2;
    const bool listed = a.seqs > 32;
    if (listed && !launch_prompt_plan(a, kBM, false, tiles, st)) return -1;
    const dim3 grid(static_cast<unsigned>(tiles * a.kv_heads));
    return launch_dependent(prompt_simt_kernel<D, T>, grid, dim3(kThreads), Smem<D, T>::kBytes, st, a, listed) ? 1 + listed : -1;
}

template <int D>
int tree_few(const ServeArgs &a, cudaStream_t st) {
    static std::atomic<uint64_t> known{0};
    if (!allow_smem(tree_few_kernel<D>, Few<D>::kBytes, &known)) return -1;
    const int blocks = a.sms * (D == 64 ? 2 : 1);   // by shared memory
    if (!launch_dependent(tree_few_kernel<D>, dim3(blocks), dim3(kThreads), Few<D>::kBytes, st, a)) return -1;
    return launch_tree_join(a, blocks, kFewRows, st) ? 2 : -1;
}

template <int D, typename T>
int tree_simt(const ServeArgs &a, cudaStream_t st) {
    static std::atomic<uint64_t> known{0};
    if (!allow_smem(tree_simt_kernel<D, T>, Smem<D, T>::kBytes, &known)) return -1;
    const int blocks = 2 * a.sms;   // two per SM fit (shared memory)
    if (!launch_dependent(tree_simt_kernel<D, T>, dim3(blocks), dim3(kThreads), Smem<D, T>::kBytes, st, a)) return -1;
    return launch_tree_join(a, blocks, kBM, st) ? 2 : -1;
}

}  // namespace

bool launch_tree_join(const ServeArgs &a, int blocks, int rows, cudaStream_t st) {
    const int used = a.max_len * a.group < rows ? a.max_len * a.group : rows;
    const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>((used + kJoinRows - 1) / kJoinRows));
    return a.d == 64 ? launch_dependent(tree_join_kernel<64>, grid, dim3(32 * kJoinRows), 0, st, a, blocks, rows)
                     : launch_dependent(tree_join_kernel<128>, grid, dim3(32 * kJoinRows), 0, st, a, blocks, rows);
}

size_t serve_prompt_workspace(bool tc, int64_t tokens, int64_t seqs, int64_t max_len, int kv_heads, int group, int sms) {
    if (tc) return prompt_tc_workspace(tokens, seqs, max_len, kv_heads, group, sms);
    return seqs > 32 ? prompt_plan_bytes(prompt_items(tokens, seqs, kBM, group)) : 0;
}

size_t serve_tree_workspace(int sms, int d) {
    // SIMT: two blocks per SM of 64 rows; tensor cores: one of up to 256 rows
    const size_t simt = 2 * static_cast<size_t>(sms) * (sizeof(TreeJoin) + 2 * tree_slot_floats(kBM, d) * sizeof(float));
    const size_t tc = static_cast<size_t>(sms) * (sizeof(TreeJoin) + 2 * tree_slot_floats(256, d) * sizeof(float));
    return simt > tc ? simt : tc;
}

int launch_prompt_simt(const ServeArgs &a, int dtype, cudaStream_t st) {
    if (a.d == 64) return dtype == 0 ? prompt_simt<64, uint16_t>(a, st) : prompt_simt<64, float>(a, st);
    return dtype == 0 ? prompt_simt<128, uint16_t>(a, st) : prompt_simt<128, float>(a, st);
}

int launch_tree_simt(const ServeArgs &a, int dtype, cudaStream_t st) {
    const bool few = dtype != 0 && a.max_len * a.group <= kFewRows;
    if (a.d == 64) return few ? tree_few<64>(a, st) : dtype == 0 ? tree_simt<64, uint16_t>(a, st) : tree_simt<64, float>(a, st);
    return few ? tree_few<128>(a, st) : dtype == 0 ? tree_simt<128, uint16_t>(a, st) : tree_simt<128, float>(a, st);
}

}  // namespace ha
