// ha_serve_short.cu -- attention over short packed prompts (at most 128 tokens), bf16: few of them, where the time of one
// chain counts, and many that are much shorter than a tile.
//
// A block has 64 query rows (token * group + head) of a key head and all keys up to its last token in shared memory; a
// warp has 16 rows and all their scores in registers: S = Q K^T by mma.sync (m16n8k16), a plain softmax, O = P V. No tensor
// maps on the host, no TMEM, no hand-over between warps; several blocks per SM hide one another's loads.
//
// What bounds it: the chain offsets -> rows -> products. One prompt of 77 tokens, 8 heads on 2, d = 64: 4.7 us against 6.9 us
// in the persistent tcgen05 kernel; 256 of up to 32 tokens, 16 heads, d = 64: 26 us against 48; but 256 of up to 128
// tokens: 71 against 52, as mma.sync multiplies at a fraction of tcgen05's rate.
//
// The weights are rounded to bf16 because the tensor core multiplies bf16; the normaliser sums the unrounded values, and the
// exponentials are the hardware's (ex2.approx, a few units in the last place of fp32: far below a weight's rounding).
// Values of keys that a row does not see may be infinities or NaN: in the 16 keys at the diagonal what is not finite is
// taken as 0, and added to the rows that see it.
#include <math.h>

#include <atomic>

#include "ha_common.cuh"
#include "ha_internal.h"
#include "ha_serve.cuh"

namespace ha {
namespace {

constexpr int kRows = 64, kThreads = 128, kMaxKeys = 128;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool ok) {
    const int n = ok ? 16 : 0;   // 0: zeros are written, nothing is read
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void ldsm(uint32_t at, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at)
                 : "memory");
}
__device__ __forceinline__ void ldsm_t(uint32_t at, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at)
                 : "memory");
}
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// An exponent of ones in either half carries into the bit above it.
__device__ __forceinline__ uint32_t bad(uint32_t u) { return ((u & 0x7f807f80u) + 0x00800080u) & 0x80008000u; }

// Byte offset of a 16-byte piece of a row of D values; eight rows' pieces of a column lie on different banks.
template <int D>
__device__ __forceinline__ int at16(int row, int piece) {
    return row * (D * 2) + ((piece ^ (row & 7)) << 4);
}

template <int D>
__global__ void __launch_bounds__(kThreads, D == 64 ? 4 : 2) prompt_short_kernel(const ServeArgs a, int per_seq, int cap) {
    extern __shared__ __align__(128) unsigned char sm[];
    grid_dependency_wait();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t pair = blockIdx.x / per_seq;
    const int kh = static_cast<int>(pair % a.kv_heads), seq = static_cast<int>(pair / a.kv_heads);
    const int row0 = static_cast<int>(blockIdx.x % per_seq) * kRows;
    int start, len;
    if (!prompt_seq(a, seq, &start, &len) && row0 == 0 && kh == 0 && tid == 0) atomicOr(a.status, kStatusData);
    if (row0 >= len * a.group) return;
    const int rows = min(kRows, len * a.group - row0);
    const int keys = (row0 + rows - 1) / a.group + 1;      // up to the last row's own
    const int padded = (keys + 15) & ~15;
    constexpr int kPieces = D / 8;
    const uint32_t qs = smem_u32(sm), ks = qs + kRows * D * 2, vs = ks + cap * D * 2;
    {
        const uint16_t *q = static_cast<const uint16_t *>(a.q);
        const uint16_t *k = static_cast<const uint16_t *>(a.k) + start * a.k_tok + kh * a.k_head;
        const uint16_t *v = static_cast<const uint16_t *>(a.v) + start * a.v_tok + kh * a.v_head;
        const int piece = tid % kPieces;
#pragma unroll
        for (int r = tid / kPieces; r < kRows; r += kThreads / kPieces) {
            const int row = row0 + min(r, rows - 1), tok = row / a.group, head = kh * a.group + row - tok * a.group;
            copy16(qs + at16<D>(r, piece), q + (start + tok) * a.q_tok + head * a.q_head + piece * 8, r < rows);
        }
        for (int r = tid / kPieces; r < padded; r += kThreads / kPieces)
            copy16(ks + at16<D>(r, piece), k + min(r, keys - 1) * a.k_tok + piece * 8, r < keys);
        asm volatile("cp.async.commit_group;" ::: "memory");
        for (int r = tid / kPieces; r < padded; r += kThreads / kPieces)
            copy16(vs + at16<D>(r, piece), v + min(r, keys - 1) * a.v_tok + piece * 8, r < keys);
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
    const int w0 = warp * 16;                              // the warp's rows of the block
    const bool busy = w0 < rows;
    // this lane's two rows: its scores are columns 2 (lane % 4) and the next of every 8 keys
    const int g = lane >> 2, col = (lane & 3) * 2;
    const int row_of[2] = {min(w0 + g, rows - 1), min(w0 + g + 8, rows - 1)};
    const int tok[2] = {(row0 + row_of[0]) / a.group, (row0 + row_of[1]) / a.group};
    const int seen = (row0 + w0) / a.group + 1;            // keys in front of this one all of the warp's rows see
    const int chunks = busy ? (row0 + min(rows, w0 + 16) - 1) / a.group / 16 + 1 : 0;
    constexpr int kChunks = kMaxKeys / 16;
    float s[kChunks][2][4];
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    __syncthreads();
    float top[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    if (busy) {
        uint32_t q[D / 16][4];
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) ldsm(qs + at16<D>(w0 + (lane & 15), kk * 2 + (lane >> 4)), q[kk]);
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
            if (c >= chunks) break;
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[c][n][e] = 0.f;
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                uint32_t b[4];
                ldsm(ks + at16<D>(c * 16 + (lane >> 4) * 8 + (lane & 7), kk * 2 + (lane >> 3 & 1)), b);
                mma(s[c][0], q[kk], b[0], b[1]);
                mma(s[c][1], q[kk], b[2], b[3]);
            }
            if (c * 16 + 16 > seen) {
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (c * 16 + n * 8 + col + (e & 1) > tok[e >> 1]) s[c][n][e] = -INFINITY;
            }
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) top[e >> 1] = fmaxf(top[e >> 1], s[c][n][e]);
        }
    }
    const float scale = a.scale * kLog2e;
    float ref[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 1));
        top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 2));
        top[i] *= scale;
        ref[i] = top[i] == -INFINITY ? 0.f : top[i];
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();
    if (!busy) return;
    float o[D / 8][4];
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
    bool odd = false;
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
        if (c >= chunks) break;
        uint32_t p[4];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            float x[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                x[e] = ex2(fmaf(s[c][n][e], scale, -ref[e >> 1]));
                l[e >> 1] += x[e];
            }
            p[2 * n] = pack(x[0], x[1]);
            p[2 * n + 1] = pack(x[2], x[3]);
        }
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
            uint32_t b[4];
            ldsm_t(vs + at16<D>(c * 16 + (lane >> 3 & 1) * 8 + (lane & 7), i * 2 + (lane >> 4)), b);
            if (c * 16 + 16 > seen) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t x = bad(b[e]);
                    if (x) {
                        odd = true;
                        b[e] &= ~((x & 0x80000000u ? 0xffff0000u : 0u) | (x & 0x8000u ? 0xffffu : 0u));
                    }
                }
            }
            mma(o[2 * i], p, b[0], b[1]);
            mma(o[2 * i + 1], p, b[2], b[3]);
        }
    }
    odd = __any_sync(0xffffffffu, odd);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
        l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
        const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];
#pragma unroll
        for (int j = 0; j < D / 8; ++j) {
            o[j][2 * i] = l[i] == 0.f ? 0.f : o[j][2 * i] * inv;
            o[j][2 * i + 1] = l[i] == 0.f ? 0.f : o[j][2 * i + 1] * inv;
        }
    }
    if (odd) {
        // values that were taken as 0, for the rows that see them
#pragma unroll
        for (int i = 0; i < 2; ++i)
            for (int key = seen & ~15; key <= tok[i]; ++key)
#pragma unroll
                for (int j = 0; j < D / 8; ++j) {
                    const uint32_t u = *reinterpret_cast<const uint32_t *>(sm + (vs - qs) + at16<D>(key, j) + col * 2);
                    if (!bad(u)) continue;
                    const float lo = bf16_bits_to_float(static_cast<uint16_t>(u)), hi = bf16_bits_to_float(static_cast<uint16_t>(u >> 16));
                    if (!(fabsf(lo) < INFINITY)) o[j][2 * i] += lo;
                    if (!(fabsf(hi) < INFINITY)) o[j][2 * i + 1] += hi;
                }
    }
    const int mine = min(16, rows - w0);
    if (a.lse && (lane & 3) == 0) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (g + 8 * i < mine) {
                const int head = kh * a.group + row0 + row_of[i] - tok[i] * a.group;
                a.lse[static_cast<int64_t>(head) * a.tokens + start + tok[i]] = l[i] == 0.f ? -INFINITY : (top[i] + log2f(l[i])) * kLn2;
            }
    }
    if (a.out_dtype == 0) {
        // through the place of the warp's queries, so that a store covers whole 16-byte pieces
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < D / 8; ++j)
                *reinterpret_cast<uint32_t *>(sm + at16<D>(w0 + g + 8 * i, j) + col * 2) = pack(o[j][2 * i], o[j][2 * i + 1]);
        __syncwarp();
#pragma unroll
        for (int x = lane; x < 16 * kPieces; x += 32) {
            const int r = x / kPieces, piece = x % kPieces, row = row0 + w0 + r, t = row / a.group;
            if (r < mine)
                *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.o) + static_cast<int64_t>(start + t) * a.o_tok +
                                           static_cast<int64_t>(kh * a.group + row - t * a.group) * a.o_head + piece * 8) =
                    *reinterpret_cast<const uint4 *>(sm + at16<D>(w0 + r, piece));
        }
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (g + 8 * i < mine) {
                const int head = kh * a.group + row0 + row_of[i] - tok[i] * a.group;
                float *dst = static_cast<float *>(a.o) + static_cast<int64_t>(start + tok[i]) * a.o_tok + static_cast<int64_t>(head) * a.o_head;
#pragma unroll
                for (int j = 0; j < D / 8; ++j)
                    *reinterpret_cast<float2 *>(dst + j * 8 + col) = make_float2(o[j][2 * i], o[j][2 * i + 1]);
            }
    }
}

template <int D>
bool launch(const ServeArgs &a, cudaStream_t st) {
    static std::atomic<uint64_t> known{0};
    const int cap = (a.max_len + 15) & ~15, bytes = (kRows + 2 * cap) * D * 2, most = (kRows + 2 * kMaxKeys) * D * 2;
    if (!allow_smem(prompt_short_kernel<D>, most, &known)) return false;
    const int per_seq = (a.max_len * a.group + kRows - 1) / kRows;
    const int64_t blocks = static_cast<int64_t>(a.seqs) * a.kv_heads * per_seq;
    return launch_dependent(prompt_short_kernel<D>, dim3(static_cast<unsigned>(blocks)), dim3(kThreads), bytes, st, a, per_seq, cap);
}

}  // namespace

// Where this kernel is the faster one, in us here and there:
// - one round of blocks (8 heads on 2 and 16 heads at d = 64, 32 on 8 at d = 128): d = 64, 128 tokens: 256 blocks 7.3 and 8.4,
//   512 blocks 8.7 and 8.7 to 11.2, 1024 blocks 15.7 and 11.6; d = 64, 32 tokens: 512 blocks 5.2 and 11.2; d = 128, 32 tokens:
//   256 blocks 6.5 and 9.3, 512 blocks 10.9 and 9.7; 128 tokens: 64 blocks 9.7 and 9.5;
// - more of them: an SM takes about 0.7 + 0.0105 n us for a block of n keys at d = 64 and 1.9 + 0.022 n at d = 128, and 3.2 and
//   4.2 us for an item of two query tiles there, full or not. 1024 prompts, 16 heads, d = 64, of 64 tokens: 148 and 182, of
//   32: 118 and 175; 8 heads on 2 of 64: 71 and 55, of 16: 16 and 27; 32 heads on 8, d = 128, of 32: 294 and 139.
bool prompt_is_short(const ServeArgs &a) {
    if (a.max_len > kMaxKeys) return false;
    const int64_t heads = static_cast<int64_t>(a.seqs) * a.kv_heads;
    const int64_t blocks = heads * ((a.max_len * a.group + kRows - 1) / kRows);
    if (blocks > 0x7fffffff) return false;
    const int shorter = kMaxKeys * 64 / (a.max_len * a.d);   // than 128 tokens at d = 64
    if (blocks <= 2 * a.sms * (shorter < 4 ? shorter : 4) * 64 / a.d) return true;
    const int tokens = 128 / a.group;                        // of a query tile there
    const int64_t items = a.max_len <= tokens ? (heads + 1) / 2 : heads * ((a.max_len + 2 * tokens - 1) / (2 * tokens));
    return a.d == 64 ? blocks * (64 + a.max_len) < items * 288 : blocks * (86 + a.max_len) < items * 190;
}

int launch_prompt_short(const ServeArgs &a, cudaStream_t st) {
    return (a.d == 64 ? launch<64>(a, st) : launch<128>(a, st)) ? 1 : -1;
}

}  // namespace ha
