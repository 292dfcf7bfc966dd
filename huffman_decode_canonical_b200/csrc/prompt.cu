// prompt.cu -- causal attention over packed prompts with grouped heads, on the
// tensor cores (tcgen05).
//
//   o_i = sum_{j <= i + klen - qlen} p_ij v_j,  p_i = softmax_j(scale q_i . k_j)
//
// A CTA takes 256 queries of one head as two tiles of 128 rows and walks the
// keys in tiles of 128.  Each query tile has its scores S, whose room its
// weights P then take, and its output O in TMEM (lane = query row): S = Q K^T
// from shared memory, P V with P read from TMEM.  One warp issues all MMAs, one
// the TMA copies; four warps for each query tile take the softmax, a row a
// thread, so that one tile's softmax runs beside the other's MMAs.  The reference
// maximum of a row is only raised when a score passes it by 2^8 (any reference
// gives the same quotient), so O is rarely rescaled.  Bound by the exponentials
// and the MMAs about alike: 128 x 128 scores take 16384 exponentials (16 a clock
// and SM) and 2 x 128 x 128 x D multiply-adds (4096 a clock).
//
// What the mask hides must not count, whatever it holds.  Scores are replaced one
// by one.  Values of a tile that some row must not see are looked over in shared
// memory before their MMA: rows past the sequence's keys are zeroed, and where a
// visible row holds an infinity or NaN (0 times it would reach rows that do not
// see it) the CTA's rows are computed again one by one.
#include <algorithm>
#include <cstring>

#include "launch.h"
#include "sm100.cuh"

namespace entro {
using namespace sm100;

struct PromptArgs {
    const void *q, *k, *v;
    void *out;
    int64_t q_token, q_head, k_token, k_head, v_token, v_head, out_token, out_head;
    const int32_t *cu_q, *cu_k;
    int32_t *status;
    int64_t tokens, keys;
    int batch, heads, group;
    float scale_log2;
    uint32_t tx_extra;
};

constexpr int kRows = 128;             // rows of a query tile, and of a key tile
constexpr int kChunk = kRows * 128;    // bytes of 128 rows of 64 channels (one TMA box)
constexpr int kPromptThreads = 384;    // 2 x 4 softmax warps, MMA, copies, 2 warps that look over values
constexpr float kLazyLog2 = 8.0f;

template <int D>
struct PromptShape {
    static constexpr int kChunks = (D + 63) / 64;              // 96 channels fill one and a half; the rest reads as zero
    static constexpr int kTileBytes = kChunks * kChunk;
    static constexpr int kStages = D == 64 ? 8 : 4;            // key and value tiles in flight
    static constexpr int kSmem = 1024 + (2 + kStages) * kTileBytes;
};

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// One row by the definition, by one warp: for rows whose tile holds an infinity
// or NaN among values that other rows do not see.
template <typename T, int D>
__device__ __noinline__ void row_by_row(const PromptArgs &a, int head, int64_t q_row, int64_t k_row, int visible) {
    const int lane = threadIdx.x % 32;
    const T *q = static_cast<const T *>(a.q) + q_row * a.q_token + head * a.q_head;
    const T *k = static_cast<const T *>(a.k) + k_row * a.k_token + (head / a.group) * a.k_head;
    const T *v = static_cast<const T *>(a.v) + k_row * a.v_token + (head / a.group) * a.v_head;
    float m = -INFINITY, l = 0.0f, o[D / 32];
#pragma unroll
    for (int i = 0; i < D / 32; i++) o[i] = 0.0f;
    for (int j0 = 0; j0 < visible; j0 += 32) {
        float s = -INFINITY;
        if (j0 + lane < visible) {
            s = 0.0f;
            const T *row = k + (j0 + lane) * a.k_token;
            for (int d = 0; d < D; d += 8) {
                const uint4 x = *reinterpret_cast<const uint4 *>(row + d), y = *reinterpret_cast<const uint4 *>(q + d);
                const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const float2 f = Half<T>::widen(xs[i]), g = Half<T>::widen(ys[i]);
                    s = fmaf(f.x, g.x, fmaf(f.y, g.y, s));
                }
            }
            s *= a.scale_log2;
        }
        float n = fmaxf(m, s);
        for (int x = 16; x; x /= 2) n = fmaxf(n, __shfl_xor_sync(~0u, n, x));
        const float base = n == -INFINITY ? 0.0f : n;
        const float f = m == n ? 1.0f : exp2_fast(m - base), p = exp2_fast(s - base);
        m = n;
        l = l * f + p;
#pragma unroll
        for (int i = 0; i < D / 32; i++) o[i] *= f;
        for (int j = 0; j < 32 && j0 + j < visible; j++) {
            const float w = __shfl_sync(~0u, p, j);
            const T *row = v + (j0 + j) * a.v_token;
#pragma unroll
            for (int i = 0; i < D / 32; i++) o[i] = fmaf(w, static_cast<float>(row[i * 32 + lane]), o[i]);
        }
    }
    for (int x = 16; x; x /= 2) l += __shfl_xor_sync(~0u, l, x);
    T *out = static_cast<T *>(a.out) + q_row * a.out_token + head * a.out_head;
#pragma unroll
    for (int i = 0; i < D / 32; i++) out[i * 32 + lane] = static_cast<T>(l == 0.0f ? 0.0f : o[i] / l);
}

template <typename T, int D>
__global__ void __launch_bounds__(kPromptThreads, 1)
    prompt_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap k_map,
                  const __grid_constant__ CUtensorMap v_map, const __grid_constant__ PromptArgs a) {
    using Shape = PromptShape<D>;
    constexpr int kStages = Shape::kStages;
    // weights are held as 2^6 times theirs in fp16: at most 2^14, and none above 2^-30 of the largest is lost
    constexpr float kBias = Half<T>::kExp == 0x7C007C00u ? 6.0f : 0.0f;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bars[2 * kStages + 1 + 2 + 2 + 2 + 3 + 3];
    __shared__ uint32_t tmem_base;
    __shared__ int failed, special, where[6];
    const uint32_t base = (smem_u32(smem_raw) + 1023) & ~1023u, ring = base + 2 * Shape::kTileBytes;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const uint32_t full = smem_u32(bars), empty = full + 8 * kStages, q_full = empty + 8 * kStages, s_full = q_full + 8,
                   p_full = s_full + 16, o_full = p_full + 16, v_sent = o_full + 16, v_seen = v_sent + 24;

    // this CTA's query tiles: (sequence, block of 256 queries), the last block of a sequence first, since it has most keys
    const int head = blockIdx.x % a.heads;
    if (warp == 0) {
        int64_t item = blockIdx.x / a.heads;
        if (lane == 0) where[0] = -1;
        __syncwarp();
        for (int b0 = 0; b0 < a.batch; b0 += 32) {
            const int b = b0 + lane;
            int q0 = 0, qn = 0, k0 = 0, kn = 0;
            if (b < a.batch) {
                q0 = a.cu_q[b], qn = a.cu_q[b + 1] - q0;
                k0 = a.cu_k[b], kn = a.cu_k[b + 1] - k0;
                if (q0 < 0 || qn < 0 || static_cast<int64_t>(q0) + qn > a.tokens || k0 < 0 || kn < 0 ||
                    static_cast<int64_t>(k0) + kn > a.keys) {
                    set_status(a.status, ENTRO_E_INVAL);
                    qn = 0;
                }
            }
            const int blocks = qn / 256 + (qn % 256 != 0);
            int sum = blocks;
            for (int o = 1; o < 32; o *= 2) {
                const int up = __shfl_up_sync(~0u, sum, o);
                if (lane >= o) sum += up;
            }
            if (item < sum && item >= sum - blocks) {
                where[0] = q0, where[1] = qn, where[2] = k0, where[3] = kn;
                where[4] = sum - 1 - static_cast<int>(item);
            }
            const int all = __shfl_sync(~0u, sum, 31);
            if (item < all) break;
            item -= all;
        }
    } else if (warp == 1 && lane == 0) {
        for (int s = 0; s < kStages; s++) {
            bar_init(full + 8 * s, 1);
            bar_init(empty + 8 * s, 1);
        }
        bar_init(q_full, 1);
        for (int t = 0; t < 2; t++) {
            bar_init(s_full + 8 * t, 1);
            bar_init(p_full + 8 * t, 4);
            bar_init(o_full + 8 * t, 1);
        }
        for (int j = 0; j < 3; j++) {
            bar_init(v_sent + 8 * j, 1);
            bar_init(v_seen + 8 * j, 2);
        }
        fence_bar_init();
        failed = special = 0;
        prefetch_map(&q_map);
        prefetch_map(&k_map);
        prefetch_map(&v_map);
    }
    __syncthreads();
    if (where[0] < 0) return;  // (the grid has a few more blocks than there may be query tiles)
    if (warp == 8) tmem_alloc<1>(smem_u32(&tmem_base), 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base;
    const int q0 = where[0], qlen = where[1], k0 = where[2], klen = where[3], row0 = where[4] * 256;
    const int offset = klen - qlen;  // query i sees keys up to i + offset
    // key tiles of each query tile (0: no rows, or none that sees a key)
    auto key_tiles = [&](int t) {
        const int first = row0 + t * kRows;
        if (first >= qlen) return 0;
        const int64_t most = static_cast<int64_t>(min(first + kRows, qlen)) + offset;
        return most <= 0 ? 0 : static_cast<int>((most + kRows - 1) / kRows);
    };
    const int n0 = key_tiles(0), n1 = key_tiles(1), n = max(n0, n1);
    // key tiles from here on (three at most) hold keys that some row of the CTA must not see
    const int masked_from = offset + row0 + 1 <= 0 ? 0 : (offset + row0 + 1) / kRows;
    bool ok = true;

    if (warp == 9) {
        // ---- copies: queries, then K0 V0 K1 V1 ...
        if (elect_one() && n > 0) {
            const int kv = head / a.group;
            bar_expect(q_full, (n1 > 0 ? 2 : 1) * Shape::kTileBytes + a.tx_extra);
            for (int t = 0; t < (n1 > 0 ? 2 : 1); t++)
                for (int c = 0; c < Shape::kChunks; c++)
                    tma_3d(base + t * Shape::kTileBytes + c * kChunk, &q_map, q_full, c * 64, head, q0 + row0 + t * kRows);
            for (int i = 0; i < 2 * n; i++) {
                const int s = i % kStages, round = i / kStages;
                if (round > 0 && !bar_wait(empty + 8 * s, (round - 1) & 1)) {
                    ok = false;
                    break;
                }
                bar_expect(full + 8 * s, Shape::kTileBytes);
                for (int c = 0; c < Shape::kChunks; c++)
                    tma_3d(ring + s * Shape::kTileBytes + c * kChunk, i % 2 ? &v_map : &k_map, full + 8 * s, c * 64, kv, k0 + i / 2 * kRows);
                // from here on the tile's barrier is in the phase that the warps below wait for
                if (i % 2 && i / 2 >= masked_from) bar_arrive(v_sent + 8 * (i / 2 - masked_from));
            }
        }
    } else if (warp == 8) {
        // ---- MMAs
        if (elect_one() && n > 0) {
            constexpr uint32_t kScores = kAccF32 | Half<T>::kA | Half<T>::kB | mma_shape(kRows, kRows);
            constexpr uint32_t kValues = kAccF32 | Half<T>::kA | Half<T>::kB | kBMajorMN | mma_shape(kRows, D);
            auto scores = [&](int t, int i) {  // S_t = Q_t K^T, with K in ring place i
                const uint32_t qa = base + t * Shape::kTileBytes, ka = ring + i % kStages * Shape::kTileBytes;
#pragma unroll
                for (int k = 0; k < D / 16; k++) {
                    const uint32_t at = k / 4 * kChunk + k % 4 * 32;
                    mma_f16(tmem + t * kRows, operand_desc(qa + at, 16, 1024), operand_desc(ka + at, 16, 1024), kScores, k > 0);
                }
                mma_commit(s_full + 8 * t);
            };
            auto arrived = [&](int i) { return bar_wait(full + 8 * (i % kStages), i / kStages & 1); };
            do {
                if (!(ok = bar_wait(q_full, 0) && arrived(0))) break;
                tc_fence_after();
                if (n0 > 0) scores(0, 0);
                if (n1 > 0) scores(1, 0);
                mma_commit(empty);
                for (int j = 0; j < n && ok; j++) {
                    const int iv = 2 * j + 1, ik = 2 * j + 2;
                    if (!(ok = arrived(iv))) break;
                    if (j >= masked_from && !(ok = bar_wait(v_seen + 8 * (j - masked_from), 0))) break;
                    if (j + 1 < n && !(ok = arrived(ik))) break;
                    for (int t = 0; t < 2; t++) {
                        const int nt = t ? n1 : n0;
                        if (j >= nt) continue;
                        if (!(ok = bar_wait(p_full + 8 * t, j & 1))) break;
                        tc_fence_after();
                        const uint32_t va = ring + iv % kStages * Shape::kTileBytes;
#pragma unroll
                        for (int k = 0; k < kRows / 16; k++)
                            mma_f16_ta(tmem + 2 * kRows + t * 128, tmem + t * kRows + k * 8, operand_desc(va + k * 2048, kChunk, 1024),
                                       kValues, j > 0 || k > 0);
                        // (MMAs run in order: the next scores overwrite P after it has been read)
                        if (j + 1 < nt) scores(t, ik);
                        else mma_commit(o_full + 8 * t);
                    }
                    if (!ok) break;
                    mma_commit(empty + 8 * (iv % kStages));
                    if (j + 1 < n) mma_commit(empty + 8 * (ik % kStages));
                }
            } while (false);
        }
    } else if (warp >= 10) {
        // ---- values that some row must not see
        for (int j = masked_from; j < n; j++) {
            const int i = 2 * j + 1;
            if (!bar_wait(v_sent + 8 * (j - masked_from), 0) || !bar_wait(full + 8 * (i % kStages), i / kStages & 1)) {
                ok = false;
                break;
            }
            const uint32_t tile = ring + i % kStages * Shape::kTileBytes;
            bool odd = false;
            for (int u = tid - 320; u < Shape::kTileBytes / 16; u += 64) {
                // (the swizzle moves 16-byte pieces inside a row of 128 bytes only)
                const int key = j * kRows + u % (kChunk / 16) / 8;
                if (key >= klen) {
                    asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(tile + u * 16), "r"(0) : "memory");
                } else {
                    uint32_t x[4];
                    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]) : "r"(tile + u * 16));
#pragma unroll
                    for (int w = 0; w < 4; w++) {
                        constexpr uint32_t kLow = Half<T>::kExp & 0xFFFF, kHigh = Half<T>::kExp & 0xFFFF0000u;
                        odd = odd || (x[w] & kLow) == kLow || (x[w] & kHigh) == kHigh;
                    }
                }
            }
            if (odd) special = 1;
            fence_async_smem();
            __syncwarp();
            if (lane == 0) bar_arrive(v_seen + 8 * (j - masked_from));
        }
    } else {
        // ---- softmax: a row a thread
        const int t = warp / 4, nt = t ? n1 : n0, row = row0 + tid;
        const uint32_t lanes = static_cast<uint32_t>(warp % 4 * 32) << 16, st = tmem + t * kRows + lanes, ot = tmem + 2 * kRows + t * 128 + lanes;
        const int first = row0 + t * kRows;
        const int sees = row + offset;  // the last key of this row
        const float c = a.scale_log2;
        float m = -INFINITY, l = 0.0f;  // m in units of the raw scores
        for (int j = 0; j < nt; j++) {
            if (!__all_sync(~0u, bar_wait(s_full + 8 * t, j & 1))) {
                ok = false;
                break;
            }
            tc_fence_after();
            uint32_t s[kRows];
#pragma unroll
            for (int x = 0; x < kRows; x += 32) tmem_ld32(st + x, s + x);
            tmem_wait_ld<kRows>(s);
            if (j * kRows + kRows - 1 > first + offset) {
                const int last = sees - j * kRows;
#pragma unroll
                for (int x = 0; x < kRows; x++)
                    if (x > last) s[x] = 0xFF800000u;
            }
            float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int x = 0; x < kRows; x++) top[x % 4] = fmaxf(top[x % 4], __uint_as_float(s[x]));
            const float n_m = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
            const bool raise = n_m * c > m * c + kLazyLog2;
            if (__any_sync(~0u, raise)) {
                const float f = raise ? exp2_fast((m - n_m) * c) : 1.0f;
                if (raise) m = n_m;
                l *= f;
                if (j > 0) {
                    // O holds everything up to the last tile: its MMAs came before the scores that were waited for
#pragma unroll 1
                    for (int x = 0; x < D; x += 32) {
                        uint32_t o[32];
                        tmem_ld32(ot + x, o);
                        tmem_wait_ld<32>(o);
#pragma unroll
                        for (int y = 0; y < 32; y++) o[y] = __float_as_uint(__uint_as_float(o[y]) * f);
                        tmem_st32(ot + x, o);
                    }
                }
            }
            const float less = (m == -INFINITY ? 0.0f : -m * c) + kBias;
            float sum[2] = {0.0f, 0.0f};
#pragma unroll
            for (int x = 0; x < kRows; x += 64) {
                uint32_t p[32];
#pragma unroll
                for (int y = 0; y < 32; y++) {
                    const float e0 = exp2_fast(fmaf(__uint_as_float(s[x + 2 * y]), c, less));
                    const float e1 = exp2_fast(fmaf(__uint_as_float(s[x + 2 * y + 1]), c, less));
                    sum[0] += e0;
                    sum[1] += e1;
                    p[y] = Half<T>::pack(e0, e1);
                }
                tmem_st32(st + x / 2, p);
            }
            l += sum[0] + sum[1];
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) bar_arrive(p_full + 8 * t);
        }
        if (ok && nt > 0) {
            ok = __all_sync(~0u, bar_wait(o_full + 8 * t, 0));
            tc_fence_after();
        }
        if (ok && first < qlen) {
            const float by = l == 0.0f ? 0.0f : 1.0f / l;
            T *out = static_cast<T *>(a.out) + (static_cast<int64_t>(q0) + row) * a.out_token + head * a.out_head;
#pragma unroll 1
            for (int x = 0; x < D; x += 32) {
                uint32_t o[32];
                if (nt > 0) {
                    tmem_ld32(ot + x, o);
                    tmem_wait_ld<32>(o);
                }
                if (row < qlen) {
#pragma unroll
                    for (int y = 0; y < 32; y += 8) {
                        uint32_t h[4];
#pragma unroll
                        for (int z = 0; z < 4; z++)
                            h[z] = l == 0.0f ? 0u : Half<T>::pack(__uint_as_float(o[y + 2 * z]) * by, __uint_as_float(o[y + 2 * z + 1]) * by);
                        *reinterpret_cast<uint4 *>(out + x + y) = make_uint4(h[0], h[1], h[2], h[3]);
                    }
                }
            }
        }
    }
    if (!ok) failed = 1;
    __syncwarp();
    __syncthreads();
    if (failed) {
        if (tid == 0) set_status(a.status, ENTRO_E_TIMEOUT);
        drain();
    } else if (special) {
        for (int r = row0 + warp; r < min(row0 + 256, qlen); r += kPromptThreads / 32)
            row_by_row<T, D>(a, head, static_cast<int64_t>(q0) + r, k0, min(max(r + offset + 1, 0), klen));
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 8) tmem_free<1>(tmem, 512);
}

template <typename T>
static const void *pick_prompt(int dim, size_t *smem) {
    *smem = dim == 64 ? PromptShape<64>::kSmem : dim == 96 ? PromptShape<96>::kSmem : PromptShape<128>::kSmem;
    return dim == 64   ? reinterpret_cast<const void *>(prompt_kernel<T, 64>)
           : dim == 96 ? reinterpret_cast<const void *>(prompt_kernel<T, 96>)
                       : reinterpret_cast<const void *>(prompt_kernel<T, 128>);
}

// [tokens][heads][dim] for TMA boxes of 128 tokens of 64 channels of a head
static int rows_map(CUtensorMap *map, int type, const void *base, int64_t tokens, int heads, int dim, int64_t token, int64_t head) {
    const uint64_t dims[3] = {static_cast<uint64_t>(dim), static_cast<uint64_t>(heads), static_cast<uint64_t>(tokens)};
    const uint64_t strides[2] = {static_cast<uint64_t>(heads > 1 ? head : dim) * 2, static_cast<uint64_t>(tokens > 1 ? token : dim) * 2};
    const uint32_t box[3] = {64, 1, kRows};
    return encode_map(map, type == ENTRO_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, base, dims, strides, box);
}

// rows that a TMA copy can read: strides above 0, in steps of 16 bytes, below 2^40 bytes
static bool tma_rows(const void *p, int64_t tokens, int heads, int64_t token, int64_t head) {
    auto good = [](int64_t s) { return s > 0 && s % 8 == 0 && s < (INT64_C(1) << 39); };
    return aligned16(p) && (tokens <= 1 || good(token)) && (heads <= 1 || good(head));
}

}  // namespace entro

using namespace entro;

extern "C" int entro_attention_prompt(int32_t type, int32_t head_dim, const void *d_q, int64_t q_token, int64_t q_head, int32_t heads,
                                      int64_t tokens, const void *d_k, int64_t k_token, int64_t k_head, const void *d_v,
                                      int64_t v_token, int64_t v_head, int32_t kv_heads, int64_t keys, const int32_t *d_cu_q,
                                      const int32_t *d_cu_k, int32_t batch, float scale, void *d_out, int64_t out_token,
                                      int64_t out_head, int32_t *d_status, void *stream) {
    if ((type != ENTRO_BF16 && type != ENTRO_F16) || (head_dim != 64 && head_dim != 96 && head_dim != 128)) return ENTRO_E_INVAL;
    if (heads < 1 || kv_heads < 1 || heads % kv_heads || tokens < 0 || keys < 0 || batch < 0 || !(scale > 0.0f) || scale > 3.0e38f) return ENTRO_E_INVAL;
    if (tokens > INT32_MAX - 256 || keys > INT32_MAX - 256) return ENTRO_E_LIMIT;
    if (tokens == 0 || batch == 0) return ENTRO_OK;
    if (!d_q || !d_cu_q || !d_out || (keys > 0 && (!d_k || !d_v))) return ENTRO_E_INVAL;
    if (!tma_rows(d_q, tokens, heads, q_token, q_head) || !tma_rows(d_k, keys, kv_heads, k_token, k_head) ||
        !tma_rows(d_v, keys, kv_heads, v_token, v_head) || !aligned16(d_out) || out_token % 8 || out_head % 8)
        return ENTRO_E_INVAL;
    if (!d_cu_k && tokens != keys) return ENTRO_E_INVAL;
    PromptArgs a;
    std::memset(&a, 0, sizeof(a));
    a.q = d_q, a.k = d_k, a.v = d_v, a.out = d_out;
    a.q_token = q_token, a.q_head = q_head, a.k_token = k_token, a.k_head = k_head, a.v_token = v_token, a.v_head = v_head;
    a.out_token = out_token, a.out_head = out_head;
    a.cu_q = d_cu_q, a.cu_k = d_cu_k ? d_cu_k : d_cu_q;
    a.status = d_status;
    a.tokens = tokens, a.keys = keys, a.batch = batch, a.heads = heads, a.group = heads / kv_heads;
    a.scale_log2 = scale * 1.4426950408889634f;
    a.tx_extra = test_tx_extra();
    const int64_t blocks = (tokens / 256 + batch) * heads;
    if (blocks > INT32_MAX) return ENTRO_E_LIMIT;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
    size_t smem;
    const void *fn = type == ENTRO_BF16 ? pick_prompt<__nv_bfloat16>(head_dim, &smem) : pick_prompt<__half>(head_dim, &smem);
    int r = allow_smem(fn, dev);
    CUtensorMap q_map, k_map, v_map;
    if (r == ENTRO_OK) r = rows_map(&q_map, type, d_q, tokens, heads, head_dim, q_token, q_head);
    // (without keys nothing is copied; the maps only have to be valid)
    if (r == ENTRO_OK) r = keys ? rows_map(&k_map, type, d_k, keys, kv_heads, head_dim, k_token, k_head) : (k_map = q_map, ENTRO_OK);
    if (r == ENTRO_OK) r = keys ? rows_map(&v_map, type, d_v, keys, kv_heads, head_dim, v_token, v_head) : (v_map = q_map, ENTRO_OK);
    if (r != ENTRO_OK) return r;
    void *args[] = {&q_map, &k_map, &v_map, &a};
    e = launch_ex(fn, dim3(static_cast<unsigned>(blocks)), kPromptThreads, smem, static_cast<cudaStream_t>(stream), 1, false, args);
    return e == cudaSuccess ? ENTRO_OK : cuda_fail(e, "entro_attention_prompt");
}
