// prompt.cu -- causal attention over packed prompts with grouped heads, on the
// tensor cores (tcgen05).
//
//   o_i = sum_{j <= i + klen - qlen} p_ij v_j,  p_i = softmax_j(scale q_i . k_j)
//
// A CTA takes 256 queries of one head as two tiles of 128 rows and walks the
// keys in tiles of 64, then goes on with another block of queries.
// S = Q K^T from shared memory and O += P V with P read from TMEM are
// tcgen05.mma; S, P and O are in TMEM (lane = query row).  A warp issues each query
// tile's MMAs, one finds the work and issues the TMA copies, one looks over values
// that are partly hidden, and four warps for each query tile take the softmax, a
// row a thread.  The reference maximum of a row is only raised when a score passes
// it by 2^8 (any reference gives the same quotient), so O is rarely rescaled.
// Bound by the exponentials and the MMAs about alike at 128 channels (128 x 128
// scores take 16384 exponentials, 16 a clock and SM, and 2 x 128 x 128 x D
// multiply-adds, 4096 a clock).  8192 tokens, 32 heads of 128 over 8: 441 us in a row of
// 9 calls (1248 TFLOP/s), 510 in a long one, at the power limit.  At 64 and 96 the
// exponentials take longer than the MMAs, but neither accounts for the time: 4096 tokens,
// 32 heads of 64: 108 us (640); 6011 tokens, 32 heads of 96: 277 to 294 us (755 to 802),
// in 5 prompts of uneven lengths 127 to 130 (600).  Taking a part of
// the exponentials by a polynomial instead, looking for the maximum only after a weight
// came out too large, or fetching the next scores beside the exponentials was slower (in
// an earlier form 463 us -> 489 to 518, 562, and 510).
//
// The weights are rounded to the inputs' type (half a step of it, of each weight): both
// operands of an MMA have one type, and values in bfloat16 do not fit fp16.  A second
// product with the weights' remainders would add half of the MMAs again.  The sums of
// the weights take them as they were in 32 bits.
//
// Few queries over many keys leave most SMs without a block: there a cluster of up
// to eight CTAs shares the keys of a block (see join_parts).
//
// What the mask hides must not count, whatever it holds.  Scores are replaced one
// by one.  Values of a tile that some row must not see are looked over in shared
// memory before their MMA: rows past the sequence's keys are zeroed, and so are
// infinities and NaN (0 times one would reach rows that do not see it), which are
// added to the outputs of the rows that do see them: a weight above 0 times an
// infinity, and whatever is finite besides, is that infinity.
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
    int parts;  // CTAs (a cluster) that share the keys of a block: 1 to 8
    float scale_log2;
    uint32_t tx_extra;
};

constexpr int kRows = 128;             // rows of a query tile
constexpr int kPromptThreads = 384;    // 2 x 4 softmax warps, an MMA warp for each query tile, copies, a look over values
constexpr float kLazyLog2 = 8.0f;
constexpr int kMarks = 8;              // barriers for masked value tiles, more than the ring holds

// TMEM has 512 columns: for each of two query tiles the scores (64 columns, a key each), two buffers of weights (32
// columns, two keys each) and the output (a column a channel).  With weights apart from scores the next scores do not
// wait for the last weights' product, so the softmax warps always find scores ready; with two buffers the weights do not
// wait for it either (step j's scores come after the product of step j - 2 in the order of the MMAs).  That is room for 64
// keys a tile at 128 channels; at 64 channels 128 keys were no faster (4096 tokens: 119 and 122 us) and worse for short
// prompts (16 of 44 tokens, 32 heads: 17.4 and 12.5 us).
template <int D>
struct PromptShape {
    static constexpr int kKeys = 64;                           // keys of a tile
    static constexpr int kChunks = (D + 63) / 64;              // 64 channels each; 96 fill one and a half, the rest reads as zero
    static constexpr int kQChunk = kRows * 128, kChunk = kKeys * 128;  // bytes of a chunk (one TMA box)
    static constexpr int kQTile = kChunks * kQChunk, kTile = kChunks * kChunk;
    static constexpr int kStages = (220 * 1024 - 2 * kQTile) / kTile < 10 ? (220 * 1024 - 2 * kQTile) / kTile : 10;  // key and value tiles in flight
    static constexpr int kSmem = 1024 + 2 * kQTile + kStages * kTile;
    static constexpr uint32_t kS = 0, kP = 2 * kKeys, kO = 4 * kKeys;  // TMEM columns: S0 S1, P0 P0 P1 P1, O0 O1
    static_assert(kO + 2 * D <= 512 && kStages / 2 < kMarks && kStages >= 4 && kKeys % 32 == 0, "");
    static_assert(2 * kRows * (D + 2) * 4 <= kSmem - 1024, "");  // a part's outputs and statistics for the join
};

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// Exponents of all ones, in either half of a word, carry into the sign bits.
template <typename T>
__device__ __forceinline__ uint32_t not_finite(uint32_t x) {
    constexpr uint32_t kOne = Half<T>::kExp == 0x7C007C00u ? 0x04000400u : 0x00800080u;
    return ((x & Half<T>::kExp) + kOne) & 0x80008000u;
}

// By a warp, a row a lane: the infinities and NaN among the values of keys [from, to) to the outputs (written before) of
// the rows that see them, keys up to `last`.  A key that scores -infinity has weight 0, and 0 times them is NaN.  A block's
// keys of this kind are some 320 at most (its queries' and the rest of a tile), so this takes no longer for a long context.
template <typename T, int D>
__device__ __forceinline__ void add_not_finite(const PromptArgs &a, int head, int64_t q_row, int64_t k_row, int from, int to, bool mine, int last) {
    const int lane = threadIdx.x % 32;
    const T *q = static_cast<const T *>(a.q) + q_row * a.q_token + head * a.q_head;
    const T *k = static_cast<const T *>(a.k) + k_row * a.k_token + (head / a.group) * a.k_head;
    const T *v = static_cast<const T *>(a.v) + k_row * a.v_token + (head / a.group) * a.v_head;
    T *out = static_cast<T *>(a.out) + q_row * a.out_token + head * a.out_head;
#pragma unroll 1
    for (int j0 = from; j0 < to; j0 += 32) {
        uint32_t odd = 0;
        if (j0 + lane < to) {
            const T *row = v + (j0 + lane) * a.v_token;
            for (int d = 0; d < D; d += 8) {
                const uint4 x = *reinterpret_cast<const uint4 *>(row + d);
                odd |= not_finite<T>(x.x) | not_finite<T>(x.y) | not_finite<T>(x.z) | not_finite<T>(x.w);
            }
        }
        for (uint32_t keys = __ballot_sync(~0u, odd != 0); keys; keys &= keys - 1) {
            const int j = j0 + __ffs(keys) - 1;
            if (!mine || j > last) continue;
            float s = 0.0f;
#pragma unroll 1
            for (int d = 0; d < D; d++) s = fmaf(static_cast<float>(q[d]), static_cast<float>(k[j * a.k_token + d]), s);
            const bool none = s * a.scale_log2 == -INFINITY;
#pragma unroll 1
            for (int d = 0; d < D; d++) {
                const float x = static_cast<float>(v[j * a.v_token + d]);
                if (!(fabsf(x) < INFINITY)) out[d] = static_cast<T>(static_cast<float>(out[d]) + (none ? __int_as_float(0x7FC00000) : x));
            }
        }
    }
}

// What a CTA works on: 256 queries of a head.
struct PromptItem {
    int q0, qlen, k0, klen, row0, head;  // head < 0: no more work
    int offset;                          // query i sees keys up to i + offset
    int skipped;                         // keys of the sequence in front of k0

    // key tiles of query tile t (0: no rows, or none that sees a key)
    template <int KEYS>
    __device__ __forceinline__ int key_tiles(int t) const {
        const int first = row0 + t * kRows;
        if (first >= qlen) return 0;
        const int64_t most = min(static_cast<int64_t>(min(first + kRows, qlen)) + offset, static_cast<int64_t>(klen));
        return most <= 0 ? 0 : static_cast<int>((most + KEYS - 1) / KEYS);
    }
    // key tiles from here on hold keys that some row must not see
    template <int KEYS>
    __device__ __forceinline__ int masked_from() const { return offset + row0 + 1 <= 0 ? 0 : (offset + row0 + 1) / KEYS; }
    // of the key tiles, part `i` of `of` (its rows see the keys that they saw)
    template <int KEYS>
    __device__ __forceinline__ void cut(int i, int of) {
        const int n = max(key_tiles<KEYS>(0), key_tiles<KEYS>(1)), from = n * i / of * KEYS, to = min(n * (i + 1) / of * KEYS, klen);
        skipped = from, k0 += from, offset -= from, klen = max(to - from, 0);
    }
    // back to the whole sequence's keys (but for their number)
    __device__ __forceinline__ void join_cut() { k0 -= skipped, offset += skipped, skipped = 0; }
};

// Block number -> item, by a warp: heads fastest, so that those of a key head meet in L2; of a sequence's blocks the
// last first, since it has most keys.  False: a block of no item (the grid is cut for the most there may be).
__device__ __forceinline__ bool find_item(const PromptArgs &a, int block, PromptItem &it) {
    const int lane = threadIdx.x % 32;
    it.head = block % a.heads;
    int left = block / a.heads;
    for (int b0 = 0; b0 < a.batch; b0 += 32) {
        const int b = b0 + lane;
        int q0 = 0, qn = 0, k0 = 0, kn = 0;
        if (b < a.batch) {
            q0 = a.cu_q[b], k0 = a.cu_k[b];
            const int q1 = a.cu_q[b + 1], k1 = a.cu_k[b + 1];
            // (compared before they are subtracted: differences of offsets may pass 32 bits)
            if (q0 < 0 || q0 > q1 || q1 > a.tokens || k0 < 0 || k0 > k1 || k1 > a.keys)
                set_status(a.status, ENTRO_E_INVAL);
            else
                qn = q1 - q0, kn = k1 - k0;
        }
        const int blocks = qn / 256 + (qn % 256 != 0);
        int sum = blocks;
        for (int o = 1; o < 32; o *= 2) {
            const int up = __shfl_up_sync(~0u, sum, o);
            if (lane >= o) sum += up;
        }
        const uint32_t here = __ballot_sync(~0u, left < sum);
        if (here) {
            const int from = __ffs(here) - 1;
            it.q0 = __shfl_sync(~0u, q0, from), it.qlen = __shfl_sync(~0u, qn, from);
            it.k0 = __shfl_sync(~0u, k0, from), it.klen = __shfl_sync(~0u, kn, from);
            it.offset = it.klen - it.qlen, it.skipped = 0;
            it.row0 = (__shfl_sync(~0u, sum, from) - 1 - left) * 256;
            return true;
        }
        left -= __shfl_sync(~0u, sum, 31);
    }
    return false;
}

// The next block that has not started, in place of which this CTA goes on (cluster launch control).
__device__ __forceinline__ void ask_next(uint32_t reply, uint32_t bar) {
    bar_expect(bar, 16);
    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(reply), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ int next_block(uint32_t reply) {  // -1: none is left
    uint32_t x;
    asm volatile(
        "{\n\t.reg .b128 r;\n\t.reg .pred p;\n\t"
        "ld.shared.b128 r, [%1];\n\t"
        "mov.u32 %0, 0xffffffff;\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %0, r;\n\t}"
        : "=r"(x)
        : "r"(reply)
        : "memory");
    fence_async_smem();  // read before the next reply is written
    return static_cast<int>(x);
}

// ---- A block whose keys are shared by a cluster.  Softmax over parts of the keys: with (m_p, l_p, o_p) of part p and
// m = max m_p, l = sum 2^(c (m_p - m)) l_p and o alike.  Each CTA holds its part's of all 256 rows; they meet in shared
// memory across the cluster, so there is no workspace and no second launch, and the sums have one order.
// 256 queries over 32768 keys, 32 heads of 128: 413 us by a CTA a block, 127 by four.

__device__ __forceinline__ void all_warps() { asm volatile("barrier.sync 1, %0;" ::"n"(kPromptThreads) : "memory"); }

// by warps that have no rows (or none that came through): every thread takes part in the barriers
__device__ __forceinline__ void skip_join() {
    __syncwarp();
    all_warps();
    cluster_sync();
    cluster_sync();
}

// By the softmax warps, a row a thread: the parts go to their CTAs' shared memory, where queries, keys and values were
// (nothing reads those any more when all warps are here), and each CTA finishes a share of the rows.
template <typename T, int D>
__device__ __forceinline__ void join_parts(const PromptArgs &a, PromptItem it, uint32_t base, uint32_t ot, float m, float l, bool any,
                                        uint32_t special) {
    const int tid = threadIdx.x, warp = tid / 32;
    const uint32_t stats = base + 256 * D * 4;
    __syncwarp();
    all_warps();
    tc_fence_after();
    const int rows = min(256, it.qlen - it.row0);
#pragma unroll 1
    for (int x = 0; x < D && warp * 32 < rows; x += 32) {
        uint32_t o[32];
        if (any) {
            tmem_ld32(ot + x, o);
            tmem_wait_ld<32>(o);
        } else {
#pragma unroll
            for (int y = 0; y < 32; y++) o[y] = 0;
        }
        // (eight lanes write 16 bytes each at a time, of rows that begin in the same bank: pieces change places with the row)
#pragma unroll
        for (int y = 0; y < 8; y++)
            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(base + tid * D * 4 + (((x / 4 + y) ^ (tid & 7)) * 16)), "r"(o[4 * y]),
                         "r"(o[4 * y + 1]), "r"(o[4 * y + 2]), "r"(o[4 * y + 3])
                         : "memory");
    }
    asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(stats + tid * 8), "f"(m), "f"(l) : "memory");
    __syncwarp();
    cluster_sync();
    const int parts = a.parts, share = (rows + parts - 1) / parts, row0 = static_cast<int>(cluster_rank()) * share;
    const int end = min(row0 + share, rows);
    uint32_t odd = 0;
    for (int p = 0; p < parts; p++) {
        uint32_t x, y;
        asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(x) : "r"(map_to(special, p)) : "memory");
        asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(y) : "r"(map_to(special + 16, p)) : "memory");
        odd |= x | y;
    }
    {
        const float c = a.scale_log2;
        for (int u = tid; u < (end - row0) * (D / 8); u += 256) {
            const int r = row0 + u / (D / 8), d = u % (D / 8) * 2;  // 8 channels: pieces d and d + 1
            float2 ml[8];
            float top = -INFINITY;
#pragma unroll
            for (int p = 0; p < 8; p++) ml[p] = p < parts ? load_cluster2(map_to(stats + r * 8, p)) : make_float2(-INFINITY, 0.0f);
#pragma unroll
            for (int p = 0; p < 8; p++) top = fmaxf(top, ml[p].x);
            float sum = 0.0f, o[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int p = 0; p < 8; p++)
                if (p < parts) {
                    const uint32_t row = map_to(base + r * D * 4, p);
                    const float4 x = load_cluster4(row + ((d ^ (r & 7)) * 16)), y = load_cluster4(row + (((d + 1) ^ (r & 7)) * 16));
                    const float f = ml[p].x == top ? 1.0f : exp2_fast((ml[p].x - top) * c);
                    sum = fmaf(f, ml[p].y, sum);
                    o[0] = fmaf(f, x.x, o[0]), o[1] = fmaf(f, x.y, o[1]), o[2] = fmaf(f, x.z, o[2]), o[3] = fmaf(f, x.w, o[3]);
                    o[4] = fmaf(f, y.x, o[4]), o[5] = fmaf(f, y.y, o[5]), o[6] = fmaf(f, y.z, o[6]), o[7] = fmaf(f, y.w, o[7]);
                }
            const float by = sum == 0.0f ? 0.0f : sum < 0.0f ? __int_as_float(0x7FC00000) : 1.0f / sum;
            uint32_t h[4];
#pragma unroll
            for (int z = 0; z < 4; z++) h[z] = sum == 0.0f ? 0u : Half<T>::pack(o[2 * z] * by, o[2 * z + 1] * by);
            T *out = static_cast<T *>(a.out) + (static_cast<int64_t>(it.q0) + it.row0 + r) * a.out_token + it.head * a.out_head;
            *reinterpret_cast<uint4 *>(out + d * 4) = make_uint4(h[0], h[1], h[2], h[3]);
        }
    }
    if (odd) {  // (of the whole cluster: all warps agree)
        asm volatile("barrier.sync 2, 256;" ::: "memory");
        it.join_cut();
        const int r = row0 + tid, top = min(row0 + warp * 32 + 31, end - 1);
        if (row0 + warp * 32 < end)
            add_not_finite<T, D>(a, it.head, static_cast<int64_t>(it.q0) + it.row0 + min(r, end - 1), it.k0, it.masked_from<PromptShape<D>::kKeys>() * PromptShape<D>::kKeys,
                                 it.row0 + top + it.offset + 1, r < end, it.row0 + r + it.offset);
    }
    __syncwarp();
    cluster_sync();  // the others have read this CTA's part
}

template <typename T, int D>
__global__ void __launch_bounds__(kPromptThreads, 1)
    prompt_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap k_map,
                  const __grid_constant__ CUtensorMap v_map, const __grid_constant__ PromptArgs a) {
    using Shape = PromptShape<D>;
    constexpr int kStages = Shape::kStages, kKeys = Shape::kKeys;
    // weights are held as 2^6 times theirs in fp16: at most 2^14, and none above 2^-30 of the largest is lost
    constexpr float kBias = Half<T>::kExp == 0x7C007C00u ? 6.0f : 0.0f;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(16) uint32_t reply[4];
    __shared__ PromptItem items[2];
    __shared__ __align__(8) uint64_t bars[2 * kStages + 23 + 2 * kMarks];
    __shared__ uint32_t tmem_base;
    __shared__ int failed, special[8];  // per query tile: items with values that are not finite (item n in place n % 4)
    const uint32_t base = (smem_u32(smem_raw) + 1023) & ~1023u, ring = base + 2 * Shape::kQTile;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    // Barriers, each with a count of its own that goes on from item to item:
    const uint32_t full = smem_u32(bars), empty = full + 8 * kStages;       // key and value tiles
    const uint32_t item_full = empty + 8 * kStages, item_empty = item_full + 16;  // item n in place n % 2
    const uint32_t q_full = item_empty + 16, q_empty = q_full + 8;          // the item's queries; (per tile) read for the last time
    const uint32_t s_full = q_empty + 16, s_read = s_full + 16;             // per tile: scores; taken into registers
    const uint32_t p_full = s_read + 16, p_read = p_full + 32;              // per tile: weights (per buffer); multiplied
    const uint32_t o_full = p_read + 16, o_empty = o_full + 16;             // per tile: the item's output; stored
    const uint32_t asked = o_empty + 16, turn = asked + 8, v_sent = turn + 8, v_seen = v_sent + 8 * kMarks;  // masked value tile g in place g % kMarks: on its way; looked over
    if (warp == 0) {
        if (lane == 0) {
            for (int s = 0; s < kStages; s++) {
                bar_init(full + 8 * s, 1);
                bar_init(empty + 8 * s, 2);
            }
            bar_init(q_full, 1);
            bar_init(asked, 1);
            bar_init(turn, 4);
            for (int t = 0; t < 2; t++) {
                bar_init(item_full + 8 * t, 1);
                bar_init(item_empty + 8 * t, 11);  // two MMA warps, the look-over, eight softmax warps
                bar_init(q_empty + 8 * t, 1);
                bar_init(s_full + 8 * t, 1);
                bar_init(s_read + 8 * t, 4);
                bar_init(p_full + 16 * t, 4);
                bar_init(p_full + 16 * t + 8, 4);
                bar_init(p_read + 8 * t, 1);
                bar_init(o_full + 8 * t, 1);
                bar_init(o_empty + 8 * t, 4);
            }
            for (int j = 0; j < kMarks; j++) {
                bar_init(v_sent + 8 * j, 1);
                bar_init(v_seen + 8 * j, 1);
            }
            fence_bar_init();
            failed = 0;
            for (int x = 0; x < 8; x++) special[x] = 0;
        }
    } else if (warp == 1 && lane == 0) {
        prefetch_map(&q_map);
        prefetch_map(&k_map);
        prefetch_map(&v_map);
    } else if (warp == 8) {
        tmem_alloc<1>(smem_u32(&tmem_base), 512);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base;
    bool ok = true;
    // item n as the other warps take it from its place; every lane waits, so that a warp leaves together
    auto take = [&](int n, PromptItem &it) {
        if (!__all_sync(~0u, bar_wait(item_full + 8 * (n % 2), n / 2 & 1))) {
            ok = false;
            return false;
        }
        it = items[n % 2];
        __syncwarp();
        if (lane == 0) bar_arrive(item_empty + 8 * (n % 2));
        return it.head >= 0;
    };

    // registers: a softmax thread holds a row of scores (the shares add up to the launch's 384 x 168)
    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
        if (warp == 10) {
            // ---- items and copies: queries, then K0 V0 K1 V1 ...
            const int rank = blockIdx.x % a.parts;
            int block = blockIdx.x / a.parts, items_out = 0, queries = 0, i = 0, g = 0, answers = 0;
            PromptItem it;
            while (ok) {
                const bool is = block >= 0 && find_item(a, block, it);
                bool soon = false;
                if (is && a.parts > 1) it.cut<kKeys>(rank, a.parts);
                if (is || block < 0) {
                    if (block < 0) it.head = -1;
                    if (items_out >= 2) ok = __all_sync(~0u, bar_wait(item_empty + 8 * (items_out % 2), (items_out / 2 - 1) & 1));
                    if (!ok) break;
                    if (lane == 0) {
                        items[items_out % 2] = it;
                        bar_arrive(item_full + 8 * (items_out % 2));
                    }
                    items_out++;
                    if (block < 0) break;
                    const int n1 = it.key_tiles<kKeys>(1), n = max(it.key_tiles<kKeys>(0), n1), masked_from = it.masked_from<kKeys>();
                    soon = n <= 4 && a.parts == 1;
                    if (soon && lane == 0) ask_next(smem_u32(reply), asked);
                    if (n > 0) {
                        if (elect_one()) {
                            const int kv = it.head / a.group, tiles = n1 > 0 ? 2 : 1;
                            for (int t = 0; t < 2 && queries > 0 && ok; t++) ok = bar_wait(q_empty + 8 * t, (queries - 1) & 1);
                            if (ok) {
                                bar_expect(q_full, tiles * Shape::kQTile + a.tx_extra);
                                for (int t = 0; t < tiles; t++)
                                    for (int c = 0; c < Shape::kChunks; c++)
                                        tma_3d(base + t * Shape::kQTile + c * Shape::kQChunk, &q_map, q_full, c * 64, it.head,
                                               it.q0 + it.row0 + t * kRows);
                            }
                            for (int u = 0; u < 2 * n && ok; u++) {
                                const int s = (i + u) % kStages, round = (i + u) / kStages, j = u / 2;
                                if (round > 0 && !(ok = bar_wait(empty + 8 * s, (round - 1) & 1))) break;
                                bar_expect(full + 8 * s, Shape::kTile);
                                for (int c = 0; c < Shape::kChunks; c++)
                                    tma_3d(ring + s * Shape::kTile + c * Shape::kChunk, u % 2 ? &v_map : &k_map, full + 8 * s, c * 64, kv,
                                           it.k0 + j * kKeys);
                                // from here on the tile's barrier is in the phase that the look-over waits for
                                if (u % 2 && j >= masked_from) bar_arrive(v_sent + 8 * ((g + j - masked_from) % kMarks));
                            }
                        }
                        ok = __all_sync(~0u, ok);
                        queries++;
                        i += 2 * n;
                        g += max(0, n - masked_from);
                    }
                }
                // The next item is asked for only now, when all of this one's copies are on their way, unless that is short:
                // a CTA that asks earlier takes work that another could begin sooner.
                if (!ok) break;
                if (a.parts > 1) {  // a block a CTA: all of them are there at once
                    block = -1;
                    continue;
                }
                if (!soon && lane == 0) ask_next(smem_u32(reply), asked);
                if (!__all_sync(~0u, bar_wait(asked, answers++ & 1))) ok = false;
                if (ok) block = next_block(smem_u32(reply));
                __syncwarp();
            }
        } else if (warp == 11) {
            // ---- values that some row must not see
            PromptItem it;
            int i = 0, g = 0;
            for (int n_item = 0; ok && take(n_item, it); n_item++) {
                const int n0 = it.key_tiles<kKeys>(0), n1 = it.key_tiles<kKeys>(1), n = max(n0, n1);
                for (int j = it.masked_from<kKeys>(); j < n; j++, g++) {
                    const int iv = i + 2 * j + 1;
                    if (!__all_sync(~0u, bar_wait(v_sent + 8 * (g % kMarks), g / kMarks & 1) && bar_wait(full + 8 * (iv % kStages), iv / kStages & 1))) {
                        ok = false;
                        break;
                    }
                    const uint32_t tile = ring + iv % kStages * Shape::kTile;
                    const int there = min(it.klen - j * kKeys, kKeys);  // keys of the tile that exist (one at least)
                    // a piece of 16 bytes is of key u / 8 (the swizzle moves pieces inside a row of 128 bytes only)
                    uint32_t odd = 0;
#pragma unroll 1
                    for (int c = 0; c < Shape::kChunks; c++) {
                        const uint32_t chunk = tile + c * Shape::kChunk;
#pragma unroll 8
                        for (int u = lane; u < there * 8; u += 32) {
                            uint32_t x[4];
                            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                                         : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
                                         : "r"(chunk + u * 16));
#pragma unroll
                            for (int w = 0; w < 4; w++) odd |= not_finite<T>(x[w]);
                        }
                        for (int u = there * 8 + lane; u < kKeys * 8; u += 32)
                            asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(chunk + u * 16), "r"(0) : "memory");
                    }
                    // For each query tile that these values are multiplied with, and no other: that one's softmax warps may
                    // be past this item.  (At most two items ahead of a softmax warp.)
                    if (odd) {  // this lane's pieces once more (rolled up: a longer loop here cost short prompts 0.4 us)
#pragma unroll 1
                        for (uint32_t at = tile + lane * 16, c = 0; c < Shape::kChunks; c++, at = tile + c * Shape::kChunk + lane * 16)
#pragma unroll 1
                            for (; at < tile + c * Shape::kChunk + there * 128; at += 512) {
                                uint32_t x[4];
                                asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]) : "r"(at));
#pragma unroll
                                for (int w = 0; w < 4; w++) x[w] &= ~__vcmpeq2(x[w] & Half<T>::kExp, Half<T>::kExp);
                                asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]) : "memory");
                            }
                        if (j < n0) special[n_item % 4] = n_item + 1;
                        if (j < n1) special[4 + n_item % 4] = n_item + 1;
                    }
                    fence_async_smem();
                    __syncwarp();
                    if (lane == 0) bar_arrive(v_seen + 8 * (g % kMarks));
                }
                i += 2 * n;
            }
        } else {
            // ---- MMAs of query tile t (a warp each: neither waits for the other's softmax)
            const int t = warp - 8;
            constexpr uint32_t kScores = kAccF32 | Half<T>::kA | Half<T>::kB | mma_shape(kRows, kKeys);
            constexpr uint32_t kValues = kAccF32 | Half<T>::kA | Half<T>::kB | kBMajorMN | mma_shape(kRows, D);
            const uint32_t tS = tmem + Shape::kS + t * kKeys, tP = tmem + Shape::kP + t * kKeys, tO = tmem + Shape::kO + t * D;
            PromptItem it;
            int i = 0, g = 0, queries = 0, steps = 0, outputs = 0, turns = 0;
            for (int n_item = 0; ok && take(n_item, it); n_item++) {
                const int n0 = it.key_tiles<kKeys>(0), n1 = it.key_tiles<kKeys>(1), n = max(n0, n1), nt = t ? n1 : n0,
                          masked_from = it.masked_from<kKeys>();
                if (n == 0) continue;
                if (elect_one()) {
                    auto arrived = [&](int k) { return bar_wait(full + 8 * ((i + k) % kStages), (i + k) / kStages & 1); };
                    // S = Q K^T for the item's key tile j, when the scores before it have been taken
                    auto scores = [&](int j) {
                        const int k = 2 * j, x0 = steps + j;
                        if (!arrived(k) || (j < nt && x0 > 0 && !bar_wait(s_read + 8 * t, (x0 - 1) & 1))) return false;
                        if (j < nt) {
                            tc_fence_after();
                            const uint32_t qa = base + t * Shape::kQTile, ka = ring + (i + k) % kStages * Shape::kTile;
#pragma unroll
                            for (int x = 0; x < D / 16; x++)
                                mma_f16(tS, operand_desc(qa + x / 4 * Shape::kQChunk + x % 4 * 32, 16, 1024),
                                        operand_desc(ka + x / 4 * Shape::kChunk + x % 4 * 32, 16, 1024), kScores, x > 0);
                            mma_commit(s_full + 8 * t);
                        }
                        if (j + 1 == max(nt, 1)) mma_commit(q_empty + 8 * t);
                        mma_commit(empty + 8 * ((i + k) % kStages));  // (without MMAs before it, this arrives at once)
                        return true;
                    };
                    // The second tile begins when the first is through most of its first exponentials: side by side the
                    // two look for maxima together and then share the exponential unit, and leave that state only
                    // slowly (2100 cycles a step in step, 1550 out of step).
                    ok = bar_wait(q_full, queries & 1) && (t == 0 || n0 == 0 || bar_wait(turn, turns & 1)) && scores(0);
                    for (int j = 0; j < n && ok; j++) {
                        if (j + 1 < n && !(ok = scores(j + 1))) break;
                        const int k = 2 * j + 1, gv = g + j - masked_from;
                        if (!(ok = arrived(k))) break;
                        if (j < nt) {
                            if (j >= masked_from && !(ok = bar_wait(v_seen + 8 * (gv % kMarks), gv / kMarks & 1))) break;
                            // the item before has taken its output away
                            if (j == 0 && outputs > 0 && !(ok = bar_wait(o_empty + 8 * t, (outputs - 1) & 1))) break;
                            if (!(ok = bar_wait(p_full + 16 * t + (steps + j) % 2 * 8, (steps + j) / 2 & 1))) break;
                            tc_fence_after();
                            const uint32_t va = ring + (i + k) % kStages * Shape::kTile;
#pragma unroll
                            for (int x = 0; x < kKeys / 16; x++)
                                mma_f16_ta(tO, tP + (steps + j) % 2 * (kKeys / 2) + x * 8, operand_desc(va + x * 2048, Shape::kChunk, 1024), kValues, j > 0 || x > 0);
                            mma_commit(p_read + 8 * t);
                            if (j + 1 == nt) mma_commit(o_full + 8 * t);
                        }
                        mma_commit(empty + 8 * ((i + k) % kStages));
                    }
                }
                ok = __all_sync(~0u, ok);
                i += 2 * n;
                g += max(0, n - masked_from);
                queries++;
                steps += nt;
                outputs += nt > 0;
                turns += n0 > 0;
            }
        }
        if (a.parts > 1) skip_join();
    } else {
        // ---- softmax: a row a thread
        asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
        const int t = warp / 4;
        const uint32_t lanes = static_cast<uint32_t>(warp % 4 * 32) << 16, st = tmem + Shape::kS + t * kKeys + lanes,
                       pt = tmem + Shape::kP + t * kKeys + lanes, ot = tmem + Shape::kO + t * D + lanes;
        const float c = a.scale_log2;
        PromptItem it;
        int steps = 0, outputs = 0;
        bool joined = false;
        for (int n_item = 0; ok && take(n_item, it); n_item++) {
            const int nt = it.key_tiles<kKeys>(t), first = it.row0 + t * kRows, row = it.row0 + tid;
            const int sees = row + it.offset;    // the last key of this row
            float m = -INFINITY, l = 0.0f;       // m in units of the raw scores
            for (int j = 0; j < nt; j++) {
                ok = ok && bar_wait(s_full + 8 * t, (steps + j) & 1);  // (a wait that gave up is the last: no vote a step)
                __syncwarp();
                tc_fence_after();
                uint32_t s[kKeys];
#pragma unroll
                for (int x = 0; x < kKeys; x += 32) tmem_ld32(st + x, s + x);
                tmem_wait_ld<kKeys>(s);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) bar_arrive(s_read + 8 * t);
                if (j * kKeys + kKeys - 1 > first + it.offset) {
                    const int last = sees - j * kKeys;
#pragma unroll
                    for (int x = 0; x < kKeys; x++)
                        if (x > last) s[x] = 0xFF800000u;
                }
                float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int x = 0; x < kKeys; x += 2) top[x / 2 % 4] = max3(top[x / 2 % 4], __uint_as_float(s[x]), __uint_as_float(s[x + 1]));
                const float n_m = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
                const bool raise = n_m * c > m * c + kLazyLog2;
                if (__any_sync(~0u, raise)) {
                    const float f = raise ? exp2_fast((m - n_m) * c) : 1.0f;
                    if (raise) m = n_m;
                    l *= f;
                    if (j > 0) {
                        // (O may be changed when the last weights have been multiplied, and none are before these are written)
                        ok = ok && bar_wait(p_read + 8 * t, (steps + j - 1) & 1);
                        __syncwarp();
                        tc_fence_after();
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
                const uint64_t c2 = pair(c, c), less2 = pair(less, less);
                uint64_t sum[4] = {pair(0.0f, 0.0f), pair(0.0f, 0.0f), pair(0.0f, 0.0f), pair(0.0f, 0.0f)};
                uint32_t p[kKeys / 2];
#pragma unroll
                for (int y = 0; y < kKeys / 2; y++) {
                    if (y == kKeys * 3 / 8 && t == 0 && j == 0 && lane == 0) bar_arrive(turn);
                    const float2 v = halves(fma2(pair(s[2 * y], s[2 * y + 1]), c2, less2));
                    const float e0 = exp2_fast(v.x), e1 = exp2_fast(v.y);
                    sum[y % 4] = add2(sum[y % 4], pair(e0, e1));
                    p[y] = Half<T>::pack(e0, e1);
                }
                tmem_st32(pt + (steps + j) % 2 * (kKeys / 2), p);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) bar_arrive(p_full + 16 * t + (steps + j) % 2 * 8);
                const float2 both = halves(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])));
                l += both.x + both.y;
            }
            if (nt > 0) {
                ok = __all_sync(~0u, ok && bar_wait(o_full + 8 * t, outputs & 1));
                tc_fence_after();
            }
            if (!ok) break;
            // (the last key of this row once more: over the loop above there is no register for it)
            int last = tid;
            asm volatile("" : "+r"(last));
            last += it.row0 + it.offset;
            // Keys that all score -infinity leave no softmax: NaN (0 / 0), unlike no keys at all.
            if (a.parts > 1) {
                // a part's row of such keys says so by a negative sum, which counts nothing beside those of other parts
                if (l == 0.0f && nt > 0 && last >= 0) l = -1.0f;
                join_parts<T, D>(a, it, base, ot, m, l, nt > 0, smem_u32(special));
                joined = true;
                break;
            }
            if (first < it.qlen) {
                const float by = 1.0f / l;
                T *out = static_cast<T *>(a.out) + (static_cast<int64_t>(it.q0) + row) * a.out_token + it.head * a.out_head;
#pragma unroll 1
                for (int x = 0; x < D; x += 32) {
                    uint32_t o[32];
                    if (nt > 0) {
                        tmem_ld32(ot + x, o);
                        tmem_wait_ld<32>(o);
                    }
                    if (row < it.qlen) {
#pragma unroll
                        for (int y = 0; y < 32; y += 8) {
                            uint32_t h[4];
#pragma unroll
                            for (int z = 0; z < 4; z++)
                                h[z] = last < 0 ? 0u : Half<T>::pack(__uint_as_float(o[y + 2 * z]) * by, __uint_as_float(o[y + 2 * z + 1]) * by);
                            *reinterpret_cast<uint4 *>(out + x + y) = make_uint4(h[0], h[1], h[2], h[3]);
                        }
                    }
                }
            }
            if (nt > 0) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) bar_arrive(o_empty + 8 * t);
                // (this tile's values have all been looked over before its output was complete)
                if (*static_cast<volatile int *>(&special[t * 4 + n_item % 4]) == n_item + 1 && it.row0 + warp * 32 < it.qlen)
                    add_not_finite<T, D>(a, it.head, static_cast<int64_t>(it.q0) + min(row, it.qlen - 1), it.k0, it.masked_from<kKeys>() * kKeys,
                                         min(it.row0 + warp * 32 + 31, it.qlen - 1) + it.offset + 1, row < it.qlen, last);
            }
            steps += nt;
            outputs += nt > 0;
        }
        if (a.parts > 1 && !joined) skip_join();
    }
    if (!ok) failed = 1;
    __syncwarp();
    __syncthreads();
    if (failed) {
        if (tid == 0) set_status(a.status, ENTRO_E_TIMEOUT);
        drain();
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

// [tokens][heads][dim] for TMA boxes of `rows` tokens of 64 channels of a head
static int rows_map(CUtensorMap *map, int type, const void *base, int64_t tokens, int heads, int dim, int64_t token, int64_t head, int rows) {
    const uint64_t dims[3] = {static_cast<uint64_t>(dim), static_cast<uint64_t>(heads), static_cast<uint64_t>(tokens)};
    const uint64_t strides[2] = {static_cast<uint64_t>(heads > 1 ? head : dim) * 2, static_cast<uint64_t>(tokens > 1 ? token : dim) * 2};
    const uint32_t box[3] = {64, 1, static_cast<uint32_t>(rows)};
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
    if (heads < 1 || kv_heads < 1 || heads % kv_heads || tokens < 0 || keys < 0 || batch < 0 || !(scale > 0.0f) || scale > 2.0e38f) return ENTRO_E_INVAL;
    if (tokens > INT32_MAX - 256 || keys > INT32_MAX - 256) return ENTRO_E_LIMIT;
    if (tokens == 0 || batch == 0) return ENTRO_OK;
    if (!d_q || !d_cu_q || !d_out || (keys > 0 && (!d_k || !d_v))) return ENTRO_E_INVAL;
    if (!tma_rows(d_q, tokens, heads, q_token, q_head) || !tma_rows(d_k, keys, kv_heads, k_token, k_head) ||
        !tma_rows(d_v, keys, kv_heads, v_token, v_head) || !aligned16(d_out) || out_token % 8 || out_head % 8 ||
        !separate_rows(tokens, heads, head_dim, out_token, out_head))
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
    const int64_t blocks = (tokens + INT64_C(255) * batch) / 256 * heads;  // the most there may be
    if (blocks > INT32_MAX) return ENTRO_E_LIMIT;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
    size_t smem;
    const void *fn = type == ENTRO_BF16 ? pick_prompt<__nv_bfloat16>(head_dim, &smem) : pick_prompt<__half>(head_dim, &smem);
    const int keys_of = PromptShape<64>::kKeys;  // (the same for all widths)
    int r = allow_smem(fn, dev);
    // Few blocks over many keys: as many CTAs share the keys of a block as all find room at once, with four key tiles each
    // at least on an average sequence.  (40 queries over 4040 keys, 32 heads of 128: 47 us alone, 20 by four; over 1024: 16
    // and 12.  With clusters that come in two waves, 16 heads by eight: 29, by four 19.  Below 1024 keys there is little to
    // gain, and results that do not depend on the batch to lose.)
    a.parts = 1;
    if (keys / batch >= 1024)
        for (int parts = static_cast<int>(std::min<int64_t>(keys / batch / 256, 8)); parts > 1 && a.parts == 1 && r == ENTRO_OK; parts--) {
            int clusters = 0;
            r = clusters_at_once(fn, dev, kPromptThreads, smem, parts, &clusters);
            if (blocks <= clusters) a.parts = parts;
        }
    CUtensorMap q_map, k_map, v_map;
    if (r == ENTRO_OK) r = rows_map(&q_map, type, d_q, tokens, heads, head_dim, q_token, q_head, kRows);
    // (without keys nothing is copied; the maps only have to be valid)
    if (r == ENTRO_OK) r = keys ? rows_map(&k_map, type, d_k, keys, kv_heads, head_dim, k_token, k_head, keys_of) : (k_map = q_map, ENTRO_OK);
    if (r == ENTRO_OK) r = keys ? rows_map(&v_map, type, d_v, keys, kv_heads, head_dim, v_token, v_head, keys_of) : (v_map = q_map, ENTRO_OK);
    if (r != ENTRO_OK) return r;
    void *args[] = {&q_map, &k_map, &v_map, &a};
    e = launch_ex(fn, dim3(static_cast<unsigned>(blocks * a.parts)), kPromptThreads, smem, static_cast<cudaStream_t>(stream), a.parts, false, args);
    return e == cudaSuccess ? ENTRO_OK : cuda_fail(e, "entro_attention_prompt");
}
