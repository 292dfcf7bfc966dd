// product.cu -- products of more activation rows than the fused GEMV takes:
// activations quantized to 8 bits per token, times 8-bit weight codes on the
// integer tensor cores (tcgen05, kind::i8), with a scale for each token and
// channel.
//
//   a_t = max_k |x[t, k]|,  q[t, k] = rint(127 x[t, k] / a_t),  s_t = a_t / 127
//   y[t, n] = s_t w_n (sum_k q[t, k] c[n, k] - z_n sum_k q[t, k])
//
// The codes c are what entro_decode_codes writes for an 8-bit tensor (unsigned,
// with the tensor's zero point z and scale w) or any other 8-bit weights.  The
// sums are exact 32-bit integers, so a result does not depend on how the work
// is split.  In the MMA the weights are operand A (their rows are the TMEM
// lanes) and the tokens operand B, so few tokens make a narrow tile instead of
// a padded one, and a warp's 32 outputs of one token are adjacent in memory.
#include <algorithm>
#include <cstring>

#include "launch.h"
#include "sm100.cuh"

namespace entro {
using namespace sm100;

// ------------------------------------------------------------------ tokens to 8 bits

struct QuantArgs {
    const uint16_t *x;
    int8_t *q;
    float *scale;
    int32_t *sum;
    int64_t tokens, cols, ldx, ldq;
};

// One CTA a token.  The row stays in registers between its two uses (VECS
// 16-byte loads a thread; 0: rows too long or too unaligned for that, read twice
// element by element).  Bound by memory, 3 bytes an element: 8192 x 14336 in 65 to
// 70 us, 5.2 TB/s; 500 x 28672 in 11 us (read twice: 29).
template <typename T, int THREADS, int VECS>
__global__ void __launch_bounds__(THREADS) quantize_kernel(const QuantArgs a) {
    __shared__ uint32_t red_max[THREADS / 32];
    __shared__ int red_sum[THREADS / 32];
    dependents_may_launch();
    const int tid = threadIdx.x;
    const int64_t t = blockIdx.x;
    const uint16_t *row = a.x + t * a.ldx;
    uint4 v[VECS ? VECS : 1];
    uint32_t m = 0;  // of the halves without their signs: ordered as their values are, infinities and NaN at the top
    if (VECS) {
#pragma unroll
        for (int i = 0; i < VECS; i++) {
            const int64_t k = (static_cast<int64_t>(i) * THREADS + tid) * 8;
            v[i] = make_uint4(0, 0, 0, 0);
            if (k + 8 <= a.cols) {
                v[i] = __ldg(reinterpret_cast<const uint4 *>(row + k));
            } else if (k < a.cols) {
                uint16_t e[8] = {0, 0, 0, 0, 0, 0, 0, 0};
                for (int j = 0; j < 8 && k + j < a.cols; j++) e[j] = row[k + j];
                std::memcpy(&v[i], e, 16);
            }
            m = __vmaxu2(m, __vmaxu2(__vmaxu2(v[i].x & 0x7FFF7FFFu, v[i].y & 0x7FFF7FFFu),
                                     __vmaxu2(v[i].z & 0x7FFF7FFFu, v[i].w & 0x7FFF7FFFu)));
        }
    } else {
        for (int64_t k = tid; k < a.cols; k += THREADS) m = max(m, static_cast<uint32_t>(row[k] & 0x7FFF));
    }
    m = max(m & 0xFFFF, m >> 16);
    m = __reduce_max_sync(~0u, m);
    if (tid % 32 == 0) red_max[tid / 32] = m;
    __syncthreads();
    m = 0;
    for (int w = 0; w < THREADS / 32; w++) m = max(m, red_max[w]);
    const BlockCode<T> code(m);
    int sum = 0;
    if (VECS) {
#pragma unroll
        for (int i = 0; i < VECS; i++) {
            const int64_t k = (static_cast<int64_t>(i) * THREADS + tid) * 8;
            if (k >= a.cols) break;
            const uint2 o = code.eight(v[i]);
            sum = __dp4a(static_cast<int>(o.x), 0x01010101, __dp4a(static_cast<int>(o.y), 0x01010101, sum));
            // the row pitch is a multiple of 16 bytes: the last vector's zeros fall inside it
            *reinterpret_cast<uint2 *>(a.q + t * a.ldq + k) = o;
        }
    } else {
        for (int64_t k = tid; k < a.cols; k += THREADS) {
            const int c = code.one(Half<T>::widen(row[k]).x);
            a.q[t * a.ldq + k] = static_cast<int8_t>(c);
            sum += c;
        }
    }
    sum = __reduce_add_sync(~0u, sum);
    if (tid % 32 == 0) red_sum[tid / 32] = sum;
    __syncthreads();
    if (tid == 0) {
        sum = 0;
        for (int w = 0; w < THREADS / 32; w++) sum += red_sum[w];
        a.sum[t] = sum;
        a.scale[t] = code.scale();
    }
}

// ------------------------------------------------------------------ codes to a byte each

// Packed 4-bit codes, or 8-bit ones in rows of any length, to a byte each in
// rows of `ld` bytes (a multiple of 16, which the product's copies need).
__global__ void __launch_bounds__(256) unpack_kernel(const uint8_t *codes, int bits, int64_t rows, int64_t cols, uint8_t *out,
                                                     int64_t ld) {
    const int64_t words = ld / 16, total = rows * words;
    for (int64_t i = blockIdx.x * 256LL + threadIdx.x; i < total; i += gridDim.x * 256LL) {
        const int64_t r = i / words, k0 = i % words * 16, first = r * cols + k0;
        uint32_t o[4] = {0, 0, 0, 0};
        if (bits == 4 && first % 2 == 0 && k0 + 16 <= cols && first % 16 == 0) {
            const uint2 v = __ldg(reinterpret_cast<const uint2 *>(codes + first / 2));
            const uint32_t w[2] = {v.x, v.y};
#pragma unroll
            for (int j = 0; j < 2; j++) {
                const uint32_t lo = w[j] & 0x0F0F0F0Fu, hi = (w[j] >> 4) & 0x0F0F0F0Fu;
                o[2 * j] = __byte_perm(lo, hi, 0x5140);
                o[2 * j + 1] = __byte_perm(lo, hi, 0x7362);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 16; j++) {
                if (k0 + j >= cols) break;
                const int64_t s = first + j;
                const uint32_t c = bits == 4 ? (codes[s / 2] >> (s % 2 * 4)) & 15u : codes[s];
                o[j / 4] |= c << (j % 4 * 8);
            }
        }
        *reinterpret_cast<uint4 *>(out + r * ld + k0) = make_uint4(o[0], o[1], o[2], o[3]);
    }
}

// ------------------------------------------------------------------ the product

enum OutType { OUT_F32 = 0, OUT_BF16T = 1, OUT_F16T = 2 };

struct ProductArgs {
    const float *x_scale;
    const int32_t *x_sum;
    const float *w_scale;   // per channel, or null: w_scale_all
    const int32_t *w_zero;  // per channel, or null: w_zero_all
    float w_scale_all;
    int32_t w_zero_all;
    void *y;
    int64_t ldy;
    int32_t *status;
    int tokens, rows, cols;
    int bn;          // tokens of a tile
    int chunks;      // 128-byte steps over cols
    int stages;
    int row_tiles, token_tiles;
    uint32_t idesc, tmem_cols, tx_extra;
};

template <int OUT>
struct OutOf;
template <>
struct OutOf<OUT_F32> {
    using Type = float;
    static __device__ __forceinline__ float of(float v) { return v; }
};
template <>
struct OutOf<OUT_BF16T> {
    using Type = __nv_bfloat16;
    static __device__ __forceinline__ __nv_bfloat16 of(float v) { return __float2bfloat16_rn(v); }
};
template <>
struct OutOf<OUT_F16T> {
    using Type = __half;
    static __device__ __forceinline__ __half of(float v) { return __float2half_rn(v); }
};

// One channel's part of the epilogue.
struct Channel {
    float scale;
    int32_t zero;
    bool wide;  // the zero point is outside the codes' range: its product may pass 32 bits

    __device__ __forceinline__ void load(const ProductArgs &a, int n) {
        scale = n < a.rows ? (a.w_scale ? a.w_scale[n] : a.w_scale_all) : 0.0f;
        zero = n < a.rows ? (a.w_zero ? a.w_zero[n] : a.w_zero_all) : 0;
        wide = zero < -256 || zero > 256;
    }
    // acc - zero * sum: in the codes' range the difference is a sum of cols products of at most 127 * 511,
    // below 2^31 for cols up to 32768; past that, or for other zero points (in64), it is taken in 64 bits
    template <bool in64>
    __device__ __forceinline__ float value(int32_t acc, int32_t sum, float x_scale) const {
        const float v = in64 ? static_cast<float>(static_cast<long long>(acc) - static_cast<long long>(zero) * sum)
                             : static_cast<float>(acc - zero * sum);
        return v * (x_scale * scale);
    }
    // N tokens' outputs of this channel, the first at y, the next ones ldy further each; `left` of them exist
    template <int OUT, int N, bool in64>
    __device__ __forceinline__ void store(const uint32_t *acc, const float *xs, const int32_t *xz, typename OutOf<OUT>::Type *y,
                                          int64_t ldy, int left) const {
        if (left >= N) {
#pragma unroll
            for (int j = 0; j < N; j++, y += ldy) *y = OutOf<OUT>::of(value<in64>(static_cast<int32_t>(acc[j]), xz[j], xs[j]));
        } else {
#pragma unroll
            for (int j = 0; j < N; j++, y += ldy)
                if (j < left) *y = OutOf<OUT>::of(value<in64>(static_cast<int32_t>(acc[j]), xz[j], xs[j]));
        }
    }
};

constexpr int kChunkBytes = 128;                 // k bytes of a stage: one swizzle row
constexpr int kTileRows = 128;                   // weight rows of a CTA's tile
constexpr int kABytes = kTileRows * kChunkBytes;

// Few tokens: one tile of 128 weight rows by all tokens (up to 256) a cluster,
// whose CTAs share the k range; the partial sums meet in shared memory over the
// cluster (each CTA finishes a share of the tokens).  Bound by reading the
// weights once; the split is what lets a projection of 16 row tiles use all SMs: 24 tokens
// x 2048 x 2048 in 6.6 us, 64 x 4096 x 4096 in 8.6.
template <int OUT>
__global__ void __launch_bounds__(192, 1) product_narrow_kernel(const __grid_constant__ CUtensorMap w_map,
                                                                const __grid_constant__ CUtensorMap x_map,
                                                                const __grid_constant__ ProductArgs a) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bars[2 * 16 + 1];
    __shared__ uint32_t tmem_base;
    __shared__ int failed;
    __shared__ float xs[256];
    __shared__ int32_t xz[256];
    const uint32_t base = (smem_u32(smem_raw) + 1023) & ~1023u;
    const int tid = threadIdx.x, warp = tid / 32;
    const int split = gridDim.x, part = blockIdx.x, tile = blockIdx.y;
    const int c0 = static_cast<int>(static_cast<int64_t>(a.chunks) * part / split);
    const int c1 = static_cast<int>(static_cast<int64_t>(a.chunks) * (part + 1) / split);
    const uint32_t full = smem_u32(bars), empty = full + 8 * a.stages, done = full + 16 * a.stages;
    const uint32_t b_bytes = a.bn * kChunkBytes, stage_bytes = kABytes + b_bytes;
    if (tid == 0) {
        for (int s = 0; s < a.stages; s++) {
            bar_init(full + 8 * s, 1);
            bar_init(empty + 8 * s, 1);
        }
        bar_init(done, 1);
        fence_bar_init();
        failed = 0;
        prefetch_map(&w_map);
        prefetch_map(&x_map);
    }
    if (warp == 0) tmem_alloc<1>(smem_u32(&tmem_base), a.tmem_cols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base;
    wait_for_prior_grid();
    bool ok = true;
    if (warp == 4) {
        if (elect_one()) {
            for (int c = c0; c < c1; c++) {
                const int i = c - c0, s = i % a.stages, round = i / a.stages;
                if (round > 0 && !bar_wait(empty + 8 * s, (round - 1) & 1)) {
                    ok = false;
                    break;
                }
                bar_expect(full + 8 * s, stage_bytes + a.tx_extra);
                tma_2d(base + s * stage_bytes, &w_map, full + 8 * s, c * kChunkBytes, tile * kTileRows);
                tma_2d(base + s * stage_bytes + kABytes, &x_map, full + 8 * s, c * kChunkBytes, 0);
            }
        }
    } else if (warp == 5) {
        if (elect_one()) {
            for (int c = c0; c < c1; c++) {
                const int i = c - c0, s = i % a.stages, round = i / a.stages;
                if (!bar_wait(full + 8 * s, round & 1)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint64_t da = operand_desc(base + s * stage_bytes, 16, 1024);
                const uint64_t db = operand_desc(base + s * stage_bytes + kABytes, 16, 1024);
#pragma unroll
                for (int k = 0; k < kChunkBytes / 32; k++) mma_i8<1>(tmem, da + 2 * k, db + 2 * k, a.idesc, i > 0 || k > 0);
                mma_commit(empty + 8 * s);
            }
            if (ok) mma_commit(done);
        }
    } else {
        for (int t = tid; t < a.tokens; t += 128) {
            xs[t] = a.x_scale[t];
            xz[t] = a.x_sum[t];
        }
        ok = bar_wait(done, 0);
        tc_fence_after();
    }
    if (!ok) failed = 1;
    __syncwarp();
    __syncthreads();
    const bool bad = failed != 0;
    if (bad) {
        if (tid == 0) set_status(a.status, ENTRO_E_TIMEOUT);
        drain();
    }
    const int per = (a.bn + split - 1) / split;  // tokens that a CTA of the cluster finishes
    const int n = tile * kTileRows + tid;        // (warps 0 to 3)
    Channel ch;
    if (warp < 4) ch.load(a, n);
    const uint32_t lanes = tmem + (static_cast<uint32_t>(warp * 32) << 16);
    const bool in64 = __any_sync(~0u, warp < 4 && ch.wide) || a.cols > 32768;
    if (split == 1) {
        if (warp < 4 && !bad) {
            for (int t0 = 0; t0 < a.bn; t0 += 16) {
                uint32_t r[16];
                tmem_ld16(lanes + t0, r);
                tmem_wait_ld<16>(r);
                if (n < a.rows) {
                    auto *y = static_cast<typename OutOf<OUT>::Type *>(a.y) + t0 * a.ldy + n;
                    if (in64) ch.template store<OUT, 16, true>(r, xs + t0, xz + t0, y, a.ldy, a.tokens - t0);
                    else ch.template store<OUT, 16, false>(r, xs + t0, xz + t0, y, a.ldy, a.tokens - t0);
                }
            }
        }
    } else {
        // [source CTA][token of the share][row]: every CTA's operands have been consumed behind the barrier
        cluster_sync();
        if (warp < 4) {
            const uint32_t mine = base + (part * per * kTileRows + tid) * 4;
            int owner = 0, in_share = 0;
            uint32_t to = map_to(mine, 0);
            for (int t0 = 0; t0 < a.bn; t0 += 16) {
                uint32_t r[16];
                tmem_ld16(lanes + t0, r);
                tmem_wait_ld<16>(r);
#pragma unroll
                for (int j = 0; j < 16; j++) {
                    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(to), "r"(r[j]) : "memory");
                    to += kTileRows * 4;
                    if (++in_share == per) {
                        in_share = 0;
                        to = map_to(mine, min(++owner, split - 1));
                    }
                }
            }
        }
        cluster_sync();
        if (warp < 4 && !bad) {
            for (int j = 0; j < per; j++) {
                const int t = part * per + j;
                if (t >= a.tokens || t >= a.bn) break;
                int32_t v[8], acc = 0;
#pragma unroll
                for (int s = 0; s < 8; s++)
                    if (s < split) asm volatile("ld.shared.s32 %0, [%1];" : "=r"(v[s]) : "r"(base + ((s * per + j) * kTileRows + tid) * 4));
#pragma unroll
                for (int s = 0; s < 8; s++)
                    if (s < split) acc += v[s];
                if (n < a.rows) {
                    auto *y = static_cast<typename OutOf<OUT>::Type *>(a.y) + t * a.ldy + n;
                    const uint32_t bits = static_cast<uint32_t>(acc);
                    if (in64) ch.template store<OUT, 1, true>(&bits, xs + t, xz + t, y, a.ldy, 1);
                    else ch.template store<OUT, 1, false>(&bits, xs + t, xz + t, y, a.ldy, 1);
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) tmem_free<1>(tmem, a.tmem_cols);
}

// Many tokens: pairs of CTAs walk the tiles of 256 weight rows by bn tokens.
// Each CTA brings its 128 rows and half of the tokens, the pair's MMAs (issued
// by CTA 0) read both halves from both SMs, so a tile of 256 x 256 costs each SM
// 32 KB of copies per 128 of k.  Two accumulators in TMEM: a tile's epilogue
// runs beside the next tile's MMAs.  Bound by the MMAs for long k (8192 tokens x 4096
// x 14336: 302 us, 3.19 P operations/s, twice the rate of 16-bit products), by copies
// from L2 and unfilled waves for few tokens (515 x 14336 x 4096: 30 us, 2.0 P).
template <int OUT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(256, 1)
    product_wide_kernel(const __grid_constant__ CUtensorMap w_map, const __grid_constant__ CUtensorMap x_map,
                        const __grid_constant__ ProductArgs a) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bars[2 * 8 + 4];
    __shared__ uint32_t tmem_base;
    __shared__ int failed, epilogue_failed;
    __shared__ float xs[2][256];
    __shared__ int32_t xz[2][256];
    const uint32_t base = (smem_u32(smem_raw) + 1023) & ~1023u;
    const int tid = threadIdx.x, warp = tid / 32;
    const uint32_t rank = cluster_rank();
    const uint32_t full = smem_u32(bars), empty = full + 8 * a.stages, acc_full = full + 16 * a.stages, acc_empty = acc_full + 16;
    const int half = a.bn / 2;
    const uint32_t b_bytes = half * kChunkBytes, stage_bytes = kABytes + b_bytes;
    if (tid == 0) {
        for (int s = 0; s < a.stages; s++) {
            bar_init(full + 8 * s, 1);
            bar_init(empty + 8 * s, 1);
        }
        for (int s = 0; s < 2; s++) {
            bar_init(acc_full + 8 * s, 1);
            bar_init(acc_empty + 8 * s, 8);  // four epilogue warps of both CTAs
        }
        fence_bar_init();
        failed = epilogue_failed = 0;
        prefetch_map(&w_map);
        prefetch_map(&x_map);
    }
    if (warp == 2) tmem_alloc<2>(smem_u32(&tmem_base), 512);
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = tmem_base;
    wait_for_prior_grid();
    const int tiles = a.row_tiles * a.token_tiles, pairs = gridDim.x / 2;
    // groups of 8 row tiles, rows fastest: the tiles in flight share weights and tokens in L2
    auto where = [&](int i, int &row, int &token) {
        const int per_group = 8 * a.token_tiles, g = i / per_group, r = i - g * per_group;
        const int high = min(8, a.row_tiles - g * 8);
        row = g * 8 + r % high;
        token = r / high;
    };
    bool ok = true;
    if (warp == 0) {
        if (elect_one()) {
            int i = 0;
            for (int tile = blockIdx.x / 2; tile < tiles && ok; tile += pairs) {
                int row, token;
                where(tile, row, token);
                for (int c = 0; c < a.chunks; c++, i++) {
                    const int s = i % a.stages, round = i / a.stages;
                    if (round > 0 && !bar_wait(empty + 8 * s, (round - 1) & 1)) {
                        ok = false;
                        break;
                    }
                    if (rank == 0) bar_expect(full + 8 * s, 2 * stage_bytes + a.tx_extra);
                    const uint32_t bar = map_to(full + 8 * s, 0);
                    tma_2d_pair(base + s * stage_bytes, &w_map, bar, c * kChunkBytes, row * 256 + rank * kTileRows);
                    tma_2d_pair(base + s * stage_bytes + kABytes, &x_map, bar, c * kChunkBytes, token * a.bn + rank * half);
                }
            }
        }
    } else if (warp == 1 && rank == 0) {
        if (elect_one()) {
            int i = 0, n = 0;
            for (int tile = blockIdx.x / 2; tile < tiles && ok; tile += pairs, n++) {
                const int acc = n & 1;
                if (n >= 2 && !bar_wait(acc_empty + 8 * acc, (n / 2 - 1) & 1)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                for (int c = 0; c < a.chunks; c++, i++) {
                    const int s = i % a.stages, round = i / a.stages;
                    if (!bar_wait(full + 8 * s, round & 1)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t da = operand_desc(base + s * stage_bytes, 16, 1024);
                    const uint64_t db = operand_desc(base + s * stage_bytes + kABytes, 16, 1024);
#pragma unroll
                    for (int k = 0; k < kChunkBytes / 32; k++)
                        mma_i8<2>(tmem + acc * 256, da + 2 * k, db + 2 * k, a.idesc, c > 0 || k > 0);
                    mma_commit_pair(empty + 8 * s);
                }
                if (ok) mma_commit_pair(acc_full + 8 * acc);
            }
        }
    } else if (warp >= 4) {
        const int e = warp - 4, et = tid - 128;
        int n = 0;
        for (int tile = blockIdx.x / 2; tile < tiles; tile += pairs, n++) {
            const int acc = n & 1;
            int row, token;
            where(tile, row, token);
            // the tile's token scales and sums, read while its MMAs run; every epilogue warp has
            // left this buffer's previous tile when the one after that tile's barrier below is passed
            for (int j = et; j < a.bn; j += 128) {
                const int t = token * a.bn + j;
                xs[acc][j] = t < a.tokens ? a.x_scale[t] : 0.0f;
                xz[acc][j] = t < a.tokens ? a.x_sum[t] : 0;
            }
            asm volatile("bar.sync 1, 128;" ::: "memory");
            const int ch_row = row * 256 + rank * kTileRows + et;
            Channel ch;
            ch.load(a, ch_row);
            const bool in64 = __any_sync(~0u, ch.wide) || a.cols > 32768;
            ok = bar_wait(acc_full + 8 * acc, (n / 2) & 1);
            if (!ok) epilogue_failed = 1;
            asm volatile("bar.sync 1, 128;" ::: "memory");  // all four warps stop at the same tile
            if (*static_cast<volatile int *>(&epilogue_failed)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const uint32_t lanes = tmem + acc * 256 + (static_cast<uint32_t>(e * 32) << 16);
            for (int t0 = 0; t0 < a.bn; t0 += 32) {
                uint32_t r[32];
                tmem_ld32(lanes + t0, r);
                tmem_wait_ld<32>(r);
                const int t = token * a.bn + t0;
                if (ch_row < a.rows && t < a.tokens) {
                    auto *y = static_cast<typename OutOf<OUT>::Type *>(a.y) + t * a.ldy + ch_row;
                    if (in64) ch.template store<OUT, 32, true>(r, xs[acc] + t0, xz[acc] + t0, y, a.ldy, a.tokens - t);
                    else ch.template store<OUT, 32, false>(r, xs[acc] + t0, xz[acc] + t0, y, a.ldy, a.tokens - t);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (tid % 32 == 0) bar_arrive_cluster(map_to(acc_empty + 8 * acc, 0));
        }
    }
    if (!ok) failed = 1;
    __syncwarp();
    __syncthreads();
    if (failed) {
        if (tid == 0) set_status(a.status, ENTRO_E_TIMEOUT);
        drain();
    }
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
    if (warp == 2) tmem_free<2>(tmem, 512);
}

// ------------------------------------------------------------------ host side

// What a call takes in cycles, roughly, by either kernel; measured over 24 to 515 tokens, 1024 to 14336 rows and 512 to
// 16384 columns on 148 SMs.  A step of 128 k costs its copies, 2.8 cycles a row of 128 bytes with all SMs copying from L2
// (540 cycles at 128 tokens a pair, 730 at 256, where the MMAs alone need 512), and some latency at least.  Wide tiles
// start and end cheaper (5000 cycles against 9000, and 60 a token for the cluster's sums); narrow ones split k and so
// keep SMs busy when there are few row tiles: 64 tokens x 4096 x 4096 8.8 us narrow, 10.7 wide; 128 tokens 12.2 and 11.1;
// 128 tokens x 14336 x 4096 (k first) 22 and 28, x 4096 x 14336 18.1 and 15.0.
static double wide_cycles(int64_t tiles, int pairs, int chunks, int bn) {
    const double busy = std::min(1.0, static_cast<double>(tiles) / pairs);
    const double step = std::max({460.0, 2.0 * bn, 2.85 * (kTileRows + bn / 2) * busy}) + 0.5 * bn;
    return static_cast<double>((tiles + pairs - 1) / pairs) * chunks * step + 5000;
}
static double narrow_cycles(int64_t row_tiles, int split, int sms, int chunks, int bn) {
    const int64_t ctas = row_tiles * split;
    const double busy = std::min(1.0, static_cast<double>(ctas) / sms);
    const double step = std::max(300.0, 2.85 * (kTileRows + bn) * busy);
    return static_cast<double>((ctas + sms - 1) / sms) * ((chunks + split - 1) / split) * step + 9000 + (split > 1 ? 60.0 * bn : 0.0);
}

// The kernel and the tile width whose waves cost least.
static entro_product_plan plan_product(int64_t tokens, int64_t rows, int chunks, int sms) {
    // wide tiles: pairs of SMs walk them
    const int pairs = sms / 2;
    const int64_t wide_rows = (rows + 255) / 256;
    double wide_cost = 1e300;
    int wide_bn = 256;
    for (int bn = 256; bn >= 32; bn -= 32) {
        const double c = wide_cycles((tokens + bn - 1) / bn * wide_rows, pairs, chunks, bn);
        if (c < wide_cost) wide_cost = c, wide_bn = bn;
    }
    // one narrow tile of all tokens: k split as long as that fills SMs
    const int narrow_bn = static_cast<int>(std::min<int64_t>((tokens + 15) / 16 * 16, 272));
    const int64_t narrow_rows = (rows + kTileRows - 1) / kTileRows;
    int split = 1;
    while (split < 8 && split * 2 <= chunks && narrow_rows * split * 2 <= sms) split *= 2;
    if (narrow_bn <= 256 && narrow_rows <= 65535 && narrow_cycles(narrow_rows, split, sms, chunks, narrow_bn) < wide_cost) {
        const int stage = kABytes + narrow_bn * kChunkBytes;
        return {0, narrow_bn, split, std::min(8, 100 * 1024 / stage < 3 ? 200 * 1024 / stage : 100 * 1024 / stage), narrow_rows, 1};
    }
    const int stage = kABytes + wide_bn / 2 * kChunkBytes;
    return {1, wide_bn, 1, std::min(8, 200 * 1024 / stage), wide_rows, (tokens + wide_bn - 1) / wide_bn};
}

// 256 threads of up to four 16-byte loads; from 8192 columns on 512 (14336: 65 to 70 us, by 256 of eight loads 74 to 81).
template <typename T>
static const void *pick_quantize(int64_t cols, bool whole, unsigned *threads) {
    *threads = whole && cols > 8192 && cols <= 32768 ? 512 : 256;
    return !whole || cols > 32768 ? reinterpret_cast<const void *>(quantize_kernel<T, 256, 0>)
           : cols <= 2048         ? reinterpret_cast<const void *>(quantize_kernel<T, 256, 1>)
           : cols <= 4096         ? reinterpret_cast<const void *>(quantize_kernel<T, 256, 2>)
           : cols <= 8192         ? reinterpret_cast<const void *>(quantize_kernel<T, 256, 4>)
           : cols <= 16384        ? reinterpret_cast<const void *>(quantize_kernel<T, 512, 4>)
                                  : reinterpret_cast<const void *>(quantize_kernel<T, 512, 8>);
}

}  // namespace entro

using namespace entro;

extern "C" int entro_quantize_tokens(const void *d_x, int32_t type, int64_t tokens, int64_t cols, int64_t ldx, int8_t *d_q,
                                     int64_t ldq, float *d_scale, int32_t *d_sum, void *stream) {
    if ((type != ENTRO_BF16 && type != ENTRO_F16) || tokens < 0 || cols < 1 || ldx < cols || ldq < cols) return ENTRO_E_INVAL;
    if (tokens > ENTRO_PRODUCT_MAX_TOKENS || cols > ENTRO_PRODUCT_MAX_COLS) return ENTRO_E_LIMIT;
    if (tokens == 0) return ENTRO_OK;
    if (!d_x || !d_q || !d_scale || !d_sum || ldq % 16 || !aligned16(d_q) || (reinterpret_cast<uintptr_t>(d_x) & 1)) return ENTRO_E_INVAL;
    QuantArgs a{static_cast<const uint16_t *>(d_x), d_q, d_scale, d_sum, tokens, cols, ldx, ldq};
    const bool whole = aligned16(d_x) && ldx % 8 == 0;  // rows in 16-byte pieces
    unsigned threads;
    const void *fn = type == ENTRO_BF16 ? pick_quantize<__nv_bfloat16>(cols, whole, &threads) : pick_quantize<__half>(cols, whole, &threads);
    void *args[] = {&a};
    cudaError_t e = launch_ex(fn, dim3(static_cast<unsigned>(tokens)), threads, 0, static_cast<cudaStream_t>(stream), 1, false, args);
    return e == cudaSuccess ? ENTRO_OK : cuda_fail(e, "entro_quantize_tokens");
}

extern "C" int entro_unpack_codes(const void *d_codes, int32_t bits, int64_t rows, int64_t cols, void *d_out, int64_t ld, void *stream) {
    if ((bits != 4 && bits != 8) || rows < 0 || cols < 0 || ld < cols || ld % 16) return ENTRO_E_INVAL;
    if (rows == 0 || cols == 0) return ENTRO_OK;
    if (!d_codes || !d_out || !aligned16(d_codes) || !aligned16(d_out) || d_codes == d_out) return ENTRO_E_INVAL;
    const int64_t words = rows * (ld / 16);
    const uint8_t *codes = static_cast<const uint8_t *>(d_codes);
    uint8_t *out = static_cast<uint8_t *>(d_out);
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
    DeviceInfo di;
    const int r = device_info(dev, &di);
    if (r != ENTRO_OK) return r;
    void *args[] = {&codes, &bits, &rows, &cols, &out, &ld};
    e = launch_ex(reinterpret_cast<const void *>(unpack_kernel), dim3(static_cast<unsigned>(std::min<int64_t>((words + 255) / 256, di.sms * 16))),
                  256, 0, static_cast<cudaStream_t>(stream), 1, false, args);
    return e == cudaSuccess ? ENTRO_OK : cuda_fail(e, "entro_unpack_codes");
}

extern "C" int entro_matmul_i8(const int8_t *d_q, int64_t ldq, const float *d_x_scale, const int32_t *d_x_sum, int64_t tokens,
                               const void *d_w, int32_t w_type, int64_t ldw, int64_t rows, int64_t cols, const float *d_w_scale,
                               float w_scale, const int32_t *d_w_zero, int32_t w_zero, void *d_y, int32_t y_type, int64_t ldy,
                               int32_t *d_status, void *stream) {
    if (tokens < 0 || rows < 0 || cols < 1 || ldq < cols || ldw < cols || ldy < rows) return ENTRO_E_INVAL;
    if ((w_type != ENTRO_U8 && w_type != ENTRO_S8) || (y_type != ENTRO_F32 && y_type != ENTRO_BF16 && y_type != ENTRO_F16)) return ENTRO_E_INVAL;
    if (tokens > ENTRO_PRODUCT_MAX_TOKENS || cols > ENTRO_PRODUCT_MAX_COLS || rows > (INT64_C(1) << 30)) return ENTRO_E_LIMIT;
    if (tokens == 0 || rows == 0) return ENTRO_OK;
    if (!d_q || !d_x_scale || !d_x_sum || !d_w || !d_y) return ENTRO_E_INVAL;
    if (ldq % 16 || ldw % 16 || !aligned16(d_q) || !aligned16(d_w)) return ENTRO_E_INVAL;
    if (reinterpret_cast<uintptr_t>(d_y) & (y_type == ENTRO_F32 ? 3 : 1)) return ENTRO_E_INVAL;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
    DeviceInfo di;
    int r = device_info(dev, &di);
    if (r != ENTRO_OK) return r;

    ProductArgs a;
    std::memset(&a, 0, sizeof(a));
    a.x_scale = d_x_scale;
    a.x_sum = d_x_sum;
    a.w_scale = d_w_scale;
    a.w_zero = d_w_zero;
    a.w_scale_all = w_scale;
    a.w_zero_all = w_zero;
    a.y = d_y;
    a.ldy = ldy;
    a.status = d_status;
    a.tokens = static_cast<int>(tokens);
    a.rows = static_cast<int>(rows);
    a.cols = static_cast<int>(cols);
    a.chunks = static_cast<int>((cols + kChunkBytes - 1) / kChunkBytes);
    a.tx_extra = test_tx_extra();
    const uint32_t types = kAccS32 | (w_type == ENTRO_S8 ? kAS8 : kAU8) | kBS8;
    const entro_product_plan plan = plan_product(tokens, rows, a.chunks, di.sms);
    const bool narrow = !plan.wide;
    a.bn = plan.tile_tokens;
    a.stages = plan.stages;
    if (plan.row_tiles * plan.token_tiles > INT32_MAX) return ENTRO_E_LIMIT;
    a.row_tiles = static_cast<int>(plan.row_tiles);
    a.token_tiles = static_cast<int>(plan.token_tiles);
    size_t smem;
    dim3 grid;
    unsigned cluster, threads;
    const void *fn;
    if (narrow) {
        const int stage = kABytes + a.bn * kChunkBytes, split = plan.split;
        a.tmem_cols = 32;
        while (a.tmem_cols < static_cast<uint32_t>(a.bn)) a.tmem_cols *= 2;
        a.idesc = types | mma_shape(kTileRows, a.bn);
        const int share = (a.bn + split - 1) / split;
        smem = 1024 + std::max<size_t>(static_cast<size_t>(a.stages) * stage, static_cast<size_t>(split) * share * kTileRows * 4);
        grid = dim3(split, a.row_tiles);
        cluster = split;
        threads = 192;
        fn = y_type == ENTRO_F32 ? reinterpret_cast<const void *>(product_narrow_kernel<OUT_F32>)
             : y_type == ENTRO_BF16 ? reinterpret_cast<const void *>(product_narrow_kernel<OUT_BF16T>)
                                    : reinterpret_cast<const void *>(product_narrow_kernel<OUT_F16T>);
    } else {
        const int stage = kABytes + a.bn / 2 * kChunkBytes;
        a.idesc = types | mma_shape(256, a.bn);
        smem = 1024 + static_cast<size_t>(a.stages) * stage;
        grid = dim3(2 * static_cast<unsigned>(std::min<int64_t>(plan.row_tiles * plan.token_tiles, di.sms / 2)));
        cluster = 1;  // the pair is the kernel's own cluster size
        threads = 256;
        fn = y_type == ENTRO_F32 ? reinterpret_cast<const void *>(product_wide_kernel<OUT_F32>)
             : y_type == ENTRO_BF16 ? reinterpret_cast<const void *>(product_wide_kernel<OUT_BF16T>)
                                    : reinterpret_cast<const void *>(product_wide_kernel<OUT_F16T>);
    }
    r = allow_smem(fn, dev);
    if (r != ENTRO_OK) return r;
    CUtensorMap w_map, x_map;
    const uint64_t w_dims[2] = {static_cast<uint64_t>(cols), static_cast<uint64_t>(rows)}, w_strides[1] = {static_cast<uint64_t>(ldw)};
    const uint64_t x_dims[2] = {static_cast<uint64_t>(cols), static_cast<uint64_t>(tokens)}, x_strides[1] = {static_cast<uint64_t>(ldq)};
    const uint32_t w_box[2] = {kChunkBytes, kTileRows}, x_box[2] = {kChunkBytes, static_cast<uint32_t>(narrow ? a.bn : a.bn / 2)};
    r = encode_map(&w_map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, d_w, w_dims, w_strides, w_box);
    if (r == ENTRO_OK) r = encode_map(&x_map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, d_q, x_dims, x_strides, x_box);
    if (r != ENTRO_OK) return r;
    void *args[] = {&w_map, &x_map, &a};
    const bool early = static_cast<int64_t>(grid.x) * grid.y <= di.sms;
    e = launch_ex(fn, grid, threads, smem, static_cast<cudaStream_t>(stream), cluster, early, args);
    return e == cudaSuccess ? ENTRO_OK : cuda_fail(e, "entro_matmul_i8");
}

extern "C" int entro_test_product_plan(int64_t tokens, int64_t rows, int64_t cols, int32_t sms, entro_product_plan *plan) {
    if (!plan || tokens < 1 || rows < 1 || cols < 1 || sms < 2) return ENTRO_E_INVAL;
    if (tokens > ENTRO_PRODUCT_MAX_TOKENS || cols > ENTRO_PRODUCT_MAX_COLS || rows > (INT64_C(1) << 30)) return ENTRO_E_LIMIT;
    *plan = plan_product(tokens, rows, static_cast<int>((cols + kChunkBytes - 1) / kChunkBytes), sms);
    return ENTRO_OK;
}
