// kvcache.cu -- a paged key/value cache in 8 bits with a scale for each block of
// tokens and head: its writer, its reader, and the attention of single tokens
// over it.
//
// A page holds P tokens of all key heads, [head][token][channel], and is the
// block that shares a scale.  A block is coded once it is full: with a the
// largest magnitude of the block and head, scale = a / 127 and codes =
// rint(127 x / a).  The tokens of a sequence's last, open block stay in 16 bits
// in the sequence's tail slot.  So codes are never coded again, and what a cache
// holds does not depend on how its tokens arrived.
#include <algorithm>
#include <cstring>
#include <type_traits>

#include "launch.h"
#include "sm100.cuh"

namespace entro {
using namespace sm100;

struct Cache {
    int8_t *codes[2];  // keys, values: [pages][kv][P][D]
    float *scale[2];   // [pages][kv]
    void *tail[2];     // [slots][kv][P][D], 16-bit
    int64_t pages, slots;
    int kv, log_page;
};

// ------------------------------------------------------------------ append

struct AppendArgs {
    Cache c;
    const void *in[2];  // [tokens][kv][D]
    int64_t in_token[2], in_head[2];  // strides, elements
    const int32_t *cu;     // [batch + 1]: a sequence's new tokens among the packed ones
    const int32_t *table;  // [batch][table_width]
    const int32_t *lens;   // [batch]: tokens with the new ones
    const int32_t *slot_of;
    int32_t *status;
    int64_t tokens, table_stride;
    int batch, table_width;
    int heads;  // key heads that a CTA takes, one after the other
};

constexpr int kAppendThreads = 128;

// The sequence's new tokens [begin, begin + n) and its first new position; n = 0
// for what the arguments do not allow (reported once).
__device__ __forceinline__ int new_tokens(const AppendArgs &a, int b, int &begin, int &start) {
    begin = a.cu[b], start = 0;
    const int end = a.cu[b + 1], len = a.lens[b];
    const int slot = a.slot_of ? a.slot_of[b] : b;
    // (compared before they are subtracted: differences of these numbers may pass 32 bits)
    const bool ok = begin >= 0 && begin <= end && end <= a.tokens && len >= 0 && end - begin <= len && slot >= 0 && slot < a.c.slots;
    const int n = ok ? end - begin : 0;
    if (!ok || (n > 0 && len >> a.c.log_page > a.table_width)) {
        set_status(a.status, ENTRO_E_INVAL);
        return 0;
    }
    start = len - n;
    return n;
}

// Work item -> (sequence, block): an item for each block that gets new tokens.
__device__ __forceinline__ bool find_block(const AppendArgs &a, int64_t item, int &b, int &block, int &begin, int &n, int &start) {
    __shared__ int warp_sum[kAppendThreads / 32];
    __shared__ int found[5];
    const int tid = threadIdx.x, lane = tid % 32;
    int64_t before = 0;
    for (int b0 = 0; b0 < a.batch; b0 += kAppendThreads) {
        const int mine = b0 + tid;
        int bg = 0, st = 0, nn = 0, blocks = 0;
        if (mine < a.batch) {
            nn = new_tokens(a, mine, bg, st);
            if (nn > 0) blocks = ((st + nn - 1) >> a.c.log_page) - (st >> a.c.log_page) + 1;
        }
        int sum = blocks;
        for (int o = 1; o < 32; o *= 2) {
            const int up = __shfl_up_sync(~0u, sum, o);
            if (lane >= o) sum += up;
        }
        if (tid == 0) found[0] = -1;
        if (lane == 31) warp_sum[tid / 32] = sum;
        __syncthreads();
        int64_t at = before + sum;
        for (int w = 0; w < tid / 32; w++) at += warp_sum[w];
        if (item < at && item >= at - blocks) {
            found[0] = mine;
            found[1] = (st >> a.c.log_page) + static_cast<int>(item - (at - blocks));
            found[2] = bg;
            found[3] = nn;
            found[4] = st;
        }
        __syncthreads();
        if (found[0] >= 0) {
            b = found[0], block = found[1], begin = found[2], n = found[3], start = found[4];
            return true;
        }
        for (int w = 0; w < kAppendThreads / 32; w++) before += warp_sum[w];
        __syncthreads();
    }
    return false;
}

// One CTA a (block, some heads, keys or values): finding the block costs as much as coding a small one, so
// long calls take four heads a CTA.  Bound by memory: 2 bytes of each new element in, 1 (or 2, in the tail) out; 36000
// tokens of 8 x 128 in 37 us, 5.9 TB/s.
template <typename T, int D, int P>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const AppendArgs a) {
    constexpr int kVecs = P * D / 8, kMine = (kVecs + kAppendThreads - 1) / kAppendThreads, kRow = D / 8;
    __shared__ uint32_t red[kAppendThreads / 32];
    int b, block, begin, n, start;
    if (!find_block(a, blockIdx.x, b, block, begin, n, start)) return;
    const int tid = threadIdx.x, kind = blockIdx.z, end = start + n;
    const int slot = a.slot_of ? a.slot_of[b] : b;
    const int first = start / P, last_open = end % P ? end / P : -1;  // the block that stays open, if any
    // When the first block's older tokens are in the tail, its CTA writes the open block's
    // tokens over them after it has read them; otherwise the open block's own CTA does.
    const bool older = start % P != 0;
    if (block == last_open && block != first && older) return;
    const int page = block != last_open ? a.table[b * a.table_stride + block] : 0;
    const bool ok = page >= 0 && page < a.c.pages;
    if (!ok) set_status(a.status, ENTRO_E_INVAL);
    for (int h = blockIdx.y * a.heads; h < min((blockIdx.y + 1) * a.heads, static_cast<unsigned>(a.c.kv)); h++) {
        T *tail = static_cast<T *>(a.c.tail[kind]) + (static_cast<int64_t>(slot) * a.c.kv + h) * (P * D);
        const T *in = static_cast<const T *>(a.in[kind]) + begin * a.in_token[kind] + h * a.in_head[kind];
        if (block != last_open) {
            uint4 v[kMine];
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < kMine; i++) {
                const int u = i * kAppendThreads + tid;
                if (kVecs % kAppendThreads && u >= kVecs) break;
                const int t = u / kRow, x = u % kRow * 8, pos = block * P + t;
                v[i] = *reinterpret_cast<const uint4 *>(pos < start ? tail + t * D + x : in + (pos - start) * a.in_token[kind] + x);
                m = __vmaxu2(m, __vmaxu2(__vmaxu2(v[i].x & 0x7FFF7FFFu, v[i].y & 0x7FFF7FFFu),
                                         __vmaxu2(v[i].z & 0x7FFF7FFFu, v[i].w & 0x7FFF7FFFu)));
            }
            m = __reduce_max_sync(~0u, max(m & 0xFFFF, m >> 16));
            if (tid % 32 == 0) red[tid / 32] = m;
            __syncthreads();
#pragma unroll
            for (int w = 0; w < kAppendThreads / 32; w++) m = max(m, red[w]);
            const BlockCode<T> code(m);
            int8_t *out = a.c.codes[kind] + (static_cast<int64_t>(ok ? page : 0) * a.c.kv + h) * (P * D);
            if (ok) {
#pragma unroll
                for (int i = 0; i < kMine; i++) {
                    const int u = i * kAppendThreads + tid;
                    if (kVecs % kAppendThreads && u >= kVecs) break;
                    *reinterpret_cast<uint2 *>(out + u * 8) = code.eight(v[i]);
                }
                if (tid == 0) a.c.scale[kind][static_cast<int64_t>(page) * a.c.kv + h] = code.scale();
            }
            __syncthreads();  // the older tokens have been read (and the maxima)
            if (block != first || !older || last_open < 0) continue;
        }
        // the open block's new tokens into the tail
        const int from = max(start, last_open * P);
        for (int u = tid; u < (end - from) * kRow; u += kAppendThreads) {
            const int pos = from + u / kRow, x = u % kRow * 8;
            *reinterpret_cast<uint4 *>(tail + pos % P * D + x) =
                __ldg(reinterpret_cast<const uint4 *>(in + (pos - start) * a.in_token[kind] + x));
        }
    }
}

// ------------------------------------------------------------------ read

struct ReadArgs {
    Cache c;
    void *out[2];  // [tokens][kv][D]
    int64_t out_token[2], out_head[2];
    const int32_t *cu;
    const int32_t *table;
    const int32_t *slot_of;
    int32_t *status;
    int64_t tokens, table_stride;
    int batch, table_width;
};

// Where a sequence's tokens lie among the packed ones; false for offsets that the call does not allow.  (Compared before
// they are subtracted: the difference of two 32-bit offsets may pass 32 bits.)
__device__ __forceinline__ bool packed_range(const ReadArgs &a, int b, int &begin, int &end) {
    begin = a.cu[b], end = a.cu[b + 1];
    return begin >= 0 && begin <= end && end <= a.tokens;
}

// One cached token back to 16 bits, by a warp: code times scale in 32 bits, rounded once.
template <typename T, int D>
__device__ __forceinline__ void read_token(const ReadArgs &a, int64_t t) {
    const int lane = threadIdx.x % 32, P = 1 << a.c.log_page;
    // the last sequence that begins at or before t
    int lo = 0, hi = a.batch;
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (a.cu[mid] <= t) lo = mid;
        else hi = mid;
    }
    const int b = lo;
    int begin, end;
    if (!packed_range(a, b, begin, end) || t < begin || t >= end) return;  // a token of no sequence: left as it is
    const int pos = static_cast<int>(t) - begin, block = pos >> a.c.log_page;
    const int slot = a.slot_of ? a.slot_of[b] : b;
    const bool open = block == (end - begin) >> a.c.log_page;
    const int page = !open && block < a.table_width ? a.table[b * a.table_stride + block] : -1;
    if (open ? slot < 0 || slot >= a.c.slots : page < 0 || page >= a.c.pages) {
        if (lane == 0) set_status(a.status, ENTRO_E_INVAL);
        return;
    }
    const int off = pos & (P - 1);
    if (open) {
        constexpr int kRow = D / 8;
        for (int u = lane; u < 2 * a.c.kv * kRow; u += 32) {
            const int x = u % kRow * 8, row = u / kRow, kind = row >= a.c.kv, h = row - kind * a.c.kv;
            const T *tail = static_cast<const T *>(a.c.tail[kind]) + ((static_cast<int64_t>(slot) * a.c.kv + h) * P + off) * D + x;
            *reinterpret_cast<uint4 *>(static_cast<T *>(a.out[kind]) + t * a.out_token[kind] + h * a.out_head[kind] + x) =
                __ldg(reinterpret_cast<const uint4 *>(tail));
        }
        return;
    }
    constexpr int kRow = D / 16;
#pragma unroll 4
    for (int u = lane; u < 2 * a.c.kv * kRow; u += 32) {
        const int x = u % kRow * 16, row = u / kRow, kind = row >= a.c.kv, h = row - kind * a.c.kv;
        const int64_t at = static_cast<int64_t>(page) * a.c.kv + h;
        const float s = __ldg(a.c.scale[kind] + at);
        const uint4 c = __ldg(reinterpret_cast<const uint4 *>(a.c.codes[kind] + (at * P + off) * D + x));
        const uint32_t w[4] = {c.x ^ 0x80808080u, c.y ^ 0x80808080u, c.z ^ 0x80808080u, c.w ^ 0x80808080u};
        uint32_t o[8];
#pragma unroll
        for (int i = 0; i < 8; i++) {
            // 2^23 + (code + 128) has the code's byte as its low bits
            const uint32_t lo = __byte_perm(w[i / 2], 0x4B000000u, 0x7540 + i % 2 * 2), hi = __byte_perm(w[i / 2], 0x4B000000u, 0x7541 + i % 2 * 2);
            const float2 v = halves(mul2(add2(pair(lo, hi), pair(-8388736.0f, -8388736.0f)), pair(s, s)));
            o[i] = Half<T>::pack(v.x, v.y);
        }
        uint4 *out = reinterpret_cast<uint4 *>(static_cast<T *>(a.out[kind]) + t * a.out_token[kind] + h * a.out_head[kind] + x);
        out[0] = make_uint4(o[0], o[1], o[2], o[3]);
        out[1] = make_uint4(o[4], o[5], o[6], o[7]);
    }
}

// Bound by memory: 36000 tokens of 8 x 128 in 46 us, 4.8 TB/s.
template <typename T, int D>
__global__ void __launch_bounds__(256) read_kernel(const ReadArgs a) {
    const int64_t t = blockIdx.x * 8LL + threadIdx.x / 32;
    if (t < a.tokens) read_token<T, D>(a, t);
    // offsets are reported whether a token finds them or not (last: the tokens do not wait for it)
    int begin, end;
    for (int64_t b = blockIdx.x * 256LL + threadIdx.x; b < a.batch; b += gridDim.x * 256LL)
        if (!packed_range(a, static_cast<int>(b), begin, end)) set_status(a.status, ENTRO_E_INVAL);
}

// ------------------------------------------------------------------ attention of single tokens

struct AttendArgs {
    Cache c;
    const void *q;  // [batch][heads][D]
    void *out;      // [batch][heads][D]
    int64_t q_token, q_head, out_token, out_head, table_stride;
    const int32_t *table;
    const int32_t *lens;
    const int32_t *slot_of;
    float *work;
    int32_t *status;
    int batch, group, chunks;  // query heads of a key head; groups of 8 of them
    int table_width, ctas;
    bool join_early;  // the join may begin, and find its place, while the pieces are computed
    float scale_log2;
};

constexpr int kAttendThreads = 128;
constexpr int kTile = 64;         // tokens a CTA takes at a time, 16 a warp
constexpr int kHeads = 8;         // query heads of an MMA
constexpr float kLazy = 8.0f;     // the reference maximum is raised when a score passes it by 2^8
// Weights are held as 2^6 times theirs, at most 2^14, in fp16: off by 2^-11 of themselves, or by 2^-31 where that is more.
// (Their products with the codes are exact in fp16 alone: a bfloat16 weight would be off by 2^-8.)
constexpr float kBias = 6.0f;

// The cached length, cut to the table's pages and an open block (both kernels agree on it).
__device__ __forceinline__ int clean_len(const AttendArgs &a, int b, bool report) {
    const int len = a.lens[b];
    const int64_t most = min(((static_cast<int64_t>(a.table_width) + 1) << a.c.log_page) - 1, static_cast<int64_t>(INT32_MAX) - kTile);
    if (len >= 0 && len <= most) return len;
    if (report) set_status(a.status, ENTRO_E_INVAL);
    return len < 0 ? 0 : static_cast<int>(most);
}

// All (sequence, head, tile)s in a row (less than 2^31) are cut into equal shares for the CTAs.
struct Shares {
    uint32_t each, more;  // the first `more` CTAs take one more than `each`
    __device__ __forceinline__ Shares(uint32_t total, uint32_t ctas) : each(total / ctas), more(total % ctas) {}
    __device__ __forceinline__ uint32_t begin(uint32_t cta) const { return cta * each + min(cta, more); }
    __device__ __forceinline__ int owner(uint32_t tile) const {
        return tile < more * (each + 1) ? tile / (each + 1) : more + (tile - more * (each + 1)) / each;
    }
};

// All tiles of one head over the batch, and the sequence that `pick` chooses with the tiles before it: pick(b, tiles
// before b, tiles of b, all tiles) is true for one sequence at most.  A batch of up to a CTA's threads is read once.
template <typename Pick>
__device__ __forceinline__ uint32_t scan_batch(const AttendArgs &a, int &seq, uint32_t &before, Pick pick) {
    __shared__ uint32_t warp_sum[kAttendThreads / 32], picked_before;
    __shared__ int picked;
    const int tid = threadIdx.x, lane = tid % 32;
    uint32_t total = 0, at = 0, tiles = 0;
    if (tid == 0) picked = -1;
    auto chunk = [&](int b) {  // at: tiles before sequence b; total: those of all chunks so far
        tiles = b < a.batch ? (static_cast<uint32_t>(clean_len(a, b, false)) + kTile - 1) / kTile : 0;
        uint32_t sum = tiles;
        for (int o = 1; o < 32; o *= 2) {
            const uint32_t up = __shfl_up_sync(~0u, sum, o);
            if (lane >= o) sum += up;
        }
        if (lane == 31) warp_sum[tid / 32] = sum;
        __syncthreads();
        at = total + sum - tiles;
        for (int w = 0; w < kAttendThreads / 32; w++) {
            if (w < tid / 32) at += warp_sum[w];
            total += warp_sum[w];
        }
        __syncthreads();
    };
    for (int b0 = 0; b0 < a.batch; b0 += kAttendThreads) chunk(b0 + tid);
    const uint32_t all = total;
    auto offer = [&](int b) {
        if (b < a.batch && pick(b, at, tiles, all)) {
            picked = b;
            picked_before = at;
        }
    };
    if (a.batch <= kAttendThreads) {
        offer(tid);
    } else {
        total = 0;
        for (int b0 = 0; b0 < a.batch; b0 += kAttendThreads) {
            chunk(b0 + tid);
            offer(b0 + tid);
        }
    }
    __syncthreads();
    seq = picked;
    before = picked_before;
    return all;
}

// Four codes to two pairs of 16-bit floats, exactly: 1024 + (code + 128) has the
// code's byte as its low bits.
__device__ __forceinline__ uint32_t sub2(uint32_t h) {
    uint32_t r;
    asm("sub.f16x2 %0, %1, %2;" : "=r"(r) : "r"(h), "r"(0x64806480u));
    return r;
}
__device__ __forceinline__ void mma16816(float *c, const uint32_t *a, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma16816_bf16(float *c, const uint32_t *a, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Asynchronous copies to shared memory, in groups a thread.
__device__ __forceinline__ void copy_async16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_async4(uint32_t dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void close_group() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void wait_groups() {  // all but the last N groups have landed
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A step's 16 tokens of codes in shared memory: rows of D bytes, their 16-byte pieces moved so that the eight lanes of
// a phase meet eight different ones -- keys: lanes read strips of D / 4 bytes of rows gid; values: strips of D / 8
// bytes of rows 2 tig.  (96: no move needed for the keys, two lanes a bank for the values.)
template <int D>
struct StepLayout {
    static constexpr int kCodes = 16 * D, kBytes = 2 * kCodes + 16;  // keys, values, their two scales
    static __device__ __forceinline__ uint32_t key(int row, int byte) {
        return D == 128 ? row * 128 + (byte ^ ((row & 1) * 16)) : row * D + byte;
    }
    static __device__ __forceinline__ uint32_t value(int row, int byte) {
        if (D == 96) return row * D + byte;
        return (row * D + byte) ^ ((row / 2 & 3) * 32);  // (rows 2 tig: a line of 128 bytes each, or two)
    }
};
template <int N>
__device__ __forceinline__ void load_shared(uint32_t *r, uint32_t at) {
    if (N == 16) asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at));
    else if (N == 8) asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(at));
    else asm volatile("ld.shared.u32 %0, [%1];" : "=r"(r[0]) : "r"(at));
}

// N bytes (16, 24, 32, 48 or 64) from an address aligned to the largest power of two in N, up to 16
template <int N>
__device__ __forceinline__ void load_bytes(uint32_t *r, const void *p) {
    static_assert(N % 8 == 0, "");
    if (N % 16 == 0) {
#pragma unroll
        for (int i = 0; i < N / 16; i++) {
            const uint4 v = __ldg(static_cast<const uint4 *>(p) + i);
            r[4 * i] = v.x, r[4 * i + 1] = v.y, r[4 * i + 2] = v.z, r[4 * i + 3] = v.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < N / 8; i++) {
            const uint2 v = __ldg(static_cast<const uint2 *>(p) + i);
            r[2 * i] = v.x, r[2 * i + 1] = v.y;
        }
    }
}
// A power of two that brings numbers of at most this magnitude (the bits of a
// 16-bit float without its sign) near 2^14, and its inverse.  A bfloat16 then fits
// fp16 exactly if its exponent is at most 31 below the largest: `exact_from` has the
// bits of the smallest that does.
template <typename T>
__device__ __forceinline__ float fit_factor(uint32_t top, float &inverse, int &exact_from) {
    exact_from = 0;
    if (Half<T>::kExp == 0x7C007C00u) {  // fp16 already
        inverse = 1.0f;
        return 1.0f;
    }
    const int e = min(max(static_cast<int>(top >> 7), 28), 254);  // biased exponent
    exact_from = (e - 31) * 128;
    inverse = __uint_as_float(static_cast<uint32_t>(e - 14) << 23);
    return __uint_as_float(static_cast<uint32_t>(254 + 14 - e) << 23);
}
template <typename T>
__device__ __forceinline__ uint32_t to_f16x2(uint32_t v, float factor) {
    if (Half<T>::kExp == 0x7C007C00u) return v;
    const float2 f = Half<T>::widen(v);
    return Half<__half>::pack(f.x * factor, f.y * factor);
}

// Scores of a step of coded tokens by products in 32 bits, of code times scale as they stand: for queries whose channels
// lie too far apart for one factor.  As in the MMA, this thread's are tokens gid and gid + 8 of heads 2 tig and 2 tig + 1
// (q0, q1); `from` holds the step's keys, in StepLayout.
template <typename T, int D>
__device__ __forceinline__ void wide_scores(float *s, uint32_t from, float scale, const T *q0, const T *q1) {
    const int gid = threadIdx.x % 32 / 4;
    s[0] = s[1] = s[2] = s[3] = 0.0f;
#pragma unroll 1
    for (int d = 0; d < D; d += 4) {
        uint32_t k[2];
        load_shared<4>(k, from + StepLayout<D>::key(gid, d));
        load_shared<4>(k + 1, from + StepLayout<D>::key(gid + 8, d));
        const uint2 x = __ldg(reinterpret_cast<const uint2 *>(q0 + d)), y = __ldg(reinterpret_cast<const uint2 *>(q1 + d));
        const float2 xs[2] = {Half<T>::widen(x.x), Half<T>::widen(x.y)}, ys[2] = {Half<T>::widen(y.x), Half<T>::widen(y.y)};
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const float a = i % 2 ? xs[i / 2].y : xs[i / 2].x, b = i % 2 ? ys[i / 2].y : ys[i / 2].x;
            const float lo = static_cast<float>(static_cast<int8_t>(k[0] >> (8 * i))) * scale;
            const float hi = static_cast<float>(static_cast<int8_t>(k[1] >> (8 * i))) * scale;
            s[0] = fmaf(a, lo, s[0]), s[1] = fmaf(b, lo, s[1]), s[2] = fmaf(a, hi, s[2]), s[3] = fmaf(b, hi, s[3]);
        }
    }
}

// A warp's running softmax over the tokens it has seen, for 8 query heads: this
// thread holds heads 2 tig and 2 tig + 1 (tig = lane % 4) of 1/8 of the channels.
// Scores and outputs are transposed products, K Q^T and V^T P^T, so that the
// codes are the 16-row operand: the rows of a thread's fragments are tokens
// (scores) or channels (outputs), and neither the order of the tokens nor that of
// the channels inside an MMA matters, so a thread reads whole strips of its rows.
template <int D>
struct Running {
    float m[2], l[2];
    float o[D / 16][4];

    __device__ __forceinline__ void clear() {
        m[0] = m[1] = -INFINITY;
        l[0] = l[1] = 0.0f;
#pragma unroll
        for (int i = 0; i < D / 16; i++) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;
    }

    // s: scores in units of log2 (tokens gid and gid + 8 of heads 2 tig, 2 tig + 1), -inf
    // where there is no token; on return their weights.
    __device__ __forceinline__ void weights(float *s) {
        const float t0 = m[0] + kLazy, t1 = m[1] + kLazy;
        if (__any_sync(~0u, s[0] > t0 || s[2] > t0 || s[1] > t1 || s[3] > t1)) {
            float n0 = fmaxf(s[0], s[2]), n1 = fmaxf(s[1], s[3]);
#pragma unroll
            for (int x = 4; x < 32; x *= 2) {
                n0 = fmaxf(n0, __shfl_xor_sync(~0u, n0, x));
                n1 = fmaxf(n1, __shfl_xor_sync(~0u, n1, x));
            }
            n0 = fmaxf(n0, m[0]), n1 = fmaxf(n1, m[1]);
            const float f0 = m[0] == n0 ? 1.0f : ex2(m[0] - n0), f1 = m[1] == n1 ? 1.0f : ex2(m[1] - n1);
            m[0] = n0, m[1] = n1;
            l[0] *= f0, l[1] *= f1;
#pragma unroll
            for (int i = 0; i < D / 16; i++) {
                o[i][0] *= f0, o[i][2] *= f0;
                o[i][1] *= f1, o[i][3] *= f1;
            }
        }
        // no score so far: any reference does
        const float r0 = (m[0] == -INFINITY ? 0.0f : m[0]) - kBias, r1 = (m[1] == -INFINITY ? 0.0f : m[1]) - kBias;
        s[0] = ex2(s[0] - r0), s[1] = ex2(s[1] - r1), s[2] = ex2(s[2] - r0), s[3] = ex2(s[3] - r1);
        l[0] += s[0] + s[2];
        l[1] += s[1] + s[3];
    }
};

// What sums of weights make of an output: 1 / l; nothing where there were no tokens; NaN where there were, but all scored
// -infinity (their sum is marked by a negative number, which counts nothing beside other sums).
__device__ __forceinline__ float by_sum(float l) { return l == 0.0f ? 0.0f : l < 0.0f ? __int_as_float(0x7FC00000) : 1.0f / l; }

// Weights as the P^T operand in fp16 (2^-11 of a weight at most).
struct Weights16 {
    uint32_t p0, p1;
    __device__ __forceinline__ explicit Weights16(const float *e)
        : p0(transpose8x8(Half<__half>::pack(e[0], e[1]))), p1(transpose8x8(Half<__half>::pack(e[2], e[3]))) {}
};

// A warp's steps in flight, the one at work among them.  Two with 16 warps on an SM keep memory as busy as it gets
// (48 sequences of 8192 to 32768 tokens, 8 key heads of 128: 391 us; three 425, four 474, in turns).
constexpr int kSteps = 2;

template <int D>
constexpr int attend_smem() {
    const int steps = 4 * kSteps * StepLayout<D>::kBytes, join = 4 * kHeads * (D + 4) * 4;
    return steps > join ? steps : join;
}

// One pass over the cache.  A CTA's share of all tiles is one row of tiles, cut
// where the (sequence, head) changes; a piece that covers all of its sequence and
// head is finished here, others leave (m, l, o) behind for the join.  Bound by
// reading the codes, 2 D bytes of a token and key head: 48 sequences of 8192 to 32768
// tokens, 8 key heads of 128: 391 to 422 us from run to run, 5.0 to 5.4 TB/s; of 625 to 2500 with 32 key heads of 96, where pieces are short: 97 us, 4.5
// TB/s; one of 1000 tokens: 8.2 us with the join, in a graph.
template <typename T, int D>
__global__ void __launch_bounds__(kAttendThreads, 4) attend_kernel(const AttendArgs a) {
    using Layout = StepLayout<D>;
    constexpr bool kBf16 = Half<T>::kExp != 0x7C007C00u;
    constexpr int kK = D / 4, kV = D / 8;  // bytes of a token's codes that a thread reads: keys (2 tokens), values (4)
    constexpr int kKLoad = kK % 16 == 0 ? 16 : 8, kVLoad = kV % 16 == 0 ? 16 : kV % 8 == 0 ? 8 : 4;
    extern __shared__ __align__(16) uint8_t smem[];  // the warps' steps, then their outputs
    __shared__ float sm_m[4][kHeads], sm_l[4][kHeads];
    float(*sm_o)[kHeads][D + 4] = reinterpret_cast<float(*)[kHeads][D + 4]>(smem);
    if (a.join_early) dependents_may_launch();
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, gid = lane / 4, tig = lane % 4;
    const uint32_t steps = smem_u32(smem) + warp * kSteps * Layout::kBytes;
    const int P = 1 << a.c.log_page, cols = a.c.kv * a.chunks;
    int seq;
    uint32_t before;
    const uint32_t total = scan_batch(a, seq, before, [&](int, uint32_t at, uint32_t tiles, uint32_t all) {
        const uint32_t first = Shares(all * cols, a.ctas).begin(blockIdx.x);
        return first >= at * cols && first < (at + tiles) * cols;
    }) * cols;
    const Shares shares(total, a.ctas);
    uint32_t at = shares.begin(blockIdx.x);
    const uint32_t stop = shares.begin(blockIdx.x + 1);
    if (at >= stop) return;
    uint32_t seq_at = before * cols;
    while (at < stop) {
        // the piece: tiles [t0, t1) of column (key head, chunk of query heads) of the sequence
        int len = clean_len(a, seq, true), tiles = (len + kTile - 1) / kTile;
        while (at >= seq_at + static_cast<uint32_t>(tiles * cols)) {  // (sequences without tokens have no tiles)
            seq_at += tiles * cols;
            seq++;
            len = clean_len(a, seq, true);
            tiles = (len + kTile - 1) / kTile;
        }
        const int col = (at - seq_at) / static_cast<uint32_t>(tiles), t0 = (at - seq_at) % static_cast<uint32_t>(tiles);
        const int t1 = min(static_cast<uint32_t>(tiles), t0 + (stop - at));
        const int h = col / a.chunks, head0 = h * a.group + col % a.chunks * kHeads;
        const int heads = min(kHeads, a.group - col % a.chunks * kHeads);
        const int full = len >> a.c.log_page << a.c.log_page;  // tokens in coded blocks
        const int32_t *pages = a.table + seq * a.table_stride;

        // Steps of 16 tokens, kSteps - 1 of them on their way; this warp's tiles up to `coded_end` are of coded blocks.  A
        // step on a page that does not exist copies nothing; bit x of `coded` says of the step in place x whether it did,
        // and its bit 31 whether this warp has had any token.
        const int coded_end = min(t1, (full - warp * 16 + kTile - 1) / kTile);
        uint32_t coded = 0;
        int place = 0;  // of the next step to be sent
        auto page_of = [&](int tile) { return tile < coded_end ? __ldg(pages + ((tile * kTile + warp * 16) >> a.c.log_page)) : -1; };
        int page = page_of(t0);
        auto send = [&](int tile) {
            const int tok = tile * kTile + warp * 16, p = page;
            page = page_of(tile + 1);
            coded &= ~(1u << place);
            if (tile < coded_end) {
                if (p >= 0 && p < a.c.pages) {
                    const int64_t block = static_cast<int64_t>(p) * a.c.kv + h, from = (block * P + (tok & (P - 1))) * D;
                    const uint32_t to = steps + place * Layout::kBytes;
#pragma unroll
                    for (int i = 0; i < D / 32; i++) {
                        const int piece = i * 32 + lane, row = piece / (D / 16), byte = piece % (D / 16) * 16;
                        copy_async16(to + Layout::key(row, byte), a.c.codes[0] + from + piece * 16);
                        copy_async16(to + Layout::kCodes + Layout::value(row, byte), a.c.codes[1] + from + piece * 16);
                    }
                    if (lane < 2) copy_async4(to + 2 * Layout::kCodes + lane * 4, a.c.scale[lane] + block);
                    coded |= 1u << place | 1u << 31;
                } else {
                    set_status(a.status, ENTRO_E_INVAL);
                }
            }
            close_group();
            place = place + 1 == kSteps ? 0 : place + 1;
        };
        for (int i = 0; i < kSteps - 1; i++) send(t0 + i);

        // Q as the second operand: head gid, channels tig D / 4 + 4 s + 0 .. 3 in step s
        uint32_t q[D / 16][2];
        float mine = 0.0f;
        bool wide = false;  // some query's channels lie too far apart for fp16 (the warp's)
        auto q_row = [&](int head) { return static_cast<const T *>(a.q) + seq * a.q_token + (head0 + min(head, heads - 1)) * a.q_head; };
        {
            uint32_t raw[D / 8], top = 0;
            load_bytes<D / 2>(raw, q_row(gid) + tig * kK);
#pragma unroll
            for (int i = 0; i < D / 8; i++) top = __vmaxu2(top, raw[i] & 0x7FFF7FFFu);
            top = max(top & 0xFFFF, top >> 16);
            top = max(top, __shfl_xor_sync(~0u, top, 1));
            top = max(top, __shfl_xor_sync(~0u, top, 2));
            int exact_from;
            const float f = fit_factor<T>(top, mine, exact_from);
            if (kBf16) {
                uint32_t low = ~0u;  // the smallest magnitude but 0, less one
#pragma unroll
                for (int i = 0; i < D / 8; i++) low = __vminu2(low, __vsub2(raw[i] & 0x7FFF7FFFu, 0x00010001u));
                wide = __any_sync(~0u, static_cast<int>(min(low & 0xFFFF, low >> 16)) + 1 < exact_from);
            }
#pragma unroll
            for (int i = 0; i < D / 8; i++) q[i / 2][i % 2] = gid < heads ? to_f16x2<T>(raw[i], f) : 0u;
            mine *= a.scale_log2;
        }
        const float qs[2] = {__shfl_sync(~0u, mine, tig * 8), __shfl_sync(~0u, mine, tig * 8 + 4)};

        Running<D> r;
        r.clear();
        // Steps of coded tokens: a thread's keys are tokens gid and gid + 8, its values tokens 2 tig, 2 tig + 1 and those + 8.
        int here = 0, tile = t0;
        auto coded_steps = [&](auto by_products) {
            for (; tile < coded_end; tile++) {
                send(tile + kSteps - 1);
                wait_groups<kSteps - 1>();
                __syncwarp();
                if (coded >> here & 1) {
                    const uint32_t from = steps + here * Layout::kBytes;
                    uint32_t kr[2][kK / 4], vr[4][kV / 4];
                    float ks, vs;
                    asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(ks), "=f"(vs) : "r"(from + 2 * Layout::kCodes));
#pragma unroll
                    for (int i = 0; i < kK; i += kKLoad) {
                        load_shared<kKLoad>(kr[0] + i / 4, from + Layout::key(gid, tig * kK + i));
                        load_shared<kKLoad>(kr[1] + i / 4, from + Layout::key(gid + 8, tig * kK + i));
                    }
#pragma unroll
                    for (int i = 0; i < kV; i += kVLoad)
#pragma unroll
                        for (int j = 0; j < 4; j++)
                            load_shared<kVLoad>(vr[j] + i / 4, from + Layout::kCodes + Layout::value(2 * tig + j / 2 * 8 + j % 2, gid * kV + i));
                    float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int s = 0; s < D / 16; s++) {
                        const uint32_t lo = kr[0][s] ^ 0x80808080u, hi = kr[1][s] ^ 0x80808080u;
                        const uint32_t f[4] = {sub2(__byte_perm(lo, 0x64646464u, 0x4140)), sub2(__byte_perm(hi, 0x64646464u, 0x4140)),
                                               sub2(__byte_perm(lo, 0x64646464u, 0x4342)), sub2(__byte_perm(hi, 0x64646464u, 0x4342))};
                        mma16816(c, f, q[s][0], q[s][1]);
                    }
                    const float f0 = qs[0] * ks, f1 = qs[1] * ks;
                    float s[4] = {c[0] * f0, c[1] * f1, c[2] * f0, c[3] * f1};
                    if (decltype(by_products)::value) {
                        wide_scores<T, D>(s, from, ks, q_row(2 * tig), q_row(2 * tig + 1));
#pragma unroll
                        for (int i = 0; i < 4; i++) s[i] *= a.scale_log2;
                    }
                    r.weights(s);
                    const Weights16 p(s);
#pragma unroll
                    for (int i = 0; i < D / 32; i++) {
                        // four channels of four tokens to the fragments of two MMAs
                        const uint32_t x0 = vr[0][i] ^ 0x80808080u, x1 = vr[1][i] ^ 0x80808080u;
                        const uint32_t x2 = vr[2][i] ^ 0x80808080u, x3 = vr[3][i] ^ 0x80808080u;
#pragma unroll
                        for (int u = 0; u < 2; u++) {
                            const uint32_t lo = __byte_perm(x0, x1, u ? 0x7362 : 0x5140), hi = __byte_perm(x2, x3, u ? 0x7362 : 0x5140);
                            const uint32_t f[4] = {sub2(__byte_perm(lo, 0x64646464u, 0x4140)), sub2(__byte_perm(lo, 0x64646464u, 0x4342)),
                                                   sub2(__byte_perm(hi, 0x64646464u, 0x4140)), sub2(__byte_perm(hi, 0x64646464u, 0x4342))};
                            float w[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                            mma16816(w, f, p.p0, p.p1);
                            float *o = r.o[2 * i + u];
                            o[0] += w[0] * vs, o[1] += w[1] * vs, o[2] += w[2] * vs, o[3] += w[3] * vs;
                        }
                    }
                }
                __syncwarp();  // the step's place is sent to again
                here = here + 1 == kSteps ? 0 : here + 1;
            }
        };
        if (kBf16 && wide) coded_steps(std::true_type());
        else coded_steps(std::false_type());

        for (; tile < t1; tile++) {
            const int tok = tile * kTile + warp * 16;
            if (tok >= len) break;
            const int slot = a.slot_of ? a.slot_of[seq] : seq;
            if (slot < 0 || slot >= a.c.slots) {
                set_status(a.status, ENTRO_E_INVAL);
            } else {
                coded |= 1u << 31;
                // Up to 16 tokens of the open block, in 16 bits: their products take them as they are, so that neither
                // a large number nor an infinity changes what the others count.
                const int64_t base = (static_cast<int64_t>(slot) * a.c.kv + h) * P + (tok & (P - 1));
                const T *kt = static_cast<const T *>(a.c.tail[0]) + base * D, *vt = static_cast<const T *>(a.c.tail[1]) + base * D;
                const int n = len - tok;  // tokens of the step that exist, if below 16
                float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                {
                    uint32_t x[2][D / 8], raw[D / 8];
#pragma unroll
                    for (int j = 0; j < 2; j++) {
                        if (gid + 8 * j < n) {
                            load_bytes<D / 2>(x[j], kt + (gid + 8 * j) * D + tig * kK);
                        } else {
#pragma unroll
                            for (int i = 0; i < D / 8; i++) x[j][i] = 0;
                        }
                    }
                    if (kBf16) load_bytes<D / 2>(raw, q_row(gid) + tig * kK);
#pragma unroll
                    for (int s = 0; s < D / 16; s++) {
                        const uint32_t f[4] = {x[0][2 * s], x[1][2 * s], x[0][2 * s + 1], x[1][2 * s + 1]};
                        if (kBf16) mma16816_bf16(c, f, gid < heads ? raw[2 * s] : 0u, gid < heads ? raw[2 * s + 1] : 0u);
                        else mma16816(c, f, q[s][0], q[s][1]);
                    }
                }
                float s[4];
#pragma unroll
                for (int i = 0; i < 4; i++) s[i] = gid + i / 2 * 8 < n ? c[i] * a.scale_log2 : -INFINITY;
                r.weights(s);
                // The weights: fp16, or a pair of bfloat16 whose sum is as near (2^-18).
                const Weights16 p(s);
                uint32_t hi[2], lo[2];
#pragma unroll
                for (int i = 0; i < 2; i++) {
                    const uint32_t x = Half<__nv_bfloat16>::pack(s[2 * i], s[2 * i + 1]);
                    const float2 f = Half<__nv_bfloat16>::widen(x);
                    hi[i] = transpose8x8(x);
                    lo[i] = transpose8x8(Half<__nv_bfloat16>::pack(s[2 * i] - f.x, s[2 * i + 1] - f.y));
                }
                uint32_t y[4][D / 16];
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    const int t = 2 * tig + j / 2 * 8 + j % 2;
                    if (t < n) {
                        load_bytes<D / 4>(y[j], vt + t * D + gid * kV);
                    } else {
#pragma unroll
                        for (int i = 0; i < D / 16; i++) y[j][i] = 0;
                    }
                }
#pragma unroll
                for (int i = 0; i < D / 16; i++) {
                    uint32_t f[4] = {__byte_perm(y[0][i], y[1][i], 0x5410), __byte_perm(y[0][i], y[1][i], 0x7632),
                                     __byte_perm(y[2][i], y[3][i], 0x5410), __byte_perm(y[2][i], y[3][i], 0x7632)};
                    if (kBf16) {
                        mma16816_bf16(r.o[i], f, hi[0], hi[1]);
                        // (infinities count once: the remainders may be 0 or below)
#pragma unroll
                        for (int j = 0; j < 4; j++) f[j] &= ~__vcmpeq2(f[j] & Half<T>::kExp, Half<T>::kExp);
                        mma16816_bf16(r.o[i], f, lo[0], lo[1]);
                    } else {
                        float w[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                        mma16816(w, f, p.p0, p.p1);
#pragma unroll
                        for (int j = 0; j < 4; j++) r.o[i][j] += w[j];
                    }
                }
            }
        }
        wait_groups<0>();

        // the four warps' parts meet in shared memory
        __syncthreads();
        if (coded >> 31) {
#pragma unroll
            for (int x = 0; x < 2; x++)
                if (r.m[x] == -INFINITY && r.l[x] == 0.0f) r.l[x] = -1.0f;
        }
#pragma unroll
        for (int x = 4; x < 32; x *= 2) {
            r.l[0] += __shfl_xor_sync(~0u, r.l[0], x);
            r.l[1] += __shfl_xor_sync(~0u, r.l[1], x);
        }
        if (gid == 0) {
            sm_m[warp][2 * tig] = r.m[0], sm_m[warp][2 * tig + 1] = r.m[1];
            sm_l[warp][2 * tig] = r.l[0], sm_l[warp][2 * tig + 1] = r.l[1];
        }
#pragma unroll
        for (int i = 0; i < D / 16; i++) {
            // rows gid and gid + 8 of tile i are channels gid D / 8 + 2 i and + 1
            const int d = gid * kV + 2 * i;
            *reinterpret_cast<float2 *>(&sm_o[warp][2 * tig][d]) = make_float2(r.o[i][0], r.o[i][2]);
            *reinterpret_cast<float2 *>(&sm_o[warp][2 * tig + 1][d]) = make_float2(r.o[i][1], r.o[i][3]);
        }
        __syncthreads();
        const bool whole = t0 == 0 && t1 == tiles;
        // a piece that does not begin its sequence and head goes to the CTA's first place, one that only does not end it to the second
        float *part = a.work + (static_cast<int64_t>(blockIdx.x) * 2 + (t0 == 0)) * (kHeads * (D + 2));
        for (int u = tid; u < heads * (D / 2); u += kAttendThreads) {
            const int head = u / (D / 2), d = u % (D / 2) * 2;
            float m = -INFINITY;
#pragma unroll
            for (int w = 0; w < 4; w++) m = fmaxf(m, sm_m[w][head]);
            float l = 0.0f, o0 = 0.0f, o1 = 0.0f;
#pragma unroll
            for (int w = 0; w < 4; w++) {
                const float f = sm_m[w][head] == m ? 1.0f : ex2(sm_m[w][head] - m);
                l += f * sm_l[w][head];
                o0 += f * sm_o[w][head][d];
                o1 += f * sm_o[w][head][d + 1];
            }
            if (whole) {
                const float by = by_sum(l);
                T *out = static_cast<T *>(a.out) + seq * a.out_token + (head0 + head) * a.out_head + d;
                *reinterpret_cast<uint32_t *>(out) = Half<T>::pack(o0 * by, o1 * by);
            } else {
                float *row = part + head * (D + 2);
                *reinterpret_cast<float2 *>(row + 2 + d) = make_float2(o0, o1);
                if (d == 0) *reinterpret_cast<float2 *>(row) = make_float2(m, l);
            }
        }
        __syncthreads();
        at += t1 - t0;
    }
}

// Joins the pieces of each sequence and query head: a CTA each, its two halves taking every other piece.  Sequences
// without tokens get zeros.
template <typename T, int D>
__global__ void __launch_bounds__(kAttendThreads) join_kernel(const AttendArgs a) {
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, heads = a.c.kv * a.group, cols = a.c.kv * a.chunks;
    const int seq = static_cast<int>(blockIdx.x) / heads, head = static_cast<int>(blockIdx.x) % heads;
    const int col = head / a.group * a.chunks + head % a.group / kHeads, in_chunk = head % a.group % kHeads;
    int got;
    uint32_t before;
    const uint32_t total = scan_batch(a, got, before, [&](int b, uint32_t, uint32_t, uint32_t) { return b == seq; }) * cols;
    const int tiles = (clean_len(a, seq, true) + kTile - 1) / kTile;
    const Shares shares(total, a.ctas);
    const uint32_t t0 = before * cols + col * tiles;
    int first = 0, last = 0;
    if (tiles > 0) {
        first = shares.owner(t0);
        last = shares.owner(t0 + tiles - 1);
    }
    wait_for_prior_grid();  // (the lengths above are no work of the grid before)
    if (tiles > 0 && first == last) return;  // one CTA had it all
    // 64 pieces at a time: their maxima and sums first (a piece's weight is 2^(its maximum - the largest)), then their
    // outputs, with nothing between the loads
    constexpr int kPieces = 64;
    __shared__ float weight[2][kPieces];
    __shared__ float2 half_o[64];
    auto row_of = [&](int i) { return a.work + ((static_cast<int64_t>(i) * 2 + (i == first)) * kHeads + in_chunk) * (D + 2); };
    const int pieces = tiles > 0 ? last - first + 1 : 0, half = tid / 64, d = tid % 64 * 2;
    float most = -INFINITY, sum = 0.0f;
    float2 o = make_float2(0.0f, 0.0f);
    for (int i0 = 0, turn = 0; i0 < pieces; i0 += kPieces, turn ^= 1) {
        const int n = min(kPieces, pieces - i0);
        float2 ml[2];  // (every warp looks at all of them: no barrier between this and what follows)
#pragma unroll
        for (int x = 0; x < 2; x++)
            ml[x] = lane + 32 * x < n ? *reinterpret_cast<const float2 *>(row_of(first + i0 + lane + 32 * x)) : make_float2(-INFINITY, 0.0f);
        float m = fmaxf(ml[0].x, ml[1].x);
        for (int x = 16; x; x /= 2) m = fmaxf(m, __shfl_xor_sync(~0u, m, x));
        const float now = fmaxf(most, m), f = most == now ? 1.0f : ex2(most - now);
        float l = 0.0f;
#pragma unroll
        for (int x = 0; x < 2; x++) {
            const float w = ml[x].x == now ? 1.0f : ex2(ml[x].x - now);
            if (warp == 0) weight[turn][lane + 32 * x] = w;
            l += w * ml[x].y;
        }
        for (int x = 16; x; x /= 2) l += __shfl_xor_sync(~0u, l, x);
        sum = sum * f + l;
        most = now;
        __syncthreads();  // (two turns' weights: a warp may be one ahead)
        o.x *= f, o.y *= f;
        if (d < D) {
#pragma unroll 8
            for (int i = half; i < n; i += 2) {
                const float2 v = *reinterpret_cast<const float2 *>(row_of(first + i0 + i) + 2 + d);
                o.x += weight[turn][i] * v.x;
                o.y += weight[turn][i] * v.y;
            }
        }
    }
    if (half == 1) half_o[tid - 64] = o;
    __syncthreads();
    if (half == 0 && d < D) {
        const float by = by_sum(sum);
        T *out = static_cast<T *>(a.out) + seq * a.out_token + head * a.out_head + d;
        *reinterpret_cast<uint32_t *>(out) = Half<T>::pack((o.x + half_o[tid].x) * by, (o.y + half_o[tid].y) * by);
    }
}

// ------------------------------------------------------------------ host side

static int make_cache(const entro_kv_cache *c, Cache *o) {
    if (!c || c->pages < 1 || c->slots < 1 || c->kv_heads < 1 || c->kv_heads > 65535) return ENTRO_E_INVAL;
    if (c->type != ENTRO_BF16 && c->type != ENTRO_F16) return ENTRO_E_INVAL;
    if (c->head_dim != 64 && c->head_dim != 96 && c->head_dim != 128) return ENTRO_E_INVAL;
    if (c->page_tokens != 16 && c->page_tokens != 32 && c->page_tokens != 64 && c->page_tokens != 128) return ENTRO_E_INVAL;
    void *const p[6] = {c->k_codes, c->v_codes, c->k_scale, c->v_scale, c->k_tail, c->v_tail};
    for (void *q : p)
        if (!q || !aligned16(q)) return ENTRO_E_INVAL;
    o->codes[0] = static_cast<int8_t *>(c->k_codes), o->codes[1] = static_cast<int8_t *>(c->v_codes);
    o->scale[0] = static_cast<float *>(c->k_scale), o->scale[1] = static_cast<float *>(c->v_scale);
    o->tail[0] = c->k_tail, o->tail[1] = c->v_tail;
    o->pages = c->pages, o->slots = c->slots, o->kv = c->kv_heads;
    o->log_page = c->page_tokens == 16 ? 4 : c->page_tokens == 32 ? 5 : c->page_tokens == 64 ? 6 : 7;
    return ENTRO_OK;
}

static bool vector_rows(const void *p, int64_t token, int64_t head) { return aligned16(p) && token % 8 == 0 && head % 8 == 0; }

template <typename T, int D>
static const void *pick_append(int log_page) {
    switch (log_page) {
        case 4: return reinterpret_cast<const void *>(append_kernel<T, D, 16>);
        case 5: return reinterpret_cast<const void *>(append_kernel<T, D, 32>);
        case 6: return reinterpret_cast<const void *>(append_kernel<T, D, 64>);
        default: return reinterpret_cast<const void *>(append_kernel<T, D, 128>);
    }
}

// f<T, D>() of the cache's type and width
#define ENTRO_BY_TYPE(c, f, ...)                                                                     \
    ((c)->type == ENTRO_BF16 ? (c)->head_dim == 64   ? f(__nv_bfloat16, 64, ##__VA_ARGS__)              \
                               : (c)->head_dim == 96 ? f(__nv_bfloat16, 96, ##__VA_ARGS__)            \
                                                     : f(__nv_bfloat16, 128, ##__VA_ARGS__)           \
                             : (c)->head_dim == 64   ? f(__half, 64, ##__VA_ARGS__)                     \
                               : (c)->head_dim == 96 ? f(__half, 96, ##__VA_ARGS__)                   \
                                                     : f(__half, 128, ##__VA_ARGS__))
#define ENTRO_APPEND(T, D, log_page) pick_append<T, D>(log_page)
#define ENTRO_READ(T, D) reinterpret_cast<const void *>(read_kernel<T, D>)
#define ENTRO_ATTEND(T, D) reinterpret_cast<const void *>(attend_kernel<T, D>)
#define ENTRO_JOIN(T, D) reinterpret_cast<const void *>(join_kernel<T, D>)

// CTAs of an attention over the cache: four on each SM.
static int attend_ctas(int *ctas) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
    DeviceInfo di;
    const int r = device_info(dev, &di);
    if (r == ENTRO_OK) *ctas = 4 * di.sms;
    return r;
}

}  // namespace entro

using namespace entro;

extern "C" int entro_kv_append(const entro_kv_cache *cache, const void *d_k, int64_t k_token, int64_t k_head, const void *d_v,
                               int64_t v_token, int64_t v_head, int64_t tokens, const int32_t *d_cu, const int32_t *d_table,
                               int64_t table_stride, int32_t table_width, const int32_t *d_lens, const int32_t *d_slots,
                               int32_t batch, int32_t *d_status, void *stream) {
    AppendArgs a;
    std::memset(&a, 0, sizeof(a));
    const int r = make_cache(cache, &a.c);
    if (r != ENTRO_OK) return r;
    if (tokens < 0 || tokens > INT32_MAX || batch < 0 || table_width < 0 || table_stride < table_width) return ENTRO_E_INVAL;
    if (tokens == 0 || batch == 0) return ENTRO_OK;
    if (!d_k || !d_v || !d_cu || (!d_table && table_width > 0) || !d_lens || !vector_rows(d_k, k_token, k_head) || !vector_rows(d_v, v_token, v_head)) return ENTRO_E_INVAL;
    if (!d_slots && batch > cache->slots) return ENTRO_E_INVAL;
    a.in[0] = d_k, a.in[1] = d_v;
    a.in_token[0] = k_token, a.in_token[1] = v_token, a.in_head[0] = k_head, a.in_head[1] = v_head;
    a.cu = d_cu, a.table = d_table, a.lens = d_lens, a.slot_of = d_slots, a.status = d_status;
    a.tokens = tokens, a.table_stride = table_stride, a.batch = batch, a.table_width = table_width;
    // blocks that get new tokens: each has one at least, and a sequence's n reach at most (n - 2) / P + 2
    const int P = 1 << a.c.log_page;
    const int64_t items = std::min<int64_t>(tokens, (tokens + static_cast<int64_t>(batch) * (P - 2)) / P + batch);
    a.heads = items * a.c.kv >= 8192 ? 4 : 1;
    const void *fn = ENTRO_BY_TYPE(cache, ENTRO_APPEND, a.c.log_page);
    void *args[] = {&a};
    const cudaError_t e = launch_ex(fn, dim3(static_cast<unsigned>(items), (a.c.kv + a.heads - 1) / a.heads, 2), kAppendThreads, 0,
                                    static_cast<cudaStream_t>(stream), 1, false, args);
    return e == cudaSuccess ? ENTRO_OK : cuda_fail(e, "entro_kv_append");
}

extern "C" int entro_kv_read(const entro_kv_cache *cache, void *d_k, int64_t k_token, int64_t k_head, void *d_v, int64_t v_token,
                             int64_t v_head, int64_t tokens, const int32_t *d_cu, const int32_t *d_table, int64_t table_stride,
                             int32_t table_width, const int32_t *d_slots, int32_t batch, int32_t *d_status, void *stream) {
    ReadArgs a;
    std::memset(&a, 0, sizeof(a));
    const int r = make_cache(cache, &a.c);
    if (r != ENTRO_OK) return r;
    if (tokens < 0 || tokens > INT32_MAX || batch < 0 || table_width < 0 || table_stride < table_width) return ENTRO_E_INVAL;
    if (tokens == 0 || batch == 0) return ENTRO_OK;
    if (!d_k || !d_v || !d_cu || (!d_table && table_width > 0) || !vector_rows(d_k, k_token, k_head) || !vector_rows(d_v, v_token, v_head)) return ENTRO_E_INVAL;
    if (!separate_rows(tokens, a.c.kv, cache->head_dim, k_token, k_head) || !separate_rows(tokens, a.c.kv, cache->head_dim, v_token, v_head))
        return ENTRO_E_INVAL;
    if (!d_slots && batch > cache->slots) return ENTRO_E_INVAL;
    a.out[0] = d_k, a.out[1] = d_v;
    a.out_token[0] = k_token, a.out_token[1] = v_token, a.out_head[0] = k_head, a.out_head[1] = v_head;
    a.cu = d_cu, a.table = d_table, a.slot_of = d_slots, a.status = d_status;
    a.tokens = tokens, a.table_stride = table_stride, a.batch = batch, a.table_width = table_width;
    void *args[] = {&a};
    const cudaError_t e = launch_ex(ENTRO_BY_TYPE(cache, ENTRO_READ), dim3(static_cast<unsigned>((tokens + 7) / 8)), 256, 0,
                                    static_cast<cudaStream_t>(stream), 1, false, args);
    return e == cudaSuccess ? ENTRO_OK : cuda_fail(e, "entro_kv_read");
}

extern "C" int entro_kv_attend_workspace(const entro_kv_cache *cache, uint64_t *bytes) {
    if (!cache || !bytes) return ENTRO_E_INVAL;
    int ctas = 0;
    const int r = attend_ctas(&ctas);
    if (r == ENTRO_OK) *bytes = static_cast<uint64_t>(ctas) * 2 * kHeads * (cache->head_dim + 2) * 4;
    return r;
}

extern "C" int entro_kv_attend(const entro_kv_cache *cache, const void *d_q, int64_t q_token, int64_t q_head, int32_t heads,
                               const int32_t *d_table, int64_t table_stride, int32_t table_width, const int32_t *d_lens,
                               const int32_t *d_slots, int32_t batch, float scale, void *d_out, int64_t out_token, int64_t out_head,
                               void *d_work, uint64_t work_bytes, int32_t *d_status, void *stream) {
    AttendArgs a;
    std::memset(&a, 0, sizeof(a));
    int r = make_cache(cache, &a.c);
    if (r != ENTRO_OK) return r;
    if (batch < 0 || heads < 1 || heads % a.c.kv || table_width < 0 || table_stride < table_width || !(scale > 0.0f) || scale > 2.0e38f)
        return ENTRO_E_INVAL;
    if (batch == 0) return ENTRO_OK;
    if (!d_q || !d_out || !d_lens || !d_work || (!d_table && table_width > 0) || !aligned16(d_work) || !vector_rows(d_q, q_token, q_head) ||
        !vector_rows(d_out, out_token, out_head) || !separate_rows(batch, heads, cache->head_dim, out_token, out_head))
        return ENTRO_E_INVAL;
    if (!d_slots && batch > cache->slots) return ENTRO_E_INVAL;
    r = attend_ctas(&a.ctas);
    if (r != ENTRO_OK) return r;
    if (work_bytes < static_cast<uint64_t>(a.ctas) * 2 * kHeads * (cache->head_dim + 2) * 4) return ENTRO_E_INVAL;
    a.q = d_q, a.out = d_out;
    a.q_token = q_token, a.q_head = q_head, a.out_token = out_token, a.out_head = out_head;
    a.table = d_table, a.table_stride = table_stride, a.table_width = table_width;
    a.lens = d_lens, a.slot_of = d_slots, a.work = static_cast<float *>(d_work), a.status = d_status;
    a.batch = batch, a.group = heads / a.c.kv, a.chunks = (a.group + kHeads - 1) / kHeads;
    a.scale_log2 = scale * 1.4426950408889634f;
    const int64_t columns = static_cast<int64_t>(batch) * a.c.kv * a.chunks;
    // all tiles are counted in 32 bits
    if (columns * (((static_cast<int64_t>(table_width) + 1) << a.c.log_page) / kTile + 1) > INT32_MAX) return ENTRO_E_LIMIT;
    const int64_t joins = static_cast<int64_t>(batch) * heads;
    if (joins > INT32_MAX) return ENTRO_E_LIMIT;
    a.join_early = joins <= a.ctas / 4;  // a CTA on each SM at most, beside the four that are there
    const size_t smem = cache->head_dim == 64 ? attend_smem<64>() : cache->head_dim == 96 ? attend_smem<96>() : attend_smem<128>();
    const void *fn = ENTRO_BY_TYPE(cache, ENTRO_ATTEND);
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
    r = allow_smem(fn, dev);
    if (r != ENTRO_OK) return r;
    void *args[] = {&a};
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    e = launch_ex(fn, dim3(a.ctas), kAttendThreads, smem, st, 1, false, args);
    if (e == cudaSuccess)
        e = launch_ex(ENTRO_BY_TYPE(cache, ENTRO_JOIN), dim3(static_cast<unsigned>(joins)), kAttendThreads, 0, st, 1, a.join_early, args);
    return e == cudaSuccess ? ENTRO_OK : cuda_fail(e, "entro_kv_attend");
}
