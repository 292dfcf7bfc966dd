// launch.h -- host-side plumbing that the launch code of all kernels shares.
// Not part of the C ABI.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace entro {

// Records the text that entro_last_cuda_error returns; returns ENTRO_E_CUDA.
int cuda_fail(cudaError_t e, const char *where);

struct DeviceInfo {
    int sms = 0;
    int smem_optin = 0;
};
int device_info(int dev, DeviceInfo *out);

// Bytes that the bounded-wait test adds to a barrier and that never arrive (0 in the product).
uint32_t test_tx_extra();

// Lets `fn` use all the shared memory a CTA of the device can have (once per kernel and device).
int allow_smem(const void *fn, int dev);

// How many clusters of `cluster` CTAs the device holds at a time (asked for once per kernel, device and size; the kernel's
// `threads` and `smem` are always the same).
int clusters_at_once(const void *fn, int dev, unsigned threads, size_t smem, int cluster, int *clusters);

// A launch with clusters of `cluster` CTAs along x if above 1.  early: it may begin while the kernel
// before it finishes (its kernel waits for that one before it touches memory).  Only grids whose
// CTAs are all resident at once start early: CTAs of a larger grid would fill the SMs and wait
// there for a kernel that may still need the room.
cudaError_t launch_ex(const void *fn, dim3 grid, unsigned threads, size_t smem, cudaStream_t st, unsigned cluster, bool early,
                      void **args);

// A tiled tensor map over `rank` dimensions (innermost first; strides in bytes of dimensions 1, 2,
// ...), 128-byte swizzle; elements outside read as zero.
int encode_map(CUtensorMap *map, CUtensorMapDataType type, int rank, const void *base, const uint64_t *dims,
               const uint64_t *strides, const uint32_t *box);

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// An output's [tokens][heads] rows of `dim` elements share none: one stride steps over all that the other spans.
inline bool separate_rows(int64_t tokens, int64_t heads, int64_t dim, int64_t token, int64_t head) {
    const auto steps = [](int64_t stride, int64_t n, int64_t span) {  // n rows of `span` elements, `stride` apart
        return n <= 1 || stride >= span;
    };
    const auto span = [dim](int64_t stride, int64_t n) {
        return n <= 1 ? dim : stride > (INT64_MAX - dim) / (n - 1) ? INT64_MAX : (n - 1) * stride + dim;
    };
    return (steps(head, heads, dim) && steps(token, tokens, span(head, heads))) ||
           (steps(token, tokens, dim) && steps(head, heads, span(token, tokens)));
}

}  // namespace entro
