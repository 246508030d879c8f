// pages.cu -- copies pages inside paged caches (bi_kv_copy_pages): the open page of a forked
// sequence, pages moved together when a pool is compacted.
//
// One launch copies the same list of pages in every plane (a layer's K, its V, their scale
// bytes, ...).  The n pages of a plane are taken as one stream of 16-byte units, cut into
// pieces of 2048 units; a CTA copies one piece, each thread eight units that it loads before
// it stores any, so that 32 KB per CTA are in flight.  A page of 16 KB or more lies in few
// pieces and a 512-byte page of scale bytes shares a piece with others.  Bound by memory:
// it reads and writes each byte once -- 1,021 pages of eight layers' 8-bit caches (1.08 GB each
// way) in 312 us, 6.9 TB/s; one page of eight layers' bf16 caches in 3.3 us, launch included.
#include "attn_common.cuh"

namespace bi {
namespace {

constexpr int COPY_THREADS = 256;
constexpr int COPY_UNITS = 8;  // 16-byte units per thread
constexpr int PIECE = COPY_THREADS * COPY_UNITS;

struct CopyArgs {
    uint4* base[kCopyPlanes];
    unsigned int units[kCopyPlanes];      // 16-byte units per page
    unsigned int first[kCopyPlanes + 1];  // first piece of each plane
};

__global__ void __launch_bounds__(COPY_THREADS)
copy_pages_kernel(const __grid_constant__ CopyArgs a, int planes, int num_pages,
                  const int32_t* __restrict__ src, const int32_t* __restrict__ dst, int n,
                  unsigned int* err) {
    pdl_wait();
    pdl_trigger();
    int lo = 0, hi = planes;  // plane of this piece
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.first[mid] <= blockIdx.x) lo = mid; else hi = mid;
    }
    uint4* base = a.base[lo];
    const unsigned int units = a.units[lo];
    const int64_t total = int64_t(n) * units;
    const int64_t at = int64_t(blockIdx.x - a.first[lo]) * PIECE + threadIdx.x;
    uint4 v[COPY_UNITS];
    int64_t to[COPY_UNITS];
#pragma unroll
    for (int k = 0; k < COPY_UNITS; ++k) {
        const int64_t i = at + k * COPY_THREADS;
        to[k] = -1;
        if (i < total) {
            const int page = int(i / units);
            const unsigned int off = unsigned(i - int64_t(page) * units);
            const int s = src[page], d = dst[page];
            if (s >= 0 && s < num_pages && d >= 0 && d < num_pages) {
                v[k] = base[int64_t(s) * units + off];
                to[k] = int64_t(d) * units + off;
            } else if (off == 0) {
                latch_error(err, kErrDeviceArg);
            }
        }
    }
#pragma unroll
    for (int k = 0; k < COPY_UNITS; ++k)
        if (to[k] >= 0) base[to[k]] = v[k];
}

}  // namespace

cudaError_t launch_copy_pages(const DeviceInfo& dev, void* const* planes,
                              const int64_t* page_bytes, int num_planes, int num_pages,
                              const int32_t* src, const int32_t* dst, int n, cudaStream_t stream) {
    for (int p0 = 0; p0 < num_planes; p0 += kCopyPlanes) {
        const int np = num_planes - p0 < kCopyPlanes ? num_planes - p0 : kCopyPlanes;
        CopyArgs a{};
        int64_t first = 0;
        for (int p = 0; p < np; ++p) {
            a.base[p] = static_cast<uint4*>(planes[p0 + p]);
            a.units[p] = unsigned(page_bytes[p0 + p] / 16);
            a.first[p] = unsigned(first);
            first += (int64_t(n) * a.units[p] + PIECE - 1) / PIECE;
            if (first > 0x7fffffffLL) return cudaErrorNotSupported;
        }
        a.first[np] = unsigned(first);
        cudaError_t e = launch_pdl(copy_pages_kernel, dim3(unsigned(first)), dim3(COPY_THREADS), 0,
                                   stream, a, np, num_pages, src, dst, n, dev.err_word);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace bi
