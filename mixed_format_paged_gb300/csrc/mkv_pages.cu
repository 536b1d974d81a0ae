// Page copies of the pool (mkv_seq_fork, mkv_seq_truncate, mkv_seq_copy): rows move, nothing is computed.
//
// Bound: memory, twice the bytes of the rows that hold tokens.  One block per (page, layer, kv head) copies
// its K and V planes; of a page that is not full, only the rows of its tokens (a V token pair is one
// 2 d-byte run, so an odd count rounds up) and their scales.  The rows past them keep what the slot held, which
// the attention kernels clear on their way.
// The list of pages travels as a kernel parameter: no upload, no buffer that a later call could overwrite.
// Measured (HBM copy rate 6,695 GB/s): 64 tail pages of 16 layers x 4 kv heads, 135 MB, 22.2 us with its launch (91 %);
// 8 sequences whole, 1.25 GB, 180.5 us (104 %: the rate is a copy of another length).
#include "mkv_internal.h"

namespace mkv {
namespace {

constexpr int kThreads = 256, kUnroll = 4;

__device__ __forceinline__ void copy16(const uint8_t* src, uint8_t* dst, int n16) {
  const uint4* s = reinterpret_cast<const uint4*>(src);
  uint4* d = reinterpret_cast<uint4*>(dst);
  for (int i = threadIdx.x; i < n16; i += kThreads * kUnroll) {
    uint4 v[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (i + u * kThreads < n16) v[u] = __ldcs(s + i + u * kThreads);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (i + u * kThreads < n16) __stcs(d + i + u * kThreads, v[u]);
  }
}

template <int N>
__global__ void __launch_bounds__(kThreads) mkv_page_copy_kernel(const __grid_constant__ PageCopyParams<N> pp) {
  const PageCopyHead& p = pp.h;
  const int h = blockIdx.x % p.Hkv;
  const int layer = (blockIdx.x / p.Hkv) % p.L;
  const PageCopy pg = pp.page[blockIdx.x / (p.Hkv * p.L)];
  const int f = pg.tq3;
  const int row = f ? 3 * kHeadDim / 8 : kHeadDim;
  const int plane = p.P * (row + 2);
  const int64_t head = int64_t(h) * 2 * plane;
  const uint8_t* src = p.src[f] + layer * p.src_layer[f] + pg.src * p.page_bytes[f] + head;
  uint8_t* dst = p.dst[f] + layer * p.dst_layer[f] + pg.dst * p.page_bytes[f] + head;
  if (pg.nvalid == p.P) {                               // both planes, one run
    copy16(src, dst, 2 * plane / 16);
    return;
  }
  for (int kv = 0; kv < 2; ++kv) {                      // (a TQ3 page is always full)
    const int rows = kv ? (pg.nvalid + 1) & ~1 : pg.nvalid;
    copy16(src, dst, rows * kHeadDim / 16);
    if (threadIdx.x < pg.nvalid)
      reinterpret_cast<uint16_t*>(dst + p.P * kHeadDim)[threadIdx.x] =
          reinterpret_cast<const uint16_t*>(src + p.P * kHeadDim)[threadIdx.x];
    src += plane;
    dst += plane;
  }
}

template <int N>
cudaError_t launch(const PageCopyHead& h, const PageCopy* pages, cudaStream_t s) {
  PageCopyParams<N> p;
  p.h = h;
  for (int i = 0; i < h.n; ++i) p.page[i] = pages[i];
  for (int i = h.n; i < N; ++i) p.page[i] = PageCopy{0, 0, 0, 0};
  mkv_page_copy_kernel<N><<<h.n * h.L * h.Hkv, kThreads, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace

// A launch pays for the parameters it carries, and short lists are the rule: 64 forks with a pass of truncations take
// 15.5 us of host time with a block of 128 entries (2 KB) and 16.4 with one of 1,024.
cudaError_t launch_page_copy(const PageCopyHead& h, const PageCopy* pages, cudaStream_t s) {
  if (h.n <= 0) return cudaSuccess;
  return h.n <= kPageCopiesFew ? launch<kPageCopiesFew>(h, pages, s) : launch<kPageCopies>(h, pages, s);
}

}  // namespace mkv
