// Append to the block-scaled 8-bit cache (mkv_blk8_append).
//
// One block per (touched page, kv head, K|V).  The page's scale is s = 2^e, e the smallest integer with
// max |x| <= 448 2^e over the tokens the page has held since its position 0 was written; codes are
// e4m3_rn(x / s).  Dividing by a power of two is exact, so a code is rounded once, whatever the order in
// which the tokens came; when a new token raises e, the older codes are brought to the new scale, which is
// exact too except where a code falls into e4m3's subnormals (then it is rounded, to nearest even).
// e4m3 has no infinity, and a scale for one would erase the page's other values: infinities become NaN codes, as NaNs
// do, and the maximum is that of the finite values (taken again, from shared memory, by a page that met one).
//
// Bound: memory, the rows in and the codes out.  A page's rows stay in shared memory between the maximum and
// the codes, so they are read once; asynchronous copies bring them there, each thread its own 64 values (no
// barrier between copy and use), so the bytes in flight cost no registers and three blocks of the largest
// pages share an SM.  A single new token's call is latency: table, length, row, maximum, store.
// Measured (HBM copy rate 6,695 GB/s): 32,768 tokens x 4 kv heads x 256, bf16, 202 MB: 35.2 us (85 %; 36.0 with the
// maximum taken in fp32; 106 with the rows held in registers, a quarter of the bytes in flight); one token for each of 64
// sequences: 5.9 us (8.4 with the owner of a page found by bisection).
#include "mkv_blk8.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>

namespace mkv {
namespace {

constexpr unsigned kFull = 0xffffffffu;

// Eight values of a row, from this thread's staging place in shared memory.
__device__ __forceinline__ void get8(const float* p, float (&x)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w; x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
__device__ __forceinline__ void get8(const __nv_bfloat16* p, float (&x)[8]) {
  const uint4 r = *reinterpret_cast<const uint4*>(p);
  const __nv_bfloat162* b = reinterpret_cast<const __nv_bfloat162*>(&r);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __bfloat1622float2(b[i]);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}
__device__ __forceinline__ void get8(const __half* p, float (&x)[8]) {
  const uint4 r = *reinterpret_cast<const uint4*>(p);
  const __half2* b = reinterpret_cast<const __half2*>(&r);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(b[i]);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}
// The largest magnitude so far: 16-bit types two at a time as they are (their order is the floats').
template <typename T> struct Most;
template <> struct Most<float> {
  float m = 0.f;
  __device__ __forceinline__ void add8(const float* p) {
    float x[8];
    get8(p, x);
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(x[i]));
  }
  __device__ __forceinline__ float get() const { return m; }
};
template <typename T, typename T2> struct Most16 {
  T2 m;
  __device__ __forceinline__ Most16() { *reinterpret_cast<uint32_t*>(&m) = 0; }
  __device__ __forceinline__ void add8(const T* p) {
    const uint4 r = *reinterpret_cast<const uint4*>(p);
    const T2* x = reinterpret_cast<const T2*>(&r);
#pragma unroll
    for (int i = 0; i < 4; ++i) m = __hmax2(m, __habs2(x[i]));
  }
};
template <> struct Most<__nv_bfloat16> : Most16<__nv_bfloat16, __nv_bfloat162> {
  __device__ __forceinline__ float get() const { return fmaxf(__low2float(m), __high2float(m)); }
};
template <> struct Most<__half> : Most16<__half, __half2> {
  __device__ __forceinline__ float get() const { return fmaxf(__low2float(m), __high2float(m)); }
};
template <typename T>
__device__ __forceinline__ void stage8(T* to, const T* from) {
  const uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(to));
#pragma unroll
  for (int i = 0; i < int(sizeof(T)) / 2; ++i)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at + 16 * i), "l"(reinterpret_cast<const char*>(from) + 16 * i)
                 : "memory");
}
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ bool finite(float x) { return fabsf(x) < INFINITY; }
// Exponent field of the scale (0: scale 0) for a largest magnitude (finite): 448 = 1.75 * 2^8.
__device__ __forceinline__ int scale_exponent(float amax) {
  if (!(amax > 0.f)) return 0;
  int x;
  const float m = frexpf(amax, &x);                     // amax = m 2^x, m in [1/2, 1)
  const int e = x - (m <= 0.875f ? 9 : 8);
  return min(max(e, -126) + 127, 248);                  // 1 .. 248
}
__device__ __forceinline__ float pow2_field(int f) { return __uint_as_float(static_cast<uint32_t>(f) << 23); }

// THREADS * 64 values cover a page; TP: the type of k and v.
template <typename TP, int THREADS>
__global__ void __launch_bounds__(THREADS, 1536 / THREADS)
mkv_blk8_append_kernel(const __grid_constant__ B8AppendParams p) {
  extern __shared__ __align__(16) uint8_t stage_raw[];  // THREADS * 64 values
  TP* const stage = reinterpret_cast<TP*>(stage_raw) + threadIdx.x * 8;
  __shared__ float warp_max[THREADS / 32];
  const int kv = blockIdx.x & 1;
  const int h = (blockIdx.x >> 1) % p.Hkv;
  const int x = (blockIdx.x >> 1) / p.Hkv;
  // sequence i owns the page numbers base(i) .. base(i + 1), base(i) = cu[i] / P + 2 i: new tokens m touch at
  // most m / P + 2 pages, and floor(a + b) >= floor(a) + floor(b) leaves that many
  // (base is increasing: the owner is the last i with base(i) <= x, and counting those takes one round of loads
  // where a bisection would chain them)
  int below = 0;
  for (int i0 = 0; i0 < p.n; i0 += THREADS) {
    const int i = i0 + threadIdx.x;
    if (i < p.n) asm volatile("prefetch.global.L1 [%0];" ::"l"(p.lens + i));
    below += __syncthreads_count(i < p.n && p.cu[min(i, p.n - 1)] / p.P + 2 * i <= x);
  }
  const int r = max(below, 1) - 1;
  const int c0 = p.cu[r], c1 = p.cu[r + 1], len = p.lens[r];
  const int add = c1 - c0;
  const int old = len - add;
  if (c1 == c0) return;
  if (c0 < 0 || c1 < c0 || c1 > p.tokens || old < 0) {  // rows that are not there, or more of them than the sequence holds
    if (threadIdx.x == 0) atomicOr(p.err, kErrBadPage);
    return;
  }
  const int nth = x - (c0 / p.P + 2 * r);
  if (nth < 0) return;
  const int pg = old / p.P + nth;
  const int start = pg * p.P;
  if (start >= len) return;
  const int page = pg < p.width ? p.table[static_cast<int64_t>(r) * p.width + pg] : -1;
  if (page < 0 || page >= p.pages) {
    if (threadIdx.x == 0) atomicOr(p.err, kErrBadPage);
    return;
  }
  const int t0 = max(old - start, 0), t1 = min(len - start, p.P);      // the page's new tokens
  const int64_t cell = static_cast<int64_t>(page) * p.Hkv + h;
  uint8_t* codes = p.codes[kv] + cell * p.P * p.D;
  const float was = t0 > 0 ? p.scale[kv][cell] : 0.f;   // position 0 starts the page anew
  const int shift = 31 - __clz(p.D) - 3;                // 2^shift units of 8 values in a row
  const int row0 = threadIdx.x >> shift, rows = THREADS >> shift;      // a thread's units lie `rows` rows apart
  const TP* src = static_cast<const TP*>(p.x[kv]) +
                  static_cast<int64_t>(c0 + start + t0 - old + row0) * p.token_stride[kv] + h * p.head_stride[kv] +
                  (threadIdx.x & ((1 << shift) - 1)) * 8;
  const int64_t hop = rows * p.token_stride[kv];
  const int work = t1 - t0 - row0;                      // row j * rows of this thread's is one of the call's while < work
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (j * rows < work) stage8(stage + j * THREADS * 8, src + j * hop);
  asm volatile("cp.async.wait_all;" ::: "memory");
  Most<TP> most;
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (j * rows < work) most.add8(stage + j * THREADS * 8);
  float amax = most.get();
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, o));
  if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = amax;
  __syncthreads();
  amax = warp_max[threadIdx.x & (THREADS / 32 - 1)];
#pragma unroll
  for (int o = THREADS / 64; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, o));
  const bool inf = amax == INFINITY;                    // (of the whole block)
  if (inf) {                                            // the scale is that of the finite values
    amax = 0.f;
#pragma unroll 1
    for (int j = 0; j < 8 && j * rows < work; ++j) {
      float y[8];
      get8(stage + j * THREADS * 8, y);
#pragma unroll
      for (int i = 0; i < 8; ++i) amax = fmaxf(amax, finite(y[i]) ? fabsf(y[i]) : 0.f);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, o));
    __syncthreads();                                    // every thread has read the first maxima
    if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = amax;
    __syncthreads();
    amax = warp_max[threadIdx.x & (THREADS / 32 - 1)];
#pragma unroll
    for (int o = THREADS / 64; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, o));
  }
  const int want = scale_exponent(amax);
  const float now = fmaxf(was, pow2_field(want));
  // 1 / now: the reciprocal of a power of two (2^-126 .. 2^121) is one; a scale that a program filled in itself may be
  // anything, and then the codes are of correctly rounded quotients
  const float inv = now > 0.f ? __frcp_rn(now) : 0.f;
  const bool odd = __float_as_uint(now) & 0x007fffffu;
  __syncthreads();                                      // every thread has read the old scale
  if (threadIdx.x == 0 && (now != was || t0 == 0)) p.scale[kv][cell] = now;
  if (now > was && was > 0.f) {                         // bring the page's older codes to the new scale
    const float ratio = was * inv;
    for (int u = threadIdx.x; u < t0 << shift; u += THREADS) {
      uint2 w = reinterpret_cast<uint2*>(codes)[u];
      uint32_t* half = &w.x;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        uint32_t o = 0;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint32_t f2;
          const uint16_t two = static_cast<uint16_t>(half[k] >> (16 * i));
          asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(f2) : "h"(two));
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&f2));
          o |= e4m3x2(f.x * ratio, f.y * ratio) << (16 * i);
        }
        half[k] = o;
      }
      reinterpret_cast<uint2*>(codes)[u] = w;
    }
  }
  auto put = [&](int j, const float (&y)[8]) {
    uint2 w;
    w.x = e4m3x2(y[0], y[1]) | (e4m3x2(y[2], y[3]) << 16);
    w.y = e4m3x2(y[4], y[5]) | (e4m3x2(y[6], y[7]) << 16);
    reinterpret_cast<uint2*>(codes)[(t0 << shift) + threadIdx.x + j * THREADS] = w;
  };
  if (inf || odd) {                                     // (apart: among the values of every page, 37.0 us became 38.8)
#pragma unroll 1
    for (int j = 0; j * rows < work; ++j) {
      float y[8];
      get8(stage + j * THREADS * 8, y);
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = !finite(y[i]) ? NAN : odd ? __fdiv_rn(y[i], now) : y[i] * inv;
      put(j, y);
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (j * rows >= work) break;
    float y[8];
    get8(stage + j * THREADS * 8, y);
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] *= inv;
    put(j, y);
  }
}

template <typename TP, int THREADS>
cudaError_t start(const B8AppendParams& p, unsigned blocks, cudaStream_t s) {
  constexpr int bytes = THREADS * 64 * int(sizeof(TP));
  if (bytes > 48 * 1024) {
    // a per-device attribute: set once per device (twice from racing threads is harmless)
    static std::atomic<uint64_t> set{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (!bit || !(set.load(std::memory_order_acquire) & bit)) {
      e = cudaFuncSetAttribute(mkv_blk8_append_kernel<TP, THREADS>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
      if (e != cudaSuccess) return e;
      set.fetch_or(bit, std::memory_order_acq_rel);
    }
  }
  mkv_blk8_append_kernel<TP, THREADS><<<blocks, THREADS, bytes, s>>>(p);
  return cudaGetLastError();
}

template <typename TP>
cudaError_t go(const B8AppendParams& p, cudaStream_t s) {
  const int64_t blocks = (int64_t(p.tokens / p.P) + 2 * int64_t(p.n)) * p.Hkv * 2;
  if (blocks <= 0) return cudaSuccess;
  if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
  const int cells = p.P * p.D;                          // 64 values a thread
  if (cells <= 4096) return start<TP, 64>(p, unsigned(blocks), s);
  if (cells <= 8192) return start<TP, 128>(p, unsigned(blocks), s);
  if (cells <= 16384) return start<TP, 256>(p, unsigned(blocks), s);
  return start<TP, 512>(p, unsigned(blocks), s);
}

}  // namespace

cudaError_t launch_b8_append(const B8AppendParams& p, cudaStream_t s) {
  return p.dtype == 0 ? go<float>(p, s) : p.dtype == 1 ? go<__nv_bfloat16>(p, s) : go<__half>(p, s);
}

}  // namespace mkv
