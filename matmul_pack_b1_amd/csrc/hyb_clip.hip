// Kernels of the 2-norm over a list of tensors and their scaling
// (include/hyb_clip.h).  Bound by memory: 872 MB of gradients are read in 129-145 us
// (6.0-6.7 TB/s) and scaled in 317-332 (5.3-5.5), 450 in all in a loop (491 with loads and
// stores that the caches keep); nine small ones take the depth of two launches, 4.6 and 6.1
// us.
//
// Squares are fp64: the converting and the fused multiply-add of an element take
// less of the vector unit than its bytes take of memory, and no sum overflows or
// loses what is small beside it.
#include <type_traits>

#include "hyb_clip_internal.h"
#include "hyb_panel.h"
#include "hyb_stream.h"

namespace hyb {
namespace {

// The tensors of one launch, at most N; tensor i has chunks start[i] ..
// start[i + 1] - 1, rows' chunks one after the other.  A list of up to twelve has a
// small table, since the host copies it for every launch: nine tensors 15.3-17.0 us a call,
// with the large one 16.3-17.4 (in each of four processes; 20 tensors with a table of 32 or
// of 64 differ by less than the processes do).
template <int N>
struct ClipTable {
  const char* data[N];
  char* out[N];
  int64_t cols[N], lda[N], ldo[N];
  int64_t start[N + 1];
  uint8_t dtype[N];
  int32_t count;
};
static_assert(sizeof(ClipTable<kClipTensors>) + 64 <= 4096, "kernel arguments");
constexpr int kClipFew = 12;

template <int N>
__device__ __forceinline__ int clip_find(const ClipTable<N>& t, int64_t chunk) {
  int lo = 0, hi = t.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.start[mid] <= chunk)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

// Sum over the workgroup's 256 threads, in a fixed order; the result is in every
// thread.
__device__ __forceinline__ double clip_block_sum(double v, double* lds) {
#pragma unroll
  for (int d = 1; d < 64; d *= 2) v += __shfl_xor(v, d);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  return (lds[0] + lds[1]) + (lds[2] + lds[3]);
}

// Sum of squares of the 16 bytes at p.
template <int DT>
__device__ __forceinline__ double clip_squares(const Bytes16& b) {
  double s = 0.0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (DT == HYB_F32) {
      const double v = double(__builtin_bit_cast(float, b.w[i]));
      s = __builtin_fma(v, v, s);
    } else {
      const double v = double(widen16<DT>(b.w[i] & 0xFFFFu)), u = double(widen16<DT>(b.w[i] >> 16));
      s = __builtin_fma(v, v, s);
      s = __builtin_fma(u, u, s);
    }
  }
  return s;
}

template <int DT>
__device__ __forceinline__ float clip_read(const char* p, int64_t i) {
  if constexpr (DT == HYB_F32)
    return reinterpret_cast<const float*>(p)[i];
  else
    return widen16<DT>(reinterpret_cast<const uint16_t*>(p)[i]);
}

// Lists beyond kStreamBytes (STREAM) are read and written around the caches.
template <bool STREAM>
__device__ __forceinline__ Bytes16 clip_load(const char* p) {
  if constexpr (STREAM)
    return stream_load(p);
  else
    return *reinterpret_cast<const Bytes16*>(p);
}
template <bool STREAM>
__device__ __forceinline__ void clip_store(char* p, const Bytes16& b) {
  if constexpr (STREAM)
    stream_store(p, b);
  else
    *reinterpret_cast<Bytes16*>(p) = b;
}

// A thread's share of the squares of `n` elements at p.
template <int DT, bool STREAM>
__device__ __forceinline__ double clip_chunk(const char* p, int32_t n) {
  constexpr int kEach = DT == HYB_F32 ? 4 : 8;  // of 16 bytes
  const int32_t whole = n / kEach;
  double s = 0.0;
  int32_t i = threadIdx.x;
  for (; i + 1792 < whole; i += 2048) {
    Bytes16 b[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) b[u] = clip_load<STREAM>(p + (i + 256 * u) * 16);
#pragma unroll
    for (int u = 0; u < 8; ++u) s += clip_squares<DT>(b[u]);
  }
  for (; i < whole; i += 256) s += clip_squares<DT>(reinterpret_cast<const Bytes16*>(p)[i]);
  const int32_t at = whole * kEach + int32_t(threadIdx.x);
  if (at < n) {
    const double v = double(clip_read<DT>(p, at));
    s = __builtin_fma(v, v, s);
  }
  return s;
}

// Chunk `chunk` of tensor i: f(data, out, elements).
template <int N, typename F>
__device__ __forceinline__ void clip_at(const ClipTable<N>& t, int i, int64_t chunk, F f) {
  const int64_t per = (t.cols[i] + kClipChunk - 1) / kClipChunk, c = chunk - t.start[i];
  const int64_t row = c / per, col = (c - row * per) * kClipChunk;
  const int32_t n = int32_t(t.cols[i] - col < kClipChunk ? t.cols[i] - col : kClipChunk);
  const int size = t.dtype[i] == HYB_F32 ? 4 : 2;
  f(t.data[i] + (row * t.lda[i] + col) * size, t.out[i] + (row * t.ldo[i] + col) * size, n);
}

template <int N, bool STREAM>
__global__ __launch_bounds__(256) void k_clip_squares(ClipTable<N> t, double* __restrict__ sums) {
  __shared__ double lds[4];
  const int64_t all = t.start[t.count];
  double s = 0.0;
  for (int64_t c = blockIdx.x; c < all; c += gridDim.x) {
    const int i = clip_find(t, c);
    clip_at(t, i, c, [&](const char* p, char*, int32_t n) {
      if (t.dtype[i] == HYB_F32)
        s += clip_chunk<HYB_F32, STREAM>(p, n);
      else if (t.dtype[i] == HYB_BF16)
        s += clip_chunk<HYB_BF16, STREAM>(p, n);
      else
        s += clip_chunk<HYB_F16, STREAM>(p, n);
    });
  }
  s = clip_block_sum(s, lds);
  if (threadIdx.x == 0) sums[blockIdx.x] = s;
}

// The norm from the partial sums, in every thread.
__device__ __forceinline__ double clip_norm(const double* __restrict__ sums, int64_t count, double* lds) {
  double s = 0.0;
  for (int64_t i = threadIdx.x; i < count; i += 256) s += sums[i];
  return __builtin_sqrt(clip_block_sum(s, lds));
}

__global__ __launch_bounds__(256) void k_clip_norm(const double* __restrict__ sums, int64_t count,
                                                   float* __restrict__ norm) {
  __shared__ double lds[4];
  const double v = clip_norm(sums, count, lds);
  if (threadIdx.x == 0) *norm = float(v);
}

template <int DT, bool STREAM>
__device__ __forceinline__ void clip_scale(const char* p, char* q, int32_t n, float f) {
  constexpr int kEach = DT == HYB_F32 ? 4 : 8;
  const int32_t whole = n / kEach;
  auto scaled = [&](const Bytes16& b) {
    Bytes16 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (DT == HYB_F32)
        r.w[i] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(float, b.w[i]) * f);
      else
        r.w[i] = round16x2<DT>(widen16<DT>(b.w[i] & 0xFFFFu) * f, widen16<DT>(b.w[i] >> 16) * f);
    }
    return r;
  };
  int32_t i = threadIdx.x;
  for (; i + 1792 < whole; i += 2048) {
    Bytes16 b[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) b[u] = clip_load<STREAM>(p + (i + 256 * u) * 16);
#pragma unroll
    for (int u = 0; u < 8; ++u) clip_store<STREAM>(q + (i + 256 * u) * 16, scaled(b[u]));
  }
  for (; i < whole; i += 256) reinterpret_cast<Bytes16*>(q)[i] = scaled(reinterpret_cast<const Bytes16*>(p)[i]);
  const int32_t at = whole * kEach + int32_t(threadIdx.x);
  if (at < n) {
    const float v = clip_read<DT>(p, at) * f;
    if constexpr (DT == HYB_F32)
      reinterpret_cast<float*>(q)[at] = v;
    else
      reinterpret_cast<uint16_t*>(q)[at] = round16<DT>(v);
  }
}

// Every workgroup takes the norm from the sums itself (they lie in the caches),
// which saves a launch.
template <int N, bool STREAM>
__global__ __launch_bounds__(256) void k_clip_scale(ClipTable<N> t, const double* __restrict__ sums, int64_t count,
                                                    float max_norm, float* __restrict__ norm) {
  __shared__ double lds[4];
  const double v = clip_norm(sums, count, lds);
  if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = float(v);
  const double r = double(max_norm) / (v + 1e-6);
  const float f = r < 1.0 || r != r ? float(r) : 1.f;
  // from the last chunk to the first: what the squares read last lies in the
  // last-level cache (872 MB, kept by the caches, 492 us, from the first on 522)
  const int64_t all = t.start[t.count];
  for (int64_t c = all - 1 - blockIdx.x; c >= 0; c -= gridDim.x) {
    const int i = clip_find(t, c);
    if (f == 1.f && t.out[i] == t.data[i]) continue;
    clip_at(t, i, c, [&](const char* p, char* q, int32_t n) {
      if (t.dtype[i] == HYB_F32)
        clip_scale<HYB_F32, STREAM>(p, q, n, f);
      else if (t.dtype[i] == HYB_BF16)
        clip_scale<HYB_BF16, STREAM>(p, q, n, f);
      else
        clip_scale<HYB_F16, STREAM>(p, q, n, f);
    });
  }
}

template <int N>
ClipTable<N> table_of(const std::vector<hyb_tensor>& tensors, const ClipLaunch& l) {
  ClipTable<N> t;
  t.count = l.count;
  t.start[0] = 0;
  for (int j = 0; j < l.count; ++j) {
    const hyb_tensor& x = tensors[l.first + j];
    t.data[j] = static_cast<const char*>(x.data);
    t.out[j] = static_cast<char*>(x.out);
    t.cols[j] = x.cols;
    t.lda[j] = x.lda;
    t.ldo[j] = x.ldo;
    t.dtype[j] = uint8_t(x.dtype);
    t.start[j + 1] = t.start[j] + x.rows * ((x.cols + kClipChunk - 1) / kClipChunk);
  }
  return t;
}

template <typename F>
void with_table(int count, F f) {
  if (count <= kClipFew)
    f(std::integral_constant<int, kClipFew>());
  else
    f(std::integral_constant<int, kClipTensors>());
}

// More bytes than the last-level cache holds?
bool streamed(const std::vector<hyb_tensor>& tensors) {
  int64_t bytes = 0;
  for (const hyb_tensor& t : tensors) bytes += t.rows * t.cols * (t.dtype == HYB_F32 ? 4 : 2);
  return bytes > kStreamBytes;
}

hipError_t launch_squares(const std::vector<hyb_tensor>& tensors, const std::vector<ClipLaunch>& plan, double* ws,
                          bool stream, hipStream_t s) {
  for (const ClipLaunch& l : plan) {
    auto go = [&](auto kernel, auto few) {
      hipLaunchKernelGGL(kernel, dim3(unsigned(l.groups)), dim3(256), 0, s, table_of<decltype(few)::value>(tensors, l),
                         ws + l.sum0);
    };
    with_table(l.count, [&](auto n) {
      constexpr int N = decltype(n)::value;
      stream ? go(&k_clip_squares<N, true>, n) : go(&k_clip_squares<N, false>, n);
    });
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_norm(const std::vector<hyb_tensor>& tensors, float* norm, double* ws, hipStream_t s) {
  int64_t sums;
  const std::vector<ClipLaunch> plan = clip_plan(tensors, &sums);
  const hipError_t e = launch_squares(tensors, plan, ws, streamed(tensors), s);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(k_clip_norm, dim3(1), dim3(256), 0, s, ws, sums, norm);
  return hipGetLastError();
}

hipError_t launch_clip(const std::vector<hyb_tensor>& tensors, float max_norm, float* norm, double* ws, hipStream_t s) {
  if (tensors.empty()) return launch_norm(tensors, norm, ws, s);
  int64_t sums;
  const std::vector<ClipLaunch> plan = clip_plan(tensors, &sums);
  const bool stream = streamed(tensors);
  hipError_t e = launch_squares(tensors, plan, ws, stream, s);
  for (size_t i = plan.size(); i-- > 0 && e == hipSuccess;) {
    const ClipLaunch& l = plan[i];
    float* to = i == 0 ? norm : nullptr;
    auto go = [&](auto kernel, auto few) {
      hipLaunchKernelGGL(kernel, dim3(unsigned(l.groups)), dim3(256), 0, s, table_of<decltype(few)::value>(tensors, l), ws,
                         sums, max_norm, to);
    };
    with_table(l.count, [&](auto n) {
      constexpr int N = decltype(n)::value;
      stream ? go(&k_clip_scale<N, true>, n) : go(&k_clip_scale<N, false>, n);
    });
    e = hipGetLastError();
  }
  return e;
}

}  // namespace hyb
