// The norm of many gradients together, and the gradients scaled back to a largest norm,
// for gfx950.
//
//   norm = sqrt(sum over tensors and elements of g^2)
//   out  = g * min(1, max_norm / norm)
//
// Both passes are bound by HBM.  The tensors of a launch come in its arguments (no table
// in device memory, so the call is captured like any other); they are cut into chunks of
// kChunk elements, workgroup b takes chunks b, b + grid, ..., and a chunk's tensor is found
// by one comparison per lane.  Squares are summed in 64 bits (bf16 and float32 squares pass
// float32's range at both ends); the sums of the workgroups meet in a fixed order, by every
// workgroup of the second pass for itself, which spares a launch between the two.  That
// pass walks the chunks from the last to the first, whose bytes the memory-side cache
// still holds (648 us from the first on, 627 so), and its results go past the caches where
// they do not fit there (659 us into them).
//
// 604 million bf16 gradients in three tensors: the norm 200 us (6.0 TB/s of 1.2 GB), norm
// and clipped copy 625 us (5.8 TB/s of 3.6 GB), in place 613, nothing to clip in place 200.
#include <hip/hip_runtime.h>

#include <float.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "ops_internal.h"
#include "row_common.h"

namespace moe {
namespace {

using namespace row;

constexpr int kThreads = 256;
constexpr int kChunk = 8192;    // elements
constexpr int kTensors = 96;    // per launch: the arguments stay below 4 KB
constexpr int kGroups = 1024;   // workgroups of a pass over everything (2048: 627 us, 623 with 1024, see below)
constexpr int64_t kCacheBytes = 192 << 20;  // gradients past this do not stay in the 256 MB memory-side cache

struct Tensors {
  const void* g[kTensors];
  void* out[kTensors];
  int64_t n[kTensors];           // elements
  uint32_t first[kTensors];      // first chunk; 2^32 - 1 past the last tensor
  uint32_t f32[kTensors / 32];   // a bit per tensor
  uint32_t chunks;
};
static_assert(sizeof(Tensors) < 3584, "with the other arguments below 4 KB");

// The tensor of chunk c: how many first chunks are not past it, less one.
__device__ __forceinline__ int tensor_of(const Tensors& t, uint32_t c) {
  const int lane = threadIdx.x & 63;
  int n = 0;
#pragma unroll
  for (int i = 0; i < (kTensors + 63) / 64; ++i) {
    const int at = i * 64 + lane;
    n += __builtin_popcountll(__ballot(at < kTensors && t.first[at < kTensors ? at : 0] <= c));
  }
  return __builtin_amdgcn_readfirstlane(n - 1);
}

__device__ __forceinline__ double wave_sum64(double v) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
  return v;
}
// Sum over the workgroup, the same bits in every thread.
__device__ __forceinline__ double block_sum64(double v) {
  __shared__ double part[kThreads / 64];
  v = wave_sum64(v);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x / 64] = v;
  __syncthreads();
  double s = part[0];
#pragma unroll
  for (int i = 1; i < kThreads / 64; ++i) s += part[i];
  return s;
}

template <typename T>
__device__ __forceinline__ double chunk_squares(const T* __restrict__ g, int n) {
  constexpr int kSteps = kChunk / (kThreads * 8);
  double s[2] = {0.0, 0.0};
  Piece<T> p[kSteps];
#pragma unroll
  for (int i = 0; i < kSteps; ++i) p[i].load(g, (i * kThreads + (int)threadIdx.x) * 8, n);
#pragma unroll
  for (int i = 0; i < kSteps; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const double v = (double)p[i].get(e);
      s[e & 1] = fma(v, v, s[e & 1]);
    }
  return s[0] + s[1];
}

__global__ __launch_bounds__(kThreads) void squares_kernel(Tensors t, double* part) {
  double s = 0.0;
  for (uint32_t c = blockIdx.x; c < t.chunks; c += gridDim.x) {
    const int i = tensor_of(t, c);
    const int64_t at = (int64_t)(c - t.first[i]) * kChunk;
    const int n = (int)min((int64_t)kChunk, t.n[i] - at);
    s += t.f32[i / 32] >> (i % 32) & 1 ? chunk_squares(static_cast<const float*>(t.g[i]) + at, n)
                                       : chunk_squares(static_cast<const uint16_t*>(t.g[i]) + at, n);
  }
  s = block_sum64(s);
  if (threadIdx.x == 0) part[blockIdx.x] = s;
}

// The norm from the workgroups' sums, in a fixed order.
__device__ __forceinline__ double norm_of(const double* part, int parts) {
  double s = 0.0;
  for (int i = threadIdx.x; i < parts; i += kThreads) s += part[i];
  return sqrt(block_sum64(s));
}

__global__ __launch_bounds__(kThreads) void norm_kernel(const double* part, int parts, float* norm) {
  const float v = (float)norm_of(part, parts);
  if (threadIdx.x == 0) *norm = v;
}

// `past_cache`: whole pieces go past the caches, for gradients too many to be read from there.
__device__ __forceinline__ void store_piece(uint16_t* out, int at, int n, const float (&v)[8], bool past_cache) {
  if (!past_cache || at + 8 > n) return store8(out, at, n, v);
  const u32x4_e2 d{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])};
  __builtin_nontemporal_store(d, reinterpret_cast<u32x4_e2*>(out + at));
}
__device__ __forceinline__ void store_piece(float* out, int at, int n, const float (&v)[8], bool past_cache) {
  if (!past_cache || at + 8 > n) return store8(out, at, n, v);
#pragma unroll
  for (int h = 0; h < 8; h += 4) {
    const u32x4_e4 d{__float_as_uint(v[h]), __float_as_uint(v[h + 1]), __float_as_uint(v[h + 2]), __float_as_uint(v[h + 3])};
    __builtin_nontemporal_store(d, reinterpret_cast<u32x4_e4*>(out + at + h));
  }
}

// `F`: the factor's type, in which the products are made.
template <typename F, typename T>
__device__ __forceinline__ void scale_chunk(const T* g, T* out, int n, F c, bool past_cache) {
  constexpr int kSteps = kChunk / (kThreads * 8);
  Piece<T> p[kSteps];
#pragma unroll
  for (int i = 0; i < kSteps; ++i) p[i].load(g, (i * kThreads + (int)threadIdx.x) * 8, n);
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int at = (i * kThreads + (int)threadIdx.x) * 8;
    if (at >= n) break;
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = (float)(p[i].get(e) * c);
    store_piece(out, at, n, v, past_cache);
  }
}

// This workgroup's chunks times c.  What stays as it is and where it is is not written.
template <typename F>
__device__ __forceinline__ void clip_chunks(const Tensors& t, F c, bool past_cache) {
  for (uint32_t k = blockIdx.x; k < t.chunks; k += gridDim.x) {
    const uint32_t id = t.chunks - 1 - k;
    const int i = tensor_of(t, id);
    if (c == 1 && t.out[i] == t.g[i]) continue;
    const int64_t at = (int64_t)(id - t.first[i]) * kChunk;
    const int n = (int)min((int64_t)kChunk, t.n[i] - at);
    if (t.f32[i / 32] >> (i % 32) & 1)
      scale_chunk(static_cast<const float*>(t.g[i]) + at, static_cast<float*>(t.out[i]) + at, n, c, past_cache);
    else
      scale_chunk(static_cast<const uint16_t*>(t.g[i]) + at, static_cast<uint16_t*>(t.out[i]) + at, n, c, past_cache);
  }
}

// `part`: the sums of the first pass, or nullptr: the norm is there already.
__global__ __launch_bounds__(kThreads) void clip_kernel(Tensors t, const double* part, int parts, float* norm, float max_norm,
                                                        int write_norm, int in_place, int past_cache) {
  double norm64;
  float v;
  if (part != nullptr) {
    norm64 = norm_of(part, parts);
    v = (float)norm64;
    if (write_norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = v;
    // the norm that is returned, so that a clip of its own gives the same bits, but where
    // float32 cannot hold it
    if (v < INFINITY) norm64 = v;
  } else {
    norm64 = v = *norm;
  }
  // a norm that is NaN or infinite scales nothing
  const bool scaled = norm64 > max_norm && norm64 < (double)INFINITY;
  const float c = scaled ? max_norm / v : 1.0f;
  if (c == 1.0f && in_place) return;
  // the factor by such a norm, or below float32's normal range, where it would have lost
  // bits, and its products are in 64 bits
  if (c < FLT_MIN)
    clip_chunks(t, (double)max_norm / norm64, past_cache);
  else
    clip_chunks(t, c, past_cache);
}

int64_t chunks_of(int64_t n) { return (n + kChunk - 1) / kChunk; }

// Workgroups of a launch with `chunks` of `total` chunks.
int groups_of(int64_t chunks, int64_t total) {
  return (int)std::max<int64_t>(1, std::min<int64_t>(chunks, chunks * kGroups / std::max<int64_t>(total, kGroups)));
}

// Calls f(tensors of one launch, workgroups) for all of them, kTensors at a time, from the
// first or from the last on; the workgroups are shared out by the launches' chunks.
template <typename F>
hipError_t for_launches(const GradTensor* list, int64_t count, bool reverse, F f) {
  int64_t total = 0;
  for (int64_t i = 0; i < count; ++i) total += chunks_of(list[i].n);
  const int64_t launches = (count + kTensors - 1) / kTensors;
  for (int64_t k = 0; k < launches; ++k) {
    const int64_t l = reverse ? launches - 1 - k : k;
    Tensors t{};
    int64_t c = 0;
    int at = 0;
    for (int64_t i = l * kTensors; i < std::min(count, (l + 1) * kTensors); ++i) {
      if (list[i].n == 0) continue;
      t.g[at] = list[i].g;
      t.out[at] = list[i].out;
      t.n[at] = list[i].n;
      t.first[at] = (uint32_t)c;
      if (list[i].f32) t.f32[at / 32] |= 1u << (at % 32);
      c += chunks_of(list[i].n);
      ++at;
    }
    if (c == 0) continue;
    t.chunks = (uint32_t)c;
    for (; at < kTensors; ++at) t.first[at] = 0xffffffffu;
    const hipError_t e = f(t, groups_of(c, total));
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

size_t grad_norm_workspace(int64_t count) { return (kGroups + (size_t)(count + kTensors - 1) / kTensors) * sizeof(double); }

bool grad_sizes_ok(const GradTensor* list, int64_t count) {
  for (int64_t l = 0; l < count; l += kTensors) {
    int64_t c = 0;
    for (int64_t i = l; i < std::min(count, l + kTensors); ++i) {
      c += chunks_of(list[i].n);
      if (c >= (int64_t)0xffffffff) return false;
    }
  }
  return true;
}

hipError_t launch_grad_squares(const GradTensor* list, int64_t count, double* part, int* parts, hipStream_t s) {
  *parts = 0;
  return for_launches(list, count, false, [&](const Tensors& t, int groups) {
    hipLaunchKernelGGL(squares_kernel, dim3(groups), dim3(kThreads), 0, s, t, part + *parts);
    *parts += groups;
    return hipGetLastError();
  });
}

hipError_t launch_grad_norm(const double* part, int parts, float* norm, hipStream_t s) {
  hipLaunchKernelGGL(norm_kernel, dim3(1), dim3(kThreads), 0, s, part, parts, norm);
  return hipGetLastError();
}

hipError_t launch_grad_clip(const GradTensor* list, int64_t count, const double* part, int parts, float* norm, float max_norm,
                            bool in_place, hipStream_t s) {
  bool first = part != nullptr;
  int64_t bytes = 0;
  for (int64_t i = 0; i < count; ++i) bytes += list[i].n * (list[i].f32 ? 4 : 2);
  return for_launches(list, count, true, [&](const Tensors& t, int groups) {
    hipLaunchKernelGGL(clip_kernel, dim3(groups), dim3(kThreads), 0, s, t, part, parts, norm, max_norm, first ? 1 : 0, in_place ? 1 : 0, bytes > kCacheBytes ? 1 : 0);
    first = false;
    return hipGetLastError();
  });
}

}  // namespace moe
