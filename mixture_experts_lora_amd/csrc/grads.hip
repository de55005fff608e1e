// The norm of all gradients together, and the gradients scaled to at most a given norm.
//
//   norm = sqrt(sum over every tensor of g^2)        g' = g min(1, max_norm / (norm + eps))
//
// Squares are summed in 64 bits: float32 would overflow from |g| = 1.8e19 on (bfloat16 reaches 3e38)
// and lose small gradients beside large sums; at two bytes an element the 64-bit sums hide behind
// HBM. The tensors' addresses travel in the kernel arguments, up to kGradTensors a launch, so no
// table has to be copied to the GPU. A launch cuts its tensors into pieces of kGradPiece elements
// and each block sums every so many-th piece into its own partial; one block then adds the partials.
// All sums have an order that depends on the sizes and on which addresses allow 16-byte pieces. Bound
// by HBM: 88 million bfloat16 elements in 48 tensors, squares 31 us (5.7 TB/s, part of it from the
// Infinity Cache), partials 4.6, scaling 61 (5.8 TB/s in and out).
#include <algorithm>

#include "launch.h"
#include "row8.h"

namespace moe {

namespace {

constexpr int kGradTensors = 80;
constexpr int kGradPiece = 16384;
constexpr int kGradBlock = 256;
// Up to so many elements one block of kGradOne threads sums and roots in a single launch (57344
// float32 elements in four tensors, the calls of norm and clip together: 11 us, against 15 with the
// norm in two launches).
constexpr int kGradOne = 1024;
constexpr int64_t kGradOneMost = 131072;
constexpr int kGradBlocks = 2048;  // most partials a launch leaves

struct GradTable {
  const void* src[kGradTensors];
  void* dst[kGradTensors];
  int64_t n[kGradTensors];
  int64_t first[kGradTensors + 1];  // piece at which a tensor starts
  uint8_t dtype[kGradTensors];
  uint8_t vec[kGradTensors];  // its addresses allow 16-byte pieces
  int count;
};
static_assert(sizeof(GradTable) < 3600, "kernel arguments");

// Calls go(tensor, first element, elements) for the pieces of this block.
template <typename F>
__device__ __forceinline__ void for_pieces(const GradTable& t, F&& go) {
  int i = 0;
  const int64_t total = t.first[t.count];
  for (int64_t p = blockIdx.x; p < total; p += gridDim.x) {
    while (p >= t.first[i + 1]) ++i;
    const int64_t at = (p - t.first[i]) * kGradPiece;
    go(i, at, static_cast<int>(min(static_cast<int64_t>(kGradPiece), t.n[i] - at)));
  }
}

template <int BLOCK, typename Elem>
__device__ __forceinline__ double squares(const Elem* g, int n, bool vec) {
  double s[2] = {0.0, 0.0};
  auto add = [&](int j, float x) __attribute__((always_inline)) {
    const double d = static_cast<double>(x);
    s[j & 1] = __builtin_fma(d, d, s[j & 1]);
  };
  int done = 0;
  if (vec) {
    done = n & ~7;
    constexpr int STEP = BLOCK * 8;
    int i = threadIdx.x * 8;
    for (; i + 3 * STEP < done; i += 4 * STEP) {
      Row8<Elem> r[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) r[u].load(g + i + u * STEP);
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        float v[8];
        r[u].get(v);
#pragma unroll
        for (int j = 0; j < 8; ++j) add(j, v[j]);
      }
    }
    for (; i < done; i += STEP) {
      Row8<Elem> r;
      r.load(g + i);
      float v[8];
      r.get(v);
#pragma unroll
      for (int j = 0; j < 8; ++j) add(j, v[j]);
    }
  }
  for (int i = done + threadIdx.x; i < n; i += BLOCK) add(0, to_f32<Elem>(g[i]));
  return s[0] + s[1];
}

// The block's sum, in thread 0: lanes by halves, then the waves in order.
template <int BLOCK>
__device__ __forceinline__ double block_sum(double s) {
  __shared__ double part[BLOCK / kWave];
#pragma unroll
  for (int d = kWave / 2; d > 0; d >>= 1) s += __shfl_xor(s, d, kWave);
  if ((threadIdx.x & (kWave - 1)) == 0) part[threadIdx.x / kWave] = s;
  __syncthreads();
  s = part[0];
#pragma unroll
  for (int w = 1; w < BLOCK / kWave; ++w) s += part[w];
  return s;
}

template <bool ONE>
__global__ __launch_bounds__(ONE ? kGradOne : kGradBlock) void grad_squares_kernel(GradTable t,
                                                                                   double* part,
                                                                                   float* norm) {
  constexpr int BLOCK = ONE ? kGradOne : kGradBlock;
  double s = 0.0;
  for_pieces(t, [&](int i, int64_t at, int n) __attribute__((always_inline)) {
    if (t.dtype[i] == MOE_F32)
      s += squares<BLOCK>(static_cast<const float*>(t.src[i]) + at, n, t.vec[i]);
    else if (t.dtype[i] == MOE_BF16)
      s += squares<BLOCK>(static_cast<const bf16_t*>(t.src[i]) + at, n, t.vec[i]);
    else
      s += squares<BLOCK>(static_cast<const f16_t*>(t.src[i]) + at, n, t.vec[i]);
  });
  s = block_sum<BLOCK>(s);
  if (threadIdx.x == 0) {
    if (ONE) *norm = static_cast<float>(sqrt(s));
    else part[blockIdx.x] = s;
  }
}

__global__ __launch_bounds__(kGradBlock) void grad_norm_kernel(const double* part, int n,
                                                               float* norm) {
  double s = 0.0;
  for (int i = threadIdx.x; i < n; i += kGradBlock) s += part[i];
  s = block_sum<kGradBlock>(s);
  if (threadIdx.x == 0) *norm = static_cast<float>(sqrt(s));
}

template <typename Elem>
__device__ __forceinline__ void scale_piece(const Elem* src, Elem* dst, int n, bool vec, float c) {
  int done = 0;
  if (vec) {
    done = n & ~7;
    for (int i = threadIdx.x * 8; i < done; i += kGradBlock * 8) {
      Row8<Elem> r;
      r.load(src + i);
      float v[8];
      r.get(v);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] *= c;
      r.set(v);
      r.store(dst + i);
    }
  }
  for (int i = done + threadIdx.x; i < n; i += kGradBlock)
    dst[i] = from_f32<Elem>(to_f32<Elem>(src[i]) * c);
}

// Where nothing is clipped (c = 1) a gradient that stays in place is neither read nor written.
__global__ __launch_bounds__(kGradBlock) void grad_clip_kernel(GradTable t, const float* norm,
                                                               float max_norm, float eps) {
  const double want = static_cast<double>(max_norm) / (static_cast<double>(*norm) + eps);
  // a NaN norm passes through, as max_norm / infinity = 0 does
  const float c = want > 1.0 ? 1.0f : static_cast<float>(want);
  for_pieces(t, [&](int i, int64_t at, int n) __attribute__((always_inline)) {
    if (c == 1.0f && t.src[i] == t.dst[i]) return;
    if (t.dtype[i] == MOE_F32)
      scale_piece(static_cast<const float*>(t.src[i]) + at, static_cast<float*>(t.dst[i]) + at, n,
                  t.vec[i], c);
    else if (t.dtype[i] == MOE_BF16)
      scale_piece(static_cast<const bf16_t*>(t.src[i]) + at, static_cast<bf16_t*>(t.dst[i]) + at, n,
                  t.vec[i], c);
    else
      scale_piece(static_cast<const f16_t*>(t.src[i]) + at, static_cast<f16_t*>(t.dst[i]) + at, n,
                  t.vec[i], c);
  });
}

// The next tensors that fit a launch; returns how many of the list were taken (empty ones among
// them). For the norm alone a dst may be anything.
int fill_table(const moe_grad* g, int count, bool norm, GradTable* t) {
  int taken = 0;
  t->count = 0;
  t->first[0] = 0;
  for (; taken < count && t->count < kGradTensors; ++taken) {
    const moe_grad& x = g[taken];
    if (x.n == 0) continue;
    const int i = t->count++;
    t->src[i] = x.src;
    t->dst[i] = x.dst;
    t->n[i] = x.n;
    t->dtype[i] = static_cast<uint8_t>(x.dtype);
    const void* dst = norm ? x.src : x.dst;
    t->vec[i] = ((reinterpret_cast<uintptr_t>(x.src) | reinterpret_cast<uintptr_t>(dst)) & 15) == 0;
    t->first[i + 1] = t->first[i] + (x.n + kGradPiece - 1) / kGradPiece;
  }
  return taken;
}

int64_t blocks_of(const GradTable& t) {
  return std::min<int64_t>(t.first[t.count], kGradBlocks);
}

// Whether one block sums the whole list: it fits a launch, and adding partials up would cost more.
bool one_block(int count, const moe_grad* grads) {
  int64_t n = 0;
  int tensors = 0;
  for (int i = 0; i < count; ++i) {
    n += grads[i].n;
    tensors += grads[i].n > 0;
    if (n > kGradOneMost || tensors > kGradTensors) return false;
  }
  return tensors > 0;
}

}  // namespace

size_t grad_norm_ws_bytes(int count, const moe_grad* grads) {
  if (one_block(count, grads)) return 0;
  int64_t parts = 0;
  for (int at = 0; at < count;) {
    GradTable t;
    at += fill_table(grads + at, count - at, true, &t);
    parts += blocks_of(t);
  }
  return static_cast<size_t>(parts) * sizeof(double);
}

hipError_t launch_grad_norm(int count, const moe_grad* grads, float* norm, void* ws, hipStream_t s,
                            KernelTimer* tm) {
  TimedScope ts(tm, MOE_K_GRAD_NORM, s);
  double* part = static_cast<double*>(ws);
  if (one_block(count, grads)) {
    GradTable t;
    fill_table(grads, count, true, &t);
    hipLaunchKernelGGL(grad_squares_kernel<true>, dim3(1), dim3(kGradOne), 0, s, t, part, norm);
    return hipGetLastError();
  }
  int64_t parts = 0;
  for (int at = 0; at < count;) {
    GradTable t;
    at += fill_table(grads + at, count - at, true, &t);
    const int64_t blocks = blocks_of(t);
    if (blocks == 0) continue;
    hipLaunchKernelGGL(grad_squares_kernel<false>, dim3(static_cast<unsigned>(blocks)),
                       dim3(kGradBlock), 0, s, t, part + parts, norm);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    parts += blocks;
  }
  // (of no elements at all: the sum of no partials)
  hipLaunchKernelGGL(grad_norm_kernel, dim3(1), dim3(kGradBlock), 0, s, part,
                     static_cast<int>(parts), norm);
  return hipGetLastError();
}

hipError_t launch_grad_clip(int count, const moe_grad* grads, const float* norm, float max_norm,
                            float eps, hipStream_t s, KernelTimer* tm) {
  TimedScope ts(tm, MOE_K_GRAD_CLIP, s);
  for (int at = 0; at < count;) {
    GradTable t;
    at += fill_table(grads + at, count - at, false, &t);
    const int64_t blocks = blocks_of(t);
    if (blocks == 0) continue;
    hipLaunchKernelGGL(grad_clip_kernel, dim3(static_cast<unsigned>(blocks)), dim3(kGradBlock), 0,
                       s, t, norm, max_norm, eps);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace moe
