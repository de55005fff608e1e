// Rows to microscaled codes and back (mx.h has the formats). Bound by HBM: a thread takes 8
// elements at a time, four lanes a block of 32, and every byte moves once (184320 x 2880 bfloat16 to
// 4 bits 256 us, 5.2 TB/s, and back 235).
#include <type_traits>

#include "launch.h"
#include "mx.h"

namespace moe {

namespace {

constexpr int kMxBlock = 256;

struct MxArgs {
  int64_t chunks;      // of 8 elements
  uint32_t row_blocks;  // blocks of 32 a row
  uint32_t scale_cols;
};

// Where block b (over all rows) has its scale, and whether it is its row's last.
__device__ __forceinline__ int64_t scale_at(const MxArgs& p, uint32_t b, bool& last) {
  const uint32_t row = b / p.row_blocks, in = b - row * p.row_blocks;
  last = in + 1 == p.row_blocks;
  return static_cast<int64_t>(row) * p.scale_cols + in;
}

template <typename Elem, int FMT>
__global__ __launch_bounds__(kMxBlock) void mx_quantize_kernel(MxArgs p, const Elem* src,
                                                               uint8_t* codes, uint8_t* scales) {
  const int64_t c = static_cast<int64_t>(blockIdx.x) * kMxBlock + threadIdx.x;
  if (c >= p.chunks) return;  // a quad is in or out as one: a row is whole blocks
  Row8<Elem> r;
  r.load(src + c * 8);
  float v[8];
  r.get(v);
  const uint32_t s = mx_scale_of<FMT>(mx_block_amax(v));
  const uint2 q = mx_encode8<FMT>(v, s);
  if constexpr (FMT == MOE_MX_FP4)
    reinterpret_cast<uint32_t*>(codes)[c] = q.x;
  else
    reinterpret_cast<uint2*>(codes)[c] = q;
  if ((threadIdx.x & 3) == 0) {
    bool last;
    uint8_t* at = scales + scale_at(p, static_cast<uint32_t>(c >> 2), last);
    *at = static_cast<uint8_t>(s);
    if (last)
      for (uint32_t i = p.row_blocks; i < p.scale_cols; ++i) at[i - p.row_blocks + 1] = 0;
  }
}

template <typename Elem, int FMT>
__global__ __launch_bounds__(kMxBlock) void mx_dequantize_kernel(MxArgs p, const uint8_t* codes,
                                                                 const uint8_t* scales, Elem* dst) {
  const int64_t c = static_cast<int64_t>(blockIdx.x) * kMxBlock + threadIdx.x;
  if (c >= p.chunks) return;
  uint2 q = make_uint2(0, 0);
  if constexpr (FMT == MOE_MX_FP4)
    q.x = reinterpret_cast<const uint32_t*>(codes)[c];
  else
    q = reinterpret_cast<const uint2*>(codes)[c];
  bool last;
  const uint32_t s = scales[scale_at(p, static_cast<uint32_t>(c >> 2), last)];
  float v[8];
  mx_decode8<FMT>(q, s, v);
  Row8<Elem> r;
  r.set(v);
  r.store(dst + c * 8);
}

MxArgs mx_args(int64_t rows, int cols) {
  return {rows * cols / 8, static_cast<uint32_t>(cols / 32),
          static_cast<uint32_t>(mx_scale_cols(cols))};
}

dim3 mx_grid(const MxArgs& a) {
  return dim3(static_cast<unsigned>((a.chunks + kMxBlock - 1) / kMxBlock));
}

}  // namespace

hipError_t launch_mx_quantize(int fmt, int dtype, int64_t rows, int cols, const void* src,
                              void* codes, uint8_t* scales, hipStream_t s, KernelTimer* tm) {
  TimedScope ts(tm, MOE_K_MX_QUANTIZE, s);
  const MxArgs a = mx_args(rows, cols);
  return by_type(dtype, [&](auto tag) {
    return by_format(fmt, [&](auto f) {
      using Elem = decltype(tag);
      hipLaunchKernelGGL((mx_quantize_kernel<Elem, decltype(f)::value>), mx_grid(a),
                         dim3(kMxBlock), 0, s, a, static_cast<const Elem*>(src),
                         static_cast<uint8_t*>(codes), scales);
      return hipGetLastError();
    });
  });
}

hipError_t launch_mx_dequantize(int fmt, int dtype, int64_t rows, int cols, const void* codes,
                                const uint8_t* scales, void* dst, hipStream_t s, KernelTimer* tm) {
  TimedScope ts(tm, MOE_K_MX_DEQUANTIZE, s);
  const MxArgs a = mx_args(rows, cols);
  return by_type(dtype, [&](auto tag) {
    return by_format(fmt, [&](auto f) {
      using Elem = decltype(tag);
      hipLaunchKernelGGL((mx_dequantize_kernel<Elem, decltype(f)::value>), mx_grid(a),
                         dim3(kMxBlock), 0, s, a, static_cast<const uint8_t*>(codes), scales,
                         static_cast<Elem*>(dst));
      return hipGetLastError();
    });
  });
}

}  // namespace moe
