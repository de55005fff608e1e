// Eight consecutive elements of a row, the unit that the residual and linear kernels load, round
// and store, and that one dropout counter covers.
#pragma once

#include "device_common.h"
#include "moe_lora.h"

namespace moe {

// One row of a tensor as a buffer resource: accesses past its end read zeros and write nothing, and
// so does everything where the row is not there (a null tensor, a row past the last). Kernels that
// load rows ahead use it, since an access that always issues leaves the compiler's count of the
// accesses in flight exact (after a branch around one it waits for all of them).
__device__ __forceinline__ __amdgpu_buffer_rsrc_t row_buf(const void* tensor, int64_t row,
                                                          int row_bytes, bool there = true) {
  const uint64_t at = reinterpret_cast<uint64_t>(tensor) + static_cast<uint64_t>(row * row_bytes);
  const uint64_t lo = static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<uint32_t>(at)));
  const uint64_t hi =
      static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<uint32_t>(at >> 32)));
  return __builtin_amdgcn_make_buffer_rsrc(
      reinterpret_cast<void*>((hi << 32) | lo), static_cast<short>(0),
      __builtin_amdgcn_readfirstlane(there && tensor ? row_bytes : 0), 0x00020000);
}

typedef uint32_t row_u32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ uint4 buf_load(const __amdgpu_buffer_rsrc_t& b, int byte) {
  const row_u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(b, byte, 0, 0);
  return make_uint4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void buf_store(const __amdgpu_buffer_rsrc_t& b, int byte, uint4 v) {
  __builtin_amdgcn_raw_buffer_store_b128(row_u32x4{v.x, v.y, v.z, v.w}, b, byte, 0, 0);
}

// Eight consecutive elements as they are stored: 16 bytes of a 16-bit type, 32 of float.
template <typename T> struct Row8;
template <> struct Row8<bf16_t> {
  uint4 a;
  __device__ void load(const bf16_t* p) { a = *reinterpret_cast<const uint4*>(p); }
  // what is computed from this value after here is not computed before
  __device__ void opaque() { asm volatile("" : "+v"(a.x), "+v"(a.y), "+v"(a.z), "+v"(a.w)); }
  __device__ void store(bf16_t* p) const { *reinterpret_cast<uint4*>(p) = a; }
  // chunk c (elements 8c ..) of a row
  __device__ void load(const __amdgpu_buffer_rsrc_t& b, int c) { a = buf_load(b, 16 * c); }
  __device__ void store(const __amdgpu_buffer_rsrc_t& b, int c) const { buf_store(b, 16 * c, a); }
  __device__ void zero() { a = make_uint4(0, 0, 0, 0); }
  __device__ void get(float (&v)[8]) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  __device__ void set(const float (&v)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = static_cast<uint32_t>(f32_to_bf16(v[2 * i])) |
             (static_cast<uint32_t>(f32_to_bf16(v[2 * i + 1])) << 16);
    a = make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <> struct Row8<f16_t> {
  uint4 a;
  __device__ void load(const f16_t* p) { a = *reinterpret_cast<const uint4*>(p); }
  // what is computed from this value after here is not computed before
  __device__ void opaque() { asm volatile("" : "+v"(a.x), "+v"(a.y), "+v"(a.z), "+v"(a.w)); }
  __device__ void store(f16_t* p) const { *reinterpret_cast<uint4*>(p) = a; }
  // chunk c (elements 8c ..) of a row
  __device__ void load(const __amdgpu_buffer_rsrc_t& b, int c) { a = buf_load(b, 16 * c); }
  __device__ void store(const __amdgpu_buffer_rsrc_t& b, int c) const { buf_store(b, 16 * c, a); }
  __device__ void zero() { a = make_uint4(0, 0, 0, 0); }
  __device__ void get(float (&v)[8]) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = static_cast<float>(__builtin_bit_cast(f16_t, static_cast<uint16_t>(w[i])));
      v[2 * i + 1] =
          static_cast<float>(__builtin_bit_cast(f16_t, static_cast<uint16_t>(w[i] >> 16)));
    }
  }
  __device__ void set(const float (&v)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = static_cast<uint32_t>(__builtin_bit_cast(uint16_t, static_cast<f16_t>(v[2 * i]))) |
             (static_cast<uint32_t>(__builtin_bit_cast(uint16_t, static_cast<f16_t>(v[2 * i + 1])))
              << 16);
    a = make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <> struct Row8<float> {
  float4 a, b;
  __device__ void opaque() {}  // nothing is unpacked
  __device__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ void store(float* p) const {
    reinterpret_cast<float4*>(p)[0] = a;
    reinterpret_cast<float4*>(p)[1] = b;
  }
  __device__ void load(const __amdgpu_buffer_rsrc_t& r, int c) {
    a = __builtin_bit_cast(float4, buf_load(r, 32 * c));
    b = __builtin_bit_cast(float4, buf_load(r, 32 * c + 16));
  }
  __device__ void store(const __amdgpu_buffer_rsrc_t& r, int c) const {
    buf_store(r, 32 * c, __builtin_bit_cast(uint4, a));
    buf_store(r, 32 * c + 16, __builtin_bit_cast(uint4, b));
  }
  __device__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ void get(float (&v)[8]) const {
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
  __device__ void set(const float (&v)[8]) {
    a = make_float4(v[0], v[1], v[2], v[3]);
    b = make_float4(v[4], v[5], v[6], v[7]);
  }
};

// Calls go with a value of the storage type of `dtype`.
template <typename F>
hipError_t by_type(int dtype, F&& go) {
  if (dtype == MOE_BF16) return go(bf16_t{});
  if (dtype == MOE_F16) return go(f16_t{});
  return go(float{});
}

}  // namespace moe
