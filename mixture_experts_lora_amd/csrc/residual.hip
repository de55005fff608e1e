// The residual stream around a block: element-wise dropout, and the fused residual operator
//
//   forward   v  = post(y)                     post, pre: none, RMS norm or layer norm
//             h' = h + alpha g drop(v)         g: 1, or a gate per channel, token or element
//             x' = pre(h')                     h' as it is stored (rounded to the layer dtype)
//   backward  D  = dh' + J_pre(h')^T dx'       the gradient at h'; dh = D
//             dg = alpha drop(v) D             summed over the gate's broadcast axis
//             e  = alpha g drop(D)             the gradient at v, under the same mask
//             dy = J_post(y)^T e
//
// A norm is n(u) = (shift + w) uhat + b with uhat = (u - mean) rstd (mean = 0 for RMS, b = 0 and
// none for RMS), rstd = 1 / sqrt(mean((u - mean)^2) + eps), and with d = (shift + w) dn its input
// gradient is rstd (d - mean(d) - uhat mean(d uhat)) (no mean(d) for RMS); dw = sum_t dn uhat,
// db = sum_t dn.
//
// Both directions are bound by HBM: they move each row once and hold it in registers between the
// reductions. All sums, means and the stored statistics are float32. A variance is the mean
// square about the mean already found (the row is at hand), not a difference of moments.
#include <algorithm>
#include <type_traits>

#include "dropout.h"
#include "launch.h"
#include "row8.h"

namespace moe {

namespace {

// ------------------------------------------------------------------ element-wise dropout
// One thread per 8 elements (one counter); VEC: both pointers on a 16-byte boundary. src and dst
// may be the same buffer: a thread reads its elements before it writes them.
template <typename Elem, bool VEC>
__global__ __launch_bounds__(256) void dropout_kernel(const Elem* src, Elem* dst, int64_t n,
                                                      DropArgs d) {
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x, i = c * 8;
  if (i >= n) return;
  const DropKey key = drop_key(d);
  Row8<Elem> r;
  const bool whole = VEC && i + 8 <= n;
  if (whole) r.load(src + i);
  const uint32_t bits = d.thr ? drop_bits(d, key, static_cast<uint64_t>(c)) : 0xffu;
  if (whole) {
    float v[8];
    r.get(v);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = (bits >> j) & 1u ? v[j] * d.scale : 0.f;
    r.set(v);
    r.store(dst + i);
  } else {
    const int m = static_cast<int>(n - i < 8 ? n - i : 8);
    for (int j = 0; j < m; ++j)
      dst[i + j] = from_f32<Elem>((bits >> j) & 1u ? to_f32<Elem>(src[i + j]) * d.scale : 0.f);
  }
}

// ------------------------------------------------------------------ reductions over a row
// A row belongs to TPR threads: one wave, or a whole block of TPR / 64 waves that meets in LDS
// (one barrier a reduction: two slots in turn, so a wave that is one reduction ahead writes the
// slot that nobody reads any more). Every thread gets the same sum, in a fixed order.
template <int TPR>
struct RowSum {
  static constexpr int W = TPR / kWave;
  float (*slots)[2 * W];
  int turn;
  __device__ float2 operator()(float a, float b) {
    a = wave_sum(a);
    b = wave_sum(b);
    if constexpr (W == 1) {
      return make_float2(a, b);
    } else {
      float* s = slots[turn];
      turn ^= 1;
      const int wave = threadIdx.x / kWave;
      if ((threadIdx.x & (kWave - 1)) == 0) {
        s[2 * wave] = a;
        s[2 * wave + 1] = b;
      }
      __syncthreads();
      a = b = 0.f;
#pragma unroll
      for (int i = 0; i < W; ++i) {
        a += s[2 * i];
        b += s[2 * i + 1];
      }
      return make_float2(a, b);
    }
  }
};

__device__ __forceinline__ float gate_value(float g, int sigmoid) {
  return sigmoid ? 1.0f / (1.0f + expf(-g)) : g;
}

// Statistics of a row held as CH chunks of 8 elements: chunk i of a thread is chunk
// lane + i TPR of the row (chunks past the row are skipped).
template <typename Elem, int TPR, int CH>
__device__ __forceinline__ void row_stats(const Row8<Elem> (&r)[CH], int lane, int cpr, int kind,
                                          float inv_h, float eps, RowSum<TPR>& sum, float& mean,
                                          float& rstd) {
  mean = 0.f;
  if (kind == MOE_NORM_LAYER) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      if (lane + i * TPR >= cpr) continue;
      float v[8];
      r[i].get(v);
#pragma unroll
      for (int j = 0; j < 8; ++j) s += v[j];
    }
    mean = sum(s, 0.f).x * inv_h;
  }
  float q = 0.f;
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    if (lane + i * TPR >= cpr) continue;
    float v[8];
    r[i].get(v);
#pragma unroll
    for (int j = 0; j < 8; ++j) q += (v[j] - mean) * (v[j] - mean);
  }
  rstd = 1.0f / sqrtf(sum(q, 0.f).x * inv_h + eps);
}

// (shift + w) u + b of one chunk; b may be null.
template <typename Elem>
__device__ __forceinline__ void affine(float (&u)[8], const Elem* w, const Elem* b, int col,
                                       float shift) {
  Row8<Elem> r;
  float f[8];
  r.load(w + col);
  r.get(f);
#pragma unroll
  for (int j = 0; j < 8; ++j) u[j] *= shift + f[j];
  if (b) {
    r.load(b + col);
    r.get(f);
#pragma unroll
    for (int j = 0; j < 8; ++j) u[j] += f[j];
  }
}

// ------------------------------------------------------------------ forward
// TPR threads a row, the row in CH chunks of 8 elements a thread. Reads h and y, writes h' and
// x' once; the norms' vectors come from cache. A thread reads all of its h and y before it writes
// anything, so h' may be h.
template <typename Elem, int TPR, int CH>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void residual_fwd_kernel(ResidualArgs p) {
  constexpr int BLOCK = TPR < 256 ? 256 : TPR;
  static_assert(TPR == kWave || TPR == BLOCK, "a row belongs to a wave or to a block");
  __shared__ float slots[2][2 * (TPR / kWave)];
  const int lane = threadIdx.x % TPR;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (BLOCK / TPR) + threadIdx.x / TPR;
  if (row >= p.T) return;  // whole waves; a block that owns one row never leaves early
  RowSum<TPR> sum{slots, 0};
  const int cpr = p.H / 8;
  const int64_t base = row * p.H;
  const Elem* h = static_cast<const Elem*>(p.h);
  const Elem* y = static_cast<const Elem*>(p.y);
  Row8<Elem> rh[CH], ry[CH];
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = lane + i * TPR;
    rh[i].zero();
    ry[i].zero();
    if (c < cpr) {
      if (y) ry[i].load(y + base + 8 * c);
      if (h) rh[i].load(h + base + 8 * c);
    }
  }
  float4 st = make_float4(0.f, 0.f, 0.f, 0.f);
  if (y) {
    if (p.post != MOE_NORM_NONE)
      row_stats<Elem, TPR, CH>(ry, lane, cpr, p.post, p.inv_h, p.eps, sum, st.x, st.y);
    const DropKey key = drop_key(p.drop);
    const Elem* gate = static_cast<const Elem*>(p.gate);
    float g = 1.f;
    if (p.gate_kind == MOE_GATE_TOKEN) g = gate_value(to_f32<Elem>(gate[row]), p.gate_sigmoid);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = lane + i * TPR;
      if (c >= cpr) continue;
      float v[8], u[8];
      ry[i].get(v);
      if (p.post != MOE_NORM_NONE) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = (v[j] - st.x) * st.y;
        affine<Elem>(v, static_cast<const Elem*>(p.w_post), static_cast<const Elem*>(p.b_post),
                     8 * c, p.shift);
      }
      if (p.drop.thr) {
        const uint32_t bits = drop_bits(p.drop, key, static_cast<uint64_t>(row * cpr + c));
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = (bits >> j) & 1u ? v[j] * p.drop.scale : 0.f;
      }
      if (p.gate_kind == MOE_GATE_CHANNEL || p.gate_kind == MOE_GATE_FULL) {
        Row8<Elem> rg;
        float f[8];
        rg.load(gate + (p.gate_kind == MOE_GATE_FULL ? base : 0) + 8 * c);
        rg.get(f);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] *= gate_value(f[j], p.gate_sigmoid);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] *= g;
      }
      rh[i].get(u);
#pragma unroll
      for (int j = 0; j < 8; ++j) u[j] += p.alpha * v[j];
      rh[i].set(u);
    }
  }
  if (p.h_out) {
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = lane + i * TPR;
      if (c < cpr) rh[i].store(static_cast<Elem*>(p.h_out) + base + 8 * c);
    }
  }
  if (p.pre != MOE_NORM_NONE) {
    row_stats<Elem, TPR, CH>(rh, lane, cpr, p.pre, p.inv_h, p.eps, sum, st.z, st.w);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = lane + i * TPR;
      if (c >= cpr) continue;
      float u[8];
      rh[i].get(u);
#pragma unroll
      for (int j = 0; j < 8; ++j) u[j] = (u[j] - st.z) * st.w;
      affine<Elem>(u, static_cast<const Elem*>(p.w_pre), static_cast<const Elem*>(p.b_pre), 8 * c,
                   p.shift);
      Row8<Elem> o;
      o.set(u);
      o.store(static_cast<Elem*>(p.x_out) + base + 8 * c);
    }
  }
  if (lane == 0 && p.stats) p.stats[row] = st;
}

// ------------------------------------------------------------------ backward
// Column sums that a launch forms; `slot` of the partials [group][slot][H].
enum ColSum { CS_W_PRE = 0, CS_B_PRE = 1, CS_W_POST = 2, CS_B_POST = 3, CS_GATE = 4, CS_COUNT = 5 };

// Each group of TPR threads walks the rows group, group + groups, ... and keeps the column sums
// of its rows (dw, db and a channel gate's gradient) in registers, float32, in row order; the
// groups' partials are added by residual_colsum_kernel in group order, so results are the same
// run to run. YPATH: a post norm or a gate is there, so y is read. LAYER: either norm is a layer
// norm (the sums of d and of db exist); without it their registers are not held.
template <typename Elem, int TPR, int CH, bool YPATH, bool LAYER>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void residual_bwd_kernel(ResidualBwdArgs q) {
  const ResidualArgs& p = q.f;
  constexpr int BLOCK = TPR < 256 ? 256 : TPR;
  static_assert(TPR == kWave || TPR == BLOCK, "a row belongs to a wave or to a block");
  __shared__ float slots[2][2 * (TPR / kWave)];
  const int lane = threadIdx.x % TPR;
  const int64_t group = static_cast<int64_t>(blockIdx.x) * (BLOCK / TPR) + threadIdx.x / TPR;
  if (group >= q.groups) return;
  RowSum<TPR> sum{slots, 0};
  const int cpr = p.H / 8;
  const bool pre = p.pre != MOE_NORM_NONE, post = YPATH && p.post != MOE_NORM_NONE;
  const Elem* gate = static_cast<const Elem*>(p.gate);
  const DropKey key = drop_key(p.drop);

  float a_wpre[CH][8], a_bpre[LAYER ? CH : 1][8], a_wpost[YPATH ? CH : 1][8],
      a_bpost[YPATH && LAYER ? CH : 1][8], a_gate[YPATH ? CH : 1][8];
#pragma unroll
  for (int i = 0; i < CH; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      a_wpre[i][j] = 0.f;
      if constexpr (LAYER) a_bpre[i][j] = 0.f;
      if constexpr (YPATH) a_wpost[i][j] = a_gate[i][j] = 0.f;
      if constexpr (YPATH && LAYER) a_bpost[i][j] = 0.f;
    }
  // the vectors along H stay in registers over the rows
  Row8<Elem> rwpre[CH], rwpost[YPATH ? CH : 1], rbpost[YPATH && LAYER ? CH : 1],
      rgate[YPATH ? CH : 1];
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = lane + i * TPR;
    rwpre[i].zero();
    if (pre && c < cpr) rwpre[i].load(static_cast<const Elem*>(p.w_pre) + 8 * c);
    if constexpr (YPATH) {
      rwpost[i].zero();
      rgate[i].zero();
      if (post && c < cpr) rwpost[i].load(static_cast<const Elem*>(p.w_post) + 8 * c);
      if (p.gate_kind == MOE_GATE_CHANNEL && c < cpr) rgate[i].load(gate + 8 * c);
      if constexpr (LAYER) {
        rbpost[i].zero();
        if (post && p.b_post && c < cpr)
          rbpost[i].load(static_cast<const Elem*>(p.b_post) + 8 * c);
      }
    }
  }

  for (int64_t row = group; row < p.T; row += q.groups) {
    const int64_t base = row * p.H;
    Row8<Elem> rd[CH], rx[CH], rh[CH], ry[YPATH ? CH : 1];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = lane + i * TPR;
      rd[i].zero();
      rx[i].zero();
      rh[i].zero();
      if constexpr (YPATH) ry[i].zero();
      if (c < cpr) {
        if (pre) {
          rx[i].load(static_cast<const Elem*>(q.dx_out) + base + 8 * c);
          rh[i].load(static_cast<const Elem*>(q.h_out) + base + 8 * c);
        }
        if (q.dh_out) rd[i].load(static_cast<const Elem*>(q.dh_out) + base + 8 * c);
        if constexpr (YPATH) ry[i].load(static_cast<const Elem*>(p.y) + base + 8 * c);
      }
    }
    const float4 st = p.stats ? p.stats[row] : make_float4(0.f, 0.f, 0.f, 0.f);
    float2 m = make_float2(0.f, 0.f);  // mean of d uhat, mean of d
    if (pre) {
      float s1 = 0.f, s2 = 0.f;
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        float x[8], h[8], w[8];
        rx[i].get(x);
        rh[i].get(h);
        rwpre[i].get(w);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float hat = (h[j] - st.z) * st.w, d = x[j] * (p.shift + w[j]);
          a_wpre[i][j] += x[j] * hat;
          s1 += d * hat;
          if constexpr (LAYER) {
            a_bpre[i][j] += x[j];
            s2 += d;
          }
        }
      }
      m = sum(s1, s2);
      m.x *= p.inv_h;
      m.y = LAYER && p.pre == MOE_NORM_LAYER ? m.y * p.inv_h : 0.f;
    }
    // D, kept in float32 for the y path; dh is its rounded copy
    float D[CH][8];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      rd[i].get(D[i]);
      if (pre) {
        float x[8], h[8], w[8];
        rx[i].get(x);
        rh[i].get(h);
        rwpre[i].get(w);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float hat = (h[j] - st.z) * st.w, d = x[j] * (p.shift + w[j]);
          D[i][j] += st.w * (d - m.y - hat * m.x);
        }
      }
      const int c = lane + i * TPR;
      if (q.dh && c < cpr) {
        Row8<Elem> o;
        o.set(D[i]);
        o.store(static_cast<Elem*>(q.dh) + base + 8 * c);
      }
    }
    if (!q.dy && !YPATH) continue;
    float gt = 1.f;
    if (YPATH && p.gate_kind == MOE_GATE_TOKEN)
      gt = gate_value(to_f32<Elem>(gate[row]), p.gate_sigmoid);
    float s1 = 0.f, s2 = 0.f, sg = 0.f;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = lane + i * TPR;
      if (c >= cpr) continue;
      const uint32_t bits =
          p.drop.thr ? drop_bits(p.drop, key, static_cast<uint64_t>(row * cpr + c)) : 0xffu;
      float g[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) g[j] = gt;
      if constexpr (YPATH) {
        float v[8], w[8];
        ry[i].get(v);
        rwpost[i].get(w);
        if (post) {
          float b[8] = {};
          if constexpr (LAYER) rbpost[i].get(b);
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] = (v[j] - st.x) * st.y * (p.shift + w[j]) + b[j];
        }
        // alpha drop(v) D: the gate's gradient before its sum and its sigmoid's slope
#pragma unroll
        for (int j = 0; j < 8; ++j)
          v[j] = (bits >> j) & 1u ? p.alpha * p.drop.scale * v[j] * D[i][j] : 0.f;
        if (p.gate_kind == MOE_GATE_CHANNEL) {
          rgate[i].get(g);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            g[j] = gate_value(g[j], p.gate_sigmoid);
            a_gate[i][j] += v[j];
          }
        } else if (p.gate_kind == MOE_GATE_TOKEN) {
#pragma unroll
          for (int j = 0; j < 8; ++j) sg += v[j];
        } else if (p.gate_kind == MOE_GATE_FULL) {
          Row8<Elem> r;
          r.load(gate + base + 8 * c);
          r.get(g);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            g[j] = gate_value(g[j], p.gate_sigmoid);
            if (p.gate_sigmoid) v[j] *= g[j] * (1.f - g[j]);
          }
          if (q.dgate) {
            r.set(v);
            r.store(static_cast<Elem*>(q.dgate) + base + 8 * c);
          }
        }
      }
      // e, in D's place
#pragma unroll
      for (int j = 0; j < 8; ++j)
        D[i][j] = (bits >> j) & 1u ? p.alpha * p.drop.scale * g[j] * D[i][j] : 0.f;
      if constexpr (YPATH) {
        if (post) {
          float u[8], w[8];
          ry[i].get(u);
          rwpost[i].get(w);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float hat = (u[j] - st.x) * st.y, d = D[i][j] * (p.shift + w[j]);
            a_wpost[i][j] += D[i][j] * hat;
            s1 += d * hat;
            if constexpr (LAYER) {
              a_bpost[i][j] += D[i][j];
              s2 += d;
            }
          }
        }
      }
    }
    m = make_float2(0.f, 0.f);
    if (post) {
      m = sum(s1, s2);
      m.x *= p.inv_h;
      m.y = LAYER && p.post == MOE_NORM_LAYER ? m.y * p.inv_h : 0.f;
    }
    if (YPATH && p.gate_kind == MOE_GATE_TOKEN) {
      sg = sum(sg, 0.f).x;
      if (p.gate_sigmoid) sg *= gt * (1.f - gt);
      if (lane == 0 && q.dgate) static_cast<Elem*>(q.dgate)[row] = from_f32<Elem>(sg);
    }
    if (!q.dy) continue;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = lane + i * TPR;
      if (c >= cpr) continue;
      if constexpr (YPATH) {
        if (post) {
          float u[8], w[8];
          ry[i].get(u);
          rwpost[i].get(w);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float hat = (u[j] - st.x) * st.y, d = D[i][j] * (p.shift + w[j]);
            D[i][j] = st.y * (d - m.y - hat * m.x);
          }
        }
      }
      Row8<Elem> o;
      o.set(D[i]);
      o.store(static_cast<Elem*>(q.dy) + base + 8 * c);
    }
  }

  auto put = [&](int which, const float (&a)[8], int c) {
    if (q.slot[which] < 0) return;
    Row8<float> o;
    o.set(a);
    o.store(q.part + (group * q.nslots + q.slot[which]) * p.H + 8 * c);
  };
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = lane + i * TPR;
    if (c >= cpr) continue;
    put(CS_W_PRE, a_wpre[i], c);
    if constexpr (LAYER) put(CS_B_PRE, a_bpre[i], c);
    if constexpr (YPATH) put(CS_W_POST, a_wpost[i], c);
    if constexpr (YPATH && LAYER) put(CS_B_POST, a_bpost[i], c);
    if constexpr (YPATH) put(CS_GATE, a_gate[i], c);
  }
}

// Adds the groups' partials: one block per 32 columns and column sum, 32 rows of 32 lanes that
// each walk every 32nd group; then the 32 row sums, in order.
template <typename Elem>
__global__ __launch_bounds__(1024) void residual_colsum_kernel(ResidualBwdArgs q) {
  __shared__ float red[32][33];
  const int cx = threadIdx.x & 31, ry = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + cx, slot = blockIdx.y;
  const int64_t H = q.f.H;
  float a = 0.f;
  if (col < H)
    for (int64_t g = ry; g < q.groups; g += 32) a += q.part[(g * q.nslots + slot) * H + col];
  red[ry][cx] = a;
  __syncthreads();
  if (ry != 0 || col >= H) return;
  a = 0.f;
#pragma unroll
  for (int i = 0; i < 32; ++i) a += red[i][cx];
  if (slot == q.slot[CS_GATE] && q.f.gate_sigmoid) {
    const float g = gate_value(to_f32<Elem>(static_cast<const Elem*>(q.f.gate)[col]), 1);
    a *= g * (1.f - g);
  }
  void* out = nullptr;
#pragma unroll
  for (int i = 0; i < CS_COUNT; ++i)
    if (q.slot[i] == slot) out = q.colsum[i];
  static_cast<Elem*>(out)[col] = from_f32<Elem>(a);
}

// Threads a row and chunks a thread. Forward: a wave holds rows up to 4096 wide.
template <typename F>
hipError_t by_width_fwd(int H, F&& go) {
  using std::integral_constant;
  if (H <= 512) return go(integral_constant<int, 64>(), integral_constant<int, 1>());
  if (H <= 1024) return go(integral_constant<int, 64>(), integral_constant<int, 2>());
  if (H <= 2048) return go(integral_constant<int, 64>(), integral_constant<int, 4>());
  if (H <= 4096) return go(integral_constant<int, 64>(), integral_constant<int, 8>());
  if (H <= 8192) return go(integral_constant<int, 256>(), integral_constant<int, 4>());
  return go(integral_constant<int, 512>(), integral_constant<int, 4>());
}

// Backward: at most two chunks a thread, since the column sums take 8 registers each per chunk.
template <typename F>
hipError_t by_width_bwd(int H, F&& go) {
  using std::integral_constant;
  if (H <= 512) return go(integral_constant<int, 64>(), integral_constant<int, 1>());
  if (H <= 2048) return go(integral_constant<int, 256>(), integral_constant<int, 1>());
  if (H <= 4096) return go(integral_constant<int, 256>(), integral_constant<int, 2>());
  if (H <= 8192) return go(integral_constant<int, 512>(), integral_constant<int, 2>());
  return go(integral_constant<int, 1024>(), integral_constant<int, 2>());
}

inline int bwd_threads(int H) { return H <= 512 ? 64 : H <= 4096 ? 256 : H <= 8192 ? 512 : 1024; }

}  // namespace

hipError_t launch_dropout(int dtype, int64_t n, const DropArgs& d, const void* src, void* dst,
                          hipStream_t s, KernelTimer* tm) {
  TimedScope ts(tm, MOE_K_DROPOUT, s);
  const bool vec = ((reinterpret_cast<uintptr_t>(src) | reinterpret_cast<uintptr_t>(dst)) & 15) == 0;
  const dim3 grid(static_cast<unsigned>(((n + 7) / 8 + 255) / 256));
  return by_type(dtype, [&](auto tag) {
    using Elem = decltype(tag);
    auto* kern = vec ? dropout_kernel<Elem, true> : dropout_kernel<Elem, false>;
    hipLaunchKernelGGL(kern, grid, dim3(256), 0, s, static_cast<const Elem*>(src),
                       static_cast<Elem*>(dst), n, d);
    return hipGetLastError();
  });
}

hipError_t launch_residual_fwd(int dtype, const ResidualArgs& a, hipStream_t s, KernelTimer* tm) {
  TimedScope ts(tm, MOE_K_RESIDUAL_NORM, s);
  return by_type(dtype, [&](auto tag) {
    return by_width_fwd(a.H, [&](auto tpr, auto ch) {
      constexpr int TPR = decltype(tpr)::value, BLOCK = TPR < 256 ? 256 : TPR, R = BLOCK / TPR;
      hipLaunchKernelGGL((residual_fwd_kernel<decltype(tag), TPR, decltype(ch)::value>),
                         dim3(static_cast<unsigned>((static_cast<int64_t>(a.T) + R - 1) / R)),
                         dim3(BLOCK), 0, s, a);
      return hipGetLastError();
    });
  });
}

// Four blocks' worth of threads a CU (1024) over 256 CUs: enough rows in flight, few partials.
int64_t residual_bwd_groups(int T, int H) {
  return std::min<int64_t>(T, 256 * 1024 / bwd_threads(H));
}

hipError_t launch_residual_bwd(int dtype, const ResidualBwdArgs& a, hipStream_t s,
                               KernelTimer* tm) {
  TimedScope ts(tm, MOE_K_RESIDUAL_NORM_BWD, s);
  const bool ypath = a.f.post != MOE_NORM_NONE || a.f.gate_kind != MOE_GATE_NONE;
  const bool layer = a.f.post == MOE_NORM_LAYER || a.f.pre == MOE_NORM_LAYER;
  return by_type(dtype, [&](auto tag) {
    using Elem = decltype(tag);
    hipError_t e = by_width_bwd(a.f.H, [&](auto tpr, auto ch) {
      constexpr int TPR = decltype(tpr)::value, CH = decltype(ch)::value;
      constexpr int BLOCK = TPR < 256 ? 256 : TPR, R = BLOCK / TPR;
      auto* kern = ypath ? (layer ? residual_bwd_kernel<Elem, TPR, CH, true, true>
                                  : residual_bwd_kernel<Elem, TPR, CH, true, false>)
                         : (layer ? residual_bwd_kernel<Elem, TPR, CH, false, true>
                                  : residual_bwd_kernel<Elem, TPR, CH, false, false>);
      hipLaunchKernelGGL(kern, dim3(static_cast<unsigned>((a.groups + R - 1) / R)), dim3(BLOCK), 0,
                         s, a);
      return hipGetLastError();
    });
    if (e != hipSuccess || a.nslots == 0) return e;
    hipLaunchKernelGGL(residual_colsum_kernel<Elem>,
                       dim3(static_cast<unsigned>((a.f.H + 31) / 32), a.nslots), dim3(1024), 0, s,
                       a);
    return hipGetLastError();
  });
}

}  // namespace moe
