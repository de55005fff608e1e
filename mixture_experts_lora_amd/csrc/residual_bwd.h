// Backward of the residual operator (residual.hip has the formulas): the row kernel and the sums
// over its blocks, instantiated for one storage type by each residual_bwd_*.hip.
#pragma once

#include <algorithm>
#include <type_traits>

#include "colsum.h"
#include "dropout.h"
#include "residual.h"
#include "row8.h"

namespace moe {

namespace {

// Column sums that a launch forms; `slot` of the partials [group][slot][H].
enum ColSum { CS_W_PRE = 0, CS_B_PRE = 1, CS_W_POST = 2, CS_B_POST = 3, CS_GATE = 4, CS_COUNT = 5 };

// TPR threads walk every so many-th row and keep the column sums of their rows (dw, db and a
// channel gate's gradient) in registers, float32, in row order; the four waves of a block whose
// rows belong to a wave add theirs in LDS, and the blocks' partials are added by
// residual_colsum_kernel in block order, so results are the same run to run. YPATH: a post norm
// or a gate is there, so y is read. LAYER: either norm is a layer norm (the sums of d and of db
// exist). GATE: the gate. What a variant does not have takes none of its registers, and they
// decide how many rows are in flight on a CU.
//
// Vector instructions cost nearly as much as the memory: with sums of 8192 x 7168 rows, both norms,
// a gate and dropout, 65 an element take 100 of 170 us. So norms are one fused multiply-add an
// element (uhat = u rstd - mean rstd), constants along a row are folded, and what a row's second
// pass needs is kept from the first (now 158.7 us, where a large copy takes 138; 8192 x 2880 bf16
// with one norm: 49.1 us, a copy 46).
template <typename Elem, int TPR, int CH, bool YPATH, bool LAYER, int GATE>
__global__ __launch_bounds__(row_block<TPR>()) void residual_bwd_kernel(ResidualBwdArgs q) {
  const ResidualArgs& p = q.f;
  constexpr int BLOCK = row_block<TPR>();
  __shared__ float slots[2][2 * (TPR / kWave)];
  const int lane = row_lane<TPR>();
  constexpr int R = BLOCK / TPR;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * R + row_in_block<TPR>();
  const int64_t stride = q.groups * R;
  RowSum<TPR> sum{slots, 0};
  const int cpr = p.H / 8;
  const bool pre = p.pre != MOE_NORM_NONE, post = YPATH && p.post != MOE_NORM_NONE;
  const bool dropout = p.drop.thr != 0;
  static_assert(YPATH || GATE == MOE_GATE_NONE, "a gate's gradient reads y");
  const DropKey key = drop_key(p.drop);
  // alpha and the kept elements' scale
  const float as = p.alpha * p.drop.scale;

  float a_wpre[CH][8], a_bpre[CH][8], a_wpost[CH][8], a_bpost[CH][8], a_gate[CH][8];
  // The vectors along H, as they are applied (shift + w, the gate's value; 0 past the row, whose
  // lanes then add nothing to a row's sums), or where those would not fit the registers (PACKED)
  // as they are stored. (For float32 that saves nothing: there the channel gate's variants at 896 and
  // 1024 threads spill 20 to 72 bytes a lane, the full gate's at 896 with a layer norm 12. No 16-bit
  // variant of one chunk spills.)
  constexpr bool PACKED = CH == 1 && TPR >= 896 && YPATH && LAYER;
  constexpr int NV = 4;  // w_pre, w_post, b_post, a channel gate
  float held[PACKED ? 1 : NV][CH][8];
  Row8<Elem> stored[PACKED ? NV : 1][CH];
  float add[CH];
  const int rb = p.H * static_cast<int>(sizeof(Elem));
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = lane + i * TPR;
    add[i] = c < cpr ? p.shift : 0.f;
    const void* from[NV] = {pre ? p.w_pre : nullptr, post ? p.w_post : nullptr,
                            post ? p.b_post : nullptr,
                            GATE == MOE_GATE_CHANNEL ? p.gate : nullptr};
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      Row8<Elem> r;
      r.load(row_buf(from[k], 0, rb), c);
      if constexpr (PACKED) stored[k][i] = r;
      else r.get(held[k][i]);
    }
    if constexpr (!PACKED) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        held[0][i][j] += add[i];
        held[1][i][j] += add[i];
        held[3][i][j] = gate_value(held[3][i][j], p.gate_sigmoid);
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
      a_wpre[i][j] = a_bpre[i][j] = a_wpost[i][j] = a_bpost[i][j] = a_gate[i][j] = 0.f;
  }
  auto vec = [&](auto kc, int i, float (&out)[8]) __attribute__((always_inline)) {
    constexpr int k = decltype(kc)::value;
    if constexpr (PACKED) {
      stored[k][i].opaque();  // unpacked here each time, not once before the rows
      stored[k][i].get(out);
      if (k < 2) {
#pragma unroll
        for (int j = 0; j < 8; ++j) out[j] += add[i];
      }
      if (k == 3) {
#pragma unroll
        for (int j = 0; j < 8; ++j) out[j] = gate_value(out[j], p.gate_sigmoid);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) out[j] = held[k][i][j];
    }
  };
  using std::integral_constant;

  // The next row is loaded while this one is reduced. Blocks of over 256 threads have registers
  // left for only what a row needs first, dx' and h' (the rest arrives during the first reduction),
  // and those with the most sums, or two chunks a thread, for nothing.
  constexpr bool AHEAD = CH == 1 && !PACKED, AHEAD_ALL = AHEAD && TPR <= 256;
  Row8<Elem> nd[CH], nx[CH], nh[CH], ny[CH];
  float4 nst = make_float4(0.f, 0.f, 0.f, 0.f);
  auto fetch_first = [&](int64_t row) __attribute__((always_inline)) {
    const bool there = row < p.T;
    const auto bx = row_buf(q.dx_out, row, rb, there && pre);
    const auto bh = row_buf(q.h_out, row, rb, there && pre);
    const auto bs = row_buf(p.stats, row, 16, there);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      nx[i].load(bx, lane + i * TPR);
      nh[i].load(bh, lane + i * TPR);
    }
    nst = __builtin_bit_cast(float4, buf_load(bs, 0));
  };
  auto fetch_rest = [&](int64_t row) __attribute__((always_inline)) {
    const bool there = row < p.T;
    const auto bd = row_buf(q.dh_out, row, rb, there);
    const auto by = row_buf(p.y, row, rb, there && YPATH);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      nd[i].load(bd, lane + i * TPR);
      if (YPATH) ny[i].load(by, lane + i * TPR);
    }
  };
  if (AHEAD) fetch_first(first);
  if (AHEAD_ALL) fetch_rest(first);
  for (int64_t row = first; row < p.T; row += stride) {
    if (!AHEAD) fetch_first(row);
    if (!AHEAD_ALL) fetch_rest(row);
    Row8<Elem> rd[CH], rx[CH], rh[CH], ry[CH], rg[CH];
    if (GATE == MOE_GATE_FULL) {
      const auto bg = row_buf(p.gate, row, rb);
#pragma unroll
      for (int i = 0; i < CH; ++i) rg[i].load(bg, lane + i * TPR);
    }
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      rd[i] = nd[i];
      rx[i] = nx[i];
      rh[i] = nh[i];
      if (YPATH) ry[i] = ny[i];
    }
    const float4 st = nst;
    if (AHEAD) fetch_first(row + stride);
    if (AHEAD_ALL) fetch_rest(row + stride);
    // the mask needs nothing from memory: drawn while the row arrives
    uint4 rnd[CH];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      rnd[i] = make_uint4(0, 0, 0, 0);
      if (dropout) rnd[i] = philox(key, static_cast<uint64_t>(row * cpr + lane + i * TPR));
    }
    // D: the gradient at h', kept in float32 for the y path; dh is its rounded copy
    float D[CH][8];
    if (pre) {
      float hat[CH][8], d[CH][8], s1 = 0.f, s2 = 0.f;
      const float off = -st.z * st.w;
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        float x[8], h[8], w[8];
        rx[i].get(x);
        rh[i].get(h);
        vec(integral_constant<int, 0>(), i, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          hat[i][j] = LAYER ? fmaf(h[j], st.w, off) : h[j] * st.w;
          d[i][j] = x[j] * w[j];
          a_wpre[i][j] = fmaf(x[j], hat[i][j], a_wpre[i][j]);
          s1 = fmaf(d[i][j], hat[i][j], s1);
          if (LAYER) {
            a_bpre[i][j] += x[j];
            s2 += d[i][j];
          }
        }
      }
      const float2 m = sum(s1, s2);
      // rstd (d - mean(d) - uhat mean(d uhat))
      const float c1 = -st.w * p.inv_h * m.x;
      const float c0 = LAYER && p.pre == MOE_NORM_LAYER ? -st.w * p.inv_h * m.y : 0.f;
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        rd[i].get(D[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float t = fmaf(hat[i][j], c1, D[i][j]);
          if (LAYER) t += c0;
          D[i][j] = fmaf(d[i][j], st.w, t);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < CH; ++i) rd[i].get(D[i]);
    }
    const auto bdh = row_buf(q.dh, row, rb);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      Row8<Elem> o;
      o.set(D[i]);
      o.store(bdh, lane + i * TPR);
    }
    if (!q.dy && !YPATH) continue;
    float gt = 1.f, slope = 1.f;
    if (GATE == MOE_GATE_TOKEN) {
      gt = to_f32<Elem>(static_cast<const Elem*>(p.gate)[row]);
      if (p.gate_sigmoid) slope = gate_slope(gt, gt);
    }
    // u: yhat (y itself without a post norm); e, the gradient at v, takes D's place
    float u[CH][8], s1 = 0.f, s2 = 0.f, sg = 0.f;
    const float off = -st.x * st.y;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = lane + i * TPR;
      float f[8];  // alpha drop(D)
      if (dropout) {
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = kept(p.drop, rnd[i], j) ? D[i][j] * as : 0.f;
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = D[i][j] * as;
      }
      if (YPATH) {
        ry[i].get(u[i]);
        float v[8], w[8], b[8];
        vec(integral_constant<int, 1>(), i, w);
        if (LAYER && GATE != MOE_GATE_NONE) vec(integral_constant<int, 2>(), i, b);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (post) u[i][j] = LAYER ? fmaf(u[i][j], st.y, off) : u[i][j] * st.y;
          if (GATE != MOE_GATE_NONE)
            v[j] = post ? (LAYER ? fmaf(u[i][j], w[j], b[j]) : u[i][j] * w[j]) : u[i][j];
        }
        if (GATE != MOE_GATE_NONE) {
          // alpha drop(v) D: the gate's gradient before its sum and its sigmoid's slope
#pragma unroll
          for (int j = 0; j < 8; ++j)
            v[j] = !dropout || kept(p.drop, rnd[i], j) ? v[j] * f[j] : 0.f;
        }
        if (GATE == MOE_GATE_CHANNEL) {
          float g[8];
          vec(integral_constant<int, 3>(), i, g);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            a_gate[i][j] += v[j];
            f[j] *= g[j];
          }
        } else if (GATE == MOE_GATE_TOKEN) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            sg += c < cpr ? v[j] : 0.f;
            f[j] *= gt;
          }
        } else if (GATE == MOE_GATE_FULL) {
          float g[8];
          rg[i].get(g);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            // a dropped element is 0 whatever its gate holds, as in the forward
            if (dropout && !kept(p.drop, rnd[i], j)) g[j] = 0.f;
            if (p.gate_sigmoid) v[j] *= gate_slope(g[j], g[j]);
            f[j] *= g[j];
          }
          Row8<Elem> o;
          o.set(v);
          o.store(row_buf(q.dgate, row, rb), c);
        }
        if (post) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            a_wpost[i][j] = fmaf(f[j], u[i][j], a_wpost[i][j]);
            if (LAYER) a_bpost[i][j] += f[j];
            f[j] *= w[j];  // d
            s1 = fmaf(f[j], u[i][j], s1);
            if (LAYER) s2 += f[j];
          }
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) D[i][j] = f[j];
    }
    if (GATE == MOE_GATE_TOKEN) {
      sg = sum(sg, 0.f).x;
      sg *= slope;
      if (lane == 0 && q.dgate) static_cast<Elem*>(q.dgate)[row] = from_f32<Elem>(sg);
    }
    if (post) {
      const float2 m = sum(s1, s2);
      const float c1 = -st.y * p.inv_h * m.x;
      const float c0 = LAYER && p.post == MOE_NORM_LAYER ? -st.y * p.inv_h * m.y : 0.f;
#pragma unroll
      for (int i = 0; i < CH; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j)
          D[i][j] = fmaf(D[i][j], st.y, LAYER ? fmaf(u[i][j], c1, c0) : u[i][j] * c1);
    }
    const auto bdy = row_buf(q.dy, row, rb);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      Row8<Elem> o;
      o.set(D[i]);
      o.store(bdy, lane + i * TPR);
    }
  }

  auto put = [&](int which, const float (&a)[CH][8]) {
    if (q.slot[which] < 0) return;
    float* out = q.part + (blockIdx.x * static_cast<int64_t>(q.nslots) + q.slot[which]) * p.H;
    if constexpr (R == 1) {
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const int c = lane + i * TPR;
        Row8<float> o;
        o.set(a[i]);
        if (c < cpr) o.store(out + 8 * c);
      }
    } else {
      static_assert(R == 1 || (R == 4 && CH == 1), "four waves of one chunk a lane");
      __shared__ float share[R == 1 ? 1 : 4][R == 1 ? 1 : 512];
      __syncthreads();  // the previous column sum is read
      Row8<float> o;
      o.set(a[0]);
      o.store(&share[threadIdx.x / TPR][8 * lane]);
      __syncthreads();
      for (int c = threadIdx.x; c < p.H; c += BLOCK)
        out[c] = (share[0][c] + share[1][c]) + (share[2][c] + share[3][c]);
    }
  };
  put(CS_W_PRE, a_wpre);
  if constexpr (LAYER) put(CS_B_PRE, a_bpre);
  if constexpr (YPATH) put(CS_W_POST, a_wpost);
  if constexpr (YPATH && LAYER) put(CS_B_POST, a_bpost);
  if constexpr (GATE == MOE_GATE_CHANNEL) put(CS_GATE, a_gate);
}

// Adds the blocks' partials: one block per 32 columns and column sum, bound by the latency of its
// few loads and the launch (4.9 us after 8192 x 2880 rows).
template <typename Elem>
__global__ __launch_bounds__(1024) void residual_colsum_kernel(ResidualBwdArgs q) {
  __shared__ float red[128][33];
  const int slot = blockIdx.y;
  const int64_t H = q.f.H;
  int col;
  float s;
  if (!block_colsum(q.part + slot * H, q.groups, q.nslots * H, blockIdx.x * 32, q.f.H, red, col, s))
    return;
  if (slot == q.slot[CS_GATE] && q.f.gate_sigmoid) {
    float g = to_f32<Elem>(static_cast<const Elem*>(q.f.gate)[col]);
    s *= gate_slope(g, g);
  }
  void* out = nullptr;
#pragma unroll
  for (int i = 0; i < CS_COUNT; ++i)
    if (q.slot[i] == slot) out = q.colsum[i];
  static_cast<Elem*>(out)[col] = from_f32<Elem>(s);
}

template <typename Elem>
hipError_t launch_bwd(ResidualBwdArgs a, hipStream_t s) {
  const bool layer = a.f.post == MOE_NORM_LAYER || a.f.pre == MOE_NORM_LAYER;
  auto go = [&](auto ypath, auto gate) {
    return by_row_width(a.f.H, [&](auto tpr, auto ch) {
      constexpr int TPR = decltype(tpr)::value, CH = decltype(ch)::value;
      constexpr int BLOCK = row_block<TPR>();
      constexpr bool Y = decltype(ypath)::value;
      constexpr int G = decltype(gate)::value;
      auto* kern = layer ? residual_bwd_kernel<Elem, TPR, CH, Y, true, G>
                         : residual_bwd_kernel<Elem, TPR, CH, Y, false, G>;
      hipLaunchKernelGGL(kern, dim3(static_cast<unsigned>(a.groups)), dim3(BLOCK), 0, s, a);
      return hipGetLastError();
    });
  };
  using std::integral_constant;
  using Yes = std::true_type;
  hipError_t e;
  if (a.f.gate_kind == MOE_GATE_CHANNEL) e = go(Yes(), integral_constant<int, MOE_GATE_CHANNEL>());
  else if (a.f.gate_kind == MOE_GATE_TOKEN) e = go(Yes(), integral_constant<int, MOE_GATE_TOKEN>());
  else if (a.f.gate_kind == MOE_GATE_FULL) e = go(Yes(), integral_constant<int, MOE_GATE_FULL>());
  else if (a.f.post != MOE_NORM_NONE) e = go(Yes(), integral_constant<int, MOE_GATE_NONE>());
  else e = go(std::false_type(), integral_constant<int, MOE_GATE_NONE>());
  if (e != hipSuccess || a.nslots == 0) return e;
  hipLaunchKernelGGL(residual_colsum_kernel<Elem>,
                     dim3(static_cast<unsigned>((a.f.H + 31) / 32), a.nslots), dim3(1024), 0, s, a);
  return hipGetLastError();
}

}  // namespace

}  // namespace moe
