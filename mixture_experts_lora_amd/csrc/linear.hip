// Dense linear operator of the residual stream, and its backward:
//
//   z = x w^T + bias        x [T, K], w [N, K]
//   y = residual + dropout(act(z))
//   dz = act'(z) kept(dy)      kept(dy): dy where the mask keeps it, else 0
//   dx = c dz w    dw = c dz^T x    dbias = c sum_t dz      c: the kept elements' scale
//
// dz is rounded to the layer dtype (it feeds MFMA, as the experts' dH does), dbias summed before
// that. c goes to the float32 results, so that without an activation dz is exact.
//
// Many tokens: MFMA tiles (gemm16 for the 16-bit types, linear_f32_kernel for float32) whose
// epilogue applies bias, activation, dropout and residual to the float32 product, so z and y move
// once. Where a product has too few tiles to fill the card, its reduction is cut into slices that
// are summed in slice order by a second kernel with the same epilogue: no atomics, so results are
// the same run to run. Up to 16 tokens the product is bound by reading w once, and
// linear_few_kernel streams it.
#include <algorithm>
#include <type_traits>

#include "colsum.h"
#include "gemm16.h"

namespace moe {

namespace {

#define MOE_TRY(x)                       \
  do {                                   \
    hipError_t err_ = (x);               \
    if (err_ != hipSuccess) return err_; \
  } while (0)

// ------------------------------------------------------------------ float32 product
// 128 x 128 tiles, four waves of 64 x 64, 16 deep, two LDS slots filled through registers.
// v_mfma_f32_32x32x2_f32 takes 64 cycles for 4 KFLOP, so the product is bound by MFMA and the
// plain loop below keeps it fed. LDS holds both operands as [k][mn]; a row of 132 floats puts the
// four k-quads that a k-contiguous fill writes for 16 rows on all 64 banks. (8192 x 4096 x 2880:
// 1669 us, 116 TFLOP/s.)
typedef float f32x16_t __attribute__((ext_vector_type(16)));

template <bool KC>
__device__ __forceinline__ void f32_fetch(const float* base, int64_t ld, int mn0, int mn_lim,
                                          int64_t k0, int64_t k_end, float4 (&r)[2]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int idx = threadIdx.x + i * 256;
    const int mn = mn0 + (KC ? idx / 4 : idx % 32 * 4);
    const int64_t k = k0 + (KC ? idx % 4 * 4 : idx / 32);
    r[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (mn < mn_lim && k < k_end)
      r[i] = *reinterpret_cast<const float4*>(base + (KC ? mn * ld + k : k * ld + mn));
  }
}

template <bool KC>
__device__ __forceinline__ void f32_put(float (&s)[16][132], const float4 (&r)[2]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int idx = threadIdx.x + i * 256;
    if (KC) {
      const int mn = idx / 4, k = idx % 4 * 4;
      s[k][mn] = r[i].x;
      s[k + 1][mn] = r[i].y;
      s[k + 2][mn] = r[i].z;
      s[k + 3][mn] = r[i].w;
    } else {
      *reinterpret_cast<float4*>(&s[idx / 32][idx % 32 * 4]) = r[i];
    }
  }
}

// out(m, n) = sum_k a(m, k) b(n, k) over the block's slice; M, N, K[0], kchunk, E, lin and out as
// EPI_LINEAR's. EPI: the output goes through linear_finish8, otherwise it is stored.
template <bool A_KC, bool B_KC, bool EPI>
__global__ __launch_bounds__(256, 2) void linear_f32_kernel(GemmArgs p) {
  constexpr int WN = 64;
  union Smem {
    float tile[2][2][16][132];
    char slab[4][32 * WN * 4];
  };
  __shared__ __attribute__((aligned(1024))) Smem sm;
  int e, n_tile, m0;
  if (!dense_tile(p, 128, e, n_tile, m0)) return;
  const int n0 = n_tile * 128, lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wm = wave >> 1, wn = wave & 1;
  const int64_t kbeg = static_cast<int64_t>(e) * p.kchunk;
  const int64_t kend = min(kbeg + p.kchunk, static_cast<int64_t>(p.K[0]));
  const float* A = static_cast<const float*>(p.a[0].ptr);
  const float* B = static_cast<const float*>(p.b[0].ptr);
  f32x16 acc[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;
  float4 ra[2], rb[2];
  f32_fetch<A_KC>(A, p.a[0].ld, m0, p.M, kbeg, kend, ra);
  f32_fetch<B_KC>(B, p.b[0].ld, n0, p.N, kbeg, kend, rb);
  f32_put<A_KC>(sm.tile[0][0], ra);
  f32_put<B_KC>(sm.tile[0][1], rb);
  __syncthreads();
  int slot = 0;
  for (int64_t k0 = kbeg; k0 < kend; k0 += 16) {
    const bool more = k0 + 16 < kend;
    if (more) {
      f32_fetch<A_KC>(A, p.a[0].ld, m0, p.M, k0 + 16, kend, ra);
      f32_fetch<B_KC>(B, p.b[0].ld, n0, p.N, k0 + 16, kend, rb);
    }
    const auto& sa = sm.tile[slot][0];
    const auto& sb = sm.tile[slot][1];
#pragma unroll
    for (int s = 0; s < 8; ++s) {
      float fa[2], fb[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        fa[i] = sa[2 * s + (lane >> 5)][wm * 64 + i * 32 + (lane & 31)];
        fb[i] = sb[2 * s + (lane >> 5)][wn * 64 + i * 32 + (lane & 31)];
      }
      // b as the MFMA's A operand: a lane ends with consecutive columns of one row
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x2f32(fb[j], fa[i], acc[i][j], 0, 0, 0);
    }
    slot ^= 1;
    if (more) {
      // the other slot was last read before the previous barrier
      f32_put<A_KC>(sm.tile[slot][0], ra);
      f32_put<B_KC>(sm.tile[slot][1], rb);
    }
    __syncthreads();
  }
  char* slab = sm.slab[wave];
#pragma unroll
  for (int mi = 0; mi < 2; ++mi) {
    if (mi) wave_lds_sync();
#pragma unroll
    for (int ni = 0; ni < 2; ++ni)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        f32x4 v;
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = acc[mi][ni][4 * q + j];
        *reinterpret_cast<f32x4*>(slab + slab_off<WN>(lane & 31, ni * 8 + 2 * q + (lane >> 5))) = v;
      }
    wave_lds_sync();
#pragma unroll
    for (int pass = 0; pass < 4; ++pass) {
      const int r = pass * 8 + lane / 8, s = lane % 8;
      const int row = m0 + wm * 64 + mi * 32 + r, col = n0 + wn * 64 + 8 * s;
      float v[8];
      read8_interleaved<WN>(slab, r, s, v);
      if (row >= p.M || col >= p.N) continue;
      if (EPI && p.E == 1) {
        linear_finish8<float>(p.lin, row, col, p.N, v);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] *= p.scale;
        Row8<float> o;
        o.set(v);
        o.store(static_cast<float*>(p.out) + (static_cast<int64_t>(e) * p.M + row) * p.N + col);
      }
    }
  }
}

// ------------------------------------------------------------------ sums over slices
// The slices' partials [E][M][N] in slice order, then the epilogue: eight columns a thread. Bound
// by reading the partials; plan() charges them at 4 TB/s, written and read, and the launch at 5 us.
template <typename Elem>
__global__ __launch_bounds__(256) void linear_sum_kernel(const float* __restrict__ part, int E,
                                                         int64_t MN, int N, LinearEpi epi) {
  const int64_t i = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 8;
  if (i >= MN) return;
  float v[8] = {};
#pragma unroll 4
  for (int e = 0; e < E; ++e) {
    Row8<float> r;
    float f[8];
    r.load(part + e * MN + i);
    r.get(f);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] += f[j];
  }
  const int64_t row = i / N;
  linear_finish8<Elem>(epi, row, static_cast<int>(i - row * N), N, v);
}

// ------------------------------------------------------------------ few tokens
// Bound by reading w once.
//
// One or two tokens: a block owns eight columns (eight rows of w) and its four waves split K in
// 16-byte pieces a lane, so each wave reads 1 KB of a row an instruction with eight rows in flight;
// x comes from cache. (7168 x 7168 bf16, one token: 21.1 us, 4.9 TB/s; by MFMA fragments, 16 rows
// of 64 bytes an instruction, 25.4 us.)
template <typename Elem, int TT>
__global__ __launch_bounds__(256) void linear_one_kernel(const Elem* __restrict__ x,
                                                         const Elem* __restrict__ w, int T, int K,
                                                         int N, LinearEpi epi) {
  __shared__ float red[4][TT * 8];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, n0 = blockIdx.x * 8;
  float acc[8][TT];
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int t = 0; t < TT; ++t) acc[i][t] = 0.f;
  for (int k = threadIdx.x * 8; k < K; k += 256 * 8) {
    Row8<Elem> rw[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) rw[i].load(w + static_cast<int64_t>(n0 + i) * K + k);
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      if (t >= T) continue;
      Row8<Elem> rx;
      float fx[8];
      rx.load(x + static_cast<int64_t>(t) * K + k);
      rx.get(fx);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float fw[8];
        rw[i].get(fw);
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[i][t] += fx[j] * fw[j];
      }
    }
  }
#pragma unroll
  for (int t = 0; t < TT; ++t)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float s = wave_sum(acc[i][t]);
      if (lane == 0) red[wave][t * 8 + i] = s;
    }
  __syncthreads();
  const int t = threadIdx.x;
  if (t >= T) return;
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    v[i] = (red[0][t * 8 + i] + red[1][t * 8 + i]) + (red[2][t * 8 + i] + red[3][t * 8 + i]);
  linear_finish8<Elem>(epi, t, n0, N, v);
}

// Up to 16 tokens, where fused multiply-adds would bound the kernel above (16 tokens, 4096 x 2880:
// 27.4 us, by MFMA 10.2): a block owns 16 columns and its eight waves deal out the reduction in
// pieces of 16 bytes x 8 steps a lane, straight into MFMA fragments: 16 rows of 64 bytes for w (the
// MFMA's A operand, so that a lane ends with four consecutive columns of a token) and for x, which
// comes from L2. Accesses past an operand read zeros. The waves' sums meet in LDS in wave order.
template <typename Elem> struct Few;
template <> struct Few<bf16_t> {
  static constexpr int KSTEP = 32;
  __device__ static f32x4 mul(const uint4& a, const uint4& b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  }
};
template <> struct Few<f16_t> {
  static constexpr int KSTEP = 32;
  typedef f16_t h8 __attribute__((ext_vector_type(8)));
  __device__ static f32x4 mul(const uint4& a, const uint4& b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8, a),
                                                  __builtin_bit_cast(h8, b), c, 0, 0, 0);
  }
};
// The four floats of a lane go through four products whose k are {j, 4 + j, 8 + j, 12 + j}.
template <> struct Few<float> {
  static constexpr int KSTEP = 16;
  __device__ static f32x4 mul(const uint4& a, const uint4& b, f32x4 c) {
    const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int j = 0; j < 4; ++j)
      c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(x[j]), __uint_as_float(y[j]), c, 0,
                                               0, 0);
    return c;
  }
};

template <typename Elem>
__global__ __launch_bounds__(512) void linear_few_kernel(const Elem* __restrict__ x,
                                                         const Elem* __restrict__ w, int T, int K,
                                                         int N, LinearEpi epi) {
  typedef Few<Elem> F;
  constexpr int ES = sizeof(Elem), STEPS = 8;
  __shared__ __attribute__((aligned(16))) float red[8][16][20];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n0 = blockIdx.x * 16, row = lane & 15, kl = (lane >> 4) * (16 / ES);
  const int kb = K * ES;  // bytes of a row
  const auto bw = row_buf(w + static_cast<int64_t>(n0) * K, 0, min(N - n0, 16) * kb);
  const auto bx = row_buf(x, 0, T * kb);
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  for (int k0 = wave * F::KSTEP * STEPS; k0 < K; k0 += 8 * F::KSTEP * STEPS) {
    uint4 fw[STEPS], fx[STEPS];
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      const int k = k0 + s * F::KSTEP + kl;
      // K is a multiple of 8: the 16 bytes are all in or all out
      const int at = k < K ? row * kb + k * ES : static_cast<int>(kOOB);
      fw[s] = buf_load(bw, at);
      fx[s] = buf_load(bx, at);
    }
#pragma unroll
    for (int s = 0; s < STEPS; ++s) acc = F::mul(fw[s], fx[s], acc);
  }
  // lane: token lane % 16, columns 4 (lane / 16) .. + 3
  *reinterpret_cast<f32x4*>(&red[wave][row][(lane >> 4) * 4]) = acc;
  __syncthreads();
  const int t = threadIdx.x >> 1, half = threadIdx.x & 1, col = n0 + half * 8;
  if (t >= T || col >= N) return;
  float v[8] = {};
#pragma unroll
  for (int q = 0; q < 8; ++q)
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] += red[q][t][half * 8 + j];
  linear_finish8<Elem>(epi, t, col, N, v);
}

// ------------------------------------------------------------------ dz and dbias
// 512 columns a block, its four waves on different rows, two rows of a wave in flight at once; rows
// are dealt to gridDim.y groups whose column sums (float32, in row order) linear_colsum_kernel adds.
// dz null: only the sums. Bound by HBM (8192 x 2880 bf16, gelu: 27.6 us, 5.1 TB/s; its column
// sums' second kernel 4.8 us).
template <typename Elem>
__global__ __launch_bounds__(256) void linear_dz_kernel(const Elem* __restrict__ dy, int T, int N,
                                                        LinearEpi epi, Elem* __restrict__ dz,
                                                        float* __restrict__ part) {
  constexpr int U = 2;
  __shared__ float red[4][512 + 8];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int chunk = blockIdx.x * 64 + lane, rb = N * static_cast<int>(sizeof(Elem));
  const DropKey key = drop_key(epi.drop);
  const bool act = epi.act != MOE_ACT_NONE;
  float sum[8] = {};
  for (int64_t t0 = blockIdx.y * 4 * U + wave; t0 < T; t0 += gridDim.y * 4 * U) {
    Row8<Elem> r[U], rz[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t t = t0 + 4 * u;
      r[u].load(row_buf(dy, t, rb, t < T), chunk);
      rz[u].load(row_buf(epi.pre, t, rb, act && t < T), chunk);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t t = t0 + 4 * u;
      float v[8];
      r[u].get(v);
      if (act) {
        float z[8];
        rz[u].get(z);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] *= act_slope<Elem>(z[j], epi.act);
      }
      // last, so that a dropped element is 0 whatever z holds, as in the forward
      if (epi.drop.thr) {
        const uint4 rnd = philox(key, static_cast<uint64_t>(t * (N / 8) + chunk));
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = kept(epi.drop, rnd, j) ? v[j] : 0.f;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) sum[j] += v[j];
      r[u].set(v);
      r[u].store(row_buf(dz, t, rb, t < T), chunk);
    }
  }
  if (!part) return;
#pragma unroll
  for (int j = 0; j < 8; ++j) red[wave][lane * 8 + j] = sum[j];
  __syncthreads();
  for (int c = threadIdx.x; c < 512; c += 256) {
    const int n = blockIdx.x * 512 + c;
    if (n < N)
      part[static_cast<int64_t>(blockIdx.y) * N + n] =
          epi.drop.scale * ((red[0][c] + red[1][c]) + (red[2][c] + red[3][c]));
  }
}

template <typename Elem>
__global__ __launch_bounds__(1024) void linear_colsum_kernel(const float* part, int groups, int N,
                                                             Elem* db) {
  __shared__ float red[128][33];
  int col;
  float s;
  if (block_colsum(part, groups, N, blockIdx.x * 32, N, red, col, s)) db[col] = from_f32<Elem>(s);
}

// ------------------------------------------------------------------ host side
constexpr int kFewTokens = 16;

// One product of M x N outputs over K: tile shape, and slices of the reduction.
enum Tile { TILE_256x256, TILE_256x192, TILE_192x192, TILE_128x128, TILE_128x64, TILE_64x64, TILE_128x256, TILE_F32 };
struct Product {
  Tile tile;
  int bm, bn, ntm, ntn, E, kchunk;
  size_t part_bytes;  // 0: one slice, no partials
};

// The plan of least estimated time: the tiles of the busiest CU at the rate a CU reaches with them
// and what a tile cannot overlap, plus the slices' partials written and read and the launch that
// sums them. `few`: the least number of tiles whose time a CU takes (tiles of four waves keep a CU
// busy by twos). Fitted to launches of 8192 x 4096 x 2880 (full CUs) and of 64 to 2048 tokens; the
// plans it gives 300 and 1000 tokens of that product take 23.6 and 43 us, 128 x 64 tiles 28.5 and 56.
struct TileModel {
  Tile tile;
  int bm, bn;
  double tflops, few, over_us;  // per CU
};
constexpr TileModel kRows16[] = {{TILE_256x256, 256, 256, 4.2, 1.0, 3.0},
                                 {TILE_256x192, 256, 192, 4.1, 1.0, 3.0},
                                 {TILE_128x128, 128, 128, 4.0, 1.2, 2.5},
                                 {TILE_128x64, 128, 64, 2.7, 1.7, 1.5},
                                 {TILE_64x64, 64, 64, 1.4, 2.0, 0.8}};
constexpr TileModel kReduceRows16[] = {{TILE_192x192, 192, 192, 4.1, 1.0, 2.5},
                                       {TILE_128x256, 128, 256, 4.1, 1.4, 1.5}};
constexpr TileModel kF32[] = {{TILE_F32, 128, 128, 0.5, 1.5, 1.5}};

Product plan(int dtype, bool reduce_rows, int64_t M, int64_t N, int64_t K) {
  const bool f32 = dtype == MOE_F32;
  const TileModel* models = f32 ? kF32 : reduce_rows ? kReduceRows16 : kRows16;
  const int count = f32 ? 1 : reduce_rows ? 2 : 5, least = f32 ? 128 : 256;
  Product best{};
  double best_us = 0.0;
  for (int i = 0; i < count; ++i) {
    const TileModel& m = models[i];
    const int64_t tiles = static_cast<int64_t>(ceil_div(M, m.bm)) * ceil_div(N, m.bn);
    // The register-staged tiles address a slice of a row reduction by 32-bit buffer offsets; the DMA
    // tiles move their buffer's 64-bit base with each k tile, and the float32 ones use pointers.
    const int64_t e0 = m.tile == TILE_192x192 ? (K * std::max(M, N) * 2 >> 30) + 1 : 1;
    const int64_t e1 = std::max<int64_t>(e0, std::min<int64_t>(32, K / least));
    for (int64_t e = e0; e <= e1; ++e) {
      const int64_t chunk = (((K + e - 1) / e) + 63) / 64 * 64, E = ceil_div(K, chunk);
      const double busiest = std::max<double>(m.few, static_cast<double>((tiles * E + 255) / 256));
      const double tile_us = 2.0 * m.bm * m.bn * std::min(chunk, K) / (m.tflops * 1e6);
      const double part_us = E > 1 ? 5.0 + 8.0 * E * M * N / 4e6 : 0.0;
      const double us = busiest * (tile_us + m.over_us) + part_us;
      if (best.E != 0 && us >= best_us) continue;
      best_us = us;
      best.tile = m.tile;
      best.bm = m.bm;
      best.bn = m.bn;
      best.ntm = ceil_div(M, m.bm);
      best.ntn = ceil_div(N, m.bn);
      best.kchunk = static_cast<int>(chunk);
      best.E = static_cast<int>(E);
      best.part_bytes = E > 1 ? static_cast<size_t>(E) * M * N * sizeof(float) : 0;
    }
  }
  return best;
}

GemmArgs dense_args(const Product& q, int dtype, int64_t M, int64_t N, int64_t K) {
  GemmArgs a{};
  a.a[1] = none();
  a.b[1] = none();
  a.K[0] = static_cast<int>(K);
  a.M = static_cast<int>(M);
  a.N = static_cast<int>(N);
  a.E = q.E;
  a.ntm = q.ntm;
  a.ntn = q.ntn;
  a.kchunk = q.kchunk;
  a.scale = 1.0f;
  a.dtype = dtype;
  return a;
}

// out = a b^T through epi (epi.y is the output); a is [M, K]; b is [N, K], or [K, N] when !B_KC.
template <bool B_KC>
hipError_t product(const Product& q, GemmArgs& a, const LinearEpi& epi, void* part, hipStream_t s) {
  a.lin = epi;
  a.out = part;
  const int grid = q.E * q.ntm * q.ntn;
  switch (q.tile) {
    case TILE_256x256:
      MOE_TRY(launch(GEMM16(a.dtype, 256, 256, 128, 64, 64, 2, 1, GROUP_M, EPI_LINEAR, false, true, B_KC, 1),
                     grid, a, s, 512));
      break;
    case TILE_256x192:
      MOE_TRY(launch(GEMM16(a.dtype, 256, 192, 64, 96, 64, 2, 1, GROUP_M, EPI_LINEAR, false, true, B_KC, 1),
                     grid, a, s, 512));
      break;
    case TILE_128x128:
      MOE_TRY(launch(GEMM16(a.dtype, 128, 128, 64, 64, 64, 2, 2, GROUP_M, EPI_LINEAR, false, true, B_KC, 1),
                     grid, a, s));
      break;
    case TILE_128x64:
      MOE_TRY(launch(GEMM16(a.dtype, 128, 64, 32, 64, 64, 3, 2, GROUP_M, EPI_LINEAR, false, true, B_KC, 0),
                     grid, a, s));
      break;
    case TILE_64x64:
      MOE_TRY(launch(GEMM16(a.dtype, 64, 64, 32, 32, 64, 5, 2, GROUP_M, EPI_LINEAR, false, true, B_KC, 0),
                     grid, a, s));
      break;
    case TILE_F32:
      MOE_TRY(launch(linear_f32_kernel<true, B_KC, true>, grid, a, s));
      break;
    default: return hipErrorInvalidValue;
  }
  if (q.E == 1) return hipSuccess;
  return by_type(a.dtype, [&](auto tag) {
    const int64_t MN = static_cast<int64_t>(a.M) * a.N;
    hipLaunchKernelGGL(linear_sum_kernel<decltype(tag)>,
                       dim3(static_cast<unsigned>((MN / 8 + 255) / 256)), dim3(256), 0, s,
                       static_cast<const float*>(part), q.E, MN, a.N, epi);
    return hipGetLastError();
  });
}

// dw [N, K] = scale dz^T x: the reduction runs over the rows of both.
hipError_t product_rows(const Product& q, GemmArgs& a, float scale, void* out, void* part,
                        hipStream_t s) {
  a.out = q.E > 1 ? part : out;
  a.scale = q.E > 1 ? 1.0f : scale;
  const int grid = q.E * q.ntm * q.ntn;
  if (a.dtype == MOE_F32)
    MOE_TRY(launch(linear_f32_kernel<false, false, false>, grid, a, s));
  else if (q.tile == TILE_192x192)
    MOE_TRY(launch(GEMM16(a.dtype, 192, 192, 96, 96, 64, 2, 1, GROUP_K, EPI_LINEAR, false, false, false, 1),
                   grid, a, s));
  else
    MOE_TRY(launch(GEMM16(a.dtype, 128, 256, 64, 128, 32, 3, 2, GROUP_K, EPI_LINEAR, false, false, false, 0),
                   grid, a, s));
  if (q.E == 1) return hipSuccess;
  LinearEpi epi{};
  epi.y = out;
  epi.scale = scale;
  return by_type(a.dtype, [&](auto tag) {
    const int64_t MN = static_cast<int64_t>(a.M) * a.N;
    hipLaunchKernelGGL(linear_sum_kernel<decltype(tag)>,
                       dim3(static_cast<unsigned>((MN / 8 + 255) / 256)), dim3(256), 0, s,
                       static_cast<const float*>(part), q.E, MN, a.N, epi);
    return hipGetLastError();
  });
}

template <typename Elem>
hipError_t few_tokens(const LinearDims& d, const void* x, const void* w, const LinearEpi& epi,
                      hipStream_t s) {
  auto* kern = d.T == 1   ? linear_one_kernel<Elem, 1>
               : d.T == 2 ? linear_one_kernel<Elem, 2>
                          : linear_few_kernel<Elem>;
  const dim3 grid(ceil_div(d.N, d.T <= 2 ? 8 : 16)), block(d.T <= 2 ? 256 : 512);
  hipLaunchKernelGGL(kern, grid, block, 0, s, static_cast<const Elem*>(x),
                     static_cast<const Elem*>(w), d.T, d.K, d.N, epi);
  return hipGetLastError();
}

// Groups of rows: about six blocks a CU.
inline int dz_groups(const LinearDims& d) {
  return std::min<int>(ceil_div(d.T, 8), std::max<int>(1, 1536 / ceil_div(d.N, 512)));
}

struct BwdPlan {
  Product dx, dw;
  size_t dz_bytes, part_bytes;
};

BwdPlan bwd_plan(const LinearDims& d, bool form_dz) {
  BwdPlan b{};
  b.dx = plan(d.dtype, false, d.T, d.K, d.N);
  b.dw = plan(d.dtype, true, d.N, d.K, d.T);
  const size_t es = d.dtype == MOE_F32 ? 4 : 2;
  b.dz_bytes = form_dz ? align_up(static_cast<size_t>(d.T) * d.N * es) : 0;
  // dbias's, dx's and dw's partials are used one after the other
  b.part_bytes = std::max({b.dx.part_bytes, b.dw.part_bytes,
                           static_cast<size_t>(dz_groups(d)) * d.N * sizeof(float)});
  return b;
}

}  // namespace

size_t linear_fwd_ws_bytes(const LinearDims& d) {
  if (d.T <= kFewTokens) return 0;
  return plan(d.dtype, false, d.T, d.N, d.K).part_bytes;
}

size_t linear_bwd_ws_bytes(const LinearDims& d, bool form_dz) {
  const BwdPlan b = bwd_plan(d, form_dz);
  return b.dz_bytes + b.part_bytes;
}

hipError_t launch_linear_fwd(const LinearDims& d, const void* x, const void* w,
                             const LinearEpi& epi, void* ws, hipStream_t s, KernelTimer* tm) {
  TimedScope ts(tm, MOE_K_LINEAR_FWD, s);
  if (d.T <= kFewTokens)
    return by_type(d.dtype, [&](auto tag) { return few_tokens<decltype(tag)>(d, x, w, epi, s); });
  const Product q = plan(d.dtype, false, d.T, d.N, d.K);
  GemmArgs a = dense_args(q, d.dtype, d.T, d.N, d.K);
  a.a[0] = opnd(x, 0, d.K, 1, true);
  a.b[0] = opnd(w, 0, d.K, 1, true);
  return product<true>(q, a, epi, ws, s);
}

hipError_t launch_linear_bwd(const LinearDims& d, const void* dy, const void* x, const void* w,
                             const LinearEpi& epi, void* dx, void* dw, void* db, void* ws,
                             hipStream_t s, KernelTimer* tm) {
  TimedScope ts(tm, MOE_K_LINEAR_BWD, s);
  const bool form_dz = epi.act != MOE_ACT_NONE || epi.drop.thr != 0;
  const BwdPlan b = bwd_plan(d, form_dz);
  void* part = static_cast<char*>(ws) + b.dz_bytes;
  const void* dz = form_dz ? ws : dy;
  if (form_dz || db) {
    MOE_TRY(by_type(d.dtype, [&](auto tag) {
      using Elem = decltype(tag);
      const int groups = dz_groups(d);
      hipLaunchKernelGGL(linear_dz_kernel<Elem>, dim3(ceil_div(d.N, 512), groups), dim3(256), 0, s,
                         static_cast<const Elem*>(dy), d.T, d.N, epi,
                         form_dz && (dx || dw) ? static_cast<Elem*>(ws) : nullptr,
                         db ? static_cast<float*>(part) : nullptr);
      MOE_TRY(hipGetLastError());
      if (!db) return hipSuccess;
      hipLaunchKernelGGL(linear_colsum_kernel<Elem>, dim3(ceil_div(d.N, 32)), dim3(1024), 0, s,
                         static_cast<const float*>(part), groups, d.N, static_cast<Elem*>(db));
      return hipGetLastError();
    }));
  }
  if (dx) {
    GemmArgs a = dense_args(b.dx, d.dtype, d.T, d.K, d.N);
    a.a[0] = opnd(dz, 0, d.N, 1, true);
    a.b[0] = opnd(w, 0, d.K, 0, true);
    LinearEpi out{};
    out.y = dx;
    out.scale = epi.drop.scale;
    MOE_TRY(product<false>(b.dx, a, out, part, s));
  }
  if (dw) {
    GemmArgs a = dense_args(b.dw, d.dtype, d.N, d.K, d.T);
    a.a[0] = opnd(dz, 0, d.N, 0, true);
    a.b[0] = opnd(x, 0, d.K, 0, true);
    MOE_TRY(product_rows(b.dw, a, epi.drop.scale, dw, part, s));
  }
  return hipSuccess;
}

}  // namespace moe
