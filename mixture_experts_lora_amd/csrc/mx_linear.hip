// Products of microscaled operands on the matrix cores: y[i] = f(a[i] w[e(i)]^T), a in 8 or 4 bits,
// w in 4, one weight matrix or one per expert, f the identity or SwiGLU of its two halves, y in 16
// bits or microscaled 8 bits (mx.h has the formats).
//
// The scaled MFMA takes the codes as they are stored, with one scale byte per row and 32 elements of
// the reduction, and accumulates in float32. Its operand layout for 32 x 32 x 64 (16 x 16 x 128): lane
// l holds row l % 32 (l % 16) and, with g = l / 32 (l / 16), in 4 bits the 32 elements of block g; in
// 8 bits the 16 elements from 16 g on and the 16 from 16 g on of the second half. The scale that lane
// (row, g) brings is that of block g. w is the first operand, so that an output row's columns lie
// along a lane's registers.
#include <algorithm>
#include <type_traits>

#include "gemm16.h"
#include "mx.h"

namespace moe {

namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr int kMxOut8 = 2;  // beside MOE_BF16 = 1; MOE_F16 stands as 0 here
template <int OUT>
using Out16 = std::conditional_t<OUT == 1, bf16_t, f16_t>;

struct MxGemm {
  const uint8_t *a, *a_scales, *w, *w_scales;
  const int32_t *rows;     // gathered: row i of the products is row rows[i] / k of a
  const int32_t *offsets;  // [E + 1]; null: one weight matrix for all M rows
  void* y;
  uint8_t* y_scales;
  int64_t a_rows;
  int M, K, N, E, k, ntn;
};

// A tile of the products: rows [row0, row0 + rows) with expert e's weights, N tile n.
struct MxTile {
  int e, row0, rows, n;
};

// Inclusive sum over the wave's lanes.
__device__ __forceinline__ int wave_scan(int v, int lane) {
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) {
    const int o = __shfl_up(v, d, kWave);
    if (lane >= d) v += o;
  }
  return v;
}

// Where logical tile `at` of an expert with `mt` M tiles lies: up to 8 M tiles swept across the N
// tiles, so that the tiles at work together share rows and weights in L2.
template <int BM>
__device__ __forceinline__ void raster(const MxGemm& p, int at, int mt, int begin, int end,
                                       MxTile& t) {
  const int gs = at / (kTileGroup * p.ntn) * kTileGroup, gsz = min(kTileGroup, mt - gs);
  const int rem = at - gs * p.ntn;
  t.n = rem / gsz;
  t.row0 = begin + (gs + rem % gsz) * BM;
  t.rows = min(BM, end - t.row0);
}

// The tile of block `b`; false: a block past the last tile. Each wave looks through the offsets by
// itself, 64 experts at a time. spread: logical tiles in eight contiguous runs, one per XCD.
template <int BM, bool SPREAD>
__device__ __forceinline__ bool find_tile(const MxGemm& p, int b, MxTile& t) {
  if (!p.offsets) {
    const int mt = (p.M + BM - 1) / BM, total = mt * p.ntn;
    if (b >= total) return false;
    t.e = 0;
    raster<BM>(p, SPREAD ? xcd_remap(b, total) : b, mt, 0, p.M, t);
    return true;
  }
  const int lane = threadIdx.x & (kWave - 1);
  auto count = [&](int e0, int& begin, int& end) __attribute__((always_inline)) {
    const int e = e0 + lane;
    begin = end = 0;
    if (e < p.E) {
      // rows outside [0, M) are nobody's (a caller's error stays in bounds)
      begin = max(p.offsets[e], 0);
      end = min(p.offsets[e + 1], p.M);
    }
    return end > begin ? (end - begin + BM - 1) / BM : 0;
  };
  int L = b;
  if (SPREAD) {
    int total = 0;
    for (int e0 = 0; e0 < p.E; e0 += kWave) {
      int begin, end;
      total += __builtin_amdgcn_readlane(wave_scan(count(e0, begin, end), lane), kWave - 1);
    }
    total *= p.ntn;
    if (b >= total) return false;
    L = xcd_remap(b, total);
  }
  int before = 0;
  for (int e0 = 0; e0 < p.E; e0 += kWave) {
    int begin, end;
    const int mine = count(e0, begin, end), upto = before + wave_scan(mine, lane);
    const uint64_t past = __ballot(L < upto * p.ntn);
    if (past != 0) {
      const int at = __builtin_ctzll(past);
      const int mt = __builtin_amdgcn_readlane(mine, at);
      const int first = __builtin_amdgcn_readlane(upto, at) - mt;
      t.e = e0 + at;
      raster<BM>(p, L - first * p.ntn, mt, __builtin_amdgcn_readlane(begin, at),
                 __builtin_amdgcn_readlane(end, at), t);
      return true;
    }
    before = __builtin_amdgcn_readlane(upto, kWave - 1);
  }
  return false;
}

template <int FMT>
__device__ __forceinline__ constexpr int row_bytes_of(int k) {
  return FMT == MOE_MX_FP4 ? k / 2 : k;
}

// ------------------------------------------------------------------ many rows: tiles through LDS
// LDS rows hold 128 elements, 16-byte chunk c of row r at c ^ swizzle(r), so that 16 lanes of a
// fragment read (16 rows, one chunk) touch every bank once.
template <int RB>  // bytes a row: 128 or 64
__device__ __forceinline__ int mx_swz(int r) {
  return RB == 128 ? (r >> 1) & 7 : (r >> 2) & 3;
}

// Rows of one operand's tile as DMA instructions of 1 KB: the lane's source offset, without the
// stage's.
template <int RB, int N>
struct MxFill {
  uint32_t vo[N];
};

template <int RB>
__device__ __forceinline__ int fill_row(int j, int lane) { return j * (1024 / RB) + lane / (RB / 16); }
template <int RB>
__device__ __forceinline__ int fill_chunk(int j, int lane) {
  return (lane % (RB / 16)) ^ mx_swz<RB>(fill_row<RB>(j, lane));
}

// Columns of the output that a block of BN weight rows gives.
template <int BN, bool SWIGLU>
constexpr int out_cols() { return SWIGLU ? BN / 2 : BN; }

template <int AF, int OUT, bool SWIGLU, int BM, int BN, int WM, int WN, int MINB>
__global__ __launch_bounds__((BM / WM) * (BN / WN) * 64, MINB) void mx_gemm_kernel(MxGemm p) {
  constexpr int WAVES_N = BN / WN, NW = (BM / WM) * WAVES_N;
  constexpr int MF = WM / 32, NF = WN / 32;
  constexpr int AB = row_bytes_of<AF>(128), WB = 64;
  constexpr int A_BYTES = BM * AB, W_BYTES = BN * WB, STAGE = A_BYTES + W_BYTES;
  constexpr int S_BYTES = (BM + BN) * 16;  // scales of 512 elements
  constexpr int AI = A_BYTES / 1024 / NW, WI = W_BYTES / 1024 / NW;
  static_assert(AI * NW * 1024 == A_BYTES && WI * NW * 1024 == W_BYTES, "whole instructions a wave");
  static_assert((BM + BN) % 64 == 0 && BM % 64 == 0, "whole scale instructions");
  __shared__ __attribute__((aligned(1024))) char smem[2 * STAGE + 2 * S_BYTES];
  char* const sscale = smem + 2 * STAGE;

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WAVES_N, wn = wave % WAVES_N;
  MxTile t;
  if (!find_tile<BM, true>(p, blockIdx.x, t)) return;
  const int n0 = t.n * out_cols<BN, SWIGLU>();
  const int n_w = SWIGLU ? 2 * p.N : p.N;
  const int a_row = row_bytes_of<AF>(p.K), w_row = p.K / 2;
  const int sc = static_cast<int>(mx_scale_cols(p.K));

  // Weight row of the tile's row r. SwiGLU: each wave's rows are half gate, half up.
  auto weight_row = [&](int r, bool& ok) __attribute__((always_inline)) {
    if (!SWIGLU) {
      ok = n0 + r < p.N;
      return n0 + r;
    }
    const int w = r / WN, in = r % WN, f = n0 + w * (WN / 2) + in % (WN / 2);
    ok = f < p.N;
    return in < WN / 2 ? f : p.N + f;
  };
  // Row of a: gathered rows as they are in a, the others from the tile's first on.
  const int64_t a_first = p.rows ? 0 : t.row0;
  auto act_row = [&](int r, bool& ok) __attribute__((always_inline)) {
    ok = r < t.rows;
    if (!p.rows) return r;
    const int pair = p.rows[t.row0 + (ok ? r : 0)];
    const int row = static_cast<int>(static_cast<uint32_t>(pair) / static_cast<uint32_t>(p.k));
    ok = ok && row < p.a_rows;
    return row;
  };
  const u32x4 ra = buffer_rsrc(p.a + a_first * a_row, clamp_records((p.a_rows - a_first) * a_row));
  const u32x4 rw = buffer_rsrc(p.w + static_cast<int64_t>(t.e) * n_w * w_row,
                               clamp_records(static_cast<int64_t>(n_w) * w_row));
  const u32x4 rsa = buffer_rsrc(p.a_scales + a_first * sc, clamp_records((p.a_rows - a_first) * sc));
  const u32x4 rsw = buffer_rsrc(p.w_scales + static_cast<int64_t>(t.e) * n_w * sc,
                                clamp_records(static_cast<int64_t>(n_w) * sc));
  uint32_t voa[AI], vow[WI];
#pragma unroll
  for (int i = 0; i < AI; ++i) {
    const int j = wave + NW * i;
    bool ok;
    const int row = act_row(fill_row<AB>(j, lane), ok);
    voa[i] = ok ? static_cast<uint32_t>(row) * a_row + fill_chunk<AB>(j, lane) * 16 : kOOB;
  }
#pragma unroll
  for (int i = 0; i < WI; ++i) {
    const int j = wave + NW * i;
    bool ok;
    const int row = weight_row(fill_row<WB>(j, lane), ok);
    vow[i] = ok ? static_cast<uint32_t>(row) * w_row + fill_chunk<WB>(j, lane) * 16 : kOOB;
  }
  // scale rows: instruction q covers 64 rows of the tile, a's first
  constexpr int SI = (S_BYTES / 1024 + NW - 1) / NW;
  uint32_t vos[SI];
#pragma unroll
  for (int i = 0; i < SI; ++i) {
    const int q = wave + NW * i;
    bool ok = false;
    int row = 0;
    if (q < BM / 64) row = act_row(q * 64 + lane, ok);
    else if (q < (BM + BN) / 64) row = weight_row((q - BM / 64) * 64 + lane, ok);
    vos[i] = ok ? static_cast<uint32_t>(row) * sc : kOOB;
  }

  const int stages = (p.K + 127) / 128;
  auto issue = [&](int s) __attribute__((always_inline)) {
    char* st = smem + (s & 1) * STAGE;
    const int left = p.K - s * 128;  // elements; a multiple of 32
    const int a_left = row_bytes_of<AF>(left), w_left = left / 2;
#pragma unroll
    for (int i = 0; i < AI; ++i) {
      const int j = wave + NW * i;
      const uint32_t vo = fill_chunk<AB>(j, lane) * 16 < a_left ? voa[i] : kOOB;
      dma16(st + j * 1024, ra, vo, static_cast<uint32_t>(s) * AB);
    }
#pragma unroll
    for (int i = 0; i < WI; ++i) {
      const int j = wave + NW * i;
      const uint32_t vo = fill_chunk<WB>(j, lane) * 16 < w_left ? vow[i] : kOOB;
      dma16(st + A_BYTES + j * 1024, rw, vo, static_cast<uint32_t>(s) * WB);
    }
    if ((s & 3) == 0) {
      char* ss = sscale + ((s >> 2) & 1) * S_BYTES;
#pragma unroll
      for (int i = 0; i < SI; ++i) {
        const int q = wave + NW * i;
        if (q < (BM + BN) / 64)
          dma16(ss + q * 1024, q < BM / 64 ? rsa : rsw, vos[i], static_cast<uint32_t>(s) * 4);
      }
    }
  };

  f32x16 acc[NF][MF] = {};
  const int r = lane & 31, g = lane >> 5;
  issue(0);
  for (int s = 0; s < stages; ++s) {
    // this stage has arrived for every wave, and nobody reads the one before any more
    wait_vmcnt<0>();
    barrier_lds();
    if (s + 1 < stages) issue(s + 1);
    const char* sa = smem + (s & 1) * STAGE + wm * WM * AB;
    const char* sw = smem + (s & 1) * STAGE + A_BYTES + wn * WN * WB;
    const char* ss = sscale + ((s >> 2) & 1) * S_BYTES + (s & 3) * 4;
    int sca[MF], scw[NF];
#pragma unroll
    for (int f = 0; f < MF; ++f)
      sca[f] = *reinterpret_cast<const int*>(ss + (wm * WM + f * 32 + r) * 16) >> (8 * g);
#pragma unroll
    for (int f = 0; f < NF; ++f)
      scw[f] = *reinterpret_cast<const int*>(ss + (BM + wn * WN + f * 32 + r) * 16) >> (8 * g);
    auto step = [&](auto jc) __attribute__((always_inline)) {
      constexpr int j = decltype(jc)::value;
      i32x8 fa[MF], fw[NF];
#pragma unroll
      for (int f = 0; f < NF; ++f) {
        const i32x4 v = *reinterpret_cast<const i32x4*>(
            sw + (f * 32 + r) * WB + (((2 * j + g) ^ mx_swz<WB>(r)) << 4));
        fw[f] = __builtin_shufflevector(v, v, 0, 1, 2, 3, -1, -1, -1, -1);
      }
#pragma unroll
      for (int f = 0; f < MF; ++f) {
        const char* row = sa + (f * 32 + r) * AB;
        if constexpr (AF == MOE_MX_FP4) {
          const i32x4 v = *reinterpret_cast<const i32x4*>(row + (((2 * j + g) ^ mx_swz<AB>(r)) << 4));
          fa[f] = __builtin_shufflevector(v, v, 0, 1, 2, 3, -1, -1, -1, -1);
        } else {
          const i32x4 lo = *reinterpret_cast<const i32x4*>(row + (((4 * j + g) ^ mx_swz<AB>(r)) << 4));
          const i32x4 hi =
              *reinterpret_cast<const i32x4*>(row + (((4 * j + 2 + g) ^ mx_swz<AB>(r)) << 4));
          fa[f] = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
        }
      }
#pragma unroll
      for (int f = 0; f < NF; ++f)
#pragma unroll
        for (int m = 0; m < MF; ++m)
          acc[f][m] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
              fw[f], fa[m], acc[f][m], 4, AF == MOE_MX_FP4 ? 4 : 0, 2 * j, scw[f], 2 * j, sca[m]);
    };
    step(std::integral_constant<int, 0>());
    step(std::integral_constant<int, 1>());
  }

  // Lane (r, g) holds row r's columns 8 q + 4 g + i at register 4 q + i; after swapping halves with
  // its partner it holds the 16 columns from 16 g on.
  auto columns = [&](const f32x16& c, float (&v)[16]) __attribute__((always_inline)) {
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
        const auto x = __builtin_amdgcn_permlane32_swap(__float_as_uint(c[4 * q + i]),
                                                        __float_as_uint(c[4 * (q + 2) + i]), false, false);
        v[8 * q + i] = __uint_as_float(x[0]);
        v[8 * q + 4 + i] = __uint_as_float(x[1]);
      }
  };
  constexpr int OF = SWIGLU ? NF / 2 : NF;  // fragments of output columns
#pragma unroll
  for (int m = 0; m < MF; ++m) {
    const int local = wm * WM + m * 32 + r;
    const bool there = local < t.rows;
    const int64_t row = t.row0 + local;
#pragma unroll
    for (int f = 0; f < OF; ++f) {
      float v[16];
      columns(acc[f][m], v);
      if constexpr (SWIGLU) {
        float u[16];
        columns(acc[f + NF / 2][m], u);
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = swiglu(v[i], u[i]);
      }
      const int base = n0 + wn * (OF * 32) + f * 32, col = base + 16 * g;
      if constexpr (OUT == kMxOut8) {
        uint32_t amax = 0;
#pragma unroll
        for (int i = 0; i < 16; ++i) amax = max(amax, __float_as_uint(v[i]) & 0x7fffffffu);
        const auto x = __builtin_amdgcn_permlane32_swap(amax, amax, false, false);
        amax = max(static_cast<uint32_t>(x[0]), static_cast<uint32_t>(x[1]));
        const uint32_t sb = mx_scale_of<MOE_MX_FP8>(amax);
        float lo[8], hi[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          lo[i] = v[i];
          hi[i] = v[8 + i];
        }
        const uint2 c0 = mx_encode8<MOE_MX_FP8>(lo, sb), c1 = mx_encode8<MOE_MX_FP8>(hi, sb);
        if (there && base < p.N) {
          *reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.y) + row * p.N + col) =
              make_uint4(c0.x, c0.y, c1.x, c1.y);
          if (g == 0) {
            const int cols = static_cast<int>(mx_scale_cols(p.N));
            uint8_t* s = p.y_scales + row * cols;
            s[base / 32] = static_cast<uint8_t>(sb);
            if (base + 32 == p.N)
              for (int i = p.N / 32; i < cols; ++i) s[i] = 0;
          }
        }
      } else {
        Out16<OUT>* y = static_cast<Out16<OUT>*>(p.y) + row * p.N + col;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float o[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) o[i] = v[8 * h + i];
          Row8<Out16<OUT>> r8;
          r8.set(o);
          if (there && col + 8 * h < p.N) r8.store(y + 8 * h);
        }
      }
    }
  }
}

// ------------------------------------------------------------------ few rows: weights streamed
// A block takes up to 16 rows and 32 output columns; its four waves split the reduction and meet in
// LDS, adding in order. Weights come straight from HBM into the matrix cores' registers, each byte
// once for 16 rows; steps of 128 elements are loaded kAhead at a time.
constexpr int kSmallRows = 16, kSmallCols = 32, kSmallWaves = 4, kAhead = 4;

template <int AF, int OUT, bool SWIGLU>
__global__ __launch_bounds__(kSmallWaves * 64) void mx_rows_kernel(MxGemm p) {
  constexpr int NF = SWIGLU ? 4 : 2;
  constexpr int AB = row_bytes_of<AF>(128), AC = AB / 64;  // bytes a step; 16-byte pieces a lane
  constexpr int LD = 20;  // floats between a row's fragments' columns, off the banks' period
  __shared__ float red[kSmallWaves][NF][16][LD];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  MxTile t;
  if (!find_tile<kSmallRows, false>(p, blockIdx.x, t)) return;
  const int n0 = t.n * kSmallCols, n_w = SWIGLU ? 2 * p.N : p.N;
  const int a_row = row_bytes_of<AF>(p.K), w_row = p.K / 2;
  const int sc = static_cast<int>(mx_scale_cols(p.K));
  const int r = lane & 15, g = lane >> 4;

  // a's row of this lane
  const bool act = r < t.rows;
  int64_t arow = t.row0 + (act ? r : 0);
  if (p.rows)
    arow = static_cast<uint32_t>(p.rows[arow]) / static_cast<uint32_t>(p.k);
  const bool a_ok = act && arow < p.a_rows;
  if (!a_ok) arow = 0;
  const uint8_t* ap = p.a + arow * a_row;
  const uint8_t* asp = p.a_scales + arow * sc;
  const uint8_t *wp[NF], *wsp[NF];
  bool w_ok[NF];
#pragma unroll
  for (int f = 0; f < NF; ++f) {
    const int half = SWIGLU ? f & 1 : f, n = n0 + 16 * half + r;
    w_ok[f] = n < p.N;
    const int64_t row = static_cast<int64_t>(t.e) * n_w + (w_ok[f] ? n : 0) + (SWIGLU && f >= 2 ? p.N : 0);
    wp[f] = p.w + row * w_row;
    wsp[f] = p.w_scales + row * sc;
  }
  const int steps = (p.K + 127) / 128, each = (steps + kSmallWaves - 1) / kSmallWaves;
  const int first = wave * each, last = min(steps, first + each);
  f32x4 acc[NF] = {};
  const i32x4 zero = {};
  for (int s0 = first; s0 < last; s0 += kAhead) {
    i32x4 w[kAhead][NF], a[kAhead][AC];
    int sw[kAhead][NF], sa[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int s = s0 + u;
      const bool in = s < last;
      const int at = in ? s : first;
      // elements of this lane's pieces that are within the row
      const int left = in ? p.K - s * 128 : 0;
#pragma unroll
      for (int f = 0; f < NF; ++f) {
        const bool ok = w_ok[f] && g * 32 < left;
        w[u][f] = ok ? __builtin_nontemporal_load(reinterpret_cast<const i32x4*>(wp[f] + at * 64 + g * 16)) : zero;
        sw[u][f] = *reinterpret_cast<const int*>(wsp[f] + at * 4) >> (8 * g);
      }
#pragma unroll
      for (int c = 0; c < AC; ++c) {
        const int byte = c * 64 + g * 16;
        const bool ok = a_ok && byte < row_bytes_of<AF>(left);
        a[u][c] = ok ? *reinterpret_cast<const i32x4*>(ap + at * AB + byte) : zero;
      }
      sa[u] = *reinterpret_cast<const int*>(asp + at * 4) >> (8 * g);
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const i32x8 fa = AC == 2 ? __builtin_shufflevector(a[u][0], a[u][AC - 1], 0, 1, 2, 3, 4, 5, 6, 7)
                               : __builtin_shufflevector(a[u][0], a[u][0], 0, 1, 2, 3, -1, -1, -1, -1);
#pragma unroll
      for (int f = 0; f < NF; ++f)
        acc[f] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
            __builtin_shufflevector(w[u][f], w[u][f], 0, 1, 2, 3, -1, -1, -1, -1), fa, acc[f], 4,
            AF == MOE_MX_FP4 ? 4 : 0, 0, sw[u][f], 0, sa[u]);
    }
  }
  // lane (r, g) has row r, columns 4 g .. 4 g + 3
#pragma unroll
  for (int f = 0; f < NF; ++f)
    *reinterpret_cast<f32x4*>(&red[wave][f][r][4 * g]) = acc[f];
  __syncthreads();
  const int m = threadIdx.x >> 4, c = (threadIdx.x & 15) * 2, col = n0 + c;
  auto total = [&](int f, int at) __attribute__((always_inline)) {
    float v = red[0][f][m][at];
#pragma unroll
    for (int w = 1; w < kSmallWaves; ++w) v += red[w][f][m][at];
    return v;
  };
  float v[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    v[i] = total(c >> 4, (c & 15) + i);
    if constexpr (SWIGLU) v[i] = swiglu(v[i], total(2 + (c >> 4), (c & 15) + i));
  }
  const bool there = m < t.rows && col < p.N;
  const int64_t row = t.row0 + m;
  if constexpr (OUT == kMxOut8) {
    uint32_t amax = max(__float_as_uint(v[0]) & 0x7fffffffu, __float_as_uint(v[1]) & 0x7fffffffu);
    amax = max(amax, static_cast<uint32_t>(dpp_i32<kDppSwap1>(static_cast<int>(amax))));
    amax = max(amax, static_cast<uint32_t>(dpp_i32<kDppSwap2>(static_cast<int>(amax))));
    amax = max(amax, static_cast<uint32_t>(dpp_i32<kDppHalfMirror>(static_cast<int>(amax))));
    amax = max(amax, static_cast<uint32_t>(dpp_i32<kDppMirror>(static_cast<int>(amax))));
    const uint32_t sb = mx_scale_of<MOE_MX_FP8>(amax);
    const float e[8] = {v[0], v[1]};
    const uint2 code = mx_encode8<MOE_MX_FP8>(e, sb);
    if (there) {
      *reinterpret_cast<uint16_t*>(static_cast<uint8_t*>(p.y) + row * p.N + col) =
          static_cast<uint16_t>(code.x);
      if (c == 0) {
        const int cols = static_cast<int>(mx_scale_cols(p.N));
        uint8_t* s = p.y_scales + row * cols;
        s[n0 / 32] = static_cast<uint8_t>(sb);
        if (n0 + 32 == p.N)
          for (int i = p.N / 32; i < cols; ++i) s[i] = 0;
      }
    }
  } else if (there) {
    const uint32_t lo = __builtin_bit_cast(uint16_t, from_f32<Out16<OUT>>(v[0]));
    const uint32_t hi = __builtin_bit_cast(uint16_t, from_f32<Out16<OUT>>(v[1]));
    *reinterpret_cast<uint32_t*>(static_cast<Out16<OUT>*>(p.y) + row * p.N + col) = lo | (hi << 16);
  }
}

// Calls go with the format of a, the output and SwiGLU as constants.
template <typename F>
hipError_t by_product(const moe_mx_linear_shape& s, F&& go) {
  using std::integral_constant;
  return by_format(s.a_format, [&](auto af) {
    auto out = [&](auto o) {
      return s.swiglu ? go(af, o, integral_constant<bool, true>())
                      : go(af, o, integral_constant<bool, false>());
    };
    if (s.out == MOE_MX_OUT_FP8) return out(integral_constant<int, kMxOut8>());
    if (s.out == MOE_BF16) return out(integral_constant<int, 1>());
    return out(integral_constant<int, 0>());
  });
}

}  // namespace

size_t mx_linear_ws_bytes(const moe_mx_linear_shape&) { return 0; }

hipError_t launch_mx_linear(const moe_mx_linear_shape& s, const void* a, const uint8_t* a_scales,
                            const int32_t* rows, const int32_t* offsets, const void* w,
                            const uint8_t* w_scales, void* y, uint8_t* y_scales, void*,
                            hipStream_t st, KernelTimer* tm) {
  TimedScope ts(tm, MOE_K_MX_LINEAR, st);
  MxGemm p{};
  p.a = static_cast<const uint8_t*>(a);
  p.a_scales = a_scales;
  p.w = static_cast<const uint8_t*>(w);
  p.w_scales = w_scales;
  p.rows = s.gather ? rows : nullptr;
  p.offsets = s.E > 0 ? offsets : nullptr;
  p.y = y;
  p.y_scales = y_scales;
  p.M = s.T * s.k;
  p.a_rows = s.gather ? s.T : p.M;
  p.K = s.K;
  p.N = s.N;
  p.E = s.E;
  p.k = s.k;
  const int experts = std::max(1, std::min(s.E, p.M));
  return by_product(s, [&](auto af, auto out, auto glu) {
    constexpr int AF = decltype(af)::value, OUT = decltype(out)::value;
    constexpr bool GLU = decltype(glu)::value;
    // at most this many M tiles of bm rows, whatever the experts' counts are
    auto tiles = [&](int bm) {
      return s.E > 0 ? p.M / bm + experts : (p.M + bm - 1) / bm;
    };
    if (p.M <= 16 * experts) {
      p.ntn = (s.N + kSmallCols - 1) / kSmallCols;
      hipLaunchKernelGGL((mx_rows_kernel<AF, OUT, GLU>),
                         dim3(static_cast<unsigned>(tiles(kSmallRows) * p.ntn)),
                         dim3(kSmallWaves * 64), 0, st, p);
    } else {
      constexpr int BM = 128, BN = 256, C = out_cols<BN, GLU>();
      p.ntn = (s.N + C - 1) / C;
      hipLaunchKernelGGL((mx_gemm_kernel<AF, OUT, GLU, BM, BN, 64, 128, 2>),
                         dim3(static_cast<unsigned>(tiles(BM) * p.ntn)), dim3(256), 0, st, p);
    }
    return hipGetLastError();
  });
}

}  // namespace moe
