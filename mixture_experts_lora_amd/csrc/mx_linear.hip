// Products of microscaled operands on the matrix cores: y[i] = f(a[i] w[e(i)]^T), a in 8 or 4 bits,
// w in 4, one weight matrix or one per expert, f the identity or SwiGLU of its two halves, y in 16
// bits or microscaled 8 bits (mx.h has the formats).
//
// The scaled MFMA takes the codes as they are stored, with one scale byte per row and 32 elements of
// the reduction, and accumulates in float32. With two 4-bit operands nothing is lost on the way. With
// 8-bit codes it aligns each eight neighbouring products to the largest of them and cuts off what lies
// below 2^-13 of its power of two (measured; sums of random rows are then off by about 4e-6, where
// float32 sums are off by 1e-7). So an 8-bit a is multiplied in two parts, the codes of 4 and more and
// the others: a product of the first is a multiple of 2^-2 and at most 2688, which is cut at 2^-2; one
// of the others is at most 22.5, cut at 2^-9, and a multiple of that unless its code is below 2^-5, where
// 2^-10 can go. Sums are then float32's (of 94 million 8-bit results of 2880-element sums 76 are not the
// nearest to the exact one, 75 by a float32 product in torch, 49764 in one part), for twice the matrix
// instructions: the experts below 790 to 880 us in two parts and 510 to 540 in one, one token 11.5 and
// 10.3. One part is a caller's choice (fast).
//
// Its operand layout for 32 x 32 x 64 (16 x 16 x 128): lane l holds row l % 32 (l % 16) and, with
// g = l / 32 (l / 16), in 4 bits the 32 elements of block g; in 8 bits the 16 elements from 16 g on and
// the 16 from 16 g on of the second half. The scale that lane (row, g) brings is that of block g. w is
// the first operand, so that an output row's columns lie along a lane's registers.
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
// 32 experts, 8192 tokens of 4, 2880 -> 2 x 2880, 8-bit result: in two parts 790 to 880 us, the matrix
// cores busy for 59 % of the cycles (executed 2.5 to 2.75 PFLOP/s, where products of such data from
// registers alone reach 3.6 to 3.9); in one 510 to 540 us, busy for 50 %. Most of the rest stands outside
// the loop: 9.5 us a tile, 13 tiles a CU one after another, are the tile's lookup, its first stages and
// its epilogue, in which nothing else runs on the CU. Power is the smaller part (zeros in the place of
// data: 749 us for 793, and 473 for 509). Dense, 4 bits by 4, 8192 x 4096 x 2880: 60 to 66 us, the matrix
// cores busy for 31 %, on zeros 53.
//
// A stage is 128 elements of every row; NST stages have places in LDS. 16-byte chunk c of row r is
// kept at c ^ swizzle(r), so that 16 lanes of a fragment read (16 rows, one chunk) touch every bank
// once.
template <int RB>  // bytes a row: 128 (8 bits) or 64 (4 bits)
__device__ __forceinline__ int mx_swz(int r) {
  return RB == 128 ? (r >> 1) & 7 : (r >> 2) & 3;
}

// Row and byte within the stage that lane `lane` of an operand's 1 KB DMA instruction j brings.
template <int RB>
__device__ __forceinline__ int fill_row(int j, int lane) { return j * (1024 / RB) + lane / (RB / 16); }
template <int RB>
__device__ __forceinline__ int fill_byte(int j, int lane) {
  return ((lane % (RB / 16)) ^ mx_swz<RB>(fill_row<RB>(j, lane))) * 16;
}

// The instruction's operand: 16 bytes of 4-bit codes (the upper half is not read), or 32 of 8-bit.
__device__ __forceinline__ i32x8 mx_operand(const i32x4& lo, const i32x4& hi, bool fp4) {
  return fp4 ? __builtin_shufflevector(lo, lo, 0, 1, 2, 3, -1, -1, -1, -1)
             : __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}

// The codes of 4 and more in magnitude, with zeros in the place of the others. Magnitude bits past 0x47
// carry into a byte's bit 7, which is then spread over the byte.
__device__ __forceinline__ i32x8 mx_large(const i32x8& x) {
  i32x8 r;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t v = static_cast<uint32_t>(x[i]);
    const uint32_t t = (v & 0x7f7f7f7fu) + 0x38383838u;
    // bytes 0 to 3 of all ones or zeros by bits 7, 15, 23 and 31 of t
    r[i] = static_cast<int>(v & __builtin_amdgcn_perm(t, t << 8, 0x0b090a08u));
  }
  return r;
}

// 16 bytes per lane, global -> LDS at byte `lds` of the block's memory (dma16 of gemm16.h, whose
// generic pointers cost a check for null each); rs and soff are uniform.
__device__ __forceinline__ void dma16_at(uint32_t lds, const u32x4& rs, uint32_t vo, uint32_t soff) {
  const uint32_t m0 = __builtin_amdgcn_readfirstlane(lds);
  u32x4 srs;
#pragma unroll
  for (int i = 0; i < 4; ++i) srs[i] = __builtin_amdgcn_readfirstlane(rs[i]);
  const uint32_t ssoff = __builtin_amdgcn_readfirstlane(soff);
  asm volatile("s_nop 4\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds" ::"{m0}"(m0), "v"(vo),
               "s"(srs), "s"(ssoff)
               : "memory");
}

// Columns of the output that a block of BN weight rows gives.
template <int BN, bool SWIGLU>
constexpr int out_cols() { return SWIGLU ? BN / 2 : BN; }

// PARTS: that a is multiplied in.
template <int AF, int PARTS, int OUT, bool SWIGLU, int BM, int BN, int WM, int WN, int NST>
__global__ __launch_bounds__((BM / WM) * (BN / WN) * 64)
    __attribute__((amdgpu_waves_per_eu(2, 2))) void mx_gemm_kernel(MxGemm p) {
  constexpr int WAVES_N = BN / WN, NW = (BM / WM) * WAVES_N;
  constexpr int MF = WM / 32, NF = WN / 32;
  constexpr int AB = row_bytes_of<AF>(128), WB = 64;
  // places for w's rows in whole instructions a wave; those past BN are not filled
  constexpr int BNL = (BN + NW * (1024 / WB) - 1) / (NW * (1024 / WB)) * (NW * (1024 / WB));
  constexpr int A_BYTES = BM * AB, W_BYTES = BNL * WB, STAGE = A_BYTES + W_BYTES;
  constexpr int S_BYTES = (BM + BN) * 16;  // scales of 512 elements, in two places
  constexpr int AI = A_BYTES / 1024 / NW, WI = W_BYTES / 1024 / NW;
  static_assert(AI * NW * 1024 == A_BYTES && WI * NW * 1024 == W_BYTES, "whole instructions a wave");
  static_assert(NW * (1024 / AB) % 16 == 0 && NW * (1024 / WB) % 16 == 0,
                "whole swizzle periods between a wave's instructions");
  static_assert(BN % 64 == 0 && BM % 64 == 0, "whole scale instructions");
  static_assert(NST >= 2 && NST <= 4, "scales: one place is read, the other filled");
  constexpr int S_AT = NST * STAGE;
  __shared__ __attribute__((aligned(1024))) char smem[S_AT + 2 * S_BYTES];

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WAVES_N, wn = wave % WAVES_N;
  MxTile t;
  if (!find_tile<BM, true>(p, blockIdx.x, t)) return;

  const int n_w = SWIGLU ? 2 * p.N : p.N;
  const int a_row = row_bytes_of<AF>(p.K), w_row = p.K / 2;
  const int sc = static_cast<int>(mx_scale_cols(p.K));
  const int stages = (p.K + 127) / 128;

  // Weight row of a tile's row r, from the tile's first on. SwiGLU: each wave's rows are half gate,
  // half up. A row past the last reads zeros (past the matrix) or a row whose column is not stored.
  auto weight_row = [&](int r) __attribute__((always_inline)) {
    if (!SWIGLU) return r;
    const int in = r % WN;
    return r / WN * (WN / 2) + in % (WN / 2) + (in < WN / 2 ? 0 : p.N);
  };
  static_assert(!SWIGLU || NW * (1024 / WB) == WN / 2 || NW * (1024 / WB) % WN == 0,
                "rows an instruction's step apart are so in w");
  // the byte a lane brings is the same in all of its wave's instructions
  const int byte_a = fill_byte<AB>(wave, lane), byte_w = fill_byte<WB>(wave, lane);
  // scale rows: instruction q covers 64 rows of a tile, a's first
  constexpr int SI = (S_BYTES / 1024 + NW - 1) / NW;
  // row of a gathered or, from the tile's first on, of its own
  auto act = [&](int r, int bytes, uint32_t byte) __attribute__((always_inline)) {
    if (!p.rows) return r < t.rows ? r * bytes + byte : kOOB;
    const int pair = p.rows[t.row0 + min(r, t.rows - 1)];
    const uint32_t row = static_cast<uint32_t>(pair) / static_cast<uint32_t>(p.k);
    return r < t.rows && row < p.a_rows ? row * bytes + byte : kOOB;
  };
  const int64_t a_first = p.rows ? 0 : t.row0, w_first = static_cast<int64_t>(t.e) * n_w;
  const u32x4 ra = buffer_rsrc(p.a + a_first * a_row, clamp_records((p.a_rows - a_first) * a_row));
  const u32x4 rsa = buffer_rsrc(p.a_scales + a_first * sc, clamp_records((p.a_rows - a_first) * sc));
  const u32x4 rw = buffer_rsrc(p.w + w_first * w_row, clamp_records(static_cast<int64_t>(n_w) * w_row));
  const u32x4 rsw = buffer_rsrc(p.w_scales + w_first * sc, clamp_records(static_cast<int64_t>(n_w) * sc));
  const int n0 = t.n * out_cols<BN, SWIGLU>();
  uint32_t voa[AI], vos[SI];
#pragma unroll
  for (int i = 0; i < AI; ++i) voa[i] = act(fill_row<AB>(wave + NW * i, lane), a_row, byte_a);
  const uint32_t vow = static_cast<uint32_t>(n0 + weight_row(fill_row<WB>(wave, lane))) * w_row + byte_w;
#pragma unroll
  for (int i = 0; i < SI; ++i) {
    const int q = wave + NW * i;
    vos[i] = q < BM / 64 ? act(q * 64 + lane, sc, 0)
                         : static_cast<uint32_t>(n0 + weight_row((q - BM / 64) * 64 + lane)) * sc;
  }

  const uint32_t lds = static_cast<uint32_t>(
      reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) const char*)(smem)));
  // Instruction i of this wave's share of stage s into place `at`; what lies past the rows' end is
  // filled with zeros.
  auto issue = [&](int s, int at, int i) __attribute__((always_inline)) {
    const uint32_t st = lds + at * STAGE;
    if (i < AI) {
      const uint32_t end = a_row - s * AB > byte_a ? 0u : kOOB;
      dma16_at(st + (wave + NW * i) * 1024, ra, voa[i < AI ? i : 0] | end, static_cast<uint32_t>(s) * AB);
    } else {
      i -= AI;
      uint32_t end = w_row - s * WB > byte_w ? 0u : kOOB;
      if (BN != BNL && (wave + NW * i) * (1024 / WB) >= BN) end = kOOB;
      dma16_at(st + A_BYTES + (wave + NW * i) * 1024, rw,
               (vow + static_cast<uint32_t>(weight_row(NW * (1024 / WB) * i)) * w_row) | end,
               static_cast<uint32_t>(s) * WB);
    }
  };
  // The scales of four stages, with the first of them.
  auto issue_scales = [&](int s) __attribute__((always_inline)) {
    if ((s & 3) != 0) return;
#pragma unroll
    for (int i = 0; i < SI; ++i) {
      const int q = wave + NW * i;
      if (q < (BM + BN) / 64)
        dma16_at(lds + S_AT + (s >> 2 & 1) * S_BYTES + q * 1024, q < BM / 64 ? rsa : rsw,
                 vos[i] | (s * 4 < sc ? 0u : kOOB), static_cast<uint32_t>(s) * 4);
    }
  };

  // A stage is two steps of 64 elements, each with its own fragment registers: the second step's are
  // read while the first is multiplied and the next stage's first while the second is. The barrier
  // stands between the two, when a wave has read all of the stage and the next one has arrived; the
  // place it frees is filled during the second step, a few instructions beside each product (all
  // before the products: 32 experts, 8192 tokens of 4, 550 us against 518; dense 73.8 / 69.0).
  f32x16 acc[NF][MF] = {};
  const int r = lane & 31, g = lane >> 5;
  struct Frags {
    i32x4 a[MF][AB / 64], w[NF];  // as loaded; widened to the instruction's operand at its use
  };
  struct Scales {
    int a[MF], w[NF];
  };
  auto load_scales = [&](int s, Scales& c) __attribute__((always_inline)) {
    const char* ss = smem + S_AT + (s >> 2 & 1) * S_BYTES + (s & 3) * 4;
#pragma unroll
    for (int f = 0; f < MF; ++f)
      c.a[f] = *reinterpret_cast<const int*>(ss + (wm * WM + f * 32 + r) * 16) >> (8 * g);
#pragma unroll
    for (int f = 0; f < NF; ++f)
      c.w[f] = *reinterpret_cast<const int*>(ss + (BM + wn * WN + f * 32 + r) * 16) >> (8 * g);
  };
  // Piece i of a step's fragments: 16 bytes of a weight fragment, or of one of a's.
  constexpr int PIECES = NF + MF * (AB / 64), PRODUCTS = NF * MF * PARTS;
  auto load = [&](int at, auto jc, int i, Frags& x) __attribute__((always_inline)) {
    constexpr int j = decltype(jc)::value;
    if (i < NF) {
      x.w[i < NF ? i : 0] = *reinterpret_cast<const i32x4*>(
          smem + at * STAGE + A_BYTES + (wn * WN + i * 32 + r) * WB + (((2 * j + g) ^ mx_swz<WB>(r)) << 4));
    } else if (i < PIECES) {
      const int f = (i - NF) / (AB / 64), h = (i - NF) % (AB / 64);
      x.a[f][h] = *reinterpret_cast<const i32x4*>(
          smem + at * STAGE + (wm * WM + f * 32 + r) * AB +
          (((AB / 32 * j + 2 * h + g) ^ mx_swz<AB>(r)) << 4));
    }
  };
  // Product i of a step. The empty statement holds it in place: neither it nor what stands beside it
  // moves across, so that the wave's other instructions go out while the matrix core is busy.
  i32x8 large, rest;
  auto multiply = [&](auto jc, int i, const Frags& x, const Scales& c) __attribute__((always_inline)) {
    constexpr int j = decltype(jc)::value;
    const int f = PARTS == 1 ? i / MF : i % NF, m = PARTS == 1 ? i % MF : i / (NF * PARTS);
    i32x8 a = mx_operand(x.a[m][0], x.a[m][AB / 64 - 1], AB == 64);
    if constexpr (PARTS == 2) {
      if (i % (NF * PARTS) == 0) {
        large = mx_large(a);
        rest = a ^ large;
      }
      a = i / NF % PARTS == 0 ? large : rest;
    }
    acc[f][m] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
        mx_operand(x.w[f], x.w[f], true), a, acc[f][m], 4, AF == MOE_MX_FP4 ? 4 : 0, 2 * j, c.w[f],
        2 * j, c.a[m]);
    asm volatile("" : "+v"(acc[f][m])::"memory");
  };
  const std::integral_constant<int, 0> first;
  const std::integral_constant<int, 1> second;
  constexpr int EACH = (PIECES + PRODUCTS - 1) / PRODUCTS;       // pieces read beside a product
  constexpr int FILL = (AI + WI + PRODUCTS - 1) / PRODUCTS;      // DMA instructions beside one
  Frags x0, x1;
  Scales c0, c1;
  // Loads of a wave complete in order: with at most so many left, the stage before the last NST - 2
  // has arrived (scales among them only make the wait stricter).
  constexpr int IN_FLIGHT = (NST - 2) * (AI + WI);
#pragma unroll
  for (int s = 0; s < NST; ++s) {
    issue_scales(s);
#pragma unroll
    for (int i = 0; i < AI + WI; ++i) issue(s, s, i);
  }
  wait_vmcnt<IN_FLIGHT + AI + WI>();
  barrier_lds();
  // a wave whose rows or columns lie past the end (an expert's last tile) only brings its share
  if (wm * WM >= t.rows || n0 + wn * out_cols<WN, SWIGLU>() >= p.N) {
    for (int s = 0, at = 0; s < stages; ++s, at = at + 1 == NST ? 0 : at + 1) {
      wait_vmcnt<IN_FLIGHT>();
      barrier_lds();
      issue_scales(s + NST);
#pragma unroll
      for (int i = 0; i < AI + WI; ++i) issue(s + NST, at, i);
    }
    wait_vmcnt<0>();
    return;
  }
  load_scales(0, c0);
#pragma unroll
  for (int i = 0; i < PIECES; ++i) load(0, first, i, x0);
  int at = 0;  // the place of stage s
  for (int s = 0; s < stages; ++s) {
#pragma unroll
    for (int i = 0; i < PRODUCTS; ++i) {
#pragma unroll
      for (int n = 0; n < EACH; ++n) load(at, second, EACH * i + n, x1);
      multiply(first, i, x0, c0);
    }
    wait_vmcnt<IN_FLIGHT>();
    barrier_lds();
    const int next = at + 1 == NST ? 0 : at + 1;
    c1 = c0;
    load_scales(s + 1, c0);  // past the last stage: not used
    issue_scales(s + NST);
#pragma unroll
    for (int i = 0; i < PRODUCTS; ++i) {
      multiply(second, i, x1, c1);
#pragma unroll
      for (int n = 0; n < EACH; ++n) load(next, first, EACH * i + n, x0);
#pragma unroll
      for (int n = 0; n < FILL; ++n)
        if (FILL * i + n < AI + WI) issue(s + NST, at, FILL * i + n);
    }
    at = next;
  }
  wait_vmcnt<0>();

  // Lane (r, g) holds row r's columns 8 q + 4 g + i at register 4 q + i. Rounded to the output's type
  // these are words of two or four columns; after swapping halves of them with its partner it holds
  // the 16 columns from 16 g on. (Swapped before the rounding and SwiGLU, two or four times the words:
  // the experts above 517 us against 513.)
  auto swap = [](uint32_t a, uint32_t b, uint32_t& lo, uint32_t& hi) __attribute__((always_inline)) {
    const auto x = __builtin_amdgcn_permlane32_swap(a, b, false, false);
    lo = x[0];
    hi = x[1];
  };

  constexpr int OF = SWIGLU ? NF / 2 : NF;  // fragments of output columns
#pragma unroll
  for (int m = 0; m < MF; ++m) {
    const int local = wm * WM + m * 32 + r;
    const bool there = local < t.rows;
    const int64_t row = t.row0 + local;
#pragma unroll
    for (int f = 0; f < OF; ++f) {
      float lo[8], hi[8];  // q = 0 and 1, q = 2 and 3
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        lo[i] = acc[f][m][i];
        hi[i] = acc[f][m][8 + i];
        if constexpr (SWIGLU) {
          lo[i] = swiglu(lo[i], acc[f + NF / 2][m][i]);
          hi[i] = swiglu(hi[i], acc[f + NF / 2][m][8 + i]);
        }
      }
      const int base = n0 + wn * (OF * 32) + f * 32, col = base + 16 * g;
      if constexpr (OUT == kMxOut8) {
        uint32_t amax = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          amax = max(amax, max(__float_as_uint(lo[i]) & 0x7fffffffu, __float_as_uint(hi[i]) & 0x7fffffffu));
        uint32_t a0, a1;
        swap(amax, amax, a0, a1);
        const uint32_t sb = mx_scale_of<MOE_MX_FP8>(max(a0, a1));
        const uint2 c0 = mx_encode8<MOE_MX_FP8>(lo, sb), c1 = mx_encode8<MOE_MX_FP8>(hi, sb);
        uint4 out;
        swap(c0.x, c1.x, out.x, out.y);
        swap(c0.y, c1.y, out.z, out.w);
        if (there && base < p.N) {
          *reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.y) + row * p.N + col) = out;
          if (g == 0) {
            const int cols = static_cast<int>(mx_scale_cols(p.N));
            uint8_t* s = p.y_scales + row * cols;
            s[base / 32] = static_cast<uint8_t>(sb);
            if (base + 32 == p.N)
              for (int i = p.N / 32; i < cols; ++i) s[i] = 0;
          }
        }
      } else {
        Row8<Out16<OUT>> w0, w1;
        w0.set(lo);
        w1.set(hi);
        uint4 out[2];
        swap(w0.a.x, w1.a.x, out[0].x, out[0].z);
        swap(w0.a.y, w1.a.y, out[0].y, out[0].w);
        swap(w0.a.z, w1.a.z, out[1].x, out[1].z);
        swap(w0.a.w, w1.a.w, out[1].y, out[1].w);
        Out16<OUT>* y = static_cast<Out16<OUT>*>(p.y) + row * p.N + col;
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (there && col + 8 * h < p.N) *reinterpret_cast<uint4*>(y + 8 * h) = out[h];
      }
    }
  }
}

// ------------------------------------------------------------------ few rows: weights streamed
// A block takes up to 16 rows and 16 or 32 output columns; its waves split the reduction and meet in
// LDS, adding in order. Weights come straight from HBM into the matrix cores' registers, each byte once
// for 16 rows, in batches of four steps of 128 elements with the next batch on its way: a row's four
// steps are 256 bytes of codes and 16 of scales. Loads go by buffer resources, whose bounds make
// zeros of steps past the operand; what a batch reads behind its own steps is not multiplied. One
// token of 4 of 32 experts, 2880 -> 2 x 2880, 11.5 us (3.1 TB/s; in one part 10.3): bound by a chain of
// latencies, the offsets, the scan over the experts, then the tile's weights (and rows[], then a). A
// wave's six steps are two batches, the second on its way while the first is multiplied. Into 8 bits 14.6
// us (13.1): with 32 columns a block there are half the blocks, at one wave a SIMD.
constexpr int kSmallRows = 16, kSmallWaves = 4, kBatch = 4;

// Output columns of a block: as few as there can be, so that even one token's experts give every CU
// several blocks; 32 where they share a scale. (32 columns for 16-bit results: 64 tokens of 4 of 32
// experts, 2880 x 2880 gate and up, 92 us against 76; one token 10.3 against 10.2.)
template <int OUT>
constexpr int small_cols() { return OUT == kMxOut8 ? 32 : 16; }

template <int AF, int PARTS, int OUT, bool SWIGLU>
__global__ __launch_bounds__(kSmallWaves * 64) void mx_rows_kernel(MxGemm p) {
  constexpr int COLS = small_cols<OUT>(), OF = COLS / 16, NF = SWIGLU ? 2 * OF : OF;
  constexpr int AB = row_bytes_of<AF>(128), AC = AB / 64;  // bytes a step; 16-byte pieces a lane
  constexpr int LD = 20;  // floats between a row's fragments' columns, off the banks' period
  __shared__ float red[kSmallWaves][NF][16][LD];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  MxTile t;
  if (!find_tile<kSmallRows, false>(p, blockIdx.x, t)) return;
  const int n0 = t.n * COLS, n_w = SWIGLU ? 2 * p.N : p.N;
  const int a_row = row_bytes_of<AF>(p.K), w_row = p.K / 2;
  const int sc = static_cast<int>(mx_scale_cols(p.K));
  const int r = lane & 15, g = lane >> 4;
  const bool act = r < t.rows;
  int64_t arow = t.row0 + (act ? r : 0);  // a's row of this lane
  int pair = 0;
  if (p.rows) pair = p.rows[arow];

  auto resource = [](const uint8_t* base, int64_t bytes) __attribute__((always_inline)) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(base), static_cast<short>(0),
                                             clamp_records(bytes), 0x00020000);
  };
  const int64_t w_first = static_cast<int64_t>(t.e) * n_w;
  const auto rw = resource(p.w + w_first * w_row, static_cast<int64_t>(n_w) * w_row);
  const auto rsw = resource(p.w_scales + w_first * sc, static_cast<int64_t>(n_w) * sc);
  uint32_t vw[NF], vsw[NF];
#pragma unroll
  for (int f = 0; f < NF; ++f) {
    const int n = n0 + 16 * (f % OF) + r;  // SwiGLU: the gate's fragments, then those of up
    const uint32_t row = n + f / OF * p.N;
    vw[f] = n < p.N ? row * w_row + g * 16 : kOOB;
    vsw[f] = n < p.N ? row * sc : kOOB;
  }
  const int steps = (p.K + 127) / 128, each = (steps + kSmallWaves - 1) / kSmallWaves;
  const int first = wave * each, last = min(steps, first + each);
  struct Batch {
    i32x4 w[kBatch][NF], sw[NF], a[kBatch][AC], sa;
  };
  auto load_w = [&](int s0, Batch& x) __attribute__((always_inline)) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      // pieces past the row's end are zeros
      const uint32_t end = (s0 + u) * 64 + g * 16 < w_row ? 0u : kOOB;
#pragma unroll
      for (int f = 0; f < NF; ++f)
        x.w[u][f] = __builtin_bit_cast(
            i32x4, __builtin_amdgcn_raw_buffer_load_b128(rw, vw[f] | end, (s0 + u) * 64, 0));
    }
#pragma unroll
    for (int f = 0; f < NF; ++f)
      x.sw[f] = __builtin_bit_cast(
          i32x4, __builtin_amdgcn_raw_buffer_load_b128(rsw, vsw[f], s0 * 4, 0));
  };
  Batch x0, x1;
  if (first < last) load_w(first, x0);
  if (p.rows) arow = static_cast<uint32_t>(pair) / static_cast<uint32_t>(p.k);
  // a tile's rows lie together, or are anywhere in a gathered a (below 2 GiB)
  const int64_t a_first = p.rows ? 0 : t.row0;
  const auto ra = resource(p.a + a_first * a_row, (p.a_rows - a_first) * a_row);
  const auto rsa = resource(p.a_scales + a_first * sc, (p.a_rows - a_first) * sc);
  const bool a_ok = act && arow < p.a_rows;
  const uint32_t va = a_ok ? static_cast<uint32_t>(arow - a_first) * a_row + g * 16 : kOOB;
  const uint32_t vsa = a_ok ? static_cast<uint32_t>(arow - a_first) * sc : kOOB;
  auto load_a = [&](int s0, Batch& x) __attribute__((always_inline)) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
#pragma unroll
      for (int c = 0; c < AC; ++c) {
        const int byte = (s0 + u) * AB + c * 64;
        const uint32_t end = byte + g * 16 < a_row ? 0u : kOOB;
        x.a[u][c] = __builtin_bit_cast(
            i32x4, __builtin_amdgcn_raw_buffer_load_b128(ra, va | end, byte, 0));
      }
    x.sa = __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(rsa, vsa, s0 * 4, 0));
  };
  f32x4 acc[NF] = {};
  auto multiply = [&](int s0, const Batch& x) __attribute__((always_inline)) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (s0 + u >= last) break;
      const i32x8 all = mx_operand(x.a[u][0], x.a[u][AC - 1], AC == 1);
      auto products = [&](const i32x8& fa) __attribute__((always_inline)) {
#pragma unroll
        for (int f = 0; f < NF; ++f)
          acc[f] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
              mx_operand(x.w[u][f], x.w[u][f], true), fa, acc[f], 4, AF == MOE_MX_FP4 ? 4 : 0, 0,
              x.sw[f][u] >> (8 * g), 0, x.sa[u] >> (8 * g));
      };
      if constexpr (PARTS == 1) {
        products(all);
      } else {
        const i32x8 large = mx_large(all);
        products(large);
        products(all ^ large);
      }
    }
  };
  if (first < last) load_a(first, x0);
  for (int s0 = first; s0 < last; s0 += 2 * kBatch) {
    if (s0 + kBatch < last) {
      load_w(s0 + kBatch, x1);
      load_a(s0 + kBatch, x1);
    }
    multiply(s0, x0);
    if (s0 + 2 * kBatch < last) {
      load_w(s0 + 2 * kBatch, x0);
      load_a(s0 + 2 * kBatch, x0);
    }
    multiply(s0 + kBatch, x1);
  }
  // lane (r, g) has row r, columns 4 g .. 4 g + 3
#pragma unroll
  for (int f = 0; f < NF; ++f)
    *reinterpret_cast<f32x4*>(&red[wave][f][r][4 * g]) = acc[f];
  __syncthreads();
  // CPT columns a thread
  constexpr int CPT = COLS / 16;
  const int m = threadIdx.x >> 4, c = (threadIdx.x & 15) * CPT, col = n0 + c;
  auto total = [&](int f, int at) __attribute__((always_inline)) {
    float v = red[0][f][m][at];
#pragma unroll
    for (int w = 1; w < kSmallWaves; ++w) v += red[w][f][m][at];
    return v;
  };
  float v[CPT];
#pragma unroll
  for (int i = 0; i < CPT; ++i) {
    v[i] = total(c >> 4, (c & 15) + i);
    if constexpr (SWIGLU) v[i] = swiglu(v[i], total(OF + (c >> 4), (c & 15) + i));
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
    static_assert(CPT == 1, "a column a thread");
    static_cast<Out16<OUT>*>(p.y)[row * p.N + col] = from_f32<Out16<OUT>>(v[0]);
  }
}

// Which kernel takes a call, measured on both sides of each line with an 8-bit a in one part and
// [in two].
//  Few rows: while its blocks (in units of 16 output columns) are at most three [four] a CU, since
//  weights are read again for every 16 rows. 4096 -> 2880, 64 rows 11.9 us against 14.5 of the smallest
//  tiles [12.9 / 21.3], 96 rows 18.3 against 14.7 [19.5 / 21.4]; 8192 -> 8192, 16 rows 15.3 / 25.3
//  [16.5 / 37], 32 rows 27.5 / 24.9 [29.4 / 37]; SwiGLU 2880 -> 2880 of 4 of 32 experts, one token
//  10.5 / 13.2 [11.5 / 17.9], 8 tokens 41.9 / 36.7 [44.8 / 43.8].
//  Larger tiles, which read less from L2 for a product: where they give three quarters of the CUs a
//  tile, and experts on average rows for half of one. 4096 -> 2880, 256 x 256 against 128 x 128:
//  4096 rows (192 tiles) 51.6 / 54.8 us [81.5 / 87], 2048 rows 43.4 / 31.4 [80 / 57]; the experts
//  above, 1024 tokens (128 rows each) 122.6 / 143.0 [177 / 176], 768 tokens 114.7 / 103.5 [136 / 138].
//  128 x 128 against 64 x 128: 1024 rows (184 tiles) 20.1 / 21.4 [33.6 / 31.6], 512 rows 17.8 / 15.6
//  [31.8 / 23.1]; the experts, 512 tokens (64 rows each) 93.5 / 111.8 [118 / 121], 256 tokens 81 / 75
//  [109 / 86].
//  256 x 192 in the place of 256 x 256 where the last round of tiles would leave many CUs idle, so
//  that rounds times columns fall by a tenth or more (without SwiGLU, whose halves of 96 rows no
//  instruction's step divides): 8192 rows of 4096 -> 2880 (480 tiles for 384) 87.3 us against 97.6
//  [140 / 160], in 4 bits 69.5 / 74.2; 2048 tokens of 4 of 32 experts, 2880 -> 2880, 94.4 / 106.3
//  [157 / 179], 8192 tokens [458 / 432]. Rounds are counted as if only the last of all tiles were not
//  full: what each expert's last tile adds is not known on the host.
constexpr int kCUs = 256, kTilesToFill = kCUs * 3 / 4;

// Calls go with the format of a, its parts, the output and SwiGLU as constants.
template <typename F>
hipError_t by_product(const moe_mx_linear_shape& s, F&& go) {
  using std::integral_constant;
  auto operand = [&](auto af, auto parts) {
    auto out = [&](auto o) {
      return s.swiglu ? go(af, parts, o, integral_constant<bool, true>())
                      : go(af, parts, o, integral_constant<bool, false>());
    };
    if (s.out == MOE_MX_OUT_FP8) return out(integral_constant<int, kMxOut8>());
    if (s.out == MOE_BF16) return out(integral_constant<int, 1>());
    return out(integral_constant<int, 0>());
  };
  typedef integral_constant<int, 1> One;
  typedef integral_constant<int, 2> Two;
  if (s.a_format == MOE_MX_FP4) return operand(integral_constant<int, MOE_MX_FP4>(), One());
  if (s.fast) return operand(integral_constant<int, MOE_MX_FP8>(), One());
  return operand(integral_constant<int, MOE_MX_FP8>(), Two());
}

}  // namespace

hipError_t launch_mx_linear(const moe_mx_linear_shape& s, const void* a, const uint8_t* a_scales,
                            const int32_t* rows, const int32_t* offsets, const void* w,
                            const uint8_t* w_scales, void* y, uint8_t* y_scales, hipStream_t st,
                            KernelTimer* tm) {
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
  return by_product(s, [&](auto af, auto parts, auto out, auto glu) {
    constexpr int AF = decltype(af)::value, PARTS = decltype(parts)::value, OUT = decltype(out)::value;
    constexpr bool GLU = decltype(glu)::value;
    // at most this many tiles of bm rows and bn weight rows, whatever the experts' counts are
    auto tiles = [&](int bm, int cols) {
      p.ntn = (s.N + cols - 1) / cols;
      return static_cast<int64_t>(s.E > 0 ? p.M / bm + experts : (p.M + bm - 1) / bm) * p.ntn;
    };
    auto tiled = [&](auto bm, auto bn, auto wm, auto wn, auto nst) {
      constexpr int BM = decltype(bm)::value, BN = decltype(bn)::value;
      constexpr int WM = decltype(wm)::value, WN = decltype(wn)::value;
      hipLaunchKernelGGL((mx_gemm_kernel<AF, PARTS, OUT, GLU, BM, BN, WM, WN, decltype(nst)::value>),
                         dim3(static_cast<unsigned>(tiles(BM, out_cols<BN, GLU>()))),
                         dim3((BM / WM) * (BN / WN) * 64), 0, st, p);
    };
    // rounds of a tile a CU that 256 x bn tiles take, in columns
    auto rounds = [&](int bn) {
      const int64_t n = (p.M + 255) / 256 * static_cast<int64_t>((s.N + bn - 1) / bn);
      return (n + kCUs - 1) / kCUs * bn;
    };
    auto fills = [&](int bm, int bn) {
      const int cols = GLU ? bn / 2 : bn;
      return p.M >= bm / 2 * static_cast<int64_t>(experts) &&
             p.M / bm * static_cast<int64_t>((s.N + cols - 1) / cols) >= kTilesToFill;
    };
    using std::integral_constant;
    if (tiles(kSmallRows, small_cols<OUT>()) * (small_cols<OUT>() / 16) <= (PARTS == 2 ? 4 : 3) * kCUs) {
      hipLaunchKernelGGL((mx_rows_kernel<AF, PARTS, OUT, GLU>),
                         dim3(static_cast<unsigned>(tiles(kSmallRows, small_cols<OUT>()))),
                         dim3(kSmallWaves * 64), 0, st, p);
    } else if (!GLU && fills(256, 256) && rounds(192) * 10 < rounds(256) * 9) {
      if constexpr (!GLU)
        tiled(integral_constant<int, 256>(), integral_constant<int, 192>(), integral_constant<int, 64>(),
              integral_constant<int, 96>(), integral_constant<int, 3>());
    } else if (fills(256, 256)) {
      tiled(integral_constant<int, 256>(), integral_constant<int, 256>(), integral_constant<int, 64>(),
            integral_constant<int, 128>(), integral_constant<int, 3>());
    } else if (fills(128, 128)) {
      tiled(integral_constant<int, 128>(), integral_constant<int, 128>(), integral_constant<int, 64>(),
            integral_constant<int, 64>(), integral_constant<int, 3>());
    } else {
      tiled(integral_constant<int, 64>(), integral_constant<int, 128>(), integral_constant<int, 32>(),
            integral_constant<int, 64>(), integral_constant<int, 4>());
    }
    return hipGetLastError();
  });
}

}  // namespace moe
