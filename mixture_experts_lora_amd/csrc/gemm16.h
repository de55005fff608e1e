// The 16-bit MFMA GEMM template (gemm16) with its operand descriptions, LDS layouts and epilogue
// helpers, shared by the grouped expert products (gemm.hip, which describes the modes) and the
// dense linear operator (linear.hip).
#pragma once

#include <algorithm>
#include <type_traits>

#include "device_common.h"
#include "launch.h"
#include "linear.h"

namespace moe {

namespace {

enum Mode { GROUP_M = 0, GROUP_K = 1, GROUP_KV = 2 };
// EPI_STORE_F32: float32 output (router logits); EPI_ADD: out = src + result
// with src = aux when given (merged export: W + s B A) else out itself (an
// accumulate); the sum formed in float32, one rounding. EPI_LINEAR: one dense
// product instead of a group per expert: no tile list or offsets, E slices of
// kchunk along the reduction, the output through linear_finish8 (GROUP_M) or
// stored (GROUP_K), or float32 partials [E][M][N] when E > 1.
enum Epi {
  EPI_STORE = 0, EPI_SWIGLU = 1, EPI_SWIGLU_BWD = 2, EPI_STORE_F32 = 3, EPI_ADD = 4,
  EPI_LINEAR = 5
};

struct Opnd {
  const void* ptr;
  int64_t estride;  // elements between consecutive experts (0: not per expert)
  int64_t ld;       // leading dimension in elements
  int kcontig;      // 1: (mn, k) at ptr[mn*ld + k]; 0: at ptr[k*ld + mn]
  int vec;          // 16-byte chunks allowed (alignment and extents are multiples of 8)
  // Gathered rows (the layer input read in token order): row i of the
  // permuted order is row rows[i] / rows_div of ptr, which holds rows_bytes
  // bytes. Null rows: the operand's rows are in permuted order. Gathered
  // are the A operand of GROUP_M (rows along mn: x or dY) and, in the weight
  // gradients, the operand whose rows run along k (dY as A of dB_d, x as B of
  // dA_gu and dW_gu).
  const int32_t* rows;
  int rows_div;
  int64_t rows_bytes;
};

struct GemmArgs {
  Opnd a[2], b[2];  // [0] main segment, [1] LoRA segment (GROUP_M only)
  int K[2];         // GROUP_M: K extent of each segment (K[1] may be 0)
  int M, N;         // GROUP_K: output extent; GROUP_M: N = output columns (features)
  int E;
  const int32_t* offsets;  // [E+1]
  const int4* tiles;       // GROUP_M: {expert, first row, valid rows, raster group}
  const int32_t* ntiles;   // GROUP_M: number of M tiles (device)
  int ntn;                 // number of N tiles
  int ntm;                 // GROUP_K: number of M tiles
  void* out;
  int64_t out_estride;  // GROUP_K: elements between experts in `out`
  int64_t ld_out;
  void* out2;  // EPI_SWIGLU: act
  int64_t ld_out2;
  const void* aux;  // EPI_SWIGLU_BWD: h
  int64_t ld_aux;
  int I;  // gate width for SwiGLU epilogues / paired weight rows
  float scale;
  int dtype;  // host side only: MOE_BF16 or MOE_F16 picks the 16-bit kernel
  // GROUP_KV: B of the side product (per expert [M, N] row-major, expert e of
  // the launch uses B[e / vsplit]) and its float32 partials vp[M tile][row][N]
  const void* vb;
  int64_t vb_estride;
  float* vp;
  int64_t vp_tstride;  // elements between M tiles of vp
  int vsplit;
  // EPI_SWIGLU_BWD (GROUP_M), both optional: roww[row] scales the product
  // before the SwiGLU derivative (dAct = w * acc); dwp receives, per output
  // row, float32 partial sums of acc * act over each wave's column slice
  // (at dwp[row * dwp_slots + n_tile * (BN / WN) + wave column]), act being
  // SwiGLU(h) recomputed from the h the epilogue loads.
  const float* roww;
  float* dwp;
  int dwp_slots;
  // EPI_LINEAR: M output rows, reduction length K[0] in slices of kchunk
  int kchunk;
  LinearEpi lin;
};

// Spread `total` logical tiles over the 8 XCDs so that each XCD works on a
// contiguous range of them (workgroup b is dispatched to XCD b % 8).
__device__ __forceinline__ int xcd_remap(int b, int total) {
  const int x = b & 7, j = b >> 3, q = total >> 3, rem = total & 7;
  return x * q + (x < rem ? x : rem) + j;
}

// Tile-list entries are {expert, first row, valid rows, group}: an expert's M
// tiles form groups of at most 8 consecutive entries, and `group` holds the
// group's first entry times 16 plus its size. Logical tiles L = gs * ntn ..
// (gs + gsz) * ntn - 1 belong to the group starting at entry gs, M tile
// fastest, so L / ntn is always one of that group's entries. Returns the
// entry of logical tile L and sets its N tile.
constexpr int kTileGroup = 8;
__device__ __forceinline__ int group_tile(const int4* tiles, int L, int ntn, int& n_tile) {
  const int g = tiles[L / ntn].w;
  const int gs = g >> 4, gsz = g & 15;
  const int rem = L - gs * ntn;
  n_tile = rem / gsz;
  return gs + rem % gsz;
}

// EPI_LINEAR's slice, N tile and first row of this block: the tile lists' raster (up to 8 M tiles
// swept across the N tiles) without a list. False: a block past the last tile.
__device__ __forceinline__ bool dense_tile(const GemmArgs& p, int bm, int& e, int& n_tile,
                                           int& m0) {
  const int per = p.ntm * p.ntn, total = p.E * per;
  if (static_cast<int>(blockIdx.x) >= total) return false;
  const int L = xcd_remap(blockIdx.x, total);
  e = L / per;
  const int at = L - e * per;
  const int gs = at / (kTileGroup * p.ntn) * kTileGroup, gsz = min(kTileGroup, p.ntm - gs);
  const int rem = at - gs * p.ntn;
  n_tile = rem / gsz;
  m0 = (gs + rem % gsz) * bm;
  return true;
}

// One operand of one tile: where element (mn, k) lives and which ones exist.
template <typename T>
struct View {
  const T* base;
  int64_t ld;
  int kcontig, vec;
  int klim;    // valid k in [0, klim)
  int mn_lim;  // valid local mn in [0, mn_lim) (simple mapping)
  int paired;  // gate_up weight rows: local n < half -> gate row pbase+n, else up row I+pbase+n-half
  int half, pbase, I;
  // gathered rows (Opnd::rows from this tile's first row on, and its divisor):
  // mn (k-contiguous) or k (output-contiguous) index i is row grow[i] / gk of base
  const int32_t* grow;
  int gk;
};

template <typename T>
__device__ __forceinline__ int64_t map_mn(const View<T>& v, int n, bool& ok) {
  if (!v.paired) {
    ok = n < v.mn_lim;
    return n;
  }
  const int f = v.pbase + (n < v.half ? n : n - v.half);
  ok = f < v.I;
  return n < v.half ? f : v.I + f;
}

template <typename T>
__device__ __forceinline__ int64_t gathered_row(const View<T>& v, int64_t i) {
  return v.grow ? static_cast<int64_t>(static_cast<uint32_t>(v.grow[i]) / static_cast<uint32_t>(v.gk))
                : i;
}

template <typename T>
__device__ __forceinline__ T load_elem(const View<T>& v, int n, int k) {
  bool ok;
  const int64_t g = map_mn(v, n, ok);
  if (!ok || k >= v.klim) return T(0);
  return v.kcontig ? v.base[gathered_row(v, g) * v.ld + k]
                   : v.base[gathered_row(v, k) * v.ld + g];
}

// ----------------------------------------------------------------- epilogue helpers
// Four consecutive columns [col, col+4) of one row; ragged column tails and
// unaligned rows fall back to element stores.
template <typename T>
__device__ __forceinline__ void store4(T* rowp, int col, int ncols, bool aligned,
                                       const float (&v)[4]) {
  if (aligned && col + 4 <= ncols) {
    Vec4<T>::store(rowp + col, v);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (col + j < ncols) rowp[col + j] = from_f32<T>(v[j]);
  }
}

template <typename T, int MODE, int EPI>
__device__ __forceinline__ void epi_store(const GemmArgs& p, int e, int64_t row0, int m_local,
                                          int rows, int n_col, const float (&v)[4]) {
  if (m_local >= rows) return;
  if (MODE == GROUP_M) {
    const int64_t row = row0 + m_local;
    if (EPI == EPI_STORE || EPI == EPI_STORE_F32 || EPI == EPI_ADD) {
      float o[4];
      T* rp = static_cast<T*>(p.out) + row * p.ld_out;
      const T* sp = EPI == EPI_ADD && p.aux ? static_cast<const T*>(p.aux) + row * p.ld_aux : rp;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        o[j] = v[j] * p.scale;
        if (EPI == EPI_ADD && n_col + j < p.N) o[j] += to_f32<T>(sp[n_col + j]);
      }
      store4<T>(rp, n_col, p.N, (p.ld_out & 3) == 0, o);
    }
  } else {
    // GROUP_K: out[e][m][n], row = feature m (rows = valid M in this tile)
    float o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = v[j] * p.scale;
    T* rp = static_cast<T*>(p.out) + static_cast<int64_t>(e) * p.out_estride +
            (row0 + m_local) * p.ld_out;
    store4<T>(rp, n_col, p.N, (p.ld_out & 3) == 0, o);
  }
}

template <typename T>
__device__ __forceinline__ void epi_swiglu(const GemmArgs& p, int64_t row0, int m_local,
                                           int rows, int f, const float (&g)[4],
                                           const float (&u)[4]) {
  if (m_local >= rows || f >= p.I) return;  // I multiple of 8: groups of 4 all in or all out
  const int64_t row = row0 + m_local;
  T* hr = static_cast<T*>(p.out) + row * p.ld_out;
  float a[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) a[j] = swiglu(g[j], u[j]);
  Vec4<T>::store(hr + f, g);
  Vec4<T>::store(hr + p.I + f, u);
  Vec4<T>::store(static_cast<T*>(p.out2) + row * p.ld_out2 + f, a);
}

// ----------------------------------------------------------------- bf16 MFMA kernel
// LDS tiles are BK (32 or 64) deep in k, unpadded, with 16-byte-chunk XOR swizzles:
//   k-contiguous tile [R][BK]: row r keeps k-chunk c at position c ^ kswz<BK>(r)
//   n-contiguous tile [BK][R]: k-row k keeps n-chunk c at position c ^ nswz<R>(k)
// chosen so that every 256-byte group of a fragment read (16 lanes of
// ds_read_b128, 32 lanes of ds_read_b64_tr_b16) touches each LDS bank once.
// Both layouts yield the same MFMA fragment: lane l holds 8 consecutive k
// (block l/32) of the row or column l%32 (the transpose read, CDNA4's
// ds_read_b64_tr_b16, gathers them from the k-major tile). Tiles are filled by
// buffer->LDS DMA with no register staging: each wave instruction writes 1 KB
// of LDS, lane l at +16 l, from a per-lane byte offset that encodes the
// swizzle; lanes outside the operand get an out-of-range offset and the
// hardware writes zeros. NST LDS stages keep NST-1 tiles in flight while one
// is multiplied.
constexpr uint32_t kOOB = 0x80000000u;

typedef __attribute__((address_space(3))) void lds_void;
typedef short v4s __attribute__((ext_vector_type(4)));
typedef short v8s __attribute__((ext_vector_type(8)));

template <int BK>
__device__ __forceinline__ int kswz(int row) {
  return BK == 64 ? ((row >> 1) & 7) : ((row >> 2) & 3);
}

template <int R>
__device__ __forceinline__ int nswz(int k) {
  // 192: rows of 24 chunks, whose last 8 a swizzle within 8 chunks keeps in the row; they shift the
  // banks as rows of 64 do
  return R == 64 || R == 192 ? (((k >> 1) & 1) << 2) : R >= 128 ? ((k & 3) << 2) : 0;
}

template <int N>
__device__ __forceinline__ void wait_vmcnt() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// Own LDS traffic finished, then a workgroup barrier.
__device__ __forceinline__ void barrier_lds() {
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// Buffer resource (V#) over [base, base + nrec bytes): raw, stride 0.
__device__ __forceinline__ u32x4 buffer_rsrc(const void* base, int nrec) {
  const uint64_t b = reinterpret_cast<uint64_t>(base);
  u32x4 r;
  r[0] = static_cast<uint32_t>(b);
  r[1] = static_cast<uint32_t>(b >> 32) & 0xffffu;
  r[2] = static_cast<uint32_t>(nrec);
  r[3] = 0x00020000u;
  return r;
}

// 16 bytes per lane, global -> LDS: lane l's bytes land at lds + 16 l. The
// instruction is issued from inline asm so that the compiler does not treat
// it as an LDS store it must wait for before every later LDS read (it would
// insert s_waitcnt vmcnt(0) and drain all tiles in flight); completion is
// tracked by the explicit vmcnt waits of the pipeline instead. The asm has no
// outputs, so no register is ever written by a load still in flight.
__device__ __forceinline__ void dma16(const char* lds, const u32x4& rs, uint32_t vo,
                                      uint32_t soff) {
  const uint32_t m0 = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(
      reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) const char*)(lds))));
  // resource and offset are wave-uniform; make that explicit for the SGPR operands
  u32x4 srs;
  srs[0] = __builtin_amdgcn_readfirstlane(rs[0]);
  srs[1] = __builtin_amdgcn_readfirstlane(rs[1]);
  srs[2] = __builtin_amdgcn_readfirstlane(rs[2]);
  srs[3] = __builtin_amdgcn_readfirstlane(rs[3]);
  const uint32_t ssoff = __builtin_amdgcn_readfirstlane(soff);
  // s_nop 4: the resource/offset SGPRs may have just been written by VALU
  // (v_readfirstlane), which a VMEM read may only follow after 5 wait states,
  // and M0 needs 1 wait state before an LDS DMA; the compiler's hazard
  // recognizer does not look inside inline asm, so the asm provides both.
  asm volatile("s_nop 4\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds" ::"{m0}"(m0), "v"(vo),
               "s"(srs), "s"(ssoff)
               : "memory");
}

__device__ __forceinline__ int clamp_records(int64_t bytes) {
  return bytes <= 0 ? 0 : (bytes > 0x7fffffff ? 0x7fffffff : static_cast<int>(bytes));
}

// Fill geometry of one operand tile of ROWS rows (or columns) x BK, filled
// by NW waves in 1 KB wave instructions (16 bytes per lane).
template <int ROWS, int BK, bool KC, int NW>
struct Geo {
  static constexpr int TI = ROWS * BK * 2 / 1024;  // 1 KB instructions per tile
  static constexpr int NIW = (TI + NW - 1) / NW;   // per wave (upper bound)
  static constexpr int MINW = TI / NW;             // issued by every wave
  static constexpr int CPR = KC ? BK / 8 : ROWS / 8;        // chunks per LDS row
  static constexpr int RPI = KC ? 512 / BK : 512 / ROWS;    // LDS rows per instruction
  // Row and chunk position that lane `lane` of instruction j fills. Where an instruction fills
  // whole rows the part that depends on j is kept apart, so that it folds into the instructions'
  // offsets (one form for both: up to 440 more instructions in a grouped product).
  __device__ static int row(int j, int lane) {
    return 64 % CPR == 0 ? RPI * j + lane / CPR : (64 * j + lane) / CPR;
  }
  __device__ static int pos(int j, int lane) {
    return 64 % CPR == 0 ? lane % CPR : (64 * j + lane) % CPR;
  }
};

// DMA plan of one operand tile: buffer (base, bytes), per-instruction lane offsets.
template <int ROWS, int BK, bool KC, int NW>
struct Plan {
  const void* base;
  int64_t bytes;  // extent of the operand from base
  int nrec;
  u32x4 rs;  // buffer resource over [base, base + nrec)
  uint32_t vo[Geo<ROWS, BK, KC, NW>::NIW];
  int vec;
  int klim;
  int64_t ld;
  View<bf16_t> view;  // element view for the slow (non-DMA) fill
};

template <int ROWS, int BK, bool KC, int NW>
__device__ __forceinline__ void make_plan(Plan<ROWS, BK, KC, NW>& P, const View<bf16_t>& v,
                                          int64_t bytes, int vec, int wave, int lane) {
  typedef Geo<ROWS, BK, KC, NW> G;
  P.view = v;
  P.vec = vec;
  P.klim = v.klim;
  P.ld = v.ld;
  P.base = v.base;
  P.bytes = bytes;
  P.nrec = clamp_records(bytes);
  P.rs = buffer_rsrc(v.base, P.nrec);
#pragma unroll
  for (int i = 0; i < G::NIW; ++i) {
    const int j = wave + NW * i;  // instruction index within the tile
    const int r = G::row(j, lane), p = G::pos(j, lane);
    uint32_t vo = kOOB;
    if (KC) {
      const int c = p ^ kswz<BK>(r);
      bool ok;
      const int64_t g = map_mn(v, r, ok);
      if (ok && r < ROWS) vo = static_cast<uint32_t>((gathered_row(v, g) * v.ld + c * 8) * 2);
    } else {
      // gathered: the offsets depend on the k tile's rows (gather_vo)
      const int cn = p ^ nswz<ROWS>(r);
      if (cn * 8 < v.mn_lim && r < BK && !v.grow) vo = static_cast<uint32_t>((r * v.ld + cn * 8) * 2);
    }
    P.vo[i] = vo;
  }
}

// Buffer resource and scalar offset of the tile at k0. A k-contiguous
// operand keeps one resource (k0 is a small byte offset). An output-contiguous
// one advances along its rows: its resource starts at row k0 (64-bit address
// arithmetic) and covers the rest of the operand, so neither the 32-bit scalar
// offset nor the 2^31-byte record count limits how many rows it spans (a
// weight gradient runs over all of an expert's rows).
template <int ROWS, int BK, bool KC, int NW>
__device__ __forceinline__ u32x4 tile_rsrc(const Plan<ROWS, BK, KC, NW>& P, int k0,
                                           uint32_t& soff) {
  if (KC) {
    soff = static_cast<uint32_t>(k0) * 2;
    return P.rs;
  }
  soff = 0;
  if (P.view.grow) return P.rs;  // gathered rows: per-lane offsets from the start
  const int64_t adv = static_cast<int64_t>(k0) * P.ld * 2;
  return buffer_rsrc(static_cast<const char*>(P.base) + adv, clamp_records(P.bytes - adv));
}

// Lane offset of instruction j of an output-contiguous tile at k0 whose rows
// are gathered: the instruction covers the tile's k rows RPI*j .. RPI*j+RPI-1
// (wave-uniform), whose row numbers come in through scalar loads (constant
// address space: they go through the scalar cache and are counted apart from
// the DMA loads in flight), so the DMA pipeline's vector-memory waits stay
// exact. table (optional): the byte offsets of the block's rows from row tw0
// on, in LDS (read instead of the scalar loads).
template <int ROWS, int BK, bool KC, int NW>
__device__ __forceinline__ uint32_t gather_vo(const Plan<ROWS, BK, KC, NW>& P, int k0, int j,
                                              int lane, const uint32_t* table = nullptr,
                                              int tw0 = 0) {
  typedef Geo<ROWS, BK, KC, NW> G;
  typedef const __attribute__((address_space(4))) int32_t* cptr;
  if (P.klim <= 0) return kOOB;
  const int r0 = k0 + G::RPI * j, last = P.klim - 1, t = lane / G::CPR;
  const int cn = (lane % G::CPR) ^ nswz<ROWS>(G::RPI * j + t);
  if (table) {
    const uint32_t off = table[min(r0 + t, last) - tw0];
    if (r0 + t > last || cn * 8 >= P.view.mn_lim) return kOOB;
    return off + static_cast<uint32_t>(cn) * 16;
  }
  const cptr rows = (cptr)(P.view.grow);
  int sp = 0;
#pragma unroll
  for (int q = 0; q < G::RPI; ++q) {
    const int v = rows[min(r0 + q, last)];
    if (t == q) sp = v;
  }
  if (r0 + t > last || cn * 8 >= P.view.mn_lim) return kOOB;
  const uint32_t row = static_cast<uint32_t>(sp) / static_cast<uint32_t>(P.view.gk);
  return static_cast<uint32_t>((static_cast<int64_t>(row) * P.ld + cn * 8) * 2);
}

// Issue one tile: DMA when possible, else an element-wise fill. GATH false:
// the operand is never gathered along k (no code for it).
template <int ROWS, int BK, bool KC, int NW, bool GATH = true>
__device__ __forceinline__ void fill(const Plan<ROWS, BK, KC, NW>& P, int k0, char* lds, int wave,
                                     int lane, const uint32_t* gtab = nullptr, int tw0 = 0) {
  typedef Geo<ROWS, BK, KC, NW> G;
  if (P.vec) {
    uint32_t soff;
    const u32x4 rs = tile_rsrc(P, k0, soff);
    const bool tail = KC && (k0 + BK > P.klim);  // n-contiguous tails hit the buffer bound
#pragma unroll
    for (int i = 0; i < G::NIW; ++i) {
      const int j = wave + NW * i;
      if (G::TI % NW == 0 || j < G::TI) {
        uint32_t vo = P.vo[i];
        if (GATH && !KC && P.view.grow) vo = gather_vo(P, k0, j, lane, gtab, tw0);
        if (tail) {
          const int r = G::RPI * j + lane / G::CPR;
          const int c = (lane % G::CPR) ^ kswz<BK>(r);
          if (k0 + c * 8 >= P.klim) vo = kOOB;
        }
        dma16(lds + j * 1024, rs, vo, soff);
      }
    }
  } else {
    bf16_t* t = reinterpret_cast<bf16_t*>(lds);
    for (int e = threadIdx.x; e < ROWS * BK; e += 64 * NW) {
      int byte;
      bf16_t val;
      if (KC) {
        const int row = e / BK, k = e % BK;
        byte = row * BK * 2 + (((k >> 3) ^ kswz<BK>(row)) << 4) + (k & 7) * 2;
        val = load_elem(P.view, row, k0 + k);
      } else {
        const int k = e / ROWS, mn = e % ROWS;
        byte = k * ROWS * 2 + (((mn >> 3) ^ nswz<ROWS>(k)) << 4) + (mn & 7) * 2;
        val = load_elem(P.view, mn, k0 + k);
      }
      t[byte >> 1] = val;
    }
  }
}

// One DMA instruction (index i of this wave's share) of a tile; DMA plans only.
// GIVEN: gvo is the lane offset, formed by the caller (the plan's own offset,
// or a gathered row's); GATH false: the operand is never gathered along k.
template <int ROWS, int BK, bool KC, int NW, bool GATH = true, bool GIVEN = false>
__device__ __forceinline__ void fill_one(const Plan<ROWS, BK, KC, NW>& P, int k0, char* lds,
                                         int wave, int lane, int i, uint32_t gvo = 0) {
  typedef Geo<ROWS, BK, KC, NW> G;
  const int j = wave + NW * i;
  if (G::TI % NW != 0 && j >= G::TI) return;
  uint32_t soff;
  const u32x4 rs = tile_rsrc(P, k0, soff);
  uint32_t vo = P.vo[i];
  if (GIVEN)
    vo = gvo;
  else if (GATH && !KC && P.view.grow)
    vo = gather_vo(P, k0, j, lane);
  if (KC && k0 + BK > P.klim) {  // k tail of a k-contiguous operand: mask by lane
    const int r = G::RPI * j + lane / G::CPR;
    const int c = (lane % G::CPR) ^ kswz<BK>(r);
    if (k0 + c * 8 >= P.klim) vo = kOOB;
  }
  dma16(lds + j * 1024, rs, vo, soff);
}

// A fill geometry tagged with its operand's k-contiguity (for generic lambdas).
template <typename G, bool KC>
struct GeoK : G {
  static constexpr bool KCV = KC;
};

// Per-lane LDS byte offsets of the MFMA fragments.
template <int ROWS, int BK, bool KC, int NFR>
struct FragAddr {
  int off[KC ? BK / 16 : NFR];  // KC: per k-step (shared by all fragments); NC: per fragment
};

template <int ROWS, int BK, bool KC, int NFR>
__device__ __forceinline__ void frag_addr(FragAddr<ROWS, BK, KC, NFR>& F,
                                          const int (&fr_base)[NFR], int lane) {
  if (KC) {
    const int h = lane >> 5, r = lane & 31;
#pragma unroll
    for (int ks = 0; ks < BK / 16; ++ks)
      F.off[ks] = r * BK * 2 + ((((2 * ks + h) ^ kswz<BK>(r))) << 4);
  } else {
    const int G = lane >> 4, li = lane & 15;
    const int kl = (G >> 1) * 8 + (li >> 2);  // k row of this lane in a k-step (first read)
#pragma unroll
    for (int f = 0; f < (KC ? 0 : NFR); ++f) {
      const int n = fr_base[f] + (G & 1) * 16 + (li & 3) * 4;
      F.off[KC ? 0 : f] = kl * ROWS * 2 + ((((n >> 3) ^ nswz<ROWS>(kl))) << 4) + (n & 7) * 2;
    }
  }
}

template <int ROWS, int BK, bool KC, int NFR>
__device__ __forceinline__ bf16x8 read_frag(const char* tile,
                                            const FragAddr<ROWS, BK, KC, NFR>& F, int f,
                                            int fr_base_f, int ks) {
  if (KC) {
    return *reinterpret_cast<const bf16x8*>(tile + fr_base_f * BK * 2 + F.off[ks]);
  } else {
    const char* p = tile + F.off[KC ? 0 : f] + ks * 16 * ROWS * 2;
    v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4s*)(p));
    v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (__attribute__((address_space(3))) v4s*)(p + 4 * ROWS * 2));
    v8s r = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    return __builtin_bit_cast(bf16x8, r);
  }
}

// ---- epilogue staging helpers
// A wave's float32 slab is 32 rows x WN columns; row r keeps 16-byte chunk c
// at c ^ sswz(r), so that 16 lanes writing one chunk column of 16 rows, or
// reading 16 row segments, hit distinct LDS banks.
template <int WN>
__device__ __forceinline__ int slab_off(int r, int c) {
  const int sw = WN >= 64 && WN % 64 == 0 ? (r & 15) : ((r >> 1) & 7);
  return r * WN * 4 + ((c ^ sw) << 4);
}

// Eight floats: chunks c and c+1 of row r.
template <int WN>
__device__ __forceinline__ void read8(const char* slab, int r, int c, float (&v)[8]) {
  const f32x4 lo = *reinterpret_cast<const f32x4*>(slab + slab_off<WN>(r, c));
  const f32x4 hi = *reinterpret_cast<const f32x4*>(slab + slab_off<WN>(r, c + 1));
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[j] = lo[j];
    v[4 + j] = hi[j];
  }
}

// Columns 8s..8s+7 of row r. Lanes of the upper half of a row read their odd
// chunk first, so that 16 lanes of either read touch 16 distinct 16-byte bank groups.
template <int WN>
__device__ __forceinline__ void read8_interleaved(const char* slab, int r, int s, float (&v)[8]) {
  const int odd = s >= WN / 16 ? 1 : 0;
  const f32x4 x = *reinterpret_cast<const f32x4*>(slab + slab_off<WN>(r, 2 * s + odd));
  const f32x4 y = *reinterpret_cast<const f32x4*>(slab + slab_off<WN>(r, 2 * s + (odd ^ 1)));
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[j] = odd ? y[j] : x[j];
    v[4 + j] = odd ? x[j] : y[j];
  }
}

// ---- the two 16-bit storage formats: bfloat16 and IEEE half, both held as
// raw 16-bit words (the tiles, DMA and LDS layouts do not care which); F16
// selects the MFMA instruction and the conversions of the epilogue.
template <bool F16>
__device__ __forceinline__ float h16_to_f32(uint16_t v) {
  if constexpr (F16) return static_cast<float>(__builtin_bit_cast(_Float16, v));
  else return __uint_as_float(static_cast<uint32_t>(v) << 16);
}

template <bool F16>
__device__ __forceinline__ uint16_t f32_to_h16(float f) {  // round to nearest even
  if constexpr (F16) return __builtin_bit_cast(uint16_t, static_cast<_Float16>(f));
  else return f32_to_bf16(f);
}

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

// acc += A B^T on a 32 x 32 tile, k = 16 (bfloat16 or half operands, float32 accumulate)
template <bool F16>
__device__ __forceinline__ f32x16 mfma32(bf16x8 a, bf16x8 b, f32x16 c) {
  if constexpr (F16)
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// Eight consecutive 16-bit values as one 16-byte global access (16-byte aligned).
// Epilogue traffic is streamed once: non-temporal loads and stores keep it
// from evicting the operand tiles the other blocks are reading from L2.
template <bool F16>
__device__ __forceinline__ void unpack8(const u32x4& r, float (&v)[8]) {
  const uint32_t w[4] = {r[0], r[1], r[2], r[3]};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = h16_to_f32<F16>(static_cast<uint16_t>(w[j] & 0xffffu));
    v[2 * j + 1] = h16_to_f32<F16>(static_cast<uint16_t>(w[j] >> 16));
  }
}

template <bool F16>
__device__ __forceinline__ void load8(const bf16_t* p, float (&v)[8]) {
  unpack8<F16>(__builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p)), v);
}

template <bool F16>
__device__ __forceinline__ void store8(bf16_t* p, const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
    w[j] = static_cast<uint32_t>(f32_to_h16<F16>(v[2 * j])) |
           (static_cast<uint32_t>(f32_to_h16<F16>(v[2 * j + 1])) << 16);
  u32x4 q;
  q[0] = w[0];
  q[1] = w[1];
  q[2] = w[2];
  q[3] = w[3];
  __builtin_nontemporal_store(q, reinterpret_cast<u32x4*>(p));
}

// LDS writes of this wave are complete (and not reordered by the compiler)
// before its lanes read what other lanes wrote.
__device__ __forceinline__ void wave_lds_sync() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

template <bool F16, int BM, int BN, int WM, int WN, int BK, int NST, int MINB, int MODE, int EPI,
          bool PAIRED, bool A_KC, bool B_KC, int VST, int GATH = 0>
__global__ __launch_bounds__((BM / WM) * (BN / WN) * 64, MINB) void gemm16(GemmArgs p) {
  constexpr int WAVES_N = BN / WN, MF = WM / 32, NF = WN / 32;
  constexpr int NW = (BM / WM) * (BN / WN);
  constexpr int A_BYTES = BM * BK * 2, B_BYTES = BN * BK * 2, ST = A_BYTES + B_BYTES;
  typedef Geo<BM, BK, A_KC, NW> GA;
  typedef Geo<BN, BK, B_KC, NW> GB;
  static_assert(NW == 4 || NW == 8, "four or eight waves per block");
  static_assert(!PAIRED || (NF % 2 == 0), "paired tiles need gate and up fragments");
  static_assert(GA::TI >= 1 && GB::TI >= 1, "tile smaller than one DMA instruction");
  static_assert(VST || (NST >= 3 && NST <= 6 && (NST - 2) * (GA::MINW + GB::MINW) <= 63),
                "vmcnt range");
  // GROUP_KV: + the block's [BM][32] tile of the side-product B
  constexpr int VB_BYTES = MODE == GROUP_KV ? BM * 32 * 2 : 0;
  // GATH (weight gradients, DMA tiles): the reduction rows of operand A
  // (GATH 1: dY's rows for the B gradient of down) or B (GATH 2: x's rows for
  // the LoRA A gradient of gate_up and dW_gu) are read through a row list, so
  // that operand's lane offsets depend on each k tile's rows: they are formed
  // a k tile ahead from a table in LDS of the byte offsets of up to GT_ROWS
  // of the block's rows (sized so that two blocks still fit a CU). A
  // separate instantiation keeps the ungathered loop as it is.
  constexpr bool GK = MODE == GROUP_K || MODE == GROUP_KV;
  static_assert(GATH == 0 || (GK && VST == 0 && !A_KC && !B_KC), "gathered rows: DMA weight gradients");
  constexpr bool GATHER_A = GATH == 1, GATHER_B = GATH == 2;
  constexpr int GT_ROWS = GATH == 0                ? 0
                          : (GATHER_B && BM <= 32) ? 4096
                          : (GATHER_A && BN <= 32) ? 2048
                                                   : 1024;
  __shared__ __attribute__((aligned(1024))) char smem[NST * ST + VB_BYTES + GT_ROWS * 4];

  const int tid = threadIdx.x, lane = tid & 63;
  // wave index as a wave-uniform (scalar) value, so that everything derived
  // from it (DMA destinations, resources) stays in SGPRs
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  // The second and later rows of waves are rotated along N: when only the
  // first column of waves holds valid columns (a narrow last N tile), its
  // waves sit on different SIMDs (wave w runs on SIMD w % 4).
  const int wm = wave / WAVES_N, wn = (wave % WAVES_N + wm) % WAVES_N;

  constexpr bool DENSE = EPI == EPI_LINEAR;
  static_assert(!DENSE || (!PAIRED && GATH == 0 && MODE != GROUP_KV), "dense products are plain");
  int e, n_tile, rows, m0 = 0, krows = 0;
  int kbeg = 0, K0 = p.K[0];  // GROUP_M: this block's part of the reduction
  int64_t row0;
  if constexpr (DENSE) {
    if (!dense_tile(p, BM, e, n_tile, m0)) return;
    rows = min(BM, p.M - m0);
    kbeg = e * p.kchunk;
    K0 = min(p.kchunk, p.K[0] - kbeg);
    row0 = MODE == GROUP_M ? m0 : kbeg;
    krows = K0;
  } else if (MODE == GROUP_M) {
    const int mtot = *p.ntiles;
    const int total = mtot * p.ntn;
    if (static_cast<int>(blockIdx.x) >= total) return;
    // XCD-contiguous ranges, then groups of up to 8 M tiles of one expert
    // swept across all N tiles, so the tiles an XCD runs together share A
    // rows and the expert's weight columns in L2.
    const int L = xcd_remap(blockIdx.x, total);
    const int4 t = p.tiles[group_tile(p.tiles, L, p.ntn, n_tile)];
    e = t.x;
    row0 = t.y;
    rows = t.z;
  } else {
    const int total = p.E * p.ntm * p.ntn;
    if (static_cast<int>(blockIdx.x) >= total) return;
    const int L = xcd_remap(blockIdx.x, total);
    e = L / (p.ntm * p.ntn);
    const int rem = L - e * (p.ntm * p.ntn);
    const int mt = rem / p.ntn;
    n_tile = rem - mt * p.ntn;
    m0 = mt * BM;
    rows = min(BM, p.M - m0);
    row0 = p.offsets[e];
    krows = p.offsets[e + 1] - static_cast<int>(row0);
  }
  const int n0 = PAIRED ? 0 : n_tile * BN;

  // ---- DMA plans for the main segment (0) and the LoRA segment (1). Kept in
  // plain variables, never indexed by a runtime value, so they stay in
  // registers: a scratch access would bring an s_waitcnt vmcnt(0) that also
  // drains every tile in flight.
  Plan<BM, BK, A_KC, NW> pa0, pa1;
  Plan<BN, BK, B_KC, NW> pb0, pb1;
  auto build = [&](int seg, Plan<BM, BK, A_KC, NW>& PA, Plan<BN, BK, B_KC, NW>& PB) {
    const Opnd& A = p.a[seg];
    const Opnd& B = p.b[seg];
    View<bf16_t> va{}, vb{};
    va.ld = A.ld; va.kcontig = A.kcontig; va.vec = A.vec;
    vb.ld = B.ld; vb.kcontig = B.kcontig; vb.vec = B.vec;
    int64_t abytes, bbytes;
    if (MODE == GROUP_M) {
      const int K = DENSE && seg == 0 ? K0 : p.K[seg];
      va.base = static_cast<const bf16_t*>(A.ptr) + row0 * A.ld + kbeg;
      va.klim = K;
      va.mn_lim = rows;
      abytes = (static_cast<int64_t>(rows) * A.ld - kbeg) * 2;
      if (A.rows) {
        va.base = static_cast<const bf16_t*>(A.ptr);
        va.grow = A.rows + row0;
        va.gk = A.rows_div;
        abytes = A.rows_bytes;
      }
      const bf16_t* wb = static_cast<const bf16_t*>(B.ptr) + static_cast<int64_t>(e) * B.estride;
      vb.klim = K;
      if (PAIRED) {
        vb.base = wb;
        vb.paired = 1;
        vb.half = BN / 2;
        vb.pbase = n_tile * (BN / 2);
        vb.I = p.I;
        vb.mn_lim = BN;
        bbytes = static_cast<int64_t>(2) * p.I * B.ld * 2;
      } else if (B_KC) {
        vb.base = wb + static_cast<int64_t>(n0) * B.ld + kbeg;
        vb.mn_lim = p.N - n0;
        bbytes = (static_cast<int64_t>(p.N - n0) * B.ld - kbeg) * 2;
      } else {
        vb.base = wb + static_cast<int64_t>(kbeg) * B.ld + n0;
        vb.mn_lim = p.N - n0;
        bbytes = static_cast<int64_t>(K) * B.ld * 2 - static_cast<int64_t>(n0) * 2;
      }
    } else {
      va.base = static_cast<const bf16_t*>(A.ptr) + row0 * A.ld + m0;
      va.klim = krows;
      va.mn_lim = p.M - m0;
      abytes = static_cast<int64_t>(krows) * A.ld * 2 - static_cast<int64_t>(m0) * 2;
      if (GATHER_A) {
        va.base = static_cast<const bf16_t*>(A.ptr) + m0;
        va.grow = A.rows + row0;
        va.gk = A.rows_div;
        abytes = A.rows_bytes - static_cast<int64_t>(m0) * 2;
      }
      vb.base = static_cast<const bf16_t*>(B.ptr) + row0 * B.ld + n0;
      vb.klim = krows;
      vb.mn_lim = p.N - n0;
      bbytes = static_cast<int64_t>(krows) * B.ld * 2 - static_cast<int64_t>(n0) * 2;
      if (GATHER_B) {
        vb.base = static_cast<const bf16_t*>(B.ptr) + n0;
        vb.grow = B.rows + row0;
        vb.gk = B.rows_div;
        bbytes = B.rows_bytes - static_cast<int64_t>(n0) * 2;
      }
    }
    make_plan<BM, BK, A_KC, NW>(PA, va, abytes, A.vec, wave, lane);
    make_plan<BN, BK, B_KC, NW>(PB, vb, bbytes, B.vec, wave, lane);
  };
  build(0, pa0, pb0);
  if (MODE == GROUP_M) {
    build(1, pa1, pb1);
  } else {
    pa1 = pa0;
    pb1 = pb0;
  }

  const int nk0 = MODE == GROUP_M ? (K0 + BK - 1) / BK : (krows + BK - 1) / BK;
  const int nk1 = MODE == GROUP_M ? (p.K[1] + BK - 1) / BK : 0;
  const int nk = nk0 + nk1;
  const bool dma0 = pa0.vec && pb0.vec, dma1 = pa1.vec && pb1.vec;

  // Gathered reduction rows (GROUP_K, GROUP_KV): the byte offsets of the rows
  // from gw0 on in LDS, when formed, for the operand whose rows they are
  const uint32_t* gtab_a = nullptr;
  const uint32_t* gtab_b = nullptr;
  int gw0 = 0;
  auto issue = [&](int j) {  // a whole stage at once (prologue, element-wise fills)
    char* sa = smem + (j % NST) * ST;
    char* sb = sa + A_BYTES;
    if (j < nk0) {
      fill<BM, BK, A_KC, NW, GATHER_A>(pa0, j * BK, sa, wave, lane, gtab_a, gw0);
      fill<BN, BK, B_KC, NW, GATHER_B>(pb0, j * BK, sb, wave, lane, gtab_b, gw0);
    } else {
      fill<BM, BK, A_KC, NW, false>(pa1, (j - nk0) * BK, sa, wave, lane);
      fill<BN, BK, B_KC, NW, false>(pb1, (j - nk0) * BK, sb, wave, lane);
    }
  };
  // A stage filled only by DMA leaves at least MINW loads per operand outstanding.
  auto dma_stage = [&](int j) { return j < nk0 ? dma0 : dma1; };

  int fa_base[MF], fb_base[NF];
#pragma unroll
  for (int mi = 0; mi < MF; ++mi) fa_base[mi] = wm * WM + mi * 32;
#pragma unroll
  for (int ni = 0; ni < NF; ++ni) {
    if (PAIRED)
      fb_base[ni] = (ni < NF / 2) ? wn * (WN / 2) + ni * 32
                                  : BN / 2 + wn * (WN / 2) + (ni - NF / 2) * 32;
    else
      fb_base[ni] = wn * WN + ni * 32;
  }
  FragAddr<BM, BK, A_KC, MF> FA;
  FragAddr<BN, BK, B_KC, NF> FB;
  frag_addr<BM, BK, A_KC, MF>(FA, fa_base, lane);
  frag_addr<BN, BK, B_KC, NF>(FB, fb_base, lane);

  // EPI_LINEAR epilogue: a slab's 32 x WN outputs in pieces of eight columns, 64 at a time. The
  // bias's and residual's pieces of a slab are loaded while the slab before it is finished; those of
  // the first one before the main loop where the tile is small enough to have registers for them
  // (there the latency counts, too). One block a CU does not overlap it with products: of the 197 us
  // that 8192 x 4096 x 2880 bf16 with bias, dropout and residual takes (983 TFLOP/s), the bare
  // product in the same run takes 190.
  typedef std::conditional_t<F16, f16_t, bf16_t> DElem;
  constexpr int DSEGS = WN / 8, DPASS = DENSE ? 32 * DSEGS / 64 : 1;
  constexpr bool DEARLY = MF * NF <= 4;
  DropKey dkey{};
  // a lane's columns repeat every DREP pieces, so its bias does
  constexpr int DREP = 64 % DSEGS == 0 ? 1 : 3;
  static_assert(!DENSE || (DREP * 64 % DSEGS == 0 && DPASS % DREP == 0), "columns repeat");
  Row8<DElem> dres[2][DPASS], dbias[DREP];
  auto dplace = [&](int mi, int pass, int& m_local, int& col) __attribute__((always_inline)) {
    m_local = wm * WM + mi * 32 + (pass * 64 + lane) / DSEGS;
    col = n0 + wn * WN + 8 * ((pass * 64 + lane) % DSEGS);
    return m_local < rows && col < p.N;  // N is a multiple of 8
  };
  auto dfetch = [&](int mi, Row8<DElem> (&r)[DPASS]) __attribute__((always_inline)) {
    const bool finish = MODE == GROUP_M && p.E == 1;
    if (mi == 0) {
      dkey = drop_key(p.lin.drop);
#pragma unroll
      for (int pass = 0; pass < DREP; ++pass) {
        int m_local, col;
        dplace(0, pass, m_local, col);
        dbias[pass].zero();
        if (finish && p.lin.bias && col < p.N)
          dbias[pass].load(static_cast<const DElem*>(p.lin.bias) + col);
      }
    }
#pragma unroll
    for (int pass = 0; pass < DPASS; ++pass) {
      int m_local, col;
      r[pass].zero();
      if (dplace(mi, pass, m_local, col) && finish && p.lin.residual)
        r[pass].load(static_cast<const DElem*>(p.lin.residual) +
                     static_cast<int64_t>(m0 + m_local) * p.N + col);
    }
  };
  if constexpr (DENSE && DEARLY) dfetch(0, dres[0]);

  f32x16 acc[MF][NF];
#pragma unroll
  for (int i = 0; i < MF; ++i)
#pragma unroll
    for (int j = 0; j < NF; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;

  // GROUP_KV: this block's feature rows of the expert's side-product B, as
  // MFMA fragments over the whole tile (k = feature, n = column of B; lane l
  // holds column l%32 and features 8(l/32)..+7 of each 16-feature step). The
  // [BM][32] tile goes through LDS in 16-byte pieces (zero-padded past M and
  // N; rows of B are 16-byte aligned, N a multiple of 8) and is read back
  // with transpose reads, like any output-contiguous operand.
  static_assert(MODE != GROUP_KV || (BM == 256 && BN == 32 && BK == 32 && !A_KC && VST == 0),
                "side-product partials assume 256 x 32 tiles, 32 rows per k tile");
  constexpr int VKS = MODE == GROUP_KV ? BM / 16 : 1;
  bf16x8 vbf[VKS];
  if constexpr (MODE == GROUP_KV) {
    const bf16_t* bm = static_cast<const bf16_t*>(p.vb) +
                       static_cast<int64_t>(e / p.vsplit) * p.vb_estride;
    char* vt = smem + NST * ST;
    for (int i = tid; i < BM * 4; i += NW * 64) {  // piece i: feature i/4, columns 8 (i%4)..
      const int f = i >> 2, c = i & 3;
      u32x4 v = {0u, 0u, 0u, 0u};
      if (m0 + f < p.M && c * 8 < p.N)
        v = *reinterpret_cast<const u32x4*>(bm + static_cast<int64_t>(m0 + f) * p.N + c * 8);
      *reinterpret_cast<u32x4*>(vt + f * 64 + c * 16) = v;
    }
    __syncthreads();
    FragAddr<32, BM, false, 1> FV;
    const int zero[1] = {0};
    frag_addr<32, BM, false, 1>(FV, zero, lane);
#pragma unroll
    for (int kk = 0; kk < VKS; ++kk) vbf[kk] = read_frag<32, BM, false, 1>(vt, FV, 0, 0, kk);
  }

  if constexpr (VST > 0) {
    // ---- Register-staged main loop: every wave loads its share of a k tile
    // into VGPRs (16 bytes per lane per 1 KB piece, the same lane offsets as
    // the DMA plans, out-of-range lanes read zeros) and writes it to the LDS
    // slot the tile belongs to. Two LDS slots and one register buffer: tile
    // it+1 is written during tile it's second k-step (its slot was last read
    // before the previous barrier), and the load of tile it+2 is issued into
    // the buffer just freed, so each load has a whole k tile of MFMAs to
    // arrive. Tile 1 is loaded together with tile 0 into a prologue-only
    // buffer (the accumulators hold nothing yet, so their registers are
    // free): a block waits for one load latency before its first MFMA.
    //
    // The steady state (the tiles whose staged load is a whole in-range tile
    // of the main segment) runs two tiles per iteration, so the LDS slot of
    // every access is a compile-time constant: fragment reads and staging
    // writes take their whole offset in the instruction's immediate field
    // from loop-invariant per-lane bases, and the loads need no masking.
    // The first tile, the tiles around the LoRA segment and the K tail, and
    // the last tile take the general path (slot chosen at run time, loads
    // masked).
    static_assert(VST == 1, "one register buffer");
    static_assert(NST == 2, "register staging uses two LDS slots");
    constexpr int KS = BK / 16;
    static_assert(KS % 2 == 0, "fragment double-buffering alternates per k-step");
    u32x4 ra[GA::NIW], rb[GB::NIW];
    // Buffer resource of a plan (wave-uniform: built in SGPRs).
    auto make_rs = [&](const auto& P) __attribute__((always_inline)) {
      // readfirstlane returns int: widen through uint32_t, never by sign extension
      const uint64_t base = reinterpret_cast<uint64_t>(P.base);
      const uint64_t lo = static_cast<uint32_t>(
          __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(base)));
      const uint64_t hi = static_cast<uint32_t>(
          __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(base >> 32)));
      return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>((hi << 32) | lo),
                                               static_cast<short>(0),
                                               __builtin_amdgcn_readfirstlane(P.nrec), 0x00020000);
    };
    __amdgpu_buffer_rsrc_t rsa = make_rs(pa0), rsb = make_rs(pb0);
    // CLEAN: the tile is a whole, in-range tile of the current plans (no
    // masking, every lane's offset as planned)
    auto vload = [&](auto& P, const __amdgpu_buffer_rsrc_t& rs, int k0, u32x4* r, auto geo,
                     bool live, auto cleanc) __attribute__((always_inline)) {
      typedef decltype(geo) G;
      constexpr bool CLEAN = decltype(cleanc)::value;
      const bool kc = decltype(geo)::KCV;
      const uint32_t soff = kc ? static_cast<uint32_t>(k0) * 2
                               : static_cast<uint32_t>(static_cast<int64_t>(k0) * P.ld * 2);
      const bool tail = !CLEAN && kc && (k0 + BK > P.klim);
#pragma unroll
      for (int i = 0; i < G::NIW; ++i) {
        const int j = wave + NW * i;
        if (G::TI % NW == 0 || j < G::TI) {
          uint32_t vo = P.vo[i];
          if constexpr (!CLEAN) {
            if (!live) vo = kOOB;
            if (tail) {
              const int rr = G::RPI * j + lane / G::CPR;
              const int c = (lane % G::CPR) ^ kswz<BK>(rr);
              if (k0 + c * 8 >= P.klim) vo = kOOB;
            }
          }
          r[i] = __builtin_amdgcn_raw_buffer_load_b128(rs, vo, __builtin_amdgcn_readfirstlane(soff), 0);
        }
      }
    };
    // Branch-free issue: the plans switch to the LoRA segment's once, before
    // its first tile is loaded (tiles are loaded in order), and live = false
    // issues the loads with every lane out of range (they return zeros and
    // touch no memory) instead of skipping them, so every path issues the
    // same loads and the compiler's waits stay exact.
    auto switch_plans = [&]() __attribute__((always_inline)) {
      pa0 = pa1;
      pb0 = pb1;
      rsa = make_rs(pa0);
      rsb = make_rs(pb0);
    };
    auto load_tile = [&](int j, u32x4* a, u32x4* b, bool live, auto cleanc) __attribute__((always_inline)) {
      const int k0 = (j >= nk0 ? j - nk0 : j) * BK;
      vload(pa0, rsa, k0, a, GeoK<GA, A_KC>(), live, cleanc);
      vload(pb0, rsb, k0, b, GeoK<GB, B_KC>(), live, cleanc);
    };
    // LDS layout [A slot 0 | A slot 1 | B slot 0 | B slot 1]: every access of
    // a slot lies within 64 KB of its operand's region start, so a per-lane
    // base register plus the instruction's immediate offset reaches it.
    constexpr int B_REGION = 2 * A_BYTES;
    static_assert(A_BYTES <= 32768 && B_BYTES <= 32768, "slot offsets fit the DS immediate");
    // slot: LDS slot (0 or 1) the tile goes to
    auto store_tile = [&](int slot, const u32x4* a, const u32x4* b) __attribute__((always_inline)) {
      char* sa = smem + slot * A_BYTES;
      char* sb = smem + B_REGION + slot * B_BYTES;
#pragma unroll
      for (int i = 0; i < GA::NIW; ++i) {
        const int jj = wave + NW * i;
        if (GA::TI % NW == 0 || jj < GA::TI)
          *reinterpret_cast<u32x4*>(sa + jj * 1024 + 16 * lane) = a[i];
      }
#pragma unroll
      for (int i = 0; i < GB::NIW; ++i) {
        const int jj = wave + NW * i;
        if (GB::TI % NW == 0 || jj < GB::TI)
          *reinterpret_cast<u32x4*>(sb + jj * 1024 + 16 * lane) = b[i];
      }
    };
    bf16x8 af[2][MF], bf[2][NF];
    // Fragment addresses: per-lane bases (per k-step for k-contiguous tiles,
    // per fragment for output-contiguous ones, which advance by a constant
    // per k-step) plus compile-time offsets. The wave's own row/column offset
    // sits in the base; the fragment index and the slot are immediates.
    // k-contiguous: base_k[ks] + (fr_base[f] - fr_base[0]) * BK * 2
    // output-contiguous: base_f[f] + ks * 16 * ROWS * 2 (+ 4 * ROWS * 2)
    const char* abase[A_KC ? KS : MF];
    const char* bbase[B_KC ? KS : NF];
#pragma unroll
    for (int q = 0; q < (A_KC ? KS : MF); ++q)
      abase[q] = smem + (A_KC ? fa_base[0] * BK * 2 + FA.off[q] : FA.off[q]);
#pragma unroll
    for (int q = 0; q < (B_KC ? KS : NF); ++q)
      bbase[q] = smem + B_REGION + (B_KC ? fb_base[0] * BK * 2 + FB.off[q] : FB.off[q]);
    // compile-time fragment offsets relative to fragment 0 (they depend on
    // the wave only through fr_base[0])
    auto frag_rd = [&](const char* const* base, auto kcc, auto rowsc, int f, int frel, int ks,
                       int slot_off) __attribute__((always_inline)) {
      constexpr bool KC = decltype(kcc)::value;
      constexpr int ROWS = decltype(rowsc)::value;
      if constexpr (KC) {
        return *reinterpret_cast<const bf16x8*>(base[ks] + slot_off + frel * BK * 2);
      } else {
        const char* q = base[f] + slot_off + ks * 16 * ROWS * 2;
        v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4s*)(q));
        v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (__attribute__((address_space(3))) v4s*)(q + 4 * ROWS * 2));
        v8s r = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
        return __builtin_bit_cast(bf16x8, r);
      }
    };
    auto read_frags = [&](int slot, int ks, int dst) __attribute__((always_inline)) {
#pragma unroll
      for (int mi = 0; mi < MF; ++mi)
        af[dst][mi] = frag_rd(abase, std::integral_constant<bool, A_KC>(),
                              std::integral_constant<int, BM>(), mi, mi * 32, ks, slot * A_BYTES);
#pragma unroll
      for (int ni = 0; ni < NF; ++ni) {
        // fr_base[ni] - fr_base[0]: compile time (paired: gate fragments, then up ones)
        const int frel = PAIRED ? (ni < NF / 2 ? ni * 32 : BN / 2 + (ni - NF / 2) * 32) : ni * 32;
        bf[dst][ni] = frag_rd(bbase, std::integral_constant<bool, B_KC>(),
                              std::integral_constant<int, BN>(), ni, frel, ks, slot * B_BYTES);
      }
    };
    u32x4 ta[GA::NIW], tb[GB::NIW];  // tile 1, prologue only
    if (nk > 0) {
      if (nk0 == 0) switch_plans();
      load_tile(0, ra, rb, true, std::false_type());
      if (1 == nk0) switch_plans();
      load_tile(1, ta, tb, 1 < nk, std::false_type());
      store_tile(0, ra, rb);
      __syncthreads();
      read_frags(0, 0, 0);
    }
    // k-steps of the last tile holding valid k (the rest of it is zeros)
    const int klast = MODE == GROUP_M ? (nk1 > 0 ? p.K[1] - (nk1 - 1) * BK : K0 - (nk0 - 1) * BK)
                                      : krows - (nk0 - 1) * BK;
    const int ns_last = (klast + 15) / 16;
    // One k tile. PAR: the tile's LDS slot when known at compile time (-1:
    // it % 2 at run time). MFMA = false: the wave's rows or columns all lie
    // past the valid ones; it still loads, stores and meets every barrier,
    // but issues no MFMAs and reads no fragments. LAST: the last tile, which
    // stages and loads nothing and leaves its k-step loop after the k-steps
    // that hold valid k (a LoRA segment of rank 16 fills one of a 64-wide
    // tile's four; the rest is zeros); one path with early exits, so the
    // accumulators stay in place. FIRST: tile 1 is stored from the prologue
    // buffer. CLEAN: the load this tile issues (tile it+2) is a whole,
    // in-range tile of the plans already in place.
    auto ktile = [&](int it, auto parc, auto mfmac, auto lastc, auto firstc,
                     auto cleanc) __attribute__((always_inline)) {
      constexpr int PAR = decltype(parc)::value;
      constexpr bool MFMA = decltype(mfmac)::value;
      constexpr bool LAST = decltype(lastc)::value;
      constexpr bool FIRST = decltype(firstc)::value;
      constexpr bool CLEAN = decltype(cleanc)::value;
      const int slot = PAR >= 0 ? PAR : (it & 1);
      if (!CLEAN && it + 2 == nk0) switch_plans();  // the tile loaded here is it+2
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        if constexpr (LAST) {
          if (ks >= ns_last) break;
        }
        const int cur = ks & 1;
        if (ks + 1 < KS) {
          if constexpr (MFMA) read_frags(slot, ks + 1, cur ^ 1);
        } else if (!LAST && it + 1 < nk) {
          // Before the last k-step's MFMAs: every wave has read all of tile
          // it (its slot may be refilled next) and has written tile it+1, so
          // one barrier covers both, and the first fragment reads of tile
          // it+1 overlap this k-step's MFMAs.
          barrier_lds();
          if constexpr (MFMA) read_frags(slot ^ 1, 0, cur ^ 1);
        }
        // tile it+1's slot was last read in tile it-1, before the last barrier
        if (!LAST && ks == 1) {
          // past the last tile this stores the zeros of an out-of-range
          // load into a slot nobody reads again
          if constexpr (FIRST) store_tile(slot ^ 1, ta, tb);
          else store_tile(slot ^ 1, ra, rb);
          const int jn = it + 2;
          if constexpr (CLEAN) load_tile(jn, ra, rb, true, std::true_type());
          else load_tile(min(jn, nk - 1), ra, rb, jn < nk, std::false_type());
        }
        if constexpr (MFMA) {
          // Instruction order within the k-step, by measurement: one LDS read
          // after each MFMA, and in the staging k-step the stores and loads
          // early, two of each after each of the first four MFMAs.
#pragma unroll
          for (int mi = 0; mi < MF; ++mi)
#pragma unroll
            for (int ni = 0; ni < NF; ++ni)
              acc[mi][ni] = mfma32<F16>(bf[cur][ni], af[cur][mi], acc[mi][ni]);
          if (!LAST && ks == 1) {
#pragma unroll
            for (int i = 0; i < MF * NF / 2; ++i) {
              __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // one MFMA
              __builtin_amdgcn_sched_group_barrier(0x200, 2, 0);  // two LDS writes
              __builtin_amdgcn_sched_group_barrier(0x020, 2, 0);  // two buffer loads
            }
#pragma unroll
            for (int i = 0; i < MF * NF / 2; ++i) {
              __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // one MFMA
              __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);  // two LDS reads
            }
          } else {
#pragma unroll
            for (int i = 0; i < MF * NF; ++i) {
              __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // one MFMA
              __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);  // one LDS read
            }
          }
        }
        // Each k-step is a scheduling region of its own: otherwise the
        // scheduler fills the groups above with MFMAs of the next k-step,
        // putting two MFMAs on one accumulator back to back (a dependent
        // 32x32x16 MFMA issues after about 52 cycles instead of 32).
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    // The wave-uniform choice is made once, outside the k loop, so the loop
    // itself has no extra branch.
    auto kloop = [&](auto mfmac) __attribute__((always_inline)) {
      using Yes = std::true_type;
      using No = std::false_type;
      using Rt = std::integral_constant<int, -1>;
      const int nkf = nk - 1;  // full tiles before the last
      // Tiles 1..C are clean: the tile each stages (it + 2) is a whole tile
      // of the main segment (K tail tile excluded).
      const int last_clean = MODE == GROUP_M || DENSE ? nk0 - 1 - (K0 % BK != 0 ? 1 : 0) : -1;
      const int C = min(nkf - 1, last_clean - 2);
      if (nkf > 0) ktile(0, Rt(), mfmac, No(), Yes(), No());
      int it = 1;
      for (; it + 1 <= C; it += 2) {
        ktile(it, std::integral_constant<int, 1>(), mfmac, No(), No(), Yes());
        ktile(it + 1, std::integral_constant<int, 0>(), mfmac, No(), No(), Yes());
      }
      if (it <= C) {
        ktile(it, std::integral_constant<int, 1>(), mfmac, No(), No(), Yes());
        ++it;
      }
      for (; it < nkf; ++it) ktile(it, Rt(), mfmac, No(), No(), No());
      if (nk > 0) ktile(nkf, Rt(), mfmac, Yes(), No(), No());
    };
    // Waves whose rows all lie past the tile's valid rows, or whose columns
    // all lie past the valid columns, neither read fragments nor multiply.
    const bool live = (MODE != GROUP_M && !DENSE) ||
                      (wm * WM < rows && (PAIRED ? n_tile * (BN / 2) + wn * (WN / 2) < p.I
                                                 : n0 + wn * WN < p.N));
    if (live) kloop(std::true_type());
    else kloop(std::false_type());
  } else {
    // Gathered reduction rows (GROUP_K, GROUP_KV): the lane offsets of a
    // refill depend on its rows' numbers, so they are formed one iteration
    // ahead (their loads then complete under a k tile of MFMAs instead of
    // delaying the refill's DMA issue).
    constexpr bool gath_a = GATHER_A, gath_b = GATHER_B, gath = GATH != 0;
    uint32_t gvo_a[GA::NIW], gvo_b[GB::NIW];
    // The rows' byte offsets, GT_ROWS at a time from row gw0 on: formed
    // before the first DMA, and again (experts of more than GT_ROWS rows)
    // when a refill passes the window, which then waits for the DMA in flight.
    uint32_t* gt = reinterpret_cast<uint32_t*>(smem + NST * ST + VB_BYTES);
    const int32_t* gt_rows = gath_a ? pa0.view.grow : pb0.view.grow;
    const uint32_t gt_div = static_cast<uint32_t>(gath_a ? pa0.view.gk : pb0.view.gk);
    const uint32_t gt_ld2 = static_cast<uint32_t>(gath_a ? pa0.ld : pb0.ld) * 2u;
    auto gather_window = [&](int w0) __attribute__((always_inline)) {
      __syncthreads();
      for (int i = tid; i < GT_ROWS && w0 + i < krows; i += NW * 64)
        gt[i] = static_cast<uint32_t>(gt_rows[w0 + i]) / gt_div * gt_ld2;
      __syncthreads();
      gw0 = w0;
    };
    if (GT_ROWS > 0 && gath) {
      gather_window(0);
      if (gath_a)
        gtab_a = gt;
      else
        gtab_b = gt;
    }
    auto gather_plan = [&](int j) __attribute__((always_inline)) {
      if (GT_ROWS > 0 && gath && (j + 1) * BK > gw0 + GT_ROWS) gather_window(j * BK);
      if (gath_a) {
#pragma unroll
        for (int i = 0; i < GA::NIW; ++i)
          gvo_a[i] = gather_vo(pa0, j * BK, wave + NW * i, lane, gtab_a, gw0);
      }
      if (gath_b) {
#pragma unroll
        for (int i = 0; i < GB::NIW; ++i)
          gvo_b[i] = gather_vo(pb0, j * BK, wave + NW * i, lane, gtab_b, gw0);
      }
    };
  #pragma unroll
    for (int s = 0; s < NST - 1; ++s)
      if (s < nk) issue(s);
    if (gath && NST - 1 < nk) gather_plan(NST - 1);
    for (int it = 0; it < nk; ++it) {
      // stage `it` must have landed; the DMA-only stages after it may stay in flight
      {
        int ahead = min(NST - 2, nk - 1 - it);
        for (int s = 1; s <= ahead; ++s)
          if (!dma_stage(it + s)) ahead = 0;
        constexpr int PER = GA::MINW + GB::MINW;
        switch (ahead) {
          case 1: wait_vmcnt<PER>(); break;
          case 2: wait_vmcnt<2 * PER>(); break;
          case 3: wait_vmcnt<3 * PER>(); break;
          case 4: wait_vmcnt<4 * PER>(); break;
          default: wait_vmcnt<0>(); break;
        }
      }
      barrier_lds();
      // Stage it+NST-1 is refilled while stage `it` is multiplied: its DMA
      // instructions are spread over the k-steps so that load issue overlaps the
      // MFMAs instead of stalling in-order issue in one burst.
      const int jn = it + NST - 1;
      const bool refill = jn < nk;
      const bool refill_dma = refill && dma_stage(jn);
      if (refill && !refill_dma) issue(jn);  // element-wise fill (rare shapes)
      const bool segn1 = jn >= nk0;
      const int k0n = (segn1 ? jn - nk0 : jn) * BK;
      const Plan<BM, BK, A_KC, NW> PA = segn1 ? pa1 : pa0;
      const Plan<BN, BK, B_KC, NW> PB = segn1 ? pb1 : pb0;
      char* san = smem + (jn % NST) * ST;
      char* sbn = san + A_BYTES;
      const char* sa = smem + (it % NST) * ST;
      const char* sb = sa + A_BYTES;
      constexpr int KS = BK / 16;
      constexpr int NT = GA::NIW + GB::NIW;
      uint32_t gcur_a[GA::NIW], gcur_b[GB::NIW];
#pragma unroll
      for (int i = 0; i < GA::NIW; ++i) gcur_a[i] = gvo_a[i];
#pragma unroll
      for (int i = 0; i < GB::NIW; ++i) gcur_b[i] = gvo_b[i];
      if (gath && jn + 1 < nk) gather_plan(jn + 1);
      // Fragments are double-buffered in registers: the LDS reads of k-step
      // ks+1 are in flight while the MFMAs of k-step ks run.
      bf16x8 af[2][MF], bf[2][NF];
  #pragma unroll
      for (int mi = 0; mi < MF; ++mi) af[0][mi] = read_frag<BM, BK, A_KC, MF>(sa, FA, mi, fa_base[mi], 0);
  #pragma unroll
      for (int ni = 0; ni < NF; ++ni) bf[0][ni] = read_frag<BN, BK, B_KC, NF>(sb, FB, ni, fb_base[ni], 0);
  #pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        const int cur = ks & 1;
        if (ks + 1 < KS) {
  #pragma unroll
          for (int mi = 0; mi < MF; ++mi)
            af[cur ^ 1][mi] = read_frag<BM, BK, A_KC, MF>(sa, FA, mi, fa_base[mi], ks + 1);
  #pragma unroll
          for (int ni = 0; ni < NF; ++ni)
            bf[cur ^ 1][ni] = read_frag<BN, BK, B_KC, NF>(sb, FB, ni, fb_base[ni], ks + 1);
        }
        if (refill_dma) {
  #pragma unroll
          for (int t = ks * NT / KS; t < (ks + 1) * NT / KS; ++t) {
            if (t < GA::NIW) {
              if constexpr (gath_a)
                fill_one<BM, BK, A_KC, NW, false, true>(PA, k0n, san, wave, lane, t, gcur_a[t]);
              else
                fill_one<BM, BK, A_KC, NW, false>(PA, k0n, san, wave, lane, t);
            } else {
              const int tb = t - GA::NIW;
              if constexpr (gath_b)
                fill_one<BN, BK, B_KC, NW, false, true>(PB, k0n, sbn, wave, lane, tb, gcur_b[tb]);
              else
                fill_one<BN, BK, B_KC, NW, false>(PB, k0n, sbn, wave, lane, tb);
            }
          }
        }
  #pragma unroll
        for (int mi = 0; mi < MF; ++mi)
  #pragma unroll
          for (int ni = 0; ni < NF; ++ni)
            acc[mi][ni] = mfma32<F16>(bf[cur][ni], af[cur][mi], acc[mi][ni]);
      }
      if constexpr (MODE == GROUP_KV) {
        // The A stage holds rows it*BK.. of the expert's D as [BK rows][BM
        // features] (output-contiguous layout). One wave per k tile, in turn,
        // multiplies those 32 rows by B over the tile's features and stores
        // the float32 partial; the stage stays valid until the next barrier.
        if (wave == it % NW) {
          f32x16 av;
#pragma unroll
          for (int v = 0; v < 16; ++v) av[v] = 0.f;
          const int kr = lane & 31, hb = lane >> 5;
#pragma unroll
          for (int kk = 0; kk < VKS; ++kk) {
            const int chunk = 2 * kk + hb;  // 8 features 16 kk + 8 hb ..
            const bf16x8 a = *reinterpret_cast<const bf16x8*>(
                sa + kr * BM * 2 + ((chunk ^ nswz<BM>(kr)) << 4));
            av = mfma32<F16>(vbf[kk], a, av);
          }
          // lane holds row kr and columns 8 q + 4 hb + (0..3) for q = 0..3
          const int rowl = it * BK + kr;
          if (rowl < krows) {
            float* vr = p.vp + static_cast<int64_t>(m0 / BM) * p.vp_tstride +
                        (row0 + rowl) * static_cast<int64_t>(p.N);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const int j = 8 * q + 4 * hb;
              if (j < p.N)
                *reinterpret_cast<f32x4*>(vr + j) = f32x4{av[4 * q], av[4 * q + 1], av[4 * q + 2], av[4 * q + 3]};
            }
          }
        }
      }
    }

  }

  // ---- Epilogue, staged through LDS. After the final wait no DMA is in
  // flight, so once every wave is past its last fragment read the whole ring
  // is free. Each wave then stages one 32-row slab of its accumulators at a
  // time as float32 and writes the outputs back as whole 16-byte row segments
  // (8 consecutive bf16), which keeps global stores, and the h loads of the
  // SwiGLU backward, coalesced along rows.
  // Accumulator layout: lane holds, for MFMA tile (mi, ni), row lane%32 of the
  // 32-row slab mi and the columns 8*(v/4) + 4*(lane/32) + v%4 of fragment ni.
  __syncthreads();
  constexpr int SLAB = 32 * WN * 4;
  static_assert(NW * SLAB <= NST * ST, "epilogue slab does not fit in the LDS ring");
  char* slab = smem + wave * SLAB;
  const int srow = lane & 31, shalf = lane >> 5;
  const bool out_vec = (reinterpret_cast<uintptr_t>(p.out) & 15) == 0 && (p.ld_out & 7) == 0 &&
                       (p.out_estride & 7) == 0;
  const bool out_vec4 = (reinterpret_cast<uintptr_t>(p.out) & 15) == 0 && (p.ld_out & 3) == 0 &&
                        (p.out_estride & 3) == 0;
  const bool aux_vec = p.aux == nullptr ||
                       ((reinterpret_cast<uintptr_t>(p.aux) & 15) == 0 && (p.ld_aux & 7) == 0);
  // SwiGLU backward: the h segments a slab needs are loaded while the previous
  // slab is finished, so one load latency per tile is exposed rather than one
  // per slab (the epilogue reads h [rows, 2I] and writes dH of the same size).
  // (wave tiles up to 64 wide: two slabs of h take 64 VGPRs; wider ones load per slab)
  constexpr bool HPRE = MODE == GROUP_M && EPI == EPI_SWIGLU_BWD && !PAIRED && WN <= 64;
  constexpr int HSEGS = WN / 8, HRPP = 64 / HSEGS, HPASS = 32 / HRPP;
  u32x4 hpre[2][HPASS][2];
  auto hfetch = [&](int mi, u32x4 (&hb)[HPASS][2]) {
    const int mb = wm * WM + mi * 32;
#pragma unroll
    for (int pass = 0; pass < HPASS; ++pass) {
      const int m_local = mb + pass * HRPP + lane / HSEGS;
      const int col = n0 + wn * WN + 8 * (lane % HSEGS);
      if (m_local < rows && col < p.N) {  // N = I, a multiple of 8
        const bf16_t* hr = static_cast<const bf16_t*>(p.aux) + (row0 + m_local) * p.ld_aux;
        hb[pass][0] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(hr + col));
        hb[pass][1] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(hr + p.I + col));
      }
    }
  };
  if constexpr (HPRE) hfetch(0, hpre[0]);
  if constexpr (DENSE) {
    if (!DEARLY) dfetch(0, dres[0]);
#pragma unroll
    for (int mi = 0; mi < MF; ++mi) {
      if (mi) wave_lds_sync();  // previous slab fully read
#pragma unroll
      for (int ni = 0; ni < NF; ++ni)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          f32x4 v;
#pragma unroll
          for (int j = 0; j < 4; ++j) v[j] = acc[mi][ni][4 * q + j];
          *reinterpret_cast<f32x4*>(slab + slab_off<WN>(srow, ni * 8 + 2 * q + shalf)) = v;
        }
      if (mi + 1 < MF) dfetch(mi + 1, dres[(mi + 1) & 1]);
      wave_lds_sync();
#pragma unroll
      for (int pass = 0; pass < DPASS; ++pass) {
        int m_local, col;
        const bool in = dplace(mi, pass, m_local, col);
        float v[8];
        read8_interleaved<WN>(slab, (pass * 64 + lane) / DSEGS, (pass * 64 + lane) % DSEGS, v);
        if (!in) continue;
        const int64_t row = m0 + m_local;
        if (p.E > 1) {
          Row8<float> o;
          o.set(v);
          o.store(static_cast<float*>(p.out) + (static_cast<int64_t>(e) * p.M + row) * p.N + col);
        } else if (MODE == GROUP_M) {
          linear_finish8<DElem>(p.lin, dkey, row, col, p.N, dbias[pass % DREP],
                                dres[mi & 1][pass], v);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] *= p.scale;
          store8<F16>(static_cast<bf16_t*>(p.out) + row * p.N + col, v);
        }
      }
    }
    return;
  }
#pragma unroll
  for (int mi = 0; mi < MF; ++mi) {
    if constexpr (HPRE) {
      if (mi + 1 < MF) hfetch(mi + 1, hpre[(mi + 1) & 1]);
    }
    if (mi) wave_lds_sync();  // previous slab fully read
#pragma unroll
    for (int ni = 0; ni < NF; ++ni)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        f32x4 v;
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = acc[mi][ni][4 * q + j];
        *reinterpret_cast<f32x4*>(slab + slab_off<WN>(srow, ni * 8 + 2 * q + shalf)) = v;
      }
    wave_lds_sync();
    const int mbase = wm * WM + mi * 32;  // first tile row of this slab
    if (PAIRED) {
      // slab columns [0, WN/2) are gate features, [WN/2, WN) the matching up features
      constexpr int SEGS = WN / 16, RPP = 64 / SEGS;
#pragma unroll
      for (int pass = 0; pass < 32 / RPP; ++pass) {
        const int r = pass * RPP + lane / SEGS, s = lane % SEGS;
        const int m_local = mbase + r;
        const int f = n_tile * (BN / 2) + wn * (WN / 2) + 8 * s;
        float g[8], u[8], a[8];
        read8<WN>(slab, r, 2 * s, g);
        read8<WN>(slab, r, WN / 8 + 2 * s, u);
        if (m_local < rows && f < p.I) {  // I is a multiple of 8
#pragma unroll
          for (int j = 0; j < 8; ++j) a[j] = swiglu(g[j], u[j]);
          const int64_t row = row0 + m_local;
          bf16_t* hr = static_cast<bf16_t*>(p.out) + row * p.ld_out;
          store8<F16>(hr + f, g);
          store8<F16>(hr + p.I + f, u);
          store8<F16>(static_cast<bf16_t*>(p.out2) + row * p.ld_out2 + f, a);
        }
      }
    } else {
      constexpr int SEGS = WN / 8, RPP = 64 / SEGS;
#pragma unroll
      for (int pass = 0; pass < 32 / RPP; ++pass) {
        const int r = pass * RPP + lane / SEGS, s = lane % SEGS;
        const int m_local = mbase + r;
        const int col = n0 + wn * WN + 8 * s;
        float v[8];
        read8_interleaved<WN>(slab, r, s, v);
        if (MODE == GROUP_M && EPI == EPI_SWIGLU_BWD) {
          // every lane stays to the end: the dw partial is summed over the
          // SEGS lanes that hold one row
          const int64_t row = row0 + m_local;
          float part = 0.f;
          if (m_local < rows && col < p.N) {  // N = I, a multiple of 8
            float g[8], u[8], dg[8], du[8];
            if constexpr (HPRE) {
              unpack8<F16>(hpre[mi & 1][pass][0], g);
              unpack8<F16>(hpre[mi & 1][pass][1], u);
            } else {
              const bf16_t* hr = static_cast<const bf16_t*>(p.aux) + row * p.ld_aux;
              load8<F16>(hr + col, g);
              load8<F16>(hr + p.I + col, u);
            }
            const float wr = p.roww ? p.roww[row] : 1.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j)
              part += v[j] * swiglu_bwd_act(g[j], u[j], wr * v[j], dg[j], du[j]);
            bf16_t* dr = static_cast<bf16_t*>(p.out) + row * p.ld_out;
            store8<F16>(dr + col, dg);
            store8<F16>(dr + p.I + col, du);
          }
          if (p.dwp) {
#pragma unroll
            for (int off = SEGS / 2; off >= 1; off >>= 1) part += __shfl_xor(part, off, kWave);
            if (s == 0 && m_local < rows)
              p.dwp[row * p.dwp_slots + n_tile * WAVES_N + wn] = part;
          }
          continue;
        }
        if (m_local >= rows) continue;
        if (EPI == EPI_STORE_F32) {
          // GROUP_M: router logits; GROUP_K: split-K partial weight gradients
          float* rp = MODE == GROUP_M
                          ? static_cast<float*>(p.out) + (row0 + m_local) * p.ld_out
                          : static_cast<float*>(p.out) + static_cast<int64_t>(e) * p.out_estride +
                                static_cast<int64_t>(m0 + m_local) * p.ld_out;
          if (out_vec4 && col + 8 <= p.N) {
            float4* q = reinterpret_cast<float4*>(rp + col);
            q[0] = make_float4(v[0] * p.scale, v[1] * p.scale, v[2] * p.scale, v[3] * p.scale);
            q[1] = make_float4(v[4] * p.scale, v[5] * p.scale, v[6] * p.scale, v[7] * p.scale);
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
              if (col + j < p.N) rp[col + j] = v[j] * p.scale;
          }
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] *= p.scale;
          // GROUP_M: an expert's row; GROUP_K: feature row m0 + m_local of expert e's gradient
          bf16_t* rp = MODE == GROUP_M
                           ? static_cast<bf16_t*>(p.out) + (row0 + m_local) * p.ld_out
                           : static_cast<bf16_t*>(p.out) + static_cast<int64_t>(e) * p.out_estride +
                                 static_cast<int64_t>(m0 + m_local) * p.ld_out;
          // EPI_ADD source row: aux (merged export) or the output row itself
          const bf16_t* sp = EPI == EPI_ADD && p.aux
                                 ? static_cast<const bf16_t*>(p.aux) + (row0 + m_local) * p.ld_aux
                                 : rp;
          if (out_vec && col + 8 <= p.N && (EPI != EPI_ADD || aux_vec)) {
            if (EPI == EPI_ADD) {
              float o[8];
              load8<F16>(sp + col, o);
#pragma unroll
              for (int j = 0; j < 8; ++j) v[j] += o[j];
            }
            store8<F16>(rp + col, v);
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
              if (col + j < p.N)
                rp[col + j] = f32_to_h16<F16>(EPI == EPI_ADD ? v[j] + h16_to_f32<F16>(sp[col + j]) : v[j]);
          }
        }
      }
    }
  }
}

// ----------------------------------------------------------------- host helpers
constexpr size_t kAlign = 256;
inline size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

inline int ceil_div(int64_t a, int64_t b) { return static_cast<int>((a + b - 1) / b); }

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

Opnd opnd(const void* ptr, int64_t estride, int64_t ld, int kcontig, bool vec_ok) {
  Opnd o;
  o.ptr = ptr;
  o.estride = estride;
  o.ld = ld;
  o.kcontig = kcontig;
  o.vec = vec_ok && (ld % 8 == 0) && aligned16(ptr) && (estride % 8 == 0);
  o.rows = nullptr;
  o.rows_div = 1;
  o.rows_bytes = 0;
  return o;
}

Opnd none() { return Opnd{nullptr, 0, 0, 1, 0, nullptr, 1, 0}; }

template <typename K>
hipError_t launch(K kern, int grid, const GemmArgs& a, hipStream_t s, int threads = 256) {
  if (grid <= 0) return hipSuccess;
  hipLaunchKernelGGL(kern, dim3(grid), dim3(threads), 0, s, a);
  return hipGetLastError();
}

// The 16-bit GEMM instantiation for a layer dtype (MOE_BF16 or MOE_F16); the
// arguments are the tile parameters of gemm16 after F16, VST last.
#define GEMM16(dtype, ...) \
  ((dtype) == MOE_F16 ? gemm16<true, __VA_ARGS__> : gemm16<false, __VA_ARGS__>)

}  // namespace

}  // namespace moe
