// Grouped expert GEMMs of the MoE-LoRA layer: forward and backward.
//
// Per expert e, over its rows X (permuted, expert after expert):
//   forward   h     = X W_gu^T + (s X A_gu^T) B_gu^T       act = silu(h_gate) h_up
//             y_exp = act W_d^T + (s act A_d^T) B_d^T
//   backward  dAct  = G W_d + (s G B_d) A_d                dH = SwiGLU'(h) dAct
//             dX    = dH W_gu + (s dH B_gu) A_gu
//             dB_d  = G^T (s act A_d^T)   dA_d  = (s G B_d)^T act
//             dB_gu = dH^T (s X A_gu^T)   dA_gu = (s dH B_gu)^T X
// The adapter is always applied in the split order (input times A, then B)
// and W + s B A is never formed (Unsloth, "Fine-tune MoE models 12x faster",
// faster-moe page, section "Faster LoRA MoE training"; the LoRA shapes and
// the frozen base weights are in its section "Implementation details"; the
// per-expert loop and the gate/up halves of gate_up_proj in its section
// "What is torch._grouped_mm?"). SwiGLU follows the fused LoRA MLP
// definition in the aiflowlearn.net Unsloth tutorial.
//
// One kernel template covers every product:
//  - GROUP_M: output rows are an expert's rows. A device-built tile list maps
//    each M tile to (expert, first row, valid rows); group sizes never leave
//    the device. The rank-r LoRA term is a second K segment appended to the
//    main K loop ([X | s X A^T] times [W | B]^T), so it costs one extra
//    K step and no extra pass over the output.
//  - GROUP_K: the reduction runs over an expert's rows (the LoRA weight
//    gradients), one block per (expert, M tile, N tile), so no atomics and
//    bit-identical results run to run.
//  - GROUP_KV: GROUP_K for dB = D^T U that also forms, from the D rows it
//    already holds in LDS, float32 partials of the side product D B over its
//    feature tile (summed over tiles by a second kernel), so that D is read
//    once for both.
// Operands are staged through LDS in 16-byte chunks, in the layout they have
// in memory (k-contiguous or output-contiguous, XOR-swizzled); fragments of
// output-contiguous tiles are read with the gfx950 transpose read. 16-bit
// products use v_mfma_f32_32x32x16_bf16 (or _f16) with float32 accumulation;
// the weight fragment is the MFMA A operand so that each lane ends up holding
// consecutive output columns of one row. float32 layers use a plain FMA
// kernel with the same tiling logic.
#include <stdlib.h>

#include <algorithm>
#include <type_traits>

#include "gemm16.h"

namespace moe {

namespace {

// ----------------------------------------------------------------- float32 FMA kernel
// 64 x 64 tiles (paired: 64 gate + 64 up columns), 4 x 4 outputs per thread.
template <int MODE, int EPI, bool PAIRED>
__global__ __launch_bounds__(256) void gemm_f32(GemmArgs p) {
  constexpr int BM = 64, BN = 64, BK = 16, NB = PAIRED ? 2 * BN : BN;
  __shared__ float sA[BK][BM + 4];
  __shared__ float sB[BK][NB + 4];
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;

  int e, n_tile, rows, m0 = 0, krows = 0;
  int64_t row0;
  if (MODE == GROUP_M) {
    const int mtot = *p.ntiles;
    const int total = mtot * p.ntn;
    if (static_cast<int>(blockIdx.x) >= total) return;
    const int mt = blockIdx.x % mtot;
    n_tile = blockIdx.x / mtot;
    const int4 t = p.tiles[mt];
    e = t.x;
    row0 = t.y;
    rows = t.z;
  } else {
    const int total = p.E * p.ntm * p.ntn;
    if (static_cast<int>(blockIdx.x) >= total) return;
    e = blockIdx.x / (p.ntm * p.ntn);
    const int rem = blockIdx.x - e * (p.ntm * p.ntn);
    const int mt = rem / p.ntn;
    n_tile = rem - mt * p.ntn;
    m0 = mt * BM;
    rows = min(BM, p.M - m0);
    row0 = p.offsets[e];
    krows = p.offsets[e + 1] - static_cast<int>(row0);
  }
  const int n0 = PAIRED ? 0 : n_tile * BN;

  float acc[4][4] = {}, accu[4][4] = {};
  const int nseg = MODE == GROUP_M ? 2 : 1;
  for (int seg = 0; seg < nseg; ++seg) {
    const Opnd& A = p.a[seg];
    const Opnd& B = p.b[seg];
    View<float> va{}, vb{};
    va.ld = A.ld; va.kcontig = A.kcontig; vb.ld = B.ld; vb.kcontig = B.kcontig;
    int K;
    if (MODE == GROUP_M) {
      K = p.K[seg];
      va.base = static_cast<const float*>(A.ptr) + row0 * A.ld;
      va.mn_lim = rows;
      if (A.rows) {
        va.base = static_cast<const float*>(A.ptr);
        va.grow = A.rows + row0;
        va.gk = A.rows_div;
      }
      const float* wb = static_cast<const float*>(B.ptr) + static_cast<int64_t>(e) * B.estride;
      if (PAIRED) {
        vb.base = wb; vb.paired = 1; vb.half = BN; vb.pbase = n_tile * BN; vb.I = p.I;
        vb.mn_lim = NB;
      } else {
        vb.base = B.kcontig ? wb + static_cast<int64_t>(n0) * B.ld : wb + n0;
        vb.mn_lim = p.N - n0;
      }
    } else {
      K = krows;
      va.base = static_cast<const float*>(A.ptr) + row0 * A.ld + m0;
      va.mn_lim = p.M - m0;
      if (A.rows) {
        va.base = static_cast<const float*>(A.ptr) + m0;
        va.grow = A.rows + row0;
        va.gk = A.rows_div;
      }
      vb.base = static_cast<const float*>(B.ptr) + row0 * B.ld + n0;
      vb.mn_lim = p.N - n0;
      if (B.rows) {
        vb.base = static_cast<const float*>(B.ptr) + n0;
        vb.grow = B.rows + row0;
        vb.gk = B.rows_div;
      }
    }
    va.klim = K;
    vb.klim = K;
    for (int k0 = 0; k0 < K; k0 += BK) {
      for (int i = tid; i < BM * BK; i += 256) sA[i % BK][i / BK] = load_elem(va, i / BK, k0 + i % BK);
      for (int i = tid; i < NB * BK; i += 256) sB[i % BK][i / BK] = load_elem(vb, i / BK, k0 + i % BK);
      __syncthreads();
#pragma unroll
      for (int kk = 0; kk < BK; ++kk) {
        float a[4], b[4], bu[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = sA[kk][ty * 4 + i];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          b[j] = sB[kk][tx * 4 + j];
          bu[j] = PAIRED ? sB[kk][BN + tx * 4 + j] : 0.f;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            acc[i][j] = fmaf(a[i], b[j], acc[i][j]);
            if (PAIRED) accu[i][j] = fmaf(a[i], bu[j], accu[i][j]);
          }
      }
      __syncthreads();
    }
  }
  if constexpr (!PAIRED && MODE == GROUP_M && EPI == EPI_SWIGLU_BWD) {
    // SwiGLU backward with optional row weights and dw partials (one slot per
    // N tile, summed over the 16 threads of a row: consecutive lanes)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int m_local = ty * 4 + i;
      const int64_t row = row0 + m_local;
      float part = 0.f;
      if (m_local < rows) {
        const float* hr = static_cast<const float*>(p.aux) + row * p.ld_aux;
        float* dr = static_cast<float*>(p.out) + row * p.ld_out;
        const float wr = p.roww ? p.roww[row] : 1.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int col = n0 + tx * 4 + j;
          if (col < p.N) {
            const float g = hr[col], u = hr[p.I + col];
            float dg, du;
            part += acc[i][j] * swiglu_bwd_act(g, u, wr * acc[i][j], dg, du);
            dr[col] = dg;
            dr[p.I + col] = du;
          }
        }
      }
      if (p.dwp) {
#pragma unroll
        for (int off = 8; off >= 1; off >>= 1) part += __shfl_xor(part, off, kWave);
        if (tx == 0 && m_local < rows) p.dwp[row * p.dwp_slots + n_tile] = part;
      }
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float v[4], u[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[j] = acc[i][j];
      u[j] = accu[i][j];
    }
    if (PAIRED) {
      epi_swiglu<float>(p, row0, ty * 4 + i, rows, n_tile * BN + tx * 4, v, u);
    } else {
      const int64_t rbase = MODE == GROUP_M ? row0 : static_cast<int64_t>(m0);
      epi_store<float, MODE, EPI>(p, e, rbase, ty * 4 + i, rows, n0 + tx * 4, v);
    }
  }
}

// ----------------------------------------------------------------- tile list
// One block of 1024 threads (E <= 1024). Two lists in one launch, for two tile
// heights: M tiles of `bm` rows per expert, in expert order, with their raster
// groups (group_tile); empty experts get none.
__global__ __launch_bounds__(1024) void tiles_kernel(const int32_t* __restrict__ offsets, int E,
                                                     int bm0, int4* __restrict__ tiles0,
                                                     int32_t* __restrict__ ntiles0, int bm1,
                                                     int4* __restrict__ tiles1,
                                                     int32_t* __restrict__ ntiles1) {
  __shared__ int wsum[2][1024 / kWave];
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const int e = threadIdx.x;
  int lo = 0, cnt = 0;
  if (e < E) {
    lo = offsets[e];
    cnt = offsets[e + 1] - lo;
  }
#pragma unroll
  for (int l = 0; l < 2; ++l) {
    const int bm = l ? bm1 : bm0;
    int4* tiles = l ? tiles1 : tiles0;
    const int nt = (cnt + bm - 1) / bm;
    int incl = nt;
#pragma unroll
    for (int off = 1; off < kWave; off <<= 1) {
      int o = __shfl_up(incl, off, kWave);
      if (lane >= off) incl += o;
    }
    if (lane == kWave - 1) wsum[l][wave] = incl;
    __syncthreads();
    int base = 0, total = 0;
    for (int w = 0; w < 1024 / kWave; ++w) {
      if (w < wave) base += wsum[l][w];
      total += wsum[l][w];
    }
    base += incl - nt;
    for (int i = 0; i < nt; ++i) {
      const int r = i * bm;
      const int g0 = i / kTileGroup * kTileGroup;
      const int grp = (base + g0) * 16 + min(kTileGroup, nt - g0);
      tiles[base + i] = make_int4(e, lo + r, min(bm, cnt - r), grp);
    }
    if (threadIdx.x == 0) *(l ? ntiles1 : ntiles0) = total;
  }
}

// ----------------------------------------------------------------- host side
inline int esz_of(const ExpertDims& d) { return d.dtype == MOE_F32 ? 4 : 2; }

// The layer input [rows, ld] as an operand: x_perm as it is, or x in token
// order read through sorted_pair.
Opnd opnd_x(const XRows& x, int64_t ld, int kcontig, int esz) {
  Opnd o = opnd(x.ptr, 0, ld, kcontig, true);
  if (x.rows) {
    o.rows = x.rows;
    o.rows_div = x.k;
    o.rows_bytes = static_cast<int64_t>(x.T) * ld * esz;
  }
  return o;
}

// Tile list capacity for `bm`-row tiles.
inline int64_t tile_cap(int64_t N, int E, int bm) { return (N + bm - 1) / bm + E + 1; }

// Two device-built tile lists: `small` (the LoRA side products and the
// float32 kernels) and `big` (the four expert GEMMs; its tile height depends
// on the tile variant).
struct TileList {
  int4* tiles;
  int32_t* ntiles;
  int bm;
};

struct WsLayout {
  TileList small, big;
  size_t bytes;
};

inline int small_rows(int dtype) { return dtype != MOE_F32 ? 128 : 64; }
// 256-row tiles for the register-staged kernel, whose LoRA segment (K = r)
// must come in 16-byte pieces.
inline int big_rows(const ExpertDims& d) {
  if (d.dtype == MOE_F32) return 64;
  return d.r % 8 == 0 ? 256 : 128;
}

WsLayout tile_ws(void* ws, const ExpertDims& d) {
  WsLayout L;
  char* p = static_cast<char*>(ws);
  size_t off = 0;
  auto list = [&](int bm) {
    TileList t;
    t.bm = bm;
    t.tiles = reinterpret_cast<int4*>(p + off);
    off += align_up(static_cast<size_t>(tile_cap(d.N, d.E, bm)) * sizeof(int4));
    t.ntiles = reinterpret_cast<int32_t*>(p + off);
    off += kAlign;
    return t;
  };
  L.small = list(small_rows(d.dtype));
  L.big = list(big_rows(d));
  L.bytes = off;
  return L;
}

inline hipError_t build_tiles(const WsLayout& L, const int32_t* offsets, int E, hipStream_t s) {
  hipLaunchKernelGGL(tiles_kernel, dim3(1), dim3(1024), 0, s, offsets, E, L.small.bm,
                     L.small.tiles, L.small.ntiles, L.big.bm, L.big.tiles, L.big.ntiles);
  return hipGetLastError();
}

// Tiles of the four expert GEMMs, chosen by measurement on MI355X:
//  - 256 x 256, eight waves of 128 x 64, BK 64, two LDS slots (128 KB),
//    operands staged through VGPRs (one k tile in flight per wave): the
//    default. A wave issues buffer->LDS DMA at about a quarter of the rate it
//    issues buffer loads into VGPRs, so register staging keeps the MFMAs fed
//    with fewer bytes in flight; 256-row tiles also halve the L2 traffic per
//    MFMA relative to 128 x 256.
//  - 256 x 256 with buffer->LDS DMA fills (128 x 128 per wave, BK 32, three
//    stages) when an operand cannot be read in 16-byte pieces (a pointer that
//    is not 16-byte aligned): the DMA fill falls back to element-wise loads.
//  - 128 x 256, four waves, buffer->LDS DMA, BK 32, three stages, two blocks
//    per CU: ranks that are not a multiple of 8 (the LoRA segment, K = r,
//    then takes element-wise fills).
inline bool all_vec(const GemmArgs& a) {
  return a.a[0].vec && a.b[0].vec && (a.K[1] == 0 || (a.a[1].vec && a.b[1].vec));
}

// Wave columns per N tile of the kernel launch_big runs (the dw partial
// slots of a SwiGLU-backward launch): 256 / 64 for the register-staged
// kernel, 256 / 128 for the other two.
inline int big_waves_n(const GemmArgs& a, int bm) { return bm == 256 && all_vec(a) ? 4 : 2; }

template <int MODE, int EPI, bool PAIRED, bool A_KC, bool B_KC>
hipError_t launch_big(int grid, const GemmArgs& a, hipStream_t s, int bm) {
  if (bm == 256) {
    if (!all_vec(a))
      return launch(GEMM16(a.dtype, 256, 256, 128, 128, 32, 3, 1, MODE, EPI, PAIRED, A_KC, B_KC, 0), grid, a, s);
    return launch(GEMM16(a.dtype, 256, 256, 128, 64, 64, 2, 1, MODE, EPI, PAIRED, A_KC, B_KC, 1), grid, a, s, 512);
  }
  return launch(GEMM16(a.dtype, 128, 256, 64, 128, 32, 3, 2, MODE, EPI, PAIRED, A_KC, B_KC, 0), grid, a, s);
}

// M-tile grid bound for GROUP_M launches over a tile list (excess blocks exit at once).
inline int gm_grid(const ExpertDims& d, const TileList& t, int ntn) {
  return static_cast<int>(tile_cap(d.N, d.E, t.bm) * ntn);
}

GemmArgs base_args(const ExpertDims& d, const int32_t* offsets, const TileList& t) {
  GemmArgs a{};
  a.a[1] = none();
  a.b[1] = none();
  a.E = d.E;
  a.offsets = offsets;
  a.tiles = t.tiles;
  a.ntiles = t.ntiles;
  a.I = d.I;
  a.scale = 1.0f;
  a.dtype = d.dtype;
  return a;
}

// out[rows, r] = scale * A[rows, K] * L_e (L_e is [r, K] when l_kcontig, else [K, r]).
hipError_t side_product(const ExpertDims& d, const int32_t* offsets, const WsLayout& L,
                        const Opnd& A, int K, const void* Lw, int64_t l_estride, int l_kcontig,
                        void* out, hipStream_t s) {
  const TileList& t = L.small;
  GemmArgs a = base_args(d, offsets, t);
  const bool r_vec = d.r % 8 == 0;
  a.a[0] = A;
  a.b[0] = l_kcontig ? opnd(Lw, l_estride, K, 1, true) : opnd(Lw, l_estride, d.r, 0, r_vec);
  a.K[0] = K;
  a.K[1] = 0;
  a.N = d.r;
  a.out = out;
  a.ld_out = d.r;
  a.scale = d.scale;
  if (d.dtype != MOE_F32) {
    a.ntn = 1;
    if (l_kcontig) {
      if (d.r <= 32)
        return launch(GEMM16(a.dtype, 128, 32, 32, 32, 64, 3, 2, GROUP_M, EPI_STORE, false, true, true, 0),
                      gm_grid(d, t, 1), a, s);
      return launch(GEMM16(a.dtype, 128, 64, 32, 64, 64, 3, 2, GROUP_M, EPI_STORE, false, true, true, 0),
                    gm_grid(d, t, 1), a, s);
    }
    if (d.r <= 32)
      return launch(GEMM16(a.dtype, 128, 32, 32, 32, 64, 3, 2, GROUP_M, EPI_STORE, false, true, false, 0),
                    gm_grid(d, t, 1), a, s);
    return launch(GEMM16(a.dtype, 128, 64, 32, 64, 64, 3, 2, GROUP_M, EPI_STORE, false, true, false, 0),
                  gm_grid(d, t, 1), a, s);
  }
  a.ntn = ceil_div(d.r, 64);
  return launch(gemm_f32<GROUP_M, EPI_STORE, false>, gm_grid(d, t, a.ntn), a, s);
}

// ---- weight gradients: out_e[P, Q] = sum over the expert's rows n of L[n, P] R[n, Q]
// (L: [rows, P], R: [rows, Q]). One workgroup owns an output tile and runs
// over all the expert's rows, so no atomics are needed and the result does not
// depend on scheduling. When the experts are too few to give every CU a tile
// (a shared expert is one expert over all T tokens), each expert's rows are
// cut into S contiguous chunks that act as experts of their own, every chunk
// writes a float32 partial into the workspace, and a second kernel sums the S
// partials of each expert in chunk order (still deterministic).

// Tiles per expert of the kernel weight_grad picks for [P, Q].
int wgrad_tiles(const ExpertDims& d, int P, int Q) {
  if (d.dtype == MOE_F32) return ceil_div(P, 64) * ceil_div(Q, 64);
  if (Q <= 64 && P > 64) return ceil_div(P, 256);
  if (P >= 256 && Q >= 256) return ceil_div(P, 128) * ceil_div(Q, 256);
  return (P <= 32 ? 1 : ceil_div(P, 64)) * ceil_div(Q, 256);
}

// Row chunks per expert: enough to reach ~512 workgroups when fewer than 256
// would run, never chunks of fewer than 256 rows on average, and only for the
// LoRA gradients of rank <= 32 (the full fine-tuning gradients have tiles
// enough and would need large partials; higher ranks are rare).
int wgrad_splits(const ExpertDims& d, int P, int Q) {
  if (std::min(P, Q) > 32) return 1;
  const int64_t blocks = static_cast<int64_t>(d.E) * wgrad_tiles(d, P, Q);
  if (blocks >= 256) return 1;
  const int64_t by_rows = static_cast<int64_t>(d.N) / (static_cast<int64_t>(d.E) * 256);
  const int64_t want = (512 + blocks - 1) / blocks;
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({want, by_rows, 64})));
}

// Workspace for the split path of one [P, Q] gradient: chunk offsets, then partials.
size_t wgrad_split_bytes(const ExpertDims& d, int P, int Q) {
  const int S = wgrad_splits(d, P, Q);
  if (S <= 1) return 0;
  const int64_t G = static_cast<int64_t>(d.E) * S;
  return align_up(static_cast<size_t>(G + 1) * 4) + align_up(static_cast<size_t>(G) * P * Q * 4);
}

// The largest split workspace over the four LoRA gradients of the backward.
size_t lora_wgrad_split_bytes(const ExpertDims& d) {
  const int H = d.H, I = d.I, r = d.r;
  return std::max({wgrad_split_bytes(d, H, r), wgrad_split_bytes(d, r, I),
                   wgrad_split_bytes(d, 2 * I, r), wgrad_split_bytes(d, r, H)});
}

// Chunk c of expert e covers rows [off[e] + cnt_e c / S, off[e] + cnt_e (c + 1) / S).
__global__ void split_offsets_kernel(const int32_t* __restrict__ off, int E, int S,
                                     int32_t* __restrict__ voff) {
  for (int i = threadIdx.x; i < E * S; i += blockDim.x) {
    const int e = i / S, c = i - e * S;
    const int64_t cnt = off[e + 1] - off[e];
    voff[i] = off[e] + static_cast<int32_t>(cnt * c / S);
  }
  if (threadIdx.x == 0) voff[E * S] = off[E];
}

template <typename Elem>
__global__ __launch_bounds__(256) void reduce_splits_kernel(const float* __restrict__ part,
                                                            Elem* __restrict__ out, int S,
                                                            int64_t PQ, int64_t total) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (i >= total) return;
  const int64_t e = i / PQ, q = i - e * PQ;
  const float* p = part + e * S * PQ + q;
  float acc = 0.f;
  for (int c = 0; c < S; ++c) acc += p[c * PQ];
  out[i] = from_f32<Elem>(acc);
}

// One weight-gradient tile shape (BK 32, three stages, two blocks per CU): the
// instantiation that reads A's rows (GA) or B's rows (GB) through their row
// list when that operand has one. Shapes without that instantiation refuse a
// row list, as does a launch with both.
template <int BM, int BN, int WM, int WN, int MODE, int EPI, bool GA, bool GB>
hipError_t launch_wg(const GemmArgs& a, int grid, hipStream_t s) {
  const bool ra = a.a[0].rows != nullptr, rb = a.b[0].rows != nullptr;
  if (ra && rb) return hipErrorInvalidValue;
  if (ra) {
    if constexpr (GA)
      return launch(GEMM16(a.dtype, BM, BN, WM, WN, 32, 3, 2, MODE, EPI, false, false, false, 0, 1),
                    grid, a, s);
    return hipErrorInvalidValue;
  }
  if (rb) {
    if constexpr (GB)
      return launch(GEMM16(a.dtype, BM, BN, WM, WN, 32, 3, 2, MODE, EPI, false, false, false, 0, 2),
                    grid, a, s);
    return hipErrorInvalidValue;
  }
  return launch(GEMM16(a.dtype, BM, BN, WM, WN, 32, 3, 2, MODE, EPI, false, false, false, 0),
                grid, a, s);
}

template <int EPI>
hipError_t weight_grad_launch(const ExpertDims& d, GemmArgs& a, int E, int P, int Q,
                              hipStream_t s) {
  if (a.vp) {  // [big, r <= 32] with side-product partials (checked by the caller)
    a.ntn = 1;
    a.ntm = ceil_div(P, 256);
    return launch_wg<256, 32, 64, 32, GROUP_KV, EPI, true, false>(a, E * a.ntm, s);
  }
  if (d.dtype != MOE_F32) {
    // Split partials (EPI_STORE_F32) only come from gradients with a side of
    // at most 32 (wgrad_splits): the other tile shapes exist for EPI_STORE only.
    constexpr bool WIDE = EPI == EPI_STORE;
    if (Q <= 64 && P > 64) {  // [big, r]
      a.ntn = 1;
      a.ntm = ceil_div(P, 256);
      if (Q <= 32) return launch_wg<256, 32, 64, 32, GROUP_K, EPI, true, false>(a, E * a.ntm, s);
      if constexpr (WIDE)
        return launch_wg<256, 64, 64, 64, GROUP_K, EPI, true, false>(a, E * a.ntm, s);
      return hipErrorInvalidValue;
    }
    if (P >= 256 && Q >= 256) {  // [big, big]: full fine-tuning weight gradients
      if constexpr (WIDE) {
        a.ntm = ceil_div(P, 128);
        a.ntn = ceil_div(Q, 256);
        return launch_wg<128, 256, 64, 128, GROUP_K, EPI, false, true>(a, E * a.ntm * a.ntn, s);
      }
      return hipErrorInvalidValue;
    }
    // [r, big] (or both small)
    a.ntn = ceil_div(Q, 256);
    if (P <= 32) {
      a.ntm = 1;
      return launch_wg<32, 256, 32, 64, GROUP_K, EPI, false, true>(a, E * a.ntn, s);
    }
    if constexpr (WIDE) {
      a.ntm = ceil_div(P, 64);
      return launch_wg<64, 256, 64, 64, GROUP_K, EPI, true, true>(a, E * a.ntm * a.ntn, s);
    }
    return hipErrorInvalidValue;
  }
  a.ntm = ceil_div(P, 64);
  a.ntn = ceil_div(Q, 64);
  return launch(gemm_f32<GROUP_K, EPI_STORE, false>, E * a.ntm * a.ntn, a, s);
}

#define MOE_TRY_WG(x)                   \
  do {                                  \
    hipError_t err_ = (x);              \
    if (err_ != hipSuccess) return err_; \
  } while (0)

// Side product fused into a LoRA B gradient (see GROUP_KV): alongside
// dB = D^T U it forms V = scale * D Bm with Bm per expert [P, Q].
struct SideOut {
  const void* bm = nullptr;   // [E][P][Q]
  void* out = nullptr;        // V [N, Q] in the layer dtype
  float* part = nullptr;      // ceil(P / 256) x N x Q float32 partials
  const float* roww = nullptr;  // optional: also out_w[n] = roww[n] V[n] (one rounding)
  void* out_w = nullptr;
};

// The fused path covers 16-bit layers, Q = r <= 32 with rows of 16 bytes.
// The partials cost ceil(P / 256) x Q float32 per row each way; past 2 KB a
// row (512 values: DeepSeek-V3's dB_d, 28 tiles at r = 32) reading D a second
// time in a plain side-product GEMM was faster on MI355X (0.45 against
// 0.53 ms), at 2 KB the two were even (DeepSeek-V3's dB_gu), below it fusing
// wins (gpt-oss-20b's dB_gu, 1.5 KB: 0.11 against 0.17 ms).
inline bool side_fusable(const ExpertDims& d, int P, int Q) {
  return d.dtype != MOE_F32 && Q <= 32 && Q % 8 == 0 && P % 8 == 0 && P > 64 &&
         ceil_div(P, 256) * Q <= 512;
}

inline size_t side_part_bytes(const ExpertDims& d) {
  int P = 0;
  for (const int p : {d.H, 2 * d.I})
    if (side_fusable(d, p, d.r)) P = std::max(P, p);
  return static_cast<size_t>(ceil_div(P, 256)) * d.N * d.r * 4;
}

// V[i] = scale * sum over tiles t (in order) of part[t][i]; with roww, also
// out_w[i] = roww[i / Q] * V[i] (from the float32 sum, one rounding).
template <typename Elem>
__global__ __launch_bounds__(256) void side_sum_kernel(const float* __restrict__ part, int tiles,
                                                       int64_t tstride, float scale,
                                                       Elem* __restrict__ out,
                                                       const float* __restrict__ roww, int Q,
                                                       Elem* __restrict__ out_w) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (i >= tstride) return;
  float acc = 0.f;
  for (int t = 0; t < tiles; ++t) acc += part[t * tstride + i];
  out[i] = from_f32<Elem>(acc * scale);
  if (roww) out_w[i] = from_f32<Elem>(roww[i / Q] * (acc * scale));
}

// dst[n][c] = w[n] * src[n][c] over rows x cols (dst may be src), one rounding.
// VEC (16-bit, cols % 8 == 0, both 16-byte aligned: the dY rows of full
// fine-tuning) one 16-byte piece per thread; otherwise (float32 rows, and the
// [N, r] side products when r % 8 != 0) one element per thread.
template <typename Elem, bool VEC>
__global__ __launch_bounds__(256) void scale_rows_kernel(const Elem* src, const float* __restrict__ w,
                                                         int64_t total, int cols, Elem* dst) {
  const int64_t i = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) * (VEC ? 8 : 1);
  if (i >= total) return;
  const float wr = w[i / cols];
  if constexpr (VEC) {
    u32x4 v = *reinterpret_cast<const u32x4*>(src + i);
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const uint16_t lo = static_cast<uint16_t>(v[t] & 0xffffu), hi = static_cast<uint16_t>(v[t] >> 16);
      const float a = wr * to_f32<Elem>(__builtin_bit_cast(Elem, lo));
      const float b = wr * to_f32<Elem>(__builtin_bit_cast(Elem, hi));
      v[t] = static_cast<uint32_t>(__builtin_bit_cast(uint16_t, from_f32<Elem>(a))) |
             (static_cast<uint32_t>(__builtin_bit_cast(uint16_t, from_f32<Elem>(b))) << 16);
    }
    *reinterpret_cast<u32x4*>(dst + i) = v;
  } else {
    dst[i] = from_f32<Elem>(wr * to_f32<Elem>(src[i]));
  }
}

hipError_t scale_rows(int dtype, const void* src, const float* w, int64_t rows, int cols,
                      void* dst, hipStream_t s) {
  const int64_t total = rows * cols;
  if (total <= 0) return hipSuccess;
  const bool vec = dtype != MOE_F32 && cols % 8 == 0 && aligned16(src) && aligned16(dst);
  const dim3 grid(static_cast<unsigned>((total / (vec ? 8 : 1) + 255) / 256));
  if (dtype == MOE_BF16) {
    auto k = vec ? scale_rows_kernel<bf16_t, true> : scale_rows_kernel<bf16_t, false>;
    hipLaunchKernelGGL(k, grid, dim3(256), 0, s, static_cast<const bf16_t*>(src), w, total, cols,
                       static_cast<bf16_t*>(dst));
  } else if (dtype == MOE_F16) {
    auto k = vec ? scale_rows_kernel<f16_t, true> : scale_rows_kernel<f16_t, false>;
    hipLaunchKernelGGL(k, grid, dim3(256), 0, s, static_cast<const f16_t*>(src), w, total, cols,
                       static_cast<f16_t*>(dst));
  } else {
    auto k = scale_rows_kernel<float, false>;
    hipLaunchKernelGGL(k, grid, dim3(256), 0, s, static_cast<const float*>(src), w, total, cols,
                       static_cast<float*>(dst));
  }
  return hipGetLastError();
}

// split_ws: at least wgrad_split_bytes(d, P, Q) bytes (unused when that is 0),
// or null: then the rows are never split (one workgroup per output tile runs
// over all of an expert's rows), whatever wgrad_splits would choose.
// side (optional, side_fusable only): also form V = scale D Bm.
hipError_t weight_grad(const ExpertDims& d, const int32_t* offsets, const void* Lm, int P,
                       const void* Rm, int Q, void* out, hipStream_t s, void* split_ws,
                       const SideOut* side = nullptr, const XRows* rx = nullptr,
                       const XRows* lx = nullptr) {
  if (lx && rx) return hipErrorInvalidValue;  // at most one operand's rows are gathered
  GemmArgs a{};
  a.vsplit = 1;
  if (side) {
    a.vb = side->bm;
    a.vb_estride = static_cast<int64_t>(P) * Q;
    a.vp = side->part;
    a.vp_tstride = d.N * Q;
  }
  a.a[1] = none();
  a.b[1] = none();
  a.M = P;
  a.N = Q;
  a.scale = 1.0f;
  a.dtype = d.dtype;
  a.out_estride = static_cast<int64_t>(P) * Q;
  a.ld_out = Q;
  a.a[0] = lx ? opnd_x(*lx, P, 0, esz_of(d)) : opnd(Lm, 0, P, 0, P % 8 == 0);
  a.b[0] = rx ? opnd_x(*rx, Q, 0, esz_of(d)) : opnd(Rm, 0, Q, 0, Q % 8 == 0);
  const int S = split_ws ? wgrad_splits(d, P, Q) : 1;
  auto side_sum = [&]() -> hipError_t {
    if (!side) return hipSuccess;
    const int tiles = ceil_div(P, 256);
    const int64_t n = d.N * Q;
    const dim3 grid(static_cast<unsigned>((n + 255) / 256));
    if (d.dtype == MOE_BF16)
      hipLaunchKernelGGL(side_sum_kernel<bf16_t>, grid, dim3(256), 0, s, side->part, tiles, n,
                         d.scale, static_cast<bf16_t*>(side->out), side->roww, Q,
                         static_cast<bf16_t*>(side->out_w));
    else
      hipLaunchKernelGGL(side_sum_kernel<f16_t>, grid, dim3(256), 0, s, side->part, tiles, n,
                         d.scale, static_cast<f16_t*>(side->out), side->roww, Q,
                         static_cast<f16_t*>(side->out_w));
    return hipGetLastError();
  };
  if (S <= 1) {
    a.E = d.E;
    a.offsets = offsets;
    a.out = out;
    MOE_TRY_WG(weight_grad_launch<EPI_STORE>(d, a, d.E, P, Q, s));
    return side_sum();
  }
  const int G = d.E * S;
  a.vsplit = S;
  int32_t* voff = static_cast<int32_t*>(split_ws);
  float* part = reinterpret_cast<float*>(static_cast<char*>(split_ws) +
                                         align_up(static_cast<size_t>(G + 1) * 4));
  hipLaunchKernelGGL(split_offsets_kernel, dim3(1), dim3(256), 0, s, offsets, d.E, S, voff);
  a.E = G;
  a.offsets = voff;
  a.out = part;
  hipError_t e = weight_grad_launch<EPI_STORE_F32>(d, a, G, P, Q, s);
  if (e != hipSuccess) return e;
  const int64_t PQ = static_cast<int64_t>(P) * Q, total = static_cast<int64_t>(d.E) * PQ;
  const dim3 grid(static_cast<unsigned>((total + 255) / 256));
  if (d.dtype == MOE_BF16)
    hipLaunchKernelGGL(reduce_splits_kernel<bf16_t>, grid, dim3(256), 0, s, part,
                       static_cast<bf16_t*>(out), S, PQ, total);
  else if (d.dtype == MOE_F16)
    hipLaunchKernelGGL(reduce_splits_kernel<f16_t>, grid, dim3(256), 0, s, part,
                       static_cast<f16_t*>(out), S, PQ, total);
  else
    hipLaunchKernelGGL(reduce_splits_kernel<float>, grid, dim3(256), 0, s, part,
                       static_cast<float*>(out), S, PQ, total);
  MOE_TRY_WG(hipGetLastError());
  return side_sum();
}

#define MOE_TRY(x)                      \
  do {                                  \
    hipError_t err_ = (x);              \
    if (err_ != hipSuccess) return err_; \
  } while (0)

}  // namespace

size_t experts_fwd_ws_bytes(const ExpertDims& d) {
  return tile_ws(nullptr, d).bytes;
}

namespace {

// dw partial slots per row of the down backward (the combine backward folded
// into it): one per wave column of every N tile of the SwiGLU-backward GEMM,
// the most any of its kernels uses (256-wide tiles of 64-wide waves; float32
// layers 64-wide tiles of one slot).
inline int dw_slots_max(const ExpertDims& d) {
  return d.dtype == MOE_F32 ? ceil_div(d.I, 64) : ceil_div(d.I, 256) * 4;
}

// Backward workspace: tile lists, G B_d and dH B_gu [N, r], dH [N, 2I],
// split-K and side-product partials; for the combine backward folded in,
// also the permuted routing weights [N] f32, w u_d and w G B_d [N, r] and
// the dw partials [slots, N] f32.
struct BwdWs {
  WsLayout L;
  void *gb, *dhb, *dh, *split;
  float* vpart;
  float* w_perm;
  void *wu_d, *gbw;
  float* dwp;
  size_t bytes;
};

BwdWs bwd_ws(void* ws, const ExpertDims& d) {
  const size_t esz = d.dtype == MOE_F32 ? 4 : 2;
  BwdWs B;
  B.L = tile_ws(ws, d);
  char* base = static_cast<char*>(ws);
  size_t off = B.L.bytes;
  auto take = [&](size_t n) {
    void* q = base ? base + off : nullptr;
    off += align_up(n);
    return q;
  };
  B.gb = take(static_cast<size_t>(d.N) * d.r * esz);
  B.dhb = take(static_cast<size_t>(d.N) * d.r * esz);
  B.dh = take(static_cast<size_t>(d.N) * 2 * d.I * esz);
  B.split = take(lora_wgrad_split_bytes(d));
  B.vpart = static_cast<float*>(take(d.dtype != MOE_F32 ? side_part_bytes(d) : 0));
  B.w_perm = static_cast<float*>(take(static_cast<size_t>(d.N) * 4));
  B.wu_d = take(static_cast<size_t>(d.N) * d.r * esz);
  B.gbw = take(static_cast<size_t>(d.N) * d.r * esz);
  B.dwp = static_cast<float*>(take(static_cast<size_t>(dw_slots_max(d)) * d.N * 4));
  B.bytes = off;
  return B;
}

}  // namespace

size_t experts_bwd_ws_bytes(const ExpertDims& d) { return bwd_ws(nullptr, d).bytes; }

namespace {

// h = X W_gu^T + u_gu B_gu^T ; act = SwiGLU(h)   (tile lists already built)
hipError_t launch_gate_up(const ExpertDims& d, const WsLayout& L, const XRows& x,
                          const int32_t* offsets, const moe_weights& w, const void* u_gu,
                          void* h, void* act, hipStream_t s, KernelTimer* tm) {
  const int H = d.H, I = d.I, r = d.r;
  GemmArgs a = base_args(d, offsets, L.big);
  a.a[0] = opnd_x(x, H, 1, esz_of(d));
  a.b[0] = opnd(w.w_gu, static_cast<int64_t>(2) * I * H, H, 1, true);
  a.a[1] = opnd(u_gu, 0, r, 1, r % 8 == 0);
  a.b[1] = opnd(w.b_gu, static_cast<int64_t>(2) * I * r, r, 1, r % 8 == 0);
  a.K[0] = H;
  a.K[1] = r;
  a.N = 2 * I;
  a.out = h;
  a.ld_out = 2 * I;
  a.out2 = act;
  a.ld_out2 = I;
  TimedScope ts(tm, MOE_K_GATE_UP_FWD, s);
  if (d.dtype != MOE_F32) {
    a.ntn = ceil_div(I, 128);
    return launch_big<GROUP_M, EPI_SWIGLU, true, true, true>(gm_grid(d, L.big, a.ntn), a, s,
                                                              L.big.bm);
  }
  a.ntn = ceil_div(I, 64);
  return launch(gemm_f32<GROUP_M, EPI_SWIGLU, true>, gm_grid(d, L.big, a.ntn), a, s);
}

// Recompute mode: h [N, 2I] and act [N, I] live in scratch after `base_bytes`.
inline size_t lean_extra_bytes(const ExpertDims& d) {
  const size_t esz = d.dtype == MOE_F32 ? 4 : 2;
  return align_up(static_cast<size_t>(d.N) * 2 * d.I * esz) +
         align_up(static_cast<size_t>(d.N) * d.I * esz);
}

inline moe_saved lean_saved(const ExpertDims& d, const moe_saved& sv, void* ws, size_t base_bytes) {
  const size_t esz = d.dtype == MOE_F32 ? 4 : 2;
  moe_saved out = sv;
  char* p = static_cast<char*>(ws) + align_up(base_bytes);
  out.h = p;
  out.act = p + align_up(static_cast<size_t>(d.N) * 2 * d.I * esz);
  return out;
}

}  // namespace

hipError_t launch_experts_fwd(const ExpertDims& d, const XRows& x, const int32_t* offsets,
                              const moe_weights& w, const moe_saved& sv, void* ws,
                              hipStream_t s, KernelTimer* tm) {
  const WsLayout L = tile_ws(ws, d);
  const int H = d.H, I = d.I, r = d.r;
  MOE_TRY(build_tiles(L, offsets, d.E, s));
  {  // u_gu = s X A_gu^T
    TimedScope ts(tm, MOE_K_LORA_SIDE, s);
    MOE_TRY(side_product(d, offsets, L, opnd_x(x, H, 1, esz_of(d)), H, w.a_gu,
                         static_cast<int64_t>(r) * H, 1, sv.u_gu, s));
  }
  MOE_TRY(launch_gate_up(d, L, x, offsets, w, sv.u_gu, sv.h, sv.act, s, tm));
  {  // u_d = s act A_d^T
    TimedScope ts(tm, MOE_K_LORA_SIDE, s);
    MOE_TRY(side_product(d, offsets, L, opnd(sv.act, 0, I, 1, true), I, w.a_d,
                         static_cast<int64_t>(r) * I, 1, sv.u_d, s));
  }
  {  // y_exp = act W_d^T + u_d B_d^T
    GemmArgs a = base_args(d, offsets, L.big);
    a.a[0] = opnd(sv.act, 0, I, 1, true);
    a.b[0] = opnd(w.w_d, static_cast<int64_t>(H) * I, I, 1, true);
    a.a[1] = opnd(sv.u_d, 0, r, 1, r % 8 == 0);
    a.b[1] = opnd(w.b_d, static_cast<int64_t>(H) * r, r, 1, r % 8 == 0);
    a.K[0] = I;
    a.K[1] = r;
    a.N = H;
    a.out = sv.y_exp;
    a.ld_out = H;
    TimedScope ts(tm, MOE_K_DOWN_FWD, s);
    if (d.dtype != MOE_F32) {
      a.ntn = ceil_div(H, 256);
      MOE_TRY((launch_big<GROUP_M, EPI_STORE, false, true, true>( gm_grid(d, L.big, a.ntn),
                     a, s, L.big.bm)));
    } else {
      a.ntn = ceil_div(H, 64);
      MOE_TRY(launch(gemm_f32<GROUP_M, EPI_STORE, false>, gm_grid(d, L.big, a.ntn), a, s));
    }
  }
  return hipSuccess;
}

hipError_t launch_experts_bwd(const ExpertDims& d, const void* g, const XRows& x,
                              const int32_t* offsets, const moe_weights& w,
                              const moe_saved& sv, void* dx_perm, const moe_lora_grads& gr,
                              const moe_base_grads* base, void* ws, hipStream_t s,
                              KernelTimer* tm, const CombineBwd* cb) {
  const BwdWs B = bwd_ws(ws, d);
  const WsLayout& L = B.L;
  const int H = d.H, I = d.I, r = d.r;
  void* gb = B.gb;    // s G B_d (with cb: s dY B_d, unweighted)
  void* dhb = B.dhb;  // s dH B_gu
  void* dh = B.dh;
  void* split = B.split;
  // The side products G B_d and dH B_gu read the same matrices as the
  // gradients dB_d = G^T u_d and dB_gu = dH^T u_gu; where the shapes allow,
  // one kernel reads each matrix once for both.
  const bool fuse_d = side_fusable(d, H, r) && aligned16(w.b_d);
  const bool fuse_gu = side_fusable(d, 2 * I, r) && aligned16(w.b_gu);

  MOE_TRY(build_tiles(L, offsets, d.E, s));
  // With the combine backward folded in, g holds dY's rows unweighted and
  // every consumer of G = w dY applies w itself: dB_d = dY^T (w u_d); the
  // down backward runs on dY and its epilogue scales the product by w (dw
  // comes from the unweighted product); dA_d = (w s dY B_d)^T act; the full
  // fine-tuning dW_d = (w dY)^T act after the rows are scaled in place.
  // With cb->gather_dy (never with base) those rows are not copied: the
  // GEMMs read row sorted_pair[i] / k of dY for permuted row i.
  const bool dyg = cb && cb->gather_dy;
  if (dyg && base) return hipErrorInvalidValue;
  const XRows dyr{cb ? cb->dy : nullptr, cb ? cb->sorted_pair : nullptr, cb ? cb->k : 1,
                  cb ? cb->T : 0};
  const Opnd g_rows = dyg ? opnd_x(dyr, H, 1, esz_of(d)) : opnd(g, 0, H, 1, true);
  const XRows* g_lx = dyg ? &dyr : nullptr;
  const void* ud_eff = sv.u_d;   // right operand of dB_d
  const void* gb_da = gb;        // left operand of dA_d
  if (cb && !dyg) {
    TimedScope ts(tm, MOE_K_DY_GATHER, s);
    const int64_t row_bytes = static_cast<int64_t>(H) * (d.dtype == MOE_F32 ? 4 : 2);
    MOE_TRY(launch_gather(cb->dy, cb->sorted_pair, offsets, d.E, cb->k, d.N, row_bytes,
                          const_cast<void*>(g), s, nullptr));
  }
  if (cb) {  // w of each permuted row, and w u_d
    TimedScope ts(tm, MOE_K_DW_SUM, s);
    MOE_TRY(launch_perm_weights(d.dtype, cb->topk_w, cb->sorted_pair, d.N, sv.u_d, r, B.w_perm,
                                B.wu_d, s));
    ud_eff = B.wu_d;
    gb_da = B.gbw;
  }
  if (fuse_d) {  // dB_d = G^T u_d [H, r] and gb = s G B_d in one pass over G
    TimedScope ts(tm, MOE_K_LORA_WGRAD, s);
    SideOut so;
    so.bm = w.b_d;
    so.out = gb;
    so.part = B.vpart;
    if (cb) {
      so.roww = B.w_perm;
      so.out_w = B.gbw;
    }
    MOE_TRY(weight_grad(d, offsets, g, H, ud_eff, r, gr.db_d, s, split, &so, nullptr, g_lx));
  } else {  // gb = s G B_d      (B_d[e] is [H, r]: K = H rows, r contiguous)
    TimedScope ts(tm, MOE_K_LORA_SIDE, s);
    MOE_TRY(side_product(d, offsets, L, g_rows, H, w.b_d,
                         static_cast<int64_t>(H) * r, 0, gb, s));
    if (cb) MOE_TRY(scale_rows(d.dtype, gb, B.w_perm, d.N, r, B.gbw, s));
  }
  {  // dAct = G W_d + gb A_d ; dH = SwiGLU'(h) dAct
    GemmArgs a = base_args(d, offsets, L.big);
    a.a[0] = g_rows;
    a.b[0] = opnd(w.w_d, static_cast<int64_t>(H) * I, I, 0, true);   // [K=H][N=I]
    a.a[1] = opnd(gb, 0, r, 1, r % 8 == 0);
    a.b[1] = opnd(w.a_d, static_cast<int64_t>(r) * I, I, 0, true);   // [K=r][N=I]
    a.K[0] = H;
    a.K[1] = r;
    a.N = I;
    a.out = dh;
    a.ld_out = 2 * I;
    a.aux = sv.h;
    a.ld_aux = 2 * I;
    a.ntn = d.dtype != MOE_F32 ? ceil_div(I, 256) : ceil_div(I, 64);
    if (cb) {
      a.roww = B.w_perm;
      a.dwp = B.dwp;
      a.dwp_slots = d.dtype != MOE_F32 ? a.ntn * big_waves_n(a, L.big.bm) : a.ntn;
    }
    {
      TimedScope ts(tm, MOE_K_DOWN_BWD, s);
      if (d.dtype != MOE_F32)
        MOE_TRY((launch_big<GROUP_M, EPI_SWIGLU_BWD, false, true, false>(
                       gm_grid(d, L.big, a.ntn), a, s, L.big.bm)));
      else
        MOE_TRY(launch(gemm_f32<GROUP_M, EPI_SWIGLU_BWD, false>, gm_grid(d, L.big, a.ntn), a, s));
    }
    if (cb) {
      TimedScope ts(tm, MOE_K_DW_SUM, s);
      MOE_TRY(launch_dw_sum(B.dwp, a.dwp_slots, cb->inv_pos,
                            static_cast<int64_t>(cb->T) * cb->k, cb->d_topk_w, s));
    }
  }
  {  // dB_d = G^T u_d  [H, r] (unless fused above) ;  dA_d = gb^T act  [r, I]
    TimedScope ts(tm, MOE_K_LORA_WGRAD, s);
    if (!fuse_d)
      MOE_TRY(weight_grad(d, offsets, g, H, ud_eff, r, gr.db_d, s, split, nullptr, nullptr, g_lx));
    MOE_TRY(weight_grad(d, offsets, gb_da, r, sv.act, I, gr.da_d, s, split));
  }
  if (base) {  // full fine-tuning: dW_d = G^T act  [H, I]
    if (cb) {
      TimedScope ts(tm, MOE_K_ROW_SCALE, s);
      MOE_TRY(scale_rows(d.dtype, g, B.w_perm, d.N, H, const_cast<void*>(g), s));
    }
    TimedScope ts(tm, MOE_K_BASE_WGRAD, s);
    MOE_TRY(weight_grad(d, offsets, g, H, sv.act, I, base->dw_d, s, nullptr));
  }
  if (fuse_gu) {  // dB_gu = dH^T u_gu [2I, r] and dhb = s dH B_gu in one pass over dH
    TimedScope ts(tm, MOE_K_LORA_WGRAD, s);
    SideOut so;
    so.bm = w.b_gu;
    so.out = dhb;
    so.part = B.vpart;
    MOE_TRY(weight_grad(d, offsets, dh, 2 * I, sv.u_gu, r, gr.db_gu, s, split, &so));
  } else {  // dhb = s dH B_gu   (B_gu[e] is [2I, r])
    TimedScope ts(tm, MOE_K_LORA_SIDE, s);
    MOE_TRY(side_product(d, offsets, L, opnd(dh, 0, 2 * I, 1, true), 2 * I, w.b_gu,
                         static_cast<int64_t>(2) * I * r, 0, dhb, s));
  }
  {  // dX = dH W_gu + dhb A_gu
    GemmArgs a = base_args(d, offsets, L.big);
    a.a[0] = opnd(dh, 0, 2 * I, 1, true);
    a.b[0] = opnd(w.w_gu, static_cast<int64_t>(2) * I * H, H, 0, true);  // [K=2I][N=H]
    a.a[1] = opnd(dhb, 0, r, 1, r % 8 == 0);
    a.b[1] = opnd(w.a_gu, static_cast<int64_t>(r) * H, H, 0, true);      // [K=r][N=H]
    a.K[0] = 2 * I;
    a.K[1] = r;
    a.N = H;
    a.out = dx_perm;
    a.ld_out = H;
    TimedScope ts(tm, MOE_K_GATE_UP_BWD, s);
    if (d.dtype != MOE_F32) {
      a.ntn = ceil_div(H, 256);
      MOE_TRY((launch_big<GROUP_M, EPI_STORE, false, true, false>( gm_grid(d, L.big, a.ntn),
                     a, s, L.big.bm)));
    } else {
      a.ntn = ceil_div(H, 64);
      MOE_TRY(launch(gemm_f32<GROUP_M, EPI_STORE, false>, gm_grid(d, L.big, a.ntn), a, s));
    }
  }
  {  // dB_gu = dH^T u_gu  [2I, r] (unless fused above) ;  dA_gu = dhb^T X  [r, H]
    TimedScope ts(tm, MOE_K_LORA_WGRAD, s);
    if (!fuse_gu) MOE_TRY(weight_grad(d, offsets, dh, 2 * I, sv.u_gu, r, gr.db_gu, s, split));
    MOE_TRY(weight_grad(d, offsets, dhb, r, x.ptr, H, gr.da_gu, s, split, nullptr, &x));
  }
  if (base) {  // full fine-tuning: dW_gu = dH^T X  [2I, H]
    TimedScope ts(tm, MOE_K_BASE_WGRAD, s);
    MOE_TRY(weight_grad(d, offsets, dh, 2 * I, x.ptr, H, base->dw_gu, s, nullptr, nullptr, &x));
  }
  return hipSuccess;
}

size_t experts_fwd_lean_ws_bytes(const ExpertDims& d) {
  return align_up(experts_fwd_ws_bytes(d)) + lean_extra_bytes(d);
}

size_t experts_bwd_lean_ws_bytes(const ExpertDims& d) {
  return align_up(experts_bwd_ws_bytes(d)) + lean_extra_bytes(d);
}

hipError_t launch_experts_fwd_lean(const ExpertDims& d, const XRows& x,
                                   const int32_t* offsets, const moe_weights& w,
                                   const moe_saved& sv, void* ws, hipStream_t s,
                                   KernelTimer* tm) {
  const moe_saved full = lean_saved(d, sv, ws, experts_fwd_ws_bytes(d));
  return launch_experts_fwd(d, x, offsets, w, full, ws, s, tm);
}

hipError_t launch_experts_bwd_recompute(const ExpertDims& d, const void* g, const XRows& x,
                                        const int32_t* offsets, const moe_weights& w,
                                        const moe_saved& sv, void* dx_perm,
                                        const moe_lora_grads& gr, const moe_base_grads* base,
                                        void* ws, hipStream_t s, KernelTimer* tm,
                                        const CombineBwd* cb) {
  const moe_saved full = lean_saved(d, sv, ws, experts_bwd_ws_bytes(d));
  const WsLayout L = tile_ws(ws, d);
  MOE_TRY(build_tiles(L, offsets, d.E, s));
  MOE_TRY(launch_gate_up(d, L, x, offsets, w, sv.u_gu, full.h, full.act, s, tm));
  return launch_experts_bwd(d, g, x, offsets, w, full, dx_perm, gr, base, ws, s, tm, cb);
}

// ----------------------------------------------------------------- router projection
// logits = x W_r^T (float32 out) and its input gradient dx += d_logits W_r, as
// grouped GEMMs over a single group of all T rows (tile list built on the
// device from offsets {0, T}).
namespace {

__global__ void range_offsets_kernel(int32_t* off, int T) {
  if (threadIdx.x == 0) {
    off[0] = 0;
    off[1] = T;
  }
}

template <typename Elem>
__global__ __launch_bounds__(256) void cast_kernel(const float* __restrict__ src,
                                                   Elem* __restrict__ dst, int64_t n) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (i < n) dst[i] = from_f32<Elem>(src[i]);
}

// dst += src; with vec, each thread takes 16 bytes (both pointers 16-byte aligned).
template <typename Elem>
__global__ __launch_bounds__(256) void accumulate_kernel(const Elem* __restrict__ src,
                                                         Elem* __restrict__ dst, int64_t n,
                                                         bool vec) {
  constexpr int V = 16 / sizeof(Elem);
  const int64_t t = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (vec) {
    const int64_t i = t * V;
    if (i + V <= n) {
      Elem a[V], b[V];
      *reinterpret_cast<uint4*>(a) = *reinterpret_cast<const uint4*>(src + i);
      *reinterpret_cast<uint4*>(b) = *reinterpret_cast<const uint4*>(dst + i);
#pragma unroll
      for (int j = 0; j < V; ++j) b[j] = from_f32<Elem>(to_f32<Elem>(b[j]) + to_f32<Elem>(a[j]));
      *reinterpret_cast<uint4*>(dst + i) = *reinterpret_cast<const uint4*>(b);
    } else {
      for (int64_t j = i; j < n; ++j)
        dst[j] = from_f32<Elem>(to_f32<Elem>(dst[j]) + to_f32<Elem>(src[j]));
    }
  } else if (t < n) {
    dst[t] = from_f32<Elem>(to_f32<Elem>(dst[t]) + to_f32<Elem>(src[t]));
  }
}

struct RouterWs {
  int32_t* offsets;
  WsLayout L;
  bf16_t* dl16;  // d_logits in bf16 (backward, bf16 layers)
  size_t bytes;
};

RouterWs router_ws(void* ws, int T, int E, int dtype) {
  ExpertDims d{};
  d.N = T;
  d.E = 1;
  d.dtype = dtype;
  d.r = 8;  // tile heights as for a LoRA-friendly rank: 128-row small list
  RouterWs R;
  char* p = static_cast<char*>(ws);
  R.offsets = reinterpret_cast<int32_t*>(p);
  size_t off = kAlign;
  R.L = tile_ws(p ? p + off : nullptr, d);
  off += align_up(R.L.bytes);
  R.dl16 = reinterpret_cast<bf16_t*>(p ? p + off : nullptr);
  off += dtype != MOE_F32 ? align_up(static_cast<size_t>(T) * E * 2) : 0;
  R.bytes = off;
  return R;
}

GemmArgs router_args(const RouterWs& R, int dtype) {
  GemmArgs a{};
  a.dtype = dtype;
  a.a[1] = none();
  a.b[1] = none();
  a.E = 1;
  a.offsets = R.offsets;
  a.tiles = R.L.small.tiles;
  a.ntiles = R.L.small.ntiles;
  a.K[1] = 0;
  a.scale = 1.0f;
  return a;
}

}  // namespace

size_t router_ws_bytes(int T, int E, int dtype) { return router_ws(nullptr, T, E, dtype).bytes; }

hipError_t launch_router_fwd(const void* x, const void* w_r, int T, int H, int E, int dtype,
                             float* logits, void* ws, hipStream_t s, KernelTimer* tm) {
  const RouterWs R = router_ws(ws, T, E, dtype);
  TimedScope ts(tm, MOE_K_ROUTER_FWD, s);
  hipLaunchKernelGGL(range_offsets_kernel, dim3(1), dim3(64), 0, s, R.offsets, T);
  MOE_TRY(build_tiles(R.L, R.offsets, 1, s));
  GemmArgs a = router_args(R, dtype);
  a.a[0] = opnd(x, 0, H, 1, true);
  a.b[0] = opnd(w_r, 0, H, 1, true);
  a.K[0] = H;
  a.N = E;
  a.out = logits;
  a.ld_out = E;
  if (dtype != MOE_F32) {
    a.ntn = ceil_div(E, 64);
    return launch(GEMM16(a.dtype, 128, 64, 32, 64, 64, 3, 2, GROUP_M, EPI_STORE_F32, false, true, true, 0),
                  static_cast<int>(tile_cap(T, 1, R.L.small.bm)) * a.ntn, a, s);
  }
  a.ntn = ceil_div(E, 64);
  return launch(gemm_f32<GROUP_M, EPI_STORE, false>,
                static_cast<int>(tile_cap(T, 1, R.L.small.bm)) * a.ntn, a, s);
}

hipError_t launch_router_bwd(const float* d_logits, const void* w_r, int T, int H, int E,
                             int dtype, void* dx, void* ws, hipStream_t s, KernelTimer* tm) {
  const RouterWs R = router_ws(ws, T, E, dtype);
  TimedScope ts(tm, MOE_K_ROUTER_BWD, s);
  hipLaunchKernelGGL(range_offsets_kernel, dim3(1), dim3(64), 0, s, R.offsets, T);
  MOE_TRY(build_tiles(R.L, R.offsets, 1, s));
  GemmArgs a = router_args(R, dtype);
  a.K[0] = E;
  a.N = H;
  a.out = dx;
  a.ld_out = H;
  if (dtype != MOE_F32) {
    const int64_t n = static_cast<int64_t>(T) * E;
    const dim3 grid(static_cast<unsigned>((n + 255) / 256));
    if (dtype == MOE_F16)
      hipLaunchKernelGGL(cast_kernel<f16_t>, grid, dim3(256), 0, s, d_logits,
                         reinterpret_cast<f16_t*>(R.dl16), n);
    else
      hipLaunchKernelGGL(cast_kernel<bf16_t>, grid, dim3(256), 0, s, d_logits, R.dl16, n);
    a.a[0] = opnd(R.dl16, 0, E, 1, true);
    a.b[0] = opnd(w_r, 0, H, 0, true);  // [K = E][N = H]
    a.ntn = ceil_div(H, 256);
    return launch(GEMM16(a.dtype, 128, 256, 64, 128, 32, 3, 2, GROUP_M, EPI_ADD, false, true, false, 0),
                  static_cast<int>(tile_cap(T, 1, R.L.small.bm)) * a.ntn, a, s);
  }
  a.a[0] = opnd(d_logits, 0, E, 1, true);
  a.b[0] = opnd(w_r, 0, H, 0, true);
  a.ntn = ceil_div(H, 64);
  return launch(gemm_f32<GROUP_M, EPI_ADD, false>,
                static_cast<int>(tile_cap(T, 1, R.L.small.bm)) * a.ntn, a, s);
}

// ----------------------------------------------------------------- merged export
// W'[e] = W[e] + s B[e] A[e] for both stacked projections. 16-bit layers use
// merge_kernel below; float32 layers a grouped GEMM whose "tokens" are the
// output rows of each expert's weight (2I for gate_up, H for down; K = r) and
// whose epilogue adds the base weight read from aux.
namespace {

// One stacked projection, 16-bit layers: W [E][R][C], B [E][R][r],
// A [E][r][C]. One block of four waves per 64-row x 256-column tile of an
// expert's W (grid: x = row tile * ntc + column tile, y = expert); wave w
// takes columns 64w .. 64w+63. The pass is bound by streaming W in and W' out,
// so each wave first issues the rank-r operand loads (small, L2-resident),
// then all of its base-weight loads (8 rows x 64 columns per instruction,
// 16 bytes a lane), and only then waits for the operands: the base weight
// arrives while the product runs on MFMA (k = 16 per step, zero past r). The
// product goes through the wave's own LDS tile, 32 rows at a time, so each
// lane ends with 8 consecutive elements of a row: W' = W + s (B A) as one
// float32 sum, rounded once, stored in 16 bytes. VEC: C % 8 == 0 and W, W'
// 16-byte aligned; otherwise every W / W' element is accessed on its own. W'
// may be W itself: each element is read and written by the same lane.
constexpr int kMergeRows = 64, kMergeCols = 256, kMergeLd = 72;

template <bool F16, bool VEC, int KS>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(VEC ? (KS < 4 ? 4 : 2)
                                                                          : (KS < 2 ? 4 : 2))))
void merge_kernel(const bf16_t* W, const bf16_t* __restrict__ Bm,
                  const bf16_t* __restrict__ Am, bf16_t* out, int R, int C, int r, int ntc,
                  float scale, bool avec, bool bvec) {
  // row stride 72 floats: the two half-waves of a fragment store (rows i and
  // i + 4) fall on disjoint banks
  __shared__ float P[4][32][kMergeLd];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int rt = blockIdx.x / ntc, ct = blockIdx.x - rt * ntc;
  const int row0 = rt * kMergeRows;
  const int col0 = ct * kMergeCols + wave * 64;
  if (col0 >= C) return;  // wave-uniform; the kernel has no block barrier
  const int64_t e = blockIdx.y;
  const bf16_t* We = W + e * R * C;
  bf16_t* Oe = out + e * R * C;
  const uint16_t* Be = reinterpret_cast<const uint16_t*>(Bm) + e * R * r;
  const uint16_t* Ae = reinterpret_cast<const uint16_t*>(Am) + e * r * C;
  const int li = lane & 31, lk = (lane >> 5) * 8;

  // Rank-r operands of all k steps (KS of them cover r, zero past r). A-side
  // fragments are B's rows (the product's rows): 16-byte loads when bvec. The
  // B-side fragments need 8 consecutive k of one column of A ([r][C]), so the
  // wave's 64 columns of A are loaded by rows (16 bytes a lane when avec) and
  // written transposed into the wave's LDS tile, At[column][k], from which
  // each fragment is one 16-byte read. The same LDS later holds the product.
  const int ks_n = (r + 15) / 16;
  uint16_t (*At)[kMergeLd] = reinterpret_cast<uint16_t (*)[kMergeLd]>(P[wave]);
  u32x4 ach[2 * KS];
#pragma unroll
  for (int i = 0; i < 2 * KS; ++i) {  // chunk m: k = m / 8, columns 8 (m % 8) .. + 7
    const int m = i * 64 + lane, k = m >> 3, c = col0 + (m & 7) * 8;
    const uint16_t* src = Ae + static_cast<int64_t>(k) * C + c;
    u32x4 v = {0u, 0u, 0u, 0u};
    if (i < 2 * ks_n && k < r && c < C) {
      if (avec) {
        v = *reinterpret_cast<const u32x4*>(src);
      } else {
#pragma unroll
        for (int t = 0; t < 4; ++t) v[t] = src[2 * t] | (static_cast<uint32_t>(src[2 * t + 1]) << 16);
      }
    }
    ach[i] = v;
  }
  u32x4 fa[KS][2], fb[KS][2];
#pragma unroll
  for (int ks = 0; ks < KS; ++ks) {
#pragma unroll
    for (int f = 0; f < 2; ++f) {
      const int n = row0 + 32 * f + li, k0 = ks * 16 + lk;
      const uint16_t* src = Be + static_cast<int64_t>(n) * r + k0;
      u32x4 v = {0u, 0u, 0u, 0u};
      if (ks < ks_n && n < R) {
        if (bvec) {
          if (k0 < r) v = *reinterpret_cast<const u32x4*>(src);
        } else {
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            const uint32_t lo = k0 + 2 * t < r ? src[2 * t] : 0u;
            const uint32_t hi = k0 + 2 * t + 1 < r ? src[2 * t + 1] : 0u;
            v[t] = lo | (hi << 16);
          }
        }
      }
      fa[ks][f] = v;
    }
  }
  __builtin_amdgcn_sched_barrier(0);

  // base weight: load j covers rows 8j .. 8j+7 of the tile, lane -> row
  // 8j + lane/8, columns lc .. lc+7
  const int lr = lane >> 3, lc = col0 + (lane & 7) * 8;
  u32x4 wv[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int row = row0 + 8 * j + lr;
    const bf16_t* src = We + static_cast<int64_t>(row) * C + lc;
    if constexpr (VEC) {
      wv[j] = row < R && lc < C ? __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(src))
                                : u32x4{0u, 0u, 0u, 0u};
    } else {
      uint32_t v[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const uint32_t lo = row < R && lc + 2 * t < C ? src[2 * t] : 0u;
        const uint32_t hi = row < R && lc + 2 * t + 1 < C ? src[2 * t + 1] : 0u;
        v[t] = lo | (hi << 16);
      }
      wv[j] = u32x4{v[0], v[1], v[2], v[3]};
    }
  }
  __builtin_amdgcn_sched_barrier(0);

  // At: every chunk of k steps below ks_n is written (zeros past r)
#pragma unroll
  for (int i = 0; i < 2 * KS; ++i) {
    if (i < 2 * ks_n) {
      const int m = i * 64 + lane, k = m >> 3, cl = (m & 7) * 8;
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        At[cl + 2 * t][k] = static_cast<uint16_t>(ach[i][t] & 0xffffu);
        At[cl + 2 * t + 1][k] = static_cast<uint16_t>(ach[i][t] >> 16);
      }
    }
  }
  wave_lds_sync();
#pragma unroll
  for (int ks = 0; ks < KS; ++ks)
#pragma unroll
    for (int g = 0; g < 2; ++g)
      fb[ks][g] = ks < ks_n ? *reinterpret_cast<const u32x4*>(&At[32 * g + li][ks * 16 + lk])
                            : u32x4{0u, 0u, 0u, 0u};

  float (*Pw)[kMergeLd] = P[wave];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    f32x16 acc[2];
#pragma unroll
    for (int g = 0; g < 2; ++g)
#pragma unroll
      for (int q = 0; q < 16; ++q) acc[g][q] = 0.0f;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
      if (ks < ks_n)
#pragma unroll
        for (int g = 0; g < 2; ++g)
          acc[g] = mfma32<F16>(__builtin_bit_cast(bf16x8, fa[ks][h]),
                               __builtin_bit_cast(bf16x8, fb[ks][g]), acc[g]);
    wave_lds_sync();  // the At reads (h = 0) or the previous half's reads are done
    // acc[g] register q: product row 8(q/4) + 4(lane/32) + q%4 of this
    // half, column 32g + lane%32 of the wave's 64
#pragma unroll
    for (int g = 0; g < 2; ++g)
#pragma unroll
      for (int q = 0; q < 16; ++q)
        Pw[8 * (q >> 2) + 4 * (lane >> 5) + (q & 3)][32 * g + li] = scale * acc[g][q];
    wave_lds_sync();
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int rl = 8 * j + lr, row = row0 + 32 * h + rl;
      const f32x4 p0 = *reinterpret_cast<const f32x4*>(&Pw[rl][(lane & 7) * 8]);
      const f32x4 p1 = *reinterpret_cast<const f32x4*>(&Pw[rl][(lane & 7) * 8 + 4]);
      float v[8];
      unpack8<F16>(wv[4 * h + j], v);
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        v[t] += p0[t];
        v[4 + t] += p1[t];
      }
      if (row >= R) continue;
      bf16_t* dst = Oe + static_cast<int64_t>(row) * C + lc;
      if constexpr (VEC) {
        if (lc < C) store8<F16>(dst, v);
      } else {
#pragma unroll
        for (int t = 0; t < 8; ++t)
          if (lc + t < C) dst[t] = f32_to_h16<F16>(v[t]);
      }
    }
  }
}

__global__ void uniform_offsets_kernel(int32_t* off, int E, int rows) {
  for (int e = threadIdx.x; e <= E; e += blockDim.x) off[e] = e * rows;
}

struct MergeWs {
  int32_t* offsets;
  WsLayout L;
  size_t bytes;
};

MergeWs merge_ws(void* ws, const ExpertDims& d) {
  MergeWs M;
  char* p = static_cast<char*>(ws);
  M.offsets = reinterpret_cast<int32_t*>(p);
  size_t off = align_up(static_cast<size_t>(d.E + 1) * 4);
  M.L = tile_ws(p ? p + off : nullptr, d);
  M.bytes = off + align_up(M.L.bytes);
  return M;
}

// rows of one expert's output, dims of the workspace-sizing view
ExpertDims merge_dims(const ExpertDims& d, int rows) {
  ExpertDims m = d;
  m.N = d.E * rows;
  return m;
}

hipError_t merge_one(const ExpertDims& d, int rows, int cols, const void* w, const void* a,
                     const void* b, void* out, void* ws, hipStream_t s) {
  if (d.dtype != MOE_F32) {
    const int64_t ntc = ceil_div(cols, kMergeCols), nt = ceil_div(rows, kMergeRows) * ntc;
    if (nt > INT32_MAX || d.r > 64) return hipErrorInvalidValue;
    const bool vec = cols % 8 == 0 && aligned16(w) && aligned16(out);
    const bool f16 = d.dtype == MOE_F16;
    auto pick = [&](auto ks) {
      constexpr int KS = decltype(ks)::value;
      return f16 ? (vec ? merge_kernel<true, true, KS> : merge_kernel<true, false, KS>)
                 : (vec ? merge_kernel<false, true, KS> : merge_kernel<false, false, KS>);
    };
    auto kern = d.r <= 16   ? pick(std::integral_constant<int, 1>())
                : d.r <= 32 ? pick(std::integral_constant<int, 2>())
                            : pick(std::integral_constant<int, 4>());
    hipLaunchKernelGGL(kern, dim3(static_cast<unsigned>(nt), d.E), dim3(256), 0, s,
                       static_cast<const bf16_t*>(w), static_cast<const bf16_t*>(b),
                       static_cast<const bf16_t*>(a), static_cast<bf16_t*>(out), rows, cols, d.r,
                       static_cast<int>(ntc), d.scale, aligned16(a),
                       d.r % 8 == 0 && aligned16(b));
    return hipGetLastError();
  }
  const ExpertDims m = merge_dims(d, rows);
  const MergeWs M = merge_ws(ws, m);
  hipLaunchKernelGGL(uniform_offsets_kernel, dim3(1), dim3(256), 0, s, M.offsets, d.E, rows);
  MOE_TRY(build_tiles(M.L, M.offsets, d.E, s));
  GemmArgs g{};
  g.dtype = d.dtype;
  g.a[1] = none();
  g.b[1] = none();
  g.E = d.E;
  g.offsets = M.offsets;
  g.tiles = M.L.small.tiles;
  g.ntiles = M.L.small.ntiles;
  g.a[0] = opnd(b, 0, d.r, 1, d.r % 8 == 0);                               // B rows: [rows, r]
  g.b[0] = opnd(a, static_cast<int64_t>(d.r) * cols, cols, 0, true);      // A[e]: [K = r][N = cols]
  g.K[0] = d.r;
  g.K[1] = 0;
  g.N = cols;
  g.out = out;
  g.ld_out = cols;
  g.aux = w;
  g.ld_aux = cols;
  g.scale = d.scale;
  const int grid_m = static_cast<int>(tile_cap(m.N, d.E, M.L.small.bm));
  g.ntn = ceil_div(cols, 64);
  return launch(gemm_f32<GROUP_M, EPI_ADD, false>, grid_m * g.ntn, g, s);
}

}  // namespace

size_t merge_ws_bytes(const ExpertDims& d) {
  return std::max(merge_ws(nullptr, merge_dims(d, 2 * d.I)).bytes,
                  merge_ws(nullptr, merge_dims(d, d.H)).bytes);
}

hipError_t launch_merge(const ExpertDims& d, const moe_weights& w, void* w_gu_out, void* w_d_out,
                        void* ws, hipStream_t s, KernelTimer* tm) {
  TimedScope ts(tm, MOE_K_MERGE, s);
  if (w_gu_out) MOE_TRY(merge_one(d, 2 * d.I, d.H, w.w_gu, w.a_gu, w.b_gu, w_gu_out, ws, s));
  if (w_d_out) MOE_TRY(merge_one(d, d.H, d.I, w.w_d, w.a_d, w.b_d, w_d_out, ws, s));
  return hipSuccess;
}

hipError_t launch_accumulate(int dtype, int64_t n, const void* src, void* dst, hipStream_t s,
                             KernelTimer* tm) {
  if (n <= 0) return hipSuccess;
  TimedScope ts(tm, MOE_K_ACCUMULATE, s);
  const dim3 grid(static_cast<unsigned>((n + 255) / 256));
  const bool vec = ((reinterpret_cast<uintptr_t>(src) | reinterpret_cast<uintptr_t>(dst)) & 15) == 0;
  auto go = [&](auto tag) {
    using Elem = decltype(tag);
    constexpr int V = 16 / sizeof(Elem);
    const int64_t threads = vec ? (n + V - 1) / V : n;
    hipLaunchKernelGGL(accumulate_kernel<Elem>, dim3(static_cast<unsigned>((threads + 255) / 256)),
                       dim3(256), 0, s, static_cast<const Elem*>(src), static_cast<Elem*>(dst), n,
                       vec);
  };
  if (dtype == MOE_BF16) go(bf16_t{});
  else if (dtype == MOE_F16) go(f16_t{});
  else go(float{});
  return hipGetLastError();
}

}  // namespace moe
