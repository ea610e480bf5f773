// gemm.hip -- bf16 MFMA GEMMs of the QLoRA linear layer.
//
// One kernel template computes  C[I][J] = sum_c Aop(i, c) * Bop(j, c)  with
// v_mfma_f32_32x32x16_bf16 (fp32 accumulation) on 256-thread workgroups.
// Operand tiles are staged through LDS as [row][64 + 8] bf16 (contraction
// contiguous, so every MFMA fragment is one 16-byte LDS read).  The operand
// producers:
//   CC    bf16 source [row][c] (contraction contiguous): 16-byte copies
//   T     bf16 source [c][row]: 16-byte loads along the row, written to LDS
//         transposed (a wave covers 64 consecutive c, so the 2-byte writes of
//         one instruction are contiguous)
//   NF4CC packed NF4 weight W[n][k] with c = k: each thread dequantizes half a
//         block (32 codes) into bf16 exactly as nf4_dequantize does
//   NF4T  packed NF4 weight W[n][k] with c = n (the backward's dX): 32 codes
//         of one row, written to LDS transposed
// Ultralytics glossary "QLoRA", "How QLoRA works": the forward dequantizes
// NF4 to bf16 right before the matrix product and adds the LoRA path; the
// backward computes gradients through the dequantized weights and only for
// the two LoRA matrices.
//
// The LoRA terms enter as a prologue of the main GEMMs: the accumulators
// start as s * (T B^T) (forward) or s * (U A) (dX), then the base product is
// accumulated on top.  The rank-r side products (T, U, dA, dB) run as split
// contractions writing fp32 partials that a second kernel sums in a fixed
// order (deterministic) and rounds to bf16.
//
// Many adapters on one weight (multi.hip sorts the tokens by adapter and
// writes the order): the same products with the rows taken through the sorted
// order, in three forms (enum Multi).
//   ROWS  T and U: a workgroup's rows are a piece of one adapter's run, so its
//         tile meets that adapter's factor alone
//   SEGS  dA and dB: the contraction runs over a piece of one adapter's tokens,
//         at most `step` of them, so that one adapter with most of the
//         tokens does not hold a few workgroups up (8 adapters of 300 to 2000
//         tokens, N = 11008, r = 64: dB 125 us with a whole adapter a
//         workgroup, 95 in pieces).  An adapter of one piece is finished there;
//         the others' fp32 sums are added up in order afterwards.  Both run
//         in one launch: on small batches each alone leaves most of the chip
//         idle and pays a launch of its own
//         (8192 tokens of 8 adapters, N = 11008, K = 4096, r = 64: U 43 us and dB
//         with dA 67 us, 4.2 and 3.7 TB/s of activations read, 128 and 256 bytes
//         a row and stage from wherever the row lies)
//   MAIN  the fused GEMMs: a tile's rows may belong to several adapters; each
//         run's LoRA term is summed apart and added to that run's rows only,
//         so nothing of one adapter (not even a NaN) reaches another's rows
#include <algorithm>
#include <type_traits>

#include "common.h"
#include "device.h"

namespace qln {

constexpr int BK = 64;
constexpr int PITCH = BK + 8;  // bf16 elements per LDS row (144 bytes)
constexpr int NTHREADS = 256;

enum { SRC_CC = 0, SRC_T = 1, SRC_NF4CC = 2, SRC_NF4T = 3, SRC_TF32S = 4,
       SRC_TR = 5,      // A from a [C][I] matrix, kept [c][i] in LDS, read with transposing loads
       SRC_TF32SR = 6   // B from an fp32 [C][J] matrix as hi + lo bf16, kept [c][j], transposing loads
};
enum { LORA_NONE = 0, LORA_FWD = 1, LORA_DX = 2 };
enum { OUT_BF16 = 0, OUT_F32 = 1 };
enum Multi { MULTI_NONE = 0, MULTI_ROWS = 1, MULTI_SEGS = 2, MULTI_MAIN = 3 };

// One of the two products of a SEGS launch: dB (operand dY, tiles of N) or dA
// (operand X, tiles of K, stored transposed).
struct SegsHalf {
  const u16* a; int64_t lda;
  const float* b;        // T or U
  int64_t I;
  int64_t step, nt;      // longest piece of an adapter's tokens, steps of all tokens
  float* part; u16* out; // sums of pieces, and the result
  bool trans;
  int tiles;             // workgroups of blockIdx.x
};

struct GemmArgs {
  // A operand (bf16), rows i
  const u16* a; int64_t lda; bool a_vec;
  // B operand: bf16 source, fp32 source (SRC_TF32S) or NF4 weight, rows j
  const void* b; int64_t ldb; bool b_vec;
  NF4View w;
  int64_t I, J, C;
  int64_t c_per_split;
  // LoRA prologue: accumulators start at s * sum_{c < r} la(i, c) * lb(j, c);
  // la is fp32 [I][r] (T or U), rounded to bf16 on its way to LDS
  const float* la; const u16* lb; int r; float s; bool la_vec; bool lb_vec;
  // output
  void* out; int64_t ldo; float out_scale;
  // many adapters: the sorted order, and elements from one adapter's factor
  // (B operand of ROWS, lb of MAIN) or output (SEGS) to the next
  MultiOrder mo; int64_t ad_stride;
  SegsHalf seg[2];       // SEGS: dB and dA
  int64_t M;             // and all tokens
};

__device__ __forceinline__ float nf4_level(const float* sL, uint32_t c) { return sL[c]; }

// ---------------------------------------------------------------------------
// producers: global -> registers (load) and registers -> LDS (store)
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint4 load8_guarded(const u16* src, int64_t row, int64_t rows,
                                               int64_t ld, int64_t c, int64_t C, bool vec) {
  if (row < rows && c + 8 <= C && vec)
    return *reinterpret_cast<const uint4*>(src + row * ld + c);
  uint32_t w[4] = {0, 0, 0, 0};
  if (row < rows) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (c + e < C) w[e >> 1] |= (uint32_t)src[row * ld + c + e] << (16 * (e & 1));
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Many adapters: a stage's loads stand in one block and nothing reads them
// before the next stage's LDS stores, so all of them are in flight while this
// stage multiplies (guarded one by one, with zeros selected beside each load,
// a stage waited for nine loads in turn).  Addresses are
// clamped into the matrix; what lies outside in an output's row or column is
// not stored, and what lies past the contraction's end is zeroed in
// registers (keep) before the last stage's LDS store.

// Tile of R rows x 64 contraction from a [rows][C] matrix (leading dim ld).
template <int R>
struct ProdCC {
  static constexpr int NV = R / 32;
  uint4 v[NV];
  __device__ void load(const u16* src, int64_t ld, int64_t rows, int64_t C, int64_t r0,
                       int64_t c0, bool vec, int tid) {
#pragma unroll
    for (int q = 0; q < NV; ++q)
      v[q] = load8_guarded(src, r0 + tid / 8 + 32 * q, rows, ld, c0 + (tid % 8) * 8, C, vec);
  }
  // rows clamped, C a multiple of 64, 16-byte aligned rows
  __device__ void load_clamped(const u16* src, int64_t ld, int64_t rows, int64_t c0, int tid) {
#pragma unroll
    for (int q = 0; q < NV; ++q) {
      const int64_t row = tid / 8 + 32 * q;
      v[q] = load16(src + (row < rows ? row : 0) * ld + c0 + (tid % 8) * 8);
    }
  }
  __device__ void store(u16* S, int tid) const {
#pragma unroll
    for (int q = 0; q < NV; ++q)
      *reinterpret_cast<uint4*>(S + (tid / 8 + 32 * q) * PITCH + (tid % 8) * 8) = v[q];
  }
};

// The same tile with its rows taken through the sorted order: position
// p = p0 + local row is matrix row perm[p] (from p1 on the last one again),
// rows of ld elements, 16-byte aligned, zeros from C to the next multiple of 8.
template <int R>
struct ProdCCRows {
  static constexpr int NV = R / 32;
  uint4 v[NV];
  int32_t row[NV];
  __device__ void init(const int32_t* perm, int64_t p0, int64_t p1, int tid) {
#pragma unroll
    for (int q = 0; q < NV; ++q) {
      row[q] = perm[min(p0 + tid / 8 + 32 * q, p1 - 1)];
    }
  }
  __device__ void load(const u16* src, int64_t ld, int64_t C, int64_t c0, int tid) {
    const int64_t c = c0 + (tid % 8) * 8;
#pragma unroll
    for (int q = 0; q < NV; ++q)
      v[q] = load16(src + row[q] * ld + (c < C ? c : 0));
  }
  __device__ void keep(int64_t n, int tid) {   // the stage's first n contraction positions
#pragma unroll
    for (int q = 0; q < NV; ++q)
      if ((tid % 8) * 8 >= n) v[q] = make_uint4(0, 0, 0, 0);
  }
  __device__ void store(u16* S, int tid) const {
#pragma unroll
    for (int q = 0; q < NV; ++q)
      *reinterpret_cast<uint4*>(S + (tid / 8 + 32 * q) * PITCH + (tid % 8) * 8) = v[q];
  }
};

// Tile of R rows x 64 contraction from a [C][cols] matrix (row index along
// the contiguous dimension): LDS row i receives column i0 + i.
template <int R>
struct ProdT {
  static constexpr int NV = R / 32;
  uint4 v[NV];
  __device__ void load(const u16* src, int64_t ld, int64_t C, int64_t cols, int64_t i0,
                       int64_t c0, bool vec, int tid) {
    const int lane = tid & 63, wv = tid >> 6;
#pragma unroll
    for (int q = 0; q < NV; ++q)
      v[q] = load8_guarded(src, c0 + lane, C, ld, i0 + (wv + 4 * q) * 8, cols, vec);
  }
  // from column 0, rows of ld = cols elements at any boundary: a row's last 8
  // may reach into the next (columns that are not stored), the matrix's last
  // 8 are gathered
  template <bool VEC>
  __device__ void load_clamped(const u16* src, int64_t C, int64_t cols, int64_t c0, int tid) {
    const int lane = tid & 63, wv = tid >> 6;
    const u16* row = src + min(c0 + lane, C - 1) * cols;
    if constexpr (VEC) {
#pragma unroll
      for (int q = 0; q < NV; ++q) {
        const int64_t i = (wv + 4 * q) * 8;
        v[q] = load16(row + (i < cols ? i : 0));
      }
    } else {
#pragma unroll
      for (int q = 0; q < NV; ++q) {
        const int64_t i = (wv + 4 * q) * 8;
        const u16* at = row + (i < cols ? i : 0);
        if (at + 8 <= src + C * cols) {
          v[q] = load16_any(at);
        } else {
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const uint32_t h = *(at + e < src + C * cols ? at + e : src);
            w[e >> 1] = e & 1 ? w[e >> 1] | (h << 16) : h;
          }
          v[q] = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
    }
  }
  __device__ void keep(int64_t n, int tid) {   // the stage's first n contraction positions
#pragma unroll
    for (int q = 0; q < NV; ++q)
      if ((tid & 63) >= n) v[q] = make_uint4(0, 0, 0, 0);
  }
  __device__ void store(u16* S, int tid) const {
    const int lane = tid & 63, wv = tid >> 6;
#pragma unroll
    for (int q = 0; q < NV; ++q) {
      const int iseg = (wv + 4 * q) * 8;
      const uint32_t w[4] = {v[q].x, v[q].y, v[q].z, v[q].w};
#pragma unroll
      for (int e = 0; e < 8; ++e)
        S[(iseg + e) * PITCH + lane] = (u16)(w[e >> 1] >> (16 * (e & 1)));
    }
  }
};

// Tiles of a matrix whose contiguous dimension is the output index (dY or X
// for dB and dA): loaded with whole 256-byte row segments (16 lanes per
// contraction row) and kept in LDS as [64 c][R + 8] rows, so both the global
// loads and the 16-byte LDS stores are contiguous; the MFMA fragments come out
// with the transposing LDS read (ds_read_b64_tr_b16).
template <int R>
constexpr int tr_pitch() { return R + 8; }

typedef __attribute__((address_space(3))) short lds_short_g;
typedef short s16x4_g __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4_g lds_s16x4_g;

// MFMA operand fragment of column block cb (32 columns) at contraction step ks
// from a [c][cols] bf16 tile: lane l receives 8 contraction values of column
// cb*32 + l%32 (within each 16-lane group, lane i gets element i%4 of the rows
// addressed by lanes 4j + i/4).
__device__ __forceinline__ bf16x8_t read_tr(const u16* S, int pitch, int col0, int ks, int lane) {
  const int L = lane & 15;
  const int col = col0 + 16 * ((lane >> 4) & 1) + 4 * (L & 3);
  const int row = ks * 16 + 8 * (lane >> 5) + (L >> 2);
  const lds_short_g* base = (const lds_short_g*)S;
  const s16x4_g lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_g*)(base + row * pitch + col));
  const s16x4_g hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_g*)(base + (row + 4) * pitch + col));
  typedef short s16x8_t __attribute__((ext_vector_type(8)));
  const s16x8_t v = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
  return __builtin_bit_cast(bf16x8_t, v);
}

// bf16 [C][cols] source, R = 128 output columns: thread t loads row
// c0 + t/16 + 16q (q < 4), columns i0 + 8 (t % 16) .. +8
template <int R>
struct ProdTR {
  static_assert(R == 128, "16 lanes x 8 columns per row");
  uint4 v[4];
  __device__ void load(const u16* src, int64_t ld, int64_t C, int64_t cols, int64_t i0,
                       int64_t c0, bool vec, int tid) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      v[q] = load8_guarded(src, c0 + tid / 16 + 16 * q, C, ld, i0 + (tid % 16) * 8, cols, vec);
  }
  // contraction positions taken through the sorted order: rows[q] is the matrix
  // row of position c0 + tid/16 + 16q (16-byte aligned rows, ld a multiple of 8)
  __device__ void load_rows(const u16* src, int64_t ld, int64_t cols, int64_t i0, const int32_t (&rows)[4], int tid) {
    const int64_t i = i0 + (tid % 16) * 8;
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] = load16(src + rows[q] * ld + (i < cols ? i : 0));
  }
  __device__ void keep(int64_t n, int tid) {   // the stage's first n contraction positions
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (tid / 16 + 16 * q >= n) v[q] = make_uint4(0, 0, 0, 0);
  }
  __device__ void store(u16* S, int tid) const {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      *reinterpret_cast<uint4*>(S + (tid / 16 + 16 * q) * tr_pitch<R>() + (tid % 16) * 8) = v[q];
  }
};

// fp32 [C][cols] source, R (32, 64 or 128) output columns, split into hi =
// bf16(x) and lo = bf16(x - hi): thread t loads row c0 + t/16 + 16q (q < 4),
// R/16 consecutive columns
template <int R>
struct ProdTF32SR {
  static constexpr int E = R / 16;
  float x[4][E];
  __device__ void load(const float* src, int64_t ld, int64_t C, int64_t cols, int64_t j0,
                       int64_t c0, bool vec, int tid) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int64_t c = c0 + tid / 16 + 16 * q, j = j0 + (tid % 16) * E;
      if (vec && c < C && j + E <= cols) {
#pragma unroll
        for (int e = 0; e < E; e += 2) {
          const float2 f = *reinterpret_cast<const float2*>(src + c * ld + j + e);
          x[q][e] = f.x;
          x[q][e + 1] = f.y;
        }
      } else {
#pragma unroll
        for (int e = 0; e < E; ++e) x[q][e] = (c < C && j + e < cols) ? src[c * ld + j + e] : 0.0f;
      }
    }
  }
  // rows through the sorted order, as ProdTR::load_rows (VEC: cols a multiple
  // of 4, so that two or four lie inside or outside)
  template <bool VEC>
  __device__ void load_rows(const float* src, int64_t ld, int64_t cols, const int32_t (&rows)[4], int tid) {
    const int64_t j = (tid % 16) * E;
    if constexpr (VEC) {
      constexpr int W = E < 4 ? E : 4;
      typedef float wide_t __attribute__((ext_vector_type(W)));
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int e = 0; e < E; e += W) {
          const wide_t f = *reinterpret_cast<const wide_t*>(src + rows[q] * ld + (j + e < cols ? j + e : 0));
#pragma unroll
          for (int k = 0; k < W; ++k) x[q][e + k] = f[k];
        }
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int e = 0; e < E; ++e) x[q][e] = src[rows[q] * ld + (j + e < cols ? j + e : 0)];
    }
  }
  __device__ void keep(int64_t n, int tid) {   // the stage's first n contraction positions
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (tid / 16 + 16 * q >= n) x[q][e] = 0.0f;
  }
  __device__ void store(u16* Shi, u16* Slo, int tid) const {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      uint32_t hi[E / 2], lo[E / 2];
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        const float h0 = bf16_to_f32(f32_to_bf16(x[q][e])), h1 = bf16_to_f32(f32_to_bf16(x[q][e + 1]));
        hi[e / 2] = pack_bf16x2(h0, h1);
        lo[e / 2] = pack_bf16x2(x[q][e] - h0, x[q][e + 1] - h1);
      }
      const int off = (tid / 16 + 16 * q) * tr_pitch<R>() + (tid % 16) * E;
#pragma unroll
      for (int e = 0; e < E / 2; ++e) {
        *reinterpret_cast<uint32_t*>(Shi + off + 2 * e) = hi[e];
        *reinterpret_cast<uint32_t*>(Slo + off + 2 * e) = lo[e];
      }
    }
  }
};

// fp32 tile of R rows x 64 contraction from a [rows][C] fp32 matrix, rounded
// to bf16 (RNE) on the way to LDS.
template <int R>
struct ProdCCF32 {
  static constexpr int NV = R / 32;
  uint4 v[NV];
  __device__ void load(const float* src, int64_t ld, int64_t rows, int64_t C, int64_t r0,
                       int64_t c0, bool vec, int tid) {
#pragma unroll
    for (int q = 0; q < NV; ++q) {
      const int64_t row = r0 + tid / 8 + 32 * q, c = c0 + (tid % 8) * 8;
      float x[8];
      if (row < rows && c + 8 <= C && vec) {
        const float4 a = *reinterpret_cast<const float4*>(src + row * ld + c);
        const float4 b = *reinterpret_cast<const float4*>(src + row * ld + c + 4);
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = (row < rows && c + e < C) ? src[row * ld + c + e] : 0.0f;
      }
      v[q] = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                        pack_bf16x2(x[6], x[7]));
    }
  }
  __device__ void store(u16* S, int tid) const {
#pragma unroll
    for (int q = 0; q < NV; ++q)
      *reinterpret_cast<uint4*>(S + (tid / 8 + 32 * q) * PITCH + (tid % 8) * 8) = v[q];
  }
};

// fp32 tile of R rows x 64 contraction from a [C][cols] fp32 matrix, split
// into hi = bf16(x) and lo = bf16(x - hi): the sum of the two MFMA products
// sees x to about 2^-17 relative precision.
template <int R>
struct ProdTF32S {
  static constexpr int NV = R / 32;
  float x[NV][8];
  __device__ void load(const float* src, int64_t ld, int64_t C, int64_t cols, int64_t i0,
                       int64_t c0, bool vec, int tid) {
    const int lane = tid & 63, wv = tid >> 6;
    const int64_t c = c0 + lane;
#pragma unroll
    for (int q = 0; q < NV; ++q) {
      const int64_t i = i0 + (wv + 4 * q) * 8;
      if (c < C && i + 8 <= cols && vec) {
        const float4 a = *reinterpret_cast<const float4*>(src + c * ld + i);
        const float4 b = *reinterpret_cast<const float4*>(src + c * ld + i + 4);
        x[q][0] = a.x; x[q][1] = a.y; x[q][2] = a.z; x[q][3] = a.w;
        x[q][4] = b.x; x[q][5] = b.y; x[q][6] = b.z; x[q][7] = b.w;
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[q][e] = (c < C && i + e < cols) ? src[c * ld + i + e] : 0.0f;
      }
    }
  }
  __device__ void store(u16* Shi, u16* Slo, int tid) const {
    const int lane = tid & 63, wv = tid >> 6;
#pragma unroll
    for (int q = 0; q < NV; ++q) {
      const int iseg = (wv + 4 * q) * 8;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const u16 hi = f32_to_bf16(x[q][e]);
        const u16 lo = f32_to_bf16(x[q][e] - bf16_to_f32(hi));
        Shi[(iseg + e) * PITCH + lane] = hi;
        Slo[(iseg + e) * PITCH + lane] = lo;
      }
    }
  }
};

// dequantize 32 packed codes (16 bytes) with block scale sc into 16 bf16 pairs
__device__ __forceinline__ void dequant32(const uint4& c, float sc, const float* sL,
                                          uint32_t o[16]) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const uint32_t byte = (w[i >> 2] >> (8 * (i & 3))) & 0xFFu;
    o[i] = pack_bf16x2(nf4_level(sL, byte & 15u) * sc, nf4_level(sL, byte >> 4) * sc);
  }
}

// restored block scale: fl32(E4M3(q) * d), or the stored fp32 scale
__device__ __forceinline__ float block_scale(const NF4View& w, int64_t blk) {
  return w.fp32_scale ? w.dscale[blk]
                      : (w.u8_scale ? (float)w.qscale[blk] : e4m3_decode(w.qscale[blk])) * w.dscale[blk >> 8];
}

// NF4 weight, rows j = n (128 of them), contraction c = k (one 64-block):
// two threads per row, 32 codes each.
struct ProdNF4CC {
  uint4 v;
  float sc;
  __device__ void load(const NF4View& w, int64_t n0, int64_t k0, int tid) {
    const int64_t n = n0 + tid / 2;
    const int half = tid & 1;
    if (n < w.N) {
      v = *reinterpret_cast<const uint4*>(w.codes + n * (w.K / 2) + k0 / 2 + half * 16);
      sc = block_scale(w, n * (w.K / 64) + k0 / 64);
    } else {
      v = make_uint4(0, 0, 0, 0);
      sc = 0.0f;
    }
  }
  __device__ void store(u16* S, const float* sL, int tid) const {
    uint32_t o[16];
    dequant32(v, sc, sL, o);
    u16* dst = S + (tid / 2) * PITCH + (tid & 1) * 32;
#pragma unroll
    for (int q = 0; q < 4; ++q)
      *reinterpret_cast<uint4*>(dst + 8 * q) = make_uint4(o[4 * q], o[4 * q + 1], o[4 * q + 2],
                                                          o[4 * q + 3]);
  }
};

// NF4 weight, rows j = k (128 columns of W), contraction c = n (64 rows of W):
// thread (lane, wave) takes 32 codes of row c0 + lane at columns
// j0 + 32*wave .. +32 and writes them to LDS transposed.
struct ProdNF4T {
  uint4 v;
  float sc;
  __device__ void load(const NF4View& w, int64_t j0, int64_t c0, int tid) {
    const int lane = tid & 63, wv = tid >> 6;
    const int64_t n = c0 + lane;
    const int64_t k = j0 + 32 * wv;
    if (n < w.N && k < w.K) {
      v = *reinterpret_cast<const uint4*>(w.codes + n * (w.K / 2) + k / 2);
      sc = block_scale(w, n * (w.K / 64) + k / 64);
    } else {
      v = make_uint4(0, 0, 0, 0);
      sc = 0.0f;
    }
  }
  __device__ void store(u16* S, const float* sL, int tid) const {
    const int lane = tid & 63, wv = tid >> 6;
    uint32_t o[16];
    dequant32(v, sc, sL, o);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      S[(32 * wv + 2 * i) * PITCH + lane] = (u16)(o[i] & 0xFFFFu);
      S[(32 * wv + 2 * i + 1) * PITCH + lane] = (u16)(o[i] >> 16);
    }
  }
};

// ---------------------------------------------------------------------------
// the kernel
// ---------------------------------------------------------------------------
template <int BM, int BN, int WM, int WN, int ASRC, int BSRC, int LORA, int OUT, bool STORE_T,
          int MULTI = MULTI_NONE, bool BVEC = true>
__global__ __launch_bounds__(NTHREADS) void k_gemm(GemmArgs p) {
  // this workgroup's product of a SEGS launch, field by field (a struct chosen
  // as a whole went through scratch memory)
  const bool seg2 = MULTI == MULTI_SEGS && (int)blockIdx.x >= p.seg[0].tiles;
  const SegsHalf &s0 = p.seg[0], &s1 = p.seg[1];
  struct {
    const u16* a; int64_t lda; const float* b; int64_t I, step, nt; float* part; u16* out; bool trans;
  } const sg = {seg2 ? s1.a : s0.a, seg2 ? s1.lda : s0.lda, seg2 ? s1.b : s0.b,
                seg2 ? s1.I : s0.I, seg2 ? s1.step : s0.step, seg2 ? s1.nt : s0.nt, seg2 ? s1.part : s0.part,
                seg2 ? s1.out : s0.out, seg2 ? s1.trans : s0.trans};
  static_assert(WM * WN == 4, "four waves");
  constexpr int TM = BM / WM / 32, TN = BN / WN / 32;
  constexpr int SA_E = ASRC == SRC_TR ? BK * (BM + 8) : BM * PITCH;
  constexpr int SB_E = BSRC == SRC_TF32SR ? BK * (BN + 8) : BN * PITCH;
  __shared__ __attribute__((aligned(16))) u16 sA[SA_E];
  __shared__ __attribute__((aligned(16))) u16 sB[SB_E];
  constexpr bool SPLIT = (BSRC == SRC_TF32S || BSRC == SRC_TF32SR);
  __shared__ __attribute__((aligned(16))) u16 sB2[SPLIT ? SB_E : 8];
  __shared__ float sL[16];

  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = wave / WN, wn = wave % WN;
  int64_t i0 = (int64_t)blockIdx.x * BM;
  if (seg2) i0 -= (int64_t)s0.tiles * BM;
  int64_t i1 = p.I;   // end of the tile's rows (many adapters: positions)
  const int64_t j0 = MULTI == MULTI_SEGS ? 0 : (int64_t)blockIdx.y * BN;
  int64_t cs0 = (int64_t)blockIdx.z * p.c_per_split;
  int64_t cs1 = min(p.C, cs0 + p.c_per_split);
  int ad = 0;         // the workgroup's adapter (ROWS, SEGS)
  if constexpr (MULTI == MULTI_ROWS) {
    if (!multi_piece(p.mo, blockIdx.x, p.I, BM, &ad, &i0, &i1)) return;
    if (ad == p.mo.count) cs1 = cs0;   // rows without an adapter: zeros
  } else if constexpr (MULTI == MULTI_SEGS) {
    if (blockIdx.y >= sg.nt + p.mo.count) return;     // (the other product has more steps)
    if (!multi_piece(p.mo, blockIdx.y, p.M, sg.step, &ad, &cs0, &cs1)) {
      ad = (int)(blockIdx.y - sg.nt);
      if (p.mo.seg[ad] != p.mo.seg[ad + 1]) return;   // counted among the multiples of the step
      cs0 = cs1 = p.mo.seg[ad];                       // no tokens: zeros
    }
    if (ad == p.mo.count) return;                     // tokens without an adapter
  } else if constexpr (MULTI == MULTI_MAIN) {
    i1 = min(p.I, i0 + BM);
  }

  if (tid < 16) sL[tid] = p.w.lv[tid];   // the weight's codebook (unused without a weight)

  f32x16_t acc[TM][TN];
#pragma unroll
  for (int a = 0; a < TM; ++a)
#pragma unroll
    for (int b = 0; b < TN; ++b)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[a][b][v] = 0.0f;

  auto mma_tile = [&]() {
#pragma unroll
    for (int ks = 0; ks < BK / 16; ++ks) {
      bf16x8_t fa[TM], fb[TN];
#pragma unroll
      for (int a = 0; a < TM; ++a) {
        if constexpr (ASRC == SRC_TR)
          fa[a] = read_tr(sA, BM + 8, wm * (BM / WM) + a * 32, ks, lane);
        else
          fa[a] = *reinterpret_cast<const bf16x8_t*>(
              sA + (wm * (BM / WM) + a * 32 + (lane & 31)) * PITCH + ks * 16 + (lane >> 5) * 8);
      }
#pragma unroll
      for (int b = 0; b < TN; ++b) {
        if constexpr (BSRC == SRC_TF32SR)
          fb[b] = read_tr(sB, BN + 8, wn * (BN / WN) + b * 32, ks, lane);
        else
          fb[b] = *reinterpret_cast<const bf16x8_t*>(
              sB + (wn * (BN / WN) + b * 32 + (lane & 31)) * PITCH + ks * 16 + (lane >> 5) * 8);
      }
#pragma unroll
      for (int a = 0; a < TM; ++a)
#pragma unroll
        for (int b = 0; b < TN; ++b)
          acc[a][b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa[a], fb[b], acc[a][b], 0, 0, 0);
      if constexpr (SPLIT) {
#pragma unroll
        for (int b = 0; b < TN; ++b) {
          if constexpr (BSRC == SRC_TF32SR)
            fb[b] = read_tr(sB2, BN + 8, wn * (BN / WN) + b * 32, ks, lane);
          else
            fb[b] = *reinterpret_cast<const bf16x8_t*>(
                sB2 + (wn * (BN / WN) + b * 32 + (lane & 31)) * PITCH + ks * 16 + (lane >> 5) * 8);
        }
#pragma unroll
        for (int a = 0; a < TM; ++a)
#pragma unroll
          for (int b = 0; b < TN; ++b)
            acc[a][b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa[a], fb[b], acc[a][b], 0, 0, 0);
      }
    }
  };

  // ---- LoRA prologue, many adapters: run by run of the tile's rows ----
  if constexpr (MULTI == MULTI_MAIN) {
    const int64_t v1 = min(i1, (int64_t)p.mo.seg[p.mo.count]);   // rows with an adapter come first
    for (int64_t q0 = i0; q0 < v1;) {
      const int a_id = p.mo.sid[q0];
      const int64_t q1 = min(i1, (int64_t)p.mo.seg[a_id + 1]);
      const float sc = p.mo.scale[a_id];
      const u16* fac = p.lb + (int64_t)a_id * p.ad_stride;
      for (int64_t c0 = 0; c0 < p.r; c0 += BK) {
        ProdCC<BN> lbc;
        ProdT<BN> lbt;
        if constexpr (LORA == LORA_FWD) lbc.load(fac, p.r, p.J, p.r, j0, c0, p.lb_vec, tid);
        else lbt.load(fac, p.J, p.r, p.J, j0, c0, p.lb_vec, tid);
        // the rows' operand as two bf16 terms, one after the other through sA
#pragma unroll 1
        for (int term = 0; term < 2; ++term) {
          __syncthreads();
#pragma unroll
          for (int q = 0; q < BM / 32; ++q) {
            const int64_t pos = i0 + tid / 8 + 32 * q, c = c0 + (tid % 8) * 8;
            float x[8];
            uint32_t hi[4], lo[4];
            const bool in = pos >= q0 && pos < q1;
            const float* src = p.la + (in ? (int64_t)p.mo.perm[pos] : 0) * p.r;
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = in && c + e < p.r ? sc * src[c + e] : 0.0f;
#pragma unroll
            for (int e = 0; e < 4; ++e) split_bf16x2(x[2 * e], x[2 * e + 1], hi[e], lo[e]);
            *reinterpret_cast<uint4*>(sA + (tid / 8 + 32 * q) * PITCH + (tid % 8) * 8) =
                make_uint4(term ? lo[0] : hi[0], term ? lo[1] : hi[1], term ? lo[2] : hi[2], term ? lo[3] : hi[3]);
          }
          if (term == 0) {
            if constexpr (LORA == LORA_FWD) lbc.store(sB, tid);
            else lbt.store(sB, tid);
          }
          __syncthreads();
#pragma unroll
          for (int a = 0; a < TM; ++a)
#pragma unroll
            for (int b = 0; b < TN; ++b) {
              f32x16_t t;
#pragma unroll
              for (int v = 0; v < 16; ++v) t[v] = 0.0f;
#pragma unroll
              for (int ks = 0; ks < BK / 16; ++ks) {
                const bf16x8_t fa = *reinterpret_cast<const bf16x8_t*>(
                    sA + (wm * (BM / WM) + a * 32 + (lane & 31)) * PITCH + ks * 16 + (lane >> 5) * 8);
                const bf16x8_t fb = *reinterpret_cast<const bf16x8_t*>(
                    sB + (wn * (BN / WN) + b * 32 + (lane & 31)) * PITCH + ks * 16 + (lane >> 5) * 8);
                t = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa, fb, t, 0, 0, 0);
              }
#pragma unroll
              for (int v = 0; v < 16; ++v) {
                const int64_t pos = i0 + wm * (BM / WM) + a * 32 + (v >> 2) * 8 + (lane >> 5) * 4 + (v & 3);
                acc[a][b][v] += pos >= q0 && pos < q1 ? t[v] : 0.0f;
              }
            }
        }
      }
      q0 = q1;
    }
  }

  // ---- LoRA prologue ----
  if constexpr (LORA != LORA_NONE && MULTI == MULTI_NONE) {
    for (int64_t c0 = 0; c0 < p.r; c0 += BK) {
      ProdCCF32<BM> la;
      la.load(p.la, p.r, p.I, p.r, i0, c0, p.la_vec, tid);
      if constexpr (LORA == LORA_FWD) {
        ProdCC<BN> lb;  // B [J][r]
        lb.load(p.lb, p.r, p.J, p.r, j0, c0, p.lb_vec, tid);
        __syncthreads();
        la.store(sA, tid);
        lb.store(sB, tid);
      } else {
        ProdT<BN> lb;   // A [r][J]
        lb.load(p.lb, p.J, p.r, p.J, j0, c0, p.lb_vec, tid);
        __syncthreads();
        la.store(sA, tid);
        lb.store(sB, tid);
      }
      __syncthreads();
      mma_tile();
    }
#pragma unroll
    for (int a = 0; a < TM; ++a)
#pragma unroll
      for (int b = 0; b < TN; ++b)
#pragma unroll
        for (int v = 0; v < 16; ++v) acc[a][b][v] *= p.s;
  }

  // ---- main contraction ----
  constexpr bool ROWS_A = MULTI == MULTI_ROWS || MULTI == MULTI_MAIN;
  using PA = typename std::conditional<
      ASRC == SRC_CC, typename std::conditional<ROWS_A, ProdCCRows<BM>, ProdCC<BM>>::type,
      typename std::conditional<ASRC == SRC_TR, ProdTR<BM>, ProdT<BM>>::type>::type;
  PA pa;
  ProdCC<BN> pbcc;
  ProdT<BN> pbt;
  ProdTF32S<BN> pbs;
  ProdTF32SR<BN> pbr;
  ProdNF4CC pn;
  ProdNF4T pnt;
  const u16* bsrc = reinterpret_cast<const u16*>(p.b);
  if constexpr (MULTI == MULTI_ROWS) bsrc += (int64_t)ad * p.ad_stride;
  if constexpr (ROWS_A) pa.init(p.mo.perm, i0, i1, tid);

  // SEGS: the matrix rows of a stage's contraction positions, looked up one
  // stage before its loads
  int32_t seg_rows[4];
  auto look_up = [&](int64_t c0) {
#pragma unroll
    for (int q = 0; q < 4; ++q) seg_rows[q] = p.mo.perm[min(c0 + tid / 16 + 16 * q, p.M - 1)];
  };
  // (nothing is computed from the rows before this point, a stage after their look-up)
  auto touch_rows = [&]() {
#pragma unroll
    for (int q = 0; q < 4; ++q) asm volatile("" : "+v"(seg_rows[q]));
  };
  auto load_stage = [&](int64_t c0) {
    if constexpr (MULTI == MULTI_SEGS) touch_rows();
    if constexpr (MULTI == MULTI_SEGS) pa.load_rows(sg.a, sg.lda, sg.I, i0, seg_rows, tid);
    else if constexpr (ROWS_A) pa.load(p.a, p.lda, p.C, c0, tid);
    else if constexpr (ASRC == SRC_CC) pa.load(p.a, p.lda, p.I, p.C, i0, c0, p.a_vec, tid);
    else pa.load(p.a, p.lda, p.C, p.I, i0, c0, p.a_vec, tid);
    if constexpr (BSRC == SRC_CC && MULTI == MULTI_ROWS) pbcc.load_clamped(bsrc, p.ldb, p.J, c0, tid);
    else if constexpr (BSRC == SRC_CC) pbcc.load(bsrc, p.ldb, p.J, p.C, j0, c0, p.b_vec, tid);
    else if constexpr (BSRC == SRC_T && MULTI == MULTI_ROWS)
      pbt.template load_clamped<BVEC>(bsrc, p.C, p.J, c0, tid);
    else if constexpr (BSRC == SRC_T) pbt.load(bsrc, p.ldb, p.C, p.J, j0, c0, p.b_vec, tid);
    else if constexpr (BSRC == SRC_TF32S)
      pbs.load(reinterpret_cast<const float*>(p.b), p.ldb, p.C, p.J, j0, c0, p.b_vec, tid);
    else if constexpr (MULTI == MULTI_SEGS)
      pbr.template load_rows<BVEC>(sg.b, p.ldb, p.J, seg_rows, tid);
    else if constexpr (BSRC == SRC_TF32SR)
      pbr.load(reinterpret_cast<const float*>(p.b), p.ldb, p.C, p.J, j0, c0, p.b_vec, tid);
    else if constexpr (BSRC == SRC_NF4CC) pn.load(p.w, j0, c0, tid);
    else pnt.load(p.w, j0, c0, tid);
  };
  auto store_stage = [&](int64_t c0) {
    if constexpr (MULTI != MULTI_NONE) {
      const int64_t end = MULTI == MULTI_SEGS ? cs1 : p.C;
      if (c0 + BK > end) {
        pa.keep(end - c0, tid);
        if constexpr (MULTI == MULTI_SEGS) pbr.keep(end - c0, tid);
        else if constexpr (BSRC == SRC_T) pbt.keep(end - c0, tid);
      }
    }
    pa.store(sA, tid);
    if constexpr (BSRC == SRC_CC) pbcc.store(sB, tid);
    else if constexpr (BSRC == SRC_T) pbt.store(sB, tid);
    else if constexpr (BSRC == SRC_TF32S) pbs.store(sB, sB2, tid);
    else if constexpr (BSRC == SRC_TF32SR) pbr.store(sB, sB2, tid);
    else if constexpr (BSRC == SRC_NF4CC) pn.store(sB, sL, tid);
    else pnt.store(sB, sL, tid);
  };

  if (cs0 < cs1) {
    if constexpr (MULTI == MULTI_SEGS) look_up(cs0);
    load_stage(cs0);
    if constexpr (MULTI == MULTI_SEGS) look_up(cs0 + BK);
    for (int64_t c0 = cs0; c0 < cs1; c0 += BK) {
      __syncthreads();
      store_stage(c0);
      __syncthreads();
      if (c0 + BK < cs1) {
        load_stage(c0 + BK);
        if constexpr (MULTI == MULTI_SEGS) look_up(c0 + 2 * BK);
      } else if constexpr (MULTI == MULTI_SEGS) {
        touch_rows();   // (else the wait for the last look-up stands behind both ways, and waits for the loads)
      }
      mma_tile();
    }
  }

  // ---- epilogue ----
  // (many adapters: what the stores need of the order is read before the
  // first of them; read in between, every store waited for such a load)
  bool seg_whole = false;
  float seg_scale = 0.0f;
  float* seg_part = nullptr;
  if constexpr (MULTI == MULTI_SEGS) {
    seg_whole = cs0 == p.mo.seg[ad] && cs1 == p.mo.seg[ad + 1];
    seg_scale = p.mo.scale[ad];
    const int64_t k = cs0 / sg.step;
    seg_part = sg.part + (cs0 % sg.step == 0 ? k : sg.nt + k) * sg.I * p.J;
  }
  int32_t out_row[TM][16];
  if constexpr (ROWS_A) {
#pragma unroll
    for (int a = 0; a < TM; ++a)
#pragma unroll
      for (int v = 0; v < 16; ++v) {
        const int64_t i = i0 + wm * (BM / WM) + a * 32 + (v >> 2) * 8 + (lane >> 5) * 4 + (v & 3);
        const int32_t row = p.mo.perm[i < i1 ? i : i0];
        out_row[a][v] = i < i1 ? row : -1;
      }
  }
#pragma unroll
  for (int a = 0; a < TM; ++a)
#pragma unroll
    for (int b = 0; b < TN; ++b) {
      const int64_t j = j0 + wn * (BN / WN) + b * 32 + (lane & 31);
#pragma unroll
      for (int v = 0; v < 16; ++v) {
        int64_t i = i0 + wm * (BM / WM) + a * 32 + (v >> 2) * 8 + (lane >> 5) * 4 + (v & 3);
        if constexpr (MULTI == MULTI_SEGS) {
          if (!seg_whole) {          // a piece's sums [slot][I][J]
            if (i < sg.I && j < p.J) seg_part[i * p.J + j] = acc[a][b][v];
          } else if (sg.trans) {     // dA [ad][J][I]: four columns a store (I a multiple of 64)
            if ((v & 3) == 0 && i < sg.I && j < p.J) {
              const uint2 x = make_uint2(pack_bf16x2(acc[a][b][v] * seg_scale, acc[a][b][v + 1] * seg_scale),
                                         pack_bf16x2(acc[a][b][v + 2] * seg_scale, acc[a][b][v + 3] * seg_scale));
              *reinterpret_cast<uint2*>(sg.out + ((int64_t)ad * p.J + j) * sg.I + i) = x;
            }
          } else if ((v & 1) == 0) {
            // dB [ad][I][J]: neighbouring lanes swap, so that an even lane stores its
            // and its neighbour's column of row i, an odd one those of row i + 1
            const bool odd = lane & 1;
            const float x0 = acc[a][b][v] * seg_scale, x1 = acc[a][b][v + 1] * seg_scale;
            const float got = dpp_f32<DPP_QUAD_XOR1>(odd ? x0 : x1);
            const int64_t ii = i + (odd ? 1 : 0), jj = j & ~(int64_t)1;
            if (ii < sg.I && jj < p.J) {
              u16* dst = sg.out + ((int64_t)ad * sg.I + ii) * p.J + jj;
              const uint32_t x = odd ? pack_bf16x2(got, x1) : pack_bf16x2(x0, got);
              if (jj + 1 < p.J) __builtin_memcpy(dst, &x, 4);   // (at any 2-byte boundary)
              else *dst = (u16)x;
            }
          }
          continue;
        }
        if constexpr (ROWS_A) i = out_row[a][v] >= 0 ? out_row[a][v] : p.I;
        if (i < p.I && j < p.J) {
          if constexpr (OUT == OUT_F32) {
            float* o = reinterpret_cast<float*>(p.out);
            o[((int64_t)blockIdx.z * p.I + i) * p.J + j] = acc[a][b][v];
          } else {
            u16* o = reinterpret_cast<u16*>(p.out);
            const u16 h = f32_to_bf16(acc[a][b][v] * p.out_scale);
            if constexpr (STORE_T) o[j * p.ldo + i] = h;
            else o[i * p.ldo + j] = h;
          }
        }
      }
    }
}

// Sum split partials [splits][I][J] in order, scale, round to bf16; store
// [I][J] (ldo) or transposed [J][I] (ldo).
template <typename OutT>
__global__ __launch_bounds__(256) void k_reduce(const float* __restrict__ part, int splits,
                                                int64_t I, int64_t J, float scale,
                                                OutT* __restrict__ out, int64_t ldo, bool trans) {
  const int64_t n = I * J;
  for (int64_t e = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; e < n;
       e += (int64_t)gridDim.x * blockDim.x) {
    float s = 0.0f;
#pragma unroll 8
    for (int z = 0; z < splits; ++z) s += part[(int64_t)z * n + e];
    const int64_t i = e / J, j = e % J;
    OutT h;
    if constexpr (sizeof(OutT) == 2) h = f32_to_bf16(s * scale);
    else h = s * scale;
    if (trans) out[j * ldo + i] = h;
    else out[i * ldo + j] = h;
  }
}

// dB and dA of the adapters of several pieces: the pieces' sums in order, times
// the scale, rounded to bf16: [ad][I][J], or [ad][J][I] through an LDS
// transpose (dA).  One workgroup per 32 x 32 tile (blockIdx.x: those of dB,
// then of dA) and multiple of the step (blockIdx.z + 1); the first multiple
// inside an adapter's tokens does it.  A piece from a multiple k of the step
// has slot k, one from the adapter's start inside step k slot nt + k.
__global__ __launch_bounds__(256) void k_reduce_multi(SegsHalf h0, SegsHalf h1, MultiOrder mo, int J) {
  __shared__ float tile[32][33];
  const int t0 = (int)((h0.I + 31) / 32);
  const bool second = (int)blockIdx.x >= t0;
  const int64_t step = second ? h1.step : h0.step, nt = second ? h1.nt : h0.nt, I = second ? h1.I : h0.I;
  const float* part = second ? h1.part : h0.part;
  u16* out = second ? h1.out : h0.out;
  const bool trans = second ? h1.trans : h0.trans;
  const int64_t k0 = (int64_t)blockIdx.z + 1;
  if (k0 >= nt) return;
  const int64_t ad = mo.sid[k0 * step];
  if (ad == mo.count) return;
  const int64_t s0 = mo.seg[ad], s1 = mo.seg[ad + 1];
  if (k0 * step <= s0 || (k0 - 1) * step > s0) return;
  const int64_t first = s0 % step == 0 ? k0 - 1 : nt + k0 - 1;   // slot of the piece up to k0 * step
  const int64_t pieces = 1 + (s1 - 1) / step - (k0 - 1);
  const int64_t i0 = (int64_t)((int)blockIdx.x - (second ? t0 : 0)) * 32, IJ = I * J;
  const int j0 = blockIdx.y * 32, x = threadIdx.x & 31, y = threadIdx.x >> 5;
  const float s = mo.scale[ad];
  float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
  for (int64_t z = 0; z < pieces; ++z) {
    const float* src = part + (z == 0 ? first : k0 + z - 1) * IJ;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int64_t i = i0 + y + 8 * k;
      v[k] += src[i < I && j0 + x < J ? i * J + j0 + x : 0];
    }
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int64_t i = i0 + y + 8 * k;
    if (trans) tile[y + 8 * k][x] = v[k] * s;
    else if (i < I && j0 + x < J) out[(ad * I + i) * J + j0 + x] = f32_to_bf16(v[k] * s);
  }
  if (trans) {
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int64_t i = i0 + x;
      const int j = j0 + y + 8 * k;
      if (i < I && j < J) out[(ad * J + j) * I + i] = f32_to_bf16(tile[x][y + 8 * k]);
    }
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
static bool vec_ok(const void* p, int64_t ld) {
  return ((uintptr_t)p % 16 == 0) && (ld % 8 == 0);
}

int rank_tile(int r) { return r <= 32 ? 32 : (r <= 64 ? 64 : 128); }

static int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Workgroups a skinny product aims for (two 128-row workgroups per CU):
// doubling it shortened no product and doubled the fixed-order reduction.
constexpr int64_t kSkinnyWorkgroups = 512;

SkinnyPlan skinny_plan(int64_t I, int64_t C) {
  const int64_t tiles = cdiv(I, 128);
  const int64_t ctiles = cdiv(C, BK);
  int64_t splits = std::max<int64_t>(1, cdiv(kSkinnyWorkgroups, tiles));
  splits = std::min<int64_t>(splits, std::max<int64_t>(1, ctiles / 4));
  splits = std::min<int64_t>(splits, 64);
  const int64_t per = cdiv(ctiles, splits) * BK;
  SkinnyPlan pl;
  pl.splits = (int)cdiv(C, per);
  pl.c_per_split = per;
  return pl;
}

int64_t skinny_partial_elems(int64_t I, int64_t C, int r) {
  const SkinnyPlan pl = skinny_plan(I, C);
  return (int64_t)pl.splits * I * r;
}

template <typename OutT>
static hipError_t launch_reduce(const float* part, int splits, int64_t I, int64_t J, float scale,
                                OutT* out, int64_t ldo, bool trans, hipStream_t st) {
  int64_t grid = std::min<int64_t>(cdiv(I * J, 256), 8192);
  hipLaunchKernelGGL(k_reduce<OutT>, dim3((unsigned)grid), dim3(256), 0, st, part, splits, I, J,
                     scale, out, ldo, trans);
  return hipGetLastError();
}

template <int ASRC, int BSRC>
static hipError_t launch_skinny(GemmArgs& p, hipStream_t st) {
  const SkinnyPlan pl = skinny_plan(p.I, p.C);
  p.c_per_split = pl.c_per_split;
  dim3 grid((unsigned)cdiv(p.I, 128), 1, (unsigned)pl.splits);
  const int rt = rank_tile((int)p.J);
  if (rt == 32)
    hipLaunchKernelGGL((k_gemm<128, 32, 4, 1, ASRC, BSRC, LORA_NONE, OUT_F32, false>), grid,
                       dim3(NTHREADS), 0, st, p);
  else if (rt == 64)
    hipLaunchKernelGGL((k_gemm<128, 64, 4, 1, ASRC, BSRC, LORA_NONE, OUT_F32, false>), grid,
                       dim3(NTHREADS), 0, st, p);
  else
    hipLaunchKernelGGL((k_gemm<128, 128, 4, 1, ASRC, BSRC, LORA_NONE, OUT_F32, false>), grid,
                       dim3(NTHREADS), 0, st, p);
  return hipGetLastError();
}

static GemmArgs zero_args() {
  GemmArgs p;
  __builtin_memset(&p, 0, sizeof(p));
  p.out_scale = 1.0f;
  return p;
}

hipError_t launch_lora_down(const u16* X, const u16* A, int64_t M, int64_t K, int r,
                            float* ws, float* T, hipStream_t st) {
  GemmArgs p = zero_args();
  p.a = X; p.lda = K; p.a_vec = vec_ok(X, K);
  p.b = A; p.ldb = K; p.b_vec = vec_ok(A, K);
  p.I = M; p.J = r; p.C = K;
  p.out = ws;
  hipError_t e = launch_skinny<SRC_CC, SRC_CC>(p, st);
  if (e != hipSuccess) return e;
  return launch_reduce(ws, skinny_plan(M, K).splits, M, r, 1.0f, T, r, false, st);
}

hipError_t launch_lora_u(const u16* dY, const u16* B, int64_t M, int64_t N, int r, float* ws,
                         float* U, hipStream_t st) {
  GemmArgs p = zero_args();
  p.a = dY; p.lda = N; p.a_vec = vec_ok(dY, N);
  p.b = B; p.ldb = r; p.b_vec = vec_ok(B, r);
  p.I = M; p.J = r; p.C = N;
  p.out = ws;
  hipError_t e = launch_skinny<SRC_CC, SRC_T>(p, st);
  if (e != hipSuccess) return e;
  return launch_reduce(ws, skinny_plan(M, N).splits, M, r, 1.0f, U, r, false, st);
}

hipError_t launch_lora_db(const u16* dY, const float* T, int64_t M, int64_t N, int r, float s,
                          float* ws, u16* dB, hipStream_t st) {
  GemmArgs p = zero_args();
  p.a = dY; p.lda = N; p.a_vec = vec_ok(dY, N);
  p.b = T; p.ldb = r; p.b_vec = vec_ok(T, r * 2);
  p.I = N; p.J = r; p.C = M;
  p.out = ws;
  hipError_t e = launch_skinny<SRC_TR, SRC_TF32SR>(p, st);
  if (e != hipSuccess) return e;
  return launch_reduce(ws, skinny_plan(N, M).splits, N, r, s, dB, r, false, st);
}

hipError_t launch_lora_da(const float* U, const u16* X, int64_t M, int64_t K, int r, float s,
                          float* ws, u16* dA, hipStream_t st) {
  // dA^T [K][r] = X^T U, stored transposed into dA [r][K]
  GemmArgs p = zero_args();
  p.a = X; p.lda = K; p.a_vec = vec_ok(X, K);
  p.b = U; p.ldb = r; p.b_vec = vec_ok(U, r * 2);
  p.I = K; p.J = r; p.C = M;
  p.out = ws;
  hipError_t e = launch_skinny<SRC_TR, SRC_TF32SR>(p, st);
  if (e != hipSuccess) return e;
  return launch_reduce(ws, skinny_plan(K, M).splits, K, r, s, dA, K, true, st);
}

// ---- many adapters ----
// T and U: pieces of at most 128 rows of one adapter's run; the run starts
// that are not multiples of 128 add up to one piece an adapter
static int64_t rows_pieces(int64_t M, int count) { return cdiv(M, 128) + count + 1; }
// (splits down to two stages of 64: a stage takes over a microsecond of latency,
// which is all of a small batch's time; about two workgroups a compute unit: with
// four, T of 4096 tokens, K = 8192, r = 64 takes 27.6 us for 25.2 with its sum, U
// of 8192 tokens, N = 11008 the same 49)
static SkinnyPlan multi_rows_plan(int64_t M, int64_t C, int count, int64_t most) {
  const int64_t nt = cdiv(M, 128), ctiles = cdiv(C, BK);
  int64_t splits = std::max<int64_t>(1, cdiv(kSkinnyWorkgroups, nt + std::min<int64_t>(count, nt)));
  splits = std::min<int64_t>({splits, std::max<int64_t>(1, ctiles / 2), most});
  const int64_t per = cdiv(ctiles, splits) * BK;
  return SkinnyPlan{(int)cdiv(C, per), per};
}
// T: up to eight slices that every column tile reads again, 16 MB in all, are
// added up by the fused kernel, for a launch less (333 tokens, 1000x1984, r = 12: a
// call 32.7 us for 33.8); with more of them the launch is cheaper (520 tokens,
// 4096^2, r = 64: 60 us for 72 in the kernel; 318, 11008x8192: 139 for 203).  A
// short contraction (40 stages) is cut into eight for it: 32.7 us for 34.1.
static bool t_sliced(int64_t slices, int64_t M, int64_t N, int r) {
  return slices <= 8 && slices * M * r * 4 * cdiv(N, 256) <= (int64_t)16 << 20;
}
static SkinnyPlan multi_t_plan(int64_t M, int64_t N, int64_t K, int r, int count) {
  return multi_rows_plan(M, K, count, cdiv(K, BK) <= 40 && t_sliced(8, M, N, r) ? 8 : 64);
}
bool multi_t_sliced(int64_t M, int64_t N, int64_t K, int r, int count) {
  return t_sliced(multi_t_plan(M, N, K, r, count).splits, M, N, r);
}
// dA and dB: the longest piece of an adapter's tokens, so that the pieces of
// evenly cut tokens fill the chip about twice (kSkinnyWorkgroups), at least 256
// (a backward with 128, 256, 512: 1030 tokens, 4096^2, r = 64 99.9, 97.3, 100.6 us;
// 2000 tokens, 2048^2, r = 100 92.0, 89.7, 99.7; 777, 1003x832, r = 3 48.5, 48.2,
// 44.9)
static int64_t segs_step(int64_t I, int64_t M) {
  const int64_t nt = std::max<int64_t>(1, std::min<int64_t>({cdiv(kSkinnyWorkgroups, cdiv(I, 128)), M / 256, 64}));
  return cdiv(cdiv(M, nt), BK) * BK;
}
static int64_t segs_elems(int64_t I, int64_t M, int r) {
  const int64_t nt = cdiv(M, segs_step(I, M));
  return nt > 1 ? 2 * nt * I * r : 0;
}
int64_t multi_partial_elems(int64_t M, int64_t N, int64_t K, int r, int count, bool backward) {
  int64_t e = (int64_t)multi_t_plan(M, N, K, r, count).splits * M * r;
  if (backward) {
    e = std::max<int64_t>(e, (int64_t)multi_rows_plan(M, N, count, 64).splits * M * r);
    e = std::max<int64_t>(e, segs_elems(N, M, r) + segs_elems(K, M, r));
  }
  return e;
}

template <int BSRC, bool BVEC>
static hipError_t launch_rows(GemmArgs& p, const SkinnyPlan& pl, float* ws, float* out, MultiParts* slices,
                              hipStream_t st) {
  p.c_per_split = pl.c_per_split;
  p.out = ws;
  const dim3 grid((unsigned)rows_pieces(p.I, p.mo.count), 1, (unsigned)pl.splits);
  const int rt = rank_tile((int)p.J);
  if (rt == 32)
    hipLaunchKernelGGL((k_gemm<128, 32, 4, 1, SRC_CC, BSRC, LORA_NONE, OUT_F32, false, MULTI_ROWS, BVEC>), grid,
                       dim3(NTHREADS), 0, st, p);
  else if (rt == 64)
    hipLaunchKernelGGL((k_gemm<128, 64, 4, 1, SRC_CC, BSRC, LORA_NONE, OUT_F32, false, MULTI_ROWS, BVEC>), grid,
                       dim3(NTHREADS), 0, st, p);
  else
    hipLaunchKernelGGL((k_gemm<128, 128, 4, 1, SRC_CC, BSRC, LORA_NONE, OUT_F32, false, MULTI_ROWS, BVEC>), grid,
                       dim3(NTHREADS), 0, st, p);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (slices) {
    *slices = MultiParts{ws, pl.splits, p.I * p.J, (int)p.J};
    return hipSuccess;
  }
  return launch_reduce(ws, pl.splits, p.I, p.J, 1.0f, out, p.J, false, st);
}

hipError_t launch_multi_t(const MultiOrder& mo, const u16* X, const u16* A, int64_t M, int64_t N, int64_t K, int r,
                          float* ws, float* T, MultiParts* slices, hipStream_t st) {
  GemmArgs p = zero_args();
  p.a = X; p.lda = K;   // (K a multiple of 64: 16-byte aligned rows)
  p.b = A; p.ldb = K; p.ad_stride = (int64_t)r * K;
  p.I = M; p.J = r; p.C = K; p.mo = mo;
  return launch_rows<SRC_CC, true>(p, multi_t_plan(M, N, K, r, mo.count), ws, T, slices, st);
}

hipError_t launch_multi_u(const MultiOrder& mo, const u16* dY, int64_t ldy, const u16* B, int64_t M, int64_t N, int r,
                          float* ws, float* U, hipStream_t st) {
  GemmArgs p = zero_args();
  p.a = dY; p.lda = ldy;   // (ldy a multiple of 8: 16-byte aligned rows)
  p.b = B; p.ldb = r; p.ad_stride = N * r;
  p.I = M; p.J = r; p.C = N; p.mo = mo;
  const SkinnyPlan pl = multi_rows_plan(M, N, mo.count, 64);
  return r % 8 == 0 ? launch_rows<SRC_T, true>(p, pl, ws, U, nullptr, st)
                    : launch_rows<SRC_T, false>(p, pl, ws, U, nullptr, st);
}

static SegsHalf segs_half(const u16* a, int64_t lda, const float* b, int64_t I, int64_t M, float* part, u16* out,
                          bool trans) {
  SegsHalf h;
  __builtin_memset(&h, 0, sizeof(h));
  h.a = a; h.lda = lda;
  h.b = b; h.I = I;
  h.step = segs_step(I, M); h.nt = cdiv(M, h.step);
  h.part = part; h.out = out; h.trans = trans;
  h.tiles = (int)cdiv(I, 128);
  return h;
}

template <bool BVEC>
static void launch_segs(const GemmArgs& p, dim3 grid, hipStream_t st) {
  const int rt = rank_tile((int)p.J);
  if (rt == 32)
    hipLaunchKernelGGL((k_gemm<128, 32, 4, 1, SRC_TR, SRC_TF32SR, LORA_NONE, OUT_F32, false, MULTI_SEGS, BVEC>), grid,
                       dim3(NTHREADS), 0, st, p);
  else if (rt == 64)
    hipLaunchKernelGGL((k_gemm<128, 64, 4, 1, SRC_TR, SRC_TF32SR, LORA_NONE, OUT_F32, false, MULTI_SEGS, BVEC>), grid,
                       dim3(NTHREADS), 0, st, p);
  else
    hipLaunchKernelGGL((k_gemm<128, 128, 4, 1, SRC_TR, SRC_TF32SR, LORA_NONE, OUT_F32, false, MULTI_SEGS, BVEC>), grid,
                       dim3(NTHREADS), 0, st, p);
}

hipError_t launch_multi_dadb(const MultiOrder& mo, const u16* dY, int64_t ldy, const float* T, const u16* X,
                             const float* U, int64_t M, int64_t N, int64_t K, int r, float* ws, u16* dA, u16* dB,
                             hipStream_t st) {
  GemmArgs p = zero_args();
  p.ldb = r;
  p.J = r; p.mo = mo; p.M = M;
  p.seg[0] = segs_half(dY, ldy, T, N, M, ws, dB, false);
  p.seg[1] = segs_half(X, K, U, K, M, ws + segs_elems(N, M, r), dA, true);
  const int64_t nt = std::max(p.seg[0].nt, p.seg[1].nt);
  const dim3 grid((unsigned)(p.seg[0].tiles + p.seg[1].tiles), (unsigned)(nt + mo.count));
  if (r % 4 == 0) launch_segs<true>(p, grid, st);
  else launch_segs<false>(p, grid, st);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || nt == 1) return e;
  hipLaunchKernelGGL(k_reduce_multi, dim3((unsigned)(cdiv(N, 32) + cdiv(K, 32)), (unsigned)cdiv(r, 32), (unsigned)(nt - 1)),
                     dim3(256), 0, st, p.seg[0], p.seg[1], mo, r);
  return hipGetLastError();
}

hipError_t launch_multi_fwd_generic(const MultiOrder& mo, const NF4View& w, const u16* X, int64_t M, const float* T,
                                    const u16* B, int r, u16* Y, hipStream_t st) {
  GemmArgs p = zero_args();
  p.a = X; p.lda = w.K;
  p.w = w;
  p.I = M; p.J = w.N; p.C = w.K; p.c_per_split = w.K;
  p.la = T; p.lb = B; p.r = r; p.lb_vec = vec_ok(B, r); p.ad_stride = w.N * r;
  p.out = Y; p.ldo = w.N; p.mo = mo;
  dim3 grid((unsigned)cdiv(M, 128), (unsigned)cdiv(w.N, 128), 1);
  hipLaunchKernelGGL((k_gemm<128, 128, 2, 2, SRC_CC, SRC_NF4CC, LORA_FWD, OUT_BF16, false, MULTI_MAIN>), grid,
                     dim3(NTHREADS), 0, st, p);
  return hipGetLastError();
}

hipError_t launch_multi_dx_generic(const MultiOrder& mo, const NF4View& w, const u16* dY, int64_t ldy, int64_t M,
                                   const float* U, const u16* A, int r, u16* dX, hipStream_t st) {
  GemmArgs p = zero_args();
  p.a = dY; p.lda = ldy;
  p.w = w;
  p.I = M; p.J = w.K; p.C = w.N; p.c_per_split = w.N;
  p.la = U; p.lb = A; p.r = r; p.lb_vec = vec_ok(A, w.K); p.ad_stride = (int64_t)r * w.K;
  p.out = dX; p.ldo = w.K; p.mo = mo;
  dim3 grid((unsigned)cdiv(M, 128), (unsigned)cdiv(w.K, 128), 1);
  hipLaunchKernelGGL((k_gemm<128, 128, 2, 2, SRC_CC, SRC_NF4T, LORA_DX, OUT_BF16, false, MULTI_MAIN>), grid,
                     dim3(NTHREADS), 0, st, p);
  return hipGetLastError();
}

// Tile-128 fused GEMMs for the shapes the buffer-load kernels of gemm_big.hip
// do not take (activation rows that are not 16-byte aligned, or operands of
// 2 GiB and more): same math, guarded loads.
hipError_t launch_fwd_generic(const NF4View& w, const u16* X, int64_t M, const float* T,
                           const u16* B, int r, float s, u16* Y, hipStream_t st) {
  GemmArgs p = zero_args();
  p.a = X; p.lda = w.K; p.a_vec = vec_ok(X, w.K);
  p.w = w;
  p.I = M; p.J = w.N; p.C = w.K; p.c_per_split = w.K;
  p.la = T; p.lb = B; p.r = r; p.s = s; p.la_vec = vec_ok(T, r * 2); p.lb_vec = vec_ok(B, r);
  p.out = Y; p.ldo = w.N;
  dim3 grid((unsigned)cdiv(M, 128), (unsigned)cdiv(w.N, 128), 1);
  hipLaunchKernelGGL((k_gemm<128, 128, 2, 2, SRC_CC, SRC_NF4CC, LORA_FWD, OUT_BF16, false>), grid,
                     dim3(NTHREADS), 0, st, p);
  return hipGetLastError();
}

hipError_t launch_dx_generic(const NF4View& w, const u16* dY, int64_t M, const float* U,
                          const u16* A, int r, float s, u16* dX, hipStream_t st) {
  GemmArgs p = zero_args();
  p.a = dY; p.lda = w.N; p.a_vec = vec_ok(dY, w.N);
  p.w = w;
  p.I = M; p.J = w.K; p.C = w.N; p.c_per_split = w.N;
  p.la = U; p.lb = A; p.r = r; p.s = s; p.la_vec = vec_ok(U, r * 2); p.lb_vec = vec_ok(A, w.K);
  p.out = dX; p.ldo = w.K;
  dim3 grid((unsigned)cdiv(M, 128), (unsigned)cdiv(w.K, 128), 1);
  hipLaunchKernelGGL((k_gemm<128, 128, 2, 2, SRC_CC, SRC_NF4T, LORA_DX, OUT_BF16, false>), grid,
                     dim3(NTHREADS), 0, st, p);
  return hipGetLastError();
}


}  // namespace qln
