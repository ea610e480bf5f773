// gemm_big.hip -- the two large fused GEMMs of the QLoRA linear layer:
//
//   forward  Y  = X W'^T + s T B^T      (contraction over k, W' rows are output columns)
//   backward dX = dY W' + s U A          (contraction over n, W' columns are output columns)
//
// W' is the bf16 dequantized NF4 weight, produced tile by tile inside the
// kernel: a thread turns one 64-code block into bf16 exactly as
// nf4_dequantize does (w' = bf16(fl32(L[code] * scale))), through a per-block
// 16-entry bf16 table held in registers and looked up with byte permutes, and
// writes it to LDS with 16-byte stores.  Ultralytics glossary "QLoRA", "How
// QLoRA works": dequantize NF4 to bfloat16 right before the matrix product,
// gradients flow through the dequantized weights.
//
// Tiling (gfx950): 512 threads = 8 waves (two per SIMD, so one wave's MFMAs
// overlap the other's dequantization), output tile 256 x 256, contraction
// step 64.  Each wave owns a 128 x 64 eighth as 4 x 2 accumulators of
// v_mfma_f32_32x32x16_bf16 (128 accumulator registers).  LDS holds two stages
// of both operand tiles (about 144 KiB); global loads run two stages ahead in
// registers, so one barrier per step separates writing stage k+1 from
// reading stage k.  A thread produces a quarter of an A-tile column chunk and
// half of one 64-code weight block per step.  The forward's weight tile is [n][k] (contraction
// contiguous: plain 16-byte fragment reads); the backward's is [n][k] with
// n the contraction, read with ds_read_b64_tr_b16 (within each 16-lane group
// lane i receives element i%4 of the rows addressed by lanes 4j + i/4, which
// yields the column fragment the MFMA needs).
//
// The LoRA term is a prologue: the accumulators start as (s T) B^T or
// (s U) A, with s T / s U rounded to bf16 on the way to LDS (rank r <= 128 in
// steps of 64), then the base product accumulates on top.
//
// Dual projection (forward only): two weights of one shape that read the
// same X, such as the gate and up projections of a Llama-style MLP (the
// models the Transformers "Bitsandbytes" and Ultralytics pages fine-tune), in
// one kernel.  A tile's 256 weight rows are 128 output columns of each
// weight, interleaved in 32-row slices (gate n0..n0+31, up n0..n0+31, gate
// n0+32.., ...), so each wave's two 32-column accumulator blocks hold the
// gate and up sums of the same outputs, and the X tile is read once for both.
// The two LoRA terms share one prologue of contraction 2r: the A side is
// [T_gate | T_up] and a gate row of the B side is [B_gate[n] | 0], an up row
// [0 | B_up[n]].  The epilogue writes both outputs, or silu(g) * u.
//
// Many adapters (MULTI): a tile's 256 rows are 256 positions of the order
// sorted by adapter (multi.hip), read and written through it.  The A side of
// the prologue, scale T of each row, does not depend on the adapter
// whose factor it meets, so it is staged once per 64 ranks, as two bf16
// terms (the rest of the first in the second: 2^-16 left out, as dA and dB
// leave out of T and U; with the first term alone the rounding of scale T was
// as large an error as that of the output); the factors of
// the tile's runs are staged after it, as many as fit the 64-deep stage
// (four of rank <= 16, two of rank <= 32), the next ones loaded while these
// multiply.  A run's product of a 32 x 32 block is summed apart and added to
// the run's rows only, so that no other row sees it, whatever values the
// factor holds.  For the same reason main-loop loads past the contraction's end
// read zeros here (elsewhere they read into the next row and meet zero
// weights, which is the same for finite values).  4096 tokens of 16 adapters, r =
// 64, 28672x8192: 1.70-1.84 ms from card to card, 1.05-1.13 PFLOP/s, bound as one
// adapter's kernel is; 8192 tokens, dX of 11008x4096: 0.65-0.70 ms, 1.05-1.14
// PFLOP/s.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "common.h"
#include "device.h"

namespace qln {
namespace big {

constexpr int BM = 256, BN = 256, BK = 64;
constexpr int APITCH = BK + 8;          // A tile [256][72] bf16 (144-byte rows)
constexpr int FPITCH = BK + 8;          // forward W tile [256 n][72]
constexpr int TPITCH = BN + 32;         // backward W tile [64 n][288] (576-byte rows)
// A tile of TMB 32-row blocks a wave: 64 TMB rows (many adapters take 1, 2 or 4)
template <int TMB>
constexpr int a_elems() { return 64 * TMB * APITCH; }   // 18432 at TMB = 4
constexpr int BF_ELEMS = BN * FPITCH;   // 18432
constexpr int BT_ELEMS = BK * TPITCH;   // 17408
constexpr int NTHREADS = 512;

enum { MODE_FWD = 0, MODE_DX = 1 };

template <int MODE>
constexpr int b_elems() { return MODE == MODE_FWD ? BF_ELEMS : BT_ELEMS; }
// epilogue staging: each wave's 128 x 64 bf16 block, rows padded to 72
constexpr int EPITCH = 72;
template <int TMB>
constexpr int e_elems() { return 32 * TMB * EPITCH; }
template <int MODE, int TMB>
constexpr size_t lds_bytes() {
  const size_t main = (size_t)2 * (a_elems<TMB>() + b_elems<MODE>()) * 2;
  const size_t epi = (size_t)(NTHREADS / 64) * e_elems<TMB>() * 2;
  return main > epi ? main : epi;
}

struct BigArgs {
  const u16* a; int64_t lda; bool a_vec;   // X [M][K] or dY [M][N]
  NF4View w;
  int64_t M, J, C;                         // output M x J, contraction C
  const float* la;                         // T or U, fp32 [M][r]
  const u16* lb;                           // B [N][r] (forward) or A [r][K] (backward)
  int r; float s; bool la_vec; bool lb_vec;
  u16* out; int64_t ldo; bool out_vec;   // out_vec: 16-byte aligned rows
  // dual projection only: the second weight, its T and B, its output
  NF4View w2; const float* la2; const u16* lb2; u16* out2;
  // many adapters only: the sorted order, elements from one adapter's factor to the next
  MultiOrder mo; int64_t ad_stride;
  // many adapters: with gridDim.z > 1 each z takes kt_per steps of the contraction (an even
  // number) and writes fp32 sums of its positions to part [z][M][J]
  float* part; int kt_per;
  // many adapters: la is the sum of la_parts slices, la_step elements apart, rows la_ld wide;
  // with t_save the sums are written there too (fp32 [M][r])
  // (la_size: elements of a slice)
  int la_parts; int64_t la_step, la_size; int la_ld; float* t_save;
};

enum { DUAL_NONE = 0, DUAL_SEPARATE = 1, DUAL_SWIGLU = 2 };

// dual projection: tile row t (0..255) holds output column n0 + dual_col(t)
// of the gate weight (dual_src(t) == 0) or of the up weight (1)
__device__ __forceinline__ int dual_col(int t) { return 32 * (t >> 6) + (t & 31); }
__device__ __forceinline__ int dual_src(int t) { return (t >> 5) & 1; }

typedef __attribute__((address_space(3))) short lds_short;
typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4_t lds_s16x4;

// ---------------------------------------------------------------------------
// dequantization of one 64-code block (32 bytes) into 32 bf16 pairs
// ---------------------------------------------------------------------------
// The two lanes that share a block (lanes 2i and 2i + 1 of a wave) build its
// table together: lane parity p scales the 8 levels 8p .. 8p + 7 and takes
// the other 8 from its partner with a DPP move.  Entries 0..7 of a lane's
// table are its own levels, so lane 1 of a pair looks codes up with bit 3
// flipped (the flip argument of dequant8), which lands every code on its own
// level.
struct Table {
  uint32_t lo[4], hi[4];   // low / high bytes of the 16 bf16 values, 4 per word
};

__device__ __forceinline__ uint32_t dpp_pair_swap(uint32_t x) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, DPP_QUAD_XOR1, 0xF, 0xF, false);
}

// mv: this lane's 8 levels; sc: the block's scale
__device__ __forceinline__ Table make_table(const float (&mv)[8], float sc) {
  uint32_t P[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) P[j] = pack_bf16x2(mv[2 * j] * sc, mv[2 * j + 1] * sc);
  Table t;
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    t.lo[q] = __builtin_amdgcn_perm(P[2 * q + 1], P[2 * q], 0x06040200u);
    t.hi[q] = __builtin_amdgcn_perm(P[2 * q + 1], P[2 * q], 0x07050301u);
  }
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    t.lo[2 + q] = dpp_pair_swap(t.lo[q]);
    t.hi[2 + q] = dpp_pair_swap(t.hi[q]);
  }
  return t;
}

// four 4-bit indices (one per byte) -> their bf16 low bytes and high bytes.
// Byte selectors past 12 read as 0xFF, so each half of the table is looked
// up with the other half's indices pushed past 16 and the two are AND-ed.
__device__ __forceinline__ void lookup4(const Table& t, uint32_t idx, uint32_t& lo, uint32_t& hi) {
  // idx | ((idx << 1) & 0x10101010) as one three-input bit operation
  const uint32_t selA = __builtin_amdgcn_bitop3_b32(idx, idx << 1, 0x10101010u, 0xF8);  // 8..15 -> 24..31 (0xFF)
  const uint32_t selB = selA ^ 0x18181818u;                // indices 0..7 -> 24..31, 8..15 -> 0..7
  lo = __builtin_amdgcn_perm(t.lo[1], t.lo[0], selA) & __builtin_amdgcn_perm(t.lo[3], t.lo[2], selB);
  hi = __builtin_amdgcn_perm(t.hi[1], t.hi[0], selA) & __builtin_amdgcn_perm(t.hi[3], t.hi[2], selB);
}

// 8 codes (one word, element e in bits 4e..4e+3) -> 4 words of bf16 pairs in
// element order.  The codes are first regrouped one per byte in element order
// (bytes of c and c >> 4 interleaved, then masked), so that each lookup's
// bytes pair up directly into two output words.
__device__ __forceinline__ void dequant8(const Table& t, uint32_t c, uint32_t flip, uint32_t o[4]) {
  const uint32_t c4 = c >> 4;
  const uint32_t i03 = (__builtin_amdgcn_perm(c4, c, 0x05010400u) ^ flip) & 0x0F0F0F0Fu;   // codes 0..3
  const uint32_t i47 = (__builtin_amdgcn_perm(c4, c, 0x07030602u) ^ flip) & 0x0F0F0F0Fu;   // codes 4..7
  uint32_t l, h;
  lookup4(t, i03, l, h);
  o[0] = __builtin_amdgcn_perm(h, l, 0x05010400u);
  o[1] = __builtin_amdgcn_perm(h, l, 0x07030602u);
  lookup4(t, i47, l, h);
  o[2] = __builtin_amdgcn_perm(h, l, 0x05010400u);
  o[3] = __builtin_amdgcn_perm(h, l, 0x07030602u);
}

// ---------------------------------------------------------------------------
// Main-loop operand loads go through buffer resources: a load whose byte
// offset is past the buffer's end returns zeros, so rows beyond M, rows of W
// beyond N and the stages past the last one need no branches.  (A row read
// past the contraction length C of the backward's dY runs into the next row;
// those values meet W rows beyond N, which read as zero codes with a zero
// scale, so they add nothing.)
// ---------------------------------------------------------------------------
typedef uint32_t u32x4v __attribute__((ext_vector_type(4)));

struct Bufs {
  __amdgpu_buffer_rsrc_t a, codes, qscale, dscale;
  uint32_t qor, dshift;   // scale format: E4M3 code OR-ed in (QOR_U8: integer scales), group shift of dscale
};

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void* p, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, (int)bytes, 0x00020000);
}

__device__ __forceinline__ uint4 bload16(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  const u32x4v v = __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0);
  return make_uint4(v.x, v.y, v.z, v.w);
}

template <int TMB>
struct StageA { uint4 v[TMB]; };                  // A tile: 16 bytes per thread and 64 rows
struct StageW { uint4 c; uint32_t q; float d; };  // half a block's codes, raw scale byte, group constant

// A tile rows m0 + tid/8 + 64q, contraction c0 + 8*(tid%8) .. +8
__device__ __forceinline__ void load_a(StageA<4>& st, const Bufs& b, uint32_t row_off0,
                                       uint32_t row_step, uint32_t c0) {
#pragma unroll
  for (int q = 0; q < 4; ++q) st.v[q] = bload16(b.a, row_off0 + q * row_step + 2 * c0);
}

// the thread's half block: row n, columns k + 32*half .. +32.  The scale is
// decoded only when the block is dequantized (one step later), so nothing
// waits for these loads now; a stage past the last one (live == false) gets
// group constant 0, so it multiplies as a zero tile.
__device__ __forceinline__ void load_w(StageW& st, const Bufs& b, uint32_t n, uint32_t k, uint32_t half,
                                       uint32_t K, bool live) {
  st.c = bload16(b.codes, n * (K / 2) + k / 2 + 16 * half);
  const uint32_t blk = n * (K / 64) + k / 64;
  st.q = __builtin_amdgcn_raw_buffer_load_b8(b.qscale, blk, 0, 0);
  // a dead stage reads past the end of the group constants, which returns 0
  st.d = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(
                                       b.dscale, live ? 4 * (blk >> b.dshift) : 0xFFFFFFF0u, 0, 0));
}

// fl32(E4M3(q) * d); with fp32 scales q reads 0 from an empty buffer and the
// OR makes it E4M3(1.0), so the product is the stored scale exactly; with
// uint8-linear scales (qor == QOR_U8) fl32(q * d)
constexpr uint32_t QOR_U8 = 0x100u;
__device__ __forceinline__ float stage_scale(const StageW& st, uint32_t qor) {
  const float v = qor == QOR_U8 ? (float)(st.q & 0xFFu)
                                : __builtin_amdgcn_cvt_f32_fp8((int)(st.q | qor), 0);
  return v * st.d;
}

template <int TMB>
__device__ __forceinline__ void store_a(const StageA<TMB>& st, u16* sA, int tid) {
#pragma unroll
  for (int q = 0; q < TMB; ++q)
    *reinterpret_cast<uint4*>(sA + (tid / 8 + 64 * q) * APITCH + (tid % 8) * 8) = st.v[q];
}

// LoRA prologue A-side tile: s times fp32 T or U, rounded to bf16 (guarded loads)
__device__ __forceinline__ void lora_a_tile(const float* src, int64_t ld, int64_t rows,
                                            int64_t C, int64_t m0, int64_t c0, bool vec,
                                            float s, u16* sA, int tid) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int64_t row = m0 + tid / 8 + 64 * q;
    const int64_t c = c0 + (tid % 8) * 8;
    float x[8];
    if (row < rows && c + 8 <= C && vec) {
      const float4 u = *reinterpret_cast<const float4*>(src + row * ld + c);
      const float4 v = *reinterpret_cast<const float4*>(src + row * ld + c + 4);
      x[0] = u.x; x[1] = u.y; x[2] = u.z; x[3] = u.w; x[4] = v.x; x[5] = v.y; x[6] = v.z; x[7] = v.w;
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = (row < rows && c + e < C) ? src[row * ld + c + e] : 0.0f;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] *= s;
    *reinterpret_cast<uint4*>(sA + (tid / 8 + 64 * q) * APITCH + (tid % 8) * 8) =
        make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                   pack_bf16x2(x[6], x[7]));
  }
}

// Dual prologue, A side: columns c < r of the contraction come from T_gate,
// columns r .. 2r - 1 from T_up (both fp32 [M][r]), times s, rounded to bf16.
__device__ __forceinline__ void lora_a_tile_dual(const float* la, const float* la2, int r,
                                                 int64_t rows, int64_t m0, int64_t c0, bool vec,
                                                 float s, u16* sA, int tid) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int64_t row = m0 + tid / 8 + 64 * q;
    const int64_t c = c0 + (tid % 8) * 8;
    float x[8];
    if (vec && row < rows && c + 8 <= 2 * r) {  // r % 8 == 0: a chunk lies in one source
      const float* src = c < r ? la + row * r + c : la2 + row * r + (c - r);
      const float4 u = *reinterpret_cast<const float4*>(src);
      const float4 v = *reinterpret_cast<const float4*>(src + 4);
      x[0] = u.x; x[1] = u.y; x[2] = u.z; x[3] = u.w; x[4] = v.x; x[5] = v.y; x[6] = v.z; x[7] = v.w;
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int64_t ce = c + e;
        x[e] = row >= rows || ce >= 2 * r ? 0.0f : ce < r ? la[row * r + ce] : la2[row * r + ce - r];
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] *= s;
    *reinterpret_cast<uint4*>(sA + (tid / 8 + 64 * q) * APITCH + (tid % 8) * 8) =
        make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                   pack_bf16x2(x[6], x[7]));
  }
}

// Many adapters: what the prologue needs of a tile's rows (positions), in LDS.
struct RunTable {
  int start[BM + 1];   // first tile row of each run; start[n] = end of the last
  int id[BM];          // its adapter
  int row[BM];         // each row's token (-1 past M)
  int live[BM];        // whether it has an adapter
  float scale[BM];     // and its scale
};

// Many adapters, A side of the prologue: row t is position m0 + t, its own T
// or U times its own adapter's scale, as two bf16 terms (zeros for a row without
// an adapter or past M).
template <int TMB>
__device__ __forceinline__ void lora_a_tile_multi(const BigArgs& p, const RunTable* rt, int c0, bool save, u16* sHi,
                                                  u16* sLo, int tid) {
#pragma unroll 2
  for (int q = 0; q < TMB; ++q) {
    const int t = tid / 8 + 64 * q, c = c0 + (tid % 8) * 8;
    const int64_t row = rt->row[t];
    const bool in = rt->live[t];
    const float sc = rt->scale[t];
    const float* src = p.la + (in ? row * p.la_ld : 0);
    float x[8];
    // 8 floats at any 4-byte boundary: a row's last ones may reach into the next
    // (not used); where they would reach past the last slice, one by one
    const float* s8 = src + (c < p.r ? c : 0);
    if (s8 + 8 <= p.la + p.la_size) {
      f32x4_t u, v;
      __builtin_memcpy(&u, s8, 16);
      __builtin_memcpy(&v, s8 + 4, 16);
      // (the smallest tile has the registers to load four slices at a time)
#pragma unroll(TMB == 1 ? 4 : 1)
      for (int z = 1; z < p.la_parts; ++z) {
        f32x4_t a, b;
        __builtin_memcpy(&a, s8 + z * p.la_step, 16);
        __builtin_memcpy(&b, s8 + z * p.la_step + 4, 16);
        u += a;
        v += b;
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[e] = u[e];
        x[4 + e] = v[e];
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = src[c + e < p.r ? c + e : p.r - 1];
#pragma unroll 1
      for (int z = 1; z < p.la_parts; ++z) {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] += src[z * p.la_step + (c + e < p.r ? c + e : p.r - 1)];
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      x[e] = in && c + e < p.r ? x[e] : 0.0f;
      if (save && row >= 0 && c + e < p.r) p.t_save[row * p.r + c + e] = x[e];
      x[e] *= sc;
    }
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) split_bf16x2(x[2 * e], x[2 * e + 1], hi[e], lo[e]);
    const int at = (tid / 8 + 64 * q) * APITCH + (tid % 8) * 8;
    *reinterpret_cast<uint4*>(sHi + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    *reinterpret_cast<uint4*>(sLo + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
  }
}

// where the thread's 32 dequantized values go: forward tile [256 n][FPITCH],
// block row tid/2; backward tile [64 n][TPITCH], block (tid/2) = 4 per row
template <int MODE>
__device__ __forceinline__ u16* w_dst(u16* sB, int tid) {
  const int blk = tid >> 1, half = tid & 1;
  if constexpr (MODE == MODE_FWD) return sB + blk * FPITCH + 32 * half;
  else return sB + (blk >> 2) * TPITCH + 64 * (blk & 3) + 32 * half;
}

// Backward tile swizzle: in row n, 16-byte chunk c (8 bf16) is stored at chunk
// c ^ x with x = 2 * bit 4 of c ^ (n & 1), a permutation inside each aligned
// group of four chunks.  A thread stores four consecutive chunks of a row and
// eight threads fill a row, so without it the chunks 16 apart (256 bytes)
// and those of the next row fell on the same LDS banks; with it the 16 lanes
// of one store cycle use 16 distinct 4-bank groups, and the transposing reads
// (4 rows x 4 aligned chunks a half-wave) still cover 64 distinct banks.
__device__ __forceinline__ uint32_t t_swz(uint32_t chunk, uint32_t row) {
  return ((chunk >> 3) & 2u) ^ (row & 1u);
}
// the XOR of the thread's own chunks (all four share it)
template <int MODE>
__device__ __forceinline__ uint32_t w_swz(int tid) {
  if constexpr (MODE == MODE_FWD) return 0u;
  else return t_swz(4u * (uint32_t)(tid & 7), (uint32_t)(tid >> 3));
}

// dequantize the thread's half block and store its 32 bf16 values at dst
__device__ __forceinline__ void store_w(const StageW& st, const float (&mv)[8], uint32_t flip,
                                        uint32_t qor, u16* dst, uint32_t swz) {
  const Table t = make_table(mv, stage_scale(st, qor));
  const uint32_t c[4] = {st.c.x, st.c.y, st.c.z, st.c.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t o[4];
    dequant8(t, c[i], flip, o);
    *reinterpret_cast<uint4*>(dst + 8 * ((uint32_t)i ^ swz)) = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

// LoRA prologue operand of the B side, bf16, in the weight tile's layout:
// forward B [J][r] row j0 + tid/2, columns c0 + 32*(tid%2) .. +32; backward
// A [r][J] row c0 + (tid/2)/4, columns j0 + 64*((tid/2)%4) + 32*(tid%2) .. +32.
template <int MODE>
__device__ __forceinline__ void lora_b_tile(const BigArgs& p, u16* sB, int64_t j0, int64_t c0,
                                            int tid) {
  u16* dst = w_dst<MODE>(sB, tid);
  const int blk = tid >> 1, half = tid & 1;
  int64_t row, col0, rows, cols, ld;
  if constexpr (MODE == MODE_FWD) {
    row = j0 + blk; col0 = c0 + 32 * half; rows = p.J; cols = p.r; ld = p.r;
  } else {
    row = c0 + (blk >> 2); col0 = j0 + 64 * (blk & 3) + 32 * half; rows = p.r; cols = p.J; ld = p.J;
  }
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int64_t c = col0 + 8 * q;
    uint32_t v[4] = {0, 0, 0, 0};
    if (row < rows && c + 8 <= cols && p.lb_vec) {
      const uint4 u = *reinterpret_cast<const uint4*>(p.lb + row * ld + c);
      v[0] = u.x; v[1] = u.y; v[2] = u.z; v[3] = u.w;
    } else if (row < rows) {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (c + e < cols) v[e >> 1] |= (uint32_t)p.lb[row * ld + c + e] << (16 * (e & 1));
    }
    *reinterpret_cast<uint4*>(dst + 8 * ((uint32_t)q ^ w_swz<MODE>(tid))) = make_uint4(v[0], v[1], v[2], v[3]);
  }
}

// Dual prologue, B side, in the forward weight tile's layout: tile row t is
// [B_gate[n] | 0] for a gate row and [0 | B_up[n]] for an up row, n = n0 +
// dual_col(t); the thread fills row tid/2, columns c0 + 32*(tid%2) .. +32.
__device__ __forceinline__ void lora_b_tile_dual(const BigArgs& p, u16* sB, int64_t n0, int64_t c0,
                                                 int tid) {
  u16* dst = sB + (tid >> 1) * FPITCH + 32 * (tid & 1);
  const int t = tid >> 1, src = dual_src(t);
  const int64_t n = n0 + dual_col(t);
  const u16* lb = src ? p.lb2 : p.lb;
  const int64_t lo = src ? p.r : 0;  // this row's nonzero contraction range: lo .. lo + r - 1
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int64_t c = c0 + 32 * (tid & 1) + 8 * q;
    uint32_t v[4] = {0, 0, 0, 0};
    if (n < p.J) {
      if (p.lb_vec && c >= lo && c + 8 <= lo + p.r) {
        const uint4 u = *reinterpret_cast<const uint4*>(lb + n * p.r + (c - lo));
        v[0] = u.x; v[1] = u.y; v[2] = u.z; v[3] = u.w;
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (c + e >= lo && c + e < lo + p.r)
            v[e >> 1] |= (uint32_t)lb[n * p.r + (c + e - lo)] << (16 * (e & 1));
      }
    }
    *reinterpret_cast<uint4*>(dst + 8 * q) = make_uint4(v[0], v[1], v[2], v[3]);
  }
}

// Many adapters, B side: contraction slot c of the stage is rank c0 + c % rp of
// the factor of run u0 + c / rp (rp = 16, 32 or 64 slots a run), in the weight
// tile's layout: chunk q (16 bytes) of the thread's four.  Runs from nruns on
// are not multiplied and columns past J not stored, so those addresses
// are only clamped; ranks past r are zeroed before the LDS store
// (lora_b_ranks), not here, so that nothing waits for the loads.
template <int MODE>
__device__ __forceinline__ int lora_b_slot(int tid, int q) {
  return MODE == MODE_FWD ? 32 * (tid & 1) + 8 * q : tid >> 3;   // forward: 8 ranks of a column; backward: 8 columns of a rank
}
template <int MODE, bool VEC>
__device__ __forceinline__ uint4 load_lora_b_multi(const BigArgs& p, const RunTable* rt, int nruns, int u0, int rp,
                                                   int64_t j0, int c0, int tid, int q) {
  const int blk = tid >> 1, half = tid & 1;
  const int slot = lora_b_slot<MODE>(tid, q);
  const int u = u0 + slot / rp, rank = c0 + slot % rp < p.r ? c0 + slot % rp : 0;
  const u16* fac = p.lb + (int64_t)rt->id[u < nruns ? u : 0] * p.ad_stride;
  const int64_t j1 = MODE == MODE_FWD ? j0 + blk : j0 + 64 * (blk & 3) + 32 * half + 8 * q, j = j1 < p.J ? j1 : 0;
  if constexpr (MODE == MODE_DX) {          // J = K, a multiple of 64
    return load16(fac + rank * p.J + j);
  } else if constexpr (VEC) {               // r a multiple of 8
    return load16(fac + j * p.r + rank);
  } else {                                  // a column's last 8 may reach into the next; the factor's last 8 are gathered
    const u16 *src = fac + j * p.r + rank, *end = fac + p.J * p.r;
    if (src + 8 <= end) return load16_any(src);
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t h = *(src + e < end ? src + e : fac);
      w[e >> 1] = e & 1 ? w[e >> 1] | (h << 16) : h;
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
}
// zeros for the chunk's ranks past r
template <int MODE, bool VEC>
__device__ __forceinline__ uint4 lora_b_ranks(const BigArgs& p, uint4 v, int rp, int c0, int tid, int q) {
  const int n = p.r - c0 - lora_b_slot<MODE>(tid, q) % rp;   // ranks from the chunk's first on
  if (MODE == MODE_DX || VEC) return n > 0 ? v : make_uint4(0, 0, 0, 0);
  uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = n > 2 * i + 1 ? w[i] : n > 2 * i ? w[i] & 0xFFFFu : 0u;
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// ---------------------------------------------------------------------------
// MFMA on one LDS stage: wave (wm, wn) owns rows wm*128 .. +128 and columns
// wn*64 .. +64 of the tile
// ---------------------------------------------------------------------------
template <int MODE>
__device__ __forceinline__ bf16x8_t read_b(const u16* sB, int wn, int b, int ks, int lane) {
  if constexpr (MODE == MODE_FWD) {
    return *reinterpret_cast<const bf16x8_t*>(
        sB + (wn * 64 + b * 32 + (lane & 31)) * FPITCH + ks * 16 + (lane >> 5) * 8);
  } else {
    const int L = lane & 15;
    const int col = wn * 64 + b * 32 + 16 * ((lane >> 4) & 1) + 4 * (L & 3);
    const int row = ks * 16 + 8 * (lane >> 5) + (L >> 2);
    // rows row and row + 4 have the same parity, so the same swizzle
    const int scol = col ^ (8 * (int)t_swz((uint32_t)col >> 3, (uint32_t)row));
    const lds_short* base = (const lds_short*)(sB);
    const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (lds_s16x4*)(base + row * TPITCH + scol));
    const s16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (lds_s16x4*)(base + (row + 4) * TPITCH + scol));
    typedef short s16x8_t __attribute__((ext_vector_type(8)));
    s16x8_t v = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    return __builtin_bit_cast(bf16x8_t, v);
  }
}

template <int MODE, int TMB>
__device__ __forceinline__ void frags(bf16x8_t (&fa)[TMB], bf16x8_t (&fb)[2], const u16* sA,
                                      const u16* sB, int wm, int wn, int ks, int lane) {
#pragma unroll
  for (int a = 0; a < TMB; ++a)
    fa[a] = *reinterpret_cast<const bf16x8_t*>(
        sA + (wm * 32 * TMB + a * 32 + (lane & 31)) * APITCH + ks * 16 + (lane >> 5) * 8);
#pragma unroll
  for (int b = 0; b < 2; ++b) fb[b] = read_b<MODE>(sB, wn, b, ks, lane);
}

template <int MODE>
__device__ __forceinline__ void mma_stage(f32x16_t (&acc)[4][2], const u16* sA, const u16* sB,
                                          int wm, int wn, int lane) {
#pragma unroll
  for (int ks = 0; ks < BK / 16; ++ks) {
    bf16x8_t fa[4], fb[2];
    frags<MODE, 4>(fa, fb, sA, sB, wm, wn, ks, lane);
#pragma unroll
    for (int a = 0; a < 4; ++a)
#pragma unroll
      for (int b = 0; b < 2; ++b)
        acc[a][b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa[a], fb[b], acc[a][b], 0, 0, 0);
  }
}

// One contraction step with the producer work for the next stage woven in:
// for each 16-wide substep ks, the fragments of ks+1 are read while the 8
// MFMAs of ks issue, then a quarter of the next stage is written to the other
// LDS buffer (one 16-byte A chunk and 8 dequantized weights).  Loads of the
// stage after next are woven in too: the A chunk is reloaded right after it
// is stored, the weight block's scale bytes right after its table is built
// and its codes once they are dequantized, so the per-CU address unit sees a
// steady trickle instead of one burst per step.
struct NextLoads {
  const Bufs* bf;
  uint32_t a_base, a_step, a_c0;   // A stage to load into ra (contraction start)
  uint32_t wn, wk, whalf, K;       // weight half block to load into w
  bool wlive;
  uint32_t a_row[4];               // many adapters: byte offsets of the thread's four rows
  uint32_t a_col;                  // and of the stage's column, or COL_PAST behind the contraction's end
};

// many adapters: offsets of a row or a column that reads zeros.  A buffer ends
// 256 rows and 1024 bytes before 2^31 (fits_32bit), and a row has 16 bytes or more
// (a dY of few columns; 8 elements), so any row plus COL_PAST is past the end, and their
// sum does not wrap.
constexpr uint32_t ROW_PAST = 0x80000000u, COL_PAST = 0x7FFFF000u;
static_assert(0x80000000ull - 256 * 16 - 8 * BK * 2 <= COL_PAST && (uint64_t)ROW_PAST + COL_PAST + 8 * 16 <= 0x100000000ull);

template <int MODE, bool MULTI, int TMB>
__device__ __forceinline__ void step_pipelined(f32x16_t (&acc)[TMB][2], const u16* sA,
                                               const u16* sB, int wm, int wn, int lane,
                                               StageA<TMB>& ra, StageW& w,
                                               u16* sA_next, u16* wdst_next, int tid,
                                               const NextLoads& nl, const float (&mv)[8],
                                               uint32_t flip, uint32_t wswz) {
  bf16x8_t fa[2][TMB], fb[2][2];
  frags<MODE, TMB>(fa[0], fb[0], sA, sB, wm, wn, 0, lane);
  const Table t = make_table(mv, stage_scale(w, nl.bf->qor));
  const uint32_t c[4] = {w.c.x, w.c.y, w.c.z, w.c.w};
  {
    // the scale byte and group constant of the weight block after next
    const uint32_t blk = nl.wn * (nl.K / 64) + nl.wk / 64;
    w.q = __builtin_amdgcn_raw_buffer_load_b8(nl.bf->qscale, blk, 0, 0);
    w.d = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(
                                        nl.bf->dscale, nl.wlive ? 4 * (blk >> nl.bf->dshift) : 0xFFFFFFF0u,
                                        0, 0));
  }
#pragma unroll
  for (int ks = 0; ks < 4; ++ks) {
    const int cur = ks & 1;
    if (ks < 3) frags<MODE, TMB>(fa[cur ^ 1], fb[cur ^ 1], sA, sB, wm, wn, ks + 1, lane);
#pragma unroll
    for (int a = 0; a < TMB; ++a)
#pragma unroll
      for (int b = 0; b < 2; ++b)
        acc[a][b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa[cur][a], fb[cur][b], acc[a][b],
                                                            0, 0, 0);
    {
      uint32_t o[4];
      dequant8(t, c[ks], flip, o);
      *reinterpret_cast<uint4*>(wdst_next + 8 * ((uint32_t)ks ^ wswz)) = make_uint4(o[0], o[1], o[2], o[3]);
      if (ks < TMB) {
        *reinterpret_cast<uint4*>(sA_next + (tid / 8 + 64 * ks) * APITCH + (tid % 8) * 8) = ra.v[ks];
        if constexpr (MULTI) ra.v[ks] = bload16(nl.bf->a, nl.a_row[ks] + nl.a_col);
        else ra.v[ks] = bload16(nl.bf->a, nl.a_base + ks * nl.a_step + 2 * nl.a_c0);
      }
    }
    if (ks == 3) w.c = bload16(nl.bf->codes, nl.wn * (nl.K / 2) + nl.wk / 2 + 16 * nl.whalf);
#ifndef QLN_NO_INTERLEAVE
    // keep the dequantization's VALU work between the MFMAs (up to five VALU
    // per MFMA in the forward, six in the backward, as measured best)
    constexpr int ILV_VALU = MODE == MODE_FWD ? 5 : 6;
    if constexpr (TMB == 4)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);          // one MFMA
      __builtin_amdgcn_sched_group_barrier(0x002, ILV_VALU, 0);   // then VALU
      if (i < 6) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);                  // next fragments
      else if (i < 7) __builtin_amdgcn_sched_group_barrier(0x200, 2, 0);             // LDS stores
      else __builtin_amdgcn_sched_group_barrier(0x020, 2, 0);                         // global loads
    }
#endif
    __builtin_amdgcn_sched_barrier(0);
  }
}

// ---------------------------------------------------------------------------
// the kernel
// ---------------------------------------------------------------------------
template <int MODE, int DUAL, bool MULTI = false, bool VEC = true, int TMB = 4>
__global__ __launch_bounds__(NTHREADS, 1) void k_gemm_big(BigArgs p) {
  static_assert(MULTI || TMB == 4, "smaller tiles are for many adapters");
  constexpr int ROWS = 64 * TMB, WROWS = 32 * TMB;   // rows of the tile and of a wave
  constexpr int A_ELEMS = a_elems<TMB>();
  extern __shared__ __attribute__((aligned(16))) u16 smem[];
  u16* sA[2] = {smem, smem + A_ELEMS};
  u16* sB[2] = {smem + 2 * A_ELEMS, smem + 2 * A_ELEMS + b_elems<MODE>()};

  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = wave >> 2, wn = wave & 3;
  const int64_t m0 = (int64_t)blockIdx.x * ROWS;
  // output column tile start (a dual tile covers BN / 2 columns of each weight)
  const int64_t j0 = (int64_t)blockIdx.y * (DUAL ? BN / 2 : BN);

  f32x16_t acc[TMB][2];
#pragma unroll
  for (int a = 0; a < TMB; ++a)
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[a][b][v] = 0.0f;

  // ---- LoRA prologue, many adapters ----
  if constexpr (MULTI) {
    __shared__ RunTable s_runs;
    __shared__ int s_wave[TMB];
    RunTable* rt = &s_runs;
    const int mine = tid < ROWS ? (m0 + tid < p.M ? p.mo.sid[m0 + tid] : p.mo.count) : p.mo.count;
    const int before = tid > 0 && tid < ROWS ? (m0 + tid - 1 < p.M ? p.mo.sid[m0 + tid - 1] : p.mo.count) : -1;
    const bool first = tid < ROWS && mine != before;   // the rows without an adapter are the last run
    const uint64_t bal = __ballot(first);
    if (tid < ROWS && lane == 0) s_wave[wave] = __popcll(bal);
    __syncthreads();
    int at = 0, nall = 0;
#pragma unroll
    for (int i = 0; i < TMB; ++i) {
      if (i < wave) at += s_wave[i];
      nall += s_wave[i];
    }
    if (first) {
      const int k = at + __popcll(bal & (((uint64_t)1 << lane) - 1));
      rt->start[k] = tid;
      rt->id[k] = mine;
    }
    if (tid == 0) rt->start[nall] = ROWS;
    if (tid < ROWS) {
      rt->row[tid] = m0 + tid < p.M ? p.mo.perm[m0 + tid] : -1;
      rt->live[tid] = mine < p.mo.count;
      rt->scale[tid] = mine < p.mo.count ? p.mo.scale[mine] : 0.0f;
    }
    __syncthreads();
    const bool save = p.t_save && blockIdx.y == 0 && blockIdx.z == 0;
    const int rp = p.r <= 16 ? 16 : p.r <= 32 ? 32 : 64, slots = 64 / rp;
    // runs ulo .. uhi - 1: all with an adapter, or with a split contraction
    // this part's share of them (at 56 tokens of 30 adapters, rank 64, the
    // first part alone took 33 us over the factors while the others waited)
    const int nruns = rt->id[nall - 1] == p.mo.count ? nall - 1 : nall;
    const int share = (nruns + slots * (int)gridDim.z - 1) / (slots * (int)gridDim.z) * slots;
    const int ulo = (int)blockIdx.z * share, uhi = min(nruns, ulo + share);
    u16* dst[2] = {w_dst<MODE>(sB[0], tid), w_dst<MODE>(sB[1], tid)};
    for (int c0 = 0; c0 < p.r && (ulo < uhi || save); c0 += BK) {
      // The next group's factors are loaded while one multiplies (two or four
      // groups ahead gained nothing); 256-row tiles have no registers to
      // gather a rank that is no multiple of 8 ahead and do it as they store
      constexpr bool AHEAD = VEC || TMB < 4;
      uint4 v[4];
      auto ahead = [&](int u) {
        if (!AHEAD || u >= uhi) return;
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] = load_lora_b_multi<MODE, VEC>(p, rt, uhi, u, rp, j0, c0, tid, q);
      };
      if (c0 > 0) __syncthreads();   // the last chunk's fragments are read
      lora_a_tile_multi<TMB>(p, rt, c0, save, sA[0], sA[1], tid);
      ahead(ulo);
      int buf = 0;
      for (int u0 = ulo; u0 < uhi; u0 += slots, buf ^= 1) {
        // (the buffer written now was last read before the previous barrier)
        u16* to = buf ? dst[1] : dst[0];
        if constexpr (AHEAD) {
#pragma unroll
          for (int q = 0; q < 4; ++q)
            *reinterpret_cast<uint4*>(to + 8 * ((uint32_t)q ^ w_swz<MODE>(tid))) =
                lora_b_ranks<MODE, VEC>(p, v[q], rp, c0, tid, q);
        } else {
#pragma unroll 1
          for (int q = 0; q < 4; ++q)
            *reinterpret_cast<uint4*>(to + 8 * ((uint32_t)q ^ w_swz<MODE>(tid))) =
                lora_b_ranks<MODE, VEC>(p, load_lora_b_multi<MODE, VEC>(p, rt, uhi, u0, rp, j0, c0, tid, q), rp, c0, tid, q);
        }
        __syncthreads();
        ahead(u0 + slots);
        const u16* sBc = buf ? sB[1] : sB[0];
        for (int s = 0; s < slots && u0 + s < uhi; ++s) {
          const int r0 = __builtin_amdgcn_readfirstlane(rt->start[u0 + s]) - wm * WROWS;
          const int r1 = __builtin_amdgcn_readfirstlane(rt->start[u0 + s + 1]) - wm * WROWS;
          if (r1 <= 0 || r0 >= WROWS) continue;
          const int k0 = s * rp / 16, k1 = k0 + rp / 16;
#pragma unroll
          for (int a = 0; a < TMB; ++a) {
            if (r1 <= 32 * a || r0 >= 32 * a + 32) continue;
#pragma unroll
            for (int b = 0; b < 2; ++b) {
              f32x16_t tmp;
#pragma unroll
              for (int i = 0; i < 16; ++i) tmp[i] = 0.0f;
              for (int ks = k0; ks < k1; ++ks) {
                const int at = (wm * WROWS + a * 32 + (lane & 31)) * APITCH + (ks - k0) * 16 + (lane >> 5) * 8;
                const bf16x8_t fb = read_b<MODE>(sBc, wn, b, ks, lane);
                tmp = __builtin_amdgcn_mfma_f32_32x32x16_bf16(*reinterpret_cast<const bf16x8_t*>(sA[0] + at), fb, tmp, 0, 0, 0);
                tmp = __builtin_amdgcn_mfma_f32_32x32x16_bf16(*reinterpret_cast<const bf16x8_t*>(sA[1] + at), fb, tmp, 0, 0, 0);
              }
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                const int row = 32 * a + (i >> 2) * 8 + (lane >> 5) * 4 + (i & 3);
                acc[a][b][i] += (uint32_t)(row - r0) < (uint32_t)(r1 - r0) ? tmp[i] : 0.0f;
              }
            }
          }
        }
      }
    }
  }

  // ---- LoRA prologue: acc = sum_{c < r} bf16(s la(m, c)) lb(j, c) ----
  if constexpr (!MULTI) {
  for (int64_t c0 = 0; c0 < (DUAL ? 2 * p.r : p.r); c0 += BK) {
    __syncthreads();
    if constexpr (DUAL) {
      lora_a_tile_dual(p.la, p.la2, p.r, p.M, m0, c0, p.la_vec, p.s, sA[0], tid);
      lora_b_tile_dual(p, sB[0], j0, c0, tid);
    } else {
      lora_a_tile(p.la, p.r, p.M, p.r, m0, c0, p.la_vec, p.s, sA[0], tid);
      lora_b_tile<MODE>(p, sB[0], j0, c0, tid);
    }
    __syncthreads();
    mma_stage<MODE>(acc, sA[0], sB[0], wm, wn, lane);
  }
  }
  __syncthreads();

  // ---- main contraction ----
  // While stage kt is multiplied out of LDS buffer kt&1, the other buffer
  // receives stage kt+1 (A tile from registers loaded one step earlier, the
  // weight block dequantized from registers loaded two steps earlier).  Loads
  // of stages past the end read zeros or unused data and are never consumed.
  Bufs bf;
  bf.a = rsrc(p.a, (uint32_t)(p.M * p.lda * 2));
  // a dual tile's wave w produces rows of the gate weight (w even) or the up
  // weight (w odd): the choice is uniform across the wave
  const int wsrc = DUAL ? (__builtin_amdgcn_readfirstlane(wave) & 1) : 0;
  const NF4View& wv = wsrc ? p.w2 : p.w;
  bf.codes = rsrc(wv.codes, (uint32_t)(wv.N * wv.K / 2));
  bf.qscale = rsrc(wv.qscale, wv.fp32_scale ? 0u : (uint32_t)(wv.N * wv.K / 64));
  bf.dscale = rsrc(wv.dscale, (uint32_t)(4 * (wv.fp32_scale ? wv.N * wv.K / 64
                                                             : (wv.N * wv.K / 64 + 255) / 256)));
  bf.qor = wv.fp32_scale ? 0x38u : wv.u8_scale ? QOR_U8 : 0u;   // 0x38: E4M3 code of 1.0
  bf.dshift = wv.fp32_scale ? 0u : 8u;
  // this lane's half of the block table: levels 8p .. 8p + 7 for lane parity p
  const bool odd_lane = tid & 1;
  const uint32_t flip = odd_lane ? 0x08080808u : 0u;
  float mv[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) mv[i] = odd_lane ? wv.lv[8 + i] : wv.lv[i];
  const uint32_t K = (uint32_t)p.w.K;
  // rows past M give offsets past the end (the host checks 32-bit room)
  const uint32_t a_base = (uint32_t)((m0 + tid / 8) * p.lda * 2) + 2 * 8 * (tid % 8);
  const uint32_t a_step = (uint32_t)(64 * p.lda * 2);
  // many adapters: the thread's rows through the sorted order, and columns
  // that read zeros from the contraction's end on
  uint32_t a_row[4] = {0, 0, 0, 0};   // (the first TMB of them)
  // (c0 below this is inside; with C no multiple of 8 the row holds zeros from C to its pitch)
  const uint32_t a_live = (uint32_t)p.C - 8u * (uint32_t)(tid % 8);
  if constexpr (MULTI) {
#pragma unroll
    for (int q = 0; q < TMB; ++q) {
      const int64_t pos = m0 + tid / 8 + 64 * q;
      a_row[q] = (pos < p.M ? (uint32_t)p.mo.perm[pos] * (uint32_t)(p.lda * 2) : ROW_PAST) + 16u * (uint32_t)(tid % 8);
    }
  }
  auto a_col = [&](uint32_t c0) { return (int)c0 < (int)a_live ? 2 * c0 : COL_PAST; };
  auto load_rows = [&](StageA<TMB>& st, uint32_t c0) {
    if constexpr (MULTI) {
#pragma unroll
      for (int q = 0; q < TMB; ++q) st.v[q] = bload16(bf.a, a_row[q] + a_col(c0));
    } else {
      load_a(st, bf, a_base, a_step, c0);
    }
  };
  const int wblk = tid >> 1;
  const uint32_t whalf = (uint32_t)(tid & 1);
  // weight block coordinates of this thread for contraction step kt
  auto w_n = [&](int64_t kt) -> uint32_t {
    if constexpr (DUAL) return (uint32_t)(j0 + dual_col(wblk));
    else if constexpr (MODE == MODE_FWD) return (uint32_t)(j0 + wblk);
    else return (uint32_t)(kt * BK + (wblk >> 2));
  };
  auto w_k = [&](int64_t kt) -> uint32_t {
    if constexpr (MODE == MODE_FWD) return (uint32_t)(kt * BK);
    else return (uint32_t)(j0 + 64 * (wblk & 3));
  };
  u16* wdst0 = w_dst<MODE>(sB[0], tid);
  u16* wdst1 = w_dst<MODE>(sB[1], tid);

  // steps kt0 .. nk - 1 (all of them, or this part's)
  int64_t nk = (p.C + BK - 1) / BK, kt0 = 0;
  if constexpr (MULTI) {
    kt0 = (int64_t)blockIdx.z * p.kt_per;
    nk = min(nk, kt0 + p.kt_per);
  }
  StageA<TMB> ra;
  StageW w0, w1;
  load_rows(ra, (uint32_t)(kt0 * BK));
  load_w(w0, bf, w_n(kt0), w_k(kt0), whalf, K, true);
  store_a(ra, sA[0], tid);
  const uint32_t wswz = w_swz<MODE>(tid);
  store_w(w0, mv, flip, bf.qor, wdst0, wswz);
  load_rows(ra, (uint32_t)((kt0 + 1) * BK));
  load_w(w1, bf, w_n(kt0 + 1), w_k(kt0 + 1), whalf, K, kt0 + 1 < nk);
  load_w(w0, bf, w_n(kt0 + 2), w_k(kt0 + 2), whalf, K, kt0 + 2 < nk);
  __syncthreads();
  // steps are taken in pairs; with an odd count the last pair's second step
  // multiplies a zero weight tile (no early exit: that would make the
  // compiler keep two copies of the accumulators)
  for (int64_t kt = kt0; kt < nk; kt += 2) {
    // buffer 0 holds stage kt; ra = A(kt+1), w1 = W(kt+1), w0 = W(kt+2)
    {
      const NextLoads nl{&bf, a_base, a_step, (uint32_t)((kt + 2) * BK), w_n(kt + 3), w_k(kt + 3), whalf, K,
                         kt + 3 < nk, {a_row[0], a_row[1], a_row[2], a_row[3]}, MULTI ? a_col((uint32_t)((kt + 2) * BK)) : 0u};
      step_pipelined<MODE, MULTI, TMB>(acc, sA[0], sB[0], wm, wn, lane, ra, w1, sA[1], wdst1, tid, nl, mv, flip, wswz);
    }
    __syncthreads();
    // buffer 1 holds stage kt+1; ra = A(kt+2), w0 = W(kt+2), w1 = W(kt+3)
    {
      const NextLoads nl{&bf, a_base, a_step, (uint32_t)((kt + 3) * BK), w_n(kt + 4), w_k(kt + 4), whalf, K,
                         kt + 4 < nk, {a_row[0], a_row[1], a_row[2], a_row[3]}, MULTI ? a_col((uint32_t)((kt + 3) * BK)) : 0u};
      step_pipelined<MODE, MULTI, TMB>(acc, sA[1], sB[1], wm, wn, lane, ra, w0, sA[0], wdst0, tid, nl, mv, flip, wswz);
    }
    __syncthreads();
  }

  // ---- epilogue ----
  // Each wave rounds its 128 x 64 block to bf16 into its own LDS region
  // (lanes l and l^1 hold neighbouring columns of the same rows, so one DPP
  // swap per pair of values gives each lane a packed pair), then writes it
  // back out as 16-byte row segments.  The main loop's last barrier has freed
  // LDS; the regions are disjoint, and a wave's LDS operations complete in
  // order, so no barrier is needed.  With the SwiGLU epilogue the block is
  // 128 x 32: h = silu(g) * u of the wave's gate and up accumulators.
  if constexpr (MULTI) {
    if (gridDim.z > 1) {   // sums of a part of the contraction, in fp32 by position
#pragma unroll
      for (int a = 0; a < TMB; ++a)
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
          for (int v = 0; v < 16; ++v) {
            const int64_t i = m0 + wm * WROWS + a * 32 + (v >> 2) * 8 + (lane >> 5) * 4 + (v & 3);
            const int64_t j = j0 + wn * 64 + b * 32 + (lane & 31);
            if (i < p.M && j < p.J) p.part[((int64_t)blockIdx.z * p.M + i) * p.J + j] = acc[a][b][v];
          }
      return;
    }
  }
  u16* sE = smem + wave * e_elems<TMB>();
  const bool odd = lane & 1;
  constexpr int NBLK = DUAL == DUAL_SWIGLU ? 1 : 2;
#pragma unroll
  for (int a = 0; a < TMB; ++a)
#pragma unroll
    for (int b = 0; b < NBLK; ++b)
#pragma unroll
      for (int v = 0; v < 16; v += 2) {
        float x0 = acc[a][b][v], x1 = acc[a][b][v + 1];
        if constexpr (DUAL == DUAL_SWIGLU) {
          x0 = x0 / (1.0f + __expf(-x0)) * acc[a][1][v];
          x1 = x1 / (1.0f + __expf(-x1)) * acc[a][1][v + 1];
        }
        const float got = dpp_f32<DPP_QUAD_XOR1>(odd ? x0 : x1);
        const int row = a * 32 + (v >> 2) * 8 + (lane >> 5) * 4 + (v & 3) + (odd ? 1 : 0);
        const int col = b * 32 + ((lane & 31) & ~1);
        *reinterpret_cast<uint32_t*>(sE + row * EPITCH + col) =
            odd ? pack_bf16x2(got, x1) : pack_bf16x2(x0, got);
      }
  // read back: 8 lanes per 64-column row (4 per 32-column row)
  constexpr int LPR = NBLK * 4;              // lanes per row
  constexpr int RPI = 64 / LPR;              // rows per instruction
  // (many adapters: the rows' places are read before the first store)
  int32_t orow[WROWS / RPI];
  if constexpr (MULTI) {
#pragma unroll
    for (int q = 0; q < WROWS / RPI; ++q) {
      const int64_t pos = m0 + wm * WROWS + q * RPI + lane / LPR;
      const int32_t row = p.mo.perm[pos < p.M ? pos : m0];
      orow[q] = pos < p.M ? row : -1;
    }
  }
#pragma unroll
  for (int q = 0; q < WROWS / RPI; ++q) {
    const int row = q * RPI + lane / LPR, col = (lane % LPR) * 8;
    const uint4 v = *reinterpret_cast<const uint4*>(sE + row * EPITCH + col);
    int64_t i = m0 + wm * WROWS + row;
    if constexpr (MULTI) i = orow[q] >= 0 ? (int64_t)orow[q] : p.M;
    int64_t j;
    u16* out;
    if constexpr (DUAL == DUAL_SEPARATE) {
      j = j0 + wn * 32 + (col & 31);
      out = col < 32 ? p.out : p.out2;
    } else if constexpr (DUAL == DUAL_SWIGLU) {
      j = j0 + wn * 32 + col;
      out = p.out;
    } else {
      j = j0 + wn * 64 + col;
      out = p.out;
    }
    if (i < p.M) {
      u16* dst = out + i * p.ldo + j;
      if (MULTI && j + 8 <= p.J) {
        store16_any(dst, v);   // (rows of any N: 2-byte stores took a third of a call with N = 20777, K = 448)
      } else if (p.out_vec && j + 8 <= p.J) {
        *reinterpret_cast<uint4*>(dst) = v;
      } else {
        const uint32_t w4[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (j + e < p.J) dst[e] = (u16)(w4[e >> 1] >> (16 * (e & 1)));
      }
    }
  }
}

static bool vec_ok(const void* ptr, int64_t ld) {
  return ((uintptr_t)ptr % 16 == 0) && (ld % 8 == 0);
}

template <int MODE, int DUAL = DUAL_NONE, bool MULTI = false, bool VEC = true, int TMB = 4>
static hipError_t launch(const BigArgs& p, hipStream_t st, int splits = 1) {
  const hipError_t e =
      set_dynamic_lds((const void*)k_gemm_big<MODE, DUAL, MULTI, VEC, TMB>, (int)lds_bytes<MODE, TMB>());
  if (e != hipSuccess) return e;
  const int64_t bn = DUAL ? BN / 2 : BN;
  dim3 grid((unsigned)((p.M + 64 * TMB - 1) / (64 * TMB)), (unsigned)((p.J + bn - 1) / bn), (unsigned)splits);
  const size_t lds = lds_bytes<MODE, TMB>();
  hipLaunchKernelGGL((k_gemm_big<MODE, DUAL, MULTI, VEC, TMB>), grid, dim3(NTHREADS), lds, st, p);
  return hipGetLastError();
}

// Many adapters, split contraction: the parts' sums of a position in order,
// rounded to bf16, written to the position's row.  Four columns a thread.
__global__ __launch_bounds__(256) void k_join(const float* __restrict__ part, int splits, int64_t M, int64_t J,
                                              const int32_t* __restrict__ perm, u16* __restrict__ out) {
  const int64_t pos = blockIdx.y, row = perm[pos], n = M * J;
  const int64_t j0 = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (j0 >= J) return;
  const float* src = part + pos * J + j0;
  if (j0 + 4 <= J) {   // (16 and 8 bytes at any boundary: J need not be a multiple of 4)
    float s[4];
    __builtin_memcpy(s, src, 16);
    for (int z = 1; z < splits; ++z) {
      float x[4];
      __builtin_memcpy(x, src + z * n, 16);
#pragma unroll
      for (int e = 0; e < 4; ++e) s[e] += x[e];
    }
    const uint32_t w[2] = {pack_bf16x2(s[0], s[1]), pack_bf16x2(s[2], s[3])};
    __builtin_memcpy(out + row * J + j0, w, 8);
  } else {
    for (int64_t e = 0; e < 4 && j0 + e < J; ++e) {
      float s = src[e];
      for (int z = 1; z < splits; ++z) s += src[z * n + e];
      out[row * J + j0 + e] = f32_to_bf16(s);
    }
  }
}

// Tile rows (64 TMB) and parts of the contraction for M x J outputs over C:
// the least of rounds of workgroups x steps x step time, plus joining the
// parts' sums (8 bytes an output and part at 4 TB/s).  A step of 64 (MI355X,
// 256 compute units, r = 16, shapes of 32 to 4096 tokens on 4096^2 to 28672x8192
// weights) takes 0.85, 1.0, 1.3 us for 64, 128 and 256 rows with few workgroups,
// 1.1, 1.4, 1.95 us with one on every compute unit.  A choice, not a
// prediction: the constant 4 us stands for a prologue that grows with the runs
// of a tile, the rank and T's slices, so a kernel of few steps takes up to 2.5
// times the sum (56 tokens of 30 adapters, r = 64: 32 us for 19; 4001 tokens,
// 344-369 for 339).  That cancels where tiles and parts are compared: of 20 calls
// timed at every tile and split (r = 3 to 128, up to 100 adapters) 15 had the
// best, 5 were 3-8% over it, three of them at 200 tokens.  Few rows take small
// tiles (64 x 28672x8192: 95 us against 126 us with 256-row tiles), few tiles
// split (64 x 8192^2: 50 us in 8 parts, 128 us whole).
struct MultiPlan {
  int tmb, splits, kt_per;
};
static MultiPlan multi_plan(int64_t M, int64_t J, int64_t C) {
  const int64_t cus = 256, steps = (C + BK - 1) / BK, jt = (J + BN - 1) / BN;
  MultiPlan best{4, 1, (int)steps + 1};
  double cost = 1e30;
  for (int tmb = 4; tmb >= 1; tmb /= 2) {
    const double alone = tmb == 4 ? 1.3 : tmb == 2 ? 1.0 : 0.85, crowd = tmb == 4 ? 0.65 : tmb == 2 ? 0.4 : 0.25;
    const int64_t tiles = (M + 64 * tmb - 1) / (64 * tmb) * jt;
    for (int s = 1; s <= 16; ++s) {
      const int64_t per = ((steps + s - 1) / s + 1) / 2 * 2, parts = (steps + per - 1) / per;
      if (s > 1 && (parts != s || per < 4 || M > 65535)) continue;
      const int64_t wgs = tiles * parts;
      const double step_us = alone + crowd * std::min(1.0, (double)wgs / (double)cus);
      const double us = (double)((wgs + cus - 1) / cus) * ((double)per * step_us + 4.0) +
                        (parts > 1 ? 5.0 + (double)parts * (double)M * (double)J * 8.0 / 4.0e6 : 0.0);
      if (us < cost) {
        cost = us;
        best = MultiPlan{tmb, (int)parts, (int)per};
      }
    }
  }
  return best;
}

template <int MODE>
static hipError_t launch_multi(BigArgs& p, float* ws, hipStream_t st) {
  const MultiPlan pl = multi_plan(p.M, p.J, p.C);
  p.part = ws;
  p.kt_per = pl.kt_per;
  hipError_t e = hipSuccess;
  bool vec = true;
  if constexpr (MODE == MODE_FWD) {
    vec = p.lb_vec;
    if (!vec)
      e = pl.tmb == 4   ? launch<MODE, DUAL_NONE, true, false, 4>(p, st, pl.splits)
          : pl.tmb == 2 ? launch<MODE, DUAL_NONE, true, false, 2>(p, st, pl.splits)
                        : launch<MODE, DUAL_NONE, true, false, 1>(p, st, pl.splits);
  }
  if (vec)
    e = pl.tmb == 4   ? launch<MODE, DUAL_NONE, true, true, 4>(p, st, pl.splits)
        : pl.tmb == 2 ? launch<MODE, DUAL_NONE, true, true, 2>(p, st, pl.splits)
                      : launch<MODE, DUAL_NONE, true, true, 1>(p, st, pl.splits);
  if (e != hipSuccess || pl.splits == 1) return e;
  const dim3 grid((unsigned)((p.J + 1023) / 1024), (unsigned)p.M);
  hipLaunchKernelGGL(k_join, grid, dim3(256), 0, st, ws, pl.splits, p.M, p.J, p.mo.perm, p.out);
  return hipGetLastError();
}

}  // namespace big

// The buffer-load kernels need 16-byte aligned activation rows and 32-bit
// byte offsets (with room for the tile overrun); other shapes take the
// tile-128 kernels of gemm.hip.
static bool fits_32bit(int64_t M, int64_t lda, const NF4View& w) {
  const int64_t lim = (int64_t)1 << 31;
  return (M + big::BM) * lda * 2 + 8 * big::BK * 2 < lim && (w.N + big::BN) * w.K / 2 < lim &&
         w.N * w.K / 64 < lim && 4 * scale_d_count(w) < lim;
}

hipError_t launch_fwd_main(const NF4View& w, const u16* X, int64_t M, const float* T,
                           const u16* B, int r, float s, u16* Y, hipStream_t st) {
  if (!big::vec_ok(X, w.K) || !fits_32bit(M, w.K, w))
    return launch_fwd_generic(w, X, M, T, B, r, s, Y, st);
  big::BigArgs p{};
  p.a = X; p.lda = w.K; p.a_vec = big::vec_ok(X, w.K);
  p.w = w;
  p.M = M; p.J = w.N; p.C = w.K;
  p.la = T; p.lb = B; p.r = r; p.s = s;
  p.la_vec = big::vec_ok(T, r * 2); p.lb_vec = big::vec_ok(B, r);
  p.out = Y; p.ldo = w.N; p.out_vec = big::vec_ok(Y, w.N);
  return big::launch<big::MODE_FWD>(p, st);
}

// Gate and up projections of one X in one kernel (epilogue: 1 = both outputs,
// 2 = bf16(silu(g) * u) into Yg).  M is cut into slices whose X fits the
// 32-bit buffer offsets.
hipError_t launch_fwd_dual(const NF4View& wg, const NF4View& wu, const u16* X, int64_t M,
                           const float* Tg, const float* Tu, const u16* Bg, const u16* Bu, int r,
                           float s, int epilogue, u16* Yg, u16* Yu, hipStream_t st) {
  const int64_t N = wg.N, K = wg.K;
  const int64_t lim = (int64_t)1 << 31;
  if ((N + big::BN) * K / 2 >= lim || N * K / 64 >= lim || 4 * scale_d_count(wg) >= lim ||
      4 * scale_d_count(wu) >= lim)
    return hipErrorInvalidValue;
  int64_t mstep = (lim - 8 * big::BK * 2) / (K * 2) - big::BM;
  mstep = mstep / big::BM * big::BM;
  if (mstep < big::BM) return hipErrorInvalidValue;
  for (int64_t m = 0; m < M; m += mstep) {
    const int64_t mc = std::min(mstep, M - m);
    big::BigArgs p{};
    p.a = X + m * K; p.lda = K; p.a_vec = true;
    p.w = wg; p.w2 = wu;
    p.M = mc; p.J = N; p.C = K;
    p.la = Tg + m * r; p.la2 = Tu + m * r;
    p.lb = Bg; p.lb2 = Bu; p.r = r; p.s = s;
    p.la_vec = r % 8 == 0 && big::vec_ok(Tg, 8) && big::vec_ok(Tu, 8);
    p.lb_vec = big::vec_ok(Bg, r) && big::vec_ok(Bu, r);
    p.out = Yg + m * N; p.out2 = epilogue == 1 ? Yu + m * N : nullptr; p.ldo = N;
    p.out_vec = big::vec_ok(Yg, N) && (epilogue != 1 || big::vec_ok(Yu, N));
    const hipError_t e = epilogue == 1 ? big::launch<big::MODE_FWD, big::DUAL_SEPARATE>(p, st)
                                       : big::launch<big::MODE_FWD, big::DUAL_SWIGLU>(p, st);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_dx_main(const NF4View& w, const u16* dY, int64_t M, const float* U,
                          const u16* A, int r, float s, u16* dX, hipStream_t st) {
  if (!big::vec_ok(dY, w.N) || !fits_32bit(M, w.N, w) || (w.N + big::BK) * w.K / 2 >= ((int64_t)1 << 31))
    return launch_dx_generic(w, dY, M, U, A, r, s, dX, st);
  big::BigArgs p{};
  p.a = dY; p.lda = w.N; p.a_vec = big::vec_ok(dY, w.N);
  p.w = w;
  p.M = M; p.J = w.K; p.C = w.N;
  p.la = U; p.lb = A; p.r = r; p.s = s;
  p.la_vec = big::vec_ok(U, r * 2); p.lb_vec = big::vec_ok(A, w.K);
  p.out = dX; p.ldo = w.K; p.out_vec = big::vec_ok(dX, w.K);
  return big::launch<big::MODE_DX>(p, st);
}

// fp32 elements of the split sums (0 if the contraction is not split)
int64_t multi_main_elems(int64_t M, int64_t J, int64_t C) {
  const big::MultiPlan pl = big::multi_plan(M, J, C);
  return pl.splits > 1 ? pl.splits * M * J : 0;
}

void multi_tiles(int64_t M, int64_t J, int64_t C, int* rows, int* parts) {
  const big::MultiPlan pl = big::multi_plan(M, J, C);
  *rows = 64 * pl.tmb;
  *parts = pl.splits;
}

bool multi_dx_fits(const u16* dY, int64_t ldy, int64_t M, const NF4View& w) {
  return big::vec_ok(dY, ldy) && fits_32bit(M, ldy, w) && (w.N + big::BK) * w.K / 2 < ((int64_t)1 << 31);
}

// whether launch_multi_fwd takes a shape itself
bool multi_fwd_fits(const u16* X, int64_t M, const NF4View& w) { return big::vec_ok(X, w.K) && fits_32bit(M, w.K, w); }

// Many adapters: the same two kernels over the sorted order.
hipError_t launch_multi_fwd(const MultiOrder& mo, const NF4View& w, const u16* X, int64_t M, float* T,
                            const MultiParts& tp, const u16* B, int r, float* ws, u16* Y, hipStream_t st) {
  if (!multi_fwd_fits(X, M, w)) return launch_multi_fwd_generic(mo, w, X, M, T, B, r, Y, st);
  big::BigArgs p{};
  p.a = X; p.lda = w.K; p.a_vec = true;
  p.w = w;
  p.M = M; p.J = w.N; p.C = w.K;
  p.la = T; p.la_parts = 1; p.la_ld = r; p.la_size = M * r; p.lb = B; p.r = r; p.lb_vec = big::vec_ok(B, r);
  if (tp.slices) {   // T comes as slices: add them up here and keep the sums
    p.la = tp.part; p.la_parts = tp.slices; p.la_step = p.la_size = tp.step; p.la_ld = tp.ld; p.t_save = T;
  }
  p.out = Y; p.ldo = w.N; p.out_vec = big::vec_ok(Y, w.N);
  p.mo = mo; p.ad_stride = w.N * r;
  return big::launch_multi<big::MODE_FWD>(p, ws, st);
}

hipError_t launch_multi_dx(const MultiOrder& mo, const NF4View& w, const u16* dY, int64_t ldy, int64_t M,
                           const float* U, const u16* A, int r, float* ws, u16* dX, hipStream_t st) {
  if (!multi_dx_fits(dY, ldy, M, w))
    return launch_multi_dx_generic(mo, w, dY, ldy, M, U, A, r, dX, st);
  big::BigArgs p{};
  p.a = dY; p.lda = ldy; p.a_vec = true;
  p.w = w;
  p.M = M; p.J = w.K; p.C = w.N;
  p.la = U; p.la_parts = 1; p.la_ld = r; p.la_size = M * r; p.lb = A; p.r = r; p.lb_vec = true;
  p.out = dX; p.ldo = w.K; p.out_vec = big::vec_ok(dX, w.K);
  p.mo = mo; p.ad_stride = (int64_t)r * w.K;
  return big::launch_multi<big::MODE_DX>(p, ws, st);
}

}  // namespace qln
