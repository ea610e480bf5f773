// optim8.hip -- AdamW over a list of tensors with both moments in 8 bits.
//
// Ultralytics glossary "QLoRA", "How QLoRA works" (paged-optimizer bullet) and
// vnread "Grokking QLoRA", "Paged Optimizers": the adapters' optimizer state
// is what grows with every adapter trained.  The step of optim.hip with the
// moments kept as OCP E4M3 codes, one fp32 scale per block of 256 elements:
//
//   m = E4M3(cm) dm,   u = E4M3(cu) du          (u is the root of the variance v)
//   m' = b1 m + (1 - b1) g,   u' = sqrt(b2 u^2 + (1 - b2) g^2)
//   theta' = theta (1 - lr wd) - (lr / (1 - b1^t)) m' / (u' / sqrt(1 - b2^t) + eps)
//   dm' = max|m'| / 448,   cm' = E4M3 nearest(m' 448 / max|m'|)
//   du' = max u' / 448,    cu' = E4M3 stochastic(u' 448 / max u'), at least 1 if u' > 0
// (a block with max|m'| < 2^-117 has dm' = cm' = 0; an element whose m' or u'
// is not finite has the NaN code there and counts in no maximum, so a gradient
// of NaN or infinity stays its own element's: blocks cross rows, and adapters),
//
// in fp32, every operation rounded on its own (this file is compiled without
// contraction, so the stored bits are defined by these lines).  The update
// takes m' and u' before they are rounded to 8 bits.
//   u, not v, is stored: its range is half of v's in octaves, and E4M3 holds
// 2^-18 .. 1 of a block's largest.  It never becomes 0 while u' > 0, so a
// denominator cannot fall to eps by underflow.
//   u is rounded stochastically: with b2 = 0.999 it moves by at most 0.05% a
// step when gradients shrink, against E4M3 steps of 6-12%, so nearest would
// round the move away every time (simulated: gradients of half a block's
// elements falling to 1/100 leave u 7.8 times too large 3500 steps later,
// against 0.91 times).  The rounding bits are a hash of a seed and the
// element's place in the list, so a step can be repeated bit for bit.
//
// A pure stream: 10 bytes per parameter (18 with a master copy) and 16 per
// block, bound by HBM.  32 lanes hold a block, 8 elements a lane, so a block's
// largest values are one reduction over half a wave; one workgroup handles 8
// blocks of one tensor, and a launch covers up to MAXT tensors.  70.8M parameters
// in 60 tensors: 146 us in two launches, 4.9 TB/s (a large copy: 5.2); 8.0M
// with masters in 32 tensors: 24.9 us; 0.5M in 8: 5.4 us, one chain of loads,
// reduction and stores in one round of workgroups (an empty launch: 1.5).
#include <hip/hip_runtime.h>

#include <cmath>

#include "common.h"
#include "device.h"

namespace qln {
namespace opt8 {

constexpr int MAXT = 48;              // the table stays within 4 KB of kernel arguments
constexpr int NTHREADS = 256;
constexpr int EPT = 8;
constexpr int BLK = 256;
constexpr int64_t CHUNK = NTHREADS * EPT;
constexpr int64_t MAX_CHUNKS = ((int64_t)1 << 24) - 1;   // a launch has fewer than 2^32 threads
static_assert(kAdamw8MaxNumel / CHUNK <= MAX_CHUNKS, "the largest tensor is one launch");
// A block of first moments that all lie under this is stored as zeros: its
// scale would be a subnormal and 448 over its largest infinite.  Gradients of
// zero, as of an adapter that no token names, bring it there in some 700
// steps.  (u is the root of an fp32 number: at least 2^-74.5, or zero.)
constexpr float LEAST = 0x1p-117f;

struct Tensor {
  u16* p; const u16* g; uint8_t* m; uint8_t* u; float* sm; float* su; float* w; int64_t n;
};

struct Args {
  Tensor t[MAXT];
  uint32_t chunk0[MAXT + 1];   // first chunk of each tensor; chunk0[count] = total
  uint32_t blk0[MAXT];         // first block of each tensor in the whole list
  int count;
  float b1, c1, b2, c2;        // c = 1 - b
  float decay, step_size, inv_sqrt_bc2, eps;
  uint32_t key;
};
static_assert(sizeof(Args) <= 4096, "kernel arguments");

// lowbias32: a published 32-bit integer mix
__host__ __device__ __forceinline__ uint32_t mix32(uint32_t x) {
  x ^= x >> 16;
  x *= 0x7feb352du;
  x ^= x >> 15;
  x *= 0x846ca68bu;
  return x ^ (x >> 16);
}

// max over each aligned group of 32 lanes
__device__ __forceinline__ float max32(float x) {
  x = max16(x);
  const uint32_t b = __float_as_uint(x);
  const auto s = __builtin_amdgcn_permlane16_swap(b, b, false, false);
  return fmaxf(__uint_as_float(s[0]), __uint_as_float(s[1]));
}

// x in [0, 448] to an E4M3 code: low20 is added below the last kept bit and
// carries; under 2^-6 (the subnormal codes) x + 2^-6 has the spacing wanted
__device__ __forceinline__ uint32_t e4m3_carry(float x, uint32_t low20) {
  const bool small = x < 0x1p-6f;
  const uint32_t b = __float_as_uint(small ? x + 0x1p-6f : x);
  const int c = (int)((b + low20) >> 20) - (small ? 121 << 3 : 120 << 3);
  const int k = c < 1 ? 1 : c > 126 ? 126 : c;
  return x > 0.0f ? (uint32_t)k : 0u;
}

template <bool MASTER>
__global__ __launch_bounds__(NTHREADS) void k_adamw8(Args a) {
  const uint32_t c = blockIdx.x;
  int lo = 0, hi = a.count;   // the chunk's tensor: the last with chunk0 <= c
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (c >= a.chunk0[mid]) lo = mid;
    else hi = mid;
  }
  const Tensor& T = a.t[lo];
  const int64_t e0 = (int64_t)(c - a.chunk0[lo]) * CHUNK + (int64_t)threadIdx.x * EPT;
  const int64_t left = T.n - e0;   // elements of this lane (all lanes stay for the reductions)
  const bool whole = left >= EPT;
  const int64_t blk = e0 / BLK;

  uint32_t pw[4] = {0, 0, 0, 0}, gw[4] = {0, 0, 0, 0}, mw[2] = {0, 0}, uw[2] = {0, 0};
  float th[EPT];
  float dm = 0.0f, du = 0.0f;
  if (left > 0) {
    dm = T.sm[blk];
    du = T.su[blk];
  }
  if (whole) {
    const uint4 pv = *reinterpret_cast<const uint4*>(T.p + e0), gv = *reinterpret_cast<const uint4*>(T.g + e0);
    const uint2 mv = *reinterpret_cast<const uint2*>(T.m + e0), uv = *reinterpret_cast<const uint2*>(T.u + e0);
    pw[0] = pv.x; pw[1] = pv.y; pw[2] = pv.z; pw[3] = pv.w;
    gw[0] = gv.x; gw[1] = gv.y; gw[2] = gv.z; gw[3] = gv.w;
    mw[0] = mv.x; mw[1] = mv.y;
    uw[0] = uv.x; uw[1] = uv.y;
    if constexpr (MASTER) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const f32x4_t v = *reinterpret_cast<const f32x4_t*>(T.w + e0 + 4 * h);
#pragma unroll
        for (int e = 0; e < 4; ++e) th[4 * h + e] = v[e];
      }
    }
  } else {   // the tensor's ragged end: elements past it read as zeros
#pragma unroll
    for (int e = 0; e < EPT; ++e) {
      if constexpr (MASTER) th[e] = 0.0f;
      if (e >= left) continue;
      pw[e >> 1] |= (uint32_t)T.p[e0 + e] << (16 * (e & 1));
      gw[e >> 1] |= (uint32_t)T.g[e0 + e] << (16 * (e & 1));
      mw[e >> 2] |= (uint32_t)T.m[e0 + e] << (8 * (e & 3));
      uw[e >> 2] |= (uint32_t)T.u[e0 + e] << (8 * (e & 3));
      if constexpr (MASTER) th[e] = T.w[e0 + e];
    }
  }

  constexpr float INF = __builtin_inff();
  float m[EPT], u[EPT], am = 0.0f, au = 0.0f;
  auto grad = [&](int e) { return __uint_as_float(e & 1 ? gw[e >> 1] & 0xFFFF0000u : gw[e >> 1] << 16); };
  auto root = [&](int e) { return __builtin_amdgcn_cvt_f32_fp8((int)(uw[e >> 2] >> (8 * (e & 3))), 0) * du; };
  uint32_t top = 0;   // of the variances' bits (not negative): infinity and NaN are the largest
#pragma unroll
  for (int e = 0; e < EPT; ++e) {
    const float g = grad(e), uo = root(e);
    if constexpr (!MASTER) th[e] = __uint_as_float(e & 1 ? pw[e >> 1] & 0xFFFF0000u : pw[e >> 1] << 16);
    m[e] = a.b1 * (__builtin_amdgcn_cvt_f32_fp8((int)(mw[e >> 2] >> (8 * (e & 3))), 0) * dm) + a.c1 * g;
    const float v = a.b2 * (uo * uo) + a.c2 * (g * g);
    top = max(top, __float_as_uint(v));
    u[e] = __builtin_sqrtf(v);
    am = fmaxf(am, fabsf(m[e]));
  }
  au = __builtin_sqrtf(__uint_as_float(top));
  // whether an m or v of this lane is not finite (fmaxf drops a NaN; m's come from a
  // gradient's, which v has too, or from a code): found by the lane (by the element 70.8M
  // parameters took 178 us for 166)
  auto nan_code = [](uint32_t w) { return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u; };
  const bool odd = !(au < INF) || !(am < INF) || !(dm < INF) || (nan_code(mw[0]) | nan_code(mw[1])) != 0;
  if (odd) {
    am = au = 0.0f;
#pragma unroll
    for (int e = 0; e < EPT; ++e) {
      if (!(u[e] < INF)) {   // g over 2^64: the same root of numbers 2^64 times smaller
        const float g = grad(e) * 0x1p-64f, uo = root(e) * 0x1p-64f;
        u[e] = __builtin_sqrtf(a.b2 * (uo * uo) + a.c2 * (g * g)) * 0x1p64f;
      }
      if (fabsf(m[e]) < INF) am = fmaxf(am, fabsf(m[e]));
      if (u[e] < INF) au = fmaxf(au, u[e]);
    }
  }
#pragma unroll
  for (int e = 0; e < EPT; ++e) th[e] = th[e] * a.decay - a.step_size * (m[e] / (u[e] * a.inv_sqrt_bc2 + a.eps));
  am = max32(am);
  au = max32(au);
  am = am >= LEAST ? am : 0.0f;
  const float im = am > 0.0f ? 448.0f / am : 0.0f, iu = au > 0.0f ? 448.0f / au : 0.0f;

  const uint32_t pair = (a.blk0[lo] * (uint32_t)BLK + (uint32_t)e0) >> 1;
  uint32_t om[2] = {0, 0}, ou[2] = {0, 0}, op[4];
#pragma unroll
  for (int e = 0; e < EPT; e += 2) {
    const uint32_t h = mix32((pair + (uint32_t)e / 2) ^ a.key);
    const uint32_t both = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(m[e] * im, m[e + 1] * im, 0, false) & 0xFFFFu;
    om[e >> 2] |= both << (8 * (e & 3));
    ou[e >> 2] |= e4m3_carry(u[e] * iu, (h & 0xFFFFu) * 16u + 8u) << (8 * (e & 3));
    ou[e >> 2] |= e4m3_carry(u[e + 1] * iu, (h >> 16) * 16u + 8u) << (8 * ((e + 1) & 3));
    op[e >> 1] = pack_bf16x2(th[e], th[e + 1]);
  }

  if (odd) {   // 0x7F, the NaN code, over what is not finite
#pragma unroll
    for (int e = 0; e < EPT; ++e) {
      const int at = 8 * (e & 3);
      if (!(fabsf(m[e]) < INF)) om[e >> 2] = (om[e >> 2] & ~(0x80u << at)) | 0x7Fu << at;
      if (!(u[e] < INF)) ou[e >> 2] |= 0x7Fu << at;
    }
  }
  if (left > 0 && e0 % BLK == 0) {
    T.sm[blk] = am * (1.0f / 448.0f);
    T.su[blk] = au * (1.0f / 448.0f);
  }
  if (whole) {
    *reinterpret_cast<uint4*>(T.p + e0) = make_uint4(op[0], op[1], op[2], op[3]);
    *reinterpret_cast<uint2*>(T.m + e0) = make_uint2(om[0], om[1]);
    *reinterpret_cast<uint2*>(T.u + e0) = make_uint2(ou[0], ou[1]);
    if constexpr (MASTER) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        *reinterpret_cast<f32x4_t*>(T.w + e0 + 4 * h) = f32x4_t{th[4 * h], th[4 * h + 1], th[4 * h + 2], th[4 * h + 3]};
    }
  } else {
#pragma unroll
    for (int e = 0; e < EPT; ++e) {
      if (e >= left) continue;
      T.p[e0 + e] = (u16)(op[e >> 1] >> (16 * (e & 1)));
      T.m[e0 + e] = (uint8_t)(om[e >> 2] >> (8 * (e & 3)));
      T.u[e0 + e] = (uint8_t)(ou[e >> 2] >> (8 * (e & 3)));
      if constexpr (MASTER) T.w[e0 + e] = th[e];
    }
  }
}

}  // namespace opt8

// Tensors with and without a master copy go to separate launches of up to
// MAXT tensors; a tensor's place in the list (its rounding bits) counts every
// tensor in blocks, whichever launch takes it.
hipError_t launch_adamw8(const Adamw8Tensor* ts, int count, double lr, double b1, double b2, double eps, double wd,
                         int64_t step, uint32_t seed, hipStream_t st) {
  opt8::Args a{};
  a.b1 = (float)b1; a.c1 = (float)(1.0 - b1); a.b2 = (float)b2; a.c2 = (float)(1.0 - b2);
  a.decay = (float)(1.0 - lr * wd);
  a.step_size = (float)(lr / (1.0 - std::pow(b1, (double)step)));
  a.inv_sqrt_bc2 = (float)(1.0 / std::sqrt(1.0 - std::pow(b2, (double)step)));
  a.eps = (float)eps;
  a.key = opt8::mix32(seed);
  for (int master = 0; master < 2; ++master) {
    a.count = 0;
    int64_t chunks = 0;
    uint64_t blocks = 0;
    auto flush = [&]() -> hipError_t {
      if (a.count == 0) return hipSuccess;
      a.chunk0[a.count] = (uint32_t)chunks;
      if (master)
        hipLaunchKernelGGL(opt8::k_adamw8<true>, dim3((unsigned)chunks), dim3(opt8::NTHREADS), 0, st, a);
      else
        hipLaunchKernelGGL(opt8::k_adamw8<false>, dim3((unsigned)chunks), dim3(opt8::NTHREADS), 0, st, a);
      a.count = 0;
      chunks = 0;
      return hipGetLastError();
    };
    for (int i = 0; i < count; ++i) {
      const Adamw8Tensor& t = ts[i];
      const uint64_t first = blocks;
      blocks += (uint64_t)((t.n + opt8::BLK - 1) / opt8::BLK);
      if (t.n <= 0 || (t.master != nullptr) != (master == 1)) continue;
      const int64_t nc = (t.n + opt8::CHUNK - 1) / opt8::CHUNK;
      if (a.count == opt8::MAXT || chunks + nc > opt8::MAX_CHUNKS) {
        const hipError_t e = flush();
        if (e != hipSuccess) return e;
      }
      a.t[a.count] = opt8::Tensor{t.param, t.grad, t.m, t.u, t.sm, t.su, t.master, t.n};
      a.chunk0[a.count] = (uint32_t)chunks;
      a.blk0[a.count] = (uint32_t)first;
      ++a.count;
      chunks += nc;
    }
    const hipError_t e = flush();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace qln
