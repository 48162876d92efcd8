// state_ops.cuh -- AdamW over many tensors with its moments in 32 or 8 bits,
// the gradient norm that clips it, and the conversion of moments between the
// two forms.  All are HBM-bound streams over lists of tensors.
//
//   adamw32_kernel     one AdamW step with fp32 moments; fp32 parameters,
//                      optionally with a bf16 working copy, or bf16 ones.
//   adamw8_kernel      the same step with 8-bit codes, one fp32 scale per 256
//                      elements.
//   grad_norm_kernel   norm = sqrt(sum g^2) over a list and the clip factor
//                      min(1, max_norm / (norm + 1e-6)), one launch.
//   state8_kernel      moments (fp32 or bf16) -> codes and scales, and back.
//
// Measured on 134M elements in one tensor, us and share of a plain copy's
// 6.54 TB/s (a share above 1 is a better mix of reads and writes than the
// copy's):
//
//   adamw32   fp32 parameters, bf16 gradients (26 B/element)     515   1.04
//             ... with a copy (28)                               554   1.04
//             bf16 parameters (22)                               437   1.03
//             ... stochastic                                     467   0.97
//   adamw8    fp32 parameters, bf16 gradients (14)               283   1.02
//             ... with a copy (16)                               324   1.02
//             ... with a copy, stochastic                        326   1.01
//             ... stochastic                                     307   0.94
//             bf16 parameters (10)                               244   0.85
//             ... stochastic                                     324   0.64
//   state8    pack from fp32 (10 for both moments)               206   1.00
//             pack from bf16 (6)                                 188   0.66
//             unpack to bf16 (6)                                 131   0.94
//   norm      fp32 gradients (4)                                  83   0.99
//             bf16 gradients (2), call after call                 42   0.97
//
// The pack from bf16 runs the fp32 one's instructions and more (29 an element)
// on 60 % of its bytes: 58 % of the issue slots used, and a warp that computes
// has no loads in flight.
// The 8-bit step on bf16 parameters and the stochastic ones are bound by
// instruction issue, not by memory (52 to 72 instructions an element, 78 % of
// the issue slots used, the integer pipe the busiest): two codes an element
// cost two roots, their rounding and its check, and a hash when stochastic.
//
// The 8-bit form.  256 consecutive elements of one tensor are a block (one
// warp, 8 elements per lane); codes keep the square root of the magnitude:
//
//   first moment    m = c |c| s,           c = -127 .. 127, s = max|m| / 127^2
//   second moment   sqrt(v) = (c + 1)^2 s, c = 0 .. 255,    s = max sqrt(v) / 256^2
//
// so a code c resolves its value to 1/c of it, over a range of 127^2 in m and
// 256^4 in v within one block.  Codes linear in the value would lose the small
// second moments; a second moment rounded to zero would divide by eps, so
// there is no zero among its codes.  A code is floor(y + u) of the real-valued
// code y: u = 1/2 rounds to nearest; u = (h + 1/2) / 2^16 with a hashed 16-bit
// h rounds up with the probability of y's fraction.  With beta2 = 0.999 a
// second moment shrinks by at most 0.1 % a step, 0.025 % of its code, which
// rounding to nearest never passes on; stochastic rounding does on average.
// It is the code whose mean is right.  A second moment is the code's fourth
// power, so its own mean lies above by a share of about (1 / c)^2 for a code
// c rounded once, and by more where a step's errors add up over many steps:
// medians measured at 1.00 of the 32-bit moment for codes above 100, 1.06 for
// 10 to 29, 1.16 for 4 to 9 (beta2 = 0.999, stationary gradients).
//
// A block whose largest magnitude is below 2^-100 is stored as zero (its
// scale's reciprocal would leave the range), one whose largest magnitude is
// not finite as NaN throughout.
//
// Codes are defined by IEEE single-precision arithmetic in the order written
// (adam_moments8, encode_m, encode_r): no contraction and no approximate function decides
// one, so the stored state does not depend on how a kernel is scheduled.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>

#include "elementwise.cuh"
#include "sm100_ptx.cuh"

namespace muon {

constexpr int ST_THREADS = 256;
constexpr int Q_BLOCK = 256;            // elements that share a scale: one warp, 8 per lane
constexpr int ST_WARPS = ST_THREADS / 32;
constexpr int ADAM8_CTAS = 4;             // resident thread blocks per SM
constexpr int ADAM8_SMEM = 55 * 1024;     // of shared memory each
constexpr int STATE8_BLOCKS = 4;          // per warp
constexpr int NORM_BYTES = 16384;         // of gradients in a chunk
constexpr int NORM_CTAS = 8;              // resident thread blocks per SM
constexpr int MAX_SLOTS = 480;          // tensors of one launch: their gradient pointers are a kernel
                                        // parameter (3840 B), so rebinding gradients touches no
                                        // device memory that a launch in flight could be reading
constexpr float Q_TINY = 7.8886090522101181e-31f;   // 2^-100

struct GradPtrs {
  const void* p[MAX_SLOTS];
};

// The work of one thread block: consecutive blocks of 256 elements of one
// tensor, the same number for each of its warps.  Pointers are those of the
// first element, so a thread block starts after one load; the hardware hands
// them out in order, so the GPU works on neighbouring addresses at any time
// and an SM that gets less bandwidth gets less work.  (Persistent warps over
// a static split were measured too: a pure stream lost 6 to 12 % to the
// slowest SMs.)
struct alignas(16) AdamChunk {
  char* param;
  char* m;                 // float or int8_t
  char* v;                 // float or uint8_t
  float* m_scale;          // 8-bit: one per block
  float* v_scale;
  __nv_bfloat16* copy;     // nullptr: none
  int64_t base;            // first element's index in its tensor
  uint32_t id;             // the tensor's place in the plan's list
  uint16_t slot;           // its gradient in the launch's GradPtrs
  uint16_t count;          // elements
};
static_assert(sizeof(AdamChunk) == 64, "one chunk is two 32-byte sectors");

struct AdamPlanScalars {
  float2 beta1, one_beta1, beta2, one_beta2;  // each twice, for packed operations; 1 - beta formed in 64 bits
  float2 eps2, minus_zero;                    // -0: adam_moments8
  float eps, decay, step_size, inv_bc2;       // 1 - lr wd, lr / (1 - beta1^t), 1 / sqrt(1 - beta2^t)
  double ln_beta1, ln_beta2, lr, wd;          // for a step count or rate that lives on the device
  const int64_t* step_ptr;
  const float* lr_ptr;
  const float* grad_scale;
  uint32_t seed_key, step;                    // mixed seed, low bits of the step
};

// 32-bit mixer: xor-shifts and odd multiplications, each a bijection; shifts
// and multipliers are those of C. Wellons, "Prospecting for Hash Functions"
// (2018).
__device__ __host__ __forceinline__ uint32_t mix32(uint32_t x) {
  x ^= x >> 16;
  x *= 0x7FEB352Du;
  x ^= x >> 15;
  x *= 0x846CA68Bu;
  return x ^ (x >> 16);
}

__device__ __forceinline__ float unit16(uint32_t h) {
  return __fmul_rn(__fadd_rn(static_cast<float>(h), 0.5f), 1.f / 65536.f);
}

// fp32 -> bf16 bits, up in magnitude with the probability of the dropped bits;
// infinities and NaN as rounding to nearest gives them.
__device__ __forceinline__ uint16_t bf16_stochastic(float x, uint32_t h16) {
  const uint32_t b = __float_as_uint(x);
  if ((b & 0x7F800000u) == 0x7F800000u) return __bfloat16_as_ushort(__float2bfloat16_rn(x));
  return static_cast<uint16_t>((b + h16) >> 16);
}

// ---------------------------------------------------------------------------
// a lane's 8 elements of a block: 4 l .. 4 l + 3 and 128 + 4 l .. 128 + 4 l + 3
// ---------------------------------------------------------------------------
// Every vector access of a warp then covers consecutive bytes, whatever the
// element's size.  `full`: the block is whole and the pointer aligned to 4
// elements; else element by element, those below `count` (of the block).
constexpr int HALF = Q_BLOCK / 2;

__device__ __forceinline__ bool inside(int lane, int k, int count) {
  return 4 * lane + (k & 3) + (k >> 2) * HALF < count;
}

template <bool BF16>
__device__ __forceinline__ void load8(const char* block, int lane, bool full, int count, float (&x)[8]) {
  if (full) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if (BF16) {
        const uint2 w = *reinterpret_cast<const uint2*>(block + 8 * lane + j * 2 * HALF);
        const float2 a = unpack_bf16x2(w.x), b = unpack_bf16x2(w.y);
        x[4 * j] = a.x; x[4 * j + 1] = a.y; x[4 * j + 2] = b.x; x[4 * j + 3] = b.y;
      } else {
        const float4 a = *reinterpret_cast<const float4*>(block + 16 * lane + j * 4 * HALF);
        x[4 * j] = a.x; x[4 * j + 1] = a.y; x[4 * j + 2] = a.z; x[4 * j + 3] = a.w;
      }
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int e = 4 * lane + (k & 3) + (k >> 2) * HALF;
      x[k] = e >= count ? 0.f
             : BF16 ? __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(block)[e])
                    : reinterpret_cast<const float*>(block)[e];
    }
  }
}

__device__ __forceinline__ void store8_f32(char* block, int lane, bool full, int count, const float (&x)[8]) {
  if (full) {
    *reinterpret_cast<float4*>(block + 16 * lane) = make_float4(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<float4*>(block + 16 * lane + 4 * HALF) = make_float4(x[4], x[5], x[6], x[7]);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (inside(lane, k, count)) reinterpret_cast<float*>(block)[4 * lane + (k & 3) + (k >> 2) * HALF] = x[k];
  }
}

// w: pairs of bf16
__device__ __forceinline__ void store8_u16(char* block, int lane, bool full, int count, const uint32_t (&w)[4]) {
  if (full) {
    *reinterpret_cast<uint2*>(block + 8 * lane) = make_uint2(w[0], w[1]);
    *reinterpret_cast<uint2*>(block + 8 * lane + 2 * HALF) = make_uint2(w[2], w[3]);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (inside(lane, k, count))
        reinterpret_cast<uint16_t*>(block)[4 * lane + (k & 3) + (k >> 2) * HALF] =
            static_cast<uint16_t>(w[k >> 1] >> (16 * (k & 1)));
  }
}

__device__ __forceinline__ void load8_codes(const char* block, int lane, bool full, int count, uint32_t (&w)[2]) {
  if (full) {
    w[0] = *reinterpret_cast<const uint32_t*>(block + 4 * lane);
    w[1] = *reinterpret_cast<const uint32_t*>(block + 4 * lane + HALF);
  } else {
    w[0] = w[1] = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (inside(lane, k, count))
        w[k >> 2] |= static_cast<uint32_t>(static_cast<uint8_t>(block[4 * lane + (k & 3) + (k >> 2) * HALF])) << (8 * (k & 3));
  }
}

__device__ __forceinline__ void store8_codes(char* block, int lane, bool full, int count, const uint32_t (&w)[2]) {
  if (full) {
    *reinterpret_cast<uint32_t*>(block + 4 * lane) = w[0];
    *reinterpret_cast<uint32_t*>(block + 4 * lane + HALF) = w[1];
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (inside(lane, k, count)) block[4 * lane + (k & 3) + (k >> 2) * HALF] = static_cast<char>(w[k >> 2] >> (8 * (k & 3)));
  }
}

__device__ __forceinline__ bool aligned(const void* p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// ---------------------------------------------------------------------------
// the 8-bit form
// ---------------------------------------------------------------------------
__device__ __forceinline__ float decode_m(uint32_t code, float s) {
  const float c = static_cast<float>(static_cast<int8_t>(code));
  return __fmul_rn(__fmul_rn(c, fabsf(c)), s);
}

__device__ __forceinline__ float decode_r(uint32_t code, float s) {
  const float c = static_cast<float>(code) + 1.f;
  return __fmul_rn(__fmul_rn(c, c), s);
}

// Scale of a block from its largest magnitude (as bits: NaN sorts above
// infinity, so it is not lost in the maximum).
__device__ __forceinline__ float block_scale(uint32_t max_bits, float inv_levels2) {
  const float s = __fmul_rn(__uint_as_float(max_bits), inv_levels2);
  return max_bits >= 0x7F800000u ? __uint_as_float(0x7FC00000u) : max_bits < __float_as_uint(Q_TINY) ? 0.f : s;
}

// ... of first moments from the largest |m|, of second ones from the largest v
// (roots keep order: the largest root is the root of the largest).
template <bool SECOND>
__device__ __forceinline__ float moment_scale(uint32_t max_bits) {
  return SECOND ? block_scale(__float_as_uint(__fsqrt_rn(__uint_as_float(max_bits))), 1.f / 65536.f)
                : block_scale(max_bits, 1.f / 16129.f);
}

// 1 / s, 0 for a block that keeps no codes.
__device__ __forceinline__ float scale_inverse(float s) { return s > 0.f ? __frcp_rn(s) : 0.f; }

// floor(sqrt(x / s) + u)
__device__ __forceinline__ float real_code(float x, float inv, float u) {
  return floorf(__fadd_rn(__fsqrt_rn(__fmul_rn(x, inv)), u));
}

__device__ __forceinline__ uint32_t encode_m(float m, float inv, float u) {
  if (inv == 0.f || m == 0.f) return 0;
  const int c = static_cast<int>(fminf(real_code(fabsf(m), inv, u), 127.f));
  return static_cast<uint32_t>(m < 0.f ? -c : c) & 0xFFu;
}

__device__ __forceinline__ uint32_t encode_r(float r, float inv, float u) {
  if (inv == 0.f) return 0;
  return static_cast<uint32_t>(fminf(fmaxf(real_code(r, inv, u), 1.f), 256.f)) - 1u;
}

// ---------------------------------------------------------------------------
// the same codes at streaming speed
// ---------------------------------------------------------------------------
// IEEE square roots and integer conversions for two codes an element made the
// 8-bit step compute bound.  The fast path forms y with sqrt.approx (relative
// error at most 2^-23) and rounds by adding 1.5 * 2^23; where y + u lies so
// near an integer that this could round to another code than the definition
// (FAR_* below, both sides' errors added up), the code is formed again by the
// definition.  A 16-bit u enters as h / 2^16 - 1/2, short of its 2^-17.
//
// Errors of y on both sides together, relative in units of 2^-23 (an IEEE
// operation has 1/2, an approximate one 1, rsqrt.approx 1.1), halved by the
// root where they stand under it:
//   m: 1 / s 1 + 1/2 here and 1 in the definition, whose 1 / 127^2 is off by
//      0.16, times m 1 -> 1.83; the root 1.5; times 127: 5.1e-5.  y + u: 2^-17 in the definition, 2^-18 twice
//      here, 2^-17 for the missing part of u: 2.3e-5.
//   r: r 1.5, 1 / s 1.1 here and 1 in the definition, the product 1 -> 2.3;
//      the root 1.5; times 256: 1.16e-4.  y + u: three times 2^-17 and 2^-18:
//      2.7e-5.
constexpr float FAR_M = 0.5f - 7.5e-5f;
constexpr float FAR_R = 0.5f - 1.46e-4f;
constexpr float ROUND_MAGIC = 12582912.f;   // 1.5 * 2^23

__device__ __forceinline__ float sqrt_fast(float x) {
  float y;
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float rcp_fast(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float rsqrt_fast(float x) {
  float y;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 1 / s on the fast path, straight from the largest |m| or v.
template <bool SECOND>
__device__ __forceinline__ float fast_inverse(uint32_t max_bits) {
  const float big = __uint_as_float(max_bits);
  return SECOND ? 65536.f * rsqrt_fast(big) : 16129.f * rcp_fast(big);
}

// max(a, |b|, |c|), NaN if any is
__device__ __forceinline__ float max_abs3(float a, float b, float c) {
  float y;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}

__device__ __forceinline__ float max_abs8(const float (&x)[8]) {
  return max_abs3(max_abs3(max_abs3(max_abs3(0.f, x[0], x[1]), x[2], x[3]), x[4], x[5]), x[6], x[7]);
}

// Two fp32 values in a register pair: sm_100a rounds both halves of a packed
// operation as the scalar one would, at one issue slot for two elements.
struct F2 {
  uint64_t v;
};
__device__ __forceinline__ F2 pack2(float lo, float hi) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpack2(F2 a, float& lo, float& hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(a.v)); }
__device__ __forceinline__ F2 both(float x) { return pack2(x, x); }

// Constants of packed operations, in constant memory: operands from there
// take neither registers nor the two moves that build a pair of literals.
enum PairConst { K_BIAS_M, K_BIAS_V, K_UP_M, K_DOWN_M, K_UP_R, K_DOWN_R, K_MINUS, K_UNIT, K_CENTRE, K_COUNT };
__constant__ float2 kPairs[K_COUNT] = {
    {-8388736.f, -8388736.f},                                  // - (2^23 + 128): a signed code
    {-8388607.f, -8388607.f},                                  // - 2^23 + 1: an unsigned code + 1
    {ROUND_MAGIC, ROUND_MAGIC}, {-ROUND_MAGIC, -ROUND_MAGIC},
    {ROUND_MAGIC - 1.f, ROUND_MAGIC - 1.f}, {1.f - ROUND_MAGIC, 1.f - ROUND_MAGIC},
    {-1.f, -1.f}, {1.f / 65536.f, 1.f / 65536.f}, {-128.5f, -128.5f}};
__device__ __forceinline__ F2 pair(const float2& x) { return {*reinterpret_cast<const uint64_t*>(&x)}; }
__device__ __forceinline__ F2 pair(PairConst k) { return {*reinterpret_cast<const uint64_t*>(&kPairs[k])}; }
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}

// byte k of w as the low mantissa byte of 2^23: 2^23 + byte
__device__ __forceinline__ float magic_byte(uint32_t w, int k) {
  return __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7650 | k));
}

// 2^23 + h of the low and the high half of w, their bytes swapped for `swap`
__device__ __forceinline__ F2 magic_halves(uint32_t w, bool swap) {
  return pack2(__uint_as_float(__byte_perm(w, 0x4B000000u, swap ? 0x7601 : 0x7610)),
               __uint_as_float(__byte_perm(w, 0x4B000000u, swap ? 0x7623 : 0x7632)));
}

__device__ __forceinline__ uint32_t pack_low_bytes(const float (&z)[8], int at) {
  const uint32_t a = __byte_perm(__float_as_uint(z[at]), __float_as_uint(z[at + 1]), 0x0040);
  const uint32_t b = __byte_perm(__float_as_uint(z[at + 2]), __float_as_uint(z[at + 3]), 0x0040);
  return __byte_perm(a, b, 0x5410);
}

// The block's real-valued codes a[k], moved by u - 1/2, rounded to nearest:
// low mantissa bytes of z[k] hold the codes, and the return value says whether
// any lies within the limits of a boundary.
template <bool SECOND, bool STOCH>
__device__ __forceinline__ bool round8(const float (&x)[8], float inv, const uint32_t (&h)[4], float (&a)[8], float (&z)[8]) {
  const F2 i2 = both(inv), up = pair(SECOND ? K_UP_R : K_UP_M), down = pair(SECOND ? K_DOWN_R : K_DOWN_M),
           minus = pair(K_MINUS);
  float f[8];
#pragma unroll
  for (int k = 0; k < 8; k += 2) {
    float lo, hi;
    unpack2(mul2(pack2(x[k], x[k + 1]), i2), lo, hi);
    lo = sqrt_fast(fabsf(lo));
    hi = sqrt_fast(fabsf(hi));
    // + h / 2^16 - 1/2; the magic 2^23 leaves 128 of it
    if (STOCH)
      unpack2(fma2(magic_halves(h[k >> 1], !SECOND), pair(K_UNIT), add2(pack2(lo, hi), pair(K_CENTRE))), lo, hi);
    a[k] = SECOND ? fmaxf(lo, 1.f) : copysignf(lo, x[k]);
    a[k + 1] = SECOND ? fmaxf(hi, 1.f) : copysignf(hi, x[k + 1]);
    const F2 a2 = pack2(a[k], a[k + 1]), z2 = add2(a2, up);
    unpack2(z2, z[k], z[k + 1]);
    unpack2(fma2(add2(z2, down), minus, a2), f[k], f[k + 1]);
  }
  return max_abs8(f) > (SECOND ? FAR_R : FAR_M);
}

// Forms the codes that round8 could not be sure of by their definition, one a
// pass: almost always a single one of a warp's 256.
template <bool SECOND, bool STOCH>
__device__ __forceinline__ void redo8(const float (&x)[8], uint32_t max_bits, const uint32_t (&h)[4], const float (&a)[8],
                                      float (&z)[8]) {
  constexpr float MAGIC = SECOND ? ROUND_MAGIC - 1.f : ROUND_MAGIC, FAR = SECOND ? FAR_R : FAR_M;
  const float inv = __frcp_rn(moment_scale<SECOND>(max_bits));
  uint32_t todo = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) todo |= (fabsf(a[k] - (z[k] - MAGIC)) > FAR ? 1u : 0u) << k;
  while (todo != 0) {
    const int at = __ffs(todo) - 1;
    todo &= todo - 1;
    float v = 0.f;
    uint32_t word = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k == at) {
        v = x[k];
        word = h[k >> 1] >> (16 * (k & 1));
      }
    word &= 0xFFFFu;
    const float u = STOCH ? unit16(SECOND ? word : ((word >> 8) | (word << 8)) & 0xFFFFu) : 0.5f;
    const float c = SECOND ? fminf(fmaxf(real_code(__fsqrt_rn(v), inv, u), 1.f), 256.f)
                           : copysignf(fminf(real_code(fabsf(v), inv, u), 127.f), v);
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k == at) z[k] = c + MAGIC;
  }
}

// Codes of 8 first moments (x = r = m) or second moments (x = v, r its fast
// root) on the fast path; max_bits: the largest |m| or v of the block.
template <bool SECOND, bool STOCH>
__device__ __forceinline__ void encode8_fast(const float (&x)[8], const float (&r)[8], uint32_t max_bits,
                                             const uint32_t (&h)[4], uint32_t (&w)[2]) {
  float a[8], z[8];
  if (round8<SECOND, STOCH>(r, fast_inverse<SECOND>(max_bits), h, a, z)) redo8<SECOND, STOCH>(x, max_bits, h, a, z);
  w[0] = pack_low_bytes(z, 0);
  w[1] = pack_low_bytes(z, 4);
}

// The moments that 8 codes stand for (decode_m, decode_r on all of them).
__device__ __forceinline__ void decode8_m(const uint32_t (&w)[2], float s, float (&m)[8]) {
  const uint32_t q[2] = {w[0] ^ 0x80808080u, w[1] ^ 0x80808080u};
  const F2 bias = pair(K_BIAS_M), s2 = both(s);
#pragma unroll
  for (int k = 0; k < 8; k += 2) {
    float lo, hi;
    unpack2(add2(pack2(magic_byte(q[k >> 2], k & 3), magic_byte(q[k >> 2], (k & 3) + 1)), bias), lo, hi);
    unpack2(mul2(pack2(__fmul_rn(lo, fabsf(lo)), __fmul_rn(hi, fabsf(hi))), s2), m[k], m[k + 1]);
  }
}

__device__ __forceinline__ void decode8_v(const uint32_t (&w)[2], float s, float (&v)[8]) {
  const F2 bias = pair(K_BIAS_V), s2 = both(s);
#pragma unroll
  for (int k = 0; k < 8; k += 2) {
    const F2 c = add2(pack2(magic_byte(w[k >> 2], k & 3), magic_byte(w[k >> 2], (k & 3) + 1)), bias);
    const F2 r = mul2(mul2(c, c), s2);
    unpack2(mul2(r, r), v[k], v[k + 1]);
  }
}

// Blocks that the fast path takes: its flushes of subnormals then change no
// code (an element whose v is subnormal lies below 2^-36 of the block's
// largest, code 0 on either path).
__device__ __forceinline__ bool fast_block(uint32_t mbits, uint32_t vbits) {
  constexpr uint32_t m_low = 0x0D800000u, m_top = 0x7B800000u;     // 2^-100, 2^120: 1 / m stays a normal number
  constexpr uint32_t v_low = 0x12800000u, v_top = 0x7F800000u;     // 2^-90, infinity
  return mbits - m_low < m_top - m_low && vbits - v_low < v_top - v_low;
}

// New moments, each operation rounded once.  A packed mul whose result goes
// into a packed add is contracted to an fma whatever their rounding modifiers,
// and so is an fma with a literal -0.  With a -0 that only the launch knows
// the products stay products: adding it changes none.
__device__ __forceinline__ void adam_moments8(float (&m)[8], float (&v)[8], const float (&g)[8], float scale,
                                              const AdamPlanScalars& s) {
  const F2 f = both(scale), b1 = pair(s.beta1), o1 = pair(s.one_beta1), b2 = pair(s.beta2), o2 = pair(s.one_beta2),
           z = pair(s.minus_zero);
#pragma unroll
  for (int k = 0; k < 8; k += 2) {
    const F2 g2 = mul2(pack2(g[k], g[k + 1]), f);
    unpack2(add2(fma2(pack2(m[k], m[k + 1]), b1, z), fma2(g2, o1, z)), m[k], m[k + 1]);
    unpack2(add2(fma2(pack2(v[k], v[k + 1]), b2, z), fma2(mul2(g2, g2), o2, z)), v[k], v[k + 1]);
  }
}

// p <- p decay - step_size m / (sqrt(v) inv_bc2 + eps).  FAST: approximate
// root and reciprocal (2^-22 of the update).
template <bool FAST>
__device__ __forceinline__ void adam_param8(float (&p)[8], const float (&m)[8], const float (&v)[8], float (&r)[8],
                                            float decay, float step_size, float inv_bc2, const float2& eps) {
  const F2 d2 = both(decay), s2 = both(-step_size), c2 = both(inv_bc2), e2 = pair(eps);
#pragma unroll
  for (int k = 0; k < 8; k += 2) {
    float lo, hi;
    r[k] = FAST ? sqrt_fast(v[k]) : __fsqrt_rn(v[k]);
    r[k + 1] = FAST ? sqrt_fast(v[k + 1]) : __fsqrt_rn(v[k + 1]);
    unpack2(fma2(pack2(r[k], r[k + 1]), c2, e2), lo, hi);
    const F2 q = FAST ? mul2(pack2(m[k], m[k + 1]), pack2(rcp_fast(lo), rcp_fast(hi))) : pack2(m[k] / lo, m[k + 1] / hi);
    unpack2(fma2(pack2(p[k], p[k + 1]), d2, mul2(q, s2)), p[k], p[k + 1]);
  }
}

// ---------------------------------------------------------------------------
// AdamW
// ---------------------------------------------------------------------------
// What a launch's scalars come to on the device.
struct AdamNow {
  float scale, step_size, inv_bc2, decay;
  uint32_t step;
  bool go;                 // false: nothing is written
};

// Every lane of a warp calls it, and all get the same answer: blocks are
// reduced over whole warps.
__device__ __forceinline__ AdamNow adam_now(const AdamPlanScalars& sc, const int* flags) {
  AdamNow d{1.f, sc.step_size, sc.inv_bc2, sc.decay, sc.step, true};
  const bool stop = halted(flags);
  if (sc.grad_scale != nullptr) {
    d.scale = *sc.grad_scale;
    d.go = isfinite(d.scale);           // a gradient was not finite
  }
  if (sc.step_ptr != nullptr || sc.lr_ptr != nullptr) {
    if ((threadIdx.x & 31) == 0) {
      const double lr = sc.lr_ptr != nullptr ? static_cast<double>(*sc.lr_ptr) : sc.lr;
      d.go = d.go && isfinite(lr);
      d.decay = static_cast<float>(1.0 - lr * sc.wd);
      if (sc.step_ptr != nullptr) {
        const int64_t t = *sc.step_ptr;
        d.go = d.go && t >= 1;
        d.step = static_cast<uint32_t>(t);
        d.step_size = static_cast<float>(lr / -expm1(static_cast<double>(t) * sc.ln_beta1));
        d.inv_bc2 = static_cast<float>(1.0 / sqrt(-expm1(static_cast<double>(t) * sc.ln_beta2)));
      } else {
        d.step_size = static_cast<float>(lr * static_cast<double>(sc.step_size));   // 1 / (1 - beta1^t) there
      }
    }
    d.go = __shfl_sync(0xffffffffu, d.go, 0);
    d.decay = __shfl_sync(0xffffffffu, d.decay, 0);
    d.step = __shfl_sync(0xffffffffu, d.step, 0);
    d.step_size = __shfl_sync(0xffffffffu, d.step_size, 0);
    d.inv_bc2 = __shfl_sync(0xffffffffu, d.inv_bc2, 0);
  }
  d.go = __all_sync(0xffffffffu, d.go && !stop);
  return d;
}

// The hashed bits of a lane's four pairs of elements: 16 for either element of
// pair q, mix32((low word of q ^ key) + high word of q * 0x9E3779B9).  e: the
// block's first element in its tensor, a multiple of 256, so that a pair's
// place in the block only sets zero bits of e / 2.
__device__ __forceinline__ void block_bits(int64_t e, int lane, uint32_t key, uint32_t (&h)[4]) {
  const uint64_t q = static_cast<uint64_t>(e) / 2;
  const uint32_t low = static_cast<uint32_t>(q) ^ key ^ (2 * lane), high = static_cast<uint32_t>(q >> 32) * 0x9E3779B9u;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    // kept as it is: the compiler would rather form it again for each of its
    // uses, 11 instructions an element more (134M elements: 350 and 314 us)
    h[k] = mix32((low ^ ((k >> 1) * (HALF / 2) + (k & 1))) + high);
    asm volatile("" : "+r"(h[k]));
  }
}

// New parameters to memory: bf16 (nearest or stochastic), or fp32 and its copy.
template <bool PBF16, bool COPY, bool STOCH>
__device__ __forceinline__ void store_param(char* param, char* copy, int lane, bool full, int count, const float (&p)[8],
                                            const uint32_t (&h)[4]) {
  uint32_t w[4];
  if (PBF16 && STOCH) {
    const bool odd = !(max_abs8(p) < INFINITY);     // a carry would turn a NaN's bits into a number
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t hp = mix32(h[k] ^ 0x5BD1E995u);
      if (odd)
        w[k] = uint32_t(bf16_stochastic(p[2 * k], hp & 0xFFFFu)) | uint32_t(bf16_stochastic(p[2 * k + 1], hp >> 16)) << 16;
      else
        w[k] = __byte_perm(__float_as_uint(p[2 * k]) + (hp & 0xFFFFu), __float_as_uint(p[2 * k + 1]) + (hp >> 16), 0x7632);
    }
    store8_u16(param, lane, full, count, w);
  } else if (PBF16 || COPY) {
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = pack_bf16x2(p[2 * k], p[2 * k + 1]);
    store8_u16(PBF16 ? param : copy, lane, full, count, w);
  }
  if (!PBF16) store8_f32(param, lane, full, count, p);
}

// The approximate root flushes one below 2^-63 to zero: eps has to cover it.
__device__ __forceinline__ bool eps_covers(float eps, float inv_bc2) { return eps >= 2e-12f * inv_bc2; }

// r receives the roots of v.
__device__ __forceinline__ void adam_param8(float (&p)[8], const float (&m)[8], const float (&v)[8], float (&r)[8],
                                            const AdamNow& now, const AdamPlanScalars& sc) {
  if (eps_covers(sc.eps, now.inv_bc2)) adam_param8<true>(p, m, v, r, now.decay, now.step_size, now.inv_bc2, sc.eps2);
  else adam_param8<false>(p, m, v, r, now.decay, now.step_size, now.inv_bc2, sc.eps2);
}

// fp32 moments: a block of 256 per warp, loaded straight to registers, ahead
// of the launch's scalars.  Bound by HBM: 28 B an element leave the arithmetic
// (27 instructions an element, start-up and all) a fifth of the issue slots.
template <bool PBF16, bool COPY, bool GBF16, bool STOCH>
__global__ void __launch_bounds__(ST_THREADS, 4)
    adamw32_kernel(const AdamChunk* __restrict__ chunks, const __grid_constant__ GradPtrs grads,
                   const __grid_constant__ AdamPlanScalars sc, const int* flags) {
  constexpr int P = PBF16 ? 2 : 4, G = GBF16 ? 2 : 4;
  // The table was complete before the first launch: it is read ahead of the
  // wait for the previous kernel.
  const AdamChunk ch = chunks[blockIdx.x];
  const int lane = threadIdx.x & 31, first = (threadIdx.x >> 5) * Q_BLOCK;
  const int count = static_cast<int>(ch.count) - first;
  if (count <= 0) return;
  const char* grad = static_cast<const char*>(grads.p[ch.slot]) + (ch.base + first) * G;
  char *const pp = ch.param + first * P, *const mp = ch.m + first * 4, *const vp = ch.v + first * 4;
  const bool full = count >= Q_BLOCK && aligned(pp, 4 * P) && aligned(grad, 4 * G) && aligned(mp, 16) &&
                    aligned(vp, 16) && (!COPY || aligned(ch.copy, 8));
  float g[8], p[8], m[8], v[8], r[8];
  pdl_wait();
  load8<GBF16>(grad, lane, full, count, g);
  load8<PBF16>(pp, lane, full, count, p);
  load8<false>(mp, lane, full, count, m);
  load8<false>(vp, lane, full, count, v);
  const AdamNow now = adam_now(sc, flags);
  if (!now.go) return;
  adam_moments8(m, v, g, now.scale, sc);
  adam_param8(p, m, v, r, now, sc);
  store8_f32(mp, lane, full, count, m);
  store8_f32(vp, lane, full, count, v);
  uint32_t h[4] = {};
  if (STOCH) block_bits(ch.base + first, lane, mix32(mix32(sc.seed_key + now.step) + ch.id), h);
  store_param<PBF16, COPY, STOCH>(pp, reinterpret_cast<char*>(ch.copy + first), lane, full, count, p, h);
}

// 8-bit moments: up to Stage8::blocks blocks per warp, fetched whole into
// shared memory by one bulk copy an array before the first is worked on.  One
// block per warp left the start-up (about 210 instructions and two loads that
// wait for one another) unpaid for: 134M elements, fp32 parameters, took 409
// us with one block, 323 with two, 294 with three; as many as ADAM8_CTAS
// resident thread blocks have shared memory for.  Four thread blocks of 64
// registers a thread beat three of 80 (304 and 310 us) and two (587 and 494 us
// in an earlier form): the arithmetic needs the warps more than registers, so
// what the loop over whole blocks keeps alive is kept small: the ragged tail
// goes first, scales stay in one register, their pointers are read again (296
// -> 285); new scales are formed once for all of a warp's blocks, from their
// largest magnitudes (285 -> 283, bf16 parameters 250 -> 244); with a copy,
// its pointer and its place in the tensor are read again for each block (327
// -> 324, stochastic 373 -> 326; the place without a copy, or m's and v's
// pointers, cost more than they freed).
template <bool PBF16, bool GBF16>
struct Stage8 {
  static constexpr int P = PBF16 ? 2 : 4, G = GBF16 ? 2 : 4;
  static constexpr int blocks = ADAM8_SMEM / (ST_WARPS * Q_BLOCK * (P + G + 2));
  static constexpr int off_g = P * Q_BLOCK * blocks, off_m = off_g + G * Q_BLOCK * blocks, off_v = off_m + Q_BLOCK * blocks,
                       bytes = off_v + Q_BLOCK * blocks;
  static constexpr int cta = ST_WARPS * bytes;
};

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
               "r"(bytes), "r"(bar) : "memory");
}

// Waits for the warp's bulk copies.  After kWaitLimitNs it records that in the
// context's flags, gives copies in flight as long again to land before the
// shared memory is given back, and returns false.  Lanes poll by their own
// clocks, so one may give up where another sees the copies land.
__device__ __forceinline__ bool lane_wait(uint64_t* bar, int* flags) {
  if (mbar_try_wait(bar, 0)) return true;
  for (int turn = 0; turn < 2; ++turn) {
    const uint64_t start = global_timer_ns();
    while (global_timer_ns() - start <= kWaitLimitNs)
      if (mbar_try_wait(bar, 0)) return turn == 0;
    atomicOr(flags, kDevErrTimeout);
  }
  return false;
}

// One answer for the warp, whose blocks need all of its lanes.
__device__ __forceinline__ bool bulk_wait(uint64_t* bar, int* flags) {
  return __all_sync(0xffffffffu, lane_wait(bar, flags));
}

// A block's new moments to codes and scales, by the definition.
template <bool STOCH>
__device__ __forceinline__ void encode8_exact(const float (&m)[8], const float (&v)[8], uint32_t mbits, uint32_t vbits,
                                              const uint32_t (&h)[4], uint32_t (&mw)[2], uint32_t (&vw)[2]) {
  const float minv = scale_inverse(moment_scale<false>(mbits)), rinv = scale_inverse(moment_scale<true>(vbits));
  mw[0] = mw[1] = vw[0] = vw[1] = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    float um = 0.5f, uv = 0.5f;
    if (STOCH) {
      const uint32_t hk = (h[k >> 1] >> (16 * (k & 1))) & 0xFFFFu;
      uv = unit16(hk);
      um = unit16(((hk >> 8) | (hk << 8)) & 0xFFFFu);
    }
    mw[k >> 2] |= encode_m(m[k], minv, um) << (8 * (k & 3));
    vw[k >> 2] |= encode_r(__fsqrt_rn(v[k]), rinv, uv) << (8 * (k & 3));
  }
}

// What a warp works on: its first element in the chunk and of each array.
struct Adam8Warp {
  char *param, *m, *v;
  int first;
  const char* grad;
  int64_t base;
  uint32_t key;
};

// Block b of a warp.  FULL: from shared memory, all 256 elements, vector
// stores.  Else `count` elements from and to global memory one by one.
// `scales`: lanes 2 b and 2 b + 1 hold the block's old scales of m and of r on
// entry, its largest new |m| and v on return, from which the warp forms the
// scales of all its blocks at once.
template <bool PBF16, bool COPY, bool GBF16, bool STOCH, bool FULL>
__device__ __forceinline__ void adam8_block(const Adam8Warp& w, const char* mine, int b, int count, float& scales,
                                            const AdamNow& now, const AdamPlanScalars& sc, const AdamChunk* ch) {
  using St = Stage8<PBF16, GBF16>;
  const int lane = threadIdx.x & 31, at = b * Q_BLOCK;
  float g[8], p[8], m[8], v[8], r[8];
  uint32_t mw[2], vw[2];
  load8<GBF16>((FULL ? mine + St::off_g : w.grad) + at * St::G, lane, FULL, count, g);
  load8<PBF16>((FULL ? mine : w.param) + at * St::P, lane, FULL, count, p);
  load8_codes((FULL ? mine + St::off_m : w.m) + at, lane, FULL, count, mw);
  load8_codes((FULL ? mine + St::off_v : w.v) + at, lane, FULL, count, vw);
  decode8_m(mw, __shfl_sync(0xffffffffu, scales, 2 * b), m);
  decode8_v(vw, __shfl_sync(0xffffffffu, scales, 2 * b + 1), v);
  adam_moments8(m, v, g, now.scale, sc);
  adam_param8(p, m, v, r, now, sc);
  uint32_t h[4] = {};
  if (STOCH) block_bits((COPY ? ch->base + w.first : w.base) + at, lane, w.key, h);
  store_param<PBF16, COPY, STOCH>(w.param + at * St::P, COPY ? reinterpret_cast<char*>(ch->copy + w.first + at) : nullptr, lane, FULL, count, p, h);
  if (!FULL) {
    // past the end m is 0 (no code, no gradient), but a code 0 of v is not
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (!inside(lane, k, count)) v[k] = 0.f;
  }
  const uint32_t mbits = __reduce_max_sync(0xffffffffu, __float_as_uint(max_abs8(m)));
  const uint32_t vbits = __reduce_max_sync(0xffffffffu, __float_as_uint(max_abs8(v)));
  if (lane >> 1 == b) scales = __uint_as_float(lane & 1 ? vbits : mbits);
  // (a stochastic tail on the fast path cost the loop over whole blocks
  // registers: 183 -> 188 us on 38.7M elements with the clip and unpacking)
  if ((FULL || !STOCH) && fast_block(mbits, vbits)) {
    encode8_fast<false, STOCH>(m, m, mbits, h, mw);
    encode8_fast<true, STOCH>(v, r, vbits, h, vw);
  } else {
    encode8_exact<STOCH>(m, v, mbits, vbits, h, mw, vw);
  }
  store8_codes(w.m + at, lane, FULL, count, mw);
  store8_codes(w.v + at, lane, FULL, count, vw);
}

template <bool PBF16, bool COPY, bool GBF16, bool STOCH>
__global__ void __launch_bounds__(ST_THREADS, ADAM8_CTAS)
    adamw8_kernel(const AdamChunk* __restrict__ chunks, int blocks, const __grid_constant__ GradPtrs grads,
                  const __grid_constant__ AdamPlanScalars sc, int* flags) {
  using St = Stage8<PBF16, GBF16>;
  extern __shared__ __align__(128) char smem[];
  __shared__ __align__(8) uint64_t bars[ST_WARPS];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, first = warp * blocks * Q_BLOCK;
  const char* mine = smem + warp * St::bytes;
  Adam8Warp w;
  AdamNow now;
  int whole, count;
  float scales = 0.f;
  {
    // The table was complete before the first launch: it is read ahead of the
    // wait for the previous kernel.
    const AdamChunk ch = chunks[blockIdx.x];
    count = min(static_cast<int>(ch.count) - first, blocks * Q_BLOCK);
    if (count <= 0) return;
    w.grad = static_cast<const char*>(grads.p[ch.slot]) + (ch.base + first) * St::G;
    w.param = ch.param + first * St::P;
    w.m = ch.m + first;
    w.v = ch.v + first;
    w.first = first;
    w.base = ch.base + first;
    // bulk copies want 16-byte boundaries; whole blocks have them when their
    // tensors do.  What is left (a tensor's last block, views at odd offsets)
    // is loaded where it is used.
    const bool vec = aligned(w.param, 16) && aligned(w.grad, 16) && aligned(w.m, 16) && aligned(w.v, 16) &&
                     (!COPY || aligned(ch.copy, 8));
    whole = vec ? count / Q_BLOCK : 0;
    if (lane == 0) {
      mbar_init(&bars[warp], 1);
      fence_barrier_init();
    }
    __syncwarp();
    pdl_wait();
    if (whole > 0 && lane == 0) {
      const uint32_t n = whole * Q_BLOCK, dst = smem_u32(mine), bar = smem_u32(&bars[warp]);
      mbar_arrive_expect_tx(&bars[warp], n * (St::P + St::G + 2));
      bulk_load(dst + St::off_g, w.grad, n * St::G, bar);
      bulk_load(dst, w.param, n * St::P, bar);
      bulk_load(dst + St::off_m, w.m, n, bar);
      bulk_load(dst + St::off_v, w.v, n, bar);
    }
    if ((lane >> 1) * Q_BLOCK < count) scales = ((lane & 1 ? ch.v_scale : ch.m_scale) + first / Q_BLOCK)[lane >> 1];
    now = adam_now(sc, flags);
    w.key = STOCH ? mix32(mix32(sc.seed_key + now.step) + ch.id) : 0u;
  }
  if (now.go) {
#pragma unroll 1
    for (int b = whole; b * Q_BLOCK < count; ++b)
      adam8_block<PBF16, COPY, GBF16, STOCH, false>(w, mine, b, count - b * Q_BLOCK, scales, now, sc, chunks + blockIdx.x);
  }
  // Scales of the blocks from `from` on.  The chunk's pointers are read again:
  // kept, they would cost the loop registers.
  auto store_scales = [&](int from) {
    const AdamChunk* ch = chunks + blockIdx.x;
    const uint32_t bits = __float_as_uint(scales);
    const float ms = moment_scale<false>(bits), rs = moment_scale<true>(bits);
    if (lane >> 1 >= from && (lane >> 1) * Q_BLOCK < min(static_cast<int>(ch->count) - first, blocks * Q_BLOCK))
      ((lane & 1 ? ch->v_scale : ch->m_scale) + first / Q_BLOCK)[lane >> 1] = lane & 1 ? rs : ms;
  };
  const bool landed = whole == 0 || bulk_wait(&bars[warp], flags);
  if (!now.go) return;
  if (!landed) {
    store_scales(whole);     // the tail's codes are already new
    return;
  }
#pragma unroll 1
  for (int b = 0; b < whole; ++b) adam8_block<PBF16, COPY, GBF16, STOCH, true>(w, mine, b, Q_BLOCK, scales, now, sc, chunks + blockIdx.x);
  store_scales(0);
}

// ---------------------------------------------------------------------------
// conversion
// ---------------------------------------------------------------------------
struct alignas(16) Q8Chunk {
  char* values;            // fp32 or bf16 moments
  char* codes;             // int8 first moments or uint8 second moments
  float* scales;
  uint16_t count;          // elements
  uint8_t second;          // 1: second moments
  uint8_t bf16;            // values' type
  uint32_t pad;
};
static_assert(sizeof(Q8Chunk) == 32, "one chunk is one sector");

// One block.  PACK: values -> codes and scale, rounded to nearest.  Else the
// values that the codes stand for, rounded once to the values' type.
template <bool SECOND>
__device__ __forceinline__ void pack8(float (&x)[8], float* scale, int lane, uint32_t (&w)[2]) {
  const uint32_t xbits = __reduce_max_sync(0xffffffffu, __float_as_uint(max_abs8(x)));
  bool plain = true;
  if (SECOND) {
    // a negative second moment has no root
    float low = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) low = fminf(low, x[k]);
    plain = __all_sync(0xffffffffu, low == 0.f);
  }
  const uint32_t bits = plain ? xbits : 0x7FC00000u;
  const float s = moment_scale<SECOND>(bits);
  if (lane == 0) *scale = s;
  const uint32_t none[4] = {};
  w[0] = w[1] = 0;
  if (fast_block(SECOND ? __float_as_uint(1.f) : bits, SECOND ? bits : __float_as_uint(1.f))) {
    float r[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) r[k] = SECOND ? sqrt_fast(x[k]) : x[k];
    encode8_fast<SECOND, false>(x, r, bits, none, w);
  } else {
    const float inv = scale_inverse(s);
#pragma unroll
    for (int k = 0; k < 8; ++k)
      w[k >> 2] |= (SECOND ? encode_r(__fsqrt_rn(x[k]), inv, 0.5f) : encode_m(x[k], inv, 0.5f)) << (8 * (k & 3));
  }
}

// A warp's blocks of a chunk, U at once: their loads first.
template <bool PACK, bool SECOND, bool BF16, int U>
__device__ __forceinline__ void convert_blocks(char* values, char* codes, float* scales, int lane, bool full, int count) {
  constexpr int V = BF16 ? 2 : 4;
  float x[U][8];
  uint32_t w[U][2];
  if (PACK) {
#pragma unroll
    for (int u = 0; u < U; ++u) load8<BF16>(values + u * Q_BLOCK * V, lane, full, count, x[u]);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      pack8<SECOND>(x[u], scales + u, lane, w[u]);
      store8_codes(codes + u * Q_BLOCK, lane, full, count, w[u]);
    }
  } else {
    float s[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      load8_codes(codes + u * Q_BLOCK, lane, full, count, w[u]);
      s[u] = scales[u];
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (SECOND) decode8_v(w[u], s[u], x[u]);
      else decode8_m(w[u], s[u], x[u]);
      if (BF16) {
        uint32_t o[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) o[k] = pack_bf16x2(x[u][2 * k], x[u][2 * k + 1]);
        store8_u16(values + u * Q_BLOCK * V, lane, full, count, o);
      } else {
        store8_f32(values + u * Q_BLOCK * V, lane, full, count, x[u]);
      }
    }
  }
}

template <bool PACK, bool SECOND, bool BF16>
__device__ __forceinline__ void convert_run(const Q8Chunk& ch, int first, int lane) {
  constexpr int V = BF16 ? 2 : 4, U = STATE8_BLOCKS;
  char *values = ch.values + first * V, *codes = ch.codes + first;
  float* scales = ch.scales + first / Q_BLOCK;
  int count = min(static_cast<int>(ch.count) - first, U * Q_BLOCK);
  const bool vec = aligned(values, 4 * V) && aligned(codes, 4);
  if (vec && count == U * Q_BLOCK) {
    convert_blocks<PACK, SECOND, BF16, U>(values, codes, scales, lane, true, Q_BLOCK);
    return;
  }
  for (; count > 0; count -= Q_BLOCK) {
    convert_blocks<PACK, SECOND, BF16, 1>(values, codes, scales, lane, vec && count >= Q_BLOCK, count);
    values += Q_BLOCK * V;
    codes += Q_BLOCK;
    ++scales;
  }
}

template <bool PACK>
__global__ void __launch_bounds__(ST_THREADS) state8_kernel(const Q8Chunk* __restrict__ chunks, const int* flags) {
  const Q8Chunk ch = chunks[blockIdx.x];
  const int lane = threadIdx.x & 31, first = (threadIdx.x >> 5) * STATE8_BLOCKS * Q_BLOCK;
  pdl_wait();
  if (first >= ch.count || __any_sync(0xffffffffu, halted(flags))) return;
  if (ch.second)
    ch.bf16 ? convert_run<PACK, true, true>(ch, first, lane) : convert_run<PACK, true, false>(ch, first, lane);
  else
    ch.bf16 ? convert_run<PACK, false, true>(ch, first, lane) : convert_run<PACK, false, false>(ch, first, lane);
}

// ---------------------------------------------------------------------------
// gradient norm
// ---------------------------------------------------------------------------
struct alignas(16) NormChunk {
  int64_t base;            // first element's index in its tensor
  uint16_t slot;
  uint16_t count;          // elements
  uint32_t bf16;
};
static_assert(sizeof(NormChunk) == 16, "");

// Sum of squares of up to 8 elements.  fp32 holds it to 2^-22 when it lies well
// inside fp32's range; if not (tiny or huge gradients, but not all zeros, as
// the rows of an embedding that no token touched have) `bad` is set and the
// squares have to be formed in 64 bits.
__device__ __forceinline__ float squares8(const float (&x)[8], bool& bad) {
  float s = 0.f;
#pragma unroll
  for (int k = 0; k < 8; ++k) s = fmaf(x[k], x[k], s);
  bad |= !(s > 1e-25f && s < 1e37f) && max_abs8(x) != 0.f;
  return s;
}

__device__ __forceinline__ double squares8_wide(const float (&x)[8]) {
  double d = 0.0;
#pragma unroll
  for (int k = 0; k < 8; ++k) d = fma(static_cast<double>(x[k]), static_cast<double>(x[k]), d);
  return d;
}

__device__ __forceinline__ double block_sum_f64(double v, double* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  double s = 0.0;
  if (threadIdx.x < 32) {
    s = threadIdx.x < ST_WARPS ? red[threadIdx.x] : 0.0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  }
  return s;    // valid in warp 0
}

// partials: one per block of this list's launches, then the block counter.
// The last block to finish adds the partials in order (no atomics on values:
// the same gradients give the same norm) and resets the counter.
struct NormOut {
  float* out;              // norm, factor
  double* partials;
  unsigned int* counter;
  double max_norm;
  unsigned int first;      // this launch's first partial
  unsigned int total;      // blocks of all launches (0: nothing to sum)
};

// One chunk: a thread's vectors of 16 bytes are ST_THREADS vectors apart, U
// loaded at once.
template <bool BF16>
__device__ __forceinline__ double square_chunk(const char* g, int count) {
  // Four vectors of a thread in flight and eight thread blocks per SM: 134M
  // bf16 gradients 42.2 us; eight vectors and four thread blocks 44.9, sixteen
  // and two 49.5.
  constexpr int V = NORM_BYTES / 16 / ST_THREADS;
  double acc = 0.0;
  if (count == NORM_BYTES / (BF16 ? 2 : 4) && aligned(g, 16)) {
    const uint4* p = reinterpret_cast<const uint4*>(g) + threadIdx.x;
    uint4 raw[V];
#pragma unroll
    for (int u = 0; u < V; ++u) raw[u] = p[u * ST_THREADS];
    auto eight = [](const uint4& w, const uint4& z, float (&x)[8]) {
      if (BF16) {
        const float2 a = unpack_bf16x2(w.x), b = unpack_bf16x2(w.y), c = unpack_bf16x2(w.z), d = unpack_bf16x2(w.w);
        x[0] = a.x; x[1] = a.y; x[2] = b.x; x[3] = b.y; x[4] = c.x; x[5] = c.y; x[6] = d.x; x[7] = d.y;
      } else {
        x[0] = __uint_as_float(w.x); x[1] = __uint_as_float(w.y); x[2] = __uint_as_float(w.z); x[3] = __uint_as_float(w.w);
        x[4] = __uint_as_float(z.x); x[5] = __uint_as_float(z.y); x[6] = __uint_as_float(z.z); x[7] = __uint_as_float(z.w);
      }
    };
    constexpr int S = BF16 ? 1 : 2;      // vectors of 8 elements
    bool bad = false;
#pragma unroll
    for (int u = 0; u < V; u += S) {
      float x[8];
      eight(raw[u], raw[u + S - 1], x);
      acc += squares8(x, bad);
    }
    if (bad) {
      acc = 0.0;
#pragma unroll 1
      for (int u = 0; u < V; u += S) {
        float x[8];
        eight(p[u * ST_THREADS], p[(u + S - 1) * ST_THREADS], x);
        acc += squares8_wide(x);
      }
    }
    return acc;
  }
  for (int b = (threadIdx.x >> 5) * Q_BLOCK; b < count; b += ST_WARPS * Q_BLOCK) {
    float x[8];
    const char* block = g + b * (BF16 ? 2 : 4);
    load8<BF16>(block, threadIdx.x & 31, count - b >= Q_BLOCK && aligned(block, 16), count - b, x);
    bool bad = false;
    const float s = squares8(x, bad);
    acc += bad ? squares8_wide(x) : static_cast<double>(s);
  }
  return acc;
}

// Thread block b takes chunks b, b + gridDim.x, ...
__global__ void __launch_bounds__(ST_THREADS, NORM_CTAS)
    grad_norm_kernel(const NormChunk* __restrict__ chunks, unsigned nchunks, const __grid_constant__ GradPtrs grads,
                     const NormOut o) {
  __shared__ double red[ST_WARPS];
  __shared__ bool last;
  double acc = 0.0;
  NormChunk ch{};
  if (blockIdx.x < nchunks) ch = chunks[blockIdx.x];
  pdl_wait();
  for (unsigned c = blockIdx.x; c < nchunks;) {
    const char* g = static_cast<const char*>(grads.p[ch.slot]) + ch.base * (ch.bf16 ? 2 : 4);
    const NormChunk now = ch;
    c += gridDim.x;
    if (c < nchunks) ch = chunks[c];
    acc += now.bf16 ? square_chunk<true>(g, now.count) : square_chunk<false>(g, now.count);
  }
  double sum = block_sum_f64(acc, red);
  if (o.total > 1) {
    if (threadIdx.x == 0) {
      o.partials[o.first + blockIdx.x] = sum;
      __threadfence();
      // wraps to 0 when every block has come by
      last = atomicInc(o.counter, o.total - 1) == o.total - 1;
    }
    __syncthreads();
    if (!last) return;
    __threadfence();
    sum = 0.0;
    for (unsigned int i = threadIdx.x; i < o.total; i += ST_THREADS) sum += __ldcg(o.partials + i);
    sum = block_sum_f64(sum, red);
  }
  if (threadIdx.x == 0) {
    const float norm = static_cast<float>(sqrt(sum));
    o.out[0] = norm;
    // a norm that is not finite leaves no factor: steps that read it write nothing
    o.out[1] = isfinite(norm) ? static_cast<float>(fmin(1.0, o.max_norm / (sqrt(sum) + 1e-6))) : __uint_as_float(0x7FC00000u);
  }
}

}  // namespace muon
