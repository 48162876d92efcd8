// state_ops.cuh -- AdamW over many tensors with its moments in 32 or 8 bits,
// the gradient norm that clips it, and the conversion of moments between the
// two forms.  All are HBM-bound streams over lists of tensors.
//
//   adamw_plan_kernel  one AdamW step.  fp32 moments, or 8-bit codes with one
//                      fp32 scale per 256 elements; fp32 or bf16 parameters,
//                      fp32 parameters optionally with a bf16 working copy.
//   grad_norm_kernel   norm = sqrt(sum g^2) over a list and the clip factor
//                      min(1, max_norm / (norm + 1e-6)), one launch.
//   state8_kernel      moments (fp32 or bf16) -> codes and scales, and back.
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
//
// A block whose largest magnitude is below 2^-100 is stored as zero (its
// scale's reciprocal would leave the range), one whose largest magnitude is
// not finite as NaN throughout.
//
// Codes are defined by IEEE single-precision arithmetic in the order written
// (adam_moments, encode_*): no contraction and no approximate function decides
// one, so the stored state does not depend on how a kernel is scheduled.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>

#include "elementwise.cuh"
#include "sm100_ptx.cuh"

namespace muon {

constexpr int ST_THREADS = 256;
constexpr int Q_BLOCK = 256;            // elements that share a scale: one warp, 8 per lane
constexpr int ST_CHUNK = 2048;          // elements of one thread block: a block of 256 for each warp
constexpr int MAX_SLOTS = 480;          // tensors of one launch: their gradient pointers are a kernel
                                        // parameter (3840 B), so rebinding gradients touches no
                                        // device memory that a launch in flight could be reading
constexpr float Q_TINY = 7.8886090522101181e-31f;   // 2^-100

struct GradPtrs {
  const void* p[MAX_SLOTS];
};

// ST_CHUNK elements of one tensor.  Pointers are those of the chunk's first
// element, so a block starts after one 64-byte load.
struct alignas(16) AdamChunk {
  void* param;
  void* m;                 // float or int8_t
  void* v;                 // float or uint8_t
  float* m_scale;          // 8-bit: one per 256 elements
  float* v_scale;
  __nv_bfloat16* copy;     // nullptr: none
  int64_t base;            // first element's index in its tensor
  uint32_t id;             // the tensor's place in the plan's list
  uint16_t slot;           // its gradient in the launch's GradPtrs
  uint16_t count;          // elements, 1 .. ST_CHUNK
};
static_assert(sizeof(AdamChunk) == 64, "one chunk is two 32-byte sectors");

struct AdamPlanScalars {
  float beta1, one_beta1, beta2, one_beta2;   // 1 - beta formed in 64 bits
  float eps, decay, step_size, inv_bc2;       // 1 - lr wd, lr / (1 - beta1^t), 1 / sqrt(1 - beta2^t)
  double ln_beta1, ln_beta2, lr, wd;          // for a step count or rate that lives on the device
  const int64_t* step_ptr;
  const float* lr_ptr;
  const float* grad_scale;
  uint32_t seed_key, step;                    // mixed seed, low bits of the step
  float minus_zero;                           // -0 (adam_moments8)
};

// 32-bit mixer: xor-shifts and odd multiplications, each a bijection.
__device__ __host__ __forceinline__ uint32_t mix32(uint32_t x) {
  x ^= x >> 16;
  x *= 0x7FEB352Du;
  x ^= x >> 15;
  x *= 0x846CA68Bu;
  return x ^ (x >> 16);
}

// 16 + 16 hashed bits for elements 2 q and 2 q + 1 of a tensor with key k.
__device__ __forceinline__ uint32_t pair_bits(uint64_t q, uint32_t key) {
  return mix32((static_cast<uint32_t>(q) ^ key) + static_cast<uint32_t>(q >> 32) * 0x9E3779B9u);
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
// 8 consecutive elements of a lane
// ---------------------------------------------------------------------------
template <int BF16>
__device__ __forceinline__ void load8_vec(const void* p, float (&x)[8]) {
  if (BF16) {
    const uint4 w = *static_cast<const uint4*>(p);
    float2 f;
    f = unpack_bf16x2(w.x); x[0] = f.x; x[1] = f.y;
    f = unpack_bf16x2(w.y); x[2] = f.x; x[3] = f.y;
    f = unpack_bf16x2(w.z); x[4] = f.x; x[5] = f.y;
    f = unpack_bf16x2(w.w); x[6] = f.x; x[7] = f.y;
  } else {
    const float4 a = static_cast<const float4*>(p)[0], b = static_cast<const float4*>(p)[1];
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w; x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  }
}

template <int BF16>
__device__ __forceinline__ void load8_some(const void* p, int n, float (&x)[8]) {
#pragma unroll
  for (int k = 0; k < 8; ++k)
    x[k] = k >= n ? 0.f : BF16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p)[k]) : static_cast<const float*>(p)[k];
}

__device__ __forceinline__ void store8_f32(float* p, const float (&x)[8], bool vec, int n) {
  if (vec) {
    reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < n) p[k] = x[k];
  }
}

__device__ __forceinline__ void store8_u16(void* p, const uint32_t (&w)[4], bool vec, int n) {
  if (vec) {
    *static_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < n) static_cast<uint16_t*>(p)[k] = static_cast<uint16_t>(w[k >> 1] >> (16 * (k & 1)));
  }
}

__device__ __forceinline__ void load8_codes(const void* p, bool vec, int n, uint32_t (&w)[2]) {
  if (vec) {
    const uint2 q = *static_cast<const uint2*>(p);
    w[0] = q.x; w[1] = q.y;
  } else {
    w[0] = w[1] = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < n) w[k >> 2] |= static_cast<uint32_t>(static_cast<const uint8_t*>(p)[k]) << (8 * (k & 3));
  }
}

__device__ __forceinline__ void store8_codes(void* p, const uint32_t (&w)[2], bool vec, int n) {
  if (vec) {
    *static_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < n) static_cast<uint8_t*>(p)[k] = static_cast<uint8_t>(w[k >> 2] >> (8 * (k & 3)));
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
// infinity, so it is not lost in the maximum), and the scale's reciprocal, 0
// for a block that keeps no codes.
__device__ __forceinline__ float block_scale(uint32_t max_bits, float inv_levels2, float& inv) {
  const float big = __uint_as_float(max_bits);
  inv = 0.f;
  if (max_bits >= 0x7F800000u) return __uint_as_float(0x7FC00000u);
  if (big < Q_TINY) return 0.f;
  const float s = __fmul_rn(big, inv_levels2);
  inv = __frcp_rn(s);
  return s;
}

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
// Errors in y, in units of 2^-23 relative unless absolute:
//   m: sqrt.approx 1, IEEE root 1/2; times 127: 2.3e-5.  y + u: 2^-17 on the
//      definition's side, 2^-18 here, 2^-17 for the missing part of u: 1.9e-5.
//   r: r itself 1 + 1/2, r * inv twice 1/2, halved by the root: 1.25; the root
//      1 + 1/2; times 256: 8.4e-5.  y + u: 2^-17 + 2^-17 + 2^-17: 2.3e-5
//      (2^-16 each above 256 only where min() decides).
constexpr float FAR_M = 0.5f - 6.1e-5f;
constexpr float FAR_R = 0.5f - 1.9e-4f;
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

// h / 2^16 - 1/2 of the low (or high) half of w, its bytes swapped for `swap`
__device__ __forceinline__ float half_unit(uint32_t w, int high, bool swap) {
  const int b0 = 2 * high + (swap ? 1 : 0), b1 = 2 * high + (swap ? 0 : 1);
  return fmaf(__uint_as_float(__byte_perm(w, 0x4B000000u, 0x7600 | (b1 << 4) | b0)), 1.f / 65536.f, -128.5f);
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
  constexpr float MAGIC = SECOND ? ROUND_MAGIC - 1.f : ROUND_MAGIC;
  const F2 i2 = both(inv), up = both(MAGIC), down = both(-MAGIC), minus = both(-1.f);
  float f[8];
#pragma unroll
  for (int k = 0; k < 8; k += 2) {
    float lo, hi;
    unpack2(mul2(pack2(x[k], x[k + 1]), i2), lo, hi);
    lo = sqrt_fast(fabsf(lo));
    hi = sqrt_fast(fabsf(hi));
    if (STOCH) {
      lo += half_unit(h[k >> 1], 0, !SECOND);
      hi += half_unit(h[k >> 1], 1, !SECOND);
    }
    a[k] = SECOND ? fmaxf(lo, 1.f) : copysignf(lo, x[k]);
    a[k + 1] = SECOND ? fmaxf(hi, 1.f) : copysignf(hi, x[k + 1]);
    const F2 a2 = pack2(a[k], a[k + 1]), z2 = add2(a2, up);
    unpack2(z2, z[k], z[k + 1]);
    unpack2(fma2(add2(z2, down), minus, a2), f[k], f[k + 1]);
  }
  return max_abs8(f) > (SECOND ? FAR_R : FAR_M);
}

template <bool STOCH>
__device__ __forceinline__ void encode8_m_fast(const float (&m)[8], float inv, const uint32_t (&h)[4], uint32_t (&w)[2]) {
  float a[8], z[8];
  if (round8<false, STOCH>(m, inv, h, a, z)) {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (fabsf(a[k] - (z[k] - ROUND_MAGIC)) > FAR_M) {
        const uint32_t hk = (h[k >> 1] >> (16 * (k & 1))) & 0xFFFFu;
        const float u = STOCH ? unit16(((hk >> 8) | (hk << 8)) & 0xFFFFu) : 0.5f;
        z[k] = copysignf(fminf(real_code(fabsf(m[k]), inv, u), 127.f), m[k]) + ROUND_MAGIC;
      }
  }
  w[0] = pack_low_bytes(z, 0);
  w[1] = pack_low_bytes(z, 4);
}

template <bool STOCH>
__device__ __forceinline__ void encode8_r_fast(const float (&v)[8], float inv, const uint32_t (&h)[4], uint32_t (&w)[2]) {
  float r[8], a[8], z[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) r[k] = sqrt_fast(v[k]);
  if (round8<true, STOCH>(r, inv, h, a, z)) {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (fabsf(a[k] - (z[k] - (ROUND_MAGIC - 1.f))) > FAR_R) {
        const float u = STOCH ? unit16((h[k >> 1] >> (16 * (k & 1))) & 0xFFFFu) : 0.5f;
        z[k] = fminf(fmaxf(real_code(__fsqrt_rn(v[k]), inv, u), 1.f), 256.f) + (ROUND_MAGIC - 1.f);
      }
  }
  w[0] = pack_low_bytes(z, 0);
  w[1] = pack_low_bytes(z, 4);
}

// The moments that 8 codes stand for (decode_m, decode_r on all of them).
__device__ __forceinline__ void decode8_m(const uint32_t (&w)[2], float s, float (&m)[8]) {
  const uint32_t q[2] = {w[0] ^ 0x80808080u, w[1] ^ 0x80808080u};
  const F2 bias = both(-8388736.f), s2 = both(s);      // 2^23 + 128
#pragma unroll
  for (int k = 0; k < 8; k += 2) {
    float lo, hi;
    unpack2(add2(pack2(magic_byte(q[k >> 2], k & 3), magic_byte(q[k >> 2], (k & 3) + 1)), bias), lo, hi);
    unpack2(mul2(pack2(__fmul_rn(lo, fabsf(lo)), __fmul_rn(hi, fabsf(hi))), s2), m[k], m[k + 1]);
  }
}

__device__ __forceinline__ void decode8_v(const uint32_t (&w)[2], float s, float (&v)[8]) {
  const F2 bias = both(-8388607.f), s2 = both(s);      // the code + 1
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
constexpr float FAST_V_MIN = 8.0779356694631609e-28f;   // 2^-90
__device__ __forceinline__ bool fast_block(uint32_t mbits, uint32_t vbits) {
  return mbits >= __float_as_uint(Q_TINY) && mbits < 0x7F800000u && vbits >= __float_as_uint(FAST_V_MIN) &&
         vbits < 0x7F800000u;
}

// New moments, each operation rounded once.  A packed mul whose result goes
// into a packed add is contracted to an fma whatever their rounding modifiers,
// and so is an fma with a literal -0.  With a -0 that only the launch knows
// the products stay products: adding it changes none.
__device__ __forceinline__ void adam_moments8(float (&m)[8], float (&v)[8], const float (&g)[8], float scale,
                                              const AdamPlanScalars& s) {
  const F2 f = both(scale), b1 = both(s.beta1), o1 = both(s.one_beta1), b2 = both(s.beta2), o2 = both(s.one_beta2),
           z = both(s.minus_zero);
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
__device__ __forceinline__ void adam_param8(float (&p)[8], const float (&m)[8], const float (&v)[8], float decay,
                                            float step_size, float inv_bc2, float eps) {
  const F2 d2 = both(decay), s2 = both(-step_size), c2 = both(inv_bc2), e2 = both(eps);
#pragma unroll
  for (int k = 0; k < 8; k += 2) {
    float lo, hi;
    const F2 r = FAST ? pack2(sqrt_fast(v[k]), sqrt_fast(v[k + 1])) : pack2(__fsqrt_rn(v[k]), __fsqrt_rn(v[k + 1]));
    unpack2(fma2(r, c2, e2), lo, hi);
    const F2 q = FAST ? mul2(pack2(m[k], m[k + 1]), pack2(rcp_fast(lo), rcp_fast(hi))) : pack2(m[k] / lo, m[k + 1] / hi);
    unpack2(fma2(pack2(p[k], p[k + 1]), d2, mul2(q, s2)), p[k], p[k + 1]);
  }
}

// ---------------------------------------------------------------------------
// AdamW
// ---------------------------------------------------------------------------
template <bool S8, bool PBF16, bool GBF16, bool STOCH>
__global__ void __launch_bounds__(ST_THREADS, 4)
    adamw_plan_kernel(const AdamChunk* __restrict__ chunks, const __grid_constant__ GradPtrs grads,
                      const __grid_constant__ AdamPlanScalars sc, const int* flags) {
  // The table was complete before the first launch: it is read ahead of the
  // wait for the previous kernel.
  const AdamChunk ch = chunks[blockIdx.x];
  const char* grad = static_cast<const char*>(grads.p[ch.slot]) + ch.base * (GBF16 ? 2 : 4);
  pdl_wait();
  if (halted(flags)) return;
  float scale = 1.f;
  if (sc.grad_scale != nullptr) {
    scale = *sc.grad_scale;
    if (!isfinite(scale)) return;       // a gradient was not finite: nothing is written
  }
  float step_size = sc.step_size, inv_bc2 = sc.inv_bc2, decay = sc.decay;
  uint32_t step = sc.step;
  if (sc.step_ptr != nullptr || sc.lr_ptr != nullptr) {
    __shared__ float dyn[3];
    __shared__ uint32_t dyn_step;
    __shared__ int dyn_ok;
    if (threadIdx.x == 0) {
      const int64_t t = sc.step_ptr != nullptr ? *sc.step_ptr : 0;
      const double lr = sc.lr_ptr != nullptr ? static_cast<double>(*sc.lr_ptr) : sc.lr;
      dyn_ok = (sc.step_ptr == nullptr || t >= 1) && isfinite(lr);
      dyn_step = sc.step_ptr != nullptr ? static_cast<uint32_t>(t) : sc.step;
      // host-side bias corrections stand in step_size / lr and inv_bc2
      const double bc1 = sc.step_ptr != nullptr ? -expm1(static_cast<double>(t) * sc.ln_beta1) : 0.0;
      const double bc2 = sc.step_ptr != nullptr ? -expm1(static_cast<double>(t) * sc.ln_beta2) : 0.0;
      dyn[0] = static_cast<float>(sc.step_ptr != nullptr ? lr / bc1 : lr * static_cast<double>(sc.step_size));
      dyn[1] = sc.step_ptr != nullptr ? static_cast<float>(1.0 / sqrt(bc2)) : sc.inv_bc2;
      dyn[2] = static_cast<float>(1.0 - lr * sc.wd);
    }
    __syncthreads();
    if (!dyn_ok) return;
    step_size = dyn[0]; inv_bc2 = dyn[1]; decay = dyn[2];
    step = dyn_step;
  }
  // the fast path flushes a root below 2^-63 to zero: eps has to cover it
  const bool eps_covers = sc.eps >= 2e-12f * inv_bc2;
  const uint32_t key = STOCH ? mix32(mix32(sc.seed_key + step) + ch.id) : 0u;
  const bool vec = aligned(ch.param, 16) && aligned(grad, 16) && aligned(ch.copy, 16) &&
                   aligned(ch.m, S8 ? 8 : 16) && aligned(ch.v, S8 ? 8 : 16);
  const int lane = threadIdx.x & 31;
  const int count = ch.count;
  for (int b = threadIdx.x >> 5; b * Q_BLOCK < count; b += ST_THREADS / 32) {
    const int e = b * Q_BLOCK + lane * 8;
    const int n = min(8, count - e);
    const bool full = vec && n == 8;
    float g[8], p[8], m[8], v[8];
    char* pp = static_cast<char*>(ch.param) + int64_t(e) * (PBF16 ? 2 : 4);
    if (full) {
      load8_vec<GBF16>(grad + int64_t(e) * (GBF16 ? 2 : 4), g);
      load8_vec<PBF16>(pp, p);
    } else {
      load8_some<GBF16>(grad + int64_t(e) * (GBF16 ? 2 : 4), n, g);
      load8_some<PBF16>(pp, n, p);
    }
    if (S8) {
      uint32_t mw[2], vw[2];
      load8_codes(static_cast<char*>(ch.m) + e, full, n, mw);
      load8_codes(static_cast<char*>(ch.v) + e, full, n, vw);
      decode8_m(mw, ch.m_scale[b], m);
      decode8_v(vw, ch.v_scale[b], v);
    } else if (full) {
      load8_vec<0>(static_cast<float*>(ch.m) + e, m);
      load8_vec<0>(static_cast<float*>(ch.v) + e, v);
    } else {
      load8_some<0>(static_cast<float*>(ch.m) + e, n, m);
      load8_some<0>(static_cast<float*>(ch.v) + e, n, v);
    }
    adam_moments8(m, v, g, scale, sc);
    if (eps_covers) adam_param8<true>(p, m, v, decay, step_size, inv_bc2, sc.eps);
    else adam_param8<false>(p, m, v, decay, step_size, inv_bc2, sc.eps);
    uint32_t h[4] = {};
    if (STOCH) {
#pragma unroll
      for (int k = 0; k < 4; ++k) h[k] = pair_bits(static_cast<uint64_t>(ch.base + e) / 2 + k, key);
    }
    if (n > 0) {
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
        store8_u16(pp, w, full, n);
      } else if (PBF16 || ch.copy != nullptr) {
#pragma unroll
        for (int k = 0; k < 4; ++k) w[k] = pack_bf16x2(p[2 * k], p[2 * k + 1]);
        store8_u16(PBF16 ? static_cast<void*>(pp) : static_cast<void*>(ch.copy + e), w, full, n);
      }
      if (!PBF16) store8_f32(reinterpret_cast<float*>(pp), p, full, n);
    }
    if (S8) {
      // past the end m is 0 (no code, no gradient), but a code 0 of v is not
      if (n < 8) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (k >= n) v[k] = 0.f;
      }
      const uint32_t mbits = __reduce_max_sync(0xffffffffu, __float_as_uint(max_abs8(m)));
      const uint32_t vbits = __reduce_max_sync(0xffffffffu, __float_as_uint(max_abs8(v)));
      float minv, rinv;
      const float mscale = block_scale(mbits, 1.f / 16129.f, minv);
      // roots keep order, so the largest root is the root of the largest
      const float rscale = block_scale(__float_as_uint(__fsqrt_rn(__uint_as_float(vbits))), 1.f / 65536.f, rinv);
      if (lane == 0) {
        ch.m_scale[b] = mscale;
        ch.v_scale[b] = rscale;
      }
      uint32_t mw[2] = {0, 0}, vw[2] = {0, 0};
      if (fast_block(mbits, vbits)) {
        encode8_m_fast<STOCH>(m, minv, h, mw);
        encode8_r_fast<STOCH>(v, rinv, h, vw);
      } else {
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
      if (n > 0) {
        store8_codes(static_cast<char*>(ch.m) + e, mw, full, n);
        store8_codes(static_cast<char*>(ch.v) + e, vw, full, n);
      }
    } else if (n > 0) {
      store8_f32(static_cast<float*>(ch.m) + e, m, full, n);
      store8_f32(static_cast<float*>(ch.v) + e, v, full, n);
    }
  }
}

// ---------------------------------------------------------------------------
// conversion
// ---------------------------------------------------------------------------
struct alignas(16) Q8Chunk {
  void* values;            // fp32 or bf16 moments
  void* codes;             // int8 first moments or uint8 second moments
  float* scales;
  uint16_t count;          // 1 .. ST_CHUNK
  uint8_t second;          // 1: second moments
  uint8_t bf16;            // values' type
  uint32_t pad;
};
static_assert(sizeof(Q8Chunk) == 32, "one chunk is one sector");

// PACK: values -> codes and scales, rounded to nearest.  Else the values that
// the codes stand for, rounded once to the values' type.
template <bool PACK>
__global__ void __launch_bounds__(ST_THREADS)
    state8_kernel(const Q8Chunk* __restrict__ chunks, const int* flags) {
  const Q8Chunk ch = chunks[blockIdx.x];
  pdl_wait();
  if (halted(flags)) return;
  const int lane = threadIdx.x & 31;
  const int count = ch.count;
  const bool vec = aligned(ch.values, 16) && aligned(ch.codes, 8);
  for (int b = threadIdx.x >> 5; b * Q_BLOCK < count; b += ST_THREADS / 32) {
    const int e = b * Q_BLOCK + lane * 8;
    const int n = min(8, count - e);
    const bool full = vec && n == 8;
    char* vp = static_cast<char*>(ch.values) + int64_t(e) * (ch.bf16 ? 2 : 4);
    float x[8];
    uint32_t w[2] = {0, 0};
    if (PACK) {
      if (ch.bf16) {
        if (full) load8_vec<1>(vp, x); else load8_some<1>(vp, n, x);
      } else {
        if (full) load8_vec<0>(vp, x); else load8_some<0>(vp, n, x);
      }
      uint32_t bits = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (ch.second) x[k] = __fsqrt_rn(x[k]);
        bits = max(bits, __float_as_uint(x[k]) & 0x7FFFFFFFu);   // 0 past the end
      }
      bits = __reduce_max_sync(0xffffffffu, bits);
      float inv;
      const float s = block_scale(bits, ch.second ? 1.f / 65536.f : 1.f / 16129.f, inv);
      if (lane == 0) ch.scales[b] = s;
#pragma unroll
      for (int k = 0; k < 8; ++k)
        w[k >> 2] |= (ch.second ? encode_r(x[k], inv, 0.5f) : encode_m(x[k], inv, 0.5f)) << (8 * (k & 3));
      if (n > 0) store8_codes(static_cast<char*>(ch.codes) + e, w, full, n);
    } else {
      load8_codes(static_cast<char*>(ch.codes) + e, full, n, w);
      const float s = ch.scales[b];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint32_t c = (w[k >> 2] >> (8 * (k & 3))) & 0xFFu;
        if (ch.second) {
          const float r = decode_r(c, s);
          x[k] = __fmul_rn(r, r);
        } else {
          x[k] = decode_m(c, s);
        }
      }
      if (n > 0) {
        if (ch.bf16) {
          uint32_t o[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) o[k] = pack_bf16x2(x[2 * k], x[2 * k + 1]);
          store8_u16(vp, o, full, n);
        } else {
          store8_f32(reinterpret_cast<float*>(vp), x, full, n);
        }
      }
    }
  }
}

// ---------------------------------------------------------------------------
// gradient norm
// ---------------------------------------------------------------------------
constexpr int NORM_CHUNK = 8192;
constexpr int NORM_BLOCKS_PER_SM = 8;

struct NormChunk {
  int64_t base;
  uint16_t slot;
  uint16_t count;          // 1 .. NORM_CHUNK
  uint8_t bf16;
  uint8_t pad[3];
};
static_assert(sizeof(NormChunk) == 16, "");

// Sum of squares of up to 8 elements in 64 bits.  fp32 holds it to 2^-22 when
// it lies well inside fp32's range; else (tiny or huge gradients) the squares
// are formed in 64 bits.
__device__ __forceinline__ double squares8(const float (&x)[8]) {
  float s = 0.f;
  uint32_t any = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    s = fmaf(x[k], x[k], s);
    any |= __float_as_uint(x[k]) << 1;
  }
  if (s > 1e-25f && s < 1e37f) return static_cast<double>(s);
  if (any == 0) return 0.0;
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
    s = threadIdx.x < ST_THREADS / 32 ? red[threadIdx.x] : 0.0;
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

__global__ void __launch_bounds__(ST_THREADS)
    grad_norm_kernel(const NormChunk* __restrict__ chunks, unsigned int nchunks,
                     const __grid_constant__ GradPtrs grads, const NormOut o) {
  __shared__ double red[ST_THREADS / 32];
  __shared__ bool last;
  pdl_wait();
  double acc = 0.0;
  for (unsigned int c = blockIdx.x; c < nchunks; c += gridDim.x) {
    const NormChunk ch = chunks[c];
    const int size = ch.bf16 ? 2 : 4;
    const char* g = static_cast<const char*>(grads.p[ch.slot]) + ch.base * size;
    const bool vec = aligned(g, 16);
#pragma unroll
    for (int it = 0; it < NORM_CHUNK / (8 * ST_THREADS); ++it) {
      const int e = (it * ST_THREADS + threadIdx.x) * 8;
      const int n = min(8, int(ch.count) - e);
      float x[8];
      if (n <= 0) continue;
      if (ch.bf16) {
        if (vec && n == 8) load8_vec<1>(g + int64_t(e) * 2, x); else load8_some<1>(g + int64_t(e) * 2, n, x);
      } else {
        if (vec && n == 8) load8_vec<0>(g + int64_t(e) * 4, x); else load8_some<0>(g + int64_t(e) * 4, n, x);
      }
      acc += squares8(x);
    }
  }
  const double mine = block_sum_f64(acc, red);
  if (threadIdx.x == 0) {
    if (nchunks > 0) o.partials[o.first + blockIdx.x] = mine;
    __threadfence();
    // wraps to 0 when every block has come by
    last = o.total == 0 || atomicInc(o.counter, o.total - 1) == o.total - 1;
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  double sum = 0.0;
  for (unsigned int i = threadIdx.x; i < o.total; i += ST_THREADS) sum += __ldcg(o.partials + i);
  sum = block_sum_f64(sum, red);
  if (threadIdx.x == 0) {
    const float norm = static_cast<float>(sqrt(sum));
    o.out[0] = norm;
    // a norm that is not finite leaves no factor: steps that read it write nothing
    o.out[1] = isfinite(norm) ? static_cast<float>(fmin(1.0, o.max_norm / (sqrt(sum) + 1e-6))) : __uint_as_float(0x7FC00000u);
  }
}

}  // namespace muon
