// AdamW over many tensors in one launch, with states in 32 or in 8 bits.
//
// Per element, in fp32 (every product and sum of m and v rounded on its own,
// so that they do not depend on the compiler's contraction):
//   g' = g * grad_scale
//   m  = m * b1 + g' * (1 - b1)         v = v * b2 + (g' * g') * (1 - b2)
//   w  = w * (1 - lr * wd) - m / (sqrt(v) / sqrt(1 - b2^t) + eps) * lr / (1 - b1^t)
// w is the fp32 master copy, or the parameter widened; the parameter is w
// rounded once to its type.
//
// 8-bit states.  256 consecutive elements share an exponent byte E, the
// exponent field of their largest magnitude once rounded up to 3 mantissa
// bits, so no element rounds past the largest code.  m keeps a sign and 7 bits
// c (4 exponent, 3 mantissa), v 8 bits c (5 exponent, 3 mantissa); c = 0 is
// zero, any other c the float with bits ((E - 15) << 23) + (c << 20), for v
// ((E - 31) << 23) + (c << 20).  Decoding is a shift and an add, and the
// bits of a float above the block's base round to a code by one add and one
// shift.  The rounding is stochastic (the 20 bits dropped against 20 random
// bits hashed from the seed, the tensor and the element): with 3 mantissa bits
// and b2 = 0.999 a nearest rounding would return v to the same code every
// step and never let it decay, while this one keeps its expectation.  E = 255
// marks a block that held an infinity or NaN: all of it reads as NaN.
//
// Bound by HBM: with a bf16 parameter and gradient and an fp32 master 28
// bytes an element with 32-bit states, 16 with 8-bit ones.  Measured on 151 M
// parameters: 0.84 ms = 5.04 TB/s with 32-bit states, 0.48-0.51 ms = 4.7-5.0
// TB/s with 8-bit ones (a copy of 1 GiB reaches 5.17); 16.5 k parameters in five
// tensors: 4.8 us.
#include "device_common.h"
#include "fp8ds.h"
#include "launch.h"

#pragma clang fp contract(off)

namespace fp8ds {

namespace {

typedef unsigned int v4u __attribute__((ext_vector_type(4)));
typedef unsigned int v2u __attribute__((ext_vector_type(2)));

constexpr int kAThreads = 256;
constexpr int kStateBlock = FP8DS_ADAMW_BLOCK;         // elements that share an exponent byte
constexpr int kPerLane = 8;                            // half a wave holds one such block
constexpr int kTile = kAThreads * kPerLane;            // elements of one pass of a workgroup
constexpr int kTilesPerGroup = 2;
constexpr int kMaxTensors = 48;                        // the table has to fit the kernel arguments

struct AdamTensor {
  void* p;
  const void* g;
  void* m;
  void* v;
  float* w;
  uint8_t* me;
  uint8_t* ve;
  const int32_t* step;           // the device step count, or null
  uint32_t numel;
  uint32_t key;      // seed and tensor number, mixed on the host
};

struct AdamArgs {
  AdamTensor t[kMaxTensors];
  uint32_t first[kMaxTensors];   // first workgroup of each tensor; unused entries hold ~0
  float b1, b2, c1, c2;          // betas and 1 - betas
  float decay, step_size, inv_sqrt_bc2, eps;
  const float* grad_scale;
  const float* lr_dev;           // with it or a tensor's step, decay, step_size and
                                 // inv_sqrt_bc2 are formed in the kernel
  float lr, wd, ln_b1, ln_b2;
  int32_t step;
};
static_assert(sizeof(AdamArgs) <= 4096, "kernel arguments");

// 32 random bits for element i: an add and two multiplications by odd numbers
// (the fractions of the golden ratio and of the square roots of 2 and 3),
// each followed by a shift that folds the high bits down.
constexpr uint32_t kGolden = 0x9E3779B1u, kRoot2 = 0x6A09E667u, kRoot3 = 0xBB67AE85u;
__device__ __forceinline__ uint32_t hash32(uint32_t i, uint32_t key) {
  uint32_t x = i * kGolden + key;
  x = (x ^ (x >> 16)) * kRoot2;
  x = (x ^ (x >> 15)) * kRoot3;
  return x ^ (x >> 16);
}

template <int T>
__device__ __forceinline__ float widen(uint32_t bits) {
  if constexpr (T == kInBf16) return __uint_as_float(bits << 16);
  else if constexpr (T == kInF16) return (float)__builtin_bit_cast(_Float16, (uint16_t)bits);
  else return __uint_as_float(bits);
}

template <int T>
__device__ __forceinline__ uint32_t narrow(float x) {
  if constexpr (T == kInBf16) return __builtin_bit_cast(uint16_t, (__bf16)x);
  else if constexpr (T == kInF16) return __builtin_bit_cast(uint16_t, (_Float16)x);
  else return __float_as_uint(x);
}

// Eight consecutive elements of type T as bit patterns.  full: one or two
// aligned 16-byte accesses; else element by element, those at or past n left out.
template <int T>
__device__ __forceinline__ void load8(const void* base, uint32_t i, uint32_t n, bool full, uint32_t (&x)[8]) {
  if constexpr (T == kInF32) {
    const uint32_t* p = static_cast<const uint32_t*>(base) + i;
    if (full) {
      const v4u a = __builtin_nontemporal_load(reinterpret_cast<const v4u*>(p));
      const v4u b = __builtin_nontemporal_load(reinterpret_cast<const v4u*>(p) + 1);
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = a[e], x[4 + e] = b[e];
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = i + e < n ? p[e] : 0u;
    }
  } else {
    const uint16_t* p = static_cast<const uint16_t*>(base) + i;
    if (full) {
      const v4u a = __builtin_nontemporal_load(reinterpret_cast<const v4u*>(p));
#pragma unroll
      for (int e = 0; e < 4; ++e) x[2 * e] = a[e] & 0xFFFFu, x[2 * e + 1] = a[e] >> 16;
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = i + e < n ? p[e] : 0u;
    }
  }
}

template <int T>
__device__ __forceinline__ void store8(void* base, uint32_t i, uint32_t n, bool full, const uint32_t (&x)[8]) {
  if constexpr (T == kInF32) {
    uint32_t* p = static_cast<uint32_t*>(base) + i;
    if (full) {
      __builtin_nontemporal_store(v4u{x[0], x[1], x[2], x[3]}, reinterpret_cast<v4u*>(p));
      __builtin_nontemporal_store(v4u{x[4], x[5], x[6], x[7]}, reinterpret_cast<v4u*>(p) + 1);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (i + e < n) p[e] = x[e];
    }
  } else {
    uint16_t* p = static_cast<uint16_t*>(base) + i;
    if (full) {
      __builtin_nontemporal_store(
          v4u{x[0] | x[1] << 16, x[2] | x[3] << 16, x[4] | x[5] << 16, x[6] | x[7] << 16},
          reinterpret_cast<v4u*>(p));
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (i + e < n) p[e] = (uint16_t)x[e];
    }
  }
}

__device__ __forceinline__ void load8_codes(const void* base, uint32_t i, uint32_t n, bool full, uint32_t (&x)[8]) {
  const uint8_t* p = static_cast<const uint8_t*>(base) + i;
  if (full) {
    const v2u a = __builtin_nontemporal_load(reinterpret_cast<const v2u*>(p));
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = (a[e / 4] >> (8 * (e % 4))) & 0xFFu;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = i + e < n ? p[e] : 0u;
  }
}

__device__ __forceinline__ void store8_codes(void* base, uint32_t i, uint32_t n, bool full, const uint32_t (&x)[8]) {
  uint8_t* p = static_cast<uint8_t*>(base) + i;
  if (full) {
    __builtin_nontemporal_store(v2u{x[0] | x[1] << 8 | x[2] << 16 | x[3] << 24,
                                    x[4] | x[5] << 8 | x[6] << 16 | x[7] << 24},
                                reinterpret_cast<v2u*>(p));
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (i + e < n) p[e] = (uint8_t)x[e];
  }
}

template <bool SIGNED>
constexpr uint32_t kSpan = SIGNED ? 15u : 31u;   // exponents below the block's largest that codes reach

// The float a code stands for, as bits.
template <bool SIGNED>
__device__ __forceinline__ uint32_t decode_bits(uint32_t code, uint32_t exp) {
  const uint32_t mag = SIGNED ? code & 0x7Fu : code;
  uint32_t b = mag == 0 ? 0u : ((exp - kSpan<SIGNED>) << 23) + (mag << 20);
  if (exp == 255u) b = 0x7FC00000u;
  return SIGNED ? b | (code & 0x80u) << 24 : b;
}

// Rounds eight values of one block (each half wave holds a block) to codes;
// returns its exponent byte.  r: 20 random bits an element.
template <bool SIGNED>
__device__ __forceinline__ uint32_t encode8(const float (&x)[8], const uint32_t (&r)[8], uint32_t (&code)[8]) {
  constexpr uint32_t kTop = SIGNED ? 127u : 255u;
  uint32_t top = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(x[e]) & 0x7FFFFFFFu);
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, d, 32));
  // Rounded up to 3 mantissa bits; blocks of tiny values share the lowest
  // exponent that keeps the smallest code a normal float.
  const uint32_t exp = top == 0 ? 0u : min(max((top + 0xFFFFFu) >> 23, kSpan<SIGNED> + 1), 255u);
  const uint32_t base = (exp - kSpan<SIGNED>) << 23;
  const float foot = __uint_as_float(base + (1u << 20));   // what code 1 stands for
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint32_t bits = __float_as_uint(x[e]) & 0x7FFFFFFFu;
    const int32_t t = (int32_t)(bits - base);
    // Below code 1 the neighbours are 0 and 1: r / 2^20 * foot is exact (20 bits times 9/8).
    const uint32_t low = (float)r[e] * 0x1p-20f * foot < __uint_as_float(bits) ? 1u : 0u;
    uint32_t c = t < (1 << 20) ? low : min((uint32_t)(t + (int32_t)r[e]) >> 20, kTop);
    if (top == 0) c = 0;
    if (SIGNED && c != 0) c |= (__float_as_uint(x[e]) >> 24) & 0x80u;
    code[e] = c;
  }
  return exp;
}

template <int PT, int GT, bool MASTER, int BITS>
__global__ __launch_bounds__(kAThreads) void adamw_kernel(AdamArgs a) {
  // This workgroup's tensor: lane l compares entry l's first workgroup.
  const int lane = threadIdx.x & 63;
  const uint32_t wg = blockIdx.x;
  const uint32_t mine = lane < kMaxTensors ? a.first[lane] : ~0u;
  const int ti = __builtin_amdgcn_readfirstlane(__popcll(__ballot(mine <= wg)) - 1);
  const AdamTensor& t = a.t[ti];
  const uint32_t n = t.numel;
  uint32_t key = t.key;
  float decay = a.decay, step_size = a.step_size, inv_sqrt_bc2 = a.inv_sqrt_bc2;
  if (a.lr_dev || t.step) {
    const float lr = a.lr_dev ? *a.lr_dev : a.lr;
    const int32_t step = t.step ? *t.step : a.step;
    // 1 - b^t = -expm1(t ln b)
    decay = 1.0f - lr * a.wd;
    step_size = lr / -expm1f((float)step * a.ln_b1);
    inv_sqrt_bc2 = 1.0f / sqrtf(-expm1f((float)step * a.ln_b2));
    if (t.step) key += (uint32_t)step * kRoot2;
  }
  const float gs = a.grad_scale ? *a.grad_scale : 1.0f;
  const uintptr_t all = reinterpret_cast<uintptr_t>(t.p) | reinterpret_cast<uintptr_t>(t.g) |
                        reinterpret_cast<uintptr_t>(t.m) | reinterpret_cast<uintptr_t>(t.v) |
                        (MASTER ? reinterpret_cast<uintptr_t>(t.w) : 0);
  const bool aligned = (all & 15u) == 0;
  const uint64_t i0 = (uint64_t)(wg - a.first[ti]) * (kTile * kTilesPerGroup) + threadIdx.x * kPerLane;
#pragma unroll
  for (int it = 0; it < kTilesPerGroup; ++it) {
    const uint64_t i64 = i0 + (uint64_t)it * kTile;
    // Half waves leave together: a state block is one half wave's 256 elements.
    if ((i64 & ~uint64_t(kStateBlock - 1)) >= n) break;
    const uint32_t i = (uint32_t)min(i64, (uint64_t)n);
    const bool full = aligned && i64 + kPerLane <= n;
    uint32_t gb[8], wb[8], mb[8], vb[8];
    load8<GT>(t.g, i, n, full, gb);
    if constexpr (MASTER) load8<kInF32>(t.w, i, n, full, wb);
    else load8<PT>(t.p, i, n, full, wb);
    uint32_t me = 0, ve = 0;
    if constexpr (BITS == 8) {
      load8_codes(t.m, i, n, full, mb);
      load8_codes(t.v, i, n, full, vb);
      me = t.me[i64 / kStateBlock];
      ve = t.ve[i64 / kStateBlock];
    } else {
      load8<kInF32>(t.m, i, n, full, mb);
      load8<kInF32>(t.v, i, n, full, vb);
    }
    float m[8], v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if constexpr (BITS == 8) {
        mb[e] = decode_bits<true>(mb[e], me);
        vb[e] = decode_bits<false>(vb[e], ve);
      }
      float g = widen<GT>(gb[e]);
      if (a.grad_scale) g = g * gs;
      m[e] = __uint_as_float(mb[e]) * a.b1 + g * a.c1;
      v[e] = __uint_as_float(vb[e]) * a.b2 + g * g * a.c2;
      float w = MASTER ? __uint_as_float(wb[e]) : widen<PT>(wb[e]);
      const float den = __builtin_amdgcn_sqrtf(v[e]) * inv_sqrt_bc2 + a.eps;
      w = w * decay - m[e] * __builtin_amdgcn_rcpf(den) * step_size;
      wb[e] = __float_as_uint(w);
      // Past the end of the tensor the state is zero, whatever was loaded.
      if (BITS == 8 && i64 + e >= n) m[e] = v[e] = 0.0f;
    }
    if constexpr (BITS == 8) {
      uint32_t r[8], c[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) r[e] = hash32((uint32_t)i64 + e, key);
      uint32_t rm[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) rm[e] = r[e] >> 12;
      const uint32_t me2 = encode8<true>(m, rm, c);
      store8_codes(t.m, i, n, full, c);
#pragma unroll
      for (int e = 0; e < 8; ++e) rm[e] = (r[e] * kGolden) >> 12;
      const uint32_t ve2 = encode8<false>(v, rm, c);
      store8_codes(t.v, i, n, full, c);
      if ((threadIdx.x & 31) == 0) {
        t.me[i64 / kStateBlock] = (uint8_t)me2;
        t.ve[i64 / kStateBlock] = (uint8_t)ve2;
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) mb[e] = __float_as_uint(m[e]), vb[e] = __float_as_uint(v[e]);
      store8<kInF32>(t.m, i, n, full, mb);
      store8<kInF32>(t.v, i, n, full, vb);
    }
    if constexpr (MASTER) store8<kInF32>(t.w, i, n, full, wb);
    uint32_t pb[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) pb[e] = narrow<PT>(__uint_as_float(wb[e]));
    store8<PT>(t.p, i, n, full, pb);
  }
}

// Codes to bf16: a code has 4 significant bits, so bf16 holds it exactly.  Bound
// by HBM: 151 M elements, 3 bytes each, in 76 us = 5.96 TB/s (right after the step
// that wrote the codes, part of which the last-level cache then still holds).
template <bool SIGNED>
__global__ __launch_bounds__(kAThreads) void state_values_kernel(const uint8_t* codes, const uint8_t* exps, int64_t n,
                                                                 uint16_t* out, bool aligned) {
  const int64_t step = (int64_t)gridDim.x * kTile;
  for (int64_t i = (int64_t)blockIdx.x * kTile + threadIdx.x * kPerLane; i < n; i += step) {
    const uint32_t exp = exps[i / kStateBlock];
    const uint32_t left = (uint32_t)min((int64_t)kPerLane, n - i);
    const bool full = aligned && left == kPerLane;
    uint32_t c[8];
    load8_codes(codes + i, 0, left, full, c);
#pragma unroll
    for (int e = 0; e < 8; ++e) c[e] = decode_bits<SIGNED>(c[e], exp) >> 16;
    store8<kInBf16>(out + i, 0, left, full, c);
  }
}

typedef void (*AdamFn)(AdamArgs);

template <int PT, int GT, bool MASTER>
AdamFn pick_bits(int bits) {
  return bits == 8 ? adamw_kernel<PT, GT, MASTER, 8> : adamw_kernel<PT, GT, MASTER, 32>;
}
template <int PT, int GT>
AdamFn pick_master(bool master, int bits) {
  return master ? pick_bits<PT, GT, true>(bits) : pick_bits<PT, GT, false>(bits);
}
template <int PT>
AdamFn pick_grad(int gt, bool master, int bits) {
  if (gt == kInBf16) return pick_master<PT, kInBf16>(master, bits);
  if (gt == kInF16) return pick_master<PT, kInF16>(master, bits);
  return pick_master<PT, kInF32>(master, bits);
}

}  // namespace

int launch_adamw(const fp8ds_adamw_tensor* ts, const int32_t* const* steps, int nt, const fp8ds_adamw_args& p,
                 bool master, hipStream_t stream) {
  AdamFn fn = p.param_type == kInBf16  ? pick_grad<kInBf16>(p.grad_type, master, p.state_bits)
              : p.param_type == kInF16 ? pick_grad<kInF16>(p.grad_type, master, p.state_bits)
                                       : pick_grad<kInF32>(p.grad_type, master, p.state_bits);
  AdamArgs a;
  a.b1 = (float)p.beta1;
  a.b2 = (float)p.beta2;
  a.c1 = (float)(1.0 - p.beta1);
  a.c2 = (float)(1.0 - p.beta2);
  a.eps = (float)p.eps;
  a.lr = (float)p.lr;
  a.wd = (float)p.weight_decay;
  a.ln_b1 = p.beta1 > 0 ? (float)__builtin_log(p.beta1) : -__builtin_inff();
  a.ln_b2 = p.beta2 > 0 ? (float)__builtin_log(p.beta2) : -__builtin_inff();
  a.step = (int32_t)p.step;
  a.decay = (float)(1.0 - p.lr * p.weight_decay);
  a.step_size = a.inv_sqrt_bc2 = 0.0f;
  if (!p.step_dev && !steps) {
    a.step_size = (float)(p.lr / (1.0 - __builtin_pow(p.beta1, (double)p.step)));
    a.inv_sqrt_bc2 = (float)(1.0 / __builtin_sqrt(1.0 - __builtin_pow(p.beta2, (double)p.step)));
  }
  a.grad_scale = p.grad_scale;
  a.lr_dev = p.lr_dev;
  int at = 0;
  while (at < nt) {
    int used = 0;
    uint64_t groups = 0;
    for (; at < nt && used < kMaxTensors; ++at) {
      const fp8ds_adamw_tensor& s = ts[at];
      if (s.numel == 0) continue;
      const uint64_t need = ((uint64_t)s.numel + kTile * kTilesPerGroup - 1) / (kTile * kTilesPerGroup);
      if (groups + need > 0x7FFFFFFFu) break;
      a.t[used] = AdamTensor{s.p, s.g, s.exp_avg, s.exp_avg_sq, s.master, s.exp_avg_exp, s.exp_avg_sq_exp,
                             steps ? steps[at] : p.step_dev, (uint32_t)s.numel, p.seed ^ (uint32_t)at * kRoot3};
      a.first[used] = (uint32_t)groups;
      groups += need;
      ++used;
    }
    for (int i = used; i < kMaxTensors; ++i) a.first[i] = ~0u;
    if (groups == 0) continue;
    hipLaunchKernelGGL(fn, dim3((unsigned)groups), dim3(kAThreads), 0, stream, a);
    if (const int st = check_launch("adamw_kernel")) return st;
  }
  return FP8DS_OK;
}

int launch_adamw_state_values(const uint8_t* codes, const uint8_t* exps, int64_t n, bool is_signed, void* out,
                              hipStream_t stream) {
  const bool aligned = ((reinterpret_cast<uintptr_t>(codes) | reinterpret_cast<uintptr_t>(out)) & 15u) == 0;
  const int64_t blocks = (n + kTile - 1) / kTile;
  const dim3 grid((unsigned)(blocks < 16384 ? blocks : 16384));
  if (is_signed)
    hipLaunchKernelGGL(state_values_kernel<true>, grid, dim3(kAThreads), 0, stream, codes, exps, n,
                       static_cast<uint16_t*>(out), aligned);
  else
    hipLaunchKernelGGL(state_values_kernel<false>, grid, dim3(kAThreads), 0, stream, codes, exps, n,
                       static_cast<uint16_t*>(out), aligned);
  return check_launch("state_values_kernel");
}

}  // namespace fp8ds
