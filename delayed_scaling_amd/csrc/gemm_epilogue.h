// The scaled FP8 GEMM with an activation epilogue:
//   z = acc * alpha + bias;  C = bf16(act(z) + residual), optionally Z = bf16(z)
// or, for the backward pass of such a product,
//   C = bf16(acc * alpha * act'(Z))
// with Z the bf16 pre-activation its forward stored.  acc, z and act(z) stay
// in fp32; C and Z are each rounded once.
//
// The bodies are those of gemm_kernel.h; only the store of a finished tile
// differs.  Each wave passes its accumulators through its share of the stage
// buffer the tile's last stage freed as fp32, in pieces of 32 rows by 32 (16
// on the 64x64 tile) columns, and reads them back row by row, 8 columns a lane:
// in that layout the residual or Z, the bias and the results are 16-byte
// accesses of neighbouring lanes, the activation runs once per element on
// eight of them at a time, and rows or columns outside C are one comparison, so
// edge tiles take the same path.
//
// Cost beside the product: 2 bytes an element for each of C, Z and the
// residual, and about 20 vector instructions an element for GELU, which at
// K = 1024 is a third of the MFMA time and overlaps it only across the
// workgroups that share a CU.  Measured (E4M3, 2048x4096x1024): 15.9 us with no
// epilogue, 19.4 with GELU, 20.5 with bias, GELU and Z kept, 19.8 for GELU's
// slope; 8192x1024x4096: 35.4, 38.4, 39.6, 45.5, with a residual 44.4 (37-38
// with the residual still in the last-level cache).
#pragma once

#include "gemm_kernel.h"

namespace fp8ds {

// Also the activation numbers of fp8ds_act.
constexpr int kActNone = 0, kActRelu = 1, kActGelu = 2, kActGeluTanh = 3, kActSilu = 4;

struct GemmEpiKArgs : GemmKArgs {
  const uint16_t* extra;      // residual, or Z when grad is set; may be null without grad
  uint16_t* preact;           // Z to store, or null
  int64_t ld_extra, stride_extra, ld_preact, stride_preact;
  int act, grad;
};

typedef void (*GemmEpiFn)(GemmEpiKArgs);
// Pickers, one per layout: tiles 6 (256x256, eight waves), 7 and 8 (the
// 128x128 and 64x64 unit tiles).
GemmEpiFn gemm_epi_fn_nt(int tile, int fa, int fb);
GemmEpiFn gemm_epi_fn_nn(int tile, int fa, int fb);
GemmEpiFn gemm_epi_fn_tn(int tile, int fa, int fb);

// The kernel's arguments, read again from the kernel-argument segment where a
// tile begins and ends: kept in scalar registers through the K loop, with what
// the epilogue needs, they push the loop's own values out to vector lanes.
static __device__ __forceinline__ GemmEpiKArgs late_args() {
  typedef __attribute__((address_space(4))) const uint64_t karg_t;
  uint64_t a = (uint64_t)(uintptr_t)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(a));
  struct Words {
    uint64_t w[sizeof(GemmEpiKArgs) / 8];
  } t;
#pragma unroll
  for (unsigned i = 0; i < sizeof(t) / 8; ++i) t.w[i] = ((karg_t*)(uintptr_t)a)[i];
  return __builtin_bit_cast(GemmEpiKArgs, t);
}

static __device__ __forceinline__ GemmEpiKArgs tile_args(const GemmEpiKArgs&) { return late_args(); }

namespace {

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float sigmoid(float x) {
  return __builtin_amdgcn_rcpf(1.0f + exp2_fast(-1.4426950408889634f * x));
}

// The normal distribution's upper tail Q(|z|) and density exponential
// e = exp(-z^2 / 2): Q = e t P(t), t = 1 / (1 + 0.36 |z|), P a degree-6
// polynomial fitted here to least maximal relative error over [0, 14]
// (8.8e-7; 1.2e-6 as evaluated in fp32), so the tail keeps its relative
// precision where 1 + erf would cancel.
__device__ __forceinline__ float normal_tail(float z, float& e) {
  e = exp2_fast(-0.72134752044448170f * z * z);
  const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.36f, __builtin_fabsf(z), 1.0f));
  float q = 0.04705688f;
  q = __builtin_fmaf(q, t, -0.17976674f);
  q = __builtin_fmaf(q, t, 0.18095683f);
  q = __builtin_fmaf(q, t, 0.026547348f);
  q = __builtin_fmaf(q, t, 0.13972001f);
  q = __builtin_fmaf(q, t, 0.14177231f);
  q = __builtin_fmaf(q, t, 0.14371306f);
  return q * t * e;
}

constexpr float kTanhA = 0.7978845608028654f;   // sqrt(2 / pi)
constexpr float kTanhB = 0.044715f;

template <int ACT>
__device__ __forceinline__ float act_value(float z) {
  if constexpr (ACT == kActRelu) return z < 0.0f ? 0.0f : z;
  if constexpr (ACT == kActGelu) {
    float e;
    const float q = normal_tail(z, e);
    return z * (z < 0.0f ? q : 1.0f - q);
  }
  // 0.5 z (1 + tanh u) = z sigmoid(2 u)
  if constexpr (ACT == kActGeluTanh) return z * sigmoid(2.0f * kTanhA * z * __builtin_fmaf(kTanhB, z * z, 1.0f));
  if constexpr (ACT == kActSilu) return z * sigmoid(z);
  return z;
}

template <int ACT>
__device__ __forceinline__ float act_slope(float z) {
  if constexpr (ACT == kActRelu) return z > 0.0f ? 1.0f : 0.0f;
  if constexpr (ACT == kActGelu) {
    float e;
    const float q = normal_tail(z, e);
    return __builtin_fmaf(0.3989422804014327f * z, e, z < 0.0f ? q : 1.0f - q);
  }
  if constexpr (ACT == kActGeluTanh) {
    // (s (1 - s) is zero long before z^2 would overflow; the two may not meet.)
    const float zz = __builtin_fminf(z * z, 0x1p64f);
    const float s = sigmoid(2.0f * kTanhA * z * __builtin_fmaf(kTanhB, zz, 1.0f));
    return __builtin_fmaf(z * s * (1.0f - s), 2.0f * kTanhA * __builtin_fmaf(3.0f * kTanhB, zz, 1.0f), s);
  }
  if constexpr (ACT == kActSilu) {
    const float s = sigmoid(z);
    return s * __builtin_fmaf(z, 1.0f - s, 1.0f);
  }
  return 1.0f;
}

template <int N>
struct Int {
  static constexpr int value = N;
};

// Calls f with the activation and the direction as constants.
template <class F>
__device__ __forceinline__ void with_act(const GemmEpiKArgs& p, const F& f) {
  if (p.grad) {
    switch (p.act) {
      case kActRelu: return f(Int<kActRelu>{}, Int<1>{});
      case kActGelu: return f(Int<kActGelu>{}, Int<1>{});
      case kActGeluTanh: return f(Int<kActGeluTanh>{}, Int<1>{});
      case kActSilu: return f(Int<kActSilu>{}, Int<1>{});
      default: return f(Int<kActNone>{}, Int<0>{});   // a slope of 1: refused by the host with an operand
    }
  }
  switch (p.act) {
    case kActRelu: return f(Int<kActRelu>{}, Int<0>{});
    case kActGelu: return f(Int<kActGelu>{}, Int<0>{});
    case kActGeluTanh: return f(Int<kActGeluTanh>{}, Int<0>{});
    case kActSilu: return f(Int<kActSilu>{}, Int<0>{});
    default: return f(Int<kActNone>{}, Int<0>{});
  }
}

__device__ __forceinline__ float bias_one(const GemmKArgs& p, int n) {
  if (p.bias_kind == 0) return 0.0f;
  if (p.bias_kind == 1) return __uint_as_float((uint32_t) static_cast<const uint16_t*>(p.bias)[n] << 16);
  if (p.bias_kind == 2) return static_cast<const float*>(p.bias)[n];
  const int c = static_cast<const uint8_t*>(p.bias)[n];
  return (p.bias_kind == 3 ? __builtin_amdgcn_cvt_f32_fp8(c, 0) : __builtin_amdgcn_cvt_f32_bf8(c, 0)) *
         p.bias_scale_inv[0];
}

// `left` (8 or fewer) 16-bit values to dst, 16 bytes at once when all are there.  The stores are streaming ones: with plain stores the epilogue
// alone ran 6 us longer at 8192x1024x4096 (41.4 against 35.2 us) and 12 us at
// 8192x4096x1024 (57.0 against 44.8).
__device__ __forceinline__ void store8_row(uint16_t* dst, int left, v4i x) {
  if (left >= 8) {
    __builtin_nontemporal_store(x, reinterpret_cast<v4i*>(dst));
    return;
  }
#pragma unroll
  for (int e = 0; e < 7; ++e)
    if (e < left) dst[e] = (uint16_t)((uint32_t)x[e / 2] >> (16 * (e & 1)));
}

}  // namespace

// The store of one wave's block of output tile v, for the bodies of
// gemm_kernel.h (same contract: `stage_buf` is the freed stage buffer, of
// which the wave uses the 1 KiB pieces its own next loads refill).  Returns
// false: the number of its memory operations varies.  (In GemmEpiKArgs's own
// namespace, where the bodies' calls look for it by their argument.)
template <int BM, int BN, int TM, int TN, int NW, int LPS, bool DRAIN = false>
static __device__ __forceinline__ bool store_c_tile(const GemmEpiKArgs&, const v16f (&acc)[TN][TM], int v, int r0, int c0,
                                             int lane, int wave, float alpha, bool staged, lds_char_t* stage_buf) {
  static_assert(sizeof(GemmEpiKArgs) % 8 == 0, "read in 8-byte words");
  const GemmEpiKArgs p = late_args();
  int bt, tmi, tni;
  map_tile(p, v, bt, tmi, tni);
  const int m0 = tmi * BM + r0, n0 = tni * BN + c0;
  uint16_t* cb = p.c + bt * p.stride_c;
  const uint16_t* xb = p.extra ? p.extra + bt * p.stride_extra : nullptr;
  uint16_t* zb = p.preact ? p.preact + bt * p.stride_preact : nullptr;
  if (!staged) {
    // K = 0: the product is zero, so z is the bias alone.
    with_act(p, [&](auto act, auto grad) {
      constexpr int A = decltype(act)::value;
      for (int i = lane; i < TM * 32 * TN * 32; i += 64) {
        const int m = m0 + i / (TN * 32), n = n0 + i % (TN * 32);
        if (m >= p.m || n >= p.n) continue;
        const float z = bias_one(p, n);
        const float x = xb ? __uint_as_float((uint32_t)xb[m * p.ld_extra + n] << 16) : 0.0f;
        const float y = decltype(grad)::value ? 0.0f * act_slope<A>(x) : act_value<A>(z) + x;
        if (zb) zb[m * p.ld_preact + n] = (uint16_t)pack_bf16x2(z, 0.0f);
        cb[m * p.ldc + n] = (uint16_t)pack_bf16x2(y, 0.0f);
      }
    });
    return false;
  }

  constexpr int SC = LPS * 1024 >= 32 * 32 * 4 ? 32 : 16;     // columns of a piece
  constexpr int RB = SC * 4, CH = RB / 16, RPP = 1024 / RB;   // bytes and 16-byte chunks of a row, rows per KiB
  constexpr int LR = SC / 8, RPI = 64 / LR, NR = 32 / RPI;    // lanes per row, rows per read, reads
  static_assert(32 * RB <= LPS * 1024, "staging area");
  const uint32_t sbase = lds_address(stage_buf) + (uint32_t)wave * 1024u;
  auto row_at = [&](uint32_t r) __attribute__((always_inline)) {
    return sbase + (r / RPP) * (NW * 1024u) + (r % RPP) * RB;
  };
  // Chunks are XOR-swizzled by row pairs (quads of the shorter rows): 16 rows
  // of one chunk fall into distinct banks.
  auto chunk_at = [&](uint32_t r, uint32_t c) __attribute__((always_inline)) {
    return row_at(r) + ((c ^ ((r / (256 / RB)) % CH)) << 4);
  };
  const uint32_t wr = lane & 31, wh = lane >> 5;              // as the MFMA left them: row, 4-column half
  const int rr = lane / LR, rc = lane % LR;                   // as read back
  // What a piece needs beside the accumulators: the residual is requested one
  // or two pieces ahead, the bias, which other tiles have left in the caches, one.
  struct Side {
    v4f b0, b1;
  };
  constexpr int AHEAD = TM * TN == 4 ? 2 : 1;     // (what the tile's registers leave room for)
  v4i x[AHEAD + 1][NR] = {};
  constexpr int PIECES = (TN * 32 / SC) * TM;
  const bool has_bias = p.bias_kind != 0;
  // Through a buffer descriptor that ends with the matrix (to the dword its last
  // element is in): no branch, so nothing waits for a load before its use.  What
  // lies past column N of a row is read, from the next row, and not used.
  const int64_t x0 = (int64_t)m0 * p.ld_extra + n0;
  const int64_t x_left = ((int64_t)(p.m - 1) * p.ld_extra + p.n - x0) * 2;
  const __amdgpu_buffer_rsrc_t x_rsrc =
      make_rsrc(xb + x0, xb && x_left > 0 ? (uint32_t)(((x_left < 0x7FFFFFF0 ? x_left : 0x7FFFFFF0) + 3) & ~3ll) : 0u);
  const uint32_t x_row = (uint32_t)p.ld_extra * 2u, x_lane = (uint32_t)rr * x_row + (uint32_t)rc * 16u;
  auto fetch_extra = [&](v4i (&f)[NR], int i) __attribute__((always_inline)) {
    const uint32_t at = x_lane + (uint32_t)(32 * (i % TM)) * x_row + (uint32_t)(i / TM * SC) * 2u;
#pragma unroll
    for (int q = 0; q < NR; ++q)
      f[q] = __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(x_rsrc, at + (uint32_t)(q * RPI) * x_row, 0, 0));
  };
  auto fetch = [&](Side& f, int i) __attribute__((always_inline)) {
    const int n = n0 + i / TM * SC + 8 * rc, left = p.n - n;
    if (has_bias) {
      f.b0 = f.b1 = v4f{};
      if (left >= 8) {
        f.b0 = bias4_full(p, n);
        f.b1 = bias4_full(p, n + 4);
      } else {
#pragma unroll
        for (int e = 0; e < 7; ++e)
          if (e < left) (e < 4 ? f.b0 : f.b1)[e % 4] = bias_one(p, n + e);
      }
    }
  };
  Side now = {}, next = {};
  fetch(now, 0);
  if (xb) {
#pragma unroll
    for (int i = 0; i < AHEAD; ++i)
      if (i < PIECES) fetch_extra(x[i], i);
  }
  // (A loop over the pieces, so the nine activations make nine copies of one
  // piece's code and not of all; the unrolled sequence was no faster.)
#pragma unroll 1
  for (int i = 0; i < PIECES; ++i) {
    if (i + 1 < PIECES) fetch(next, i + 1);
    if (xb && i + AHEAD < PIECES) fetch_extra(x[AHEAD], i + AHEAD);
    // (Accumulators have no run-time index: one of these writes is taken.)
#pragma unroll
    for (int c = 0; c < PIECES; ++c) {
      if (c != i) continue;
      const v16f& a = acc[c / TM * SC / 32][c % TM];
#pragma unroll
      for (int g = 0; g < SC / 8; ++g) {
        const int rq = (c / TM * SC % 32) / 8 + g;
        *(__attribute__((address_space(3))) v4f*)(lds_char_t*)(uintptr_t)chunk_at(wr, 2 * g + wh) =
            v4f{a[4 * rq], a[4 * rq + 1], a[4 * rq + 2], a[4 * rq + 3]};
      }
    }
    const int n = n0 + i / TM * SC + 8 * rc, left = p.n - n;
    const int mq = m0 + 32 * (i % TM) + rr;
    float z[NR][8], y[NR][8];
#pragma unroll
    for (int q = 0; q < NR; ++q) {
      const uint32_t r = q * RPI + rr;
      const v4f lo = *(const __attribute__((address_space(3))) v4f*)(lds_char_t*)(uintptr_t)chunk_at(r, 2 * rc);
      const v4f hi = *(const __attribute__((address_space(3))) v4f*)(lds_char_t*)(uintptr_t)chunk_at(r, 2 * rc + 1);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        z[q][e] = __builtin_fmaf(e < 4 ? lo[e] : hi[e - 4], alpha, e < 4 ? now.b0[e] : now.b1[e - 4]);
    }
    auto extra = [&](int q, int e) __attribute__((always_inline)) {
      const int w = x[0][q][e / 2];
      return __uint_as_float(e & 1 ? (uint32_t)w & 0xFFFF0000u : (uint32_t)w << 16);
    };
    with_act(p, [&](auto act, auto grad) __attribute__((always_inline)) {
      constexpr int A = decltype(act)::value;
#pragma unroll
      for (int q = 0; q < NR; ++q)
#pragma unroll
        for (int e = 0; e < 8; ++e)
          y[q][e] = decltype(grad)::value ? z[q][e] * act_slope<A>(extra(q, e)) : act_value<A>(z[q][e]);
    });
    if (xb && !p.grad) {
#pragma unroll
      for (int q = 0; q < NR; ++q)
#pragma unroll
        for (int e = 0; e < 8; ++e) y[q][e] += extra(q, e);
    }
    auto row_of = [](const float (&v)[8]) __attribute__((always_inline)) {
      return v4i{(int)pack_bf16x2(v[0], v[1]), (int)pack_bf16x2(v[2], v[3]), (int)pack_bf16x2(v[4], v[5]),
                 (int)pack_bf16x2(v[6], v[7])};
    };
#pragma unroll
    for (int q = 0; q < NR; ++q) {
      const int m = mq + q * RPI;
      if (m < p.m && left > 0) {
        if (zb) store8_row(zb + m * p.ld_preact + n, left, row_of(z[q]));
        store8_row(cb + m * p.ldc + n, left, row_of(y[q]));
      }
    }
    now = next;
#pragma unroll
    for (int a = 0; a < AHEAD; ++a)
#pragma unroll
      for (int q = 0; q < NR; ++q) x[a][q] = x[a + 1][q];
  }
  // The staging reads have returned before the caller's next loads refill the area.
  __builtin_amdgcn_s_waitcnt(lgkmcnt_zero_imm());
  if constexpr (DRAIN) __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));
  return false;
}

namespace {

template <bool A_KC, bool B_KC, int FA, int FB>
__global__ __launch_bounds__(512, 1) void gemm_epi_256_kernel(GemmEpiKArgs p) {
  __shared__ __attribute__((aligned(1024))) char smem_raw[smem_bytes<256, 256, 4>()];
  gemm_body<256, 256, 4, 2, 4, A_KC, B_KC, FA, FB>(p, (lds_char_t*)smem_raw, (int)blockIdx.x, (int)gridDim.x);
}

template <bool A_KC, bool B_KC, int FA, int FB>
__global__ __launch_bounds__(256, 2) void gemm_epi_128_kernel(GemmEpiKArgs p) {
  __shared__ __attribute__((aligned(1024))) char smem_raw[kUSlots * 128 * kKU];
  gemm_body_u128<A_KC, B_KC, FA, FB, 128>(p, (lds_char_t*)smem_raw, (int)blockIdx.x, (int)gridDim.x);
}

template <bool A_KC, bool B_KC, int FA, int FB>
__global__ __launch_bounds__(256, 4) void gemm_epi_64_kernel(GemmEpiKArgs p) {
  __shared__ __attribute__((aligned(1024))) char smem_raw[kUSlots * 64 * kKU];
  gemm_body_u128<A_KC, B_KC, FA, FB, 64>(p, (lds_char_t*)smem_raw, (int)blockIdx.x, (int)gridDim.x);
}

template <bool AKC, bool BKC, int FA, int FB>
GemmEpiFn pick_epi_tile(int tile) {
  if (tile == 6) return gemm_epi_256_kernel<AKC, BKC, FA, FB>;
  return tile == 7 ? gemm_epi_128_kernel<AKC, BKC, FA, FB> : gemm_epi_64_kernel<AKC, BKC, FA, FB>;
}
template <bool AKC, bool BKC>
GemmEpiFn pick_epi(int tile, int fa, int fb) {
  if (fa == 0) return fb == 0 ? pick_epi_tile<AKC, BKC, 0, 0>(tile) : pick_epi_tile<AKC, BKC, 0, 1>(tile);
  return fb == 0 ? pick_epi_tile<AKC, BKC, 1, 0>(tile) : pick_epi_tile<AKC, BKC, 1, 1>(tile);
}

}  // namespace
}  // namespace fp8ds
