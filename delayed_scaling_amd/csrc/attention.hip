// Attention and its backward pass on gfx950 16-bit MFMA, fp32 accumulation.
//
// For one head, with c = scale * log2(e) and visible(i, j) the mask:
//   S = Q K^T;  P_ij = 2^(c S_ij - m_i) over visible j, m_i the running maximum;
//   O_i = sum_j P_ij V_j / l_i;  lse_i = ln 2 (m_i + log2 l_i)
// and backward, from the stored lse (nothing of the size of S is kept):
//   P = 2^(c S - lse / ln 2);  delta_i = dO_i . O_i;  dS = P (dO V^T - delta)
//   dQ = scale dS K;  dK = scale dS^T Q;  dV = P^T dO
//
// Design:
//  * Every product is v_mfma_f32_32x32x16 with the operands arranged so that
//    softmax needs no shuffles and P never leaves its registers: the forward
//    forms S^T = K Q^T, so a lane owns one query (its column) and holds 16 of
//    the 32 keys of a tile, the other half of the lanes the other 16.  Row
//    statistics are one value a lane.  The same registers, packed to 16 bits,
//    are the B operand of O^T = V^T P^T: the order in which a lane holds its
//    keys (4 of each 8) is matched by loading V^T's fragments in that order.
//    dK / dV take S = Q K^T instead (a lane owns one key), and dQ the
//    transposed form again.
//  * A workgroup is four waves of 32 rows each (128 queries, or keys for dK
//    and dV); the operand they share streams through LDS in tiles of 64 rows,
//    two in flight (global -> LDS without a register round trip).
//  * One LDS layout serves both ways a tile is read: 16-byte pieces of a row
//    (K in S = Q K^T) and 4 x 16 blocks transposed on the way
//    (ds_read_b64_tr_b16: V^T, K^T, Q^T, dO^T).  Piece p of row r sits at
//    piece p ^ f(r), f chosen so that 16 consecutive rows of one piece, and 4
//    consecutive rows of 4 neighbouring pieces, fall into distinct banks.
//  * The grid runs the longest (latest) causal rows first, and all work of
//    one key / value head on one XCD, whose L2 then holds its K and V.
//  * Results do not depend on scheduling: every output has one writer that
//    sums in a fixed order (dK and dV loop over the query heads of their
//    group, in a fixed number of parts for the shapes; dQ has a kernel of its
//    own, two products more than a fused pass with atomic sums).
#include <algorithm>

#include "device_common.h"
#include "fp8ds.h"
#include "launch.h"

namespace fp8ds {

namespace {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
typedef _Float16 v2h __attribute__((ext_vector_type(2)));
typedef float v2f __attribute__((ext_vector_type(2)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) v4s lds_v4s_t;
typedef __attribute__((address_space(3))) v4f lds_v4f_t;
typedef __attribute__((address_space(3))) float lds_float_t;

constexpr int kWaves = 4;
constexpr int kTile = 64;                  // rows of one LDS tile
constexpr int kRows = 32 * kWaves;         // rows a workgroup owns
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNegInf = -__builtin_inff();
// The backward pass carries P times 2^24 in bf16 (whose range is fp32's) and
// takes the factor out of its sums: the hardware exponential flushes results
// below 2^-126, and gradients of keys that every query all but ignores would
// vanish there.  It costs nothing: the exponent rides on lse.  fp16 ends at 2^16
// and is coarse below 2^-14, so there P carries 2^15, which keeps it and dS = P
// (dP - delta) of gradients down to 1e-9 off the coarse end (unlifted, dS of
// 2e-7 was rounded to multiples of 6e-8); Fit below keeps large ones off the other.
template <bool BF>
constexpr float kLift = BF ? 24.0f : 15.0f;
template <bool BF>
constexpr float kDrop = BF ? 0x1p-24f : 0x1p-15f;
constexpr uint32_t kOut = 0x80000000u;     // offset past every buffer: loads give zero

template <int N>
struct Const {
  static constexpr int value = N;
};

struct View {
  char* p;
  int64_t batch, row, head;                // strides in bytes
};

struct AttnArgs {
  View q, k, v, o, dout, dq, dk, dv;
  float* lse;                              // [batch][heads_q][max_q], packed [heads_q][rows]
  float* delta;                            // same layout; stat_size further on, lse / ln 2 - kLift
  int64_t stat_size;
  const int32_t* cu_q;                     // packed: first row of each sequence, and one past the last
  const int32_t* cu_k;
  int64_t lse_head, lse_batch;             // strides of lse and delta in elements
  int64_t rows_q, rows_k;                  // packed: rows of the whole tensors
  int heads_q, heads_kv, group, batch, dim, max_q, max_k, blocks;
  int causal, window, paired;              // paired: a workgroup runs row blocks i and blocks - 1 - i
  int parts;                               // dK / dV: workgroups that share a block's query rows
  int64_t units;                           // blocks of 128 keys, over all sequences and heads
  float* partial;                          // [parts][units][dk, dv][wave]: sums of each part, as the lanes hold them
  float scale;
};

// One sequence of the batch: the first row and the number of rows of each side.
struct Seq {
  int64_t q0, k0;
  int nq, nk, b;
};
__device__ __forceinline__ Seq sequence(const AttnArgs& a, int b) {
  Seq s{0, 0, a.max_q, a.max_k, b};
  if (a.cu_q) {
    // Clamped to the tensors' rows and to the promised maxima (which the grid
    // was sized by), so no offset leads outside the tensors.
    s.q0 = max((int64_t)0, min((int64_t)a.cu_q[b], a.rows_q));
    s.nq = (int)max((int64_t)0, min(min((int64_t)a.cu_q[b + 1], a.rows_q) - s.q0, (int64_t)a.max_q));
    s.k0 = max((int64_t)0, min((int64_t)a.cu_k[b], a.rows_k));
    s.nk = (int)max((int64_t)0, min(min((int64_t)a.cu_k[b + 1], a.rows_k) - s.k0, (int64_t)a.max_k));
    s.b = 0;
  }
  return s;
}

// Workgroup -> (row block, head, sequence).  Index i runs on XCD i mod 8; the
// last row blocks, the longest causal ones, go first.  Dense: all blocks and
// query heads of one (sequence, key / value head) pair go to one XCD, whose L2
// keeps their K and V.  Packed sequences differ in length, so a pair is worth
// more or less work than another and some hold none: there the heads of all
// sequences are dealt round, which spreads every sequence over the XCDs
// (8192 tokens in nine ragged sequences, 16 heads on 4: forward 118 us with
// pairs bound to XCDs, 64 us dealt round; one sequence of 1750 tokens
// among eight empty ones: 92 against 39 us).
struct Work {
  int block, head, b;
};
__device__ __forceinline__ Work work_of(const AttnArgs& a, int heads, bool last_first, int i) {
  const int sub = heads / a.heads_kv;               // heads of this kernel per key / value head
  const int pairs = a.batch * a.heads_kv;
  int pair, u;                                      // u: index among the pair's sub * blocks workgroups
  if (a.cu_q) {
    const int all = pairs * sub, blk = i / all, r = i - blk * all;
    Work w;
    w.block = last_first ? a.blocks - 1 - blk : blk;
    w.b = r / heads;
    w.head = r - w.b * heads;
    return w;
  }
  const int whole = pairs & ~7;                     // pairs dealt to the XCDs in full rounds
  const int rounds_of = a.paired ? (a.blocks + 1) / 2 : a.blocks;
  const int per = sub * rounds_of;
  if (i < whole * per) {
    const int xcd = i & 7, j = i >> 3, rounds = whole >> 3;
    pair = (j % rounds) * 8 + xcd;
    u = j / rounds;
  } else {
    const int r = pairs - whole, j = i - whole * per;
    pair = whole + j % r;
    u = j / r;
  }
  Work w;
  const int blk = u / sub;
  w.block = last_first ? a.blocks - 1 - blk : blk;
  w.b = pair / a.heads_kv;
  w.head = (pair - w.b * a.heads_kv) * sub + u % sub;
  return w;
}

template <bool BF>
__device__ __forceinline__ v16f mfma(v4i x, v4i y, v16f c) {
  if constexpr (BF)
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8bf, x), __builtin_bit_cast(v8bf, y), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(v8h, x), __builtin_bit_cast(v8h, y), c, 0, 0, 0);
}

// Two floats to the 16-bit type, nearest even, the first in the low half.
template <bool BF>
__device__ __forceinline__ int pack2(float x, float y) {
  if constexpr (BF) return __builtin_bit_cast(int, __builtin_convertvector(v2f{x, y}, v2bf));
  else return __builtin_bit_cast(int, __builtin_convertvector(v2f{x, y}, v2h));
}

template <bool BF>
__device__ __forceinline__ float widen(int bits, int half) {
  if constexpr (BF) return __uint_as_float(half ? (uint32_t)bits & 0xFFFF0000u : (uint32_t)bits << 16);
  else return (float)__builtin_bit_cast(v2h, bits)[half];
}

// Sums of products of the 16-bit pairs of two registers.
template <bool BF>
__device__ __forceinline__ float dot8(v4i x, v4i y, float s) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    s = __builtin_fmaf(widen<BF>(x[e], 0), widen<BF>(y[e], 0), s);
    s = __builtin_fmaf(widen<BF>(x[e], 1), widen<BF>(y[e], 1), s);
  }
  return s;
}

// The larger of three.  (The builtins, which compile to one v_max3_f32, and not
// that instruction as inline asm: its operands are results of matrix products,
// and the compiler puts the wait states those need only before instructions it
// knows.  A NaN loses against a number here; it comes back through the
// exponential.)
__device__ __forceinline__ float max3(float x, float y, float z) {
  return __builtin_fmaxf(__builtin_fmaxf(x, y), z);
}

// fp16's end for dS: a factor (a power of two, one for the wave) under which every
// value packed so far has stayed below 2^15.  It falls, and the sums formed under
// the old one with it, when a value outgrows that: a test of the largest of 16 for
// each block, and a product an element once it is not 1 (nine packed sequences of
// 8192 tokens, forward and backward: 329 -> 337 us).  It goes to 16 times less than
// it has to at most, so what is lost of a value is its own rounding or 2^-36 of
// the largest.
template <bool BF>
struct Fit {
  float f = 1.0f;
  template <int N>
  __device__ __forceinline__ void operator()(v16f& x, v16f (&sums)[N]) {
    if constexpr (!BF) {
      float top = __builtin_fabsf(x[0]);
#pragma unroll
      for (int r = 1; r < 15; r += 2) top = max3(top, __builtin_fabsf(x[r]), __builtin_fabsf(x[r + 1]));
      top = __builtin_fmaxf(top, __builtin_fabsf(x[15])) * f;
      // (An infinity stays one, in a row or column of its lane's that is lost to it.)
      const bool finite = top < __builtin_inff();
      if (__any(finite && top > 0x1p15f)) {
        float shrink = 1.0f;
        do shrink *= 0x1p-4f;
        while (__any(finite && top * shrink > 0x1p15f));
        f *= shrink;
#pragma unroll
        for (int i = 0; i < N; ++i) sums[i] *= shrink;
      }
      if (f != 1.0f) x *= f;
    }
  }
};

// The value of the lane 32 away.
__device__ __forceinline__ float other_half(float x, bool hi) {
  const uint32_t u = __float_as_uint(x);
  const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return __uint_as_float(hi ? r[0] : r[1]);
}

__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}
// Wait for all of the wave's vector memory operations.  The loads into LDS
// below are counted by no one else; the builtin (unlike inline asm) also tells
// the compiler that loads of its own are done, so it puts no wait of its own,
// which would cover the tile just requested, into the loop.
__device__ __forceinline__ void wait_loads() { __builtin_amdgcn_s_waitcnt((7 << 4) | (15 << 8)); }

// ---------------------------------------------------------------------------
// LDS tiles: kTile rows of DP elements (2 DP bytes).

template <int DP>
__device__ __forceinline__ int swz(int r) {
  if constexpr (DP == 128) return ((r & 3) << 2) | ((r >> 2) & 3);
  else return (((r >> 1) & 1) << 2) | ((r >> 2) & 3);
}

// Brings rows row0 .. row0 + kTile of one head's matrix (n rows of dim
// elements, `stride` bytes apart) into the tile at `lds`; rows past n and
// columns past dim land as zeros.  The caller waits for the wave's loads and
// then for a barrier.
template <int DP>
struct TileLoad {
  static constexpr int kPieces = DP / 8;              // 16-byte pieces of a row
  static constexpr int kLoads = kTile * kPieces / 64 / kWaves;
  uint32_t voff[kLoads];

  __device__ __forceinline__ void init(int wave, int lane, int64_t stride, int dim) {
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      const int slot = (j * kWaves + wave) * 64 + lane;
      const int row = slot / kPieces, piece = (slot % kPieces) ^ swz<DP>(row);
      voff[j] = piece * 8 < dim ? (uint32_t)row * (uint32_t)stride + piece * 16u : kOut;
    }
  }
  // `left`: rows from the tile's first to the matrix's end.
  __device__ __forceinline__ void issue(const char* tile, uint32_t stride, int left, int dim, uint32_t lds,
                                        int wave) const {
    const uint32_t bytes = left > 0 ? (uint32_t)(min(left, kTile) - 1) * stride + (uint32_t)dim * 2u : 0u;
    const v4i rsrc = rsrc_words(tile, bytes);
    lds = __builtin_amdgcn_readfirstlane(lds + wave * 1024);
#pragma unroll
    for (int j = 0; j < kLoads; ++j) load_lds16(rsrc, lds + j * kWaves * 1024, voff[j], 0);
  }
};

// Row fragment: lane l gets 8 elements, from column 16 * slab + 8 * (l / 32),
// of row 32 * blk + l % 32.
template <int DP>
__device__ __forceinline__ v4i row_frag(const lds_char_t* tile, int blk, int slab, int lane) {
  const int r = lane & 31;
  const int piece = (2 * slab + (lane >> 5)) ^ swz<DP>(r);
  return *(const lds_v4i_t*)(tile + blk * (32 * DP * 2) + r * (DP * 2) + piece * 16);
}

// The same read, and a transposed one, with the lane's part of the address
// worked out once: a block's or slab's rows, and a tile's place in LDS up to
// 64 KB, are immediates.  Transposed: lane l gets, of column 32 * dblk + l % 32,
// the elements of rows 16 * slab + 4 h + {0..3} and 16 * slab + 8 + 4 h +
// {0..3}, h = l / 32: the order in which a lane holds 16 consecutive rows of an
// MFMA result.
template <int DP>
struct FragAddr {
  uint32_t row[DP / 16], col[DP / 32][2];
  __device__ __forceinline__ void init(int lane, uint32_t base = 0) {
    const int r = lane & 31, q = lane & 15, h = lane >> 5;
#pragma unroll
    for (int d = 0; d < DP / 16; ++d) row[d] = base + r * (DP * 2) + ((2 * d + h) ^ swz<DP>(r)) * 16;
#pragma unroll
    for (int i = 0; i < DP / 32; ++i)
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const int cr = 8 * t + 4 * h + (q >> 2);
        col[i][t] = base + cr * (DP * 2) + ((4 * i + 2 * ((lane >> 4) & 1) + ((q & 3) >> 1)) ^ swz<DP>(cr)) * 16 + (q & 1) * 8;
      }
  }
};
__device__ __forceinline__ v4i read_row(uint32_t addr, int imm) {
  return *(const lds_v4i_t*)((const lds_char_t*)(uintptr_t)addr + imm);
}
__device__ __forceinline__ v4i read_col(const uint32_t (&addr)[2], int imm) {
  const v2i lo = __builtin_bit_cast(v2i, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s_t*)((lds_char_t*)(uintptr_t)addr[0] + imm)));
  const v2i hi = __builtin_bit_cast(v2i, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s_t*)((lds_char_t*)(uintptr_t)addr[1] + imm)));
  return v4i{lo[0], lo[1], hi[0], hi[1]};
}

// Row of a 32-row MFMA result that register r of lane half h holds.
__device__ __forceinline__ int result_row(int r, int h) { return 8 * (r >> 2) + 4 * h + (r & 3); }

// 32 rows of one head's matrix as the B operand over all columns, straight
// from global memory: lane l holds row l % 32; zeros outside.
template <int DP>
__device__ __forceinline__ void load_rows(v4i (&f)[DP / 16], const char* base, int64_t stride, int row0, int n,
                                          int dim, int lane) {
  const int row = row0 + (lane & 31);
#pragma unroll
  for (int s = 0; s < DP / 16; ++s) {
    const int col = 16 * s + 8 * (lane >> 5);
    f[s] = row < n && col < dim ? *reinterpret_cast<const v4i*>(base + (int64_t)row * stride + col * 2) : v4i{};
  }
}

// 16-bit rows out of a transposed result: lane l holds row l % 32 and, of each
// 8 columns, 4.
template <int DP, bool BF>
__device__ __forceinline__ void store_rows(const v16f (&acc)[DP / 32], float factor, char* base, int64_t stride,
                                           int row0, int n, int dim, int lane) {
  const int row = row0 + (lane & 31), h = lane >> 5;
  if (row >= n) return;
  char* p = base + (int64_t)row * stride;
#pragma unroll
  for (int i = 0; i < DP / 32; ++i)
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int col = 32 * i + 8 * g + 4 * h;
      if (col < dim)
        *reinterpret_cast<v2i*>(p + col * 2) =
            v2i{pack2<BF>(acc[i][4 * g] * factor, acc[i][4 * g + 1] * factor),
                pack2<BF>(acc[i][4 * g + 2] * factor, acc[i][4 * g + 3] * factor)};
    }
}

// Keys that some row of [row0, row0 + rows) sees, as a range; `off` is
// nk - nq, the shift that aligns the last query with the last key.
__device__ __forceinline__ void key_range(const AttnArgs& a, const Seq& s, int row0, int rows, int& lo, int& hi) {
  lo = 0;
  hi = s.nk;
  const int last = min(row0 + rows, s.nq) - 1;
  const int64_t off = (int64_t)s.nk - s.nq;
  if (a.causal) hi = (int)max((int64_t)0, min((int64_t)s.nk, last + off + 1));
  if (a.window) lo = (int)max((int64_t)0, min((int64_t)s.nk, row0 + off - a.window + 1));
}

// ---------------------------------------------------------------------------
// Forward.

// Two waves a SIMD cover each other's latencies.  What bounds it is issue: per
// 64-key tile a wave spends as long issuing 32 exponentials, about 100 vector
// instructions and its LDS reads as its 32 products keep the matrix unit busy,
// and the two waves' shares overlap only in part (MFMA busy 49 % of SIMD
// cycles, no LDS conflicts, 85 MB from HBM at 2 x 4096).  Measured, causal bf16:
// 8192 tokens, 16 heads of 128 on 4: 267-287 us = 0.96-1.03 PFLOP/s; 2 x 4096,
// 16 heads on 8: 150-169 us; 4 x 512, 16 heads of 64: 12-13 us.
template <int DP, bool BF>
__global__ __launch_bounds__(64 * kWaves, 2) void attn_fwd_kernel(AttnArgs a) {
  constexpr int kTileBytes = kTile * DP * 2;
  __shared__ __attribute__((aligned(1024))) char smem_raw[4 * kTileBytes];   // K and V of two tiles
  lds_char_t* smem = (lds_char_t*)smem_raw;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), h = lane >> 5;
  const Work w = work_of(a, a.heads_q, a.causal != 0, blockIdx.x);
  const Seq s = sequence(a, w.b);
  const int kvh = w.head / a.group;
  const char* qp = a.q.p + s.b * a.q.batch + s.q0 * a.q.row + w.head * a.q.head;
  const char* kp = a.k.p + s.b * a.k.batch + s.k0 * a.k.row + kvh * a.k.head;
  const char* vp = a.v.p + s.b * a.v.batch + s.k0 * a.v.row + kvh * a.v.head;
  const uint32_t krow = (uint32_t)a.k.row, vrow = (uint32_t)a.v.row;
  const uint32_t base = lds_address(smem);
  const float c = a.scale * kLog2e;
  TileLoad<DP> lk, lv;
  lk.init(wave, lane, a.k.row, a.dim);
  lv.init(wave, lane, a.v.row, a.dim);
  FragAddr<DP> at;
  at.init(lane, base);

  for (int pass = 0; pass < (a.paired ? 2 : 1); ++pass) {
    const int block = pass == 0 ? w.block : a.blocks - 1 - w.block;
    const int row0 = block * kRows, wrow = row0 + 32 * wave;
    if (row0 >= s.nq || (pass == 1 && block == w.block)) continue;
    if (pass == 1) lds_barrier();           // every wave has read its last tile of the first pass

    int klo, khi;
    key_range(a, s, row0, kRows, klo, khi);
    const int t0 = klo / kTile, t1 = (khi + kTile - 1) / kTile;
    const char* kt = kp + (int64_t)t0 * kTile * krow;        // the next tile to request
    const char* vt = vp + (int64_t)t0 * kTile * vrow;
    int left = s.nk - t0 * kTile;
    auto issue = [&](int n) __attribute__((always_inline)) {   // into the buffer of n's parity
      const uint32_t to = base + (uint32_t)(n & 1) * 2 * kTileBytes;
      lk.issue(kt, krow, left, a.dim, to, wave);
      lv.issue(vt, vrow, left, a.dim, to + kTileBytes, wave);
      kt += (uint64_t)krow * kTile;
      vt += (uint64_t)vrow * kTile;
      left -= kTile;
    };
    if (t0 < t1) issue(0);
    v4i qf[DP / 16];
    load_rows<DP>(qf, qp, a.q.row, wrow, s.nq, a.dim, lane);

    v16f o[DP / 32] = {};
    float m = kNegInf, l = 0.0f;            // m in units of S; l: this lane's half of the row
    int jlo, jhi;                            // keys this lane's query sees
    key_range(a, s, wrow + (lane & 31), 1, jlo, jhi);
    int wlo, whi;                            // keys some query of this wave sees
    key_range(a, s, wrow, 32, wlo, whi);
    if (wrow >= s.nq) whi = 0;
    int clo, chi;                            // and keys all of them see
    {
      int x;
      key_range(a, s, wrow, 1, x, chi);
      key_range(a, s, wrow + 31, 1, clo, x);
    }

    // (Unrolled over the two buffers, so that theirs are constants and every LDS
    // read is a lane's address and an immediate.)
    auto step = [&](auto parity, int t) __attribute__((always_inline)) {
      constexpr int B = decltype(parity)::value, kK = B * 2 * kTileBytes, kV = kK + kTileBytes;
      wait_loads();
      lds_barrier();
      if (t + 1 < t1) issue(1 - B);
      const int j0 = t * kTile;
      if (j0 >= whi || j0 + kTile <= wlo) return;
      v16f st[2] = {};
#pragma unroll
      for (int d = 0; d < DP / 16; ++d)
#pragma unroll
        for (int b = 0; b < 2; ++b) st[b] = mfma<BF>(read_row(at.row[d], kK + b * (32 * DP * 2)), qf[d], st[b]);
      if (j0 < clo || j0 + kTile > chi) {
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            const int j = j0 + 32 * b + result_row(r, h);
            st[b][r] = ((j < jhi) & (j >= jlo)) ? st[b][r] : kNegInf;
          }
      }
      float top = max3(st[0][0], st[1][0], kNegInf);
#pragma unroll
      for (int r = 1; r < 16; ++r) top = max3(top, st[0][r], st[1][r]);
      top = fmaxf(top, other_half(top, h));
      // The maximum moves only when a row outgrows it by 2^8 (or had none): until
      // then P stays below 2^8 and O and l need no rescaling; the quotient O / l is
      // the same either way.
      if (__any(!((top - m) * c <= 8.0f))) {
        const float next = fmaxf(m, top);
        const float safe = next == kNegInf ? 0.0f : next;
        const float shrink = __builtin_amdgcn_exp2f((m - safe) * c);
        m = next;
        l *= shrink;
#pragma unroll
        for (int i = 0; i < DP / 32; ++i) o[i] *= shrink;
      }
      const float mc = m == kNegInf ? 0.0f : m * c;
      float sum[2] = {};
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          st[b][r] = __builtin_amdgcn_exp2f(__builtin_fmaf(st[b][r], c, -mc));
          sum[r & 1] += st[b][r];
        }
      l += sum[0] + sum[1];
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          v4i p;
#pragma unroll
          for (int e = 0; e < 4; ++e) p[e] = pack2<BF>(st[b][8 * k + 2 * e], st[b][8 * k + 2 * e + 1]);
#pragma unroll
          for (int i = 0; i < DP / 32; ++i)
            o[i] = mfma<BF>(read_col(at.col[i], kV + (2 * b + k) * (16 * DP * 2)), p, o[i]);
        }
    };
    for (int t = t0; t < t1; t += 2) {
      step(Const<0>{}, t);
      if (t + 1 < t1) step(Const<1>{}, t + 1);
    }

    if (wrow >= s.nq) continue;
    l += other_half(l, h);
    const float inv = l > 0.0f ? 1.0f / l : l == 0.0f ? 0.0f : __builtin_nanf("");
    char* op = a.o.p + s.b * a.o.batch + s.q0 * a.o.row + w.head * a.o.head;
    store_rows<DP, BF>(o, inv, op, a.o.row, wrow, s.nq, a.dim, lane);
    const int row = wrow + lane;
    if (lane < 32 && row < s.nq)
      a.lse[s.b * a.lse_batch + w.head * a.lse_head + s.q0 + row] =
          l == 0.0f ? kNegInf : m * a.scale + kLn2 * __builtin_amdgcn_logf(l);
  }
}

// ---------------------------------------------------------------------------
// Backward: dQ (and delta, which the dK / dV kernel after it reads).  Bound as
// the forward is, with three products a tile for its two (MFMA busy 50 %); at
// head_dim 128 without FIX addresses of the output go to memory before the loop
// and come back after it (92 bytes a lane: 12 MB at 2 x 4096).  Measured, causal bf16: 2 x 4096, 16 heads of 128 on 8:
// 220-245 us = 0.84-0.94 PFLOP/s; 4 x 512, 16 heads of 64: 18-19 us.
//
// delta from the rounded O carries O's rounding.  The rows of dS should sum to
// zero, so the sum r_i of those formed with delta' is the error of delta', and
// the dK / dV kernel gets delta' + r (2 x 4096: dK 2.43e-3 off in all without it,
// 2.34e-3 with; 16 additions a lane and block of 32 keys, 1.2 % of the whole step).  For dQ itself
// the error is little beside the rounding of dS over many keys, but as much
// again over few (64 keys: 2.9e-3 off in all instead of 2.4e-3).  There FIX
// removes it too:
//   dQ = scale (dS' K - r (P K))
// with one product more.
template <int DP, bool BF, bool FIX>
__global__ __launch_bounds__(64 * kWaves, FIX && DP == 128 ? 1 : 2) void attn_dq_kernel(AttnArgs a) {
  constexpr int kTileBytes = kTile * DP * 2;
  __shared__ __attribute__((aligned(1024))) char smem_raw[4 * kTileBytes];
  lds_char_t* smem = (lds_char_t*)smem_raw;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), h = lane >> 5;
  const Work w = work_of(a, a.heads_q, a.causal != 0, blockIdx.x);
  const Seq s = sequence(a, w.b);
  const int kvh = w.head / a.group;
  const char* qp = a.q.p + s.b * a.q.batch + s.q0 * a.q.row + w.head * a.q.head;
  const char* kp = a.k.p + s.b * a.k.batch + s.k0 * a.k.row + kvh * a.k.head;
  const char* vp = a.v.p + s.b * a.v.batch + s.k0 * a.v.row + kvh * a.v.head;
  const char* gp = a.dout.p + s.b * a.dout.batch + s.q0 * a.dout.row + w.head * a.dout.head;
  const char* op = a.o.p + s.b * a.o.batch + s.q0 * a.o.row + w.head * a.o.head;
  TileLoad<DP> lk, lv;
  lk.init(wave, lane, a.k.row, a.dim);
  lv.init(wave, lane, a.v.row, a.dim);
  const uint32_t base = lds_address(smem);
  const uint32_t krow = (uint32_t)a.k.row, vrow = (uint32_t)a.v.row;
  FragAddr<DP> at;
  at.init(lane, base);

  for (int pass = 0; pass < (a.paired ? 2 : 1); ++pass) {
    const int block = pass == 0 ? w.block : a.blocks - 1 - w.block;
    const int row0 = block * kRows, wrow = row0 + 32 * wave, row = wrow + (lane & 31);
    if (row0 >= s.nq || (pass == 1 && block == w.block)) continue;
    if (pass == 1) lds_barrier();            // every wave has read its last tile of the first pass
    int klo, khi;
    key_range(a, s, row0, kRows, klo, khi);
    const int t0 = klo / kTile, t1 = (khi + kTile - 1) / kTile;
    const char* kt = kp + (int64_t)t0 * kTile * krow;        // the next tile to request
    const char* vt = vp + (int64_t)t0 * kTile * vrow;
    int left = s.nk - t0 * kTile;
    auto issue = [&](int n) __attribute__((always_inline)) {   // into the buffer of n's parity
      const uint32_t to = base + (uint32_t)(n & 1) * 2 * kTileBytes;
      lk.issue(kt, krow, left, a.dim, to, wave);
      lv.issue(vt, vrow, left, a.dim, to + kTileBytes, wave);
      kt += (uint64_t)krow * kTile;
      vt += (uint64_t)vrow * kTile;
      left -= kTile;
    };
    if (t0 < t1) issue(0);

    v4i qf[DP / 16], gf[DP / 16];
    load_rows<DP>(qf, qp, a.q.row, wrow, s.nq, a.dim, lane);
    load_rows<DP>(gf, gp, a.dout.row, wrow, s.nq, a.dim, lane);
    float delta = 0.0f;
    {
      v4i of[DP / 16];
      load_rows<DP>(of, op, a.o.row, wrow, s.nq, a.dim, lane);
#pragma unroll
      for (int d = 0; d < DP / 16; ++d) delta = dot8<BF>(gf[d], of[d], delta);
    }
    delta += other_half(delta, h);
    const int64_t stat = s.b * a.lse_batch + w.head * a.lse_head + s.q0 + row;
    float lse = 0.0f;
    if (row < s.nq) {
      lse = a.lse[stat];
      // A row that sees nothing: its P is 2^(S - infinity) = 0 in the kernel that reads this.
      if (h == 0) a.delta[a.stat_size + stat] = lse == kNegInf ? -kNegInf : lse * kLog2e - kLift<BF>;
    }
    const float c = a.scale * kLog2e;
    const float mc = lse == kNegInf ? 0.0f : lse * kLog2e - kLift<BF>;   // (an empty row: every key is masked)
    int jlo, jhi;                            // keys this lane's query sees
    key_range(a, s, row, 1, jlo, jhi);
    int wlo, whi;
    key_range(a, s, wrow, 32, wlo, whi);
    if (wrow >= s.nq) whi = 0;
    v16f dq[DP / 32] = {}, pk[FIX ? DP / 32 : 1] = {};
    float rest = 0.0f;                       // this lane's half of r, times 2^kLift
    Fit<BF> fit;

    int clo, chi;                            // keys every query of this wave sees
    {
      int x;
      key_range(a, s, wrow, 1, x, chi);
      key_range(a, s, wrow + 31, 1, clo, x);
    }
    // (Unrolled over the two buffers, so that theirs are constants.)
    auto step = [&](auto parity, int t) __attribute__((always_inline)) {
      constexpr int kK = decltype(parity)::value * 2 * kTileBytes, kV = kK + kTileBytes;
      wait_loads();
      lds_barrier();
      if (t + 1 < t1) issue(1 - decltype(parity)::value);
      const int j0 = t * kTile;
      if (j0 >= whi || j0 + kTile <= wlo) return;
      const bool edge = j0 < clo || j0 + kTile > chi;
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        v16f st = {}, dp = {};
#pragma unroll
        for (int d = 0; d < DP / 16; ++d) {
          st = mfma<BF>(read_row(at.row[d], kK + b * (32 * DP * 2)), qf[d], st);
          dp = mfma<BF>(read_row(at.row[d], kV + b * (32 * DP * 2)), gf[d], dp);
        }
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(st[r], c, -mc));
          st[r] = p * (dp[r] - delta);
          if (FIX) dp[r] = p;
        }
        if (edge) {
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            const int j = j0 + 32 * b + result_row(r, h);
            const bool see = (j < jhi) & (j >= jlo);
            st[r] = see ? st[r] : 0.0f;
            if (FIX) dp[r] = see ? dp[r] : 0.0f;
          }
        }
#pragma unroll
        for (int r = 0; r < 16; ++r) rest += st[r];
        fit(st, dq);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          v4i x, p;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            x[e] = pack2<BF>(st[8 * k + 2 * e], st[8 * k + 2 * e + 1]);
            if (FIX) p[e] = pack2<BF>(dp[8 * k + 2 * e], dp[8 * k + 2 * e + 1]);
          }
#pragma unroll
          for (int i = 0; i < DP / 32; ++i) {
            const v4i f = read_col(at.col[i], kK + (2 * b + k) * (16 * DP * 2));
            dq[i] = mfma<BF>(f, x, dq[i]);
            if constexpr (FIX) pk[i] = mfma<BF>(f, p, pk[i]);
          }
        }
      }
    };
    for (int t = t0; t < t1; t += 2) {
      step(Const<0>{}, t);
      if (t + 1 < t1) step(Const<1>{}, t + 1);
    }
    rest = (rest + other_half(rest, h)) * kDrop<BF>;
    if (row < s.nq && h == 0) a.delta[stat] = delta + rest;
    if constexpr (!BF) {
#pragma unroll
      for (int i = 0; i < DP / 32; ++i) dq[i] *= 1.0f / fit.f;
    }
    if constexpr (FIX) {
#pragma unroll
      for (int i = 0; i < DP / 32; ++i) dq[i] -= rest * pk[i];
    }
    char* dst = a.dq.p + s.b * a.dq.batch + s.q0 * a.dq.row + w.head * a.dq.head;
    store_rows<DP, BF>(dq, a.scale * kDrop<BF>, dst, a.dq.row, wrow, s.nq, a.dim, lane);
  }
}

// ---------------------------------------------------------------------------
// Backward: dK and dV.  A workgroup owns 128 keys and runs over the query
// heads of their group and the query rows that see them.

// One wave a SIMD at head_dim 128 (its 128 accumulators, the K and V fragments
// and two score tiles in flight take the registers of two), so nothing but the
// wave itself hides a latency: the loop is pipelined by hand over blocks of 32
// query rows.  Step t runs the S and dP products of block t + 1 under the
// exponentials of block t and the transposed reads its dV and dK products
// need, then those products under the row reads of block t + 2.  Three LDS
// buffers keep tiles n and n + 1 readable while n + 2 arrives, so one barrier
// a tile is enough.  Bound by that one wave's issue (MFMA busy 47 % of SIMD
// cycles, LDS reads 29 % of CU cycles without conflicts).  Measured, causal
// bf16: 2 x 4096, 16 heads of 128 on 8: 309-352 us = 0.78-0.89 PFLOP/s (478
// before the pipelining); 4 x 512, 16 heads of 64: 20-21 us.
//
// Few keys, or few key / value heads, make fewer workgroups than keep the
// device busy.  Then `parts` workgroups share a block's query tiles (of all
// its heads, one range of them each) and leave their sums as fp32 in the
// workspace, in the order the lanes hold them; attn_join_kernel adds them, in
// the order of the parts, and rounds once.  Measured (causal bf16, dQ and dK / dV
// together, alone and shared): 1 x 8192, 16 heads of 128 on 4: 1257 and 913 us;
// 1 x 2048: 297 and 133; 1 x 1024, 8 heads of 64 on 1: 203 and 48.  Nine packed
// fp16 sequences of 8192 tokens in all (16 heads of 128 on 4, window 1024): 170 us,
// or 143 and 18 for the join (148 since Fit).
//
// Where one part's sums of a wave's 32 keys stand: which = 0 dK, 1 dV.  Packed
// sequences: sequence b's blocks are numbered from k0 / 128 + b on, so no two
// blocks share a number and the last is below rows / 128 + batch.
template <int DP>
__device__ __forceinline__ float* partial_of(const AttnArgs& a, const Seq& s, const Work& w, int block, int blocks,
                                             int part, int which, int wave) {
  const int64_t id = (a.cu_q ? s.k0 / kRows + w.b : (int64_t)w.b * blocks) + block;
  return a.partial + (((part * a.units + id * a.heads_kv + w.head) * 2 + which) * kWaves + wave) * (32 * DP);
}

template <int DP, bool BF>
__global__ __launch_bounds__(64 * kWaves, 1) void attn_dkv_kernel(AttnArgs a) {
  constexpr int kTileBytes = kTile * DP * 2, kSlabs = DP / 16, kBlocks = DP / 32, kBufs = 3;
  __shared__ __attribute__((aligned(1024))) char smem_raw[kBufs * 2 * kTileBytes];   // a Q and a dO tile each
  __shared__ __attribute__((aligned(16))) float stats_raw[kBufs][2][kTile];          // lse / ln 2 - kLift, delta
  lds_char_t* smem = (lds_char_t*)smem_raw;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), h = lane >> 5;
  const Work w = work_of(a, a.heads_kv, false, blockIdx.x);
  const Seq s = sequence(a, w.b);
  // Packed: blocks of one distance from their sequence's end, which see as many
  // rows, run together, the longest first.
  const int from = w.block / a.parts, part = w.block - from * a.parts;
  const int block = a.cu_q ? from - (a.blocks / a.parts - (s.nk + kRows - 1) / kRows) : from;
  const int key0 = block * kRows;
  if (block < 0 || key0 >= s.nk) return;
  const char* kp = a.k.p + s.b * a.k.batch + s.k0 * a.k.row + w.head * a.k.head;
  const char* vp = a.v.p + s.b * a.v.batch + s.k0 * a.v.row + w.head * a.v.head;
  const int wkey = key0 + 32 * wave, key = wkey + (lane & 31);

  // Query rows that see one of the workgroup's keys, and this lane's key.
  const int64_t off = (int64_t)s.nk - s.nq;
  auto row_range = [&](int k0, int n, int& lo, int& hi) __attribute__((always_inline)) {
    lo = 0;
    hi = s.nq;
    const int last = min(k0 + n, s.nk) - 1;
    if (a.causal) lo = (int)max((int64_t)0, min((int64_t)s.nq, k0 - off));
    if (a.window) hi = (int)max((int64_t)0, min((int64_t)s.nq, (int64_t)last + a.window - off));
  };
  int rlo, rhi, ilo, ihi;
  row_range(key0, kRows, rlo, rhi);
  row_range(key, 1, ilo, ihi);
  if (key >= s.nk) ihi = 0;
  const int t0 = rlo / kTile, t1 = (rhi + kTile - 1) / kTile;
  // The tiles of all heads in a row, and this part's share [first, first + total).
  const int per = max(0, t1 - t0), all = per * a.group;
  const int first = (int)((int64_t)all * part / a.parts), total = (int)((int64_t)all * (part + 1) / a.parts) - first;
  // Rows every key of this wave is seen by: tiles inside need no mask.
  int clo, chi;
  {
    int x;
    row_range(wkey + 31, 1, clo, x);
    row_range(wkey, 1, x, chi);
    if (wkey + 32 > s.nk) chi = 0;
  }

  TileLoad<DP> lq, lg;
  lq.init(wave, lane, a.q.row, a.dim);
  lg.init(wave, lane, a.dout.row, a.dim);
  const uint32_t base = lds_address(smem);
  const uint32_t stats_base = lds_address((const lds_char_t*)&stats_raw[0][0][0]);
  // The next tile to request: its query head, its addresses, its buffer.
  const uint32_t qrow = (uint32_t)a.q.row, grow = (uint32_t)a.dout.row;
  int ih = 0, left = 0, togo = 0, ibuf = 0, todo = total;
  const char *qp, *gp;
  const float* sp;                         // waves 0 and 1: lse / ln 2 and delta
  auto first_tile = [&]() __attribute__((always_inline)) {
    const int qh = w.head * a.group + ih;
    const int64_t r0 = s.q0 + (int64_t)t0 * kTile;
    qp = a.q.p + s.b * a.q.batch + r0 * a.q.row + qh * a.q.head;
    gp = a.dout.p + s.b * a.dout.batch + r0 * a.dout.row + qh * a.dout.head;
    sp = a.delta + (wave == 0 ? a.stat_size : 0) + s.b * a.lse_batch + qh * a.lse_head + r0;
    left = s.nq - t0 * kTile;
    togo = per;
  };
  if (total > 0) ih = first / per;
  const int skip = first - ih * per;                  // tiles of the first head that are another part's
  first_tile();
  qp += (uint64_t)qrow * kTile * skip;
  gp += (uint64_t)grow * kTile * skip;
  sp += kTile * skip;
  left -= kTile * skip;
  togo -= skip;
  auto issue = [&]() __attribute__((always_inline)) {
    if (todo-- > 0) {
      const uint32_t at = base + (uint32_t)ibuf * 2 * kTileBytes;
      lq.issue(qp, qrow, left, a.dim, at, wave);
      lg.issue(gp, grow, left, a.dim, at + kTileBytes, wave);
      if (wave < 2)   // 64 values; zeros past the sequence
        load_lds4(rsrc_words(sp, (uint32_t)max(0, min(left, kTile)) * 4u),
                  __builtin_amdgcn_readfirstlane(stats_base + (uint32_t)(ibuf * 2 + wave) * (kTile * 4)),
                  (uint32_t)lane * 4u);
    }
    ibuf = ibuf == kBufs - 1 ? 0 : ibuf + 1;
    if (--togo == 0) {
      ++ih;
      first_tile();
    } else {
      qp += (uint64_t)qrow * kTile;
      gp += (uint64_t)grow * kTile;
      sp += kTile;
      left -= kTile;
    }
  };

  v16f dk[kBlocks] = {}, dv[kBlocks] = {};
  Fit<BF> fit;
  if (total > 0) {
    issue();
    issue();
    v4i kf[kSlabs], vf[kSlabs];
    load_rows<DP>(kf, kp, a.k.row, wkey, s.nk, a.dim, lane);
    load_rows<DP>(vf, vp, a.v.row, wkey, s.nk, a.dim, lane);
    const float c = a.scale * kLog2e;
    wait_loads();
    lds_barrier();

    v4i rq[kSlabs], rg[kSlabs];                       // row fragments of the next block
    v16f st[2], dp[2];
    auto load_block = [&](const lds_char_t* qt, int b) __attribute__((always_inline)) {
#pragma unroll
      for (int d = 0; d < kSlabs; ++d) {
        rq[d] = row_frag<DP>(qt, b, d, lane);
        rg[d] = row_frag<DP>(qt + kTileBytes, b, d, lane);
      }
    };
    auto scores = [&](v16f& x, v16f& y) __attribute__((always_inline)) {
      x = v16f{};
      y = v16f{};
#pragma unroll
      for (int d = 0; d < kSlabs; ++d) {
        x = mfma<BF>(rq[d], kf[d], x);
        y = mfma<BF>(rg[d], vf[d], y);
      }
    };
    int buf = 0, r0 = (t0 + skip) * kTile;
    load_block(smem, 0);
    scores(st[0], dp[0]);
    load_block(smem, 1);
    FragAddr<DP> lane_at, at;
    lane_at.init(lane);

    auto step = [&](auto half) __attribute__((always_inline)) {
      constexpr int B = decltype(half)::value;
      const lds_float_t* stats = (const lds_float_t*)(lds_char_t*)(uintptr_t)(stats_base + (uint32_t)buf * (2 * kTile * 4));
      v4f lse[4], delta[4];
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        lse[g] = *(const lds_v4f_t*)(stats + 32 * B + 8 * g + 4 * h);
        delta[g] = *(const lds_v4f_t*)(stats + kTile + 32 * B + 8 * g + 4 * h);
      }
      // The order of this loop and the next is the order of issue (the
      // scheduler, left alone, gathers the products at the ends): one product,
      // then the vector and LDS instructions that fit under it.
      v4i cg[2][kBlocks], cq[2][kBlocks];
      v16f &p = st[B], &x = dp[B], &pn = st[1 - B], &xn = dp[1 - B];
      pn = v16f{};
      xn = v16f{};
      auto expo = [&](int r) __attribute__((always_inline)) {
        p[r] = __builtin_amdgcn_exp2f(__builtin_fmaf(p[r], c, -lse[r >> 2][r & 3]));
        x[r] -= delta[r >> 2][r & 3];
      };
      constexpr int kPer = 16 / (2 * kSlabs);         // elements a product
#pragma unroll
      for (int q = 0; q < 2 * kSlabs; ++q) {
        const int d = q >> 1, k = q / kSlabs, i = (q % kSlabs) >> 1;
        if (q & 1) {
          xn = mfma<BF>(rg[d], vf[d], xn);
          cq[k][i] = read_col(at.col[i], (2 * B + k) * (16 * DP * 2));
        } else {
          pn = mfma<BF>(rq[d], kf[d], pn);
          cg[k][i] = read_col(at.col[i], kTileBytes + (2 * B + k) * (16 * DP * 2));
        }
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
          const int r = q * kPer + e;
          if (r > 0) x[r - 1] *= p[r - 1];            // (one behind: the exponential's latency)
          expo(r);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      x[15] *= p[15];
      if (r0 < clo || r0 + kTile > chi) {
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const int row = r0 + 32 * B + result_row(r, h);
          const bool see = (row >= ilo) & (row < ihi);
          p[r] = see ? p[r] : 0.0f;
          x[r] = see ? x[r] : 0.0f;
        }
      }
      fit(x, dk);
      auto pack8 = [&](const v16f& y, int k) __attribute__((always_inline)) {
        return v4i{pack2<BF>(y[8 * k], y[8 * k + 1]), pack2<BF>(y[8 * k + 2], y[8 * k + 3]),
                   pack2<BF>(y[8 * k + 4], y[8 * k + 5]), pack2<BF>(y[8 * k + 6], y[8 * k + 7])};
      };
      v4i pp[2], ds[2];
      pp[0] = pack8(p, 0);
      ds[0] = pack8(x, 0);
#pragma unroll
      for (int q = 0; q < 2 * kBlocks; ++q) {
        const int k = q / kBlocks, i = q % kBlocks;
        dv[i] = mfma<BF>(cg[k][i], pp[k], dv[i]);
        rq[q] = read_row(at.row[q], B * (32 * DP * 2));
        if (q == 0) pp[1] = pack8(p, 1);
        __builtin_amdgcn_sched_barrier(0);
        dk[i] = mfma<BF>(cq[k][i], ds[k], dk[i]);
        rg[q] = read_row(at.row[q], kTileBytes + B * (32 * DP * 2));
        if (q == 0) ds[1] = pack8(x, 1);
        __builtin_amdgcn_sched_barrier(0);
      }
    };

    for (int n = 0; n < total; ++n) {
      // (After the last tile the reads of the next one find what is there, and
      // what is computed from them is not used.)
      const int nbuf = buf == kBufs - 1 ? 0 : buf + 1;
      // This tile's transposed reads, and the next one's row reads.
#pragma unroll
      for (int i = 0; i < kBlocks; ++i)
#pragma unroll
        for (int t = 0; t < 2; ++t) at.col[i][t] = lane_at.col[i][t] + (base + (uint32_t)buf * 2 * kTileBytes);
#pragma unroll
      for (int d = 0; d < kSlabs; ++d) at.row[d] = lane_at.row[d] + (base + (uint32_t)nbuf * 2 * kTileBytes);
      // Operands that stay the whole loop belong in the accumulation registers,
      // the score tiles, which vector instructions read, outside them.
#pragma unroll
      for (int d = 0; d < kSlabs; ++d) asm volatile("" : "+a"(kf[d]), "+a"(vf[d]));
      if (n > 0) {
        wait_loads();                                 // tile n + 1, requested a tile ago
        lds_barrier();
      }
      issue();                                        // tile n + 2, where tile n - 1 was
      step(Const<0>{});
      step(Const<1>{});
      buf = nbuf;
      r0 += kTile;
      if (r0 == t1 * kTile) r0 = t0 * kTile;
    }
  }
  if constexpr (!BF) {
#pragma unroll
    for (int i = 0; i < kBlocks; ++i) dk[i] *= 1.0f / fit.f;
  }
  if (a.parts > 1) {
    const int blocks = a.blocks / a.parts;
    auto leave = [&](const v16f (&x)[kBlocks], int which) __attribute__((always_inline)) {
      v4f* p = reinterpret_cast<v4f*>(partial_of<DP>(a, s, w, block, blocks, part, which, wave)) + lane;
#pragma unroll
      for (int i = 0; i < kBlocks; ++i)
#pragma unroll
        for (int g = 0; g < 4; ++g)
          p[(4 * i + g) * 64] = v4f{x[i][4 * g], x[i][4 * g + 1], x[i][4 * g + 2], x[i][4 * g + 3]};
    };
    leave(dk, 0);
    leave(dv, 1);
    return;
  }
  store_rows<DP, BF>(dk, a.scale * kDrop<BF>, a.dk.p + s.b * a.dk.batch + s.k0 * a.dk.row + w.head * a.dk.head, a.dk.row, wkey,
                     s.nk, a.dim, lane);
  store_rows<DP, BF>(dv, kDrop<BF>, a.dv.p + s.b * a.dv.batch + s.k0 * a.dv.row + w.head * a.dv.head, a.dv.row, wkey,
                     s.nk, a.dim, lane);
}

// dK and dV from their parts.  A wave takes 32 keys and 32 columns of one of the
// two, so that few blocks still spread over the device.  Bound by the reads of
// the partial sums (packed fp16 case above: 71 MB in 18 us = 4 TB/s).
template <int DP, bool BF>
__global__ __launch_bounds__(64 * kWaves) void attn_join_kernel(AttnArgs a) {
  constexpr int kBlocks = DP / 32;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, h = lane >> 5;
  const int piece = blockIdx.x % (2 * kBlocks), which = piece / kBlocks, i = piece % kBlocks;
  const Work w = work_of(a, a.heads_kv, false, blockIdx.x / (2 * kBlocks));
  const Seq s = sequence(a, w.b);
  const int key0 = w.block * kRows + 32 * wave, key = key0 + (lane & 31);
  if (key0 >= s.nk) return;
  v4f sum[4] = {};
#pragma unroll 4
  for (int part = 0; part < a.parts; ++part) {
    const v4f* p = reinterpret_cast<const v4f*>(partial_of<DP>(a, s, w, w.block, a.blocks, part, which, wave)) + lane;
#pragma unroll
    for (int g = 0; g < 4; ++g) sum[g] += p[(4 * i + g) * 64];
  }
  if (key >= s.nk) return;
  const View& out = which ? a.dv : a.dk;
  const float factor = which ? kDrop<BF> : a.scale * kDrop<BF>;
  char* p = out.p + s.b * out.batch + (s.k0 + key) * out.row + w.head * out.head;
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    const int col = 32 * i + 8 * g + 4 * h;
    if (col < a.dim)
      *reinterpret_cast<v2i*>(p + col * 2) = v2i{pack2<BF>(sum[g][0] * factor, sum[g][1] * factor),
                                                pack2<BF>(sum[g][2] * factor, sum[g][3] * factor)};
  }
}

// ---------------------------------------------------------------------------
// Host side.

View view(const fp8ds_attn_view& v) {
  return View{static_cast<char*>(const_cast<void*>(v.p)), v.stride_batch * 2, v.stride_row * 2, v.stride_head * 2};
}

// Blocks of 128 keys over all sequences and key / value heads (packed: a bound
// on them, from the rows there are).
int64_t dkv_units(const fp8ds_attn_args& p) {
  const int64_t blocks = p.cu_seqlens_q ? (p.rows_k + kRows - 1) / kRows + p.batch
                                        : ((int64_t)p.max_k + kRows - 1) / kRows * p.batch;
  return blocks * p.heads_kv;
}
// Into how many parts dK / dV cuts the query tiles of each.  A CU runs one of
// its workgroups at a time.  Blocks of one length (every key sees as many rows)
// are cut until they fill the 256 CUs once; causal and packed ones differ, half
// as long on average as the longest, and even out over 512.  No part is made
// shorter than 8 tiles, about the time of the launch that joins them (with 4:
// 4 x 512, 16 heads of 64: 51 against 38 us for the backward; 1 x 1024, 16 heads of
// 128 on 4: 81 against 73).  The quotient is rounded: 3 x 1500, 12 heads of 64, 432
// blocks: 116 us in two parts each, 111 in one.
int dkv_parts(const fp8ds_attn_args& p) {
  constexpr int64_t kCus = 256, kLeast = 8;
  const int64_t units = dkv_units(p);
  if (units <= 0) return 1;
  const int64_t rows = p.window > 0 ? std::min<int64_t>(p.max_q, (int64_t)p.window + kRows) : p.max_q;
  const int64_t tiles = (rows + kTile - 1) / kTile * (p.heads_q / p.heads_kv);
  const bool even = !p.cu_seqlens_q && (!p.causal || rows < p.max_q);
  const int64_t fill = even ? kCus / units : (2 * kCus + units / 2) / units;
  return (int)std::max<int64_t>(1, std::min(fill, tiles / kLeast));
}
size_t stats_bytes(const fp8ds_attn_args& p) {
  const size_t rows = (size_t)p.heads_q * (size_t)p.lse_stride_head * (p.cu_seqlens_q ? 1 : (size_t)p.batch);
  return (rows * 8 + 15) & ~(size_t)15;
}

AttnArgs make_args(const fp8ds_attn_args& p) {
  AttnArgs a{};
  a.q = view(p.q);
  a.k = view(p.k);
  a.v = view(p.v);
  a.o = view(p.out);
  a.dout = view(p.dout);
  a.dq = view(p.dq);
  a.dk = view(p.dk);
  a.dv = view(p.dv);
  a.lse = p.lse;
  a.delta = static_cast<float*>(p.workspace);
  a.cu_q = p.cu_seqlens_q;
  a.cu_k = p.cu_seqlens_k;
  a.lse_head = p.lse_stride_head;
  a.lse_batch = p.cu_seqlens_q ? 0 : p.lse_stride_head * p.heads_q;
  a.rows_q = p.rows_q;
  a.rows_k = p.rows_k;
  a.heads_q = p.heads_q;
  a.heads_kv = p.heads_kv;
  a.stat_size = (int64_t)p.heads_q * p.lse_stride_head * (p.cu_seqlens_q ? 1 : p.batch);
  a.group = p.heads_q / p.heads_kv;
  a.batch = p.batch;
  a.dim = p.head_dim;
  a.max_q = p.max_q;
  a.max_k = p.max_k;
  a.causal = p.causal != 0;
  a.window = p.window;
  a.scale = p.scale;
  a.parts = 1;
  return a;
}

typedef void (*AttnFn)(AttnArgs);

int blocks_of(int rows) { return (int)(((int64_t)rows + kRows - 1) / kRows); }

// Causal rows differ in length: the first block of 128 sees one or two tiles,
// the last all.  Once there are more workgroups than the device holds (two a
// CU), a workgroup takes block i and block n - 1 - i, so all are as long and
// none runs on alone at the end (8192 tokens, 16 heads of 128: forward 303 us
// one by one, 281 us in pairs; 2 x 4096: 160 and 150).
// pieces: workgroups a block.
int launch(const char* name, AttnFn fn, AttnArgs a, int heads, int blocks, int pieces, bool may_pair, hipStream_t stream) {
  constexpr int64_t kResident = 512;
  a.blocks = blocks;
  a.paired = may_pair && a.causal && !a.window && !a.cu_q && (int64_t)a.batch * heads * blocks > kResident;
  const int64_t groups = (int64_t)a.batch * heads * (a.paired ? (blocks + 1) / 2 : blocks) * pieces;
  if (groups == 0) return FP8DS_OK;
  if (groups > 0x7FFFFFFF) return set_error(FP8DS_EUNSUPPORTED, "%s: %lld workgroups exceed the grid limit", name, (long long)groups);
  hipLaunchKernelGGL(fn, dim3((unsigned)groups), dim3(64 * kWaves), 0, stream, a);
  return check_launch(name);
}

#define FP8DS_ATTN_PICK(kernel, dim, bf) \
  ((dim) > 64 ? ((bf) ? kernel<128, true> : kernel<128, false>) : ((bf) ? kernel<64, true> : kernel<64, false>))

}  // namespace

int launch_attn_forward(const fp8ds_attn_args& p, hipStream_t stream) {
  const AttnArgs a = make_args(p);
  return launch("attn_forward", FP8DS_ATTN_PICK(attn_fwd_kernel, p.head_dim, p.type == FP8DS_IN_BF16), a, p.heads_q,
                blocks_of(p.max_q), 1, true, stream);
}

int launch_attn_backward(const fp8ds_attn_args& p, hipStream_t stream) {
  const AttnArgs a = make_args(p);
  const bool bf = p.type == FP8DS_IN_BF16;
  // The rounding of O adds 22 % to dQ's error at 64 keys, 4 % at 512, 2 % at 1024;
  // taking it out costs a product in four (4 x 512, heads of 64: 16.8 -> 18.3 us).
  const int keys = p.window > 0 && p.window < p.max_k ? p.window : p.max_k;
  const bool fix = keys <= 512, wide = p.head_dim > 64;
  const AttnFn dq = fix ? (wide ? (bf ? attn_dq_kernel<128, true, true> : attn_dq_kernel<128, false, true>)
                                : (bf ? attn_dq_kernel<64, true, true> : attn_dq_kernel<64, false, true>))
                        : (wide ? (bf ? attn_dq_kernel<128, true, false> : attn_dq_kernel<128, false, false>)
                                : (bf ? attn_dq_kernel<64, true, false> : attn_dq_kernel<64, false, false>));
  if (const int st = launch("attn_backward", dq, a, p.heads_q, blocks_of(p.max_q), 1, true, stream)) return st;
  AttnArgs b = a;
  b.parts = dkv_parts(p);
  b.units = dkv_units(p);
  b.partial = reinterpret_cast<float*>(static_cast<char*>(p.workspace) + stats_bytes(p));
  const AttnFn dkv = FP8DS_ATTN_PICK(attn_dkv_kernel, p.head_dim, bf);
  const int blocks = blocks_of(p.max_k);
  if (const int st = launch("attn_backward", dkv, b, p.heads_kv, blocks * b.parts, 1, false, stream)) return st;
  if (b.parts == 1) return FP8DS_OK;
  return launch("attn_backward", FP8DS_ATTN_PICK(attn_join_kernel, p.head_dim, bf), b, p.heads_kv, blocks, wide ? 8 : 4,
                false, stream);
}

size_t attn_backward_workspace(const fp8ds_attn_args& p) {
  if (p.heads_kv <= 0 || p.head_dim <= 0 || p.max_q < 0 || p.max_k < 0 || p.rows_k < 0) return stats_bytes(p);
  const int parts = dkv_parts(p);
  const size_t width = p.head_dim > 64 ? 128 : 64;
  return stats_bytes(p) + (parts > 1 ? (size_t)parts * (size_t)dkv_units(p) * (2 * kRows * width * sizeof(float)) : 0);
}

}  // namespace fp8ds
