// Dense product with packed weights and a fused epilogue,
//   out = bf16( [residual +] [mul *] act( x . W + bias ) ),
// W[k][n] = scale[n][k/32] * (level[n][k] - offset) in the packed format of
// include/moe.h.  (The pages name the code families of the weights, "Xolotl"
// card, README "Quick start"; the product and its epilogue are this library's.)
//
// Two kernels, by the number of rows T:
//   few rows: bound by the packed bytes.  Exact bf16 levels on 16x16x32 ops,
//     each 32-group's partial sum multiplied by its fp16 scale in fp32, K
//     split over the waves of a block.  One launch.
//   many rows: bound by the matrix cores.  The scale goes into an fp16
//     operand, so that one 32x32x16 op follows another over the whole of K.
//     Rows and columns are first given powers of two (staging launch).
#include <hip/hip_runtime.h>

#include <type_traits>

#include "device_common.h"
#include "moe_internal.h"

namespace bqmoe {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) void lds_void;

// --------------------------------------------------------------- epilogue
__device__ __forceinline__ float sigmoid_f(float v) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.4426950408889634f * v));
}

// act(v) in fp32 (exponential and reciprocal by the hardware, one unit in the
// last place each; the result is rounded to bf16 right after)
__device__ __forceinline__ float activate(int act, float v) {
  switch (act) {
    case MOE_ACT_SILU: return v * sigmoid_f(v);
    case MOE_ACT_GELU: return 0.5f * v * erfcf(-0.70710678118654752f * v);
    case MOE_ACT_GELU_TANH:
      return v * sigmoid_f(1.5957691216057308f * (v + 0.044715f * v * v * v));
    case MOE_ACT_RELU: return v < 0.f ? 0.f : v;
    case MOE_ACT_RELU2: return v < 0.f ? 0.f : v * v;
    case MOE_ACT_SIGMOID: return sigmoid_f(v);
  }
  return v;
}

__device__ __forceinline__ void finish(const LinArgs& A, float v, int t, int n) {
  if (A.bias) v += A.bias[n];
  v = activate(A.act, v);
  if (A.mul) v *= bf16_to_f32(A.mul[(int64_t)t * A.ldm + n]);
  if (A.res) v += bf16_to_f32(A.res[(int64_t)t * A.ldr + n]);
  A.out[(int64_t)t * A.ldo + n] = (uint16_t)f32_to_bf16(v);
}

// Eight consecutive columns at once (16-byte loads and stores).
__device__ __forceinline__ void finish8(const LinArgs& A, float (&v)[8], int t, int n) {
  if (A.bias) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] += A.bias[n + j];
  }
  if (A.act != MOE_ACT_NONE) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = activate(A.act, v[j]);
  }
  if (A.mul) {
    const u32x4 m = *reinterpret_cast<const u32x4*>(A.mul + (int64_t)t * A.ldm + n);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] *= bf16_to_f32((m[j >> 1] >> (16 * (j & 1))) & 0xFFFFu);
  }
  if (A.res) {
    const u32x4 m = *reinterpret_cast<const u32x4*>(A.res + (int64_t)t * A.ldr + n);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] += bf16_to_f32((m[j >> 1] >> (16 * (j & 1))) & 0xFFFFu);
  }
  u32x4 o;
#pragma unroll
  for (int j = 0; j < 4; ++j) o[j] = f32_to_bf16(v[2 * j]) | (f32_to_bf16(v[2 * j + 1]) << 16);
  *reinterpret_cast<u32x4*>(A.out + (int64_t)t * A.ldo + n) = o;
}

// --------------------------------------------------------------- few rows
// Levels as bf16 values on two bases, without a subtraction: a 2-bit field at
// bit 2 of a mantissa under 1.0 makes it 1 + u/32, at bit 4 under 0.25 makes
// it 0.25 + u/32 (the third bit of a 3-bit level goes above the field).  The
// fields of k-slots (2v, 2v + 1), v = 0, 1, are shifted to bit 2, those of
// v = 2, 3 to bit 4.  The constant part is taken off by a second op whose
// operand is -(base + offset/32) in every column (exact in bf16 for the three
// offsets): it gives the first op's C operand, so D = sum_k x_k (u - offset) / 32.
struct LevelK {
  uint32_t m2, m4, b2, b4, c2, c4;  // masks, bases and constants at bits 2 and 4
};

template <bool Q3, int GB>
__device__ __forceinline__ u32x4 levels_bf16(uint32_t w, uint32_t w1, const LevelK& k) {
  u32x4 r;
  if (GB & 1) {
    r[0] = ((w >> 6) & k.m2) | k.b2;
    r[1] = ((w >> 8) & k.m2) | k.b2;
    r[2] = ((w >> 8) & k.m4) | k.b4;
    r[3] = ((w >> 10) & k.m4) | k.b4;
  } else {
    r[0] = ((w << 2) & k.m2) | k.b2;
    r[1] = (w & k.m2) | k.b2;
    r[2] = (w & k.m4) | k.b4;
    r[3] = ((w >> 2) & k.m4) | k.b4;
  }
  if (Q3) {  // bit 2 of the level: to bit 4 (v = 0, 1) or 6 (v = 2, 3)
    constexpr int s = GB == 0 ? 0 : GB == 1 ? 1 : GB == 2 ? 6 : 7;
    const uint32_t h0 = s <= 2 ? w1 << (2 - s) : w1 >> (s - 2), h12 = w1 >> s;
    const uint32_t h3 = GB == 0 ? w1 << 6 : GB == 1 ? w1 << 5 : GB == 2 ? w1 >> 8 : w1 >> 9;
    r[0] = bit_insert(0x00100010u, h0, r[0]);
    r[1] = bit_insert(0x00100010u, h12, r[1]);
    r[2] = bit_insert(0x00400040u, h12, r[2]);
    r[3] = bit_insert(0x00400040u, h3, r[3]);
  }
  return r;
}

// Block: one n-tile (16 columns), W waves, wave w the k-blocks w, w + W, ...
// Operand A is x: lane l supplies row l%16, which is token
// 16 mt + (l%16)/4 + 4 (l%4), so that accumulator register i holds tokens
// 4i .. 4i+3 (one per lane quarter) and RI = ceil(T/4) registers do (MT = 1).
template <bool Q3, int MT, int RI, int KU>
__global__ __launch_bounds__(512) void k_lin_few(LinArgs A, LevelK lk, int T) {
  extern __shared__ __attribute__((aligned(16))) float s_part[];  // [W][MT][16][16]
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int W = blockDim.x >> 6, nt = blockIdx.x, KB = A.K / 128;
  const int r = lane & 15, q = lane >> 4;
  LevelK k = lk;
  k.b2 = lane_copy(lk.b2);
  k.b4 = lane_copy(lk.b4);
  const u32x4 cb = {lane_copy(lk.c2), lane_copy(lk.c2), lane_copy(lk.c4), lane_copy(lk.c4)};
  const uint8_t* w0 = A.w + (size_t)nt * KB * 512 + lane * 8;
  const uint8_t* w1 = A.w + A.plane1 + (size_t)nt * KB * 256 + lane * 4;
  const uint8_t* sc = A.w + A.scales + (size_t)nt * KB * 128 + r * 8;
  const uint16_t* xr[MT];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    const int t = 16 * mt + (r >> 2) + 4 * (r & 3);  // rows past T repeat the last (not stored)
    xr[mt] = A.x + (int64_t)min(t, T - 1) * A.ldx + 8 * q;
  }
  float acc[MT][RI];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int i = 0; i < RI; ++i) acc[mt][i] = 0.f;

  struct Chunk {
    u32x2 w[KU], s[KU];
    uint32_t w1[KU];
    u32x4 x[KU][MT][4];
  };
  auto load = [&](int kb0, Chunk& c) __attribute__((always_inline)) {
#pragma unroll
    for (int u = 0; u < KU; ++u) {
      const int kb = min(kb0 + u * W, KB - 1);
      c.w[u] = *reinterpret_cast<const u32x2*>(w0 + (size_t)kb * 512);
      if (Q3) c.w1[u] = *reinterpret_cast<const uint32_t*>(w1 + (size_t)kb * 256);
      c.s[u] = *reinterpret_cast<const u32x2*>(sc + (size_t)kb * 128);
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int g = 0; g < 4; ++g)
          c.x[u][mt][g] = *reinterpret_cast<const u32x4*>(xr[mt] + (size_t)kb * 128 + 32 * g);
    }
  };
  auto group = [&](auto gc, const Chunk& c, int u) __attribute__((always_inline)) {
    constexpr int GB = decltype(gc)::value;
    const u32x4 b = levels_bf16<Q3, GB>(c.w[u][GB / 2], Q3 ? c.w1[u] : 0u, k);
    const float s = f16_to_f32((c.s[u][GB / 2] >> (16 * (GB & 1))) & 0xFFFFu);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      f32x4 d = mfma32(c.x[u][mt][GB], cb, f32x4{0.f, 0.f, 0.f, 0.f});
      d = mfma32(c.x[u][mt][GB], b, d);
#pragma unroll
      for (int i = 0; i < RI; ++i) acc[mt][i] = fmaf(s, d[i], acc[mt][i]);
    }
  };
  Chunk c;
  for (int kb0 = wave; kb0 < KB; kb0 += W * KU) {
    load(kb0, c);
#pragma unroll
    for (int u = 0; u < KU; ++u)
      if (kb0 + u * W < KB) {
        group(std::integral_constant<int, 0>{}, c, u);
        group(std::integral_constant<int, 1>{}, c, u);
        group(std::integral_constant<int, 2>{}, c, u);
        group(std::integral_constant<int, 3>{}, c, u);
      }
  }
  // sum over the waves in order; register i of lane (r, q) is token 16 mt + 4 i + q, column r
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int i = 0; i < RI; ++i)
      s_part[((wave * MT + mt) * 16 + 4 * i + q) * 16 + r] = acc[mt][i];
  __syncthreads();
  const int outs = min(T, 16 * MT) * 16;
  for (int o = tid; o < outs; o += blockDim.x) {
    float v = 0.f;
    for (int w = 0; w < W; ++w) v += s_part[w * MT * 256 + o];
    finish(A, v * 32.f, o >> 4, nt * 16 + (o & 15));
  }
}

// --------------------------------------------------------------- many rows
// Staging.  One wave per row: e = (exponent of max|x|) - 14, in [-100, 114];
// xs = fp16(x * 2^-e), exact for values down to 2^-31 of the row's maximum,
// rscale = 2^e.  The blocks after the rows take 256 columns each: cscale =
// 2^-f, where 2^f (in fp16, f at most 15) brings the column's largest |scale|
// to [2^13, 2^14), so that scale * level keeps 11 bits however small a
// column's scales are.
__global__ __launch_bounds__(256) void k_lin_stage(LinArgs A, int T, uint16_t* __restrict__ xs,
                                                   float* __restrict__ rscale,
                                                   float* __restrict__ cscale, int row_blocks) {
  const int K = A.K;
  if ((int)blockIdx.x >= row_blocks) {
    const int n = ((int)blockIdx.x - row_blocks) * 256 + threadIdx.x;
    if (n >= A.N) return;
    const int KB = K / 128;
    const uint8_t* sc = A.w + A.scales + (size_t)(n >> 4) * KB * 128 + (n & 15) * 8;
    uint32_t m = 0;
    for (int kb = 0; kb < KB; ++kb) {
      const u32x2 v = *reinterpret_cast<const u32x2*>(sc + (size_t)kb * 128);
      m = max(m, max(max(v[0] & 0x7FFFu, (v[0] >> 16) & 0x7FFFu),
                     max(v[1] & 0x7FFFu, (v[1] >> 16) & 0x7FFFu)));
    }
    // exponent of the largest scale (a subnormal one counts as 2^-15, an
    // infinite or zero one leaves the column as it is)
    const int ex = (int)(m >> 10) - 15;
    const int f = m == 0 || m >= 0x7C00u ? 0 : min(15, 13 - ex);
    cscale[n] = __uint_as_float((uint32_t)(127 - f) << 23);
    return;
  }
  const int row = blockIdx.x * 4 + (threadIdx.x >> 6), lane = threadIdx.x & 63;
  if (row >= T) return;
  const uint16_t* s = A.x + (int64_t)row * A.ldx;
  uint16_t* d = xs + (size_t)row * K;
  uint32_t m = 0;
  for (int i = lane * 8; i < K; i += 512) {
    const uint4 v = *reinterpret_cast<const uint4*>(s + i);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) m = max(m, max(w[j] & 0x7FFFu, (w[j] >> 16) & 0x7FFFu));
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, o));
  const int e = min(114, max(-100, (int)(m >> 7) - 127 - 14));
  const float f = __uint_as_float((uint32_t)(127 - e) << 23);
  for (int i = lane * 8; i < K; i += 512) {
    const uint4 v = *reinterpret_cast<const uint4*>(s + i);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const _Float16 lo = (_Float16)(bf16_to_f32(w[j] & 0xFFFFu) * f);
      const _Float16 hi = (_Float16)(bf16_to_f32(w[j] >> 16) * f);
      o[j] = (uint32_t)__builtin_bit_cast(uint16_t, lo) |
             ((uint32_t)__builtin_bit_cast(uint16_t, hi) << 16);
    }
    *reinterpret_cast<uint4*>(d + i) = make_uint4(o[0], o[1], o[2], o[3]);
  }
  if (lane == 0) rscale[row] = __uint_as_float((uint32_t)(127 + e) << 23);
}

// Weight operand of one lane: 8 values of one column and 32-group GB as fp16,
// s * (u - offset) * fac with fac = 1, 1/2, 1/4 (ternary, 2-bit, 3-bit; so
// that no factor overflows): a mask-and-or puts the level into the mantissa of
// an fp16 base where its lowest bit is worth 1 (bit 2 under 256, bit 4 under
// 64, bit 6 under 16), one packed FMA gives (u - offset) * fac exactly, one
// packed multiply by the scale rounds to fp16's 11 bits.  That rounding is
// exact for ternary weights and at most 2^-12 of a 2- or 3-bit weight
// otherwise: an error of about 1e-4 of the result's size, against 1.7e-3 of
// its rounding to bf16; keeping the scales out of the operand would cost a
// vector FMA per result and 32-group, as much time as the matrix cores'.
struct OperandK {
  uint32_t m2, m4, m6, b2, b4, b6, o2, o4, o6;
};

template <int Q, int GB>
__device__ __forceinline__ u32x4 weights_f16(uint32_t w, uint32_t w1, uint32_t s2,
                                             const OperandK& k) {
  const uint32_t x1 = (GB & 1) ? w >> 8 : w, x0 = (GB & 1) ? w >> 6 : w << 2;
  uint32_t f[4] = {(x0 & k.m2) | k.b2, (x1 & k.m2) | k.b2, (x1 & k.m4) | k.b4,
                   (x1 & k.m6) | k.b6};
  if (Q == MOE_Q_INT3) {
    constexpr int s = GB == 0 ? 0 : GB == 1 ? 1 : GB == 2 ? 6 : 7;
    const uint32_t h0 = s <= 2 ? w1 << (2 - s) : w1 >> (s - 2), h12 = w1 >> s;
    const uint32_t h3 = GB == 0 ? w1 << 8 : GB == 1 ? w1 << 7 : GB == 2 ? w1 >> 6 : w1 >> 7;
    f[0] = bit_insert(0x00100010u, h0, f[0]);
    f[1] = bit_insert(0x00100010u, h12, f[1]);
    f[2] = bit_insert(0x00400040u, h12, f[2]);
    f[3] = bit_insert(0x01000100u, h3, f[3]);
  }
  constexpr uint32_t fac = Q == MOE_Q_INT3 ? 0x34003400u : 0x38003800u;  // 1/4, 1/2
  u32x4 r;
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    const f16x2 o = __builtin_bit_cast(f16x2, v < 2 ? k.o2 : v == 2 ? k.o4 : k.o6);
    const f16x2 c = Q == MOE_Q_TERNARY
                        ? __builtin_bit_cast(f16x2, f[v]) + o
                        : __builtin_bit_cast(f16x2, f[v]) * __builtin_bit_cast(f16x2, fac) + o;
    r[v] = __builtin_bit_cast(uint32_t, c * __builtin_bit_cast(f16x2, s2));
  }
  return r;
}

__device__ __forceinline__ f32x16 mfma_lin(u32x4 a, u32x4 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a),
                                                __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// s_waitcnt immediate: vector-memory count vm (0..63), LDS count lgkm
constexpr int wait_vm_lgkm(int vm, int lgkm) {
  return (vm & 15) | (7 << 4) | ((lgkm & 15) << 8) | ((vm >> 4) << 14);
}

constexpr int kRsrcLin = 0x00020000;  // buffer resource word 3: raw 32-bit dwords

// 64 lanes x 16 bytes straight into LDS, lane l's at at + 16 l
__device__ __forceinline__ void load_lds16(const void* base, uint8_t* at, uint32_t off, int soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(
      __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, -1, kRsrcLin), (lds_void*)at,
      16, off, soff, 0, 0);
}

// Block: a tile of 32 NRT rows and W waves of 32 CT columns each.  Per 128-wide
// k-step the block's fp16 rows go into a ring of three LDS stages (direct
// loads two steps ahead), each wave's packed words and scales into registers
// one step ahead; the wave builds its weight operands in registers, each
// feeding NRT matrix-core ops.
template <int Q, int NRT, int W, int CT>
__global__ __launch_bounds__(64 * W, 1) void k_lin_gemm(LinArgs A, OperandK kk,
                                                        const uint16_t* __restrict__ xs,
                                                        const float* __restrict__ rscale,
                                                        const float* __restrict__ cscale, int T,
                                                        int row_tiles, int ncol) {
  extern __shared__ __attribute__((aligned(16))) uint8_t sbuf[];
  constexpr int R = 32 * NRT, kStage = R * 256, kDma = R / (4 * W);
  static_assert(R % (4 * W) == 0, "row split");
  constexpr bool Q3 = Q == MOE_Q_INT3;
  // work item = (row tile, column group), tile-major; each XCD takes one
  // contiguous chunk of the items (blocks go to the 8 XCDs round-robin)
  const int n_items = row_tiles * ncol, chunk = (n_items + 7) / 8;
  const int local = blockIdx.x / 8, item = (blockIdx.x % 8) * chunk + local;
  if (local >= chunk || item >= n_items) return;
  const int tile = item / ncol, col = item % ncol;
  const int tid = threadIdx.x, lane = tid & 63, l32 = lane & 31, hl = lane >> 5, r = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int K = A.K, N = A.N, S = K / 128, NT = N / 16;
  const int row0 = tile * R;

  // LDS: row i of a stage at i * 256, its 16-byte chunk c (8 k) in slot
  // c ^ (i % 16); 16 lanes load one row.  Rows past T repeat the last one.
  const uint16_t* const xrow = xs + (size_t)row0 * K;
  uint32_t aoffs[kDma];
#pragma unroll
  for (int i = 0; i < kDma; ++i) {
    const int row = 4 * kDma * wave + 4 * i + (lane >> 4);
    aoffs[i] = (uint32_t)min(row, T - 1 - row0) * (uint32_t)(2 * K) +
               (((lane & 15) ^ (row & 15)) << 4);
  }
  const uint32_t la = (uint32_t)(l32 * 256) | ((uint32_t)(hl ^ (l32 & 15)) << 4);

  OperandK k = kk;
  k.b2 = lane_copy(kk.b2);
  k.b4 = lane_copy(kk.b4);
  k.b6 = lane_copy(kk.b6);

  // packed weights: column tile ct of the wave is n-tiles 2c, 2c + 1 of
  // c = (col W + wave) CT + ct; tiles past N repeat the last one (not stored)
  uint32_t wo[CT], po[CT], so[CT];
  uint32_t cm[CT];  // 2^f of the lane's column, twice
#pragma unroll
  for (int ct = 0; ct < CT; ++ct) {
    const int c32 = (col * W + wave) * CT + ct;
    const uint32_t nt = (uint32_t)min(2 * c32 + (l32 >> 4), NT - 1);
    wo[ct] = nt * S * 512 + (16 * hl + r) * 8;
    po[ct] = (uint32_t)A.plane1 + nt * S * 256 + (16 * hl + r) * 4;
    so[ct] = (uint32_t)A.scales + nt * S * 128 + r * 8;
    const uint32_t ex = (__float_as_uint(cscale[nt * 16 + r]) >> 23) & 0xFFu;  // 127 - f
    const uint32_t h = (127u + 15u - ex) << 10;
    cm[ct] = h | (h << 16);
  }

  f32x16 acc[NRT][CT];
#pragma unroll
  for (int rt = 0; rt < NRT; ++rt)
#pragma unroll
    for (int ct = 0; ct < CT; ++ct)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[rt][ct][i] = 0.f;

  struct Words {
    u32x2 w[CT][2], s[CT];
    uint32_t w1[CT][2];
  };
  auto issue = [&](int s, int buf) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < kDma; ++i)
      load_lds16(xrow, sbuf + buf * kStage + (kDma * wave + i) * 1024, aoffs[i], s * 256);
  };
  auto loadb = [&](int s, Words& b) __attribute__((always_inline)) {
    const __amdgpu_buffer_rsrc_t rB =
        __builtin_amdgcn_make_buffer_rsrc((void*)A.w, 0, -1, kRsrcLin);
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        b.w[ct][h] = __builtin_bit_cast(
            u32x2, __builtin_amdgcn_raw_buffer_load_b64(rB, (int)wo[ct], s * 512 + 256 * h, 0));
        if (Q3)
          b.w1[ct][h] = __builtin_amdgcn_raw_buffer_load_b32(rB, (int)po[ct], s * 256 + 128 * h, 0);
      }
      b.s[ct] = __builtin_bit_cast(
          u32x2, __builtin_amdgcn_raw_buffer_load_b64(rB, (int)so[ct], s * 128, 0));
    }
  };
  auto build = [&](auto qc, const Words& b, u32x4 (&o)[CT]) __attribute__((always_inline)) {
    constexpr int GB = decltype(qc)::value >> 1, h = decltype(qc)::value & 1;
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
      const uint32_t sh = (b.s[ct][GB >> 1] >> (16 * (GB & 1))) & 0xFFFFu;
      const uint32_t s2 = __builtin_bit_cast(
          uint32_t, __builtin_bit_cast(f16x2, sh | (sh << 16)) * __builtin_bit_cast(f16x2, cm[ct]));
      o[ct] = weights_f16<Q, GB>(b.w[ct][h][GB >> 1], Q3 ? b.w1[ct][h] : 0u, s2, k);
    }
  };
  auto loada = [&](uint32_t at, int q, u32x4 (&a)[NRT]) __attribute__((always_inline)) {
    const uint8_t* p = sbuf + (at ^ (uint32_t)((2 * q) << 4));
#pragma unroll
    for (int rt = 0; rt < NRT; ++rt) a[rt] = *reinterpret_cast<const u32x4*>(p + rt * 8192);
  };
  auto mfmas = [&](const u32x4 (&a)[NRT], const u32x4 (&b)[CT]) __attribute__((always_inline)) {
#pragma unroll
    for (int rt = 0; rt < NRT; ++rt)
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) acc[rt][ct] = mfma_lin(a[rt], b[ct], acc[rt][ct]);
  };
  // sub-step q of a step (group q/2, k-half q%2): the next sub-step's rows are
  // read and its weights built while this one's matrix-core ops run
  auto sub = [&](auto qc, uint32_t at, const Words& b, const Words& bn, u32x4 (&a0)[NRT],
                 u32x4 (&a1)[NRT], u32x4 (&o0)[CT], u32x4 (&o1)[CT])
      __attribute__((always_inline)) {
    constexpr int q = decltype(qc)::value;
    if constexpr (q < 7) loada(at, q + 1, a1);
    if constexpr (q < 7)
      build(std::integral_constant<int, q + 1>{}, b, o1);
    else
      build(std::integral_constant<int, 0>{}, bn, o1);
    mfmas(a0, o0);
#pragma unroll
    for (int i = 0; i < NRT * CT; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x002, Q3 ? 7 : 5, 0);
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  Words wa, wb;
  u32x4 a0[NRT], a1[NRT], o0[CT], o1[CT];
  issue(0, 0);
  loadb(0, wa);
  issue(min(1, S - 1), 1);
  build(std::integral_constant<int, 0>{}, wa, o0);
  int st = 0;  // ring stage of step s
  auto step = [&](int s, const Words& b, Words& bn) __attribute__((always_inline)) {
    // step s is in LDS for every wave (step s + 1's direct loads may remain in
    // flight) and every wave is done with step s - 1's stage, which the loads
    // of step s + 2 overwrite
    __builtin_amdgcn_s_waitcnt(wait_vm_lgkm(kDma, 0));
    __builtin_amdgcn_s_barrier();
    const int st2 = st == 0 ? 2 : st - 1;
    const uint32_t at = la + (uint32_t)(st * kStage);
    loada(at, 0, a0);
    __builtin_amdgcn_sched_barrier(0);
    // loads past the last step repeat it, so that a step has no branch
    loadb(min(s + 1, S - 1), bn);
    issue(min(s + 2, S - 1), st2);
    __builtin_amdgcn_sched_barrier(0);
    sub(std::integral_constant<int, 0>{}, at, b, bn, a0, a1, o0, o1);
    sub(std::integral_constant<int, 1>{}, at, b, bn, a1, a0, o1, o0);
    sub(std::integral_constant<int, 2>{}, at, b, bn, a0, a1, o0, o1);
    sub(std::integral_constant<int, 3>{}, at, b, bn, a1, a0, o1, o0);
    sub(std::integral_constant<int, 4>{}, at, b, bn, a0, a1, o0, o1);
    sub(std::integral_constant<int, 5>{}, at, b, bn, a1, a0, o1, o0);
    sub(std::integral_constant<int, 6>{}, at, b, bn, a0, a1, o0, o1);
    sub(std::integral_constant<int, 7>{}, at, b, bn, a1, a0, o1, o0);
    st = st == 2 ? 0 : st + 1;
  };
  int s = 0;
  for (; s + 1 < S; s += 2) {
    step(s, wa, wb);
    step(s + 1, wb, wa);
  }
  if (s < S) step(s, wa, wb);
  __builtin_amdgcn_s_waitcnt(wait_vm_lgkm(0, 0));  // the repeated last loads have landed

  // Epilogue: register i of acc[rt][ct] is row rt*32 + 8(i/4) + 4 hl + i%4,
  // column l32.  Each wave turns 64 x 32 results at a time in LDS of its own
  // (rows 40 floats apart, free of bank conflicts), so that a lane finishes 8
  // consecutive columns.
  __builtin_amdgcn_s_barrier();  // the ring is free
  constexpr int kTurn = 40, kRt = NRT < 2 ? 1 : 2;
  static_assert(W * kRt * 32 * kTurn * 4 <= 3 * kStage && NRT % kRt == 0, "turning area");
  float* const turn = reinterpret_cast<float*>(sbuf) + wave * kRt * 32 * kTurn;
  constexpr float unfac = Q == MOE_Q_TERNARY ? 1.f : Q == MOE_Q_INT2 ? 2.f : 4.f;
#pragma unroll
  for (int ct = 0; ct < CT; ++ct) {
    const int n0 = ((col * W + wave) * CT + ct) * 32;
    const float cs = unfac * cscale[min(n0 + l32, N - 1)];
#pragma unroll
    for (int r0 = 0; r0 < NRT; r0 += kRt) {
#pragma unroll
      for (int rt = 0; rt < kRt; ++rt)
#pragma unroll
        for (int i = 0; i < 16; ++i)
          turn[(rt * 32 + 8 * (i >> 2) + 4 * hl + (i & 3)) * kTurn + l32] = acc[r0 + rt][ct][i] * cs;
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
      const int n = n0 + 8 * (lane & 3);
#pragma unroll 1
      for (int p = 0; p < 2 * kRt; ++p) {
        const int m = 16 * p + (lane >> 2), t = row0 + r0 * 32 + m;
        if (t < T && n < N) {
          const f32x4 v0 = *reinterpret_cast<const f32x4*>(turn + m * kTurn + 8 * (lane & 3));
          const f32x4 v1 = *reinterpret_cast<const f32x4*>(turn + m * kTurn + 8 * (lane & 3) + 4);
          const float rs = rscale[t];
          float v[8];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            v[j] = v0[j] * rs;
            v[4 + j] = v1[j] * rs;
          }
          finish8(A, v, t, n);
        }
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
    }
  }
}

// ------------------------------------------------------------------ launch
LinWs lin_ws_layout(int K, int N, int T) {
  LinWs w{};
  if (T <= kLinFewRows) {
    w.total = 256;
    return w;
  }
  const auto up = [](size_t v) { return (v + 255) & ~size_t(255); };
  w.xs = 0;
  w.rscale = up((size_t)T * K * 2);
  w.cscale = up(w.rscale + (size_t)T * 4);
  w.total = up(w.cscale + (size_t)N * 4);
  return w;
}

template <bool Q3>
static void few(const LinArgs& A, int T, hipStream_t s) {
  const int KB = A.K / 128, W = KB < 8 ? KB : 8;
  const uint32_t off = A.q == MOE_Q_TERNARY ? 2u : A.q == MOE_Q_INT2 ? 3u : 7u;  // 2 * offset
  // -(32 + offset) / 32 and -(8 + offset) / 32 as bf16 pairs
  const auto pair = [](float v) {
    uint32_t u;
    __builtin_memcpy(&u, &v, 4);
    return (u >> 16) | (u & 0xFFFF0000u);
  };
  const LevelK lk = {0x000C000Cu,          0x00300030u,
                     0x3F803F80u,          0x3E803E80u,
                     pair(-(64.f + off) / 64.f), pair(-(16.f + off) / 64.f)};
  const dim3 g(A.N / 16), b(64 * W);
#define BQ_LF(MT, RI, KU) \
  hipLaunchKernelGGL((k_lin_few<Q3, MT, RI, KU>), g, b, W * MT * 1024, s, A, lk, T)
  if (T <= 4)
    BQ_LF(1, 1, 4);
  else if (T <= 8)
    BQ_LF(1, 2, 4);
  else if (T <= 16)
    BQ_LF(1, 4, 4);
  else if (T <= 32)
    BQ_LF(2, 4, 2);
  else
    BQ_LF(4, 4, 1);
#undef BQ_LF
}

template <int Q, int NRT, int W, int CT>
static int gemm(const LinArgs& A, const OperandK& k, int T, uint8_t* ws, const LinWs& L,
                hipStream_t s) {
  const int tiles = (T + 32 * NRT - 1) / (32 * NRT), ncol = (A.N + 32 * CT * W - 1) / (32 * CT * W);
  const size_t lds = 3 * 32 * NRT * 256;
  if (lds > 65536 &&
      hipFuncSetAttribute((const void*)k_lin_gemm<Q, NRT, W, CT>,
                          hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds) != hipSuccess)
    return (int)hipErrorInvalidConfiguration;
  const int items = tiles * ncol;
  hipLaunchKernelGGL((k_lin_gemm<Q, NRT, W, CT>), dim3((items + 7) / 8 * 8), dim3(64 * W), lds, s,
                     A, k, (const uint16_t*)(ws + L.xs), (const float*)(ws + L.rscale),
                     (const float*)(ws + L.cscale), T, tiles, ncol);
  return (int)hipGetLastError();
}

template <int Q>
static int many(const LinArgs& A, int T, uint8_t* ws, hipStream_t s) {
  const LinWs L = lin_ws_layout(A.K, A.N, T);
  const int row_blocks = (T + 3) / 4;
  hipLaunchKernelGGL(k_lin_stage, dim3(row_blocks + (A.N + 255) / 256), dim3(256), 0, s, A, T,
                     (uint16_t*)(ws + L.xs), (float*)(ws + L.rscale), (float*)(ws + L.cscale),
                     row_blocks);
  // -(base + offset) * fac for the bases 256, 64, 16
  OperandK k = {0x000C000Cu, 0x00300030u, 0x00C000C0u, 0x5C005C00u, 0x54005400u, 0x4C004C00u,
                0, 0, 0};
  const auto pair = [](float v) {
    const _Float16 h = (_Float16)v;
    uint16_t u;
    __builtin_memcpy(&u, &h, 2);
    return (uint32_t)u | ((uint32_t)u << 16);
  };
  const float off = qtype_offset(Q), fac = Q == MOE_Q_TERNARY ? 1.f : Q == MOE_Q_INT2 ? .5f : .25f;
  k.o2 = pair(-(256.f + off) * fac);
  k.o4 = pair(-(64.f + off) * fac);
  k.o6 = pair(-(16.f + off) * fac);
  const long blocks = (long)((T + 127) / 128) * ((A.N + 511) / 512);
  if (blocks >= 192) return gemm<Q, 4, 8, 2>(A, k, T, ws, L, s);
  return gemm<Q, 2, 4, 1>(A, k, T, ws, L, s);
}

int launch_linear(const LinArgs& A, int T, uint8_t* ws, void* stream) {
  hipStream_t s = (hipStream_t)stream;
  if (T <= kLinFewRows) {
    if (A.q == MOE_Q_INT3)
      few<true>(A, T, s);
    else
      few<false>(A, T, s);
    return (int)hipGetLastError();
  }
  if (A.q == MOE_Q_TERNARY) return many<MOE_Q_TERNARY>(A, T, ws, s);
  if (A.q == MOE_Q_INT2) return many<MOE_Q_INT2>(A, T, ws, s);
  return many<MOE_Q_INT3>(A, T, ws, s);
}

}  // namespace bqmoe
