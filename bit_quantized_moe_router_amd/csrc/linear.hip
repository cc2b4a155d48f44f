// Dense product with packed weights and a fused epilogue,
//   out = bf16( [residual +] [mul *] act( x . W + bias ) ),
// W[k][n] = scale[n][k/32] * (level[n][k] - offset) in the packed format of
// include/moe.h.  (The pages name the code families of the weights, "Xolotl"
// card, README "Quick start"; the product and its epilogue are this library's.)
//
// Three kernels, by the number of rows T and tiles:
//   few rows: bound by the packed bytes.  Exact bf16 levels on 16x16x32 ops,
//     each 32-group's partial sum multiplied by its fp16 scale in fp32, K
//     split over the waves of a block.  One launch.
//   some rows: too few tiles to fill the chip, bound by latency.  The operands
//     of the next kernel, K split over blocks, their fp32 partial results
//     joined by a second launch with the epilogue.
//   many rows: bound by the matrix cores.  The scale goes into an fp16
//     operand, so that one 32x32x16 op follows another over the whole of K,
//     and the rows are turned to fp16 on their way into LDS.
#include <hip/hip_runtime.h>

#include <type_traits>
#include <utility>

#include "device_common.h"
#include "moe_internal.h"
#include "topk_common.h"

namespace bqmoe {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

// --------------------------------------------------------------- epilogue
__device__ __forceinline__ float sigmoid_f(float v) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.4426950408889634f * v));
}

// act(v) in fp32 (exponential and reciprocal by the hardware, one unit in the
// last place each; the result is rounded to bf16 right after).  The erf of
// GELU is Abramowitz and Stegun's 7.1.26 (absolute error 1.5e-7), in the form
// that gives erfc(|z|) = poly(t) exp(-z^2), t = 1 / (1 + 0.3275911 |z|).
template <int ACT>
__device__ __forceinline__ float activate(float v) {
  if (ACT == MOE_ACT_SILU) return v * sigmoid_f(v);
  if (ACT == MOE_ACT_GELU) {
    const float z = fabsf(v) * 0.70710678118654752f;
    const float t = __builtin_amdgcn_rcpf(fmaf(0.3275911f, z, 1.0f));
    const float p = t * fmaf(t, fmaf(t, fmaf(t, fmaf(t, 1.061405429f, -1.453152027f), 1.421413741f),
                                     -0.284496736f), 0.254829592f);
    const float c = 0.5f * p * __builtin_amdgcn_exp2f(-1.4426950408889634f * z * z);
    return v * (v < 0.f ? c : 1.0f - c);
  }
  if (ACT == MOE_ACT_GELU_TANH)
    return v * sigmoid_f(1.5957691216057308f * (v + 0.044715f * v * v * v));
  if (ACT == MOE_ACT_RELU) return v < 0.f ? 0.f : v;
  if (ACT == MOE_ACT_RELU2) return v < 0.f ? 0.f : v * v;
  if (ACT == MOE_ACT_SIGMOID) return sigmoid_f(v);
  return v;
}

// f(integral constant of the activation): one copy of f's code for each
template <typename F>
__device__ __forceinline__ void for_act(int act, F f) {
  switch (act) {
    case MOE_ACT_SILU: f(std::integral_constant<int, MOE_ACT_SILU>{}); break;
    case MOE_ACT_GELU: f(std::integral_constant<int, MOE_ACT_GELU>{}); break;
    case MOE_ACT_GELU_TANH: f(std::integral_constant<int, MOE_ACT_GELU_TANH>{}); break;
    case MOE_ACT_RELU: f(std::integral_constant<int, MOE_ACT_RELU>{}); break;
    case MOE_ACT_RELU2: f(std::integral_constant<int, MOE_ACT_RELU2>{}); break;
    case MOE_ACT_SIGMOID: f(std::integral_constant<int, MOE_ACT_SIGMOID>{}); break;
    default: break;
  }
}

__device__ __forceinline__ void finish(const LinArgs& A, float v, int t, int n) {
  if (A.bias) v += A.bias[n];
  for_act(A.act, [&](auto ac) { v = activate<decltype(ac)::value>(v); });
  if (A.mul) v *= bf16_to_f32(A.mul[(int64_t)t * A.ldm + n]);
  if (A.res) v += bf16_to_f32(A.res[(int64_t)t * A.ldr + n]);
  A.out[(int64_t)t * A.ldo + n] = (uint16_t)f32_to_bf16(v);
}

// Four consecutive columns at once (8-byte loads and stores).
__device__ __forceinline__ void finish4(const LinArgs& A, f32x4 v, int t, int n) {
  if (A.bias) {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] += A.bias[n + j];
  }
  for_act(A.act, [&](auto ac) {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = activate<decltype(ac)::value>(v[j]);
  });
  if (A.mul) {
    const u32x2 m = *reinterpret_cast<const u32x2*>(A.mul + (int64_t)t * A.ldm + n);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] *= bf16_to_f32((m[j >> 1] >> (16 * (j & 1))) & 0xFFFFu);
  }
  if (A.res) {
    const u32x2 m = *reinterpret_cast<const u32x2*>(A.res + (int64_t)t * A.ldr + n);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] += bf16_to_f32((m[j >> 1] >> (16 * (j & 1))) & 0xFFFFu);
  }
  u32x2 o;
#pragma unroll
  for (int j = 0; j < 2; ++j) o[j] = f32_to_bf16(v[2 * j]) | (f32_to_bf16(v[2 * j + 1]) << 16);
  *reinterpret_cast<u32x2*>(A.out + (int64_t)t * A.ldo + n) = o;
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
// Bound by the latency of one pass over the packed bytes: 4.6 us for 1 x 4096 x
// 4096 of 2 bits (5.3 MB, 1.1 TB/s; 4.0 back to back in a graph), 6.1 for
// 8 x 4096 x 2048 of 3 bits.
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
// Weight operand of one lane: 8 values of one column and 32-group GB as fp16,
// s * (u - offset) * fac, fac = 32 (16 for 3-bit levels: then the largest
// weight of a scale up to 2^10 is finite).  A mask-and-or puts the level into
// the mantissa of an fp16 base where its lowest bit is worth 1 (bit 2 under
// 256, bit 4 under 64, bit 6 under 16), one packed FMA gives (u - offset) * fac
// exactly, one packed multiply by the scale (half GB%2 of sp, for both halves
// by operand selection) rounds to fp16's 11 bits.  That rounding is exact for
// ternary weights and at most 2^-11 of a 2- or 3-bit weight otherwise: an
// error of about 1e-4 of the result's size, against 1.7e-3 of its rounding to
// bf16; keeping the scales out of the operand would cost a vector FMA per
// result and 32-group, as much time as the matrix cores'.
struct OperandK {
  uint32_t m2, m4, m6, b2, b4, b6, o2, o4, o6;
};
template <int Q>
constexpr float kFac = Q == MOE_Q_INT3 ? 16.f : 32.f;

template <int Q, int GB>
__device__ __forceinline__ u32x4 weights_f16(uint32_t w, uint32_t w1, f16x2 sp,
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
  const f16x2 s2 = __builtin_shufflevector(sp, sp, GB & 1, GB & 1);
  const f16x2 fac = {(_Float16)kFac<Q>, (_Float16)kFac<Q>};
  u32x4 r;
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    const f16x2 o = __builtin_bit_cast(f16x2, v < 2 ? k.o2 : v == 2 ? k.o4 : k.o6);
    r[v] = __builtin_bit_cast(uint32_t, (__builtin_bit_cast(f16x2, f[v]) * fac + o) * s2);
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

// 16, 8 or 4 bytes per lane at base + off + soff
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc_of(const void* base) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, -1, kRsrcLin);
}
__device__ __forceinline__ u32x4 load_b128(const void* base, int off, int soff) {
  return __builtin_bit_cast(u32x4,
                            __builtin_amdgcn_raw_buffer_load_b128(rsrc_of(base), off, soff, 0));
}
__device__ __forceinline__ u32x2 load_b64(const void* base, int off, int soff) {
  return __builtin_bit_cast(u32x2,
                            __builtin_amdgcn_raw_buffer_load_b64(rsrc_of(base), off, soff, 0));
}
__device__ __forceinline__ uint32_t load_b32(const void* base, int off, int soff) {
  return __builtin_amdgcn_raw_buffer_load_b32(rsrc_of(base), off, soff, 0);
}

// f(integral constants 0 .. N-1)
template <int... I, typename F>
__device__ __forceinline__ void for_ints_impl(std::integer_sequence<int, I...>, F f) {
  (f(std::integral_constant<int, I>{}), ...);
}
template <int N, typename F>
__device__ __forceinline__ void for_ints(F f) {
  for_ints_impl(std::make_integer_sequence<int, N>{}, f);
}

__device__ __forceinline__ uint32_t pk_max_u16(uint32_t a, uint32_t b) {
  typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a),
                                                                __builtin_bit_cast(u16x2, b)));
}

// Epilogue of the matrix-core kernels: register i of acc[rt][ct] is row
// rt*32 + 8(i/4) + 4(lane/32) + i%4 and column l32 of its 32 x 32 tile.  Bias
// and activation are applied there; then each wave turns 32 rows of its
// columns at a time in LDS of its own, so that a lane holds 8 consecutive
// columns and whole cache lines are read and written.  The factor (or, without
// one, the residual) of the next 32 rows is loaded meanwhile.  srow: the tile
// rows' powers of two in LDS; cscale: those of the lane's columns.
template <int CT>
constexpr int kTurnRow = 32 * CT + 8;  // floats; rows 4 apart are half the banks apart
template <int CT>
constexpr int kTurnBytes = 32 * kTurnRow<CT> * 4;

template <int NRT, int CT>
__device__ __forceinline__ void store_tile(const LinArgs& A, f32x16 (&acc)[NRT][CT], float unfac,
                                           const float* srow, const float (&cscale)[CT],
                                           uint8_t* area, int T, int row0, int col0) {
  constexpr int kLanes = 4 * CT, kRows = 64 / kLanes, P = 32 / kRows;  // lanes a row, passes
  const int lane = threadIdx.x & 63, l32 = lane & 31, hl = lane >> 5;
  float* const turn = reinterpret_cast<float*>(area);
  const int lr = lane / kLanes, n = col0 + 8 * (lane % kLanes);
  // rows and columns past the end repeat the last ones (read, not stored)
  const int nc = min(n, A.N - 8);
  const uint16_t* const first = A.mul ? A.mul : A.res;
  const int64_t ldf = A.mul ? A.ldm : A.ldr;
  u32x4 op[2][P], op2[P];
  auto fetch = [&](const uint16_t* base, int64_t ld, int rt, u32x4 (&o)[P])
      __attribute__((always_inline)) {
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int t = min(row0 + rt * 32 + p * kRows + lr, T - 1);
      o[p] = *reinterpret_cast<const u32x4*>(base + (int64_t)t * ld + nc);
    }
  };
  if (first) fetch(first, ldf, 0, op[0]);
  float cs[CT], bi[CT];
#pragma unroll
  for (int ct = 0; ct < CT; ++ct) {
    const int c = min(col0 + 32 * ct + l32, A.N - 1);
    cs[ct] = unfac * cscale[ct];
    bi[ct] = A.bias ? A.bias[c] : 0.f;
  }
#pragma unroll
  for (int rt = 0; rt < NRT; ++rt)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const f32x4 rs = *reinterpret_cast<const f32x4*>(srow + rt * 32 + 8 * j + 4 * hl);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int ct = 0; ct < CT; ++ct)
          acc[rt][ct][4 * j + i] = acc[rt][ct][4 * j + i] * cs[ct] * rs[i] + bi[ct];
    }
  for_act(A.act, [&](auto ac) __attribute__((always_inline)) {
#pragma unroll
    for (int rt = 0; rt < NRT; ++rt)
#pragma unroll
      for (int ct = 0; ct < CT; ++ct)
#pragma unroll
        for (int i = 0; i < 16; ++i)
          acc[rt][ct][i] = activate<decltype(ac)::value>(acc[rt][ct][i]);
  });
  // one straight copy for each of: neither, factor, residual, both
  auto rows = [&](auto has_mul, auto has_res) __attribute__((always_inline)) {
    constexpr bool M = decltype(has_mul)::value, S = decltype(has_res)::value;
#pragma unroll
    for (int rt = 0; rt < NRT; ++rt) {
      if (M && S) fetch(A.res, A.ldr, rt, op2);
      if ((M || S) && rt + 1 < NRT) fetch(first, ldf, rt + 1, op[(rt + 1) & 1]);
#pragma unroll
      for (int ct = 0; ct < CT; ++ct)
#pragma unroll
        for (int i = 0; i < 16; ++i)
          turn[(8 * (i >> 2) + 4 * hl + (i & 3)) * kTurnRow<CT> + 32 * ct + l32] = acc[rt][ct][i];
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const int m = p * kRows + lr, t = row0 + rt * 32 + m;
        const float* at = turn + m * kTurnRow<CT> + 8 * (lane % kLanes);
        const f32x4 v0 = *reinterpret_cast<const f32x4*>(at);
        const f32x4 v1 = *reinterpret_cast<const f32x4*>(at + 4);
        float v[8] = {v0[0], v0[1], v0[2], v0[3], v1[0], v1[1], v1[2], v1[3]};
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float f = bf16_to_f32((op[rt & 1][p][j >> 1] >> (16 * (j & 1))) & 0xFFFFu);
          if (M) v[j] *= f;
          if (!M && S) v[j] += f;
          if (M && S) v[j] += bf16_to_f32((op2[p][j >> 1] >> (16 * (j & 1))) & 0xFFFFu);
        }
        u32x4 o;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          o[j] = f32_to_bf16(v[2 * j]) | (f32_to_bf16(v[2 * j + 1]) << 16);
        if (t < T && n < A.N) *reinterpret_cast<u32x4*>(A.out + (int64_t)t * A.ldo + n) = o;
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
    }
  };
  if (!first)
    rows(std::false_type{}, std::false_type{});
  else if (!A.res)
    rows(std::true_type{}, std::false_type{});
  else if (!A.mul)
    rows(std::false_type{}, std::true_type{});
  else
    rows(std::true_type{}, std::true_type{});
}

// Block: a tile of 32 NRT rows and W waves of 32 CT columns each.  Per 128-wide
// k-step the block's rows go through registers into one of two LDS stages as
// fp16 (a step ahead), each wave's packed words and scales into registers one
// step ahead; the wave builds its weight operands in registers, each feeding
// NRT matrix-core ops.
//
// fp16 holds a bf16 value exactly down to 2^-17 and rounds smaller ones by at
// most 2^-24, and the operand keeps 11 bits of a weight of scale down to 2^-17.  So
// where each row's largest value is 0 or lies in [2^-6, 2^15] and each
// column's largest scale is 0 or in [2^-14, 2^10], plain conversion changes a
// value by at most 2^-18 of its row's largest, which does not show in a sum
// that this largest value takes part in, rounded to bf16 (2^-8), and hardly
// elsewhere.  The block learns both maxima on the way; if one is
// outside, it runs the product again with each row's values and each column's
// scales brought to the upper end of the range by powers of two (pass 2).
// (Giving every row its power of two beforehand took a launch of its own that
// read and wrote all rows: 46 us of 180 at 8192 x 4096 x 2048.)
//
// Measured: 8192 x 4096 x 2048 131 us (1.05 PFLOP/s), 16384 x 4096 x 4096 536
// (1.03); the matrix cores are busy in 64 and 60 % of the cycles, at the clock
// that the power limit leaves (about 1.6 GHz).  The rest is the build of the
// operands, 5 to 7 vector ops for each matrix-core op of 8 passes, and the
// epilogue, which nothing covers as one block fills a CU: 17 us for 256 blocks
// of 128 x 512.  Loading its factor's lines during the last two steps gained
// 1.5 % at the first size and nothing at the second.
template <int Q, int NRT, int W, int CT>
__global__ __launch_bounds__(64 * W, 1) void k_lin_gemm(LinArgs A, OperandK kk, int T,
                                                        int row_tiles, int ncol) {
  extern __shared__ __attribute__((aligned(16))) uint8_t sbuf[];
  // small tiles have registers to spare and short steps: their rows are loaded
  // two steps ahead of their conversion, their words a whole step
  constexpr int R = 32 * NRT, kStage = R * 256, kCh = R / (4 * W), kDeep = NRT * CT <= 2 ? 2 : 1;
  static_assert(R % (4 * W) == 0 && kCh <= 8, "row split");
  constexpr bool Q3 = Q == MOE_Q_INT3;
  __shared__ __attribute__((aligned(16))) float srow[R];
  __shared__ int s_redo;
  // work item = (row tile, column group), tile-major; each XCD takes one
  // contiguous chunk of the items (blocks go to the 8 XCDs round-robin)
  const int n_items = row_tiles * ncol, chunk = (n_items + 7) / 8;
  const int local = blockIdx.x / 8, item = (blockIdx.x % 8) * chunk + local;
  if (local >= chunk || item >= n_items) return;
  const int tile = item / ncol, col = item % ncol;
  const int tid = threadIdx.x, lane = tid & 63, l32 = lane & 31, hl = lane >> 5, r = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int K = A.K, S = K / 128, NT = A.N / 16;
  const int row0 = tile * R;
  if (tid == 0) s_redo = 0;

  // LDS: row i of a stage at i * 256, its 16-byte chunk c (8 k) in slot
  // c ^ (i % 16); 16 lanes convert one row.  Rows past T repeat the last one.
  const uint16_t* const xrow = A.x + (int64_t)row0 * A.ldx;
  uint32_t xo[kCh];
#pragma unroll
  for (int i = 0; i < kCh; ++i) {
    const int row = 4 * (kCh * wave + i) + (lane >> 4);
    xo[i] = (uint32_t)min(row, T - 1 - row0) * (uint32_t)(2 * A.ldx) + (lane & 15) * 16;
  }
  // (rows 4 i on: the swizzle's 4 i is XORed in where a chunk is stored)
  const uint32_t lo = (uint32_t)((4 * kCh * wave + (lane >> 4)) * 256) |
                      (((lane & 15) ^ (((4 * kCh * wave) & 15) + (lane >> 4))) << 4);
  const uint32_t la = (uint32_t)(l32 * 256) | ((uint32_t)(hl ^ (l32 & 15)) << 4);

  OperandK k = kk;
  k.b2 = lane_copy(kk.b2);
  k.b4 = lane_copy(kk.b4);
  k.b6 = lane_copy(kk.b6);

  // packed weights: column tile ct of the wave is n-tiles 2c, 2c + 1 of
  // c = (col W + wave) CT + ct; tiles past N repeat the last one (not stored)
  uint32_t wo[CT], po[CT], so[CT];
#pragma unroll
  for (int ct = 0; ct < CT; ++ct) {
    const int c32 = (col * W + wave) * CT + ct;
    const uint32_t nt = (uint32_t)min(2 * c32 + (l32 >> 4), NT - 1);
    wo[ct] = nt * S * 512 + (16 * hl + r) * 8;
    po[ct] = (uint32_t)A.plane1 + nt * S * 256 + (16 * hl + r) * 4;
    so[ct] = (uint32_t)A.scales + nt * S * 128 + r * 8;
  }

  struct Words {
    u32x2 w[CT][2], s[CT];
    uint32_t w1[CT][2];
  };
  u32x4 xv[kDeep][kCh];        // bf16 rows of the steps after this one
  float rmax[kCh], rfac[kCh];  // the rows' largest |x| so far, 2^-e of pass 2
  uint32_t cmax[CT], cm[CT];   // the column's largest |scale| (two halves), 2^f twice
  f32x16 acc[NRT][CT];
  auto loadx = [&](int s, int i, u32x4 (&x)[kCh]) __attribute__((always_inline)) {
    x[i] = load_b128(xrow, (int)xo[i], min(s, S - 1) * 256);
  };
  auto loadb = [&](int s, Words& b) __attribute__((always_inline)) {
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        b.w[ct][h] = load_b64(A.w, (int)wo[ct], s * 512 + 256 * h);
        if (Q3) b.w1[ct][h] = load_b32(A.w, (int)po[ct], s * 256 + 128 * h);
      }
      b.s[ct] = load_b64(A.w, (int)so[ct], s * 128);
    }
  };
  auto loada = [&](uint32_t at, int q, u32x4 (&a)[NRT]) __attribute__((always_inline)) {
    const uint8_t* p = sbuf + (at ^ (uint32_t)((2 * q) << 4));
#pragma unroll
    for (int rt = 0; rt < NRT; ++rt) a[rt] = *reinterpret_cast<const u32x4*>(p + rt * 8192);
  };

  // One product over K; SCALED: pass 2.
  auto product = [&](auto scaled) __attribute__((always_inline)) {
    constexpr bool SC = decltype(scaled)::value;
#pragma unroll
    for (int rt = 0; rt < NRT; ++rt)
#pragma unroll
      for (int ct = 0; ct < CT; ++ct)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[rt][ct][i] = 0.f;
    auto build = [&](auto qc, const Words& b, u32x4 (&o)[CT]) __attribute__((always_inline)) {
      constexpr int GB = decltype(qc)::value >> 1, h = decltype(qc)::value & 1;
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) {
        const uint32_t sw = b.s[ct][GB >> 1];  // (a bit cast of the element itself takes element 0)
        f16x2 sp = __builtin_bit_cast(f16x2, sw);
        if (SC) sp = sp * __builtin_bit_cast(f16x2, cm[ct]);
        o[ct] = weights_f16<Q, GB>(b.w[ct][h][GB >> 1], Q3 ? b.w1[ct][h] : 0u, sp, k);
      }
    };
    // chunk i of x as fp16 into LDS stage st
    auto convert = [&](int i, int st, const u32x4 (&x)[kCh]) __attribute__((always_inline)) {
      u32x4 o;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float a = __uint_as_float(x[i][j] << 16), b = __uint_as_float(x[i][j] & 0xFFFF0000u);
        if (SC) {
          a *= rfac[i];
          b *= rfac[i];
        } else {
          // (the library function would first canonicalise each operand)
          __asm__("v_max3_f32 %0, %0, |%1|, |%2|" : "+v"(rmax[i]) : "v"(a), "v"(b));
        }
        o[j] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_pkrtz(a, b));
      }
      *reinterpret_cast<u32x4*>(sbuf + st * kStage + i * 1024 + (lo ^ ((i & 3) << 6))) = o;
    };
    // sub-step q of a step (group q/2, k-half q%2): the next sub-step's rows
    // are read, its weights built and a part of the next step's rows
    // converted while this one's matrix-core ops run
    auto sub = [&](auto qc, int s, uint32_t at, const Words& b, const Words& bn, u32x4 (&x)[kCh],
                   u32x4 (&a0)[NRT], u32x4 (&a1)[NRT], u32x4 (&o0)[CT], u32x4 (&o1)[CT])
        __attribute__((always_inline)) {
      constexpr int q = decltype(qc)::value;
      if constexpr (q < 7) loada(at, q + 1, a1);
      if constexpr (q < 7)
        build(std::integral_constant<int, q + 1>{}, b, o1);
      else
        build(std::integral_constant<int, 0>{}, bn, o1);
      if constexpr (q < kCh) convert(q, (s + 1) & 1, x);
#pragma unroll
      for (int rt = 0; rt < NRT; ++rt)
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) acc[rt][ct] = mfma_lin(a0[rt], o0[ct], acc[rt][ct]);
#pragma unroll
      for (int i = 0; i < NRT * CT; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x002, Q3 ? 8 : 6, 0);
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      }
      __builtin_amdgcn_sched_barrier(0);
      if constexpr (q < kCh) loadx(s + 1 + kDeep, q, x);
      __builtin_amdgcn_sched_barrier(0);
    };
    Words wa, wb;
    u32x4 a0[NRT], a1[NRT], o0[CT], o1[CT];
    // step s converts x of step s + 1, from xv[s % kDeep]
#pragma unroll
    for (int i = 0; i < kCh; ++i) loadx(0, i, xv[kDeep - 1]);
    loadb(0, wa);
    if (kDeep == 2) {
      loadb(min(1, S - 1), wb);
#pragma unroll
      for (int i = 0; i < kCh; ++i) loadx(1, i, xv[0]);
    }
#pragma unroll
    for (int i = 0; i < kCh; ++i) convert(i, 0, xv[kDeep - 1]);
#pragma unroll
    for (int i = 0; i < kCh; ++i) loadx(kDeep, i, xv[kDeep - 1]);
    build(std::integral_constant<int, 0>{}, wa, o0);
    auto step = [&](int s, Words& b, Words& bn, u32x4 (&x)[kCh]) __attribute__((always_inline)) {
      // step s's rows are in LDS for every wave, and every wave is done with
      // the stage that step s + 1's overwrite
      __builtin_amdgcn_s_waitcnt(wait_vm_lgkm(63, 0));
      __builtin_amdgcn_s_barrier();
      const uint32_t at = la + (uint32_t)((s & 1) * kStage);
      loada(at, 0, a0);
      __builtin_amdgcn_sched_barrier(0);
      if (!SC) {
#pragma unroll
        for (int ct = 0; ct < CT; ++ct)
#pragma unroll
          for (int i = 0; i < 2; ++i) cmax[ct] = pk_max_u16(cmax[ct], b.s[ct][i] & 0x7FFF7FFFu);
      }
      __builtin_amdgcn_sched_barrier(0);
      sub(std::integral_constant<int, 0>{}, s, at, b, bn, x, a0, a1, o0, o1);
      sub(std::integral_constant<int, 1>{}, s, at, b, bn, x, a1, a0, o1, o0);
      sub(std::integral_constant<int, 2>{}, s, at, b, bn, x, a0, a1, o0, o1);
      // the next step's words, where half of this one's are done with (past
      // the last step they repeat it, so that there is no branch)
      if (kDeep == 1) loadb(min(s + 1, S - 1), bn);
      __builtin_amdgcn_sched_barrier(0);
      sub(std::integral_constant<int, 3>{}, s, at, b, bn, x, a1, a0, o1, o0);
      sub(std::integral_constant<int, 4>{}, s, at, b, bn, x, a0, a1, o0, o1);
      sub(std::integral_constant<int, 5>{}, s, at, b, bn, x, a1, a0, o1, o0);
      sub(std::integral_constant<int, 6>{}, s, at, b, bn, x, a0, a1, o0, o1);
      sub(std::integral_constant<int, 7>{}, s, at, b, bn, x, a1, a0, o1, o0);
      if (kDeep == 2) loadb(min(s + 2, S - 1), b);
      __builtin_amdgcn_sched_barrier(0);
    };
    int s = 0;
    for (; s + 1 < S; s += 2) {
      step(s, wa, wb, xv[0]);
      step(s + 1, wb, wa, xv[kDeep - 1]);
    }
    if (s < S) step(s, wa, wb, xv[0]);
    __syncthreads();  // the stages are free
  };

#pragma unroll
  for (int i = 0; i < kCh; ++i) rmax[i] = 0.f;
#pragma unroll
  for (int ct = 0; ct < CT; ++ct) cmax[ct] = 0u;
  product(std::false_type{});

  // the maxima: rows over their 16 lanes, columns over the two halves
  float cscale[CT];
  bool redo = false;
#pragma unroll
  for (int i = 0; i < kCh; ++i) {
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) rmax[i] = fmaxf(rmax[i], __shfl_xor(rmax[i], o, 64));
    redo |= rmax[i] != 0.f && !(rmax[i] >= 0x1p-6f && rmax[i] <= 0x1p15f);
    if ((lane & 15) == 0) srow[4 * (kCh * wave + i) + (lane >> 4)] = 1.f;
  }
#pragma unroll
  for (int ct = 0; ct < CT; ++ct) {
    cmax[ct] = max(cmax[ct] & 0xFFFFu, cmax[ct] >> 16);
    redo |= cmax[ct] != 0u && !(cmax[ct] >= 0x0400u && cmax[ct] <= 0x6400u);
    cscale[ct] = 1.f;
  }
  if (redo) s_redo = 1;
  __syncthreads();
  if (s_redo) {
#pragma unroll
    for (int i = 0; i < kCh; ++i) {
      // 2^e brings the largest value to [2^14, 2^15); an infinite one counts as 2^114
      const int e = min(114, max(-100, (int)(__float_as_uint(rmax[i]) >> 23) - 127 - 14));
      rfac[i] = __uint_as_float((uint32_t)(127 - e) << 23);
      if ((lane & 15) == 0)
        srow[4 * (kCh * wave + i) + (lane >> 4)] = __uint_as_float((uint32_t)(127 + e) << 23);
    }
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
      // 2^f brings the largest scale to [2^7, 2^8) (f at most 15: a subnormal
      // one to 2^-9 at least); an infinite or zero one leaves the column as it is
      const int f = cmax[ct] == 0u || cmax[ct] >= 0x7C00u
                        ? 0
                        : min(15, 7 - ((int)(cmax[ct] >> 10) - 15));
      cm[ct] = (uint32_t)(f + 15) << 10;
      cm[ct] |= cm[ct] << 16;
      cscale[ct] = __uint_as_float((uint32_t)(127 - f) << 23);
    }
    product(std::true_type{});
  }
  store_tile<NRT, CT>(A, acc, 1.f / kFac<Q>, srow, cscale, sbuf + wave * kTurnBytes<CT>, T, row0,
                      (col * W + wave) * CT * 32);
}

// --------------------------------------------------------------- some rows
// Block: 32 NRT rows x 128 columns (4 waves of 32) and a run of k-chunks of
// four k-blocks.  A chunk is loaded as a whole (every load of it in flight at
// once, the next chunk's while this one is multiplied), so its rows' and
// columns' largest values are known before anything is converted: each gets
// its power of two, and the chunk's product is brought back to scale as it is
// added to the block's sum.  77 x 4096 x 2064: 9.3 us and 2.6 for the join.
// part: where K is split, the partial sums [split][T][N].
constexpr int kSomeKb = 4;
template <int Q, int NRT>
__global__ __launch_bounds__(256, 2) void k_lin_some(LinArgs A, OperandK kk, int T, int row_tiles,
                                                     int ncol, int run, float* __restrict__ part) {
  extern __shared__ __attribute__((aligned(16))) uint8_t sbuf[];  // kSomeKb stages
  constexpr int R = 32 * NRT, kStage = R * 256, kCh = R / 16;
  constexpr bool Q3 = Q == MOE_Q_INT3;
  __shared__ __attribute__((aligned(16))) float srow[R];
  const int tiles = row_tiles * ncol, split = blockIdx.x / tiles, item = blockIdx.x % tiles;
  const int tile = item / ncol, col = item % ncol;
  const int tid = threadIdx.x, lane = tid & 63, l32 = lane & 31, hl = lane >> 5, r = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int K = A.K, S = K / 128, NT = A.N / 16;
  const int row0 = tile * R, n0 = col * 128 + 32 * wave;
  const int c0 = split * run, c1 = min((S + kSomeKb - 1) / kSomeKb, c0 + run);
  const uint16_t* const xrow = A.x + (int64_t)row0 * A.ldx;
  uint32_t xo[kCh];
#pragma unroll
  for (int i = 0; i < kCh; ++i)
    xo[i] = (uint32_t)min(4 * (kCh * wave + i) + (lane >> 4), T - 1 - row0) *
                (uint32_t)(2 * A.ldx) + (lane & 15) * 16;
  const uint32_t la = (uint32_t)(l32 * 256) | ((uint32_t)(hl ^ (l32 & 15)) << 4);
  OperandK k = kk;
  k.b2 = lane_copy(kk.b2);
  k.b4 = lane_copy(kk.b4);
  k.b6 = lane_copy(kk.b6);
  const uint32_t nt = (uint32_t)min((n0 >> 4) + (l32 >> 4), NT - 1);
  const uint32_t wo = nt * S * 512 + (16 * hl + r) * 8;
  const uint32_t po = (uint32_t)A.plane1 + nt * S * 256 + (16 * hl + r) * 4;
  const uint32_t so = (uint32_t)A.scales + nt * S * 128 + r * 8;

  u32x4 xv[kSomeKb][kCh];
  u32x2 w[kSomeKb][2], sc[kSomeKb];
  uint32_t w1[kSomeKb][2];
  // (k-blocks past the end repeat the last one's loads and count as zero rows)
  auto load = [&](int c) __attribute__((always_inline)) {
#pragma unroll
    for (int u = 0; u < kSomeKb; ++u) {
      const int kb = min(c * kSomeKb + u, S - 1);
#pragma unroll
      for (int i = 0; i < kCh; ++i) xv[u][i] = load_b128(xrow, (int)xo[i], kb * 256);
    }
  };
  auto loadw = [&](int c) __attribute__((always_inline)) {
#pragma unroll
    for (int u = 0; u < kSomeKb; ++u) {
      const int kb = min(c * kSomeKb + u, S - 1);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        w[u][h] = load_b64(A.w, (int)wo, kb * 512 + 256 * h);
        if (Q3) w1[u][h] = load_b32(A.w, (int)po, kb * 256 + 128 * h);
      }
      sc[u] = load_b64(A.w, (int)so, kb * 128);
    }
  };
  f32x16 sum[NRT][1], acc[NRT];
#pragma unroll
  for (int rt = 0; rt < NRT; ++rt)
#pragma unroll
    for (int i = 0; i < 16; ++i) sum[rt][0][i] = 0.f;
  loadw(c0);
  load(c0);
  for (int c = c0; c < c1; ++c) {
    // rows: 2^e brings the largest value to [2^14, 2^15) (16 lanes hold a row)
    float fac[kCh];
    __syncthreads();  // the last chunk's rows are read
#pragma unroll
    for (int i = 0; i < kCh; ++i) {
      uint32_t m = 0;
#pragma unroll
      for (int u = 1; u < kSomeKb; ++u)
        if (c * kSomeKb + u >= S) xv[u][i] = u32x4{0u, 0u, 0u, 0u};
#pragma unroll
      for (int u = 0; u < kSomeKb; ++u)
#pragma unroll
        for (int j = 0; j < 4; ++j) m = pk_max_u16(m, xv[u][i][j] & 0x7FFF7FFFu);
      m = max(m & 0xFFFFu, m >> 16);
      m = max(m, dpp_u32<0xB1>(m));
      m = max(m, dpp_u32<0x4E>(m));
      m = max(m, dpp_u32<0x141>(m));
      m = max(m, dpp_u32<0x140>(m));
      const int e = min(114, max(-100, (int)(m >> 7) - 127 - 14));
      fac[i] = __uint_as_float((uint32_t)(127 - e) << 23);
      const int row = 4 * (kCh * wave + i) + (lane >> 4);
      if ((lane & 15) == 0) srow[row] = __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
      for (int u = 0; u < kSomeKb; ++u) {
        u32x4 o;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          o[j] = __builtin_bit_cast(
              uint32_t, __builtin_amdgcn_cvt_pkrtz(__uint_as_float(xv[u][i][j] << 16) * fac[i],
                                                   __uint_as_float(xv[u][i][j] & 0xFFFF0000u) *
                                                       fac[i]));
        *reinterpret_cast<u32x4*>(sbuf + u * kStage + row * 256 +
                                  (((lane & 15) ^ (row & 15)) << 4)) = o;
      }
    }
    // the column: 2^f brings the largest scale to [2^7, 2^8), f at most 15
    uint32_t cm = 0;
#pragma unroll
    for (int u = 0; u < kSomeKb; ++u)
#pragma unroll
      for (int i = 0; i < 2; ++i) cm = pk_max_u16(cm, sc[u][i] & 0x7FFF7FFFu);
    cm = max(cm & 0xFFFFu, cm >> 16);
    const int f = cm == 0u || cm >= 0x7C00u ? 0 : min(15, 7 - ((int)(cm >> 10) - 15));
    const uint32_t fh = (uint32_t)(f + 15) << 10, f2 = fh | (fh << 16);
    const float cs = __uint_as_float((uint32_t)(127 - f) << 23) / kFac<Q>;
    __syncthreads();
    if (c + 1 < c1) load(c + 1);
#pragma unroll
    for (int rt = 0; rt < NRT; ++rt)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[rt][i] = 0.f;
    // 32 sub-steps of 16 k: the next one's rows are read and its weights built
    // while this one's matrix-core ops run
    auto rows = [&](auto qc, u32x4 (&a)[NRT]) __attribute__((always_inline)) {
      constexpr int u = decltype(qc)::value >> 3, q = decltype(qc)::value & 7;
      const uint8_t* p = sbuf + u * kStage + (la ^ (uint32_t)((2 * q) << 4));
#pragma unroll
      for (int rt = 0; rt < NRT; ++rt) a[rt] = *reinterpret_cast<const u32x4*>(p + rt * 8192);
    };
    auto build = [&](auto qc) __attribute__((always_inline)) {
      constexpr int u = decltype(qc)::value >> 3, q = decltype(qc)::value & 7;
      constexpr int GB = q >> 1, h = q & 1;
      const uint32_t sw = sc[u][GB >> 1];
      const f16x2 sp = __builtin_bit_cast(f16x2, sw) * __builtin_bit_cast(f16x2, f2);
      return weights_f16<Q, GB>(w[u][h][GB >> 1], Q3 ? w1[u][h] : 0u, sp, k);
    };
    u32x4 a[2][NRT], o[2];
    rows(std::integral_constant<int, 0>{}, a[0]);
    o[0] = build(std::integral_constant<int, 0>{});
    __builtin_amdgcn_sched_barrier(0);
    for_ints<8 * kSomeKb>([&](auto qc) __attribute__((always_inline)) {
      constexpr int q = decltype(qc)::value;
      if constexpr (q + 1 < 8 * kSomeKb) {
        rows(std::integral_constant<int, q + 1>{}, a[(q + 1) & 1]);
        o[(q + 1) & 1] = build(std::integral_constant<int, q + 1>{});
      }
#pragma unroll
      for (int rt = 0; rt < NRT; ++rt) acc[rt] = mfma_lin(a[q & 1][rt], o[q & 1], acc[rt]);
#pragma unroll
      for (int i = 0; i < NRT; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x002, 24 / NRT, 0);
      }
      __builtin_amdgcn_sched_barrier(0);
    });
    if (c + 1 < c1) loadw(c + 1);
#pragma unroll
    for (int rt = 0; rt < NRT; ++rt)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const f32x4 rs = *reinterpret_cast<const f32x4*>(srow + rt * 32 + 8 * j + 4 * hl);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          sum[rt][0][4 * j + i] = fmaf(acc[rt][4 * j + i] * cs, rs[i], sum[rt][0][4 * j + i]);
      }
  }
  if (part) {
    const int n = n0 + l32;
    float* o = part + ((size_t)split * T + row0) * A.N + n;
#pragma unroll
    for (int rt = 0; rt < NRT; ++rt)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int m = rt * 32 + 8 * (i >> 2) + 4 * hl + (i & 3);
        if (row0 + m < T && n < A.N) o[(size_t)m * A.N] = sum[rt][0][i];
      }
    return;
  }
  __syncthreads();
  if (tid < R) srow[tid] = 1.f;
  __syncthreads();
  const float one[1] = {1.f};
  store_tile<NRT, 1>(A, sum, 1.f, srow, one, sbuf + wave * kTurnBytes<1>, T, row0, n0);
}

// Joins the partial sums, in the order of the splits, and finishes: one
// thread per four columns, eight splits' loads in flight at once.
__global__ __launch_bounds__(256) void k_lin_join(LinArgs A, int T, int splits,
                                                  const float* __restrict__ part) {
  const int per_row = A.N / 4;
  const long i = (long)blockIdx.x * 256 + threadIdx.x;
  if (i >= (long)T * per_row) return;
  const int t = (int)(i / per_row), n = (int)(i % per_row) * 4;
  const float* p = part + (size_t)t * A.N + n;
  const size_t step = (size_t)T * A.N;
  f32x4 sum = {0.f, 0.f, 0.f, 0.f};
  for (int s0 = 0; s0 < splits; s0 += 8) {
    f32x4 v[8];
#pragma unroll
    for (int s = 0; s < 8; ++s)  // (past the last split: it again, not added)
      v[s] = *reinterpret_cast<const f32x4*>(p + min(s0 + s, splits - 1) * step);
#pragma unroll
    for (int s = 0; s < 8; ++s)
      if (s0 + s < splits) sum += v[s];
  }
  finish4(A, sum, t, n);
}

// ------------------------------------------------------------------ launch
// Which kernel takes a call: the one whose time, in us, is the least by these
// estimates, fitted to sweeps of T = 1 .. 3000 at (K, N) from (512, 8192) to
// (8192, 1024), S = K / 128 steps and b blocks of each kernel:
//   few     2.5 + S * 0.24 (T <= 32) or 0.54, more where b exceeds the CUs
//           (4096 x 4096: 10.3 us at T = 32, 21.5 at 64)
//   some    3.8 + run * b * 0.0095 (32 rows a tile) or 0.022 (64), and the
//           second launch (4096 x 2064, T = 77: 13.5 us; the smallest tiles of
//           the next kernel unsplit 24.6)
//   tiles   3 + S steps and an epilogue.  A step takes a latency-bound time
//           while the CUs have a block or less and grows with the blocks
//           beyond it; of the 128-row tiles a CU takes one block at a time, so
//           that nothing covers their epilogues.  Measured, by tile, at
//             1000 x 4096 x 4096   42.5 us (64 x 256), 48 (64 x 128, 128 x 256), 83 (128 x 512)
//             2048 x 4096 x 1024   34.0 (64 x 128), 37.7 (64 x 256), 49.5, 83
//             2048 x 4096 x 4096   74.9 (128 x 256), 83 (64 x 256), 97, 98
//             4096 x 4096 x 4096   136 (128 x 512), 148 (128 x 256), 161, 183
//             16384 x 512 x 1024   31.1 (128 x 256), 31.9 (64 x 256), 38, 40
// Up to 16 rows are always few (their exact weights).
struct LinTile {
  int nrt, waves, ct;        // rows / 32, waves, columns of a wave / 32
  float floor, base, slope;  // us a step: max(floor, base + slope * b / 256)
  float end;                 // us of epilogue for 256 blocks
};
constexpr LinTile kLinTiles[] = {{1, 4, 1, 0.62f, 0.27f, 0.43f, 0.9f},
                                 {2, 4, 1, 0.77f, 0.27f, 0.62f, 1.8f},
                                 {2, 8, 1, 1.00f, 0.05f, 1.13f, 2.6f},
                                 {4, 8, 1, 1.32f, 0.55f, 1.55f, 5.2f},
                                 {4, 8, 2, 2.40f, 2.00f, 1.55f, 17.0f}};
struct LinPlan {
  int kind;  // -2 few, -1 some, else the tile's place in kLinTiles
  int rows, tiles, ncol, run, splits;  // some
};
static LinPlan lin_plan(int K, int N, int T) {
  LinPlan best{};
  best.kind = -2;
  if (T <= 16) return best;
  const int S = K / 128;
  float cost = 1e30f;
  if (T <= kLinFewRows) {
    const float over = N > 4096 ? (float)N / 4096.f : 1.f;
    cost = 2.5f + S * (T <= 32 ? 0.24f : 0.54f) * over;
  }
  {
    LinPlan p{};
    p.kind = -1;
    p.ncol = (N + 127) / 128;
    const int chunks = (S + kSomeKb - 1) / kSomeKb;
    // 32-row tiles, three blocks to a CU, where they fit; else 64-row ones, two
    p.rows = (long)((T + 31) / 32) * p.ncol * chunks <= 768 ? 32 : 64;
    p.tiles = (T + p.rows - 1) / p.rows;
    const long want = (p.rows == 32 ? 768 : 512) / ((long)p.tiles * p.ncol);
    p.splits = want < 1 ? 1 : want < chunks ? (int)want : chunks;
    p.run = (chunks + p.splits - 1) / p.splits;
    p.splits = (chunks + p.run - 1) / p.run;
    const float b = (float)p.tiles * p.ncol * p.splits;
    float c = 3.8f + p.run * b * (p.rows == 32 ? 0.0095f : 0.022f) + 1.5f * (p.run - 1);
    if (p.splits > 1) c += 2.5f + (float)p.splits * T * N * 1.0e-6f;
    if (c < cost && (long)p.tiles * p.ncol * p.splits <= 1 << 20) {
      cost = c;
      best = p;
    }
  }
  for (int i = 0; i < 5; ++i) {
    const LinTile& v = kLinTiles[i];
    const long b = (long)((T + 32 * v.nrt - 1) / (32 * v.nrt)) *
                   ((N + 32 * v.ct * v.waves - 1) / (32 * v.ct * v.waves));
    // the fullest CU sets the time; of the 128-row tiles it takes one block at a time
    const float f = b <= 256 ? (float)b / 256.f : (float)((b + 255) / 256);
    float step = v.nrt == 4 && f > 1.f ? (v.base + v.slope) * f : v.base + v.slope * f;
    step = step < v.floor ? v.floor : step;
    const float c = 3.f + v.end * f + S * step;
    if (c < cost) {
      cost = c;
      best.kind = i;
    }
  }
  return best;
}

// What a call for T rows needs, and what any call for up to T rows may (a
// split needs at most 512 64-row or 768 32-row tiles of 128 columns).
size_t lin_ws_need(int K, int N, int T) {
  const LinPlan p = lin_plan(K, N, T);
  return p.kind == -1 && p.splits > 1 ? (size_t)p.splits * T * N * 4 : 0;
}
size_t lin_ws_bytes(int K, int N, int T) {
  if (T <= 16) return 256;
  const size_t most = (size_t)512 * 64 * 128 * 4;
  const size_t all = (size_t)((K / 128 + kSomeKb - 1) / kSomeKb) * T * N * 4;
  return ((all < most ? all : most) + 255) & ~size_t(255);
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
static int gemm(const LinArgs& A, const OperandK& k, int T, hipStream_t s) {
  const int tiles = (T + 32 * NRT - 1) / (32 * NRT), ncol = (A.N + 32 * CT * W - 1) / (32 * CT * W);
  constexpr size_t stages = 2 * 32 * NRT * 256, turn = W * kTurnBytes<CT>;
  constexpr size_t lds = stages > turn ? stages : turn;
  if (lds > 64000 &&
      hipFuncSetAttribute((const void*)k_lin_gemm<Q, NRT, W, CT>,
                          hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds) != hipSuccess)
    return (int)hipErrorInvalidConfiguration;
  const int items = tiles * ncol;
  hipLaunchKernelGGL((k_lin_gemm<Q, NRT, W, CT>), dim3((items + 7) / 8 * 8), dim3(64 * W), lds, s,
                     A, k, T, tiles, ncol);
  return (int)hipGetLastError();
}

template <int Q>
static int many(const LinArgs& A, const LinPlan& p, int T, uint8_t* ws, hipStream_t s) {
  // -(base + offset) * fac for the bases 256, 64, 16
  OperandK k = {0x000C000Cu, 0x00300030u, 0x00C000C0u, 0x5C005C00u, 0x54005400u, 0x4C004C00u,
                0, 0, 0};
  const auto pair = [](float v) {
    const _Float16 h = (_Float16)v;
    uint16_t u;
    __builtin_memcpy(&u, &h, 2);
    return (uint32_t)u | ((uint32_t)u << 16);
  };
  const float off = qtype_offset(Q), fac = kFac<Q>;
  k.o2 = pair(-(256.f + off) * fac);
  k.o4 = pair(-(64.f + off) * fac);
  k.o6 = pair(-(16.f + off) * fac);
  switch (p.kind) {
    case 0: return gemm<Q, 1, 4, 1>(A, k, T, s);
    case 1: return gemm<Q, 2, 4, 1>(A, k, T, s);
    case 2: return gemm<Q, 2, 8, 1>(A, k, T, s);
    case 3: return gemm<Q, 4, 8, 1>(A, k, T, s);
    case 4: return gemm<Q, 4, 8, 2>(A, k, T, s);
  }
  float* part = p.splits > 1 ? (float*)ws : nullptr;
  const dim3 g((unsigned)(p.tiles * p.ncol * p.splits));
  constexpr int stages = kSomeKb * 256, turn = 4 * kTurnBytes<1>;
  if (p.rows == 32)
    hipLaunchKernelGGL((k_lin_some<Q, 1>), g, dim3(256), 32 * stages, s, A, k, T, p.tiles, p.ncol,
                       p.run, part);
  else
    hipLaunchKernelGGL((k_lin_some<Q, 2>), g, dim3(256), 64 * stages, s, A, k, T, p.tiles, p.ncol,
                       p.run, part);
  static_assert(turn <= 32 * stages, "turning area");
  if (part)
    hipLaunchKernelGGL(k_lin_join, dim3((unsigned)(((long)T * (A.N / 4) + 255) / 256)), dim3(256),
                       0, s, A, T, p.splits, part);
  return (int)hipGetLastError();
}

int launch_linear(const LinArgs& A, int T, uint8_t* ws, void* stream) {
  hipStream_t s = (hipStream_t)stream;
  const LinPlan p = lin_plan(A.K, A.N, T);
  if (p.kind == -2) {
    if (A.q == MOE_Q_INT3)
      few<true>(A, T, s);
    else
      few<false>(A, T, s);
    return (int)hipGetLastError();
  }
  if (A.q == MOE_Q_TERNARY) return many<MOE_Q_TERNARY>(A, p, T, ws, s);
  if (A.q == MOE_Q_INT2) return many<MOE_Q_INT2>(A, p, T, ws, s);
  return many<MOE_Q_INT3>(A, p, T, ws, s);
}

}  // namespace bqmoe
