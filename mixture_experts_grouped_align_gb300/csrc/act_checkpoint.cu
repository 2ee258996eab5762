// The expert activation with an MXFP8 checkpoint, and its backward pass from the checkpoint.
//
// Forward, per row of pre-activations z (SwiGLU: gate | up, 2I values; relu^2: I values) with
// an optional row weight w:
//   h = w * silu(g) * u   or   h = w * max(z, 0)^2           (fp32, rounded once to bf16)
//   checkpoint = MXFP8(z): E4M3 codes and one E8M0 scale per 32 values (mx_quant.cuh)
// Backward, with z~ the checkpoint's values, s = sigmoid(g~) and a the activation of z~:
//   d g = w dh u~ s (1 + g~ (1 - s)),  d u = w dh g~ s   or   d z = 2 w dh max(z~, 0)
//   d w = sum_i dh_i a_i,  h~ = w a (the operand of the weight gradient, recomputed)
// The checkpoint keeps 33/64 of the bytes of bf16 pre-activations between the passes.
//
// Both are streams: the forward reads 2 N1 and writes 2 I + 33/32 N1 bytes per row, the
// backward reads 33/32 N1 + 2 I and writes 2 N1 + 2 I (N1 = 2I or I), and nothing is read
// twice.  A thread owns eight consecutive columns (16 bytes of bf16, 8 of codes), so the four
// lanes of a quad own one 32-value block of each half: its maximum takes two shuffles.  A
// row's columns belong to one warp (LANES < 32 lanes of it for narrow rows), or with few values
// to one block, and d w is a shuffle reduction over them in a fixed order.
//
// Measured: 65536 x 2048 SwiGLU 161 us forward and 197 us backward (6.7 and 6.9 TB/s, HBM's copy
// rate); 12345 x 1856 relu^2 19.8 and 26.1 us (5.8 and 6.2 TB/s, a launch's start and end being a
// tenth of it); 100000 x 352 SwiGLU 49.6 and 57 us (5.7 and 6.2 TB/s); 168 x 928 SwiGLU 1.8 us each, a
// launch.
#include <cuda_fp8.h>

#include "moe_common.cuh"
#include "moe_launch.h"
#include "mx_quant.cuh"

namespace {

using moe_launch::ActBackward;
using moe_launch::ActCheckpoint;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr unsigned kAll = 0xffffffffu;

MOE_DEV void unpack8(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
MOE_DEV uint4 pack8(const float (&f)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// MXFP8 of a 32-value block held eight values (bf16 pairs `raw`, fp32 `v`) a lane by four
// neighbouring lanes, all of which call: this lane's codes, and the block's scale byte.  The rule
// of mxq::quant32; the largest magnitude is found on the bf16 pairs, where NaN is the largest.
MOE_DEV uint2 quant8(const uint4& raw, const float (&v)[8], uint32_t& scale) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
  uint32_t m = 0;  // magnitudes are ordered like their bits
#pragma unroll
  for (int i = 0; i < 4; ++i) m = __vmaxu2(m, w[i] & 0x7fff7fffu);
  uint32_t b = max(m << 16, m & 0xffff0000u);
  b = max(b, __shfl_xor_sync(kAll, b, 1));
  b = max(b, __shfl_xor_sync(kAll, b, 2));
  if (b > 0x7f800000u) {
    scale = 255u;
    return make_uint2(0x7f7f7f7fu, 0x7f7f7f7fu);
  }
  const int e = mxq::block_exponent(__uint_as_float(b));
  scale = (uint32_t)(e + 127);
  const float inv = e >= 127 ? __uint_as_float(0x00400000u) : __uint_as_float((uint32_t)(127 - e) << 23);
  uint32_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    h[i] = __nv_cvt_float2_to_fp8x2(make_float2(v[2 * i] * inv, v[2 * i + 1] * inv), __NV_SATFINITE, __NV_E4M3);
  return make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
}

// Eight E4M3 codes under one E8M0 scale -> their values (exact).
MOE_DEV void dequant8(uint2 c, uint32_t scale, float (&v)[8]) {
  const float s = moe::e8m0_to_f32(scale);
  uint32_t h[4];
  moe::e4m3x4_to_f16x2(c.x, h[0], h[1]);
  moe::e4m3x4_to_f16x2(c.y, h[2], h[3]);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
    v[2 * i] = f.x * s;
    v[2 * i + 1] = f.y * s;
  }
}

// 1 / (1 + 2^(-g log2 e)) with the hardware's exponential and reciprocal (2 ulp and 1 ulp).
MOE_DEV float sigmoid(float g) {
  float e, s;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(g * -1.44269504f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(1.f + e));
  return s;
}

// The rows of a block: WIDE = the whole block on one row, otherwise 32 / LANES rows a warp.
// A row's lanes take kTurns turns of 8 LANES columns at a time, all loads first: that many bytes in
// flight are what the stream needs, and the turns' scale bytes lie together, moved by one byte per
// lane.
template <int LANES, bool WIDE, int TURNS>
struct Map {
  static constexpr int kRowsPerBlock = WIDE ? 1 : kWarps * (32 / LANES);
  static constexpr int kStep = WIDE ? kThreads : LANES;  // columns of eight per turn
  static constexpr int kTurns = TURNS;
  MOE_DEV static int64_t row() {
    if (WIDE) return blockIdx.x;
    return (int64_t)blockIdx.x * kRowsPerBlock + threadIdx.x / LANES;
  }
  MOE_DEV static int col() { return WIDE ? threadIdx.x : threadIdx.x % LANES; }
};

template <bool GATED, int LANES, bool WIDE, int TURNS>
__global__ void __launch_bounds__(kThreads, TURNS > 1 ? 3 : 4) act_checkpoint_kernel(ActCheckpoint a) {
  using M = Map<LANES, WIDE, TURNS>;
  constexpr int kT = M::kTurns, kH = GATED ? 2 : 1;
  moe::wait_for_stream();
  moe::let_next_start();
  const int64_t row = M::row();
  const bool in = row < a.rows;
  const int units = a.I / 8, lane = threadIdx.x & 31;
  const int64_t N1 = GATED ? 2 * (int64_t)a.I : a.I;
  const float w = !in ? 0.f : (a.row_w ? a.row_w[row] : 1.f);
  const uint4* z = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.gu) + row * N1);
  uint4* h = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.h) + row * a.I);
  uint2* codes = reinterpret_cast<uint2*>(a.codes + row * N1);
  uint8_t* scales = a.scales + row * (N1 / 32);
  // every lane makes every turn: the shuffles of a quad need its four lanes
  for (int c0 = 0; c0 < units; c0 += kT * M::kStep) {
    uint4 raw[kT][kH];
    uint32_t packed[kH] = {};
#pragma unroll
    for (int t = 0; t < kT; ++t) {
      const int c = c0 + t * M::kStep + M::col();
#pragma unroll
      for (int p = 0; p < kH; ++p)  // a row of weight 0 is left out: nothing of it is read, its outputs are zeros
        raw[t][p] = in && c < units && w != 0.f ? __ldcs(z + p * units + c) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int t = 0; t < kT; ++t) {
      const int c = c0 + t * M::kStep + M::col();
      const bool live = in && c < units;
      float g[8], u[8], o[8];
      unpack8(raw[t][0], g);
      if (GATED) unpack8(raw[t][kH - 1], u);
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = w == 0.f ? 0.f : w * (GATED ? g[i] * sigmoid(g[i]) * u[i] : moe::relu2(g[i]));
      uint32_t sg, su = 0;
      const uint2 cg = quant8(raw[t][0], g, sg);
      uint2 cu = make_uint2(0, 0);
      if (GATED) cu = quant8(raw[t][kH - 1], u, su);
      if (live) {
        if (a.h) __stcs(h + c, pack8(o));
        __stcs(codes + c, cg);
        if (GATED) __stcs(codes + units + c, cu);
        if (kT == 1 && (c & 3) == 0) {
          scales[c >> 2] = (uint8_t)sg;
          if (GATED) scales[(units + c) >> 2] = (uint8_t)su;
        }
      }
      packed[0] |= sg << (8 * t);
      if (GATED) packed[kH - 1] |= su << (8 * t);
    }
    if (kT > 1) {  // lane kQ t + q of a row stores the scale of turn t's quad q
      constexpr int kQ = LANES / 4;
      const int sub = lane % LANES, b = c0 / 4 + sub;
#pragma unroll
      for (int p = 0; p < kH; ++p) {
        const uint32_t v = __shfl_sync(kAll, packed[p], (sub % kQ) * 4, LANES);
        if (in && sub < kQ * kT && b * 4 < units) scales[p * (units / 4) + b] = (uint8_t)(v >> (8 * (sub / kQ)));
      }
    }
  }
}

template <bool GATED, int LANES, bool WIDE, int TURNS>
__global__ void __launch_bounds__(kThreads, TURNS > 1 ? 3 : 4) act_backward_kernel(ActBackward a) {
  using M = Map<LANES, WIDE, TURNS>;
  constexpr int kT = M::kTurns, kH = GATED ? 2 : 1;
  moe::wait_for_stream();
  moe::let_next_start();
  const int64_t row = M::row();
  const bool in = row < a.rows;
  const int units = a.I / 8, lane = threadIdx.x & 31;
  const int64_t N1 = GATED ? 2 * (int64_t)a.I : a.I;
  const float w = !in ? 0.f : (a.row_w ? a.row_w[row] : 1.f);
  const uint2* codes = reinterpret_cast<const uint2*>(a.codes + row * N1);
  const uint8_t* scales = a.scales + row * (N1 / 32);
  const uint4* dh = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.dh) + row * a.I);
  uint4* dz = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.d_gu) + row * N1);
  uint4* h = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.h) + row * a.I);
  float dot = 0.f;
  for (int c0 = 0; c0 < units; c0 += kT * M::kStep) {
    uint4 rd[kT];
    uint2 rc[kT][kH];
    uint32_t rs[kT][kH], turns[kH] = {};
    // a row of weight 0 is left out: nothing of it is read, its outputs are zeros
    const bool read = in && w != 0.f;
#pragma unroll
    for (int t = 0; t < kT; ++t) {
      const int c = c0 + t * M::kStep + M::col();
      const bool live = read && c < units;
      rd[t] = live ? __ldcs(dh + c) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int p = 0; p < kH; ++p) {
        rc[t][p] = live ? __ldcs(codes + p * units + c) : make_uint2(0, 0);
        if (kT == 1) rs[t][p] = live ? scales[(p * units + c) >> 2] : 0;
      }
    }
    if (kT > 1) {  // lane kQ t + q of a row holds the scale of turn t's quad q
      constexpr int kQ = LANES / 4;
      const int sub = lane % LANES, b = c0 / 4 + sub;
#pragma unroll
      for (int p = 0; p < kH; ++p) {
        turns[p] = read && sub < kQ * kT && b * 4 < units ? scales[p * (units / 4) + b] : 0;
#pragma unroll
        for (int t = 0; t < kT; ++t) rs[t][p] = __shfl_sync(kAll, turns[p], kQ * t + (sub >> 2), LANES);
      }
    }
#pragma unroll
    for (int t = 0; t < kT; ++t) {
      const int c = c0 + t * M::kStep + M::col();
      if (!in || c >= units) continue;
      float g[8], u[8], d[8], dg[8], du[8], o[8];
      unpack8(rd[t], d);
      dequant8(rc[t][0], rs[t][0], g);
      if (GATED) dequant8(rc[t][kH - 1], rs[t][kH - 1], u);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float wt = w * d[i];
        if (GATED) {
          const float s = sigmoid(g[i]), gs = g[i] * s;
          dot += d[i] * (gs * u[i]);
          o[i] = w * (gs * u[i]);
          du[i] = wt * gs;
          dg[i] = wt * u[i] * (s + gs * (1.f - s));
        } else {
          const float r = g[i] < 0.f ? 0.f : g[i];
          dot += d[i] * (r * r);
          o[i] = w * (r * r);
          dg[i] = 2.f * wt * r;
        }
      }
      __stcs(dz + c, pack8(dg));
      if (GATED) __stcs(dz + units + c, pack8(du));
      if (a.h) __stcs(h + c, pack8(o));
    }
  }
  if (a.d_row_w == nullptr) return;
#pragma unroll
  for (int o = (WIDE ? 32 : LANES) / 2; o > 0; o >>= 1) dot += __shfl_xor_sync(kAll, dot, o);
  if (WIDE) {
    __shared__ float red[kWarps];
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = dot;
    __syncthreads();
    dot = 0.f;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) dot += red[i];
    if (threadIdx.x == 0) a.d_row_w[row] = dot;
  } else if (in && threadIdx.x % LANES == 0) {
    a.d_row_w[row] = dot;
  }
}

constexpr int64_t kFew = 400000;  // eights of columns in all

template <int LANES, bool WIDE, int TURNS>
struct Pick {
  using M = Map<LANES, WIDE, TURNS>;
  static constexpr int kLanes = LANES, kTurns = TURNS;
  static constexpr bool kWide = WIDE;
};

// Few values: as many threads as there are eights, so that SMs are not left empty (a block per row
// above 512 columns: 1500 rows of I = 2048, forward 7.1 us so and 9.7 as warps; 3000 of 512: 3.0 as
// 32 lanes and 3.7 as 16).  Many: the fewest lanes that hold a row in three or four turns, whichever
// leaves fewer of them idle (two where that is all), at most a warp, which then takes the turns over (forward and backward:
// 20000 rows of 2048, 134 us as blocks and 114 as warps; 100000 of 352, 140 us as 32 lanes in two
// turns and 107 as 16 in three; 80000 of 512, 125 and 113; 60000 of 768, 136 in four turns and 130
// in three).
template <typename Args, typename F>
cudaError_t pick(const Args& a, F launch) {
  const int units = a.I / 8, warps = (units + 31) / 32;
  if (a.rows * units < kFew) {
    if (units <= 4) return launch(Pick<4, false, 1>{});
    if (units <= 8) return launch(Pick<8, false, 1>{});
    if (units <= 16) return launch(Pick<16, false, 1>{});
    if (units <= 32) return launch(Pick<32, false, 1>{});
    if (units <= 64) return launch(Pick<32, false, 2>{});
    return launch(Pick<32, true, 1>{});
  }
  if (units <= 4) return launch(Pick<4, false, 1>{});
  if (units <= 8) return launch(Pick<4, false, 2>{});
  if (units <= 12) return launch(Pick<4, false, 3>{});
  if (units <= 16) return launch(Pick<4, false, 4>{});
  if (units <= 24) return launch(Pick<8, false, 3>{});
  if (units <= 32) return launch(Pick<8, false, 4>{});
  if (units <= 48) return launch(Pick<16, false, 3>{});
  if (units <= 64) return launch(Pick<16, false, 4>{});
  if ((warps + 2) / 3 * 3 < (warps + 3) / 4 * 4) return launch(Pick<32, false, 3>{});
  return launch(Pick<32, false, 4>{});
}

template <bool GATED>
cudaError_t checkpoint(const ActCheckpoint& a, cudaStream_t s) {
  return pick(a, [&](auto p) {
    using P = decltype(p);
    const int64_t blocks = (a.rows + P::M::kRowsPerBlock - 1) / P::M::kRowsPerBlock;
    return moe_launch::launch_staged(act_checkpoint_kernel<GATED, P::kLanes, P::kWide, P::kTurns>, dim3((unsigned)blocks),
                                     dim3(kThreads), 0, s, 1, a);
  });
}

template <bool GATED>
cudaError_t backward(const ActBackward& a, cudaStream_t s) {
  return pick(a, [&](auto p) {
    using P = decltype(p);
    const int64_t blocks = (a.rows + P::M::kRowsPerBlock - 1) / P::M::kRowsPerBlock;
    return moe_launch::launch_staged(act_backward_kernel<GATED, P::kLanes, P::kWide, P::kTurns>, dim3((unsigned)blocks),
                                     dim3(kThreads), 0, s, 1, a);
  });
}

}  // namespace

namespace moe_launch {

cudaError_t act_checkpoint(const ActCheckpoint& a, cudaStream_t stream) {
  if (a.rows == 0) return cudaSuccess;
  return a.gated ? checkpoint<true>(a, stream) : checkpoint<false>(a, stream);
}

cudaError_t act_backward(const ActBackward& a, cudaStream_t stream) {
  if (a.rows == 0) return cudaSuccess;
  return a.gated ? backward<true>(a, stream) : backward<false>(a, stream);
}

}  // namespace moe_launch
