// Residual addition with dropout and the root-mean-square norm, with 8-bit outputs, and the backward
// pass.
//
// Forward, per row of K values that counts (mask):
//   s = residual + drop(x)                          stored in the stream's type (bf16 or fp32)
//   n = s r w,  r = (mean(s^2) + eps)^(-1/2)        from the unrounded s, in fp32
//   out = bf16(n);  MX: mxq's rule per 32 values;  row: max |n| / 448 and E4M3(n 448 / max |n|)
// Backward, from the stored stream s alone (its row gives r again), with g = d_out w:
//   ds = r (g - s r^2 mean(g s)) + d_stream;  d_residual = ds;  d_x = drop'(ds)
//   d_w = sum over rows of d_out s r
// Dropout draws its numbers again in both passes, so there is no mask to write or read: Philox 4x32
// with ten rounds (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as easy as 1, 2, 3", SC
// 2011) on the counter (index / 8, step, stream) under the seed.  Its 128 bits are eight 16-bit
// numbers, one for each of the eight values that a thread moves as 16 bytes: 20 wide multiplications
// for eight values instead of the 40 that 32-bit numbers would take, at the price of a probability in
// steps of 2^-16.
//
// Both passes are bound by memory: every tensor is read or written once, and a row stays in registers from
// its sums to its outputs.  Measured (replayed graphs): 8192 x 7168 to bf16, stream and MX codes 81 us, 6.56
// TB/s (a copy moves 6.78); 61440 x 2880 with an fp32 stream and dropout, forward and back, 735 us, 6.6 TB/s;
// 8192 x 7168 in bf16 the same 177 us, 6.0 TB/s (171 without dropout: what the generator computes is not all
// hidden).  Few rows are bound by the launch and two latencies: 64 x 2880 1.5 us.
// With the backward pass's loads into registers these were 283 us (no room for loads ahead beside the sums
// of d_w), with rings of bulk copies, which need a barrier and a thread that issues them, 238.
#include <cuda_fp8.h>

#include <algorithm>

#include "cp_async.cuh"
#include "moe_common.cuh"
#include "moe_launch.h"
#include "mx_quant.cuh"
#include "per_device.h"
#include "tcgen05.cuh"

namespace {

using moe_launch::ResidualNorm;
using moe_launch::ResidualNormBackward;

constexpr unsigned kAll = 0xffffffffu;
constexpr int kThreads = 256;  // of a block whose rows are narrow

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

// Eight values of the residual stream as they are loaded and stored.
template <bool F32>
struct Eight {
  uint4 v[F32 ? 2 : 1];
  MOE_DEV void load(const void* p, int64_t unit) {
#pragma unroll
    for (int i = 0; i < (F32 ? 2 : 1); ++i) v[i] = __ldcs(static_cast<const uint4*>(p) + unit * (F32 ? 2 : 1) + i);
  }
  MOE_DEV void zero() {
#pragma unroll
    for (int i = 0; i < (F32 ? 2 : 1); ++i) v[i] = make_uint4(0, 0, 0, 0);
  }
  MOE_DEV void get(float (&f)[8]) const {
    if (F32) {
      const uint32_t w[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[F32].x, v[F32].y, v[F32].z, v[F32].w};
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(w[i]);
    } else {
      unpack8(v[0], f);
    }
  }
  MOE_DEV static void store(void* p, int64_t unit, const float (&f)[8]) {
    uint4* q = static_cast<uint4*>(p) + unit * (F32 ? 2 : 1);
    if (F32) {
      __stcs(q, make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3])));
      __stcs(q + 1, make_uint4(__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]), __float_as_uint(f[7])));
    } else {
      __stcs(q, pack8(f));
    }
  }
};

// The generator's key and the counter's constant half; below is what drops an element (16 bits).
struct Dropout {
  uint32_t k0, k1, step, stream, below;
  float gain;
  MOE_DEV void init(const int64_t* rng, uint32_t stream_id, uint32_t drop_below, float kept_gain) {
    below = drop_below << 16;
    gain = kept_gain;
    stream = stream_id;
    k0 = k1 = step = 0;
    if (below) {
      const uint64_t seed = (uint64_t)rng[0];
      k0 = (uint32_t)seed;
      k1 = (uint32_t)(seed >> 32);
      step = (uint32_t)rng[1];
    }
  }
  // f = gain f or 0, for the eight values of unit `unit` of the flat tensor
  MOE_DEV void apply(int64_t unit, float (&f)[8]) const {
    if (!below) return;
    uint32_t c0 = (uint32_t)unit, c1 = (uint32_t)((uint64_t)unit >> 32), c2 = step, c3 = stream, a = k0, b = k1;
#pragma unroll
    for (int i = 0; i < 10; ++i) {
      const uint64_t p0 = (uint64_t)0xD2511F53u * c0, p1 = (uint64_t)0xCD9E8D57u * c2;
      c0 = (uint32_t)(p1 >> 32) ^ c1 ^ a;
      c1 = (uint32_t)p1;
      c2 = (uint32_t)(p0 >> 32) ^ c3 ^ b;
      c3 = (uint32_t)p0;
      a += 0x9E3779B9u;
      b += 0xBB67AE85u;
    }
    const uint32_t w[4] = {c0, c1, c2, c3};
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // `below` is in the upper half: the lower half of w does not change the comparison
      f[2 * i] = (w[i] << 16) >= below ? __fmul_rn(f[2 * i], gain) : 0.f;
      f[2 * i + 1] = w[i] >= below ? __fmul_rn(f[2 * i + 1], gain) : 0.f;
    }
  }
};

// Rows of a block: WIDE = the whole block on one row, otherwise 32 / LANES rows a warp.  A thread
// holds V eights of its row, kStep apart, so that a row is loaded at once and read once.
template <int LANES, bool WIDE, int V>
struct Map {
  static constexpr int kLanes = LANES, kV = V;
  static constexpr bool kWide = WIDE;
  static constexpr int kMost = WIDE ? 1024 : kThreads;  // threads of a block
  MOE_DEV static int rows() { return WIDE ? 1 : kThreads / LANES; }
  MOE_DEV static int group() { return WIDE ? 0 : threadIdx.x / LANES; }
  MOE_DEV static int col() { return WIDE ? threadIdx.x : threadIdx.x % LANES; }
  MOE_DEV static int step() { return WIDE ? blockDim.x : LANES; }
};

// Sums of a and b (MAX: the largest of b's non-negative bits, NaN above all) over the threads of a row,
// in a fixed order.  `red`: shared memory for WIDE; the caller separates two uses of it by a barrier.
template <typename M, bool MAX = false>
MOE_DEV void reduce_pair(float& a, float& b, float2* red) {
  const auto lanes = [&](int n) {
    const bool whole = MAX && n == 32;  // shuffles bound row scales: 8192 x 7168 to codes alone 64 us without this, 58
    if (whole) b = __uint_as_float(__reduce_max_sync(kAll, __float_as_uint(b)));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      if (o >= n) continue;
      a += __shfl_xor_sync(kAll, a, o);
      if (whole) continue;
      const float c = __shfl_xor_sync(kAll, b, o);
      b = MAX ? __uint_as_float(max(__float_as_uint(b), __float_as_uint(c))) : b + c;
    }
  };
  lanes(M::kLanes);
  if (M::kWide) {
    const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) red[threadIdx.x >> 5] = make_float2(a, b);
    __syncthreads();
    const float2 v = lane < warps ? red[lane] : make_float2(0.f, 0.f);
    a = v.x;
    b = v.y;
    lanes(32);
  }
}

// (sum / K + eps)^(-1/2): rsqrtf and a Newton step, within 2 units of the last place; 0 for an infinite
// sum.
MOE_DEV float inverse_rms(float sum, float inv_k, float eps) {
  const float m = __fmaf_rn(sum, inv_k, eps), r = rsqrtf(m);
  const float e = __fmaf_rn(-m * r, r, 1.f);
  return m <= 3.4028235e38f ? __fmaf_rn(0.5f * r, e, r) : (m > 3.4028235e38f ? 0.f : m);
}

// E4M3 codes of eight values, saturated at 448, NaN kept.
MOE_DEV uint2 codes8(const float (&v)[8], float by) {
  uint32_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    h[i] = __nv_cvt_float2_to_fp8x2(make_float2(v[2 * i] * by, v[2 * i + 1] * by), __NV_SATFINITE, __NV_E4M3);
  return make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
}

// MXFP8 of a 32-value block held eight values a lane by four neighbouring lanes, all of which call:
// mxq::quant32's rule.
MOE_DEV uint2 quant8(const float (&v)[8], uint32_t& scale) {
  uint32_t b = 0;  // magnitudes are ordered like their bits, NaN above all
#pragma unroll
  for (int i = 0; i < 8; ++i) b = max(b, __float_as_uint(v[i]) & 0x7fffffffu);
  b = max(b, __shfl_xor_sync(kAll, b, 1));
  b = max(b, __shfl_xor_sync(kAll, b, 2));
  if (b > 0x7f800000u) {
    scale = 255u;
    return make_uint2(0x7f7f7f7fu, 0x7f7f7f7fu);
  }
  const int e = mxq::block_exponent(__uint_as_float(b));
  scale = (uint32_t)(e + 127);
  return codes8(v, e >= 127 ? __uint_as_float(0x00400000u) : __uint_as_float((uint32_t)(127 - e) << 23));
}

// The smallest scale of a row: zero rows have it, and 1 / scale stays finite.
constexpr float kRowScaleMin = 0x1p-120f;

// How a row becomes codes: of s `first` w `by`.
struct RowCodes {
  float scale, first, by;
};
// Below this 448 / max |s w| may be infinite, and the products s w lose bits (or all of them).
constexpr float kTopMin = 0x1p-119f;
// The scale of a row whose largest |s w| is `top`, finite and kTopMin at least.  Its codes are those of s w 448 /
// top, which is n 448 / max |n| without r's rounding, or of n 2^120 where the scale is the smallest.
MOE_DEV RowCodes row_codes(float top, float r) {
  const float most = top * r, nan = __uint_as_float(0x7fc00000u);
  if (!(most <= 3.4028235e38f)) return RowCodes{nan, 1.f, nan};  // an infinity, too, leaves NaN in its row
  if (most / 448.f < kRowScaleMin) return RowCodes{kRowScaleMin, r, 1.f / kRowScaleMin};
  return RowCodes{most / 448.f, 1.f, 448.f / top};
}
// The same from the largest |n|, for other rows: of n 448 / most, at most n 2^120.
MOE_DEV RowCodes row_codes_of_n(float most, float r) {
  const RowCodes rc = row_codes(most, 1.f);
  return RowCodes{rc.scale, r, rc.by};
}
// How the row of s becomes codes.  Small rows (those of zeros among them) and those in which s w overflows (n is 0
// where the sum of squares did) go over their products again, so all threads of a row call, and of a warp; `red`:
// as reduce_pair's, this thread's last use of it is over.
template <typename M>
MOE_DEV RowCodes codes_of(const float (&s)[M::kV][8], const uint4 (&w)[M::kV], float top, float r, float2* red) {
  const bool other = !(top >= kTopMin && top <= 3.4028235e38f);
  if (!(M::kWide ? other : __any_sync(kAll, other))) return row_codes(top, r);
  float none = 0.f, most = 0.f;
#pragma unroll
  for (int t = 0; t < M::kV; ++t) {
    float f[8];
    unpack8(w[t], f);
#pragma unroll
    for (int i = 0; i < 8; ++i) most = __uint_as_float(max(__float_as_uint(most), __float_as_uint(s[t][i] * r * f[i]) & 0x7fffffffu));
  }
  if (M::kWide) __syncthreads();  // the first sums have been read
  reduce_pair<M, true>(none, most, red);
  return other ? row_codes_of_n(most, r) : row_codes(top, r);
}

// The outputs of eight values s of unit u (c: its unit in the row); every lane calls.
template <int QUANT>
MOE_DEV void finish(const ResidualNorm& p, const float (&s)[8], const uint4& w, float r, const RowCodes& rc, int64_t u, int c, bool on) {
  float f[8];
  unpack8(w, f);
  if (QUANT == 2) {
    float q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = s[i] * rc.first * f[i];
    if (on) __stcs(reinterpret_cast<uint2*>(p.codes) + u, codes8(q, rc.by));
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = s[i] * r * f[i];  // zeros where a row does not count: its s and w are
  if (on && p.out) __stcs(static_cast<uint4*>(p.out) + u, pack8(f));
  if (QUANT == 1) {
    uint32_t e;
    const uint2 q = quant8(f, e);
    if (on) {
      __stcs(reinterpret_cast<uint2*>(p.codes) + u, q);
      if ((c & 3) == 0) static_cast<uint8_t*>(p.scales)[u >> 2] = (uint8_t)e;
    }
  }
}

// The outputs of eight values of a row that does not count, but for a row's scale.
template <bool F32, int QUANT>
MOE_DEV void store_zeros(const ResidualNorm& p, int64_t u, int c) {
  const float z[8] = {};
  if (p.stream) Eight<F32>::store(p.stream, u, z);
  if (p.out) __stcs(static_cast<uint4*>(p.out) + u, make_uint4(0, 0, 0, 0));
  if (QUANT) __stcs(reinterpret_cast<uint2*>(p.codes) + u, make_uint2(0, 0));
  if (QUANT == 1 && (c & 3) == 0) static_cast<uint8_t*>(p.scales)[u >> 2] = 0;
}

// QUANT: 0 no codes, 1 a power of two per 32 values, 2 a scale per row.
template <bool F32, int QUANT, typename M>
__global__ void __launch_bounds__(M::kMost) residual_norm_kernel(ResidualNorm p) {
  constexpr int V = M::kV;
  __shared__ float2 red[32];
  moe::wait_for_stream();
  moe::let_next_start();
  const int64_t row = (int64_t)blockIdx.x * M::rows() + M::group();
  const int units = p.K / 8;
  const bool in = row < p.T;
  const bool live = in && (p.mask == nullptr || p.mask[row] != 0);
  const int64_t u0 = row * units;
  Dropout drop;
  drop.init(p.rng, p.rng_stream, p.x ? p.drop_below : 0u, p.gain);

  Eight<F32> res[V];
  uint4 x[V], w[V];
#pragma unroll
  for (int t = 0; t < V; ++t) {
    const int c = M::col() + t * M::step();
    const bool on = live && c < units;
    if (on && p.residual) res[t].load(p.residual, u0 + c);
    else res[t].zero();
    x[t] = on && p.x ? __ldcs(static_cast<const uint4*>(p.x) + u0 + c) : make_uint4(0, 0, 0, 0);
    w[t] = c < units ? static_cast<const uint4*>(p.weight)[c] : make_uint4(0, 0, 0, 0);
    if (!live) w[t] = make_uint4(0, 0, 0, 0);  // its outputs are zeros, whatever the weight holds
  }
  float s[V][8], sum = 0.f, top = 0.f;
#pragma unroll
  for (int t = 0; t < V; ++t) {
    const int c = M::col() + t * M::step();
    float f[8];
    res[t].get(s[t]);
    if (p.x) {
      unpack8(x[t], f);
      if (live && c < units) drop.apply(u0 + c, f);
      // a product and a sum, each rounded: the stored stream does not depend on how they are contracted
#pragma unroll
      for (int i = 0; i < 8; ++i) s[t][i] = __fadd_rn(s[t][i], f[i]);
    }
    if (p.stream && in && c < units) Eight<F32>::store(p.stream, u0 + c, s[t]);
    if (QUANT == 2) unpack8(w[t], f);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      sum += s[t][i] * s[t][i];
      if (QUANT == 2) top = __uint_as_float(max(__float_as_uint(top), __float_as_uint(s[t][i] * f[i]) & 0x7fffffffu));
    }
  }
  reduce_pair<M, QUANT == 2>(sum, top, red);
  const float r = inverse_rms(sum, 1.f / (float)p.K, p.eps);
  RowCodes rc{};
  if (QUANT == 2) {
    rc = codes_of<M>(s, w, top, r, red);
    if (in && M::col() == 0) static_cast<float*>(p.scales)[row] = rc.scale;
  }
#pragma unroll
  for (int t = 0; t < V; ++t) {
    const int c = M::col() + t * M::step();
    finish<QUANT>(p, s[t], w[t], r, rc, u0 + c, c, in && c < units);
  }
}

// ---------------------------------------------------------------------------------------------
// Many rows.  A block walks over batches of rows (one, or as many narrow ones as its threads hold), so
// that a thread keeps its columns.  Its lanes bring their columns of the next kAhead batches into
// shared memory by asynchronous copies and read nobody else's, so the ring needs no barrier of the
// block: the copies of the next rows are in flight through the sums and stores of this one, whatever
// the registers hold.

// Planes of 16 bytes a thread; a stage has several.
template <typename M>
struct Ring {
  uint32_t base, step;  // the first thread of this one's row group in plane 0, bytes of a plane
  int lane;             // within the row group
  MOE_DEV void init(uint8_t* smem) {
    lane = threadIdx.x % M::kLanes;
    base = tc::smem_addr(smem) + (threadIdx.x - lane) * 16;
    step = blockDim.x * 16;
  }
  static MOE_DEV uint4 read(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
  }
  static MOE_DEV void write(uint32_t a, const uint4& v) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
  }
  MOE_DEV uint32_t at(int plane) const { return base + plane * step + lane * 16; }
  // Chunk j < 2 kLanes of the group's, in two planes: lanes that copy neighbours and lanes that read
  // every second one both meet each bank once.
  MOE_DEV uint32_t pair_at(int plane, int j) const {
    const int p = j ^ ((j >> 3) & 1);
    return base + (plane + p / M::kLanes) * step + (p % M::kLanes) * 16;
  }
  // This lane's eight bf16 of unit u (c: its unit in the row), into one plane.
  MOE_DEV void fetch16(int plane, const void* p, int64_t u, int c, int units) const {
    if (c < units) cpa::cp_async16(at(plane), static_cast<const uint4*>(p) + u);
  }
  // The same of a stream's values.  fp32: two planes; a lane copies two chunks of its group that lie
  // kLanes apart, so that a warp copies whole lines, and reads its own two after stream_ready().
  template <bool F32>
  MOE_DEV void fetch_stream(int plane, const void* p, int64_t u, int c, int units) const {
    if (!F32) return fetch16(plane, p, u, c, units);
    const int64_t first = 2 * (u - lane);
    const int last = 2 * (units - (c - lane));
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int j = h * M::kLanes + lane;
      if (j < last) cpa::cp_async16(pair_at(plane, j), static_cast<const uint4*>(p) + first + j);
    }
  }
  template <bool F32>
  MOE_DEV Eight<F32> stream(int plane) const {
    Eight<F32> e;
    if (!F32) {
      e.v[0] = read(at(plane));
    } else {
      e.v[0] = read(pair_at(plane, 2 * lane));
      e.v[F32] = read(pair_at(plane, 2 * lane + 1));
    }
    return e;
  }
};

// Backward.  HOLD: a row's values stay in registers from the sums to the outputs and its stage is filled
// again at once; otherwise (two eights a thread of a large block) they are read again.
template <bool F32, typename M, int kAhead>
__global__ void __launch_bounds__(M::kMost) residual_norm_backward_kernel(ResidualNormBackward p) {
  constexpr int V = M::kV, kS = F32 ? 2 : 1, kPer = 1 + 2 * kS, kChunks = V * kPer;  // a stage's: d_out, stream, d_stream
  constexpr bool kHold = !M::kWide || V == 1;
  constexpr int kHeld = kHold ? V : 1;
  // A row that does not count is zeros, whatever the weight holds: as products with a weight of zeros for fp32
  // streams (61440 x 2880 forward and back 735 us, as a branch 752), as a branch otherwise (8192 x 7168 177, as
  // products 184).
  constexpr bool kBranch = !F32;
  const auto weight = [](bool live, const uint4& z) { return kBranch || live ? z : make_uint4(0, 0, 0, 0); };
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float2 red[2][32];
  moe::wait_for_stream();
  moe::let_next_start();
  const int rows = M::rows(), units = p.K / 8;
  const int64_t stride = (int64_t)gridDim.x * rows;
  const float inv_k = 1.f / (float)p.K;
  Dropout drop;
  drop.init(p.rng, p.rng_stream, p.d_x ? p.drop_below : 0u, p.gain);
  Ring<M> ring;
  ring.init(smem);
  uint4 w[kHeld];
  float dw[V][8];
#pragma unroll
  for (int t = 0; t < V; ++t) {
    const int c = M::col() + t * M::step();
    const uint4 z = c < units ? static_cast<const uint4*>(p.weight)[c] : make_uint4(0, 0, 0, 0);
    if (kHold) w[t] = z;
    else ring.write(ring.at(kAhead * kChunks + t), z);  // planes of their own
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[t][i] = 0.f;
  }
  const auto fetch = [&](int64_t row, int s) {
    if (row < p.T) {
#pragma unroll
      for (int t = 0; t < V; ++t) {
        const int c = M::col() + t * M::step(), k = s * kChunks + t * kPer;
        const int64_t u = row * units + c;
        ring.fetch16(k, p.d_out, u, c, units);
        ring.template fetch_stream<F32>(k + 1, p.stream, u, c, units);
        if (p.d_stream) ring.template fetch_stream<F32>(k + 1 + kS, p.d_stream, u, c, units);
      }
    }
    cpa::cp_async_commit();
  };
  int64_t row = (int64_t)blockIdx.x * rows + M::group();
  for (int s = 0; s < kAhead; ++s) fetch(row + s * stride, s);
  uint32_t counts = p.mask == nullptr || (row < p.T && p.mask[row] != 0);
  int s = 0, turn = 0;
  for (int64_t row0 = (int64_t)blockIdx.x * rows; row0 < p.T; row0 += stride, row += stride, turn ^= 1) {
    const bool in = row < p.T, live = in && counts;
    if (p.mask) counts = row + stride < p.T ? p.mask[row + stride] : 0;  // the next row's, a turn ahead
    cpa::cp_async_wait<kAhead - 1>();
    if (F32) __syncwarp();  // other lanes' copies
    Eight<F32> st[kHeld], ds[kHeld];
    uint4 d[kHeld];
    float sum = 0.f, dot = 0.f;
#pragma unroll
    for (int t = 0; t < V; ++t) {
      const int k = s * kChunks + t * kPer, h = kHold ? t : 0, c = M::col() + t * M::step();
      d[h] = make_uint4(0, 0, 0, 0);
      st[h].zero();
      ds[h].zero();
      if (!kHold) w[0] = ring.read(ring.at(kAhead * kChunks + t));
      if (live && c < units) {
        d[h] = ring.read(ring.at(k));
        st[h] = ring.template stream<F32>(k + 1);
        if (kHold && p.d_stream) ds[h] = ring.template stream<F32>(k + 1 + kS);
      }
      float v[8], g[8], f[8];
      st[h].get(v);
      unpack8(d[h], g);
      unpack8(weight(live, w[h]), f);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        sum += v[i] * v[i];
        dot += g[i] * f[i] * v[i];
      }
    }
    const int stage = s;
    s = s + 1 == kAhead ? 0 : s + 1;
    if (kHold) {
      if (F32) __syncwarp();
      fetch(row + kAhead * stride, stage);
    }
    reduce_pair<M>(sum, dot, red[turn]);  // two sets in turn: one barrier a row is enough
    const float r = inverse_rms(sum, inv_k, p.eps);
    const float q = r == 0.f ? 0.f : r * r * (dot * inv_k);  // the norm of such a row is 0, whatever overflows in dot
#pragma unroll
    for (int t = 0; t < V; ++t) {
      const int c = M::col() + t * M::step(), h = kHold ? t : 0, k = stage * kChunks + t * kPer;
      if (!in || c >= units) continue;
      const int64_t u = row * units + c;
      if (kBranch && !live) {
        const float z[8] = {};
        if (p.d_residual) Eight<F32>::store(p.d_residual, u, z);
        if (p.d_x) __stcs(static_cast<uint4*>(p.d_x) + u, make_uint4(0, 0, 0, 0));
        continue;
      }
      if (!kHold && live) {
        d[0] = ring.read(ring.at(k));
        st[0] = ring.template stream<F32>(k + 1);
        if (p.d_stream) ds[0] = ring.template stream<F32>(k + 1 + kS);
        w[0] = ring.read(ring.at(kAhead * kChunks + t));
      }
      float v[8], g[8], f[8], o[8];
      st[h].get(v);
      unpack8(d[h], g);
      unpack8(weight(live, w[h]), f);
      ds[h].get(o);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        o[i] = r * (g[i] * f[i] - v[i] * q) + o[i];
        dw[t][i] += g[i] * (v[i] * r);
      }
      if (p.d_residual) Eight<F32>::store(p.d_residual, u, o);
      if (p.d_x) {
        if (live) drop.apply(u, o);
        __stcs(static_cast<uint4*>(p.d_x) + u, pack8(o));
      }
    }
    if (!kHold) {
      if (F32) __syncwarp();
      fetch(row + kAhead * stride, stage);
    }
  }
  if (p.parts == nullptr) return;
  float* mine = p.parts + (int64_t)blockIdx.x * p.K;
  if (M::kWide) {
#pragma unroll
    for (int t = 0; t < V; ++t) {
      const int c = M::col() + t * M::step();
      if (c < units) {
        reinterpret_cast<float4*>(mine)[2 * c] = make_float4(dw[t][0], dw[t][1], dw[t][2], dw[t][3]);
        reinterpret_cast<float4*>(mine)[2 * c + 1] = make_float4(dw[t][4], dw[t][5], dw[t][6], dw[t][7]);
      }
    }
  } else {
    constexpr int kCols = 8 * V * M::kLanes;
    float* shares = reinterpret_cast<float*>(smem);  // [groups][columns], once no thread reads the ring
    cpa::cp_async_wait<0>();
    __syncthreads();
#pragma unroll
    for (int t = 0; t < V; ++t)
#pragma unroll
      for (int i = 0; i < 8; ++i) shares[M::group() * kCols + (M::col() + t * M::step()) * 8 + i] = dw[t][i];
    __syncthreads();
    for (int k = threadIdx.x; k < p.K; k += kThreads) {
      float a = 0.f;
      for (int g = 0; g < rows; ++g) a += shares[g * kCols + k];
      mine[k] = a;
    }
  }
}

// Forward.
template <bool F32, int QUANT, typename M, int kAhead>
__global__ void __launch_bounds__(M::kMost) residual_norm_walk_kernel(ResidualNorm p) {
  constexpr int V = M::kV, kS = F32 ? 2 : 1, kPer = 1 + kS, kChunks = V * kPer;  // a stage's: x, residual
  // With codes, a row's outputs all leave at once and two rows are read ahead (8192 x 7168 MX: 80 us; the
  // stream before the sums 86, and with four rows ahead 91: memory that turns between reads and writes less
  // often moves more); dropout spreads them well enough (forward and back 178 us, otherwise 184).
  constexpr bool kLate = QUANT != 0;
  static_assert(M::kWide, "whether a row counts is the same for the whole block");
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float2 red[2][32];
  moe::wait_for_stream();
  moe::let_next_start();
  const int rows = M::rows(), units = p.K / 8;
  const int64_t stride = (int64_t)gridDim.x * rows;
  const float inv_k = 1.f / (float)p.K;
  Dropout drop;
  drop.init(p.rng, p.rng_stream, p.x ? p.drop_below : 0u, p.gain);
  Ring<M> ring;
  ring.init(smem);
  uint4 w[V];
#pragma unroll
  for (int t = 0; t < V; ++t) {
    const int c = M::col() + t * M::step();
    w[t] = c < units ? static_cast<const uint4*>(p.weight)[c] : make_uint4(0, 0, 0, 0);
  }
  const auto fetch = [&](int64_t row, int s) {
    if (row < p.T) {
#pragma unroll
      for (int t = 0; t < V; ++t) {
        const int c = M::col() + t * M::step(), k = s * kChunks + t * kPer;
        const int64_t u = row * units + c;
        if (p.x) ring.fetch16(k, p.x, u, c, units);
        if (p.residual) ring.template fetch_stream<F32>(k + 1, p.residual, u, c, units);
      }
    }
    cpa::cp_async_commit();
  };
  int64_t row = (int64_t)blockIdx.x * rows + M::group();
  for (int s = 0; s < kAhead; ++s) fetch(row + s * stride, s);
  uint32_t counts = p.mask == nullptr || (row < p.T && p.mask[row] != 0);
  int stage = 0, turn = 0;
  for (int64_t row0 = (int64_t)blockIdx.x * rows; row0 < p.T; row0 += stride, row += stride) {
    const bool in = row < p.T, live = in && counts;
    if (p.mask) counts = row + stride < p.T ? p.mask[row + stride] : 0;  // the next row's, a turn ahead
    cpa::cp_async_wait<kAhead - 1>();
    if (F32) __syncwarp();  // other lanes' copies
    Eight<F32> res[V];
    uint4 x[V];
#pragma unroll
    for (int t = 0; t < V; ++t) {
      const int k = stage * kChunks + t * kPer;
      const bool on = live && M::col() + t * M::step() < units;
      x[t] = make_uint4(0, 0, 0, 0);
      res[t].zero();
      if (on && p.x) x[t] = ring.read(ring.at(k));
      if (on && p.residual) res[t] = ring.template stream<F32>(k + 1);
    }
    if (F32) __syncwarp();
    fetch(row + kAhead * stride, stage);
    stage = stage + 1 == kAhead ? 0 : stage + 1;
    if (!live) {  // all zeros, whatever the weight holds
#pragma unroll
      for (int t = 0; t < V; ++t) {
        const int c = M::col() + t * M::step();
        if (c < units) store_zeros<F32, QUANT>(p, row * units + c, c);
      }
      if (QUANT == 2 && M::col() == 0) static_cast<float*>(p.scales)[row] = kRowScaleMin;
      continue;
    }
    float s[V][8], sum = 0.f, top = 0.f;
#pragma unroll
    for (int t = 0; t < V; ++t) {
      const int c = M::col() + t * M::step();
      const int64_t u = row * units + c;
      float f[8];
      res[t].get(s[t]);
      if (p.x) {
        unpack8(x[t], f);
        if (live && c < units) drop.apply(u, f);
#pragma unroll
        for (int i = 0; i < 8; ++i) s[t][i] = __fadd_rn(s[t][i], f[i]);
      }
      if (!kLate && p.stream && in && c < units) Eight<F32>::store(p.stream, u, s[t]);
      if (QUANT == 2) unpack8(w[t], f);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        sum += s[t][i] * s[t][i];
        if (QUANT == 2) top = __uint_as_float(max(__float_as_uint(top), __float_as_uint(s[t][i] * f[i]) & 0x7fffffffu));
      }
    }
    reduce_pair<M, QUANT == 2>(sum, top, red[turn]);  // two sets in turn: one barrier a row is enough
    const float r = inverse_rms(sum, inv_k, p.eps);
    RowCodes rc{};
    if (QUANT == 2) {
      rc = codes_of<M>(s, w, top, r, red[turn]);
      if (in && M::col() == 0) static_cast<float*>(p.scales)[row] = rc.scale;
    }
#pragma unroll
    for (int t = 0; t < V; ++t) {
      const int c = M::col() + t * M::step();
      if (kLate && p.stream && in && c < units) Eight<F32>::store(p.stream, row * units + c, s[t]);
      finish<QUANT>(p, s[t], w[t], r, rc, row * units + c, c, in && c < units);
    }
    turn ^= 1;
  }
}

// out[k] = the sum over n parts of parts[i][k], in a fixed order: 32 columns a block, eight lanes of
// four of them, 32 groups of parts.
__global__ void __launch_bounds__(kThreads) column_parts_kernel(const float* parts, int n, int K, float* out) {
  __shared__ float4 sums[32][8];
  moe::wait_for_stream();
  moe::let_next_start();
  const int lane = threadIdx.x & 7, group = threadIdx.x >> 3;
  const int k4 = blockIdx.x * 8 + lane;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
  if (4 * k4 < K)
    for (int i = group; i < n; i += 32) {
      const float4 v = reinterpret_cast<const float4*>(parts + (int64_t)i * K)[k4];
      a.x += v.x;
      a.y += v.y;
      a.z += v.z;
      a.w += v.w;
    }
  sums[group][lane] = a;
  __syncthreads();
  if (group == 0 && 4 * k4 < K) {
    for (int i = 1; i < 32; ++i) {
      const float4 v = sums[i][lane];
      a.x += v.x;
      a.y += v.y;
      a.z += v.z;
      a.w += v.w;
    }
    reinterpret_cast<float4*>(out)[k4] = a;
  }
}

constexpr int64_t kFew = 200000;  // eights of columns in all

// A block or a part of a warp for each row: as many threads as there are eights in wide rows and in few
// narrow ones, which leaves registers for most threads an SM has (8192 x 7168 80 us as four eights a
// thread, 78 as one), up to four eights a lane in many narrow ones, so that a row stays within a warp.
// With codes or dropout, what every thread does for the row counts beside its eights: two of them a thread
// (20000 x 2880: MX 81 us as one, 78 as two; row scales 82 and 75, to codes alone 74 and 66, with four 67;
// dropout, forward and back, 189 and 182).
template <typename F>
cudaError_t pick_once(int64_t T, int K, bool more, F launch) {
  const int units = K / 8;
  if (units <= 8) return launch(Map<8, false, 1>{});
  const bool few = T * units < kFew;
  if (units <= 32) return few ? launch(Map<32, false, 1>{}) : launch(Map<8, false, 4>{});
  if (units <= 64 && !few) return launch(Map<16, false, 4>{});
  if (units <= 128 && !few && !more) return launch(Map<32, false, 4>{});
  if (units <= 1024 && (few || !more)) return launch(Map<32, true, 1>{});
  return launch(Map<32, true, 2>{});
}

template <typename M>
int threads_of(int K) {
  return M::kWide ? ((K / 8 + M::kV - 1) / M::kV + 31) / 32 * 32 : kThreads;
}
template <typename M>
int64_t blocks_of(int64_t T) {
  const int rows = M::kWide ? 1 : kThreads / M::kLanes;
  return (T + rows - 1) / rows;
}

// Blocks of an SM that walk over rows: as many small ones as hold 1024 threads (40000 x 1024, dropout, forward
// and back: 187 us with four, 131 with eight).
constexpr int walkers_most(int threads) { return std::max(4, std::min(8, 1024 / threads)); }
// Blocks that leave a part of d_w.
int parts_most(int K) {
  const int units = K / 8;
  return 152 * walkers_most(units <= 64 ? kThreads : (units + 31) / 32 * 32);  // 1024 eights and more: four
}
constexpr int kRingMost = 224 * 1024;  // shared memory of an SM for the rings of its blocks

// Columns of a thread where blocks walk over rows: narrow rows share warps; wide ones have a block.
template <typename F>
cudaError_t pick_walk(int K, F launch) {
  const int units = K / 8;
  if (units <= 8) return launch(Map<8, false, 1>{});
  if (units <= 32) return launch(Map<16, false, 2>{});
  if (units <= 64) return launch(Map<32, false, 2>{});
  if (units <= 1024) return launch(Map<32, true, 1>{});
  return launch(Map<32, true, 2>{});
}

// Blocks of `kern` that walk over T rows: as many as fit beside one another.  `known`: one for each kernel.
template <typename M, typename K>
int64_t walkers(int64_t T, K kern, int threads, int smem, moe_host::PerDevice<33>& known) {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) dev = -1;
  const int fit = known.get(dev, threads / 32, 1, [&] {
    int n = 0;
    return cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kern, threads, smem) == cudaSuccess ? n : 0;
  });
  return std::min<int64_t>(blocks_of<M>(T), (int64_t)std::min(fit, walkers_most(threads)) * moe_launch::sm_count_current());
}

template <bool F32, int QUANT>
cudaError_t forward(const ResidualNorm& p, cudaStream_t stream) {
  // Blocks that walk over rows pay where a block of its own leaves a row too few neighbours beside it to
  // hide what it computes: wide rows with dropout or codes, and those above 1024 eights, in bf16
  // (8192 x 7168: dropout 79 us and 88 as blocks of their own, row scales 82 and 84, MX 80 and 92, the
  // norm alone 82 and 78; 4778 x 12288: 80 and 86, dropout 78 and 103; 14336 x 4096 MX 95 and 81; fp32
  // streams 121 and 101 and more).  A thread has two eights where a row becomes codes of its own scale alone
  // (66 us as one and as two; without x and the stream, 58 and 50), otherwise one (with the bf16 rows beside
  // the codes 82 as one and 94 as two).
  if constexpr (!F32) {
    if (p.K > 8192 ? p.T * (p.K / 8) >= kFew : p.K > 4096 && p.T * (p.K / 8) >= 4 * kFew && (p.drop_below || QUANT)) {
      const auto walk = [&](auto m) {
        using M = decltype(m);
        static std::atomic<uint64_t> done[2] = {};
        static moe_host::PerDevice<33> known[2];
        const int threads = threads_of<M>(p.K), stage = threads * 16 * M::kV * 2;
        const bool deep = QUANT == 0 && 4 * stage <= kRingMost;  // rows ahead: four, or two with codes and where they do not fit
        const auto kern = deep ? residual_norm_walk_kernel<F32, QUANT, M, 4> : residual_norm_walk_kernel<F32, QUANT, M, 2>;
        const int smem = (deep ? 4 : 2) * stage;
        const cudaError_t e = moe_launch::allow_smem((const void*)kern, kRingMost, done[deep]);
        if (e != cudaSuccess) return e;
        const int64_t blocks = walkers<M>(p.T, kern, threads, smem, known[deep]);
        return moe_launch::launch_staged(kern, dim3((unsigned)blocks), dim3((unsigned)threads), smem, stream, 1, p);
      };
      return p.K <= 8192 && (QUANT != 2 || p.out) ? walk(Map<32, true, 1>{}) : walk(Map<32, true, 2>{});
    }
  }
  return pick_once(p.T, p.K, QUANT != 0 || p.drop_below != 0, [&](auto m) {
    using M = decltype(m);
    return moe_launch::launch_staged(residual_norm_kernel<F32, QUANT, M>, dim3((unsigned)blocks_of<M>(p.T)),
                                     dim3((unsigned)threads_of<M>(p.K)), 0, stream, 1, p);
  });
}

template <bool F32>
cudaError_t backward(ResidualNormBackward p, float* d_weight, cudaStream_t stream) {
  int64_t parts = 0;
  cudaError_t err = pick_walk(p.K, [&](auto m) {
    using M = decltype(m);
    static std::atomic<uint64_t> done[2] = {};
    static moe_host::PerDevice<33> known[2];
    const int threads = threads_of<M>(p.K), chunk = threads * 16 * M::kV, chunks = F32 ? 5 : 3;
    // two rows ahead (three: 8192 x 7168 forward and back 178 us in place of 177, without dropout 176 and
    // 171), one where they do not fit; the weights of a row that is not held
    const int stage = chunks * chunk, weights = M::kWide && M::kV > 1 ? chunk : 0;
    const int ahead = std::min(2, (kRingMost - weights) / stage), which = ahead - 1;
    const auto kern = ahead == 2 ? residual_norm_backward_kernel<F32, M, 2> : residual_norm_backward_kernel<F32, M, 1>;
    const int smem = std::max(ahead * stage + weights, M::kWide ? 0 : kThreads * 8 * M::kV * 4);
    const cudaError_t e = moe_launch::allow_smem((const void*)kern, kRingMost, done[which]);
    if (e != cudaSuccess) return e;
    parts = std::min<int64_t>(walkers<M>(p.T, kern, threads, smem, known[which]), parts_most(p.K));
    return moe_launch::launch_staged(kern, dim3((unsigned)parts), dim3((unsigned)threads), smem, stream, 1, p);
  });
  if (err != cudaSuccess || d_weight == nullptr) return err;
  return moe_launch::launch_staged(column_parts_kernel, dim3((unsigned)((p.K + 31) / 32)), dim3(kThreads), 0, stream, 1,
                                   (const float*)p.parts, (int)parts, p.K, d_weight);
}

}  // namespace

namespace moe_launch {

size_t residual_norm_workspace_bytes(int K) { return (size_t)parts_most(K) * K * 4; }

cudaError_t residual_norm(const ResidualNorm& p, cudaStream_t stream) {
  if (p.T == 0) return cudaSuccess;
  if (p.stream_f32)
    return p.quant == 0 ? forward<true, 0>(p, stream) : p.quant == 1 ? forward<true, 1>(p, stream) : forward<true, 2>(p, stream);
  return p.quant == 0 ? forward<false, 0>(p, stream) : p.quant == 1 ? forward<false, 1>(p, stream) : forward<false, 2>(p, stream);
}

cudaError_t residual_norm_backward(ResidualNormBackward p, float* d_weight, cudaStream_t stream) {
  if (p.T == 0) return d_weight ? zero_f32(d_weight, p.K, stream) : cudaSuccess;
  return p.stream_f32 ? backward<true>(p, d_weight, stream) : backward<false>(p, d_weight, stream);
}

}  // namespace moe_launch
