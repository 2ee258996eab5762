// Low-rank adapters of many requests beside a dense product: few rows a request.
//
//   out[m] = base[m] + scale[a] (x[m] A[a]^T) B[a]^T,  a the adapter of m's request
//
// Bound by the adapters' bytes: with few rows each of them is read for a handful of rows.  So rows
// are gathered by adapter, whatever their order: a block looks at 512 rows, finds each one's
// occurrence among the rows of its adapter, and every sixteenth is the first of a tile of up to
// sixteen rows of one adapter, the rows of an m16n8k16 MMA.  (250 rows over five adapters are 20
// tiles, and not 250 readings of an adapter.)  Two kernels, v = x A^T and out = base + v B^T; in each
// every CTA takes an equal run of all tiles' blocks of K, or of features, so that one tile and 500
// alike use every SM.  A tile's pieces of v are added in order by those who read them.  The second
// kernel starts under the first one: its tables, the rows without an adapter and B's way into L2 do
// not wait for v.
// The operands of an MMA are read from global memory in their own layout, 16 or 8 bytes a lane: the
// order of K within the products is the lanes', for both operands alike.  v is fp32 and enters the
// second product as two bf16 numbers, 2^-17 of itself off.  Rows are never in one accumulator with
// another adapter's: a request's weights that are not finite stay its own.
#include <algorithm>

#include "moe_common.cuh"
#include "moe_launch.h"

namespace {

using moe_launch::Adapter;

constexpr int kThreads = 512, kWarps = 16;
constexpr int kChunk = 512;   // rows that a block looks at
constexpr int kTile = 16;     // rows of a tile
constexpr int kRankMost = 128;
constexpr unsigned kAll = 0xffffffffu;

struct Rows {
  alignas(16) int32_t id[kChunk];  // a row's adapter, -1: none, -2: of no request
  int16_t occ[kChunk];       // rows of its adapter before it
  int16_t leader[kChunk];    // first rows of the tiles
  int32_t start[kChunk];     // the last request that starts at a row, -1: none
  int32_t start_id[kChunk];  // its adapter and its end
  int32_t start_end[kChunk];
  int32_t warp_sum[kWarps];
  int32_t tiles;
  int32_t rows[kTile];       // of the tile at hand
};
// Read and written 8 or 16 bytes at a time.
struct DownSmem {
  Rows t;
  alignas(16) float part[kWarps * kTile * 32];              // shares of v: [slice][row][rank]
};
struct UpSmem {
  Rows t;
  alignas(16) uint32_t vb[2][kTile * (kRankMost + 8) / 2];  // v's high and low parts: [row][rank], rows 8 ranks apart
};

// A CTA's run over the tiles' blocks: `blocks` a tile, in pieces of one tile each.
struct Run {
  int64_t at, end;
  int blocks;
  MOE_DEV Run(int64_t total, int blocks, int cta, int ctas) : blocks(blocks) {
    at = cta < ctas ? total * cta / ctas : 0;
    end = cta < ctas ? total * (cta + 1) / ctas : 0;
  }
  MOE_DEV bool next(int& tile, int& b0, int& b1) {
    if (at >= end) return false;
    tile = (int)(at / blocks);
    b0 = (int)(at - (int64_t)tile * blocks);
    b1 = (int)min((int64_t)blocks, b0 + end - at);
    at += b1 - b0;
    return true;
  }
};
// The CTA whose run has block x (no run is empty).
MOE_DEV int owner(int64_t x, int64_t total, int ctas) { return (int)(((x + 1) * ctas - 1) / total); }
// CTAs of the first kernel on `tiles` tiles of `blocks` blocks: a tile is cut into at most kPieces
// pieces, or kPieces / 2 + 1 where there are several, whose sums cost as much as they gain.
constexpr int kPieces = 32;
MOE_DEV int down_ctas(int tiles, int blocks, int ctas) {
  return min(ctas, min(tiles <= 4 ? kPieces - 1 : kPieces / 2, blocks) * tiles);
}

MOE_DEV void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// A K step of 32: this lane's eight values of two x rows and of a weight row each.
MOE_DEV void mma32(float (&d)[4], const uint4& x0, const uint4& x1, const uint4& w) {
  const uint32_t a[4] = {x0.x, x1.x, x0.y, x1.y}, b[4] = {x0.z, x1.z, x0.w, x1.w};
  moe::mma_bf16(d, a, w.x, w.y, d);
  moe::mma_bf16(d, b, w.z, w.w, d);
}

// The chunk's rows: adapters, occurrences and tiles.
__device__ __forceinline__ void make_tables(const Adapter& p, Rows& sm, int64_t row0, int rows, bool report) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // Where a request starts in the chunk, or -1.  Of several at one place (offsets that decrease) the last
  // is taken, by every CTA: they meet in the barriers of the same tiles.
  const auto place = [&](int i, int& end, int& id) {
    const int64_t lo = p.row_offsets[i], hi = p.row_offsets[i + 1];
    id = p.adapter[i];
    end = (int)(hi - row0 < rows ? hi - row0 : rows);
    const bool bounds = lo >= 0 && lo <= hi && hi <= p.M, known = id >= -1 && id < p.L;
    if (report && !(bounds && known)) moe::set_status(p.status, bounds ? MOE_ERR_INVALID_EXPERT : MOE_ERR_CAPACITY);
    if (!known) id = -1;
    if (!bounds || lo == hi || hi <= row0 || lo >= row0 + rows) return -1;
    return lo > row0 ? (int)(lo - row0) : 0;
  };
  int end, a;
  sm.start[tid] = -1;
  __syncthreads();
  for (int i = tid; i < p.R; i += kThreads) {
    const int at = place(i, end, a);
    if (at >= 0) atomicMax(&sm.start[at], i);
  }
  __syncthreads();
  for (int i = tid; i < p.R; i += kThreads) {
    const int at = place(i, end, a);
    if (at >= 0 && sm.start[at] == i) {
      sm.start_id[at] = a;
      sm.start_end[at] = end;
    }
  }
  __syncthreads();
  // the request of a row is the last that starts at or before it
  int at = sm.start[tid] >= 0 ? tid : -1;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int up = __shfl_up_sync(kAll, at, o);
    if (lane >= o && up > at) at = up;
  }
  if (lane == 31) sm.warp_sum[warp] = at;
  __syncthreads();
  for (int w = 0; w < warp; ++w) at = max(at, sm.warp_sum[w]);
  const int id = tid < rows && at >= 0 && tid < sm.start_end[at] ? sm.start_id[at] : -2;
  sm.id[tid] = id;
  __syncthreads();
  int occ = 0;
  if (id >= 0) {
    const int4* ids = reinterpret_cast<const int4*>(sm.id);
    for (int j = 0; j < tid / 4; ++j) {
      const int4 q = ids[j];
      occ += (q.x == id) + (q.y == id) + (q.z == id) + (q.w == id);
    }
    for (int j = tid & ~3; j < tid; ++j) occ += sm.id[j] == id;
  }
  sm.occ[tid] = (int16_t)occ;
  const unsigned leads = __ballot_sync(kAll, id >= 0 && occ % kTile == 0);
  if (lane == 0) sm.warp_sum[warp] = __popc(leads);
  __syncthreads();
  int before = 0, all = 0;
  for (int w = 0; w < kWarps; ++w) {
    const int n = sm.warp_sum[w];
    before += w < warp ? n : 0;
    all += n;
  }
  if (leads >> lane & 1) sm.leader[before + __popc(leads & ((1u << lane) - 1))] = (int16_t)tid;
  if (tid == 0) sm.tiles = all;
  __syncthreads();
}

// Eight features of a row: base (or zeros) plus add, to out.
template <bool F32>
__device__ __forceinline__ void add_to_base(const Adapter& p, int64_t at, const float (&add)[8]) {
  if (F32) {
    float4 b[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
    if (p.base) {
      b[0] = reinterpret_cast<const float4*>(static_cast<const float*>(p.base) + at)[0];
      b[1] = reinterpret_cast<const float4*>(static_cast<const float*>(p.base) + at)[1];
    }
    float4* o = reinterpret_cast<float4*>(static_cast<float*>(p.out) + at);
    o[0] = make_float4(b[0].x + add[0], b[0].y + add[1], b[0].z + add[2], b[0].w + add[3]);
    o[1] = make_float4(b[1].x + add[4], b[1].y + add[5], b[1].z + add[6], b[1].w + add[7]);
  } else {
    uint4 b = make_uint4(0, 0, 0, 0);
    if (p.base) b = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.base) + at);
    uint32_t w[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 s = __floats2bfloat162_rn(__uint_as_float(w[i] << 16) + add[2 * i],
                                                     __uint_as_float(w[i] & 0xffff0000u) + add[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&s);
    }
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + at) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// The rows of tile t, -1 where it has fewer than sixteen; every thread calls.
__device__ __forceinline__ int tile_rows(Rows& sm, int t) {
  const int tid = threadIdx.x, lead = sm.leader[t], id = sm.id[lead], from = sm.occ[lead];
  if (tid < kTile) sm.rows[tid] = -1;
  __syncthreads();
  if (sm.id[tid] == id && sm.occ[tid] >= from && sm.occ[tid] < from + kTile) sm.rows[sm.occ[tid] - from] = tid;
  __syncthreads();
  return id;
}

// blockIdx.x: a chunk of 512 rows, a CTA of the chunk's.
__global__ void __launch_bounds__(kThreads, 2) adapter_few_down_kernel(Adapter p, int ctas) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  DownSmem& sm = *reinterpret_cast<DownSmem*>(smem_raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, q = lane & 3;
  const int chunk = blockIdx.x / ctas, cta = blockIdx.x - chunk * ctas;
  const int64_t row0 = (int64_t)chunk * kChunk;
  const int rows = p.M - row0 < kChunk ? (int)(p.M - row0) : kChunk;
  moe::wait_for_stream();
  moe::let_next_start();
  make_tables(p, sm.t, row0, rows, blockIdx.x == 0);

  const int nk = (p.K + 31) / 32, used = down_ctas(sm.t.tiles, nk, ctas);
  const int64_t total = (int64_t)sm.t.tiles * nk;
  const int groups = (p.r + 31) / 32;  // of 32 ranks
  const int slices = kWarps / groups, rg = warp % groups, slice = warp / groups, rp = groups * 32;
  const uint16_t* x = static_cast<const uint16_t*>(p.x);
  Run run(total, nk, cta, used);
  int t, k0, k1;
  while (run.next(t, k0, k1)) {
    const int id = tile_rows(sm.t, t);
    const uint16_t* A = static_cast<const uint16_t*>(p.a) + (int64_t)id * p.r * p.K;
    if (slice < slices) {
      const int ra = sm.t.rows[g], rb = sm.t.rows[g + 8];
      float d[4][4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) d[j][i] = 0.f;
      const uint4 none = make_uint4(0, 0, 0, 0);
      const uint16_t* xa = x + (row0 + (ra < 0 ? 0 : ra)) * p.K;
      const uint16_t* xb = x + (row0 + (rb < 0 ? 0 : rb)) * p.K;
      for (int c = k0 + slice; c < k1; c += slices) {
        const int k = c * 32 + q * 8;
        const bool on = k < p.K;
        uint4 w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int n = rg * 32 + j * 8 + g;
          w[j] = on && n < p.r ? moe::ldg_nc_u128(A + (int64_t)n * p.K + k) : none;
        }
        const uint4 x0 = on && ra >= 0 ? *reinterpret_cast<const uint4*>(xa + k) : none;
        const uint4 x1 = on && rb >= 0 ? *reinterpret_cast<const uint4*>(xb + k) : none;
#pragma unroll
        for (int j = 0; j < 4; ++j) mma32(d[j], x0, x1, w[j]);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float* at = sm.part + (slice * kTile + g) * rp + rg * 32 + j * 8 + q * 2;
        *reinterpret_cast<float2*>(at) = make_float2(d[j][0], d[j][1]);
        *reinterpret_cast<float2*>(at + 8 * rp) = make_float2(d[j][2], d[j][3]);
      }
    }
    __syncthreads();
    const int piece = cta - owner((int64_t)t * nk, total, used);
    float* v = p.v + ((int64_t)piece * p.M + row0) * p.r;
    for (int i = tid; i < kTile * rp / 2; i += kThreads) {  // two ranks each
      const int m = sm.t.rows[2 * i / rp], k = 2 * i % rp;
      float2 s = make_float2(0.f, 0.f);
      for (int c = 0; c < slices; ++c) {
        const float2 u = *reinterpret_cast<const float2*>(sm.part + c * kTile * rp + 2 * i);
        s.x += u.x;
        s.y += u.y;
      }
      if (m >= 0 && k < p.r) *reinterpret_cast<float2*>(v + (int64_t)m * p.r + k) = s;
    }
    __syncthreads();
  }
}

template <bool F32>
__global__ void __launch_bounds__(kThreads, 2) adapter_few_up_kernel(Adapter p, int ctas) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  UpSmem& sm = *reinterpret_cast<UpSmem*>(smem_raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, q = lane & 3;
  const int chunk = blockIdx.x / ctas, cta = blockIdx.x - chunk * ctas;
  const int64_t row0 = (int64_t)chunk * kChunk;
  const int rows = p.M - row0 < kChunk ? (int)(p.M - row0) : kChunk;
  // The first kernel lets this one start when all before it is complete: what is not v can be read and
  // written already.
  make_tables(p, sm.t, row0, rows, false);
  const int nk = (p.K + 31) / 32, nb = (p.N + 31) / 32, used = down_ctas(sm.t.tiles, nk, ctas);
  const int64_t total = (int64_t)sm.t.tiles * nk;
  const int rp = (p.r + 31) / 32 * 32, vs = (kRankMost + 8) / 2, steps = (p.r + 15) / 16;
  Run run((int64_t)sm.t.tiles * nb, nb, cta, ctas);
  int t, b0, b1;
  {  // this CTA's parts of B on their way into L2
    Run ahead = run;
    while (ahead.next(t, b0, b1)) {
      const uint16_t* B = static_cast<const uint16_t*>(p.b) + ((int64_t)sm.t.id[sm.t.leader[t]] * p.N + b0 * 32) * p.r;
      const int64_t bytes = ((int64_t)min(b1 * 32, p.N) - b0 * 32) * p.r * 2;
      for (int64_t i = (int64_t)tid * 128; i < bytes; i += kThreads * 128) prefetch_l2(reinterpret_cast<const char*>(B) + i);
    }
  }
  // rows of requests without an adapter: base as it is
  if (p.base != p.out) {
    const int units = p.N / 8 * (F32 ? 2 : 1);
    for (int i = cta; i < rows; i += ctas)
      if (sm.t.id[i] == -1)
        for (int c = tid; c < units; c += kThreads) {
          const int64_t at = (row0 + i) * units + c;
          static_cast<uint4*>(p.out)[at] = p.base ? static_cast<const uint4*>(p.base)[at] : make_uint4(0, 0, 0, 0);
        }
  }
  moe::wait_for_stream();
  moe::let_next_start();
  while (run.next(t, b0, b1)) {
    const int id = tile_rows(sm.t, t);
    const uint16_t* B = static_cast<const uint16_t*>(p.b) + (int64_t)id * p.N * p.r;
    const int c0 = owner((int64_t)t * nk, total, used), pieces = owner((int64_t)(t + 1) * nk - 1, total, used) - c0 + 1;
    const float scale = p.scale ? p.scale[id] : 1.f;
    for (int i = tid; i < kTile * rp / 2; i += kThreads) {  // two ranks each
      const int j = 2 * i / rp, m = sm.t.rows[j], k = 2 * i % rp;
      float2 s = make_float2(0.f, 0.f);
      if (m >= 0 && k < p.r) {
        const float* v = p.v + (row0 + m) * p.r + k;
        for (int c = 0; c < pieces; ++c) {
          const float2 u = *reinterpret_cast<const float2*>(v + (int64_t)c * p.M * p.r);
          s.x += u.x;
          s.y += u.y;
        }
      }
      s.x *= scale;
      s.y *= scale;
      const __nv_bfloat162 hi = __floats2bfloat162_rn(s.x, s.y);
      const __nv_bfloat162 lo = __floats2bfloat162_rn(s.x - __low2float(hi), s.y - __high2float(hi));
      sm.vb[0][j * vs + k / 2] = *reinterpret_cast<const uint32_t*>(&hi);
      sm.vb[1][j * vs + k / 2] = *reinterpret_cast<const uint32_t*>(&lo);
    }
    __syncthreads();
    const int ra = sm.t.rows[g], rb = sm.t.rows[g + 8];
    // v B^T, 32 features at a time: feature 8 (c / 2) + 2 j + c % 2 is column c of product j, so that a
    // lane ends with eight neighbouring ones of its rows
    for (int b = b0 + warp; b < b1; b += kWarps) {
      float d[4][4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) d[j][i] = 0.f;
      const int f0 = b * 32 + 8 * (g >> 1) + (g & 1);
      for (int s = 0; s < steps; ++s) {
        const int k = s * 16 + q * 4;
        uint2 w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          w[j] = f0 + 2 * j < p.N && k < p.r ? moe::ldg_nc_u64(B + (int64_t)(f0 + 2 * j) * p.r + k) : make_uint2(0, 0);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint2 va = *reinterpret_cast<const uint2*>(&sm.vb[h][g * vs + k / 2]);
          const uint2 vc = *reinterpret_cast<const uint2*>(&sm.vb[h][(g + 8) * vs + k / 2]);
          const uint32_t a[4] = {va.x, vc.x, va.y, vc.y};
#pragma unroll
          for (int j = 0; j < 4; ++j) moe::mma_bf16(d[j], a, w[j].x, w[j].y, d[j]);
        }
      }
      const int n = b * 32 + 8 * q;
      if (n < p.N) {
        const float u[8] = {d[0][0], d[0][1], d[1][0], d[1][1], d[2][0], d[2][1], d[3][0], d[3][1]};
        const float v[8] = {d[0][2], d[0][3], d[1][2], d[1][3], d[2][2], d[2][3], d[3][2], d[3][3]};
        if (ra >= 0) add_to_base<F32>(p, (row0 + ra) * p.N + n, u);
        if (rb >= 0) add_to_base<F32>(p, (row0 + rb) * p.N + n, v);
      }
    }
    __syncthreads();
  }
}

constexpr int kCtasMost = 160;  // of a call, where its chunks are fewer

int64_t chunks_of(int64_t M) { return (M + kChunk - 1) / kChunk; }
int ctas_of(int64_t M, int sms) { return (int)std::max<int64_t>(1, std::min(sms, kCtasMost) / chunks_of(M)); }

}  // namespace

namespace moe_launch {

// v by row, as often as a tile has pieces at most.
size_t adapter_few_workspace_bytes(int64_t M, int r) {
  const int ctas = ctas_of(M, kCtasMost);
  return (size_t)std::min(kPieces, ctas) * M * r * 4;
}

cudaError_t adapter_few(const Adapter& p, cudaStream_t stream) {
  static std::atomic<uint64_t> done[3] = {};
  const auto up = p.out_f32 ? adapter_few_up_kernel<true> : adapter_few_up_kernel<false>;
  cudaError_t e = allow_smem((const void*)adapter_few_down_kernel, sizeof(DownSmem), done[0]);
  if (e == cudaSuccess) e = allow_smem((const void*)up, sizeof(UpSmem), done[1 + (p.out_f32 != 0)]);
  if (e != cudaSuccess) return e;
  const int ctas = ctas_of(p.M, sm_count_current());
  const dim3 grid((unsigned)(chunks_of(p.M) * ctas));
  e = launch_staged(adapter_few_down_kernel, grid, dim3(kThreads), sizeof(DownSmem), stream, 1, p, ctas);
  if (e != cudaSuccess) return e;
  return launch_staged(up, grid, dim3(kThreads), sizeof(UpSmem), stream, 1, p, ctas);
}

}  // namespace moe_launch
