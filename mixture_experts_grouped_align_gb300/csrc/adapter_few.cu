// Low-rank adapters of many requests beside a dense product: few rows a request.
//
//   out[m] = base[m] + scale[a] (x[m] A[a]^T) B[a]^T,  a the adapter of m's request
//
// Bound by the adapters' bytes: with few rows each of them is read for a handful of rows.  So rows
// are gathered by adapter, whatever their order: a block looks at 512 rows, finds each one's
// occurrence among the rows of its adapter, and every sixteenth is the first of a tile of up to
// sixteen rows of one adapter, the rows of an m16n8k16 MMA.  (250 rows over five adapters are 20
// tiles, and not 250 readings of an adapter.)  A tile belongs to a cluster of up to eight CTAs:
//   v = x A^T   K is split over the cluster and over the warps; the shares are added in order through
//               shared memory and then distributed shared memory;
//   v B^T       each CTA takes its share of the features, whose part of B it has brought into L2
//               meanwhile.
// The operands of an MMA are read from global memory in their own layout, 16 or 8 bytes a lane: the
// order of K within the products is the lanes', for both operands alike.  v is fp32 and enters the
// second product as two bf16 numbers, 2^-17 of itself off.  Rows are never in one accumulator with
// another adapter's: a request's weights that are not finite stay its own.
#include <algorithm>

#include "moe_common.cuh"
#include "moe_launch.h"
#include "tcgen05.cuh"

namespace {

using moe_launch::Adapter;

constexpr int kThreads = 512, kWarps = 16;
constexpr int kChunk = 512;   // rows that a block looks at
constexpr int kTile = 16;     // rows of a tile
constexpr int kRankMost = 128;
constexpr unsigned kAll = 0xffffffffu;

struct Smem {
  alignas(16) int32_t id[kChunk];  // a row's adapter, -1: none, -2: of no request
  int16_t occ[kChunk];       // rows of its adapter before it
  int16_t leader[kChunk];    // first rows of the tiles
  int32_t start[kChunk];     // the last request that starts at a row, -1: none
  int32_t start_id[kChunk];  // its adapter and its end
  int32_t start_end[kChunk];
  int32_t warp_sum[kWarps];
  int32_t tiles;
  int32_t rows[kTile];
  // read and written 8 or 16 bytes at a time
  alignas(16) float part[kWarps * kTile * 32];             // shares of v: [slice][row][rank]
  alignas(16) float v[2][kTile * kRankMost];               // this CTA's share, two tiles in turn
  alignas(16) uint32_t vb[2][kTile * (kRankMost + 8) / 2]; // v as bf16, high and low parts: [row][rank], rows 8 ranks apart
};

MOE_DEV void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// A K step of 32: this lane's eight values of two x rows and of a weight row each.
MOE_DEV void mma32(float (&d)[4], const uint4& x0, const uint4& x1, const uint4& w) {
  const uint32_t a[4] = {x0.x, x1.x, x0.y, x1.y}, b[4] = {x0.z, x1.z, x0.w, x1.w};
  moe::mma_bf16(d, a, w.x, w.y, d);
  moe::mma_bf16(d, b, w.z, w.w, d);
}

// The chunk's rows: adapters, occurrences and tiles.
__device__ __forceinline__ void make_tables(const Adapter& p, Smem& sm, int64_t row0, int rows) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // Where a request starts in the chunk, or -1.  Of several at one place (offsets that decrease) the last
  // is taken, by every CTA: they meet in the barriers of the same tiles.
  const auto place = [&](int i, int& end, int& id) {
    const int64_t lo = p.row_offsets[i], hi = p.row_offsets[i + 1];
    id = p.adapter[i];
    end = (int)(hi - row0 < rows ? hi - row0 : rows);
    const bool bounds = lo >= 0 && lo <= hi && hi <= p.M, known = id >= -1 && id < p.L;
    if (blockIdx.x == 0 && !(bounds && known)) moe::set_status(p.status, bounds ? MOE_ERR_INVALID_EXPERT : MOE_ERR_CAPACITY);
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

template <bool F32>
__global__ void __launch_bounds__(kThreads) adapter_few_kernel(Adapter p, int C, int clusters) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  Smem& sm = *reinterpret_cast<Smem*>(smem_raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, q = lane & 3;
  const int rank = C > 1 ? (int)tc::cluster_ctarank() : 0;
  const int cluster = blockIdx.x / C, chunk = cluster / clusters, mine = cluster - chunk * clusters;
  const int64_t row0 = (int64_t)chunk * kChunk;
  const int rows = p.M - row0 < kChunk ? (int)(p.M - row0) : kChunk;
  moe::wait_for_stream();
  moe::let_next_start();
  make_tables(p, sm, row0, rows);

  const int nk = (p.K + 31) / 32, nb = (p.N + 31) / 32;
  const int k0 = (int)((int64_t)nk * rank / C), k1 = (int)((int64_t)nk * (rank + 1) / C);
  const int b0 = (int)((int64_t)nb * rank / C), b1 = (int)((int64_t)nb * (rank + 1) / C);
  const int groups = (p.r + 31) / 32;  // of 32 ranks
  const int slices = kWarps / groups, rg = warp % groups, slice = warp / groups;
  const int rp = groups * 32, vs = (kRankMost + 8) / 2;
  const int steps = (p.r + 15) / 16;
  const uint16_t* x = static_cast<const uint16_t*>(p.x);

  // rows of requests without an adapter: base as it is
  if (p.base != p.out) {
    const int size = F32 ? 32 : 16;  // of eight features
    const int first = b0 * 4 * (size / 16), units = std::min(b1 * 4, p.N / 8) * (size / 16) - first;
    for (int i = mine; i < rows; i += clusters)
      if (sm.id[i] == -1) {
        const int64_t at = (row0 + i) * (p.N / 8) * (size / 16) + first;
        for (int c = tid; c < units; c += kThreads)
          static_cast<uint4*>(p.out)[at + c] = p.base ? static_cast<const uint4*>(p.base)[at + c] : make_uint4(0, 0, 0, 0);
      }
  }
  int turn = 0;
  for (int t = mine; t < sm.tiles; t += clusters, turn ^= 1) {
    const int lead = sm.leader[t], id = sm.id[lead], from = sm.occ[lead];
    if (tid < kTile) sm.rows[tid] = -1;
    __syncthreads();
    if (sm.id[tid] == id && sm.occ[tid] >= from && sm.occ[tid] < from + kTile) sm.rows[sm.occ[tid] - from] = tid;
    __syncthreads();
    const uint16_t* A = static_cast<const uint16_t*>(p.a) + (int64_t)id * p.r * p.K;
    const uint16_t* B = static_cast<const uint16_t*>(p.b) + (int64_t)id * p.N * p.r;
    const int ra = sm.rows[g], rb = sm.rows[g + 8];
    {  // this CTA's part of B on its way into L2
      const char* lo = reinterpret_cast<const char*>(B + (int64_t)b0 * 32 * p.r);
      const int64_t bytes = ((int64_t)std::min(b1 * 32, p.N) - b0 * 32) * p.r * 2;
      for (int64_t i = (int64_t)tid * 128; i < bytes; i += kThreads * 128) prefetch_l2(lo + i);
    }
    // v = x A^T over this CTA's K
    if (slice < slices) {
      float d[4][4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) d[j][i] = 0.f;
      const uint4 none = make_uint4(0, 0, 0, 0);
      const uint16_t* xa = x + (row0 + (ra < 0 ? 0 : ra)) * p.K;
      const uint16_t* xb = x + (row0 + (rb < 0 ? 0 : rb)) * p.K;
      constexpr int kU = 2;
      for (int kc = k0 + slice; kc < k1; kc += kU * slices) {
        uint4 x0[kU], x1[kU], w[kU][4];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          const int c = kc + u * slices, k = c * 32 + q * 8;
          const bool on = c < k1 && k < p.K;
          x0[u] = on && ra >= 0 ? *reinterpret_cast<const uint4*>(xa + k) : none;
          x1[u] = on && rb >= 0 ? *reinterpret_cast<const uint4*>(xb + k) : none;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int n = rg * 32 + j * 8 + g;
            w[u][j] = on && n < p.r ? moe::ldg_nc_u128(A + (int64_t)n * p.K + k) : none;
          }
        }
#pragma unroll
        for (int u = 0; u < kU; ++u)
#pragma unroll
          for (int j = 0; j < 4; ++j) mma32(d[j], x0[u], x1[u], w[u][j]);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float* at = sm.part + (slice * kTile + g) * rp + rg * 32 + j * 8 + q * 2;
        *reinterpret_cast<float2*>(at) = make_float2(d[j][0], d[j][1]);
        *reinterpret_cast<float2*>(at + 8 * rp) = make_float2(d[j][2], d[j][3]);
      }
    }
    __syncthreads();
    for (int i = tid; i < kTile * rp; i += kThreads) {
      float s = 0.f;
      for (int k = 0; k < slices; ++k) s += sm.part[k * kTile * rp + i];
      sm.v[turn][i] = s;
    }
    if (C > 1) tc::cluster_sync();
    else __syncthreads();
    const float scale = p.scale ? p.scale[id] : 1.f;
    for (int i = tid; i < kTile * rp / 2; i += kThreads) {  // two ranks each
      const uint32_t at = tc::smem_addr(&sm.v[turn][2 * i]);
      float2 s = make_float2(0.f, 0.f);
      for (int c = 0; c < C; ++c) {
        uint32_t a = at;
        float2 v;
        if (C > 1) asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(at), "r"(c));
        if (C > 1) asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a) : "memory");
        else v = *reinterpret_cast<const float2*>(&sm.v[turn][2 * i]);
        s.x += v.x;
        s.y += v.y;
      }
      s.x *= scale;
      s.y *= scale;
      const __nv_bfloat162 hi = __floats2bfloat162_rn(s.x, s.y);
      const __nv_bfloat162 lo = __floats2bfloat162_rn(s.x - __low2float(hi), s.y - __high2float(hi));
      const int m = 2 * i / rp, k = 2 * i % rp;
      sm.vb[0][m * vs + k / 2] = *reinterpret_cast<const uint32_t*>(&hi);
      sm.vb[1][m * vs + k / 2] = *reinterpret_cast<const uint32_t*>(&lo);
    }
    __syncthreads();
    // v B^T over this CTA's features, 32 at a time: feature 8 (c / 2) + 2 j + c % 2 is column c of
    // product j, so that a lane ends with eight neighbouring ones of its rows
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
  if (C > 1) tc::cluster_sync();  // no CTA leaves while another reads its share
}

}  // namespace

namespace moe_launch {

cudaError_t adapter_few(const Adapter& p, cudaStream_t stream) {
  static std::atomic<uint64_t> done[2] = {};
  const auto kern = p.out_f32 ? adapter_few_kernel<true> : adapter_few_kernel<false>;
  const cudaError_t e = allow_smem((const void*)kern, sizeof(Smem), done[p.out_f32 != 0]);
  if (e != cudaSuccess) return e;
  const int C = 8;
  const int64_t chunks = (p.M + kChunk - 1) / kChunk;
  // two CTAs fit an SM; a chunk has at most as many tiles as rows
  const int64_t at_once = std::max<int64_t>(1, 2 * (int64_t)sm_count_current() / C / chunks);
  const int clusters = (int)std::min<int64_t>(std::min<int64_t>(p.M, kChunk), at_once);
  return launch_staged(kern, dim3((unsigned)(chunks * clusters * C)), dim3(kThreads), sizeof(Smem), stream, C, p, C, clusters);
}

}  // namespace moe_launch
