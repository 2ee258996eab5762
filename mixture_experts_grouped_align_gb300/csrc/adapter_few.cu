// Low-rank adapters of many requests beside a dense product: few rows a request.
//
//   out[m] = base[m] + scale[a] (x[m] A[a]^T) B[a]^T,  a the adapter of m's request
//
// Bound by the adapters' bytes: with few rows each of them is read for a handful of rows.  So rows
// are gathered by adapter, whatever their order: a block looks at 256 rows, finds each one's
// occurrence among the rows of its adapter, and every sixteenth is the first of a tile of up to
// sixteen rows of one adapter, the rows of an m16n8k16 MMA.  (250 rows over five adapters are 20
// tiles, and not 250 readings of an adapter.)  Two kernels, v = x A^T and out = base + v B^T; in each
// the CTAs share the tiles' blocks of K, or of features, so that one tile and 200 alike use many SMs.
// A tile's pieces of v are added in order by those who read them.  The second kernel starts under the
// first one: its tables, the rows without an adapter and the way of B and base into shared memory and
// L2 do not wait for v.
// The operands of an MMA are read from global memory in their own layout, 16 or 8 bytes a lane: the
// order of K within the products is the lanes', for both operands alike.  v is fp32 and enters the
// second product as a sum of bf16 numbers: two, 2^-17 of itself off, or three for fp32 outputs.  Rows
// are never in one accumulator with another adapter's: a request's weights that are not finite stay its
// own.
// Measured (replayed graphs, us): one token of rank 16, 2880 -> 2880: 6.2; 64 tokens over 100 adapters of
// rank 16, 2880 -> 5760: 10.5 (19.5 MB; 11.7 from HBM); 250 rows over five adapters of rank 64, 7168 ->
// 4096: 13.1 (14.5).  Not the bytes bound these but the chain: the launch, the tables (1.3), the first loads
// of A (2.5), the pieces' sum and its way to the second kernel (1.7), the products and stores.  In one
// kernel of clusters, which wait for the slowest piece in place of the launch, they took 7.4, 31 and 29.
#include <algorithm>

#include "cp_async.cuh"
#include "moe_launch.h"

namespace {

using moe_launch::Adapter;

constexpr int kThreads = 256, kWarps = 8;       // of the first kernel
constexpr int kUpThreads = 512, kUpWarps = 16;  // of the second
constexpr int kChunk = 256;                     // rows that a block looks at
constexpr int kSlotBits = 9, kSlots = 1 << kSlotBits;  // twice the rows: a free place is near
constexpr int kTile = 16;     // rows of a tile
constexpr int kFewest = 4;    // rows of a tile that the second kernel takes without the tensor cores
constexpr int kRankMost = 128;
constexpr unsigned kAll = 0xffffffffu;

struct Rows {
  alignas(16) int32_t id[kChunk];  // a row's adapter, -1: none, -2: of no request
  int16_t occ[kChunk];       // rows of its adapter before it
  int16_t leader[kChunk];    // first rows of the tiles
  int32_t slot_id[kSlots];   // adapters of the chunk's rows, hashed; -1: free
  // an adapter's rows; later the first kernel's shares of v, and the second's operands
  alignas(16) uint32_t slot_rows[kSlots][kChunk / 32];
  int32_t start[kChunk];     // the last request that starts at a row, -1: none
  int32_t start_id[kChunk];  // its adapter and its end
  int32_t start_end[kChunk];
  int32_t warp_sum[kChunk / 32], lead_sum[kChunk / 32];
  int32_t tiles;
  int32_t rows[kTile];       // of the tile at hand
};
// Read and written 8 or 16 bytes at a time, after the tables are made.
constexpr int kVs = (kRankMost + 8) / 2;  // words of a row of v's bf16 parts
struct DownSmem {
  Rows t;
  MOE_DEV float* part() { return reinterpret_cast<float*>(t.slot_rows); }  // shares of v: [slice][row][rank]
};
static_assert(sizeof(Rows::slot_rows) >= kWarps * kTile * 32 * 4 && sizeof(Rows::slot_rows) >= 3 * kTile * kVs * 4, "");
// What a thread of the second kernel reads first of B and of base is copied into shared memory while the
// first kernel still runs, in places of its own, so that no thread waits for another's copies: 64 bytes of
// B (32 for fp32 outputs), and of base what it adds to in its first block of features.
template <bool F32>
struct UpSmem {
  Rows t;
  static constexpr int kAhead = F32 ? 2 : 4;  // of 16 bytes
  alignas(16) uint8_t b[kAhead * kUpThreads * 16];
  alignas(16) uint8_t base[(F32 ? 4 : 2) * kUpThreads * 16];
  // v's h-th bf16 parts: [row][rank], rows 8 ranks apart
  MOE_DEV uint32_t* vb(int h) { return &t.slot_rows[0][0] + h * kTile * kVs; }
  // the i-th place of n bytes of this thread
  static MOE_DEV uint8_t* place(uint8_t* mem, int i, int n) { return mem + (i * kUpThreads + (int)threadIdx.x) * n; }
};

// Equal shares of the tiles' blocks for the CTAs of a chunk.  Up to as many tiles as CTAs: `parts` CTAs a
// tile, a piece of one tile each, as every further piece costs a CTA the latency of its first loads (64
// tokens over 100 adapters: 3.2 us of loads for two pieces, 1.6 for one).  More tiles: whole ones in turn, or
// up to four pieces of each where that fills the last turn better; a block of 32 takes a CTA about 2.3 ns a
// rank, and a piece 1500 ns more (500 rows over 150 adapters of rank 64, 4096 -> 4096: 102 us in whole tiles,
// 86; 2000 rows of 100 requests over 8 of rank 16 39 and 35).
constexpr int kPieces = 32;
struct Share {
  int tiles, blocks, parts, cta, ctas;
  MOE_DEV Share(int tiles, int blocks, int most, int r, int cta, int ctas) : tiles(tiles), blocks(blocks), parts(1), cta(cta), ctas(ctas) {
    if (tiles <= ctas) {
      if (tiles) parts = max(1, min(min(most, blocks), ctas / tiles));
      return;
    }
    // in integers, as both kernels have to find the same; `parts` pieces where they save 4 per cent
    const int tile = 23 * min(blocks, 4096) / 10 * r, whole = tiles / ctas, rest = tiles - whole * ctas;
    int least = (whole + (rest > 0)) * ((tile + 1500) / 25 * 24);
#pragma unroll
    for (int n = 2; n <= 4; ++n) {
      if (n > most || n > blocks || n > ctas) break;
      const int turns = n * whole + (n * rest > 0) + (n * rest > ctas) + (n * rest > 2 * ctas) + (n * rest > 3 * ctas);
      const int time = turns * (tile / n + 1500);
      if (time < least) {
        least = time;
        parts = n;
      }
    }
  }
  // The n-th piece of this CTA: its tile, its number among the tile's, and its blocks.
  MOE_DEV bool get(int n, int& tile, int& part, int& b0, int& b1) const {
    const int i = cta + n * ctas;
    if (i >= tiles * parts) return false;
    tile = parts > 1 ? i / parts : i;
    part = i - tile * parts;
    b0 = (int)((int64_t)blocks * part / parts);
    b1 = (int)((int64_t)blocks * (part + 1) / parts);
    return true;
  }
};

MOE_DEV void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// A K step of 32: this lane's eight values of two x rows and of a weight row each.
MOE_DEV void mma32(float (&d)[4], const uint4& x0, const uint4& x1, const uint4& w) {
  const uint32_t a[4] = {x0.x, x1.x, x0.y, x1.y}, b[4] = {x0.z, x1.z, x0.w, x1.w};
  moe::mma_bf16(d, a, w.x, w.y, d);
  moe::mma_bf16(d, b, w.z, w.w, d);
}

// What make_tables wants to find.
__device__ __forceinline__ void clear_tables(Rows& sm) {
  for (int i = threadIdx.x; i < kSlots; i += blockDim.x) sm.slot_id[i] = -1;
  for (int i = threadIdx.x; i < kSlots * kChunk / 32; i += blockDim.x) (&sm.slot_rows[0][0])[i] = 0;
  if (threadIdx.x < kChunk) sm.start[threadIdx.x] = -1;
}

// The chunk's rows: adapters, occurrences and tiles, after clear_tables and a barrier.  Every thread calls,
// the first kChunk of them have a row.
__device__ __forceinline__ void make_tables(const Adapter& p, Rows& sm, int64_t row0, int rows, bool report) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool mine = tid < kChunk;
  // Where a request starts in the chunk, or -1.  Of several at one place (offsets that decrease) the last
  // is taken, by every CTA and in both kernels.
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
  int first_end = 0, first_id = 0, end, id_of;
  const int first_at = mine && tid < p.R ? place(tid, first_end, first_id) : -1;  // most calls have no more requests
  if (first_at >= 0) atomicMax(&sm.start[first_at], tid);
  for (int i = kChunk + tid; i < p.R; i += blockDim.x) {
    const int at = place(i, end, id_of);
    if (at >= 0) atomicMax(&sm.start[at], i);
  }
  __syncthreads();
  if (first_at >= 0 && sm.start[first_at] == tid) {
    sm.start_id[first_at] = first_id;
    sm.start_end[first_at] = first_end;
  }
  for (int i = kChunk + tid; i < p.R; i += blockDim.x) {
    const int at = place(i, end, id_of);
    if (at >= 0 && sm.start[at] == i) {
      sm.start_id[at] = id_of;
      sm.start_end[at] = end;
    }
  }
  // the request of a row is the last that starts at or before it
  int at = mine && sm.start[tid] >= 0 ? tid : -1;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int up = __shfl_up_sync(kAll, at, o);
    if (lane >= o && up > at) at = up;
  }
  if (mine && lane == 31) sm.warp_sum[warp] = at;
  __syncthreads();
  int id = -2;
  if (mine) {
    const int before = lane < warp ? sm.warp_sum[lane] : -1;
    at = max(at, __reduce_max_sync(kAll, before));
    if (tid < rows && at >= 0 && tid < sm.start_end[at]) id = sm.start_id[at];
    sm.id[tid] = id;
  }
  // an adapter's rows as bits, in a place of its own in a table: its occurrence is the bits before a row's
  int place_of = 0;
  if (id >= 0) {
    place_of = (int)(((uint32_t)id * 2654435769u) >> (32 - kSlotBits));
    for (int old; (old = atomicCAS(&sm.slot_id[place_of], -1, id)) != -1 && old != id;) place_of = (place_of + 1) & (kSlots - 1);
    atomicOr(&sm.slot_rows[place_of][warp], 1u << lane);
  }
  __syncthreads();
  unsigned leads = 0;
  if (mine) {
    int occ = 0;
    if (id >= 0)
#pragma unroll
      for (int w = 0; w < kChunk / 32; ++w) {
        const uint32_t bits = sm.slot_rows[place_of][w];
        occ += __popc(w < warp ? bits : w == warp ? bits & ((1u << lane) - 1) : 0u);
      }
    sm.occ[tid] = (int16_t)occ;
    leads = __ballot_sync(kAll, id >= 0 && occ % kTile == 0);
    if (lane == 0) sm.lead_sum[warp] = __popc(leads);
  }
  __syncthreads();
  if (mine) {
    const int n = lane < kChunk / 32 ? sm.lead_sum[lane] : 0;
    const int before = __reduce_add_sync(kAll, lane < warp ? n : 0), all = __reduce_add_sync(kAll, n);
    if (leads >> lane & 1) sm.leader[before + __popc(leads & ((1u << lane) - 1))] = (int16_t)tid;
    if (tid == 0) sm.tiles = all;
  }
  __syncthreads();
}

// Eight features of a row.
template <bool F32>
struct Out8 {
  uint4 v[F32 ? 2 : 1];
  MOE_DEV void load(const void* base, int64_t at, bool on) {
#pragma unroll
    for (int i = 0; i < (F32 ? 2 : 1); ++i)
      v[i] = on && base ? static_cast<const uint4*>(base)[at / 8 * (F32 ? 2 : 1) + i] : make_uint4(0, 0, 0, 0);
  }
  // The same by way of shared memory, piece i of its places.
  static MOE_DEV void fetch(UpSmem<F32>& sm, int i, const void* base, int64_t at) {
#pragma unroll
    for (int j = 0; j < (F32 ? 2 : 1); ++j)
      cpa::cp_async16(tc::smem_addr(sm.place(sm.base, i * (F32 ? 2 : 1) + j, 16)),
                      static_cast<const uint4*>(base) + at / 8 * (F32 ? 2 : 1) + j);
  }
  MOE_DEV void take(UpSmem<F32>& sm, int i, bool on) {
#pragma unroll
    for (int j = 0; j < (F32 ? 2 : 1); ++j)
      v[j] = on ? *reinterpret_cast<const uint4*>(sm.place(sm.base, i * (F32 ? 2 : 1) + j, 16)) : make_uint4(0, 0, 0, 0);
  }
  MOE_DEV void add_and_store(void* out, int64_t at, const float (&f)[8]) const {
    uint32_t w[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[F32].x, v[F32].y, v[F32].z, v[F32].w};
    uint4* o = static_cast<uint4*>(out) + at / 8 * (F32 ? 2 : 1);
    if (F32) {
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(__uint_as_float(w[i]) + f[i]);
      o[0] = make_uint4(w[0], w[1], w[2], w[3]);
      o[F32] = make_uint4(w[4], w[5], w[6], w[7]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 s = __floats2bfloat162_rn(__uint_as_float(w[i] << 16) + f[2 * i],
                                                       __uint_as_float(w[i] & 0xffff0000u) + f[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&s);
      }
      o[0] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
};

// The rows of tile t, -1 where it has fewer than sixteen; every thread calls.
__device__ __forceinline__ int tile_rows(Rows& sm, int t) {
  const int tid = threadIdx.x, lead = sm.leader[t], id = sm.id[lead], from = sm.occ[lead];
  __syncthreads();  // the rows of the tile before have been read
  if (tid < kTile) sm.rows[tid] = -1;
  __syncthreads();
  if (tid < kChunk && sm.id[tid] == id && sm.occ[tid] >= from && sm.occ[tid] < from + kTile) sm.rows[sm.occ[tid] - from] = tid;
  __syncthreads();
  return id;
}

// blockIdx.x: a chunk of 256 rows, a CTA of the chunk's.  A warp takes NJ eights of ranks and a share of
// the run's blocks, U of them at once: what the loads in flight take of registers is what the run's time
// goes by (512 threads of one block at a time: 250 rows of rank 64 over five adapters 23 us).
template <int NJ, int U>
__global__ void __launch_bounds__(kThreads, 2) adapter_few_down_kernel(Adapter p, int ctas) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  DownSmem& sm = *reinterpret_cast<DownSmem*>(smem_raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, q = lane & 3;
  const int chunk = blockIdx.x / ctas, cta = blockIdx.x - chunk * ctas;
  const int64_t row0 = (int64_t)chunk * kChunk;
  const int rows = p.M - row0 < kChunk ? (int)(p.M - row0) : kChunk;
  clear_tables(sm.t);
  __syncthreads();
  moe::wait_for_stream();
  moe::let_next_start();
  make_tables(p, sm.t, row0, rows, blockIdx.x == 0);

  const int nk = (p.K + 31) / 32;
  const Share share(sm.t.tiles, nk, kPieces, p.r, cta, ctas);
  const int groups = (p.r + 8 * NJ - 1) / (8 * NJ);
  const int slices = kWarps / groups, rg = warp % groups, slice = warp / groups, rp = groups * 8 * NJ;
  const uint16_t* x = static_cast<const uint16_t*>(p.x);
  int t, part, k0, k1;
  for (int turn = 0; share.get(turn, t, part, k0, k1); ++turn) {
    int t1, part1, l0, l1;
    if (share.get(turn + 1, t1, part1, l0, l1)) {  // the next piece's A on its way into L2 meanwhile
      const char* A = reinterpret_cast<const char*>(static_cast<const uint16_t*>(p.a) + (int64_t)sm.t.id[sm.t.leader[t1]] * p.r * p.K);
      const int first = l0 * 64, bytes = min(l1 * 64, p.K * 2) - first, lines = (bytes + 127) / 128;
      for (int i = tid; i < p.r * lines; i += kThreads) prefetch_l2(A + (int64_t)(i / lines) * p.K * 2 + first + i % lines * 128);
    }
    const int id = tile_rows(sm.t, t);
    const uint16_t* A = static_cast<const uint16_t*>(p.a) + (int64_t)id * p.r * p.K;
    if (slice < slices) {
      const int ra = sm.t.rows[g], rb = sm.t.rows[g + 8];
      float d[NJ][4];
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) d[j][i] = 0.f;
      const uint4 none = make_uint4(0, 0, 0, 0);
      const uint16_t* xa = x + (row0 + (ra < 0 ? 0 : ra)) * p.K;
      const uint16_t* xb = x + (row0 + (rb < 0 ? 0 : rb)) * p.K;
      const uint16_t* wa = A + (int64_t)(rg * 8 * NJ + g) * p.K;
      for (int c = k0 + slice; c < k1; c += U * slices) {
        uint4 w[U][NJ], x0[U], x1[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int k = (c + u * slices) * 32 + q * 8;
          const bool on = c + u * slices < k1 && k < p.K;
#pragma unroll
          for (int j = 0; j < NJ; ++j)
            w[u][j] = on && rg * 8 * NJ + j * 8 + g < p.r ? moe::ldg_nc_u128(wa + (int64_t)j * 8 * p.K + k) : none;
          x0[u] = on && ra >= 0 ? moe::ldg_nc_u128(xa + k) : none;
          x1[u] = on && rb >= 0 ? moe::ldg_nc_u128(xb + k) : none;
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int j = 0; j < NJ; ++j) mma32(d[j], x0[u], x1[u], w[u][j]);
      }
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        float* at = sm.part() + (slice * kTile + g) * rp + (rg * NJ + j) * 8 + q * 2;
        *reinterpret_cast<float2*>(at) = make_float2(d[j][0], d[j][1]);
        *reinterpret_cast<float2*>(at + 8 * rp) = make_float2(d[j][2], d[j][3]);
      }
    }
    __syncthreads();
    float* v = p.v + ((int64_t)part * p.M + row0) * p.r;
    for (int i = tid; i < kTile * rp / 2; i += kThreads) {  // two ranks each
      const int m = sm.t.rows[2 * i / rp], k = 2 * i % rp;
      float2 s = make_float2(0.f, 0.f);
      for (int c = 0; c < slices; ++c) {
        const float2 u = *reinterpret_cast<const float2*>(sm.part() + c * kTile * rp + 2 * i);
        s.x += u.x;
        s.y += u.y;
      }
      if (m >= 0 && k < p.r) *reinterpret_cast<float2*>(v + (int64_t)m * p.r + k) = s;
    }
    __syncthreads();
  }
}

// The sum of a row's pieces of v, four ranks, in the order of the pieces.
MOE_DEV float4 pieces_of(const Adapter& p, int64_t row, int k, int from, int step, int pieces) {
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  const float* v = p.v + row * p.r + k;
  for (int c0 = from; c0 < pieces; c0 += 8 * step) {
    float4 u[8];
#pragma unroll
    for (int c = 0; c < 8; ++c)
      u[c] = c0 + c * step < pieces ? *reinterpret_cast<const float4*>(v + (int64_t)(c0 + c * step) * p.M * p.r)
                                    : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      s.x += u[c].x;
      s.y += u[c].y;
      s.z += u[c].z;
      s.w += u[c].w;
    }
  }
  return s;
}

// The tile's v times the scale as PARTS bf16 numbers: four ranks to a lane, or to 2 or 4 lanes with every
// second or fourth piece, as many as fill the block.  lr: log2 of the ranks, rounded up.
template <int PARTS, bool F32>
__device__ __forceinline__ void sum_pieces(const Adapter& p, UpSmem<F32>& sm, int64_t row0, int pieces, int lr, float scale) {
  const int by = 128 >> lr, mine = threadIdx.x & (by - 1), i = threadIdx.x >> (7 - lr);
  const int j = 4 * i >> lr, m = sm.t.rows[j], k = 4 * i & ((1 << lr) - 1);
  float4 s = m >= 0 && k < p.r ? pieces_of(p, row0 + m, k, mine, by, pieces) : make_float4(0.f, 0.f, 0.f, 0.f);
  for (int o = 1; o < by; o <<= 1) {
    s.x += __shfl_xor_sync(kAll, s.x, o);
    s.y += __shfl_xor_sync(kAll, s.y, o);
    s.z += __shfl_xor_sync(kAll, s.z, o);
    s.w += __shfl_xor_sync(kAll, s.w, o);
  }
  if (mine == 0) {
    float f[4] = {s.x * scale, s.y * scale, s.z * scale, s.w * scale};
    uint32_t w[PARTS][2];
    moe::split_bf16_any<PARTS>(f, w);
#pragma unroll
    for (int h = 0; h < PARTS; ++h) *reinterpret_cast<uint2*>(sm.vb(h) + j * kVs + k / 2) = make_uint2(w[h][0], w[h][1]);
  }
}

// A tile of up to kFewest rows, without the tensor cores: a lane has two neighbouring features at a time,
// whose weights it reads whole, and multiplies them with v in fp32.  Most of a tile of sixteen rows would
// be empty, and what an MMA wants around it is five times the instructions (64 tokens over 100 adapters:
// 0.9 us for 32 features of each warp).  Where the features leave most threads without any, four or eight lanes
// share two of them, every eight ranks another lane (one row of rank 128, 928 -> 4104: 9.9 us without, 7.5; with
// ranks below 64, or two lanes a pair, no gain: 6.2 and 6.4 for rank 16, 10.3 and 11.4 for 8 rows of rank 64).  16 bytes of B are number 2 (pair * eights + eight) +
// feature of the thread's.
template <bool SHARED>
struct Lanes {
  int log, first, step;  // of a pair of features; this thread's first feature, and how far its next one is
  MOE_DEV Lanes(int n0, int n1, int r) {
    const int pairs = (n1 - n0) / 2;
    log = !SHARED || r < 64 ? 0 : pairs <= kUpThreads / 8 ? 3 : pairs <= kUpThreads / 4 ? 2 : 0;
    first = n0 + 2 * ((int)threadIdx.x >> log);
    step = 2 * (kUpThreads >> log);
  }
  MOE_DEV int rank() const { return SHARED ? ((int)threadIdx.x & ((1 << log) - 1)) * 8 : 0; }
};

template <bool F32, bool SHARED>
__device__ __forceinline__ void fetch_few(const Adapter& p, UpSmem<F32>& sm, int id, int64_t row0, int n0, int n1) {
  constexpr int kSize = F32 ? 8 : 4, kAhead = UpSmem<F32>::kAhead;  // bytes of a pair of base
  const uint16_t* B = static_cast<const uint16_t*>(p.b) + (int64_t)id * p.N * p.r;
  const Lanes<SHARED> lanes(n0, n1, p.r);
  for (int i = 0, k = lanes.rank(), n = lanes.first; i < kAhead && n < n1; i += 2) {
    if (k < p.r) {
      cpa::cp_async16(tc::smem_addr(sm.place(sm.b, i, 16)), B + (int64_t)n * p.r + k);
      cpa::cp_async16(tc::smem_addr(sm.place(sm.b, i + 1, 16)), B + (int64_t)(n + 1) * p.r + k);
    }
    if ((k += 8 << lanes.log) >= p.r) {
      k = lanes.rank();
      n += lanes.step;
    }
  }
  if (!p.base || lanes.rank() > 0) return;  // the first lane stores the sums
  for (int u = 0, n = lanes.first; u < 2 && n < n1; ++u, n += lanes.step)
    for (int j = 0; j < kFewest; ++j) {
      const int m = sm.t.rows[j];
      if (m < 0) break;
      const char* from = static_cast<const char*>(p.base) + ((row0 + m) * p.N + n) * (kSize / 2);
      const uint32_t to = tc::smem_addr(sm.place(sm.base, u * kFewest + j, kSize));
      if (F32) cpa::cp_async8(to, from);
      else cpa::cp_async4(to, from);
    }
}

template <bool F32, bool SHARED>
__device__ __forceinline__ void few_rows(const Adapter& p, UpSmem<F32>& sm, int id, int64_t row0, int n0, int n1, int pieces, int lr,
                                         float scale) {
  constexpr int kAhead = UpSmem<F32>::kAhead;
  const int tid = threadIdx.x;
  float* v = reinterpret_cast<float*>(sm.vb(0));  // [row][rank] in fp32
  {
    const int i = tid >> 2, j = 4 * i >> lr, k = 4 * i & ((1 << lr) - 1);  // four lanes a sum
    const int m = j < kFewest ? sm.t.rows[j] : -1;
    float4 s = m >= 0 && k < p.r ? pieces_of(p, row0 + m, k, tid & 3, 4, pieces) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      s.x += __shfl_xor_sync(kAll, s.x, o);
      s.y += __shfl_xor_sync(kAll, s.y, o);
      s.z += __shfl_xor_sync(kAll, s.z, o);
      s.w += __shfl_xor_sync(kAll, s.w, o);
    }
    if ((tid & 3) == 0 && j < kFewest)
      reinterpret_cast<float4*>(v)[i] = make_float4(s.x * scale, s.y * scale, s.z * scale, s.w * scale);
  }
  cpa::cp_async_wait_all();
  __syncthreads();
  int rows = 0;
#pragma unroll
  for (int j = 0; j < kFewest; ++j) rows += sm.t.rows[j] >= 0;
  const uint16_t* B = static_cast<const uint16_t*>(p.b) + (int64_t)id * p.N * p.r;
  const Lanes<SHARED> lanes(n0, n1, p.r);
  const unsigned together = ((1u << (1 << lanes.log)) - 1) << (tid & 31 & -(1 << lanes.log));
  for (int n = lanes.first, u = 0, i = 0; n < n1; n += lanes.step, ++u) {
    float d[kFewest][2];
#pragma unroll
    for (int j = 0; j < kFewest; ++j) d[j][0] = d[j][1] = 0.f;
    for (int k = lanes.rank(); k < p.r; k += 8 << lanes.log, i += 2) {
      uint4 w[2];
#pragma unroll
      for (int h = 0; h < 2; ++h)
        w[h] = i < kAhead ? *reinterpret_cast<const uint4*>(sm.place(sm.b, i + h, 16)) : moe::ldg_nc_u128(B + (int64_t)(n + h) * p.r + k);
#pragma unroll
      for (int j = 0; j < kFewest; ++j) {
        if (j >= rows) break;
        const float4 e = *reinterpret_cast<const float4*>(v + (j << lr) + k);
        const float4 f = *reinterpret_cast<const float4*>(v + (j << lr) + k + 4);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          d[j][h] = __fmaf_rn(e.x, __uint_as_float(w[h].x << 16), d[j][h]);
          d[j][h] = __fmaf_rn(e.y, __uint_as_float(w[h].x & 0xffff0000u), d[j][h]);
          d[j][h] = __fmaf_rn(e.z, __uint_as_float(w[h].y << 16), d[j][h]);
          d[j][h] = __fmaf_rn(e.w, __uint_as_float(w[h].y & 0xffff0000u), d[j][h]);
          d[j][h] = __fmaf_rn(f.x, __uint_as_float(w[h].z << 16), d[j][h]);
          d[j][h] = __fmaf_rn(f.y, __uint_as_float(w[h].z & 0xffff0000u), d[j][h]);
          d[j][h] = __fmaf_rn(f.z, __uint_as_float(w[h].w << 16), d[j][h]);
          d[j][h] = __fmaf_rn(f.w, __uint_as_float(w[h].w & 0xffff0000u), d[j][h]);
        }
      }
    }
    for (int o = 1; SHARED && o < 1 << lanes.log; o <<= 1)
#pragma unroll
      for (int j = 0; j < kFewest; ++j) {
        if (j >= rows) break;
        d[j][0] += __shfl_xor_sync(together, d[j][0], o);
        d[j][1] += __shfl_xor_sync(together, d[j][1], o);
      }
    if (lanes.rank() > 0) continue;
#pragma unroll
    for (int j = 0; j < kFewest; ++j) {
      if (j >= rows) break;
      const int64_t at = ((row0 + sm.t.rows[j]) * p.N + n) / 2;
      if (F32) {
        float2 e = make_float2(0.f, 0.f);
        if (p.base) e = u < 2 ? *reinterpret_cast<const float2*>(sm.place(sm.base, u * kFewest + j, 8)) : static_cast<const float2*>(p.base)[at];
        static_cast<float2*>(p.out)[at] = make_float2(e.x + d[j][0], e.y + d[j][1]);
      } else {
        uint32_t e = 0;
        if (p.base) e = u < 2 ? *reinterpret_cast<const uint32_t*>(sm.place(sm.base, u * kFewest + j, 4)) : static_cast<const uint32_t*>(p.base)[at];
        const __nv_bfloat162 o = __floats2bfloat162_rn(__uint_as_float(e << 16) + d[j][0], __uint_as_float(e & 0xffff0000u) + d[j][1]);
        static_cast<uint32_t*>(p.out)[at] = *reinterpret_cast<const uint32_t*>(&o);
      }
    }
  }
}

// A warp takes a block of 32 features at a time, its weights S steps of 16 ranks at a time; up to S steps
// in all (WHOLE) the next block's loads are under way meanwhile.
template <bool F32, int S, bool WHOLE>
__global__ void __launch_bounds__(kUpThreads, 2) adapter_few_up_kernel(Adapter p, int ctas) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  UpSmem<F32>& sm = *reinterpret_cast<UpSmem<F32>*>(smem_raw);
  constexpr int kParts = F32 ? 3 : 2;  // bf16 numbers that carry a value of v
  constexpr int kAhead = UpSmem<F32>::kAhead;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, q = lane & 3;
  const int chunk = blockIdx.x / ctas, cta = blockIdx.x - chunk * ctas;
  const int64_t row0 = (int64_t)chunk * kChunk;
  const int rows = p.M - row0 < kChunk ? (int)(p.M - row0) : kChunk;
  clear_tables(sm.t);
  __syncthreads();
  // The first kernel lets this one start when all before it is complete: what is not v can be read and
  // written already.
  make_tables(p, sm.t, row0, rows, false);
  const int nk = (p.K + 31) / 32, nb = (p.N + 31) / 32, pieces = Share(sm.t.tiles, nk, kPieces, p.r, 0, ctas).parts;
  const int lr = p.r <= 32 ? 5 : p.r <= 64 ? 6 : 7, steps = (p.r + 15) / 16;
  const Share share(sm.t.tiles, nb, nb, p.r, cta, ctas);
  float scale = 1.f;
  int t, part, b0, b1;
  // A tile's rows; its scale, and its part of B and of its rows of base on their way: what each thread
  // reads first into shared memory, the rest into L2.
  const auto begin = [&] {
    const int id = tile_rows(sm.t, t), wide = min(b1 * 32, p.N) - b0 * 32;
    if (p.scale) scale = p.scale[id];
    if (sm.t.rows[kFewest] < 0) {
      fetch_few<F32, !WHOLE>(p, sm, id, row0, b0 * 32, min(b1 * 32, p.N));
    } else {
      // a step of 16 ranks of a block of 32 features is number (block * steps + step) of the warp's
      const uint16_t* B = static_cast<const uint16_t*>(p.b) + ((int64_t)id * p.N + 8 * (g >> 1) + (g & 1)) * p.r + q * 4;
      int b = b0 + warp;
      for (int i = 0, s = 0; i < kAhead / 2 && b < b1; ++i) {
        if (b * 32 + 8 * (g >> 1) < p.N && s * 16 + q * 4 < p.r)
          for (int j = 0; j < 4; ++j)
            cpa::cp_async8(tc::smem_addr(sm.place(sm.b, i * 4 + j, 8)), B + (int64_t)b * 32 * p.r + 2 * j * p.r + s * 16);
        if (++s == steps) {
          s = 0;
          b += kUpWarps;
        }
      }
      b = b0 + warp;
      if (p.base && b < b1 && b * 32 + 8 * q < p.N) {
        const int ra = sm.t.rows[g], rb = sm.t.rows[g + 8];
        if (ra >= 0) Out8<F32>::fetch(sm, 0, p.base, (row0 + ra) * p.N + 8 * q + b * 32);
        if (rb >= 0) Out8<F32>::fetch(sm, 1, p.base, (row0 + rb) * p.N + 8 * q + b * 32);
      }
    }
    const char* from = reinterpret_cast<const char*>(static_cast<const uint16_t*>(p.b) + ((int64_t)id * p.N + b0 * 32) * p.r);
    for (int64_t i = kAhead * kUpThreads * 16 + (int64_t)tid * 128; i < (int64_t)wide * p.r * 2; i += kUpThreads * 128) prefetch_l2(from + i);
    constexpr int kSize = F32 ? 4 : 2;
    const int m = sm.t.rows[warp];
    if (p.base && m >= 0) {
      const char* at = static_cast<const char*>(p.base) + ((row0 + m) * p.N + b0 * 32) * kSize;
      for (int i = 32 * kUpWarps * kSize + lane * 128; i < wide * kSize; i += 32 * 128) prefetch_l2(at + i);
    }
    return id;
  };
  int id = share.get(0, t, part, b0, b1) ? begin() : 0;
  // rows of requests without an adapter: base as it is
  if (p.base != p.out) {
    const int units = p.N / 8 * (F32 ? 2 : 1);
    for (int i = cta; i < rows; i += ctas)
      if (sm.t.id[i] == -1)
        for (int c = tid; c < units; c += kUpThreads) {
          const int64_t at = (row0 + i) * units + c;
          static_cast<uint4*>(p.out)[at] = p.base ? static_cast<const uint4*>(p.base)[at] : make_uint4(0, 0, 0, 0);
        }
  }
  moe::wait_for_stream();
  moe::let_next_start();
  for (int turn = 0; share.get(turn, t, part, b0, b1); ++turn) {
    if (turn > 0) id = begin();
    if (sm.t.rows[kFewest] < 0) {
      few_rows<F32, !WHOLE>(p, sm, id, row0, b0 * 32, min(b1 * 32, p.N), pieces, lr, scale);
      continue;
    }
    sum_pieces<kParts>(p, sm, row0, pieces, lr, scale);
    cpa::cp_async_wait_all();
    __syncthreads();
    // v B^T, 32 features at a time: feature 8 (c / 2) + 2 j + c % 2 is column c of product j, so that a
    // lane ends with eight neighbouring ones of its rows
    const int ra = sm.t.rows[g], rb = sm.t.rows[g + 8];
    const uint16_t* B = static_cast<const uint16_t*>(p.b) + ((int64_t)id * p.N + 8 * (g >> 1) + (g & 1)) * p.r + q * 4;
    const int64_t at_a = (row0 + ra) * p.N + 8 * q, at_b = (row0 + rb) * p.N + 8 * q;
    uint2 w[S][4];
    Out8<F32> oa, ob;  // base
    const auto load_w = [&](int b, int s0) {  // eight features are all within N, or none
      const bool on = b < b1 && b * 32 + 8 * (g >> 1) < p.N;
      const uint16_t* at = B + (int64_t)b * 32 * p.r + s0 * 16;
      const int n = (b - b0) / kUpWarps * steps + s0;
#pragma unroll
      for (int s = 0; s < S; ++s)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          w[s][j] = !on || (s0 + s) * 16 + q * 4 >= p.r ? make_uint2(0, 0)
                    : n + s < kAhead / 2 ? *reinterpret_cast<const uint2*>(sm.place(sm.b, (n + s) * 4 + j, 8))
                                         : moe::ldg_nc_u64(at + 2 * j * p.r + s * 16);
    };
    const auto load_o = [&](int b) {
      const bool on = b < b1 && b * 32 + 8 * q < p.N;
      if (b == b0 + warp) {
        oa.take(sm, 0, on && p.base && ra >= 0);
        ob.take(sm, 1, on && p.base && rb >= 0);
      } else {
        oa.load(p.base, at_a + b * 32, on && ra >= 0);
        ob.load(p.base, at_b + b * 32, on && rb >= 0);
      }
    };
    if (WHOLE) {
      load_w(b0 + warp, 0);
      load_o(b0 + warp);
    }
    for (int b = b0 + warp; b < b1; b += kUpWarps) {
      float d[4][4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) d[j][i] = 0.f;
      if (!WHOLE) load_o(b);
      for (int s0 = 0; s0 < (WHOLE ? S : steps); s0 += S) {
        if (!WHOLE) load_w(b, s0);
#pragma unroll
        for (int s = 0; s < S; ++s) {
          if (s0 + s >= steps) break;
#pragma unroll
          for (int h = 0; h < kParts; ++h) {
            const int at = (s0 + s) * 8 + q * 2;
            const uint2 va = *reinterpret_cast<const uint2*>(sm.vb(h) + g * kVs + at);
            const uint2 vc = *reinterpret_cast<const uint2*>(sm.vb(h) + (g + 8) * kVs + at);
            const uint32_t a[4] = {va.x, vc.x, va.y, vc.y};
#pragma unroll
            for (int j = 0; j < 4; ++j) moe::mma_bf16(d[j], a, w[s][j].x, w[s][j].y, d[j]);
          }
        }
      }
      const Out8<F32> ea = oa, eb = ob;
      if (WHOLE) {
        load_w(b + kUpWarps, 0);
        load_o(b + kUpWarps);
      }
      if (b * 32 + 8 * q < p.N) {
        const float lo[8] = {d[0][0], d[0][1], d[1][0], d[1][1], d[2][0], d[2][1], d[3][0], d[3][1]};
        const float hi[8] = {d[0][2], d[0][3], d[1][2], d[1][3], d[2][2], d[2][3], d[3][2], d[3][3]};
        if (ra >= 0) ea.add_and_store(p.out, at_a + b * 32, lo);
        if (rb >= 0) eb.add_and_store(p.out, at_b + b * 32, hi);
      }
    }
  }
}

constexpr int kCtasMost = 160;  // of a call, where its chunks are fewer

constexpr int kCarveout = 44;  // per cent of 228 KB
static_assert(sizeof(DownSmem) + std::max(sizeof(UpSmem<false>), sizeof(UpSmem<true>)) + 2 * 1024 <= 100 * 1024, "");

cudaError_t share_sm(const void* kernel, std::atomic<uint64_t>& done) {
  int dev = -1;
  const bool known = cudaGetDevice(&dev) == cudaSuccess && dev >= 0 && dev < 64;
  if (known && (done.load(std::memory_order_relaxed) >> dev & 1)) return cudaSuccess;
  const cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, kCarveout);
  if (err == cudaSuccess && known) done.fetch_or(uint64_t{1} << dev, std::memory_order_relaxed);
  return err;
}

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
  const int ctas = ctas_of(p.M, sm_count_current());
  const dim3 grid((unsigned)(chunks_of(p.M) * ctas));
  const auto down = p.r <= 16 ? adapter_few_down_kernel<2, 4> : adapter_few_down_kernel<4, 3>;
  // An SM that is set up for the shared memory of the first kernel's blocks alone would take the second's
  // only when it is empty; and what is not shared memory is L1, which the first kernel's loads need.  So both
  // ask for 100 KB, a block of each (250 rows of rank 64 over five adapters: 13.2 us; with nothing asked for
  // 14.6, with 164 KB and twice as much copied ahead 13.5, with all of it 14.4).
  static std::atomic<uint64_t> set[2] = {};
  cudaError_t e = share_sm((const void*)down, set[p.r > 16]);
  if (e != cudaSuccess) return e;
  e = launch_staged(down, grid, dim3(kThreads), sizeof(DownSmem), stream, 1, p, ctas);
  if (e != cudaSuccess) return e;
  const auto up = p.r <= 16   ? (p.out_f32 ? adapter_few_up_kernel<true, 1, true> : adapter_few_up_kernel<false, 1, true>)
                  : p.r <= 32 ? (p.out_f32 ? adapter_few_up_kernel<true, 2, true> : adapter_few_up_kernel<false, 2, true>)
                              : (p.out_f32 ? adapter_few_up_kernel<true, 2, false> : adapter_few_up_kernel<false, 2, false>);
  const int smem = p.out_f32 ? sizeof(UpSmem<true>) : sizeof(UpSmem<false>);
  static std::atomic<uint64_t> done[6] = {}, set_up[6] = {};
  e = allow_smem((const void*)up, smem, done[(p.out_f32 ? 3 : 0) + (p.r <= 16 ? 0 : p.r <= 32 ? 1 : 2)]);
  if (e == cudaSuccess) e = share_sm((const void*)up, set_up[(p.out_f32 ? 3 : 0) + (p.r <= 16 ? 0 : p.r <= 32 ? 1 : 2)]);
  if (e != cudaSuccess) return e;
  return launch_staged(up, grid, dim3(kUpThreads), smem, stream, 1, p, ctas);
}

}  // namespace moe_launch
