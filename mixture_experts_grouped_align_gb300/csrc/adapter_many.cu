// Low-rank adapters of many requests beside a dense product: long requests, on tcgen05.
//
//   v = x A[a]^T  (adapter_down_kernel);   out = base + scale[a] v B[a]^T  (adapter_up_kernel)
//
// Both are streams: x is read once, base and out once each, and the products are 2 r operations a
// value of them, far below the tensor cores' rate.  Tiles are up to 128 rows of one request (so of one
// adapter: no accumulator row has two, and what a box reads past the request is dropped).  Their number
// is known on the device only; every block adds up the requests' tiles, and each takes an equal run of
// all tiles' blocks of K (first kernel) or of N (second), however the runs cut the tiles.
//   down: stages of 64 of K, 128 rows of x and the adapter's r rows by TMA; M = 128, N = r, K = 16 MMAs
//         into one of two accumulators; the sum of a tile's piece goes to the workspace in fp32.  The
//         accumulator loses up to a unit in the last place with every MMA, always towards zero, which a
//         bf16 output hides: for fp32 outputs it takes kChunk stages at most, which are added there.
//   up:   the builder warps add the pieces of a tile's v, scale it and leave it as two bf16 operands whose
//         sum it is to 2^-17 of itself (three for fp32 outputs), the rows of MMAs against 128 features of B
//         at a time; base comes in boxes of 128 bytes x 128 rows, six ahead, in which the epilogue warps add
//         the accumulator and from which they store whole lines of the request's rows.
// Every wait is bounded; one that runs out sets MOE_ERR_TIMEOUT and all roles leave their loops.
// Measured (replayed graphs): 58879 rows of 16 requests of rank 64, 2880 -> 2880, 187 us for 1022 MB: down 62 (5.6
// TB/s), up 119 (6.1 TB/s; a copy moves 6.8); 8192 rows of rank 32, 7168 -> 4096, 54 us: 25 (4.7 TB/s) and 31, of
// which 6 are the first v and the last stores.  The kernels follow one another on an SM, as each fills its
// shared memory; what is not v of the second one starts where the first has left (56 us with a wait for all).
#include <algorithm>

#include "dense_common.cuh"

namespace {

using moe_launch::Adapter;

constexpr int kRows = 128, kRequestsMost = 1024;
constexpr int kBox = kRows * 128;  // bytes of a box of 128 rows x 128 bytes
constexpr int kPart = 32;          // rows of the boxes that a shorter tile takes instead

// Of the requests: tiles before one [R + 1], and of those with an adapter [R + 1], first row, the row
// behind the last, adapter (-1: none).
struct Tables {
  const int32_t *first, *own, *start, *end, *id;
  int R;
};

struct Tile {
  int id, rows, own;  // own: its number among those with an adapter
  int64_t row0;
};

__host__ __device__ inline int table_bytes(int R) { return (5 * R + 2) * 4; }

__device__ __forceinline__ Tables tables_of(const int32_t* mem, int R) {
  return Tables{mem, mem + R + 1, mem + 2 * R + 2, mem + 3 * R + 2, mem + 4 * R + 2, R};
}

// The requests' tiles, by one warp; `bare`: requests without an adapter have tiles too.  A request that
// starts before the highest offset so far has none: rows are in one request at most, whatever the
// offsets, and there are no more tiles than the workspace has places for.
__device__ __forceinline__ void make_tables(const Adapter& p, int32_t* mem, bool bare, bool report) {
  int32_t *first = mem, *own = mem + p.R + 1, *start = own + p.R + 1, *end = start + p.R, *id = end + p.R;
  const int lane = threadIdx.x & 31;
  int32_t tiles = 0, owned = 0, top = 0;
  for (int i0 = 0; i0 < p.R; i0 += 32) {
    const int i = i0 + lane;
    int32_t lo = 0, hi = 0, a = -1, n = 0, m = 0;
    if (i < p.R) {
      lo = p.row_offsets[i];
      hi = p.row_offsets[i + 1];
      a = p.adapter[i];
    }
    int32_t high = lo >= 0 && lo <= p.M ? lo : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t v = __shfl_up_sync(0xffffffffu, high, o);
      if (lane >= o) high = max(high, v);
    }
    high = max(high, top);
    top = __shfl_sync(0xffffffffu, high, 31);
    if (i < p.R) {
      const bool bounds = lo >= high && lo <= hi && hi <= p.M, known = a >= -1 && a < p.L;
      if (report && !(bounds && known)) moe::set_status(p.status, bounds ? MOE_ERR_INVALID_EXPERT : MOE_ERR_CAPACITY);
      if (!known) a = -1;
      if (bounds) n = (hi - lo + kRows - 1) / kRows;
      if (a >= 0) m = n;
      else if (!bare) n = 0;
    }
    int32_t sn = n, sm = m;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t u = __shfl_up_sync(0xffffffffu, sn, o), v = __shfl_up_sync(0xffffffffu, sm, o);
      if (lane >= o) {
        sn += u;
        sm += v;
      }
    }
    if (i < p.R) {
      first[i] = tiles + sn - n;
      own[i] = owned + sm - m;
      start[i] = lo;
      end[i] = hi;
      id[i] = a;
    }
    tiles += __shfl_sync(0xffffffffu, sn, 31);
    owned += __shfl_sync(0xffffffffu, sm, 31);
  }
  if (lane == 0) {
    first[p.R] = tiles;
    own[p.R] = owned;
  }
}

__device__ __forceinline__ Tile tile_of(const Tables& t, int n) {
  int lo = 0, hi = t.R;  // the last request with first <= n (requests without tiles share it with the next)
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (t.first[mid] <= n) lo = mid;
    else hi = mid;
  }
  const int row = t.start[lo] + (n - t.first[lo]) * kRows;
  return Tile{t.id[lo], min(kRows, t.end[lo] - row), t.own[lo] + n - t.first[lo], row};
}

// A CTA's run over the tiles' blocks: `blocks` a tile, in pieces of one tile each.
struct Run {
  int64_t at, end;
  int blocks;
  __device__ __forceinline__ Run(int64_t total, int blocks, int cta, int ctas) : blocks(blocks) {
    at = cta < ctas ? total * cta / ctas : 0;
    end = cta < ctas ? total * (cta + 1) / ctas : 0;
  }
  __device__ __forceinline__ bool next(int& tile, int& b0, int& b1) {
    if (at >= end) return false;
    tile = (int)(at / blocks);
    b0 = (int)(at - (int64_t)tile * blocks);
    b1 = (int)min((int64_t)blocks, b0 + end - at);
    at += b1 - b0;
    return true;
  }
};

// The first kernel's CTAs: each has a block at least, and few tiles are cut into few pieces, the fewer the
// wider v is, since every CTA of the second kernel that has features of a tile reads all of its pieces.
__device__ __forceinline__ int down_ctas(int tiles, int blocks, int ctas, int r) {
  const int most = r <= 32 ? 8 : r <= 64 ? 4 : 2;
  return min(ctas, min(most, blocks) * tiles);
}
// The CTA whose run has block x.
__device__ __forceinline__ int owner(int64_t x, int64_t total, int ctas) { return (int)(((x + 1) * ctas - 1) / total); }
// A piece's place in the workspace is its tile's number plus its CTA's: no two pieces share one, as from
// piece to piece one of the two at least goes up.

// A tile's rows of 128 bytes at x: one box, or boxes of 32 rows for a tile of fewer than 128.
__device__ __forceinline__ void load_rows(uint32_t dst, const CUtensorMap* whole, const CUtensorMap* part, int x, const Tile& tl,
                                              uint64_t* bar) {
  if (tl.rows == kRows) {
    tma::load_2d(dst, whole, x, (int32_t)tl.row0, bar);
  } else {
    for (int r = 0; r < tl.rows; r += kPart) tma::load_2d(dst + r * 128, part, x, (int32_t)tl.row0 + r, bar);
  }
}
__device__ __forceinline__ uint32_t rows_bytes(const Tile& tl) {
  return tl.rows == kRows ? kBox : (uint32_t)((tl.rows + kPart - 1) / kPart * kPart * 128);
}

// ------------------------------------------------------------------------------------------ down

constexpr int kDownThreads = 256, kDownStages = 10;
constexpr int kChunk = 12;  // stages of an accumulator for fp32 outputs

__global__ void __launch_bounds__(kDownThreads, 1)
    adapter_down_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_x32,
                        const __grid_constant__ CUtensorMap tm_a, Adapter p, int stages) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ uint64_t full[kDownStages], empty[kDownStages], tfull[2], tempty[2], drain;
  __shared__ uint32_t taddr_s;
  __shared__ volatile int abort_flag;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int rp = (p.r + 15) / 16 * 16, slot = kBox + rp * 128;
  const uint32_t smem_s = tc::smem_addr(smem);
  int32_t* tab = reinterpret_cast<int32_t*>(smem + stages * slot);
  const uint64_t wb = p.wait_ns > 0 ? (uint64_t)p.wait_ns : tc::kWaitNs;
  if (tid == 0) {
    for (int s = 0; s < stages; ++s) {
      tc::mbar_init(&full[s], 1);
      tc::mbar_init(&empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&tfull[i], 1);
      tc::mbar_init(&tempty[i], 4);
    }
    tc::mbar_init(&drain, 1);
    abort_flag = 0;
    tc::mbar_fence_init();
  }
  moe::wait_for_stream();
  moe::let_next_start();
  if (warp == 1) {
    tc::tmem_alloc(&taddr_s, 256);
    tc::tmem_relinquish();
  } else if (warp == 2) {
    make_tables(p, tab, false, blockIdx.x == 0);
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t taddr = __shfl_sync(0xffffffffu, taddr_s, 0);
  const Tables t = tables_of(tab, p.R);
  const int nk = (p.K + 63) / 64, tiles = t.first[p.R], ctas = down_ctas(tiles, nk, gridDim.x, p.r);
  Run run((int64_t)tiles * nk, nk, blockIdx.x, ctas);
  int tile, k0, k1;

  if (warp == 0 && !p.stall) {
    const bool leader = dense::elect_one();
    int s = 0, n = 0;
    uint32_t ph = 1;  // a slot's first use waits for nothing
    bool ok = true;
    while (ok && run.next(tile, k0, k1)) {
      const Tile tl = tile_of(t, tile);
      for (int k = k0; k < k1; ++k) {
        if (abort_flag || !tc::mbar_wait(&empty[s], ph, wb)) {
          if (!abort_flag) moe::set_status(p.status, MOE_ERR_TIMEOUT);
          abort_flag = 1;
          ok = false;
          break;
        }
        if (leader) {
          const uint32_t at = smem_s + s * slot;
          tma::mbar_arrive_expect_tx(&full[s], rows_bytes(tl) + (uint32_t)(rp * 128));
          load_rows(at, &tm_x, &tm_x32, k * 128, tl, &full[s]);
          tma::load_2d(at + kBox, &tm_a, k * 128, tl.id * p.r, &full[s]);
        }
        __syncwarp();
        ++n;
        if (++s == stages) {
          s = 0;
          ph ^= 1;
        }
      }
    }
    // every load lands before the block may end, also when another role has given up
    for (int j = n > stages ? n - stages : 0; j < n; ++j)
      if (!tc::mbar_wait(&full[j % stages], (j / stages) & 1, wb)) moe::set_status(p.status, MOE_ERR_TIMEOUT);
  } else if (warp == 1 && !p.stall) {
    const bool leader = dense::elect_one();
    const uint32_t idesc = tc::idesc_f16(kRows, rp, 1);
    int s = 0, acc_it = 0;
    uint32_t ph = 0;
    bool ok = true;
    while (ok && run.next(tile, k0, k1))
      for (int from = k0, until; ok && from < k1; from = until, ++acc_it) {
        until = p.out_f32 ? min(k1, from + kChunk) : k1;
        const int acc = acc_it & 1;
        ok = tc::mbar_wait(&tempty[acc], ((acc_it >> 1) & 1) ^ 1, wb);
        tc::tc_fence_after();
        for (int k = from; k < until && ok; ++k) {
          if (abort_flag || !tc::mbar_wait(&full[s], ph, wb)) {
            ok = false;
            break;
          }
          tc::tc_fence_after();
          if (leader) {
            const uint64_t xd = tc::sdesc_sw128(smem_s + s * slot), ad = tc::sdesc_sw128(smem_s + s * slot + kBox);
#pragma unroll
            for (int j = 0; j < 4; ++j) tc::mma_f16_ss(taddr + acc * 128, xd + 2 * j, ad + 2 * j, idesc, k > from || j > 0);
            tc::mma_commit(&empty[s]);
          }
          __syncwarp();
          if (++s == stages) {
            s = 0;
            ph ^= 1;
          }
        }
        if (!ok) {
          if (!abort_flag) moe::set_status(p.status, MOE_ERR_TIMEOUT);
          abort_flag = 1;
        } else if (leader) {
          tc::mma_commit(&tfull[acc]);
        }
        __syncwarp();
      }
    if (leader) {
      tc::mma_commit(&drain);
      if (!tc::mbar_wait(&drain, 0, wb)) moe::set_status(p.status, MOE_ERR_TIMEOUT);
    }
    __syncwarp();
  } else if (warp >= 4) {
    const int quarter = warp & 3, row = quarter * 32 + lane;
    int acc_it = 0;
    bool ok = true;
    while (ok && run.next(tile, k0, k1)) {
      const Tile tl = tile_of(t, tile);
      float* at = p.v + ((int64_t)(tile + blockIdx.x) * kRows + row) * p.r;
      for (int from = k0, until; from < k1; from = until, ++acc_it) {
        until = p.out_f32 ? min(k1, from + kChunk) : k1;
        const int acc = acc_it & 1;
        if (abort_flag || !tc::mbar_wait(&tfull[acc], (acc_it >> 1) & 1, wb)) {
          if (!abort_flag) moe::set_status(p.status, MOE_ERR_TIMEOUT);
          abort_flag = 1;
          ok = false;
          break;
        }
        tc::tc_fence_after();
        for (int c = 0; c < rp; c += 16) {
          uint32_t v[16];
          dense::tmem_ld16(taddr + acc * 128 + ((uint32_t)(quarter * 32) << 16) + c, v);
          tc::tmem_ld_wait();
          if (row < tl.rows)
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (c + 4 * j < p.r) {
                float4* to = reinterpret_cast<float4*>(at + c) + j;
                float4 e = make_float4(__uint_as_float(v[4 * j]), __uint_as_float(v[4 * j + 1]), __uint_as_float(v[4 * j + 2]),
                                       __uint_as_float(v[4 * j + 3]));
                if (from > k0) {  // this thread's own, of the accumulator before
                  const float4 b = *to;
                  e = make_float4(b.x + e.x, b.y + e.y, b.z + e.z, b.w + e.w);
                }
                *to = e;
              }
        }
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&tempty[acc]);
      }
    }
  }
  __syncwarp();
  tc::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc::tc_fence_after();
    tc::tmem_dealloc(taddr, 256);
  }
}

// -------------------------------------------------------------------------------------------- up

constexpr int kUpThreads = 512;
constexpr int kFeat = 128;      // features of an accumulator
constexpr int kAccs = 4;
constexpr int kBaseSlots = 6;   // at most, and always even: see UpPlan
constexpr int kWeightSlots = 3;

struct UpPlan {
  int blocks;                   // of 64 ranks
  int bufs;                     // operands of v
  // Base's slots are even in number, so that a slot's boxes are always the same drain group's: a wait by
  // parity holds for the phase at hand or the next only, and a group that passed over the other's use of a
  // slot would take that use's end for its own.
  int base_slots, weight_slots;
  int a, b, base, tab;          // offsets in shared memory
  int smem;
};

__device__ __forceinline__ uint32_t chunk_at(int r, int q) { return (uint32_t)(r * 128 + ((q ^ (r & 7)) << 4)); }
__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void sts8(uint32_t a, uint32_t x, uint32_t y) {
  asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(a), "r"(x), "r"(y) : "memory");
}
__device__ __forceinline__ void sts16(uint32_t a, const uint4& v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// Warps: 0 loads base, 1 issues the MMAs, 2 makes the tables, 3 loads B, 4..7 build v's operands,
// 8..15 drain (the two of a lane quarter take turns at boxes).
template <bool F32>
__global__ void __launch_bounds__(kUpThreads, 1)
    adapter_up_kernel(const __grid_constant__ CUtensorMap tm_base, const __grid_constant__ CUtensorMap tm_base32,
                      const __grid_constant__ CUtensorMap tm_b, Adapter p, UpPlan pl,
                      int down_grid) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ uint64_t bfull[kBaseSlots], bempty[kBaseSlots], wfull[kWeightSlots], wempty[kWeightSlots];
  __shared__ uint64_t afull[2], aempty[2], tfull[kAccs], tempty[kAccs], drain;
  __shared__ uint32_t taddr_s;
  __shared__ volatile int abort_flag;
  constexpr int kParts = F32 ? 3 : 2;  // bf16 numbers that carry a value of v
  constexpr int kCols = F32 ? 32 : 64, kTurns = kFeat / kCols;  // columns of a base box, boxes of an accumulator
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const uint32_t smem_s = tc::smem_addr(smem);
  int32_t* tab = reinterpret_cast<int32_t*>(smem + pl.tab);
  const uint64_t wb = p.wait_ns > 0 ? (uint64_t)p.wait_ns : tc::kWaitNs;
  if (tid == 0) {
    for (int s = 0; s < kBaseSlots; ++s) {
      tc::mbar_init(&bfull[s], 1);
      tc::mbar_init(&bempty[s], 4);
    }
    for (int s = 0; s < kWeightSlots; ++s) {
      tc::mbar_init(&wfull[s], 1);
      tc::mbar_init(&wempty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&afull[i], 4);
      tc::mbar_init(&aempty[i], 1);
    }
    for (int i = 0; i < kAccs; ++i) {
      tc::mbar_init(&tfull[i], 1);
      tc::mbar_init(&tempty[i], 8);
    }
    tc::mbar_init(&drain, 1);
    abort_flag = 0;
    tc::mbar_fence_init();
  }
  if (warp == 1) {
    tc::tmem_alloc(&taddr_s, kAccs * kFeat);
    tc::tmem_relinquish();
  }
  // The first kernel lets this one start when all before it is complete: only v is waited for, by the
  // warps that read it (of every CTA, so that this kernel never ends before the first).  What follows this
  // kernel waits for its end before it touches memory (launch_staged).
  moe::let_next_start();
  if (warp == 2) make_tables(p, tab, p.base != p.out, false);
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t taddr = __shfl_sync(0xffffffffu, taddr_s, 0);
  const Tables t = tables_of(tab, p.R);
  const int nb = (p.N + kFeat - 1) / kFeat;
  Run run((int64_t)t.first[p.R] * nb, nb, blockIdx.x, gridDim.x);
  int tile, b0, b1;
  const auto give_up = [&] {
    if (!abort_flag) moe::set_status(p.status, MOE_ERR_TIMEOUT);
    abort_flag = 1;
  };
  // boxes of base that part of an accumulator's features has
  const auto turns_of = [&](int b) { return min(kTurns, (p.N - b * kFeat + kCols - 1) / kCols); };

  if (warp == 0 && !p.stall) {
    const bool leader = dense::elect_one();
    int s = 0, n = 0;
    uint32_t ph = 1;
    bool ok = true;
    while (ok && run.next(tile, b0, b1)) {
      const Tile tl = tile_of(t, tile);
      for (int b = b0; b < b1 && ok; ++b)
        for (int c = 0; c < turns_of(b); ++c) {
          if (abort_flag || !tc::mbar_wait(&bempty[s], ph, wb)) {
            give_up();
            ok = false;
            break;
          }
          if (leader) {
            if (p.base) {
              tma::mbar_arrive_expect_tx(&bfull[s], rows_bytes(tl));
              load_rows(smem_s + pl.base + s * kBox, &tm_base, &tm_base32, (b * kFeat + c * kCols) * (F32 ? 4 : 2), tl, &bfull[s]);
            } else {
              tc::mbar_arrive(&bfull[s]);
            }
          }
          __syncwarp();
          ++n;
          if (++s == pl.base_slots) {
            s = 0;
            ph ^= 1;
          }
        }
    }
    for (int j = n > pl.base_slots ? n - pl.base_slots : 0; j < n; ++j)
      if (!tc::mbar_wait(&bfull[j % pl.base_slots], (j / pl.base_slots) & 1, wb)) give_up();
  } else if (warp == 3 && !p.stall) {
    const bool leader = dense::elect_one();
    int s = 0, n = 0;
    uint32_t ph = 1;
    bool ok = true;
    while (ok && run.next(tile, b0, b1)) {
      const Tile tl = tile_of(t, tile);
      if (tl.id < 0) continue;
      for (int b = b0; b < b1; ++b) {
        if (abort_flag || !tc::mbar_wait(&wempty[s], ph, wb)) {
          give_up();
          ok = false;
          break;
        }
        if (leader) {
          tma::mbar_arrive_expect_tx(&wfull[s], (uint32_t)(pl.blocks * kBox));
          for (int k = 0; k < pl.blocks; ++k)  // past the rank: zeros
            tma::load_2d(smem_s + pl.b + (s * pl.blocks + k) * kBox, &tm_b, k * 128, tl.id * p.N + b * kFeat, &wfull[s]);
        }
        __syncwarp();
        ++n;
        if (++s == pl.weight_slots) {
          s = 0;
          ph ^= 1;
        }
      }
    }
    for (int j = n > pl.weight_slots ? n - pl.weight_slots : 0; j < n; ++j)
      if (!tc::mbar_wait(&wfull[j % pl.weight_slots], (j / pl.weight_slots) & 1, wb)) give_up();
  } else if (warp == 1 && !p.stall) {
    const bool leader = dense::elect_one();
    const uint32_t idesc = tc::idesc_f16(kRows, kFeat, 1);
    const int steps = (p.r + 15) / 16;
    int s = 0, acc_it = 0, tile_it = 0;
    uint32_t ph = 0;
    bool ok = true;
    while (ok && run.next(tile, b0, b1)) {
      const Tile tl = tile_of(t, tile);
      if (tl.id < 0) continue;
      const int buf = tile_it % pl.bufs;
      if (abort_flag || !tc::mbar_wait(&afull[buf], (tile_it / pl.bufs) & 1, wb)) ok = false;
      for (int b = b0; b < b1 && ok; ++b, ++acc_it) {
        const int acc = acc_it % kAccs;
        if (abort_flag || !tc::mbar_wait(&tempty[acc], ((acc_it / kAccs) & 1) ^ 1, wb) || !tc::mbar_wait(&wfull[s], ph, wb)) {
          ok = false;
          break;
        }
        tc::tc_fence_after();
        if (leader) {
          for (int h = 0; h < kParts; ++h)
            for (int k = 0; k < steps; ++k) {
              const uint64_t ad = tc::sdesc_sw128(smem_s + pl.a + ((buf * kParts + h) * pl.blocks + k / 4) * kBox) + 2 * (k & 3);
              const uint64_t bd = tc::sdesc_sw128(smem_s + pl.b + (s * pl.blocks + k / 4) * kBox) + 2 * (k & 3);
              tc::mma_f16_ss(taddr + acc * kFeat, ad, bd, idesc, h > 0 || k > 0);
            }
          tc::mma_commit(&wempty[s]);
          tc::mma_commit(&tfull[acc]);
        }
        __syncwarp();
        if (++s == pl.weight_slots) {
          s = 0;
          ph ^= 1;
        }
      }
      if (!ok) {
        give_up();
      } else if (leader) {
        tc::mma_commit(&aempty[buf]);
      }
      __syncwarp();
      ++tile_it;
    }
    if (leader) {
      tc::mma_commit(&drain);
      if (!tc::mbar_wait(&drain, 0, wb)) moe::set_status(p.status, MOE_ERR_TIMEOUT);
    }
    __syncwarp();
  } else if (warp >= 4 && warp < 8) {
    // v of a tile: the pieces' sum times the adapter's scale, as bf16 numbers
    moe::wait_for_stream();
    const int row = tid - 128, nk = (p.K + 63) / 64, own = t.own[p.R], ctas = down_ctas(own, nk, down_grid, p.r);
    const int64_t total = (int64_t)own * nk;
    const int per = p.r / 4;
    int tile_it = 0;
    while (run.next(tile, b0, b1)) {
      const Tile tl = tile_of(t, tile);
      if (tl.id < 0) continue;
      const int buf = tile_it % pl.bufs;
      if (abort_flag || !tc::mbar_wait(&aempty[buf], ((tile_it / pl.bufs) & 1) ^ 1, wb)) {
        give_up();
        break;
      }
      const float scale = p.scale ? p.scale[tl.id] : 1.f;
      const int c0 = owner((int64_t)tl.own * nk, total, ctas), pieces = owner((int64_t)(tl.own + 1) * nk - 1, total, ctas) - c0 + 1;
      const float4* at = reinterpret_cast<const float4*>(p.v + (int64_t)(tl.own + c0) * kRows * p.r);
      const uint32_t mem = smem_s + pl.a + buf * kParts * pl.blocks * kBox;
      const int quads = tl.rows * per, piece = kRows * per;  // four ranks each
      for (int i0 = tid - 128; i0 < quads; i0 += 4 * kRows) {
        float4 s[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) s[u] = i0 + u * kRows < quads ? at[i0 + u * kRows] : make_float4(0.f, 0.f, 0.f, 0.f);
        for (int c = 1; c < pieces; ++c) {
          float4 e[4];
#pragma unroll
          for (int u = 0; u < 4; ++u)
            e[u] = i0 + u * kRows < quads ? at[(int64_t)c * piece + i0 + u * kRows] : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            s[u].x += e[u].x;
            s[u].y += e[u].y;
            s[u].z += e[u].z;
            s[u].w += e[u].w;
          }
        }
        const auto put = [&](int u, const uint32_t (&w)[kParts][2]) {
          const int i = i0 + u * kRows, m = i / per, k = (i - m * per) * 4;
          const uint32_t to = mem + (k >> 6) * kBox + tc::sw128_offset(m, (k & 63) >> 3) + (k & 4) * 2;
#pragma unroll
          for (int h = 0; h < kParts; ++h) sts8(to + h * pl.blocks * kBox, w[h][0], w[h][1]);
        };
        float top = 0.f;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          if (i0 + u * kRows >= quads) break;
          float f[4] = {s[u].x * scale, s[u].y * scale, s[u].z * scale, s[u].w * scale};
          uint32_t w[kParts][2];
          top = fmaxf(top, moe::largest4(f));
          moe::split_bf16<kParts>(f, w);
          put(u, w);
        }
        if (top > moe::kBf16Most) {  // again, with care (2048 rows of rank 128 33.0 us; 33.7 with a check of each four)
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            if (i0 + u * kRows >= quads) break;
            float f[4] = {s[u].x * scale, s[u].y * scale, s[u].z * scale, s[u].w * scale};
            uint32_t w[kParts][2];
            moe::split_bf16_any<kParts>(f, w);
            put(u, w);
          }
        }
      }
      if (p.r & 8) {  // the MMA's last ranks, past the adapters'
        const uint32_t to = mem + (p.r >> 6) * kBox + tc::sw128_offset(row, (p.r & 63) >> 3);
#pragma unroll
        for (int h = 0; h < kParts; ++h) sts16(to + h * pl.blocks * kBox, make_uint4(0, 0, 0, 0));
      }
      tc::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&afull[buf]);
      ++tile_it;
    }
  } else if (warp >= 8) {
    const int quarter = warp & 3, group = (warp - 8) >> 2;
    int s = 0, acc_it = 0;
    int64_t box = 0;
    uint32_t ph = 0;
    bool ok = true;
    while (ok && run.next(tile, b0, b1)) {
      const Tile tl = tile_of(t, tile);
      const bool has = tl.id >= 0, live = quarter * 32 < tl.rows;
      for (int b = b0; b < b1 && ok; ++b) {
        const int acc = acc_it % kAccs;
        if (abort_flag || (has && !tc::mbar_wait(&tfull[acc], (acc_it / kAccs) & 1, wb))) {
          give_up();
          ok = false;
          break;
        }
        tc::tc_fence_after();
        for (int c = 0; c < turns_of(b); ++c, ++box) {
          const int slot = s;
          const uint32_t par = ph;
          if (++s == pl.base_slots) {
            s = 0;
            ph ^= 1;
          }
          if ((box & 1) != group) continue;
          if (!tc::mbar_wait(&bfull[slot], par, wb)) {
            give_up();
            ok = false;
            break;
          }
          if (live) {
            const uint32_t mem = smem_s + pl.base + slot * kBox + quarter * 32 * 128;  // this warp's rows
            if (has || !p.base) {
              const uint32_t from = taddr + acc * kFeat + ((uint32_t)(quarter * 32) << 16) + c * kCols;
#pragma unroll
              for (int h = 0; h < (F32 ? 1 : 2); ++h) {
                uint32_t v[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = 0;
                if (has) {
                  tc::tmem_ld32(from + h * 32, v);
                  tc::tmem_ld_wait();
                }
#pragma unroll
                for (int q = 0; q < (F32 ? 8 : 4); ++q) {
                  const uint32_t at = mem + chunk_at(lane, h * 4 + q);
                  uint4 e = p.base ? lds16(at) : make_uint4(0, 0, 0, 0);
                  if (F32) {
                    e.x = __float_as_uint(__uint_as_float(e.x) + __uint_as_float(v[4 * q]));
                    e.y = __float_as_uint(__uint_as_float(e.y) + __uint_as_float(v[4 * q + 1]));
                    e.z = __float_as_uint(__uint_as_float(e.z) + __uint_as_float(v[4 * q + 2]));
                    e.w = __float_as_uint(__uint_as_float(e.w) + __uint_as_float(v[4 * q + 3]));
                  } else {
                    uint32_t w[4] = {e.x, e.y, e.z, e.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                      const int j = (8 * q + 2 * i) & 31;
                      const __nv_bfloat162 o = __floats2bfloat162_rn(__uint_as_float(w[i] << 16) + __uint_as_float(v[j]),
                                                                     __uint_as_float(w[i] & 0xffff0000u) + __uint_as_float(v[j + 1]));
                      w[i] = *reinterpret_cast<const uint32_t*>(&o);
                    }
                    e = make_uint4(w[0], w[1], w[2], w[3]);
                  }
                  sts16(at, e);
                }
              }
            }
            __syncwarp();
            // whole lines of the rows: eight lanes a row
            const int col = b * kFeat + c * kCols + (lane & 7) * (kCols / 8);
            uint8_t* out = static_cast<uint8_t*>(p.out) + ((tl.row0 + quarter * 32 + (lane >> 3)) * p.N + col) * (F32 ? 4 : 2);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int r = i * 4 + (lane >> 3);
              const uint4 e = lds16(mem + chunk_at(r, lane & 7));
              if (quarter * 32 + r < tl.rows && col < p.N) *reinterpret_cast<uint4*>(out + (int64_t)i * 4 * p.N * (F32 ? 4 : 2)) = e;
            }
            tc::fence_proxy_async_smem();  // this box's writes, before the next one's load
          }
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&bempty[slot]);
        }
        if (has) {
          tc::tc_fence_before();
          __syncwarp();
          if (lane == 0 && ok) tc::mbar_arrive(&tempty[acc]);
          ++acc_it;
        }
      }
    }
  }
  __syncwarp();
  tc::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc::tc_fence_after();
    tc::tmem_dealloc(taddr, kAccs * kFeat);
  }
}

constexpr int kSmemMost = 226 * 1024;
constexpr int kCtasMost = 256;

}  // namespace

namespace moe_launch {

bool adapter_many_can(int64_t M, int R) { return M >= 256 && R <= kRequestsMost; }

// The estimated time against that of the kernels for few rows, in ns: a tile costs about the same whatever
// it has of rows, since its adapter's B comes once for it, and a request ends with a tile that is not full
// (0.62 of a tile a request in the fit, over 21 sizes: the slower was chosen in four, by 5% at most); the
// others' time goes by the rows and the rank.  Times measured at both (us, tiles of 128 rows first): 4096 -> 4096
// of rank 16: 1000 rows of 16 requests 17.1 and 15.6, of 100 46.7 and 18.1, 2000 of 60 33.1 and 29.2, 512 of 8
// 14.1 and 11.6; 2880 -> 2880 of rank 64: 1000 of 16 19.7 and 23.9, 4096 of 128 51 and 101, of 400 123 and 103;
// 520 -> 256 of rank 16: 8000 of 100 17 and 26.
bool adapter_many_takes(int64_t M, int R, int r, int N, int K) {
  if (!adapter_many_can(M, R)) return false;
  const double size = ((double)N + K) / 8192;
  const double many = 9300 + 92.0 * r + 480 * (M / 128.0 + 0.62 * R) * size, few = 5100 + M * (1.1 + (6.2 + 0.38 * r) * size);
  return many < few;
}

// The pieces of v: one for each tile and one for each CTA.
size_t adapter_many_workspace_bytes(int64_t M, int R, int r) {
  return (size_t)(M / kRows + R + kCtasMost) * kRows * r * 4;
}

cudaError_t adapter_many(const Adapter& p, cudaStream_t stream) {
  const int rp = (p.r + 15) / 16 * 16, slot = kBox + rp * 128;
  const int tables = table_bytes(p.R);
  CUtensorMap tm_x, tm_x32, tm_a, tm_base, tm_base32, tm_b;
  const int size = p.out_f32 ? 4 : 2;
  if (!tma::encode_2d_u8(&tm_x, p.x, (uint64_t)p.K * 2, p.M, (uint64_t)p.K * 2, 128, kRows, true) ||
      !tma::encode_2d_u8(&tm_x32, p.x, (uint64_t)p.K * 2, p.M, (uint64_t)p.K * 2, 128, kPart, true) ||
      !tma::encode_2d_u8(&tm_base32, p.base ? p.base : p.out, (uint64_t)p.N * size, p.M, (uint64_t)p.N * size, 128, kPart, true) ||
      !tma::encode_2d_u8(&tm_a, p.a, (uint64_t)p.K * 2, (uint64_t)p.L * p.r, (uint64_t)p.K * 2, 128, rp, true) ||
      !tma::encode_2d_u8(&tm_b, p.b, (uint64_t)p.r * 2, (uint64_t)p.L * p.N, (uint64_t)p.r * 2, 128, kFeat, true) ||
      !tma::encode_2d_u8(&tm_base, p.base ? p.base : p.out, (uint64_t)p.N * size, p.M, (uint64_t)p.N * size, 128, kRows, true))
    return cudaErrorInvalidValue;
  static std::atomic<uint64_t> done[3] = {};
  const int sms = std::min(sm_count_current(), kCtasMost);
  const int stages = std::min(kDownStages, (kSmemMost - 1024 - tables) / slot);
  cudaError_t e = allow_smem((const void*)adapter_down_kernel, kSmemMost, done[0]);
  if (e == cudaSuccess)
    e = launch_staged(adapter_down_kernel, dim3((unsigned)sms), dim3(kDownThreads), stages * slot + tables + 1024, stream, 1, tm_x,
                      tm_x32, tm_a, p, stages);
  if (e != cudaSuccess) return e;
  UpPlan pl{};
  pl.blocks = (p.r + 63) / 64;
  pl.bufs = pl.blocks == 1 ? 2 : 1;
  pl.weight_slots = pl.blocks == 1 && !p.out_f32 ? kWeightSlots : 2;  // six boxes of base fit beside them
  pl.a = 0;
  pl.b = pl.bufs * (p.out_f32 ? 3 : 2) * pl.blocks * kBox;
  pl.base = pl.b + pl.weight_slots * pl.blocks * kBox;
  pl.base_slots = std::min(kBaseSlots, (kSmemMost - 1024 - tables - pl.base) / kBox) & ~1;
  pl.tab = pl.base + pl.base_slots * kBox;
  pl.smem = pl.tab + tables + 1024;
  const auto kern = p.out_f32 ? adapter_up_kernel<true> : adapter_up_kernel<false>;
  e = allow_smem((const void*)kern, kSmemMost, done[1 + (p.out_f32 != 0)]);
  if (e != cudaSuccess) return e;
  return launch_staged(kern, dim3((unsigned)sms), dim3(kUpThreads), pl.smem, stream, 1, tm_base, tm_base32, tm_b, p, pl, sms);
}

}  // namespace moe_launch
