// The router's auxiliary losses with their gradient, and the gradient of the routing weights.
//
// With n real tokens (mask != 0), c_e the number of their top-k choices that name expert e,
// p_t = softmax(logits_t) over all experts and lse_t = log sum_e exp(logits_te):
//   balance = sum_e f_e P_e,  f_e = E c_e / (n k),  P_e = (1/n) sum_t p_te
//   z       = (1/n) sum_t lse_t^2
//   loss    = a * balance + b * z
//   d loss / d logits_te = (a/n) p_te (g_e - sum_e' g_e' p_te') + (2b/n) lse_t p_te,
// where g_e = f_e - 1 may stand for f_e because sum_e p_te = 1: g is formed from integers, so
// a well balanced router (all f_e near 1) loses nothing to cancellation.  The routing weights
// w_t = softmax over the token's k chosen logits add
//   [e = id_tj] w_tj (dw_tj - sum_i w_ti dw_ti).
//
// The counts f are no function of the logits' values, so one pass over the logits gives both
// the sums of p and the gradient: T E floats read once and written once, which is the floor.
// Two launches: the counts (T k ids), then the pass (above 512 experts a third for the column
// sums); a small batch is one launch of one cluster, which counts for itself.
//
// The pass gives a row to LANES lanes (4 to 32, NV vectors of four values each) and keeps it in
// registers from the load to the store.
// Every lane keeps the column sums of its own columns over its rows; blocks add theirs in a
// fixed order into one row of partial sums each, and the last block to finish adds those rows
// in order, so that repeated calls give the same bits (no floating-point atomics).
//
// Measured: 61440 x 128, k 4: 20 us for 62.9 MB of rows (3.1 TB/s), 22 with a mask; 8192 x 256, k 8:
// 12.7 us; 30000 x 1024, k 8: 53 us (4.6 TB/s); 64 x 128: 4.9 us.  Bound, in that order, by the counts before
// the pass and the sums behind it (about 6 and 4 us; the rows between them run at 6.6 TB/s), by
// that chain alone, by the rows, and by one launch with two rounds of loads.
#include "moe_common.cuh"
#include "moe_launch.h"
#include "tcgen05.cuh"

namespace {

using moe_launch::RouterLoss;

constexpr int kCountThreads = 512;
constexpr int kMaxCountBlocks = 64;
constexpr int kMaxPassBlocks = 256;       // one block per SM
constexpr int kClusterBlocks = 8;
constexpr int kFinishThreads = 256;       // >= the pass's blocks and the vectors of a block's columns
constexpr unsigned kAll = 0xffffffffu;

// Workspace: ticket (256 bytes) | the choices' counts [E], then the real tokens | counts of the
// count blocks [kMaxCountBlocks][count_pitch(E)] (their word E: its real tokens) | column sums of the
// pass's blocks [kMaxPassBlocks][part_pitch(E)] | their sums of lse^2 [kMaxPassBlocks].
__host__ __device__ inline int part_pitch(int E) { return (E + 3) / 4 * 4; }
__host__ __device__ inline int count_pitch(int E) { return (E + 4) / 4 * 4; }
struct Ws {
  unsigned* ticket;
  int* total;
  int* counts;
  float* part;
};
__host__ __device__ inline Ws carve(void* ws, int E) {
  uint8_t* p = static_cast<uint8_t*>(ws);
  Ws w;
  w.ticket = reinterpret_cast<unsigned*>(p);
  w.total = reinterpret_cast<int*>(p + 256);
  w.counts = w.total + count_pitch(E);
  w.part = reinterpret_cast<float*>(p + 256 + ((size_t)(kMaxCountBlocks + 1) * count_pitch(E) * 4 + 255) / 256 * 256);
  return w;
}

// Counts of tokens [t0, t1) (t0 a multiple of 4) into hist[E] (shared) and their real tokens into
// *n_real (shared).  Four ids a load, four loads in flight per thread.
template <int kThreads>
__device__ void count_tokens(const RouterLoss& a, int64_t t0, int64_t t1, int* hist, int* n_real) {
  for (int e = threadIdx.x; e < a.E; e += kThreads) hist[e] = 0;
  if (threadIdx.x == 0) *n_real = 0;
  __syncthreads();
  const uint32_t p0 = (uint32_t)(t0 * a.k), n = (uint32_t)((t1 - t0) * a.k), k = (uint32_t)a.k;
  bool bad = false;
  auto add = [&](int id) {
    if ((uint32_t)id < (uint32_t)a.E) atomicAdd(&hist[id], 1);
    else bad = true;
  };
  const int4* v = reinterpret_cast<const int4*>(a.ids + p0);
  const uint32_t n4 = n / 4;
  for (uint32_t i = threadIdx.x; i < n4; i += 4 * kThreads) {
    int4 q[4];
    bool live[16];  // all loads before the first count
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const uint32_t j = i + u * kThreads, p = p0 + 4 * j;
      if (j < n4) q[u] = __ldg(v + j);
      const bool in = j < n4;
#pragma unroll
      for (int c = 0; c < 4; ++c) live[4 * u + c] = in;
      if (a.mask && in) {
        const uint32_t t = p / k, r = p - t * k;  // four ids: of tokens t and t + 1 at most where k >= 4
        if (k >= 4) {
          const bool m0 = a.mask[t] != 0, m1 = r + 3 < k ? m0 : a.mask[t + 1] != 0;
#pragma unroll
          for (int c = 0; c < 4; ++c) live[4 * u + c] = r + c < k ? m0 : m1;
        } else {
#pragma unroll
          for (int c = 0; c < 4; ++c) live[4 * u + c] = a.mask[(p + c) / k] != 0;
        }
      }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (live[4 * u]) add(q[u].x);
      if (live[4 * u + 1]) add(q[u].y);
      if (live[4 * u + 2]) add(q[u].z);
      if (live[4 * u + 3]) add(q[u].w);
    }
  }
  if (threadIdx.x < n - 4 * n4) {
    const uint32_t p = p0 + 4 * n4 + threadIdx.x;
    if (!a.mask || a.mask[p / k] != 0) add(a.ids[p]);
  }
  if (bad) moe::set_status(a.status, MOE_ERR_INVALID_EXPERT);
  if (a.mask) {
    int c = 0;
    for (int64_t t = t0 + threadIdx.x; t < t1; t += kThreads) c += a.mask[t] != 0;
    c = __reduce_add_sync(kAll, c);
    if ((threadIdx.x & 31) == 0 && c) atomicAdd(n_real, c);
  } else if (threadIdx.x == 0) {
    *n_real = (int)(t1 - t0);
  }
  __syncthreads();
}

__global__ void __launch_bounds__(kCountThreads) router_count_kernel(RouterLoss a, int64_t per_block) {
  extern __shared__ int sm_count[];
  __shared__ int n_real;
  moe::wait_for_stream();
  moe::let_next_start();  // the pass: what its first loads read is complete by now
  const Ws w = carve(a.ws, a.E);
  const int64_t t0 = blockIdx.x * per_block;
  const int64_t t1 = t0 + per_block < a.T ? t0 + per_block : a.T;
  count_tokens<kCountThreads>(a, t0, t1 > t0 ? t1 : t0, sm_count, &n_real);
  int* out = w.counts + (size_t)blockIdx.x * count_pitch(a.E);
  for (int e = threadIdx.x; e < a.E; e += kCountThreads) out[e] = sm_count[e];
  if (threadIdx.x == 0) {
    out[a.E] = n_real;
    if (blockIdx.x == 0) *w.ticket = 0;
  }
}

template <int LANES>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
  return v;
}
template <int LANES>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}

// 2^x with the hardware's exponential and 1/x with its reciprocal (1 to 2 ulp), results below the
// normal range flushed to 0: probabilities that small add nothing in fp32.
MOE_DEV float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
MOE_DEV float rcp_fast(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two fp32 values in a register pair, and the instructions that work on both at once: the pass
// is bound by the instructions it issues, not by its loads, where every value takes its own.
typedef unsigned long long f2;
MOE_DEV f2 pack2(float lo, float hi) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
MOE_DEV float lo2(f2 v) { return __uint_as_float((uint32_t)v); }
MOE_DEV float hi2(f2 v) { return __uint_as_float((uint32_t)(v >> 32)); }
MOE_DEV f2 add2(f2 a, f2 b) {
  f2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
MOE_DEV f2 mul2(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
MOE_DEV f2 fma2(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// A row's LANES lanes hold 2 NV pairs each.  Column of the pair's two values: adjacent where rows
// are whole 16-byte vectors (VEC), LANES apart otherwise.
template <int LANES, bool VEC>
__device__ __forceinline__ int col_of(int sub, int pair, int half) {
  return VEC ? (pair >> 1) * 4 * LANES + sub * 4 + (pair & 1) * 2 + half : (2 * pair + half) * LANES + sub;
}

// Reads a row of E values (or, WHOLE, of as many as the lanes hold): -inf past E.
template <int LANES, int NV, bool VEC, bool WHOLE>
__device__ __forceinline__ void load_row(const float* row, int E, int sub, f2 (&x)[2 * NV]) {
  const f2 none = pack2(-INFINITY, -INFINITY);
  if (VEC) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = v * 4 * LANES + sub * 4;
      if (WHOLE || c < E) {
        const longlong2 f = *reinterpret_cast<const longlong2*>(row + c);
        x[2 * v] = (f2)f.x;
        x[2 * v + 1] = (f2)f.y;
      } else {
        x[2 * v] = x[2 * v + 1] = none;
      }
    }
  } else {
#pragma unroll
    for (int p = 0; p < 2 * NV; ++p) {
      const int c0 = col_of<LANES, VEC>(sub, p, 0), c1 = col_of<LANES, VEC>(sub, p, 1);
      x[p] = pack2(c0 < E ? row[c0] : -INFINITY, c1 < E ? row[c1] : -INFINITY);
    }
  }
}

template <int LANES, int NV, bool VEC, bool WHOLE>
__device__ __forceinline__ void store_row(float* row, int E, int sub, const f2 (&d)[2 * NV]) {
  if (VEC) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = v * 4 * LANES + sub * 4;
      if (WHOLE || c < E)
        __stcs(reinterpret_cast<longlong2*>(row + c), make_longlong2((long long)d[2 * v], (long long)d[2 * v + 1]));
    }
  } else {
#pragma unroll
    for (int p = 0; p < 2 * NV; ++p) {
      const int c0 = col_of<LANES, VEC>(sub, p, 0), c1 = col_of<LANES, VEC>(sub, p, 1);
      if (c0 < E) __stcs(row + c0, lo2(d[p]));
      if (c1 < E) __stcs(row + c1, hi2(d[p]));
    }
  }
}

// The lanes' columns of a shared row of kCols values.
template <int LANES, int NV, bool VEC>
__device__ __forceinline__ void shared_row(const float* r, int sub, f2 (&v)[2 * NV]) {
  if (VEC) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const ulonglong2 f = *reinterpret_cast<const ulonglong2*>(r + i * 4 * LANES + sub * 4);
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  } else {
#pragma unroll
    for (int p = 0; p < 2 * NV; ++p) v[p] = pack2(r[col_of<LANES, VEC>(sub, p, 0)], r[col_of<LANES, VEC>(sub, p, 1)]);
  }
}

// Sum over the block's threads of v (every thread gets it; `red` holds a float per warp).
template <int kThreads>
__device__ float block_sum(float v, float* red) {
  v = group_sum<32>(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) s += red[i];
  return s;
}

// Threads of the pass: what the register file holds of a row, the next row, the columns' sums and
// their g at sixteen or at 32 values a lane.
__host__ __device__ constexpr int pass_threads(int nv) { return nv <= 4 ? 640 : 384; }

MOE_DEV uint32_t cluster_addr(const void* p, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(tc::smem_addr(p)), "r"(rank));
  return a;
}
MOE_DEV int ld_cluster_s32(const int* p, uint32_t rank) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(cluster_addr(p, rank)) : "memory");
  return v;
}
MOE_DEV float ld_cluster_f32(const float* p, uint32_t rank) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(cluster_addr(p, rank)) : "memory");
  return v;
}

// g_e = f_e - 1 of expert e's count c among n real tokens' k choices, the numerator from integers.
MOE_DEV float g_of(int E, int k, int n, int c) {
  const int64_t nk = (int64_t)n * k;
  return n > 0 ? (float)((int64_t)E * c - nk) / (float)nk : 0.f;
}

MOE_DEV void store_loss(const RouterLoss& a, float bal, float zs) {
  // a part whose coefficient is 0 is off, also where its value is infinite
  a.loss[0] = (a.balance_coef != 0.f ? a.balance_coef * bal : 0.f) + (a.z_coef != 0.f ? a.z_coef * zs : 0.f);
  a.loss[1] = bal;
  a.loss[2] = zs;
}

// CLUSTER: the grid is one cluster, whose blocks count a share of the choices each and exchange
// counts and column sums through distributed shared memory.  Otherwise the counts come from
// router_count_kernel, and the last block to finish adds the blocks' column sums.  Above 512
// experts that is router_finish_kernel's: one SM alone would read up to 152 rows of 4 KB (7000
// tokens of 1001 experts: 33 us so, 26 with a cluster of its own; 20000 of 64: 11.3 and 12.1).
// Shared memory: g [kCols] | this block's counts, later its column sums [kCols] | at the end the
// column sums of its warps [kWarps][kCols], or four of other blocks a thread.
template <int LANES, int NV, bool VEC, bool WHOLE, bool CLUSTER>
__global__ void __launch_bounds__(pass_threads(NV), 1) router_pass_kernel(RouterLoss a) {
  constexpr int kThreads = pass_threads(NV), kWarps = kThreads / 32;
  constexpr int kGroups = 32 / LANES;       // rows of a warp
  constexpr int kCols = 4 * NV * LANES;     // columns the lanes can hold, >= E
  constexpr bool kFinish = !CLUSTER && NV > 4;  // router_finish_kernel follows
  extern __shared__ float sm[];
  __shared__ int n_sh;
  __shared__ unsigned last;
  __shared__ float red[kWarps];
  __shared__ float z_sh;
  const int E = a.E, k = a.k;
  float* gs = sm;
  float* mine = sm + kCols;
  float* sums = sm + 2 * kCols;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, sub = lane % LANES, grp = lane / LANES;
  const Ws ws = carve(a.ws, E);
  const int pitch = part_pitch(E);

  const bool with_dw = a.dw != nullptr && a.d_logits != nullptr;
  const uint32_t T = (uint32_t)a.T, step = gridDim.x * kWarps * kGroups;  // T k < 2^31
  uint32_t t = (blockIdx.x * kWarps + warp) * kGroups + grp;              // this group's row
  // What a row needs is under way a turn ahead: its logits, its mask byte and this lane's choice
  // (and, once that is there, the choice's own logit).  Rows that the mask leaves out are read
  // like the others, so that no load waits for the mask.
  f2 next[2 * NV];
  int id_n = -1;
  float w_n = 0.f, dw_n = 0.f;
  bool real_n = false;
  auto load = [&](uint32_t tr) {
    real_n = tr < T;
    if (!real_n) return;
    load_row<LANES, NV, VEC, WHOLE>(a.logits + (size_t)tr * E, E, sub, next);
    if (a.mask) real_n = a.mask[tr] != 0;
    if (with_dw && sub < k) {
      id_n = a.ids[tr * k + sub];
      w_n = a.w[tr * k + sub];
      dw_n = a.dw[tr * k + sub];
    }
  };
  auto chosen = [&](uint32_t tr) { return (uint32_t)id_n < (uint32_t)E ? a.logits[(size_t)tr * E + id_n] : 0.f; };
  if (CLUSTER) {
    moe::wait_for_stream();
    moe::let_next_start();
  }
  load(t);  // before the counts are waited for
  float l0 = chosen(t);
  int* cs = reinterpret_cast<int*>(gs);
  if (CLUSTER) {
    int* hist = reinterpret_cast<int*>(mine);
    const uint32_t share = ((T + gridDim.x - 1) / gridDim.x + 3) / 4 * 4;
    const uint32_t t0 = blockIdx.x * share < T ? blockIdx.x * share : T, t1 = t0 + share < T ? t0 + share : T;
    count_tokens<kThreads>(a, t0, t1, hist, &n_sh);
    if (gridDim.x > 1) tc::cluster_sync();
    int n = 0;
#pragma unroll 1
    for (uint32_t r = 0; r < gridDim.x; ++r) n += ld_cluster_s32(&n_sh, r);
    for (int e = tid; e < E; e += kThreads) {
      int s = 0;
#pragma unroll 1
      for (uint32_t r = 0; r < gridDim.x; ++r) s += ld_cluster_s32(hist + e, r);
      cs[e] = s;
    }
    if (gridDim.x > 1) tc::cluster_sync();  // every block has read the others' counts
    else __syncthreads();
    if (tid == 0) n_sh = n;
    __syncthreads();
  } else {
    moe::wait_for_stream();
    moe::let_next_start();
    // four columns a thread, kShare threads sharing a column's count blocks, all loads in flight
    constexpr int kAcross = kCols / 4, kShare = kThreads / kAcross < 16 ? kThreads / kAcross : 16, kBatch = 8;
    if (warp == 0) {
      int c = 0;
      for (int b = lane; b < a.count_blocks; b += 32) c += __ldcg(ws.counts + (size_t)b * count_pitch(E) + E);
      c = __reduce_add_sync(kAll, c);
      if (lane == 0) n_sh = c;
    }
    const int c = (tid % kAcross) * 4, r0 = tid / kAcross;
    int4 s = make_int4(0, 0, 0, 0);
    if (c < E && r0 < kShare)
      for (int b0 = r0; b0 < a.count_blocks; b0 += kShare * kBatch) {
        int4 v[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const int b = b0 + i * kShare;
          v[i] = b < a.count_blocks ? __ldcg(reinterpret_cast<const int4*>(ws.counts + (size_t)b * count_pitch(E) + c))
                                    : make_int4(0, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          s.x += v[i].x;
          s.y += v[i].y;
          s.z += v[i].z;
          s.w += v[i].w;
        }
      }
    int* shares = reinterpret_cast<int*>(sums);
    if (r0 < kShare) *reinterpret_cast<int4*>(shares + r0 * kCols + c) = s;
    __syncthreads();
    for (int e = tid; e < E; e += kThreads) {
      int s = 0;
#pragma unroll
      for (int i = 0; i < kShare; ++i) s += shares[i * kCols + e];
      cs[e] = s;
    }
    __syncthreads();
  }
  const int n = n_sh;
  const float inv_n = n > 0 ? 1.f / (float)n : 0.f;
  const float ca = a.balance_coef * inv_n, cz = 2.f * a.z_coef * inv_n;
  for (int e = tid; e < kCols; e += kThreads) {
    float g = 0.f;
    if (e < E) {
      const int c = cs[e];
      if (blockIdx.x == 0) {
        if (a.counts) a.counts[e] = c;
        if (kFinish) {
          ws.total[e] = c;
          if (e == 0) ws.total[E] = n;
        }
      }
      g = g_of(E, k, n, c);
    }
    gs[e] = g;  // the same word cs[e] was read from, by the same thread
  }
  __syncthreads();

  f2 acc[2 * NV], g[2 * NV];
  float zacc = 0.f;
  shared_row<LANES, NV, VEC>(gs, sub, g);
#pragma unroll
  for (int p = 0; p < 2 * NV; ++p) acc[p] = 0ull;
  while (t - grp < T) {  // the same turns for every lane of a warp: the shuffles need them all
    f2 x[2 * NV];
#pragma unroll
    for (int p = 0; p < 2 * NV; ++p) x[p] = next[p];
    const bool real = real_n;
    const int id0 = id_n;
    const float w0 = w_n, dw0 = dw_n;
    if (t - grp + step < T) load(t + step);
    if (!__all_sync(kAll, real)) {  // pad rows and rows past the end look like rows with nothing left
      if (!real)
#pragma unroll
        for (int p = 0; p < 2 * NV; ++p) x[p] = pack2(-INFINITY, -INFINITY);
    }
    float m = fmaxf(lo2(x[0]), hi2(x[0]));
#pragma unroll
    for (int p = 1; p < 2 * NV; ++p) m = fmaxf(m, fmaxf(lo2(x[p]), hi2(x[p])));
    m = group_max<LANES>(m);
    // a row with nothing left by its mask (all -inf), a pad row or a row past the end: p = 0.
    // fmaxf passes over NaN, so a row of -inf and NaN looks the same and is told apart here.
    bool some = m > -INFINITY;
    if (__any_sync(kAll, !some && real)) {
      bool nan = false;
#pragma unroll
      for (int p = 0; p < 2 * NV; ++p) nan |= lo2(x[p]) != lo2(x[p]) || hi2(x[p]) != hi2(x[p]);
      const unsigned lanes = __ballot_sync(kAll, nan) >> (grp * LANES);
      some |= (LANES == 32 ? lanes : lanes & ((1u << (LANES & 31)) - 1u)) != 0;
    }
    const float m0 = m > -INFINITY ? m : 0.f;
    const f2 minus = pack2(-m0, -m0), log2e = pack2(1.44269504f, 1.44269504f);
    f2 tot2 = 0ull, s2 = 0ull;
#pragma unroll
    for (int p = 0; p < 2 * NV; ++p) {
      const f2 y = mul2(add2(x[p], minus), log2e);  // -inf stays -inf, the largest becomes 0
      x[p] = pack2(exp2_fast(lo2(y)), exp2_fast(hi2(y)));
      tot2 = add2(tot2, x[p]);
      s2 = fma2(x[p], g[p], s2);
    }
    const float tot = group_sum<LANES>(lo2(tot2) + hi2(tot2));
    const float s = group_sum<LANES>(lo2(s2) + hi2(s2));
    const float inv = some ? rcp_fast(tot) : 0.f;
    const float lse = some ? m + logf(tot) : 0.f;
    if (sub == 0) zacc += lse * lse;
    const float caz = ca * inv, lin = (cz * lse - caz * s) * inv;
    const f2 inv2 = pack2(inv, inv), caz2 = pack2(caz, caz), lin2 = pack2(lin, lin);
#pragma unroll
    for (int p = 0; p < 2 * NV; ++p) {
      acc[p] = fma2(x[p], inv2, acc[p]);
      x[p] = mul2(x[p], fma2(caz2, g[p], lin2));
    }
    if (a.d_logits && t < T) store_row<LANES, NV, VEC, WHOLE>(a.d_logits + (size_t)t * E, E, sub, x);
    if (with_dw) {
      // The chosen columns are stored once more with the routing weights' share, by the lane
      // that holds the choice, from the choice's own logit.  Choices that repeat an expert, or
      // more of them than lanes, are added to the stored row by one lane in order instead.
      const bool live = real && some, mine = live && (uint32_t)id0 < (uint32_t)E;
      const uint32_t c0 = t * k;
      float wd = mine ? w0 * dw0 : 0.f;
      if (k > LANES && live)
        for (int j = sub + LANES; j < k; j += LANES)
          if ((uint32_t)a.ids[c0 + j] < (uint32_t)E) wd += a.w[c0 + j] * a.dw[c0 + j];
      wd = group_sum<LANES>(wd);
      const unsigned same = __match_any_sync(kAll, mine ? (grp << 16) + id0 : (int)(0x80000000u + lane));
      const bool one_by_one = __any_sync(kAll, k > LANES || (same & (same - 1)) != 0);
      __syncwarp();  // the row's stores come before these
      if (!one_by_one) {
        if (mine)
          a.d_logits[(size_t)t * E + id0] =
              exp2_fast((l0 - m0) * 1.44269504f) * (caz * gs[id0] + lin) + w0 * (dw0 - wd);
      } else if (live && sub == 0) {
        float* d = a.d_logits + (size_t)t * E;
        for (int j = 0; j < k; ++j) {
          const int e = a.ids[c0 + j];
          if ((uint32_t)e < (uint32_t)E) d[e] += a.w[c0 + j] * (a.dw[c0 + j] - wd);
        }
      }
    }
    t += step;
    if (t < T) l0 = chosen(t);
  }

  // column sums of the block: groups of a warp by shuffles, warps through shared memory
  __syncthreads();
#pragma unroll
  for (int p = 0; p < 2 * NV; ++p)
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      float v = half ? hi2(acc[p]) : lo2(acc[p]);
#pragma unroll
      for (int o = LANES; o < 32; o <<= 1) v += __shfl_xor_sync(kAll, v, o);
      if (grp == 0) sums[(size_t)warp * kCols + col_of<LANES, VEC>(sub, p, half)] = v;
    }
  const float z = block_sum<kThreads>(zacc, red);  // its barriers also publish the warps' sums
  float* part = ws.part + (size_t)blockIdx.x * pitch;  // rows of partial sums, their pad words zero
  float* zpart = ws.part + (size_t)kMaxPassBlocks * pitch;
  for (int e = tid; e < (CLUSTER ? E : pitch); e += kThreads) {
    float s = 0.f;
    if (e < E)
#pragma unroll
      for (int i = 0; i < kWarps; ++i) s += sums[(size_t)i * kCols + e];
    if (CLUSTER) mine[e] = s;
    else part[e] = s;
  }
  float bal = 0.f, zs = 0.f;
  if (CLUSTER) {
    if (tid == 0) z_sh = z;
    if (gridDim.x > 1) tc::cluster_sync();
    else __syncthreads();
    if (blockIdx.x == 0) {
      for (int e = tid; e < E; e += kThreads) {
        float s = 0.f;
#pragma unroll 1
        for (uint32_t r = 0; r < gridDim.x; ++r) s += ld_cluster_f32(mine + e, r);
        s *= inv_n;
        if (a.prob_mean) a.prob_mean[e] = s;
        bal += (gs[e] + 1.f) * s;
      }
#pragma unroll 1
      for (uint32_t r = 0; r < gridDim.x; ++r) zs += ld_cluster_f32(&z_sh, r);
      zs *= inv_n;
    }
    if (gridDim.x > 1) tc::cluster_sync();  // no block leaves before its sums are read
    if (blockIdx.x != 0) return;
  } else if (kFinish) {
    if (tid == 0) zpart[blockIdx.x] = z;
    return;
  } else {
    if (tid == 0) zpart[blockIdx.x] = z;
    __threadfence();
    __syncthreads();
    if (tid == 0) last = atomicAdd(ws.ticket, 1u) == gridDim.x - 1;
    __syncthreads();
    if (!last) return;
    __threadfence();
    // the last block: four columns a thread, kRowsAt threads sharing a column's blocks, eight
    // blocks in flight
    constexpr int kAcross = kCols / 4, kRowsAt = kThreads / kAcross < 32 ? kThreads / kAcross : 32, kBatch = 8;
    const int c = (tid % kAcross) * 4, r0 = tid / kAcross;
    float4 s4 = make_float4(0.f, 0.f, 0.f, 0.f);
    if (c < E && r0 < kRowsAt)
      for (unsigned b0 = r0; b0 < gridDim.x; b0 += kRowsAt * kBatch) {
        float4 v[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const unsigned b = b0 + i * kRowsAt;
          v[i] = b < gridDim.x ? __ldcg(reinterpret_cast<const float4*>(ws.part + (size_t)b * pitch + c))
                               : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          s4.x += v[i].x;
          s4.y += v[i].y;
          s4.z += v[i].z;
          s4.w += v[i].w;
        }
      }
    zs = tid < gridDim.x ? __ldcg(zpart + tid) : 0.f;
    zs = block_sum<kThreads>(zs, red) * inv_n;
    if (r0 < kRowsAt) *reinterpret_cast<float4*>(sums + (size_t)r0 * kCols + c) = s4;
    __syncthreads();
    for (int e = tid; e < E; e += kThreads) {
      float s = 0.f;
#pragma unroll 8
      for (int i = 0; i < kRowsAt; ++i) s += sums[(size_t)i * kCols + e];
      s *= inv_n;
      if (a.prob_mean) a.prob_mean[e] = s;
      bal += (gs[e] + 1.f) * s;
    }
  }
  bal = block_sum<kThreads>(bal, red);
  if (tid == 0) store_loss(a, bal, zs);
}

// The column sums of the pass's blocks, added in order, and the losses from them.  One cluster whose
// blocks own a range of columns each, four of them a thread, the other threads sharing the rows.
__global__ void __launch_bounds__(kFinishThreads) router_finish_kernel(RouterLoss a, int rows) {
  constexpr int kBatch = 8;
  __shared__ float4 sums[kFinishThreads];
  __shared__ float red[kFinishThreads / 32];
  __shared__ float bal_sh;
  moe::wait_for_stream();
  moe::let_next_start();
  const int E = a.E, pitch = part_pitch(E), tid = threadIdx.x;
  const Ws ws = carve(a.ws, E);
  const int per = (pitch / 4 + gridDim.x - 1) / gridDim.x;  // vectors of four columns of this block
  const int across = kFinishThreads / per, c = (blockIdx.x * per + tid % per) * 4, r0 = tid / per;
  const int n = ws.total[E];
  const float inv_n = n > 0 ? 1.f / (float)n : 0.f;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  if (c < pitch && r0 < across)
    for (int b0 = r0; b0 < rows; b0 += across * kBatch) {
      float4 v[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int b = b0 + i * across;
        v[i] = b < rows ? __ldcg(reinterpret_cast<const float4*>(ws.part + (size_t)b * pitch + c)) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        s.x += v[i].x;
        s.y += v[i].y;
        s.z += v[i].z;
        s.w += v[i].w;
      }
    }
  const float z = blockIdx.x == 0 && tid < rows ? __ldcg(ws.part + (size_t)kMaxPassBlocks * pitch + tid) : 0.f;
  int cnt[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) cnt[i] = tid < per && c + i < E ? ws.total[c + i] : 0;
  sums[tid] = s;
  __syncthreads();
  float bal = 0.f;
  if (tid < per && c < pitch) {
#pragma unroll 8
    for (int r = 1; r < across; ++r) {
      const float4 v = sums[r * per + tid];
      s.x += v.x;
      s.y += v.y;
      s.z += v.z;
      s.w += v.w;
    }
    const float p[4] = {s.x * inv_n, s.y * inv_n, s.z * inv_n, s.w * inv_n};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (c + i < E) {
        if (a.prob_mean) a.prob_mean[c + i] = p[i];
        bal += (g_of(E, a.k, n, cnt[i]) + 1.f) * p[i];
      }
  }
  bal = block_sum<kFinishThreads>(bal, red);
  const float zs = block_sum<kFinishThreads>(z, red) * inv_n;
  if (tid == 0) bal_sh = bal;
  if (gridDim.x > 1) tc::cluster_sync();
  if (blockIdx.x == 0 && tid == 0) {
    for (uint32_t r = 1; r < gridDim.x; ++r) bal += ld_cluster_f32(&bal_sh, r);
    store_loss(a, bal, zs);
  }
  if (gridDim.x > 1) tc::cluster_sync();
}

template <int LANES, int NV, bool VEC, bool WHOLE>
cudaError_t launch_pass(RouterLoss a, cudaStream_t stream) {
  constexpr int kCols = 4 * NV * LANES, kThreads = pass_threads(NV), kWarps = kThreads / 32;
  constexpr int kRows = kWarps * (32 / LANES);  // rows of a block per turn
  constexpr size_t kSmem = 4 * (2 * kCols + (kWarps * kCols > 4 * kThreads ? kWarps * kCols : 4 * kThreads));
  const int64_t turns = (a.T + kRows - 1) / kRows;  // of one block alone
  const bool cluster = turns <= kClusterBlocks;
  auto kern = cluster ? router_pass_kernel<LANES, NV, VEC, WHOLE, true> : router_pass_kernel<LANES, NV, VEC, WHOLE, false>;
  if (kSmem > 48 * 1024) {
    static std::atomic<uint64_t> sized[2] = {};
    const cudaError_t err = moe_launch::allow_smem(reinterpret_cast<const void*>(kern), (int)kSmem, sized[cluster]);
    if (err != cudaSuccess) return err;
  }
  if (cluster) {
    const int c = (int)(turns < 1 ? 1 : turns);
    return moe_launch::launch_staged(kern, dim3((unsigned)c), dim3(kThreads), kSmem, stream, c, a);
  }
  int64_t blocks = (a.T * a.k + 4095) / 4096;
  if (blocks > kMaxCountBlocks) blocks = kMaxCountBlocks;
  const int64_t per = ((a.T + blocks - 1) / blocks + 3) / 4 * 4;  // ids of a block start on 16 bytes
  a.count_blocks = (int)((a.T + per - 1) / per);
  const cudaError_t err = moe_launch::launch_staged(router_count_kernel, dim3((unsigned)a.count_blocks), dim3(kCountThreads),
                                                    (size_t)a.E * 4, stream, 1, a, per);
  if (err != cudaSuccess) return err;
  int64_t cap = moe_launch::sm_count_current();
  if (cap > kMaxPassBlocks) cap = kMaxPassBlocks;
  // the pass's first loads run under the counts, which it then waits for
  const unsigned pass = (unsigned)(turns < cap ? turns : cap);
  const cudaError_t passed = moe_launch::launch_staged(kern, dim3(pass), dim3(kThreads), kSmem, stream, 1, a);
  if (NV <= 4 || passed != cudaSuccess) return passed;
  return moe_launch::launch_staged(router_finish_kernel, dim3(kClusterBlocks), dim3(kFinishThreads), 0, stream, kClusterBlocks, a,
                                   (int)pass);
}

template <int LANES, int NV>
cudaError_t launch_rows(const RouterLoss& a, cudaStream_t s) {
  if (a.E % 4) return launch_pass<LANES, NV, false, false>(a, s);
  return a.E == 4 * NV * LANES ? launch_pass<LANES, NV, true, true>(a, s) : launch_pass<LANES, NV, true, false>(a, s);
}

// The fewest lanes that hold a row at sixteen values each (32 above 512 experts): fewer lanes mean
// fewer shuffle steps per row and more rows in flight per warp.  Above 16 experts at least eight,
// so that each of up to eight choices has a lane of its own.
cudaError_t launch(const RouterLoss& a, cudaStream_t s) {
  const int E = a.E;
  if (E <= 16) return launch_rows<4, 1>(a, s);
  if (E <= 32) return launch_rows<8, 1>(a, s);
  if (E <= 64) return launch_rows<8, 2>(a, s);
  if (E <= 128) return launch_rows<8, 4>(a, s);
  if (E <= 256) return launch_rows<16, 4>(a, s);
  if (E <= 512) return launch_rows<32, 4>(a, s);
  return launch_rows<32, 8>(a, s);
}

}  // namespace

namespace moe_launch {

size_t router_loss_workspace_bytes(int E) {
  return 512 + (size_t)(kMaxCountBlocks + 1) * count_pitch(E) * 4 + (size_t)kMaxPassBlocks * (part_pitch(E) + 1) * 4;
}

cudaError_t router_loss(const RouterLoss& a, cudaStream_t stream) {
  return launch(a, stream);
}

}  // namespace moe_launch
