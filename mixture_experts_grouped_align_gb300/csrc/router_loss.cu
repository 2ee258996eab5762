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
// Two launches: the counts (T k ids), then the pass; a batch of at most kOneBlockElems logits
// is one launch of one block, which counts for itself.
//
// The pass gives a row to LANES lanes (8, 16 or 32: the fewest that hold it at four values a
// lane, then NV vectors of four a lane) and keeps it in registers from the load to the store.
// Every lane keeps the column sums of its own columns over its rows; blocks add theirs in a
// fixed order into one row of partial sums each, and the last block to finish adds those rows
// in order, so that repeated calls give the same bits (no floating-point atomics).
#include "moe_common.cuh"
#include "moe_launch.h"

namespace {

using moe_launch::RouterLoss;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCountBlocks = 64;
constexpr int64_t kOneBlockElems = 16384;
constexpr unsigned kAll = 0xffffffffu;

// Workspace: ticket (256 bytes) | counts of the count blocks [kMaxCountBlocks][E + 1] (the last
// word: its real tokens) | partial sums of the pass [blocks][E + 1] (the last word: sum lse^2).
struct Ws {
  unsigned* ticket;
  int* counts;
  float* part;
};
__host__ __device__ inline Ws carve(void* ws, int E) {
  uint8_t* p = static_cast<uint8_t*>(ws);
  Ws w;
  w.ticket = reinterpret_cast<unsigned*>(p);
  w.counts = reinterpret_cast<int*>(p + 256);
  w.part = reinterpret_cast<float*>(p + 256 + (size_t)kMaxCountBlocks * (E + 1) * 4);
  return w;
}

// Counts of tokens [t0, t1) into hist[E] (shared) and their real tokens into *n_real (shared).
__device__ void count_tokens(const RouterLoss& a, int64_t t0, int64_t t1, int* hist, int* n_real) {
  for (int e = threadIdx.x; e < a.E; e += kThreads) hist[e] = 0;
  if (threadIdx.x == 0) *n_real = 0;
  __syncthreads();
  const int64_t p1 = t1 * a.k;
  for (int64_t p = t0 * a.k + threadIdx.x; p < p1; p += kThreads) {
    const int64_t t = p / a.k;
    if (a.mask && a.mask[t] == 0) continue;
    const int id = a.ids[p];
    if (id < 0 || id >= a.E) moe::set_status(a.status, MOE_ERR_INVALID_EXPERT);
    else atomicAdd(&hist[id], 1);
  }
  if (a.mask) {
    int n = 0;
    for (int64_t t = t0 + threadIdx.x; t < t1; t += kThreads) n += a.mask[t] != 0;
    n = __reduce_add_sync(kAll, n);
    if ((threadIdx.x & 31) == 0 && n) atomicAdd(n_real, n);
  } else if (threadIdx.x == 0) {
    *n_real = (int)(t1 - t0);
  }
  __syncthreads();
}

__global__ void __launch_bounds__(kThreads) router_count_kernel(RouterLoss a, int64_t per_block) {
  extern __shared__ int sm_count[];
  __shared__ int n_real;
  const Ws w = carve(a.ws, a.E);
  const int64_t t0 = blockIdx.x * per_block;
  const int64_t t1 = t0 + per_block < a.T ? t0 + per_block : a.T;
  count_tokens(a, t0, t1 > t0 ? t1 : t0, sm_count, &n_real);
  int* out = w.counts + (size_t)blockIdx.x * (a.E + 1);
  for (int e = threadIdx.x; e < a.E; e += kThreads) out[e] = sm_count[e];
  if (threadIdx.x == 0) {
    out[a.E] = n_real;
    if (blockIdx.x == 0) *w.ticket = 0;
  }
}

template <int LANES>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) {
    const float x = __shfl_xor_sync(kAll, v, o);
    v = (v != v || x != x) ? __int_as_float(0x7fc00000) : fmaxf(v, x);
  }
  return v;
}
template <int LANES>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}

// Column of value i (0 .. 4 NV - 1) of lane `sub` of a row's LANES lanes.
template <int LANES, int VEC>
__device__ __forceinline__ int col_of(int sub, int i) {
  return VEC == 4 ? (i >> 2) * 4 * LANES + sub * 4 + (i & 3) : i * LANES + sub;
}

template <int LANES, int NV, int VEC>
__device__ __forceinline__ void load_row(const float* row, int E, int sub, float (&x)[4 * NV]) {
  if (VEC == 4) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = v * 4 * LANES + sub * 4;
      float4 f = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      if (c < E) f = __ldcs(reinterpret_cast<const float4*>(row + c));
      x[4 * v] = f.x; x[4 * v + 1] = f.y; x[4 * v + 2] = f.z; x[4 * v + 3] = f.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4 * NV; ++i) {
      const int c = i * LANES + sub;
      x[i] = c < E ? __ldcs(row + c) : -INFINITY;
    }
  }
}

template <int LANES, int NV, int VEC>
__device__ __forceinline__ void store_row(float* row, int E, int sub, const float (&d)[4 * NV]) {
  if (VEC == 4) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = v * 4 * LANES + sub * 4;
      if (c < E) __stcs(reinterpret_cast<float4*>(row + c), make_float4(d[4 * v], d[4 * v + 1], d[4 * v + 2], d[4 * v + 3]));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4 * NV; ++i) {
      const int c = i * LANES + sub;
      if (c < E) __stcs(row + c, d[i]);
    }
  }
}

// Sum over the block's threads of v (every thread gets it; `red` holds kWarps floats).
__device__ float block_sum(float v, float* red) {
  v = group_sum<32>(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.f;
  for (int i = 0; i < kWarps; ++i) s += red[i];
  return s;
}

// ONE: the grid is one block, which counts the choices itself.
// Shared memory: g [E] | the routing weights' gradient of one row per group [groups][E] (the
// column sums of one warp each at the end, [kWarps][4 NV 32]).
template <int LANES, int NV, int VEC, bool ONE>
__global__ void __launch_bounds__(kThreads) router_pass_kernel(RouterLoss a) {
  constexpr int kGroups = 32 / LANES;       // rows of a warp
  constexpr int kCols = 4 * NV * LANES;     // columns the lanes can hold, >= E
  constexpr int kRows = NV == 1 ? 2 : 1;    // rows in flight per group
  extern __shared__ float sm[];
  __shared__ int n_sh;
  __shared__ unsigned last;
  __shared__ float red[kWarps];
  const int E = a.E, k = a.k;
  float* gs = sm;
  float* up_all = sm + kCols;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, sub = lane % LANES, grp = lane / LANES;
  float* up = up_all + (size_t)(warp * kGroups + grp) * kCols;
  const Ws ws = carve(a.ws, E);

  int* cs = reinterpret_cast<int*>(gs);
  if (ONE) {
    count_tokens(a, 0, a.T, cs, &n_sh);
  } else {
    for (int e = tid; e <= E; e += kThreads) {
      int s = 0;
      for (int b = 0; b < a.count_blocks; ++b) s += ws.counts[(size_t)b * (E + 1) + e];
      if (e == E) n_sh = s;
      else cs[e] = s;
    }
    __syncthreads();
  }
  const int n = n_sh;
  const float inv_n = n > 0 ? 1.f / (float)n : 0.f;
  for (int e = tid; e < kCols; e += kThreads) {
    float g = 0.f;
    if (e < E) {
      const int c = cs[e];
      if (blockIdx.x == 0 && a.counts) a.counts[e] = c;
      if (n > 0) g = (float)((double)((int64_t)E * c - (int64_t)n * k) / (double)((int64_t)n * k));
    }
    gs[e] = g;  // the same word cs[e] was read from, by the same thread
  }
  for (int i = tid; i < kWarps * kGroups * kCols; i += kThreads) up_all[i] = 0.f;
  __syncthreads();

  float acc[4 * NV], zacc = 0.f;
#pragma unroll
  for (int i = 0; i < 4 * NV; ++i) acc[i] = 0.f;
  const float ca = a.balance_coef * inv_n, cz = 2.f * a.z_coef * inv_n;
  const int64_t per = (int64_t)kGroups * kRows;  // rows of a warp per turn
  const int64_t step = (int64_t)gridDim.x * kWarps * per;
  // every lane of a warp makes the same number of turns (the shuffles need them all)
  for (int64_t base = ((int64_t)blockIdx.x * kWarps + warp) * per; base < a.T; base += step) {
    float x[kRows][4 * NV];
    bool in[kRows], real[kRows];
    int id[kRows];
    float w[kRows], dw[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const int64_t t = base + (int64_t)r * kGroups + grp;
      in[r] = t < a.T;
      real[r] = in[r] && (!a.mask || a.mask[t] != 0);
      if (real[r]) {
        load_row<LANES, NV, VEC>(a.logits + t * E, E, sub, x[r]);
      } else {
#pragma unroll
        for (int i = 0; i < 4 * NV; ++i) x[r][i] = -INFINITY;
      }
    }
    const bool with_dw = a.dw != nullptr && a.d_logits != nullptr;
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const int64_t t = base + (int64_t)r * kGroups + grp;
      float m = x[r][0];
#pragma unroll
      for (int i = 1; i < 4 * NV; ++i) m = (m != m || x[r][i] != x[r][i]) ? __int_as_float(0x7fc00000) : fmaxf(m, x[r][i]);
      m = group_max<LANES>(m);
      // a row with nothing left by its mask (all -inf), a pad row or a row past the end: p = 0
      const bool some = m != -INFINITY;
      float p[4 * NV], tot = 0.f;
#pragma unroll
      for (int i = 0; i < 4 * NV; ++i) {
        p[i] = some ? __expf(x[r][i] - m) : 0.f;
        tot += p[i];
      }
      tot = group_sum<LANES>(tot);
      const float inv = some ? 1.f / tot : 0.f;
      const float lse = some ? m + logf(tot) : 0.f;
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < 4 * NV; ++i) {
        p[i] *= inv;
        acc[i] += p[i];
        s += p[i] * gs[col_of<LANES, VEC>(sub, i)];
      }
      s = group_sum<LANES>(s);
      if (sub == 0) zacc += lse * lse;
      if (a.d_logits == nullptr) continue;
      float d[4 * NV];
      const float lin = cz * lse - ca * s;
#pragma unroll
      for (int i = 0; i < 4 * NV; ++i) d[i] = p[i] * (ca * gs[col_of<LANES, VEC>(sub, i)] + lin);
      if (with_dw) {
        // the k choices, one after another (k may exceed the group's lanes); ids of a token may
        // repeat, so each choice's share is added by one lane in the order of j
        float wd = 0.f;
        if (real[r] && some)
          for (int j = sub; j < k; j += LANES) {
            const int e = a.ids[t * k + j];
            if (e >= 0 && e < E) wd += a.w[t * k + j] * a.dw[t * k + j];
          }
        wd = group_sum<LANES>(wd);
        if (real[r] && some && sub == 0)
          for (int j = 0; j < k; ++j) {
            const int e = a.ids[t * k + j];
            if (e >= 0 && e < E) up[e] += a.w[t * k + j] * (a.dw[t * k + j] - wd);
          }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4 * NV; ++i) d[i] += up[col_of<LANES, VEC>(sub, i)];
        __syncwarp();
        if (real[r] && some && sub == 0)
          for (int j = 0; j < k; ++j) {
            const int e = a.ids[t * k + j];
            if (e >= 0 && e < E) up[e] = 0.f;
          }
        __syncwarp();
      }
      if (in[r]) store_row<LANES, NV, VEC>(a.d_logits + t * E, E, sub, d);
    }
  }

  // column sums of the block: groups of a warp by shuffles, warps through shared memory
#pragma unroll
  for (int i = 0; i < 4 * NV; ++i)
#pragma unroll
    for (int o = LANES; o < 32; o <<= 1) acc[i] += __shfl_xor_sync(kAll, acc[i], o);
  __syncthreads();
  if (grp == 0)
#pragma unroll
    for (int i = 0; i < 4 * NV; ++i) up_all[(size_t)warp * kCols + col_of<LANES, VEC>(sub, i)] = acc[i];
  const float z = block_sum(zacc, red);
  __syncthreads();
  float* part = ws.part + (size_t)blockIdx.x * (E + 1);
  for (int e = tid; e < E; e += kThreads) {
    float s = 0.f;
    for (int i = 0; i < kWarps; ++i) s += up_all[(size_t)i * kCols + e];
    part[e] = s;
  }
  if (tid == 0) part[E] = z;
  if (!ONE) {
    __threadfence();
    __syncthreads();
    if (tid == 0) last = atomicAdd(ws.ticket, 1u) == gridDim.x - 1;
    __syncthreads();
    if (!last) return;
    __threadfence();
  } else {
    __syncthreads();
  }
  // the last block: P, and the three losses
  float bal = 0.f;
  for (int e = tid; e < E; e += kThreads) {
    float s = 0.f;
    for (unsigned b = 0; b < gridDim.x; ++b) s += __ldcg(ws.part + (size_t)b * (E + 1) + e);
    s *= inv_n;
    if (a.prob_mean) a.prob_mean[e] = s;
    bal += (gs[e] + 1.f) * s;
  }
  float zs = 0.f;
  for (unsigned b = tid; b < gridDim.x; b += kThreads) zs += __ldcg(ws.part + (size_t)b * (E + 1) + E);
  bal = block_sum(bal, red);
  zs = block_sum(zs, red) * inv_n;
  if (tid == 0) {
    if (n == 0) bal = zs = 0.f;
    // a part whose coefficient is 0 is off, also where its value is infinite
    a.loss[0] = (a.balance_coef != 0.f ? a.balance_coef * bal : 0.f) + (a.z_coef != 0.f ? a.z_coef * zs : 0.f);
    a.loss[1] = bal;
    a.loss[2] = zs;
  }
}

template <int LANES, int NV, int VEC>
cudaError_t launch_pass(const RouterLoss& a, int blocks, bool one, cudaStream_t stream) {
  constexpr int kCols = 4 * NV * LANES;
  const size_t smem = (size_t)kCols * 4 * (1 + kWarps * (32 / LANES));
  auto kern = one ? router_pass_kernel<LANES, NV, VEC, true> : router_pass_kernel<LANES, NV, VEC, false>;
  cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (err != cudaSuccess) return err;
  kern<<<blocks, kThreads, smem, stream>>>(a);
  return cudaGetLastError();
}

template <int VEC>
cudaError_t launch_width(const RouterLoss& a, int blocks, bool one, cudaStream_t s) {
  const int E = a.E;
  if (E <= 32) return launch_pass<8, 1, VEC>(a, blocks, one, s);
  if (E <= 64) return launch_pass<16, 1, VEC>(a, blocks, one, s);
  if (E <= 128) return launch_pass<32, 1, VEC>(a, blocks, one, s);
  if (E <= 256) return launch_pass<32, 2, VEC>(a, blocks, one, s);
  if (E <= 512) return launch_pass<32, 4, VEC>(a, blocks, one, s);
  return launch_pass<32, 8, VEC>(a, blocks, one, s);
}

int pass_blocks(int64_t T, int E) {
  const int lanes = E <= 32 ? 8 : (E <= 64 ? 16 : 32);
  const int64_t rows = (int64_t)kWarps * (32 / lanes) * (E <= 128 ? 2 : 1);
  const int64_t need = (T + rows - 1) / rows, cap = (int64_t)moe_launch::sm_count_current() * 2;
  return (int)(need < 1 ? 1 : (need < cap ? need : cap));
}

}  // namespace

namespace moe_launch {

size_t router_loss_workspace_bytes(int E) {
  // the partial sums of at most two blocks per SM (up to 256 SMs)
  return 256 + (size_t)kMaxCountBlocks * (E + 1) * 4 + (size_t)512 * (E + 1) * 4;
}

cudaError_t router_loss(RouterLoss a, cudaStream_t stream) {
  const bool one = a.T * a.E <= kOneBlockElems;
  if (!one) {
    int64_t blocks = (a.T * a.k + 4095) / 4096;
    if (blocks > kMaxCountBlocks) blocks = kMaxCountBlocks;
    const int64_t per = (a.T + blocks - 1) / blocks;
    a.count_blocks = (int)blocks;
    router_count_kernel<<<(unsigned)blocks, kThreads, (size_t)a.E * 4, stream>>>(a, per);
    const cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess) return err;
  }
  int blocks = one ? 1 : pass_blocks(a.T, a.E);
  if (blocks > 512) blocks = 512;
  return a.E % 4 == 0 ? launch_width<4>(a, blocks, one, stream) : launch_width<1>(a, blocks, one, stream);
}

}  // namespace moe_launch
