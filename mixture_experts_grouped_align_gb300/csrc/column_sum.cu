// Column sums of a bf16 matrix: the gradient of a bias that every row was given,
// d_b[n] = sum_m dz[m, n], in fp32.
//
// A stream of 2 M N bytes.  A cluster of eight CTAs owns 128 columns and shares the rows among
// its CTAs; a thread adds eight columns (16 bytes a row) of every sixteenth row of its share,
// eight rows in flight.  The sixteen row groups of a CTA and then the eight CTAs (distributed
// shared memory) are added in order: the same bits every time, one launch, no workspace.
#include "moe_common.cuh"
#include "moe_launch.h"
#include "tcgen05.cuh"

namespace {

constexpr int kThreads = 256, kCols = 128, kSplit = 8;

template <bool VEC>
__global__ void __cluster_dims__(kSplit, 1, 1) __launch_bounds__(kThreads)
    column_sum_kernel(const uint16_t* __restrict__ x, int64_t M, int64_t N, float* __restrict__ out) {
  __shared__ float part[16][kCols];
  __shared__ float mine[kCols];
  const int tid = threadIdx.x, cg = tid & 15, rg = tid >> 4;
  const int rank = (int)tc::cluster_ctarank();
  const int64_t n0 = (int64_t)(blockIdx.x / kSplit) * kCols + cg * 8;
  const int64_t r0 = M * rank / kSplit, r1 = M * (rank + 1) / kSplit;
  float acc[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = 0.f;
  constexpr int kU = 8;
  for (int64_t r = r0 + rg; r < r1; r += 16 * kU) {
    uint32_t v[kU][4];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int64_t m = r + 16 * u;
#pragma unroll
      for (int i = 0; i < 4; ++i) v[u][i] = 0;
      if (m < r1) {
        if (VEC) {
          if (n0 < N) {
            const uint4 w = __ldcs(reinterpret_cast<const uint4*>(x + m * N + n0));
            v[u][0] = w.x; v[u][1] = w.y; v[u][2] = w.z; v[u][3] = w.w;
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (n0 + i < N) v[u][i >> 1] |= (uint32_t)x[m * N + n0 + i] << (16 * (i & 1));
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kU; ++u)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc[2 * i] += __uint_as_float(v[u][i] << 16);
        acc[2 * i + 1] += __uint_as_float(v[u][i] & 0xffff0000u);
      }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) part[rg][cg * 8 + i] = acc[i];
  __syncthreads();
  if (tid < kCols) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) s += part[i][tid];
    mine[tid] = s;
  }
  tc::cluster_sync();
  const int64_t n = (int64_t)(blockIdx.x / kSplit) * kCols + tid;
  if (rank == 0 && tid < kCols && n < N) {
    float s = 0.f;
    for (int r = 0; r < kSplit; ++r) {
      uint32_t a;
      float v;
      asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(tc::smem_addr(&mine[tid])), "r"(r));
      asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
      s += v;
    }
    out[n] = s;
  }
  tc::cluster_sync();
}

}  // namespace

namespace moe_launch {

cudaError_t column_sum(const void* x, int64_t M, int64_t N, float* out, cudaStream_t stream) {
  const int64_t blocks = (N + kCols - 1) / kCols * kSplit;
  if (N % 8 == 0)
    column_sum_kernel<true><<<(unsigned)blocks, kThreads, 0, stream>>>(static_cast<const uint16_t*>(x), M, N, out);
  else
    column_sum_kernel<false><<<(unsigned)blocks, kThreads, 0, stream>>>(static_cast<const uint16_t*>(x), M, N, out);
  return cudaGetLastError();
}

}  // namespace moe_launch
