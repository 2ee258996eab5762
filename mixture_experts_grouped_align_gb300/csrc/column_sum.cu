// Column sums of a bf16 matrix: the gradient of a bias that every row was given,
// d_b[n] = sum_m dz[m, n], in fp32.
//
// A stream of 2 M N bytes.  A cluster of eight CTAs owns 64 columns (one 128-byte line of a row),
// or 32, and shares the rows among its CTAs; a thread adds eight columns (16 bytes a row) of
// every 32nd (64th) row of its share, eight rows in flight, the last ones included.  The row
// groups of a CTA and then the eight CTAs (distributed shared memory) are added in order: the
// same bits every time, one launch, no workspace.
//
// Measured: 8191 x 4096 13.6 us (5.0 TB/s), 60000 x 2048 42 us (5.8 TB/s), 16000 x 64 4.0 us.  Bound
// by HBM for long matrices; for short ones by the loads in flight that the columns leave.
#include "moe_common.cuh"
#include "moe_launch.h"
#include "tcgen05.cuh"

namespace {

constexpr int kThreads = 256, kSplit = 8;

__device__ __forceinline__ void add8(float (&acc)[8], const uint4& v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    acc[2 * i] += __uint_as_float(w[i] << 16);
    acc[2 * i + 1] += __uint_as_float(w[i] & 0xffff0000u);
  }
}

// VEC: rows are whole 16-byte units.
template <int kCols, bool VEC>
__global__ void __launch_bounds__(kThreads)
    column_sum_kernel(const uint16_t* __restrict__ x, int64_t M, int64_t N, float* __restrict__ out) {
  moe::wait_for_stream();
  moe::let_next_start();
  constexpr int kLanes = kCols / 8, kGroups = kThreads / kLanes;
  __shared__ float part[kGroups][kCols];
  __shared__ float mine[kCols];
  const int tid = threadIdx.x, cg = tid % kLanes, rg = tid / kLanes;
  const int rank = (int)tc::cluster_ctarank();
  const int64_t n0 = (int64_t)(blockIdx.x / kSplit) * kCols + cg * 8;
  const int64_t r1 = M * (rank + 1) / kSplit;
  int64_t r = M * rank / kSplit + rg;
  float acc[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = 0.f;
  if (VEC) {
    constexpr int kU = 8;
    if (n0 < N) {
      const uint4* p = reinterpret_cast<const uint4*>(x + r * N + n0);
      const int64_t step = kGroups * N / 8;
      for (; r + (kU - 1) * kGroups < r1; r += kU * kGroups, p += kU * step) {
        uint4 v[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) v[u] = __ldcs(p + u * step);
#pragma unroll
        for (int u = 0; u < kU; ++u) add8(acc, v[u]);
      }
      if (r < r1) {  // the last rows, together as well
        uint4 v[kU - 1];
#pragma unroll
        for (int u = 0; u < kU - 1; ++u) v[u] = r + u * kGroups < r1 ? __ldcs(p + u * step) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int u = 0; u < kU - 1; ++u) add8(acc, v[u]);
      }
    }
  } else {
    for (; r < r1; r += kGroups)
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (n0 + i < N) acc[i] += moe::bf16_bits_to_f32(x[r * N + n0 + i]);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) part[rg][cg * 8 + i] = acc[i];
  __syncthreads();
  if (tid < kCols) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kGroups; ++i) s += part[i][tid];
    mine[tid] = s;
  }
  tc::cluster_sync();
  const int64_t n = (int64_t)(blockIdx.x / kSplit) * kCols + tid;
  if (rank == 0 && tid < kCols && n < N) {
    float v[kSplit];
#pragma unroll
    for (int r = 0; r < kSplit; ++r) {
      uint32_t a;
      asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(tc::smem_addr(&mine[tid])), "r"(r));
      asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v[r]) : "r"(a) : "memory");
    }
#pragma unroll
    for (int r = 1; r < kSplit; ++r) v[0] += v[r];
    out[n] = v[0];
  }
  tc::cluster_sync();
}

}  // namespace

namespace moe_launch {

cudaError_t column_sum(const void* x, int64_t M, int64_t N, float* out, cudaStream_t stream) {
  // Few columns and many rows: 32 columns a cluster, for twice the CTAs (60000 x 2048: 60 us with 64,
  // 42 with 32; 8191 x 2688: 11.6 and 10.2; 16000 x 64: 6.0 and 4.0).  Else whole lines are read faster
  // and there are fewer clusters to meet (8191 x 4096: 13.6 us with 64, 17.0 with 32; 1000 x 2880: 3.6
  // and 4.5).
  const int64_t wide = (N + 63) / 64 * kSplit;
  const bool narrow = M >= 2000 && 4 * wide <= 9 * sm_count_current();
  const int64_t blocks = narrow ? (N + 31) / 32 * kSplit : wide;
  const bool vec = N % 8 == 0;
  const auto kern = narrow ? (vec ? column_sum_kernel<32, true> : column_sum_kernel<32, false>)
                           : (vec ? column_sum_kernel<64, true> : column_sum_kernel<64, false>);
  return launch_staged(kern, dim3((unsigned)blocks), dim3(kThreads), 0, stream, kSplit, static_cast<const uint16_t*>(x), M, N,
                       out);
}

}  // namespace moe_launch
