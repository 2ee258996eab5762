// The dense product (dense_gemm.cu) where its 128 x 256 tiles would leave SMs idle: few rows,
// or few columns.
//
// Bound with few rows: reading W once.  A tile is 128 features x BN rows of x with the roles of
// the operands exchanged (A = the 128 weight rows, B = the rows of x), so that one row of x
// costs an MMA of N = 16 and not of M = 128.  K is split over the C CTAs of a cluster, which
// makes tiles x C CTAs pull on W at once; each accumulates its share in TMEM, leaves it in its
// shared memory as fp32 (token-major, so that lanes are consecutive features), and the C shares
// are added in rank order through distributed shared memory by the CTA that stores the row: no
// workspace, no second launch, the same bits every time.  SwiGLU keeps two accumulators (gate
// and up features in the same lane).
//   warp 0 loads stages (64 of K: the weight tile(s), BN rows of x) by TMA, as many stages as
//   fit; warp 1 issues the MMAs; then all eight warps drain, add and store.
#include "dense_common.cuh"

namespace {

using namespace dense;

constexpr int kThreads = 256;
constexpr int kFeat = 128;
constexpr int kMaxStages = 12;
constexpr int kRing = 208 * 1024;  // shared memory of the stages, at most

struct Split {
  int BN;        // rows of x per tile: 16, 32, 64, 128 or (not SwiGLU) 256
  int C;         // CTAs of a cluster: the shares of K
  int stages;
  int slot;      // bytes of a stage
  int smem;
  int cols;      // TMEM columns
  int64_t n_tiles, m_tiles;
};

__device__ __forceinline__ float2 ld_cluster_f2(uint32_t addr, uint32_t rank) {
  uint32_t a;
  float2 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a) : "memory");
  return v;
}

template <bool GATED>
__global__ void __launch_bounds__(kThreads, 1)
    dense_split_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w, Dense d,
                       Split sp) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ uint64_t full[kMaxStages], empty[kMaxStages], done;
  __shared__ uint32_t taddr_s;
  __shared__ volatile int abort_flag;
  constexpr int kNA = GATED ? 2 : 1;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = sp.C > 1 ? (int)tc::cluster_ctarank() : 0;
  if (tid == 0) {
    for (int s = 0; s < sp.stages; ++s) {
      tc::mbar_init(&full[s], 1);
      tc::mbar_init(&empty[s], 1);
    }
    tc::mbar_init(&done, 1);
    abort_flag = 0;
    tc::mbar_fence_init();
  }
  if (warp == 1) {
    tc::tmem_alloc(&taddr_s, sp.cols);
    tc::tmem_relinquish();
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t taddr = taddr_s, smem_s = tc::smem_addr(smem);
  const bool kn = d.w_kn != 0;
  const uint64_t wb = d.wait_ns > 0 ? (uint64_t)d.wait_ns : tc::kWaitNs;
  const int64_t tile = blockIdx.x / sp.C;
  const int64_t nt = tile % sp.n_tiles, mt = tile / sp.n_tiles;
  const int nk = (d.K + kBK - 1) / kBK;
  const int k0 = (int)((int64_t)nk * rank / sp.C), k1 = (int)((int64_t)nk * (rank + 1) / sp.C);
  const int kx = kNA * kFeat * 128;  // x rows of a stage, behind the weight tiles

  if (warp == 0 && lane == 0 && !d.stall) {
    int issued = 0;
    for (int kb = k0; kb < k1; ++kb) {
      const int it = kb - k0, s = it % sp.stages;
      if (!tc::mbar_wait(&empty[s], ((it / sp.stages) & 1) ^ 1, wb)) {
        moe::set_status(d.status, MOE_ERR_TIMEOUT);
        abort_flag = 1;
        break;
      }
      issued = it + 1;
      const uint32_t sl = smem_s + s * sp.slot;
      tma::mbar_arrive_expect_tx(&full[s], (uint32_t)(kx + sp.BN * 128));
      load_w(sl, &tm_w, kn, nt * kFeat, kFeat, kb, &full[s]);
      if (GATED) load_w(sl + kFeat * 128, &tm_w, kn, d.N + nt * kFeat, kFeat, kb, &full[s]);
      tma::load_2d(sl + kx, &tm_x, kb * 128, (int32_t)(mt * sp.BN), &full[s]);
    }
    // every load lands before the block may end, also when another role has given up
    for (int j = issued > sp.stages ? issued - sp.stages : 0; j < issued; ++j)
      if (!tc::mbar_wait(&full[j % sp.stages], (j / sp.stages) & 1, wb)) {
        moe::set_status(d.status, MOE_ERR_TIMEOUT);
        abort_flag = 1;
      }
  } else if (warp == 1 && lane == 0 && !d.stall) {
    const uint32_t idesc = tc::idesc_f16(kFeat, sp.BN, 1) | (kn ? 1u << 15 : 0u);
    for (int kb = k0; kb < k1; ++kb) {
      const int it = kb - k0, s = it % sp.stages;
      if (!tc::mbar_wait(&full[s], (it / sp.stages) & 1, wb)) {
        moe::set_status(d.status, MOE_ERR_TIMEOUT);
        abort_flag = 1;
        break;
      }
      tc::tc_fence_after();
      const uint32_t sl = smem_s + s * sp.slot;
#pragma unroll
      for (int a = 0; a < kNA; ++a)
#pragma unroll
        for (int j = 0; j < kBK / 16; ++j)
          tc::mma_f16_ss(taddr + a * sp.BN, w_desc(sl + a * kFeat * 128, kn, j), tc::sdesc_sw128(sl + kx + j * 32), idesc,
                         it > 0 || j > 0);
      tc::mma_commit(&empty[s]);
    }
    tc::mma_commit(&done);
  }
  __syncwarp();
  bool ok = true;
  // every thread waits for the last product (the loader's lane too: a timeout ends its loop)
  if (!tc::mbar_wait(&done, 0, wb)) {
    moe::set_status(d.status, MOE_ERR_TIMEOUT);
    ok = false;
  }
  if (abort_flag) ok = false;
  tc::tc_fence_after();
  // the accumulators -> this CTA's shared memory, [accumulator][token][feature] fp32 (the ring
  // is free: every load has landed and every product has read it)
  float* part = reinterpret_cast<float*>(smem);
  const int feat = (warp & 3) * 32 + lane;
  const int64_t m0 = mt * sp.BN;
  const int rows = d.M - m0 < sp.BN ? (int)(d.M - m0) : sp.BN;
  if (ok) {
    const uint32_t tb = taddr + ((uint32_t)((warp & 3) * 32) << 16);
    // warps 0-3 take the even groups of 16 columns, warps 4-7 the odd ones
    for (int a = 0; a < kNA; ++a)
      for (int c = (warp >> 2) * 16; c < sp.BN; c += 32) {
        if (c >= rows) break;  // tokens past M: nothing is read of them
        uint32_t v[16];
        asm volatile(
            "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
            "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
            : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
              "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
            : "r"(tb + a * sp.BN + c));
        tc::tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 16; ++j) part[((size_t)a * sp.BN + c + j) * kFeat + feat] = __uint_as_float(v[j]);
      }
  }
  tc::tc_fence_before();
  if (sp.C > 1) tc::cluster_sync();
  else __syncthreads();
  if (warp == 1) {
    tc::tc_fence_after();
    tc::tmem_dealloc(taddr, sp.cols);
  }
  // rows rank, rank + C, ... of the tile: four rows at a time, two features a thread
  if (ok) {
    const int f = (tid & 63) * 2;
    const int64_t n = nt * kFeat + f;
    const uint32_t base = tc::smem_addr(part);
    float b0 = 0.f, b1 = 0.f, u0 = 0.f, u1 = 0.f;
    if (d.bias) {
      if (n < d.N) b0 = bias_at(d.bias, n);
      if (n + 1 < d.N) b1 = bias_at(d.bias, n + 1);
      if (GATED && n < d.N) u0 = bias_at(d.bias, d.N + n);
      if (GATED && n + 1 < d.N) u1 = bias_at(d.bias, d.N + n + 1);
    }
    for (int t = rank + sp.C * (tid >> 6); t < rows; t += sp.C * 4) {
      float2 z = make_float2(0.f, 0.f), u = make_float2(0.f, 0.f);
      const uint32_t at = base + (uint32_t)(t * kFeat + f) * 4;
      for (int r = 0; r < sp.C; ++r) {
        const float2 v = ld_cluster_f2(at, r);
        z.x += v.x;
        z.y += v.y;
        if (GATED) {
          const float2 w = ld_cluster_f2(at + (uint32_t)(sp.BN * kFeat * 4), r);
          u.x += w.x;
          u.y += w.y;
        }
      }
      z.x += b0;
      z.y += b1;
      if (GATED) {
        z.x = moe::silu(z.x) * (u.x + u0);
        z.y = moe::silu(z.y) * (u.y + u1);
      } else if (d.relu2) {
        z.x = moe::relu2(z.x);
        z.y = moe::relu2(z.y);
      }
      const int64_t at_o = (m0 + t) * d.N + n;
      if (n + 1 < d.N && d.N % 2 == 0) {
        if (d.out_f32) {
          if (d.residual) {
            const float2 r = *reinterpret_cast<const float2*>(static_cast<const float*>(d.residual) + at_o);
            z.x += d.residual_scale * r.x;
            z.y += d.residual_scale * r.y;
          }
          *reinterpret_cast<float2*>(static_cast<float*>(d.out) + at_o) = z;
        } else {
          if (d.residual) {
            const uint32_t r = *reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(d.residual) + at_o);
            z.x += d.residual_scale * __uint_as_float(r << 16);
            z.y += d.residual_scale * __uint_as_float(r & 0xffff0000u);
          }
          *reinterpret_cast<__nv_bfloat162*>(static_cast<uint16_t*>(d.out) + at_o) = __floats2bfloat162_rn(z.x, z.y);
        }
      } else {
        const float zz[2] = {z.x, z.y};
        for (int i = 0; i < 2; ++i)
          if (n + i < d.N) {
            const float o = zz[i] + (d.residual ? d.residual_scale * residual_at(d, at_o + i) : 0.f);
            if (d.out_f32) static_cast<float*>(d.out)[at_o + i] = o;
            else static_cast<uint16_t*>(d.out)[at_o + i] = moe::f32_to_bf16_bits(o);
          }
      }
    }
  }
  if (sp.C > 1) tc::cluster_sync();  // no CTA leaves while another still reads its share
}

int tile_rows(const Dense& d) {
  const int most = d.gated ? 128 : 256;
  int bn = 16;
  while (bn < most && bn < d.M) bn *= 2;
  return bn;
}

Split plan(const Dense& d) {
  Split s{};
  const int64_t sms = moe_launch::sm_count_current();
  s.BN = tile_rows(d);
  s.n_tiles = (d.N + kFeat - 1) / kFeat;
  s.m_tiles = (d.M + s.BN - 1) / s.BN;
  const int64_t tiles = s.n_tiles * s.m_tiles, nk = (d.K + kBK - 1) / kBK;
  int64_t c = sms / tiles;
  if (c > 8) c = 8;
  if (c > nk) c = nk;
  s.C = c < 1 ? 1 : (int)c;
  s.slot = ((d.gated ? 2 : 1) * kFeat + s.BN) * 128;
  s.stages = kRing / s.slot;
  if (s.stages > kMaxStages) s.stages = kMaxStages;
  const int share = (int)((nk + s.C - 1) / s.C);
  if (s.stages > share) s.stages = share;
  const int part = (d.gated ? 2 : 1) * s.BN * kFeat * 4;
  s.smem = (s.stages * s.slot > part ? s.stages * s.slot : part) + 1024;
  s.cols = 32;
  while (s.cols < (d.gated ? 2 : 1) * s.BN) s.cols *= 2;
  return s;
}

template <bool GATED>
cudaError_t launch(const Dense& d, const Split& s, cudaStream_t stream) {
  const uint64_t K2 = (uint64_t)d.K * 2, N1 = GATED ? 2 * (uint64_t)d.N : (uint64_t)d.N;
  CUtensorMap mx{}, mw{};
  if (!tma::encode_2d_u8(&mx, d.x, K2, (uint64_t)d.M, K2, 128, (uint32_t)s.BN, true)) return cudaErrorInvalidValue;
  const bool okw = d.w_kn ? tma::encode_2d_u8(&mw, d.w, N1 * 2, (uint64_t)d.K, N1 * 2, 128, kBK, true)
                          : tma::encode_2d_u8(&mw, d.w, K2, N1, K2, 128, kFeat, true);
  if (!okw) return cudaErrorInvalidValue;
  auto kern = dense_split_kernel<GATED>;
  cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kRing + 1024);
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(s.n_tiles * s.m_tiles * s.C));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = s.smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = s.C;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  err = cudaLaunchKernelEx(&cfg, kern, mx, mw, d, s);
  return err == cudaSuccess ? cudaGetLastError() : err;
}

}  // namespace

namespace moe_launch {

bool dense_split_takes(const Dense& d) {
  const Split s = plan(d);
  const int64_t sms = sm_count_current(), nk = (d.K + kBK - 1) / kBK;
  const int64_t ctas = s.n_tiles * s.m_tiles * s.C;
  if (ctas >= ((int64_t)1 << 31)) return false;
  // tensor-core time of both kernels in units of one 128 x 256 stage
  const int64_t tiles = ((d.M + 127) / 128) * ((d.N + (d.gated ? 127 : 255)) / (d.gated ? 128 : 256));
  const int64_t big = (tiles + sms - 1) / sms * nk * 256;
  const int64_t small = (ctas + sms - 1) / sms * ((nk + s.C - 1) / s.C) * (d.gated ? 2 : 1) * s.BN;
  return small < big;
}

cudaError_t dense_split(const Dense& d, cudaStream_t stream) {
  const Split s = plan(d);
  return d.gated ? launch<true>(d, s, stream) : launch<false>(d, s, stream);
}

}  // namespace moe_launch
