// The dense product where the 256 x 256 tiles of dense_gemm.cu's CTA pairs would leave SMs idle (few
// rows, or few columns).
//
// Bound with few rows: reading W once.  A tile is 128 NA features x BN rows of x with the roles
// of the operands exchanged (A = 128 weight rows, B = the rows of x), so that one row of x costs
// an MMA of N = 16 and not of M = 128.  K is split over the C CTAs of a cluster, which makes
// tiles x C CTAs pull on W at once; each accumulates its share in TMEM, leaves it in its shared
// memory as fp32 (token-major, so that lanes are consecutive features), and the C shares are
// added through distributed shared memory by the CTA that stores the row, from its own share on
// in rank order: no workspace, no second launch, the same bits every time.  A SwiGLU weight tile
// is 64 gate rows and the 64 up rows of the same features, which meet in that sum.  NA = 2 keeps
// two accumulators that share one load of x.
//
// The tensor core's accumulator loses up to one unit in the last place with every MMA, always
// towards zero, which a bf16 output hides and an fp32 output does not (relative error 6e-8 for
// every 64 of K, measured).  For fp32 outputs K is therefore also split over G accumulators in
// TMEM of at most kGroupBlocks blocks of 64 each, which are added in fp32 registers.
//   warp 0 loads stages (64 or 128 of K: the weight tiles, BN rows of x) by TMA, as many stages as
//   fit, from before the block's other roles are ready;
//   warp 1 issues the MMAs; then all sixteen warps drain, add and store.
//
// Measured back to back in a graph.  Weights from HBM (inputs of 270 MB, twice the L2, in turn): 64 x
// 2880 -> 2 x 2880 SwiGLU 10.7 us, the weight at 3.1 TB/s; 64 x 7168 -> 2048 10.3 us, 2.8 TB/s; one row
// 2688 -> 1856 5.7 us; 4099 x 7168 -> 256 in fp32 21.5 us.  With three sets of inputs in turn, whose
// weights stay in L2: 9.1, 7.4, 5.3 and 20.4.  Of the small ones about 3 us are the launch's start, the
// ring's first loads and the cluster's sum, which a longer K hides no part of.  Clocks from the work
// before to the first MMA, the last one, the cluster's meeting, the end (from HBM): 64 rows 5000, 10100,
// 13500, 17000; one row 3700, 4800, 7400, 9600; 4099 rows 3900, 23200, 27600, 35600.
#include <math.h>

#include <atomic>

#include "dense_common.cuh"
#include "per_device.h"

namespace {

using namespace dense;

constexpr int kThreads = 512;
constexpr int kFeat = 128;
constexpr int kMaxStages = 12;
constexpr int kAlone = 116 * 1024;  // more than half of an SM's shared memory
constexpr int kRing = 208 * 1024;  // shared memory of the stages, at most

constexpr int kGroupBlocks = 14;   // blocks of 64 of K an accumulator takes for fp32 outputs

struct Split {
  int BN;        // rows of x per tile: 16, 32, or 64 to 256 in steps of 16
  int NA;        // weight tiles (128 features) per tile
  int C;         // CTAs of a cluster: the shares of K
  int G;         // accumulators a share is split over
  int sub;       // blocks of 64 of K in a stage
  int phase;     // rows of x that leave through shared memory at a time, a multiple of 16
  int stages;
  int slot;      // bytes of a stage
  int smem;
  int cols;      // TMEM columns
  int64_t n_tiles, m_tiles;
};

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr, uint32_t rank) {
  uint32_t a;
  float4 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
  return v;
}

// The epilogue of four neighbouring features of a row: z (SwiGLU: the gate) and u (the up part).
template <bool GATED>
__device__ __forceinline__ void store4(const Dense& d, int64_t m, int64_t n, float4 z4, float4 u4) {
  if (n >= d.N) return;
  float z[4] = {z4.x, z4.y, z4.z, z4.w}, u[4] = {u4.x, u4.y, u4.z, u4.w};
  const int some = d.N - n < 4 ? (int)(d.N - n) : 4;
  if (d.bias)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < some) {
        z[i] += bias_at(d.bias, n + i);
        if (GATED) u[i] += bias_at(d.bias, d.N + n + i);
      }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (GATED) z[i] = (d.out_f32 ? moe::silu_f32(z[i]) : moe::silu(z[i])) * u[i];
    else if (d.relu2) z[i] = moe::relu2(z[i]);
  }
  const int64_t at = m * d.N + n;
  if (some == 4 && d.N % 4 == 0) {
    if (d.out_f32) {
      if (d.residual) {
        const float4 r = *reinterpret_cast<const float4*>(static_cast<const float*>(d.residual) + at);
        z[0] += d.residual_scale * r.x;
        z[1] += d.residual_scale * r.y;
        z[2] += d.residual_scale * r.z;
        z[3] += d.residual_scale * r.w;
      }
      *reinterpret_cast<float4*>(static_cast<float*>(d.out) + at) = make_float4(z[0], z[1], z[2], z[3]);
    } else {
      if (d.residual) {
        const uint2 r = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(d.residual) + at);
        z[0] += d.residual_scale * __uint_as_float(r.x << 16);
        z[1] += d.residual_scale * __uint_as_float(r.x & 0xffff0000u);
        z[2] += d.residual_scale * __uint_as_float(r.y << 16);
        z[3] += d.residual_scale * __uint_as_float(r.y & 0xffff0000u);
      }
      const __nv_bfloat162 lo = __floats2bfloat162_rn(z[0], z[1]), hi = __floats2bfloat162_rn(z[2], z[3]);
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(d.out) + at) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < some) {
        const float o = z[i] + (d.residual ? d.residual_scale * residual_at(d, at + i) : 0.f);
        if (d.out_f32) static_cast<float*>(d.out)[at + i] = o;
        else static_cast<uint16_t*>(d.out)[at + i] = moe::f32_to_bf16_bits(o);
      }
  }
}

template <int NA, bool GATED, int SUB>
__global__ void __launch_bounds__(kThreads, 1)
    dense_split_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w, Dense d,
                       Split sp) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ uint64_t full[kMaxStages], empty[kMaxStages], done;
  __shared__ uint32_t taddr_s;
  __shared__ volatile int abort_flag;
  constexpr int kOut = GATED ? kFeat / 2 : kFeat;  // output features of a weight tile
  // from lane 0: values the compiler can keep in uniform registers
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int rank = sp.C > 1 ? __shfl_sync(0xffffffffu, (int)tc::cluster_ctarank(), 0) : 0;
  const uint32_t smem_s = tc::smem_addr(smem);
  const bool kn = d.w_kn != 0;
  const uint64_t wb = d.wait_ns > 0 ? (uint64_t)d.wait_ns : tc::kWaitNs;
  const uint32_t tile = blockIdx.x / (uint32_t)sp.C, mt = tile / (uint32_t)sp.n_tiles, nt = tile - mt * (uint32_t)sp.n_tiles;
  const int64_t n0 = (int64_t)nt * NA * kOut;  // the tile's first output feature
  const int nk = (d.K + SUB * kBK - 1) / (SUB * kBK);
  const int k0 = (int)((int64_t)nk * rank / sp.C), share = (int)((int64_t)nk * (rank + 1) / sp.C) - k0;
  const int kx = NA * kFeat * 128;  // x rows of a stage, behind the weight tiles
  const int sub_bytes = kx + sp.BN * 128;
  auto load_stage = [&](int it, int s) {
    tma::mbar_arrive_expect_tx(&full[s], (uint32_t)(SUB * sub_bytes));
#pragma unroll
    for (int sub = 0; sub < SUB; ++sub) {  // past K: zeros
      const uint32_t sl = smem_s + s * sp.slot + sub * sub_bytes;
      const int kb = (k0 + it) * SUB + sub;
#pragma unroll
      for (int a = 0; a < NA; ++a) {
        const uint32_t w = sl + a * kFeat * 128;
        if (GATED) {
          load_w(w, &tm_w, kn, n0 + a * kOut, kOut, kb, &full[s]);
          load_w(w + kOut * 128, &tm_w, kn, d.N + n0 + a * kOut, kOut, kb, &full[s]);
        } else {
          load_w(w, &tm_w, kn, n0 + a * kOut, kOut, kb, &full[s]);
        }
      }
      tma::load_2d(sl + kx, &tm_x, kb * 128, (int32_t)(mt * sp.BN), &full[s]);
    }
  };
  // two stages are under way before the block's other warps are ready
  const int first = share < 2 ? share : (sp.stages < 2 ? sp.stages : 2);
  if (tid == 0) {
    for (int s = 0; s < sp.stages; ++s) {
      tc::mbar_init(&full[s], 1);
      tc::mbar_init(&empty[s], 1);
    }
    tc::mbar_init(&done, 1);
    abort_flag = 0;
    tc::mbar_fence_init();
    tc::fence_proxy_async_smem();
    moe::wait_for_stream();
    if (!d.stall)
      for (int it = 0; it < first; ++it) load_stage(it, it);
  }
  if (warp == 1) {
    tc::tmem_alloc(&taddr_s, sp.cols);
    tc::tmem_relinquish();
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t taddr = __shfl_sync(0xffffffffu, taddr_s, 0);
  moe::wait_for_stream();
  moe::let_next_start();

  if (warp == 0 && !d.stall) {
    const bool leader = elect_one();
    int s = first == sp.stages ? 0 : first, issued = first;
    uint32_t ph = first == sp.stages ? 0 : 1;  // a slot's first use waits for nothing
    for (int it = first; it < share; ++it) {
      if (!tc::mbar_wait(&empty[s], ph, wb)) {
        moe::set_status(d.status, MOE_ERR_TIMEOUT);
        abort_flag = 1;
        break;
      }
      if (leader) load_stage(it, s);
      __syncwarp();
      issued = it + 1;
      if (++s == sp.stages) {
        s = 0;
        ph ^= 1;
      }
    }
    // every load lands before the block may end, also when another role has given up
    for (int j = issued > sp.stages ? issued - sp.stages : 0; j < issued; ++j)
      if (!tc::mbar_wait(&full[j % sp.stages], (j / sp.stages) & 1, wb)) {
        moe::set_status(d.status, MOE_ERR_TIMEOUT);
        abort_flag = 1;
      }
  } else if (warp == 1 && !d.stall) {
    // The whole warp runs the loop and one lane issues: descriptors and addresses are the same in
    // every lane, so they stay in uniform registers and a stage's issue takes few instructions.
    const bool leader = elect_one();
    const uint32_t idesc = tc::idesc_f16(kFeat, sp.BN, 1) | (kn ? 1u << 15 : 0u);
    const uint32_t wstep = w_step(kn), slot16 = (uint32_t)sp.slot / 16, sub16 = (uint32_t)sub_bytes / 16;
    const uint64_t w0 = w_desc(smem_s, kn, 0), x0 = tc::sdesc_sw128(smem_s + kx);
    // accumulator group g takes the stages up to (g + 1) share / G
    int s = 0, g = 0, last_of_g = share / sp.G;
    uint32_t ph = 0, d_tmem = taddr, fresh = 1;
    uint64_t wd = w0, xd = x0;
    for (int it = 0; it < share; ++it) {
      if (it == last_of_g) {
        ++g;
        last_of_g = (int)((int64_t)share * (g + 1) / sp.G);
        d_tmem += NA * sp.BN;
        fresh = 1;
      }
      if (!tc::mbar_wait(&full[s], ph, wb)) {
        moe::set_status(d.status, MOE_ERR_TIMEOUT);
        abort_flag = 1;
        break;
      }
      tc::tc_fence_after();
      if (leader) {
#pragma unroll
        for (int sub = 0; sub < SUB; ++sub)
#pragma unroll
          for (int a = 0; a < NA; ++a)
#pragma unroll
            for (int j = 0; j < kBK / 16; ++j)
              tc::mma_f16_ss(d_tmem + a * sp.BN, wd + sub * sub16 + a * (kFeat * 128 / 16) + j * wstep, xd + sub * sub16 + j * kXStep,
                             idesc, sub > 0 || j > 0 || !fresh);
        tc::mma_commit(&empty[s]);
      }
      __syncwarp();
      fresh = 0;
      wd += slot16;
      xd += slot16;
      if (++s == sp.stages) {
        s = 0;
        ph ^= 1;
        wd = w0;
        xd = x0;
      }
    }
    if (leader) tc::mma_commit(&done);
  }
  // One warp watches for the last product; the others sleep at the block's barrier and leave the
  // issue slots to it.
  if (warp == 1 && !tc::mbar_wait(&done, 0, wb)) {
    moe::set_status(d.status, MOE_ERR_TIMEOUT);
    abort_flag = 1;
  }
  __syncthreads();
  const bool ok = !abort_flag;
  tc::tc_fence_after();
  const int64_t m0 = (int64_t)mt * sp.BN;
  const int rows = d.M - m0 < sp.BN ? (int)(d.M - m0) : sp.BN;
  const int phase = sp.phase;
  // `phase` rows at a time: accumulators -> this CTA's shared memory, [weight tile][row][feature]
  // fp32 (the ring is free: every load has landed and every product has read it), then the sum
  // over the cluster.  The same turns for every CTA of the cluster: they share the tile's rows.
  float* part = reinterpret_cast<float*>(smem);
  const uint32_t base = tc::smem_addr(part);
  for (int p0 = 0; p0 < rows; p0 += phase) {
    const int prow = rows - p0 < phase ? rows - p0 : phase;
    if (ok) {
      const uint32_t tb = taddr + ((uint32_t)((warp & 3) * 32) << 16) + p0;
      // a warp takes its 32 lanes of every fourth group of 16 rows
#pragma unroll
      for (int a = 0; a < NA; ++a)
        for (int c = (warp >> 2) * 16; c < prow; c += 64) {
          float* dst = part + (a * phase + c) * kFeat + (warp & 3) * 32 + lane;
          uint32_t v[16];
          tmem_ld16(tb + a * sp.BN + c, v);
          tc::tmem_ld_wait();
          for (int g = 1; g < sp.G; ++g) {
            uint32_t r[16];
            tmem_ld16(tb + (g * NA + a) * sp.BN + c, r);
            tc::tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] = __float_as_uint(__uint_as_float(v[j]) + __uint_as_float(r[j]));
          }
#pragma unroll
          for (int j = 0; j < 16; ++j) dst[j * kFeat] = __uint_as_float(v[j]);
        }
    }
    if (sp.C > 1) tc::cluster_sync();
    else __syncthreads();
    // rows rank, rank + C, ... of the phase: four features a lane, kOut / 4 lanes a row
    constexpr int kLanes = kOut / 4, kRows = kThreads / kLanes;
    const int f = (tid % kLanes) * 4, t0 = rank + sp.C * (tid / kLanes);
    if (ok && sp.C == 1) {
      for (int t = t0; t < prow; t += kRows)
#pragma unroll
        for (int a = 0; a < NA; ++a) {
          const float* at = part + (a * phase + t) * kFeat + f;
          const float4 v = *reinterpret_cast<const float4*>(at);
          store4<GATED>(d, m0 + p0 + t, n0 + a * kOut + f, v, GATED ? *reinterpret_cast<const float4*>(at + kOut) : v);
        }
    } else if (ok) {
      for (int t = t0; t < prow; t += sp.C * kRows)
#pragma unroll
        for (int a = 0; a < NA; ++a) {
          const uint32_t at = base + (uint32_t)((a * phase + t) * kFeat + f) * 4;
          float4 v[8], u[8];
#pragma unroll
          for (int r = 0; r < 8; ++r) {
            // from this CTA's own share on, so that the CTAs do not all read the same one at once
            const int from = rank + r < sp.C ? rank + r : rank + r - sp.C;
            v[r] = r < sp.C ? ld_cluster_f4(at, from) : make_float4(0.f, 0.f, 0.f, 0.f);
            if (GATED) u[r] = r < sp.C ? ld_cluster_f4(at + kOut * 4, from) : make_float4(0.f, 0.f, 0.f, 0.f);
          }
#pragma unroll
          for (int r = 1; r < 8; ++r) {
            v[0].x += v[r].x;
            v[0].y += v[r].y;
            v[0].z += v[r].z;
            v[0].w += v[r].w;
            if (GATED) {
              u[0].x += u[r].x;
              u[0].y += u[r].y;
              u[0].z += u[r].z;
              u[0].w += u[r].w;
            }
          }
          store4<GATED>(d, m0 + p0 + t, n0 + a * kOut + f, v[0], GATED ? u[0] : v[0]);
        }
    }
    // before the next phase overwrites, or the CTA leaves, every CTA has read its share
    if (sp.C > 1) tc::cluster_sync();
    else __syncthreads();
  }
  tc::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc::tc_fence_after();
    tc::tmem_dealloc(taddr, sp.cols);
  }
}

// CTAs of clusters of C, 1 to 8, that the current device holds at once with one CTA per SM (queried
// once per device).
void resident_ctas(int (&at_once)[9]) {
  static moe_host::PerDevice<9> seen;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) dev = -1;
  const int sms = moe_launch::sm_count_current();
  at_once[0] = 0;
  at_once[1] = sms;
  for (int C = 2; C <= 8; ++C)
    at_once[C] = seen.get(dev, C, C, [=] {
      cudaLaunchConfig_t cfg{};
      cfg.gridDim = dim3((unsigned)(C * sms));
      cfg.blockDim = dim3(kThreads);
      cfg.dynamicSmemBytes = kRing + 1024;
      cudaLaunchAttribute at[1];
      at[0].id = cudaLaunchAttributeClusterDimension;
      at[0].val.clusterDim.x = C;
      at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
      cfg.attrs = at;
      cfg.numAttrs = 1;
      int clusters = 0;
      if (cudaFuncSetAttribute(dense_split_kernel<1, false, 1>, cudaFuncAttributeMaxDynamicSharedMemorySize, kRing + 1024) !=
              cudaSuccess ||
          cudaOccupancyMaxActiveClusters(&clusters, dense_split_kernel<1, false, 1>, &cfg) != cudaSuccess) {
        (void)cudaGetLastError();
        return 0;
      }
      return clusters * C;
    });
}

// The variant with the least estimated time in clocks.  Per CTA a stage costs what its operands
// take from L2 (about 60 bytes a clock and SM) or its MMAs on the tensor core (BN / 2 clocks
// each), whichever is more; a wave of CTAs is as long as its longest share; the sum over the
// cluster moves about 16 bytes a clock into an SM.  Against every variant timed, over 25 shapes of 1
// to 16000 rows with weights from HBM: within 2% of the best in 20, 4 to 5% off in three (128 x 2048 x 2048
// 6.9 us against 6.7; 4099 x 256 x 7168 fp32 21.6 against 20.6; 2000 x 2 x 2048 x 2048 SwiGLU 26.0 against
// 24.9 on CTA pairs), 8% in one (47 x 520 x 2880 5.4 against 5.0), and 17% in the worst: 512 x 2 x 2048 x
// 7168 SwiGLU, 33.4 us as 2 x 256 split in four against 28.6 as 128-row tiles whole in K, whose loads it
// takes for slower than they are.  Above 64 rows BN goes in steps of 16, which fits ragged M and the
// number of SMs.
Split plan(const Dense& d, double* clocks) {
  const int kOut = d.gated ? kFeat / 2 : kFeat;
  Split best{};
  double least = 0;
  int resident[9];
  resident_ctas(resident);
  for (int NA = 1; NA <= 2; ++NA)
    for (int BN = 16; BN <= 256; BN = BN < 64 ? BN * 2 : BN + 16) {
      Split s{};
      s.NA = NA;
      s.BN = BN;
      s.n_tiles = (d.N + NA * kOut - 1) / (NA * kOut);
      s.m_tiles = (d.M + BN - 1) / BN;
      // small tiles' MMAs take less than a stage's handshake (about 190 clocks), so two blocks of
      // 64 share one (64 x 7168 x 2048: 8.1 -> 7.5 us); large tiles need the ring's finer slots
      // (4099 x 256 x 7168: 21.1 us so, 22.5 with two)
      s.sub = BN <= 64 ? 2 : 1;
      const uint32_t nk = (uint32_t)(d.K + s.sub * kBK - 1) / (uint32_t)(s.sub * kBK);
      const int64_t tiles = s.n_tiles * s.m_tiles;
      if (tiles < (1 << 27)) {
        const double load = s.sub * (NA * kFeat + BN) * (128 / 60.0), mma = s.sub * BN * 2.0 * NA, stage = mma > load ? mma : load;
        for (uint32_t C = 1; C <= 8 && C <= nk; ++C) {
          const uint32_t at_once = (uint32_t)resident[C];
          // more shares than fill a wave only shorten fp32 sums
          if (C > 1 && (uint32_t)tiles * (C - 1) >= at_once && !d.out_f32) break;
          const uint32_t share = (nk + C - 1) / C, waves = ((uint32_t)tiles * C + at_once - 1) / at_once;
          uint32_t G = 1;
          if (d.out_f32) {
            G = (share * s.sub + kGroupBlocks - 1) / kGroupBlocks;
            if (G > (uint32_t)(512 / (NA * BN))) continue;  // too long a sum in one accumulator
          }
          // each wave: its stages, about 3000 clocks to start, the drain and the cluster's sum
          const double bytes = NA * BN * kFeat * 4.0;
          const double t = waves * (share * stage + 3000 + bytes * G / 100 + (C > 1 ? 2500 + bytes / 16 * (C - 1) / C : 0));
          if (best.BN == 0 || t < least) {
            least = t;
            best = s;
            best.C = (int)C;
            best.G = (int)G;
          }
        }
      }
      if (BN >= d.M) break;
    }
  if (best.BN == 0) {  // more tiles, or longer fp32 sums, than this kernel is for
    *clocks = INFINITY;
    return best;
  }
  const int nk = (d.K + best.sub * kBK - 1) / (best.sub * kBK), share = (nk + best.C - 1) / best.C;
  best.slot = best.sub * (best.NA * kFeat + best.BN) * 128;
  best.stages = kRing / best.slot;
  if (best.stages > kMaxStages) best.stages = kMaxStages;
  if (best.stages > share) best.stages = share;
  const int fit = kRing / (best.NA * kFeat * 4) / 16 * 16, turns = (best.BN + fit - 1) / fit;
  best.phase = (best.BN + 16 * turns - 1) / (16 * turns) * 16;
  const int part = best.NA * best.phase * kFeat * 4;
  best.smem = (best.stages * best.slot > part ? best.stages * best.slot : part) + 1024;
  // Never two CTAs of this kernel on an SM: one could wait for tensor memory that the other holds
  // until its cluster has met, while the clusters' other CTAs wait the other way round.
  if (best.smem < kAlone) best.smem = kAlone;
  best.cols = 32;
  while (best.cols < best.NA * best.BN * best.G) best.cols *= 2;
  *clocks = least;
  return best;
}

template <int NA, bool GATED, int SUB>
cudaError_t launch(const Dense& d, const Split& s, cudaStream_t stream) {
  const uint64_t K2 = (uint64_t)d.K * 2, N1 = GATED ? 2 * (uint64_t)d.N : (uint64_t)d.N;
  CUtensorMap mx{}, mw{};
  if (!tma::encode_2d_u8(&mx, d.x, K2, (uint64_t)d.M, K2, 128, (uint32_t)s.BN, true)) return cudaErrorInvalidValue;
  const bool okw = d.w_kn ? tma::encode_2d_u8(&mw, d.w, N1 * 2, (uint64_t)d.K, N1 * 2, 128, kBK, true)
                          : tma::encode_2d_u8(&mw, d.w, K2, N1, K2, 128, GATED ? kFeat / 2 : kFeat, true);
  if (!okw) return cudaErrorInvalidValue;
  auto kern = dense_split_kernel<NA, GATED, SUB>;
  static std::atomic<uint64_t> sized{0};
  cudaError_t err = moe_launch::allow_smem(reinterpret_cast<const void*>(kern), kRing + 1024, sized);
  if (err != cudaSuccess) return err;
  return moe_launch::launch_staged(kern, dim3((unsigned)(s.n_tiles * s.m_tiles * s.C)), dim3(kThreads), (size_t)s.smem, stream,
                                   s.C, mx, mw, d, s);
}

// Whether the split kernel is estimated faster than the pairs', and how it would run.
bool pick(const Dense& d, Split* s) {
  double split = 0;
  *s = plan(d, &split);
  // the pairs' kernel: 512 clocks a stage of a 256 x 256 tile, its start and its last epilogue
  const int64_t pairs = moe_launch::sm_count_current() / 2, nk = (d.K + kBK - 1) / kBK;
  const int64_t tiles = ((d.M + 255) / 256) * ((d.N + (d.gated ? 127 : 255)) / (d.gated ? 128 : 256));
  return split < (double)((tiles + pairs - 1) / pairs) * nk * 512 + 7000;
}

}  // namespace

namespace moe_launch {

bool dense_split(const Dense& d, cudaStream_t stream, cudaError_t* err) {
  Split s;
  if (!pick(d, &s)) return false;
  const int which = (d.gated ? 4 : 0) + (s.NA == 2 ? 2 : 0) + (s.sub == 2 ? 1 : 0);
  using Launch = cudaError_t (*)(const Dense&, const Split&, cudaStream_t);
  static const Launch launches[8] = {launch<1, false, 1>, launch<1, false, 2>, launch<2, false, 1>, launch<2, false, 2>,
                                     launch<1, true, 1>,  launch<1, true, 2>,  launch<2, true, 1>,  launch<2, true, 2>};
  *err = launches[which](d, s, stream);
  return true;
}

void dense_plan(const Dense& d, int32_t* p) {
  Split s;
  if (pick(d, &s)) {
    const int32_t v[8] = {1, s.BN, s.NA, s.C, s.G, s.sub, s.phase, s.stages};
    for (int i = 0; i < 8; ++i) p[i] = v[i];
  } else {
    for (int i = 0; i < 8; ++i) p[i] = 0;
  }
}

}  // namespace moe_launch
