// Dense matrix product with its bias, activation and residual in the epilogue, on tcgen05.
//
//   z = x . W^T + b;   out = act(z) + residual_scale * residual
// x [M, K] bf16; W stored [N1, K] or (contracted over its rows, as an input gradient needs the
// forward weight) [K, N1]; act = none, relu^2 or SwiGLU (N1 = 2N: gate features, then up).
// fp32 accumulation, one rounding to the output type (shapes of few tiles: dense_split.cu).
//
// Bound: 2 M N1 K operations on the tensor cores, as long as the operands arrive: an SM takes
// about 64 bytes a clock from L2, and a 128 x 256 tile on one SM (48 KB of operands per 512 clocks
// of MMAs) was held to 70% of the tensor cores by that.  So two CTAs, a cluster on two SMs, share
// a 256 x 256 tile: the MMAs (cta_group::2, M 256, N 256, K 16) read 128 rows of x and 128 of W
// from either CTA's shared memory, 32 KB per CTA and stage, and leave 128 rows of the tile in
// each CTA's TMEM.  Persistent pairs over the tiles (SwiGLU: 128 gate columns from the first CTA
// and 128 up columns from the second, so both lie in the same TMEM lane and thread), two fp32
// accumulators of 256 TMEM columns so that a tile's epilogue runs under the next tile's products:
//   warp 0  loads this CTA's half of a stage (64 of K) by TMA, completing on the first CTA's
//           barrier, five stages;
//   warp 1  of the first CTA issues the MMAs; their commits free the stage, and announce the
//           accumulator, in both CTAs;
//   warps 4..19  drain the accumulator, four per TMEM lane quarter with a quarter of the columns
//           each: bias, activation, residual (a TMA box loaded into the staging box the result
//           then replaces), rounding, and a TMA store of a box of 32 rows, which drops what lies
//           past M or N.  Rows of out that are no multiple of 16 bytes are stored by plain stores.
// The tensor core's accumulator loses up to one unit in the last place with every MMA, always
// towards zero, which a bf16 output hides.  For fp32 outputs an accumulator therefore takes at
// most kChunk stages, and the epilogue warps add the chunks up in registers meanwhile.
// Tiles are taken sixteen row tiles at a time, the column tile slower, so that the pairs running at
// once share their operands in L2 (8191 x 7168 x 4096, long runs under the power limit: 4 row tiles
// 308 us, 8 303, 16 296, 32 317).
// Measured: 8192 x 7168 -> 2 x 2048 SwiGLU with bias, short runs 253 us (1.90 PFLOP/s, the library's
// rate for the product alone; 284 us on single CTAs' 128 x 256 tiles), under the power limit 290 to
// 300; 8191 x 4096 -> 7168 on the other layout with the residual 279 us.  fp32 outputs cost the drain of
// every chunk besides twice the bytes: 8000 x 4104 -> 7168 368 us (bf16 308, both under the power
// limit), 4096 x 1032 -> 4104 47 (38), 8192 x 7168 -> 2 x 2048 SwiGLU 263 to 269 (250 to 253).
// Every wait is bounded; one that runs out sets MOE_ERR_TIMEOUT, all roles leave their loops,
// the loads in flight are waited for, and both CTAs meet before either ends.
#include "dense_common.cuh"

namespace {

using namespace dense;

constexpr int kThreads = 640;
constexpr int kBM = 128, kBN = 256;             // a CTA's rows and the pair's columns of a tile
constexpr int kStages = 5;
constexpr int kA = 0, kB = kBM * 128, kSlot = 2 * kBM * 128;  // x rows | this CTA's 128 W rows
constexpr int kStg = kStages * kSlot;           // staging boxes, 4 KB per epilogue warp
constexpr int kEpiWarp0 = 4, kEpiWarps = 16;
constexpr int kBars = kStg + kEpiWarps * 4096;
constexpr int kSmem = kBars + 512 + 1024;
constexpr int kGroupM = 16;
constexpr int kChunk = 12;                      // stages (64 of K) an accumulator takes for fp32 outputs

struct Tiles {
  int64_t m, n, total;
};

// The tensor-core instructions of a CTA pair.
namespace pair {

// Allocation, release and deallocation are executed by a warp of each CTA of the pair.
__device__ __forceinline__ void tmem_alloc(uint32_t* dst, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(tc::smem_addr(dst)), "r"(ncols)
               : "memory");
}
__device__ __forceinline__ void tmem_relinquish() {
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
// D (+)= A . B^T, M = 256: rows 0..127 of A and D are the first CTA's, 128..255 the second's, and
// so are the halves of B's rows, each at the same shared-memory offset.
__device__ __forceinline__ void mma_f16_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Arrives on the barrier at this offset in both CTAs when the MMAs issued before have completed.
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          tc::smem_addr(bar)),
      "h"((uint16_t)3)
      : "memory");
}
// Cluster address of a barrier of the first CTA.
__device__ __forceinline__ uint32_t first_cta_addr(const uint64_t* bar) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(a) : "r"(tc::smem_addr(bar)));
  return a;
}
__device__ __forceinline__ void arrive_first_cta(uint64_t* bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(first_cta_addr(bar)) : "memory");
}
// Loads a box into this CTA's shared memory; its bytes complete on a barrier of either CTA.
__device__ __forceinline__ void load_2d(uint32_t dst, const CUtensorMap* map, int32_t x, int32_t y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
      : "memory");
}

}  // namespace pair

__device__ __forceinline__ void tile_of(const Tiles& ts, int64_t t, int64_t& mt, int64_t& nt) {
  const int64_t per = kGroupM * ts.n, g = t / per, r = t - g * per;
  const int64_t rows = ts.m - g * kGroupM < kGroupM ? ts.m - g * kGroupM : kGroupM;
  nt = r / rows;
  mt = g * kGroupM + (r - nt * rows);
}

// Byte offset of 16-byte unit q of row r of a staging box: rows of 128 bytes in the 128-byte
// swizzle, or of 64 bytes as they are.
template <int BYTES>
__device__ __forceinline__ uint32_t box_offset(int r, int q) {
  return BYTES == 128 ? (uint32_t)(r * 128 + ((q ^ (r & 7)) << 4)) : (uint32_t)(r * BYTES + (q << 4));
}
__device__ __forceinline__ void lds128(uint32_t at, uint32_t (&r)[4]) {
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ void sts128(uint32_t at, const uint32_t (&r)[4]) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]) : "memory");
}

// Bias of the 8 features n .. n + 7 (zeros past N); `base` is the first feature's index.
__device__ __forceinline__ void bias8(const void* bias, int64_t base, int64_t n, int64_t N, bool vec, float (&b)[8]) {
  if (vec && n + 8 <= N) {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(bias) + base + n));
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      b[2 * i] = __uint_as_float(w[i] << 16);
      b[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) b[i] = n + i < N ? bias_at(bias, base + n + i) : 0.f;
  }
}

template <bool GATED, bool F32>
__global__ void __launch_bounds__(kThreads, 1)
    dense_gemm_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w,
                      const __grid_constant__ CUtensorMap tm_o, const __grid_constant__ CUtensorMap tm_r, Dense d,
                      Tiles ts) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kBars);
  uint64_t* empty = full + kStages;
  uint64_t* tfull = empty + kStages;   // [2]
  uint64_t* tempty = tfull + 2;        // [2]
  uint64_t* drain = tempty + 2;
  uint64_t* rfull = drain + 1;         // [kEpiWarps] residual box landed
  uint32_t* taddr_s = reinterpret_cast<uint32_t*>(rfull + kEpiWarps);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(taddr_s + 1);
  // from lane 0: values the compiler can keep in uniform registers
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const uint32_t rank = __shfl_sync(0xffffffffu, tc::cluster_ctarank(), 0);
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      tc::mbar_init(&full[s], 1);
      tc::mbar_init(&empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&tfull[i], 1);
      tc::mbar_init(&tempty[i], 2 * kEpiWarps);
    }
    tc::mbar_init(drain, 1);
    for (int i = 0; i < kEpiWarps; ++i) tc::mbar_init(&rfull[i], 1);
    *abort_flag = 0;
    tc::mbar_fence_init();
  }
  if (warp == 1) {
    pair::tmem_alloc(taddr_s, 512);
    pair::tmem_relinquish();
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::cluster_sync();  // both CTAs' barriers are there before either is signalled
  tc::tc_fence_after();
  moe::wait_for_stream();
  moe::let_next_start();
  const uint32_t taddr = __shfl_sync(0xffffffffu, *taddr_s, 0), smem_s = tc::smem_addr(smem);
  const int nk = (d.K + kBK - 1) / kBK;
  const bool kn = d.w_kn != 0;
  const uint64_t wb = d.wait_ns > 0 ? (uint64_t)d.wait_ns : tc::kWaitNs;
  constexpr int kOutN = GATED ? 128 : kBN;  // output columns of a tile
  const int64_t pair0 = blockIdx.x / 2, pairs = gridDim.x / 2;

  if (warp == 0 && !d.stall) {
    // ------------------------------------------------------------------ loads
    const bool leader = elect_one();
    if (leader) {
      tma::prefetch_map(&tm_x);
      tma::prefetch_map(&tm_w);
    }
    uint32_t s = 0, ph = 1, it = 0;
    bool ok = true;
    for (int64_t t = pair0; t < ts.total && ok && !*abort_flag; t += pairs) {
      int64_t mt, nt;
      tile_of(ts, t, mt, nt);
      const int32_t row = (int32_t)(mt * 2 * kBM + rank * kBM);
      const int64_t n0 = GATED ? nt * 128 + (rank ? d.N : 0) : nt * kBN + rank * 128;
      for (int kb = 0; kb < nk; ++kb, ++it) {
        if (!tc::mbar_wait(&empty[s], ph, wb)) {
          ok = false;
          break;
        }
        if (leader) {
          const uint32_t sl = smem_s + s * kSlot, bar = pair::first_cta_addr(&full[s]);
          if (rank == 0) tma::mbar_arrive_expect_tx(&full[s], 2 * kSlot);  // both CTAs' halves
          pair::load_2d(sl + kA, &tm_x, kb * 128, row, bar);
          if (kn) {
            pair::load_2d(sl + kB, &tm_w, (int32_t)n0 * 2, kb * kBK, bar);
            pair::load_2d(sl + kB + kAtomCol, &tm_w, (int32_t)(n0 + 64) * 2, kb * kBK, bar);
          } else {
            pair::load_2d(sl + kB, &tm_w, kb * 128, (int32_t)n0, bar);
          }
        }
        __syncwarp();
        if (++s == kStages) {
          s = 0;
          ph ^= 1;
        }
      }
    }
    if (!ok) {
      moe::set_status(d.status, MOE_ERR_TIMEOUT);
      *abort_flag = 1;
    }
    // every load lands before the pair may end, also when another role has given up (the first
    // CTA's barriers count both CTAs' loads)
    if (rank == 0)
      for (uint32_t j = it > (uint32_t)kStages ? it - kStages : 0; j < it; ++j)
        if (!tc::mbar_wait(&full[j % kStages], (j / kStages) & 1, wb)) moe::set_status(d.status, MOE_ERR_TIMEOUT);
    __syncwarp();
  } else if (warp == 1 && rank == 0 && !d.stall) {
    // ------------------------------------------------------------------ MMA issuer
    // The whole warp runs the loop and one lane issues: descriptors and addresses are the same in
    // every lane, so they stay in uniform registers and a stage's issue takes few instructions.
    const bool leader = elect_one();
    const uint32_t idesc = tc::idesc_f16(2 * kBM, kBN, 1) | (kn ? 1u << 16 : 0u);
    const uint32_t wstep = w_step(kn);
    const uint64_t a0 = tc::sdesc_sw128(smem_s + kA), b0 = w_desc(smem_s + kB, kn, 0);
    uint32_t s = 0, ph = 0, acc = 0, acc_ph = 1;
    bool ok = true;
    for (int64_t t = pair0; t < ts.total && ok && !*abort_flag; t += pairs) {
      // fp32 outputs: kChunk stages an accumulator, which the epilogue adds up in registers
      for (int k0 = 0; k0 < nk && ok; k0 += F32 ? kChunk : nk) {
        const int k1 = F32 && k0 + kChunk < nk ? k0 + kChunk : nk;
        if (!tc::mbar_wait(&tempty[acc], acc_ph, wb)) {
          ok = false;
          break;
        }
        tc::tc_fence_after();
        const uint32_t d_tmem = taddr + acc * kBN;
        for (int kb = k0; kb < k1; ++kb) {
          if (!tc::mbar_wait(&full[s], ph, wb)) {
            ok = false;
            break;
          }
          tc::tc_fence_after();
          if (leader) {
            const uint64_t ad = a0 + s * (kSlot / 16), bd = b0 + s * (kSlot / 16);
#pragma unroll
            for (int j = 0; j < kBK / 16; ++j) pair::mma_f16_ss(d_tmem, ad + j * kXStep, bd + j * wstep, idesc, kb > k0 || j > 0);
            pair::mma_commit(&empty[s]);
          }
          __syncwarp();
          if (++s == kStages) {
            s = 0;
            ph ^= 1;
          }
        }
        if (!ok) break;
        if (leader) pair::mma_commit(&tfull[acc]);
        __syncwarp();
        acc ^= 1;
        if (acc == 0) acc_ph ^= 1;
      }
    }
    if (!ok) {
      moe::set_status(d.status, MOE_ERR_TIMEOUT);
      *abort_flag = 1;
    }
    if (leader) pair::mma_commit(drain);
    if (!tc::mbar_wait(drain, 0, wb)) moe::set_status(d.status, MOE_ERR_TIMEOUT);
    __syncwarp();
  } else if (warp >= kEpiWarp0) {
    // ------------------------------------------------------------------ epilogue
    const int ew = warp - kEpiWarp0, quarter = warp & 3;
    constexpr int kPer = kOutN / (kEpiWarps / 4);     // output columns of a warp
    constexpr int kCols = F32 ? 32 : 64;              // columns of a 128-byte staging row
    constexpr int kBoxes = kPer < kCols ? 1 : kPer / kCols, kBlocks = (kPer < kCols ? kPer : kCols) / 32;
    const int col0 = (ew >> 2) * kPer;
    const uint32_t box = smem_s + kStg + ew * 4096;
    const bool vec = d.N % 8 == 0;
    const bool res_box = d.residual != nullptr && d.tma_out;
    uint32_t acc = 0, acc_ph = 0, rph = 0;
    float sum[F32 ? kPer : 1], sum_u[F32 && GATED ? kPer : 1];  // fp32 outputs: the chunks' sums
    bool ok = true;
    for (int64_t t = pair0; t < ts.total && ok && !*abort_flag; t += pairs) {
      int64_t mt, nt;
      tile_of(ts, t, mt, nt);
      const uint32_t lane_quarter = (uint32_t)(quarter * 32) << 16;
      for (int k0 = 0; k0 < nk; k0 += F32 ? kChunk : nk) {
        if (!tc::mbar_wait(&tfull[acc], acc_ph, wb)) {
          ok = false;
          break;
        }
        tc::tc_fence_after();
        if (!F32) break;
        const uint32_t tb = taddr + acc * kBN + lane_quarter + col0;
#pragma unroll
        for (int c = 0; c < kPer; c += 16) {
          uint32_t v[16];
          tmem_ld16(tb + c, v);
          tc::tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 16; ++i) sum[F32 ? c + i : 0] = (k0 ? sum[F32 ? c + i : 0] : 0.f) + __uint_as_float(v[i]);
          if (GATED) {
            tmem_ld16(tb + 128 + c, v);
            tc::tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; ++i)
              sum_u[F32 && GATED ? c + i : 0] = (k0 ? sum_u[F32 && GATED ? c + i : 0] : 0.f) + __uint_as_float(v[i]);
          }
        }
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) pair::arrive_first_cta(&tempty[acc]);
        acc ^= 1;
        if (acc == 0) acc_ph ^= 1;
      }
      if (!ok) break;
      const uint32_t tb = taddr + acc * kBN + lane_quarter + col0;
      const int64_t m0 = mt * 2 * kBM + rank * kBM + quarter * 32, m = m0 + lane;
#pragma unroll
      for (int bx = 0; bx < kBoxes; ++bx) {
        const int64_t n0 = nt * kOutN + col0 + bx * kCols;
        if (n0 >= d.N || m0 >= d.M) continue;  // the same for the whole warp
        if (lane == 0 && d.tma_out) {
          tma::bulk_wait_read_all();  // the last store has read the box
          if (res_box) {
            tma::mbar_arrive_expect_tx(&rfull[ew], 32 * kBlocks * 32 * (F32 ? 4 : 2));
            tma::load_2d(box, &tm_r, (int32_t)(n0 * (F32 ? 4 : 2)), (int32_t)m0, &rfull[ew]);
          }
        }
        __syncwarp();
        bool have = !res_box;
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) {
          uint32_t v[32], u[32];
          if (F32) {
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              v[i] = __float_as_uint(sum[F32 ? bx * kCols + 32 * b + i : 0]);
              if (GATED) u[i] = __float_as_uint(sum_u[F32 && GATED ? bx * kCols + 32 * b + i : 0]);
            }
          } else {
            tc::tmem_ld32(tb + bx * kCols + 32 * b, v);
            if (GATED) tc::tmem_ld32(tb + 128 + bx * kCols + 32 * b, u);
            tc::tmem_ld_wait();
          }
          if (!have) {
            if (!tc::mbar_wait(&rfull[ew], rph, wb)) ok = false;
            have = true;
          }
#pragma unroll
          for (int q = 0; q < 4; ++q) {  // eight columns
            const int64_t n = n0 + 32 * b + 8 * q;
            float o[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = __uint_as_float(v[8 * q + i]);
            if (d.bias) {
              float bb[8];
              bias8(d.bias, 0, n, d.N, vec, bb);
#pragma unroll
              for (int i = 0; i < 8; ++i) o[i] += bb[i];
            }
            if (GATED) {
              float up[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) up[i] = __uint_as_float(u[8 * q + i]);
              if (d.bias) {
                float bb[8];
                bias8(d.bias, d.N, n, d.N, vec, bb);
#pragma unroll
                for (int i = 0; i < 8; ++i) up[i] += bb[i];
              }
#pragma unroll
              for (int i = 0; i < 8; ++i) o[i] = (F32 ? moe::silu_f32(o[i]) : moe::silu(o[i])) * up[i];
            } else if (d.relu2) {
#pragma unroll
              for (int i = 0; i < 8; ++i) o[i] = moe::relu2(o[i]);
            }
            if (d.residual && !res_box) {
#pragma unroll
              for (int i = 0; i < 8; ++i)
                if (m < d.M && n + i < d.N) o[i] += d.residual_scale * residual_at(d, m * d.N + n + i);
            }
            if (F32) {
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                const uint32_t at = box + box_offset<4 * kBlocks * 32>(lane, 2 * q + j);
                if (res_box) {
                  uint32_t r[4];
                  lds128(at, r);
#pragma unroll
                  for (int i = 0; i < 4; ++i) o[4 * j + i] += d.residual_scale * __uint_as_float(r[i]);
                }
                const uint32_t w[4] = {__float_as_uint(o[4 * j]), __float_as_uint(o[4 * j + 1]), __float_as_uint(o[4 * j + 2]),
                                       __float_as_uint(o[4 * j + 3])};
                sts128(at, w);
              }
            } else {
              const uint32_t at = box + box_offset<2 * kBlocks * 32>(lane, 4 * b + q);
              if (res_box) {
                uint32_t r[4];
                lds128(at, r);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  o[2 * i] += d.residual_scale * __uint_as_float(r[i] << 16);
                  o[2 * i + 1] += d.residual_scale * __uint_as_float(r[i] & 0xffff0000u);
                }
              }
              uint32_t pk[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(o[2 * i], o[2 * i + 1]);
                pk[i] = *reinterpret_cast<const uint32_t*>(&h);
              }
              sts128(at, pk);
            }
          }
        }
        if (res_box) rph ^= 1;
        if (d.tma_out) {
          tc::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma::store_2d(&tm_o, (int32_t)(n0 * (F32 ? 4 : 2)), (int32_t)m0, box);
            tma::bulk_commit();
          }
        } else {  // rows of out not a multiple of 16 bytes: a row's columns by the lanes
          __syncwarp();
          constexpr int kBoxCols = 32 * kBlocks;
          const int rows = d.M - m0 < 32 ? (int)(d.M - m0) : 32;
          const int cols = d.N - n0 < kBoxCols ? (int)(d.N - n0) : kBoxCols;
          for (int r = 0; r < rows; ++r)
            for (int c = lane; c < cols; c += 32) {
              if (F32) {
                uint32_t w;
                asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w) : "r"(box + box_offset<4 * kBoxCols>(r, c >> 2) + (c & 3) * 4) : "memory");
                static_cast<uint32_t*>(d.out)[(m0 + r) * d.N + n0 + c] = w;
              } else {
                uint16_t w;
                asm volatile("ld.shared.b16 %0, [%1];" : "=h"(w) : "r"(box + box_offset<2 * kBoxCols>(r, c >> 3) + (c & 7) * 2) : "memory");
                static_cast<uint16_t*>(d.out)[(m0 + r) * d.N + n0 + c] = w;
              }
            }
          __syncwarp();
        }
      }
      if (!F32) {
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) pair::arrive_first_cta(&tempty[acc]);
        acc ^= 1;
        if (acc == 0) acc_ph ^= 1;
      }
    }
    if (!ok) {
      moe::set_status(d.status, MOE_ERR_TIMEOUT);
      *abort_flag = 1;
    }
    if (lane == 0) tma::bulk_wait_read_all();  // the stores need the boxes no more; they end with the grid
    __syncwarp();
  }
  tc::tc_fence_before();
  __syncthreads();
  // the last commit reaches the second CTA too: it is waited for there before the CTA may end
  if (warp == 1 && rank == 1 && !d.stall && !tc::mbar_wait(drain, 0, wb)) moe::set_status(d.status, MOE_ERR_TIMEOUT);
  __syncwarp();
  tc::cluster_sync();  // neither CTA leaves while the other's products or signals may reach it
  if (warp == 1) {
    tc::tc_fence_after();
    pair::tmem_dealloc(taddr, 512);
  }
}

template <bool GATED, bool F32>
cudaError_t launch(const Dense& d, cudaStream_t stream) {
  Tiles ts;
  ts.m = (d.M + 2 * kBM - 1) / (2 * kBM);
  ts.n = (d.N + (GATED ? 127 : kBN - 1)) / (GATED ? 128 : kBN);
  ts.total = ts.m * ts.n;
  const uint64_t K2 = (uint64_t)d.K * 2, N1 = GATED ? 2 * (uint64_t)d.N : (uint64_t)d.N;
  CUtensorMap mx{}, mw{}, mo{}, mr{};
  if (!tma::encode_2d_u8(&mx, d.x, K2, (uint64_t)d.M, K2, 128, kBM, true)) return cudaErrorInvalidValue;
  const bool okw = d.w_kn ? tma::encode_2d_u8(&mw, d.w, N1 * 2, (uint64_t)d.K, N1 * 2, 128, kBK, true)
                          : tma::encode_2d_u8(&mw, d.w, K2, N1, K2, 128, 128, true);
  if (!okw) return cudaErrorInvalidValue;
  if (d.tma_out) {
    const uint64_t row = (uint64_t)d.N * (F32 ? 4 : 2);
    constexpr uint32_t kBox = GATED && !F32 ? 64 : 128;  // bytes of a staging row
    if (!tma::encode_2d_u8(&mo, d.out, row, (uint64_t)d.M, row, kBox, 32, kBox == 128)) return cudaErrorInvalidValue;
    if (d.residual && !tma::encode_2d_u8(&mr, d.residual, row, (uint64_t)d.M, row, kBox, 32, kBox == 128))
      return cudaErrorInvalidValue;
  }
  static std::atomic<uint64_t> sized{0};
  cudaError_t err = moe_launch::allow_smem(reinterpret_cast<const void*>(&dense_gemm_kernel<GATED, F32>), kSmem, sized);
  if (err != cudaSuccess) return err;
  const int64_t most = moe_launch::sm_count_current() / 2;
  return moe_launch::launch_staged(dense_gemm_kernel<GATED, F32>, dim3((unsigned)(2 * (ts.total < most ? ts.total : most))),
                                   dim3(kThreads), kSmem, stream, 2, mx, mw, mo, mr, d, ts);
}

}  // namespace

namespace moe_launch {

cudaError_t dense_gemm(Dense d, cudaStream_t stream) {
  if (d.M == 0) return cudaSuccess;
  cudaError_t err;
  if (dense_split(d, stream, &err)) return err;
  d.tma_out = ((int64_t)d.N * (d.out_f32 ? 4 : 2)) % 16 == 0;
  if (d.gated) return d.out_f32 ? launch<true, true>(d, stream) : launch<true, false>(d, stream);
  return d.out_f32 ? launch<false, true>(d, stream) : launch<false, false>(d, stream);
}

}  // namespace moe_launch
