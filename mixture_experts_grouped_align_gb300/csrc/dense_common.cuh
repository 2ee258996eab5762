// What the two dense matrix-product kernels share: their arguments, the tile loads of both
// weight layouts and the epilogue's arithmetic.
#pragma once

#include "moe_common.cuh"
#include "moe_launch.h"
#include "tcgen05.cuh"
#include "tma.cuh"

namespace dense {

using moe_launch::Dense;

constexpr int kBK = 64;              // K elements of a stage: 128 bytes of bf16
constexpr int kAtomCol = 64 * 128;   // [K, N] weights: 64 K rows x 64 columns, the MN-major atoms of a stage

// A weight tile of `rows` output features (a multiple of 64) from feature n0 on, at K block kb.
// [N, K] weights: one box of `rows` rows x 128 bytes, the K-major 128-byte-swizzled layout.
// [K, N] weights: boxes of 64 K rows x 64 features, each an MN-major atom column.
MOE_DEV void load_w(uint32_t dst, const CUtensorMap* map, bool kn, int64_t n0, int rows, int kb, uint64_t* bar) {
  if (!kn) {
    tma::load_2d(dst, map, kb * 128, (int32_t)n0, bar);
  } else {
    for (int j = 0; j < rows / 64; ++j)
      tma::load_2d(dst + j * kAtomCol, map, (int32_t)(n0 + 64 * j) * 2, kb * kBK, bar);
  }
}

// Descriptor of K step j (16 elements) of a weight tile loaded by load_w.
MOE_DEV uint64_t w_desc(uint32_t tile, bool kn, int j) {
  return kn ? tc::sdesc_sw128_mn(tile + j * 2 * 1024, kAtomCol, 1024) : tc::sdesc_sw128(tile + j * 32);
}

// The warp's elected lane: true in exactly one lane, in warp-uniform code.
MOE_DEV bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

// Descriptor steps, in the descriptor's units of 16 bytes: a K step of 16 elements of the weight
// tile (w_desc's j) and of a K-major tile.
MOE_DEV uint32_t w_step(bool kn) { return kn ? 2 * 1024 / 16 : 2; }
constexpr uint32_t kXStep = 2;

// 32 lanes x 16 columns of TMEM -> 16 registers a thread.
MOE_DEV void tmem_ld16(uint32_t taddr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(taddr));
}

MOE_DEV float bias_at(const void* bias, int64_t i) {
  return moe::bf16_bits_to_f32(static_cast<const uint16_t*>(bias)[i]);
}

MOE_DEV float residual_at(const Dense& d, int64_t i) {
  return d.out_f32 ? static_cast<const float*>(d.residual)[i]
                   : moe::bf16_bits_to_f32(static_cast<const uint16_t*>(d.residual)[i]);
}

}  // namespace dense
