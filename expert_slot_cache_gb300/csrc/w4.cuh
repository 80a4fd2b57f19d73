// 4-bit weights with group scales: the packed format and the device helpers its kernels share.
//
// A K x N matrix W (y = x W) holds W[k][n] = (code[k][n] - 8) * scale[k / G][n] with codes 0..15 and
// one scale per G = 32, 64 or 128 consecutive inputs of an output column.  Packed:
//
//   codes   [Mt][Kb][512 B]  Mt = ceil(N / 16) tiles of 16 output columns, Kb = ceil(K / 64) blocks of
//                            64 inputs.  A tile block is 32 lanes x 16 bytes: lane 4g + q holds, for
//                            columns g and g + 8 of the tile, the 16 inputs 32h + 8q + i (h = 0, 1;
//                            i = 0..7) in four 32-bit words.  Word s covers the four inputs
//                            k0 = 32(s >> 1) + 8q + 4(s & 1): nibbles 0 and 4 are column g's inputs
//                            k0, k0 + 1, nibbles 1 and 5 column g + 8's, nibbles 2, 6 and 3, 7 the same
//                            for k0 + 2, k0 + 3.  That is the A fragment of a 16 x 16 MMA: one 16-byte
//                            load per lane feeds four of them, and the matching B fragment is 16
//                            consecutive bytes of a bf16 row.
//   scales  [Mt][Kg][8 words] Kg groups per tile; word g = (column g, column g + 8) as two fp16, divided
//                            by the column's multiplier
//   mult    [Mt * 16] fp32   power of two per column: 2^floor(log2(max |scale|)), 1 where that is 0 or
//                            not finite.  fp16 scales below 2 then keep every bit of a bf16 scale down
//                            to 2^-14 of the column's largest one, and (code - 8) * scale has at most 11
//                            significant bits: exact in fp16.
//   meta    [4] fp32         [0] the largest column 2-norm of W (bounds |x W| by |x| times it), 0 0 0
//
// Inputs beyond K and columns beyond N have code 8 (weight 0) and scale 0.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace moe {

struct W4Dims {
  int K, N, G, Kb, Mt, Kg;
  size_t codes, scales, mult, meta, bytes;  // byte offsets of the parts, total size
};

__host__ __device__ inline W4Dims w4_dims(int K, int N, int G) {
  W4Dims d;
  d.K = K;
  d.N = N;
  d.G = G;
  d.Kb = (K + 63) / 64;
  d.Mt = (N + 15) / 16;
  d.Kg = (d.Kb * 64 + G - 1) / G;
  d.codes = 0;
  d.scales = (size_t)d.Mt * d.Kb * 512;
  d.mult = d.scales + (size_t)d.Mt * d.Kg * 32;
  d.meta = d.mult + (size_t)d.Mt * 64;
  d.bytes = d.meta + 16;
  return d;
}

inline bool w4_group_ok(int G) { return G == 32 || G == 64 || G == 128; }
// Shapes of a packed matrix: rows of x are read 16 bytes at a time (K % 8), indexes fit 32 bits.
inline bool w4_shape_ok(int K, int N, int G) {
  return w4_group_ok(G) && K >= 8 && K % 8 == 0 && K <= (1 << 20) && N >= 1 && N <= (1 << 24);
}

// Slab shapes: those of the other FFN entry points (H % 64, I % 32), in the packed matrices' range.
inline bool w4_slab_ok(int H, int I, int G) {
  return H >= 64 && H % 64 == 0 && I >= 32 && I % 32 == 0 && w4_shape_ok(H, I, G) && w4_shape_ok(I, H, G);
}

// The three matrices of an expert slab: gate and up (H x I), down (I x H).
struct W4Slab {
  W4Dims gu, dn;
  size_t bytes;
};
__host__ __device__ inline W4Slab w4_slab(int H, int I, int G) {
  W4Slab s;
  s.gu = w4_dims(H, I, G);
  s.dn = w4_dims(I, H, G);
  s.bytes = 2 * s.gu.bytes + s.dn.bytes;
  return s;
}

// Word w of a lane's 16 bytes -> the four bf16x2 registers of a 16 x 16 A fragment, as code - 8:
// a nibble in the low mantissa bits of 0x4300 is 128 + code, and 128 + code - 136 is exact.
__device__ __forceinline__ void w4_frag_bf16(uint32_t w, uint32_t (&a)[4]) {
  const uint32_t off = 0x43084308u;  // 136, 136
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t v = ((w >> (4 * i)) & 0x000f000fu) | 0x43004300u;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(a[i]) : "r"(v), "r"(off));
  }
}

// C += A(16 x 16, bf16) B(16 x 8, bf16), fp32 accumulators.
__device__ __forceinline__ void mma_bf16_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

}  // namespace moe
