// 4-bit weights with group scales: the packed format and the device helpers its kernels share.
//
// A K x N matrix W (y = x W) holds W[k][n] = (code[k][n] - 8) * scale[k / G][n] with codes 0..15 and
// one scale per G = 32, 64 or 128 consecutive inputs of an output column.  Packed:
//
//   codes   [Mt / 8][Kb][8][512 B]  Mt = ceil(N / 16) tiles of 16 output columns, Kb = ceil(K / 64)
//                            blocks of 64 inputs; eight tiles' blocks are neighbours (the last tiles, fewer
//                            than eight, among themselves), so 128 columns x 64 inputs are one copy of
//                            4 KB.  A tile block is 32 chunks of 16 bytes, four for each pair of
//                            columns g and g + 8 (g = 0..7): chunk 4g + (q + g / 2) % 4 holds inputs
//                            8q .. 8q + 7 and 32 + 8q .. 32 + 8q + 7 of column g, then the same of
//                            column g + 8, one 32-bit word for eight inputs.  In a word, the codes of
//                            inputs 0, 2, 4, 6 start at bits 3, 7, 11, 15, those of 1, 3, 5, 7 sixteen
//                            bits further (the last one's bits 32-34 wrap to 0-2).
//   The two readers this serves: in a warp, lane 4g + q's chunk is its A fragment of four 16 x 16 MMAs
//   (one coalesced 16-byte load each), whose B fragment is 16 consecutive bytes of a bf16 row; and a
//   thread that owns one column reads its 64 inputs as four 8-byte pieces from shared memory, where the
//   rotation by g / 2 spreads sixteen columns over all banks.  A code in bits 3-6 of a half is the top of
//   a bf16 mantissa (0x4180 | code << 3 is 16 + code), one in bits 6-9 the top of an fp16 mantissa
//   (0x4c00 | code << 6 is 16 + code): there (code - 8) * scale is one fused multiply-add with -24 * scale,
//   exact for a scale of 8 significant bits.
//   scales  [Mt / 8][Kg][8 words][8] Kg groups, neighbours as for the codes (word g of all eight tiles, then
//                            word g + 1); word g = (column g, column g + 8) of the tile as two fp16, divided
//                            by the column's multiplier
//   mult    [Mt * 16] fp32   power of two per column: 2^floor(log2(max |scale|)), 1 where that is 0 or
//                            not finite.  fp16 scales below 2 then keep every bit of a bf16 scale down
//                            to 2^-14 of the column's largest one, and (code - 8) * scale has at most 11
//                            significant bits: exact in fp16.
//   meta    [4] fp32         [0] the largest column 2-norm of W (bounds |x W| by |x| times it; columns whose norm
//                            is not finite are left out), 0 0 0
//
// Inputs beyond K and columns beyond N have code 8 (weight 0) and scale 0.
#pragma once

#include <cuda_fp16.h>

#include "internal.cuh"

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

// Tiles that lie together with tile mt, and the place of its block kb (512 B units) and of word g of its group
// kg (4 B units).
__host__ __device__ __forceinline__ int w4_mates(const W4Dims& d, int mt) {
  const int left = d.Mt - (mt & ~7);
  return left < 8 ? left : 8;
}
__host__ __device__ __forceinline__ size_t w4_code_at(const W4Dims& d, int mt, int kb) {
  return (size_t)(mt & ~7) * d.Kb + (size_t)kb * w4_mates(d, mt) + (mt & 7);
}
__host__ __device__ __forceinline__ size_t w4_scale_at(const W4Dims& d, int mt, int kg, int g) {
  return ((size_t)(mt & ~7) * d.Kg + (size_t)kg * w4_mates(d, mt)) * 8 + g * w4_mates(d, mt) + (mt & 7);
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

// An expert slab: gate and up as one H x 2I matrix whose tiles of 16 columns alternate (gate 0, up 0,
// gate 1, ..), so that a feature's two products are neighbours; a second meta (its own holds the gate
// columns' largest norm, this one the up columns'); then down (I x H).
struct W4Slab {
  W4Dims gu, dn;
  size_t up_meta, dn_at, bytes;
};
__host__ __device__ inline W4Slab w4_slab(int H, int I, int G) {
  W4Slab s;
  s.gu = w4_dims(H, 2 * I, G);
  s.dn = w4_dims(I, H, G);
  s.up_meta = s.gu.bytes;
  s.dn_at = s.gu.bytes + 16;
  s.bytes = s.dn_at + s.dn.bytes;
  return s;
}

// First bit of the code of input i (0..7) in a word.
__host__ __device__ constexpr int w4_code_bit(int i) {
  return 3 + 4 * (i >> 1) + 16 * (i & 1);
}
__host__ __device__ inline uint32_t w4_put(int code, int bit) {
  const uint32_t c = (uint32_t)code;
  return bit > 28 ? (c << bit) | (c >> (32 - bit)) : c << bit;
}

// A lane's chunk within a tile block.
__device__ __forceinline__ int w4_chunk(int g, int q) { return 4 * g + ((q + (g >> 1)) & 3); }

// The words of columns g (w0) and g + 8 (w1) for one run of eight inputs -> the A fragments (bf16x2) of two
// 16 x 16 MMAs, inputs 0-3 and 4-7 of the run, as code - 8: 16 + code, then 24 off, both exact.
__device__ __forceinline__ void w4_frag_bf16(uint32_t w0, uint32_t w1, uint32_t (&a0)[4], uint32_t (&a1)[4]) {
  auto conv = [](uint32_t v) {  // two operations: the constants in registers
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(v), "r"(0x00780078u), "r"(0x41804180u));
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(r), "r"(0x41c041c0u));
    return r;
  };
  a0[0] = conv(w0);
  a0[1] = conv(w1);
  a0[2] = conv(w0 >> 4);
  a0[3] = conv(w1 >> 4);
  a1[0] = conv(w0 >> 8);
  a1[1] = conv(w1 >> 8);
  a1[2] = conv(__funnelshift_r(w0, w0, 12));
  a1[3] = conv(__funnelshift_r(w1, w1, 12));
}

// D = A(16 x 16, bf16) B(16 x 8, bf16) + C, fp32.
__device__ __forceinline__ void mma_bf16_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1,
                                               float c0, float c1, float c2, float c3) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}

// The tensor-core path (w4_gemm.cu).
size_t w4_linear_gemm_ws(int T, const W4Dims& d);
int launch_w4_linear_gemm(const uint16_t* x, size_t ldx, int T, const uint8_t* w, const W4Dims& d, void* out,
                          size_t ldo, int out_f32, void* ws, int32_t* status, cudaStream_t s);
size_t w4_ffn_gemm_ws(size_t n, int H, int I, bool yh);
int launch_ffn_w4_gemm(const FfnArgs& f, const int32_t* ids, const int32_t* pos, int group, void* ws,
                       const uint16_t** yh, const int32_t** yexp, cudaStream_t s, Prof* prof);
int launch_w4_combine(const uint16_t* yh, const int32_t* yexp, const float* w, const int32_t* pos, int T, int k, int H,
                      void* out, cudaStream_t s);

}  // namespace moe
