// Packing of 4-bit matrices (format: w4.cuh), from codes and scales or from bf16 weights.  Done once
// per matrix, before serving.
#include <algorithm>

#include "internal.cuh"
#include "w4.cuh"

namespace moe {

// One matrix of a call: where its columns come from and where it goes.
struct W4PackMat {
  W4Dims d;
  int paired;           // gate and up: tile t of 16 columns is tile t / 2 of source t % 2 (N / 2 columns each)
  size_t src, scale;    // first element of its codes or weights, and of its scales, in an item
  size_t dst, meta;     // byte offsets in an item's packed form: the matrix, and a paired one's second meta
};

// The matrices of one call: `count` items of one matrix or, for a slab, two (gate / up, down).
struct W4PackArgs {
  int mats;
  W4PackMat m[2];
  const uint8_t* codes;     // [item][...] bytes 0..15, or NULL: quantise `w`
  const uint16_t* scales;   // bf16 [item][...]
  const uint16_t* w;        // bf16 [item][...] weights
  size_t src_item, scale_item, dst_item;  // elements / elements / bytes per item
  uint8_t* dst;
};

// Groups of the source's scale array: ceil(K / G) (the packed form may hold one more).
__host__ __device__ __forceinline__ int src_groups(const W4Dims& d) { return (d.K + d.G - 1) / d.G; }
// Source column of packed column n: its offset among the rows' first elements (of codes: k = 0; of scales: group 0).
__device__ __forceinline__ size_t src_col(const W4PackMat& m, int n, int rows) {
  if (!m.paired) return n;
  const int t = n >> 4;
  return (size_t)(t & 1) * rows * (m.d.N / 2) + (t >> 1) * 16 + (n & 15);
}
__device__ __forceinline__ int src_ld(const W4PackMat& m) { return m.paired ? m.d.N / 2 : m.d.N; }

constexpr int kPackCols = 128;  // output columns of a CTA: 8 tiles
constexpr int kPackRows = 128;  // inputs of a CTA: whole groups for every group size

// One CTA: 128 inputs x 128 output columns of one matrix; codes are staged as bytes in shared memory.
// The scales are left in the packed array as raw bf16; w4_scale_kernel normalises them.
__global__ void __launch_bounds__(256) w4_pack_kernel(const W4PackArgs a) {
  __shared__ uint8_t sc[kPackRows][kPackCols + 4];
  const W4PackMat& m = a.m[blockIdx.z % a.mats];
  const size_t item = blockIdx.z / a.mats;
  const W4Dims& d = m.d;
  const int k0 = blockIdx.y * kPackRows, n0 = blockIdx.x * kPackCols, ld = src_ld(m);
  if (k0 >= d.Kb * 64 || n0 >= d.Mt * 16) return;
  uint8_t* dst = a.dst + item * a.dst_item + m.dst;
  uint16_t* dsc = reinterpret_cast<uint16_t*>(dst + d.scales);
  const int rows = min(kPackRows, d.Kb * 64 - k0);
  const int gpc = kPackRows / d.G;  // groups of this CTA's inputs
  if (a.codes) {
    const uint8_t* src = a.codes + item * a.src_item + m.src;
    for (int i = threadIdx.x; i < rows * kPackCols; i += 256) {
      const int r = i / kPackCols, c = i % kPackCols, k = k0 + r, n = n0 + c;
      sc[r][c] = k < d.K && n < d.N ? src[src_col(m, n, d.K) + (size_t)k * ld] & 15 : 8;
    }
    const uint16_t* ss = a.scales + item * a.scale_item + m.scale;
    for (int i = threadIdx.x; i < gpc * kPackCols; i += 256) {
      const int g = k0 / d.G + i / kPackCols, n = n0 + i % kPackCols;
      if (g < d.Kg && n < d.Mt * 16)
        dsc[w4_scale_at(d, n >> 4, g, n & 7) * 2 + ((n >> 3) & 1)] =
            g < src_groups(d) && n < d.N ? ss[src_col(m, n, src_groups(d)) + (size_t)g * ld] : 0;
    }
  } else {
    const uint16_t* src = a.w + item * a.src_item + m.src;
    for (int i = threadIdx.x; i < gpc * kPackCols; i += 256) {
      const int lg = i / kPackCols, c = i % kPackCols, g = k0 / d.G + lg, n = n0 + c;
      if (g >= d.Kg) continue;
      const int kb = k0 + lg * d.G, ke = min(kb + d.G, d.K);
      // the weight furthest from zero gets code 0: scale = w / -8, rounded to bf16; NaN where a weight is, as no code can
      // say so
      float hi = 0.f, lo = 0.f, nan = 0.f;
      const uint16_t* col = src + src_col(m, min(n, d.N - 1), d.K);
      if (n < d.N)
        for (int k = kb; k < ke; ++k) {
          const float v = bf16_to_f32(col[(size_t)k * ld]);
          hi = fmaxf(hi, v);
          lo = fminf(lo, v);
          if (v != v) nan = v;
        }
      const uint16_t sb = f32_to_bf16((hi > -lo ? hi : lo) * -0.125f + nan);
      const float s = bf16_to_f32(sb);
      for (int k = kb; k < min(kb + d.G, d.Kb * 64); ++k) {
        int code = 8;
        if (n < d.N && k < ke && s != 0.f) {
          const float q = rintf(__fdiv_rn(bf16_to_f32(col[(size_t)k * ld]), s));
          code = (int)fminf(fmaxf(q, -8.f), 7.f) + 8;
        }
        sc[k - k0][c] = (uint8_t)code;
      }
      if (n < d.Mt * 16) dsc[w4_scale_at(d, n >> 4, g, n & 7) * 2 + ((n >> 3) & 1)] = sb;
    }
  }
  __syncthreads();
  // words: [tile][block][lane][s]
  const int nb = rows / 64, nt = min(kPackCols / 16, d.Mt - n0 / 16);
  uint32_t* out = reinterpret_cast<uint32_t*>(dst);
  for (int i = threadIdx.x; i < nt * nb * 128; i += 256) {
    const int wd = i & 127, b = (i >> 7) % nb, t = (i >> 7) / nb;
    const int ch = wd >> 2, g = ch >> 2, q = (ch - (g >> 1)) & 3;
    const int k = b * 64 + 32 * (wd & 1) + 8 * q, c = t * 16 + g + 8 * ((wd >> 1) & 1);
    uint32_t v = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) v |= w4_put(sc[k + j][c], w4_code_bit(j));
    out[w4_code_at(d, n0 / 16 + t, k0 / 64 + b) * 128 + wd] = v;
  }
}

// One thread per output column: the column's multiplier, its scales as normalised fp16, and the
// largest column 2-norm of the matrix (meta[0], zeroed before; an integer maximum of non-negative
// floats, so the order of the columns does not matter).
__global__ void __launch_bounds__(128) w4_scale_kernel(const W4PackArgs a) {
  const W4PackMat& m = a.m[blockIdx.y % a.mats];
  const size_t item = blockIdx.y / a.mats;
  const W4Dims& d = m.d;
  const int n = blockIdx.x * 128 + threadIdx.x;
  if (n >= d.Mt * 16) return;
  uint8_t* dst = a.dst + item * a.dst_item + m.dst;
  const int tile = n >> 4, g = n & 7, h = (n >> 3) & 1;
  uint16_t* sc = reinterpret_cast<uint16_t*>(dst + d.scales) + h;
  float amax = 0.f;
  for (int i = 0; i < d.Kg; ++i) amax = fmaxf(amax, fabsf(bf16_to_f32(sc[w4_scale_at(d, tile, i, g) * 2])));
  const int e = amax > 0.f && amax < INFINITY ? ilogbf(amax) : 0;
  // 2^-e as two factors, so that a subnormal largest scale does not overflow it
  const float f0 = ldexpf(1.f, -e / 2), f1 = ldexpf(1.f, -(e - e / 2));
  const uint32_t* words = reinterpret_cast<const uint32_t*>(dst);
  float norm = 0.f;
  for (int i = 0; i < d.Kg; ++i) {
    const size_t at = w4_scale_at(d, tile, i, g) * 2;
    const float raw = bf16_to_f32(sc[at]);
    int sq = 0;  // sum of (code - 8)^2 of the group: at most 128 * 64
    for (int b = i * d.G / 32; b < (i + 1) * d.G / 32 && b < d.Kb * 2; ++b)  // blocks of 32 inputs
      for (int q = 0; q < 4; ++q) {
        const uint32_t v = words[w4_code_at(d, tile, b >> 1) * 128 + w4_chunk(g, q) * 4 + 2 * h + (b & 1)];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int c = (int)(__funnelshift_r(v, v, w4_code_bit(j)) & 15) - 8;
          sq += c * c;
        }
      }
    const float r = raw * f0 * f1;
    norm = fmaf(r * r, (float)sq, norm);
    sc[at] = __half_as_ushort(__float2half_rn(r));
  }
  reinterpret_cast<float*>(dst + d.mult)[n] = ldexpf(1.f, e);
  // 1e-3 up: the sum above is rounded, the bound must not be below the norm.  A column with a scale that is not finite
  // has no results to bound; the others keep theirs.
  uint8_t* meta = m.paired && (tile & 1) ? a.dst + item * a.dst_item + m.meta : dst + d.meta;
  const float bound = ldexpf(sqrtf(norm) * 1.001f, e);
  if (bound < INFINITY) atomicMax(reinterpret_cast<int*>(meta), __float_as_int(bound));
}

__global__ void w4_meta_kernel(const W4PackArgs a, int n) {
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= n) return;
  const W4PackMat& m = a.m[i % a.mats];
  uint8_t* item = a.dst + (size_t)(i / a.mats) * a.dst_item;
  *reinterpret_cast<float4*>(item + m.dst + m.d.meta) = make_float4(0.f, 0.f, 0.f, 0.f);
  if (m.paired) *reinterpret_cast<float4*>(item + m.meta) = make_float4(0.f, 0.f, 0.f, 0.f);
}

static int launch_pack(const W4PackArgs& a, int count, cudaStream_t s) {
  int kc = 0, nc = 0, sc = 0;
  for (int i = 0; i < a.mats; ++i) {
    const W4Dims& d = a.m[i].d;
    kc = std::max(kc, (d.Kb * 64 + kPackRows - 1) / kPackRows);
    nc = std::max(nc, (d.Mt * 16 + kPackCols - 1) / kPackCols);
    sc = std::max(sc, (d.Mt * 16 + 127) / 128);
  }
  const int per = 65535 / a.mats;  // items per launch: the grid's z
  for (int i0 = 0; i0 < count; i0 += per) {
    const int n = std::min(per, count - i0);
    W4PackArgs b = a;
    if (b.codes) b.codes += i0 * a.src_item, b.scales += i0 * a.scale_item;
    if (b.w) b.w += i0 * a.src_item;
    b.dst += i0 * a.dst_item;
    w4_meta_kernel<<<(n * a.mats + 127) / 128, 128, 0, s>>>(b, n * a.mats);
    w4_pack_kernel<<<dim3(nc, kc, n * a.mats), 256, 0, s>>>(b);  // (kc <= 8192, nc up to 2^17: the grid's x)
    w4_scale_kernel<<<dim3(sc, n * a.mats), 128, 0, s>>>(b);
    MOE_LAUNCH_CHECK();
  }
  return MOE_OK;
}

size_t w4_slab_bytes_h(int H, int I, int group) { return w4_slab(H, I, group).bytes; }
bool w4_slab_shape_ok(int H, int I, int group) { return w4_slab_ok(H, I, group); }

static int pack_matrix(const uint8_t* codes, const uint16_t* scales, const uint16_t* w, int n, int K, int N, int G,
                       void* dst, cudaStream_t s) {
  if (!dst || n < 1 || !w4_shape_ok(K, N, G)) return MOE_ERR_ARG;
  if ((uintptr_t)dst % 16) return MOE_ERR_ALIGN;
  W4PackArgs a{};
  a.mats = 1;
  a.m[0].d = w4_dims(K, N, G);
  a.codes = codes, a.scales = scales, a.w = w;
  a.src_item = (size_t)K * N;
  a.scale_item = (size_t)((K + G - 1) / G) * N;
  a.dst_item = a.m[0].d.bytes;
  a.dst = (uint8_t*)dst;
  return launch_pack(a, n, s);
}

static int pack_slabs(const uint8_t* codes, const uint16_t* scales, const uint16_t* w, int n, int H, int I, int G,
                      void* dst, cudaStream_t s) {
  if (!dst || n < 1 || !w4_slab_ok(H, I, G)) return MOE_ERR_ARG;
  if ((uintptr_t)dst % 16) return MOE_ERR_ALIGN;
  const W4Slab sl = w4_slab(H, I, G);
  W4PackArgs a{};
  a.mats = 2;
  a.m[0] = W4PackMat{sl.gu, 1, 0, 0, 0, sl.up_meta};
  a.m[1] = W4PackMat{sl.dn, 0, (size_t)2 * H * I, (size_t)2 * ((H + G - 1) / G) * I, sl.dn_at, 0};
  a.codes = codes, a.scales = scales, a.w = w;
  a.src_item = (size_t)3 * H * I;
  a.scale_item = (size_t)2 * ((H + G - 1) / G) * I + (size_t)((I + G - 1) / G) * H;
  a.dst_item = sl.bytes;
  a.dst = (uint8_t*)dst;
  return launch_pack(a, n, s);
}

}  // namespace moe

using namespace moe;

extern "C" size_t moe_w4_bytes(int K, int N, int group) {
  return w4_shape_ok(K, N, group) ? w4_dims(K, N, group).bytes : 0;
}

extern "C" size_t moe_w4_slab_bytes(int H, int I, int group) {
  return w4_slab_ok(H, I, group) ? w4_slab(H, I, group).bytes : 0;
}

extern "C" int moe_w4_pack(const uint8_t* codes, const void* scales, int n, int K, int N, int group, void* dst,
                           moe_stream_t stream) {
  if (!codes || !scales) return MOE_ERR_ARG;
  return pack_matrix(codes, (const uint16_t*)scales, nullptr, n, K, N, group, dst, (cudaStream_t)stream);
}

extern "C" int moe_w4_quantize(const void* w, int n, int K, int N, int group, void* dst, moe_stream_t stream) {
  if (!w) return MOE_ERR_ARG;
  return pack_matrix(nullptr, nullptr, (const uint16_t*)w, n, K, N, group, dst, (cudaStream_t)stream);
}

extern "C" int moe_w4_pack_slabs(const uint8_t* codes, const void* scales, int n, int H, int I, int group, void* dst,
                                 moe_stream_t stream) {
  if (!codes || !scales) return MOE_ERR_ARG;
  return pack_slabs(codes, (const uint16_t*)scales, nullptr, n, H, I, group, dst, (cudaStream_t)stream);
}

extern "C" int moe_w4_quantize_slabs(const void* w, int n, int H, int I, int group, void* dst, moe_stream_t stream) {
  if (!w) return MOE_ERR_ARG;
  return pack_slabs(nullptr, nullptr, (const uint16_t*)w, n, H, I, group, dst, (cudaStream_t)stream);
}
