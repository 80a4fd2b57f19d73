// Low-rank adapters of many requests beside a shared projection, and their gradients.
//
// Sequence q of a batch is the rows [seq[q], seq[q + 1]) and has the adapter l = ids[q], or none:
//   v = s_l x A_l^T  (R values a row),   out = base + v B_l;
//   dv = s_l dy B_l^T,   dx = base + dv A_l,   dA_l = sum_t dv_t x_t^T,   dB_l = sum_t v_t dy_t^T.
// A [L][R][K] and B [L][R][N] both run along the features, so the gradient's dx is the forward pass with A and B
// exchanged, and dA and dB are one kernel.
#include <algorithm>

#include "adapters.cuh"

namespace moe {

constexpr int kRowThreads = 256;
constexpr int kRowCluster = 8;

__device__ __forceinline__ uint32_t ad_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void ad_cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void ad_cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void ad_store_remote(float* p, uint32_t rank, float v) {
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
               : "=r"(at)
               : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(p))), "r"(rank));
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at), "f"(v) : "memory");
}

__device__ __forceinline__ float ad_dot8(uint4 x, uint4 w, float s) {
  const uint32_t a[4] = {x.x, x.y, x.z, x.w}, b[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    s = fmaf(bf16_lo(a[i]), bf16_lo(b[i]), s);
    s = fmaf(bf16_hi(a[i]), bf16_hi(b[i]), s);
  }
  return s;
}
__device__ __forceinline__ void ad_axpy8(float v, uint4 w, float (&acc)[8]) {
  const uint32_t b[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    acc[2 * i] = fmaf(v, bf16_lo(b[i]), acc[2 * i]);
    acc[2 * i + 1] = fmaf(v, bf16_hi(b[i]), acc[2 * i + 1]);
  }
}

// out = base + acc over 8 values, one rounding.
template <bool F32>
__device__ __forceinline__ void ad_add8(const void* base, void* out, long long ib, long long io, const float (&acc)[8]) {
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = acc[i];
  if (F32) {
    if (base) {
      const float4* p = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(base) + ib);
      const float4 b0 = p[0], b1 = p[1];
      v[0] += b0.x, v[1] += b0.y, v[2] += b0.z, v[3] += b0.w, v[4] += b1.x, v[5] += b1.y, v[6] += b1.z, v[7] += b1.w;
    }
    float4* q = reinterpret_cast<float4*>(reinterpret_cast<float*>(out) + io);
    q[0] = make_float4(v[0], v[1], v[2], v[3]);
    q[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    if (base) {
      const uint4 b = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(base) + ib);
      const uint32_t u[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) v[2 * i] += bf16_lo(u[i]), v[2 * i + 1] += bf16_hi(u[i]);
    }
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 q = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      o[i] = *reinterpret_cast<const uint32_t*>(&q);
    }
    *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(out) + io) = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

// One cluster of CTAs per row, or per sequence of up to max_rows rows: CTA c takes its share of the K inputs for all R
// products, the partial sums meet in every CTA's shared memory, and CTA c computes its share of the N outputs.  One
// launch, no workspace.  One row of R 16 (2048 x 2048) 3.9 us, 64 rows of 64 adapters (2048 x 4096, 1.3 us of weight bytes)
// 5.5: the launch, ids -> weights -> cluster -> outputs.  With 64 registers four CTAs are resident (three: 8.6, five: 7.0).
template <bool F32>
__global__ void __launch_bounds__(kRowThreads, 4) adapters_row_kernel(const AdArgs a, int max_rows) {
  __shared__ __align__(16) float s_red[kRowThreads * 8];
  __shared__ float s_part[2][kRowCluster][kAdMaxR];
  __shared__ float s_v[kAdMaxR];
  pdl_wait();
  pdl_trigger();  // what follows waits for this kernel, or has other rows
  const int c = (int)ad_rank(), unit = blockIdx.x / kRowCluster;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int s = unit, t0 = unit, t1 = unit + 1;
  if (max_rows) {
    t0 = min(max(a.seq[s], 0), a.T);
    t1 = min(max(a.seq[s + 1], 0), a.T);
    if (t1 - t0 > max_rows || t1 <= t0) return;
  } else {
    s = ad_sequence(a, unit);
    if (unit == 0 && a.seq)
      for (int q = c * kRowThreads + tid; q < a.n_seq; q += kRowCluster * kRowThreads)
        if (a.seq[q + 1] < a.seq[q]) set_status(a.status, MOE_DEV_BAD_GROUPS);
  }
  const int l = s < 0 ? -1 : ad_adapter(a, s);
  const int nv = a.N / 8, n0 = nv * c / kRowCluster, n1 = nv * (c + 1) / kRowCluster;
  if (l < 0) {
    const float none[8] = {};
    for (int t = t0; t < t1; ++t) {
      if (a.kept && c == 0)
        for (int r = tid; r < a.R; r += kRowThreads) a.kept[(size_t)t * a.R + r] = 0.f;
      if (a.out && (a.out != a.base || a.ldo != a.ldb))
        for (int j = n0 + tid; j < n1; j += kRowThreads)
          ad_add8<F32>(a.base, a.out, t * a.ldb + 8 * j, t * a.ldo + 8 * j, none);
    }
    return;
  }
  ad_cluster_arrive();
  const int kv = a.K / 8, k0 = kv * c / kRowCluster, k1 = kv * (c + 1) / kRowCluster, kn = k1 - k0;
  const uint4* w1 = reinterpret_cast<const uint4*>(a.w1 + (size_t)l * a.R * a.K) + k0;
  const uint4* w2 = reinterpret_cast<const uint4*>(a.w2 + (size_t)l * a.R * a.N);
  // outputs: `wide` threads side by side, the ranks divided among groups of them.  The first weights of both products
  // are on their way before anything is waited for.
  int wide = 32;
  while (wide < n1 - n0 && wide < kRowThreads) wide *= 2;
  const int groups = kRowThreads / wide, rg = tid / wide, j0 = n0 + tid % wide;
  constexpr int P1 = 2, P2 = 4;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  uint4 h1[P1], h2[P2];
#pragma unroll
  for (int i = 0; i < P1; ++i) {
    const int r = warp + i * (kRowThreads / 32);
    h1[i] = lane < kn && r < a.R ? w1[(size_t)r * kv + lane] : zero;
  }
#pragma unroll
  for (int i = 0; i < P2; ++i) {
    const int r = rg + i * groups;
    h2[i] = a.out && j0 < n1 && r < a.R ? w2[(size_t)r * nv + j0] : zero;
  }
  const float scale = a.scale[l];
  ad_cluster_wait();  // the other CTAs have started
  for (int t = t0; t < t1; ++t) {
    float(*part)[kAdMaxR] = s_part[t & 1];
    const uint4* xr = reinterpret_cast<const uint4*>(a.x + t * a.ldx) + k0;
    const uint4 x0 = lane < kn ? xr[lane] : zero;
#pragma unroll 2
    for (int i = 0; warp + i * (kRowThreads / 32) < a.R; ++i) {
      const int r = warp + i * (kRowThreads / 32);
      const uint4 first = i == 0 ? h1[0] : i == 1 ? h1[1] : lane < kn ? w1[(size_t)r * kv + lane] : zero;
      float sum = ad_dot8(x0, first, 0.f);
      for (int k = lane + 32; k < kn; k += 32) sum = ad_dot8(xr[k], w1[(size_t)r * kv + k], sum);
#pragma unroll
      for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(MOE_FULL_MASK, sum, o);
      if (lane < kRowCluster) ad_store_remote(&part[c][r], lane, sum);
    }
    ad_cluster_arrive();
    ad_cluster_wait();
    for (int r = tid; r < a.R; r += kRowThreads) {
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < kRowCluster; ++i) sum += part[i][r];
      sum *= scale;
      s_v[r] = sum;
      if (a.kept && c == 0) a.kept[(size_t)t * a.R + r] = sum;
    }
    __syncthreads();
    if (a.parts && c == 0) {
      const int Rk = (a.R + 15) / 16 * 16, g8 = Rk / 8;
      for (int i = tid; i < 2 * g8; i += kRowThreads) {
        const int which = i / g8, r = i % g8 * 8;
        float v[8];
        if (which) {
          ad_load8(a.fwd + (size_t)t * a.R, a.R, r, v);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] = r + j < a.R ? s_v[r + j] : 0.f;
        }
        ad_put_parts(a.parts + ((size_t)which * a.T + t) * 3 * Rk, Rk, r, v);
      }
    }
    if (a.out)
      for (int from = n0; from < n1; from += wide) {  // (the same rounds for every thread)
        const int j = from + tid % wide;
        float acc[8] = {};
        if (j < n1) {
#pragma unroll
          for (int i = 0; i < P2; ++i) {
            const int r = rg + i * groups;
            if (r < a.R) ad_axpy8(s_v[r], from == n0 ? h2[i] : w2[(size_t)r * nv + j], acc);
          }
#pragma unroll 4
          for (int r = rg + P2 * groups; r < a.R; r += groups) ad_axpy8(s_v[r], w2[(size_t)r * nv + j], acc);
        }
        if (groups > 1) {
          if (rg > 0)
#pragma unroll
            for (int i = 0; i < 8; i += 4)
              *reinterpret_cast<float4*>(&s_red[(tid - wide) * 8 + i]) = make_float4(acc[i], acc[i + 1], acc[i + 2], acc[i + 3]);
          __syncthreads();
          if (rg == 0)
            for (int q = 0; q < groups - 1; ++q)
#pragma unroll
              for (int i = 0; i < 8; ++i) acc[i] += s_red[(q * wide + tid) * 8 + i];
        }
        if (rg == 0 && j < n1) ad_add8<F32>(a.base, a.out, t * a.ldb + 8 * j, t * a.ldo + 8 * j, acc);
      }
    __syncthreads();  // s_v and s_red are free again
  }
}

static int ad_launch_rows(const AdArgs& a, bool f32, int units, int max_rows, cudaStream_t s) {
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = kRowCluster;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)units * kRowCluster);
  cfg.blockDim = dim3(kRowThreads);
  cfg.stream = s;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  if (f32) MOE_CUDA_TRY(cudaLaunchKernelEx(&cfg, adapters_row_kernel<true>, a, max_rows));
  else MOE_CUDA_TRY(cudaLaunchKernelEx(&cfg, adapters_row_kernel<false>, a, max_rows));
  return MOE_OK;
}

static int ad_sms(int* sms) {
  int dev = 0;
  MOE_CUDA_TRY(cudaGetDevice(&dev));
  MOE_CUDA_TRY(cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev));
  return MOE_OK;
}

// Sequences of up to so many rows take the row kernel in a batch of short and long ones (36 single rows and four prompts of
// 1001 rows: 15.4 us; a tile of 32 rows takes 8 us for one row, too).
constexpr int kShortRows = 4;

static int ad_run(const AdArgs& a, bool f32, cudaStream_t s) {
  if (!a.seq || a.T <= kShortRows) return ad_launch_rows(a, f32, a.T, 0, s);
  if (a.n_seq == 1 || a.T >= 64ll * a.n_seq) return ad_launch_tiles(a, f32, 0, false, s);
  if (int rc = ad_launch_rows(a, f32, a.n_seq, kShortRows, s)) return rc;
  return ad_launch_tiles(a, f32, kShortRows, true, s);
}

static bool ad_shape(int T, int K, int N, int R, int L, const int32_t* seq, int n_seq) {
  return T >= 1 && T <= (1 << 24) && K >= 8 && K <= (1 << 17) && N >= 8 && N <= (1 << 17) && R >= 1 && R <= kAdMaxR &&
         L >= 1 && L <= 65535 && n_seq >= 1 && n_seq <= (1 << 24) && (seq || n_seq == T);
}
// Rows of n elements, ld apart.
static bool ad_ld_ok(long long ld, int n) { return ld >= n && ld < (1ll << 31); }
// Rows of `ld` elements of `size` bytes start on 16 bytes.
static bool ad_rows_ok(const void* p, long long ld, int size) { return (uintptr_t)p % 16 == 0 && ld * size % 16 == 0; }
// Whether T rows of n bytes, ld apart, and T rows of m bytes, le apart, have no byte in common: apart, or side by side in
// rows of one stride.  (Rows of two strides over one range count as overlapping.)
static bool ad_apart(const void* p, long long ld, long long n, const void* q, long long le, long long m, int T) {
  const long long a = (long long)(uintptr_t)p, b = (long long)(uintptr_t)q;
  if (a + (T - 1) * ld + n <= b || b + (T - 1) * le + m <= a) return true;
  if (T == 1 || ld != le) return false;
  const long long d = ((b - a) % ld + ld) % ld;  // q's rows begin d bytes into p's
  return d >= n && d + m <= ld;
}
static size_t ad256(size_t v) { return (v + 255) & ~size_t(255); }

}  // namespace moe

using namespace moe;

extern "C" int moe_adapters(const void* x, long long ldx, const void* base, long long ldb, int T, int K, int N, int R,
                            int L, const void* a, const void* b, const float* scale, const int32_t* ids,
                            const int32_t* seq_start, int n_seq, void* out, long long ldo, int out_f32, float* kept,
                            int32_t* dev_status, moe_stream_t stream) {
  if (!x || !a || !b || !scale || !ids || !out || (out_f32 != 0 && out_f32 != 1)) return MOE_ERR_ARG;
  if (!ad_shape(T, K, N, R, L, seq_start, n_seq)) return MOE_ERR_ARG;
  if (!ad_ld_ok(ldx, K) || !ad_ld_ok(ldo, N) || (base && !ad_ld_ok(ldb, N))) return MOE_ERR_ARG;
  const int size = out_f32 ? 4 : 2;
  if (!ad_apart(x, ldx * 2, K * 2, out, ldo * size, N * size, T) ||
      (base && (base != out || ldb != ldo) && !ad_apart(base, ldb * size, N * size, out, ldo * size, N * size, T)))
    return MOE_ERR_ARG;
  if (K % 8 || N % 8 || !ad_rows_ok(x, ldx, 2) || !ad_rows_ok(out, ldo, size) || (base && !ad_rows_ok(base, ldb, size)) || (uintptr_t)a % 16 || (uintptr_t)b % 16)
    return MOE_ERR_ALIGN;
  const AdArgs g{(const uint16_t*)x, (const uint16_t*)a, (const uint16_t*)b, scale, ids, seq_start, base, out, kept,
                 nullptr, nullptr, dev_status, ldx, base ? ldb : 0, ldo, T, K, N, R, L, n_seq};
  return ad_run(g, out_f32 != 0, (cudaStream_t)stream);
}

extern "C" size_t moe_adapters_grad_workspace_bytes(int T, int R) {
  if (T < 1 || R < 1 || R > kAdMaxR) return 0;
  return ad256((size_t)T * R * 4) + (size_t)T * ((R + 15) / 16 * 16) * 12;
}

extern "C" int moe_adapters_grad(const void* dy, long long ldy, const void* x, long long ldx, const float* kept,
                                 const void* base, long long ldb, int T, int K, int N, int R, int L, const void* a,
                                 const void* b, const float* scale, const int32_t* ids, const int32_t* seq_start,
                                 int n_seq, void* dx, long long lddx, float* da, float* db, void* workspace,
                                 size_t workspace_bytes, int32_t* dev_status, moe_stream_t stream) {
  if (!dy || !a || !b || !scale || !ids || !workspace || (!dx && !da) || (!da != !db) || (da && (!x || !kept)))
    return MOE_ERR_ARG;
  if (!ad_shape(T, K, N, R, L, seq_start, n_seq)) return MOE_ERR_ARG;
  // each block of features of each adapter looks at all sequences: about a second's work at the limit
  if (da && (long long)L * n_seq > (1ll << 44) / (K + N)) return MOE_ERR_ARG;
  if (!ad_ld_ok(ldy, N) || (da && !ad_ld_ok(ldx, K)) || (dx && !ad_ld_ok(lddx, K)) || (dx && base && !ad_ld_ok(ldb, K)))
    return MOE_ERR_ARG;
  if (dx && (dx == x || !ad_apart(dy, ldy * 2, N * 2, dx, lddx * 2, K * 2, T) ||
             (da && !ad_apart(x, ldx * 2, K * 2, dx, lddx * 2, K * 2, T)) ||
             (base && (base != dx || ldb != lddx) && !ad_apart(base, ldb * 2, K * 2, dx, lddx * 2, K * 2, T))))
    return MOE_ERR_ARG;
  if (K % 8 || N % 8 || !ad_rows_ok(dy, ldy, 2) || (da && !ad_rows_ok(x, ldx, 2)) || (dx && !ad_rows_ok(dx, lddx, 2)) ||
      (dx && base && !ad_rows_ok(base, ldb, 2)) || (uintptr_t)a % 16 ||
      (uintptr_t)b % 16 || (uintptr_t)da % 16 || (uintptr_t)db % 16 || (uintptr_t)workspace % 256 ||
      workspace_bytes < moe_adapters_grad_workspace_bytes(T, R))
    return MOE_ERR_ALIGN;
  cudaStream_t s = (cudaStream_t)stream;
  // dv in fp32 for the short sequences' kernel, in parts (with kept) for the tiles'
  float* dv = (float*)workspace;
  uint16_t* parts = (uint16_t*)((char*)workspace + ad256((size_t)T * R * 4));
  const AdOuter by = ad_outer_by(T, n_seq, seq_start);
  const bool tiles = by != AdOuter::kShort;
  const AdArgs g{(const uint16_t*)dy, (const uint16_t*)b, (const uint16_t*)a, scale, ids, seq_start, dx ? base : nullptr,
                 dx, da && by != AdOuter::kTiles ? dv : nullptr, kept, da && tiles ? parts : nullptr, dev_status, ldy,
                 dx && base ? ldb : 0, lddx, T, N, K, R, L, n_seq};
  if (int rc = ad_run(g, false, s)) return rc;
  if (!da) return MOE_OK;
  const AdGradArgs o{(const uint16_t*)x, (const uint16_t*)dy, dv, kept, ids, seq_start, da, db, tiles ? parts : nullptr,
                     dev_status, ldx, ldy, T, K, N, R, L, n_seq, by == AdOuter::kBoth};
  int sms = 0;
  if (int rc = ad_sms(&sms)) return rc;
  return ad_launch_outer(o, sms, s);
}
