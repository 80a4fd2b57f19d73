// The router's balance loss over packed sequences: counts, loss, and the gradient in the logits.
//
// For a sequence s with T_s valid tokens, c[s][e] routings of expert e among them, and the router's
// probabilities p[t] (softmax of the logits, or sigmoids divided by their sum):
//   f[s][e] = E c[s][e] / (k T_s),   d[t] = sum_e f[s][e] p[t][e],   loss = coef / T_v sum_t d[t]
// over the T_v valid tokens of all sequences.  f is a constant of the gradient, so
//   dloss / dlogit[t][e] = coef / T_v p[t][e] (f[s][e] - d[t])          (softmax)
//                          ... times (1 - sigmoid(logit[t][e]))          (sigmoid)
// The counts come from the ids alone, so one pass over the logits gives loss and gradient: the bytes of
// the logits, read once, and of the gradient, written once, are what bounds it.  Two launches: the counts
// (one cluster of CTAs per sequence, its histograms meet in distributed shared memory, so nothing has to
// be zeroed), and the pass, which starts beside the first and has its first rows in registers by the time
// the counts are there.
#include <algorithm>

#include "internal.cuh"

namespace moe {

struct BalArgs {
  const void* logits;
  const int32_t* ids;
  const uint8_t* mask;        // [T] or NULL
  const int32_t* seq;         // [n_seq + 1] or NULL: one sequence of T tokens
  const float* grad_out;      // [1] or NULL: 1
  int T, E, k, n_seq;
  float coef;
  int32_t* counts;            // [n_seq][E]
  float* f;                   // [n_seq][E] (workspace)
  int32_t* seqid;             // [T] sequence of a valid token, -1 of the others (workspace)
  int32_t* tokens;            // [n_seq] valid tokens (workspace)
  double* part;               // [grid] partial losses (workspace)
  int32_t* ticket;            // [1] (workspace)
  float* loss;                // [1] or NULL
  void* grad;                 // [T][E] or NULL
  int32_t* status;
};

__device__ __forceinline__ int bal_seq_start(const BalArgs& a, int s) {
  return a.seq ? min(max(a.seq[s], 0), a.T) : (s ? a.T : 0);
}

constexpr int kCntThreads = 512;
constexpr int kCntCluster = 16;  // CTAs of a cluster, at most
constexpr int kCntIds = 1024;    // ids per CTA that a cluster size aims at

__device__ __forceinline__ uint32_t bal_cluster_ctas() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t bal_cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void bal_cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The sum of the 32-bit words at shared::cta address p of the cluster's CTAs, all of them in flight at once.
__device__ __forceinline__ int bal_cluster_sum(const int* p, uint32_t nc) {
  const uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(p));
  int v[kCntCluster], sum = 0;
#pragma unroll
  for (uint32_t r = 0; r < kCntCluster; ++r) {
    v[r] = 0;
    if (r < nc) {
      uint32_t at;
      asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(a), "r"(r));
      asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v[r]) : "r"(at));
    }
  }
#pragma unroll
  for (int r = 0; r < kCntCluster; ++r) sum += v[r];
  return sum;
}

// One cluster per sequence: its expert counts, f, valid tokens, and the tokens' sequence ids.  Integer sums:
// any order gives the same.
__global__ void __launch_bounds__(kCntThreads) balance_count_kernel(const BalArgs a) {
  __shared__ int cnt[kMaxE];
  __shared__ int ntok;
  pdl_trigger();  // the pass may start: it waits for this kernel before it reads anything of it
  const uint32_t rank = bal_cluster_rank(), nc = bal_cluster_ctas();
  const int s = blockIdx.x / nc;
  for (int e = threadIdx.x; e < a.E; e += kCntThreads) cnt[e] = 0;
  if (threadIdx.x == 0) ntok = 0;
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.ticket = 0;
  const int b0 = bal_seq_start(a, s), b1 = bal_seq_start(a, s + 1);
  if (b1 < b0 && rank == 0 && threadIdx.x == 0) set_status(a.status, MOE_DEV_BAD_GROUPS);
  __syncthreads();
  // this CTA's tokens
  const int len = max(b1 - b0, 0), per = (len + (int)nc - 1) / (int)nc;
  const int t0 = b0 + min((int)rank * per, len), t1 = b0 + min(((int)rank + 1) * per, len);
  int mine = 0;
  for (int t = t0 + (int)threadIdx.x; t < t1; t += kCntThreads) {
    const bool ok = !a.mask || a.mask[t];
    mine += ok;
    a.seqid[t] = ok ? s : -1;
  }
  mine = __reduce_add_sync(MOE_FULL_MASK, mine);
  if ((threadIdx.x & 31) == 0 && mine) atomicAdd(&ntok, mine);
  const int32_t* ids = a.ids + (size_t)t0 * a.k;
  const int n = (t1 - t0) * a.k;
  constexpr int U = 4;
  for (int i0 = threadIdx.x; i0 < n; i0 += U * kCntThreads) {
    int e[U];
    bool ok[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * kCntThreads;
      ok[u] = i < n && (!a.mask || a.mask[t0 + i / a.k]);
      e[u] = i < n ? ids[i] : 0;
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (ok[u]) {
        if (e[u] < 0 || e[u] >= a.E) set_status(a.status, MOE_DEV_BAD_EXPERT);
        else atomicAdd(&cnt[e[u]], 1);
      }
  }
  // tokens before the first sequence and after the last belong to none
  if (s == 0)
    for (int t = (int)(rank * kCntThreads + threadIdx.x); t < b0; t += (int)nc * kCntThreads) a.seqid[t] = -1;
  if (s == a.n_seq - 1)
    for (int t = b1 + (int)(rank * kCntThreads + threadIdx.x); t < a.T; t += (int)nc * kCntThreads) a.seqid[t] = -1;
  bal_cluster_sync();
  const int tok = bal_cluster_sum(&ntok, nc);
  const float u = (float)a.E / ((float)a.k * (float)max(tok, 1));
  for (int e = (int)(rank * kCntThreads + threadIdx.x); e < a.E; e += (int)nc * kCntThreads) {
    const int c = bal_cluster_sum(&cnt[e], nc);
    a.counts[(size_t)s * a.E + e] = c;
    a.f[(size_t)s * a.E + e] = (float)c * u;
  }
  if (rank == 0 && threadIdx.x == 0) a.tokens[s] = tok;
  bal_cluster_sync();  // no CTA leaves while another one reads its shared memory
}

constexpr int kBalThreads = 256;
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float bal_exp2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float bal_rcp(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// V consecutive values of a row (16 bytes, or one value).
template <bool BF16, int V>
struct BalVec {
  uint32_t r[V == 1 ? 1 : 4];
  __device__ __forceinline__ void load(const void* p, size_t i) {
    if constexpr (V == 1) {
      r[0] = BF16 ? (uint32_t)reinterpret_cast<const uint16_t*>(p)[i] << 16
                  : __float_as_uint(reinterpret_cast<const float*>(p)[i]);
    } else {
      const uint4 v = ldg_stream(reinterpret_cast<const uint8_t*>(p) + i * (BF16 ? 2 : 4));
      r[0] = v.x, r[1] = v.y, r[2] = v.z, r[3] = v.w;
    }
  }
  __device__ __forceinline__ float at(int j) const {
    if constexpr (V == 1 || !BF16) return __uint_as_float(r[j]);
    else return j & 1 ? bf16_hi(r[j / 2]) : bf16_lo(r[j / 2]);
  }
  __device__ __forceinline__ static void store(void* p, size_t i, const float (&v)[V]) {
    if constexpr (V == 1) {
      if (BF16) reinterpret_cast<uint16_t*>(p)[i] = f32_to_bf16(v[0]);
      else reinterpret_cast<float*>(p)[i] = v[0];
    } else if constexpr (BF16) {
      uint32_t o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const __nv_bfloat162 q = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
        o[j] = *reinterpret_cast<const uint32_t*>(&q);
      }
      *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(p) + i) = make_uint4(o[0], o[1], o[2], o[3]);
    } else {
      *reinterpret_cast<float4*>(reinterpret_cast<float*>(p) + i) = make_float4(v[0], v[1], v[2], v[3]);
    }
  }
};

// Groups of L lanes take a token each; a lane holds NC chunks of V values, chunk c of lane l being the row's
// (c L + l)-th.  CTA b takes `per` consecutive tokens.
//
// The usual row costs few instructions: exp of the logits as they are (or 1 / (1 + exp(-l))), no maximum.  A row whose
// sum leaves [2^-20, 2^100] is done again with the maximum taken off; for the others whatever underflows is below
// 2^-106 of the sum.  The price is the rounding of the larger argument, 2^-24 of it: the gradient's largest error is
// 2e-7 of p (f + d) for logits around 0, 4e-7 around 30, 7e-7 around 62.
// Issue slots are 44 to 49% busy and the memory 14 to 24%: the pass waits for its loads and, between a row's two
// reductions, for itself.  (16,384 x 512 bf16 with gradient 17.1 us with the counts, 30,011 x 288 sigmoid 19.8.)
template <int V, int NC, int L, bool BF16, bool SIG>
__global__ void __launch_bounds__(kBalThreads) balance_kernel(const BalArgs a, int per) {
  constexpr int W = kBalThreads / 32, G = kBalThreads / L, N = NC * V;
  __shared__ int s_red[W];
  __shared__ double s_loss[W];
  __shared__ int s_last;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gl = threadIdx.x % L, g = threadIdx.x / L;
  const int t_end = min((int)(blockIdx.x + 1) * per, a.T);
  bool has[NC];
  BalVec<BF16, V> x[NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    has[c] = (c * L + gl) * V < a.E;
#pragma unroll
    for (int j = 0; j < (V == 1 ? 1 : 4); ++j) x[c].r[j] = V > 1 && BF16 ? 0xff80ff80u : 0xff800000u;  // -inf past the row
  }
  int t = blockIdx.x * per + g;
  size_t row = (size_t)t * a.E + gl * V;  // the lane's first value
  auto fetch = [&](bool in, size_t at) {
#pragma unroll
    for (int c = 0; c < NC; ++c)
      if (in && has[c]) x[c].load(a.logits, at + c * (L * V));
  };
  fetch(t < t_end, row);
  pdl_wait();
  // valid tokens of all sequences
  int tv = 0;
  for (int s = threadIdx.x; s < a.n_seq; s += kBalThreads) tv += a.tokens[s];
  tv = __reduce_add_sync(MOE_FULL_MASK, tv);
  if (lane == 0) s_red[warp] = tv;
  int sid = t < t_end ? a.seqid[t] : -1, sid_f = -1;
  __syncthreads();
  tv = 0;
  for (int w = 0; w < W; ++w) tv += s_red[w];
  const float gscale = a.coef / (float)max(tv, 1) * (a.grad && a.grad_out ? *a.grad_out : 1.f);
  auto group_sum = [](float v) {
#pragma unroll
    for (int o = L / 2; o; o >>= 1) v += __shfl_xor_sync(MOE_FULL_MASK, v, o);
    return v;
  };

  double loss = 0.;  // (in 32 bits the roundings add up: 2^24 equal tokens were 2e-5 off)
  float f[N];
#pragma unroll
  for (int i = 0; i < N; ++i) f[i] = 0.f;
  for (; t - g < t_end; t += G, row += (size_t)G * a.E) {  // the same number of rounds for every lane
    const bool in = t < t_end, valid = in && sid >= 0 && sid < a.n_seq;
    const int sn = t + G < t_end ? a.seqid[t + G] : -1;
    if (valid && sid != sid_f) {
      sid_f = sid;
      const float* fr = a.f + (size_t)sid * a.E + gl * V;
#pragma unroll
      for (int c = 0; c < NC; ++c)
        if (has[c]) {
          if constexpr (V == 1) {
            f[c] = fr[c * L];
          } else {
#pragma unroll
            for (int j = 0; j < V; j += 4) {
              const float4 w = *reinterpret_cast<const float4*>(fr + c * (L * V) + j);
              f[c * V + j] = w.x, f[c * V + j + 1] = w.y, f[c * V + j + 2] = w.z, f[c * V + j + 3] = w.w;
            }
          }
        }
    }
    float l[N], q[N], keep[SIG ? N : 1], sum = 0.f, dot = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      l[i] = x[i / V].at(i % V);
      q[i] = bal_exp2(SIG ? -kLog2e * l[i] : kLog2e * l[i]);
      if (SIG) {
        const float em = q[i];
        q[i] = bal_rcp(1.f + em);
        keep[i] = fminf(em, 3e38f) * q[i];  // 1 - sigma
      }
      sum += q[i];
      dot = fmaf(q[i], f[i], dot);
    }
    sum = group_sum(sum);
    dot = group_sum(dot);
    const bool rare = valid && !(sum >= 0x1p-20f && sum <= 0x1p100f);
    if (__any_sync(MOE_FULL_MASK, rare)) {
      float mx = -INFINITY;
#pragma unroll
      for (int i = 0; i < N; ++i) mx = fmaxf(mx, l[i]);
#pragma unroll
      for (int o = L / 2; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(MOE_FULL_MASK, mx, o));
      const float ref = mx == -INFINITY ? 0.f : mx;
      float sum2 = 0.f, dot2 = 0.f;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        float v;
        if (SIG) {
          // sigma(l) / exp(min(max, 0)) = exp(min(l, 0) - min(max, 0)) / (1 + exp(-|l|)); NaN stays NaN
          const float em = expf(-fabsf(l[i])), r = 1.f / (1.f + em);
          v = expf(fminf(l[i], 0.f) - fminf(ref, 0.f)) * r;
          if (rare) keep[i] = (l[i] >= 0.f ? em : 1.f) * r;
        } else {
          v = expf(l[i] - ref);
        }
        sum2 += v;
        dot2 = fmaf(v, f[i], dot2);
        if (rare) q[i] = v;
      }
      sum2 = group_sum(sum2);
      dot2 = group_sum(dot2);
      if (rare) {
        sum = sum2;
        dot = dot2;
      }
    }
    fetch(t + G < t_end, row + (size_t)G * a.E);
    const float inv = sum == 0.f ? 0.f : 1.f / sum;  // a row of -inf has no probabilities
    const float dt = dot * inv;
    if (valid) loss += dt;
    if (a.grad) {
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        float v[V];
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const int i = c * V + j;
          v[j] = gscale * (q[i] * inv * (f[i] - dt));  // gscale * inv alone could leave fp32's range
          if (SIG) v[j] *= keep[i];
          if (!valid) v[j] = 0.f;
        }
        if (in && has[c]) BalVec<BF16, V>::store(a.grad, row + c * (L * V), v);
      }
    }
    sid = sn;
  }
  if (!a.loss) return;
  // one value per token group, then the groups of a warp, the warps, the CTAs: a fixed order
#pragma unroll
  for (int o = 16; o >= L; o >>= 1) loss += __shfl_xor_sync(MOE_FULL_MASK, loss, o);  // (a group's lanes hold the same)
  if (lane == 0) s_loss[warp] = loss;
  __syncthreads();
  if (threadIdx.x == 0) {
    double v = 0.;
    for (int w = 0; w < W; ++w) v += s_loss[w];
    a.part[blockIdx.x] = v;
    __threadfence();
    s_last = atomicAdd(a.ticket, 1) == (int)gridDim.x - 1;
  }
  __syncthreads();
  if (s_last) {
    // the last CTA adds the parts: strided sums, each warp's tree, the warps in order
    __threadfence();
    double v = 0.;
    for (int i = threadIdx.x; i < (int)gridDim.x; i += kBalThreads) v += __ldcg(a.part + i);
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(MOE_FULL_MASK, v, o);
    if (lane == 0) s_loss[warp] = v;
    __syncthreads();
    if (threadIdx.x == 0) {
      v = 0.;
      for (int w = 0; w < W; ++w) v += s_loss[w];
      *a.loss = (float)(v * ((double)a.coef / max(tv, 1)));
    }
  }
}

constexpr int kBalMaxGrid = 4096;

static size_t bal256(size_t v) { return (v + 255) & ~size_t(255); }

// CTAs of whole rounds of tokens, as many as are resident at once.
template <int V, int NC, int L, bool BF16>
static int launch_pass(const BalArgs& a, bool sig, int sms, cudaStream_t s) {
  auto run = [&](auto kernel, int (&resident)[64]) -> int {
    int dev = 0;
    MOE_CUDA_TRY(cudaGetDevice(&dev));
    if (dev < 0 || dev >= 64) return MOE_ERR_CUDA;
    if (resident[dev] == 0) {
      int n = 0;
      MOE_CUDA_TRY(cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, kBalThreads, 0));
      resident[dev] = std::max(n, 1);
    }
    constexpr int G = kBalThreads / L;
    const int64_t most = std::min(sms * resident[dev], kBalMaxGrid);
    const int per = (int)((a.T + most * G - 1) / (most * G)) * G;
    MOE_CUDA_TRY(launch_pdl(kernel, dim3((a.T + per - 1) / per), dim3(kBalThreads), 0, s, a, per));
    return MOE_OK;
  };
  static int r0[64] = {}, r1[64] = {};
  return sig ? run(balance_kernel<V, NC, L, BF16, true>, r1) : run(balance_kernel<V, NC, L, BF16, false>, r0);
}

// Workspace: ticket, partial losses, valid tokens per sequence, sequence of each token, f.
struct BalWs {
  size_t part, tokens, seqid, f, bytes;
};
static BalWs bal_ws(int T, int E, int n_seq) {
  BalWs w;
  w.part = 256;
  w.tokens = w.part + 8 * (size_t)kBalMaxGrid;
  w.seqid = w.tokens + bal256(4 * (size_t)n_seq);
  w.f = w.seqid + bal256(4 * (size_t)T);
  w.bytes = w.f + bal256(4 * (size_t)n_seq * E);
  return w;
}

}  // namespace moe

using namespace moe;

extern "C" size_t moe_balance_workspace_bytes(int T, int E, int n_seq) {
  if (T < 1 || E < 1 || E > kMaxE || n_seq < 1) return 0;
  return bal_ws(T, E, n_seq).bytes;
}

extern "C" int moe_balance_loss(const void* logits, int bf16, const int32_t* ids, const uint8_t* token_mask,
                                const int32_t* seq_start, int n_seq, int T, int E, int k, int rflags, float coef,
                                const float* grad_loss, int32_t* counts, float* loss, void* grad_logits,
                                void* workspace, size_t workspace_bytes, int32_t* dev_status, moe_stream_t stream) {
  if (!logits || !ids || !counts || !workspace || (!loss && !grad_logits)) return MOE_ERR_ARG;
  if (T < 1 || T > (1 << 26) || E < 1 || E > kMaxE || k < 1 || k > kMaxK || k > E || n_seq < 1 || n_seq > (1 << 26) ||
      (!seq_start && n_seq != 1))
    return MOE_ERR_ARG;
  if ((bf16 != 0 && bf16 != 1) || (rflags & ~MOE_ROUTE_SIGMOID)) return MOE_ERR_ARG;
  const BalWs w = bal_ws(T, E, n_seq);
  if ((uintptr_t)logits % (bf16 ? 2 : 4) || (uintptr_t)grad_logits % (bf16 ? 2 : 4) || (uintptr_t)workspace % 256 ||
      workspace_bytes < w.bytes)
    return MOE_ERR_ALIGN;
  int dev = 0, sms = 0;
  MOE_CUDA_TRY(cudaGetDevice(&dev));
  MOE_CUDA_TRY(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev));
  char* ws = (char*)workspace;
  const BalArgs a{logits, ids, token_mask, seq_start, grad_loss, T, E, k, n_seq, coef, counts, (float*)(ws + w.f),
                  (int32_t*)(ws + w.seqid), (int32_t*)(ws + w.tokens), (double*)(ws + w.part), (int32_t*)ws, loss,
                  grad_logits, dev_status};
  cudaStream_t s = (cudaStream_t)stream;
  // the cluster of a sequence of average length
  int nc = 1;
  while (nc < kCntCluster && (int64_t)T * k > (int64_t)n_seq * nc * kCntIds) nc *= 2;
  if (nc > 8) {
    static bool wide[64] = {};
    if (dev < 0 || dev >= 64) return MOE_ERR_CUDA;
    if (!wide[dev]) {
      MOE_CUDA_TRY(cudaFuncSetAttribute(balance_count_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1));
      wide[dev] = true;
    }
  }
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = nc;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)n_seq * nc);
  cfg.blockDim = dim3(kCntThreads);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  MOE_CUDA_TRY(cudaLaunchKernelEx(&cfg, balance_count_kernel, a));
  const bool sig = rflags & MOE_ROUTE_SIGMOID;
  // 16-byte chunks where every row starts on one; at most 16 values (bf16: 24) a lane, so that few sums cross
  // lanes and a warp has several rows in flight
  const int v = bf16 ? 8 : 4;
  const bool vec = E % v == 0 && (uintptr_t)logits % 16 == 0 && (uintptr_t)grad_logits % 16 == 0;
  if (!vec) {
    if (bf16) {
      if (E <= 128) return launch_pass<1, 4, 32, true>(a, sig, sms, s);
      if (E <= 384) return launch_pass<1, 12, 32, true>(a, sig, sms, s);
      return launch_pass<1, 32, 32, true>(a, sig, sms, s);
    }
    if (E <= 128) return launch_pass<1, 4, 32, false>(a, sig, sms, s);
    if (E <= 384) return launch_pass<1, 12, 32, false>(a, sig, sms, s);
    return launch_pass<1, 32, 32, false>(a, sig, sms, s);
  }
  const int chunks = E / v;
  if (bf16) {
    if (chunks <= 16) return launch_pass<8, 2, 8, true>(a, sig, sms, s);
    if (chunks <= 32) return launch_pass<8, 2, 16, true>(a, sig, sms, s);
    if (chunks <= 48) return launch_pass<8, 3, 16, true>(a, sig, sms, s);
    if (chunks <= 64) return launch_pass<8, 2, 32, true>(a, sig, sms, s);
    return launch_pass<8, 4, 32, true>(a, sig, sms, s);
  }
  if (chunks <= 16) return launch_pass<4, 2, 8, false>(a, sig, sms, s);
  if (chunks <= 32) return launch_pass<4, 4, 8, false>(a, sig, sms, s);
  if (chunks <= 64) return launch_pass<4, 4, 16, false>(a, sig, sms, s);
  if (chunks <= 96) return launch_pass<4, 3, 32, false>(a, sig, sms, s);
  if (chunks <= 128) return launch_pass<4, 4, 32, false>(a, sig, sms, s);
  return launch_pass<4, 8, 32, false>(a, sig, sms, s);
}
