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
constexpr int kCntIds = 4096;    // ids per CTA that a cluster size aims at

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
// The 32-bit word at shared::cta address p of CTA `rank` of the cluster.
__device__ __forceinline__ int bal_peer(const int* p, uint32_t rank) {
  uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(p)), r;
  int v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(r) : "memory");
  return v;
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
  int tok = 0;
  for (uint32_t r = 0; r < nc; ++r) tok += bal_peer(&ntok, r);
  const float u = (float)a.E / ((float)a.k * (float)max(tok, 1));
  for (int e = (int)(rank * kCntThreads + threadIdx.x); e < a.E; e += (int)nc * kCntThreads) {
    int c = 0;
    for (uint32_t r = 0; r < nc; ++r) c += bal_peer(&cnt[e], r);
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
  asm("ex2.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
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

// Groups of `lanes` lanes (a power of two) take a token each; a lane holds NC chunks of V values, chunk c of
// lane l being the row's (c * lanes + l)-th.  CTA b takes `per` consecutive tokens.
template <int V, int NC, bool BF16, bool SIG>
__global__ void __launch_bounds__(kBalThreads) balance_kernel(const BalArgs a, int lanes, int per) {
  constexpr int W = kBalThreads / 32;
  __shared__ int s_red[W];
  __shared__ double s_loss[W];
  __shared__ int s_last;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gl = lane & (lanes - 1), groups = kBalThreads / lanes, g = threadIdx.x / lanes;
  const int t_end = min((int)(blockIdx.x + 1) * per, a.T);
  auto fetch = [&](int t, BalVec<BF16, V> (&x)[NC]) {
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int e = (c * lanes + gl) * V;
      if (t < t_end && e < a.E) x[c].load(a.logits, (size_t)t * a.E + e);
    }
  };
  BalVec<BF16, V> x[NC];
  int t = blockIdx.x * per + g;
  fetch(t, x);
  pdl_wait();
  // valid tokens of all sequences
  int tv = 0;
  for (int s = threadIdx.x; s < a.n_seq; s += kBalThreads) tv += a.tokens[s];
  tv = __reduce_add_sync(MOE_FULL_MASK, tv);
  if (lane == 0) s_red[warp] = tv;
  int sid = t < t_end ? a.seqid[t] : -1;
  __syncthreads();
  tv = 0;
  for (int w = 0; w < W; ++w) tv += s_red[w];
  const float gscale = a.coef / (float)max(tv, 1) * (a.grad && a.grad_out ? *a.grad_out : 1.f);

  float loss = 0.f;
  for (; t - g < t_end; t += groups) {  // the same number of rounds for every lane
    const bool in = t < t_end, valid = in && sid >= 0 && sid < a.n_seq;
    const float* fr = a.f + (size_t)(valid ? sid : 0) * a.E;
    const int tn = t + groups;
    const int sn = tn < t_end ? a.seqid[tn] : -1;
    float mx = -INFINITY;
    float q[NC * V], keep[SIG ? NC * V : 1];
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const bool has = valid && (c * lanes + gl) * V < a.E;
        q[c * V + j] = has ? x[c].at(j) : -INFINITY;
        mx = fmaxf(mx, q[c * V + j]);
      }
    fetch(tn, x);
    for (int o = lanes >> 1; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(MOE_FULL_MASK, mx, o));
    float sum = 0.f, dot = 0.f;
    // softmax: exp(l - max).  sigmoid: sigma(l), or, where the largest logit is below -20, sigma(l) / exp(max):
    // the sum takes the factor out, and nothing underflows that counts.
    const float ref = SIG ? (mx < -20.f ? mx : 0.f) : mx;
    const float shift = -(ref == -INFINITY ? 0.f : ref) * kLog2e;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int e0 = (c * lanes + gl) * V;
      float f[V];
      if constexpr (V == 1) {
        f[0] = e0 < a.E ? __ldg(fr + e0) : 0.f;
      } else {
#pragma unroll
        for (int j = 0; j < V; j += 4) {
          const float4 w = e0 < a.E ? __ldg(reinterpret_cast<const float4*>(fr + e0 + j)) : make_float4(0.f, 0.f, 0.f, 0.f);
          f[j] = w.x, f[j + 1] = w.y, f[j + 2] = w.z, f[j + 3] = w.w;
        }
      }
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int i = c * V + j;
        const float l = q[i];
        if (SIG) {
          const float em = bal_exp2(-fabsf(l) * kLog2e);  // sigma = 1 / (1 + em) or em / (1 + em)
          const float inv = __fdividef(1.f, 1.f + em);
          const float lo = mx < -20.f ? bal_exp2(fmaf(l, kLog2e, shift)) : em;
          keep[i] = (l >= 0.f ? em : 1.f) * inv;
          q[i] = (l >= 0.f ? 1.f : lo) * inv;
        } else {
          q[i] = bal_exp2(fmaf(l, kLog2e, shift));
        }
        sum += q[i];
        dot = fmaf(q[i], f[j], dot);
      }
    }
    for (int o = lanes >> 1; o; o >>= 1) {
      sum += __shfl_xor_sync(MOE_FULL_MASK, sum, o);
      dot += __shfl_xor_sync(MOE_FULL_MASK, dot, o);
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;  // a row of -inf has no probabilities, nor has one left out
    const float dt = dot * inv;
    loss += dt;
    if (a.grad && in) {
      const float gs = gscale * inv;
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int e0 = (c * lanes + gl) * V;
        if (e0 >= a.E) continue;
        float v[V];
        if constexpr (V == 1) {
          v[0] = __ldg(fr + e0);
        } else {
#pragma unroll
          for (int j = 0; j < V; j += 4) {
            const float4 w = __ldg(reinterpret_cast<const float4*>(fr + e0 + j));
            v[j] = w.x, v[j + 1] = w.y, v[j + 2] = w.z, v[j + 3] = w.w;
          }
        }
#pragma unroll
        for (int j = 0; j < V; ++j) {
          v[j] = gs * q[c * V + j] * (v[j] - dt);
          if (SIG) v[j] *= keep[c * V + j];
        }
        BalVec<BF16, V>::store(a.grad, (size_t)t * a.E + e0, v);
      }
    }
    sid = sn;
  }
  if (!a.loss) return;
  // one value per token group, then the groups of a warp, the warps, the CTAs: a fixed order
  if (gl != 0) loss = 0.f;
#pragma unroll
  for (int o = 16; o; o >>= 1) loss += __shfl_xor_sync(MOE_FULL_MASK, loss, o);
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
  if (s_last && warp == 0) {
    // the last CTA adds the parts: 32 strided sums, then their tree
    __threadfence();
    double v = 0.;
    for (int i = lane; i < (int)gridDim.x; i += 32) v += *(volatile double*)(a.part + i);
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(MOE_FULL_MASK, v, o);
    if (lane == 0) *a.loss = (float)(v * ((double)a.coef / max(tv, 1)));
  }
}

constexpr int kBalMaxGrid = 4096;

static size_t bal256(size_t v) { return (v + 255) & ~size_t(255); }

template <int V, int NC>
static int launch_pass(const BalArgs& a, bool bf16, bool sig, int lanes, int sms, cudaStream_t s) {
  // CTAs of whole rounds of tokens, up to six per SM
  const int groups = kBalThreads / lanes, most = std::min(sms * 6, kBalMaxGrid);
  const int rounds = (int)(((int64_t)a.T + (int64_t)most * groups - 1) / ((int64_t)most * groups));
  const int per = rounds * groups;
  const dim3 grid((a.T + per - 1) / per), block(kBalThreads);
  cudaError_t e;
  if (bf16) {
    e = sig ? launch_pdl(balance_kernel<V, NC, true, true>, grid, block, 0, s, a, lanes, per)
            : launch_pdl(balance_kernel<V, NC, true, false>, grid, block, 0, s, a, lanes, per);
  } else if constexpr (V <= 4) {
    e = sig ? launch_pdl(balance_kernel<V, NC, false, true>, grid, block, 0, s, a, lanes, per)
            : launch_pdl(balance_kernel<V, NC, false, false>, grid, block, 0, s, a, lanes, per);
  } else {
    e = cudaErrorInvalidValue;
  }
  MOE_CUDA_TRY(e);
  return MOE_OK;
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
  // 16-byte chunks where every row starts on one; lanes: about 16 values each, so that few reductions are
  // needed and a warp has several rows in flight
  const int v = bf16 ? 8 : 4;
  const bool vec = E % v == 0 && (uintptr_t)logits % 16 == 0 && (uintptr_t)grad_logits % 16 == 0;
  const int chunks = vec ? E / v : E;
  if (!vec) {
    if (E <= 128) return launch_pass<1, 4>(a, bf16, sig, 32, sms, s);
    if (E <= 384) return launch_pass<1, 12>(a, bf16, sig, 32, sms, s);
    return launch_pass<1, 32>(a, bf16, sig, 32, sms, s);
  }
  int lanes = 1;
  while (lanes < 32 && lanes * (bf16 ? 2 : 4) < chunks) lanes *= 2;
  const int nc2 = (chunks + lanes - 1) / lanes;
  if (bf16) {
    if (nc2 <= 2) return launch_pass<8, 2>(a, bf16, sig, lanes, sms, s);
    return launch_pass<8, 4>(a, bf16, sig, lanes, sms, s);
  }
  if (nc2 <= 3) return launch_pass<4, 3>(a, bf16, sig, lanes, sms, s);
  if (nc2 <= 4) return launch_pass<4, 4>(a, bf16, sig, lanes, sms, s);
  return launch_pass<4, 8>(a, bf16, sig, lanes, sms, s);
}
