// The router's balance loss over packed sequences: counts, loss, and the gradient in the logits.
//
// For a sequence s with T_s valid tokens, c[s][e] routings of expert e among them, and the router's
// probabilities p[t] (softmax of the logits, or sigmoids divided by their sum):
//   f[s][e] = E c[s][e] / (k T_s),   d[t] = sum_e f[s][e] p[t][e],   loss = coef / T_v sum_t d[t]
// over the T_v valid tokens of all sequences.  f is a constant of the gradient, so
//   dloss / dlogit[t][e] = coef / T_v p[t][e] (f[s][e] - d[t])          (softmax)
//                          ... times (1 - sigmoid(logit[t][e]))          (sigmoid)
// The counts come from the ids alone, so one pass over the logits gives loss and gradient.
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

constexpr int kCntThreads = 1024;

// One CTA per sequence: its expert counts and valid tokens.  Integer sums: any order gives the same.
__global__ void __launch_bounds__(kCntThreads) balance_count_kernel(const BalArgs a) {
  __shared__ int cnt[kMaxE];
  __shared__ int ntok;
  const int s = blockIdx.x;
  for (int e = threadIdx.x; e < a.E; e += kCntThreads) cnt[e] = 0;
  if (threadIdx.x == 0) {
    ntok = 0;
    if (s == 0) *a.ticket = 0;
  }
  __syncthreads();
  const int t0 = bal_seq_start(a, s), t1 = bal_seq_start(a, s + 1);
  if (t1 < t0 && threadIdx.x == 0) set_status(a.status, MOE_DEV_BAD_GROUPS);
  int mine = 0;
  for (int t = t0 + (int)threadIdx.x; t < t1; t += kCntThreads) {
    if (a.mask && !a.mask[t]) continue;
    ++mine;
    for (int j = 0; j < a.k; ++j) {
      const int e = a.ids[(size_t)t * a.k + j];
      if (e < 0 || e >= a.E) set_status(a.status, MOE_DEV_BAD_EXPERT);
      else atomicAdd(&cnt[e], 1);
    }
  }
  mine = __reduce_add_sync(MOE_FULL_MASK, mine);
  if ((threadIdx.x & 31) == 0 && mine) atomicAdd(&ntok, mine);
  __syncthreads();
  for (int e = threadIdx.x; e < a.E; e += kCntThreads) a.counts[(size_t)s * a.E + e] = cnt[e];
  if (threadIdx.x == 0) a.tokens[s] = ntok;
}

constexpr int kBalWarps = 8;

template <bool BF16>
__device__ __forceinline__ float bal_load(const void* p, size_t i) {
  return BF16 ? bf16_to_f32(reinterpret_cast<const uint16_t*>(p)[i]) : reinterpret_cast<const float*>(p)[i];
}
template <bool BF16>
__device__ __forceinline__ void bal_store(void* p, size_t i, float v) {
  if (BF16) reinterpret_cast<uint16_t*>(p)[i] = f32_to_bf16(v);
  else reinterpret_cast<float*>(p)[i] = v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(MOE_FULL_MASK, v, o);
  return v;
}
__device__ __forceinline__ float warp_maxf(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(MOE_FULL_MASK, v, o));
  return v;
}

// A warp per token, VPL logits per lane (E <= 32 VPL); a warp takes `per` consecutive tokens.
template <int VPL, bool BF16, bool SIG>
__global__ void __launch_bounds__(32 * kBalWarps) balance_kernel(const BalArgs a, int per) {
  __shared__ int s_red[kBalWarps];
  __shared__ double s_loss[kBalWarps];
  __shared__ int s_last;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // valid tokens of all sequences
  int tv = 0;
  for (int s = threadIdx.x; s < a.n_seq; s += 32 * kBalWarps) tv += a.tokens[s];
  tv = __reduce_add_sync(MOE_FULL_MASK, tv);
  if (lane == 0) s_red[warp] = tv;
  __syncthreads();
  tv = 0;
  for (int w = 0; w < kBalWarps; ++w) tv += s_red[w];
  const float unit = a.coef / (float)max(tv, 1);
  const float gscale = a.grad ? unit * (a.grad_out ? *a.grad_out : 1.f) : 0.f;

  const int t0 = min((int)(blockIdx.x * kBalWarps + warp) * per, a.T), t1 = min(t0 + per, a.T);
  int s = -1, s_end = -1;  // the sequence at hand ends before token s_end
  if (t0 < t1) {
    int lo = 0, hi = a.n_seq;  // the first sequence that ends after t0
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (bal_seq_start(a, mid + 1) > t0) hi = mid;
      else lo = mid + 1;
    }
    s = lo - 1;
    s_end = t0;
  }
  float f[VPL];
  double loss = 0.;
  for (int t = t0; t < t1; ++t) {
    if (t >= s_end) {
      do ++s;
      while (s < a.n_seq && bal_seq_start(a, s + 1) <= t);
      s_end = s < a.n_seq ? bal_seq_start(a, s + 1) : a.T;
      const float u = s < a.n_seq ? (float)a.E / ((float)a.k * (float)max(a.tokens[s], 1)) : 0.f;
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        const int e = lane + 32 * i;
        f[i] = s < a.n_seq && e < a.E ? (float)a.counts[(size_t)s * a.E + e] * u : 0.f;
      }
    }
    // tokens of no sequence count as masked
    const bool valid = s < a.n_seq && t >= bal_seq_start(a, s) && (!a.mask || a.mask[t]);
    const size_t row = (size_t)t * a.E;
    if (!valid) {
      if (a.grad)
#pragma unroll
        for (int i = 0; i < VPL; ++i)
          if (lane + 32 * i < a.E) bal_store<BF16>(a.grad, row + lane + 32 * i, 0.f);
      continue;
    }
    float l[VPL], mx = -INFINITY;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      l[i] = lane + 32 * i < a.E ? bal_load<BF16>(a.logits, row + lane + 32 * i) : -INFINITY;
      mx = fmaxf(mx, l[i]);
    }
    mx = warp_maxf(mx);
    // softmax: exp(l - max).  sigmoid: sigma(l) / sigma(max), the same up to the factor that the
    // division by the sum takes out: exp(l - max) (1 + exp(-|..|)) forms stay finite for any l.
    float sum = 0.f, dot = 0.f, q[VPL], keep[SIG ? VPL : 1];
    const float ref = mx == -INFINITY ? 0.f : mx;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      if (SIG) {
        // sigma(l) = exp(min(l, 0)) / (1 + exp(-|l|)); relative to exp(min(max, 0))
        const float em = expf(-fabsf(l[i]));
        const float inv = 1.f / (1.f + em);
        q[i] = expf(fminf(l[i], 0.f) - fminf(ref, 0.f)) * inv;
        keep[i] = l[i] >= 0.f ? em * inv : inv;  // 1 - sigma(l)
      } else {
        q[i] = expf(l[i] - ref);
      }
      sum += q[i];
      dot = fmaf(q[i], f[i], dot);
    }
    sum = warp_sum(sum);
    dot = warp_sum(dot);
    const float inv = sum == 0.f ? 0.f : 1.f / sum;  // a row of -inf has no probabilities
    const float dt = dot * inv;
    loss += dt;
    if (a.grad) {
      const float gs = gscale * inv;
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (lane + 32 * i < a.E) {
          float g = gs * q[i] * (f[i] - dt);
          if (SIG) g *= keep[i];
          bal_store<BF16>(a.grad, row + lane + 32 * i, g);
        }
    }
  }
  if (!a.loss) return;
  if (lane == 0) s_loss[warp] = loss;
  __syncthreads();
  if (threadIdx.x == 0) {
    double v = 0.;
    for (int w = 0; w < kBalWarps; ++w) v += s_loss[w];
    a.part[blockIdx.x] = v;
    __threadfence();
    s_last = atomicAdd(a.ticket, 1) == (int)gridDim.x - 1;
  }
  __syncthreads();
  if (s_last && warp == 0) {
    // the last CTA adds the parts: 32 strided sums, then their tree, always in the same order
    __threadfence();
    double v = 0.;
    for (int i = lane; i < (int)gridDim.x; i += 32) v += *(volatile double*)(a.part + i);
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(MOE_FULL_MASK, v, o);
    if (lane == 0) *a.loss = (float)(v * ((double)a.coef / max(tv, 1)));
  }
}

constexpr int kBalMaxGrid = 4096;

template <int VPL>
static int launch_balance(const BalArgs& a, bool bf16, bool sig, int grid, int per, cudaStream_t s) {
  const dim3 b(32 * kBalWarps);
  if (bf16) {
    if (sig) balance_kernel<VPL, true, true><<<grid, b, 0, s>>>(a, per);
    else balance_kernel<VPL, true, false><<<grid, b, 0, s>>>(a, per);
  } else {
    if (sig) balance_kernel<VPL, false, true><<<grid, b, 0, s>>>(a, per);
    else balance_kernel<VPL, false, false><<<grid, b, 0, s>>>(a, per);
  }
  MOE_LAUNCH_CHECK();
  return MOE_OK;
}

static size_t bal256(size_t v) { return (v + 255) & ~size_t(255); }

}  // namespace moe

using namespace moe;

extern "C" size_t moe_balance_workspace_bytes(int n_seq) {
  if (n_seq < 1) return 0;
  return 256 + 8 * (size_t)kBalMaxGrid + bal256(4 * (size_t)n_seq);
}

extern "C" int moe_balance_loss(const void* logits, int bf16, const int32_t* ids, const uint8_t* token_mask,
                                const int32_t* seq_start, int n_seq, int T, int E, int k, int rflags, float coef,
                                const float* grad_loss, int32_t* counts, float* loss, void* grad_logits,
                                void* workspace, size_t workspace_bytes, int32_t* dev_status, moe_stream_t stream) {
  if (!logits || !ids || !counts || !workspace || (!loss && !grad_logits)) return MOE_ERR_ARG;
  if (T < 1 || E < 1 || E > kMaxE || k < 1 || k > kMaxK || k > E || n_seq < 1 || (!seq_start && n_seq != 1))
    return MOE_ERR_ARG;
  if ((bf16 != 0 && bf16 != 1) || (rflags & ~MOE_ROUTE_SIGMOID)) return MOE_ERR_ARG;
  if ((uintptr_t)logits % (bf16 ? 2 : 4) || (uintptr_t)grad_logits % (bf16 ? 2 : 4) || (uintptr_t)workspace % 256 ||
      workspace_bytes < moe_balance_workspace_bytes(n_seq))
    return MOE_ERR_ALIGN;
  int dev = 0, sms = 0;
  MOE_CUDA_TRY(cudaGetDevice(&dev));
  MOE_CUDA_TRY(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev));
  char* ws = (char*)workspace;
  BalArgs a{logits, ids, token_mask, seq_start, grad_loss, T, E, k, n_seq, coef, counts,
            (int32_t*)(ws + 256 + 8 * (size_t)kBalMaxGrid), (double*)(ws + 256), (int32_t*)ws, loss, grad_logits,
            dev_status};
  cudaStream_t s = (cudaStream_t)stream;
  balance_count_kernel<<<n_seq, kCntThreads, 0, s>>>(a);
  MOE_LAUNCH_CHECK();
  const int warps = std::min(sms * 4, kBalMaxGrid) * kBalWarps;
  const int per = (T + warps - 1) / warps;
  const int grid = (T + per * kBalWarps - 1) / (per * kBalWarps);
  const bool sig = rflags & MOE_ROUTE_SIGMOID;
  if (E <= 128) return launch_balance<4>(a, bf16, sig, grid, per, s);
  if (E <= 256) return launch_balance<8>(a, bf16, sig, grid, per, s);
  if (E <= 512) return launch_balance<16>(a, bf16, sig, grid, per, s);
  return launch_balance<32>(a, bf16, sig, grid, per, s);
}
