// Group-limited routing from given logits, and the gradient of its weights.
//
// The E experts are n_group groups of E / n_group neighbours.  With s = softmax(l) or sigmoid(l) and c = s + bias (no
// bias: c is ordered as l is), a group's score is the sum of its two best c (or its best one), the topk_group best
// groups stay, and the k best c among their experts are picked; w_j = scale s_j (/ sum_j s_j).  Equal values: the lower
// index first.
//
// The picks are whole numbers, so they are those of 64-bit arithmetic: c is formed in fp32, and where two neighbours in
// the order are closer than the fp32 error bound (and not the same logit with the same bias), the candidates of the token,
// or the best of its groups, are compared again in fp64.  That is some tokens in a thousand.
//
// The bytes of the logits, read once, would bound a large batch (16,384 x 512 fp32: 5.2 us); the instructions of a warp
// for a token, about 1,250, bound it in practice (31.7 us, issued in 61% of the cycles), and the launch a small one (one token 3.1 us).
#include <algorithm>

#include "internal.cuh"

namespace moe {

struct GroupArgs {
  const void* logits;   // [T][E], fp32 or bf16
  const float* bias;    // [E] or NULL
  const uint8_t* mask;  // [T] or NULL
  int T, E, k;
  int n_group, group, topk_group;  // group = E / n_group experts
  int lanes;                       // lanes of a group: a power of two
  int live;                        // lanes that hold experts of the best groups, about
  uint32_t magic;                  // ceil(2^20 / group): e magic / 2^20 is the group of e < 1024
  int flags;
  float scale;
  int32_t* ids;
  float* w;
};

constexpr int kGrpThreads = 256;

// Order of 32-bit floats as unsigned integers: absent 0, NaN 1, -inf, ..., +inf; -0 counts as 0.
__device__ __forceinline__ uint32_t grp_key(float v) {
  const uint32_t b = __float_as_uint(v + 0.f);
  return v != v ? 1u : b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float grp_value(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
}
__device__ __forceinline__ uint64_t grp_key64(double v) {
  const uint64_t b = (uint64_t)__double_as_longlong(v + 0.);
  return v != v ? 1ull : b ^ ((uint64_t)((int64_t)b >> 63) | 0x8000000000000000ull);
}
__device__ __forceinline__ uint64_t grp_max64(uint64_t v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = max(v, __shfl_xor_sync(MOE_FULL_MASK, v, o));
  return v;
}

template <bool BF16>
__device__ __forceinline__ float grp_logit(const void* p, size_t i) {
  return BF16 ? bf16_to_f32(reinterpret_cast<const uint16_t*>(p)[i]) : reinterpret_cast<const float*>(p)[i];
}

// sigmoid(l).  In units of 2^-24 of itself: e is off by 4 (its instruction) and 1.5 |l| (the rounding of its argument),
// which counts e / (1 + e) times, the sum by 1, the reciprocal by 2.
__device__ __forceinline__ float grp_sigmoid(float l) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(l * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
  return r;
}
// How far apart two scores have to be for fp32 to tell their order: rel (|c| + max |bias|) + kGrpTiny.
// Sigmoid, rel = 2^-19 (32 units): two scores are off by 2 (3 + (4 + 1.5 |l|) e / (1 + e)) units of s <= |c| + |bias| and by
// one each from the addition of the bias: below 32 for l > -5.3; further down 3 (|l| - 5.3) units of s < e^l more, at most
// 3.3e-10.  Softmax, rel = 2^-17 (128 units): 2 (4 + |l - max| + 44) + 2, for sums of 37 additions; beyond |l - max| = 15
// the rest is below 1e-14.
constexpr float kGrpTiny = 0x1p-31f;  // 4.7e-10
// Whether fp32 does not tell the order of two scores of these keys (m at most ml).
__device__ __forceinline__ bool grp_close(uint32_t ml, uint32_t m, float rel, float bmax) {
  if (m <= 1u) return false;  // nothing, or a NaN
  const float a = grp_value(ml), b = grp_value(m);
  return !(a - b > rel * (fabsf(a) + bmax) + kGrpTiny) && !(isinf(a) && a == b);
}

// V consecutive logits (16 bytes, or one), as they are.
template <bool BF16, int V>
struct GrpRaw {
  uint32_t r[V == 1 ? 1 : 4];
  __device__ __forceinline__ void load(const void* p, size_t i) {
    if constexpr (V == 1) {
      r[0] = __float_as_uint(grp_logit<BF16>(p, i));
    } else {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(reinterpret_cast<const uint8_t*>(p) + i * (BF16 ? 2 : 4)));
      r[0] = v.x, r[1] = v.y, r[2] = v.z, r[3] = v.w;
    }
  }
  __device__ __forceinline__ float at(int j) const {
    if constexpr (V == 1 || !BF16) return __uint_as_float(r[j]);
    else return j & 1 ? bf16_hi(r[j / 2]) : bf16_lo(r[j / 2]);
  }
};
template <bool BF16, int V>
__device__ __forceinline__ void grp_load(const void* p, size_t i, float* v) {
  GrpRaw<BF16, V> x;
  x.load(p, i);
#pragma unroll
  for (int j = 0; j < V; ++j) v[j] = x.at(j);
}

// sum_e exp(logit - mx) of a token in fp64, by the whole warp.
template <bool BF16>
__device__ __noinline__ double grp_sum64(const GroupArgs& a, size_t row, float mx) {
  double s = 0.;
  for (int e = threadIdx.x & 31; e < a.E; e += 32) s += exp((double)grp_logit<BF16>(a.logits, row + e) - (double)mx);
  for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(MOE_FULL_MASK, s, o);
  return s;
}

// A group's score from its two best.  One of +inf (a bias that pins an expert) is the score, whatever stands beside it.
template <class F>
__device__ __forceinline__ F grp_score(F b1, F b2, bool one) {
  return one || b1 == (F)INFINITY ? b1 : b1 + b2;
}

// One expert's s in fp64.
__device__ __noinline__ double grp_score64(float l, bool sig, float mx, double sum) {
  return sig ? 1. / (1. + exp(-(double)l)) : exp((double)l - (double)mx) / sum;
}

// A warp's exclusive prefix sum of n; `n` becomes the total.
__device__ __forceinline__ int grp_scan(int& n) {
  int at = n;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(MOE_FULL_MASK, at, o);
    if ((threadIdx.x & 31) >= o) at += x;
  }
  at -= n;
  n = __shfl_sync(MOE_FULL_MASK, at + n, 31);
  return at;
}

// The picks of one token in fp64, by the whole warp; lane j returns pick j.  A lane holds every lanes-th expert of
// group lane / lanes, which are at most 64.
template <bool BF16>
__device__ __noinline__ int grp_pick64(const GroupArgs& a, size_t row) {
  const int lane = threadIdx.x & 31, g = lane / a.lanes, i0 = lane % a.lanes;
  const bool sig = a.flags & MOE_ROUTE_SIGMOID;
  constexpr int NE = 64;
  uint64_t key[NE];
  const int held = g < a.n_group ? (a.group - i0 + a.lanes - 1) / a.lanes : 0;
  double mx = -INFINITY, sum = 0.;
  auto at = [&](int u) { return u < held ? g * a.group + u * a.lanes + i0 : -1; };  // the lane's u-th expert, or -1
  if (!sig) {
    for (int u = 0; u < held; ++u)
      if (at(u) >= 0) mx = fmax(mx, (double)grp_logit<BF16>(a.logits, row + at(u)));
    for (int o = 16; o; o >>= 1) mx = fmax(mx, __shfl_xor_sync(MOE_FULL_MASK, mx, o));
    for (int u = 0; u < held; ++u)
      if (at(u) >= 0) sum += exp((double)grp_logit<BF16>(a.logits, row + at(u)) - mx);
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(MOE_FULL_MASK, sum, o);
  }
  const bool best = a.flags & MOE_ROUTE_GROUP_MAX;
  double b1 = -INFINITY, b2 = -INFINITY;
  for (int u = 0; u < held; ++u) {
    const int e = at(u);
    key[u] = 0;
    if (e < 0) continue;
    const double l = (double)grp_logit<BF16>(a.logits, row + e);
    const double s = sig ? 1. / (1. + exp(-l)) : exp(l - mx) / sum;
    const double c = a.bias ? s + (double)a.bias[e] : l, v = a.bias || best ? c : s;
    b2 = fmax(b2, fmin(b1, v == v ? v : -INFINITY));
    b1 = fmax(b1, v);
    key[u] = grp_key64(c);
  }
  if (a.topk_group < a.n_group) {
    for (int o = a.lanes / 2; o; o >>= 1) {
      const double o1 = __shfl_xor_sync(MOE_FULL_MASK, b1, o), o2 = __shfl_xor_sync(MOE_FULL_MASK, b2, o);
      b2 = fmax(fmin(b1, o1), fmax(b2, o2));
      b1 = fmax(b1, o1);
    }
    const uint64_t gk = g < a.n_group ? grp_key64(grp_score(b1, b2, best || a.group == 1)) : 0ull;
    int before = 0;
    for (int h = 0; h < a.n_group; ++h) {
      const uint64_t ok = __shfl_sync(MOE_FULL_MASK, gk, h * a.lanes);
      before += ok > gk || (ok == gk && h < g);
    }
    if (before >= a.topk_group)
      for (int u = 0; u < held; ++u) key[u] = 0;
  }
  int mine = -1;
  for (int j = 0; j < a.k; ++j) {
    uint64_t best = 0;
    for (int u = 0; u < held; ++u) best = max(best, key[u]);
    const uint64_t m = grp_max64(best);
    int e = INT_MAX;
    for (int u = held - 1; u >= 0; --u)
      if (key[u] == m && at(u) >= 0) e = at(u);
    e = __reduce_min_sync(MOE_FULL_MASK, e);
    for (int u = 0; u < held; ++u)
      if (at(u) == e) key[u] = 0;
    if (lane == j) mine = e;
  }
  return mine;
}

// Whether the next logits and the bias of a lane's elements wait in shared memory: with more than 8 (256 bf16 logits: 15.2
// us in registers, 15.6 so; 16,384 x 512: 33.6 and 31.5; 8192 x 1024 77.8 and 74.4).
template <int V, int NE, bool FLAT>
constexpr bool kGrpAhead = !FLAT && V > 1 && NE > 8;
// CTAs of a SM (16,384 x 512, 16 elements a lane, in shared memory: 34 us with two, 31.5 with three, 32.8 with four;
// 8192 x 288, 12 in registers: 34.8 with two, 35.9 with three).
template <int V, int NE, bool FLAT>
constexpr int kGrpResident = NE <= 8 || (kGrpAhead<V, NE, FLAT> && NE <= 16) ? 3 : 2;
// One warp routes a token.  Where the groups fill the lanes, lane (g, i) holds the vectors i, i + lanes, ... of V experts
// of group g, so that a group's score takes log2(lanes) shuffles.  FLAT: the lanes hold the row's vectors in turn, and the
// groups' scores are taken from shared memory.
//
// The k best: k of the lanes' best elements are at or above the k-th largest of them, so only elements at or above it (a
// tolerance below it, with a bias) can be picked.  They are some 12 to 16 as a rule; a lane takes each, and its place is
// the number of those that are larger.  (k maxima one after the other, each over all elements, took twice as long;
// they remain for tokens with more than 32 such elements: many equal logits.)
template <int V, int NQ, bool BF16, bool FLAT>
__global__ void __launch_bounds__(kGrpThreads, kGrpResident<V, NQ * V, FLAT>) group_route_kernel(const GroupArgs a) {
  constexpr int NE = NQ * V;
  constexpr bool kAhead = kGrpAhead<V, NE, FLAT>;
  __shared__ uint4 s_x[kAhead ? kGrpThreads / 32 : 1][kAhead ? NQ : 1][32];  // a lane's next logits
  __shared__ float4 s_b[kAhead ? NE / 4 : 1][32];                             // and the bias of its experts
  __shared__ uint16_t s_e[kGrpThreads / 32][32];
  __shared__ __align__(16) uint32_t s_top[kGrpThreads / 32][32];
  __shared__ float s_c[FLAT ? kGrpThreads / 32 : 1][FLAT ? kMaxE : 1], s_least[FLAT ? kGrpThreads / 32 : 1][32];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane / a.lanes, i0 = lane % a.lanes;
  const bool sig = a.flags & MOE_ROUTE_SIGMOID, raw = a.flags & MOE_ROUTE_RAW, gmax = a.flags & MOE_ROUTE_GROUP_MAX;
  const bool limited = a.topk_group < a.n_group;
  const bool scores = a.bias || (limited && !gmax);  // scores are needed for the choice
  const bool total = !sig && (scores || raw);         // the softmax over all experts is
  const int e0 = FLAT ? lane * V : g * a.group + i0 * V;  // vector q starts at expert e0 + q step
  const int step = FLAT ? 32 * V : a.lanes * V;
  const float kNone = __uint_as_float(0x7fffffffu);  // NaN: at or above nothing
  float bias[kAhead ? 1 : NE], bmax = 0.f;
  auto expert = [&](int u) { return e0 + u / V * step + u % V; };
  auto there = [&](int u) { return !FLAT || expert(u) < a.E; };
  auto group_of = [&](int u) { return FLAT ? (int)((uint32_t)expert(u) * a.magic >> 20) : g; };
  // a token's logits are on their way while the one before is routed (a lane reads what it copied itself)
  GrpRaw<BF16, V> next[kAhead ? 1 : NQ];
  bool valid = true;
  auto fetch = [&](int t) {
#pragma unroll
    for (int q = 0; q < NQ; ++q)
      if constexpr (kAhead) {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(&s_x[warp][q][lane])),
                     "l"(reinterpret_cast<const uint8_t*>(a.logits) + ((size_t)t * a.E + e0 + q * step) * (BF16 ? 2 : 4))
                     : "memory");
      } else {
        if (there(q * V)) next[q].load(a.logits, (size_t)t * a.E + e0 + q * step);
      }
    valid = !a.mask || a.mask[t];
  };
  const int warps = gridDim.x * (kGrpThreads / 32);
  int t = blockIdx.x * (kGrpThreads / 32) + warp;
  if (t < a.T) fetch(t);
  if (a.bias) {
#pragma unroll
    for (int u = 0; u < NE; ++u) {
      const float b = there(u) ? a.bias[expert(u)] : 0.f;
      if constexpr (!kAhead) bias[u] = b;
      else if (warp == 0) reinterpret_cast<float*>(&s_b[u / 4][lane])[u % 4] = b;
      if (fabsf(b) < INFINITY) bmax = fmaxf(bmax, fabsf(b));
    }
    bmax = __uint_as_float(__reduce_max_sync(MOE_FULL_MASK, __float_as_uint(bmax)));
    if constexpr (kAhead) __syncthreads();
  }
  auto bias_of = [&](int u) { return kAhead ? reinterpret_cast<const float*>(&s_b[u / 4][lane])[u % 4] : bias[kAhead ? 0 : u]; };
  for (; t < a.T; t += warps) {
    const size_t row = (size_t)t * a.E;
    float c[NE];  // the logits, then what is compared; kNone for what is not there
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      GrpRaw<BF16, V> x;
      if constexpr (kAhead) {
        if (q == 0) asm volatile("cp.async.wait_all;" ::: "memory");
        const uint4 v = s_x[warp][q][lane];
        x.r[0] = v.x, x.r[1] = v.y, x.r[2] = v.z, x.r[3] = v.w;
      } else {
        x = next[q];
      }
#pragma unroll
      for (int v = 0; v < V; ++v) c[q * V + v] = there(q * V) ? x.at(v) : kNone;
    }
    const bool padding = !valid;
    if (t + warps < a.T) fetch(t + warps);
    if (padding) {
      if (lane < a.k) {
        a.ids[(size_t)t * a.k + lane] = -1;
        a.w[(size_t)t * a.k + lane] = 0.f;
      }
      continue;
    }
    float mx = 0.f, sum = 1.f, inv = 1.f;
    if (total) {
      mx = -INFINITY;
#pragma unroll
      for (int u = 0; u < NE; ++u) mx = fmaxf(mx, c[u]);
#pragma unroll
      for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(MOE_FULL_MASK, mx, o));
      sum = 0.f;
#pragma unroll
      for (int u = 0; u < NE; ++u)
        if (there(u)) sum += expf(c[u] - mx);
#pragma unroll
      for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(MOE_FULL_MASK, sum, o);
      inv = 1.f / sum;
    }
    auto score = [&](float l) { return sig ? grp_sigmoid(l) : expf(l - mx) * inv; };
    if (a.bias) {
#pragma unroll
      for (int u = 0; u < NE; u += 4) {
        float4 b;
        if constexpr (kAhead) b = s_b[u / 4][lane];
        else b = make_float4(bias[u], bias[u + 1], bias[u + 2], bias[u + 3]);
        c[u] = score(c[u]) + b.x;
        c[u + 1] = score(c[u + 1]) + b.y;
        c[u + 2] = score(c[u + 2]) + b.z;
        c[u + 3] = score(c[u + 3]) + b.w;
      }
    }
    // the two best of the lane's part of its group (without a sum of scores: of what is compared)
    float b1 = -INFINITY, b2 = -INFINITY;
    if (limited) {
      auto better = [&](float v) {
        b2 = fmaxf(b2, fminf(b1, v == v ? v : -INFINITY));
        b1 = fmaxf(b1, v);
      };
      const bool compared = a.bias || gmax;
      if constexpr (FLAT) {
#pragma unroll
        for (int u = 0; u < NE; ++u)
          if (there(u)) s_c[warp][expert(u)] = compared ? c[u] : score(c[u]);
        __syncwarp();
        if (g < a.n_group)
          for (int i = i0; i < a.group; i += a.lanes) better(s_c[warp][g * a.group + i]);
        __syncwarp();
      } else {
#pragma unroll
        for (int u = 0; u < NE; ++u) better(compared ? c[u] : score(c[u]));
      }
    }
    const float rel = sig ? 0x1p-19f : 0x1p-17f;
    double sum64 = 0.;
    if (limited) {
      const bool one = gmax || a.group == 1;
      for (int o = a.lanes / 2; o; o >>= 1) {
        const float o1 = __shfl_xor_sync(MOE_FULL_MASK, b1, o), o2 = __shfl_xor_sync(MOE_FULL_MASK, b2, o);
        b2 = fmaxf(fminf(b1, o1), fmaxf(b2, o2));
        b1 = fmaxf(b1, o1);
      }
      const float best = grp_score(b1, b2, one);
      const uint32_t gk = g < a.n_group ? grp_key(best) : 0u;
      int before = 0;
      for (int h = 0; h < a.n_group; ++h) {
        const uint32_t ok = __shfl_sync(MOE_FULL_MASK, gk, h * a.lanes);
        before += ok > gk || (ok == gk && h < g);
      }
      bool in = before < a.topk_group && g < a.n_group;
      if (scores) {
        const float lo = grp_value(__reduce_min_sync(MOE_FULL_MASK, in ? gk : 0xffffffffu));
        const float hi = grp_value(__reduce_max_sync(MOE_FULL_MASK, !in ? gk : 0u));
        if (!(lo - hi > 2.f * (rel * (fabsf(lo) + 2.f * bmax) + kGrpTiny))) {
          // the groups in fp64, of what may be their best (without a bias a softmax's sum does not matter)
          sum64 = !sig && a.bias ? grp_sum64<BF16>(a, row, mx) : 1.;
          const float low = one ? b1 : b2;
          const float least = isinf(low) ? low : low - 2.f * (rel * (fabsf(low) + bmax) + kGrpTiny);
          if constexpr (FLAT) {
            if (i0 == 0) s_least[warp][g] = least;
            __syncwarp();
          }
          auto near = [&](int u) { return (a.bias ? c[u] : score(c[u])) >= (FLAT ? s_least[warp][group_of(u) & 31] : least); };
          int m = 0;
#pragma unroll
          for (int u = 0; u < NE; ++u) m += near(u);
          const int first = grp_scan(m);
          double x1 = -INFINITY, x2 = -INFINITY;
          for (int from = 0; from < m; from += 32) {  // a lane computes one of them
            int i = first - from;
#pragma unroll
            for (int u = 0; u < NE; ++u)
              if (near(u)) {
                if (i >= 0 && i < 32) s_e[warp][i] = (uint16_t)expert(u);
                ++i;
              }
            __syncwarp();
            const int x = from + lane < m ? s_e[warp][lane] : -1;
            double v = 0.;
            if (x >= 0) v = grp_score64(grp_logit<BF16>(a.logits, row + x), sig, mx, sum64) + (a.bias ? (double)a.bias[x] : 0.);
            for (int j = 0; j < min(32, m - from); ++j) {
              const double o = __shfl_sync(MOE_FULL_MASK, v, j);
              if (__shfl_sync(MOE_FULL_MASK, x, j) / a.group == g) {
                x2 = fmax(x2, fmin(x1, o));
                x1 = fmax(x1, o);
              }
            }
            __syncwarp();
          }
          const uint64_t gk64 = g < a.n_group ? grp_key64(grp_score(x1, x2, one)) : 0ull;
          before = 0;
          for (int h = 0; h < a.n_group; ++h) {
            const uint64_t ok = __shfl_sync(MOE_FULL_MASK, gk64, h * a.lanes);
            before += ok > gk64 || (ok == gk64 && h < g);
          }
          in = before < a.topk_group && g < a.n_group;
        }
      }
      if constexpr (FLAT) {
        const unsigned live = __ballot_sync(MOE_FULL_MASK, in);  // (bit h lanes: group h)
#pragma unroll
        for (int u = 0; u < NE; ++u) c[u] = live >> ((group_of(u) * a.lanes) & 31) & 1 ? c[u] : kNone;
      } else {
#pragma unroll
        for (int u = 0; u < NE; ++u) c[u] = in ? c[u] : kNone;
      }
    }
    // the k-th largest of the lanes' best elements, or where lanes are few of the best of each 2 or 4: with k lanes the
    // lowest of their best has more than 32 elements above it too often (8192 x 1024, 8 lanes, k 8: 75 us, so 41; 8192 x
    // 512, 16 lanes, k 16: 82 and 26), with 5 k / 4 it has 12 to 20
    float thr = -INFINITY;
    {
      constexpr int CH = V == 1 ? 1 : NE <= 8 ? 2 : 4, NT = NE / CH;
      float top[NT], best = -INFINITY;
#pragma unroll
      for (int q = 0; q < NT; ++q) {
        top[q] = c[q * CH];
#pragma unroll
        for (int v = 1; v < CH; ++v) top[q] = fmaxf(top[q], c[q * CH + v]);
        best = fmaxf(best, top[q]);
      }
      constexpr uint32_t kLowest = 0x007fffffu;  // -inf
      if (V == 1 || 4 * a.live >= 5 * a.k) {
        uint32_t mine = grp_key(best);
        if (a.k > 4) {  // (4: 20.0 us either way, 2: 17.0 one after the other and 17.5, 10: 33.6 counted and 35)
          s_top[warp][lane] = mine;
          __syncwarp();
          int above = 0;  // lanes at or above this one's
#pragma unroll
          for (int j = 0; j < 32; j += 4) {
            const uint4 o = *reinterpret_cast<const uint4*>(&s_top[warp][j]);
            above += (o.x >= mine) + (o.y >= mine) + (o.z >= mine) + (o.w >= mine);
          }
          __syncwarp();
          const uint32_t m = __reduce_max_sync(MOE_FULL_MASK, above >= a.k ? mine : 0u);
          if (m > kLowest) thr = grp_value(m);
        } else {
          for (int seen = 0; seen < a.k;) {
            const uint32_t m = __reduce_max_sync(MOE_FULL_MASK, mine);
            if (m <= kLowest) break;
            seen += __popc(__ballot_sync(MOE_FULL_MASK, mine == m));
            if (seen >= a.k) thr = grp_value(m);
            if (mine == m) mine = 0;
          }
        }
      } else {
        for (int seen = 0; seen < a.k;) {
          const uint32_t m = __reduce_max_sync(MOE_FULL_MASK, grp_key(best));
          if (m <= kLowest) break;
          const float f = grp_value(m);
          int here = 0;
          best = -INFINITY;
#pragma unroll
          for (int q = 0; q < NT; ++q) {
            here += top[q] == f;
            if (top[q] == f) top[q] = -INFINITY;
            best = fmaxf(best, top[q]);
          }
          seen += __reduce_add_sync(MOE_FULL_MASK, here);
          if (seen >= a.k) thr = f;
        }
      }
    }
    if (a.bias && fabsf(thr) < INFINITY) thr -= rel * (fabsf(thr) + bmax) + kGrpTiny;
    int n = 0;
#pragma unroll
    for (int u = 0; u < NE; ++u) n += c[u] >= thr;
    int at = grp_scan(n);
    int place = lane, e = -1;  // of the expert that this lane has, if place < k
    float z = -INFINITY;
    bool exact = n < a.k;  // NaN among the picks
    if (n <= 32 && !exact) {
#pragma unroll
      for (int u = 0; u < NE; ++u)
        if (c[u] >= thr) s_e[warp][at++] = (uint16_t)expert(u);
      __syncwarp();
      const bool on = lane < n;
      float bb = 0.f;
      uint32_t mine = 0u;
      if (on) {
        e = s_e[warp][lane];
        z = grp_logit<BF16>(a.logits, row + e);
        if (a.bias) bb = a.bias[e];
        mine = grp_key(a.bias ? score(z) + bb : z);
      }
      __syncwarp();
      uint32_t above = 0xffffffffu;  // the next larger one
      int same = 0;
      place = 0;
#pragma unroll 4
      for (int j = 0; j < n; ++j) {
        const uint32_t o = __shfl_sync(MOE_FULL_MASK, mine, j);
        place += o > mine;
        same += o == mine;
        if (o > mine) above = min(above, o);
      }
      const bool close = a.bias && on && place >= 1 && above != 0xffffffffu && grp_close(above, mine, rel, bmax);
      bool unsure = close && place <= a.k;
      if (__any_sync(MOE_FULL_MASK, on && same > 1)) {
        int larger = 0;  // than the next larger one: with several of that, one may have a place though this one has none
        for (int j = 0; j < n; ++j) {
          const uint32_t o = __shfl_sync(MOE_FULL_MASK, mine, j);
          larger += o > above;
          const int oe = __shfl_sync(MOE_FULL_MASK, e, j);
          const float oz = __shfl_sync(MOE_FULL_MASK, z, j), ob = __shfl_sync(MOE_FULL_MASK, bb, j);
          if (on && o == mine) {
            place += oe < e;
            // equal scores of other logits are equal in fp32 alone (but for infinities)
            unsure |= a.bias && fabsf(grp_value(mine)) < INFINITY && (oz != z || ob != bb);
          }
        }
        unsure |= close && larger < a.k;
      }
      if (!on) place = 32;
      if (__any_sync(MOE_FULL_MASK, unsure)) {
        if (!sig && sum64 == 0.) sum64 = grp_sum64<BF16>(a, row, mx);
        const double s = grp_score64(z, sig, mx, sum64);
        const uint64_t x = on ? grp_key64(s + (double)bb) : 0ull;
        place = on ? 0 : 32;
        for (int j = 0; j < n; ++j) {
          const uint64_t o = __shfl_sync(MOE_FULL_MASK, x, j);
          const int oe = __shfl_sync(MOE_FULL_MASK, e, j);
          place += o > x || (o == x && oe < e);
        }
      }
    } else if (!exact) {
      // one after the other: many are equal
      int last = -1;
      uint32_t ml = 0;
      for (int j = 0; j < a.k && !exact; ++j) {
        float best = -INFINITY;
#pragma unroll
        for (int u = 0; u < NE; ++u) best = fmaxf(best, c[u]);
        const uint32_t m = __reduce_max_sync(MOE_FULL_MASK, grp_key(best));
        const float f = grp_value(m);
        int x = INT_MAX;
#pragma unroll
        for (int u = NE - 1; u >= 0; --u)
          if (c[u] == f) x = expert(u);
        x = __reduce_min_sync(MOE_FULL_MASK, x);
#pragma unroll
        for (int u = 0; u < NE; ++u)
          if (expert(u) == x) c[u] = kNone;
        if (a.bias) {
          if (j > 0 && grp_close(ml, m, rel, bmax))
            exact = grp_logit<BF16>(a.logits, row + x) != grp_logit<BF16>(a.logits, row + last) || a.bias[x] != a.bias[last];
          ml = m;
          last = x;
        }
        if (lane == j) e = x;
      }
      if (a.bias && !exact) {
        // the last pick and what is left
        const float ll = grp_logit<BF16>(a.logits, row + last), lb = a.bias[last], fl = grp_value(ml);
        float next = -INFINITY;
#pragma unroll
        for (int u = 0; u < NE; ++u) {
          if (c[u] == fl) exact |= fabsf(fl) < INFINITY && (grp_logit<BF16>(a.logits, row + expert(u)) != ll || bias_of(u) != lb);
          else next = fmaxf(next, c[u]);
        }
        const uint32_t m = __reduce_max_sync(MOE_FULL_MASK, grp_key(next));
        exact = __any_sync(MOE_FULL_MASK, exact) || grp_close(ml, m, rel, bmax);
      }
      if (lane < a.k && !exact) z = grp_logit<BF16>(a.logits, row + e);
    }
    if (exact) {
      place = lane;
      e = grp_pick64<BF16>(a, row);
      if (lane < a.k) z = grp_logit<BF16>(a.logits, row + e);
    }
    // weights, over the lanes with a place
    const bool on = place < a.k;
    float w = 0.f;
    if (raw) {
      if (on) w = sig ? 1.f / (1.f + expf(-z)) : expf(z - mx) / sum;
    } else {
      const uint32_t m = __reduce_max_sync(MOE_FULL_MASK, on ? grp_key(z) : 0u);
      const float top = m > 0x007fffffu ? grp_value(m) : 0.f;  // (0 in the place of -inf)
      if (on) {
        // sigmoid(z) / exp(min(top, 0)): a row of large negative logits keeps its proportions
        w = sig ? expf(fminf(z, 0.f) - fminf(top, 0.f)) / (1.f + expf(-fabsf(z))) : expf(z - top);
      }
      float all = w;
#pragma unroll
      for (int o = 16; o; o >>= 1) all += __shfl_xor_sync(MOE_FULL_MASK, all, o);
      w = all == 0.f ? 0.f : w / all;  // picks of -inf alone have no weight
    }
    if (on) {
      a.ids[(size_t)t * a.k + place] = e;
      a.w[(size_t)t * a.k + place] = w * a.scale;
    }
  }
}

struct GroupGradArgs {
  const void* logits;
  const int32_t* ids;
  const float* gw;  // [T][k]
  int T, E, k, flags;
  float scale;
  void* grad;
  int32_t* status;
};

template <bool BF16>
__device__ __forceinline__ void grp_put(void* p, size_t i, float v) {
  if (BF16) reinterpret_cast<uint16_t*>(p)[i] = f32_to_bf16(v);
  else reinterpret_cast<float*>(p)[i] = v;
}

// The gradient of a token's weights, L lanes (at least its picks) a token.  With W = sum_i g_i w_i / scale over its picks:
//   renormalised      w_j (g_j - W)   [sigmoid: (1 - s_j)]         in the picks alone
//   not, sigmoid      scale g_j s_j (1 - s_j)                      in the picks alone
//   not, softmax      s_e (scale G_e - sum_i scale g_i s_i)        everywhere (DENSE); G_e: the g of the picks of e
// The row is written in whole vectors first (NC a lane) and the picks' values over it by the same warp.  A pick that is
// there twice adds up, in the order of the picks.  30,011 x 288 bf16, every logit: 12.8 us where the bytes take 5.5; the
// chain ids -> logits -> sums -> row is what a CTA waits for, and three rounds of CTAs follow each other (a warp a token
// and the row read three times took 23).
template <int V, int NC, int L, bool BF16, bool DENSE>
__global__ void __launch_bounds__(kGrpThreads) group_grad_kernel(const GroupGradArgs a) {
  pdl_wait();
  pdl_trigger();
  constexpr float kNone = -INFINITY;
  const int lane = threadIdx.x & 31, gl = lane % L, lead = lane - gl;
  const bool sig = a.flags & MOE_ROUTE_SIGMOID, raw = a.flags & MOE_ROUTE_RAW;
  const int t = (int)((blockIdx.x * (unsigned)kGrpThreads + threadIdx.x) / L);
  const bool in = t < a.T;
  const size_t row = (size_t)t * a.E;
  auto total = [](float v) {
#pragma unroll
    for (int o = L / 2; o; o >>= 1) v += __shfl_xor_sync(MOE_FULL_MASK, v, o);
    return v;
  };
  GrpRaw<BF16, V> x[DENSE ? NC : 1];
  if (DENSE) {
#pragma unroll
    for (int c = 0; c < NC; ++c)
      if (in && (c * L + gl) * V < a.E) x[c].load(a.logits, row + (c * L + gl) * V);
  }
  int e = -1;
  if (in && gl < a.k) {
    e = a.ids[(size_t)t * a.k + gl];
    if (e < -1 || e >= a.E) set_status(a.status, MOE_DEV_BAD_EXPERT);
    if (e >= a.E) e = -1;
  }
  const bool on = e >= 0;
  const float gj = on ? a.gw[(size_t)t * a.k + gl] * a.scale : 0.f;
  const unsigned group = L == 32 ? MOE_FULL_MASK : ((1u << (L & 31)) - 1u) << lead;
  const bool any = (__ballot_sync(MOE_FULL_MASK, on) & group) != 0;
  const float z = on ? grp_logit<BF16>(a.logits, row + e) : kNone;
  float p = 0.f, jac = 1.f, dot = 0.f;  // the pick's share of the sum that its weight is over
  float q[DENSE ? NC * V : 1], inv = 0.f, mx = z;
  if (DENSE) {
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        q[c * V + j] = any && (c * L + gl) * V < a.E ? x[c].at(j) : kNone;
        mx = fmaxf(mx, q[c * V + j]);
      }
  }
  if (DENSE || !raw) {
#pragma unroll
    for (int o = L / 2; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(MOE_FULL_MASK, mx, o));
    if (mx == -INFINITY) mx = 0.f;
  }
  float sum = 0.f;
  if (DENSE) {
#pragma unroll
    for (int u = 0; u < NC * V; ++u) sum += q[u] = expf(q[u] - mx);
  }
  if (on) {
    const float em = expf(-fabsf(z));
    if (sig) jac = (z >= 0.f ? em : 1.f) / (1.f + em);
    if (sig && raw) p = (z >= 0.f ? 1.f : em) / (1.f + em);
    else p = sig ? expf(fminf(z, 0.f) - fminf(mx, 0.f)) / (1.f + em) : expf(z - mx);
  }
  if (DENSE || !raw) {
    sum = total(DENSE ? sum : p);
    inv = sum == 0.f ? 0.f : 1.f / sum;
    p *= inv;
    dot = total(on ? p * gj : 0.f);
  }
  // the row without its picks
  if (in) {
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int i = (c * L + gl) * V;
      if (i >= a.E) break;
      float v[V];
#pragma unroll
      for (int j = 0; j < V; ++j) v[j] = DENSE && any ? q[c * V + j] * inv * -dot : 0.f;
      if constexpr (V == 1) {
        grp_put<BF16>(a.grad, row + i, v[0]);
      } else {
        uint32_t o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (BF16) {
            const __nv_bfloat162 w = __floats2bfloat162_rn(v[(2 * j) % V], v[(2 * j + 1) % V]);
            o[j] = *reinterpret_cast<const uint32_t*>(&w);
          } else {
            o[j] = __float_as_uint(v[j]);
          }
        }
        *reinterpret_cast<uint4*>(reinterpret_cast<uint8_t*>(a.grad) + (row + i) * (BF16 ? 2 : 4)) =
            make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
  }
  __syncwarp();
  // the picks: the first lane of a repeated one adds all of them
  const unsigned same = __match_any_sync(MOE_FULL_MASK, on ? e : -1 - lane) & group;
  float v = DENSE ? gj : raw ? p * gj * jac : p * (gj - dot) * jac;
  if (__any_sync(MOE_FULL_MASK, on && (same & (same - 1)))) {
    float all = 0.f;
    for (int j = 0; j < a.k; ++j) {
      const float o = __shfl_sync(MOE_FULL_MASK, v, lead + j);
      if (same >> (lead + j) & 1) all += o;
    }
    v = all;
  }
  if (DENSE) v = p * (v - dot);
  if (on && (same & lanemask_lt()) == 0) grp_put<BF16>(a.grad, row + e, v);
}

template <int V, int NC, int L, bool BF16>
static int launch_group_grad(const GroupGradArgs& a, cudaStream_t s) {
  constexpr int per = kGrpThreads / L;
  const dim3 grid((a.T + per - 1) / per), block(kGrpThreads);
  if ((a.flags & MOE_ROUTE_RAW) && !(a.flags & MOE_ROUTE_SIGMOID))
    MOE_CUDA_TRY(launch_pdl(group_grad_kernel<V, NC, L, BF16, true>, grid, block, 0, s, a));
  else
    MOE_CUDA_TRY(launch_pdl(group_grad_kernel<V, NC, L, BF16, false>, grid, block, 0, s, a));
  return MOE_OK;
}

static int grp_sms(int* sms) {
  static int seen[64] = {};
  int dev = 0;
  MOE_CUDA_TRY(cudaGetDevice(&dev));
  if (dev < 0 || dev >= 64) return MOE_ERR_CUDA;
  if (seen[dev] == 0) MOE_CUDA_TRY(cudaDeviceGetAttribute(&seen[dev], cudaDevAttrMultiProcessorCount, dev));
  *sms = seen[dev];
  return MOE_OK;
}

template <int V, int NQ, bool BF16, bool FLAT>
static int launch_groups_as(GroupArgs a, int sms, cudaStream_t s) {
  a.live = std::min(32, a.topk_group * (FLAT ? std::max(a.group / V, 1) : a.lanes));
  // as many CTAs as are resident: a warp keeps the bias and has the next token's logits on their way
  constexpr int W = kGrpThreads / 32;
  const dim3 grid(std::min((a.T + W - 1) / W, sms * kGrpResident<V, NQ * V, FLAT>)), block(kGrpThreads);
  MOE_CUDA_TRY(launch_pdl(group_route_kernel<V, NQ, BF16, FLAT>, grid, block, 0, s, a));
  return MOE_OK;
}

template <int V, int NQ, bool BF16>
static int launch_groups(const GroupArgs& a, int sms, cudaStream_t s) {
  if (V > 1 && a.lanes * a.n_group == 32 && a.group == a.lanes * NQ * V)
    return launch_groups_as<V, NQ, BF16, (V == 1)>(a, sms, s);
  return launch_groups_as<V, NQ, BF16, true>(a, sms, s);
}

}  // namespace moe

using namespace moe;

extern "C" int moe_route_groups(const void* logits, int bf16, const float* sel_bias, const uint8_t* token_mask, int T,
                                int E, int k, int n_group, int topk_group, int rflags, float scale, int32_t* ids,
                                float* w, moe_stream_t stream) {
  if (!logits || !ids || !w || (bf16 != 0 && bf16 != 1)) return MOE_ERR_ARG;
  if (T < 1 || T > (1 << 26) || E < 1 || E > kMaxE || n_group < 1 || n_group > 32 || E % n_group || topk_group < 1 ||
      topk_group > n_group || k < 1 || k > kMaxK || k > topk_group * (E / n_group))
    return MOE_ERR_ARG;
  if (rflags & ~(MOE_ROUTE_SIGMOID | MOE_ROUTE_RAW | MOE_ROUTE_GROUP_MAX)) return MOE_ERR_ARG;
  if ((uintptr_t)logits % (bf16 ? 2 : 4)) return MOE_ERR_ALIGN;
  int sms = 0;
  if (int rc = grp_sms(&sms)) return rc;
  int lanes = 32;
  while (lanes * n_group > 32) lanes /= 2;
  const int group = E / n_group;
  const int v = bf16 ? 8 : 4;
  const GroupArgs a{logits, sel_bias, token_mask, T, E, k, n_group, group, topk_group, lanes, 0,
                    (uint32_t)(((1 << 20) + group - 1) / group), rflags, scale, ids, w};
  cudaStream_t s = (cudaStream_t)stream;
  // 16-byte vectors where every row starts on one
  const int each = (E + 31) / 32, vecs = (E / v + 31) / 32;  // of a lane
  if (E % v == 0 && (uintptr_t)logits % 16 == 0) {
    if (bf16) {
      if (vecs <= 1) return launch_groups<8, 1, true>(a, sms, s);
      if (vecs <= 2) return launch_groups<8, 2, true>(a, sms, s);
      return launch_groups<8, 4, true>(a, sms, s);
    }
    if (vecs <= 1) return launch_groups<4, 1, false>(a, sms, s);
    if (vecs <= 2) return launch_groups<4, 2, false>(a, sms, s);
    if (vecs <= 4) return launch_groups<4, 4, false>(a, sms, s);
    return launch_groups<4, 8, false>(a, sms, s);
  }
  if (bf16) {
    if (each <= 4) return launch_groups<1, 4, true>(a, sms, s);
    if (each <= 16) return launch_groups<1, 16, true>(a, sms, s);
    return launch_groups<1, 32, true>(a, sms, s);
  }
  if (each <= 4) return launch_groups<1, 4, false>(a, sms, s);
  if (each <= 16) return launch_groups<1, 16, false>(a, sms, s);
  return launch_groups<1, 32, false>(a, sms, s);
}

extern "C" int moe_route_groups_grad(const void* logits, int bf16, const int32_t* ids, const float* grad_w, int T, int E,
                                     int k, int rflags, float scale, void* grad_logits, int32_t* dev_status,
                                     moe_stream_t stream) {
  if (!logits || !ids || !grad_w || !grad_logits || (bf16 != 0 && bf16 != 1)) return MOE_ERR_ARG;
  if (T < 1 || T > (1 << 26) || E < 1 || E > kMaxE || k < 1 || k > kMaxK) return MOE_ERR_ARG;
  if (rflags & ~(MOE_ROUTE_SIGMOID | MOE_ROUTE_RAW)) return MOE_ERR_ARG;
  if ((uintptr_t)logits % (bf16 ? 2 : 4) || (uintptr_t)grad_logits % (bf16 ? 2 : 4)) return MOE_ERR_ALIGN;
  const GroupGradArgs a{logits, ids, grad_w, T, E, k, rflags, scale, grad_logits, dev_status};
  const int v = bf16 ? 8 : 4;
  const bool vec = E % v == 0 && (uintptr_t)logits % 16 == 0 && (uintptr_t)grad_logits % 16 == 0;
  cudaStream_t s = (cudaStream_t)stream;
  const int chunks = E / v;
  if (!vec) {
    if (bf16) {
      if (E <= 128) return launch_group_grad<1, 4, 32, true>(a, s);
      if (E <= 384) return launch_group_grad<1, 12, 32, true>(a, s);
      return launch_group_grad<1, 32, 32, true>(a, s);
    }
    if (E <= 128) return launch_group_grad<1, 4, 32, false>(a, s);
    if (E <= 384) return launch_group_grad<1, 12, 32, false>(a, s);
    return launch_group_grad<1, 32, 32, false>(a, s);
  }
  if (bf16) {
    if (chunks <= 16) return launch_group_grad<8, 1, 16, true>(a, s);
    if (chunks <= 32) return launch_group_grad<8, 2, 16, true>(a, s);
    if (chunks <= 48) return launch_group_grad<8, 3, 16, true>(a, s);
    if (chunks <= 64) return launch_group_grad<8, 2, 32, true>(a, s);
    return launch_group_grad<8, 4, 32, true>(a, s);
  }
  if (chunks <= 32) return launch_group_grad<4, 2, 16, false>(a, s);
  if (chunks <= 64) return launch_group_grad<4, 2, 32, false>(a, s);
  if (chunks <= 96) return launch_group_grad<4, 3, 32, false>(a, s);
  if (chunks <= 128) return launch_group_grad<4, 4, 32, false>(a, s);
  return launch_group_grad<4, 8, 32, false>(a, s);
}
