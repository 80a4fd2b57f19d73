// Products with 4-bit weights and group scales (format: w4.cuh) for few rows: the linear layer and the
// grouped SwiGLU expert FFN as weight streams.
//
//   y[t][n] = sum_k x[t][k] (code[k][n] - 8) scale[k / G][n]
//
// The codes become the A operand of 16 x 16 x 8 MMAs as the exact bf16 integers code - 8, the bf16 activations
// the B operand; a 64-input block's products (32 inputs where G = 32) are summed in fp32 by the tensor core,
// multiplied by their fp32 scale and added in fp32.  No weight and no activation is rounded.
// (16 + code needs one operation less for every pair of codes, but its surplus, 24 times the block's sum of
// activations, has to come off again: an input far above the rest then costs accuracy in columns where its weight
// is 0, infinities become NaN, and sums overflow early.  The extra MMAs for the surplus cost as much as they save:
// us, with it / as it is, 8 tokens through the experts 46.6 / 45.4, 32 tokens 101.7 / 99.3, head 28.8 / 29.1.)
//
// A warp streams CM neighbouring tiles of 16 columns (CM x 512 bytes a block of 64 inputs, one 16-byte load
// per lane and tile), every ks-th block of the inputs, two blocks ahead and on across the end of a unit, so
// that its loads do not pause; the activations of a block travel with its codes.  (A ring in shared memory, filled
// by bulk copies or by cp.async, took 8 tokens 58 and 59 us when registers took 51; 45 since the shares are finer and
// the products exact.)  The ks warps that share a unit add up in shared memory, in warp order.  ks is the split that
// costs least for the unit count at hand (w4_split): few long shares while there are units for every warp, short ones
// for a few small matrices.
#include <algorithm>

#include "internal.cuh"
#include "w4.cuh"

namespace moe {

constexpr int kW4Warps = 8;
constexpr int kW4Threads = 32 * kW4Warps;
constexpr int kW4Ctas = 2;   // resident CTAs per SM that the registers allow
constexpr int kW4Slots = 512;  // routing slots that the stream kernels group themselves; more are grouped before them
// Rows of an expert, on average, from which the tensor-core path takes over: a stream pays for every eight rows of an
// expert, a large tile hardly for any of its 256.  us, streams / tensor cores: 8 experts, 12 rows each 25.0 / 32.3, 24
// rows 39.3 / 34.1, 48 rows 64.8 / 34.2; 32 experts, 8 rows 29.0 / 37.3, 12 rows 35.7 / 36.2, 16 rows 41.5 / 36.6; 128
// experts, 6 rows 120 / 156, 8 rows 142 / 157, 10 rows 172 / 159; 288 experts, 8 rows 233 / 238, 10 rows 274 / 240.
// The average counts all experts and the figures are for even loads: how many rows the experts in use have is known on
// the device alone.
constexpr int kGemmRows = 10;

// One block of 64 inputs in registers: a lane's codes of CM tiles, their columns' scales, and the lane's inputs
// of NB groups of eight rows (LO: as the sum of two bf16).
template <int CM, int NB, bool LO, bool G32>
struct W4Block {
  uint4 w[CM];
  uint32_t s[G32 ? 2 : 1][CM];
  uint4 x[NB][LO ? 2 : 1][2];
};

// What a warp streams of one unit: its tiles' codes and scales, and the rows they meet.
template <int NB>
struct W4Unit {
  const uint8_t* codes;   // the lane's chunk in block 0 of the first tile
  const uint8_t* scales;  // the lane's columns in group 0
  int mates;              // tiles that lie between one block and the next
  int nm;                 // tiles that exist (0: nothing to do)
  const uint16_t* x[NB];  // the lane's row of each group, at input 8 (lane & 3)
};
template <int NB>
__device__ __forceinline__ void w4_at(W4Unit<NB>& u, const uint8_t* m, const W4Dims& d, int tile, int nm, int lane) {
  u.codes = m + w4_code_at(d, tile, 0) * 512 + 16 * w4_chunk(lane >> 2, lane & 3);
  u.scales = m + d.scales + w4_scale_at(d, tile, 0, lane >> 2) * 4;
  u.mates = w4_mates(d, tile);
  u.nm = nm;
}

template <int CM, int NB, bool LO, bool G32>
__device__ __forceinline__ void w4_load_codes(W4Block<CM, NB, LO, G32>& b, const W4Unit<NB>& u, const W4Dims& d, int kb) {
  const uint8_t* c = u.codes + (size_t)(uint32_t)(kb * u.mates) * 512;
  const int kg = G32 ? 2 * kb : d.G == 128 ? kb >> 1 : kb;
  const uint8_t* s = u.scales + (uint32_t)(kg * u.mates) * 32u;
  if (u.nm == CM && (CM == 1 || u.mates == 8)) {  // (units start on a multiple of CM: a lane's scales are one load)
#pragma unroll
    for (int m = 0; m < CM; ++m) b.w[m] = ldg_stream(c + m * 512);
#pragma unroll
    for (int p = 0; p < (G32 ? 2 : 1); ++p) {
      const uint8_t* sp = s + p * u.mates * 32;
      if constexpr (CM == 4) {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(sp));
        b.s[p][0] = v.x, b.s[p][1] = v.y, b.s[p][2] = v.z, b.s[p][3] = v.w;
      } else if constexpr (CM == 2) {
        const uint2 v = __ldg(reinterpret_cast<const uint2*>(sp));
        b.s[p][0] = v.x, b.s[p][1] = v.y;
      } else {
        b.s[p][0] = __ldg(reinterpret_cast<const uint32_t*>(sp));
      }
    }
    return;
  }
#pragma unroll
  for (int m = 0; m < CM; ++m) {  // the last tiles; those that do not exist repeat the last one
    const int mm = min(m, u.nm - 1);
    b.w[m] = ldg_stream(c + mm * 512);
#pragma unroll
    for (int p = 0; p < (G32 ? 2 : 1); ++p)
      b.s[p][m] = __ldg(reinterpret_cast<const uint32_t*>(s + p * u.mates * 32) + mm);
  }
}

// Rows written by the kernel before (LO) are read by plain loads after the wait, x through the read-only path.
template <int CM, int NB, bool LO, bool G32>
__device__ __forceinline__ void w4_load_rows(W4Block<CM, NB, LO, G32>& b, const W4Unit<NB>& u, const W4Dims& d, int kb, int q,
                                             size_t lo) {
  if (kb * 64 + 64 <= d.K) {
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int p = 0; p < (LO ? 2 : 1); ++p) {
        const uint4* at = reinterpret_cast<const uint4*>(u.x[nb] + p * lo + kb * 64);
#pragma unroll
        for (int h = 0; h < 2; ++h) b.x[nb][p][h] = LO ? at[4 * h] : __ldg(at + 4 * h);
      }
    return;
  }
#pragma unroll
  for (int nb = 0; nb < NB; ++nb)
#pragma unroll
    for (int p = 0; p < (LO ? 2 : 1); ++p) {
      const uint16_t* x = u.x[nb] + p * lo + kb * 64;
#pragma unroll
      for (int h = 0; h < 2; ++h) {  // K % 8 == 0: a lane's eight inputs are inside or outside together
        const uint4* at = reinterpret_cast<const uint4*>(x + 32 * h);
        b.x[nb][p][h] = kb * 64 + 32 * h + 8 * q < d.K ? (LO ? *at : __ldg(at)) : make_uint4(0, 0, 0, 0);
      }
    }
}

template <int CM, int NB, bool LO, bool G32>
__device__ __forceinline__ void w4_load(W4Block<CM, NB, LO, G32>& b, const W4Unit<NB>& u, const W4Dims& d, int kb, int q,
                                        size_t lo) {
  w4_load_codes<CM, NB, LO, G32>(b, u, d, kb);
  w4_load_rows<CM, NB, LO, G32>(b, u, d, kb, q, lo);
}

template <int CM, int NB, bool LO, bool G32>
__device__ __forceinline__ void w4_block(const W4Block<CM, NB, LO, G32>& b, float (&acc)[CM][NB][4]) {
  constexpr int P = LO ? 2 : 1;
#pragma unroll
  for (int part = 0; part < (G32 ? 2 : 1); ++part) {
    constexpr int H = G32 ? 1 : 2;  // halves of the block per scale
#pragma unroll
    for (int m = 0; m < CM; ++m) {
      float c[NB][4];
#pragma unroll
      for (int h = 0; h < H; ++h) {
        uint32_t a0[4], a1[4];
        w4_frag_bf16(part + h ? b.w[m].y : b.w[m].x, part + h ? b.w[m].w : b.w[m].z, a0, a1);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int p = 0; p < P; ++p) {
            const uint4 v = b.x[nb][p][part + h];
            if (h == 0 && p == 0) mma_bf16_16816(c[nb], a0, v.x, v.y, 0.f, 0.f, 0.f, 0.f);
            else mma_bf16_16816(c[nb], a0, v.x, v.y, c[nb][0], c[nb][1], c[nb][2], c[nb][3]);
            mma_bf16_16816(c[nb], a1, v.z, v.w, c[nb][0], c[nb][1], c[nb][2], c[nb][3]);
          }
      }
      const uint32_t sw = b.s[part][m];
      const float2 s = __half22float2(*reinterpret_cast<const __half2*>(&sw));
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        acc[m][nb][0] = fmaf(s.x, c[nb][0], acc[m][nb][0]);
        acc[m][nb][1] = fmaf(s.x, c[nb][1], acc[m][nb][1]);
        acc[m][nb][2] = fmaf(s.y, c[nb][2], acc[m][nb][2]);
        acc[m][nb][3] = fmaf(s.y, c[nb][3], acc[m][nb][3]);
      }
    }
  }
}

// Sums of the ks warps of a subgroup, in warp order: red[warp][m][nb][4][32].  Element (i, lane) is column
// (lane >> 2) + 8 * (i >> 1), row 2 * (lane & 3) + (i & 1).
template <int CM, int NB>
__device__ __forceinline__ void w4_put_part(float* red, int warp, int lane, const float (&acc)[CM][NB][4]) {
#pragma unroll
  for (int m = 0; m < CM; ++m)
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int i = 0; i < 4; ++i) red[(((warp * CM + m) * NB + nb) * 4 + i) * 32 + lane] = acc[m][nb][i];
}
template <int CM, int NB>
__device__ __forceinline__ float w4_sum_part(const float* red, int w0, int ks, int m, int row, int col) {
  const int nb = row >> 3, i = 2 * (col >> 3) + (row & 1), lane = 4 * (col & 7) + ((row & 7) >> 1);
  float s = 0.f;
  for (int w = 0; w < ks; ++w) s += red[((((w0 + w) * CM + m) * NB + nb) * 4 + i) * 32 + lane];
  return s;
}

// Whether a row has neither infinities nor NaN (those have given the formula's result already); by a whole warp.
__device__ __noinline__ bool w4_finite(const uint16_t* x, int K) {
  const uint4* at = reinterpret_cast<const uint4*>(x);
  uint32_t bad = 0;
#pragma unroll 4
  for (int k = threadIdx.x & 31; k < K / 8; k += 32) {
    const uint4 v = at[k];
    for (uint32_t u : {v.x, v.y, v.z, v.w}) bad |= __vcmpeq2(u & 0x7f807f80u, 0x7f807f80u);
  }
  return !__any_sync(MOE_FULL_MASK, bad);
}

// One result in 64 bits, for a sum of finite inputs that left fp32's range on its way: inputs above some 2^100.
// Reached by such results alone, and in a pass of its own after a kernel's stream (called from the stream's rounds it
// took registers from them: 32 tokens 98.3 / 101.5 us), so in no hurry.  codes: the packed column's words in its tile's
// block 0 (g: its place among the tile's first or second eight), sc: its scale of group 0, mates: w4_mates.
template <bool LO>
__device__ __noinline__ float w4_dot_at(const uint32_t* codes, const __half* sc, int mates, int g, float mult, int K, int G,
                                        const uint16_t* x, size_t lo) {
  double sum = 0.;
  for (int k = 0; k < K; k += 8) {
    const int b = k >> 5, q = (k >> 3) & 3;
    const uint32_t v = codes[(size_t)(b >> 1) * mates * 128 + w4_chunk(g, q) * 4 + (b & 1)];
    const double s = __half2float(sc[(size_t)(k / G) * mates * 16]);
    for (int j = 0; j < 8; ++j) {
      double xv = bf16_to_f32(x[k + j]);
      if (LO) xv += bf16_to_f32(x[lo + k + j]);
      sum += xv * (((int)(__funnelshift_r(v, v, w4_code_bit(j)) & 15) - 8) * s);
    }
  }
  return (float)(sum * mult);
}
// Of packed column n of the matrix at w, for the inputs at x (LO: as the sum with those at x + lo).
template <bool LO>
__device__ __forceinline__ float w4_dot(const uint8_t* w, const W4Dims& d, int n, const uint16_t* x, size_t lo) {
  const int tile = n >> 4, g = n & 7, h = (n >> 3) & 1;
  return w4_dot_at<LO>(reinterpret_cast<const uint32_t*>(w) + w4_code_at(d, tile, 0) * 128 + 2 * h,
                       reinterpret_cast<const __half*>(w + d.scales) + w4_scale_at(d, tile, 0, g) * 2 + h, w4_mates(d, tile), g,
                       reinterpret_cast<const float*>(w + d.mult)[n], d.K, d.G, x, lo);
}

// Warps per unit: the power of two with the least rounds x (blocks of a share + the cost of ending a round, about
// one block: with 3 in its place 8 tokens took 51 us, with 1 46; 32 tokens over 288 experts 108 and 101; now 44.5 and 99).
__host__ __device__ inline int w4_split(int units, int Kb, int ctas) {
  int best = 1;
  int64_t least = 0;
  for (int ks = 1; ks <= kW4Warps; ks *= 2) {
    const int64_t sub = (int64_t)ctas * (kW4Warps / ks), rounds = (units + sub - 1) / sub;
    const int64_t cost = rounds * ((Kb + ks - 1) / ks + 1);
    if (ks == 1 || cost < least) {
      best = ks;
      least = cost;
    }
  }
  return best;
}

// The stream of one CTA: rounds 0 .. rounds - 1 of units; unit(round) gives this warp's unit (of its subgroup)
// and done(round, red) is called by all threads once the subgroups' parts of a round are in red.  The first
// blocks' codes are loaded before a programmatic dependent's wait, the rows after it.
template <int CM, int NB, bool LO, bool G32, class Unit, class Done>
__device__ __forceinline__ void w4_stream(const W4Dims& d, int ks, int rounds, size_t lo, float* red, Unit&& unit,
                                          Done&& done) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, q = lane & 3, part = warp % ks;
  const int steps = ((d.Kb + ks - 1) / ks + 1) / 2;  // of two blocks
  W4Block<CM, NB, LO, G32> ring[2];
  W4Unit<NB> cur, nxt = unit(0);
#pragma unroll
  for (int j = 0; j < 2; ++j)
    if (nxt.nm > 0 && part + j * ks < d.Kb) w4_load_codes<CM, NB, LO, G32>(ring[j], nxt, d, part + j * ks);
  pdl_wait();
#pragma unroll
  for (int j = 0; j < 2; ++j)
    if (nxt.nm > 0 && part + j * ks < d.Kb) w4_load_rows<CM, NB, LO, G32>(ring[j], nxt, d, part + j * ks, q, lo);
  for (int r = 0; r < rounds; ++r) {
    cur = nxt;
    if (r + 1 < rounds) nxt = unit(r + 1);
    else nxt.nm = 0;
    float acc[CM][NB][4] = {};
    int kb = part;
    for (int s = 0; s + 1 < steps; ++s, kb += 2 * ks)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        if (cur.nm > 0) w4_block<CM, NB, LO, G32>(ring[j], acc);  // all but a share's last two blocks exist
        const int kn = kb + (2 + j) * ks;
        if (cur.nm > 0 && kn < d.Kb) w4_load<CM, NB, LO, G32>(ring[j], cur, d, kn, q, lo);
      }
#pragma unroll
    for (int j = 0; j < 2; ++j) {  // the slots' next blocks are the next unit's
      if (cur.nm > 0 && kb + j * ks < d.Kb) w4_block<CM, NB, LO, G32>(ring[j], acc);
      if (nxt.nm > 0 && part + j * ks < d.Kb) w4_load<CM, NB, LO, G32>(ring[j], nxt, d, part + j * ks, q, lo);
    }
    float* buf = red + (r & 1) * (kW4Warps * CM * NB * 128);  // two buffers: one barrier per round
    w4_put_part<CM, NB>(buf, warp, lane, acc);
    __syncthreads();
    done(r, buf);
  }
}

struct W4LinArgs {
  const uint16_t* x;
  size_t ldx, ldo;
  int T, ks;  // ks warps share CM tiles
  const uint8_t* w;
  W4Dims d;
  void* out;
  int out_f32;
};

// grid (CTAs, ceil(T / (8 NB))).
template <int CM, int NB, bool G32>
__global__ void __launch_bounds__(kW4Threads, kW4Ctas) w4_linear_kernel(const W4LinArgs a) {
  __shared__ float red[2 * kW4Warps * CM * NB * 128];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int ks = a.ks, sub = kW4Warps / ks;  // subgroups of the CTA
  const int groups = (a.d.Mt + CM - 1) / CM;
  const int rounds = (groups - (int)blockIdx.x * sub + (int)gridDim.x * sub - 1) / ((int)gridDim.x * sub);
  const int t0 = blockIdx.y * 8 * NB, nt = min(8 * NB, a.T - t0);
  const float* mult = reinterpret_cast<const float*>(a.w + a.d.mult);
  __shared__ bool fin[8 * NB];  // rows without infinities and NaN; only where a result was lost
  auto first = [&](int r, int g) { return ((r * (int)gridDim.x + (int)blockIdx.x) * sub + g) * CM; };  // tile
  auto unit = [&](int r) {
    W4Unit<NB> u;
    const int tile = first(r, warp / ks);
    w4_at(u, a.w, a.d, min(tile, a.d.Mt - 1), max(0, min(CM, a.d.Mt - tile)), lane);
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)  // rows past the batch repeat its last one; their results are dropped
      u.x[nb] = a.x + (size_t)(t0 + min(8 * nb + (lane >> 2), nt - 1)) * a.ldx + 8 * (lane & 3);
    return u;
  };
  if (rounds <= 0) return;
  bool lost = false;  // a result of this thread is not finite
  auto put = [&](int r, const float* buf, bool again) {
    for (int i = threadIdx.x; i < sub * CM * 16 * nt; i += kW4Threads) {
      const int col = i % (CM * 16), row = i / (CM * 16) % nt, g = i / (CM * 16 * nt);
      const int n = first(r, g) * 16 + col;
      if (n >= a.d.N) continue;
      const size_t o = (size_t)(t0 + row) * a.ldo + n;
      float v;
      if (again) {
        if (!fin[row]) continue;
        if (isfinite(a.out_f32 ? reinterpret_cast<float*>(a.out)[o] : bf16_to_f32(reinterpret_cast<uint16_t*>(a.out)[o]))) continue;
        v = w4_dot<false>(a.w, a.d, n, a.x + (size_t)(t0 + row) * a.ldx, 0);
      } else {
        v = w4_sum_part<CM, NB>(buf, g * ks, ks, col >> 4, row, col & 15) * mult[n];
        lost |= !isfinite(v);
      }
      if (a.out_f32) reinterpret_cast<float*>(a.out)[o] = v;
      else reinterpret_cast<uint16_t*>(a.out)[o] = f32_to_bf16(v);
    }
  };
  w4_stream<CM, NB, false, G32>(a.d, ks, rounds, 0, red, unit, [&](int r, const float* buf) { put(r, buf, false); });
  if (!__syncthreads_or(lost)) return;
  for (int row = warp; row < nt; row += kW4Warps) {
    const bool f = w4_finite(a.x + (size_t)(t0 + row) * a.ldx, a.d.K);
    if (lane == 0) fin[row] = f;
  }
  __syncthreads();
  if (lost)
    for (int r = 0; r < rounds; ++r) put(r, nullptr, true);
}

struct W4FfnArgs {
  FfnArgs f;              // f.pool: bytes of the 4-bit slot pool
  W4Slab sl;
  uint16_t* h;            // bf16 [2][n][I]: h = h[0] + h[1]
  int n;                  // routing slots
  // Routed form: the groups come from the ids (row = flat routing slot), the combine follows in w4_sum_kernel.
  const int32_t* ids;     // [n], or NULL: f.offset / f.rows / f.list_e / f.n_list (row = grouped position)
  const int32_t* sum_ids; // [n] where the combine follows: the ids, whichever form the groups come in
  const int32_t* pos;     // [n] row of y of every slot, where the groups are given and the combine follows
  int cap;                // row batches that there can be
  const float* w;         // [n]
  uint16_t* out;          // bf16 [T][H]
};

// At most eight rows of one expert.
constexpr int kW4Rows = 8;
struct W4Batch {
  int slot, n;            // slot -1: no slot
  uint16_t row[kW4Rows];  // rows of h and y
};


// The row batches of the listed experts, or of the ids, by ascending expert, in shared memory: `tab` holds
// cap entries, `cnt` (2 kMaxE + n ints, free afterwards) is scratch.  Built by all threads; returns their number.
// Every CTA builds the same batches, though the order of the rows inside one may vary: no row's result depends
// on its neighbours.
__device__ __forceinline__ int w4_batches(const W4FfnArgs& g, W4Batch* tab, int* cnt, int* tmp) {
  const FfnArgs& a = g.f;
  const int n = g.n;
  if (g.ids) {
    int *first = cnt + kMaxE, *ids = cnt + 2 * kMaxE;  // an expert's first batch; the ids
    for (int e = threadIdx.x; e < a.E; e += kW4Threads) cnt[e] = 0;
    __syncthreads();
    constexpr int U = kW4Slots / kW4Threads;  // routing slots per thread
    int id[U], rank[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = threadIdx.x + u * kW4Threads;
      id[u] = i < n ? g.ids[i] : -1;
      if (i < n && (id[u] < 0 || id[u] >= a.E)) {
        set_status(a.status, MOE_DEV_BAD_EXPERT);
        id[u] = -1;
      }
      if (i < n) ids[i] = id[u];
      rank[u] = id[u] >= 0 ? atomicAdd(&cnt[id[u]], 1) : 0;
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (id[u] >= 0 && cnt[id[u]] > kW4Rows) {  // several batches: the row's place is its place among the ids
        rank[u] = 0;
        for (int j = 0; j < (int)threadIdx.x + u * kW4Threads; ++j) rank[u] += ids[j] == id[u];
      }
    int base = 0;
    for (int e0 = 0; e0 < a.E; e0 += kW4Threads) {
      const int e = e0 + threadIdx.x, rows = e < a.E ? cnt[e] : 0, c = (rows + kW4Rows - 1) / kW4Rows;
      int tot;
      const int b = base + block_exclusive_scan(c, tmp, &tot);
      if (c > 0) {
        int slot = a.e2s ? a.e2s[e] : e;
        if (slot < 0 || slot >= a.S) {
          set_status(a.status, MOE_DEV_BAD_SLOT);
          slot = -1;
        }
        first[e] = b;
        for (int i = 0; i < c; ++i) {
          tab[b + i].slot = slot;
          tab[b + i].n = min(kW4Rows, rows - kW4Rows * i);
        }
      }
      base += tot;
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (id[u] >= 0)
        tab[first[id[u]] + rank[u] / kW4Rows].row[rank[u] % kW4Rows] = (uint16_t)(threadIdx.x + u * kW4Threads);
    __syncthreads();
    return base;
  }
  const int nl = min(*a.n_list, kMaxE);
  int base = 0;
  for (int l0 = 0; l0 < nl; l0 += kW4Threads) {
    const int li = l0 + threadIdx.x;
    int c = 0, p0 = 0, rows = 0, slot = -1;
    if (li < nl) {
      const int e = a.list_e[li];
      if (e >= 0 && e < a.E) {
        slot = a.list_s ? a.list_s[li] : a.e2s ? a.e2s[e] : e;
        p0 = a.offset[e];
        rows = min(max(a.offset[e + 1] - p0, 0), n);
        c = (rows + kW4Rows - 1) / kW4Rows;
        if (slot < 0 || slot >= a.S) {
          if (c > 0) set_status(a.status, MOE_DEV_BAD_SLOT);
          slot = -1;
        }
      }
    }
    int tot;
    const int ex = base + block_exclusive_scan(c, tmp, &tot);
    for (int i = 0; i < c && ex + i < g.cap; ++i) {
      W4Batch& b = tab[ex + i];
      b.slot = slot;
      b.n = min(kW4Rows, rows - kW4Rows * i);
      for (int j = 0; j < b.n; ++j) b.row[j] = (uint16_t)(p0 + kW4Rows * i + j);
    }
    base += tot;
  }
  __syncthreads();
  if (base > g.cap && threadIdx.x == 0) set_status(a.status, MOE_DEV_BAD_GROUPS);
  return min(base, g.cap);
}

// Gate and up: unit = (row batch, two tiles of gate with their neighbours of up); an expert's batches follow
// each other, so that their weights come from memory once.
constexpr int kGuTiles = 4;  // (I % 32 == 0 and H % 64 == 0: both matrices have whole units)
template <bool G32>
__global__ void __launch_bounds__(kW4Threads, kW4Ctas) w4_gateup_kernel(const W4FfnArgs a) {
  extern __shared__ W4Batch tab[];
  __shared__ float red[2 * kW4Warps * kGuTiles * 128];
  __shared__ int tmp[33];
  pdl_trigger();  // the down kernel may start: it waits for this one before it reads h
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const W4Dims& d = a.sl.gu;
  const int nbat = w4_batches(a, tab, reinterpret_cast<int*>(red), tmp);
  const int FT = (d.Mt + kGuTiles - 1) / kGuTiles, I = d.N / 2, units = nbat * FT;
  const int ks = w4_split(units, d.Kb, gridDim.x), sub = kW4Warps / ks;
  const int rounds = (units - (int)blockIdx.x * sub + (int)gridDim.x * sub - 1) / ((int)gridDim.x * sub);
  if (rounds <= 0) return;
  auto index = [&](int r, int g) { return (r * (int)gridDim.x + (int)blockIdx.x) * sub + g; };
  auto slab = [&](int slot) { return reinterpret_cast<const uint8_t*>(a.f.pool) + (size_t)slot * a.sl.bytes; };
  auto unit = [&](int r) {
    W4Unit<1> u;
    u.nm = 0;
    const int i = index(r, warp / ks);
    if (i >= units) return u;
    const W4Batch& b = tab[i / FT];
    if (b.slot < 0) return u;
    const int tile = i % FT * kGuTiles;
    w4_at(u, slab(b.slot), d, tile, min(kGuTiles, d.Mt - tile), lane);
    const int row = b.row[min(lane >> 2, b.n - 1)];  // rows past the batch repeat its last one
    u.x[0] = a.f.x + (size_t)((a.ids ? row : a.f.rows[row]) / a.f.k) * a.f.H + 8 * (lane & 3);
    return u;
  };
  bool lost = false;  // a gate or up value, or h, of this thread is not finite (h is not wherever one of the others is not)
  auto put = [&](int r, const float* buf, bool again) {
    for (int i = threadIdx.x; i < sub * 32 * kW4Rows; i += kW4Threads) {
      const int col = i & 31, row = (i >> 5) % kW4Rows, g = (i >> 5) / kW4Rows, u = index(r, g);
      if (u >= units) continue;
      const W4Batch& b = tab[u / FT];
      const int tile = u % FT * kGuTiles, m = 2 * (col >> 4), f = tile / 2 * 16 + col;
      if (b.slot < 0 || row >= b.n || tile + m >= d.Mt) continue;
      const float* mg = reinterpret_cast<const float*>(slab(b.slot) + d.mult) + (tile + m) * 16 + (col & 15);
      const size_t o = (size_t)b.row[row] * I + f;
      float gv, uv;
      if (again) {
        // (a warp has 32 columns of one row, and gets here as a whole)
        const bool bad = !isfinite(bf16_to_f32(a.h[o]));
        const uint16_t* x = a.f.x + (size_t)((a.ids ? b.row[row] : a.f.rows[b.row[row]]) / a.f.k) * a.f.H;
        if (!__any_sync(MOE_FULL_MASK, bad) || !w4_finite(x, d.K) || !bad) continue;
        const int n = (tile + m) * 16 + (col & 15);
        gv = w4_dot<false>(slab(b.slot), d, n, x, 0);
        uv = w4_dot<false>(slab(b.slot), d, n + 16, x, 0);
      } else {
        gv = w4_sum_part<kGuTiles, 1>(buf, g * ks, ks, m, row, col & 15) * mg[0];
        uv = w4_sum_part<kGuTiles, 1>(buf, g * ks, ks, m + 1, row, col & 15) * mg[16];
      }
      const float h = gv / (1.f + __expf(-gv)) * uv;
      // h as the sum of two bf16: 16 significant bits reach the down product
      const uint16_t hi = f32_to_bf16(h);
      const bool fin = isfinite(bf16_to_f32(hi));
      lost |= !fin;
      a.h[o] = hi;
      a.h[(size_t)a.n * I + o] = fin ? f32_to_bf16(h - bf16_to_f32(hi)) : 0;
    }
  };
  w4_stream<kGuTiles, 1, false, G32>(d, ks, rounds, 0, red, unit, [&](int r, const float* buf) { put(r, buf, false); });
  if (__any_sync(MOE_FULL_MASK, lost))
    for (int r = 0; r < rounds; ++r) put(r, nullptr, true);
}

// out[t] = bf16(sum_j w[t][j] y[slot]), fp32, j ascending: grid (T, H / 512).  (Sums by the CTAs of the down kernel
// that finish last save this launch, which overlaps, and cost as much: one token 16.6 us with them and 16.1
// without when that was measured, 8 tokens 45.4 and 46.0; 15.7 and 44.5 now.)
__global__ void __launch_bounds__(128) w4_sum_kernel(const W4FfnArgs a) {
  pdl_wait();
  const int H = a.f.H, k = a.f.k, t = blockIdx.x, c = (blockIdx.y * 128 + threadIdx.x) * 4;
  if (c >= H) return;
  float4 y[kMaxK], s = make_float4(0.f, 0.f, 0.f, 0.f);
  float w[kMaxK];
  int e[kMaxK];
#pragma unroll
  for (int j = 0; j < kMaxK; ++j) {
    e[j] = j < k ? a.sum_ids[t * k + j] : -1;
    w[j] = j < k ? a.w[t * k + j] : 0.f;
  }
#pragma unroll
  for (int j = 0; j < kMaxK; ++j) {
    y[j] = make_float4(0.f, 0.f, 0.f, 0.f);
    const bool expert = e[j] >= 0 && e[j] < a.f.E;  // others have no row
    if (expert) y[j] = *reinterpret_cast<const float4*>(a.f.y + (size_t)(a.pos ? a.pos[t * k + j] : t * k + j) * H + c);
    e[j] = !expert ? -1 : a.f.e2s ? a.f.e2s[e[j]] : e[j];  // its slot
  }
#pragma unroll
  for (int j = 0; j < kMaxK; ++j)  // an expert without a slot has a row of zeros; its weight may be anything
    if (e[j] < 0 || e[j] >= a.f.S) w[j] = 0.f;
#pragma unroll
  for (int j = 0; j < kMaxK; ++j) {
    s.x = fmaf(w[j], y[j].x, s.x), s.y = fmaf(w[j], y[j].y, s.y);
    s.z = fmaf(w[j], y[j].z, s.z), s.w = fmaf(w[j], y[j].w, s.w);
  }
  *reinterpret_cast<uint2*>(a.out + (size_t)t * H + c) =
      make_uint2(uint32_t(f32_to_bf16(s.x)) | uint32_t(f32_to_bf16(s.y)) << 16,
                 uint32_t(f32_to_bf16(s.z)) | uint32_t(f32_to_bf16(s.w)) << 16);
}

// Down: unit = (row batch, four tiles of 16 output columns).
constexpr int kDnTiles = 4;
template <bool G32>
__global__ void __launch_bounds__(kW4Threads, kW4Ctas) w4_down_kernel(const W4FfnArgs a) {
  extern __shared__ W4Batch tab[];
  __shared__ float red[2 * kW4Warps * kDnTiles * 128];
  __shared__ int tmp[33];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const W4Dims& d = a.sl.dn;
  const int nbat = w4_batches(a, tab, reinterpret_cast<int*>(red), tmp);
  const int FT = (d.Mt + kDnTiles - 1) / kDnTiles, units = nbat * FT;
  const int ks = w4_split(units, d.Kb, gridDim.x), sub = kW4Warps / ks;
  const int rounds = (units - (int)blockIdx.x * sub + (int)gridDim.x * sub - 1) / ((int)gridDim.x * sub);
  if (rounds <= 0) {
    pdl_wait();
    return;
  }
  auto index = [&](int r, int g) { return (r * (int)gridDim.x + (int)blockIdx.x) * sub + g; };
  auto down = [&](int slot) {
    return reinterpret_cast<const uint8_t*>(a.f.pool) + (size_t)slot * a.sl.bytes + a.sl.dn_at;
  };
  auto unit = [&](int r) {
    W4Unit<1> u;
    u.nm = 0;
    const int i = index(r, warp / ks);
    if (i >= units) return u;
    const W4Batch& b = tab[i / FT];
    if (b.slot < 0) return u;
    const int tile = i % FT * kDnTiles;
    w4_at(u, down(b.slot), d, tile, min(kDnTiles, d.Mt - tile), lane);
    u.x[0] = a.h + (size_t)b.row[min(lane >> 2, b.n - 1)] * d.K + 8 * (lane & 3);
    return u;
  };
  bool lost = false;  // a result of this thread is not finite
  auto put = [&](int r, const float* buf, bool again) {
    for (int i = threadIdx.x; i < sub * 16 * kDnTiles * kW4Rows; i += kW4Threads) {
      const int col = i % (16 * kDnTiles), row = i / (16 * kDnTiles) % kW4Rows, g = i / (16 * kDnTiles * kW4Rows);
      const int u = index(r, g);
      if (u >= units) continue;
      const W4Batch& b = tab[u / FT];
      const int n = u % FT * (16 * kDnTiles) + col;
      if (row >= b.n || n >= d.N) continue;
      // an expert without a slot adds nothing: its rows are zero
      float* y = a.f.y + (size_t)b.row[row] * d.N + n;
      float v = 0.f;
      if (again) {
        // (a warp has 32 columns of one row, and gets here as a whole)
        const bool bad = !isfinite(*y);
        const uint16_t* h = a.h + (size_t)b.row[row] * d.K;
        if (!__any_sync(MOE_FULL_MASK, bad) || !w4_finite(h, d.K) || !bad) continue;
        v = w4_dot<true>(down(b.slot), d, n, h, (size_t)a.n * d.K);
      } else if (b.slot >= 0) {
        v = w4_sum_part<kDnTiles, 1>(buf, g * ks, ks, col >> 4, row, col & 15) *
            reinterpret_cast<const float*>(down(b.slot) + d.mult)[n];
        lost |= !isfinite(v);
      }
      *y = v;
    }
  };
  w4_stream<kDnTiles, 1, true, G32>(d, ks, rounds, (size_t)a.n * d.K, red, unit,
                                    [&](int r, const float* buf) { put(r, buf, false); });
  if (__any_sync(MOE_FULL_MASK, lost))
    for (int r = 0; r < rounds; ++r) put(r, nullptr, true);
}

static int w4_sms(int* sms) {
  int dev = 0;
  MOE_CUDA_TRY(cudaGetDevice(&dev));
  MOE_CUDA_TRY(cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev));
  return MOE_OK;
}

static bool w4_gemm_ffn(int n, int E) { return n > 128 && n >= kGemmRows * E; }

size_t w4_ws_bytes(int n, int H, int I) {
  const size_t h = ((size_t)n * I * 4 + 255) & ~size_t(255);
  return w4_gemm_ffn(n, 0) ? std::max(h, w4_ffn_gemm_ws(n, H, I, false)) : h;  // (enough for any number of experts)
}

// The two weight streams; the second one's CTAs start as the first one's leave.
static int launch_ffn_w4_stream(W4FfnArgs a, int group, int sms, cudaStream_t stream, Prof* prof) {
  static bool d0[64] = {}, d1[64] = {}, d2[64] = {}, d3[64] = {};
  a.cap = std::min(a.n, a.f.E + a.n / kW4Rows);  // a batch that is not full is an expert's last
  const size_t smem = (size_t)a.cap * sizeof(W4Batch);
  constexpr int most = (kMaxE + kMaxE * kGemmRows / kW4Rows) * (int)sizeof(W4Batch);
  if (group == 32) {
    MOE_CUDA_TRY(ensure_smem(w4_gateup_kernel<true>, most, d0));
    MOE_CUDA_TRY(ensure_smem(w4_down_kernel<true>, most, d1));
  } else {
    MOE_CUDA_TRY(ensure_smem(w4_gateup_kernel<false>, most, d2));
    MOE_CUDA_TRY(ensure_smem(w4_down_kernel<false>, most, d3));
  }
  const dim3 grid(sms * kW4Ctas), block(kW4Threads);
  if (prof) prof->begin(MOE_PROF_FFN_GATEUP, stream);
  if (group == 32) w4_gateup_kernel<true><<<grid, block, smem, stream>>>(a);
  else w4_gateup_kernel<false><<<grid, block, smem, stream>>>(a);
  MOE_LAUNCH_CHECK();
  if (prof) prof->end(stream);
  if (prof) prof->begin(MOE_PROF_FFN_DOWN, stream);
  MOE_CUDA_TRY(launch_pdl(group == 32 ? w4_down_kernel<true> : w4_down_kernel<false>, grid, block, smem, stream, a));
  if (prof) prof->end(stream);
  if (a.out)
    MOE_CUDA_TRY(launch_pdl(w4_sum_kernel, dim3(a.f.T, (a.f.H + 511) / 512), dim3(128), 0, stream, a));
  return MOE_OK;
}

// y rows of the listed experts; ws holds h (w4_ws_bytes).
int launch_ffn_w4(const FfnArgs& f, int group, void* ws, size_t ws_bytes, int max_list, cudaStream_t stream,
                  Prof* prof) {
  const int n = f.T * f.k;
  if (ws_bytes < w4_ws_bytes(n, f.H, f.I)) return MOE_ERR_ALIGN;
  if (max_list <= 0) return MOE_OK;
  if (w4_gemm_ffn(n, f.E)) return launch_ffn_w4_gemm(f, nullptr, nullptr, group, ws, nullptr, nullptr, stream, prof);
  int sms = 0;
  const int r = w4_sms(&sms);
  if (r != MOE_OK) return r;
  W4FfnArgs a{};
  a.f = f, a.sl = w4_slab(f.H, f.I, group), a.h = (uint16_t*)ws, a.n = n;
  return launch_ffn_w4_stream(a, group, sms, stream, prof);
}

static size_t al256(size_t v) { return (v + 255) & ~size_t(255); }

// Workspace of moe_experts_w4: the groups of the permute, then y and the FFN's own.
struct W4ExpWs {
  int32_t *count, *offset, *rows, *pos, *act_e, *n_act, *perm;
  float* y;
  void* ffn;
  size_t ffn_bytes, bytes;
};
static W4ExpWs w4_exp_ws(void* base, int T, int H, int I, int k, int E) {
  const int n = T * k;
  W4ExpWs w{};
  char* b = (char*)base;
  size_t off = 0;
  auto take = [&](size_t bytes) -> void* {
    char* p = b ? b + off : nullptr;
    off += al256(bytes);
    return p;
  };
  w.count = (int32_t*)take(4 * (size_t)E);
  w.offset = (int32_t*)take(4 * (size_t)(E + 1));
  w.rows = (int32_t*)take(4 * (size_t)n);
  w.pos = (int32_t*)take(4 * (size_t)n);
  w.act_e = (int32_t*)take(4 * (size_t)E);
  w.n_act = (int32_t*)take(4);
  w.perm = (int32_t*)take(moe_permute_scratch_bytes(n, E) + 4);
  const bool gemm = w4_gemm_ffn(n, E);  // its y is fp16 inside its own workspace
  w.y = gemm ? nullptr : (float*)take(4 * (size_t)n * H);
  w.ffn_bytes = gemm ? w4_ffn_gemm_ws(n, H, I, true) : 4 * (size_t)n * I;
  w.ffn = take(w.ffn_bytes);
  w.bytes = off;
  return w;
}

// Streams take a pass over the weights per 32 rows, about 0.4 us for 10^6 of them; the tensor-core path costs 8 us
// and more (rows, launches, the pipeline's start) and then little.  us, streams / tensor cores: 17 rows, 4096 x 4096
// 8.8 / 12.0, x 16384 25.5 / 19.0; 33 rows, 4096 x 4096 16.0 / 12.5, 1024 x 8192 11.2 / 10.5; 128 rows, 2048 x 2048
// 12.4 / 11.7, 1024 x 1024 5.5 / 10.6; 512 rows, 1024 x 1024 16.2 / 12.7, 512 x 512 7.6 / 11.3.
static bool w4_gemm_linear(int T, int K, int N) {
  const double work = (double)((T + 31) / 32) * K * N;
  return T > 16 && work >= (T > 32 ? 1 << 24 : 1 << 25);
}

// Routing slots and hidden sizes whose products the kernels index with 32 bits.
static bool w4_rows_ok(int T, int k) { return (int64_t)T * k <= (1 << 24); }

}  // namespace moe

using namespace moe;

extern "C" size_t moe_w4_linear_workspace_bytes(int T, int K, int N, int group) {
  if (T < 1 || !w4_shape_ok(K, N, group)) return 0;
  return w4_gemm_linear(T, K, N) ? w4_linear_gemm_ws(T, w4_dims(K, N, group)) : 0;
}

extern "C" int moe_w4_linear(const void* x, long long ldx, int T, int K, int N, int group, const void* w, void* out,
                             long long ldo, int out_f32, void* workspace, size_t workspace_bytes,
                             int32_t* dev_status, moe_stream_t stream) {
  if (!x || !w || !out || T < 1 || T > (1 << 24) || !w4_shape_ok(K, N, group) || ldx < K || ldo < N)
    return MOE_ERR_ARG;
  if (out_f32 != 0 && out_f32 != 1) return MOE_ERR_ARG;
  if ((uintptr_t)x % 16 || ldx % 8 || (uintptr_t)w % 16 || (uintptr_t)out % (out_f32 ? 4 : 2)) return MOE_ERR_ALIGN;
  if (workspace_bytes < moe_w4_linear_workspace_bytes(T, K, N, group) || (uintptr_t)workspace % 256)
    return MOE_ERR_ALIGN;
  if (w4_gemm_linear(T, K, N))
    return launch_w4_linear_gemm((const uint16_t*)x, (size_t)ldx, T, (const uint8_t*)w, w4_dims(K, N, group), out,
                                 (size_t)ldo, out_f32, workspace, dev_status, (cudaStream_t)stream);
  int sms = 0;
  const int r = w4_sms(&sms);
  if (r != MOE_OK) return r;
  W4LinArgs a{(const uint16_t*)x, (size_t)ldx, (size_t)ldo, T, 1, (const uint8_t*)w, w4_dims(K, N, group), out, out_f32};
  // rows of a pass, and tiles of a warp: four where that leaves a unit for every other warp, as many rows need
  // the registers for their sums
  const int rows = T <= 8 ? 8 : T <= 16 ? 16 : 32, ctas = sms * kW4Ctas;
  const int cm = rows == 32 ? 1 : rows == 16 ? 2 : a.d.Mt >= 8 * ctas ? 4 : a.d.Mt >= ctas ? 2 : 1;
  const int groups = (a.d.Mt + cm - 1) / cm;
  a.ks = w4_split(groups, a.d.Kb, ctas);
  const int gx = std::min((groups + kW4Warps / a.ks - 1) / (kW4Warps / a.ks), ctas);
  const bool g32 = group == 32;
  for (int t0 = 0; t0 < T; t0 += 65535 * rows) {  // the grid's y
    W4LinArgs b = a;
    b.x += (size_t)t0 * ldx;
    b.out = (char*)out + (size_t)t0 * ldo * (out_f32 ? 4 : 2);
    b.T = std::min(T - t0, 65535 * rows);
    const dim3 grid(gx, (b.T + rows - 1) / rows);
    auto go = [&](auto kernel, auto kernel32) { (g32 ? kernel32 : kernel)<<<grid, kW4Threads, 0, (cudaStream_t)stream>>>(b); };
    if (rows == 32) go(w4_linear_kernel<1, 4, false>, w4_linear_kernel<1, 4, true>);
    else if (rows == 16) go(w4_linear_kernel<2, 2, false>, w4_linear_kernel<2, 2, true>);
    else if (cm == 4) go(w4_linear_kernel<4, 1, false>, w4_linear_kernel<4, 1, true>);
    else if (cm == 2) go(w4_linear_kernel<2, 1, false>, w4_linear_kernel<2, 1, true>);
    else go(w4_linear_kernel<1, 1, false>, w4_linear_kernel<1, 1, true>);
    MOE_LAUNCH_CHECK();
  }
  return MOE_OK;
}

extern "C" size_t moe_ffn_w4_workspace_bytes(int T, int H, int k, int I) {
  if (T < 1 || H < 1 || k < 1 || I < 1 || !w4_rows_ok(T, k)) return 0;
  return w4_ws_bytes(T * k, H, I);
}

extern "C" int moe_expert_ffn_w4(const void* x, int T, int H, int I, int k, int E, int group, const int32_t* offset,
                                 const int32_t* rows, const int32_t* list_e, const int32_t* n_list, int max_list,
                                 const void* pool, int S, const int32_t* e2s, float* y, void* workspace,
                                 size_t workspace_bytes, int32_t* dev_status, moe_stream_t stream) {
  if (!x || !offset || !rows || !list_e || !n_list || !pool || !y || !workspace) return MOE_ERR_ARG;
  if (!shape_ok(T, H, I, k, E) || !w4_slab_ok(H, I, group) || !w4_rows_ok(T, k) || max_list < 0 || S < 1 ||
      (!e2s && S < E))
    return MOE_ERR_ARG;
  if ((uintptr_t)pool % 16 || (uintptr_t)y % 16 || (uintptr_t)workspace % 256 || (uintptr_t)x % 16)
    return MOE_ERR_ALIGN;
  FfnArgs f{};
  f.x = (const uint16_t*)x;
  f.T = T, f.H = H, f.I = I, f.k = k, f.E = E;
  f.offset = offset, f.rows = rows, f.list_e = list_e, f.n_list = n_list;
  f.pool = (const uint16_t*)pool, f.e2s = e2s, f.S = S, f.pool_only = 1;
  f.y = y, f.status = dev_status;
  return launch_ffn_w4(f, group, workspace, workspace_bytes, std::min(max_list, E), (cudaStream_t)stream, nullptr);
}

extern "C" size_t moe_experts_w4_workspace_bytes(int T, int H, int I, int k, int E) {
  if (!shape_ok(T, H, I, k, E) || !w4_rows_ok(T, k)) return 0;
  // fewer tokens may need more: the streams' y is fp32
  const int most = std::min((std::max(kGemmRows * E, 129) - 1) / k, T);
  return std::max(w4_exp_ws(nullptr, T, H, I, k, E).bytes, most > 0 ? w4_exp_ws(nullptr, most, H, I, k, E).bytes : 0);
}

extern "C" int moe_experts_w4(const void* x, const int32_t* ids, const float* w, int T, int H, int I, int k, int E,
                              int group, const void* pool, int S, const int32_t* e2s, void* out, void* workspace,
                              size_t workspace_bytes, int32_t* dev_status, moe_stream_t stream) {
  if (!x || !ids || !w || !pool || !out || !workspace) return MOE_ERR_ARG;
  if (!shape_ok(T, H, I, k, E) || !w4_slab_ok(H, I, group) || !w4_rows_ok(T, k) || S < 1 || (!e2s && S < E))
    return MOE_ERR_ARG;
  if ((uintptr_t)pool % 16 || (uintptr_t)out % 8 || (uintptr_t)workspace % 256 || (uintptr_t)x % 16)
    return MOE_ERR_ALIGN;
  const int n = T * k;
  const W4ExpWs ws = w4_exp_ws(workspace, T, H, I, k, E);
  if (workspace_bytes < ws.bytes) return MOE_ERR_ALIGN;
  cudaStream_t s = (cudaStream_t)stream;
  FfnArgs f{};
  f.x = (const uint16_t*)x;
  f.T = T, f.H = H, f.I = I, f.k = k, f.E = E;
  f.pool = (const uint16_t*)pool, f.e2s = e2s, f.S = S, f.pool_only = 1;
  f.y = ws.y, f.status = dev_status;
  const bool gemm = w4_gemm_ffn(n, E);
  int sms = 0, r = w4_sms(&sms);
  if (r != MOE_OK) return r;
  W4FfnArgs a{};
  a.f = f, a.sl = w4_slab(H, I, group), a.h = (uint16_t*)ws.ffn, a.n = n;
  a.w = w, a.sum_ids = ids, a.out = (uint16_t*)out;
  if (!gemm && n <= kW4Slots) {
    a.ids = ids;
    return launch_ffn_w4_stream(a, group, sms, s, nullptr);
  }
  r = launch_permute(ids, n, E, ws.count, ws.offset, ws.rows, ws.pos, ws.act_e, ws.n_act, dev_status, ws.perm, s);
  if (r != MOE_OK) return r;
  f.offset = ws.offset, f.rows = ws.rows, f.list_e = ws.act_e, f.n_list = ws.n_act;
  if (!gemm) {
    a.f = f, a.pos = ws.pos;
    return launch_ffn_w4_stream(a, group, sms, s, nullptr);
  }
  const uint16_t* yh = nullptr;
  const int32_t* yexp = nullptr;
  if ((r = launch_ffn_w4_gemm(f, ids, ws.pos, group, ws.ffn, &yh, &yexp, s, nullptr)) != MOE_OK) return r;
  return launch_w4_combine(yh, yexp, w, ws.pos, T, k, H, out, s);
}
