// The weights' gradients of the adapters: dA_l = sum_t dv_t x_t^T and dB_l = sum_t v_t dy_t^T over the rows of the
// sequences with adapter l, in one launch.
//
// Longer sequences: tcgen05.  D [128 features][R] of one adapter and one block of 128 features of x or dy, summed over
// tiles of 64 rows by TMA as they lie (features run along, so x is MN-major, and v is too).  The kernels before write
// each fp32 value of v and dv as three bf16 numbers (24 bits, nothing is rounded) next to each other, as columns of one
// product that are added in the end: done by this kernel's own warps, once for every block of features, it took three
// times as long as the product.  The tensor cores truncate what they add, so that an error grows with every
// step in one direction: after four tiles the sums are taken over into shared memory by additions that round.
// A cluster of CTAs divides the rows of an adapter where blocks are few; their sums meet in distributed shared memory in
// a fixed order.  x and dy are read once from HBM, x's tile and v's by every block of features from L2: 8192 rows of R 32,
// 2048 x 4096, 33 us where HBM's bytes take 16, at 60 B a clock and SM.
//
// Many short sequences: a thread per two features, on the CUDA cores (the tiles would be mostly empty).
#include <algorithm>

#include "adapters.cuh"

namespace moe {

constexpr int kAoThreads = 192;  // TMA warp, MMA warp, four warps that take the sums over
constexpr int kAoFeat = 128;     // features of a block (MMA M)
constexpr int kAoRows = 64;      // rows of a tile
constexpr int kAoXBytes = kAoRows * kAoFeat * 2;
constexpr int kAoAtom = kAoRows * 128;  // 64 columns of a tile
constexpr int kAoDrain = 4;             // tiles between two drains of an accumulator

struct AoGeo {
  int S, Rk, atoms, stages;       // CTAs of a cluster, R in sixteens, 64-column atoms of v, ring slots
  int acc, tmem;                  // accumulators, TMEM columns
  int off_part, off_bar;          // sums, barriers
  int blocks_a;                   // blocks of features of x
};

// The tiles [lo, hi) of the rows of one adapter, by a whole warp: sequence after sequence, 64 rows at a time.
struct AoTiles {
  const AdGradArgs& a;
  int l, lo, hi;
  int s = 0, at = 0, t = 0, left = 0, t0 = 0, n = 0;
  unsigned m = 0;
  __device__ __forceinline__ bool next(int& row0, int& rows) {
    for (;;) {
      if (at >= hi) return false;
      if (left > 0) {
        row0 = t;
        rows = min(kAoRows, left);
        t += kAoRows;
        left -= kAoRows;
        ++at;
        return true;
      }
      if (m == 0) {
        if (s >= a.n_seq) return false;
        // the next 32 sequences with one of l's, four times 32 looked at at once
        int q = s + (threadIdx.x & 31), id[4];
        unsigned any[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) id[i] = q + 32 * i < a.n_seq ? a.ids[q + 32 * i] : -1;
#pragma unroll
        for (int i = 0; i < 4; ++i) any[i] = __ballot_sync(MOE_FULL_MASK, id[i] == l);
        const int skip = any[0] ? 0 : any[1] ? 1 : any[2] ? 2 : 3;
        q += 32 * skip;
        s += 32 * (skip + 1);
        t0 = n = 0;
        if ((any[0] ? id[0] : any[1] ? id[1] : any[2] ? id[2] : id[3]) == l) {
          t0 = a.seq ? min(max(a.seq[q], 0), a.T) : q;
          n = a.seq ? max(min(max(a.seq[q + 1], 0), a.T) - t0, 0) : 1;
        }
        m = __ballot_sync(MOE_FULL_MASK, n > 0);
        continue;
      }
      const int j = __ffs(m) - 1;
      m &= m - 1;
      t = __shfl_sync(MOE_FULL_MASK, t0, j);
      left = __shfl_sync(MOE_FULL_MASK, n, j);
      const int skip = min((left + kAoRows - 1) / kAoRows, max(lo - at, 0));  // tiles of other CTAs
      at += skip;
      t += skip * kAoRows;
      left -= skip * kAoRows;
    }
  }
};

__device__ __forceinline__ float4 ao_remote(const float* p, uint32_t rank) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(mapa_shared(smem_u32(p), rank)));
  return v;
}

__global__ void __launch_bounds__(kAoThreads)
    adapters_outer_tile_kernel(const AdGradArgs a, const AoGeo g, const __grid_constant__ CUtensorMap mapX,
                               const __grid_constant__ CUtensorMap mapY, const __grid_constant__ CUtensorMap mapV) {
  extern __shared__ __align__(1024) unsigned char sm[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_rank(), S = g.S;
  const int block = blockIdx.x / S, l = blockIdx.y;
  const bool first = block < g.blocks_a;
  const int F = first ? a.K : a.N, f0 = (block - (first ? 0 : g.blocks_a)) * kAoFeat;
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + g.off_bar);  // a tile is ready
  uint64_t* landed = full + 4;                                   // one whose last rows are to be cleared has landed
  uint64_t* empty = landed + 4;
  uint64_t* tfull = empty + 4;   // an accumulator's tiles are done
  uint64_t* tempty = tfull + 2;  // and taken over
  uint64_t* done = tempty + 2;   // every product is
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(done + 1);
  int* s_total = reinterpret_cast<int*>(s_tmem + 1);
  volatile int* abort_flag = s_total + 1;
  unsigned* s_excess = reinterpret_cast<unsigned*>(s_total + 2);
  float* part = reinterpret_cast<float*>(sm + g.off_part);  // [Rk][128]
  const int stage = kAoXBytes + g.atoms * kAoAtom;
  if (threadIdx.x == 0) {
    prefetch_tmap(first ? &mapX : &mapY);
    prefetch_tmap(&mapV);
    for (int i = 0; i < g.stages; ++i) mbar_init(&full[i], 1), mbar_init(&landed[i], 1), mbar_init(&empty[i], 1);
    mbar_init(done, 1);
    for (int i = 0; i < g.acc; ++i) mbar_init(&tfull[i], 1), mbar_init(&tempty[i], 4);
    *abort_flag = 0;
    *s_total = 0;
    *s_excess = 0;
    mbar_fence_init();
  }
  pdl_wait();
  if (warp == 1) {  // (after the wait: a kernel before this one may have tensor memory to allocate yet)
    tmem_alloc(s_tmem, g.tmem);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_trigger();
  // An adapter has no more tiles than `most`: starts that descend (flagged by the kernels before) make its sequences overlap,
  // and no more work.
  const int most = a.T / kAoRows + a.n_seq;
  int mine = 0;
  unsigned excess = 0;
  for (int q0 = threadIdx.x; q0 < a.n_seq; q0 += 4 * kAoThreads) {
    int id[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) id[i] = q0 + i * kAoThreads < a.n_seq ? a.ids[q0 + i * kAoThreads] : -1;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (id[i] == l) {
        const int q = q0 + i * kAoThreads, n = a.seq ? min(max(a.seq[q + 1], 0), a.T) - min(max(a.seq[q], 0), a.T) : 1;
        if (n > 0) mine = min(mine + (n + kAoRows - 1) / kAoRows, most), excess += (unsigned)(n - kAdLong);
      }
  }
  __syncwarp();
  mine = min((int)__reduce_add_sync(MOE_FULL_MASK, mine), most);  // (a warp's sum is below 2^30)
  if (lane == 0 && mine) atomicAdd(s_total, mine);
  if (a.both) {
    excess = __reduce_add_sync(MOE_FULL_MASK, excess);
    if (lane == 0) atomicAdd(s_excess, excess);
  }
  __syncthreads();
  const uint32_t tmem = *s_tmem;
  if (a.both && (int)*s_excess < 0) {  // (the whole cluster) rows fewer than kAdLong a sequence: the other kernel's
    if (warp == 1) tmem_dealloc(tmem, g.tmem);
    return;
  }
  const int total = min(*s_total, most);
  AoTiles tiles{a, l, (int)((long long)total * rank / S), (int)((long long)total * (rank + 1) / S)};
  const int nt = tiles.hi - tiles.lo;
  bool dead = false;  // (of a whole warp) nothing is waited for or issued after a timeout
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (!dead) dead = !ad_wait(bar, parity, abort_flag, a.status);
  };
  int row0 = 0, rows = 0;
  // The loops that issue copies and products are run by whole warps, so that their operands stay in uniform registers.
  if (warp == 0) {
    const bool lead = elect_one();
    const CUtensorMap* map = first ? &mapX : &mapY;
    int s = 0, issued = 0;
    uint32_t ph = 1, cleared = 0, last = 0;  // of a slot: the number of its tiles to be cleared, whether its last is one
    while (tiles.next(row0, rows) && !dead) {
      if (issued >= g.stages) wait(&empty[s], ph);
      if (dead) break;
      uint64_t* bar = rows % 16 ? &landed[s] : &full[s];
      last = rows % 16 ? last | 1u << s : last & ~(1u << s);
      cleared ^= rows % 16 ? 1u << s : 0u;  // (its parity)
      if (lead) {
        unsigned char* st = sm + s * stage;
        mbar_expect_tx(bar, (uint32_t)stage);
        tma_load_3d(st, map, bar, f0, row0, 0);
        tma_load_3d(st + kAoAtom, map, bar, f0 + 64, row0, 0);
        for (int n = 0; n < g.atoms; ++n)
          tma_load_3d(st + kAoXBytes + n * kAoAtom, &mapV, bar, n * 64, row0, first ? 0 : 1);
      }
      __syncwarp();
      ++issued;
      if (++s == g.stages) s = 0, ph ^= 1;
    }
    // after a timeout every copy lands before the CTA may go
    if (dead || *abort_flag)
      for (int j = max(0, issued - g.stages); j < issued; ++j) {
        const int q = j % g.stages;
        if (last >> q & 1) mbar_wait(&landed[q], ~(cleared >> q) & 1);
        else mbar_wait(&full[q], (j / g.stages) & 1);
      }
    __syncwarp();
  } else if (warp == 1) {
    const bool lead = elect_one();
    const int cols = 3 * g.Rk, n1 = cols <= 256 ? cols : 192;
    const uint32_t id1 = idesc_bf16(kAoFeat, n1, 1, 1), id2 = idesc_bf16(kAoFeat, max(cols - n1, 16), 1, 1);
    const uint64_t a0 = smem_desc_l(smem_u32(sm), kAoAtom, 1024, kLayoutSw128);
    const uint64_t b0 = smem_desc_l(smem_u32(sm) + kAoXBytes, kAoAtom, 1024, kLayoutSw128);
    constexpr uint32_t kStep = 2048 >> 4;  // 16 rows
    int s = 0, n = 0, b = 0;  // slot; tile of the accumulator; accumulator
    uint32_t ph = 0, tph = 1;  // phases of slots and accumulators
    for (int i = 0; tiles.next(row0, rows); ++i) {
      if (n == 0 && i >= kAoDrain * g.acc) wait(&tempty[b], tph);
      wait(&full[s], ph);
      tc_fence_after();
      const bool last = ++n == kAoDrain || i == nt - 1;
      if (lead && !dead) {
        const uint32_t d = tmem + b * cols;
        const uint64_t ad = a0 + (uint64_t)(s * (stage >> 4)), bd = b0 + (uint64_t)(s * (stage >> 4));
        if (rows > 48) {
          umma_f16_k64(d, ad, bd, id1, n > 1, kStep, kStep);
          if (cols > n1) umma_f16_k64(d + n1, ad, bd + (3 * kAoAtom >> 4), id2, n > 1, kStep, kStep);
        } else {
          for (int k = 0; k * 16 < rows; ++k) {
            umma_f16(d, ad + k * kStep, bd + k * kStep, id1, n > 1 || k);
            if (cols > n1) umma_f16(d + n1, ad + k * kStep, bd + (3 * kAoAtom >> 4) + k * kStep, id2, n > 1 || k);
          }
        }
      }
      if (lead) {
        umma_commit(&empty[s]);
        if (last) umma_commit(&tfull[b]);
      }
      __syncwarp();
      if (++s == g.stages) s = 0, ph ^= 1;
      if (last) {
        n = 0;
        if (++b == g.acc) b = 0, tph ^= 1;
      }
    }
    if (lead) umma_commit(done);
    __syncwarp();
    mbar_wait(done, 0);  // also after a timeout: nothing of this CTA is read or written any more
  } else {
    const int q = warp & 3, f = q * 32 + lane;  // of the sums: lane = feature
    int drained = 0, cleared = 0;
    auto drain = [&] {  // the parts of a rank are Rk columns apart
      const int j = drained++, b = j % g.acc;
      wait(&tfull[b], (j / g.acc) & 1);
      tc_fence_after();
      for (int c = 0; c < g.Rk; c += 16) {
        float v[16], w[16], x[16];
        const uint32_t at = tmem + ((uint32_t)(q * 32) << 16) + b * 3 * g.Rk + c;
        tmem_ld_w<16>(at, v);
        tmem_ld_w<16>(at + g.Rk, w);
        tmem_ld_w<16>(at + 2 * g.Rk, x);
        tmem_ld_wait();
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          float* p = part + (c + k) * kAoFeat + f;
          const float sum = v[k] + (w[k] + x[k]);
          *p = j ? *p + sum : sum;
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&tempty[b]);
    };
    for (int i = 0; tiles.next(row0, rows); ++i) {
      const int s = i % g.stages;
      // The rest of the last 16 rows belongs to others, whatever it is: each slot has a warp that clears it, and makes the
      // tile ready in the place of its copies.  (The warp waits for such tiles alone, on a barrier of their own: the slot
      // is not used again before, so that it can be neither behind nor ahead of the barrier's phases.)
      if (s == warp - 2 && rows % 16) {
        wait(&landed[s], cleared & 1);
        ++cleared;
        const int rest = 16 - rows % 16, pieces = (2 + g.atoms) * 8;
        for (int u = lane; u < rest * pieces; u += 32) {
          const int r = rows + u / pieces, p = u % pieces;
          *reinterpret_cast<uint4*>(sm + s * stage + (p / 8) * kAoAtom + r * 128 + (p % 8) * 16) = make_uint4(0, 0, 0, 0);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[s]);
      }
      // with two accumulators the one before last's sums are taken over while the products of the last one run
      if (i % kAoDrain == kAoDrain - 1 && i / kAoDrain >= g.acc - 1) drain();
    }
    while (drained * kAoDrain < nt) drain();
    if (nt == 0)
      for (int r = 0; r < g.Rk; ++r) part[r * kAoFeat + f] = 0.f;
    __syncwarp();
  }
  if (S > 1) cluster_sync();
  else __syncthreads();
  {
    const int r0 = a.R * rank / S, r1 = a.R * (rank + 1) / S;
    float* out = (first ? a.da : a.db) + (size_t)l * a.R * F + f0;
    for (int i = threadIdx.x; i < (r1 - r0) * (kAoFeat / 4); i += kAoThreads) {
      const int r = r0 + i / (kAoFeat / 4), f = i % (kAoFeat / 4) * 4;
      float4 p[8], v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int c = 0; c < 8; ++c) p[c] = c < S ? ao_remote(part + r * kAoFeat + f, c) : v;
#pragma unroll
      for (int c = 0; c < 8; ++c) v.x += p[c].x, v.y += p[c].y, v.z += p[c].z, v.w += p[c].w;
      if (f0 + f < F) *reinterpret_cast<float4*>(out + (size_t)r * F + f) = v;
    }
    __syncwarp();
  }
  if (S > 1) cluster_sync();  // no CTA leaves while another one reads its shared memory
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, g.tmem);
  }
}

// Whether an adapter's rows are kAdLong a sequence or more, as the kernel above finds it (by all threads of the CTA).
__device__ __forceinline__ bool ao_long(const AdGradArgs& a, int l, unsigned* excess) {
  if (threadIdx.x == 0) *excess = 0;
  __syncthreads();
  unsigned mine = 0;
  for (int q0 = threadIdx.x; q0 < a.n_seq; q0 += 4 * blockDim.x) {
    int id[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) id[i] = q0 + i * blockDim.x < a.n_seq ? a.ids[q0 + i * blockDim.x] : -1;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (id[i] == l) {
        const int q = q0 + i * blockDim.x, n = min(max(a.seq[q + 1], 0), a.T) - min(max(a.seq[q], 0), a.T);
        if (n > 0) mine += (unsigned)(n - kAdLong);
      }
  }
  __syncwarp();
  mine = __reduce_add_sync(MOE_FULL_MASK, mine);
  if ((threadIdx.x & 31) == 0) atomicAdd(excess, mine);
  __syncthreads();
  return (int)*excess >= 0;
}

// Short sequences: a thread has two features and 16 ranks; the rows of the adapter are listed in shared memory.
constexpr int kAsThreads = 128;
constexpr int kAsRanks = 16;
constexpr int kAsList = 1024;
__device__ __forceinline__ void ao_short(const AdGradArgs& a, int blocks_a) {
  __shared__ int s_row[kAsList], s_scan[33];
  const bool first = (int)blockIdx.x < blocks_a;
  const int F = first ? a.K : a.N, f = (((int)blockIdx.x - (first ? 0 : blocks_a)) * kAsThreads + threadIdx.x) * 2;
  const int l = blockIdx.y, r0 = blockIdx.z * kAsRanks, nr = min(kAsRanks, a.R - r0);
  const uint16_t* x = (first ? a.x : a.dy) + (f < F ? f : 0);
  const long long ld = first ? a.ldx : a.ldy;
  const float* v = (first ? a.dv : a.v) + r0;
  float acc[2 * kAsRanks] = {};
  unsigned left = (unsigned)a.T;  // rows: sequences that overlap (starts that descend, flagged before) are no more work
  // sequences 128 at a time (512 without any of l's are passed over at once); their rows listed in order, up to kAsList of
  // them at a time
  for (int q0 = 0; q0 < a.n_seq && left > 0; q0 += kAsThreads) {
    const int q = q0 + (int)threadIdx.x;
    if (q0 % (4 * kAsThreads) == 0 && a.n_seq > 4 * kAsThreads) {
      bool any = false;
#pragma unroll
      for (int i = 0; i < 4; ++i) any |= q + i * kAsThreads < a.n_seq && a.ids[q + i * kAsThreads] == l;
      if (!__syncthreads_or(any)) {
        q0 += 3 * kAsThreads;
        continue;
      }
    }
    int t = 0, n = 0;
    if (q < a.n_seq && a.ids[q] == l) {
      t = a.seq ? min(max(a.seq[q], 0), a.T) : q;
      n = a.seq ? max(min(max(a.seq[q + 1], 0), a.T) - t, 0) : 1;
    }
    int sum;
    const int at = block_exclusive_scan(n, s_scan, &sum);  // (at most 2^31)
    const int total = (int)min((unsigned)sum, left);
    left -= (unsigned)total;
    for (int base = 0; base < total; base += kAsList) {
      for (int i = max(base - at, 0); i < min(n, base + kAsList - at); ++i) s_row[at + i - base] = t + i;
      __syncthreads();
      const int m = min(kAsList, total - base);
      for (int i = 0; i < m; i += 4) {
        uint32_t xv[4];
        float vv[4][kAsRanks];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int row = s_row[min(i + u, m - 1)];
          xv[u] = i + u < m ? *reinterpret_cast<const uint32_t*>(x + row * ld) : 0u;
#pragma unroll
          for (int j = 0; j < kAsRanks; ++j) vv[u][j] = j < nr && i + u < m ? v[(size_t)row * a.R + j] : 0.f;
        }
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
          for (int j = 0; j < kAsRanks; ++j) {
            acc[2 * j] = fmaf(vv[u][j], bf16_lo(xv[u]), acc[2 * j]);
            acc[2 * j + 1] = fmaf(vv[u][j], bf16_hi(xv[u]), acc[2 * j + 1]);
          }
      }
      __syncthreads();
    }
  }
  if (f >= F) return;
  float* o = (first ? a.da : a.db) + ((size_t)l * a.R + r0) * F + f;
#pragma unroll
  for (int j = 0; j < kAsRanks; ++j)
    if (j < nr) *reinterpret_cast<float2*>(o + (size_t)j * F) = make_float2(acc[2 * j], acc[2 * j + 1]);
}
__global__ void __launch_bounds__(kAsThreads) adapters_outer_short_kernel(const AdGradArgs a, int blocks_a) {
  if (!a.both) {
    pdl_wait();
    ao_short(a, blocks_a);
    return;
  }
  // The kernel of the tiles has waited for what came before it and writes other adapters: only the end has to be in order.
  __shared__ unsigned s_excess;
  if (!ao_long(a, blockIdx.y, &s_excess)) ao_short(a, blocks_a);
  if (blockIdx.x + blockIdx.y + blockIdx.z == 0) pdl_wait();
}

static int ad_launch_outer_short(const AdGradArgs& a, cudaStream_t s) {
  const int per = 2 * kAsThreads, blocks_a = (a.K + per - 1) / per, blocks = blocks_a + (a.N + per - 1) / per;
  MOE_CUDA_TRY(launch_pdl(adapters_outer_short_kernel, dim3(blocks, a.L, (a.R + kAsRanks - 1) / kAsRanks), dim3(kAsThreads), 0, s,
                          a, blocks_a));
  return MOE_OK;
}

int ad_launch_outer(const AdGradArgs& a, int sms, cudaStream_t s) {
  if (!a.parts) return ad_launch_outer_short(a, s);
  AoGeo g = {};
  g.Rk = (a.R + 15) / 16 * 16;
  g.atoms = (3 * g.Rk + 63) / 64;
  g.acc = 6 * g.Rk <= 512 ? 2 : 1;
  g.tmem = 32;
  while (g.tmem < g.acc * 3 * g.Rk) g.tmem *= 2;
  const int stage = kAoXBytes + g.atoms * kAoAtom;
  // two CTAs a SM up to 32 ranks, else one; a slot for each of the four warps that clear rows at most
  g.stages = std::min(4, ((g.Rk <= 32 ? 112 : 224) * 1024 - g.Rk * kAoFeat * 4) / stage);
  g.off_part = g.stages * stage;
  g.off_bar = g.off_part + g.Rk * kAoFeat * 4;
  g.blocks_a = (a.K + kAoFeat - 1) / kAoFeat;
  const int blocks = g.blocks_a + (a.N + kAoFeat - 1) / kAoFeat;
  const int bytes = g.off_bar + 512;
  // CTAs for about two a SM; the adapters in use are at most the sequences
  const long long busy = (long long)blocks * std::min(a.L, a.n_seq);
  g.S = 1;
  while (g.S < 8 && busy * g.S * 2 <= 2ll * sms && a.T >= 128 * g.S) g.S *= 2;
  CUtensorMap mx, my, mv;
  for (int w = 0; w < 2; ++w) {
    const uint64_t ld = (uint64_t)(w ? a.ldy : a.ldx) * 2;
    const uint64_t dims[3] = {(uint64_t)(w ? a.N : a.K), (uint64_t)a.T, 1}, st[2] = {ld, ld};
    const uint32_t box[3] = {64, kAoRows, 1};
    if (int rc = encode_tmap_3d_bf16(w ? &my : &mx, w ? a.dy : a.x, dims, st, box, CU_TENSOR_MAP_SWIZZLE_128B)) return rc;
  }
  {
    const uint64_t ld = (uint64_t)g.Rk * 6;
    const uint64_t dims[3] = {(uint64_t)g.Rk * 3, (uint64_t)a.T, 2}, st[2] = {ld, ld * a.T};
    const uint32_t box[3] = {64, kAoRows, 1};
    if (int rc = encode_tmap_3d_bf16(&mv, a.parts, dims, st, box, CU_TENSOR_MAP_SWIZZLE_128B)) return rc;
  }
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = g.S;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(blocks * g.S), (unsigned)a.L);
  cfg.blockDim = dim3(kAoThreads);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = s;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  static bool done[64] = {};
  MOE_CUDA_TRY(ensure_smem(adapters_outer_tile_kernel, 227 * 1024 - 512, done));
  MOE_CUDA_TRY(cudaLaunchKernelEx(&cfg, adapters_outer_tile_kernel, a, g, mx, my, mv));
  return a.both ? ad_launch_outer_short(a, s) : MOE_OK;
}

}  // namespace moe
