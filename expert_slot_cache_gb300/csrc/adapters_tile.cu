// Adapters of longer sequences on the tcgen05 tensor cores: out = base + (scale_l x A_l^T) B_l in one launch.
//
// A cluster of 2, 4 or 8 CTAs has a tile of 32, 64 or 128 rows of one sequence.  CTA c multiplies its share of the K inputs by
// all R ranks (D1 [rows][R] in TMEM: x by TMA, K-major; A_l K-major); the shares meet in distributed shared memory, where
// each CTA adds up some of the rows in a fixed order, scales them and hands them to all; then CTA c multiplies them by
// its share of the N outputs (D2 [rows][128], double-buffered; B_l as it lies, MN-major) and adds base on the way out.
// Nothing but x, A, B, base and out crosses the memory, so those bytes bound a large batch: 4096 rows of R 64, 2048 x 4096,
// take 27.6 us where they take 13; the second product with its 67 MB takes 8, some 13 go to dependent steps before (x's way
// in 3, sums through the cluster 3, v's way to the other CTAs some 3.7, at 14 B a clock and SM).  64 rows of R 16 take 8.3 us.
// Sending base to L2 while the first product runs costs more than it hides (4096 rows 3.6 us more, 16,384 of R 16 8.3).
//
// The rows of a tile of 32 or 64 stand in the 128 lanes of D several times, so that all four epilogue warps (each reads
// 32 lanes) have columns to store.  The tensor cores truncate what they add, so that an error grows with every step in one
// direction: D1 is several accumulators in turn, of 16 additions each at most, added by additions that round.  Where four of
// them are not enough (DRAINS: more than 1024 inputs a CTA), the epilogue warps take each over into a sum in TMEM while the
// others are filled.  (200 rows of 131,072 inputs, R 16: 87 us; with four accumulators of 256 additions 73, and v off by
// 5e-6.  A kernel of its own: as a branch of the one kernel it cost the others 1 to 3%.)
//
// v = scale x A^T enters the second product as a sum of three bf16 numbers, which are its 24 bits: with two (16 bits) a
// result in which ranks nearly cancel was off by more than fp32 sums are.  (The third costs 4096 rows of R 64 1.2 us of 27.6,
// on v's way to the other CTAs.)  The products cost little beside the bytes: 2 R flops a byte of x.
#include <algorithm>

#include "adapters.cuh"

namespace moe {

constexpr int kAtThreads = 192;  // TMA warp, MMA warp, four epilogue warps
constexpr int kAtRows = 128;     // rows of a tile, at most (MMA M)
constexpr int kAtCols = 128;     // outputs of a step of the second product
constexpr int kAtXBytes = kAtRows * 128;  // 64 inputs of a tile's rows
constexpr int kAtStage = 4096;            // 32 rows x 128 bytes of results
constexpr int kAtStages2 = 2;
constexpr int kAtAcc = 4;    // accumulators of D1; or three and their sum,
constexpr int kAtDrain = 4;  // after so many steps of 64 inputs (four additions each)
constexpr int kAtParts = 3;  // bf16 numbers that v's fp32 is the sum of

struct AtGeo {
  int tile, Rk, stages1;        // rows of a tile, R in sixteens, slots of the first ring
  int tmem;                     // TMEM columns: kAtAcc accumulators, two steps of D2
  int off2, off_part, off_bar;  // second ring, partial sums / staging, barriers
  int short_rows;               // sequences of up to so many rows are the row kernel's,
  int beside;                   // which has been launched before this one and may still run
};

__device__ __forceinline__ uint64_t at_desc(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
  return smem_desc_l(saddr, lbo, sbo, kLayoutSw128);
}
__device__ __forceinline__ void at_cluster_arrive_relaxed() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void at_cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void at_cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void at_fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void at_store4(uint32_t caddr, float a, float b, float c, float d) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(caddr), "f"(a), "f"(b), "f"(c), "f"(d) : "memory");
}
// Shared memory of this CTA to another one's; the bytes count on an mbarrier there.
__device__ __forceinline__ void at_send(uint32_t to, uint32_t from, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(to),
               "r"(from), "r"(bytes), "r"(bar)
               : "memory");
}
__device__ __forceinline__ void at_copy16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}

// Bounds of segment j: the rows before the first sequence, the sequences, the rows behind the last.
__device__ __forceinline__ void at_segment(const AdArgs& a, int j, int& t0, int& t1) {
  t0 = j == 0 ? 0 : min(max(a.seq[j - 1], 0), a.T);
  t1 = j == a.n_seq + 1 ? a.T : min(max(a.seq[j], 0), a.T);
}

struct AtTile {
  int row0, rows, l;  // rows 0: there is no such tile
};
// Rows of a segment that are the tiles'.
__device__ __forceinline__ int at_rows(const AdArgs& a, const AtGeo& g, bool seq, int t0, int t1, int l) {
  const bool copies = a.kept || (a.out && (a.out != a.base || a.ldo != a.ldb));
  return (seq && t1 - t0 <= g.short_rows) || (l < 0 && !copies) ? 0 : max(t1 - t0, 0);
}

// Tile `ti` of the batch where a thread has a segment: the tiles follow one another, so that clusters without one are the
// last.  By all threads of the CTA.
__device__ __forceinline__ AtTile at_find_few(const AdArgs& a, const AtGeo& g, int ti, int* tmp, int* tile) {
  const int j = (int)threadIdx.x;
  int t0 = 0, t1 = 0, l = -1, n = 0;
  if (j == 0) tile[1] = 0;
  if (j < a.n_seq + 2) {
    at_segment(a, j, t0, t1);
    const bool seq = j >= 1 && j <= a.n_seq;
    if (seq) {
      l = ad_adapter(a, j - 1);
      if (a.seq[j] < a.seq[j - 1]) set_status(a.status, MOE_DEV_BAD_GROUPS);
    }
    n = (at_rows(a, g, seq, t0, t1, l) + g.tile - 1) / g.tile;
  }
  int total;
  const int at = block_exclusive_scan(n, tmp, &total);
  if (ti >= at && ti < at + n) {
    tile[0] = t0 + (ti - at) * g.tile;
    tile[1] = min(g.tile, t1 - tile[0]);
    tile[2] = l;
  }
  __syncthreads();
  return {tile[0], tile[1], tile[2]};
}

// The same with any number of segments, by each warp for itself.  Segment j's tiles begin at floor(t0 / tile) + j, which
// leaves room for them: floor(t1 / tile) + 1 - floor(t0 / tile) is ceil((t1 - t0) / tile) at least.  So the segment is found
// in the starts themselves, 32 of them looked at at once.  (A walk through all of them took 16 ms for 32,768 sequences of 8
// rows, this one 1.9.  With 40 and 100 sequences the clusters without a tile among the others cost 0.7 and 2.4 us.)
__device__ __forceinline__ AtTile at_find_many(const AdArgs& a, const AtGeo& g, int ti) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = a.n_seq + 1;  // the last segment that begins at or before ti lies in [lo, hi]
  for (;;) {
    const int step = (hi - lo) / 32 + 1, j = lo + lane * step;
    int t0 = 0, t1 = 0, l = -1;
    if (j <= hi) {
      at_segment(a, j, t0, t1);
      if (step == 1 && j >= 1 && j <= a.n_seq) l = ad_adapter(a, j - 1);
    }
    const int last = 31 - __clz(__ballot_sync(MOE_FULL_MASK, j <= hi && t0 / g.tile + j <= ti) | 1u);
    lo += last * step;
    hi = min(hi, lo + step - 1);
    if (step > 1) continue;
    const int from = __shfl_sync(MOE_FULL_MASK, t0, last), end = __shfl_sync(MOE_FULL_MASK, t1, last);
    l = __shfl_sync(MOE_FULL_MASK, l, last);
    const int row0 = from + (ti - from / g.tile - lo) * g.tile;
    return {row0, at_rows(a, g, lo >= 1 && lo <= a.n_seq, from, end, l) > 0 ? max(min(g.tile, end - row0), 0) : 0, l};
  }
}
// Whether a thread has a segment.
__host__ __device__ inline bool at_few(const AdArgs& a) { return a.n_seq + 2 <= kAtThreads; }

// Where 16-byte piece i of the partial sums lies: rows a power of two apart meet no bank twice.
__device__ __forceinline__ uint32_t at_piece(uint32_t i) { return (i ^ ((i >> 3) & 7)) * 16; }

template <bool F32, int C, bool DRAINS>
__global__ void __launch_bounds__(kAtThreads, 2)
    adapters_tile_kernel(const AdArgs a, const AtGeo g, const __grid_constant__ CUtensorMap mapX,
                         const __grid_constant__ CUtensorMap mapA, const __grid_constant__ CUtensorMap mapB) {
  constexpr int kSize = F32 ? 4 : 2;
  extern __shared__ __align__(1024) unsigned char sm[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_rank();
  uint64_t* full1 = reinterpret_cast<uint64_t*>(sm + g.off_bar);
  uint64_t* empty1 = full1 + 4;
  uint64_t* full2 = empty1 + 4;
  uint64_t* empty2 = full2 + kAtStages2;
  uint64_t* tfull = empty2 + kAtStages2;
  uint64_t* tempty = tfull + 2;
  uint64_t* d1full = tempty + 2;
  uint64_t* vfull = d1full + 1;                    // v of all rows is there,
  uint64_t* vrep = vfull + 1;                      // in all the lanes
  uint64_t* done = vrep + 1;                       // every product is
  uint64_t* afull = done + 1;                      // an accumulator of D1 is done,
  uint64_t* aempty = afull + kAtAcc - 1;           // and taken over
  int* s_tile = reinterpret_cast<int*>(aempty + kAtAcc - 1);  // [4]
  int* s_scan = s_tile + 4;                                   // [33]
  volatile int* abort_flag = s_scan + 33;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(s_scan + 34);
  if (threadIdx.x == 0) {
    prefetch_tmap(&mapX);
    prefetch_tmap(&mapA);
    prefetch_tmap(&mapB);
    for (int i = 0; i < g.stages1; ++i) mbar_init(&full1[i], 1), mbar_init(&empty1[i], 1);
    for (int i = 0; i < kAtStages2; ++i) mbar_init(&full2[i], 1), mbar_init(&empty2[i], 1);
    for (int i = 0; i < 2; ++i) mbar_init(&tfull[i], 1), mbar_init(&tempty[i], 4);
    mbar_init(d1full, 1);
    mbar_init(vfull, 2);
    mbar_init(vrep, 4);
    mbar_init(done, 1);
    if (DRAINS)
      for (int i = 0; i < kAtAcc - 1; ++i) mbar_init(&afull[i], 1), mbar_init(&aempty[i], 4);
    *abort_flag = 0;
    mbar_fence_init();
  }
  // The row kernel waited for what came before it and reads and writes other rows: only the end has to be in order.
  if (!g.beside) pdl_wait();
  if (warp == 1) {  // (after the wait: a kernel before this one may have tensor memory to allocate yet)
    tmem_alloc(s_tmem, g.tmem);
    tmem_relinquish();
  }
  tc_fence_before();
  const int ti = (int)cluster_index();
  AtTile found;
  if (at_few(a)) {
    found = at_find_few(a, g, ti, s_scan, s_tile);
  } else {
    found = at_find_many(a, g, ti);
    // (there are more clusters than sequences, so that every sequence is looked at once)
    if (threadIdx.x == kAtThreads - 1 && rank == 0 && ti < a.n_seq) {
      ad_adapter(a, ti);
      if (a.seq[ti + 1] < a.seq[ti]) set_status(a.status, MOE_DEV_BAD_GROUPS);
    }
    __syncthreads();
  }
  const int row0 = found.row0, rows = found.rows, l = found.l;
  tc_fence_after();
  const uint32_t tmem = *s_tmem;
  if (rows == 0 || l < 0) {  // (the whole cluster)
    if (warp == 1) tmem_dealloc(tmem, g.tmem);
    if (rows == 0) {  // the last one waits for all that have no tile, and leave room for those that have
      if (g.beside && ti == (int)cluster_count() - 1) pdl_wait();
      return;
    }
    if (g.beside) pdl_wait();
  }
  const int NT = (a.N + kAtCols - 1) / kAtCols, nt0 = NT * rank / C, nt1 = NT * (rank + 1) / C;
  if (l < 0) {
    if (a.kept && rank == 0)
      for (int i = threadIdx.x; i < rows * a.R; i += kAtThreads) a.kept[(size_t)row0 * a.R + i] = 0.f;
    if (!a.out || (a.out == a.base && a.ldo == a.ldb)) return;
    const int p0 = nt0 * kAtCols * kSize / 16, np = min(nt1 * kAtCols, a.N) * kSize / 16 - p0;
    for (int i = threadIdx.x; i < rows * np; i += kAtThreads) {
      const long long t = row0 + i / np, p = p0 + i % np;
      uint4 v = make_uint4(0, 0, 0, 0);
      if (a.base) v = reinterpret_cast<const uint4*>(reinterpret_cast<const uint8_t*>(a.base) + t * a.ldb * kSize)[p];
      reinterpret_cast<uint4*>(reinterpret_cast<uint8_t*>(a.out) + t * a.ldo * kSize)[p] = v;
    }
    return;
  }
  unsigned char* ring2 = sm + g.off2;
  unsigned char* part = sm + g.off_part;
  const int stage1 = kAtXBytes + g.Rk * 128, stage2 = g.Rk * 256;
  const int nt = a.out ? nt1 - nt0 : 0;
  at_cluster_arrive_relaxed();    // waited for where another CTA's shared memory is written first
  if (!g.beside) pdl_trigger();  // (after the allocation: a kernel that starts now may allocate, too)
  bool dead = false;  // (of a whole warp) nothing is waited for or issued after a timeout
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (!dead) dead = !ad_wait(bar, parity, abort_flag, a.status);
  };
  const int kc = (a.K + 63) / 64, kc0 = kc * rank / C, kc1 = kc * (rank + 1) / C, nk = kc1 - kc0;
  const int nacc = DRAINS ? kAtAcc - 1 : (nk + kAtDrain - 1) / kAtDrain;  // accumulators of D1, taken in turn
  const int copies = kAtRows / g.tile;                    // of a tile's rows in the 128 lanes
  const int per = g.tile / C;                             // rows that a CTA adds up
  const int mine = max(0, min(per, rows - rank * per));
  const int atoms = (kAtParts * g.Rk + 63) / 64;                // of v: 128 lanes x 128 bytes
  // ---- the first product.  The loops that issue copies and products are run by whole warps, so that their operands
  // stay in uniform registers.
  const bool lead = elect_one();
  int loaded1 = 0, loaded2 = 0;
  auto load2 = [&] {  // the next step of the second product
    const int i = loaded2 % kAtStages2;
    if (lead) {
      unsigned char* st = ring2 + i * stage2;
      mbar_expect_tx(&full2[i], (uint32_t)stage2);
      tma_load_3d(st, &mapB, &full2[i], (nt0 + loaded2) * kAtCols, 0, l);
      tma_load_3d(st + g.Rk * 128, &mapB, &full2[i], (nt0 + loaded2) * kAtCols + 64, 0, l);
    }
    __syncwarp();
    ++loaded2;
  };
  if (warp == 0) {
    int s = 0;
    uint32_t ph = 1;
    for (int i = 0; i < nk && !dead; ++i) {
      if (i >= g.stages1) wait(&empty1[s], ph);
      if (dead) break;
      if (lead) {
        unsigned char* st = sm + s * stage1;
        mbar_expect_tx(&full1[s], (uint32_t)(g.tile + g.Rk) * 128);
        tma_load_3d(st, &mapX, &full1[s], (kc0 + i) * 64, row0, 0);
        tma_load_3d(st + kAtXBytes, &mapA, &full1[s], (kc0 + i) * 64, 0, l);
      }
      __syncwarp();
      ++loaded1;
      if (++s == g.stages1) s = 0, ph ^= 1;
    }
    while (loaded2 < min(nt, kAtStages2) && !dead) load2();
    if (lead) mbar_expect_tx(vfull, (uint32_t)(atoms * 128 * (rows - mine)));
    __syncwarp();
  } else if (warp == 1 && nk > 0) {
    const uint32_t idesc = idesc_bf16(kAtRows, g.Rk, 0, 0);
    const uint64_t a0 = at_desc(smem_u32(sm), 16, 1024), b0 = at_desc(smem_u32(sm) + kAtXBytes, 16, 1024);
    int s = 0, n = 0;
    uint32_t ph = 0, aph = 1;
    auto step = [&](bool first) {
      wait(&full1[s], ph);
      tc_fence_after();
      const uint64_t at = (uint64_t)(s * (stage1 >> 4));
      if (lead && !dead) umma_f16_k64(tmem + n * g.Rk, a0 + at, b0 + at, idesc, !first, 2, 2);
      if (lead) umma_commit(&empty1[s]);
      __syncwarp();
      if (++s == g.stages1) s = 0, ph ^= 1;
    };
    if constexpr (DRAINS) {
      for (int i = 0; i < nk; i += kAtDrain) {
        if (i >= kAtDrain * nacc) wait(&aempty[n], aph);
        for (int k = i; k < min(i + kAtDrain, nk); ++k) step(k == i);
        if (lead) umma_commit(&afull[n]);
        __syncwarp();
        if (++n == nacc) n = 0, aph ^= 1;
      }
    } else {
      for (int i = 0; i < nk; ++i) {
        step(i < nacc);
        if (++n == nacc) n = 0;
      }
    }
    if (lead) umma_commit(d1full);
    __syncwarp();
  }
  const int q = warp & 3, row = (q * 32 + lane) % g.tile, copy = q * 32 / g.tile;
  const uint32_t lanes = (uint32_t)(q * 32) << 16;
  float scale = 0.f;
  if (warp >= 2) {
    scale = a.scale[l];
    if constexpr (DRAINS) {
      const uint32_t sum = tmem + lanes + (kAtAcc - 1) * g.Rk;
      for (int j = 0; j * kAtDrain < nk; ++j) {
        const int n = j % nacc;
        wait(&afull[n], (j / nacc) & 1);
        tc_fence_after();
        for (int c = 0; c < g.Rk && copy == 0; c += 16) {
          float v[16], w[16];
          tmem_ld_w<16>(tmem + lanes + n * g.Rk + c, v);
          if (j) tmem_ld_w<16>(sum + c, w);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 16; ++i) v[i] = j ? v[i] + w[i] : v[i];
          tmem_st16(sum + c, v);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&aempty[n]);
      }
    }
    if (nk > 0) {
      wait(d1full, 0);
      tc_fence_after();
    }
    const uint32_t dst = mapa_shared(smem_u32(part), (uint32_t)(row / per));
    const int first = (rank * per + row % per) * (g.Rk / 4);
    at_cluster_wait();  // every CTA of the cluster has started
    const uint32_t d1 = tmem + lanes + (DRAINS ? (kAtAcc - 1) * g.Rk : 0);  // what is left to be added up
    const int left = DRAINS ? min(nk, 1) : nacc;
    for (int c = 0; c < g.Rk && copy == 0; c += 16) {
      float w[kAtAcc][16];
#pragma unroll
      for (int n = 0; n < kAtAcc; ++n)
        if (n < left) tmem_ld_w<16>(d1 + n * g.Rk + c, w[n]);
      tmem_ld_wait();
      float v[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        v[i] = 0.f;
#pragma unroll
        for (int n = 0; n < kAtAcc; ++n)
          if (n < left) v[i] += w[n][i];
      }
      if (row < rows) {
#pragma unroll
        for (int i = 0; i < 16; i += 4) at_store4(dst + at_piece(first + (c + i) / 4), v[i], v[i + 1], v[i + 2], v[i + 3]);
      }
    }
    tc_fence_before();
    __syncwarp();
  } else {
    at_cluster_wait();
  }
  cluster_sync();  // partial sums are there; the first ring is free in every CTA (its products are done)
  if (warp >= 2) {
    // piece p (8 of the 3 Rk values) of row t
    auto v_at = [&](int t, int p) { return (uint32_t)((p / 8) * kAtXBytes + t * 128 + ((p % 8) ^ (t & 7)) * 16); };
    const int g8 = g.Rk / 8;
    for (int i = threadIdx.x - 64; i < mine * g8; i += 128) {
      const int r = i / g8, c = (i % g8) * 8, t = rank * per + r;
      float v[8] = {};
#pragma unroll
      for (int p = 0; p < C; ++p) {
        const uint32_t at = (p * per + r) * (g.Rk / 4) + c / 4;
        const float4 x = *reinterpret_cast<const float4*>(part + at_piece(at));
        const float4 y = *reinterpret_cast<const float4*>(part + at_piece(at + 1));
        v[0] += x.x, v[1] += x.y, v[2] += x.z, v[3] += x.w, v[4] += y.x, v[5] += y.y, v[6] += y.z, v[7] += y.w;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[j] = c + j < a.R ? v[j] * scale : 0.f;  // beyond R: zero rows of A, but x may be infinite
        if (a.kept && c + j < a.R) a.kept[(size_t)(row0 + t) * a.R + c + j] = v[j];
      }
      if (a.parts) ad_put_parts(a.parts + (size_t)(row0 + t) * 3 * g.Rk, g.Rk, c, v);
      if (!a.out) continue;
      uint4 o[kAtParts];
      ad_split8(v, o);
#pragma unroll
      for (int s = 0; s < kAtParts; ++s) *reinterpret_cast<uint4*>(sm + v_at(t, s * g8 + c / 8)) = o[s];
    }
    at_fence_async();
    named_sync(1, 128);
    if (a.out && warp == 2) {
      // this CTA's rows to the other CTAs: rows are 128 bytes, one behind the other
      for (int i = lane; i < atoms * C && mine > 0; i += 32)
        if (i % C != rank) {
          const uint32_t from = smem_u32(sm) + (uint32_t)(i / C * kAtXBytes + rank * per * 128);
          at_send(mapa_shared(from, i % C), from, mine * 128, mapa_shared(smem_u32(vfull), i % C));
        }
      if (lane == 0) mbar_arrive(vfull);
      __syncwarp();
    }
    if (a.parts)
      for (int i = threadIdx.x - 64; i < mine * g8; i += 128) {
        const int c = (i % g8) * 8, t = row0 + rank * per + i / g8;
        float v[8];
        ad_load8(a.fwd + (size_t)t * a.R, a.R, c, v);
        ad_put_parts(a.parts + ((size_t)a.T + t) * 3 * g.Rk, g.Rk, c, v);
      }
    if (a.out && copies > 1) {
      wait(vfull, 0);
      for (int i = threadIdx.x - 64; i < rows * kAtParts * g8; i += 128) {
        const uint32_t at = v_at(i / (kAtParts * g8), i % (kAtParts * g8));
        const uint4 v = *reinterpret_cast<const uint4*>(sm + at);
        for (int n = 1; n < copies; ++n) *reinterpret_cast<uint4*>(sm + at + n * g.tile * 128) = v;
      }
      at_fence_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(vrep);
    }
    at_cluster_arrive();
  }
  // (a CTA goes when all have their v: until then its shared memory is read)
  // ---- the second product
  if (warp == 0) {
    at_cluster_arrive();
    while (loaded2 < nt && !dead) {
      wait(&empty2[loaded2 % kAtStages2], (loaded2 / kAtStages2 - 1) & 1);
      if (!dead) load2();
    }
    // after a timeout every copy lands before the CTA may go
    if (dead || *abort_flag) {
      for (int j = max(0, loaded1 - g.stages1); j < loaded1; ++j) mbar_wait(&full1[j % g.stages1], (j / g.stages1) & 1);
      for (int j = max(0, loaded2 - kAtStages2); j < loaded2; ++j) mbar_wait(&full2[j % kAtStages2], (j / kAtStages2) & 1);
    }
    __syncwarp();
  } else if (warp == 1) {
    if (a.out) {
      wait(vfull, 0);
      if (copies > 1) wait(vrep, 0);
      at_fence_async();
    }
    at_cluster_arrive();
    const uint32_t idesc = idesc_bf16(kAtRows, kAtCols, 0, 1);
    const uint64_t a0 = at_desc(smem_u32(sm), 16, 1024), b0 = at_desc(smem_u32(ring2), g.Rk * 128, 1024);
    for (int i = 0; i < nt; ++i) {
      const int s = i % kAtStages2, b = i & 1;
      wait(&full2[s], (i / kAtStages2) & 1);
      if (i >= 2) wait(&tempty[b], (i / 2 - 1) & 1);
      tc_fence_after();
      if (lead && !dead) {
        uint64_t bd = b0 + (uint64_t)(s * (stage2 >> 4));
        int r = 0;  // 16 ranks of B at a time, three times over
        for (int k = 0; k < kAtParts * g.Rk; k += 16) {
          umma_f16(tmem + b * kAtCols, a0 + (uint64_t)((k / 64) * (kAtXBytes >> 4) + (k % 64) / 8), bd, idesc, k != 0);
          r += 16;
          bd += 2048 >> 4;
          if (r == g.Rk) r = 0, bd = b0 + (uint64_t)(s * (stage2 >> 4));
        }
      }
      if (lead) {
        umma_commit(&empty2[s]);
        umma_commit(&tfull[b]);
      }
      __syncwarp();
    }
    if (lead) umma_commit(done);
    __syncwarp();
    mbar_wait(done, 0);  // also after a timeout: nothing of this CTA is read or written any more
  } else {
    constexpr int kChunk = F32 ? 32 : 64, kPer = kAtCols / kChunk;  // outputs of a chunk (128 bytes); chunks of a step
    unsigned char* buf = part + (warp - 2) * 2 * kAtStage;
    const int nch = nt * kPer;              // this warp's chunks: copy, copy + copies, ...
    const int pr = lane >> 3, pc = lane & 7;  // of a 4-row copy: row, 16-byte piece
    const int r0 = q * 32 % g.tile;         // first row of this warp
    const int have = min(32, rows - r0);    // (none: it waits and arrives only)
    auto col = [&](int ch) { return (nt0 + ch / kPer) * kAtCols + ch % kPer * kChunk; };
    int slot = 0;
    auto fetch = [&](int ch, int to) {
      if (ch < nch && a.base) {
        const int n = col(ch) + pc * (16 / kSize);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int r = i * 4 + pr;
          if (r < have && n < a.N)
            at_copy16(buf + to * kAtStage + r * 128 + ((pc ^ (r & 7)) * 16),
                      reinterpret_cast<const uint8_t*>(a.base) + ((row0 + r0 + r) * a.ldb + n) * kSize);
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    fetch(copy, 0);
    for (int i = 0; i < nt; ++i) {
      const int b = i & 1;
      const int c0 = i * kPer, from = c0 + (copy - c0 % copies + copies) % copies;  // the step's first chunk of this warp
      bool waited = false;
      for (int ch = from; ch < c0 + kPer; ch += copies) {
        fetch(ch + copies, slot ^ 1);
        if (!waited) {
          wait(&tfull[b], (i / 2) & 1);
          tc_fence_after();
          waited = true;
        }
        float v[kChunk];
        const uint32_t at = tmem + lanes + b * kAtCols + ch % kPer * kChunk;
#pragma unroll
        for (int j = 0; j < kChunk; j += 32) tmem_ld32(at + j, *reinterpret_cast<float(*)[32]>(v + j));
        tmem_ld_wait();
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        __syncwarp();
        unsigned char* st = buf + slot * kAtStage;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          uint4* p = reinterpret_cast<uint4*>(st + lane * 128 + ((j ^ (lane & 7)) * 16));
          uint4 x = make_uint4(0, 0, 0, 0);
          if (a.base) x = *p;
          uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (F32) {
              u[k] = __float_as_uint(__uint_as_float(u[k]) + v[j * 4 + k]);
            } else {
              const __nv_bfloat162 z = __floats2bfloat162_rn(bf16_lo(u[k]) + v[(j * 8 + 2 * k) % kChunk],
                                                             bf16_hi(u[k]) + v[(j * 8 + 2 * k + 1) % kChunk]);
              u[k] = *reinterpret_cast<const uint32_t*>(&z);
            }
          }
          *p = make_uint4(u[0], u[1], u[2], u[3]);
        }
        __syncwarp();
        const int n = col(ch) + pc * (16 / kSize);
        const bool store = n < a.N && !dead;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int r = k * 4 + pr;
          if (store && r < have)
            *reinterpret_cast<uint4*>(reinterpret_cast<uint8_t*>(a.out) + ((row0 + r0 + r) * a.ldo + n) * kSize) =
                *reinterpret_cast<const uint4*>(st + r * 128 + ((pc ^ (r & 7)) * 16));
        }
        __syncwarp();
        slot ^= 1;
      }
      if (!waited) {  // nothing of this step: in step with the others all the same
        wait(&tfull[b], (i / 2) & 1);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&tempty[b]);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    tc_fence_before();
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, g.tmem);
    __syncwarp();
  }
  at_cluster_wait();
  if (g.beside) pdl_wait();
}

template <bool F32, int C, bool DRAINS>
static int at_launch_as(const AdArgs& a, const AtGeo& g, int bytes, const CUtensorMap& mx, const CUtensorMap& ma,
                     const CUtensorMap& mb, cudaStream_t s) {
  long long tiles = a.T / g.tile + a.n_seq + 2ll;
  if (at_few(a)) tiles = std::min<long long>(tiles, a.T);
  if (tiles * C > 0x7fffffffll) return MOE_ERR_ARG;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = C;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(tiles * C));
  cfg.blockDim = dim3(kAtThreads);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = s;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  static bool done[64] = {};
  constexpr int kMost = 227 * 1024 - 512;
  if (bytes > kMost) return MOE_ERR_ARG;
  MOE_CUDA_TRY(ensure_smem(adapters_tile_kernel<F32, C, DRAINS>, kMost, done));
  MOE_CUDA_TRY(cudaLaunchKernelEx(&cfg, adapters_tile_kernel<F32, C, DRAINS>, a, g, mx, ma, mb));
  return MOE_OK;
}

template <bool F32, int C>
static int at_launch(const AdArgs& a, const AtGeo& g, int bytes, const CUtensorMap& mx, const CUtensorMap& ma,
                     const CUtensorMap& mb, cudaStream_t s) {
  return a.K > 64 * C * kAtDrain * kAtAcc ? at_launch_as<F32, C, true>(a, g, bytes, mx, ma, mb, s)
                                          : at_launch_as<F32, C, false>(a, g, bytes, mx, ma, mb, s);
}

int ad_launch_tiles(const AdArgs& a, bool f32, int short_rows, bool beside, cudaStream_t s) {
  AtGeo g = {};
  g.Rk = (a.R + 15) / 16 * 16;
  // CTAs of a cluster and rows of a tile, by an estimate of the time: rounds of as many clusters as run at once, in each a
  // CTA takes 9 us and its share of the tile's bytes at 40 KB/us, less where the CTAs' sum would pass 6.6 MB/us.
  // Measured: 4096 rows of R 64 (2048 x 4096) 27.3 us with 8 and 128, 28.8 with 4 and 64, 31.9 with 4 and 128; 12,000 rows
  // 67 with 2 and 128, 76 with 4 or 8; 16,384 of R 16 (2048 x 2048) 56 with 8 and 128, 45 with 4, 41 with 2; 1024 of R 16
  // 11.0 with 8 and 128, 10.3 with 8 and 64, 10.9 with 8 and 32; 2000 of R 128 (4096 x 4096) 30 with 4 and 64, 35 with 4 and
  // 128, 46 with 8 and 128.
  int C = 8;
  double best = 0.;
  for (int c = 2; c <= 8; c *= 2)
    for (int tile = 32; tile <= kAtRows; tile *= 2) {
      if (g.Rk > 64 && f32 && tile > 64) continue;
      const double bytes = (tile * (2. * a.K + (f32 ? 4. : 2.) * (a.base ? 2 : 1) * (a.out ? a.N : 0)) + 2. * a.R * ((double)a.K + a.N)) / c;
      const int most = g.Rk > 64 ? (c == 8 ? 15 : c == 4 ? 36 : 76) : (c == 8 ? 35 : c == 4 ? 75 : 152);
      const long long n = (a.T + tile - 1) / tile + a.n_seq / 2;
      auto round = [&](long long clusters) { return 9. + bytes / std::min(40e3, 6.6e6 / ((double)clusters * c)); };
      const double t = (double)(n / most) * round(most) + (n % most ? round(n % most) : 0.);
      if (best == 0. || t < best) best = t, C = c, g.tile = tile;
    }
  g.short_rows = short_rows;
  g.beside = beside;
  g.tmem = g.Rk <= 64 ? 256 : 512;  // (above 64 ranks a CTA has its SM for itself)
  const int stage1 = kAtXBytes + g.Rk * 128;
  // two CTAs a SM up to 64 ranks
  g.stages1 = g.Rk <= 16 ? 4 : g.Rk <= 32 ? 3 : g.Rk <= 64 ? 2 : 3;
  const int ring1 = std::max(g.stages1 * stage1, (kAtParts * g.Rk + 63) / 64 * kAtXBytes);
  g.off2 = ring1;
  g.off_part = g.off2 + kAtStages2 * g.Rk * 256;
  g.off_bar = g.off_part + std::max(8 * kAtStage, g.tile * g.Rk * 4);
  const int bytes = g.off_bar + 512;
  CUtensorMap mx, ma, mb;
  {
    const uint64_t dims[3] = {(uint64_t)a.K, (uint64_t)a.T, 1}, st[2] = {(uint64_t)a.ldx * 2, (uint64_t)a.ldx * 2};
    const uint32_t box[3] = {64, (uint32_t)g.tile, 1};
    if (int rc = encode_tmap_3d_bf16(&mx, a.x, dims, st, box, CU_TENSOR_MAP_SWIZZLE_128B)) return rc;
  }
  for (int w = 0; w < 2; ++w) {
    const uint64_t F = w ? a.N : a.K;
    const uint64_t dims[3] = {F, (uint64_t)a.R, (uint64_t)a.L}, st[2] = {F * 2, F * 2 * a.R};
    const uint32_t box[3] = {64, (uint32_t)g.Rk, 1};
    if (int rc = encode_tmap_3d_bf16(w ? &mb : &ma, w ? a.w2 : a.w1, dims, st, box, CU_TENSOR_MAP_SWIZZLE_128B)) return rc;
  }
  if (C == 8) return f32 ? at_launch<true, 8>(a, g, bytes, mx, ma, mb, s) : at_launch<false, 8>(a, g, bytes, mx, ma, mb, s);
  if (C == 2) return f32 ? at_launch<true, 2>(a, g, bytes, mx, ma, mb, s) : at_launch<false, 2>(a, g, bytes, mx, ma, mb, s);
  return f32 ? at_launch<true, 4>(a, g, bytes, mx, ma, mb, s) : at_launch<false, 4>(a, g, bytes, mx, ma, mb, s);
}

}  // namespace moe
