// Adapters of longer sequences on the tcgen05 tensor cores: out = base + (scale_l x A_l^T) B_l in one launch.
//
// A cluster of C CTAs has a tile of up to 128 rows of one sequence.  CTA c multiplies its share of the K inputs by all R
// ranks (D1 [rows][R] in TMEM: x by TMA, K-major; A_l K-major); the shares meet in distributed shared memory, where each
// CTA adds up some of the rows in a fixed order, scales them and hands them to all; then CTA c multiplies them by its
// share of the N outputs (D2 [rows][128], double-buffered; B_l as it lies, MN-major) and adds base on the way out.
// Nothing but x, A, B, base and out crosses the memory, so those bytes bound it.
//
// v = scale x A^T enters the second product as a sum of two (bf16 results) or three (fp32 results) bf16 numbers: 16 or
// 24 significant bits.  The products cost little beside the bytes: 2 R flops a byte of x.
#include <algorithm>

#include "adapters.cuh"
#include "tc05.cuh"

namespace moe {

constexpr int kAtThreads = 192;  // TMA warp, MMA warp, four epilogue warps
constexpr int kAtRows = 128;     // rows of a tile, at most (MMA M)
constexpr int kAtCols = 128;     // outputs of a step of the second product
constexpr uint32_t kAtTmem = 256;
constexpr int kAtXBytes = kAtRows * 128;  // 64 inputs of a tile's rows
constexpr int kAtStage = 4096;            // 32 rows x 128 bytes of results
constexpr int kAtStages2 = 2;

struct AtGeo {
  int C, tile, Rk, stages1;     // CTAs, rows of a tile, R in sixteens, slots of the first ring
  int off2, off_part, off_bar;  // second ring, partial sums / staging, barriers
  int short_rows;               // sequences of up to so many rows are the row kernel's
};

__device__ __forceinline__ uint64_t at_desc(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
  return smem_desc_l(saddr, lbo, sbo, kLayoutSw128);
}
__device__ __forceinline__ void at_fence_async() { asm volatile("fence.proxy.async;" ::: "memory"); }
__device__ __forceinline__ void at_store4(uint32_t caddr, float a, float b, float c, float d) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(caddr), "f"(a), "f"(b), "f"(c), "f"(d) : "memory");
}
__device__ __forceinline__ void at_store16(uint32_t caddr, uint4 v) {
  asm volatile("st.shared::cluster.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(caddr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
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

// Tile `ti` of the batch: its first row, rows and adapter; rows 0: there is no such tile.
__device__ void at_find(const AdArgs& a, const AtGeo& g, int ti, int* tmp, int* tile) {
  const bool copies = a.kept || (a.out && (a.out != a.base || a.ldo != a.ldb));
  int before = 0;
  if (threadIdx.x == 0) tile[1] = 0;
  for (int j0 = 0; j0 < a.n_seq + 2; j0 += kAtThreads) {
    const int j = j0 + (int)threadIdx.x;
    int t0 = 0, t1 = 0, l = -1, n = 0;
    if (j < a.n_seq + 2) {
      at_segment(a, j, t0, t1);
      const bool seq = j >= 1 && j <= a.n_seq;
      if (seq) {
        l = ad_adapter(a, j - 1);
        if (a.seq[j] < a.seq[j - 1]) set_status(a.status, MOE_DEV_BAD_GROUPS);
      }
      n = max(t1 - t0, 0);
      if ((seq && n <= g.short_rows) || (l < 0 && !copies)) n = 0;
      n = (n + g.tile - 1) / g.tile;
    }
    int total;
    const int at = before + block_exclusive_scan(n, tmp, &total);
    if (ti >= at && ti < at + n) {
      tile[0] = t0 + (ti - at) * g.tile;
      tile[1] = min(g.tile, t1 - tile[0]);
      tile[2] = l;
    }
    before += total;
    if (ti < before) break;
  }
  __syncthreads();
}

template <bool F32>
__global__ void __launch_bounds__(kAtThreads, 1)
    adapters_tile_kernel(const AdArgs a, const AtGeo g, const __grid_constant__ CUtensorMap mapX,
                         const __grid_constant__ CUtensorMap mapA, const __grid_constant__ CUtensorMap mapB) {
  constexpr int NS = F32 ? 3 : 2;
  extern __shared__ __align__(16) unsigned char at_raw[];
  unsigned char* sm = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(at_raw) + 1023) & ~uintptr_t(1023));
  __shared__ int s_tile[3], s_scan[33], s_abort;
  __shared__ uint32_t s_tmem;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_rank(), C = g.C;
  pdl_wait();
  at_find(a, g, (int)cluster_index(), s_scan, s_tile);
  const int row0 = s_tile[0], rows = s_tile[1], l = s_tile[2];
  if (rows == 0) return;  // (the whole cluster)
  const int NT = (a.N + kAtCols - 1) / kAtCols, nt0 = NT * rank / C, nt1 = NT * (rank + 1) / C;
  constexpr int kSize = F32 ? 4 : 2;
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
  uint64_t* full1 = reinterpret_cast<uint64_t*>(sm + g.off_bar);
  uint64_t* empty1 = full1 + 8;
  uint64_t* full2 = empty1 + 8;
  uint64_t* empty2 = full2 + kAtStages2;
  uint64_t* tfull = empty2 + kAtStages2;
  uint64_t* tempty = tfull + 2;
  uint64_t* d1full = tempty + 2;
  unsigned char* ring2 = sm + g.off2;
  unsigned char* part = sm + g.off_part;
  const int stage1 = kAtXBytes + g.Rk * 128, stage2 = g.Rk * 256;
  if (threadIdx.x == 0) {
    for (int i = 0; i < g.stages1; ++i) mbar_init(&full1[i], 1), mbar_init(&empty1[i], 1);
    for (int i = 0; i < kAtStages2; ++i) mbar_init(&full2[i], 1), mbar_init(&empty2[i], 1);
    for (int i = 0; i < 2; ++i) mbar_init(&tfull[i], 1), mbar_init(&tempty[i], 4);
    mbar_init(d1full, 1);
    s_abort = 0;
    mbar_fence_init();
  }
  if (warp == 1) {
    tmem_alloc(&s_tmem, kAtTmem);
    tmem_relinquish();
  }
  __syncthreads();
  tc_fence_before();
  cluster_sync();  // every CTA of the cluster has started: its shared memory may be written
  tc_fence_after();
  const uint32_t tmem = s_tmem, d1 = tmem + 128;
  volatile int* abort_flag = &s_abort;
  auto give_up = [&] {
    *abort_flag = 1;
    set_status(a.status, MOE_DEV_TIMEOUT);
  };
  auto wait = [&](uint64_t* bar, uint32_t parity) {  // bounded; nothing is waited for after a timeout
    if (!*abort_flag && !mbar_wait(bar, parity)) give_up();
  };
  const int kc = (a.K + 63) / 64, kc0 = kc * rank / C, kc1 = kc * (rank + 1) / C, nk = kc1 - kc0;
  const int boxes = (rows + 31) / 32;
  const int nt = a.out ? nt1 - nt0 : 0;
  int loaded2 = 0;
  auto load2 = [&](int i) {  // step i of the second product
    unsigned char* st = ring2 + (i % kAtStages2) * stage2;
    uint64_t* bar = &full2[i % kAtStages2];
    mbar_expect_tx(bar, (uint32_t)stage2);
    tma_load_3d(st, &mapB, bar, (nt0 + i) * kAtCols, 0, l);
    tma_load_3d(st + g.Rk * 128, &mapB, bar, (nt0 + i) * kAtCols + 64, 0, l);
  };
  // ---- the first product
  if (warp == 0) {
    if (lane == 0) {
      for (int i = 0; i < nk && !*abort_flag; ++i) {
        const int s = i % g.stages1, use = i / g.stages1;
        if (use > 0) wait(&empty1[s], (use - 1) & 1);
        if (*abort_flag) break;
        unsigned char* st = sm + s * stage1;
        mbar_expect_tx(&full1[s], (uint32_t)(boxes * 4096 + g.Rk * 128));
        for (int b = 0; b < boxes; ++b) tma_load_3d(st + b * 4096, &mapX, &full1[s], (kc0 + i) * 64, row0 + 32 * b, 0);
        tma_load_3d(st + kAtXBytes, &mapA, &full1[s], (kc0 + i) * 64, 0, l);
      }
      for (; loaded2 < min(nt, kAtStages2) && !*abort_flag; ++loaded2) load2(loaded2);
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0 && nk > 0) {
      const uint32_t idesc = idesc_bf16(kAtRows, g.Rk, 0, 0);
      const uint32_t base = smem_u32(sm);
      for (int i = 0; i < nk; ++i) {
        const int s = i % g.stages1, use = i / g.stages1;
        wait(&full1[s], use & 1);
        tc_fence_after();
        if (!*abort_flag) {
          const uint64_t ad = at_desc(base + s * stage1, 16, 1024), bd = at_desc(base + s * stage1 + kAtXBytes, 16, 1024);
#pragma unroll
          for (int q = 0; q < 4; ++q) umma_f16(d1, ad + 2 * q, bd + 2 * q, idesc, i + q != 0);
        }
        umma_commit(&empty1[s]);
      }
      umma_commit(d1full);
    }
    __syncwarp();
  }
  const int per = g.tile / C;            // rows that a CTA adds up
  const int pitch = g.Rk + 4;            // floats of a row of partial sums
  const int q = warp & 3, row = q * 32 + lane;
  if (warp >= 2) {
    if (nk > 0) {
      wait(d1full, 0);
      __syncwarp();
      tc_fence_after();
    }
    const uint32_t dst = mapa_shared(smem_u32(part), (uint32_t)min(row / per, C - 1)) +
                         (uint32_t)((rank * per + row % per) * pitch) * 4;
    for (int c = 0; c < g.Rk; c += 16) {
      float v[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = 0.f;
      if (nk > 0) {
        tmem_ld_w<16>(d1 + ((uint32_t)(q * 32) << 16) + c, v);
        tmem_ld_wait();
      }
      if (row < rows) {
#pragma unroll
        for (int i = 0; i < 16; i += 4) at_store4(dst + (c + i) * 4, v[i], v[i + 1], v[i + 2], v[i + 3]);
      }
    }
    tc_fence_before();
  }
  cluster_sync();  // partial sums are there; the first ring is free in every CTA (its products are done)
  if (warp >= 2) {
    const float scale = a.scale[l];
    const int g8 = g.Rk / 8, mine = max(0, min(per, rows - rank * per));
    for (int i = threadIdx.x - 64; i < mine * g8; i += 128) {
      const int r = i / g8, c = (i % g8) * 8, t = rank * per + r;
      float v[8] = {};
      for (int p = 0; p < C; ++p) {
        const float4* src = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(part) + (p * per + r) * pitch + c);
        const float4 x = src[0], y = src[1];
        v[0] += x.x, v[1] += x.y, v[2] += x.z, v[3] += x.w, v[4] += y.x, v[5] += y.y, v[6] += y.z, v[7] += y.w;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[j] = c + j < a.R ? v[j] * scale : 0.f;  // beyond R: zero rows of A, but x may be infinite
        if (a.kept && c + j < a.R) a.kept[(size_t)(row0 + t) * a.R + c + j] = v[j];
      }
      uint4 o[NS];
      ad_split8<NS>(v, o);
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        const int k = s * g.Rk + c;
        const uint32_t off = smem_u32(sm) + (uint32_t)((k / 64) * kAtXBytes + t * 128 + (((k % 64) / 8) ^ (t & 7)) * 16);
        for (int p = 0; p < C; ++p) at_store16(mapa_shared(off, p), o[s]);
      }
    }
    at_fence_async();
  }
  cluster_sync();  // v of all rows is there
  // ---- the second product
  if (warp == 0) {
    if (lane == 0) {
      for (; loaded2 < nt && !*abort_flag; ++loaded2) {
        wait(&empty2[loaded2 % kAtStages2], (loaded2 / kAtStages2 - 1) & 1);
        if (*abort_flag) break;
        load2(loaded2);
      }
      // after a timeout every copy lands before the CTA may go
      if (*abort_flag) {
        for (int s = 0; s < g.stages1 && s < nk; ++s) mbar_wait(&full1[s], ((nk - 1 - s) / g.stages1) & 1);
        for (int s = 0; s < kAtStages2 && s < loaded2; ++s) mbar_wait(&full2[s], ((loaded2 - 1 - s) / kAtStages2) & 1);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0 && nt > 0) {
      at_fence_async();
      const uint32_t idesc = idesc_bf16(kAtRows, kAtCols, 0, 1);
      const uint32_t base = smem_u32(sm);
      for (int i = 0; i < nt; ++i) {
        const int s = i % kAtStages2, b = i & 1;
        wait(&full2[s], (i / kAtStages2) & 1);
        if (i >= 2) wait(&tempty[b], (i / 2 - 1) & 1);
        tc_fence_after();
        if (!*abort_flag) {
          const uint64_t bd = at_desc(smem_u32(ring2) + s * stage2, g.Rk * 128, 1024);
          for (int k = 0; k < NS * g.Rk; k += 16) {
            const uint64_t ad = at_desc(base + (k / 64) * kAtXBytes + (k % 64) * 2, 16, 1024);
            umma_f16(tmem + b * kAtCols, ad, bd + (uint64_t)(k % g.Rk / 16) * (2048 >> 4), idesc, k != 0);
          }
        }
        umma_commit(&empty2[s]);
        umma_commit(&tfull[b]);
      }
    }
    __syncwarp();
  } else {
    constexpr int kChunk = F32 ? 32 : 64, kPer = kAtCols / kChunk;  // outputs of a chunk (128 bytes); chunks of a step
    unsigned char* buf = part + (warp - 2) * 2 * kAtStage;
    const int nch = nt * kPer;
    const int pr = lane >> 3, pc = lane & 7;  // of a 4-row copy: row, 16-byte piece
    auto col = [&](int ch) { return (nt0 + ch / kPer) * kAtCols + ch % kPer * kChunk; };
    auto fetch = [&](int ch) {
      if (ch < nch && a.base) {
        const int n = col(ch) + pc * (16 / kSize);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int r = i * 4 + pr;
          if (q * 32 + r < rows && n < a.N)
            at_copy16(buf + (ch & 1) * kAtStage + r * 128 + ((pc ^ (r & 7)) * 16),
                      reinterpret_cast<const uint8_t*>(a.base) + ((row0 + q * 32 + r) * a.ldb + n) * kSize);
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    fetch(0);
    for (int ch = 0; ch < nch; ++ch) {
      const int i = ch / kPer, b = i & 1;
      fetch(ch + 1);
      if (ch % kPer == 0) {
        wait(&tfull[b], (i / 2) & 1);
        __syncwarp();
        tc_fence_after();
      }
      float v[kChunk];
      const uint32_t at = tmem + ((uint32_t)(q * 32) << 16) + b * kAtCols + ch % kPer * kChunk;
#pragma unroll
      for (int j = 0; j < kChunk; j += 32) tmem_ld32(at + j, *reinterpret_cast<float(*)[32]>(v + j));
      tmem_ld_wait();
      if (ch % kPer == kPer - 1) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&tempty[b]);
      }
      asm volatile("cp.async.wait_group 1;" ::: "memory");
      __syncwarp();
      unsigned char* st = buf + (ch & 1) * kAtStage;
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
            const __nv_bfloat162 z = __floats2bfloat162_rn(bf16_lo(u[k]) + v[(j * 8 + 2 * k) % kChunk], bf16_hi(u[k]) + v[(j * 8 + 2 * k + 1) % kChunk]);
            u[k] = *reinterpret_cast<const uint32_t*>(&z);
          }
        }
        *p = make_uint4(u[0], u[1], u[2], u[3]);
      }
      __syncwarp();
      const int n = col(ch) + pc * (16 / kSize);
      const bool store = n < a.N && !*abort_flag;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int r = k * 4 + pr;
        if (store && q * 32 + r < rows)
          *reinterpret_cast<uint4*>(reinterpret_cast<uint8_t*>(a.out) + ((row0 + q * 32 + r) * a.ldo + n) * kSize) =
              *reinterpret_cast<const uint4*>(st + r * 128 + ((pc ^ (r & 7)) * 16));
      }
      __syncwarp();
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    tc_fence_before();
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kAtTmem);
  }
}

int ad_launch_tiles(const AdArgs& a, bool f32, int short_rows, cudaStream_t s) {
  AtGeo g = {};
  const int NS = f32 ? 3 : 2;
  g.Rk = (a.R + 15) / 16 * 16;
  g.C = 4;
  g.tile = g.Rk > 64 ? 64 : kAtRows;  // (the partial sums of 128 rows of more ranks do not fit beside the rings)
  g.short_rows = short_rows;
  const int stage1 = kAtXBytes + g.Rk * 128;
  g.stages1 = g.Rk > 64 ? 3 : 4;
  const int ring1 = std::max(g.stages1 * stage1, (NS * g.Rk + 63) / 64 * kAtXBytes);
  g.off2 = ring1;
  g.off_part = g.off2 + kAtStages2 * g.Rk * 256;
  g.off_bar = g.off_part + std::max(8 * kAtStage, (g.tile * (g.Rk + 4) * 4 + 1023) / 1024 * 1024);
  const int bytes = g.off_bar + 256 + 1024;
  CUtensorMap mx, ma, mb;
  {
    const uint64_t dims[3] = {(uint64_t)a.K, (uint64_t)a.T, 1}, st[2] = {(uint64_t)a.ldx * 2, (uint64_t)a.ldx * 2};
    const uint32_t box[3] = {64, 32, 1};
    if (int rc = encode_tmap_3d_bf16(&mx, a.x, dims, st, box, CU_TENSOR_MAP_SWIZZLE_128B)) return rc;
  }
  for (int w = 0; w < 2; ++w) {
    const uint64_t F = w ? a.N : a.K;
    const uint64_t dims[3] = {F, (uint64_t)a.R, (uint64_t)a.L}, st[2] = {F * 2, F * 2 * a.R};
    const uint32_t box[3] = {64, (uint32_t)g.Rk, 1};
    if (int rc = encode_tmap_3d_bf16(w ? &mb : &ma, w ? a.w2 : a.w1, dims, st, box, CU_TENSOR_MAP_SWIZZLE_128B)) return rc;
  }
  const long long tiles = std::min<long long>(a.T, a.T / g.tile + a.n_seq + 2ll);
  if (tiles * g.C > 0x7fffffffll) return MOE_ERR_ARG;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = g.C;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(tiles * g.C));
  cfg.blockDim = dim3(kAtThreads);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = s;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  static bool d0[64] = {}, d1[64] = {};
  constexpr int kMost = 227 * 1024 - 512;
  if (bytes > kMost) return MOE_ERR_ARG;
  if (f32) {
    MOE_CUDA_TRY(ensure_smem(adapters_tile_kernel<true>, kMost, d1));
    MOE_CUDA_TRY(cudaLaunchKernelEx(&cfg, adapters_tile_kernel<true>, a, g, mx, ma, mb));
  } else {
    MOE_CUDA_TRY(ensure_smem(adapters_tile_kernel<false>, kMost, d0));
    MOE_CUDA_TRY(cudaLaunchKernelEx(&cfg, adapters_tile_kernel<false>, a, g, mx, ma, mb));
  }
  return MOE_OK;
}

}  // namespace moe
