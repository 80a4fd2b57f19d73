// 4-bit products of many rows on the tcgen05 tensor cores: the linear layer, and the grouped gate / up
// and down products of the expert FFN.
//
// Computed transposed, D^T = W^T X^T: a CTA's tile is two blocks of 128 output features (gate and up of
// the same features, or 256 consecutive ones) x up to 128 rows.  The weights are the A operand and come
// from TMEM: worker threads own one feature each, turn its 64 codes of a stage into fp16 with one fused
// multiply-add per pair and write them to TMEM, so the weights cross shared memory only once, as 4-bit
// codes.  The rows are the B operand, fp16 in shared memory (TMA, 128-byte swizzle).
//
// fp16, not bf16: (code - 8) * scale has up to 11 significant bits, exact in fp16.  The ranges are kept
// by powers of two: scales are stored relative to their column's largest (w4.cuh), each row of x is
// scaled so that its largest element is in [2^14, 2^15), h by the bound |h| <= |x|^2 |Wg| |Wu| (column
// 2-norms), y by the bound that follows.  A value keeps all 11 bits while it is above 2^-29 of its row's
// bound; typical values are 2^-11 (h) and 2^-16 (y) of it.  So x (8 bits) is exact and only h and, on its
// way to the combine, y are rounded, to 11 bits.
//
// Warps: 0 TMA producer, 1 TMEM allocation and MMA issue (one thread), 2-17 workers (two sets that
// dequantise 128 inputs in turn; all drain the accumulators).  TMEM: 2 x 128 accumulator columns, 4 weight stages of 2 x 32 columns.
#include <limits.h>

#include <algorithm>

#include "internal.cuh"
#include "tc05.cuh"
#include "w4.cuh"

namespace moe {

constexpr int kGM = 128;       // features per accumulator
constexpr int kGN = 128;       // rows per tile
constexpr int kGK = 64;        // inputs per stage
constexpr int kGXRing = 5;     // stages of rows in shared memory
constexpr int kGChunk = 4;     // stages of codes that are copied together
constexpr int kGWRing = 2;     // chunks of codes in shared memory
constexpr int kGVisit = 2;     // stages that a worker dequantises at a time
constexpr int kGSet = 8;       // worker warps of a visit
constexpr int kGWorkers = 16;  // worker warps: two sets, taking visits in turn, each with its TMEM columns
constexpr int kGThreads = 64 + 32 * kGWorkers;
constexpr int kGXBytes = kGN * kGK * 2;
constexpr int kGCodeBlock = kGChunk * 4096;    // a chunk's codes of 128 features
constexpr int kGScaleBlock = kGChunk * 2 * 256;  // its fp16 scales (two groups a stage at most)
constexpr int kGWBytes = 2 * (kGCodeBlock + kGScaleBlock);
constexpr int kGEpiBytes = 32 * 32 * 4 + 256;  // per worker warp: staging, and its 32 rows' powers of two
static_assert(kGChunk == 2 * kGVisit, "a chunk is one visit of each set");
constexpr uint32_t kGTmemCols = 512;
constexpr uint32_t kGACol = 2 * kGN;           // first weight column

enum { kGateUp = 0, kDown = 1, kLinear = 2 };

struct W4GemmArgs {
  const uint8_t* w;        // slab pool, or the packed matrix
  size_t slab;             // bytes between slabs (0: one matrix)
  W4Dims d;
  size_t mat0, mat1;       // offsets of the two blocks' matrices (gate, up) or of the one matrix
  int K, NF;               // K of the rows; feature tiles
  int n;                   // rows
  // grouped rows
  const int32_t *offset, *list_e, *n_list, *e2s, *list_s;
  int E, S;
  int32_t* status;
  const int32_t* rexp;     // [n] the B operand's row p is 2^-rexp[p] times the true one
  const int32_t* oexp;     // [n] kGateUp: the same of h
  // outputs
  uint16_t* h;             // kGateUp: fp16 [n][N]
  uint16_t* yh;            // kDown: fp16 [n][N], 2^-(rexp + w4_y_exp) times y, or NULL
  float* y;                // kDown: fp32 [n][N]
  void* out;               // kLinear
  size_t ldo;
  int out_f32;
};

// One lane of the (converged) warp.  The loops that issue copies and MMAs are run by whole warps, so that
// their operands stay in uniform registers; only the issue itself is one lane's.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(p));
  return p != 0;
}

// D[tmem] (+)= A[tmem] x B[smem].
__device__ __forceinline__ void umma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n"
      " .reg .pred p;\n"
      " setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n"
      "}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// 2^e >= 1.001 |column|_2 of every column (0 for a matrix of zeros or a norm that is not finite).
__device__ __forceinline__ int w4_norm_exp(const uint8_t* m, const W4Dims& d) {
  const float c = *reinterpret_cast<const float*>(m + d.meta);
  return c > 0.f && c < INFINITY ? ilogbf(c) + 1 : 0;
}
// |y| <= |h|_2 |column|_2 <= sqrt(I) 2^15 2^hexp 2^norm_exp: the exponent that takes y / 2^hexp below 2^15.
__device__ __forceinline__ int w4_y_exp(const uint8_t* m, const W4Dims& d) {
  return (32 - __clz(d.K) + 1) / 2 + w4_norm_exp(m, d);
}

// 32 lanes x 32 consecutive 32-bit columns from registers.
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Instruction descriptor: fp16 A and B (both K-major), fp32 accumulation.
__device__ __forceinline__ uint32_t idesc_f16(int M, int N) {
  return (1u << 4) | (uint32_t(N >> 3) << 17) | (uint32_t(M >> 4) << 24);
}

__device__ __forceinline__ bool w4g_slot(const W4GemmArgs& a, int li, int& e, int& slot) {
  e = a.list_e[li];
  if (e < 0 || e >= a.E) return false;
  slot = a.list_s ? a.list_s[li] : a.e2s ? a.e2s[e] : e;
  return slot >= 0 && slot < a.S;
}

struct W4GTile {
  const uint8_t* base;  // the slab or matrix
  int ft, row0, ntok;
};

// Tile t: row tile t / NF (by the prefix of row tiles over the list), feature tile t % NF.
template <int kMode>
__device__ __forceinline__ W4GTile w4g_tile(const W4GemmArgs& a, const int* pre, int nl, int t) {
  W4GTile r;
  const int i = t / a.NF;
  r.ft = t - i * a.NF;
  if (kMode == kLinear) {
    r.base = a.w;
    r.row0 = i * kGN;
    r.ntok = min(kGN, a.n - r.row0);
  } else {
    int lo = 0, hi = nl;  // pre[lo] <= i < pre[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (pre[mid] <= i) lo = mid;
      else hi = mid;
    }
    int e, slot;
    w4g_slot(a, lo, e, slot);
    r.base = a.w + (size_t)slot * a.slab;
    r.row0 = a.offset[e] + (i - pre[lo]) * kGN;
    r.ntok = min(kGN, a.offset[e + 1] - r.row0);
  }
  return r;
}

// First tile of 16 columns of block b, and its matrix.
template <int kMode>
__device__ __forceinline__ int w4g_mt0(int ft, int b) {
  return kMode == kGateUp ? ft * 8 : (2 * ft + b) * 8;
}

// Eight codes of a word (w4.cuh) times their scale, fp16, inputs in order.
__device__ __forceinline__ void w4_expand(uint32_t w, __half2 s, uint32_t* o) {
  const __half2 m24s = __hmul2(s, __float2half2_rn(-24.f));
  auto top = [&](uint32_t v) {  // codes in bits 6-9: 16 + code; (16 + code) s - 24 s is exact
    v = (v & 0x03c003c0u) | 0x4c004c00u;
    const __half2 r = __hfma2(*reinterpret_cast<const __half2*>(&v), s, m24s);
    return *reinterpret_cast<const uint32_t*>(&r);
  };
  o[0] = top(w);
  // codes in bits 2-5: 256 + code; the shift is saved and one more half-precision operation spent,
  // which keeps the integer and the floating-point pipe equally busy
  const uint32_t v = (w & 0x003c003cu) | 0x5c005c00u;
  const __half2 c = __hsub2(*reinterpret_cast<const __half2*>(&v), __float2half2_rn(264.f)), p = __hmul2(c, s);
  o[1] = *reinterpret_cast<const uint32_t*>(&p);
  o[2] = top(w >> 4);
  o[3] = top(__funnelshift_r(w, w, 8));
}

__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }  // -126 <= e <= 127

// Drains 32 rows (of chunk `chunk`) x this warp's 32 features of both accumulators: to registers, the
// accumulators are handed back, then scaled, transposed through shared memory and stored.
template <int kMode, class Wait>
__device__ __forceinline__ void w4g_drain(const W4GemmArgs& a, const W4Dims& d, const W4GTile& ti, uint32_t taddr, int q,
                                          int chunk, int lane, unsigned char* stage, uint64_t* tfull,
                                          uint64_t* tempty, uint32_t tc, Wait&& wait, volatile int* abort_flag) {
  const int tok0 = 32 * chunk;
  const bool any = tok0 < ti.ntok, mine = tok0 + lane < ti.ntok;
  const size_t row0 = (size_t)ti.row0 + tok0;
  // the rows' powers of two, one lane each, for all lanes to read
  float* fac = reinterpret_cast<float*>(stage + 4096);
  if (any) {
    const float rx = mine ? pow2(a.rexp[row0 + lane]) : 0.f;
    if (kMode == kGateUp) {
      fac[2 * lane] = rx;
      fac[2 * lane + 1] = mine ? pow2(-a.oexp[row0 + lane]) : 0.f;
    } else {
      fac[lane] = kMode == kDown && a.yh ? 1.f : rx;  // scaled rows of y keep the row's own power of two apart
    }
  }
  __syncwarp();
  wait(tfull, tc & 1u);
  tc_fence_after();
  auto release = [&] {
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(tempty);
  };
  if (!any) {
    release();
    return;
  }
  const bool store = !*abort_flag;
  if (kMode == kGateUp) {
    float v0[32], v1[32];
    tmem_ld32(taddr + tok0, v0);
    tmem_ld32(taddr + kGN + tok0, v1);
    tmem_ld_wait();
    release();
    const int f0 = ti.ft * kGM + 32 * q, f = f0 + lane;
    const float* mg = reinterpret_cast<const float*>(ti.base + a.mat0 + d.mult);
    const float* mu = reinterpret_cast<const float*>(ti.base + a.mat1 + d.mult);
    const float cg = f < d.N ? mg[f] : 0.f, cu = f < d.N ? mu[f] : 0.f;
    uint16_t* st = reinterpret_cast<uint16_t*>(stage);
#pragma unroll
    for (int j = 0; j < 32; j += 2) {
      const float4 m = *reinterpret_cast<const float4*>(fac + 2 * j);  // x, 1 / h of rows j, j + 1
      const float g0 = v0[j] * cg * m.x, g1 = v0[j + 1] * cg * m.z;
      const float u0 = v1[j] * cu * m.x, u1 = v1[j + 1] * cu * m.z;
      st[j * 32 + lane] = __half_as_ushort(__float2half_rn(__fdividef(g0, 1.f + __expf(-g0)) * u0 * m.y));
      st[(j + 1) * 32 + lane] = __half_as_ushort(__float2half_rn(__fdividef(g1, 1.f + __expf(-g1)) * u1 * m.w));
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // 32 rows x 64 B: four 16-byte pieces per lane
      const int idx = i * 32 + lane, row = idx >> 2, seg = idx & 3;
      const uint4 v = *reinterpret_cast<const uint4*>(st + row * 32 + seg * 8);
      if (store && tok0 + row < ti.ntok && f0 + seg * 8 < d.N)
        *reinterpret_cast<uint4*>(a.h + (row0 + row) * d.N + f0 + seg * 8) = v;
    }
    __syncwarp();
    return;
  }
  const float* mc = reinterpret_cast<const float*>(ti.base + a.mat0 + d.mult);
#pragma unroll 1
  for (int blk = 0; blk < 2; ++blk) {
    float v[32];
    tmem_ld32(taddr + blk * kGN + tok0, v);
    tmem_ld_wait();
    if (blk == 1) release();
    const int f0 = (2 * ti.ft + blk) * kGM + 32 * q, f = f0 + lane;
    if (f0 >= d.N) continue;
    float cm = f < d.N ? mc[f] : 0.f;
    if (kMode == kDown && a.yh) cm = ldexpf(cm, -w4_y_exp(ti.base + a.mat0, d));
#pragma unroll
    for (int j = 0; j < 32; j += 4) {
      const float4 m = *reinterpret_cast<const float4*>(fac + j);
      v[j] = v[j] * cm * m.x;
      v[j + 1] = v[j + 1] * cm * m.y;
      v[j + 2] = v[j + 2] * cm * m.z;
      v[j + 3] = v[j + 3] * cm * m.w;
    }
    if (kMode == kLinear && !(a.ldo % 8 == 0 && (uintptr_t)a.out % 16 == 0 && f0 + 32 <= d.N)) {
      // unaligned or ragged rows of out: element stores, 32 consecutive features per row
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (store && tok0 + j < ti.ntok && f < d.N) {
          const size_t at = (row0 + j) * a.ldo + f;
          if (a.out_f32) reinterpret_cast<float*>(a.out)[at] = v[j];
          else reinterpret_cast<uint16_t*>(a.out)[at] = f32_to_bf16(v[j]);
        }
      continue;
    }
    const bool f32 = kMode == kLinear ? a.out_f32 != 0 : a.yh == nullptr;
    const size_t ld = kMode == kLinear ? a.ldo : (size_t)d.N;
    if (f32) {
      float* st = reinterpret_cast<float*>(stage);
      float* out = kMode == kLinear ? reinterpret_cast<float*>(a.out) : a.y;
#pragma unroll
      for (int j = 0; j < 32; ++j) st[j * 32 + lane] = v[j];
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 8; ++i) {  // 32 rows x 128 B
        const int idx = i * 32 + lane, row = idx >> 3, seg = idx & 7;
        const uint4 o = *reinterpret_cast<const uint4*>(st + row * 32 + seg * 4);
        if (store && tok0 + row < ti.ntok && f0 + seg * 4 < d.N)
          *reinterpret_cast<uint4*>(out + (row0 + row) * ld + f0 + seg * 4) = o;
      }
    } else {
      uint16_t* st = reinterpret_cast<uint16_t*>(stage);
      uint16_t* out = kMode == kLinear ? reinterpret_cast<uint16_t*>(a.out) : a.yh;
#pragma unroll
      for (int j = 0; j < 32; ++j)
        st[j * 32 + lane] = kMode == kLinear ? f32_to_bf16(v[j]) : __half_as_ushort(__float2half_rn(v[j]));
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 4; ++i) {  // 32 rows x 64 B
        const int idx = i * 32 + lane, row = idx >> 2, seg = idx & 3;
        const uint4 o = *reinterpret_cast<const uint4*>(st + row * 32 + seg * 8);
        if (store && tok0 + row < ti.ntok && f0 + seg * 8 < d.N)
          *reinterpret_cast<uint4*>(out + (row0 + row) * ld + f0 + seg * 8) = o;
      }
    }
    __syncwarp();
  }
}

template <int kMode>
__global__ void __launch_bounds__(kGThreads, 1) w4_gemm_kernel(const W4GemmArgs a, const __grid_constant__ CUtensorMap mapX) {
  extern __shared__ __align__(16) unsigned char gsm_raw[];
  unsigned char* sm =
      reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(gsm_raw) + 1023) & ~uintptr_t(1023));
  unsigned char* xs = sm;                             // [ring][16 KB]
  unsigned char* wsm = sm + kGXRing * kGXBytes;       // [ring][codes of both blocks | scales of both blocks]
  unsigned char* epi = wsm + kGWRing * kGWBytes;      // [workers][4 KB]
  uint64_t* xfull = reinterpret_cast<uint64_t*>(epi + kGWorkers * kGEpiBytes);
  uint64_t* xempty = xfull + kGXRing;
  uint64_t* wfull = xempty + kGXRing;
  uint64_t* wempty = wfull + kGWRing;
  uint64_t* afull = wempty + kGWRing;
  uint64_t* aempty = afull + 2;
  uint64_t* tfull = aempty + 2;
  uint64_t* tempty = tfull + 1;
  uint64_t* done = tempty + 1;
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  __shared__ int s_pre[kMode == kLinear ? 1 : kMaxE + 1];
  __shared__ int s_tmp[33];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const W4Dims& d = a.d;
  const int nkb = d.Kb;
  int nl = 0, total;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kGXRing; ++s) {
      mbar_init(&xfull[s], 1);
      mbar_init(&xempty[s], 1);
    }
    for (int s = 0; s < kGWRing; ++s) {
      mbar_init(&wfull[s], 1);
      mbar_init(&wempty[s], kGWorkers);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&afull[s], kGSet);
      mbar_init(&aempty[s], 1);
    }
    mbar_init(tfull, 1);
    mbar_init(tempty, kGWorkers);
    mbar_init(done, 1);
    s_abort = 0;
    mbar_fence_init();
  }
  if (warp == 1) {
    tmem_alloc(&s_tmem, kGTmemCols);
    tmem_relinquish();
  }
  if (kMode == kLinear) {
    total = (a.n + kGN - 1) / kGN * a.NF;
    __syncthreads();
  } else {
    // prefix of the listed experts' row tiles
    nl = min(*a.n_list, kMaxE);
    int carry = 0;
    for (int l0 = 0; l0 < nl; l0 += kGThreads) {
      const int li = l0 + threadIdx.x;
      int e, slot, c = 0;
      if (li < nl && w4g_slot(a, li, e, slot)) c = (max(a.offset[e + 1] - a.offset[e], 0) + kGN - 1) / kGN;
      int tot;
      const int ex = block_exclusive_scan(c, s_tmp, &tot);
      if (li < nl) s_pre[li] = carry + ex;
      carry += tot;
    }
    if (threadIdx.x == 0) s_pre[nl] = carry;
    __syncthreads();
    total = carry * a.NF;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  volatile int* abort_flag = &s_abort;
  // a wait that gives up ends the work of every role; the barriers are then no longer waited for
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (!mbar_try_wait(bar, parity) && !*abort_flag && !mbar_wait(bar, parity)) {
      *abort_flag = 1;
      set_status(a.status, MOE_DEV_TIMEOUT);
    }
  };

  if (warp == 0) {
    uint32_t xi = 0, wi = 0;  // stages of rows and chunks of codes issued
    bool dead = false;
    const bool lead = elect_one();
    for (int t = blockIdx.x; t < total && !dead; t += gridDim.x) {
      const W4GTile ti = w4g_tile<kMode>(a, s_pre, nl, t);
      const int mt0 = w4g_mt0<kMode>(ti.ft, 0), mt1 = w4g_mt0<kMode>(ti.ft, 1);
      // the tiles of 16 columns that exist, per block
      const uint32_t nm0 = min(8, d.Mt - mt0), nm1 = max(0, min(8, d.Mt - mt1));
      const uint8_t *m0 = ti.base + a.mat0, *m1 = ti.base + a.mat1;
      for (int kb = 0; kb < nkb; ++kb, ++xi) {
        if (kb % kGChunk == 0) {
          const uint32_t s = wi % kGWRing, use = wi / kGWRing, nb = min(kGChunk, nkb - kb);
          const uint32_t ng = d.G == 128 ? (nb + 1) / 2 : d.G == 64 ? nb : 2 * nb;
          const int kg = kb * kGK / d.G;
          if (use > 0) wait(&wempty[s], (use - 1) & 1u);
          dead = __any_sync(MOE_FULL_MASK, *abort_flag);
          if (dead) break;
          unsigned char* dst = wsm + s * kGWBytes;
          if (lead) {
            mbar_expect_tx(&wfull[s], (nm0 + nm1) * (512 * nb + 32 * ng));
            bulk_load(dst, m0 + w4_code_at(d, mt0, kb) * 512, nm0 * 512 * nb, &wfull[s]);
            bulk_load(dst + 2 * kGCodeBlock, m0 + d.scales + w4_scale_at(d, mt0, kg) * 32, nm0 * 32 * ng, &wfull[s]);
            if (nm1 > 0) {
              bulk_load(dst + kGCodeBlock, m1 + w4_code_at(d, mt1, kb) * 512, nm1 * 512 * nb, &wfull[s]);
              bulk_load(dst + 2 * kGCodeBlock + kGScaleBlock, m1 + d.scales + w4_scale_at(d, mt1, kg) * 32,
                        nm1 * 32 * ng, &wfull[s]);
            }
          }
          __syncwarp();
          ++wi;
        }
        const uint32_t s = xi % kGXRing, use = xi / kGXRing;
        if (use > 0) wait(&xempty[s], (use - 1) & 1u);
        dead = __any_sync(MOE_FULL_MASK, *abort_flag);
        if (dead) break;
        if (lead) {
          mbar_expect_tx(&xfull[s], kGXBytes);
          tma_load_3d(xs + s * kGXBytes, &mapX, &xfull[s], kb * kGK, ti.row0, 0);
        }
        __syncwarp();
      }
    }
    // after a timeout: let every copy land before the CTA can exit
    if (dead) {
      for (uint32_t j = xi > kGXRing ? xi - kGXRing : 0; j < xi; ++j) mbar_wait(&xfull[j % kGXRing], (j / kGXRing) & 1u);
      for (uint32_t j = wi > kGWRing ? wi - kGWRing : 0; j < wi; ++j) mbar_wait(&wfull[j % kGWRing], (j / kGWRing) & 1u);
    }
  } else if (warp == 1) {
    const uint64_t bd0 = smem_desc_l(smem_u32(xs), 16, 1024, kLayoutSw128);
    const bool lead = elect_one();
    uint32_t xi = 0, vi = 0, tc = 0;  // stages of rows, visits, tiles
    for (int t = blockIdx.x; t < total && !__any_sync(MOE_FULL_MASK, *abort_flag); t += gridDim.x, ++tc) {
      const W4GTile ti = w4g_tile<kMode>(a, s_pre, nl, t);
      const uint32_t idesc = idesc_f16(kGM, (ti.ntok + 15) & ~15);
      const bool two = kMode == kGateUp || w4g_mt0<kMode>(ti.ft, 1) < d.Mt;
      if (tc > 0) wait(tempty, (tc - 1) & 1u);
      for (int kb = 0; kb < nkb; ++vi) {
        const uint32_t as = vi & 1;
        wait(&afull[as], (vi >> 1) & 1u);
#pragma unroll
        for (int h = 0; h < kGVisit; ++h, ++kb, ++xi) {
          if (kb >= nkb) break;
          const uint32_t s = xi % kGXRing;
          wait(&xfull[s], (xi / kGXRing) & 1u);
          tc_fence_after();
          const uint32_t ac = tmem + kGACol + as * 128 + h * 32;
          const uint64_t bd = bd0 + (uint64_t)(s * (kGXBytes >> 4));
          if (lead) {
#pragma unroll
            for (int k = 0; k < 4; ++k) umma_f16_ts(tmem, ac + 8 * k, bd + 2 * k, idesc, kb > 0 || k > 0);
            if (two)
#pragma unroll
              for (int k = 0; k < 4; ++k) umma_f16_ts(tmem + kGN, ac + 64 + 8 * k, bd + 2 * k, idesc, kb > 0 || k > 0);
            umma_commit(&xempty[s]);
          }
          __syncwarp();
        }
        if (lead) umma_commit(&aempty[as]);
        __syncwarp();
      }
      if (lead) umma_commit(tfull);
      __syncwarp();
    }
    if (lead) umma_commit(done);
    __syncwarp();
    mbar_wait(done, 0);
  } else {
    // TMEM lane quarter; block and set (dequantising); 32-row chunk of the tile (draining)
    const int q = warp & 3, b = ((warp - 2) >> 2) & 1, set = (warp - 2) >> 3, chunk = (warp - 2) >> 2;
    const int r = 32 * q + lane, g = r & 7, hi = (r >> 3) & 1;
    const uint32_t lane_addr = (uint32_t)(q * 32) << 16;
    const uint32_t a_addr = tmem + lane_addr + kGACol + set * 128 + b * 64;
    unsigned char* stage = epi + (warp - 2) * kGEpiBytes;
    uint32_t vi = 0, wi = 0, tc = 0;  // visits, chunks before this tile, tiles drained
    W4GTile prev = {};
    bool pending = false;  // prev has not been drained
    for (int t = blockIdx.x;; t += gridDim.x) {
      const bool real = t < total && !__any_sync(MOE_FULL_MASK, *abort_flag);
      W4GTile ti = {};
      if (real) ti = w4g_tile<kMode>(a, s_pre, nl, t);
      const int nm = max(1, min(8, d.Mt - w4g_mt0<kMode>(ti.ft, b))), nk = real ? nkb : 0;
      // one visit of each set, the last tile's drain, the other visits
      int kb = 0;
#pragma unroll 1
      for (int phase = 0; phase < 2; ++phase) {
#pragma unroll 1
      for (const int end = phase ? nk : min(nk, 2 * kGVisit); kb < end; kb += kGVisit, ++vi) {
        // a chunk of codes holds two visits, one of each set; a tile starts a chunk of its own
        const uint32_t c = wi + kb / kGChunk, ws = c % kGWRing;
        if ((vi & 1) != (uint32_t)set) {
          if (kb % kGChunk == 0 && kb + kGVisit >= nkb) {  // a last chunk without a visit of this set
            wait(&wfull[ws], (c / kGWRing) & 1u);
            __syncwarp();
            if (lane == 0) mbar_arrive(&wempty[ws]);
          }
          continue;
        }
        wait(&wfull[ws], (c / kGWRing) & 1u);
        const unsigned char* wst = wsm + ws * kGWBytes;
        uint32_t o[32];
#pragma unroll
        for (int h = 0; h < kGVisit; ++h) {
          if (kb + h >= nkb) break;
          const int j4 = kb % kGChunk + h;
          const unsigned char* code = wst + b * kGCodeBlock + (j4 * nm + (r >> 4)) * 512 + g * 64 + hi * 8;
          const int gi = d.G == 128 ? j4 >> 1 : d.G == 64 ? j4 : 2 * j4;
          const __half* sp = reinterpret_cast<const __half*>(wst + 2 * kGCodeBlock + b * kGScaleBlock +
                                                             (gi * nm + (r >> 4)) * 32 + g * 4) + hi;
          uint2 w[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) w[j] = *reinterpret_cast<const uint2*>(code + ((j + (g >> 1)) & 3) * 16);
          const __half2 s0 = __half2half2(sp[0]), s1 = d.G == 32 ? __half2half2(sp[16 * nm]) : s0;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            w4_expand(w[j].x, s0, &o[4 * j]);
            w4_expand(w[j].y, s1, &o[16 + 4 * j]);
          }
          if (h == 0 && vi >= 2) wait(&aempty[set], ((vi >> 1) - 1) & 1u);
          tc_fence_after();
          tmem_st32(a_addr + 32 * h, o);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&afull[set]);
          mbar_arrive(&wempty[ws]);
        }
      }
      if (phase == 0 && pending) {
        w4g_drain<kMode>(a, d, prev, tmem + lane_addr, q, chunk, lane, stage, tfull, tempty, tc, wait, abort_flag);
        ++tc;
      }
      }
      if (!real) break;
      prev = ti;
      pending = true;
      wi += (nkb + kGChunk - 1) / kGChunk;
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kGTmemCols);
  }
}

// ---------------------------------------------------------------------------
// Rows: x -> fp16 times a power of two per row, in grouped order; one warp per row.
// ---------------------------------------------------------------------------
constexpr int kRowThreads = 256;
constexpr int kNoRow = INT_MIN;  // yexp of a row whose expert has no slot

struct W4RowArgs {
  const uint16_t* x;
  size_t ldx;
  int n, K;
  uint16_t* xp;            // fp16 [n][K]
  int32_t* xexp;           // [n]
  // grouped rows (list_e != NULL)
  W4GemmArgs g;
  const int32_t* rows;
  int k;
  W4Dims dn;               // the down matrix, and where it starts in a slab
  size_t mat2;
  int32_t *hexp, *yexp;    // [n]
  float* y;                // rows of experts without a slot are zeroed, or NULL (yexp says so)
};

// One row: returns its exponent and ceil(log2 |x'|^2) (x' = the scaled row).
__device__ __forceinline__ void w4_scale_row(const uint16_t* x, uint16_t* xp, int K, int lane, int& xe, int& ln) {
  float amax = 0.f;
  auto take = [&](uint32_t v) {
    const float lo = fabsf(bf16_lo(v)), hi = fabsf(bf16_hi(v));
    amax = fmaxf(amax, lo < INFINITY ? lo : 0.f);  // infinities and NaN do not set the scale
    amax = fmaxf(amax, hi < INFINITY ? hi : 0.f);
  };
  for (int c = lane; c < K / 8; c += 32) {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(x) + c);
    take(v.x), take(v.y), take(v.z), take(v.w);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(MOE_FULL_MASK, amax, o));
  xe = amax > 0.f ? max(ilogbf(amax) - 14, -126) : 0;
  const float f0 = ldexpf(1.f, -xe / 2), f1 = ldexpf(1.f, -xe - (-xe / 2));  // 2^-xe may overflow by itself
  float nrm = 0.f;
  auto conv = [&](uint32_t v) {
    const float lo = bf16_lo(v) * f0 * f1, hi = bf16_hi(v) * f0 * f1;
    nrm += fabsf(lo) < INFINITY ? lo * lo : 0.f;
    nrm += fabsf(hi) < INFINITY ? hi * hi : 0.f;
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  };
  for (int c = lane; c < K / 8; c += 32) {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(x) + c);
    reinterpret_cast<uint4*>(xp)[c] = make_uint4(conv(v.x), conv(v.y), conv(v.z), conv(v.w));
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) nrm += __shfl_xor_sync(MOE_FULL_MASK, nrm, o);
  ln = nrm > 0.f ? ilogbf(nrm * 1.001f) + 1 : 0;
}

__global__ void __launch_bounds__(kRowThreads) w4_rows_kernel(const W4RowArgs a) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = gridDim.x * (kRowThreads / 32);
  for (int p = blockIdx.x * (kRowThreads / 32) + warp; p < a.n; p += nw) {
    int xe, ln;
    w4_scale_row(a.x + (size_t)p * a.ldx, a.xp + (size_t)p * a.K, a.K, lane, xe, ln);
    if (lane == 0) a.xexp[p] = xe;
  }
}

__global__ void __launch_bounds__(kRowThreads) w4_group_rows_kernel(const W4RowArgs a) {
  __shared__ int s_pre[kMaxE + 1];
  __shared__ int s_tmp[33];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = gridDim.x * (kRowThreads / 32);
  const int nl = min(*a.g.n_list, kMaxE);
  int carry = 0;
  for (int l0 = 0; l0 < nl; l0 += kRowThreads) {
    const int li = l0 + threadIdx.x, e = li < nl ? a.g.list_e[li] : -1;
    const int c = e >= 0 && e < a.g.E ? max(a.g.offset[e + 1] - a.g.offset[e], 0) : 0;
    int tot;
    const int ex = block_exclusive_scan(c, s_tmp, &tot);
    if (li < nl) s_pre[li] = carry + ex;
    carry += tot;
  }
  if (threadIdx.x == 0) s_pre[nl] = carry;
  __syncthreads();
  for (int i = blockIdx.x * (kRowThreads / 32) + warp; i < carry; i += nw) {
    int lo = 0, hi = nl;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (s_pre[mid] <= i) lo = mid;
      else hi = mid;
    }
    int e, slot;
    const bool ok = w4g_slot(a.g, lo, e, slot);
    const int p = a.g.offset[e] + i - s_pre[lo];
    if (!ok) {
      if (lane == 0) {
        set_status(a.g.status, MOE_DEV_BAD_SLOT);
        a.yexp[p] = kNoRow;
      }
      if (a.y)
        for (int c = lane; c < a.dn.N / 4; c += 32)
          reinterpret_cast<float4*>(a.y + (size_t)p * a.dn.N)[c] = make_float4(0.f, 0.f, 0.f, 0.f);
      continue;
    }
    int xe, ln;
    w4_scale_row(a.x + (size_t)(a.rows[p] / a.k) * a.ldx, a.xp + (size_t)p * a.K, a.K, lane, xe, ln);
    if (lane == 0) {
      const uint8_t* base = a.g.w + (size_t)slot * a.g.slab;
      // |h| <= |g| |u| <= |x|^2 |Wg| |Wu|; h 2^-hexp stays below 2^15
      const int b = ln + 2 * xe + w4_norm_exp(base + a.g.mat0, a.g.d) + w4_norm_exp(base + a.g.mat1, a.g.d);
      const int he = min(max(b - 15, -126), 126);
      a.xexp[p] = xe;
      a.hexp[p] = he;
      a.yexp[p] = he + w4_y_exp(base + a.mat2, a.dn);
    }
  }
}

// out[t] = bf16(sum_j w[t][j] y[pos[t][j]]) from the scaled fp16 rows, fp32, j ascending; 8 columns a thread.
__global__ void __launch_bounds__(128) w4_combine_kernel(const uint16_t* __restrict__ yh,
                                                         const int32_t* __restrict__ yexp,
                                                         const float* __restrict__ w, const int32_t* __restrict__ pos,
                                                         int k, int H, uint16_t* __restrict__ out) {
  const int t = blockIdx.x, c = (blockIdx.y * 128 + threadIdx.x) * 8;
  if (c >= H) return;
  float acc[8] = {};
  for (int j = 0; j < k; ++j) {
    const int p = pos[(size_t)t * k + j];
    if (p < 0) continue;
    const int e = yexp[p];
    if (e == kNoRow) continue;
    const uint4 v = *reinterpret_cast<const uint4*>(yh + (size_t)p * H + c);
    const float wj = ldexpf(w[(size_t)t * k + j], e / 2), m = ldexpf(1.f, e - e / 2);  // 2^e may overflow by itself
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
      acc[2 * i] = fmaf(wj, f.x * m, acc[2 * i]);
      acc[2 * i + 1] = fmaf(wj, f.y * m, acc[2 * i + 1]);
    }
  }
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = uint32_t(f32_to_bf16(acc[2 * i])) | (uint32_t(f32_to_bf16(acc[2 * i + 1])) << 16);
  *reinterpret_cast<uint4*>(out + (size_t)t * H + c) = make_uint4(o[0], o[1], o[2], o[3]);
}

constexpr size_t kGSmem = 1024 + (size_t)kGXRing * kGXBytes + (size_t)kGWRing * kGWBytes +
                          (size_t)kGWorkers * kGEpiBytes + 64 * sizeof(uint64_t);
static_assert(kGSmem <= 222 * 1024, "shared memory of a CTA, with the 4.3 KB of static arrays");

// [n][K] 16-bit rows; a box is one stage of one row tile (128 rows x 64 inputs; what lies outside reads as 0).
static int row_map(CUtensorMap* m, const void* base, int n, int K) {
  const uint64_t d[3] = {(uint64_t)K, (uint64_t)n, 1};
  const uint64_t s[2] = {(uint64_t)K * 2, (uint64_t)n * K * 2};
  const uint32_t b[3] = {kGK, kGN, 1};
  return encode_tmap_3d_bf16(m, base, d, s, b, CU_TENSOR_MAP_SWIZZLE_128B);
}

template <int kMode>
static int launch_gemm(const W4GemmArgs& g, const void* rows, cudaStream_t s) {
  static bool done[64] = {};
  MOE_CUDA_TRY(ensure_smem(w4_gemm_kernel<kMode>, (int)kGSmem, done));
  int dev = 0, sms = 0;
  MOE_CUDA_TRY(cudaGetDevice(&dev));
  MOE_CUDA_TRY(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev));
  CUtensorMap m;
  if (row_map(&m, rows, g.n, g.K) != MOE_OK) return MOE_ERR_CUDA;
  w4_gemm_kernel<kMode><<<sms, kGThreads, kGSmem, s>>>(g, m);
  MOE_LAUNCH_CHECK();
  return MOE_OK;
}

static size_t g256(size_t v) { return (v + 255) & ~size_t(255); }

size_t w4_linear_gemm_ws(int T, int K) { return g256(2 * (size_t)T * K) + g256(4 * (size_t)T); }

int launch_w4_linear_gemm(const uint16_t* x, size_t ldx, int T, const uint8_t* w, const W4Dims& d, void* out,
                          size_t ldo, int out_f32, void* ws, int32_t* status, cudaStream_t s) {
  W4RowArgs r{};
  r.x = x, r.ldx = ldx, r.n = T, r.K = d.K;
  r.xp = (uint16_t*)ws;
  r.xexp = (int32_t*)((char*)ws + g256(2 * (size_t)T * d.K));
  w4_rows_kernel<<<std::min((T + 7) / 8, 1216), kRowThreads, 0, s>>>(r);
  MOE_LAUNCH_CHECK();
  W4GemmArgs g{};
  g.w = w, g.d = d, g.K = d.K, g.n = T;
  g.NF = (d.N + 2 * kGM - 1) / (2 * kGM);
  g.status = status, g.rexp = r.xexp;
  g.out = out, g.ldo = ldo, g.out_f32 = out_f32;
  return launch_gemm<kLinear>(g, r.xp, s);
}

// Workspace: x' [n][H] fp16, h [n][I] fp16, exponents, and y [n][H] fp16 where the caller combines.
size_t w4_ffn_gemm_ws(size_t n, int H, int I, bool yh) {
  return g256(2 * n * H) + g256(2 * n * I) + 3 * g256(4 * n) + (yh ? g256(2 * n * H) : 0);
}

// y rows of the listed experts (fp32 f.y, or scaled fp16 with *yh / *yexp set for launch_w4_combine).
int launch_ffn_w4_gemm(const FfnArgs& f, int group, void* ws, const uint16_t** yh, const int32_t** yexp,
                       cudaStream_t s, Prof* prof) {
  const size_t n = (size_t)f.T * f.k;
  const W4Slab sl = w4_slab(f.H, f.I, group);
  char* b = (char*)ws;
  auto take = [&](size_t bytes) {
    char* p = b;
    b += g256(bytes);
    return p;
  };
  W4RowArgs r{};
  r.x = f.x, r.ldx = f.H, r.n = (int)n, r.K = f.H;
  r.xp = (uint16_t*)take(2 * n * f.H);
  uint16_t* h = (uint16_t*)take(2 * n * f.I);
  r.xexp = (int32_t*)take(4 * n);
  r.hexp = (int32_t*)take(4 * n);
  r.yexp = (int32_t*)take(4 * n);
  W4GemmArgs g{};
  g.w = (const uint8_t*)f.pool, g.slab = sl.bytes, g.d = sl.gu, g.mat0 = 0, g.mat1 = sl.gu.bytes;
  g.K = f.H, g.n = (int)n, g.NF = (f.I + kGM - 1) / kGM;
  g.offset = f.offset, g.list_e = f.list_e, g.n_list = f.n_list, g.e2s = f.e2s, g.list_s = f.list_s;
  g.E = f.E, g.S = f.S, g.status = f.status;
  g.rexp = r.xexp, g.oexp = r.hexp, g.h = h;
  r.g = g, r.rows = f.rows, r.k = f.k, r.dn = sl.dn, r.mat2 = 2 * sl.gu.bytes;
  r.y = yh ? nullptr : f.y;
  if (prof) prof->begin(MOE_PROF_FFN_ROWS, s);
  w4_group_rows_kernel<<<(int)std::min((n + 7) / 8, (size_t)1216), kRowThreads, 0, s>>>(r);
  MOE_LAUNCH_CHECK();
  if (prof) prof->end(s);
  if (prof) prof->begin(MOE_PROF_FFN_GATEUP, s);
  int rc = launch_gemm<kGateUp>(g, r.xp, s);
  if (rc != MOE_OK) return rc;
  if (prof) prof->end(s);
  W4GemmArgs gd = g;
  gd.d = sl.dn, gd.mat0 = gd.mat1 = 2 * sl.gu.bytes;
  gd.K = f.I, gd.NF = (f.H + 2 * kGM - 1) / (2 * kGM);
  gd.rexp = r.hexp, gd.oexp = nullptr, gd.h = nullptr;
  gd.y = f.y;
  if (yh) {
    gd.yh = (uint16_t*)take(2 * n * f.H);
    *yh = gd.yh;
    *yexp = r.yexp;
  }
  if (prof) prof->begin(MOE_PROF_FFN_DOWN, s);
  if ((rc = launch_gemm<kDown>(gd, h, s)) != MOE_OK) return rc;
  if (prof) prof->end(s);
  return MOE_OK;
}

int launch_w4_combine(const uint16_t* yh, const int32_t* yexp, const float* w, const int32_t* pos, int T, int k, int H,
                      void* out, cudaStream_t s) {
  w4_combine_kernel<<<dim3(T, (H / 8 + 127) / 128), 128, 0, s>>>(yh, yexp, w, pos, k, H, (uint16_t*)out);
  MOE_LAUNCH_CHECK();
  return MOE_OK;
}

}  // namespace moe
