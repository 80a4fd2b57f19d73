// 4-bit products of many rows on the tcgen05 tensor cores: the linear layer, and the grouped gate / up
// and down products of the expert FFN.
//
// Computed transposed, D^T = W^T X^T, by CTA pairs (a cluster of two): a tile is 256 packed columns of
// W (128 in each CTA) x up to 256 rows (half of them in each CTA's shared memory).  The weights are the A
// operand and come from TMEM: worker threads own one column each, turn its codes into fp16 with about one
// fused multiply-add per pair and write them to TMEM, so the weights cross shared memory only once, as
// 4-bit codes.  The rows are the B operand, fp16 in shared memory (TMA, 128-byte swizzle).
//
// fp16, not bf16: (code - 8) * scale has up to 11 significant bits, exact in fp16.  The ranges are kept
// by powers of two: scales are stored relative to their column's largest (w4.cuh), each row of x is
// scaled so that its largest element is in [2^14, 2^15), h by the bound |h| <= |x|^2 |Wg| |Wu| (column
// 2-norms), y by the bound that follows.  A value keeps all 11 bits while it is above 2^-29 of its row's
// bound; typical values are 2^-11 (h) and 2^-16 (y) of it.  So x (8 bits) is exact, down to 2^-29 of the
// row's largest, and only h and, on its way to the combine, y are rounded, to 11 bits.
// The bound can be far too large: for a row with a few inputs far above the rest whose weights are small.  A row
// all of whose h are below 2^-17 of the bound is noticed on the way (w4g_small), its tile's gate / up product
// done again in a second launch (kRedo), scaled by the row's largest |h|, and y by what follows from that.
// (Inputs of 10^4 and 10^5 times the rest with zero weights, 2048 inputs: y off by 3% and 100% without that, as
// for ordinary rows with it.  Where no row needs it: 4096 tokens 346 -> 350 us, 1.4 of them the launch.)
//
// Why pairs and 256 rows: an MMA over 256 x 256 x 16 runs 128 cycles in each SM and one thread can issue
// it in that time; a pair's SM needs 32 B of rows and 8 B of codes a cycle from L2, near the 40 B that
// an SM gets; and each code is dequantised once per 256 rows.  (One CTA, 2 x 128 columns x 128 rows, took
// 87 us for 4096 rows through 2048 x 4096: its MMAs of 64 cycles could not be issued fast enough.)
//
// Warps: 0-15 are workers: four sets of four warps (one per TMEM lane quarter) that dequantise 128 inputs (a
// visit) in turn, each set into TMEM columns of its own; all drain the accumulators.  16 loads the rows, 18 the
// codes, 17 allocates TMEM and, in the pair's first CTA, issues the MMAs (one lane).
// A visit has one barrier for its rows' bytes and its workers' arrivals, and one commit gives both rings back:
// with a barrier and a commit per stage and ring the issuing warp needed 390 cycles a stage, and 4096 rows
// through 2048 x 4096 took 73 us instead of 66 (53 since the drain spills no registers and launches overlap; its
// MMAs alone would take 34).  Before a tile is drained three sets have dequantised inputs of the
// next one, so the MMAs go on while the drained values are stored.
// TMEM: 256 accumulator columns, 4 x 64 columns of weights.
#include <limits.h>

#include <algorithm>

#include "internal.cuh"
#include "tc05.cuh"
#include "w4.cuh"

namespace moe {

constexpr int kGM = 128;       // packed columns per CTA
constexpr int kGN = 256;       // rows per tile
constexpr int kGRows = 128;    // of them in one CTA's shared memory, at most
constexpr int kGK = 64;        // inputs per stage
constexpr int kGVisit = 2;     // stages that are copied, dequantised and multiplied at a time
constexpr int kGSets = 4;      // sets of four worker warps, taking visits in turn; visits of rows in shared memory
// Visits of codes in shared memory.  A multiple of the sets, so that a slot always belongs to the same set: copies
// can land out of order, and a set that met another set's slot could take a phase that is still open, by its
// parity, for the one after it.
constexpr int kGWRing = kGSets;
constexpr int kGWorkers = 4 * kGSets;
constexpr int kGThreads = 96 + 32 * kGWorkers;
constexpr int kGXBytes = kGRows * kGK * 2;      // a stage's rows
constexpr int kGCodeBytes = kGVisit * 4096;     // a visit's codes of 128 columns
constexpr int kGScaleBytes = kGVisit * 2 * 256; // its fp16 scales (two groups a stage at most)
constexpr int kGWBytes = kGCodeBytes + kGScaleBytes;
constexpr int kGEpiRows = 16;                   // rows that a worker warp stores at a time
constexpr int kGLd = 36;                        // staging: floats per row of 32 (padded against bank conflicts)
constexpr int kGEpiBytes = kGEpiRows * kGLd * 4;  // per worker warp
constexpr uint32_t kGTmemCols = 512;
constexpr uint32_t kGACol = kGN;                // first weight column
static_assert(kGN == 64 * kGSets, "each set drains 64 rows");
static_assert(kGWRing % kGSets == 0, "a slot of codes belongs to one set");

constexpr int kNoRow = INT_MIN;  // yexp of a row whose expert has no slot

enum { kGateUp = 0, kDown = 1, kLinear = 2, kRedo = 3 };  // kRedo: kGateUp of the tiles that hold a row to scale anew

struct W4GemmArgs {
  const uint8_t* w;        // slab pool, or the packed matrix
  size_t slab;             // bytes between slabs (0: one matrix)
  W4Dims d;
  size_t mat;              // offset of the matrix in a slab
  int K, NF;               // K of the rows; column tiles of 256
  int n;                   // rows
  int parts, stages;       // kLinear: parts of the inputs, stages in one (even); 1 and d.Kb elsewhere
  // grouped rows
  const int32_t *offset, *list_e, *n_list, *e2s, *list_s;
  int E, S;
  int32_t* status;
  const int32_t* rexp;     // [n] the B operand's row p is 2^-rexp[p] times the true one
  const int32_t* oexp;     // [n] kGateUp: the same of h, by its bound
  // grouped rows: of a row's runs of 16 h, how many are small, their largest |h 2^-oexp| (its bits), and whether
  // there is a row all of whose runs are; yexp of such rows is corrected by kRedo
  int32_t *hcnt, *hmax, *redo, *yexp;
  // outputs
  uint16_t* h;             // kGateUp: fp16 [n][ldh]
  int ldh;
  uint16_t* yh;            // kDown: fp16 [n][N], 2^-(rexp + w4_y_exp) times y, or NULL
  float* y;                // kDown: fp32 [n][N]
  void* out;               // kLinear
  size_t ldo;
  int out_f32;
};

// The rows as tensor maps with boxes of 16, 32, ... 128 rows x two stages: one copy a visit.
constexpr int kGBoxes = kGRows / 16;
struct W4RowMaps {
  CUtensorMap m[kGBoxes];
};
// Rows are kept in whole stages, the rest zeros.
__host__ __device__ inline int w4g_ld(int K) { return (K + kGK - 1) / kGK * kGK; }

// D[tmem of both CTAs] (+)= A[tmem of both] x B[smem of both], over one 64-deep stage: four MMAs; the first
// accumulates when `accumulate` is nonzero.
__device__ __forceinline__ void umma_f16_ts_pair_k64(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                                     uint32_t accumulate) {
  asm volatile(
      "{\n"
      " .reg .pred p, t;\n"
      " setp.ne.b32 p, %4, 0;\n"
      " setp.eq.b32 t, 0, 0;\n"
      " tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n"
      " tcgen05.mma.cta_group::2.kind::f16 [%0], [%5], %6, %3, t;\n"
      " tcgen05.mma.cta_group::2.kind::f16 [%0], [%7], %8, %3, t;\n"
      " tcgen05.mma.cta_group::2.kind::f16 [%0], [%9], %10, %3, t;\n"
      "}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(a_tmem + 8), "l"(bdesc + 2), "r"(a_tmem + 16),
      "l"(bdesc + 4), "r"(a_tmem + 24), "l"(bdesc + 6)
      : "memory");
}

// Arrive on an mbarrier of either CTA of the pair, by its shared::cluster address.  What such an arrival
// hands over is in TMEM, which the tcgen05 waits and fences order; a release at cluster scope would wait for
// the thread's global stores as well (about 1,000 cycles after a drain).
__device__ __forceinline__ void mbar_arrive_pair(uint32_t caddr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(caddr) : "memory");
}

// Waits for a barrier's phase, kGPolls tests at most, in as few instructions as there can be: waiting warps
// share their schedulers with the workers.
constexpr uint32_t kGPolls = 64;  // between looks at the abort flag
__device__ __forceinline__ bool mbar_poll(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n"
      " .reg .pred p, q;\n"
      " .reg .u32 n;\n"
      " mov.u32 n, %3;\n"
      "POLL:\n"
      " mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      " @p bra DONE;\n"
      " sub.u32 n, n, 1;\n"
      " setp.ne.u32 q, n, 0;\n"
      " @q bra POLL;\n"
      "DONE:\n"
      " selp.u32 %0, 1, 0, p;\n"
      "}\n"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity), "n"(kGPolls)
      : "memory");
  return ok != 0;
}

// 2^e >= 1.001 |column|_2 of every column whose norm is finite (0 for a matrix of zeros).
__device__ __forceinline__ int w4_norm_exp(const uint8_t* meta) {
  const float c = *reinterpret_cast<const float*>(meta);
  return c > 0.f ? ilogbf(c) + 1 : 0;
}
// |y| <= |h|_2 |column|_2 <= sqrt(I) 2^15 2^hexp 2^norm_exp: the exponent that takes y / 2^hexp below 2^15.
__device__ __forceinline__ int w4_y_exp(const uint8_t* m, const W4Dims& d) {
  return (32 - __clz(d.K) + 1) / 2 + w4_norm_exp(m + d.meta);
}

// Of a row all of whose h are small: the exponent, <= 0, that takes 2^he times it to the row's largest |h| (in
// [2^14, 2^15) of it).  0 for other rows, and for rows of zeros.
constexpr float kGSmall = 0.25f;  // |h 2^-he| below it is small: 2^-25, which fp16 rounds by, is 2^-23 of it
__device__ __forceinline__ int w4_h_shift(const W4GemmArgs& a, int runs, size_t p, int he) {
  const float m = __int_as_float(a.hmax[p]);
  return a.hcnt[p] == runs && m > 0.f ? max(ilogbf(m) - 14, -126 - he) : 0;
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
  const uint8_t* base;  // the matrix
  int ft, row0, ntok;
  int k0, nk;           // first stage, stages
  int part;
};

// Tile t: column tile t % NF, row tile t / NF (by the prefix of row tiles over the list); kLinear: of part
// t / (NF x row tiles) of the inputs.
template <int kMode>
__device__ __forceinline__ W4GTile w4g_tile(const W4GemmArgs& a, const int* pre, int nl, int t) {
  W4GTile r;
  const int i = t / a.NF;
  r.ft = t - i * a.NF;
  r.k0 = r.part = 0, r.nk = a.d.Kb;
  if (kMode == kLinear) {
    const int rt = (a.n + kGN - 1) / kGN;
    r.part = i / rt;
    r.k0 = r.part * a.stages, r.nk = min(a.stages, a.d.Kb - r.k0);
    r.base = a.w;
    r.row0 = (i - r.part * rt) * kGN;
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
    r.base = a.w + (size_t)slot * a.slab + a.mat;
    r.row0 = a.offset[e] + (i - pre[lo]) * kGN;
    r.ntok = min(kGN, a.offset[e + 1] - r.row0);
  }
  return r;
}

// Rows of a tile in each CTA: half the MMA's N, which is a multiple of 32.
__host__ __device__ __forceinline__ int w4g_half(int ntok) { return ((ntok + 31) & ~31) >> 1; }

// Eight codes of a word (w4.cuh) times their scale, fp16, inputs in order.
__device__ __forceinline__ void w4_expand(uint32_t w, __half2 s, uint32_t* o) {
  const __half2 m24s = __hmul2(s, __float2half2_rn(-24.f));
  auto top = [&](uint32_t v) {  // codes in bits 6-9: 16 + code; (16 + code) s - 24 s is exact
    asm("lop3.b32 %0, %0, %1, %2, 0xEA;" : "+r"(v) : "r"(0x03c003c0u), "r"(0x4c004c00u));
    const __half2 r = __hfma2(*reinterpret_cast<const __half2*>(&v), s, m24s);
    return *reinterpret_cast<const uint32_t*>(&r);
  };
  // codes in bits 3-6: 128 + code; the shift is saved and one more half-precision operation spent, which
  // keeps the integer and the floating-point pipe equally busy
  uint32_t v;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(v) : "r"(w), "r"(0x00780078u), "r"(0x58005800u));
  const __half2 c = __hsub2(*reinterpret_cast<const __half2*>(&v), __float2half2_rn(136.f)), p = __hmul2(c, s);
  o[0] = *reinterpret_cast<const uint32_t*>(&p);
  o[1] = top(w >> 1);
  o[2] = top(w >> 5);
  o[3] = top(__funnelshift_r(w, w, 9));
}

__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }  // -126 <= e <= 127

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&p);
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 p = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&p);
}

// What the drain of 64 rows (of set `set`) multiplies with: the rows' exponents (two rows a lane) and the
// lane's column's power of two.  Loaded a visit before they are needed.
struct W4GFactors {
  int r[2], o[2];
  float cm;
};
template <int kMode>
__device__ __forceinline__ W4GFactors w4g_factors(const W4GemmArgs& a, const W4GTile& ti, int blk, int q, int set,
                                                  int lane) {
  const W4Dims& d = a.d;
  const int tok0 = 64 * set, nrow = ti.ntok - tok0, c = blk * kGM + 32 * q + lane;
  W4GFactors f = {};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const size_t p = (size_t)ti.row0 + tok0 + 32 * i + lane;
    if (32 * i + lane < nrow) {
      // scaled rows of y keep the row's own power of two apart, and parts of the inputs theirs, up to their sum
      if (!(kMode == kDown && a.yh) && !(kMode == kLinear && a.parts > 1)) f.r[i] = a.rexp[p];
      if (kMode == kDown && !a.yh) f.r[i] += w4_h_shift(a, d.K / 16, p, f.r[i]);
      if (kMode == kGateUp || kMode == kRedo) f.o[i] = a.oexp[p];
      if (kMode == kRedo) f.o[i] += w4_h_shift(a, d.N / 32, p, f.o[i]);
    }
  }
  if (c < d.N) f.cm = reinterpret_cast<const float*>(ti.base + d.mult)[c];
  if (kMode == kDown && a.yh) f.cm = ldexpf(f.cm, -w4_y_exp(ti.base, d));
  return f;
}

// 16 rows x 32 packed columns of a warp, as 16-bit values times the column's power of two (v[row pair], a
// column per lane), through shared memory (st) to their place: the rows 16 i, ... of the 64 of f.
template <int kMode>
__device__ __forceinline__ void w4g_store16(const W4GemmArgs& a, const uint32_t* v, uint32_t* st, const W4GFactors& f,
                                            int i, size_t row0, int nrow, int c0, int lane) {
  const W4Dims& d = a.d;
  const size_t ld = kMode == kLinear ? a.ldo : (size_t)d.N;
#pragma unroll
  for (int j = 0; j < kGEpiRows / 2; ++j) st[j * kGLd + lane] = v[j];
  __syncwarp();
  uint16_t* out = kMode == kLinear ? reinterpret_cast<uint16_t*>(a.out) : a.yh;
  auto row_fac = [&](int row) { return pow2(__shfl_sync(MOE_FULL_MASK, f.r[i >> 1], 16 * (i & 1) + row)); };
  auto scaled = [](uint32_t w, float m) {
    const __nv_bfloat162 p = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&w), __float2bfloat162_rn(m));
    return *reinterpret_cast<const uint32_t*>(&p);
  };
  if (kMode == kLinear && !(ld % 8 == 0 && (uintptr_t)a.out % 16 == 0 && c0 + 32 <= d.N)) {
    // unaligned or ragged rows of out: element stores, 32 consecutive columns per row
    for (int j = 0; j < nrow; ++j) {
      const float m = row_fac(j);
      if (c0 + lane < d.N) {
        const uint32_t w = scaled(st[j / 2 * kGLd + lane], m);
        out[(row0 + j) * ld + c0 + lane] = uint16_t(j & 1 ? w >> 16 : w);
      }
    }
  } else {
    const int rp = lane >> 2, seg = (lane & 3) * 8;  // 8 row pairs x 4 runs of 8 columns
    const uint4 w0 = *reinterpret_cast<const uint4*>(st + rp * kGLd + seg);
    const uint4 w1 = *reinterpret_cast<const uint4*>(st + rp * kGLd + seg + 4);
    float m[2] = {1.f, 1.f};
    if (kMode == kLinear) m[0] = row_fac(2 * rp), m[1] = row_fac(2 * rp + 1);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t sel = h ? 0x7632 : 0x5410;
      uint32_t o[4] = {__byte_perm(w0.x, w0.y, sel), __byte_perm(w0.z, w0.w, sel), __byte_perm(w1.x, w1.y, sel),
                       __byte_perm(w1.z, w1.w, sel)};
      if (kMode == kLinear)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] = scaled(o[j], m[h]);
      if (2 * rp + h < nrow)
        *reinterpret_cast<uint4*>(out + (row0 + 2 * rp + h) * ld + c0 + seg) = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
  __syncwarp();
}

// Notes the rows of a warp's 16 rows x 16 h whose run is small.  most: the largest |h| of a lane's half of a run.
__device__ __forceinline__ void w4g_small(const W4GemmArgs& a, float most, size_t row0, int nrow, int lane) {
  const unsigned big = __ballot_sync(MOE_FULL_MASK, most >= kGSmall);
  if (((big | big >> 1) & 0x55555555u) == 0x55555555u) return;  // as usual
  most = fmaxf(most, __shfl_xor_sync(MOE_FULL_MASK, most, 1));
  if ((lane & 1) || (lane >> 1) >= nrow || most >= kGSmall) return;
  const size_t p = row0 + (lane >> 1);
  atomicMax(a.hmax + p, __float_as_int(most));
  __threadfence();
  if (atomicAdd(a.hcnt + p, 1) == a.d.N / 32 - 1 && atomicMax(a.hmax + p, 0) > 0) *a.redo = 1;
}

// The same of fp32 values (v[row], without the column's power of two): to fp32 results, or (kGateUp, kRedo) to h.
template <int kMode>
__device__ __forceinline__ void w4g_store32(const W4GemmArgs& a, const float* v, float* st, const W4GFactors& f, int i,
                                            int part, size_t row0, int nrow, int c0, int lane) {
  const W4Dims& d = a.d;
  auto row_fac = [&](int row) { return pow2(__shfl_sync(MOE_FULL_MASK, f.r[i >> 1], 16 * (i & 1) + row)); };
#pragma unroll
  for (int j = 0; j < kGEpiRows; ++j) st[j * kGLd + lane] = v[j] * f.cm;
  __syncwarp();
  if (kMode == kGateUp || kMode == kRedo) {  // columns 0-15: gate, 16-31: up of the same 16 features
    const int f0 = c0 / 2, row = lane >> 1, seg = (lane & 1) * 8;
    const float x = row_fac(row),
                xh = x * pow2(-__shfl_sync(MOE_FULL_MASK, f.o[i >> 1], 16 * (i & 1) + row));
    uint32_t o[4];
    float most = 0.f;
#pragma unroll
    for (int j = 0; j < 8; j += 4) {
      const float4 g = *reinterpret_cast<const float4*>(st + row * kGLd + seg + j);
      const float4 u = *reinterpret_cast<const float4*>(st + row * kGLd + 16 + seg + j);
      auto h = [&](float gv, float uv) {
        gv *= x;
        const float hv = __fdividef(gv, 1.f + __expf(-gv)) * (uv * xh);
        if (kMode == kGateUp) most = fmaxf(most, fabsf(hv));
        return hv;
      };
      o[j / 2] = pack_f16(h(g.x, u.x), h(g.y, u.y));
      o[j / 2 + 1] = pack_f16(h(g.z, u.z), h(g.w, u.w));
    }
    if (row < nrow) *reinterpret_cast<uint4*>(a.h + (row0 + row) * a.ldh + f0 + seg) = make_uint4(o[0], o[1], o[2], o[3]);
    if (kMode == kGateUp) w4g_small(a, most, row0, nrow, lane);
  } else {
    // (a part of the inputs writes sums of its own)
    float* out = kMode == kLinear ? reinterpret_cast<float*>(a.out) + (size_t)part * a.n * a.ldo : a.y;
    const size_t ld = kMode == kLinear ? a.ldo : (size_t)d.N;
    if (kMode == kLinear && !(ld % 4 == 0 && (uintptr_t)a.out % 16 == 0 && c0 + 32 <= d.N)) {
      for (int row = 0; row < nrow; ++row) {
        const float m = row_fac(row);
        if (c0 + lane < d.N) out[(row0 + row) * ld + c0 + lane] = st[row * kGLd + lane] * m;
      }
    } else {
#pragma unroll
      for (int n = 0; n < kGEpiRows / 4; ++n) {  // rows of 128 B
        const int idx = n * 32 + lane, row = idx >> 3, seg = (idx & 7) * 4;
        float4 o = *reinterpret_cast<const float4*>(st + row * kGLd + seg);
        const float m = row_fac(row);
        o.x *= m, o.y *= m, o.z *= m, o.w *= m;
        if (row < nrow) *reinterpret_cast<float4*>(out + (row0 + row) * ld + c0 + seg) = o;
      }
    }
  }
  __syncwarp();
}

// Drains 64 rows (of set `set`) x this warp's 32 columns: to registers, the accumulators are handed back
// (tempty of the pair's first CTA), then 16 rows at a time through shared memory to their place.  16-bit results
// are rounded on their way to the registers, which takes half as many.
template <int kMode, class Wait>
__device__ __forceinline__ void w4g_drain(const W4GemmArgs& a, const W4GTile& ti, int blk, uint32_t taddr, int q, int set,
                                          int lane, float* st, const W4GFactors& f, uint64_t* tfull,
                                          uint32_t tempty0, uint32_t parity, Wait&& wait, const bool& dead) {
  const W4Dims& d = a.d;
  const int tok0 = 64 * set, nrow = ti.ntok - tok0, c0 = blk * kGM + 32 * q;
  const bool any = nrow > 0 && c0 < d.N;
  const bool half = kMode == kLinear ? !a.out_f32 : kMode == kDown && a.yh != nullptr;
  const size_t row0 = (size_t)ti.row0 + tok0;
  __syncwarp();
  wait(tfull, parity);
  tc_fence_after();
  auto hand_back = [&] {
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive_pair(tempty0);
  };
  if (!any) {
    hand_back();
    return;
  }
  if (half) {
    // two rows of a column in a word; the rows' powers of two are exact after the rounding too (a bf16 has
    // fp32's range; y's fp16 rows carry none)
    uint32_t v[32];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float t[32];
      tmem_ld32(taddr + tok0 + 32 * i, t);
      tmem_ld_wait();
#pragma unroll
      for (int j = 0; j < 32; j += 2)
        v[16 * i + j / 2] = kMode == kLinear ? pack_bf16(t[j] * f.cm, t[j + 1] * f.cm) : pack_f16(t[j] * f.cm, t[j + 1] * f.cm);
    }
    hand_back();
    if (dead) return;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (nrow > 16 * i)
        w4g_store16<kMode>(a, v + 8 * i, reinterpret_cast<uint32_t*>(st), f, i, row0 + 16 * i,
                           min(nrow - 16 * i, 16), c0, lane);
  } else {
    float v0[32], v1[32];
    tmem_ld32(taddr + tok0, v0);
    tmem_ld32(taddr + tok0 + 32, v1);
    tmem_ld_wait();
    hand_back();
    if (dead) return;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (nrow > 16 * i)
        w4g_store32<kMode>(a, (i < 2 ? v0 : v1) + 16 * (i & 1), st, f, i, ti.part, row0 + 16 * i,
                           min(nrow - 16 * i, 16), c0, lane);
  }
}

template <int kMode>
__global__ void __launch_bounds__(kGThreads, 1) w4_gemm_kernel(const W4GemmArgs a, const __grid_constant__ W4RowMaps mapX) {
  extern __shared__ __align__(16) unsigned char gsm_raw[];
  unsigned char* sm = gsm_raw + ((0u - smem_u32(gsm_raw)) & 1023u);  // (an offset: the accesses stay shared ones)
  unsigned char* xs = sm;                             // [ring][stages of a visit][16 KB]
  unsigned char* wsm = sm + kGSets * kGVisit * kGXBytes;  // [ring][codes | scales]
  float* epi = reinterpret_cast<float*>(wsm + kGWRing * kGWBytes);   // [workers][kGEpiRows][kGLd]
  // of a visit: its rows have landed and its weights are in TMEM, in both CTAs (the first one's barrier counts);
  // its MMAs have read both
  uint64_t* full = reinterpret_cast<uint64_t*>(epi + kGWorkers * (kGEpiBytes / 4));
  uint64_t* empty = full + kGSets;
  uint64_t* wfull = empty + kGSets;
  uint64_t* wempty = wfull + kGWRing;
  uint64_t* tfull = wempty + kGWRing;
  uint64_t* tempty = tfull + 1;
  uint64_t* done = tempty + 1;
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  __shared__ int s_pre[kMode == kLinear ? 1 : kMaxE + 1];
  __shared__ int s_tmp[33];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int cl = (int)cluster_index(), ncl = (int)cluster_count();
  const W4Dims& d = a.d;
  int nl = 0, total;

  if (kMode == kRedo) {
    pdl_wait();
    pdl_trigger();
    if (*a.redo == 0) return;  // in every CTA
    for (int p = blockIdx.x * kGThreads + threadIdx.x; p < a.n; p += gridDim.x * kGThreads)
      if (a.yexp[p] != kNoRow) a.yexp[p] += w4_h_shift(a, d.N / 32, p, a.oexp[p]);
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < kGWRing; ++s) {
      mbar_init(&wfull[s], 1);
      mbar_init(&wempty[s], 4);  // a set's four warps
    }
    for (int s = 0; s < kGSets; ++s) {
      mbar_init(&full[s], 9);  // a set's four warps in each CTA, and the bytes
      mbar_init(&empty[s], 1);
    }
    mbar_init(tfull, 1);
    mbar_init(tempty, 2 * kGWorkers);
    mbar_init(done, 1);
    s_abort = 0;
    mbar_fence_init();
  }
  if (warp == kGWorkers + 1) {
    tmem_alloc_pair(&s_tmem, kGTmemCols);
    tmem_relinquish_pair();
  }
  if (kMode != kRedo) {
    pdl_wait();
    pdl_trigger();
  }
  if (kMode == kLinear) {
    total = (a.n + kGN - 1) / kGN * a.NF * a.parts;
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
    total = carry * a.NF;
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync();  // barriers of both CTAs initialised, TMEM allocated on both, prefix complete
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  volatile int* abort_flag = &s_abort;
  // Waits as a whole warp, first with one test (the loops that issue copies are short of instructions: 4096 tokens
  // 358 us, 350 with it).  A wait that gives up (or sees that another one did) ends the work of its role: `dead`,
  // the same in every lane; a role that is dead waits no more.
  bool dead = false;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (__all_sync(MOE_FULL_MASK, mbar_try_wait(bar, parity)) || dead) return;
    bool ok = false;
    for (int i = 0; i < int(kWaitPolls / kGPolls) && !ok && !*abort_flag; ++i) ok = mbar_poll(bar, parity);
    if (!ok && !*abort_flag) {
      *abort_flag = 1;
      set_status(a.status, MOE_DEV_TIMEOUT);
    }
    dead = __any_sync(MOE_FULL_MASK, !ok);
  };

  // the first tile from t on that there is work in
  auto next = [&](int t) {
    if (kMode == kRedo)
      for (; t < total; t += ncl) {
        const W4GTile ti = w4g_tile<kMode>(a, s_pre, nl, t);
        bool any = false;
        for (int i = lane; i < ti.ntok; i += 32) {
          const size_t p = (size_t)ti.row0 + i;
          any |= w4_h_shift(a, d.N / 32, p, a.oexp[p]) != 0;
        }
        if (__any_sync(MOE_FULL_MASK, any)) break;
      }
    return t;
  };

  if (warp == kGWorkers) {
    const bool lead = elect_one();
    uint32_t s = 0, ph = 1, issued = 0;
    for (int t = next(cl); t < total && !dead; t = next(t + ncl)) {
      const W4GTile ti = w4g_tile<kMode>(a, s_pre, nl, t);
      const int r = w4g_half(ti.ntok), row = ti.row0 + (int)rank * r;
      const CUtensorMap* map = &mapX.m[r / 16 - 1];
      for (int kb = ti.k0; kb < ti.k0 + ti.nk; kb += kGVisit) {
        wait(&empty[s], ph);
        if (dead) break;
        if (lead) {
          // the first CTA's barrier counts the bytes of both (of two stages: past the last one zeros are read)
          if (rank == 0) mbar_expect_tx(&full[s], 2u * kGVisit * (uint32_t)r * (kGK * 2));
          tma_load_3d_pair(xs + s * (kGVisit * kGXBytes), map, mapa_shared(smem_u32(&full[s]), 0), 0, row, kb);
        }
        __syncwarp();
        ++issued;
        s = (s + 1) % kGSets;
        ph ^= s == 0;
      }
    }
    // after a timeout: let every copy land before the CTAs can exit (the workers' arrivals may be missing, so
    // that the barriers can only show it where they complete: the wait is short and bounded)
    if (dead && rank == 0)
      for (uint32_t j = issued > kGSets ? issued - kGSets : 0; j < issued; ++j)
        for (int i = 0; i < 1024 && !mbar_poll(&full[j % kGSets], (j / kGSets) & 1u); ++i) {
        }
  } else if (warp == kGWorkers + 2) {
    const bool lead = elect_one();
    uint32_t s = 0, ph = 1, issued = 0;
    for (int t = next(cl); t < total && !dead; t = next(t + ncl)) {
      const W4GTile ti = w4g_tile<kMode>(a, s_pre, nl, t);
      const int blk = 2 * ti.ft + (int)rank;
      const uint32_t nm = max(0, min(8, d.Mt - 8 * blk));  // the tiles of 16 columns that exist
      const uint8_t* code = ti.base + w4_code_at(d, 8 * blk, ti.k0) * 512;
      const uint8_t* scale = ti.base + d.scales + w4_scale_at(d, 8 * blk, ti.k0 * kGK / d.G, 0) * 4;
      const uint32_t cb = nm * 512 * kGVisit, sb = nm * 32 * (kGVisit * kGK / d.G);  // of a whole visit
      for (int kb = 0; kb < ti.nk; kb += kGVisit) {
        wait(&wempty[s], ph);
        if (dead) break;
        if (lead) {
          unsigned char* dst = wsm + s * kGWBytes;
          const bool whole = kb + kGVisit <= ti.nk;  // else one stage
          const uint32_t c1 = whole ? cb : cb / 2, s1 = whole || d.G == 128 ? sb : sb / 2;
          if (nm > 0) {
            mbar_expect_tx(&wfull[s], c1 + s1);
            bulk_load(dst, code, c1, &wfull[s]);
            bulk_load(dst + kGCodeBytes, scale, s1, &wfull[s]);
          } else {
            mbar_arrive(&wfull[s]);  // the pair's second CTA has no columns here: its results are dropped
          }
        }
        __syncwarp();
        code += cb, scale += sb;
        ++issued;
        s = (s + 1) % kGWRing;
        ph ^= s == 0;
      }
    }
    if (dead)
      for (uint32_t j = issued > kGWRing ? issued - kGWRing : 0; j < issued; ++j)
        mbar_wait(&wfull[j % kGWRing], (j / kGWRing) & 1u);
  } else if (warp == kGWorkers + 1) {
    if (rank == 0) {
      const uint64_t bd0 = smem_desc_l(smem_u32(xs), 16, 1024, kLayoutSw128);
      const bool lead = elect_one();
      uint32_t s = 0, ph = 0, tp = 1;  // of the ring, of the accumulators
      for (int t = next(cl); t < total && !dead; t = next(t + ncl)) {
        const W4GTile ti = w4g_tile<kMode>(a, s_pre, nl, t);
        const int r = w4g_half(ti.ntok);
        const uint32_t idesc = idesc_f16(2 * kGM, 2 * r);
        wait(tempty, tp);
        tp ^= 1;
        for (int kb = 0; kb < ti.nk; kb += kGVisit) {
          wait(&full[s], ph);
          tc_fence_after();
          if (lead && !dead) {
            const uint32_t at = tmem + kGACol + s * 64;
            const uint64_t bd = bd0 + (uint64_t)(s * kGVisit * (kGXBytes >> 4));
            umma_f16_ts_pair_k64(tmem, at, bd, idesc, kb > 0);
            if (kb + 1 < ti.nk) umma_f16_ts_pair_k64(tmem, at + 32, bd + (uint64_t)(r * (kGK * 2 >> 4)), idesc, 1);
          }
          if (lead) umma_commit_pair(&empty[s]);
          __syncwarp();
          s = (s + 1) % kGSets;
          ph ^= s == 0;
        }
        if (lead) umma_commit_pair(tfull);
        __syncwarp();
      }
      if (lead) umma_commit_pair(done);  // completes in both CTAs once every MMA has finished
      __syncwarp();
    }
    mbar_wait(done, 0);
  } else if (warp < kGWorkers) {
    const int q = warp & 3, set = warp >> 2;  // TMEM lane quarter; visits (dequantising) and rows (draining)
    const int r = 32 * q + lane, g = r & 7, hi = (r >> 3) & 1;
    const uint32_t lane_addr = tmem + ((uint32_t)(q * 32) << 16);
    const uint32_t a_addr = lane_addr + kGACol + set * 64;
    float* st = epi + warp * (kGEpiBytes / 4);
    const uint32_t full0 = mapa_shared(smem_u32(&full[set]), 0), tempty0 = mapa_shared(smem_u32(tempty), 0);
    uint32_t vi = 0, tc = 0;          // visits before this tile, tiles drained
    uint32_t uses = 0;                // this set's visits
    W4GTile prev = {};
    bool pending = false;  // prev has not been drained
    W4GFactors f = {};
    for (int t = next(cl);; t = next(t + ncl)) {
      const bool real = t < total && !dead;
      W4GTile ti = {};
      if (real) ti = w4g_tile<kMode>(a, s_pre, nl, t);
      const int nm = max(1, min(8, d.Mt - 8 * (2 * ti.ft + (int)rank))), nk = real ? ti.nk : 0;
      // a visit of every set but one (whose columns the last tile's final MMAs still read), the last tile's
      // drain, the other visits; this set's are every fourth one of the CTA's sequence
      int kb = (int)((set - vi) % kGSets) * kGVisit;
#pragma unroll 1
      for (int phase = 0; phase < 2; ++phase) {
        const int end = phase ? nk : min(nk, (kGSets - 1) * kGVisit);
#pragma unroll 1
        for (; kb < end; kb += kGSets * kGVisit) {
          const uint32_t v = vi + kb / kGVisit, ws = v % kGWRing;
          wait(&wfull[ws], (v / kGWRing) & 1u);
          const unsigned char* wst = wsm + ws * kGWBytes;
          uint32_t o[32];
#pragma unroll
          for (int h = 0; h < kGVisit; ++h) {
            if (kb + h >= nk) break;
            const unsigned char* code = wst + (h * nm + (r >> 4)) * 512 + g * 64 + hi * 8;
            const int gi = d.G == 128 ? 0 : d.G == 64 ? h : 2 * h;
            const __half* sp = reinterpret_cast<const __half*>(wst + kGCodeBytes + (gi * nm * 8 + g * nm + (r >> 4)) * 4) + hi;
            uint2 w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = *reinterpret_cast<const uint2*>(code + ((j + (g >> 1)) & 3) * 16);
            const __half2 s0 = __half2half2(sp[0]), s1 = d.G == 32 ? __half2half2(sp[16 * nm]) : s0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              w4_expand(w[j].x, s0, &o[4 * j]);
              w4_expand(w[j].y, s1, &o[16 + 4 * j]);
            }
            if (h == 0) wait(&empty[set], (uses & 1u) ^ 1u);
            tc_fence_after();
            tmem_st32(a_addr + 32 * h, o);
          }
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive_pair(full0);
            mbar_arrive(&wempty[ws]);
          }
          ++uses;
        }
        if (phase == 0 && pending) {
          w4g_drain<kMode>(a, prev, 2 * prev.ft + (int)rank, lane_addr, q, set, lane, st, f, tfull, tempty0, tc & 1u,
                           wait, dead);
          ++tc;
        }
      }
      if (!real) break;
      prev = ti;
      pending = true;
      f = w4g_factors<kMode>(a, ti, 2 * ti.ft + (int)rank, q, set, lane);
      vi += (nk + kGVisit - 1) / kGVisit;
    }
  }
  // reconverge before the cluster barrier, which also keeps each CTA's shared memory alive while its peer
  // may still signal it
  __syncwarp();
  tc_fence_before();
  cluster_sync();
  if (warp == kGWorkers + 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, kGTmemCols);
  }
}

// ---------------------------------------------------------------------------
// Rows: x -> fp16 times a power of two per row, in grouped order; one warp per row.
// ---------------------------------------------------------------------------
constexpr int kRowThreads = 256, kTokenThreads = 128;

struct W4RowArgs {
  const uint16_t* x;
  size_t ldx;
  int n, K;                // rows of xp, or of x with ids and pos
  uint16_t* xp;            // fp16 [n][ld], zeros past K
  int ld;
  int32_t* xexp;           // [n]
  // grouped rows (list_e != NULL)
  W4GemmArgs g;
  const int32_t* rows;
  const int32_t *ids, *pos;  // every slot is grouped: rows by token (w4_token_rows_kernel)
  int k;
  W4Slab sl;
  int32_t *hexp, *yexp;    // [n]
  float* y;                // rows of experts without a slot are zeroed, or NULL (yexp says so)
};

// The share of a row x of K inputs that one of `step` threads (the i0-th) has: 16 bytes of every 16 step.  It is
// read once, all of it in flight at a time, up to NC loads; what is beyond them is read again.
template <int NC>
struct W4Row {
  const uint4* x;
  int n, i0, step, xe;
  float f0, f1;
  uint4 v[NC];  // scaled, after scale()

  __device__ __forceinline__ uint32_t conv(uint32_t u) const { return pack_f16(bf16_lo(u) * f0 * f1, bf16_hi(u) * f0 * f1); }
  __device__ __forceinline__ uint4 conv(uint4 u) const { return make_uint4(conv(u.x), conv(u.y), conv(u.z), conv(u.w)); }

  // The largest magnitude, as bits (bf16 magnitudes are ordered like integers); infinities and NaN do not count.
  __device__ __forceinline__ uint32_t load(const uint16_t* row, int K, int i0_, int step_) {
    x = reinterpret_cast<const uint4*>(row), n = K / 8, i0 = i0_, step = step_;
#pragma unroll
    for (int i = 0; i < NC; ++i) v[i] = step * i + i0 < n ? __ldg(x + step * i + i0) : make_uint4(0, 0, 0, 0);
    uint32_t amax = 0;
    auto take = [&](uint32_t u) {
      const uint32_t lo = u & 0x7fffu, hi = (u >> 16) & 0x7fffu;
      amax = max(amax, lo < 0x7f80u ? lo : 0u);
      amax = max(amax, hi < 0x7f80u ? hi : 0u);
    };
#pragma unroll
    for (int i = 0; i < NC; ++i) take(v[i].x), take(v[i].y), take(v[i].z), take(v[i].w);
    for (int c = step * NC + i0; c < n; c += step) {
      const uint4 u = __ldg(x + c);
      take(u.x), take(u.y), take(u.z), take(u.w);
    }
    return amax;
  }
  // With the whole row's largest: xe, and this share times 2^-xe; with kNorm its sum of squares.
  template <bool kNorm>
  __device__ __forceinline__ float scale(uint32_t amax) {
    xe = amax ? max(ilogbf(__uint_as_float(amax << 16)) - 14, -126) : 0;
    f0 = ldexpf(1.f, -xe / 2), f1 = ldexpf(1.f, -xe - (-xe / 2));  // 2^-xe may overflow by itself
    float nrm = 0.f;
    auto square = [&](uint32_t u) {
      const float lo = bf16_lo(u) * f0 * f1, hi = bf16_hi(u) * f0 * f1;
      nrm += fabsf(lo) < INFINITY ? lo * lo : 0.f;
      nrm += fabsf(hi) < INFINITY ? hi * hi : 0.f;
    };
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      if (kNorm) square(v[i].x), square(v[i].y), square(v[i].z), square(v[i].w);
      v[i] = conv(v[i]);
    }
    if (kNorm)
      for (int c = step * NC + i0; c < n; c += step) {
        const uint4 u = __ldg(x + c);
        square(u.x), square(u.y), square(u.z), square(u.w);
      }
    return nrm;
  }
  // To ld values, zeros past the row's own.
  __device__ __forceinline__ void store(uint16_t* row, int ld) const {
    uint4* o = reinterpret_cast<uint4*>(row);
#pragma unroll
    for (int i = 0; i < NC; ++i)
      if (step * i + i0 < ld / 8) o[step * i + i0] = v[i];
    for (int c = step * NC + i0; c < ld / 8; c += step) o[c] = c < n ? conv(__ldg(x + c)) : make_uint4(0, 0, 0, 0);
  }
};

// A row by one warp: loaded and scaled; with kNorm, returns ceil(log2 |x'|^2) (x' = the scaled row).
template <bool kNorm, int NC>
__device__ __forceinline__ int w4_warp_row(W4Row<NC>& r, const uint16_t* row, int K, int lane) {
  float nrm = r.template scale<kNorm>(__reduce_max_sync(MOE_FULL_MASK, r.load(row, K, lane, 32)));
  if (kNorm)
#pragma unroll
    for (int o = 16; o; o >>= 1) nrm += __shfl_xor_sync(MOE_FULL_MASK, nrm, o);
  return nrm > 0.f ? ilogbf(nrm * 1.001f) + 1 : 0;
}

// Rows of a linear layer, a warp to a row.
template <int NC>
__global__ void __launch_bounds__(kRowThreads) w4_rows_kernel(const W4RowArgs a) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = gridDim.x * (kRowThreads / 32);
  pdl_wait();
  pdl_trigger();
  for (int p = blockIdx.x * (kRowThreads / 32) + warp; p < a.n; p += nw) {
    W4Row<NC> r;
    w4_warp_row<false>(r, a.x + (size_t)p * a.ldx, a.K, lane);
    r.store(a.xp + (size_t)p * a.ld, a.ld);
    if (lane == 0) a.xexp[p] = r.xe;
  }
}

// The same of few rows: `per` warps (a power of two) to a row, four loads a thread.
__global__ void __launch_bounds__(kRowThreads) w4_few_rows_kernel(const W4RowArgs a, int per) {
  constexpr int kWarps = kRowThreads / 32;
  __shared__ uint32_t s_max[2][kWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = warp & (per - 1), rows = kWarps / per;
  pdl_wait();
  pdl_trigger();
  int buf = 0;
  for (int p0 = blockIdx.x * rows; p0 < a.n; p0 += gridDim.x * rows, buf ^= 1) {
    const int p = min(p0 + warp / per, a.n - 1);  // (a last row may be done twice, with the same result)
    W4Row<4> r;
    uint32_t amax = __reduce_max_sync(MOE_FULL_MASK, r.load(a.x + (size_t)p * a.ldx, a.K, 32 * sub + lane, 32 * per));
    if (lane == 0) s_max[buf][warp] = amax;
    __syncthreads();
    for (int i = 0; i < per; ++i) amax = max(amax, s_max[buf][warp - sub + i]);
    r.scale<false>(amax);
    r.store(a.xp + (size_t)p * a.ld, a.ld);
    if (sub == 0 && lane == 0) a.xexp[p] = r.xe;
  }
}

// The exponents of row p: of x, of h, of y.
__device__ __forceinline__ void w4_row_exps(const W4RowArgs& a, int slot, int p, int xe, int ln) {
  const uint8_t* base = a.g.w + (size_t)slot * a.g.slab;
  // |h| <= |g| |u| <= |x|^2 |Wg| |Wu|; h 2^-hexp stays below 2^15
  const int b = ln + 2 * xe + w4_norm_exp(base + a.sl.gu.meta) + w4_norm_exp(base + a.sl.up_meta);
  const int he = min(max(b - 15, -126), 126);
  a.xexp[p] = xe;
  a.hexp[p] = he;
  a.yexp[p] = he + w4_y_exp(base + a.sl.dn_at, a.sl.dn);
  a.g.hcnt[p] = a.g.hmax[p] = 0;
}

// Zeros past a row of h.
__device__ __forceinline__ void w4_pad_h(const W4RowArgs& a, size_t p, int lane) {
  for (int c = a.sl.dn.K / 8 + lane; c < a.g.ldh / 8; c += 32)
    reinterpret_cast<uint4*>(a.g.h + p * a.g.ldh)[c] = make_uint4(0, 0, 0, 0);
}

template <int NC>
__global__ void __launch_bounds__(kRowThreads) w4_group_rows_kernel(const W4RowArgs a) {
  __shared__ int s_pre[kMaxE + 1];
  __shared__ int s_tmp[33];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = gridDim.x * (kRowThreads / 32);
  pdl_wait();
  pdl_trigger();
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.g.redo = 0;
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
        for (int c = lane; c < a.sl.dn.N / 4; c += 32)
          reinterpret_cast<float4*>(a.y + (size_t)p * a.sl.dn.N)[c] = make_float4(0.f, 0.f, 0.f, 0.f);
      continue;
    }
    W4Row<NC> r;
    const int ln = w4_warp_row<true>(r, a.x + (size_t)(a.rows[p] / a.k) * a.ldx, a.K, lane);
    r.store(a.xp + (size_t)p * a.ld, a.ld);
    w4_pad_h(a, p, lane);
    if (lane == 0) w4_row_exps(a, slot, p, r.xe, ln);
  }
}

// The same by token, where every slot is grouped: a row is read and scaled once and stored k times, its slots'
// exponents found by a lane each.  (4096 tokens of 2048, top 8: 26 us for the 128 MB it stores, 5.2 TB/s; by slot,
// with the same arithmetic eight times, 50 us.)
template <int NC>
__global__ void __launch_bounds__(kTokenThreads) w4_token_rows_kernel(const W4RowArgs a) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = gridDim.x * (kTokenThreads / 32);
  pdl_wait();
  pdl_trigger();
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.g.redo = 0;
  for (int t = blockIdx.x * (kTokenThreads / 32) + warp; t < a.n; t += nw) {
    W4Row<NC> r;
    const int ln = w4_warp_row<true>(r, a.x + (size_t)t * a.ldx, a.K, lane);
    for (int j0 = 0; j0 < a.k; j0 += 32) {
      int p = j0 + lane < a.k ? a.pos[(size_t)t * a.k + j0 + lane] : -1;  // -1: not an expert
      if (p >= 0) {
        const int e = a.ids[(size_t)t * a.k + j0 + lane], slot = a.g.e2s ? a.g.e2s[e] : e;
        if (slot >= 0 && slot < a.g.S) {
          w4_row_exps(a, slot, p, r.xe, ln);
        } else {
          set_status(a.g.status, MOE_DEV_BAD_SLOT);
          a.yexp[p] = kNoRow;
          p = -1;
        }
      }
      for (unsigned m = __ballot_sync(MOE_FULL_MASK, p >= 0); m; m &= m - 1) {
        const size_t at = __shfl_sync(MOE_FULL_MASK, p, __ffs(m) - 1);
        r.store(a.xp + at * a.ld, a.ld);
        w4_pad_h(a, at, lane);
      }
    }
  }
}

// out[t] = bf16(sum_j w[t][j] y[pos[t][j]]) from the scaled fp16 rows, fp32, j ascending; 8 columns a thread.
// Bound by memory: 144 MB for 4096 tokens of 2048, top 8, in 31 us (4.7 TB/s; with eight rows in flight 35 us).
__global__ void __launch_bounds__(128) w4_combine_kernel(const uint16_t* __restrict__ yh,
                                                         const int32_t* __restrict__ yexp,
                                                         const float* __restrict__ w, const int32_t* __restrict__ pos,
                                                         int k, int H, uint16_t* __restrict__ out) {
  const int t = blockIdx.x, c = (blockIdx.y * 128 + threadIdx.x) * 8;
  pdl_wait();
  if (c >= H) return;
  float acc[8] = {};
  for (int j0 = 0; j0 < k; j0 += 4) {  // four rows in flight
    int p[4], e[4];
    float wj[4];
    uint4 v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) p[j] = j0 + j < k ? pos[(size_t)t * k + j0 + j] : -1;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      e[j] = p[j] >= 0 ? yexp[p[j]] : kNoRow;
      wj[j] = p[j] >= 0 ? w[(size_t)t * k + j0 + j] : 0.f;
      if (p[j] >= 0) v[j] = __ldcs(reinterpret_cast<const uint4*>(yh + (size_t)p[j] * H + c));
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (e[j] == kNoRow) continue;
      const float we = ldexpf(wj[j], e[j] / 2), m = ldexpf(1.f, e[j] - e[j] / 2);  // 2^e may overflow by itself
      const uint32_t u[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
        acc[2 * i] = fmaf(we, f.x * m, acc[2 * i]);
        acc[2 * i + 1] = fmaf(we, f.y * m, acc[2 * i + 1]);
      }
    }
  }
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = uint32_t(f32_to_bf16(acc[2 * i])) | (uint32_t(f32_to_bf16(acc[2 * i + 1])) << 16);
  uint16_t* at = out + (size_t)t * H + c;
  if ((uintptr_t)at % 16 == 0) {
    *reinterpret_cast<uint4*>(at) = make_uint4(o[0], o[1], o[2], o[3]);
  } else {  // out is 8-byte aligned
    *reinterpret_cast<uint2*>(at) = make_uint2(o[0], o[1]);
    *reinterpret_cast<uint2*>(at + 4) = make_uint2(o[2], o[3]);
  }
}

constexpr size_t kGSmem = 1024 + (size_t)kGSets * kGVisit * kGXBytes + (size_t)kGWRing * kGWBytes +
                          (size_t)kGWorkers * kGEpiBytes + 64 * sizeof(uint64_t);
static_assert(kGSmem <= 222 * 1024, "shared memory of a CTA, with the 4.3 KB of static arrays");

// [n][ld] 16-bit rows as [stages][n][64]; what lies outside reads as 0.
static int row_maps(W4RowMaps* rm, const void* base, int n, int K, unsigned boxes) {
  const uint64_t ld = w4g_ld(K), d[3] = {kGK, (uint64_t)n, ld / kGK}, s[2] = {ld * 2, kGK * 2};
  for (int i = 0; i < kGBoxes; ++i) {
    if (!(boxes >> i & 1)) continue;
    const uint32_t b[3] = {kGK, 16u * (i + 1), kGVisit};
    const int r = encode_tmap_3d_bf16(&rm->m[i], base, d, s, b, CU_TENSOR_MAP_SWIZZLE_128B);
    if (r != MOE_OK) return r;
  }
  return MOE_OK;
}

// Persistent CTA pairs: as many clusters of two as fit at once (one CTA per SM).
template <int kMode>
static int launch_gemm(const W4GemmArgs& g, const void* rows, cudaStream_t s) {
  static bool done[64] = {};
  static int clusters[64] = {};
  MOE_CUDA_TRY(ensure_smem(w4_gemm_kernel<kMode>, (int)kGSmem, done));
  int dev = 0;
  MOE_CUDA_TRY(cudaGetDevice(&dev));
  // one matrix has full row tiles and a last one; groups have any
  unsigned boxes = (1u << kGBoxes) - 1;
  if (kMode == kLinear) {
    boxes = g.n >= kGN ? 1u << (kGBoxes - 1) : 0;
    if (g.n % kGN) boxes |= 1u << (w4g_half(g.n % kGN) / 16 - 1);
  }
  W4RowMaps m = {};
  if (row_maps(&m, rows, g.n, g.K, boxes) != MOE_OK) return MOE_ERR_CUDA;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kGThreads);
  cfg.dynamicSmemBytes = kGSmem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if (clusters[dev] == 0) {
    int sms = 0, n = 0;
    MOE_CUDA_TRY(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev));
    cfg.gridDim = dim3((unsigned)(sms & ~1));
    MOE_CUDA_TRY(cudaOccupancyMaxActiveClusters(&n, (void*)w4_gemm_kernel<kMode>, &cfg));
    if (n < 1) return MOE_ERR_CUDA;
    clusters[dev] = n;
  }
  cfg.gridDim = dim3((unsigned)(2 * clusters[dev]));
  MOE_CUDA_TRY(cudaLaunchKernelEx(&cfg, w4_gemm_kernel<kMode>, g, m));
  return MOE_OK;
}

static size_t g256(size_t v) { return (v + 255) & ~size_t(255); }

// Parts of the inputs: where there are fewer tiles than pairs of SMs, as many as there are pairs for, of kGPart
// stages or more, kGMostParts at most: each adds its sums to write and read.  (256 rows through 4096 x 4096, four
// parts: 17.2 us, undivided 26.4; 8192 x 1024, eight parts of 16 stages 17.7, sixteen of 8 20.0, undivided 42.9;
// 2048 x 2048, four parts of 8 stages 13.7, two of 16 15.0, undivided 17.9.)
constexpr int kGPairs = 76, kGPart = 8, kGMostParts = 8;
static void w4_parts(int T, const W4Dims& d, int& parts, int& stages) {
  const int64_t tiles = (int64_t)((T + kGN - 1) / kGN) * ((d.N + 2 * kGM - 1) / (2 * kGM));
  parts = (int)std::min<int64_t>(kGPairs / tiles, std::min(d.Kb / kGPart, kGMostParts));
  stages = parts < 2 ? d.Kb : ((d.Kb + parts - 1) / parts + kGVisit - 1) / kGVisit * kGVisit;
  parts = (d.Kb + stages - 1) / stages;
}
static int w4_part_ld(int N) { return (N + 3) & ~3; }

// Enough for any number of rows up to T: parts x rows <= kGPairs / (column tiles) x min(T, kGN).
size_t w4_linear_gemm_ws(int T, const W4Dims& d) {
  const size_t nf = (d.N + 2 * kGM - 1) / (2 * kGM);
  return g256(2 * (size_t)T * w4g_ld(d.K)) + g256(4 * (size_t)T) +
         (2 * nf > kGPairs ? 0 : 4 * (kGPairs / nf) * std::min(T, kGN) * w4_part_ld(d.N));
}

// out = the sums of the parts, in order, times the row's power of two; four columns a thread.
__global__ void __launch_bounds__(256) w4_parts_kernel(const float* __restrict__ part, const int32_t* __restrict__ rexp,
                                                       int parts, int T, int N, int ldp, void* out, size_t ldo,
                                                       int out_f32) {
  const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x, per = ldp / 4, t = i / per, c = (i - t * per) * 4;
  pdl_wait();
  if (t >= (size_t)T) return;
  const float* p = part + t * ldp + c;
  float4 s = __ldcs(reinterpret_cast<const float4*>(p));
#pragma unroll 4
  for (int j = 1; j < parts; ++j) {
    const float4 v = __ldcs(reinterpret_cast<const float4*>(p + (size_t)j * T * ldp));
    s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
  }
  const float m = pow2(rexp[t]);
  s.x *= m, s.y *= m, s.z *= m, s.w *= m;
  const float v[4] = {s.x, s.y, s.z, s.w};
  const size_t at = t * ldo + c;
  if (out_f32) {
    float* o = reinterpret_cast<float*>(out) + at;
    if ((uintptr_t)o % 16 == 0 && c + 4 <= (size_t)N) {
      *reinterpret_cast<float4*>(o) = s;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (c + j < (size_t)N) o[j] = v[j];
    }
  } else {
    uint16_t* o = reinterpret_cast<uint16_t*>(out) + at;
    if ((uintptr_t)o % 8 == 0 && c + 4 <= (size_t)N) {
      *reinterpret_cast<uint2*>(o) = make_uint2(pack_bf16(s.x, s.y), pack_bf16(s.z, s.w));
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (c + j < (size_t)N) o[j] = f32_to_bf16(v[j]);
    }
  }
}

int launch_w4_linear_gemm(const uint16_t* x, size_t ldx, int T, const uint8_t* w, const W4Dims& d, void* out,
                          size_t ldo, int out_f32, void* ws, int32_t* status, cudaStream_t s) {
  W4RowArgs r{};
  r.x = x, r.ldx = ldx, r.n = T, r.K = d.K;
  r.xp = (uint16_t*)ws, r.ld = w4g_ld(d.K);
  r.xexp = (int32_t*)((char*)ws + g256(2 * (size_t)T * r.ld));
  // a warp to a row while there is a row for every scheduler twice; several warps where a row's latency is what
  // counts (33 rows of 4096: 15.6 us with one, 12.7 with four; 4096 rows of 2048: 53.5 with one, 55 with two)
  if (T >= 1216) {
    MOE_CUDA_TRY(launch_pdl(d.K <= 2048 ? w4_rows_kernel<8> : w4_rows_kernel<16>, dim3(std::min((T + 7) / 8, 1216)),
                            dim3(kRowThreads), 0, s, r));
  } else {
    const int per = d.K <= 1024 ? 1 : d.K <= 2048 ? 2 : d.K <= 4096 ? 4 : 8, rows = kRowThreads / 32 / per;
    MOE_CUDA_TRY(launch_pdl(w4_few_rows_kernel, dim3((T + rows - 1) / rows), dim3(kRowThreads), 0, s, r, per));
  }
  W4GemmArgs g{};
  g.w = w, g.d = d, g.K = d.K, g.n = T;
  g.NF = (d.N + 2 * kGM - 1) / (2 * kGM);
  g.status = status, g.rexp = r.xexp;
  g.out = out, g.ldo = ldo, g.out_f32 = out_f32;
  w4_parts(T, d, g.parts, g.stages);
  if (g.parts == 1) return launch_gemm<kLinear>(g, r.xp, s);
  float* part = (float*)((char*)r.xexp + g256(4 * (size_t)T));
  const int ldp = w4_part_ld(d.N);
  g.out = part, g.ldo = ldp, g.out_f32 = 1;
  const int rc = launch_gemm<kLinear>(g, r.xp, s);
  if (rc != MOE_OK) return rc;
  MOE_CUDA_TRY(launch_pdl(w4_parts_kernel, dim3((unsigned)(((size_t)T * (ldp / 4) + 255) / 256)), dim3(256), 0, s,
                          (const float*)part, (const int32_t*)r.xexp, g.parts, T, d.N, ldp, out, ldo, out_f32));
  return MOE_OK;
}

// Workspace: x' [n][H] and h [n][I] fp16 in whole stages, exponents, what tells of small h, and y [n][H] fp16 where the caller combines.
size_t w4_ffn_gemm_ws(size_t n, int H, int I, bool yh) {
  return g256(2 * n * w4g_ld(H)) + g256(2 * n * w4g_ld(I)) + 5 * g256(4 * n) + 256 + (yh ? g256(2 * n * H) : 0);
}

// y rows of the listed experts (fp32 f.y, or scaled fp16 with *yh / *yexp set for launch_w4_combine).  ids and pos:
// every slot's expert and row, where the list holds every expert with rows (else NULL).
int launch_ffn_w4_gemm(const FfnArgs& f, const int32_t* ids, const int32_t* pos, int group, void* ws,
                       const uint16_t** yh, const int32_t** yexp, cudaStream_t s, Prof* prof) {
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
  r.ld = w4g_ld(f.H);
  r.xp = (uint16_t*)take(2 * n * r.ld);
  uint16_t* h = (uint16_t*)take(2 * n * w4g_ld(f.I));
  r.xexp = (int32_t*)take(4 * n);
  r.hexp = (int32_t*)take(4 * n);
  r.yexp = (int32_t*)take(4 * n);
  int32_t *hcnt = (int32_t*)take(4 * n), *hmax = (int32_t*)take(4 * n), *redo = (int32_t*)take(4);
  W4GemmArgs g{};
  g.w = (const uint8_t*)f.pool, g.slab = sl.bytes, g.d = sl.gu, g.mat = 0;
  g.K = f.H, g.n = (int)n, g.NF = (2 * f.I + 2 * kGM - 1) / (2 * kGM);
  g.offset = f.offset, g.list_e = f.list_e, g.n_list = f.n_list, g.e2s = f.e2s, g.list_s = f.list_s;
  g.E = f.E, g.S = f.S, g.status = f.status;
  g.rexp = r.xexp, g.oexp = r.hexp, g.h = h, g.ldh = w4g_ld(f.I);
  g.hcnt = hcnt, g.hmax = hmax, g.redo = redo, g.yexp = r.yexp;
  r.g = g, r.rows = f.rows, r.k = f.k, r.sl = sl;
  r.y = yh ? nullptr : f.y;
  if (prof) prof->begin(MOE_PROF_FFN_ROWS, s);
  if (ids) {
    r.ids = ids, r.pos = pos, r.n = f.T;
    MOE_CUDA_TRY(launch_pdl(f.H <= 2048 ? w4_token_rows_kernel<8> : w4_token_rows_kernel<16>,
                            dim3((unsigned)std::min((f.T + 3) / 4, 2432)), dim3(kTokenThreads), 0, s, r));
  } else {
    MOE_CUDA_TRY(launch_pdl(f.H <= 2048 ? w4_group_rows_kernel<8> : w4_group_rows_kernel<16>,
                            dim3((unsigned)std::min((n + 7) / 8, (size_t)1216)), dim3(kRowThreads), 0, s, r));
  }
  if (prof) prof->end(s);
  if (prof) prof->begin(MOE_PROF_FFN_GATEUP, s);
  int rc = launch_gemm<kGateUp>(g, r.xp, s);
  if (rc == MOE_OK) rc = launch_gemm<kRedo>(g, r.xp, s);
  if (rc != MOE_OK) return rc;
  if (prof) prof->end(s);
  W4GemmArgs gd = g;
  gd.d = sl.dn, gd.mat = sl.dn_at;
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
  MOE_CUDA_TRY(launch_pdl(w4_combine_kernel, dim3(T, (H / 8 + 127) / 128), dim3(128), 0, s, yh, yexp, w, pos, k, H,
                          (uint16_t*)out));
  return MOE_OK;
}

}  // namespace moe
