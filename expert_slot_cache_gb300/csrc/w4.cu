// Products with 4-bit weights and group scales (format: w4.cuh): the linear layer and the grouped
// SwiGLU expert FFN.
//
//   y[t][n] = sum_k x[t][k] (code[k][n] - 8) scale[k / G][n]
//
// The codes become the A operand of 16 x 16 x 8 MMAs as exact bf16 integers, the bf16 activations the B
// operand; a 64-input block's products (32 inputs where G = 32) are summed in fp32 by the tensor core,
// then multiplied by their fp32 scale and added in fp32.  No weight and no activation is rounded.
#include <algorithm>

#include "internal.cuh"
#include "w4.cuh"

namespace moe {

constexpr int kW4Warps = 8;
constexpr int kW4Threads = 32 * kW4Warps;

// One matrix's view for a tile: lane's code words, the tile's scale words, the multipliers.
struct W4Tile {
  const uint4* codes;      // + kb * 32 * mates
  const uint32_t* scales;  // + kg * 8 * mates
  int mates;
};

__device__ __forceinline__ W4Tile w4_tile(const uint8_t* m, const W4Dims& d, int tile, int lane) {
  W4Tile t;
  t.codes = reinterpret_cast<const uint4*>(m) + w4_code_at(d, tile, 0) * 32 + w4_chunk(lane >> 2, lane & 3);
  t.scales = reinterpret_cast<const uint32_t*>(m + d.scales) + w4_scale_at(d, tile, 0) * 8 + (lane >> 2);
  t.mates = w4_mates(d, tile);
  return t;
}

// acc[m][nb] += tile products of blocks [kb0, kb1): NM matrices that share the rows of x, NB groups of
// eight rows.  xr[nb]: the lane's row (column lane >> 2 of the group), already offset by 8 * (lane & 3).
// LO: the rows come as a sum of two bf16 arrays, xr[nb] and xr[nb] + lo.
template <int NM, int NB, bool LO>
__device__ __forceinline__ void w4_accumulate(const W4Tile (&t)[NM], const uint16_t* const (&xr)[NB], size_t lo,
                                              int K, int G, int kb0, int kb1, int q, float (&acc)[NM][NB][4]) {
#pragma unroll 2
  for (int kb = kb0; kb < kb1; ++kb) {
    uint4 w[NM];
#pragma unroll
    for (int m = 0; m < NM; ++m) w[m] = ldg_stream(t[m].codes + (size_t)kb * (32 * t[0].mates));
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = kb * 64 + 32 * h;
      const bool in = k + 8 * q < K;  // K % 8 == 0: a lane's eight inputs are inside or outside together
      uint4 x[NB], xl[NB];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        x[nb] = in ? __ldg(reinterpret_cast<const uint4*>(xr[nb] + k)) : make_uint4(0, 0, 0, 0);
        if (LO) xl[nb] = in ? __ldg(reinterpret_cast<const uint4*>(xr[nb] + lo + k)) : make_uint4(0, 0, 0, 0);
      }
      const int kg = k / G;
#pragma unroll
      for (int m = 0; m < NM; ++m) {
        uint32_t a0[4], a1[4];
        w4_frag_bf16(h ? w[m].y : w[m].x, h ? w[m].w : w[m].z, a0, a1);
        const uint32_t sw = __ldg(t[m].scales + (size_t)kg * (8 * t[0].mates));
        const float2 s = __half22float2(*reinterpret_cast<const __half2*>(&sw));
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          float c[4] = {0.f, 0.f, 0.f, 0.f};
          mma_bf16_16816(c, a0, x[nb].x, x[nb].y);
          mma_bf16_16816(c, a1, x[nb].z, x[nb].w);
          if (LO) {
            mma_bf16_16816(c, a0, xl[nb].x, xl[nb].y);
            mma_bf16_16816(c, a1, xl[nb].z, xl[nb].w);
          }
          acc[m][nb][0] = fmaf(s.x, c[0], acc[m][nb][0]);
          acc[m][nb][1] = fmaf(s.x, c[1], acc[m][nb][1]);
          acc[m][nb][2] = fmaf(s.y, c[2], acc[m][nb][2]);
          acc[m][nb][3] = fmaf(s.y, c[3], acc[m][nb][3]);
        }
      }
    }
  }
}

// Sum of the `ks` warps' accumulators of one tile, parts in warp order: red[warp][m][nb][4][32].
// Element (i, lane) is column (lane >> 2) + 8 * (i >> 1), row 2 * (lane & 3) + (i & 1).
template <int NM, int NB>
__device__ __forceinline__ void w4_store_part(float* red, int warp, int lane, const float (&acc)[NM][NB][4]) {
#pragma unroll
  for (int m = 0; m < NM; ++m)
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int i = 0; i < 4; ++i) red[(((warp * NM + m) * NB + nb) * 4 + i) * 32 + lane] = acc[m][nb][i];
}

template <int NM, int NB>
__device__ __forceinline__ float w4_sum_part(const float* red, int w0, int ks, int m, int row, int col) {
  const int nb = row >> 3, i = 2 * (col >> 3) + (row & 1), lane = 4 * (col & 7) + ((row & 7) >> 1);
  float s = 0.f;
  for (int w = 0; w < ks; ++w) s += red[((((w0 + w) * NM + m) * NB + nb) * 4 + i) * 32 + lane];
  return s;
}

struct W4LinArgs {
  const uint16_t* x;
  size_t ldx, ldo;
  int T, ks;  // ks warps share a tile
  const uint8_t* w;
  W4Dims d;
  void* out;
  int out_f32;
};

// grid (ceil(Mt / (8 / ks)), ceil(T / (8 NB))).
template <int NB>
__global__ void __launch_bounds__(kW4Threads) w4_linear_kernel(const W4LinArgs a) {
  __shared__ float red[kW4Warps * NB * 4 * 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int ks = a.ks, tpc = kW4Warps / ks;
  const int tile0 = blockIdx.x * tpc, tile = tile0 + warp / ks, part = warp % ks;
  const int t0 = blockIdx.y * 8 * NB, nt = min(8 * NB, a.T - t0);
  float acc[1][NB][4] = {};
  if (tile < a.d.Mt) {
    const uint16_t* xr[NB];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)  // rows past the batch repeat its last one; their results are dropped
      xr[nb] = a.x + (size_t)(t0 + min(8 * nb + (lane >> 2), nt - 1)) * a.ldx + 8 * (lane & 3);
    const W4Tile t[1] = {w4_tile(a.w, a.d, tile, lane)};
    const int per = (a.d.Kb + ks - 1) / ks;
    w4_accumulate<1, NB, false>(t, xr, 0, a.d.K, a.d.G, min(part * per, a.d.Kb), min((part + 1) * per, a.d.Kb),
                                lane & 3, acc);
  }
  w4_store_part<1, NB>(red, warp, lane, acc);
  __syncthreads();
  const float* mult = reinterpret_cast<const float*>(a.w + a.d.mult);
  for (int i = threadIdx.x; i < tpc * 16 * nt; i += kW4Threads) {
    const int col = i & 15, row = (i >> 4) % nt, tl = (i >> 4) / nt;
    const int n = (tile0 + tl) * 16 + col;
    if (n >= a.d.N) continue;
    const float v = w4_sum_part<1, NB>(red, tl * ks, ks, 0, row, col) * mult[n];
    const size_t o = (size_t)(t0 + row) * a.ldo + n;
    if (a.out_f32) reinterpret_cast<float*>(a.out)[o] = v;
    else reinterpret_cast<uint16_t*>(a.out)[o] = f32_to_bf16(v);
  }
}

struct W4FfnArgs {
  FfnArgs f;      // f.pool: bytes of the 4-bit slot pool
  W4Slab sl;
  uint16_t* h;    // bf16 [2][n][I]: h = h[0] + h[1]
  size_t n;
};

__device__ __forceinline__ bool w4_slot(const FfnArgs& a, int li, int& e, int& slot) {
  e = a.list_e[li];
  if (e < 0 || e >= a.E) return false;
  slot = a.list_s ? a.list_s[li] : a.e2s ? a.e2s[e] : e;
  return true;
}

// Gate and up: unit = (listed expert, tile of 16 h features); eight warps split the inputs.
template <int NB>
__global__ void __launch_bounds__(kW4Threads) w4_gateup_kernel(const W4FfnArgs a) {
  __shared__ float red[kW4Warps * 2 * NB * 4 * 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const W4Dims& d = a.sl.gu;
  const int nl = *a.f.n_list, FT = d.Mt / 2, I = d.N / 2;  // a tile of gate and its neighbour of up
  for (int u = blockIdx.x; u < nl * FT; u += gridDim.x) {
    int e, slot;
    if (!w4_slot(a.f, u / FT, e, slot)) continue;
    if (slot < 0 || slot >= a.f.S) {
      if (threadIdx.x == 0) set_status(a.f.status, MOE_DEV_BAD_SLOT);
      continue;
    }
    const int tile = u % FT, pe = a.f.offset[e + 1];
    const uint8_t* base = reinterpret_cast<const uint8_t*>(a.f.pool) + (size_t)slot * a.sl.bytes;
    const W4Tile t[2] = {w4_tile(base, d, 2 * tile, lane), w4_tile(base, d, 2 * tile + 1, lane)};
    const float* mg = reinterpret_cast<const float*>(base + d.mult) + tile * 32;
    const float* mu = mg + 16;
    const int per = (d.Kb + kW4Warps - 1) / kW4Warps;
    for (int p0 = a.f.offset[e]; p0 < pe; p0 += 8 * NB) {
      const int nt = min(8 * NB, pe - p0);
      const uint16_t* xr[NB];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
        xr[nb] = a.f.x + (size_t)(a.f.rows[p0 + min(8 * nb + (lane >> 2), nt - 1)] / a.f.k) * a.f.H + 8 * (lane & 3);
      float acc[2][NB][4] = {};
      w4_accumulate<2, NB, false>(t, xr, 0, d.K, d.G, min(warp * per, d.Kb), min((warp + 1) * per, d.Kb), lane & 3,
                                  acc);
      __syncthreads();
      w4_store_part<2, NB>(red, warp, lane, acc);
      __syncthreads();
      for (int i = threadIdx.x; i < 16 * nt; i += kW4Threads) {
        const int col = i & 15, row = i >> 4;
        const float g = w4_sum_part<2, NB>(red, 0, kW4Warps, 0, row, col) * mg[col];
        const float v = w4_sum_part<2, NB>(red, 0, kW4Warps, 1, row, col) * mu[col];
        const float h = g / (1.f + __expf(-g)) * v;
        // h as the sum of two bf16: 16 significant bits reach the down product
        const uint16_t hi = f32_to_bf16(h);
        const size_t o = (size_t)(p0 + row) * I + tile * 16 + col;
        a.h[o] = hi;
        a.h[a.n * I + o] = isfinite(bf16_to_f32(hi)) ? f32_to_bf16(h - bf16_to_f32(hi)) : 0;
      }
    }
  }
}

// Down: unit = (listed expert, two tiles of 16 output columns); four warps split the inputs of a tile.
template <int NB>
__global__ void __launch_bounds__(kW4Threads) w4_down_kernel(const W4FfnArgs a) {
  constexpr int KS = 4, TPC = kW4Warps / KS;
  __shared__ float red[kW4Warps * NB * 4 * 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const W4Dims& d = a.sl.dn;
  const int nl = *a.f.n_list, FT = (d.Mt + TPC - 1) / TPC;
  for (int u = blockIdx.x; u < nl * FT; u += gridDim.x) {
    int e, slot;
    if (!w4_slot(a.f, u / FT, e, slot)) continue;
    const int tile0 = u % FT * TPC, tile = tile0 + warp / KS, part = warp % KS, pe = a.f.offset[e + 1];
    const bool ok = slot >= 0 && slot < a.f.S;
    const uint8_t* base =
        reinterpret_cast<const uint8_t*>(a.f.pool) + (size_t)(ok ? slot : 0) * a.sl.bytes + a.sl.dn_at;
    const float* mult = reinterpret_cast<const float*>(base + d.mult);
    const int per = (d.Kb + KS - 1) / KS;
    for (int p0 = a.f.offset[e]; p0 < pe; p0 += 8 * NB) {
      const int nt = min(8 * NB, pe - p0);
      float acc[1][NB][4] = {};
      if (ok && tile < d.Mt) {
        const W4Tile t[1] = {w4_tile(base, d, tile, lane)};
        const uint16_t* xr[NB];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
          xr[nb] = a.h + (size_t)(p0 + min(8 * nb + (lane >> 2), nt - 1)) * d.K + 8 * (lane & 3);
        w4_accumulate<1, NB, true>(t, xr, a.n * d.K, d.K, d.G, min(part * per, d.Kb), min((part + 1) * per, d.Kb),
                                   lane & 3, acc);
      }
      __syncthreads();
      w4_store_part<1, NB>(red, warp, lane, acc);
      __syncthreads();
      for (int i = threadIdx.x; i < TPC * 16 * nt; i += kW4Threads) {
        const int col = i & 15, row = (i >> 4) % nt, tl = (i >> 4) / nt, n = (tile0 + tl) * 16 + col;
        // an expert without a slot adds nothing: its rows are zero
        if (n < d.N)
          a.f.y[(size_t)(p0 + row) * d.N + n] = ok ? w4_sum_part<1, NB>(red, tl * KS, KS, 0, row, col) * mult[n] : 0.f;
      }
    }
  }
}

static int w4_sms(int* sms) {
  int dev = 0;
  MOE_CUDA_TRY(cudaGetDevice(&dev));
  MOE_CUDA_TRY(cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev));
  return MOE_OK;
}

// Rows from which the tensor-core path takes over.
constexpr int kGemmRows = 512;

static bool w4_gemm_ffn(int n) { return n >= kGemmRows; }

size_t w4_ws_bytes(int n, int H, int I) {
  const size_t h = ((size_t)n * I * 4 + 255) & ~size_t(255);
  return w4_gemm_ffn(n) ? std::max(h, w4_ffn_gemm_ws(n, H, I, false)) : h;
}

// y rows of the listed experts; ws holds h (w4_ws_bytes).
int launch_ffn_w4(const FfnArgs& f, int group, void* ws, size_t ws_bytes, int max_list, cudaStream_t stream,
                  Prof* prof) {
  const int n = f.T * f.k;
  if (ws_bytes < w4_ws_bytes(n, f.H, f.I)) return MOE_ERR_ALIGN;
  if (max_list <= 0) return MOE_OK;
  if (w4_gemm_ffn(n)) return launch_ffn_w4_gemm(f, group, ws, nullptr, nullptr, stream, prof);
  int sms = 0;
  const int r = w4_sms(&sms);
  if (r != MOE_OK) return r;
  W4FfnArgs a{f, w4_slab(f.H, f.I, group), (uint16_t*)ws, (size_t)n};
  const int g1 = std::min(max_list * (a.sl.gu.Mt / 2), sms * 8), g2 = std::min(max_list * ((a.sl.dn.Mt + 1) / 2), sms * 8);
  if (prof) prof->begin(MOE_PROF_FFN_GATEUP, stream);
  if (f.T <= 8) w4_gateup_kernel<1><<<g1, kW4Threads, 0, stream>>>(a);
  else w4_gateup_kernel<2><<<g1, kW4Threads, 0, stream>>>(a);
  MOE_LAUNCH_CHECK();
  if (prof) prof->end(stream);
  if (prof) prof->begin(MOE_PROF_FFN_DOWN, stream);
  if (f.T <= 8) w4_down_kernel<1><<<g2, kW4Threads, 0, stream>>>(a);
  else w4_down_kernel<2><<<g2, kW4Threads, 0, stream>>>(a);
  MOE_LAUNCH_CHECK();
  if (prof) prof->end(stream);
  return MOE_OK;
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
  const bool gemm = w4_gemm_ffn(n);  // its y is fp16 inside its own workspace
  w.y = gemm ? nullptr : (float*)take(4 * (size_t)n * H);
  w.ffn_bytes = gemm ? w4_ffn_gemm_ws(n, H, I, true) : w4_ws_bytes(n, H, I);
  w.ffn = take(w.ffn_bytes);
  w.bytes = off;
  return w;
}

static bool w4_gemm_linear(int T) { return T >= 64; }

// Routing slots and hidden sizes whose products the kernels index with 32 bits.
static bool w4_rows_ok(int T, int k) { return (int64_t)T * k <= (1 << 24); }

}  // namespace moe

using namespace moe;

extern "C" size_t moe_w4_linear_workspace_bytes(int T, int K, int N, int group) {
  if (T < 1 || !w4_shape_ok(K, N, group)) return 0;
  return w4_gemm_linear(T) ? w4_linear_gemm_ws(T, K) : 0;
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
  if (w4_gemm_linear(T))
    return launch_w4_linear_gemm((const uint16_t*)x, (size_t)ldx, T, (const uint8_t*)w, w4_dims(K, N, group), out,
                                 (size_t)ldo, out_f32, workspace, dev_status, (cudaStream_t)stream);
  int sms = 0;
  const int r = w4_sms(&sms);
  if (r != MOE_OK) return r;
  W4LinArgs a{(const uint16_t*)x, (size_t)ldx, (size_t)ldo, T, 1, (const uint8_t*)w, w4_dims(K, N, group), out, out_f32};
  while (a.ks < kW4Warps && a.d.Mt * a.ks < sms * 32) a.ks *= 2;
  const int gx = (a.d.Mt + kW4Warps / a.ks - 1) / (kW4Warps / a.ks);
  const int rows = T <= 8 ? 8 : T <= 16 ? 16 : 32;
  for (int t0 = 0; t0 < T; t0 += 65535 * rows) {  // the grid's y
    W4LinArgs b = a;
    b.x += (size_t)t0 * ldx;
    b.out = (char*)out + (size_t)t0 * ldo * (out_f32 ? 4 : 2);
    b.T = std::min(T - t0, 65535 * rows);
    const dim3 grid(gx, (b.T + rows - 1) / rows);
    if (rows == 8) w4_linear_kernel<1><<<grid, kW4Threads, 0, (cudaStream_t)stream>>>(b);
    else if (rows == 16) w4_linear_kernel<2><<<grid, kW4Threads, 0, (cudaStream_t)stream>>>(b);
    else w4_linear_kernel<4><<<grid, kW4Threads, 0, (cudaStream_t)stream>>>(b);
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
  return w4_exp_ws(nullptr, T, H, I, k, E).bytes;
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
  int r = launch_permute(ids, n, E, ws.count, ws.offset, ws.rows, ws.pos, ws.act_e, ws.n_act, dev_status, ws.perm, s);
  if (r != MOE_OK) return r;
  FfnArgs f{};
  f.x = (const uint16_t*)x;
  f.T = T, f.H = H, f.I = I, f.k = k, f.E = E;
  f.offset = ws.offset, f.rows = ws.rows, f.list_e = ws.act_e, f.n_list = ws.n_act;
  f.pool = (const uint16_t*)pool, f.e2s = e2s, f.S = S, f.pool_only = 1;
  f.y = ws.y, f.status = dev_status;
  if (w4_gemm_ffn(n)) {
    const uint16_t* yh = nullptr;
    const int32_t* yexp = nullptr;
    if ((r = launch_ffn_w4_gemm(f, group, ws.ffn, &yh, &yexp, s, nullptr)) != MOE_OK) return r;
    return launch_w4_combine(yh, yexp, w, ws.pos, T, k, H, out, s);
  }
  if ((r = launch_ffn_w4(f, group, ws.ffn, ws.ffn_bytes, std::min(n, E), s, nullptr)) != MOE_OK) return r;
  return launch_combine(ws.y, w, ws.pos, ids, nullptr, T, k, H, E, 0, out, nullptr, nullptr, s);
}
