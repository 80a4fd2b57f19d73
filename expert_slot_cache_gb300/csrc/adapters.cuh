// Low-rank adapters beside a shared projection: arguments and launchers shared by adapters.cu and its kernels.
#pragma once

#include "internal.cuh"
#include "tc05.cuh"

namespace moe {

constexpr int kAdMaxR = 128;

// out = base + (scale_l x W1_l^T) W2_l over the rows of each sequence; the gradient's dx is the same with dy for x, W1
// and W2 exchanged.
struct AdArgs {
  const uint16_t* x;   // [T] rows of K, ldx apart
  const uint16_t* w1;  // [L][R][K]
  const uint16_t* w2;  // [L][R][N]
  const float* scale;  // [L]
  const int32_t* ids;  // [n_seq], -1: no adapter
  const int32_t* seq;  // [n_seq + 1] or NULL: row t is sequence t
  const void* base;    // [T] rows of N, ldb apart, or NULL
  void* out;           // [T] rows of N, ldo apart, or NULL: the product x W1^T alone
  float* kept;         // [T][R] scale_l x W1_l^T, or NULL
  const float* fwd;    // [T][R] or NULL: the forward pass's values,
  uint16_t* parts;     // which go, with this pass's, into bf16 [2][T][3 Rk]: three numbers each (or NULL)
  int32_t* status;
  long long ldx, ldb, ldo;
  int T, K, N, R, L, n_seq;
};

// The adapter of sequence s, or -1 (flagged, where it is neither one nor -1).
__device__ __forceinline__ int ad_adapter(const AdArgs& a, int s) {
  const int l = a.ids[s];
  if (l < -1 || l >= a.L) set_status(a.status, MOE_DEV_BAD_EXPERT);
  return l < a.L ? l : -1;
}

// The sequence of row t: the last s with seq[s] <= t < seq[s + 1]; -1 for a row in none.
__device__ __forceinline__ int ad_sequence(const AdArgs& a, int t) {
  if (!a.seq) return t;
  int lo = 0, hi = a.n_seq + 1;  // the first s with seq[s] > t lies in [lo, hi]
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (a.seq[mid] > t) hi = mid;
    else lo = mid + 1;
  }
  return lo >= 1 && lo <= a.n_seq ? lo - 1 : -1;
}

// The sequences of more than short_rows rows (and the rows of none), by tiles.
int ad_launch_tiles(const AdArgs& a, bool f32, int short_rows, bool beside, cudaStream_t s);

// v as a sum of three bf16 numbers, eight values at once (packed pairs): truncation leaves an exact rest, so that they are
// all 24 bits.  A rest of an infinity or a NaN counts as 0.
__device__ __forceinline__ void ad_split8(const float (&v)[8], uint4 (&o)[3]) {
  uint32_t w[3][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float x = v[2 * i], y = v[2 * i + 1];
#pragma unroll
    for (int s = 0; s < 3; ++s) {
      if (s == 2) {
        const __nv_bfloat162 q = __floats2bfloat162_rn(x, y);
        w[s][i] = *reinterpret_cast<const uint32_t*>(&q);
      } else {
        const uint32_t xb = __float_as_uint(x) & 0xffff0000u, yb = __float_as_uint(y) & 0xffff0000u;
        w[s][i] = (xb >> 16) | yb;
        x = fabsf(x) < INFINITY ? x - __uint_as_float(xb) : 0.f;
        y = fabsf(y) < INFINITY ? y - __uint_as_float(yb) : 0.f;
      }
    }
  }
#pragma unroll
  for (int s = 0; s < 3; ++s) o[s] = make_uint4(w[s][0], w[s][1], w[s][2], w[s][3]);
}

// Values c .. c + 7 of a row (R of them; zeros beyond) as three numbers each, [first | second | third][Rk].
__device__ __forceinline__ void ad_put_parts(uint16_t* row, int Rk, int c, const float (&v)[8]) {
  uint4 o[3];
  ad_split8(v, o);
#pragma unroll
  for (int k = 0; k < 3; ++k) *reinterpret_cast<uint4*>(row + k * Rk + c) = o[k];
}
__device__ __forceinline__ void ad_load8(const float* row, int R, int c, float (&v)[8]) {
  const float* p = row + c;
  if (c + 8 <= R && (reinterpret_cast<uintptr_t>(p) & 15) == 0) {
    const float4 x = reinterpret_cast<const float4*>(p)[0], y = reinterpret_cast<const float4*>(p)[1];
    v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w, v[4] = y.x, v[5] = y.y, v[6] = y.z, v[7] = y.w;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = c + j < R ? p[j] : 0.f;
  }
}

// Bounded wait of a whole warp; false after a timeout, its own (flagged) or another warp's.
__device__ __forceinline__ bool ad_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int32_t* status) {
  for (int i = 0; i < kWaitPolls; ++i) {
    if (__all_sync(MOE_FULL_MASK, mbar_try_wait(bar, parity))) return true;
    if ((i & 255) == 255 && __any_sync(MOE_FULL_MASK, *abort_flag)) return false;
  }
  *abort_flag = 1;
  set_status(status, MOE_DEV_TIMEOUT);
  return false;
}

struct AdGradArgs {
  const uint16_t* x;   // [T] rows of K
  const uint16_t* dy;  // [T] rows of N
  const float* dv;     // [T][R]
  const float* v;      // [T][R]
  const int32_t* ids;
  const int32_t* seq;
  float* da;           // [L][R][K]
  float* db;           // [L][R][N]
  const uint16_t* parts;  // bf16 [2][T][3 Rk]: dv and v as three numbers each, for the rows of adapters, or NULL
  int32_t* status;
  long long ldx, ldy;
  int T, K, N, R, L, n_seq;
  int both;  // both kernels are launched, each takes its adapters
};

// Which kernel computes dA and dB: tiles from 16 rows a sequence on, counted by adapter over the sequences that have rows.
// The host knows it where all sequences together are that long; else both kernels are launched and find out by themselves:
// 8192 rows in two sequences and 1022 empty ones (2048 x 4096, R 32) take 137 us, 1,075 where empty ones counted; 2400 rows in
// 300 sequences 216, 207 without the launch that they do not need.  Below 512 rows that launch (4 us of 42 for 400 rows) costs
// about what it could save.
enum class AdOuter { kShort, kTiles, kBoth };
constexpr int kAdLong = 16;
inline AdOuter ad_outer_by(int T, int n_seq, const int32_t* seq) {
  return !seq ? AdOuter::kShort : T >= (long long)kAdLong * n_seq ? AdOuter::kTiles : T >= 512 ? AdOuter::kBoth : AdOuter::kShort;
}
// dA and dB.
int ad_launch_outer(const AdGradArgs& a, int sms, cudaStream_t s);

}  // namespace moe
