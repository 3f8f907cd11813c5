// RMS norms around the scan of a Mamba-2 block on gfx950.
//
// Before a block (pre-norm with the residual update; Mamba-3-Lite block page:
// RMSNorm, pre-norm, eps 1e-5):
//   r = residual + scale o x
//   out = r rsqrt(mean(r^2) + eps) o w
// and its gradient at the given r, with n = r rstd, dn = dout o w:
//   g = dres + rstd (dn - n mean(dn o n))
//   dresidual = g, dx = scale o g, dw = sum_rows dout o n, dscale = sum_rows g o x
//
// After the scan (the Mamba-2 layer's norm between the scan and out_proj), per
// group of L = D / groups channels, s = silu(z):
//   out = rms(y o s) o w            or, norm_before_gate,  rms(y) o w o s
// with its gradient.
//
// All of it streams: about 10 flops per element against 6 to 18 bytes, so HBM
// bounds it.  A team of TPR lanes owns a row segment and holds it in registers
// (K vectors of 8 elements per lane), so every input is read once, all of a
// row's loads issued before the first is used: the sum of squares is taken and
// the values are normalised from the same registers.  Sums, statistics and the
// residual are float32; the norm is taken of r before it is rounded to the
// residual's type, and each output is rounded once.  The sums over rows (dw,
// dscale) stay in registers while a team walks its rows; teams of a workgroup
// join them in LDS and write one row of a partial-sum table, which a second
// kernel adds up in a fixed order (no atomics).
//
// Measured in a captured graph, and for a backward its two kernels in a trace (a
// 1 GiB copy reaches 4.98 TB/s, a 64 MB one in the cache 6.8):
//   residual norm, 16384 x 2048, bf16 x and out, float32 r:  79.0 us, 5.1 TB/s
//     backward, 4096 x 2048, with dscale:  32.8 us (4.6 TB/s), 29.9 + 4.1 for
//     the sums; two library adds over the same bytes take 31.1 us
//     backward, 1237 x 1027, float32:  13.8 us, 10.6 + 4.1 (in the cache; 1027
//     channels are 129 vectors for 256 lanes, and 512 workgroups walk 2 or 3 rows)
//     one row of 2048:  2.5 us (a launch)
//   gated norm, 4096 x 4096 bf16, z in rows of 8512:  17.6 us, 5.7 TB/s
//     backward in 8 groups:  34.4 us (4.9 TB/s), 31.8 + 4.0
//     256 x 4096, float32 y:  3.4 us
// Set aside: the next row's loads issued before a row is processed (residual
// backward 37.5 -> 36.9 us, gated 39.9 -> 42.5, before the weights stayed in
// registers).

#include "ssd_chunk_common.h"
#include "ssd_internal.h"
#include "ssd_rows.h"

namespace ssd {

namespace {

__device__ __forceinline__ float fast_sigmoid(float v) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(v * -1.4426950408889634f));
}

// Sums of NV values per thread over a team of TPR lanes, returned in every
// lane.  Teams wider than a wave go through LDS (red: 2 x 16 x NV floats,
// alternating between calls, so that one barrier a call is enough).
template <int TPR, int NV>
__device__ __forceinline__ void team_sum(float (&v)[NV], float* red, int parity) {
  constexpr int W = TPR < kWave ? TPR : kWave;  // TPR > kWave: the team is the workgroup
#pragma unroll
  for (int o = W / 2; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] += __shfl_xor(v[i], o, kWave);
  if constexpr (TPR > kWave) {
    constexpr int NW = TPR / kWave;
    float* slot = red + parity * 16 * NV;
    if ((threadIdx.x & (kWave - 1)) == 0)
#pragma unroll
      for (int i = 0; i < NV; ++i) slot[(threadIdx.x / kWave) * NV + i] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float s = 0.0f;
#pragma unroll
      for (int k = 0; k < NW; ++k) s += slot[k * NV + i];
      v[i] = s;
    }
  }
}

// sum over the lane's own elements of f(i), i >= drop
template <typename F>
__device__ __forceinline__ void own_sum(float& acc, int drop, F f) {
  if (drop == 0) {
#pragma unroll
    for (int i = 0; i < 8; ++i) acc += f(i);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) acc += i >= drop ? f(i) : 0.0f;
  }
}

// A lane's sum of squares is scaled by a power of two before the team's sum and
// back in the mean.  No bit of an ordinary row changes, and 16384 squares of
// 1e18 stay inside float32 (2.6e38); unscaled they pass it, rsqrt gives 0 and
// the row is lost.  The other end moves by 2^3: squares of 1e-18 stay whole.
constexpr float kDown = 1.0f / 64.0f, kUp = 64.0f;

// Threads of a workgroup: `several` shared by teams of up to a wave, which
// need no barrier in their row loops; a wider team has a workgroup of its own.
template <int TPR>
constexpr int team_block(int several) {
  return TPR > kWave ? TPR : several;
}
constexpr int kFwdThreads = 256, kBwdThreads = 512;

template <int TPR, int K, bool SHORT, typename TX, typename TR, typename TO>
__global__ __launch_bounds__(team_block<TPR>(kFwdThreads)) void ssd_add_norm_kernel(
    const TX* __restrict__ x, const float* __restrict__ scale, const TR* residual,
    const float* __restrict__ w, float eps, TR* r_out, TO* __restrict__ out, int M, int D) {
  constexpr int BT = team_block<TPR>(kFwdThreads), TEAMS = BT / TPR;
  __shared__ float red[TPR > kWave ? 32 : 1];
  const int lane = threadIdx.x % TPR;
  const float inv = kUp / static_cast<float>(D);
  Place pl[K];
#pragma unroll
  for (int k = 0; k < K; ++k) pl[k] = place_of<SHORT>(lane + k * TPR, D);
  int parity = 0;
  for (long long row = static_cast<long long>(blockIdx.x) * TEAMS + threadIdx.x / TPR; row < M;
       row += static_cast<long long>(gridDim.x) * TEAMS) {
    const size_t base = static_cast<size_t>(row) * D;
    float r[K][8];
    Row8<float> wv[K];
    {
      Row8<TX> xv[K];
#pragma unroll
      for (int k = 0; k < K; ++k) xv[k] = row_load<SHORT>(x + base, pl[k], D);
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) r[k][i] = xv[k][i];
    }
    if (scale) {
      Row8<float> sv[K];
#pragma unroll
      for (int k = 0; k < K; ++k) sv[k] = row_load<SHORT>(reload<(K > 1)>(scale), pl[k], D);
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) r[k][i] *= sv[k][i];
    }
    if (residual) {
      Row8<TR> rv[K];
#pragma unroll
      for (int k = 0; k < K; ++k) rv[k] = row_load<SHORT>(residual + base, pl[k], D);
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) r[k][i] += rv[k][i];
    }
#pragma unroll
    for (int k = 0; k < K; ++k) wv[k] = row_load<SHORT>(reload<(K > 1)>(w), pl[k], D);
    float ss[1] = {0.0f};
#pragma unroll
    for (int k = 0; k < K; ++k) own_sum(ss[0], pl[k].drop, [&](int i) { return r[k][i] * r[k][i]; });
    ss[0] *= kDown;
    team_sum<TPR, 1>(ss, red, parity);
    parity ^= 1;
    const float rstd = rsqrtf(ss[0] * inv + eps);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float o[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = r[k][i] * rstd * wv[k][i];
      if (r_out) row_store<SHORT>(r_out + base, pl[k], D, r[k]);
      row_store<SHORT>(out + base, pl[k], D, o);
    }
  }
}

// Backward: what is loaded or made again rather than kept (see reload, remake):
// where two vectors a lane meet 128 registers.
template <int TPR, int K>
constexpr bool kHide = K > 1 && TPR > kWave;

// The team's column sums (K vectors of 8 per lane) joined over the workgroup's
// teams and written as columns 0 .. L-1 of `part`.
template <int TPR, int K, bool SHORT>
__device__ __forceinline__ void write_part(const float (&acc)[K][8], const Place (&pl)[K], float* buf,
                                           float* part, int L) {
  constexpr int BT = team_block<TPR>(kBwdThreads), TEAMS = BT / TPR;
  const int lane = threadIdx.x % TPR, team = threadIdx.x / TPR;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    if constexpr (TEAMS > 1) {
      // buf[i][team][lane]: element i of the lane's vector; column j of the
      // sums is element j / TPR of lane j % TPR
#pragma unroll
      for (int i = 0; i < 8; ++i) buf[(i * TEAMS + team) * TPR + lane] = acc[k][i];
      __syncthreads();
      for (int j = threadIdx.x; j < TPR * 8; j += BT) {  // BT is a multiple of TPR: lane stays
        const int i = j / TPR;
        float s = 0.0f;
#pragma unroll 8
        for (int t = 0; t < TEAMS; ++t) s += buf[(i * TEAMS + t) * TPR + lane];
        const Place p = place_of<SHORT>(lane + k * TPR, L);
        if (i >= p.drop && i < (SHORT ? L : 8)) part[p.off + i] = s;
      }
      __syncthreads();
    } else {
      row_store<SHORT>(part, pl[k], L, acc[k]);
    }
  }
}

template <int TPR, int K, bool SHORT, typename TX, typename TR, typename TO>
__global__ __launch_bounds__(team_block<TPR>(kBwdThreads)) void ssd_add_norm_bwd_kernel(
    const TO* __restrict__ dout, const TR* __restrict__ dres, const TR* __restrict__ r,
    const TX* __restrict__ x, const float* __restrict__ scale, const float* __restrict__ w,
    float eps, TR* __restrict__ dresidual, TX* __restrict__ dx, float* __restrict__ part, int M,
    int D, int want_dscale) {
  constexpr int BT = team_block<TPR>(kBwdThreads), TEAMS = BT / TPR;
  __shared__ float red[TPR > kWave ? 64 : 1];
  __shared__ float buf[TEAMS > 1 ? BT * 8 : 1];
  const int lane = threadIdx.x % TPR;
  const float inv = 1.0f / static_cast<float>(D);
  Place pl[K];
#pragma unroll
  for (int k = 0; k < K; ++k) pl[k] = place_of<SHORT>(lane + k * TPR, D);
  float dw[K][8] = {}, ds[K][8] = {};
  int parity = 0;
  for (long long row = static_cast<long long>(blockIdx.x) * TEAMS + threadIdx.x / TPR; row < M;
       row += static_cast<long long>(gridDim.x) * TEAMS) {
    const size_t base = static_cast<size_t>(row) * D;
    Row8<TR> rv[K], ev[K];
    Row8<TO> dv[K];
    Row8<TX> xv[K];
#pragma unroll
    for (int k = 0; k < K; ++k) rv[k] = row_load<SHORT>(r + base, pl[k], D), dv[k] = row_load<SHORT>(dout + base, pl[k], D);
    // what the second half needs arrives during the first (without dres or
    // dscale the row itself is loaded again, from the cache, and not used)
    const TR* second = dres ? dres : r;
#pragma unroll
    for (int k = 0; k < K; ++k) ev[k] = row_load<SHORT>(second + base, pl[k], D);
    if (want_dscale) {
#pragma unroll
      for (int k = 0; k < K; ++k) xv[k] = row_load<SHORT>(x + base, pl[k], D);
    }
    float s[2] = {0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const Row8<float> wv = row_load<SHORT>(reload<kHide<TPR, K>>(w), pl[k], D);
      own_sum(s[0], pl[k].drop, [&](int i) { return rv[k][i] * rv[k][i]; });
      own_sum(s[1], pl[k].drop, [&](int i) { return dv[k][i] * wv[i] * rv[k][i]; });
    }
    s[0] *= kDown;
    team_sum<TPR, 2>(s, red, parity);
    parity ^= 1;
    const float rstd = rsqrtf(s[0] * (kUp * inv) + eps);
    const float m = s[1] * rstd * inv;  // mean(dn o n)
#pragma unroll
    for (int k = 0; k < K; ++k) {
      remake<kHide<TPR, K>>(rv[k]);
      remake<kHide<TPR, K>>(dv[k]);
      const Row8<float> wv = row_load<SHORT>(reload<kHide<TPR, K>>(w), pl[k], D);
      float g[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float n = rv[k][i] * rstd;
        dw[k][i] = fmaf(dv[k][i], n, dw[k][i]);
        g[i] = rstd * fmaf(-n, m, dv[k][i] * wv[i]);
        if (dres) g[i] += ev[k][i];
      }
      if (dresidual) row_store<SHORT>(dresidual + base, pl[k], D, g);
      if (want_dscale) {
#pragma unroll
        for (int i = 0; i < 8; ++i) ds[k][i] = fmaf(g[i], xv[k][i], ds[k][i]);
      }
      if (dx) {
        if (scale) {
          const Row8<float> sv = row_load<SHORT>(reload<kHide<TPR, K>>(scale), pl[k], D);
#pragma unroll
          for (int i = 0; i < 8; ++i) g[i] *= sv[i];
        }
        row_store<SHORT>(dx + base, pl[k], D, g);
      }
    }
  }
  float* p = part + static_cast<size_t>(blockIdx.x) * (want_dscale ? 2 : 1) * D;
  write_part<TPR, K, SHORT>(dw, pl, buf, p, D);
  if (want_dscale) write_part<TPR, K, SHORT>(ds, pl, buf, p + D, D);
}

// Grid: x = row blocks, y = groups.
template <int TPR, int K, bool SHORT, typename TY, typename TZ, typename TO>
__global__ __launch_bounds__(team_block<TPR>(kFwdThreads)) void ssd_gated_norm_kernel(
    const TY* __restrict__ y, const TZ* __restrict__ z, long long ldz, const float* __restrict__ w,
    float eps, int before, TO* __restrict__ out, int M, int D, int L) {
  constexpr int BT = team_block<TPR>(kFwdThreads), TEAMS = BT / TPR;
  __shared__ float red[TPR > kWave ? 32 : 1];
  const int lane = threadIdx.x % TPR;
  const float inv = kUp / static_cast<float>(L);
  const size_t c0 = static_cast<size_t>(blockIdx.y) * L;
  Place pl[K];
#pragma unroll
  for (int k = 0; k < K; ++k) pl[k] = place_of<SHORT>(lane + k * TPR, L);
  int parity = 0;
  for (long long row = static_cast<long long>(blockIdx.x) * TEAMS + threadIdx.x / TPR; row < M;
       row += static_cast<long long>(gridDim.x) * TEAMS) {
    const size_t base = static_cast<size_t>(row) * D + c0;
    Row8<TY> yv[K];
    Row8<TZ> zv[K];
    Row8<float> wv[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      yv[k] = row_load<SHORT>(y + base, pl[k], L);
      zv[k] = row_load<SHORT>(z + static_cast<size_t>(row) * ldz + c0, pl[k], L);
    }
#pragma unroll
    for (int k = 0; k < K; ++k) wv[k] = row_load<SHORT>(reload<(K > 1)>(w) + c0, pl[k], L);
    float u[K][8], gt[K][8];
    float ss[1] = {0.0f};
#pragma unroll
    for (int k = 0; k < K; ++k) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float s = zv[k][i] * fast_sigmoid(zv[k][i]);
        u[k][i] = before ? yv[k][i] : yv[k][i] * s;
        gt[k][i] = before ? s : 1.0f;
      }
      own_sum(ss[0], pl[k].drop, [&](int i) { return u[k][i] * u[k][i]; });
    }
    ss[0] *= kDown;
    team_sum<TPR, 1>(ss, red, parity);
    parity ^= 1;
    const float rstd = rsqrtf(ss[0] * inv + eps);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float o[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = u[k][i] * rstd * wv[k][i] * gt[k][i];
      row_store<SHORT>(out + base, pl[k], L, o);
    }
  }
}

template <int TPR, int K, bool SHORT, typename TY, typename TZ, typename TO>
__global__ __launch_bounds__(team_block<TPR>(kBwdThreads)) void ssd_gated_norm_bwd_kernel(
    const TO* __restrict__ dout, const TY* __restrict__ y, const TZ* __restrict__ z, long long ldz,
    const float* __restrict__ w, float eps, int before, TY* __restrict__ dy, TZ* __restrict__ dz,
    long long lddz, float* __restrict__ part, int M, int D, int L) {
  constexpr int BT = team_block<TPR>(kBwdThreads), TEAMS = BT / TPR;
  __shared__ float red[TPR > kWave ? 64 : 1];
  __shared__ float buf[TEAMS > 1 ? BT * 8 : 1];
  const int lane = threadIdx.x % TPR;
  const float inv = 1.0f / static_cast<float>(L);
  const size_t c0 = static_cast<size_t>(blockIdx.y) * L;
  Place pl[K];
#pragma unroll
  for (int k = 0; k < K; ++k) pl[k] = place_of<SHORT>(lane + k * TPR, L);
  float dw[K][8] = {};
  int parity = 0;
  for (long long row = static_cast<long long>(blockIdx.x) * TEAMS + threadIdx.x / TPR; row < M;
       row += static_cast<long long>(gridDim.x) * TEAMS) {
    const size_t base = static_cast<size_t>(row) * D + c0;
    Row8<TY> yv[K];
    Row8<TZ> zv[K];
    Row8<TO> dv[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      yv[k] = row_load<SHORT>(y + base, pl[k], L);
      zv[k] = row_load<SHORT>(z + static_cast<size_t>(row) * ldz + c0, pl[k], L);
      dv[k] = row_load<SHORT>(dout + base, pl[k], L);
    }
    float s[2] = {0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const Row8<float> wv = row_load<SHORT>(reload<kHide<TPR, K>>(w) + c0, pl[k], L);
      float u[8], dn[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float gate = zv[k][i] * fast_sigmoid(zv[k][i]);
        u[i] = before ? yv[k][i] : yv[k][i] * gate;
        dn[i] = before ? dv[k][i] * gate : dv[k][i];
      }
      own_sum(s[0], pl[k].drop, [&](int i) { return u[i] * u[i]; });
      own_sum(s[1], pl[k].drop, [&](int i) { return dn[i] * wv[i] * u[i]; });
    }
    s[0] *= kDown;
    team_sum<TPR, 2>(s, red, parity);
    parity ^= 1;
    const float rstd = rsqrtf(s[0] * (kUp * inv) + eps);
    const float m = s[1] * rstd * inv;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      remake<kHide<TPR, K>>(yv[k]);
      remake<kHide<TPR, K>>(zv[k]);
      remake<kHide<TPR, K>>(dv[k]);
      const Row8<float> wv = row_load<SHORT>(reload<kHide<TPR, K>>(w) + c0, pl[k], L);
      float gy[8], gz[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float zz = zv[k][i], sig = fast_sigmoid(zz), gate = zz * sig;
        const float u = before ? yv[k][i] : yv[k][i] * gate;
        const float n = u * rstd;
        const float dn = before ? dv[k][i] * gate : dv[k][i];
        dw[k][i] = fmaf(dn, n, dw[k][i]);
        const float du = rstd * fmaf(-n, m, dn * wv[i]);
        gy[i] = before ? du : du * gate;
        const float dg = before ? dv[k][i] * n * wv[i] : du * yv[k][i];
        gz[i] = dg * sig * fmaf(zz, 1.0f - sig, 1.0f);
      }
      row_store<SHORT>(dy + base, pl[k], L, gy);
      row_store<SHORT>(dz + static_cast<size_t>(row) * lddz + c0, pl[k], L, gz);
    }
  }
  write_part<TPR, K, SHORT>(dw, pl, buf, part + static_cast<size_t>(blockIdx.x) * D + c0, L);
}

// Grid: blocks of 64 columns; the 16 waves of a block split the parts, each
// with eight loads in flight.
constexpr int kSumWaves = 16;
__global__ __launch_bounds__(kSumWaves* kWave) void ssd_sum_parts_kernel(
    const float* __restrict__ part, int nparts, int n, float* __restrict__ a, int na,
    float* __restrict__ b) {
  constexpr int U = 8;
  __shared__ float s[kSumWaves][kWave];
  const int lane = threadIdx.x & (kWave - 1), wv = wave_id();
  const int col = blockIdx.x * kWave + lane;
  float acc = 0.0f;
  if (col < n) {
    for (int p0 = wv; p0 < nparts; p0 += U * kSumWaves) {
      float v[U];
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const int p = p0 + k * kSumWaves;  // past the table: the last row, not added
        v[k] = part[static_cast<size_t>(p < nparts ? p : nparts - 1) * n + col];
      }
#pragma unroll
      for (int k = 0; k < U; ++k) acc += p0 + k * kSumWaves < nparts ? v[k] : 0.0f;
    }
  }
  s[wv][lane] = acc;
  __syncthreads();
  if (wv == 0 && col < n) {
    float t = 0.0f;
#pragma unroll
    for (int k = 0; k < kSumWaves; ++k) t += s[k][lane];
    if (col < na)
      a[col] = t;
    else
      b[col - na] = t;
  }
}

struct Shape {
  int tpr, k;
};
// Lanes of a team and vectors per lane for a row segment of L elements, in both
// directions.
// Forward: one vector per lane, but for the longest rows and for 513 to 1024
// elements, whose backward is the faster with two (below).  The few instructions
// per wave set the time of a small batch (one row of 2048: 256 lanes 2.7 us, 64
// lanes of four vectors 3.4; one row of 1024 with two 2.6), and large batches
// stream either way (4096 x 2048: 17.1 and 16.9 us, 8192 x 1024 with two 16.9;
// 512 x 16384: 19.7 and, with 512 lanes of four, 17.5).
// Backward: each lane also holds the column sums of its vectors.  Measured for
// the residual norm (bf16 x and dout, float32 r and dres, 2^23 elements) and,
// after the slash, the gated one (bf16, 2^24), floors 30.3 / 33.7 us: L = 512
// 32.6 / 33.4 us; 1024 with 64 lanes of two 33.1 / 34.0, 128 of one 35.0 / 42.1;
// 2048 32.2 / 36.5; 4096 34.7 / 36.6; 8192 with 1024 of one 37.3 / 41.0, 512 of
// two 44.5 / 44.1; 16384 with 1024 of two 44.1, 512 of four 45.8.
// Other types cross register limits, but not the time: the gated backward of 2049
// to 4096 channels with float32 y and bf16 z takes 130 registers, so one workgroup
// a CU instead of two (4096 x 4096: 1.14 of its floor; all bf16, 123 registers,
// 1.17); of 4097 to 8192 channels it spills 1 to 4 with a float32 among its types
// (1.01 to 1.05; all bf16, none, 1.22); the residual backward of 8193 to 16384
// channels spills 2 to 17 (512 x 16384: 1.41 to 1.46; all bf16, none, 1.68).
Shape shape_of(int L) {
  if (L <= 128) return {16, 1};
  if (L <= 512) return {64, 1};
  if (L <= 1024) return {64, 2};
  if (L <= 2048) return {256, 1};
  if (L <= 4096) return {512, 1};
  if (L <= 8192) return {1024, 1};
  return {1024, 2};
}
// workgroups of `several` threads (or one team) along the rows: enough for
// every row, at most `cap` over all groups
int row_blocks(int M, Shape s, int groups, int several, int cap) {
  const int t = s.tpr > kWave ? 1 : several / s.tpr;
  const long long need = (static_cast<long long>(M) + t - 1) / t;
  const long long most = cap / groups > 0 ? cap / groups : 1;
  return static_cast<int>(need < most ? need : most);
}
constexpr int kFwdBlocks = 4096;
// Backward: every workgroup writes a row of `sums` vectors of partial sums, so
// few are wanted, but their waves have to keep the memory busy: 512; 256 with
// two vectors a lane (8192 rows of 1024: residual norm 33.1 us, gated 34.0 at
// 16384 rows; at 512 36.4 and 38.0) or sixteen waves (1024 x 8192: 37.3 and, at
// 512, 42.8); 1024 where teams of four waves write one sum (4096 x 2 norms of
// 2048: 37.1 us, at 512 40.6; the residual norm's two sums there 36.7 and 32.5).
int bwd_blocks(int L, int sums) {
  const Shape s = shape_of(L);
  return s.k == 2 || s.tpr == 1024 ? 256 : s.tpr == 256 && sums == 1 ? 1024 : 512;
}

// KERNEL<TPR, K, SHORT, types> for segments of L elements
#define SSD_ROW_CASE(KERNEL, TPR, K, grid, several, st, ...)                                   \
  case TPR * 8 + K:                                                                            \
    launch_k(true, KERNEL<TPR, K, false, T0, T1, T2>, grid, dim3(team_block<TPR>(several)), st, \
             nullptr, __VA_ARGS__);                                                            \
    break;
#define SSD_ROW_LAUNCH(KERNEL, L, grid, several, st, ...)                                         \
  do {                                                                                            \
    if (L < 8) {                                                                                  \
      launch_k(true, KERNEL<16, 1, true, T0, T1, T2>, grid, dim3(team_block<16>(several)), st,     \
               nullptr, __VA_ARGS__);                                                             \
      break;                                                                                      \
    }                                                                                             \
    const Shape shape = shape_of(L);                                                              \
    switch (shape.tpr * 8 + shape.k) {                                                            \
      SSD_ROW_CASE(KERNEL, 16, 1, grid, several, st, __VA_ARGS__)                                 \
      SSD_ROW_CASE(KERNEL, 64, 1, grid, several, st, __VA_ARGS__)                                 \
      SSD_ROW_CASE(KERNEL, 64, 2, grid, several, st, __VA_ARGS__)                                 \
      SSD_ROW_CASE(KERNEL, 256, 1, grid, several, st, __VA_ARGS__)                                \
      SSD_ROW_CASE(KERNEL, 512, 1, grid, several, st, __VA_ARGS__)                                \
      SSD_ROW_CASE(KERNEL, 1024, 1, grid, several, st, __VA_ARGS__)                               \
      SSD_ROW_CASE(KERNEL, 1024, 2, grid, several, st, __VA_ARGS__)                               \
    }                                                                                             \
  } while (0)

template <typename T0, typename T1, typename T2>
hipError_t add_norm_fwd_t(const AddNormArgs& a, hipStream_t st) {
  const dim3 grid(row_blocks(a.M, shape_of(a.D), 1, kFwdThreads, kFwdBlocks));
  SSD_ROW_LAUNCH(ssd_add_norm_kernel, a.D, grid, kFwdThreads, st, static_cast<const T0*>(a.x), a.scale,
                 static_cast<const T1*>(a.residual), a.w, a.eps, static_cast<T1*>(a.r_out),
                 static_cast<T2*>(a.out), a.M, a.D);
  return hipGetLastError();
}

template <typename T0, typename T1, typename T2>
hipError_t add_norm_bwd_t(const AddNormArgs& a, hipStream_t st) {
  const int nparts = add_norm_parts(a.M, a.D);
  float* part = static_cast<float*>(a.workspace);
  if (nparts > 0) {  // no rows: the sums are zero
    SSD_ROW_LAUNCH(ssd_add_norm_bwd_kernel, a.D, dim3(nparts), kBwdThreads, st, static_cast<const T2*>(a.dout),
                   static_cast<const T1*>(a.dres), static_cast<const T1*>(a.r), static_cast<const T0*>(a.x),
                   a.scale, a.w, a.eps, static_cast<T1*>(a.dresidual), static_cast<T0*>(a.dx), part, a.M, a.D,
                   static_cast<int>(a.dscale != nullptr));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return sum_parts(part, nparts, a.dscale ? 2 * a.D : a.D, a.dw, a.D, a.dscale, st);
}

template <typename T0, typename T1, typename T2>
hipError_t gated_norm_fwd_t(const GatedNormArgs& a, hipStream_t st) {
  const int L = a.D / a.groups;
  const dim3 grid(row_blocks(a.M, shape_of(L), a.groups, kFwdThreads, kFwdBlocks), a.groups);
  SSD_ROW_LAUNCH(ssd_gated_norm_kernel, L, grid, kFwdThreads, st, static_cast<const T0*>(a.y),
                 static_cast<const T1*>(a.z), a.ldz, a.w, a.eps, a.before, static_cast<T2*>(a.out), a.M, a.D, L);
  return hipGetLastError();
}

template <typename T0, typename T1, typename T2>
hipError_t gated_norm_bwd_t(const GatedNormArgs& a, hipStream_t st) {
  const int L = a.D / a.groups;
  const int nparts = gated_norm_parts(a.M, a.D, a.groups);
  float* part = static_cast<float*>(a.workspace);
  if (nparts > 0) {
    SSD_ROW_LAUNCH(ssd_gated_norm_bwd_kernel, L, dim3(nparts, a.groups), kBwdThreads, st,
                   static_cast<const T2*>(a.dout), static_cast<const T0*>(a.y), static_cast<const T1*>(a.z), a.ldz,
                   a.w, a.eps, a.before, static_cast<T0*>(a.dy), static_cast<T1*>(a.dz), a.lddz, part, a.M, a.D, L);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return sum_parts(part, nparts, a.D, a.dw, a.D, nullptr, st);
}

// the three element types of a call, each float32 (0) or bfloat16 (1)
#define SSD_TYPES3(FN, a, t0, t1, t2, st)                            \
  switch ((t0) * 4 + (t1) * 2 + (t2)) {                              \
    case 0: return FN<float, float, float>(a, st);                   \
    case 1: return FN<float, float, uint16_t>(a, st);                \
    case 2: return FN<float, uint16_t, float>(a, st);                \
    case 3: return FN<float, uint16_t, uint16_t>(a, st);             \
    case 4: return FN<uint16_t, float, float>(a, st);                \
    case 5: return FN<uint16_t, float, uint16_t>(a, st);             \
    case 6: return FN<uint16_t, uint16_t, float>(a, st);             \
    default: return FN<uint16_t, uint16_t, uint16_t>(a, st);         \
  }

}  // namespace

hipError_t sum_parts(const float* part, int nparts, int n, float* a, int na, float* b,
                     hipStream_t st) {
  launch_k(true, ssd_sum_parts_kernel, dim3((n + kWave - 1) / kWave), dim3(kSumWaves * kWave), st,
           nullptr, part, nparts, n, a, na, b);
  return hipGetLastError();
}

int add_norm_parts(int M, int D) { return row_blocks(M, shape_of(D), 1, kBwdThreads, bwd_blocks(D, 2)); }
int gated_norm_parts(int M, int D, int groups) {
  const int L = D / groups;
  return row_blocks(M, shape_of(L), groups, kBwdThreads, bwd_blocks(L, 1));
}

hipError_t run_add_norm(const AddNormArgs& a, hipStream_t st) {
  SSD_TYPES3(add_norm_fwd_t, a, a.x_dtype, a.res_dtype, a.out_dtype, st)
}
hipError_t run_add_norm_bwd(const AddNormArgs& a, hipStream_t st) {
  SSD_TYPES3(add_norm_bwd_t, a, a.x_dtype, a.res_dtype, a.out_dtype, st)
}
hipError_t run_gated_norm(const GatedNormArgs& a, hipStream_t st) {
  SSD_TYPES3(gated_norm_fwd_t, a, a.y_dtype, a.z_dtype, a.out_dtype, st)
}
hipError_t run_gated_norm_bwd(const GatedNormArgs& a, hipStream_t st) {
  SSD_TYPES3(gated_norm_bwd_t, a, a.y_dtype, a.z_dtype, a.out_dtype, st)
}

}  // namespace ssd
