// Backward of the Mamba-2 layer's depthwise causal convolution (kernel size 4,
// bias, SiLU; the forward is ssd_conv.hip) on gfx950.
//
// With v_t = bias + sum_j w_j in_{t-3+j} and out_t = act(v_t), per channel:
//   g_t   = dout_t act'(v_t),   SiLU'(v) = s (1 + v (1 - s)), s = 1/(1+e^-v)
//   din_p = w_3 g_p + w_2 g_{p+1} + w_1 g_{p+2} + w_0 g_{p+3}   (g outside 0..T-1 is 0)
//           + dstate_out[p - (T-3)] where p >= T-3
//   dw_j  = sum_{b,t} g_t in_{t-3+j},   dbias = sum_{b,t} g_t
// where in_p for p < 0 is the carried state, whose gradient din_{-3..-1} is
// dstate_in.  v_t is recomputed from the inputs; nothing is saved by the
// forward.
//
// The operation streams (x and dout in, dx out).  A lane owns 4 channels and
// walks a run of tokens with the windows in_{t-3..t} and g_{t-3..t} and the
// channel's five sums in registers, so a row is read once per run (plus 3
// rows of halo on either side).  The four waves of a workgroup take runs of
// the same channels and join their sums in LDS; each workgroup writes one row
// of a partial-sum table that a second kernel adds up in a fixed order.

#include "ssd_chunk_common.h"
#include "ssd_internal.h"
#include "ssd_rows.h"

namespace ssd {

namespace {

constexpr int kV = 4;        // channels per lane
constexpr int kRun = 32;     // tokens per run
constexpr int kMaxParts = 256;

template <typename T>
__device__ __forceinline__ void load4(const T* p, float* f);
template <>
__device__ __forceinline__ void load4<float>(const float* p, float* f) {
  const float4 q = *reinterpret_cast<const float4*>(p);
  f[0] = q.x, f[1] = q.y, f[2] = q.z, f[3] = q.w;
}
template <>
__device__ __forceinline__ void load4<uint16_t>(const uint16_t* p, float* f) {
  const uint2 q = *reinterpret_cast<const uint2*>(p);
  f[0] = __uint_as_float(q.x << 16), f[1] = __uint_as_float(q.x & 0xFFFF0000u);
  f[2] = __uint_as_float(q.y << 16), f[3] = __uint_as_float(q.y & 0xFFFF0000u);
}
__device__ __forceinline__ void store4(float* p, const float* f) {
  *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
}
__device__ __forceinline__ void store4(uint16_t* p, const float* f) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]));
}

// Grid: x = channel blocks of 64 lanes, y = workgroups over the (sequence,
// run) units, four units at a time.
template <typename T, bool SILU>
__global__ __launch_bounds__(kThreads) void ssd_conv1d_bwd_kernel(
    const T* __restrict__ xbc, long long ld, const float* __restrict__ w,
    const float* __restrict__ bias, const float* __restrict__ state_in, const T* __restrict__ dx,
    const float* __restrict__ dB, const float* __restrict__ dC,
    const float* __restrict__ dstate_out, T* __restrict__ dxbc, long long lddx,
    float* __restrict__ dstate_in, float* __restrict__ part, int Bsz, int Tn, int HP, int GN) {
  const int Ch = HP + 2 * GN;
  const int wid = wave_id();
  const int c = (blockIdx.x * kWave + (threadIdx.x & (kWave - 1))) * kV;
  const bool active = c < Ch;
  const int nruns = Tn > 0 ? (Tn + kRun - 1) / kRun : 1;
  const long long units = static_cast<long long>(Bsz) * nruns;
  float wt[kV][4], bs[kV] = {}, dw[kV][4] = {}, db[kV] = {};
#pragma unroll
  for (int v = 0; v < kV; ++v) {
    load4(w + static_cast<size_t>(active ? c + v : 0) * 4, wt[v]);
  }
  if (bias && active) load4(bias + c, bs);

  for (long long u = static_cast<long long>(blockIdx.y) * 4 + wid; u < units;
       u += static_cast<long long>(gridDim.y) * 4) {
    if (!active) continue;
    const int b = static_cast<int>(u / nruns);
    const int t0 = static_cast<int>(u % nruns) * kRun;
    const int t1 = min(t0 + kRun, Tn);
    const size_t row0 = static_cast<size_t>(b) * Tn;
    const float* st = state_in ? state_in + static_cast<size_t>(b) * 3 * Ch + c : nullptr;
    auto in_at = [&](int p, float* f) {
      if (p >= 0) {
        load4(xbc + (row0 + p) * ld + c, f);
      } else if (st) {
        load4(st + static_cast<size_t>(3 + p) * Ch, f);
      } else {
        f[0] = f[1] = f[2] = f[3] = 0.0f;
      }
    };
    auto dout_at = [&](int t, float* f) {
      if (c < HP)
        load4(dx + (row0 + t) * HP + c, f);
      else if (c < HP + GN)
        load4(dB + (row0 + t) * GN + (c - HP), f);
      else
        load4(dC + (row0 + t) * GN + (c - HP - GN), f);
    };
    float win[4][kV], gw[4][kV] = {};
#pragma unroll
    for (int j = 0; j < 3; ++j) in_at(t0 - 3 + j, win[j + 1]);
    for (int t = t0; t < t1 + 3; ++t) {
#pragma unroll
      for (int j = 0; j < 3; ++j)
#pragma unroll
        for (int v = 0; v < kV; ++v) win[j][v] = win[j + 1][v], gw[j][v] = gw[j + 1][v];
      if (t < Tn) {
        float d[kV];
        in_at(t, win[3]);
        dout_at(t, d);
#pragma unroll
        for (int v = 0; v < kV; ++v) {
          float g = d[v];
          if (SILU) {
            float a = bs[v];
#pragma unroll
            for (int j = 0; j < 4; ++j) a = fmaf(wt[v][j], win[j][v], a);
            const float s = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(a * -1.4426950408889634f));
            g *= s * fmaf(a, 1.0f - s, 1.0f);
          }
          gw[3][v] = g;
          if (t < t1) {
            db[v] += g;
#pragma unroll
            for (int j = 0; j < 4; ++j) dw[v][j] = fmaf(g, win[j][v], dw[v][j]);
          }
        }
      } else {
#pragma unroll
        for (int v = 0; v < kV; ++v) gw[3][v] = 0.0f;
      }
      const int p = t - 3;
      if (p < t0 && t0 > 0) continue;  // the run before writes those
      float o[kV];
#pragma unroll
      for (int v = 0; v < kV; ++v)
        o[v] = fmaf(wt[v][3], gw[0][v], fmaf(wt[v][2], gw[1][v], fmaf(wt[v][1], gw[2][v], wt[v][0] * gw[3][v])));
      if (dstate_out && p >= Tn - 3) {
        float e[kV];
        load4(dstate_out + (static_cast<size_t>(b) * 3 + (p - (Tn - 3))) * Ch + c, e);
#pragma unroll
        for (int v = 0; v < kV; ++v) o[v] += e[v];
      }
      if (p >= 0)
        store4(dxbc + (row0 + p) * lddx + c, o);
      else if (dstate_in)
        store4(dstate_in + (static_cast<size_t>(b) * 3 + (3 + p)) * Ch + c, o);
    }
  }

  // join the four waves: columns c*4 + j hold dw, 4 Ch + c dbias
  __shared__ float buf[3][kWave][kV * 5];
  const int lane = threadIdx.x & (kWave - 1);
  if (wid > 0) {
#pragma unroll
    for (int v = 0; v < kV; ++v) {
#pragma unroll
      for (int j = 0; j < 4; ++j) buf[wid - 1][lane][v * 4 + j] = dw[v][j];
      buf[wid - 1][lane][16 + v] = db[v];
    }
  }
  __syncthreads();
  if (wid == 0 && active) {
    float* p = part + static_cast<size_t>(blockIdx.y) * 5 * Ch;
#pragma unroll
    for (int v = 0; v < kV; ++v) {
#pragma unroll
      for (int j = 0; j < 4; ++j) dw[v][j] += buf[0][lane][v * 4 + j] + buf[1][lane][v * 4 + j] + buf[2][lane][v * 4 + j];
      db[v] += buf[0][lane][16 + v] + buf[1][lane][16 + v] + buf[2][lane][16 + v];
      store4(p + static_cast<size_t>(c + v) * 4, dw[v]);
    }
    store4(p + 4 * static_cast<size_t>(Ch) + c, db);
  }
}

template <typename T>
void launch_conv_bwd(const ConvBwdArgs& a, hipStream_t st) {
  const int Ch = a.HP + 2 * a.GN;
  const dim3 grid((Ch / kV + kWave - 1) / kWave, conv_bwd_parts(a.Bsz, a.T));
  const T* xbc = static_cast<const T*>(a.xbc);
  const T* dx = static_cast<const T*>(a.dx);
  T* dxbc = static_cast<T*>(a.dxbc);
  float* part = static_cast<float*>(a.workspace);
  if (a.act)
    launch_k(true, ssd_conv1d_bwd_kernel<T, true>, grid, dim3(kThreads), st, nullptr, xbc, a.ld, a.w,
             a.bias, a.state_in, dx, a.dB, a.dC, a.dstate_out, dxbc, a.lddx, a.dstate_in, part, a.Bsz,
             a.T, a.HP, a.GN);
  else
    launch_k(true, ssd_conv1d_bwd_kernel<T, false>, grid, dim3(kThreads), st, nullptr, xbc, a.ld, a.w,
             a.bias, a.state_in, dx, a.dB, a.dC, a.dstate_out, dxbc, a.lddx, a.dstate_in, part, a.Bsz,
             a.T, a.HP, a.GN);
}

}  // namespace

// rows of the partial-sum table: one per workgroup of four runs
int conv_bwd_parts(int Bsz, int T) {
  const long long units = static_cast<long long>(Bsz) * (T > 0 ? (T + kRun - 1) / kRun : 1);
  const long long need = (units + 3) / 4;
  return static_cast<int>(need < kMaxParts ? need : kMaxParts);
}

hipError_t run_conv1d_bwd(const ConvBwdArgs& a, hipStream_t st) {
  if (a.dtype == 1)
    launch_conv_bwd<uint16_t>(a, st);
  else
    launch_conv_bwd<float>(a, st);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int Ch = a.HP + 2 * a.GN;
  return sum_parts(static_cast<const float*>(a.workspace), conv_bwd_parts(a.Bsz, a.T), 5 * Ch, a.dw,
                   4 * Ch, a.dbias, st);
}

}  // namespace ssd
