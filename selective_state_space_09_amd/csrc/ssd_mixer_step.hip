// One token of the Mamba-2 layer between in_proj and the gated norm, in one
// launch on a pool of per-sequence states: the causal convolution's step
// (ssd_conv.hip) and the recurrence's step (ssd_decode.hip).
//
// Row b of the batch belongs to slot s = slots[b] of the pool.  With
// in = [conv rows 0..2 of the slot, xbc row b], per channel
//   v = bias + sum_j w_j in_j, out = act(v), split into x (H P), B, C (G N)
// then per head h of group g
//   delta = clamp(softplus(dt + dt_bias)), a = exp(A delta)
//   state <- a state + delta x B^T,  y = state C + D x
// and the conv rows move up by one.
//
// The state (P N floats per head, read and written once) is nearly all of the
// traffic, so HBM bounds a large batch and latency a small one.  One workgroup
// per (row, head): it convolves its head's P channels and its group's B and C
// into LDS (the H/G heads of a group repeat B and C: 2N channels against P N
// state values, from the cache), then walks the state as the decode kernel
// does.  A head's own conv rows are shifted by its workgroup; those of B and C
// are still being read by the group's other workgroups, so each counts itself
// in at the slot's arrivals counter once it has read them, and the last one
// shifts them (the counter wraps to zero by itself).  No workgroup waits for
// another.

#include "ssd_chunk_common.h"
#include "ssd_internal.h"

namespace ssd {

namespace {

typedef float f4v __attribute__((ext_vector_type(4)));

template <typename T>
__device__ __forceinline__ float elem(T v);
template <>
__device__ __forceinline__ float elem<float>(float v) {
  return v;
}
template <>
__device__ __forceinline__ float elem<uint16_t>(uint16_t v) {
  return bf16_bits_to_f32(v);
}

template <int N, typename T>
__global__ __launch_bounds__(kThreads) void ssd_mixer_step_kernel(
    float* __restrict__ conv, float* __restrict__ hpool, unsigned* __restrict__ arrivals,
    const int* __restrict__ slots, int nslots, const T* __restrict__ xbc, long long ldx,
    const T* __restrict__ dt, long long lddt, const float* __restrict__ w,
    const float* __restrict__ bias, int act, const float* __restrict__ A,
    const float* __restrict__ D, const float* __restrict__ dt_bias, float lo, float hi,
    void* __restrict__ y, int y_bf16, int H, int P, int G) {
  extern __shared__ float lds[];  // x (P), B (N), C (N)
  constexpr int LPR = N / 4;            // lanes per state row
  constexpr int RPP = kThreads / LPR;   // rows covered by one pass of the block
  constexpr int UNR = 8;                // rows in flight per thread
  constexpr int CI = 2;                 // convolved channels in flight per thread
  const int b = blockIdx.x / H, hh = blockIdx.x % H, g = hh / (H / G);
  const int tid = threadIdx.x;
  const int HP = H * P, GN = G * N, Ch = HP + 2 * GN, nch = P + 2 * N;
  const size_t yrow = static_cast<size_t>(blockIdx.x) * P;

  // a row takes part if its slot exists and no earlier row has it; until that
  // is known it reads (only) slot 0's states
  const int named = slots ? slots[b] : b;
  const int slot = named >= 0 && named < nslots ? named : 0;
  int skip = named != slot;
  if (slots)
    for (int j = tid; j < b; j += kThreads) skip |= slots[j] == named;

  // loads in the order of their use: the convolution's, then the first pass of
  // the state, which is in flight while the convolution is computed
  float* cs = conv + static_cast<size_t>(slot) * 3 * Ch;
  const T* row = xbc + static_cast<size_t>(b) * ldx;
  auto channel = [&](int i) {
    return i < P ? hh * P + i : i < P + N ? HP + g * N + (i - P) : HP + GN + g * N + (i - P - N);
  };
  float s0[CI], s1[CI], s2[CI], s3[CI], bs[CI];
  float4 q[CI];
#pragma unroll
  for (int k = 0; k < CI; ++k) {
    const int c = channel(min(tid + k * kThreads, nch - 1));
    s0[k] = cs[c], s1[k] = cs[Ch + c], s2[k] = cs[2 * Ch + c], s3[k] = elem<T>(row[c]);
    q[k] = *reinterpret_cast<const float4*>(w + static_cast<size_t>(c) * 4);
    bs[k] = bias ? bias[c] : 0.0f;
  }
  const int col = tid % LPR, rsub = tid / LPR;
  float* hrow = hpool + (static_cast<size_t>(slot) * H + hh) * P * N + col * 4;
  f4v v[UNR];
  auto load_rows = [&](int r0) {
#pragma unroll
    for (int k = 0; k < UNR; ++k) {
      const int r = min(r0 + k * RPP, P - 1);
      v[k] = __builtin_nontemporal_load(reinterpret_cast<const f4v*>(hrow + static_cast<size_t>(r) * N));
    }
  };
  load_rows(rsub);

  auto conv_value = [&](float a0, float a1, float a2, float a3, float4 t, float bb) {
    float o = fmaf(t.w, a3, fmaf(t.z, a2, fmaf(t.y, a1, fmaf(t.x, a0, bb))));
    if (act) o *= __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(o * -1.4426950408889634f));
    return o;
  };
#pragma unroll
  for (int k = 0; k < CI; ++k) {
    const int i = tid + k * kThreads;
    if (i < nch) lds[i] = conv_value(s0[k], s1[k], s2[k], s3[k], q[k], bs[k]);
  }
  for (int i = tid + CI * kThreads; i < nch; i += kThreads) {  // P + 2N > 512
    const int c = channel(i);
    lds[i] = conv_value(cs[c], cs[Ch + c], cs[2 * Ch + c], elem<T>(row[c]),
                        *reinterpret_cast<const float4*>(w + static_cast<size_t>(c) * 4), bias ? bias[c] : 0.0f);
  }
  skip = __syncthreads_or(skip);
  if (skip) {  // a padding row
    for (int p = tid; p < P; p += kThreads) {
      if (y_bf16)
        static_cast<uint16_t*>(y)[yrow + p] = 0;
      else
        static_cast<float*>(y)[yrow + p] = 0.0f;
    }
    return;
  }
  // every conv value of this workgroup has arrived: count it in at the group's
  // B and C, and move this head's own channels up
  const bool alone = H == G;
  unsigned arrived = 0;
  if (!alone && tid == 0)
    arrived = atomicInc(arrivals + static_cast<size_t>(slot) * G + g, static_cast<unsigned>(H / G - 1));
  const int own = alone ? nch : P;
#pragma unroll
  for (int k = 0; k < CI; ++k) {
    const int i = tid + k * kThreads;
    if (i < own) {
      const int c = channel(i);
      cs[c] = s1[k], cs[Ch + c] = s2[k], cs[2 * Ch + c] = s3[k];
    }
  }
  for (int i = tid + CI * kThreads; i < own; i += kThreads) {
    const int c = channel(i);
    const float m1 = cs[Ch + c], m2 = cs[2 * Ch + c];
    cs[c] = m1, cs[Ch + c] = m2, cs[2 * Ch + c] = elem<T>(row[c]);
  }

  const float delta = step_size(elem<T>(dt[static_cast<size_t>(b) * lddt + hh]), dt_bias ? dt_bias[hh] : 0.0f, lo, hi);
  const float a = __expf(A[hh] * delta);
  const float Dh = D ? D[hh] : 0.0f;
  float bq[4], cq[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) bq[k] = lds[P + col * 4 + k], cq[k] = lds[P + N + col * 4 + k];
  for (int r0 = rsub; r0 < P; r0 += UNR * RPP) {
    if (r0 != rsub) load_rows(r0);
#pragma unroll
    for (int k = 0; k < UNR; ++k) {
      const int r = r0 + k * RPP;
      float part = 0.0f, xv = 0.0f;
      if (r < P) {
        xv = lds[r];
        const float u = delta * xv;
        f4v n;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          n[i] = a * v[k][i] + u * bq[i];
          part = fmaf(n[i], cq[i], part);
        }
        __builtin_nontemporal_store(n, reinterpret_cast<f4v*>(hrow + static_cast<size_t>(r) * N));
      }
#pragma unroll
      for (int o = LPR / 2; o > 0; o >>= 1) part += __shfl_xor(part, o, kWave);
      if (r < P && col == 0) {
        const float out = part + Dh * xv;
        if (y_bf16)
          static_cast<uint16_t*>(y)[yrow + r] = static_cast<uint16_t>(pack_bf16x2(out, 0.0f) & 0xFFFFu);
        else
          static_cast<float*>(y)[yrow + r] = out;
      }
    }
  }

  if (alone) return;
  __shared__ int last;
  if (tid == 0) last = arrived == static_cast<unsigned>(H / G - 1);
  __syncthreads();
  if (!last) return;
  for (int i = tid; i < 2 * N; i += kThreads) {
    const int c = channel(P + i);
    const float m1 = cs[Ch + c], m2 = cs[2 * Ch + c];
    cs[c] = m1, cs[Ch + c] = m2, cs[2 * Ch + c] = elem<T>(row[c]);
  }
}

template <typename T>
hipError_t mixer_step_t(const MixerStepArgs& a, hipStream_t st) {
  const dim3 grid(a.Bsz * a.H);
  const size_t shared = static_cast<size_t>(a.P + 2 * a.N) * sizeof(float);
#define SSD_STEP_CASE(NN)                                                                            \
  case NN:                                                                                           \
    hipLaunchKernelGGL((ssd_mixer_step_kernel<NN, T>), grid, dim3(kThreads), shared, st, a.conv,   \
                         a.h, a.arrivals, a.slots, a.nslots, static_cast<const T*>(a.xbc), a.ldx,    \
                         static_cast<const T*>(a.dt), a.lddt, a.w, a.bias, a.act, a.A, a.D,          \
                         a.dt_bias, a.dt_min, a.dt_max, a.y, a.y_dtype, a.H, a.P, a.G);              \
    break;
  switch (a.N) {
    SSD_STEP_CASE(16)
    SSD_STEP_CASE(32)
    SSD_STEP_CASE(64)
    SSD_STEP_CASE(128)
    SSD_STEP_CASE(256)
    default:
      return hipErrorInvalidValue;
  }
#undef SSD_STEP_CASE
  return hipGetLastError();
}

}  // namespace

hipError_t run_mixer_step(const MixerStepArgs& a, hipStream_t st) {
  return a.dtype == 1 ? mixer_step_t<uint16_t>(a, st) : mixer_step_t<float>(a, st);
}

}  // namespace ssd
