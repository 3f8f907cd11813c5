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
// traffic, so HBM bounds a large batch and latency a small one.  A workgroup
// serves HB heads of one row and group: 256 threads per head for the state, as
// in the decode kernel, and one more wave for the convolution.  The state's
// first rows are in flight while that wave convolves the heads' P channels and
// the group's B and C into LDS (a group's workgroups repeat B and C: 2N channels
// against HB P N state values, from the cache).  The roles are separate waves
// because a wave waits for its memory operations in their order: with both in
// one wave the state's arithmetic would wait for the counter and the shifted
// rows behind its loads (256 rows of 64 heads: 189 us, in one role 193; one row:
// 6.5 us against 6.8).
//
// The conv rows of a workgroup's own x channels are moved up by its conv wave;
// those of B and C are still being read by the group's other workgroups, so
// each counts itself in at the slot's arrivals counter once it has read them,
// and the last one moves them (the counter wraps to zero by itself).  No
// workgroup waits for another.  Two heads a workgroup halve the counting and
// the repeated B and C: 8 rows of 64 heads in one group 9.9 us, with one head
// 12.3 us; one row 6.5 and 6.2.
//
// A row looks through the slots of the rows before it (no workspace, no second
// launch); past 256 rows in vectors of four, eight in flight: 4096 rows of
// H = P = 64, N = 128 2976 us, without a slot map 2797, with one load at a time
// 3631; 16384 rows of H = 8, P = 32, N = 16 767, 492 and 2521.
//
// Measured at 256 rows of H = P = 64, N = 128, one group (1.11 GB): 190 us, 5.8
// TB/s.  ssd_conv1d_step and ssd_step_decode on the same states, their float32
// inputs ready and row b on slot b, take 6.1 + 180 us there, 3.4 + 45.0 at 64 rows
// (this kernel 53.5), 2.8 + 24.8 at 32 (30.3), 2.7 + 13.4 at 16 (16.7), 2.6 + 7.7
// at 8 (10.2) and 2.5 + 4.8 at one (6.7).  From 16 rows on the one launch takes
// more than the two together, most at 32 rows: 1024 workgroups of nine waves and
// 72 registers, of which 768 are resident.  What it gives for that are slots and
// padding in a pool, and bf16 in_proj rows read in place, which the two kernels'
// caller first has to gather and widen.

#include "ssd_chunk_common.h"
#include "ssd_internal.h"

namespace ssd {

namespace {

typedef float f4v __attribute__((ext_vector_type(4)));
typedef int i4_e4 __attribute__((ext_vector_type(4), aligned(4)));  // at any element

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

template <int N, int HB, typename T>
__global__ __launch_bounds__(kThreads* HB + kWave) void ssd_mixer_step_kernel(
    float* __restrict__ conv, float* __restrict__ hpool, unsigned* __restrict__ arrivals,
    const int* __restrict__ slots, int nslots, const T* __restrict__ xbc, long long ldx,
    const T* __restrict__ dt, long long lddt, const float* __restrict__ w,
    const float* __restrict__ bias, int act, const float* __restrict__ A,
    const float* __restrict__ D, const float* __restrict__ dt_bias, float lo, float hi,
    void* __restrict__ y, int y_bf16, int H, int P, int G) {
  extern __shared__ float lds[];  // x (HB P), B (N), C (N)
  __shared__ int padding;
  constexpr int LPR = N / 4;            // lanes per state row
  constexpr int RPP = kThreads / LPR;   // rows covered by one pass of a head's threads
  constexpr int UNR = 8;                // rows in flight per thread
  constexpr int CI = 6;                 // convolved channels in flight per lane
  const int HW = H / HB;                // workgroups per row
  const int b = blockIdx.x / HW, h0 = (blockIdx.x % HW) * HB, g = h0 / (H / G);
  const int HP = H * P, GN = G * N, Ch = HP + 2 * GN, xch = HB * P, nch = xch + 2 * N;

  // a row takes part if its slot exists and no earlier row has it; until that
  // is known the workgroup reads (only) slot 0's states
  const int named = slots ? slots[b] : b;
  const int slot = named >= 0 && named < nslots ? named : 0;

  if (wave_id() == HB * (kThreads / kWave)) {  // the wave that convolves
    const int lane = threadIdx.x & (kWave - 1);
    float* cs = conv + static_cast<size_t>(slot) * 3 * Ch;
    const T* row = xbc + static_cast<size_t>(b) * ldx;
    auto channel = [&](int i) {
      return i < xch       ? h0 * P + i
             : i < xch + N ? HP + g * N + (i - xch)
                           : HP + GN + g * N + (i - xch - N);
    };
    // the slots of the rows before it are looked at after the convolution; the
    // first ones are in flight with its loads
    const int* map = slots ? slots : reinterpret_cast<const int*>(A);
    constexpr int FI = 4;
    int first[FI];
#pragma unroll
    for (int k = 0; k < FI; ++k) first[k] = map[slots ? min(lane + k * kWave, b) : 0];
#pragma unroll 1
    for (int k0 = lane; k0 < nch; k0 += CI * kWave) {
      float s0[CI], s1[CI], s2[CI], s3[CI], bs[CI];
      float4 q[CI];
#pragma unroll
      for (int k = 0; k < CI; ++k) {
        const int c = channel(min(k0 + k * kWave, nch - 1));
        s3[k] = elem<T>(row[c]);
        q[k] = *reinterpret_cast<const float4*>(w + static_cast<size_t>(c) * 4);
        bs[k] = bias ? bias[c] : 0.0f;
        s0[k] = cs[c], s1[k] = cs[Ch + c], s2[k] = cs[2 * Ch + c];
      }
#pragma unroll
      for (int k = 0; k < CI; ++k) {
        float o = fmaf(q[k].w, s3[k], fmaf(q[k].z, s2[k], fmaf(q[k].y, s1[k], fmaf(q[k].x, s0[k], bs[k]))));
        if (act) o *= __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(o * -1.4426950408889634f));
        if (k0 + k * kWave < nch) lds[k0 + k * kWave] = o;
      }
    }
    int skip = named != slot;
#pragma unroll
    for (int k = 0; k < FI; ++k) skip |= slots && lane + k * kWave < b && first[k] == named;
    if (slots) {  // the rest, b >= FI kWave: vectors of four, the last ones shifted back into the rows before b
      constexpr int U = 8;
#pragma unroll 1
      for (int j0 = FI * kWave; j0 < b; j0 += U * 4 * kWave) {
        i4_e4 q[U];
#pragma unroll
        for (int k = 0; k < U; ++k)
          q[k] = *reinterpret_cast<const i4_e4*>(slots + min(j0 + (k * kWave + lane) * 4, b - 4));
#pragma unroll
        for (int k = 0; k < U; ++k)
#pragma unroll
          for (int i = 0; i < 4; ++i) skip |= q[k][i] == named;
      }
    }
    skip = __any(skip);
    if (lane == 0) padding = skip;
    __syncthreads();
    if (skip) return;
    // Every conv value of this workgroup has arrived.  Count it in at the
    // group's B and C, move the channels up that no other workgroup reads (all
    // of them if there is none), and, as the last one in, those of B and C.
    const unsigned others = H / G / HB - 1;  // workgroups of the group besides this one
    unsigned arrived = 0;
    if (others && lane == 0) arrived = atomicInc(arrivals + static_cast<size_t>(slot) * G + g, others);
    auto shift = [&](int from, int to) {  // channels i, from <= i < to
      for (int i = from + lane; i < to; i += kWave) {
        const int c = channel(i);
        const float m1 = cs[Ch + c], m2 = cs[2 * Ch + c], m3 = elem<T>(row[c]);
        cs[c] = m1, cs[Ch + c] = m2, cs[2 * Ch + c] = m3;
      }
    };
    shift(0, xch);
    if (__shfl(arrived, 0) == others) shift(xch, nch);
    return;
  }

  // the waves of the state: their first rows are in flight while the
  // convolution is computed
  const int ht = wave_id() / (kThreads / kWave), hh = h0 + ht, tid = threadIdx.x % kThreads;
  const int col = tid % LPR, rsub = tid / LPR;
  const float dtv = elem<T>(dt[static_cast<size_t>(b) * lddt + hh]), dtb = dt_bias ? dt_bias[hh] : 0.0f;
  const float Ah = A[hh], Dh = D ? D[hh] : 0.0f;
  float* state = hpool + (static_cast<size_t>(slot) * H + hh) * P * N;  // uniform; 32-bit offsets per lane
  const size_t yrow = (static_cast<size_t>(b) * H + hh) * P;
  auto put_y = [&](int r, float v) {
    if (y_bf16)
      static_cast<uint16_t*>(y)[yrow + r] = static_cast<uint16_t>(pack_bf16x2(v, 0.0f) & 0xFFFFu);
    else
      static_cast<float*>(y)[yrow + r] = v;
  };
  f4v v[UNR];
  auto load_rows = [&](int r0) {
#pragma unroll
    for (int k = 0; k < UNR; ++k) {
      const uint32_t at = min(r0 + k * RPP, P - 1) * N + col * 4;
      v[k] = __builtin_nontemporal_load(reinterpret_cast<const f4v*>(state + at));
    }
  };
  load_rows(rsub);
  const float delta = step_size(dtv, dtb, lo, hi);
  const float a = __expf(Ah * delta);
  __syncthreads();
  if (padding) {
    for (int p = tid; p < P; p += kThreads) put_y(p, 0.0f);
    return;
  }
  float bq[4], cq[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) bq[k] = lds[xch + col * 4 + k], cq[k] = lds[xch + N + col * 4 + k];
  for (int r0 = rsub; r0 < P; r0 += UNR * RPP) {
    if (r0 != rsub) load_rows(r0);
#pragma unroll
    for (int k = 0; k < UNR; ++k) {
      const int r = r0 + k * RPP;
      float part = 0.0f, xv = 0.0f;
      if (r < P) {
        xv = lds[ht * P + r];
        const float u = delta * xv;
        f4v n;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          n[i] = a * v[k][i] + u * bq[i];
          part = fmaf(n[i], cq[i], part);
        }
        const uint32_t at = r * N + col * 4;
        __builtin_nontemporal_store(n, reinterpret_cast<f4v*>(state + at));
      }
#pragma unroll
      for (int o = LPR / 2; o > 0; o >>= 1) part += __shfl_xor(part, o, kWave);
      if (r < P && col == 0) put_y(r, part + Dh * xv);
    }
  }
}

template <int HB, typename T>
hipError_t mixer_step_t(const MixerStepArgs& a, hipStream_t st) {
  const dim3 grid(static_cast<unsigned>(a.Bsz) * (a.H / HB));
  const size_t shared = static_cast<size_t>(HB * a.P + 2 * a.N) * sizeof(float);
#define SSD_STEP_CASE(NN)                                                                              \
  case NN:                                                                                             \
    hipLaunchKernelGGL((ssd_mixer_step_kernel<NN, HB, T>), grid, dim3(kThreads * HB + kWave), shared, st, a.conv, \
                       a.h, a.arrivals, a.slots, a.nslots, static_cast<const T*>(a.xbc), a.ldx,        \
                       static_cast<const T*>(a.dt), a.lddt, a.w, a.bias, a.act, a.A, a.D, a.dt_bias,   \
                       a.dt_min, a.dt_max, a.y, a.y_dtype, a.H, a.P, a.G);                             \
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
  if (a.H / a.G % 2 == 0)  // two heads of a group per workgroup (figures above)
    return a.dtype == 1 ? mixer_step_t<2, uint16_t>(a, st) : mixer_step_t<2, float>(a, st);
  return a.dtype == 1 ? mixer_step_t<1, uint16_t>(a, st) : mixer_step_t<1, float>(a, st);
}

}  // namespace ssd
