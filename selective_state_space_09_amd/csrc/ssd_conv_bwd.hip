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
// The operation streams (x and dout in, dx out).  A lane owns V channels and
// walks a run of kRun tokens with the windows of inputs and gradients and the
// channels' five sums in registers, so a row is read once per run (plus halo
// rows that the cache serves).  To write din_p it needs g up to p + 3: it
// starts with g_{t0..t0+2} and then, for each p, makes g_{p+3} and din_p.  The
// sums take the tokens t = p + 3 (and 0..2 in a sequence's first run), so every
// token is counted once without a mask.  Loads and stores are buffer accesses whose offsets are
// pushed out of range where nothing may be touched, so no access sits in a
// branch, and a block of kBlk tokens is loaded while the one before it is
// computed.
//
// Workgroups own channels of one of the three outputs x, B, C (whose gradients
// differ in type).  The four waves of a workgroup take runs of the same
// channels and join their sums in LDS; each workgroup writes one row of a
// partial-sum table that a second kernel adds up in a fixed order.

#include <type_traits>

#include "ssd_chunk_common.h"
#include "ssd_internal.h"
#include "ssd_rows.h"

namespace ssd {

namespace {

// Measured at 2 x 2048 tokens of 4352 bf16 channels (both kernels): V = 2, runs
// of 32, blocks of 8 30.9 us; blocks of 4 31.9; runs of 16 31.9, of 64 33.3
// (fewer waves); V = 4 42.9 (half the waves at twice the registers).
constexpr int kV = 2;      // channels per lane
constexpr int kRun = 32;   // tokens per run
constexpr int kBlk = 8;    // tokens loaded together
constexpr int kMaxParts = 256;
constexpr uint32_t kOOB = 0xFFFFFFF0u;

// V elements of type T at a byte offset of a buffer, as raw words
template <typename T, int V>
struct Raw {
  static constexpr int BYTES = sizeof(T) * V, WORDS = BYTES / 4;
  uint32_t w[WORDS];
  __device__ __forceinline__ void load(buf_t b, uint32_t off) {
    if constexpr (BYTES == 4) {
      w[0] = __builtin_amdgcn_raw_buffer_load_b32(b, off, 0, 0);
    } else if constexpr (BYTES == 8) {
      const uint2 q = buf_load8(b, off);
      w[0] = q.x, w[1] = q.y;
    } else {
      const uint4 q = buf_load16(b, off);
      w[0] = q.x, w[1] = q.y, w[2] = q.z, w[3] = q.w;
    }
  }
  __device__ __forceinline__ float at(int v) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(w[v]);
    return __uint_as_float(v & 1 ? w[v >> 1] & 0xFFFF0000u : w[v >> 1] << 16);
  }
  __device__ __forceinline__ static void store(buf_t b, uint32_t off, const float* f) {
    uint32_t w[WORDS];
#pragma unroll
    for (int i = 0; i < WORDS; ++i)
      w[i] = sizeof(T) == 4 ? __float_as_uint(f[i]) : pack_bf16x2(f[2 * i], f[2 * i + 1]);
    if constexpr (BYTES == 4)
      __builtin_amdgcn_raw_buffer_store_b32(w[0], b, off, 0, 0);
    else if constexpr (BYTES == 8)
      buf_store8(b, off, make_uint2(w[0], w[1]));
    else
      buf_store16(b, off, make_uint4(w[0], w[1], w[2], w[3]));
  }
};

// One workgroup's share of a channel region of TD gradients: lane channels c
// .. c+V-1 of the row (region channel cr of width W), runs `first`, first +
// stride, ...
template <typename T, typename TD, bool SILU>
__device__ __forceinline__ void conv_bwd_body(
    const T* __restrict__ xbc, long long ld, const float* __restrict__ w,
    const float* __restrict__ bias, const float* __restrict__ state_in, const TD* __restrict__ dout,
    const float* __restrict__ dstate_out, T* __restrict__ dxbc, long long lddx,
    float* __restrict__ dstate_in, int Bsz, int Tn, int Ch, int c, int cr, int W, bool active,
    long long first, long long stride, float (&dw)[kV][4], float (&db)[kV]) {
  constexpr int V = kV;
  const int nruns = Tn > 0 ? (Tn + kRun - 1) / kRun : 1;
  const long long units = static_cast<long long>(Bsz) * nruns;
  float wt[V][4], bs[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const float4 q = *reinterpret_cast<const float4*>(w + static_cast<size_t>(active ? c + v : 0) * 4);
    wt[v][0] = q.x, wt[v][1] = q.y, wt[v][2] = q.z, wt[v][3] = q.w;
    bs[v] = bias && active ? bias[c + v] : 0.0f;
  }
  const uint32_t lim = 3u * static_cast<uint32_t>(Ch) * 4u;

  for (long long u = first; u < units; u += stride) {
    const int b = static_cast<int>(u / nruns);
    const int t0 = static_cast<int>(u % nruns) * kRun;
    const int base = t0 >= 3 ? t0 - 3 : 0;           // first row that the run reads
    const int rows = min(Tn - base, kRun + 6);       // rows it may read
    const size_t r0 = static_cast<size_t>(b) * Tn + base;
    const buf_t xb = make_buf(xbc + r0 * ld, static_cast<uint32_t>(rows * ld * sizeof(T)));
    const buf_t gb = make_buf(dout + r0 * W, static_cast<uint32_t>(static_cast<size_t>(rows) * W * sizeof(TD)));
    const buf_t ob = make_buf(dxbc + r0 * lddx, static_cast<uint32_t>(rows * lddx * sizeof(T)));
    const size_t so = static_cast<size_t>(b) * 3 * Ch;
    const buf_t sb = make_buf(state_in + so, state_in ? lim : 0u);
    const buf_t eb = make_buf(dstate_out + so, dstate_out ? lim : 0u);
    auto off_x = [&](int p, long long pitch) -> uint32_t {  // row p of the sequence
      return active && p >= 0 && p < Tn ? static_cast<uint32_t>(((p - base) * pitch + c) * sizeof(T)) : kOOB;
    };
    auto off_g = [&](int p) -> uint32_t {
      return active && p < Tn ? static_cast<uint32_t>(((p - base) * static_cast<long long>(W) + cr) * sizeof(TD)) : kOOB;
    };
    auto off_s = [&](int row) -> uint32_t {  // row of a (3, Ch) state
      return active && row >= 0 && row < 3 ? (static_cast<uint32_t>(row) * Ch + c) * 4u : kOOB;
    };
    Raw<T, V> px[6];
    Raw<float, V> ps[3];
    Raw<TD, V> pg[3];
#pragma unroll
    for (int j = 0; j < 3; ++j) {
      px[j].load(xb, off_x(t0 - 3 + j, ld));
      ps[j].load(sb, off_s(t0 + j));  // position t0 - 3 + j where that is negative
    }
#pragma unroll
    for (int j = 0; j < 3; ++j) {
      px[3 + j].load(xb, off_x(t0 + j, ld));
      pg[j].load(gb, off_g(t0 + j));
    }
    Raw<T, V> nx[kBlk];
    Raw<TD, V> ng[kBlk];
#pragma unroll
    for (int i = 0; i < kBlk; ++i) {
      nx[i].load(xb, off_x(t0 + 3 + i, ld));
      ng[i].load(gb, off_g(t0 + 3 + i));
    }

    float win[3][V], gw[3][V];  // inputs t-3 .. t-1, gradients t-3 .. t-1
    // a state row is read only where the position is negative (t0 = 0), and
    // there the input row reads as zero: one of the two is zero
#pragma unroll
    for (int j = 0; j < 3; ++j)
#pragma unroll
      for (int v = 0; v < V; ++v) win[j][v] = px[j].at(v) + (t0 == 0 ? ps[j].at(v) : 0.0f);

    auto grad = [&](float x, float d, int v) -> float {
      if constexpr (!SILU) return d;
      float a = bs[v];
#pragma unroll
      for (int j = 0; j < 3; ++j) a = fmaf(wt[v][j], win[j][v], a);
      a = fmaf(wt[v][3], x, a);
      const float s = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(a * -1.4426950408889634f));
      return d * s * fmaf(a, 1.0f - s, 1.0f);
    };
    auto count = [&](float x, float g, int v) {
      db[v] += g;
#pragma unroll
      for (int j = 0; j < 3; ++j) dw[v][j] = fmaf(g, win[j][v], dw[v][j]);
      dw[v][3] = fmaf(g, x, dw[v][3]);
    };
#pragma unroll
    for (int i = 0; i < 3; ++i) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float x = px[3 + i].at(v);
        float g = 0.0f;
        if (t0 + i < Tn) {
          g = grad(x, pg[i].at(v), v);
          if (t0 == 0) count(x, g, v);
        }
        gw[i][v] = g;
        win[0][v] = win[1][v], win[1][v] = win[2][v], win[2][v] = x;
      }
    }
    if (t0 == 0 && dstate_in) {  // positions -3, -2, -1: the carried state's gradient
      const buf_t db_ = make_buf(dstate_in + so, lim);
#pragma unroll
      for (int j = 0; j < 3; ++j) {
        Raw<float, V> e;
        e.load(eb, off_s(j - Tn));  // dstate_out row p - (T - 3), p = j - 3
        float o[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
          o[v] = e.at(v);
#pragma unroll
          for (int i = 0; i <= j; ++i) o[v] = fmaf(wt[v][j - i], gw[i][v], o[v]);
        }
        Raw<float, V>::store(db_, off_s(j), o);
      }
    }
    // the gradients of positions p0 .. p0 + kBlk - 1; at the sequence's end
    // (EDGE) tokens past it count for nothing and dstate_out is added
    auto block = [&](auto edge, int p0, const Raw<T, V>* cx, const Raw<TD, V>* cg) {
#pragma unroll
      for (int i = 0; i < kBlk; ++i) {
        const int p = p0 + i;
        float o[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const float x = cx[i].at(v);
          float g = 0.0f;
          if (!edge.value || p + 3 < Tn) {
            g = grad(x, cg[i].at(v), v);
            count(x, g, v);
          }
          o[v] = fmaf(wt[v][3], gw[0][v], fmaf(wt[v][2], gw[1][v], fmaf(wt[v][1], gw[2][v], wt[v][0] * g)));
          gw[0][v] = gw[1][v], gw[1][v] = gw[2][v], gw[2][v] = g;
          win[0][v] = win[1][v], win[1][v] = win[2][v], win[2][v] = x;
        }
        if constexpr (edge.value) {
          if (dstate_out && p >= Tn - 3) {
            Raw<float, V> e;
            e.load(eb, off_s(p - (Tn - 3)));
#pragma unroll
            for (int v = 0; v < V; ++v) o[v] += e.at(v);
          }
        }
        Raw<T, V>::store(ob, off_x(p, lddx), o);
      }
    };
#pragma unroll 1
    for (int p0 = t0; p0 < min(t0 + kRun, Tn); p0 += kBlk) {
      Raw<T, V> cx[kBlk];
      Raw<TD, V> cg[kBlk];
#pragma unroll
      for (int i = 0; i < kBlk; ++i) cx[i] = nx[i], cg[i] = ng[i];
      if (p0 + kBlk < t0 + kRun) {
#pragma unroll
        for (int i = 0; i < kBlk; ++i) {
          nx[i].load(xb, off_x(p0 + kBlk + 3 + i, ld));
          ng[i].load(gb, off_g(p0 + kBlk + 3 + i));
        }
      }
      if (p0 + kBlk + 3 <= Tn)
        block(std::false_type{}, p0, cx, cg);
      else
        block(std::true_type{}, p0, cx, cg);
    }
  }
}

// channel blocks of one output
inline __host__ __device__ int region_blocks(int W) { return (W / kV + kWave - 1) / kWave; }

// Grid: x = channel blocks of x, then B, then C; y = workgroups over the
// (sequence, run) units, four at a time.
template <typename T, bool SILU>
__global__ __launch_bounds__(kThreads) void ssd_conv1d_bwd_kernel(
    const T* __restrict__ xbc, long long ld, const float* __restrict__ w,
    const float* __restrict__ bias, const float* __restrict__ state_in, const T* __restrict__ dx,
    const float* __restrict__ dB, const float* __restrict__ dC,
    const float* __restrict__ dstate_out, T* __restrict__ dxbc, long long lddx,
    float* __restrict__ dstate_in, float* __restrict__ part, int Bsz, int Tn, int HP, int GN) {
  const int Ch = HP + 2 * GN;
  const int wid = wave_id(), lane = threadIdx.x & (kWave - 1);
  const long long first = static_cast<long long>(blockIdx.y) * 4 + wid, stride = static_cast<long long>(gridDim.y) * 4;
  const int nx = region_blocks(HP), ng = region_blocks(GN), bx = blockIdx.x;
  float dw[kV][4] = {}, db[kV] = {};
  int c;
  bool active;
  if (bx < nx) {
    c = (bx * kWave + lane) * kV;
    active = c < HP;
    conv_bwd_body<T, T, SILU>(xbc, ld, w, bias, state_in, dx, dstate_out, dxbc, lddx, dstate_in, Bsz, Tn, Ch, c, c,
                              HP, active, first, stride, dw, db);
  } else {
    const bool isC = bx >= nx + ng;
    const int cr = ((bx - nx - (isC ? ng : 0)) * kWave + lane) * kV;
    c = HP + (isC ? GN : 0) + cr;
    active = cr < GN;
    conv_bwd_body<T, float, SILU>(xbc, ld, w, bias, state_in, isC ? dC : dB, dstate_out, dxbc, lddx, dstate_in, Bsz,
                                  Tn, Ch, c, cr, GN, active, first, stride, dw, db);
  }

  // join the four waves: columns 4 c + j hold dw, 4 Ch + c dbias
  __shared__ float buf[3][kV * 5][kWave];
  if (wid > 0) {
#pragma unroll
    for (int v = 0; v < kV; ++v) {
#pragma unroll
      for (int j = 0; j < 4; ++j) buf[wid - 1][v * 5 + j][lane] = dw[v][j];
      buf[wid - 1][v * 5 + 4][lane] = db[v];
    }
  }
  __syncthreads();
  if (wid == 0 && active) {
    float* p = part + static_cast<size_t>(blockIdx.y) * 5 * Ch;
#pragma unroll
    for (int v = 0; v < kV; ++v) {
#pragma unroll
      for (int k = 0; k < 3; ++k) {
#pragma unroll
        for (int j = 0; j < 4; ++j) dw[v][j] += buf[k][v * 5 + j][lane];
        db[v] += buf[k][v * 5 + 4][lane];
      }
      *reinterpret_cast<float4*>(p + static_cast<size_t>(c + v) * 4) = make_float4(dw[v][0], dw[v][1], dw[v][2], dw[v][3]);
      p[4 * static_cast<size_t>(Ch) + c + v] = db[v];
    }
  }
}

template <typename T>
void launch_conv_bwd(const ConvBwdArgs& a, hipStream_t st) {
  const dim3 grid(region_blocks(a.HP) + 2 * region_blocks(a.GN), conv_bwd_parts(a.Bsz, a.T));
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
