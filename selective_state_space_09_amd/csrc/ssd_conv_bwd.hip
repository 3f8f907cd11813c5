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
// walks a run of 8 to 32 tokens with the windows of inputs and gradients and the
// channels' five sums in registers, so a row is read once per run (plus halo
// rows that the cache serves).  To write din_p it needs g up to p + 3: it
// starts with g_{t0..t0+2} and then, for each p, makes g_{p+3} and din_p.  The
// sums take the tokens t = p + 3 (and 0..2 in a sequence's first run), so every
// token is counted once without a mask.  Loads and stores are buffer accesses
// with one descriptor per row, made in scalar registers: a row outside the
// sequence has an empty one (loads give zero, stores are dropped), a lane
// without channels an offset past every row.  So no access sits in a branch, a
// lane's offset never changes, and a block of kBlk tokens is loaded while the
// one before it is computed.
//
// Workgroups own channels of one of the three outputs x, B, C (whose gradients
// differ in type).  The four waves of a workgroup take runs of the same
// channels and join their sums in LDS; each workgroup writes one row of a
// partial-sum table that a second kernel adds up in a fixed order.
//
// What bounds it: the bytes (2 x 2048 tokens of 4352 bf16 channels: 109 MB, 21.7
// us as one elementwise library kernel) and, close behind, the instructions: 30
// of the VALU per element, two of them quarter-rate, 14.8 us, and three scalar
// ones to every four of them (the descriptors; with SiLU 13 or 14 scalar registers
// are spilled to vector lanes).  28.3 us a call, 3.9 TB/s; in a trace 26.9 us (25.4
// at least) for this kernel and 4.0 for the sums.  Few channels leave lanes idle:
// 8 x 4096 tokens of 80 bf16 channels 21.7 us, 0.8 TB/s.

#include "ssd_chunk_common.h"
#include "ssd_internal.h"
#include "ssd_rows.h"

namespace ssd {

namespace {

// Measured at 2 x 2048 tokens of 4352 bf16 channels (both kernels; the whole
// call's bytes as one elementwise library kernel: 21.7 us), runs of 32: V = 2,
// blocks of 4 31.4 us, blocks of 8 34.3; with a second copy of the block's code
// for its last tokens 33.4 (4) and 32.0 (8); one descriptor per run and the row
// in the lane's offset 34.4 (8); V = 4 42.9 (half the waves).
constexpr int kV = 2;       // channels per lane
constexpr int kRunMax = 32;  // tokens per run, at most (a multiple of kBlk)
constexpr int kBlk = 4;    // tokens loaded together
constexpr int kMaxParts = 256;
// past every row and every (3, Ch) state, also with a state row's offset added
constexpr uint32_t kOut = 0x60000000u;

// V elements of type T at a byte offset of a buffer, as raw words
template <typename T, int V>
struct Raw {
  static constexpr int BYTES = sizeof(T) * V, WORDS = BYTES / 4;
  static_assert(BYTES == 4 || BYTES == 8, "one or two words");
  uint32_t w[WORDS];
  __device__ __forceinline__ void load(buf_t b, uint32_t off) {
    if constexpr (BYTES == 4) {
      w[0] = __builtin_amdgcn_raw_buffer_load_b32(b, off, 0, 0);
    } else {
      const uint2 q = buf_load8(b, off);
      w[0] = q.x, w[1] = q.y;
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
    else
      buf_store8(b, off, make_uint2(w[0], w[1]));
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
    int run, long long first, long long stride, float (&dw)[kV][4], float (&db)[kV]) {
  constexpr int V = kV;
  const int nruns = Tn > 0 ? (Tn - 1) / run + 1 : 1;
  const long long units = static_cast<long long>(Bsz) * nruns;
  float wt[V][4], bs[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const float4 q = *reinterpret_cast<const float4*>(w + static_cast<size_t>(active ? c + v : 0) * 4);
    wt[v][0] = q.x, wt[v][1] = q.y, wt[v][2] = q.z, wt[v][3] = q.w;
    bs[v] = bias && active ? bias[c + v] : 0.0f;
  }
  const uint32_t xlane = active ? static_cast<uint32_t>(c * sizeof(T)) : kOut;
  const uint32_t glane = active ? static_cast<uint32_t>(cr * sizeof(TD)) : kOut;
  const uint32_t slane = active ? static_cast<uint32_t>(c) * 4u : kOut;
  const long long xpitch = ld * static_cast<long long>(sizeof(T)), opitch = lddx * static_cast<long long>(sizeof(T));
  const long long gpitch = W * static_cast<long long>(sizeof(TD));
  const uint32_t xbytes = static_cast<uint32_t>(Ch * sizeof(T)), gbytes = static_cast<uint32_t>(W * sizeof(TD));
  const uint32_t sbytes = 3u * static_cast<uint32_t>(Ch) * 4u;

  for (long long u = first; u < units; u += stride) {
    const int b = static_cast<int>(u / nruns);
    const int t0 = static_cast<int>(u % nruns) * run;
    const long long r0 = static_cast<long long>(b) * Tn;
    // rows are taken in order, each stream by a pointer that moves a row at a
    // time: inputs from t0 - 3, gradients and results from t0
    const char* xp = reinterpret_cast<const char*>(xbc) + (r0 + t0 - 3) * xpitch;
    const char* gp = reinterpret_cast<const char*>(dout) + (r0 + t0) * gpitch;
    char* op = reinterpret_cast<char*>(dxbc) + (r0 + t0) * opitch;
    auto xrow = [&](int p) {
      const buf_t r = make_buf(xp, p >= 0 && p < Tn ? xbytes : 0u);
      xp += xpitch;
      return r;
    };
    auto grow = [&](int p) {
      const buf_t r = make_buf(gp, p < Tn ? gbytes : 0u);
      gp += gpitch;
      return r;
    };
    auto orow = [&](int p) {
      const buf_t r = make_buf(op, p < Tn ? xbytes : 0u);
      op += opitch;
      return r;
    };
    const size_t so = static_cast<size_t>(b) * 3 * Ch;
    const buf_t sb = make_buf(state_in + so, state_in ? sbytes : 0u);
    const buf_t eb = make_buf(dstate_out + so, dstate_out ? sbytes : 0u);
    auto st = [&](int row) { return row >= 0 && row < 3 ? static_cast<uint32_t>(row) * Ch * 4u : kOut; };
    Raw<T, V> px[6];
    Raw<float, V> ps[3];
    Raw<TD, V> pg[3];
#pragma unroll
    for (int j = 0; j < 3; ++j) {
      px[j].load(xrow(t0 - 3 + j), xlane);
      ps[j].load(sb, st(t0 + j) + slane);  // position t0 - 3 + j where that is negative
    }
#pragma unroll
    for (int j = 0; j < 3; ++j) {
      px[3 + j].load(xrow(t0 + j), xlane);
      pg[j].load(grow(t0 + j), glane);
    }
    Raw<T, V> nx[kBlk];
    Raw<TD, V> ng[kBlk];
#pragma unroll
    for (int i = 0; i < kBlk; ++i) {
      nx[i].load(xrow(t0 + 3 + i), xlane);
      ng[i].load(grow(t0 + 3 + i), glane);
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
        const bool in = t0 + i < Tn;
        const float g = in ? grad(x, pg[i].at(v), v) : 0.0f;
        if (t0 == 0 && in) count(x, g, v);
        gw[i][v] = g;
        win[0][v] = win[1][v], win[1][v] = win[2][v], win[2][v] = x;
      }
    }
    if (t0 == 0 && dstate_in) {  // positions -3, -2, -1: the carried state's gradient
#pragma unroll
      for (int j = 0; j < 3; ++j) {
        Raw<float, V> e;
        e.load(eb, st(j - Tn) + slane);  // row p - (T - 3) of dstate_out, p = j - 3
        float o[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
          o[v] = e.at(v);
#pragma unroll
          for (int i = 0; i <= j; ++i) o[v] = fmaf(wt[v][j - i], gw[i][v], o[v]);
        }
        Raw<float, V>::store(make_buf(dstate_in + so, sbytes), st(j) + slane, o);
      }
    }
#pragma unroll 1
    for (int p0 = t0; p0 < min(t0 + run, Tn); p0 += kBlk) {
      Raw<T, V> cx[kBlk];
      Raw<TD, V> cg[kBlk];
#pragma unroll
      for (int i = 0; i < kBlk; ++i) cx[i] = nx[i], cg[i] = ng[i];
      if (p0 + kBlk < t0 + run) {
#pragma unroll
        for (int i = 0; i < kBlk; ++i) {
          nx[i].load(xrow(p0 + kBlk + 3 + i), xlane);
          ng[i].load(grow(p0 + kBlk + 3 + i), glane);
        }
      }
#pragma unroll
      for (int i = 0; i < kBlk; ++i) {
        const int p = p0 + i;
        const bool end = p + 3 >= Tn;  // past the sequence: g = 0, nothing counted
        float o[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const float x = cx[i].at(v);
          const float g = end ? 0.0f : grad(x, cg[i].at(v), v);
          if (!end) count(x, g, v);
          o[v] = fmaf(wt[v][3], gw[0][v], fmaf(wt[v][2], gw[1][v], fmaf(wt[v][1], gw[2][v], wt[v][0] * g)));
          gw[0][v] = gw[1][v], gw[1][v] = gw[2][v], gw[2][v] = g;
          win[0][v] = win[1][v], win[1][v] = win[2][v], win[2][v] = x;
        }
        if (end && dstate_out) {
          Raw<float, V> e;
          e.load(eb, st(p - (Tn - 3)) + slane);
#pragma unroll
          for (int v = 0; v < V; ++v) o[v] += e.at(v);
        }
        Raw<T, V>::store(orow(p), xlane, o);
      }
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
    float* __restrict__ dstate_in, float* __restrict__ part, int Bsz, int Tn, int HP, int GN, int run) {
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
                              HP, active, run, first, stride, dw, db);
  } else {
    const bool isC = bx >= nx + ng;
    const int cr = ((bx - nx - (isC ? ng : 0)) * kWave + lane) * kV;
    c = HP + (isC ? GN : 0) + cr;
    active = cr < GN;
    conv_bwd_body<T, float, SILU>(xbc, ld, w, bias, state_in, isC ? dC : dB, dstate_out, dxbc, lddx, dstate_in, Bsz,
                                  Tn, Ch, c, cr, GN, active, run, first, stride, dw, db);
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

// Run length and workgroups of a call.  A run of n tokens costs about n + 5 (its
// halo: three more gradients, six more rows), and the CU with the most
// workgroups ends last, so of the runs that give kMinWaves waves (four per SIMD)
// the one with the least ceil(workgroups / CUs) (n + 5); without enough waves
// the shortest.  The ranking counts a workgroup for every four runs, also past the
// kMaxParts per channel block that are launched (waves then walk several runs), so
// few channels with many tokens are ranked by a grid that is not quite theirs.
// Measured (both kernels): 2 x 2048 tokens of 4352 bf16 channels,
// 1258 workgroups of 28-token runs 28.1 us, 1088 of 32 30.0 (five on some CUs,
// 4.25 on average), 1768 of 20 29.1; 3 x 509 tokens of 1024 + 2 x 1024 float32
// channels, runs of 8 (4608 waves) 16.4, of 12 17.0, of 32 18.5.
constexpr long long kMinWaves = 4096;
constexpr int kRunMin = 8, kCUs = 256;
struct Plan {
  int run, blocks, parts;
};
Plan plan_of(int Bsz, int T, int HP, int GN) {
  Plan p;
  p.blocks = region_blocks(HP) + 2 * region_blocks(GN);
  p.run = kRunMin;
  long long best = -1, groups = 0;
  for (int run = kRunMin; run <= kRunMax; run += kBlk) {
    const long long units = static_cast<long long>(Bsz) * (T > 0 ? (T - 1) / run + 1 : 1);
    const long long wgs = (units + 3) / 4;
    const long long cost = (wgs * p.blocks + kCUs - 1) / kCUs * (run + 5);
    if (run == kRunMin || (units * p.blocks >= kMinWaves && cost < best)) {
      p.run = run;
      best = cost;
      groups = wgs;
    }
  }
  p.parts = static_cast<int>(groups < kMaxParts ? groups : kMaxParts);
  return p;
}

template <typename T>
void launch_conv_bwd(const ConvBwdArgs& a, hipStream_t st) {
  const Plan plan = plan_of(a.Bsz, a.T, a.HP, a.GN);
  const dim3 grid(plan.blocks, plan.parts);
  const T* xbc = static_cast<const T*>(a.xbc);
  const T* dx = static_cast<const T*>(a.dx);
  T* dxbc = static_cast<T*>(a.dxbc);
  float* part = static_cast<float*>(a.workspace);
  if (a.act)
    launch_k(true, ssd_conv1d_bwd_kernel<T, true>, grid, dim3(kThreads), st, nullptr, xbc, a.ld, a.w,
             a.bias, a.state_in, dx, a.dB, a.dC, a.dstate_out, dxbc, a.lddx, a.dstate_in, part, a.Bsz,
             a.T, a.HP, a.GN, plan.run);
  else
    launch_k(true, ssd_conv1d_bwd_kernel<T, false>, grid, dim3(kThreads), st, nullptr, xbc, a.ld, a.w,
             a.bias, a.state_in, dx, a.dB, a.dC, a.dstate_out, dxbc, a.lddx, a.dstate_in, part, a.Bsz,
             a.T, a.HP, a.GN, plan.run);
}

}  // namespace

// rows of the partial-sum table
int conv_bwd_parts(int Bsz, int T, int HP, int GN) { return plan_of(Bsz, T, HP, GN).parts; }

hipError_t run_conv1d_bwd(const ConvBwdArgs& a, hipStream_t st) {
  if (a.dtype == 1)
    launch_conv_bwd<uint16_t>(a, st);
  else
    launch_conv_bwd<float>(a, st);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int Ch = a.HP + 2 * a.GN;
  return sum_parts(static_cast<const float*>(a.workspace), conv_bwd_parts(a.Bsz, a.T, a.HP, a.GN), 5 * Ch, a.dw,
                   4 * Ch, a.dbias, st);
}

}  // namespace ssd
