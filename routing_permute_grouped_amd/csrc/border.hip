// The border of an expert block: combine, the norm after the block, its gate and scale, the
// residual sum and the norm before the next block, in one pass, and the backward of that pass.
//   u = sum_j w[t,j] y[dst[t,j]] + shared[t]        z = u rp gp, rp = 1/sqrt(mean u^2 + eps)
//   out = resid + scale gate[t] z                   x_next = out rn gn, rn likewise of out
// (z = u without gp). Backward, with f = scale gate[t], uh = u rp, oh = out rn:
//   G  = dout + rn (dx gn - oh mean(dx gn oh))      dresid = G
//   S  = sum_d G gp uh                              dgate = scale S
//   du = rp f (gp G - uh S / D)                     dgp = sum_t f G uh,  dgn = sum_t dx oh
//
// Bound by HBM: the forward reads k + 2 rows a token and writes two (three kept ones for a
// backward), the backward reads four and writes two. So a token's row is held in registers from
// its one read to its last use: VC values a lane, G waves a token (G the power of two that
// holds D), sums over a wave by lane exchange and over the G waves through LDS. Everything is
// float32 between the reads and the one rounding of each result; out is not rounded before the
// next norm.
//
// The gains' gradients are sums over all tokens. A workgroup keeps those of the tokens it takes
// in registers (a lane's columns stay the same) and writes one row of partial sums; a second
// kernel adds the rows. Fixed grids, so equal calls give equal bits.
#include <algorithm>

#include "border.hpp"
#include "common.hpp"
#include "kernels.hpp"
#include "wave.hpp"

namespace moe {
namespace {

constexpr int kParts = 256;      // most rows of partial sums
// Most workgroups of the forward; longer batches take several turns of each. One for every few tokens
// would pass the 2^32 threads of a launch from 2^26 tokens, of which the runtime then keeps the low 32
// bits. Far fewer are slower: each turn begins with its loads (65536 x 4096, top-4: 656 us, 64
// workgroups a CU 709; 262144 x 1024: 667 and 724).
constexpr int kMostGroups = 1 << 21;

typedef float f32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// Sum of v over the G waves of a token (of the one wave for G = 1), the same in every lane.
// `turn` alternates between the two halves of red, so one barrier a sum is enough: a half is
// written again only behind the next sum's barrier.
template <int WPB>
__device__ __forceinline__ float token_sum(float v, int G, int wave, float (*red)[WPB], int& turn) {
  v = wave_sum(v);
  if (G == 1) return v;
  if ((threadIdx.x & 63) == 0) red[turn][wave] = v;
  lds_barrier();
  const int first = wave & ~(G - 1);
  v = 0.0f;
  for (int i = 0; i < G; ++i) v += red[turn][first + i];
  turn ^= 1;
  return v;
}

// VC: values a lane holds; kJ: slots whose rows are read together.
template <typename TIn, int VC, int WPB, int kJ>
__global__ __launch_bounds__(WPB * 64) void border_kernel(const BorderCall a, int G) {
  constexpr int V = Chunk<TIn>::V, C = VC / V;
  __shared__ float red[2][WPB];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int gw = wave & (G - 1), tpb = WPB / G, nck = a.D / V;
  const float inv = 1.0f / (float)a.D;
  int turn = 0;
  int ck[C];
  bool in[C];
#pragma unroll
  for (int i = 0; i < C; ++i) {
    ck[i] = (i * G + gw) * 64 + lane;
    in[i] = ck[i] < nck;
  }
  // every wave makes the same number of turns, for the barriers
  for (int t0 = blockIdx.x * tpb; t0 < a.T; t0 += gridDim.x * tpb) {
    const bool there = t0 + wave / G < a.T;
    const int t = min(t0 + wave / G, a.T - 1);
    const size_t base = (size_t)t * a.D;
    u32x4 raw[C];
#pragma unroll
    for (int i = 0; i < C; ++i) {
      raw[i] = u32x4{0, 0, 0, 0};
      if (in[i]) raw[i] = ld16_nt(static_cast<const TIn*>(a.resid) + base + (size_t)ck[i] * V);
    }
    float o[VC];
    if (a.block) {
      float u[VC];
#pragma unroll
      for (int v = 0; v < VC; ++v) u[v] = 0.0f;
      if (a.y) {
        for (int j0 = 0; j0 < a.k; j0 += kJ) {
          u32x4 yv[kJ][C];
          int d[kJ];
          float w[kJ];
#pragma unroll
          for (int j = 0; j < kJ; ++j) {
            d[j] = -1;
            w[j] = 1.0f;
            if (j0 + j < a.k) {
              d[j] = a.dst[(size_t)t * a.k + j0 + j];
              if (a.w) w[j] = a.w[(size_t)t * a.k + j0 + j];
            }
            if (d[j] >= a.m_cap) d[j] = -1;
          }
#pragma unroll
          for (int j = 0; j < kJ; ++j)
            if (d[j] >= 0)
#pragma unroll
              for (int i = 0; i < C; ++i)
                if (in[i])
                  yv[j][i] = ld16_nt(static_cast<const TIn*>(a.y) + (size_t)d[j] * a.D + (size_t)ck[i] * V);
#pragma unroll
          for (int j = 0; j < kJ; ++j)
            if (d[j] >= 0)
#pragma unroll
              for (int i = 0; i < C; ++i)
                if (in[i]) {
                  float f[V];
                  Chunk<TIn>::widen(yv[j][i], f);
#pragma unroll
                  for (int v = 0; v < V; ++v) u[i * V + v] = __builtin_fmaf(w[j], f[v], u[i * V + v]);
                }
        }
      }
      if (a.shared) {
#pragma unroll
        for (int i = 0; i < C; ++i)
          if (in[i]) {
            float f[V];
            Chunk<TIn>::widen(ld16_nt(static_cast<const TIn*>(a.shared) + base + (size_t)ck[i] * V), f);
#pragma unroll
            for (int v = 0; v < V; ++v) u[i * V + v] += f[v];
          }
      }
      if (a.u && there) {
#pragma unroll
        for (int i = 0; i < C; ++i)
          if (in[i]) st16_nt(static_cast<TIn*>(a.u) + base + (size_t)ck[i] * V, Chunk<TIn>::narrow(u + i * V));
      }
      float f = a.scale;
      if (a.gate) f *= a.gate[t];
      if (a.gamma_post) {
        float s = 0.0f;
#pragma unroll
        for (int v = 0; v < VC; ++v) s = __builtin_fmaf(u[v], u[v], s);
        const float rp = 1.0f / sqrtf(token_sum<WPB>(s, G, wave, red, turn) * inv + a.eps);
        if (a.rstd_post && there && gw == 0 && lane == 0) a.rstd_post[t] = rp;
#pragma unroll
        for (int i = 0; i < C; ++i)
          if (in[i]) {
            float g[V];
            Chunk<TIn>::widen(ld16(static_cast<const TIn*>(a.gamma_post) + (size_t)ck[i] * V), g);
#pragma unroll
            for (int v = 0; v < V; ++v) u[i * V + v] *= rp * g[v];
          }
      }
#pragma unroll
      for (int i = 0; i < C; ++i) {
        Chunk<TIn>::widen(raw[i], o + i * V);
#pragma unroll
        for (int v = 0; v < V; ++v) o[i * V + v] = __builtin_fmaf(f, u[i * V + v], o[i * V + v]);
      }
      if (there) {
#pragma unroll
        for (int i = 0; i < C; ++i)
          if (in[i]) st16(static_cast<TIn*>(a.out) + base + (size_t)ck[i] * V, Chunk<TIn>::narrow(o + i * V));
      }
    } else {
#pragma unroll
      for (int i = 0; i < C; ++i) Chunk<TIn>::widen(raw[i], o + i * V);
    }
    if (!a.gamma_next) continue;
    float s = 0.0f;
#pragma unroll
    for (int v = 0; v < VC; ++v) s = __builtin_fmaf(o[v], o[v], s);
    const float rn = 1.0f / sqrtf(token_sum<WPB>(s, G, wave, red, turn) * inv + a.eps);
    if (!there) continue;
    if (a.rstd_next && gw == 0 && lane == 0) a.rstd_next[t] = rn;
#pragma unroll
    for (int i = 0; i < C; ++i)
      if (in[i]) {
        float g[V];
        Chunk<TIn>::widen(ld16(static_cast<const TIn*>(a.gamma_next) + (size_t)ck[i] * V), g);
#pragma unroll
        for (int v = 0; v < V; ++v) g[v] *= o[i * V + v] * rn;
        st16(static_cast<TIn*>(a.x_next) + base + (size_t)ck[i] * V, Chunk<TIn>::narrow(g));
      }
  }
}

// AHEAD: the next token's rows are loaded while this one's sums are taken.
template <typename TIn, int VC, int WPB, bool AHEAD>
__global__ __launch_bounds__(WPB * 64) void border_bwd_kernel(const BorderBwdCall a, int G) {
  constexpr int V = Chunk<TIn>::V, C = VC / V;
  __shared__ float red[2][WPB];
  __shared__ f32x4 sums[WPB * 64 * VC / 4];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int gw = wave & (G - 1), tpb = WPB / G, nck = a.D / V;
  const float inv = 1.0f / (float)a.D;
  const bool next = a.dx_next, post = a.gamma_post, dot = post || a.dgate;
  int turn = 0;
  int ck[C];
  bool in[C];
  float accp[VC], accn[VC];
  u32x4 gainp[C], gainn[C];   // the lane's columns stay the same, and so do their gains
#pragma unroll
  for (int i = 0; i < C; ++i) {
    ck[i] = (i * G + gw) * 64 + lane;
    in[i] = ck[i] < nck;
    gainp[i] = gainn[i] = u32x4{0, 0, 0, 0};
    if (in[i] && post) gainp[i] = ld16(static_cast<const TIn*>(a.gamma_post) + (size_t)ck[i] * V);
    if (in[i] && next) gainn[i] = ld16(static_cast<const TIn*>(a.gamma_next) + (size_t)ck[i] * V);
  }
#pragma unroll
  for (int v = 0; v < VC; ++v) accp[v] = accn[v] = 0.0f;

  struct Raw {
    u32x4 g[C], x[C], o[C], u[C];
    float rn, rp, gate;
  };
  auto read = [&](const void* p, size_t base, u32x4 (&raw)[C]) {
#pragma unroll
    for (int i = 0; i < C; ++i) {
      raw[i] = u32x4{0, 0, 0, 0};
      if (p && in[i]) raw[i] = ld16_nt(static_cast<const TIn*>(p) + base + (size_t)ck[i] * V);
    }
  };
  auto load = [&](Raw& r, int t0) {
    const int t = min(t0 + wave / G, a.T - 1);
    const size_t base = (size_t)t * a.D;
    read(a.dout, base, r.g);
    read(a.dx_next, base, r.x);
    read(next ? a.out : nullptr, base, r.o);
    read(dot ? a.u : nullptr, base, r.u);
    r.rn = next ? a.rstd_next[t] : 0.0f;
    r.rp = post ? a.rstd_post[t] : 1.0f;
    r.gate = a.block && a.gate ? a.gate[t] : 1.0f;
  };
  auto token = [&](const Raw& r, int t0) {
    const bool there = t0 + wave / G < a.T;
    const int t = min(t0 + wave / G, a.T - 1);
    const size_t base = (size_t)t * a.D;
    float g[VC];
#pragma unroll
    for (int i = 0; i < C; ++i) Chunk<TIn>::widen(r.g[i], g + i * V);
    if (next) {
      float s = 0.0f;
#pragma unroll
      for (int i = 0; i < C; ++i) {
        float x[V], o[V], gn[V];
        Chunk<TIn>::widen(r.x[i], x);
        Chunk<TIn>::widen(r.o[i], o);
        Chunk<TIn>::widen(gainn[i], gn);
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const float oh = o[v] * r.rn;
          s = __builtin_fmaf(x[v] * gn[v], oh, s);
          if (there) accn[i * V + v] = __builtin_fmaf(x[v], oh, accn[i * V + v]);
        }
      }
      const float m = token_sum<WPB>(s, G, wave, red, turn) * inv;
#pragma unroll
      for (int i = 0; i < C; ++i) {
        float x[V], o[V], gn[V];
        Chunk<TIn>::widen(r.x[i], x);
        Chunk<TIn>::widen(r.o[i], o);
        Chunk<TIn>::widen(gainn[i], gn);
#pragma unroll
        for (int v = 0; v < V; ++v)
          g[i * V + v] = __builtin_fmaf(r.rn, x[v] * gn[v] - o[v] * r.rn * m, g[i * V + v]);
      }
    }
    if (there) {
#pragma unroll
      for (int i = 0; i < C; ++i)
        if (in[i]) st16(static_cast<TIn*>(a.dresid) + base + (size_t)ck[i] * V, Chunk<TIn>::narrow(g + i * V));
    }
    if (!a.block) return;
    const float f = a.scale * r.gate;
    if (dot) {
      float s = 0.0f;
#pragma unroll
      for (int i = 0; i < C; ++i) {
        float u[V], gp[V];
        Chunk<TIn>::widen(r.u[i], u);
        Chunk<TIn>::widen(gainp[i], gp);
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const float uh = u[v] * r.rp;
          s = __builtin_fmaf(post ? g[i * V + v] * gp[v] : g[i * V + v], uh, s);
          if (there) accp[i * V + v] = __builtin_fmaf(f * g[i * V + v], uh, accp[i * V + v]);
        }
      }
      s = token_sum<WPB>(s, G, wave, red, turn);
      if (a.dgate && there && gw == 0 && lane == 0) a.dgate[t] = a.scale * s;
      if (post) {
        const float m = s * inv;
#pragma unroll
        for (int i = 0; i < C; ++i) {
          float u[V], gp[V];
          Chunk<TIn>::widen(r.u[i], u);
          Chunk<TIn>::widen(gainp[i], gp);
#pragma unroll
          for (int v = 0; v < V; ++v)
            g[i * V + v] = r.rp * (g[i * V + v] * gp[v] - u[v] * r.rp * m);
        }
      }
    }
    if (there) {
#pragma unroll
      for (int v = 0; v < VC; ++v) g[v] *= f;
#pragma unroll
      for (int i = 0; i < C; ++i)
        if (in[i]) st16(static_cast<TIn*>(a.du) + base + (size_t)ck[i] * V, Chunk<TIn>::narrow(g + i * V));
    }
  };
  // every wave makes the same number of turns, for the barriers
  const int step = gridDim.x * tpb;
  if constexpr (AHEAD) {   // past the end the last token is read again
    Raw raw[2];
    load(raw[0], blockIdx.x * tpb);
    for (int t0 = blockIdx.x * tpb; t0 < a.T; t0 += 2 * step) {
      load(raw[1], t0 + step);
      token(raw[0], t0);
      if (t0 + step >= a.T) break;
      load(raw[0], t0 + 2 * step);
      token(raw[1], t0 + step);
    }
  } else {
    for (int t0 = blockIdx.x * tpb; t0 < a.T; t0 += step) {
      Raw raw;
      load(raw, t0);
      token(raw, t0);
    }
  }
  // the workgroup's sums over its token groups, in group order, to its row of the partial sums
  auto put = [&](const float (&acc)[VC], float* rows) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < VC / 4; ++i)
      sums[(i * WPB + wave) * 64 + lane] = f32x4{acc[4 * i], acc[4 * i + 1], acc[4 * i + 2], acc[4 * i + 3]};
    __syncthreads();
    // column quad c of wave position w: chunk (i * G + w) * 64 + l, quad i * V/4 + j of a lane
    for (int c = threadIdx.x; c < a.D / 4; c += WPB * 64) {
      const int chunk = c / (V / 4), j = c % (V / 4);
      const int l = chunk & 63, w = (chunk >> 6) & (G - 1), i = (chunk >> 6) / G;
      f32x4 s = {0.0f, 0.0f, 0.0f, 0.0f};
      for (int q = 0; q < tpb; ++q) s += sums[((i * (V / 4) + j) * WPB + q * G + w) * 64 + l];
      *reinterpret_cast<f32x4*>(rows + (size_t)blockIdx.x * a.D + 4 * c) = s;
    }
  };
  if (a.dgamma_next) put(accn, a.partial);
  if (a.dgamma_post) put(accp, a.partial + (size_t)gridDim.x * a.D);
}

// out[d] = sum of rows[0..n)[d]: 64 columns a workgroup, each of its 16 waves every 16th row,
// the waves' sums in wave order.
__global__ __launch_bounds__(1024) void column_sums_kernel(const float* __restrict__ partial, int n,
                                                           int D, float* __restrict__ out0,
                                                           float* __restrict__ out1) {
  __shared__ float red[16][64];
  float* out = blockIdx.y ? out1 : out0;
  if (!out) return;
  const float* rows = partial + (size_t)blockIdx.y * n * D;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int d = blockIdx.x * 64 + lane;
  float s = 0.0f;
#pragma unroll 8
  for (int r = wave; r < n; r += 16) s += rows[(size_t)r * D + d];
  red[wave][lane] = s;
  __syncthreads();
  if (wave == 0) {
    s = 0.0f;
#pragma unroll
    for (int w = 0; w < 16; ++w) s += red[w][lane];
    out[d] = s;
  }
}

int waves_for(int D, int VC) {
  int g = 1;
  while (g * 64 * VC < D) g *= 2;
  return g;
}

// rows of partial sums: one a workgroup, of at most 16 waves' tokens
int parts_of(int T) { return std::min(kParts, T); }

template <typename TIn, int VC, int WPB, bool AHEAD>
int launch_bwd(const BorderBwdCall& c, hipStream_t s) {
  const int G = waves_for(c.D, VC), tpb = WPB / G;
  const int n = std::min(kParts, (c.T + tpb - 1) / tpb);
  hipLaunchKernelGGL((border_bwd_kernel<TIn, VC, WPB, AHEAD>), dim3(n), dim3(WPB * 64), 0, s, c, G);
  return n;
}

template <typename TIn, int VC, int WPB, int kJ>
void launch_vc(const BorderCall& c, hipStream_t s) {
  const int G = waves_for(c.D, VC), tpb = WPB / G;
  const int n = std::min(kMostGroups, (c.T + tpb - 1) / tpb);
  hipLaunchKernelGGL((border_kernel<TIn, VC, WPB, kJ>), dim3(n), dim3(WPB * 64), 0, s, c, G);
}

template <typename TIn>
void launch_typed(const BorderCall& c, hipStream_t s) {
  // Few tokens are a chain of latencies: more waves a token, more rows on the way (4 tokens, top-6,
  // D = 2048: 5.2 against 6.3 us). Many fill the card: two rows at a time leave the most waves (8192
  // tokens 70.7 us, four 73.2, one 71.8).
  const bool few = c.T <= cu_count();
  if (few && waves_for(c.D, 8) <= 4)
    launch_vc<TIn, 8, 4, 8>(c, s);
  else if (few && waves_for(c.D, 8) <= 16)
    launch_vc<TIn, 8, 16, 8>(c, s);
  else if (waves_for(c.D, 16) <= 4)
    launch_vc<TIn, 16, 4, 2>(c, s);
  else
    launch_vc<TIn, 16, 16, 2>(c, s);
}

}  // namespace

hipError_t launch_border(int dt, const BorderCall& c, hipStream_t s) {
  if (dt == kF32)
    launch_typed<float>(c, s);
  else
    launch_typed<bf16_t>(c, s);
  return hipGetLastError();
}

size_t border_workspace_bytes(int T, int D) { return (size_t)2 * parts_of(T) * D * sizeof(float); }

hipError_t launch_border_backward(int dt, const BorderBwdCall& c, hipStream_t s) {
  // bf16: 8 waves of 16 values a lane, from D = 4096 16 waves of 8, which keep more loads on the way
  // (16384 tokens, us: D = 1024 40.4 against 43.9, 2048 75 both, 2880 108.7 against 104.2, 4096 137.3
  // against 134.7, 5120 204.6 against 202.6; 8192 x 7168 126.3 against 129.4). float32: 8 waves of 8 values.
  // Wider rows take 16 waves of 16 values, at most 128 registers each, without loads ahead: bf16 past D =
  // 8192 spills 52 registers (8192 x 16384: 526 us, 3.1 TB/s), float32 past 4096 87 (8192 x 7168: 375 us, 3.8
  // TB/s; 8192 x 4096, which does not, 133 us, 6.1).
  int n;
  if (dt == kF32)
    n = c.D <= 4096 ? launch_bwd<float, 8, 8, true>(c, s) : launch_bwd<float, 16, 16, false>(c, s);
  else if (c.D < 4096)
    n = launch_bwd<bf16_t, 16, 8, true>(c, s);
  else
    n = c.D <= 8192 ? launch_bwd<bf16_t, 8, 16, true>(c, s) : launch_bwd<bf16_t, 16, 16, false>(c, s);
  if (c.dgamma_next || c.dgamma_post)
    hipLaunchKernelGGL(column_sums_kernel, dim3(c.D / 64, c.dgamma_post ? 2 : 1), dim3(1024), 0, s,
                       c.partial, n, c.D, c.dgamma_next, c.dgamma_post);
  return hipGetLastError();
}

}  // namespace moe
