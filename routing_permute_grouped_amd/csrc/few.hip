// The whole expert layer for a few tokens (at most 32) in three kernels: the router's logits, then
// top-k + fc1, then fc2 + combine. Per token t and slot j with expert e = topk_idx[t,j]:
//   h[t,j] = silu(x[t] w1[e]^T) * (x[t] w3[e]^T), rounded to the layer type,
//   out[t] = sum_j topk_w[t,j] * (h[t,j] w2[e]^T) + hs[t] ws2^T  (hs: the shared experts' h),
// all sums in float32, out rounded once. h is rounded because it is the matrix instruction's
// operand in fc2 and the layer's storage point everywhere else; y is not rounded here.
//
// Bound by one read of the active experts' weights. With so few tokens no row is moved: the
// weights are the matrix instruction's first operand (16 output columns of the layer), tokens its
// second (16 columns). Up to as many tokens as an instruction takes, its columns are the tokens
// themselves, an expert's product is taken for all of them and kept for those that chose it; more
// tokens than that are taken expert by expert, each one's own tokens in the columns, 16 (or in fc2
// RC) at a time, and only an expert with more of them has its weights read again (from the L2: its
// groups run side by side). An expert with such a group of tokens is a segment below.
//   * few_logits: over the whole card; every workgroup of few_fc1 chooses from them for itself.
//   * few_fc1: an item is 16 rows of w1 and of w3 of one active expert (or of the shared
//     experts). KS waves of a workgroup's 16 share an item's k, KS chosen on the device so that
//     the items fill whole rounds of the card; their sums meet in LDS in wave order. The tokens'
//     rows lie in LDS where they fit (from the L2 they cost 14% of the stream at 16 tokens).
//   * few_fc2: a workgroup owns RC output columns and reads their w2 rows of every active
//     expert; its waves take equal shares of all those k, and their sums meet in LDS in wave
//     order, so there are no atomics and equal calls give equal bits. The rows of h lie in LDS
//     where they fit; the first weights are on the way before they are.
// A lane loads 16 bytes of a weight row at a time, PF units ahead. Tokens past T read as zeros
// through the buffer descriptor's range, or as another token's row, and are not stored.
#include <algorithm>
#include <type_traits>

#include "common.hpp"
#include "few.hpp"
#include "kernels.hpp"
#include "route_core.hpp"

namespace moe {
namespace {

constexpr int WAVES = 16;
constexpr int THREADS = WAVES * 64;
constexpr int MAXT = kFewTokens;
constexpr int MAXSLOTS = MAXT * kMaxTopK;
constexpr int MAXE = 1024;
constexpr uint32_t PAST = 0x7ffffff0u;   // a lane offset past every buffer here
// LDS: 160 KiB less the slots' tables (indices, weights, tokens of an expert, segments)
constexpr int TABLES = MAXSLOTS * 8 + MAXE * 4 + MAXSLOTS * 2 + 64;
constexpr int POOL = (160 * 1024 - TABLES) / 256 * 256;
constexpr int RED = WAVES * 2 * 64 * 16;   // fc1: a slot of sums a wave

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2v __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// This wave's LDS accesses are complete, then every wave of the workgroup meets; loads in
// flight keep flying.
__device__ __forceinline__ void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// a / b for 0 <= a < 2^24, 0 < b with a quotient under 2^22 (the reciprocal is then off by less than
// one): a few instructions where the compiler's division takes some hundred clocks (five plans of
// an item's share with it: 2.5 us).
__device__ __forceinline__ int quot(int a, int b) {
  int q = (int)((float)a * __builtin_amdgcn_rcpf((float)b));
  const int r = a - q * b;
  if (r < 0) --q;
  if (r >= b) ++q;
  return q;
}
// The same of values that the whole wave shares, in scalar registers.
__device__ __forceinline__ int quot_wave(int a, int b) { return __builtin_amdgcn_readfirstlane(quot(a, b)); }

// Weight formats. A unit is what a wave multiplies at a time: UK values of k, of which lane
// group g = lane / 16 holds the 16-byte pieces that the NF instructions take; x's pieces lie
// at the same k, XL bytes apart from group to group and XF from instruction to instruction.
template <int W> struct Fmt;
template <> struct Fmt<kFewF32> {
  typedef float Act;
  static constexpr int UK = 32, NF = 2, NV = 2, WB = 128, XB = 128, XL = 16, XF = 64;
};
template <> struct Fmt<kFewBf16> {
  typedef bf16_t Act;
  static constexpr int UK = 64, NF = 2, NV = 2, WB = 128, XB = 128, XL = 16, XF = 64;
};
// 4-bit: a lane's 16 bytes are one block of 32 codes with its scale
template <> struct Fmt<kFewMx4> {
  typedef bf16_t Act;
  static constexpr int UK = 128, NF = 4, NV = 1, WB = 64, XB = 256, XL = 64, XF = 16;
};

// float32: the instructions' sum is one chain of products; every CHAIN units it is added to a sum beside it and
// begun again, so that a sum over k is a chain of 256 products and one of those sums in place of up to
// 65536 products (8 tokens, D = 4544: out off by 4.7e-7 of its size, 1.9e-6 in one chain). Every unit apart
// costs the wait for its products (32 tokens over 8 experts of 4096 x 2048: 218 us, every 8 187, one chain 191).
// In bf16 the roundings of h and out are some thousand times what that saves.
constexpr int CHAIN = 8;
template <int W>
__device__ __forceinline__ bool chain_ends(int step) {
  return W == kFewF32 && step % CHAIN == CHAIN - 1;
}

template <int W> struct WReg {
  u32x4 v[Fmt<W>::NV];
  uint32_t s;
};

// One matrix [E, N, K]: the lane's row of expert e, and its scale bytes (4-bit).
struct Rows {
  const uint8_t* row;
  const uint8_t* scale;
};

template <int W>
__device__ __forceinline__ Rows rows_at(const void* q, const void* s, int e, int N, int K, int n,
                                        int g) {
  const size_t r = (size_t)e * N + n;
  Rows o;
  o.row = static_cast<const uint8_t*>(q) + r * ((size_t)K / Fmt<W>::UK * Fmt<W>::WB) + 16 * g;
  o.scale = W == kFewMx4 ? static_cast<const uint8_t*>(s) + r * 4 + g : nullptr;
  return o;
}

template <int W>
__device__ __forceinline__ void load_unit(WReg<W>& w, const Rows& m, size_t sstep, int u) {
#pragma unroll
  for (int i = 0; i < Fmt<W>::NV; ++i) w.v[i] = ld16(m.row + (size_t)u * Fmt<W>::WB + 64 * i);
  if (W == kFewMx4) w.s = m.scale[(size_t)u * sstep];
}

// Instruction f of a unit: acc += rows x columns.
template <int W>
__device__ __forceinline__ void mul(const WReg<W>& w, const u32x4& x, int f, f32x4& acc) {
  if constexpr (W == kFewF32) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      acc = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(w.v[f][i]), __uint_as_float(x[i]),
                                                 acc, 0, 0, 0);
  } else {
    bf16x8 wf;
    if constexpr (W == kFewBf16) {
      wf = __builtin_bit_cast(bf16x8, w.v[f]);
    } else {   // eight codes and the block's scale: exact in bf16
      const float scale = __uint_as_float(w.s << 23);
      const uint32_t c = w.v[0][f];
      const bf16x2v p = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 0);
      const bf16x2v q = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 1);
      const bf16x2v r = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 2);
      const bf16x2v t = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 3);
      wf = bf16x8{p[0], p[1], q[0], q[1], r[0], r[1], t[0], t[1]};
    }
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf, __builtin_bit_cast(bf16x8, x), acc, 0, 0, 0);
  }
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t act_rsrc(const void* p, size_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, (int)bytes, 0x00020000);
}

template <int W, int XF = Fmt<W>::XF>
__device__ __forceinline__ void load_x(u32x4 (&x)[Fmt<W>::NF], __amdgpu_buffer_rsrc_t rs,
                                       uint32_t off, int more) {
#pragma unroll
  for (int f = 0; f < Fmt<W>::NF; ++f)
    x[f] = __builtin_amdgcn_raw_buffer_load_b128(rs, (int)off, more + f * XF, 0);
}

// Rows in LDS: 16-byte piece c of row r, of `bytes` bytes (a multiple of 128), at c ^ key, key
// the row's token modulo 8, so that eight tokens' pieces of one c fall on distinct banks.
__device__ __forceinline__ void fill_rows(char* lds, const void* src, int rows, int bytes, int per) {
  const int n = bytes / 16;
  for (int i = threadIdx.x; i < rows * n; i += THREADS) {
    const int r = quot(i, n), c = i - r * n;
    st16(lds + (size_t)r * bytes + ((c ^ (quot(r, per) & 7)) << 4), ld16(static_cast<const char*>(src) + (size_t)i * 16));
  }
}
// The lane's pieces of unit u: `row` its row's LDS address, t its token.
template <int W, int XL = Fmt<W>::XL, int XF = Fmt<W>::XF>
__device__ __forceinline__ u32x4 lds_piece(const char* row, int t, int g, int u, int f) {
  const int low = g * (XL / 16) + f * (XF / 16);
  return ld16(row + u * Fmt<W>::XB + ((low ^ (t & 7)) << 4));
}

// A workgroup's tables: the slots' indices and weights, the tokens of every expert as bits (only
// where there are more tokens than columns), and the segments: an expert, and in the bits above
// the group of its tokens that the columns hold.
struct Tables {
  int idx[MAXSLOTS];
  float w[MAXSLOTS];
  uint32_t tokens[MAXE];
  int16_t seg[MAXSLOTS];
  int sums[WAVES];
};
static_assert(sizeof(Tables) == TABLES, "the pool is what the tables leave");
constexpr int SEGE = 1024;   // a segment is expert + SEGE * group

// The segments for `cols` columns, from the slots in LDS (an index outside [0, E) is no expert).
// Returns their number. At most 64 slots of at most `cols` tokens: every wave for itself without a
// barrier, `mine` the lane's slot's index (all waves write the same list, in the slots' order).
// Else in the experts' order, behind barriers.
__device__ __forceinline__ int segments(Tables& tb, int mine, int T, int k, int E, int cols) {
  const int tid = threadIdx.x, lane = tid & 63, slots = T * k;
  if (slots <= 64 && T <= cols) {
    bool first = lane < slots && mine >= 0 && mine < E;
    for (int s = 0; s + 1 < slots; ++s)
      if (lane > s && __builtin_amdgcn_readlane(mine, s) == mine) first = false;
    const uint64_t m = __ballot(first);
    if (first) tb.seg[__popcll(m & ((1ull << lane) - 1))] = (int16_t)mine;
    return __popcll(m);
  }
  if (tid < E) tb.tokens[tid] = 0;
  __syncthreads();
  for (int i = tid; i < slots; i += THREADS) {
    const int e = tb.idx[i];
    if (e >= 0 && e < E) atomicOr(&tb.tokens[e], 1u << quot(i, k));
  }
  __syncthreads();
  const int n = tid < E ? (__popc(tb.tokens[tid]) + cols - 1) / cols : 0;
  int inc = n;   // prefix sums over the wave, then over the waves
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(inc, d);
    if (lane >= d) inc += o;
  }
  if (lane == 63) tb.sums[tid >> 6] = inc;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < WAVES; ++w) {
    const int s = tb.sums[w];
    all += s;
    if (w < tid >> 6) before += s;
  }
  for (int g = 0; g < n; ++g) tb.seg[before + inc - n + g] = (int16_t)(tid + SEGE * g);
  __syncthreads();
  return all;
}

// The n-th set bit of m (n below their number).
__device__ __forceinline__ int nth_bit(uint32_t m, int n) {
  int at = 0;
#pragma unroll
  for (int s = 16; s >= 1; s >>= 1) {
    const int c = __popc(m >> at & ((1u << s) - 1));
    if (n >= c) {
      n -= c;
      at += s;
    }
  }
  return at;
}

// The token in column c of a segment, -1 for none; of a group of the shared experts' (shared).
__device__ __forceinline__ int column_token(const Tables& tb, int seg, bool shared, int group, int c,
                                            int T, int cols) {
  if (shared || T <= cols) {
    const int t = (shared ? group * cols : 0) + c;
    return t < T ? t : -1;
  }
  const uint32_t m = tb.tokens[seg % SEGE];
  const int n = seg / SEGE * cols + c;
  return n < __popc(m) ? nth_bit(m, n) : -1;
}

// Where h's value n of a row lies (n a multiple of 4), and h's piece distances. For 4-bit weights the
// lanes of an instruction take every fourth 16-byte piece of a unit's 256 bytes, so those lie side by
// side (16 tokens over 8 experts of F = 14336: the call 187 us, with h in order 194).
constexpr int H_LANE = 16, H_NEXT = 64;   // bytes from group to group, instruction to instruction
template <int W>
__device__ __forceinline__ int h_at(int n) {
  return W == kFewMx4 ? (n & ~127) + (n >> 3 & 3) * 32 + (n >> 5 & 3) * 8 + (n & 7) : n;
}

template <typename Act>
__device__ __forceinline__ void store4(Act* p, const f32x4& v) {
  if constexpr (sizeof(Act) == 2)
    *reinterpret_cast<uint2*>(p) = uint2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
  else
    *reinterpret_cast<f32x4*>(p) = v;
}

// silu(a) * b. bf16: the hardware's approximate reciprocal, about 1 ulp of float32, below the
// rounding of h; float32: the exact quotient.
template <typename Act>
__device__ __forceinline__ float silu_mul(float a, float b) {
  if constexpr (sizeof(Act) == 2) return a * __builtin_amdgcn_rcpf(1.0f + __expf(-a)) * b;
  return a / (1.0f + expf(-a)) * b;
}

// The logits [T][E], bit for bit what the routing kernel gives: NT tokens with one expert a wave,
// STEPS chunk steps in flight, four experts a workgroup. A chain of loads bounds it, so it is a
// launch over the whole card: by every workgroup of the first kernel itself one token over 64
// experts of D = 2048 took as long in all (41.7 us), two 4 us more and 16 over 64 of D = 128 8 us
// more (4 over 4 of D = 128, where the launch is all there is, 3 us less).
constexpr int LOGIT_WAVES = 4;
template <typename TIn, int NT>
__global__ __launch_bounds__(64 * LOGIT_WAVES) void few_logits(
    const TIn* __restrict__ x, const TIn* __restrict__ wg, const float* __restrict__ bias, int T, int D,
    int E, float* __restrict__ logits) {
  constexpr int V = Chunk<TIn>::V, STEPS = NT == 1 ? 8 : 4, LANES = 64 / NT;
  const int lane = threadIdx.x & 63;
  const int e = blockIdx.x * LOGIT_WAVES + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int t0 = blockIdx.y * NT;
  if (e >= E) return;
  const TIn* wr = wg + (size_t)e * D;
  const int nchunk = D / V;
  float acc[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) acc[t] = 0.0f;
  for (int c0 = lane; c0 < nchunk; c0 += 64 * STEPS) {
    u32x4 xc[STEPS][NT], wc[STEPS];
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      const int c = min(c0 + 64 * s, nchunk - 1);
      wc[s] = ld16(wr + (size_t)c * V);
#pragma unroll
      for (int t = 0; t < NT; ++t) xc[s][t] = ld16(x + (size_t)min(t0 + t, T - 1) * D + (size_t)c * V);
    }
#pragma unroll
    for (int s = 0; s < STEPS; ++s)
      if (c0 + 64 * s < nchunk) {
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
          for (int t = 0; t < NT; ++t) dot_step(acc[t], elem<TIn>(xc[s][t], i), elem<TIn>(wc[s], i), TIn());
      }
  }
  const float v = reduce_pairs<NT, 32>(acc, lane);
  const int t = t0 + lane / LANES;
  if (lane % LANES == 0 && t < T) logits[t * E + e] = bias ? v + bias[e] : v;
}

struct FewArgs {
  const void *x, *wg;
  const float* bias;
  int T, D, F, E, k, renorm, Fs;
  const void *w1, *w3, *w2, *s1, *s3, *s2;   // s: scales of 4-bit weights
  const void *ws1, *ws3, *ws2;               // shared experts [Fs, D], [D, Fs]
  int32_t* topk_idx;
  float* topk_w;
  void *h, *hs, *out;                        // h [T*k, F], hs [T, Fs]
  uint32_t hs_off;                           // bytes of h: hs lies behind it
  float* logits;                             // [T, E], of the call that routes
  int most_ks;                               // waves that may share an item of fc1, as a power of two
};

// Waves that share an item, as a power of two: the fewest units of k in a chain over all rounds,
// counting what a round costs beside them (its first loads and the meeting) as 4 units. items over
// `grid` workgroups of 2^waves waves each. (The rounds may be off by one here, which is no harm.)
__device__ __forceinline__ int share_of(int items, int grid, int waves, int units, int most) {
  const float per = (float)items * __builtin_amdgcn_rcpf((float)(grid << waves));
  float cost = INFINITY;
  int best = 0;
#pragma unroll
  for (int i = 0; i <= 4; ++i) {
    const float c = ceilf(per * (float)(1 << i)) * (float)(((units + (1 << i) - 1) >> i) + 4);
    if (i <= most && c < cost) {
      cost = c;
      best = i;
    }
  }
  return __builtin_amdgcn_readfirstlane(best);
}

// Steps 0 .. n-1 with the loads PF steps ahead. Within the loop every load is made, so that the
// waits count exactly; the last ones are made only where a step takes them. FIRST: the first PF
// loads too, else the caller has made them.
template <int PF, bool FIRST = true, typename Load, typename Compute>
__device__ __forceinline__ void ring(int n, Load load, Compute compute) {
  if constexpr (FIRST) {
#pragma unroll
    for (int j = 0; j < PF; ++j)
      if (j < n) load(j, j);
  }
  int s = 0;
  for (; s + 2 * PF <= n; s += PF) {
#pragma unroll
    for (int j = 0; j < PF; ++j) {
      compute(j, s + j);
      load(j, s + j + PF);
    }
  }
#pragma unroll
  for (int j = 0; j < PF; ++j) {
    if (s + j < n) compute(j, s + j);
    if (s + j + PF < n) load(j, s + j + PF);
  }
  s += PF;
#pragma unroll
  for (int j = 0; j < PF; ++j)
    if (s + j < n) compute(j, s + j);
}

// A wave's part of one item of fc1: rows n .. n+15 of w1 and of w3 times the tokens, over units
// kw, kw + KS, ... t: the lane's column's token (-1: none). The tokens' rows come from LDS (xl) or
// from memory (XL false).
template <int W, int PF, bool XL>
__device__ __forceinline__ void fc1_item(const Rows& m1, const Rows& m3, size_t sstep, const void* x,
                                         const char* xl, int T, int t, int xrow, int units, int kw,
                                         int KS, f32x4 (&acc)[2]) {
  constexpr int NF = Fmt<W>::NF;
  if (kw >= units) return;
  const int n = quot_wave(units - kw + KS - 1, KS);
  const int g = (threadIdx.x & 63) >> 4;
  const __amdgpu_buffer_rsrc_t xrs = act_rsrc(x, (size_t)T * xrow);
  WReg<W> wr[PF][2];
  u32x4 xr[XL ? 1 : PF][NF];
  const int tl = max(t, 0);   // a column without a token takes another row; nothing of it is kept
  const uint32_t off = t >= 0 ? t * (uint32_t)xrow + g * Fmt<W>::XL : PAST;
  const char* row = XL ? xl + tl * xrow : nullptr;
  f32x4 sum[2] = {};   // of the chains that have ended
  auto load = [&](int j, int s) {
    const int u = kw + s * KS;
    load_unit<W>(wr[j][0], m1, sstep, u);
    load_unit<W>(wr[j][1], m3, sstep, u);
    if constexpr (!XL) load_x<W>(xr[j], xrs, off, u * Fmt<W>::XB);
  };
  auto compute = [&](int j, int s) {
    if constexpr (XL) {
#pragma unroll
      for (int f = 0; f < NF; ++f) xr[0][f] = lds_piece<W>(row, tl, g, kw + s * KS, f);
    }
#pragma unroll
    for (int f = 0; f < NF; ++f) {
      mul<W>(wr[j][0], xr[XL ? 0 : j][f], f, acc[0]);
      mul<W>(wr[j][1], xr[XL ? 0 : j][f], f, acc[1]);
    }
    if (chain_ends<W>(s)) {
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        sum[m] += acc[m];
        acc[m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      }
    }
  };
  ring<PF>(n, load, compute);
  if constexpr (W == kFewF32) {
    acc[0] += sum[0];
    acc[1] += sum[1];
  }
}

// W: the routed weights' format, S: the shared experts'. NE: 0 with routing given, else the
// logits a lane holds in the choice made here. XL: the tokens' rows in LDS.
template <int W, int S, int NE, bool XL>
__global__ __launch_bounds__(THREADS) void few_fc1(const FewArgs a) {
  typedef typename Fmt<W>::Act Act;
  // units in flight: more of them were slower (bf16, 16 tokens over 8 experts: 2 341 us, 4 349; one
  // token, 4 bits: 2 20.6, 4 25.6, where registers spill). With the rows from the L2 a third one
  // hides their way, but for 4 bits, where it spills (32 tokens over 64 experts of 4096: the call
  // 84 us, with 2 71)
  constexpr int PW = XL || W == kFewMx4 ? 2 : 3, PS = 2;
  __shared__ Tables tb;
  // the waves' sums, then the rows (which take the sums' place where no two waves share an item)
  __shared__ __attribute__((aligned(256))) char pool[XL ? POOL : RED];
  f32x4* red = reinterpret_cast<f32x4*>(pool);
  char* xl = pool + (a.most_ks > 0 ? RED : 0);
  const int lane = threadIdx.x & 63, fr = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int slots = a.T * a.k;
  const int xrow = a.D * (int)sizeof(Act);
  f32x4 acc[2];

  if constexpr (XL) fill_rows(xl, a.x, a.T, xrow, 1);
  if constexpr (NE > 0) {
    for (int t = wave; t < a.T; t += WAVES)
      route_token<(NE > 0 ? NE : 1)>(a.logits + t * a.E, t, a.E, a.k, a.renorm, tb.idx, tb.w, nullptr, lane);
    __syncthreads();
    if (blockIdx.x == 0)
      for (int i = threadIdx.x; i < slots; i += THREADS) {
        a.topk_idx[i] = tb.idx[i];
        a.topk_w[i] = tb.w[i];
      }
  } else {
    for (int i = threadIdx.x; i < slots; i += THREADS) tb.idx[i] = a.topk_idx[i];
    __syncthreads();
  }
  const int nseg = segments(tb, lane < slots ? tb.idx[lane] : -1, a.T, a.k, a.E, 16);

  // The items: of the shared experts, then of the segments. Where their formats differ (and so
  // their units) each kind has half of the waves.
  const int cols = a.F / 16, scols = a.Fs / 16;
  const int shared = (a.T + 15) / 16 * scols, items = shared + nseg * cols;
  const bool two = S != W && shared > 0 && nseg > 0;
  const int mine = two ? 3 : 4;   // the waves of a kind, as a power of two, as KS
  auto plan = [&](int n, int units, int& KS, int& rounds) {
    KS = share_of(n, gridDim.x, mine, units, min(mine, a.most_ks));
    const int step = gridDim.x << (mine - KS);
    rounds = quot_wave(n + step - 1, step);
  };
  int KS, rounds, KS2 = 0, rounds2 = 0;
  plan(two ? shared : items, a.D / (shared > 0 ? Fmt<S>::UK : Fmt<W>::UK), KS, rounds);
  if (two) plan(items - shared, a.D / Fmt<W>::UK, KS2, rounds2);
  const bool meet = KS > 0 || KS2 > 0, second = two && wave >= WAVES / 2;
  const int turns = max(rounds, rounds2);   // the same for all waves, for the barriers
  if (second) KS = KS2;
  const int w = wave & ((1 << mine) - 1), kw = w & ((1 << KS) - 1);
  const int from = (second ? shared : 0) + (w >> KS) * gridDim.x + blockIdx.x;
  const int end = two && !second ? shared : items;

  for (int r = 0; r < turns; ++r) {
    const int item = from + r * (gridDim.x << (mine - KS));
    const bool there = item < end, sh = item < shared;
    const int at = there ? (sh ? item : item - shared) : 0;
    const int group = quot_wave(at, sh ? scols : cols), n0 = (at - group * (sh ? scols : cols)) * 16;
    const int seg = sh || !there ? 0 : tb.seg[group];
    const int e = seg % SEGE;
    const int t = column_token(tb, seg, sh, group, fr, a.T, 16);
    acc[0] = acc[1] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    if (there) {
      const int N = sh ? a.Fs : a.F;
      if (S == W || !sh) {
        const Rows m1 = rows_at<W>(sh ? a.ws1 : a.w1, a.s1, e, N, a.D, n0 + fr, g);
        const Rows m3 = rows_at<W>(sh ? a.ws3 : a.w3, a.s3, e, N, a.D, n0 + fr, g);
        fc1_item<W, PW, XL>(m1, m3, (size_t)a.E * a.F * 4, a.x, xl, a.T, t, xrow,
                            a.D / Fmt<W>::UK, kw, 1 << KS, acc);
      } else {
        const Rows m1 = rows_at<S>(a.ws1, nullptr, 0, N, a.D, n0 + fr, g);
        const Rows m3 = rows_at<S>(a.ws3, nullptr, 0, N, a.D, n0 + fr, g);
        fc1_item<S, PS, XL>(m1, m3, 0, a.x, xl, a.T, t, xrow, a.D / Fmt<S>::UK, kw, 1 << KS, acc);
      }
    }
    if (meet) {   // the waves' sums in wave order
      if (kw > 0)
#pragma unroll
        for (int m = 0; m < 2; ++m) red[(wave * 2 + m) * 64 + lane] = acc[m];
      lds_barrier();
      if (kw == 0)
        for (int o = wave + 1; o < wave + (1 << KS); ++o)
#pragma unroll
          for (int m = 0; m < 2; ++m) acc[m] += red[(o * 2 + m) * 64 + lane];
      lds_barrier();
    }
    if (kw > 0 || !there || t < 0) continue;
    // lane l holds column l%16 and rows 4*(l/16) .. +3 of the item's 16
    f32x4 v;
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] = silu_mul<Act>(acc[0][q], acc[1][q]);
    if (sh) {
      store4(static_cast<Act*>(a.hs) + (size_t)t * a.Fs + n0 + 4 * g, v);
    } else {
      // the first of the token's slots that hold e; a second one shares its h
      for (int j = 0; j < a.k; ++j)
        if (tb.idx[t * a.k + j] == e) {
          store4(static_cast<Act*>(a.h) + ((size_t)t * a.k + j) * a.F + h_at<W>(n0 + 4 * g), v);
          break;
        }
    }
  }
}

// Token t's weight of expert e (the sum over its slots that hold e) and the first such slot,
// -1 if there is none.
__device__ __forceinline__ int find_slot(const int* idx, const float* tw, int t, int k, int e,
                                         float& w) {
  int at = -1;
  w = 0.0f;
  for (int j = k - 1; j >= 0; --j)
    if (idx[t * k + j] == e) {
      at = t * k + j;
      w += tw[at];
    }
  return at;
}

// Wave `wave`'s share (of `waves`) of the units of segments [first, nseg), then (nsh > 0) of the
// shared experts' groups of tokens, added to the wave's sums `tot` in LDS ([NS][T][RC] float32).
// With NS > 1 the instruction's 16 rows and columns are NS streams: rows and columns
// [s * RC, (s + 1) * RC) hold the same output columns, and RC tokens, at the units of another share, so all of
// a load's 16 rows are new bytes; of the products only those of one stream's rows with its own
// columns are taken. A lane then follows its stream (lane % 16 / RC) for loads and sums alike.
// HL: h (and hs behind it) in LDS at hl; `filled` is called once the first weights are on the way.
template <int W, int NS, int PF, bool HL, typename Filled>
__device__ __forceinline__ void fc2_units(const FewArgs& a, const Tables& tb, int first, int nseg,
                                          int nsh, int n0, int wave, int waves, const char* hl,
                                          Filled filled, float* tot) {
  typedef typename Fmt<W>::Act Act;
  constexpr int NF = Fmt<W>::NF, RC = 16 / NS;
  const int lane = threadIdx.x & 63, fr = lane & 15, g = lane >> 4;
  const int stream = fr / RC, c = fr % RC;
  const int U = a.F / Fmt<W>::UK, Us = a.Fs / Fmt<W>::UK;
  const int routed = (nseg - first) * U, all = routed + nsh * Us;
  const int share = wave * NS + (NS == 1 ? 0 : stream);
  // even shares, the first `rest` of them one longer (all < 2^22, the segments' units of k)
  const int even = quot_wave(all, waves * NS), rest = all - even * (waves * NS);
  const int lo = share * even + min(share, rest), n = even + (share < rest ? 1 : 0);
  const int most = NS == 1 ? n : even + (rest > 0 ? 1 : 0);   // the longest share
  if (most <= 0) {
    filled();
    return;
  }
  const size_t sstep = (size_t)a.E * a.D * 4;
  const __amdgpu_buffer_rsrc_t rs = act_rsrc(a.h, a.hs_off + (size_t)a.T * a.Fs * sizeof(Act));
  // where this lane's four results of a sum go, if its rows are its columns' stream's
  const bool own = NS == 1 || g / (RC / 4) == stream;
  float* sums = tot + (size_t)stream * a.T * RC + (4 * g) % RC;

  WReg<W> wr[PF];
  u32x4 xr[HL ? 1 : PF][NF];
  // the load side's segment and unit, and the sums'; a share without units reads the first
  const int begin = n > 0 ? lo : 0;
  const bool bs = begin >= routed;
  const int bu = bs ? Us : U, bq = NS == 1 ? quot_wave(bs ? begin - routed : begin, bu)
                                                 : quot(bs ? begin - routed : begin, bu);
  int ls = (bs ? nseg : first) + bq, lu = (bs ? begin - routed : begin) - bq * bu;
  int cs = ls, cu = lu;
  Rows m;
  uint32_t off;     // the column's row: bytes into h (hs behind it)
  int tok;          // its token, -1: none
  float weight;     // and the weight of its sums
  auto weights = [&]() {
    m = ls >= nseg ? rows_at<W>(a.ws2, nullptr, 0, a.D, a.Fs, n0 + c, g)
                   : rows_at<W>(a.w2, a.s2, tb.seg[ls] % SEGE, a.D, a.F, n0 + c, g);
  };
  auto column = [&](int s) {
    const bool sh = s >= nseg;
    const int seg = sh ? 0 : tb.seg[s];
    tok = column_token(tb, seg, sh, s - nseg, c, a.T, RC);
    weight = 1.0f;
    int at = tok;
    if (tok >= 0 && !sh) {
      at = find_slot(tb.idx, tb.w, tok, a.k, seg % SEGE, weight);
      if (at < 0) tok = -1;
    }
    off = (uint32_t)at * (uint32_t)((sh ? a.Fs : a.F) * sizeof(Act)) + (sh ? a.hs_off : 0u);
    if (HL)
      off = tok < 0 ? 0u : off;   // some row; nothing of it is kept
    else
      off = tok < 0 ? PAST : off + g * H_LANE;
  };
  auto load = [&](int j, int s) {
    load_unit<W>(wr[j], m, sstep, lu);
    if constexpr (!HL) load_x<W, H_NEXT>(xr[j], rs, off == PAST ? PAST : off + lu * Fmt<W>::XB, 0);
    if (s + 1 < n) {   // a stream past its share's end reads its last unit again
      ++lu;
      if (lu == (ls >= nseg ? Us : U)) {
        lu = 0;
        ++ls;
        weights();
        if constexpr (!HL) column(ls);
      }
    }
  };
  f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f}, sum = acc;
  auto flush = [&]() {   // the segment's sums, weighted
    if constexpr (W == kFewF32) {
      acc += sum;
      sum = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
    const uint32_t keep = off;
    const int kt = tok;
    if constexpr (!HL) column(cs);   // (the load side is further on)
    if (own && tok >= 0) {
      f32x4* p = reinterpret_cast<f32x4*>(sums + tok * RC);
      f32x4 v = *p;
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] = __builtin_fmaf(weight, acc[q], v[q]);
      *p = v;
    }
    if constexpr (!HL) {
      off = keep;
      tok = kt;
    }
    acc = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  };
  auto compute = [&](int j, int s) {
    if constexpr (HL) {
#pragma unroll
      for (int f = 0; f < NF; ++f) xr[0][f] = lds_piece<W, H_LANE, H_NEXT>(hl + off, max(tok, 0), g, cu, f);
    }
#pragma unroll
    for (int f = 0; f < NF; ++f) mul<W>(wr[j], xr[HL ? 0 : j][f], f, acc);
    if (chain_ends<W>(s)) {
      sum += acc;
      acc = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
    if (s + 1 < n) {
      ++cu;
      if (cu == (cs >= nseg ? Us : U)) {
        flush();
        cu = 0;
        ++cs;
        if constexpr (HL) column(cs);
      }
    } else if (s + 1 == n) {   // what a stream multiplies past its end is not taken
      flush();
    }
  };
  weights();
  column(ls);
#pragma unroll
  for (int j = 0; j < PF; ++j)
    if (j < most) load(j, j);
  filled();
  ring<PF, false>(most, load, compute);
}

template <int W, int S, int NS, bool HL>
__global__ __launch_bounds__(THREADS) void few_fc2(const FewArgs a) {
  typedef typename Fmt<W>::Act Act;
  // units in flight. They matter where rows of h come from the L2 (16 tokens over 8 experts of 14336, the
  // call in us: bf16 2 506, 3 482, 4 502; 32 tokens, 4 bits: 1 254, 2 251, 3 249, 4 251); with h in LDS one
  // token over 64 experts takes 40 to 41 with one to four, 4-bit 27.7 with two or three, 28.6 with four or six
  constexpr int PW = W == kFewMx4 ? (HL ? 4 : 2) : (HL ? 2 : 3), PS = 2, RC = 16 / NS;
  __shared__ Tables tb;
  __shared__ __attribute__((aligned(256))) char pool[HL ? POOL : MAXT * 1024];
  float* tot = reinterpret_cast<float*>(pool);   // [WAVES][NS][T][RC]
  char* hl = pool + a.T * 1024;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int slots = a.T * a.k;
  int mine = -1;
  if (slots <= 64) {   // every wave for itself, the same values
    if (lane < slots) {
      mine = a.topk_idx[lane];
      tb.idx[lane] = mine;
      tb.w[lane] = a.topk_w[lane];
    }
  } else {
    for (int i = threadIdx.x; i < slots; i += THREADS) {
      tb.idx[i] = a.topk_idx[i];
      tb.w[i] = a.topk_w[i];
    }
    __syncthreads();
  }
  const int nseg = segments(tb, mine, a.T, a.k, a.E, RC);
  const int nsh = a.Fs > 0 ? (a.T + RC - 1) / RC : 0;
  bool fill = HL;
  auto filled = [&]() {
    if (!fill) return;
    fill = false;
    fill_rows(hl, a.h, slots, a.F * (int)sizeof(Act), a.k);
    if (a.Fs) fill_rows(hl + a.hs_off, a.hs, a.T, a.Fs * (int)sizeof(Act), 1);
    __syncthreads();
  };
  // where the formats differ, the waves are shared out by the bytes of each
  int ws = 0;
  if (S != W && nsh > 0) {
    const float bs = 64.0f * (float)(nsh * a.Fs), br = 17.0f * (float)(nseg * a.F);
    ws = nseg == 0 ? WAVES : max(1, min(WAVES - 1, (int)(WAVES * bs * __builtin_amdgcn_rcpf(bs + br) + 0.5f)));
    ws = __builtin_amdgcn_readfirstlane(ws);
  }
  float* sums = tot + (size_t)wave * 16 * a.T;
  for (int ch = blockIdx.x; ch < a.D / RC; ch += gridDim.x) {
    for (int i = lane; i < 4 * a.T; i += 64) reinterpret_cast<f32x4*>(sums)[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    if (S == W)
      fc2_units<W, NS, PW, HL>(a, tb, 0, nseg, nsh, ch * RC, wave, WAVES, hl, filled, sums);
    else if (wave < ws)
      fc2_units<S, NS, PS, HL>(a, tb, nseg, nseg, nsh, ch * RC, wave, ws, hl, filled, sums);
    else
      fc2_units<W, NS, PW, HL>(a, tb, 0, nseg, 0, ch * RC, wave - ws, WAVES - ws, hl, filled, sums);
    lds_barrier();
    for (int o = threadIdx.x; o < RC * a.T; o += THREADS) {   // the waves' sums in wave order
      float v = 0.0f;
#pragma unroll
      for (int s = 0; s < WAVES * NS; ++s) v += tot[(size_t)s * RC * a.T + o];
      Act* out = static_cast<Act*>(a.out) + (size_t)(o / RC) * a.D + ch * RC + o % RC;
      if constexpr (sizeof(Act) == 2)
        *out = (Act)f32_to_bf16(v);
      else
        *out = v;
    }
    lds_barrier();
  }
}

template <int W, int S, int NS>
void launch_fc2(const FewArgs& a, hipStream_t s) {
  typedef typename Fmt<W>::Act Act;
  const dim3 grid(std::min(cu_count(), a.D * NS / 16)), block(THREADS);
  const bool hl = (int64_t)a.hs_off + (int64_t)a.T * (a.Fs * sizeof(Act) + 1024) <= POOL;
  if (hl)
    hipLaunchKernelGGL((few_fc2<W, S, NS, true>), grid, block, 0, s, a);
  else
    hipLaunchKernelGGL((few_fc2<W, S, NS, false>), grid, block, 0, s, a);
}

template <int W, int S>
void launch_fmt(FewArgs a, hipStream_t s) {
  typedef typename Fmt<W>::Act Act;
  const int cus = cu_count();
  const dim3 block(THREADS);
  const int most = std::min(a.E * ((a.T + 15) / 16), a.T * a.k) * (a.F / 16) + (a.T + 15) / 16 * (a.Fs / 16);
  const dim3 grid1(std::min(cus, most));
  // The tokens' rows in LDS beside the waves' sums, or, where they need all of it, with one wave
  // an item; rows that do not fit come from the L2.
  const int64_t rows = (int64_t)a.T * a.D * sizeof(Act);
  const bool xl = rows <= POOL;
  a.most_ks = !xl || rows + RED <= POOL ? 4 : 0;
  const int ne = !a.wg ? 0 : (a.E <= 64 ? 1 : (a.E <= 256 ? 4 : 16));
  const auto fc1 = xl ? (ne == 0 ? few_fc1<W, S, 0, true> : ne == 1 ? few_fc1<W, S, 1, true>
                         : ne == 4 ? few_fc1<W, S, 4, true> : few_fc1<W, S, 16, true>)
                      : (ne == 0 ? few_fc1<W, S, 0, false> : ne == 1 ? few_fc1<W, S, 1, false>
                         : ne == 4 ? few_fc1<W, S, 4, false> : few_fc1<W, S, 16, false>);
  hipLaunchKernelGGL(fc1, grid1, block, 0, s, a);
  // Output columns at a time, RC of 16, 8 and 4: those with the least of rounds * (RC + 8), the 8 for
  // what a round costs beside its columns (one token and 8 tokens over 32 experts, in us: D = 1152
  // 16 25.7 67.9, 8 25.1 57.5, 4 26.8 58.8; D = 2304 29.9 94.7, 33.8 99.9, 35.4 95.1; D = 5120 59.0
  // 177, 60.0 170, 64.9 170).
  auto cost = [&](int rc) { return (a.D / rc + cus - 1) / cus * (rc + 8); };
  if (cost(16) <= std::min(cost(8), cost(4)))
    launch_fc2<W, S, 1>(a, s);
  else if (cost(8) <= cost(4))
    launch_fc2<W, S, 2>(a, s);
  else
    launch_fc2<W, S, 4>(a, s);
}

template <typename TIn>
void launch_logits(const FewArgs& a, hipStream_t s) {
  // a token at a time where that does not fill the card (8 tokens, 256 experts of D = 7168: the call
  // 143.5 us, four at a time 148; calls with F = 128 and top-1, one at a time against four: 12 tokens over
  // these 41 and 43.5, 16 46 and 48, 24 50 both, 32 58 and 57.5; over 8 experts of 4096 12 tokens 23.8 and 25.9,
  // 24 25.5 and 27.7, 32 26.1 and 28.3)
  const bool one = a.T < 16;
  const auto f = one ? few_logits<TIn, 1> : few_logits<TIn, 4>;
  const dim3 grid((a.E + LOGIT_WAVES - 1) / LOGIT_WAVES, one ? a.T : (a.T + 3) / 4);
  hipLaunchKernelGGL(f, grid, dim3(64 * LOGIT_WAVES), 0, s, static_cast<const TIn*>(a.x),
                     static_cast<const TIn*>(a.wg), a.bias, a.T, a.D, a.E, a.logits);
}

// h and hs
size_t rows_bytes(int fmt, int T, int k, int F, int Fs) {
  const size_t b = fmt == kFewF32 ? 4 : 2;
  return ((size_t)T * k * F + (size_t)T * Fs) * b;
}

}  // namespace

size_t few_workspace_bytes(int fmt, int T, int k, int F, int Fs) {
  return rows_bytes(fmt, T, k, F, Fs) + (size_t)T * MAXE * sizeof(float);
}

hipError_t launch_few(int fmt, const FewCall& c, hipStream_t s) {
  FewArgs a;
  a.x = c.x;
  a.wg = c.wg;
  a.bias = c.bias;
  a.T = c.T;
  a.D = c.D;
  a.F = c.F;
  a.E = c.E;
  a.k = c.k;
  a.renorm = c.renorm;
  a.Fs = c.Fs;
  a.w1 = c.w[0];
  a.w3 = c.w[1];
  a.w2 = c.w[2];
  a.s1 = c.s[0];
  a.s3 = c.s[1];
  a.s2 = c.s[2];
  a.ws1 = c.ws[0];
  a.ws3 = c.ws[1];
  a.ws2 = c.ws[2];
  a.topk_idx = c.topk_idx;
  a.topk_w = c.topk_w;
  a.h = c.workspace;
  a.hs_off = (uint32_t)((size_t)c.T * c.k * c.F * (fmt == kFewF32 ? 4 : 2));   // at most 2^28
  a.hs = static_cast<char*>(c.workspace) + a.hs_off;
  a.out = c.out;
  a.logits = reinterpret_cast<float*>(static_cast<char*>(c.workspace) + rows_bytes(fmt, c.T, c.k, c.F, c.Fs));
  if (c.wg) {
    if (fmt == kFewF32)
      launch_logits<float>(a, s);
    else
      launch_logits<bf16_t>(a, s);
  }
  if (fmt == kFewF32)
    launch_fmt<kFewF32, kFewF32>(a, s);
  else if (fmt == kFewBf16)
    launch_fmt<kFewBf16, kFewBf16>(a, s);
  else
    launch_fmt<kFewMx4, kFewBf16>(a, s);
  return hipGetLastError();
}

}  // namespace moe
