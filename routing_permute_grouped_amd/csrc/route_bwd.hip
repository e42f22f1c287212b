// The router's backward, from the gradient of the top-k weights. With p = softmax(logits):
//   weights p[idx]:             dl_e = p_e (dp_e - sum_i p_i dp_i), dp_e the sum of dw over the
//                               token's slots that hold e
//   weights made to sum to one: dl_e = sum over those slots of w_j (dw_j - sum_i w_i dw_i)
//   dl += dlogits_add;  dx = dl wg (+ dx_add);  dwg = dl^T x;  dbias = sum_t dl
//
// Bound by HBM: x and dx_add are read once, dx is written once. The products are thin (E of
// some tens), so they run on the matrix cores without LDS tiles: both sum over the rows of a
// row-major matrix (wg over e, x over t), and a lane builds the instruction's operand from
// loads of 16 bytes of RL consecutive rows, taking every element's RL rows together
// (byte permutes in bf16, nothing in float32). A block of 16 columns is then every
// CL-th column, and a lane's results over the CL blocks are CL neighbours, stored at once.
//   * bf16: dl enters as bf16 summands (dl = hi + mid + lo, the first two for dx, whose own
//     rounding is 2^8 times coarser than their 2^-17, all three for the float32 dwg). x and
//     wg are exact in bf16, so the products are those of float32 dl. float32: the float32
//     matrix instruction.
//   * dwg sums over the tokens: a workgroup's waves take slices of a range of tokens, their sums
//     meet in LDS in wave order, and a last kernel adds the ranges in order. Equal calls give
//     equal bits.
// dl is written in the operands' form (rows and transposed, padded with zeros) by the first
// kernel beside its float32 output.
#include <algorithm>
#include <type_traits>

#include "common.hpp"
#include "kernels.hpp"
#include "route_bwd.hpp"
#include "wave.hpp"

namespace moe {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kTok = 32;       // tokens of a workgroup of the first kernel, and T's padding
constexpr int kDlWaves = 16;
// Most workgroups of the first kernel along the grid's x, the others along its y: one for every kTok tokens
// along x alone would pass the 2^32 threads of that dimension from 2^27 tokens, of which the runtime then
// keeps the low 32 bits. (Turns of fewer workgroups instead: 65536 tokens over 64 experts 43.8 us against 41.6.)
constexpr int kMostX = 1 << 16;
// Tokens of a short batch, whose ranges are one: a launch less, which counts where the call waits for the
// host (20 us of it), against more workgroups. On the GPU alone, as in a graph, one range against more: to
// 700 tokens the same, 1024 tokens over 64 experts of 2048 23.6 us against 19.3, over 8 of 512 in float32
// 18.3 against 13.6.
constexpr int kShort = 1024;
constexpr int kWaves = 8;          // waves of a workgroup of the products
constexpr int kDxWaves = 2048;     // and dx

// RL: rows of k in a lane's 16-byte operand; CL: columns a lane loads of each; KS: k of a step;
// SP: summands of dl in dwg, SX in dx; DW: waves that dwg is cut into (float32, bound by its matrix
// instruction, 3489 tokens over 78 experts of D = 2816: 2048 68 us, 1024 94; bf16, bound by memory,
// 8192 over 64 of 2048: 1024 41.6, 2048 46).
template <typename T> struct Op;
template <> struct Op<bf16_t> {
  typedef bf16_t Part;
  static constexpr int RL = 8, CL = 8, KS = 32, SP = 3, SX = 2, DW = 1024;
};
template <> struct Op<float> {
  typedef float Part;
  static constexpr int RL = 4, CL = 4, KS = 16, SP = 1, SX = 1, DW = 2048;
};

// Element q of the RL rows a lane has loaded, as one operand.
__device__ __forceinline__ u32x4 column(const u32x4 (&r)[8], int q) {
  const uint32_t sel = q & 1 ? 0x07060302u : 0x05040100u;
  u32x4 f;
#pragma unroll
  for (int j = 0; j < 4; ++j) f[j] = __builtin_amdgcn_perm(r[2 * j + 1][q >> 1], r[2 * j][q >> 1], sel);
  return f;
}
__device__ __forceinline__ u32x4 column(const u32x4 (&r)[4], int q) {
  return u32x4{r[0][q], r[1][q], r[2][q], r[3][q]};
}

template <typename T>
__device__ __forceinline__ f32x4 mma(const u32x4& a, const u32x4& b, f32x4 c) {
  if constexpr (sizeof(T) == 2) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a[i]), __uint_as_float(b[i]), c, 0, 0, 0);
    return c;
  }
}

// Where the workspace's parts lie.
struct Parts {
  void* rows;        // [SX][T][Ep]
  void* cols;        // [SP][Tp / kTok][Ep][kTok]: a step's rows lie side by side
  float* dbias;      // [Tp / kTok][E]
  float* dwg;        // [S][E][D]
};

// dl of R tokens (t0, t0 + step, ...) by one wave, their chains side by side; NE experts a lane.
// Tokens past T leave zeros in LDS.
template <int NE, int R>
__device__ __forceinline__ void token_dl(const RouteBwdCall& a, int t0, int step, int lane,
                                         float* rows, int ld) {
  int e[R], t[R];
  float slot[R];   // what the lane's slot adds to its expert's dl (renorm) or dp
  float l[R][NE], add[R][NE], dl[R][NE];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    t[r] = min(t0 + r * step, a.T - 1);
    e[r] = -1;
    slot[r] = 0.0f;
    if (lane < a.k) {
      e[r] = a.topk_idx[(size_t)t[r] * a.k + lane];
      slot[r] = a.dtopk_w[(size_t)t[r] * a.k + lane];
      if (e[r] < 0 || e[r] >= a.E) {
        e[r] = -1;
        slot[r] = 0.0f;
      }
    }
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      const int x = lane + 64 * i;
      dl[r][i] = add[r][i] = 0.0f;
      l[r][i] = -INFINITY;
      if (x < a.E) {
        l[r][i] = a.logits[(size_t)t[r] * a.E + x];
        if (a.dlogits_add) add[r][i] = a.dlogits_add[(size_t)t[r] * a.E + x];
      }
    }
  }
  if (a.renorm) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      // the slot's logit sits in lane e % 64
      float s = -INFINITY;
#pragma unroll
      for (int i = 0; i < NE; ++i) {
        const float v = __shfl(l[r][i], e[r] & 63);
        if (e[r] >= 0 && e[r] >> 6 == i) s = v;
      }
      const float mx = wave_max(s);   // every lane takes part
      const float ex = e[r] >= 0 ? expf(s - mx) : 0.0f;
      const float w = ex / wave_sum(ex);
      const float c = wave_sum(e[r] >= 0 ? w * slot[r] : 0.0f);
      slot[r] = e[r] >= 0 ? w * (slot[r] - c) : 0.0f;
    }
  }
  for (int j = 0; j < a.k; ++j)
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int ej = __builtin_amdgcn_readlane(e[r], j);
      const float sj = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(slot[r]), j));
#pragma unroll
      for (int i = 0; i < NE; ++i) dl[r][i] += lane + 64 * i == ej ? sj : 0.0f;
    }
  if (!a.renorm) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float mx = l[r][0];
#pragma unroll
      for (int i = 1; i < NE; ++i) mx = fmaxf(mx, l[r][i]);
      mx = wave_max(mx);
      float sum = 0.0f, dot = 0.0f;
#pragma unroll
      for (int i = 0; i < NE; ++i) {
        l[r][i] = lane + 64 * i < a.E ? expf(l[r][i] - mx) : 0.0f;
        sum += l[r][i];
      }
      sum = wave_sum(sum);
#pragma unroll
      for (int i = 0; i < NE; ++i) {
        l[r][i] /= sum;
        dot = __builtin_fmaf(l[r][i], dl[r][i], dot);
      }
      dot = wave_sum(dot);
      const bool any = __ballot(e[r] >= 0) != 0;   // without a slot nothing reaches the logits, NaN ones too
#pragma unroll
      for (int i = 0; i < NE; ++i) dl[r][i] = any ? l[r][i] * (dl[r][i] - dot) : 0.0f;
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const bool there = t0 + r * step < a.T;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      const int x = lane + 64 * i;
      if (x < a.E) {
        const float v = dl[r][i] + add[r][i];
        if (there) a.dlogits[(size_t)t[r] * a.E + x] = v;
        rows[r * step * ld + x] = there ? v : 0.0f;
      }
    }
  }
}

// Summand s of v: the first is v rounded, each next the rounded rest.
template <int S>
__device__ __forceinline__ void summands(float v, uint32_t (&o)[S]) {
#pragma unroll
  for (int s = 0; s < S; ++s) {
    o[s] = f32_to_bf16(v);
    v -= bf16_to_f32(o[s]);
  }
}

template <typename TIn, int NE>
__global__ __launch_bounds__(kDlWaves * 64) void route_dl_kernel(const RouteBwdCall a, Parts p, int Ep, int Tp) {
  constexpr int R = NE == 16 ? 1 : kTok / kDlWaves, W = kDlWaves;
  __shared__ float tile[kTok * (64 * NE + 1)];   // [kTok][Ep + 1]
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int group = blockIdx.y * gridDim.x + blockIdx.x;
  if (group >= Tp / kTok) return;
  const int t0 = group * kTok, ld = Ep + 1;
  for (int r = wave; r < kTok; r += W)
    for (int e = a.E + lane; e < Ep; e += 64) tile[r * ld + e] = 0.0f;
  for (int r = wave; r < kTok; r += W * R) token_dl<NE, R>(a, t0 + r, W, lane, tile + r * ld, ld);
  __syncthreads();
  constexpr int SP = Op<TIn>::SP, SX = Op<TIn>::SX;
  const size_t nrow = (size_t)a.T * Ep, ncol = (size_t)Ep * Tp;
  // the operands' forms, four neighbours a thread
  auto put = [&](void* base, size_t at, size_t part, const float (&v)[4], auto S) {
    if constexpr (sizeof(TIn) == 2) {
      uint32_t o[4][S.value];
#pragma unroll
      for (int i = 0; i < 4; ++i) summands<S.value>(v[i], o[i]);
#pragma unroll
      for (int s = 0; s < S.value; ++s)
        *reinterpret_cast<uint2*>(static_cast<bf16_t*>(base) + s * part + at) =
            uint2{o[0][s] | o[1][s] << 16, o[2][s] | o[3][s] << 16};
    } else {
      *reinterpret_cast<f32x4*>(static_cast<float*>(base) + at) = f32x4{v[0], v[1], v[2], v[3]};
    }
  };
  if (a.dx) {
    const int q = Ep / 4;   // quads of a row: 8, or a multiple of 16
    for (int i = threadIdx.x; i < kTok * q; i += W * 64) {
      const int r = i / q, e = i % q * 4;
      if (t0 + r >= a.T) break;
      const float* v = tile + r * ld + e;
      put(p.rows, (size_t)(t0 + r) * Ep + e, nrow, {v[0], v[1], v[2], v[3]}, std::integral_constant<int, SX>());
    }
  }
  if (a.dwg) {
    const int r = 4 * (lane & 7);
    for (int e = wave * 8 + (lane >> 3); e < Ep; e += 8 * W) {
      const float* v = tile + r * ld + e;
      put(p.cols, ((size_t)group * Ep + e) * kTok + r, ncol, {v[0], v[ld], v[2 * ld], v[3 * ld]},
          std::integral_constant<int, SP>());
    }
  }
  if (a.dbias)
    for (int e = threadIdx.x; e < a.E; e += W * 64) {
      float s = 0.0f;
      for (int r = 0; r < kTok; ++r) s += tile[r * ld + e];
      p.dbias[(size_t)group * a.E + e] = s;
    }
}

// dx of one block of 16 tokens and 16*CL columns from the sums: lane l holds columns
// CL*(l%16) .. +CL-1 of tokens 4*(l/16) + r, so 16 lanes write a token's columns side by side.
template <typename TIn>
__device__ __forceinline__ void store_dx(const RouteBwdCall& a, const f32x4 (&acc)[Op<TIn>::CL],
                                         const u32x4 (&add)[4], int t0, int col, int g) {
  constexpr int CL = Op<TIn>::CL;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int t = t0 + 4 * g + r;
    if (t >= a.T || col >= a.D) continue;
    float v[CL];
#pragma unroll
    for (int q = 0; q < CL; ++q) v[q] = acc[q][r];
    if (a.dx_add) {
      float f[CL];
      Chunk<TIn>::widen(add[r], f);
#pragma unroll
      for (int q = 0; q < CL; ++q) v[q] += f[q];
    }
    st16(static_cast<TIn*>(a.dx) + (size_t)t * a.D + col, Chunk<TIn>::narrow(v));
  }
}
template <typename TIn>
__device__ __forceinline__ void load_add(const RouteBwdCall& a, u32x4 (&add)[4], int t0, int col, int g) {
  if (!a.dx_add) return;
#pragma unroll
  for (int r = 0; r < 4; ++r)
    add[r] = ld16(static_cast<const TIn*>(a.dx_add) + (size_t)min(t0 + 4 * g + r, a.T - 1) * a.D +
                     min(col, a.D - Op<TIn>::CL));
}

// dx for at most 64 experts: a wave builds the operands of its 16*CL columns of wg once and takes
// `per` blocks of 16 tokens, the next one's dl and dx_add on the way.
template <typename TIn, int STEPS>
__device__ __forceinline__ void dx_body(const RouteBwdCall& a, const Parts& p, int strips, int per,
                                        int64_t id) {
  typedef Op<TIn> O;
  typedef typename O::Part Part;
  constexpr int Ep = STEPS * O::KS;
  const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
  const int blocks = (a.T + 15) / 16;
  const int first = (int)(id / strips) * per, last = min(first + per, blocks);
  if (first >= last) return;
  const int col = (int)(id % strips) * 16 * O::CL + n * O::CL;
  const size_t nrow = (size_t)a.T * Ep;
  const Part* rows = static_cast<const Part*>(p.rows);
  u32x4 d[2][STEPS][O::SX], add[2][4];
  auto load = [&](int j, int b) {
    const Part* at = rows + (size_t)min(16 * b + n, a.T - 1) * Ep + g * O::RL;
#pragma unroll
    for (int s = 0; s < STEPS; ++s)
#pragma unroll
      for (int i = 0; i < O::SX; ++i) d[j][s][i] = ld16(at + i * nrow + s * O::KS);
    load_add<TIn>(a, add[j], 16 * b, col, g);
  };
  load(0, first);
  u32x4 f[STEPS][O::CL];
#pragma unroll
  for (int s = 0; s < STEPS; ++s) {
    u32x4 w[O::RL];
#pragma unroll
    for (int i = 0; i < O::RL; ++i)   // rows past E meet zeros of dl
      w[i] = ld16(static_cast<const TIn*>(a.wg) + (size_t)min(s * O::KS + g * O::RL + i, a.E - 1) * a.D +
                  min(col, a.D - O::CL));
#pragma unroll
    for (int q = 0; q < O::CL; ++q) f[s][q] = column(w, q);
  }
  for (int b = first; b < last; b += 2)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if (b + j >= last) break;
      load(j ^ 1, min(b + j + 1, last - 1));
      f32x4 acc[O::CL];
#pragma unroll
      for (int q = 0; q < O::CL; ++q) {
        acc[q] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int s = 0; s < STEPS; ++s)
#pragma unroll
          for (int i = O::SX - 1; i >= 0; --i) acc[q] = mma<TIn>(d[j][s][i], f[s][q], acc[q]);
      }
      store_dx<TIn>(a, acc, add[j], 16 * (b + j), col, g);
    }
}

// dx for more experts: a wave takes 64 tokens and 16*CL columns, k = e in steps.
template <typename TIn>
__device__ __forceinline__ void dx_wide_body(const RouteBwdCall& a, const Parts& p, int Ep,
                                             int strips, int64_t id) {
  typedef Op<TIn> O;
  typedef typename O::Part Part;
  constexpr int NB = 4;
  const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
  const int t0 = (int)(id / strips) * 16 * NB;
  if (t0 >= a.T) return;
  const int col = (int)(id % strips) * 16 * O::CL + n * O::CL;
  const size_t nrow = (size_t)a.T * Ep;
  f32x4 acc[NB][O::CL];
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int q = 0; q < O::CL; ++q) acc[b][q] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  const Part* rows = static_cast<const Part*>(p.rows);
  for (int e0 = 0; e0 < a.E; e0 += O::KS) {
    u32x4 w[O::RL], d[O::SX][NB];
#pragma unroll
    for (int i = 0; i < O::RL; ++i)
      w[i] = ld16(static_cast<const TIn*>(a.wg) + (size_t)min(e0 + g * O::RL + i, a.E - 1) * a.D + min(col, a.D - O::CL));
#pragma unroll
    for (int s = 0; s < O::SX; ++s)
#pragma unroll
      for (int b = 0; b < NB; ++b)
        d[s][b] = ld16(rows + s * nrow + (size_t)min(t0 + 16 * b + n, a.T - 1) * Ep + e0 + g * O::RL);
#pragma unroll
    for (int q = 0; q < O::CL; ++q) {
      const u32x4 f = column(w, q);
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int s = O::SX - 1; s >= 0; --s) acc[b][q] = mma<TIn>(d[s][b], f, acc[b][q]);
    }
  }
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    u32x4 add[4];
    load_add<TIn>(a, add, t0 + 16 * b, col, g);
    store_dx<TIn>(a, acc[b], add, t0 + 16 * b, col, g);
  }
}

// dwg: a workgroup takes 16*MB experts, 16*CL columns and a range of tokens.
template <typename TIn, int MB>
__device__ __forceinline__ void dwg_body(const RouteBwdCall& a, const Parts& p, int Ep, int Tp,
                                         int strips, int chunks, int S, int block,
                                         float* __restrict__ out) {
  typedef Op<TIn> O;
  typedef typename O::Part Part;
  constexpr int COLS = 16 * O::CL;
  constexpr int HALF = MB % 2 == 0 ? MB / 2 : 1;   // expert blocks that meet in LDS at a time
  __shared__ f32x4 red[kWaves * HALF * 16 * COLS / 4];
  const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int strip = block % strips, chunk = block / strips % chunks;
  const int split = block / (strips * chunks);
  const int c0 = strip * COLS, e0 = chunk * 16 * MB, col = c0 + n * O::CL;
  const bool in = col < a.D;
  const size_t ncol = (size_t)Ep * Tp;
  const int steps = Tp / O::KS, slices = S * kWaves;
  const int sl = split * kWaves + wave;
  const int lo = (int)((int64_t)steps * sl / slices), hi = (int)((int64_t)steps * (sl + 1) / slices);
  f32x4 acc[MB][O::CL];
#pragma unroll
  for (int m = 0; m < MB; ++m)
#pragma unroll
    for (int q = 0; q < O::CL; ++q) acc[m][q] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  const Part* cols = static_cast<const Part*>(p.cols);
  u32x4 x[2][O::RL];
  auto load_x = [&](int j, int s) {
#pragma unroll
    for (int i = 0; i < O::RL; ++i)   // tokens past T meet zeros of dl
      x[j][i] = ld16_nt(static_cast<const TIn*>(a.x) + (size_t)min(s * O::KS + g * O::RL + i, a.T - 1) * a.D + (in ? col : 0));
  };
  if (lo < hi) load_x(0, lo);
  for (int s0 = lo; s0 < hi; s0 += 2)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int s = s0 + j, t0 = s * O::KS;
      if (s >= hi) break;
      u32x4 d[O::SP][MB];
#pragma unroll
      for (int i = 0; i < O::SP; ++i)
#pragma unroll
        for (int m = 0; m < MB; ++m)
          d[i][m] = ld16(cols + i * ncol + ((size_t)(t0 / kTok) * Ep + e0 + 16 * m + n) * kTok + t0 % kTok + g * O::RL);
      load_x(j ^ 1, min(s + 1, hi - 1));
#pragma unroll
      for (int q = 0; q < O::CL; ++q) {
        const u32x4 f = column(x[j], q);
#pragma unroll
        for (int i = O::SP - 1; i >= 0; --i)
#pragma unroll
          for (int m = 0; m < MB; ++m) acc[m][q] = mma<TIn>(d[i][m], f, acc[m][q]);
      }
    }
  // lane l holds columns CL*(l%16) .. +CL-1 of experts 4*(l/16) .. +3 of each block
#pragma unroll
  for (int h = 0; h < MB / HALF; ++h) {
    __syncthreads();
#pragma unroll
    for (int m = 0; m < HALF; ++m)
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int q = 0; q < O::CL; q += 4)
          red[(((wave * HALF + m) * 16 + 4 * g + r) * COLS + n * O::CL + q) / 4] =
              f32x4{acc[h * HALF + m][q][r], acc[h * HALF + m][q + 1][r],
                    acc[h * HALF + m][q + 2][r], acc[h * HALF + m][q + 3][r]};
    __syncthreads();
    for (int i = threadIdx.x; i < HALF * 16 * COLS / 4; i += kWaves * 64) {
      f32x4 s = red[i];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) s += red[w * HALF * 16 * COLS / 4 + i];
      const int e = e0 + h * HALF * 16 + i / (COLS / 4), c = c0 + i % (COLS / 4) * 4;
      if (e < a.E && c < a.D)
        *reinterpret_cast<f32x4*>(out + ((size_t)split * a.E + e) * a.D + c) = s;
    }
  }
}

// The token groups' sums of dbias: a wave takes 16 experts, four lanes each every fourth group.
__device__ __forceinline__ void dbias_body(const float* __restrict__ db, int groups, int E,
                                           float* __restrict__ dbias, int wave) {
  const int lane = threadIdx.x & 63;
  const int e = wave * 16 + (lane & 15);
  float s = 0.0f;
  if (e < E)
#pragma unroll 8
    for (int r = lane >> 4; r < groups; r += 4) s += db[(size_t)r * E + e];
  s += __shfl_xor(s, 16);
  s += __shfl_xor(s, 32);
  if (e < E && lane < 16) dbias[e] = s;
}

// dwg, dx and dbias side by side in one launch: dwg reads x, dx writes (and reads dx_add), and
// neither waits for the other's last workgroups (8192 tokens over 64 experts, D = 2048: 41.5 us in
// all, as launches of their own 49.4; 16384 over 32, D = 4096: 85 against 109; 389 over 8, float32: 20.9
// against 25.9). STEPS: dx's steps of k, 0 for more than 64 experts.
template <typename TIn, int STEPS, int MB>
__global__ __launch_bounds__(kWaves * 64) void route_products_kernel(const RouteBwdCall a, Parts p,
                                                                     int Ep, int Tp, int strips,
                                                                     int chunks, int S, int per,
                                                                     int dwg, int dx,
                                                                     float* __restrict__ out) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int block = blockIdx.x;
  if (block < dwg) {
    dwg_body<TIn, MB>(a, p, Ep, Tp, strips, chunks, S, block, out);
  } else if (block < dwg + dx) {
    const int64_t id = (int64_t)(block - dwg) * kWaves + wave;
    if constexpr (STEPS > 0)
      dx_body<TIn, STEPS>(a, p, strips, per, id);
    else
      dx_wide_body<TIn>(a, p, Ep, strips, id);
  } else {
    dbias_body(p.dbias, Tp / kTok, a.E, a.dbias, (block - dwg - dx) * kWaves + wave);
  }
}

// The ranges' sums of dwg, in order.
__global__ __launch_bounds__(256) void route_sum_kernel(const f32x4* __restrict__ dwg, int S, int64_t n4,
                                                        f32x4* __restrict__ out) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n4) return;
  f32x4 s = dwg[i];
#pragma unroll 8
  for (int r = 1; r < S; ++r) s += dwg[r * n4 + i];
  out[i] = s;
}

struct Plan {
  int Ep, Tp, strips, MB, chunks, S;
  size_t rows, cols, dbias, dwg;   // bytes
};

template <typename TIn>
Plan plan(int T, int D, int E) {
  typedef Op<TIn> O;
  Plan p;
  p.Ep = E <= 32 ? 32 : (E + 63) / 64 * 64;
  p.Tp = (T + kTok - 1) / kTok * kTok;
  p.strips = (D + 16 * O::CL - 1) / (16 * O::CL);
  // of more than 64 experts 48 at a time where they pad them less than 64 (78 of float32: 94 us, 64 at
  // a time 117)
  p.MB = E <= 16 ? 1 : E <= 32 ? 2 : E > 64 && (E + 47) / 48 * 48 < (E + 63) / 64 * 64 ? 3 : 4;
  p.chunks = (E + 16 * p.MB - 1) / (16 * p.MB);
  // ranges of tokens: enough waves for the card, at least one step of k a wave
  const int steps = p.Tp / O::KS;
  const int want = O::DW / kWaves / (p.strips * p.chunks);
  p.S = std::max(1, std::min(want, steps / kWaves));
  if (T <= kShort) p.S = 1;   // no launch for the sums
  p.rows = (size_t)O::SX * T * p.Ep * sizeof(TIn);
  p.cols = (size_t)O::SP * p.Ep * p.Tp * sizeof(TIn);
  p.dbias = ((size_t)(p.Tp / kTok) * E * 4 + 15) / 16 * 16;
  p.dwg = p.S > 1 ? (size_t)p.S * E * D * 4 : 0;
  return p;
}

template <typename TIn>
hipError_t launch_typed(const RouteBwdCall& c, hipStream_t s) {
  const Plan p = plan<TIn>(c.T, c.D, c.E);
  char* at = static_cast<char*>(c.workspace);
  Parts w;
  w.rows = at;
  w.cols = at + p.rows;
  w.dbias = reinterpret_cast<float*>(at + p.rows + p.cols);
  w.dwg = reinterpret_cast<float*>(at + p.rows + p.cols + p.dbias);
  const int groups = p.Tp / kTok;
  const auto dl = c.E <= 64    ? route_dl_kernel<TIn, 1>
                  : c.E <= 128 ? route_dl_kernel<TIn, 2>
                               : (c.E <= 256 ? route_dl_kernel<TIn, 4> : route_dl_kernel<TIn, 16>);
  const int gx = std::min(groups, kMostX);
  hipLaunchKernelGGL(dl, dim3(gx, (groups + gx - 1) / gx), dim3(kDlWaves * 64), 0, s, c, w, p.Ep, p.Tp);
  const int blocks16 = (c.T + 15) / 16;
  const int per = std::max<int>(1, (int)(((int64_t)blocks16 * p.strips + kDxWaves - 1) / kDxWaves));
  const int64_t dxw = p.Ep <= 64 ? (int64_t)((blocks16 + per - 1) / per) * p.strips
                                 : (int64_t)((c.T + 63) / 64) * p.strips;
  const int dwg = c.dwg ? p.strips * p.chunks * p.S : 0;
  const int dx = c.dx ? (int)((dxw + kWaves - 1) / kWaves) : 0;
  const int db = c.dbias ? (c.E + 16 * kWaves - 1) / (16 * kWaves) : 0;
  constexpr int S32 = 32 / Op<TIn>::KS, S64 = 64 / Op<TIn>::KS;
  const auto products = c.E <= 16   ? route_products_kernel<TIn, S32, 1>
                        : c.E <= 32 ? route_products_kernel<TIn, S32, 2>
                        : c.E <= 64 ? route_products_kernel<TIn, S64, 4>
                                    : p.MB == 3 ? route_products_kernel<TIn, 0, 3>
                                    : route_products_kernel<TIn, 0, 4>;
  if (dwg + dx + db > 0)
    hipLaunchKernelGGL(products, dim3(dwg + dx + db), dim3(kWaves * 64), 0, s, c, w, p.Ep, p.Tp, p.strips,
                       p.chunks, p.S, per, dwg, dx, p.S > 1 ? w.dwg : c.dwg);
  if (c.dwg && p.S > 1) {
    const int64_t n4 = (int64_t)c.E * c.D / 4;
    hipLaunchKernelGGL(route_sum_kernel, dim3((unsigned)((n4 + 255) / 256)), dim3(256), 0, s,
                       reinterpret_cast<const f32x4*>(w.dwg), p.S, n4, reinterpret_cast<f32x4*>(c.dwg));
  }
  return hipGetLastError();
}

template <typename TIn>
size_t bytes_typed(int T, int D, int E) {
  const Plan p = plan<TIn>(T, D, E);
  return p.rows + p.cols + p.dbias + p.dwg;
}

}  // namespace

size_t route_bwd_workspace_bytes(int dt, int T, int D, int E) {
  return dt == kF32 ? bytes_typed<float>(T, D, E) : bytes_typed<bf16_t>(T, D, E);
}

hipError_t launch_route_backward(int dt, const RouteBwdCall& c, hipStream_t s) {
  return dt == kF32 ? launch_typed<float>(c, s) : launch_typed<bf16_t>(c, s);
}

}  // namespace moe
