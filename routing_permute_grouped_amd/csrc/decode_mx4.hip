// Grouped SwiGLU for decode with MXFP4 weights: bf16 rows in the masked layout's slabs
// against expert weights held as E2M1 codes (two a byte, the even k in the low half) with
// one E8M0 scale per 32 values, in k-step words. Per expert e and valid row:
//   h = silu(x w1^T) * (x w3^T) rounded to bf16, y = h w2^T, float32 sums.
// h is rounded once to bf16, its type as an output and as an operand of fc2's matrix
// instruction, as in the masked path with bf16 weights (y is then off by about 2.4e-3 of its size,
// with a float32 h by 1.7e-3).
//
// Bound by the stream of the active experts' weights, 17/32 byte a value, a quarter of the
// bf16 stream; per weight byte there is four times the work on the rows. Hence
//   * a work item is 64 output columns for up to 64 rows of one expert; a workgroup of four
//     waves takes one item after the other, each wave 16 of the columns: rows of w1 and of w3
//     (fc1: one row fragment feeds both), or of w2. Where such items are too few for the CUs,
//     an item is 32 columns, and two waves halve the k of 16;
//   * a lane loads 16 bytes of a weight row: one whole MX block, so one scale serves them.
//     Lane group g holds block g of a 128-value chunk, and its 8-code words are the four
//     MFMA slices; the rows' fragments follow the same order (any order of k serves that
//     both operands share). One load brings KS chunks' scale words to the four lane groups,
//     which exchange them by lane swaps: a byte load per chunk cost 12 to 15%;
//   * v_cvt_scalef32_pk_bf16_fp4 turns two codes and the block's scale into two bf16
//     values, exactly (one fraction bit, and a power of two), and v_mfma_f32_16x16x32_bf16
//     multiplies;
//   * rows come through LDS, KS chunks at a time, double-buffered through registers, one
//     barrier per KS chunks. A group's weights lie in registers and are refilled with the next
//     group's once they are multiplied. All loads are ordinary ones, so every wait is the
//     compiler's own;
//   * four workgroups a CU hide the latency; deeper prefetch at three or two was slower (64
//     experts of D = 2048, F = 1408, one row each: 57 us, at two workgroups and 16 chunks
//     ahead 94), and so was splitting k over all four waves (100 us);
//   * the items that exist are found on the device from the counts, so that experts without
//     rows and unused row groups cost no workgroup (one that looks up its count and leaves
//     holds its place for more than a microsecond: 20 of 87 us with half of them empty).
// Rows behind counts[e] are neither read nor written; an expert without rows reads nothing.
#include <algorithm>

#include "common.hpp"
#include "kernels.hpp"

namespace moe {
namespace {

constexpr int DW = 4;           // waves per workgroup
constexpr int GROUP = 64;       // rows of an item
constexpr int XBYTES = 32768;   // two row buffers: 16*NB rows of KS chunks (256 bytes) each
constexpr int XCDS = 8;

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2v __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// Eight codes and their block's scale as eight bf16 values.
__device__ __forceinline__ bf16x8 dequant8(uint32_t w, float scale) {
  const bf16x2v a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0);
  const bf16x2v b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1);
  const bf16x2v c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2);
  const bf16x2v d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3);
  return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

__device__ __forceinline__ void store4(bf16_t* p, float a, float b, float c, float d) {
  *reinterpret_cast<uint2*>(p) = uint2{pack_bf16x2(a, b), pack_bf16x2(c, d)};
}

// silu(a) * b; the sigmoid's reciprocal from the hardware's approximate reciprocal
// (about 1 ulp of float32, below the bf16 rounding of h)
__device__ __forceinline__ float silu_mul(float a, float b) {
  return a * __builtin_amdgcn_rcpf(1.0f + __expf(-a)) * b;
}

// This wave's LDS accesses are complete, then every wave of the workgroup meets; loads in
// flight keep flying.
__device__ __forceinline__ void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

struct Mx4Weights {
  const uint8_t* q1;    // [E][N][K/2]
  const uint8_t* q2;    // fc1: w3's; fc2: w2's again
  const uint32_t* s1;   // [K/128][E*N] words
  const uint32_t* s2;
};

// The scale words of KS chunks, held by the lane groups (group g: chunk g % KS), to byte g of
// each chunk's word as a power of two: the swaps put group pairs, then halves, side by side.
template <int KS>
__device__ __forceinline__ void spread(uint32_t word, int g, float (&scale)[KS]) {
  uint32_t w[4] = {word, word, word, word};
  if (KS == 4) {
    const auto h = __builtin_amdgcn_permlane32_swap(word, word, false, false);
    w[0] = (uint32_t)h[0];
    w[2] = (uint32_t)h[1];
  }
  if (KS >= 2) {
    const auto a = __builtin_amdgcn_permlane16_swap(w[0], w[0], false, false);
    w[0] = (uint32_t)a[0];
    w[1] = (uint32_t)a[1];
  }
  if (KS == 4) {
    const auto b = __builtin_amdgcn_permlane16_swap(w[2], w[2], false, false);
    w[2] = (uint32_t)b[0];
    w[3] = (uint32_t)b[1];
  }
#pragma unroll
  for (int i = 0; i < KS; ++i)
    scale[i] = __uint_as_float(__builtin_amdgcn_ubfe(w[i], 8 * g, 8) << 23);
}

// NB: row blocks of 16 of the item's rows; KS: 128-value chunks per LDS buffer, and of weights in
// flight; KW: waves that share 16 columns, each taking every KW-th chunk (the item is 64 / KW
// columns, and their sums are added in wave order). cols: the item's first column.
template <bool FC1, int NB, int KS, int KW>
__device__ __forceinline__ void dec4_body(char* xs, const bf16_t* __restrict__ X, int cols, int e,
                                          int r0, int rows, int K, int N, int E,
                                          const Mx4Weights& wt, bf16_t* __restrict__ out) {
  constexpr int NW = FC1 ? 2 : 1;                 // weight fragments a wave multiplies
  constexpr int ROWB = KS * 256;                  // bytes of a row's group of chunks
  constexpr int NX = NB * KS;                     // 16-byte units per thread and group
  constexpr int KC = KS / KW;                     // chunks of a group a wave takes
  static_assert(2 * NB * 16 * ROWB <= XBYTES, "two row buffers");
  // opaque per item, so that addresses derived from it are not kept across the items: with
  // six bodies in the item loop they would not fit the registers
  int tid = threadIdx.x;
  asm volatile("" : "+v"(tid));
  const int lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int fr = lane & 15, g = lane >> 4;
  const int kw = KW > 1 ? wave / (DW / KW) : 0;
  const int n0 = cols + wave % (DW / KW) * 16;
  const int nch = K / 128;
  const int ngr = (nch + KS - 1) / KS;

  // this lane's weight rows, and their scale words of the wave's chunk g % KC of a group
  const size_t row = (size_t)e * N + n0 + fr;
  const uint8_t* wrow[2] = {wt.q1 + row * (K / 2) + 16 * g, wt.q2 + row * (K / 2) + 16 * g};
  const uint32_t* srow[2] = {wt.s1 + row, wt.s2 + row};
  const size_t sstep = (size_t)E * N;
  u32x4 wr[NW][KC];
  uint32_t sr[NW];
  // past the last chunk of a group that K ends in, the last one again; its rows are zeros there
  auto wload = [&](int gr) {
#pragma unroll
    for (int i = 0; i < KC; ++i) {
      const int c = min(gr * KS + i * KW + kw, nch - 1);
#pragma unroll
      for (int w = 0; w < NW; ++w) wr[w][i] = ld16(wrow[w] + (size_t)c * 64);
    }
#pragma unroll
    for (int w = 0; w < NW; ++w)
      sr[w] = srow[w][min(gr * KS + g % KC * KW + kw, nch - 1) * sstep];
  };

  // unit q of a group: row q / (16*KS), 16-byte unit q % (16*KS) of the row's group
  u32x4 xr[NX];
  auto xload = [&](int gr) {
#pragma unroll
    for (int i = 0; i < NX; ++i) {
      const int q = tid + i * DW * 64;
      const int r = q / (16 * KS), u = q % (16 * KS);
      const int k0 = gr * (KS * 128) + u * 8;
      xr[i] = u32x4{0u, 0u, 0u, 0u};
      if (r < rows && k0 < K) xr[i] = ld16(X + (size_t)(r0 + r) * K + k0);
    }
  };
  // unit u of row r at u ^ (r % 16): the 16 rows of a quarter-wave's read hit distinct banks
  auto xstore = [&](int buf) {
#pragma unroll
    for (int i = 0; i < NX; ++i) {
      const int q = tid + i * DW * 64;
      const int r = q / (16 * KS), u = q % (16 * KS);
      st16(xs + buf * (XBYTES / 2) + r * ROWB + ((u ^ (r & 15)) << 4), xr[i]);
    }
  };

  f32x4 acc[NW][NB];
#pragma unroll
  for (int w = 0; w < NW; ++w)
#pragma unroll
    for (int b = 0; b < NB; ++b) acc[w][b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

  auto compute = [&](int buf) {
    const char* xb = xs + buf * (XBYTES / 2);
    float scale[NW][KC];
#pragma unroll
    for (int w = 0; w < NW; ++w) spread<KC>(sr[w], g, scale[w]);
#pragma unroll
    for (int i = 0; i < KC; ++i) {
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        bf16x8 wf[NW];
#pragma unroll
        for (int w = 0; w < NW; ++w) wf[w] = dequant8(wr[w][i][s], scale[w][i]);
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const int r = 16 * b + fr;
          const bf16x8 xf = __builtin_bit_cast(
              bf16x8, ld16(xb + r * ROWB + (i * KW + kw) * 256 + (((4 * g + s) ^ (r & 15)) << 4)));
#pragma unroll
          for (int w = 0; w < NW; ++w)
            acc[w][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf[w], xf, acc[w][b], 0, 0, 0);
        }
      }
    }
  };

  xload(0);
  wload(0);
  lds_barrier();   // the item before is done with the buffers
  xstore(0);
  xload(1);
  lds_barrier();
  for (int gr = 0; gr < ngr; ++gr) {
    compute(gr & 1);
    // the other buffer's readers passed the barrier that ended the step before
    xstore((gr + 1) & 1);
    xload(gr + 2);
    if (gr + 1 < ngr) wload(gr + 1);
    lds_barrier();
  }

  if (KW > 1) {   // every wave is past its last read of the row buffers
    f32x4* red = reinterpret_cast<f32x4*>(xs) + wave % (DW / KW) * ((KW - 1) * NW * NB * 64) + lane;
    if (kw > 0) {
#pragma unroll
      for (int w = 0; w < NW; ++w)
#pragma unroll
        for (int b = 0; b < NB; ++b) red[(((kw - 1) * NW + w) * NB + b) * 64] = acc[w][b];
    }
    lds_barrier();
    if (kw == 0) {
#pragma unroll
      for (int o = 0; o < KW - 1; ++o)
#pragma unroll
        for (int w = 0; w < NW; ++w)
#pragma unroll
          for (int b = 0; b < NB; ++b) acc[w][b] += red[((o * NW + w) * NB + b) * 64];
    }
    if (kw > 0) return;   // from this item; the next one begins with a barrier
  }
  // lane l holds row 16*b + l%16 and output columns 4*(l/16) .. +3 of its 16
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    const int r = 16 * b + fr;
    if (r < rows) {
      bf16_t* p = out + ((size_t)r0 + r) * N + n0 + 4 * g;
      const f32x4 &a = acc[0][b], &u = acc[NW - 1][b];
      if (FC1)
        store4(p, silu_mul(a[0], u[0]), silu_mul(a[1], u[1]), silu_mul(a[2], u[2]),
               silu_mul(a[3], u[3]));
      else
        store4(p, a[0], a[1], a[2], a[3]);
    }
  }
}

// Rows of expert e (none past the last expert), and their row groups of 64.
__device__ __forceinline__ int rows_of(const int32_t* counts, int e, int E, int cap) {
  return e < E ? max(0, min(counts[e], cap)) : 0;
}
__device__ __forceinline__ int groups_of(int rows) { return (rows + GROUP - 1) / GROUP; }

// Exclusive prefix sum over the wave; total: the whole sum.
__device__ __forceinline__ int wave_scan(int v, int& total) {
  const int lane = threadIdx.x & 63;
  int inc = v;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(inc, d);
    if (lane >= d) inc += o;
  }
  total = __builtin_amdgcn_readlane(inc, 63);
  return inc - v;
}

// The last lane whose prefix sum is not past v.
__device__ __forceinline__ int last_lane(int prefix, bool in, int v) {
  return 63 - __clzll(__ballot(in && prefix <= v));
}

// Every wave holds the row groups' prefix sums over the experts, `per` experts a lane, and
// numbers the items expert by expert: expert e, whose groups start at s, owns items
// [s, s + its groups) * ncols. Of one expert's items, the row groups of eight column blocks
// follow each other at a distance of eight, so those of one column block run on one XCD,
// close in time, and the second finds the weights in its L2.
template <bool FC1>
__global__ __launch_bounds__(DW * 64, 4) void dec4_kernel(const bf16_t* __restrict__ X,
                                                          const int32_t* __restrict__ counts,
                                                          int cap, int E, int K, int N,
                                                          int cus, Mx4Weights wt,
                                                          bf16_t* __restrict__ out) {
  __shared__ __attribute__((aligned(1024))) char xs[XBYTES];
  const int lane = threadIdx.x & 63;
  const int per = (E + 63) / 64;
  int sum = 0, groups, mine = 0;   // mine: rows of the lane's (last) expert
  bool tall = false;               // an expert with more than 32 rows
  for (int i = 0; i < per; ++i) {
    mine = rows_of(counts, lane * per + i, E, cap);
    sum += groups_of(mine);
    tall |= mine > 32;
  }
  const int start = wave_scan(sum, groups);
  // with at most one 64-column item a CU, two waves share 16 columns: twice the items, half
  // the chain of loads (one token over 6 of 64 experts 17.9 -> 15.9 us; at two items a CU, K =
  // 14336, 158 -> 179 us). Two LDS chunks of more than 32 rows would not fit.
  const bool halve = groups * (N / 64) <= cus && __ballot(tall) == 0;
  const int width0 = halve ? 32 : 64, ncols = N / width0;
  const int items = groups * ncols;
  for (int item = blockIdx.x; item < items; item += gridDim.x) {
    const int grp = item / ncols;
    int e = last_lane(start, true, grp);
    int s = __builtin_amdgcn_readlane(start, e);
    int n = __builtin_amdgcn_readlane(mine, e);
    if (per > 1) {   // the lane's experts, one a lane
      int all;
      const int c = lane < per ? rows_of(counts, e * per + lane, E, cap) : 0;
      const int at = wave_scan(groups_of(c), all);
      const int l = last_lane(at, lane < per, grp - s);
      s += __builtin_amdgcn_readlane(at, l);
      n = __builtin_amdgcn_readlane(c, l);
      e = e * per + l;
    }
    const int ng = groups_of(n);
    const int local = item - s * ncols;
    const int base = local / (XCDS * ng) * XCDS, in = local - base * ng;
    const int width = min(XCDS, ncols - base);
    const int first = in / width * GROUP, cols = (base + in % width) * width0;
    const int rows = min(n - first, GROUP), r0 = e * cap + first;
    if (rows <= 16 && halve)
      dec4_body<FC1, 1, 4, 2>(xs, X, cols, e, r0, rows, K, N, E, wt, out);
    else if (rows <= 16)
      dec4_body<FC1, 1, 4, 1>(xs, X, cols, e, r0, rows, K, N, E, wt, out);
    else if (rows <= 32 && halve)
      dec4_body<FC1, 2, 2, 2>(xs, X, cols, e, r0, rows, K, N, E, wt, out);
    else if (rows <= 32)
      dec4_body<FC1, 2, 2, 1>(xs, X, cols, e, r0, rows, K, N, E, wt, out);
    else if (rows <= 48)
      dec4_body<FC1, 3, 1, 1>(xs, X, cols, e, r0, rows, K, N, E, wt, out);
    else
      dec4_body<FC1, 4, 1, 1>(xs, X, cols, e, r0, rows, K, N, E, wt, out);
  }
}

template <bool FC1>
void launch_dec4(const void* X, const int32_t* counts, int cap, int E, int K, int N,
                 const Mx4Weights& wt, void* out, hipStream_t s) {
  const int64_t most = (int64_t)E * ((cap + GROUP - 1) / GROUP) * (N / 32);
  const int grid = (int)std::min<int64_t>(4 * cu_count(), most);
  hipLaunchKernelGGL(dec4_kernel<FC1>, dim3(grid), dim3(DW * 64), 0, s,
                     static_cast<const bf16_t*>(X), counts, cap, E, K, N, cu_count(), wt,
                     static_cast<bf16_t*>(out));
}

}  // namespace

hipError_t launch_decode_mx4(const void* x, const int32_t* counts, int E, int D, int F, int cap,
                             const void* w1q, const void* w1s, const void* w3q, const void* w3s,
                             const void* w2q, const void* w2s, void* h, void* y, hipStream_t s) {
  const auto q = [](const void* p) { return static_cast<const uint8_t*>(p); };
  const auto w = [](const void* p) { return static_cast<const uint32_t*>(p); };
  launch_dec4<true>(x, counts, cap, E, D, F, Mx4Weights{q(w1q), q(w3q), w(w1s), w(w3s)}, h, s);
  launch_dec4<false>(h, counts, cap, E, F, D, Mx4Weights{q(w2q), q(w2q), w(w2s), w(w2s)}, y, s);
  return hipGetLastError();
}

}  // namespace moe
