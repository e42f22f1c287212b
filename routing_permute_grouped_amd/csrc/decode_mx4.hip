// Grouped SwiGLU for decode with MXFP4 weights: bf16 rows in the masked layout's slabs
// against expert weights held as E2M1 codes (two a byte, the even k in the low half) with
// one E8M0 scale per 32 values, in k-step words. Per expert e and valid row:
//   h = silu(x w1^T) * (x w3^T) rounded to bf16, y = h w2^T, float32 sums.
//
// Bound by the stream of the active experts' weights, 17/32 byte a value, a quarter of the
// bf16 stream; per weight byte there is four times the work on the rows. Hence
//   * a workgroup (4 waves) takes one expert; every row fragment read from LDS feeds two
//     weight fragments: 16 columns of w1 and of w3 (fc1), or 32 columns of w2 (fc2);
//   * a lane loads 16 bytes of a weight row: one whole MX block, so one scale serves them.
//     Lane group g holds block g of a 128-value chunk, and its 8-code words are the four
//     MFMA slices; the rows' fragments follow the same order (any order of k serves that
//     both operands share);
//   * v_cvt_scalef32_pk_bf16_fp4 turns two codes and the block's scale into two bf16
//     values, exactly (one fraction bit, and a power of two), and v_mfma_f32_16x16x32_bf16
//     multiplies;
//   * rows come through LDS, KS chunks at a time, double-buffered through registers, one
//     barrier per KS chunks; weights run PD groups ahead in registers. All loads are
//     ordinary ones, so every wait is the compiler's own.
// Rows behind counts[e] are neither read nor written; an expert without rows reads nothing.
#include <algorithm>

#include "common.hpp"
#include "kernels.hpp"

namespace moe {
namespace {

constexpr int DW = 4;   // waves per workgroup

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
  const uint8_t* s1;    // [K/128][E*N] words, as bytes
  const uint8_t* s2;
};

// NB: row blocks of 16 of this workgroup's rows; KS: 128-value chunks per LDS buffer;
// PD: groups of KS weight chunks in flight.
template <bool FC1, int NB, int KS, int PD>
__device__ __forceinline__ void dec4_body(char* xs, int xbytes, const bf16_t* __restrict__ X,
                                          int e, int r0, int rows, int K, int N, int E,
                                          const Mx4Weights& wt, bf16_t* __restrict__ out) {
  constexpr int ROWB = KS * 256;                  // bytes of a row's group of chunks
  constexpr int NX = NB * KS;                     // 16-byte units per thread and group
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int fr = lane & 15, g = lane >> 4;
  const int n0 = (blockIdx.x * DW + wave) * (FC1 ? 16 : 32);
  const int nch = K / 128;
  const int ngr = (nch + KS - 1) / KS;

  // this lane's two weight rows and their scale bytes (byte g of a chunk's word)
  const size_t row1 = (size_t)e * N + n0 + fr, row2 = FC1 ? row1 : row1 + 16;
  const uint8_t* wrow[2] = {wt.q1 + row1 * (K / 2) + 16 * g,
                            (FC1 ? wt.q2 : wt.q1) + row2 * (K / 2) + 16 * g};
  const uint8_t* srow[2] = {wt.s1 + row1 * 4 + g, (FC1 ? wt.s2 : wt.s1) + row2 * 4 + g};
  const size_t sstep = (size_t)E * N * 4;
  u32x4 wr[PD][2][KS];
  uint32_t sr[PD][2][KS];
  // past the last chunk the last one is read again; its rows are zeros there
  auto wload = [&](int slot, int gr) {
#pragma unroll
    for (int i = 0; i < KS; ++i) {
      const int c = min(gr * KS + i, nch - 1);
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        wr[slot][w][i] = ld16(wrow[w] + (size_t)c * 64);
        sr[slot][w][i] = srow[w][c * sstep];
      }
    }
  };

  // unit q of a group: row q / (16*KS), 16-byte unit q % (16*KS) of the row's group
  u32x4 xr[NX];
  auto xload = [&](int gr) {
#pragma unroll
    for (int i = 0; i < NX; ++i) {
      const int q = threadIdx.x + i * DW * 64;
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
      const int q = threadIdx.x + i * DW * 64;
      const int r = q / (16 * KS), u = q % (16 * KS);
      st16(xs + buf * xbytes + r * ROWB + ((u ^ (r & 15)) << 4), xr[i]);
    }
  };

  f32x4 acc[2][NB];
#pragma unroll
  for (int w = 0; w < 2; ++w)
#pragma unroll
    for (int b = 0; b < NB; ++b) acc[w][b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

  auto compute = [&](int buf, int slot) {
    const char* xb = xs + buf * xbytes;
#pragma unroll
    for (int i = 0; i < KS; ++i) {
      float sc[2];
#pragma unroll
      for (int w = 0; w < 2; ++w) sc[w] = __uint_as_float(sr[slot][w][i] << 23);
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        bf16x8 wf[2];
#pragma unroll
        for (int w = 0; w < 2; ++w) wf[w] = dequant8(wr[slot][w][i][s], sc[w]);
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const int r = 16 * b + fr;
          const bf16x8 xf = __builtin_bit_cast(
              bf16x8, ld16(xb + r * ROWB + i * 256 + (((4 * g + s) ^ (r & 15)) << 4)));
#pragma unroll
          for (int w = 0; w < 2; ++w)
            acc[w][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf[w], xf, acc[w][b], 0, 0, 0);
        }
      }
    }
  };

  xload(0);
#pragma unroll
  for (int p = 0; p < PD; ++p) wload(p, p);
  xstore(0);
  xload(1);
  lds_barrier();
  for (int g0 = 0; g0 < ngr; g0 += PD) {
#pragma unroll
    for (int j = 0; j < PD; ++j) {
      const int gr = g0 + j;
      if (gr < ngr) {
        compute(gr & 1, j);
        // the other buffer's readers passed the barrier that ended the step before
        xstore((gr + 1) & 1);
        xload(gr + 2);
        wload(j, gr + PD);
        lds_barrier();
      }
    }
  }

  // lane l holds row 16*b + l%16 and output columns 4*(l/16) .. +3 of its 16
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    const int r = 16 * b + fr;
    if (r < rows) {
      bf16_t* p = out + ((size_t)r0 + r) * N + n0 + 4 * g;
      const f32x4 &a = acc[0][b], &u = acc[1][b];
      if (FC1) {
        store4(p, silu_mul(a[0], u[0]), silu_mul(a[1], u[1]), silu_mul(a[2], u[2]),
               silu_mul(a[3], u[3]));
      } else {
        store4(p, a[0], a[1], a[2], a[3]);
        store4(p + 16, u[0], u[1], u[2], u[3]);
      }
    }
  }
}

// One workgroup per (64 fc1 or 128 fc2 columns, expert, 16*TB of its rows). The body is
// chosen by the rows that are there.
template <bool FC1, int TB, int KS, int PD>
__global__ __launch_bounds__(DW * 64) void dec4_kernel(const bf16_t* __restrict__ X,
                                                       const int32_t* __restrict__ counts,
                                                       int cap, int K, int N, Mx4Weights wt,
                                                       bf16_t* __restrict__ out) {
  constexpr int XBYTES = TB * 16 * KS * 256;
  __shared__ __attribute__((aligned(1024))) char xs[2 * XBYTES];
  const int e = blockIdx.y;
  const int first = blockIdx.z * (16 * TB);
  const int rows = min(max(0, min(counts[e], cap)) - first, 16 * TB);
  if (rows <= 0) return;   // uniform over the workgroup: the weights stay unread
  const int r0 = e * cap + first;
#define DEC4_CASE(n)                                                                          \
  case n:                                                                                     \
    if (TB >= n)                                                                              \
      dec4_body<FC1, (TB >= n ? n : 1), KS, PD>(xs, XBYTES, X, e, r0, rows, K, N, gridDim.y,  \
                                                wt, out);                                     \
    break;
  switch ((rows + 15) >> 4) {
    DEC4_CASE(1)
    DEC4_CASE(2)
    DEC4_CASE(3)
    DEC4_CASE(4)
    DEC4_CASE(5)
    DEC4_CASE(6)
    DEC4_CASE(7)
    default:
      if (TB >= 8)
        dec4_body<FC1, (TB >= 8 ? 8 : 1), KS, PD>(xs, XBYTES, X, e, r0, rows, K, N, gridDim.y,
                                                  wt, out);
      break;
  }
#undef DEC4_CASE
}

template <bool FC1>
void launch_dec4(const void* X, const int32_t* counts, int cap, int E, int K, int N,
                 const Mx4Weights& wt, void* out, hipStream_t s) {
  const int cols = FC1 ? 64 : 128;
  const bf16_t* x = static_cast<const bf16_t*>(X);
  bf16_t* o = static_cast<bf16_t*>(out);
  const auto go = [&](auto kern, int tb) {
    const dim3 grid(N / cols, E, (cap + 16 * tb - 1) / (16 * tb));
    hipLaunchKernelGGL(kern, grid, dim3(DW * 64), 0, s, x, counts, cap, K, N, wt, o);
  };
  if (cap <= 16)
    go(dec4_kernel<FC1, 1, 4, 2>, 1);
  else if (cap <= 32)
    go(dec4_kernel<FC1, 2, 4, 2>, 2);
  else if (cap <= 64)
    go(dec4_kernel<FC1, 4, 2, 2>, 4);
  else
    go(dec4_kernel<FC1, 8, 2, 2>, 8);
}

}  // namespace

hipError_t launch_decode_mx4(const void* x, const int32_t* counts, int E, int D, int F, int cap,
                             const void* w1q, const void* w1s, const void* w3q, const void* w3s,
                             const void* w2q, const void* w2s, void* h, void* y, hipStream_t s) {
  const auto b = [](const void* p) { return static_cast<const uint8_t*>(p); };
  launch_dec4<true>(x, counts, cap, E, D, F, Mx4Weights{b(w1q), b(w3q), b(w1s), b(w3s)}, h, s);
  launch_dec4<false>(h, counts, cap, E, F, D, Mx4Weights{b(w2q), b(w2q), b(w2s), b(w2s)}, y, s);
  return hipGetLastError();
}

}  // namespace moe
