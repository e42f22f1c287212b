// MXFP4 quantisation of rows, and the values of MXFP4 and MXFP8 rows.
//
// Every 32 consecutive values of a row share a power of two 2^X, stored as the byte X + 127
// (E8M0). MXFP4: X is the smallest integer >= -127 with max|v| <= 6 * 2^X (6 is the largest
// E2M1 value), so nothing saturates; with max|v| = 1.f * 2^e that is e - 2, or e - 1 when
// 1.f > 1.5, read off the float's bits. Each value becomes the E2M1 code of v / 2^X, to
// nearest, ties to the even code, by the hardware's scaled conversion; sign kept, -0
// included; two codes a byte, the even element in the low half. A block that holds an
// infinity or a NaN has no scale: its byte is 255 (E8M0's NaN) and its codes are zero, and
// every reader gives NaN for it.
//
// Scales go row by row ([R, C/32] bytes) or in the products' k-step words ([C/128][R] words,
// byte j of word (s, r) for block 4*s + j of row r).
//
// Bound by HBM: 2 or 4 bytes in and 17/32 out a value (and the reverse). A block is four
// neighbouring lanes of 8 values, so a wave reads and writes whole lines; the four lanes
// share the block's maximum by two lane swaps. The values to quantise are read past the
// caches: they are not needed again, and what the kernel before left in the caches then is
// not written back against the reads (69632 x 2048 bf16 to k-step words and back: 168 -> 129
// us, 5.6 TB/s; 1 GiB copies run at 5.0).
#include <algorithm>

#include "common.hpp"
#include "kernels.hpp"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 2;   // groups of 8 values a thread has in flight (4: 7.2 us for 6.0 on 64 x 4096)

typedef __bf16 bf16x2v __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

// max over the four lanes of a quad
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, true));   // xor 1
  return max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, true));   // xor 2
}

// 8 values of type T, their largest magnitude as float bits, and their codes.
template <typename T> struct Eight;
template <> struct Eight<bf16_t> {
  u32x4 a;
  __device__ void load(const bf16_t* p) { a = ld16_nt(p); }
  __device__ void zero() { a = u32x4{0u, 0u, 0u, 0u}; }
  __device__ uint32_t amax() const {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = max(m, max(a[i] & 0x7fffu, (a[i] >> 16) & 0x7fffu));
    return m << 16;
  }
  __device__ uint32_t codes(float scale) const {
    uint32_t w = 0;
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2v, (uint32_t)a[0]), scale, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2v, (uint32_t)a[1]), scale, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2v, (uint32_t)a[2]), scale, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2v, (uint32_t)a[3]), scale, 3);
    return w;
  }
};
template <> struct Eight<float> {
  u32x4 a, b;
  __device__ void load(const float* p) {
    a = ld16_nt(p);
    b = ld16_nt(p + 4);
  }
  __device__ void zero() { a = b = u32x4{0u, 0u, 0u, 0u}; }
  __device__ uint32_t amax() const {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = max(m, max(a[i] & 0x7fffffffu, b[i] & 0x7fffffffu));
    return m;
  }
  __device__ uint32_t codes(float scale) const {
    auto f = [](uint32_t u) { return __uint_as_float(u); };
    uint32_t w = 0;
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f(a[0]), f(a[1]), scale, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f(a[2]), f(a[3]), scale, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f(b[0]), f(b[1]), scale, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f(b[2]), f(b[3]), scale, 3);
    return w;
  }
};

// The E8M0 byte of a block whose largest magnitude has the float bits u.
__device__ __forceinline__ uint32_t mx4_scale_byte(uint32_t u) {
  const int e = (int)(u >> 23);
  if (e == 255) return 255u;
  return (uint32_t)max(0, e - 2 + ((u & 0x7fffffu) > 0x400000u ? 1 : 0));
}

// Where group i of this thread's work item lies: its row and its first column (a multiple of
// 8), or row -1. In rows, an item is kThreads * kUnroll consecutive groups of the matrix; in
// k-step words it is 32 rows of one 128-column step, 8 rows a wave, so that the words an
// item writes are 128 consecutive bytes.
template <bool KSTEPS>
__device__ __forceinline__ bool place(int64_t item, int i, int64_t R, int C, int64_t& row, int& col) {
  const int t = threadIdx.x;
  if (KSTEPS) {
    const int steps = C / 128;
    const int64_t tile = item / steps;
    row = tile * 32 + (t >> 6) * 8 + i * 4 + ((t & 63) >> 4);
    col = (int)(item - tile * steps) * 128 + (t & 15) * 8;
    return row < R;
  }
  const int per = C / 8;
  const int64_t q = (item * kUnroll + i) * kThreads + t;
  row = q / per;
  col = (int)(q - row * per) * 8;
  return row < R;
}

template <typename T, bool KSTEPS>
__global__ __launch_bounds__(kThreads) void quantize_mx4_kernel(const T* __restrict__ x,
                                                               int64_t items, int64_t R, int C,
                                                               uint8_t* __restrict__ q,
                                                               uint8_t* __restrict__ scales) {
  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    Eight<T> v[kUnroll];
    int64_t row[kUnroll];
    int col[kUnroll];
    bool in[kUnroll];
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      in[i] = place<KSTEPS>(item, i, R, C, row[i], col[i]);
      v[i].zero();
      if (in[i]) v[i].load(x + row[i] * C + col[i]);
    }
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const uint32_t sb = mx4_scale_byte(quad_max(v[i].amax()));
      const uint32_t w = sb == 255u ? 0u : v[i].codes(__uint_as_float(sb << 23));
      if (KSTEPS) {
        // the four blocks of a row's 128 columns are the 16 lanes of a DPP row: each puts its
        // byte in place and the lanes gather the word
        uint32_t word = sb << (8 * ((threadIdx.x >> 2) & 3));
        word |= (uint32_t)__shfl_xor((int)word, 4);
        word |= (uint32_t)__shfl_xor((int)word, 8);
        if (in[i] && (threadIdx.x & 15) == 0)
          reinterpret_cast<uint32_t*>(scales)[(int64_t)(col[i] / 128) * R + row[i]] = word;
      } else if (in[i] && (threadIdx.x & 3) == 0) {
        scales[row[i] * (C / 32) + col[i] / 32] = (uint8_t)sb;
      }
      if (in[i]) *reinterpret_cast<uint32_t*>(q + (row[i] * C + col[i]) / 2) = w;
    }
  }
}

template <typename T>
__device__ __forceinline__ void store8(T* p, const float* v);
template <>
__device__ __forceinline__ void store8<bf16_t>(bf16_t* p, const float* v) {
  st16(p, Chunk<bf16_t>::narrow(v));
}
template <>
__device__ __forceinline__ void store8<float>(float* p, const float* v) {
  st16(p, Chunk<float>::narrow(v));
  st16(p + 4, Chunk<float>::narrow(v + 4));
}

// FP4: packed E2M1 codes, else E4M3 bytes. Values are exact in float32 where float32 holds
// them (the largest scales overflow to infinity, as the value does); bf16 rounds them once,
// which only values below 2^-126 notice.
template <typename T, bool FP4, bool KSTEPS>
__global__ __launch_bounds__(kThreads) void dequantize_mx_kernel(const uint8_t* __restrict__ q,
                                                                const uint8_t* __restrict__ scales,
                                                                int64_t items, int64_t R, int C,
                                                                T* __restrict__ out) {
  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    uint2 w[kUnroll];
    uint32_t sb[kUnroll];
    int64_t at[kUnroll];
    bool in[kUnroll];
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      int64_t row;
      int col;
      in[i] = place<KSTEPS>(item, i, R, C, row, col);
      at[i] = row * C + col;
      w[i] = uint2{0u, 0u};
      sb[i] = 0u;
      if (in[i]) {
        if (FP4) w[i].x = *reinterpret_cast<const uint32_t*>(q + at[i] / 2);
        else w[i] = *reinterpret_cast<const uint2*>(q + at[i]);
        sb[i] = KSTEPS ? scales[((int64_t)(col / 128) * R + row) * 4 + ((col >> 5) & 3)]
                       : scales[row * (C / 32) + col / 32];
      }
    }
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const float s = __uint_as_float(sb[i] == 255u ? 0x7fc00000u : sb[i] << 23);
      f32x2 p0, p1, p2, p3;
      if (FP4) {
        p0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[i].x, s, 0);
        p1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[i].x, s, 1);
        p2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[i].x, s, 2);
        p3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[i].x, s, 3);
      } else {
        p0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w[i].x, s, false);
        p1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w[i].x, s, true);
        p2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w[i].y, s, false);
        p3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w[i].y, s, true);
      }
      const float v[8] = {p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
      if (in[i]) store8<T>(out + at[i], v);
    }
  }
}

int64_t work_items(int64_t R, int C, bool ksteps) {
  return ksteps ? (R + 31) / 32 * (C / 128)
                : (R * (C / 8) + kThreads * kUnroll - 1) / (kThreads * kUnroll);
}

int grid_for(int64_t items) { return (int)std::min<int64_t>(64 * cu_count(), items); }

template <typename T, bool FP4>
void launch_dequant_t(const void* q, const void* scales, int64_t R, int C, bool ksteps, void* out,
                      hipStream_t s) {
  const int64_t items = work_items(R, C, ksteps);
  const auto kern = ksteps ? dequantize_mx_kernel<T, FP4, true> : dequantize_mx_kernel<T, FP4, false>;
  hipLaunchKernelGGL(kern, dim3(grid_for(items)), dim3(kThreads), 0, s,
                     static_cast<const uint8_t*>(q), static_cast<const uint8_t*>(scales), items, R,
                     C, static_cast<T*>(out));
}

template <typename T>
void launch_quant_t(const void* x, int64_t R, int C, void* q, void* scales, bool ksteps,
                    hipStream_t s) {
  const int64_t items = work_items(R, C, ksteps);
  const auto kern = ksteps ? quantize_mx4_kernel<T, true> : quantize_mx4_kernel<T, false>;
  hipLaunchKernelGGL(kern, dim3(grid_for(items)), dim3(kThreads), 0, s, static_cast<const T*>(x),
                     items, R, C, static_cast<uint8_t*>(q), static_cast<uint8_t*>(scales));
}

}  // namespace

hipError_t launch_quantize_mx4(int dt, const void* x, int64_t R, int C, void* q, void* scales,
                               bool ksteps, hipStream_t s) {
  if (dt == kF32) launch_quant_t<float>(x, R, C, q, scales, ksteps, s);
  else launch_quant_t<bf16_t>(x, R, C, q, scales, ksteps, s);
  return hipGetLastError();
}

hipError_t launch_dequantize_mx(int dt, bool fp4, const void* q, const void* scales, int64_t R,
                                int C, bool ksteps, void* out, hipStream_t s) {
  if (dt == kF32)
    fp4 ? launch_dequant_t<float, true>(q, scales, R, C, ksteps, out, s)
        : launch_dequant_t<float, false>(q, scales, R, C, ksteps, out, s);
  else
    fp4 ? launch_dequant_t<bf16_t, true>(q, scales, R, C, ksteps, out, s)
        : launch_dequant_t<bf16_t, false>(q, scales, R, C, ksteps, out, s);
  return hipGetLastError();
}

}  // namespace moe
