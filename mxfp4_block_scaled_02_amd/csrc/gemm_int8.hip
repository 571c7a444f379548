// gemm_a8w8: C[m, n] = T(acc * a_s[m] * b_s[n] (+ bias[n])), acc the exact int32
// sum over k of Aq[m, k] * Bq[n, k] on the integer matrix instructions.
//
// The order of k inside a matrix instruction is free as long as both operands
// use the same one. For the 16x16x64 instruction lane l supplies 16 bytes of row
// l%16; here two instructions cover a 128-byte step, lane l loading the 32
// contiguous bytes k = 32*(l/16) .. +31 of its row, so that a row's 128-byte line
// is used whole by one pair of loads.
// Result: lane l, register r = D[4*(l/16) + r][l%16], row = first operand's.
#include "host_common.hpp"
#include "mx_device.hpp"

#pragma clang fp contract(off)

namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v16i __attribute__((ext_vector_type(16)));

struct GemmArgs {
  const uint8_t* A;
  int64_t lda;
  const float* as;
  const uint8_t* B;
  int64_t ldb;
  const float* bs;
  const void* bias;
  void* C;
  int64_t ldc;
  int M, N, K;
  int ctype;
};

constexpr int kOut = 0x7fffffff;  // an offset past every window: reads zeros

__device__ __forceinline__ __amdgpu_buffer_rsrc_t window(const uint8_t* base, int64_t rows, int64_t ld, int K) {
  const int64_t n = (rows - 1) * ld + K;  // < 2^31 by the host's check of ld
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(base), (short)0, (int)n, 0x00020000);
}
__device__ __forceinline__ v4i load16(__amdgpu_buffer_rsrc_t r, int voff, int soff) {
  return __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(r, voff, soff, 0));
}

__device__ __forceinline__ float bias_at(const GemmArgs& p, int n) {
  if (p.ctype == MXFP4_TYPE_F32) return ((const float*)p.bias)[n];
  const uint16_t b = ((const uint16_t*)p.bias)[n];
  if (p.ctype == MXFP4_TYPE_BF16) return __builtin_bit_cast(float, (uint32_t)b << 16);
  return (float)__builtin_bit_cast(_Float16, b);
}
__device__ __forceinline__ void store_one(const GemmArgs& p, int64_t m, int n, float v) {
  const int64_t at = m * p.ldc + n;
  if (p.ctype == MXFP4_TYPE_F32)
    ((float*)p.C)[at] = v;
  else if (p.ctype == MXFP4_TYPE_BF16)
    ((uint16_t*)p.C)[at] = mx::f32_to_bf16(v);
  else
    ((_Float16*)p.C)[at] = (_Float16)v;
}

// A workgroup owns 16*MT rows x 16*NT columns of C; its W waves take contiguous
// shares of K, load their operands straight into registers, and add their
// integer sums into one tile in LDS (integer sums: their order does not matter).
template <int MT, int NT, int W>
__global__ __launch_bounds__(64 * W) void gemm_direct_kernel(GemmArgs p) {
  constexpr int MS = 16 * MT, NS = 16 * NT;
  __shared__ int tile[MS * NS];
  const int l = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int mt = (p.M + MS - 1) / MS;
  const int m0 = (int)(blockIdx.x % (unsigned)mt) * MS, n0 = (int)(blockIdx.x / (unsigned)mt) * NS;
  const int rows = min(MS, p.M - m0), cols = min(NS, p.N - n0);
  for (int i = threadIdx.x; i < MS * NS; i += 64 * W) tile[i] = 0;
  const __amdgpu_buffer_rsrc_t ar = window(p.A + (int64_t)m0 * p.lda, rows, p.lda, p.K);
  const __amdgpu_buffer_rsrc_t br = window(p.B + (int64_t)n0 * p.ldb, cols, p.ldb, p.K);
  const int steps = (p.K + 127) / 128;
  const int s0 = (int)((int64_t)steps * wave / W), s1 = (int)((int64_t)steps * (wave + 1) / W);
  v4i acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = v4i{0, 0, 0, 0};
  for (int s = s0; s < s1; ++s) {
    const int k = 128 * s + 32 * (l >> 4);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const bool in = k + 16 * h < p.K;  // past K both operands read zeros
      v4i a[MT], b[NT];
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        const int r = 16 * i + (l & 15);
        a[i] = load16(ar, in && r < rows ? (int)(r * p.lda) + k + 16 * h : kOut, 0);
      }
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const int r = 16 * j + (l & 15);
        b[j] = load16(br, in && r < cols ? (int)(r * p.ldb) + k + 16 * h : kOut, 0);
      }
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a[i], b[j], acc[i][j], 0, 0, 0);
    }
  }
  __syncthreads();  // the tile's zeros
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        atomicAdd(&tile[(16 * i + 4 * (l >> 4) + r) * NS + 16 * j + (l & 15)], acc[i][j][r]);
  __syncthreads();
  for (int i = threadIdx.x; i < MS * NS; i += 64 * W) {
    const int m = i / NS, n = i % NS;
    if (m < rows && n < cols) {
      float v = (float)tile[i] * p.as[m0 + m] * p.bs[n0 + n];
      if (p.bias) v = v + bias_at(p, n0 + n);
      store_one(p, m0 + m, n0 + n, v);
    }
  }
}

template <int MT, int NT, int W>
hipError_t launch_direct(GemmArgs& p, hipStream_t st) {
  const int64_t grid = mxh::cdiv(p.M, 16 * MT) * mxh::cdiv(p.N, 16 * NT);
  void* args[] = {&p};
  return hipLaunchKernel((const void*)gemm_direct_kernel<MT, NT, W>, dim3((unsigned)grid), dim3(64 * W), args, 0, st);
}

constexpr int64_t kMaxStride = (int64_t)1 << 22;  // 256 rows of a window stay below 2^31 bytes
constexpr int64_t kMaxK = 131056;                 // 128 * 128 * K < 2^31

}  // namespace

extern "C" int gemm_a8w8(const void* Aq, int64_t lda, const float* as, const void* Bq, int64_t ldb, const float* bs,
                         const void* bias, void* C, int64_t ldc, int ctype, int64_t M, int64_t N, int64_t K,
                         void* stream) {
  if (M < 1 || N < 1 || K < 1) return MXFP4_ERR_SHAPE;  // first: an empty tensor's pointer may be NULL
  if (!Aq || !as || !Bq || !bs || !C) return MXFP4_ERR_NULL;
  if (ctype != MXFP4_TYPE_BF16 && ctype != MXFP4_TYPE_F16 && ctype != MXFP4_TYPE_F32) return MXFP4_ERR_ARG;
  if (K < 16 || K % 16 != 0 || K > kMaxK) return MXFP4_ERR_SHAPE;
  if (M > ((int64_t)1 << 24) || N > ((int64_t)1 << 24) || mxh::cdiv(M, 16) * mxh::cdiv(N, 16) > ((int64_t)1 << 30))
    return MXFP4_ERR_SHAPE;
  if (lda < K || lda > kMaxStride || ldb < K || ldb > kMaxStride || ldc < N || ldc > ((int64_t)1 << 36))
    return MXFP4_ERR_SHAPE;
  const int64_t size = ctype == MXFP4_TYPE_F32 ? 4 : 2;
  if (!mxh::aligned(Aq, 16) || lda % 16 != 0 || !mxh::aligned(Bq, 16) || ldb % 16 != 0 || !mxh::aligned(as, 4) ||
      !mxh::aligned(bs, 4) || !mxh::aligned(C, (uintptr_t)size) || (bias && !mxh::aligned(bias, (uintptr_t)size)))
    return MXFP4_ERR_ALIGN;
  GemmArgs p{(const uint8_t*)Aq, lda, as, (const uint8_t*)Bq, ldb, bs, bias, C, ldc, (int)M, (int)N, (int)K, ctype};
  const hipStream_t st = (hipStream_t)stream;
  if (M <= 16) return mxh::launch_status(launch_direct<1, 1, 16>(p, st));
  if (M <= 32) return mxh::launch_status(launch_direct<2, 1, 16>(p, st));
  return mxh::launch_status(launch_direct<4, 4, 4>(p, st));
}
