// lora_add: y[t] += scale * (x[t] . A^T) . B^T with the adapter (A, B) of each row, for
// low-rank adapters of many requests beside a shared projection.
//
// Two launches. shrink: 16 rows and a share of K to a workgroup, x . A^T in fp32 partial
// sums [split][T][R]. expand: 16 rows and 256 columns to a workgroup, which adds the
// partial sums in their order, holds them as 16-bit pieces and multiplies with B.
// A tile's rows may have any adapters: each distinct one is multiplied with all 16 rows,
// and a row keeps the result of its own. (Selection, not masking with zeros: an adapter
// that is not finite stays with its rows.)
#include "host_common.hpp"
#include "mx_device.hpp"

namespace {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef u32x4 u32x4_at4 __attribute__((aligned(4)));
typedef u32x4 u32x4_at2 __attribute__((aligned(2)));

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
constexpr int kCols = 64 * kWaves;  // columns of y to a workgroup of expand

struct LoraArgs {
  uint8_t* y;
  int64_t ldy;  // elements
  const uint8_t* x;
  int64_t ldx;  // bytes
  const uint8_t* a;
  const uint8_t* b;
  const int32_t* index;
  const float* scale;
  float* part;
  int T, N, K, R, n, splits;
};

// The 16-bit types' matrix instruction and conversions.
template <int DT>
struct Half;
template <>
struct Half<MXFP4_TYPE_BF16> {
  typedef v8bf V;
  static __device__ __forceinline__ mx::v4f mfma(V a, V b, mx::v4f c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
  static __device__ __forceinline__ __bf16 round(float f) { return (__bf16)f; }
};
template <>
struct Half<MXFP4_TYPE_F16> {
  typedef v8h V;
  static __device__ __forceinline__ mx::v4f mfma(V a, V b, mx::v4f c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
  }
  static __device__ __forceinline__ _Float16 round(float f) { return (_Float16)f; }
};

// The adapter of lane l's row (row0 + l % 16), -1 without one.
__device__ __forceinline__ int adapter_of(const LoraArgs& a, int row0) {
  const int row = row0 + (threadIdx.x & 15);
  const int i = row < a.T ? a.index[row] : -1;
  return (uint32_t)i < (uint32_t)a.n ? i : -1;
}

template <int DT, int RT>
__global__ __launch_bounds__(kThreads) void shrink_kernel(LoraArgs a) {
  typedef typename Half<DT>::V V;
  __shared__ __align__(16) mx::v4f red[kWaves][RT][64];
  const int tid = threadIdx.x, l = tid & 63, c = l & 15, g = l >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int row0 = 16 * blockIdx.x, q = blockIdx.y;
  const int idx = adapter_of(a, row0);
  const uint64_t some = __ballot(idx >= 0) & 0xffffu;
  if (some == 0) return;  // the same on every wave
  const int steps = (a.K + 31) / 32;
  const int begin = (int)((int64_t)steps * q / a.splits), end = (int)((int64_t)steps * (q + 1) / a.splits);
  const uint8_t* xr = a.x + (int64_t)min(row0 + c, a.T - 1) * a.ldx;
  mx::v4f keep[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) keep[r] = mx::v4f{0.f, 0.f, 0.f, 0.f};
  for (uint64_t todo = some; todo != 0;) {
    const int i = __builtin_amdgcn_readlane(idx, __ffsll((unsigned long long)todo) - 1);
    const bool mine = idx == i;
    todo &= ~__ballot(mine);
    const uint8_t* ar[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) ar[r] = a.a + ((int64_t)i * a.R + min(16 * r + c, a.R - 1)) * a.K * 2;
    mx::v4f acc[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) acc[r] = mx::v4f{0.f, 0.f, 0.f, 0.f};
    for (int s = begin + wave; s < end; s += kWaves) {
      const int k = 32 * s + 8 * g;
      const bool in = k < a.K;  // K % 8 == 0: a piece is wholly inside or outside
      const int64_t at = in ? 2 * (int64_t)k : 0;
      V xv = *reinterpret_cast<const V*>(xr + at);
      if (!in) xv = V{0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
      for (int r = 0; r < RT; ++r) acc[r] = Half<DT>::mfma(*reinterpret_cast<const V*>(ar[r] + at), xv, acc[r]);
    }
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int e = 0; e < 4; ++e) keep[r][e] = mine ? acc[r][e] : keep[r][e];
  }
#pragma unroll
  for (int r = 0; r < RT; ++r) red[wave][r][l] = keep[r];
  __syncthreads();
  for (int r = wave; r < RT; r += kWaves) {
    mx::v4f v = red[0][r][l];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) v = v + red[w][r][l];
    const int rank = 16 * r + 4 * g;
    if (row0 + c < a.T && rank < a.R)
      *reinterpret_cast<mx::v4f*>(a.part + ((int64_t)q * a.T + row0 + c) * a.R + rank) = v;
  }
}

// 16 values of a row of y from column n on, and back.
template <int YT>
struct Row16 {
  static constexpr int kSize = YT == MXFP4_TYPE_F32 ? 4 : 2;
  static constexpr int kWords = 16 * kSize / 4;
  static __device__ __forceinline__ float one(const uint8_t* at) {
    if constexpr (YT == MXFP4_TYPE_F32) return *(const float*)at;
    const uint16_t b = *(const uint16_t*)at;
    if constexpr (YT == MXFP4_TYPE_BF16) return __builtin_bit_cast(float, (uint32_t)b << 16);
    return (float)__builtin_bit_cast(_Float16, b);
  }
  static __device__ __forceinline__ void put(uint8_t* at, float v) {
    if constexpr (YT == MXFP4_TYPE_F32)
      *(float*)at = v;
    else if constexpr (YT == MXFP4_TYPE_BF16)
      *(uint16_t*)at = mx::f32_to_bf16(v);
    else
      *(_Float16*)at = (_Float16)v;
  }
  static __device__ __forceinline__ void load(const uint8_t* at, int left, float (&v)[16]) {
    if (left >= 16) {
      uint32_t w[kWords];
#pragma unroll
      for (int i = 0; i < kWords / 4; ++i) {
        u32x4 p;
        if constexpr (kSize == 4)
          p = reinterpret_cast<const u32x4_at4*>(at)[i];
        else
          p = reinterpret_cast<const u32x4_at2*>(at)[i];
        w[4 * i] = p.x;
        w[4 * i + 1] = p.y;
        w[4 * i + 2] = p.z;
        w[4 * i + 3] = p.w;
      }
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        if constexpr (YT == MXFP4_TYPE_F32) {
          v[i] = __builtin_bit_cast(float, w[i]);
        } else if constexpr (YT == MXFP4_TYPE_BF16) {
          v[2 * i] = __builtin_bit_cast(float, w[i] << 16);
          v[2 * i + 1] = __builtin_bit_cast(float, w[i] & 0xffff0000u);
        } else {
          typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
          const f16x2 p = __builtin_bit_cast(f16x2, w[i]);
          v[2 * i] = (float)p[0];
          v[2 * i + 1] = (float)p[1];
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = i < left ? one(at + i * kSize) : 0.0f;
    }
  }
  static __device__ __forceinline__ void store(uint8_t* at, int left, const float (&v)[16]) {
    if (left >= 16) {
      uint32_t w[kWords];
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        if constexpr (YT == MXFP4_TYPE_F32) {
          w[i] = __builtin_bit_cast(uint32_t, v[i]);
        } else if constexpr (YT == MXFP4_TYPE_BF16) {
          w[i] = mx::pack_bf16x2(v[2 * i], v[2 * i + 1]);
        } else {
          typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
          const f16x2 p = {(_Float16)v[2 * i], (_Float16)v[2 * i + 1]};
          w[i] = __builtin_bit_cast(uint32_t, p);
        }
      }
#pragma unroll
      for (int i = 0; i < kWords / 4; ++i) {
        const u32x4 p = {w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]};
        if constexpr (kSize == 4)
          reinterpret_cast<u32x4_at4*>(at)[i] = p;
        else
          reinterpret_cast<u32x4_at2*>(at)[i] = p;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (i < left) put(at + i * kSize, v[i]);
    }
  }
};

// RS steps of 32 ranks (R <= 32 RS). The second product takes x . A^T as 16-bit pieces whose
// sum it is: two are within 2^-16 of it (bf16; fp16 2^-22), three, where y is fp32, within
// 2^-23. fp16 pieces are of the row times a power of two that brings its largest value to
// 2^14: they neither overflow nor lose bits to subnormals that would count.
template <int DT, int YT, int RS>
__global__ __launch_bounds__(kThreads) void expand_kernel(LoraArgs a) {
  typedef typename Half<DT>::V V;
  constexpr int kPieces = YT == MXFP4_TYPE_F32 ? 3 : 2;
  __shared__ __align__(16) float u[16][32 * RS + 4];
  const int tid = threadIdx.x, l = tid & 63, c = l & 15, g = l >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int row0 = 16 * blockIdx.x, n0 = kCols * blockIdx.y + 64 * wave;
  const int idx = adapter_of(a, row0);
  const uint64_t some = __ballot(idx >= 0) & 0xffffu;
  if (some == 0) return;  // the same on every wave
  for (int i = tid; i < 16 * 8 * RS; i += kThreads) {
    const int t = i / (8 * RS), rank = 4 * (i % (8 * RS));
    mx::v4f v = {0.f, 0.f, 0.f, 0.f};
    if (row0 + t < a.T && ((some >> t) & 1) && rank < a.R)
      for (int q = 0; q < a.splits; ++q)
        v = v + *reinterpret_cast<const mx::v4f*>(a.part + ((int64_t)q * a.T + row0 + t) * a.R + rank);
    *reinterpret_cast<mx::v4f*>(&u[t][rank]) = v;
  }
  __syncthreads();
  V piece[RS][kPieces];
  float back = 1.0f;  // undoes the power of two
  {
    float f[RS][8];
#pragma unroll
    for (int s = 0; s < RS; ++s)
#pragma unroll
      for (int e = 0; e < 8; ++e) f[s][e] = u[c][32 * s + 8 * g + e];
    if constexpr (DT == MXFP4_TYPE_F16) {
      uint32_t m = 0;
#pragma unroll
      for (int s = 0; s < RS; ++s)
#pragma unroll
        for (int e = 0; e < 8; ++e) m = max(m, __builtin_bit_cast(uint32_t, f[s][e]) & 0x7fffffffu);
      m = max(m, (uint32_t)__shfl_xor((int)m, 16, 64));
      m = max(m, (uint32_t)__shfl_xor((int)m, 32, 64));
      const int up = m == 0 || m >= 0x7f800000u ? 0 : min(14 + 127 - (int)(m >> 23), 126);
      const float by = __builtin_bit_cast(float, (uint32_t)(127 + up) << 23);
      back = __builtin_bit_cast(float, (uint32_t)(127 - up) << 23);
#pragma unroll
      for (int s = 0; s < RS; ++s)
#pragma unroll
        for (int e = 0; e < 8; ++e) f[s][e] *= by;
    }
#pragma unroll
    for (int s = 0; s < RS; ++s)
#pragma unroll
      for (int p = 0; p < kPieces; ++p)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          piece[s][p][e] = Half<DT>::round(f[s][e]);
          f[s][e] = f[s][e] - (float)piece[s][p][e];
        }
  }
  if (n0 >= a.N) return;  // whole waves, and there is no barrier below
  mx::v4f keep[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) keep[j] = mx::v4f{0.f, 0.f, 0.f, 0.f};
  for (uint64_t todo = some; todo != 0;) {
    const int i = __builtin_amdgcn_readlane(idx, __ffsll((unsigned long long)todo) - 1);
    const bool mine = idx == i;
    todo &= ~__ballot(mine);
    // Group j of 16 columns: the operand's row c is column 16 (c / 4) + 4 j + c % 4, so that the
    // four groups leave a lane with 16 neighbouring columns, 16 g .. 16 g + 15.
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int n = min(n0 + 16 * (c >> 2) + 4 * j + (c & 3), a.N - 1);
      const uint8_t* br = a.b + ((int64_t)i * a.N + n) * a.R * 2;
      mx::v4f acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int s = 0; s < RS; ++s) {
        const int rank = 32 * s + 8 * g;
        const bool in = rank < a.R;
        V bv = *reinterpret_cast<const V*>(br + (in ? 2 * rank : 0));
        if (!in) bv = V{0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
        for (int p = 0; p < kPieces; ++p) acc = Half<DT>::mfma(bv, piece[s][p], acc);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) keep[j][e] = mine ? acc[e] : keep[j][e];
    }
  }
  const int col = n0 + 16 * g;
  if (idx >= 0 && col < a.N) {
    const float by = a.scale ? a.scale[idx] : 1.0f;
    uint8_t* at = a.y + ((int64_t)(row0 + c) * a.ldy + col) * Row16<YT>::kSize;
    float v[16];
    Row16<YT>::load(at, a.N - col, v);
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) v[4 * j + e] = v[4 * j + e] + by * (keep[j][e] * back);
    Row16<YT>::store(at, a.N - col, v);
  }
}

bool shape_ok(int64_t T, int64_t K, int64_t R) {
  constexpr int64_t kMax = (int64_t)1 << 20;
  return T >= 1 && T <= kMax && K >= 8 && K <= kMax && K % 8 == 0 && R >= 8 && R <= 128 && R % 8 == 0;
}
// Workgroups that share a row tile's K: enough to occupy the chip, each wave one step at least.
int splits_of(int64_t T, int64_t K) {
  const int64_t tiles = mxh::cdiv(T, 16), most = mxh::cdiv(mxh::cdiv(K, 32), kWaves);
  const int64_t want = mxh::cdiv(512, tiles);
  return (int)(want < most ? want : most);
}

template <int DT, int RT>
hipError_t launch_shrink(LoraArgs& a, hipStream_t st) {
  void* args[] = {&a};
  return hipLaunchKernel((const void*)shrink_kernel<DT, RT>, dim3((unsigned)mxh::cdiv(a.T, 16), (unsigned)a.splits),
                         dim3(kThreads), args, 0, st);
}
template <int DT, int YT, int RS>
hipError_t launch_expand(LoraArgs& a, hipStream_t st) {
  void* args[] = {&a};
  return hipLaunchKernel((const void*)expand_kernel<DT, YT, RS>,
                         dim3((unsigned)mxh::cdiv(a.T, 16), (unsigned)mxh::cdiv(a.N, kCols)), dim3(kThreads), args, 0,
                         st);
}
template <int DT, int YT>
int launch(LoraArgs& a, hipStream_t st) {
  hipError_t e = a.R <= 16   ? launch_shrink<DT, 1>(a, st)
                 : a.R <= 32 ? launch_shrink<DT, 2>(a, st)
                 : a.R <= 64 ? launch_shrink<DT, 4>(a, st)
                             : launch_shrink<DT, 8>(a, st);
  if (e != hipSuccess) return MXFP4_ERR_HIP;
  e = a.R <= 32   ? launch_expand<DT, YT, 1>(a, st)
      : a.R <= 64 ? launch_expand<DT, YT, 2>(a, st)
                  : launch_expand<DT, YT, 4>(a, st);
  return mxh::launch_status(e);
}

}  // namespace

extern "C" size_t lora_add_workspace_bytes(int64_t T, int64_t K, int64_t R) {
  return shape_ok(T, K, R) ? (size_t)splits_of(T, K) * (size_t)T * (size_t)R * 4 : 0;
}

extern "C" int lora_add(void* y, int64_t ldy, int ytype, const void* x, int64_t ldx, int xtype, const void* a,
                        const void* b, const int32_t* index, const float* scale, int64_t T, int64_t N, int64_t K,
                        int64_t R, int64_t n, void* workspace, size_t workspace_bytes, void* stream) {
  if (T < 1 || N < 1 || n < 1) return MXFP4_ERR_SHAPE;  // first: an empty tensor's pointer may be NULL
  if (!y || !x || !a || !b || !index) return MXFP4_ERR_NULL;
  if (xtype != MXFP4_TYPE_BF16 && xtype != MXFP4_TYPE_F16) return MXFP4_ERR_ARG;
  if (ytype != xtype && ytype != MXFP4_TYPE_F32) return MXFP4_ERR_ARG;
  constexpr int64_t kMax = (int64_t)1 << 20, kMaxLd = (int64_t)1 << 36;
  if (!shape_ok(T, K, R) || N > kMax || n > kMax || ldx < K || ldx > kMaxLd || ldy < N || ldy > kMaxLd)
    return MXFP4_ERR_SHAPE;
  if (!mxh::aligned(x, 16) || ldx % 8 != 0 || !mxh::aligned(a, 16) || !mxh::aligned(b, 16) ||
      !mxh::aligned(y, ytype == MXFP4_TYPE_F32 ? 4 : 2) || !mxh::aligned(index, 4) || !mxh::aligned(scale, 4))
    return MXFP4_ERR_ALIGN;
  if (!workspace || !mxh::aligned(workspace, 16) || workspace_bytes < lora_add_workspace_bytes(T, K, R))
    return MXFP4_ERR_WORKSPACE;
  LoraArgs p{(uint8_t*)y, ldy,   (const uint8_t*)x, ldx * 2, (const uint8_t*)a, (const uint8_t*)b, index, scale,
             (float*)workspace, (int)T, (int)N, (int)K, (int)R, (int)n, splits_of(T, K)};
  const hipStream_t st = (hipStream_t)stream;
  if (xtype == MXFP4_TYPE_BF16)
    return ytype == MXFP4_TYPE_F32 ? launch<MXFP4_TYPE_BF16, MXFP4_TYPE_F32>(p, st)
                                   : launch<MXFP4_TYPE_BF16, MXFP4_TYPE_BF16>(p, st);
  return ytype == MXFP4_TYPE_F32 ? launch<MXFP4_TYPE_F16, MXFP4_TYPE_F32>(p, st)
                                 : launch<MXFP4_TYPE_F16, MXFP4_TYPE_F16>(p, st);
}
