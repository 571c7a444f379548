// int8_quant and int8_rmsnorm_quant: one int8 code per element and one fp32
// scale per row, of the row itself or of its root-mean-square norm (with the
// residual's addition in front). The rule, for the fp32 values y of a row:
//   s = max(fl(max|y| * fl(1/127)), 2^-126),  r = fl(1/s),  code = rint(fl(y*r)).
// |y| <= max|y| makes |fl(y*r)| <= 127 (1 + 2^-21), whose nearest integer is at
// most 127, so the codes need no clamp; the lower bound on s keeps r finite for
// rows of zeros or of subnormals. The maximum runs over the magnitude bits as
// integers, which order like the values with Inf and NaN on top: a row that
// holds one gets the scale NaN and codes 0, so that what is computed from the
// row shows it.
//
// A row is read once: thread t of the row's threads takes the 16-byte pieces t,
// t + threads, ..., keeps them in registers, and between the reductions (sum of
// squares, maximum) nothing goes to memory. The bytes bound it from about a thousand
// rows on: M4096 K7168 bf16 with a residual, 205 MB, 39 us with everything from memory
// (5.3 TB/s; a large copy reaches 5.4), without norm, 88 MB, 17.5 us; 31.5 and 14.6 us
// where the Infinity Cache holds part of it. A few rows take one trip to memory and two
// reductions: 16 rows 3.7 us in a graph, of which the launch is 1.7.
#include "host_common.hpp"
#include "mx_device.hpp"

#pragma clang fp contract(off)  // every fp32 step of the rule rounds by itself

namespace {

struct RowArgs {
  const uint8_t* x;  // strides in bytes
  int64_t ldx;
  const uint8_t* res;
  int64_t ldr;
  const uint8_t* w;
  uint8_t* h;
  int64_t ldh;
  uint8_t* q;
  int64_t ldq;
  float* s;
  int64_t M;
  int K;
  float eps;
};

typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

// Workgroups go kGridX to a row of the grid: one dimension of a launch holds fewer than
// 2^32 threads, which eight million rows of 512 would pass.
constexpr int64_t kGridX = (int64_t)1 << 20;
inline dim3 row_grid(int64_t groups) {
  return dim3((unsigned)(groups < kGridX ? groups : kGridX), (unsigned)mxh::cdiv(groups, kGridX));
}

enum Mode { kQuant, kNorm, kNormResidual };

// 16 bytes of a row as fp32 values, and back (round to nearest even).
template <int DT>
struct Piece {
  static constexpr int kElems = DT == MXFP4_TYPE_F32 ? 4 : 8;
  static constexpr int kSize = DT == MXFP4_TYPE_F32 ? 4 : 2;
  static __device__ __forceinline__ void unpack(const u32x4& v, float (&f)[kElems]) {
    const uint32_t wd[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (DT == MXFP4_TYPE_F32) {
        f[i] = __builtin_bit_cast(float, wd[i]);
      } else if constexpr (DT == MXFP4_TYPE_BF16) {
        f[2 * i] = __builtin_bit_cast(float, wd[i] << 16);
        f[2 * i + 1] = __builtin_bit_cast(float, wd[i] & 0xffff0000u);
      } else {
        const f16x2 p = __builtin_bit_cast(f16x2, wd[i]);
        f[2 * i] = (float)p.x;
        f[2 * i + 1] = (float)p.y;
      }
    }
  }
  static __device__ __forceinline__ u32x4 pack(const float (&f)[kElems]) {
    uint32_t wd[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (DT == MXFP4_TYPE_F32) {
        wd[i] = __builtin_bit_cast(uint32_t, f[i]);
      } else if constexpr (DT == MXFP4_TYPE_BF16) {
        wd[i] = mx::pack_bf16x2(f[2 * i], f[2 * i + 1]);
      } else {
        const f16x2 p = {(_Float16)f[2 * i], (_Float16)f[2 * i + 1]};
        wd[i] = __builtin_bit_cast(uint32_t, p);
      }
    }
    return u32x4{wd[0], wd[1], wd[2], wd[3]};
  }
};

// Loads go through a buffer resource over the row's bytes: a piece past the row
// reads zeros by the range check, which changes neither the sum nor the maximum.
// (K % 16 == 0: a piece lies wholly inside the row or wholly past it.)
__device__ __forceinline__ __amdgpu_buffer_rsrc_t row_rsrc(const void* base, int bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, bytes, 0x00020000);
}
__device__ __forceinline__ u32x4 load_piece(__amdgpu_buffer_rsrc_t r, int piece) {
  return __builtin_amdgcn_raw_buffer_load_b128(r, 16 * piece, 0, 0);
}

template <int E>
__device__ __forceinline__ uint32_t max_bits(uint32_t m, const float (&f)[E]) {
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const uint32_t b = __builtin_bit_cast(uint32_t, f[e]) & 0x7fffffffu;
    m = m > b ? m : b;
  }
  return m;
}

struct RowScale {
  float s, r;
  bool bad;
};
__device__ __forceinline__ RowScale row_scale(uint32_t amax_bits) {
  RowScale o;
  o.bad = amax_bits >= 0x7f800000u;
  const float t = __builtin_bit_cast(float, amax_bits) * (1.0f / 127.0f);
  o.s = t > 1.17549435e-38f ? t : 1.17549435e-38f;
  o.r = 1.0f / o.s;
  if (o.bad) o.s = __builtin_bit_cast(float, 0x7fc00000u);
  return o;
}

// Four codes in a dword. Adding 1.5 * 2^23 rounds a value of magnitude <= 127 to
// the nearest integer (ties to even), whose two's complement is the sum's low byte.
__device__ __forceinline__ uint32_t pack_codes(float a, float b, float c, float d) {
  constexpr float kMagic = 12582912.0f;
  const uint32_t ab = __builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, b + kMagic),
                                            __builtin_bit_cast(uint32_t, a + kMagic), 0x0c0c0400u);
  const uint32_t cd = __builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, d + kMagic),
                                            __builtin_bit_cast(uint32_t, c + kMagic), 0x04000c0cu);
  return ab | cd;
}

template <int E>
__device__ __forceinline__ void store_codes(uint8_t* at, const float (&y)[E], const RowScale& sc) {
  const uint32_t keep = sc.bad ? 0u : ~0u;
  const uint32_t lo = pack_codes(y[0] * sc.r, y[1] * sc.r, y[2] * sc.r, y[3] * sc.r) & keep;
  if constexpr (E == 8) {
    const uint32_t hi = pack_codes(y[4] * sc.r, y[5] * sc.r, y[6] * sc.r, y[7] * sc.r) & keep;
    *reinterpret_cast<u32x2*>(at) = u32x2{lo, hi};
  } else {
    *reinterpret_cast<uint32_t*>(at) = lo;
  }
}

// Sum and maximum over the W waves of a row, the same on every thread and the
// same on every run: a butterfly over the lanes, then the waves in order.
template <int W>
__device__ __forceinline__ double row_sum(double v, double* part) {
#pragma unroll
  for (int s = 32; s >= 1; s >>= 1) v = v + __shfl_xor(v, s, 64);
  if constexpr (W > 1) {
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    v = part[0];
#pragma unroll
    for (int u = 1; u < W; ++u) v = v + part[u];
  }
  return v;
}
template <int W>
__device__ __forceinline__ uint32_t row_max(uint32_t v, uint32_t* part) {
#pragma unroll
  for (int s = 32; s >= 1; s >>= 1) {
    const uint32_t o = (uint32_t)__shfl_xor((int)v, s, 64);
    v = v > o ? v : o;
  }
  if constexpr (W > 1) {
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    v = part[0];
#pragma unroll
    for (int u = 1; u < W; ++u) v = v > part[u] ? v : part[u];
  }
  return v;
}

__device__ __forceinline__ float norm_factor(double ss, int K, float eps) {
  return (float)(1.0 / __builtin_sqrt(ss / (double)K + (double)eps));
}

// Rows of at most 64 * W * R pieces: W waves to a row, one row to a workgroup
// (W > 1) or one to each of its four waves (W == 1).
template <int DT, int MODE, int W, int R>
__global__ __launch_bounds__(W == 1 ? 256 : 64 * W) void row_kernel(RowArgs a) {
  using P = Piece<DT>;
  constexpr int E = P::kElems;
  __shared__ double part_sum[W];
  __shared__ uint32_t part_max[W];
  const int t = W == 1 ? threadIdx.x & 63 : threadIdx.x;
  const int64_t group = (int64_t)blockIdx.y * kGridX + blockIdx.x;
  // a wave's row is uniform; without saying so the loads below loop over their lanes' descriptors
  const int64_t row = W == 1 ? group * 4 + __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6)) : group;
  if (row >= a.M) return;  // whole workgroups; with W == 1 whole waves, and then there is no barrier
  const int bytes = a.K * P::kSize;
  const __amdgpu_buffer_rsrc_t xr = row_rsrc(a.x + row * a.ldx, bytes);
  u32x4 v[R], w[R];
#pragma unroll
  for (int i = 0; i < R; ++i) v[i] = load_piece(xr, t + 64 * W * i);
  if constexpr (MODE == kNormResidual) {
    const __amdgpu_buffer_rsrc_t rr = row_rsrc(a.res + row * a.ldr, bytes);
    u32x4 u[R];
#pragma unroll
    for (int i = 0; i < R; ++i) u[i] = load_piece(rr, t + 64 * W * i);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      float f[E], g[E];
      P::unpack(v[i], f);
      P::unpack(u[i], g);
#pragma unroll
      for (int e = 0; e < E; ++e) f[e] = f[e] + g[e];
      v[i] = P::pack(f);
    }
  }
  if constexpr (MODE != kQuant) {
    const __amdgpu_buffer_rsrc_t wr = row_rsrc(a.w, bytes);
#pragma unroll
    for (int i = 0; i < R; ++i) w[i] = load_piece(wr, t + 64 * W * i);
  }
  if constexpr (MODE == kNormResidual) {
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int p = t + 64 * W * i;
      if (p * E < a.K) *reinterpret_cast<u32x4*>(a.h + row * a.ldh + 16 * p) = v[i];
    }
  }
  float inv = 1.0f;
  if constexpr (MODE != kQuant) {
    double ss = 0.0;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      float f[E];
      P::unpack(v[i], f);
#pragma unroll
      for (int e = 0; e < E; ++e) ss = __builtin_fma((double)f[e], (double)f[e], ss);
    }
    inv = norm_factor(row_sum<W>(ss, part_sum), a.K, a.eps);
  }
  auto values = [&](int i, float (&y)[E]) {
    P::unpack(v[i], y);
    if constexpr (MODE != kQuant) {
      float g[E];
      P::unpack(w[i], g);
#pragma unroll
      for (int e = 0; e < E; ++e) y[e] = (y[e] * inv) * g[e];
    }
  };
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    float y[E];
    values(i, y);
    m = max_bits<E>(m, y);
  }
  const RowScale sc = row_scale(row_max<W>(m, part_max));
  if (t == 0) a.s[row] = sc.s;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int p = t + 64 * W * i;
    if (p * E < a.K) {
      float y[E];
      values(i, y);
      store_codes<E>(a.q + row * a.ldq + p * E, y, sc);
    }
  }
}

// Rows longer than the registers of a workgroup hold: one workgroup to a row,
// which reads the row again for each of its phases. With a residual the first
// phase writes h and the later ones read it back, each thread its own pieces. Quantising
// 4096 bf16 rows of K 36864 takes 103 us (4.4 TB/s; the last length that the registers
// hold, K 32768, 71 us, 5.6 TB/s), 8192 fp32 rows of K 28672 297 us (4.0 TB/s).
constexpr int kLongWaves = 16;
template <int DT, int MODE>
__global__ __launch_bounds__(64 * kLongWaves) void row_long_kernel(RowArgs a) {
  using P = Piece<DT>;
  constexpr int E = P::kElems, T = 64 * kLongWaves;
  __shared__ double part_sum[kLongWaves];
  __shared__ uint32_t part_max[kLongWaves];
  const int64_t row = (int64_t)blockIdx.y * kGridX + blockIdx.x;
  if (row >= a.M) return;
  const int pieces = a.K / E;
  const uint8_t* src = a.x + row * a.ldx;
  float inv = 1.0f;
  if constexpr (MODE != kQuant) {
    double ss = 0.0;
    for (int p = threadIdx.x; p < pieces; p += T) {
      float f[E];
      u32x4 v = *reinterpret_cast<const u32x4*>(src + (int64_t)16 * p);
      P::unpack(v, f);
      if constexpr (MODE == kNormResidual) {
        float g[E];
        P::unpack(*reinterpret_cast<const u32x4*>(a.res + row * a.ldr + (int64_t)16 * p), g);
#pragma unroll
        for (int e = 0; e < E; ++e) f[e] = f[e] + g[e];
        v = P::pack(f);
        *reinterpret_cast<u32x4*>(a.h + row * a.ldh + (int64_t)16 * p) = v;
        P::unpack(v, f);
      }
#pragma unroll
      for (int e = 0; e < E; ++e) ss = __builtin_fma((double)f[e], (double)f[e], ss);
    }
    inv = norm_factor(row_sum<kLongWaves>(ss, part_sum), a.K, a.eps);
    if constexpr (MODE == kNormResidual) src = a.h + row * a.ldh;
  }
  auto values = [&](int p, float (&y)[E]) {
    P::unpack(*reinterpret_cast<const u32x4*>(src + (int64_t)16 * p), y);
    if constexpr (MODE != kQuant) {
      float g[E];
      P::unpack(*reinterpret_cast<const u32x4*>(a.w + (int64_t)16 * p), g);
#pragma unroll
      for (int e = 0; e < E; ++e) y[e] = (y[e] * inv) * g[e];
    }
  };
  uint32_t m = 0;
  for (int p = threadIdx.x; p < pieces; p += T) {
    float y[E];
    values(p, y);
    m = max_bits<E>(m, y);
  }
  const RowScale sc = row_scale(row_max<kLongWaves>(m, part_max));
  if (threadIdx.x == 0) a.s[row] = sc.s;
  for (int p = threadIdx.x; p < pieces; p += T) {
    float y[E];
    values(p, y);
    store_codes<E>(a.q + row * a.ldq + (int64_t)p * E, y, sc);
  }
}

template <int DT, int MODE, int W, int R>
hipError_t launch_row(RowArgs& a, hipStream_t st) {
  void* args[] = {&a};
  return hipLaunchKernel((const void*)row_kernel<DT, MODE, W, R>, row_grid(W == 1 ? mxh::cdiv(a.M, 4) : a.M),
                         dim3(W == 1 ? 256 : 64 * W), args, 0, st);
}

// Waves to a row and pieces to a thread, by the row's pieces; both were measured over K 256
// to 16384, 16 to 4096 rows, bf16 and fp32. Up to 1024 pieces a thread has one or two: more
// pieces are added up in turn (norm of 16 rows of 896 pieces: 2 waves 4.8 us, 8 waves 3.9),
// more waves cost their barriers and leave the last ones empty (norm of 4096 rows of 258
// bf16 pieces: 16 waves 31.8 us, 4 waves 15.4). Two waves with one piece rather than one
// with two take 65 to 128 pieces (norm of 16 rows of 128: 3.12 us, 3.26). Past 1024 pieces a
// thread has four: eight waves as long as they hold the row (quantising 2112 rows of 1792
// fp32 pieces: 16 waves with two 16.9 us, 8 waves with four 14.8).
template <int DT, int MODE>
hipError_t launch_mode(RowArgs& a, hipStream_t st) {
  const int pieces = a.K / Piece<DT>::kElems;
  if (pieces <= 64) return launch_row<DT, MODE, 1, 1>(a, st);
  if (pieces <= 128) return launch_row<DT, MODE, 2, 1>(a, st);
  if (pieces <= 256) return launch_row<DT, MODE, 2, 2>(a, st);
  if (pieces <= 512) return launch_row<DT, MODE, 4, 2>(a, st);
  if (pieces <= 1024) return launch_row<DT, MODE, 8, 2>(a, st);
  if (pieces <= 2048) return launch_row<DT, MODE, 8, 4>(a, st);
  if (pieces <= 4096) return launch_row<DT, MODE, 16, 4>(a, st);
  void* args[] = {&a};
  return hipLaunchKernel((const void*)row_long_kernel<DT, MODE>, row_grid(a.M), dim3(64 * kLongWaves), args, 0, st);
}

template <int MODE>
int launch(RowArgs& a, int dtype, void* stream) {
  const hipStream_t st = (hipStream_t)stream;
  switch (dtype) {
    case MXFP4_TYPE_BF16: return mxh::launch_status(launch_mode<MXFP4_TYPE_BF16, MODE>(a, st));
    case MXFP4_TYPE_F16: return mxh::launch_status(launch_mode<MXFP4_TYPE_F16, MODE>(a, st));
    default: return mxh::launch_status(launch_mode<MXFP4_TYPE_F32, MODE>(a, st));
  }
}

// K <= 2^28: a row's byte offsets (at most 4 K) stay below 2^31.
int check_rows(const void* x, int64_t ldx, const void* q, int64_t ldq, const void* s, int dtype, int64_t M, int64_t K) {
  if (M < 1 || K < 1) return MXFP4_ERR_SHAPE;  // first: an empty tensor's pointer may be NULL
  if (!x || !q || !s) return MXFP4_ERR_NULL;
  if (dtype != MXFP4_TYPE_BF16 && dtype != MXFP4_TYPE_F16 && dtype != MXFP4_TYPE_F32) return MXFP4_ERR_ARG;
  if (M > mxh::kMaxDim || K < 16 || K % 16 != 0 || K > ((int64_t)1 << 28)) return MXFP4_ERR_SHAPE;
  if (ldx < K || ldx > INT64_MAX / 8 / M || ldq < K || ldq > INT64_MAX / 2 / M) return MXFP4_ERR_SHAPE;
  const int64_t size = dtype == MXFP4_TYPE_F32 ? 4 : 2;
  if (!mxh::aligned(x, 16) || (ldx * size) % 16 != 0 || !mxh::aligned(q, 16) || ldq % 16 != 0 || !mxh::aligned(s, 4))
    return MXFP4_ERR_ALIGN;
  return MXFP4_OK;
}

}  // namespace

extern "C" int int8_quant(const void* x, int64_t ldx, int dtype, void* q, int64_t ldq, float* s, int64_t M, int64_t K,
                          void* stream) {
  const int rc = check_rows(x, ldx, q, ldq, s, dtype, M, K);
  if (rc != MXFP4_OK) return rc;
  const int64_t size = dtype == MXFP4_TYPE_F32 ? 4 : 2;
  RowArgs a{};
  a.x = (const uint8_t*)x;
  a.ldx = ldx * size;
  a.q = (uint8_t*)q;
  a.ldq = ldq;
  a.s = s;
  a.M = M;
  a.K = (int)K;
  return launch<kQuant>(a, dtype, stream);
}

extern "C" int int8_rmsnorm_quant(const void* x, int64_t ldx, const void* residual, int64_t ldr, const void* w,
                                  float eps, int dtype, void* h, int64_t ldh, void* q, int64_t ldq, float* s, int64_t M,
                                  int64_t K, void* stream) {
  const int rc = check_rows(x, ldx, q, ldq, s, dtype, M, K);
  if (rc != MXFP4_OK) return rc;
  if (!w || !residual != !h) return MXFP4_ERR_NULL;
  const int64_t size = dtype == MXFP4_TYPE_F32 ? 4 : 2;
  if (residual && (ldr < K || ldr > INT64_MAX / 8 / M || ldh < K || ldh > INT64_MAX / 8 / M)) return MXFP4_ERR_SHAPE;
  if (!(eps > 0.0f) || !(eps <= 3.4028235e38f)) return MXFP4_ERR_ARG;  // also rejects NaN
  if (!mxh::aligned(w, 16)) return MXFP4_ERR_ALIGN;
  if (residual && (!mxh::aligned(residual, 16) || (ldr * size) % 16 != 0 || !mxh::aligned(h, 16) ||
                   (ldh * size) % 16 != 0))
    return MXFP4_ERR_ALIGN;
  RowArgs a{(const uint8_t*)x, ldx * size, (const uint8_t*)residual, residual ? ldr * size : 0, (const uint8_t*)w,
            (uint8_t*)h, residual ? ldh * size : 0, (uint8_t*)q, ldq, s, M, (int)K, eps};
  return residual ? launch<kNormResidual>(a, dtype, stream) : launch<kNorm>(a, dtype, stream);
}
