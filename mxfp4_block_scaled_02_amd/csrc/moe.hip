// moe_a16w4: the experts' gated MLP of a mixture of experts on MXFP4 weights for a few
// tokens (bf16 activations; the weights' bytes bound it, so the activations are not
// quantised).
#include "host_common.hpp"
#include "mx_device.hpp"

namespace {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
constexpr int kMaxE = 1024;

struct MoeArgs {
  const uint8_t* x;  // strides in bytes
  int64_t ldx;
  const int32_t* ids;
  const float* weights;
  const uint8_t* w13;
  int64_t stride13;
  const uint8_t* w2;
  int64_t stride2;
  uint8_t* y;
  int64_t ldy;
  uint8_t* h;   // bf16 [pairs, I]
  float* part;  // fp32 [pairs, H]
  int T, k, E, H, I;
};

// Packed weight of one expert: see mxfp4_pack_B.
struct Packed {
  const uint8_t* units;
  const uint8_t* scales;
  int KU, KG;
};
__device__ __forceinline__ Packed packed(const uint8_t* base, int N, int K) {
  Packed p;
  p.KU = (K + 63) / 64;
  p.KG = (p.KU + 3) / 4;
  p.units = base;
  p.scales = base + (int64_t)(N / 32) * p.KU * 1024;
  return p;
}

// The expert of a slot (the slot-th of those that any pair takes, in rising order), and its
// pairs. Returns the number of pairs, 0 for a slot past the last expert.
struct Rows {
  uint32_t bits[kMaxE / 32];
  int count;
  uint16_t pair[MXFP4_MOE_MAX_PAIRS];
};
__device__ __forceinline__ int find_rows(const MoeArgs& a, int slot, Rows& s, int& expert) {
  const int tid = threadIdx.x, l = tid & 63, P = a.T * a.k;
  if (tid < kMaxE / 32) s.bits[tid] = 0;
  if (tid == 0) s.count = 0;
  __syncthreads();
  for (int i = tid; i < P; i += kThreads) {
    const uint32_t e = (uint32_t)a.ids[i];
    if (e < (uint32_t)a.E) atomicOr(&s.bits[e >> 5], 1u << (e & 31));
  }
  __syncthreads();
  const uint32_t word = l < kMaxE / 32 ? s.bits[l] : 0;
  int upto = __popc(word);  // experts in this and the words before
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(upto, d, 64);
    if (l >= d) upto += o;
  }
  const uint64_t has = __ballot(upto > slot);
  if (has == 0) return 0;  // the same on every thread
  const int at = __ffsll((unsigned long long)has) - 1;
  uint32_t w = (uint32_t)__builtin_amdgcn_readlane((int)word, at);
  int skip = slot - (__builtin_amdgcn_readlane(upto, at) - __popc(w));
  for (; skip > 0; --skip) w &= w - 1;
  expert = 32 * at + __ffs(w) - 1;
  for (int i = tid; i < P; i += kThreads)
    if (a.ids[i] == expert) s.pair[atomicAdd(&s.count, 1)] = (uint16_t)i;
  __syncthreads();
  return s.count;
}

__device__ __forceinline__ v8bf expand(uint32_t codes, float scale) {
  const mx::v2bf p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 0);
  const mx::v2bf p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 1);
  const mx::v2bf p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 2);
  const mx::v2bf p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 3);
  return v8bf{p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
}

// acc[r][c] (+)= rows 16r.. of the activations times 16-column group c of two 32-column
// tiles (c / 2 the tile, c % 2 its half) over this wave's share of K: scale groups of 256 k,
// wave, wave + kWaves, .... The weights are the first operand, so that result register i of
// lane l is column 4 * (l / 16) + i of the group for row l % 16. Lane l supplies the 32
// codes of column l % 16, k = 32 * (l / 16) .. +31 of a 128-k step, and the same k of its row.
template <int NT>
__device__ __forceinline__ void multiply(const Packed& p, const int (&tile)[2], const uint8_t* const (&row)[NT], int K,
                                         int wave, mx::v4f (&acc)[NT][4]) {
  const int l = threadIdx.x & 63, c = l & 15, g = l >> 4;
  const uint8_t* unit[2];
  const uint8_t* scale[2];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    unit[t] = p.units + (int64_t)tile[t] * p.KU * 1024;
    scale[t] = p.scales + (int64_t)tile[t] * p.KG * 256;
  }
  const int lane = (g & 1) * 32 + c;  // of the unit's lanes, first half of its columns
  for (int q = wave; q < p.KG; q += kWaves) {
    u32x4 code[2][4];  // [step][column group]
    uint32_t sc[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int at = lane + 16 * (i & 1);
      sc[i] = *reinterpret_cast<const uint32_t*>(scale[i >> 1] + (int64_t)q * 256 + 4 * at) >> (8 * (g >> 1));
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const int u = 4 * q + 2 * s + (g >> 1);
        const bool in = u < p.KU;
        const u32x4 v = *reinterpret_cast<const u32x4*>(unit[i >> 1] + (int64_t)(in ? u : p.KU - 1) * 1024 + 16 * at);
        code[s][i] = in ? v : u32x4{0, 0, 0, 0};
      }
    }
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int k0 = min(256 * q + 128 * s + 32 * g, K - 32);  // past the end: the codes are zero
      v8bf f[NT][4];
#pragma unroll
      for (int r = 0; r < NT; ++r)
#pragma unroll
        for (int j = 0; j < 4; ++j) f[r][j] = *reinterpret_cast<const v8bf*>(row[r] + 2 * (int64_t)k0 + 16 * j);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float e = __builtin_bit_cast(float, ((sc[i] >> (16 * s)) & 0xffu) << 23);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const v8bf w = expand(code[s][i][j], e);
#pragma unroll
          for (int r = 0; r < NT; ++r) acc[r][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, f[r][j], acc[r][i], 0, 0, 0);
        }
      }
    }
  }
}

constexpr int kMaxNT = 4;
struct Smem {
  Rows rows;
  mx::v4f red[kWaves][kMaxNT * 4][64];
};

template <int NT>
__device__ __forceinline__ void store_parts(const mx::v4f (&acc)[NT][4], int wave, Smem& sm) {
  const int l = threadIdx.x & 63;
  __syncthreads();
#pragma unroll
  for (int r = 0; r < NT; ++r)
#pragma unroll
    for (int i = 0; i < 4; ++i) sm.red[wave][r * 4 + i][l] = acc[r][i];
  __syncthreads();
}
__device__ __forceinline__ mx::v4f sum_parts(const Smem& sm, int i, int l) {
  mx::v4f v = sm.red[0][i][l];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) v = v + sm.red[w][i][l];
  return v;
}

// 32 columns of gate and of up of one expert for 16 * NT of its pairs, and h.
template <int NT>
__device__ __forceinline__ void up_rows(const MoeArgs& a, const Packed& p, int tile, int first, int n, Smem& sm) {
  const int tid = threadIdx.x, l = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const uint8_t* row[NT];
#pragma unroll
  for (int r = 0; r < NT; ++r) row[r] = a.x + (sm.rows.pair[min(first + 16 * r + (l & 15), n - 1)] / a.k) * a.ldx;
  mx::v4f acc[NT][4];
#pragma unroll
  for (int r = 0; r < NT; ++r)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[r][i] = mx::v4f{0.f, 0.f, 0.f, 0.f};
  const int tiles[2] = {tile, a.I / 32 + tile};
  multiply<NT>(p, tiles, row, a.H, wave, acc);
  store_parts<NT>(acc, wave, sm);
  for (int i = tid; i < NT * 2 * 64; i += kThreads) {
    const int r = i >> 7, half = (i >> 6) & 1;
    const int at = first + 16 * r + (l & 15);
    const mx::v4f g = sum_parts(sm, 4 * r + half, l), u = sum_parts(sm, 4 * r + 2 + half, l);
    float h[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) h[e] = g[e] / (1.0f + expf(-g[e])) * u[e];
    if (at < n)
      *reinterpret_cast<u32x2*>(a.h + ((int64_t)sm.rows.pair[at] * a.I + 32 * tile + 16 * half + 4 * (l >> 4)) * 2) =
          u32x2{mx::pack_bf16x2(h[0], h[1]), mx::pack_bf16x2(h[2], h[3])};
  }
}

// 64 columns of the down product of one expert for 16 * NT of its pairs.
template <int NT>
__device__ __forceinline__ void down_rows(const MoeArgs& a, const Packed& p, int block, int first, int n, Smem& sm) {
  const int tid = threadIdx.x, l = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const uint8_t* row[NT];
#pragma unroll
  for (int r = 0; r < NT; ++r) row[r] = a.h + (int64_t)sm.rows.pair[min(first + 16 * r + (l & 15), n - 1)] * a.I * 2;
  mx::v4f acc[NT][4];
#pragma unroll
  for (int r = 0; r < NT; ++r)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[r][i] = mx::v4f{0.f, 0.f, 0.f, 0.f};
  const int tiles[2] = {2 * block, min(2 * block + 1, a.H / 32 - 1)};
  multiply<NT>(p, tiles, row, a.I, wave, acc);
  store_parts<NT>(acc, wave, sm);
  for (int i = tid; i < NT * 4 * 64; i += kThreads) {
    const int r = i >> 8, c = (i >> 6) & 3;
    const int at = first + 16 * r + (l & 15), col = 64 * block + 16 * c + 4 * (l >> 4);
    if (at < n && col < a.H)
      *reinterpret_cast<mx::v4f*>(a.part + (int64_t)sm.rows.pair[at] * a.H + col) = sum_parts(sm, 4 * r + c, l);
  }
}

template <bool UP>
__global__ __launch_bounds__(kThreads) void experts_kernel(MoeArgs a) {
  __shared__ __align__(16) Smem sm;
  int expert = 0;
  const int n = find_rows(a, blockIdx.y, sm.rows, expert);
  if (n == 0) return;
  expert = __builtin_amdgcn_readfirstlane(expert);
  const Packed p = UP ? packed(a.w13 + expert * a.stride13, 2 * a.I, a.H) : packed(a.w2 + expert * a.stride2, a.H, a.I);
  for (int first = 0; first < n; first += 16 * kMaxNT) {
    const int left = n - first;
    if (left <= 16)
      UP ? up_rows<1>(a, p, blockIdx.x, first, n, sm) : down_rows<1>(a, p, blockIdx.x, first, n, sm);
    else if (left <= 32)
      UP ? up_rows<2>(a, p, blockIdx.x, first, n, sm) : down_rows<2>(a, p, blockIdx.x, first, n, sm);
    else
      UP ? up_rows<4>(a, p, blockIdx.x, first, n, sm) : down_rows<4>(a, p, blockIdx.x, first, n, sm);
    __syncthreads();
  }
}

// y[t] = sum over the token's pairs, in their order.
__global__ __launch_bounds__(256) void combine_kernel(MoeArgs a) {
  const int t = blockIdx.y, col = 4 * (blockIdx.x * 256 + threadIdx.x);
  if (col >= a.H) return;
  mx::v4f v = {0.f, 0.f, 0.f, 0.f};
  for (int j = 0; j < a.k; ++j) {
    const int64_t p = (int64_t)t * a.k + j;
    if ((uint32_t)a.ids[p] < (uint32_t)a.E) {
      const mx::v4f q = *reinterpret_cast<const mx::v4f*>(a.part + p * a.H + col);
      v = v + a.weights[p] * q;
    }
  }
  *reinterpret_cast<u32x2*>(a.y + t * a.ldy + 2 * col) = u32x2{mx::pack_bf16x2(v[0], v[1]), mx::pack_bf16x2(v[2], v[3])};
}

bool shape_ok(int64_t T, int64_t k, int64_t H, int64_t I) {
  constexpr int64_t kMaxRow = (int64_t)1 << 20;
  return T >= 1 && k >= 1 && T <= MXFP4_MOE_MAX_PAIRS && k <= MXFP4_MOE_MAX_PAIRS && T * k <= MXFP4_MOE_MAX_PAIRS &&
         H >= 32 && H <= kMaxRow && H % 32 == 0 && I >= 32 && I <= kMaxRow && I % 32 == 0;
}
size_t h_bytes(int64_t T, int64_t k, int64_t I) { return (size_t)(T * k * I * 2 + 255) / 256 * 256; }

}  // namespace

extern "C" size_t moe_a16w4_workspace_bytes(int64_t T, int64_t k, int64_t H, int64_t I) {
  if (!shape_ok(T, k, H, I)) return 0;
  return h_bytes(T, k, I) + (size_t)(T * k * H) * 4;
}

extern "C" int moe_a16w4(const void* x, int64_t ldx, const int32_t* ids, const float* weights, const void* w13,
                         int64_t stride13, const void* w2, int64_t stride2, void* y, int64_t ldy, int64_t T, int64_t k,
                         int64_t E, int64_t H, int64_t I, void* workspace, size_t workspace_bytes, void* stream) {
  if (T < 1 || k < 1) return MXFP4_ERR_SHAPE;  // first: an empty tensor's pointer may be NULL
  if (!x || !ids || !weights || !w13 || !w2 || !y) return MXFP4_ERR_NULL;
  if (!shape_ok(T, k, H, I) || E < 1 || E > kMaxE) return MXFP4_ERR_SHAPE;
  constexpr int64_t kMaxLd = (int64_t)1 << 36, kMaxStride = (int64_t)1 << 40;
  if (ldx < H || ldx > kMaxLd || ldy < H || ldy > kMaxLd) return MXFP4_ERR_SHAPE;
  if (stride13 < (int64_t)mxfp4_pack_B_bytes(2 * I, H) || stride13 > kMaxStride ||
      stride2 < (int64_t)mxfp4_pack_B_bytes(H, I) || stride2 > kMaxStride)
    return MXFP4_ERR_SHAPE;
  if (!mxh::aligned(x, 16) || ldx % 8 != 0 || !mxh::aligned(ids, 4) || !mxh::aligned(weights, 4) ||
      !mxh::aligned(w13, 16) || stride13 % 16 != 0 || !mxh::aligned(w2, 16) || stride2 % 16 != 0 ||
      !mxh::aligned(y, 8) || ldy % 4 != 0)
    return MXFP4_ERR_ALIGN;
  if (!workspace || !mxh::aligned(workspace, 16) || workspace_bytes < moe_a16w4_workspace_bytes(T, k, H, I))
    return MXFP4_ERR_WORKSPACE;
  MoeArgs a{(const uint8_t*)x, ldx * 2,       ids,      weights, (const uint8_t*)w13, stride13, (const uint8_t*)w2,
            stride2,           (uint8_t*)y,   ldy * 2,  (uint8_t*)workspace,
            (float*)((uint8_t*)workspace + h_bytes(T, k, I)), (int)T, (int)k, (int)E, (int)H, (int)I};
  void* args[] = {&a};
  const hipStream_t st = (hipStream_t)stream;
  const unsigned slots = (unsigned)(T * k < E ? T * k : E);
  hipError_t e = hipLaunchKernel((const void*)experts_kernel<true>, dim3((unsigned)(I / 32), slots), dim3(kThreads), args,
                                 0, st);
  if (e != hipSuccess) return MXFP4_ERR_HIP;
  e = hipLaunchKernel((const void*)experts_kernel<false>, dim3((unsigned)mxh::cdiv(H, 64), slots), dim3(kThreads), args,
                      0, st);
  if (e != hipSuccess) return MXFP4_ERR_HIP;
  return mxh::launch_status(hipLaunchKernel((const void*)combine_kernel, dim3((unsigned)mxh::cdiv(H, 1024), (unsigned)T),
                                            dim3(256), args, 0, st));
}
