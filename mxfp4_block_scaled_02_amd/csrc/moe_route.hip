// moe_route: the k experts of each token and their weights, from the router's logits.
//
// One wave to a row; lane l holds the S neighbouring logits from l * S on. Without a bias the
// rank is the logit itself, as an integer that orders like it (32 bits), with one it is score +
// bias in float64 (64 bits): a last bit of a rounded score would change choices that lie close
// together, and a row has too few values for the float64 work to show. k rounds take the
// largest rank over the wave; equal ranks go to the lowest lane, and a lane's own candidate is
// its first, so that the lowest index wins without being compared. Reductions run over DPP
// moves, a few cycles each; a shuffle through LDS takes over 100, and a row needs about 60 in
// turn. 16 rows of 256 logits with k 8 take 5.4 us for the launch (sigmoid and bias, 64-bit ranks),
// 4096 rows (4 MB) 6.4, 777 rows of 60 with k 3 3.3. Not bytes but latencies bound few rows, from
// replays of a launch at k 1, 8 and 16: of 5.2 us 1.8 are a smallest kernel's, 1.7 the rounds (0.22 each,
// 0.17 on 32-bit ranks), the rest the loads (each bias and each 16-bit logit is waited for by itself)
// and the float64 scores. With 4096 rows, four waves to a SIMD, a round takes 0.29 (biased 0.41):
// there the instructions issued count.
#include <type_traits>

#include "host_common.hpp"

// The float64 steps are the definition's: none are joined.
#pragma clang fp contract(off)

namespace {

struct RouteArgs {
  const void* logits;
  int64_t ldl;
  const float* bias;
  float* weights;
  int32_t* ids;
  int64_t T;
  int E, k, sigmoid, renormalize;
  float scale;
};

template <int DT>
__device__ __forceinline__ float logit_at(const void* p, int64_t i) {
  if constexpr (DT == MXFP4_TYPE_F32) return ((const float*)p)[i];
  const uint16_t b = ((const uint16_t*)p)[i];
  if constexpr (DT == MXFP4_TYPE_BF16) return __builtin_bit_cast(float, (uint32_t)b << 16);
  return (float)__builtin_bit_cast(_Float16, b);
}

// An integer that orders like the value (-0 below +0 would split a tie: they are equal).
__device__ __forceinline__ uint32_t order32(float v) {
  const uint32_t b = __builtin_bit_cast(uint32_t, v == 0.0f ? 0.0f : v);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ uint64_t order64(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v == 0.0 ? 0.0 : v);
  return b >> 63 ? ~b : b | 0x8000000000000000ull;
}

// v of the lane that the step's move takes it from; `none` for lanes without one. After the
// steps 0 to 5, each combined with the lane's own, lane 63 has all lanes' values.
template <int STEP>
__device__ __forceinline__ uint32_t moved(uint32_t v, uint32_t none) {
  constexpr int kCtrl[6] = {0x111, 0x112, 0x114, 0x118, 0x142, 0x143};  // row_shr 1, 2, 4, 8, row_bcast 15, 31
  constexpr int kRowMask[6] = {0xf, 0xf, 0xf, 0xf, 0xa, 0xc};
  return (uint32_t)__builtin_amdgcn_update_dpp((int)none, (int)v, kCtrl[STEP], kRowMask[STEP], 0xf, false);
}
template <int STEP = 0>
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  if constexpr (STEP == 6) {
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
  } else {
    const uint32_t o = moved<STEP>(v, 0);
    return wave_max<STEP + 1>(v > o ? v : o);
  }
}
template <int STEP = 0>
__device__ __forceinline__ double wave_sum(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  if constexpr (STEP == 6) {
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)b, 63);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), 63);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
  } else {
    const uint64_t o = (uint64_t)moved<STEP>((uint32_t)(b >> 32), 0) << 32 | moved<STEP>((uint32_t)b, 0);
    return wave_sum<STEP + 1>(v + __builtin_bit_cast(double, o));
  }
}
// The value of the largest key (0 if all are), the same on every lane.
__device__ __forceinline__ uint32_t largest(uint32_t k) { return wave_max(k); }
__device__ __forceinline__ uint64_t largest(uint64_t k) {
  const uint32_t hi = wave_max((uint32_t)(k >> 32));
  const uint32_t lo = wave_max((uint32_t)(k >> 32) == hi ? (uint32_t)k : 0u);
  return (uint64_t)hi << 32 | lo;
}

constexpr int kRows = 4;  // rows (waves) to a workgroup

// E <= 64 S.
template <int DT, int S, bool BIAS>
__global__ __launch_bounds__(64 * kRows) void route_kernel(RouteArgs a) {
  typedef typename std::conditional<BIAS, uint64_t, uint32_t>::type Key;
  const int l = threadIdx.x & 63;
  const int64_t row = (int64_t)blockIdx.x * kRows + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (row >= a.T) return;  // whole waves, and there is no barrier
  const int64_t base = row * a.ldl;
  float v[S], bias[S];
#pragma unroll
  for (int i = 0; i < S; ++i) {
    const int e = S * l + i;
    v[i] = e < a.E ? logit_at<DT>(a.logits, base + e) : -__builtin_inff();
    if constexpr (BIAS) bias[i] = e < a.E ? a.bias[e] : 0.0f;
  }
  uint32_t order[S], best32 = 0;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < S; ++i) {
    bad |= !(v[i] < __builtin_inff());  // NaN or +Inf
    order[i] = v[i] > -__builtin_inff() ? order32(v[i]) : 0;
    best32 = best32 > order[i] ? best32 : order[i];
  }
  // The row's largest logit (any value for a row without one).
  const uint32_t top32 = largest(best32);
  const double top = (double)__builtin_bit_cast(float, top32 & 0x80000000u ? top32 & 0x7fffffffu : ~top32);
  // The softmax's sum over the row is needed for its scores as ranks or as weights.
  double total = 0.0, scores[S];
  const bool sums = !a.sigmoid && (BIAS || !a.renormalize);
  if (sums) {
#pragma unroll
    for (int i = 0; i < S; ++i) {
      scores[i] = v[i] > -__builtin_inff() ? exp((double)v[i] - top) : 0.0;
      total = total + scores[i];
    }
    total = wave_sum(total);
  }
  auto score = [&](float x) {
    if (a.sigmoid) return 1.0 / (1.0 + exp(-(double)x));
    const double p = exp((double)x - top);
    return sums ? p / total : p;
  };
  Key key[S];  // 0: cannot be chosen (the order of every real value is larger)
#pragma unroll
  for (int i = 0; i < S; ++i) {
    if constexpr (BIAS) {
      key[i] = 0;
      if (order[i] != 0) {
        const double r = (a.sigmoid ? score(v[i]) : scores[i] / total) + (double)bias[i];
        bad |= !(r < __builtin_inf());
        key[i] = r > -__builtin_inf() ? order64(r) : 0;
      }
    } else {
      key[i] = order[i];
    }
  }
  if (__ballot(bad)) {
    if (l < a.k) {
      a.ids[row * a.k + l] = l;
      a.weights[row * a.k + l] = __builtin_nanf("");
    }
    return;
  }
  // A lane's candidate: its largest key, the lowest index among equals.
  Key best;
  int at;
  float val;
  auto candidate = [&]() {
    best = key[0];
    at = 0;
    val = v[0];
#pragma unroll
    for (int i = 1; i < S; ++i)
      if (key[i] > best) {
        best = key[i];
        at = i;
        val = v[i];
      }
  };
  candidate();
  int id = -1;  // lane j keeps choice j
  float chosen = 0.0f;
  for (int j = 0; j < a.k; ++j) {
    const Key b = largest(best);
    if (b == 0) break;  // nothing left, the same on every lane
    const int lane = __ffsll((unsigned long long)__ballot(best == b)) - 1;
    const int i0 = __builtin_amdgcn_readlane(at, lane);
    const float x = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, val), lane));
    if (l == j) {
      id = S * lane + i0;
      chosen = x;
    }
    if (l == lane) {
#pragma unroll
      for (int i = 0; i < S; ++i)
        if (i == i0) key[i] = 0;
      candidate();
    }
  }
  double w = id >= 0 ? score(chosen) : 0.0;
  if (a.renormalize) {
    const double sum = wave_sum(w);
    w = sum > 0.0 ? w / sum : 0.0;
  }
  if (l < a.k) {
    a.ids[row * a.k + l] = id;
    a.weights[row * a.k + l] = (float)(w * (double)a.scale);
  }
}

template <int DT, int S>
hipError_t launch_bias(RouteArgs& a, hipStream_t st) {
  void* args[] = {&a};
  const void* f = a.bias ? (const void*)route_kernel<DT, S, true> : (const void*)route_kernel<DT, S, false>;
  return hipLaunchKernel(f, dim3((unsigned)mxh::cdiv(a.T, kRows)), dim3(64 * kRows), args, 0, st);
}
template <int DT>
hipError_t launch_size(RouteArgs& a, hipStream_t st) {
  if (a.E <= 64) return launch_bias<DT, 1>(a, st);
  if (a.E <= 128) return launch_bias<DT, 2>(a, st);
  if (a.E <= 256) return launch_bias<DT, 4>(a, st);
  if (a.E <= 512) return launch_bias<DT, 8>(a, st);
  return launch_bias<DT, 16>(a, st);
}

}  // namespace

extern "C" int moe_route(const void* logits, int64_t ldl, int dtype, const float* bias, int score, int renormalize,
                         float scale, float* weights, int32_t* ids, int64_t T, int64_t E, int64_t k, void* stream) {
  if (T < 1 || E < 1 || k < 1) return MXFP4_ERR_SHAPE;  // first: an empty tensor's pointer may be NULL
  if (!logits || !weights || !ids) return MXFP4_ERR_NULL;
  if (dtype != MXFP4_TYPE_BF16 && dtype != MXFP4_TYPE_F16 && dtype != MXFP4_TYPE_F32) return MXFP4_ERR_ARG;
  if (score != MXFP4_SCORE_SOFTMAX && score != MXFP4_SCORE_SIGMOID) return MXFP4_ERR_ARG;
  if (!(scale >= -3.4028235e38f) || !(scale <= 3.4028235e38f)) return MXFP4_ERR_ARG;  // also rejects NaN
  if (T > ((int64_t)1 << 24) || E > 1024 || k > 64 || k > E || ldl < E || ldl > ((int64_t)1 << 36))
    return MXFP4_ERR_SHAPE;
  if (!mxh::aligned(logits, dtype == MXFP4_TYPE_F32 ? 4 : 2) || !mxh::aligned(bias, 4) || !mxh::aligned(weights, 4) ||
      !mxh::aligned(ids, 4))
    return MXFP4_ERR_ALIGN;
  RouteArgs a{logits, ldl, bias, weights, ids, T, (int)E, (int)k, score == MXFP4_SCORE_SIGMOID, renormalize != 0,
              scale};
  const hipStream_t st = (hipStream_t)stream;
  switch (dtype) {
    case MXFP4_TYPE_BF16: return mxh::launch_status(launch_size<MXFP4_TYPE_BF16>(a, st));
    case MXFP4_TYPE_F16: return mxh::launch_status(launch_size<MXFP4_TYPE_F16>(a, st));
    default: return mxh::launch_status(launch_size<MXFP4_TYPE_F32>(a, st));
  }
}
