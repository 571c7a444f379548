// moe_route: the k experts of each token and their weights, from the router's logits.
//
// One wave to a row. Lane l holds the logits l, l + 64, ...; without a bias the rank is
// the logit itself, as an integer that orders like it (32 bits), with one it is score +
// bias in float64 (64 bits): a last bit of a rounded score would change choices that lie
// close together, and a row has too few values for the float64 work to show. k rounds take
// the largest (rank, lowest index) over the wave; a lane looks for its next candidate only
// after one of its own was taken.
#include "host_common.hpp"

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

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int s = 32; s >= 1; s >>= 1) v = fmaxf(v, __shfl_xor(v, s, 64));
  return v;
}
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int s = 32; s >= 1; s >>= 1) v = v + __shfl_xor(v, s, 64);
  return v;
}

constexpr int kRows = 4;  // rows (waves) to a workgroup

// S logits to a lane (E <= 64 S).
template <int DT, int S, bool BIAS>
__global__ __launch_bounds__(64 * kRows) void route_kernel(RouteArgs a) {
  typedef typename std::conditional<BIAS, uint64_t, uint32_t>::type Key;
  const int l = threadIdx.x & 63;
  const int64_t row = (int64_t)blockIdx.x * kRows + (threadIdx.x >> 6);
  if (row >= a.T) return;  // whole waves, and there is no barrier
  const int64_t base = row * a.ldl;
  float v[S];
#pragma unroll
  for (int i = 0; i < S; ++i) v[i] = l + 64 * i < a.E ? logit_at<DT>(a.logits, base + l + 64 * i) : -__builtin_inff();
  float top = -__builtin_inff();
  bool bad = false;
#pragma unroll
  for (int i = 0; i < S; ++i) {
    bad |= !(v[i] < __builtin_inff());  // NaN or +Inf
    top = fmaxf(top, v[i]);
  }
  top = wave_max(top);
  // The softmax's sum over the row is needed for its scores as ranks or as weights.
  double total = 0.0;
  const bool sums = !a.sigmoid && (BIAS || !a.renormalize);
  if (sums) {
#pragma unroll
    for (int i = 0; i < S; ++i) total = total + (v[i] > -__builtin_inff() ? exp((double)v[i] - (double)top) : 0.0);
    total = wave_sum(total);
  }
  auto score = [&](float x) {
    if (a.sigmoid) return 1.0 / (1.0 + exp(-(double)x));
    const double p = exp((double)x - (double)top);
    return sums ? p / total : p;
  };
  Key key[S];  // 0: cannot be chosen (the order of every real value is larger)
#pragma unroll
  for (int i = 0; i < S; ++i) {
    if constexpr (BIAS) {
      key[i] = 0;
      if (v[i] > -__builtin_inff()) {
        const double r = score(v[i]) + (double)a.bias[l + 64 * i];
        bad |= !(r < __builtin_inf());
        key[i] = r > -__builtin_inf() ? order64(r) : 0;
      }
    } else {
      key[i] = v[i] > -__builtin_inff() ? order32(v[i]) : 0;
    }
  }
  if (__ballot(bad)) {
    for (int j = l; j < a.k; j += 64) {
      a.ids[row * a.k + j] = j;
      a.weights[row * a.k + j] = __builtin_nanf("");
    }
    return;
  }
  // A lane's candidate: its largest key, the lowest index among equals.
  Key best;
  int at;
  float val;
  auto candidate = [&]() {
    best = key[0];
    at = l;
    val = v[0];
#pragma unroll
    for (int i = 1; i < S; ++i)
      if (key[i] > best) {
        best = key[i];
        at = l + 64 * i;
        val = v[i];
      }
  };
  candidate();
  int id = -1;      // lane j keeps choice j
  float chosen = 0.0f;
  for (int j = 0; j < a.k; ++j) {
    Key b = best;
    int e = at;
    float x = val;
#pragma unroll
    for (int s = 32; s >= 1; s >>= 1) {
      const Key ob = __shfl_xor(b, s, 64);
      const int oe = __shfl_xor(e, s, 64);
      const float ox = __shfl_xor(x, s, 64);
      if (ob > b || (ob == b && oe < e)) {
        b = ob;
        e = oe;
        x = ox;
      }
    }
    if (b == 0) break;  // nothing left, the same on every lane
    if (l == j) {
      id = e;
      chosen = x;
    }
    if (at == e) {
#pragma unroll
      for (int i = 0; i < S; ++i)
        if (l + 64 * i == e) key[i] = 0;
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
  if (a.E <= 256) return launch_bias<DT, 4>(a, st);
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
  if (T > ((int64_t)1 << 24) || E > 1024 || k > 64 || k > E || ldl < E || ldl > ((int64_t)1 << 36)) return MXFP4_ERR_SHAPE;
  if (!mxh::aligned(logits, dtype == MXFP4_TYPE_F32 ? 4 : 2) || !mxh::aligned(bias, 4) || !mxh::aligned(weights, 4) ||
      !mxh::aligned(ids, 4))
    return MXFP4_ERR_ALIGN;
  RouteArgs a{logits, ldl, bias, weights, ids, T, (int)E, (int)k, score == MXFP4_SCORE_SIGMOID, renormalize != 0, scale};
  const hipStream_t st = (hipStream_t)stream;
  switch (dtype) {
    case MXFP4_TYPE_BF16: return mxh::launch_status(launch_size<MXFP4_TYPE_BF16>(a, st));
    case MXFP4_TYPE_F16: return mxh::launch_status(launch_size<MXFP4_TYPE_F16>(a, st));
    default: return mxh::launch_status(launch_size<MXFP4_TYPE_F32>(a, st));
  }
}
