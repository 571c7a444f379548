// lora_add: y[t] += scale * (x[t] . A^T) . B^T with the adapter (A, B) of each row, for
// low-rank adapters of many requests beside a shared projection.
//
// Two launches. shrink: x . A^T in fp32 partial sums [split][T][R]. expand: 512 columns to
// a workgroup, which adds the partial sums in their order, holds them as 16-bit pieces and
// multiplies with B. Both take 64 neighbouring rows and an adapter at a time: the rows that
// have it are gathered into 16-row tiles, so that A and B are read once for all of them, and
// no row meets another one's adapter.
#include "host_common.hpp"
#include "mx_device.hpp"

namespace {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef u32x4 u32x4_at4 __attribute__((aligned(4)));
typedef u32x4 u32x4_at2 __attribute__((aligned(2)));

constexpr int kBlock = 64;          // rows, one to a lane
constexpr int kStage = 64;          // k of a step of shrink: 128 bytes, a cache line of a row
constexpr int kShrinkWaves = 4;
constexpr int kShrinkThreads = 64 * kShrinkWaves;
constexpr int kExpandWaves = 4;
constexpr int kExpandThreads = 64 * kExpandWaves;
constexpr int kCols = 64 * kExpandWaves;  // columns of y to a workgroup of expand

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
  int T, N, K, R, n;
  int unit;           // 16-row tiles that a workgroup of expand takes together
  int splits, slice;  // workgroups that share K, steps of kStage to each
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

// The adapter of lane l's row, -1 without one.
__device__ __forceinline__ int adapter_of(const LoraArgs& a, int row0) {
  const int row = row0 + (threadIdx.x & 63);
  const int i = row < a.T ? a.index[row] : -1;
  return (uint32_t)i < (uint32_t)a.n ? i : -1;
}
// The groups of rows (of the 64) with the same adapter, in units of `tiles` 16-row tiles, of
// which gridDim.z workgroups take every gridDim.z-th; f(adapter, rows, first) is called by all
// waves alike, first the unit's first row within its group. One block of rows has a workgroup
// for each row instead, which goes on if its row is the first of a unit: the count of units
// before it need not be known.
template <typename F>
__device__ __forceinline__ void for_units(const LoraArgs& a, int idx, int tiles, F f) {
  if (gridDim.y == 1) {
    const int r = blockIdx.z, adapter = __builtin_amdgcn_readlane(idx, r);
    if (adapter < 0) return;
    const uint64_t rows = __ballot(idx == adapter);
    const int before = __popcll(rows & (((uint64_t)1 << r) - 1));
    if (before % (16 * tiles) == 0) f(adapter, rows, before);
    return;
  }
  int turn = blockIdx.z;
  for (uint64_t todo = __ballot(idx >= 0); todo != 0;) {
    const int adapter = __builtin_amdgcn_readlane(idx, __ffsll((unsigned long long)todo) - 1);
    const uint64_t rows = __ballot(idx == adapter);
    todo &= ~rows;
    for (int first = 0; first < __popcll(rows); first += 16 * tiles) {
      if (turn == 0) {
        f(adapter, rows, first);
        turn = gridDim.z;
      }
      --turn;
    }
  }
}
// Lane p gets the p-th of the rows (past the last one: some other row).
__device__ __forceinline__ int gathered(uint64_t rows) {
  const int l = threadIdx.x & 63;
  const uint64_t below = ((uint64_t)1 << l) - 1;
  const int at = (rows >> l) & 1 ? __popcll(rows & below) : __popcll(rows) + __popcll(~rows & below);
  return __builtin_amdgcn_ds_permute(4 * at, l);
}

// More than 16 rows (R <= 16 RT): rows of x and of A go through LDS a step at a time, as whole
// cache lines, each read once for the workgroup; wave w multiplies the rows 16 w .. 16 w + 15.
// Rows lie in LDS as 128 bytes of 8 pieces, piece p of row r at p ^ ((r / 2) % 8), which keeps
// the operands' reads free of bank conflicts. kAhead steps' loads are under way in registers.
// The ranks are the first operand: result register e of lane l is rank 4 * (l / 16) + e of
// row l % 16.
constexpr int kAhead = 4;
template <int RT>
struct TileSmem {
  u32x4 line[2][kBlock + 16 * RT][8];
};
template <int DT, int RT>
__device__ __forceinline__ void shrink_tile(const LoraArgs& a, int adapter, int row0, int order, int count, int begin,
                                            int end, TileSmem<RT>& sm, mx::v4f (&acc)[RT]) {
  typedef typename Half<DT>::V V;
  constexpr int kLoads = (8 * (kBlock + 16 * RT) + kShrinkThreads - 1) / kShrinkThreads;
  constexpr int kRows = kShrinkThreads / 8;  // rows that a load of all threads covers
  const int tid = threadIdx.x, l = tid & 63, c = l & 15, g = l >> 4, wave = tid >> 6;
  const int p = tid & 7, slot = p ^ ((tid >> 4) & 7);
  const uint8_t* src[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int r = kRows * i + (tid >> 3);
    src[i] = i < kBlock / kRows
                 ? a.x + (int64_t)(row0 + __shfl(order, min(r, count - 1), 64)) * a.ldx
                 : a.a + ((int64_t)adapter * a.R + min(r - kBlock, a.R - 1)) * a.K * 2;
  }
  // Steps past the end are zeros: the loop has no branch around a load, so that the waits count
  // the loads that are under way.
  u32x4 held[kAhead][kLoads];
  auto inside = [&](int s) { return s < end && kStage * s + 8 * p < a.K; };  // K % 8 == 0: a piece is in or out
  auto load = [&](int s, u32x4 (&v)[kLoads]) {
    const int64_t at = inside(s) ? 2 * (int64_t)(kStage * s + 8 * p) : 0;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) v[i] = *reinterpret_cast<const u32x4*>(src[i] + at);
  };
  auto put = [&](int s, const u32x4 (&v)[kLoads], int buf) {
    const bool in = inside(s);
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int r = kRows * i + (tid >> 3);
      if (r < kBlock + 16 * RT) sm.line[buf][r][slot] = in || i >= kBlock / kRows ? v[i] : u32x4{0, 0, 0, 0};
    }
  };
#pragma unroll
  for (int i = 0; i < kAhead; ++i) load(begin + i, held[i]);
  __syncthreads();  // the last group's reads
  put(begin, held[0], 0);
  load(begin + kAhead, held[0]);
  for (int s0 = begin; s0 < end; s0 += kAhead) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      static_assert(kAhead % 2 == 0, "the buffer follows from i alone");
      __syncthreads();
      V xv[2], av[2][RT];
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
        const int at = (4 * kk + g) ^ ((c >> 1) & 7);
        xv[kk] = __builtin_bit_cast(V, sm.line[i & 1][16 * wave + c][at]);
#pragma unroll
        for (int r = 0; r < RT; ++r) av[kk][r] = __builtin_bit_cast(V, sm.line[i & 1][kBlock + 16 * r + c][at]);
      }
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int kk = 0; kk < 2; ++kk)
#pragma unroll
        for (int r = 0; r < RT; ++r) acc[r] = Half<DT>::mfma(av[kk][r], xv[kk], acc[r]);
      put(s0 + i + 1, held[(i + 1) % kAhead], (i + 1) & 1);
      load(s0 + i + 1 + kAhead, held[(i + 1) % kAhead]);
    }
  }
}

// At most 16 rows: the operands go straight to registers, the waves share the K steps of 32
// and add up in LDS; U steps' loads are under way together.
template <int DT, int RT, int U>
__device__ __forceinline__ void shrink_few(const LoraArgs& a, int adapter, int row, int begin, int end,
                                           mx::v4f (&acc)[RT]) {
  typedef typename Half<DT>::V V;
  const int l = threadIdx.x & 63, c = l & 15, g = l >> 4;
  const uint8_t* xr = a.x + (int64_t)row * a.ldx;
  const uint8_t* ar[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) ar[r] = a.a + ((int64_t)adapter * a.R + min(16 * r + c, a.R - 1)) * a.K * 2;
  for (int s = begin; s < end; s += U) {
    V av[U][RT], xv[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = 32 * (s + u) + 8 * g;
      const bool in = s + u < end && k < a.K;
      const int64_t at = in ? 2 * (int64_t)k : 0;
      xv[u] = *reinterpret_cast<const V*>(xr + at);
      if (!in) xv[u] = V{0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
      for (int r = 0; r < RT; ++r) av[u][r] = *reinterpret_cast<const V*>(ar[r] + at);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int r = 0; r < RT; ++r) acc[r] = Half<DT>::mfma(av[u][r], xv[u], acc[r]);
  }
}

template <int DT, int RT, int U>
__global__ __launch_bounds__(kShrinkThreads) void shrink_kernel(LoraArgs a) {
  __shared__ union {
    TileSmem<RT> tile;
    mx::v4f red[kShrinkWaves][RT][64];
  } sm;
  const int tid = threadIdx.x, l = tid & 63, c = l & 15, g = l >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int row0 = kBlock * blockIdx.y, q = blockIdx.x;
  const int idx = adapter_of(a, row0);
  const int stages = (a.K + kStage - 1) / kStage, begin = q * a.slice, end = min(begin + a.slice, stages);
  for_units(a, idx, kBlock / 16, [&](int adapter, uint64_t rows, int) {
    const int order = gathered(rows), count = __popcll(rows);
    mx::v4f acc[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) acc[r] = mx::v4f{0.f, 0.f, 0.f, 0.f};
    auto store = [&](int t, int r, const mx::v4f& v) {
      const int row = row0 + __shfl(order, min(t, count - 1), 64), rank = 16 * r + 4 * g;
      if (t < count && rank < a.R) *reinterpret_cast<mx::v4f*>(a.part + ((int64_t)q * a.T + row) * a.R + rank) = v;
    };
    if (count > 16) {
      shrink_tile<DT, RT>(a, adapter, row0, order, count, begin, end, sm.tile, acc);
#pragma unroll
      for (int r = 0; r < RT; ++r) store(16 * wave + c, r, acc[r]);
    } else {
      const int share = (2 * a.slice + kShrinkWaves - 1) / kShrinkWaves, first = 2 * begin + wave * share;
      const int row = row0 + __shfl(order, min(c, count - 1), 64);
      shrink_few<DT, RT, U>(a, adapter, row, first, min(first + share, 2 * end), acc);
      __syncthreads();
#pragma unroll
      for (int r = 0; r < RT; ++r) sm.red[wave][r][l] = acc[r];
      __syncthreads();
      for (int r = wave; r < RT; r += kShrinkWaves) {
        mx::v4f v = sm.red[0][r][l];
#pragma unroll
        for (int w = 1; w < kShrinkWaves; ++w) v = v + sm.red[w][r][l];
        store(c, r, v);
      }
    }
  });
}

// The 16 of a wave's 64 columns of a row of y that lane group g (of four) has, as pieces of 16
// bytes: the four groups' pieces of one number are 64 neighbouring bytes of the row.
template <int YT>
struct Row16 {
  static constexpr int kSize = YT == MXFP4_TYPE_F32 ? 4 : 2;
  static constexpr int kWords = 16 * kSize / 4;
  static constexpr int kPieces = kWords / 4, kPer = 16 / kSize;  // columns to a piece
  // The column of value 4 j of group g.
  static __device__ __forceinline__ int column(int g, int j) {
    return 4 * kPer * (4 * j / kPer) + kPer * g + 4 * j % kPer;
  }
  // `row`: the wave's first column; `left` of its columns are there (FULL: all).
  template <bool FULL>
  static __device__ __forceinline__ void load(const uint8_t* row, int g, int left, uint32_t (&w)[kWords]) {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int n = 4 * kPer * i + kPer * g;
      const uint8_t* at = row + n * kSize;
      if constexpr (FULL) {
        u32x4 p;
        if constexpr (kSize == 4)
          p = *reinterpret_cast<const u32x4_at4*>(at);
        else
          p = *reinterpret_cast<const u32x4_at2*>(at);
        w[4 * i] = p.x;
        w[4 * i + 1] = p.y;
        w[4 * i + 2] = p.z;
        w[4 * i + 3] = p.w;
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if constexpr (kSize == 4) {
            w[4 * i + e] = n + e < left ? *(const uint32_t*)(at + 4 * e) : 0;
          } else {
            const uint32_t lo = n + 2 * e < left ? *(const uint16_t*)(at + 4 * e) : 0;
            const uint32_t hi = n + 2 * e + 1 < left ? *(const uint16_t*)(at + 4 * e + 2) : 0;
            w[4 * i + e] = lo | hi << 16;
          }
        }
      }
    }
  }
  static __device__ __forceinline__ void unpack(const uint32_t (&w)[kWords], float (&v)[16]) {
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
  }
  template <bool FULL>
  static __device__ __forceinline__ void store(uint8_t* row, int g, int left, const float (&v)[16]) {
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
    for (int i = 0; i < kPieces; ++i) {
      const int n = 4 * kPer * i + kPer * g;
      uint8_t* at = row + n * kSize;
      if constexpr (FULL) {
        const u32x4 p = {w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]};
        if constexpr (kSize == 4)
          *reinterpret_cast<u32x4_at4*>(at) = p;
        else
          *reinterpret_cast<u32x4_at2*>(at) = p;
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if constexpr (kSize == 4) {
            if (n + e < left) *(uint32_t*)(at + 4 * e) = w[4 * i + e];
          } else {
            if (n + 2 * e < left) *(uint16_t*)(at + 4 * e) = (uint16_t)w[4 * i + e];
            if (n + 2 * e + 1 < left) *(uint16_t*)(at + 4 * e + 2) = (uint16_t)(w[4 * i + e] >> 16);
          }
        }
      }
    }
  }
};

// RS steps of 32 ranks (R <= 32 RS). The second product takes x . A^T as 16-bit pieces whose
// sum it is: two are within 2^-16 of it (bf16; fp16 2^-22), three, where y is fp32, within
// 2^-23. fp16 pieces are of the row times a power of two that brings its largest value to
// 2^14: they neither overflow nor lose bits to subnormals that would count.
template <int YT, int RS>
constexpr int expand_tiles() {  // row tiles that go together: their rows of y are held in registers
  return YT == MXFP4_TYPE_F32 || RS == 4 ? 2 : 4;
}
template <int DT, int YT, int RS>
struct ExpandSmem {
  // Ranks of a row in pieces of 8, one row 16 bytes longer than its ranks.
  typename Half<DT>::V u[YT == MXFP4_TYPE_F32 ? 3 : 2][16 * expand_tiles<YT, RS>()][4 * RS + 1];
  float back[16 * expand_tiles<YT, RS>()];  // undoes the power of two
};
// 64 columns, from n0 on, of a unit's rows. FULL: y has all of them.
template <int DT, int YT, int RS>
struct Columns {
  typedef typename Half<DT>::V V;
  typedef Row16<YT> Y;
  static constexpr int kPieces = YT == MXFP4_TYPE_F32 ? 3 : 2, kTiles = expand_tiles<YT, RS>();
  V bv[4][RS];
  uint8_t* at[kTiles];
  uint32_t held[kTiles][Y::kWords];

  template <bool FULL>
  __device__ __forceinline__ void load(const LoraArgs& a, int adapter, int row0, int n0, int order, int first, int count) {
    const int l = threadIdx.x & 63, c = l & 15, g = l >> 4;
    // Row c of the operand of column group j is column Y::column(c / 4, j) + c % 4: result register e of
    // group j of lane l is column Y::column(g, j) + e. Past R the pieces are zeros, and B's are any.
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int n = min(n0 + Y::column(c >> 2, j) + (c & 3), a.N - 1);
      const uint8_t* br = a.b + ((int64_t)adapter * a.N + n) * a.R * 2;
#pragma unroll
      for (int s = 0; s < RS; ++s) {
        const int rank = 32 * s + 8 * g;
        bv[j][s] = *reinterpret_cast<const V*>(br + (rank < a.R ? 2 * rank : 0));
      }
    }
#pragma unroll
    for (int m = 0; m < kTiles; ++m) {
      const int row = row0 + __shfl(order, first + min(16 * m + c, count - 1), 64);
      at[m] = a.y + ((int64_t)row * a.ldy + n0) * Y::kSize;
      if (16 * m < count) Y::template load<FULL>(at[m], g, a.N - n0, held[m]);
    }
  }
  template <bool FULL>
  __device__ __forceinline__ void add(const LoraArgs& a, const ExpandSmem<DT, YT, RS>& sm, int n0, int count, float scale) {
    const int l = threadIdx.x & 63, c = l & 15, g = l >> 4;
#pragma unroll
    for (int m = 0; m < kTiles; ++m) {
      if (16 * m >= count) break;
      const int t = min(16 * m + c, count - 1);
      V piece[RS][kPieces];
#pragma unroll
      for (int s = 0; s < RS; ++s)
#pragma unroll
        for (int p = 0; p < kPieces; ++p) piece[s][p] = sm.u[p][t][4 * s + g];
      float v[16], by = scale;
      if constexpr (DT == MXFP4_TYPE_F16) by = by * sm.back[t];
      Y::unpack(held[m], v);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        mx::v4f acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < RS; ++s)
#pragma unroll
          for (int p = 0; p < kPieces; ++p) acc = Half<DT>::mfma(bv[j][s], piece[s][p], acc);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[4 * j + e] = v[4 * j + e] + by * acc[e];
      }
      if (16 * m + c < count) Y::template store<FULL>(at[m], g, a.N - n0, v);
    }
  }
};

template <int DT, int YT, int RS>
__global__ __launch_bounds__(kExpandThreads, RS == 4 || (RS == 2 && YT == MXFP4_TYPE_F32) ? 2 : 3) void expand_kernel(LoraArgs a) {
  typedef typename Half<DT>::V V;
  constexpr int kPieces = YT == MXFP4_TYPE_F32 ? 3 : 2;
  constexpr int kTiles = expand_tiles<YT, RS>();
  __shared__ __align__(16) ExpandSmem<DT, YT, RS> sm;
  const int tid = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int row0 = kBlock * blockIdx.y, n0 = kCols * blockIdx.x + 64 * wave;
  const int idx = adapter_of(a, row0);
  for_units(a, idx, a.unit, [&](int adapter, uint64_t rows, int first) {
    const int order = gathered(rows), count = min(__popcll(rows) - first, 16 * a.unit);
    const float scale = a.scale ? a.scale[adapter] : 1.0f;
    __syncthreads();
    // 8 ranks of a row to kAdders neighbouring threads, which share the partial sums; 4 RS such
    // groups to a row.
    auto sums = [&](auto adders) {
      constexpr int kAdders = decltype(adders)::value;
      for (int i0 = 0; i0 < 64 * kTiles * RS * kAdders; i0 += kExpandThreads) {
        const int i = i0 + tid, t = i / (4 * RS * kAdders), at = i / kAdders % (4 * RS);
        if (i0 >= 4 * RS * kAdders * count) break;
        const int row = row0 + __shfl(order, min(first + t, kBlock - 1), 64);
        float f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (t < count && 8 * at < a.R) {
          const float* p = a.part + (int64_t)row * a.R + 8 * at;
#pragma unroll 4
          for (int q = i % kAdders; q < a.splits; q += kAdders) {
            const float* pq = p + (int64_t)q * a.T * a.R;
            const mx::v4f lo = *reinterpret_cast<const mx::v4f*>(pq), hi = *reinterpret_cast<const mx::v4f*>(pq + 4);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              f[e] = f[e] + lo[e];
              f[4 + e] = f[4 + e] + hi[e];
            }
          }
        }
#pragma unroll
        for (int d = 1; d < kAdders; d <<= 1)
#pragma unroll
          for (int e = 0; e < 8; ++e) f[e] = f[e] + __shfl_xor(f[e], d, 64);
        if constexpr (DT == MXFP4_TYPE_F16) {
          uint32_t top = 0;
#pragma unroll
          for (int e = 0; e < 8; ++e) top = max(top, __builtin_bit_cast(uint32_t, f[e]) & 0x7fffffffu);
#pragma unroll
          for (int d = kAdders; d < 4 * RS * kAdders; d <<= 1) top = max(top, (uint32_t)__shfl_xor((int)top, d, 64));
          const int up = top == 0 || top >= 0x7f800000u ? 0 : min(14 + 127 - (int)(top >> 23), 126);
          const float by = __builtin_bit_cast(float, (uint32_t)(127 + up) << 23);
          if (at == 0 && i % kAdders == 0 && t < count) sm.back[t] = __builtin_bit_cast(float, (uint32_t)(127 - up) << 23);
#pragma unroll
          for (int e = 0; e < 8; ++e) f[e] *= by;
        }
        if (i % kAdders == 0 && t < count)
#pragma unroll
          for (int p = 0; p < kPieces; ++p) {
            V v;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              v[e] = Half<DT>::round(f[e]);
              f[e] = f[e] - (float)v[e];
            }
            sm.u[p][t][at] = v;
          }
      }
    };
    if (a.splits > 12)
      sums(std::integral_constant<int, (RS == 4 ? 4 : 8)>());  // a row's threads are of one wave
    else
      sums(std::integral_constant<int, 1>());
    Columns<DT, YT, RS> columns;
    const bool full = n0 + 64 <= a.N;  // the same for a wave
    if (full)
      columns.template load<true>(a, adapter, row0, n0, order, first, count);
    else
      columns.template load<false>(a, adapter, row0, n0, order, first, count);
    __syncthreads();
    if (full)
      columns.template add<true>(a, sm, n0, count, scale);
    else
      columns.template add<false>(a, sm, n0, count, scale);
  });
}

bool shape_ok(int64_t T, int64_t K, int64_t R) {
  constexpr int64_t kMax = (int64_t)1 << 20;
  return T >= 1 && T <= kMax && K >= 8 && K <= kMax && K % 8 == 0 && R >= 8 && R <= 128 && R % 8 == 0;
}
// Workgroups that share a block's units of `tiles` row tiles (see for_units). Most blocks of a
// prompt have one group, some two; a decode batch has as many as it has rows or adapters.
int workgroups_of(int64_t T, int64_t n, int tiles, int64_t target) {
  const int64_t blocks = mxh::cdiv(T, kBlock), most = kBlock / 16 / tiles + n - 1;
  if (blocks == 1) return (int)T;
  const int64_t z = target / blocks;
  return (int)(z < 1 ? 1 : z > 8 ? (8 < most ? 8 : most) : (z < most ? z : most));
}
// Workgroups that share K: enough to occupy the chip, each wave one step of 32 at least; from 65
// rows on at most 10, as every workgroup of expand adds up their sums (777 rows, K 2064, N 2113,
// R 24: 17 splits 6.4 + 10.0 us for the two kernels, 9 splits 5.2 + 8.8).
int splits_of(int64_t T, int64_t K) {
  const int64_t blocks = mxh::cdiv(T, kBlock), stages = mxh::cdiv(K, kStage), most = mxh::cdiv(stages, 2);
  const int64_t want = blocks == 1 ? mxh::cdiv(512, T < 32 ? T : 32) : blocks < 26 ? 10 : mxh::cdiv(256, blocks);
  return (int)mxh::cdiv(stages, mxh::cdiv(stages, want < most ? want : most));
}

template <int DT, int RT, int U>
hipError_t launch_shrink(LoraArgs& a, hipStream_t st) {
  void* args[] = {&a};
  return hipLaunchKernel((const void*)shrink_kernel<DT, RT, U>,
                         dim3((unsigned)a.splits, (unsigned)mxh::cdiv(a.T, kBlock), (unsigned)workgroups_of(a.T, a.n, kBlock / 16, 256)),
                         dim3(kShrinkThreads), args, 0, st);
}
template <int DT, int YT, int RS>
hipError_t launch_expand(LoraArgs& a, hipStream_t st) {
  a.unit = a.T <= 2048 ? 1 : expand_tiles<YT, RS>();
  void* args[] = {&a};
  return hipLaunchKernel((const void*)expand_kernel<DT, YT, RS>,
                         dim3((unsigned)mxh::cdiv(a.N, kCols), (unsigned)mxh::cdiv(a.T, kBlock),
                              (unsigned)workgroups_of(a.T, a.n, a.unit, a.unit == 1 ? 256 : 128)),
                         dim3(kExpandThreads), args, 0, st);
}
template <int DT, int YT>
int launch(LoraArgs& a, hipStream_t st) {
  hipError_t e = a.R <= 16   ? launch_shrink<DT, 1, 4>(a, st)
                 : a.R <= 32 ? launch_shrink<DT, 2, 4>(a, st)
                 : a.R <= 64 ? launch_shrink<DT, 4, 4>(a, st)
                             : launch_shrink<DT, 8, 2>(a, st);
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
  const int splits = splits_of(T, K);
  LoraArgs p{(uint8_t*)y, ldy,   (const uint8_t*)x, ldx * 2, (const uint8_t*)a, (const uint8_t*)b, index, scale,
             (float*)workspace, (int)T, (int)N, (int)K, (int)R, (int)n,
             0, splits, (int)mxh::cdiv(mxh::cdiv(K, kStage), splits)};
  const hipStream_t st = (hipStream_t)stream;
  if (xtype == MXFP4_TYPE_BF16)
    return ytype == MXFP4_TYPE_F32 ? launch<MXFP4_TYPE_BF16, MXFP4_TYPE_F32>(p, st)
                                   : launch<MXFP4_TYPE_BF16, MXFP4_TYPE_BF16>(p, st);
  return ytype == MXFP4_TYPE_F32 ? launch<MXFP4_TYPE_F16, MXFP4_TYPE_F32>(p, st)
                                 : launch<MXFP4_TYPE_F16, MXFP4_TYPE_F16>(p, st);
}
