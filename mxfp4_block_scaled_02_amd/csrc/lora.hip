// lora_add: y[t] += scale * (x[t] . A^T) . B^T with the adapter (A, B) of each row, for
// low-rank adapters of many requests beside a shared projection.
//
// shrink: x . A^T in fp32 partial sums [split][T][R]. expand: 256 columns to a workgroup, which
// adds the partial sums in their order, holds them as 16-bit pieces and multiplies with B. Both
// take units of up to 64 rows with the same adapter, wherever they lie among the rows, in 16-row
// tiles: A and B are read once for a unit, and no row meets another one's adapter. The units of
// up to 64 rows are found by every wave itself; of more by a launch in front (plan).
//
// Measured on the MI355X (bf16; a copy of memory reaches 5.2 TB/s):
//   T    K    N    R   n   us for the launches   what bounds it
//   1    7168 2112 16  8   3.6 + 4.8             latency (a call takes 11 us on the host)
//   64   7168 4096 32  24  6.7 + 5.2             latency: 12 and 7 MB
//   777  2064 2113 24  5   3.6 + 4.9 + 7.6       latency (x fp16, y fp32)
//   4096 7168 4096 64  8   4.9 + 16 + 21.5       x once at 3.6 TB/s; y in and out at 3.1, beside the
//                                                partial sums, which 16 workgroups add up each
//   4096 4096 4096 32  28  5.5 + 12.8 + 18.3     the same (adapters in any order of rows)
#include <type_traits>

#include "host_common.hpp"
#include "mx_device.hpp"

namespace {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef u32x4 u32x4_at4 __attribute__((aligned(4)));
typedef u32x4 u32x4_at2 __attribute__((aligned(2)));

constexpr int kFew = 64;            // rows of a call that a wave looks through by itself
constexpr int kBlock = 4096;        // rows of a block of plan
constexpr int kMaxN = 4096;
constexpr int kUnit = 64;           // rows with one adapter that go together at most
constexpr int kThreads = 256;
constexpr int kStage = 64;          // k of a step of shrink: 128 bytes, a cache line of a row
constexpr int kShrinkWaves = 4;
static_assert(kThreads == 64 * kShrinkWaves);
constexpr int kExpandWaves = 4;
static_assert(kThreads == 64 * kExpandWaves);
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
  int tiles;  // 16-row tiles that a workgroup of expand takes together
  struct Unit* units;
  int slots;          // units that a block may have
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

// The adapter of a row, -1 without one.
__device__ __forceinline__ int adapter_of(const LoraArgs& a, int row) {
  const int i = row < a.T ? a.index[row] : -1;
  return (uint32_t)i < (uint32_t)a.n ? i : -1;
}
// Up to 64 rows with one adapter.
struct __align__(16) Unit {
  int adapter, count;     // no rows in a slot that is not needed
  uint16_t rows[kUnit];   // within the block
};
// At most: a unit for every 64 rows, and one that is not full for each adapter.
__host__ __device__ inline int64_t slots_of(int64_t T, int64_t n) {
  const int64_t here = T < kBlock ? T : kBlock;
  return here / kUnit + (n < here ? n : here);
}

// The units of a block of rows, by rising adapter, the rows of each in an order that the indices
// alone decide: a counting sort. A wave counts the adapters of its rows (every 16th run of 64;
// which rows of a run have the same adapter follows from a ballot for each bit of the index), the
// counts are added up over the waves, and over the adapters the units. Latency: 777 rows of 5
// adapters 3.6 us (4.0 with room for 4096 rows), 2000 of 28 4.2 (4.8), 4096 of 28 5.5; a round for
// each adapter in a wave's rows instead of the ballots took 3.3, 8.2 and 13.7. Past 64 rows it pays:
// 64 rows of 24 adapters, K 7168, N 4096, take 6.7 + 5.2 us without it, and 6.0 + 6.5 beside the
// plan with it; but without it each row is a workgroup that looks through all rows.
constexpr int kPlanWaves = 16;
template <int kWords>  // runs of 64 rows to a wave
__global__ __launch_bounds__(64 * kPlanWaves) void plan_kernel(LoraArgs a) {
  __shared__ uint16_t before[kPlanWaves][kMaxN];  // rows with the adapter in the waves before
  __shared__ uint16_t unit0[kMaxN];               // the adapter's first unit
  __shared__ int sums[kPlanWaves];
  const int tid = threadIdx.x, l = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const uint64_t below = ((uint64_t)1 << l) - 1;
  const int row0 = kBlock * blockIdx.x;
  auto row_of = [&](int w) { return 64 * (kPlanWaves * w + wave) + l; };
  Unit* const units = a.units + (int64_t)blockIdx.x * a.slots;
  int idx[kWords], rank[kWords];
#pragma unroll
  for (int w = 0; w < kWords; ++w) idx[w] = adapter_of(a, row0 + row_of(w));
  for (int i = l; i < a.n; i += 64) before[wave][i] = 0;
  const int bits = 32 - __builtin_clz(a.n - 1 | 1);
#pragma unroll
  for (int w = 0; w < kWords; ++w) {
    uint64_t same = __ballot(idx[w] >= 0);  // the run's rows with the lane's adapter
    for (int b = 0; b < bits; ++b) {
      const bool bit = idx[w] >> b & 1;
      const uint64_t set = __ballot(bit);
      same &= bit ? set : ~set;
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");  // a lane reads what another has written
    if (idx[w] >= 0) {
      const int upto = before[wave][idx[w]];
      rank[w] = upto + __popcll(same & below);
      if ((same & below) == 0) before[wave][idx[w]] = (uint16_t)(upto + __popcll(same));
    }
  }
  __syncthreads();
  int units_before = 0;  // of the adapters of the rounds before
  for (int i0 = 0; i0 < a.n; i0 += 64 * kPlanWaves) {
    const int i = i0 + tid;
    int total = 0;
    if (i < a.n)
#pragma unroll
      for (int w = 0; w < kPlanWaves; ++w) {
        const int c = before[w][i];
        before[w][i] = (uint16_t)total;
        total += c;
      }
    const int count = (total + kUnit - 1) / kUnit;
    int upto = count;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(upto, d, 64);
      if (l >= d) upto += o;
    }
    if (l == 63) sums[wave] = upto;
    __syncthreads();
    int first = units_before + upto - count;
#pragma unroll
    for (int w = 0; w < kPlanWaves; ++w) {
      if (w < wave) first += sums[w];
      units_before += sums[w];
    }
    if (i < a.n) unit0[i] = (uint16_t)first;
    for (int u = 0; u < count; ++u) {
      units[first + u].adapter = i;
      units[first + u].count = min(total - kUnit * u, kUnit);
    }
    __syncthreads();
  }
  for (int u = units_before + tid; u < a.slots; u += 64 * kPlanWaves) units[u].count = 0;
#pragma unroll
  for (int w = 0; w < kWords; ++w)
    if (idx[w] >= 0) {
      const int at = before[wave][idx[w]] + rank[w];
      units[unit0[idx[w]] + at / kUnit].rows[at % kUnit] = (uint16_t)row_of(w);
    }
}

// Calls f(adapter, row0, order, count) for the unit of this workgroup, if it has one, by all waves
// alike: lane p < count's `order` is the unit's p-th row, from row0 on. Units are taken apart into
// pieces of up to `size` rows. FEW (T <= 64): a workgroup (blockIdx.z) for each row, which goes on
// if its row is the first of a piece.
template <bool FEW, typename F>
__device__ __forceinline__ void with_unit(const LoraArgs& a, int size, F f) {
  const int l = threadIdx.x & 63;
  if constexpr (FEW) {
    const int idx = adapter_of(a, l);
    const int r = blockIdx.z, adapter = __builtin_amdgcn_readlane(idx, r);
    if (adapter < 0) return;
    const uint64_t rows = __ballot(idx == adapter), below = ((uint64_t)1 << l) - 1;
    const int first = __popcll(rows & (((uint64_t)1 << r) - 1));
    if (first % size != 0) return;
    // Lane p gets the p-th of the rows (past the last one: some other row), then the first + p-th.
    const int at = (rows >> l) & 1 ? __popcll(rows & below) : __popcll(rows) + __popcll(~rows & below);
    const int order = __builtin_amdgcn_ds_permute(4 * at, l);
    f(adapter, 0, __shfl(order, min(first + l, 63), 64), min(__popcll(rows) - first, size));
  } else {
    const int pieces = kUnit / size, first = (int)(blockIdx.z % pieces) * size;
    const Unit& u = a.units[(int64_t)blockIdx.y * a.slots + blockIdx.z / pieces];
    const int adapter = u.adapter, count = min(u.count - first, size), order = u.rows[min(first + l, kUnit - 1)];
    if (count > 0) f(adapter, kBlock * (int)blockIdx.y, order, count);
  }
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
  u32x4 line[2][kUnit + 16 * RT][8];
};
template <int DT, int RT>
__device__ __forceinline__ void shrink_tile(const LoraArgs& a, int adapter, int row0, int order, int count, int begin,
                                            int end, TileSmem<RT>& sm, mx::v4f (&acc)[RT]) {
  typedef typename Half<DT>::V V;
  constexpr int kLoads = (8 * (kUnit + 16 * RT) + kThreads - 1) / kThreads;
  constexpr int kRows = kThreads / 8;  // rows that a load of all threads covers
  const int tid = threadIdx.x, l = tid & 63, c = l & 15, g = l >> 4, wave = tid >> 6;
  const int p = tid & 7, slot = p ^ ((tid >> 4) & 7);
  const uint8_t* src[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int r = kRows * i + (tid >> 3);
    src[i] = i < kUnit / kRows
                 ? a.x + (int64_t)(row0 + __shfl(order, min(r, count - 1), 64)) * a.ldx
                 : a.a + ((int64_t)adapter * a.R + min(r - kUnit, a.R - 1)) * a.K * 2;
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
      if (r < kUnit + 16 * RT) sm.line[buf][r][slot] = in || i >= kUnit / kRows ? v[i] : u32x4{0, 0, 0, 0};
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
        for (int r = 0; r < RT; ++r) av[kk][r] = __builtin_bit_cast(V, sm.line[i & 1][kUnit + 16 * r + c][at]);
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

// The second launch bound keeps the sums out of accumulation registers, and the moves to and from them.
template <int DT, int RT, int U, bool FEW>
__global__ __launch_bounds__(kThreads, RT == 8 ? 2 : 3) void shrink_kernel(LoraArgs a) {
  __shared__ union {
    TileSmem<RT> tile;
    mx::v4f red[kShrinkWaves][RT][64];
  } sm;
  const int tid = threadIdx.x, l = tid & 63, c = l & 15, g = l >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int q = blockIdx.x;
  const int stages = (a.K + kStage - 1) / kStage, begin = q * a.slice, end = min(begin + a.slice, stages);
  with_unit<FEW>(a, kUnit, [&](int adapter, int row0, int order, int count) {
    mx::v4f acc[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) acc[r] = mx::v4f{0.f, 0.f, 0.f, 0.f};
    auto store = [&](int t, int r, const mx::v4f& v) {
      const int row = row0 + __shfl(order, min(t, count - 1), 64), rank = 16 * r + 4 * g;
      if (t < count && rank < a.R) *reinterpret_cast<mx::v4f*>(a.part + ((int64_t)q * a.T + row) * a.R + rank) = v;
    };
    // 24 rows of 6 adapters, K 4096: 3.6 us, 4.4 if all went through LDS; 64 of 24, K 7168: 6.7 and 8.1.
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
  // Ranks of a row in pieces of 8, piece p of row t at p ^ swizzle(t): see TileSmem.
  typename Half<DT>::V u[YT == MXFP4_TYPE_F32 ? 3 : 2][16 * expand_tiles<YT, RS>()][4 * RS];
  static __device__ __forceinline__ int swizzle(int t) {
    return RS == 1 ? 0 : RS == 2 ? t >> 1 & 7 : (t & 1) << 3 | (t & 2) << 1 | (t >> 2 & 3);
  }
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
  __device__ __forceinline__ void load(const LoraArgs& a, int adapter, int row0, int n0, int order, int count) {
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
      const int row = row0 + __shfl(order, min(16 * m + c, count - 1), 64);
      at[m] = a.y + ((int64_t)row * a.ldy + n0) * Y::kSize;
      if (16 * m < count) Y::template load<FULL>(at[m], g, a.N - n0, held[m]);
    }
  }
  template <bool FULL>
  __device__ __forceinline__ void add(const LoraArgs& a, const ExpandSmem<DT, YT, RS>& sm, int n0, int count,
                                      float scale) {
    const int l = threadIdx.x & 63, c = l & 15, g = l >> 4;
#pragma unroll
    for (int m = 0; m < kTiles; ++m) {
      if (16 * m >= count) break;
      const int t = min(16 * m + c, count - 1);
      V piece[RS][kPieces];
#pragma unroll
      for (int s = 0; s < RS; ++s)
#pragma unroll
        for (int p = 0; p < kPieces; ++p) piece[s][p] = sm.u[p][t][(4 * s + g) ^ sm.swizzle(t)];
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

template <int DT, int YT, int RS, bool FEW>
__global__ __launch_bounds__(kThreads, RS == 4 || (RS == 2 && YT == MXFP4_TYPE_F32) ? 2 : 3) void expand_kernel(
    LoraArgs a) {
  typedef typename Half<DT>::V V;
  constexpr int kPieces = YT == MXFP4_TYPE_F32 ? 3 : 2;
  constexpr int kTiles = expand_tiles<YT, RS>();
  __shared__ __align__(16) ExpandSmem<DT, YT, RS> sm;
  const int tid = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n0 = kCols * blockIdx.x + 64 * wave;
  with_unit<FEW>(a, 16 * a.tiles, [&](int adapter, int row0, int order, int count) {
    const float scale = a.scale ? a.scale[adapter] : 1.0f;
    __syncthreads();
    // 8 ranks of a row to kAdders neighbouring threads, which share the partial sums; 4 RS such
    // groups to a row.
    auto sums = [&](auto adders) {
      constexpr int kAdders = decltype(adders)::value;
      for (int i0 = 0; i0 < 64 * kTiles * RS * kAdders; i0 += kThreads) {
        const int i = i0 + tid, t = i / (4 * RS * kAdders), at = i / kAdders % (4 * RS);
        if (i0 >= 4 * RS * kAdders * count) break;
        const int row = row0 + __shfl(order, min(t, count - 1), 64);
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
          if (at == 0 && i % kAdders == 0 && t < count)
            sm.back[t] = __builtin_bit_cast(float, (uint32_t)(127 - up) << 23);
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
            sm.u[p][t][at ^ sm.swizzle(t)] = v;
          }
      }
    };
    // One thread for a row's 8 ranks is less work, several shorten the chain of loads: one row, 56 splits
    // 8.6 us with one thread, 4.8 with 8; 4096 rows, 4 splits 21.4 and 35.6.
    if (a.splits > 12)
      sums(std::integral_constant<int, (RS == 4 ? 4 : 8)>());  // a row's threads are of one wave
    else
      sums(std::integral_constant<int, 1>());
    Columns<DT, YT, RS> columns;
    const bool full = n0 + 64 <= a.N;  // the same for a wave
    if (full)
      columns.template load<true>(a, adapter, row0, n0, order, count);
    else
      columns.template load<false>(a, adapter, row0, n0, order, count);
    __syncthreads();
    if (full)
      columns.template add<true>(a, sm, n0, count, scale);
    else
      columns.template add<false>(a, sm, n0, count, scale);
  });
}

bool shape_ok(int64_t T, int64_t K, int64_t R, int64_t n) {
  constexpr int64_t kMax = (int64_t)1 << 20;
  return T >= 1 && T <= kMax && K >= 8 && K <= kMax && K % 8 == 0 && R >= 8 && R <= 128 && R % 8 == 0 &&
         n >= 1 && n <= kMaxN;
}
// Workgroups that share K: enough to occupy the chip, each wave one step of 32 at least; from 65
// rows on at most 10, as every workgroup of expand adds up their sums (777 rows, K 2064, N 2113,
// R 24: 17 splits 6.4 + 10.0 us for the two kernels, 9 splits 5.2 + 8.8). Half and double as many:
// 64 rows of 24 adapters, K 7168, 6.7 + 5.2 us against 8.0 + 4.9 and 9.3 + 6.2; 4096 rows, K 7168,
// R 64, 16.0 + 21.2 against 23.3 + 20.2 and 17.5 + 24.9.
int splits_of(int64_t T, int64_t K) {
  const int64_t stages = mxh::cdiv(K, kStage), most = mxh::cdiv(stages, 2);
  const int64_t want = T <= kFew ? mxh::cdiv(512, T < 32 ? T : 32) : T < 26 * 64 ? 10 : mxh::cdiv(16384, T);
  return (int)mxh::cdiv(stages, mxh::cdiv(stages, want < most ? want : most));
}

// The grid's y and z for pieces of `rows` rows (see with_unit).
dim3 grid_of(const LoraArgs& a, unsigned x, int rows) {
  if (a.T <= kFew) return dim3(x, 1, (unsigned)a.T);
  return dim3(x, (unsigned)mxh::cdiv(a.T, kBlock), (unsigned)(a.slots * (kUnit / rows)));
}
template <int DT, int RT, int U>
hipError_t launch_shrink(LoraArgs& a, hipStream_t st) {
  void* args[] = {&a};
  const void* f =
      a.T <= kFew ? (const void*)shrink_kernel<DT, RT, U, true> : (const void*)shrink_kernel<DT, RT, U, false>;
  return hipLaunchKernel(f, grid_of(a, (unsigned)a.splits, kUnit), dim3(kThreads), args, 0, st);
}
template <int DT, int YT, int RS>
hipError_t launch_expand(LoraArgs& a, hipStream_t st) {
  // A whole unit while that occupies the chip (4096 rows of 8 adapters, R 64: 21.6 us, 26.9 a tile at a
  // time; 256 of 24, R 16 5.4 and 6.6), else a tile (227 rows of 2 adapters, N 3797: 6.2, whole units 12.5;
  // 533 of 3, N 7088, R 32 6.8 and 11.4). All blocks of rows count (65536 rows of 8 adapters, K and N 1024,
  // R 32: 99 us for the call, 110 a tile at a time; 8192, R 16 20.4 and 21.4, in spans 23.3 and 23.0).
  a.tiles = mxh::cdiv(a.N, kCols) * slots_of(a.T, a.n) * mxh::cdiv(a.T, kBlock) < 384 ? 1 : expand_tiles<YT, RS>();
  void* args[] = {&a};
  const void* f =
      a.T <= kFew ? (const void*)expand_kernel<DT, YT, RS, true> : (const void*)expand_kernel<DT, YT, RS, false>;
  return hipLaunchKernel(f, grid_of(a, (unsigned)mxh::cdiv(a.N, kCols), 16 * a.tiles), dim3(kThreads),
                         args, 0, st);
}
size_t part_bytes(int64_t T, int64_t K, int64_t R) { return (size_t)splits_of(T, K) * (size_t)T * (size_t)R * 4; }

template <int DT, int YT>
int launch(LoraArgs& a, hipStream_t st) {
  hipError_t e = hipSuccess;
  if (a.T > kFew) {
    void* args[] = {&a};
    const void* f = a.T <= 1024   ? (const void*)plan_kernel<1>
                    : a.T <= 2048 ? (const void*)plan_kernel<2>
                                  : (const void*)plan_kernel<kBlock / (64 * kPlanWaves)>;
    e = hipLaunchKernel(f, dim3((unsigned)mxh::cdiv(a.T, kBlock)), dim3(64 * kPlanWaves), args, 0, st);
    if (e != hipSuccess) return MXFP4_ERR_HIP;
  }
  e = a.R <= 16   ? launch_shrink<DT, 1, 4>(a, st)
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

extern "C" size_t lora_add_workspace_bytes(int64_t T, int64_t K, int64_t R, int64_t n) {
  if (!shape_ok(T, K, R, n)) return 0;
  return part_bytes(T, K, R) + (T <= kFew ? 0 : (size_t)(mxh::cdiv(T, kBlock) * slots_of(T, n)) * sizeof(Unit));
}

extern "C" int lora_add(void* y, int64_t ldy, int ytype, const void* x, int64_t ldx, int xtype, const void* a,
                        const void* b, const int32_t* index, const float* scale, int64_t T, int64_t N, int64_t K,
                        int64_t R, int64_t n, void* workspace, size_t workspace_bytes, void* stream) {
  if (T < 1 || N < 1 || n < 1) return MXFP4_ERR_SHAPE;  // first: an empty tensor's pointer may be NULL
  if (!y || !x || !a || !b || !index) return MXFP4_ERR_NULL;
  if (xtype != MXFP4_TYPE_BF16 && xtype != MXFP4_TYPE_F16) return MXFP4_ERR_ARG;
  if (ytype != xtype && ytype != MXFP4_TYPE_F32) return MXFP4_ERR_ARG;
  constexpr int64_t kMax = (int64_t)1 << 20, kMaxLd = (int64_t)1 << 36;
  if (!shape_ok(T, K, R, n) || N > kMax || ldx < K || ldx > kMaxLd || ldy < N || ldy > kMaxLd)
    return MXFP4_ERR_SHAPE;
  if (!mxh::aligned(x, 16) || ldx % 8 != 0 || !mxh::aligned(a, 16) || !mxh::aligned(b, 16) ||
      !mxh::aligned(y, ytype == MXFP4_TYPE_F32 ? 4 : 2) || !mxh::aligned(index, 4) || !mxh::aligned(scale, 4))
    return MXFP4_ERR_ALIGN;
  if (!workspace || !mxh::aligned(workspace, 16) || workspace_bytes < lora_add_workspace_bytes(T, K, R, n))
    return MXFP4_ERR_WORKSPACE;
  const int splits = splits_of(T, K);
  LoraArgs p{(uint8_t*)y, ldy, (const uint8_t*)x, ldx * 2, (const uint8_t*)a, (const uint8_t*)b, index, scale,
             (float*)workspace, (int)T, (int)N, (int)K, (int)R, (int)n,
             0, (Unit*)((uint8_t*)workspace + part_bytes(T, K, R)), (int)slots_of(T, n), splits,
             (int)mxh::cdiv(mxh::cdiv(K, kStage), splits)};
  const hipStream_t st = (hipStream_t)stream;
  if (xtype == MXFP4_TYPE_BF16)
    return ytype == MXFP4_TYPE_F32 ? launch<MXFP4_TYPE_BF16, MXFP4_TYPE_F32>(p, st)
                                   : launch<MXFP4_TYPE_BF16, MXFP4_TYPE_BF16>(p, st);
  return ytype == MXFP4_TYPE_F32 ? launch<MXFP4_TYPE_F16, MXFP4_TYPE_F32>(p, st)
                                 : launch<MXFP4_TYPE_F16, MXFP4_TYPE_F16>(p, st);
}
