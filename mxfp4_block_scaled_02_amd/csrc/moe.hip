// moe_a16w4: the experts' gated MLP of a mixture of experts on MXFP4 weights for a few
// tokens (bf16 activations; the weights' bytes bound it, so the activations are not
// quantised).
//
// Two or three launches: gate, up and SwiGLU into h; the down product; where a token's experts
// are not added up in that product (tokens_kernel), their sum (combine_kernel). A workgroup has
// some columns of one expert, finds the rows that take it in `ids` by itself, and reads its part of
// the weight once for up to 16 (few_kernel) or 64 (many_kernel) of them: no launch sorts the rows,
// and nothing goes back to the host. Up to 10 rows an expert on average one workgroup takes all of an
// expert's rows in turns of 16, so that an expert with many more of them holds the call up (256 tokens,
// k 8, 256 experts, H 2048, I 512: 105 us with 8 rows of each, 140 with 204 of one).
//
// Measured on the MI355X (a linear read of memory reaches 5.5 to 5.8 TB/s, a copy 5.2):
//   T   k  E   H    I     us for the launches    what bounds it
//   1   8  32  7168 2048  21.6 + 15.2            the weights of 8 experts, 187 MB: 5.8 and 4.1 TB/s
//   64  8  64  7168 2048  181 + 98 + 4.9         all weights, 1.50 GB: 5.5 and 5.1 TB/s
//   37  3  24  2112 1056  16.3 + 11.3 + 3.9      latency: one pass of 33 and 17 workgroups an expert
//   124 4  6   2240 1568  42.3 + 4.6             latency: 150 and 108 workgroups for 32 rows each
//   256 4  32  2048 1024  21.9 + 20.4 + 4.7      vector instructions, 60 % of the cycles: conversions
//   2   2  8   512  256   4.2 + 4.7              latency (a call takes 11 us on the host)
#include "host_common.hpp"
#include "mx_device.hpp"

// Sums in the order that the code gives them, whichever variant computes a row.
#pragma clang fp contract(off)

namespace {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
constexpr int kMaxE = 1024;
constexpr int kNonTemporal = 2;  // the nt bit of the buffer instructions

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
  uint8_t* h;   // bf16 [2, pairs, I]
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

// The pairs (t, j) of a slot's expert. A launch has a slot for each expert (slot_is_expert: it is
// known at once) or, where there are fewer pairs, for each pair: then a slot stands for its own
// pair's expert (up to 64 pairs: one ballot, no pass over LDS; 2 tokens, k 2, E 8, H 512: 4.2 us
// for the launch and 5.7 without, one token, k 8, H 7168: 21.6 and 23.1) or for the slot-th of the
// experts that are taken. `list` has the slot's pairs in an order that the ids alone decide.
// Returns their number, 0 for a slot to skip.
struct Rows {
  uint32_t bits[kMaxE / 32];
  int count[kWaves];
  uint16_t list[MXFP4_MOE_MAX_PAIRS];
};
__device__ __forceinline__ bool slot_is_expert(const MoeArgs& a) { return a.T * a.k >= a.E; }
__device__ __forceinline__ int find_rows(const MoeArgs& a, int slot, Rows& s, int& expert) {
  const int tid = threadIdx.x, l = tid & 63, P = a.T * a.k;
  if (P <= 64 && !slot_is_expert(a)) {
    // It goes on if its pair is the first with the expert.
    const int id = l < P ? a.ids[l] : -1;
    expert = __builtin_amdgcn_readlane(id, slot);
    const uint64_t mine = __ballot(id == expert);
    if ((uint32_t)expert >= (uint32_t)a.E || __ffsll((unsigned long long)mine) - 1 != slot) return 0;
    if (tid < 64 && id == expert) s.list[__popcll(mine & (((uint64_t)1 << l) - 1))] = (uint16_t)l;
    __syncthreads();
    return __popcll(mine);
  }
  // A thread's ids stay in registers from one pass to the next (4096 pairs: 16 to a thread).
  constexpr int kEach = MXFP4_MOE_MAX_PAIRS / kThreads;
  const int wave = tid >> 6, each = (P + kThreads - 1) / kThreads;
  uint32_t id[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i)
    id[i] = i < each && tid + kThreads * i < P ? (uint32_t)a.ids[tid + kThreads * i] : ~0u;
  if (slot_is_expert(a)) {
    expert = slot;
  } else {  // the slot-th of the experts that any pair takes, in rising order
    if (tid < kMaxE / 32) s.bits[tid] = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kEach; ++i)
      if (i < each && id[i] < (uint32_t)a.E) atomicOr(&s.bits[id[i] >> 5], 1u << (id[i] & 31));
    __syncthreads();
    const uint32_t word = l < kMaxE / 32 ? s.bits[l] : 0;
    int before = 0, at = 0;  // experts before word `at`
    uint32_t w = 0;
    for (; at < kMaxE / 32; ++at) {
      w = (uint32_t)__builtin_amdgcn_readlane((int)word, at);
      if (before + __popc(w) > slot) break;
      before += __popc(w);
    }
    if (at == kMaxE / 32) return 0;  // the same on every thread
    const bool mine = l < 32 && (w >> l & 1) && __popc(w & ((1u << l) - 1)) == slot - before;
    expert = 32 * at + __ffsll((unsigned long long)__ballot(mine)) - 1;
  }
  int sum = 0;  // of this wave
#pragma unroll
  for (int i = 0; i < kEach; ++i)
    if (i < each) sum += __popcll(__ballot(id[i] == (uint32_t)expert));
  if (l == 0) s.count[wave] = sum;
  __syncthreads();
  int n = 0, pos = 0;
#pragma unroll
  for (int u = 0; u < kWaves; ++u) {
    if (u == wave) pos = n;
    n += s.count[u];
  }
#pragma unroll
  for (int i = 0; i < kEach; ++i)
    if (i < each) {
      const uint64_t has = __ballot(id[i] == (uint32_t)expert);
      if (id[i] == (uint32_t)expert)
        s.list[pos + __popcll(has & (((uint64_t)1 << l) - 1))] = (uint16_t)(tid + kThreads * i);
      pos += __popcll(has);
    }
  __syncthreads();
  return n;
}

__device__ __forceinline__ v8bf expand(uint32_t codes, float scale) {
  const mx::v2bf p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 0);
  const mx::v2bf p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 1);
  const mx::v2bf p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 2);
  const mx::v2bf p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 3);
  return v8bf{p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
}
__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const uint8_t* base, int bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(base), (short)0, bytes, 0x00020000);
}

// A 32-column tile of a packed weight. Loads go through buffer resources over the tile's units
// and scales: what lies past its K reads zeros, and makes no traffic.
struct Tile {
  __amdgpu_buffer_rsrc_t units, scales;
};
__device__ __forceinline__ Tile tile_at(const Packed& p, int tile) {
  return Tile{make_rsrc(p.units + (int64_t)tile * p.KU * 1024, p.KU * 1024),
              make_rsrc(p.scales + (int64_t)tile * p.KG * 256, p.KG * 256)};
}

// Lane l of a wave supplies column l % 16 of each of NC 16-column groups (group c: half c % 2
// of tile c / 2), and row l % 16 of the activations, both for k = 32 * (l / 16) .. +31 of a
// 128-k step. The weights are the matrix instruction's first operand: result register i of
// lane l is column 4 * (l / 16) + i of the group for row l % 16.
// A step's codes and the dwords of scales that it shares with its neighbour.
template <int NC>
struct Codes {
  u32x4 w[NC];
  uint32_t scale[NC];
};
// Group i is half i % 2 of tile i / 2; with `split` half `h` of tile i.
template <int NC, bool SPLIT = false>
__device__ __forceinline__ void load_codes(const Tile* t, int step, Codes<NC>& c, int h = 0) {
  const int l = threadIdx.x & 63, g = l >> 4, lane = 32 * (g & 1) + (l & 15);
#pragma unroll
  for (int i = 0; i < NC; ++i)
    c.scale[i] = __builtin_amdgcn_raw_buffer_load_b32(t[SPLIT ? i : i / 2].scales,
                                                      256 * (step >> 1) + 4 * (lane + 16 * (SPLIT ? h : i & 1)), 0,
                                                      kNonTemporal);
#pragma unroll
  for (int i = 0; i < NC; ++i)
    c.w[i] = __builtin_amdgcn_raw_buffer_load_b128(
        t[SPLIT ? i : i / 2].units, 2048 * step + 1024 * (g >> 1) + 16 * (lane + 16 * (SPLIT ? h : i & 1)), 0,
        kNonTemporal);
}
// acc[r][i] += rows 16 r .. times column group i over a step; f(r, pl, j): the lane's elements
// 8 j .. 8 j + 7 of its row of tile r, of the row's PL parts whose sum it is.
template <int NT, int PL, int NC, typename F>
__device__ __forceinline__ void multiply(const Codes<NC>& c, int step, F f, mx::v4f (&acc)[NT][NC]) {
  const int byte = 16 * (step & 1) + 8 * ((threadIdx.x & 63) >> 5);  // the lane's unit of the step's two
  float e[NC];
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    uint32_t sc = c.scale[i];
    asm volatile("" : "+v"(sc));  // else the shift follows its load, which it would wait for, a step before its use
    e[i] = __builtin_bit_cast(float, (sc >> byte & 0xffu) << 23);
  }
  // A quarter's operands are asked for before the products of the quarter in front of it.
  v8bf x[2][NT][PL];
  auto get = [&](int j) {
#pragma unroll
    for (int r = 0; r < NT; ++r)
#pragma unroll
      for (int pl = 0; pl < PL; ++pl) x[j & 1][r][pl] = f(r, pl, j);
  };
  get(0);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (j < 3) get(j + 1);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const v8bf w = expand(c.w[i][j], e[i]);
#pragma unroll
      for (int pl = 0; pl < PL; ++pl)
#pragma unroll
        for (int r = 0; r < NT; ++r)
          acc[r][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, x[j & 1][r][pl], acc[r][i], 0, 0, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
  }
}

template <int NT, int NC>
__device__ __forceinline__ void clear(mx::v4f (&acc)[NT][NC]) {
#pragma unroll
  for (int r = 0; r < NT; ++r)
#pragma unroll
    for (int i = 0; i < NC; ++i) acc[r][i] = mx::v4f{0.f, 0.f, 0.f, 0.f};
}

// h of a pair is kept as two bf16 parts, the value's rounding and the rest's (within 2^-17 of it
// together): one part alone would put an error into y as large as y's own rounding. The second
// part costs a matrix instruction more (256 tokens, k 4, 32 experts, H 2048, I 1024: 48.6 us for the
// call with one, 49.3 with both).
__device__ __forceinline__ const uint8_t* h_row(const MoeArgs& a, int part, int pair) {
  return a.h + ((int64_t)part * a.T * a.k + pair) * a.I * 2;
}
// Four columns of h of a pair, times the pair's weight.
__device__ __forceinline__ void store_h(const MoeArgs& a, int pair, int col, const mx::v4f& g, const mx::v4f& u) {
  const float w = a.weights[pair];
  float h[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) h[e] = g[e] / (1.0f + expf(-g[e])) * u[e] * w;
#pragma unroll
  for (int part = 0; part < 2; ++part) {
    const u32x2 v = {mx::pack_bf16x2(h[0], h[1]), mx::pack_bf16x2(h[2], h[3])};
    *reinterpret_cast<u32x2*>(const_cast<uint8_t*>(h_row(a, part, pair)) + 2 * col) = v;
    h[0] -= __builtin_bit_cast(float, v.x << 16);
    h[1] -= __builtin_bit_cast(float, v.x & 0xffff0000u);
    h[2] -= __builtin_bit_cast(float, v.y << 16);
    h[3] -= __builtin_bit_cast(float, v.y & 0xffff0000u);
  }
}

// ---------------------------------------------------------------------------
// Gate and up, few rows to an expert: 32 columns of each to a workgroup, K split over its waves
// ---------------------------------------------------------------------------
// Steps of 128 k: wave, wave + kWaves, .... Activations come straight from L2. No step is fetched
// ahead: the registers that it would take leave room for fewer waves, which hide more (64
// tokens through 64 experts of H 7168, I 2048: no step ahead 177 us, one 184, three 200).
struct FewSmem {
  Rows rows;
  mx::v4f red[kWaves][4][64];
};
__global__ __launch_bounds__(kThreads) void few_kernel(MoeArgs a) {
  __shared__ __align__(16) FewSmem sm;
  const int tid = threadIdx.x, l = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), b = blockIdx.x;
  int expert = 0;
  const int n = find_rows(a, blockIdx.y, sm.rows, expert);
  if (n == 0) return;
  const Packed p = packed(a.w13 + __builtin_amdgcn_readfirstlane(expert) * a.stride13, 2 * a.I, a.H);
  const Tile t[2] = {tile_at(p, b), tile_at(p, a.I / 32 + b)};
  for (int first = 0; first < n; first += 16) {
    const int at = first + (l & 15), pair = sm.rows.list[min(at, n - 1)];
    const uint8_t* row = a.x + pair / a.k * a.ldx;
    mx::v4f acc[1][4];
    clear(acc);
    const int steps = (a.H + 127) / 128, g = l >> 4;
#pragma unroll 1
    for (int s = wave; s < steps; s += kWaves) {
      Codes<4> code;
      v8bf x[4];
      load_codes<4>(t, s, code);
      const int k = min(128 * s + 32 * g, a.H - 32);  // past the end: the codes are zero
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = *reinterpret_cast<const v8bf*>(row + 2 * (int64_t)k + 16 * j);
      multiply<1, 1, 4>(code, s, [&](int, int, int j) { return x[j]; }, acc);
    }
    __syncthreads();  // the last rows' sums
#pragma unroll
    for (int i = 0; i < 4; ++i) sm.red[wave][i][l] = acc[0][i];
    __syncthreads();
    if (wave < 2) {  // a half of the columns each
      mx::v4f g = sm.red[0][wave][l], u = sm.red[0][2 + wave][l];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) {
        g = g + sm.red[w][wave][l];
        u = u + sm.red[w][2 + wave][l];
      }
      if (at < n) store_h(a, pair, 32 * b + 16 * wave + 4 * (l >> 4), g, u);
    }
  }
}

// ---------------------------------------------------------------------------
// More rows to an expert, and the down product: 32 columns to a wave, activations through LDS
// ---------------------------------------------------------------------------
// A 128-k step of up to 64 rows lies in LDS as 16 pieces of 16 bytes to a row, piece p of row r
// at p ^ swizzle(r). LDS serves a wave's 16-byte accesses eight lanes at a time, four and four from
// neighbouring groups of 16 (lanes 0 .. 3 with 20 .. 23, 4 .. 7 with 16 .. 19, ...): with the row's low
// bits on top these hit distinct banks, in the reads (4 rows of a piece, 4 of the next group's) and in
// the writes (4 pieces of a row, 4 of the next). p ^ (r % 16) made each read collide once (1024
// tokens, k 4, 32 experts, H 2048, I 1024: 67 + 58 us, so 63 + 56; no difference at 256 tokens).
// Two buffers, one barrier to a step. PL: the rows' parts.
__device__ __forceinline__ int swizzle(int row) { return (row & 1) << 3 | (row & 2) << 1 | (row >> 2 & 3); }
template <int MAXNT, int PL>
struct ManySmem {
  Rows rows;
  u32x4 x[2][PL][16 * MAXNT][16];
};
template <int NT, int PL>
struct ManyStep {
  Codes<2> code;
  u32x4 x[PL][NT];
};
// A wave's columns: 16 of gate and of up, or 32 of the down product. A wave past the last ones repeats
// them and stores nothing: it still fetches its share of rows. Twice as many columns to a wave
// (half the reads of LDS) took 128 tokens, k 8, 64 experts, H 7168, I 2048 211 + 138 us against 206 + 129,
// 256 tokens, k 8, 128 experts, H 2048, I 768 53 + 45 against 51 + 40; 512 tokens, k 8, 64 experts,
// H 7168, I 2048 402 + 333 against 442 + 335.
template <bool UP>
struct Columns {
  Tile t[2];
  int unit, units, half;
  __device__ __forceinline__ Columns(const MoeArgs& a, int expert) {
    const Packed p =
        UP ? packed(a.w13 + expert * a.stride13, 2 * a.I, a.H) : packed(a.w2 + expert * a.stride2, a.H, a.I);
    unit = kWaves * blockIdx.x + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    units = UP ? a.I / 16 : a.H / 32;
    const int u = min(unit, units - 1);
    half = u & 1;
    t[0] = tile_at(p, UP ? u / 2 : u);
    if constexpr (UP) t[1] = tile_at(p, a.I / 32 + u / 2);
  }
  __device__ __forceinline__ void load(int step, Codes<2>& c) const { load_codes<2, UP>(t, step, c, half); }
};
template <bool UP, int NT, typename SMEM>
__device__ __forceinline__ void many_rows(const MoeArgs& a, const Columns<UP>& o, int first, int n, SMEM& sm,
                                          const Codes<2> (&begin)[2]) {
  constexpr int PL = UP ? 1 : 2;
  const int tid = threadIdx.x, l = tid & 63, c = l & 15, g = l >> 4;
  const int K = UP ? a.H : a.I;
  const int piece = tid & 15;
  const uint8_t* row[PL][NT];  // of the rows that this thread fetches a piece of
#pragma unroll
  for (int r = 0; r < NT; ++r) {
    const int pair = sm.rows.list[min(first + 16 * r + (tid >> 4), n - 1)];
#pragma unroll
    for (int pl = 0; pl < PL; ++pl) row[pl][r] = (UP ? a.x + pair / a.k * a.ldx : h_row(a, pl, pair)) + 16 * piece;
  }
  mx::v4f acc[NT][2];
  clear(acc);
  const int steps = (K + 127) / 128;
  auto load = [&](int s, ManyStep<NT, PL>& v) {
    if (s >= 2) o.load(s, v.code);
    const int64_t at = 128 * s + 8 * piece < K ? 256 * (int64_t)s : -16 * (int64_t)piece;  // past K: the row's start
#pragma unroll
    for (int pl = 0; pl < PL; ++pl)
#pragma unroll
      for (int r = 0; r < NT; ++r) v.x[pl][r] = *reinterpret_cast<const u32x4*>(row[pl][r] + at);
  };
  auto put = [&](const ManyStep<NT, PL>& v, int buf) {
#pragma unroll
    for (int pl = 0; pl < PL; ++pl)
#pragma unroll
      for (int r = 0; r < NT; ++r) sm.x[buf][pl][16 * r + (tid >> 4)][piece ^ swizzle(tid >> 4)] = v.x[pl][r];
  };
  ManyStep<NT, PL> v[2];
  load(0, v[0]);
  load(1, v[1]);
  v[0].code = begin[0];
  v[1].code = begin[1];
  put(v[0], 0);
  for (int s = 0; s < steps; s += 2) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      __syncthreads();
      put(v[1 - i], 1 - i);
      const Codes<2> code = v[i].code;
      load(s + i + 2, v[i]);
      __builtin_amdgcn_sched_barrier(0);  // keeps the loads ahead of the products
      if (s + i < steps)
        multiply<NT, PL, 2>(code, i, [&](int r, int pl, int j) {
          return __builtin_bit_cast(v8bf, sm.x[i][pl][16 * r + c][(4 * g + j) ^ swizzle(c)]);
        }, acc);
    }
  }
  if (o.unit >= o.units) return;  // whole waves; the caller's barrier is after the loop
#pragma unroll
  for (int r = 0; r < NT; ++r) {
    const int at = first + 16 * r + c;
    if (at >= n) continue;
    const int pair = sm.rows.list[at];
    if constexpr (UP) {
      store_h(a, pair, 16 * o.unit + 4 * g, acc[r][0], acc[r][1]);
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        *reinterpret_cast<mx::v4f*>(a.part + (int64_t)pair * a.H + 32 * o.unit + 16 * i + 4 * g) = acc[r][i];
    }
  }
}

// `tiles` <= MAXNT row tiles go together; the workgroups along z share an expert's rows.
// Two waves to a SIMD are asked for, so that no more than 256 registers are there to use: with more
// the sums would live in accumulation registers and move out and back in every step (256 tokens, k 4,
// 32 experts, H 2048, I 1024: 21.9 us for gate and up, 23.5 that way).
template <bool UP, int MAXNT>
__global__ __launch_bounds__(kThreads, 2) void many_kernel(MoeArgs a, int tiles) {
  __shared__ __align__(16) ManySmem<MAXNT, UP ? 1 : 2> sm;
  int expert = blockIdx.y;
  Codes<2> begin[2];
  auto start = [&]() {
    const Columns<UP> o(a, __builtin_amdgcn_readfirstlane(expert));
    o.load(0, begin[0]);
    o.load(1, begin[1]);
  };
  // The weight is asked for before the rows are known, where the expert is.
  const bool direct = slot_is_expert(a);
  if (direct) start();
  const int n = find_rows(a, blockIdx.y, sm.rows, expert);
  if (n == 0) return;
  if (!direct) start();
  const Columns<UP> o(a, __builtin_amdgcn_readfirstlane(expert));
  const int rows = 16 * tiles, step = rows * gridDim.z;
  for (int first = rows * blockIdx.z; first < n; first += step) {
    const int left = min(n - first, rows);
    if (MAXNT == 1 || left <= 16)
      many_rows<UP, 1>(a, o, first, n, sm, begin);
    else if (left <= 32)
      many_rows<UP, MAXNT == 1 ? 1 : 2>(a, o, first, n, sm, begin);
    else if (left <= 48)
      many_rows<UP, MAXNT == 1 ? 1 : 3>(a, o, first, n, sm, begin);
    else
      many_rows<UP, MAXNT>(a, o, first, n, sm, begin);
    __syncthreads();
    if (first + step < n) start();
  }
}

// y[t] = sum over the token's pairs, in their order. What lies in the place of a pair without an
// expert is read like the others, at the same time as the ids, and left out.
__global__ __launch_bounds__(256) void combine_kernel(MoeArgs a) {
  const int t = blockIdx.y, col = 4 * (blockIdx.x * 256 + threadIdx.x);
  if (col >= a.H) return;
  mx::v4f v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
  for (int j = 0; j < a.k; ++j) {
    const int64_t p = (int64_t)t * a.k + j;
    const bool there = (uint32_t)a.ids[p] < (uint32_t)a.E;
    const mx::v4f q = *reinterpret_cast<const mx::v4f*>(a.part + p * a.H + col);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = v[e] + (there ? q[e] : 0.0f);
  }
  *reinterpret_cast<u32x2*>(a.y + t * a.ldy + 2 * col) =
      u32x2{mx::pack_bf16x2(v[0], v[1]), mx::pack_bf16x2(v[2], v[3])};
}

// ---------------------------------------------------------------------------
// Few tokens: the down product over all their experts, 32 or 16 columns to a workgroup
// ---------------------------------------------------------------------------
// The rows are the tokens, so that the sum over a token's experts is the matrix instruction's
// own: no partial products in memory, no launch to add them. The work is a list of (expert,
// 128 k), taken in turn by the waves; h of all pairs lies in LDS, piece p (8 k) of a row of
// token t at p ^ t, which spreads a piece of the tokens over distinct banks. A token without the
// expert has a row of zeros, and keeps its sums: zeros times a weight that is not finite are NaN.
// Up to 10 pairs, past which the other two launches are as fast or faster. The call, replayed, this way and
// with many_kernel and combine_kernel (E 32): one token, k 8, H 7168, I 2048 37.0 us and 39.4; 2 tokens,
// k 2, H 512, I 256 7.9 and 8.7; 5 tokens, k 2, H 4096, I 1024 22.7 and 23.4, H 2048 17.0 and 16.2; 6 tokens,
// k 2, H 2048, I 1024 18.1 and 16.5; 4 tokens, k 4, H 512, I 512 13.1 and 11.3, H 7168 26.2 and 26.8; 8
// tokens, k 8, H 4096, I 256 27.6 and 20.7.
constexpr int kTokens = 16;  // columns of the matrix instruction
constexpr int kTokenPairs = 10;
static_assert(kTokenPairs <= kTokens);
// Of 8 k: all pairs' I, each rounded up to 128; three to a thread (5 tokens, k 2, H 3392, I 1856, which
// needs more than two: 22.5 us this way, 25.5 the other).
constexpr int kTokenWaves = 16;
constexpr int kTokenPieces = 3 * 64 * kTokenWaves;
template <int NC>
struct TokenSmem {
  int slots;
  u32x4 h[2][kTokenPieces];
  u32x4 zero;
  int expert[kTokenPairs];             // of a slot
  int16_t pair[kTokenPairs][kTokens];  // of a slot's token, -1 without one
  mx::v4f red[kTokenWaves][NC][64];
};
// Slots are the distinct (expert, turn) in the order of their first pairs; a pair's turn is how
// often its token has its expert before. One wave finds them: lane p has pair p.
template <int NC>
__device__ __forceinline__ void find_slots(const MoeArgs& a, TokenSmem<NC>& s) {
  const int tid = threadIdx.x, l = tid & 63, P = a.T * a.k;
  const int id = l < P ? a.ids[l] : -1, token = l / a.k;
  for (int i = tid; i < kTokenPairs * kTokens / 2; i += 64 * kTokenWaves)
    reinterpret_cast<uint32_t*>(s.pair)[i] = ~0u;
  __syncthreads();
  if (tid >= 64) return;
  const bool there = (uint32_t)id < (uint32_t)a.E;
  int lead = l;  // one token: every pair is a slot of its own
  if (a.T > 1) {
    int turn = 0;
    for (int i = 0; i < P; ++i) turn += i < l && __builtin_amdgcn_readlane(id, i) == id && i / a.k == token;
    for (int i = P - 1; i >= 0; --i)
      if (__builtin_amdgcn_readlane(id, i) == id && __builtin_amdgcn_readlane(turn, i) == turn && i < l) lead = i;
  }
  const uint64_t leads = __ballot(there && lead == l);
  const int slot = __popcll(leads & (((uint64_t)1 << lead) - 1));
  if (there) {
    if (lead == l) s.expert[slot] = id;
    s.pair[slot][token] = (int16_t)l;
  }
  if (l == 0) s.slots = __popcll(leads);
}
// 16 NC columns to a workgroup.
template <int NC>
__global__ __launch_bounds__(64 * kTokenWaves) void tokens_kernel(MoeArgs a) {
  __shared__ __align__(16) TokenSmem<NC> sm;
  const int tid = threadIdx.x, l = tid & 63, c = l & 15, g = l >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int P = a.T * a.k, steps = (a.I + 127) / 128, pieces = 16 * steps;  // of a row
  // Everyone's h is asked for before the slots are known.
  constexpr int kEach = kTokenPieces / (64 * kTokenWaves);
  u32x4 held[2][kEach];
  int at[kEach];
  {
    int pair = tid / pieces, p = tid - pair * pieces;
    const int by = 64 * kTokenWaves / pieces, rest = 64 * kTokenWaves - by * pieces;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      at[i] = pair < P ? pair * pieces + (p ^ (pair / a.k)) : -1;
#pragma unroll
      for (int pl = 0; pl < 2; ++pl) {
        held[pl][i] = u32x4{0, 0, 0, 0};
        if (pair < P && 8 * p < a.I) held[pl][i] = *reinterpret_cast<const u32x4*>(h_row(a, pl, pair) + 16 * p);
      }
      pair += by;
      p += rest;
      if (p >= pieces) {
        p -= pieces;
        ++pair;
      }
    }
  }
  if (tid == 0) sm.zero = u32x4{0, 0, 0, 0};
  find_slots(a, sm);
#pragma unroll
  for (int i = 0; i < kEach; ++i)
#pragma unroll
    for (int pl = 0; pl < 2; ++pl)
      if (at[i] >= 0) sm.h[pl][at[i]] = held[pl][i];
  __syncthreads();
  const int slots = sm.slots;
  mx::v4f acc[1][NC];
  clear(acc);
  int slot = wave / steps, s = wave - slot * steps;
  const int by = kTokenWaves / steps, rest = kTokenWaves - by * steps;
#pragma unroll 1
  while (slot < slots) {
    const Packed p = packed(a.w2 + __builtin_amdgcn_readfirstlane(sm.expert[slot]) * a.stride2, a.H, a.I);
    const Tile t[1] = {tile_at(p, NC == 2 ? blockIdx.x : blockIdx.x / 2)};
    Codes<NC> code;
    load_codes<NC, NC == 1>(t, s, code, blockIdx.x & 1);
    const int pair = sm.pair[slot][c];  // of the lane's token, in the operand and in the result alike
    mx::v4f kept[NC];
#pragma unroll
    for (int i = 0; i < NC; ++i) kept[i] = acc[0][i];
    multiply<1, 2, NC>(code, s, [&](int, int pl, int j) {
      const u32x4* x = pair >= 0 ? &sm.h[pl][pair * pieces + ((16 * s + 4 * g + j) ^ c)] : &sm.zero;
      return __builtin_bit_cast(v8bf, *x);
    }, acc);
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[0][i][e] = pair >= 0 ? acc[0][i][e] : kept[i][e];
    slot += by;
    s += rest;
    if (s >= steps) {
      s -= steps;
      ++slot;
    }
  }
#pragma unroll
  for (int i = 0; i < NC; ++i) sm.red[wave][i][l] = acc[0][i];
  __syncthreads();
  if (wave >= NC || c >= a.T) return;
  mx::v4f y = sm.red[0][wave][l];
#pragma unroll
  for (int w = 1; w < kTokenWaves; ++w) y = y + sm.red[w][wave][l];
  *reinterpret_cast<u32x2*>(a.y + c * a.ldy + 2 * (16 * NC * (int)blockIdx.x + 16 * wave + 4 * g)) =
      u32x2{mx::pack_bf16x2(y[0], y[1]), mx::pack_bf16x2(y[2], y[3])};
}

// Up to 64 rows go together, so that a weight is expanded once for them; 32 where 64 would leave the chip
// short of workgroups (124 tokens, k 4, 6 experts, H 2240, I 1568: 42.3 us for the two launches, 47.2
// with 64, 58.8 with 16; 512 tokens, k 8, 16 experts, H 7168, I 512 202 with 64, 223 with 32).
// Workgroups along z for an expert's further rows, up to 512 in all and as many as one expert's rows may
// take: those without rows end after find_rows (the same two cases: one workgroup for all of an
// expert's rows 65 and 312 us).
template <bool UP, int MAXNT>
hipError_t launch_many(MoeArgs& a, unsigned slots, hipStream_t st) {
  const int64_t P = (int64_t)a.T * a.k;
  const unsigned units = (unsigned)mxh::cdiv(UP ? a.I : a.H, (UP ? 16 : 32) * kWaves);
  const int64_t groups = (int64_t)units * slots;
  int tiles = MAXNT;
  unsigned z = 1;
  if (MAXNT > 1) {
    if (groups * mxh::cdiv(P, (int64_t)slots * 16 * MAXNT) < 512) tiles = 2;
    const int64_t most = mxh::cdiv(P, 16 * tiles), want = mxh::cdiv(512, groups);
    z = (unsigned)(most < want ? most : want);
  }
  void* args[] = {&a, &tiles};
  return hipLaunchKernel((const void*)many_kernel<UP, MAXNT>, dim3(units, slots, z), dim3(kThreads), args, 0, st);
}

bool shape_ok(int64_t T, int64_t k, int64_t H, int64_t I) {
  constexpr int64_t kMaxRow = (int64_t)1 << 20;
  return T >= 1 && k >= 1 && T <= MXFP4_MOE_MAX_PAIRS && k <= MXFP4_MOE_MAX_PAIRS && T * k <= MXFP4_MOE_MAX_PAIRS &&
         H >= 32 && H <= kMaxRow && H % 32 == 0 && I >= 32 && I <= kMaxRow && I % 32 == 0;
}
size_t h_bytes(int64_t T, int64_t k, int64_t I) { return (size_t)(T * k * I * 4 + 255) / 256 * 256; }  // two parts

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
  const int64_t P = T * k;
  // Rows to an expert: up to 10 on average few is as fast or faster (H 2048, I 1024, 32 experts: gate and up
  // 18.6 us, many 17.9; H 4096, I 1536, 16 experts 24.4 and 26.8), with 12 many is (22.0 and 18.6; 29.9 and
  // 26.7): few goes over the weight again for every 16 rows.
  const bool many = P > 10 * E;
  const unsigned slots = (unsigned)(P < E ? P : E), tiles = (unsigned)(I / 32);
  hipError_t e = many ? launch_many<true, 4>(a, slots, st)
                      : hipLaunchKernel((const void*)few_kernel, dim3(tiles, slots), dim3(kThreads), args, 0, st);
  if (e != hipSuccess) return MXFP4_ERR_HIP;
  if (P <= kTokenPairs && P * mxh::cdiv(I, 128) * 16 <= kTokenPieces) {
    // 16 columns to a workgroup while there is a CU for each (the call, replayed: 2 tokens, k 4, H 4096, I 1024,
    // 256 workgroups 19.6 us, 128 of 32 columns 20.1), else 32: LDS lets one workgroup to a CU (H 4128: 258
    // workgroups 26.8 us, 129 of 32 columns 20.6; one token, k 8, H 7168, I 2048 45.4 and 37.8).
    const bool narrow = H <= 16 * 256;
    const void* f = narrow ? (const void*)tokens_kernel<1> : (const void*)tokens_kernel<2>;
    const dim3 grid((unsigned)(narrow ? H / 16 : H / 32));
    return mxh::launch_status(hipLaunchKernel(f, grid, dim3(64 * kTokenWaves), args, 0, st));
  }
  e = many ? launch_many<false, 4>(a, slots, st) : launch_many<false, 1>(a, slots, st);
  if (e != hipSuccess) return MXFP4_ERR_HIP;
  const dim3 grid((unsigned)mxh::cdiv(H, 1024), (unsigned)T);
  return mxh::launch_status(hipLaunchKernel((const void*)combine_kernel, grid, dim3(256), args, 0, st));
}
