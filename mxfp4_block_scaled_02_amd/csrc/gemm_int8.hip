// gemm_a8w8: C[m, n] = T(acc * a_s[m] * b_s[n] (+ bias[n])), acc the exact int32
// sum over k of Aq[m, k] * Bq[n, k] on the integer matrix instructions.
//
// Every kernel multiplies with the 16x16x64 instruction: lane l supplies the 16
// bytes k = 16*(l/16) .. +15 of row l%16 of its operand, and result register r of
// lane l is D[4*(l/16) + r][l%16]. B is the first operand, so that a lane holds four
// neighbouring columns of C. K goes in steps of 128 bytes, a cache line of a row,
// and operands reach LDS by loads that bypass the registers.
//
// Three kernels, chosen from (M, N, K) by a ranking of them (kTiles below):
//  * skinny: 16 or 32 rows x 16 or 32 columns, K split over four waves (few tokens);
//  * ring: 32 x 32 to 128 x 256 tiles, a ring of LDS stages;
//  * large: 256 x 256 tiles, a ring of finer units, more under way per CU.
// What bounds them: the ring kernels take in 54 to 66 GB/s of operands a CU over their
// whole time (76 to 85 lines under way at 315 to 330 cycles each; a loop of such loads
// alone 55 to 75), so up to a thousand rows the bytes per CU decide (M256 N4096 K7168,
// 917 KB a CU: 13.8 to 15 us with the operands in the Infinity Cache, 1.0 to 1.1 POP/s,
// and 19 us from memory); a whole chip of 256 x 256 tiles is held by the power limit (M4096
// N4096 K7168: 86 to 91 us, 2.65 to 2.8 POP/s, from memory 90 to 95; on codes of zero 75).
#include "host_common.hpp"
#include "mx_device.hpp"

#pragma clang fp contract(off)

namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));

// Several elements of C at any element's address (rows need not be aligned to more):
// the hardware takes such stores, one instruction each. Non-temporal: C passes through
// once, and the operands keep their place in L2 (M2048 N7168 K2048: 28.8 -> 28.0 us).
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef u32x4 u32x4_at4 __attribute__((aligned(4)));
typedef u32x4 u32x4_at2 __attribute__((aligned(2)));
typedef u32x2 u32x2_at2 __attribute__((aligned(2)));
template <int CT>
struct Packed {
  static constexpr int kSize = CT == MXFP4_TYPE_F32 ? 4 : 2;
  static __device__ __forceinline__ void store16(void* at, const u32x4& v) {
    if constexpr (kSize == 4)
      __builtin_nontemporal_store(v, reinterpret_cast<u32x4_at4*>(at));
    else
      __builtin_nontemporal_store(v, reinterpret_cast<u32x4_at2*>(at));
  }
};

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
};

constexpr int kOut = 0x7fffffff;  // an offset past every window: zeros

template <int CT>
__device__ __forceinline__ float bias_at(const GemmArgs& p, int n) {
  if constexpr (CT == MXFP4_TYPE_F32) return ((const float*)p.bias)[n];
  const uint16_t b = ((const uint16_t*)p.bias)[n];
  if constexpr (CT == MXFP4_TYPE_BF16) return __builtin_bit_cast(float, (uint32_t)b << 16);
  return (float)__builtin_bit_cast(_Float16, b);
}
template <int CT>
__device__ __forceinline__ void store_one(const GemmArgs& p, int64_t m, int n, float v) {
  const int64_t at = m * p.ldc + n;
  if constexpr (CT == MXFP4_TYPE_F32)
    ((float*)p.C)[at] = v;
  else if constexpr (CT == MXFP4_TYPE_BF16)
    ((uint16_t*)p.C)[at] = mx::f32_to_bf16(v);
  else
    ((_Float16*)p.C)[at] = (_Float16)v;
}

// ---------------------------------------------------------------------------
// What the kernels share
// ---------------------------------------------------------------------------
// Operand rows lie in LDS as 128-byte rows of 8 pieces; piece c of row r is at slot
// c ^ ((r >> 1) & 7), which spreads the same piece of 16 neighbouring rows over 256
// bytes' worth of distinct banks (with c ^ (r & 7) every read collided twice: +38 %
// LDS cycles). Buffer-to-LDS loads fill 1 KB units of 8 rows: lane l's 16 bytes land
// at 16*l, so lane l fetches the piece that belongs in slot l%8 of row l/8.
__device__ __forceinline__ int unit_piece(int l, int unit_parity) {
  return 16 * ((l & 7) ^ (l >> 4)) ^ (64 * unit_parity);
}
// Where lane l finds its 16 bytes of half kk of a step, in a block of 16 rows.
__device__ __forceinline__ int frag_at(int l, int kk) {
  return (l & 15) * 128 + 16 * ((4 * kk + (l >> 4)) ^ ((l >> 1) & 7));
}

// A buffer resource over `rows` rows of K bytes at stride ld, as the scalar words that
// the loads written in assembly take: an offset past the last row's end reads zeros.
__device__ __forceinline__ u32x4 window_words(const uint8_t* base, int64_t rows, int64_t ld, int K) {
  const uintptr_t at = (uintptr_t)base;
  return u32x4{(uint32_t)at, (uint32_t)(at >> 32), (uint32_t)((rows - 1) * ld + K), 0x00020000u};
}
// 1 KB from memory to LDS (16 bytes a lane; lanes out of range write zeros). In
// assembly: for the intrinsic the compiler waits before every LDS read that follows,
// which would drain the ring. The kernels wait themselves (wait_loads, and a barrier
// where other waves read). The LDS address goes to m0, which is an output, so that the
// compiler does not count on what it had there itself. (As an input that it writes itself,
// loads of the large kernel came closer together: 350 cycles of latency for 240, +0.5 % time.)
__device__ __forceinline__ void load_to_lds(uint32_t at, int voff, const u32x4& r) {
  uint32_t m0;
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tbuffer_load_dwordx4 %2, %3, 0 offen lds"
               : "={m0}"(m0)
               : "s"(at), "v"(voff), "s"(r)
               : "memory");
}
template <int N>
__device__ __forceinline__ void wait_loads() {  // at most N of this wave's loads still outstanding
  static_assert(N < 64, "the counter's width");
  asm volatile("s_waitcnt vmcnt(%0)" ::"i"(N) : "memory");
}

// Workgroup ids of one residue mod 8 share an XCD (and its L2): each XCD gets a
// contiguous run of tiles, walked in bands of 8 row tiles, so that a run is compact
// in both directions and its tiles share rows of A and B in L2.
struct TileAt {
  int m, n;
};
__device__ __forceinline__ TileAt tile_at(int b, int mt, int nt) {
  constexpr int kBand = 8;
  const int G = mt * nt, q = G / 8, r = G % 8, x = b % 8;
  const int id = x * q + (x < r ? x : r) + b / 8;
  const int band = id / (kBand * nt), in = id - band * kBand * nt, bh = min(kBand, mt - band * kBand);
  return TileAt{band * kBand + in % bh, in / bh};
}

// A tile's scales and biases: fetched into registers while the first operand loads
// are under way, and put into LDS when the ring is no longer in use.
template <int CT, int BM, int BN, int T>
struct TileScales {
  static constexpr int kRegs = (BM + BN + T - 1) / T;
  static constexpr int kBytes = 4 * (BM + 2 * BN);
  float s[kRegs], b[kRegs];
  __device__ __forceinline__ void fetch(const GemmArgs& p, int m0, int n0, int rows, int cols) {
#pragma unroll
    for (int c = 0; c < kRegs; ++c) {
      const int e = threadIdx.x + T * c;
      s[c] = e < BN ? p.bs[n0 + min(e, cols - 1)] : p.as[m0 + min(e - BN, rows - 1)];
      b[c] = p.bias && e < BN ? bias_at<CT>(p, n0 + min(e, cols - 1)) : 0.0f;
    }
  }
  __device__ __forceinline__ void put(float* at) const {  // BN column scales, BM row scales, BN biases
#pragma unroll
    for (int c = 0; c < kRegs; ++c) {
      const int e = threadIdx.x + T * c;
      if (e < BM + BN) at[e] = s[c];
      if (e < BN) at[BM + BN + e] = b[c];
    }
  }
};

// 16 rows of a wave's part of C. acc[j] lane l register r is row l%16, column
// 16*j + 4*(l/16) + r of it (B is the matrix instruction's first operand). The rows go
// through the wave's own LDS block (kPitch bytes a row) and out in pieces of 16 bytes.
// Strip by strip: the stores of one drain while the next is converted (eight strips
// put first and stored after: M4096 N4096 K128 10.0 -> 10.9 us).
template <int CT, int NI>
struct Strip {
  static constexpr int kSize = Packed<CT>::kSize;
  static constexpr int kPitch = 16 * NI * kSize + 16;
  static constexpr int kBytes = 16 * kPitch;
  static __device__ __forceinline__ void store(const GemmArgs& p, uint8_t* epi, const v4i (&acc)[NI], float as,
                                               const float4 (&bs)[NI], const float4 (&bias)[NI], int m0, int n0,
                                               int l) {
#pragma unroll
    for (int j = 0; j < NI; ++j) {
      const float sc[4] = {bs[j].x, bs[j].y, bs[j].z, bs[j].w}, bi[4] = {bias[j].x, bias[j].y, bias[j].z, bias[j].w};
      float v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[e] = (float)acc[j][e] * as * sc[e];
        if (p.bias) v[e] = v[e] + bi[e];
      }
      uint8_t* const t = epi + (l & 15) * kPitch + (16 * j + 4 * (l >> 4)) * kSize;
      if constexpr (CT == MXFP4_TYPE_F32) {
        *reinterpret_cast<float4*>(t) = make_float4(v[0], v[1], v[2], v[3]);
      } else if constexpr (CT == MXFP4_TYPE_BF16) {
        *reinterpret_cast<uint2*>(t) = make_uint2(mx::pack_bf16x2(v[0], v[1]), mx::pack_bf16x2(v[2], v[3]));
      } else {
        *reinterpret_cast<f16x4*>(t) = f16x4{(_Float16)v[0], (_Float16)v[1], (_Float16)v[2], (_Float16)v[3]};
      }
    }
    __builtin_amdgcn_wave_barrier();
    const uint8_t* const from = epi;
    uint8_t* const to = (uint8_t*)p.C + ((int64_t)m0 * p.ldc + n0) * kSize;
    const int rows = min(16, p.M - m0), cols = min(16 * NI, p.N - n0);  // either may be below 1
    if (cols >= 16 * NI) {
      constexpr int kPieces = NI * kSize;  // of 16 bytes, in a row
#pragma unroll
      for (int i = 0; i < 16 * kPieces; i += 64) {
        const int r = (i + l) / kPieces, c = (i + l) % kPieces * 16;
        if (r < rows)
          Packed<CT>::store16(to + r * p.ldc * kSize + c, *reinterpret_cast<const u32x4*>(from + r * kPitch + c));
      }
    } else {  // the last columns element by element, neighbouring lanes on neighbouring columns
#pragma unroll 4
      for (int i = l; i < 256 * NI; i += 64) {
        const int r = i / (16 * NI), c = i % (16 * NI);
        if (r < rows && c < cols) {
          if constexpr (kSize == 4)
            *(uint32_t*)(to + (r * p.ldc + c) * 4) = *(const uint32_t*)(from + r * kPitch + c * 4);
          else
            *(uint16_t*)(to + (r * p.ldc + c) * 2) = *(const uint16_t*)(from + r * kPitch + c * 2);
        }
      }
    }
    __builtin_amdgcn_wave_barrier();
  }
};
// Four neighbouring elements of C, of which the first `left` exist.
template <int CT>
__device__ __forceinline__ void store_four(const GemmArgs& p, int64_t m, int n, const float (&v)[4], int left) {
  if (left < 4) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e < left) store_one<CT>(p, m, n + e, v[e]);
    return;
  }
  uint8_t* const t = (uint8_t*)p.C + (m * p.ldc + n) * Packed<CT>::kSize;
  if constexpr (CT == MXFP4_TYPE_F32) {
    Packed<CT>::store16(t, u32x4{__builtin_bit_cast(uint32_t, v[0]), __builtin_bit_cast(uint32_t, v[1]),
                                 __builtin_bit_cast(uint32_t, v[2]), __builtin_bit_cast(uint32_t, v[3])});
  } else if constexpr (CT == MXFP4_TYPE_BF16) {
    *reinterpret_cast<u32x2_at2*>(t) = u32x2{mx::pack_bf16x2(v[0], v[1]), mx::pack_bf16x2(v[2], v[3])};
  } else {
    const f16x4 h = {(_Float16)v[0], (_Float16)v[1], (_Float16)v[2], (_Float16)v[3]};
    *reinterpret_cast<u32x2_at2*>(t) = __builtin_bit_cast(u32x2, h);
  }
}

// ---------------------------------------------------------------------------
// Skinny kernel: a workgroup owns 16*MT rows x NC columns of C; its W waves take
// contiguous shares of K, each with a ring of S steps of its own in LDS, and run
// without a barrier until their integer sums meet in LDS (integers: their order does
// not matter).
// ---------------------------------------------------------------------------
template <int CT, int MT, int NC, int W, int S>
__global__ __launch_bounds__(64 * W) void gemm_skinny_kernel(GemmArgs p, int mt) {
  constexpr int MS = 16 * MT, NI = NC / 16, T = 64 * W;
  constexpr int UA = 2 * MT, UB = NC / 8, L = UA + UB, kRing = S * L * 1024, kSums = NI * MT * 64;
  static_assert(NI * MT <= S * L, "a wave's sums fit its ring");
  static_assert(NC % 16 == 0 && (kSums % T == 0 || kSums < T), "whole fragments, whole rounds of threads");
  constexpr int kRounds = (kSums + T - 1) / T;
  __shared__ __align__(16) uint8_t lds[W * kRing];
  const int l = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int m0 = (int)(blockIdx.x % (unsigned)mt) * MS, n0 = (int)(blockIdx.x / (unsigned)mt) * NC;
  const int rows = min(MS, p.M - m0), cols = min(NC, p.N - n0);
  const int lda = (int)p.lda, ldb = (int)p.ldb;
  const u32x4 ar = window_words(p.A + (int64_t)m0 * lda, rows, lda, p.K);
  const u32x4 br = window_words(p.B + (int64_t)n0 * ldb, cols, ldb, p.K);
  uint8_t* const own = lds + wave * kRing;
  const uint32_t own0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)lds + wave * kRing;
  const int steps = (p.K + 127) / 128;
  const int s0 = (int)((int64_t)steps * wave / W), s1 = (int)((int64_t)steps * (wave + 1) / W);
  const int avo = (l >> 3) * lda, bvo = (l >> 3) * ldb;
  auto load = [&](int s, int slot) {  // past K and past the share zeros
#pragma unroll
    for (int u = 0; u < L; ++u) {
      const bool isA = u < UA;
      const int q = isA ? u : u - UA, k = 128 * s + unit_piece(l, q & 1);
      const int off = isA ? avo + 8 * q * lda : bvo + 8 * q * ldb;
      load_to_lds(own0 + (slot * L + u) * 1024, s < s1 && k < p.K ? off + k : kOut, isA ? ar : br);
    }
  };
#pragma unroll
  for (int f = 0; f < S; ++f) load(s0 + f, f);
  // this thread's share of the tile, four neighbouring columns of one row a round
  float as[kRounds], bs[kRounds][4], bias[kRounds][4];
#pragma unroll
  for (int c = 0; c < kRounds; ++c) {
    const int t = (int)threadIdx.x + T * c;
    const int m = 16 * ((t >> 6) % MT) + (t & 15), n = 16 * ((t >> 6) / MT) + 4 * (t >> 4 & 3);
    as[c] = p.as[m0 + min(m, rows - 1)];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      bs[c][e] = p.bs[n0 + min(n + e, cols - 1)];
      bias[c][e] = p.bias ? bias_at<CT>(p, n0 + min(n + e, cols - 1)) : 0.0f;
    }
  }
  v4i acc[MT][NI];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NI; ++j) acc[i][j] = v4i{0, 0, 0, 0};
  int slot = 0;
  for (int s = s0; s < s1; ++s) {
    wait_loads<(S - 1) * L>();
    const uint8_t* const at = own + slot * L * 1024;
    v4i a[2][MT], b[2][NI];
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
#pragma unroll
      for (int i = 0; i < MT; ++i) a[kk][i] = *reinterpret_cast<const v4i*>(at + frag_at(l, kk) + 2048 * i);
#pragma unroll
      for (int j = 0; j < NI; ++j) b[kk][j] = *reinterpret_cast<const v4i*>(at + UA * 1024 + frag_at(l, kk) + 2048 * j);
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the step is in registers: its slot is free
    load(s + S, slot);
#pragma unroll
    for (int kk = 0; kk < 2; ++kk)
#pragma unroll
      for (int j = 0; j < NI; ++j)
#pragma unroll
        for (int i = 0; i < MT; ++i)
          acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(b[kk][j], a[kk][i], acc[i][j], 0, 0, 0);
    slot = slot == S - 1 ? 0 : slot + 1;
  }
  wait_loads<0>();  // nothing may still land where the sums go
#pragma unroll
  for (int j = 0; j < NI; ++j)
#pragma unroll
    for (int i = 0; i < MT; ++i) *reinterpret_cast<v4i*>(own + ((j * MT + i) * 64 + l) * 16) = acc[i][j];
  __syncthreads();
#pragma unroll
  for (int c = 0; c < kRounds; ++c) {
    const int t = (int)threadIdx.x + T * c;
    const int m = 16 * ((t >> 6) % MT) + (t & 15), n = 16 * ((t >> 6) / MT) + 4 * (t >> 4 & 3);
    if (t >= kSums || m >= rows || n >= cols) continue;
    v4i sum = *reinterpret_cast<const v4i*>(lds + t * 16);
#pragma unroll
    for (int w = 1; w < W; ++w) sum += *reinterpret_cast<const v4i*>(lds + w * kRing + t * 16);
    float v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[e] = (float)sum[e] * as[c] * bs[c][e];
      if (p.bias) v[e] = v[e] + bias[c][e];
    }
    store_four<CT>(p, m0 + m, n0 + n, v, cols - n);
  }
}

template <int CT, int MT, int NC, int W, int S>
hipError_t launch_skinny(GemmArgs& p, hipStream_t st) {
  int mt = (int)mxh::cdiv(p.M, 16 * MT);
  const int64_t grid = mt * mxh::cdiv(p.N, NC);
  void* args[] = {&p, &mt};
  return hipLaunchKernel((const void*)gemm_skinny_kernel<CT, MT, NC, W, S>, dim3((unsigned)grid), dim3(64 * W), args,
                         0, st);
}

// ---------------------------------------------------------------------------
// Ring kernel: WM x WN waves own BM x BN of C. LDS holds a ring of S stages, each the
// operands of one 128-byte step of K; a stage is loaded again, S steps on, as soon as it
// is read. One barrier per step, between its two 64-byte halves' matrix work: when it is
// passed, the next stage has arrived for every wave and this one is read by every wave.
// ---------------------------------------------------------------------------
template <int CT, int BM, int BN, int WM, int WN, int S>
__global__ __launch_bounds__(64 * WM * WN) void gemm_ring_kernel(GemmArgs p, int mt, int nt) {
  constexpr int W = WM * WN, T = 64 * W, TM = BM / WM, TN = BN / WN, MI = TM / 16, NI = TN / 16;
  constexpr int LA = BM / 8 / W, LB = BN / 8 / W, L = LA + LB;  // units per wave and step
  static_assert(BM % (8 * W) == 0 && BN % (8 * W) == 0, "every wave loads whole units of both operands");
  constexpr int kStage = (BM + BN) * 128;
  using St = Strip<CT, NI>;
  using Sc = TileScales<CT, BM, BN, T>;
  static_assert(W * St::kBytes + Sc::kBytes <= S * kStage, "the epilogue reuses the ring");
  __shared__ __align__(16) uint8_t lds[S * kStage];
  const int l = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const TileAt tile = tile_at(blockIdx.x, mt, nt);
  const int m0 = tile.m * BM, n0 = tile.n * BN, rows = min(BM, p.M - m0), cols = min(BN, p.N - n0);
  const int lda = (int)p.lda, ldb = (int)p.ldb;
  const u32x4 ar = window_words(p.A + (int64_t)m0 * lda, rows, lda, p.K);
  const u32x4 br = window_words(p.B + (int64_t)n0 * ldb, cols, ldb, p.K);
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)lds;
  const int avo = (8 * wave * LA + (l >> 3)) * lda, bvo = (8 * wave * LB + (l >> 3)) * ldb;
  auto load = [&](int s, int slot) {  // past K (and in steps past the last) zeros
    const uint32_t at = lds0 + slot * kStage;
#pragma unroll
    for (int i = 0; i < LA; ++i) {
      const int k = 128 * s + unit_piece(l, (wave * LA + i) & 1);
      load_to_lds(at + (wave * LA + i) * 1024, k < p.K ? avo + 8 * i * lda + k : kOut, ar);
    }
#pragma unroll
    for (int i = 0; i < LB; ++i) {
      const int k = 128 * s + unit_piece(l, (wave * LB + i) & 1);
      load_to_lds(at + BM * 128 + (wave * LB + i) * 1024, k < p.K ? bvo + 8 * i * ldb + k : kOut, br);
    }
  };
  const int steps = (p.K + 127) / 128;
#pragma unroll
  for (int s = 0; s < S; ++s) load(s, s);
  Sc sc;
  sc.fetch(p, m0, n0, rows, cols);
  const int wm = wave / WN, wn = wave % WN;
  v4i acc[MI][NI];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NI; ++j) acc[i][j] = v4i{0, 0, 0, 0};
  v4i a[2][MI], b[2][NI];
  auto read = [&](int slot, int kk) {
    const uint8_t* const at = lds + slot * kStage + wm * TM * 128 + frag_at(l, kk);
    const uint8_t* const bt = lds + slot * kStage + (BM + wn * TN) * 128 + frag_at(l, kk);
#pragma unroll
    for (int i = 0; i < MI; ++i) a[kk][i] = *reinterpret_cast<const v4i*>(at + 2048 * i);
#pragma unroll
    for (int j = 0; j < NI; ++j) b[kk][j] = *reinterpret_cast<const v4i*>(bt + 2048 * j);
  };
  auto mul = [&](int kk) {
#pragma unroll
    for (int j = 0; j < NI; ++j)
#pragma unroll
      for (int i = 0; i < MI; ++i)
        acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(b[kk][j], a[kk][i], acc[i][j], 0, 0, 0);
    __builtin_amdgcn_sched_barrier(0);
  };
  wait_loads<(S - 1) * L>();
  __syncthreads();
  read(0, 0);
  int slot = 0;
  for (int s = 0; s < steps; ++s) {
    const int next = slot == S - 1 ? 0 : slot + 1;
    read(slot, 1);
    __builtin_amdgcn_sched_barrier(0);
    mul(0);
    wait_loads<(S - 2) * L>();  // stage s+1 is here
    __syncthreads();            // for every wave, and stage s is read by every wave
    read(next, 0);
    __builtin_amdgcn_sched_barrier(0);
    load(s + S, slot);
    mul(1);
    slot = next;
  }
  wait_loads<0>();
  __syncthreads();
  float* const scales = reinterpret_cast<float*>(lds + W * St::kBytes);
  sc.put(scales);
  __syncthreads();
  float4 bs[NI], bias[NI];
#pragma unroll
  for (int j = 0; j < NI; ++j) {
    const float* const at = scales + wn * TN + 16 * j + 4 * (l >> 4);
    bs[j] = *reinterpret_cast<const float4*>(at);
    bias[j] = *reinterpret_cast<const float4*>(at + BM + BN);
  }
#pragma unroll
  for (int i = 0; i < MI; ++i)
    St::store(p, lds + wave * St::kBytes, acc[i], scales[BN + wm * TM + 16 * i + (l & 15)], bs, bias,
              m0 + wm * TM + 16 * i, n0 + wn * TN, l);
}

// ---------------------------------------------------------------------------
// Large kernel: 8 waves (2 x 4) own 256 x 256 of C. The ring holds ten units of 128
// rows x 128 bytes; a step of K is the units A rows 0..127, B rows 0..127, B rows
// 128..255, A rows 128..255, in this order of need. A step has two halves, the upper
// and the lower 128 rows of C; a wave owns 64 rows x 64 columns of each half, reads
// the columns' operands in the first and keeps them for the second. After each half
// the units that only it needs are free (three, then one), so that 96 to 112 KB of
// loads are always under way and a unit has about 1.5 steps to arrive.
// Every group of four matrix instructions is followed by the LDS reads and loads that
// run beside it, in source order: the scheduler is kept from collecting them.
// The 16x16x64 instruction, not 32x32x32: on random codes the whole chip sustains
// 4150 TOP/s with it and 3450 with the other (4850 and 4900 on zeros): the power
// limit, not the issue rate, decides.
// ---------------------------------------------------------------------------
template <int CT>
__global__ __launch_bounds__(512) void gemm_large_kernel(GemmArgs p, int mt, int nt) {
  constexpr int BM = 256, BN = 256, kUnit = 16384, kUnits = 10;
  using St = Strip<CT, 4>;
  using Sc = TileScales<CT, BM, BN, 512>;
  static_assert(8 * St::kBytes + Sc::kBytes <= kUnits * kUnit, "the epilogue reuses the ring");
  __shared__ __align__(16) uint8_t lds[kUnits * kUnit];
  const int l = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const TileAt tile = tile_at(blockIdx.x, mt, nt);
  const int m0 = tile.m * BM, n0 = tile.n * BN, rows = min(BM, p.M - m0), cols = min(BN, p.N - n0);
  const int lda = (int)p.lda, ldb = (int)p.ldb;
  const u32x4 ar = window_words(p.A + (int64_t)m0 * lda, rows, lda, p.K);
  const u32x4 br = window_words(p.B + (int64_t)n0 * ldb, cols, ldb, p.K);
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)lds;
  const int avo = (16 * wave + (l >> 3)) * lda, bvo = (16 * wave + (l >> 3)) * ldb;
  // half i of this wave's 16 rows of unit q of step s; past K (and in steps past the last) zeros
  auto load = [&](int s, int q, int slot, int i) {
    const int k = 128 * s + unit_piece(l, i);
    const int off = q == 0   ? avo + 8 * i * lda
                    : q == 1 ? bvo + 8 * i * ldb
                    : q == 2 ? bvo + (128 + 8 * i) * ldb
                             : avo + (128 + 8 * i) * lda;
    load_to_lds(lds0 + slot * kUnit + wave * 2048 + 1024 * i, k < p.K ? off + k : kOut, q == 0 || q == 3 ? ar : br);
  };
  const int steps = (p.K + 127) / 128;
#pragma unroll
  for (int u = 0; u < 2 * kUnits; ++u) load(u >> 3, (u >> 1) & 3, u >> 1, u & 1);
  Sc sc;
  sc.fetch(p, m0, n0, rows, cols);
  const int wm = wave >> 2, wn = wave & 3, bsel = wn >> 1;
  const uint8_t* const at = lds + wm * 64 * 128;
  const uint8_t* const bt = lds + (wn & 1) * 64 * 128;
  v4i a[2][4], b[2][4], acc[8][4];  // acc rows: 4 of the upper half, 4 of the lower
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = v4i{0, 0, 0, 0};
  auto readA = [&](int slot, int kk, int i) {
    a[kk][i] = *reinterpret_cast<const v4i*>(at + slot * kUnit + frag_at(l, kk) + 2048 * i);
  };
  auto readB = [&](int slot, int kk, int j) {
    b[kk][j] = *reinterpret_cast<const v4i*>(bt + slot * kUnit + frag_at(l, kk) + 2048 * j);
  };
  auto mul = [&](int h, int kk, int j) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      acc[4 * h + i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(b[kk][j], a[kk][i], acc[4 * h + i][j], 0, 0, 0);
    __builtin_amdgcn_sched_barrier(0);
  };
  auto wrap = [](int x) { return x >= kUnits ? x - kUnits : x; };
  // Two loads a wave and unit. Units issued when step s begins: up to 4s+9, needed 4s .. 4s+2: seven younger
  // (on later steps 4s+9 follows the wait: six).
  wait_loads<14>();
  __syncthreads();
  int s0 = 0;  // slot of unit 4*s
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    readA(0, 0, j);
    readB(1 + bsel, 0, j);
  }
  for (int s = 0; s < steps; ++s) {
    const int s1 = wrap(s0 + 1), s2 = wrap(s0 + 2), s3 = wrap(s0 + 3), next = wrap(s0 + 4);
    const int sb = bsel ? s2 : s1, nb = wrap(next + 1 + bsel);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      readA(s0, 1, j);
      readB(sb, 1, j);
      mul(0, 0, j);
    }
    wait_loads<12>();  // unit 4s+3; younger: 4s+4 .. 4s+9
    __syncthreads();   // and units 4s .. 4s+2 are read by every wave
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      readA(s3, 0, j);
      load(s + 2, j < 2 ? 2 : 3, j < 2 ? s0 : s1, j & 1);
      mul(0, 1, j);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      readA(s3, 1, j);
      if (j < 2) load(s + 3, 0, s2, j);
      mul(1, 0, j);
    }
    wait_loads<12>();  // units 4s+4 .. 4s+6; younger: 4s+7 .. 4s+12
    __syncthreads();   // and unit 4s+3 is read by every wave
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      readA(next, 0, j);
      readB(nb, 0, j);
      if (j < 2) load(s + 3, 1, s3, j);
      mul(1, 1, j);
    }
    s0 = next;
  }
  wait_loads<0>();
  __syncthreads();
  float* const scales = reinterpret_cast<float*>(lds + 8 * St::kBytes);
  sc.put(scales);
  __syncthreads();
  float4 bs[4], bias[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float* const from = scales + wn * 64 + 16 * j + 4 * (l >> 4);
    bs[j] = *reinterpret_cast<const float4*>(from);
    bias[j] = *reinterpret_cast<const float4*>(from + BM + BN);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int m = 128 * (i >> 2) + wm * 64 + 16 * (i & 3);
    St::store(p, lds + wave * St::kBytes, acc[i], scales[BN + m + (l & 15)], bs, bias, m0 + m, n0 + wn * 64, l);
  }
}

template <int CT, int BM, int BN, int WM, int WN, int S>
hipError_t launch_ring(GemmArgs& p, hipStream_t st) {
  int mt = (int)mxh::cdiv(p.M, BM), nt = (int)mxh::cdiv(p.N, BN);
  void* args[] = {&p, &mt, &nt};
  return hipLaunchKernel((const void*)gemm_ring_kernel<CT, BM, BN, WM, WN, S>, dim3((unsigned)(mt * nt)),
                         dim3(64 * WM * WN), args, 0, st);
}
template <int CT>
hipError_t launch_large(GemmArgs& p, hipStream_t st) {
  int mt = (int)mxh::cdiv(p.M, 256), nt = (int)mxh::cdiv(p.N, 256);
  void* args[] = {&p, &mt, &nt};
  return hipLaunchKernel((const void*)gemm_large_kernel<CT>, dim3((unsigned)(mt * nt)), dim3(512), args, 0, st);
}

// The kernels a call may take, and a figure that ranks them as a function of a kernel's
// tiles per CU n (rounded up over kModelCUs) and 128-byte steps of K t:
//   start + tile * n + step * t + tile_step * n * t.
// The constants are least-squares fits of relative error to times in us over 255 shapes (M
// 1 to 4096, N 256 to 7168, K 512 to 7168, operands from memory, graph replay;
// profiles/int8_tile_fit.csv). The figure is not the time: it has no term for the memory
// that all tiles read, which falls out where it is the same for all of them. For the kernel
// taken it is 0.63 to 1.27 of the time over these shapes, and 0.46 to 1.13 (median 0.66)
// with N or K of 8192 to 28672, where reading the weight bounds a call of few rows.
// The choice, over every kernel measured on every shape (profiles/int8_tile_check.csv),
// costs 0.8 % more than always taking the fastest on the 255 shapes (at most 23 %, M4096
// N2112 K512: 16.4 us on 256 x 256, 13.3 on 128 x 64) and 1.0 % on 36 shapes with the
// larger extents (at most 11 %, M1 N28672 K8192: 47.6 us on the 32 x 32 ring, 42.8 on 16 x 16).
// What decides: below about 200 tiles the chip idles, so small tiles win (M16 N2112 K7168:
// 7.7 us on 16 x 16, 17.0 on 64 x 64); past it the bytes per CU do, as BM + BN per BM * BN
// (M1024 N4096 K7168: 36.9 us on 128 x 128, 58.2 on 64 x 64).
struct TileModel {
  int bm, bn;
  float start, tile, step, tile_step;
};
constexpr TileModel kTiles[] = {
    {16, 16, 2.391f, 0.724f, -0.025f, 0.072f},     // 1: skinny
    {32, 16, 2.620f, 0.622f, -0.041f, 0.102f},     // 2: skinny
    {32, 32, 2.535f, 0.802f, -0.095f, 0.185f},     // 3: skinny
    {32, 32, 2.604f, 0.469f, 0.051f, 0.081f},      // 4: ring
    {64, 32, 2.601f, 0.621f, 0.051f, 0.128f},      // 5: ring
    {64, 64, 2.407f, 1.033f, 0.015f, 0.195f},      // 6: ring
    {128, 64, 2.303f, 1.378f, 0.012f, 0.298f},     // 7: ring
    {128, 128, 1.296f, 3.422f, -0.160f, 0.549f},   // 8: ring
    {128, 256, 0.285f, 5.266f, -0.195f, 0.861f},   // 9: ring
    {256, 256, -0.505f, 8.197f, -0.549f, 1.620f},  // 10: large
};
constexpr int kModelCUs = 256;

// 1-based index of the kernel for a valid shape.
int choose_tile(int64_t M, int64_t N, int64_t K) {
  const float t = (float)K / 128.0f;
  int best = 0;
  float least = 0.0f;
  for (int i = 0; i < (int)(sizeof(kTiles) / sizeof(kTiles[0])); ++i) {
    const TileModel& m = kTiles[i];
    const float n = (float)mxh::cdiv(mxh::cdiv(M, m.bm) * mxh::cdiv(N, m.bn), kModelCUs);
    const float cost = m.start + m.tile * n + (m.step + m.tile_step * n) * t;
    if (!best || cost < least) {
      best = i + 1;
      least = cost;
    }
  }
  return best;
}

template <int CT>
hipError_t launch(GemmArgs& p, hipStream_t st) {
  switch (choose_tile(p.M, p.N, p.K)) {
    case 1: return launch_skinny<CT, 1, 16, 4, 4>(p, st);
    case 2: return launch_skinny<CT, 2, 16, 4, 3>(p, st);
    case 3: return launch_skinny<CT, 2, 32, 4, 2>(p, st);
    case 4: return launch_ring<CT, 32, 32, 2, 2, 5>(p, st);
    case 5: return launch_ring<CT, 64, 32, 4, 1, 4>(p, st);
    case 6: return launch_ring<CT, 64, 64, 4, 2, 4>(p, st);
    case 7: return launch_ring<CT, 128, 64, 4, 2, 3>(p, st);
    case 8: return launch_ring<CT, 128, 128, 4, 4, 4>(p, st);
    case 9: return launch_ring<CT, 128, 256, 4, 4, 3>(p, st);
    default: return launch_large<CT>(p, st);
  }
}

constexpr int64_t kMaxStride = (int64_t)1 << 22;  // 256 rows of a window stay below 2^31 bytes
constexpr int64_t kMaxK = 131056;                 // 128 * 128 * K < 2^31

int check_shape(int64_t M, int64_t N, int64_t K) {
  if (M < 1 || N < 1 || K < 16 || K % 16 != 0 || K > kMaxK) return MXFP4_ERR_SHAPE;
  if (M > ((int64_t)1 << 24) || N > ((int64_t)1 << 24) || mxh::cdiv(M, 16) * mxh::cdiv(N, 16) > ((int64_t)1 << 30))
    return MXFP4_ERR_SHAPE;
  return MXFP4_OK;
}

}  // namespace

extern "C" int gemm_a8w8_path(int64_t M, int64_t N, int64_t K) {
  return check_shape(M, N, K) == MXFP4_OK ? choose_tile(M, N, K) : 0;
}

extern "C" int gemm_a8w8(const void* Aq, int64_t lda, const float* as, const void* Bq, int64_t ldb, const float* bs,
                         const void* bias, void* C, int64_t ldc, int ctype, int64_t M, int64_t N, int64_t K,
                         void* stream) {
  if (M < 1 || N < 1 || K < 1) return MXFP4_ERR_SHAPE;  // first: an empty tensor's pointer may be NULL
  if (!Aq || !as || !Bq || !bs || !C) return MXFP4_ERR_NULL;
  if (ctype != MXFP4_TYPE_BF16 && ctype != MXFP4_TYPE_F16 && ctype != MXFP4_TYPE_F32) return MXFP4_ERR_ARG;
  if (check_shape(M, N, K) != MXFP4_OK) return MXFP4_ERR_SHAPE;
  if (lda < K || lda > kMaxStride || ldb < K || ldb > kMaxStride || ldc < N || ldc > ((int64_t)1 << 36))
    return MXFP4_ERR_SHAPE;
  const int64_t size = ctype == MXFP4_TYPE_F32 ? 4 : 2;
  if (!mxh::aligned(Aq, 16) || lda % 16 != 0 || !mxh::aligned(Bq, 16) || ldb % 16 != 0 || !mxh::aligned(as, 4) ||
      !mxh::aligned(bs, 4) || !mxh::aligned(C, (uintptr_t)size) || (bias && !mxh::aligned(bias, (uintptr_t)size)))
    return MXFP4_ERR_ALIGN;
  GemmArgs p{(const uint8_t*)Aq, lda, as, (const uint8_t*)Bq, ldb, bs, bias, C, ldc, (int)M, (int)N, (int)K};
  const hipStream_t st = (hipStream_t)stream;
  switch (ctype) {
    case MXFP4_TYPE_BF16: return mxh::launch_status(launch<MXFP4_TYPE_BF16>(p, st));
    case MXFP4_TYPE_F16: return mxh::launch_status(launch<MXFP4_TYPE_F16>(p, st));
    default: return mxh::launch_status(launch<MXFP4_TYPE_F32>(p, st));
  }
}
