// Single-token decode attention over a paged cache (include/fc_paged.h).
//
// What it computes, per sequence and kv head, over the tokens t a row sees:
//   s_t = sigma q.k_t,  out = sum e^(s_t - m) v_t / sum e^(s_t - m)
// for the G query heads that share the kv head.
//
// What bounds it: HBM. Every seen K and V row is read once per kv head and
// serves its whole group; at G = 8 and bf16 that is four multiply-adds per byte
// and a conversion per element, most of what the CUDA cores can do at full
// bandwidth and little of what the tensor cores can (12 % busy). So both
// products run as mma.sync m16n8k16 (fp32 out) with the TOKENS (and for V the
// channels) on the 16-wide side and the heads on the 8-wide one:
//   S^T (16 tokens x 8 heads)  = K (16 x D) . Q^T,
//   O^T (16 channels x 8 heads) += V^T (16 x 16 tokens) . P^T.
// A 128-row tcgen05 tile would have to be gathered from several pages into
// shared memory first; here every warp takes its fragments straight from HBM
// into registers, 16 bytes per lane. The order of the contracted index is
// free, so lane (r = lane / 4, c = lane % 4) loads 16 contiguous bytes of K row
// r and calls them its k-indices; for V it loads 16 contiguous bytes of its
// four token rows and pairs them with byte permutes. No staging, no barrier
// in the loop; the next tile's K loads are issued once S is done, its V loads
// once O is, so loads are in flight all the time.
//
// Precision. bf16 rows are exact as they are; the query is one bf16 limb, or
// three (24 bits) when it is fp32; P is split into two limbs (2^-17) for a bf16
// output and three for an fp32 one; fp32 pages are split into three limbs,
// products below 2^-24 of the largest dropped. int8 codes are exact in fp16,
// which takes fewer instructions than bf16 and holds 11 bits a limb: the query
// (brought to fp16's range by a power of two per head) is one limb, two when
// it is fp32, and P times V's scale (by a power of two per head that follows the
// running maximum and the products themselves, not the scales: a large V row of
// little weight leaves the others their bits) is two.
// Maxima, sums and accumulators are fp32. Sums that stay in the tensor cores'
// accumulators are truncated, not rounded (7e-6 over 8,000 tokens), so each
// tile's V products, and for an fp32 result each step's leading score product,
// are added in fp32 (int8: for an fp32 query). Against 64 bits, in the 2-norm of a
// head: 6e-7 and less in fp32 for scores below 2^4 (log2 domain; beyond that a
// score's own half step shows), 1.4e-7 over a batch; the output's own rounding in
// bf16.
//
// Measured (B200, calls back to back): one bf16 sequence of 131,075 tokens, 32
// query and 8 kv heads of 128: 90 to 91 us, 5.9 TB/s, 0.90 of the copy rate. 64
// int8 sequences of up to 8,199 tokens, 64 / 8 heads: 172 us, 4.1 TB/s, bound by
// its 503 instructions per tile. One fp32 sequence of 256 tokens, 4 heads of 64:
// 9.7 us, all latency.
//
// Softmax: each warp keeps its own running maximum per head and raises it only
// when a tile exceeds it by more than 2^8 (a vote); until then p <= 2^8 and the
// sums stay exact enough in fp32, and no shuffle is needed.
//
// Split: the batch's tiles (16 tokens of one row and kv head) form one line,
// cut evenly over the CTAs and their warps, whatever the rows' lengths. A warp
// finishes the (row, head) segments it holds whole; the others it leaves as
// (m, l, acc) fragments, at most two per warp. The CTA joins its warps'
// fragments in order and leaves at most two to the workspace; the last CTA of
// a segment (an atomic ticket, no waiting) joins those in order. The result
// does not depend on which CTA is last.
#pragma once

#include <cuda_fp16.h>

#include <atomic>

#include "fc_paged.cuh"

namespace fc {

struct PagedArgs {
  PageView pages;
  TokenView q, kn, vn;   // kn.p null: no fused append
  int32_t q_dtype, new_dtype;
  int32_t q_vec, new_vec, out_vec;  // aligned for vector access
  int32_t G;
  float scale_log2e;
  int32_t window, sinks;
  void* out;
  int64_t os_b, os_h;
  int32_t out_dtype;
  float* lse;
  uint32_t* tickets;   // one per CTA
  char* partials;      // two fragments per CTA
};

int launch_paged_attention_bf16_12(const PagedArgs& a, int64_t D, cudaStream_t s);
int launch_paged_attention_bf16_13(const PagedArgs& a, int64_t D, cudaStream_t s);
int launch_paged_attention_bf16_33(const PagedArgs& a, int64_t D, cudaStream_t s);
int launch_paged_attention_f32_33(const PagedArgs& a, int64_t D, cudaStream_t s);
int launch_paged_attention_i8_12(const PagedArgs& a, int64_t D, cudaStream_t s);
int launch_paged_attention_i8_22(const PagedArgs& a, int64_t D, cudaStream_t s);

// CTAs a launch may have (the workspace is sized for them).
constexpr int kPagedCtasPerSm = 1;
// Bytes of one fragment in the workspace.
inline size_t paged_fragment_bytes(int64_t D, int64_t G) {
  const size_t nt = G > 8 ? 2 : 1;
  return nt * size_t(D) / 16 * 512 + nt * 64;
}

#ifdef __CUDACC__

constexpr int kTile = 16;          // tokens per tile
constexpr int kSetup = 2;          // what beginning a segment costs, in tiles
constexpr int kJoin = 3;           // what a join over the workspace costs, in tiles per warp

// What a warp left of a segment (row, head): tiles [from, to) of n.
struct Piece {
  int32_t row, head, from, to, n;
};
// A segment left to other CTAs as well (row -1: none).
struct Open {
  int32_t row, head, cta0, cta1;
};

// QL, PL: limbs of the query and of P.
template <typename T, int D_, int NT_, int QL_, int PL_>
struct PagedCfg {
  static constexpr int D = D_, NT = NT_, QL = QL_, PL = PL_;  // NT: groups of 8 heads
  static constexpr int ES = int(sizeof(T));
  // log2 of how far p may exceed 1 (int8: the largest scale, 2^121, times it is
  // a finite fp32 number)
  static constexpr float kLazy = ES == 1 ? 6.0f : 8.0f;
  static constexpr float kMostScale = 8.507059173023462e37f;  // 2^126
  static constexpr int KW = D / 4 * ES / 4;   // words of a K row per lane
  static constexpr int VW = D / 8 * ES / 4;   // words of a V row per lane
  static constexpr int KL = 16 / ES < D / 4 ? 16 / ES : D / 4;  // elements per load
  static constexpr int VL = 16 / ES < D / 8 ? 16 / ES : D / 8;
  // tiles per iteration: more than one only where a tile is a few loads (two for
  // int8 rows of 128 spilled far more than one's 16 bytes: 250 us against 195 for
  // 64 sequences of 8K; one for int8 rows of 64: 104 us against 96)
  static constexpr int U = KW >= 8 ? 1 : 2;
  // Rows too wide for the registers are taken in parts (two, or four), and only
  // the first part of K and of V is loaded ahead. fp32 and int8 rows need room
  // for their limbs and conversions besides (16 heads of 128 in fp32: 2.6 TB/s
  // whole, 3.4 in two parts; 16 of 256 in int8: 1.5 and 1.6).
  static constexpr int kRegs = NT * D / 4 + U * (2 * KW + 4 * VW);
  static constexpr int CH = kRegs <= (ES == 2 ? 192 : 160) ? 1 : NT * D / 4 + 2 * U * KW <= (ES == 4 ? 176 : 192) ? 2 : 4;
  static constexpr bool kPrefetch = CH == 1;
  static constexpr int NQ = NT * D / 16;      // float4 accumulators per lane
  // 16 warps of 128 registers where a tile needs few (bf16 rows of 64: 5.1 TB/s
  // with 12, 5.5 with 16; int8 rows of 64 spill 132 bytes with 16 and none with
  // 12: 96 and 97 us for 64 sequences of 8K)
  static constexpr int WARPS = NQ >= 32 ? 4 : NQ >= 16 || kRegs > 96 ? 8 : kRegs > 48 || NT > 1 ? 12 : 16;
  static constexpr size_t kFragment = size_t(NQ) * 512 + NT * 64;
  static constexpr size_t kQuery = size_t(QL) * NT * (D / 32) * 512;
  static constexpr size_t kShared = WARPS * (2 * kFragment + kQuery);
  // besides: two pieces and their number for each warp, two open segments
  static constexpr size_t kStatic = WARPS * (2 * sizeof(Piece) + sizeof(int)) + 2 * sizeof(Open);
  static_assert(kShared + kStatic <= 232448, "shared memory of a CTA");
  static constexpr int kMostCtas = int(WARPS * 2 * kFragment / (NT * 8 * 4));  // of one segment: see the joins
};

// d += A B, or d = A B where FIRST (16 x 8 x 16; bf16, or fp16 for int8 pages).
template <typename T, bool FIRST>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  const float c0 = FIRST ? 0.0f : d[0], c1 = FIRST ? 0.0f : d[1], c2 = FIRST ? 0.0f : d[2], c3 = FIRST ? 0.0f : d[3];
  if constexpr (sizeof(T) == 1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
  } else {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
  }
}

// 2^e for -126 <= e <= 127.
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }
// The exponent of a positive finite x (its floor of log2; subnormals -127).
__device__ __forceinline__ int exponent_of(float x) { return int(__float_as_uint(x) >> 23) - 127; }

// A power of two g >= 1 that makes up for a factor e in [0, 1], e g <= 1, and
// leaves x (a power of two) times it at 2^126 or below.
__device__ __forceinline__ float lower_power(float e, float x) {
  const int most = 126 - exponent_of(x), k = -1 - exponent_of(e);  // e in [2^(-k - 1), 2^-k)
  return pow2i(k < 0 ? 0 : k < most ? k : most);
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

// Two bf16 (lo in the low half), rounded to nearest even.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

// Two fp16 (lo in the low half), rounded to nearest even.
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

// Exact int8 -> fp16 of two codes: x holds 0x6400 | (code + 128) in each half,
// the fp16 numbers 1024 + code + 128; 1152 is subtracted. (The codes plus 128 as
// fp16 subnormals take one instruction less a pair, but then 128 times the sum of
// the query, or of P, runs through sums that are truncated at its size: 4e-6 to
// 2.5e-5 of the output for queries that have a mean.)
__device__ __forceinline__ uint32_t codes_to_f16(uint32_t x) {
  const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&x), __half2half2(__ushort_as_half(0x6480)));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// The fp16 limb of (lo, hi), rounded to nearest, and what remains (exact).
__device__ __forceinline__ uint32_t take_limb_f16(float& lo, float& hi) {
  const uint32_t w = pack_f16(lo, hi);
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
  lo -= f.x;
  hi -= f.y;
  return w;
}

// The limb of (lo, hi) as packed bf16, and what remains. Truncation keeps eight
// bits and cannot overflow; three limbs hold all 24.
__device__ __forceinline__ uint32_t take_limb(float& lo, float& hi) {
  const uint32_t a = __float_as_uint(lo), b = __float_as_uint(hi);
  lo -= __uint_as_float(a & 0xffff0000u);
  hi -= __uint_as_float(b & 0xffff0000u);
  return __byte_perm(a, b, 0x7632);
}

__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The tiles of one row: the sinks' tiles, then those from the window's first.
struct RowTiles {
  int32_t len, lo, sinks;  // seen: t < len and (t >= lo or t < sinks)
  int32_t ns, w0, n;       // tile i starts at 16 (i < ns ? i : i - ns + w0)
  __device__ __forceinline__ RowTiles(const BatchRow& b, int32_t window, int32_t sink) {
    len = b.slot < 0 ? 0 : b.len;
    lo = window > 0 && len > window ? len - window : 0;
    sinks = sink < lo ? sink : lo;
    ns = (sinks + kTile - 1) / kTile;
    w0 = lo / kTile;
    if (ns > w0) ns = w0;
    n = ns + (len + kTile - 1) / kTile - w0;
    if (n < 1) n = 1;  // an empty row is one masked tile: its output is written
  }
  __device__ __forceinline__ int32_t start(int32_t i) const { return kTile * (i < ns ? i : i - ns + w0); }
  __device__ __forceinline__ bool sees(int32_t t) const { return t < len && (t >= lo || t < sinks); }
};

// Exponents that join two parts: 2^(m - M), 1 where both are -infinity (the
// part is empty, or all its scores are NaN and have to stay so).
__device__ __forceinline__ float join_factor(float m, float M) { return m == M ? 1.0f : fast_exp2(m - M); }

// Writes accumulator quad q of one lane, times f0 and f1: heads 8 nt + 2c and
// + 1, two neighbouring channels of D; any output type and alignment.
template <typename C>
__device__ __noinline__ void store_quad(const PagedArgs& a, int32_t row, int32_t head, int q, float4 acc, float f0,
                                        float f1) {
  const int lane = int(threadIdx.x & 31), r = lane >> 2, c = lane & 3;
  const int nt = q / (C::D / 16), idx = 2 * (q % (C::D / 16));
  const int d = idx / C::VL * 8 * C::VL + r * C::VL + idx % C::VL;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int g = nt * 8 + 2 * c + j;
    if (g >= a.G) continue;
    const int64_t at = row * a.os_b + (int64_t(head) * a.G + g) * a.os_h + d;
    const float x0 = (j ? acc.y : acc.x) * (j ? f1 : f0), x1 = (j ? acc.w : acc.z) * (j ? f1 : f0);
    if (a.out_dtype == FC_DTYPE_F32) {
      float* o = static_cast<float*>(a.out) + at;
      o[0] = x0;
      o[1] = x1;
    } else if (a.out_vec) {
      *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(a.out) + at) = pack_bf16(x0, x1);
    } else {
      __nv_bfloat16* o = static_cast<__nv_bfloat16*>(a.out) + at;
      o[0] = __float2bfloat16_rn(x0);
      o[1] = __float2bfloat16_rn(x1);
    }
  }
}

// The same for all quads of a segment that one warp holds whole, to aligned
// outputs.
template <typename C, typename TO>
__device__ __forceinline__ void store_all(const PagedArgs& a, int32_t row, int32_t head,
                                          const float (&acc)[C::NQ][4], const float (&f)[C::NT][2]) {
  constexpr int MT = C::D / 16;
  const int lane = int(threadIdx.x & 31), r = lane >> 2, c = lane & 3;
#pragma unroll
  for (int nt = 0; nt < C::NT; ++nt)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int g = nt * 8 + 2 * c + j;
      if (g >= a.G) continue;
      TO* o = static_cast<TO*>(a.out) + row * a.os_b + (int64_t(head) * a.G + g) * a.os_h + r * C::VL;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        const int idx = 2 * mt, d = idx / C::VL * 8 * C::VL + idx % C::VL;
        const float x0 = acc[nt * MT + mt][j] * f[nt][j], x1 = acc[nt * MT + mt][2 + j] * f[nt][j];
        if constexpr (sizeof(TO) == 4) *reinterpret_cast<float2*>(o + d) = make_float2(x0, x1);
        else *reinterpret_cast<uint32_t*>(o + d) = pack_bf16(x0, x1);
      }
    }
}

// lse = ln 2 (m + log2 l) of query head g of a kv head's group.
__device__ __forceinline__ void store_lse(const PagedArgs& a, int32_t row, int32_t head, int g, float m, float l) {
  if (a.lse && g < a.G)
    a.lse[(int64_t(row) * a.pages.H + head) * a.G + g] =
        l == 0.0f ? -__builtin_huge_valf() : 0.6931471805599453f * (m + log2f(l));
}

// A segment's part in shared memory or the workspace: NQ x 32 float4
// accumulators, then NT x 8 maxima (log2 domain), then NT x 8 sums.
template <typename C>
struct Fragment {
  char* p;
  __device__ __forceinline__ float4& acc(int q, int lane) const { return reinterpret_cast<float4*>(p)[q * 32 + lane]; }
  __device__ __forceinline__ float& m(int h) const { return reinterpret_cast<float*>(p + size_t(C::NQ) * 512)[h]; }
  __device__ __forceinline__ float& l(int h) const { return m(h + C::NT * 8); }
};

// Four query elements at q[at ..], of either type and any alignment.
static __device__ __noinline__ float4 load_query_slow(const void* q, int64_t at, int dtype) {
  return make_float4(load_elem(q, at, dtype), load_elem(q, at + 1, dtype), load_elem(q, at + 2, dtype),
                     load_elem(q, at + 3, dtype));
}

// The new token's K and V rows of a kv head, to their page.
template <typename T, int D>
__device__ __noinline__ void store_new_rows(const PagedArgs& a, int32_t row, int32_t head, int64_t page, int32_t in) {
  constexpr int E = D / 32;
  const PageView& pv = a.pages;
  const int lane = int(threadIdx.x & 31);
  float x[2][E];
  load_token_row<E>(a.kn.p, row * a.kn.sb + head * a.kn.sh, a.new_dtype, a.new_vec & 1, x[0], lane);
  load_token_row<E>(a.vn.p, row * a.vn.sb + head * a.vn.sh, a.new_dtype, a.new_vec & 2, x[1], lane);
  const int64_t at = page * pv.stride_page + head * pv.stride_head + int64_t(in) * D + lane * E;
  const int64_t se = page * pv.sstride_page + head * pv.sstride_head + in;
#pragma unroll 1
  for (int kv = 0; kv < 2; ++kv) {
    store_row<T, E>(x[0], reinterpret_cast<T*>(kv ? pv.v : pv.k) + at, (kv ? pv.vs : pv.ks) + se, lane);
#pragma unroll
    for (int i = 0; i < E; ++i) x[0][i] = x[1][i];
  }
}

// What a warp has of a segment: a lane's accumulators, maxima and sums.
template <typename C>
struct Share {
  float acc[C::NQ][4], m[C::NT][2], l[C::NT][2];
};
template <typename C>
__device__ __forceinline__ void copy_share(float (&acc)[C::NQ][4], float (&m)[C::NT][2], float (&l)[C::NT][2],
                                           const float (&acc0)[C::NQ][4], const float (&m0)[C::NT][2],
                                           const float (&l0)[C::NT][2]) {
#pragma unroll
  for (int q = 0; q < C::NQ; ++q)
#pragma unroll
    for (int k = 0; k < 4; ++k) acc[q][k] = acc0[q][k];
#pragma unroll
  for (int nt = 0; nt < C::NT; ++nt)
#pragma unroll
    for (int j = 0; j < 2; ++j) m[nt][j] = m0[nt][j], l[nt][j] = l0[nt][j];
}

// Tiles [tile, end) of a segment once more, token by token in fp32: what the
// kernel's loop leaves of the heads that have a NaN in a lane, without limbs, so
// that infinities and NaN act as the formula has them. Five to eight times the
// loop's time: 131,072 bf16 tokens, 32 / 8 heads of 128, 90 us without a NaN, 712
// with NaN in every V row, 589 with one infinity.
template <typename T, typename C>
__device__ __noinline__ void attend_plain(const PagedArgs& a, int32_t slot, int32_t row, int32_t head,
                                          RowTiles rt, int32_t tile, int32_t end, Share<C>& x) {
  constexpr int MT = C::D / 16, NT = C::NT;
  constexpr float kNone = -__builtin_huge_valf();
  const PageView& pv = a.pages;
  const int lane = int(threadIdx.x & 31), r = lane >> 2, c = lane & 3;
  float acc[C::NQ][4], m[NT][2], l[NT][2];
  copy_share<C>(acc, m, l, x.acc, x.m, x.l);
  bool redo[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      bool bad = l[nt][j] != l[nt][j];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
        bad |= acc[nt * MT + mt][j] != acc[nt * MT + mt][j] || acc[nt * MT + mt][2 + j] != acc[nt * MT + mt][2 + j];
      redo[nt][j] = (__ballot_sync(0xffffffffu, bad) >> c & 0x11111111u) != 0;
      if (!redo[nt][j]) continue;
      m[nt][j] = kNone;
      l[nt][j] = 0.0f;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) acc[nt * MT + mt][j] = acc[nt * MT + mt][2 + j] = 0.0f;
    }
  // lane r's eighth of the channels of heads 2c and 2c + 1
  constexpr int E = C::D / 8;
  float qv[NT][2][E];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int g = nt * 8 + 2 * c + j;
      const int64_t qh = row * a.q.sb + (int64_t(head) * a.G + g) * a.q.sh + r * E;
#pragma unroll
      for (int d = 0; d < E; ++d) qv[nt][j][d] = g < a.G && redo[nt][j] ? load_elem(a.q.p, qh + d, a.q_dtype) : 0.0f;
    }
#pragma unroll 1
  for (int32_t i = tile; i < end; ++i) {
#pragma unroll 1
    for (int32_t t = rt.start(i); t < rt.start(i) + kTile; ++t) {
      const int32_t page = rt.sees(t) ? page_of(pv, slot, t) : -1;
      if (page < 0) continue;
      const int64_t at = page * pv.stride_page + head * pv.stride_head + int64_t(t & ((1 << pv.log2P) - 1)) * C::D;
      float k[E], v[MT][2], e[NT][2], p[NT][2];
      load_elems<T, E>(reinterpret_cast<const T*>(pv.k) + at + r * E, k);
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        const int idx = 2 * mt, d = idx / C::VL * 8 * C::VL + r * C::VL + idx % C::VL;
        load_elems<T, 2>(reinterpret_cast<const T*>(pv.v) + at + d, v[mt]);
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float s = 0.0f;
#pragma unroll
          for (int d = 0; d < E; ++d) s += k[d] * qv[nt][j][d];
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
          s *= a.scale_log2e;
          const float top = fmaxf(m[nt][j], s);
          e[nt][j] = join_factor(m[nt][j], top);
          p[nt][j] = fast_exp2(s - (top == kNone ? 0.0f : top));
          if (!redo[nt][j]) continue;
          m[nt][j] = top;
          l[nt][j] = l[nt][j] * e[nt][j] + (r == 0 ? p[nt][j] : 0.0f);  // (summed over the lanes later)
        }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int n = 0; n < 4; ++n)
            if (redo[nt][n & 1])
              acc[nt * MT + mt][n] = acc[nt * MT + mt][n] * e[nt][n & 1] + p[nt][n & 1] * v[mt][n >> 1];
    }
  }
  copy_share<C>(x.acc, x.m, x.l, acc, m, l);
}

template <typename T, int D, int NT, int QL, int PL>
__global__ void __launch_bounds__(PagedCfg<T, D, NT, QL, PL>::WARPS * 32, 1)
    paged_attention_kernel(const __grid_constant__ PagedArgs a) {
  using C = PagedCfg<T, D, NT, QL, PL>;
  constexpr int U = C::U, KW = C::KW, VW = C::VW, CH = C::CH, MT = D / 16;
  constexpr int KB = C::KL * C::ES, VB = C::VL * C::ES;  // bytes per load
  constexpr int kRow = D * C::ES;                        // bytes of a token's row
  constexpr float kNone = -__builtin_huge_valf();
  // an fp32 result (int8: of an fp32 query; a bf16 one's eight bits let the sums
  // of its products be nearly exact, and 6e-7 holds without it)
  constexpr bool kFine = C::ES == 1 ? QL == 2 : PL == 3;
  extern __shared__ __align__(16) char smem[];
  __shared__ Piece pieces[C::WARPS * 2];
  __shared__ int n_pieces[C::WARPS];
  __shared__ Open open[2];
  const int warp = int(threadIdx.x >> 5), lane = int(threadIdx.x & 31), r = lane >> 2, c = lane & 3;
  char* fragments = smem;  // two per warp
  uint4* qs = reinterpret_cast<uint4*>(smem + C::WARPS * 2 * C::kFragment + warp * C::kQuery);
  // (the queries' memory, once they are done with)
  float(*factors)[NT * 8] = reinterpret_cast<float(*)[NT * 8]>(smem + C::WARPS * 2 * C::kFragment);
  const PageView& pv = a.pages;
  const int H = pv.H;

  after_previous();
  if (threadIdx.x < 2) open[threadIdx.x].row = -1;

  // ---- the warp's share of the line of units: a segment (row, kv head) is its
  // tiles behind kSetup units, what it costs to begin one
  const int per = (pv.n_rows + 31) / 32;
  int64_t mine = 0;
  int32_t longest = 0;
#pragma unroll 1
  for (int i = 0; i < per; ++i) {
    const int b = lane * per + i;
    if (b < pv.n_rows) {
      const int32_t n = RowTiles(pv.batch[b], a.window, a.sinks).n;
      mine += n + kSetup;
      longest = n > longest ? n : longest;
    }
  }
  mine *= H;
  int64_t before = mine;  // inclusive, then exclusive prefix
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, before, o);
    if (lane >= o) before += x;
  }
  const int64_t total = __shfl_sync(0xffffffffu, before, 31);
  before -= mine;
  longest = __reduce_max_sync(0xffffffffu, longest);
  // `chunk` units per warp, no fewer than U + kSetup: a small batch takes fewer CTAs
  constexpr uint32_t kFew = C::WARPS * (U + kSetup);
  const uint32_t ctas = total >= int64_t(gridDim.x) * kFew ? gridDim.x : (uint32_t(total) + kFew - 1) / kFew;
  const uint32_t workers = ctas * C::WARPS;
  int64_t chunk = total >> 31 ? (total + workers - 1) / workers : (uint32_t(total) + workers - 1) / workers;
  // A CTA per segment, if that takes its warps at most kJoin more tiles each
  // than an even split (which joins over the workspace instead).
  const uint32_t segments = uint32_t(pv.n_rows) * uint32_t(H);
  const int32_t each = (longest + C::WARPS - 1) / C::WARPS;
  const bool alone = segments <= gridDim.x && each <= chunk + kJoin;

  int32_t row = 0, head = 0, unit = 0;
  int64_t from = 0, to = 0, cta_chunk = 1;
  if (alone) {
    if (blockIdx.x >= segments) return;
    row = int32_t(blockIdx.x / uint32_t(H));
    head = int32_t(blockIdx.x % uint32_t(H));
    const int32_t n = RowTiles(pv.batch[row], a.window, a.sinks).n, share = (n + C::WARPS - 1) / C::WARPS;
    from = share * warp;
    to = from + share < n ? from + share : n;
    unit = int32_t(from) + kSetup;
  } else {
    cta_chunk = chunk * C::WARPS;
    const int64_t cta_from = cta_chunk * blockIdx.x;
    if (cta_from >= total) return;
    const int64_t cta_to = cta_from + cta_chunk < total ? cta_from + cta_chunk : total;
    from = cta_from + chunk * warp;
    to = from + chunk < cta_to ? from + chunk : cta_to;
    if (from < to) {
      const unsigned who = __ballot_sync(0xffffffffu, before <= from && from < before + mine);
      const int src = __ffs(int(who)) - 1;
      if (lane == src) {
        int64_t base = before;
        row = lane * per;
#pragma unroll 1
        while (row < pv.n_rows) {
          const int32_t n = RowTiles(pv.batch[row], a.window, a.sinks).n + kSetup;
          if (from < base + int64_t(n) * H) {
            const int64_t x = from - base;
            head = x >> 31 ? int32_t(x / n) : int32_t(uint32_t(x) / uint32_t(n));
            unit = int32_t(x - int64_t(head) * n);
            break;
          }
          base += int64_t(n) * H;
          ++row;
        }
      }
      row = __shfl_sync(0xffffffffu, row, src);
      head = __shfl_sync(0xffffffffu, head, src);
      unit = __shfl_sync(0xffffffffu, unit, src);
    }
  }

  // ---- the segments of the share
  int made = 0;  // fragments left in shared memory
  int64_t at = from;
#pragma unroll 1
  while (at < to && row < pv.n_rows) {
    const BatchRow br = pv.batch[row];
    const RowTiles rt(br, a.window, a.sinks);
    const int32_t last = int64_t(rt.n + kSetup - unit) < to - at ? rt.n + kSetup : unit + int32_t(to - at);
    const int32_t tile = unit > kSetup ? unit - kSetup : 0, end = last - kSetup;
    at += last - unit;
    unit = 0;
    if (end <= tile) {  // only of what comes before the tiles
      if (last == rt.n + kSetup && ++head == H) head = 0, ++row;
      continue;
    }
    const int32_t Pm = (1 << pv.log2P) - 1;

    // The table ahead of its use: lane j holds the pages of tile held + j (-1:
    // nothing to read; a page of 8 tokens holds half a tile), and of the 32
    // tiles after them; a bit per tile: all its tokens are seen.
    struct Ahead {
      int32_t page[2];
      uint32_t full;
    } cur, nxt;
    int32_t held = tile;
    auto fetch = [&](int32_t i, Ahead& g) {
      g.page[0] = g.page[1] = -1;  // past the end: the last loads ahead read nothing
      g.full = 0;
      if (i >= end) return;
      const int32_t t = rt.start(i + lane);
      bool all = t + kTile <= rt.len && (t >= rt.lo || t + kTile <= rt.sinks);
      g.page[0] = i + lane < end && t < rt.len ? page_of(pv, br.slot, t) : -1;
      g.page[1] = g.page[0];
      if (pv.log2P == 3) g.page[1] = i + lane < end && t + 8 < rt.len ? page_of(pv, br.slot, t + 8) : -1;
      g.full = __ballot_sync(0xffffffffu, all && (g.page[0] | g.page[1]) >= 0);
    };
    float acc[C::NQ][4] = {};
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt][0] = m[nt][1] = kNone;
      l[nt][0] = l[nt][1] = 0.0f;
    }
    if (rt.len > 0) {
    // query fragments, pre-split into limbs, to this warp's shared memory
    __syncwarp();
    float qf[NT][2];  // int8: what the scores of heads 2c and 2c + 1 are scaled by
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int g = nt * 8 + r;
      const int64_t qh = row * a.q.sb + (int64_t(head) * a.G + g) * a.q.sh;
      if (C::ES == 2 && QL == 1 && (a.q_vec & 2)) {  // eight bf16 as they are
        uint4 w[D / 32];
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          w[i] = make_uint4(0, 0, 0, 0);
          if (g < a.G)
            load_words<16>(&w[i].x, static_cast<const __nv_bfloat16*>(a.q.p) + qh + i * 32 + c * 8);
        }
        if (nt == 0) fetch(held, cur);  // the table's latency with the query's
#pragma unroll
        for (int i = 0; i < D / 32; ++i) qs[(nt * (D / 32) + i) * 32 + lane] = w[i];
        continue;
      }
      float x[D / 32][8];
#pragma unroll
      for (int i = 0; i < D / 32; ++i)
#pragma unroll
        for (int j = 0; j < 8; j += 4) {
          const int idx = i * 8 + j, d = idx / C::KL * 4 * C::KL + c * C::KL + idx % C::KL;
          float y[4] = {0.0f, 0.0f, 0.0f, 0.0f};
          if (g < a.G) {
            if (!a.q_vec) {
              const float4 z = load_query_slow(a.q.p, qh + d, a.q_dtype);
              y[0] = z.x, y[1] = z.y, y[2] = z.z, y[3] = z.w;
            } else if (QL == 1 || a.q_dtype != FC_DTYPE_F32) {
              load_elems<__nv_bfloat16, 4>(static_cast<const __nv_bfloat16*>(a.q.p) + qh + d, y);
            } else {
              load_elems<float, 4>(static_cast<const float*>(a.q.p) + qh + d, y);
            }
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) x[i][j + e] = y[e];
        }
      if (nt == 0) fetch(held, cur);  // the table's latency with the query's
      if constexpr (C::ES == 1) {
        // a power of two brings the head's largest |q| to [2^14, 2^15)
        float top = 0.0f;
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
#pragma unroll
          for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(x[i][e]));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // (a zero row or one with an infinity: any scale will do)
        int e = top > 0.0f && top <= 3.402823466e+38f ? exponent_of(top) : 14;
        e = e < -100 ? -100 : e;
        const float up = pow2i(14 - e);
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
#pragma unroll
          for (int k = 0; k < 8; ++k) x[i][k] *= up;
        const float down = pow2i(e - 14);
        qf[nt][0] = __shfl_sync(0xffffffffu, down, 8 * c) * a.scale_log2e;
        qf[nt][1] = __shfl_sync(0xffffffffu, down, 8 * c + 4) * a.scale_log2e;
      }
#pragma unroll
      for (int limb = 0; limb < QL; ++limb)
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            w[e] = C::ES == 1 ? take_limb_f16(x[i][2 * e], x[i][2 * e + 1]) : take_limb(x[i][2 * e], x[i][2 * e + 1]);
          qs[((limb * NT + nt) * (D / 32) + i) * 32 + lane] = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
    if (a.kn.p && br.count > 0 && end == rt.n && rt.len > 0) {
      // the fused append: the warp with the segment's last tile stores the new
      // token's rows, which no other warp reads
      const int32_t page = page_of(pv, br.slot, rt.len - 1);
      if (page >= 0) store_new_rows<T, D>(a, row, head, page, (rt.len - 1) & Pm);
    }
    __syncwarp();  // the query's fragments and the new token's rows are visible
    fetch(held + 32, nxt);

    // int8: a head's accumulators hold sum p v times this power of two, so that
    // P times V's scale fits fp16; it begins as high as there is one with a
    // reciprocal in fp32
    float vm[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) vm[nt][0] = vm[nt][1] = C::kMostScale;

    uint32_t kr[U][2][KW / CH] = {}, vr[U][4][VW / CH] = {};
    // where the tiles' halves are: bytes into the layer's pool, scales
    int64_t off[U][2], soff[U][2];
    const int64_t page_bytes = pv.stride_page * C::ES;
    float sk[U][2] = {}, sv[U][2] = {};  // int8: scales of tokens r and r + 8
    bool full = false;                   // every token of the iteration is seen
    // this lane's K row r and V row 2c within a half
    const char* const kp = pv.k + head * (pv.stride_head * C::ES) + r * kRow + c * KB;
    const char* const vp = pv.v + head * (pv.stride_head * C::ES) + 2 * c * kRow + r * VB;

    auto advance = [&](int32_t i) {  // to the tiles from i on
      if (i - held == 32) {
        held = i;
        cur = nxt;
        fetch(held + 32, nxt);
      }
      const int j = i - held;
      constexpr uint32_t kAll = (1u << U) - 1;
      full = (cur.full >> j & kAll) == kAll;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int32_t in = rt.start(i + u) & Pm;
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          const int32_t x = hh == 0 || pv.log2P == 3 ? __shfl_sync(0xffffffffu, cur.page[hh], j + u) : -1;
          if (hh == 0 || pv.log2P == 3) {
            off[u][hh] = x < 0 ? -1 : x * page_bytes + ((in + 8 * hh) & Pm) * kRow;
            if constexpr (C::ES == 1) soff[u][hh] = x * pv.sstride_page + ((in + 8 * hh) & Pm);
          } else {
            off[u][1] = off[u][0] < 0 ? -1 : off[u][0] + 8 * kRow;
            if constexpr (C::ES == 1) soff[u][1] = soff[u][0] + 8;
          }
        }
      }
    };
    auto load_k = [&](int32_t i, int part) {
      auto rows = [&](auto on) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            const char* p = kp + off[u][hh] + part * (KW / CH) * 16;
            if (on(u, hh)) {
#pragma unroll
              for (int j = 0; j < KW / CH; j += KB / 4) load_words<KB>(&kr[u][hh][j], p + j * 16);
            }
            if constexpr (C::ES == 1) {
              const int64_t se = soff[u][hh] + head * pv.sstride_head + r;
              if (on(u, hh)) {
                load_words<4>(reinterpret_cast<uint32_t*>(&sk[u][hh]), pv.ks + se);
                load_words<4>(reinterpret_cast<uint32_t*>(&sv[u][hh]), pv.vs + se);
              } else {
                sv[u][hh] = 0.0f;  // (a masked K row may hold anything: its score is replaced)
              }
            }
          }
      };
      if (full) rows([](int, int) { return true; });
      else rows([&](int u, int hh) { return off[u][hh] >= 0 && rt.sees(rt.start(i + u) + hh * 8 + r); });
    };
    auto load_v = [&](int32_t i, int part) {
      auto rows = [&](auto on) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const char* p = vp + off[u][k >> 1] + (k & 1) * kRow + part * (VW / CH) * 32;
            if (on(u, k)) {
#pragma unroll
              for (int j = 0; j < VW / CH; j += VB / 4) load_words<VB>(&vr[u][k][j], p + j * 32);
            } else {
#pragma unroll
              for (int j = 0; j < VW / CH; ++j) vr[u][k][j] = 0;
            }
          }
      };
      if (full) rows([](int, int) { return true; });
      else
        rows([&](int u, int k) {
          return off[u][k >> 1] >= 0 && rt.sees(rt.start(i + u) + (k >> 1) * 8 + 2 * c + (k & 1));
        });
    };

    if constexpr (!C::kPrefetch) {
      advance(tile);
      load_k(tile, 0);
    }
    // The first pass only loads (the loads' code is there once).
#pragma unroll 1
    for (int32_t i = C::kPrefetch ? tile - U : tile; i < end; i += U) {
      const bool work = !C::kPrefetch || i >= tile;
      float s[U][NT][4], svc[U][2];
      if constexpr (!C::kPrefetch) load_v(i, 0);
      if (work) {
        // ---- S^T = K Q^T
        // a second chain of dependent products; in an fp32 result, whose last
        // bits the tensor cores' truncated sums would bias, the small ones
        float odd[U][NT][4] = {};
#pragma unroll
        for (int part = 0; part < CH; ++part) {
          if (part > 0) load_k(i, part);
          constexpr int STEPS = D / 16 / CH;  // k-steps of 16 channels per part
          static_assert(STEPS % 2 == 0, "two chains");
          uint4 qb[QL][NT];  // the query's words of two k-steps
#pragma unroll
          for (int ks = 0; ks < STEPS; ++ks) {
            const int kk = part * STEPS + ks;
            // fp32 pages have three limbs; the others are exact as they are
            constexpr int KLIMBS = C::ES == 4 ? 3 : 1;
            uint32_t ka[U][KLIMBS][4];
#pragma unroll
            for (int u = 0; u < U; ++u) {
              if constexpr (C::ES == 4) {
                float x[2][4];
#pragma unroll
                for (int hh = 0; hh < 2; ++hh)
#pragma unroll
                  for (int e = 0; e < 4; ++e) x[hh][e] = __uint_as_float(kr[u][hh][4 * ks + e]);
#pragma unroll
                for (int k = 0; k < 3; ++k)
#pragma unroll
                  for (int e = 0; e < 4; ++e) ka[u][k][e] = take_limb(x[e & 1][e & 2], x[e & 1][(e & 2) + 1]);
              } else if constexpr (C::ES == 2) {
#pragma unroll
                for (int e = 0; e < 4; ++e) ka[u][0][e] = kr[u][e & 1][2 * ks + (e >> 1)];
              } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  ka[u][0][e] = codes_to_f16(
                      __byte_perm(kr[u][e & 1][ks] ^ 0x80808080u, 0x64646464u, e < 2 ? 0x4140 : 0x4342));
              }
            }
#pragma unroll
            for (int ql = 0; ql < QL; ++ql)
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                if ((kk & 1) == 0) qb[ql][nt] = qs[((ql * NT + nt) * (D / 32) + kk / 2) * 32 + lane];
                const uint2 b = kk & 1 ? make_uint2(qb[ql][nt].z, qb[ql][nt].w) : make_uint2(qb[ql][nt].x, qb[ql][nt].y);
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                  for (int k = 0; k < KLIMBS; ++k) {
                    if (k + ql > 2) continue;
                    if constexpr (kFine) {
                      // each step's leading product on its own, added in fp32;
                      // the small ones (2^-8 and less) in a sum of their own
                      if (ql == 0 && k == 0) {
                        float t[4];
                        mma<T, true>(t, ka[u][k], b.x, b.y);
#pragma unroll
                        for (int e = 0; e < 4; ++e) s[u][nt][e] = kk == 0 ? t[e] : s[u][nt][e] + t[e];
                      } else if (kk == 0 && (KLIMBS > 1 ? ql == 0 && k == 1 : ql == 1)) {
                        mma<T, true>(odd[u][nt], ka[u][k], b.x, b.y);
                      } else {
                        mma<T, false>(odd[u][nt], ka[u][k], b.x, b.y);
                      }
                      continue;
                    }
                    auto& d = kk & 1 ? odd[u][nt] : s[u][nt];
                    if (kk <= 1 && ql == 0 && k == 0) mma<T, true>(d, ka[u][k], b.x, b.y);
                    else mma<T, false>(d, ka[u][k], b.x, b.y);
                  }
              }
          }
        }
        // ---- scores in the log2 domain, masked
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int hh = 0; hh < 2; ++hh)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                float& x = s[u][nt][2 * hh + j];
                x += odd[u][nt][2 * hh + j];
                if constexpr (C::ES == 1) x *= sk[u][hh] * qf[nt][j];
                else x *= a.scale_log2e;
              }
        if (!full) {
#pragma unroll
          for (int u = 0; u < U; ++u)
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
              if (off[u][hh] >= 0 && rt.sees(rt.start(i + u) + hh * 8 + r)) continue;
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) s[u][nt][2 * hh] = s[u][nt][2 * hh + 1] = kNone;
            }
        }
        if constexpr (C::ES == 1) {
#pragma unroll
          for (int u = 0; u < U; ++u) {
            svc[u][0] = sv[u][0];  // before the next ones are loaded
            svc[u][1] = sv[u][1];
          }
        }
      }
      if constexpr (C::kPrefetch) {
        advance(i + U);
        load_k(i + U, 0);
      }
      if (work) {
        // ---- running maximum, raised only where a score passes it by 2^kLazy
        bool raise = false;
        float top[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float x = fmaxf(s[0][nt][j], s[0][nt][2 + j]);
#pragma unroll
            for (int u = 1; u < U; ++u) x = fmaxf(x, fmaxf(s[u][nt][j], s[u][nt][2 + j]));
            top[nt][j] = x;
            raise |= x > m[nt][j] + C::kLazy;
          }
        if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              float x = top[nt][j];
#pragma unroll
              for (int o = 4; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
              x = fmaxf(x, m[nt][j]);
              float e = join_factor(m[nt][j], x);
              m[nt][j] = x;
              l[nt][j] *= e;
              if constexpr (C::ES == 1) {
                // what the maximum takes away the scale may give back, or the
                // tokens before would set the later ones' precision
                const float g = lower_power(e, vm[nt][j]);
                vm[nt][j] *= g;
                e *= g;
              }
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) {
                acc[nt * MT + mt][j] *= e;
                acc[nt * MT + mt][2 + j] *= e;
              }
            }
        }

        // ---- P, and its limbs as B operands (heads x tokens)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          // no score yet: the maximum is -infinity and p is to be 0
          const float b0 = m[nt][0] == kNone ? 0.0f : m[nt][0], b1 = m[nt][1] == kNone ? 0.0f : m[nt][1];
#pragma unroll
          for (int u = 0; u < U; ++u)
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
              float& p0 = s[u][nt][2 * hh];
              float& p1 = s[u][nt][2 * hh + 1];
              p0 = fast_exp2(p0 - b0);
              p1 = fast_exp2(p1 - b1);
              l[nt][0] += p0;
              l[nt][1] += p1;
              if constexpr (C::ES == 1) {
                p0 *= svc[u][hh];
                p1 *= svc[u][hh];
              }
            }
        }
        if constexpr (C::ES == 1) {
          // P times V's scale, in the head's power of two: lowered where a
          // product passes 2^15, to bring the largest of the tile to [2^7, 2^8)
          bool low = false;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              float x = fmaxf(fabsf(s[0][nt][j]), fabsf(s[0][nt][2 + j]));
#pragma unroll
              for (int u = 1; u < U; ++u) x = fmaxf(x, fmaxf(fabsf(s[u][nt][j]), fabsf(s[u][nt][2 + j])));
              top[nt][j] = x;
              low |= top[nt][j] * vm[nt][j] > 32768.0f;
            }
          if (__any_sync(0xffffffffu, low)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                float x = top[nt][j];
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
                if (x * vm[nt][j] <= 32768.0f) continue;
                const int now = 7 - exponent_of(x), e = now - exponent_of(vm[nt][j]);
                vm[nt][j] = pow2i(now);
                const float f = pow2i(e < -126 ? -126 : e);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                  acc[nt * MT + mt][j] *= f;
                  acc[nt * MT + mt][2 + j] *= f;
                }
              }
          }
        }
        uint32_t pb[U][PL][NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int u = 0; u < U; ++u)
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
              float p0 = s[u][nt][2 * hh], p1 = s[u][nt][2 * hh + 1];
              if constexpr (C::ES == 1) {
                p0 *= vm[nt][0];
                p1 *= vm[nt][1];
              }
#pragma unroll
              for (int k = 0; k < PL; ++k) {
                // bf16: the last limb is rounded, the ones before are cut at eight bits
                const uint32_t w = C::ES == 1 ? take_limb_f16(p0, p1)
                                              : k == PL - 1 ? pack_bf16(p0, p1) : take_limb(p0, p1);
                pb[u][k][nt][hh] = transpose8x8(w);
              }
            }

        // ---- O^T += V^T P^T: the iteration's products in accumulators of their
        // own, added in fp32 (the tensor cores' running sums are truncated)
#pragma unroll
        for (int part = 0; part < CH; ++part) {
          if (part > 0) load_v(i, part);
          if (!C::kPrefetch && part == CH - 1) {
            advance(i + U);
            load_k(i + U, 0);
          }
#pragma unroll
          for (int mt = 0; mt < MT / CH; ++mt) {
            float o[NT][4];
#pragma unroll
            for (int u = 0; u < U; ++u) {
              constexpr int VLIMBS = C::ES == 4 ? 3 : 1;
              uint32_t va[VLIMBS][4];
              if constexpr (C::ES == 4) {
                float x[4][2];
#pragma unroll
                for (int k = 0; k < 4; ++k)
#pragma unroll
                  for (int e = 0; e < 2; ++e) x[k][e] = __uint_as_float(vr[u][k][2 * mt + e]);
#pragma unroll
                for (int k = 0; k < 3; ++k)
#pragma unroll
                  for (int e = 0; e < 4; ++e) va[k][e] = take_limb(x[e & 2][e & 1], x[(e & 2) + 1][e & 1]);
              } else if constexpr (C::ES == 2) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  va[0][e] = __byte_perm(vr[u][e & 2][mt], vr[u][(e & 2) + 1][mt], e & 1 ? 0x7632 : 0x5410);
              } else {
                // codes 2 mt and 2 mt + 1 of each token: bytes of word mt / 2
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const uint32_t sel = (mt & 1 ? 0x0602u : 0x0400u) + (e & 1 ? 0x0101u : 0u);
                  va[0][e] = codes_to_f16(
                      (__byte_perm(vr[u][e & 2][mt / 2], vr[u][(e & 2) + 1][mt / 2], sel) & 0x00ff00ffu) ^ 0x64806480u);
                }
              }
#pragma unroll
              for (int v = VLIMBS - 1; v >= 0; --v)
#pragma unroll
                for (int k = PL - 1; k >= 0; --k) {  // the small products first
                  if (v + k > 2) continue;
#pragma unroll
                  for (int nt = 0; nt < NT; ++nt) {
                    if (u == 0 && v == VLIMBS - 1 && k == (PL - 1 < 3 - VLIMBS ? PL - 1 : 3 - VLIMBS))
                      mma<T, true>(o[nt], va[v], pb[u][k][nt][0], pb[u][k][nt][1]);
                    else mma<T, false>(o[nt], va[v], pb[u][k][nt][0], pb[u][k][nt][1]);
                  }
                }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 4; ++e) acc[nt * MT + part * (MT / CH) + mt][e] += o[nt][e];
          }
        }
      }
      if constexpr (C::kPrefetch) load_v(i + U, 0);
    }

    // ---- an infinity's limbs (inf - inf, or inf times a limb that is 0) are NaN
    // where its products are not: heads with a NaN are done again without limbs.
    // (An int8 row with one reads as NaN.)
    if constexpr (C::ES != 1) {
      bool bad = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) bad |= l[nt][0] != l[nt][0] || l[nt][1] != l[nt][1];
#pragma unroll
      for (int q = 0; q < C::NQ; ++q)
#pragma unroll
        for (int k = 0; k < 4; ++k) bad |= acc[q][k] != acc[q][k];
      if (__any_sync(0xffffffffu, bad)) {
        Share<C> x;  // (through memory: the loop's registers stay its own)
        copy_share<C>(x.acc, x.m, x.l, acc, m, l);
        attend_plain<T, C>(a, br.slot, row, head, rt, tile, end, x);
        copy_share<C>(acc, m, l, x.acc, x.m, x.l);
      }
    }

    // ---- the segment's sums over the lanes' tokens; whole segments are done
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) l[nt][j] += __shfl_xor_sync(0xffffffffu, l[nt][j], o);
    if constexpr (C::ES == 1) {
#pragma unroll
      for (int q = 0; q < C::NQ; ++q)
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[q][k] *= pow2i(-exponent_of(vm[q / MT][k & 1]));
    }
    }  // rt.len > 0
    if (tile == 0 && end == rt.n) {
      float f[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          f[nt][j] = l[nt][j] == 0.0f ? 0.0f : 1.0f / l[nt][j];
          if (r == 0) store_lse(a, row, head, nt * 8 + 2 * c + j, m[nt][j], l[nt][j]);
        }
      if (!a.out_vec) {
#pragma unroll
        for (int q = 0; q < C::NQ; ++q)
          store_quad<C>(a, row, head, q, make_float4(acc[q][0], acc[q][1], acc[q][2], acc[q][3]), f[q / MT][0], f[q / MT][1]);
      } else if (a.out_dtype == FC_DTYPE_F32) {
        store_all<C, float>(a, row, head, acc, f);
      } else {
        store_all<C, __nv_bfloat16>(a, row, head, acc, f);
      }
    } else {
      const Fragment<C> f{fragments + (warp * 2 + made) * C::kFragment};
#pragma unroll
      for (int q = 0; q < C::NQ; ++q) f.acc(q, lane) = make_float4(acc[q][0], acc[q][1], acc[q][2], acc[q][3]);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          if (r == 0) {
            f.m(nt * 8 + 2 * c + j) = m[nt][j];
            f.l(nt * 8 + 2 * c + j) = l[nt][j];
          }
      if (lane == 0) pieces[warp * 2 + made] = Piece{row, head, tile, end, rt.n};
      ++made;
    }
    if (++head == H) head = 0, ++row;
  }
  if (lane == 0) n_pieces[warp] = made;
  __syncthreads();

  // ---- join the CTA's fragments, segment by segment. A segment's fragments
  // are the last one of the warp it begins in (or, where it began before this
  // CTA, the first one of warp 0) and the first ones of the warps after it, up
  // to the warp that ends it.
  const int held_by = lane < C::WARPS ? n_pieces[lane] : 0;
  const Piece p0 = pieces[2 * (lane < C::WARPS ? lane : 0)];
  const Piece pl = pieces[held_by > 0 ? 2 * lane + held_by - 1 : 0];
  const unsigned used = __ballot_sync(0xffffffffu, held_by > 0);
  const unsigned ends = __ballot_sync(0xffffffffu, held_by > 0 && p0.to == p0.n);
  // bit 0: a segment that began before; bit w + 1: one that begins in warp w
  const unsigned starts = __ballot_sync(0xffffffffu, held_by > 0 && pl.from == 0) << 1 |
                          (__ballot_sync(0xffffffffu, lane == 0 && held_by > 0 && p0.from > 0) ? 1u : 0u);
  const int groups = __popc(starts), last_warp = 31 - __clz(int(used | 1u));
  const uint32_t span = cta_chunk >> 31 ? 0x7fffffffu : uint32_t(cta_chunk);
  // the slot a segment's fragments begin at (bit: its bit in `starts`), and the
  // warp that holds its last one
  auto first_slot = [&](int bit) { return bit > 0 ? 2 * (bit - 1) + n_pieces[bit - 1] - 1 : 0; };
  auto end_warp = [&](int slot) {
    const unsigned after = ends & (0xfffffffeu << (slot >> 1));
    return pieces[slot].to == pieces[slot].n ? slot >> 1 : after ? __ffs(int(after)) - 1 : last_warp;
  };
  auto upto = [&](int slot, int w1) { return pieces[w1 > slot >> 1 ? 2 * w1 : slot].to; };

  // what each fragment is multiplied by: a thread per fragment and head
  {
    const int slot = int(threadIdx.x) / (NT * 8), h = int(threadIdx.x) % (NT * 8), w = slot >> 1;
    if (slot < 2 * C::WARPS && (slot & 1) < n_pieces[w]) {
      const int lead = pieces[slot].from == 0 ? slot : first_slot(31 - __clz(int(starts & ((2u << w) - 1))));
      const int w1 = end_warp(lead), n = w1 - (lead >> 1) + 1;
      auto at_ = [&](int i) { return Fragment<C>{fragments + (i == 0 ? lead : (lead & ~1) + 2 * i) * C::kFragment}; };
      float M = kNone, L = 0.0f;
#pragma unroll 4
      for (int i = 0; i < n; ++i) M = fmaxf(M, at_(i).m(h));
#pragma unroll 4
      for (int i = 0; i < n; ++i) L += at_(i).l(h) * join_factor(at_(i).m(h), M);
      const Piece first = pieces[lead];
      const int32_t to = upto(lead, w1);
      const bool whole = first.from == 0 && to == first.n;
      const float e = join_factor(Fragment<C>{fragments + slot * C::kFragment}.m(h), M);
      factors[slot][h] = !whole ? e : L == 0.0f ? 0.0f : e / L;
      if (slot == lead && whole) store_lse(a, first.row, first.head, h, M, L);
      if (slot == lead && !whole) {
        const int j = first.from > 0 ? 0 : 1;
        const Fragment<C> f{a.partials + (int64_t(blockIdx.x) * 2 + j) * C::kFragment};
        f.m(h) = M;
        f.l(h) = L;
        if (h == 0)  // the CTAs it lies in: its tiles before and after this one's
          open[j] = Open{first.row, first.head, int32_t(blockIdx.x - (uint32_t(first.from) + span - 1) / span),
                         int32_t(blockIdx.x + (uint32_t(first.n - to) + span - 1) / span)};
      }
    }
  }
  __syncthreads();
#pragma unroll 1
  for (int i = warp; i < groups * C::NQ; i += C::WARPS) {
    unsigned rest = starts;  // its (i / NQ)-th bit
    for (int k = i / C::NQ; k > 0; --k) rest &= rest - 1;
    const int lead = first_slot(__ffs(int(rest)) - 1), w1 = end_warp(lead), n = w1 - (lead >> 1) + 1;
    const int q = i % C::NQ, hc = q / MT * 8 + 2 * c;
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
    for (int k = 0; k < n; ++k) {
      const int slot = k == 0 ? lead : (lead & ~1) + 2 * k;
      const float4 v = Fragment<C>{fragments + slot * C::kFragment}.acc(q, lane);
      const float2 e = *reinterpret_cast<const float2*>(&factors[slot][hc]);
      acc.x += v.x * e.x;
      acc.y += v.y * e.y;
      acc.z += v.z * e.x;
      acc.w += v.w * e.y;
    }
    const Piece first = pieces[lead];
    if (first.from == 0 && upto(lead, w1) == first.n) {
      store_quad<C>(a, first.row, first.head, q, acc, 1.0f, 1.0f);
    } else {
      Fragment<C>{a.partials + (int64_t(blockIdx.x) * 2 + (first.from > 0 ? 0 : 1)) * C::kFragment}.acc(q, lane) = acc;
    }
  }
  __syncthreads();

  // ---- the last CTA of a segment joins the CTAs' fragments (an atomic ticket
  // at the segment's first CTA; the fence makes the CTA's fragments, ordered
  // before it by the barrier, visible to the CTA that comes last)
  if (threadIdx.x < 2 && open[threadIdx.x].row >= 0) {
    Open& o = open[threadIdx.x];
    __threadfence();
    const uint32_t n = atomicAdd(&a.tickets[o.cta0], 1u);
    if (n == uint32_t(o.cta1 - o.cta0)) {
      a.tickets[o.cta0] = 0;
      __threadfence();
    } else {
      o.row = -1;
    }
  }
  __syncthreads();
#pragma unroll 1
  for (int j = 0; j < 2; ++j) {
    const Open o = open[j];
    if (o.row < 0) continue;
    // fragment 0 is its CTA's second, every later one its CTA's first
    const int n = o.cta1 - o.cta0 + 1;
    auto at_ = [&](int i) {
      return Fragment<C>{a.partials + (int64_t(o.cta0 + i) * 2 + (i == 0 ? 1 : 0)) * C::kFragment};
    };
    constexpr int N = 16;  // loads in flight per lane
    float4 v[N];
    auto load = [&](int q, int i0) {
#pragma unroll
      for (int k = 0; k < N; ++k)
        v[k] = i0 + k < n ? at_(i0 + k).acc(q, lane) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    };
    if (warp < C::NQ) load(warp, 0);  // before the factors are known
    float* fs = reinterpret_cast<float*>(smem);  // [n][NT 8], by a warp per head
#pragma unroll 1
    for (int h = warp; h < NT * 8; h += C::WARPS) {
      float M = kNone, L = 0.0f;
#pragma unroll 1
      for (int k = lane; k < n; k += 32) M = fmaxf(M, at_(k).m(h));
      M = warp_max(M);
#pragma unroll 1
      for (int k = lane; k < n; k += 32) L += at_(k).l(h) * join_factor(at_(k).m(h), M);
      L = warp_sum(L);
#pragma unroll 1
      for (int k = lane; k < n; k += 32) fs[k * NT * 8 + h] = L == 0.0f ? 0.0f : join_factor(at_(k).m(h), M) / L;
      if (lane == 0) store_lse(a, o.row, o.head, h, M, L);
    }
    __syncthreads();
#pragma unroll 1
    for (int q = warp; q < C::NQ; q += C::WARPS) {
      const int hc = q / MT * 8 + 2 * c;
      if (q != warp) load(q, 0);
      float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 1
      for (int i0 = 0;;) {
#pragma unroll
        for (int k = 0; k < N; ++k)
          if (i0 + k < n) {
            const float2 e = *reinterpret_cast<const float2*>(&fs[(i0 + k) * NT * 8 + hc]);
            acc.x += v[k].x * e.x;
            acc.y += v[k].y * e.y;
            acc.z += v[k].z * e.x;
            acc.w += v[k].w * e.y;
          }
        if ((i0 += N) >= n) break;
        load(q, i0);
      }
      store_quad<C>(a, o.row, o.head, q, acc, 1.0f, 1.0f);
    }
    __syncthreads();
  }
}

template <typename T, int D, int NT, int QL, int PL>
int launch_paged(const PagedArgs& a, cudaStream_t s) {
  using C = PagedCfg<T, D, NT, QL, PL>;
  auto* kernel = paged_attention_kernel<T, D, NT, QL, PL>;
  static std::atomic<bool> set[64];  // once per device
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return FC_ERR_CUDA;
  if (!set[dev]) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(C::kShared)) != cudaSuccess)
      return FC_ERR_CUDA;
    set[dev] = true;
  }
  const int ctas = sm_count() * kPagedCtasPerSm;
  return launch_after(kernel, dim3(unsigned(ctas < C::kMostCtas ? ctas : C::kMostCtas)), C::WARPS * 32, C::kShared, s,
                      a);
}

template <typename T, int QL, int PL>
int launch_paged_sizes(const PagedArgs& a, int64_t D, cudaStream_t s) {
  const bool two = a.G > 8;
  switch (D) {
    case 32:
      return two ? launch_paged<T, 32, 2, QL, PL>(a, s) : launch_paged<T, 32, 1, QL, PL>(a, s);
    case 64:
      return two ? launch_paged<T, 64, 2, QL, PL>(a, s) : launch_paged<T, 64, 1, QL, PL>(a, s);
    case 128:
      return two ? launch_paged<T, 128, 2, QL, PL>(a, s) : launch_paged<T, 128, 1, QL, PL>(a, s);
    case 256:
      return two ? launch_paged<T, 256, 2, QL, PL>(a, s) : launch_paged<T, 256, 1, QL, PL>(a, s);
  }
  return FC_ERR_UNSUPPORTED;
}

#endif  // __CUDACC__

}  // namespace fc
