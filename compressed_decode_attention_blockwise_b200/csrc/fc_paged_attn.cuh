// Single-token decode attention over a paged cache (include/fc_paged.h).
//
// What it computes, per sequence and kv head, over the tokens t a row sees:
//   s_t = sigma q.k_t,  out = sum e^(s_t - m) v_t / sum e^(s_t - m)
// for the G query heads that share the kv head.
//
// What bounds it: HBM. Every seen K and V row is read once per kv head and
// serves its whole group; at G = 8 and bf16 that is 8 multiply-adds per byte,
// above what CUDA-core FMAs sustain at full bandwidth and a small share of the
// tensor cores' rate. So both products run as mma.sync m16n8k16 (bf16 in, fp32
// out) with the TOKENS (and for V the channels) on the 16-wide side and the
// heads on the 8-wide one:
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
// it is fp32, and P times V's scale (by a power of two per warp) is two.
// Maxima, sums and accumulators are fp32.
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
  int32_t q_limbs, p_limbs;
  float scale_log2e;
  int32_t window, sinks;
  void* out;
  int64_t os_b, os_h;
  int32_t out_dtype;
  float* lse;
  uint32_t* tickets;   // one per CTA
  char* partials;      // two fragments per CTA
};

int launch_paged_attention_bf16(const PagedArgs& a, int64_t D, cudaStream_t s);
int launch_paged_attention_f32(const PagedArgs& a, int64_t D, cudaStream_t s);
int launch_paged_attention_i8(const PagedArgs& a, int64_t D, cudaStream_t s);

// CTAs a launch may have (the workspace is sized for them).
constexpr int kPagedCtasPerSm = 1;
// Bytes of one fragment in the workspace.
inline size_t paged_fragment_bytes(int64_t D, int64_t G) {
  const size_t nt = G > 8 ? 2 : 1;
  return nt * size_t(D) / 16 * 512 + nt * 64;
}

#ifdef __CUDACC__

constexpr int kTile = 16;          // tokens per tile
constexpr float kLazy = 8.0f;      // log2 of how far p may exceed 1

template <typename T, int D_, int NT_>
struct PagedCfg {
  static constexpr int D = D_, NT = NT_;      // NT: groups of 8 heads
  static constexpr int ES = int(sizeof(T));
  static constexpr int KW = D / 4 * ES / 4;   // words of a K row per lane
  static constexpr int VW = D / 8 * ES / 4;   // words of a V row per lane
  static constexpr int KL = 16 / ES < D / 4 ? 16 / ES : D / 4;  // elements per load
  static constexpr int VL = 16 / ES < D / 8 ? 16 / ES : D / 8;
  // tiles per iteration: as many as keep 4 KB of K in flight per warp
  static constexpr int U = KW >= 16 ? 1 : KW == 8 ? 2 : 4;
  // rows too wide for the registers are taken in parts, without prefetch
  static constexpr int kRegs = NT * D / 4 + U * (2 * KW + 4 * VW);
  static constexpr int CH = kRegs <= 192 ? 1 : kRegs <= 256 ? 2 : 4;
  static constexpr bool kPrefetch = CH == 1;
  static constexpr int NQ = NT * D / 16;      // float4 accumulators per lane
  static constexpr int WARPS = NQ >= 32 ? 4 : kRegs <= 96 ? 12 : 8;
  static constexpr size_t kFragment = size_t(NQ) * 512 + NT * 64;
  static constexpr size_t q_bytes(int limbs) { return size_t(limbs) * NT * (D / 32) * 512; }
};

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
template <typename T>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                    uint32_t b0, uint32_t b1) {
  if constexpr (sizeof(T) == 1) mma_f16(d, a0, a1, a2, a3, b0, b1);
  else mma_bf16(d, a0, a1, a2, a3, b0, b1);
}

// 2^e for -126 <= e <= 127.
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }
// The exponent of a positive finite x (its floor of log2; subnormals -127).
__device__ __forceinline__ int exponent_of(float x) { return int(__float_as_uint(x) >> 23) - 127; }

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
// the fp16 numbers 1024 + code + 128; 1152 is subtracted.
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
  __device__ __forceinline__ RowTiles(int32_t slot, int32_t length, int32_t window, int32_t sink) {
    len = slot < 0 ? 0 : length;
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

// Writes the (already joined) accumulator quad q of one lane: heads 8 nt + 2c
// and + 1, channels d and d + 1 of D.
template <typename C, typename T>
__device__ __forceinline__ void store_quad(const PagedArgs& a, int32_t row, int32_t head, int q, int lane,
                                           const float (&acc)[4], const float (&l)[2]) {
  const int nt = q / (C::D / 16), mt = q % (C::D / 16), r = lane >> 2, c = lane & 3;
  const int idx = 2 * mt, d = idx / C::VL * 8 * C::VL + r * C::VL + idx % C::VL;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int g = nt * 8 + 2 * c + j;
    if (g >= a.G) continue;
    const float inv = l[j] == 0.0f ? 0.0f : 1.0f / l[j];
    const float x0 = l[j] == 0.0f ? 0.0f : acc[j] * inv, x1 = l[j] == 0.0f ? 0.0f : acc[2 + j] * inv;
    const int64_t at = row * a.os_b + (int64_t(head) * a.G + g) * a.os_h + d;
    if (a.out_dtype == FC_DTYPE_F32) {
      float* o = static_cast<float*>(a.out) + at;
      if (a.out_vec) {
        *reinterpret_cast<float2*>(o) = make_float2(x0, x1);
      } else {
        o[0] = x0;
        o[1] = x1;
      }
    } else {
      __nv_bfloat16* o = static_cast<__nv_bfloat16*>(a.out) + at;
      if (a.out_vec) {
        *reinterpret_cast<uint32_t*>(o) = pack_bf16(x0, x1);
      } else {
        o[0] = __float2bfloat16_rn(x0);
        o[1] = __float2bfloat16_rn(x1);
      }
    }
  }
}

// lse = ln 2 (m + log2 l) of the lane's two heads, by the lanes of row r = 0.
__device__ __forceinline__ void store_lse(const PagedArgs& a, int32_t row, int32_t head, int nt, int lane,
                                          const float (&m)[2], const float (&l)[2]) {
  if (!a.lse || lane >= 4) return;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int g = nt * 8 + 2 * lane + j;
    if (g < a.G)
      a.lse[(int64_t(row) * a.pages.H + head) * a.G + g] =
          l[j] == 0.0f ? __int_as_float(0xff800000) : 0.6931471805599453f * (m[j] + log2f(l[j]));
  }
}

// A segment's part in shared memory or the workspace: NQ x 32 float4
// accumulators, then NT x 8 maxima (log2 domain), then NT x 8 sums.
template <typename C>
struct Fragment {
  const char* p;
  __device__ __forceinline__ float4 acc(int q, int lane) const {
    return reinterpret_cast<const float4*>(p)[q * 32 + lane];
  }
  __device__ __forceinline__ float2 m(int nt, int c) const {
    return reinterpret_cast<const float2*>(p + size_t(C::NQ) * 512)[nt * 4 + c];
  }
  __device__ __forceinline__ float2 l(int nt, int c) const {
    return reinterpret_cast<const float2*>(p + size_t(C::NQ) * 512 + C::NT * 32)[nt * 4 + c];
  }
};

// What a warp left of a segment (row, head): tiles [from, to) of n.
struct Piece {
  int32_t row, head, from, to, n;
};

// Joins n fragments (at(i)) for quad q: the lane's accumulators, maxima, sums.
template <typename C, typename At>
__device__ __forceinline__ void join(int n, At at, int q, int lane, float (&acc)[4], float (&m)[2],
                                     float (&l)[2]) {
  const int nt = q / (C::D / 16), c = lane & 3;
  m[0] = m[1] = __int_as_float(0xff800000);
  for (int i = 0; i < n; ++i) {
    const float2 x = Fragment<C>{at(i)}.m(nt, c);
    m[0] = fmaxf(m[0], x.x);
    m[1] = fmaxf(m[1], x.y);
  }
  acc[0] = acc[1] = acc[2] = acc[3] = l[0] = l[1] = 0.0f;
#pragma unroll 4
  for (int i = 0; i < n; ++i) {
    const Fragment<C> f{at(i)};
    const float2 mi = f.m(nt, c), li = f.l(nt, c);
    const float4 v = f.acc(q, lane);
    const float e0 = join_factor(mi.x, m[0]), e1 = join_factor(mi.y, m[1]);
    l[0] += li.x * e0;
    l[1] += li.y * e1;
    acc[0] += v.x * e0;
    acc[1] += v.y * e1;
    acc[2] += v.z * e0;
    acc[3] += v.w * e1;
  }
}

template <typename C>
__device__ __forceinline__ void store_fragment(char* p, int q, int lane, const float (&acc)[4],
                                               const float (&m)[2], const float (&l)[2]) {
  reinterpret_cast<float4*>(p)[q * 32 + lane] = make_float4(acc[0], acc[1], acc[2], acc[3]);
  const int nt = q / (C::D / 16);
  if (q % (C::D / 16) == 0 && lane < 4) {
    reinterpret_cast<float2*>(p + size_t(C::NQ) * 512)[nt * 4 + lane] = make_float2(m[0], m[1]);
    reinterpret_cast<float2*>(p + size_t(C::NQ) * 512 + C::NT * 32)[nt * 4 + lane] = make_float2(l[0], l[1]);
  }
}

template <typename T, int D, int NT>
__global__ void __launch_bounds__(PagedCfg<T, D, NT>::WARPS * 32, 1)
    paged_attention_kernel(const __grid_constant__ PagedArgs a) {
  using C = PagedCfg<T, D, NT>;
  constexpr int U = C::U, KW = C::KW, VW = C::VW, CH = C::CH, MT = D / 16;
  constexpr int KB = C::KL * C::ES, VB = C::VL * C::ES;  // bytes per load
  extern __shared__ __align__(16) char smem[];
  __shared__ Piece pieces[C::WARPS * 2];
  __shared__ int n_pieces[C::WARPS];
  __shared__ int last_of[2];
  const int warp = int(threadIdx.x >> 5), lane = int(threadIdx.x & 31), r = lane >> 2, c = lane & 3;
  char* fragments = smem;  // two per warp
  uint4* qs = reinterpret_cast<uint4*>(smem + C::WARPS * 2 * C::kFragment + warp * C::q_bytes(a.q_limbs));
  const PageView& pv = a.pages;
  const int H = pv.H;

  // ---- the warp's share of the line of tiles
  const int per = (pv.n_rows + 31) / 32;
  int64_t mine = 0;
  for (int i = 0; i < per; ++i) {
    const int b = lane * per + i;
    if (b < pv.n_rows) mine += RowTiles(pv.batch[b].slot, pv.batch[b].len, a.window, a.sinks).n;
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
  // no fewer than U tiles per warp: a small batch takes fewer CTAs
  int64_t ctas = (total + C::WARPS * U - 1) / (C::WARPS * U);
  if (ctas > int64_t(gridDim.x)) ctas = gridDim.x;
  if (int64_t(blockIdx.x) >= ctas) return;
  const int64_t cta_from = total * blockIdx.x / ctas, cta_to = total * (blockIdx.x + 1) / ctas;
  const int64_t from = cta_from + (cta_to - cta_from) * warp / C::WARPS;
  const int64_t to = cta_from + (cta_to - cta_from) * (warp + 1) / C::WARPS;

  int32_t row = 0, head = 0, tile = 0;
  if (from < to) {
    const unsigned who = __ballot_sync(0xffffffffu, before <= from && from < before + mine);
    const int src = __ffs(int(who)) - 1;
    if (lane == src) {
      int64_t base = before;
      row = lane * per;
      while (row < pv.n_rows) {
        const int32_t n = RowTiles(pv.batch[row].slot, pv.batch[row].len, a.window, a.sinks).n;
        if (from < base + int64_t(n) * H) {
          head = int32_t((from - base) / n);
          tile = int32_t((from - base) % n);
          break;
        }
        base += int64_t(n) * H;
        ++row;
      }
    }
    row = __shfl_sync(0xffffffffu, row, src);
    head = __shfl_sync(0xffffffffu, head, src);
    tile = __shfl_sync(0xffffffffu, tile, src);
  }

  // ---- the segments of the share
  int made = 0;  // fragments left in shared memory
  int64_t at = from;
  while (at < to && row < pv.n_rows) {
    const BatchRow br = pv.batch[row];
    const RowTiles rt(br.slot, br.len, a.window, a.sinks);
    const int32_t end = int64_t(rt.n - tile) < to - at ? rt.n : tile + int32_t(to - at);

    // query fragments, pre-split into limbs, to this warp's shared memory
    __syncwarp();
    float qf[NT][2];  // int8: what the scores of heads 2c and 2c + 1 are scaled by
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int g = nt * 8 + r;
      const int64_t qh = row * a.q.sb + (int64_t(head) * a.G + g) * a.q.sh;
      float x[D / 32][8];
#pragma unroll
      for (int i = 0; i < D / 32; ++i)
#pragma unroll
        for (int j = 0; j < 8; j += 4) {
          const int idx = i * 8 + j, d = idx / C::KL * 4 * C::KL + c * C::KL + idx % C::KL;
          float y[4] = {0.0f, 0.0f, 0.0f, 0.0f};
          if (g < a.G) {
            if (!a.q_vec) {
#pragma unroll
              for (int e = 0; e < 4; ++e) y[e] = load_any(a.q.p, qh + d + e, a.q_dtype);
            } else if (a.q_dtype == FC_DTYPE_F32) {
              load_vec<float, 4>(static_cast<const float*>(a.q.p) + qh + d, y);
            } else {
              load_vec<__nv_bfloat16, 4>(static_cast<const __nv_bfloat16*>(a.q.p) + qh + d, y);
            }
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) x[i][j + e] = y[e];
        }
      if constexpr (C::ES == 1) {
        // a power of two brings the head's largest |q| to [2^14, 2^15)
        float top = 0.0f;
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
#pragma unroll
          for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(x[i][e]));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // (0 and NaN rows, and infinities: any scale will do)
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
      for (int limb = 0; limb < a.q_limbs; ++limb)
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if constexpr (C::ES == 1) w[e] = take_limb_f16(x[i][2 * e], x[i][2 * e + 1]);
            else w[e] = take_limb(x[i][2 * e], x[i][2 * e + 1]);
          }
          qs[((limb * NT + nt) * (D / 32) + i) * 32 + lane] = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
    const char* kh = pv.k + int64_t(head) * pv.stride_head * C::ES;
    const char* vh = pv.v + int64_t(head) * pv.stride_head * C::ES;
    if (a.kn.p && br.count > 0 && end == rt.n && rt.len > 0) {
      // the fused append: the warp with the segment's last tile stores the new
      // token's rows, which no other warp reads
      const int32_t pos = rt.len - 1, pg = page_of(pv, br.slot, pos);
      if (pg >= 0) {
        const int32_t in = pos & ((1 << pv.log2P) - 1);
        const int64_t e = pg * pv.stride_page + int64_t(in) * D;
        const int64_t se = pg * pv.sstride_page + head * pv.sstride_head + in;
        store_token_row<T, D>(a.kn.p, row * a.kn.sb + head * a.kn.sh, a.new_dtype, a.new_vec & 1,
                              reinterpret_cast<T*>(const_cast<char*>(kh)) + e, pv.ks + se, lane);
        store_token_row<T, D>(a.vn.p, row * a.vn.sb + head * a.vn.sh, a.new_dtype, a.new_vec & 2,
                              reinterpret_cast<T*>(const_cast<char*>(vh)) + e, pv.vs + se, lane);
      }
    }
    __syncwarp();  // the query's fragments and the new token's rows are visible

    float acc[C::NQ][4];
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int q = 0; q < C::NQ; ++q) acc[q][0] = acc[q][1] = acc[q][2] = acc[q][3] = 0.0f;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt][0] = m[nt][1] = __int_as_float(0xff800000);
      l[nt][0] = l[nt][1] = 0.0f;
    }
    int ve = 0;                                       // int8: see below
    float v_most = -1.0f, v_mul = 0.0f, svc[U][2];

    uint32_t kr[U][2][KW / CH] = {}, vr[U][4][VW / CH] = {};
    int32_t pg[U][2];                 // pages of the tiles' two halves
    float sk[U][2] = {}, sv[U][2] = {};  // int8: scales of tokens r and r + 8
    bool full;                        // every token of the iteration is seen

    const int32_t Pm = (1 << pv.log2P) - 1;
    // The table ahead of its use: lane j holds the pages of tiles `held` + j
    // (a page of 8 tokens holds half a tile) and of the 32 tiles after them.
    int32_t held = tile, cur[2], nxt[2];
    auto fetch = [&](int32_t i, int32_t (&g)[2]) {
      const int32_t t = rt.start(i + lane);
      const bool in = i + lane < end && t < rt.len;
      g[0] = in ? page_of(pv, br.slot, t) : -1;
      g[1] = pv.log2P > 3 ? g[0] : in && t + 8 < rt.len ? page_of(pv, br.slot, t + 8) : -1;
    };
    fetch(held, cur);
    fetch(held + 32, nxt);
    auto pages_of = [&](int32_t i) {
      if (i - held == 32) {
        held = i;
        cur[0] = nxt[0];
        cur[1] = nxt[1];
        fetch(held + 32, nxt);
      }
      full = true;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        pg[u][0] = __shfl_sync(0xffffffffu, cur[0], i - held + u);
        pg[u][1] = __shfl_sync(0xffffffffu, cur[1], i - held + u);
        const int32_t t = rt.start(i + u);
        full &= pg[u][0] >= 0 && pg[u][1] >= 0 && t + kTile <= rt.len && (t >= rt.lo || t + kTile <= rt.sinks);
      }
    };
    auto load_k = [&](int32_t i, int part) {
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          const int32_t t = rt.start(i + u) + hh * 8 + r;
          const char* p = kh + (pg[u][hh] * pv.stride_page + int64_t(t & Pm) * D) * C::ES + c * KB;
          if (full || (pg[u][hh] >= 0 && rt.sees(t))) {
#pragma unroll
            for (int j = 0; j < KW / CH; j += KB / 4)
              load_words<KB>(&kr[u][hh][j], p + (j * 4 + part * (KW / CH) * 4) * 4);
            if constexpr (C::ES == 1) {
              const int64_t se = pg[u][hh] * pv.sstride_page + head * pv.sstride_head + (t & Pm);
              load_words<4>(reinterpret_cast<uint32_t*>(&sk[u][hh]), pv.ks + se);
              load_words<4>(reinterpret_cast<uint32_t*>(&sv[u][hh]), pv.vs + se);
            }
          } else if constexpr (C::ES == 1) {
            sv[u][hh] = 0.0f;  // (a masked K row may hold anything: its score is replaced)
          }
        }
    };
    auto load_v = [&](int32_t i, int part) {
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int32_t g = pg[u][k >> 1], t = rt.start(i + u) + (k >> 1) * 8 + 2 * c + (k & 1);
          const char* p = vh + (g * pv.stride_page + int64_t(t & Pm) * D) * C::ES + r * VB;
          if (full || (g >= 0 && rt.sees(t))) {
#pragma unroll
            for (int j = 0; j < VW / CH; j += VB / 4)
              load_words<VB>(&vr[u][k][j], p + (j * 8 + part * (VW / CH) * 8) * 4);
          } else {
#pragma unroll
            for (int j = 0; j < VW / CH; ++j) vr[u][k][j] = 0;
          }
        }
    };

    pages_of(tile);
    if constexpr (C::kPrefetch) {
      load_k(tile, 0);
      load_v(tile, 0);
    }
    for (int32_t i = tile; i < end; i += U) {
      // ---- S^T = K Q^T
      float s[U][NT][4];
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) s[u][nt][0] = s[u][nt][1] = s[u][nt][2] = s[u][nt][3] = 0.0f;
#pragma unroll
      for (int part = 0; part < CH; ++part) {
        if constexpr (!C::kPrefetch) load_k(i, part);
        constexpr int STEPS = D / 16 / CH;  // k-steps of 16 channels per part
        if constexpr (C::ES == 4) {
#pragma unroll
          for (int ks = 0; ks < STEPS; ++ks)
#pragma unroll
            for (int u = 0; u < U; ++u) {
              float x[2][4];
#pragma unroll
              for (int hh = 0; hh < 2; ++hh)
#pragma unroll
                for (int e = 0; e < 4; ++e) x[hh][e] = __uint_as_float(kr[u][hh][4 * ks + e]);
#pragma unroll
              for (int kl = 0; kl < 3; ++kl) {
                const uint32_t a0 = take_limb(x[0][0], x[0][1]), a2 = take_limb(x[0][2], x[0][3]);
                const uint32_t a1 = take_limb(x[1][0], x[1][1]), a3 = take_limb(x[1][2], x[1][3]);
#pragma unroll
                for (int ql = 0; ql < 3 - kl; ++ql) {
                  if (ql >= a.q_limbs) break;
#pragma unroll
                  for (int nt = 0; nt < NT; ++nt) {
                    const int kk = part * STEPS + ks;
                    const uint2 b = reinterpret_cast<const uint2*>(
                        &qs[((ql * NT + nt) * (D / 32) + kk / 2) * 32 + lane])[kk & 1];
                    mma_bf16(s[u][nt], a0, a1, a2, a3, b.x, b.y);
                  }
                }
              }
            }
        } else {
          // bf16, int8: K is exact in one limb; the limbs of the query
          float odd[U][NT][4] = {};  // a second chain of dependent products
#pragma unroll
          for (int ks = 0; ks < STEPS; ++ks) {
            const int kk = part * STEPS + ks;
            uint32_t k0[U], k1[U], k2[U], k3[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
              if constexpr (C::ES == 2) {
                k0[u] = kr[u][0][2 * ks];
                k1[u] = kr[u][1][2 * ks];
                k2[u] = kr[u][0][2 * ks + 1];
                k3[u] = kr[u][1][2 * ks + 1];
              } else {
                const uint32_t x0 = kr[u][0][ks] ^ 0x80808080u, x1 = kr[u][1][ks] ^ 0x80808080u;
                k0[u] = codes_to_f16(__byte_perm(x0, 0x64646464u, 0x4140));
                k1[u] = codes_to_f16(__byte_perm(x1, 0x64646464u, 0x4140));
                k2[u] = codes_to_f16(__byte_perm(x0, 0x64646464u, 0x4342));
                k3[u] = codes_to_f16(__byte_perm(x1, 0x64646464u, 0x4342));
              }
            }
#pragma unroll
            for (int ql = 0; ql < (C::ES == 1 ? 2 : 3); ++ql) {
              if (ql >= a.q_limbs) break;
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                const uint2 b = reinterpret_cast<const uint2*>(
                    &qs[((ql * NT + nt) * (D / 32) + kk / 2) * 32 + lane])[kk & 1];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                  if (ks & 1) mma<T>(odd[u][nt], k0[u], k1[u], k2[u], k3[u], b.x, b.y);
                  else mma<T>(s[u][nt], k0[u], k1[u], k2[u], k3[u], b.x, b.y);
                }
              }
            }
          }
#pragma unroll
          for (int u = 0; u < U; ++u)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 4; ++e) s[u][nt][e] += odd[u][nt][e];
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
              if constexpr (C::ES == 1) s[u][nt][2 * hh + j] *= sk[u][hh] * qf[nt][j];
              else s[u][nt][2 * hh + j] *= a.scale_log2e;
            }
      if (!full) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            if (pg[u][hh] >= 0 && rt.sees(rt.start(i + u) + hh * 8 + r)) continue;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              s[u][nt][2 * hh] = s[u][nt][2 * hh + 1] = __int_as_float(0xff800000);
          }
      }
      if constexpr (C::ES == 1) {
        // V's scales are multiplied into P as 2^(7 - ve) scale, ve above the
        // exponent of every scale so far, so that fp16 holds them (p <= 2^8)
        float x = 0.0f;
#pragma unroll
        for (int u = 0; u < U; ++u) x = fmaxf(x, fmaxf(sv[u][0], sv[u][1]));
        if (__any_sync(0xffffffffu, x > v_most)) {
          x = warp_max(x);
          int e = exponent_of(x) + 1;
          e = e < -100 ? -100 : e > 120 ? 120 : e;
          const float f = v_most < 0.0f ? 0.0f : pow2i(ve - e < -126 ? -126 : ve - e);
          ve = e;
          v_most = pow2i(e);
          v_mul = pow2i(7 - e);
#pragma unroll
          for (int q = 0; q < C::NQ; ++q)
#pragma unroll
            for (int k = 0; k < 4; ++k) acc[q][k] *= f;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          svc[u][0] = sv[u][0] * v_mul;  // before the prefetch
          svc[u][1] = sv[u][1] * v_mul;
        }
      }
      if constexpr (C::kPrefetch) {
        pages_of(i + U);
        load_k(i + U, 0);
      }

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
          raise |= x > m[nt][j] + kLazy;
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
            const float e = join_factor(m[nt][j], x);
            m[nt][j] = x;
            l[nt][j] *= e;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              acc[nt * MT + mt][j] *= e;
              acc[nt * MT + mt][2 + j] *= e;
            }
          }
      }

      // ---- P, and its limbs as B operands (heads x tokens)
      uint32_t pb[U][3][NT][2];
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            float p[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              // no score yet: the maximum is -infinity and p is to be 0
              const float base = m[nt][j] == __int_as_float(0xff800000) ? 0.0f : m[nt][j];
              p[j] = fast_exp2(s[u][nt][2 * hh + j] - base);
              l[nt][j] += p[j];
              if constexpr (C::ES == 1) p[j] *= svc[u][hh];
            }
#pragma unroll
            for (int k = 0; k < 3; ++k) {
              if constexpr (C::ES == 1) {
                if (k < 2) pb[u][k][nt][hh] = transpose8x8(take_limb_f16(p[0], p[1]));
                continue;
              }
              // the last limb is rounded, the ones before keep eight bits each
              if (k < a.p_limbs - 1) pb[u][k][nt][hh] = transpose8x8(take_limb(p[0], p[1]));
              else if (k < a.p_limbs) pb[u][k][nt][hh] = transpose8x8(pack_bf16(p[0], p[1]));
            }
          }

      // ---- O^T += V^T P^T: the iteration's products in accumulators of their
      // own, added in fp32 (the tensor cores' running sums are truncated)
#pragma unroll
      for (int part = 0; part < CH; ++part) {
        if constexpr (!C::kPrefetch) load_v(i, part);
#pragma unroll
        for (int mt = 0; mt < MT / CH; ++mt) {
          const int q = part * (MT / CH) + mt;
          float o[NT][4] = {};
#pragma unroll
          for (int u = 0; u < U; ++u) {
            if constexpr (C::ES == 4) {
              float x[4][2];
#pragma unroll
              for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int e = 0; e < 2; ++e) x[k][e] = __uint_as_float(vr[u][k][2 * mt + e]);
#pragma unroll
              for (int vl = 0; vl < 3; ++vl) {
                const uint32_t a0 = take_limb(x[0][0], x[1][0]), a1 = take_limb(x[0][1], x[1][1]);
                const uint32_t a2 = take_limb(x[2][0], x[3][0]), a3 = take_limb(x[2][1], x[3][1]);
#pragma unroll
                for (int k = 0; k < 3 - vl; ++k)
                  if (k < a.p_limbs) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                      mma_bf16(o[nt], a0, a1, a2, a3, pb[u][k][nt][0], pb[u][k][nt][1]);
                  }
              }
            } else {
              uint32_t a0, a1, a2, a3;
              if constexpr (C::ES == 2) {
                a0 = __byte_perm(vr[u][0][mt], vr[u][1][mt], 0x5410);
                a1 = __byte_perm(vr[u][0][mt], vr[u][1][mt], 0x7632);
                a2 = __byte_perm(vr[u][2][mt], vr[u][3][mt], 0x5410);
                a3 = __byte_perm(vr[u][2][mt], vr[u][3][mt], 0x7632);
              } else {
                // codes 2 mt and 2 mt + 1 of each token: bytes of word mt / 2
                const uint32_t lo = mt & 1 ? 0x0602u : 0x0400u, hi = mt & 1 ? 0x0703u : 0x0501u;
                auto pair = [](uint32_t w0, uint32_t w1, uint32_t sel) {
                  return codes_to_f16((__byte_perm(w0, w1, sel) & 0x00ff00ffu) ^ 0x64806480u);
                };
                a0 = pair(vr[u][0][mt / 2], vr[u][1][mt / 2], lo);
                a1 = pair(vr[u][0][mt / 2], vr[u][1][mt / 2], hi);
                a2 = pair(vr[u][2][mt / 2], vr[u][3][mt / 2], lo);
                a3 = pair(vr[u][2][mt / 2], vr[u][3][mt / 2], hi);
              }
              constexpr int kMost = C::ES == 1 ? 2 : 3;
#pragma unroll
              for (int k = 0; k < kMost; ++k)
                if (C::ES == 1 || k < a.p_limbs) {
#pragma unroll
                  for (int nt = 0; nt < NT; ++nt)
                    mma<T>(o[nt], a0, a1, a2, a3, pb[u][k][nt][0], pb[u][k][nt][1]);
                }
            }
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[nt * MT + q][e] += o[nt][e];
        }
      }
      if constexpr (C::kPrefetch) load_v(i + U, 0);
      else pages_of(i + U);
    }

    // ---- the segment's sums over the lanes' tokens; whole segments are done
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) l[nt][j] += __shfl_xor_sync(0xffffffffu, l[nt][j], o);
    if constexpr (C::ES == 1) {
      const float f = v_most < 0.0f ? 0.0f : pow2i(ve - 7);
#pragma unroll
      for (int q = 0; q < C::NQ; ++q)
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[q][k] *= f;
    }
    const bool whole = tile == 0 && end == rt.n;
    char* frag = fragments + (warp * 2 + made) * C::kFragment;
#pragma unroll
    for (int q = 0; q < C::NQ; ++q) {
      if (whole) store_quad<C, T>(a, row, head, q, lane, acc[q], l[q / MT]);
      else store_fragment<C>(frag, q, lane, acc[q], m[q / MT], l[q / MT]);
    }
    if (whole) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) store_lse(a, row, head, nt, lane, m[nt], l[nt]);
    } else {
      if (lane == 0) pieces[warp * 2 + made] = Piece{row, head, tile, end, rt.n};
      ++made;
    }
    at += end - tile;
    tile = 0;
    if (++head == H) head = 0, ++row;
  }
  if (lane == 0) n_pieces[warp] = made;
  __syncthreads();

  // ---- join the CTA's fragments, segment by segment, in order
  int open = 0;                       // segments left to other CTAs as well
  int32_t seg_row[2], seg_head[2], seg_n[2];
  int64_t first_pos[2];               // line position of the segment's tile 0
  {
    // line position of the fragments: walk the CTA's range
    int w = 0, k = 0;
    while (w < C::WARPS) {
      if (k >= n_pieces[w]) {
        ++w;
        k = 0;
        continue;
      }
      const Piece first = pieces[w * 2 + k];
      int ids[C::WARPS], n = 0;
      int32_t upto = first.from;
      // consecutive fragments of one segment: at most one per warp
      while (w < C::WARPS) {
        if (k >= n_pieces[w]) {
          ++w;
          k = 0;
          continue;
        }
        const Piece p = pieces[w * 2 + k];
        if (p.row != first.row || p.head != first.head) break;
        ids[n++] = w * 2 + k;
        upto = p.to;
        ++k;
      }
      const bool whole = first.from == 0 && upto == first.n;
      char* to_ws = a.partials + (int64_t(blockIdx.x) * 2 + (first.from > 0 ? 0 : 1)) * C::kFragment;
      for (int q = warp; q < C::NQ; q += C::WARPS) {
        float o[4], mm[2], ll[2];
        join<C>(n, [&](int i) { return fragments + ids[i] * C::kFragment; }, q, lane, o, mm, ll);
        if (whole) {
          store_quad<C, T>(a, first.row, first.head, q, lane, o, ll);
          if (q % MT == 0) store_lse(a, first.row, first.head, q / MT, lane, mm, ll);
        } else {
          store_fragment<C>(to_ws, q, lane, o, mm, ll);
        }
      }
      if (!whole) {
        const int j = open++ & 1;
        seg_row[j] = first.row;
        seg_head[j] = first.head;
        seg_n[j] = first.n;
        // a segment that began before this CTA starts `from` tiles before its
        // range; one that runs past its end begins upto - from tiles before it
        first_pos[j] = first.from > 0 ? cta_from - first.from : cta_to - upto;
      }
    }
  }
  if (open == 0) return;

  // ---- the last CTA of a segment joins the CTAs' fragments
  __threadfence();
  __syncthreads();
  for (int j = 0; j < open; ++j) {
    // the CTA of position p is the largest c with total c / ctas <= p
    const int64_t p0 = first_pos[j], p1 = p0 + seg_n[j] - 1;
    const int32_t c0 = int32_t(((p0 + 1) * ctas - 1) / total), c1 = int32_t(((p1 + 1) * ctas - 1) / total);
    if (threadIdx.x == 0) {
      const uint32_t n = atomicAdd(&a.tickets[c0], 1u);
      last_of[j] = n == uint32_t(c1 - c0);
      if (last_of[j]) a.tickets[c0] = 0;
    }
    __syncthreads();
    if (!last_of[j]) continue;
    __threadfence();
    for (int q = warp; q < C::NQ; q += C::WARPS) {
      float o[4], mm[2], ll[2];
      join<C>(c1 - c0 + 1,
              [&](int i) { return a.partials + (int64_t(c0 + i) * 2 + (i == 0 ? 1 : 0)) * C::kFragment; }, q,
              lane, o, mm, ll);
      store_quad<C, T>(a, seg_row[j], seg_head[j], q, lane, o, ll);
      if (q % MT == 0) store_lse(a, seg_row[j], seg_head[j], q / MT, lane, mm, ll);
    }
  }
}

template <typename T, int D, int NT>
int launch_paged(const PagedArgs& a, cudaStream_t s) {
  using C = PagedCfg<T, D, NT>;
  const size_t smem = C::WARPS * (2 * C::kFragment + C::q_bytes(a.q_limbs));
  auto* kernel = paged_attention_kernel<T, D, NT>;
  // once per device: the attribute allows the largest form (three limbs)
  static std::atomic<bool> set[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return FC_ERR_CUDA;
  if (!set[dev]) {
    const size_t most = C::WARPS * (2 * C::kFragment + C::q_bytes(3));
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(most)) != cudaSuccess)
      return FC_ERR_CUDA;
    set[dev] = true;
  }
  const unsigned grid = unsigned(sm_count() * kPagedCtasPerSm);
  kernel<<<grid, C::WARPS * 32, smem, s>>>(a);
  return cuda_status(cudaGetLastError());
}

template <typename T>
int launch_paged_dtype(const PagedArgs& a, int64_t D, cudaStream_t s) {
  const bool two = a.G > 8;
  switch (D) {
    case 32:
      return two ? launch_paged<T, 32, 2>(a, s) : launch_paged<T, 32, 1>(a, s);
    case 64:
      return two ? launch_paged<T, 64, 2>(a, s) : launch_paged<T, 64, 1>(a, s);
    case 128:
      return two ? launch_paged<T, 128, 2>(a, s) : launch_paged<T, 128, 1>(a, s);
    case 256:
      return two ? launch_paged<T, 256, 2>(a, s) : launch_paged<T, 256, 1>(a, s);
  }
  return FC_ERR_UNSUPPORTED;
}

#endif  // __CUDACC__

}  // namespace fc
