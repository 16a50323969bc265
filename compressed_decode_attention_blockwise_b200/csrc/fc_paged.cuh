// Internal helpers of the paged cache's translation units (not part of the ABI).
#pragma once

#include "fc_internal.cuh"
#include "fc_paged.h"

namespace fc {

// Host validation of a paged cache's descriptor (storage, map pointers).
int check_pages(const fc_pages* p);
// FC_ERR_INVALID while `stream` is being captured (bookkeeping is a host
// decision that a replay could not repeat).
int check_not_capturing(fc_stream stream);

inline bool paged_group_ok(int64_t Hq, int64_t H) {
  if (H < 1 || Hq < 1 || Hq % H) return false;
  const int64_t g = Hq / H;
  return g == 1 || g == 2 || g == 4 || g == 8 || g == 16;
}
inline bool paged_dim_ok(int64_t D) { return D == 32 || D == 64 || D == 128 || D == 256; }

// One row of the open batch as the kernels read it.
struct BatchRow {
  int32_t slot, len, first, count;
};

// Where one layer's pages are, by value for the kernels (strides in elements).
struct PageView {
  char* k;
  char* v;
  float* ks;
  float* vs;
  int64_t stride_page, stride_head, sstride_page, sstride_head;
  const int32_t* table;
  const BatchRow* batch;
  int32_t max_pages, n_pages, n_slots, n_rows, log2P, H;
};
PageView page_view(const fc_pages* p, int64_t layer);

// A bf16 or fp32 input of (B, H, M, D) with element strides.
struct TokenView {
  const void* p;
  int64_t sb, sh, sm;
};

// Launches a kernel that may be set up while the kernel before it on the stream
// still runs (a programmatic dependent): its blocks begin with after_previous(),
// which waits until that kernel is complete and its writes are visible, so only
// the launch itself overlaps. A launch of this file saves about a microsecond
// behind another one.
template <typename Arg>
inline int launch_after(void (*kernel)(Arg), dim3 grid, unsigned block, size_t smem, cudaStream_t stream,
                        const Arg& arg) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cuda_status(cudaLaunchKernelEx(&cfg, kernel, arg));
}

// ------------------------------------------------------------------ device

// The first thing every block of a launch_after kernel does: nothing of global
// memory may be touched before it. It then lets the next launch be set up.
__device__ __forceinline__ void after_previous() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// The page that holds position t of a slot, -1 when the map has none (so that
// a stale map masks the token instead of sending a load astray).
__device__ __forceinline__ int32_t page_of(const PageView& a, int32_t slot, int32_t t) {
  const int32_t i = t >> a.log2P;
  if (uint32_t(slot) >= uint32_t(a.n_slots) || uint32_t(i) >= uint32_t(a.max_pages)) return -1;
  const int32_t pg = a.table[int64_t(slot) * a.max_pages + i];
  return uint32_t(pg) < uint32_t(a.n_pages) ? pg : -1;
}

template <int BYTES>
__device__ __forceinline__ void load_words(uint32_t* w, const void* p) {
  // plain (coherent) loads: the fused step reads rows its own warp has stored
  if constexpr (BYTES == 16) {
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "l"(p));
  } else if constexpr (BYTES == 8) {
    asm volatile("ld.global.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "l"(p));
  } else {
    static_assert(BYTES == 4, "load width");
    asm volatile("ld.global.L1::no_allocate.u32 %0, [%1];" : "=r"(w[0]) : "l"(p));
  }
}

// VEC consecutive elements as floats, by vector loads where p is aligned to
// them. Coherent loads here and below: what a kernel reads may have been written
// after its launch, before after_previous() returned.
template <typename T, int VEC>
__device__ __forceinline__ void load_elems(const T* p, float (&out)[VEC]) {
  constexpr int kBytes = VEC * int(sizeof(T)), kStep = kBytes < 16 ? kBytes : 16, kPerWord = 4 / int(sizeof(T));
  if constexpr (kBytes >= 4) {
#pragma unroll
    for (int i = 0; i < kBytes / kStep; ++i) {
      uint32_t w[kStep / 4];
      load_words<kStep>(w, reinterpret_cast<const char*>(p) + i * kStep);
#pragma unroll
      for (int k = 0; k < kStep / 4; ++k) unpack_word<T>(w[k], &out[(i * (kStep / 4) + k) * kPerWord]);
    }
  } else {
    static_assert(kBytes == 2 && VEC == 1, "one bf16");
    unsigned short h;
    asm volatile("ld.global.L1::no_allocate.u16 %0, [%1];" : "=h"(h) : "l"(p));
    out[0] = __uint_as_float(uint32_t(h) << 16);
  }
}
// One element of a runtime dtype.
__device__ __forceinline__ float load_elem(const void* p, int64_t i, int dtype) {
  float x[1];
  if (dtype == FC_DTYPE_F32) load_elems<float, 1>(static_cast<const float*>(p) + i, x);
  else load_elems<__nv_bfloat16, 1>(static_cast<const __nv_bfloat16*>(p) + i, x);
  return x[0];
}

// int8: code = x / (absmax / 127) to nearest, ties to even. y = |x| (127 / absmax)
// in fp32 decides it unless y lies within 2^-12 of a half-integer (its error is
// below 127 * 2^-22); there the exact comparison of 254 |x| with
// (2k + 1) absmax, both exact in fp64 (24 + 8 bits), decides.
__device__ __forceinline__ int quantise_one(float x, float r, float top) {
  const float y = fabsf(x) * r;
  int c = __float2int_rn(y);
  if (fabsf(y - float(c)) > 0.5f - 0.000244140625f) {
    const int k = int(floorf(y));  // the border k + 1/2 is the near one
    const double a = 254.0 * double(fabsf(x)), b = (2.0 * k + 1.0) * double(top);
    c = a > b ? k + 1 : a < b ? k : k + (k & 1);
  }
  c = c > 127 ? 127 : c;
  return x < 0.0f ? -c : c;
}

template <int E>
__device__ __forceinline__ void quantise_row(const float (&x)[E], int8_t* dst, float* scale, int lane) {
  float top = 0.0f;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    top = fmaxf(top, fabsf(x[i]));
    bad |= !(fabsf(x[i]) <= 3.402823466e+38f);
  }
  top = warp_max(top);
  bad = __any_sync(0xffffffffu, bad);
  // 127 / top overflows below 2^-121; such rows take the quotient in fp64
  const bool tiny = top < 1e-36f;
  const float r = bad || top == 0.0f ? 0.0f : __fdiv_rn(127.0f, top);
  int8_t c[E];
#pragma unroll
  for (int i = 0; i < E; ++i) {
    if (bad || top == 0.0f) {
      c[i] = 0;
    } else if (tiny) {
      c[i] = int8_t(__double2int_rn(127.0 * double(x[i]) / double(top)));
    } else {
      c[i] = int8_t(quantise_one(x[i], r, top));
    }
  }
  if constexpr (E == 1) {
    dst[0] = c[0];
  } else if constexpr (E == 2) {
    *reinterpret_cast<char2*>(dst) = make_char2(c[0], c[1]);
  } else {
#pragma unroll
    for (int i = 0; i < E / 4; ++i)
      reinterpret_cast<char4*>(dst)[i] = make_char4(c[4 * i], c[4 * i + 1], c[4 * i + 2], c[4 * i + 3]);
  }
  if (lane == 0) *scale = bad ? __int_as_float(0x7fc00000) : float(double(top) / 127.0);
}

// A lane's share of a token row: elements [lane E, lane E + E) of the bf16 or
// fp32 row at src[elem ..]. vec: the row is aligned for vector loads of it.
template <int E>
__device__ __forceinline__ void load_token_row(const void* src, int64_t elem, int src_dtype, bool vec,
                                               float (&x)[E], int lane) {
  if (vec && src_dtype == FC_DTYPE_BF16) {
    load_elems<__nv_bfloat16, E>(static_cast<const __nv_bfloat16*>(src) + elem + lane * E, x);
  } else if (vec) {
    load_elems<float, E>(static_cast<const float*>(src) + elem + lane * E, x);
  } else {
#pragma unroll
    for (int i = 0; i < E; ++i) x[i] = load_elem(src, elem + lane * E + i, src_dtype);
  }
}

// Stores a lane's share of a token row as the pages hold it (a warp per row).
template <typename T, int E>
__device__ __forceinline__ void store_row(const float (&x)[E], T* dst, float* scale, int lane) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < E; ++i) dst[i] = x[i];
  } else if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int i = 0; i < E; ++i) dst[i] = __float2bfloat16_rn(x[i]);
  } else {
    quantise_row<E>(x, dst, scale, lane);
  }
}

}  // namespace fc
