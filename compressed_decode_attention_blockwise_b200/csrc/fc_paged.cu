// The paged cache's data calls: append, read, and the host side of attention
// and the fused step. Declared in include/fc_paged.h.
#include <climits>
#include <type_traits>

#include "fc_paged_attn.cuh"

namespace fc {
namespace {

constexpr int kAppendThreads = 256;
constexpr int kAhead = 8;  // 16-byte loads in flight per thread of a copy

struct AppendArgs {
  PageView pages;
  TokenView k, v;
  int32_t dtype, vec;
  int64_t M, offered;    // tokens per batch entry of the source, B * M
  int32_t ahead, side;   // tokens per thread and CTA: see the kernels
};

// The page and the row in it of new token n of the open batch (false: none).
// Rows are found by their first token. Empty rows, which a captured launch of
// more rows than the open batch has finds behind the others, hold no first
// token that the search could go by (an earlier batch's, or -1 after a reset).
__device__ __forceinline__ bool locate_token(const PageView& p, int64_t n, int32_t* page, int32_t* in) {
  int lo = 0, hi = p.n_rows;  // the last row in use with first <= n
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    const int4 b = reinterpret_cast<const int4*>(p.batch)[mid];  // slot, length, first, count
    if (b.x >= 0 && b.z <= n) lo = mid;
    else hi = mid;
  }
  const BatchRow b = p.batch[lo];
  if (b.slot < 0 || n < b.first || n >= int64_t(b.first) + b.count) return false;
  const int32_t pos = b.len - b.count + int32_t(n - b.first);
  if (pos < 0) return false;
  *page = page_of(p, b.slot, pos);
  *in = pos & ((1 << p.log2P) - 1);
  return *page >= 0;
}

// Where up to N tokens of a CTA come from (element offsets of head 0) and go
// to (page -1: nowhere), for all its threads. Thread i does token i.
template <int N>
struct Tokens {
  int64_t k[N], v[N];
  int32_t page[N], in[N];
  __device__ __forceinline__ void sources(const AppendArgs& a, int64_t n0, int count) {
    if (int(threadIdx.x) < count) {
      const uint32_t n = uint32_t(n0) + threadIdx.x, M = uint32_t(a.M);  // (offered < 2^31)
      const uint32_t b = n < M ? 0 : n / M, m = n - b * M;
      k[threadIdx.x] = b * a.k.sb + m * a.k.sm;
      v[threadIdx.x] = b * a.v.sb + m * a.v.sm;
    }
    __syncthreads();
  }
  __device__ __forceinline__ void places(const AppendArgs& a, int64_t n0, int count) {
    if (int(threadIdx.x) < count) {
      int32_t g = -1, i = 0;
      if (n0 + threadIdx.x >= a.offered || !locate_token(a.pages, n0 + threadIdx.x, &g, &i)) g = -1;
      page[threadIdx.x] = g;
      in[threadIdx.x] = i;
    }
    __syncthreads();
  }
};

// bf16 and fp32 pages: a pass of 16-byte moves (read + write, HBM-bound). A
// thread keeps one word of one head's K or V row and takes it for `ahead`
// tokens at once, their loads issued before the pages are known; narrow caches
// have `side` tokens side by side in a CTA. 49 K tokens, 8 heads of 128 in bf16:
// 67 us, 6.0 TB/s, 0.91 of the copy rate (80 us when every thread found its
// tokens by division).
template <typename T, int D>
__global__ void __launch_bounds__(kAppendThreads) append_copy_kernel(const __grid_constant__ AppendArgs a) {
  constexpr int V = D * int(sizeof(T)) / 16;  // 16-byte words per row
  __shared__ Tokens<kAppendThreads> at;
  const int H = a.pages.H, words = 2 * H * V, count = a.ahead * a.side;
  const int64_t n0 = int64_t(blockIdx.x) * count;
  after_previous();
  at.sources(a, n0, count);
  const int sub = a.side > 1 ? int(threadIdx.x) / words : 0;
  for (int item = int(threadIdx.x) - sub * words; item < words || item == int(threadIdx.x); item += kAppendThreads) {
    const bool on = item < words && sub < a.side;
    const int row = item / V, w = item % V, kv = row >= H, h = row - kv * H;
    const TokenView& s = kv ? a.v : a.k;
    uint4 x[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int t = u * a.side + sub;
      if (!on || u >= a.ahead || n0 + t >= a.offered) continue;
      const T* p = static_cast<const T*>(s.p) + (kv ? at.v : at.k)[t] + h * s.sh;
      if (a.vec) {
        x[u] = __ldcs(reinterpret_cast<const uint4*>(p) + w);
      } else {
        uint32_t y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if constexpr (sizeof(T) == 4) {
            y[e] = __float_as_uint(p[w * 4 + e]);
          } else {
            const unsigned short* q = reinterpret_cast<const unsigned short*>(p) + w * 8 + 2 * e;
            y[e] = uint32_t(q[0]) | uint32_t(q[1]) << 16;
          }
        }
        x[u] = make_uint4(y[0], y[1], y[2], y[3]);
      }
    }
    if (item < kAppendThreads) at.places(a, n0, count);  // (every thread's first pass)
    T* const d = reinterpret_cast<T*>(kv ? a.pages.v : a.pages.k) + h * a.pages.stride_head;
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int t = u * a.side + sub;
      if (!on || u >= a.ahead || at.page[t] < 0) continue;
      reinterpret_cast<uint4*>(d + at.page[t] * a.pages.stride_page + int64_t(at.in[t]) * D)[w] = x[u];
    }
  }
}

// int8 pages: a warp per row (token, head, K or V), four rows' loads at once;
// see quantise_row. 666 tokens of 8 heads of 128: 9.2 us, latency; 49,152: 327 us,
// 0.93 TB/s, the quantiser's instructions.
template <int D>
__global__ void __launch_bounds__(kAppendThreads) append_i8_kernel(const __grid_constant__ AppendArgs a) {
  constexpr int E = D / 32, W = kAppendThreads / 32, kRows = 4;
  __shared__ Tokens<kAhead> at;
  const int64_t n0 = int64_t(blockIdx.x) * a.ahead;
  const int warp = int(threadIdx.x >> 5), lane = int(threadIdx.x & 31);
  const int H = a.pages.H, rows = a.ahead * 2 * H;
  after_previous();
  at.sources(a, n0, a.ahead);
  for (int base = 0; base < rows; base += kRows * W) {
    float x[kRows][E];
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const int row = base + u * W + warp, tok = row / (2 * H), kv = row / H & 1, h = row % H;
      if (row >= rows || n0 + tok >= a.offered) continue;
      const TokenView& s = kv ? a.v : a.k;
      load_token_row<E>(s.p, (kv ? at.v : at.k)[tok] + h * s.sh, a.dtype, a.vec, x[u], lane);
    }
    if (base == 0) at.places(a, n0, a.ahead);
    // one copy of the quantiser's code: a short launch waits for its code first
#pragma unroll 1
    for (int u = 0; u < kRows; ++u) {
      float y[E];
#pragma unroll
      for (int i = 0; i < E; ++i) {
        y[i] = x[0][i];
#pragma unroll
        for (int k = 1; k < kRows; ++k) x[k - 1][i] = x[k][i];
      }
      const int row = base + u * W + warp, tok = row / (2 * H), kv = row / H & 1, h = row % H;
      if (row >= rows || at.page[tok] < 0) continue;
      int8_t* d = reinterpret_cast<int8_t*>(kv ? a.pages.v : a.pages.k) + at.page[tok] * a.pages.stride_page +
                  h * a.pages.stride_head + int64_t(at.in[tok]) * D;
      float* sc = (kv ? a.pages.vs : a.pages.ks) + at.page[tok] * a.pages.sstride_page +
                  h * a.pages.sstride_head + at.in[tok];
      quantise_row<E>(y, d + lane * E, sc, lane);
    }
  }
}

struct ReadArgs {
  PageView pages;
  void* k;
  void* v;
  int64_t ks_h, ks_t, vs_h, vs_t;
  int32_t slot, len;
};

// Dense rows of one slot, 16-byte loads or stores, AHEAD rows in flight per
// thread; bound by HBM (pages read + rows written). Rows that keep their type
// are moved as they are. 32,768 tokens, 8 heads of 128 in bf16: 40 us, at the copy
// rate; 333 int8 tokens: 5.3 us with one row per thread, 10 with eight; 49,152 int8
// tokens: 107 us, 2.8 TB/s.
template <typename T, typename TO, int D, int AHEAD>
__global__ void __launch_bounds__(256) paged_read_kernel(const __grid_constant__ ReadArgs a) {
  constexpr bool kMove = std::is_same<T, TO>::value;
  constexpr int E = kMove ? 16 / int(sizeof(T)) : 8;  // elements per thread and row
  constexpr int V = D / E, kRows = 256 / V;
  const int group = int(threadIdx.x) / V, w = int(threadIdx.x) % V;
  const int h = int(blockIdx.y) >> 1, kv = int(blockIdx.y) & 1;
  const int32_t t0 = int32_t(blockIdx.x) * (AHEAD * kRows) + group;
  const T* const pool = reinterpret_cast<const T*>(kv ? a.pages.v : a.pages.k) + h * a.pages.stride_head + w * E;
  TO* const out = static_cast<TO*>(kv ? a.v : a.k) + h * (kv ? a.vs_h : a.ks_h) + w * E;
  const int64_t os = kv ? a.vs_t : a.ks_t;
  int32_t page[AHEAD];
  after_previous();
#pragma unroll
  for (int u = 0; u < AHEAD; ++u) {
    const int32_t t = t0 + u * kRows;
    page[u] = t < a.len ? page_of(a.pages, a.slot, t) : -1;
  }
  uint4 x[AHEAD];
  float f[AHEAD][kMove ? 1 : E];
#pragma unroll
  for (int u = 0; u < AHEAD; ++u) {
    if (page[u] < 0) continue;
    const int32_t in = (t0 + u * kRows) & ((1 << a.pages.log2P) - 1);
    const T* p = pool + page[u] * a.pages.stride_page + int64_t(in) * D;
    if constexpr (kMove) {
      x[u] = __ldcs(reinterpret_cast<const uint4*>(p));
    } else {
      load_elems<T, E>(p, f[u]);
      if constexpr (sizeof(T) == 1) {
        const float s = (kv ? a.pages.vs : a.pages.ks)[page[u] * a.pages.sstride_page + h * a.pages.sstride_head + in];
#pragma unroll
        for (int e = 0; e < E; ++e) f[u][e] *= s;
      }
    }
  }
#pragma unroll
  for (int u = 0; u < AHEAD; ++u) {
    if (page[u] < 0) continue;
    TO* o = out + (t0 + u * kRows) * os;
    if constexpr (kMove) {
      __stcs(reinterpret_cast<uint4*>(o), x[u]);
    } else if constexpr (sizeof(TO) == 4) {
      reinterpret_cast<float4*>(o)[0] = make_float4(f[u][0], f[u][1], f[u][2], f[u][3]);
      reinterpret_cast<float4*>(o)[1] = make_float4(f[u][4], f[u][5], f[u][6], f[u][7]);
    } else {
      *reinterpret_cast<uint4*>(o) = make_uint4(pack_bf16(f[u][0], f[u][1]), pack_bf16(f[u][2], f[u][3]),
                                                pack_bf16(f[u][4], f[u][5]), pack_bf16(f[u][6], f[u][7]));
    }
  }
}

// Tokens per thread: eight, two below 32 tokens per SM, one below 8 (a launch of
// few tokens is all latency). Narrow caches, whose CTAs take `side` tokens side
// by side, go by the same numbers: fewer CTAs with more loads in flight are the
// faster ones there (one kv head of 128 in bf16, 4,800 tokens: 3.5 us in 75 CTAs
// of eight tokens per thread, 4.1 in 300 of two; 10,000: 4.2 in 157, 4.8 in 625).
template <int D>
int launch_append(AppendArgs a, int pages_dtype, cudaStream_t s) {
  a.ahead = a.offered < int64_t(sm_count()) * 8 ? 1 : a.offered < int64_t(sm_count()) * 32 ? 2 : kAhead;
  a.side = 1;
  if (pages_dtype != FC_DTYPE_I8) {
    const int words = 2 * a.pages.H * (D * dtype_size(pages_dtype) / 16);
    if (words < kAppendThreads) a.side = kAppendThreads / words;
    if (a.side > kAppendThreads / kAhead) a.side = kAppendThreads / kAhead;
  }
  const int64_t per = int64_t(a.ahead) * a.side;
  const unsigned grid = unsigned((a.offered + per - 1) / per);
  auto* kernel = pages_dtype == FC_DTYPE_I8    ? append_i8_kernel<D>
                 : pages_dtype == FC_DTYPE_F32 ? append_copy_kernel<float, D>
                                               : append_copy_kernel<__nv_bfloat16, D>;
  return launch_after(kernel, dim3(grid), kAppendThreads, 0, s, a);
}

template <typename T, typename TO, int D>
int launch_read_as(const ReadArgs& a, cudaStream_t s) {
  constexpr int E = std::is_same<T, TO>::value ? 16 / int(sizeof(T)) : 8;
  constexpr unsigned kRows = 256 / (D / E);  // rows of a CTA in one pass
  const unsigned heads = unsigned(a.pages.H) * 2, len = unsigned(a.len);
  // eight rows per thread, or one while the CTAs of eight would not fill the GPU
  if (int64_t(len) * heads < int64_t(sm_count()) * 2 * kAhead * kRows)
    return launch_after(paged_read_kernel<T, TO, D, 1>, dim3((len + kRows - 1) / kRows, heads), 256, 0, s, a);
  constexpr unsigned kTile = kAhead * kRows;
  return launch_after(paged_read_kernel<T, TO, D, kAhead>, dim3((len + kTile - 1) / kTile, heads), 256, 0, s, a);
}
template <typename T, int D>
int launch_read(const ReadArgs& a, int out_dtype, cudaStream_t s) {
  return out_dtype == FC_DTYPE_F32 ? launch_read_as<T, float, D>(a, s) : launch_read_as<T, __nv_bfloat16, D>(a, s);
}

template <int D>
int launch_read_dtype(const ReadArgs& a, int dtype, int out_dtype, cudaStream_t s) {
  if (dtype == FC_DTYPE_I8) return launch_read<int8_t, D>(a, out_dtype, s);
  if (dtype == FC_DTYPE_F32) return launch_read<float, D>(a, out_dtype, s);
  return launch_read<__nv_bfloat16, D>(a, out_dtype, s);
}

bool float_dtype(int32_t dt) { return dt == FC_DTYPE_F32 || dt == FC_DTYPE_BF16; }

// Aligned for accesses of `bytes`: base and every stride (elements of size es).
bool aligned_for(const void* p, const int64_t* st, int n, int64_t es, int64_t bytes) {
  if (reinterpret_cast<uintptr_t>(p) % uintptr_t(bytes)) return false;
  for (int i = 0; i < n; ++i)
    if (st[i] * es % bytes) return false;
  return true;
}

int check_layer(const fc_pages* p, int64_t layer) {
  const int st = check_pages(p);
  if (st != FC_OK) return st;
  return layer < 0 || layer >= p->n_layers ? FC_ERR_INVALID : FC_OK;
}

// Tokens written to pages of p: their dtype is the pages', or any for int8.
bool token_dtype_ok(const fc_pages* p, int32_t dtype) {
  return float_dtype(dtype) && (p->dtype == FC_DTYPE_I8 || p->dtype == dtype);
}

struct PagedWorkspace {
  size_t tickets, partials, total;
};
PagedWorkspace paged_workspace(int64_t D, int64_t G) {
  const size_t ctas = size_t(sm_count()) * kPagedCtasPerSm;
  PagedWorkspace w;
  w.tickets = 0;
  w.partials = pad256(ctas * 4);
  w.total = w.partials + 2 * ctas * paged_fragment_bytes(D, G);
  return w;
}

int attention(const fc_pages* p, int64_t layer, const void* q, int32_t q_dtype, const int64_t* q_strides,
              int64_t Hq, bool step, const void* k_new, const void* v_new, int32_t new_dtype,
              const int64_t* k_strides, const int64_t* v_strides, float softmax_scale, int64_t window,
              int64_t sinks, void* workspace, size_t workspace_bytes, void* out, int32_t out_dtype,
              const int64_t* out_strides, float* lse, fc_stream stream) {
  const int st = check_layer(p, layer);
  if (st != FC_OK) return st;
  if (!q || !q_strides || !out || !out_strides || !workspace) return FC_ERR_INVALID;
  if (!float_dtype(q_dtype) || !float_dtype(out_dtype)) return FC_ERR_INVALID;
  if (q_strides[3] != 1 || out_strides[3] != 1 || window < 0 || sinks < 0) return FC_ERR_INVALID;
  if (softmax_scale != softmax_scale || Hq < 1 || Hq % p->H) return FC_ERR_INVALID;
  if (!paged_group_ok(Hq, p->H)) return FC_ERR_UNSUPPORTED;
  if (p->n_rows < 1 || p->n_rows > p->n_slots) return FC_ERR_INVALID;
  const int64_t q_es = dtype_size(q_dtype), o_es = dtype_size(out_dtype);
  if (reinterpret_cast<uintptr_t>(q) % uintptr_t(q_es) || reinterpret_cast<uintptr_t>(out) % uintptr_t(o_es) ||
      reinterpret_cast<uintptr_t>(lse) % 4 || reinterpret_cast<uintptr_t>(workspace) % 256)
    return FC_ERR_INVALID;
  const int64_t G = Hq / p->H;
  const PagedWorkspace ws = paged_workspace(p->D, G);
  if (workspace_bytes < ws.total) return FC_ERR_INVALID;
  PagedArgs a{};
  if (step) {
    if (!k_new || !v_new || !k_strides || !v_strides || !token_dtype_ok(p, new_dtype)) return FC_ERR_INVALID;
    if (k_strides[3] != 1 || v_strides[3] != 1 || !p->one_each) return FC_ERR_INVALID;
    const int64_t es = dtype_size(new_dtype), bytes = es * p->D / 32 > 16 ? 16 : es * p->D / 32;
    if (reinterpret_cast<uintptr_t>(k_new) % uintptr_t(es) || reinterpret_cast<uintptr_t>(v_new) % uintptr_t(es))
      return FC_ERR_INVALID;
    a.kn = TokenView{k_new, k_strides[0], k_strides[1], 0};
    a.vn = TokenView{v_new, v_strides[0], v_strides[1], 0};
    a.new_dtype = new_dtype;
    a.new_vec = (aligned_for(k_new, k_strides, 2, es, bytes) ? 1 : 0) |
                (aligned_for(v_new, v_strides, 2, es, bytes) ? 2 : 0);
  }
  a.pages = page_view(p, layer);
  a.q = TokenView{q, q_strides[0], q_strides[1], 0};
  a.q_dtype = q_dtype;
  a.q_vec = (aligned_for(q, q_strides, 2, q_es, 4 * q_es) ? 1 : 0) | (aligned_for(q, q_strides, 2, q_es, 16) ? 2 : 0);
  a.out_vec = aligned_for(out, out_strides, 2, o_es, 2 * o_es) ? 1 : 0;
  a.G = int32_t(G);
  const double sigma = softmax_scale > 0.0f ? double(softmax_scale) : 1.0 / sqrt(double(p->D));
  a.scale_log2e = float(sigma * 1.4426950408889634);
  a.window = int32_t(window < INT_MAX ? window : INT_MAX);
  a.sinks = int32_t(sinks < INT_MAX - kTile ? sinks : INT_MAX - kTile);
  a.out = out;
  a.os_b = out_strides[0];
  a.os_h = out_strides[1];
  a.out_dtype = out_dtype;
  a.lse = lse;
  a.tickets = reinterpret_cast<uint32_t*>(static_cast<char*>(workspace) + ws.tickets);
  a.partials = static_cast<char*>(workspace) + ws.partials;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  // limbs of (query, P): as many as the query's and the output's type need
  const bool fine_q = q_dtype == FC_DTYPE_F32, fine_out = out_dtype == FC_DTYPE_F32;
  if (p->dtype == FC_DTYPE_F32) return launch_paged_attention_f32_33(a, p->D, s);
  if (p->dtype == FC_DTYPE_I8)
    return fine_q ? launch_paged_attention_i8_22(a, p->D, s) : launch_paged_attention_i8_12(a, p->D, s);
  if (fine_q) return launch_paged_attention_bf16_33(a, p->D, s);
  return fine_out ? launch_paged_attention_bf16_13(a, p->D, s) : launch_paged_attention_bf16_12(a, p->D, s);
}

}  // namespace
}  // namespace fc

using namespace fc;

extern "C" int fc_paged_append(const fc_pages* p, int64_t layer, const void* k, const void* v, int32_t dtype,
                               const int64_t* k_strides, const int64_t* v_strides, int64_t B, int64_t M,
                               fc_stream stream) {
  const int st = check_layer(p, layer);
  if (st != FC_OK) return st;
  if (p->n_rows < 1 || p->n_rows > p->n_slots || B < 0 || M < 0 || !token_dtype_ok(p, dtype))
    return FC_ERR_INVALID;
  if ((M > 0 && B > INT_MAX / M) || B * M < p->n_tokens) return FC_ERR_INVALID;
  // nothing to write; a captured launch is there for later batches
  if (B * M == 0 || (p->n_tokens == 0 && check_not_capturing(stream) == FC_OK)) return FC_OK;
  if (!k || !v || !k_strides || !v_strides || k_strides[3] != 1 || v_strides[3] != 1) return FC_ERR_INVALID;
  const int64_t es = dtype_size(dtype);
  if (reinterpret_cast<uintptr_t>(k) % uintptr_t(es) || reinterpret_cast<uintptr_t>(v) % uintptr_t(es))
    return FC_ERR_INVALID;
  AppendArgs a{};
  a.pages = page_view(p, layer);
  a.k = TokenView{k, k_strides[0], k_strides[1], k_strides[2]};
  a.v = TokenView{v, v_strides[0], v_strides[1], v_strides[2]};
  a.dtype = dtype;
  a.vec = aligned_for(k, k_strides, 3, es, 16) && aligned_for(v, v_strides, 3, es, 16) ? 1 : 0;
  a.M = M;
  a.offered = B * M;
  // the grid covers every offered token, so that a captured launch serves any
  // later batch of as many
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  switch (p->D) {
    case 32:
      return launch_append<32>(a, p->dtype, s);
    case 64:
      return launch_append<64>(a, p->dtype, s);
    case 128:
      return launch_append<128>(a, p->dtype, s);
    default:
      return launch_append<256>(a, p->dtype, s);
  }
}

extern "C" size_t fc_paged_workspace_bytes(int64_t Hq, int64_t H, int64_t D) {
  if (!paged_group_ok(Hq, H) || !paged_dim_ok(D)) return 0;
  return paged_workspace(D, Hq / H).total;
}

extern "C" uint64_t fc_paged_capture_id(fc_stream stream) {
  cudaStreamCaptureStatus c = cudaStreamCaptureStatusNone;
  unsigned long long id = 0;
  if (cudaStreamGetCaptureInfo(static_cast<cudaStream_t>(stream), &c, &id) != cudaSuccess) {
    (void)cudaGetLastError();  // no device: nothing can be capturing
    return 0;
  }
  return c == cudaStreamCaptureStatusNone ? 0 : uint64_t(id) + 1;
}

extern "C" int fc_paged_attention(const fc_pages* p, int64_t layer, const void* q, int32_t q_dtype,
                                  const int64_t* q_strides, int64_t Hq, float softmax_scale, int64_t window,
                                  int64_t sinks, void* workspace, size_t workspace_bytes, void* out,
                                  int32_t out_dtype, const int64_t* out_strides, float* lse,
                                  fc_stream stream) {
  return attention(p, layer, q, q_dtype, q_strides, Hq, false, nullptr, nullptr, 0, nullptr, nullptr,
                   softmax_scale, window, sinks, workspace, workspace_bytes, out, out_dtype, out_strides, lse,
                   stream);
}

extern "C" int fc_paged_step(const fc_pages* p, int64_t layer, const void* q, int32_t q_dtype,
                             const int64_t* q_strides, int64_t Hq, const void* k_new, const void* v_new,
                             int32_t new_dtype, const int64_t* k_strides, const int64_t* v_strides,
                             float softmax_scale, int64_t window, int64_t sinks, void* workspace,
                             size_t workspace_bytes, void* out, int32_t out_dtype, const int64_t* out_strides,
                             float* lse, fc_stream stream) {
  return attention(p, layer, q, q_dtype, q_strides, Hq, true, k_new, v_new, new_dtype, k_strides, v_strides,
                   softmax_scale, window, sinks, workspace, workspace_bytes, out, out_dtype, out_strides, lse,
                   stream);
}

extern "C" int fc_paged_read(const fc_pages* p, int64_t layer, int64_t slot, void* k_out, void* v_out,
                             int32_t out_dtype, const int64_t* k_strides, const int64_t* v_strides, int64_t T,
                             fc_stream stream) {
  const int st = check_layer(p, layer);
  if (st != FC_OK) return st;
  if (slot < 0 || slot >= p->n_slots || !float_dtype(out_dtype)) return FC_ERR_INVALID;
  const int32_t len = p->h_lens[slot];
  if (T < len) return FC_ERR_INVALID;
  if (len == 0) return FC_OK;
  if (!k_out || !v_out || !k_strides || !v_strides || k_strides[3] != 1 || v_strides[3] != 1)
    return FC_ERR_INVALID;
  const int64_t es = dtype_size(out_dtype);
  if (!aligned_for(k_out, k_strides, 3, es, 16) || !aligned_for(v_out, v_strides, 3, es, 16))
    return FC_ERR_INVALID;
  if (p->H > 32767) return FC_ERR_UNSUPPORTED;
  ReadArgs a{};
  a.pages = page_view(p, layer);
  a.k = k_out;
  a.v = v_out;
  a.ks_h = k_strides[1];
  a.ks_t = k_strides[2];
  a.vs_h = v_strides[1];
  a.vs_t = v_strides[2];
  a.slot = int32_t(slot);
  a.len = len;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  switch (p->D) {
    case 32:
      return launch_read_dtype<32>(a, p->dtype, out_dtype, s);
    case 64:
      return launch_read_dtype<64>(a, p->dtype, out_dtype, s);
    case 128:
      return launch_read_dtype<128>(a, p->dtype, out_dtype, s);
    default:
      return launch_read_dtype<256>(a, p->dtype, out_dtype, s);
  }
}
