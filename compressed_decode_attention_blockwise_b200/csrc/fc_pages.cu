// Bookkeeping of the paged cache: which pages a sequence has, taking, sharing,
// copying, packing and freeing them. Declared in include/fc_paged.h.
//
// The decisions are host integers (lowest free page first, reference counts),
// made on the caller's arrays and taken back if the call fails. What the
// device needs of them travels as kernel parameters: no staging buffer, no
// copy call, nothing that the host could change before the GPU has read it.
// Page copies are one pass over the moved pages of all layers, a warp per
// 4 KB piece of one head's run, so they are bound by HBM (read + write).
#include <memory>
#include <new>
#include <utility>
#include <vector>

#include "fc_paged.cuh"

namespace fc {
namespace {

// ------------------------------------------------------------- edit records

enum RecOp : int32_t {
  kRow,    // batch[a] = {b, c, d, e}; lens[b] = c when b >= 0
  kRun,    // table[a][b + i] = c + i, i < d
  kCrop,   // lens[a] = b; table[a][c + i] = -1, i < d
  kFork    // table[b][i] = table[a][i], i < c; lens[b] = d
};
struct Rec {
  int32_t op, a, b, c, d, e;
};

struct MapView {
  int32_t* table;
  int32_t* lens;
  int32_t* batch;
  int64_t max_pages;
};

// Two parameter sizes: a step's edits fit the small one; a long prompt's need
// fewer launches with the large one (28 KB of the 32 KB a launch may carry).
constexpr int kFewRecs = 160, kManyRecs = 1200;
template <int N>
struct Recs {
  MapView m;
  int32_t n;
  Rec r[N];
};

// One warp per record. Records of one call never touch the same entry.
__device__ __forceinline__ void apply_record(const MapView& m, const Rec& r) {
  const int lane = int(threadIdx.x & 31);
  switch (r.op) {
    case kRow:
      if (lane == 0) {
        reinterpret_cast<int4*>(m.batch)[r.a] = make_int4(r.b, r.c, r.d, r.e);
        if (r.b >= 0) m.lens[r.b] = r.c;
      }
      break;
    case kRun:
      for (int j = lane; j < r.d; j += 32) m.table[int64_t(r.a) * m.max_pages + r.b + j] = r.c + j;
      break;
    case kCrop:
      for (int j = lane; j < r.d; j += 32) m.table[int64_t(r.a) * m.max_pages + r.c + j] = -1;
      if (lane == 0) m.lens[r.a] = r.b;
      break;
    case kFork:
      for (int j = lane; j < r.c; j += 32)
        m.table[int64_t(r.b) * m.max_pages + j] = m.table[int64_t(r.a) * m.max_pages + j];
      if (lane == 0) m.lens[r.b] = r.d;
      break;
  }
}

template <int N>
__global__ void __launch_bounds__(256) edit_map_kernel(const __grid_constant__ Recs<N> p) {
  const int i = int(blockIdx.x) * 8 + int(threadIdx.x >> 5);
  after_previous();
  if (i < p.n) apply_record(p.m, p.r[i]);
}

template <int N>
int launch_recs(const MapView& m, const Rec* r, int n, cudaStream_t s) {
  Recs<N> a;
  a.m = m;
  a.n = n;
  for (int i = 0; i < n; ++i) a.r[i] = r[i];
  return launch_after(edit_map_kernel<N>, dim3(unsigned((n + 7) / 8)), 256, 0, s, a);
}

int launch_edits(const fc_pages* p, const std::vector<Rec>& recs, cudaStream_t s) {
  const MapView m{p->table, p->lens, p->batch, p->max_pages};
  for (size_t at = 0; at < recs.size();) {
    const size_t left = recs.size() - at;
    const int n = int(left > size_t(kManyRecs) ? size_t(kManyRecs) : left);
    const int st = n <= kFewRecs ? launch_recs<kFewRecs>(m, &recs[at], n, s)
                                 : launch_recs<kManyRecs>(m, &recs[at], n, s);
    if (st != FC_OK) return st;
    at += size_t(n);
  }
  return FC_OK;
}

// -------------------------------------------------------------- page copies

struct Pair {
  int32_t src, dst;
};
constexpr int kFewPairs = 440, kManyPairs = 3500;

struct CopyShape {
  char* base[4];  // k, v, k_scales, v_scales (null scales: two parts only)
  int64_t layer[2], page[2], head[2];  // byte strides of the rows / the scales
  int64_t run[2];                      // bytes of one head's rows / scales
  uint32_t n_layers, H, pieces;        // pieces: 4 KB parts of a head's rows
  uint32_t row_units, all_units;       // warps' units: rows of k and v, then scales
  int32_t* table;                      // remapped when not null
  int64_t table_entries;
  int32_t first_moved;                 // entries below it stay
  unsigned copy_blocks;
};
template <int N, int NR>
struct Pairs {
  CopyShape s;
  int32_t n, n_recs;
  Pair p[N];  // ascending in src where a table is remapped
  MapView m;
  Rec r[NR > 0 ? NR : 1];
};

constexpr int kPieceBytes = 4096;

// A warp per unit: (pair, layer, k or v, head, 4 KB piece), all its loads in
// flight before the first store. Sources and destinations are disjoint pages.
// 255 MB moved (compaction, 4 layers of 8 heads of 128): 75 us, 6.8 TB/s.
// The blocks past copy_blocks see to the map: they apply the NR records that
// came along (a step's copies and edits in one launch), or rewrite the table,
// where an entry that names a moved page gets the page's new place (binary
// search in the pairs).
template <int N, int NR>
__global__ void __launch_bounds__(256) copy_pages_kernel(const __grid_constant__ Pairs<N, NR> a) {
  const CopyShape& s = a.s;
  after_previous();
  const int lane = int(threadIdx.x & 31);
  if (NR > 0 && blockIdx.x >= s.copy_blocks) {
    const int i = int(blockIdx.x - s.copy_blocks) * 8 + int(threadIdx.x >> 5);
    if (i < a.n_recs) apply_record(a.m, a.r[i]);
    return;
  }
  if (blockIdx.x >= s.copy_blocks) {
    __shared__ Pair sp[NR > 0 ? 1 : N];
    for (int i = int(threadIdx.x); i < a.n; i += 256) sp[i] = a.p[i];
    __syncthreads();
    const int64_t step = int64_t(gridDim.x - s.copy_blocks) * 256;
    for (int64_t i = int64_t(blockIdx.x - s.copy_blocks) * 256 + threadIdx.x; i < s.table_entries; i += step) {
      const int32_t e = s.table[i];
      if (e < s.first_moved) continue;
      int lo = 0, hi = a.n;
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (sp[mid].src < e) lo = mid + 1;
        else hi = mid;
      }
      if (lo < a.n && sp[lo].src == e) s.table[i] = sp[lo].dst;
    }
    return;
  }
  const uint32_t warps = s.copy_blocks * 8;
  for (uint32_t u = blockIdx.x * 8 + (threadIdx.x >> 5); u < s.all_units; u += warps) {
    const bool scale = u >= s.row_units;
    uint32_t i = scale ? u - s.row_units : u;
    const uint32_t pieces = scale ? 1 : s.pieces;
    const int64_t piece = i % pieces;
    i /= pieces;
    const int64_t h = i % s.H;
    i /= s.H;
    const int kv = int(i & 1);
    i >>= 1;
    const int64_t layer = i % s.n_layers;
    const Pair pr = a.p[i / s.n_layers];
    char* b = s.base[(scale ? 2 : 0) + kv] + layer * s.layer[scale] + h * s.head[scale] + piece * kPieceBytes;
    const char* from = b + pr.src * s.page[scale];
    char* to = b + pr.dst * s.page[scale];
    int64_t bytes = s.run[scale] - piece * kPieceBytes;
    if (bytes > kPieceBytes) bytes = kPieceBytes;
    uint4 w[kPieceBytes / 512];
#pragma unroll
    for (int j = 0; j < kPieceBytes / 512; ++j)
      if (j * 512 + lane * 16 < bytes) w[j] = __ldcs(reinterpret_cast<const uint4*>(from + j * 512 + lane * 16));
#pragma unroll
    for (int j = 0; j < kPieceBytes / 512; ++j)
      if (j * 512 + lane * 16 < bytes) __stcs(reinterpret_cast<uint4*>(to + j * 512 + lane * 16), w[j]);
  }
}

template <int N, int NR>
int launch_pairs(const CopyShape& shape, const Pair* pr, int n, const MapView& m, const std::vector<Rec>* recs,
                 cudaStream_t stream) {
  Pairs<N, NR> a;
  a.s = shape;
  a.n = n;
  a.n_recs = 0;
  if (NR > 0) {
    a.m = m;
    a.n_recs = int32_t(recs->size());
    for (int i = 0; i < a.n_recs; ++i) a.r[i] = (*recs)[size_t(i)];
  }
  for (int i = 0; i < n; ++i) a.p[i] = pr[i];
  a.s.row_units = uint32_t(n) * shape.n_layers * 2 * shape.H * shape.pieces;
  a.s.all_units = a.s.row_units + (shape.base[2] ? uint32_t(n) * shape.n_layers * 2 * shape.H : 0);
  const int64_t most = int64_t(sm_count()) * 8;  // eight CTAs of eight warps per SM
  int64_t blocks = (int64_t(a.s.all_units) + 7) / 8;
  if (blocks > most) blocks = most;
  a.s.copy_blocks = unsigned(blocks);
  blocks += (a.n_recs + 7) / 8;
  if (shape.table) {
    int64_t t = (shape.table_entries + 1023) / 1024;
    blocks += t > 64 ? 64 : t;
    a.s.first_moved = pr[0].src;
  }
  return launch_after(copy_pages_kernel<N, NR>, dim3(unsigned(blocks)), 256, 0, stream, a);
}

// Copies the pairs' pages; remap: rewrites the table by them; recs (or null):
// edits of the map that go along.
int launch_copies(const fc_pages* p, const std::vector<Pair>& pairs, bool remap, const std::vector<Rec>* recs,
                  cudaStream_t stream) {
  const MapView m{p->table, p->lens, p->batch, p->max_pages};
  CopyShape s{};
  const int64_t es = dtype_size(p->dtype);
  s.base[0] = static_cast<char*>(p->k);
  s.base[1] = static_cast<char*>(p->v);
  s.base[2] = reinterpret_cast<char*>(p->k_scales);
  s.base[3] = reinterpret_cast<char*>(p->v_scales);
  s.layer[0] = p->stride_layer * es;
  s.page[0] = p->stride_page * es;
  s.head[0] = p->stride_head * es;
  s.run[0] = p->page_size * p->D * es;
  s.layer[1] = p->scale_stride_layer * 4;
  s.page[1] = p->scale_stride_page * 4;
  s.head[1] = p->scale_stride_head * 4;
  s.run[1] = int64_t(p->page_size) * 4;
  s.n_layers = uint32_t(p->n_layers);
  s.H = uint32_t(p->H);
  s.pieces = uint32_t((s.run[0] + kPieceBytes - 1) / kPieceBytes);
  // units are counted in 32 bits (below 2^31, so that a stride cannot wrap)
  const int64_t per_pair = p->n_layers * 2 * p->H * (s.pieces + 1);
  const int64_t fit = (int64_t(1) << 31) / per_pair - 1;
  if (fit < 1) return FC_ERR_UNSUPPORTED;
  const size_t most = size_t(fit < kManyPairs ? fit : kManyPairs);
  if (remap) {
    s.table = p->table;
    s.table_entries = p->n_slots * p->max_pages;
  }
  if (recs && !pairs.empty() && pairs.size() <= size_t(kFewPairs) && pairs.size() <= most &&
      recs->size() <= size_t(kFewRecs))
    return launch_pairs<kFewPairs, kFewRecs>(s, pairs.data(), int(pairs.size()), m, recs, stream);
  for (size_t at = 0; at < pairs.size();) {
    const size_t left = pairs.size() - at;
    const int n = int(left > most ? most : left);
    const int st = n <= kFewPairs ? launch_pairs<kFewPairs, 0>(s, &pairs[at], n, m, nullptr, stream)
                                  : launch_pairs<kManyPairs, 0>(s, &pairs[at], n, m, nullptr, stream);
    if (st != FC_OK) return st;
    at += size_t(n);
  }
  return recs ? launch_edits(p, *recs, stream) : FC_OK;
}

// ----------------------------------------------------- uploading a whole map

constexpr int kSegs = 200, kInts = 6000;
struct MapChunk {
  MapView m;
  int32_t n;
  struct {
    int32_t slot, at, n, off;  // table[slot][at ..] (slot < 0: lens[at ..]) = v[off ..]
  } seg[kSegs];
  int32_t v[kInts];
};

__global__ void __launch_bounds__(128) upload_map_kernel(const __grid_constant__ MapChunk c) {
  const auto& g = c.seg[blockIdx.x];
  after_previous();
  int32_t* to = g.slot < 0 ? c.m.lens + g.at : c.m.table + int64_t(g.slot) * c.m.max_pages + g.at;
  for (int i = int(threadIdx.x); i < g.n; i += 128) to[i] = c.v[g.off + i];
}

struct MapUpload {
  MapChunk c;
  int used = 0;
  cudaStream_t s;
  explicit MapUpload(const fc_pages* p, cudaStream_t stream) : s(stream) {
    c.m = MapView{p->table, p->lens, p->batch, p->max_pages};
    c.n = 0;
  }
  int flush() {
    if (c.n == 0) return FC_OK;
    const int st = launch_after(upload_map_kernel, dim3(unsigned(c.n)), 128, 0, s, c);
    c.n = used = 0;
    return st;
  }
  int add(int32_t slot, const int32_t* v, int64_t n) {
    for (int64_t at = 0; at < n;) {
      if (c.n == kSegs || used == kInts) {
        const int st = flush();
        if (st != FC_OK) return st;
      }
      const int64_t m = n - at < kInts - used ? n - at : kInts - used;
      auto& g = c.seg[c.n++];
      g.slot = slot;
      g.at = int32_t(at);
      g.n = int32_t(m);
      g.off = used;
      for (int64_t i = 0; i < m; ++i) c.v[used + i] = v[at + i];
      used += int(m);
      at += m;
    }
    return FC_OK;
  }
};

// ------------------------------------------------------------ host decisions

// Changes of the host map that can be taken back.
class HostEdit {
 public:
  explicit HostEdit(fc_pages* p) : p_(p), saved_(*p) {}
  ~HostEdit() {
    if (done_) return;
    for (size_t i = log_.size(); i-- > 0;) *log_[i].first = log_[i].second;
    *p_ = saved_;
  }
  void set(int32_t* at, int32_t v) {
    log_.emplace_back(at, *at);
    *at = v;
  }
  void keep() { done_ = true; }

  int32_t* entry(int32_t slot, int64_t i) { return p_->h_table + int64_t(slot) * p_->max_pages + i; }
  // The lowest free page, now used once; the caller has seen that one is free.
  int32_t take() {
    int64_t g = p_->first_free;
    while (g < p_->n_pages && p_->h_refs[g] != 0) ++g;
    if (g >= p_->n_pages) return -1;
    set(&p_->h_refs[g], 1);
    p_->first_free = g + 1;
    --p_->n_free;
    return int32_t(g);
  }
  void drop(int32_t g) {
    set(&p_->h_refs[g], p_->h_refs[g] - 1);
    if (p_->h_refs[g] == 0) {
      ++p_->n_free;
      if (g < p_->first_free) p_->first_free = g;
    }
  }

 private:
  fc_pages* p_;
  fc_pages saved_;
  std::vector<std::pair<int32_t*, int32_t>> log_;
  bool done_ = false;
};

inline int64_t pages_for(const fc_pages* p, int64_t len) { return (len + p->page_size - 1) / p->page_size; }

// Runs a call's body; no exception leaves it (bad_alloc of the host lists).
template <typename F>
int guarded(F body) {
  try {
    return body();
  } catch (...) {
    return FC_ERR_CAPACITY;
  }
}

int check_slots(const fc_pages* p, const int32_t* slots, int64_t n, std::vector<uint8_t>* seen) {
  if (n < 0 || n > p->n_slots || (n > 0 && !slots)) return FC_ERR_INVALID;
  seen->assign(size_t(p->n_slots), 0);
  for (int64_t i = 0; i < n; ++i) {
    if (slots[i] < 0 || slots[i] >= p->n_slots || (*seen)[size_t(slots[i])]) return FC_ERR_INVALID;
    (*seen)[size_t(slots[i])] = 1;
  }
  return FC_OK;
}

// Empties a slot's entries from page index `from` on (after its edit is queued).
void drop_pages(fc_pages* p, int32_t slot, int64_t from) {
  int32_t* row = p->h_table + int64_t(slot) * p->max_pages;
  for (int64_t i = from, n = pages_for(p, p->h_lens[slot]); i < n; ++i) {
    const int32_t g = row[i];
    row[i] = -1;
    if (--p->h_refs[g] == 0) {
      ++p->n_free;
      if (g < p->first_free) p->first_free = g;
    }
  }
}

void close_batch(fc_pages* p) {
  p->n_rows = p->n_tokens = 0;
  p->one_each = 0;
}

int start_call(const fc_pages* p, fc_stream stream) {
  const int st = check_pages(p);
  return st != FC_OK ? st : check_not_capturing(stream);
}

}  // namespace

int check_pages(const fc_pages* p) {
  if (!p || !p->k || !p->v || !p->table || !p->lens || !p->batch || !p->h_table || !p->h_lens || !p->h_refs)
    return FC_ERR_INVALID;
  const int64_t es = dtype_size(p->dtype);
  if (es == 0) return FC_ERR_INVALID;
  const bool quant = p->dtype == FC_DTYPE_I8;
  if (quant != (p->k_scales != nullptr) || quant != (p->v_scales != nullptr)) return FC_ERR_INVALID;
  if (p->n_layers < 1 || p->n_pages < 1 || p->H < 1 || p->n_slots < 1 || p->max_pages < 1) return FC_ERR_INVALID;
  if (p->page_size < 1 || (p->page_size & (p->page_size - 1))) return FC_ERR_INVALID;
  if (!paged_dim_ok(p->D) || p->page_size < 8 || p->page_size > 1024) return FC_ERR_UNSUPPORTED;
  constexpr int64_t kMost = int64_t(1) << 30;
  if (p->n_pages > kMost || p->n_slots > kMost || p->max_pages > kMost || p->H > 65535 || p->n_layers > 65535 ||
      p->max_pages * p->page_size > kMost || p->n_slots > kMost / p->max_pages)
    return FC_ERR_UNSUPPORTED;
  if (!aligned16(p->k) || !aligned16(p->v) || !aligned16(p->batch)) return FC_ERR_INVALID;
  const int64_t run = p->page_size * p->D;
  if (p->stride_head < run || p->stride_page < run || p->stride_layer < 0) return FC_ERR_INVALID;
  if (p->stride_head * es % 16 || p->stride_page * es % 16 || p->stride_layer * es % 16) return FC_ERR_INVALID;
  if (quant) {
    if (!aligned16(p->k_scales) || !aligned16(p->v_scales)) return FC_ERR_INVALID;
    if (p->scale_stride_head < p->page_size || p->scale_stride_page < p->page_size || p->scale_stride_layer < 0)
      return FC_ERR_INVALID;
    if (p->scale_stride_head % 4 || p->scale_stride_page % 4 || p->scale_stride_layer % 4) return FC_ERR_INVALID;
  }
  return FC_OK;
}

int check_not_capturing(fc_stream stream) {
  cudaStreamCaptureStatus c = cudaStreamCaptureStatusNone;
  const cudaError_t e = cudaStreamIsCapturing(static_cast<cudaStream_t>(stream), &c);
  if (e != cudaSuccess) {
    // no device (host-only use of the validation): nothing can be capturing
    (void)cudaGetLastError();
    return e == cudaErrorNoDevice || e == cudaErrorInsufficientDriver ? FC_OK : FC_ERR_CUDA;
  }
  return c == cudaStreamCaptureStatusNone ? FC_OK : FC_ERR_INVALID;
}

PageView page_view(const fc_pages* p, int64_t layer) {
  PageView a{};
  const int64_t es = dtype_size(p->dtype);
  a.k = static_cast<char*>(p->k) + layer * p->stride_layer * es;
  a.v = static_cast<char*>(p->v) + layer * p->stride_layer * es;
  if (p->k_scales) {
    a.ks = p->k_scales + layer * p->scale_stride_layer;
    a.vs = p->v_scales + layer * p->scale_stride_layer;
  }
  a.stride_page = p->stride_page;
  a.stride_head = p->stride_head;
  a.sstride_page = p->scale_stride_page;
  a.sstride_head = p->scale_stride_head;
  a.table = p->table;
  a.batch = reinterpret_cast<const BatchRow*>(p->batch);
  a.max_pages = int32_t(p->max_pages);
  a.n_pages = int32_t(p->n_pages);
  a.n_slots = int32_t(p->n_slots);
  a.n_rows = int32_t(p->n_rows);
  a.H = int32_t(p->H);
  while ((1 << a.log2P) < p->page_size) ++a.log2P;
  return a;
}

}  // namespace fc

using namespace fc;

extern "C" int fc_pages_reset(fc_pages* p, fc_stream stream) {
  const int st = start_call(p, stream);
  if (st != FC_OK) return st;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const size_t entries = size_t(p->n_slots) * size_t(p->max_pages);
  cudaError_t e = cudaMemsetAsync(p->table, 0xff, entries * 4, s);
  if (e == cudaSuccess) e = cudaMemsetAsync(p->lens, 0, size_t(p->n_slots) * 4, s);
  if (e == cudaSuccess) e = cudaMemsetAsync(p->batch, 0xff, size_t(p->n_slots) * 16, s);  // slot -1
  if (e != cudaSuccess) return FC_ERR_CUDA;
  for (size_t i = 0; i < entries; ++i) p->h_table[i] = -1;
  for (int64_t i = 0; i < p->n_slots; ++i) p->h_lens[i] = 0;
  for (int64_t i = 0; i < p->n_pages; ++i) p->h_refs[i] = 0;
  p->first_free = 0;
  p->n_free = p->n_pages;
  p->device_rows = 0;
  close_batch(p);
  return FC_OK;
}

extern "C" int fc_pages_restore(fc_pages* p, const int32_t* table, const int32_t* lens, fc_stream stream) {
  const int st0 = start_call(p, stream);
  if (st0 != FC_OK) return st0;
  if (!table || !lens) return FC_ERR_INVALID;
  return guarded([&]() -> int {
    std::vector<int32_t> refs(size_t(p->n_pages), 0), last(size_t(p->n_pages), -1);
    int64_t used = 0;
    for (int64_t s = 0; s < p->n_slots; ++s) {
      if (lens[s] < 0 || lens[s] > p->max_pages * p->page_size) return FC_ERR_INVALID;
      const int64_t n = pages_for(p, lens[s]);
      for (int64_t i = 0; i < n; ++i) {
        const int32_t g = table[s * p->max_pages + i];
        if (g < 0 || g >= p->n_pages || last[size_t(g)] == s) return FC_ERR_INVALID;
        last[size_t(g)] = int32_t(s);
        used += refs[size_t(g)]++ == 0;
      }
    }
    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
    if (cudaMemsetAsync(p->table, 0xff, size_t(p->n_slots) * size_t(p->max_pages) * 4, cs) != cudaSuccess)
      return FC_ERR_CUDA;
    const std::unique_ptr<MapUpload> up(new MapUpload(p, cs));  // 28 KB: kept off the stack
    int st = up->add(-1, lens, p->n_slots);
    for (int64_t s = 0; s < p->n_slots && st == FC_OK; ++s)
      st = up->add(int32_t(s), table + s * p->max_pages, pages_for(p, lens[s]));
    if (st == FC_OK) st = up->flush();
    if (st != FC_OK) return st;
    for (int64_t s = 0; s < p->n_slots; ++s) {
      const int64_t n = pages_for(p, lens[s]);
      for (int64_t i = 0; i < p->max_pages; ++i) {
        const int64_t at = s * p->max_pages + i;
        p->h_table[at] = i < n ? table[at] : -1;
      }
      p->h_lens[s] = lens[s];
    }
    for (int64_t g = 0; g < p->n_pages; ++g) p->h_refs[g] = refs[size_t(g)];
    p->first_free = 0;
    p->n_free = p->n_pages - used;
    close_batch(p);
    return FC_OK;
  });
}

extern "C" int fc_pages_begin(fc_pages* p, const int32_t* slots, const int32_t* counts, int64_t n,
                              int64_t n_rows, fc_stream stream) {
  const int st0 = start_call(p, stream);
  if (st0 != FC_OK) return st0;
  if (n < 1 || n_rows < n || n_rows > p->n_slots) return FC_ERR_INVALID;
  return guarded([&]() -> int {
    std::vector<uint8_t> seen;
    int st = check_slots(p, slots, n, &seen);
    if (st != FC_OK) return st;
    int64_t total = 0;
    bool one_each = true;
    for (int64_t i = 0; i < n; ++i) {
      const int64_t c = counts ? counts[i] : 1;
      if (c < 0) return FC_ERR_INVALID;
      if (p->h_lens[slots[i]] + c > p->max_pages * p->page_size) return FC_ERR_CAPACITY;
      total += c;
      one_each = one_each && c == 1;
    }
    if (total > INT32_MAX) return FC_ERR_UNSUPPORTED;
    std::vector<Rec> recs;
    std::vector<Pair> copies;
    HostEdit ed(p);
    int32_t first = 0;
    for (int64_t i = 0; i < n; ++i) {
      const int32_t slot = slots[i], len = p->h_lens[slot];
      const int32_t c = counts ? counts[i] : 1, now = len + c;
      int64_t at = pages_for(p, len);
      if (c > 0 && len % p->page_size) {
        const int32_t old = *ed.entry(slot, at - 1);
        if (p->h_refs[old] > 1) {  // shared: copied before it is written
          const int32_t g = ed.take();
          if (g < 0) return FC_ERR_CAPACITY;
          ed.drop(old);
          ed.set(ed.entry(slot, at - 1), g);
          copies.push_back({old, g});
          recs.push_back({kRun, slot, int32_t(at - 1), g, 1, 0});
        }
      }
      for (const int64_t end = pages_for(p, now); at < end; ++at) {
        const int32_t g = ed.take();
        if (g < 0) return FC_ERR_CAPACITY;
        ed.set(ed.entry(slot, at), g);
        if (!recs.empty() && recs.back().op == kRun && recs.back().a == slot &&
            recs.back().b + recs.back().d == at && recs.back().c + recs.back().d == g)
          ++recs.back().d;
        else
          recs.push_back({kRun, slot, int32_t(at), g, 1, 0});
      }
      ed.set(&p->h_lens[slot], now);
      recs.push_back({kRow, int32_t(i), slot, now, first, c});
      first += c;
    }
    // padding, and what a larger batch left behind (a captured launch may read it)
    const int64_t rows = p->device_rows > n_rows ? p->device_rows : n_rows;
    for (int64_t i = n; i < rows; ++i) recs.push_back({kRow, int32_t(i), -1, 0, first, 0});
    p->n_rows = n_rows;
    p->device_rows = int32_t(n_rows);
    p->n_tokens = total;
    p->one_each = one_each ? 1 : 0;
    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
    if ((st = launch_copies(p, copies, false, &recs, cs)) != FC_OK) return st;
    ed.keep();
    return FC_OK;
  });
}

extern "C" int fc_pages_fork(fc_pages* p, const int32_t* src, const int32_t* dst, int64_t n, fc_stream stream) {
  const int st0 = start_call(p, stream);
  if (st0 != FC_OK) return st0;
  return guarded([&]() -> int {
    std::vector<uint8_t> seen;
    int st = check_slots(p, dst, n, &seen);
    if (st != FC_OK) return st;
    if (n > 0 && !src) return FC_ERR_INVALID;
    for (int64_t i = 0; i < n; ++i) {
      if (src[i] < 0 || src[i] >= p->n_slots || seen[size_t(src[i])] || p->h_lens[dst[i]] != 0)
        return FC_ERR_INVALID;
    }
    std::vector<Rec> recs;
    for (int64_t i = 0; i < n; ++i)
      recs.push_back({kFork, src[i], dst[i], int32_t(pages_for(p, p->h_lens[src[i]])), p->h_lens[src[i]], 0});
    if ((st = launch_edits(p, recs, static_cast<cudaStream_t>(stream))) != FC_OK) return st;
    for (int64_t i = 0; i < n; ++i) {
      const int32_t* from = p->h_table + int64_t(src[i]) * p->max_pages;
      int32_t* to = p->h_table + int64_t(dst[i]) * p->max_pages;
      for (int64_t j = 0, m = pages_for(p, p->h_lens[src[i]]); j < m; ++j) ++p->h_refs[to[j] = from[j]];
      p->h_lens[dst[i]] = p->h_lens[src[i]];
    }
    close_batch(p);
    return FC_OK;
  });
}

extern "C" int fc_pages_free(fc_pages* p, const int32_t* slots, int64_t n, fc_stream stream) {
  const int st0 = start_call(p, stream);
  if (st0 != FC_OK) return st0;
  return guarded([&]() -> int {
    std::vector<uint8_t> seen;
    int st = check_slots(p, slots, n, &seen);
    if (st != FC_OK) return st;
    std::vector<Rec> recs;
    for (int64_t i = 0; i < n; ++i) {
      if (p->h_lens[slots[i]] == 0) continue;
      recs.push_back({kCrop, slots[i], 0, 0, int32_t(pages_for(p, p->h_lens[slots[i]])), 0});
    }
    if ((st = launch_edits(p, recs, static_cast<cudaStream_t>(stream))) != FC_OK) return st;
    for (int64_t i = 0; i < n; ++i) {
      drop_pages(p, slots[i], 0);
      p->h_lens[slots[i]] = 0;
    }
    close_batch(p);
    return FC_OK;
  });
}

extern "C" int fc_pages_crop(fc_pages* p, int32_t slot, int64_t tokens_to_remove, fc_stream stream) {
  const int st0 = start_call(p, stream);
  if (st0 != FC_OK) return st0;
  if (slot < 0 || slot >= p->n_slots || tokens_to_remove > 0) return FC_ERR_INVALID;
  const int64_t len = p->h_lens[slot];
  const int64_t now = tokens_to_remove < -len ? 0 : len + tokens_to_remove;
  if (now == len) return FC_OK;
  return guarded([&]() -> int {
    const int64_t kept = pages_for(p, now);
    const std::vector<Rec> recs{{kCrop, slot, int32_t(now), int32_t(kept), int32_t(pages_for(p, len) - kept), 0}};
    const int st = launch_edits(p, recs, static_cast<cudaStream_t>(stream));
    if (st != FC_OK) return st;
    drop_pages(p, slot, kept);
    p->h_lens[slot] = int32_t(now);
    close_batch(p);
    return FC_OK;
  });
}

extern "C" int fc_pages_compact(fc_pages* p, int64_t* n_live, fc_stream stream) {
  const int st0 = start_call(p, stream);
  if (st0 != FC_OK) return st0;
  return guarded([&]() -> int {
    const int64_t live = p->n_pages - p->n_free;
    std::vector<Pair> moves;
    int64_t hole = 0;
    for (int64_t g = live; g < p->n_pages; ++g) {
      if (p->h_refs[g] == 0) continue;
      while (p->h_refs[hole] != 0) ++hole;  // as many holes as moved pages
      moves.push_back({int32_t(g), int32_t(hole++)});
    }
    if (!moves.empty()) {
      std::vector<int32_t> to(size_t(p->n_pages - live), -1);
      for (const Pair& m : moves) to[size_t(m.src - live)] = m.dst;
      const int st = launch_copies(p, moves, true, nullptr, static_cast<cudaStream_t>(stream));
      if (st != FC_OK) return st;
      for (int64_t s = 0; s < p->n_slots; ++s) {
        int32_t* row = p->h_table + s * p->max_pages;
        const int64_t m = pages_for(p, p->h_lens[s]);
        for (int64_t i = 0; i < m; ++i)
          if (row[i] >= live) row[i] = to[size_t(row[i] - live)];
      }
      for (const Pair& m : moves) {
        p->h_refs[m.dst] = p->h_refs[m.src];
        p->h_refs[m.src] = 0;
      }
    }
    p->first_free = live;
    if (n_live) *n_live = live;
    return FC_OK;
  });
}
