// api_paged.cu -- C ABI of the caches in pages: argument checks on the host, then launches (csa.h has the contracts).

#include <algorithm>
#include <cmath>

#include "host.cuh"
#include "kernels.cuh"

namespace csa {

int check_table(const csa_page_table* pt, int B) {
  CSA_CHECK_ARG(pt != nullptr, "page table is null");
  CSA_CHECK_ARG(pt->slots > 0 && pt->max_pages > 0 && pt->num_pages > 0, "slots, max_pages and num_pages must be positive");
  CSA_CHECK_SUP(pt->page_size >= 16 && pt->page_size <= 1024 && (pt->page_size & (pt->page_size - 1)) == 0,
                "page_size must be a power of two in [16, 1024]");
  CSA_CHECK_SUP((long long)pt->num_pages * pt->page_size < (1ll << 31) &&
                    (long long)pt->max_pages * pt->page_size < (1ll << 31) &&
                    (long long)pt->slots * pt->max_pages < (1ll << 31),
                "page table too large for 32-bit rows");
  CSA_CHECK_ARG(pt->table && pt->refs && aligned(pt->table, 4) && aligned(pt->refs, 4), "table or refs null or misaligned");
  CSA_CHECK_ARG(B > 0 && B <= pt->slots, "B must be in [1, slots]");
  return CSA_OK;
}

namespace {

int check_cache(const csa_page_table* pt, const csa_paged_cache* c) {
  CSA_CHECK_ARG(c != nullptr && c->pages != nullptr && aligned(c->pages, 16), "cache or its pages null or misaligned");
  if (c->scales != nullptr) {
    CSA_CHECK_SUP(c->d == 512, "an 8-bit cache has rows of 512");
    CSA_CHECK_SUP(c->block >= 1 && c->block <= kAppendMaxUnit && (c->block & (c->block - 1)) == 0 && c->block <= pt->page_size,
                  "block must be a power of two in [1, %d], at most page_size", kAppendMaxUnit);
    CSA_CHECK_ARG(aligned(c->scales, 16), "scales misaligned");
  } else {
    CSA_CHECK_SUP(c->d >= 8 && c->d <= 512 && c->d % 8 == 0, "a bf16 cache has rows of 8 .. 512 values, a multiple of 8");
  }
  return CSA_OK;
}

struct PagesWs {
  size_t n_moves, list_a, list_b, move_src, move_dst, heir, need, copy, last, rows, total;
};

PagesWs pages_ws_layout(long long slots, long long max_pages, long long num_pages) {
  PagesWs w{};
  size_t off = kStatusBytes;
  auto take = [&](long long ints) {
    const size_t at = off;
    off = round_up(off + (size_t)ints * 4, 256);
    return at;
  };
  w.n_moves = take(1);
  w.list_a = take(num_pages);
  w.list_b = take(num_pages);
  w.move_src = take(num_pages);
  w.move_dst = take(num_pages);
  w.heir = take(num_pages);
  w.need = take(slots);
  w.copy = take(slots);
  w.last = take(slots);
  w.rows = take(slots * max_pages);
  w.total = off;
  return w;
}

int pages_params(const csa_page_table* pt, void* ws, size_t ws_bytes, PagesParams* P) {
  const PagesWs w = pages_ws_layout(pt->slots, pt->max_pages, pt->num_pages);
  if (int rc = check_ws(ws, ws_bytes, w.total)) return rc;
  char* base = static_cast<char*>(ws);
  *P = PagesParams{};
  P->slots = pt->slots;
  P->max_pages = pt->max_pages;
  P->num_pages = pt->num_pages;
  P->page_shift = log2_int(pt->page_size);
  P->table = pt->table;
  P->refs = pt->refs;
  P->n_moves = reinterpret_cast<int*>(base + w.n_moves);
  P->list_a = reinterpret_cast<int*>(base + w.list_a);
  P->list_b = reinterpret_cast<int*>(base + w.list_b);
  P->move_src = reinterpret_cast<int*>(base + w.move_src);
  P->move_dst = reinterpret_cast<int*>(base + w.move_dst);
  P->heir = reinterpret_cast<int*>(base + w.heir);
  P->need = reinterpret_cast<int*>(base + w.need);
  P->copy = reinterpret_cast<int*>(base + w.copy);
  P->last = reinterpret_cast<int*>(base + w.last);
  P->rows = reinterpret_cast<int*>(base + w.rows);
  P->status = reinterpret_cast<uint32_t*>(ws);
  return CSA_OK;
}

cudaError_t launch_table(void (*one)(PagesParams), void (*cluster)(PagesParams), const PagesParams& P, cudaStream_t st) {
  const bool small = (long long)P.slots * P.max_pages + P.num_pages <= kPagesSmall && P.slots <= kPagesSmallSlots;
  return launch_pdl(small ? one : cluster, dim3(small ? 1 : kPagesCluster), dim3(kPagesThreads), 0, st, P);
}

int check_caches(const csa_page_table* pt, const csa_paged_cache* caches, int n) {
  CSA_CHECK_ARG(n >= 0 && n <= 1024 && (n == 0 || caches != nullptr), "n_caches must be in [0, 1024]");
  for (int i = 0; i < n; ++i)
    if (int rc = check_cache(pt, caches + i)) return rc;
  return CSA_OK;
}

// The moves that a table operation left in its workspace, in every cache (kMaxCaches a launch).
int copy_pages(const csa_page_table* pt, const csa_paged_cache* caches, int n, long long max_moves, const PagesParams& T,
               const DeviceInfo& dev, cudaStream_t st) {
  for (int c0 = 0; c0 < n; c0 += kMaxCaches) {
    CopyParams P{};
    P.n_moves = T.n_moves;
    P.move_src = T.move_src;
    P.move_dst = T.move_dst;
    int np = 0;
    long long units = 0;
    auto pool = [&](void* base, long long bytes) {
      PagePool& q = P.pool[np++];
      q.base = static_cast<uint8_t*>(base);
      q.page_bytes = (int)bytes;
      q.units = (int)((bytes + kCopyChunk - 1) / kCopyChunk);
      units += q.units;
    };
    for (int c = c0; c < std::min(n, c0 + kMaxCaches); ++c) {
      const csa_paged_cache& k = caches[c];
      pool(k.pages, (long long)pt->page_size * k.d * (k.scales ? 1 : 2));
      if (k.scales) pool(k.scales, (long long)pt->page_size / k.block * 4);
    }
    P.units_per_page = (int)units;
    const long long grid = std::min<long long>(max_moves * units, (long long)dev.sms * 8);
    CSA_CUDA(launch_pdl(pages_copy_kernel, dim3((unsigned)std::max<long long>(1, grid)), dim3(kCopyThreads), 0, st, P));
  }
  return CSA_OK;
}

int run_attn8(const csa_attn8_args* args, bool list, cudaStream_t st) {
  CSA_CHECK_ARG(args != nullptr, "args is null");
  const csa_attn8_args& a = *args;
  const csa_page_table* pt = a.pt;
  const csa_paged_cache* c = a.cache;
  if (int rc = check_paged(pt, c, a.B, true)) return rc;
  CSA_CHECK_ARG(a.S > 0, "S must be positive");
  CSA_CHECK_SUP(a.H >= 1 && a.H <= 128, "H must be in [1, 128]");
  CSA_CHECK_SUP(a.rope_dim >= 2 && a.rope_dim % 2 == 0 && a.rope_dim / 2 <= kMaxRopePairs, "rope_dim must be even and <= 128");
  CSA_CHECK_ARG(std::isfinite(a.rope_base) && a.rope_base > 0.f, "rope_base must be positive");
  CSA_CHECK_ARG(std::isfinite(a.scale), "scale must be finite");
  CSA_CHECK_ARG(a.ratio > 0, "ratio must be positive");
  CSA_CHECK_SUP(a.window >= 1 && a.window <= kAttnMaxWindow, "window must be in [1, %d]", kAttnMaxWindow);
  CSA_CHECK_ARG(a.ring_cap >= a.window, "ring_cap must be >= window");
  CSA_CHECK_ARG(a.q_pos && a.q && a.ring && a.sink && a.out, "null pointer argument");
  CSA_CHECK_ARG(aligned(a.q, 16) && aligned(a.ring, 16) && aligned(a.out, 16) && aligned(a.sink, 4) && aligned(a.q_pos, 4),
                "misaligned pointer");
  CSA_CHECK_ARG(a.ring_bstride % 8 == 0 && a.ring_bstride >= (int64_t)a.ring_cap * 512,
                "ring_bstride must be a multiple of 8 and >= ring_cap*512");
  CSA_CHECK_SUP((long long)a.B * a.S * a.H < (1ll << 31), "too many query rows");
  CSA_CHECK_SUP((long long)a.B * a.S < (1ll << 29), "at most 2^29 queries");
  if (list) {
    CSA_CHECK_ARG(a.topk_idx != nullptr && aligned(a.topk_idx, 4), "topk_idx null or misaligned");
    CSA_CHECK_SUP(a.topk >= 1 && a.topk <= kAttnMaxTopk, "topk must be in [1, %d]", kAttnMaxTopk);
  }
  if (int rc = check_ws(a.ws, a.ws_bytes, kStatusBytes)) return rc;
  DeviceInfo* dev;
  if (int rc = device_info(&dev)) return rc;
  Attn8Params P{};
  P.B = a.B;
  P.S = a.S;
  P.H = a.H;
  P.rope_dim = a.rope_dim;
  const double step = std::pow((double)a.rope_base, -2.0 / a.rope_dim);
  P.inv_freq[0] = 1.0;
  for (int i = 1; i < a.rope_dim / 2; ++i) P.inv_freq[i] = P.inv_freq[i - 1] * step;
  P.scale_log2 = a.scale * 1.4426950408889634f;
  P.window = a.window;
  P.ring_cap = a.ring_cap;
  P.ring_bstride = a.ring_bstride;
  P.ring = a.ring;
  P.pages = static_cast<const uint8_t*>(c->pages);
  P.scales = c->scales;
  P.table = pt->table;
  P.num_pages = pt->num_pages;
  P.page_shift = log2_int(pt->page_size);
  P.block_shift = log2_int(c->block);
  P.max_pages = pt->max_pages;
  P.max_entries = pt->max_pages * pt->page_size;
  P.ratio = a.ratio;
  P.q_pos = a.q_pos;
  P.q = a.q;
  P.topk_idx = list ? a.topk_idx : nullptr;
  P.topk = list ? a.topk : 0;
  P.sink = a.sink;
  P.out = a.out;
  P.out_is_f32 = a.out_is_f32 ? 1 : 0;
  P.status = reinterpret_cast<uint32_t*>(a.ws);
  const size_t smem = attn8_smem_bytes();
  CSA_CHECK_SUP(smem <= (size_t)dev->max_smem, "shared memory too small for the attention kernel");
  // Splits: as many as the device's CTA pairs allow per query (and the workspace holds), two tiles of the longest
  // candidate list a split at least; and only where the tiles that a split saves outweigh the partials and their
  // merge, which cost as much as 2 tiles and 0.27 a query (of 128 heads). Measured on a B200, one split against all: 24
  // queries of 12 tiles 27.8 and 28.9 us, of 20 tiles 37.1 and 32.6; 37 queries of 20 tiles 38.5 and 40.3, of 36 tiles 58.1
  // and 52.5; 8 queries of 8 tiles 22.2 and 20.7, of 5 tiles 19.2 and 21.2; one query of 8 tiles 22.0 and 18.1.
  const long long queries = (long long)a.B * a.S;
  const long long max_tiles = (a.window + 31) / 32 + ((long long)(list ? a.topk : P.max_entries) + 63) / 64;
  int splits = (int)std::min<long long>(attn_ws_splits(queries), std::max<long long>(1, (dev->sms / 2) / queries));
  splits = (int)std::max<long long>(1, std::min<long long>(splits, max_tiles / 2));
  if (max_tiles * (splits - 1) * 128 * 100 <= splits * (200 * 128 + 27 * queries * a.H)) splits = 1;
  if (splits > 1 && a.ws_bytes < kStatusBytes + attn_part_bytes(queries, splits)) splits = 1;
  P.splits = splits;
  if (splits > 1) {
    P.part_o = reinterpret_cast<float*>(static_cast<char*>(a.ws) + kStatusBytes);
    P.part_ml = P.part_o + (size_t)queries * splits * 128 * 512;
  }
  CSA_CUDA(launch_pdl(attn8_kernel, dim3((unsigned)(2 * queries * splits)), dim3(kAttn8Threads), smem, st, P));
  if (splits > 1) {
    AttnCombineParams C{};
    C.splits = splits;
    C.H = a.H;
    C.d = 512;
    C.rope_dim = a.rope_dim;
    for (int i = 0; i < a.rope_dim / 2; ++i) C.inv_freq[i] = P.inv_freq[i];
    C.q_pos = a.q_pos;
    C.part_o = P.part_o;
    C.part_ml = P.part_ml;
    C.out = a.out;
    C.out_is_f32 = P.out_is_f32;
    C.status = P.status;
    CSA_CUDA(launch_pdl(attn_combine_kernel, dim3((unsigned)a.H, (unsigned)queries), dim3(kAttnCombineThreads), 0, st, C));
  }
  return CSA_OK;
}

}  // namespace

int check_paged(const csa_page_table* pt, const csa_paged_cache* c, int B, bool quantised) {
  if (int rc = check_table(pt, B)) return rc;
  if (int rc = check_cache(pt, c)) return rc;
  CSA_CHECK_ARG((c->scales != nullptr) == quantised, quantised ? "the cache must be an 8-bit one" : "the cache must be a bf16 one");
  return CSA_OK;
}

size_t pages_ws_bytes(long long slots, long long max_pages, long long num_pages) {
  return pages_ws_layout(slots, max_pages, num_pages).total;
}

}  // namespace csa

using namespace csa;

extern "C" {

int csa_cache_append(const csa_page_table* pt, const csa_paged_cache* c, int B, int S, int ratio,
                     const int32_t* start_pos, const uint16_t* rows, int64_t rows_bstride, int max_rows, void* ws,
                     size_t ws_bytes, void* stream) {
  if (int rc = check_table(pt, B)) return rc;
  if (int rc = check_cache(pt, c)) return rc;
  CSA_CHECK_ARG(S > 0 && ratio > 0 && max_rows > 0, "S, ratio and max_rows must be positive");
  CSA_CHECK_ARG(start_pos && rows && aligned(start_pos, 4) && aligned(rows, 16), "start_pos or rows null or misaligned");
  CSA_CHECK_ARG(rows_bstride % 8 == 0 && rows_bstride >= 0, "rows_bstride must be a multiple of 8");
  CSA_CHECK_SUP(B <= 65535, "at most 65535 requests");
  if (int rc = check_ws(ws, ws_bytes, kStatusBytes)) return rc;
  DeviceInfo* dev;
  if (int rc = device_info(&dev)) return rc;
  AppendParams P{};
  P.S = S;
  P.ratio = ratio;
  P.start_pos = start_pos;
  P.rows = rows;
  P.rows_bstride = rows_bstride;
  P.max_rows = max_rows;
  P.d = c->d;
  P.pages = static_cast<uint8_t*>(c->pages);
  P.scales = c->scales;
  P.table = pt->table;
  P.refs = pt->refs;
  P.slots = pt->slots;
  P.num_pages = pt->num_pages;
  P.page_shift = log2_int(pt->page_size);
  P.block_shift = c->scales ? log2_int(c->block) : 0;
  P.max_pages = pt->max_pages;
  P.status = reinterpret_cast<uint32_t*>(ws);
  // A segment of S tokens completes at most ceil(S / ratio) entries; they begin anywhere in a unit.
  const long long n = ((long long)S + ratio - 1) / ratio;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (c->scales != nullptr) {
    P.unit = std::max(c->block, 16);
    const unsigned gx = (unsigned)((n + P.unit - 2) / P.unit + 1);
    void (*kernel)(AppendParams) = P.unit == 16 ? cache_append_kernel<2> : P.unit == 32 ? cache_append_kernel<4> : cache_append_kernel<8>;
    CSA_CUDA(launch_pdl(kernel, dim3(gx, (unsigned)B), dim3(kAppendThreads), 0, st, P));
  } else {
    const unsigned gx = (unsigned)((n + kAppendThreads / 32 - 1) / (kAppendThreads / 32));
    CSA_CUDA(launch_pdl(cache_append_bf16_kernel, dim3(gx, (unsigned)B), dim3(kAppendThreads), 0, st, P));
  }
  return CSA_OK;
}

int csa_cache_read(const csa_page_table* pt, const csa_paged_cache* c, int B, int n, const int32_t* idx, uint16_t* out,
                   void* ws, size_t ws_bytes, void* stream) {
  if (int rc = check_table(pt, B)) return rc;
  if (int rc = check_cache(pt, c)) return rc;
  CSA_CHECK_ARG(n > 0, "n must be positive");
  CSA_CHECK_ARG(idx && out && aligned(idx, 4) && aligned(out, 16), "idx or out null or misaligned");
  if (int rc = check_ws(ws, ws_bytes, kStatusBytes)) return rc;
  DeviceInfo* dev;
  if (int rc = device_info(&dev)) return rc;
  ReadParams P{};
  P.B = B;
  P.n = n;
  P.d = c->d;
  P.idx = idx;
  P.pages = static_cast<const uint8_t*>(c->pages);
  P.scales = c->scales;
  P.table = pt->table;
  P.num_pages = pt->num_pages;
  P.page_shift = log2_int(pt->page_size);
  P.block_shift = c->scales ? log2_int(c->block) : 0;
  P.max_pages = pt->max_pages;
  P.out = out;
  P.status = reinterpret_cast<uint32_t*>(ws);
  const long long grid = ((long long)B * n + kReadThreads / 32 - 1) / (kReadThreads / 32);
  CSA_CHECK_SUP(grid < (1ll << 31), "too many rows");
  CSA_CUDA(launch_pdl(cache_read_kernel, dim3((unsigned)grid), dim3(kReadThreads), 0, static_cast<cudaStream_t>(stream), P));
  return CSA_OK;
}

int csa_pages_reserve(const csa_page_table* pt, const int32_t* entries, void* ws, size_t ws_bytes, void* stream) {
  if (int rc = check_table(pt, 1)) return rc;
  CSA_CHECK_ARG(entries != nullptr && aligned(entries, 4), "entries null or misaligned");
  PagesParams P;
  if (int rc = pages_params(pt, ws, ws_bytes, &P)) return rc;
  DeviceInfo* dev;
  if (int rc = device_info(&dev)) return rc;
  P.entries = entries;
  CSA_CUDA(launch_table(pages_reserve_kernel, pages_reserve_cluster_kernel, P, static_cast<cudaStream_t>(stream)));
  return CSA_OK;
}

int csa_pages_fork(const csa_page_table* pt, const csa_paged_cache* caches, int n_caches, const int32_t* parent,
                   const int32_t* entries, void* ws, size_t ws_bytes, void* stream) {
  if (int rc = check_table(pt, 1)) return rc;
  if (int rc = check_caches(pt, caches, n_caches)) return rc;
  CSA_CHECK_ARG(parent && entries && aligned(parent, 4) && aligned(entries, 4), "parent or entries null or misaligned");
  PagesParams P;
  if (int rc = pages_params(pt, ws, ws_bytes, &P)) return rc;
  DeviceInfo* dev;
  if (int rc = device_info(&dev)) return rc;
  P.parent = parent;
  P.entries = entries;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  CSA_CUDA(launch_table(pages_fork_kernel, pages_fork_cluster_kernel, P, st));
  return copy_pages(pt, caches, n_caches, std::min(pt->slots, pt->num_pages), P, *dev, st);
}

int csa_pages_compact(const csa_page_table* pt, const csa_paged_cache* caches, int n_caches, int32_t* map, int32_t* live,
                      void* ws, size_t ws_bytes, void* stream) {
  if (int rc = check_table(pt, 1)) return rc;
  if (int rc = check_caches(pt, caches, n_caches)) return rc;
  CSA_CHECK_ARG(map && live && aligned(map, 4) && aligned(live, 4), "map or live null or misaligned");
  PagesParams P;
  if (int rc = pages_params(pt, ws, ws_bytes, &P)) return rc;
  DeviceInfo* dev;
  if (int rc = device_info(&dev)) return rc;
  P.map = map;
  P.live = live;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  CSA_CUDA(launch_table(pages_compact_kernel, pages_compact_cluster_kernel, P, st));
  return copy_pages(pt, caches, n_caches, pt->num_pages / 2 + 1, P, *dev, st);
}

int csa_sparse_attn8(const csa_attn8_args* a, void* stream) { return run_attn8(a, true, static_cast<cudaStream_t>(stream)); }

int hca_attn8(const csa_attn8_args* a, void* stream) { return run_attn8(a, false, static_cast<cudaStream_t>(stream)); }

}  // extern "C"
