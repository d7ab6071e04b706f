// paged.cu -- caches in pages: entries written into and read out of the pages, and the page table's life
// (reserve, fork / free, compact).
//
// A page table maps each slot (request) to pages of a pool: entry e of slot r is row e % page_size of page
// table[r][e / page_size]; refs[p] counts the table entries (and other holders) of page p, 0: free. Every
// cache laid out behind one table (a layer's main and index entries, every layer of a model) has a pool
// of the same page numbers. All of it lives in device memory and changes in stream order, so a captured decode
// step may contain these calls. Every choice is deterministic: new pages are the lowest free ones, in slot order.

#include <math_constants.h>

#include "attn_util.cuh"
#include "kernels.cuh"
#include "ptx.cuh"

namespace csa {

namespace {

__device__ __forceinline__ int ld_cg(const int* p) { return __ldcg(p); }

// Exclusive prefix sum over the block's threads (blockDim.x a multiple of 32, at most 1024); `total` in every
// thread. Begins and ends with a barrier.
__device__ __forceinline__ int block_scan(int v, int* smem /* 33 ints */, int& total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, nw = blockDim.x >> 5;
  int inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  __syncthreads();
  if (lane == 31) smem[w] = inc;
  __syncthreads();
  if (w == 0) {
    const int x = lane < nw ? smem[lane] : 0;
    int xi = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, xi, o);
      if (lane >= o) xi += y;
    }
    smem[lane] = xi - x;
    if (lane == 31) smem[32] = xi;
  }
  __syncthreads();
  total = smem[32];
  const int r = smem[w] + inc - v;
  __syncthreads();
  return r;
}

// A page-table operation runs on C CTAs: a cluster of 8, or one CTA where the table is small (then barriers are the
// CTA's, and the slots' arguments are in shared memory).
template <int C>
__device__ __forceinline__ void all_sync() {
  if (C == 1) __syncthreads();
  else cluster_sync();
}
template <int C>
__device__ __forceinline__ unsigned rank() {
  return C == 1 ? 0u : cluster_ctarank();
}

// Items [lo, hi) of [0, n) that this CTA walks, and of those the run of this thread.
template <int C>
__device__ __forceinline__ void my_run(unsigned n, unsigned& lo, unsigned& hi) {
  const unsigned c = rank<C>(), each = (n + C - 1) / C;
  const unsigned a = min(n, c * each), b = min(n, a + each);
  const unsigned per = (b - a + blockDim.x - 1) / blockDim.x;
  lo = min(b, a + per * threadIdx.x);
  hi = min(b, lo + per);
}

// N scans over all CTAs' threads at once: v[k] becomes the sum of v[k] in the threads before this one, total[k] that in
// all. Ends with a barrier of all, which also orders what was written before it. CTAs exchange their sums through
// shared memory: `sums` [2][3][kPagesCluster] of each CTA gets every CTA's; `turn`: calls take 0 and 1 in turn, so that a CTA ahead
// does not overwrite what another still reads.
template <int C, int N>
__device__ __forceinline__ void all_scan(int (&v)[N], int (&total)[N], int* smem, int (*sums)[3][kPagesCluster], int turn) {
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = block_scan(v[k], smem, total[k]);
  if (C == 1) return;
  if (threadIdx.x < C) {
    const uint32_t far = mapa_shared(smem_u32(&sums[turn][0][rank<C>()]), threadIdx.x);
#pragma unroll
    for (int k = 0; k < N; ++k)
      asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(far + (uint32_t)(k * kPagesCluster * 4)), "r"(total[k]) : "memory");
  }
  __syncwarp();
  all_sync<C>();
  const int c = (int)rank<C>();
#pragma unroll
  for (int k = 0; k < N; ++k) {
    total[k] = 0;
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int x = sums[turn][k][i];
      v[k] += i < c ? x : 0;
      total[k] += x;
    }
  }
}

}  // namespace

// ------------------------------------------------------------------------------------------------ append

// Whether a slot other than b has `page` at place lp too (a fork gives copies their pages at the parent's places). The threads
// of a warp or a CTA, `first` of `step`, look at their part of the slots; looked at only where the page has several holders.
__device__ __forceinline__ bool others_page(const AppendParams& P, int b, long long lp, int page, int first, int step) {
  bool other = false;
  for (int s = first; s < P.slots; s += step) other |= s != b && P.table[(long long)s * P.max_pages + lp] == page;
  return other;
}

// Entries [e0, e1) that a segment of S tokens at start_pos completes, from `rows` into the pages (e4m3).
// A CTA takes one unit of max(block, 16) entries (a block's rows share its scale, and a unit lies inside
// one page); a warp takes a row at a time, 16 dims a lane, and keeps it in registers between the block's maximum
// and the rounding, so every row is read once. Bound by latency: the position, then rows and page, then the page's holders and the
// block's scale, the codes. B200, blocks of 16: one entry of 64 requests 2.5 us, 8192 entries of four (8.4 MB read, 4.2 written) 4.3,
// 32768 of one 11.7 (2.7, 4.6 and 10.3 without the look at the holders and with the scale read behind the rows; with 16 warps a CTA
// 2 us more). Four CTAs an SM (64 registers; two for blocks of 64): for blocks of 16, five of 48 take 5.1 us at 8192 entries, for
// blocks of 32 three of 80 take 4.7 instead of 4.4.
//   scale of a block = the least power of two 2^k with max |x| <= 448 * 2^k over its rows, and never less
//   than before: when new rows raise it, the earlier rows' codes are rounded again to the new step (by an exact
//   power of two; only codes below e4m3's normal range lose bits).
// A power of two costs e4m3 nothing (its steps are relative) and makes every value of the cache
// exact in bf16. A row with a value that is not finite makes its block's scale NaN.
// kMax: rows a warp takes, unit / 8.
template <int kMax>
__global__ void __launch_bounds__(kAppendThreads, kMax == 8 ? 2 : 4) cache_append_kernel(AppendParams P) {
  __shared__ int row_k[kAppendMaxUnit];
  __shared__ float s_new[kAppendMaxUnit], s_old[kAppendMaxUnit];
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.y, warp = warp_id(), lane = lane_id();
  const int start = P.start_pos[b];
  if (start < 0) return;  // a padding request
  const long long e0 = start / P.ratio, e1 = ((long long)start + P.S) / P.ratio;
  const long long u0 = (e0 / P.unit + blockIdx.x) * P.unit;
  if (u0 >= e1 || e1 <= e0) return;
  const long long lp = u0 >> P.page_shift;
  const int page = lp < P.max_pages ? P.table[(long long)b * P.max_pages + lp] : -1;  // looked at behind the rows' reads
  constexpr int kWarps = kAppendThreads / 32;
  uint4 a[kMax], c[kMax];
  bool is_new[kMax];
#pragma unroll
  for (int i = 0; i < kMax; ++i) {
    const int r = warp + kWarps * i;
    const long long e = u0 + r;
    is_new[i] = r < P.unit && e >= e0 && e < e1;
    if (is_new[i] && e >= P.max_rows) {
      if (lane == 0) record_status(P.status, CSA_DEV_BOUNDS);
      is_new[i] = false;
    }
    if (is_new[i]) {
      const uint4* src = reinterpret_cast<const uint4*>(P.rows + (long long)b * P.rows_bstride + e * 512);
      a[i] = src[lane];
      c[i] = src[32 + lane];
    }
  }
  if (page < 0 || page >= P.num_pages) {
    if (threadIdx.x == 0) record_status(P.status, CSA_DEV_BOUNDS);
    return;
  }
  const long long row0 = ((long long)page << P.page_shift) + (u0 & ((1 << P.page_shift) - 1));
  // The page's holders, and the scale so far of the block that the thread's row begins: on their way beside the rows.
  const int held = P.refs[page], r0 = threadIdx.x, block = 1 << P.block_shift;
  const bool begins = r0 < P.unit && (r0 & (block - 1)) == 0;
  const float old = begins && u0 + r0 < e0 ? P.scales[(row0 + r0) >> P.block_shift] : 0.f;  // (a block without earlier rows has none)
#pragma unroll
  for (int i = 0; i < kMax; ++i) {
    const int r = warp + kWarps * i;
    if (r < P.unit) {
      int k = -1000;                               // no new row
      if (is_new[i]) {
        const uint32_t w[8] = {a[i].x, a[i].y, a[i].z, a[i].w, c[i].x, c[i].y, c[i].z, c[i].w};
        uint32_t mx = w[0];
#pragma unroll
        for (int v = 1; v < 8; ++v) mx = max_abs_bf16x2(mx, w[v]);
        mx = __reduce_max_sync(0xffffffffu, max(mx & 0x7FFFu, (mx >> 16) & 0x7FFFu));
        const int e = (int)(mx >> 7);              // biased exponent; 448 = 1.75 * 2^8
        k = e == 255 ? 1000 : max(-100, e - 127 - 8 + ((mx & 0x7Fu) > 0x60u ? 1 : 0));
      }
      if (lane == 0) row_k[r] = k;
    }
  }
  __syncthreads();
  // A thread a row of the unit; the first of each block settles its scale.
  if (threadIdx.x < (unsigned)P.unit) {  // (16, 32 or 64 of them: whole half warps)
    const int r = r0;
    const uint32_t in = P.unit < 32 ? 0xFFFFu : 0xffffffffu;
    int k = row_k[r];
    if (block == 64) k = max(k, row_k[r ^ 32]);
    for (int o = min(block, 32) >> 1; o > 0; o >>= 1) k = max(k, __shfl_xor_sync(in, k, o));
    if (begins) {
      float s = k == 1000 ? CUDART_NAN_F : __uint_as_float((uint32_t)(127 + max(k, -100)) << 23);
      if (old != old || old > s) s = old;
      s_old[r >> P.block_shift] = old;
      s_new[r >> P.block_shift] = k == -1000 ? 0.f : s;  // 0: nothing new in the block
    }
  }
  __syncthreads();
  // Nothing is written over another slot's rows. (Looked at here, behind both barriers, the holders have arrived.)
  if (held > 1 && __syncthreads_or(others_page(P, b, lp, page, threadIdx.x, kAppendThreads))) {
    if (threadIdx.x == 0) record_status(P.status, CSA_DEV_BOUNDS);
    return;
  }
  if (begins && s_new[r0 >> P.block_shift] != 0.f) P.scales[(row0 + r0) >> P.block_shift] = s_new[r0 >> P.block_shift];
#pragma unroll
  for (int i = 0; i < kMax; ++i) {
    const int r = warp + kWarps * i;
    if (r >= P.unit) continue;
    const float s = s_new[r >> P.block_shift];
    uint2* dst = reinterpret_cast<uint2*>(P.pages + (row0 + r) * 512);
    if (is_new[i]) {
      const float inv = s == s ? 1.f / s : 0.f;    // exact: s is a power of two
      const uint32_t w[8] = {a[i].x, a[i].y, a[i].z, a[i].w, c[i].x, c[i].y, c[i].z, c[i].w};
      uint16_t h[8];
#pragma unroll
      for (int v = 0; v < 8; ++v) {
        const float x0 = __uint_as_float(w[v] << 16) * inv, x1 = __uint_as_float(w[v] & 0xFFFF0000u) * inv;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(h[v]) : "f"(s == s ? x0 : 0.f), "f"(s == s ? x1 : 0.f));
      }
      dst[lane] = make_uint2(h[0] | ((uint32_t)h[1] << 16), h[2] | ((uint32_t)h[3] << 16));
      dst[32 + lane] = make_uint2(h[4] | ((uint32_t)h[5] << 16), h[6] | ((uint32_t)h[7] << 16));
    } else if (u0 + r < e0 && s > s_old[r >> P.block_shift]) {
      const float f = s_old[r >> P.block_shift] / s;
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        uint2 q = dst[32 * v + lane];
        uint32_t* w = reinterpret_cast<uint32_t*>(&q);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          uint32_t out = 0;
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            uint32_t hh;
            uint16_t cc;
            asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(hh) : "h"((uint16_t)(w[x] >> (16 * y))));
            float lo, hi;
            asm("{.reg .b16 l, h; mov.b32 {l, h}, %2; cvt.f32.f16 %0, l; cvt.f32.f16 %1, h;}" : "=f"(lo), "=f"(hi) : "r"(hh));
            asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(cc) : "f"(lo * f), "f"(hi * f));
            out |= (uint32_t)cc << (16 * y);
          }
          w[x] = out;
        }
        dst[32 * v + lane] = q;
      }
    }
  }
}

template __global__ void cache_append_kernel<2>(AppendParams);
template __global__ void cache_append_kernel<4>(AppendParams);
template __global__ void cache_append_kernel<8>(AppendParams);

// The same for bf16 pages (the index cache): rows of d values copied as they are, a warp a row.
__global__ void __launch_bounds__(kAppendThreads) cache_append_bf16_kernel(AppendParams P) {
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.y, lane = lane_id();
  const int start = P.start_pos[b];
  if (start < 0) return;
  const long long e0 = start / P.ratio, e1 = ((long long)start + P.S) / P.ratio;
  const long long e = e0 + (long long)blockIdx.x * (kAppendThreads / 32) + warp_id();
  if (e >= e1) return;
  const long long lp = e >> P.page_shift;
  const int page = lp < P.max_pages ? P.table[(long long)b * P.max_pages + lp] : -1;
  if (page < 0 || page >= P.num_pages || e >= P.max_rows) {
    if (lane == 0) record_status(P.status, CSA_DEV_BOUNDS);
    return;
  }
  const long long row = ((long long)page << P.page_shift) + (e & ((1 << P.page_shift) - 1));
  const uint4* src = reinterpret_cast<const uint4*>(P.rows + (long long)b * P.rows_bstride + e * P.d);
  uint4* dst = reinterpret_cast<uint4*>(P.pages + row * P.d * 2);
  const int held = P.refs[page];
  uint4 v[2];  // d is at most 512
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (lane + 32 * i < P.d / 8) v[i] = src[lane + 32 * i];
  if (held > 1 && __any_sync(0xffffffffu, others_page(P, b, lp, page, lane, 32))) {
    if (lane == 0) record_status(P.status, CSA_DEV_BOUNDS);
    return;
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (lane + 32 * i < P.d / 8) dst[lane + 32 * i] = v[i];
}

// ------------------------------------------------------------------------------------------------ read

// Rows idx[b][i] of each request as bf16: out[b][i]. A warp a row; -1 leaves the output row as it was. The
// value of an e4m3 row (4 significant bits times a power of two) is exact in bf16. Bound by its three dependent reads
// (index, page, row): B200: 64 x 16 rows 1.9 us, 4 x 2065 rows 4.0.
__global__ void __launch_bounds__(kReadThreads) cache_read_kernel(ReadParams P) {
  pdl_wait();
  pdl_trigger();
  const long long i = (long long)blockIdx.x * (kReadThreads / 32) + warp_id();
  const int lane = lane_id();
  if (i >= (long long)P.B * P.n) return;
  const int e = P.idx[i];
  if (e < 0) return;
  const int b = (int)(i / P.n);
  const int lp = e >> P.page_shift;
  const int page = lp < P.max_pages ? P.table[(long long)b * P.max_pages + lp] : -1;
  if (page < 0 || page >= P.num_pages) {
    if (lane == 0) record_status(P.status, CSA_DEV_BOUNDS);
    return;
  }
  const long long row = ((long long)page << P.page_shift) + (e & ((1 << P.page_shift) - 1));
  uint16_t* out = P.out + i * P.d;
  if (P.scales == nullptr) {
    const uint4* src = reinterpret_cast<const uint4*>(P.pages + row * P.d * 2);
    for (int c = lane; c < P.d / 8; c += 32) reinterpret_cast<uint4*>(out)[c] = src[c];
    return;
  }
  const float s = P.scales[row >> P.block_shift];
  const uint4 q = reinterpret_cast<const uint4*>(P.pages + row * 512)[lane];
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
  uint32_t o[8];
#pragma unroll
  for (int v = 0; v < 8; ++v) {
    uint32_t hh;
    float lo, hi;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(hh) : "h"((uint16_t)(w[v >> 1] >> (16 * (v & 1)))));
    asm("{.reg .b16 l, h; mov.b32 {l, h}, %2; cvt.f32.f16 %0, l; cvt.f32.f16 %1, h;}" : "=f"(lo), "=f"(hi) : "r"(hh));
    asm("cvt.rn.bf16x2.f32 %0, %2, %1;" : "=r"(o[v]) : "f"(lo * s), "f"(hi * s));
  }
  reinterpret_cast<uint4*>(out)[2 * lane] = make_uint4(o[0], o[1], o[2], o[3]);
  reinterpret_cast<uint4*>(out)[2 * lane + 1] = make_uint4(o[4], o[5], o[6], o[7]);
}

// ------------------------------------------------------------------------------------------------ page table
//
// The three table operations are integer scans over the table and the reference counts (64 KB for 64 requests at
// 32K, a few hundred at a million tokens) in one launch. What they cost is latency: the barriers and dependent loads of
// each phase, so loads are issued four at a time, and a cluster's CTAs exchange their sums through shared memory (through global
// memory a reservation took 7.2 us instead of 3.7). Up to kPagesSmall places and pages one CTA is quicker, beyond a
// cluster of 8; B200, back to back: 4 slots x 8 places, 64 pages: reserve 2.6 (cluster: 3.5), fork 5.0 (7.2), compact
// 2.8 (4.5) us; 64 x 32, 2048 pages: 3.3 (3.7), 6.9 (8.5), 3.8 (4.9); 64 x 64, 4096 pages: 4.0 (3.7), 8.9 (9.0), 4.9 (5.1); one CTA
// at 64 x 128, 8192 pages: 6.2, 17.7 and 11.0 against the cluster's 3.9, 9.4 and 5.3 (a fork takes 0.1 more since it looks for
// places without a page). At a million tokens a slot: 8 x 4096 places, 16384 pages: 7.1, 17.2, 9.6; 64 x 4096, 131072 pages: 33.0,
// 92.0, 58.3. What depends on a slot alone is
// worked out first, by every CTA in its own shared memory (S), or for more than kPagesSmallSlots slots once, in the workspace.

// f(i, g(i)) for i = first, first + step, ... below n, with four g under way.
template <typename G, typename F>
__device__ __forceinline__ void batched(unsigned n, unsigned first, unsigned step, G g, F f) {
  for (unsigned i = first; i < n; i += 4 * step) {
    decltype(g(0u)) v[4];
#pragma unroll
    for (unsigned u = 0; u < 4; ++u)
      if (i + u * step < n) v[u] = g(i + u * step);
#pragma unroll
    for (unsigned u = 0; u < 4; ++u)
      if (i + u * step < n) f(i + u * step, v[u]);
  }
}

// Pages for entries[r] entries of every slot: unmapped places below ceil(entries[r] / page_size), in (slot,
// place) order, get the lowest free pages. With fewer free pages than places nothing changes.
template <int C, bool S>
__device__ __forceinline__ void pages_reserve(const PagesParams& P) {
  __shared__ int scan[33], sums[2][3][kPagesCluster];
  __shared__ int s_entries[S ? kPagesSmallSlots : 1];
  if (C > 1) cluster_arrive_relaxed();  // waited for before the first access to another CTA's shared memory
  pdl_wait();
  pdl_trigger();
  const int ps = 1 << P.page_shift, mp = P.max_pages;
  int bad = 0;
  for (unsigned r = threadIdx.x; r < (unsigned)P.slots; r += kPagesThreads) {
    const int e = P.entries[r];
    if (S) s_entries[r] = e;
    if (e < 0 || (long long)e > ((long long)mp << P.page_shift)) bad = 1;
  }
  __syncthreads();
  auto need = [&](int r) -> int {
    const int e = S ? s_entries[r] : P.entries[r];
    return e <= 0 ? 0 : (int)(((long long)e + ps - 1) >> P.page_shift);
  };
  unsigned t0, t1, f0, f1;
  my_run<C>((unsigned)P.slots * mp, t0, t1);
  my_run<C>((unsigned)P.num_pages, f0, f1);
  int want = 0, nfree = 0;
  batched(t1, t0, 1, [&](unsigned i) { return P.table[i]; }, [&](unsigned i, int v) {
    const unsigned r = i / (unsigned)mp;
    if (v < -1 || v >= P.num_pages) bad = 1;
    if (v < 0 && (int)(i - r * mp) < need(r)) ++want;
  });
  batched(f1, f0, 1, [&](unsigned i) { return P.refs[i]; }, [&](unsigned, int v) { nfree += v == 0 ? 1 : 0; });
  int at[3] = {want, nfree, bad}, all[3];
  if (C > 1) cluster_wait();
  all_scan<C>(at, all, scan, sums, 0);
  int w = at[0], f = at[1];
  const int wall = all[0], fall = all[1], ball = all[2];
  if (ball > 0 || wall > fall) {  // the same in every thread
    if (rank<C>() == 0 && threadIdx.x == 0) record_status(P.status, ball > 0 ? CSA_DEV_BOUNDS : CSA_DEV_NO_PAGES);
    return;
  }
  if (wall == 0) return;  // (no CTA touches another's shared memory after the scan's barrier)
  for (unsigned i = f0; i < f1 && f < wall; ++i)
    if (P.refs[i] == 0) {
      P.list_a[f++] = (int)i;
      P.refs[i] = 1;
    }
  all_sync<C>();
  if (want > 0)
    for (unsigned i = t0; i < t1; ++i) {
      const unsigned r = i / (unsigned)mp;
      if ((int)(i - r * mp) < need(r) && P.table[i] < 0) P.table[i] = ld_cg(P.list_a + w++);
    }
}

// Slot r becomes a copy of slot parent[r] (-1: empty, r: unchanged), all slots at once. Pages are shared by
// reference, but for a partly filled last page: rows will be appended to it, so it goes to the lowest of the slots that take
// it over (`heir`, per page) only if nobody else holds it after the call, and the others get fresh pages, which
// pages_copy_kernel fills. (The page copied thus always keeps a holder and is never itself a fresh one.) Nothing is
// committed before the free pages are known to suffice: reference counts, without those of partly filled last pages taken
// over, are worked out in `list_b`, changed rows in `rows`.
template <int C, bool S>
__device__ __forceinline__ void pages_fork(const PagesParams& P) {
  __shared__ int scan[33], sums[2][3][kPagesCluster];
  __shared__ int s_parent[S ? kPagesSmallSlots : 1], s_need[S ? kPagesSmallSlots : 1], s_copy[S ? kPagesSmallSlots : 1];
  __shared__ int s_last[S ? kPagesSmallSlots : 1];
  if (C > 1) cluster_arrive_relaxed();  // waited for before the first access to another CTA's shared memory
  pdl_wait();
  pdl_trigger();
  const unsigned tid = rank<C>() * kPagesThreads + threadIdx.x;
  constexpr unsigned kAll = C * kPagesThreads;
  const int ps = 1 << P.page_shift, cap = P.max_pages << P.page_shift;
  const unsigned cells = (unsigned)P.slots * P.max_pages, mp = P.max_pages;
  // Slots are walked by every CTA where their arrays are its own, by all together otherwise.
  const unsigned s_first = S ? threadIdx.x : tid, s_step = S ? kPagesThreads : kAll;
  int* need = S ? s_need : P.need;    // pages that the slot takes over
  int* copy = S ? s_copy : P.copy;    // the place of its partly filled last page, -1: none; then: if it takes a copy
  int* last = S ? s_last : P.last;    // that page
  auto at = [](int* p, unsigned i) { return S ? p[i] : ld_cg(p + i); };
  auto parent_of = [&](unsigned r) { return S ? s_parent[r] : P.parent[r]; };
  constexpr int kNone = 0x7FFFFFFF;
  // Phase 0: check, copy the counts, clear the heirs.
  int bad = 0;
  for (unsigned r = s_first; r < (unsigned)P.slots; r += s_step) {
    const int p = P.parent[r], e = P.entries[r];
    if (p < -1 || p >= P.slots || e < 0 || e > cap) bad = 1;
    if (S) s_parent[r] = p;
  }
  batched(cells, tid, kAll, [&](unsigned i) { return P.table[i]; }, [&](unsigned, int v) {
    if (v < -1 || v >= P.num_pages) bad = 1;
  });
  batched((unsigned)P.num_pages, tid, kAll, [&](unsigned i) { return P.refs[i]; }, [&](unsigned i, int v) {
    P.list_b[i] = v;
    P.heir[i] = kNone;
  });
  if (tid == 0) *P.n_moves = 0;
  int nbad[1] = {bad}, ball[1];
  if (C > 1) cluster_wait();
  all_scan<C>(nbad, ball, scan, sums, 0);
  if (ball[0] > 0) {
    if (tid == 0) record_status(P.status, CSA_DEV_BOUNDS);
    return;
  }
  // Phase 1: what each slot takes; the lowest heir of each partly filled last page.
  for (unsigned r = s_first; r < (unsigned)P.slots; r += s_step) {
    const int s = parent_of(r);
    int n = 0, c = -1, p = -1;
    if (s >= 0 && s != (int)r) {
      const int e = P.entries[s];
      n = (int)(((long long)e + ps - 1) >> P.page_shift);
      p = (e & (ps - 1)) != 0 ? P.table[s * mp + n - 1] : -1;
      if (p >= 0) {
        c = n - 1;
        if (!S || r % C == rank<C>()) atomicMin(P.heir + p, (int)r);
      }
    }
    need[r] = n;
    copy[r] = c;
    last[r] = p;
  }
  S ? __syncthreads() : all_sync<C>();
  // Phase 2: changed rows and counts. A place without a page among those that are taken over is told by n_moves = -1 (as a third
  // sum of the next scan it cost every call 0.4 us).
  batched(cells, tid, kAll,
          [&](unsigned i) {
            const unsigned r = i / mp, lp = i - r * mp;
            const int s = parent_of(r);
            if (s == (int)r) return make_int2(-1, -1);
            return make_int2(P.table[i], (int)lp < at(need, r) ? P.table[s * mp + lp] : -1);
          },
          [&](unsigned i, int2 v) {  // (what the place held, what it takes over)
            const unsigned r = i / mp, lp = i - r * mp;
            if (parent_of(r) == (int)r) return;
            if (v.x >= 0) atomicAdd(P.list_b + v.x, -1);
            if (v.y < 0 && (int)lp < at(need, r)) *P.n_moves = -1;
            if (v.y >= 0 && at(copy, r) != (int)lp) atomicAdd(P.list_b + v.y, 1);
            P.rows[i] = v.y;
          });
  int want = 0;
  unsigned r0, r1, f0, f1;
  my_run<C>((unsigned)P.slots, r0, r1);
  my_run<C>((unsigned)P.num_pages, f0, f1);
  all_sync<C>();
  const int hole = ld_cg(P.n_moves);
  for (unsigned r = r0; r < r1; ++r) {  // (these slots' `copy` is this thread's from here on)
    const int p = at(last, r);
    if (p < 0) continue;
    if (ld_cg(P.list_b + p) == 0 && ld_cg(P.heir + p) == (int)r) copy[r] = -1;
    else ++want;
  }
  // Phase 3: free pages. A page without holders but with an heir stays with that.
  int nfree = 0;
  auto count = [&](unsigned i) { return make_int2(ld_cg(P.list_b + i), ld_cg(P.heir + i)); };
  batched(f1, f0, 1, count, [&](unsigned, int2 v) { nfree += v.x == 0 && v.y == kNone ? 1 : 0; });
  int at2[2] = {want, nfree}, all2[2];
  all_scan<C>(at2, all2, scan, sums, 1);
  int w = at2[0], f = at2[1];
  const int wall = all2[0], fall = all2[1];
  if (hole < 0 || wall > fall) {  // the same in every thread
    if (tid == 0) {
      *P.n_moves = 0;
      record_status(P.status, hole < 0 ? CSA_DEV_BOUNDS : CSA_DEV_NO_PAGES);
    }
    return;
  }
  batched(f1, f0, 1, count, [&](unsigned i, int2 v) {
    if (v.x == 0 && v.y != kNone) {
      v.x = 1;
    } else if (v.x == 0 && f < wall) {
      P.list_a[f++] = (int)i;
      v.x = 1;
    }
    P.refs[i] = v.x;
  });
  all_sync<C>();
  // Phase 4: the moves and the changed places (the parents' rows are read before any row changes).
  for (unsigned r = r0; r < r1; ++r) {
    const int lp = at(copy, r);
    if (lp < 0) continue;
    const int dst = ld_cg(P.list_a + w);
    P.move_src[w] = at(last, r);
    P.move_dst[w] = dst;
    ++w;
    P.rows[r * mp + lp] = dst;
  }
  if (tid == 0) *P.n_moves = wall;
  all_sync<C>();
  batched(cells, tid, kAll, [&](unsigned i) { return ld_cg(P.rows + i); }, [&](unsigned i, int v) {
    if (parent_of(i / mp) != (int)(i / mp)) P.table[i] = v;
  });
}

// Live pages (refs > 0) move to the front: with L of them, the k-th live page at or behind L goes to the k-th
// free page before L. map[p]: where page p is now (-1: it was free).
template <int C, bool>
__device__ __forceinline__ void pages_compact(const PagesParams& P) {
  __shared__ int scan[33], sums[2][3][kPagesCluster];
  if (C > 1) cluster_arrive_relaxed();  // waited for before the first access to another CTA's shared memory
  pdl_wait();
  pdl_trigger();
  const unsigned tid = rank<C>() * kPagesThreads + threadIdx.x;
  constexpr unsigned kAll = C * kPagesThreads;
  unsigned f0, f1;
  my_run<C>((unsigned)P.num_pages, f0, f1);
  int nlive = 0;
  batched(f1, f0, 1, [&](unsigned i) { return P.refs[i]; }, [&](unsigned, int v) { nlive += v != 0 ? 1 : 0; });
  int at[1] = {nlive}, all[1];
  if (C > 1) cluster_wait();
  all_scan<C>(at, all, scan, sums, 0);
  const int before = at[0], L = all[0];  // live pages before f0, in all
  // Holes (free pages before L), numbered from the front. As many live pages lie at or behind L, and L - 1 - k of
  // them follow page i with k live pages before it, so its number from the front is M - 1 - (L - 1 - k).
  int holes = 0;
  for (int i = (int)f0, k = before; i < (int)f1; ++i) {
    const bool live = P.refs[i] != 0;
    if (!live && i < L) {
      P.list_a[i - k] = i;
      ++holes;
    }
    k += live ? 1 : 0;
  }
  int at1[1] = {holes}, all1[1];
  all_scan<C>(at1, all1, scan, sums, 1);
  const int M = all1[0];
  for (int i = (int)f0, k = before; i < (int)f1; ++i) {
    const bool live = P.refs[i] != 0;
    int to = live ? i : -1;
    if (live && i >= L) {
      const int m = M - 1 - (L - 1 - k);
      to = ld_cg(P.list_a + m);
      P.move_src[m] = i;
      P.move_dst[m] = to;
    }
    P.map[i] = to;
    k += live ? 1 : 0;
  }
  if (tid == 0) {
    *P.n_moves = M;
    *P.live = L;
  }
  all_sync<C>();
  for (int m = tid; m < M; m += kAll) {
    const int src = ld_cg(P.move_src + m), dst = ld_cg(P.move_dst + m);
    P.refs[dst] = P.refs[src];
    P.refs[src] = 0;
  }
  batched((unsigned)P.slots * P.max_pages, tid, kAll,
          [&](unsigned i) {
            const int v = P.table[i];
            return make_int2(v, v >= 0 && v < P.num_pages ? ld_cg(P.map + v) : -1);
          },
          [&](unsigned i, int2 v) {  // (page, where it is now)
            if (v.x == -1) return;
            if (v.y < 0) record_status(P.status, CSA_DEV_BOUNDS);  // a place that maps no live page: left as it is
            else if (v.y != v.x) P.table[i] = v.y;
          });
}

#define CSA_PAGES_KERNELS(name)                                                                                        \
  __global__ void __launch_bounds__(kPagesThreads) name##_kernel(PagesParams P) { name<1, true>(P); }                   \
  __global__ void __cluster_dims__(kPagesCluster, 1, 1) __launch_bounds__(kPagesThreads)                                 \
      name##_cluster_kernel(PagesParams P) {                                                                            \
    if (P.slots <= kPagesSmallSlots) name<kPagesCluster, true>(P);                                                      \
    else name<kPagesCluster, false>(P);                                                                                 \
  }
CSA_PAGES_KERNELS(pages_reserve)
CSA_PAGES_KERNELS(pages_fork)
CSA_PAGES_KERNELS(pages_compact)
#undef CSA_PAGES_KERNELS

// The moves of a fork or a compaction, in every pool: work unit = (move, chunk of a pool's page), 16 bytes a thread
// and load, four loads in flight. Sources and destinations of one call never overlap. Bound by DRAM: a page's bytes
// are read and written once. B200: 4016 pages of 32 KB (half of 16384 live) to the front in 41.3 us, 263 MB read and written at
// 6.4 TB/s, 0.97 of the HBM copy rate (chunks of 8 or 32 KB: 43).
__global__ void __launch_bounds__(kCopyThreads) pages_copy_kernel(CopyParams P) {
  pdl_wait();
  pdl_trigger();
  const int n = *P.n_moves;
  const long long units = (long long)n * P.units_per_page;
  for (long long u = blockIdx.x; u < units; u += gridDim.x) {
    const int m = (int)(u / P.units_per_page);
    int c = (int)(u - (long long)m * P.units_per_page), p = 0;
    while (c >= P.pool[p].units) c -= P.pool[p++].units;
    const PagePool& pool = P.pool[p];
    const long long off = (long long)c * kCopyChunk;
    const int bytes = (int)min((long long)kCopyChunk, (long long)pool.page_bytes - off);
    const uint8_t* src = pool.base + (long long)P.move_src[m] * pool.page_bytes + off;
    uint8_t* dst = pool.base + (long long)P.move_dst[m] * pool.page_bytes + off;
    if (pool.page_bytes % 16 == 0) {
      constexpr int kIn = kCopyChunk / 16 / kCopyThreads;
      uint4 v[kIn];
#pragma unroll
      for (int i = 0; i < kIn; ++i) {
        const int x = 16 * (threadIdx.x + i * kCopyThreads);
        if (x < bytes) v[i] = *reinterpret_cast<const uint4*>(src + x);
      }
#pragma unroll
      for (int i = 0; i < kIn; ++i) {
        const int x = 16 * (threadIdx.x + i * kCopyThreads);
        if (x < bytes) *reinterpret_cast<uint4*>(dst + x) = v[i];
      }
    } else {  // scale pages of fewer than four blocks
      for (int x = 4 * threadIdx.x; x < bytes; x += 4 * kCopyThreads)
        *reinterpret_cast<uint32_t*>(dst + x) = *reinterpret_cast<const uint32_t*>(src + x);
    }
  }
}

}  // namespace csa
