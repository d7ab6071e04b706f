// paged.cu -- caches in pages: entries written into and read out of the pages, and the page table's life
// (reserve, fork / free, compact).
//
// A page table maps each slot (request) to pages of a pool: entry e of slot r is row e % page_size of page
// table[r][e / page_size]; refs[p] counts the table entries (and other holders) of page p, 0: free. Every
// cache laid out behind one table (a layer's main and index entries, every layer of a model) has a pool
// of the same page numbers. All of it lives in device memory and changes in stream order, so a captured decode
// step may contain these calls. Every choice is deterministic: new pages are the lowest free ones, in slot order.

#include <math_constants.h>

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

// Items [lo, hi) of [0, n) that this CTA of the cluster walks, and of those the run of this thread.
__device__ __forceinline__ void my_run(long long n, long long& lo, long long& hi) {
  const long long c = cluster_ctarank();
  const long long a = n * c / kPagesCluster, b = n * (c + 1) / kPagesCluster;
  const long long per = (b - a + blockDim.x - 1) / blockDim.x;
  lo = min(b, a + per * threadIdx.x);
  hi = min(b, lo + per);
}

// Sum of slot `what` of every earlier CTA of the cluster, and of all of them (each published its own before a
// cluster barrier).
__device__ __forceinline__ int cluster_prefix(const int* counts, int what, int& total) {
  int before = 0;
  total = 0;
  const int c = (int)cluster_ctarank();
#pragma unroll
  for (int i = 0; i < kPagesCluster; ++i) {
    const int v = ld_cg(counts + kPagesCluster * what + i);
    before += i < c ? v : 0;
    total += v;
  }
  return before;
}

}  // namespace

// ------------------------------------------------------------------------------------------------ append

// Entries [e0, e1) that a segment of S tokens at start_pos completes, from `rows` into the pages (e4m3).
// A CTA takes one unit of max(block, 16) entries (a block's rows share its scale, and a unit lies inside
// one page); a warp takes a row at a time, 16 dims a lane, and keeps it in registers between the block's maximum
// and the rounding, so every row is read once. Bound by the rows' bytes (1 KB read, 512 B written).
//   scale of a block = the least power of two 2^k with max |x| <= 448 * 2^k over its rows, and never less
//   than before: when new rows raise it, the earlier rows' codes are rounded again to the new step (by an exact
//   power of two; only codes below e4m3's normal range lose bits).
// A power of two costs e4m3 nothing (its steps are relative) and makes every value of the cache
// exact in bf16. A row with a value that is not finite makes its block's scale NaN.
__global__ void __launch_bounds__(kAppendThreads) cache_append_kernel(AppendParams P) {
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
  const int page = lp < P.max_pages ? P.table[(long long)b * P.max_pages + lp] : -1;
  if (page < 0 || page >= P.num_pages) {
    if (threadIdx.x == 0) record_status(P.status, CSA_DEV_BOUNDS);
    return;
  }
  const long long row0 = ((long long)page << P.page_shift) + (u0 & ((1 << P.page_shift) - 1));
  constexpr int kWarps = kAppendThreads / 32, kMax = kAppendMaxUnit / kWarps;
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
#pragma unroll
  for (int i = 0; i < kMax; ++i) {
    const int r = warp + kWarps * i;
    if (r < P.unit) {
      int k = -1000;                               // no new row
      if (is_new[i]) {
        const uint32_t w[8] = {a[i].x, a[i].y, a[i].z, a[i].w, c[i].x, c[i].y, c[i].z, c[i].w};
        uint32_t mx = 0;
#pragma unroll
        for (int v = 0; v < 8; ++v) mx = __vmaxu2(mx, w[v] & 0x7FFF7FFFu);
        mx = max(mx & 0xFFFFu, mx >> 16);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        const int e = (int)(mx >> 7);              // biased exponent; 448 = 1.75 * 2^8
        k = e == 255 ? 1000 : max(-100, e - 127 - 8 + ((mx & 0x7Fu) > 0x60u ? 1 : 0));
      }
      if (lane == 0) row_k[r] = k;
    }
  }
  __syncthreads();
  const int nblk = P.unit >> P.block_shift, block = 1 << P.block_shift;
  if (threadIdx.x < (unsigned)nblk) {
    int k = -1000;
    for (int r = 0; r < block; ++r) k = max(k, row_k[threadIdx.x * block + r]);
    float* sp = P.scales + (row0 >> P.block_shift) + threadIdx.x;
    const float old = u0 + (long long)threadIdx.x * block < e0 ? *sp : 0.f;  // a block without earlier rows has none
    float s = k == 1000 ? CUDART_NAN_F : __uint_as_float((uint32_t)(127 + max(k, -100)) << 23);
    if (old != old || old > s) s = old;
    s_old[threadIdx.x] = old;
    s_new[threadIdx.x] = k == -1000 ? 0.f : s;     // 0: nothing new in the block
    if (k != -1000) *sp = s;
  }
  __syncthreads();
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
  for (int i = lane; i < P.d / 8; i += 32) dst[i] = src[i];
}

// ------------------------------------------------------------------------------------------------ read

// Rows idx[b][i] of each request as bf16: out[b][i]. A warp a row; -1 leaves the output row as it was. The
// value of an e4m3 row (4 significant bits times a power of two) is exact in bf16.
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
// The three table operations are integer scans over the table and the reference counts (a few hundred KB for
// 64 requests at a million tokens): one cluster of 8 CTAs walks them, a contiguous run per thread, with
// cluster barriers between the phases, so an operation on the table is one launch. What they cost is
// latency: the barriers and dependent loads of each phase.

// Pages for entries[r] entries of every slot: unmapped places below ceil(entries[r] / page_size), in (slot,
// place) order, get the lowest free pages. With fewer free pages than places nothing changes.
__global__ void __cluster_dims__(kPagesCluster, 1, 1) __launch_bounds__(kPagesThreads) pages_reserve_kernel(PagesParams P) {
  __shared__ int scan[33];
  pdl_wait();
  pdl_trigger();
  const int ps = 1 << P.page_shift;
  const int c = (int)cluster_ctarank();
  auto need = [&](int r) -> long long {
    const int e = P.entries[r];
    return e <= 0 ? 0 : ((long long)e + ps - 1) >> P.page_shift;
  };
  long long t0, t1, f0, f1;
  my_run((long long)P.slots * P.max_pages, t0, t1);
  my_run(P.num_pages, f0, f1);
  int want = 0, bad = 0;
  for (long long i = t0; i < t1; ++i) {
    const int r = (int)(i / P.max_pages), lp = (int)(i - (long long)r * P.max_pages);
    const long long n = need(r);
    if (lp == 0 && (n > P.max_pages || P.entries[r] < 0)) bad = 1;
    const int v = P.table[i];
    if (v < -1 || v >= P.num_pages) bad = 1;
    if (lp < n && v < 0) ++want;
  }
  int nfree = 0;
  for (long long i = f0; i < f1; ++i) nfree += P.refs[i] == 0 ? 1 : 0;
  int wtot, ftot, btot;
  const int wpos = block_scan(want, scan, wtot);
  const int fpos = block_scan(nfree, scan, ftot);
  block_scan(bad, scan, btot);
  if (threadIdx.x == 0) {
    P.counts[c] = wtot;
    P.counts[kPagesCluster + c] = ftot;
    P.counts[2 * kPagesCluster + c] = btot;
  }
  cluster_sync();
  int wall, fall, ball;
  int w = cluster_prefix(P.counts, 0, wall) + wpos;
  int f = cluster_prefix(P.counts, 1, fall) + fpos;
  cluster_prefix(P.counts, 2, ball);
  if (ball > 0 || wall > fall) {  // the same in every thread
    if (c == 0 && threadIdx.x == 0) record_status(P.status, ball > 0 ? CSA_DEV_BOUNDS : CSA_DEV_NO_PAGES);
    cluster_sync();
    return;
  }
  for (long long i = f0; i < f1 && f < wall; ++i)
    if (P.refs[i] == 0) {
      P.list_a[f++] = (int)i;
      P.refs[i] = 1;
    }
  cluster_sync();
  if (want > 0)
    for (long long i = t0; i < t1; ++i) {
      const int r = (int)(i / P.max_pages), lp = (int)(i - (long long)r * P.max_pages);
      if (lp < need(r) && P.table[i] < 0) P.table[i] = ld_cg(P.list_a + w++);
    }
}

// Slot r becomes a copy of slot parent[r] (-1: empty, r: unchanged), all slots at once. Pages are shared by
// reference, except that of several heirs of a partly filled last page one keeps it (the parent's own slot, else
// the lowest heir) and the others get fresh pages, which pages_copy_kernel fills. Nothing is committed before the
// free pages are known to suffice: reference counts are worked out in `list_b`, changed rows in `rows`.
__global__ void __cluster_dims__(kPagesCluster, 1, 1) __launch_bounds__(kPagesThreads) pages_fork_kernel(PagesParams P) {
  __shared__ int scan[33];
  pdl_wait();
  pdl_trigger();
  const int ps = 1 << P.page_shift;
  const int c = (int)cluster_ctarank();
  const int tid = c * kPagesThreads + threadIdx.x;
  constexpr int kAll = kPagesCluster * kPagesThreads;
  const int cap = P.max_pages << P.page_shift;
  // Phase 0: check, copy the counts, clear the heirs.
  int bad = 0;
  for (int r = tid; r < P.slots; r += kAll) {
    const int p = P.parent[r], e = P.entries[r];
    if (p < -1 || p >= P.slots || e < 0 || e > cap) bad = 1;
    P.heir[r] = 0x7FFFFFFF;
  }
  const long long cells = (long long)P.slots * P.max_pages;
  for (long long i = tid; i < cells; i += kAll) {
    const int v = P.table[i];
    if (v < -1 || v >= P.num_pages) bad = 1;
  }
  for (int i = tid; i < P.num_pages; i += kAll) P.list_b[i] = P.refs[i];
  int btot;
  block_scan(bad, scan, btot);
  if (threadIdx.x == 0) P.counts[c] = btot;
  if (tid == 0) *P.n_moves = 0;
  cluster_sync();
  int ball;
  cluster_prefix(P.counts, 0, ball);
  if (ball > 0) {
    if (tid == 0) record_status(P.status, CSA_DEV_BOUNDS);
    cluster_sync();
    return;
  }
  // Phase 1: the lowest heir of each slot that does not keep itself.
  for (int r = tid; r < P.slots; r += kAll) {
    const int s = P.parent[r];
    if (s >= 0) atomicMin(P.heir + s, s == r ? -1 : r);
  }
  cluster_sync();
  // Slot r takes a copy of its parent's last page?
  auto copies = [&](int r, int& s, int& lp) -> bool {
    s = P.parent[r];
    if (s < 0 || s == r || (P.entries[s] & (ps - 1)) == 0 || ld_cg(P.heir + s) == r) return false;
    lp = P.entries[s] >> P.page_shift;
    return P.table[(long long)s * P.max_pages + lp] >= 0;
  };
  // Phase 2: changed rows and counts.
  for (long long i = tid; i < cells; i += kAll) {
    const int r = (int)(i / P.max_pages), lp = (int)(i - (long long)r * P.max_pages);
    const int s = P.parent[r];
    if (s == r) continue;
    const int was = P.table[i];
    if (was >= 0) atomicAdd(P.list_b + was, -1);
    int now = -1;
    if (s >= 0 && lp < (int)(((long long)P.entries[s] + ps - 1) >> P.page_shift)) {
      now = P.table[(long long)s * P.max_pages + lp];
      int s2, lp2;
      if (now >= 0 && !(copies(r, s2, lp2) && lp2 == lp)) atomicAdd(P.list_b + now, 1);
    }
    P.rows[i] = now;
  }
  int want = 0;
  long long r0, r1, f0, f1;
  my_run(P.slots, r0, r1);
  my_run(P.num_pages, f0, f1);
  for (long long r = r0; r < r1; ++r) {
    int s, lp;
    want += copies((int)r, s, lp) ? 1 : 0;
  }
  int wtot;
  const int wpos = block_scan(want, scan, wtot);
  if (threadIdx.x == 0) P.counts[kPagesCluster + c] = wtot;
  cluster_sync();
  // Phase 3: free pages.
  int nfree = 0, ftot;
  for (long long i = f0; i < f1; ++i) nfree += ld_cg(P.list_b + i) == 0 ? 1 : 0;
  const int fpos = block_scan(nfree, scan, ftot);
  if (threadIdx.x == 0) P.counts[2 * kPagesCluster + c] = ftot;
  cluster_sync();
  int wall, fall;
  int w = cluster_prefix(P.counts, 1, wall) + wpos;
  int f = cluster_prefix(P.counts, 2, fall) + fpos;
  if (wall > fall) {
    if (tid == 0) record_status(P.status, CSA_DEV_NO_PAGES);
    cluster_sync();
    return;
  }
  for (long long i = f0; i < f1; ++i) {
    const int v = ld_cg(P.list_b + i);
    int now = v;
    if (v == 0 && f < wall) {
      P.list_a[f++] = (int)i;
      now = 1;
    }
    P.refs[i] = now;
  }
  cluster_sync();
  // Phase 4: the moves and the changed places (the parents' rows are read before any row changes).
  for (long long r = r0; r < r1; ++r) {
    int s, lp;
    if (!copies((int)r, s, lp)) continue;
    const int dst = ld_cg(P.list_a + w);
    P.move_src[w] = P.table[(long long)s * P.max_pages + lp];
    P.move_dst[w] = dst;
    ++w;
    P.rows[r * P.max_pages + lp] = dst;
  }
  if (tid == 0) *P.n_moves = wall;
  cluster_sync();
  for (long long i = tid; i < cells; i += kAll) {
    const int r = (int)(i / P.max_pages);
    if (P.parent[r] != r) P.table[i] = ld_cg(P.rows + i);
  }
}

// Live pages (refs > 0) move to the front: with L of them, the k-th live page at or behind L goes to the k-th
// free page before L. map[p]: where page p is now (-1: it was free).
__global__ void __cluster_dims__(kPagesCluster, 1, 1) __launch_bounds__(kPagesThreads) pages_compact_kernel(PagesParams P) {
  __shared__ int scan[33];
  pdl_wait();
  pdl_trigger();
  const int c = (int)cluster_ctarank();
  const int tid = c * kPagesThreads + threadIdx.x;
  constexpr int kAll = kPagesCluster * kPagesThreads;
  long long f0, f1;
  my_run(P.num_pages, f0, f1);
  int nlive = 0, ltot;
  for (long long i = f0; i < f1; ++i) nlive += P.refs[i] != 0 ? 1 : 0;
  const int pos = block_scan(nlive, scan, ltot);
  if (threadIdx.x == 0) P.counts[c] = ltot;
  cluster_sync();
  int L;
  const int before = cluster_prefix(P.counts, 0, L) + pos;  // live pages before f0
  // Holes (free pages before L), numbered from the front. As many live pages lie at or behind L, and L - 1 - k of
  // them follow page i with k live pages before it, so its number from the front is M - 1 - (L - 1 - k).
  int holes = 0;
  for (long long i = f0, k = before; i < f1; ++i) {
    const bool live = P.refs[i] != 0;
    if (!live && i < L) {
      P.list_a[i - k] = (int)i;
      ++holes;
    }
    k += live ? 1 : 0;
  }
  int htot;
  block_scan(holes, scan, htot);
  if (threadIdx.x == 0) P.counts[kPagesCluster + c] = htot;
  cluster_sync();
  int M;
  cluster_prefix(P.counts, 1, M);
  for (long long i = f0, k = before; i < f1; ++i) {
    const bool live = P.refs[i] != 0;
    int to = live ? (int)i : -1;
    if (live && i >= L) {
      const int m = M - 1 - (int)(L - 1 - k);
      to = ld_cg(P.list_a + m);
      P.move_src[m] = (int)i;
      P.move_dst[m] = to;
    }
    P.map[i] = to;
    k += live ? 1 : 0;
  }
  if (tid == 0) {
    *P.n_moves = M;
    *P.live = L;
  }
  cluster_sync();
  for (int m = tid; m < M; m += kAll) {
    const int src = ld_cg(P.move_src + m), dst = ld_cg(P.move_dst + m);
    P.refs[dst] = P.refs[src];
    P.refs[src] = 0;
  }
  const long long cells = (long long)P.slots * P.max_pages;
  for (long long i = tid; i < cells; i += kAll) {
    const int v = P.table[i];
    if (v == -1) continue;
    const int to = v >= 0 && v < P.num_pages ? ld_cg(P.map + v) : -1;
    if (to < 0) record_status(P.status, CSA_DEV_BOUNDS);  // a place that maps no live page: left as it is
    else if (to != v) P.table[i] = to;
  }
}

// The moves of a fork or a compaction, in every pool: work unit = (move, chunk of a pool's page), 16 bytes a thread
// and load, four loads in flight. Sources and destinations of one call never overlap. Bound by DRAM: a page's bytes
// are read and written once.
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
