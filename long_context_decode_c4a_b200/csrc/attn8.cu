// attn8.cu -- sparse MQA with a learned sink and inverse RoPE over a cache held in 8 bits, in pages.
//
// For query t of request b and head h, over the window rows (bf16, ring) and the compressed entries
// (e4m3 codes c_j in pages, one power-of-two scale s_j for each block of entries):
//   l_j = scale * q_h . (s_j c_j),  m = max(max_j l_j, sink_h),
//   o_h = sum_j e^(l_j - m) s_j c_j / (sum_j e^(l_j - m) + e^(sink_h - m)), then rotate o_h[448:] by -t.
// The entries are the query's selected ones (list form) or every visible one (range form).
//
// The cached bytes go to the tensor cores as they are (tcgen05.mma kind::f8f6f4, both operands e4m3);
// what meets them is split into e4m3 pieces instead of the cache being widened to bf16:
//   q_h = 2^k_h (q1 + q2): q1 is q_h 2^-k_h (largest element in (224, 448]) rounded to e4m3 (4 significant bits),
//     q2 the remainder in e5m2. A bf16 value has 8 significant bits, so the remainder of rounding to 4 is at most 8
//     units of the last: 3 bits hold it. q1 + q2 is exact down to 2^-14 of the head's largest element (where q1
//     becomes subnormal), and off by at most 2^-21 of the largest below.
//   A window row is split the same way, c = 2^k (c1 + c2), both e4m3 (they are rows of one tile: 32 candidates
//     a tile); exact down to 2^-10 of the row's largest element, off by at most 2^-17 of it below. Its score is the
//     sum of the two columns, its P stands in both.
//   P = p1 + p2: p1 is P rounded to e4m3 (4 significant bits), p2 the remainder rounded to e5m2 (3 bits), so
//     P is off by at most 2^-8 of itself (p1 leaves 2^-4, p2 leaves 2^-4 of that: a step below a bf16 P's
//     2^-9), or by 2^-22 of the row's running maximum where that is more: e5m2's smallest step is 2^-7 of
//     e4m3's, which keeps a long flat tail behind one large weight (an e4m3 p2 would round each weight below
//     2^-15 of the maximum to nothing; thousands of entries of that size are a weight to be counted).
// P carries the scale of its column (O += (p_j s_j) c_j), so the running maximum is that of
// y_j = l_j + log2 s_j; the denominator takes P back to p_j with 1 / s_j. The sink enters at the end
// only: it must not push P below e4m3's range.
//
// Layout: two CTAs per query; CTA `half` accumulates O[:, 256 half .. 256 half + 256) (128 heads x 256
// columns of fp32 are half of TMEM) and computes the scores over all 512 dims itself. Both CTAs so gather
// whole rows: 512 bytes, as many as the half row of a bf16 cache, and no partial score crosses the pair.
//   TMEM (512 columns): [0,128) q1 (four e4m3 values a column); [128,192) and [192,256) two 64-column
//     score tiles, whose first 32 columns P (p1, then p2) takes over; [256,512) O.
//   SMEM: four 32 KB stages of 64 rows (four 128-byte blocks in the 128B-swizzled layout, which serves the
//     scores as a K-major and PV as an MN-major operand); q2 (64 KB); the candidate list.
//   Warps: 0..3 build the list, split window rows and gather entries (16-byte cp.async, a warp covering
//     one row an instruction); 4 and 5 issue the score MMAs of even and odd tiles, 6 the PV MMAs (and owns
//     TMEM); 7..10 and 11..14 are the softmax groups of even and odd tiles, one head (TMEM lane) a
//     thread; both first split q, and share the epilogue.
// Split-candidate mode (few queries): as in attn.cu; attn_combine_kernel merges the partials.

#include <cuda_fp16.h>
#include <math_constants.h>

#include <cstddef>

#include "attn_util.cuh"
#include "kernels.cuh"
#include "ptx.cuh"
#include "rope.cuh"

namespace csa {

namespace {

constexpr int kProd = 128;                      // warps 0..3
constexpr int kQkWarp = 4;                      // warps 4, 5
constexpr int kPvWarp8 = 6;
constexpr int kSoftWarp = 7;                    // warps 7..10 (even tiles), 11..14 (odd tiles)
constexpr int kGroup = 128;                     // threads of a softmax group
constexpr int kRows = 64;                       // rows of a tile
constexpr int kWinRows = 32;                    // window candidates of a tile (two rows each)
constexpr int kStages8 = 4;
constexpr uint32_t kBlk = kRows * 128;          // one 128-dim block of a stage
constexpr uint32_t kStage = 4 * kBlk;           // 32 KB
constexpr uint32_t kQBlk = 128 * 128;           // one 128-dim block of a q piece
constexpr uint32_t kQ2Bytes = 4 * kQBlk;        // 64 KB
constexpr uint32_t kRowPitch = 512 + 16;        // output staging: 256 bf16 dims, padded against bank conflicts
// P is formed relative to 2^(m + kHead): a later row may exceed the maximum that P refers to by 2^kHead
// before O is rescaled, and P (at most 1 = e4m3 code value 256 after the shift by 2^8) stays in range.
constexpr float kHead = 3.f;
static_assert(kAttn8Threads == 32 * (kSoftWarp + 8), "warp roles");

struct Smem8 {
  uint64_t kv_full[kStages8], kv_free[kStages8];
  uint64_t s_full[2];      // scores of tile j written (score tile j % 2)
  uint64_t s_free[2];      // PV(j) completed: score tile j % 2 (scores, then P) is free, O holds PV(0..j)
  uint64_t p_full[2];      // P of tile j stored
  uint64_t q_done;         // q1 is in TMEM, q2 in shared memory, the staging area (stages 2, 3) is free
  uint64_t list_ready;
  uint64_t hand[2][4];     // softmax group g published the running maximum after its tile (quadrant q)
  uint64_t drain[3];
  uint32_t tmem_base;
  int abort_flag, bad, epi_bad;
  int n_tiles, tile0, win_tiles;
  uint32_t scan[kProd / 32];
  float rope_cs[kMaxRopePairs][2];
  float qf[128];           // per head: 2^k_h * scale * log2(e)
  float m_hand[4][32];
  float l_g[2][128], m_g[2][128];
  float scale[kStages8][kRows];                       // the rows' scales, as gathered
  alignas(16) float col_a[8][kRows], col_k[8][kRows], col_i[8][kRows];  // (read four at a time) per softmax warp: s_j, log2 s_j, 1 / s_j of its tile's columns
  int32_t list[kAttnMaxTopk];                         // list form: pool rows of the selected entries
};

static_assert(offsetof(Smem8, col_a) % 16 == 0 && sizeof(Smem8::col_a[0]) % 16 == 0, "float4 reads of the column factors");

// 8-bit pieces of two fp32 values (|x| <= 448): hi in e4m3, the remainder lo in e5m2 or e4m3. Through fp16, which
// holds every bf16 value scaled into e4m3's range exactly (below 2^-14: to 2^-25).
template <bool kLoE5M2>
__device__ __forceinline__ void split_fp8x2(float x0, float x1, uint16_t& hi, uint16_t& lo) {
  uint32_t h, back, r;
  asm("cvt.rn.f16x2.f32 %0, %2, %1;" : "=r"(h) : "f"(x0), "f"(x1));
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(hi) : "r"(h));
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(back) : "h"(hi));
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(h), "r"(back));
  if (kLoE5M2) asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(lo) : "r"(r));
  else asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(lo) : "r"(r));
}

// Split of a 512-dim bf16 row held by a warp: lane l has dims [8 l, 8 l + 8) in a and [256 + 8 l, ...) in b.
// Returns 2^k with max |x| <= 448 * 2^k (k >= -100), or NaN (and zero pieces) if a value is not finite.
struct RowPieces {
  uint2 hi[2], lo[2];
};
template <bool kLoE5M2>
__device__ __forceinline__ float split_row(const uint4& a, const uint4& b, RowPieces& out) {
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  uint32_t mx = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) mx = __vmaxu2(mx, w[i] & 0x7FFF7FFFu);
  mx = max(mx & 0xFFFFu, mx >> 16);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  const int e = (int)(mx >> 7);  // biased exponent of the largest magnitude; 448 = 1.75 * 2^8, 0x60 / 128 = 0.75
  const int k = max(-100, e - 127 - 8 + ((mx & 0x7Fu) > 0x60u ? 1 : 0));
  const bool fin = e < 255;
  const float inv = fin ? __uint_as_float((uint32_t)(127 - k) << 23) : 0.f;
  uint16_t h[8], l[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float x0 = __uint_as_float(w[i] << 16), x1 = __uint_as_float(w[i] & 0xFFFF0000u);
    split_fp8x2<kLoE5M2>(fin ? x0 * inv : 0.f, fin ? x1 * inv : 0.f, h[i], l[i]);
  }
#pragma unroll
  for (int v = 0; v < 2; ++v) {
    out.hi[v] = make_uint2(h[4 * v] | ((uint32_t)h[4 * v + 1] << 16), h[4 * v + 2] | ((uint32_t)h[4 * v + 3] << 16));
    out.lo[v] = make_uint2(l[4 * v] | ((uint32_t)l[4 * v + 1] << 16), l[4 * v + 2] | ((uint32_t)l[4 * v + 3] << 16));
  }
  return fin ? __uint_as_float((uint32_t)(127 + k) << 23) : CUDART_NAN_F;
}

// Store lane l's 8 + 8 codes of row `row` into a [4 blocks][rows][128 B] swizzled region of block size `blk`.
__device__ __forceinline__ void store_codes(uint8_t* base, uint32_t blk, int row, int lane, const uint2 (&v)[2]) {
  const uint32_t off = sw128_offset((uint32_t)row, (uint32_t)((lane & 15) >> 1)) + (uint32_t)(lane & 1) * 8u;
#pragma unroll
  for (int i = 0; i < 2; ++i)
    *reinterpret_cast<uint2*>(base + (uint32_t)(2 * i + (lane >> 4)) * blk + off) = v[i];
}

// 2^8 (a - b) of two fp16 pairs; exact where the difference is.
__device__ __forceinline__ uint32_t rest2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(r), "r"(0x5C005C00u));
  return r;
}

// P (fp32 in [0, 1], standing for 2^8 P in 8-bit units) to its two pieces, four columns at a time. An fp16
// value below 2 shifted right by 7 is the e4m3 code of 2^8 times it (same mantissa alignment, exponent
// biases 15 and 7), subnormals included: p1 is the code of P rounded at that bit. The remainder is exact in
// fp16; the upper byte of an fp16 value is its e5m2 code, rounded by adding half a step of the lower byte.
__device__ __forceinline__ void split_p(const float* p, uint32_t& p1, uint32_t& p2) {
  uint32_t h0, h1;
  asm("cvt.rn.f16x2.f32 %0, %2, %1;" : "=r"(h0) : "f"(p[0]), "f"(p[1]));
  asm("cvt.rn.f16x2.f32 %0, %2, %1;" : "=r"(h1) : "f"(p[2]), "f"(p[3]));
  const uint32_t a0 = (h0 + 0x00400040u) & 0xFF80FF80u, a1 = (h1 + 0x00400040u) & 0xFF80FF80u;
  const uint32_t r0 = rest2(h0, a0) + 0x00800080u, r1 = rest2(h1, a1) + 0x00800080u;
  p1 = __byte_perm(a0 >> 7, a1 >> 7, 0x6420);
  p2 = __byte_perm(r0, r1, 0x7531);
}

}  // namespace

__global__ void __launch_bounds__(kAttn8Threads, 1) attn8_kernel(Attn8Params P) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* stages = base;
  uint8_t* q2 = base + kStages8 * kStage;
  uint8_t* q1s = stages + 2 * kStage;            // q1 on its way to TMEM: stages 2 and 3
  Smem8& sm = *reinterpret_cast<Smem8*>(q2 + kQ2Bytes);

  const int warp = warp_id(), lane = lane_id();
  const int half = blockIdx.x & 1;
  const int nq = P.B * P.S;
  const int item = nq * P.splits - 1 - (int)(blockIdx.x >> 1);  // later queries (more candidates) first
  const int qi = item / P.splits, sp = item % P.splits, b = qi / P.S;
  volatile int* abort_flag = &sm.abort_flag;
  uint32_t* status = P.status;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages8; ++i) {
      mbar_init(&sm.kv_full[i], kProd);
      mbar_init(&sm.kv_free[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.s_full[i], 1);
      mbar_init(&sm.s_free[i], 1);
      mbar_init(&sm.p_full[i], kGroup);
      for (int q = 0; q < 4; ++q) mbar_init(&sm.hand[i][q], 32);
    }
    mbar_init(&sm.q_done, 2 * kGroup);
    mbar_init(&sm.list_ready, 1);
    for (int i = 0; i < 3; ++i) mbar_init(&sm.drain[i], 1);
    sm.abort_flag = 0;
    sm.bad = 0;
    sm.epi_bad = 0;
    fence_mbar_init();
  }
  if (warp == kPvWarp8) {
    tmem_alloc(&sm.tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  pdl_wait();
  pdl_trigger();
  const int t = P.q_pos[qi];
  // A negative position marks a padding query: it has no candidates and its output is zero.
  const int nwin = t < 0 ? 0 : (t < P.window ? t + 1 : P.window);
  const int p0 = t - nwin + 1;
  const int Tw = (nwin + kWinRows - 1) / kWinRows;
  const int ecap = t < 0 ? 0 : min((int)(((long long)t + 1) / P.ratio), P.max_entries);

  if (warp < kProd / 32) {
    // ------------------------------------------------------------ candidate list, window split, gathers
    const int pt = threadIdx.x;
    const int32_t* table = P.table + (long long)b * P.max_pages;
    const uint16_t* ring = P.ring + (long long)b * P.ring_bstride;
    bool bad = false;
    // Pool row of entry e (0 <= e < ecap), or -1 when its page is not mapped.
    auto pool_row = [&](int e) -> int {
      const int pg = table[e >> P.page_shift];
      if (pg < 0 || pg >= P.num_pages) {
        bad = true;
        return -1;
      }
      return (pg << P.page_shift) | (e & ((1 << P.page_shift) - 1));
    };
    // Window tile w of the query into `stage`: candidate r of the tile in rows r and r + 32.
    auto window_tile = [&](int w, int stage) {
      uint8_t* st = stages + (size_t)stage * kStage;
#pragma unroll 1
      for (int r0 = 0; r0 < 8; r0 += 4) {
        uint4 a[4], c[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = 8 * warp + r0 + i, k = w * kWinRows + r;
          a[i] = c[i] = make_uint4(0, 0, 0, 0);
          if (k < nwin) {
            const uint4* src = reinterpret_cast<const uint4*>(ring + (long long)((p0 + k) % P.ring_cap) * 512);
            a[i] = src[lane];
            c[i] = src[32 + lane];
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = 8 * warp + r0 + i;
          RowPieces pc;
          const float s = split_row<false>(a[i], c[i], pc);
          store_codes(st, kBlk, r, lane, pc.hi);
          store_codes(st, kBlk, r + kWinRows, lane, pc.lo);
          if (lane == 0) sm.scale[stage][r] = sm.scale[stage][r + kWinRows] = (w * kWinRows + r < nwin) ? s : 0.f;
        }
      }
      fence_proxy_async_smem();
      mbar_arrive(&sm.kv_full[stage]);
    };
    // One pair per query: its first two tiles (stages 0 and 1) are window tiles and need no list.
    int done = 0;
    if (P.splits == 1)
      for (; done < min(Tw, 2); ++done) window_tile(done, done);

    int n;  // entries
    if (P.topk_idx != nullptr) {
      // Each thread takes a contiguous run of the selection; runs are compacted in order.
      const int32_t* sel = P.topk_idx + (long long)qi * P.topk;
      const int per = (P.topk + kProd - 1) / kProd;
      const int lo = min(P.topk, pt * per), hi = min(P.topk, lo + per);
      int rows[kAttnMaxTopk / kProd];
      uint32_t cnt = 0;
#pragma unroll
      for (int u = 0; u < kAttnMaxTopk / kProd; ++u) {
        const int j = lo + u;
        const int s = (u < per && j < hi) ? sel[j] : -1;
        bad |= s >= ecap;
        rows[u] = (s >= 0 && s < ecap) ? s : -1;
      }
#pragma unroll
      for (int u = 0; u < kAttnMaxTopk / kProd; ++u) {
        if (rows[u] >= 0) rows[u] = pool_row(rows[u]);
        cnt += rows[u] >= 0 ? 1u : 0u;
      }
      uint32_t inc = cnt;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
      }
      if (lane == 31) sm.scan[warp] = inc;
      named_bar_sync(2, kProd);
      uint32_t pos = inc - cnt, total = 0;
#pragma unroll
      for (int i = 0; i < kProd / 32; ++i) {
        pos += i < warp ? sm.scan[i] : 0u;
        total += sm.scan[i];
      }
#pragma unroll
      for (int u = 0; u < kAttnMaxTopk / kProd; ++u)
        if (rows[u] >= 0) sm.list[pos++] = rows[u];
      n = (int)total;
    } else {
      n = ecap;
      bad = t >= 0 && ((long long)t + 1) / P.ratio > P.max_entries;
    }
    const int Jq = Tw + (n + kRows - 1) / kRows;
    const int tile0 = (int)(((long long)Jq * sp) / P.splits);
    const int J = (int)(((long long)Jq * (sp + 1)) / P.splits) - tile0;
    named_bar_sync(2, kProd);  // the list is complete
    if (pt == 0) {
      sm.n_tiles = J;
      sm.tile0 = tile0;
      sm.win_tiles = Tw;
      mbar_arrive(&sm.list_ready);
    }

    // Lane i < 16 of a warp holds the pool row of the tile's row warp + 4 i, fetched one tile ahead.
    auto fetch = [&](int j) -> int {
      const int k = (tile0 + j - Tw) * kRows + warp + 4 * (lane & 15);
      if (j >= J || tile0 + j < Tw || k >= n) return -1;
      return P.topk_idx != nullptr ? sm.list[k] : pool_row(k);
    };
    int next_row = fetch(done);
    for (int j = done; j < J; ++j) {
      const int stage = j & (kStages8 - 1);
      if (j >= kStages8) {
        if (!mbar_wait(&sm.kv_free[stage], (uint32_t)((j / kStages8 - 1) & 1), abort_flag, status, 302)) break;
      } else if (j >= 2) {
        if (!mbar_wait(&sm.q_done, 0, abort_flag, status, 301)) break;
      }
      const int my_row = next_row;
      next_row = fetch(j + 1);
      if (tile0 + j < Tw) {
        window_tile(tile0 + j, stage);
        continue;
      }
      const uint32_t st = smem_u32(stages + (size_t)stage * kStage) + (uint32_t)(lane >> 3) * kBlk;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int row = __shfl_sync(0xffffffffu, my_row, i);
        cp_async_16_zfill(st + sw128_offset((uint32_t)(warp + 4 * i), (uint32_t)(lane & 7)),
                          P.pages + (long long)max(row, 0) * 512 + lane * 16, row >= 0);
      }
      if (lane < 16)
        cp_async_4_zfill(smem_u32(&sm.scale[stage][warp + 4 * lane]), P.scales + (max(my_row, 0) >> P.block_shift),
                         my_row >= 0);
      cp_async_arrive_noinc(&sm.kv_full[stage]);
    }
    cp_async_wait_all();  // after an abort: let the copies land before teardown
    if (bad && half == 0) record_status(status, CSA_DEV_BOUNDS);
  } else if (warp < kPvWarp8) {
    // ------------------------------------------------------------ score MMAs: tiles j = w, w + 2, ...
    if (lane == 0) {
      const int w = warp - kQkWarp;
      const bool ok = mbar_wait(&sm.q_done, 0, abort_flag, status, 311) &&
                      mbar_wait(&sm.list_ready, 0, abort_flag, status, 312);
      const int J = ok ? sm.n_tiles : 0;
      const uint32_t idesc1 = idesc_fp8_f32(kE4M3, kE4M3, 128, kRows, 0, 0);
      const uint32_t idesc2 = idesc_fp8_f32(kE5M2, kE4M3, 128, kRows, 0, 0);
      const uint32_t qa = smem_u32(q2), d_s = tmem + 128 + kRows * w;
      for (int j = w; j < J; j += 2) {
        const int stage = j & (kStages8 - 1);
        if (j >= 2 && !mbar_wait(&sm.s_free[w], (uint32_t)((j / 2 - 1) & 1), abort_flag, status, 313)) break;
        if (!mbar_wait(&sm.kv_full[stage], (uint32_t)((j / kStages8) & 1), abort_flag, status, 314)) break;
        fence_proxy_async_smem();  // rows written by cp.async before the MMAs read them
        tc_fence_after();
        const uint32_t kb = smem_u32(stages + (size_t)stage * kStage);
#pragma unroll
        for (int ks = 0; ks < 16; ++ks)
          mma8_ts(d_s, tmem + 8 * ks, smem_desc_sw128(kb + (ks >> 2) * kBlk + (ks & 3) * 32, 16, 1024), idesc1,
                  ks > 0 ? 1u : 0u);
#pragma unroll
        for (int ks = 0; ks < 16; ++ks)
          mma8_ss(d_s, smem_desc_sw128(qa + (ks >> 2) * kQBlk + (ks & 3) * 32, 16, 1024),
                  smem_desc_sw128(kb + (ks >> 2) * kBlk + (ks & 3) * 32, 16, 1024), idesc2, 1u);
        mma_commit(&sm.s_full[w]);
      }
      // Every MMA issued above completes on its own; wait for them before TMEM is released.
      mma_commit(&sm.drain[w]);
      mbar_wait_drain(&sm.drain[w], 0, status, 315);
    }
  } else if (warp == kPvWarp8) {
    // ------------------------------------------------------------ PV MMAs, in tile order
    if (lane == 0) {
      const int J = mbar_wait(&sm.list_ready, 0, abort_flag, status, 321) ? sm.n_tiles : 0;
      const uint32_t idesc[2] = {idesc_fp8_f32(kE4M3, kE4M3, 128, 256, 0, 1), idesc_fp8_f32(kE5M2, kE4M3, 128, 256, 0, 1)};
      for (int j = 0; j < J; ++j) {
        const int stage = j & (kStages8 - 1), g = j & 1;
        if (!mbar_wait(&sm.p_full[g], (uint32_t)((j / 2) & 1), abort_flag, status, 322)) break;
        fence_proxy_async_smem();
        tc_fence_after();
        const uint32_t vb = smem_u32(stages + (size_t)stage * kStage) + (uint32_t)half * 2 * kBlk;
        const uint32_t pc = tmem + 128 + kRows * g;
#pragma unroll
        for (int part = 0; part < 2; ++part)
#pragma unroll
          for (int ks = 0; ks < 2; ++ks)
            mma8_ts(tmem + 256, pc + 16 * part + 8 * ks, smem_desc_sw128(vb + ks * 4096, kBlk, 1024), idesc[part],
                    (j > 0 || part > 0 || ks > 0) ? 1u : 0u);
        mma_commit(&sm.kv_free[stage]);
        mma_commit(&sm.s_free[g]);
      }
      mma_commit(&sm.drain[2]);
      mbar_wait_drain(&sm.drain[2], 0, status, 323);
    }
  } else {
    // ------------------------------------------------------------ q split, softmax, epilogue
    const int sw = warp - kSoftWarp;           // 0..7
    const int g = sw >> 2;                     // softmax group
    const int quad = warp & 3;                 // TMEM lane quadrant
    const int h = quad * 32 + lane;            // head = TMEM lane
    const uint32_t lane_addr = (uint32_t)(quad * 32) << 16;
    // q rows 16 sw .. 16 sw + 15, eight in flight.
#pragma unroll 1
    for (int r0 = 0; r0 < 16; r0 += 8) {
      uint4 a[8], c[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = 16 * sw + r0 + i;
        a[i] = c[i] = make_uint4(0, 0, 0, 0);
        if (r < P.H) {
          const uint4* src = reinterpret_cast<const uint4*>(P.q + ((long long)qi * P.H + r) * 512);
          a[i] = src[lane];
          c[i] = src[32 + lane];
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = 16 * sw + r0 + i;
        RowPieces pc;
        const float f = split_row<true>(a[i], c[i], pc);
        store_codes(q1s, kQBlk, r, lane, pc.hi);
        store_codes(q2, kQBlk, r, lane, pc.lo);
        if (lane == 0) sm.qf[r] = f * P.scale_log2;
      }
    }
    // Inverse-RoPE table for position t.
    const int st = threadIdx.x - kSoftWarp * 32;  // 0..255
    if (st < P.rope_dim / 2) {
      float cs, sn;
      rope_cos_sin(t, P.inv_freq[st], &cs, &sn);
      sm.rope_cs[st][0] = cs;
      sm.rope_cs[st][1] = -sn;
    }
    fence_proxy_async_smem();  // q2 before the MMAs read it
    named_bar_sync(1, 2 * kGroup);
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {  // q1 -> TMEM: group g brings blocks 2 g and 2 g + 1
      const int kb = 2 * g + kk;
      uint32_t r[32];
#pragma unroll
      for (int ch = 0; ch < 8; ++ch) {
        const uint4 v = *reinterpret_cast<const uint4*>(q1s + kb * kQBlk + sw128_offset(h, ch));
        r[4 * ch + 0] = v.x;
        r[4 * ch + 1] = v.y;
        r[4 * ch + 2] = v.z;
        r[4 * ch + 3] = v.w;
      }
      tmem_st32(tmem + lane_addr + 32 * kb, r);
    }
    tmem_wait_st();
    tc_fence_before();
    mbar_arrive(&sm.q_done);

    bool ok = __all_sync(0xffffffffu, mbar_wait(&sm.list_ready, 0, abort_flag, status, 331));
    const int J = ok ? sm.n_tiles : 0;
    const int tile0 = sm.tile0;
    const float qf = sm.qf[h];
    // s_free[i % 2] completes once per PV(i). A wait for PV(i) by parity is unambiguous while PV(i - 2) is
    // known to have completed and PV(i + 2) cannot have: scores of tile j exist only after PV(j - 2), and
    // PV(j + 1) needs the maximum that the group of tile j has not yet published.
    auto wait_pv = [&](int i) -> bool {
      return i < 0 || __all_sync(0xffffffffu, mbar_wait(&sm.s_free[i & 1], (uint32_t)((i / 2) & 1), abort_flag, status, 332));
    };
    float m_used = -CUDART_INF_F, l = 0.f;
    for (int j = g; j < J; j += 2) {
      const int stage = j & (kStages8 - 1);
      const bool win = tile0 + j < Tw;
      // Column factors, two columns a lane, while the score MMAs run. A window candidate's second column
      // adds nothing to the denominator.
      if (!__all_sync(0xffffffffu, mbar_wait(&sm.kv_full[stage], (uint32_t)((j / kStages8) & 1), abort_flag, status, 333))) {
        ok = false;
        break;
      }
      __syncwarp();  // the last tile's factors have been read
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int c = 32 * i + lane;
        const float s = sm.scale[stage][c];
        sm.col_a[sw][c] = s;
        sm.col_k[sw][c] = log2f(s);  // 0 (a masked column): -inf
        sm.col_i[sw][c] = (s == 0.f || (win && c >= kWinRows)) ? 0.f : 1.f / s;
      }
      __syncwarp();
      if (!__all_sync(0xffffffffu, mbar_wait(&sm.s_full[g], (uint32_t)((j / 2) & 1), abort_flag, status, 334))) {
        ok = false;
        break;
      }
      tc_fence_after();
      const uint32_t s_addr = tmem + lane_addr + 128 + kRows * g;
      float y[kRows];
      {
        uint32_t v0[32], v1[32];
        tmem_ld32(s_addr, v0);
        tmem_ld32(s_addr + 32, v1);
        tmem_wait_ld();
        if (win) {
#pragma unroll
          for (int c = 0; c < 32; ++c) y[c] = y[c + 32] = __uint_as_float(v0[c]) + __uint_as_float(v1[c]);
        } else {
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            y[c] = __uint_as_float(v0[c]);
            y[c + 32] = __uint_as_float(v1[c]);
          }
        }
      }
      float mx[4] = {-CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F};
#pragma unroll
      for (int c = 0; c < kRows; c += 4) {
        const float4 a = *reinterpret_cast<const float4*>(&sm.col_a[sw][c]);
        const float4 k = *reinterpret_cast<const float4*>(&sm.col_k[sw][c]);
        y[c] = fmaf(y[c] * qf, a.x, k.x);
        y[c + 1] = fmaf(y[c + 1] * qf, a.y, k.y);
        y[c + 2] = fmaf(y[c + 2] * qf, a.z, k.z);
        y[c + 3] = fmaf(y[c + 3] * qf, a.w, k.w);
#pragma unroll
        for (int e = 0; e < 4; ++e) mx[e] = fmaxf(mx[e], y[c + e]);
      }
      const float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
      // The running maximum after tile j - 1, from the other group (it only grows).
      if (j > 0) {
        if (!__all_sync(0xffffffffu, mbar_wait(&sm.hand[1 - g][quad], (uint32_t)(((j - 1) / 2) & 1), abort_flag, status, 335))) {
          ok = false;
          break;
        }
        const float mp = sm.m_hand[quad][lane];
        if (mp != m_used) {
          l = l != 0.f ? l * exp2f(m_used - mp) : 0.f;
          m_used = mp;
        }
      }
      // Lazy rescale; the TMEM accesses are warp-collective, so the warp takes the branch if any lane must.
      const bool need = mt > m_used + kHead || (m_used == -CUDART_INF_F && mt > m_used);
      if (__any_sync(0xffffffffu, need)) {
        const float alpha = need ? exp2f(m_used - mt) : 1.f;
        if (j > 0) {
          if (!wait_pv(j - 1)) {
            ok = false;
            break;
          }
          tc_fence_after();
#pragma unroll 1
          for (int cc = 0; cc < 16; ++cc) {
            uint32_t o[16];
            const uint32_t oa = tmem + lane_addr + 256 + 16 * cc;
            tmem_ld16(oa, o);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
            tmem_st16(oa, o);
          }
          tmem_wait_st();
          tc_fence_before();
        }
        if (need) {
          l *= alpha;
          m_used = mt;
        }
      }
      if (j + 1 < J) {
        sm.m_hand[quad][lane] = m_used;
        mbar_arrive(&sm.hand[g][quad]);
      }
      const float ref = (m_used == -CUDART_INF_F ? 0.f : m_used) + kHead;
      uint32_t p1[16], p2[16];
      float ls[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < kRows; c += 4) {
        const float4 ki = *reinterpret_cast<const float4*>(&sm.col_i[sw][c]);
        float p[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) p[e] = ex2_approx(y[c + e] - ref);
        ls[0] = fmaf(p[0], ki.x, ls[0]);
        ls[1] = fmaf(p[1], ki.y, ls[1]);
        ls[2] = fmaf(p[2], ki.z, ls[2]);
        ls[3] = fmaf(p[3], ki.w, ls[3]);
        split_p(p, p1[c / 4], p2[c / 4]);
      }
      l += (ls[0] + ls[1]) + (ls[2] + ls[3]);
      tmem_st16(s_addr, p1);
      tmem_st16(s_addr + 16, p2);
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(&sm.p_full[g]);
    }
    // Every PV completed. PV(J - 2) first: only then is the parity of PV(J - 1) unambiguous.
    if (ok && J > 0 && (!wait_pv(J - 2) || !wait_pv(J - 1))) ok = false;
    sm.l_g[g][h] = l;
    sm.m_g[g][h] = m_used;
    if (!ok && lane == 0) sm.epi_bad = 1;
    named_bar_sync(1, 2 * kGroup);
    tc_fence_after();
    const bool fin = !sm.epi_bad;
    // The last published maximum (it only grows) is what O refers to.
    const float m_fin = fmaxf(sm.m_g[0][h], sm.m_g[1][h]);
    float den = 0.f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float li = sm.l_g[i][h];
      if (li != 0.f) den += li * exp2f(sm.m_g[i][h] - m_fin);
    }
    const bool any = m_fin != -CUDART_INF_F || den != den;  // some candidate counted (or the row is NaN)
    float ref = m_fin + kHead;
    const float sl = h < P.H ? P.sink[h] * 1.4426950408889634f : -CUDART_INF_F;
    float f;                                   // what O is multiplied by
    if (P.splits == 1) {
      den += exp2f(sl - ref);
      f = any ? (1.f / 256.f) / den : 0.f;
    } else {
      // A partial refers to its own maximum; split 0's denominator holds the sink, and refers to the
      // sink if that is larger.
      f = 1.f / 256.f;
      if (sp == 0 && sl > -CUDART_INF_F) {
        const float r = fmaxf(ref, sl);
        const float w = any ? exp2f(ref - r) : 0.f;
        den = (den != 0.f ? den * w : 0.f) + exp2f(sl - r);
        f *= w;
        ref = r;
      }
      if (g == 0 && half == 0 && h < P.H && fin) {
        const long long r = (long long)item * 2 * P.H + h;
        P.part_ml[r] = ref;
        P.part_ml[r + P.H] = den;
      }
    }
    const bool read_o = J > 0 && any;
    if (fin) {
      const int rope0 = 512 - P.rope_dim;
      uint8_t* srow = stages + (size_t)h * kRowPitch;  // every gather and MMA that reads the stages completed
#pragma unroll 1
      for (int cc = 0; cc < 4; ++cc) {
        const int lc = 128 * g + 32 * cc, col0 = 256 * half + lc;
        uint32_t o[32];
        tmem_ld32(tmem + lane_addr + 256 + lc, o);
        tmem_wait_ld();
        float v[32];
#pragma unroll
        for (int c = 0; c < 32; ++c) v[c] = read_o ? __uint_as_float(o[c]) * f : 0.f;
        if (P.splits == 1 && col0 + 32 > rope0) {
#pragma unroll
          for (int c = 0; c < 32; c += 2) {
            const int dim = col0 + c;
            if (dim >= rope0) {
              const float cs = sm.rope_cs[(dim - rope0) >> 1][0], sn = sm.rope_cs[(dim - rope0) >> 1][1];
              const float e = v[c], od = v[c + 1];
              v[c] = e * cs - od * sn;
              v[c + 1] = e * sn + od * cs;
            }
          }
        }
        if (P.splits > 1 || P.out_is_f32) {
          if (h < P.H) {
            float* dst = P.splits > 1 ? P.part_o + ((long long)item * P.H + h) * 512 + col0
                                      : static_cast<float*>(P.out) + ((long long)qi * P.H + h) * 512 + col0;
#pragma unroll
            for (int c = 0; c < 8; ++c)
              reinterpret_cast<float4*>(dst)[c] = make_float4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
          }
        } else {
          uint4* dst = reinterpret_cast<uint4*>(srow + 2 * lc);
#pragma unroll
          for (int c = 0; c < 4; ++c)
            dst[c] = make_uint4(pack_bf16(v[8 * c], v[8 * c + 1]), pack_bf16(v[8 * c + 2], v[8 * c + 3]),
                                pack_bf16(v[8 * c + 4], v[8 * c + 5]), pack_bf16(v[8 * c + 6], v[8 * c + 7]));
        }
      }
      if (P.splits == 1 && !P.out_is_f32) {
        // Each head row's 512 bytes leave in one bulk store, once both groups staged their halves.
        fence_proxy_async_smem();
        named_bar_sync(1, 2 * kGroup);
        if (g == 0 && h < P.H) {
          bulk_store_global(static_cast<uint16_t*>(P.out) + ((long long)qi * P.H + h) * 512 + 256 * half, smem_u32(srow), 512);
          bulk_commit();
          bulk_wait_read_all();
        }
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kPvWarp8) tmem_dealloc(tmem, 512);
}

size_t attn8_smem_bytes() { return 1024 + kStages8 * kStage + kQ2Bytes + sizeof(Smem8); }

}  // namespace csa
