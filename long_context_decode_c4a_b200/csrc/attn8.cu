// attn8.cu -- sparse MQA with a learned sink and inverse RoPE over a cache held in 8 bits, in pages.
//
// For query t of request b and head h, over the window rows (bf16, ring) and the compressed entries
// (e4m3 codes c_j in pages, one power-of-two scale s_j for each block of entries):
//   l_j = scale * q_h . (s_j c_j),  m = max(max_j l_j, sink_h),
//   o_h = sum_j e^(l_j - m) s_j c_j / (sum_j e^(l_j - m) + e^(sink_h - m)), then rotate o_h[448:] by -t.
// The entries are the query's selected ones (list form) or every visible one (range form).
//
// The cached bytes go to the tensor cores as they are (tcgen05.mma kind::f8f6f4, both operands e4m3);
// what meets them is split into 8-bit pieces instead of the cache being widened to bf16:
//   q_h = 2^k_h (q1 + q2): q1 is q_h 2^-k_h (largest element in (224, 448]) rounded to e4m3 (4 significant bits),
//     q2 the remainder in e5m2. A bf16 value has 8 significant bits, so the remainder of rounding to 4 is at most 8
//     units of the last: 3 bits hold it. q1 + q2 is exact down to 2^-14 of the head's largest element (where q1
//     becomes subnormal), and off by at most 2^-21 of the largest below.
//   A window row is split the same way, c = 2^k (c1 + c2), both e4m3 (they are rows of one tile: 32 candidates
//     a tile); exact down to 2^-10 of the row's largest element, off by at most 2^-17 of it below. Its score is the
//     sum of the two columns, its P stands in both.
//   P = p1 + p2: p1 is P rounded to e4m3 (4 significant bits), p2 the remainder rounded to e5m2 (3 bits), so
//     P is off by at most 2^-8 of itself (p1 leaves 2^-4 of its binade, p2 2^-4 of that). A bf16 P's worst case is the same,
//     its mean square 2.8 times as large; the P_hi + P_lo of attn.cu (2^-16) would take a third and a fourth piece
//     here, and the tensor memory that holds P is full with two. P below 2^-14, where p1 is subnormal, is off by at most
//     2^-22; below 2^-18 p2 alone has it, by at most 2^-3 of itself (and fp16's 2^-25); below 2^-25 nothing is left.
//     (In units where the largest P lies between 2^-4.25 and 2^0.75; kHeadMost says what that means for a long tail.)
// P carries the scale of its column (O += (p_j s_j) c_j), so the running maximum is that of
// y_j = l_j + log2 s_j; the denominator takes P back to p_j with 1 / s_j. The sink enters at the end
// only: it must not push P below e4m3's range.
//
// Layout: a cluster of two CTAs per query. CTA `half` accumulates O[:, 256 half .. 256 half + 256) (128 heads x 256
// columns of fp32 are half of TMEM) over all tiles of 64 rows; the scores and the softmax of a tile are one
// CTA's (tile j: CTA j % 2's own), which sends P (16 KB) to the other. So of a tile its owner gathers whole rows and the other
// CTA its half of them, and the tensor cores spend 1264 cycles a tile and CTA (scores 1504 every other tile, PV 512).
//   TMEM (512 columns): [0,128) q1 (four codes a column); [128,192) the scores of an own tile; [192,224)
//     and [224,256) P of even and odd own tiles (p1, then p2); [256,512) O. The scores leave for registers as soon
//     as they are there, so the score MMAs of the next own tile run during the softmax of this one.
//   SMEM (128B-swizzled blocks of 64 rows x 128 dims, which serve the scores as a K-major and PV as an MN-major
//     operand): six slots A of this CTA's 256 dims (a slot a tile, until its PV completed), two slots B of the other
//     256 dims (own tiles, until their scores are there), a buffer for the other CTA's P; q2 (64 KB).
//   Warps: 0..3 split window rows and gather entries (16-byte cp.async); 4 issues the score MMAs, 5 the PV MMAs
//     (and owns TMEM); 6..9 and 10..13 are the softmax groups of even and odd own tiles, one head (TMEM lane)
//     a thread; both first split q (each CTA half of the heads, for both) and own tile 1's window rows, and share the epilogue.
//   The reference of P and O (the maximum, when it last had to be raised) is handed from tile to tile, so across the
//     CTAs each time: the group of tile j takes over that of tile j - 1, rescales its CTA's O if it changed, allows
//     PV(j - 1) (ack), raises it if its own scores ask for it, and hands it on before it forms P.
// Split-candidate mode (few queries): as in attn.cu; attn_combine_kernel merges the partials.
//
// One B200, in a graph: 64 requests at 32K (1024 of 8192 entries and 128 window rows each) 42.8 us, 0.27 of the time that the
// operations need at the dense bf16 rate and 0.21 of the HBM copy rate; a segment of 2000 queries 1105 us (0.33 of the
// former); 24 requests of 1500 entries 36.8 us; one request of 39 entries 19.8 us. (Fewer heads than 128 are padded to 128: 16 heads
// of the first case take 40.3 us.) No unit is near its limit (tensor pipe 23 %, issue slots 26 %): bound by the way of a tile through its stations, gather to PV, that six slots cover, and by
// 5 us before the first scores (list, q and its split) and 3 after the last PV.

#include <math_constants.h>

#include <cstddef>

#include "attn_util.cuh"
#include "kernels.cuh"
#include "ptx.cuh"
#include "rope.cuh"

namespace csa {

namespace {

constexpr int kProd = 128;                      // warps 0..3
constexpr int kQkWarp = 4;
constexpr int kPvWarp8 = 5;
constexpr int kSoftWarp = 6;                    // warps 6..9 (even tiles), 10..13 (odd tiles)
constexpr int kGroup = 128;                     // threads of a softmax group
constexpr int kRows = 64;                       // rows of a tile
constexpr int kWinRows = 32;                    // window candidates of a tile (two rows each)
constexpr int kA = 6;                           // slots A
constexpr uint32_t kBlk = kRows * 128;          // a block: 64 rows x 128 dims
constexpr uint32_t kSlot = 2 * kBlk;            // a slot: 256 dims (16 KB); a P buffer of 128 heads x (p1, p2) is as large
constexpr uint32_t kQBlk = 128 * 128;           // one 128-dim block of a q piece
constexpr uint32_t kQ2Bytes = 4 * kQBlk;        // 64 KB
// TMEM columns.
constexpr uint32_t kScoreCol = 128, kPCol = 192, kOCol = 256;
// P is formed relative to 2^ref, the reference ref = m + head, m the running maximum when O was last rescaled: later rows may
// exceed ref by 2^kOver before O has to be rescaled again, P staying at or below 1.75 (e4m3's 448). Headroom costs the weights
// far below the largest: P below 2^-14 is off by up to 2^-22, its pieces' steps there, which J tiles can add up to
// 64 J 2^(head - 22) of the largest weight. So head is what keeps that below 2^-7 (P's own precision is 2^-8): kHeadMost up to 26
// tiles, then a binade less for each doubling, and none from 854 tiles on (54592 candidates a pair), beyond which the bound grows with
// the number of tiles. Less for few tiles would cost: 64 queries of 20 tiles took 42.8 us at 4.25, 44.4 at 3.7, as one of a
// warp's 32 heads needs a rescale more often; on long lists new maxima are rare.
constexpr float kHeadMost = 4.25f, kHeadLeast = -0.75f, kOver = 0.75f;
static_assert(kAttn8Threads == 32 * (kSoftWarp + 8), "warp roles");

struct Smem8 {
  uint64_t a_full[kA];     // this CTA's producers are done with the tile (for the other CTA's window tile: nothing to do)
  uint64_t w_full[kA];     // rows of a window tile that the other CTA owns
  uint64_t a_free[kA];     // PV of the slot's tile completed in both CTAs
  uint64_t b_free[2];      // the scores of own tile i are there: slot B i % 2 is free
  uint64_t s_full[2];      // the same, for the softmax (barrier i % 2: a group looks at its own tiles only)
  uint64_t s_free;         // ... and have left for registers (phase i)
  uint64_t p_full[2];      // P of own tile i stored (TMEM buffer i % 2)
  uint64_t pb_full[2];     // P of the other CTA's own tile i (i % 2) arrived
  uint64_t pb_free[2];     // PV of own tile i (i % 2) completed in the other CTA: its P buffer is free
  uint64_t ack[2];         // group g took over the reference of the other CTA's tile: O is ready for its PV
  uint64_t pv_done[4];     // PV(j) completed (barrier j % 4): O holds PV(0..j)
  uint64_t hand[2][4];     // the reference after the other CTA's tile of its group g (quadrant q) arrived
  uint64_t ex_full;        // the other CTA's denominators
  uint64_t q_ready;        // both CTAs' pieces of q are in shared memory
  uint64_t q_done;         // q1 is in TMEM in both CTAs: the staging area (slots A 3 to 5, the P buffer) is free
  uint64_t list_ready;
  uint64_t drain[2];
  uint32_t tmem_base;
  int abort_flag, epi_bad;
  int n_tiles, tile0, entry_tiles;
  float head;              // how far the reference is set above the maximum
  int last[kProd / 32];
  float rope_cs[kMaxRopePairs][2];
  float qf[128];           // per head: 2^k_h * scale * log2(e)
  float2 hand_m[2][128];   // (the reference before that tile, after it)
  float l_g[4][128], m_g[4][128];                     // of this CTA's groups, then of the other's
  float scale[4][kRows];                              // scales of own tile i's rows (i % 4), as gathered
  alignas(16) float col_a[8][kRows], col_k[8][kRows], col_i[8][kRows];  // (read four at a time) per softmax warp: s_j, log2 s_j, 1 / s_j of its tile's columns
};

constexpr size_t kTileBytes = (kA + 3) * (size_t)kSlot;  // slots A, P buffer, slots B
static_assert(128 * (1024 + 16) <= kTileBytes + kQ2Bytes, "output staging");
static_assert(offsetof(Smem8, col_a) % 16 == 0 && sizeof(Smem8::col_a[0]) % 16 == 0, "float4 reads of the column factors");

// The upper bytes of two fp16 pairs (their e5m2 codes, the lower bits dropped).
__device__ __forceinline__ uint32_t codes_e5m2(uint32_t v0, uint32_t v1) { return __byte_perm(v0, v1, 0x7531); }

// 2^8 (a - b) of two fp16 pairs; exact where the difference is.
__device__ __forceinline__ uint32_t rest2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(r), "r"(0x5C005C00u));
  return r;
}
// Round an fp16 pair to e4m3's 4 significant bits (half a unit away from zero: the code's carry is fp16's).
__device__ __forceinline__ uint32_t round_e4m3(uint32_t h) { return (h + 0x00400040u) & 0xFF80FF80u; }

// Split of a 512-dim bf16 row held by a warp: lane l has dims [8 l, 8 l + 8) in a and [256 + 8 l, ...) in b. The row
// is scaled to at most 448 in magnitude and taken through fp16, which holds every scaled bf16 value above 2^-14
// exactly and the rest to 2^-25. Returns 2^k with max |x| <= 448 * 2^k (k >= -100), or NaN if a value is not finite (its
// pieces are then whatever they are: a row's scale, or a head's factor, of NaN makes NaN of all that it meets).
// Two integer instructions in three run at half rate here, the conversions to 8 bits at a quarter: a row costs a
// warp about 200 cycles, which is what the split of q and of the window rows is bound by.
struct RowPieces {
  uint2 hi[2], lo[2];
};
template <bool kLoE5M2>
__device__ __forceinline__ float split_row(const uint4& a, const uint4& b, RowPieces& out) {
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  uint32_t mx = w[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) mx = max_abs_bf16x2(mx, w[i]);
  mx = __reduce_max_sync(0xffffffffu, max(mx & 0x7FFFu, (mx >> 16) & 0x7FFFu));
  const int e = (int)(mx >> 7);  // biased exponent of the largest magnitude; 448 = 1.75 * 2^8, 0x60 / 128 = 0.75
  const int k = max(-100, e - 127 - 8 + ((mx & 0x7Fu) > 0x60u ? 1 : 0));
  const float inv = __uint_as_float((uint32_t)(127 - k) << 23);
  uint16_t h[8];
  uint32_t r[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    uint32_t v, back;
    asm("cvt.rn.f16x2.f32 %0, %2, %1;" : "=r"(v) : "f"(__uint_as_float(w[i] << 16) * inv), "f"(__uint_as_float(w[i] & 0xFFFF0000u) * inv));
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(h[i]) : "r"(v));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(back) : "h"(h[i]));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r[i]) : "r"(v), "r"(back));
  }
#pragma unroll
  for (int v = 0; v < 2; ++v)
    out.hi[v] = make_uint2(h[4 * v] | ((uint32_t)h[4 * v + 1] << 16), h[4 * v + 2] | ((uint32_t)h[4 * v + 3] << 16));
  if (kLoE5M2) {
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] += 0x00800080u;  // round the byte that leaves
#pragma unroll
    for (int v = 0; v < 2; ++v)
      out.lo[v] = make_uint2(codes_e5m2(r[4 * v], r[4 * v + 1]), codes_e5m2(r[4 * v + 2], r[4 * v + 3]));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(h[i]) : "r"(r[i]));
#pragma unroll
    for (int v = 0; v < 2; ++v)
      out.lo[v] = make_uint2(h[4 * v] | ((uint32_t)h[4 * v + 1] << 16), h[4 * v + 2] | ((uint32_t)h[4 * v + 3] << 16));
  }
  return e < 255 ? __uint_as_float((uint32_t)(127 + k) << 23) : CUDART_NAN_F;
}

// Bytes that a CTA gets from the other: of a window tile (two pieces of 32 half rows), of q (64 heads, two pieces and a
// factor each), of a tile's P, a warp's references, the denominators.
constexpr uint32_t kPeerTile = 2 * 32 * 256, kPeerQ = 64 * (2 * 512 + 4), kPeerP = 128 * 128, kPeerRef = 32 * 8, kPeerSum = 2 * 128 * 8;

__device__ __forceinline__ void st_shared_v2(uint32_t addr, uint2 v) {
  asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(addr), "r"(v.x), "r"(v.y) : "memory");
}

// Both run once for each row and are not inlined: eight copies each are 60 KB of code beside the softmax's, and instruction
// fetch is what this kernel's warps wait for most after their turn (64 requests at 32K: 46.5 us inlined, 44.0 so).
//
// Split a head's row and store lane l's 8 + 8 codes of each piece at q1 / q2 + off + {0, 2} blocks: of this CTA and of the
// other (at cluster address + far, the bytes counted on its barrier `bar`). Returns the row's factor.
__device__ __noinline__ float split_q_row(uint4 a, uint4 c, uint32_t q1, uint32_t q2, uint32_t far1, uint32_t far2, uint32_t bar) {
  RowPieces pc;
  const float f = split_row<true>(a, c, pc);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t at = 2u * i * kQBlk;
    st_shared_v2(q1 + at, pc.hi[i]);
    st_async_v2(far1 + at, pc.hi[i].x, pc.hi[i].y, bar);
    st_shared_v2(q2 + at, pc.lo[i]);
    st_async_v2(far2 + at, pc.lo[i].x, pc.lo[i].y, bar);
  }
  return f;
}
// Split a window row: its codes of this CTA's 256 dims to `mine`, of the other's to `other` and to the other CTA's
// slot (cluster address `far`); the second piece kWinRows rows on. Returns the row's scale.
__device__ __noinline__ float split_window_row(uint4 a, uint4 c, uint32_t mine, uint32_t other, uint32_t far, uint32_t bar, int half) {
  RowPieces pc;
  const float s = split_row<false>(a, c, pc);
#pragma unroll
  for (int lo = 0; lo < 2; ++lo) {
    const uint2 v0 = lo ? pc.lo[0] : pc.hi[0], v1 = lo ? pc.lo[1] : pc.hi[1];
    const uint2 m = half ? v1 : v0, o = half ? v0 : v1;
    const uint32_t at = lo * kWinRows * 128u;   // (a multiple of 8 rows: the same swizzle)
    st_shared_v2(mine + at, m);
    st_shared_v2(other + at, o);
    st_async_v2(far + at, o.x, o.y, bar);
  }
  return s;
}

// Two 512-dim bf16 rows of a warp, as split_row takes them.
struct RowPair {
  uint4 a[2], c[2];
};
__device__ __forceinline__ void read_row(RowPair& r, int i, const uint16_t* src, bool valid) {
  r.a[i] = r.c[i] = make_uint4(0, 0, 0, 0);
  if (valid) {
    r.a[i] = reinterpret_cast<const uint4*>(src)[lane_id()];
    r.c[i] = reinterpret_cast<const uint4*>(src)[32 + lane_id()];
  }
}

// P (fp32 in [0, 1.75), standing for 2^8 P in 8-bit units) to its two pieces, four columns at a time.
__device__ __forceinline__ void split_p(float p0, float p1, float p2, float p3, uint32_t& c1, uint32_t& c2) {
  uint32_t h0, h1;
  asm("cvt.rn.f16x2.f32 %0, %2, %1;" : "=r"(h0) : "f"(p0), "f"(p1));
  asm("cvt.rn.f16x2.f32 %0, %2, %1;" : "=r"(h1) : "f"(p2), "f"(p3));
  const uint32_t a0 = round_e4m3(h0), a1 = round_e4m3(h1);
  c1 = __byte_perm(a0 >> 7, a1 >> 7, 0x6420);  // P >= 0: no sign to move
  c2 = codes_e5m2(rest2(h0, a0) + 0x00800080u, rest2(h1, a1) + 0x00800080u);
}

// Order of a query's tiles. Three window tiles or more (the usual window of 128 has four): four of them first, which the
// gathering and the softmax warps split while there is nothing else to do. Then, or with fewer from the start, two entry
// tiles, then pairs of window and of entry tiles in turn while both last, the rest of the window, the rest of the
// entries: further on the split of a window tile takes the gathering warps longer than the tensor cores need for a tile. (Pairs,
// so that each CTA owns half of the window.) B200, 64 queries of 1024 entries, window first and entries first: 16 rows 39.9 and
// 38.0 us, 64 rows 40.2 and 39.0, 80 rows 40.9 and 42.2, 128 rows 42.2 and 44.0, 512 rows 73.5 and 75.7.
__device__ __forceinline__ int first_window(int Tw) { return Tw >= 3 ? min(Tw, 4) : 0; }
// The index of tile p among those of its kind.
__device__ __forceinline__ int tile_of(int p, int Tw, int Te, bool& win) {
  const int first = first_window(Tw), rest = Tw - first;
  win = p < first;
  if (win) return p;
  p -= first;
  if (rest == 0) return p;
  const int alt = Te < 2 ? 0 : min(rest >> 1, (Te - 2) >> 1), e0 = Te < 2 ? 0 : 2, q = p - e0;
  if (q < 0) return p;
  if (q < 4 * alt) {
    win = (q & 2) == 0;
    return (q >> 2) * 2 + (q & 1) + (win ? first : e0);
  }
  const int w = 2 * alt + q - 4 * alt;  // the first of what is left is the (2 alt)-th of the rest
  win = w < rest;
  return win ? first + w : e0 + 2 * alt + (w - rest);
}
// No window tile lies at this position or behind it.
__device__ __forceinline__ int window_end(int Tw) { return Tw == first_window(Tw) ? Tw : 2 * Tw + 2 - first_window(Tw); }

// Two fp32 operations an instruction.
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

}  // namespace

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kAttn8Threads, 1) attn8_kernel(Attn8Params P) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* slots_a = base;
  uint8_t* pb = slots_a + kA * kSlot;
  uint8_t* slots_b = pb + kSlot;
  uint8_t* q2 = base + kTileBytes;
  uint8_t* q1s = slots_a + 3 * kSlot;            // q1 on its way to TMEM: slots A 3 to 5, the P buffer
  Smem8& sm = *reinterpret_cast<Smem8*>(q2 + kQ2Bytes);

  const int warp = warp_id(), lane = lane_id();
  const int half = (int)cluster_ctarank();
  const uint32_t peer = (uint32_t)half ^ 1u;
  const int nq = P.B * P.S;
  const int item = nq * P.splits - 1 - (int)(blockIdx.x >> 1);  // later queries (more candidates) first
  const int qi = item / P.splits, sp = item % P.splits, b = qi / P.S;
  volatile int* abort_flag = &sm.abort_flag;
  uint32_t* status = P.status;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kA; ++i) {
      mbar_init(&sm.a_full[i], kProd);
      mbar_init(&sm.w_full[i], 1);
      mbar_init(&sm.a_free[i], 2);
    }
    mbar_init(&sm.s_free, kGroup);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.b_free[i], 1);
      mbar_init(&sm.s_full[i], 1);
      mbar_init(&sm.p_full[i], kGroup);
      mbar_init(&sm.pb_full[i], 1);
      mbar_init(&sm.pb_free[i], 1);
      mbar_init(&sm.ack[i], kGroup);
      for (int q = 0; q < 4; ++q) mbar_init(&sm.hand[i][q], 1);
    }
    for (int i = 0; i < 4; ++i) mbar_init(&sm.pv_done[i], 1);
    mbar_init(&sm.ex_full, 1);
    mbar_init(&sm.q_ready, 2 * kGroup + 1);
    mbar_init(&sm.q_done, 4 * kGroup);
    mbar_init(&sm.list_ready, 1);
    for (int i = 0; i < 2; ++i) mbar_init(&sm.drain[i], 1);
    sm.abort_flag = 0;
    sm.epi_bad = 0;
    fence_mbar_init();
  }
  if (warp == kPvWarp8) {
    tmem_alloc(&sm.tmem_base, 512);
    tmem_relinquish();
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync();  // the barriers of both CTAs are initialised
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
  // Tile j (of this item's J) is CTA j % 2's own, the (j >> 1)-th of them; it lies in slot A j % kA.

  // N candidates of window tile w, from the r0-th on, into a warp's registers ...
  auto window_read = [&](auto& rows, int w, int r0) {
    constexpr int N = 2 * sizeof(rows) / sizeof(RowPair);
    const uint16_t* ring = P.ring + (long long)b * P.ring_bstride;
    const int k0 = w * kWinRows + r0;
    int slot = (p0 + (k0 < nwin ? k0 : 0)) % P.ring_cap;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      read_row(rows[i >> 1], i & 1, ring + (long long)slot * 512, k0 + i < nwin);
      slot = slot + 1 == P.ring_cap ? 0 : slot + 1;
    }
  };
  // ... and their pieces into slots A `slot` and B own % 2 of own tile `own`, and the other CTA's slot A (its half of the
  // dims): candidate r in rows r and r + 32.
  auto window_store = [&](auto& rows, int w, int r0, int slot, int own) {
    constexpr int N = 2 * sizeof(rows) / sizeof(RowPair);
    const uint32_t mine = smem_u32(slots_a + (size_t)slot * kSlot), other = smem_u32(slots_b + (size_t)(own & 1) * kSlot);
    const uint32_t far = mapa_shared(mine, peer), bar = mapa_shared(smem_u32(&sm.w_full[slot]), peer);
    const uint32_t lane_off = (uint32_t)(lane >> 4) * kBlk + (uint32_t)(lane & 1) * 8u;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int r = r0 + i;
      const uint32_t off = lane_off + sw128_offset((uint32_t)r, (uint32_t)((lane & 15) >> 1));
      float s = split_window_row(rows[i >> 1].a[i & 1], rows[i >> 1].c[i & 1], mine + off, other + off, far + off, bar, half);
      if (w * kWinRows + r >= nwin) s = 0.f;
      if (lane < 2) sm.scale[own & 3][r + kWinRows * lane] = s;
    }
    fence_proxy_async_smem();
  };

  if (warp < kProd / 32) {
    // ------------------------------------------------------------ window split, gathers
    const int pt = threadIdx.x;
    const int32_t* table = P.table + (long long)b * P.max_pages;
    const int32_t* sel = P.topk_idx == nullptr ? nullptr : P.topk_idx + (long long)qi * P.topk;
    bool bad = false;
    // Number of candidates: up to the last valid place of the list (-1 in between is a masked row), or every entry.
    const int lk = warp + 4 * (lane & 15);  // the row of a tile that lane i < 16 looks after
    // The gathering warps split own tile 0, if it is of the window (8 rows a warp), and own tiles from 2 on; the softmax warps
    // own tile 1.
    RowPair wr[4];
    const bool early = P.splits == 1 && half < first_window(Tw);
    if (early) window_read(wr, half, 8 * warp);  // in flight while the list is looked through
    int n = ecap, s0 = lk, s1 = lk + kRows;
    if (sel != nullptr) {
      s0 = lk < P.topk ? sel[lk] : -1;
      s1 = lk + kRows < P.topk ? sel[lk + kRows] : -1;
      int last = 0;
      for (int j = pt; j < P.topk; j += kProd)
        if (sel[j] >= 0) last = j + 1;
      last = t < 0 ? 0 : __reduce_max_sync(0xffffffffu, last);
      if (lane == 0) sm.last[warp] = last;
      named_bar_sync(2, kProd);
      n = max(max(sm.last[0], sm.last[1]), max(sm.last[2], sm.last[3]));
    } else {
      bad = t >= 0 && ((long long)t + 1) / P.ratio > P.max_entries;
    }
    const int Te = (n + kRows - 1) / kRows, Jq = Tw + Te;
    const int tile0 = (int)(((long long)Jq * sp) / P.splits);
    const int J = (int)(((long long)Jq * (sp + 1)) / P.splits) - tile0;
    if (pt == 0) {
      sm.n_tiles = J;
      sm.tile0 = tile0;
      sm.entry_tiles = Te;
      sm.head = fminf(kHeadMost, fmaxf(kHeadLeast, 9.f - log2f((float)max(J, 1))));
      mbar_arrive(&sm.list_ready);
    }

    // Lane i < 16 of a warp has the tile's row warp + 4 i: its entry is read two tiles ahead, its page one tile ahead.
    auto entry_of = [&](int j) -> int {
      bool win;
      const int k = tile_of(tile0 + j, Tw, Te, win) * kRows + lk;
      if (j >= J || win || k >= n) return -1;
      return sel != nullptr ? sel[k] : k;
    };
    auto pool_row = [&](int e) -> int {
      if (e < 0) return -1;
      if (e >= ecap) {
        bad = true;
        return -1;
      }
      const int pg = table[e >> P.page_shift];
      if (pg < 0 || pg >= P.num_pages) {
        bad = true;
        return -1;
      }
      return (pg << P.page_shift) | (e & ((1 << P.page_shift) - 1));
    };
    auto begin = [&](int j) -> int {
      bool win;
      const int i = tile_of(tile0 + j, Tw, Te, win), k = i * kRows + lk;
      if (j >= J || win || k >= n) return -1;
      return i == 0 ? s0 : i == 1 ? s1 : sel != nullptr ? sel[k] : k;
    };
    int next_row = pool_row(begin(0)), next_entry = begin(1);
    // The next own window tile behind tile j that these warps split, into registers.
    auto next_window = [&](int j) {
      for (j += 2; j < J && tile0 + j < window_end(Tw); j += 2) {
        bool win;
        const int w = tile_of(tile0 + j, Tw, Te, win);
        if (win && j >> 1 != 1) {
          window_read(wr, w, 8 * warp);
          return;
        }
      }
    };
    if (!early) next_window(half - 2);
    int slot = 0;
    uint32_t ph = 0;
    // A lane whose wait ran out stays in the loop (its later waits return at once, and the output is given up): the warp's
    // shuffles need all lanes, and a vote on each wait costs 2.5 % of the kernel.
    for (int j = 0; j < J; ++j) {
      const int my_row = next_row;
      next_row = pool_row(next_entry);
      next_entry = entry_of(j + 2);
      if (j >= kA) mbar_wait_cluster(&sm.a_free[slot], ph ^ 1u, abort_flag, status, 302);
      else if (j >= 3) mbar_wait_cluster(&sm.q_done, 0, abort_flag, status, 301);
      bool win;
      const int index = tile_of(tile0 + j, Tw, Te, win), i0 = j >> 1;
      const uint32_t sa = smem_u32(slots_a + (size_t)slot * kSlot);
      if ((j & 1) == half) {
        if (i0 >= 2) mbar_wait(&sm.b_free[i0 & 1], (uint32_t)((i0 >> 1) & 1) ^ 1u, abort_flag, status, 304);
        if (win) {
          if (i0 != 1) {
            window_store(wr, index, 8 * warp, slot, i0);
            mbar_arrive(&sm.a_full[slot]);
            next_window(j);
          }
        } else {
          const uint32_t sb = smem_u32(slots_b + (size_t)(i0 & 1) * kSlot);
          const uint32_t st = ((lane >> 4) == half ? sa : sb) + (uint32_t)((lane >> 3) & 1) * kBlk;
          const uint8_t* src = P.pages + lane * 16;
          // Rows 8 apart have the same swizzle: two offsets serve all.
          const uint32_t st0 = st + sw128_offset((uint32_t)warp, (uint32_t)(lane & 7)),
                         st1 = st + sw128_offset((uint32_t)(warp + 4), (uint32_t)(lane & 7));
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int row = __shfl_sync(0xffffffffu, my_row, i);
            cp_async_16_zfill(((i & 1) ? st1 : st0) + (uint32_t)(i >> 1) * 1024u, src + (size_t)(uint32_t)max(row, 0) * 512u, row >= 0);
          }
          if (lane < 16)
            cp_async_4_zfill(smem_u32(&sm.scale[i0 & 3][warp + 4 * lane]), P.scales + (max(my_row, 0) >> P.block_shift),
                             my_row >= 0);
          cp_async_arrive_noinc(&sm.a_full[slot]);
        }
      } else if (win) {
        if (pt == 0) mbar_arrive_expect_tx(&sm.w_full[slot], kPeerTile);
        mbar_arrive(&sm.a_full[slot]);
      } else {
        // Two half rows an instruction: rows warp + 4 i and warp + 4 (i + 1).
        const uint32_t st = sa + (uint32_t)((lane >> 3) & 1) * kBlk + sw128_offset((uint32_t)(warp + 4 * (lane >> 4)), (uint32_t)(lane & 7));
        const uint8_t* src = P.pages + 256 * half + (lane & 15) * 16;
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
          const int row = __shfl_sync(0xffffffffu, my_row, i + (lane >> 4));
          cp_async_16_zfill(st + (uint32_t)(i >> 1) * 1024u, src + (size_t)(uint32_t)max(row, 0) * 512u, row >= 0);
        }
        cp_async_arrive_noinc(&sm.a_full[slot]);
      }
      if (++slot == kA) {
        slot = 0;
        ph ^= 1u;
      }
    }
    // The other CTA's last commits have arrived here too (this CTA's shared memory may be given up after the end).
    for (int j = max(0, J - kA); j < J; ++j)
      if (!mbar_wait_cluster(&sm.a_free[j % kA], (uint32_t)((j / kA) & 1), abort_flag, status, 303)) break;
    cp_async_wait_all();  // after an abort: let the copies land before teardown
    if (bad && half == 0) record_status(status, CSA_DEV_BOUNDS);
    __syncwarp();
    cluster_arrive_relaxed();
  } else if (warp == kQkWarp) {
    // ------------------------------------------------------------ score MMAs of the own tiles
    // The whole warp walks the loop, so that addresses and descriptors stay in uniform registers (a thread by
    // itself in a divergent branch took 80 cycles to issue each MMA of 47); one thread issues.
    const bool leader = elect_one();
    const bool ok = __all_sync(0xffffffffu, mbar_wait_cluster(&sm.q_ready, 0, abort_flag, status, 310)) &&
                    __all_sync(0xffffffffu, mbar_wait_cluster(&sm.q_done, 0, abort_flag, status, 311)) &&
                    __all_sync(0xffffffffu, mbar_wait(&sm.list_ready, 0, abort_flag, status, 312));
    const int J = ok ? sm.n_tiles : 0;
    constexpr uint32_t idesc1 = idesc_fp8_f32(kE4M3, kE4M3, 128, kRows, 0, 0);
    constexpr uint32_t idesc2 = idesc_fp8_f32(kE5M2, kE4M3, 128, kRows, 0, 0);
    const uint64_t da = smem_desc_sw128(smem_u32(slots_a), 16, 1024), db = smem_desc_sw128(smem_u32(slots_b), 16, 1024);
    // Blocks of q: this CTA's dims first (slot A), then the other's (slot B).
    const uint64_t dq = smem_desc_sw128(smem_u32(q2), 16, 1024);
    const uint32_t near = 2 * (uint32_t)half, far = 2 * peer;
    int slot = half;
    uint32_t ph = 0;
    for (int i = 0, j = half; j < J; ++i, j += 2) {
      if (!__all_sync(0xffffffffu, mbar_wait(&sm.a_full[slot], ph, abort_flag, status, 314))) break;
      if (i > 0 && !__all_sync(0xffffffffu, mbar_wait(&sm.s_free, (uint32_t)((i - 1) & 1), abort_flag, status, 313))) break;
      fence_proxy_async_smem();  // rows written by cp.async before the MMAs read them
      tc_fence_after();
      const uint64_t ka = da + (uint64_t)((uint32_t)slot * (kSlot >> 4)), kb = db + (uint64_t)((uint32_t)(i & 1) * (kSlot >> 4));
      if (leader) {
#pragma unroll
        for (int ks = 0; ks < 16; ++ks) {
          const uint32_t blk = (ks < 8 ? near : far) + ((ks >> 2) & 1);
          mma8_ts(tmem + kScoreCol, tmem + 32 * blk + 8 * (ks & 3), (ks < 8 ? ka : kb) + ((((ks >> 2) & 1) * kBlk + (ks & 3) * 32) >> 4),
                  idesc1, ks > 0 ? 1u : 0u);
        }
#pragma unroll
        for (int ks = 0; ks < 16; ++ks) {
          const uint32_t blk = (ks < 8 ? near : far) + ((ks >> 2) & 1);
          mma8_ss(tmem + kScoreCol, dq + ((blk * kQBlk + (ks & 3) * 32) >> 4),
                  (ks < 8 ? ka : kb) + ((((ks >> 2) & 1) * kBlk + (ks & 3) * 32) >> 4), idesc2, 1u);
        }
        mma_commit(&sm.s_full[i & 1]);
        mma_commit(&sm.b_free[i & 1]);
      }
      __syncwarp();
      slot += 2;
      if (slot >= kA) {
        slot -= kA;
        ph ^= 1u;
      }
    }
    // Every MMA issued above completes on its own; wait for them before TMEM is released.
    if (leader) {
      mma_commit(&sm.drain[0]);
      mbar_wait_drain(&sm.drain[0], 0, status, 315);
    }
    __syncwarp();
    cluster_arrive_relaxed();
  } else if (warp == kPvWarp8) {
    // ------------------------------------------------------------ PV MMAs of every tile
    const bool leader = elect_one();
    const int J = __all_sync(0xffffffffu, mbar_wait(&sm.list_ready, 0, abort_flag, status, 321)) ? sm.n_tiles : 0;
    const int tile0 = sm.tile0, Te = sm.entry_tiles;
    constexpr uint32_t idesc[2] = {idesc_fp8_f32(kE4M3, kE4M3, 128, 256, 0, 1), idesc_fp8_f32(kE5M2, kE4M3, 128, 256, 0, 1)};
    const uint64_t dv = smem_desc_sw128(smem_u32(slots_a), kBlk, 1024), dp = smem_desc_sw128(smem_u32(pb), 16, 1024);
    int slot = 0;
    uint32_t ph = 0, w_phase = 0;  // bit s of w_phase: parity of slot s's next window tile of the other CTA
    for (int j = 0; j < J; ++j) {
      const int i = j >> 1, g = i & 1;
      const uint32_t phase = (uint32_t)((i >> 1) & 1);
      const bool own = (j & 1) == half;
      if (own) {
        if (!__all_sync(0xffffffffu, mbar_wait(&sm.p_full[g], phase, abort_flag, status, 322))) break;
      } else {
        bool win;
        tile_of(tile0 + j, Tw, Te, win);
        if (!__all_sync(0xffffffffu, mbar_wait(&sm.a_full[slot], ph, abort_flag, status, 324))) break;
        if (win) {
          if (!__all_sync(0xffffffffu, mbar_wait_cluster(&sm.w_full[slot], (w_phase >> slot) & 1u, abort_flag, status, 325))) break;
          w_phase ^= 1u << slot;
        }
        if (!__all_sync(0xffffffffu, mbar_wait(&sm.ack[((j + 1) >> 1) & 1], (uint32_t)(((j + 1) >> 2) & 1), abort_flag, status, 326))) break;
        if (leader) mbar_arrive_expect_tx(&sm.pb_full[g], kPeerP);
        if (!__all_sync(0xffffffffu, mbar_wait_cluster(&sm.pb_full[g], phase, abort_flag, status, 327))) break;
      }
      fence_proxy_async_smem();
      tc_fence_after();
      const uint64_t vb = dv + (uint64_t)((uint32_t)slot * (kSlot >> 4));
      if (leader) {
        if (own) {
#pragma unroll
          for (int part = 0; part < 2; ++part)
#pragma unroll
            for (int ks = 0; ks < 2; ++ks)
              mma8_ts(tmem + kOCol, tmem + kPCol + 32 * g + 16 * part + 8 * ks, vb + ((ks * 4096) >> 4), idesc[part],
                      (j > 0 || part > 0 || ks > 0) ? 1u : 0u);
        } else {
#pragma unroll
          for (int part = 0; part < 2; ++part)
#pragma unroll
            for (int ks = 0; ks < 2; ++ks)
              mma8_ss(tmem + kOCol, dp + ((64 * part + 32 * ks) >> 4), vb + ((ks * 4096) >> 4), idesc[part],
                      (j > 0 || part > 0 || ks > 0) ? 1u : 0u);
          mma_commit_cluster(&sm.pb_free[g], (uint16_t)(1u << peer));
        }
        mma_commit_cluster(&sm.a_free[slot], 3);
        mma_commit(&sm.pv_done[j & 3]);
      }
      __syncwarp();
      if (++slot == kA) {
        slot = 0;
        ph ^= 1u;
      }
    }
    if (leader) {
      mma_commit(&sm.drain[1]);
      mbar_wait_drain(&sm.drain[1], 0, status, 323);
    }
    __syncwarp();
    cluster_arrive_relaxed();
  } else {
    // ------------------------------------------------------------ q split, softmax, epilogue
    const int sw = warp - kSoftWarp;           // 0..7
    const int g = sw >> 2;                     // softmax group
    const int quad = warp & 3;                 // TMEM lane quadrant
    const int h = quad * 32 + lane;            // head = TMEM lane
    const uint32_t lane_addr = (uint32_t)(quad * 32) << 16;
    // q rows 64 half + 8 sw .. + 7.
    {
      const int row0 = 64 * half + 8 * sw;
      const uint32_t q1_peer = mapa_shared(smem_u32(q1s), peer), q2_peer = mapa_shared(smem_u32(q2), peer),
                     qf_peer = mapa_shared(smem_u32(&sm.qf[0]), peer), bar = mapa_shared(smem_u32(&sm.q_ready), peer);
      if (sw == 0 && lane == 0) mbar_arrive_expect_tx(&sm.q_ready, kPeerQ);
      RowPair w[4];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        read_row(w[i >> 1], i & 1, P.q + ((long long)qi * P.H + (row0 + i)) * 512, row0 + i < P.H);
      const uint32_t lane_off = (uint32_t)(lane >> 4) * kQBlk + (uint32_t)(lane & 1) * 8u;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t off = lane_off + sw128_offset((uint32_t)(row0 + i), (uint32_t)((lane & 15) >> 1));
        const float f = split_q_row(w[i >> 1].a[i & 1], w[i >> 1].c[i & 1], smem_u32(q1s) + off, smem_u32(q2) + off, q1_peer + off,
                                    q2_peer + off, bar) * P.scale_log2;
        if (lane == 0) {
          sm.qf[row0 + i] = f;
          st_async_b32(qf_peer + 4 * (row0 + i), __float_as_uint(f), bar);
        }
      }
    }
    fence_proxy_async_smem();  // q2 before the MMAs read it
    mbar_arrive(&sm.q_ready);
    bool ok = __all_sync(0xffffffffu, mbar_wait_cluster(&sm.q_ready, 0, abort_flag, status, 330));
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
    mbar_arrive_remote_relaxed(mapa_shared(smem_u32(&sm.q_done), peer));  // this thread has read its part of the staging area

    // Own tile 1, if it is of the window: four rows a warp.
    ok = __all_sync(0xffffffffu, mbar_wait(&sm.list_ready, 0, abort_flag, status, 331)) && ok;
    {
      bool win = false;
      const int j = half + 2, w = ok && j < sm.n_tiles ? tile_of(sm.tile0 + j, Tw, sm.entry_tiles, win) : 0;
      if (win) {
        RowPair rows[2];
        window_read(rows, w, 4 * sw);
        // (Slot A 3 is in the staging area, here and in the other CTA.)
        ok = __all_sync(0xffffffffu, mbar_wait_cluster(&sm.q_done, 0, abort_flag, status, 340)) && ok;
        if (ok) window_store(rows, w, 4 * sw, j, 1);
        __syncwarp();
        if (ok && lane < 16) mbar_arrive(&sm.a_full[j]);  // eight warps: kProd arrivals
      }
    }

    // Inverse-RoPE table for position t, while the first scores are on their way (the epilogue's barrier orders it).
    const int st = threadIdx.x - kSoftWarp * 32;  // 0..255
    if (st < P.rope_dim / 2) {
      float cs, sn;
      rope_cos_sin(t, P.inv_freq[st], &cs, &sn);
      sm.rope_cs[st][0] = cs;
      sm.rope_cs[st][1] = -sn;
    }
    const int J = ok ? sm.n_tiles : 0;
    const int tile0 = sm.tile0, Te = sm.entry_tiles;
    const float qf = sm.qf[h];
    const uint64_t qf2 = pack2(qf, qf);
    // pv_done[i % 4] completes once per PV(i). A wait for PV(i) by parity is unambiguous while PV(i - 4) is known to have
    // completed and PV(i + 4) cannot have. A group waits for PV(j - 4) first of all at tile j (its P buffer's last
    // reader), and PVs complete in order; PV(j) needs this group's P, PV(j + 1) the reference that it hands on.
    auto wait_pv = [&](int i) -> bool {
      return i < 0 || __all_sync(0xffffffffu, mbar_wait(&sm.pv_done[i & 3], (uint32_t)((i / 4) & 1), abort_flag, status, 332));
    };
    float ref = -CUDART_INF_F, l = 0.f;
    // O from reference r0 to r (in the lanes where that is larger).
    auto rescale = [&](float r0, float r) {
      const float alpha = r > r0 ? exp2f(r0 - r) : 1.f;
      const uint64_t alpha2 = pack2(alpha, alpha);
      tc_fence_after();
#pragma unroll 1
      for (int cc = 0; cc < 8; ++cc) {
        uint32_t o[32];
        const uint32_t oa = tmem + lane_addr + kOCol + 32 * cc;
        tmem_ld32(oa, o);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          float a0, a1;
          unpack2(mul2(pack2(__uint_as_float(o[e]), __uint_as_float(o[e + 1])), alpha2), a0, a1);
          o[e] = __float_as_uint(a0);
          o[e + 1] = __float_as_uint(a1);
        }
        tmem_st32(oa, o);
      }
      tmem_wait_st();
      tc_fence_before();
    };
    // This group's sum from reference ref to r.
    auto refer_to = [&](float r) {
      if (r > ref) {
        l = l != 0.f ? l * exp2f(ref - r) : 0.f;
        ref = r;
      }
    };
    // Take over the reference after tile j - 1, the other CTA's, and allow its PV here.
    auto take_over = [&](int j) -> bool {
      const int from = ((j - 1) >> 1) & 1;
      if (lane == 0) mbar_arrive_expect_tx(&sm.hand[from][quad], kPeerRef);
      if (!__all_sync(0xffffffffu, mbar_wait_cluster(&sm.hand[from][quad], (uint32_t)(((j - 1) >> 2) & 1), abort_flag, status, 335)))
        return false;
      const float2 mp = sm.hand_m[from][h];
      if (j >= 2 && __any_sync(0xffffffffu, mp.y > mp.x)) {
        if (!wait_pv(j - 2)) return false;
        rescale(mp.x, mp.y);
      }
      refer_to(mp.y);
      mbar_arrive(&sm.ack[g]);
      return true;
    };
    const uint32_t hand_peer = mapa_shared(smem_u32(&sm.hand_m[g][h]), peer), hand_bar = mapa_shared(smem_u32(&sm.hand[g][quad]), peer),
                   pb_peer = mapa_shared(smem_u32(pb), peer), pb_bar = mapa_shared(smem_u32(&sm.pb_full[g]), peer);
    int last_own = -1;
    for (int i = g, j = 2 * g + half; j < J; i += 2, j += 4) {
      const int slot = j % kA;
      bool win;
      tile_of(tile0 + j, Tw, Te, win);
      // Column factors, two columns a lane, while the score MMAs run. A window candidate's second column
      // adds nothing to the denominator.
      if (!__all_sync(0xffffffffu, mbar_wait(&sm.a_full[slot], (uint32_t)((j / kA) & 1), abort_flag, status, 333))) {
        ok = false;
        break;
      }
      __syncwarp();  // the last tile's factors have been read
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int c = 32 * u + lane;
        const float s = sm.scale[i & 3][c];
        sm.col_a[sw][c] = s;
        sm.col_k[sw][c] = log2f(s);  // 0 (a masked column): -inf
        sm.col_i[sw][c] = (s == 0.f || (win && c >= kWinRows)) ? 0.f : 1.f / s;
      }
      __syncwarp();
      if (!__all_sync(0xffffffffu, mbar_wait(&sm.s_full[g], (uint32_t)((i >> 1) & 1), abort_flag, status, 334))) {
        ok = false;
        break;
      }
      tc_fence_after();
      uint64_t y[kRows / 2];
      {
        uint32_t v0[32], v1[32];
        tmem_ld32(tmem + lane_addr + kScoreCol, v0);
        tmem_ld32(tmem + lane_addr + kScoreCol + 32, v1);
        tmem_wait_ld();
        tc_fence_before();
        mbar_arrive(&sm.s_free);
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          y[c] = pack2(__uint_as_float(v0[2 * c]), __uint_as_float(v0[2 * c + 1]));
          y[c + 16] = pack2(__uint_as_float(v1[2 * c]), __uint_as_float(v1[2 * c + 1]));
        }
        if (win) {
#pragma unroll
          for (int c = 0; c < 16; ++c) y[c] = y[c + 16] = add2(y[c], y[c + 16]);
        }
      }
      float mx[2] = {-CUDART_INF_F, -CUDART_INF_F};
#pragma unroll
      for (int c = 0; c < kRows / 2; c += 2) {
        const ulonglong2 a = *reinterpret_cast<const ulonglong2*>(&sm.col_a[sw][2 * c]);
        const ulonglong2 k = *reinterpret_cast<const ulonglong2*>(&sm.col_k[sw][2 * c]);
        y[c] = fma2(mul2(y[c], qf2), a.x, k.x);
        y[c + 1] = fma2(mul2(y[c + 1], qf2), a.y, k.y);
        float e0, e1, e2, e3;
        unpack2(y[c], e0, e1);
        unpack2(y[c + 1], e2, e3);
        mx[0] = fmaxf(mx[0], fmaxf(e0, e1));
        mx[1] = fmaxf(mx[1], fmaxf(e2, e3));
      }
      const float mt = fmaxf(mx[0], mx[1]);
      if (!wait_pv(j - 4) || (j > 0 && !take_over(j))) {
        ok = false;
        break;
      }
      if (j == 0) mbar_arrive(&sm.ack[g]);  // (keeps the barrier's phases in step)
      // Raise the reference where the scores ask for it; the TMEM accesses are warp-collective, so the warp takes
      // the branch if any lane must.
      const float ref_before = ref;
      const bool need = mt > ref + kOver || (ref == -CUDART_INF_F && mt > ref);
      if (__any_sync(0xffffffffu, need)) {
        if (!wait_pv(j - 1)) {
          ok = false;
          break;
        }
        const float to = mt + sm.head;  // (the same in both CTAs)
        if (j > 0) rescale(ref_before, need ? to : ref_before);
        if (need) refer_to(to);
      }
      st_async_v2(hand_peer, __float_as_uint(ref_before), __float_as_uint(ref), hand_bar);
      const float minus = ref == -CUDART_INF_F ? 0.f : -ref;
      const uint64_t ref2 = pack2(minus, minus);
      uint32_t p1[16], p2[16];
      uint64_t ls[2] = {0, 0};
#pragma unroll
      for (int c = 0; c < kRows / 2; c += 2) {
        const ulonglong2 ki = *reinterpret_cast<const ulonglong2*>(&sm.col_i[sw][2 * c]);
        float e0, e1, e2, e3;
        unpack2(add2(y[c], ref2), e0, e1);
        unpack2(add2(y[c + 1], ref2), e2, e3);
        e0 = ex2_approx(e0);
        e1 = ex2_approx(e1);
        e2 = ex2_approx(e2);
        e3 = ex2_approx(e3);
        ls[0] = fma2(pack2(e0, e1), ki.x, ls[0]);
        ls[1] = fma2(pack2(e2, e3), ki.y, ls[1]);
        split_p(e0, e1, e2, e3, p1[c / 2], p2[c / 2]);
      }
      {
        float s0, s1;
        unpack2(add2(ls[0], ls[1]), s0, s1);
        l += s0 + s1;
      }
      const uint32_t pa = tmem + lane_addr + kPCol + 32 * g;
      tmem_st16(pa, p1);
      tmem_st16(pa + 16, p2);
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(&sm.p_full[g]);
      // ... and to the other CTA: head h's row of 64 + 64 bytes.
      if (i >= 1 && !__all_sync(0xffffffffu, mbar_wait_cluster(&sm.pb_free[g ^ 1], (uint32_t)(((i - 1) >> 1) & 1), abort_flag, status, 337))) {
        ok = false;
        break;
      }
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        st_async_v4(pb_peer + sw128_offset((uint32_t)h, (uint32_t)c), p1[4 * c], p1[4 * c + 1], p1[4 * c + 2], p1[4 * c + 3], pb_bar);
        st_async_v4(pb_peer + sw128_offset((uint32_t)h, (uint32_t)c + 4), p2[4 * c], p2[4 * c + 1], p2[4 * c + 2], p2[4 * c + 3], pb_bar);
      }
      last_own = i;
    }
    // The last tile is the other CTA's: the group whose tile would be next allows its PV.
    if (ok && J > 0 && (J & 1) == half && ((J >> 1) & 1) == g) ok = wait_pv(J - 4) && take_over(J);
    // The other CTA is done with this group's P (its commits arrive in this CTA's shared memory).
    if (ok && last_own >= 0)
      ok = __all_sync(0xffffffffu, mbar_wait_cluster(&sm.pb_free[g], (uint32_t)((last_own >> 1) & 1), abort_flag, status, 338));
    // Every PV completed: that of this group's last tile first (of J - 1 - 4 by a wait for J - 1 alone nothing is known).
    if (ok && J > 0 && ((last_own >= 0 && !wait_pv(2 * last_own + half)) || !wait_pv(J - 1))) ok = false;
    sm.l_g[g][h] = l;
    sm.m_g[g][h] = ref;
    {
      const uint32_t bar = mapa_shared(smem_u32(&sm.ex_full), peer);
      st_async_b32(mapa_shared(smem_u32(&sm.l_g[2 + g][h]), peer), __float_as_uint(l), bar);
      st_async_b32(mapa_shared(smem_u32(&sm.m_g[2 + g][h]), peer), __float_as_uint(ref), bar);
      if (sw == 0 && lane == 0) mbar_arrive_expect_tx(&sm.ex_full, kPeerSum);
    }
    ok = __all_sync(0xffffffffu, mbar_wait_cluster(&sm.ex_full, 0, abort_flag, status, 339)) && ok;
    if (!ok && lane == 0) sm.epi_bad = 1;
    __syncwarp();
    cluster_arrive_relaxed();
    named_bar_sync(1, 2 * kGroup);
    tc_fence_after();
    const bool fin = !sm.epi_bad;
    // The last reference (it only grows) is what O refers to.
    const float fin_ref = fmaxf(fmaxf(sm.m_g[0][h], sm.m_g[1][h]), fmaxf(sm.m_g[2][h], sm.m_g[3][h]));
    float den = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float li = sm.l_g[i][h];
      if (li != 0.f) den += li * exp2f(sm.m_g[i][h] - fin_ref);
    }
    const bool any = fin_ref != -CUDART_INF_F || den != den;  // some candidate counted (or the row is NaN)
    ref = fin_ref;
    const float sl = h < P.H ? P.sink[h] * 1.4426950408889634f : -CUDART_INF_F;
    float f;                                   // what O is multiplied by
    if (P.splits == 1) {
      den += exp2f(sl - ref);
      f = any ? (1.f / 256.f) / den : 0.f;
    } else {
      // A partial refers to its own maximum; split 0's denominator holds the sink, and refers to the
      // sink if that is larger (+inf too: the sink then has all of the weight). A padding query has neither.
      f = 1.f / 256.f;
      if (sp == 0 && Tw > 0 && sl != -CUDART_INF_F) {
        const float r = fmaxf(ref, sl);
        const float w = any ? exp2f(ref - r) : 0.f;
        den = (den != 0.f ? den * w : 0.f) + exp2f(sl == r ? 0.f : sl - r);
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
      // Rows are staged in shared memory (in place of the tiles: every gather and MMA completed), 16 bytes apart
      // against bank conflicts; each warp then sends off the rows of its quadrant, half of them, whole.
      const bool wide = P.splits > 1 || P.out_is_f32;
      const uint32_t row_bytes = wide ? 1024 : 512;
      uint8_t* srow = base + (size_t)h * (row_bytes + 16);
#pragma unroll 1
      for (int cc = 0; cc < 4; ++cc) {
        const int lc = 128 * g + 32 * cc, col0 = 256 * half + lc;
        uint32_t o[32];
        tmem_ld32(tmem + lane_addr + kOCol + lc, o);
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
        if (wide) {
          float4* s4 = reinterpret_cast<float4*>(srow + 4 * lc);
#pragma unroll
          for (int c = 0; c < 8; ++c) s4[c] = make_float4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
        } else {
          uint4* s4 = reinterpret_cast<uint4*>(srow + 2 * lc);
#pragma unroll
          for (int c = 0; c < 4; ++c)
            s4[c] = make_uint4(pack_bf16(v[8 * c], v[8 * c + 1]), pack_bf16(v[8 * c + 2], v[8 * c + 3]),
                               pack_bf16(v[8 * c + 4], v[8 * c + 5]), pack_bf16(v[8 * c + 6], v[8 * c + 7]));
        }
      }
      named_bar_sync(1, 2 * kGroup);
      const long long at = (long long)(P.splits > 1 ? item : qi) * P.H * 512 + 256 * half;
      uint4* out = reinterpret_cast<uint4*>(P.splits > 1 ? static_cast<void*>(P.part_o) : P.out);
      const int r0 = 32 * quad + 16 * g, r1 = min(P.H, r0 + 16);
      if (wide) {
        for (int r = r0; r < r1; ++r) {
          const uint4* src = reinterpret_cast<const uint4*>(base + (size_t)r * 1040);
          uint4* dst = out + (at + (long long)r * 512) / 4;
          dst[lane] = src[lane];
          dst[32 + lane] = src[32 + lane];
        }
      } else {
#pragma unroll 4
        for (int r = r0; r < r1; ++r)
          out[(at + (long long)r * 512) / 8 + lane] = reinterpret_cast<const uint4*>(base + (size_t)r * 528)[lane];
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kPvWarp8) tmem_dealloc(tmem, 512);
  // Every role arrived when it was done with the other CTA's shared memory, and saw to it that what the other
  // CTA sends here had come: relaxed, so that the outputs need not have landed.
  __syncwarp();
  cluster_wait();
}

size_t attn8_smem_bytes() { return 1024 + kTileBytes + kQ2Bytes + sizeof(Smem8); }

}  // namespace csa
