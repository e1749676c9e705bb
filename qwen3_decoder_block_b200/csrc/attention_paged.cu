// Causal grouped-query attention of a ragged batch's new tokens over a paged KV cache:
//   o_t = sum_p w_p V_p,  w = softmax_p(q_t K_p / sqrt(128)),  p <= ctx + t,
// for every query head of a KV group. Two forms: the decode form below (every sequence brings
// at most one token; the K/V stream bounds it) and the chunk form further down.
#include <mutex>
#include "paged.cuh"
#include "internal.h"

namespace q3 {

int make_tmap_2d(CUtensorMap* map, const void* base, long long rows, long long cols, long long ld, int box_rows);
int make_tmap_3d(CUtensorMap* map, const void* base, long long inner, long long mid, long long outer,
                 long long mid_stride_bytes, long long outer_stride_bytes, int box_inner, int box_mid, int box_outer);
int make_tmap_bytes(CUtensorMap* map, const void* base, long long rows, long long ld, int box_rows);

namespace {

constexpr int kD = 128;
constexpr int kTileK = 128;                // keys per tile
constexpr int kMaxCtas = 256;              // grid bound
constexpr int kPartFloats = kD + 2;        // one query row's partial: o[128], running max, sum
constexpr float kScaleLog2 = 0.12751743074380304f;  // log2(e) / sqrt(128)
constexpr float kRescaleThreshold = 8.0f;
constexpr uint32_t kTile8 = 128 * 128;     // [128 rows][128 bytes], 128-byte swizzle: 16 KB

// Where a CTA's share of the work list starts (written by the plan kernel, so that a CTA finds
// it with one load).
struct __align__(32) CtaStart {
  long long units;  // all units of the call
  int b, g, j;      // sequence, KV group and tile of its first unit
  int n_keys;       // keys of that row
};

struct PagedAttn {
  PagedBatch pb;
  KvPages kv;
  int n_tokens, max_q, Hq, o_f16;
  const uint16_t* q;
  long long ldq;
  uint16_t* out;
  long long ldo;
  long long* plan;   // [B + 1] work-unit prefix of the sequences
  CtaStart* start;   // [n_cta]
  int n_cta;         // CTAs of the attention kernel
  int* counters;     // merge counters
  float* part;       // partial results
  uint8_t* q8;       // decode form, e4m3 pages: the queries' e4m3 terms [B][Hkv][2G][128]
  float* q8_scale;   // [B][Hq]
  int* err;
};

// ----------------------------------------------------------------------------
// The work list. A sequence's work is counted in units (decode form: 128-key tiles of its
// Hkv rows; chunk form: see chunk_units); plan[b] is the unit at which sequence b starts,
// plan[B] all units, and CTA c of n takes units [c U / n, (c + 1) U / n): the same share
// for every CTA whatever the lengths. A sequence that cannot be served holds no units and
// is reported.
// ----------------------------------------------------------------------------
__device__ __forceinline__ bool paged_seq_ok(const PagedAttn& a, int b, int* n_q, int* ctx, int* err) {
  const int q0 = a.pb.q_start[b], q1 = a.pb.q_start[b + 1], c = a.pb.ctx_len[b];
  *n_q = q1 - q0;
  *ctx = c;
  if (q0 < 0 || q1 < q0 || q1 > a.n_tokens || q1 - q0 > a.max_q || c < 0) {
    record_error(err, kErrInvalid);
    return false;
  }
  if (q1 > q0 && (((long long)c + (q1 - q0) - 1) >> a.kv.page_shift) >= a.pb.max_pages) {
    record_error(err, kErrCapacity);
    return false;
  }
  return true;
}

// CTA holding unit t when U units are divided among n CTAs as [c U / n, (c + 1) U / n).
__device__ __forceinline__ int cta_of(long long t, long long U, int n) { return (int)(((t + 1) * n - 1) / U); }
// Whether CTA c's range is empty (only when U < n).
__device__ __forceinline__ bool cta_empty(int c, long long U, int n) { return U * c / n == U * (c + 1) / n; }

// First unit of CTA c's range.
__device__ __forceinline__ long long share(long long U, int c, int n) {
  return U < (1 << 22) ? (long long)((unsigned)U * (unsigned)c / (unsigned)n) : U * c / n;  // c, n <= 256
}

constexpr int kPlanThreads = 256;
constexpr int kPlanShared = 1024;  // sequences whose prefix is also kept in shared memory

// Exclusive prefix sums of v over the block, in order of the threads; *total: the block's sum.
__device__ __forceinline__ long long block_prefix(long long v, long long* wsum, long long* total) {
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  long long x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) wsum[wid] = x;
  __syncthreads();
  long long before = 0, all = 0;
  for (int w = 0; w < kPlanThreads / 32; ++w) {
    if (w < wid) before += wsum[w];
    all += wsum[w];
  }
  __syncthreads();
  *total = all;
  return before + x - v;
}

}  // namespace

// Decode form, before the attention: block 0 writes the work list and clears the merge
// counters; with e4m3 pages the other blocks split each query head (one per warp) into two
// e4m3 terms, q = 2^e (t1 + t2 / 16): t1 keeps 4 significant bits, the remainder of a bf16
// value (8 bits) fits the 4 of t2 exactly, down to 2^-14 of the head's largest value, below
// which the error stays under 2^-23 of that value.
__global__ void __launch_bounds__(kPlanThreads) paged_decode_prep_kernel(const PagedAttn a) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int B = a.pb.B, Hkv = a.kv.Hkv;
  if (blockIdx.x == 0) {
    __shared__ long long wsum[kPlanThreads / 32];
    __shared__ long long plan_s[kPlanShared];
    long long carry = 0;
    for (int base = 0; base < B; base += kPlanThreads) {
      const int b = base + (int)threadIdx.x;
      long long v = 0, total;
      int n_q, ctx;
      if (b < B && paged_seq_ok(a, b, &n_q, &ctx, a.err) && n_q > 0)
        v = (long long)Hkv * ((ctx + kTileK) / kTileK);
      const long long at = block_prefix(v, wsum, &total);
      if (b < B) a.plan[b] = carry + at;
      if (b < kPlanShared) plan_s[b] = carry + at;
      carry += total;
    }
    const long long* plan = B <= kPlanShared ? plan_s : a.plan;
    if (threadIdx.x == 0) a.plan[B] = carry;
    for (int i = threadIdx.x; i < B * Hkv; i += kPlanThreads) a.counters[i] = 0;
    __syncthreads();
    for (int c = threadIdx.x; c < a.n_cta; c += kPlanThreads) {
      CtaStart s;
      s.units = carry;
      s.b = s.g = s.j = s.n_keys = 0;
      const long long t = share(carry, c, a.n_cta);
      if (t < share(carry, c + 1, a.n_cta)) {
        int lo = 0, hi = B - 1;  // the last sequence that starts at or before unit t
        while (lo < hi) {
          const int mid = (lo + hi + 1) / 2;
          if (plan[mid] <= t) lo = mid; else hi = mid - 1;
        }
        s.b = lo;
        s.n_keys = a.pb.ctx_len[lo] + 1;
        const int nt = (s.n_keys + kTileK - 1) / kTileK, at = (int)(t - plan[lo]);
        s.g = at / nt;
        s.j = at % nt;
      }
      a.start[c] = s;
    }
    return;
  }
  const long long row = (long long)(blockIdx.x - 1) * (kPlanThreads / 32) + (threadIdx.x >> 5);
  const int b = (int)(row / a.Hq), h = (int)(row % a.Hq);
  if (b >= B) return;
  int n_q, ctx;
  if (!paged_seq_ok(a, b, &n_q, &ctx, nullptr) || n_q == 0) return;
  const int G = a.Hq / Hkv, g = h / G, j = h % G;
  const uint2 u = *reinterpret_cast<const uint2*>(a.q + a.pb.q_start[b] * a.ldq + (long long)h * kD + 4 * lane);
  float x[4] = {bf16_lo(u.x), bf16_hi(u.x), bf16_lo(u.y), bf16_hi(u.y)};
  const float mx = warp_max(fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3]))));
  // the largest value scaled into [128, 256): 2^-e exact, a power of two in the normal range
  const int ex = (int)((__float_as_uint(mx) >> 23) & 0xff);
  const int e = min(max(ex - 127 - 7, -119), 119);
  const float down = __uint_as_float((uint32_t)(127 - e) << 23), up = __uint_as_float((uint32_t)(127 + e) << 23);
  uint32_t t1 = 0, t2 = 0;
#pragma unroll
  for (int i = 0; i < 4; i += 2) {
    const float s0 = x[i] * down, s1 = x[i + 1] * down;
    const uint16_t p = pack_e4m3x2(s0, s1);
    const float2 f = e4m3x2_to_f32x2(p);
    t1 |= (uint32_t)p << (8 * i);
    t2 |= (uint32_t)pack_e4m3x2((s0 - f.x) * 16.f, (s1 - f.y) * 16.f) << (8 * i);
  }
  uint8_t* dst = a.q8 + (((long long)b * Hkv + g) * 2 * G + j) * kD + 4 * lane;
  *reinterpret_cast<uint32_t*>(dst) = t1;
  *reinterpret_cast<uint32_t*>(dst + G * kD) = t2;
  // a head with an infinity or a NaN: every score of it becomes NaN
  if (lane == 0) a.q8_scale[row] = ex == 255 ? __uint_as_float(0x7fc00000u) : up;
}

// ============================================================================
// Decode form. The 128-key tiles of every (sequence, KV group) row form one list that is
// divided evenly among persistent CTAs. Both products of a tile are tcgen05 MMAs with the
// cache on the 128-row side and the group's G query heads as columns:
//   S^T[key][j] = sum_d K[key][d] q_j[d]        A = K tile (K-major),  B = q (K-major)
//   O^T[d][j]  += sum_key V[key][d] P[j][key]   A = V tile (MN-major), B = P (K-major)
// so K and V go from the pages to the tensor core as they are: bf16 pages with kind::f16,
// e4m3 pages with kind::f8f6f4, never widened in shared memory. What e4m3 operands would
// cost in precision is bought back in the columns, which are nearly free here: q enters as
// two e4m3 terms (exact for bf16 queries) and P as three, each 16 times finer than the last
// (P scaled so that the running maximum is 2^5 to 2^8 of e4m3's 448: relative error 2^-12, or
// 2^-23 of the row's largest weight, finer than bf16), in columns [t G, t G + G) of term t.
// Two TMA warps fill rings of K and of V tiles, one box per page; one warp issues S, one P.V; two sets of softmax warps take alternate tiles,
// a thread owning one key (S) and one head dim (O). A row that spans CTAs leaves partials; the last of them to arrive merges
// them in CTA order, so the result does not depend on which one that is, and nobody waits.
// ============================================================================
template <int G, bool FP8>
struct DecodeCfg {
  static constexpr int kQTerms = FP8 ? 2 : 1, kPTerms = FP8 ? 3 : 1;
  static constexpr int kCols = (kPTerms * G + 15) / 16 * 16;          // MMA N
  static constexpr int kHeadWarps = G >= 8 ? 2 : 1;                   // softmax warps of a set per lane quarter
  static constexpr int kSetWarps = 4 * kHeadWarps;
  static constexpr int kSoftmaxWarps = 2 * kSetWarps;                 // set X takes the CTA's tiles of parity X
  static constexpr int kThreads = 32 * (kSoftmaxWarps + 4);
  static constexpr int kStages = FP8 ? (G == 16 ? 5 : 6) : 3;
  static constexpr uint32_t kKV = FP8 ? kTile8 : 2 * kTile8;          // K or V of one tile
  static constexpr uint32_t kQB = (FP8 ? 1 : 2) * kCols * 128;        // q of one row
  static constexpr uint32_t kOffV = kStages * kKV;                    // K ring, V ring, q of two rows
  static constexpr uint32_t kOffQ = 2 * kStages * kKV;
  static constexpr uint32_t kPB = (FP8 ? 1 : 2) * kCols * 128;        // one P buffer
  static constexpr uint32_t kOffP = kOffQ + 2 * kQB;
  static constexpr uint32_t kOffRed = kOffP + 2 * kPB;                // per set: maxima [2][4][16], sums [4][16]
  static constexpr uint32_t kOffX = kOffRed + 2 * 3 * 64 * 4;         // set 1's row: o [G][128], m [16], l [16]
  static constexpr uint32_t kOffBar = kOffX + G * kD * 4 + 2 * 16 * 4;
  static constexpr uint32_t kSmem = kOffBar + (4 * kStages + 14) * 8 + 16 + 1024;
  // tensor memory: S of set 0 and 1, O of set 0 and 1
  static constexpr uint32_t kTmem = 4 * kCols <= 64 ? 64 : (4 * kCols <= 128 ? 128 : 256);
};

// Walk over the (sequence, group) rows that meet this CTA's tiles: tiles [j0, j1) of the row.
struct RowWalk {
  const long long* plan;
  const int* ctx_len;
  int B, Hkv, b, g, j0, j1, nt, n_keys;
  int left;  // the CTA's tiles from the current row on
  __device__ RowWalk(const PagedAttn& a, const CtaStart& s, int n_tiles)
      : plan(a.plan), ctx_len(a.pb.ctx_len), B(a.pb.B), Hkv(a.kv.Hkv), b(s.b), g(s.g), j0(s.j), n_keys(s.n_keys),
        left(n_tiles) {
    set_row();
  }
  __device__ void set_row() {
    nt = (n_keys + kTileK - 1) / kTileK;
    j1 = min(nt, j0 + left);
  }
  __device__ bool valid() const { return left > 0; }
  __device__ void next() {
    left -= j1 - j0;
    if (left <= 0) return;
    j0 = 0;
    if (++g == Hkv) {
      g = 0;
      do { ++b; } while (b < B && plan[b + 1] == plan[b]);
      n_keys = ctx_len[b < B ? b : B - 1] + 1;
    }
    set_row();
  }
};

// One arrival for a warp, once all its lanes are here (32 arrivals on one barrier would queue
// up at one shared-memory word).
__device__ __forceinline__ void arrive_warp(uint64_t* bar, int lane) {
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}

__device__ __forceinline__ void named_bar(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// Element base + hh * GH + jj of a register array for the warp's head group hh (run time)
// and head jj (a constant after unrolling): constant indices keep the array in registers.
template <int HW, int GH, int N>
__device__ __forceinline__ float pick(const uint32_t (&a)[N], int base, int hh, int jj) {
  uint32_t v = a[base + jj];
#pragma unroll
  for (int h = 1; h < HW; ++h)
    if (hh == h) v = a[base + h * GH + jj];
  return __uint_as_float(v);
}
// N columns of 32 lanes from tensor memory (N a multiple of 16), waited for.
template <int N>
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, uint32_t (&r)[N]) {
  uint32_t v[N / 16][16];
#pragma unroll
  for (int c = 0; c < N / 16; ++c) tmem_ld16(taddr + 16 * c, v[c]);
#pragma unroll
  for (int c = 0; c < N / 16; ++c) tmem_wait_ld_regs16(v[c]);
#pragma unroll
  for (int c = 0; c < N / 16; ++c)
#pragma unroll
    for (int i = 0; i < 16; ++i) r[16 * c + i] = v[c][i];
}

// Maximum (MAX) or sum over the 32 lanes of each of G per-lane values: log2(G) halving
// exchanges, each leaving a lane the half of the heads its lane bit selects, then a butterfly
// over the other lane bits. Lane l ends with head l >> (5 - log2 G).
template <int G, bool MAX>
__device__ __forceinline__ float reduce_heads(const float (&x)[G], int lane) {
  float a[G];
#pragma unroll
  for (int j = 0; j < G; ++j) a[j] = x[j];
#pragma unroll
  for (int half = G / 2, bit = 16; half >= 1; half >>= 1, bit >>= 1) {
    const bool upper = (lane & bit) != 0;
#pragma unroll
    for (int k = 0; k < half; ++k) {
      const float send = upper ? a[k] : a[k + half];
      const float keep = upper ? a[k + half] : a[k];
      const float got = __shfl_xor_sync(0xffffffffu, send, bit);
      a[k] = MAX ? fmaxf(keep, got) : keep + got;
    }
  }
#pragma unroll
  for (int o = 16 / G; o > 0; o >>= 1) {
    const float got = __shfl_xor_sync(0xffffffffu, a[0], o);
    a[0] = MAX ? fmaxf(a[0], got) : a[0] + got;
  }
  return a[0];
}

template <int G, bool FP8>
__global__ void __launch_bounds__(DecodeCfg<G, FP8>::kThreads, 1)
    attn_paged_decode_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                             const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmK16,
                             const __grid_constant__ CUtensorMap tmV16, const PagedAttn a) {
  using C = DecodeCfg<G, FP8>;
  constexpr int SW = C::kSoftmaxWarps, XW = C::kSetWarps, HW = C::kHeadWarps, GH = G / HW, NC = C::kCols, NS = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + C::kOffBar);  // [NS] K (and q) loaded
  uint64_t* k_empty = k_full + NS;                                    // [NS] ... consumed
  uint64_t* v_full = k_full + 2 * NS;                                 // [NS] V loaded
  uint64_t* v_empty = k_full + 3 * NS;                                // [NS] ... consumed
  uint64_t* q_full = k_full + 4 * NS;  // [2] q of a row loaded
  uint64_t* q_empty = q_full + 2;      // [2] ... consumed
  uint64_t* s_full = q_full + 4;       // [2] scores of set X ready
  uint64_t* s_empty = s_full + 2;  // [2] scores of set X read
  uint64_t* p_full = s_full + 4;   // [2] P of set X written (and its O rescaled)
  uint64_t* pv_done = s_full + 6;  // [2] P.V of set X's tile complete
  uint64_t* drain = s_full + 8;    // [2] an issuer's MMAs complete
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(s_full + 10);
  volatile int* s_abort = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* s_last = s_abort + 1;  // this CTA merges the row
  int* err = a.err;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 4 * NS + 4; ++i) mbar_init(&k_full[i], 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1); mbar_init(&s_empty[i], XW);
      mbar_init(&p_full[i], XW); mbar_init(&pv_done[i], 1); mbar_init(&drain[i], 1);
    }
    *s_abort = 0;
    fence_barrier_init();
  }
  // Unused rows of the Q and P operand tiles are never written: clear all of them once.
  for (int i = threadIdx.x; i < (int)((2 * C::kQB + 2 * C::kPB) / 16); i += blockDim.x)
    reinterpret_cast<uint4*>(smem + C::kOffQ)[i] = make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();
  if (threadIdx.x == 32 * SW) {
    tma_prefetch_desc(&tmQ); tma_prefetch_desc(&tmK); tma_prefetch_desc(&tmV);
    tma_prefetch_desc(&tmK16); tma_prefetch_desc(&tmV16);
  }
  if (warp == SW + 1) { tmem_alloc(tmem_slot, C::kTmem); tmem_relinquish(); }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t tmO = tmem + 2 * NC;
  pdl_wait();
  pdl_trigger();
  const int Hkv = a.kv.Hkv, n_cta = (int)gridDim.x;
  const CtaStart start = a.start[blockIdx.x];
  const long long U = start.units;
  const int n_tiles = (int)(share(U, blockIdx.x + 1, n_cta) - share(U, blockIdx.x, n_cta));

  if (warp == SW || warp == SW + 3) {
    // -------------------------------------------------- TMA producers: K and q; V
    // One box per page of a tile, min(page, 128) keys each (16 in a row's last tile, so that
    // nothing past its last 16 keys is read), twice for the two 64-dim halves of bf16. Lane i
    // finds box i's page, a tile ahead, and its cache row; the rows go round by shuffles and
    // one elected lane issues the copies (about 30 clocks each; found by that lane alone, or
    // issued from a lane loop, a box costs about 180 or 95).
    const bool is_v = warp == SW + 3;
    const CUtensorMap* map = is_v ? &tmV : &tmK;
    const CUtensorMap* map16 = is_v ? &tmV16 : &tmK16;
    uint64_t* full = is_v ? v_full : k_full;
    uint64_t* empty = is_v ? v_empty : k_empty;
    uint8_t* ring = smem + (is_v ? C::kOffV : 0);
    const int shift = a.kv.page_shift, in_page = (1 << shift) - 1, box_shift = min(shift, 7);
    const int n_pages = a.kv.n_pages, rows_all = (n_pages * Hkv) << shift;
    RowWalk w(a, start, n_tiles);
    int j = w.j0;
    // the page of this lane's box in tile j of row w (0 where it has none)
    auto look_up = [&]() {
      const int left = w.n_keys - j * kTileK;
      const int off = lane << (left >= kTileK ? box_shift : 4);
      if (off >= kTileK || off >= left) return 0;
      return __ldg(a.pb.table + (long long)w.b * a.pb.max_pages + ((j * kTileK + off) >> shift));
    };
    int page = w.valid() ? look_up() : 0;
    int st = 0, done = 0, rows_seen = 0;
    uint32_t phase = 0;
    bool ok = true, new_row = true;
    while (w.valid()) {
      const int b = w.b, g = w.g, k0 = j * kTileK, left = w.n_keys - k0;
      const bool tail = left < kTileK;
      const int bs = tail ? 4 : box_shift;
      const int n = tail ? (left + 15) >> 4 : kTileK >> bs;
      // a bad page reads as zeros: behind the tensor map's last row
      const bool in = (unsigned)page < (unsigned)n_pages;
      if (!in) record_error(err, kErrInvalid);
      const int my_row = in ? ((page * Hkv + g) << shift) + ((k0 + (lane << bs)) & in_page) : rows_all;
      int row[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) row[i] = __shfl_sync(0xffffffffu, my_row, i);
      if (!is_v && new_row) {
        const int qs = rows_seen & 1;
        ok = !*s_abort && mbar_wait(&q_empty[qs], (uint32_t)((rows_seen >> 1) & 1) ^ 1u, err);
        if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
        const int tok = FP8 ? 0 : a.pb.q_start[b];
        uint8_t* dst = smem + C::kOffQ + qs * C::kQB;
        if (elect_one()) {
          mbar_arrive_expect_tx(&q_full[qs], C::kQTerms * G * 128 * (FP8 ? 1 : 2));
          if (FP8) {
            tma_load_2d(dst, &tmQ, &q_full[qs], 0, (b * Hkv + g) * 2 * G);
          } else {
            tma_load_3d(dst, &tmQ, &q_full[qs], 0, g * G, tok);
            tma_load_3d(dst + NC * 128, &tmQ, &q_full[qs], 64, g * G, tok);
          }
        }
        __syncwarp();
        ++rows_seen;
      }
      new_row = ++j == w.j1;
      if (new_row) {
        w.next();
        j = w.j0;
      }
      if (w.valid()) page = look_up();
      ok = !*s_abort && mbar_wait(&empty[st], phase ^ 1u, err);
      if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
      uint8_t* dst = ring + st * C::kKV;
      if (elect_one()) {
        const CUtensorMap* m = tail ? map16 : map;
        mbar_arrive_expect_tx(&full[st], (n << bs) * 128 * (FP8 ? 1 : 2));
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (i < n) {
            tma_load_2d(dst + ((i << bs) * 128), m, &full[st], 0, row[i]);
            if (!FP8) tma_load_2d(dst + kTile8 + ((i << bs) * 128), m, &full[st], 64, row[i]);
          }
      }
      __syncwarp();
      ++done;
      if (++st == NS) { st = 0; phase ^= 1u; }
    }
    if (!ok) {
      *s_abort = 1;
      // let the copies still in flight land before the CTA exits
      for (int i = done > NS ? done - NS : 0; i < done; ++i) mbar_wait(&full[i % NS], (uint32_t)((i / NS) & 1), err);
      if (!is_v)
        for (int i = rows_seen > 2 ? rows_seen - 2 : 0; i < rows_seen; ++i)
          mbar_wait(&q_full[i & 1], (uint32_t)((i >> 1) & 1), err);
    }
  } else if (warp == SW + 1) {
    if (lane == 0) {
      // ------------------------------------------------------------ S issuer: S = K q
      constexpr uint32_t idesc = FP8 ? idesc_e4m3_f32(128, NC, 0, 0) : idesc_bf16_f32(128, NC, 0, 0);
      int tc = 0, st = 0, rows_seen = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (RowWalk w(a, start, n_tiles); w.valid() && ok; w.next(), ++rows_seen) {
        const int qs = rows_seen & 1;
        if (*s_abort || !mbar_wait(&q_full[qs], (uint32_t)((rows_seen >> 1) & 1), err)) { ok = false; break; }
        const uint32_t sQ = smem_u32(smem + C::kOffQ + qs * C::kQB);
        for (int j = w.j0; j < w.j1; ++j, ++tc) {
          const int sb = tc & 1;
          if (*s_abort || !mbar_wait(&k_full[st], phase, err)) { ok = false; break; }
          if (tc >= 2 && (*s_abort || !mbar_wait(&s_empty[sb], (uint32_t)(((tc - 2) >> 1) & 1), err))) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sK = smem_u32(smem + st * C::kKV);
          if (FP8) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_e4m3_ss(tmem + NC * sb, sdesc_kmajor_sw128(sK) + 2 * kk, sdesc_kmajor_sw128(sQ) + 2 * kk, idesc,
                          kk ? 1u : 0u);
          } else {
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              mma_bf16_ss(tmem + NC * sb, sdesc_kmajor_sw128(sK + (kk >> 2) * kTile8) + 2 * (kk & 3),
                          sdesc_kmajor_sw128(sQ + (kk >> 2) * NC * 128) + 2 * (kk & 3), idesc, kk ? 1u : 0u);
          }
          mma_commit(&s_full[sb]);
          mma_commit(&k_empty[st]);
          if (++st == NS) { st = 0; phase ^= 1u; }
        }
        if (ok) mma_commit(&q_empty[qs]);
      }
      if (!ok) *s_abort = 1;
      mma_commit(&drain[0]);  // every MMA completes before the tensor memory is released
      mbar_wait(&drain[0], 0, err);
    }
  } else if (warp == SW + 2) {
    if (lane == 0) {
      // -------------------------------------------- P.V issuer: O^T += V^T P^T
      constexpr uint32_t idesc = FP8 ? idesc_e4m3_f32(128, NC, 1, 0) : idesc_bf16_f32(128, NC, 1, 0);
      int tc = 0, st = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (RowWalk w(a, start, n_tiles); w.valid() && ok; w.next()) {
        const int jb = w.j0, je = w.j1;
        for (int j = jb; j < je; ++j, ++tc) {
          const int pb = tc & 1;
          if (*s_abort || !mbar_wait(&v_full[st], phase, err) ||
              !mbar_wait(&p_full[pb], (uint32_t)((tc >> 1) & 1), err)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sV = smem_u32(smem + C::kOffV + st * C::kKV);
          const uint32_t sP = smem_u32(smem + C::kOffP + pb * C::kPB), tO = tmO + pb * NC;
          if (FP8) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)  // 32 keys an instruction
              mma_e4m3_ss(tO, sdesc_mnmajor_sw128(sV + kk * 32 * 128, kTile8, 1024), sdesc_kmajor_sw128(sP) + 2 * kk,
                          idesc, (j < jb + 2 && kk == 0) ? 0u : 1u);
          } else {
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)  // 16 keys an instruction
              mma_bf16_ss(tO, sdesc_mnmajor_sw128(sV + kk * 16 * 128, kTile8, 1024),
                          sdesc_kmajor_sw128(sP + (kk >> 2) * NC * 128) + 2 * (kk & 3), idesc,
                          (j < jb + 2 && kk == 0) ? 0u : 1u);
          }
          mma_commit(&pv_done[pb]);
          mma_commit(&v_empty[st]);
          if (++st == NS) { st = 0; phase ^= 1u; }
        }
      }
      if (!ok) *s_abort = 1;
      mma_commit(&drain[1]);
      mbar_wait(&drain[1], 0, err);
    }
  } else {
    // -------------------------------------------------------------------- softmax
    // warp (set X, quarter qd, half hh): key / head dim t of lanes [32 qd, 32 qd + 32), heads
    // [j0, j0 + GH) of the group, the CTA's tiles of parity X. Two sets, each with its own S,
    // P, O, maxima and sums, keep two tiles' softmax chains in flight (one chain takes longer
    // than an e4m3 tile's share of the memory bandwidth); a row's two halves meet at its end.
    const int X = warp / XW, qd = warp & 3, hh = (warp % XW) >> 2, j0 = hh * GH;
    const int t = qd * 32 + lane;
    const uint32_t lanes = (uint32_t)(qd * 32) << 16;
    const uint32_t tS = tmem + lanes + NC * X, tO = tmO + lanes + NC * X;
    float* red_max = reinterpret_cast<float*>(smem + C::kOffRed) + X * 3 * 64;  // [2][4][16]
    float* red_sum = red_max + 2 * 64;                                          // [4][16]
    float* x_o = reinterpret_cast<float*>(smem + C::kOffX);                     // [G][128]
    float* x_ml = x_o + G * kD;                                                 // m [16], l [16]
    uint8_t* p_buf = smem + C::kOffP + X * C::kPB;
    // e4m3: the running maximum is kept 5 below the scores', so that P lies in (0, 2^8]
    constexpr float kShift = FP8 ? 5.f : 0.f;
    constexpr int kSCols = (C::kQTerms * G + 15) / 16 * 16;
    int tc0 = 0;  // the CTA's tiles before the current row
    int u = 0;    // the set's tiles so far
    bool ok = true;
    for (RowWalk w(a, start, n_tiles); w.valid(); w.next()) {
      const int b = w.b, g = w.g, bg = b * Hkv + g;
      const int jb = w.j0, je = w.j1;
      float factor[GH], m_run[GH], l_part[GH];
#pragma unroll
      for (int jj = 0; jj < GH; ++jj) {
        factor[jj] = FP8 ? kScaleLog2 * a.kv.k_scale[g] * a.q8_scale[b * a.Hq + g * G + j0 + jj] : kScaleLog2;
        m_run[jj] = -INFINITY;
        l_part[jj] = 0.f;
      }
      const int j_first = jb + ((tc0 ^ X) & 1);
      for (int j = j_first; j < je; j += 2, ++u) {
        const int nk = min(kTileK, w.n_keys - j * kTileK);
        const uint32_t par = (uint32_t)(u & 1);
        ok = ok && !*s_abort && mbar_wait(&s_full[X], par, err);
        ok = __all_sync(0xffffffffu, ok);
        uint32_t sv[kSCols];
#pragma unroll
        for (int i = 0; i < kSCols; ++i) sv[i] = 0u;
        if (ok) {
          tc_fence_after();
          tmem_ld_cols<kSCols>(tS, sv);
        }
        tc_fence_before();
        arrive_warp(&s_empty[X], lane);
        float s[GH];
#pragma unroll
        for (int jj = 0; jj < GH; ++jj) {
          float x = pick<HW, GH>(sv, 0, hh, jj);
          if (FP8) x += pick<HW, GH>(sv, FP8 ? G : 0, hh, jj) * 0.0625f;
          s[jj] = (ok && t < nk) ? x * factor[jj] : -INFINITY;
        }
        // tile maximum per head: the warp's 32 keys, then the 4 quarters
        float* rm = red_max + par * 64;
        {
          const float wm = reduce_heads<GH, true>(s, lane);
          if ((lane & (32 / GH - 1)) == 0) rm[qd * 16 + j0 + lane / (32 / GH)] = wm;
        }
        named_bar(1 + X, 32 * XW);
        float alpha[GH], p[GH];
        bool rescale = false;
#pragma unroll
        for (int jj = 0; jj < GH; ++jj) {
          const int hd = j0 + jj;
          const float mt = fmaxf(fmaxf(rm[hd], rm[16 + hd]), fmaxf(rm[32 + hd], rm[48 + hd])) - kShift;
          alpha[jj] = 1.f;
          if (mt > m_run[jj] + (kRescaleThreshold - kShift) || m_run[jj] == -INFINITY) {
            alpha[jj] = (m_run[jj] == -INFINITY) ? 0.f : ex2_approx(m_run[jj] - mt);
            m_run[jj] = mt;
            rescale = true;
          }
          p[jj] = (t < nk && m_run[jj] != -INFINITY) ? ex2_approx(s[jj] - m_run[jj]) : 0.f;
          l_part[jj] = l_part[jj] * alpha[jj] + p[jj];
        }
        // the set's P buffer and O are free once the P.V of its previous tile is complete
        if (u >= 1) {
          ok = ok && !*s_abort && mbar_wait(&pv_done[X], par ^ 1u, err);
          ok = __all_sync(0xffffffffu, ok);
        }
        if (ok) {
          tc_fence_after();
          if (j > j_first && rescale) {  // uniform within the warp: its lanes hold the same maxima
            uint32_t ov[NC];
            tmem_ld_cols<NC>(tO, ov);
#pragma unroll
            for (int term = 0; term < C::kPTerms; ++term)
#pragma unroll
              for (int jj = 0; jj < GH; ++jj)
                tmem_st1(tO + term * G + j0 + jj, __float_as_uint(pick<HW, GH>(ov, term * G, hh, jj) * alpha[jj]));
            tmem_wait_st();
          }
          // P[row][t] into the K-major B tile: row term * G + head, 128-byte swizzle
          if (FP8) {
            uint8_t* pb = p_buf + (t & 15);
#pragma unroll
            for (int jj = 0; jj < GH; jj += 2) {
              float r0 = p[jj], r1 = jj + 1 < GH ? p[jj + 1 < GH ? jj + 1 : jj] : 0.f;
#pragma unroll
              for (int term = 0; term < 3; ++term) {
                const uint16_t e = pack_e4m3x2(r0, r1);
                const int row = term * G + j0 + jj;
                pb[row * 128 + (((t >> 4) ^ (row & 7)) << 4)] = (uint8_t)e;
                if (jj + 1 < GH) pb[(row + 1) * 128 + (((t >> 4) ^ ((row + 1) & 7)) << 4)] = (uint8_t)(e >> 8);
                if (term < 2) {
                  const float2 f = e4m3x2_to_f32x2(e);
                  r0 = (r0 - f.x) * 16.f;
                  r1 = (r1 - f.y) * 16.f;
                }
              }
            }
          } else {
            uint8_t* pb = p_buf + (t >> 6) * NC * 128 + (t & 7) * 2;
            const int chunk = (t & 63) >> 3;
#pragma unroll
            for (int jj = 0; jj < GH; ++jj) {
              const int row = j0 + jj;
              *reinterpret_cast<uint16_t*>(pb + row * 128 + ((chunk ^ (row & 7)) << 4)) = to_bf16_bits(p[jj]);
            }
          }
          // keys past the last one: zero their V rows (0 * NaN would poison O)
          if (hh == 0 && nk < kTileK) {
            const int tc = tc0 + (j - jb), st = tc % NS;
            ok = __all_sync(0xffffffffu, mbar_wait(&v_full[st], (uint32_t)((tc / NS) & 1), err));
            if (ok && t >= nk) {
              uint4* v = reinterpret_cast<uint4*>(smem + C::kOffV + st * C::kKV + t * 128);
#pragma unroll
              for (int c = 0; c < 8; ++c) {
                v[c] = make_uint4(0, 0, 0, 0);
                if (!FP8) v[c + kTile8 / 16] = make_uint4(0, 0, 0, 0);
              }
            }
          }
          fence_proxy_async_smem();
        }
        tc_fence_before();
        arrive_warp(&p_full[X], lane);
      }
      tc0 += je - jb;
      // end of the row's tiles in this CTA: O from tensor memory, the sums of the quarters
      const bool any = j_first < je;
      uint32_t ov[NC];
#pragma unroll
      for (int i = 0; i < NC; ++i) ov[i] = 0u;
      if (any) {
        ok = ok && !*s_abort && mbar_wait(&pv_done[X], (uint32_t)((u - 1) & 1), err);
        ok = __all_sync(0xffffffffu, ok);
        if (ok) {
          tc_fence_after();
          tmem_ld_cols<NC>(tO, ov);
        }
      }
      {
        const float ws = reduce_heads<GH, false>(l_part, lane);
        if ((lane & (32 / GH - 1)) == 0) red_sum[qd * 16 + j0 + lane / (32 / GH)] = ws;
      }
      named_bar(1 + X, 32 * XW);
      float o[GH], l[GH];
#pragma unroll
      for (int jj = 0; jj < GH; ++jj) {
        const int hd = j0 + jj;
        o[jj] = pick<HW, GH>(ov, 0, hh, jj);
        if (FP8) {
          o[jj] += pick<HW, GH>(ov, FP8 ? G : 0, hh, jj) * 0.0625f;
          o[jj] += pick<HW, GH>(ov, FP8 ? 2 * G : 0, hh, jj) * 0.00390625f;
        }
        l[jj] = red_sum[hd] + red_sum[16 + hd] + red_sum[32 + hd] + red_sum[48 + hd];
      }
      // set 1 hands its half of the row to set 0, which carries on with the whole
      if (X == 1) {
#pragma unroll
        for (int jj = 0; jj < GH; ++jj) {
          x_o[(j0 + jj) * kD + t] = o[jj];
          if (t == jj) {
            x_ml[j0 + jj] = m_run[jj];
            x_ml[16 + j0 + jj] = l[jj];
          }
        }
      }
      named_bar(3, 32 * SW);
      if (X == 0) {
#pragma unroll
        for (int jj = 0; jj < GH; ++jj) {
          const int hd = j0 + jj;
          const float m1 = x_ml[hd], M = fmaxf(m_run[jj], m1);
          const float w0 = m_run[jj] == M ? 1.f : ex2_approx(m_run[jj] - M), w1 = m1 == M ? 1.f : ex2_approx(m1 - M);
          o[jj] = o[jj] * w0 + x_o[hd * kD + t] * w1;
          l[jj] = l[jj] * w0 + x_ml[16 + hd] * w1;
          m_run[jj] = M;
        }
      }
      named_bar(3, 32 * SW);
      if (X == 1) continue;
      const float vs = FP8 ? a.kv.v_scale[g] : 1.f;
      uint16_t* out_row = a.out + a.pb.q_start[b] * a.ldo + (long long)g * G * kD + t;
      if (jb == 0 && je == w.nt) {
        if (ok) {
#pragma unroll
          for (int jj = 0; jj < GH; ++jj)
            out_row[(j0 + jj) * kD] = to_op_bits(a.o_f16 != 0, o[jj] * vs / l[jj]);
        }
        continue;
      }
      // a row shared by several CTAs: partial to slot row + CTA (unique: rows and CTA ranges
      // are both in tile order), then count it
      const long long rs = a.plan[b] + (long long)g * w.nt;
      const int c_first = cta_of(rs, U, n_cta), c_last = cta_of(rs + w.nt - 1, U, n_cta);
      const bool sparse = U < n_cta;  // one tile a CTA, some CTAs without any
      float* row_part = a.part + (long long)bg * G * kPartFloats;
      const long long stride = (long long)G * kPartFloats;
      {
        float* mine = row_part + blockIdx.x * stride;
#pragma unroll
        for (int jj = 0; jj < GH; ++jj) {
          float* dst = mine + (j0 + jj) * kPartFloats;
          __stcg(dst + t, o[jj]);
          if (t == jj) {
            __stcg(dst + kD, m_run[jj]);
            __stcg(dst + kD + 1, l[jj]);
          }
        }
      }
      named_bar(1, 32 * XW);  // every thread's stores precede the count
      if (threadIdx.x == 0) {
        const int n = sparse ? w.nt : c_last - c_first + 1;
        *s_last = ok && atom_add_acq_rel_gpu(&a.counters[bg], 1) == n - 1;
      }
      named_bar(1, 32 * XW);
      if (!*s_last) continue;
      // all partials are there: lane i weighs CTA c_first + i, 32 at a time, then the thread
      // sums its dim of them, kBatch loads in flight (one at a time they cost 8 us a row)
      constexpr int kBatch = 32 / GH;
      const float* part = row_part + j0 * kPartFloats;
      auto piece = [&](int c) { return c <= c_last && !(sparse && cta_empty(c, U, n_cta)); };
      float M[GH], m0[GH], l0[GH], L[GH], acc[GH];
#pragma unroll
      for (int jj = 0; jj < GH; ++jj) {
        m0[jj] = -INFINITY;
        l0[jj] = L[jj] = acc[jj] = 0.f;
        if (piece(c_first + lane)) {
          m0[jj] = __ldcg(part + (c_first + lane) * stride + jj * kPartFloats + kD);
          l0[jj] = __ldcg(part + (c_first + lane) * stride + jj * kPartFloats + kD + 1);
        }
        M[jj] = m0[jj];
      }
      for (int c = c_first + 32 + lane; c <= c_last; c += 32)
        if (piece(c))
#pragma unroll
          for (int jj = 0; jj < GH; ++jj) M[jj] = fmaxf(M[jj], __ldcg(part + c * stride + jj * kPartFloats + kD));
#pragma unroll
      for (int jj = 0; jj < GH; ++jj) M[jj] = warp_max(M[jj]);
      for (int base = c_first; base <= c_last; base += 32) {
        const int c = base + lane;
        float wgt[GH];
#pragma unroll
        for (int jj = 0; jj < GH; ++jj) {
          if (base != c_first) {
            m0[jj] = piece(c) ? __ldcg(part + c * stride + jj * kPartFloats + kD) : -INFINITY;
            l0[jj] = piece(c) ? __ldcg(part + c * stride + jj * kPartFloats + kD + 1) : 0.f;
          }
          wgt[jj] = piece(c) ? exp2f(m0[jj] - M[jj]) : 0.f;
          L[jj] += l0[jj] * wgt[jj];
        }
        const int n = min(32, c_last - base + 1);
        for (int i0 = 0; i0 < n; i0 += kBatch) {
          float v[kBatch][GH];
#pragma unroll
          for (int i = 0; i < kBatch; ++i)
#pragma unroll
            for (int jj = 0; jj < GH; ++jj)
              v[i][jj] = i0 + i < n ? __ldcg(part + (base + i0 + i) * stride + jj * kPartFloats + t) : 0.f;
#pragma unroll
          for (int i = 0; i < kBatch; ++i)
#pragma unroll
            for (int jj = 0; jj < GH; ++jj) {
              const float wi = __shfl_sync(0xffffffffu, wgt[jj], (i0 + i) & 31);
              acc[jj] += wi != 0.f ? v[i][jj] * wi : 0.f;  // the slot of an empty CTA holds anything
            }
        }
      }
#pragma unroll
      for (int jj = 0; jj < GH; ++jj)
        out_row[(j0 + jj) * kD] = to_op_bits(a.o_f16 != 0, acc[jj] * vs / warp_sum(L[jj]));
    }
    if (!ok) *s_abort = 1;
  }

  tc_fence_before();
  __syncthreads();
  if (warp == SW + 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmem);
  }
}

// One warp per (token, query head): 32 keys at a time, a lane's dot product per key, online
// softmax over the warp, then 4 output dims per lane.
template <bool FP8>
__global__ void __launch_bounds__(128) attn_paged_simple_kernel(const PagedBatch pb, const KvPages kv, int Hq,
                                                                int n_tokens, int max_q, const uint16_t* q,
                                                                long long ldq, uint16_t* out, long long ldo,
                                                                int o_f16, int* err) {
  __shared__ float qs[4][128];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const long long item = (long long)blockIdx.x * 4 + w;
  const int tok = (int)(item / Hq), h = (int)(item % Hq);
  if (tok >= n_tokens) return;
  const int b = paged_seq_of(pb, tok, lane);
  if (b >= pb.B) return;
  const int start = pb.q_start[b], t = tok - start, n_q = pb.q_start[b + 1] - start, ctx = pb.ctx_len[b];
  if (t < 0 || ctx < 0 || n_q > max_q || start < 0) {
    if (lane == 0) record_error(err, kErrInvalid);
    return;
  }
  if (((long long)ctx + n_q - 1) >> kv.page_shift >= pb.max_pages) {
    if (lane == 0) record_error(err, kErrCapacity);
    return;
  }
  const int g = h / (Hq / kv.Hkv);
  const float ks = FP8 ? kv.k_scale[g] : 1.f, vs = FP8 ? kv.v_scale[g] : 1.f;
  const uint2 qv = *reinterpret_cast<const uint2*>(q + tok * ldq + (long long)h * 128 + 4 * lane);
  qs[w][4 * lane] = bf16_lo(qv.x);
  qs[w][4 * lane + 1] = bf16_hi(qv.x);
  qs[w][4 * lane + 2] = bf16_lo(qv.y);
  qs[w][4 * lane + 3] = bf16_hi(qv.y);
  __syncwarp();
  const int n = ctx + t + 1;
  const float scale = 0.12751743074380304f * ks;  // log2(e) / sqrt(128)
  float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
  for (int k0 = 0; k0 < n; k0 += 32) {
    const int p = k0 + lane;
    float s = -INFINITY;
    long long cell = -1;
    if (p < n) {
      cell = paged_row(pb, kv, b, p, err);
      s = 0.f;
      if (cell >= 0) {
        cell += (long long)g << kv.page_shift;
        if (FP8) {
          const uint4* r = reinterpret_cast<const uint4*>(kv.k + cell * 128);
          for (int i = 0; i < 8; ++i) {
            const uint4 u = r[i];
            const uint32_t x[4] = {u.x, u.y, u.z, u.w};
            for (int j = 0; j < 8; ++j) {
              const float2 f = e4m3x2_to_f32x2((uint16_t)(x[j >> 1] >> (16 * (j & 1))));
              s += f.x * qs[w][16 * i + 2 * j] + f.y * qs[w][16 * i + 2 * j + 1];
            }
          }
        } else {
          const uint4* r = reinterpret_cast<const uint4*>(kv.k + cell * 256);
          for (int i = 0; i < 16; ++i) {
            const uint4 u = r[i];
            const uint32_t x[4] = {u.x, u.y, u.z, u.w};
            for (int j = 0; j < 4; ++j)
              s += bf16_lo(x[j]) * qs[w][8 * i + 2 * j] + bf16_hi(x[j]) * qs[w][8 * i + 2 * j + 1];
          }
        }
        s *= scale;
      }
    }
    const float mn = fmaxf(m, warp_max(s));
    const float pr = s == -INFINITY ? 0.f : exp2f(s - mn);
    const float alpha = m == -INFINITY ? 0.f : exp2f(m - mn);
    m = mn;
    l = l * alpha + warp_sum(pr);
    for (int i = 0; i < 4; ++i) o[i] *= alpha;
    const int nk = min(32, n - k0);
    for (int j = 0; j < nk; ++j) {
      const float pj = __shfl_sync(0xffffffffu, pr, j);
      const long long c = __shfl_sync(0xffffffffu, cell, j);
      if (c < 0) continue;
      if (FP8) {
        const uint32_t u = *reinterpret_cast<const uint32_t*>(kv.v + c * 128 + 4 * lane);
        const float2 a = e4m3x2_to_f32x2((uint16_t)u), e = e4m3x2_to_f32x2((uint16_t)(u >> 16));
        o[0] += pj * a.x; o[1] += pj * a.y; o[2] += pj * e.x; o[3] += pj * e.y;
      } else {
        const uint2 u = *reinterpret_cast<const uint2*>(kv.v + c * 256 + 8 * lane);
        o[0] += pj * bf16_lo(u.x); o[1] += pj * bf16_hi(u.x); o[2] += pj * bf16_lo(u.y); o[3] += pj * bf16_hi(u.y);
      }
    }
  }
  const float inv = vs / l;
  uint2 r;
  r.x = pack_op_x2(o_f16 != 0, o[0] * inv, o[1] * inv);
  r.y = pack_op_x2(o_f16 != 0, o[2] * inv, o[3] * inv);
  *reinterpret_cast<uint2*>(out + tok * ldo + (long long)h * 128 + 4 * lane) = r;
}

// ----------------------------------------------------------------------------
// Host side
// ----------------------------------------------------------------------------
namespace {

// Scratch of a call, in order: work list, CTA starts, merge counters, partials, e4m3 query terms and scales.
struct Scratch {
  size_t plan, start, counters, part, q8, q8_scale, bytes;
};
size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }
Scratch scratch_of(int B, int Hq, int Hkv, int max_q) {
  Scratch s;
  s.plan = 0;
  s.start = s.plan + up256(((size_t)B + 1) * sizeof(long long));
  s.counters = s.start + kMaxCtas * sizeof(CtaStart);
  const bool decode = max_q == 1;
  const int G = Hq / Hkv;
  s.part = s.counters + up256(decode ? (size_t)B * Hkv * sizeof(int) : 256);
  s.q8 = s.part + up256(decode ? ((size_t)B * Hkv + kMaxCtas) * G * kPartFloats * sizeof(float) : 256);
  s.q8_scale = s.q8 + up256(decode ? (size_t)B * Hq * 2 * kD : 0);
  s.bytes = s.q8_scale + up256(decode ? (size_t)B * Hq * sizeof(float) : 0);
  return s;
}

// Tensor maps of the pages: full-tile boxes of min(page, 128) rows and 16-row boxes.
int page_maps(const KvPages& kv, CUtensorMap* k, CUtensorMap* v, CUtensorMap* k16, CUtensorMap* v16) {
  const long long rows = ((long long)kv.n_pages * kv.Hkv) << kv.page_shift;
  const int box = kv.page_shift < 7 ? 1 << kv.page_shift : kTileK;
  auto make = [&](CUtensorMap* m, const void* p, int r) {
    return kv.fp8 ? make_tmap_bytes(m, p, rows, kD, r) : make_tmap_2d(m, p, rows, kD, kD, r);
  };
  if (make(k, kv.k, box) || make(v, kv.v, box) || make(k16, kv.k, 16) || make(v16, kv.v, 16)) {
    set_last_error("attention_paged: cannot encode the pages' tensor maps");
    return -6;
  }
  return 0;
}

template <int G, bool FP8>
int launch_decode(const PagedAttn& a, const CUtensorMap& tmQ, cudaStream_t s) {
  using C = DecodeCfg<G, FP8>;
  CUtensorMap tmK, tmV, tmK16, tmV16;
  if (page_maps(a.kv, &tmK, &tmV, &tmK16, &tmV16)) return -6;
  auto kernel = attn_paged_decode_kernel<G, FP8>;
  if (ensure_smem_attr(reinterpret_cast<const void*>(kernel), C::kSmem)) return -6;
  q3_launch(kernel, a.n_cta, C::kThreads, C::kSmem, s, tmQ, tmK, tmV, tmK16, tmV16, a);
  return 0;
}

int attention_decode(const PagedAttn& a, cudaStream_t s) {
  const int G = a.Hq / a.kv.Hkv, B = a.pb.B;
  CUtensorMap tmQ;
  if (a.kv.fp8 ? make_tmap_bytes(&tmQ, a.q8, (long long)B * a.Hq * 2, kD, 2 * G)
               : make_tmap_3d(&tmQ, a.q, kD, a.Hq, a.n_tokens, kD * 2, a.ldq * 2, 64, G, 1)) {
    set_last_error("attention_paged: cannot encode the query tensor map");
    return -6;
  }
  const long long split = a.kv.fp8 ? ((long long)B * a.Hq + kPlanThreads / 32 - 1) / (kPlanThreads / 32) : 0;
  q3_launch(paged_decode_prep_kernel, (unsigned)(1 + split), kPlanThreads, 0, s, a);
  switch (G * 2 + a.kv.fp8) {
    case 2: return launch_decode<1, false>(a, tmQ, s);
    case 3: return launch_decode<1, true>(a, tmQ, s);
    case 4: return launch_decode<2, false>(a, tmQ, s);
    case 5: return launch_decode<2, true>(a, tmQ, s);
    case 8: return launch_decode<4, false>(a, tmQ, s);
    case 9: return launch_decode<4, true>(a, tmQ, s);
    case 16: return launch_decode<8, false>(a, tmQ, s);
    case 17: return launch_decode<8, true>(a, tmQ, s);
    case 32: return launch_decode<16, false>(a, tmQ, s);
    case 33: return launch_decode<16, true>(a, tmQ, s);
  }
  set_last_error("attention_paged: %d query heads per KV group is not supported (1, 2, 4, 8 or 16)", G);
  return -2;
}

}  // namespace

size_t paged_attention_bytes(int B, int Hq, int Hkv, int max_q) { return scratch_of(B, Hq, Hkv, max_q).bytes; }

int launch_attention_paged(const uint16_t* q, long long ldq, int n_tokens, int max_q, const PagedBatch& pb,
                           const KvPages& kv, int Hq, void* scratch, uint16_t* out, long long ldo, int* err,
                           cudaStream_t s, bool o_f16) {
  const Scratch off = scratch_of(pb.B, Hq, kv.Hkv, max_q);
  uint8_t* base = static_cast<uint8_t*>(scratch);
  PagedAttn a;
  a.pb = pb;
  a.kv = kv;
  a.n_tokens = n_tokens; a.max_q = max_q; a.Hq = Hq; a.o_f16 = o_f16 ? 1 : 0;
  a.q = q; a.ldq = ldq;
  a.out = out; a.ldo = ldo;
  a.plan = reinterpret_cast<long long*>(base + off.plan);
  a.start = reinterpret_cast<CtaStart*>(base + off.start);
  a.n_cta = num_sms() < kMaxCtas ? num_sms() : kMaxCtas;
  a.counters = reinterpret_cast<int*>(base + off.counters);
  a.part = reinterpret_cast<float*>(base + off.part);
  a.q8 = base + off.q8;
  a.q8_scale = reinterpret_cast<float*>(base + off.q8_scale);
  a.err = err;
  int rc = 0;
  if (max_q == 1) {
    rc = attention_decode(a, s);
  } else {
    const long long blocks = ((long long)n_tokens * Hq + 3) / 4;
    if (blocks >= (1ll << 31)) {
      set_last_error("attention_paged: %d tokens exceed the grid limit", n_tokens);
      return -2;
    }
    q3_launch(kv.fp8 ? attn_paged_simple_kernel<true> : attn_paged_simple_kernel<false>, (unsigned)blocks, 128, 0, s,
              pb, kv, Hq, n_tokens, max_q, q, ldq, out, ldo, o_f16 ? 1 : 0, err);
  }
  if (rc) return rc;
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) {
    set_last_error("attention_paged launch failed: %s", cudaGetErrorString(e));
    return -6;
  }
  return 0;
}

}  // namespace q3
