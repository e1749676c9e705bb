// Causal grouped-query attention of a ragged batch's new tokens over a paged KV cache:
//   o_t = sum_p w_p V_p,  w = softmax_p(q_t K_p / sqrt(128)),  p <= ctx + t,
// for every query head of a KV group. Two forms: the decode form below (every sequence brings
// at most one token; the K/V stream bounds it) and the chunk form further down.
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
constexpr float kTinyWeight = 7.888609e-31f;  // 2^-100
constexpr float kMinFactor = 1.1754944e-38f;  // 2^-126
constexpr uint32_t kTile8 = 128 * 128;     // [128 rows][128 bytes], 128-byte swizzle: 16 KB

// Where a CTA's share of the work list starts (written by the plan kernel, so that a CTA finds
// it with one load). Its alignment is the one that a workspace has to have.
struct __align__(16) CtaStart {
  long long units;  // all units of the call
  int b, g, j;      // sequence, KV group and tile (decode form) or item (chunk form) of its first unit
  int rest;         // decode form: keys of that row; chunk form: units of the item before the CTA's
};

struct ChunkMeta;

struct PagedAttn {
  PagedBatch pb;
  KvPages kv;
  int n_tokens, max_q, Hq, g_shift, o_f16;  // g_shift: log2 of the query heads per KV group
  int min_q;         // chunk form: it takes the sequences with at least this many new tokens
  const uint16_t* q;
  long long ldq;
  uint16_t* out;
  long long ldo;
  long long* plan;   // [B + 1] work-unit prefix of the sequences
  CtaStart* start;   // [n_cta]
  int n_cta;         // CTAs of the attention kernel
  int* counters;     // decode form: merge counters [B * Hkv]
  ChunkMeta* meta;   // chunk form: [n_cta][2]
  float* part;       // partial results
  uint8_t* q8;       // decode form, e4m3 pages: the queries' e4m3 terms [B][Hkv][2G][128]
  float* q8_scale;   // [B][Hq]
  int* err;
};

// ----------------------------------------------------------------------------
// The work list. A sequence's work is counted in units (decode form: 128-key tiles of its
// Hkv rows; chunk form: see ChunkSeq); plan[b] is the unit at which sequence b starts,
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

namespace {

// Sum over p < P of the KV tiles of pair p, floor((ctx + min((p + 1) s, n_q) - 1) / 128) + 1, for
// s = 2 TQ (a power of two, 16 to 256) and P <= ceil(n_q / s).
__device__ __forceinline__ long long pair_tiles(int ctx, int n_q, int s, int P) {
  if (P <= 0) return 0;
  long long cut = 0;
  if ((long long)P * s > n_q) {  // the last pair ends with the sequence
    cut = ((long long)ctx + n_q - 1) / kTileK + 1;
    --P;
  }
  const long long a = (long long)ctx + s - 1;
  if (s >= kTileK) return cut + P * (a / kTileK + 1) + (long long)(s / kTileK) * P * (P - 1) / 2;
  const int r = kTileK / s;  // floor((a + p s) / 128) = floor((floor(a / s) + p) / r)
  auto F = [&](long long n) {
    const long long m = n / r;
    return r * (m * (m - 1) / 2) + m * (n - m * r);
  };
  return cut + P + F(a / s + P) - F(a / s);
}
struct ChunkSeq {
  int n_q, ctx, s, pairs, odd;
  long long head_units;  // of one KV head
  __device__ ChunkSeq(int nq, int c, int g_shift) : n_q(nq), ctx(c), s(256 >> g_shift) {
    const int tiles = (int)((((long long)nq << g_shift) + 127) >> 7);
    pairs = tiles >> 1;
    odd = tiles & 1;
    head_units = 2 * pair_tiles(ctx, n_q, s, pairs) + (odd ? ((long long)ctx + n_q - 1) / kTileK + 1 : 0);
  }
};

// One form's work list, CTA starts and cleared counters, by one block.
template <bool CHUNK>
__device__ void write_plan(const PagedAttn& a, long long* wsum, long long* plan_s) {
  const int B = a.pb.B, Hkv = a.kv.Hkv;
  long long carry = 0;
  for (int base = 0; base < B; base += kPlanThreads) {
    const int b = base + (int)threadIdx.x;
    long long v = 0, total;
    int n_q, ctx;
    if (b < B && paged_seq_ok(a, b, &n_q, &ctx, a.err)) {
      if (CHUNK) {
        if (n_q >= a.min_q) v = Hkv * ChunkSeq(n_q, ctx, a.g_shift).head_units;
      } else if (n_q == 1) {
        v = (long long)Hkv * ((ctx + kTileK) / kTileK);
      }
    }
    const long long at = block_prefix(v, wsum, &total);
    if (b < B) a.plan[b] = carry + at;
    if (b < kPlanShared) plan_s[b] = carry + at;
    carry += total;
  }
  const long long* plan = B <= kPlanShared ? plan_s : a.plan;
  if (threadIdx.x == 0) a.plan[B] = carry;
  if (!CHUNK)
    for (int i = threadIdx.x; i < B * Hkv; i += kPlanThreads) a.counters[i] = 0;
  __syncthreads();
  for (int c = threadIdx.x; c < a.n_cta; c += kPlanThreads) {
    CtaStart s;
    s.units = carry;
    s.b = s.g = s.j = s.rest = 0;
    const long long t = share(carry, c, a.n_cta);
    if (t < share(carry, c + 1, a.n_cta)) {
      int lo = 0, hi = B - 1;  // the last sequence that starts at or before unit t
      while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (plan[mid] <= t) lo = mid; else hi = mid - 1;
      }
      s.b = lo;
      if (!CHUNK) {
        s.rest = a.pb.ctx_len[lo] + 1;
        const int nt = (s.rest + kTileK - 1) / kTileK, at = (int)(t - plan[lo]);
        s.g = at / nt;
        s.j = at % nt;
      } else {
        const ChunkSeq q(a.pb.q_start[lo + 1] - a.pb.q_start[lo], a.pb.ctx_len[lo], a.g_shift);
        long long r = t - plan[lo];
        s.g = (int)(r / q.head_units);
        r -= s.g * q.head_units;
        lo = 0;
        hi = q.pairs + q.odd - 1;  // the last item that starts at or before unit r of the head
        while (lo < hi) {
          const int mid = (lo + hi + 1) / 2;
          if (2 * pair_tiles(q.ctx, q.n_q, q.s, mid) <= r) lo = mid; else hi = mid - 1;
        }
        s.j = lo;
        s.rest = (int)(r - 2 * pair_tiles(q.ctx, q.n_q, q.s, lo));
      }
    }
    a.start[c] = s;
  }
}

}  // namespace

// Before the attention: block 0 writes the decode form's work list, block 1 the chunk form's
// (`forms`: bit 0 and 1). With e4m3 pages the other blocks split each query head of the decode
// form (one per warp) into two e4m3 terms, q = 2^e (t1 + t2 / 16): t1 keeps 4 significant
// bits, the remainder of a bf16 value (8 bits) fits the 4 of t2 exactly, down to 2^-13 of
// the head's largest value, below which the error is at most 2^-21 of that value.
__global__ void __launch_bounds__(kPlanThreads) paged_plan_kernel(const PagedAttn a, const PagedAttn chunk, int forms) {
  pdl_wait();
  pdl_trigger();
  __shared__ long long wsum[kPlanThreads / 32];
  __shared__ long long plan_s[kPlanShared];
  if (blockIdx.x == 0) {
    if (forms & 1) write_plan<false>(a, wsum, plan_s);
    return;
  }
  if (blockIdx.x == 1) {
    if (forms & 2) write_plan<true>(chunk, wsum, plan_s);
    return;
  }
  const int lane = threadIdx.x & 31;
  const int B = a.pb.B, Hkv = a.kv.Hkv;
  const long long row = (long long)(blockIdx.x - 2) * (kPlanThreads / 32) + (threadIdx.x >> 5);
  const int b = (int)(row / a.Hq), h = (int)(row % a.Hq);
  if (b >= B) return;
  int n_q, ctx;
  if (!paged_seq_ok(a, b, &n_q, &ctx, nullptr) || n_q != 1) return;
  const int G = 1 << a.g_shift, g = h >> a.g_shift, j = h & (G - 1);
  const uint2 u = *reinterpret_cast<const uint2*>(a.q + a.pb.q_start[b] * a.ldq + (long long)h * kD + 4 * lane);
  float x[4] = {bf16_lo(u.x), bf16_hi(u.x), bf16_lo(u.y), bf16_hi(u.y)};
  const float mx = warp_max(fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3]))));
  // the largest value scaled into [128, 256): 2^-e exact, a power of two in the normal range
  const int ex = (int)((__float_as_uint(mx) >> 23) & 0xff);
  const int e = min(max(ex - 127 - 7, -119), 120);
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
// two e4m3 terms (exact for bf16 values down to 2^-13 of the head's largest) and P as three, each 16 times finer than the last
// (P scaled so that the running maximum is 2^5 to 2^8 of e4m3's 448: relative error 2^-12, or
// 2^-23 of the row's largest weight, finer than bf16), in columns [t G, t G + G) of term t. With
// bf16 pages P enters as two bf16 terms, its leading 8 bits and the rest (2^-15), in the same way.
// Two TMA warps fill rings of K and of V tiles, one box per page; one warp issues S, one P.V; two sets of softmax warps take alternate tiles,
// a thread owning one key (S) and one head dim (O). A row that spans CTAs leaves partials; the last of them to arrive merges
// them in CTA order, so the result does not depend on which one that is, and nobody waits.
// ============================================================================
template <int G, bool FP8>
struct DecodeCfg {
  static constexpr int kQTerms = FP8 ? 2 : 1, kPTerms = FP8 ? 3 : 2;
  static constexpr int kSCols = (kQTerms * G + 15) / 16 * 16;         // N of S
  static constexpr int kCols = (kPTerms * G + 15) / 16 * 16;          // N of P.V
  static constexpr int kHeadWarps = G >= 8 ? 2 : 1;                   // softmax warps of a set per lane quarter
  static constexpr int kSetWarps = 4 * kHeadWarps;
  static constexpr int kSoftmaxWarps = 2 * kSetWarps;                 // set X takes the CTA's tiles of parity X
  static constexpr int kThreads = 32 * (kSoftmaxWarps + 4);
  static constexpr int kStages = FP8 ? (G == 16 ? 5 : 6) : 3;
  static constexpr uint32_t kKV = FP8 ? kTile8 : 2 * kTile8;          // K or V of one tile
  static constexpr uint32_t kQB = (FP8 ? 1 : 2) * kSCols * 128;       // q of one row
  static constexpr uint32_t kOffV = kStages * kKV;                    // K ring, V ring, q of two rows
  static constexpr uint32_t kOffQ = 2 * kStages * kKV;
  static constexpr uint32_t kPB = (FP8 ? 1 : 2) * kCols * 128;        // one P buffer
  static constexpr uint32_t kOffP = kOffQ + 2 * kQB;
  static constexpr uint32_t kOffRed = kOffP + 2 * kPB;                // per set: maxima [2][4][16], sums [4][16]
  static constexpr uint32_t kOffX = kOffRed + 2 * 3 * 64 * 4;         // set 1's row: o [G][128], m [16], l [16]
  static constexpr uint32_t kOffBar = kOffX + G * kD * 4 + 2 * 16 * 4;
  static constexpr uint32_t kSmem = kOffBar + (4 * kStages + 14) * 8 + 16 + 1024;
  // tensor memory: S of set 0 and 1, O of set 0 and 1
  static constexpr uint32_t kTmem = 2 * (kSCols + kCols) <= 64 ? 64 : (2 * (kSCols + kCols) <= 128 ? 128 : 256);
};

// Walk over the (sequence, group) rows that meet this CTA's tiles: tiles [j0, j1) of the row.
struct RowWalk {
  const long long* plan;
  const int* ctx_len;
  int B, Hkv, b, g, j0, j1, nt, n_keys;
  int left;  // the CTA's tiles from the current row on
  __device__ RowWalk(const PagedAttn& a, const CtaStart& s, int n_tiles)
      : plan(a.plan), ctx_len(a.pb.ctx_len), B(a.pb.B), Hkv(a.kv.Hkv), b(s.b), g(s.g), j0(s.j), n_keys(s.rest),
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
  // predicated, not branched: the lanes stay together
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.eq.s32 p, %1, 0;\n\t@p mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}" ::"r"(
          smem_u32(bar)),
      "r"(lane)
      : "memory");
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

template <int G, bool FP8>
__global__ void __launch_bounds__(DecodeCfg<G, FP8>::kThreads, 1)
    attn_paged_decode_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                             const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmK16,
                             const __grid_constant__ CUtensorMap tmV16, const PagedAttn a) {
  using C = DecodeCfg<G, FP8>;
  constexpr int SW = C::kSoftmaxWarps, XW = C::kSetWarps, HW = C::kHeadWarps, GH = G / HW, NC = C::kCols, SC = C::kSCols,
                NS = C::kStages;
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
  const uint32_t tmO = tmem + 2 * SC;
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
            tma_load_3d(dst + SC * 128, &tmQ, &q_full[qs], 64, g * G, tok);
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
    if (elect_one()) {
      // ------------------------------------------------------------ S issuer: S = K q
      constexpr uint32_t idesc = FP8 ? idesc_e4m3_f32(128, SC, 0, 0) : idesc_bf16_f32(128, SC, 0, 0);
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
              mma_e4m3_ss(tmem + SC * sb, sdesc_kmajor_sw128(sK) + 2 * kk, sdesc_kmajor_sw128(sQ) + 2 * kk, idesc,
                          kk ? 1u : 0u);
          } else {
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              mma_bf16_ss(tmem + SC * sb, sdesc_kmajor_sw128(sK + (kk >> 2) * kTile8) + 2 * (kk & 3),
                          sdesc_kmajor_sw128(sQ + (kk >> 2) * SC * 128) + 2 * (kk & 3), idesc, kk ? 1u : 0u);
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
    if (elect_one()) {
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
    const uint32_t tS = tmem + lanes + SC * X, tO = tmO + lanes + NC * X;
    float* red_max = reinterpret_cast<float*>(smem + C::kOffRed) + X * 3 * 64;  // [2][4][16]
    float* red_sum = red_max + 2 * 64;                                          // [4][16]
    float* x_o = reinterpret_cast<float*>(smem + C::kOffX);                     // [G][128]
    float* x_ml = x_o + G * kD;                                                 // m [16], l [16]
    uint8_t* p_buf = smem + C::kOffP + X * C::kPB;
    // e4m3: the running maximum is kept 5 below the scores', so that P lies in (0, 2^8]
    constexpr float kShift = FP8 ? 5.f : 0.f;
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
        ok = ok && mbar_wait_warp(&s_full[X], par, err);
        uint32_t sv[SC];
#pragma unroll
        for (int i = 0; i < SC; ++i) sv[i] = 0u;
        if (ok) {
          tc_fence_after();
          tmem_ld_cols<SC>(tS, sv);
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
          const float wm = warp_reduce_heads<GH, true>(s, lane);
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
          // (no maximum yet: every score is -inf, of weight 0, or NaN, which stays)
          p[jj] = t < nk ? ex2_approx(s[jj] - (m_run[jj] == -INFINITY ? 0.f : m_run[jj])) : 0.f;
          l_part[jj] = l_part[jj] * alpha[jj] + p[jj];
        }
        // the set's P buffer and O are free once the P.V of its previous tile is complete
        if (u >= 1) {
          ok = ok && mbar_wait_warp(&pv_done[X], par ^ 1u, err);
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
              const int row = j0 + jj, low = G + row;
              // hi is cut, not rounded, and the rest kept above 0 (by 2^-100 of the largest weight), so
              // that an infinity in V meets weights of one sign only and stays one
              const uint32_t hi = __float_as_uint(p[jj]) & 0xffff0000u;
              const float rest = fmaxf(p[jj] - __uint_as_float(hi), kTinyWeight);
              *reinterpret_cast<uint16_t*>(pb + row * 128 + ((chunk ^ (row & 7)) << 4)) = (uint16_t)(hi >> 16);
              *reinterpret_cast<uint16_t*>(pb + low * 128 + ((chunk ^ (low & 7)) << 4)) = to_bf16_bits(rest);
            }
          }
          // keys past the last one: zero their V rows (0 * NaN would poison O)
          if (hh == 0 && nk < kTileK) {
            const int tc = tc0 + (j - jb), st = tc % NS;
            ok = mbar_wait_warp(&v_full[st], (uint32_t)((tc / NS) & 1), err);
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
        ok = ok && mbar_wait_warp(&pv_done[X], (uint32_t)((u - 1) & 1), err);
        if (ok) {
          tc_fence_after();
          tmem_ld_cols<NC>(tO, ov);
        }
      }
      {
        const float ws = warp_reduce_heads<GH, false>(l_part, lane);
        if ((lane & (32 / GH - 1)) == 0) red_sum[qd * 16 + j0 + lane / (32 / GH)] = ws;
      }
      named_bar(1 + X, 32 * XW);
      float o[GH], l[GH];
#pragma unroll
      for (int jj = 0; jj < GH; ++jj) {
        const int hd = j0 + jj;
        o[jj] = pick<HW, GH>(ov, 0, hh, jj) + pick<HW, GH>(ov, G, hh, jj) * (FP8 ? 0.0625f : 1.f);
        if (FP8) o[jj] += pick<HW, GH>(ov, FP8 ? 2 * G : 0, hh, jj) * 0.00390625f;
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
      // (applied last: before the division by the sum it may overflow, folded into 1 / sum be subnormal)
      const float vs = FP8 ? a.kv.v_scale[g] : 1.f;
      uint16_t* out_row = a.out + a.pb.q_start[b] * a.ldo + (long long)g * G * kD + t;
      if (jb == 0 && je == w.nt) {
        if (ok) {
#pragma unroll
          for (int jj = 0; jj < GH; ++jj)
            out_row[(j0 + jj) * kD] = to_op_bits(a.o_f16 != 0, o[jj] / l[jj] * vs);
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
        out_row[(j0 + jj) * kD] = to_op_bits(a.o_f16 != 0, acc[jj] / warp_sum(L[jj]) * vs);
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

// ============================================================================
// Chunk form: any number of new tokens a sequence, decode tokens among them. The 128-row MMA
// tile packs TQ = 128 / G tokens x the G query heads of one KV group, so every K/V tile is
// loaded once for the group; one softmax warpgroup X (one row a thread) per S_X, P_X, O_X in
// tensor memory, two of them a CTA. An item of work is
//   pair:   two Q tiles of a sequence and KV group; warpgroup X takes Q tile X through every
//           KV tile, both Q tiles sharing the tile's loads;
//   single: the last Q tile of an odd count (all a decode token or a short chunk has);
//           warpgroup X takes every second KV tile, and warpgroup 0 joins the halves at the
//           end, reading O_1 from tensor memory (the lanes are the same).
// Work units are KV tiles (two for a pair's tile); each CTA gets the same share of the units,
// so a long context is split over the SMs as far as the batch leaves them idle, and few Q
// tiles cost no idle SM. An item that spans CTAs leaves partials (at most four a CTA), joined
// by a kernel that follows.
//
// e4m3 pages: S takes K as it is (kind::f8f6f4) against q split into two e4m3 terms of one
// scale (exact for bf16 values down to 2^-9 of the row's largest; below, off by at most 2^-16
// of it). For P.V a third warpgroup widens V to fp16 in shared memory, which is exact, and P is
// fp16 scaled to at most 2^15: 2^-11 of each weight, or 2^-31 of the row's largest, is finer
// than bf16, and one cvt widens two values.
//
// bf16 pages: V may hold any bf16, which fp16 cannot, and both operands of a product share
// their type, so P is rounded to bf16: at most 2^-8 of each weight, of random sign, beside the 2^-8 of
// the output's own rounding (0.0023 of the output's norm from the exact result, 0.0017 with an
// exact P). A second term as in the decode form would double the P.V products; the row sum takes
// P before it is rounded. So a decode token over bf16 pages gets weights of 2^-15 from the decode form
// and of 2^-8 here, where a chunk in a small batch brings it; the header says so.
// ============================================================================
namespace {

constexpr int kChunkCtas = 152;                       // grid bound (partials are sized by it)
constexpr int kChunkPart = kD * 128 + 2 * 128;        // o [32][128 rows][4 dims], m [128], l [128]

struct ChunkMeta {
  int split;   // the CTA's last item of warpgroup X goes on in other CTAs
  int c_last;  // the last of them
  int n_rows;  // valid rows of the Q tile
  int tok;     // first token row
  int g;
  int has;     // the CTA left a partial of an item that an earlier CTA began
  int pad[2];
};

}  // namespace

// Walk over the items that meet this CTA's units.
struct ChunkWalk {
  const PagedAttn& a;
  int TQ, b, g, p;
  int q0, n_q, ctx, pairs, odd;  // of the sequence
  long long before, left;        // units of the item before the CTA's range, units from there on in the range
  bool pair;
  int t0, n_keys, nk0, n;  // first token; keys of the item; KV tiles of Q tile 0 (pair), of the item
  int k0, k1;              // the CTA's KV tiles
  __device__ ChunkWalk(const PagedAttn& a_, const CtaStart& s, long long units)
      : a(a_), TQ(128 >> a_.g_shift), b(s.b), g(s.g), p(s.j), before(s.rest), left(units), k0(0), k1(0) {
    if (left > 0) {
      set_seq();
      set_item();
      if (k0 >= k1) next();
    }
  }
  __device__ bool valid() const { return left > 0; }
  __device__ void set_seq() {
    q0 = a.pb.q_start[b];
    n_q = a.pb.q_start[b + 1] - q0;
    ctx = a.pb.ctx_len[b];
    const int tiles = (int)((((long long)n_q << a.g_shift) + 127) >> 7);
    pairs = tiles >> 1;
    odd = tiles & 1;
  }
  __device__ void set_item() {
    pair = p < pairs;
    t0 = p * 2 * TQ;
    n_keys = ctx + min(t0 + (pair ? 2 : 1) * TQ, n_q);
    n = ((n_keys - 1) >> 7) + 1;
    nk0 = pair ? ((ctx + t0 + TQ - 1) >> 7) + 1 : n;
    const int w = pair ? 1 : 0;  // log2 of a tile's units
    k0 = (int)((before + w) >> w);
    k1 = (int)min((long long)n, (before + left + w) >> w);
  }
  // the next item with tiles in the range, if any
  __device__ void next() {
    do {
      left -= (pair ? 2ll : 1ll) * n - before;
      if (left <= 0) return;
      before = 0;
      if (++p >= pairs + odd) {
        p = 0;
        if (++g == a.kv.Hkv) {
          g = 0;
          do { ++b; } while (b < a.pb.B && a.plan[b + 1] == a.plan[b]);
          if (b >= a.pb.B) { left = 0; return; }
          set_seq();
        }
      }
      set_item();
    } while (k0 >= k1);
  }
  // KV tiles of warpgroup X in the CTA's range: first, step, end
  __device__ int first(int X) const { return pair ? k0 : k0 + X; }
  __device__ int step() const { return pair ? 1 : 2; }
  __device__ int end(int X) const { return pair && X == 0 ? min(k1, nk0) : k1; }
  __device__ bool any(int X) const { return first(X) < end(X); }
  // 64-key halves of tile k that warpgroup X needs (the last tile's second half may lie behind every row)
  __device__ int halves(int X, int k) const {
    const int keys = pair && X == 0 ? ctx + t0 + TQ : n_keys;
    return k * kTileK + 64 < keys ? 2 : 1;
  }
  __device__ bool loads_q(int X) const { return pair ? any(X) : X == 0; }
};

// 16 bytes of global memory, or zeros. Volatile: the compiler keeps a run of these together (it
// would sink plain loads to their uses, one latency each).
__device__ __forceinline__ uint4 ld_or_zero(const void* p, bool there) {
  uint4 v;
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %5, 0;\n\t"
      "mov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t"
      "@p ld.global.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
      : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
      : "l"(p), "r"((int)there));
  return v;
}

// A shared-memory matrix descriptor moved by `bytes` (addresses stay below 2^18, so the 14-bit
// field of 16-byte units does not overflow).
__device__ __forceinline__ uint64_t desc_step(uint64_t d, uint32_t bytes) { return d + (bytes >> 4); }

template <bool FP8>
struct ChunkCfg {
  static constexpr int kThreads = FP8 ? 512 : 384;  // softmax 0, 1; control (K, MMA 0, MMA 1, V); V widening
  // registers a thread of the softmax, control and widening warpgroups: the sum of the shares must fit
  // what the block is launched with
  static constexpr int kRegsSoftmax = FP8 ? 184 : 200, kRegsCtl = FP8 ? 72 : 88, kRegsWiden = 72;
  static constexpr int kRegBudget = (2 * kRegsSoftmax + kRegsCtl + (FP8 ? kRegsWiden : 0)) * 128;
  static constexpr uint32_t kQTile = 2 * kTile8;                  // bf16: 2 halves; e4m3: 2 terms
  static constexpr uint32_t kKTile = FP8 ? kTile8 : 2 * kTile8;
  static constexpr uint32_t kVTile = 2 * kTile8;                  // 16-bit
  // even ring depths: warpgroup X's consecutive tiles of a single item are two apart, so a
  // stage's previous tile is one that the waiting thread has seen (or lies in an item that is over)
  static constexpr int kKStages = FP8 ? 4 : 2, kVStages = 2, kRaw = FP8 ? 2 : 0;
  static constexpr uint32_t kOffK = 2 * kQTile;
  static constexpr uint32_t kOffV = kOffK + kKStages * kKTile;
  static constexpr uint32_t kOffRaw = kOffV + kVStages * kVTile;  // e4m3 V tiles as loaded
  static constexpr uint32_t kOffML = kOffRaw + kRaw * kTile8;     // m [128], l [128] of warpgroup 1; q factors [128]
  static constexpr uint32_t kOffBar = kOffML + 3 * 128 * 4;
  static constexpr uint32_t kSmem = kOffBar + 40 * 8 + 16 + 1024;
};

// Byte offset in a Q tile of 16-byte piece c (0 to 15) of a row: two halves of 128 bytes a row,
// each with the 128-byte swizzle. The next item's q is written by the warps that stage finished
// rows in the same tile, and no barrier stands between the two: all 16 pieces of a row lie in its own
// 128 bytes of either half, so that a warp touches the bytes of its 32 rows only, and its own
// __syncwarp orders them. Staged at 256 bytes a row, a warp's rows would lie on another warp's q.
__host__ __device__ constexpr uint32_t q_tile_at(int row, int c) {
  return (uint32_t)(c >> 3) * kTile8 + (uint32_t)row * 128 + (uint32_t)(((c & 7) ^ (row & 7)) << 4);
}
constexpr bool q_tile_rows_apart() {
  for (int row = 0; row < 128; ++row)
    for (int c = 0; c < 16; ++c)
      if (q_tile_at(row, c) % kTile8 / 128 != (uint32_t)row || q_tile_at(row, c) / kTile8 != (uint32_t)(c >> 3)) return false;
  return true;
}
static_assert(q_tile_rows_apart(), "a row's pieces stay in its own bytes of the Q tile");

// Tensor memory (512 columns): warpgroup X owns columns [256 X, 256 X + 256): two buffers of 64 for the
// fp32 scores of half a KV tile, each reused for its 16-bit probabilities, and O_X in the other 128. While
// the softmax works on one buffer, the tensor core does P.V from the other and the scores that
// replace it: with whole tiles in one buffer that round trip was part of every tile (4930 clocks
// a tile of a pair).
template <bool FP8>
__global__ void __launch_bounds__(ChunkCfg<FP8>::kThreads, 1)
    attn_paged_chunk_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                            const __grid_constant__ CUtensorMap tmK16, const __grid_constant__ CUtensorMap tmV16,
                            const PagedAttn a) {
  using C = ChunkCfg<FP8>;
  constexpr int NK = C::kKStages, NV = C::kVStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint64_t* q_full = bars;          // [2] Q tile X written
  uint64_t* k_full = bars + 2;      // [NK <= 4]
  uint64_t* k_empty = bars + 6;     // [NK] two arrivals a tile
  uint64_t* v_full = bars + 10;     // [NV = 2] 16-bit V tile there
  uint64_t* v_empty = bars + 12;    // [NV] two arrivals a tile
  uint64_t* raw_full = bars + 14;   // [2] e4m3 V tile loaded
  uint64_t* raw_empty = bars + 16;  // [2]
  uint64_t* s_full = bars + 18;     // [X][buffer] scores of a half tile ready
  uint64_t* p_full = bars + 22;     // [X][buffer] P written (and O_X rescaled)
  uint64_t* pv_done = bars + 26;    // [X][buffer] P.V of the half tile complete
  uint64_t* drain = bars + 30;      // [2] an issuer's MMAs complete
  // both warpgroups and both issuers are through with an item: nobody gets more than one item
  // ahead, so that no wait can take an older phase of a barrier for the one it means
  uint64_t* item_done = bars + 32;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 33);
  volatile int* s_abort = reinterpret_cast<volatile int*>(tmem_slot + 1);
  float* ml = reinterpret_cast<float*>(smem + C::kOffML);
  int* err = a.err;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 4);
      mbar_init(&v_full[i], FP8 ? 4 : 1);
      mbar_init(&v_empty[i], 2);
      mbar_init(&raw_full[i], 1);
      mbar_init(&raw_empty[i], 4);
      mbar_init(&drain[i], 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);
      mbar_init(&pv_done[i], 1);
    }
    for (int i = 0; i < NK; ++i) { mbar_init(&k_full[i], 1); mbar_init(&k_empty[i], 2); }
    mbar_init(item_done, 8 + 2);
    *s_abort = 0;
    fence_barrier_init();
  }
  if (warp == 8 && lane == 0) {
    tma_prefetch_desc(&tmK); tma_prefetch_desc(&tmV); tma_prefetch_desc(&tmK16); tma_prefetch_desc(&tmV16);
  }
  if (warp == 9) { tmem_alloc(tmem_slot, 512); tmem_relinquish(); }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
  pdl_trigger();
  const int Hkv = a.kv.Hkv, n_cta = (int)gridDim.x;
  const CtaStart start = a.start[blockIdx.x];
  const long long U = start.units;
  const long long units = share(U, blockIdx.x + 1, n_cta) - share(U, blockIdx.x, n_cta);

  if (warp >= 12) {
    // ------------------------------------------------------------ V widening (e4m3 pages)
    regs_decrease<C::kRegsWiden>();
    const int t = threadIdx.x - 384;
    int c = 0;
    bool ok = true;
    for (ChunkWalk w(a, start, units); w.valid(); w.next()) {
      for (int k = w.k0; k < w.k1; ++k, ++c) {
        const int rs = c & 1, vs = c % NV;
        const uint32_t rphase = (uint32_t)((c >> 1) & 1), vphase = (uint32_t)((c / NV) & 1);
        ok = ok && !*s_abort && mbar_wait(&raw_full[rs], rphase, err) && mbar_wait(&v_empty[vs], vphase ^ 1u, err);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) continue;
        const uint8_t* src = smem + C::kOffRaw + rs * kTile8;
        uint8_t* dst = smem + C::kOffV + vs * C::kVTile;
        const int valid = w.n_keys - k * kTileK;  // rows past the last key become zero (0 * NaN would poison O)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int row = i * 16 + (t >> 3), ch = t & 7;  // 16 dims [16 ch, 16 ch + 16) of a row
          uint4 u = *reinterpret_cast<const uint4*>(src + row * 128 + ((ch ^ (row & 7)) << 4));
          if (row >= valid) u = make_uint4(0, 0, 0, 0);
          uint4 lo, hi;
          lo.x = e4m3x2_to_f16x2((uint16_t)u.x); lo.y = e4m3x2_to_f16x2((uint16_t)(u.x >> 16));
          lo.z = e4m3x2_to_f16x2((uint16_t)u.y); lo.w = e4m3x2_to_f16x2((uint16_t)(u.y >> 16));
          hi.x = e4m3x2_to_f16x2((uint16_t)u.z); hi.y = e4m3x2_to_f16x2((uint16_t)(u.z >> 16));
          hi.z = e4m3x2_to_f16x2((uint16_t)u.w); hi.w = e4m3x2_to_f16x2((uint16_t)(u.w >> 16));
          uint8_t* d = dst + (ch >> 2) * kTile8 + row * 128;
          const int c2 = 2 * (ch & 3);
          *reinterpret_cast<uint4*>(d + ((c2 ^ (row & 7)) << 4)) = lo;
          *reinterpret_cast<uint4*>(d + (((c2 + 1) ^ (row & 7)) << 4)) = hi;
        }
        fence_proxy_async_smem();
        arrive_warp(&v_full[vs], lane);
        if (lane == 0) mbar_arrive(&raw_empty[rs]);
      }
    }
    if (!ok) *s_abort = 1;
  } else if (warp >= 8) {
    regs_decrease<C::kRegsCtl>();
    if (warp == 8 || warp == 11) {
      // -------------------------------------------------------- TMA producers: K; V
      // As in the decode form: lane i finds box i's page a tile ahead, one lane issues.
      const bool is_v = warp == 11;
      const CUtensorMap* map = is_v ? &tmV : &tmK;
      const CUtensorMap* map16 = is_v ? &tmV16 : &tmK16;
      uint64_t* full = is_v ? (FP8 ? raw_full : v_full) : k_full;
      uint64_t* empty = is_v ? (FP8 ? raw_empty : v_empty) : k_empty;
      const int ns = is_v ? 2 : NK;
      uint8_t* ring = smem + (is_v ? (FP8 ? C::kOffRaw : C::kOffV) : C::kOffK);
      const int shift = a.kv.page_shift, in_page = (1 << shift) - 1, box_shift = min(shift, 7);
      const int n_pages = a.kv.n_pages, rows_all = (n_pages * Hkv) << shift;
      ChunkWalk w(a, start, units);
      int k = w.k0;
      auto look_up = [&]() {
        const int rest = w.n_keys - k * kTileK;
        const int off = lane << (rest >= kTileK ? box_shift : 4);
        if (off >= kTileK || off >= rest) return 0;
        return __ldg(a.pb.table + (long long)w.b * a.pb.max_pages + ((k * kTileK + off) >> shift));
      };
      int page = w.valid() ? look_up() : 0;
      int st = 0, done = 0;
      uint32_t phase = 0;
      bool ok = true;
      while (w.valid()) {
        const int g = w.g, kv0 = k * kTileK, rest = w.n_keys - kv0;
        const bool tail = rest < kTileK;
        const int bs = tail ? 4 : box_shift;
        const int n = tail ? (rest + 15) >> 4 : kTileK >> bs;
        // a bad page reads as zeros: behind the tensor map's last row
        const bool in = (unsigned)page < (unsigned)n_pages;
        if (!in) record_error(err, kErrInvalid);
        const int my_row = in ? ((page * Hkv + g) << shift) + ((kv0 + (lane << bs)) & in_page) : rows_all;
        int row[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) row[i] = __shfl_sync(0xffffffffu, my_row, i);
        if (++k == w.k1) {
          w.next();
          k = w.k0;
        }
        if (w.valid()) page = look_up();
        ok = !*s_abort && mbar_wait(&empty[st], phase ^ 1u, err);
        if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
        uint8_t* dst = ring + st * (FP8 ? kTile8 : 2 * kTile8);
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
        if (++st == ns) { st = 0; phase ^= 1u; }
      }
      if (!ok) {
        *s_abort = 1;
        // let the copies still in flight land before the CTA exits
        for (int i = done > ns ? done - ns : 0; i < done; ++i) mbar_wait(&full[i % ns], (uint32_t)((i / ns) & 1), err);
      }
    } else if (elect_one()) {
      // --------------------------------------------------- MMA issuers, one per warpgroup X
      const int X = warp - 9;
      constexpr uint32_t idesc_s = FP8 ? idesc_e4m3_f32(128, 64, 0, 0) : idesc_bf16_f32(128, 64, 0, 0);
      constexpr uint32_t idesc_o = FP8 ? idesc_f16_f32(128, kD, 0, 1) : idesc_bf16_f32(128, kD, 0, 1);
      // One thread issues every product of X, so its instructions count: elected rather than
      // picked by lane number (eight products take 141 clocks to issue, not 510), descriptors
      // built once and stepped by constants.
      const uint64_t k_desc = sdesc_kmajor_sw128(smem_u32(smem + C::kOffK));
      const uint64_t v_desc = sdesc_mnmajor_sw128(smem_u32(smem + C::kOffV), kTile8, 1024);
      int c0 = 0, u = 0, q_loads[2] = {0, 0}, it = 0;
      bool ok = true;
      for (ChunkWalk w(a, start, units); w.valid() && ok; w.next(), ++it) {
        if (it > 0) {
          ok = !*s_abort && mbar_wait(item_done, (uint32_t)((it - 1) & 1), err);
          if (!ok) break;
        }
        const int kb = w.first(X), ke = w.end(X), step = w.step();
        const int qt = w.pair ? X : 0;  // the Q tile
        const uint64_t qd = desc_step(sdesc_kmajor_sw128(smem_u32(smem)), qt * C::kQTile);
        q_loads[0] += w.loads_q(0);
        q_loads[1] += w.loads_q(1);
        // arrivals this issuer owes a stage of tile k: its own, and the other's where that one skips it
        const int twice_from = w.pair ? (X == 1 ? w.nk0 : w.k1) : 0;
        // scores of half h of tile k, X's nth half tile, into buffer n & 1
        auto issue_s = [&](int k, int h, int n, bool last_half) -> bool {
          const int c = c0 + (k - w.k0), st = c & (NK - 1);
          if (h == 0) {
            if (!mbar_wait(&k_full[st], (uint32_t)((c / NK) & 1), err)) return false;
            tc_fence_after();
          }
          const uint64_t kd = desc_step(k_desc, st * C::kKTile + h * 64 * 128);
          const uint32_t d = tmem + 256 * X + 64 * (n & 1);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            const uint64_t ad = desc_step(qd, (kk >> 2) * kTile8 + 32 * (kk & 3));
            if (FP8)  // both terms of q against the same K
              mma_e4m3_ss(d, ad, desc_step(kd, 32 * (kk & 3)), idesc_s, kk ? 1u : 0u);
            else
              mma_bf16_ss(d, ad, desc_step(kd, (kk >> 2) * kTile8 + 32 * (kk & 3)), idesc_s, kk ? 1u : 0u);
          }
          mma_commit(&s_full[2 * X + (n & 1)]);
          if (last_half) {
            mma_commit(&k_empty[st]);
            if (k >= twice_from) mma_commit(&k_empty[st]);
          }
          return true;
        };
        // P.V of half h of tile k, then the scores of half h of the next tile, which take its buffer
        auto issue_half = [&](int k, int h, bool last_half, int next_halves) -> bool {
          const int c = c0 + (k - w.k0), st = c & (NV - 1), bi = 2 * X + (u & 1);
          const uint32_t par = (uint32_t)((u >> 1) & 1);
          if (h == 0 && !mbar_wait(&v_full[st], (uint32_t)((c / NV) & 1), err)) return false;
          if (!mbar_wait(&p_full[bi], par, err)) return false;
          tc_fence_after();
          const uint64_t vd = desc_step(v_desc, st * C::kVTile + h * 64 * 128);
          const uint32_t tp = tmem + 256 * X + 64 * (u & 1);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_bf16_ts(tmem + 256 * X + 128, tp + kk * 8, desc_step(vd, kk * 16 * 128), idesc_o,
                        (k != kb || h || kk) ? 1u : 0u);
          mma_commit(&pv_done[bi]);
          if (last_half) {
            mma_commit(&v_empty[st]);
            if (k >= twice_from) mma_commit(&v_empty[st]);
          }
          if (h < next_halves) {  // P must have been read
            if (!mbar_wait(&pv_done[bi], par, err)) return false;
            tc_fence_after();
            if (!issue_s(k + step, h, u + 2, h + 1 == next_halves)) return false;
          }
          ++u;
          return true;
        };
        // (only the item's last tile can have a single half)
        if (kb < ke) {
          // the item's first two half tiles: both buffers are free since the last item ended
          const int nh = w.halves(X, kb);
          ok = !*s_abort && mbar_wait(&q_full[qt], (uint32_t)((q_loads[qt] - 1) & 1), err);
          if (ok) {
            tc_fence_after();
            ok = issue_s(kb, 0, u, nh == 1) && (nh == 1 || issue_s(kb, 1, u + 1, true));
          }
        }
        for (int k = kb; k < ke && ok; k += step) {
          const int nh = k + step < ke ? 2 : w.halves(X, k);
          const int next_halves = k + step >= ke ? 0 : k + 2 * step < ke ? 2 : w.halves(X, k + step);
          ok = !*s_abort && issue_half(k, 0, nh == 1, next_halves) && (nh == 1 || issue_half(k, 1, true, next_halves));
        }
        c0 += w.k1 - w.k0;
        mbar_arrive(item_done);
      }
      if (!ok) *s_abort = 1;
      mma_commit(&drain[X]);  // every MMA completes before the tensor memory is released
      mbar_wait(&drain[X], 0, err);
    }
  } else {
    regs_increase<C::kRegsSoftmax>();
    // ---------------------------------------------------------------- softmax
    const int X = warp >> 2, quad = warp & 3;
    const int r = quad * 32 + lane;  // row of the Q tile, tensor-memory lane
    const int gs = a.g_shift, G = 1 << gs, TQ = 128 >> gs;
    const uint32_t tS = tmem + 256 * X + ((uint32_t)(quad * 32) << 16), tO = tS + 128;
    // fp16 probabilities: the running maximum is kept 7 below the scores', so that P <= 2^15
    constexpr float kShift = FP8 ? 7.f : 0.f;
    int c0 = 0, u = 0, q_loads0 = 0, it = 0;
    bool ok = true;
    ChunkMeta meta = {};
    for (ChunkWalk w(a, start, units); w.valid(); w.next(), ++it) {
      const int qt = w.pair ? X : 0, tile_t0 = w.t0 + qt * TQ;
      const int n_rows = min(TQ, w.n_q - tile_t0) << gs;
      const bool valid = r < n_rows;
      const bool warp_valid = quad * 32 < n_rows;
      const int qpos = valid ? w.ctx + tile_t0 + (r >> gs) : w.n_keys - 1;
      const int qpos_first = __shfl_sync(0xffffffffu, qpos, 0);  // the warp's smallest
      q_loads0 += w.loads_q(0);
      float factor = kScaleLog2;
      if (w.loads_q(X)) {
        // the warp's 32 rows of Q tile X into shared memory, 128-byte swizzle (zeros behind the
        // last): 16 lanes a row, so that a load instruction takes two whole rows (a row a thread
        // would be 32 separate lines an instruction, 3.6 us a tile)
        const int d8 = lane & 15;  // dims [8 d8, 8 d8 + 8)
        uint4 v[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int row = quad * 32 + 2 * i + (lane >> 4);
          v[i] = ld_or_zero(a.q + (long long)(w.q0 + tile_t0 + (row >> gs)) * a.ldq +
                                ((long long)(w.g * G + (row & (G - 1))) * kD + 8 * d8),
                            row < n_rows);
        }
        float down = 1.f;  // e4m3: of row 2 d8 + (lane >> 4), the row that the exchange below leaves here
        if (FP8) {
          // q = 2^e (t1 + t2), the row's largest value scaled into [128, 256): t1 the leading 4
          // significant bits, t2 the other 4 (a remainder from the rounded t1 would halve the
          // error of the smallest values, and cost 1 % of a call). Largest values by halving
          // exchanges over the 16 lanes of a row: 15 shuffles for 16 rows.
          uint32_t mx[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const uint32_t m2 = __vmaxu2(__vmaxu2(v[i].x & 0x7fff7fffu, v[i].y & 0x7fff7fffu),
                                         __vmaxu2(v[i].z & 0x7fff7fffu, v[i].w & 0x7fff7fffu));
            mx[i] = max(m2 & 0xffffu, m2 >> 16);
          }
#pragma unroll
          for (int half = 8; half >= 1; half >>= 1) {
            const bool upper = (lane & half) != 0;
#pragma unroll
            for (int i = 0; i < half; ++i) {
              const uint32_t send = upper ? mx[i] : mx[i + half], keep = upper ? mx[i + half] : mx[i];
              mx[i] = max(keep, __shfl_xor_sync(0xffffffffu, send, half));
            }
          }
          const int ex = (int)(mx[0] >> 7);
          const int e = min(max(ex - 127 - 7, -119), 120);
          down = __uint_as_float((uint32_t)(127 - e) << 23);
          const float up = ex == 255 ? __uint_as_float(0x7fc00000u) : __uint_as_float((uint32_t)(127 + e) << 23);
          factor = kScaleLog2 * a.kv.k_scale[w.g] * __shfl_sync(0xffffffffu, up, (lane & 1) * 16 + (lane >> 1));
          // a row of zeros (2^-119) against a small scale: never 0, which times a masked score's -inf is
          // NaN (the scores, at most 2^24 before it, stay below 2^-100; a NaN stays)
          if (factor < kMinFactor) factor = kMinFactor;
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int row = quad * 32 + 2 * i + (lane >> 4);
          uint8_t* dst = smem + X * C::kQTile;
          if (!FP8) {
            *reinterpret_cast<uint4*>(dst + q_tile_at(row, d8)) = v[i];
          } else {
            const float dn = __shfl_sync(0xffffffffu, down, (lane & 16) + i);
            const uint32_t x[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
            uint32_t t1[4], t2[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint32_t h = x[j] & 0xfff0fff0u;
              const float h0 = bf16_lo(h) * dn, h1 = bf16_hi(h) * dn;
              t1[j] = pack_e4m3x2(h0, h1);
              t2[j] = pack_e4m3x2(bf16_lo(x[j]) * dn - h0, bf16_hi(x[j]) * dn - h1);
            }
            uint8_t* d = dst + q_tile_at(row, d8 >> 1) + (d8 & 1) * 8;
            *reinterpret_cast<uint2*>(d) = make_uint2(t1[0] | (t1[1] << 16), t1[2] | (t1[3] << 16));
            *reinterpret_cast<uint2*>(d + kTile8) = make_uint2(t2[0] | (t2[1] << 16), t2[2] | (t2[3] << 16));
          }
        }
        if (FP8 && !w.pair) ml[256 + r] = factor;  // for warpgroup 1
        fence_proxy_async_smem();
        arrive_warp(&q_full[X], lane);
      } else if (FP8 && w.any(X)) {
        ok = ok && !*s_abort && (it == 0 || mbar_wait(item_done, (uint32_t)((it - 1) & 1), err)) &&
             mbar_wait(&q_full[0], (uint32_t)((q_loads0 - 1) & 1), err);
        ok = __all_sync(0xffffffffu, ok);
        factor = ml[256 + r];
      }
      float m_run = -INFINITY, l_run = 0.f;
      const int kb = w.first(X), ke = w.end(X), step = w.step();
      // the half tiles in order: keys kv0 .. kv0 + 63 (the loop carries little: its serial
      // instructions, not the waits, are what a half tile costs besides its exponentials)
      const int n_half = kb < ke ? 2 * ((ke - kb - 1) / step) + w.halves(X, kb + (ke - kb - 1) / step * step) : 0;
      int kv0 = kb * kTileK;
      for (int n = 0; n < n_half; ++n, ++u, kv0 += n & 1 ? 64 : step * kTileK - 64) {
        const int bi = 2 * X + (u & 1);
        const uint32_t tSb = tS + 64 * (u & 1);
        ok = ok && mbar_wait_warp(&s_full[bi], (uint32_t)((u >> 1) & 1), err);
        // bf16 V: zero the tile's rows past the last key (0 * NaN would poison O); both
        // warpgroups of a pair do so before they release their P (zeros over zeros)
        if (!FP8 && kv0 + kTileK > w.n_keys && !(n & 1)) {
          const int c = c0 + ((kv0 >> 7) - w.k0), st = c % NV;
          ok = ok && mbar_wait_warp(&v_full[st], (uint32_t)((c / NV) & 1), err);
          if (ok && kv0 + r >= w.n_keys) {
            uint4* v0 = reinterpret_cast<uint4*>(smem + C::kOffV + st * C::kVTile + r * 128);
#pragma unroll
            for (int i = 0; i < 8; ++i) v0[i] = v0[i + kTile8 / 16] = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
        }
        if (!ok || !warp_valid) {  // (a warp of rows behind the last token only keeps step)
          tc_fence_before();
          arrive_warp(&p_full[bi], lane);
          continue;
        }
        tc_fence_after();
        const bool need_mask = kv0 + 63 > qpos_first;
        uint32_t v[2][32];
        tmem_ld32(tSb, v[0]);
        tmem_ld32(tSb + 32, v[1]);
        tmem_wait_ld_regs(v[0]);
        tmem_wait_ld_regs(v[1]);
        if (need_mask) {
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (kv0 + c * 32 + i > qpos) v[c][i] = __float_as_uint(-INFINITY);
        }
        float mc[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint32_t* x = v[c >> 1] + 16 * (c & 1);
          mc[c] = __uint_as_float(x[0]);
#pragma unroll
          for (int i = 1; i < 15; i += 2) mc[c] = fmax3(mc[c], __uint_as_float(x[i]), __uint_as_float(x[i + 1]));
          mc[c] = fmaxf(mc[c], __uint_as_float(x[15]));
        }
        const float mxs = fmaxf(fmaxf(mc[0], mc[1]), fmaxf(mc[2], mc[3])) * factor - kShift;
        float alpha = 1.f;
        if (mxs > m_run + kRescaleThreshold || m_run == -INFINITY) {
          alpha = (m_run == -INFINITY) ? 0.f : ex2_approx(m_run - mxs);
          m_run = mxs;
        }
        // p = 2^(s factor - m); a row that has seen no key yet (its causal limit lies before
        // this half tile) keeps m = -inf and p = 2^-inf = 0
        const float neg = m_run == -INFINITY ? 0.f : -m_run;
        const uint64_t scale2 = f2_pack(__float_as_uint(factor), __float_as_uint(factor));
        const uint64_t neg2 = f2_pack(__float_as_uint(neg), __float_as_uint(neg));
        uint64_t acc2[2] = {0ull, 0ull};
#pragma unroll
        for (int c = 0; c < 2; ++c) {
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            const uint64_t e = f2_fma(f2_pack(v[c][i], v[c][i + 1]), scale2, neg2);
            const float p0 = ex2_approx(f2_lo(e));
            const float p1 = ex2_approx(f2_hi(e));
            acc2[(i >> 1) & 1] = f2_add(acc2[(i >> 1) & 1], f2_pack(__float_as_uint(p0), __float_as_uint(p1)));
            v[c][i >> 1] = FP8 ? pack_f16x2(p0, p1) : pack_bf16x2(p0, p1);
          }
          tmem_st16(tSb + c * 16, v[c]);
        }
        const uint64_t acc = f2_add(acc2[0], acc2[1]);
        l_run = l_run * alpha + f2_lo(acc) + f2_hi(acc);
        if (n > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
          // O_X is stable once the previous half tile's P.V is complete
          ok = mbar_wait_warp(&pv_done[bi ^ 1], (uint32_t)(((u - 1) >> 1) & 1), err);
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t o[32];
            tmem_ld32(tO + c * 32, o);
            tmem_wait_ld_regs(o);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
            tmem_st32(tO + c * 32, o);
          }
        }
        tmem_wait_st();
        tc_fence_before();
        arrive_warp(&p_full[bi], lane);
      }
      c0 += w.k1 - w.k0;
      const bool any = kb < ke;
      if (any) {
        ok = ok && !*s_abort && mbar_wait(&pv_done[2 * X + ((u - 1) & 1)], (uint32_t)(((u - 1) >> 1) & 1), err);
        ok = __all_sync(0xffffffffu, ok);
      }
      // a single item's other half: warpgroup 1 leaves m, l in shared memory and O_1 in place
      float w0 = 1.f, w1 = 0.f;
      bool other = false;
      if (!w.pair) {
        if (X == 1) {
          ml[r] = any ? m_run : -INFINITY;
          ml[128 + r] = l_run;
        }
        tc_fence_before();
        named_bar(1, 256);
        tc_fence_after();
        if (X == 0) {
          const float m1 = ml[r], M = fmaxf(m_run, m1);
          other = w.any(1);
          if (other && M != -INFINITY) {
            w0 = ex2_approx(m_run - M);
            w1 = ex2_approx(m1 - M);
            l_run = l_run * w0 + ml[128 + r] * w1;
            m_run = M;
          }
        }
      }
      const int nk = w.pair && X == 0 ? w.nk0 : w.n;  // KV tiles of this Q tile
      const bool writes = any && (w.pair || X == 0);
      if (writes && warp_valid && ok) {
        tc_fence_after();
        const bool whole = w.k0 == 0 && w.k1 >= nk;
        const float vs = FP8 ? a.kv.v_scale[w.g] : 1.f;
        const float inv = whole ? 1.f / l_run : 1.f;
        // one value of a finished row; the scale last, as in the decode form
        auto done = [&](uint32_t x) { return FP8 ? __uint_as_float(x) * inv * vs : __uint_as_float(x) * inv; };
        float* part = a.part + ((long long)(blockIdx.x * 2 + (w.k0 > 0 ? 0 : 1)) * 2 + X) * kChunkPart;
        // finished rows go through the Q tile (whose scores are all done), where the warp's own q
        // lay: a row a thread into shared memory, two whole rows an instruction from there
        uint8_t* stage = smem + X * C::kQTile;
        const bool f16 = a.o_f16 != 0;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t o[32];
          tmem_ld32(tO + c * 32, o);
          tmem_wait_ld_regs(o);
          if (other) {  // the same for all threads
            uint32_t o1[32];
            tmem_ld32(tO + 256 + c * 32, o1);
            tmem_wait_ld_regs(o1);
#pragma unroll
            for (int i = 0; i < 32; ++i)
              o[i] = __float_as_uint(__uint_as_float(o[i]) * w0 + (w1 != 0.f ? __uint_as_float(o1[i]) * w1 : 0.f));
          }
          if (whole) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint4 q;
              q.x = pack_op_x2(f16, done(o[8 * i + 0]), done(o[8 * i + 1]));
              q.y = pack_op_x2(f16, done(o[8 * i + 2]), done(o[8 * i + 3]));
              q.z = pack_op_x2(f16, done(o[8 * i + 4]), done(o[8 * i + 5]));
              q.w = pack_op_x2(f16, done(o[8 * i + 6]), done(o[8 * i + 7]));
              *reinterpret_cast<uint4*>(stage + q_tile_at(r, c * 4 + i)) = q;
            }
          } else if (valid) {
#pragma unroll
            for (int i = 0; i < 32; i += 4)
              __stcg(reinterpret_cast<float4*>(part + (c * 32 + i) * 128 + r * 4),
                     make_float4(__uint_as_float(o[i]), __uint_as_float(o[i + 1]), __uint_as_float(o[i + 2]),
                                 __uint_as_float(o[i + 3])));
          }
        }
        __syncwarp();
        if (whole) {
          const int d8 = lane & 15;
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int row = quad * 32 + 2 * i + (lane >> 4);
            if (row < n_rows)
              *reinterpret_cast<uint4*>(a.out + (long long)(w.q0 + tile_t0 + (row >> gs)) * a.ldo +
                                        ((long long)(w.g * G + (row & (G - 1))) * kD + 8 * d8)) =
                  *reinterpret_cast<const uint4*>(stage + q_tile_at(row, d8));
          }
          __syncwarp();
        }
        if (!whole && valid) {
          __stcg(part + kD * 128 + r, m_run);
          __stcg(part + kD * 128 + 128 + r, l_run);
        }
      }
      if (writes && ok) {
        if (w.k0 > 0) meta.has = 1;
        if (w.k0 == 0 && w.k1 < nk) {
          const int wgt = w.pair ? 2 : 1;
          const long long us = share(U, blockIdx.x, n_cta) + (units - w.left);  // the item's first unit
          meta.split = 1;
          meta.c_last = cta_of(us + (long long)wgt * (nk - 1), U, n_cta);
          meta.n_rows = n_rows;
          meta.tok = w.q0 + tile_t0;
          meta.g = w.g;
        }
      }
      if (!w.pair) named_bar(1, 256);  // O_1, m and l are read
      arrive_warp(item_done, lane);
    }
    if (!ok) *s_abort = 1;
    if (r == 0) a.meta[blockIdx.x * 2 + X] = meta;
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the partials of the Q tiles that span CTAs: blocks (c, X, 16 dims) with the tiles that
// CTA c began and did not end. o = sum_i o_i 2^(m_i - M) / sum_i l_i 2^(m_i - M) over the CTAs in order.
__global__ void __launch_bounds__(128) paged_chunk_join_kernel(const PagedAttn a) {
  pdl_wait();
  pdl_trigger();
  const int cx = blockIdx.x >> 3, d0 = (blockIdx.x & 7) * 16, c = cx >> 1, X = cx & 1;
  const ChunkMeta m = a.meta[cx];
  const int r = threadIdx.x, lane = r & 31;
  if (!m.split) return;
  const bool valid = r < m.n_rows;
  auto part = [&](int i) { return a.part + ((long long)(i * 2 + (i == c ? 1 : 0)) * 2 + X) * kChunkPart; };
  float M = -INFINITY, L = 0.f, o[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) o[j] = 0.f;
  for (int base = c; base <= m.c_last; base += 32) {
    const int i = base + lane;
    unsigned left = __ballot_sync(0xffffffffu, i == c || (i <= m.c_last && a.meta[2 * i + X].has != 0));
    // kBatch partials at a time, their loads in flight together (one after the other they cost
    // three latencies each, 13 us for a call)
    constexpr int kBatch = 4;
    while (left) {
      const float* p[kBatch];
      float mi[kBatch], li[kBatch];
      float4 v[kBatch][4];
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int f = __ffs(left) - 1;
        left &= left - 1;
        p[b] = f < 0 ? nullptr : part(base + f);
        mi[b] = -INFINITY;
        li[b] = 0.f;
        if (valid && p[b]) {
          mi[b] = __ldcg(p[b] + kD * 128 + r);
          li[b] = __ldcg(p[b] + kD * 128 + 128 + r);
#pragma unroll
          for (int j = 0; j < 4; ++j) v[b][j] = __ldcg(reinterpret_cast<const float4*>(p[b] + (d0 + 4 * j) * 128 + r * 4));
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) v[b][j] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
      }
      float Mn = M;
#pragma unroll
      for (int b = 0; b < kBatch; ++b) Mn = fmaxf(Mn, mi[b]);
      const float old = M == -INFINITY ? 0.f : exp2f(M - Mn);
      M = Mn;
      L *= old;
#pragma unroll
      for (int j = 0; j < 16; ++j) o[j] *= old;
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const float w = mi[b] == -INFINITY ? 0.f : exp2f(mi[b] - Mn);
        L += li[b] * w;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          // (a row that saw no key of a part has weight 0 there, whatever its o holds)
          o[4 * j] += w != 0.f ? v[b][j].x * w : 0.f;
          o[4 * j + 1] += w != 0.f ? v[b][j].y * w : 0.f;
          o[4 * j + 2] += w != 0.f ? v[b][j].z * w : 0.f;
          o[4 * j + 3] += w != 0.f ? v[b][j].w * w : 0.f;
        }
      }
    }
  }
  if (!valid) return;
  const int gs = a.g_shift, G = 1 << gs;
  const float inv = 1.f / L, vs = a.kv.fp8 ? a.kv.v_scale[m.g] : 1.f;  // (the scale last, as above)
#pragma unroll
  for (int j = 0; j < 16; ++j) o[j] = o[j] * inv * vs;
  uint16_t* dst = a.out + (long long)(m.tok + (r >> gs)) * a.ldo + (long long)(m.g * G + (r & (G - 1))) * kD + d0;
  const bool f16 = a.o_f16 != 0;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint4 q;
    q.x = pack_op_x2(f16, o[8 * h], o[8 * h + 1]);
    q.y = pack_op_x2(f16, o[8 * h + 2], o[8 * h + 3]);
    q.z = pack_op_x2(f16, o[8 * h + 4], o[8 * h + 5]);
    q.w = pack_op_x2(f16, o[8 * h + 6], o[8 * h + 7]);
    *reinterpret_cast<uint4*>(dst + 8 * h) = q;
  }
}

// ----------------------------------------------------------------------------
// Host side
// ----------------------------------------------------------------------------
namespace {

// Scratch of one form, in order: work list, CTA starts, merge counters (decode form) or what the
// CTAs leave to join (chunk form), partials, e4m3 query terms and scales (decode form).
struct Scratch {
  size_t plan, start, counters, part, q8, q8_scale, bytes;
};
static_assert(alignof(CtaStart) <= 16 && alignof(ChunkMeta) <= 16, "a workspace is aligned to 16 bytes");
size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }
Scratch scratch_of(bool chunk, int B, int Hq, int Hkv) {
  Scratch s;
  const size_t G = Hq / Hkv, rows = (size_t)B * Hkv;
  s.plan = 0;
  s.start = s.plan + up256(((size_t)B + 1) * sizeof(long long));
  s.counters = s.start + kMaxCtas * sizeof(CtaStart);
  s.part = s.counters + up256(chunk ? 2 * kChunkCtas * sizeof(ChunkMeta) : rows * sizeof(int));
  s.q8 = s.part + up256((chunk ? (size_t)4 * kChunkCtas * kChunkPart : (rows + kMaxCtas) * G * kPartFloats) * sizeof(float));
  s.q8_scale = s.q8 + up256(chunk ? 0 : (size_t)B * Hq * 2 * kD);
  s.bytes = s.q8_scale + up256(chunk ? 0 : (size_t)B * Hq * sizeof(float));
  return s;
}

// The forms a call runs (bit 0: decode, bit 1: chunk). With more than one new token allowed, the
// chunk form can take every sequence. A large batch likely decodes most of them, which the
// decode form streams faster. Both forms against the chunk form alone, in us, for two chunks of 300 to
// 512 tokens in batches of decode tokens at 100 to 4000 cached:
//   sequences        4          8         12         16         32
//   bf16       45 / 32    59 / 58    72 / 88    85 / 84   99 / 132
//   e4m3       50 / 38    59 / 66   69 / 110    82 / 96   91 / 162
// The lengths, which would tell, are on the device; 16 leaves small batches one form and costs
// little either way: 15 decode tokens and one chunk 73 / 84 (e4m3 66 / 97). A batch of 16 without a decode
// token pays the decode form's launch and plan: 16 x 7 tokens 71 / 67 (82 / 79), at 10 to 100
// cached 20 / 17 (25 / 20).
constexpr int kMixedBatch = 16;
int forms_of(int B, int max_q) { return max_q == 1 ? 1 : B >= kMixedBatch ? 3 : 2; }

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

// A kernel as it is launched.
using DecodeKernel = void (*)(CUtensorMap, CUtensorMap, CUtensorMap, CUtensorMap, CUtensorMap, PagedAttn);
using ChunkKernel = void (*)(CUtensorMap, CUtensorMap, CUtensorMap, CUtensorMap, PagedAttn);
template <typename K>
struct Launch {
  K kernel = nullptr;
  int threads = 0, smem = 0, min_regs = 0;
  int ready() const { return ensure_smem_attr(reinterpret_cast<const void*>(kernel), smem, min_regs); }
};

template <int G, bool FP8>
Launch<DecodeKernel> decode_kernel() {
  using C = DecodeCfg<G, FP8>;
  return {attn_paged_decode_kernel<G, FP8>, C::kThreads, (int)C::kSmem, 0};
}
Launch<DecodeKernel> decode_kernel(int G, int fp8) {
  switch (G * 2 + fp8) {
    case 2: return decode_kernel<1, false>();
    case 3: return decode_kernel<1, true>();
    case 4: return decode_kernel<2, false>();
    case 5: return decode_kernel<2, true>();
    case 8: return decode_kernel<4, false>();
    case 9: return decode_kernel<4, true>();
    case 16: return decode_kernel<8, false>();
    case 17: return decode_kernel<8, true>();
    case 32: return decode_kernel<16, false>();
    case 33: return decode_kernel<16, true>();
  }
  return {};
}

template <bool FP8>
Launch<ChunkKernel> chunk_kernel() {
  using C = ChunkCfg<FP8>;
  // the register split must fit what the block is launched with, or the increase never returns
  return {attn_paged_chunk_kernel<FP8>, C::kThreads, (int)C::kSmem, (C::kRegBudget + C::kThreads - 1) / C::kThreads};
}

}  // namespace

size_t paged_attention_bytes(int B, int Hq, int Hkv, int max_q) {
  const int forms = forms_of(B, max_q);
  return (forms & 1 ? scratch_of(false, B, Hq, Hkv).bytes : 0) + (forms & 2 ? scratch_of(true, B, Hq, Hkv).bytes : 0);
}

int launch_attention_paged(const uint16_t* q, long long ldq, int n_tokens, int max_q, const PagedBatch& pb,
                           const KvPages& kv, int Hq, void* scratch, uint16_t* out, long long ldo, int* err,
                           cudaStream_t s, bool o_f16) {
  PagedAttn base = {};
  base.pb = pb;
  base.kv = kv;
  base.n_tokens = n_tokens; base.max_q = max_q; base.Hq = Hq; base.o_f16 = o_f16 ? 1 : 0;
  while ((kv.Hkv << base.g_shift) < Hq) ++base.g_shift;
  base.q = q; base.ldq = ldq;
  base.out = out; base.ldo = ldo;
  base.err = err;
  const int forms = forms_of(pb.B, max_q);
  uint8_t* ws = static_cast<uint8_t*>(scratch);
  PagedAttn form[2] = {base, base};  // decode, chunk
  for (int f = 0; f < 2; ++f) {
    if (!(forms >> f & 1)) continue;
    const Scratch off = scratch_of(f == 1, pb.B, Hq, kv.Hkv);
    PagedAttn& a = form[f];
    a.plan = reinterpret_cast<long long*>(ws + off.plan);
    a.start = reinterpret_cast<CtaStart*>(ws + off.start);
    a.counters = reinterpret_cast<int*>(ws + off.counters);
    a.meta = reinterpret_cast<ChunkMeta*>(ws + off.counters);
    a.part = reinterpret_cast<float*>(ws + off.part);
    a.q8 = ws + off.q8;
    a.q8_scale = reinterpret_cast<float*>(ws + off.q8_scale);
    const int cap = f == 1 ? kChunkCtas : kMaxCtas;
    a.n_cta = num_sms() < cap ? num_sms() : cap;
    ws += off.bytes;
  }
  form[1].min_q = forms == 3 ? 2 : 1;
  const long long split = forms & 1 && kv.fp8 ? ((long long)pb.B * Hq + kPlanThreads / 32 - 1) / (kPlanThreads / 32) : 0;
  // all that can fail comes before the first launch: a refused call leaves nothing on the stream
  CUtensorMap tmQ, tmK, tmV, tmK16, tmV16;
  if (page_maps(kv, &tmK, &tmV, &tmK16, &tmV16)) return -6;
  Launch<DecodeKernel> decode;
  Launch<ChunkKernel> chunk;
  if (forms & 1) {
    const int G = 1 << base.g_shift;
    decode = decode_kernel(G, kv.fp8);
    if (!decode.kernel) {
      set_last_error("attention_paged: %d query heads per KV group is not supported (1, 2, 4, 8 or 16)", G);
      return -2;
    }
    if (decode.ready()) return -6;
    if (kv.fp8 ? make_tmap_bytes(&tmQ, form[0].q8, (long long)pb.B * Hq * 2, kD, 2 * G)
               : make_tmap_3d(&tmQ, q, kD, Hq, n_tokens, kD * 2, ldq * 2, 64, G, 1)) {
      set_last_error("attention_paged: cannot encode the query tensor map (ldq %lld)", ldq);
      return -6;
    }
  }
  if (forms & 2) {
    chunk = kv.fp8 ? chunk_kernel<true>() : chunk_kernel<false>();
    if (chunk.ready()) return -6;
  }
  q3_launch(paged_plan_kernel, (unsigned)(2 + split), kPlanThreads, 0, s, form[0], form[1], forms);
  if (forms & 1)
    q3_launch(decode.kernel, form[0].n_cta, decode.threads, decode.smem, s, tmQ, tmK, tmV, tmK16, tmV16, form[0]);
  if (forms & 2) {
    q3_launch(chunk.kernel, form[1].n_cta, chunk.threads, chunk.smem, s, tmK, tmV, tmK16, tmV16, form[1]);
    q3_launch(paged_chunk_join_kernel, form[1].n_cta * 16, 128, 0, s, form[1]);
  }
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) {
    set_last_error("attention_paged launch failed: %s", cudaGetErrorString(e));
    return -6;
  }
  return 0;
}

}  // namespace q3
