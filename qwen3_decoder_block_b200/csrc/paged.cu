// Writing and moving a paged KV cache: the per-head QK norm with the rotation and the
// cache write of a ragged batch, and the copies between pages and a contiguous cache. All
// of them are bound by the bytes they move; e4m3 pages quantise as they are written
// (byte = e4m3(x / scale[head]), saturating) and widen as they are read (byte * scale).
//
// One scale per KV head, given by the caller: a key leaves its RMSNorm with a norm of at most
// sqrt(128) max |w|, and e4m3 keeps its 3 mantissa bits over 15 binades, so a scale per
// token would gain nothing; a scale per head folds into the attention's softmax factor and
// epilogue.
#include "paged.cuh"
#include "internal.h"

namespace q3 {

namespace {

// Rows of 128 values in flight per warp: 4 (token, head) rows at a time, 8 lanes each, of a
// token's slots. At 6.5 TB/s and about 2 us from a warp's first load to its last store an SM
// needs some 90 KB in flight: 4 KB a warp, 24 warps an SM (80 registers), in small blocks that
// are replaced one by one. 8192 tokens: 28.3 us (4.8 TB/s); 2 KB a warp or blocks of 256 31 to 32 us.
constexpr int kSlotsPerWarp = 16;
constexpr int kNormWarps = 4;
constexpr int kWarps = 8;  // of the moves

struct NormRopeArgs {
  PagedBatch pb;
  KvPages kv;
  const uint16_t* qkv;
  long long ldqkv;
  uint16_t* q_out;
  long long ldq;
  const uint16_t* qw;
  const uint16_t* kw;
  const float* rope;
  int n_tokens, Hq, max_pos, n_blocks_tok;
  float eps;
  int* err;
};

// Blocks of `warps` warps for the items of the tokens and, behind them, the check of the lists.
long long blocks_of(long long items, int B, int warps) { return (items + ((long long)B + 31) / 32 + warps - 1) / warps; }

// 8 bf16 as four pairs of fp32, and back
__device__ __forceinline__ void unpack8(const uint4& u, uint64_t (&f)[4]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = f2_pack(w[i] << 16, w[i] & 0xffff0000u);
}
__device__ __forceinline__ uint4 pack8(const uint64_t (&f)[4]) {
  return make_uint4(pack_bf16x2(f2_lo(f[0]), f2_hi(f[0])), pack_bf16x2(f2_lo(f[1]), f2_hi(f[1])),
                    pack_bf16x2(f2_lo(f[2]), f2_hi(f[2])), pack_bf16x2(f2_lo(f[3]), f2_hi(f[3])));
}
// x * inv as e4m3, 8 values
__device__ __forceinline__ uint2 quant8(const uint64_t (&f)[4], float inv) {
  const uint64_t inv2 = f2_pack(__float_as_uint(inv), __float_as_uint(inv));
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint64_t v = f2_mul(f[i], inv2);
    w[i] = pack_e4m3x2(f2_lo(v), f2_hi(v));
  }
  return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

}  // namespace

// A group of 8 lanes owns one (token, head) row: lane l of the group holds dims [8l, 8l + 8)
// and [64 + 8l, 64 + 8l + 8), so that the pairs of the rotation (i, i + 64) meet in one lane,
// each load of 16 bytes is part of 128 contiguous ones, and the sum of squares takes three
// shuffles. A warp owns kSlotsPerWarp consecutive head slots of a token.
template <bool FP8>
__global__ void __launch_bounds__(32 * kNormWarps, 6) qk_norm_rope_paged_kernel(const NormRopeArgs a) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const long long item = (long long)blockIdx.x * kNormWarps + (threadIdx.x >> 5);
  const long long items = (long long)a.n_tokens * a.n_blocks_tok;
  if (item >= items) {
    paged_check_lists(a.pb, a.n_tokens, item - items, lane, a.err);
    return;
  }
  const int tok = (int)(item / a.n_blocks_tok);
  const int Hkv = a.kv.Hkv, slots = a.Hq + 2 * Hkv;
  const int slot0 = (int)(item % a.n_blocks_tok) * kSlotsPerWarp + (lane >> 3);
  const int d = (lane & 7) * 8;
  constexpr int kIter = kSlotsPerWarp / 4;
  uint4 lo[kIter], hi[kIter];
#pragma unroll
  for (int i = 0; i < kIter; ++i) {
    lo[i] = hi[i] = make_uint4(0, 0, 0, 0);
    if (slot0 + 4 * i < slots) {
      const uint16_t* row = a.qkv + tok * a.ldqkv + (long long)(slot0 + 4 * i) * 128;
      lo[i] = *reinterpret_cast<const uint4*>(row + d);
      hi[i] = *reinterpret_cast<const uint4*>(row + 64 + d);
    }
  }
  PagedToken at;
  if (!paged_seq_of(a.pb, a.n_tokens, tok, lane, &at)) return;
  const int t = tok - at.start;
  if (at.ctx >= a.max_pos - t) {
    if (lane == 0) record_error(a.err, kErrCapacity);
    return;
  }
  const int pos = at.ctx + t;
  uint64_t cs[4], sn[4];  // of dims d + 2 j, d + 2 j + 1
  {
    // (a negative position is reported below; its row is not read)
    const float4* r = reinterpret_cast<const float4*>(a.rope + ((long long)max(pos, 0) * 64 + d) * 2);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float4 v = r[j];
      cs[j] = f2_pack(__float_as_uint(v.x), __float_as_uint(v.z));
      sn[j] = f2_pack(__float_as_uint(v.y), __float_as_uint(v.w));
    }
  }
  const long long cell = paged_row(a.pb, a.kv, at.b, pos, lane == 0 ? a.err : nullptr);
  if (cell < 0) return;
#pragma unroll
  for (int i = 0; i < kIter; ++i) {
    const int slot = slot0 + 4 * i;
    const bool is_q = slot < a.Hq, is_v = slot >= a.Hq + Hkv;
    // two values an instruction: these operations, not the bytes, bound the plain form
    uint64_t x[4], y[4];
    unpack8(lo[i], x);
    unpack8(hi[i], y);
    if (__any_sync(0xffffffffu, !is_v)) {
      uint64_t s2 = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) s2 = f2_fma(y[j], y[j], f2_fma(x[j], x[j], s2));
      float ss = f2_lo(s2) + f2_hi(s2);
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      if (!is_v) {
        const float r = rsqrtf(ss * (1.0f / 128.0f) + a.eps);
        const uint64_t r2 = f2_pack(__float_as_uint(r), __float_as_uint(r));
        const uint64_t n2 = f2_pack(__float_as_uint(-r), __float_as_uint(-r));
        const uint16_t* wn = is_q ? a.qw : a.kw;
        uint64_t wx[4], wy[4];
        unpack8(*reinterpret_cast<const uint4*>(wn + d), wx);
        unpack8(*reinterpret_cast<const uint4*>(wn + 64 + d), wy);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint64_t u = f2_mul(x[j], wx[j]), w = f2_mul(y[j], wy[j]);
          const uint64_t c = f2_mul(cs[j], r2), s = f2_mul(sn[j], r2), ns = f2_mul(sn[j], n2);
          x[j] = f2_fma(w, ns, f2_mul(u, c));
          y[j] = f2_fma(w, c, f2_mul(u, s));
        }
      }
    }
    if (slot >= slots) continue;
    if (is_q) {
      uint16_t* dst = a.q_out + tok * a.ldq + (long long)slot * 128;
      *reinterpret_cast<uint4*>(dst + d) = pack8(x);
      *reinterpret_cast<uint4*>(dst + 64 + d) = pack8(y);
      continue;
    }
    const int g = is_v ? slot - a.Hq - Hkv : slot - a.Hq;
    const long long at = (cell + ((long long)g << a.kv.page_shift)) * 128 + d;
    uint8_t* pool = is_v ? a.kv.v : a.kv.k;
    if (FP8) {
      const float inv = 1.0f / (is_v ? a.kv.v_scale : a.kv.k_scale)[g];
      *reinterpret_cast<uint2*>(pool + at) = quant8(x, inv);
      *reinterpret_cast<uint2*>(pool + at + 64) = quant8(y, inv);
    } else {
      *reinterpret_cast<uint4*>(pool + 2 * at) = is_v ? lo[i] : pack8(x);
      *reinterpret_cast<uint4*>(pool + 2 * at + 128) = is_v ? hi[i] : pack8(y);
    }
  }
}

int launch_qk_norm_rope_paged(const uint16_t* qkv, long long ldqkv, int n_tokens, const PagedBatch& pb,
                              const KvPages& kv, int Hq, const uint16_t* qw, const uint16_t* kw, const float* rope,
                              int max_pos, float eps, uint16_t* q_out, long long ldq, int* err, cudaStream_t s) {
  NormRopeArgs a;
  a.pb = pb;
  a.kv = kv;
  a.qkv = qkv; a.ldqkv = ldqkv;
  a.q_out = q_out; a.ldq = ldq;
  a.qw = qw; a.kw = kw; a.rope = rope;
  a.n_tokens = n_tokens; a.Hq = Hq; a.max_pos = max_pos;
  a.n_blocks_tok = (Hq + 2 * kv.Hkv + kSlotsPerWarp - 1) / kSlotsPerWarp;
  a.eps = eps;
  a.err = err;
  const long long blocks = blocks_of((long long)n_tokens * a.n_blocks_tok, pb.B, kNormWarps);
  if (blocks >= (1ll << 31)) {
    set_last_error("qk_norm_rope_paged: %d tokens exceed the grid limit", n_tokens);
    return -2;
  }
  q3_launch(kv.fp8 ? qk_norm_rope_paged_kernel<true> : qk_norm_rope_paged_kernel<false>, (unsigned)blocks,
            32 * kNormWarps, 0, s, a);
  return cudaGetLastError() == cudaSuccess ? 0 : -6;
}

// ---------------------------------------------------------------------------
// Copies between pages and a contiguous cache [B][Hkv][s_max][128] bf16: the batch's new
// positions of every head, k and v. A warp takes kHeads heads of a token: 16 lanes per row of
// 128 values (16 bytes of bf16, 8 of e4m3, a lane), kHeads rows of k and as many of v in flight.
// Instructions count here (issue slots were 63 to 77 % busy with addresses computed row by
// row): two base addresses, stepped by constant strides.
// ---------------------------------------------------------------------------
namespace {
constexpr int kHeads = 8;
struct MoveArgs {
  PagedBatch pb;
  KvPages kv;
  uint16_t* ck;
  uint16_t* cv;
  int s_max, n_tokens, n_blocks_tok;
  int* err;
};
}  // namespace

template <bool FP8, bool TO_PAGES>
__global__ void __launch_bounds__(32 * kWarps) kv_move_kernel(const MoveArgs a) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const long long item = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const long long items = (long long)a.n_tokens * a.n_blocks_tok;
  if (item >= items) {
    paged_check_lists(a.pb, a.n_tokens, item - items, lane, a.err);
    return;
  }
  const int tok = (int)(item / a.n_blocks_tok);
  const int Hkv = a.kv.Hkv;
  PagedToken at;
  if (!paged_seq_of(a.pb, a.n_tokens, tok, lane, &at)) return;
  const int t = tok - at.start;
  if (at.ctx >= a.s_max - t) {
    if (lane == 0) record_error(a.err, kErrCapacity);
    return;
  }
  const int pos = at.ctx + t;
  const long long cell = paged_row(a.pb, a.kv, at.b, pos, lane == 0 ? a.err : nullptr);
  if (cell < 0) return;
  constexpr int kIter = kHeads / 2;
  const int h0 = (int)(item % a.n_blocks_tok) * kHeads + (lane >> 4);  // heads h0, h0 + 2, ...
  const int d = (lane & 15) * 8;
  const int n = min(kIter, (Hkv - h0 + 1) >> 1);
  constexpr int kCell = FP8 ? 1 : 2;  // bytes a value in the pages
  const long long flat = (((long long)at.b * Hkv + h0) * a.s_max + pos) * 128 + d, flat_step = 256ll * a.s_max;
  const long long page = ((cell + ((long long)h0 << a.kv.page_shift)) * 128 + d) * kCell,
                  page_step = (256ll << a.kv.page_shift) * kCell;
  uint16_t* flat_kv[2] = {a.ck + flat, a.cv + flat};
  uint8_t* page_kv[2] = {a.kv.k + page, a.kv.v + page};
  uint4 in[2][kIter];
#pragma unroll
  for (int z = 0; z < 2; ++z)
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
      if (i >= n) continue;
      if (TO_PAGES) {
        in[z][i] = *reinterpret_cast<const uint4*>(flat_kv[z] + i * flat_step);
      } else if (FP8) {
        const uint2 u = *reinterpret_cast<const uint2*>(page_kv[z] + i * page_step);
        in[z][i] = make_uint4(u.x, u.y, 0, 0);
      } else {
        in[z][i] = *reinterpret_cast<const uint4*>(page_kv[z] + i * page_step);
      }
    }
#pragma unroll
  for (int z = 0; z < 2; ++z)
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
      if (i >= n) continue;
      uint16_t* fp = flat_kv[z] + i * flat_step;
      uint8_t* pp = page_kv[z] + i * page_step;
      if (!FP8) {
        *reinterpret_cast<uint4*>(TO_PAGES ? pp : reinterpret_cast<uint8_t*>(fp)) = in[z][i];
        continue;
      }
      const float scale = (z ? a.kv.v_scale : a.kv.k_scale)[h0 + 2 * i];
      uint64_t f[4];
      if (TO_PAGES) {
        unpack8(in[z][i], f);
        *reinterpret_cast<uint2*>(pp) = quant8(f, 1.0f / scale);
      } else {
        const uint64_t s2 = f2_pack(__float_as_uint(scale), __float_as_uint(scale));
        const uint32_t w[2] = {in[z][i].x, in[z][i].y};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 p = e4m3x2_to_f32x2((uint16_t)(w[j >> 1] >> (16 * (j & 1))));
          f[j] = f2_mul(f2_pack(__float_as_uint(p.x), __float_as_uint(p.y)), s2);
        }
        *reinterpret_cast<uint4*>(fp) = pack8(f);
      }
    }
}

int launch_kv_move(bool to_pages, uint16_t* ck, uint16_t* cv, int s_max, int n_tokens, const PagedBatch& pb,
                   const KvPages& kv, int* err, cudaStream_t s) {
  MoveArgs a;
  a.pb = pb;
  a.kv = kv;
  a.ck = ck;
  a.cv = cv;
  a.s_max = s_max;
  a.n_tokens = n_tokens;
  a.n_blocks_tok = (kv.Hkv + kHeads - 1) / kHeads;
  a.err = err;
  const long long blocks = blocks_of((long long)n_tokens * a.n_blocks_tok, pb.B, kWarps);
  if (blocks >= (1ll << 31)) {
    set_last_error("kv move: %d tokens exceed the grid limit", n_tokens);
    return -2;
  }
  auto k = to_pages ? (kv.fp8 ? kv_move_kernel<true, true> : kv_move_kernel<false, true>)
                    : (kv.fp8 ? kv_move_kernel<true, false> : kv_move_kernel<false, false>);
  q3_launch(k, (unsigned)blocks, 32 * kWarps, 0, s, a);
  return cudaGetLastError() == cudaSuccess ? 0 : -6;
}

}  // namespace q3
