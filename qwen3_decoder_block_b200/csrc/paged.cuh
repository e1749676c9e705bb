// Device view of a ragged batch over a paged KV cache, shared by the kernels that write,
// read and attend to it.
#pragma once
#include <cstdint>
#include "common.cuh"

namespace q3 {

// Sequence b's new tokens are rows q_start[b] .. q_start[b + 1] - 1 of the token buffers, at
// positions ctx_len[b] + 0, 1, ...; position p of sequence b lives in page
// table[b * max_pages + p / page_size], slot p % page_size.
struct PagedBatch {
  const int* q_start;
  const int* ctx_len;
  const int* table;
  int B, max_pages;
};

// Pages [n_pages][Hkv][page_size][128] of k and of v: bf16, or e4m3 with an fp32 scale per head.
struct KvPages {
  uint8_t* k;
  uint8_t* v;
  const float* k_scale;
  const float* v_scale;
  int n_pages, page_shift, Hkv, fp8;
};

// Whether sequence i's rows [first, end) can be rows of a buffer of n_tokens.
__device__ __forceinline__ bool paged_rows_ok(int first, int end, int n_tokens) {
  return first >= 0 && end >= first && end <= n_tokens;
}

// Reports an entry of q_start that decreases or lies outside [0, n_tokens], wherever it is: 32
// sequences a warp, in warps of their own behind those of the tokens (which leave a token at or
// behind such an entry alone, below), so that no token's chain of loads grows by the check.
__device__ __forceinline__ void paged_check_lists(const PagedBatch& pb, int n_tokens, long long warp, int lane, int* err) {
  const long long i = 32 * warp + lane;
  if (i < pb.B && !paged_rows_ok(pb.q_start[i], pb.q_start[i + 1], n_tokens)) record_error(err, kErrInvalid);
}

// The sequence holding row `tok` (the first that ends behind it), with its first row and cached
// length. Every lane of the warp calls it: 32 sequences a round, one memory latency each. False
// for a row of no sequence (before the first or behind the last), or at or behind a bad entry of
// q_start.
struct PagedToken {
  int b, start, ctx;
};
__device__ __forceinline__ bool paged_seq_of(const PagedBatch& pb, int n_tokens, int tok, int lane, PagedToken* out) {
  for (int base = 0; base < pb.B; base += 32) {
    const int i = base + lane;
    const bool in = i < pb.B;
    const int end = in ? pb.q_start[i + 1] : 0, first = in ? pb.q_start[i] : 0, ctx = in ? pb.ctx_len[i] : 0;
    const unsigned here = __ballot_sync(0xffffffffu, in && end > tok);
    const unsigned bad = __ballot_sync(0xffffffffu, in && !paged_rows_ok(first, end, n_tokens));
    // (up to the sequence found: the lowest bit of `here` and those below it)
    if (bad & (here ? here ^ (here - 1) : 0xffffffffu)) return false;
    if (here) {
      const int f = __ffs(here) - 1;
      out->b = base + f;
      out->start = __shfl_sync(0xffffffffu, first, f);
      out->ctx = __shfl_sync(0xffffffffu, ctx, f);
      return tok >= out->start;
    }
  }
  return false;
}

// Index of the cache row [page][0][slot] of position pos of sequence b (add head *
// page_size rows), or -1 with the reason recorded.
__device__ __forceinline__ long long paged_row(const PagedBatch& pb, const KvPages& kv, int b, int pos, int* err) {
  if (pos < 0) {
    record_error(err, kErrInvalid);
    return -1;
  }
  const int pi = pos >> kv.page_shift;
  if (pi >= pb.max_pages) {
    record_error(err, kErrCapacity);
    return -1;
  }
  const int page = pb.table[(long long)b * pb.max_pages + pi];
  if (page < 0 || page >= kv.n_pages) {
    record_error(err, kErrInvalid);
    return -1;
  }
  return (((long long)page * kv.Hkv) << kv.page_shift) + (pos & ((1 << kv.page_shift) - 1));
}

// Two fp32 as e4m3 (round to nearest even, magnitudes above 448 to 448; NaN stays NaN), the
// first in the low byte.
__device__ __forceinline__ uint16_t pack_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// Two e4m3 (low byte first) as two fp16, exactly.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t v) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(v));
  return r;
}
__device__ __forceinline__ float2 e4m3x2_to_f32x2(uint16_t v) {
  const uint32_t h = e4m3x2_to_f16x2(v);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

}  // namespace q3
