// Causal grouped-query attention of a ragged batch's new tokens over a paged KV cache.
#include "paged.cuh"
#include "internal.h"

namespace q3 {

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

size_t paged_attention_bytes(int B, int Hq, int Hkv, int max_q) { return 256; }

int launch_attention_paged(const uint16_t* q, long long ldq, int n_tokens, int max_q, const PagedBatch& pb,
                           const KvPages& kv, int Hq, void* scratch, uint16_t* out, long long ldo, int* err,
                           cudaStream_t s, bool o_f16) {
  const long long blocks = ((long long)n_tokens * Hq + 3) / 4;
  if (blocks >= (1ll << 31)) {
    set_last_error("attention_paged: %d tokens exceed the grid limit", n_tokens);
    return -2;
  }
  q3_launch(kv.fp8 ? attn_paged_simple_kernel<true> : attn_paged_simple_kernel<false>, (unsigned)blocks, 128, 0, s, pb,
            kv, Hq, n_tokens, max_q, q, ldq, out, ldo, o_f16 ? 1 : 0, err);
  return cudaGetLastError() == cudaSuccess ? 0 : -6;
}

}  // namespace q3
