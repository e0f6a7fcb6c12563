// Dense causal MLA attention of new tokens over the paged latent caches.
//
// For query token t of request b (position pos) and head h:
//   s_i = scale * q[t,h,:] . kv[i,:]   for the keys i <= pos
//   out = sum_i softmax(s)_i * kv[i, :512]     lse = log sum_i exp(s_i)
//
// The simple form: one warp per (token, head), the 8 warps of a CTA taking 8
// heads of a token; a lane holds dims {2 lane + 64 i, 2 lane + 64 i + 1} of q
// and of the output, and the softmax runs over the keys one at a time.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>

#include "common.cuh"
#include "ptx.cuh"

namespace dsa {
namespace {

constexpr int kDk = 576, kDv = 512, kF8Row = 656;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct DenseParams {
  const uint16_t* q;
  const uint8_t* kv;
  int64_t block_bytes;
  int32_t num_blocks;
  const int32_t* block_table;
  int32_t bt_stride;
  const int32_t *seq_lens, *qsl;
  int32_t B, T, H, block_size;
  float scale_log2;
  uint16_t* out;
  float* lse;
  int32_t* dev_status;
};

template <bool F8>
__global__ void __launch_bounds__(256) dense_mla_simple_kernel(const __grid_constant__ DenseParams p) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = blockIdx.x, h = blockIdx.y * 8 + warp;
  if (h >= p.H || t >= __ldg(p.qsl + p.B)) return;
  int lo = 0, hi = p.B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (__ldg(p.qsl + mid) <= t) lo = mid; else hi = mid - 1;
  }
  const int q0 = __ldg(p.qsl + lo), q1 = __ldg(p.qsl + lo + 1);
  int64_t valid = static_cast<int64_t>(__ldg(p.seq_lens + lo)) - (q1 - q0) + (t - q0) + 1;
  const int64_t cap = static_cast<int64_t>(p.bt_stride) * p.block_size;
  if (valid < 1 || valid > cap) {
    if (lane == 0) report(p.dev_status, DSA_DEVERR_SEQ_LEN);
    valid = max(int64_t(0), min(valid, cap));
  }
  const int64_t row = static_cast<int64_t>(t) * p.H + h;
  float2 q[9], acc[8];
  for (int i = 0; i < 9; ++i)
    q[i] = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(p.q + row * kDk + 64 * i + 2 * lane));
  for (int i = 0; i < 8; ++i) acc[i] = make_float2(0.f, 0.f);
  float m = kNegSentinel, l = 0.f;
  const int32_t* bt = p.block_table + static_cast<int64_t>(lo) * p.bt_stride;
  for (int64_t key = 0; key < valid; ++key) {
    const int j = static_cast<int>(key / p.block_size);
    const int blk = __ldg(bt + j);
    if (blk < 0 || blk >= p.num_blocks) {
      if (lane == 0) report(p.dev_status, DSA_DEVERR_BLOCK_OOB);
      key = static_cast<int64_t>(j + 1) * p.block_size - 1;
      continue;
    }
    const int64_t off = key - static_cast<int64_t>(j) * p.block_size;
    const uint8_t* src = p.kv + blk * p.block_bytes + off * (F8 ? kF8Row : 2 * kDk);
    float2 k[9];
    if constexpr (F8) {
      const float4 sc = __ldg(reinterpret_cast<const float4*>(src + kDv));
      const float s4[4] = {sc.x, sc.y, sc.z, sc.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        uint32_t two;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(two) : "h"(__ldg(reinterpret_cast<const uint16_t*>(src + 64 * i) + lane)));
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&two));
        k[i] = make_float2(f.x * s4[i >> 1], f.y * s4[i >> 1]);
      }
      const uint32_t r = __ldg(reinterpret_cast<const uint32_t*>(src + kDv + 16) + lane);
      k[8] = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&r));
    } else {
#pragma unroll
      for (int i = 0; i < 9; ++i) {
        const uint32_t r = __ldg(reinterpret_cast<const uint32_t*>(src) + 32 * i + lane);
        k[i] = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&r));
      }
    }
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 9; ++i) s = fmaf(q[i].x, k[i].x, fmaf(q[i].y, k[i].y, s));
#pragma unroll
    for (int off2 = 16; off2 > 0; off2 >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, off2);
    s *= p.scale_log2;
    const float m_new = fmaxf(m, s);
    const float a = exp2f(m - m_new), w = exp2f(s - m_new);
    l = l * a + w;
    m = m_new;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      acc[i].x = fmaf(w, k[i].x, acc[i].x * a);
      acc[i].y = fmaf(w, k[i].y, acc[i].y * a);
    }
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    *reinterpret_cast<__nv_bfloat162*>(p.out + row * kDv + 64 * i + 2 * lane) =
        __floats2bfloat162_rn(acc[i].x * inv, acc[i].y * inv);
  if (lane == 0 && p.lse != nullptr) p.lse[row] = l > 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
}

dsa_status_t dense_impl(const void* q, const void* kv_cache, int64_t kv_block_stride, int32_t num_blocks,
                        const int32_t* block_table, int32_t bt_stride, const int32_t* seq_lens,
                        const int32_t* query_start_loc, int32_t B, int32_t T, int32_t H, int32_t Dk, int32_t Dv,
                        int32_t block_size, float softmax_scale, int32_t num_kv_splits, void* out, float* lse,
                        void* workspace, size_t ws_bytes, int32_t* dev_status, dsa_stream_t stream, bool f8,
                        const char* name) {
  if (B < 0 || T < 0 || H <= 0 || block_size <= 0 || num_blocks < 0 || bt_stride < 0)
    return fail(DSA_ERR_INVALID_ARG, "%s: negative or zero size argument", name);
  if (Dk != kDk || Dv != kDv)
    return fail(DSA_ERR_UNSUPPORTED, "%s: (Dk, Dv) = (%d, %d), only (576, 512)", name, Dk, Dv);
  if (H > 128) return fail(DSA_ERR_UNSUPPORTED, "%s: H=%d > 128", name, H);
  if (block_size % 64) return fail(DSA_ERR_UNSUPPORTED, "%s: block_size %d not a multiple of 64", name, block_size);
  if (!(softmax_scale > 0.f) || !std::isfinite(softmax_scale))
    return fail(DSA_ERR_INVALID_ARG, "%s: softmax_scale must be positive and finite", name);
  if (num_kv_splits < DSA_KV_SPLITS_BATCH_INVARIANT || num_kv_splits > 1)
    return fail(DSA_ERR_INVALID_ARG, "%s: num_kv_splits %d not in {-1, 0, 1}", name, num_kv_splits);
  if (T > 0 && B == 0) return fail(DSA_ERR_INVALID_ARG, "%s: T > 0 with B == 0", name);
  if (T == 0) return DSA_OK;
  if (!q || !kv_cache || !block_table || !seq_lens || !query_start_loc || !out)
    return fail(DSA_ERR_INVALID_ARG, "%s: null pointer", name);
  if (!aligned16(q) || !aligned16(kv_cache) || !aligned16(out))
    return fail(DSA_ERR_INVALID_ARG, "%s: q, kv_cache and out must be 16-byte aligned", name);
  const int64_t row = f8 ? kF8Row : kDk;  // a cache row in the units of kv_block_stride
  if (kv_block_stride < block_size * row)
    return fail(DSA_ERR_INVALID_ARG, "%s: kv_block_stride %lld < block_size rows of %lld", name,
                static_cast<long long>(kv_block_stride), static_cast<long long>(row));
  if (kv_block_stride % row)
    return fail(DSA_ERR_UNSUPPORTED, "%s: kv_block_stride %lld is not a whole number of %lld-unit rows", name,
                static_cast<long long>(kv_block_stride), static_cast<long long>(row));
  if (num_blocks * (kv_block_stride / row) >= (int64_t(1) << 31))
    return fail(DSA_ERR_UNSUPPORTED, "%s: the cache holds 2^31 rows or more", name);
  dsa_status_t st = check_device();
  if (st != DSA_OK) return st;
  const size_t need = dense_mla_workspace_size(T, H, Dv, num_kv_splits);
  if (need && (workspace == nullptr || ws_bytes < need || !aligned16(workspace)))
    return fail(DSA_ERR_WORKSPACE, "%s: needs %zu workspace bytes (16-byte aligned), got %zu", name, need, ws_bytes);
  DenseParams p;
  p.q = static_cast<const uint16_t*>(q);
  p.kv = static_cast<const uint8_t*>(kv_cache);
  p.block_bytes = f8 ? kv_block_stride : 2 * kv_block_stride;
  p.num_blocks = num_blocks;
  p.block_table = block_table;
  p.bt_stride = bt_stride;
  p.seq_lens = seq_lens;
  p.qsl = query_start_loc;
  p.B = B;
  p.T = T;
  p.H = H;
  p.block_size = block_size;
  p.scale_log2 = softmax_scale * kLog2e;
  p.out = static_cast<uint16_t*>(out);
  p.lse = lse;
  p.dev_status = dev_status;
  const dim3 grid(static_cast<unsigned>(T), static_cast<unsigned>((H + 7) / 8));
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (f8) dense_mla_simple_kernel<true><<<grid, 256, 0, s>>>(p);
  else dense_mla_simple_kernel<false><<<grid, 256, 0, s>>>(p);
  return check_launch("dense_mla_simple_kernel");
}

}  // namespace
}  // namespace dsa

using namespace dsa;

extern "C" size_t dense_mla_workspace_size(int32_t T, int32_t H, int32_t Dv, int32_t num_kv_splits) {
  (void)T, (void)H, (void)Dv, (void)num_kv_splits;
  return 0;
}

extern "C" dsa_status_t dense_mla_attention(const void* q, const void* kv_cache, int64_t kv_block_stride,
                                            int32_t num_blocks, const int32_t* block_table, int32_t bt_stride,
                                            const int32_t* seq_lens, const int32_t* query_start_loc, int32_t B,
                                            int32_t T, int32_t H, int32_t Dk, int32_t Dv, int32_t block_size,
                                            float softmax_scale, int32_t num_kv_splits, void* out, float* lse,
                                            void* workspace, size_t ws_bytes, int32_t* dev_status,
                                            dsa_stream_t stream) {
  return dense_impl(q, kv_cache, kv_block_stride, num_blocks, block_table, bt_stride, seq_lens, query_start_loc, B, T,
                    H, Dk, Dv, block_size, softmax_scale, num_kv_splits, out, lse, workspace, ws_bytes, dev_status,
                    stream, false, "dense_mla_attention");
}

extern "C" dsa_status_t dense_mla_attention_fp8(const void* q, const uint8_t* kv_cache, int64_t kv_block_stride_bytes,
                                                int32_t num_blocks, const int32_t* block_table, int32_t bt_stride,
                                                const int32_t* seq_lens, const int32_t* query_start_loc, int32_t B,
                                                int32_t T, int32_t H, int32_t Dk, int32_t Dv, int32_t block_size,
                                                float softmax_scale, int32_t num_kv_splits, void* out, float* lse,
                                                void* workspace, size_t ws_bytes, int32_t* dev_status,
                                                dsa_stream_t stream) {
  return dense_impl(q, kv_cache, kv_block_stride_bytes, num_blocks, block_table, bt_stride, seq_lens, query_start_loc,
                    B, T, H, Dk, Dv, block_size, softmax_scale, num_kv_splits, out, lse, workspace, ws_bytes,
                    dev_status, stream, true, "dense_mla_attention_fp8");
}
