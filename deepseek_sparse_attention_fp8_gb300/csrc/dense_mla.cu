// Dense causal MLA attention of new tokens over the paged latent caches.
//
// For query token t of request b (position pos) and head h:
//   s_i = scale * q[t,h,:] . kv[i,:]   for the keys i <= pos
//   out = sum_i softmax(s)_i * kv[i, :512]     lse = log sum_i exp(s_i)
//
// Three kernels do it. All cut the batch's rows into row tiles (the rows of a
// request see the same latent rows, whatever their head) and the row tiles'
// steps of 128 keys into equal runs, one per group of CTAs, on the device:
//   single CTAs    (dense_mla_rows.cu)  16 or 32 rows, keys along M: few rows a
//                  request, memory bound;
//   pairs          (here, dense_mla_pair.cuh)  128 rows: single tokens of many
//                  heads, short prompts;
//   clusters of 4  (dense_mla_quad.cu)  256 rows: chunks over long contexts;
//                  they work as two pairs each where that is faster.
// A row tile cut by a run's end leaves fp32 partials, at most two per run, which
// dense_mla_merge_kernel joins. Behind 32 requests of 8192 keys and 128 heads, in
// runs of 27 steps, it reads 28 MB of them (106 parts) and takes, with its launch,
// 10 of the call's 95 us (caches cold).
#include <algorithm>

#include "dense_mla_pair.cuh"

namespace dsa {
namespace {

using namespace dense;

// Joins the partials of the row tile that starts in run blockIdx.y and goes on
// behind it: out = sum_j 2^(m_j - M) o_j / sum_j 2^(m_j - M) l_j. A thread takes
// 16 columns, i.e. dims, of a row: one 32-byte sector of the result. Partials
// lie as the accumulators do in tensor memory: the four-CTA kernel's in 512
// columns of 128 rows per CTA, the pair kernel's in 256 columns, a row's upper
// dims in lane + 64.
template <bool QUAD>
__device__ __forceinline__ void merge_tile(const DenseParams& p, const int4 d, int run) {
  constexpr int kRows = QUAD ? 256 : 128, kGroups = QUAD ? 32 : 16;
  const int r = blockIdx.x / kGroups, g = blockIdx.x % kGroups;  // CTA, 16 columns
  if (r > 1) return;
  const int lane = threadIdx.x, in_tile = QUAD ? 128 * r + lane : 64 * r + (lane & 63);
  const int dim = QUAD ? 128 * (g >> 4) + 16 * (g & 7) + ((g >> 3) & 1) * 256 : 256 * (lane >> 6) + 16 * g;
  if (in_tile >= d.y) return;
  const int parts = d.z + 1;
  const auto slot = [&](int j) { return j == 0 ? 2 * run + 1 : 2 * (run + j); };
  float M = kNegSentinel;
  for (int j = 0; j < parts; ++j) M = fmaxf(M, p.ml_part[slot(j) * kRows + in_tile].x);
  float den = 0.f;
  float4 acc[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int j = 0; j < parts; ++j) {
    const float2 ml = p.ml_part[slot(j) * kRows + in_tile];
    const float w = exp2f(ml.x - M);
    den = fmaf(w, ml.y, den);
    const float4* o = p.o_part + (static_cast<int64_t>(2 * slot(j) + r) * (4 * kGroups) + 4 * g) * 128 + lane;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 v = o[i * 128];
      acc[i].x = fmaf(w, v.x, acc[i].x);
      acc[i].y = fmaf(w, v.y, acc[i].y);
      acc[i].z = fmaf(w, v.z, acc[i].z);
      acc[i].w = fmaf(w, v.w, acc[i].w);
    }
  }
  const float inv = den != 0.f ? 1.f / den : 0.f;
  const int64_t row = static_cast<int64_t>(d.x) + in_tile;
  uint4* dst = reinterpret_cast<uint4*>(p.out + row * kDv + dim);
#pragma unroll
  for (int e = 0; e < 2; ++e)
    dst[e] = make_uint4(pack_bf16(acc[2 * e].x * inv, acc[2 * e].y * inv), pack_bf16(acc[2 * e].z * inv, acc[2 * e].w * inv),
                        pack_bf16(acc[2 * e + 1].x * inv, acc[2 * e + 1].y * inv),
                        pack_bf16(acc[2 * e + 1].z * inv, acc[2 * e + 1].w * inv));
  if (dim == 0 && p.lse != nullptr) p.lse[row] = den != 0.f ? (M + log2f(den)) * kLn2 : -INFINITY;
}

// The kernel of few rows leaves them row by row: a block takes a row, a thread
// four dims.
__device__ __forceinline__ void merge_rows(const DenseParams& p, const int4 d, int run) {
  const int row = blockIdx.x, parts = d.z + 1;
  if (row >= d.y) return;
  const auto slot = [&](int j) { return static_cast<int64_t>(j == 0 ? 2 * run + 1 : 2 * (run + j)) * p.single_rows + row; };
  float M = kNegSentinel, den = 0.f;
  for (int j = 0; j < parts; ++j) M = fmaxf(M, p.ml_part[slot(j)].x);
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int j = 0; j < parts; ++j) {
    const float2 ml = p.ml_part[slot(j)];
    const float4 v = p.o_part[slot(j) * (kDv / 4) + threadIdx.x];
    const float w = exp2f(ml.x - M);
    den = fmaf(w, ml.y, den);
    acc.x = fmaf(w, v.x, acc.x);
    acc.y = fmaf(w, v.y, acc.y);
    acc.z = fmaf(w, v.z, acc.z);
    acc.w = fmaf(w, v.w, acc.w);
  }
  const float inv = den != 0.f ? 1.f / den : 0.f;
  const int64_t g = static_cast<int64_t>(d.x) + row;
  reinterpret_cast<uint2*>(p.out + g * kDv)[threadIdx.x] =
      make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
  if (threadIdx.x == 0 && p.lse != nullptr) p.lse[g] = den != 0.f ? (M + log2f(den)) * kLn2 : -INFINITY;
}

__global__ void __launch_bounds__(128) dense_mla_merge_kernel(const __grid_constant__ DenseParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int4 d = p.desc[blockIdx.y];
  if (d.z <= 0) return;
  if (d.w == kSingle) merge_rows(p, d, blockIdx.y);
  else if (d.w == kQuad) merge_tile<true>(p, d, blockIdx.y);
  else merge_tile<false>(p, d, blockIdx.y);
}

template <bool F8>
__global__ void __launch_bounds__(pairs::threads(F8), 1) dense_mla_kernel(const __grid_constant__ DenseParams p,
                                                                          const __grid_constant__ Maps maps,
                                                                          const __grid_constant__ CodeMaps code_maps) {
  extern __shared__ __align__(1024) uint8_t smem[];
  if (misaligned(p, smem)) return;
  pairs::set_up<F8>(reinterpret_cast<pairs::Bars*>(smem + pairs::kSmBar), maps);  // overlaps the kernel before
  asm volatile("griddepcontrol.wait;" ::: "memory");
  plan_run<pairs::threads(F8), kPair>(p, reinterpret_cast<Run*>(smem + kSmRun), smem);
  pairs::run_pair<F8>(p, maps, code_maps, smem);
}

FuncAttrOnce g_smem_dense[2], g_smem_merge;

int num_pairs() { return std::max(1, num_sms() / 2); }
// partials of 128 rows per pair; a quad's 256 rows take two pairs' worth, and
// there are at most half as many; a single CTA's 32 rows take a quarter
size_t o_part_bytes(int pairs) { return static_cast<size_t>(2 * pairs) * 128 * kDv * sizeof(float); }
size_t ml_part_bytes(int pairs) { return static_cast<size_t>(2 * pairs) * 128 * sizeof(float2); }
size_t workspace_bytes(int pairs) { return o_part_bytes(pairs) + ml_part_bytes(pairs) + num_sms() * sizeof(int4); }

template <bool F8>
dsa_status_t launch_pairs(const DenseParams& p, const void* q, const void* kv, cudaStream_t s) {
  Maps maps;
  CodeMaps code_maps = {};
  dsa_status_t st = make_maps(&maps, p, F8, q, kv, 64, 9);
  if (st == DSA_OK && F8) st = make_code_maps(&code_maps, p, kv);
  if (st != DSA_OK) return st;
  if ((st = allow_smem(dense_mla_kernel<F8>, kSmTotal, g_smem_dense[F8])) != DSA_OK) return st;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * p.pairs));
  cfg.blockDim = dim3(pairs::threads(F8));
  cfg.dynamicSmemBytes = kSmTotal;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  cudaError_t e = cudaLaunchKernelEx(&cfg, dense_mla_kernel<F8>, p, maps, code_maps);
  if (e != cudaSuccess) return fail(DSA_ERR_CUDA, "dense_mla_kernel launch failed: %s", cudaGetErrorString(e));
  return DSA_OK;
}

dsa_status_t launch_merge(const DenseParams& p, cudaStream_t s) {
  dsa_status_t st = allow_smem(dense_mla_merge_kernel, 0, g_smem_merge);
  if (st != DSA_OK) return st;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = p.singles > 0 ? dim3(p.single_rows, p.singles) : dim3(p.quads > 0 ? 64 : 32, p.pairs);
  cfg.blockDim = dim3(128);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, dense_mla_merge_kernel, p);
  if (e != cudaSuccess) return fail(DSA_ERR_CUDA, "dense_mla_merge_kernel launch failed: %s", cudaGetErrorString(e));
  return DSA_OK;
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
  if (static_cast<int64_t>(T) * H >= (int64_t(1) << 31))
    return fail(DSA_ERR_UNSUPPORTED, "%s: 2^31 query rows or more", name);
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
  if (kv_block_stride / row >= (int64_t(1) << 31) || num_blocks * (kv_block_stride / row) >= (int64_t(1) << 31))
    return fail(DSA_ERR_UNSUPPORTED, "%s: the cache holds 2^31 rows or more", name);
  dsa_status_t st = check_device();
  if (st != DSA_OK) return st;
  const size_t need = dense_mla_workspace_size(T, H, Dv, num_kv_splits);
  if (need && (workspace == nullptr || ws_bytes < need || !aligned16(workspace)))
    return fail(DSA_ERR_WORKSPACE, "%s: needs %zu workspace bytes (16-byte aligned), got %zu", name, need, ws_bytes);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int pairs = num_pairs();
  DenseParams d = {};
  d.num_blocks = num_blocks;
  d.rows_per_block = static_cast<int32_t>(kv_block_stride / row);
  d.total_rows = static_cast<int32_t>(std::max<int64_t>(num_blocks * (kv_block_stride / row), 1));
  d.block_table = block_table;
  d.bt_stride = bt_stride;
  d.seq_lens = seq_lens;
  d.qsl = query_start_loc;
  d.B = B;
  d.T = T;
  d.H = H;
  d.tpt[0] = 128 / H;
  d.tpt[1] = 256 / H;
  d.block_size = block_size;
  d.bs64 = block_size / 64;
  d.scale_log2 = softmax_scale * kLog2e;
  d.kv = static_cast<const uint8_t*>(kv_cache);
  d.cut = num_kv_splits == 0;
  d.out32 = (reinterpret_cast<uintptr_t>(out) & 31u) == 0;
  d.out = static_cast<uint16_t*>(out);
  d.lse = lse;
  if (d.cut) {
    d.o_part = static_cast<float4*>(workspace);
    d.ml_part = reinterpret_cast<float2*>(static_cast<uint8_t*>(workspace) + o_part_bytes(pairs));
    d.desc = reinterpret_cast<int4*>(reinterpret_cast<uint8_t*>(d.ml_part) + ml_part_bytes(pairs));
  }
  d.dev_status = dev_status;
  // Where requests have two row tiles and more on average, quads of CTAs may
  // be faster than pairs; the device decides (plan_run). Not when row tiles may
  // not be cut: then a token's result must not depend on the other requests.
  d.quads = d.cut && static_cast<int64_t>(T) * H >= int64_t(256) * B ? num_quads(f8) : 0;
  d.pairs = d.quads > 0 ? 2 * d.quads : pairs;
  d.single_rows = d.cut ? single_rows(B, T, H, f8) : 0;
  if (d.single_rows > 0) {
    d.singles = num_sms();
    d.tpt[kSingle] = d.single_rows / H;
    st = launch_singles(d, f8, q, kv_cache, s);
  } else if (d.quads > 0) {
    st = launch_quads(d, f8, q, kv_cache, s);
  } else {
    st = f8 ? launch_pairs<true>(d, q, kv_cache, s) : launch_pairs<false>(d, q, kv_cache, s);
  }
  if (st == DSA_OK && d.cut) st = launch_merge(d, s);
  return st == DSA_OK ? check_launch(name) : st;
}

}  // namespace
}  // namespace dsa

using namespace dsa;

extern "C" size_t dense_mla_workspace_size(int32_t T, int32_t H, int32_t Dv, int32_t num_kv_splits) {
  if (T <= 0 || H <= 0 || Dv <= 0 || num_kv_splits != 0) return 0;
  return dsa::workspace_bytes(dsa::num_pairs());
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
