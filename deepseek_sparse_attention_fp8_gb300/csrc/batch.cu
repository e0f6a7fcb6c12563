// Batch metadata from the requests' lengths: the exclusive prefix sum of the
// new tokens (query_start_loc), the blocks each request takes from the queue
// of free blocks (another prefix sum, of ceil((ctx+new)/bs) - ceil(ctx/bs)),
// and per token its request, position and cache slot.
//
// The requests are taken in chunks of one per thread: a chunk's two prefix
// sums are block scans with a carry, then the threads share the chunk's
// tokens, each finding its request by binary search in shared memory. A
// token at the first position of a new block stores the block in the table,
// so no thread walks a long request's blocks alone.
#include "common.cuh"
#include "ptx.cuh"

namespace dsa {
namespace {

constexpr int kThreads = 1024;

struct BatchParams {
  const int32_t *ctx, *add, *free_blocks, *free_head;
  int32_t* free_head_out;
  int32_t* table;
  int32_t B, block_size, num_free, bt_stride, max_tokens;
  int32_t *seq_lens, *qsl, *token_req, *positions;
  int64_t* slot_map;
  int32_t* dev_status;
};

// Inclusive scan over the block; *total is the block's sum.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* warp_sums, int64_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int64_t u = __shfl_up_sync(0xFFFFFFFFu, v, off);
    if (lane >= off) v += u;
  }
  if (lane == 31) warp_sums[warp] = v;
  __syncthreads();
  int64_t before = 0, sum = 0;
  for (int w = 0; w < kThreads / 32; ++w) {
    const int64_t s = warp_sums[w];
    if (w < warp) before += s;
    sum += s;
  }
  *total = sum;
  __syncthreads();  // the sums may be overwritten
  return v + before;
}

__global__ void __launch_bounds__(kThreads) build_batch_kernel(const __grid_constant__ BatchParams p) {
  __shared__ int64_t warp_sums[kThreads / 32];
  __shared__ int32_t s_start[kThreads + 1], s_ctx[kThreads], s_take[kThreads];
  const int tid = threadIdx.x;
  uint32_t err = 0;
  const int64_t head = p.free_blocks != nullptr ? *p.free_head : 0;
  const bool head_ok = head >= 0 && head <= p.num_free;
  int64_t tokens = 0, taken = 0;  // of the chunks before
  for (int b0 = 0; b0 < p.B; b0 += kThreads) {
    const int n = min(kThreads, p.B - b0), b = b0 + tid;
    int64_t c = 0, a = 0;
    if (tid < n) {
      c = p.ctx[b];
      a = p.add[b];
      if (c < 0 || a < 0 || c + a > INT32_MAX) {
        err |= DSA_DEVERR_SEQ_LEN;
        c = c < 0 ? 0 : c;
        a = 0;
      }
    }
    int64_t sum;
    const int64_t last = tokens + block_scan(a, warp_sums, &sum);
    const int64_t cap = p.max_tokens;
    const int64_t start = min(last - a, cap);
    if (last > cap) err |= a > 0 ? DSA_DEVERR_SEQ_LEN : 0u;
    a = min(last, cap) - start;
    const int64_t held = (c + p.block_size - 1) / p.block_size;
    int64_t take = 0;
    if (tid < n && p.free_blocks != nullptr)
      take = max(int64_t(0), min((c + a + p.block_size - 1) / p.block_size, int64_t(p.bt_stride)) - held);
    int64_t sum_take;
    const int64_t take_end = taken + block_scan(take, warp_sums, &sum_take);
    if (tid < n) {
      s_start[tid] = static_cast<int32_t>(start);
      s_ctx[tid] = static_cast<int32_t>(c);
      // first index of the request's blocks in the queue; past the queue's
      // end all are alike (none left)
      s_take[tid] = static_cast<int32_t>(min(head + take_end - take, int64_t(INT32_MAX)));
      if (tid == n - 1) s_start[n] = static_cast<int32_t>(start + a);
      p.seq_lens[b] = static_cast<int32_t>(c + a);
      p.qsl[b] = static_cast<int32_t>(start);
      if (b == p.B - 1) p.qsl[p.B] = static_cast<int32_t>(start + a);
    }
    tokens += sum;
    taken += sum_take;
    __syncthreads();
    for (int t = s_start[0] + tid; t < s_start[n]; t += kThreads) {
      int lo = 0, hi = n - 1;  // the last request that starts at or before t
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (s_start[mid] <= t) lo = mid; else hi = mid - 1;
      }
      const int req = b0 + lo;
      const int32_t pos = s_ctx[lo] + (t - s_start[lo]);
      const int j = pos / p.block_size, off = pos - j * p.block_size;
      const int held_r = (s_ctx[lo] - 1) / p.block_size + (s_ctx[lo] > 0 ? 1 : 0);
      int64_t slot = -1;
      if (j >= p.bt_stride) {
        err |= DSA_DEVERR_SEQ_LEN;
      } else {
        int32_t* entry = p.table + static_cast<int64_t>(req) * p.bt_stride + j;
        int32_t blk;
        if (j >= held_r && p.free_blocks != nullptr) {
          const int64_t at = static_cast<int64_t>(s_take[lo]) + (j - held_r);
          const bool got = head_ok && at < p.num_free;
          blk = got ? __ldg(p.free_blocks + at) : -1;
          if (!got) err |= DSA_DEVERR_NO_BLOCKS;
          else if (blk < 0) err |= DSA_DEVERR_BLOCK_OOB;
          if (off == 0) *entry = blk;
        } else {
          blk = *entry;
          if (blk < 0) err |= DSA_DEVERR_BLOCK_OOB;
        }
        if (blk >= 0) slot = static_cast<int64_t>(blk) * p.block_size + off;
      }
      p.token_req[t] = req;
      p.positions[t] = pos;
      p.slot_map[t] = slot;
    }
    __syncthreads();
  }
  if (p.B == 0 && tid == 0) p.qsl[0] = 0;
  for (int64_t t = min(tokens, int64_t(p.max_tokens)) + tid; t < p.max_tokens; t += kThreads) {
    p.token_req[t] = -1;
    p.positions[t] = 0;
    p.slot_map[t] = -1;
  }
  if (tid == 0 && p.free_blocks != nullptr)
    *p.free_head_out = static_cast<int32_t>(head_ok ? min(head + taken, int64_t(p.num_free)) : head);
  if (err) report(p.dev_status, err);
}

}  // namespace
}  // namespace dsa

using namespace dsa;

extern "C" dsa_status_t dsa_build_batch(const int32_t* ctx_lens, const int32_t* new_lens, int32_t B,
                                        int32_t block_size, const int32_t* free_blocks, int32_t num_free,
                                        const int32_t* free_head, int32_t* free_head_out, int32_t* block_table,
                                        int32_t bt_stride, int32_t max_tokens, int32_t* seq_lens,
                                        int32_t* query_start_loc, int32_t* token_req, int32_t* positions,
                                        int64_t* slot_map, int32_t* dev_status, dsa_stream_t stream) {
  if (B < 0 || block_size <= 0 || num_free < 0 || bt_stride < 0 || max_tokens < 0)
    return fail(DSA_ERR_INVALID_ARG, "dsa_build_batch: negative or zero size argument");
  if (block_size % 64)
    return fail(DSA_ERR_UNSUPPORTED, "dsa_build_batch: block_size %d not a multiple of 64", block_size);
  if (!query_start_loc || (B > 0 && (!ctx_lens || !new_lens || !block_table || !seq_lens)) ||
      (max_tokens > 0 && (!token_req || !positions || !slot_map)))
    return fail(DSA_ERR_INVALID_ARG, "dsa_build_batch: null pointer");
  if (free_blocks && (!free_head || !free_head_out))
    return fail(DSA_ERR_INVALID_ARG, "dsa_build_batch: free_blocks without free_head and free_head_out");
  if (!free_blocks && num_free > 0)
    return fail(DSA_ERR_INVALID_ARG, "dsa_build_batch: num_free without free_blocks");
  dsa_status_t st = check_device();
  if (st != DSA_OK) return st;
  BatchParams p;
  p.ctx = ctx_lens;
  p.add = new_lens;
  p.free_blocks = free_blocks;
  p.free_head = free_head;
  p.free_head_out = free_head_out;
  p.table = block_table;
  p.B = B;
  p.block_size = block_size;
  p.num_free = num_free;
  p.bt_stride = bt_stride;
  p.max_tokens = max_tokens;
  p.seq_lens = seq_lens;
  p.qsl = query_start_loc;
  p.token_req = token_req;
  p.positions = positions;
  p.slot_map = slot_map;
  p.dev_status = dev_status;
  build_batch_kernel<<<1, kThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(p);
  return check_launch("build_batch_kernel");
}
