// Batch metadata from the requests' lengths: the exclusive prefix sum of the
// new tokens (query_start_loc), the blocks each request takes from the queue
// of free blocks (another prefix sum, of ceil((ctx+new)/bs) - ceil(ctx/bs)),
// and per token its request, position and cache slot.
//
// The requests are taken in chunks of one per thread: every CTA makes a chunk's
// two prefix sums (one block scan of both, with a carry) itself, then all
// threads share the chunk's tokens, four in a row each: one binary search in
// shared memory, and full 16-byte stores. A token at the first position of a
// new block stores the block in the table, so no thread walks a long request's
// blocks alone. Latency bounds it: a launch, the lengths, the free ids, the
// stores. When the queue's head is advanced in place the CTAs form one cluster,
// whose barrier keeps the head until all have read it; else there are as many
// as the tokens fill. From a graph, 512 requests with 131000 tokens: 7.0 us (a
// cluster of 8: 18, one CTA: 141); 32 requests with a token each: 5.2 us.
#include <algorithm>

#include "common.cuh"
#include "ptx.cuh"

namespace dsa {
namespace {

constexpr int kThreads = 1024;
constexpr int kCluster = 8;

struct BatchParams {
  const int32_t *ctx, *add, *free_blocks, *free_head;
  int32_t* free_head_out;
  int32_t* table;
  int32_t B, block_size, num_free, bt_stride, max_tokens;
  int32_t *seq_lens, *qsl, *token_req, *positions;
  int64_t* slot_map;
  int32_t vec;  // token_req, positions and slot_map are 16-byte aligned
  int32_t* dev_status;
};

// Inclusive scans of two values over the block; total: the block's sums.
__device__ __forceinline__ longlong2 block_scan(longlong2 v, longlong2* warp_sums, longlong2* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const auto scan = [&](longlong2 x) {
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int64_t a = __shfl_up_sync(0xFFFFFFFFu, x.x, off), b = __shfl_up_sync(0xFFFFFFFFu, x.y, off);
      if (lane >= off) {
        x.x += a;
        x.y += b;
      }
    }
    return x;
  };
  v = scan(v);
  if (lane == 31) warp_sums[warp] = v;
  __syncthreads();
  static_assert(kThreads == 1024, "a lane per warp");
  const longlong2 s = scan(warp_sums[lane]);
  total->x = __shfl_sync(0xFFFFFFFFu, s.x, 31);
  total->y = __shfl_sync(0xFFFFFFFFu, s.y, 31);
  const int64_t bx = __shfl_sync(0xFFFFFFFFu, s.x, (warp - 1) & 31), by = __shfl_sync(0xFFFFFFFFu, s.y, (warp - 1) & 31);
  if (warp > 0) {
    v.x += bx;
    v.y += by;
  }
  __syncthreads();  // the sums may be overwritten
  return v;
}

__global__ void __launch_bounds__(kThreads) build_batch_kernel(const __grid_constant__ BatchParams p) {
  __shared__ longlong2 warp_sums[kThreads / 32];
  __shared__ int32_t s_start[kThreads + 1], s_ctx[kThreads], s_take[kThreads];
  const int tid = threadIdx.x, rank = blockIdx.x;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kThreads;
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
    const int64_t cap = p.max_tokens, held = (c + p.block_size - 1) / p.block_size;
    const auto blocks_taken = [&](int64_t add) {
      return tid < n && p.free_blocks != nullptr
                 ? max(int64_t(0), min((c + add + p.block_size - 1) / p.block_size, int64_t(p.bt_stride)) - held)
                 : int64_t(0);
    };
    int64_t take = blocks_taken(a);
    longlong2 sum;
    longlong2 upto = block_scan(make_longlong2(a, take), warp_sums, &sum);
    const int64_t last = tokens + upto.x, start = min(last - a, cap);
    if (tokens + sum.x > cap) {  // the buffers are full: tokens are dropped, and their blocks not taken
      if (last > cap && a > 0) err |= DSA_DEVERR_SEQ_LEN;
      a = min(last, cap) - start;
      take = blocks_taken(a);
      longlong2 less;
      upto = block_scan(make_longlong2(a, take), warp_sums, &less);
      sum.y = less.y;
    }
    const int64_t take_end = taken + upto.y;
    if (tid < n) {
      s_start[tid] = static_cast<int32_t>(start);
      s_ctx[tid] = static_cast<int32_t>(c);
      // first index of the request's blocks in the queue; past the queue's
      // end all are alike (none left)
      s_take[tid] = static_cast<int32_t>(min(head + take_end - take, int64_t(INT32_MAX)));
      if (tid == n - 1) s_start[n] = static_cast<int32_t>(start + a);
      if (rank == 0) {
        p.seq_lens[b] = static_cast<int32_t>(c + a);
        p.qsl[b] = static_cast<int32_t>(start);
        if (b == p.B - 1) p.qsl[p.B] = static_cast<int32_t>(start + a);
      }
    }
    tokens += sum.x;
    taken += sum.y;
    __syncthreads();
    const int first = s_start[0], end = s_start[n];
    // four tokens from a multiple of 4 on; the chunk may begin and end inside
    for (int64_t t0 = (first & ~3) + int64_t(4) * (rank * kThreads + tid); t0 < end; t0 += 4 * step) {
      const int ta = max(static_cast<int>(t0), first);
      int lo = 0, hi = n - 1;  // the last request that starts at or before the first token
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (s_start[mid] <= ta) lo = mid; else hi = mid - 1;
      }
      int32_t req[4], pos[4];
      int64_t slot[4];
      int last_req = -1, last_j = -1;
      int32_t blk = -1;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t t = t0 + i;
        req[i] = pos[i] = 0;
        slot[i] = 0;
        if (t < first || t >= end) continue;
        while (t >= s_start[lo + 1]) ++lo;  // ends before n: t < s_start[n]
        pos[i] = s_ctx[lo] + (static_cast<int>(t) - s_start[lo]);
        req[i] = b0 + lo;
        const int j = pos[i] / p.block_size, off = pos[i] - j * p.block_size;
        slot[i] = -1;
        if (j >= p.bt_stride) {
          err |= DSA_DEVERR_SEQ_LEN;
          continue;
        }
        if (lo != last_req || j != last_j) {
          last_req = lo;
          last_j = j;
          int32_t* entry = p.table + static_cast<int64_t>(b0 + lo) * p.bt_stride + j;
          const int held = (s_ctx[lo] - 1) / p.block_size + (s_ctx[lo] > 0 ? 1 : 0);
          if (j >= held && p.free_blocks != nullptr) {
            const int64_t at = static_cast<int64_t>(s_take[lo]) + (j - held);
            const bool got = head_ok && at < p.num_free;
            blk = got ? __ldg(p.free_blocks + at) : -1;
            if (!got) err |= DSA_DEVERR_NO_BLOCKS;
            else if (blk < 0) err |= DSA_DEVERR_BLOCK_OOB;
            if (off == 0) *entry = blk;
          } else {
            blk = *entry;
            if (blk < 0) err |= DSA_DEVERR_BLOCK_OOB;
          }
        }
        if (blk >= 0) slot[i] = static_cast<int64_t>(blk) * p.block_size + off;
      }
      if (p.vec && t0 >= first && t0 + 4 <= end) {
        *reinterpret_cast<int4*>(p.token_req + t0) = make_int4(req[0], req[1], req[2], req[3]);
        *reinterpret_cast<int4*>(p.positions + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
        reinterpret_cast<longlong2*>(p.slot_map + t0)[0] = make_longlong2(slot[0], slot[1]);
        reinterpret_cast<longlong2*>(p.slot_map + t0)[1] = make_longlong2(slot[2], slot[3]);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (t0 + i < first || t0 + i >= end) continue;
          p.token_req[t0 + i] = req[i];
          p.positions[t0 + i] = pos[i];
          p.slot_map[t0 + i] = slot[i];
        }
      }
    }
    __syncthreads();
  }
  if (p.B == 0 && rank == 0 && tid == 0) p.qsl[0] = 0;
  for (int64_t t = min(tokens, int64_t(p.max_tokens)) + rank * kThreads + tid; t < p.max_tokens; t += step) {
    p.token_req[t] = -1;
    p.positions[t] = 0;
    p.slot_map[t] = -1;
  }
  if (p.free_head == p.free_head_out && gridDim.x > 1) ptx::cluster_sync_all();  // every CTA has read the head
  if (rank == 0 && tid == 0 && p.free_blocks != nullptr)
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
  // (every CTA reads all lengths, at any time)
  const auto share = [B](const int32_t* out, int64_t n, const int32_t* in) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(out), b = reinterpret_cast<uintptr_t>(in);
    return a < b + 4 * static_cast<uintptr_t>(B) && b < a + 4 * static_cast<uintptr_t>(n);
  };
  if (share(seq_lens, B, ctx_lens) || share(seq_lens, B, new_lens) ||
      share(query_start_loc, int64_t(B) + 1, ctx_lens) || share(query_start_loc, int64_t(B) + 1, new_lens))
    return fail(DSA_ERR_INVALID_ARG, "dsa_build_batch: seq_lens and query_start_loc must not share the inputs' memory");
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
  p.vec = aligned16(token_req) && aligned16(positions) && aligned16(slot_map);
  const bool in_place = free_blocks && free_head == free_head_out;
  const int64_t fill = (int64_t(max_tokens) + kThreads * 4 - 1) / (kThreads * 4);
  const int64_t ctas = std::min<int64_t>(fill, in_place ? kCluster : num_sms());
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(std::max<int64_t>(ctas, 1)));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cfg.gridDim.x;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = in_place ? 1 : 0;
  cudaError_t e = cudaLaunchKernelEx(&cfg, build_batch_kernel, p);
  if (e != cudaSuccess) return fail(DSA_ERR_CUDA, "build_batch_kernel launch failed: %s", cudaGetErrorString(e));
  return check_launch("build_batch_kernel");
}
