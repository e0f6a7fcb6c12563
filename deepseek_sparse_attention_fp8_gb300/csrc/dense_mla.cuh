// Shared by the dense MLA attention kernels: a batch as work (row tiles and
// steps of 128 keys, cut into runs), its block table, and the loads of keys.
//
// Rows: the (token, head) rows of a request, whole tokens at a time, form row
// tiles of at most 16, 32, 128 or 256 rows (by kernel); all rows of a request
// see the same latent rows. The steps of all row tiles form one sequence, cut
// into equal runs, one per group of CTAs (one persistent wave). A row tile cut
// by a run's end leaves fp32 partials, at most two per run.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>

#include "common.cuh"
#include "dense_steps.h"
#include "ptx.cuh"

namespace dsa {
namespace dense {

using namespace ptx;

constexpr int kDk = 576, kDv = 512, kF8Row = 656;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kSlot = 16384;  // 64 keys x 128 dims
constexpr float kRescaleThreshold = 8.f;  // log2 units
constexpr long long kWaitLimitCycles = 2000000000ll;
constexpr int kAhead = 3;   // steps that the fp8 cache's rows are asked into L2 ahead

struct DenseParams {
  int32_t num_blocks, rows_per_block, total_rows;
  const int32_t* block_table;
  int32_t bt_stride;
  const int32_t *seq_lens, *qsl;
  int32_t B, T, H, tpt[3];   // tokens per row tile of a pair, of a quad, of a single CTA
  int32_t pairs, quads;      // pairs and quads of CTAs launched; quads = 0: pairs only
  int32_t singles, single_rows;  // single CTAs launched (the kernel of few rows), rows of their row tiles
  int32_t block_size, bs64;  // bs64 = block_size / 64
  float scale_log2;
  const uint8_t* kv;  // the fp8 cache
  int32_t cut;    // row tiles may be cut
  int32_t out32;  // out is 32-byte aligned
  uint16_t* out;
  float* lse;
  // Partials, two per run: slot 2 n is the row tile that run n goes on with
  // from the run before, 2 n + 1 the one it leaves to the next
  float4* o_part;   // [slot][row halves][groups of 4 TMEM columns][128 lanes]
  float2* ml_part;  // [slot][rows of a row tile]: max (log2 units), sum
  int4* desc;       // per run: the cut row tile that starts in it (first row, rows, further parts, kind)
  int32_t* dev_status;
};

// The run of a group of CTAs: its first request, row tile and step, and its
// steps [pos, end) of all; per: steps of every run. At the end of shared memory.
enum Kind { kPair = 0, kQuad = 1, kSingle = 2 };
struct Run {
  int32_t b, tile, k0, index;
  int64_t pos, end, per;
  int32_t kind;  // what works on the batch
};
constexpr int kSmTotal = 232448, kSmRun = kSmTotal - 64;
static_assert(sizeof(Run) <= 64, "run block too large");

// The tiles need 1024-byte alignment (without static arrays the dynamic part of
// shared memory starts there). Without it the call does nothing, and there is
// nothing to join.
__device__ __forceinline__ bool misaligned(const DenseParams& p, const uint8_t* smem) {
  if ((smem_u32(smem) & 1023u) == 0) return false;
  if (threadIdx.x == 0) {
    report(p.dev_status, DSA_DEVERR_TIMEOUT);
    if (p.cut && blockIdx.x < max(p.pairs, p.singles)) p.desc[blockIdx.x] = make_int4(0, 0, 0, 0);
  }
  return true;
}

// The request b of the batch, as work.
__device__ __forceinline__ Request load_request(const DenseParams& p, int tpt, int b) {
  const int q0 = min(max(__ldg(p.qsl + b), 0), p.T), q1 = min(max(__ldg(p.qsl + b + 1), 0), p.T);
  const int64_t sl = __ldg(p.seq_lens + b), cap = static_cast<int64_t>(p.bt_stride) * p.block_size;
  return make_request(q0, q1, sl, cap, tpt);
}

// A run of steps, segment by segment (a segment: the steps of one row tile).
template <Kind KIND>
struct Cursor {
  Request req;
  int32_t b, tile, nk, k0, k1;
  int32_t left;  // steps of the run from this segment on
  __device__ __forceinline__ void cut(const DenseParams& p) {
    nk = steps_of(req, p.tpt[KIND], tile);
    k1 = p.cut ? min(nk, k0 + left) : nk;
  }
  __device__ __forceinline__ bool start(const DenseParams& p, const Run* s) {
    b = s->b;
    tile = s->tile;
    k0 = k1 = nk = s->k0;
    left = static_cast<int32_t>(s->end - s->pos);
    if (left <= 0) return false;
    req = load_request(p, p.tpt[KIND], b);
    cut(p);
    return true;
  }
  __device__ __forceinline__ bool next(const DenseParams& p) {
    left -= k1 - k0;
    if (left <= 0) return false;
    k0 = 0;
    if (++tile >= req.n_tiles) {
      tile = 0;
      do {
        if (++b >= p.B) return false;
        req = load_request(p, p.tpt[KIND], b);
      } while (req.n_tiles == 0);
    }
    cut(p);
    return true;
  }
};

// The cache rows of a unit of 64 keys: their first row (total_rows, which
// reads as zeros, where there is none) and how many of them exist.
struct Rows {
  int32_t row, n;
};
// A warp's view of a row tile's part of the block table: lane l holds the
// entry of unit base + l, and the entries of the 32 units behind are in flight,
// so that no step waits for the table. Called by whole warps.
struct Units {
  int32_t base, row, ahead;
  template <class C>
  __device__ __forceinline__ int32_t entry(const DenseParams& p, const C& c, int unit) const {
    const int64_t key = static_cast<int64_t>(unit) * 64;
    return key < c.req.kv_len ? __ldg(p.block_table + static_cast<int64_t>(c.b) * p.bt_stride + unit / p.bs64) : 0;
  }
  template <class C>
  __device__ __forceinline__ int32_t first_row(const DenseParams& p, const C& c, int32_t blk, int unit, bool rep) const {
    if (blk < 0 || blk >= p.num_blocks) {
      if (rep && static_cast<int64_t>(unit) * 64 < c.req.kv_len) report(p.dev_status, DSA_DEVERR_BLOCK_OOB);
      return -1;
    }
    return blk * p.rows_per_block + (unit % p.bs64) * 64;
  }
  template <class C>
  __device__ __forceinline__ void start(const DenseParams& p, const C& c, int lane, bool rep) {
    base = 2 * c.k0;
    row = entry(p, c, base + lane);
    ahead = entry(p, c, base + 32 + lane);
    row = first_row(p, c, row, base + lane, rep);
  }
  // units are asked for in ascending order, at most 32 behind the last
  template <class C>
  __device__ __forceinline__ Rows get(const DenseParams& p, const C& c, int unit, int lane, bool rep) {
    if (unit >= base + 32) {
      base += 32;
      row = first_row(p, c, ahead, base + lane, rep);
      ahead = entry(p, c, base + 32 + lane);
    }
    const int left = c.req.kv_len - unit * 64;
    const int32_t first = __shfl_sync(0xFFFFFFFFu, row, (unit - base) & 31);
    if (left <= 0 || first < 0) return {p.total_rows, 0};
    return {first, min(left, 64)};
  }
  // one of a step's two units
  template <class C>
  __device__ __forceinline__ Rows of(const DenseParams& p, const C& c, int kt, int which) const {
    const int left = c.req.kv_len - kt * kTile - 64 * which;
    const int32_t first = __shfl_sync(0xFFFFFFFFu, row, (2 * kt - base + which) & 31);
    return {first < 0 ? p.total_rows : first, first < 0 ? 0 : min(left, 64)};  // (no rows with n < 0 either)
  }
  // makes the units of step kt those that `of` finds; steps in ascending order
  template <class C>
  __device__ __forceinline__ void advance(const DenseParams& p, const C& c, int kt, int lane, bool rep) {
    if (2 * kt >= base + 32) {
      base += 32;
      row = first_row(p, c, ahead, base + lane, rep);
      ahead = entry(p, c, base + 32 + lane);
    }
  }
};

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
// mbar_wait with one answer for the warp
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) {
  return __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity));
}

// Loads 64 keys x 64 * blocks dims (dim block d0 on) by the whole warp. The
// rows behind a request's last key are not its own and may hold anything,
// NaN included, so they are gathered from past the cache's end, as zeros.
__device__ __forceinline__ void load_keys(uint32_t dst, const CUtensorMap* box, const CUtensorMap* row_map,
                                          uint32_t bar, Rows x, int32_t total_rows, int d0, int blocks, int lane) {
  if (x.n == 0 || x.n == 64) {
    if (lane == 0) tma_load_3d_pair(dst, box, bar, 0, x.row, d0);
  } else {
    const int g = lane & 15, d = lane >> 4;
    if (d < blocks) {
      int r[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) r[i] = 4 * g + i < x.n ? x.row + 4 * g + i : total_rows;
      tma_gather4_pair(dst + d * 8192 + g * 512, row_map, bar, (d0 + d) * 64, r[0], r[1], r[2], r[3]);
    }
  }
  __syncwarp();
}

// ---- fp8 cache: a key's 128 codes of a group are 8 lanes' 16, decoded (code *
// scale in fp32, rounded to bf16: the tensor cores take bf16) and stored as the
// swizzled tile that the copies of the bf16 cache would bring.
__device__ __forceinline__ float2 mul2(float2 a, float s) {  // two products in one instruction
  float2 r;
  asm("{\n\t.reg .b64 a, b, c;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %4};\n\tmul.rn.f32x2 c, a, b;\n\t"
      "mov.b64 {%0, %1}, c;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(s));
  return r;
}
__device__ __forceinline__ uint32_t decode2(uint32_t two, float sc) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(two)));
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
  const float2 v = mul2(f, sc);
  return pack_bf16(v.x, v.y);
}
__device__ __forceinline__ uint4 decode8(uint2 c, float sc) {
  return make_uint4(decode2(c.x, sc), decode2(c.x >> 16, sc), decode2(c.y, sc), decode2(c.y >> 16, sc));
}

// A decoding warp's part, 8 keys from key0 on, of slots of 64 keys x 128 dims.
// A slot's codes land where its dims 64-127 belong, each key's in its own row:
// the warp that has read its keys' codes may write their values in place.
struct Decoder {
  int key0;
  uint32_t at0, at1, from;
  __device__ __forceinline__ Decoder(int w, int lane) {
    const int lane8 = lane & 7, key = 8 * w + (lane >> 3);  // and key + 4
    // the order of a lane's two 16-byte chunks, and of the codes behind them,
    // that leaves no bank conflicts
    const uint32_t swap = ((lane8 >> 2) ^ (lane >> 3)) & 1;
    const uint32_t blk = (lane8 >> 2) * 8192, c0 = 2 * (lane8 & 3);
    key0 = 8 * w;
    at0 = blk + sw128_offset(key, c0 + swap);
    at1 = blk + sw128_offset(key, c0 + (swap ^ 1));
    from = 8192 + key * 128 + 16 * lane8 + 8 * swap;  // and the other 8 codes: ^ 8
  }
  // the scale of this warp's key lane >> 2
  __device__ __forceinline__ float scale(const DenseParams& p, Rows x, int group, int lane) const {
    float v = 0.f;
    const int k = key0 + (lane >> 2);
    if (k < x.n)  // volatile: issued here, a step ahead
      asm volatile("ld.global.nc.f32 %0, [%1];"
                   : "=f"(v)
                   : "l"(p.kv + static_cast<int64_t>(x.row + k) * kF8Row + kDv + 4 * group));
    return v;
  }
  // this lane's codes in a slot: [key][chunk]
  __device__ __forceinline__ void read(const uint8_t* slot, uint2 (&code)[2][2]) const {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      code[i][0] = *reinterpret_cast<const uint2*>(slot + 512 * i + from);
      code[i][1] = *reinterpret_cast<const uint2*>(slot + 512 * i + (from ^ 8));
    }
  }
  // Two slots' values, behind their codes' read; scales: key k's in lanes 4 k +
  // sc0 and 4 k + sc0 + 1. Keys from n on (counted from this lane's first) do
  // not exist; behind them may lie anything.
  __device__ __forceinline__ void write(uint8_t* slot0, uint8_t* slot1, uint2 (&code)[2][2][2], float scales, int sc0,
                                        int n, int lane) const {
    __syncwarp();
    if (__any_sync(0xFFFFFFFFu, n < 5)) {
#pragma unroll
      for (int g = 0; g < 2; ++g) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
          if (4 * i >= n) code[g][i][0] = code[g][i][1] = make_uint2(0u, 0u);
      }
    }
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      uint8_t* dst = g ? slot1 : slot0;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float sc = __shfl_sync(0xFFFFFFFFu, scales, 4 * ((lane >> 3) + 4 * i) + sc0 + g);
        *reinterpret_cast<uint4*>(dst + (i ? (at0 + 512) ^ 64 : at0)) = decode8(code[g][i][0], sc);
        *reinterpret_cast<uint4*>(dst + (i ? (at1 + 512) ^ 64 : at1)) = decode8(code[g][i][1], sc);
      }
    }
    fence_proxy_async_smem();
    __syncwarp();
  }
};

// The run of this pair, quad or single CTA: every CTA sums the requests' steps.
// `scratch` is shared memory that nothing else uses yet.
//
// kQuad: in clusters of four CTAs the lengths, which only the device knows,
// decide here whether each cluster works as a quad or as two pairs. A row tile
// costs a pair about 7100 + 4400 clocks a step (128 rows, 2 SMs), a quad 12300
// + 2700 (256 rows, 4 SMs) and ~12000 more to begin with: fitted to 16 prompts
// of 256 tokens (128 heads: 380 us on pairs, 477 on quads) and to 1024 tokens
// over a context of 16384 (3580 and 2600 us, single launches). Between: 64 x 2 tokens over 4096
// keys 156 and 125, 8 x 16 over 2048 84 and 83, 32 x 2 over 2048 56 and 61.
// Pairs in clusters of four (144 of 152 SMs, and this choice) take 5-9% longer
// than launched as pairs.
template <int kThreads, Kind KIND>
__device__ __forceinline__ void plan_run(const DenseParams& p, Run* s, uint8_t* scratch) {
  int64_t* sums = reinterpret_cast<int64_t*>(scratch);  // [4][warps]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int kWarps = kThreads / 32;
  const bool once = p.B <= kThreads;
  int64_t total = 0;
  bool quad = false;
  if constexpr (KIND == kQuad) {
    int64_t tiles[2] = {0, 0}, steps[2] = {0, 0};
    for (int b = tid; b < p.B; b += kThreads) {
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const Request r = load_request(p, p.tpt[q], b);
        tiles[q] += r.n_tiles;
        steps[q] += steps_before(r, p.tpt[q], r.n_tiles, r.n_tiles);
      }
    }
    int64_t cost[2] = {71 * tiles[0] + 44 * steps[0], 123 * tiles[1] + 27 * steps[1]};
#pragma unroll
    for (int q = 0; q < 2; ++q) {
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) cost[q] += __shfl_xor_sync(0xFFFFFFFFu, cost[q], off);
      if (lane == 0) sums[q * kWarps + warp] = cost[q];
    }
    __syncthreads();
    cost[0] = cost[1] = 0;
    for (int i = 0; i < kWarps; ++i) {
      cost[0] += sums[i];
      cost[1] += sums[kWarps + i];
    }
    quad = cost[1] * p.pairs + int64_t(120) * p.pairs * p.quads < cost[0] * p.quads;
    __syncthreads();
  }
  const Kind kind = KIND == kSingle ? kSingle : quad ? kQuad : kPair;
  const int tpt = p.tpt[kind], index = blockIdx.x >> (kind == kSingle ? 0 : kind == kQuad ? 2 : 1);
  const int n_runs = kind == kSingle ? p.singles : kind == kQuad ? p.quads : p.pairs;
  int64_t w = 0, incl = 0;
  Request r = {};
  const auto scan = [&](int b, bool first) {  // steps of request b, and their inclusive sum over the block's requests
    w = 0;
    if (b < p.B) {
      r = load_request(p, tpt, b);
      if (first && r.uneven && r.q_len > 0 && index == 0) report(p.dev_status, DSA_DEVERR_SEQ_LEN);
      w = steps_before(r, tpt, r.n_tiles, r.n_tiles);
    }
    incl = w;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int64_t u = __shfl_up_sync(0xFFFFFFFFu, incl, off);
      if (lane >= off) incl += u;
    }
    __syncthreads();
    if (lane == 31) sums[warp] = incl;
    __syncthreads();
    int64_t all = 0;
    for (int i = 0; i < kWarps; ++i) {
      if (i < warp) incl += sums[i];
      all += sums[i];
    }
    return all;
  };
  for (int b0 = 0; b0 < p.B; b0 += kThreads) total += scan(b0 + tid, true);
  int64_t per = (total + n_runs - 1) / n_runs;
  // Runs of at least two steps (a request of 1000 keys, 128 heads: 27.8 us
  // with the caches cold, 31.9 at four, 27.8 at one; 32 of 512 keys: 30.9
  // at one, 29.9 at two), of one in the kernel of few rows (16 requests of 512
  // keys: 20.6 us, 23.7 at two, 31 at four).
  if (p.cut) per = max(per, int64_t(KIND == kSingle ? 1 : 2));
  const int64_t u0 = per * index, u1 = min(u0 + per, total);
  if (tid == 0) {
    s->index = index;
    s->kind = kind;
    s->per = per;
    s->pos = s->end = 0;
  }
  __syncthreads();
  if (u0 < u1) {
    int64_t base = 0;
    for (int b0 = 0; b0 < p.B; b0 += kThreads) {
      const int64_t all = once ? total : scan(b0 + tid, false);
      const int64_t from = base + incl - w;
      if (w > 0 && from <= u0 && u0 < from + w) {
        const int64_t u = u0 - from;
        int lo = 0, hi = r.n_tiles - 1;  // the last row tile that starts at or before u
        while (lo < hi) {
          const int mid = (lo + hi + 1) >> 1;
          if (steps_before(r, tpt, r.n_tiles, mid) <= u) lo = mid; else hi = mid - 1;
        }
        const int64_t at = steps_before(r, tpt, r.n_tiles, lo);
        s->b = b0 + tid;
        s->tile = lo;
        s->k0 = static_cast<int32_t>(u - at);
        s->pos = u0;
        s->end = u1;
        if (!p.cut && u > at) {  // the row tile belongs to the run it starts in: begin with the next
          s->k0 = 0;
          s->pos = from + steps_before(r, tpt, r.n_tiles, lo + 1);
          if (lo + 1 < r.n_tiles) {
            s->tile = lo + 1;
          } else if (s->pos < u1) {
            int b = b0 + tid;
            do ++b; while (load_request(p, tpt, b).n_tiles == 0);
            s->b = b;
            s->tile = 0;
          }
        }
      }
      base += all;
    }
  }
  fence_proxy_async_smem();  // the copies that follow write where the scratch was
  __syncthreads();
}

// Tensor maps of a call: q in boxes of q_rows x 64 x q_blocks dims; the cache
// as 9 blocks of 64 dims a row, block-major boxes (keys: 64 keys x 128 dims;
// rope: 64 keys x 64; row: one row x 64, for gathers). fp8: the cache's maps
// cover the rope dims only (128 bytes from byte 528 of a row).
struct Maps {
  CUtensorMap q, keys, rope, row;
};
// fp8: 64 rows' codes of a group, and their 16 bytes of scales.
struct CodeMaps {
  CUtensorMap codes, scales;
};
inline dsa_status_t make_maps(Maps* m, const DenseParams& p, bool f8, const void* q, const void* kv, uint32_t q_rows,
                              uint32_t q_blocks) {
  const void* base = f8 ? static_cast<const uint8_t*>(kv) + kDv + 16 : kv;
  const uint64_t rows = static_cast<uint64_t>(p.total_rows), blocks = f8 ? 1 : 9;
  const uint64_t q_strides[2] = {kDk * 2, 128}, strides[2] = {f8 ? uint64_t(kF8Row) : uint64_t(kDk * 2), 128};
  const uint64_t q_dims[3] = {64, static_cast<uint64_t>(p.T) * p.H, 9}, dims[3] = {64, rows, blocks};
  const uint64_t row_dims[2] = {64 * blocks, rows};
  const uint32_t q_box[3] = {64, q_rows, q_blocks}, keys_box[3] = {64, 64, f8 ? 1u : 2u}, rope_box[3] = {64, 64, 1};
  const uint32_t row_box[2] = {64, 1};
  const CUtensorMapDataType bf16 = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const CUtensorMapSwizzle sw = CU_TENSOR_MAP_SWIZZLE_128B;
  dsa_status_t st;
  if ((st = make_tmap(&m->q, bf16, 3, q, q_dims, q_strides, q_box, sw)) != DSA_OK) return st;
  if ((st = make_tmap(&m->keys, bf16, 3, base, dims, strides, keys_box, sw)) != DSA_OK) return st;
  if ((st = make_tmap(&m->rope, bf16, 3, base, dims, strides, rope_box, sw)) != DSA_OK) return st;
  return make_tmap(&m->row, bf16, 2, base, row_dims, strides, row_box, sw);
}

inline dsa_status_t make_code_maps(CodeMaps* m, const DenseParams& p, const void* kv) {
  const uint64_t dims[2] = {kF8Row, static_cast<uint64_t>(p.total_rows)}, strides[1] = {kF8Row};
  const uint32_t codes[2] = {128, 64}, scales[2] = {16, 64};
  const CUtensorMapDataType u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
  const dsa_status_t st = make_tmap(&m->codes, u8, 2, kv, dims, strides, codes, CU_TENSOR_MAP_SWIZZLE_NONE);
  return st != DSA_OK ? st : make_tmap(&m->scales, u8, 2, kv, dims, strides, scales, CU_TENSOR_MAP_SWIZZLE_NONE);
}

// Number of 4-CTA clusters the current device runs at once, 0 when it cannot.
int num_quads(bool f8);
// Enqueues the kernel of clusters of four CTAs, p.quads of them, which work as
// quads or as 2 p.quads = p.pairs pairs.
dsa_status_t launch_quads(const DenseParams& p, bool f8, const void* q, const void* kv, cudaStream_t s);
// Rows of a row tile in the kernel of few rows, 0 where that kernel does not
// serve; enqueues it on p.singles CTAs.
int single_rows(int32_t B, int32_t T, int32_t H, bool f8);
dsa_status_t launch_singles(const DenseParams& p, bool f8, const void* q, const void* kv, cudaStream_t s);

}  // namespace dense
}  // namespace dsa
