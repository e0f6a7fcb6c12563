// Dense MLA attention for few rows (single tokens of one rank's share of the
// heads): row tiles of N = 16 or 32 rows, one CTA each, with keys and value
// dims along M, where the MMAs need 128, and the rows along N:
//   S^T = K Q^T     M = 128 keys, N rows, K = 576 dims;
//   softmax         thread = key: the rows' maxima across the 128 lanes;
//   O^T += V^T P^T  M = 128 dims (four times), N rows, K = 128 keys.
// A step moves 144 KB of keys into the SM, once for both products: at an SM's
// share of the memory bandwidth 6300 clocks (at the ~32 bytes a clock that an SM
// takes in from L2, 4600), and it issues 68 small MMAs. Memory bounds it: a step
// takes 6600-7300 clocks in the middle of a long run; the pair kernel, whose
// MMAs of 128 rows are mostly empty here, spends 4400 clocks of two SMs.
// 64 requests, 16 heads, 248000 keys in all (286 MB): 81.0 us with the launches
// from a graph and the caches cold, 99.4 on pairs; 42 us is what the bytes take.
// Of the rest ~9 us are the way to the first S (the plan, the table, the first
// 144 KB), ~2 us results, ~5 us the joining of partials.
//
// fp8 cache (16 rows): codes are copied to where half of their values belong
// and decoded in place, a slot of 128 keys x 128 dims at a time. 64 requests of
// 4096 keys, 16 heads (172 MB, 25 us): 87 us, 110 on pairs; 82 without the
// arithmetic of decoding. Decoding from loads into registers a step ahead took
// 108, 77 without those loads. 14 warps leave a thread 128 registers, and one is
// spilled (4 bytes stored, 16 loaded).
//
// Rope dims come first in a step: their slots are free again after S, so that a
// third of the next step is loaded while this one's weights are made. Results
// are written by code that fits few cache lines of instructions, and a row's
// sum and factor are one thread's: unrolled over rows in one thread the end of
// a row tile took 10000-30000 clocks, most of them waits for instructions.
#include <algorithm>

#include "dense_mla.cuh"

namespace dsa {
namespace dense {
namespace {

// warps 0-3 softmax and results, 4 loads, 5 MMA; fp8 cache: 6-13 decode
constexpr int kLoadWarp = 4, kMmaWarp = 5, kDecodeWarp = 6, kDecodeWarps = 8;
constexpr int threads(bool f8) { return 32 * (kDecodeWarp + (f8 ? kDecodeWarps : 0)); }
constexpr int kRing = 5, kPairSlot = 32768;  // slots of 128 keys x 128 dims (two blocks of 64), four per step

template <int N>
struct Layout {
  static constexpr int kRopes = N == 16 ? 2 : 1;  // buffers of 128 keys x 64 rope dims
  static constexpr int kRope = kRing * kPairSlot, kQ = kRope + kRopes * 16384;
  static constexpr int kP = kQ + 9 * N * 128;  // q as 9 blocks of N rows x 64 dims; P: 2 blocks of N rows x 64 keys
  static constexpr int kRed = kP + 2 * N * 128, kLim = kRed + 2 * 4 * N * 4,
                       kScales = kLim + 128, kBar = kScales + 4096;
  static constexpr uint32_t kColS = 0, kColO = 2 * N, kTmemCols = N == 16 ? 128 : 256;  // S 2 x N, O 4 x N
  static_assert(kBar + 256 <= kSmRun, "shared memory");
};

struct Bars {
  uint64_t full[kRing], empty[kRing], rope_full[2], rope_empty[2];
  uint64_t q_full, q_free;  // q_free: the row tile's last S has read q
  uint64_t s_full[2], p_full, pv_done[2], meet;
  uint64_t codes[kRing];  // fp8: a slot's codes landed
  uint32_t tmem;
  volatile int abort;
};
static_assert(sizeof(Bars) <= 256, "barrier block too large");

__device__ __forceinline__ float warp_max(float x) {
  float y;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}

// Loads dim blocks [d0, d0 + BLOCKS) (64 dims) of two units of 64 keys, each
// block a tile of 128 keys, by the whole warp (load_keys for a CTA of its own).
template <int BLOCKS>
__device__ __forceinline__ void load_blocks(uint32_t dst, const Maps& maps, uint64_t* bar, Rows x0, Rows x1,
                                            int32_t total_rows, int d0, int lane) {
  const bool whole0 = (x0.n & 63) == 0, whole1 = (x1.n & 63) == 0;
  if (lane < 2 * BLOCKS && ((lane & 1) ? whole1 : whole0))
    tma_load_3d(dst + lane * 8192, &maps.rope, bar, 0, (lane & 1) ? x1.row : x0.row, d0 + (lane >> 1));
  if (!whole0 || !whole1) {
    const int g = lane & 15, j = lane >> 4;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const Rows x = h ? x1 : x0;
      if ((x.n & 63) == 0 || j >= BLOCKS) continue;
      int r[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) r[i] = 4 * g + i < x.n ? x.row + 4 * g + i : total_rows;
      tma_gather4(dst + j * 16384 + h * 8192 + g * 512, &maps.row, bar, (d0 + j) * 64, r[0], r[1], r[2], r[3]);
    }
  }
  __syncwarp();
}

template <int N, bool F8>
__global__ void __launch_bounds__(threads(F8), 1) dense_mla_rows_kernel(const __grid_constant__ DenseParams p,
                                                                       const __grid_constant__ Maps maps,
                                                                       const __grid_constant__ CodeMaps code_maps) {
  using L = Layout<N>;
  extern __shared__ __align__(1024) uint8_t smem[];
  if (misaligned(p, smem)) return;
  Bars* s = reinterpret_cast<Bars*>(smem + L::kBar);
  const Run* run = reinterpret_cast<const Run*>(smem + kSmRun);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&s->full[i], F8 ? kDecodeWarps : 1);
      mbar_init(&s->empty[i], 1);
      mbar_init(&s->codes[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s->rope_full[i], 1);
      mbar_init(&s->rope_empty[i], 1);
      mbar_init(&s->s_full[i], 1);
      mbar_init(&s->pv_done[i], 1);
    }
    mbar_init(&s->q_full, 1);
    mbar_init(&s->q_free, 1);
    mbar_init(&s->p_full, 4);
    mbar_init(&s->meet, 4);
    fence_mbar_init();
    s->abort = 0;
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&s->tmem, L::kTmemCols);
    tmem_relinquish();
  }
  if (tid == kLoadWarp * 32) {
    prefetch_tmap(&maps.q);
    prefetch_tmap(&maps.rope);
    prefetch_tmap(&maps.row);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s->tmem;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  plan_run<threads(F8), kSingle>(p, reinterpret_cast<Run*>(smem + kSmRun), smem);

  const auto abort_now = [&] {
    s->abort = 1;
    report(p.dev_status, DSA_DEVERR_TIMEOUT);
  };
  Cursor<kSingle> c;
  bool ok = true;

  if (warp == kLoadWarp) {
    // ---------------- q of each row tile, and the keys: per step the rope dims,
    // then four slots of 128 dims (fp8: their codes)
    int slot = 0, it = 0, seg = 0;
    uint32_t turn = 0;
    for (bool more = c.start(p, run); more && ok; more = c.next(p), ++seg) {
      if (seg > 0) ok = warp_wait(&s->q_free, (seg - 1) & 1);
      if (!ok) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(&s->q_full, 9 * N * 128);
        tma_load_3d(smem_u32(smem + L::kQ), &maps.q, &s->q_full, 0, (c.req.q0 + c.tile * p.tpt[kSingle]) * p.H, 0);
      }
      __syncwarp();
      Units u;
      u.start(p, c, lane, true);
      for (int kt = c.k0; kt < c.k1 && ok; ++kt, ++it) {
        const Rows x0 = u.get(p, c, 2 * kt, lane, true), x1 = u.get(p, c, 2 * kt + 1, lane, true);
        const int rb = it % L::kRopes, rt = it / L::kRopes;
        ok = rt == 0 || warp_wait(&s->rope_empty[rb], (rt - 1) & 1);
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(&s->rope_full[rb], 16384);
        __syncwarp();
        load_blocks<1>(smem_u32(smem + L::kRope + rb * 16384), maps, &s->rope_full[rb], x0, x1, p.total_rows, F8 ? 0 : 8,
                       lane);
        for (int k = 0; k < 4; ++k) {
          if (turn > 0 && !warp_wait(&s->empty[slot], (turn - 1) & 1)) {
            ok = false;
            break;
          }
          if constexpr (F8) {
            // the codes to where their own keys' dims 64-127 will be
            if (lane == 0) mbar_arrive_expect_tx(&s->codes[slot], 16384 + (k == 0 ? 2048 : 0));
            __syncwarp();
            const int row = (lane & 1) ? x1.row : x0.row;
            if (lane < 2)
              tma_load_2d(smem_u32(smem + slot * kPairSlot + 16384 + lane * 8192), &code_maps.codes, &s->codes[slot],
                          128 * k, row);
            else if (k == 0 && lane < 4)
              tma_load_2d(smem_u32(smem + L::kScales + (it & 1) * 2048 + (lane & 1) * 1024), &code_maps.scales,
                          &s->codes[slot], kDv, row);
            __syncwarp();
            if (++slot == kRing) {
              slot = 0;
              ++turn;
            }
            continue;
          }
          if (lane == 0) mbar_arrive_expect_tx(&s->full[slot], kPairSlot);
          __syncwarp();
          load_blocks<2>(smem_u32(smem + slot * kPairSlot), maps, &s->full[slot], x0, x1, p.total_rows, 2 * k, lane);
          if (++slot == kRing) {
            slot = 0;
            ++turn;
          }
        }
      }
    }
    if (!ok && lane == 0) abort_now();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  } else if (F8 && warp >= kDecodeWarp) {
    // ---------------- fp8: a step's four slots, 16 keys per warp. A slot's codes
    // land where its dims 64-127 belong, each key's in its own row: the warp that
    // has read its keys' codes may write their values in place
    const int w = warp - kDecodeWarp, lane8 = lane & 7, key = w * 16 + (lane >> 3);  // and key + 4, 8, 12
    // the order of a lane's two 16-byte chunks, and of the codes behind them,
    // that leaves no bank conflicts
    const uint32_t swap = ((lane8 >> 2) ^ (lane >> 3)) & 1;
    const uint32_t blk = (lane8 >> 2) * 16384, c0 = 2 * (lane8 & 3);
    const uint32_t at0 = blk + sw128_offset(key, c0 + swap), at1 = blk + sw128_offset(key, c0 + (swap ^ 1));
    const uint32_t from = 16384 + key * 128 + 16 * lane8 + 8 * swap;  // and the other 8 codes: ^ 8
    int slot = 0, it = 0;
    uint32_t turn = 0;
    for (bool more = c.start(p, run); more && ok; more = c.next(p)) {
      for (int kt = c.k0; kt < c.k1 && ok; ++kt, ++it) {
        // keys of this warp that exist: behind them may lie anything
        const int n = c.req.kv_len - kt * kTile - w * 16 - (lane >> 3);
        const uint8_t* scales = smem + L::kScales + (it & 1) * 2048 + key * 16;
#pragma unroll 1
        for (int g = 0; g < 4; ++g) {
          ok = warp_wait(&s->codes[slot], turn & 1);
          if (!ok) break;
          uint8_t* dst = smem + slot * kPairSlot;
          uint2 code[4][2];
          float sc[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            code[i][0] = *reinterpret_cast<const uint2*>(dst + 512 * i + from);
            code[i][1] = *reinterpret_cast<const uint2*>(dst + 512 * i + (from ^ 8));
            sc[i] = *reinterpret_cast<const float*>(scales + 64 * i + 4 * g);
          }
          __syncwarp();
          if (__any_sync(0xFFFFFFFFu, n < 13)) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if (4 * i < n) continue;
              code[i][0] = code[i][1] = make_uint2(0u, 0u);
              sc[i] = 0.f;
            }
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t up = (i >> 1) * 1024;
            *reinterpret_cast<uint4*>(dst + up + ((i & 1) ? (at0 + 512) ^ 64 : at0)) = decode8(code[i][0], sc[i]);
            *reinterpret_cast<uint4*>(dst + up + ((i & 1) ? (at1 + 512) ^ 64 : at1)) = decode8(code[i][1], sc[i]);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&s->full[slot]);
          if (++slot == kRing) {
            slot = 0;
            ++turn;
          }
        }
      }
    }
    if (!ok && lane == 0) abort_now();
  } else if (warp == kMmaWarp) {
    // ---------------- MMA: whatever is ready, PV of the oldest step first. The
    // warp stays converged, so that the descriptors live in uniform registers;
    // one lane issues
    const uint32_t idesc_qk = idesc_bf16(128, N, false, false), idesc_pv = idesc_bf16(128, N, true, false);
    // K-major tiles (keys, q, P): 8-row groups 1024 bytes apart; values (dims
    // along M): 64-dim blocks 16384 bytes apart, 8 keys 1024
    const uint64_t dk = smem_desc(smem_u32(smem), 16, 1024, kSwizzle128B);
    const uint64_t dv = smem_desc(smem_u32(smem), 16384, 1024, kSwizzle128B);
    const auto all = [](bool x) { return __all_sync(0xFFFFFFFFu, x) != 0; };
    bool more = c.start(p, run);
    int iq = 0, ip = 0, sub = 0, segs = 0;  // the next S and its part, the next PV
    int kt = c.k0, sq = 0, sp = 0;          // their slots
    uint32_t tq = 0, first = 0;             // S's turn of the ring; bit i & 1: step i begins a row tile
    long long idle_since = clock64();
    while ((more || ip < iq) && !__any_sync(0xFFFFFFFFu, s->abort)) {
      bool progressed = false;
      if (ip < iq && all(mbar_test_wait(&s->p_full, ip & 1))) {
        tc_fence_after();
        const int buf = ip & 1;
        const uint32_t acc0 = ~(first >> buf) & 1u;
#pragma unroll 1
        for (int mb = 0; mb < 4; ++mb) {
          const uint64_t a0 = dv + static_cast<uint64_t>((sp * kPairSlot) >> 4), b0 = dk + static_cast<uint64_t>(L::kP >> 4);
          if (elect_one()) {
#pragma unroll
            for (int ks = 0; ks < 8; ++ks)  // 16 keys each
              mma_bf16_ss(tmem + L::kColO + mb * N, a0 + ((ks * 2048) >> 4),
                          b0 + (((ks >> 2) * N * 128 + (ks & 3) * 32) >> 4), idesc_pv, ks > 0 ? 1u : acc0);
            mma_commit(&s->empty[sp]);
            if (mb == 3) mma_commit(&s->pv_done[buf]);
          }
          __syncwarp();
          if (++sp == kRing) sp = 0;
        }
        ++ip;
        progressed = true;
      }
      if (more && iq < ip + 2) {  // PV of step iq - 2 has been issued: S was read
        const int buf = iq & 1, rb = iq % L::kRopes;
        bool ready = sub > 0 ? mbar_test_wait(&s->full[sq], tq & 1)
                             : mbar_test_wait(&s->rope_full[rb], (iq / L::kRopes) & 1);
        if (sub == 0 && kt == c.k0) ready = ready && mbar_test_wait(&s->q_full, segs & 1);
        if (all(ready)) {
          tc_fence_after();
          const uint32_t d = tmem + L::kColS + N * buf;
          if (sub == 0) {
            const uint64_t a0 = dk + static_cast<uint64_t>((L::kRope + rb * 16384) >> 4);
            const uint64_t b0 = dk + static_cast<uint64_t>((L::kQ + 8 * N * 128) >> 4);
            if (elect_one()) {
#pragma unroll
              for (int st = 0; st < 4; ++st)
                mma_bf16_ss(d, a0 + ((st * 32) >> 4), b0 + ((st * 32) >> 4), idesc_qk, st > 0 ? 1u : 0u);
              mma_commit(&s->rope_empty[rb]);
            }
            ++sub;
          } else {
            const uint64_t a0 = dk + static_cast<uint64_t>((sq * kPairSlot) >> 4);
            const uint64_t b0 = dk + static_cast<uint64_t>((L::kQ + 2 * (sub - 1) * N * 128) >> 4);
            const bool last = kt + 1 == c.k1;
            if (elect_one()) {
#pragma unroll
              for (int st = 0; st < 8; ++st)
                mma_bf16_ss(d, a0 + (((st >> 2) * 16384 + (st & 3) * 32) >> 4),
                            b0 + (((st >> 2) * N * 128 + (st & 3) * 32) >> 4), idesc_qk, 1u);
              if (sub == 4) {
                mma_commit(&s->s_full[buf]);
                if (last) mma_commit(&s->q_free);
              }
            }
            if (++sq == kRing) {
              sq = 0;
              ++tq;
            }
            if (++sub > 4) {
              first = (first & ~(1u << buf)) | (kt == c.k0 ? 1u << buf : 0u);
              sub = 0;
              ++iq;
              if (++kt == c.k1) {
                ++segs;
                more = c.next(p);
                kt = c.k0;
              }
            }
          }
          __syncwarp();
          progressed = true;
        }
      }
      if (progressed) idle_since = clock64();
      else if (all(clock64() - idle_since > kWaitLimitCycles) && lane == 0) abort_now();
    }
  } else if (warp < kLoadWarp) {
    // ---------------- softmax: TMEM lane = key (then, of O^T, dim), columns = rows
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(warp * 32) << 16);
    float* red = reinterpret_cast<float*>(smem + L::kRed);  // [step parity][warp][row]
    int* lims = reinterpret_cast<int*>(smem + L::kLim);
    uint8_t* p_dst = smem + L::kP + (tid >> 6) * N * 128;
    const uint32_t p_chunk = (tid & 63) >> 3, p_at = (tid & 7) * 2;
    int it = 0;
    uint32_t meets = 0;
    const auto meet = [&] {  // what each of the four warps wrote is seen by all
      __syncwarp();
      if (lane == 0) mbar_arrive(&s->meet);
      return warp_wait(&s->meet, meets++ & 1);
    };
    for (bool more = c.start(p, run); more && ok; more = c.next(p)) {
      const int row0 = (c.req.q0 + c.tile * p.tpt[kSingle]) * p.H;
      const int rows = (min(c.req.q_len, (c.tile + 1) * p.tpt[kSingle]) - c.tile * p.tpt[kSingle]) * p.H;
      if (tid < N) lims[tid] = tid < rows ? visible(c.req, c.tile * p.tpt[kSingle] + tid / p.H) : 0;
      const int lim0 = visible(c.req, c.tile * p.tpt[kSingle]);  // the fewest keys that a row sees
      float m[N], l[N];
#pragma unroll
      for (int i = 0; i < N; ++i) {
        m[i] = kNegSentinel;
        l[i] = 0.f;
      }
      ok = meet();
      Units u;
      u.start(p, c, lane, false);
      for (int kt = c.k0; kt < c.k1 && ok; ++kt, ++it) {
        const int buf = it & 1, key = kt * kTile + tid;
        const Rows x = u.get(p, c, 2 * kt + (warp >> 1), lane, false);
        ok = warp_wait(&s->s_full[buf], (it >> 1) & 1);
        if (!ok) break;
        tc_fence_after();
        float sc[N];
#pragma unroll
        for (int h = 0; h < N / 16; ++h) {
          uint32_t v[16];
          tmem_ld16_sync(lane_base + L::kColS + N * buf + 16 * h, v);
#pragma unroll
          for (int i = 0; i < 16; ++i) sc[16 * h + i] = __uint_as_float(v[i]);
        }
        tc_fence_before();
        if (x.n == 0 || (kt + 1) * kTile > lim0) {  // (rows that do not exist are not looked at)
#pragma unroll
          for (int i = 0; i < N; ++i) sc[i] = x.n > 0 && key < lims[i] ? sc[i] : -INFINITY;
        }
        float mine = -INFINITY;  // lane i: the maximum of row i over this warp's keys
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const float y = warp_max(sc[i]);
          if (lane == i) mine = y;
        }
        float* rd = red + buf * 4 * N;
        if (lane < N) rd[warp * N + lane] = mine;
        ok = meet();
        if (!ok) break;
        bool grown = false;
        float alpha[N];
#pragma unroll
        for (int i = 0; i < N; i += 4) {
          const float4 a = *reinterpret_cast<const float4*>(rd + i), b = *reinterpret_cast<const float4*>(rd + N + i);
          const float4 e = *reinterpret_cast<const float4*>(rd + 2 * N + i), f = *reinterpret_cast<const float4*>(rd + 3 * N + i);
          const float mt[4] = {fmaxf(fmaxf(a.x, b.x), fmaxf(e.x, f.x)), fmaxf(fmaxf(a.y, b.y), fmaxf(e.y, f.y)),
                               fmaxf(fmaxf(a.z, b.z), fmaxf(e.z, f.z)), fmaxf(fmaxf(a.w, b.w), fmaxf(e.w, f.w))};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float t = mt[j] * p.scale_log2;
            const bool g = t > m[i + j] + kRescaleThreshold;
            alpha[i + j] = 1.f;
            if (g) {
              alpha[i + j] = ex2_approx(m[i + j] - t);
              m[i + j] = t;
              grown = true;
            }
          }
        }
        uint32_t pk[N / 2];
#pragma unroll
        for (int i = 0; i < N; i += 2) {
          // the sum takes the fp32 weights; the product takes them rounded to bf16
          const float e0 = ex2_approx(fmaf(sc[i], p.scale_log2, -m[i])), e1 = ex2_approx(fmaf(sc[i + 1], p.scale_log2, -m[i + 1]));
          l[i] = l[i] * alpha[i] + e0;
          l[i + 1] = l[i + 1] * alpha[i + 1] + e1;
          pk[i / 2] = pack_bf16(e0, e1);
        }
        // P and O are free once PV of the step before is done
        if (it >= 1) ok = warp_wait(&s->pv_done[(it - 1) & 1], ((it - 1) >> 1) & 1);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int i = 0; i < N; ++i)
          *reinterpret_cast<uint16_t*>(p_dst + sw128_offset(i, p_chunk) + p_at) =
              static_cast<uint16_t>(pk[i / 2] >> (16 * (i & 1)));
        if (kt > c.k0 && grown) {  // the same in all threads
#pragma unroll 1
          for (int q = 0; q < 4 * N; q += N) {
#pragma unroll
            for (int h = 0; h < N / 16; ++h) {
              uint32_t o[16];
              tmem_ld16_sync(lane_base + L::kColO + q + 16 * h, o);
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha[16 * h + i]);
              tmem_st16(lane_base + L::kColO + q + 16 * h, o);
            }
          }
          tmem_st_wait();
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s->p_full);
      }
      if (!ok) break;
      // the row tile's (or its part's) result. The sums over the keys first: each
      // exchange halves the rows that a lane holds, until it has one
#pragma unroll
      for (int half = N / 2, off = 16; off > 0; half >>= 1, off >>= 1) {
        const bool up = (lane & off) != 0;
        if (half == 0) l[0] += __shfl_xor_sync(0xFFFFFFFFu, l[0], off);
#pragma unroll
        for (int i = 0; i < half; ++i)
          l[i] = (up ? l[i + half] : l[i]) + __shfl_xor_sync(0xFFFFFFFFu, up ? l[i] : l[i + half], off);
      }
      float* sums = red + (it & 1) * 4 * N;  // the maxima of the step before the last: read by all
      sums[warp * N + lane / (32 / N)] = l[0];
      const bool whole = c.k0 == 0 && c.k1 == c.nk;
      const int slot = 2 * run->index + (c.k0 > 0 ? 0 : 1);
      ok = meet() && warp_wait(&s->pv_done[(it - 1) & 1], ((it - 1) >> 1) & 1);
      if (!ok) break;
      tc_fence_after();
      float m_row = 0.f;  // thread = row
#pragma unroll
      for (int i = 0; i < N; ++i) m_row = tid == i ? m[i] : m_row;
      if (tid < rows) {
        const float l_row = (sums[tid] + sums[N + tid]) + (sums[2 * N + tid] + sums[3 * N + tid]);
        if (!whole) p.ml_part[slot * N + tid] = make_float2(m_row, l_row);
        else if (p.lse != nullptr) p.lse[row0 + tid] = l_row != 0.f ? (m_row + log2f(l_row)) * kLn2 : -INFINITY;
      }
      if (whole) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const float l_row = (sums[i] + sums[N + i]) + (sums[2 * N + i] + sums[3 * N + i]);
          m[i] = l_row != 0.f ? __fdividef(1.f, l_row) : 0.f;
        }
      }
      const int64_t first_row = whole ? row0 : static_cast<int64_t>(slot) * N;
      const int64_t at = first_row * kDv + tid;
#pragma unroll 1
      for (int mb = 0; mb < 4 * (N / 16); ++mb) {
        uint32_t o[16];
        const int h = mb % (N / 16) * 16;
        tmem_ld16_sync(lane_base + L::kColO + 16 * mb, o);
        const int64_t to = at + h * kDv + 128 * (mb / (N / 16));
        if (whole) {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float inv = N == 32 && h ? m[(i + 16) % N] : m[i];
            if (h + i < rows)
              p.out[to + i * kDv] = static_cast<uint16_t>(pack_bf16(__uint_as_float(o[i]) * inv, 0.f));
          }
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (h + i < rows) reinterpret_cast<float*>(p.o_part)[to + i * kDv] = __uint_as_float(o[i]);
        }
        __syncwarp();
      }
      if (tid == 0 && c.k0 == 0 && !whole) {
        // runs that hold the rest of this row tile
        const int last = static_cast<int>((run->end - c.left + c.nk - 1) / run->per);
        p.desc[run->index] = make_int4(row0, rows, last - run->index, kSingle);
      }
      ok = meet();  // the sums have been read
      tc_fence_before();
    }
    if (!ok && lane == 0) abort_now();
    if (p.cut && tid == 0) {
      // nothing to join: no row tile that starts in this run goes on behind it
      if (!ok || run->pos >= run->end || c.k0 > 0 || c.k1 == c.nk) p.desc[run->index] = make_int4(0, 0, 0, 0);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (s->abort) {
    // a wait ran out: let copies and MMAs in flight end before the memory they use is given up
    const long long t0 = clock64();
    while (clock64() - t0 < 20000000ll) __nanosleep(1000);
  }
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tmem, L::kTmemCols);
}

FuncAttrOnce g_smem[3];

template <int N, bool F8>
dsa_status_t launch(const DenseParams& p, const void* q, const void* kv, cudaStream_t s) {
  Maps maps;
  CodeMaps code_maps = {};
  dsa_status_t st = make_maps(&maps, p, F8, q, kv, N, 9);
  if (st == DSA_OK && F8) st = make_code_maps(&code_maps, p, kv);
  if (st != DSA_OK) return st;
  if ((st = allow_smem(dense_mla_rows_kernel<N, F8>, kSmTotal, g_smem[F8 ? 2 : N == 32])) != DSA_OK) return st;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.singles));
  cfg.blockDim = dim3(threads(F8));
  cfg.dynamicSmemBytes = kSmTotal;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, dense_mla_rows_kernel<N, F8>, p, maps, code_maps);
  if (e != cudaSuccess) return fail(DSA_ERR_CUDA, "dense_mla_rows_kernel launch failed: %s", cudaGetErrorString(e));
  return DSA_OK;
}

}  // namespace

// Few rows a request on average. A chunk among them still works, 16 or 32 rows
// at a time. Against pairs (us, from a graph, caches cold): 64 requests of 4096
// keys and 32 heads 90 and 95; 128 of 1000 and 8 heads 52 and 69; 8 of 8192 and
// 16 heads 40 and 48; one of 1000 keys 20 and 30; one of 64 keys 21.6 and 20.
int single_rows(int32_t B, int32_t T, int32_t H, bool f8) {
  for (int n = 16; n <= (f8 ? 16 : 32); n *= 2)
    if (H <= n && static_cast<int64_t>(T) * H <= static_cast<int64_t>(n) * B) return n;
  return 0;
}

dsa_status_t launch_singles(const DenseParams& p, bool f8, const void* q, const void* kv, cudaStream_t s) {
  if (f8) return launch<16, true>(p, q, kv, s);
  return p.single_rows == 16 ? launch<16, false>(p, q, kv, s) : launch<32, false>(p, q, kv, s);
}

}  // namespace dense
}  // namespace dsa
