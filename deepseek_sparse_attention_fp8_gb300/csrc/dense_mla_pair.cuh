// The pair kernel of dense MLA attention: row tiles of 128 rows on two CTAs.
// Rows: the (token, head) rows of a request, 128 / H whole tokens at a time,
// form row tiles of at most 128 rows; all of them see the same latent rows. A
// row tile is worked on by a CTA pair, in steps of 128 keys:
//   S = Q K^T   one cta_group::2 MMA, M = 128 (64 rows per CTA), N = 128:
//               each CTA brings the 64 q rows it owns and 64 of the keys;
//   softmax     thread = row and 32 keys; lazy rescaling of O (only when the
//               row maximum grows by more than 2^8);
//   O += P V    M = 128, N = 2 x 256: CTA r brings its rows of P and value
//               dims [256 r, 256 r + 256) of all 128 keys.
// CTA r needs all dims of its own 64 keys for S, and its own 256 dims of the
// other 64 keys for O. The MMA takes the same offsets in both CTAs, so the
// blocks of the other keys replace, after S, exactly those blocks of the own
// keys that O does not need: a step holds 64 KB per CTA, and two steps are in
// flight.
//
// What bounds it: an MMA of M = 128 on two CTAs runs at half the tensor rate
// (measured: 131 clocks at N = 256, 82 at N = 128), 36 and 16 of them a step; a
// step also moves 104 KB into each SM, 3330 clocks at the ~32 bytes a clock that
// an SM takes in (measured: 62 GB/s, from L2 or memory, multicast or not). A
// step takes 4400-4800 clocks. 32 requests of 8192 keys, 128 heads: 86 us; 8 of
// 131072: 279 us (floors: 46 and 178 by bytes). Of the 86, about 10 pass until
// the first S (the plan, the table, 208 KB from memory into every pair), 6 go
// into partials and 10 into joining them, a launch included.
// With the fp8 cache codes are copied to where half of their values belong and
// decoded in place: one more stage between a slot's being free and its MMA, and
// only two steps are in flight. 32 requests of 8192 keys: 104 us, 98 without the
// arithmetic of decoding, 2 more without asking rows into L2 ahead.
//
// Work: the steps of all row tiles form one sequence, cut into equal runs, one
// per CTA pair (one persistent wave). A row tile cut by a run's end leaves
// fp32 partials, at most two per pair, joined by dense_mla_merge_kernel.
#pragma once
#include "dense_mla.cuh"

namespace dsa {
namespace dense {
namespace pairs {

// Warps 0-7 softmax, 8 q / rope (bf16 cache: and the other keys), 9 MMA, then
// the own keys: one warp of TMA copies, or (fp8 cache) 8 decoding warps, which
// take the other keys too, and one that copies codes. Nothing may spill: beside 227 KB of shared memory
// the L1 is so small that spilled registers come back from L2.
constexpr int kAuxWarp = 8, kMmaWarp = 9, kKeyWarp = 10, kDecodeWarps = 8;
constexpr int kCodeWarp = kKeyWarp + kDecodeWarps;
constexpr int threads(bool f8) { return 32 * (kKeyWarp + (f8 ? kDecodeWarps + 1 : 1)); }
constexpr uint32_t kTmemCols = 512, kColO = 0, kColS = 256;  // O 256 columns, S 2 x 64

// Shared memory: q as 9 blocks of 64 rows x 64 dims, two steps of 4 key slots,
// the rope dims of a step's own keys, P as 2 blocks of 64 rows x 64 keys (all
// 128-byte swizzled), row maxima [2][4][64], barriers.
constexpr int kSmQ = 0, kSmKv = kSmQ + 9 * 8192, kSmRope = kSmKv + 8 * kSlot, kSmP = kSmRope + 8192,
              kSmRed = kSmP + 2 * 8192, kSmBar = kSmRed + 2 * 4 * 64 * 4;
static_assert(kSmBar + 448 <= kSmRun, "more than 227 KB of shared memory");

struct Bars {
  // the first three are the even CTA's barriers, for both CTAs
  uint64_t full[2][4];   // a slot's own keys, of both CTAs
  uint64_t other[2][2];  // a step's other keys: those of CTA r, for CTA r ^ 1
  uint64_t rope, q, p_full;  // the two TMA copies; P written by the 16 softmax warps of the pair
  uint64_t s_half[2];    // the first two slots of a step have entered S (in both CTAs)
  uint64_t s_full[2];    // S of a step complete (in both CTAs)
  uint64_t pv_half[2];   // the first 64 keys of a step have entered O (in both CTAs)
  uint64_t pv_done[2];   // O += P V of a step complete (in both CTAs)
  uint64_t rows[2];      // the four softmax warps that share 32 rows
  uint64_t codes[2][4], other_codes[2][2];  // fp8: a slot's codes landed
  uint64_t first;        // q and the rope dims of the run's first step have been asked for
  uint32_t tmem;
  volatile int abort;
};
static_assert(sizeof(Bars) <= 448, "barrier block too large");

// Barriers and tensor memory, behind a cluster barrier.
template <bool F8>
__device__ __forceinline__ void set_up(Bars* s, const Maps& maps) {
  const int tid = threadIdx.x, warp = tid >> 5;
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      for (int k = 0; k < 4; ++k) mbar_init(&s->full[i][k], F8 ? 2 * kDecodeWarps : 1);
      for (int k = 0; k < 2; ++k) mbar_init(&s->other[i][k], F8 ? kDecodeWarps : 1);
      for (int k = 0; k < 4; ++k) mbar_init(&s->codes[i][k], 1);
      for (int k = 0; k < 2; ++k) mbar_init(&s->other_codes[i][k], 1);
      mbar_init(&s->s_half[i], 1);
      mbar_init(&s->pv_half[i], 1);
      mbar_init(&s->s_full[i], 1);
      mbar_init(&s->pv_done[i], 1);
      mbar_init(&s->rows[i], 4);
    }
    mbar_init(&s->first, 1);
    mbar_init(&s->rope, 1);
    mbar_init(&s->q, 1);
    mbar_init(&s->p_full, 16);
    fence_mbar_init();
    s->abort = 0;
  }
  if (warp == kMmaWarp) {
    tmem_alloc_pair(&s->tmem, kTmemCols);
    tmem_relinquish_pair();
  }
  if (tid == kKeyWarp * 32) {
    prefetch_tmap(&maps.q);
    prefetch_tmap(&maps.keys);
    prefetch_tmap(&maps.rope);
    prefetch_tmap(&maps.row);
  }
  tc_fence_before();
  cluster_sync_all();  // the other CTA's barriers exist
  tc_fence_after();
}

// Works on this pair's run, and ends with a cluster barrier. A pair is cluster
// ranks 2 n and 2 n + 1.
template <bool F8>
__device__ __forceinline__ void run_pair(const DenseParams& p, const Maps& maps, const CodeMaps& code_maps,
                                         uint8_t* smem) {
  Bars* s = reinterpret_cast<Bars*>(smem + kSmBar);
  const Run* run = reinterpret_cast<const Run*>(smem + kSmRun);
  float* red = reinterpret_cast<float*>(smem + kSmRed);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_ctarank(), base = rank & ~1u;
  const int r = static_cast<int>(rank & 1u), pair = run->index;
  const uint16_t both = static_cast<uint16_t>(3u << base);
  const uint32_t tmem = s->tmem;
  const auto abort_now = [&] {
    s->abort = 1;
    report(p.dev_status, DSA_DEVERR_TIMEOUT);
  };
  // fp8: 64 keys' codes of a group, to where their dims 64-127 will be
  const auto load_codes = [&](uint64_t* bar, int slot, int group, int row) {
    if (lane == 0) {
      mbar_arrive_expect_tx(bar, 8192);
      tma_load_2d(smem_u32(smem + kSmKv + slot * kSlot + 8192), &code_maps.codes, bar, 128 * group, row);
    }
    __syncwarp();
  };
  // a barrier's address in the even CTA
  const auto even = [&](uint64_t* bar) { return mapa_shared(smem_u32(bar), base); };

  if (F8 && warp >= kKeyWarp && warp < kKeyWarp + kDecodeWarps) {
    // ---------------- fp8: the own keys of each step, 8 per warp, two groups
    // (slots) at a time, then the other keys of the step before
    const Decoder d(warp - kKeyWarp, lane);
    Cursor<kPair> c;
    bool more = c.start(p, run), ok = true;
    int kt = c.k0;
    Units u;
    float own_next = 0.f, other_next = 0.f;  // scales of the next step
    const auto fetch_scales = [&] {
      if (kt == c.k0) u.start(p, c, lane, false);
      else u.advance(p, c, kt, lane, false);
      own_next = d.scale(p, u.of(p, c, kt, r), lane & 3, lane);
      other_next = d.scale(p, u.of(p, c, kt, r ^ 1), 2 * r + (lane & 1), lane);
    };
    if (more) fetch_scales();
    const auto all = [](bool x) { return __all_sync(0xFFFFFFFFu, x) != 0; };
    float other_scales = 0.f;
    int other_n = 0;
    for (int it = 0; ok && (more || it > 0); ++it) {
      const int buf = it & 1, b1 = buf ^ 1;
      const bool last = !more;  // only the other keys of the last step are left
      const float own_scales = own_next, old_scales = other_scales;
      const int left = c.req.kv_len - kt * kTile - d.key0 - (lane >> 3), old_n = other_n;
      other_scales = other_next;
      other_n = left - 64 * (r ^ 1);
      if (!last) {
        if (++kt == c.k1) {
          more = c.next(p);
          kt = c.k0;
        }
        if (more) fetch_scales();
      }
      int h = last ? 2 : 0;
      bool other_left = it > 0;
      long long idle_since = clock64();
#pragma unroll 1
      while (h < 2 || other_left) {  // whichever has landed; the other keys are waited for more urgently
        if (other_left && all(mbar_test_wait(&s->other_codes[b1][0], ((it - 1) >> 1) & 1) &&
                              mbar_test_wait(&s->other_codes[b1][1], ((it - 1) >> 1) & 1))) {
          uint8_t* slot = smem + kSmKv + (b1 * 4 + 2 * (r ^ 1)) * kSlot;
          uint2 code[2][2][2];
          d.read(slot, code[0]);
          d.read(slot + kSlot, code[1]);
          d.write(slot, slot + kSlot, code, old_scales, 0, old_n, lane);
          fence_release_smem();
          if (lane == 0) mbar_arrive_remote_relaxed(even(&s->other[b1][r ^ 1]));
          other_left = false;
        } else if (h < 2 && all(mbar_test_wait(&s->codes[buf][2 * h], (it >> 1) & 1) &&
                                mbar_test_wait(&s->codes[buf][2 * h + 1], (it >> 1) & 1))) {
          uint8_t* slot = smem + kSmKv + (buf * 4 + 2 * h) * kSlot;
          uint2 code[2][2][2];
          d.read(slot, code[0]);
          d.read(slot + kSlot, code[1]);
          d.write(slot, slot + kSlot, code, own_scales, 2 * h, left - 64 * r, lane);
          fence_release_smem();
          if (lane < 2) mbar_arrive_remote_relaxed(even(&s->full[buf][2 * h + lane]));
          ++h;
        } else if (all(clock64() - idle_since > kWaitLimitCycles)) {
          if (lane == 0) abort_now();
          ok = false;
          break;
        }
      }
      if (last) break;
    }
  } else if (F8 && warp == kCodeWarp) {
    // ---------------- fp8: the codes of each step's own keys
    Cursor<kPair> c;
    int it = 0;
    bool ok = true;
    for (bool more = c.start(p, run); more && ok; more = c.next(p)) {
      Units u;
      u.start(p, c, lane, true);
      for (int kt = c.k0; kt < c.k1 && ok; ++kt, ++it) {
        const int buf = it & 1;
        const Rows x = u.get(p, c, 2 * kt + r, lane, true);
        for (int k = 0; k < 4; ++k) {
          if (it >= 2 && (k & 1) == 0 && !warp_wait(k == 0 ? &s->pv_half[buf] : &s->pv_done[buf], ((it >> 1) - 1) & 1)) {
            if (lane == 0) abort_now();
            ok = false;
            break;
          }
          load_codes(&s->codes[buf][k], buf * 4 + k, k, x.row);
        }
      }
    }
  } else if (!F8 && warp == kKeyWarp) {
    // ---------------- the own keys of each step, all 512 latent dims
    Cursor<kPair> c;
    int it = 0;
    bool ok = true;
    for (bool more = c.start(p, run); more && ok; more = c.next(p)) {
      Units u;
      u.start(p, c, lane, true);
      for (int kt = c.k0; kt < c.k1; ++kt, ++it) {
        const int buf = it & 1;
        const Rows x = u.get(p, c, 2 * kt + r, lane, true);
        // copies are served in order: the second step's wait for what the first S needs
        if (it == 1 && !warp_wait(&s->first, 0)) {
          if (lane == 0) abort_now();
          ok = false;
          break;
        }
#pragma unroll 1
        for (int k = 0; k < 4; ++k) {
          if (it >= 2 && (k & 1) == 0 && !warp_wait(k == 0 ? &s->pv_half[buf] : &s->pv_done[buf], ((it >> 1) - 1) & 1)) {
            if (lane == 0) abort_now();
            ok = false;
            break;
          }
          if (r == 0 && lane == 0) mbar_arrive_expect_tx(&s->full[buf][k], 2 * kSlot);
          load_keys(smem_u32(smem + kSmKv + (buf * 4 + k) * kSlot), &maps.keys, &maps.row, even(&s->full[buf][k]), x,
                    p.total_rows, 2 * k, 2, lane);
        }
        if (!ok) break;
      }
    }
  } else if (warp == kAuxWarp) {
    // ---------------- each step's other keys (fp8: their codes), as soon as S no
    // longer needs the dims they replace (CTA 1: after the first two slots,
    // CTA 0: after all), the rope dims of the next step's own keys, and q when
    // a row tile begins
    Cursor<kPair> c;
    int it = 0;
    Rows other{0, 0};
    const auto load_other = [&](int i) {
      const int buf = i & 1;
      if constexpr (F8) {
        for (int k = 0; k < 2; ++k) load_codes(&s->other_codes[buf][k], buf * 4 + 2 * (r ^ 1) + k, 2 * r + k, other.row);
        return;
      }
      if (r == 0 && lane == 0) {
        mbar_arrive_expect_tx(&s->other[buf][0], 2 * kSlot);
        mbar_arrive_expect_tx(&s->other[buf][1], 2 * kSlot);
      }
#pragma unroll 1
      for (int k = 0; k < 2; ++k)
        load_keys(smem_u32(smem + kSmKv + (buf * 4 + 2 * (r ^ 1) + k) * kSlot), &maps.keys, &maps.row,
                  even(&s->other[buf][r ^ 1]), other, p.total_rows, 2 * (2 * r + k), 2, lane);
    };
    bool ok = true;
    const auto after_s = [&](int i) {  // what follows S of step i; false when a wait ran out
      const int ph = (i >> 1) & 1;
      if (r == 1) {
        ok = warp_wait(&s->s_half[i & 1], ph);
        if (ok) load_other(i);
      }
      ok = ok && warp_wait(&s->s_full[i & 1], ph);
      if (!ok && lane == 0) abort_now();
      return ok;
    };
    const auto load_q = [&](int row0) {  // this CTA's 64 rows of the row tile
      if (lane == 0) {
        if (r == 0) mbar_arrive_expect_tx(&s->q, 2 * 9 * 8192);
        tma_load_3d_pair(smem_u32(smem + kSmQ), &maps.q, even(&s->q), 0, row0 + 64 * r, 0);
      }
      __syncwarp();
    };
    for (bool more = c.start(p, run); more && ok; more = c.next(p)) {
      const int row0 = (c.req.q0 + c.tile * p.tpt[kPair]) * p.H;
      if (it == 0) load_q(row0);  // needs nothing else: ahead of the block table's entries
      Units u;
      u.start(p, c, lane, false);
      // fp8: slots are free too late for copies to hide memory's latency; the own
      // keys of the step kAhead further on are asked into L2
      Units far = u;
      const auto ask = [&](int kt) {
        const Rows x = far.get(p, c, 2 * kt + r, lane, false);
        if (x.n > 0 && lane == 0) prefetch_l2(p.kv + static_cast<int64_t>(x.row) * kF8Row, x.n * kF8Row);
      };
      for (int kt = c.k0; F8 && kt < min(c.k0 + kAhead, c.k1); ++kt) ask(kt);
      for (int kt = c.k0; kt < c.k1; ++kt, ++it) {
        if (F8 && kt + kAhead < c.k1) ask(kt + kAhead);
        const Rows a = u.get(p, c, 2 * kt, lane, false), b = u.get(p, c, 2 * kt + 1, lane, false);
        const Rows x = r ? b : a, next_other = r ? a : b;
        if (it >= 1 && !after_s(it - 1)) break;
        if (r == 0 && lane == 0) mbar_arrive_expect_tx(&s->rope, 2 * 8192);
        load_keys(smem_u32(smem + kSmRope), &maps.rope, &maps.row, even(&s->rope), x, p.total_rows, F8 ? 0 : 8, 1,
                  lane);
        if (!F8 && it == 0 && lane == 0) mbar_arrive(&s->first);
        if (it >= 1 && r == 0) load_other(it - 1);
        if (it >= 1 && kt == c.k0) load_q(row0);
        other = next_other;
      }
    }
    if (ok && it >= 1 && after_s(it - 1) && r == 0) load_other(it - 1);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  } else if (warp == kMmaWarp) {
    // ---------------- MMA: the even CTA issues for the pair whatever is
    // ready, PV of the oldest step first. The warp stays converged, so that the
    // descriptors live in uniform registers, and one lane issues.
    if (r == 0) {
      const uint32_t idesc_qk = idesc_bf16(128, kTile, false, false);
      const uint32_t idesc_pv = idesc_bf16(128, 256, false, true);
      // K-major tiles (q, keys, P): 8-row groups 1024 bytes apart; keys as
      // values (dims along N): 64-dim blocks 8192 bytes apart
      const uint64_t dk = smem_desc(smem_u32(smem), 16, 1024, kSwizzle128B);
      const uint64_t dv = smem_desc(smem_u32(smem), 8192, 1024, kSwizzle128B);
      const uint32_t k_lo = static_cast<uint32_t>(dk), k_hi = static_cast<uint32_t>(dk >> 32);
      const uint32_t v_lo = static_cast<uint32_t>(dv), v_hi = static_cast<uint32_t>(dv >> 32);
      Cursor<kPair> c;
      bool more = c.start(p, run);
      int iq = 0, ip = 0, sub = 0, half = 0, segs = 0;  // the next S and PV, and the parts of them
      int kt = c.k0;
      uint32_t first = 0;  // bit i & 1: step i begins a segment
      const auto all = [](bool x) { return __all_sync(0xFFFFFFFFu, x) != 0; };
      long long idle_since = clock64();
      while ((more || ip < iq) && !__any_sync(0xFFFFFFFFu, s->abort)) {
        bool progressed = false;
        if (ip < iq && all((half == 1 || mbar_test_wait_relaxed(&s->p_full, ip & 1)) &&
                           mbar_test_wait_relaxed(&s->other[ip & 1][half], (ip >> 1) & 1))) {
          fence_acquire_smem();
          tc_fence_after();
          const int buf = ip & 1;
          const uint32_t a0 = k_lo + ((kSmP + half * 8192) >> 4);
          const uint32_t b0 = v_lo + ((kSmKv + (buf * 4 + 2 * half) * kSlot) >> 4);
          const uint32_t acc0 = half ? 1u : ~(first >> buf) & 1u;
          if (elect_one()) {
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) {  // 16 keys each
#pragma unroll
              for (int j = 0; j < 2; ++j)
                mma_bf16_ss_pair(tmem + kColO + 128 * j, a0 + ((ks * 32) >> 4), k_hi,
                                 b0 + ((j * kSlot + ks * 2048) >> 4), v_hi, idesc_pv, ks > 0 ? 1u : acc0);
            }
            mma_commit_to(half ? &s->pv_done[buf] : &s->pv_half[buf], both);
          }
          __syncwarp();
          ip += half;
          half ^= 1;
          progressed = true;
        }
        if (more && iq < ip + 2) {  // PV of step iq - 2 has been issued: S was read
          const int buf = iq & 1;
          bool ready = sub < 4 ? mbar_test_wait_relaxed(&s->full[buf][sub], (iq >> 1) & 1)
                               : mbar_test_wait_relaxed(&s->rope, iq & 1);
          if (sub == 0 && kt == c.k0) ready = ready && mbar_test_wait_relaxed(&s->q, segs & 1);
          if (all(ready)) {
            fence_acquire_smem();
            tc_fence_after();
            const uint32_t d = tmem + kColS + 64 * buf;
            if (sub < 4) {
              const uint32_t a0 = k_lo + ((kSmQ + sub * 2 * 8192) >> 4);
              const uint32_t b0 = k_lo + ((kSmKv + (buf * 4 + sub) * kSlot) >> 4);
              const uint32_t acc0 = sub > 0 ? 1u : 0u;
              if (elect_one()) {
#pragma unroll
                for (int st = 0; st < 8; ++st)
                  mma_bf16_ss_pair(d, a0 + (((st >> 2) * 8192 + (st & 3) * 32) >> 4), k_hi,
                                   b0 + (((st >> 2) * 8192 + (st & 3) * 32) >> 4), k_hi, idesc_qk, st > 0 ? 1u : acc0);
                if (sub == 1) mma_commit_to(&s->s_half[buf], both);
              }
              ++sub;
            } else {
              if (elect_one()) {
#pragma unroll
                for (int st = 0; st < 4; ++st)
                  mma_bf16_ss_pair(d, k_lo + ((kSmQ + 8 * 8192 + st * 32) >> 4), k_hi,
                                   k_lo + ((kSmRope + st * 32) >> 4), k_hi, idesc_qk, 1u);
                mma_commit_to(&s->s_full[buf], both);
              }
              first = (first & ~(1u << buf)) | (kt == c.k0 ? 1u << buf : 0u);
              sub = 0;
              ++iq;
              if (++kt == c.k1) {
                ++segs;
                more = c.next(p);
                kt = c.k0;
              }
            }
            __syncwarp();
            progressed = true;
          }
        }
        if (progressed) idle_since = clock64();
        else if (all(clock64() - idle_since > kWaitLimitCycles) && lane == 0) abort_now();
      }
    }
    __syncwarp();
  } else if (warp < kAuxWarp) {
    // ---------------- softmax: TMEM lane = 32 (warp % 4) + lane holds row
    // lane % 64 against the keys of CTA lane / 64; the two warps of a lane
    // group take 32 keys (and 128 columns of O) each
    const int l128 = (warp & 3) * 32 + lane, row = l128 & 63, kh = l128 >> 6, half = warp >> 2;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    // P stays in this CTA's shared memory, whose tensor core reads it there: the
    // proxy fence makes it visible to that core, the release of shared memory to
    // the even CTA, which issues the MMA. (A release at cluster scope of all
    // memory instead took 1300-2000 clocks per step.)
    const uint32_t p_full = even(&s->p_full);
    uint8_t* p_dst = smem + kSmP + kh * 8192;
    Cursor<kPair> c;
    int it = 0;
    uint32_t meets = 0;
    bool ok = true;
    // the four warps that hold the same 32 rows: what each wrote is seen by all
    const auto meet = [&] {
      __syncwarp();
      if (lane == 0) mbar_arrive(&s->rows[warp & 1]);
      return warp_wait(&s->rows[warp & 1], meets++ & 1);
    };
    for (bool more = c.start(p, run); more && ok; more = c.next(p)) {
      const int in_tile = 64 * r + row;  // row of the row tile
      const int tok = c.tile * p.tpt[kPair] + in_tile / p.H;
      const bool live = in_tile < p.tpt[kPair] * p.H && tok < c.req.q_len;
      const int lim = live ? visible(c.req, tok) : 0;
      float m = kNegSentinel, l = 0.f;
      Units u;
      u.start(p, c, lane, false);
      for (int kt = c.k0; kt < c.k1; ++kt, ++it) {
        const int buf = it & 1;
        const Rows x = u.get(p, c, 2 * kt + kh, lane, false);
        const int n = x.n == 0 ? 0 : lim - kt * kTile - kh * 64 - half * 32;  // of this thread's 32 keys, visible ones
        if (!warp_wait(&s->s_full[buf], (it >> 1) & 1)) {
          if (lane == 0) abort_now();
          ok = false;
          break;
        }
        tc_fence_after();
        float sc[32];
        {
          uint32_t v[32];
          tmem_ld32_sync(lane_base + kColS + 64 * buf + 32 * half, v);
#pragma unroll
          for (int i = 0; i < 32; ++i) sc[i] = __uint_as_float(v[i]) * p.scale_log2;
        }
        if (n < 32) {
#pragma unroll
          for (int i = 0; i < 32; ++i) sc[i] = i < n ? sc[i] : -INFINITY;
        }
        float mt = sc[0];
#pragma unroll
        for (int i = 1; i < 32; ++i) mt = fmaxf(mt, sc[i]);
        float* rd = red + buf * 256;
        rd[(2 * half + kh) * 64 + row] = mt;
        if (!meet()) {
          if (lane == 0) abort_now();
          ok = false;
          break;
        }
        mt = fmaxf(fmaxf(rd[row], rd[64 + row]), fmaxf(rd[128 + row], rd[192 + row]));
        const bool rescale = mt > m + kRescaleThreshold;
        const float m_new = rescale ? mt : m, neg_m = -m_new;
        float s0 = 0.f, s1 = 0.f;
        uint32_t pk[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          // the sum takes the fp32 weights; the product takes them rounded to bf16
          const float a = ex2_approx(sc[2 * i] + neg_m), b = ex2_approx(sc[2 * i + 1] + neg_m);
          s0 += a;
          s1 += b;
          pk[i] = pack_bf16(a, b);
        }
        const float alpha = rescale ? ex2_approx(m - m_new) : 1.f;
        l = l * alpha + (s0 + s1);
        m = m_new;
        // P and O are free once PV of the step before is done
        if (it >= 1 && !warp_wait(&s->pv_done[(it - 1) & 1], ((it - 1) >> 1) & 1)) {
          if (lane == 0) abort_now();
          ok = false;
          break;
        }
        tc_fence_after();
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *reinterpret_cast<uint4*>(p_dst + sw128_offset(row, 4 * half + i)) =
              make_uint4(pk[4 * i], pk[4 * i + 1], pk[4 * i + 2], pk[4 * i + 3]);
        if (kt > c.k0 && __any_sync(0xFFFFFFFFu, rescale)) {
#pragma unroll 1
          for (int q = 0; q < 128; q += 32) {
            uint32_t o[32];
            tmem_ld32_sync(lane_base + kColO + 128 * half + q, o);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
            tmem_st32(lane_base + kColO + 128 * half + q, o);
          }
          tmem_st_wait();
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        fence_release_smem();
        if (lane == 0) mbar_arrive_remote_relaxed(p_full);
      }
      if (!ok) break;
      // ---- the row tile's (or its part's) result
      float* sums = red + (it & 1) * 256;  // the maxima of the step before the last: read by all
      sums[(2 * half + kh) * 64 + row] = l;
      ok = meet();
      l = sums[row] + sums[64 + row] + sums[128 + row] + sums[192 + row];
      ok = ok && meet() && warp_wait(&s->pv_done[(it - 1) & 1], ((it - 1) >> 1) & 1);
      if (!ok) {
        if (lane == 0) abort_now();
        break;
      }
      tc_fence_after();
      const uint32_t o_base = lane_base + kColO + 128 * half;
      if (c.k0 == 0 && c.k1 == c.nk) {
        const int64_t grow = static_cast<int64_t>(c.req.q0 + c.tile * p.tpt[kPair]) * p.H + in_tile;
        const float inv = l != 0.f ? 1.f / l : 0.f;
        uint16_t* dst = p.out + grow * kDv + 256 * kh + 128 * half;
#pragma unroll 1
        for (int q = 0; q < 128; q += 32) {
          uint32_t o[32];
          tmem_ld32_sync(o_base + q, o);
#pragma unroll
          for (int e = 0; e < 2 && live; ++e) {
            uint32_t w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
              w[i] = pack_bf16(__uint_as_float(o[16 * e + 2 * i]) * inv, __uint_as_float(o[16 * e + 2 * i + 1]) * inv);
            uint16_t* d = dst + q + 16 * e;
            if (p.out32) {
              st_global_v8(d, w);
            } else {
              reinterpret_cast<uint4*>(d)[0] = make_uint4(w[0], w[1], w[2], w[3]);
              reinterpret_cast<uint4*>(d)[1] = make_uint4(w[4], w[5], w[6], w[7]);
            }
          }
          __syncwarp();
        }
        if (live && kh == 0 && half == 0 && p.lse != nullptr)
          p.lse[grow] = l != 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
      } else {
        const int slot = 2 * pair + (c.k0 > 0 ? 0 : 1);
        float4* dst = p.o_part + (static_cast<int64_t>(2 * slot + r) * 64 + 32 * half) * 128 + l128;
#pragma unroll 1
        for (int q = 0; q < 128; q += 32) {
          uint32_t o[32];
          tmem_ld32_sync(o_base + q, o);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            dst[(q / 4 + i) * 128] = make_float4(__uint_as_float(o[4 * i]), __uint_as_float(o[4 * i + 1]),
                                                 __uint_as_float(o[4 * i + 2]), __uint_as_float(o[4 * i + 3]));
        }
        if (kh == 0 && half == 0) p.ml_part[slot * 128 + in_tile] = make_float2(m, l);
        if (c.k0 == 0 && r == 0 && tid == 0) {
          // pairs whose runs hold the rest of this row tile
          const int64_t at = run->end - c.left;
          const int last = static_cast<int>((at + c.nk - 1) / run->per);
          const int rows = (min(c.req.q_len, (c.tile + 1) * p.tpt[kPair]) - c.tile * p.tpt[kPair]) * p.H;
          p.desc[pair] = make_int4((c.req.q0 + c.tile * p.tpt[kPair]) * p.H, rows, last - pair, kPair);
        }
      }
      tc_fence_before();
    }
    if (p.cut && r == 0 && tid == 0) {
      // nothing to join: no row tile that starts in this run goes on behind it
      if (!ok || run->pos >= run->end || c.k0 > 0 || c.k1 == c.nk) p.desc[pair] = make_int4(0, 0, 0, 0);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (s->abort) {
    // a wait ran out: let copies and MMAs in flight end before the memory they use is given up
    const long long t0 = clock64();
    while (clock64() - t0 < 20000000ll) __nanosleep(1000);
  }
  cluster_sync_all();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc_pair(tmem, kTmemCols);
}

}  // namespace pairs
}  // namespace dense
}  // namespace dsa
