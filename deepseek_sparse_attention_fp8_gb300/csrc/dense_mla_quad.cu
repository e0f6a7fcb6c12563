// Dense causal MLA attention for requests of several row tiles (chunks of a
// prompt, multi-token steps): row tiles of 256 rows on clusters of four CTAs.
//
// The pair kernel's M = 128 MMAs fill half of the tensor cores' rate; M = 256
// fills it, but 256 rows x 512 dims of fp32 output take the whole tensor
// memory of two CTAs. So two more CTAs make the scores:
//   CTAs 0, 1   S = Q K^T for rows [128 a, 128 a + 128), M = 256, N = 128: q's
//               latent dims in tensor memory (256 columns), its rope dims in
//               shared memory, each CTA bringing 64 of the step's 128 keys;
//               softmax; P (bf16) goes to CTA 2 + a through distributed shared
//               memory, with the factor by which the row's output shrinks;
//   CTAs 2, 3   O += P V, M = 256, N = 2 x 256: CTA 2 + a holds the outputs of
//               rows [128 a, 128 a + 128) in all 512 columns and brings value
//               dims [256 a, 256 a + 256) of all 128 keys.
// Per step an SM takes in 72 KB of keys (CTAs 0, 1), or 64 KB of values and 32
// KB of P (CTAs 2, 3): ~3000 clocks at the ~32 bytes per clock that an SM
// takes in, against 2300 and 2050 of MMA, for twice the rows of a pair's step.
// Measured: 2600-2800 clocks a step; 1024 tokens over a context of 16384 (128
// heads) 2.69 ms, 1.68 PFLOP/s or 0.90 of the measured tensor rate; a launch by
// itself 2.49 ms, with 8.9 TB/s taken in by the 144 SMs in use: both are nearly
// full (pairs: 3.58 ms).
// With the fp8 cache CTAs 0, 1 decode their 64 keys, CTAs 2, 3 their dims of
// all keys. Codes are copied to where half of their values belong and decoded
// in place. Five chunks of up to 700 tokens over up to 9000 keys: 1.75 ms (1.70
// before the odd CTAs' slots were handed on in order, then 1.45 without the
// arithmetic of decoding). With the codes loaded into registers a step ahead it
// was 1.80, and 1.43 without those loads: the few KB of L1 beside 227 KB of
// shared memory hold too few lines in flight.
#include <algorithm>

#include "dense_mla_pair.cuh"

namespace dsa {
namespace dense {
namespace {

// Warps 0-7: softmax (CTAs 0, 1), rescaling and results (CTAs 2, 3); 8 TMA
// loads, 9 MMA, 10 P on its way (CTAs 0, 1); with the fp8 cache 12-19 decode
// keys and values, 11 tells the even CTA of the odd one's.
constexpr int kWorkers = 8, kLoadWarp = 8, kMmaWarp = 9, kSendWarp = 10, kHandWarp = 11, kDecodeWarp = 12, kDecodeWarps = 8;
template <bool F8>
constexpr int kThreadsOf = F8 ? 640 : 352;
constexpr uint32_t kTmemCols = 512, kColS = 0, kColQ = 256;  // CTAs 0, 1: S 2 x 128, q 256; CTAs 2, 3: O 512

// Shared memory. CTAs 0, 1: a ring of 10 slots of 16 KB (q's 8 latent blocks of
// 128 rows x 64 dims when a row tile begins, then per step 4 slots of 64 keys
// x 128 dims), the rope dims of two steps' 64 keys, q's rope block, P and
// factors on their way to CTA 2 + a, row maxima.
// CTAs 2, 3: a ring of 10 slots (per step 4 of 64 keys x 128 dims), P as two
// buffers of 2 blocks of 128 rows x 64 keys, factors, (max, sum).
constexpr int kRing = 10;
constexpr int kSmRopeK = kRing * kSlot, kSmRopeQ = kSmRopeK + 2 * 8192, kSmPOut = kSmRopeQ + 16384, kSmRed = kSmPOut + 32768, kSmAlphaOut = kSmRed + 2048;
constexpr int kSmP = kRing * kSlot, kSmAlpha = kSmP + 2 * 32768, kSmMl = kSmAlpha + 2 * 128 * 4;
constexpr int kSmBar = kSmAlphaOut + 512;
static_assert(kSmBar + 448 <= kSmRun && kSmMl + 1024 <= kSmBar, "shared memory");

struct Bars {  // at the same offset in every CTA
  uint64_t full[kRing], empty[kRing];  // ring slots; full: of both CTAs of a pair, the even one's barrier
  uint64_t codes[kRing];               // fp8: a slot's codes landed
  // CTAs 0, 1
  uint64_t q_full, q_copied;  // q landed in the ring; copied to tensor memory by this CTA's warps
  uint64_t q_ready;           // ... by both CTAs' (CTA 0's barrier)
  uint64_t q_rope_free;       // the row tile's last S has read q's rope block
  uint64_t rope_full[2];      // the rope dims of a step's keys, of both CTAs (CTA 0's barrier); free again with S
  uint64_t s_full[2], s_free[2];  // S complete; S read by both CTAs' warps (CTA 0's barrier)
  uint64_t maxima;            // every warp has written its rows' maxima (or sums)
  uint64_t staged, sent;      // ... its part of P; P has been read by the copy to CTA 2 + a
  uint64_t ml_free;           // CTA 2 + a has read the row tile's (max, sum)
  // CTAs 2, 3
  uint64_t p_full[2], p_ready[2];  // P landed; O rescaled in both CTAs (CTA 2's barrier)
  uint64_t ml_full;
  // all: O += P V of a step complete, i.e. the P buffer is free
  uint64_t pv_done[2];
  uint32_t tmem;
  volatile int abort;
};
static_assert(sizeof(Bars) <= 448, "barrier block too large");

__device__ __forceinline__ void mma_bf16_ts_pair(uint32_t d_tmem, uint32_t a_tmem, uint32_t bdesc_lo, uint32_t bdesc_hi,
                                                 uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\tsetp.ne.b32 p, %5, 0;\n\tmov.b64 b, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "r"(bdesc_lo), "r"(bdesc_hi), "r"(idesc), "r"(accumulate));
}
// Bulk copy from this CTA's shared memory into another's, counted on a barrier
// there; bulk_read_done: the sources of this thread's copies may be overwritten.
__device__ __forceinline__ void bulk_copy_s2c(uint32_t cluster_dst, uint32_t src, uint32_t bytes, uint32_t cluster_bar) {
  asm volatile("cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   cluster_dst),
               "r"(src), "r"(bytes), "r"(cluster_bar)
               : "memory");
}
__device__ __forceinline__ void bulk_read_done() {
  asm volatile("cp.async.bulk.commit_group;\n\tcp.async.bulk.wait_group.read 0;" ::: "memory");
}
__device__ __forceinline__ void st_async_v2(uint32_t cluster_addr, uint32_t cluster_bar, uint32_t a, uint32_t b) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.b32 [%0], {%1, %2}, [%3];" ::"r"(cluster_addr),
               "r"(a), "r"(b), "r"(cluster_bar)
               : "memory");
}
// for phases that other CTAs' arrivals complete, behind a release of their
// shared memory (of tensor memory alone: behind tc_fence_before)
__device__ __forceinline__ bool warp_wait_acquire_smem(uint64_t* bar, uint32_t parity) {
  const bool ok = mbar_wait_relaxed(bar, parity);
  fence_acquire_smem();
  return __all_sync(0xFFFFFFFFu, ok);
}
__device__ __forceinline__ bool warp_wait_cluster(uint64_t* bar, uint32_t parity) {
  return __all_sync(0xFFFFFFFFu, mbar_wait_cluster(bar, parity));
}

// A ring position that walks its slots; every slot's empty barrier changes
// phase once per turn (full too, but for slots that held q).
struct Ring {
  int slot = 0;
  uint32_t turn = 0;
  __device__ __forceinline__ void next(int n = 1) {
    slot += n;
    if (slot >= kRing) {
      slot -= kRing;
      ++turn;
    }
  }
};

// Works on this quad's run, and ends with a cluster barrier.
template <bool F8>
__device__ __forceinline__ void run_quad(const DenseParams& p, const Maps& maps, const CodeMaps& code_maps,
                                         uint8_t* smem) {
  Bars* s = reinterpret_cast<Bars*>(smem + kSmBar);
  const Run* run = reinterpret_cast<const Run*>(smem + kSmRun);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = static_cast<int>(cluster_ctarank()), a = rank & 1;  // a: row half
  const bool values = rank >= 2;
  const int quad = run->index;

  if (tid == 0) {
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&s->full[i], F8 ? kDecodeWarps + (a == 0 ? 1 : 0) : 1);  // even CTAs: and the odd one's, handed on
      mbar_init(&s->empty[i], 1);
      mbar_init(&s->codes[i], 1);
    }
    mbar_init(&s->q_full, 1);
    mbar_init(&s->q_copied, kWorkers);
    mbar_init(&s->q_ready, 2 * kWorkers);
    mbar_init(&s->q_rope_free, 1);
    mbar_init(&s->rope_full[0], 1);
    mbar_init(&s->rope_full[1], 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s->s_full[i], 1);
      mbar_init(&s->s_free[i], 2 * kWorkers);
      mbar_init(&s->p_full[i], 1);
      mbar_init(&s->p_ready[i], 2 * kWorkers);
      mbar_init(&s->pv_done[i], 1);
    }
    mbar_init(&s->maxima, kWorkers);
    mbar_init(&s->staged, kWorkers);
    mbar_init(&s->sent, 1);
    mbar_init(&s->ml_free, kWorkers);
    mbar_init(&s->ml_full, 1);
    fence_mbar_init();
    s->abort = 0;
  }
  if (warp == kMmaWarp) {
    tmem_alloc_pair(&s->tmem, kTmemCols);
    tmem_relinquish_pair();
  }
  if (tid == kLoadWarp * 32) {
    prefetch_tmap(&maps.q);
    prefetch_tmap(&maps.keys);
    prefetch_tmap(&maps.rope);
    prefetch_tmap(&maps.row);
  }
  tc_fence_before();
  cluster_sync_all();  // all CTAs' barriers exist
  tc_fence_after();
  const uint32_t tmem = s->tmem;

  const auto abort_now = [&] {
    s->abort = 1;
    report(p.dev_status, DSA_DEVERR_TIMEOUT);
  };
  // a barrier's or buffer's address in another CTA
  const auto in_cta = [&](const void* x, int cta) { return mapa_shared(smem_u32(x), static_cast<uint32_t>(cta)); };
  const int even = rank & ~1;
  // fp8: 64 keys' codes of a group, to where their dims 64-127 will be
  const auto load_codes = [&](int slot, int group, int row) {
    if (lane == 0) {
      mbar_arrive_expect_tx(&s->codes[slot], 8192);
      tma_load_2d(smem_u32(smem + slot * kSlot + 8192), &code_maps.codes, &s->codes[slot], 128 * group, row);
    }
    __syncwarp();
  };
  Cursor<kQuad> c;

  if (warp == kLoadWarp && !values) {
    // ---------------- q of each row tile, then the own keys of its steps (fp8:
    // the codes of the latent dims)
    Ring ring;
    bool ok = true;
    int it = 0, seg = 0;
    const auto claim = [&] {  // the slot's former content has been used
      if (ring.turn > 0 && !warp_wait(&s->empty[ring.slot], (ring.turn - 1) & 1)) ok = false;
      return ok;
    };
    for (bool more = c.start(p, run); more && ok; more = c.next(p), ++seg) {
      const int row0 = (c.req.q0 + c.tile * p.tpt[kQuad]) * p.H + 128 * a;
      if (seg > 0 && !warp_wait(&s->q_rope_free, (seg - 1) & 1)) {
        ok = false;
        break;
      }
      if (lane == 0) {
        mbar_arrive_expect_tx(&s->q_full, 9 * 16384);
        tma_load_3d_pair(smem_u32(smem + kSmRopeQ), &maps.q, in_cta(&s->q_full, rank), 0, row0, 8);
      }
      __syncwarp();
      for (int i = 0; i < 8 && claim(); ++i, ring.next()) {
        if (lane == 0)
          tma_load_3d_pair(smem_u32(smem + ring.slot * kSlot), &maps.q, in_cta(&s->q_full, rank), 0, row0, i);
        __syncwarp();
      }
      Units u;
      u.start(p, c, lane, true);
      for (int kt = c.k0; kt < c.k1 && ok; ++kt, ++it) {
        const int buf = it & 1;
        const Rows x = u.get(p, c, 2 * kt + a, lane, true);
        for (int k = 0; k < 4 && claim(); ++k, ring.next()) {
          if constexpr (F8) {
            load_codes(ring.slot, k, x.row);
            continue;
          }
          if (a == 0 && lane == 0) mbar_arrive_expect_tx(&s->full[ring.slot], 2 * kSlot);
          load_keys(smem_u32(smem + ring.slot * kSlot), &maps.keys, &maps.row, in_cta(&s->full[ring.slot], even), x,
                    p.total_rows, 2 * k, 2, lane);
        }
        // the rope dims: their buffer is free with S of the step before the last
        ok = ok && (it < 2 || warp_wait(&s->s_full[buf], ((it >> 1) - 1) & 1));
        if (!ok) break;
        if (a == 0 && lane == 0) mbar_arrive_expect_tx(&s->rope_full[buf], 2 * 8192);
        load_keys(smem_u32(smem + kSmRopeK + buf * 8192), &maps.rope, &maps.row, in_cta(&s->rope_full[buf], even), x,
                  p.total_rows, F8 ? 0 : 8, 1, lane);
      }
    }
    if (!ok && lane == 0) abort_now();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  } else if (F8 && warp >= kDecodeWarp) {
    // ---------------- fp8: a step's 4 slots of 64 keys x 128 dims (CTAs 0, 1:
    // the 4 groups of the own keys; CTAs 2, 3: the 2 own groups of both units
    // of keys), 8 keys per warp
    const Decoder d(warp - kDecodeWarp, lane);
    Ring ring;
    uint32_t phases = 0;  // of the slots' code barriers: q's uses of a slot do not count there
    Units u;
    bool more = c.start(p, run), ok = true;
    int kt = c.k0;
    // the 32 scales of a step and this warp's keys, one per lane: slot lane & 3
    // of key lane >> 2; those of the next step are in flight
    float scale_next = 0.f;
    const auto fetch_scales = [&] {
      if (kt == c.k0) u.start(p, c, lane, false);
      else u.advance(p, c, kt, lane, false);
      Rows x = u.of(p, c, kt, values ? 0 : a);
      if (values) {
        const Rows x1 = u.of(p, c, kt, 1);
        if (lane & 2) x = x1;
      }
      scale_next = d.scale(p, x, values ? 2 * a + (lane & 1) : lane & 3, lane);
    };
    if (more) fetch_scales();
    while (more && ok) {
      if (!values && kt == c.k0) ring.next(8);  // q's slots
      const int left = c.req.kv_len - kt * kTile - d.key0 - (lane >> 3);  // keys that exist
      const float scales = scale_next;
      if (++kt == c.k1) {
        more = c.next(p);
        kt = c.k0;
      }
      if (more) fetch_scales();
#pragma unroll
      for (int h = 0; h < 2; ++h) {  // two slots at a time
        int to[2];
        uint2 code[2][2][2];
#pragma unroll
        for (int g = 0; g < 2; ++g, ring.next()) {
          to[g] = ring.slot;
          ok = ok && warp_wait(&s->codes[ring.slot], (phases >> ring.slot) & 1);
          phases ^= 1u << ring.slot;
          d.read(smem + to[g] * kSlot, code[g]);
        }
        if (!ok) break;
        d.write(smem + to[0] * kSlot, smem + to[1] * kSlot, code, scales, 2 * h, left - 64 * (values ? h : a), lane);
        if (lane < 2) mbar_arrive(&s->full[lane ? to[1] : to[0]]);
      }
    }
    if (!ok && lane == 0) abort_now();
  } else if (F8 && warp == kHandWarp) {
    // ---------------- fp8: the odd CTA's decoded slots to the even one, whose warp
    // issues the MMAs, two at a time. A fence in the decoding warps themselves
    // would wait for the scales that they have in flight
    if (a == 1) {
      const uint32_t full0 = in_cta(&s->full[0], even);
      Ring ring;
      uint32_t phases = 0;
      bool ok = true;
      for (bool more = c.start(p, run); more && ok; more = c.next(p)) {
        if (!values) ring.next(8);
        for (int i = 2 * (c.k1 - c.k0); i > 0 && ok; --i) {
          int of[2];
#pragma unroll
          for (int g = 0; g < 2; ++g, ring.next()) {
            of[g] = ring.slot;
            ok = ok && warp_wait(&s->full[ring.slot], (phases >> ring.slot) & 1);
            phases ^= 1u << ring.slot;
          }
          if (!ok) break;
          fence_release_smem();
          if (lane < 2) mbar_arrive_remote_relaxed(full0 + 8 * (lane ? of[1] : of[0]));
        }
      }
      if (!ok && lane == 0) abort_now();
    }
    __syncwarp();
  } else if (warp == kLoadWarp) {
    // ---------------- all keys of each step, the own value dims
    Ring ring;
    bool ok = true;
    for (bool more = c.start(p, run); more && ok; more = c.next(p)) {
      Units u;
      u.start(p, c, lane, false);
      for (int kt = c.k0; kt < c.k1 && ok; ++kt) {
        const Rows x0 = u.get(p, c, 2 * kt, lane, false), x1 = u.get(p, c, 2 * kt + 1, lane, false);
        for (int k = 0; k < 4; ++k, ring.next()) {
          if (ring.turn > 0 && !warp_wait(&s->empty[ring.slot], (ring.turn - 1) & 1)) {
            if (lane == 0) abort_now();
            ok = false;
            break;
          }
          if constexpr (F8) {
            load_codes(ring.slot, 2 * a + (k & 1), k < 2 ? x0.row : x1.row);
            continue;
          }
          if (a == 0 && lane == 0) mbar_arrive_expect_tx(&s->full[ring.slot], 2 * kSlot);
          load_keys(smem_u32(smem + ring.slot * kSlot), &maps.keys, &maps.row, in_cta(&s->full[ring.slot], even),
                    k < 2 ? x0 : x1, p.total_rows, 2 * (2 * a + (k & 1)), 2, lane);
        }
      }
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  } else if (warp == kMmaWarp && !values) {
    // ---------------- S, issued by CTA 0 for both. The warp stays converged,
    // so that the descriptors live in uniform registers; one lane issues
    if (rank == 0) {
      const uint32_t idesc = idesc_bf16(256, kTile, false, false);
      const uint64_t dk = smem_desc(smem_u32(smem), 16, 1024, kSwizzle128B);
      const uint32_t k_lo = static_cast<uint32_t>(dk), k_hi = static_cast<uint32_t>(dk >> 32);
      Ring ring;
      uint32_t phases = 0;  // of the slots' full barriers: q's uses of a slot do not count there
      bool ok = true;
      int it = 0, seg = 0;
      for (bool more = c.start(p, run); more && ok; more = c.next(p), ++seg) {
        ring.next(8);
        ok = warp_wait_acquire_smem(&s->q_ready, seg & 1);
        for (int kt = c.k0; kt < c.k1 && ok; ++kt, ++it) {
          const int buf = it & 1;
          if (it >= 2) ok = warp_wait_acquire_smem(&s->s_free[buf], ((it >> 1) - 1) & 1);
          const uint32_t d = tmem + kColS + 128 * buf;
#pragma unroll 1
          for (int k = 0; k < 4 && ok; ++k, ring.next()) {
            ok = warp_wait_acquire_smem(&s->full[ring.slot], (phases >> ring.slot) & 1);
            if (!ok) break;
            phases ^= 1u << ring.slot;
            tc_fence_after();
            const uint32_t b0 = k_lo + ((ring.slot * kSlot) >> 4), q0 = tmem + kColQ + k * 64, acc0 = k > 0 ? 1u : 0u;
            if (elect_one()) {
#pragma unroll
              for (int st = 0; st < 8; ++st)
                mma_bf16_ts_pair(d, q0 + st * 8, b0 + (((st >> 2) * 8192 + (st & 3) * 32) >> 4), k_hi, idesc,
                                 st > 0 ? 1u : acc0);
              mma_commit_to(&s->empty[ring.slot], 0x3);
            }
            __syncwarp();
          }
          ok = ok && warp_wait_acquire_smem(&s->rope_full[buf], (it >> 1) & 1);
          if (!ok) break;
          tc_fence_after();
          const uint32_t b0 = k_lo + ((kSmRopeK + buf * 8192) >> 4);
          const bool last = kt + 1 == c.k1;
          if (elect_one()) {
#pragma unroll
            for (int st = 0; st < 4; ++st)
              mma_bf16_ss_pair(d, k_lo + ((kSmRopeQ + st * 32) >> 4), k_hi, b0 + ((st * 32) >> 4), k_hi, idesc, 1u);
            mma_commit_to(&s->s_full[buf], 0x3);
            if (last) mma_commit_to(&s->q_rope_free, 0x3);
          }
          __syncwarp();
        }
      }
      if (!ok && lane == 0) abort_now();
    }
    __syncwarp();
  } else if (warp == kMmaWarp) {
    // ---------------- O += P V, issued by CTA 2 for both
    if (rank == 2) {
      const uint32_t idesc = idesc_bf16(256, 256, false, true);
      // P: 8-row groups 1024 bytes apart; values (dims along N): 64-dim blocks 8192 bytes apart
      const uint64_t dp = smem_desc(smem_u32(smem), 16, 1024, kSwizzle128B);
      const uint64_t dv = smem_desc(smem_u32(smem), 8192, 1024, kSwizzle128B);
      const uint32_t p_lo = static_cast<uint32_t>(dp), p_hi = static_cast<uint32_t>(dp >> 32);
      const uint32_t v_lo = static_cast<uint32_t>(dv), v_hi = static_cast<uint32_t>(dv >> 32);
      Ring ring;
      bool ok = true;
      int it = 0;
      for (bool more = c.start(p, run); more && ok; more = c.next(p)) {
        for (int kt = c.k0; kt < c.k1 && ok; ++kt, ++it) {
          const int buf = it & 1;
          ok = warp_wait_acquire_smem(&s->p_ready[buf], (it >> 1) & 1);
#pragma unroll 1
          for (int kh = 0; kh < 2 && ok; ++kh) {  // 64 keys each: a slot of 128 dims after the other
            const int s0 = ring.slot;
            ok = warp_wait_acquire_smem(&s->full[ring.slot], ring.turn & 1);
            ring.next();
            const int s1 = ring.slot;
            ok = ok && warp_wait_acquire_smem(&s->full[ring.slot], ring.turn & 1);
            ring.next();
            if (!ok) break;
            tc_fence_after();
            const uint32_t a0 = p_lo + ((kSmP + buf * 32768 + kh * 16384) >> 4);
            const uint32_t b0 = v_lo + ((s0 * kSlot) >> 4), b1 = v_lo + ((s1 * kSlot) >> 4);
            const uint32_t acc0 = (kt > c.k0 || kh > 0) ? 1u : 0u;
            if (elect_one()) {
#pragma unroll
              for (int ks = 0; ks < 4; ++ks) {  // 16 keys each
                mma_bf16_ss_pair(tmem, a0 + ((ks * 32) >> 4), p_hi, b0 + ((ks * 2048) >> 4), v_hi, idesc, ks > 0 ? 1u : acc0);
                mma_bf16_ss_pair(tmem + 256, a0 + ((ks * 32) >> 4), p_hi, b1 + ((ks * 2048) >> 4), v_hi, idesc,
                                 ks > 0 ? 1u : acc0);
              }
              mma_commit_to(&s->empty[s0], 0xC);
              mma_commit_to(&s->empty[s1], 0xC);
              if (kh == 1) mma_commit_to(&s->pv_done[buf], 0xF);
            }
            __syncwarp();
          }
        }
      }
      if (!ok && lane == 0) abort_now();
    }
    __syncwarp();
  } else if (warp == kSendWarp) {
    // ---------------- P and the factors of each step to CTA 2 + a
    if (!values) {
      const uint32_t p_dst = in_cta(smem + kSmP, 2 + a), p_full = in_cta(&s->p_full[0], 2 + a);
      const uint32_t alpha_dst = in_cta(smem + kSmAlpha, 2 + a);
      bool ok = true;
      int it = 0;
      for (bool more = c.start(p, run); more && ok; more = c.next(p)) {
        for (int kt = c.k0; kt < c.k1; ++kt, ++it) {
          const int buf = it & 1;
          // P is staged, and its buffer there is free: PV of the step before the last is done
          ok = warp_wait(&s->staged, it & 1) && (it < 2 || warp_wait(&s->pv_done[buf], ((it >> 1) - 1) & 1));
          if (!ok) {
            if (lane == 0) abort_now();
            break;
          }
          if (lane == 0) {
            bulk_copy_s2c(p_dst + buf * 32768, smem_u32(smem + kSmPOut), 32768, p_full + 8 * buf);
            bulk_copy_s2c(alpha_dst + buf * 512, smem_u32(smem + kSmAlphaOut), 512, p_full + 8 * buf);
            bulk_read_done();
            mbar_arrive(&s->sent);
          }
          __syncwarp();
        }
      }
    }
  } else if (warp < kWorkers && !values) {
    // ---------------- softmax: TMEM lane = row; the two warps of a lane group
    // take 64 keys each
    const int row = (warp & 3) * 32 + lane, half = warp >> 2;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    float* red = reinterpret_cast<float*>(smem + kSmRed);  // [step parity][half][row]
    const uint32_t q_ready = in_cta(&s->q_ready, 0), s_free = in_cta(&s->s_free[0], 0);
    uint8_t* p_out = smem + kSmPOut + half * 16384;
    Ring ring;
    bool ok = true;
    int it = 0, seg = 0;
    uint32_t meets = 0;
    const auto meet = [&] {  // what every warp wrote is seen by all
      __syncwarp();
      if (lane == 0) mbar_arrive(&s->maxima);
      return warp_wait(&s->maxima, meets++ & 1);
    };
    for (bool more = c.start(p, run); more && ok; more = c.next(p), ++seg) {
      // q's latent dims -> tensor memory (the A operand); its slots are then free
      if (!warp_wait(&s->q_full, seg & 1)) {
        if (lane == 0) abort_now();
        break;
      }
      for (int i = 0; i < 8; ++i, ring.next()) {
        if ((i & 1) != half) continue;
        const uint8_t* blk = smem + ring.slot * kSlot;
        uint32_t v[32];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint4 w = *reinterpret_cast<const uint4*>(blk + sw128_offset(row, k));
          v[4 * k] = w.x;
          v[4 * k + 1] = w.y;
          v[4 * k + 2] = w.z;
          v[4 * k + 3] = w.w;
        }
        tmem_st32(lane_base + kColQ + 32 * i, v);
      }
      tmem_st_wait();
      fence_proxy_async_smem();  // the slots are refilled by TMA
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&s->q_copied);
        mbar_arrive_remote_relaxed(q_ready);
      }
      if (warp == 0) {
        if (!warp_wait(&s->q_copied, seg & 1)) {
          if (lane == 0) abort_now();
          break;
        }
        if (lane < 8) mbar_arrive(&s->empty[(ring.slot + kRing - 8 + lane) % kRing]);
        __syncwarp();
      }
      ring.slot = (ring.slot + 4 * ((c.k1 - c.k0) % kRing)) % kRing;  // the steps' slots

      const int in_tile = 128 * a + row;
      const int tok = c.tile * p.tpt[kQuad] + in_tile / p.H;
      const bool live = in_tile < p.tpt[kQuad] * p.H && tok < c.req.q_len;
      const int lim = live ? visible(c.req, tok) : 0;
      float m = kNegSentinel, l = 0.f;
      Units u;
      u.start(p, c, lane, false);
      for (int kt = c.k0; kt < c.k1; ++kt, ++it) {
        const int buf = it & 1;
        const Rows x = u.get(p, c, 2 * kt + half, lane, false);
        const int n = x.n == 0 ? 0 : lim - kt * kTile - half * 64;  // of this thread's 64 keys, visible ones
        if (!warp_wait(&s->s_full[buf], (it >> 1) & 1)) {
          if (lane == 0) abort_now();
          ok = false;
          break;
        }
        tc_fence_after();
        // 32 scores at a time: once for the maximum, once more for the weights,
        // as 64 registers of them would spill beside the decoding warps'
        const auto scores = [&](int h, float (&sc)[32]) {
          uint32_t v[32];
          tmem_ld32_sync(lane_base + kColS + 128 * buf + 64 * half + 32 * h, v);
#pragma unroll
          for (int i = 0; i < 32; ++i) sc[i] = __uint_as_float(v[i]);
          if (n < 32 * h + 32) {
#pragma unroll
            for (int i = 0; i < 32; ++i) sc[i] = 32 * h + i < n ? sc[i] : -INFINITY;
          }
        };
        float mt = -INFINITY;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float sc[32];
          scores(h, sc);
#pragma unroll
          for (int i = 0; i < 32; ++i) mt = fmaxf(mt, sc[i]);
        }
        float* rd = red + buf * 256;
        rd[half * 128 + row] = mt;
        if (!meet()) {
          if (lane == 0) abort_now();
          ok = false;
          break;
        }
        mt = fmaxf(rd[row], rd[128 + row]) * p.scale_log2;
        const bool rescale = mt > m + kRescaleThreshold;
        const float m_new = rescale ? mt : m, neg_m = -m_new;
        const float alpha = rescale ? ex2_approx(m - m_new) : 1.f;
        m = m_new;
        float s0 = 0.f, s1 = 0.f;
        uint32_t pk[32];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float sc[32];
          scores(h, sc);
          if (h == 1) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_remote_relaxed(s_free + 8 * buf);
          }
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            // the sum takes the fp32 weights; the product takes them rounded to bf16
            const float e0 = ex2_approx(fmaf(sc[2 * i], p.scale_log2, neg_m));
            const float e1 = ex2_approx(fmaf(sc[2 * i + 1], p.scale_log2, neg_m));
            s0 += e0;
            s1 += e1;
            pk[16 * h + i] = pack_bf16(e0, e1);
          }
        }
        // P's staging memory is free once the last step's copy has read it
        if (it > 0) ok = warp_wait(&s->sent, (it - 1) & 1);
        if (!ok) {
          if (lane == 0) abort_now();
          break;
        }
#pragma unroll
        for (int k = 0; k < 8; ++k)
          *reinterpret_cast<uint4*>(p_out + sw128_offset(row, k)) =
              make_uint4(pk[4 * k], pk[4 * k + 1], pk[4 * k + 2], pk[4 * k + 3]);
        if (half == 0) *reinterpret_cast<float*>(smem + kSmAlphaOut + 4 * row) = alpha;
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s->staged);
        l = l * alpha + (s0 + s1);
      }
      if (!ok) break;
      // the row tile's (or its part's) maximum and sum
      float* sums = red + (it & 1) * 256;  // the maxima of the step before the last: read by both
      sums[half * 128 + row] = l;
      ok = meet();
      l = sums[row] + sums[128 + row];
      ok = ok && meet();
      if (ok && seg > 0 && half == 0) ok = warp_wait_acquire_smem(&s->ml_free, (seg - 1) & 1);
      if (!ok) {
        if (lane == 0) abort_now();
        break;
      }
      if (half == 0)
        st_async_v2(in_cta(smem + kSmMl, 2 + a) + row * 8, in_cta(&s->ml_full, 2 + a), __float_as_uint(m), __float_as_uint(l));
    }
  } else if (warp < kWorkers) {
    // ---------------- O: rescaling when a row's maximum has grown, and the
    // results; TMEM lane = row, the two warps of a lane group take 256 columns each
    const int row = (warp & 3) * 32 + lane, half = warp >> 2;
    const uint32_t o_base = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + 256 * half;
    const float* alphas = reinterpret_cast<const float*>(smem + kSmAlpha);
    const float2* mls = reinterpret_cast<const float2*>(smem + kSmMl);
    const uint32_t p_ready = in_cta(&s->p_ready[0], 2), ml_free = in_cta(&s->ml_free, a);
    bool ok = true;
    int it = 0, seg = 0;
    for (bool more = c.start(p, run); more && ok; more = c.next(p), ++seg) {
      for (int kt = c.k0; kt < c.k1; ++kt, ++it) {
        const int buf = it & 1;
        if (tid == 0) mbar_arrive_expect_tx(&s->p_full[buf], 32768 + 512);
        __syncwarp();
        ok = warp_wait_cluster(&s->p_full[buf], (it >> 1) & 1);
        const float alpha = ok && kt > c.k0 ? alphas[buf * 128 + row] : 1.f;  // (a row tile begins with any)
        if (__any_sync(0xFFFFFFFFu, alpha != 1.f)) {
          ok = warp_wait(&s->pv_done[buf ^ 1], ((it - 1) >> 1) & 1);
          if (ok) {
            tc_fence_after();
#pragma unroll 1
            for (int q = 0; q < 256; q += 32) {
              uint32_t o[32];
              tmem_ld32_sync(o_base + q, o);
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
              tmem_st32(o_base + q, o);
            }
            tmem_st_wait();
          }
        }
        if (!ok) {
          if (lane == 0) abort_now();
          break;
        }
        tc_fence_before();
        __syncwarp();
        fence_release_smem();  // P and the factors have landed, O is rescaled
        if (lane == 0) mbar_arrive_remote_relaxed(p_ready + 8 * buf);
      }
      if (!ok) break;
      if (tid == 0) mbar_arrive_expect_tx(&s->ml_full, 128 * 8);
      __syncwarp();
      ok = warp_wait_cluster(&s->ml_full, seg & 1);
      const float2 ml = ok ? mls[row] : make_float2(0.f, 0.f);
      ok = ok && warp_wait(&s->pv_done[(it - 1) & 1], ((it - 1) >> 1) & 1);
      if (!ok) {
        if (lane == 0) abort_now();
        break;
      }
      // the reads come before the arrival that lets CTA a write the next row tile's
      __syncwarp();
      fence_release_smem();
      if (lane == 0) mbar_arrive_remote_relaxed(ml_free);
      tc_fence_after();
      const int in_tile = 128 * a + row;
      const int tok = c.tile * p.tpt[kQuad] + in_tile / p.H;
      const bool live = in_tile < p.tpt[kQuad] * p.H && tok < c.req.q_len;
      if (c.k0 == 0 && c.k1 == c.nk) {
        const int64_t grow = static_cast<int64_t>(c.req.q0 + c.tile * p.tpt[kQuad]) * p.H + in_tile;
        const float inv = ml.y != 0.f ? 1.f / ml.y : 0.f;
#pragma unroll 1
        for (int q = 0; q < 256; q += 32) {  // columns 0-127 of a half: dims 128 half on; 128-255: 256 + 128 half on
          uint32_t o[32];
          tmem_ld32_sync(o_base + q, o);
          uint16_t* dst = p.out + grow * kDv + 128 * half + (q & 127) + 256 * (q >> 7);
#pragma unroll
          for (int e = 0; e < 2 && live; ++e) {
            uint32_t w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
              w[i] = pack_bf16(__uint_as_float(o[16 * e + 2 * i]) * inv, __uint_as_float(o[16 * e + 2 * i + 1]) * inv);
            if (p.out32) {
              st_global_v8(dst + 16 * e, w);
            } else {
              reinterpret_cast<uint4*>(dst + 16 * e)[0] = make_uint4(w[0], w[1], w[2], w[3]);
              reinterpret_cast<uint4*>(dst + 16 * e)[1] = make_uint4(w[4], w[5], w[6], w[7]);
            }
          }
          __syncwarp();
        }
        if (live && half == 0 && p.lse != nullptr) p.lse[grow] = ml.y != 0.f ? (ml.x + log2f(ml.y)) * kLn2 : -INFINITY;
      } else {
        const int slot = 2 * quad + (c.k0 > 0 ? 0 : 1);
        float4* dst = p.o_part + (static_cast<int64_t>(2 * slot + a) * 128 + 64 * half) * 128 + row;
#pragma unroll 1
        for (int q = 0; q < 256; q += 32) {
          uint32_t o[32];
          tmem_ld32_sync(o_base + q, o);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            dst[(q / 4 + i) * 128] = make_float4(__uint_as_float(o[4 * i]), __uint_as_float(o[4 * i + 1]),
                                                 __uint_as_float(o[4 * i + 2]), __uint_as_float(o[4 * i + 3]));
        }
        if (half == 0) p.ml_part[slot * 256 + in_tile] = ml;
        if (c.k0 == 0 && rank == 2 && tid == 0) {
          // runs that hold the rest of this row tile
          const int64_t at = run->end - c.left;
          const int last = static_cast<int>((at + c.nk - 1) / run->per);
          const int rows = (min(c.req.q_len, (c.tile + 1) * p.tpt[kQuad]) - c.tile * p.tpt[kQuad]) * p.H;
          p.desc[quad] = make_int4((c.req.q0 + c.tile * p.tpt[kQuad]) * p.H, rows, last - quad, kQuad);
        }
      }
      tc_fence_before();
    }
    if (rank == 2 && tid == 0) {
      // nothing to join: no row tile that starts in this run goes on behind it;
      // and the pair kernel's runs beyond leave nothing
      if (!ok || run->pos >= run->end || c.k0 > 0 || c.k1 == c.nk) p.desc[quad] = make_int4(0, 0, 0, 0);
      for (int i = quad + p.quads; i < p.pairs; i += p.quads) p.desc[i] = make_int4(0, 0, 0, 0);
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

// The lengths decide whether a cluster works as a quad or as two pairs.
template <bool F8>
__global__ void __launch_bounds__(kThreadsOf<F8>, 1) dense_mla_quad_kernel(const __grid_constant__ DenseParams p,
                                                                          const __grid_constant__ Maps quad_maps,
                                                                          const __grid_constant__ Maps pair_maps,
                                                                          const __grid_constant__ CodeMaps code_maps) {
  extern __shared__ __align__(1024) uint8_t smem[];
  if (misaligned(p, smem)) return;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Run* run = reinterpret_cast<const Run*>(smem + kSmRun);
  plan_run<kThreadsOf<F8>, kQuad>(p, reinterpret_cast<Run*>(smem + kSmRun), smem);
  if (run->kind == kQuad) {
    run_quad<F8>(p, quad_maps, code_maps, smem);
  } else {
    pairs::set_up<F8>(reinterpret_cast<pairs::Bars*>(smem + pairs::kSmBar), pair_maps);
    pairs::run_pair<F8>(p, pair_maps, code_maps, smem);
  }
}

FuncAttrOnce g_smem[2];
std::atomic<int> g_quads[2][kMaxDeviceOrdinals];  // clusters at once + 1, 0 = not asked yet

template <bool F8>
void config(cudaLaunchConfig_t* cfg, cudaLaunchAttribute* attr, int quads, cudaStream_t s) {
  *cfg = {};
  cfg->gridDim = dim3(static_cast<unsigned>(4 * quads));
  cfg->blockDim = dim3(kThreadsOf<F8>);
  cfg->dynamicSmemBytes = kSmTotal;
  cfg->stream = s;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 4;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg->attrs = attr;
  cfg->numAttrs = 2;
}

template <bool F8>
int clusters_at_once() {
  int clusters = 0;
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[2];
  config<F8>(&cfg, attr, 1, nullptr);
  cfg.numAttrs = 1;
  if (allow_smem(dense_mla_quad_kernel<F8>, kSmTotal, g_smem[F8]) != DSA_OK ||
      cudaOccupancyMaxActiveClusters(&clusters, dense_mla_quad_kernel<F8>, &cfg) != cudaSuccess) {
    cudaGetLastError();
    clusters = 0;
  }
  return std::min(clusters, num_sms() / 4);
}

template <bool F8>
dsa_status_t launch(const DenseParams& p, const void* q, const void* kv, cudaStream_t s) {
  Maps quad_maps, pair_maps;
  CodeMaps code_maps = {};
  dsa_status_t st;
  if ((st = make_maps(&quad_maps, p, F8, q, kv, 128, 1)) != DSA_OK) return st;
  if ((st = make_maps(&pair_maps, p, F8, q, kv, 64, 9)) != DSA_OK) return st;
  if (F8 && (st = make_code_maps(&code_maps, p, kv)) != DSA_OK) return st;
  if ((st = allow_smem(dense_mla_quad_kernel<F8>, kSmTotal, g_smem[F8])) != DSA_OK) return st;
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[2];
  config<F8>(&cfg, attr, p.quads, s);
  cudaError_t e = cudaLaunchKernelEx(&cfg, dense_mla_quad_kernel<F8>, p, quad_maps, pair_maps, code_maps);
  if (e != cudaSuccess) return fail(DSA_ERR_CUDA, "dense_mla_quad_kernel launch failed: %s", cudaGetErrorString(e));
  return DSA_OK;
}

}  // namespace

int num_quads(bool f8) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDeviceOrdinals) return 0;
  std::atomic<int>& known = g_quads[f8][dev];
  int n = known.load(std::memory_order_acquire);
  if (n == 0) {
    n = (f8 ? clusters_at_once<true>() : clusters_at_once<false>()) + 1;
    known.store(n, std::memory_order_release);
  }
  return n - 1;
}

dsa_status_t launch_quads(const DenseParams& p, bool f8, const void* q, const void* kv, cudaStream_t s) {
  return f8 ? launch<true>(p, q, kv, s) : launch<false>(p, q, kv, s);
}

}  // namespace dense
}  // namespace dsa
