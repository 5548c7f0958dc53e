// mla_fp4.cuh -- paged MLA decode / spec-verify over the 400-byte mxfp4 record.
//
// A record holds 512 E2M1 codes of kv_c_normed (value 2i in the low half of byte i), the 16 exponents of
// the scales of its groups of 32 values (a byte each, 2^(byte - 127)), then 64 bf16 of k_pe.  With
// K = max_g k_g a value is code * 2^(k_g - K) * 2^K; an insert keeps K - k_g <= 14, so that
// v = code * 2^(6 + k_g - K) is an E4M3 number exactly (at most 6 * 2^6 = 384, at least 0.5 * 2^-8 = 2^-9), and
//   key = [2^(K - 6) v | k_pe],  value = 2^(K - 6) v:
// one power of two a key in front of E4M3 operands.  (Groups further below K, which no insert writes, read
// as zero.)
//
// How (GB300 design):
//   * The key tiles of all requests, one after the other, are cut into equal runs, one for each CTA of a group of NQ query
//     columns (a column is a (query token, head) pair); the CTAs of all groups take the same run side by side and meet
//     its records in L2.  Where a run begins or ends inside a request its part is a partial result, at most two a CTA,
//     which a second kernel joins; the lengths are read on the GPU, so a captured graph stays balanced.  (Splits of
//     equal length, handed out by a counter: 32 requests of 1024 to 8192 keys 63 us, 39 so.)
//   * Two tiles in shared memory, each four slots of E4M3 codes of 128 values and bf16 k_pe, K-major with 128-byte swizzle, read by
//     both products.  A group has up to 64 columns: what bounds a tile is its conversion and the products' reads of it, whose
//     cost hardly depends on the columns (4 x 16 rows over 16k to 128k keys, 64 requests, with two terms a weight: two groups of
//     32 1350 us, one of 64 1030).  64 columns and three terms leave room for two tiles of 96 keys (12 a loader warp): QK takes
//     the other 32 of its 128 rows from what lies behind, and their scores are masked.  Where groups of 48 are as many, they
//     take tiles of 128 keys in less time (128 requests of 96 heads over 8k to 32k keys, two terms: three groups of 32 1147 us, two
//     of 64 1126, two of 48 951).
//   * Eight loader warps take 16 (12) keys of a tile each: 16-byte loads straight from the pages one tile ahead in
//     registers, block ids two tiles ahead.  A group's exponent below K picks two words that hold the E4M3 bytes of the eight
//     magnitudes at that scale; a byte permute turns four codes into four bytes.  That is 1.5 instructions a code,
//     where the conversion instructions by way of f16 take as many but run at half rate.
//   * Products on the 5th-generation tensor cores with keys (latents) as M = 128 and query columns as N.
//     S^T = V Q^T: the bf16 query of a column as two E4M3 terms hi + 2^-4 lo of 2^e q (they carry its 8 bits down to 2^-6
//     of the scaled range's 448); k_pe . q_pe as a bf16 product of its own.
//   * Online softmax over s' = s + K - 6: the weight of a key's codes is w = 2^(s' - m), its share of the row
//     sum w 2^(6 - K) = 2^(s - m), so the key's scale costs one multiplication.  The weights enter
//     O^T += V^T P as three E5M2 terms, each the rest rounded to nearest: a weight is off by 2^-10 of itself at most (half a step
//     of the last term, 2^-11, and of the f16 that is split, 2^-11), and nothing is lost above 2^-27 of the reference, which
//     may stand far above most weights of a row (one large key in front; two E4M3 terms ended at 2^-15 and dropped 4 to
//     35 % of such a row's output).  Over 2^17 keys that is 2^-10 of the largest weight.  The reference m moves only when a
//     logit passes it by kTau, a move costs 2.8 us: the higher kTau, the earlier E5M2 ends below the reference (4 x 16 rows as
//     above, 128 requests of 96 heads as above and 32 requests of 1024 to 8192 keys: kTau 4.75 1127, 1005 and 39.5 us, 5.75
//     1099, 1003 and 39.1; the two E4M3 terms took 1025, 939 and 37.2).  The largest weight of an item's first tile is 2^kPExp, a term exactly.
//   * The tensor cores add in fp32 and cut off: 2^-23 of an accumulator a product, of 32 keys.  Terms of both signs make less
//     of it (131072 flat keys behind one of 15 nats more: output 0.0009 too small; 2^20 keys: 0.002).
//   * The terms of a weight stand side by side along N with accumulators of their own that the epilogue adds (16 columns), or as
//     many as the tensor memory has room for, and the others add to the last accumulators by products of their own, one after the
//     other along K (32 columns: two and one; more: one each).
//   * hi and lo terms of the query are stacked along N; from 48 columns on the tensor memory has no room for that, and hi and the
//     plain rest lo = x - hi go to the same scores.  A rest is then kept to 2^-10 of the scaled range: a query's value to 2^-18
//     of the column's largest.
//   * Roles hand over through mbarriers, each waited with a time limit.  Waits between the products and what feeds them are
//     polled: a suspended thread (try_wait) was woken 0.5 to 1 us late, four times a tile (1390 -> 1095 us; of 16 columns 43 ->
//     39).
//
// What bounds it now, 64 columns (3.3 us a tile of 96 keys; 48: 3.7 us of 128): loaders (load latency, then conversion and
// stores), softmax (ordered after QK) and the tensor pipe, whose operand reads (6 KB a product of 33 cycles) share the data
// path of shared memory with both: 72 (84) products a tile at 75 cycles each.  Up to 32 columns: the chain of load, conversion, QK, softmax and PV of two tiles (2.5 us a tile).
//
// Warps: 0 scheduler, 1 QK issuer (TMEM owner), 2 PV issuer, then the softmax warps (which also prepare the query and
// write the results), then 8 loaders.
#pragma once
#include "mla_ds.cuh"

namespace mla {

constexpr int kFp4Entry = 400;          // bytes: 256 codes, 16 exponents, 128 k_pe
constexpr int kFp4Exps = 256, kFp4Rope = 272;

struct Fp4Params {
  const uint8_t* q;               // bf16 [rows][H][>=576]
  int64_t q_s0b, q_s1b;
  const uint8_t* kv;
  uint32_t blk_stride, ent_stride;
  int H, q_len, B, G, cols;       // G groups of NQ columns of the q_len * H
  const int32_t* block_table;
  int64_t bt_stride;
  const int32_t* seq_lens;
  uint32_t num_blocks;
  int block_size, bs_shift;       // n / block_size = n bs_magic / 2^(31 + bs_shift) for n < 2^31: bs_shift = ceil(log2(block_size)),
  uint32_t bs_magic;              // bs_magic = ceil(2^(31 + bs_shift) / block_size)
  int W;                          // runs of tiles: the grid is (G, W)
  int w_shift;                    // as bs_magic, for W
  uint32_t w_magic;
  float sig2;                     // softmax scale * log2(e)
  uint8_t* out;
  int64_t o_s0b, o_s1b;
  float* lse;
  float* part_o;                  // [2 W][q_len * H][512] fp32: slot 2 w + 1 a request that begins in run w and goes on,
  float* part_lse;                // slot 2 w one that began before
  int2* span;                     // [W]: the request that begins in run w and goes on (-1: none), and how many runs have part of it
  uint32_t* err;
  int wait_us, stall;             // test aids, as in PagedParams
  uint32_t two16, two31;          // 2^16, 2^31
};

template <int NQ_>
struct Fp4Cfg {
  static_assert(NQ_ == 16 || NQ_ == 32 || NQ_ == 48 || NQ_ == 64, "columns per item");
  static constexpr int NQ = NQ_;
  static constexpr bool kWide = NQ >= 48;                         // hi and lo terms along K, one slot of k_pe (see above)
  static constexpr int kN = kWide ? NQ : 2 * NQ;                  // columns of a code product
  // keys of a tile: 128, or 96 where the columns leave two tiles of 128 no room
  static constexpr int kKeys = NQ == 64 ? 96 : 128, kSlot = kKeys * 128, kRopes = kWide ? 1 : 2;
  // terms of a weight, and how many of them stand side by side along N
  static constexpr int kTerms = 3, kStack = NQ == 16 ? 3 : NQ == 32 ? 2 : 1, kNO = kStack * NQ;
  // columns of a softmax thread, and the softmax warps: 16 (of 32 in 8 warps instead of 32 in 4: 32 requests of 1024 to 8192 keys
  // 54 -> 47 us), 32 of 64, where four times four warps would leave a thread 64 registers
  static constexpr int NC = NQ == 64 ? 32 : 16, kSW = 4 * (NQ / NC);
  static constexpr bool kSetRegs = NQ > 16;
  static constexpr int kLoadWarps = 8, kPvWarp = 2, kFirstSm = kSetRegs ? 4 : 3, kFirstLoad = kFirstSm + kSW;
  static constexpr int kThreads = 32 * (kFirstLoad + kLoadWarps);
  // The threads start with the same registers each, by eights; the warps of the issuers leave the others what those need
  static constexpr int kStartRegs = 65536 / kThreads / 8 * 8;
  static constexpr int kIssueRegs = 32, kSoftmaxRegs = NQ == 64 ? 120 : NQ == 48 ? 80 : 112, kLoadRegs = NQ == 32 ? 112 : 104;
  static_assert(!kSetRegs || (kSW % 4 == 0 && 4 * kIssueRegs + kSW * kSoftmaxRegs + kLoadWarps * kLoadRegs <= kThreads / 32 * kStartRegs), "registers of the launch");
  // (an increase below the start, or a decrease above it, is an illegal instruction)
  static_assert(!kSetRegs || (kIssueRegs <= kStartRegs && kSoftmaxRegs >= kStartRegs && kLoadRegs >= kStartRegs), "directions of the changes");
  static constexpr int kRing = 0;                                 // code tiles
  static constexpr int kRope = kRing + 8 * kSlot;                 // k_pe
  static constexpr int kQ = kRope + kRopes * kSlot;               // 4 x (2 NQ rows x 128 B): hi rows, then lo rows
  static constexpr int kQRope = kQ + 4 * 2 * NQ * 128;            // NQ x 128 B
  static constexpr int kP = kQRope + NQ * 128;                    // keys x 3 NQ
  static constexpr int kScale = kP + kKeys * kTerms * NQ;         // [2][128] fp32: 2^(K - 6), -1 masked
  static constexpr int kRed = kScale + 2 * kTile * 4;             // [2][NQ][4] max, [NQ][4] sum
  static constexpr int kColF = kRed + 3 * NQ * 4 * 4;             // [NQ] sig2 2^-e
  static constexpr int kMref = kColF + NQ * 4;                    // [NQ]
  static constexpr int kAlph = kMref + NQ * 4;                    // [NQ]
  static constexpr int kLut = kAlph + NQ * 4;                     // [16] x 8 B
  static constexpr int kBelow = kLut + 16 * 8;                    // [128] x 16 B
  static constexpr int kItems = kBelow + kTile * 16;
  static constexpr int kBar = kItems + kItemDepth * 32;
  static constexpr int kParts = 2;                    // commits of a tile's PV
  static constexpr int kNumBars = 4 + 2 + 2 + 2 * kParts + 4 + 2 * kItemDepth;
  static constexpr int kMisc = kBar + kNumBars * 8;
  static constexpr int kTotal = kMisc + 16;
  static constexpr int kAlloc = kTotal + 1024;
  static_assert(kAlloc <= kSmemLimit, "shared memory budget");
  static constexpr int kS = kN + NQ;                              // S: codes, then rope columns; two of them
  static constexpr int kTmemO = 2 * kS;                           // O_j at kTmemO + kNO j
  static constexpr int kTmemCols = kTmemO + 4 * kNO <= 256 ? 256 : 512;
  static_assert(kTmemO + 4 * kNO <= kTmemCols, "TMEM budget");
  // The query's lo terms: 16 times the rest where they have columns of their own, the rest itself where they add to
  // the hi terms' (rests below 2^-10 are lost).  The weights are 2^(kPExp + kTau) = 2^15.75 at most, of E5M2's 1.75 * 2^15.
  static constexpr float kLo = kWide ? 1.f : 16.f, kTau = 5.75f, kPExp = 10.f;
};

// The E4M3 bytes of eight codes: the magnitudes picked by permutes from the eight bytes of lut, with the codes as
// selectors, the sign bits by permutes from 0x00 and 0x80.  Permutes, logic and shifts share a pipe of half rate, the
// one that bounds the loaders, so the three right shifts are made by products (the high word of x 2^16 and x 2^31, whose
// factors come as arguments: a constant would become the shift again).
__device__ __forceinline__ uint2 fp4x8_to_e4m3(uint2 lut, uint32_t w, uint32_t two16, uint32_t two31) {
  const uint32_t mag = w & 0x77777777u, sgn = __umulhi(w, two31) & 0x44444444u;
  uint32_t m0, m1, s0, s1;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(m0) : "r"(lut.x), "r"(lut.y), "r"(mag));
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(m1) : "r"(lut.x), "r"(lut.y), "r"(__umulhi(mag, two16)));
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(s0) : "r"(0u), "r"(0x80u), "r"(sgn));
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(s1) : "r"(0u), "r"(0x80u), "r"(__umulhi(sgn, two16)));
  return make_uint2(m0 | s0, m1 | s1);
}

// One lane of a warp that goes along as a whole: which, the hardware says.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xFFFFFFFF;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
  return r != 0;
}
// The products and commits of mla_ptx.cuh, issued where `on`.
__device__ __forceinline__ void mma_f8_if(bool on, uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(id), "r"(acc), "r"(on ? 1u : 0u)
      : "memory");
}
__device__ __forceinline__ void mma_f16_if(bool on, uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(id), "r"(acc), "r"(on ? 1u : 0u)
      : "memory");
}
__device__ __forceinline__ void mma_commit_if(bool on, uint64_t* bar) {
  asm volatile(
      "{\n .reg .pred q;\n setp.ne.b32 q, %1, 0;\n"
      " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(smem_u32(bar)),
      "r"(on ? 1u : 0u)
      : "memory");
}

// A wait that is in a hurry: an issuer's, polled.
__device__ __forceinline__ bool spin_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
  uint64_t t0 = 0;
  for (uint32_t i = 1;; ++i) {
    if (mbar_test_wait(bar, parity)) return true;
    if ((i & 255u) == 0) {
      if (*abort_flag) return false;
      const uint64_t now = globaltimer();
      if (t0 == 0) t0 = now;
      if (now - t0 > wait_limit_ns(abort_flag)) {
        *abort_flag = 2;
        return false;
      }
    }
  }
}
// The same by one lane of a warp.
__device__ __forceinline__ bool warp_spin(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
  bool w = true;
  if ((threadIdx.x & 31) == 0) w = spin_wait(bar, parity, abort_flag);
  w = __shfl_sync(0xFFFFFFFFu, w ? 1 : 0, 0) != 0;
  __syncwarp();
  return w;
}
// A group of warps waits through its first one, the others at a hardware barrier: a warp that polls takes issue slots from
// the others (polled by every softmax and loader warp, the waits were 4500 of 10000 instructions a tile).  Every thread of the group leaves with the same answer.
// `so_far`: false where a wait of this warp's own ran out before, which ends the group.
__device__ __forceinline__ bool group_wait(bool first, uint32_t id, uint32_t threads, uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                                           bool so_far = true) {
  bool w = so_far;
  if (first && w) w = warp_spin(bar, parity, abort_flag);
  return named_bar_and(id, threads, w);
}
// A wait that is in no hurry.
__device__ __forceinline__ bool slow_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
  const uint64_t t0 = globaltimer();
  while (!mbar_test_wait(bar, parity)) {
    __nanosleep(500);
    if (*abort_flag) return false;
    // (work items last as long as they last: this is no pipeline's wait)
    if (globaltimer() - t0 > 10 * kWaitNs) {
      *abort_flag = 2;
      return false;
    }
  }
  return true;
}

template <int NQ>
__global__ void __launch_bounds__(Fp4Cfg<NQ>::kThreads, 1) mla_fp4_kernel(const __grid_constant__ Fp4Params p) {
  using C = Fp4Cfg<NQ>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);      // (known to be shared: no generic accesses)
  uint8_t* ring = smem + C::kRing;
  uint8_t* qs = smem + C::kQ;
  uint8_t* qr = smem + C::kQRope;
  uint8_t* ps = smem + C::kP;
  float* scl = reinterpret_cast<float*>(smem + C::kScale);        // [2][128]
  float* red_m = reinterpret_cast<float*>(smem + C::kRed);        // [2][NQ][4]
  float* red_l = red_m + 2 * NQ * 4;                              // [NQ][4]
  float* colf = reinterpret_cast<float*>(smem + C::kColF);
  float* mref = reinterpret_cast<float*>(smem + C::kMref);
  float* alph = reinterpret_cast<float*>(smem + C::kAlph);
  uint2* lut = reinterpret_cast<uint2*>(smem + C::kLut);
  WorkItem* items = reinterpret_cast<WorkItem*>(smem + C::kItems);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kBar);
  uint64_t* full = bars;                  // [2][2] the loader warps have written two code tiles, and k_pe and the scales with one of them
  uint64_t* s_full = full + 4;            // [2] QK done
  uint64_t* s_free = s_full + 2;          // [2] the softmax has read S
  uint64_t* pv_part = s_free + 2;         // [2][kParts] PV of the value tiles done
  uint64_t* p_full = pv_part + 2 * C::kParts;      // P is written (one arrival per softmax warp)
  uint64_t* q_full = p_full + 1;
  uint64_t* fin = p_full + 2;
  uint64_t* fin_pv = p_full + 3;
  uint64_t* item_full = p_full + 4;
  uint64_t* item_empty = item_full + kItemDepth;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kMisc + 4);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  TL_DECL;

  if (tid == 0) TL(0, 1);
  // the merge may be scheduled now; it waits for this grid to complete
  if (tid == 0) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (warp == 0) {
    for (int i = lane; i < C::kNumBars; i += 32) {
      uint32_t count = 1;
      if (i < 4) count = C::kLoadWarps;
      if (&bars[i] == p_full) count = C::kSW;                                // the softmax warps
      if (&bars[i] >= item_empty) count = 3 + C::kLoadWarps;                 // the roles
      mbar_init(&bars[i], count);
    }
    if (lane == 0) {
      *abort_flag = 0;
      abort_flag[1] = p.wait_us;
    }
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, C::kTmemCols);
    tmem_relinquish();
  }
  if (warp == 0 && lane < 16) {
    // magnitudes 0, .5, 1, 1.5 | 2, 3, 4, 6 times 2^(6 - lane) in E4M3: exact down to 2^-9, zero below
    // (entry 15 is all zeros)
    uint32_t w[2] = {0u, 0u};
    if (lane < 15) {
      const float mag[8] = {0.f, .5f, 1.f, 1.5f, 2.f, 3.f, 4.f, 6.f};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t b = __nv_cvt_float_to_fp8(mag[i] * pow2i(6 - lane), __NV_SATFINITE, __NV_E4M3);
        w[i >> 2] |= b << (8 * (i & 3));
      }
    }
    lut[lane] = make_uint2(w[0], w[1]);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // launched as a programmatic dependent of the previous kernel in the stream: its writes (the query, the
  // cache) are visible past this wait
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (tid == 0) TL(0, 2);

  // (the registers are set inside the roles' branches: the compiler gives a branch what it sets)
  if (warp < C::kFirstSm) {
    if constexpr (C::kSetRegs) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kIssueRegs));
    if (warp == 0) {
      // ------------------------------------------------------------------ scheduler
      auto tiles_of = [&](int b) -> int64_t { return static_cast<int64_t>((static_cast<uint32_t>(max(p.seq_lens[b], 0)) + (C::kKeys - 1)) / C::kKeys); };
      // a lane sums a run of requests; the lane that holds this CTA's first tile looks for its request
      const int per_lane = (p.B + 31) / 32, b0 = min(lane * per_lane, p.B), b1 = min(b0 + per_lane, p.B);
      int64_t sum = 0;
#pragma unroll 4
      for (int b = b0; b < b1; ++b) sum += tiles_of(b);
      int64_t end = sum;
#pragma unroll
      for (int o = 1; o < 32; o *= 2) {
        const int64_t v = __shfl_up_sync(0xFFFFFFFFu, end, o);
        if (lane >= o) end += v;
      }
      const int64_t total = __shfl_sync(0xFFFFFFFFu, end, 31);
      // tiles / W, rounded up (divided by way of the product where 32 bits are enough: a lone lane's division is 0.3 us)
      const int64_t up = total + p.W - 1;
      const int64_t run = total <= 0                  ? 1
                          : up < (int64_t(1) << 31) ? static_cast<int64_t>(__umulhi(2u * static_cast<uint32_t>(up), p.w_magic) >> p.w_shift)
                                                    : up / p.W;
      const int w = static_cast<int>(blockIdx.y), g = static_cast<int>(blockIdx.x);
      const int64_t lo = min(w * run, total), hi = min(lo + run, total);
      int b = p.B;
      int64_t t0 = end - sum;      // first tile of request b
      if (lo < hi && t0 <= lo && lo < end) {
        b = b0;
        for (int64_t n; (n = tiles_of(b)) <= lo - t0; ++b) t0 += n;
      }
      const uint32_t who = __ballot_sync(0xFFFFFFFFu, b < p.B);
      const int src = who ? __ffs(who) - 1 : 0;
      b = __shfl_sync(0xFFFFFFFFu, b, src);
      t0 = __shfl_sync(0xFFFFFFFFu, t0, src);
      if (lane == 0) TL(0, 3);
      int64_t t = lo, on_t = 0;      // last tile of the request that goes on
      int on_b = -1;
      for (int nitem = 0;; ++nitem) {
        WorkItem it{};
        it.b = -1;
        if (t < hi) {
          const int64_t n = tiles_of(b);
          it.b = b;
          it.g = g;
          it.L = p.seq_lens[b];
          it.ntiles = static_cast<int>(min(hi, t0 + n) - t);
          it.k0 = static_cast<int>((t - t0) * C::kKeys);
          it.n = static_cast<int>(min(static_cast<int64_t>(it.L) - it.k0, static_cast<int64_t>(it.ntiles) * C::kKeys));
          it.pad = it.ntiles == n;                      // the whole request: final
          it.s = 2 * w + (t == t0 ? 1 : 0);
          if (t == t0 && it.ntiles < n) on_t = t0 + n - 1, on_b = b;
          t += it.ntiles;
          if (t < hi) {      // the next request with keys, 32 at a time (a padded batch has many without)
            t0 = t;
            uint32_t some = 0;
            for (++b; b < p.B; b += 32) {
              some = __ballot_sync(0xFFFFFFFFu, b + lane < p.B && p.seq_lens[b + lane] > 0);
              if (some) break;
            }
            if (some) b += __ffs(some) - 1;
          }
        }
        const int k = nitem % kItemDepth;
        bool w_ok = true;
        if (lane == 0 && nitem >= kItemDepth) w_ok = slow_wait(&item_empty[k], static_cast<uint32_t>((nitem / kItemDepth) - 1) & 1u, abort_flag);
        if (!__all_sync(0xFFFFFFFFu, w_ok)) break;
        if (lane == 0) {
          items[k] = it;
          mbar_arrive(&item_full[k]);
        }
        if (it.b < 0) break;
      }
      if (lane == 0 && g == 0) p.span[w] = make_int2(on_b, on_b < 0 ? 0 : static_cast<int>(on_t / run) - w + 1);
      __syncwarp();
      // requests without keys: zeros, every W-th one
      for (int z = w; z < p.B; z += p.W) {
        if (p.seq_lens[z] > 0) continue;
        for (int c = g * NQ; c < min(g * NQ + NQ, p.cols); ++c) {
          const int64_t r = static_cast<int64_t>(z) * p.q_len + c / p.H;
          uint8_t* o = p.out + r * p.o_s0b + static_cast<int64_t>(c % p.H) * p.o_s1b;
          for (int d = lane; d < kLora; d += 32) *reinterpret_cast<uint16_t*>(o + 2 * d) = 0;
          if (p.lse && lane == 0) p.lse[r * p.H + c % p.H] = -CUDART_INF_F;
        }
      }
    } else if (warp == 1) {
      // ------------------------------------------------------------------ QK issuer
      // (the warp goes along as a whole, so that the descriptors stay in uniform registers; one lane issues)
      {
        const bool one = elect_one();
        const uint64_t dK0 = smem_desc(smem_u32(ring), 16, 1024, kSwizzle128B);
        const uint64_t dR0 = smem_desc(smem_u32(smem + C::kRope), 16, 1024, kSwizzle128B);
        const uint64_t dQ0 = smem_desc(smem_u32(qs), 16, 1024, kSwizzle128B);
        const uint64_t dQr = smem_desc(smem_u32(qr), 16, 1024, kSwizzle128B);
        constexpr uint32_t kIdNope = idesc_e4m3(128, C::kN, 0, 0);
        constexpr uint32_t kIdRope = idesc_f16(128, NQ, 1, 1, 0, 0);
        bool ok = true;
        int nit = 0, nq = 0, g = 0;
        while (ok) {
          const int k = nit % kItemDepth;
          if (!warp_spin(&item_full[k], (nit / kItemDepth) & 1, abort_flag)) break;
          const WorkItem it = items[k];
          __syncwarp();
          if (one) mbar_arrive(&item_empty[k]);
          ++nit;
          if (it.b < 0) break;
          if (!warp_spin(q_full, nq & 1, abort_flag)) break;
          ++nq;
          for (int t = 0; t < it.ntiles && ok; ++t) {
            const int gt = g + t, h = gt & 1;
            if (gt >= 2 && !warp_spin(&s_free[h], static_cast<uint32_t>((gt - 2) >> 1) & 1u, abort_flag)) ok = false;
            if (!ok) break;
            if (lane == 0) TL(1, 1);
            const uint32_t dS = tmem + h * C::kS;
            const uint32_t use = static_cast<uint32_t>(gt >> 1) & 1u;
            // as the loaders finish the slots: two code tiles, then the other two; k_pe comes with the first ones, or last
            // where it has one slot only
            auto rope_product = [&]() {
              const uint64_t aK = desc_add(dR0, static_cast<uint32_t>((gt % C::kRopes) * (C::kSlot >> 4)));
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                mma_f16_if(one, dS + C::kN, desc_add(aK, (kk * 32) >> 4), desc_add(dQr, (kk * 32) >> 4), kIdRope, kk > 0 ? 1u : 0u);
            };
#pragma unroll 1
            for (int b = 0; b < 4 && ok; ++b) {
              if ((b & 1) == 0) {
                ok = __all_sync(0xFFFFFFFFu, spin_wait(&full[2 * h + (b >> 1)], use, abort_flag));
                if (!ok) break;
                tc_fence_after();
                if (lane == 0) TL(1, 2);
                if (b == (C::kRopes == 1 ? 2 : 0)) rope_product();
              }
              const uint64_t aK = desc_add(dK0, static_cast<uint32_t>((4 * h + b) * (C::kSlot >> 4)));
              const uint64_t bQ = desc_add(dQ0, static_cast<uint32_t>(b * (2 * NQ * 128 >> 4)));
#pragma unroll
              for (int kk = 0; kk < 4; ++kk) {
                mma_f8_if(one, dS, desc_add(aK, (kk * 32) >> 4), desc_add(bQ, (kk * 32) >> 4), kIdNope, (b | kk) ? 1u : 0u);
                if constexpr (C::kWide) mma_f8_if(one, dS, desc_add(aK, (kk * 32) >> 4), desc_add(bQ, (NQ * 128 + kk * 32) >> 4), kIdNope, 1u);
              }
            }
            if (!ok) break;
            mma_commit_if(one, &s_full[h]);
            if (lane == 0) TL(1, 3);
          }
          g += it.ntiles;
        }
        mma_commit_if(one, fin);
        volatile int no_abort[2] = {0, 0};
        mbar_wait(fin, 0, no_abort);
      }
      __syncwarp();
    } else if (warp == C::kPvWarp) {
      // ------------------------------------------------------------------ PV issuer
      {
        const bool one = elect_one();
        const uint64_t dV0 = smem_desc(smem_u32(ring), C::kSlot, 1024, kSwizzle128B);
        const uint64_t dP0 = smem_desc(smem_u32(ps), C::kTerms * NQ * 8, 128, kSwizzleNone);
        // (B, the weights, in E5M2)
        constexpr uint32_t kIdStack = idesc_e4m3(128, C::kNO, 1, 1) | (1u << 10), kIdTerm = idesc_e4m3(128, NQ, 1, 1) | (1u << 10);
        bool ok = true;
        int nit = 0, g = 0;
        while (ok) {
          const int k = nit % kItemDepth;
          if (!warp_wait(&item_full[k], (nit / kItemDepth) & 1, abort_flag)) break;
          const WorkItem it = items[k];
          __syncwarp();
          if (one) mbar_arrive(&item_empty[k]);
          ++nit;
          if (it.b < 0) break;
          for (int t = 0; t < it.ntiles; ++t) {
            const int gt = g + t;
            if (!__all_sync(0xFFFFFFFFu, spin_wait(p_full, static_cast<uint32_t>(gt) & 1u, abort_flag))) {
              ok = false;
              break;
            }
            tc_fence_after();
            if (lane == 0) TL(2, 1);
            const uint32_t acc0 = t == 0 ? 0u : 1u;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint64_t aV = desc_add(dV0, static_cast<uint32_t>((4 * (gt & 1) + j) * (C::kSlot >> 4)));
#pragma unroll
              for (int kk = 0; kk < C::kKeys / 32; ++kk) {
                // (32 keys are four groups of eight; the terms beyond the stacked ones add to the last of those)
                const uint32_t dO = tmem + C::kTmemO + C::kNO * j, at = kk * 4 * C::kTerms * NQ * 8;
                mma_f8_if(one, dO, desc_add(aV, (kk * 4096) >> 4), desc_add(dP0, at >> 4), kIdStack, kk > 0 ? 1u : acc0);
#pragma unroll
                for (int x = C::kStack; x < C::kTerms; ++x)
                  mma_f8_if(one, dO + C::kNO - NQ, desc_add(aV, (kk * 4096) >> 4), desc_add(dP0, (at + x * NQ * 8) >> 4), kIdTerm, 1u);
              }
              if ((j + 1) % (4 / C::kParts) == 0) mma_commit_if(one, &pv_part[(gt & 1) * C::kParts + j / (4 / C::kParts)]);
            }
            if (lane == 0) TL(2, 2);
          }
          g += it.ntiles;
        }
        mma_commit_if(one, fin_pv);
        volatile int no_abort[2] = {0, 0};
        mbar_wait(fin_pv, 0, no_abort);
      }
      __syncwarp();
    }
  } else if (warp >= C::kFirstLoad) {
    if constexpr (C::kSetRegs) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kLoadRegs));
    // ------------------------------------------------------------------ loaders
    // Warp w owns keys KW w .. KW w + KW - 1 of every tile.  Lane k < 16 finds key k's record and has its exponents; the
    // codes and k_pe are loaded eight lanes a key, 128 bytes in a row: lane 16 a + 8 b + 4 c + u takes, of keys 4 m + 2 a + c, the
    // groups 8 h + 4 b + u (code tile 2 h + b) and a piece of k_pe.  A quarter of the warp so stores an even and the next odd
    // row, whose columns the swizzle keeps apart.  (Four lanes a key, 64 bytes in a row: a third more time in the loads.)
    constexpr int KW = C::kKeys / C::kLoadWarps, KM = KW / 4;      // 16 or 12
    static_assert(KW <= 16 && KW % 4 == 0, "a lane of half a warp for each key, four keys a step");
    const int w = warp - C::kFirstLoad;
    const int u = lane & 3, kb = (lane >> 3) & 1, key0 = 2 * (lane >> 4) + ((lane >> 2) & 1);      // key of m: 4 m + key0
    uint4* below = reinterpret_cast<uint4*>(smem + C::kBelow) + 16 * w;                             // [key] 16 bytes: exponents below K
    struct Cursor {
      const int32_t* table;      // the request's block ids; null: past the last tile
      int kp, end, left;         // this lane's key of the tile, the item's end, tiles after this one
    };
    // ok is every loader warp's alike.  mine: this warp's waits have not run out; one of them may, at the edge of its limit, where
    // another warp's on the same barrier does not: the warp leaves its tiles and goes on to the barrier of the next item, where
    // all of them stop.
    int nit = 0;
    bool ok = true, mine = true;
    auto next_item = [&](Cursor& c) {
      const int k = nit % kItemDepth;
      if (!group_wait(w == 0, 2, 32 * C::kLoadWarps, &item_full[k], (nit / kItemDepth) & 1, abort_flag, mine)) {
        ok = false;
        c.table = nullptr;
        return;
      }
      const int b = items[k].b, k0 = items[k].k0, n = items[k].n, ntiles = items[k].ntiles;
      __syncwarp();
      if (lane == 0) mbar_arrive(&item_empty[k]);
      ++nit;
      c.table = b < 0 ? nullptr : p.block_table + static_cast<int64_t>(b) * p.bt_stride;
      c.kp = k0 + KW * w + lane;
      c.end = k0 + n;
      c.left = ntiles - 1;
    };
    auto advance = [&](Cursor& c) {
      if (!c.table) return;
      c.kp += C::kKeys;
      if (--c.left < 0) next_item(c);
    };
    uint32_t errbits = 0;
    // this lane's key of a tile: block id (as read: looked at a tile later, by found; kNoKey: there is none) and place there
    constexpr int kNoKey = -0x7FFFFFFF;
    struct Ask {
      int id, at;
    };
    auto ask = [&](const Cursor& c) -> Ask {
      Ask a{kNoKey, 0};
      if (c.table && lane < KW && c.kp < c.end) {
        const int col = static_cast<int>(__umulhi(2u * static_cast<uint32_t>(c.kp), p.bs_magic) >> p.bs_shift);      // kp / block_size
        a.at = c.kp - col * p.block_size;
        a.id = __ldg(c.table + col);
      }
      return a;
    };
    auto found = [&](const Ask& a) -> const uint8_t* {      // null: no such key or block
      const bool good = static_cast<uint32_t>(a.id) < p.num_blocks;
      if (!good && a.id != kNoKey) errbits |= 2u;
      return good ? p.kv + static_cast<uint64_t>(static_cast<uint32_t>(a.id)) * p.blk_stride +
                        static_cast<uint64_t>(static_cast<uint32_t>(a.at)) * p.ent_stride
                  : nullptr;
    };
    // A tile's records are asked of memory into L2 one tile before its loads: the loads of a tile, issued together
    // when the registers of the tile before are free, then find them there.  (Loads issued register by
    // register between the conversions ran at a load's whole latency a step: the few scoreboards of a warp
    // are shared by old and new loads.)
    auto prefetch = [&](const uint8_t* r, int at) {
      if (!r) return;
      if (p.ent_stride == kFp4Entry) {      // one for the records that lie together (one a key takes the loaders longer)
        if (lane == 0 || at == 0) bulk_prefetch_l2(r, min(KW - lane, p.block_size - at) * kFp4Entry);
      } else {
        bulk_prefetch_l2(r, kFp4Entry);
      }
    };
    // k_pe's piece of this lane: the halves of 64 bytes in the other order in odd rows (whose columns the swizzle takes to
    // the even rows' then)
    const int piece = u + 4 * (kb ^ (key0 & 1));
    uint4 code[KM][2], rope[KM], ex = make_uint4(0, 0, 0, 0);
    bool live = false;      // lane k: key k is there
    auto load_tile = [&](const uint8_t* own) {
      live = own != nullptr;
      ex = live ? __ldg(reinterpret_cast<const uint4*>(own + kFp4Exps)) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int m = 0; m < KM; ++m) {
        const uint8_t* r = reinterpret_cast<const uint8_t*>(__shfl_sync(0xFFFFFFFFu, reinterpret_cast<unsigned long long>(own), 4 * m + key0));
        if (r) {
          rope[m] = __ldg(reinterpret_cast<const uint4*>(r + kFp4Rope) + piece);
#pragma unroll
          for (int h = 0; h < 2; ++h) code[m][h] = __ldg(reinterpret_cast<const uint4*>(r) + 8 * h + 4 * kb + u);
        } else {      // an absent key is all zeros
          rope[m] = code[m][0] = code[m][1] = make_uint4(0, 0, 0, 0);
        }
      }
    };
    Cursor c{};
    next_item(c);
    if (p.stall && ok) {
      // test aid: write nothing, so that the other roles' waits run out under the launch's short limit
      ok = false;
    }
    // tile 0 in the registers, records of tile 1, block ids of tile 2.  (Behind tile t the loaders look at tile t + 3, which may be
    // three items ahead: the item kItemDepth before that one has to be done without their next tile.)
    static_assert(kItemDepth > 3, "the loaders would wait for themselves");
    bool have = c.table != nullptr, have1, have2;
    load_tile(found(ask(c)));
    advance(c);
    have1 = c.table != nullptr;
    Ask asked = ask(c);
    const uint8_t* next = found(asked);
    prefetch(next, asked.at);
    advance(c);
    have2 = c.table != nullptr;
    asked = ask(c);
    // row 4 m + key0 of this warp's in a slot, and there column 2 u (column 2 u + 1 is 16 away, by exclusive or) and k_pe's
    // piece; with m the swizzle's row changes by four
    const int row0 = KW * w + key0;
    const uint32_t o0 = row0 * 128 + (((2 * u) ^ (row0 & 7)) << 4), r0 = row0 * 128 + ((piece ^ (row0 & 7)) << 4);
    for (int gt = 0; ok && have; ++gt) {
      const int h = gt & 1;
      const uint32_t used = static_cast<uint32_t>((gt - 2) >> 1) & 1u;      // phase of tile gt - 2
      // the slots of code tiles 2 i and 2 i + 1: free after the PV that read what lay there
      auto free_slots = [&](int i) -> bool { return gt < 2 || warp_spin(&pv_part[h * C::kParts + i], used, abort_flag); };
      uint8_t* tile = ring + 4 * h * C::kSlot;
      auto written = [&](int slot) {
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[2 * h + slot]);
      };
      if (w == 0 && lane == 0) TL(4, 1);
      // the record's largest exponent, at least 2^-60: what is smaller than 2^-74 reads as zero, and the sums over
      // keys stay inside fp32
      uint32_t K;
      {
        const uint32_t word[4] = {ex.x, ex.y, ex.z, ex.w};
        uint32_t top = 0u;      // of the even and the odd bytes
#pragma unroll
        for (int i = 0; i < 4; ++i) top = __vmaxu2(top, __vmaxu2(word[i] & 0x00FF00FFu, (word[i] >> 8) & 0x00FF00FFu));
        K = max(max(top & 0xFFFFu, top >> 16), 67u);
        const uint32_t K4 = K * 0x01010101u;      // (no byte of K4 - word borrows)
        if (lane < KW) below[lane] = make_uint4(K4 - ex.x, K4 - ex.y, K4 - ex.z, K4 - ex.w);
        __syncwarp();
      }
      // k_pe and the scale.  Of two slots of k_pe this tile's is free after QK of tile gt - 2, and so after its PV; the only one
      // after QK of tile gt - 1.  The scale of tile gt - 2 was read before its PV.
      auto put_rope = [&]() {
        uint8_t* at = smem + C::kRope + (gt % C::kRopes) * C::kSlot;
#pragma unroll
        for (int m = 0; m < KM; ++m)
          *reinterpret_cast<uint4*>(at + 512 * m + (r0 ^ ((m & 1) << 6))) = rope[m];
        if (lane < KW)      // exponent 255: a NaN in the record; -1: no such key
          scl[h * kTile + KW * w + lane] = !live ? -1.f : K == 255u ? CUDART_NAN_F : __uint_as_float((K - 6u) << 23);
      };
      const uint8_t* low = reinterpret_cast<const uint8_t*>(below + key0) + 4 * kb + u;      // of key 4 m + key0 64 m on
      auto convert = [&](int i, int m, uint4 (&v)[2]) {
        const uint2 l2 = lut[min(static_cast<uint32_t>(low[64 * m + 8 * i]), 15u)];
        const uint4 x = code[m][i];
        const uint2 a0 = fp4x8_to_e4m3(l2, x.x, p.two16, p.two31), a1 = fp4x8_to_e4m3(l2, x.y, p.two16, p.two31);
        const uint2 a2 = fp4x8_to_e4m3(l2, x.z, p.two16, p.two31), a3 = fp4x8_to_e4m3(l2, x.w, p.two16, p.two31);
        v[0] = make_uint4(a0.x, a0.y, a1.x, a1.y);
        v[1] = make_uint4(a2.x, a2.y, a3.x, a3.y);
      };
      auto put = [&](int i) {
#pragma unroll
        for (int m = 0; m < KM; ++m) {
          uint4 v[2];
          convert(i, m, v);
          uint8_t* at = tile + (2 * i + kb) * C::kSlot + 512 * m;
          const uint32_t o = o0 ^ ((m & 1) << 6);
          *reinterpret_cast<uint4*>(at + o) = v[0];
          *reinterpret_cast<uint4*>(at + (o ^ 16u)) = v[1];
        }
        written(i);
      };
      if (!(mine = free_slots(0))) break;
      if (w == 0 && lane == 0) TL(4, 2);
      if constexpr (C::kRopes == 2) put_rope();
      put(0);
      if (w == 0 && lane == 0) TL(4, 4);
      mine = free_slots(1);
      if constexpr (C::kRopes == 1) {
        mine = mine && (gt < 1 || warp_spin(&s_full[h ^ 1], static_cast<uint32_t>((gt - 1) >> 1) & 1u, abort_flag));
        if (mine) put_rope();
      }
      if (!mine) break;
      if (w == 0 && lane == 0) TL(4, 5);
      put(1);
      if (w == 0 && lane == 0) TL(4, 3);
      // (the block ids are looked at before new loads are on their way, whose scoreboards they may share)
      const uint8_t* after = found(asked);
      prefetch(after, asked.at);
      load_tile(next);
      advance(c);
      asked = ask(c);
      next = after;
      have = have1;
      have1 = have2;
      have2 = c.table != nullptr;
    }
    if (!mine)
      while (c.table) advance(c);
    errbits = __reduce_or_sync(0xFFFFFFFFu, errbits);
    if (lane == 0 && errbits) set_device_error(p.err, errbits);
  } else {
    if constexpr (C::kSetRegs) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kSoftmaxRegs));
    // ------------------------------------------------------------------ softmax, query, epilogue
    constexpr int NT = 32 * C::kSW, NC = C::NC;
    const int quad = warp & 3;
    const int row = quad * 32 + lane;           // key of the tile (S^T lane), latent of a block (O^T lane)
    const int stid = tid - 32 * C::kFirstSm;
    const int c0 = (stid >> 7) * NC;            // first column of this thread
    const uint32_t tl = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    // w = 2^(s' - m + kPExp) <= 2^(kTau + kPExp).  mref holds m - kPExp.
    constexpr float kTau = C::kTau, kPExp = C::kPExp;
    // the query of an item: thread (c = stid / 8, part = stid % 8) takes elements 64 part .. + 63 of a column
    auto prep_query = [&](const WorkItem& qi) {
#pragma unroll 1
      for (int c = stid >> 3; c < NQ; c += NT / 8) {
        const int part = stid & 7;
        const int cg = qi.g * NQ + c;
        const bool live = cg < p.cols;
        const uint8_t* qrow = live ? p.q + (static_cast<int64_t>(qi.b) * p.q_len + cg / p.H) * p.q_s0b + (cg % p.H) * p.q_s1b
                                   : nullptr;
        uint4 v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = live ? *reinterpret_cast<const uint4*>(qrow + part * 128 + 16 * i) : make_uint4(0, 0, 0, 0);
        const uint4 rv = live ? *reinterpret_cast<const uint4*>(qrow + 1024 + 16 * part) : make_uint4(0, 0, 0, 0);
        uint32_t amax = 0;      // of the magnitudes' bits: a NaN is the largest
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t wv[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) amax = max(max(amax, (wv[e] << 16) & 0x7FFF0000u), wv[e] & 0x7FFF0000u);
        }
        amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
        amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
        amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 4));
        const bool finite = amax < 0x7F800000u;
        const int e = finite ? e4m3_fit_exponent(__uint_as_float(amax)) : 0;
        const float sc = pow2i(e);
        if (part == 0) colf[c] = finite ? p.sig2 * pow2i(-e) : CUDART_NAN_F;
        uint8_t* base = qs + (part >> 1) * (2 * NQ * 128);
#pragma unroll
        for (int i = 0; i < 4; ++i) {     // 16 elements per 16-byte chunk of hi and of lo
          uint32_t hw[4], lw[4];
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const uint4 a = v[2 * i + (y >> 1)];
            const uint32_t w0 = (y & 1) ? a.z : a.x, w1 = (y & 1) ? a.w : a.y;
            const float x0 = __uint_as_float(w0 << 16) * sc, x1 = __uint_as_float(w0 & 0xFFFF0000u) * sc;
            const float x2 = __uint_as_float(w1 << 16) * sc, x3 = __uint_as_float(w1 & 0xFFFF0000u) * sc;
            const uint32_t h01 = e4m3x2_sat(x0, x1), h23 = e4m3x2_sat(x2, x3);
            const float2 f01 = e4m3x2_to_float2(h01), f23 = e4m3x2_to_float2(h23);
            hw[y] = h01 | (h23 << 16);
            lw[y] = e4m3x2_sat(C::kLo * (x0 - f01.x), C::kLo * (x1 - f01.y)) |
                    (e4m3x2_sat(C::kLo * (x2 - f23.x), C::kLo * (x3 - f23.y)) << 16);
          }
          const int chunk = (part & 1) * 4 + i;
          *reinterpret_cast<uint4*>(base + sw128(c, chunk)) = make_uint4(hw[0], hw[1], hw[2], hw[3]);
          *reinterpret_cast<uint4*>(base + sw128(NQ + c, chunk)) = make_uint4(lw[0], lw[1], lw[2], lw[3]);
        }
        *reinterpret_cast<uint4*>(qr + sw128(c, part)) = rv;
      }
      fence_proxy_async_smem();
      named_bar_sync(1, NT);
      if (stid == 0) mbar_arrive(q_full);
    };
    int nit = 0, g = 0;
    bool ok = true, failed = false;      // failed: a wait of this thread's warp ran out in the tile before
    bool q_ready = false;                // the item's query was prepared during the one before
    while (ok) {
      const int k = nit % kItemDepth;
      bool w = group_wait(warp == C::kFirstSm, 1, NT, &item_full[k], (nit / kItemDepth) & 1, abort_flag);
      const WorkItem it = items[k];
      ++nit;
      if (stid < NQ) mref[stid] = -3e38f;         // no reference yet: every logit passes it, and -inf - m is no NaN
      if (!w || it.b < 0) break;
      if (stid == 0) TL(3, 20);
      if (!q_ready) prep_query(it);
      if (stid == 0) TL(3, 21);
      q_ready = false;
      const int cgb = it.g * NQ + c0;             // global column of this thread's first
      float l_part[NC];
#pragma unroll
      for (int c = 0; c < NC; ++c) l_part[c] = 0.f;
      // s' of this thread's key for its columns, masked; ks: the key's 2^(K - 6)
      auto load_s = [&](float (&s)[NC], int gt, int t, float ks) {
        const uint32_t ts = tl + (gt & 1) * C::kS + c0;
        const int kpos = it.k0 + t * C::kKeys + row;
        const bool rv = kpos < it.k0 + it.n && !(ks < 0.f);
        // (the rows of absent keys are zeros: 0 * 0 - inf)
        const float kexp = rv ? static_cast<float>(static_cast<int>(__float_as_uint(ks) >> 23) - 127) : -CUDART_INF_F;
        const float km = rv ? ks : 0.f;
#pragma unroll
        for (int c1 = 0; c1 < NC; c1 += 16) {
          float a[16], r[16];
          tmem_ld16(ts + c1, a);
          if constexpr (!C::kWide) {
            tmem_ld16(ts + NQ + c1, r);
            tmem_ld_wait();
#pragma unroll
            for (int c = 0; c < 16; ++c) a[c] = fmaf(r[c], 0.0625f, a[c]);
          }
          tmem_ld16(ts + C::kN + c1, r);
          tmem_ld_wait();
#pragma unroll
          for (int c = 0; c < 16; c += 4) {
            const float4 f4 = *reinterpret_cast<const float4*>(colf + c0 + c1 + c);
            const float ff[4] = {f4.x, f4.y, f4.z, f4.w};
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              s[c1 + c + y] = fmaf(a[c + y], ff[y] * km, fmaf(r[c + y], p.sig2, kexp));
              if (C::kKeys < kTile && !rv) s[c1 + c + y] = -CUDART_INF_F;      // (rows past the tile are anything)
            }
          }
        }
        // spec-verify: query token qi sees keys up to L - q_len + qi
        const int dq = kpos - it.L + p.q_len;
        if (rv && dq > 0) {
#pragma unroll
          for (int c = 0; c < NC; ++c)
            if ((cgb + c) / p.H < dq) s[c] = -CUDART_INF_F;
        }
      };
      for (int t = 0; t < it.ntiles; ++t) {
        const int gt = g + t;
        // (the tile's scales, written with its first slots, are there long before S)
        w = true;
        if (warp == C::kFirstSm)
          w = warp_spin(&full[2 * (gt & 1) + (C::kRopes == 1 ? 1 : 0)], static_cast<uint32_t>(gt >> 1) & 1u, abort_flag) &&
              warp_spin(&s_full[gt & 1], static_cast<uint32_t>(gt >> 1) & 1u, abort_flag);
        w = named_bar_and(1, NT, w);
        tc_fence_after();
        const float ks = row < C::kKeys ? scl[(gt & 1) * kTile + row] : -1.f;
        if (stid == 0) TL(3, 1);
        float d[NC];              // s', then s' - m + kPExp, then the weights
        auto against = [&]() {
#pragma unroll
          for (int c = 0; c < NC; c += 4) {
            const float4 m4 = *reinterpret_cast<const float4*>(mref + c0 + c);
            d[c] -= m4.x;
            d[c + 1] -= m4.y;
            d[c + 2] -= m4.z;
            d[c + 3] -= m4.w;
          }
        };
        // (an item begins without a reference; more columns have no registers for the shorter way: 1030 -> 1070 us)
        bool rare = NQ == 16 && t == 0;
        if (!rare) {
          load_s(d, gt, t, ks);
          if (stid == 0) TL(3, 2);
          against();
          float most = d[0];
#pragma unroll
          for (int c = 1; c < NC; ++c) most = fmaxf(most, d[c]);
          // (the weights for the reference as it is, while the other warps come to the barrier)
#pragma unroll
          for (int c = 0; c < NC; ++c) d[c] = ex2(d[c]);
          tc_fence_before();
          rare = named_bar_or(1, NT, most > kTau + kPExp || !w || failed);
        }
        bool pv_waited = false;
        // every thread has read S[gt & 1]; a tile that moves the reference reads it again below
        if (stid == 0 && !rare) mbar_arrive(&s_free[gt & 1]);
        if (rare) {
          ok = named_bar_and(1, NT, w && !failed);
          if (!ok) break;
          float* rb = red_m + (gt & 1) * NQ * 4;
          load_s(d, gt, t, ks);
          {
            const float wm = warp_col_reduce<NC, true>(d, lane);      // (it leaves d in pieces)
            if (lane < NC) rb[(c0 + lane) * 4 + quad] = wm;
          }
          named_bar_sync(1, NT);
          const int cl = c0 + (lane % NC);
          const float4 q4 = reinterpret_cast<const float4*>(rb)[cl];
          const float mt_l = fmaxf(fmaxf(q4.x, q4.y), fmaxf(q4.z, q4.w)) - kPExp;
          const float mo_l = mref[cl];
          const float mn_l = fmaxf(mo_l, mt_l);
          const float alpha_lane = ex2(mo_l - mn_l);
          const bool resc = __any_sync(0xFFFFFFFFu, mn_l != mo_l);
          named_bar_sync(1, NT);
          if (quad == 0 && lane < NC) {
            mref[cl] = mn_l;
            alph[cl] = alpha_lane;
          }
          named_bar_sync(1, NT);
#pragma unroll
          for (int c = 0; c < NC; ++c) l_part[c] *= alph[c0 + c];
          // O of the previous tiles moves to the new reference once PV of the last tile is done
          if (t > 0) {
            w = warp_spin(&pv_part[((gt - 1) & 1) * C::kParts + C::kParts - 1], static_cast<uint32_t>((gt - 1) >> 1) & 1u, abort_flag);
            tc_fence_after();
            pv_waited = true;
            if (w && resc) {
#pragma unroll 1
              for (int x = 0; x < 4 * C::kNO; x += NQ) {      // this thread's columns of every O_j
#pragma unroll 1
                for (int c1 = c0; c1 < c0 + NC; c1 += 16) {
                  float o[16];
                  tmem_ld16(tl + C::kTmemO + x + c1, o);
                  tmem_ld_wait();
#pragma unroll
                  for (int c = 0; c < 16; ++c) o[c] *= alph[c1 + c];
                  tmem_st16(tl + C::kTmemO + x + c1, o);
                }
              }
              tmem_st_wait();
            }
          }
          load_s(d, gt, t, ks);
          against();
#pragma unroll
          for (int c = 0; c < NC; ++c) d[c] = ex2(d[c]);
          tc_fence_before();
          named_bar_sync(1, NT);
          if (stid == 0) mbar_arrive(&s_free[gt & 1]);
        }
        if (stid == 0) TL(3, rare ? 30 : 3);
        const float ik = __uint_as_float((254u << 23) - __float_as_uint(ks < 0.f ? 1.f : ks));      // 1 / ks
        // A weight in f16 (11 bits, steps of 2^-24 below 2^-14) as three E5M2 terms, each the rest rounded to nearest (three bits and
        // a sign; the next rest is an f16 exactly, and an E5M2 the upper byte of an f16): to 2^-11 of the weight, or 2^-17
        // where E5M2 ends.
        uint32_t pw[C::kTerms][NC / 4];
#pragma unroll
        for (int y = 0; y < NC / 4; ++y) {
          uint32_t e[C::kTerms][2];
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            __half2 rest = __floats2half2_rn(d[4 * y + 2 * z], d[4 * y + 2 * z + 1]);
#pragma unroll
            for (int x = 0; x < C::kTerms; ++x) {
              e[x][z] = __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(rest), __NV_SATFINITE, __NV_E5M2);
              const uint32_t term = __byte_perm(e[x][z], 0u, 0x1404);
              if (x + 1 < C::kTerms) rest = __hsub2(rest, *reinterpret_cast<const __half2*>(&term));
            }
          }
#pragma unroll
          for (int x = 0; x < C::kTerms; ++x) pw[x][y] = __byte_perm(e[x][0], e[x][1], 0x5410);
        }
        if (t > 0 && !pv_waited) {
          w = warp_spin(&pv_part[((gt - 1) & 1) * C::kParts + C::kParts - 1], static_cast<uint32_t>((gt - 1) >> 1) & 1u, abort_flag);   // P is free
          tc_fence_after();
        }
        if (stid == 0) TL(3, 4);
        // 8 keys x 16 columns core matrices, 8-key groups 8 NQ bytes a term apart; one term's columns after the other's
        if (C::kKeys == kTile || row < C::kKeys) {
          uint8_t* prow = ps + (row >> 3) * (C::kTerms * 8 * NQ) + (row & 7) * 16;
#pragma unroll
          for (int x = 0; x < C::kTerms; ++x)
#pragma unroll
            for (int y = 0; y < NC / 4; y += 4)
              *reinterpret_cast<uint4*>(prow + ((x * NQ + c0) / 16 + y / 4) * 128) = make_uint4(pw[x][y], pw[x][y + 1], pw[x][y + 2], pw[x][y + 3]);
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0 && w) mbar_arrive(p_full);      // (where w is false the next barrier of the group ends the item)
        failed = failed || !w;
        if (stid == 0) TL(3, 5);
#pragma unroll
        for (int c = 0; c < NC; ++c) l_part[c] = fmaf(d[c], ik, l_part[c]);      // while PV runs
      }
      if (!ok) break;
      // the next item's query while PV runs and the results are written
      if (group_wait(warp == C::kFirstSm, 1, NT, &item_full[nit % kItemDepth], (nit / kItemDepth) & 1, abort_flag)) {
        const WorkItem qi = items[nit % kItemDepth];
        if (qi.b >= 0) {
          prep_query(qi);
          q_ready = true;
        }
      }
      // ---- epilogue: O / l and the LSE of every column of the item
      if (stid == 0) TL(3, 6);
      {
        w = warp_spin(&pv_part[((g + it.ntiles - 1) & 1) * C::kParts + C::kParts - 1], static_cast<uint32_t>((g + it.ntiles - 1) >> 1) & 1u, abort_flag);
        tc_fence_after();
      }
      g += it.ntiles;
      {
        const float lw = warp_col_reduce<NC, false>(l_part, lane);
        if (lane < NC) red_l[(c0 + lane) * 4 + quad] = lw;
      }
      ok = named_bar_and(1, NT, w && !failed);
      if (!ok) break;
      const int cl = c0 + (lane % NC);
      float inv_l, lse_l;
      {
        const float4 q4 = reinterpret_cast<const float4*>(red_l)[cl];
        const float l = (q4.x + q4.y) + (q4.z + q4.w);
        const bool none = l == 0.f;             // no visible key (a NaN goes on)
        inv_l = none ? 0.f : __fdividef(1.f, l);
        lse_l = none ? -CUDART_INF_F : (mref[cl] + __log2f(l)) * 0.69314718055994531f;
      }
      const bool final_out = it.pad != 0;
      // (row, head) of column cg: the flat index row * H + head is b * q_len * H + cg; a partial's is s * q_len * H + cg
      const int64_t flat0 = static_cast<int64_t>(final_out ? it.b : it.s) * p.cols + cgb;
      const int ncol = min(NC, p.cols - cgb);       // may be none
      const int64_t o_wrap = p.o_s0b - static_cast<int64_t>(p.H) * p.o_s1b;
#pragma unroll 1
      for (int jc = 0; jc < 4 * (NC / 16); ++jc) {
        const int jj = jc / (NC / 16), c1 = 16 * (jc % (NC / 16));
        if (c1 >= ncol) continue;
        float part[C::kStack][16];
#pragma unroll
        for (int x = 0; x < C::kStack; ++x) tmem_ld16(tl + C::kTmemO + C::kNO * jj + x * NQ + c0 + c1, part[x]);
        tmem_ld_wait();
        float (&o)[16] = part[0];
#pragma unroll
        for (int x = 1; x < C::kStack; ++x)
#pragma unroll
          for (int c = 0; c < 16; ++c) o[c] += part[x][c];
        const int d = 128 * jj + row;
        if (final_out) {
          int h = (cgb + c1) % p.H;
          uint8_t* ptr = p.out + (static_cast<int64_t>(it.b) * p.q_len + (cgb + c1) / p.H) * p.o_s0b +
                         static_cast<int64_t>(h) * p.o_s1b + 2 * d;
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            const float iv = __shfl_sync(0xFFFFFFFFu, inv_l, c1 + c);
            if (c1 + c < ncol) *reinterpret_cast<__nv_bfloat16*>(ptr) = __float2bfloat16_rn(o[c] * iv);
            ptr += p.o_s1b;
            if (++h == p.H) {
              h = 0;
              ptr += o_wrap;
            }
          }
        } else {
          float* dst = p.part_o + ((flat0 + c1) * kLora + d);
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            const float iv = __shfl_sync(0xFFFFFFFFu, inv_l, c1 + c);
            if (c1 + c < ncol) dst[static_cast<int64_t>(c) * kLora] = o[c] * iv;
          }
        }
      }
      if (quad == 0 && lane < ncol) {
        if (final_out) {
          if (p.lse) p.lse[flat0 + lane] = lse_l;
        } else {
          p.part_lse[flat0 + lane] = lse_l;
        }
      }
      tc_fence_before();
      named_bar_sync(1, NT);
      if (stid == 0) TL(3, 7);
      if (stid == 0) mbar_arrive(&item_empty[k]);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (tid == 0) TL(0, 9);
  if (tid == 0 && *abort_flag == 2) set_device_error(p.err, 16u);
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

}  // namespace mla
