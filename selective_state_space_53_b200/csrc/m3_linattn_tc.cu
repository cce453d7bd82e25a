// m3_linattn_tc.cu -- the linear attention core (m3_linattn.cuh) on the sm_100a tensor cores: bf16
// operands, key and value dims of 64 or 128.
//
// Chunks of Q = 128 tokens (the M of one MMA), a CTA walks the chunks of one (batch, head) for 64
// value columns with the state S (KD x 64, fp32) in registers.  With a = e^{log_decay}, token t at place
// t of a chunk of nv valid tokens, in time order
//   A   = q k^T                                          (M 128, N 128, K = KD)
//   A'  = s_upd s_out a^{t-s} A for s <= t, else 0       (bf16, tensor memory)
//   Yi  = q bf16(S)                                      (M 128, N 64, K = KD)
//   Ya  = A' v                                           (M 128, N 64, K 128, A' from tensor memory)
//   out = s_out a^{t+1} Yi + Ya
//   S  <- a^nv S + k^T (s_upd a^{nv-1-s} v)              (M = KD, N 192, K 128)
// and against time s >= t, a^{s-t}, a^{nv-1-t} and a^{s+1} in their places (the incoming state then
// carries its decay past the chunk before).  The weights a^e come from one table per CTA taken in
// 64 bits; a pair's weight is one factor of its row times one of its column within 32 x 32 blocks,
// both at most 1, so nothing overflows for any decay.
//
// Roundings: A' and the copy of S that q meets are bf16: an output is off by at most 2^-8 of the sum of
// the absolute values of its terms, beside its own rounding to bf16.  Where the terms do not cancel the two are
// alike (b2 L32768 H32 N = P = 128: relative 2-norm 2.3e-3 against 1.7e-3 of the final rounding alone), and
// a second part of A' and S would cost the tensor pipe two more products a chunk and 16 KiB that a head of
// 128 does not have.  The state is an fp32 result, so its update must not lose bits: the weighted v enters as
// three bf16 parts (8 bits each: all 24 of the product) side by side as N = 192 columns of one product, so k is
// read once for all three, and a^128 is a two-float constant.
//
// fp32 outputs (MODE 2) are a head's shares of a gradient that heads share: they are summed over the heads,
// where they may cancel, so their operands keep more.  A' and S enter as two bf16 parts each (2^-16 of a value
// is left), Yi and Ya are two products each into one accumulator, and an output is off by at most 2^-14 of its
// terms.  No caller reads the state of such a pass, so its weighted v has two parts (the second rounded: 2^-15 is
// left); the third part's shared memory then holds the low part of S and its accumulator columns that of A'.
// With one valid token and twelve heads dq and dk were 3e-2 off (relative 2-norm) with one part each, 1.6e-3 with two,
// the final rounding's own; the gradients at b4 L2048 H24 G1 N = P = 64 take 140 us, 108 with one part.
//
// Warp roles (20 warps; every mbarrier wait is bounded by %globaltimer):
//   0      producer: TMA loads of q, k, v into two stages (128-byte swizzle)
//   1      MMA issue; tensor-memory allocation
//   2      signals for the score warps; output store: TMA from the tile that the outputs were staged in
//          (over the chunk's q)
//   3      signals for the state warps
//   4-11   scores A -> A', 64 columns a warp, and the outputs of 32 value columns
//   12-19  the state of 32 value columns in registers, its copy bf16(S), and the weighted v
// Each kind has two warps on every scheduler, so that the tasks of one fill the latencies of the other.
// The signal warps wait for the products and the copies and meet the others on named barriers, where a
// waiting warp takes no issue slots (polling took a third of them).
// MMA order per chunk i: update(i), Yi(i), Ya(i), A(i+1).  The scores of i run behind update and Yi, the
// outputs behind A(i+1) and the next update; the weighted v of i + 1 (whose buffer the update of i has
// read then) and the state behind Yi to A(i+1).
// Why this split: q, k (32 KiB each at KD = 128), v and the three parts of the weighted v take 208 KiB at 64
// value columns with two stages of q, k and v, so a head of 128 value columns is two CTAs, which repeat A and
// its scores and share q and k in L2.
// Measured: b2 L32768 H32 N = P = 128 with own q and k 0.54 ms, 4.0 TB/s of algorithmic traffic (61 % of the
// measured copy rate); with shared q and k 0.50 ms.  Under a sustained load the board's power cap brings the
// clock to 1.47 GHz and the call to 0.65 ms.  A chunk takes about 3900 cycles against 2500 of products and 2900
// of shared-memory traffic: what bounds it is the latency of the SIMT tasks between the products (39 % of
// the issue slots and 43 % of the tensor pipe are used at 4096 tokens), not a pipe.
#include <cuda.h>

#include "m3_linattn.cuh"
#include "m3_ptx.cuh"

namespace m3 {
namespace {

constexpr int LQ = kLaChunk;  // tokens of a chunk
constexpr int LV = 64;   // value columns of a CTA
constexpr int L_PROD = 0, L_MMA = 1, L_STORE = 2, L_SIGNAL = 3;  // L_STORE also signals the score group
constexpr int L_CTRL = 4;       // control warps
constexpr int L_THREADS = 640;
constexpr int L_PREFETCH = 3;  // chunks that L2 is asked for ahead of their loads
constexpr int L_GROUP = 8;     // warps of the score group and of the state group
constexpr int LSC = LV / 2;    // value columns of a warp of either group
// named barriers of a signal warp and its group: what the group waits for
constexpr uint32_t LN_SC = 1, LN_Y = 2, LN_H = 3, LN_YI = 4, LN_THREADS = 32 * (L_GROUP + 1);
constexpr unsigned long long L_WAIT_NS = 2000000000ull;  // 2 s bound on any wait
constexpr int LBLK = 128 * 128;                          // one 64-column block of a 128-row tile, bytes
constexpr int L_MAXPOW = LQ + 1;  // and one word for the rest of a^128

// Barriers (pairs: one per stage).  None can complete two phases past a waiter (a parity wait would then
// miss one): each phase needs what the waiter does after it has seen the one before, of the same pair entry.
enum {
  LB_LQK = 0,  // [2] q and k of a stage landed (TMA bytes)
  LB_LV = 2,   // [2] v landed
  LB_FK = 4,   // [2] k free: the update read it (MMA commit)
  LB_FQ = 6,   // [2] q free: the outputs staged over it are stored (store warp)
  LB_FV = 8,   // [2] v free: Ya complete (MMA commit; state pass: the update)
  LB_YW = 10,  // [2] outputs staged over q
  LB_SC = 12,  // A complete (MMA commit)
  LB_SP,       // A' complete
  LB_ST,       // bf16(S) in shared memory
  LB_H,        // the update's parts complete (MMA commit)
  LB_HC,       // the update's parts read
  LB_VT,       // weighted v in shared memory
  LB_YI,       // Yi complete (MMA commit)
  LB_Y,        // Ya complete (MMA commit)
  LB_YE,       // Yi and Ya read
  LB_DRAIN,    // every MMA complete
  LNBAR
};

template <int KD>
struct LaCfg {
  static constexpr int TILE_K = (KD / 64) * LBLK;
  static constexpr int STAGE = 2 * TILE_K + LBLK;  // q, k, v
  static constexpr int OFF_VT = 2 * STAGE;         // three parts of the weighted v
  static constexpr int OFF_S = OFF_VT + 3 * LBLK;  // bf16(S), KD rows of 64
  static constexpr int OFF_POW = OFF_S + KD * 128;
  static constexpr int OFF_COL = OFF_POW + (((L_MAXPOW + 1) * 4 + 15) & ~15);  // column factors of a 32-column score block
  static constexpr int OFF_BAR = OFF_COL + 32 * 4;
  static constexpr int OFF_MISC = OFF_BAR + LNBAR * 8;
  static constexpr int SMEM = OFF_MISC + 32 + 1024;
  static constexpr uint32_t TM_A = 0, TM_AP = 128, TM_YA = 192, TM_YI = 256, TM_H = 320, TM_COLS = 512;
  static constexpr uint32_t TM_AL = TM_H + 2 * LV;  // low part of A' (shares: the update has two parts)
  static constexpr int OFF_SL = OFF_VT + 2 * LBLK;  // low part of S (shares)
  static constexpr uint32_t ID_A = idesc_bf16(128, 128, false, false);
  static constexpr uint32_t ID_Y = idesc_bf16(128, LV, false, true);
  static constexpr uint32_t ID_H = idesc_bf16(KD, 3 * LV, true, true);
  static constexpr uint32_t ID_H2 = idesc_bf16(KD, 2 * LV, true, true);
  static_assert(SMEM <= 227 * 1024, "shared memory");
};

// Waits.  The plain try_wait suspends the warp for a while by itself; a wait that goes on looks at the
// abort flag and the clock only every 256 tries, so that waiting warps leave the issue slots to the others
// (the form with a suspend-time hint and a look at the clock each time took a third of all instructions).
__device__ __forceinline__ bool la_try(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(done)
      : "r"(bar), "r"(parity)
      : "memory");
  return done != 0;
}
__device__ __noinline__ bool la_wait_long(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  const uint64_t t0 = globaltimer();
  for (;;) {
    for (int k = 0; k < 256; ++k)
      if (la_try(bar, parity)) return true;
    if (abort_flag && *abort_flag) return false;
    if (globaltimer() - t0 > L_WAIT_NS) {
      if (abort_flag) *abort_flag = 1;
      return false;
    }
  }
}
__device__ __forceinline__ bool la_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
#pragma unroll 1
  for (int k = 0; k < 64; ++k)
    if (la_try(bar, parity)) return true;
  return la_wait_long(bar, parity, abort_flag);
}
// Bounded by time only: drains copies and MMAs in flight before the CTA exits.
__device__ __forceinline__ void la_drain(uint32_t bar, uint32_t parity) { la_wait_long(bar, parity, nullptr); }
__device__ __forceinline__ float lds32(uint32_t addr) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t f2_bits(uint32_t lo, uint32_t hi) { return f2(__uint_as_float(lo), __uint_as_float(hi)); }
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&v)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
               : "r"(taddr));
}
// MMA issue and commit by the one thread that executes them.
__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile("{\n .reg .pred p;\n .reg .b32 r;\n elect.sync r|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(e));
  return e != 0;
}
__device__ __forceinline__ void mma_ss1(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc));
}
__device__ __forceinline__ void mma_ts1(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(
          d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc));
}
__device__ __forceinline__ void mma_commit1(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}
// Asks L2 for a tile that a load will want later.
__device__ __forceinline__ void tma_prefetch_4d(const CUtensorMap* map, int c0, int c1, int c2, int c3) {
  asm volatile("cp.async.bulk.prefetch.tensor.4d.L2.global.tile [%0, {%1, %2, %3, %4}];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(c0), "r"(c1), "r"(c2), "r"(c3)
               : "memory");
}
// TMA tile store from shared memory, in bulk groups.
__device__ __forceinline__ void tma_store_4d(const CUtensorMap* map, uint32_t src, int c0, int c1, int c2, int c3) {
  asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3, %4}], [%5];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(src)
               : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
__device__ __forceinline__ void la_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// Up to three passes in one launch (blockIdx.y): the gradients of one layer, whose CTAs then fill the
// machine together.
struct LaPass {
  CUtensorMap q, k, v, o;
  LaCore a;
};
struct LaJob {
  LaPass p[3];
};

// MODE 0: outputs in bf16; 1: the state pass of a segment; 2: some of the passes are shares (fp32 outputs).
template <int KD, int MODE>
__global__ void __launch_bounds__(L_THREADS, 1) la_tc_kernel(const __grid_constant__ LaJob job) {
  const CUtensorMap& tmQ = job.p[blockIdx.y].q;
  const CUtensorMap& tmK = job.p[blockIdx.y].k;
  const CUtensorMap& tmV = job.p[blockIdx.y].v;
  const CUtensorMap& tmO = job.p[blockIdx.y].o;
  const LaCore& a = job.p[blockIdx.y].a;
  using C = LaCfg<KD>;
  constexpr bool FULL = MODE != 1;
  const bool share = MODE == 2 && a.out_f32;  // (the outputs' code asks a.out_f32 itself: without that branch the
                                              // bf16 form interleaves its blocks, 1.5 % slower at 32K)
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  // the warp index as a uniform value: addresses and branches that hang on it stay off the vector registers
  const int tid = threadIdx.x, warp = __shfl_sync(kFull, tid >> 5, 0), lane = tid & 31, q4 = warp & 3;
  const int vtiles = a.VD / LV;
  unsigned blk = blockIdx.x;
  const int vt = vtiles == 2 ? (int)(blk & 1) : 0;
  if (vtiles == 2) blk >>= 1;
  const unsigned nseg_grid = FULL ? a.nseg : a.nseg - 1;
  const int seg = (int)(blk % nseg_grid), bh = (int)(blk / nseg_grid);
  const int bi = bh / a.H, h = bh % a.H;

  uint64_t* bar = reinterpret_cast<uint64_t*>(sm + C::OFF_BAR);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + C::OFF_MISC + 4);
  float* pw = reinterpret_cast<float*>(sm + C::OFF_POW);
  const uint32_t sBase = smem_u32(sm);
  auto B = [&](int k) { return sBase + C::OFF_BAR + 8 * k; };
  auto sQ = [&](int s) { return sBase + (uint32_t)(s * C::STAGE); };
  auto sK = [&](int s) { return sBase + (uint32_t)(s * C::STAGE + C::TILE_K); };
  auto sV = [&](int s) { return sBase + (uint32_t)(s * C::STAGE + 2 * C::TILE_K); };
  const uint32_t sVT = sBase + C::OFF_VT, sS = sBase + C::OFF_S, sSL = sBase + C::OFF_SL;

  // ---- setup
  if (warp == L_MMA) {
    tmem_alloc(tmem_slot, C::TM_COLS);
    tmem_relinquish();
  }
  if (tid == 0) {
    for (int s = 0; s < 2; ++s) {
      for (int k : {LB_LQK, LB_LV, LB_FK, LB_FQ, LB_FV}) mbar_init(&bar[k + s], 1);
      mbar_init(&bar[LB_YW + s], L_GROUP);
    }
    for (int k : {LB_SC, LB_H, LB_YI, LB_Y}) mbar_init(&bar[k], 1);
    for (int k : {LB_SP, LB_ST, LB_HC, LB_VT, LB_YE}) mbar_init(&bar[k], L_GROUP);
    mbar_init(&bar[LB_DRAIN], 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  const float ld = a.log_decay[h];
  float* colf = reinterpret_cast<float*>(sm + C::OFF_COL);
  if (tid < L_MAXPOW) {
    const double wd = la_pow(ld, tid);
    const float w = (float)wd;
    pw[tid] = w;
    if (tid == LQ) pw[LQ + 1] = (float)(wd - (double)w);  // a^128 as two floats
    if (tid < 32) {
      colf[a.rev ? tid : 31 - tid] = w;
    }
  }
  const int64_t page = la_page_block(a.pages, a.npages, bi, a.status);
  const int len = page < 0 ? 0 : la_len(a, bi);
  const ChunkSpan cs = la_chunks(a, seg, len);
  const int n = cs.n;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(kFull, *tmem_slot, 0);
  const uint32_t lane_base = (uint32_t)(32 * q4) << 16;
  auto chunk = [&](int i) { return a.rev ? cs.first - i : cs.first + i; };
  auto valid = [&](int i) {  // tokens of chunk i within the length
    const int left = len - chunk(i) * LQ;
    return left < LQ ? left : LQ;
  };

  const int part = a.rev ? 0 : n - 1;  // the one chunk that the sequence's end may cut
  const int nv_part = n > 0 ? valid(part) : LQ;
  const uint32_t sPow = sBase + C::OFF_POW;
  auto arrive = [&](int k) {
    __syncwarp();
    if (lane == 0) la_arrive(B(k));
  };

  if (warp < L_CTRL) {
    if (warp == L_PROD) {
      // =============================================================== producer
      if (lane == 0) {
        const int gq = h / (a.H / a.hq), gk = h / (a.H / a.hk), gv = h / (a.H / a.hv);
        // chunk i into L2 (q and k by the CTA of the first value columns only): two stages in shared memory
        // alone leave a load's latency, three thousand cycles from HBM, uncovered
        auto prefetch = [&](int i) {
          if (i >= n) return;
          const int tok = chunk(i) * LQ;
          tma_prefetch_4d(&tmV, LV * vt, gv, tok, bi);
          if (vt > 0) return;
#pragma unroll
          for (int b = 0; b < KD / 64; ++b) {
            tma_prefetch_4d(&tmK, 64 * b, gk, tok, bi);
            if constexpr (FULL) tma_prefetch_4d(&tmQ, 64 * b, gq, tok, bi);
          }
        };
        for (int i = 2; i < L_PREFETCH; ++i) prefetch(i);
        int done = 0;
        for (int i = 0; i < n; ++i) {
          prefetch(i + L_PREFETCH);
          const int s = i & 1, tok = chunk(i) * LQ;
          const uint32_t before = (uint32_t)(((i >> 1) & 1) ^ 1);  // phase of the stage's chunk i - 2
          if (i >= 2 && !la_wait(B(LB_FK + s), before, abort_flag)) break;
          mbar_expect_tx(&bar[LB_LQK + s], FULL ? 2 * C::TILE_K : C::TILE_K);
#pragma unroll
          for (int b = 0; b < KD / 64; ++b) tma_load_4d(sK(s) + b * LBLK, &tmK, 64 * b, gk, tok, bi, &bar[LB_LQK + s]);
          if (i >= 2) la_wait(B(LB_FV + s), before, abort_flag);  // a timeout still completes the barriers
          mbar_expect_tx(&bar[LB_LV + s], LBLK);
          tma_load_4d(sV(s), &tmV, LV * vt, gv, tok, bi, &bar[LB_LV + s]);
          if constexpr (FULL) {
            if (i >= 2) la_wait(B(LB_FQ + s), before, abort_flag);
#pragma unroll
            for (int b = 0; b < KD / 64; ++b) tma_load_4d(sQ(s) + b * LBLK, &tmQ, 64 * b, gq, tok, bi, &bar[LB_LQK + s]);
          }
          ++done;
        }
        // every copy issued has landed before the CTA may exit
        for (int s = 0; s < 2; ++s) {
          const int k = (done + 1 - s) / 2;  // copies into stage s
          if (k > 0) la_drain(B(LB_LQK + s), (uint32_t)((k - 1) & 1));
          if (k > 0) la_drain(B(LB_LV + s), (uint32_t)((k - 1) & 1));
        }
      }
    } else if (warp == L_STORE) {
      // =============================================================== signals to the score group, output store
      // After a timeout a signal warp meets its group without waiting, so that the group runs through its
      // chunks (within bounds, the results void) and everyone leaves.
      if constexpr (FULL) {
        bool ok = true;
        auto store = [&](int i) {  // the staged outputs of chunk i; tokens past L are not written
          const int s = i & 1;
          ok = ok && la_wait(B(LB_YW + s), (uint32_t)((i >> 1) & 1), abort_flag);
          if (lane == 0 && ok) {
            if (!a.out_f32) {
              tma_store_4d(&tmO, sQ(s), LV * vt, h, chunk(i) * LQ, bi);
              bulk_commit();
              bulk_wait_read();
            }
            la_arrive(B(LB_FQ + s));
          }
          __syncwarp();
        };
        for (int i = 0; i < n; ++i) {
          const uint32_t p = (uint32_t)(i & 1);
          ok = ok && la_wait(B(LB_SC), p, abort_flag);
          named_bar_sync(LN_SC, LN_THREADS);
          if (i > 0) store(i - 1);
          ok = ok && la_wait(B(LB_Y), p, abort_flag);
          named_bar_sync(LN_Y, LN_THREADS);
        }
        if (n > 0) store(n - 1);
        if (lane == 0) bulk_wait_all();
      }
    } else if (warp == L_SIGNAL) {
      // =============================================================== signals to the state group
      bool ok = true;
      for (int i = -1; n > 0 && i < n; ++i) {  // the update of i complete (i = -1: none yet), v of i + 1 landed
        const uint32_t p = (uint32_t)(i & 1);
        if (i >= 0) ok = ok && la_wait(B(LB_H), p, abort_flag);
        if (i + 1 < n) {
          const int s = (i + 1) & 1;
          const uint32_t ps = (uint32_t)(((i + 1) >> 1) & 1);
          ok = ok && la_wait(B(LB_LV + s), ps, abort_flag);
          // k as well where the sequence's end cuts the chunk
          if (i + 1 == part && nv_part < LQ) ok = ok && la_wait(B(LB_LQK + s), ps, abort_flag);
        }
        named_bar_sync(LN_H, LN_THREADS);
        if (FULL && i >= 0 && i + 1 < n) {
          ok = ok && la_wait(B(LB_YI), p, abort_flag);
          named_bar_sync(LN_YI, LN_THREADS);
        }
      }
    } else if (warp == L_MMA && n > 0) {
      // =============================================================== MMA issue
      // Operand descriptors of stage 0; a stage, a block and a K-step are plain address offsets.
      const uint64_t dQ = sdesc(sQ(0), 16, 1024), dK = sdesc(sK(0), 16, 1024);          // K-major
      const uint64_t dKt = sdesc(sK(0), LBLK, 1024), dVm = sdesc(sV(0), LBLK, 1024);    // MN-major
      const uint64_t dS = sdesc(sS, LBLK, 1024), dVT = sdesc(sVT, LBLK, 1024);
      const uint64_t dSL = sdesc(sSL, LBLK, 1024);
      auto stage = [&](int i) { return (uint64_t)((i & 1) * (C::STAGE >> 4)); };
      auto kstep = [](int k) { return (uint64_t)(((k >> 2) * LBLK + (k & 3) * 32) >> 4); };
      auto mstep = [](int k) { return (uint64_t)((k * 2048) >> 4); };
      const bool lead = elect_one();
      auto scores = [&](int i) -> bool {  // A of chunk i
        const int s = i & 1;
        if (!la_wait(B(LB_LQK + s), (uint32_t)((i >> 1) & 1), abort_flag)) return false;
        if constexpr (FULL) {
          tc_fence_after();
          if (lead) {
#pragma unroll
            for (int k = 0; k < KD / 16; ++k)
              mma_ss1(tmem + C::TM_A, dQ + stage(i) + kstep(k), dK + stage(i) + kstep(k), C::ID_A, k > 0);
            mma_commit1(&bar[LB_SC]);
          }
          __syncwarp();
        }
        return true;
      };
      bool ok = scores(0);
      for (int i = 0; ok && i < n; ++i) {
        const int s = i & 1;
        const uint32_t p = (uint32_t)(i & 1);
        ok = la_wait(B(LB_VT), p, abort_flag);
        if (ok && i > 0) ok = la_wait(B(LB_HC), p ^ 1, abort_flag);
        if (!ok) break;
        tc_fence_after();
        if (lead) {
#pragma unroll
          for (int k = 0; k < LQ / 16; ++k)
            mma_ss1(tmem + C::TM_H, dKt + stage(i) + mstep(k), dVT + mstep(k), share ? C::ID_H2 : C::ID_H, k > 0);
          mma_commit1(&bar[LB_H]);
          mma_commit1(&bar[LB_FK + s]);
          if (!FULL) mma_commit1(&bar[LB_FV + s]);
        }
        __syncwarp();
        if constexpr (FULL) {
          ok = la_wait(B(LB_ST), p, abort_flag);
          if (ok && i > 0) ok = la_wait(B(LB_YE), p ^ 1, abort_flag);
          if (!ok) break;
          tc_fence_after();
          if (lead) {
#pragma unroll
            for (int k = 0; k < KD / 16; ++k)
              mma_ss1(tmem + C::TM_YI, dQ + stage(i) + kstep(k), dS + mstep(k), C::ID_Y, k > 0);
            if (share) {
#pragma unroll
              for (int k = 0; k < KD / 16; ++k)
                mma_ss1(tmem + C::TM_YI, dQ + stage(i) + kstep(k), dSL + mstep(k), C::ID_Y, 1);
            }
            mma_commit1(&bar[LB_YI]);
          }
          __syncwarp();
          ok = la_wait(B(LB_SP), p, abort_flag);
          if (!ok) break;
          tc_fence_after();
          if (lead) {
#pragma unroll
            for (int k = 0; k < LQ / 16; ++k)
              mma_ts1(tmem + C::TM_YA, tmem + C::TM_AP + 8 * k, dVm + stage(i) + mstep(k), C::ID_Y, k > 0);
            if (share) {
#pragma unroll
              for (int k = 0; k < LQ / 16; ++k)
                mma_ts1(tmem + C::TM_YA, tmem + C::TM_AL + 8 * k, dVm + stage(i) + mstep(k), C::ID_Y, 1);
            }
            mma_commit1(&bar[LB_Y]);
            mma_commit1(&bar[LB_FV + s]);
          }
          __syncwarp();
        }
        if (i + 1 < n) ok = scores(i + 1);
      }
      // every MMA issued has completed before tensor memory is released
      if (lead) mma_commit1(&bar[LB_DRAIN]);
      __syncwarp();
      la_drain(B(LB_DRAIN), 0);
    }
  } else if (warp < L_CTRL + L_GROUP) {
    // =============================================================== scores and outputs
    if constexpr (FULL) {
      const int w = (warp - L_CTRL) >> 2;  // score blocks w and 3 - w (of 32 columns), value columns 32 w ..
      const int t = 32 * q4 + lane;        // this thread's token of a chunk
      const uint32_t ro = (uint32_t)t * 128u;
      const int64_t col = LV * vt + LSC * w;
      const uint32_t sCol = sBase + C::OFF_COL;
      const float sc = a.s_upd * a.s_out;
      auto out_row = [&](int64_t tok) { return (((int64_t)bi * a.L + tok) * a.H + h) * (int64_t)a.VD + col; };
      // Blocks between the rows and a block of columns: below 0 it lies ahead and stays zero throughout.  The
      // weights of one block are kept in registers: the diagonal one if the warp has it (zero where the column
      // is ahead of the row), else its first; those of the other are made from a row and a column factor.
      auto dist = [&](int cb) { return a.rev ? cb - q4 : q4 - cb; };
      const bool swap = dist(w) != 0 && (dist(3 - w) == 0 || dist(w) < 0);
      const int cb0 = swap ? 3 - w : w, cb1 = swap ? w : 3 - w, d0 = dist(cb0), d1 = dist(cb1);
      uint64_t W[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int x0 = 32 * d0 + (a.rev ? 2 * e - lane : lane - 2 * e), x1 = x0 + (a.rev ? 1 : -1);
        const float w0 = sc * lds32(sPow + 4 * (x0 < 0 ? 0 : x0)), w1 = sc * lds32(sPow + 4 * (x1 < 0 ? 0 : x1));
        W[e] = f2(x0 < 0 ? 0.0f : w0, x1 < 0 ? 0.0f : w1);
      }
      {
        uint32_t o[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) o[e] = 0u;
        if (d0 < 0) tmem_st16(tmem + lane_base + C::TM_AP + 16 * cb0, o);
        if (d1 < 0) tmem_st16(tmem + lane_base + C::TM_AP + 16 * cb1, o);
        if (share && d0 < 0) tmem_st16(tmem + lane_base + C::TM_AL + 16 * cb0, o);
        if (share && d1 < 0) tmem_st16(tmem + lane_base + C::TM_AL + 16 * cb1, o);
      }
      const float r1 = d1 > 0 ? sc * lds32(sPow + 4 * (a.rev ? 32 * d1 - lane : 32 * d1 - 31 + lane)) : 0.0f;
      for (int i = 0; i < n; ++i) {
        const int s = i & 1;
        const int nv = i == part ? nv_part : LQ;
        named_bar_sync(LN_SC, LN_THREADS);
        tc_fence_after();
        auto finish = [&](uint32_t to, int cb, uint32_t (&o)[16]) {
          if (32 * cb + 32 > nv) {  // columns past the length
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              if (32 * cb + 2 * e >= nv) o[e] = 0u;
              else if (32 * cb + 2 * e + 1 >= nv) o[e] &= 0xffffu;
            }
          }
          tmem_st16(tmem + lane_base + to + 16 * cb, o);
        };
        auto rest = [&](int cb, const float (&x)[32]) {  // what the rounding of a block left
          uint32_t o[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const uint32_t hi = pack_bf16(x[2 * e], x[2 * e + 1]);
            o[e] = pack_bf16(x[2 * e] - bf_lo(hi), x[2 * e + 1] - bf_hi(hi));
          }
          finish(C::TM_AL, cb, o);
        };
        if (d0 >= 0) {
          uint32_t v[32], o[16];
          float x[32];
          tmem_ld32(tmem + lane_base + C::TM_A + 32 * cb0, v);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            f2_split(f2_mul(f2_bits(v[2 * e], v[2 * e + 1]), W[e]), x[2 * e], x[2 * e + 1]);
            o[e] = pack_bf16(x[2 * e], x[2 * e + 1]);
          }
          finish(C::TM_AP, cb0, o);
          if (share) rest(cb0, x);
        }
        if (d1 >= 0) {
          uint32_t v[32], o[16];
          float x[32];
          tmem_ld32(tmem + lane_base + C::TM_A + 32 * cb1, v);
          tmem_wait_ld();
          const uint64_t r2 = f2(r1, r1);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const uint4 u = lds128(sCol + 16 * e);
            f2_split(f2_mul(f2_bits(v[4 * e], v[4 * e + 1]), f2_mul(f2_bits(u.x, u.y), r2)), x[4 * e], x[4 * e + 1]);
            f2_split(f2_mul(f2_bits(v[4 * e + 2], v[4 * e + 3]), f2_mul(f2_bits(u.z, u.w), r2)), x[4 * e + 2], x[4 * e + 3]);
            o[2 * e] = pack_bf16(x[4 * e], x[4 * e + 1]);
            o[2 * e + 1] = pack_bf16(x[4 * e + 2], x[4 * e + 3]);
          }
          finish(C::TM_AP, cb1, o);
          if (share) rest(cb1, x);
        }
        tmem_wait_st();
        tc_fence_before();
        arrive(LB_SP);
        // ---- outputs of the chunk
        named_bar_sync(LN_Y, LN_THREADS);
        tc_fence_after();
        const bool on = t < nv;
        const float f = on ? a.s_out * lds32(sPow + 4 * (a.rev ? nv - 1 - t : t + 1)) : 0.0f;
#pragma unroll
        for (int c = 0; c < LSC / 16; ++c) {
          uint32_t x[16], y[16];
          tmem_ld16(tmem + lane_base + C::TM_YI + LSC * w + 16 * c, x);
          tmem_ld16(tmem + lane_base + C::TM_YA + LSC * w + 16 * c, y);
          tmem_wait_ld();
          if (c == LSC / 16 - 1) {
            tc_fence_before();
            arrive(LB_YE);
          }
          float v[16];
#pragma unroll
          for (int e = 0; e < 8; ++e)
            f2_split(f2_fma(f2(f, f), f2_bits(x[2 * e], x[2 * e + 1]), f2_bits(y[2 * e], y[2 * e + 1])), v[2 * e], v[2 * e + 1]);
          if (!on) {
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] = 0.0f;
          }
          if (a.out_f32) {
            // the warp's 32 rows of 16 values over its 2 KB of q's tile (64-byte rows, 16-byte chunks rotated
            // by the row), then four lanes to a row: full sectors, an eighth of the lines per store
            const uint32_t sW = sQ(s) + 2048u * (warp - L_CTRL);
#pragma unroll
            for (int e = 0; e < 4; ++e)
              sts128(sW + lane * 64 + (((e + (lane >> 1)) & 3) << 4),
                     make_uint4(__float_as_uint(v[4 * e]), __float_as_uint(v[4 * e + 1]), __float_as_uint(v[4 * e + 2]),
                                __float_as_uint(v[4 * e + 3])));
            __syncwarp();
            const int ch = lane & 3;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int r = 8 * e + (lane >> 2), rt = chunk(i) * LQ + 32 * q4 + r;
              const uint4 x4 = lds128(sW + r * 64 + (((ch + (r >> 1)) & 3) << 4));
              if (rt < a.L) reinterpret_cast<uint4*>(static_cast<float*>(a.out) + out_row(rt))[4 * c + ch] = x4;
            }
            __syncwarp();
          } else {  // over q of the stage, which Yi was the last to read
#pragma unroll
            for (int e = 0; e < 2; ++e)
              sts128(sQ(s) + ro + (((4 * w + 2 * c + e) ^ (t & 7)) << 4),
                     make_uint4(pack_bf16(v[8 * e], v[8 * e + 1]), pack_bf16(v[8 * e + 2], v[8 * e + 3]),
                                pack_bf16(v[8 * e + 4], v[8 * e + 5]), pack_bf16(v[8 * e + 6], v[8 * e + 7])));
          }
        }
        fence_async_smem();
        arrive(LB_YW + s);
      }
      // chunks past the sequence's length
      for (int j = cs.z0; j < cs.z1; ++j) {
        const int tok = j * LQ + t;
        if (tok >= a.L) continue;
        const int e = a.out_f32 ? 4 : 2;
        uint4* g = reinterpret_cast<uint4*>(static_cast<char*>(a.out) + out_row(tok) * e);
        for (int c = 0; c < LSC * e / 16; ++c) g[c] = make_uint4(0, 0, 0, 0);
      }
    }
  } else {
    // =============================================================== state and weighted v
    const int w = (warp - L_CTRL - L_GROUP) >> 2;  // value columns 32 w .. 32 w + 31
    const int t = 32 * q4 + lane;                  // this thread's token of a chunk (weighted v)
    const uint32_t ro = (uint32_t)t * 128u;
    // accumulator row of the state (M = 128: the lane; M = 64: lanes 0-15 of each quarter)
    const bool owner = KD == 128 || lane < 16;
    const int row = KD == 128 ? t : 16 * q4 + (lane & 15);
    const int64_t col = LV * vt + LSC * w;

    // ---- the state entering the segment, in pairs
    uint64_t S[LSC / 2];
#pragma unroll
    for (int e = 0; e < LSC / 2; ++e) S[e] = 0;
    auto slot = [&](int s) { return a.ws + (((int64_t)bh * a.nseg + s) * KD + row) * a.VD + col; };
    const int64_t sbase = (page * a.H + h) * (int64_t)KD * a.VD + row * a.s_i + col * a.s_j;
    auto store_slot = [&](int s) {
      float4* p = reinterpret_cast<float4*>(slot(s));
#pragma unroll
      for (int e = 0; e < LSC / 4; ++e) {
        float4 v;
        f2_split(S[2 * e], v.x, v.y);
        f2_split(S[2 * e + 1], v.z, v.w);
        p[e] = v;
      }
    };
    if (owner && page >= 0) {
      const bool from_ws = FULL && a.nseg > 1;
      if (from_ws || (seg == 0 && a.s_in)) {
        const float* src = from_ws ? slot(seg) : a.s_in + sbase;
        const int sj = from_ws ? 1 : (int)a.s_j;
#pragma unroll
        for (int e = 0; e < LSC / 2; ++e) S[e] = f2(src[2 * e * sj], src[(2 * e + 1) * sj]);
      }
      if (!FULL && seg == 0) store_slot(0);
    }
    auto publish = [&]() {  // bf16(S), the B operand of Yi
      if (owner) {
#pragma unroll
        for (int c = 0; c < LSC / 8; ++c) {
          uint32_t o[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float lo, hi;
            f2_split(S[4 * c + e], lo, hi);
            o[e] = pack_bf16(lo, hi);
          }
          const uint32_t to = row * 128 + (((c + 4 * w) ^ (row & 7)) << 4);
          sts128(sS + to, make_uint4(o[0], o[1], o[2], o[3]));
          if (share) {  // what the rounding left
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float lo, hi;
              f2_split(S[4 * c + e], lo, hi);
              o[e] = pack_bf16(lo - bf_lo(o[e]), hi - bf_hi(o[e]));
            }
            sts128(sSL + to, make_uint4(o[0], o[1], o[2], o[3]));
          }
        }
      }
      fence_async_smem();
      arrive(LB_ST);
    };

    // ---- the weighted v of chunk i: three parts of 8 values; each part takes the upper 16 bits of what
    // is left, 24 bits in all (shares: two parts, the second rounded)
    auto weight = [&](int i) {
      const int nv = i == part ? nv_part : LQ;
      return t < nv ? a.s_upd * lds32(sPow + 4 * (a.rev ? t + 1 : nv - 1 - t)) : 0.0f;
    };
    auto vchunk = [&](int c) { return ro + (uint32_t)(((c + 4 * w) ^ (t & 7)) << 4); };
    auto weigh = [&](int i) {
      if (i == part && nv_part < LQ) {  // no infinity or NaN found past the length meets a product
        if (t >= nv_part) {
          const int s = i & 1;
          const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
          for (int c = 0; c < LSC / 8; ++c) {
            sts128(sV(s) + vchunk(c), zero);
#pragma unroll
            for (int b = 0; b < KD / 64; ++b) sts128(sK(s) + b * LBLK + vchunk(c), zero);
          }
        }
      }
      const float wt = weight(i);
      const uint64_t w2 = f2(wt, wt), minus = f2(-1.0f, -1.0f);
#pragma unroll
      for (int c = 0; c < LSC / 8; ++c) {
        const uint4 raw = lds128(sV(i & 1) + vchunk(c));
        uint64_t f[4] = {f2_mul(f2(bf_lo(raw.x), bf_hi(raw.x)), w2), f2_mul(f2(bf_lo(raw.y), bf_hi(raw.y)), w2),
                         f2_mul(f2(bf_lo(raw.z), bf_hi(raw.z)), w2), f2_mul(f2(bf_lo(raw.w), bf_hi(raw.w)), w2)};
#pragma unroll
        for (int q = 0; q < 3; ++q) {
          uint32_t b[4];
          if (share && q == 2) break;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float lo, hi;
            f2_split(f[e], lo, hi);
            if (share && q == 1) b[e] = pack_bf16(lo, hi);
            else b[e] = __byte_perm(__float_as_uint(lo), __float_as_uint(hi), 0x7632);
            if (q < 2)  // exact
              f[e] = f2_fma(f2(__uint_as_float(__float_as_uint(lo) & 0xffff0000u),
                               __uint_as_float(__float_as_uint(hi) & 0xffff0000u)), minus, f[e]);
          }
          sts128(sVT + q * LBLK + vchunk(c), make_uint4(b[0], b[1], b[2], b[3]));
        }
      }
      fence_async_smem();
      arrive(LB_VT);
    };

    // the decay of a full chunk as two floats: a long memory multiplies it in hundreds of times
    const float a128 = lds32(sPow + 4 * LQ), a128_lo = lds32(sPow + 4 * LQ + 4);
    if (n > 0) {
      if constexpr (FULL) publish();
      named_bar_sync(LN_H, LN_THREADS);
      weigh(0);
    }
    for (int i = 0; i < n; ++i) {
      const int nv = i == part ? nv_part : LQ;
      // ---- the next chunk's weighted v, once the update has read this one's
      named_bar_sync(LN_H, LN_THREADS);
      tc_fence_after();
      if (i + 1 < n) weigh(i + 1);
      // ---- the state after this chunk
      const float ghi = nv == LQ ? a128 : lds32(sPow + 4 * nv), glo = nv == LQ ? a128_lo : 0.0f;
#pragma unroll
      for (int c = 0; c < LSC / 8; ++c) {
        uint32_t x[8], y[8], z[8];
        tmem_ld8(tmem + lane_base + C::TM_H + LSC * w + 8 * c, x);
        tmem_ld8(tmem + lane_base + C::TM_H + LV + LSC * w + 8 * c, y);
        if (share) {
#pragma unroll
          for (int e = 0; e < 8; ++e) z[e] = 0u;
        } else {
          tmem_ld8(tmem + lane_base + C::TM_H + 2 * LV + LSC * w + 8 * c, z);
        }
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint64_t hs = f2_add(f2_bits(x[2 * e], x[2 * e + 1]),
                                     f2_add(f2_bits(y[2 * e], y[2 * e + 1]), f2_bits(z[2 * e], z[2 * e + 1])));
          S[4 * c + e] = f2_fma(f2(ghi, ghi), S[4 * c + e], f2_fma(f2(glo, glo), S[4 * c + e], hs));
        }
      }
      tc_fence_before();
      arrive(LB_HC);
      if (FULL && i + 1 < n) {
        named_bar_sync(LN_YI, LN_THREADS);  // Yi has read the copy before
        publish();
      }
    }
    if (!*abort_flag && owner && page >= 0) {
      if (!FULL) {
        store_slot(seg + 1);
      } else if (seg == a.nseg - 1 && a.s_fin) {
        float* dst = a.s_fin + sbase;
        const int sj = (int)a.s_j;
#pragma unroll
        for (int e = 0; e < LSC / 2; ++e) {
          float lo, hi;
          f2_split(S[e], lo, hi);
          dst[2 * e * sj] = lo;
          dst[(2 * e + 1) * sj] = hi;
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (tid == 0 && *abort_flag) set_status(a.status, M3_ERR_TIMEOUT);
  if (warp == L_MMA) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TM_COLS);
  }
}

// (b, L, heads, D) bf16 in boxes of 64 columns x 128 tokens of one head; tokens past L read as zero.
bool la_map(CUtensorMap* m, const LaCore& a, const void* base, int heads, int D) {
  auto fn = tma_encode_fn();
  if (!fn) return false;
  const cuuint64_t row = (cuuint64_t)D * 2, tok = row * heads;
  const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)a.L, (cuuint64_t)a.b};
  const cuuint64_t str[3] = {row, tok, tok * (cuuint64_t)a.L};
  const cuuint32_t box[4] = {64, 1, LQ, 1};
  const cuuint32_t es[4] = {1, 1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, str, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int KD, int MODE>
cudaError_t launch_tc_mode(const LaJob& job, int n, cudaStream_t stream) {
  static SmemAttr attr;
  auto kern = la_tc_kernel<KD, MODE>;
  const cudaError_t e = attr.ensure(kern, LaCfg<KD>::SMEM);
  if (e != cudaSuccess) return e;
  const LaCore& a = job.p[0].a;
  const int64_t grid = a.b * a.H * (a.VD / LV) * (MODE == 1 ? a.nseg - 1 : a.nseg);
  if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
  kern<<<dim3((unsigned)grid, (unsigned)n), L_THREADS, LaCfg<KD>::SMEM, stream>>>(job);
  return cudaGetLastError();
}

template <int KD>
cudaError_t launch_tc_kd(const LaCores& cores, int n, cudaStream_t stream) {
  LaJob job;
  for (int i = 0; i < n; ++i) {
    LaPass& p = job.p[i];
    const LaCore& a = p.a = cores.p[i];
    if (!la_map(&p.q, a, a.q, a.hq, KD) || !la_map(&p.k, a, a.k, a.hk, KD) || !la_map(&p.v, a, a.v, a.hv, a.VD))
      return cudaErrorInvalidValue;
    if (a.out_f32) p.o = p.v;  // unused: fp32 outputs are written from registers
    else if (!la_map(&p.o, a, a.out, a.H, a.VD)) return cudaErrorInvalidValue;
  }
  if (cores.p[0].nseg > 1) {
    cudaError_t e = launch_tc_mode<KD, 1>(job, n, stream);
    if (e == cudaSuccess) e = launch_la_prefix(cores, n, true, stream);
    if (e != cudaSuccess) return e;
  }
  for (int i = 0; i < n; ++i)
    if (cores.p[i].out_f32) return launch_tc_mode<KD, 2>(job, n, stream);
  return launch_tc_mode<KD, 0>(job, n, stream);
}

}  // namespace

bool la_tc_supported(const LaCore& a) {
  return a.bf16 && a.L >= a.tc_from && (a.KD == 64 || a.KD == 128) && (a.VD == 64 || a.VD == 128);
}

// Segments of a sequence: the count with the least modelled time, in units of one chunk of the full
// pass (2.0 us at 64 rows, 2.6 at 128): a wave of CTAs takes its chunks and 3 units to start and end (8.6 us a wave
// of one chunk at 64 rows, 11.5 at 128), a wave of the state pass 0.7 a chunk and 2, the prefix and the launches 4.
// Against the best count of 396 measured shapes (dims 64 and 128, 1 to 256 heads, 512 to 16384 tokens) the choice
// takes 0.4 % more on average and 11 % at most; without the waves' own cost it took 12 % and up to 4.8 times (b1 H80
// L4096 N = P = 64: 247 us in 32 segments, 69 in one).
void la_tc_plan(LaCore* a, int sms, int passes) {
  const int64_t nch = (a->L + LQ - 1) / LQ, units = a->b * a->H * (a->VD / LV) * passes;
  const int64_t most = nch < 32 ? nch : 32;
  double best = 0.0;
  int64_t segc = nch;
  for (int64_t s = 1; s <= most; ++s) {
    const int64_t per = (nch + s - 1) / s, n = (nch + per - 1) / per;
    const double waves = (double)((units * n + sms - 1) / sms), swaves = (double)((units * (n - 1) + sms - 1) / sms);
    const double t = waves * (per + 3.0) + (n > 1 ? swaves * (0.7 * per + 2.0) + 4.0 : 0.0);
    if (s == 1 || t < best) {
      best = t;
      segc = per;
    }
  }
  a->seg_tok = segc * LQ;
  a->nseg = (int)((nch + segc - 1) / segc);
}

cudaError_t launch_la_tc(const LaCores& cores, int n, cudaStream_t stream) {
  return cores.p[0].KD == 64 ? launch_tc_kd<64>(cores, n, stream) : launch_tc_kd<128>(cores, n, stream);
}

}  // namespace m3
