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
// Roundings: A' and the copy of S that q meets are bf16 (each moves the result by less than its own
// final rounding to bf16 does).  The state is an fp32 result, so its update must not lose bits: the
// weighted v enters as three bf16 parts (hi + mid + lo hold 24 bits) side by side as N = 192 columns
// of one product, so k is read once for all three, and a^128 is a two-float constant.
//
// Warp roles (20 warps; waits are mbarrier waits that sleep in the instruction, bounded by %globaltimer):
//   0      producer: TMA loads of q, k, v into two stages (128-byte swizzle)
//   1      MMA issue; tensor-memory allocation
//   4-7    scores: A from tensor memory -> A' back to tensor memory
//   8-11, 16-19  state and epilogue, 32 value columns each: the three parts of the update from tensor
//          memory, S in registers, bf16(S) to shared memory; then Yi, Ya from tensor memory -> out
//   12-15  weighted v: three bf16 parts to shared memory; zeroes rows past the sequence's length
// MMA order per chunk i: Yi(i), update(i), Ya(i), A(i+1).  The scores of i have Yi(i) and update(i) to
// finish in, the state of i+1 has Ya(i) and A(i+1), the weighted v of i+1 has all three.
#include <cuda.h>
#include <cudaTypedefs.h>

#include "m3_linattn.cuh"
#include "m3_ptx.cuh"

namespace m3 {
namespace {

constexpr int LQ = 128;  // tokens of a chunk
constexpr int LV = 64;   // value columns of a CTA
constexpr int L_PROD = 0, L_MMA = 1;
constexpr int L_THREADS = 640;
constexpr int LSC = LV / 2;  // state columns of one of the two state warpgroups
constexpr unsigned long long L_WAIT_NS = 2000000000ull;  // 2 s bound on any wait
constexpr int LBLK = 128 * 128;                          // one 64-column block of a 128-row tile, bytes
constexpr int L_MAXPOW = LQ + 1;

enum { LB_LD = 0, LB_FREE = 2, LB_SC = 4, LB_SP, LB_ST, LB_H, LB_VT, LB_Y, LB_YE, LB_DRAIN, LNBAR };

template <int KD>
struct LaCfg {
  static constexpr int TILE_K = (KD / 64) * LBLK;
  static constexpr int STAGE = 2 * TILE_K + LBLK;  // q, k, v
  static constexpr int OFF_VT = 2 * STAGE;         // three parts of the weighted v
  static constexpr int OFF_S = OFF_VT + 3 * LBLK;  // bf16(S), KD rows of 64
  static constexpr int OFF_POW = OFF_S + KD * 128;
  static constexpr int OFF_BAR = OFF_POW + ((L_MAXPOW * 4 + 15) & ~15);
  static constexpr int OFF_MISC = OFF_BAR + LNBAR * 8;
  static constexpr int SMEM = OFF_MISC + 32 + 1024;
  static constexpr uint32_t TM_A = 0, TM_AP = 128, TM_YI = 192, TM_YA = 256, TM_H = 320, TM_COLS = 512;
  static constexpr uint32_t ID_A = idesc_bf16(128, 128, false, false);
  static constexpr uint32_t ID_Y = idesc_bf16(128, LV, false, true);
  static constexpr uint32_t ID_H = idesc_bf16(KD, 3 * LV, true, true);
  static_assert(SMEM <= 227 * 1024, "shared memory");
};

__device__ __forceinline__ bool la_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
  if (mbar_try_wait_sleep(bar, parity, 1000000)) return true;
  const uint64_t t0 = globaltimer();
  while (!mbar_try_wait_sleep(bar, parity, 1000000)) {
    if (*abort_flag) return false;
    if (globaltimer() - t0 > L_WAIT_NS) {
      *abort_flag = 1;
      return false;
    }
  }
  return true;
}
__device__ __forceinline__ void la_drain(uint64_t* bar, uint32_t parity) {
  const uint64_t t0 = globaltimer();
  while (!mbar_try_wait_sleep(bar, parity, 1000000))
    if (globaltimer() - t0 > L_WAIT_NS) return;
}
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&v)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
               : "r"(taddr));
}
__device__ __forceinline__ void la_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// The valid chunks of a segment, in processing order: chunk(i), i < n; chunks [z0, z1) of it lie
// past the sequence's length.  A segment's tokens: those that are valid.
struct ChunkSpan {
  int64_t first, z0, z1, tokens;
  int n;
};
__device__ __forceinline__ ChunkSpan la_chunks(const LaCore& a, int seg, int64_t len) {
  const int64_t nch = (a.L + LQ - 1) / LQ, segc = a.seg_tok / LQ, nvc = (len + LQ - 1) / LQ;
  const int64_t p0 = seg * segc < nch ? seg * segc : nch, p1 = p0 + segc < nch ? p0 + segc : nch;
  ChunkSpan c;
  const int64_t lo = a.rev ? nch - p1 : p0, hi = a.rev ? nch - p0 : p1;  // chunks [lo, hi)
  const int64_t top = hi < nvc ? hi : nvc;
  c.n = top > lo ? (int)(top - lo) : 0;
  c.first = a.rev ? top - 1 : lo;
  c.z0 = top > lo ? top : lo;
  c.z1 = hi;
  const int64_t end = top * LQ < len ? top * LQ : len;
  c.tokens = c.n > 0 ? end - lo * LQ : 0;
  return c;
}

template <int KD, int MODE>
__global__ void __launch_bounds__(L_THREADS, 1)
    la_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                 const __grid_constant__ CUtensorMap tmV, const __grid_constant__ LaCore a) {
  using C = LaCfg<KD>;
  constexpr bool FULL = MODE == 0;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, wg = warp >> 2, q4 = warp & 3;
  const int vtiles = a.VD / LV;
  int64_t blk = blockIdx.x;
  const int vt = (int)(blk % vtiles);
  blk /= vtiles;
  const int nseg_grid = FULL ? a.nseg : a.nseg - 1;
  const int seg = (int)(blk % nseg_grid);
  const int64_t bh = blk / nseg_grid;
  const int bi = (int)(bh / a.H), h = (int)(bh % a.H);

  uint64_t* bar = reinterpret_cast<uint64_t*>(sm + C::OFF_BAR);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + C::OFF_MISC + 4);
  float* pw = reinterpret_cast<float*>(sm + C::OFF_POW);
  const uint32_t sBase = smem_u32(sm);
  auto sQ = [&](int s) { return sBase + (uint32_t)(s * C::STAGE); };
  auto sK = [&](int s) { return sBase + (uint32_t)(s * C::STAGE + C::TILE_K); };
  auto sV = [&](int s) { return sBase + (uint32_t)(s * C::STAGE + 2 * C::TILE_K); };
  const uint32_t sVT = sBase + C::OFF_VT, sS = sBase + C::OFF_S;

  // ---- setup
  if (warp == L_MMA) {
    tmem_alloc(tmem_slot, C::TM_COLS);
    tmem_relinquish();
  }
  if (tid == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bar[LB_LD + s], 1);
      mbar_init(&bar[LB_FREE + s], 1);
    }
    mbar_init(&bar[LB_SC], 1);
    mbar_init(&bar[LB_SP], 4);
    mbar_init(&bar[LB_ST], 8);
    mbar_init(&bar[LB_H], 1);
    mbar_init(&bar[LB_VT], 4);
    mbar_init(&bar[LB_Y], 1);
    mbar_init(&bar[LB_YE], 8);
    mbar_init(&bar[LB_DRAIN], 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  const float ld = a.log_decay[h];
  if (tid < L_MAXPOW) pw[tid] = (float)la_pow(ld, tid);
  const int64_t page = la_page_block(a.pages, a.npages, bi, a.status);
  const int64_t len = page < 0 ? 0 : la_len(a, bi);
  const ChunkSpan cs = la_chunks(a, seg, len);
  const int n = cs.n;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t lane_base = (uint32_t)(32 * q4) << 16;
  auto chunk = [&](int i) { return a.rev ? cs.first - i : cs.first + i; };
  auto valid = [&](int i) {  // tokens of chunk i within the length
    const int64_t left = len - chunk(i) * LQ;
    return left < LQ ? (int)left : LQ;
  };

  if (wg == 0) {
    if (warp == L_PROD) {
      // =============================================================== producer
      if (lane == 0) {
        const int gq = h / (a.H / a.hq), gk = h / (a.H / a.hk), gv = h / (a.H / a.hv);
        uint32_t ph = 0;  // phase bits of LB_FREE
        int done = 0;
        for (int i = 0; i < n; ++i) {
          const int s = i & 1;
          if (i >= 2) {
            if (!la_wait(&bar[LB_FREE + s], (ph >> s) & 1, abort_flag)) break;
            ph ^= 1u << s;
          }
          const int tok = (int)(chunk(i) * LQ);
          mbar_expect_tx(&bar[LB_LD + s], FULL ? C::STAGE : C::STAGE - C::TILE_K);
#pragma unroll
          for (int b = 0; b < KD / 64; ++b) {
            if constexpr (FULL) tma_load_4d(sQ(s) + b * LBLK, &tmQ, 64 * b, gq, tok, bi, &bar[LB_LD + s]);
            tma_load_4d(sK(s) + b * LBLK, &tmK, 64 * b, gk, tok, bi, &bar[LB_LD + s]);
          }
          tma_load_4d(sV(s), &tmV, LV * vt, gv, tok, bi, &bar[LB_LD + s]);
          ++done;
        }
        // every copy issued has landed before the CTA may exit
        for (int s = 0; s < 2; ++s) {
          const int k = (done + 1 - s) / 2;  // copies into stage s
          if (k > 0) la_drain(&bar[LB_LD + s], (uint32_t)((k - 1) & 1));
        }
      }
    } else if (warp == L_MMA && n > 0) {
      // =============================================================== MMA issue
      auto kdesc = [&](uint32_t base, int k) {  // K-major operand, K-step k of 16
        return sdesc(base + (uint32_t)(k >> 2) * LBLK + (uint32_t)(k & 3) * 32, 16, 1024);
      };
      auto mdesc = [&](uint32_t base, int k) { return sdesc(base + (uint32_t)k * 2048, LBLK, 1024); };  // MN-major
      uint32_t ph_ld = 0;
      auto scores = [&](int i) -> bool {
        const int s = i & 1;
        if (!la_wait(&bar[LB_LD + s], (ph_ld >> s) & 1, abort_flag)) return false;
        ph_ld ^= 1u << s;
        if constexpr (FULL) {
          tc_fence_after();
#pragma unroll
          for (int k = 0; k < KD / 16; ++k) mma_ss_w(tmem + C::TM_A, kdesc(sQ(s), k), kdesc(sK(s), k), C::ID_A, k > 0);
          mma_commit_w(&bar[LB_SC]);
        }
        return true;
      };
      bool ok = scores(0);
      for (int i = 0; ok && i < n; ++i) {
        const int s = i & 1;
        const uint32_t p = (uint32_t)(i & 1);
        ok = la_wait(&bar[LB_ST], p, abort_flag);
        if (FULL && ok && i > 0) ok = la_wait(&bar[LB_YE], p ^ 1, abort_flag);
        if (!ok) break;
        tc_fence_after();
        if constexpr (FULL) {
#pragma unroll
          for (int k = 0; k < KD / 16; ++k) mma_ss_w(tmem + C::TM_YI, kdesc(sQ(s), k), mdesc(sS, k), C::ID_Y, k > 0);
        }
        ok = la_wait(&bar[LB_VT], p, abort_flag);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int k = 0; k < LQ / 16; ++k) mma_ss_w(tmem + C::TM_H, mdesc(sK(s), k), mdesc(sVT, k), C::ID_H, k > 0);
        mma_commit_w(&bar[LB_H]);
        if constexpr (FULL) {
          ok = la_wait(&bar[LB_SP], p, abort_flag);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int k = 0; k < LQ / 16; ++k)
            mma_ts_w(tmem + C::TM_YA, tmem + C::TM_AP + 8 * k, mdesc(sV(s), k), C::ID_Y, k > 0);
          mma_commit_w(&bar[LB_Y]);
        }
        mma_commit_w(&bar[LB_FREE + s]);
        if (i + 1 < n) ok = scores(i + 1);
      }
      // every MMA issued has completed before tensor memory is released
      mma_commit_w(&bar[LB_DRAIN]);
      la_drain(&bar[LB_DRAIN], 0);
    }
  } else if (wg == 1) {
    if constexpr (FULL) {
      // =============================================================== scores
      const float sc = a.s_upd * a.s_out;
      uint64_t u[16];  // the columns' factors within a 32-column block
#pragma unroll
      for (int e = 0; e < 16; ++e)
        u[e] = a.rev ? f2(pw[2 * e], pw[2 * e + 1]) : f2(pw[31 - 2 * e], pw[30 - 2 * e]);
      for (int i = 0; i < n; ++i) {
        if (!la_wait(&bar[LB_SC], (uint32_t)(i & 1), abort_flag)) break;
        tc_fence_after();
        const int nv = valid(i);
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint32_t o[16];
          const int d = a.rev ? c - q4 : q4 - c;  // blocks between the row's and the column's
          if (d < 0) {
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = 0u;
          } else {
            uint32_t v[32];
            tmem_ld32(tmem + lane_base + C::TM_A + 32 * c, v);
            if (d > 0) {
              const float r = sc * pw[a.rev ? 32 * d - lane : 32 * d - 31 + lane];
              const uint64_t r2 = f2(r, r);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                float x, y;
                f2_split(f2_mul(f2_mul(f2(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1])), u[e]), r2), x, y);
                v[2 * e] = __float_as_uint(x);
                v[2 * e + 1] = __float_as_uint(y);
              }
            } else {
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) {
                const int dd = a.rev ? e - lane : lane - e;
                v[e] = dd >= 0 ? __float_as_uint(__uint_as_float(v[e]) * (sc * pw[dd < 0 ? 0 : dd])) : 0u;
              }
            }
            if (32 * c + 32 > nv) {  // columns past the length
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (32 * c + e >= nv) v[e] = 0u;
            }
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = pack_bf16(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1]));
          }
          tmem_st16(tmem + lane_base + C::TM_AP + 16 * c, o);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) la_arrive(&bar[LB_SP]);
      }
    }
  } else if (wg == 3) {
    // =============================================================== weighted v
    const int r = 32 * q4 + lane;  // token of the chunk
    uint32_t ph_ld = 0;
    for (int i = 0; i < n; ++i) {
      const int s = i & 1;
      if (!la_wait(&bar[LB_LD + s], (ph_ld >> s) & 1, abort_flag)) break;
      ph_ld ^= 1u << s;
      if (i > 0 && !la_wait(&bar[LB_H], (uint32_t)((i - 1) & 1), abort_flag)) break;  // the parts are read
      const int nv = valid(i);
      const uint32_t ro = (uint32_t)r * 128u;
      if (r < nv) {
        const float w = a.s_upd * pw[a.rev ? r + 1 : nv - 1 - r];
#pragma unroll 2
        for (int c = 0; c < 8; ++c) {
          const uint32_t off = ro + (uint32_t)((c ^ (r & 7)) << 4);
          float f[8];
          unpack8(lds128(sV(s) + off), f);
#pragma unroll
          for (int e = 0; e < 8; ++e) f[e] *= w;
#pragma unroll
          for (int part = 0; part < 3; ++part) {
            const uint4 p = pack8(f);
            sts128(sVT + part * LBLK + off, p);
            if (part < 2) {
              float g[8];
              unpack8(p, g);
#pragma unroll
              for (int e = 0; e < 8; ++e) f[e] -= g[e];  // exact
            }
          }
        }
      } else {
        // rows past the length: zero, so that nothing found there (infinities, NaN) meets a product
        const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          sts128(sV(s) + ro + 16 * c, zero);
#pragma unroll
          for (int b = 0; b < KD / 64; ++b) sts128(sK(s) + b * LBLK + ro + 16 * c, zero);
#pragma unroll
          for (int part = 0; part < 3; ++part) sts128(sVT + part * LBLK + ro + 16 * c, zero);
        }
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) la_arrive(&bar[LB_VT]);
    }
  } else {
    // =============================================================== state and epilogue
    // Two warpgroups, LSC value columns each.  Per chunk: the state after it (needed by the next chunk's Yi
    // and update) first, then the outputs of the chunk.
    const int c0 = wg == 2 ? 0 : LSC;  // first column, within the CTA's
    // accumulator row of this thread (M = 128: its lane; M = 64: lanes 0-15 of each quarter)
    const bool owner = KD == 128 || lane < 16;
    const int row = KD == 128 ? 32 * q4 + lane : 16 * q4 + (lane & 15);
    const int64_t col = LV * vt + c0;
    float S[LSC];
#pragma unroll
    for (int e = 0; e < LSC; ++e) S[e] = 0.0f;
    auto slot = [&](int s) { return a.ws + ((bh * a.nseg + s) * KD + row) * (int64_t)a.VD + col; };
    const int64_t sbase = (page * a.H + h) * (int64_t)KD * a.VD + row * a.s_i + col * a.s_j;
    auto store_slot = [&](int s) {
      float4* w = reinterpret_cast<float4*>(slot(s));
#pragma unroll
      for (int e = 0; e < LSC / 4; ++e) w[e] = make_float4(S[4 * e], S[4 * e + 1], S[4 * e + 2], S[4 * e + 3]);
    };
    if (owner && page >= 0) {
      if (seg == 0) {
        const bool from_ws = FULL && a.nseg > 1;
        if (from_ws || a.s_in) {
          const float* src = from_ws ? slot(0) : a.s_in + sbase;
          const int64_t sj = from_ws ? 1 : a.s_j;
#pragma unroll
          for (int e = 0; e < LSC; ++e) S[e] = src[e * sj];
        }
        if (!FULL) store_slot(0);
      } else if (FULL) {
        for (int m = 0; m < seg; ++m) {
          const float f = (float)la_pow(ld, la_chunks(a, m, len).tokens);
          const float4* z = reinterpret_cast<const float4*>(slot(m + 1));
#pragma unroll
          for (int e = 0; e < LSC / 4; ++e) {
            const float4 v = z[e];
            S[4 * e] = fmaf(f, S[4 * e], v.x);
            S[4 * e + 1] = fmaf(f, S[4 * e + 1], v.y);
            S[4 * e + 2] = fmaf(f, S[4 * e + 2], v.z);
            S[4 * e + 3] = fmaf(f, S[4 * e + 3], v.w);
          }
        }
      }
    }
    auto publish = [&]() {  // bf16(S), the B operand of Yi
      if constexpr (FULL) {
        if (owner) {
#pragma unroll
          for (int c = 0; c < LSC / 8; ++c) {
            float f[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = S[8 * c + e];
            sts128(sS + row * 128 + (((c + c0 / 8) ^ (row & 7)) << 4), pack8(f));
          }
        }
        fence_async_smem();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) la_arrive(&bar[LB_ST]);
    };
    // the decay of a full chunk as two floats: a long memory multiplies it in hundreds of times
    const float a128_lo = (float)(la_pow(ld, LQ) - (double)pw[LQ]);
    const int t = 32 * q4 + lane;  // token of the chunk whose outputs this thread writes
    auto out_row = [&](int64_t tok) { return (((int64_t)bi * a.L + tok) * a.H + h) * (int64_t)a.VD + col; };
    bool ok = true;
    if (n > 0) publish();
    for (int i = 0; i < n; ++i) {
      ok = la_wait(&bar[LB_H], (uint32_t)(i & 1), abort_flag);
      if (!ok) break;
      tc_fence_after();
      const int nv = valid(i);
      const float ghi = pw[nv], glo = nv == LQ ? a128_lo : 0.0f;
#pragma unroll
      for (int c = 0; c < LSC / 8; ++c) {
        uint32_t x[8], y[8], z[8];
        tmem_ld8(tmem + lane_base + C::TM_H + c0 + 8 * c, x);
        tmem_ld8(tmem + lane_base + C::TM_H + LV + c0 + 8 * c, y);
        tmem_ld8(tmem + lane_base + C::TM_H + 2 * LV + c0 + 8 * c, z);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float hsum = __uint_as_float(x[e]) + (__uint_as_float(y[e]) + __uint_as_float(z[e]));
          S[8 * c + e] = fmaf(ghi, S[8 * c + e], fmaf(glo, S[8 * c + e], hsum));
        }
      }
      if (i + 1 < n) publish();
      if constexpr (FULL) {
        ok = la_wait(&bar[LB_Y], (uint32_t)(i & 1), abort_flag);
        if (!ok) break;
        tc_fence_after();
        const int64_t tok = chunk(i) * LQ + t;
        const bool on = t < nv, write = tok < a.L;
        const float f = on ? a.s_out * pw[a.rev ? nv - 1 - t : t + 1] : 0.0f;
        const int64_t o = out_row(tok);
#pragma unroll
        for (int c = 0; c < LSC / 16; ++c) {
          uint32_t x[16], y[16];
          tmem_ld16(tmem + lane_base + C::TM_YI + c0 + 16 * c, x);
          tmem_ld16(tmem + lane_base + C::TM_YA + c0 + 16 * c, y);
          tmem_wait_ld();
          if (c == LSC / 16 - 1) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) la_arrive(&bar[LB_YE]);
          }
          float v[16];
#pragma unroll
          for (int e = 0; e < 16; ++e)
            v[e] = on ? fmaf(f, __uint_as_float(x[e]), __uint_as_float(y[e])) : 0.0f;
          if (write) {
            if (a.out_f32) {
              float4* p = reinterpret_cast<float4*>(static_cast<float*>(a.out) + o) + 4 * c;
#pragma unroll
              for (int e = 0; e < 4; ++e) p[e] = make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
            } else {
              uint4* p = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + o) + 2 * c;
              p[0] = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
              p[1] = make_uint4(pack_bf16(v[8], v[9]), pack_bf16(v[10], v[11]), pack_bf16(v[12], v[13]),
                                pack_bf16(v[14], v[15]));
            }
          }
        }
      }
    }
    if (ok && owner && page >= 0) {
      if (!FULL) {
        store_slot(seg + 1);
      } else if (seg == a.nseg - 1 && a.s_fin) {
#pragma unroll
        for (int e = 0; e < LSC; ++e) a.s_fin[sbase + e * a.s_j] = S[e];
      }
    }
    if constexpr (FULL) {  // chunks past the sequence's length
      for (int64_t j = cs.z0; j < cs.z1; ++j) {
        const int64_t tok = j * LQ + t;
        if (tok >= a.L) continue;
        const int e = a.out_f32 ? 4 : 2;
        uint4* p = reinterpret_cast<uint4*>(static_cast<char*>(a.out) + out_row(tok) * e);
        for (int c = 0; c < LSC * e / 16; ++c) p[c] = make_uint4(0, 0, 0, 0);
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

PFN_cuTensorMapEncodeTiled_v12000 la_encode_fn() {
  static std::once_flag once;
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  std::call_once(once, [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  });
  return fn;
}

// (b, L, heads, D) bf16 in boxes of 64 columns x 128 tokens of one head; tokens past L read as zero.
bool la_map(CUtensorMap* m, const LaCore& a, const void* base, int heads, int D) {
  auto fn = la_encode_fn();
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
cudaError_t launch_tc_mode(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, const LaCore& a,
                           cudaStream_t stream) {
  static SmemAttr attr;
  auto kern = la_tc_kernel<KD, MODE>;
  const cudaError_t e = attr.ensure(kern, LaCfg<KD>::SMEM);
  if (e != cudaSuccess) return e;
  const int64_t grid = a.b * a.H * (a.VD / LV) * (MODE == 0 ? a.nseg : a.nseg - 1);
  if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
  kern<<<(unsigned)grid, L_THREADS, LaCfg<KD>::SMEM, stream>>>(q, k, v, a);
  return cudaGetLastError();
}

template <int KD>
cudaError_t launch_tc_kd(const LaCore& a, cudaStream_t stream) {
  CUtensorMap q, k, v;
  if (!la_map(&q, a, a.q, a.hq, KD) || !la_map(&k, a, a.k, a.hk, KD) || !la_map(&v, a, a.v, a.hv, a.VD))
    return cudaErrorInvalidValue;
  if (a.nseg > 1) {
    const cudaError_t e = launch_tc_mode<KD, 1>(q, k, v, a, stream);
    if (e != cudaSuccess) return e;
  }
  return launch_tc_mode<KD, 0>(q, k, v, a, stream);
}

}  // namespace

bool la_tc_supported(const LaCore& a) {
  return a.bf16 && a.L > 0 && (a.KD == 64 || a.KD == 128) && (a.VD == 64 || a.VD == 128);
}

// Segments of a sequence: the count with the least modelled time, in units of one chunk of the full
// pass: waves of CTAs times chunks each, a state-pass chunk at half a unit, and four units for the
// second launch.
void la_tc_plan(LaCore* a, int sms) {
  const int64_t nch = (a->L + LQ - 1) / LQ, units = a->b * a->H * (a->VD / LV);
  const int64_t most = nch < 32 ? nch : 32;
  double best = 0.0;
  int64_t segc = nch;
  for (int64_t s = 1; s <= most; ++s) {
    const int64_t per = (nch + s - 1) / s, n = (nch + per - 1) / per;
    const double waves = (double)((units * n + sms - 1) / sms), swaves = (double)((units * (n - 1) + sms - 1) / sms);
    const double t = waves * per + (n > 1 ? 0.5 * swaves * per + 4.0 : 0.0);
    if (s == 1 || t < best) {
      best = t;
      segc = per;
    }
  }
  a->seg_tok = segc * LQ;
  a->nseg = (int)((nch + segc - 1) / segc);
}

cudaError_t launch_la_tc(const LaCore& a, cudaStream_t stream) {
  return a.KD == 64 ? launch_tc_kd<64>(a, stream) : launch_tc_kd<128>(a, stream);
}

}  // namespace m3
