// m3_linattn.cu -- linear attention with a decay per head: the recurrent core for every type and
// size (m3_linattn.cuh), the sum over a group's heads, and the one-token step.
//
// The core walks a sequence token by token with the state in registers: a thread holds 8 rows x 4
// columns of S as packed fp32 row pairs (f32x2), so a token costs three packed operations per two
// state elements (k v, the decayed update, the readout) and the operand rows come from shared
// memory as broadcast 128-bit loads.  LN = KD / 8 lanes share a column, their readouts are summed
// by a shuffle reduce-scatter.  It is bound by the latency of a token's chain (loads, updates,
// shuffles) at few warps and by the fp32 pipe, 6 KD VD flops a token and head, at many.  At b5 L1037 H6
// N40 P56 fp32 a call takes 56 us (its floor by bytes is 1.4 us), about 125 instructions a token and warp, half of
// them the packed arithmetic; 16 rows a thread took 168 registers and 97 us.
// Few sequences are cut into segments: every segment but the last is walked from a zero start (MODE 1)
// and leaves its end state, a prefix pass turns the end states into entering states, and the full pass
// starts from those.
//
// g itself is rounded to fp32, and a product of d of them is off by up to d 2^-24, all one way.  So the first
// token of every block of n <= 16 multiplies the state by g (1 + e + r) in g's place, e = e^{n log_decay} / g^n - 1
// taken in 64 bits and r what the rounding of that factor left in the blocks before: a call's decay over any
// number of blocks is off by half a step (2^-24) beside the factors within the last block, for a few operations a block.
// (Adding S e to k v^T at the first token, which leaves no rest at all, took 8 to 10 % more time.)
#include "m3_linattn.cuh"
#include "m3_ptx.cuh"

namespace m3 {
namespace {

constexpr int kTB = 16;       // tokens staged at once
constexpr int kMaxSeg = 64;   // segments of a sequence at most
constexpr int kLaWarps = 8;   // warps of a CTA at most

__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// Four consecutive values of a staged row.
template <bool BF16>
__device__ __forceinline__ float4 row4(const void* p, int i) {
  if constexpr (BF16) {
    const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p) + i);
    return make_float4(bf_lo(w.x), bf_hi(w.x), bf_lo(w.y), bf_hi(w.y));
  } else {
    return *reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
  }
}

template <bool BF16, bool OUT_F32, int LN, int MODE>
__global__ void __launch_bounds__(32 * kLaWarps) la_core_kernel(const __grid_constant__ LaCores job, int coltiles, int cols) {
  const LaCore& a = job.p[blockIdx.y];
  constexpr bool FULL = MODE == 0;
  constexpr int KDP = 8 * LN, CPW = 128 / LN, E = BF16 ? 2 : 4;
  using T = typename std::conditional<BF16, __nv_bfloat16, float>::type;
  extern __shared__ __align__(16) uint8_t sm[];
  const int bufsz = kTB * (2 * KDP + cols);                   // q, k, v of a token block, elements
  T* buf = reinterpret_cast<T*>(sm);                          // two of them
  float* ybuf = reinterpret_cast<float*>(sm + 2 * bufsz * E);  // [kTB][cols]
  const int tid = threadIdx.x, nthr = blockDim.x, warp = tid >> 5, lane = tid & 31, ln = lane % LN;
  unsigned blk = blockIdx.x;
  const int ct = (int)(blk % (unsigned)coltiles);
  blk /= (unsigned)coltiles;
  const unsigned nseg_grid = FULL ? a.nseg : a.nseg - 1;
  const int seg = (int)(blk % nseg_grid);
  const int bh = (int)(blk / nseg_grid);
  const int bi = bh / a.H, h = bh % a.H;
  const int c0 = ct * cols;                     // first column of the block
  const int cb = warp * CPW + (lane / LN) * 4;  // first column of the thread, within the block
  const int ncol = a.VD - c0 < cols ? a.VD - c0 : cols;
  const int64_t page = la_page_block(a.pages, a.npages, bi, a.status);
  const int len = page < 0 ? 0 : la_len(a, bi);
  const SegSpan sp = la_span(a, seg, len);
  const float ld = a.log_decay[h];
  // g and e^{n log_decay} / g^n - 1 of a full block and of the segment's last one, by one warp (64-bit exponentials
  // are slow to issue)
  __shared__ float factors[4];
  if (warp == 0) {
    const int e = lane == 0 ? 1 : lane == 1 ? kTB : (sp.tb - sp.ta) % kTB;
    const double w = la_pow(ld, e);
    double gi = (double)(float)__shfl_sync(kFull, w, 0), gp = 1.0;
    if (lane == 0) {
      factors[0] = (float)w;
      factors[3] = w > 1e-30 ? (float)(1.0 / w) : 0.0f;
    }
#pragma unroll
    for (int i = 1; i <= kTB; i *= 2) {
      if (e & i) gp *= gi;
      gi *= gi;
    }
    if (lane == 1 || lane == 2) factors[lane] = gp > 1e-30 ? (float)(w / gp - 1.0) : 0.0f;
  }

  // ---- the state entering the segment: rows 4 (ln + LN j) + e as pairs, columns cb..cb+3
  uint64_t S[4][4];
  auto row_of = [&](int rp) { return 4 * (ln + LN * (rp >> 1)) + 2 * (rp & 1); };
  auto slot = [&](int s) { return a.ws + ((int64_t)bh * a.nseg + s) * (a.KD * a.VD) + c0 + cb; };
  const int64_t sbase = (page * a.H + h) * (a.KD * a.VD) + (c0 + cb) * a.s_j;
#pragma unroll
  for (int rp = 0; rp < 4; ++rp)
#pragma unroll
    for (int c = 0; c < 4; ++c) S[rp][c] = 0;
  const bool has_col = cb < ncol;  // columns come in fours: VD is a multiple of 8
  auto put = [&](float* dst, int si, int sj, float f) {  // within one state: 32-bit offsets
#pragma unroll
    for (int rp = 0; rp < 4; ++rp)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int i = row_of(rp);
        float lo, hi;
        f2_split(S[rp][c], lo, hi);
        if (i < a.KD) {
          dst[i * si + c * sj] = f * lo;
          dst[(i + 1) * si + c * sj] = f * hi;
        }
      }
  };
  if (has_col && page >= 0) {
    if (FULL && a.nseg > 1) {
      const float* z = slot(seg);
#pragma unroll
      for (int rp = 0; rp < 4; ++rp) {
        const int i = row_of(rp);
        if (i >= a.KD) continue;
        const float4 lo = *reinterpret_cast<const float4*>(z + (int64_t)i * a.VD);
        const float4 hi = *reinterpret_cast<const float4*>(z + (int64_t)(i + 1) * a.VD);
        S[rp][0] = f2(lo.x, hi.x);
        S[rp][1] = f2(lo.y, hi.y);
        S[rp][2] = f2(lo.z, hi.z);
        S[rp][3] = f2(lo.w, hi.w);
      }
    } else if (seg == 0) {
      if (a.s_in) {
        const float* src = a.s_in + sbase;
        const int si = (int)a.s_i, sj = (int)a.s_j;
#pragma unroll
        for (int rp = 0; rp < 4; ++rp)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int i = row_of(rp);
            if (i < a.KD) S[rp][c] = f2(src[i * si + c * sj], src[(i + 1) * si + c * sj]);
          }
      }
      if (!FULL) put(slot(0), a.VD, 1, 1.0f);
    }
  }

  // ---- token blocks, in processing order; padding rows and columns of the buffers stay zero
  if (a.KD < KDP || ncol < cols)
    for (int i = tid; i < 2 * bufsz * E / 16; i += nthr) reinterpret_cast<uint4*>(sm)[i] = make_uint4(0, 0, 0, 0);
  __syncthreads();
  const float g = factors[0], ginv = factors[3];
  float left = 0.0f;  // of the decays' roundings so far, relative
  const int ntok = sp.tb - sp.ta;
  const int nblk = (ntok + kTB - 1) / kTB;
  const int gq = h / (a.H / a.hq), gk = h / (a.H / a.hk), gv = h / (a.H / a.hv);
  // token of position i of the segment
  auto token = [&](int i) { return a.rev ? sp.tb - 1 - i : sp.ta + i; };
  const int kc = a.KD * E / 16, vc = ncol * E / 16;  // 16-byte chunks of a row
  // A thread copies chunk lane & 15 (+ 16 j) of the rows warp * 2 + (lane >> 4) + 2 warps * i of a block.
  const int sl = lane & 15, sr = 2 * warp + (lane >> 4), sstep = nthr >> 4;
  const T* qg = static_cast<const T*>(a.q) + ((int64_t)bi * a.L * a.hq + gq) * a.KD;
  const T* kg = static_cast<const T*>(a.k) + ((int64_t)bi * a.L * a.hk + gk) * a.KD;
  const T* vg = static_cast<const T*>(a.v) + ((int64_t)bi * a.L * a.hv + gv) * a.VD + c0;
  const int64_t qs = (int64_t)a.hq * a.KD, ks = (int64_t)a.hk * a.KD, vs = (int64_t)a.hv * a.VD;
  constexpr int CE = 16 / E;  // elements of a chunk
  auto stage = [&](int blk_i, int s) {
    const int i0 = blk_i * kTB;
    const int nt = ntok - i0 < kTB ? ntok - i0 : kTB;
    T* bq = buf + s * bufsz;
    T* bk = bq + kTB * KDP;
    T* bv = bk + kTB * KDP;
    for (int t = sr; t < nt; t += sstep) {
      const int64_t tok = token(i0 + t);
      for (int ch = sl; ch < kc; ch += 16) {
        if (FULL) cp_async16(bq + t * KDP + ch * CE, qg + tok * qs + ch * CE);
        cp_async16(bk + t * KDP + ch * CE, kg + tok * ks + ch * CE);
      }
      for (int ch = sl; ch < vc; ch += 16) cp_async16(bv + t * cols + ch * CE, vg + tok * vs + ch * CE);
    }
  };
  // against time the first token of the sequence meets the incoming state undecayed
  const bool first = a.rev && sp.tb == len;
  const float u = a.s_upd;
  if (nblk > 0) stage(0, 0);
  cp_async_commit();
  for (int ib = 0; ib < nblk; ++ib) {
    const int s = ib & 1;
    if (ib + 1 < nblk) stage(ib + 1, s ^ 1);
    cp_async_commit();
    cp_async_wait<1>();
    __syncthreads();
    const int i0 = ib * kTB;
    const int nt = ntok - i0 < kTB ? ntok - i0 : kTB;
    const T* bq = buf + s * bufsz + 4 * ln;
    const T* bk = bq + kTB * KDP;
    const T* bv = buf + s * bufsz + 2 * kTB * KDP + cb;
    // the decay of the block's first token
    const bool plain = first && ib == 0;
    const float g1 = plain ? 1.0f : g, want = left + factors[nt == kTB ? 1 : 2], gh = fmaf(g1, want, g1);
    left = want - (gh - g1) * (plain ? 1.0f : ginv);
    // one token: the state's update, and this thread's share of the four readouts
    auto walk = [&](int t, float (&y)[4], bool head) {
      const float gt = head ? gh : g;
      const uint64_t g2 = f2(gt, gt);
      const float4 v4 = row4<BF16>(bv, t * cols);
      const uint64_t v2[4] = {f2(v4.x * u, v4.x * u), f2(v4.y * u, v4.y * u), f2(v4.z * u, v4.z * u),
                              f2(v4.w * u, v4.w * u)};
      uint64_t ya[4], yb[4];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float4 k4 = row4<BF16>(bk, t * KDP + 4 * LN * j);
        const uint64_t ka = f2(k4.x, k4.y), kb = f2(k4.z, k4.w);
        uint64_t qa = 0, qb = 0;
        if (FULL) {
          const float4 q4 = row4<BF16>(bq, t * KDP + 4 * LN * j);
          qa = f2(q4.x, q4.y);
          qb = f2(q4.z, q4.w);
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          S[2 * j][c] = f2_fma(S[2 * j][c], g2, f2_mul(ka, v2[c]));
          S[2 * j + 1][c] = f2_fma(S[2 * j + 1][c], g2, f2_mul(kb, v2[c]));
          if (FULL) {  // two short chains
            ya[c] = j == 0 ? f2_mul(qa, S[2 * j][c]) : f2_fma(qa, S[2 * j][c], ya[c]);
            yb[c] = j == 0 ? f2_mul(qb, S[2 * j + 1][c]) : f2_fma(qb, S[2 * j + 1][c], yb[c]);
          }
        }
      }
      if constexpr (FULL) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          float a0, a1, b0, b1;
          f2_split(ya[c], a0, a1);
          f2_split(yb[c], b0, b1);
          y[c] = (a0 + a1) + (b0 + b1);
        }
      }
    };
    // sum over the LN lanes of a column, two halving exchanges, then plain butterflies; lane ln then holds
    // `have` columns from `col`
    constexpr int have = LN >= 4 ? 1 : LN == 2 ? 2 : 4;
    const int col = (LN >= 2 && (ln & (LN / 2)) ? 2 : 0) + (LN >= 4 && (ln & (LN / 4)) ? 1 : 0);
    auto reduce = [&](float (&y)[4]) {
      if constexpr (LN >= 2) {
        const bool up = ln & (LN / 2);
        const float s0 = up ? y[0] : y[2], s1 = up ? y[1] : y[3];
        y[0] = (up ? y[2] : y[0]) + __shfl_xor_sync(kFull, s0, LN / 2);
        y[1] = (up ? y[3] : y[1]) + __shfl_xor_sync(kFull, s1, LN / 2);
      }
      if constexpr (LN >= 4) {
        const bool up = ln & (LN / 4);
        const float s0 = up ? y[0] : y[1];
        y[0] = (up ? y[1] : y[0]) + __shfl_xor_sync(kFull, s0, LN / 4);
      }
#pragma unroll
      for (int o = LN / 8; o > 0; o >>= 1) y[0] += __shfl_xor_sync(kFull, y[0], o);
    };
    auto keep = [&](int t, const float (&y)[4]) {
      if (LN < 8 || (ln & (LN / 4 - 1)) == 0) {
#pragma unroll
        for (int c = 0; c < have; ++c) ybuf[t * cols + cb + col + c] = a.s_out * y[c];
      }
    };
    // four tokens at a time: their sums over the lanes overlap (one by one a token took 400 cycles)
    int t = 0;
#pragma unroll 1
    for (; t + 4 <= nt; t += 4) {
      float y[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) walk(t + i, y[i], i == 0 && t == 0);
      if constexpr (FULL) {
#pragma unroll
        for (int i = 0; i < 4; ++i) reduce(y[i]);
#pragma unroll
        for (int i = 0; i < 4; ++i) keep(t + i, y[i]);
      }
    }
#pragma unroll 1
    for (; t < nt; ++t) {
      float y[4];
      walk(t, y, t == 0);
      if constexpr (FULL) {
        reduce(y);
        keep(t, y);
      }
    }
    __syncthreads();  // the block's readouts are complete, its operands read
    if constexpr (FULL) {
      for (int t = sr; t < nt; t += sstep)
        for (int c = 4 * sl; c < ncol; c += 64) {
          const float4 y = *reinterpret_cast<const float4*>(ybuf + t * cols + c);
          const int64_t o = (((int64_t)bi * a.L + token(i0 + t)) * a.H + h) * a.VD + c0 + c;
          if constexpr (OUT_F32) *reinterpret_cast<float4*>(static_cast<float*>(a.out) + o) = y;
          else *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + o) = make_uint2(pack_bf16(y.x, y.y), pack_bf16(y.z, y.w));
        }
      // ybuf is rewritten after the next block's first barrier
    }
  }
  cp_async_wait<0>();
  if constexpr (FULL) {  // tokens past the sequence's length
    for (int t = (sp.tb > sp.lo ? sp.tb : sp.lo) + sr; t < sp.hi; t += sstep)
      for (int c = 4 * sl; c < ncol; c += 64) {
        const int64_t o = (((int64_t)bi * a.L + t) * a.H + h) * a.VD + c0 + c;
        if constexpr (OUT_F32) *reinterpret_cast<float4*>(static_cast<float*>(a.out) + o) = make_float4(0, 0, 0, 0);
        else *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + o) = make_uint2(0, 0);
      }
  }

  // ---- the state left behind
  if (!has_col || page < 0) return;
  if (!FULL) put(slot(seg + 1), a.VD, 1, 1.0f);
  else if (seg == a.nseg - 1 && a.s_fin)  // against time: decayed once more past the first token
    put(a.s_fin + sbase, (int)a.s_i, (int)a.s_j, a.rev && len > 0 ? g : 1.0f);
}

// The states entering the segments: slot m + 1 holds the end state of segment m from a zero start (segment 0:
// from slot 0) and becomes the state entering segment m + 1.  One thread per four state elements, the
// segments in order; the loads do not wait for the sums.
__global__ void __launch_bounds__(128) la_prefix_kernel(const __grid_constant__ LaCores job, int per, int tc) {
  const LaCore& a = job.p[blockIdx.z];
  const int bh = blockIdx.x, e4 = blockIdx.y * 128 + threadIdx.x;
  const int bi = bh / a.H, h = bh % a.H;
  __shared__ float f[kMaxSeg];  // the decay over each segment
  if (threadIdx.x < a.nseg) {
    const int len = la_len(a, bi), m = threadIdx.x;
    int e;
    if (tc) {
      e = la_chunks(a, m, len).tokens;
    } else {
      const SegSpan sp = la_span(a, m, len);
      // (against time, the sequence's first token takes the incoming state undecayed)
      e = sp.tb - sp.ta - (a.rev && sp.tb == len && sp.tb > sp.ta);
    }
    f[m] = (float)la_pow(a.log_decay[h], e);
  }
  float4* z = reinterpret_cast<float4*>(a.ws) + (int64_t)bh * a.nseg * per + e4;
  __syncthreads();
  if (e4 >= per) return;
  float4 s = z[per];
  constexpr int U = 8;
  for (int m0 = 1; m0 < a.nseg - 1; m0 += U) {
    float4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (m0 + u < a.nseg - 1) v[u] = z[(int64_t)(m0 + u + 1) * per];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int m = m0 + u;
      if (m < a.nseg - 1) {
        s = make_float4(fmaf(f[m], s.x, v[u].x), fmaf(f[m], s.y, v[u].y), fmaf(f[m], s.z, v[u].z), fmaf(f[m], s.w, v[u].w));
        z[(int64_t)(m + 1) * per] = s;
      }
    }
  }
}

// out (rows, G, D) = sum over the H / G heads of a group of part (rows, H, D), in head order.
template <bool BF16>
__global__ void __launch_bounds__(256) la_head_sum_kernel(int64_t n4, int H, int G, int D4, const float4* part0, void* out0, const float4* part1, void* out1) {
  const float4* part = blockIdx.y ? part1 : part0;
  void* out = blockIdx.y ? out1 : out0;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n4) return;
  const int d = (int)(i % D4);
  const int64_t rg = i / D4;  // (row, group)
  const int per = H / G;
  const float4* p = part + rg * per * D4 + d;
  float4 s = make_float4(0, 0, 0, 0);
#pragma unroll 4
  for (int k = 0; k < per; ++k) {
    const float4 v = __ldcs(p + (int64_t)k * D4);
    s.x += v.x;
    s.y += v.y;
    s.z += v.z;
    s.w += v.w;
  }
  if constexpr (BF16) {
    reinterpret_cast<uint2*>(out)[i] = make_uint2(pack_bf16(s.x, s.y), pack_bf16(s.z, s.w));
  } else {
    reinterpret_cast<float4*>(out)[i] = s;
  }
}

// One token: S <- g S + k v^T, y = scale S^T q.  A CTA takes COLS columns of one (row, head) state:
// COLS / 4 lanes read a state row's segment, the other threads share the rows, and the column sums meet in
// shared memory.  Bound by HBM: the state is read and written once.  The state's loads are issued
// before the page is checked against the earlier rows' (the check decides what is stored, not what is
// read), and marked as streaming: b128 H32 N = P = 128 takes 86 us (6.3 TB/s, 96 % of the measured copy
// rate), 94 without the mark, 98 with the check first; b1 2.1 us and 3.9 with the check first.
constexpr int kStepThreads = 128;

template <bool BF16, int ITER, int COLS>
__global__ void __launch_bounds__(kStepThreads) la_step_kernel(const LaStep a, int tiles) {
  constexpr int LC = COLS / 4, RG = kStepThreads / LC;  // lanes of a row segment, row groups
  __shared__ float4 part[4][LC];
  const int tid = threadIdx.x, c4 = tid % LC, rg = tid / LC, warp = tid >> 5, lane = tid & 31;
  const unsigned tile = blockIdx.x % (unsigned)tiles, bh = blockIdx.x / (unsigned)tiles;
  const int bi = (int)(bh / (unsigned)a.H), h = (int)(bh % (unsigned)a.H);
  const int p0 = tile * COLS + 4 * c4;
  const bool on = p0 < a.P;
  const int64_t page = a.pages ? a.pages[bi] : bi;
  const bool there = page >= 0 && (!a.pages || page < a.npages);
  float* S = a.state + (page * a.H + h) * (int64_t)a.N * a.P + p0;
  float4 s[ITER];
#pragma unroll
  for (int i = 0; i < ITER; ++i) {
    const int n = rg + RG * i;
    s[i] = (on && there && n < a.N) ? __ldcs(reinterpret_cast<const float4*>(S + (int64_t)n * a.P)) : make_float4(0, 0, 0, 0);
  }
  const int64_t yi = (int64_t)bh * a.P + p0;
  const int64_t kq = ((int64_t)bi * a.G + h / (a.H / a.G)) * a.N;
  float v[4], k[ITER], q[ITER];
#pragma unroll
  for (int c = 0; c < 4; ++c) v[c] = on ? load_in<BF16>(a.v, yi + c) : 0.0f;
#pragma unroll
  for (int i = 0; i < ITER; ++i) {
    const int n = rg + RG * i;
    k[i] = n < a.N ? load_in<BF16>(a.k, kq + n) : 0.0f;
    q[i] = n < a.N ? load_in<BF16>(a.q, kq + n) : 0.0f;
  }
  // the decay as two floats: a long memory multiplies it in once a token
  const double gd = exp((double)a.log_decay[h]);
  const float g = (float)gd, gl = (float)(gd - (double)g);
  if (a.pages && la_page_block(a.pages, a.npages, bi, a.status) < 0) {
    if (on && rg == 0)
#pragma unroll
      for (int c = 0; c < 4; ++c) store_out<BF16>(a.y, yi + c, 0.0f);
    return;
  }
  float4 y = make_float4(0, 0, 0, 0);
#pragma unroll
  for (int i = 0; i < ITER; ++i) {
    const int n = rg + RG * i;
    s[i].x = fmaf(g, s[i].x, fmaf(gl, s[i].x, k[i] * v[0]));
    s[i].y = fmaf(g, s[i].y, fmaf(gl, s[i].y, k[i] * v[1]));
    s[i].z = fmaf(g, s[i].z, fmaf(gl, s[i].z, k[i] * v[2]));
    s[i].w = fmaf(g, s[i].w, fmaf(gl, s[i].w, k[i] * v[3]));
    if (on && n < a.N) __stcs(reinterpret_cast<float4*>(S + (int64_t)n * a.P), s[i]);
    y.x = fmaf(q[i], s[i].x, y.x);
    y.y = fmaf(q[i], s[i].y, y.y);
    y.z = fmaf(q[i], s[i].z, y.z);
    y.w = fmaf(q[i], s[i].w, y.w);
  }
#pragma unroll
  for (int o = LC; o < 32; o <<= 1) {
    y.x += __shfl_xor_sync(kFull, y.x, o);
    y.y += __shfl_xor_sync(kFull, y.y, o);
    y.z += __shfl_xor_sync(kFull, y.z, o);
    y.w += __shfl_xor_sync(kFull, y.w, o);
  }
  if (lane < LC) part[warp][lane] = y;
  __syncthreads();
  if (tid < LC && on) {
    float o[4] = {0, 0, 0, 0};
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const float4 f = part[w][tid];
      o[0] += f.x;
      o[1] += f.y;
      o[2] += f.z;
      o[3] += f.w;
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) store_out<BF16>(a.y, yi + c, a.scale * o[c]);
  }
}

int sm_count() {
  int dev = 0, n = 148;
  if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
  return n;
}

int lanes_of(int KD) {
  int ln = 1;
  while (8 * ln < KD) ln *= 2;
  return ln;
}

// Columns and warps of a CTA: the value dim over as few CTAs of at most kLaWarps warps as it takes.
int warps_of(const LaCore& a) {
  const int cpw = 128 / lanes_of(a.KD), need = (a.VD + cpw - 1) / cpw;
  const int ctas = (need + kLaWarps - 1) / kLaWarps, warps = (need + ctas - 1) / ctas;
  // eight columns at least to a step: a CTA's columns start on 16 bytes in bf16 (above 128 rows a warp has four)
  return cpw < 8 ? (warps + 1) & ~1 : warps;
}
int cols_of(const LaCore& a) { return warps_of(a) * (128 / lanes_of(a.KD)); }

// Segments of a sequence: enough for 16 warps per SM (about what the registers allow), each at
// least 32 tokens long so that the walk outweighs reading the earlier segments' states.  Against the best count of
// 320 measured shapes (state 16 x 24 to 128 x 128, 1 to 512 heads, 64 to 4096 tokens) that takes 12 % more on average
// and 57 % at most (64 tokens of 64 heads in two segments: 37 us, 24 in one).
void plan_core(LaCore* a, int passes) {
  if (la_tc_supported(*a)) return la_tc_plan(a, sm_count(), passes);
  const int cols = cols_of(*a);
  const int64_t warps = a->b * a->H * ((a->VD + cols - 1) / cols) * warps_of(*a) * passes;
  int64_t nseg = warps > 0 ? (int64_t)sm_count() * 16 / warps : 1;
  const int64_t most = a->L / 32;
  if (nseg > most) nseg = most;
  if (nseg > kMaxSeg) nseg = kMaxSeg;
  if (nseg < 2) nseg = 1;
  a->seg_tok = (a->L + nseg - 1) / nseg;
  if (a->seg_tok < 1) a->seg_tok = 1;
  a->nseg = (int)(a->L > 0 ? (a->L + a->seg_tok - 1) / a->seg_tok : 1);
}

template <bool BF16, bool OUT_F32, int LN, int MODE>
cudaError_t launch_core_cfg(const LaCores& job, int n, cudaStream_t stream) {
  const LaCore& a = job.p[0];
  const int cols = cols_of(a);
  const int bytes = 2 * kTB * (2 * 8 * LN + cols) * (BF16 ? 2 : 4) + kTB * cols * 4;
  static SmemAttr attr;
  auto k = la_core_kernel<BF16, OUT_F32, LN, MODE>;
  const cudaError_t e = attr.ensure(k, bytes);
  if (e != cudaSuccess) return e;
  const int tiles = (a.VD + cols - 1) / cols;
  const int64_t grid = a.b * a.H * tiles * (MODE == 0 ? a.nseg : a.nseg - 1);
  if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
  k<<<dim3((unsigned)grid, (unsigned)n), 32 * warps_of(a), bytes, stream>>>(job, tiles, cols);
  return cudaGetLastError();
}

template <bool BF16, bool OUT_F32, int LN>
cudaError_t launch_core_ln(const LaCores& job, int n, cudaStream_t stream) {
  if (job.p[0].nseg > 1) {
    cudaError_t e = launch_core_cfg<BF16, BF16 ? false : true, LN, 1>(job, n, stream);
    if (e == cudaSuccess) e = launch_la_prefix(job, n, false, stream);
    if (e != cudaSuccess) return e;
  }
  return launch_core_cfg<BF16, OUT_F32, LN, 0>(job, n, stream);
}

template <bool BF16, bool OUT_F32>
cudaError_t launch_core_type(const LaCores& job, int n, cudaStream_t stream) {
  switch (lanes_of(job.p[0].KD)) {
    case 1: return launch_core_ln<BF16, OUT_F32, 1>(job, n, stream);
    case 2: return launch_core_ln<BF16, OUT_F32, 2>(job, n, stream);
    case 4: return launch_core_ln<BF16, OUT_F32, 4>(job, n, stream);
    case 8: return launch_core_ln<BF16, OUT_F32, 8>(job, n, stream);
    case 16: return launch_core_ln<BF16, OUT_F32, 16>(job, n, stream);
    default: return launch_core_ln<BF16, OUT_F32, 32>(job, n, stream);
  }
}

template <int ITER, int COLS>
cudaError_t launch_step_cfg(const LaStep& a, cudaStream_t stream) {
  const int tiles = (a.P + COLS - 1) / COLS;
  const int64_t grid = a.b * a.H * tiles;
  if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
  if (a.bf16) la_step_kernel<true, ITER, COLS><<<(unsigned)grid, kStepThreads, 0, stream>>>(a, tiles);
  else la_step_kernel<false, ITER, COLS><<<(unsigned)grid, kStepThreads, 0, stream>>>(a, tiles);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_la_prefix(const LaCores& job, int n, bool tc, cudaStream_t stream) {
  const LaCore& a = job.p[0];
  if (a.nseg < 3) return cudaSuccess;  // slot 1 is the end state of segment 0 already
  const int per = a.KD * a.VD / 4;
  la_prefix_kernel<<<dim3((unsigned)(a.b * a.H), (unsigned)((per + 127) / 128), (unsigned)n), 128, 0, stream>>>(job, per, tc);
  return cudaGetLastError();
}

// A chunk costs the tensor cores the same for one token as for 128, 9 us a wave of CTAs at 64 rows and 12 at 128, the
// recurrent core 4 to 7 us and 0.2 to 0.3 a token while the SMs have room for its warps.  Measured, recurrent against
// tensor cores in us: one wave, b1 H24 64/64 at L16 7.4 and 9.0, L32 11 and 9; 128/128 at L16 10.5 and 12.4, L32 15
// and 12.4.  More waves: b32 H32 64/64 at L48 49 and 60, L64 62 and 61 (b8: 19 and 18, 35 and 19); 128/128 at L32
// 143 and 160, L48 191 and 162 (b8: 44 and 47, 57 and 47).  Gradients of own heads likewise: b1 H24 64/64 at L16 7.2
// and 9.4, b32 H32 at L48 130 and 146, L64 168 and 148; 128/128 b8 H32 at L32 96 and 92.  Gradients of shared heads
// take the recurrent core two launches and a sum: b1 H24 G1 64/64 at L8 15 and 15, L16 19 and 14; 128/128 20 and 19
// at L12; with more waves b32 H32 G1 64/64 at L48 142 and 172, 128/128 b8 H32 G1 at L32 105 and 109.
int la_tc_from(const LaCore& a, int passes, bool shares) {
  if (a.b * a.H * ((a.VD + 63) / 64) * passes > sm_count()) return a.KD <= 64 ? 49 : 33;
  return shares ? 13 : 25;
}

bool la_alike(const LaCore& a, const LaCore& b) {
  const bool tc = la_tc_supported(a);
  return tc == la_tc_supported(b) && a.KD == b.KD && a.VD == b.VD && (tc || a.out_f32 == b.out_f32);
}

namespace {
size_t pass_ws_bytes(const LaCore& a) {  // of a planned pass
  return a.nseg > 1 ? sizeof(float) * (size_t)(a.b * a.H) * a.nseg * a.KD * a.VD : 0;
}
}  // namespace

size_t la_group_ws_bytes(const LaCore& a0, int n) {
  LaCore a = a0;
  plan_core(&a, n);
  return n * pass_ws_bytes(a);
}

cudaError_t launch_la_group(LaCores* job, int n, void* ws, size_t ws_bytes, cudaStream_t stream) {
  for (int i = 0; i < n; ++i) {
    plan_core(&job->p[i], n);
    job->p[i].ws = static_cast<float*>(ws) + i * (pass_ws_bytes(job->p[i]) / sizeof(float));
  }
  const LaCore& a = job->p[0];
  if (n * pass_ws_bytes(a) > ws_bytes) return cudaErrorInvalidValue;
  if (la_tc_supported(a)) return launch_la_tc(*job, n, stream);
  if (!a.bf16) return launch_core_type<false, true>(*job, n, stream);
  return a.out_f32 ? launch_core_type<true, true>(*job, n, stream) : launch_core_type<true, false>(*job, n, stream);
}

cudaError_t launch_la_head_sum(int64_t rows, int H, int G, int D, int bf16, const float* const* part, void* const* out,
                               int n, cudaStream_t stream) {
  const int64_t n4 = rows * G * (D / 4);
  if (n4 == 0) return cudaSuccess;
  const int64_t grid = (n4 + 255) / 256;
  if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
  const float4* p0 = reinterpret_cast<const float4*>(part[0]);
  const float4* p1 = reinterpret_cast<const float4*>(part[n - 1]);
  const dim3 g((unsigned)grid, (unsigned)n);
  if (bf16) la_head_sum_kernel<true><<<g, 256, 0, stream>>>(n4, H, G, D / 4, p0, out[0], p1, out[n - 1]);
  else la_head_sum_kernel<false><<<g, 256, 0, stream>>>(n4, H, G, D / 4, p0, out[0], p1, out[n - 1]);
  return cudaGetLastError();
}

// Columns of a CTA: 32, twice as many with at most 64 rows once that still gives every SM four CTAs (half the CTAs,
// the same bytes in flight each; b61 H24 N = P = 64: 7.0 us against 7.8; b1 H32 N = P = 128 with 32: 2.1 us against
// 2.6 with 64).
cudaError_t launch_la_step(const LaStep& a, cudaStream_t stream) {
  if (a.N <= 64) {
    if (a.b * a.H * ((a.P + 63) / 64) >= 4 * (int64_t)sm_count()) return launch_step_cfg<8, 64>(a, stream);
    return launch_step_cfg<4, 32>(a, stream);
  }
  if (a.N <= 128) return launch_step_cfg<8, 32>(a, stream);
  return launch_step_cfg<16, 32>(a, stream);
}

}  // namespace m3
