// m3_linattn.cuh -- linear attention with a decay per head: what its kernels share.
//
// One operator serves the forward pass and all three gradients.  Per (batch, head), over the
// tokens in time order (rev = 0) or against it (rev = 1), with g = e^{log_decay},
//   S <- g S + s_upd k_t v_t^T            (KD x VD, fp32)
//   out_t = s_out S^T q_t
// forward:  y  = (q, k, v) in time order,  S from state_in, left in state_out
// gradients: dq = (dy, v, k) in time order, S^T from state_in
//            dk = (v, dy, q) against time,  from dstate_out^T
//            dv = (k, q, dy) against time,  from dstate_out, left in dstate_in
// Against time the incoming state meets the last token undecayed (dL/dS_{L-1} includes
// dstate_out itself) and the state left behind is decayed once more (S_0 = g S_{-1} + ...).
#pragma once

#include "m3_common.cuh"

namespace m3 {

struct LaCore {
  int64_t b, L;
  int H, KD, VD;
  const void *q, *k, *v;  // (b, L, hq | hk | hv, KD | KD | VD); head h of the pass reads h / (H / hx)
  int hq, hk, hv;
  int bf16;               // operands bf16 (else fp32)
  int out_f32;            // out fp32 (else bf16)
  void* out;              // (b, L, H, VD)
  int rev;
  float s_upd, s_out;
  const float* log_decay;  // (H)
  const int32_t* lens;     // (b) or null
  const int32_t* pages;    // (b) or null: the state row of each batch row
  int64_t npages;
  const float* s_in;       // state row + head * KD * VD + i * s_i + j * s_j (key index i, value index j); may be null
  float* s_fin;            // the same layout; may be null, may be s_in
  int64_t s_i, s_j;
  int tc_from;             // the fewest tokens that the tensor-core form takes (its chunk costs the same for one as for 128)
  int nseg;                // segments of a sequence walked in parallel
  int64_t seg_tok;         // tokens of a segment (in processing order)
  float* ws;               // (b * H, nseg, KD, VD) when nseg > 1: slot 0 the incoming state, slot m + 1
                           // the end state of segment m from a zero start (segment 0: from slot 0), then
                           // the state entering segment m + 1
  int* status;
};

// Token indices fit 32 bits (L is at most 2^31 - 256); 64-bit divisions, repeated 64-bit exponentials and
// unrolled set-up code are kept out of the kernels' prologues, where an instruction is fetched for one use.
// Tokens of batch row bi that are read.
__device__ __forceinline__ int la_len(const LaCore& a, int bi) {
  const int L = (int)a.L;
  if (!a.lens) return L;
  const int n = a.lens[bi];
  return n < 0 ? 0 : n > L ? L : n;
}
// g^e for a whole exponent e >= 0, rounded once to fp32: computed in 64 bits, so that distant tokens keep
// their weight to fp32 accuracy.  g = 0 (log_decay = -inf) keeps g^0 = 1.
static __device__ __noinline__ double la_pow(float log_decay, int e) {
  return e <= 0 ? 1.0 : exp((double)log_decay * (double)e);
}
// Tokens of segment m: [lo, hi) of the padded sequence, and how many of them are valid.
struct SegSpan {
  int lo, hi, ta, tb;
};
__device__ __forceinline__ SegSpan la_span(const LaCore& a, int m, int len) {
  SegSpan s;
  const unsigned L = (unsigned)a.L, seg = (unsigned)a.seg_tok;
  const unsigned q0 = (unsigned)m * seg, p0 = q0 < L ? q0 : L, p1 = L - p0 > seg ? p0 + seg : L;
  s.lo = (int)(a.rev ? L - p1 : p0);
  s.hi = (int)(a.rev ? L - p0 : p1);
  s.ta = s.lo < len ? s.lo : len;
  s.tb = s.hi < len ? s.hi : len;
  return s;
}
constexpr int kLaChunk = 128;  // tokens of a chunk of the tensor-core form
// The valid chunks of a segment, in processing order: chunk(i), i < n; chunks [z0, z1) of it lie
// past the sequence's length.  A segment's tokens: those that are valid.
struct ChunkSpan {
  int first, z0, z1, tokens, n;
};
__device__ __forceinline__ ChunkSpan la_chunks(const LaCore& a, int seg, int len) {
  const int nch = ((int)a.L + kLaChunk - 1) / kLaChunk, segc = (int)a.seg_tok / kLaChunk;
  const int nvc = (len + kLaChunk - 1) / kLaChunk;
  const int p0 = seg * segc < nch ? seg * segc : nch, p1 = p0 + segc < nch ? p0 + segc : nch;
  ChunkSpan c;
  const int lo = a.rev ? nch - p1 : p0, hi = a.rev ? nch - p0 : p1;  // chunks [lo, hi)
  const int top = hi < nvc ? hi : nvc;
  c.n = top > lo ? top - lo : 0;
  c.first = a.rev ? top - 1 : lo;
  c.z0 = top > lo ? top : lo;
  c.z1 = hi;
  const int end = top * kLaChunk < len ? top * kLaChunk : len;
  c.tokens = c.n > 0 ? end - lo * kLaChunk : 0;
  return c;
}
// The state row of batch row bi, or -1 for a row without one: a negative page (padding), a page past the
// pool or a page that an earlier row of the batch holds already (both recorded in the status word).
// Every thread of the block calls it; the same answer goes to all of them.
__device__ __forceinline__ int64_t la_page_block(const int32_t* pages, int64_t npages, int bi, int* status) {
  if (!pages) return bi;
  const int p = pages[bi];
  if (p < 0) return -1;
  int bad = p >= npages;
  for (int j = threadIdx.x; j < bi; j += blockDim.x) bad |= pages[j] == p;
  if (__syncthreads_or(bad)) {
    if (threadIdx.x == 0) set_status(status, M3_ERR_STATE);
    return -1;
  }
  return p;
}

// Launchers.
bool la_tc_supported(const LaCore& a);     // the tensor-core form takes this pass
int la_tc_from(const LaCore& a, int passes, bool shares);  // the fewest tokens for which it should (LaCore::tc_from)
void la_tc_plan(LaCore* a, int sms, int passes);
// Passes that one launch can take together, up to three of them (the gradients of a layer): their kernels fill the
// machine side by side, and a chain of launches is paid once.
struct LaCores {
  LaCore p[3];
};
bool la_alike(const LaCore& a, const LaCore& b);
size_t la_group_ws_bytes(const LaCore& a, int n);  // scratch of n passes like this one (plans their segments)
cudaError_t launch_la_group(LaCores* cores, int n, void* ws, size_t ws_bytes, cudaStream_t stream);
cudaError_t launch_la_tc(const LaCores& cores, int n, cudaStream_t stream);                // planned, scratch set
cudaError_t launch_la_prefix(const LaCores& cores, int n, bool tc, cudaStream_t stream);  // entering states from end states
// out[i] (rows, G, D) = the sums over a group's heads of part[i] (rows, H, D), i < n <= 2
cudaError_t launch_la_head_sum(int64_t rows, int H, int G, int D, int bf16, const float* const* part, void* const* out,
                               int n, cudaStream_t stream);
struct LaStep {
  int64_t b;
  int H, G, N, P, bf16;
  const void *q, *k, *v;
  const float* log_decay;
  float scale;
  float* state;
  int64_t npages;
  const int32_t* pages;
  void* y;
  int* status;
};
cudaError_t launch_la_step(const LaStep& a, cudaStream_t stream);

cudaError_t launch_pages_copy(const m3_pages& pg, int64_t n, const int32_t* src, const int32_t* dst, int* status,
                              cudaStream_t stream);
cudaError_t launch_pages_fork(const m3_pages& pg, int32_t* live, int64_t n, const int32_t* src, int32_t* dst,
                              int* status, cudaStream_t stream);
cudaError_t launch_pages_free(int64_t npages, int32_t* live, int64_t n, const int32_t* idx, int* status,
                              cudaStream_t stream);
cudaError_t launch_pages_compact(const m3_pages& pg, int32_t* live, int32_t* map, int32_t* order, int32_t* count,
                                 cudaStream_t stream);

}  // namespace m3
