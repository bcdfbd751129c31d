// kv_attention.cuh -- attention of new tokens over the mixed-precision K/V cache (decode).
//
// "Search your block floating-point scales!" (gist.science summary of arXiv 2605.12464),
// ScaleSearchAttention > attention-sink-aware mixed-precision caching: the cache that nvfp4_kv_append
// fills is read where it lies.  Per sequence the tokens are, in order,
//   sink (BF16) | middle (NVFP4, rotated by H16/4 along head_dim when `rotate`) | window (BF16 ring).
// For query token i of Tq (the newest tokens of the sequence, L tokens in all) and key t at position t:
//   s_t = scale q . k_t for t <= L - Tq + i (causal) or every t;  O = sum softmax(s)_t v_t.
// In the middle k_t = H16/4 (code e4m3 g_k), so q . k_t = (H16/4 q) . (code e4m3) g_k: the query is rotated
// once and the keys never; O's middle part is accumulated in rotated space and turned back once.
//
// One pass over the tokens with a running maximum and sum (kv_attn_kernel); what a CTA did not finish of a
// job (sequence, K/V head, tile of query rows) is joined by kv_attn_combine_kernel.  Bytes to move: 2 (D/2 + D/16) per
// middle token and K/V head, which at the copy rate of a B200 (6549 GB/s) is 92.5 us for 16 sequences of
// 32768 tokens, 8 K/V heads, D = 128; the kernel takes 139 us there in a CUDA graph, 4.35 TB/s (back-to-back calls
// 142 to 157).  Neither the bytes nor any one pipe is full: DRAM 54 %, issue slots 56 % (2.26 instructions per cycle and
// SM), converts' pipe 43 %, FP16 23 %, tensor pipe 35 %; in 44 % of a scheduler's cycles none of its 2.8 warps is
// eligible, and the largest stall is the fixed latency of the instruction before (1.3 cycles per instruction).  Latency
// at three warps per scheduler bounds it: registers (159) allow no more, and a warp has 623 instructions per tile of 32
// tokens, among them 128 converts (e2m1x2) and 128 multiplies (f16x2) of two cycles each and 48 products.  Of its 2815
// cycles per tile 20 wait for copies, 820 go into issuing them and 1880 compute.  The design keeps copies in
// flight and instructions per byte low:
// * every warp owns its tiles of 32 tokens and its own ring of shared-memory stages filled by cp.async: no
//   CTA-wide barrier inside the loop, rows behind the end arrive as zeros.  Bulk copies take the same bytes with
//   one instruction per row group, but each lane's copy is issued by itself (78 cycles): 157 us issued by every
//   warp, 147 by a fifth warp for all four;
// * code * e4m3 has at most 6 significant bits and lies in [2^-10, 2688], so the products' operands are exact
//   in FP16: one convert and one multiply give two elements, and m16n8k16 products with FP32 accumulators
//   take keys (or values' channels) as the 16 rows and query rows as the 8 columns.  A decode step has 1 to 16
//   query rows per K/V head: tcgen05 would spend a 128-row tile on them.  Keys can go to it as stored (block-scaled
//   FP4, the query as 8 FP4 terms of 16 columns each); built and measured, it took 180 us where this takes
//   140, since 128-token operands need their copies, fences and TMEM reads in step and the values still have to be
//   expanded;
// * the rotated query is split into two FP16 terms (22 bits after a power-of-two row scale), so scores
//   keep FP32 accuracy; the numerators are rounded to FP16 once, scaled by 2^10 (11 significant bits, so up to 2^-11
//   relative error each, down to 2^-24 of the row's maximum; the denominators are FP32 sums taken before that
//   rounding, so the error of a token that holds all the weight does not cancel: a second term of 11 bits would take a
//   second product over the values);
// * S^T = K Q^T leaves (token, query) fragments; movmatrix turns the FP16 numerators into the second
//   product's operand; V is packed along channels, so pairs of tokens are interleaved nibble by nibble
//   (two logic operations per 8 codes and token) before the converts;
// * the reference that numerators are taken against follows the maximum only when a score passes it by 2^5, so almost
//   no tile rescales the accumulators;
// * one job per CTA leaves SMs idle when sequences differ in length: all tokens of the call are cut evenly instead
//   (see ka_units).  In a graph: one sequence of 32768 tokens 18.4 us; 48 of up to 8191 47; 8 draft steps of 4 tokens,
//   D = 64, 13.4; D = 256 with 16 query heads on one K/V head 35.7; 301 tokens 8.2 to 8.9 (of which launch, the query's
//   rotation and three dependent rounds of loads are most).
#pragma once

#include <float.h>
#include <limits.h>
#include <math.h>

#include <type_traits>

#include "device.cuh"

namespace nvfp4 {

constexpr int kKaWarps = 4;            // warps per CTA, each with its own tiles
constexpr int kKaTile = 32;            // middle tokens per tile
// What starting and ending a job costs, in units of work (4 tiles).  Measured with 3 / 5 / 8 (us in a graph): 48 ragged
// sequences 47.5 / 48.5 / 51.8, draft tokens 13.4 / 13.6 / 13.9, one long sequence 18.2 / 18.2 / 18.9, 16 sequences of
// 32768 138.9 / 139.0 / 140.4, D = 256 with 16 rows, where a unit of work is longer, 35.6 / 33.6 / 36.8.  (1 and 2 were
// slower in an earlier form, ragged 52.4 and 51.6 against 49.2.)
constexpr int kKaJobUnits = 3;
// Least units of a part.  At most one more than kKaJobUnits: whole jobs of the least work are then never cut, which the
// host counts on.  Measured with 2 / 3 / 4 / 6 / 8 (us, D = 128, 4 rows): one sequence of 2048 tokens and 8 heads 9.2 / 9.8 /
// 10.7 / 13.0 / 14.2, 4 of 1024 9.9 / 10.2 / 11.1 / 13.1 / 14.5; the draft tokens 12.7 / 13.0 / 13.4 / 15.5 / 17.2; calls
// whose parts are longer anyway do not differ.  4 makes every part longer than a job's start, so that each has work of
// its own; 2 and 3, faster here, would need that given up.
constexpr int kKaMinUnits = 4;
constexpr int kKaMaxSplits = 65535;
constexpr int kKaJoinWarps = 8;        // warps that join the pieces of one query row
constexpr float kKaPShift = 10.0f;     // numerators of the middle are scaled by 2^10 before FP16
constexpr float kKaSlack = 5.0f;       // how far (base 2) a score may pass its row's reference: 2^15 fits FP16

struct KvSide {
  const char* sink;        // BF16 [slots, Hkv, sink_rows, D]
  const char* window;      // BF16 ring [slots, Hkv, window_rows, D]
  const uint8_t* codes;    // [pages, Hkv, page_rows, D/2]
  const uint8_t* scales;   // [pages, Hkv, page_rows, D/16] or tile layout
  const float* gscale;     // one, or one per slot
  int64_t gstride;         // 0 or 1
  int64_t mat_bytes;       // tile layout: bytes of one [page_rows, D] matrix
  int rotate, tile, vec16; // vec16: scale rows may be copied 16 bytes at a time
};

struct KvAttnParams {
  const char* q;
  char* out;
  float* lse;              // [B, Hq, Tq] or null
  int64_t q_sb, q_sh, q_st, o_sb, o_sh, o_st;   // strides in elements
  KvSide k, v;
  int Hq, Hkv, G, Tq, R, row_tiles;             // R = G Tq rows per K/V head, row r = token r / G, head r % G
  int sink_rows, window_rows, page_rows, page_shift;
  int64_t slots, pages, cols;
  const int32_t* slot;     // [B] or null: sequence b is slot b
  const int32_t* table;    // [slots, cols] or null: slot s is page s
  const int32_t* lens;     // [slots, 4] (n_sink, n_mid, head, n_window) or null: host_lens for every slot
  int host_lens[4];
  int B, causal, q_vec;
  float scale_log2;        // scale * log2(e)
  float* ws_o;             // [parts, 2, rows, D] sums of the jobs that a part shares with the part before / after it
  float2* ws_ml;           // [parts, 2, rows] their references (base 2) and denominators
  int4* ws_meta;           // jobs that are cut: sequence, head and row tile, first part, last part (-1: not cut)
  int by_job;              // ws_meta is indexed by the job (no more of them than parts); else by the part that begins it
};

template <int D>
struct KaShape {
  static constexpr int kCodeRow = D / 2, kScaleRow = D / 16;
  static constexpr int kKC = 0, kVC = kKaTile * kCodeRow, kKS = 2 * kKaTile * kCodeRow, kVS = kKS + kKaTile * kScaleRow;
  static constexpr int kStageBytes = 2 * kKaTile * (kCodeRow + kScaleRow);
  // (three stages at D = 128 gain nothing: the copies are never waited for)
  static constexpr int kStages = D == 64 ? 4 : 2;
  static constexpr int kRing = kKaWarps * kStages * kStageBytes;
};
template <int D, int NT, bool QBF>
struct KaSmem {
  static constexpr int kAccRow = D + 4;                                   // floats, padded
  static constexpr int kAcc = kKaWarps * 8 * NT * kAccRow * 4;            // the join of the warps reuses the ring
  static constexpr int kRing = KaShape<D>::kRing > kAcc ? KaShape<D>::kRing : kAcc;
  static constexpr int kQ = NT * (D / 16) * 32 * 16;                      // the rotated query's fragments (hi and lo)
  static constexpr int kQE = QBF ? kQ / 2 : kQ;                           // the query as given (a BF16 one is its first term)
  static constexpr int kStat = kKaWarps * 8 * NT * 8;
  static constexpr int kBytes = kRing + kQ + kQE + kStat + 8 * NT * 8 + kKaWarps * KaShape<D>::kStages * 4;
};

// ---- small instruction wrappers ----
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ uint32_t smem_u32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {   // the rest is zero-filled
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

template <bool BF>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  if constexpr (BF)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// the same from zero
__device__ __forceinline__ void mma16816_zero(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}
__device__ __forceinline__ uint32_t movmatrix(uint32_t a) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
// the four bytes of w (two E2M1 codes each) as f16x2
__device__ __forceinline__ void e2m1x8(uint32_t w, uint32_t (&h)[4]) {
  asm("{ .reg .b8 a, b, c, d; mov.b32 {a, b, c, d}, %4;\n"
      "cvt.rn.f16x2.e2m1x2 %0, a; cvt.rn.f16x2.e2m1x2 %1, b; cvt.rn.f16x2.e2m1x2 %2, c; cvt.rn.f16x2.e2m1x2 %3, d; }"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}
// two E4M3 bytes (low, high) as f16x2
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t b2) {
  uint32_t r;
  asm("{ .reg .b16 t; cvt.u16.u32 t, %1; cvt.rn.f16x2.e4m3x2 %0, t; }" : "=r"(r) : "r"(b2));
  return r;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// bits of a where m is set, of b elsewhere, in one operation
__device__ __forceinline__ uint32_t pick(uint32_t a, uint32_t b, uint32_t m) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xE4;" : "=r"(r) : "r"(a), "r"(b), "r"(m));
  return r;
}
__device__ __forceinline__ uint32_t both_lo(uint32_t h) {
  uint32_t r;
  asm("{ .reg .b16 a, b; mov.b32 {a, b}, %1; mov.b32 %0, {a, a}; }" : "=r"(r) : "r"(h));
  return r;
}
__device__ __forceinline__ uint32_t both_hi(uint32_t h) {
  uint32_t r;
  asm("{ .reg .b16 a, b; mov.b32 {a, b}, %1; mov.b32 %0, {b, b}; }" : "=r"(r) : "r"(h));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// (lo, hi) as two f16x2 terms: the rounded values and what they leave
__device__ __forceinline__ void split_f16(float lo, float hi, uint32_t& a, uint32_t& b) {
  a = pack_f16(lo, hi);
  b = pack_f16(__fsub_rn(lo, f16lo(a)), __fsub_rn(hi, f16hi(a)));
}
// (lo, hi) as two bf16x2 terms of the same sign, neither of them zero unless the value is: a factor times an
// infinite element of K or V then stays that infinity (a zero term would make it NaN).  The first term is the
// value cut to 8 bits, the second the rest rounded to 8 (relative error 2^-16); without a rest both are halves.
__device__ __forceinline__ void split_bf16(float lo, float hi, uint32_t& a, uint32_t& b) {
  float h0 = __uint_as_float(__float_as_uint(lo) & 0xFFFF0000u), h1 = __uint_as_float(__float_as_uint(hi) & 0xFFFF0000u);
  float r0 = __fsub_rn(lo, h0), r1 = __fsub_rn(hi, h1);
  if (r0 == 0.0f) h0 = r0 = 0.5f * lo;
  if (r1 == 0.0f) h1 = r1 = 0.5f * hi;
  a = pack_bf16(h0, h1);
  b = pack_bf16(r0, r1);
}
// a bf16x2 with halves that are infinite or NaN replaced by zero
__device__ __forceinline__ uint32_t finite_bf16x2(uint32_t u) {
  if ((u & 0x7F80u) == 0x7F80u) u &= 0xFFFF0000u;
  if ((u & 0x7F800000u) == 0x7F800000u) u &= 0x0000FFFFu;
  return u;
}
__device__ __forceinline__ float finite_or_zero(float m) { return m == -INFINITY ? 0.0f : m; }

// The lengths of the sequence of batch row b, bounded by the buffers (an unknown slot is an empty sequence).
struct KaSeq {
  int s, ns, nm, head, nw;
  int len;
};
__device__ __forceinline__ KaSeq ka_sequence(const KvAttnParams& p, int b) {
  KaSeq q;
  const int64_t s = p.slot ? p.slot[b] : b;
  const bool ok = s >= 0 && s < p.slots;
  q.s = ok ? (int)s : 0;
  int n[4];
  if (p.lens) {
#pragma unroll
    for (int k = 0; k < 4; ++k) n[k] = p.lens[4 * (int64_t)q.s + k];
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) n[k] = p.host_lens[k];
  }
  const int64_t most = p.table ? p.cols * p.page_rows : p.page_rows;
  q.ns = ok ? min(max(n[0], 0), p.sink_rows) : 0;
  q.nm = ok ? (int)min((int64_t)max(n[1], 0), most) : 0;
  q.nw = ok ? min(max(n[3], 0), p.window_rows) : 0;
  q.head = p.window_rows > 0 ? (int)((uint32_t)n[2] % (uint32_t)p.window_rows) : 0;
  q.len = q.ns + q.nm + q.nw;
  return q;
}
// The call's work in units: of a job (a sequence, K/V head and tile of query rows) kKaJobUnits for starting and ending
// it, then one per 4 tiles of the middle (a tile per warp) and one per 4 tiles of the BF16 ends, at least one.
// Units are numbered job after job and cut into equal parts, one per CTA: whatever the lengths, the CTAs do the same
// work in one wave, and only the jobs that a cut falls into have to be joined.  A cut among a job's first
// kKaJobUnits units moves to its beginning.
__device__ __forceinline__ int ka_mid_units(const KaSeq& q) { return (q.nm + kKaTile * kKaWarps - 1) / (kKaTile * kKaWarps); }
__device__ __forceinline__ int ka_end_tiles(const KaSeq& q) { return (q.ns + 15) / 16 + (q.nw + 15) / 16; }
__device__ __forceinline__ int ka_units(const KaSeq& q) {
  return kKaJobUnits + max(ka_mid_units(q) + (ka_end_tiles(q) + kKaWarps - 1) / kKaWarps, 1);
}
struct KaParts {
  int64_t base, rem;                    // part c starts at c base + min(c, rem)
  int n;
  __host__ __device__ __forceinline__ KaParts(int64_t total, int most) {
    n = (int)min((int64_t)most, max(total / kKaMinUnits, (int64_t)1));
    base = total / n;
    rem = total - base * n;
  }
  __host__ __device__ __forceinline__ int64_t start(int c) const { return c * base + min((int64_t)c, rem); }
  __host__ __device__ __forceinline__ int of(int64_t u) const {
    return (int)(u < rem * (base + 1) ? u / (base + 1) : rem + (u - rem * (base + 1)) / base);
  }
};
// What a part that has come to unit u (before its end u_end) does of the job there, one of a sequence whose jobs begin at
// seq_start and cost `cost` units each.
struct KaPiece {
  int job, first, last, units;          // units of work [first, last) of the job's
  int64_t next;                         // the job's end
  bool mine;                            // false: only units of starting the job are left, the next part begins it
  __host__ __device__ __forceinline__ KaPiece(int64_t u, int64_t u_end, int64_t seq_start, int cost) {
    job = (int)((u - seq_start) / cost);
    units = cost - kKaJobUnits;
    const int64_t work = seq_start + (int64_t)job * cost + kKaJobUnits;
    mine = u_end > work;
    first = (int)max(u - work, (int64_t)0);
    last = (int)min((int64_t)units, u_end - work);
    next = work + units;
  }
  __host__ __device__ __forceinline__ bool begun() const { return first == 0; }
  __host__ __device__ __forceinline__ bool done() const { return last == units; }
};

template <bool BF>
__device__ __forceinline__ void ka_store(char* out, int64_t i, float x) {
  if constexpr (BF) reinterpret_cast<__nv_bfloat16*>(out)[i] = __float2bfloat16_rn(x);
  else reinterpret_cast<__half*>(out)[i] = __float2half_rn(x);
}

// D: head_dim; NT: query rows / 8 of a CTA; QBF: q and out are BF16 (else FP16).
// CTAs per SM: as many as registers allow.  D = 128, NT = 1 with 3 (159 registers, no spills) against 4 (128, 56 bytes
// spilled): one long sequence 18.3 / 21.5 us, ragged 47.5 / 52.0, large 138.9 / 141.8.  D = 256, NT = 2 needs all 255
// registers of two CTAs and spills 40 (BF16) or 72 (FP16) bytes; the other forms spill nothing.
template <int D, int NT, bool QBF>
__global__ void __launch_bounds__(kKaWarps * 32, D == 256 ? 2 : D == 128 ? (NT == 1 ? 3 : 2) : (NT == 1 ? 4 : 3))
    kv_attn_kernel(const __grid_constant__ KvAttnParams p) {
  using Sh = KaShape<D>;
  using Sm = KaSmem<D, NT, QBF>;
  constexpr int ST = Sh::kStages, NS = D / 16 /* k16 steps */, NO = D / 16 /* m16 tiles of channels */;
  constexpr int KW = D >= 128 ? 4 : 2, KCH = D == 256 ? 2 : 1;      // code words per key chunk, chunks per thread
  constexpr int VW = D / 64;                                         // code words of V per thread and token
  constexpr int VB = D == 256 ? 2 : 1;                               // scale blocks of V per thread and token
  constexpr int ROWS = 8 * NT;
  extern __shared__ __align__(128) unsigned char smem[];
  uint4* qf = reinterpret_cast<uint4*>(smem + Sm::kRing);            // rotated query, FP16 hi / lo, fragment order
  uint2* qe = reinterpret_cast<uint2*>(smem + Sm::kRing + Sm::kQ);   // query as given, BF16: first terms,
  uint2* qr = qe + NT * NS * 32;                                     // and (FP16 only) second terms
  float2* stat = reinterpret_cast<float2*>(smem + Sm::kRing + Sm::kQ + Sm::kQE);
  float* rowfac = reinterpret_cast<float*>(smem + Sm::kRing + Sm::kQ + Sm::kQE + Sm::kStat);
  int* limit = reinterpret_cast<int*>(rowfac + ROWS);
  uint32_t* vms = reinterpret_cast<uint32_t*>(limit + ROWS);         // [warp][stage]: the tile's tokens that exist
  __shared__ int64_t scan[kKaWarps + 1];
  __shared__ int found_b;

  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, g = lane >> 2, t = lane & 3;
  const int part = blockIdx.x, jobs_per_seq = p.Hkv * p.row_tiles;

  // ---- this CTA's units, and the sequence that holds the first ----
  int64_t total, seq_start;
  int b;
  if (p.lens == nullptr && p.slot == nullptr) {                       // all sequences alike
    const int64_t per_seq = (int64_t)ka_units(ka_sequence(p, 0)) * jobs_per_seq;
    total = per_seq * p.B;
    const KaParts parts(total, gridDim.x);
    b = part < parts.n ? (int)(parts.start(part) / per_seq) : 0;
    seq_start = b * per_seq;
  } else {
    const int each = (p.B + kKaWarps * 32 - 1) / (kKaWarps * 32), b0 = min(tid * each, p.B), b1 = min(b0 + each, p.B);
    int64_t sum = 0;
    for (int i = b0; i < b1; ++i) sum += (int64_t)ka_units(ka_sequence(p, i)) * jobs_per_seq;
    int64_t upto = sum;                                               // inclusive prefix over the CTA's threads
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(0xFFFFFFFFu, upto, o);
      if (lane >= o) upto += v;
    }
    if (lane == 31) scan[w] = upto;
    __syncthreads();
    total = 0;
#pragma unroll
    for (int i = 0; i < kKaWarps; ++i) {
      if (i < w) upto += scan[i];
      total += scan[i];
    }
    __syncthreads();                                                  // scan is written again below
    const KaParts parts(total, gridDim.x);
    const int64_t u0 = part < parts.n ? parts.start(part) : total;
    int64_t at = upto - sum;
    if (u0 >= at && u0 < upto) {
      int i = b0;
      for (;; ++i) {
        const int64_t n = (int64_t)ka_units(ka_sequence(p, i)) * jobs_per_seq;
        if (u0 < at + n) break;
        at += n;
      }
      scan[0] = at;
      found_b = i;
    }
    __syncthreads();
    seq_start = scan[0];
    b = found_b;
  }
  const KaParts parts(total, gridDim.x);
  if (gridDim.x > 1 && tid == kKaWarps * 32 - 1 && !p.by_job) p.ws_meta[part].w = -1;
  if (part >= parts.n) return;
  int64_t u = parts.start(part);
  const int64_t u_end = parts.start(part + 1);
  KaSeq sq = ka_sequence(p, b);
  int cost = ka_units(sq);
  while (u < u_end) {
    if (u - seq_start >= (int64_t)cost * jobs_per_seq) {
      seq_start += (int64_t)cost * jobs_per_seq;
      sq = ka_sequence(p, ++b);
      cost = ka_units(sq);
    }
    const KaPiece piece(u, u_end, seq_start, cost);
    if (!piece.mine) break;
    const int job = piece.job, units = piece.units, first_unit = piece.first, last_unit = piece.last;
    u = piece.next;
    const int kvh = job / p.row_tiles, row_tile = job - kvh * p.row_tiles;
    const int mid_units = ka_mid_units(sq), tiles = (sq.nm + kKaTile - 1) / kKaTile;
    const int t_first = min(first_unit, mid_units) * kKaWarps + w, t_end = min(tiles, min(last_unit, mid_units) * kKaWarps);
    const int n_my = t_first < t_end ? (t_end - t_first + kKaWarps - 1) / kKaWarps : 0;

    // ---- the warp's ring: tile i of this warp goes to stage i % ST ----
    unsigned char* ring = smem + w * ST * Sh::kStageBytes;
    const uint32_t ring_u = smem_u32(ring);
    // Rows of the middle are numbered page by page (below 2^32, checked on the host): row (page Hkv + head) page_rows +
    // r.  Keys are read as rows r and r + 4 together, values as rows r .. r + 3: each order gets its own exchange of
    // 64- (32-) byte halves in shared memory so that both read without bank conflicts; a lane's exchange is the
    // same in every instruction but for D = 256 keys.
    constexpr int CPR = Sh::kCodeRow / 16, ITS = kKaTile * CPR / 32, HALF = ITS / 2;   // pieces per row, instructions
    const uint32_t lane_row = lane / CPR;
    const uint32_t k_at = ring_u + Sh::kKC + (lane * 16 ^ (D == 256 ? 0u : (lane_row >> 2 & 1u) << 6));
    const uint32_t v_at = ring_u + Sh::kVC + (D == 128 ? lane * 16 ^ (lane_row >> 1 & 1u) << 5 : D == 256 ? lane * 16 ^ (lane_row & 3u) << 5 : lane * 16);
    const uint8_t* kc = p.k.codes + lane * 16;
    const uint8_t* vc = p.v.codes + lane * 16;
    constexpr int RPP = 16 / Sh::kScaleRow, NP = kKaTile / RPP;        // scale rows per 16 bytes, pieces per tile and side
    const uint8_t* sc = (NP == 32 || lane < NP ? p.k.scales : p.v.scales) + lane % (NP / 2) * 16;   // NP < 32: keys', then values'
    const int32_t* my_table = p.table ? p.table + (int64_t)sq.s * p.cols : nullptr;
    const bool pieces16 = p.k.vec16 && p.v.vec16, tiles32 = p.k.tile && p.v.tile && !(my_table && p.page_rows & 31);
    const uint32_t head_rows = (uint32_t)p.Hkv * (uint32_t)p.page_rows, my_rows = (uint32_t)kvh * (uint32_t)p.page_rows;
    const int mask = p.page_shift >= 0 ? p.page_rows - 1 : 0;
    auto page_of = [&](int tok) -> int {          // the page holding middle token tok, -1: none
      if (tok >= sq.nm) return -1;
      if (!my_table) return sq.s;
      const int pg = __ldg(my_table + (p.page_shift >= 0 ? tok >> p.page_shift : tok / p.page_rows));
      return (uint32_t)pg < (uint32_t)p.pages ? pg : -1;
    };
    auto row_in_page = [&](int tok) -> int { return !my_table ? tok : p.page_shift >= 0 ? tok & mask : tok % p.page_rows; };
    uint32_t partial = 0;                         // bit i % 32: tile i does not hold 32 tokens (which it holds: vms)
    const bool split_tiles = my_table && (p.page_rows & 31);   // a tile may lie in two pages
    auto issue = [&](int i, int st, int pg0, int pg1) {
      const int tok = (t_first + i * kKaWarps) * kKaTile;
      const uint32_t so = st * Sh::kStageBytes;
      const int r0 = row_in_page(tok), r1 = split_tiles ? row_in_page(tok + 16) : r0 + 16;
      const uint32_t row0 = (uint32_t)pg0 * head_rows + my_rows + r0;
      const uint32_t row1 = split_tiles ? (uint32_t)pg1 * head_rows + my_rows + r1 : row0 + 16;
      const bool whole = (pg0 | pg1) >= 0 && tok + kKaTile <= sq.nm;
      uint32_t vm = 0xFFFFFFFFu;
      if (whole) {
        const uint8_t *k0 = kc + (uint64_t)row0 * Sh::kCodeRow, *k1 = kc + (uint64_t)row1 * Sh::kCodeRow;
        const uint8_t *v0 = vc + (uint64_t)row0 * Sh::kCodeRow, *v1 = vc + (uint64_t)row1 * Sh::kCodeRow;
#pragma unroll
        for (int it = 0; it < ITS; ++it) {
          const uint32_t ka = D == 256 ? k_at ^ (uint32_t)(it & 1) << 6 : k_at;
          cp_async16(ka + so + it * 512, (it < HALF ? k0 : k1) + (it % HALF) * 512);
          cp_async16(v_at + so + it * 512, (it < HALF ? v0 : v1) + (it % HALF) * 512);
        }
        const uint32_t sa = ring_u + so + Sh::kKS;
        if (pieces16) {
          if constexpr (NP == 32) {
            const uint64_t o = (uint64_t)(lane < 16 ? row0 : row1) * Sh::kScaleRow;
            cp_async16(sa + lane * 16, sc + o);
            cp_async16(sa + lane * 16 + Sh::kVS - Sh::kKS, sc + (p.v.scales - p.k.scales) + o);
          } else if (lane < 2 * NP) {
            cp_async16(sa + lane * 16, sc + (uint64_t)(lane % NP < NP / 2 ? row0 : row1) * Sh::kScaleRow);
          }
          return;
        }
        if (tiles32 && (r0 & 31) == 0) {          // 32 rows of a scale tile: every fourth word of its 512 bytes
          const uint64_t o = (uint64_t)((uint32_t)pg0 * (uint32_t)p.Hkv + kvh) * p.k.mat_bytes +
                             (uint64_t)(r0 >> 7) * (D / 64 * 512) + 4 * (r0 >> 5 & 3) + lane * 16;
#pragma unroll
          for (int j = 0; j < D / 64; ++j) {
            cp_async4(sa + lane * Sh::kScaleRow + 4 * j, p.k.scales + o + j * 512);
            cp_async4(sa + Sh::kVS - Sh::kKS + lane * Sh::kScaleRow + 4 * j, p.v.scales + o + j * 512);
          }
          return;
        }
      } else {
        const int n0 = pg0 >= 0 ? min(max(sq.nm - tok, 0), 16) : 0, n1 = pg1 >= 0 ? min(max(sq.nm - tok - 16, 0), 16) : 0;
        vm = ((1u << n0) - 1u) | ((1u << n1) - 1u) << 16;
        partial |= 1u << (i & 31);
        if (lane == 0) vms[w * ST + st] = vm;
#pragma unroll
        for (int it = 0; it < ITS; ++it) {
          const int ok = vm >> (it * (32 / CPR) + lane_row) & 1u;
          const uint64_t o = ok ? (uint64_t)(it < HALF ? row0 : row1) * Sh::kCodeRow + (it % HALF) * 512 : 0;
          const uint32_t ka = D == 256 ? k_at ^ (uint32_t)(it & 1) << 6 : k_at;
          cp_async16(ka + so + it * 512, kc + o, ok ? 16 : 0);
          cp_async16(v_at + so + it * 512, vc + o, ok ? 16 : 0);
        }
      }
#pragma unroll
      for (int side = 0; side < 2; ++side) {
        const uint8_t* s = side ? p.v.scales : p.k.scales;
        const bool tile = side ? p.v.tile : p.k.tile;
        const int64_t mb = side ? p.v.mat_bytes : p.k.mat_bytes;
        const uint32_t sd = ring_u + so + (side ? Sh::kVS : Sh::kKS) + lane * Sh::kScaleRow;
        const int ok = (vm >> lane) & 1u, r = (lane < 16 ? r0 : r1) + (lane & 15);
        const uint32_t row = (lane < 16 ? row0 : row1) + (lane & 15);
        const int64_t m = (int64_t)(lane < 16 ? pg0 : pg1) * p.Hkv + kvh;
#pragma unroll
        for (int j = 0; j < D / 64; ++j) {
          int64_t off = 0;
          if (ok)
            off = tile ? m * mb + ((int64_t)(r >> 7) * (D / 64) + j) * 512 + 16 * (r & 31) + 4 * (r >> 5 & 3)
                       : (int64_t)row * Sh::kScaleRow + 4 * j;
          cp_async4(sd + 4 * j, s + off, ok ? 4 : 0);
        }
      }
    };
    int next[2] = {-1, -1};                       // pages of the tile that is issued next
    auto look_up = [&](int i) {
      if (i >= n_my) return;
      const int tok = (t_first + i * kKaWarps) * kKaTile;
      next[0] = page_of(tok);
      next[1] = split_tiles ? page_of(tok + 16) : next[0];
    };
    look_up(0);
#pragma unroll
    for (int i = 0; i < ST - 1; ++i) {
      const int a = next[0], c = next[1];
      look_up(i + 1);
      if (i < n_my) issue(i, i, a, c);
      cp_async_commit();
    }

    // the BF16 ends are read last: ask for them now
    const int sink_tiles = (sq.ns + 15) / 16, e_end = min(ka_end_tiles(sq), (last_unit - mid_units) * kKaWarps);
    const int e_first = max(first_unit - mid_units, 0) * kKaWarps + w;
    if (e_first < e_end && n_my > 0) {
      const int in = e_first < sink_tiles, r = 16 * (in ? e_first : e_first - sink_tiles) + (lane & 15);
      if (r < (in ? sq.ns : sq.nw)) {
        const int rows = in ? p.sink_rows : p.window_rows, at = in ? r : r + sq.head >= rows ? r + sq.head - rows : r + sq.head;
        const KvSide& s = lane < 16 ? p.k : p.v;
        const char* src = (in ? s.sink : s.window) + (((int64_t)sq.s * p.Hkv + kvh) * rows + at) * (D * 2);
#pragma unroll
        for (int k = 0; k < D * 2; k += 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(src + k));
      }
    }

    // ---- the query rows: 16-channel blocks, rotated, scaled by a power of two per row, in fragment order ----
    constexpr int BPR = D / 16;                   // blocks per row, handled by adjacent lanes
#pragma unroll
    for (int i0 = 0; i0 < ROWS * BPR; i0 += kKaWarps * 32) {
      const int item = i0 + tid;
      if (ROWS * BPR % (kKaWarps * 32) != 0 && item >= ROWS * BPR) break;   // whole warps leave (ROWS * BPR is a multiple of 32)
      const int row = item / BPR, blk = item % BPR, r = row_tile * ROWS + row;
      float a[16];
      if (r < p.R) {
        const int i = r / p.G, hq = kvh * p.G + r % p.G;
        const int64_t at = b * p.q_sb + hq * p.q_sh + i * p.q_st + blk * 16;
        uint32_t wd[8];
        if (p.q_vec) {
          ld_v4(p.q + at * 2, wd);
          ld_v4(p.q + at * 2 + 16, wd + 4);
        } else {
          const unsigned short* s = reinterpret_cast<const unsigned short*>(p.q) + at;
#pragma unroll
          for (int k = 0; k < 8; ++k) wd[k] = s[2 * k] | (uint32_t)s[2 * k + 1] << 16;
        }
        widen_words<QBF ? DT_BF16 : DT_F16>(wd, a, 8);
      } else {
#pragma unroll
        for (int k = 0; k < 16; ++k) a[k] = 0.0f;
      }
      // channel c of the row sits in key chunk c / CD, read by thread t of the fragment; 4 channels per step
      constexpr int CD = D >= 128 ? 32 : 16;
      const int c0 = blk * 16, chunk = c0 / CD, ft = chunk & 3, j0 = (chunk >> 2) * 8 + (c0 % CD) / 4;
      const int fl = (row & 7) * 4 + ft, nt = row >> 3;
      const int fo = (nt * NS + j0) * 32 + fl;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (QBF) {
          qe[fo + j * 32] = make_uint2(pack_bf16(a[4 * j], a[4 * j + 1]), pack_bf16(a[4 * j + 2], a[4 * j + 3]));
        } else {
          uint4 v;
          split_bf16(a[4 * j], a[4 * j + 1], v.x, v.z);
          split_bf16(a[4 * j + 2], a[4 * j + 3], v.y, v.w);
          qe[fo + j * 32] = make_uint2(v.x, v.y);
          qr[fo + j * 32] = make_uint2(v.z, v.w);
        }
      }
      if (p.k.rotate) fwht16(a);
      const float sign = p.scale_log2 < 0.0f ? -1.0f : 1.0f;            // carried by the query, so that factors are >= 0
      float mx = 0.0f;
#pragma unroll
      for (int k = 0; k < 16; ++k) mx = fmaxf(mx, fabsf(a[k]));
#pragma unroll
      for (int o = BPR / 2; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
      int e = (int)(__float_as_uint(mx) >> 23) - 127;                  // floor(log2), exact for normal values
      e = mx > 0.0f && mx <= FLT_MAX ? max(-126, min(126, e)) : 0;    // 2^e and 2^-e are normal
      const float down = sign * __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint4 v;
        split_f16(a[4 * j] * down, a[4 * j + 1] * down, v.x, v.z);
        split_f16(a[4 * j + 2] * down, a[4 * j + 3] * down, v.y, v.w);
        qf[fo + j * 32] = v;
      }
      if (blk == 0) {
        rowfac[row] = __uint_as_float((uint32_t)(127 + e) << 23);
        // positions this row sees: all before the limit (rows past R restrict nothing and are not written)
        limit[row] = p.causal && r < p.R ? max(sq.len - p.Tq + r / p.G + 1, 0) : sq.len;
      }
    }
    if (gridDim.x > 1 && tid == kKaWarps * 32 - 1) {   // (the last warps have no query row of most calls)
      int4* e = p.ws_meta + (p.by_job ? (int64_t)b * jobs_per_seq + job : part);
      const bool begun = piece.begun(), done = piece.done();
      if (begun && !done) *reinterpret_cast<int2*>(e) = make_int2(b, job), e->z = part;
      if (p.by_job ? done : begun && !done) e->w = p.by_job ? (begun ? -1 : part) : parts.of(u - 1);
    }
    __syncthreads();

    float O[NO][NT][4], m[NT][2], l[NT][2], fac[NT][2];
    int lim[NT][2];                               // positions each column's row sees: all before this one
    int lim_min = INT_MAX;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        m[n][c] = -INFINITY;
        l[n][c] = 0.0f;
        lim[n][c] = limit[8 * n + 2 * t + c];
        lim_min = min(lim_min, lim[n][c]);
        fac[n][c] = rowfac[8 * n + 2 * t + c];
      }
#pragma unroll
      for (int i = 0; i < NO; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) O[i][n][c] = 0.0f;
    }
    lim_min = min(lim_min, __shfl_xor_sync(0xFFFFFFFFu, lim_min, 1));
    lim_min = min(lim_min, __shfl_xor_sync(0xFFFFFFFFu, lim_min, 2));
    const int perm = (g >> 1) + 4 * (g & 1);      // the token of fragment row g (row g + 8: + 8)

    // the tile's tokens (bit k: token k) that a column's row sees
    auto seen_of = [&](int n, int c, int tok0, uint32_t vm) -> uint32_t {
      const int rel = max(min(lim[n][c] - sq.ns - tok0, kKaTile), 0);
      return vm & (rel >= 32 ? 0xFFFFFFFFu : (1u << rel) - 1u);
    };

    // The reference m of a row's numerators follows its maximum lazily: while no score of the tile passes it by more
    // than kKaSlack, m and everything summed under it stay (one vote); else m becomes the tile's maximum and the
    // sums are rescaled.
    auto raise = [&](float (&mx)[NT][2]) {
      bool up = false;
#pragma unroll
      for (int n = 0; n < NT; ++n) up |= mx[n][0] > m[n][0] + kKaSlack || mx[n][1] > m[n][1] + kKaSlack;
      if (!__any_sync(0xFFFFFFFFu, up)) return;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) mx[n][c] = fmaxf(mx[n][c], __shfl_xor_sync(0xFFFFFFFFu, mx[n][c], o));
          // (each row by its own scores alone: what other rows see changes no bit of it)
          const float mn = mx[n][c] > m[n][c] + kKaSlack ? mx[n][c] : m[n][c];
          const float al = ex2(m[n][c] - finite_or_zero(mn));
          m[n][c] = mn;
          l[n][c] *= al;
#pragma unroll
          for (int i = 0; i < NO; ++i) {
            O[i][n][c] *= al;
            O[i][n][c + 2] *= al;
          }
        }
    };

    if (n_my > 0) {
      const float gk = p.k.gscale[p.k.gstride * sq.s] * fabsf(p.scale_log2);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        fac[n][0] *= gk;
        fac[n][1] *= gk;
      }
    }
    // A lane's offsets in a stage: rows are added as constants (the exchanges of halves depend on bits of the row
    // that those constants leave alone).
    const int k_read = Sh::kKC + ((perm * Sh::kCodeRow + t * (KW * 4)) ^ (perm >> 2 & 1) << 6);
    const int k_read2 = Sh::kKC + ((perm * Sh::kCodeRow + (t + 4) * (KW * 4)) ^ (perm >> 2 & 1) << 6);   // D = 256
    const int v_read = Sh::kVC + ((t * Sh::kCodeRow + g * (VW * 4)) ^ (D == 256 ? t << 5 : D == 128 ? (t >> 1 & 1) << 5 : 0));
    const int ks_read = Sh::kKS + perm * Sh::kScaleRow + (KW == 4 ? 2 * t : t);
    const int vs_read = Sh::kVS + t * Sh::kScaleRow + (D == 256 ? 2 * g : D == 128 ? g : g >> 1);

    // One tile of 32 tokens.  FULL: all of them exist and every row sees them.
    auto work = [&](auto full, const unsigned char* st, int tok0, uint32_t vm) {
      constexpr bool FULL = decltype(full)::value;
      // ---- S^T = K Q^T: rows are tokens (two tiles of 16), columns query rows ----
      float S[2][NT][4];
#pragma unroll
      for (int cc = 0; cc < KCH; ++cc) {
        uint32_t kw[2][2][KW], ks[2][2][KW / 2];   // [token tile][rows perm and perm + 8]; scales doubled into both halves
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int row = 8 * k + 16 * a;        // + perm, in the lane's offsets
            if constexpr (KW == 4) {
              const uint4 v = *reinterpret_cast<const uint4*>(st + (cc ? k_read2 : k_read) + row * Sh::kCodeRow);
              kw[a][k][0] = v.x, kw[a][k][1] = v.y, kw[a][k][2] = v.z, kw[a][k][3] = v.w;
              const uint32_t h = e4m3x2_f16x2(*reinterpret_cast<const unsigned short*>(st + ks_read + row * Sh::kScaleRow + 8 * cc));
              ks[a][k][0] = both_lo(h);
              ks[a][k][1] = both_hi(h);
            } else {
              const uint2 v = *reinterpret_cast<const uint2*>(st + k_read + row * Sh::kCodeRow);
              kw[a][k][0] = v.x, kw[a][k][1] = v.y;
              ks[a][k][0] = both_lo(e4m3x2_f16x2(st[ks_read + row * Sh::kScaleRow]));
            }
          }
        // a word of 8 codes feeds two steps; both token tiles take the query's fragments while they are in registers
        // (tile after tile: D = 256 38.6 against 38.0 us, ragged D = 128 47.2 against 46.8)
#pragma unroll
        for (int wd = 0; wd < KW; ++wd)
#pragma unroll
          for (int a = 0; a < 2; ++a) {
            uint32_t h[2][4];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              e2m1x8(kw[a][k][wd], h[k]);
#pragma unroll
              for (int c = 0; c < 4; ++c) h[k][c] = hmul2(h[k][c], ks[a][k][wd >> 1]);
            }
#pragma unroll
            for (int j2 = 0; j2 < 2; ++j2) {
              const int j = cc * 8 + wd * 2 + j2;
#pragma unroll
              for (int n = 0; n < NT; ++n) {
                const uint4 qv = qf[(n * NS + j) * 32 + lane];
                if (j == 0) mma16816_zero(S[a][n], h[0][2 * j2], h[1][2 * j2], h[0][2 * j2 + 1], h[1][2 * j2 + 1], qv.x, qv.y);
                else mma16816<false>(S[a][n], h[0][2 * j2], h[1][2 * j2], h[0][2 * j2 + 1], h[1][2 * j2 + 1], qv.x, qv.y);
                mma16816<false>(S[a][n], h[0][2 * j2], h[1][2 * j2], h[0][2 * j2 + 1], h[1][2 * j2 + 1], qv.z, qv.w);
              }
            }
          }
      }
      // ---- numerators (fac >= 0: maxima are taken before it is applied) ----
      float mx[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          if constexpr (!FULL) {
            const uint32_t seen = seen_of(n, c, tok0, vm);
#pragma unroll
            for (int a = 0; a < 2; ++a)
#pragma unroll
              for (int h = 0; h < 2; ++h)
                if (!(seen >> (16 * a + 8 * h + perm) & 1u)) S[a][n][c + 2 * h] = -INFINITY;
          }
          mx[n][c] = fac[n][c] * fmaxf(fmaxf(S[0][n][c], S[0][n][c + 2]), fmaxf(S[1][n][c], S[1][n][c + 2]));
        }
      raise(mx);
      uint32_t pb[2][NT][2];                       // the second product's B fragments (tokens x query rows)
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const float s0 = kKaPShift - finite_or_zero(m[n][0]), s1 = kKaPShift - finite_or_zero(m[n][1]);
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float p0 = ex2(fmaf(S[a][n][2 * h], fac[n][0], s0)), p1 = ex2(fmaf(S[a][n][2 * h + 1], fac[n][1], s1));
            if constexpr (!FULL) {                           // -Inf times a zero factor would be NaN
              p0 = S[a][n][2 * h] == -INFINITY ? 0.0f : p0;
              p1 = S[a][n][2 * h + 1] == -INFINITY ? 0.0f : p1;
            }
            l[n][0] += p0;
            l[n][1] += p1;
            pb[a][n][h] = movmatrix(pack_f16(p0, p1));
          }
      }
      // ---- O^T += V^T P^T: rows are channels, the 16 k positions the tokens 4 r + t of the fragment order ----
#pragma unroll
      for (int a = 0; a < 2; ++a) {
        uint32_t vw[4][VW], vs[2][VB];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int row = 16 * a + 4 * r;        // + t, in the lane's offset
          if constexpr (VW == 4) {
            const uint4 v = *reinterpret_cast<const uint4*>(st + v_read + row * Sh::kCodeRow);
            vw[r][0] = v.x, vw[r][1] = v.y, vw[r][2] = v.z, vw[r][3] = v.w;
          } else if constexpr (VW == 2) {
            const uint2 v = *reinterpret_cast<const uint2*>(st + v_read + row * Sh::kCodeRow);
            vw[r][0] = v.x, vw[r][1] = v.y;
          } else {
            vw[r][0] = *reinterpret_cast<const uint32_t*>(st + v_read + row * Sh::kCodeRow);
          }
        }
#pragma unroll
        for (int q2 = 0; q2 < 2; ++q2) {
          const unsigned char* s0 = st + vs_read + (16 * a + 8 * q2) * Sh::kScaleRow;
          const unsigned char* s1 = s0 + 4 * Sh::kScaleRow;
          if constexpr (VB == 2) {
            const uint32_t u0 = *reinterpret_cast<const unsigned short*>(s0), u1 = *reinterpret_cast<const unsigned short*>(s1);
            vs[q2][0] = e4m3x2_f16x2(__byte_perm(u0, u1, 0x0040));
            vs[q2][1] = e4m3x2_f16x2(__byte_perm(u0, u1, 0x0051));
          } else {
            vs[q2][0] = e4m3x2_f16x2(__byte_perm(*s0, *s1, 0x0040));
          }
        }
        uint32_t nan_tok[VB];
        if constexpr (!FULL) {
          // a poisoned block (scale NaN) of a token that only some of the columns see: 0 * NaN would reach the
          // others through the product, so its scale becomes 0 and the columns that do see it turn NaN below
#pragma unroll
          for (int vb = 0; vb < VB; ++vb) {
            nan_tok[vb] = 0;
#pragma unroll
            for (int q2 = 0; q2 < 2; ++q2) {
              const uint32_t u = vs[q2][vb];
              if ((u & 0x7FFFu) > 0x7C00u) nan_tok[vb] |= 1u << (16 * a + 8 * q2 + t), vs[q2][vb] &= 0xFFFF0000u;
              if ((u >> 16 & 0x7FFFu) > 0x7C00u) nan_tok[vb] |= 1u << (16 * a + 8 * q2 + 4 + t), vs[q2][vb] &= 0x0000FFFFu;
            }
            nan_tok[vb] |= __shfl_xor_sync(0xFFFFFFFFu, nan_tok[vb], 1);
            nan_tok[vb] |= __shfl_xor_sync(0xFFFFFFFFu, nan_tok[vb], 2);
          }
        }
#pragma unroll
        for (int wd = 0; wd < VW; ++wd) {
          constexpr uint32_t LO = 0x0F0F0F0Fu;
          uint32_t hx[2][4], hy[2][4];             // even and odd channels, (token 4 r + t, token 4 (r + 1) + t)
#pragma unroll
          for (int q2 = 0; q2 < 2; ++q2) {
            const uint32_t u = vw[2 * q2][wd], v = vw[2 * q2 + 1][wd];
            e2m1x8(pick(u, v << 4, LO), hx[q2]);
            e2m1x8(pick(u >> 4, v, LO), hy[q2]);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              hx[q2][k] = hmul2(hx[q2][k], vs[q2][VB == 2 ? wd >> 1 : 0]);
              hy[q2][k] = hmul2(hy[q2][k], vs[q2][VB == 2 ? wd >> 1 : 0]);
            }
          }
#pragma unroll
          for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int n = 0; n < NT; ++n)
              mma16816<false>(O[4 * wd + k][n], hx[0][k], hy[0][k], hx[1][k], hy[1][k], pb[a][n][0], pb[a][n][1]);
        }
        if constexpr (!FULL) {
#pragma unroll
          for (int vb = 0; vb < VB; ++vb)
            if (nan_tok[vb]) {
#pragma unroll
              for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                  if (nan_tok[vb] & seen_of(n, c, tok0, vm)) {
#pragma unroll
                    for (int k = 0; k < NO / VB; ++k) O[vb * (NO / VB) + k][n][c] = O[vb * (NO / VB) + k][n][c + 2] = NAN;
                  }
                }
            }
        }
      }
    };
    const int mid_seen = lim_min - sq.ns;         // every row sees the middle's tokens before this one
    int stage = 0, ahead = ST - 1;                // stages of tile i and of the tile issued with it
    for (int i = 0; i < n_my; ++i) {
      cp_async_wait<ST - 2>();
      __syncwarp();
      {
        const int a = next[0], c = next[1], k = i + ST - 1;
        look_up(k + 1);
        if (k < n_my) issue(k, ahead, a, c);
        cp_async_commit();
      }
      const unsigned char* st = ring + stage * Sh::kStageBytes;
      const int tok0 = (t_first + i * kKaWarps) * kKaTile;
      if (!(partial >> (i & 31) & 1u) && tok0 + kKaTile <= mid_seen) {
        work(std::true_type{}, st, tok0, 0xFFFFFFFFu);
      } else {
        const uint32_t vm = partial >> (i & 31) & 1u ? vms[w * ST + stage] : 0xFFFFFFFFu;
        partial &= ~(1u << (i & 31));
        work(std::false_type{}, st, tok0, vm);
      }
      stage = stage == ST - 1 ? 0 : stage + 1;
      ahead = ahead == ST - 1 ? 0 : ahead + 1;
    }

    // ---- the middle's sums: undo the numerators' scale, apply g_v, turn back along the channels ----
    if (n_my > 0) {
      constexpr float kUndo = 1.0f / 1024.0f;
      const float gv = p.v.gscale[p.v.gstride * sq.s] * kUndo;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          l[n][c] *= kUndo;
          if (p.v.rotate) {
            if constexpr (D == 64) {
              // 8 channels here, the other 8 of the block in the lane of g ^ 1
              float a[8];
#pragma unroll
              for (int i = 0; i < 4; ++i) a[2 * i] = O[i][n][c], a[2 * i + 1] = O[i][n][c + 2];
#pragma unroll
              for (int h = 1; h < 8; h <<= 1)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                  if ((i & h) == 0) {
                    const float u = a[i], v = a[i + h];
                    a[i] = u + v;
                    a[i + h] = u - v;
                  }
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const float o = __shfl_xor_sync(0xFFFFFFFFu, a[i], 4);
                a[i] = 0.25f * (g & 1 ? o - a[i] : a[i] + o);
              }
#pragma unroll
              for (int i = 0; i < 4; ++i) O[i][n][c] = a[2 * i], O[i][n][c + 2] = a[2 * i + 1];
            } else {
#pragma unroll
              for (int blk = 0; blk < NO / 8; ++blk) {
                float a[16];
#pragma unroll
                for (int i = 0; i < 8; ++i) a[2 * i] = O[8 * blk + i][n][c], a[2 * i + 1] = O[8 * blk + i][n][c + 2];
                fwht16(a);
#pragma unroll
                for (int i = 0; i < 8; ++i) O[8 * blk + i][n][c] = a[2 * i], O[8 * blk + i][n][c + 2] = a[2 * i + 1];
              }
            }
          }
#pragma unroll
          for (int i = 0; i < NO; ++i) {
            O[i][n][c] *= gv;
            O[i][n][c + 2] *= gv;
          }
        }
    }

    // ---- the BF16 ends, 16 tokens a tile ----
    for (int e = e_first; e < e_end; e += kKaWarps) {
      const bool in_sink = e < sink_tiles;
      const int r0 = 16 * (in_sink ? e : e - sink_tiles), cnt = min(16, (in_sink ? sq.ns : sq.nw) - r0);
      const int pos0 = in_sink ? r0 : sq.ns + sq.nm + r0;
      const int rows = in_sink ? p.sink_rows : p.window_rows;
      const int64_t mat = ((int64_t)sq.s * p.Hkv + kvh) * rows;
      const bool cut = pos0 + cnt > lim_min;       // some row does not see all of the tile
      auto row_at = [&](const KvSide& s, int r) -> const char* {
        int at = r0 + r;
        if (!in_sink) {
          at += sq.head;
          if (at >= rows) at -= rows;
        }
        return (in_sink ? s.sink : s.window) + (mat + at) * (D * 2);
      };
      float S[NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 4; ++c) S[n][c] = 0.0f;
      const bool ok0 = perm < cnt, ok1 = perm + 8 < cnt;
      const char* k0 = row_at(p.k, ok0 ? perm : 0);
      const char* k1 = row_at(p.k, ok1 ? perm + 8 : 0);
#pragma unroll
      for (int cc = 0; cc < KCH; ++cc)
#pragma unroll
        for (int v8 = 0; v8 < KW; ++v8) {          // 8 channels of the chunk: two steps
          uint4 u = make_uint4(0, 0, 0, 0), v = u;
          const int at = ((t + 4 * cc) * (KW * 8) + v8 * 8) * 2;
          if (ok0) u = *reinterpret_cast<const uint4*>(k0 + at);
          if (ok1) v = *reinterpret_cast<const uint4*>(k1 + at);
          const int j = cc * 8 + v8 * 2;
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const int at = (n * NS + j) * 32 + lane;
            mma16816<true>(S[n], u.x, v.x, u.y, v.y, qe[at].x, qe[at].y);
            mma16816<true>(S[n], u.z, v.z, u.w, v.w, qe[at + 32].x, qe[at + 32].y);
            if constexpr (!QBF) {
              mma16816<true>(S[n], u.x, v.x, u.y, v.y, qr[at].x, qr[at].y);
              mma16816<true>(S[n], u.z, v.z, u.w, v.w, qr[at + 32].x, qr[at + 32].y);
            }
          }
        }
      float mx[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          mx[n][c] = -INFINITY;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int r = perm + 8 * h;
            float& s = S[n][c + 2 * h];
            s = r < cnt && pos0 + r < lim[n][c] ? s * p.scale_log2 : -INFINITY;
            mx[n][c] = fmaxf(mx[n][c], s);
          }
        }
      raise(mx);
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const float ms = finite_or_zero(m[n][c]);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            S[n][c + 2 * h] = ex2(S[n][c + 2 * h] - ms);
            l[n][c] += S[n][c + 2 * h];
          }
        }
      uint32_t ph[NT][2], pl[NT][2];               // numerators as two BF16 terms
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t a, c;
          split_bf16(S[n][2 * h], S[n][2 * h + 1], a, c);
          ph[n][h] = movmatrix(a);
          pl[n][h] = movmatrix(c);
        }
#pragma unroll
      for (int v8 = 0; v8 < D / 64; ++v8) {        // 8 channels of the thread's chunk
        uint4 vv[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const bool ok = 4 * r + t < cnt;
          vv[r] = make_uint4(0, 0, 0, 0);
          if (ok) vv[r] = *reinterpret_cast<const uint4*>(row_at(p.v, 4 * r + t) + (g * (D / 8) + v8 * 8) * 2);
        }
        bool odd = false;                          // an infinity or NaN in a tile that some row does not see all of
        if (cut) {
#pragma unroll
          for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int k = 0; k < 4; ++k) odd |= (&vv[r].x)[k] != finite_bf16x2((&vv[r].x)[k]);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t w0 = (&vv[0].x)[k], w1 = (&vv[1].x)[k], w2 = (&vv[2].x)[k], w3 = (&vv[3].x)[k];
          if (cut) w0 = finite_bf16x2(w0), w1 = finite_bf16x2(w1), w2 = finite_bf16x2(w2), w3 = finite_bf16x2(w3);
          const uint32_t a0 = __byte_perm(w0, w1, 0x5410), a1 = __byte_perm(w0, w1, 0x7632);
          const uint32_t a2 = __byte_perm(w2, w3, 0x5410), a3 = __byte_perm(w2, w3, 0x7632);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            mma16816<true>(O[4 * v8 + k][n], a0, a1, a2, a3, ph[n][0], ph[n][1]);
            mma16816<true>(O[4 * v8 + k][n], a0, a1, a2, a3, pl[n][0], pl[n][1]);
          }
        }
        if (__any_sync(0xFFFFFFFFu, odd)) {
          // infinities and NaN are added token by token to the rows that see them (the product would multiply a
          // hidden token's by its zero numerator and make every row NaN)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            for (int tt = 0; tt < 4; ++tt) {
              uint32_t wd[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) wd[k] = __shfl_sync(0xFFFFFFFFu, (&vv[r].x)[k], g * 4 + tt);
              const int tk = 4 * r + tt, fr = 2 * tt + (r & 1);     // the token's fragment row is fr + 8 (r >> 1)
#pragma unroll
              for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                  const float pr = __shfl_sync(0xFFFFFFFFu, S[n][c + 2 * (r >> 1)], fr * 4 + t);
                  if (tk < cnt && pos0 + tk < lim[n][c]) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                      const uint32_t f = finite_bf16x2(wd[k]);
                      if ((wd[k] ^ f) & 0xFFFFu) O[4 * v8 + k][n][c] += pr * bf16lo(wd[k]);
                      if ((wd[k] ^ f) >> 16) O[4 * v8 + k][n][c + 2] += pr * bf16hi(wd[k]);
                    }
                  }
                }
            }
          }
        }
      }
    }

    // ---- join the warps ----
    // The joining kernel may be launched from here on: earlier, its waiting CTAs fill the SMs that have room first and
    // stay together there (one long sequence 21.9 against 19.9 us).
    if (u >= u_end) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) l[n][c] += __shfl_xor_sync(0xFFFFFFFFu, l[n][c], o);
        if (g == 0) stat[w * ROWS + 8 * n + 2 * t + c] = make_float2(m[n][c], l[n][c]);
      }
    cp_async_wait<0>();
    __syncthreads();                               // every warp is done with its ring: the accumulators take its place
    float* acc = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int row = 8 * n + 2 * t + c;
        float mm = -INFINITY;
#pragma unroll
        for (int k = 0; k < kKaWarps; ++k) mm = fmaxf(mm, stat[k * ROWS + row].x);
        const float f = ex2(m[n][c] - finite_or_zero(mm));
        float* a = acc + (w * ROWS + row) * Sm::kAccRow + g * (D / 8);
#pragma unroll
        for (int i = 0; i < NO; ++i) *reinterpret_cast<float2*>(a + 2 * i) = make_float2(O[i][n][c] * f, O[i][n][c + 2] * f);
      }
    __syncthreads();
    for (int v = tid; v < ROWS * (D / 4); v += kKaWarps * 32) {
      const int row = v / (D / 4), d = 4 * (v % (D / 4)), r = row_tile * ROWS + row;
      if (r >= p.R) continue;
      float mm = -INFINITY, ll = 0.0f;
#pragma unroll
      for (int k = 0; k < kKaWarps; ++k) mm = fmaxf(mm, stat[k * ROWS + row].x);
      float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int k = 0; k < kKaWarps; ++k) {
        const float2 ml = stat[k * ROWS + row];
        ll = fmaf(ml.y, ex2(ml.x - finite_or_zero(mm)), ll);
        const float4 x = *reinterpret_cast<const float4*>(acc + (k * ROWS + row) * Sm::kAccRow + d);
        s.x += x.x, s.y += x.y, s.z += x.z, s.w += x.w;
      }
      const int i = r / p.G, hq = kvh * p.G + r % p.G;
      if (first_unit > 0 || last_unit < units) {     // shared with other parts
        const int64_t at = ((int64_t)part * 2 + (first_unit > 0 ? 0 : 1)) * ROWS + row;
        *reinterpret_cast<float4*>(p.ws_o + at * D + d) = s;
        if (d == 0) p.ws_ml[at] = make_float2(mm, ll);
      } else {
        const float inv = ll == 0.0f ? 0.0f : 1.0f / ll;   // no visible token: zeros
        const int64_t at = b * p.o_sb + hq * p.o_sh + i * p.o_st + d;
        ka_store<QBF>(p.out, at, s.x * inv);
        ka_store<QBF>(p.out, at + 1, s.y * inv);
        ka_store<QBF>(p.out, at + 2, s.z * inv);
        ka_store<QBF>(p.out, at + 3, s.w * inv);
        if (d == 0 && p.lse) p.lse[((int64_t)b * p.Hq + hq) * p.Tq + i] = ll == 0.0f ? -INFINITY : (mm + log2f(ll)) * 0.6931471805599453f;
      }
    }
    __syncthreads();                             // the next job takes the shared memory
  }
}

// Joins the jobs that cuts fall into, a CTA per entry of ws_meta and query row.  Entries per part alone would launch
// thousands of CTAs that find nothing to do: draft tokens 15.3 against 13.7 us, D = 256 38.0 / 35.7, one long sequence
// 20.8 / 19.9; 48 ragged sequences, where nearly every part begins a job that is cut, 46.3 / 47.2.
template <int D, int NT, bool QBF>
__global__ void __launch_bounds__(kKaJoinWarps * 32) kv_attn_combine_kernel(const __grid_constant__ KvAttnParams p) {
  constexpr int E = D / 32, ROWS = 8 * NT;       // channels per lane
  __shared__ float part[kKaJoinWarps][D];
  __shared__ float2 stat[kKaJoinWarps];          // the warps' references and denominators
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int4 job = p.ws_meta[blockIdx.x];
  if (job.w < 0) return;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, row = blockIdx.y, pieces = job.w - job.z + 1;
  const int kvh = job.y / p.row_tiles, r = (job.y - kvh * p.row_tiles) * ROWS + row, b = job.x;
  if (r >= p.R) return;
  // piece 0: the end of the part that begins the job; piece i: the beginning of the i-th part after it
  auto piece = [&](int i) -> int64_t { return ((int64_t)(job.z + i) * 2 + (i == 0 ? 1 : 0)) * ROWS + row; };
  // every warp its pieces under its own maximum, statistics and sums fetched together: one round trip, not two (one long
  // sequence 19.9 -> 18.3 us)
  float m = -INFINITY, l = 0.0f, s[E];
#pragma unroll
  for (int k = 0; k < E; ++k) s[k] = 0.0f;
  for (int i = w; i < pieces; i += 4 * kKaJoinWarps) {
    float2 st[4];
    float v[4][E];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int at = i + j * kKaJoinWarps;
      st[j] = make_float2(-INFINITY, 0.0f);
#pragma unroll
      for (int k = 0; k < E; ++k) v[j][k] = 0.0f;
      if (at < pieces) {
        st[j] = p.ws_ml[piece(at)];
#pragma unroll
        for (int k = 0; k < E; k += 2) {
          const float2 x = *reinterpret_cast<const float2*>(p.ws_o + piece(at) * D + lane * E + k);
          v[j][k] = x.x, v[j][k + 1] = x.y;
        }
      }
    }
    const float mn = fmaxf(m, fmaxf(fmaxf(st[0].x, st[1].x), fmaxf(st[2].x, st[3].x))), ms = finite_or_zero(mn);
    const float f = ex2(m - ms);
    m = mn;
    l *= f;
#pragma unroll
    for (int k = 0; k < E; ++k) s[k] *= f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float fj = ex2(st[j].x - ms);
      l = fmaf(st[j].y, fj, l);
#pragma unroll
      for (int k = 0; k < E; ++k) s[k] = fmaf(v[j][k], fj, s[k]);
    }
  }
#pragma unroll
  for (int k = 0; k < E; ++k) part[w][lane * E + k] = s[k];
  if (lane == 0) stat[w] = make_float2(m, l);
  __syncthreads();
  float mm = -INFINITY, ll = 0.0f, fw[kKaJoinWarps];
#pragma unroll
  for (int k = 0; k < kKaJoinWarps; ++k) mm = fmaxf(mm, stat[k].x);
#pragma unroll
  for (int k = 0; k < kKaJoinWarps; ++k) {
    fw[k] = ex2(stat[k].x - finite_or_zero(mm));
    ll = fmaf(stat[k].y, fw[k], ll);
  }
  const float inv = ll == 0.0f ? 0.0f : 1.0f / ll;
  const int i = r / p.G, hq = kvh * p.G + r % p.G;
  const int64_t at = b * p.o_sb + hq * p.o_sh + i * p.o_st;
  for (int d = threadIdx.x; d < D; d += kKaJoinWarps * 32) {
    float x = 0.0f;
#pragma unroll
    for (int k = 0; k < kKaJoinWarps; ++k) x = fmaf(part[k][d], fw[k], x);
    ka_store<QBF>(p.out, at + d, x * inv);
  }
  if (threadIdx.x == 0 && p.lse)
    p.lse[((int64_t)b * p.Hq + hq) * p.Tq + i] = ll == 0.0f ? -INFINITY : (mm + log2f(ll)) * 0.6931471805599453f;
}

}  // namespace nvfp4
