// decode_api.cu -- C ABI of the decode path (include/nvfp4.h): attention over the K/V cache, rotary
// positions, page copies.  Argument validation and kernel launches.
#include <cuda_runtime.h>
#include <stdint.h>
#include <stdlib.h>
#include <string.h>

#include <algorithm>
#include <atomic>

#include "../../include/nvfp4.h"
#include "api_util.cuh"
#include "kv_attention.cuh"
#include "pages.cuh"
#include "rope.cuh"

using namespace nvfp4;

namespace {

// Raises a kernel's shared-memory limit once per device.
template <auto* kernel>
int raise_smem(int bytes) {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return NVFP4_ERR_CUDA;
  if (done.load(std::memory_order_acquire) >> dev & 1u) return NVFP4_OK;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess ||
      cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, 100) != cudaSuccess) {
    cudaGetLastError();
    return NVFP4_ERR_CUDA;
  }
  done.fetch_or(uint64_t(1) << dev, std::memory_order_release);
  return NVFP4_OK;
}

template <int D, int NT, bool QBF>
int launch_kv_attention(const KvAttnParams& p, unsigned parts, unsigned join, cudaStream_t s) {
  constexpr int smem = KaSmem<D, NT, QBF>::kBytes;
  if (int rc = raise_smem<kv_attn_kernel<D, NT, QBF>>(smem)) return rc;
  kv_attn_kernel<D, NT, QBF><<<parts, kKaWarps * 32, smem, s>>>(p);
  if (int rc = last_error()) return rc;
  if (join) {
    // launched while the first kernel drains; it waits for that kernel's results itself
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(join, std::min(p.R, 8 * NT));
    cfg.blockDim = dim3(kKaJoinWarps * 32);
    cfg.stream = s;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kv_attn_combine_kernel<D, NT, QBF>, p) != cudaSuccess) {
      cudaGetLastError();
      return NVFP4_ERR_CUDA;
    }
  }
  return last_error();
}

template <int D>
int launch_kv_attention_d(const KvAttnParams& p, bool bf, int nt, unsigned parts, unsigned join, cudaStream_t s) {
  if (nt == 1) return bf ? launch_kv_attention<D, 1, true>(p, parts, join, s) : launch_kv_attention<D, 1, false>(p, parts, join, s);
  return bf ? launch_kv_attention<D, 2, true>(p, parts, join, s) : launch_kv_attention<D, 2, false>(p, parts, join, s);
}

// Query rows of a CTA in units of 8: one K/V head's rows fit 8 for most decode steps; more rows share the
// expansion of the codes in tiles of 16.  16 sequences of 8192 tokens, 2 K/V heads, 16 rows, tiles of 16 against 8 (us):
// D = 64 17.9 / 20.4, D = 128 24.1 / 27.0, D = 256 41.6 / 44.0; 64 rows: 41.8 / 54.8, 62.4 / 78.9, 111.4 / 136.6.  Every
// tile expands the whole cache again, so many rows are far from the bytes' time (5.8 us at D = 128).
int ka_row_units(int64_t rows) { return rows <= 8 ? 1 : 2; }

// CTAs of the attention kernel that an SM holds (its launch bounds and shared memory).
int ka_ctas_per_sm(int64_t D, int nt) { return D == 256 ? 2 : D == 128 ? (nt == 1 ? 3 : 2) : (nt == 1 ? 4 : 3); }

// One side of the cache: pointers and layout into the kernel's form.  mid_rows: the longest middle that a sequence may
// have.  Its tensor scale is read even where all of its pages lie outside the pool (pages == 0: tokens that count but
// are hidden); codes and scales are not.
int ka_side(const nvfp4_kv_store& c, const nvfp4_kv_attention_desc& d, int64_t mid_rows, KvSide& o) {
  if ((c.rotate != 0 && c.rotate != 1) || (c.scale_layout != 0 && c.scale_layout != 1) ||
      (c.gscale_stride != 0 && c.gscale_stride != 1))
    return NVFP4_ERR_ARG;
  if ((d.sink_rows > 0 && c.sink == nullptr) || (d.window_rows > 0 && c.window == nullptr) ||
      (mid_rows > 0 && (c.gscale == nullptr || (d.pages > 0 && (c.codes == nullptr || c.scales == nullptr)))))
    return NVFP4_ERR_ARG;
  if (!aligned(c.sink, 16) || !aligned(c.window, 16) || !aligned(c.codes, 16) || !aligned(c.scales, 4) || !aligned(c.gscale, 4))
    return NVFP4_ERR_ALIGN;
  o.sink = static_cast<const char*>(c.sink);
  o.window = static_cast<const char*>(c.window);
  o.codes = c.codes;
  o.scales = c.scales;
  o.gscale = c.gscale;
  o.gstride = c.gscale_stride;
  o.rotate = c.rotate;
  o.tile = c.scale_layout;
  o.mat_bytes = (d.page_rows + 127) / 128 * 128 * (d.D / 64) * 4;
  o.vec16 = !c.scale_layout && d.page_rows * (d.D / 16) % 16 == 0 && aligned(c.scales, 16);
  return NVFP4_OK;
}

constexpr int64_t kMaxInt = INT_MAX;

}  // namespace

extern "C" {

int nvfp4_kv_attention_splits(int64_t B, int64_t Hkv, int64_t rows, int64_t D, int64_t max_mid, int* splits) {
  if (splits == nullptr) return NVFP4_ERR_ARG;
  if (B < 0 || Hkv < 0 || rows < 0 || max_mid < 0 || max_mid > kMaxInt || (D != 64 && D != 128 && D != 256) ||
      checked_prod({B, Hkv, rows}) < 0)
    return NVFP4_ERR_SIZE;
  *splits = 1;
  const int nt = ka_row_units(rows);
  const int64_t jobs = checked_prod({B, Hkv, (rows + 8 * nt - 1) / (8 * nt)});
  const int64_t units = (max_mid + kKaTile * kKaWarps - 1) / (kKaTile * kKaWarps) + 1 + kKaJobUnits;   // of a job, ends of up to 4 tiles
  const int64_t slots = (int64_t)sm_count() * ka_ctas_per_sm(D, nt);
  const int64_t work = checked_prod({jobs, units});
  if (jobs <= 0 || work < 0) return NVFP4_OK;
  // Short jobs (up to 4 units of work) that leave room for all of them at once keep a CTA each: nothing to join.  Against
  // parts of kKaMinUnits (us, D = 128, 8 heads, 4 rows): 64 tokens 7.4 / 9.4, 301 tokens 8.8 / 10.1, 8 and 32 sequences of 301
  // 8.9 / 10.4 and 10.0 / 13.7; just past it, 480 tokens (5 units of work) 10.2 / 10.8, 600 (6 units) 11.7 / 10.7.
  *splits = (int)(units <= 4 + kKaJobUnits && jobs <= slots ? jobs : std::min(slots, std::max<int64_t>(work / kKaMinUnits, 1)));
  return NVFP4_OK;
}

size_t nvfp4_kv_attention_workspace_bytes(int64_t rows, int64_t D, int splits) {
  if (splits <= 1 || splits > kKaMaxSplits || rows <= 0 || D <= 0 || D > 256) return 0;
  return (size_t)splits * (2 * 8 * ka_row_units(rows) * (D + 2) * 4 + 16);
}

int nvfp4_kv_attention(const nvfp4_kv_attention_desc* desc, int splits, void* workspace, size_t workspace_bytes,
                       void* stream) {
  if (desc == nullptr || splits < 1 || splits > kKaMaxSplits) return NVFP4_ERR_ARG;
  const nvfp4_kv_attention_desc& d = *desc;
  if ((d.dtype != NVFP4_BF16 && d.dtype != NVFP4_F16) || (d.causal != 0 && d.causal != 1)) return NVFP4_ERR_ARG;
  if (d.D != 64 && d.D != 128 && d.D != 256) return NVFP4_ERR_SIZE;
  if (d.B < 0 || d.Hq < 0 || d.Hkv < 0 || d.Tq < 0 || d.slots < 0 || d.sink_rows < 0 || d.window_rows < 0 || d.pages < 0 ||
      d.page_rows < 0 || d.table_cols < 0)
    return NVFP4_ERR_SIZE;
  // positions are counted in 32 bits, with room for the largest sum of the three parts
  constexpr int64_t kMaxPart = kMaxInt / 4;
  if (d.B > kMaxInt || d.Hq > kMaxInt || d.Tq > kMaxPart || d.slots > kMaxInt || d.sink_rows > kMaxPart ||
      d.window_rows > kMaxPart || d.pages > kMaxInt || d.page_rows > kMaxPart)
    return NVFP4_ERR_SIZE;
  if (d.B == 0 || d.Hq == 0 || d.Tq == 0) return NVFP4_OK;
  if (d.Hkv == 0 || d.Hq % d.Hkv != 0) return NVFP4_ERR_SIZE;
  if (d.slot == nullptr && d.B > d.slots) return NVFP4_ERR_SIZE;
  int64_t mid_rows = d.page_rows;                      // a sequence's middle at most
  if (d.table != nullptr) {
    if (d.page_rows == 0 || d.page_rows % 16 != 0) return NVFP4_ERR_SIZE;
    mid_rows = checked_prod({d.table_cols, d.page_rows});
    if (mid_rows < 0 || mid_rows > kMaxPart || checked_prod({d.slots, d.table_cols, 4}) < 0) return NVFP4_ERR_SIZE;
  } else if (d.pages < d.slots) {
    return NVFP4_ERR_SIZE;                             // slot s is page s
  }
  if (checked_prod({d.slots, d.Hkv, d.sink_rows + d.window_rows, d.D, 2}) < 0 ||
      checked_prod({d.pages, d.Hkv, (d.page_rows + 127) / 128 * 128, d.D}) < 0 ||
      d.pages * d.Hkv * d.page_rows >= (int64_t(1) << 32))       // rows are numbered in 32 bits
    return NVFP4_ERR_SIZE;
  if (d.lens == nullptr &&
      (d.n_sink < 0 || d.n_sink > d.sink_rows || d.n_mid < 0 || d.n_mid > mid_rows || d.n_window < 0 ||
       d.n_window > d.window_rows || d.head < 0 || d.head > std::max<int64_t>(d.window_rows - 1, 0)))
    return NVFP4_ERR_ARG;
  if (d.q == nullptr || d.out == nullptr) return NVFP4_ERR_ARG;
  if (!aligned(d.q, 2) || !aligned(d.out, 2) || !aligned(d.lse, 4) || !aligned(d.slot, 4) || !aligned(d.table, 4) ||
      !aligned(d.lens, 4) || !aligned(workspace, 16))
    return NVFP4_ERR_ALIGN;
  KvAttnParams p{};
  if (int rc = ka_side(d.k, d, mid_rows, p.k)) return rc;
  if (int rc = ka_side(d.v, d, mid_rows, p.v)) return rc;
  const int64_t G = d.Hq / d.Hkv, R = checked_prod({G, d.Tq});
  if (R < 0 || R > kMaxInt) return NVFP4_ERR_SIZE;
  const int nt = ka_row_units(R);
  const int64_t row_tiles = (R + 8 * nt - 1) / (8 * nt), jobs = checked_prod({d.B, d.Hkv, row_tiles});
  if (jobs < 0 || jobs > kMaxInt) return NVFP4_ERR_SIZE;
  if (splits > 1) {
    if (workspace == nullptr) return NVFP4_ERR_ARG;
    if (workspace_bytes < nvfp4_kv_attention_workspace_bytes(R, d.D, splits)) return NVFP4_ERR_SIZE;
  }
  p.q = static_cast<const char*>(d.q);
  p.out = static_cast<char*>(d.out);
  p.lse = d.lse;
  p.q_sb = d.q_sb, p.q_sh = d.q_sh, p.q_st = d.q_st;
  p.o_sb = d.out_sb, p.o_sh = d.out_sh, p.o_st = d.out_st;
  p.Hq = (int)d.Hq, p.Hkv = (int)d.Hkv, p.G = (int)G, p.Tq = (int)d.Tq, p.R = (int)R, p.row_tiles = (int)row_tiles;
  p.sink_rows = (int)d.sink_rows, p.window_rows = (int)d.window_rows, p.page_rows = (int)d.page_rows;
  p.page_shift = -1;
  if (d.page_rows > 0 && (d.page_rows & (d.page_rows - 1)) == 0) p.page_shift = __builtin_ctzll((unsigned long long)d.page_rows);
  p.slots = d.slots, p.pages = d.pages, p.cols = d.table_cols;
  p.slot = d.slot, p.table = d.table;
  p.lens = d.slots > 0 ? d.lens : nullptr;             // the kernel reads slot 0's for an unknown slot: none there is not read
  p.host_lens[0] = d.n_sink, p.host_lens[1] = d.n_mid, p.host_lens[2] = d.head, p.host_lens[3] = d.n_window;
  p.B = (int)d.B;
  p.causal = d.causal;
  p.q_vec = aligned(d.q, 16) && d.q_sb % 8 == 0 && d.q_sh % 8 == 0 && d.q_st % 8 == 0;
  p.scale_log2 = d.scale * 1.4426950408889634f;
  const int64_t ws_rows = (int64_t)splits * 2 * 8 * nt;
  p.ws_meta = static_cast<int4*>(workspace);
  p.ws_o = reinterpret_cast<float*>(p.ws_meta + splits);
  p.ws_ml = reinterpret_cast<float2*>(p.ws_o + ws_rows * d.D);
  // sequences that are all alike and parts that hold whole jobs: no cut inside a job (a job is enough for a part)
  static_assert(kKaJobUnits + 1 >= kKaMinUnits, "jobs of the least work must not be cut");
  const bool cuts = splits > 1 && !(d.lens == nullptr && d.slot == nullptr && jobs % splits == 0);
  p.by_job = jobs <= splits;
  const unsigned join = !cuts ? 0 : p.by_job ? (unsigned)jobs : (unsigned)splits;   // entries of ws_meta
  const bool bf = d.dtype == NVFP4_BF16;
  cudaStream_t s = S(stream);
  if (d.D == 64) return launch_kv_attention_d<64>(p, bf, nt, (unsigned)splits, join, s);
  if (d.D == 128) return launch_kv_attention_d<128>(p, bf, nt, (unsigned)splits, join, s);
  return launch_kv_attention_d<256>(p, bf, nt, (unsigned)splits, join, s);
}

int nvfp4_rope(const nvfp4_rope_tensor* tensors, int count, int64_t B, int64_t T, int64_t D, int64_t rot, int interleaved,
               int dtype, const void* positions, int positions64, int64_t pos_sb, int64_t pos_st, const double* freqs,
               float mscale, int inverse, void* stream) {
  if (count < 0 || count > kRopeMaxTensors || (count > 0 && tensors == nullptr) || !dtype_ok(dtype) ||
      (interleaved != 0 && interleaved != 1) || (positions64 != 0 && positions64 != 1) || (inverse != 0 && inverse != 1))
    return NVFP4_ERR_ARG;
  if (B < 0 || T < 0 || D < 0 || rot < 0 || rot > D || rot % 2 != 0 || rot / 2 > kRopeMaxPairs || D > kMaxInt || T > kMaxInt / 2 ||
      checked_prod({B, T}) < 0)
    return NVFP4_ERR_SIZE;
  RopeParams p{};
  int64_t heads = 0;
  const int es = esize(dtype), V = 16 / es;
  bool vec = D % V == 0 && rot % V == 0 && (interleaved || (rot / 2) % V == 0);
  for (int k = 0; k < count; ++k) {
    const nvfp4_rope_tensor& a = tensors[k];
    if (a.heads < 0 || a.heads > kMaxInt) return NVFP4_ERR_SIZE;
    if (a.heads == 0 || B == 0 || T == 0 || D == 0) continue;
    if (a.x == nullptr || a.out == nullptr) return NVFP4_ERR_ARG;
    if (!aligned(a.x, es) || !aligned(a.out, es)) return NVFP4_ERR_ALIGN;
    // in place only element by element: every element is written where it was read
    if (a.x == a.out && (a.x_sb != a.out_sb || a.x_sh != a.out_sh || a.x_st != a.out_st)) return NVFP4_ERR_ARG;
    vec = vec && aligned(a.x, 16) && aligned(a.out, 16) && a.x_sb % V == 0 && a.x_sh % V == 0 && a.x_st % V == 0 &&
          a.out_sb % V == 0 && a.out_sh % V == 0 && a.out_st % V == 0;
    p.a[p.count++] = RopeTensor{static_cast<const char*>(a.x), static_cast<char*>(a.out), (int)a.heads, a.x_sb, a.x_sh,
                                a.x_st, a.out_sb, a.out_sh, a.out_st};
    heads += a.heads;
  }
  if (p.count == 0) return NVFP4_OK;
  if (positions == nullptr || (rot > 0 && freqs == nullptr)) return NVFP4_ERR_ARG;
  if (!aligned(positions, positions64 ? 8 : 4) || !aligned(freqs, 8)) return NVFP4_ERR_ALIGN;
  if (heads > kMaxInt / 4096) return NVFP4_ERR_SIZE;   // (token, head) rows of a CTA are counted in 32 bits
  p.heads = (int)heads;
  p.T = (int)T;
  p.D = (int)D;
  p.rot = (int)rot;
  p.interleaved = interleaved;
  p.pos64 = positions64;
  p.pos = positions;
  p.pos_b = pos_sb;
  p.pos_t = pos_st;
  p.freqs = freqs;
  p.mscale = mscale;
  p.sign = inverse ? -1.0f : 1.0f;
  const int v = vec ? V : (interleaved ? 2 : 1);
  // odd D - rot with single pairs: pieces of two channels would miss the last one
  if (!vec && interleaved && (D - rot) % 2 != 0) return NVFP4_ERR_SIZE;
  const int64_t half = rot / 2, pieces = (interleaved ? rot : half) / v + (D - rot) / v;
  const int64_t per_pass = std::max<int64_t>(1, kRopeThreads / std::max<int64_t>(1, pieces));
  const int sms = sm_count();
  // Tokens per CTA (of one sequence): as few as make one wave of CTAs, or two or more waves where its angles would pass
  // the shared memory.  A wave that is not full costs as much as a full one; 8192 tokens of 40 heads with tiles
  // of 8 (1.4 waves) / 10 / 12 (0.9) / 16 / 24: 34.8 / 37.8 / 31.4 / 33.6 / 39.4 us, 2 x 2047 tokens of 32 heads of 64 FP32
  // channels with 4 / 6 (0.9) / 8 / 12: 16.8 / 15.0 / 16.0 / 18.7 us (into kept outputs; into new ones the
  // chosen tiles take 32.6 to 32.9 and 15.4 to 15.6).
  const int64_t most = std::min<int64_t>(std::max<int64_t>(T, 1), std::min<int64_t>(32, half ? kRopeSmemPairs / half : 32));
  const int64_t wave = (int64_t)sms * kRopeCtasPerSm, waves = (B * T + wave * most - 1) / (wave * most);
  int64_t tile = std::max<int64_t>(1, (B * T + wave * waves - 1) / (wave * waves));
  while (tile < most && B * ((T + tile - 1) / tile) > wave * waves) ++tile;    // sequences end in short tiles
  p.tile = (int)tile;
  p.tiles = (int)((T + tile - 1) / tile);
  const int64_t gx = B * p.tiles;
  if (gx > kMaxInt) return NVFP4_ERR_SIZE;
  // few tokens (a decode step): the heads of a token are shared among CTAs until there are two per SM
  const int64_t passes = (tile * heads + per_pass - 1) / per_pass;
  const int64_t gy = gx >= 2 * sms ? 1 : std::max<int64_t>(1, std::min<int64_t>({passes, (2 * sms + gx - 1) / gx, 64}));
  const dim3 grid((unsigned)gx, (unsigned)gy);
  cudaStream_t s = S(stream);
#define NVFP4_ROPE(DT)                                                              \
  do {                                                                              \
    if (interleaved) {                                                              \
      if (vec) rope_kernel<DT, true, true><<<grid, kRopeThreads, 0, s>>>(p);        \
      else rope_kernel<DT, true, false><<<grid, kRopeThreads, 0, s>>>(p);           \
    } else {                                                                        \
      if (vec) rope_kernel<DT, false, true><<<grid, kRopeThreads, 0, s>>>(p);       \
      else rope_kernel<DT, false, false><<<grid, kRopeThreads, 0, s>>>(p);          \
    }                                                                               \
  } while (0)
  if (dtype == NVFP4_F32) NVFP4_ROPE(DT_F32);
  else if (dtype == NVFP4_BF16) NVFP4_ROPE(DT_BF16);
  else NVFP4_ROPE(DT_F16);
#undef NVFP4_ROPE
  return last_error();
}

int nvfp4_copy_pages(const nvfp4_pages_array* arrays, int count, const int32_t* src, const int32_t* dst, int64_t n,
                     void* stream) {
  if (count < 0 || count > kPagesMaxArrays || (count > 0 && arrays == nullptr)) return NVFP4_ERR_ARG;
  if (n < 0 || n > kMaxInt) return NVFP4_ERR_SIZE;
  if (n > 0 && (src == nullptr || dst == nullptr)) return NVFP4_ERR_ARG;
  int64_t pages = kMaxInt;                             // pages that every array has
  for (int k = 0; k < count; ++k) {
    const nvfp4_pages_array& a = arrays[k];
    if (a.outer < 0 || a.outer > kMaxInt || a.item < 0 || a.pages < 0 || a.stride < 0) return NVFP4_ERR_SIZE;
    if (checked_prod({a.pages, a.item}) < 0 || checked_prod({a.outer, a.stride}) < 0) return NVFP4_ERR_SIZE;
    if (a.outer > 1 && a.stride < a.pages * a.item) return NVFP4_ERR_SIZE;   // pieces of pages must not overlap
    if (a.outer > 0 && a.item > 0 && a.pages > 0 && a.base == nullptr) return NVFP4_ERR_ARG;
    pages = std::min(pages, a.pages);
  }
  if (n == 0 || count == 0) return NVFP4_OK;
  for (int64_t i = 0; i < n; ++i)
    if (src[i] < 0 || src[i] >= pages || dst[i] < 0 || dst[i] >= pages) return NVFP4_ERR_ARG;
  // every destination once and none a source: all pairs move at the same time
  int32_t* v = static_cast<int32_t*>(malloc((size_t)n * 2 * sizeof(int32_t)));
  if (v == nullptr) return NVFP4_ERR_SIZE;
  memcpy(v, dst, (size_t)n * sizeof(int32_t));
  memcpy(v + n, src, (size_t)n * sizeof(int32_t));
  std::sort(v, v + n);
  std::sort(v + n, v + 2 * n);
  bool clash = false;
  for (int64_t i = 0, j = 0; i < n; ++i) {
    clash |= i > 0 && v[i] == v[i - 1];
    while (j < n && v[n + j] < v[i]) ++j;
    clash |= j < n && v[n + j] == v[i];
  }
  free(v);
  if (clash) return NVFP4_ERR_ARG;
  PagesParams p{};
  int64_t per_pair = 0;                                // CTAs for one page of every array
  for (int k = 0; k < count; ++k) {
    const nvfp4_pages_array& a = arrays[k];
    if (a.outer == 0 || a.item == 0) continue;
    PagesArray& o = p.a[p.count++];
    o.base = static_cast<char*>(a.base);
    o.stride = a.outer > 1 ? a.stride : 0;
    o.item = a.item;
    o.outer = (int)a.outer;
    o.parts = (a.item + kPagesPiece - 1) / kPagesPiece;
    const uint64_t bits = (uint64_t)reinterpret_cast<uintptr_t>(a.base) | (uint64_t)o.stride | (uint64_t)a.item;
    o.width = bits % 32 == 0 ? 32 : bits % 16 == 0 ? 16 : bits % 4 == 0 ? 4 : 1;
    const int64_t ctas = checked_prod({a.outer, o.parts});
    if (ctas < 0 || ctas > kMaxInt - per_pair) return NVFP4_ERR_SIZE;
    per_pair += ctas;
  }
  if (p.count == 0) return NVFP4_OK;
  const int64_t step = std::min<int64_t>(kPagesPairs, kMaxInt / per_pair);
  for (int64_t i = 0; i < n; i += step) {
    p.n = (int)std::min(step, n - i);
    memcpy(p.src, src + i, (size_t)p.n * sizeof(int32_t));
    memcpy(p.dst, dst + i, (size_t)p.n * sizeof(int32_t));
    int64_t total = 0;
    for (int k = 0; k < p.count; ++k) {
      p.start[k] = total;
      total += (int64_t)p.a[k].outer * p.a[k].parts * p.n;
    }
    p.start[p.count] = total;
    copy_pages_kernel<<<(unsigned)total, kPagesThreads, 0, S(stream)>>>(p);
    if (int rc = last_error()) return rc;
  }
  return NVFP4_OK;
}

}  // extern "C"
