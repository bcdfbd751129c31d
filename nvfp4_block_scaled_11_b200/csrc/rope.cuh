// rope.cuh -- rotary positions for query and key heads, ahead of the cache's rotation and quantizer.
//
// Channel pair i of the first `rot` channels of every head turns by the angle a_i = pos * freq_i:
//   (x, y) -> mscale (x cos a_i - y sin a_i, x sin a_i + y cos a_i)
// with pairs (i, i + rot/2) ("half") or (2i, 2i + 1) ("interleaved"); the other channels pass.  The inverse
// direction turns by -a_i: with the same mscale it is the adjoint, i.e. the gradient's pass.
//
// Each element is read and written once, so the kernel is bound by memory, or by latency when a call is small.  The
// angle is formed in FP64 (positions reach millions, where an FP32 product is off by whole radians) and reduced to a
// fraction of a turn before FP32 sincospi (that rounds it by up to 2^-25 half turns, 9.4e-8 radians, at any position:
// about the FP32 sine's own error, and nothing beside BF16's or FP16's rounding); a CTA does that once per token and
// pair and keeps it in shared memory for all heads of all tensors of the call.  Threads then walk (token, head) rows
// with 16-byte accesses: a thread keeps its place in the row, so no index is divided in the loop, and its first rows
// are fetched before the angles are computed.  Measured in a graph, into kept outputs and into new ones: 8192 tokens
// of 32 + 8 heads, 128 channels, BF16: 31.8 and 32.6 to 32.9 us for 168 MB, 5.1 to 5.3 TB/s; 2 x 2047 tokens of 16 +
// 16 heads, 64 channels, FP32, interleaved, 32 of them turning: 15.1 and 15.4 to 15.6 us for 67 MB; one token of 48
// sequences: 2.9 to 3.1 us, a launch and two dependent loads.  What is left is each CTA's start, which all CTAs of a
// wave share: positions, frequencies, angles and the barrier, with one row per thread in flight.
#pragma once

#include "device.cuh"

namespace nvfp4 {

constexpr int kRopeMaxTensors = 8, kRopeThreads = 256, kRopeMaxPairs = 512;
constexpr int kRopeCtasPerSm = 5;          // 48 registers (40 for six CTAs: no faster)
constexpr int kRopeSmemPairs = 2048;       // (token, pair) angles of a CTA: 16 KB

struct RopeTensor {
  const char* x;
  char* out;
  int heads;
  int64_t xb, xh, xt, ob, oh, ot;          // strides in elements
};
struct RopeParams {
  RopeTensor a[kRopeMaxTensors];
  int count, heads;                        // tensors; heads of all of them
  int T, tiles;                            // tokens of a sequence, and the CTAs that share them
  int D, rot, interleaved, pos64, tile;    // tile: tokens per CTA (of one sequence)
  const void* pos;                         // int32 / int64, element b * pos_b + t * pos_t
  int64_t pos_b, pos_t;
  const double* freqs;                     // rot / 2
  float mscale, sign;
};

template <int DT>
__device__ __forceinline__ float rope_widen(const char* p, int64_t i) {
  if (DT == DT_F32) return reinterpret_cast<const float*>(p)[i];
  if (DT == DT_BF16) return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p)[i]);
  return __half2float(reinterpret_cast<const __half*>(p)[i]);
}
template <int DT>
__device__ __forceinline__ void rope_narrow(char* p, int64_t i, float x) {
  if (DT == DT_F32) reinterpret_cast<float*>(p)[i] = x;
  else if (DT == DT_BF16) reinterpret_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(x);
  else reinterpret_cast<__half*>(p)[i] = __float2half_rn(x);
}
// V consecutive elements as they lie: one 16-byte access (V = 16 / size), or V single ones.  Plain loads, since `out` may
// be x itself.
template <int DT, int V, bool VEC>
struct RopePiece {
  uint4 raw;
  float one[VEC ? 1 : V];
  __device__ __forceinline__ void load(const char* p, int64_t i) {
    if constexpr (VEC) {
      raw = *reinterpret_cast<const uint4*>(p + i * (16 / V));
    } else {
#pragma unroll
      for (int k = 0; k < V; ++k) one[k] = rope_widen<DT>(p, i + k);
    }
  }
  __device__ __forceinline__ void widen(float (&f)[V]) const {
    if constexpr (VEC) {
      const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
      widen_words<DT>(w, f, 4);
    } else {
#pragma unroll
      for (int k = 0; k < V; ++k) f[k] = one[k];
    }
  }
};
template <int DT, int V, bool VEC>
__device__ __forceinline__ void rope_store(char* p, int64_t i, const float (&f)[V]) {
  if constexpr (VEC) {
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if constexpr (DT == DT_F32) {
        w[k] = __float_as_uint(f[k]);
      } else if constexpr (DT == DT_BF16) {
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[k]) : "f"(f[2 * k + 1]), "f"(f[2 * k]));
      } else {
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w[k]) : "f"(f[2 * k + 1]), "f"(f[2 * k]));
      }
    }
    *reinterpret_cast<uint4*>(p + i * (16 / V)) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
#pragma unroll
    for (int k = 0; k < V; ++k) rope_narrow<DT>(p, i + k, f[k]);
  }
}

// VEC: every row, pair half and passing part is a whole number of aligned 16-byte pieces.
template <int DT, bool INTER, bool VEC>
__global__ void __launch_bounds__(kRopeThreads, kRopeCtasPerSm) rope_kernel(const __grid_constant__ RopeParams p) {
  constexpr int V = VEC ? (DT == DT_F32 ? 4 : 8) : (INTER ? 2 : 1);   // elements per piece
  constexpr int PP = INTER ? V / 2 : V;                               // pairs per piece (divides rot / 2)
  __shared__ float2 cs[kRopeSmemPairs];
  constexpr int ES = DT == DT_F32 ? 4 : 2, U = INTER ? 2 : 1;          // rows per step (a row of the half layout is two loads)
  const int half = p.rot / 2, tid = threadIdx.x;
  const int seq = blockIdx.x / p.tiles, t0 = (blockIdx.x - seq * p.tiles) * p.tile, ntok = min(p.tile, p.T - t0);
  __shared__ const char* xs[kRopeMaxTensors];                             // the tensors' first rows of this CTA
  __shared__ char* os[kRopeMaxTensors];
  if (tid < p.count) {
    xs[tid] = p.a[tid].x + (seq * p.a[tid].xb + t0 * p.a[tid].xt) * ES;
    os[tid] = p.a[tid].out + (seq * p.a[tid].ob + t0 * p.a[tid].ot) * ES;
  }
  __syncthreads();
  // pieces of a row: pairs first (two pieces in the half layout), then the channels that pass
  const int turning = INTER ? p.rot / V : half / V, pieces = turning + (p.D - p.rot) / V;
  bool ready = false;
  for (int pc0 = 0; pc0 < pieces || !ready; pc0 += kRopeThreads) {      // rows of more than 256 pieces take several rounds
    const int width = max(min(kRopeThreads, pieces - pc0), 1), rows = kRopeThreads / width;
    const int pc = pc0 + tid % width, step = rows * (int)gridDim.y, first = tid / width + (int)blockIdx.y * rows;
    int tok = tid < rows * width && pc0 < pieces ? first / p.heads : ntok, h = first % p.heads;
    const int dt = step / p.heads, dh = step - dt * p.heads;
    const bool turns = pc < turning;
    const int at = turns ? pc * V : p.rot + (pc - turning) * V;          // the piece's first channel
    struct Rows {
      char* o[U];                                                        // null: no row
      const float2* c[U];
      RopePiece<DT, V, VEC> f[U], s[U];
    } cur;
    auto fetch = [&](Rows& n) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        n.o[u] = nullptr;
        if (tok >= ntok) continue;
        int k = 0, hh = h;
        while (hh >= p.a[k].heads) hh -= p.a[k++].heads;
        const RopeTensor& a = p.a[k];
        const char* x = xs[k] + (hh * a.xh + tok * a.xt) * ES;
        n.o[u] = os[k] + (hh * a.oh + tok * a.ot) * ES;
        n.c[u] = cs + tok * half;
        n.f[u].load(x, at);
        if (!INTER && turns) n.s[u].load(x, half + at);
        tok += dt;
        h += dh;
        if (h >= p.heads) h -= p.heads, ++tok;
      }
    };
    fetch(cur);
    if (!ready) {                                                        // while the first rows are on their way
      const int lanes = max(min(half, kRopeThreads), 1), abreast = kRopeThreads / lanes, i0 = tid % lanes;
      for (int j = tid < lanes * abreast ? tid / lanes : ntok; j < ntok; j += abreast) {
        const int64_t pos_at = seq * p.pos_b + (t0 + j) * p.pos_t;
        const double pos = p.pos64 ? (double)reinterpret_cast<const long long*>(p.pos)[pos_at]
                                   : (double)reinterpret_cast<const int*>(p.pos)[pos_at];
        for (int i = i0; i < half; i += lanes) {
          const double turn = pos * p.freqs[i] * 0.15915494309189535;    // / (2 pi)
          float s, c;
          sincospif((float)(2.0 * (turn - rint(turn))), &s, &c);
          // kept so that the pairs of neighbouring pieces lie side by side (threads of a warp read those together)
          cs[j * half + (i % PP) * (half / PP) + i / PP] = make_float2(c * p.mscale, s * (p.mscale * p.sign));
        }
      }
      __syncthreads();
      ready = true;
    }
    while (cur.o[0] != nullptr) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (cur.o[u] == nullptr) continue;
        float f[V];
        cur.f[u].widen(f);
        if (turns) {
          if constexpr (INTER) {
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
              const float2 r = cur.c[u][i * (half / PP) + pc];
              const float a = f[2 * i], b = f[2 * i + 1];
              f[2 * i] = a * r.x - b * r.y;
              f[2 * i + 1] = a * r.y + b * r.x;
            }
          } else {
            float s[V];
            cur.s[u].widen(s);
#pragma unroll
            for (int i = 0; i < V; ++i) {
              const float2 r = cur.c[u][i * (half / PP) + pc];
              const float a = f[i], b = s[i];
              f[i] = a * r.x - b * r.y;
              s[i] = a * r.y + b * r.x;
            }
            rope_store<DT, V, VEC>(cur.o[u], half + at, s);
          }
        }
        rope_store<DT, V, VEC>(cur.o[u], at, f);
      }
      fetch(cur);
    }
  }
}

}  // namespace nvfp4
