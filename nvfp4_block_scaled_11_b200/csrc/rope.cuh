// rope.cuh -- rotary positions for query and key heads, ahead of the cache's rotation and quantizer.
//
// Channel pair i of the first `rot` channels of every head turns by the angle a_i = pos * freq_i:
//   (x, y) -> mscale (x cos a_i - y sin a_i, x sin a_i + y cos a_i)
// with pairs (i, i + rot/2) ("half") or (2i, 2i + 1) ("interleaved"); the other channels pass.  The inverse
// direction turns by -a_i: with the same mscale it is the adjoint, i.e. the gradient's pass.
//
// Each element is read and written once, so the kernel is bound by memory.  The angle is formed in FP64
// (positions reach millions, where an FP32 product is off by whole radians) and reduced to a
// fraction of a turn before FP32 sincospi; a CTA does that once per token and pair and keeps it in shared
// memory for all heads of all tensors of the call.  Threads then walk (token, head) rows with 16-byte
// accesses: a thread keeps its place in the row, so no index is divided in the loop.
#pragma once

#include "device.cuh"

namespace nvfp4 {

constexpr int kRopeMaxTensors = 8, kRopeThreads = 256, kRopeMaxPairs = 512;
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
  int64_t tokens, T;                       // B * T; token j is (j / T, j % T)
  int D, rot, interleaved, pos64, tile;    // tile: tokens per CTA
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
// V consecutive elements: one 16-byte access (V = 16 / size) or V single ones.  Plain loads, since `out`
// may be x itself.
template <int DT, int V, bool VEC>
__device__ __forceinline__ void rope_load(const char* p, int64_t i, float (&f)[V]) {
  if constexpr (VEC) {
    const uint4 u = *reinterpret_cast<const uint4*>(p + i * (16 / V));
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    widen_words<DT>(w, f, 4);
  } else {
#pragma unroll
    for (int k = 0; k < V; ++k) f[k] = rope_widen<DT>(p, i + k);
  }
}
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
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeParams p) {
  constexpr int V = VEC ? (DT == DT_F32 ? 4 : 8) : (INTER ? 2 : 1);   // elements per piece
  constexpr int PP = INTER ? V / 2 : V;                               // pairs per piece (divides rot / 2)
  __shared__ float2 cs[kRopeSmemPairs];
  const int half = p.rot / 2, tid = threadIdx.x;
  const int64_t tok0 = (int64_t)blockIdx.x * p.tile;
  const int ntok = (int)min((int64_t)p.tile, p.tokens - tok0);
  for (int u = tid; u < ntok * half; u += kRopeThreads) {
    const int j = u / half, i = u - j * half;
    const int64_t tok = tok0 + j, b = tok / p.T, at = b * p.pos_b + (tok - b * p.T) * p.pos_t;
    const double pos = p.pos64 ? (double)reinterpret_cast<const long long*>(p.pos)[at]
                               : (double)reinterpret_cast<const int*>(p.pos)[at];
    const double turns = pos * p.freqs[i] * 0.15915494309189535;   // / (2 pi)
    float s, c;
    sincospif((float)(2.0 * (turns - rint(turns))), &s, &c);
    // kept so that the pairs of neighbouring pieces lie side by side (threads of a warp read those together)
    cs[j * half + (i % PP) * (half / PP) + i / PP] = make_float2(c * p.mscale, s * (p.mscale * p.sign));
  }
  __syncthreads();
  // pieces of a row: pairs first (two pieces in the half layout), then the channels that pass
  const int turning = INTER ? p.rot / V : half / V, pieces = turning + (p.D - p.rot) / V;
  const int64_t total = (int64_t)pieces;
  for (int64_t pc0 = 0; pc0 < total; pc0 += kRopeThreads) {   // rows of more than 256 pieces take several rounds
    const int width = (int)min((int64_t)kRopeThreads, total - pc0), rows = kRopeThreads / width;
    if (tid >= rows * width) continue;
    const int pc = (int)pc0 + tid % width;
    int row = tid / width + (int)blockIdx.y * rows, h, tok;
    const int step = rows * (int)gridDim.y;
    tok = row / p.heads;
    h = row - tok * p.heads;
    const int dt = step / p.heads, dh = step - dt * p.heads;
    for (; tok < ntok; tok += dt, h += dh) {
      if (h >= p.heads) {
        h -= p.heads;
        if (++tok >= ntok) break;
      }
      int k = 0, hh = h;
      while (hh >= p.a[k].heads) hh -= p.a[k++].heads;
      const RopeTensor& a = p.a[k];
      const int64_t g = tok0 + tok, b = g / p.T, t = g - b * p.T;
      const char* x = a.x + (b * a.xb + hh * a.xh + t * a.xt) * (DT == DT_F32 ? 4 : 2);
      char* o = a.out + (b * a.ob + hh * a.oh + t * a.ot) * (DT == DT_F32 ? 4 : 2);
      const float2* c = cs + tok * half;
      if (pc >= turning) {
        const int at = p.rot + (pc - turning) * V;
        float f[V];
        rope_load<DT, V, VEC>(x, at, f);
        rope_store<DT, V, VEC>(o, at, f);
      } else if constexpr (INTER) {
        float f[V];
        rope_load<DT, V, VEC>(x, pc * V, f);
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
          const float2 r = c[i * (half / PP) + pc];
          const float u = f[2 * i], v = f[2 * i + 1];
          f[2 * i] = u * r.x - v * r.y;
          f[2 * i + 1] = u * r.y + v * r.x;
        }
        rope_store<DT, V, VEC>(o, pc * V, f);
      } else {
        float f[V], s[V];
        rope_load<DT, V, VEC>(x, pc * V, f);
        rope_load<DT, V, VEC>(x, half + pc * V, s);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float2 r = c[i * (half / PP) + pc];
          const float u = f[i], v = s[i];
          f[i] = u * r.x - v * r.y;
          s[i] = u * r.y + v * r.x;
        }
        rope_store<DT, V, VEC>(o, pc * V, f);
        rope_store<DT, V, VEC>(o, half + pc * V, s);
      }
    }
  }
}

}  // namespace nvfp4
