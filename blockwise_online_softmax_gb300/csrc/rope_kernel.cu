// Per-head RMS norm of q and k with rotary positions, its gradient, and the
// form that writes k and v into their pages.
//
// For a row x of d columns (one head of one token at position p):
//   r = rsqrt(mean(x^2) + eps),  y = x r w          (or y = x without a weight)
//   pair i < R/2 of the rotated columns (i, i + R/2), or (2i, 2i + 1) when
//   interleaved:  (a, b) -> mscale (a cos t - b sin t, b cos t + a sin t),
//   t = 2 pi frac(p f_i); the other columns keep y.
// Gradient, with g the incoming gradient turned back by -t (times mscale):
//   dw = sum over rows of g x r,   u = g w,
//   dx = r (u - x r^2 mean(u x)).
//
// The frequency f_i comes as turns per position in units of 2^-64, so
// p f_i modulo one turn is a wrapping 64-bit product: exact for any 32-bit
// position, where fp32 angles lose all their bits near a million positions
// and fp64 arithmetic runs at 1/64 of the fp32 rate.  The top 32 bits go to
// sincospif.  Sums, the norm and the rotation are fp32; the one rounding to
// bf16 is at the store.
#include <cstdint>

#include <cuda_bf16.h>

#include "serve_internal.h"

namespace ra {
namespace {

constexpr int kWarps = 8;  // per CTA
constexpr unsigned kAll = 0xffffffffu;

// Eight consecutive columns as a lane loads and stores them.
template <typename T>
struct Vec;
template <>
struct Vec<__nv_bfloat16> {
  uint4 w;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    w = *reinterpret_cast<const uint4*>(p);  // not __ldg: the output may be the input
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(u[i] << 16);
      x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, const float (&x)[8]) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      u[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
  }
};
template <>
struct Vec<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = *reinterpret_cast<const float4*>(p);
    b = *(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  }
  static __device__ __forceinline__ void store(float* p, const float (&x)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
  }
};

__device__ __forceinline__ void load_weight(const void* w, int bf16, int col, float (&x)[8]) {
  if (bf16) {
    Vec<__nv_bfloat16> v;
    v.load(static_cast<const __nv_bfloat16*>(w) + col);
    v.get(x);
  } else {
    Vec<float> v;
    v.load(static_cast<const float*>(w) + col);
    v.get(x);
  }
}

__device__ __forceinline__ long long row_position(const RopeArgs& a, long long t) {
  if (a.positions) return a.positions[t];
  if (a.layout == kContiguous) return t;
  const PosMap m{a.layout, a.P, a.c, t / a.c, 0};
  return pos_of(m, t % a.c);
}

// What a lane needs to rotate its eight columns: out[e] = x[e] cs[e] +
// partner[e] sn[e], where the partner column is x[e ^ 1] (interleaved) or
// column e of lane `mate`, and sn carries the sign.
template <int D, bool INTER>
struct Rot {
  static constexpr int LPR = D / 8;  // lanes per row
  float cs[8], sn[8];
  int mate;     // lane that holds the partner columns
  bool on;      // this lane's columns are rotated

  __device__ __forceinline__ void place(int rot, int lane) {
    const int s = lane % LPR, half = rot / 16;
    on = s < rot / 8;
    mate = !on ? lane : (s < half ? lane + half : lane - half);
  }
  __device__ __forceinline__ void angles(const RopeArgs& a, long long pos, int lane) {
    const int s = lane % LPR, half = a.rot / 16;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      cs[e] = 1.f;
      sn[e] = 0.f;
    }
    if (!on) return;
    constexpr int N = INTER ? 4 : 8;
    const int i0 = INTER ? 4 * s : 8 * (s < half ? s : s - half);
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const unsigned long long turn = static_cast<unsigned long long>(pos) * __ldg(a.phases + i0 + j);
      float sv, cv;
      sincospif(static_cast<float>(static_cast<int>(turn >> 32)) * 0x1p-31f, &sv, &cv);
      sv *= a.mscale;
      cv *= a.mscale;
      if (INTER) {
        cs[2 * j] = cs[2 * j + 1] = cv;
        sn[2 * j] = -sv;
        sn[2 * j + 1] = sv;
      } else {
        cs[j] = cv;
        sn[j] = s < half ? -sv : sv;
      }
    }
  }
  // dir = 1: rotate; dir = -1: turn back (the transpose).
  template <int DIR>
  __device__ __forceinline__ void apply(float (&x)[8]) const {
    float p[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
      p[e] = INTER ? x[e ^ 1] : __shfl_sync(kAll, x[e], mate);
    if (!on) return;
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = x[e] * cs[e] + (DIR > 0 ? p[e] : -p[e]) * sn[e];
  }
};

template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}

// Forward (APPEND: with k and v written to their pages).  A warp takes a
// token, or one of a.parts shares of its rows; LPR lanes hold a row, so an
// iteration covers 32 / LPR rows.  cos and sin are computed once per token.
template <typename T, int D, bool INTER, bool APPEND>
__global__ void __launch_bounds__(kWarps * 32) rope_forward_kernel(const RopeArgs a) {
  constexpr int LPR = D / 8, RPI = 32 / LPR;
  const int lane = threadIdx.x & 31, col = 8 * (lane % LPR), sub = lane / LPR;
  const int rows = a.heads + a.kv_heads + (APPEND ? a.kv_heads : 0);
  const int groups = (rows + RPI - 1) / RPI;
  const int per = (groups + a.parts - 1) / a.parts;
  const long long items = a.T * a.parts;
  const long long nwarps = static_cast<long long>(gridDim.x) * kWarps;
  float wq[8], wk[8];
  if (a.qw) load_weight(a.qw, a.w_bf16, col, wq);
  if (a.kw) load_weight(a.kw, a.w_bf16, col, wk);
  Rot<D, INTER> rot;
  rot.place(a.rot, lane);
  for (long long it = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5); it < items;
       it += nwarps) {
    const long long t = it / a.parts;
    const int g0 = static_cast<int>(it % a.parts) * per;
    const int g1 = g0 + per < groups ? g0 + per : groups;
    long long slot = 0;
    if (APPEND) {
      slot = a.slots[t];
      if (slot < 0 || slot >= a.n_slots) continue;  // a padding row: nothing is written
    }
    rot.angles(a, row_position(a, t), lane);
    for (int g = g0; g < g1; ++g) {
      const int row = g * RPI + sub;
      const bool valid = row < rows;
      const bool is_q = row < a.heads, is_v = APPEND && row >= a.heads + a.kv_heads;
      const int h = is_q ? row : (is_v ? row - a.heads - a.kv_heads : row - a.heads);
      const T* src = static_cast<const T*>(is_q ? a.q : (is_v ? a.v : a.k)) +
                     t * (is_q ? a.q_str : (is_v ? a.v_str : a.k_str)) + h * D + col;
      T* dst;
      if (is_q) {
        dst = static_cast<T*>(a.qo) + t * a.qo_str + h * D + col;
      } else if (APPEND) {
        const long long page = slot >> a.page_shift;
        const long long in = slot & ((1LL << a.page_shift) - 1);
        dst = static_cast<T*>(is_v ? a.vc : a.kc) + page * (is_v ? a.vc_page : a.kc_page) +
              (in * a.kv_heads + h) * D + col;
      } else {
        dst = static_cast<T*>(a.ko) + t * a.ko_str + h * D + col;
      }
      Vec<T> raw;
      float x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = 0.f;
      if (valid) {
        raw.load(src);
        raw.get(x);
      }
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
      ss = row_sum<LPR>(ss);
      const float r = rsqrtf(ss * (1.f / D) + a.eps);
      float y[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        y[e] = x[e];
        if (is_q ? a.qw != nullptr : a.kw != nullptr) y[e] = x[e] * r * (is_q ? wq[e] : wk[e]);
      }
      rot.template apply<1>(y);
      if (valid) Vec<T>::store(dst, is_v ? x : y);
    }
  }
}

// Backward.  Rows as in the forward; the weight gradients are summed in the
// lanes, over the CTA's warps in shared memory, and written as one partial
// sum per CTA, so their order is fixed.
template <typename T, int D, bool INTER>
__global__ void __launch_bounds__(kWarps * 32) rope_backward_kernel(const RopeArgs a) {
  constexpr int LPR = D / 8, RPI = 32 / LPR;
  __shared__ float s_dw[kWarps][2][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = 8 * (lane % LPR), sub = lane / LPR;
  const int rows = a.heads + a.kv_heads;
  const int groups = (rows + RPI - 1) / RPI;
  const long long nwarps = static_cast<long long>(gridDim.x) * kWarps;
  float wq[8], wk[8], dwq[8], dwk[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) wq[e] = wk[e] = dwq[e] = dwk[e] = 0.f;
  if (a.qw) load_weight(a.qw, a.w_bf16, col, wq);
  if (a.kw) load_weight(a.kw, a.w_bf16, col, wk);
  Rot<D, INTER> rot;
  rot.place(a.rot, lane);
  for (long long t = static_cast<long long>(blockIdx.x) * kWarps + warp; t < a.T; t += nwarps) {
    rot.angles(a, row_position(a, t), lane);
    for (int g = 0; g < groups; ++g) {
      const int row = g * RPI + sub;
      const bool valid = row < rows, is_q = row < a.heads;
      const int h = is_q ? row : row - a.heads;
      float x[8], gy[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = gy[e] = 0.f;
      if (valid) {
        Vec<T> raw;
        Vec<float> gr;
        raw.load(static_cast<const T*>(is_q ? a.q : a.k) + t * (is_q ? a.q_str : a.k_str) + h * D + col);
        gr.load((is_q ? a.dqo : a.dko) + (t * (is_q ? a.heads : a.kv_heads) + h) * D + col);
        raw.get(x);
        gr.get(gy);
      }
      rot.template apply<-1>(gy);
      const bool norm = is_q ? a.qw != nullptr : a.kw != nullptr;
      float ss = 0.f, ux = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        ss = fmaf(x[e], x[e], ss);
        ux = fmaf(gy[e] * (is_q ? wq[e] : wk[e]), x[e], ux);
      }
      ss = row_sum<LPR>(ss);
      ux = row_sum<LPR>(ux);
      const float r = rsqrtf(ss * (1.f / D) + a.eps);
      const float m = r * r * ux * (1.f / D);
      float dx[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float hat = x[e] * r;
        if (is_q) dwq[e] = fmaf(gy[e], hat, dwq[e]);
        else dwk[e] = fmaf(gy[e], hat, dwk[e]);
        dx[e] = norm ? r * (gy[e] * (is_q ? wq[e] : wk[e]) - x[e] * m) : gy[e];
      }
      if (valid)
        Vec<T>::store(static_cast<T*>(is_q ? a.qo : a.ko) + t * (is_q ? a.qo_str : a.ko_str) + h * D + col, dx);
    }
  }
  if (!a.dw) return;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
#pragma unroll
    for (int o = LPR; o < 32; o <<= 1) {
      dwq[e] += __shfl_xor_sync(kAll, dwq[e], o);
      dwk[e] += __shfl_xor_sync(kAll, dwk[e], o);
    }
    if (sub == 0) {
      s_dw[warp][0][col + e] = dwq[e];
      s_dw[warp][1][col + e] = dwk[e];
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * D; i += kWarps * 32) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) s += s_dw[w][i / D][i % D];
    a.dw[static_cast<long long>(blockIdx.x) * 2 * D + i] = s;
  }
}

// One CTA per 32 of the 2 d weight gradients: warp w sums the partials w,
// w + 8, ... of its 32 columns, then the warps' sums meet in shared memory.
__global__ void __launch_bounds__(kWarps * 32) rope_weight_grad_kernel(const RopeArgs a, int n, int d) {
  __shared__ float s[kWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int i = blockIdx.x * 32 + lane;
  float x = 0.f;
  for (int p = warp; p < n; p += kWarps) x += a.dw[static_cast<long long>(p) * 2 * d + i];
  s[warp][lane] = x;
  __syncthreads();
  if (warp) return;
#pragma unroll
  for (int w = 1; w < kWarps; ++w) x += s[w][lane];
  float* dst = i < d ? a.dqw : a.dkw;
  if (dst) dst[i % d] = x;
}

int sm_count() {
  int dev = 0, sms = 152;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return sms;
}

template <typename T, bool APPEND>
cudaError_t forward_t(RopeArgs a, int d, cudaStream_t st) {
  if (a.T == 0) return cudaSuccess;
  a.parts = 1;
  long long ctas = (a.T * a.parts + kWarps - 1) / kWarps;
  const long long most = 8LL * sm_count();
  const unsigned grid = static_cast<unsigned>(ctas < most ? ctas : most);
  if (d == 128) {
    if (a.interleaved) rope_forward_kernel<T, 128, true, APPEND><<<grid, kWarps * 32, 0, st>>>(a);
    else rope_forward_kernel<T, 128, false, APPEND><<<grid, kWarps * 32, 0, st>>>(a);
  } else {
    if (a.interleaved) rope_forward_kernel<T, 64, true, APPEND><<<grid, kWarps * 32, 0, st>>>(a);
    else rope_forward_kernel<T, 64, false, APPEND><<<grid, kWarps * 32, 0, st>>>(a);
  }
  return cudaGetLastError();
}

template <typename T>
cudaError_t backward_t(const RopeArgs& a, int d, cudaStream_t st) {
  const unsigned grid = static_cast<unsigned>(rope_grad_ctas(a));
  if (d == 128) {
    if (a.interleaved) rope_backward_kernel<T, 128, true><<<grid, kWarps * 32, 0, st>>>(a);
    else rope_backward_kernel<T, 128, false><<<grid, kWarps * 32, 0, st>>>(a);
  } else {
    if (a.interleaved) rope_backward_kernel<T, 64, true><<<grid, kWarps * 32, 0, st>>>(a);
    else rope_backward_kernel<T, 64, false><<<grid, kWarps * 32, 0, st>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace

int rope_grad_ctas(const RopeArgs& a) {
  const long long ctas = (a.T + kWarps - 1) / kWarps, most = 4LL * sm_count();
  return static_cast<int>(ctas < 1 ? 1 : (ctas < most ? ctas : most));
}

cudaError_t launch_rope_forward(const RopeArgs& a, int d, bool bf16, cudaStream_t st) {
  return bf16 ? forward_t<__nv_bfloat16, false>(a, d, st) : forward_t<float, false>(a, d, st);
}

cudaError_t launch_rope_append(const RopeArgs& a, int d, cudaStream_t st) {
  return forward_t<__nv_bfloat16, true>(a, d, st);
}

cudaError_t launch_rope_backward(const RopeArgs& a, int d, bool bf16, cudaStream_t st) {
  return bf16 ? backward_t<__nv_bfloat16>(a, d, st) : backward_t<float>(a, d, st);
}

cudaError_t launch_rope_weight_grad(const RopeArgs& a, int n, int d, cudaStream_t st) {
  rope_weight_grad_kernel<<<2 * d / 32, kWarps * 32, 0, st>>>(a, n, d);
  return cudaGetLastError();
}

}  // namespace ra
