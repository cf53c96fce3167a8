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
// and fp64 arithmetic runs at 1/64 of the fp32 rate.  The top 24 bits go to
// sincospif, the next 24 in as a small turn after it: cos and sin come good to
// an ulp (with the top 32 bits rounded to fp32 for it they were off by twice
// that; 0.8 us of the 442 below).  Sums, the norm and the rotation are fp32; the
// one rounding to bf16 is at the store.
#include <cstdint>

#include <cuda_bf16.h>

#include "launch.cuh"
#include "ptx.cuh"
#include "serve_internal.h"

namespace ra {
namespace {

constexpr int kWarps = 8;  // per CTA
constexpr float kRest = 6.283185307179586f * 0x1p-48f;  // radians of 2^-48 turns
constexpr unsigned kAll = 0xffffffffu;

// Eight consecutive columns as a lane loads and stores them.
template <typename T>
struct Vec;
template <>
struct Vec<__nv_bfloat16> {
  uint4 w;
  __device__ __forceinline__ Vec() : w(make_uint4(0u, 0u, 0u, 0u)) {}
  static __device__ __forceinline__ Vec ones() {
    Vec v;
    v.w = make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u);
    return v;
  }
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
  __device__ __forceinline__ void put(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = w; }
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
  __device__ __forceinline__ Vec() : a(make_float4(0.f, 0.f, 0.f, 0.f)), b(a) {}
  static __device__ __forceinline__ Vec ones() {
    Vec v;
    v.a = v.b = make_float4(1.f, 1.f, 1.f, 1.f);
    return v;
  }
  __device__ __forceinline__ void load(const float* p) {
    a = *reinterpret_cast<const float4*>(p);
    b = *(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  }
  __device__ __forceinline__ void put(float* p) const {
    reinterpret_cast<float4*>(p)[0] = a;
    reinterpret_cast<float4*>(p)[1] = b;
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
  unsigned long long ph[2];  // phases of pairs 2 lane, 2 lane + 1
  float cs[8], sn[8];
  int mate;     // lane that holds the partner columns
  int from;     // lane that computed this lane's first pair
  bool on;      // this lane's columns are rotated
  bool minus;   // its columns are the `a` of their pairs (half layout)

  __device__ __forceinline__ void place(const RopeArgs& a, int lane) {
    const int s = lane % LPR, half = a.rot / 16;
    on = s < a.rot / 8;
    minus = s < half;
    mate = !on ? lane : (minus ? lane + half : lane - half);
    from = !on ? lane : (INTER ? 2 * s : 4 * (minus ? s : s - half));
#pragma unroll
    for (int j = 0; j < 2; ++j) ph[j] = 2 * lane + j < a.rot / 2 ? a.phases[2 * lane + j] : 0;
  }
  // cos and sin at a position: each lane computes two of the (up to 64)
  // pairs and the lanes exchange them, since every row of the warp and both
  // halves of a row need the same ones.
  __device__ __forceinline__ void angles(const RopeArgs& a, long long pos) {
    float c[2], s[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const unsigned long long turn = static_cast<unsigned long long>(pos) * ph[j];
      // The argument is the turn's top 24 bits, which fp32 holds exactly; the
      // next 24 turn the result on by an angle below 4e-7, to first order.
      float s0, c0;
      sincospif(static_cast<float>(static_cast<int>(turn >> 32) >> 8) * 0x1p-23f, &s0, &c0);
      const float rest = static_cast<float>(static_cast<unsigned>(turn >> 16) & 0xffffffu) * kRest;
      s[j] = fmaf(c0, rest, s0) * a.mscale;
      c[j] = fmaf(-s0, rest, c0) * a.mscale;
    }
    constexpr int N = INTER ? 4 : 8;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const float cv = __shfl_sync(kAll, c[j & 1], from + j / 2);
      const float sv = __shfl_sync(kAll, s[j & 1], from + j / 2);
      if (INTER) {
        cs[2 * j] = cs[2 * j + 1] = on ? cv : 1.f;
        sn[2 * j] = on ? -sv : 0.f;
        sn[2 * j + 1] = on ? sv : 0.f;
      } else {
        cs[j] = on ? cv : 1.f;
        sn[j] = on ? (minus ? -sv : sv) : 0.f;
      }
    }
  }
  // The partner's value of each column; 0 where nothing is rotated, so an
  // infinity there does not turn into a NaN with sn = 0.
  __device__ __forceinline__ void partner(const float (&x)[8], float (&p)[8]) const {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      p[e] = INTER ? x[e ^ 1] : __shfl_sync(kAll, x[e], mate);
      if (!on) p[e] = 0.f;
    }
  }
};

// The same for a row as loaded: bf16 travels packed, two columns a shuffle.
template <int D, bool INTER>
__device__ __forceinline__ void partner_row(const Rot<D, INTER>& rot, const Vec<__nv_bfloat16>& v,
                                            const float (&x)[8], float (&p)[8]) {
  if (INTER) {
    rot.partner(x, p);
    return;
  }
  Vec<__nv_bfloat16> m;
  m.w.x = __shfl_sync(kAll, v.w.x, rot.mate);
  m.w.y = __shfl_sync(kAll, v.w.y, rot.mate);
  m.w.z = __shfl_sync(kAll, v.w.z, rot.mate);
  m.w.w = __shfl_sync(kAll, v.w.w, rot.mate);
  if (!rot.on) m.w = make_uint4(0u, 0u, 0u, 0u);
  m.get(p);
}
template <int D, bool INTER>
__device__ __forceinline__ void partner_row(const Rot<D, INTER>& rot, const Vec<float>&,
                                            const float (&x)[8], float (&p)[8]) {
  rot.partner(x, p);
}

template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}

// Forward.  A warp takes a token, or a share of its rows (see share()); LPR
// lanes hold a row, so a group is 32 / LPR rows, of q or k alone, and the loads
// of kBatch groups are in flight together.  A row costs two products and a sum
// per column and one exchange of its packed columns with the partner lane.
// The 128K-token GQA q and k (32/8 heads, d = 128) take 442 us, 0.91 of the copy
// bandwidth; with the arithmetic one column at a time 469, with 2 or 4 CTAs per
// SM or other batches 450 to 585.  (The row is written out here: through turn()
// below the compiler's schedule costs 6%.)
constexpr int kBatch = 4;
template <typename T>
constexpr int kFwdCtas = sizeof(T) == 2 ? 3 : 2;  // per SM: 80 or 128 registers

template <typename T, int D, bool INTER>
__global__ void __launch_bounds__(kWarps * 32, kFwdCtas<T>) rope_forward_kernel(const RopeArgs a) {
  let_next_start();
  wait_for_previous();
  constexpr int LPR = D / 8, RPI = 32 / LPR;
  const int lane = threadIdx.x & 31, col = 8 * (lane % LPR), sub = lane / LPR;
  const int gq = (a.heads + RPI - 1) / RPI, gk = (a.kv_heads + RPI - 1) / RPI;
  const int groups = gq + gk;
  const int per = (groups + a.parts - 1) / a.parts;
  const long long items = a.whole + (a.T - a.whole) * a.parts;
  const long long nwarps = static_cast<long long>(gridDim.x) * kWarps;
  Rot<D, INTER> rot;
  rot.place(a, lane);
  for (long long it = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5); it < items;
       it += nwarps) {
    const bool cut = it >= a.whole;
    // (64-bit divisions: with 32-bit ones the compiler's schedule costs long calls 2.5%.)
    const long long t = cut ? a.whole + (it - a.whole) / a.parts : it;
    const int g0 = cut ? static_cast<int>(it - a.whole - (t - a.whole) * a.parts) * per : 0;
    const int g1 = cut && g0 + per < groups ? g0 + per : groups;
    // A last share may be empty.  (The test also keeps the compiler from moving
    // row loads above the angles, which costs 7%.)
    if (g0 < groups) rot.angles(a, row_position(a, t));
    auto rows = [&](int ga, int gb, int n, const T* src, T* dst, const void* weight) {
      // Groups [ga, gb) of a tensor's n rows of this token.
      uint64_t cw[4], sw[4];  // pairs of columns: the arithmetic is two-wide
      float w[8], wp[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = wp[e] = 1.f;
      if (weight) {
        load_weight(weight, a.w_bf16, col, w);
        rot.partner(w, wp);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        cw[e] = f2pack(rot.cs[2 * e] * w[2 * e], rot.cs[2 * e + 1] * w[2 * e + 1]);
        sw[e] = f2pack(rot.sn[2 * e] * wp[2 * e], rot.sn[2 * e + 1] * wp[2 * e + 1]);
      }
      src += sub * D + col;
      dst += sub * D + col;
      for (int g = ga; g < gb; g += kBatch) {
        Vec<T> raw[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
          raw[j] = Vec<T>();
          if (g + j < gb && (g + j) * RPI + sub < n) raw[j].load(src + (g + j) * RPI * D);
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
          if (g + j >= gb) break;
          const bool valid = (g + j) * RPI + sub < n;
          float x[8], p[8];
          raw[j].get(x);
          partner_row(rot, raw[j], x, p);
          uint64_t x2[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) x2[e] = f2pack(x[2 * e], x[2 * e + 1]);
          float r = 1.f;
          if (weight) {
            uint64_t s2 = fmul2(x2[0], x2[0]);
#pragma unroll
            for (int e = 1; e < 4; ++e) s2 = ffma2(x2[e], x2[e], s2);
            float sa, sb;
            f2unpack(s2, sa, sb);
            r = rsqrtf(row_sum<LPR>(sa + sb) * (1.f / D) + a.eps);
          }
          const uint64_t r2 = f2pack(r, r);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            f2unpack(fmul2(r2, ffma2(f2pack(p[2 * e], p[2 * e + 1]), sw[e], fmul2(x2[e], cw[e]))), x[2 * e],
                     x[2 * e + 1]);
          if (valid) Vec<T>::store(dst + (g + j) * RPI * D, x);
        }
      }
    };
    if (g0 < gq)
      rows(g0, g1 < gq ? g1 : gq, a.heads, static_cast<const T*>(a.q) + t * a.q_str,
           static_cast<T*>(a.qo) + t * a.qo_str, a.qw);
    if (g1 > gq)
      rows((g0 > gq ? g0 : gq) - gq, g1 - gq, a.kv_heads, static_cast<const T*>(a.k) + t * a.k_str,
           static_cast<T*>(a.ko) + t * a.ko_str, a.kw);
  }
}

// Norm weight and rotation of a token, folded: a row is out = r (x cw + partner
// sw) with cw = w cos and sw = w_partner sin, two columns at a time.
template <int D, bool INTER>
__device__ __forceinline__ void fold(const RopeArgs& a, const Rot<D, INTER>& rot, const void* weight, int col,
                                     uint64_t (&cw)[4], uint64_t (&sw)[4]) {
  float w[8], wp[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) w[e] = wp[e] = 1.f;
  if (weight) {
    load_weight(weight, a.w_bf16, col, w);
    rot.partner(w, wp);
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    cw[e] = f2pack(rot.cs[2 * e] * w[2 * e], rot.cs[2 * e + 1] * w[2 * e + 1]);
    sw[e] = f2pack(rot.sn[2 * e] * wp[2 * e], rot.sn[2 * e + 1] * wp[2 * e + 1]);
  }
}

// The rows of one group, normed and turned, to dst.
template <typename T, int D, bool INTER>
__device__ __forceinline__ void turn(const Rot<D, INTER>& rot, const Vec<T>& v, bool norm, float eps,
                                     const uint64_t (&cw)[4], const uint64_t (&sw)[4], bool valid, T* dst) {
  constexpr int LPR = D / 8;
  float x[8], p[8];
  v.get(x);
  partner_row(rot, v, x, p);
  uint64_t x2[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) x2[e] = f2pack(x[2 * e], x[2 * e + 1]);
  float r = 1.f;
  if (norm) {
    uint64_t s2 = fmul2(x2[0], x2[0]);
#pragma unroll
    for (int e = 1; e < 4; ++e) s2 = ffma2(x2[e], x2[e], s2);
    float sa, sb;
    f2unpack(s2, sa, sb);
    r = rsqrtf(row_sum<LPR>(sa + sb) * (1.f / D) + eps);
  }
  const uint64_t r2 = f2pack(r, r);
#pragma unroll
  for (int e = 0; e < 4; ++e)
    f2unpack(fmul2(r2, ffma2(f2pack(p[2 * e], p[2 * e + 1]), sw[e], fmul2(x2[e], cw[e]))), x[2 * e],
             x[2 * e + 1]);
  if (valid) Vec<T>::store(dst, x);
}

// Append: the same with k and v written to their pages.  Its calls are short,
// so a token's first loads, of q, k and v, go out before its angles are
// computed, its slot and position come with the token before, and k and v share
// a batch of loads.  17K tokens of 12/4 heads, d = 64, without norm, partly from
// L2: 20.0 us as the forward does it, 15.7 with q's loads and the slots early (80
// registers), 13.8 with the first group of k and v early too, at two CTAs per SM
// (in three that spills: 16.9); from HBM 17.8.  The forward done this way takes 0.5 us less of a call of
// 300 tokens and 1.2 times as long over 60K of 32/8 heads, d = 128.
constexpr int kAppendCtas = 2;  // per SM
template <int D, bool INTER>
__global__ void __launch_bounds__(kWarps * 32, kAppendCtas) rope_append_kernel(const RopeArgs a) {
  let_next_start();
  wait_for_previous();
  using T = __nv_bfloat16;
  constexpr int LPR = D / 8, RPI = 32 / LPR, N = kBatch / 2;
  const int lane = threadIdx.x & 31, col = 8 * (lane % LPR), sub = lane / LPR;
  const int gq = (a.heads + RPI - 1) / RPI, gk = (a.kv_heads + RPI - 1) / RPI;
  const int groups = gq + gk;  // v goes with k
  const int per = (groups + a.parts - 1) / a.parts;
  const long long items = a.whole + (a.T - a.whole) * a.parts;
  const long long nwarps = static_cast<long long>(gridDim.x) * kWarps;
  const int off = sub * D + col;
  Rot<D, INTER> rot;
  rot.place(a, lane);
  auto token = [&](long long it) {
    return it < a.whole ? it : a.whole + static_cast<unsigned>(it - a.whole) / static_cast<unsigned>(a.parts);
  };
  // Group g of n rows from src, if it is below gb.
  auto fetch = [&](Vec<T>& raw, const T* src, int g, int gb, int n) {
    raw = Vec<T>();
    if (g < gb && g * RPI + sub < n) raw.load(src + g * RPI * D + off);
  };
  uint64_t cw[4], sw[4];
  long long it = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (it >= items) return;
  long long t = token(it), pos = a.positions[t], slot = a.slots[t];
  for (;;) {
    const bool cut = it >= a.whole;
    const int g0 = cut ? (static_cast<int>(it - a.whole) - static_cast<int>(t - a.whole) * a.parts) * per : 0;
    const int g1 = cut && g0 + per < groups ? g0 + per : groups;
    const int q1 = g1 < gq ? g1 : gq;  // q groups [g0, q1), then k and v groups [k0, k1)
    const int k0 = g0 > gq ? g0 - gq : 0, k1 = g1 - gq;
    const bool real = slot >= 0 && slot < a.n_slots;  // else padding: nothing is written
    const T* const qsrc = static_cast<const T*>(a.q) + t * a.q_str;
    Vec<T> raw[kBatch];
    if (real && g0 < q1) {
#pragma unroll
      for (int j = 0; j < kBatch; ++j) fetch(raw[j], qsrc, g0 + j, q1, a.heads);
    }
    const T* const ksrc = static_cast<const T*>(a.k) + t * a.k_str;
    const T* const vsrc = static_cast<const T*>(a.v) + t * a.v_str;
    Vec<T> k_raw, v_raw;  // the first group's
    if (real && k0 < k1) {
      fetch(k_raw, ksrc, k0, k1, a.kv_heads);
      fetch(v_raw, vsrc, k0, k1, a.kv_heads);
    }
    long long pos2 = 0, slot2 = 0;
    if (it + nwarps < items) {
      const long long t2 = token(it + nwarps);
      pos2 = a.positions[t2];
      slot2 = a.slots[t2];
    }
    if (real) {
      rot.angles(a, pos);
      if (g0 < q1) {
        fold(a, rot, a.qw, col, cw, sw);
        T* const dst = static_cast<T*>(a.qo) + t * a.qo_str + off;
        for (int g = g0; g < q1; g += kBatch) {
          if (g > g0) {
#pragma unroll
            for (int j = 0; j < kBatch; ++j) fetch(raw[j], qsrc, g + j, q1, a.heads);
          }
#pragma unroll
          for (int j = 0; j < kBatch; ++j) {
            if (g + j >= q1) break;
            turn(rot, raw[j], a.qw != nullptr, a.eps, cw, sw, (g + j) * RPI + sub < a.heads,
                 dst + (g + j) * RPI * D);
          }
        }
      }
      if (k0 < k1) {
        fold(a, rot, a.kw, col, cw, sw);
        const long long page = slot >> a.page_shift;
        const long long in = (slot & ((1LL << a.page_shift) - 1)) * a.kv_heads * D + off;
        T* const kdst = static_cast<T*>(a.kc) + page * a.kc_page + in;
        T* const vdst = static_cast<T*>(a.vc) + page * a.vc_page + in;
        if (k0 * RPI + sub < a.kv_heads) v_raw.put(vdst + k0 * RPI * D);
        turn(rot, k_raw, a.kw != nullptr, a.eps, cw, sw, k0 * RPI + sub < a.kv_heads, kdst + k0 * RPI * D);
        for (int g = k0 + 1; g < k1; g += N) {
#pragma unroll
          for (int j = 0; j < N; ++j) {
            fetch(raw[j], ksrc, g + j, k1, a.kv_heads);
            fetch(raw[N + j], vsrc, g + j, k1, a.kv_heads);
          }
#pragma unroll
          for (int j = 0; j < N; ++j) {
            if (g + j >= k1) break;
            const bool valid = (g + j) * RPI + sub < a.kv_heads;
            turn(rot, raw[j], a.kw != nullptr, a.eps, cw, sw, valid, kdst + (g + j) * RPI * D);
            if (valid) raw[N + j].put(vdst + (g + j) * RPI * D);
          }
        }
      }
    }
    it += nwarps;
    if (it >= items) return;
    t = token(it);
    pos = pos2;
    slot = slot2;
  }
}

// A sum in two words: hi + lo takes x, and lo what that addition rounds off
// (Knuth's two-sum; six fp32 operations, where one in fp64 takes the time of
// 64).
__device__ __forceinline__ void add_to(float2& s, float x) {
  const float t = s.x + x, b = t - s.x;
  s.y += (s.x - (t - b)) + (x - b);
  s.x = t;
}
__device__ __forceinline__ void add_to(float2& s, const float2& x) {
  add_to(s, x.x);
  s.y += x.y;
}
// (An infinity stays one; its lo is NaN.)
__device__ __forceinline__ float value(const float2& s) { return isfinite(s.x) ? s.x + s.y : s.x; }

// Backward.  Groups as in the forward.  The weight gradients are summed in a
// fixed order: in the lanes over at most kRun rows (or a token's), then in two
// words, from run to run (shared memory), over the CTA's warps and over the CTAs
// (another launch).  In one word throughout, a lane added some 860 rows at 128K
// tokens, and the sums were 5.1e-7 off, 7 times the plain form's error, now
// 1.7e-7 (4099 tokens of 8/8 heads: 2.2e-7, now 0.9e-7); that took 864 us
// instead of 871, runs of 32 rows 873.  CUT: some tokens are taken in shares;
// without it that arithmetic stays out, whose registers cost a long call 3%
// (128K tokens of 32/8 heads, d = 128: 871 us, 0.92 of the copy bandwidth).
constexpr int kGradBatch = 3;
constexpr int kRun = 64;
constexpr int kGradCtas = 2;  // per SM

template <typename T, int D, bool INTER, bool CUT>
__global__ void __launch_bounds__(kWarps * 32, kGradCtas) rope_backward_kernel(const RopeArgs a) {
  let_next_start();
  wait_for_previous();
  constexpr int LPR = D / 8, RPI = 32 / LPR;
  __shared__ float2 s_dw[kWarps][16][32];  // [warp][q's eight columns, k's][lane]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = 8 * (lane % LPR), sub = lane / LPR;
  const int gq = (a.heads + RPI - 1) / RPI, gk = (a.kv_heads + RPI - 1) / RPI;
  const int groups = gq + gk, per = (groups + a.parts - 1) / a.parts;
  const unsigned items = static_cast<unsigned>(CUT ? a.whole + (a.T - a.whole) * a.parts : a.T);
  const unsigned nwarps = gridDim.x * kWarps;
  float wq[8], wk[8], dwq[8], dwk[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) wq[e] = wk[e] = dwq[e] = dwk[e] = 0.f;
  if (a.qw) load_weight(a.qw, a.w_bf16, col, wq);
  if (a.kw) load_weight(a.kw, a.w_bf16, col, wk);
  Rot<D, INTER> rot;
  rot.place(a, lane);
  // The runs' sums so far, and this one's added to them.
  auto keep = [&](bool first) {
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      float2 x = first ? make_float2(0.f, 0.f) : s_dw[warp][e][lane];
      add_to(x, e < 8 ? dwq[e] : dwk[e - 8]);
      s_dw[warp][e][lane] = x;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) dwq[e] = dwk[e] = 0.f;
  };
  const int turns = gq < kRun ? kRun / gq : 1;  // tokens of a run (k has no more groups than q)
  unsigned it = blockIdx.x * kWarps + warp;
  // (32-bit counters: with 64-bit ones 878 us instead of 871 below.)
  bool first = true;
  int left = turns;
  for (; it < items; it += nwarps) {
    const bool cut = CUT && it >= a.whole;
    const long long t = cut ? a.whole + (it - a.whole) / a.parts : it;
    const int g0 = cut ? static_cast<int>(it - a.whole - (t - a.whole) * a.parts) * per : 0;
    const int g1 = cut && g0 + per < groups ? g0 + per : groups;
    if (!CUT || g0 < groups) rot.angles(a, row_position(a, t));
    auto rows = [&](int ga, int gb, int n, const T* src, const float* grad, T* dst, bool norm,
                    const float (&w)[8], float (&dw)[8]) {
      src += sub * D + col;
      grad += sub * D + col;
      dst += sub * D + col;
      for (int g = CUT ? ga : 0; g < gb; g += kGradBatch) {
        // Rows of nobody are ones with no gradient: without eps, the norm of a row
        // of zeros would be infinite.
        Vec<T> raw[kGradBatch];
        Vec<float> gr[kGradBatch];
#pragma unroll
        for (int j = 0; j < kGradBatch; ++j) {
          raw[j] = Vec<T>::ones();
          gr[j] = Vec<float>();
          if (g + j < gb && (g + j) * RPI + sub < n) {
            raw[j].load(src + (g + j) * RPI * D);
            gr[j].load(grad + (g + j) * RPI * D);
          }
        }
#pragma unroll
        for (int j = 0; j < kGradBatch; ++j) {
          if (g + j >= gb) break;
          float x[8], gy[8], p[8];
          raw[j].get(x);
          gr[j].get(gy);
          rot.partner(gy, p);
#pragma unroll
          for (int e = 0; e < 8; ++e) gy[e] = fmaf(-p[e], rot.sn[e], gy[e] * rot.cs[e]);
          if (norm) {
            float ss = 0.f, ux = 0.f, u[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              u[e] = gy[e] * w[e];
              ss = fmaf(x[e], x[e], ss);
              ux = fmaf(u[e], x[e], ux);
            }
            ss = row_sum<LPR>(ss);
            ux = row_sum<LPR>(ux);
            const float r = rsqrtf(ss * (1.f / D) + a.eps);
            const float m = r * r * ux * (1.f / D);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              dw[e] = fmaf(gy[e], x[e] * r, dw[e]);
              gy[e] = r * fmaf(-x[e], m, u[e]);
            }
          }
          if ((g + j) * RPI + sub < n) Vec<T>::store(dst + (g + j) * RPI * D, gy);
        }
      }
    };
    rows(g0, CUT && g1 < gq ? g1 : gq, a.heads, static_cast<const T*>(a.q) + t * a.q_str, a.dqo + t * a.heads * D,
         static_cast<T*>(a.qo) + t * a.qo_str, a.qw != nullptr, wq, dwq);
    rows(g0 > gq ? g0 - gq : 0, CUT ? g1 - gq : gk, a.kv_heads, static_cast<const T*>(a.k) + t * a.k_str, a.dko + t * a.kv_heads * D,
         static_cast<T*>(a.ko) + t * a.ko_str, a.kw != nullptr, wk, dwk);
    if (--left == 0 && a.dw) {
      asm volatile("" ::: "memory");  // the sums' loads stay in here: their registers are the rows'
      keep(first);
      first = false;
      left = turns;
      asm volatile("" ::: "memory");
    }
  }
  if (!a.dw) return;
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    float2 x = first ? make_float2(0.f, 0.f) : s_dw[warp][e][lane];
    add_to(x, e < 8 ? dwq[e] : dwk[e - 8]);
#pragma unroll
    for (int o = LPR; o < 32; o <<= 1) {
      x.x += __shfl_xor_sync(kAll, x.x, o);
      x.y += __shfl_xor_sync(kAll, x.y, o);
    }
    if (sub == 0) s_dw[warp][e][lane] = x;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * D; i += kWarps * 32) {
    const int e = i / D * 8 + i % 8, l = i % D / 8;
    float2 x = s_dw[0][e][l];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) add_to(x, s_dw[w][e][l]);
    a.dw[static_cast<long long>(blockIdx.x) * 2 * D + i] = x;
  }
}

// One CTA per 32 of the 2 d weight gradients: warp w sums the partials w,
// w + 32, ... of its 32 columns, then the warps' sums of column w.
constexpr int kSumWarps = 32;
__global__ void __launch_bounds__(kSumWarps * 32) rope_weight_grad_kernel(const RopeArgs a, int n, int d) {
  let_next_start();
  wait_for_previous();
  __shared__ float2 s[kSumWarps][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float2 x = make_float2(0.f, 0.f);
  for (int p = warp; p < n; p += kSumWarps)
    add_to(x, a.dw[static_cast<long long>(p) * 2 * d + blockIdx.x * 32 + lane]);
  s[warp][lane] = x;
  __syncthreads();
  x = s[lane][warp];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    add_to(x, make_float2(__shfl_xor_sync(kAll, x.x, o), __shfl_xor_sync(kAll, x.y, o)));
  const int i = blockIdx.x * 32 + warp;
  float* dst = i < d ? a.dqw : a.dkw;
  if (lane == 0 && dst) dst[i % d] = value(x);
}

// Tokens are taken whole, one warp each, in turns of all warps of the grid; the
// rest of them, or all when there are few, by shares of their rows, a batch of
// loads each or more, so that the last turn is not a few warps' long one.  Whole
// and in shares, us, 32/8 heads, d = 128, from HBM: forward of 300 tokens 9.4 and
// 5.0, 2000 13.6 and 14.3, 4096 23.4 and 18.8, 8192 36.6 and 32.7, 20000 75.1 and
// 71.8; gradient of 300 16.6 and 11.0, 1000 21.0 and 16.5, 3000 37.7 and 31.8,
// 8192 70.9 and 70.0; append of 256 10.1 and 5.3, 1000 11.8 and 8.7, 8192 45.9 and
// 42.9.  A share computes the token's angles again, so the rest fills no more than
// one turn (forward of 6000 tokens, partly from L2: 26.0, with more 26.8), but for
// few tokens in the forward's three CTAs per SM, which come to some 16 warps per SM
// (2000 tokens so: 10.3; in one turn at most 11.6).  After more than eight turns
// the last is too small a part of the call to matter.
unsigned share(RopeArgs& a, int d, int ctas, int batch) {
  const int rpi = 256 / d, groups = (a.heads + rpi - 1) / rpi + (a.kv_heads + rpi - 1) / rpi;
  const long long warps = static_cast<long long>(ctas) * kWarps * sm_count();
  a.whole = a.T / warps * warps;
  const long long rest = a.T - a.whole, most = groups / batch;
  long long want = rest && a.whole <= 8 * warps ? warps / rest : 1;
  if (rest && !a.whole && ctas > 2) want = (16LL * sm_count() + rest - 1) / rest;
  if (want > most) want = most;
  a.parts = want < 1 ? 1 : static_cast<int>(want);
  if (a.parts == 1) a.whole = a.T;
  const long long items = a.whole + (a.T - a.whole) * a.parts, need = (items + kWarps - 1) / kWarps;
  return static_cast<unsigned>(need < warps / kWarps ? need : warps / kWarps);
}

template <typename T>
cudaError_t forward_t(RopeArgs a, int d, cudaStream_t st) {
  if (a.T == 0) return cudaSuccess;
  const unsigned grid = share(a, d, kFwdCtas<T>, kBatch);
  auto* kernel = d == 128 ? (a.interleaved ? rope_forward_kernel<T, 128, true> : rope_forward_kernel<T, 128, false>)
                         : (a.interleaved ? rope_forward_kernel<T, 64, true> : rope_forward_kernel<T, 64, false>);
  return launch_early(kernel, dim3(grid), kWarps * 32, 0, st, a);
}

template <typename T, bool CUT>
cudaError_t backward_t(const RopeArgs& a, int ctas, int d, cudaStream_t st) {
  auto* kernel = d == 128 ? (a.interleaved ? rope_backward_kernel<T, 128, true, CUT> : rope_backward_kernel<T, 128, false, CUT>)
                         : (a.interleaved ? rope_backward_kernel<T, 64, true, CUT> : rope_backward_kernel<T, 64, false, CUT>);
  return launch_early(kernel, dim3(static_cast<unsigned>(ctas)), kWarps * 32, 0, st, a);
}

}  // namespace

int rope_grad_ctas(RopeArgs& a, int d) { return static_cast<int>(share(a, d, kGradCtas, kGradBatch)); }

cudaError_t launch_rope_forward(const RopeArgs& a, int d, bool bf16, cudaStream_t st) {
  return bf16 ? forward_t<__nv_bfloat16>(a, d, st) : forward_t<float>(a, d, st);
}

cudaError_t launch_rope_append(const RopeArgs& args, int d, cudaStream_t st) {
  RopeArgs a = args;
  if (a.T == 0) return cudaSuccess;
  const unsigned grid = share(a, d, kAppendCtas, kBatch);
  auto* kernel = d == 128 ? (a.interleaved ? rope_append_kernel<128, true> : rope_append_kernel<128, false>)
                         : (a.interleaved ? rope_append_kernel<64, true> : rope_append_kernel<64, false>);
  return launch_early(kernel, dim3(grid), kWarps * 32, 0, st, a);
}

cudaError_t launch_rope_backward(const RopeArgs& a, int ctas, int d, bool bf16, cudaStream_t st) {
  if (a.parts == 1) return bf16 ? backward_t<__nv_bfloat16, false>(a, ctas, d, st) : backward_t<float, false>(a, ctas, d, st);
  return bf16 ? backward_t<__nv_bfloat16, true>(a, ctas, d, st) : backward_t<float, true>(a, ctas, d, st);
}

cudaError_t launch_rope_weight_grad(const RopeArgs& a, int n, int d, cudaStream_t st) {
  return launch_early(rope_weight_grad_kernel, dim3(2 * d / 32), kSumWarps * 32, 0, st, a, n, d);
}

}  // namespace ra
