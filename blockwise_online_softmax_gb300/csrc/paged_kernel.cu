// Decode attention over paged keys and values: the newest tokens of many
// requests, each against its own pages (include/ra.h, ra_paged_decode).
//
// For a row (one head of one new token) with allowed keys t:
//   s_t = q.k_t / sqrt(d),  m = max s,  l = sum exp(s_t - m),
//   out = sum exp(s_t - m) v_t / l,  lse = m + ln l.
//
// The work is the read of the pages: each key meets only the rows of its KV
// head (g heads x the request's new tokens).  Its units are 64-key tiles, in
// the order (request, row tile, KV head, key tile), with one unit more for what
// an item (request, row tile, KV head) costs besides its tiles, and every CTA
// of a grid of two per SM takes an equal run of them, whatever the lengths are:
// the lengths stay on the device.  (Without that unit the CTA with the short
// requests ended last: 16 requests of up to 2K keys, 18.3 against 14.4 us, one set
// of pages over and over, so partly from L2; from HBM 16.1 now.)  A
// CTA finds its run by a prefix sum over the requests.  An item that falls into
// one CTA is finished there; one cut by a border between CTAs leaves a partial
// state (m, l, O~) on each side, and a second launch joins them in CTA order.
//
// Two warps feed a ring of stages with TMA, one K, one V (a page, or 64 rows
// of a larger one, is a box of one KV head; lane p looks up and requests page
// p of the tile).  The K warp also walks the items ahead of everybody, leaves
// a record of each in shared memory and copies its query rows there.  Four
// warps consume; each takes 16 keys of a tile and keeps its own running (m, l,
// O~), so nothing in the loop waits for another warp, and the states meet at
// the item's end.  Two such CTAs on an SM hide each other's item ends, which
// one CTA of twice the warps and tile did not (a 128-key item: 2.4 against 1.6
// us).  The products are mma.sync m16n8k16 with the keys, then the columns of
// V, as the 16-wide side and 8 query rows as the other: a tcgen05 tile would be
// 128 rows for the 4 or 8 there are, and its S -> P round trip through TMEM is
// the longer chain.
#include <atomic>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include <cuda_bf16.h>

#include "paged_mma.cuh"

namespace ra {

__device__ int g_paged_status = 0;

namespace {

using namespace paged;

constexpr int kThreads = kMmaThreads;

template <int D, int NT>
struct Cfg {
  static constexpr int DIM = D, BT = 64;         // keys per tile
  static constexpr int HEADS = 1;
  static constexpr int NCH = D / 64, BOX = 6;
  static constexpr uint32_t CHROW = 128, CHB = BT * CHROW;  // a 64-column chunk of a tile, 128-byte swizzle
  static constexpr bool SCALES = false;
  static constexpr int RT = 8 * NT;              // query rows of an item
  // Registers of the two warpgroups; together the launch's 2 x 128.  (200 and
  // 56 spill in the producers: 152 requests of 128 keys, from L2, 19.3 against 18.5 us.)
  static constexpr int CONS_REGS = NT == 1 ? 152 : 192, PROD_REGS = 256 - CONS_REGS;
  static constexpr int ITEMS = NT == 1 ? 3 : 2;  // records and query tiles in flight
  static constexpr uint32_t TILE = BT * D * 2, STAGE = 2 * TILE;
  static constexpr int NST = D == 128 ? 3 : 6;   // stages of one K and one V tile
  static constexpr uint32_t QT = RT * D * 2;     // query rows, 16-byte chunks swizzled
  static constexpr uint32_t REC = 32 + 8 * RT;   // Item, then rows and ends of its query rows
  static constexpr uint32_t OFF_Q = NST * 2 * TILE;
  static constexpr uint32_t OFF_BUF = OFF_Q + ITEMS * QT;        // [kCons][8][D / 2] fp32
  static constexpr uint32_t OFF_ML = OFF_BUF + kCons * 4 * D * 4;  // [2][RT][kCons] fp32
  static constexpr uint32_t OFF_ITEM = OFF_ML + 2 * kCons * RT * 4;
  static constexpr uint32_t OFF_BAR = OFF_ITEM + ITEMS * REC;
  static constexpr uint32_t OFF_MISC = OFF_BAR + (3 * NST + 2 * ITEMS) * 8;
  static constexpr uint32_t SMEM = OFF_MISC + 16;
  static_assert(SMEM <= 115712, "two CTAs per SM");
};

// ------------------------------------------------------------------ the kernel
// NT: 8-row groups of query rows of an item.
template <int D, int NT, int MODE>
__global__ void __launch_bounds__(kThreads, 2)
paged_decode_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                    const PagedArgs a) {
  using C = Cfg<D, NT>;
  constexpr int RT = C::RT, BT = C::BT;
  constexpr uint32_t CHB = C::CHB;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sb = smem_u32(smem);
  auto kfull = [&](int s) -> uint32_t { return sb + C::OFF_BAR + 8u * s; };
  auto vfull = [&](int s) -> uint32_t { return sb + C::OFF_BAR + 8u * (C::NST + s); };
  auto empty = [&](int s) -> uint32_t { return sb + C::OFF_BAR + 8u * (2 * C::NST + s); };
  auto ifull = [&](int s) -> uint32_t { return sb + C::OFF_BAR + 8u * (3 * C::NST + s); };
  auto iempty = [&](int s) -> uint32_t { return sb + C::OFF_BAR + 8u * (3 * C::NST + C::ITEMS + s); };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = a.heads / a.kv_heads;
  start_early<MODE>();
  if (tid == 0) {
    for (int s = 0; s < C::NST; ++s) {
      mbar_init(kfull(s), 1);
      mbar_init(vfull(s), 1);
      mbar_init(empty(s), kCons);
    }
    for (int s = 0; s < C::ITEMS; ++s) {
      mbar_init(ifull(s), 33);  // every lane's copies, and the record
      mbar_init(iempty(s), kCons);
    }
    int abort = *reinterpret_cast<volatile int*>(&g_paged_status);
    // The swizzled tiles need 1024-byte alignment, which the declaration asks
    // for; a loader that ignored it would be reported, not computed with.
    if (sb & 1023u) abort = atomicCAS(&g_paged_status, 0, 0x8f) | 0x8f;
    *abort_flag = abort;
    fence_mbar_init();
  }
  start_wait<MODE>();
  if (MODE == kPlain && tid == 0) static_cast<Cut*>(a.cuts)[blockIdx.x].last = -1;
  const Run run = find_run<BT, kExtra, MODE, kThreads>(a, g, RT, smem + C::OFF_BUF, abort_flag);  // synchronizes
  if (run.first >= run.last || run.stop) return end_wait<MODE>();
  const long long lim = a.wait_limit;

  if (warp >= kCons) {
    // ---------------------------------------------------------------- producers
    regs_dec<C::PROD_REGS>();
    if (warp >= kCons + 2) return end_wait<MODE>();
    const bool is_k = warp == kCons;
    produce<C, MODE>(a, is_k ? static_cast<const void*>(&tmK) : static_cast<const void*>(&tmV), is_k, run, g, smem, sb, lane,
                     abort_flag, &g_paged_status);
    return end_wait<MODE>();
  }

  // ------------------------------------------------------------------ consumers
  regs_inc<C::CONS_REGS>();
  // After a wait that gave up, a warp runs on without waiting (the status
  // word says that the results are void) to the item's first barrier, where
  // all of them learn of it and leave together.  Every warp waits for every
  // tile: a wait names its phase by parity alone, so no warp may be a whole
  // turn of the ring away from another.
  float* buf = reinterpret_cast<float*>(smem + C::OFF_BUF);
  float* s_m = reinterpret_cast<float*>(smem + C::OFF_ML);  // [row][warp]
  float* s_l = s_m + kCons * RT;
  const float sl2 = a.scale_log2;
  const int win = static_cast<int>(a.window);
  bool ok = true;
  int st = 0;                // stage and phase of the next tile
  uint32_t par = 0;
  // ldmatrix addresses inside a 64-column chunk of a tile: K rows are keys
  // (8 x 8 blocks: keys 0-7 / 8-15 first, then columns), V the same blocks
  // with columns first, read transposed.
  const int kr = warp * 16 + (lane & 15), kc0 = lane >> 4;
  const int vr = warp * 16 + (lane & 7) + ((lane >> 4) << 3), vc0 = (lane >> 3) & 1;
  for (int it = 0;; ++it) {
    const int is = it % C::ITEMS;
    ok = ok && wait_bar(ifull(is), static_cast<uint32_t>(it / C::ITEMS) & 1u, abort_flag,
                        &g_paged_status, 0x85, lim);
    ok = __all_sync(kAll, ok);
    const int* rec = reinterpret_cast<const int*>(smem + C::OFF_ITEM + is * C::REC);
    Item item = *reinterpret_cast<const Item*>(rec);
    if (!ok || item.last == 2) item.tiles = 0;
    // Keys [lo, hi) of the lane's rows 8 nt + 2 (lane & 3) + {0, 1}; the keys
    // that every row of the item sees are [lo_all, hi_all).
    auto begin_of = [&](int end) {
      return win > 0 && end + item.base > win ? end - win : -item.base;
    };
    int rlo[NT][2], rhi[NT][2];
    const int hi_all = rec[8 + RT], lo_all = begin_of(rec[8 + 2 * RT - 1]);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        rhi[nt][c] = rec[8 + RT + 8 * nt + 2 * (lane & 3) + c];
        rlo[nt][c] = begin_of(rhi[nt][c]);
      }
    float m[NT][2], l[NT][2], o[NT][D / 16][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt][0] = m[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
      for (int x = 0; x < D / 16; ++x) o[nt][x][0] = o[nt][x][1] = o[nt][x][2] = o[nt][x][3] = 0.f;
    }
    // Query rows as the B side: one ldmatrix gives two 16-column steps.
    const uint32_t qb = sb + C::OFF_Q + is * C::QT + (lane & 7) * (D * 2);
    const int qc0 = lane >> 3, qx = lane & 7;
    for (int k = 0; k < item.tiles; ++k) {
      const uint32_t kb = sb + st * 2 * C::TILE, vb = kb + C::TILE;
      const int k0 = (item.k0 + k) * BT + warp * 16;  // the warp's first key
      ok = ok && wait_bar(kfull(st), par, abort_flag, &g_paged_status, 0x82, lim) &&
           wait_bar(vfull(st), par, abort_flag, &g_paged_status, 0x83, lim);
      ok = __all_sync(kAll, ok);  // (both waits ahead of the work: 1M keys 800 -> 794 us)
      const bool some = k0 < item.hi && k0 + 16 > item.lo;
      if (some) {
        float sc[NT][4];
        uint32_t pb[NT][3][2];
        float al[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) sc[nt][0] = sc[nt][1] = sc[nt][2] = sc[nt][3] = 0.f;
#pragma unroll
        for (int k2 = 0; k2 < D / 32; ++k2) {
          uint32_t bq[NT][4];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            ldsm4(qb + nt * 8 * (D * 2) + (((4 * k2 + qc0) ^ qx) << 4), bq[nt]);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int kk = 2 * k2 + h, ch = (2 * kk + kc0) & 7;
            uint32_t af[4];
            ldsm4(kb + (kk >> 2) * CHB + kr * 128 + ((ch ^ (kr & 7)) << 4), af);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma16816(sc[nt], af, bq[nt][2 * h], bq[nt][2 * h + 1]);
          }
        }
        if (k0 < lo_all || k0 + 16 > hi_all) {
          const int k1 = k0 + (lane >> 2);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const int key = k1 + (c >> 1) * 8;
              if (key < rlo[nt][c & 1] || key >= rhi[nt][c & 1]) sc[nt][c] = -INFINITY;
            }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float x = fmaxf(sc[nt][c], sc[nt][c + 2]);
            x = fmaxf(x, __shfl_xor_sync(kAll, x, 4));
            x = fmaxf(x, __shfl_xor_sync(kAll, x, 8));
            x = fmaxf(x, __shfl_xor_sync(kAll, x, 16));
            const float mn = fmaxf(m[nt][c], x * sl2);
            const float ref = mn == -INFINITY ? 0.f : mn;
            al[nt][c] = ex2(m[nt][c] - ref);
            m[nt][c] = mn;
            const float p0 = ex2(fmaf(sc[nt][c], sl2, -ref)), p1 = ex2(fmaf(sc[nt][c + 2], sl2, -ref));
            l[nt][c] = fmaf(l[nt][c], al[nt][c], p0 + p1);
            sc[nt][c] = p0;
            sc[nt][c + 2] = p1;
          }
        // P as three bf16 terms (8 + 8 + 8 bits): the product with V then has
        // the weights' fp32 value, which an fp32 output shows; one bf16 term
        // is off by 2^-9 of each weight.
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            float x = sc[nt][2 * half], y = sc[nt][2 * half + 1];
#pragma unroll
            for (int term = 0; term < 3; ++term) {
              const uint32_t h = bf16x2_rn(x, y);
              pb[nt][term][half] = transpose8x8(h);
              x -= __uint_as_float(h << 16);
              y -= __uint_as_float(h & 0xffff0000u);
            }
          }
        const bool edge = k0 < item.lo || k0 + 16 > item.hi;
        uint32_t keep[2] = {kAll, kAll};  // V rows outside [lo, hi) may hold anything
        if (edge) {
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const int key = k0 + 8 * half + 2 * (lane & 3);
            keep[half] = (key >= item.lo && key < item.hi ? 0xffffu : 0u) |
                         (key + 1 >= item.lo && key + 1 < item.hi ? 0xffff0000u : 0u);
          }
        }
#pragma unroll
        for (int dm = 0; dm < D / 16; ++dm) {
          uint32_t af[4];
          const int ch = (2 * dm + vc0) & 7;
          ldsm4_t(vb + (dm >> 2) * CHB + vr * 128 + ((ch ^ (vr & 7)) << 4), af);
          if (edge) {
            af[0] &= keep[0];
            af[1] &= keep[0];
            af[2] &= keep[1];
            af[3] &= keep[1];
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            // The tile's product apart, small terms first, then one rounded
            // fp32 step: the tensor core's own accumulation truncates.
            float t[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int term = 2; term >= 0; --term) mma16816(t, af, pb[nt][term][0], pb[nt][term][1]);
#pragma unroll
            for (int c = 0; c < 4; ++c) o[nt][dm][c] = fmaf(o[nt][dm][c], al[nt][c & 1], t[c]);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(empty(st));
      if (++st == C::NST) {
        st = 0;
        par ^= 1u;
      }
    }
    if (!join_warps<D, NT, false, MODE>(a, item, rec, 0, m, l, o, ok, s_m, s_l, buf, buf + 2 * (4 * D), warp, lane)) break;
    if (item.last) break;
    __syncwarp();
    if (lane == 0) mbar_arrive(iempty(is));
  }
  end_wait<MODE>();
}

// Joins the partial states of the item that CTA c = blockIdx.x began and
// others went on with: slots 2c + 1, 2(c + 1), 2(c + 2), ...; a CTA takes every
// gridDim.y-th of its rows.  Its warps take every fourth partial, each with a
// running maximum of its own, and meet in shared memory.  A short launch's time
// is its chain of loads, so a warp's first partial is requested together with
// the record that says whether there is one (16 requests of up to 2K keys partly in
// L2, both launches: 13.3 us; 14.1 with the record, the maxima and the partials in
// turn; from HBM 16.1).
constexpr int kJoin = 4;
template <int D, bool TWO>
__global__ void __launch_bounds__(32 * kJoin) paged_combine_kernel(const PagedArgs a, int RT) {
  constexpr int CPL = D / 32;
  struct Part {
    float m, l, o[CPL];
  };
  __shared__ float s_m[kJoin], s_l[kJoin], s_o[kJoin][D];
  const int c = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto load = [&](int p, int r) {
    const long long at = static_cast<long long>(p == 0 ? 2 * c + 1 : 2 * (c + p)) * RT + r;
    Part x;
    x.m = a.pm[at];
    x.l = a.pl[at];
    const float* o = a.po + at * D + CPL * lane;
    if constexpr (CPL == 4) {
      const float4 v = *reinterpret_cast<const float4*>(o);
      x.o[0] = v.x, x.o[1] = v.y, x.o[2] = v.z, x.o[3] = v.w;
    } else {
      const float2 v = *reinterpret_cast<const float2*>(o);
      x.o[0] = v.x, x.o[1] = v.y;
    }
    return x;
  };
  let_next_start();
  wait_for_previous();
  const Cut cut = static_cast<const Cut*>(a.cuts)[c];
  // Row h tile + r of a slot is row r of the item's head h (of one, or of two).
  const int tile = TWO ? RT >> 1 : RT, turn = static_cast<int>(TWO ? gridDim.y >> 1 : gridDim.y);
  const int h = TWO && static_cast<int>(blockIdx.y) >= turn ? 1 : 0, r0 = static_cast<int>(blockIdx.y) - h * turn;
  // Of the CTA's first row, and of the two partials that most cut items have;
  // whatever the scratch holds when the item has no such partial.
  Part x{};
  const bool early = warp < 2 && c + warp < static_cast<int>(gridDim.x);
  if (early) x = load(warp, h * tile + r0);
  if (cut.last < 0) return;
  const int np = cut.last - c + 1, g = a.heads / (TWO ? 2 * a.kv_heads : a.kv_heads);
  for (int r = r0; r < cut.rows; r += turn) {
    float m = -INFINITY, l = 0.f, acc[CPL] = {};
    for (int p = warp; p < np; p += kJoin) {
      if (!early || p != warp || r != r0) x = load(p, h * tile + r);
      const float mn = fmaxf(m, x.m), ref = mn == -INFINITY ? 0.f : mn;
      const float e0 = ex2(m - ref), e1 = ex2(x.m - ref);
      m = mn;
      l = fmaf(x.l, e1, l * e0);
#pragma unroll
      for (int i = 0; i < CPL; ++i) acc[i] = fmaf(x.o[i], e1, acc[i] * e0);
    }
#pragma unroll
    for (int i = 0; i < CPL; ++i) s_o[warp][CPL * lane + i] = acc[i];
    if (lane == 0) {
      s_m[warp] = m;
      s_l[warp] = l;
    }
    __syncthreads();
    float mx = s_m[0];
#pragma unroll
    for (int w = 1; w < kJoin; ++w) mx = fmaxf(mx, s_m[w]);
    const float ref = mx == -INFINITY ? 0.f : mx;
    float e[kJoin];
    l = 0.f;
#pragma unroll
    for (int w = 0; w < kJoin; ++w) {
      e[w] = ex2(s_m[w] - ref);
      l = fmaf(s_l[w], e[w], l);
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const int rr = cut.rr0 + r, j = rr / g;
    const long long row =
        static_cast<long long>(cut.row0 + j) * a.heads + (TWO ? 2 * cut.kh + h : cut.kh) * g + (rr - j * g);
    for (int i = threadIdx.x; i < D; i += 32 * kJoin) {
      float y = 0.f;
#pragma unroll
      for (int w = 0; w < kJoin; ++w) y = fmaf(s_o[w][i], e[w], y);
      if (a.out_bf16) static_cast<__nv_bfloat16*>(a.out)[row * D + i] = __float2bfloat16_rn(y * inv);
      else static_cast<float*>(a.out)[row * D + i] = y * inv;
    }
    if (threadIdx.x == 0) a.lse[row] = l == 0.f ? -INFINITY : mx * kLn2 + logf(l);
    __syncthreads();
  }
}

// Joins the states of a row over its own keys and over its prefix, WPR warps a row;
// warp w of them takes partials w, w + WPR, ..., own ones first.  Its lanes take a
// partial each for the maximum and the weights, so that all of them are requested
// at once; then a lane sums D / 32 columns over the partials, in the order of the
// CTAs.  A row mostly has one or two partials of each launch, and a warp is enough;
// with few rows and a long prefix it has some 20, and eight warps share them (8
// requests of 4 rows of 8 KV heads, a call in three launches: 4K keys 35.0 -> 24.0 us,
// 1K keys 23.6 -> 21.4).
constexpr int kRowWarps = 8;
template <int D, int WPR>
__global__ void __launch_bounds__(32 * kRowWarps)
paged_join_kernel(const PagedArgs own, const PagedArgs shared, int own_tile, int shared_tile) {
  constexpr int CPL = D / 32, kEarly = WPR == 1 ? 2 : 4, kRows = kRowWarps / WPR, kFew = WPR == 1 ? 2 : 0;
  __shared__ float s_m[kRowWarps], s_l[kRowWarps], s_o[WPR > 1 ? kRowWarps : 1][D];
  let_next_start();
  wait_for_previous();
  const int w0 = WPR == 1 ? 0 : threadIdx.x >> 5;  // the warp's first partial
  const int lane = threadIdx.x & 31;
  long long first = 0, end = own.T;
  if (own.cu_q) {
    first = own.cu_q[0] < 0 ? 0 : own.cu_q[0];
    if (own.cu_q[own.n_req] < end) end = own.cu_q[own.n_req];
  }
  first *= own.heads;
  end *= own.heads;
  // A row's partials of one launch: index of the first and how many.
  struct Parts {
    long long at;
    int n, step;
    __device__ __forceinline__ Parts(const PagedArgs& a, int2 rec, int tile, long long row, bool any) : step(2 * tile) {
      at = a.whole + row;
      n = any ? 1 : 0;
      if (any && rec.x >= 0) {
        // (Records of rows that arrays in disorder left to nobody must not lead outside.)
        at = rec.x;
        n = rec.y & (kWithPrefix - 1);
        const long long most = at < a.whole ? (a.whole - 1 - at) / step + 1 : 0;
        if (n > most) n = static_cast<int>(most);
      }
    }
    __device__ __forceinline__ long long index(int p) const {
      return p == 0 ? at : at + static_cast<long long>(p) * step - step / 2;
    }
  };
  struct Columns {
    float v[CPL];
    __device__ __forceinline__ void load(const float* p) {
      if constexpr (CPL == 4) {
        const float4 x = *reinterpret_cast<const float4*>(p);
        v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
      } else {
        const float2 x = *reinterpret_cast<const float2*>(p);
        v[0] = x.x, v[1] = x.y;
      }
    }
  };
  for (long long row = first + static_cast<long long>(blockIdx.x) * kRows + (WPR == 1 ? threadIdx.x >> 5 : 0); row < end;
       row += static_cast<long long>(gridDim.x) * kRows) {
    const int2 r0 = own.parts[row], r1 = shared.parts[row];
    const Parts a(own, r0, own_tile, row, true), b(shared, r1, shared_tile, row, r0.y & kWithPrefix);
    const int n = a.n + b.n;
    auto state = [&](int p) { return p < a.n ? own.po + a.index(p) * D : shared.po + b.index(p - a.n) * D; };
    float m = -INFINITY, l = 0.f, acc[CPL] = {};
    // Two, as mostly, are weighed by every lane, without an exchange (81K rows, d = 64: the
    // call 122 -> 114 us; four 1.02 times slower where items are cut often).
    if (n <= kFew) {
      Columns x[kFew + 1];
      float xm[kFew + 1], xl[kFew + 1];
#pragma unroll
      for (int p = 0; p < kFew; ++p) {
        xm[p] = -INFINITY;
        xl[p] = 0.f;
        if (p < n) {
          const long long at = p < a.n ? a.index(p) : b.index(p - a.n);
          xm[p] = (p < a.n ? own.pm : shared.pm)[at];
          xl[p] = (p < a.n ? own.pl : shared.pl)[at];
          x[p].load((p < a.n ? own.po : shared.po) + at * D + CPL * lane);
        }
        m = fmaxf(m, xm[p]);
      }
      const float ref = m == -INFINITY ? 0.f : m;
#pragma unroll
      for (int p = 0; p < kFew; ++p) {
        if (p >= n) break;
        const float w = ex2(xm[p] - ref);
        l = fmaf(xl[p], w, l);
#pragma unroll
        for (int i = 0; i < CPL; ++i) acc[i] = fmaf(x[p].v[i], w, acc[i]);
      }
    }
    for (int p0 = n <= kFew ? n : w0; p0 < n; p0 += 32 * WPR) {
      const int p = p0 + lane * WPR;
      const bool mine = p < n;
      const float* pm = p < a.n ? own.pm + a.index(p) : shared.pm + b.index(p - a.n);
      const float* pl = p < a.n ? own.pl + a.index(p) : shared.pl + b.index(p - a.n);
      Columns early[kEarly];
#pragma unroll
      for (int q = 0; q < kEarly; ++q)
        if (p0 + q * WPR < n) early[q].load(state(p0 + q * WPR) + CPL * lane);
      const float xm = mine ? *pm : -INFINITY, xl = mine ? *pl : 0.f;
      float mx = xm;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, o));
      const float mn = fmaxf(m, mx), ref = mn == -INFINITY ? 0.f : mn;
      const float old = ex2(m - ref), w = ex2(xm - ref);
      m = mn;
      float part = xl * w;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) part += __shfl_xor_sync(kAll, part, o);
      l = fmaf(l, old, part);
#pragma unroll
      for (int i = 0; i < CPL; ++i) acc[i] *= old;
      const int np = min(32, (n - p0 + WPR - 1) / WPR);
      auto add = [&](const Columns& x, int q) {
        const float e = __shfl_sync(kAll, w, q);
#pragma unroll
        for (int i = 0; i < CPL; ++i) acc[i] = fmaf(x.v[i], e, acc[i]);
      };
#pragma unroll
      for (int q = 0; q < kEarly; ++q)
        if (q < np) add(early[q], q);
#pragma unroll 4
      for (int q = kEarly; q < np; ++q) {
        Columns x;
        x.load(state(p0 + q * WPR) + CPL * lane);
        add(x, q);
      }
    }
    if constexpr (WPR > 1) {  // the warps' sums meet in the first
      if (lane == 0) {
        s_m[w0] = m;
        s_l[w0] = l;
      }
#pragma unroll
      for (int i = 0; i < CPL; ++i) s_o[w0][CPL * lane + i] = acc[i];
      __syncthreads();
      if (w0 == 0) {
        m = s_m[0];
#pragma unroll
        for (int w = 1; w < WPR; ++w) m = fmaxf(m, s_m[w]);
        const float ref = m == -INFINITY ? 0.f : m;
        l = 0.f;
#pragma unroll
        for (int i = 0; i < CPL; ++i) acc[i] = 0.f;
#pragma unroll
        for (int w = 0; w < WPR; ++w) {
          const float e = ex2(s_m[w] - ref);
          l = fmaf(s_l[w], e, l);
#pragma unroll
          for (int i = 0; i < CPL; ++i) acc[i] = fmaf(s_o[w][CPL * lane + i], e, acc[i]);
        }
      }
      __syncthreads();
      if (w0 != 0) continue;
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int i = 0; i < CPL; ++i) acc[i] *= inv;
    const long long at = row * D + CPL * lane;
    if (own.out_bf16) {
      auto* out = static_cast<__nv_bfloat16*>(own.out) + at;
      if constexpr (CPL == 4)
        *reinterpret_cast<uint2*>(out) = make_uint2(bf16x2_rn(acc[0], acc[1]), bf16x2_rn(acc[2], acc[3]));
      else
        *reinterpret_cast<uint32_t*>(out) = bf16x2_rn(acc[0], acc[1]);
    } else {
      float* out = static_cast<float*>(own.out) + at;
      if constexpr (CPL == 4) *reinterpret_cast<float4*>(out) = make_float4(acc[0], acc[1], acc[2], acc[3]);
      else *reinterpret_cast<float2*>(out) = make_float2(acc[0], acc[1]);
    }
    if (lane == 0) own.lse[row] = l == 0.f ? -INFINITY : m * kLn2 + logf(l);
  }
}

template <int D, int NT, int MODE>
cudaError_t decode_t(const PagedArgs& a, int ctas, const CUtensorMap& tk, const CUtensorMap& tv,
                     cudaStream_t st) {
  static std::atomic<unsigned long long> done{0};
  cudaError_t e = allow_smem(paged_decode_kernel<D, NT, MODE>, Cfg<D, NT>::SMEM, done);
  if (e != cudaSuccess) return e;
  return launch_early(paged_decode_kernel<D, NT, MODE>, dim3(static_cast<unsigned>(ctas)), kThreads, Cfg<D, NT>::SMEM, st, tk, tv,
                      a);
}

}  // namespace

// Rows per request and KV head: exact without cu_q; with it those that the
// caller expects, or T / n_req, which counts padding rows too.  It picks the
// kernel; any mix is computed right by each.  A request's rows past a tile read
// its pages again, and a 128-row tile takes its time for fewer rows.  16-row tiles
// against 128-row tiles, us, 8 KV heads, requests x keys, from HBM:
//   d = 128      20 rows    40 rows        d = 64    20 rows    40 rows
//   152 x 1K    189/140    303/144                  132/122    194/123
//   64 x 2K     172/116    252/120                  108/102    155/105
//   64 x 500   56.8/52.5  77.0/55.3                41.7/42.0  56.1/45.0
//   16 x 300   20.8/21.4  24.1/23.4                17.0/19.1  19.5/21.2
// (16 rows, d = 128: 113/139, d = 64: 74/121.)  At d = 64 up to 32 rows the border
// leaves some 7% to the large works, for 4 to 19% of those below 35 us.
int paged_row_tile(const PagedArgs& a, int d) {
  const long long rows = a.n_q * (a.heads / a.kv_heads);
  return rows <= 8 ? 8 : (rows <= (d == 64 ? 32 : 16) ? 16 : 128);
}

// A group's rows on 16-row tiles beside the own rows, in one launch, or on 128-row
// tiles in a launch of their own (paged_prefix_kernel.cu), which costs some 8 us more.
// From there the tiles decide: 16 rows take 1.4 us per 64 keys and CTA, and an item as
// much as 256 keys more; 128 rows 1.5 us per 128 keys, and 384.  Keys are those the
// prefix table has room for.  One launch and two, us, 8 KV heads, d = 128, 4 rows a
// request, own histories of up to 300 keys, groups x requests x keys of the prefix:
//   1 x 8 x 1000   13.3/20.9    1 x 16 x 4000   22.0/24.4    1 x 256 x 64    56.7/44.3
//   1 x 64 x 300   23.9/30.2    1 x 8 x 30000   46.2/42.3    1 x 128 x 900   47.9/40.2
//   10 x 32 x 100  48.8/44.8    20 x 8 x 1000   51.1/49.8    1 x 16 x 16000  49.0/33.6
// (With at most 16 rows one launch always: 300 x 2 x 300 98/111, 1 x 4 x 30000 33.5/39.4.)
bool paged_prefix_both(const PagedArgs& group) {
  const long long rows = group.n_q * (group.heads / group.kv_heads);
  const double keys = static_cast<double>(group.max_pages) * (1 << group.page_shift);
  const double heads = static_cast<double>(group.n_req) * group.kv_heads / sm_count();
  const double one = heads / 2 * ((rows + 15) / 16) * (keys / 64 + 4) * 1.4;
  const double two = 8 + heads * ((rows + 127) / 128) * (keys / 128 + 3) * 1.5;
  return rows <= 16 || one <= two;
}

size_t paged_cut_bytes(int ctas) { return sizeof(Cut) * static_cast<size_t>(ctas); }

cudaError_t launch_paged_decode(const PagedArgs& a, int mode, int d, int ctas, int row_tile,
                                const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t st) {
  // Groups alone are taken 128 rows at a time, groups and own rows in one launch 8 or 16.
  if (mode == kShared) return row_tile == 128 ? launch_paged_prefix(a, d, ctas, tk, tv, st) : cudaErrorInvalidValue;
  if (mode == kBoth && row_tile > 16) return cudaErrorInvalidValue;
  if (row_tile == 128) return launch_paged_tc(a, mode, d, ctas, tk, tv, st);
  auto run = [&](auto m) {
    constexpr int MODE = decltype(m)::value;
    if (d == 128)
      return row_tile == 8 ? decode_t<128, 1, MODE>(a, ctas, tk, tv, st) : decode_t<128, 2, MODE>(a, ctas, tk, tv, st);
    return row_tile == 8 ? decode_t<64, 1, MODE>(a, ctas, tk, tv, st) : decode_t<64, 2, MODE>(a, ctas, tk, tv, st);
  };
  return mode == kOwn ? run(std::integral_constant<int, kOwn>{})
                      : (mode == kBoth ? run(std::integral_constant<int, kBoth>{})
                                       : run(std::integral_constant<int, kPlain>{}));
}

cudaError_t launch_paged_join(const PagedArgs& own, const PagedArgs& shared, int d, int own_tile,
                              int shared_tile, cudaStream_t st) {
  const long long rows = own.T * own.heads, most = 8LL * sm_count();  // CTAs that are resident together
  const bool share = rows <= most;
  const long long need = share ? rows : (rows + kRowWarps - 1) / kRowWarps;
  const dim3 grid(static_cast<unsigned>(need < most ? need : most));
  auto* kernel = d == 128 ? (share ? paged_join_kernel<128, kRowWarps> : paged_join_kernel<128, 1>)
                          : (share ? paged_join_kernel<64, kRowWarps> : paged_join_kernel<64, 1>);
  return launch_early(kernel, grid, 32 * kRowWarps, 0, st, own, shared, own_tile, shared_tile);
}

cudaError_t launch_paged_combine(const PagedArgs& a, int d, int ctas, int row_tile, cudaStream_t st) {
  // A CTA per row; no more than an item can have, where that is known here.
  long long rows = row_tile < 16 ? row_tile : 16;
  const int g = a.heads / (a.kv_heads * a.item_heads);
  if (!a.cu_q && a.n_q * g < rows) rows = a.n_q * g;
  rows *= a.item_heads;
  const dim3 grid(static_cast<unsigned>(ctas), static_cast<unsigned>(rows));
  auto* kernel = d == 128 ? paged_combine_kernel<128, false>  // (pairs of heads: d = 64)
                          : (a.item_heads == 2 ? paged_combine_kernel<64, true> : paged_combine_kernel<64, false>);
  return launch_early(kernel, grid, 32 * kJoin, 0, st, a, row_tile * a.item_heads);
}

cudaError_t take_paged_status(int* code) {
  int zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(code, g_paged_status, sizeof(int));
  if (e != cudaSuccess) return e;
  return cudaMemcpyToSymbol(g_paged_status, &zero, sizeof(int));
}

}  // namespace ra
