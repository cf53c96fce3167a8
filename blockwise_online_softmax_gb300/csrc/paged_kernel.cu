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

#include <cuda_bf16.h>

#include "paged_walk.cuh"

namespace ra {

__device__ int g_paged_status = 0;

namespace {

using namespace paged;

constexpr int BT = 64;           // keys per tile
constexpr int kCons = 4;         // consumer warps
constexpr int kThreads = 256;    // a consumer warpgroup and one with the producers
constexpr int kExtra = 1;        // what an item's beginning and end cost, in tiles
constexpr uint32_t CHB = BT * 128;  // one 64-column chunk of a tile, 128-byte swizzle

template <int D, int NT>
struct Cfg {
  static constexpr int NCH = D / 64;
  static constexpr int RT = 8 * NT;              // query rows of an item
  // Registers of the two warpgroups; together the launch's 2 x 128.  (200 and
  // 56 spill in the producers: 152 requests of 128 keys, from L2, 19.3 against 18.5 us.)
  static constexpr int CONS_REGS = NT == 1 ? 152 : 192, PROD_REGS = 256 - CONS_REGS;
  static constexpr int ITEMS = NT == 1 ? 3 : 2;  // records and query tiles in flight
  static constexpr uint32_t TILE = BT * D * 2;
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

// An item, or the part of it that a CTA has, as its consumers need it.
// Positions are relative to the item's first key tile.  The record goes on
// with row[RT], each query row's index in out, and end[RT], the end of the
// keys that it sees.
struct Item {
  int rows;            // query rows
  int base;            // position of the item's first key tile
  int lo, hi;          // keys that any row sees
  int k0;              // first key tile here
  int tiles;           // key tiles here
  int slot;            // partial slot, or -1: the item is whole
  int last;            // the CTA's last item; 2: not even an item
};
static_assert(sizeof(Item) == 32, "record layout");

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// ------------------------------------------------------------------ the kernel
// NT: 8-row groups of query rows of an item.
template <int D, int NT>
__global__ void __launch_bounds__(kThreads, 2)
paged_decode_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                    const PagedArgs a) {
  using C = Cfg<D, NT>;
  constexpr int RT = C::RT;
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
  Cut* cuts = static_cast<Cut*>(a.cuts);
  let_next_start();
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
  wait_for_previous();
  if (tid == 0) cuts[blockIdx.x].last = -1;
  const Run run = find_run<BT, kExtra, kThreads>(a, g, RT, smem + C::OFF_BUF, abort_flag);  // synchronizes
  if (run.first >= run.last || run.stop) return;
  const long long lim = a.wait_limit;

  if (warp >= kCons) {
    // ---------------------------------------------------------------- producers
    regs_dec<C::PROD_REGS>();
    if (warp >= kCons + 2) return;
    const bool is_k = warp == kCons;
    const void* tm = is_k ? static_cast<const void*>(&tmK) : static_cast<const void*>(&tmV);
    const int sh = a.page_shift;
    const int rows = sh < 6 ? 1 << sh : BT;  // of a box
    const int npg = BT / rows;
    const uint32_t box = static_cast<uint32_t>(rows) * 128u;
    auto full = [&](int s) -> uint32_t { return is_k ? kfull(s) : vfull(s); };
    Walk<BT, kExtra> w;
    w.start(a, g, RT, run.r, run.x);
    long long u = run.first;
    if (w.k >= w.t.nt) {  // the run begins behind an item's last tile
      u += w.t.nt + kExtra - w.k;
      if (u < run.last) w.next(a, g, RT);
      else if (is_k && lane == 0) {
        reinterpret_cast<Item*>(smem + C::OFF_ITEM)->last = 2;
        mbar_arrive(ifull(0));
      }
      if (u >= run.last && is_k) copies_arrive(ifull(0));
    }
    bool ok = true;
    int i = 0;   // tiles requested
    int it = 0;  // items begun
    while (ok && u < run.last) {
      const long long left = run.last - u;
      const int tiles = left < w.t.nt - w.k ? static_cast<int>(left) : w.t.nt - w.k;
      const long long after = u + tiles + (w.k + tiles == w.t.nt ? kExtra : 0);
      PageIds ids;  // first: the record and the query rows hide its latency
      ids.start(a, w.r, w.t.lo, w.t.hi, (w.t.t0 + w.k) * BT, lane);
      if (is_k) {
        const int s = it % C::ITEMS;
        if (it >= C::ITEMS) {
          ok = wait_bar(iempty(s), (static_cast<uint32_t>(it / C::ITEMS) & 1u) ^ 1u, abort_flag,
                        &g_paged_status, 0x84, lim);
          ok = __all_sync(kAll, ok);
          if (!ok) break;
        }
        const int n = w.t.rr1 - w.t.rr0, base = w.t.t0 * BT;
        int* rec = reinterpret_cast<int*>(smem + C::OFF_ITEM + s * C::REC);
        int row = 0;
        if (lane < RT) {  // rows past the item's get its last row's keys, and no output
          const int rr = w.t.rr0 + (lane < n ? lane : n - 1), j = token_of(rr, g);
          row = (w.q.row0 + j) * a.heads + w.kh * g + (rr - j * g);
          rec[8 + lane] = row;
          rec[8 + RT + lane] = key_end(w.q, j) - base;
        }
        if (lane == 0) {
          const long long item0 = u - w.k;
          const int c0 = cta_of(item0, run), c1 = cta_of(item0 + w.t.nt - 1, run);
          const int me = static_cast<int>(blockIdx.x);
          *reinterpret_cast<Item*>(rec) =
              Item{n, base, w.t.lo - base, w.t.hi - base, w.k, tiles, c0 == c1 ? -1 : 2 * me + (me == c0 ? 1 : 0), after >= run.last};
          if (c0 != c1 && me == c0) cuts[me] = Cut{c1, w.q.row0, w.t.rr0, n, w.kh};
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(ifull(s));
        // Chunk c of row r at c ^ (r % 8): the ldmatrix rows of a column
        // block fall into different banks.
#pragma unroll
        for (int x0 = 0; x0 < RT * D / 8; x0 += 32) {
          const int x = x0 + lane, r = x / (D / 8), c = x % (D / 8);
          const long long at = static_cast<long long>(__shfl_sync(kAll, row, r)) * D + c * 8;
          copy16(sb + C::OFF_Q + s * C::QT + r * (D * 2) + ((c ^ (r & 7)) << 4),
                 static_cast<const __nv_bfloat16*>(a.q) + at, r < n ? 16u : 0u);
        }
        copies_arrive(ifull(s));
        ++it;
      }
      for (int k = 0; k < tiles; ++k, ++i) {
        const int key0 = (w.t.t0 + w.k + k) * BT;
        const int page = ids.get(a, key0, rows, npg, lane);
        const bool have = page >= 0;
        const uint32_t n = static_cast<uint32_t>(__popc(__ballot_sync(kAll, have)));
        const int s = i % C::NST;
        if (i >= C::NST) {
          ok = wait_bar(empty(s), (static_cast<uint32_t>(i / C::NST) & 1u) ^ 1u, abort_flag,
                        &g_paged_status, 0x81, lim);
          ok = __all_sync(kAll, ok);
          if (!ok) break;
        }
        if (lane == 0) mbar_arrive_expect_tx(full(s), n * box * C::NCH);
        __syncwarp();
        if (have) {
          const uint32_t dst = sb + s * 2 * C::TILE + (is_k ? 0 : C::TILE) + lane * box;
          const int row = key0 & ((1 << sh) - 1);
#pragma unroll
          for (int ch = 0; ch < C::NCH; ++ch)
            tma_load_4d(dst + ch * CHB, tm, full(s), ch * 64, w.kh, row, page);
        }
      }
      u = after;
      if (ok && u < run.last) w.next(a, g, RT);
    }
    if (!ok) {  // let the copies in flight land before the CTA leaves
      volatile int no_abort = 0;
      for (int j = i > C::NST ? i - C::NST : 0; j < i; ++j)
        wait_bar(full(j % C::NST), static_cast<uint32_t>(j / C::NST) & 1u, &no_abort, nullptr, 0, lim);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    return;
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
      ok = ok && wait_bar(kfull(st), par, abort_flag, &g_paged_status, 0x82, lim);
      ok = __all_sync(kAll, ok);
      const bool some = k0 < item.hi && k0 + 16 > item.lo;
      float sc[NT][4];
      uint32_t pb[NT][3][2];
      float al[NT][2];
      if (some) {
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
      }
      ok = ok && wait_bar(vfull(st), par, abort_flag, &g_paged_status, 0x83, lim);
      ok = __all_sync(kAll, ok);
      if (some) {
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
    // ---------------------------------------------------------------- the warps' states meet
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float x = l[nt][c];
        x += __shfl_xor_sync(kAll, x, 4);
        x += __shfl_xor_sync(kAll, x, 8);
        x += __shfl_xor_sync(kAll, x, 16);
        l[nt][c] = x;
        if (lane < 4) {
          s_m[(8 * nt + 2 * lane + c) * kCons + warp] = m[nt][c];
          s_l[(8 * nt + 2 * lane + c) * kCons + warp] = x;
        }
      }
    if (!named_bar_and(1, 32 * kCons, ok) || item.last == 2) return;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      constexpr int H = D / 32, Q = D / 64;  // 16-column groups of a half and of a quarter
      float inv[2], mx[2], lt[2];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int r = 8 * nt + 2 * (lane & 3) + c;
        const float4 vm = *reinterpret_cast<const float4*>(s_m + r * kCons);
        const float4 vl = *reinterpret_cast<const float4*>(s_l + r * kCons);
        mx[c] = fmaxf(fmaxf(vm.x, vm.y), fmaxf(vm.z, vm.w));
        const float ref = mx[c] == -INFINITY ? 0.f : mx[c];
        lt[c] = (vl.x * ex2(vm.x - ref) + vl.y * ex2(vm.y - ref)) +
                (vl.z * ex2(vm.z - ref) + vl.w * ex2(vm.w - ref));
        inv[c] = item.slot >= 0 ? 1.f : (lt[c] == 0.f ? 0.f : 1.f / lt[c]);
        const float e = ex2(m[nt][c] - ref);
#pragma unroll
        for (int dm = 0; dm < D / 16; ++dm) {
          o[nt][dm][c] *= e;
          o[nt][dm][c + 2] *= e;
        }
      }
      // Warps w and w ^ 1 swap halves of the columns and add, then w and
      // w ^ 2 quarters: warp w ends with columns [D / 4 * (2 (w & 1) + w / 2)
      // ..) of the sum.  A warp's second message goes where it read its first.
      const bool odd = warp & 1, high = warp & 2;
      float* from = buf + warp * (4 * D);
      float* to = buf + (warp ^ 1) * (4 * D);
      if (nt > 0) named_bar_sync(1, 32 * kCons);  // the messages of group nt - 1 are read
      float h[H][4];
#pragma unroll
      for (int x = 0; x < H; ++x) {
        float y[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          h[x][c] = odd ? o[nt][H + x][c] : o[nt][x][c];
          y[c] = odd ? o[nt][x][c] : o[nt][H + x][c];
        }
        *reinterpret_cast<float4*>(to + (x * 32 + lane) * 4) = make_float4(y[0], y[1], y[2], y[3]);
      }
      named_bar_sync(1, 32 * kCons);
#pragma unroll
      for (int x = 0; x < H; ++x) {
        const float4 z = *reinterpret_cast<const float4*>(from + (x * 32 + lane) * 4);
        h[x][0] += z.x;
        h[x][1] += z.y;
        h[x][2] += z.z;
        h[x][3] += z.w;
      }
      __syncwarp();
      float q[Q][4];
#pragma unroll
      for (int x = 0; x < Q; ++x) {
        float y[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          q[x][c] = high ? h[Q + x][c] : h[x][c];
          y[c] = high ? h[x][c] : h[Q + x][c];
        }
        *reinterpret_cast<float4*>(from + (x * 32 + lane) * 4) = make_float4(y[0], y[1], y[2], y[3]);
      }
      named_bar_sync(1, 32 * kCons);
      const float* last = buf + (warp ^ 2) * (4 * D);
#pragma unroll
      for (int x = 0; x < Q; ++x) {
        const float4 z = *reinterpret_cast<const float4*>(last + (x * 32 + lane) * 4);
        q[x][0] += z.x;
        q[x][1] += z.y;
        q[x][2] += z.z;
        q[x][3] += z.w;
      }
      const int d0 = (odd ? D / 2 : 0) + (high ? D / 4 : 0) + (lane >> 2);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int r = 8 * nt + 2 * (lane & 3) + c;
        if (r >= item.rows) continue;
        const long long row = item.slot >= 0 ? item.slot * RT + r : rec[8 + r];
#pragma unroll
        for (int x = 0; x < Q; ++x)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float y = q[x][c + 2 * e] * inv[c];
            const long long at = row * D + d0 + 16 * x + 8 * e;
            if (item.slot >= 0) a.po[at] = y;
            else if (a.out_bf16) static_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(y);
            else static_cast<float*>(a.out)[at] = y;
          }
        if (warp == 0 && lane < 4) {
          if (item.slot >= 0) {
            a.pm[row] = mx[c];
            a.pl[row] = lt[c];
          } else {
            a.lse[row] = lt[c] == 0.f ? -INFINITY : mx[c] * kLn2 + logf(lt[c]);  // (NaN stays)
          }
        }
      }
    }
    if (item.last) return;
    __syncwarp();
    if (lane == 0) mbar_arrive(iempty(is));
  }
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
template <int D>
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
  // Of the CTA's first row, and of the two partials that most cut items have;
  // whatever the scratch holds when the item has no such partial.
  Part x{};
  const bool early = warp < 2 && c + warp < static_cast<int>(gridDim.x);
  if (early) x = load(warp, blockIdx.y);
  if (cut.last < 0) return;
  const int np = cut.last - c + 1, g = a.heads / a.kv_heads;
  for (int r = blockIdx.y; r < cut.rows; r += gridDim.y) {
    float m = -INFINITY, l = 0.f, acc[CPL] = {};
    for (int p = warp; p < np; p += kJoin) {
      if (!early || p != warp || r != static_cast<int>(blockIdx.y)) x = load(p, r);
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
    const long long row = static_cast<long long>(cut.row0 + j) * a.heads + cut.kh * g + (rr - j * g);
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

template <int D, int NT>
cudaError_t decode_t(const PagedArgs& a, int ctas, const CUtensorMap& tk, const CUtensorMap& tv,
                     cudaStream_t st) {
  static std::atomic<unsigned long long> done{0};
  cudaError_t e = allow_smem(paged_decode_kernel<D, NT>, Cfg<D, NT>::SMEM, done);
  if (e != cudaSuccess) return e;
  return launch_early(paged_decode_kernel<D, NT>, dim3(static_cast<unsigned>(ctas)), kThreads, Cfg<D, NT>::SMEM, st, tk, tv,
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

size_t paged_cut_bytes(int ctas) { return sizeof(Cut) * static_cast<size_t>(ctas); }

cudaError_t launch_paged_decode(const PagedArgs& a, int d, int ctas, int row_tile,
                                const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t st) {
  if (row_tile == 128) return launch_paged_tc(a, d, ctas, tk, tv, st);
  if (d == 128)
    return row_tile == 8 ? decode_t<128, 1>(a, ctas, tk, tv, st) : decode_t<128, 2>(a, ctas, tk, tv, st);
  return row_tile == 8 ? decode_t<64, 1>(a, ctas, tk, tv, st) : decode_t<64, 2>(a, ctas, tk, tv, st);
}

cudaError_t launch_paged_combine(const PagedArgs& a, int d, int ctas, int row_tile, cudaStream_t st) {
  // A CTA per row; no more than an item can have, where that is known here.
  long long rows = row_tile < 16 ? row_tile : 16;
  if (!a.cu_q && a.n_q * (a.heads / a.kv_heads) < rows) rows = a.n_q * (a.heads / a.kv_heads);
  const dim3 grid(static_cast<unsigned>(ctas), static_cast<unsigned>(rows));
  return launch_early(d == 128 ? paged_combine_kernel<128> : paged_combine_kernel<64>, grid, 32 * kJoin, 0, st, a,
                      row_tile);
}

cudaError_t take_paged_status(int* code) {
  int zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(code, g_paged_status, sizeof(int));
  if (e != cudaSuccess) return e;
  return cudaMemcpyToSymbol(g_paged_status, &zero, sizeof(int));
}

}  // namespace ra
