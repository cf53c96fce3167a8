// What the two mma.sync decode kernels share (paged_kernel.cu, bf16 pages, and
// paged_fp8_kernel.cu, pages in 8 bits): the item records, the producer warps and
// the meeting of the consumer warps' states.  Device code only.
//
// A kernel's configuration C gives the KV heads of an item HEADS (their rows lie side
// by side in the tiles; a.kv_heads then counts their groups), the key tiles BT, the ring (NST stages of STAGE
// bytes: a K and a V tile of TILE bytes; where SCALES, BT scales of each in another),
// the tile's NCH chunks of CHB bytes with rows of CHROW, log2 of the rows of a
// box BOX, the row tile RT, the item ring (ITEMS) and the offsets in shared memory.
#pragma once
#include <cuda_bf16.h>

#include "paged_walk.cuh"

namespace ra {
namespace paged {

constexpr int kCons = 4;      // consumer warps
constexpr int kMmaThreads = 256;  // a consumer warpgroup and one with the producers
constexpr int kExtra = 1;     // what an item's beginning and end cost, in tiles

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
// `bytes` (a multiple of 16) from global to shared memory, both 16-byte aligned.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar)
      : "memory");
}

// A producer warp: K (which also walks the items ahead of everybody, leaves a
// record of each and copies its query rows) or V.
template <class C, int MODE>
__device__ __forceinline__ void produce(const PagedArgs& a, const void* tm, bool is_k, const Run& run, int g,
                                        uint8_t* smem, uint32_t sb, int lane, volatile int* abort_flag, int* status) {
  constexpr int BT = C::BT, RT = C::RT, D = C::DIM;
  const long long lim = a.wait_limit;
  const int sh = a.page_shift;
  const int rows = sh < C::BOX ? 1 << sh : 1 << C::BOX;  // of a box
  const int npg = BT / rows;
  const uint32_t box = static_cast<uint32_t>(rows) * C::CHROW;
  auto full = [&](int s) -> uint32_t { return sb + C::OFF_BAR + 8u * ((is_k ? 0 : C::NST) + s); };
  auto empty = [&](int s) -> uint32_t { return sb + C::OFF_BAR + 8u * (2 * C::NST + s); };
  auto ifull = [&](int s) -> uint32_t { return sb + C::OFF_BAR + 8u * (3 * C::NST + s); };
  auto iempty = [&](int s) -> uint32_t { return sb + C::OFF_BAR + 8u * (3 * C::NST + C::ITEMS + s); };
  const Joined joined(a);
  Walk<BT, kExtra, MODE> w;
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
    ids.start<MODE>(a, w.r, w.t.lo, w.t.hi, (w.t.t0 + w.k) * BT, lane);
    if (is_k) {
      const int s = it % C::ITEMS;
      if (it >= C::ITEMS) {
        ok = wait_bar(iempty(s), (static_cast<uint32_t>(it / C::ITEMS) & 1u) ^ 1u, abort_flag,
                      status, 0x84, lim);
        ok = __all_sync(kAll, ok);
        if (!ok) break;
      }
      const int n = w.t.rr1 - w.t.rr0, base = w.t.t0 * BT;
      int* rec = reinterpret_cast<int*>(smem + C::OFF_ITEM + s * C::REC);
      int row = 0;
      const int states = MODE == kBoth && w.q.group ? static_cast<int>(a.T) * a.heads : 0;  // behind those of own rows
      if (lane < RT) {  // rows past the item's get its last row's keys, and no output
        const int rr = w.t.rr0 + (lane < n ? lane : n - 1), j = token_of(rr, g);
        row = (w.q.row0 + j) * a.heads + w.kh * (C::HEADS * g) + (rr - j * g);
        rec[8 + lane] = row + states;
        rec[8 + RT + lane] = key_end<MODE>(w.q, j) - base;
      }
      if (MODE != kPlain || lane == 0) {
        const long long item0 = u - w.k;
        const int c0 = cta_of(item0, run), c1 = cta_of(item0 + w.t.nt - 1, run);
        const int me = static_cast<int>(blockIdx.x);
        if (MODE != kPlain && lane < n && me == c0)
          a.parts[row + states] = part_record(c0 == c1 ? -1 : (2 * me + 1) * RT + lane, c1 - c0 + 1 + (MODE == kOwn || MODE == kBoth ? joined.mark(w.r) : 0));
        if (lane == 0) {
          *reinterpret_cast<Item*>(rec) =
              Item{n, base, w.t.lo - base, w.t.hi - base, w.k, tiles, c0 == c1 ? -1 : 2 * me + (me == c0 ? 1 : 0), after >= run.last};
          if (MODE == kPlain && c0 != c1 && me == c0)
            static_cast<Cut*>(a.cuts)[me] = Cut{c1, w.q.row0, w.t.rr0, n, w.kh};
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(ifull(s));
      // Chunk c of row r at c ^ (r % 8): the ldmatrix rows of a column
      // block fall into different banks.
#pragma unroll
      for (int h = 0; h < C::HEADS; ++h)
#pragma unroll
        for (int x0 = 0; x0 < RT * D / 8; x0 += 32) {
          const int x = x0 + lane, r = x / (D / 8), c = x % (D / 8);
          const long long at = static_cast<long long>(__shfl_sync(kAll, row, r) + h * g) * D + c * 8;
          copy16(sb + C::OFF_Q + s * C::QT + (h * RT + r) * (D * 2) + ((c ^ (r & 7)) << 4),
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
                      status, 0x81, lim);
        ok = __all_sync(kAll, ok);
        if (!ok) break;
      }
      if (lane == 0) mbar_arrive_expect_tx(full(s), n * (box * C::NCH + (C::SCALES && is_k ? 2u * C::HEADS * rows : 0u)));
      __syncwarp();
      if (have) {
        const uint32_t dst = sb + s * C::STAGE + (is_k ? 0 : C::TILE) + lane * box;
        const int row = key0 & ((1 << sh) - 1);
#pragma unroll
        for (int ch = 0; ch < C::NCH; ++ch)
          tma_load_4d(dst + ch * C::CHB, tm, full(s), ch * 64, w.kh, row, page);
        if constexpr (C::SCALES) {
          if (is_k) {  // both tensors' scales come with the keys
#pragma unroll
            for (int h = 0; h < C::HEADS; ++h) {
              const uint32_t to = sb + C::OFF_SCALE + (s * 2 * C::HEADS + h) * BT + lane * rows;
              const long long at = (static_cast<long long>(w.kh * C::HEADS + h) << sh) + row;
              bulk_load(to, a.ks + page * a.ks_page + at, rows, full(s));
              bulk_load(to + C::HEADS * BT, a.vs + page * a.vs_page + at, rows, full(s));
            }
          }
        }
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
}

// The states (m, l, o) of the consumer warps, each over its own keys of the item,
// become one, and go to out and lse, or to partial states.  o[nt][x][c + 2 e] is
// row 8 nt + 2 (lane % 4) + c, column 16 x + 8 e + lane / 4, or, with PAIRS, column
// 16 x + 2 (lane / 4) + e.  head is added to the record's rows.  buf and buf2 hold two
// warps' messages each, 4 D floats.  False: the CTA gives up.
template <int D, int NT, bool PAIRS, int MODE>
__device__ __forceinline__ bool join_warps(const PagedArgs& a, const Item& item, const int* rec, int head, const float (&m)[NT][2],
                                           float (&l)[NT][2], float (&o)[NT][D / 16][4], bool ok, float* s_m, float* s_l,
                                           float* buf, float* buf2, int warp, int lane) {
  auto message = [&](int w) { return (w & 2 ? buf2 : buf) + (w & 1) * (4 * D); };
  constexpr int RT = 8 * NT;
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
  if (!named_bar_and(1, 32 * kCons, ok) || item.last == 2) return false;
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
      inv[c] = MODE != kPlain || item.slot >= 0 ? 1.f : (lt[c] == 0.f ? 0.f : 1.f / lt[c]);
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
    float* from = message(warp);
    float* to = message(warp ^ 1);
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
    const float* last = message(warp ^ 2);
#pragma unroll
    for (int x = 0; x < Q; ++x) {
      const float4 z = *reinterpret_cast<const float4*>(last + (x * 32 + lane) * 4);
      q[x][0] += z.x;
      q[x][1] += z.y;
      q[x][2] += z.z;
      q[x][3] += z.w;
    }
    const int d0 = (odd ? D / 2 : 0) + (high ? D / 4 : 0) + (PAIRS ? 2 : 1) * (lane >> 2);
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int r = 8 * nt + 2 * (lane & 3) + c;
      if (r >= item.rows) continue;
      const bool state = MODE != kPlain || item.slot >= 0;
      long long row = item.slot >= 0 ? item.slot * RT + r : rec[8 + r] + head;
      if (MODE != kPlain && item.slot < 0) row += a.whole;
#pragma unroll
      for (int x = 0; x < Q; ++x) {
        const long long at = row * D + d0 + 16 * x;
        const float y0 = q[x][c] * inv[c], y1 = q[x][c + 2] * inv[c];
        if constexpr (PAIRS) {
          if (state) *reinterpret_cast<float2*>(a.po + at) = make_float2(y0, y1);
          else if (a.out_bf16) *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(a.out) + at) = bf16x2_rn(y0, y1);
          else *reinterpret_cast<float2*>(static_cast<float*>(a.out) + at) = make_float2(y0, y1);
        } else {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float y = e ? y1 : y0;
            if (state) a.po[at + 8 * e] = y;
            else if (a.out_bf16) static_cast<__nv_bfloat16*>(a.out)[at + 8 * e] = __float2bfloat16_rn(y);
            else static_cast<float*>(a.out)[at + 8 * e] = y;
          }
        }
      }
      if (warp == 0 && lane < 4) {
        if (state) {
          a.pm[row] = mx[c];
          a.pl[row] = lt[c];
        } else {
          a.lse[row] = lt[c] == 0.f ? -INFINITY : mx[c] * kLn2 + logf(lt[c]);  // (NaN stays)
        }
      }
    }
  }
  return true;
}

}  // namespace paged
}  // namespace ra
