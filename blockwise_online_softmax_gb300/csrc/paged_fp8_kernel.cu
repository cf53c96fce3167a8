// Decode attention over pages in 8 bits (include/ra.h, ra_paged_decode_fp8; the
// rows as fp8.cuh holds them).  Row, keys, work list, roles and joining launch
// are those of paged_kernel.cu; with key t held as codes kc_t and scale 2^a_t,
// value t as vc_t and 2^b_t:
//   s_t = 2^a_t (q.kc_t) / sqrt(d),  m = max s,  p_t = exp(s_t - m),
//   out = sum p_t 2^b_t vc_t / sum p_t.
//
// The pages' bytes are half of bf16's, so a tile's arithmetic has half the time.
// - Codes go to the tensor core as fp16 (cvt.rn.f16x2.e4m3x2, exact, one
//   instruction for two).  The conversion is in registers, so the order of the
//   reduced index is free: a lane's four neighbouring bytes of a key's row are
//   the two register halves of one m16n8k16 fragment, and the query's columns
//   are read in the same order.  For P V, ldmatrix transposes pairs of bytes, and
//   one byte permutation gives the pairs of keys of two neighbouring columns: of
//   the fragment's rows g and g + 8.
// - q is turned to fp16 once an item, with a power of two per row that brings its
//   largest entry to [2^14, 2^15): its 8 bits are exact down to 2^-28 of that entry,
//   and below it is off by at most 2^-39 of it.
// - The weight of a value is p_t 2^b_t.  fp16 has no room for all of them, so a row
//   scales its weights of a warp's 32 keys by a power of two, the largest to [2^14,
//   2^15), and gives it back in fp32 when the tile's product is added to O.  Held
//   in two fp16 terms (22 bits and the sign of the second) a weight is off by at
//   most 2^-23 of itself, or 2^-39 of the row's largest there.  Rows have powers of
//   their own: what one weighs, another may not see.  (One power for the warp, found by
//   one instruction, took 487 for 503 us at 1M keys and 155 for 162 at 1.2M, d = 64, 9
//   rows, and lost a row's weights beside another's of a far larger scale.  bf16 pages
//   need three terms of 8 bits.)
// - A consumer warp takes 32 keys of a tile, and O is scaled only under a new maximum
//   (with 16, scaled each time: 128 requests of up to 8K keys 156 against 128 us, 1M
//   keys 680 against 512).
//
// 32/8 heads, d = 128, one row: 128 requests of up to 8K keys 123 to 136 us with the
// machine, 5.4 to 5.9 TB/s (0.79 to 0.87 of the copy rate; rows of 128 bytes some
// distance apart); bound by HBM and the ends of items.  16 rows (1M and some keys, 4
// new tokens): 503 us, 5.4 TB/s (0.79); d = 64 with 9 rows (1.2M keys, 4 heads) 162 us,
// 3.8 TB/s, with 3 rows, two heads an item, 141 us, 4.4 TB/s.  These three are bound by
// the latency of a tile's chain (products, maximum, exponentials, weights' power,
// products) with two consumer warps a scheduler: of the issue slots 42, 46 and 40% are
// busy, of the tensor pipe 40, 31 and 18%, of DRAM 63, 48 and 58%.  16 requests of up to
// 2000 keys 13.5 us: two launches and their chains of loads.
#include <atomic>
#include <cmath>
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fp8.cuh"
#include "paged_mma.cuh"

namespace ra {

__device__ int g_paged_fp8_status = 0;

namespace {

using namespace paged;

constexpr int kThreads = kMmaThreads;
constexpr int KB = 2;  // blocks of 16 keys that a warp takes of a tile

// NT: 8-row groups of query rows, HP: KV heads of an item.
template <int D, int NT, int HP>
struct Cfg {
  static constexpr int DIM = D, BT = 16 * kCons * KB, HEADS = HP;
  static constexpr int NCH = 1, BOX = 7;
  static constexpr uint32_t CHROW = D * HP, CHB = BT * CHROW;  // rows of 128 or 64 bytes, swizzled over as many
  static constexpr bool SCALES = true;
  static constexpr int RT = 8 * NT;
  // (What leaves the consumers least in memory: with 152 and 192 they spill, and are
  // up to 2% slower.)
  static constexpr int CONS_REGS = NT == 1 ? 168 : (D == 64 ? 176 : 192), PROD_REGS = 256 - CONS_REGS;
  static constexpr int ITEMS = NT == 1 ? 3 : 2;
  static constexpr uint32_t TILE = CHB;
  static constexpr uint32_t STAGE = 2 * TILE;
  static constexpr uint32_t QT = HP * RT * D * 2;
  static constexpr uint32_t REC = 32 + 8 * RT;
  // The messages of warps 2 and 3 at an item's end take the place of its query rows,
  // which are in registers by then, where they fit (at d = 128 that is a third stage: 1M
  // keys, 16 rows 512 -> 488 us, with both waits of a tile ahead of it).
  static constexpr bool IN_Q = NT == 2;
  static constexpr uint32_t BUF = (IN_Q ? 2 : kCons) * 4 * D * 4;
  static_assert(!IN_Q || QT >= 2 * 4 * D * 4, "messages fit");
  static constexpr uint32_t REST = ITEMS * QT + BUF + 2 * kCons * RT * 4 + ITEMS * REC + 16;
  static constexpr int NST = (115712 - REST - 2 * ITEMS * 8) / (STAGE + 2 * HP * BT + 24);  // what two CTAs per SM leave
  static constexpr uint32_t OFF_SCALE = NST * STAGE;  // of stage s: K's by head, then V's
  static constexpr uint32_t OFF_Q = OFF_SCALE + NST * 2 * HP * BT;
  static constexpr uint32_t OFF_BUF = OFF_Q + ITEMS * QT;
  static constexpr uint32_t OFF_ML = OFF_BUF + BUF;
  static constexpr uint32_t OFF_ITEM = OFF_ML + 2 * kCons * RT * 4;
  static constexpr uint32_t OFF_BAR = OFF_ITEM + ITEMS * REC;
  static constexpr uint32_t OFF_MISC = OFF_BAR + (3 * NST + 2 * ITEMS) * 8;
  static constexpr uint32_t SMEM = OFF_MISC + 16;
  static_assert(SMEM <= 115712 && NST >= 2, "two CTAs per SM");
};

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The same with c = 0 before.
__device__ __forceinline__ void mma_f16_first(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%10, %10, %10, %10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ uint32_t f16x2_rn(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ float2 halves(uint32_t h) { return __half22float2(*reinterpret_cast<const __half2*>(&h)); }
__device__ __forceinline__ uint32_t low2(uint32_t x) { return halves2(static_cast<uint16_t>(x)); }
__device__ __forceinline__ uint32_t high2(uint32_t x) { return halves2(static_cast<uint16_t>(x >> 16)); }
__device__ __forceinline__ uint32_t lds_u8(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint2 lds_v2(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
  return v;
}

template <int D, int NT, int HP>
__global__ void __launch_bounds__(kThreads, 2)
paged_fp8_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const PagedArgs a) {
  using C = Cfg<D, NT, HP>;
  // AHEAD: the scores of a tile are multiplied while the softmax of the one before, a
  // long chain of dependent steps, is under way.  Without and with, us: 128 requests of
  // up to 8K keys 145 and 136, 600K keys 228 and 215 (16 requests of up to 2000 keys 13.3
  // and 13.6).  At d = 64 a tile's products are half as long: 60 requests of a 4K window,
  // 9 rows 34.3 and 36.0, 1.2M keys 163 and 166, 16 requests of up to 2000 keys 10.7 and
  // 11.4.  16 rows at d = 128 have few registers left for it: 64 requests of up to 4000
  // keys and 64 rows 199 and 218, 1M keys 504 and 500.
  constexpr bool AHEAD = D == 128 && NT == 1;
  static_assert(!AHEAD || HP == 1, "one head's scores ahead");
  constexpr int RT = C::RT, BT = C::BT, ROW = D * HP;  // bytes of a key's row
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sb = smem_u32(smem);
  auto kfull = [&](int s) -> uint32_t { return sb + C::OFF_BAR + 8u * s; };
  auto vfull = [&](int s) -> uint32_t { return sb + C::OFF_BAR + 8u * (C::NST + s); };
  auto empty = [&](int s) -> uint32_t { return sb + C::OFF_BAR + 8u * (2 * C::NST + s); };
  auto ifull = [&](int s) -> uint32_t { return sb + C::OFF_BAR + 8u * (3 * C::NST + s); };
  auto iempty = [&](int s) -> uint32_t { return sb + C::OFF_BAR + 8u * (3 * C::NST + C::ITEMS + s); };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = a.heads / (a.kv_heads * HP);
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
    int abort = *reinterpret_cast<volatile int*>(&g_paged_fp8_status);
    // The swizzled tiles need 1024-byte alignment, which the declaration asks
    // for; a loader that ignored it would be reported, not computed with.
    if (sb & 1023u) abort = atomicCAS(&g_paged_fp8_status, 0, 0xaf) | 0xaf;
    *abort_flag = abort;
    fence_mbar_init();
  }
  wait_for_previous();
  if (tid == 0) static_cast<Cut*>(a.cuts)[blockIdx.x].last = -1;
  const Run run = find_run<BT, kExtra, kPlain, kThreads>(a, g, RT, smem + C::OFF_BUF, abort_flag);  // synchronizes
  if (run.first >= run.last || run.stop) return;
  const long long lim = a.wait_limit;

  if (warp >= kCons) {
    // ---------------------------------------------------------------- producers
    regs_dec<C::PROD_REGS>();
    if (warp >= kCons + 2) return;
    const bool is_k = warp == kCons;
    produce<C, kPlain>(a, is_k ? static_cast<const void*>(&tmK) : static_cast<const void*>(&tmV), is_k, run, g, smem, sb, lane,
                       abort_flag, &g_paged_fp8_status);
    return;
  }

  // ------------------------------------------------------------------ consumers
  // (After a wait that gave up a warp runs on to the item's first barrier, as in
  // paged_kernel.cu.)
  regs_inc<C::CONS_REGS>();
  float* buf = reinterpret_cast<float*>(smem + C::OFF_BUF);
  float* s_m = reinterpret_cast<float*>(smem + C::OFF_ML);  // [row][warp]
  float* s_l = s_m + kCons * RT;
  const int win = static_cast<int>(a.window);
  bool ok = true;
  int st = 0;  // stage and phase of the next tile
  uint32_t par = 0;
  constexpr int CPR = D / 16;  // 16-byte chunks of a row
  // Of a row r: the swizzle over its chunks (128-byte rows over 8 rows, 64-byte
  // rows over pairs of 8).
  auto swz = [](int r) { return ROW == 128 ? r & 7 : (r >> 1) & 3; };
  const int key0 = warp * 16 * KB;  // of the tile
  const int kr = lane & 15, c2 = lane >> 4;  // ldmatrix: row of a block, chunk of a pair
  for (int it = 0;; ++it) {
    const int is = it % C::ITEMS;
    ok = ok && wait_bar(ifull(is), static_cast<uint32_t>(it / C::ITEMS) & 1u, abort_flag, &g_paged_fp8_status, 0xa5, lim);
    ok = __all_sync(kAll, ok);
    const int* rec = reinterpret_cast<const int*>(smem + C::OFF_ITEM + is * C::REC);
    Item item = *reinterpret_cast<const Item*>(rec);
    if (!ok || item.last == 2) item.tiles = 0;
    // Keys [lo, hi) of the lane's rows 8 nt + 2 (lane & 3) + {0, 1}; the keys
    // that every row of the item sees are [lo_all, hi_all).
    auto begin_of = [&](int end) { return win > 0 && end + item.base > win ? end - win : -item.base; };
    int rlo[NT][2], rhi[NT][2];
    const int hi_all = rec[8 + RT], lo_all = begin_of(rec[8 + 2 * RT - 1]);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        rhi[nt][c] = rec[8 + RT + 8 * nt + 2 * (lane & 3) + c];
        rlo[nt][c] = begin_of(rhi[nt][c]);
      }
    // The query rows in fp16: columns 16 c + 4 (lane % 4) + 0..3 of row lane / 4,
    // and the factor on the lane's two scores of a key.
    uint32_t qf[HP][NT][CPR][2];
    float sl2[HP][NT][2];
#pragma unroll
    for (int sn = 0; sn < HP * NT; ++sn) {
      const int s = sn / NT, nt = sn % NT;
      const int r = 8 * nt + (lane >> 2);
      unsigned top = 0;
#pragma unroll
      for (int c = 0; c < CPR; ++c) {
        const int ch = 2 * c + ((lane & 3) >> 1);
        const uint2 w = lds_v2(sb + C::OFF_Q + is * C::QT + (s * RT + r) * (D * 2) + ((ch ^ (r & 7)) << 4) + (lane & 1) * 8);
        qf[s][nt][c][0] = w.x;
        qf[s][nt][c][1] = w.y;
        top = max(top, max(max(w.x << 16 & 0x7fff0000u, w.x & 0x7fff0000u), max(w.y << 16 & 0x7fff0000u, w.y & 0x7fff0000u)));
      }
      top = max(top, __shfl_xor_sync(kAll, top, 1));
      top = max(top, __shfl_xor_sync(kAll, top, 2));
      int e = static_cast<int>(top >> 23);  // largest entry in [2^(e - 127), 2^(e - 126))
      e = e < 27 ? 27 : e;
      const float up = __uint_as_float(static_cast<unsigned>(268 - e) << 23);  // 2^(14 - (e - 127))
#pragma unroll
      for (int c = 0; c < CPR; ++c)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          qf[s][nt][c][h] = f16x2_rn(__uint_as_float(qf[s][nt][c][h] << 16) * up, __uint_as_float(qf[s][nt][c][h] & 0xffff0000u) * up);
      const float down = a.scale_log2 * __uint_as_float(static_cast<unsigned>(e - 14) << 23);
#pragma unroll
      for (int c = 0; c < 2; ++c) sl2[s][nt][c] = __shfl_sync(kAll, down, 8 * (lane & 3) + 4 * c);
    }
    float m[HP][NT][2], l[HP][NT][2];
    uint64_t o2[HP][NT][D / 16][2];  // rows 2 (lane % 4) + {0, 1} of a column
#pragma unroll
    for (int sn = 0; sn < HP * NT; ++sn) {
      const int s = sn / NT, nt = sn % NT;
      m[s][nt][0] = m[s][nt][1] = -INFINITY;
      l[s][nt][0] = l[s][nt][1] = 0.f;
#pragma unroll
      for (int x = 0; x < D / 16; ++x) o2[s][nt][x][0] = o2[s][nt][x][1] = f2pack(0.f, 0.f);
    }
    // Raw scores of the warp's keys of a tile.  Independent products alternate: each
    // waits for the one before it of the same sum.  With one group of rows a sum has
    // two halves.
    constexpr int HALVES = NT == 1 ? 2 : 1;
    float part[HALVES][KB][NT][4];
    auto products = [&](int stage, int s) {
      const uint32_t kb = sb + stage * C::STAGE;
#pragma unroll
      for (int c = 0; c < CPR; c += 2) {
        uint32_t w[KB][4];  // (keys 0-7, 8-15) of chunk c, then of chunk c + 1
#pragma unroll
        for (int b = 0; b < KB; ++b) {
          const int r = key0 + 16 * b + kr;
          ldsm4(kb + r * ROW + (((s * CPR + c + c2) ^ swz(r)) << 4), w[b]);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int b = 0; b < KB; ++b) {
            const uint32_t af[4] = {low2(w[b][2 * h]), low2(w[b][2 * h + 1]), high2(w[b][2 * h]), high2(w[b][2 * h + 1])};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              float(&t)[4] = part[h % HALVES][b][nt];
              if (c + h < HALVES) mma_f16_first(t, af, qf[s][nt][c + h][0], qf[s][nt][c + h][1]);
              else mma_f16(t, af, qf[s][nt][c + h][0], qf[s][nt][c + h][1]);
            }
          }
      }
    };
    if (AHEAD && item.tiles > 0) {
      ok = ok && wait_bar(kfull(st), par, abort_flag, &g_paged_fp8_status, 0xa2, lim);
      ok = __all_sync(kAll, ok);
      products(st, 0);
    }
    for (int k = 0; k < item.tiles; ++k) {
      const uint32_t vb = sb + st * C::STAGE + C::TILE, scales = sb + C::OFF_SCALE + st * 2 * HP * BT + key0;
      const int k0 = (item.k0 + k) * BT + key0;  // the warp's first key
      const bool some = AHEAD || (k0 < item.hi && k0 + 16 * KB > item.lo);
      const bool edge = k0 < item.lo || k0 + 16 * KB > item.hi;
      const bool more = k + 1 < item.tiles;
      const int then = st + 1 == C::NST ? 0 : st + 1;
      // Both waits ahead of the tile's work, which is then one block of straight code.
      ok = ok && (AHEAD || wait_bar(kfull(st), par, abort_flag, &g_paged_fp8_status, 0xa2, lim)) &&
           wait_bar(vfull(st), par, abort_flag, &g_paged_fp8_status, 0xa3, lim) &&
           (!AHEAD || !more || wait_bar(kfull(then), then ? par : par ^ 1u, abort_flag, &g_paged_fp8_status, 0xa2, lim));
      ok = __all_sync(kAll, ok);
#pragma unroll
      for (int s = 0; s < HP; ++s) {  // the item's heads in turn: their columns of the rows
        uint64_t sc[KB][NT][2];  // of the lane's two rows, keys lane / 4 and lane / 4 + 8 of a block
        uint32_t pb[KB][NT][2][2];
        float al[NT][2];
        uint64_t back2[NT];
        bool turned = false;  // some row's maximum is a new one
        if (some) {
          if (!AHEAD) products(st, s);
#pragma unroll
          for (int b = 0; b < KB; ++b)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                sc[b][nt][h] = f2pack(part[0][b][nt][2 * h], part[0][b][nt][2 * h + 1]);
                if (HALVES == 2) sc[b][nt][h] = fadd2(sc[b][nt][h], f2pack(part[HALVES - 1][b][nt][2 * h], part[HALVES - 1][b][nt][2 * h + 1]));
              }
          // Scales of the lane's keys lane / 4 and lane / 4 + 8 of each block.
          float vs[KB][2];
#pragma unroll
          for (int b = 0; b < KB; ++b)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int j = 16 * b + 8 * h + (lane >> 2);
              const float ks = scale_of(lds_u8(scales + s * BT + j));
              vs[b][h] = scale_of(lds_u8(scales + (HP + s) * BT + j));
              if (edge && (k0 + j < item.lo || k0 + j >= item.hi)) vs[b][h] = 0.f;  // nobody's: anything may stand there
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) sc[b][nt][h] = fmul2(sc[b][nt][h], f2pack(ks, ks));
            }
          if (k0 < lo_all || k0 + 16 * KB > hi_all) {
#pragma unroll
            for (int b = 0; b < KB; ++b)
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  const int key = k0 + 16 * b + (lane >> 2) + h * 8;
                  float x[2];
                  f2unpack(sc[b][nt][h], x[0], x[1]);
#pragma unroll
                  for (int c = 0; c < 2; ++c)
                    if (key < rlo[nt][c] || key >= rhi[nt][c]) x[c] = -INFINITY;
                  sc[b][nt][h] = f2pack(x[0], x[1]);
                }
          }
          auto softmax = [&] {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              float x[KB][2][2], ref[2], sum[2];
#pragma unroll
              for (int b = 0; b < KB; ++b)
#pragma unroll
                for (int h = 0; h < 2; ++h) f2unpack(sc[b][nt][h], x[b][h][0], x[b][h][1]);
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                float mx = fmaxf(x[0][0][c], x[0][1][c]);
#pragma unroll
                for (int b = 1; b < KB; ++b) mx = fmax3(mx, x[b][0][c], x[b][1][c]);
                mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, 4));
                mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, 8));
                mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, 16));
                const float mn = fmaxf(m[s][nt][c], mx * sl2[s][nt][c]);
                ref[c] = mn == -INFINITY ? 0.f : mn;
                al[nt][c] = ex2(m[s][nt][c] - ref[c]);
                turned |= mn != m[s][nt][c];
                m[s][nt][c] = mn;
              }
              // Two rows at a time: exponentials, their sum, and times the values' scales.
              const uint64_t nref = f2pack(-ref[0], -ref[1]), by = f2pack(sl2[s][nt][0], sl2[s][nt][1]);
              uint64_t both = f2pack(0.f, 0.f);
#pragma unroll
              for (int b = 0; b < KB; ++b)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  float p0, p1;
                  f2unpack(ffma2(sc[b][nt][h], by, nref), p0, p1);
                  const uint64_t p = f2pack(ex2(p0), ex2(p1));
                  both = fadd2(both, p);
                  sc[b][nt][h] = fmul2(p, f2pack(vs[b][h], vs[b][h]));
                }
              f2unpack(both, sum[0], sum[1]);
#pragma unroll
              for (int c = 0; c < 2; ++c) l[s][nt][c] = fmaf(l[s][nt][c], al[nt][c], sum[c]);
            }
            turned = __any_sync(kAll, turned);
            // The weights in two fp16 terms, by a power of two per row that brings its
            // largest to [2^14, 2^15).  Its exponent is in the high half of an fp32 word,
            // so the lane's two rows go through the exchanges as one.  (Weights are not
            // negative; a NaN is passed by.)
            uint64_t f2[NT];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              float most[2] = {0.f, 0.f};
#pragma unroll
              for (int b = 0; b < KB; ++b) {
                float w[2][2];
#pragma unroll
                for (int h = 0; h < 2; ++h) f2unpack(sc[b][nt][h], w[h][0], w[h][1]);
#pragma unroll
                for (int c = 0; c < 2; ++c) most[c] = fmax3(most[c], w[0][c], w[1][c]);
              }
              uint32_t top = __byte_perm(__float_as_uint(most[0]), __float_as_uint(most[1]), 0x7632);
#pragma unroll
              for (int o = 4; o < 32; o <<= 1) top = __vmaxu2(top, __shfl_xor_sync(kAll, top, o));
              const uint32_t e0 = max(top >> 7 & 0x1ffu, 15u), e1 = max(top >> 23, 15u);
              f2[nt] = f2pack(__uint_as_float((268 - e0) << 23), __uint_as_float((268 - e1) << 23));  // 2^(14 - (e - 127))
              back2[nt] = f2pack(__uint_as_float((e0 - 14) << 23), __uint_as_float((e1 - 14) << 23));
            }
#pragma unroll
            for (int b = 0; b < KB; ++b)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                  const uint64_t w = fmul2(sc[b][nt][h], f2[nt]);
                  float x, y;
                  f2unpack(w, x, y);
                  const uint32_t hi = f16x2_rn(x, y);
                  const float2 v = halves(hi);
                  f2unpack(ffma2(f2pack(v.x, v.y), f2pack(-1.f, -1.f), w), x, y);
                  pb[b][nt][0][h] = transpose8x8(hi);
                  pb[b][nt][1][h] = transpose8x8(f16x2_rn(x, y));
                }
              }
          };
          if (AHEAD && more) {
            products(then, 0);
            softmax();
          } else {
            softmax();
          }
        }
        if (some) {
          if (turned) {  // seldom after an item's first tiles
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const uint64_t al2 = f2pack(al[nt][0], al[nt][1]);
#pragma unroll
              for (int x = 0; x < D / 16; ++x) {
                o2[s][nt][x][0] = fmul2(o2[s][nt][x][0], al2);
                o2[s][nt][x][1] = fmul2(o2[s][nt][x][1], al2);
              }
            }
          }
          uint32_t keep[KB][2];  // V rows outside [lo, hi) may hold anything
#pragma unroll
          for (int b = 0; b < KB; ++b)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int key = k0 + 16 * b + 8 * h + 2 * (lane & 3);
              keep[b][h] = !edge ? kAll : (key >= item.lo && key < item.hi ? 0xffffu : 0u) |
                                              (key + 1 >= item.lo && key + 1 < item.hi ? 0xffff0000u : 0u);
            }
          constexpr int PAIRS = NT == 1 ? 2 : 1;  // of 32 columns together: four sums alternate
#pragma unroll
          for (int c0 = 0; c0 < CPR; c0 += 2 * PAIRS) {
            uint32_t w[PAIRS][KB][4];  // (keys 0-7, 8-15) of 16 columns, then of the next 16
#pragma unroll
            for (int x = 0; x < PAIRS; ++x)
#pragma unroll
              for (int b = 0; b < KB; ++b) {
                const int r = key0 + 16 * b + kr;
                ldsm4_t(vb + r * ROW + (((s * CPR + c0 + 2 * x + c2) ^ swz(r)) << 4), w[x][b]);
                if (edge) {
#pragma unroll
                  for (int y = 0; y < 4; ++y) w[x][b][y] &= keep[b][y & 1];
                }
              }
            uint32_t af[2 * PAIRS][KB][4];
#pragma unroll
            for (int x = 0; x < 2 * PAIRS; ++x)
#pragma unroll
              for (int b = 0; b < KB; ++b)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  const uint32_t y = __byte_perm(w[x >> 1][b][2 * (x & 1) + h], 0, 0x3120);
                  af[x][b][2 * h] = low2(y);  // column 2 (lane / 4) of two keys
                  af[x][b][2 * h + 1] = high2(y);  // the next column
                }
            // A tile's product apart, small terms first, then one rounded fp32 step:
            // the tensor core's own accumulation truncates.
            float t[2 * PAIRS][NT][4];
#pragma unroll
            for (int term = 1; term >= 0; --term)
#pragma unroll
              for (int b = 0; b < KB; ++b)
#pragma unroll
                for (int x = 0; x < 2 * PAIRS; ++x)
#pragma unroll
                  for (int nt = 0; nt < NT; ++nt) {
                    if (term == 1 && b == 0) mma_f16_first(t[x][nt], af[x][b], pb[b][nt][1][0], pb[b][nt][1][1]);
                    else mma_f16(t[x][nt], af[x][b], pb[b][nt][term][0], pb[b][nt][term][1]);
                  }
#pragma unroll
            for (int x = 0; x < 2 * PAIRS; ++x)
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                  o2[s][nt][c0 + x][e] = ffma2(f2pack(t[x][nt][2 * e], t[x][nt][2 * e + 1]), back2[nt], o2[s][nt][c0 + x][e]);
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
    float* buf2 = C::IN_Q ? reinterpret_cast<float*>(smem + C::OFF_Q + is * C::QT) : buf + 2 * (4 * D);
#pragma unroll
    for (int s = 0; s < HP; ++s) {
      float o[NT][D / 16][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int x = 0; x < D / 16; ++x) {
          f2unpack(o2[s][nt][x][0], o[nt][x][0], o[nt][x][1]);
          f2unpack(o2[s][nt][x][1], o[nt][x][2], o[nt][x][3]);
        }
      Item part = item;
      if (item.slot >= 0) part.slot = item.slot * HP + s;
      if (!join_warps<D, NT, true, kPlain>(a, part, rec, s * g, m[s], l[s], o, ok, s_m, s_l, buf, buf2, warp, lane)) return;
    }
    if (item.last) return;
    __syncwarp();
    if (lane == 0) mbar_arrive(iempty(is));
  }
}

template <int D, int NT, int HP>
cudaError_t decode_t(const PagedArgs& a, int ctas, const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t st) {
  static std::atomic<unsigned long long> done{0};
  constexpr uint32_t smem = Cfg<D, NT, HP>::SMEM;
  cudaError_t e = allow_smem(paged_fp8_kernel<D, NT, HP>, smem, done);
  if (e != cudaSuccess) return e;
  return launch_early(paged_fp8_kernel<D, NT, HP>, dim3(static_cast<unsigned>(ctas)), kThreads, smem, st, tk, tv, a);
}

}  // namespace

int paged_fp8_row_tile(const PagedArgs& a) { return a.n_q * (a.heads / a.kv_heads) <= 8 ? 8 : 16; }
// At d = 64 and up to 8 rows two KV heads make an item, where they come in pairs: a
// key's rows of both are 128 bytes, which HBM gives at a better rate than 64.  One
// head and two, us: 1.2M keys, 4 heads, 3 rows 168 and 141; 152 requests of up to 6K
// keys, 4 heads 52.8 and 45.4, 8 heads 80.6 and 75.2; 64 of up to 500, 16 heads 18.9
// and 18.7.  A short call takes a longer step with two: 16 requests of up to 2000
// keys, 4 heads 10.8 and 11.8, 8 heads 11.9 and 13.5, 4 of up to 300 9.2 and 11.0; so
// not where the block table has no room for more than 48 MB of pages.  With 16 rows
// the arithmetic is the longer part, and half as many items share the work worse: 60
// requests of 4K keys, 4 heads, 9 rows 36.5 and 46.3, 1.2M keys 176 and 182.  At d =
// 128 pairs take 0.92 of the time for 600K keys, and more for all shorter ones (152
// requests of up to 3000 keys 69 and 78, 16 of up to 2000 13.4 and 16.1; these and
// those of 16 rows with the scores ahead and one power of two for a warp's weights).
int paged_fp8_item_heads(const PagedArgs& a, int d, int row_tile) {
  const long long tokens = (static_cast<long long>(a.n_req) * a.max_pages) << a.page_shift;
  return d == 64 && a.kv_heads % 2 == 0 && row_tile == 8 && tokens * a.kv_heads > (48LL << 20) / (2 * 64) ? 2 : 1;
}
int paged_fp8_box_rows() { return 16 * kCons * KB; }

cudaError_t launch_paged_fp8(const PagedArgs& a, int d, int ctas, int row_tile, const CUtensorMap& tk,
                             const CUtensorMap& tv, cudaStream_t st) {
  if (d == 128)
    return row_tile == 8 ? decode_t<128, 1, 1>(a, ctas, tk, tv, st) : decode_t<128, 2, 1>(a, ctas, tk, tv, st);
  if (a.item_heads == 2) return decode_t<64, 1, 2>(a, ctas, tk, tv, st);
  return row_tile == 8 ? decode_t<64, 1, 1>(a, ctas, tk, tv, st) : decode_t<64, 2, 1>(a, ctas, tk, tv, st);
}

cudaError_t take_paged_fp8_status(int* code) {
  int zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(code, g_paged_fp8_status, sizeof(int));
  if (e != cudaSuccess) return e;
  return cudaMemcpyToSymbol(g_paged_fp8_status, &zero, sizeof(int));
}

}  // namespace ra
