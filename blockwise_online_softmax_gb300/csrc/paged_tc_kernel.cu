// Paged decode for more than 16 query rows of a KV head (many new tokens, or
// many heads on one KV head): row tiles of 128 on tcgen05.  Same mathematics,
// work list, partial states and joining launch as paged_kernel.cu, with key
// tiles of 128 and one CTA per SM.
//
// With rows this many the mma.sync form is bound by its products (each 8 rows
// cost another 13 cycles per 16 x 16 block and SM quarter; 152 requests of 1K
// keys, 8 KV heads, d = 128, 16-row tiles: 3.3 TB/s of pages at 20 and 32 rows,
// 0.9 at 128); here a tile's products are 128 rows at once (4.5 TB/s at 20 rows,
// 3.8 at 128; at d = 64, where a tile takes as long, 2.6 and 2.4).
//
// Roles of the 16 warps: 0-3 and 4-7 softmax, a thread has a row, the two groups
// take a CTA's tiles in turn and hand the running maximum from one to the other;
// 8-11 the output sum (a thread has a row), 12 K loads and the walk over the
// items, 13 V loads, 14 the P V products, 15 the query rows and the Q K products
// (one issuer for both, waiting for each in turn, took 163 us where two took 152).
//   S(k) = Q K(k)^T, two buffers in TMEM.  The softmax cuts P(k) into three bf16
//   terms of 8 bits each, exactly, so that the fp32 result has all 24 of the
//   weights: for each 16 keys two terms where their scores were, one beside.
//   T = P(k) V(k), the small terms first, goes to a buffer of its own, and the
//   output sum takes it as o = o alpha + T in fp32 registers: the tensor core's
//   own accumulation over many tiles truncates, and O never needs a rescale in
//   TMEM.
// The softmax loops are rolled, 16 keys of weights to a turn.  Unrolled over a
// tile their code outgrew the instruction cache next to the other warps' and was
// fetched again for every tile: 152 requests of 1K keys, 128 rows, took 267 us,
// with 32 keys to a turn 167, with 16 166 (20 rows 218, 151, 142).  What bounds it
// now is a tile's chain: a group's pass over its scores, P V, then the next Q K
// into the same columns (2.0 us a tile of 128 keys, its loads 1.5).
// Rows of V outside the item's keys may hold anything (NaN times a zero weight
// is NaN): in tiles that such rows are part of, the softmax warps zero them in
// shared memory before P(k) is handed over.
#include <atomic>
#include <cmath>
#include <cstdint>

#include <cuda_bf16.h>

#include "paged_walk.cuh"

namespace ra {

__device__ int g_paged_tc_status = 0;

namespace {

using namespace paged;

constexpr int BT = 128;          // keys per tile
constexpr int RT = 128;          // query rows of an item
constexpr int kThreads = 512;
constexpr uint32_t CHB = BT * 128;  // one 64-column chunk of a tile, 128-byte swizzle

// An item, or the part of it that a CTA has.  Positions are relative to the
// item's first key tile.
struct Item {
  int rows;   // query rows
  int rr0;    // the first: row rr is token rr / g, head kh * g + rr % g
  int row0;   // q row of the request's first token
  int kh;
  int end0;   // keys that token 0 of the request sees end here
  int base;   // position of the item's first key tile
  int lo, hi; // keys that any row sees
  int k0;     // first key tile here
  int tiles;  // key tiles here
  int slot;   // partial slot, or -1: the item is whole
  int pad;
};

template <int D>
struct Cfg {
  static constexpr int NCH = D / 64;
  static constexpr uint32_t TILE = BT * D * 2;
  static constexpr int NST = D == 128 ? 3 : 6;  // stages of one K and one V tile
  static constexpr uint32_t OFF_Q = 0;
  static constexpr uint32_t OFF_ST = TILE;      // stage s: K at OFF_ST + 2 s TILE, V after it
  static constexpr uint32_t OFF_AL = OFF_ST + NST * 2 * TILE;  // alpha of two tiles
  static constexpr uint32_t OFF_X = OFF_AL + 2 * RT * 4;       // running maximum after two tiles
  static constexpr uint32_t OFF_INV = OFF_X + 2 * RT * 4;      // l of one group, then 1 / l, of an item's rows
  static constexpr uint32_t OFF_ITEM = OFF_INV + RT * 4;
  // Barriers: K and V tiles in, stage free; S(k); P(k); T(k) ready, which also
  // frees P(k)'s columns; T(k) and alpha(k) read; alpha(k) there; query rows
  // read; item record in and read; an item's 1 / l in and read; the two
  // issuers' drains.  Those of a tile come in pairs, by its parity.
  static constexpr int B_KF = 0, B_VF = B_KF + NST, B_E = B_VF + NST, B_S = B_E + NST,
                       B_P = B_S + 2, B_T = B_P + 2, B_TF = B_T + 2, B_AL = B_TF + 2,
                       B_M = B_AL + 2, B_QF = B_M + 2, B_I = B_QF + 1, B_IF = B_I + 2,
                       B_L = B_IF + 2, B_ML = B_L + 1, B_MLF = B_ML + 1, B_DRAIN = B_MLF + 2, NBAR = B_DRAIN + 2;
  static constexpr uint32_t OFF_BAR = OFF_ITEM + 2 * sizeof(Item);
  static constexpr uint32_t OFF_MISC = OFF_BAR + NBAR * 8;
  static constexpr uint32_t SMEM = OFF_MISC + 16;
  static_assert(SMEM <= 232448, "shared memory budget");
  // TMEM columns: S buffers (fp32; P's first two terms over them), the third
  // terms, T.
  static constexpr uint32_t C_S = 0, C_LO = 256, C_T = 384;
};

// 32 lanes x 8 consecutive 32-bit columns.
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// 32 lanes x 16 consecutive 32-bit columns.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
      "[%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
  // (valid after tmem_wait_ld)
}

// The two values cut to bf16, the first in the low half.
__device__ __forceinline__ uint32_t high_halves(float a, float b) {
  return __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
}
// What that leaves of them, exactly.
__device__ __forceinline__ void drop_high(float& a, float& b) {
  const float na = __uint_as_float((__float_as_uint(a) & 0xffff0000u) ^ 0x80000000u);
  const float nb = __uint_as_float((__float_as_uint(b) & 0xffff0000u) ^ 0x80000000u);
  f2unpack(fadd2(f2pack(a, b), f2pack(na, nb)), a, b);
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
paged_tc_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                const PagedArgs a) {
  using C = Cfg<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sb = smem_u32(smem);
  auto bar = [&](int i) -> uint32_t { return sb + C::OFF_BAR + 8u * static_cast<uint32_t>(i); };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);
  int* const status = &g_paged_tc_status;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = a.heads / a.kv_heads;
  Cut* cuts = static_cast<Cut*>(a.cuts);
  let_next_start();
  if (tid == 0) {
    for (int i = 0; i < C::NBAR; ++i) {
      uint32_t n = 1;
      if ((i >= C::B_P && i < C::B_P + 2) || (i >= C::B_TF && i < C::B_M + 2) || (i >= C::B_L && i < C::B_DRAIN)) n = 128;
      if (i == C::B_IF || i == C::B_IF + 1) n = 13;  // warps 0-11 and 15
      mbar_init(bar(i), n);
    }
    int abort = *reinterpret_cast<volatile int*>(status);
    // The swizzled tiles need 1024-byte alignment, which the declaration asks
    // for; a loader that ignored it would be reported, not computed with.
    if (sb & 1023u) abort = atomicCAS(status, 0, 0x9f) | 0x9f;
    *abort_flag = abort;
    fence_mbar_init();
  }
  wait_for_previous();
  if (tid == 0) cuts[blockIdx.x].last = -1;
  const Run run = find_run<BT, 0, kThreads>(a, g, RT, smem + C::OFF_AL, abort_flag);  // synchronizes
  if (run.first >= run.last || run.stop) return;
  if (warp == 14) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();  // also: the scratch of find_run has been read
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const long long lim = a.wait_limit;
  const int total = static_cast<int>(run.last - run.first);  // tiles of this CTA
  Item* items = reinterpret_cast<Item*>(smem + C::OFF_ITEM);
  float* s_al = reinterpret_cast<float*>(smem + C::OFF_AL);
  float* s_m = reinterpret_cast<float*>(smem + C::OFF_X);
  float* s_inv = reinterpret_cast<float*>(smem + C::OFF_INV);
  auto wait = [&](int b, uint32_t parity, int code) {
    const bool w = wait_bar(bar(b), parity & 1u, abort_flag, status, code, lim);
    return static_cast<bool>(__all_sync(kAll, w));
  };
  auto wait1 = [&](int b, uint32_t parity, int code) {  // one lane alone
    return wait_bar(bar(b), parity & 1u, abort_flag, status, code, lim);
  };
  // The record of item n, once it is there; its reader releases it itself.
  auto wait_item = [&](int n) { return wait(C::B_I + (n & 1), static_cast<uint32_t>(n >> 1), 0x91); };
  auto free_item = [&](int n) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(C::B_IF + (n & 1)));
  };

  if (warp >= 12) {
    regs_dec<88>();
    if (warp == 12 || warp == 13) {
      // -------------------------------------------------------------- K and V loads
      const bool is_k = warp == 12;
      const void* tm = is_k ? static_cast<const void*>(&tmK) : static_cast<const void*>(&tmV);
      const int full = is_k ? C::B_KF : C::B_VF;
      const int sh = a.page_shift;
      const int rows = sh < 6 ? 1 << sh : 64;  // of a box
      const int boxes = BT / rows;
      const uint32_t box = static_cast<uint32_t>(rows) * 128u;
      Walk<BT, 0> w;
      w.start(a, g, RT, run.r, run.x);
      long long u = run.first;
      bool ok = true;
      int i = 0, it = 0;
      while (ok && u < run.last) {
        const long long left = run.last - u;
        const int tiles = left < w.t.nt - w.k ? static_cast<int>(left) : w.t.nt - w.k;
        if (is_k) {
          if (it >= 2) ok = wait(C::B_IF + (it & 1), static_cast<uint32_t>(it >> 1) ^ 1u, 0x92);
          if (!ok) break;
          if (lane == 0) {
            const long long item0 = u - w.k;
            const int c0 = cta_of(item0, run), c1 = cta_of(item0 + w.t.nt - 1, run);
            const int me = static_cast<int>(blockIdx.x);
            const int base = w.t.t0 * BT, n = w.t.rr1 - w.t.rr0;
            items[it & 1] = Item{n, w.t.rr0, w.q.row0, w.kh, w.q.len - w.q.n + 1 - base, base,
                                 w.t.lo - base, w.t.hi - base, w.k, tiles,
                                 c0 == c1 ? -1 : 2 * me + (me == c0 ? 1 : 0), 0};
            if (c0 != c1 && me == c0) cuts[me] = Cut{c1, w.q.row0, w.t.rr0, n, w.kh};
            mbar_arrive(bar(C::B_I + (it & 1)));
          }
          __syncwarp();
          ++it;
        }
        PageIds ids;
        ids.start(a, w.r, w.t.lo, w.t.hi, (w.t.t0 + w.k) * BT, lane);
        for (int k = 0; k < tiles; ++k, ++i) {
          const int key0 = (w.t.t0 + w.k + k) * BT;
          const int page = ids.get(a, key0, rows, boxes, lane);
          const uint32_t n = static_cast<uint32_t>(__popc(__ballot_sync(kAll, page >= 0)));
          const int s = i % C::NST;
          if (i >= C::NST) ok = wait(C::B_E + s, static_cast<uint32_t>(i / C::NST) ^ 1u, 0x93);
          if (!ok) break;
          if (lane == 0) mbar_arrive_expect_tx(bar(full + s), n * box * C::NCH);
          __syncwarp();
          if (page >= 0) {
            const uint32_t dst = sb + C::OFF_ST + s * 2 * C::TILE + (is_k ? 0 : C::TILE) + lane * box;
            const int row = (key0 + lane * rows) & ((1 << sh) - 1);
#pragma unroll
            for (int ch = 0; ch < C::NCH; ++ch)
              tma_load_4d(dst + ch * CHB, tm, bar(full + s), ch * 64, w.kh, row, page);
          }
        }
        u += tiles;
        if (ok && u < run.last) w.next(a, g, RT);
      }
      if (!ok) {  // let the copies in flight land before the CTA leaves
        volatile int no_abort = 0;
        for (int j = i > C::NST ? i - C::NST : 0; j < i; ++j)
          wait_bar(bar(full + j % C::NST), static_cast<uint32_t>(j / C::NST) & 1u, &no_abort, nullptr, 0, lim);
      }
    } else if (warp == 15) {
      // -------------------------------------------------------------- query rows, S(k) = Q K(k)^T
      constexpr uint32_t idesc_qk = idesc_bf16(RT, BT, 0);
      const uint64_t qdesc = sdesc_sw128(sb + C::OFF_Q, 16, 1024);
      bool ok = true;
      for (int it = 0, k = 0; ok && k < total; ++it) {
        ok = wait_item(it);
        if (!ok) break;
        const Item x = items[it & 1];
        free_item(it);
        // Rows lane, lane + 32, ...: their index in q, found once.
        int row[RT / 32];
#pragma unroll
        for (int y = 0; y < RT / 32; ++y) {
          const int r = 32 * y + lane, rr = x.rr0 + (r < x.rows ? r : 0), j = rr / g;
          row[y] = (x.row0 + j) * a.heads + x.kh * g + (rr - j * g);
        }
        if (it > 0) ok = wait(C::B_QF, static_cast<uint32_t>(it - 1), 0x94);
        if (!ok) break;
        // Chunk c of row r at c ^ (r % 8) inside its 64 columns, as a TMA load
        // with 128-byte swizzle would put it.  Of 32 rows those past the item's
        // are zero; where all are, they keep what they hold (a row's scores and
        // output come from that row alone).
        constexpr int CPR = D / 8;  // chunks of a row
#pragma unroll
        for (int y = 0; y < RT / 32; ++y) {
          if (32 * y >= x.rows) break;
#pragma unroll 4
          for (int z = 0; z < CPR; ++z) {
            const int r = 32 * y + (z * 32 + lane) / CPR, c = (z * 32 + lane) % CPR;
            const long long at = static_cast<long long>(__shfl_sync(kAll, row[y], r & 31)) * D + c * 8;
            copy16(sb + C::OFF_Q + (c >> 3) * CHB + r * 128 + (((c & 7) ^ (r & 7)) << 4),
                   static_cast<const __nv_bfloat16*>(a.q) + at, r < x.rows ? 16u : 0u);
          }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {  // one lane issues at the pipe's rate, a predicated warp does not
          for (int t = 0; t < x.tiles && ok; ++t, ++k) {
            const int st = k % C::NST;
            ok = wait1(C::B_KF + st, static_cast<uint32_t>(k / C::NST), 0x96) &&
                 (k < 2 || wait1(C::B_T + (k & 1), static_cast<uint32_t>((k - 2) >> 1), 0x95));
            if (!ok) break;
            tc_fence_after();
            const uint32_t sbuf = tmem + C::C_S + static_cast<uint32_t>(k & 1) * BT;
            const uint64_t kd = sdesc_sw128(sb + C::OFF_ST + st * 2 * C::TILE, 16, 1024);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint64_t off = ((kk >> 2) * CHB + (kk & 3) * 32) >> 4;
              mma_ss(sbuf, qdesc + off, kd + off, idesc_qk, kk > 0 ? 1u : 0u);
            }
            tc_commit(bar(C::B_S + (k & 1)));
          }
          if (ok) tc_commit(bar(C::B_QF));
        }
        k = __shfl_sync(kAll, k, 0);
        ok = __shfl_sync(kAll, ok ? 1 : 0, 0) != 0;
      }
      if (lane == 0) {
        volatile int no_abort = 0;
        tc_commit(bar(C::B_DRAIN));
        wait_bar(bar(C::B_DRAIN), 0, &no_abort, nullptr, 0, lim);
      }
    } else {
      // -------------------------------------------------------------- T(k) = P(k) V(k) (warp 14)
      if (lane == 0) {
        constexpr uint32_t idesc_pv = idesc_bf16(RT, D, 1);
        bool ok = true;
        for (int k = 0; k < total && ok; ++k) {
          const int st = k % C::NST;
          ok = wait1(C::B_VF + st, static_cast<uint32_t>(k / C::NST), 0x98) &&
               (k == 0 || wait1(C::B_TF + ((k - 1) & 1), static_cast<uint32_t>((k - 1) >> 1), 0x99)) &&
               wait1(C::B_P + (k & 1), static_cast<uint32_t>(k >> 1), 0x97);
          if (!ok) break;
          tc_fence_after();
          const uint64_t vd = sdesc_sw128(sb + C::OFF_ST + st * 2 * C::TILE + C::TILE, CHB, 1024);
          const uint32_t pbuf = tmem + C::C_S + static_cast<uint32_t>(k & 1) * BT;
          // 16 keys: eight columns of each term, the first two side by side.
          const uint32_t third = tmem + C::C_LO + static_cast<uint32_t>(k & 1) * 64;
#pragma unroll 1
          for (int x = 0; x < 3; ++x)
#pragma unroll
            for (int kk = 0; kk < BT / 16; ++kk)
              mma_ts(tmem + C::C_T, x ? pbuf + (2 - x) * 8 + kk * 16 : third + kk * 8, vd + static_cast<uint64_t>((kk * 2048) >> 4),
                     idesc_pv, x + kk > 0 ? 1u : 0u);
          tc_commit(bar(C::B_E + st));
          tc_commit(bar(C::B_T + (k & 1)));
        }
        volatile int no_abort = 0;
        tc_commit(bar(C::B_DRAIN + 1));
        wait_bar(bar(C::B_DRAIN + 1), 0, &no_abort, nullptr, 0, lim);
      }
    }
    __syncwarp();
  } else if (warp < 8) {
    // ---------------------------------------------------------------- softmax
    // Warps 0-3 take the CTA's even tiles, warps 4-7 the odd ones.
    regs_dec<120>();
    const int r = tid & 127, gi = warp >> 2;
    const uint32_t tl = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const float sl2 = a.scale_log2;
    const uint64_t sl2x2 = f2pack(sl2, sl2);
    const int win = static_cast<int>(a.window);
    const uint32_t s_col = tl + C::C_S + static_cast<uint32_t>(gi) * BT;
    const uint32_t lo_col = tl + C::C_LO + static_cast<uint32_t>(gi) * (BT / 2);
    bool ok = true;
    int joins = 0;  // items so far that both groups had tiles of
    for (int it = 0, first = 0; ok && first < total; ++it) {
      ok = wait_item(it);
      if (!ok) break;
      const Item x = items[it & 1];
      free_item(it);
      // Keys [lo, hi) of the row (rows past the item's do as its last).
      const int rr = x.rr0 + (r < x.rows ? r : x.rows - 1);
      int hi = x.end0 + rr / g;
      if (hi < -x.base) hi = -x.base;
      const int lo = win > 0 && hi + x.base > win ? hi - win : -x.base;
      float m = -INFINITY, l = 0.f, alpha = 0.f;
      for (int t = (first ^ gi) & 1; t < x.tiles; t += 2) {
        const int k = first + t;
        const int k0 = (x.k0 + t) * BT;
        const int lo_j = lo - k0, hi_j = hi - k0;
        // Of any of the warp's rows: the branches below hold warp-wide accesses.
        const bool cut = __any_sync(kAll, lo_j > 0 || hi_j < BT);
        ok = wait(C::B_S + gi, static_cast<uint32_t>(k >> 1), 0x9a);
        if (!ok) break;
        tc_fence_after();
        float mine = -INFINITY;
#pragma unroll 1
        for (int c0 = 0; c0 < BT; c0 += 32) {
          uint32_t v[32];
          tmem_ld32(s_col + c0, v);
          tmem_wait_ld();
          reg_fence32(v);
          if (cut) {  // masked keys become -inf in place
#pragma unroll
            for (int j = 0; j < 32; j += 8) {
              uint32_t w[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                if (c0 + j + e < lo_j || c0 + j + e >= hi_j) v[j + e] = 0xff800000u;
                w[e] = v[j + e];
              }
              tmem_st8(s_col + c0 + j, w);
            }
          }
#define RA_S(j) __uint_as_float(v[j])
          float mx0 = fmaxf(RA_S(0), RA_S(2)), mx1 = fmaxf(RA_S(1), RA_S(3));
#pragma unroll
          for (int j = 4; j < 32; j += 4) {
            mx0 = fmax3(mx0, RA_S(j + 0), RA_S(j + 2));
            mx1 = fmax3(mx1, RA_S(j + 1), RA_S(j + 3));
          }
          mine = fmax3(mine, mx0, mx1);
        }
        // The running maximum goes from group to group.
        if (k > 0) ok = wait(C::B_M + (gi ^ 1), static_cast<uint32_t>((k - 1) >> 1), 0xa2);
        if (!ok) break;
        const float mp = t > 0 ? s_m[(gi ^ 1) * RT + r] : -INFINITY;
        const float mn = fmaxf(mp, mine * sl2);
        s_m[gi * RT + r] = mn;
        mbar_arrive(bar(C::B_M + gi));
        const float ref = mn == -INFINITY ? 0.f : mn;
        alpha = ex2(mp - ref);
        l *= ex2(m - ref);
        m = mn;
        // alpha(k - 2), in the same place, has been read.
        if (k >= 2) ok = wait(C::B_TF + gi, static_cast<uint32_t>((k - 2) >> 1), 0xa1);
        if (!ok) break;
        s_al[gi * RT + r] = alpha;
        mbar_arrive(bar(C::B_AL + gi));
        const uint64_t nm2 = f2pack(-ref, -ref);
        uint64_t acc0 = f2pack(0.f, 0.f), acc1 = acc0;
        if (cut) tmem_wait_st();
#pragma unroll 1
        for (int c0 = 0; c0 < BT; c0 += 16) {  // the terms of 16 keys go where S was
          uint32_t v[16];
          tmem_ld16(s_col + c0, v);
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 16; ++j) asm volatile("" : "+r"(v[j]));
          uint32_t p0[8], p1[8], p2[8];
#pragma unroll
          for (int j = 0; j < 16; j += 2) {
            float y0, y1;
            f2unpack(ffma2(f2pack(RA_S(j), RA_S(j + 1)), sl2x2, nm2), y0, y1);
            y0 = ex2(y0);
            y1 = ex2(y1);
            const uint64_t y = f2pack(y0, y1);
            if (j & 2) acc1 = fadd2(acc1, y);
            else acc0 = fadd2(acc0, y);
            p0[j / 2] = high_halves(y0, y1);
            drop_high(y0, y1);
            p1[j / 2] = high_halves(y0, y1);
            drop_high(y0, y1);
            p2[j / 2] = high_halves(y0, y1);
          }
          tmem_st8(s_col + c0, p0);
          tmem_st8(s_col + c0 + 8, p1);
          tmem_st8(lo_col + c0 / 2, p2);
        }
#undef RA_S
        if (x.lo > k0 || x.hi < k0 + BT) {
          // Key row r of this tile may be nobody's: zero it for the product.
          const int st = k % C::NST;
          ok = wait(C::B_VF + st, static_cast<uint32_t>(k / C::NST), 0x9b);
          if (!ok) break;
          const int key = k0 + r;
          if (key < x.lo || key >= x.hi) {
#pragma unroll
            for (int ch = 0; ch < C::NCH; ++ch)
#pragma unroll
              for (int c = 0; c < 8; ++c)
                st_shared_v4(sb + C::OFF_ST + st * 2 * C::TILE + C::TILE + ch * CHB + r * 128 + c * 16, 0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(bar(C::B_P + gi));
        float sa, sc;
        f2unpack(fadd2(acc0, acc1), sa, sc);
        l += sa + sc;
      }
      if (!ok) break;
      // A row's two sums meet in the group that had the item's last tile: the
      // other's refers to the maximum of the tile before, alpha joins them.
      // That group hands 1 / l to the output and writes the row's statistics.
      const bool last = ((first + x.tiles - 1) & 1) == gi;
      first += x.tiles;
      // s_inv may be written once the item before has been read.  A group that
      // had no tile of that item did not wait for the one before it, hence two
      // barriers by parity: among three items in a row it had one.
      if (it > 0 && last == (x.tiles == 1))
        ok = wait(C::B_MLF + ((it - 1) & 1), static_cast<uint32_t>((it - 1) >> 1), 0x9c);
      if (!ok) break;
      if (!last && x.tiles > 1) {
        s_inv[r] = l;
        mbar_arrive(bar(C::B_L));
      }
      if (last) {
        if (x.tiles > 1) {
          ok = wait(C::B_L, static_cast<uint32_t>(joins), 0xa3);
          if (!ok) break;
          l = fmaf(s_inv[r], alpha, l);
        }
        s_inv[r] = x.slot >= 0 ? 1.f : (l == 0.f ? 0.f : 1.f / l);
        mbar_arrive(bar(C::B_ML));
        if (r < x.rows) {
          if (x.slot >= 0) {
            a.pm[x.slot * RT + r] = m;
            a.pl[x.slot * RT + r] = l;
          } else {
            const int j = rr / g;
            a.lse[static_cast<long long>(x.row0 + j) * a.heads + x.kh * g + (rr - j * g)] =
                l == 0.f ? -INFINITY : m * kLn2 + logf(l);
          }
        }
      }
      if (x.tiles > 1) ++joins;
    }
  } else {
    // ---------------------------------------------------------------- output sum
    regs_inc<184>();
    const int r = tid & 127;
    const uint32_t tl = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    bool ok = true;
    int k = 0;
    for (int it = 0; ok && k < total; ++it) {
      ok = wait_item(it);
      if (!ok) break;
      const Item x = items[it & 1];
      free_item(it);
      uint64_t o[D / 2];
#pragma unroll
      for (int j = 0; j < D / 2; ++j) o[j] = f2pack(0.f, 0.f);
      for (int t = 0; t < x.tiles; ++t, ++k) {
        ok = wait(C::B_AL + (k & 1), static_cast<uint32_t>(k >> 1), 0x9d);
        if (!ok) break;
        const float al = s_al[(k & 1) * RT + r];
        const uint64_t al2 = f2pack(al, al);
        ok = wait(C::B_T + (k & 1), static_cast<uint32_t>(k >> 1), 0x9e);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int cc = 0; cc < D / 32; ++cc) {
          uint32_t v[32];
          tmem_ld32(tl + C::C_T + cc * 32, v);
          tmem_wait_ld();
          reg_fence32(v);
#pragma unroll
          for (int j = 0; j < 32; j += 2)
            o[cc * 16 + j / 2] = ffma2(o[cc * 16 + j / 2], al2,
                                       f2pack(__uint_as_float(v[j]), __uint_as_float(v[j + 1])));
        }
        tc_fence_before();
        mbar_arrive(bar(C::B_TF + (k & 1)));
      }
      if (!ok) break;
      ok = wait(C::B_ML, static_cast<uint32_t>(it), 0xa0);
      if (!ok) break;
      const float inv = s_inv[r];
      mbar_arrive(bar(C::B_MLF + (it & 1)));
      if (r >= x.rows) continue;
      const int rr = x.rr0 + r, j0 = rr / g;
      const long long row = x.slot >= 0 ? static_cast<long long>(x.slot) * RT + r
                                        : static_cast<long long>(x.row0 + j0) * a.heads + x.kh * g + (rr - j0 * g);
      const bool bf16 = x.slot < 0 && a.out_bf16;
      float* dst = (x.slot >= 0 ? a.po : static_cast<float*>(a.out)) + row * D;
      __nv_bfloat16* dst16 = static_cast<__nv_bfloat16*>(a.out) + row * D;
#pragma unroll
      for (int j = 0; j < D / 2; j += 4) {
        float y[8];
#pragma unroll
        for (int c = 0; c < 4; ++c) f2unpack(o[j + c], y[2 * c], y[2 * c + 1]);
#pragma unroll
        for (int c = 0; c < 8; ++c) y[c] *= inv;
        if (bf16) {
          *reinterpret_cast<uint4*>(dst16 + 2 * j) = make_uint4(bf16x2_rn(y[0], y[1]), bf16x2_rn(y[2], y[3]),
                                                                bf16x2_rn(y[4], y[5]), bf16x2_rn(y[6], y[7]));
        } else {
          reinterpret_cast<float4*>(dst + 2 * j)[0] = make_float4(y[0], y[1], y[2], y[3]);
          reinterpret_cast<float4*>(dst + 2 * j)[1] = make_float4(y[4], y[5], y[6], y[7]);
        }
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 14) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D>
cudaError_t launch_d(const PagedArgs& a, int ctas, const CUtensorMap& tk, const CUtensorMap& tv,
                     cudaStream_t st) {
  static std::atomic<unsigned long long> done{0};
  cudaError_t e = allow_smem(paged_tc_kernel<D>, Cfg<D>::SMEM, done);
  if (e != cudaSuccess) return e;
  return launch_early(paged_tc_kernel<D>, dim3(static_cast<unsigned>(ctas)), kThreads, Cfg<D>::SMEM, st, tk, tv, a);
}

}  // namespace

cudaError_t launch_paged_tc(const PagedArgs& a, int d, int ctas, const CUtensorMap& tk,
                            const CUtensorMap& tv, cudaStream_t st) {
  return d == 128 ? launch_d<128>(a, ctas, tk, tv, st) : launch_d<64>(a, ctas, tk, tv, st);
}

cudaError_t take_paged_tc_status(int* code) {
  int zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(code, g_paged_tc_status, sizeof(int));
  if (e != cudaSuccess) return e;
  return cudaMemcpyToSymbol(g_paged_tc_status, &zero, sizeof(int));
}

}  // namespace ra
