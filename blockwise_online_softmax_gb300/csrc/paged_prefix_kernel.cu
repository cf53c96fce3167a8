// Shared prefixes of groups with more than 16 rows of a KV head, but for the smallest
// works (include/ra.h, ra_paged_decode_prefix; paged_walk.cuh, kShared; the border,
// paged_prefix_both): row tiles of 128 on tcgen05.
// Every row sees the same keys, so a group's rows are one matrix Q and the launch
// is S = Q K^T, P = exp(S - m), O = P V with no mask but at a prefix's end:
// matrix products, bound by the tensor cores where the decode is bound by HBM.
//
// Mathematics, work list, partial states and the P V arithmetic are those of
// paged_tc_kernel.cu (weights in bf16 terms, each tile's product T summed in fp32
// registers, since the tensor core's own accumulation truncates); this kernel
// differs in what stands between the products:
// - TMEM is a ring of slots (Cfg), so neither Q K of a tile waits for P V of the
//   tile whose softmax group it goes to, nor P V for the sum to have read the product
//   before it.  With two S buffers and one T a tile was Q K, a pass of the softmax
//   and P V in turn, halved over the two groups; with three and one, P V and the
//   read of T in turn.
// - The third terms go to shared memory (K-major, 128-byte swizzle, as Q lies) for
//   want of columns.  With bf16 output there is none: two terms, rounded, leave
//   2^-17 of a weight at most, half a step of the output is 2^-8.
// - K and V slots of their own, two each, freed by the product that reads them.
// - One lane issues the products, the one that elect.sync names (elect_one), and what
//   the next tile's P V needs is waited for under this one's.
// 2048 rows of each of 8 KV heads, 16K keys, us (the launch): d = 128 bf16 output 145
// (948 TFLOP/s), fp32 179; d = 64 115 and 150.  What bounds it: at d = 128 the products,
// 24 or 32 of 128 x 128 x 16 a tile at 77 to 65 cycles each (the tensor pipe is 64 and
// 69% busy), and the chain from one to the next, for there are four slots; at d = 64
// a softmax warp's chain (scores from TMEM, exponentials, three cuts, stores, 16 keys at
// a time), which two softmax warps and one of the sum on a scheduler do not cover: no
// unit is full (issue slots 61%, tensor pipe 49%).  Tried on top and no faster: scores and T requested ahead of use
// (146 to 155 and 192 to 198), P V by halves of the keys as their weights come (165,
// 217), a reference that is raised only for scores far above it, so one pass over S
// and no maximum to hand on (the call 227 -> 242 us for fp32 at d = 128, 191 for bf16
// either way).
//
// Roles of the 16 warps: 0-3 and 4-7 softmax, a thread has a row, the two groups
// take a CTA's tiles in turn and hand the running maximum on; 8-11 the output sum;
// 12 K loads and the walk, 13 V loads, 14 the P V products, 15 the query rows and
// the Q K products.
#include <atomic>
#include <cmath>
#include <cstdint>

#include <cuda_bf16.h>

#include "paged_umma.cuh"

namespace ra {

__device__ int g_paged_prefix_status = 0;

namespace {

using namespace paged;
using namespace paged::umma;

constexpr int kA = 3;  // alpha slots

// An item, or the part of it that a CTA has.
struct Item {
  int rows;   // query rows
  int rr0;    // the first: row rr is token rr / g, head kh * g + rr % g
  int row0;   // q row of the group's first token
  int kh;
  int len;    // keys
  int k0;     // first key tile here
  int tiles;  // key tiles here
  int slot;   // partial slot, or -1: the item is whole
  int parts;  // CTAs that it is cut between
  int pad;
};

// True in one lane of the warp.  (With `lane == 0` in its place a product took some 97
// cycles to issue whatever its width; with this it is 46 to 80.  The likely reason is
// that the compiler knows of this form that one lane is left, and so keeps what the
// products share in uniform registers; that has not been looked at.)
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

template <int D, int TERMS>
struct Cfg {
  static constexpr int NCH = D / 64;
  static constexpr uint32_t TILE = BT * D * 2;
  static constexpr uint32_t LOW = TERMS == 3 ? RT * BT * 2 : 0;  // third terms of a tile
  static constexpr int NL = D == 64 ? 4 : 2;                     // of them in flight
  static constexpr uint32_t OFF_Q = 0;
  static constexpr uint32_t OFF_K = TILE, OFF_V = OFF_K + 2 * TILE, OFF_LOW = OFF_V + 2 * TILE;
  static constexpr uint32_t OFF_AL = OFF_LOW + NL * LOW;  // alpha of three tiles
  static constexpr uint32_t OFF_X = OFF_AL + kA * RT * 4;  // running maximum
  static constexpr uint32_t OFF_INV = OFF_X + RT * 4;      // l of one group
  static constexpr uint32_t OFF_ITEM = OFF_INV + RT * 4;
  // Barriers: K and V slots filled and free; S(k) (four by turns); P(k) (four); T(k)
  // ready, which also frees P(k) and its third terms (four); T(k) and alpha(k) read
  // (four); alpha(k) (three); running maximum after k, by group; query rows read;
  // item records in and read; an item's l handed over and its end read; the two
  // issuers' drains.  A wait names its phase by parity: each is for a phase whose
  // successor on the same barrier needs what follows the wait.  And the warps of a
  // role may be tiles apart: where they arrive together, the barrier's next phase
  // needs the one before it complete.  (A group's warp may be at its weights of k + 2
  // while another is at those of k, so P(k) and P(k + 2) have barriers of their own;
  // P(k + 4) needs S(k + 4), that needs T(k + 1), and that P(k).)
  static constexpr int B_KF = 0, B_KE = B_KF + 2, B_VF = B_KE + 2, B_VE = B_VF + 2, B_S = B_VE + 2, B_P = B_S + 4,
                       B_T = B_P + 4, B_TF = B_T + 4, B_AL = B_TF + 4, B_M = B_AL + kA, B_QF = B_M + 2, B_I = B_QF + 1,
                       B_IF = B_I + 2, B_L = B_IF + 2, B_ML = B_L + 1, B_MLF = B_ML + 1, B_DRAIN = B_MLF + 2,
                       NBAR = B_DRAIN + 2;
  static constexpr uint32_t OFF_BAR = OFF_ITEM + 2 * sizeof(Item);
  static constexpr uint32_t OFF_MISC = OFF_BAR + NBAR * 8;
  static constexpr uint32_t SMEM = OFF_MISC + 16;
  static_assert(SMEM <= 232448, "shared memory budget");
  // TMEM columns of S(k) (fp32; P's first two terms over them) and of T(k).  At
  // d = 128 four slots: T(k) takes the one of P(k - 1), which P V of k - 1 has
  // read, S(k + 3) that of T(k) when it has been read.  At d = 64 three for S, two
  // halves of the fourth for T.
  static __device__ __forceinline__ uint32_t s_col(int k) { return static_cast<uint32_t>(D == 128 ? k & 3 : k % 3) * BT; }
  static __device__ __forceinline__ uint32_t t_col(int k) {
    return D == 128 ? static_cast<uint32_t>((k + 3) & 3) * BT : 384u + static_cast<uint32_t>(k & 1) * D;
  }
};

__device__ __forceinline__ void reg_fence16(uint32_t (&r)[16]) {
#pragma unroll
  for (int j = 0; j < 16; ++j) asm volatile("" : "+r"(r[j]));
}

// What a pair of rounded bf16 values leaves of two, exactly (drop_high: of cut ones).
__device__ __forceinline__ void drop(float& a, float& b, uint32_t h) {
  const float na = __uint_as_float((h << 16) ^ 0x80000000u), nb = __uint_as_float((h & 0xffff0000u) ^ 0x80000000u);
  f2unpack(fadd2(f2pack(a, b), f2pack(na, nb)), a, b);
}

template <int D, int TERMS>
__global__ void __launch_bounds__(kThreads, 1)
paged_prefix_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                    const PagedArgs a) {
  using C = Cfg<D, TERMS>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sb = smem_u32(smem);
  auto bar = [&](int i) -> uint32_t { return sb + C::OFF_BAR + 8u * static_cast<uint32_t>(i); };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);
  int* const status = &g_paged_prefix_status;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = a.heads / a.kv_heads;
  start_early<kShared>();
  if (tid == 0) {
    for (int i = 0; i < C::NBAR; ++i) {
      uint32_t n = 1;
      if ((i >= C::B_P && i < C::B_T) || (i >= C::B_TF && i < C::B_QF) || (i >= C::B_L && i < C::B_DRAIN)) n = 128;
      if (i == C::B_IF || i == C::B_IF + 1) n = 13;  // warps 0-11 and 15
      mbar_init(bar(i), n);
    }
    int abort = *reinterpret_cast<volatile int*>(status);
    // The swizzled tiles need 1024-byte alignment, which the declaration asks
    // for; a loader that ignored it would be reported, not computed with.
    if (sb & 1023u) abort = atomicCAS(status, 0, 0xcf) | 0xcf;
    *abort_flag = abort;
    fence_mbar_init();
  }
  start_wait<kShared>();
  const Run run = find_run<BT, 0, kShared, kThreads>(a, g, RT, smem + C::OFF_AL, abort_flag);  // synchronizes
  if (run.first >= run.last || run.stop) return end_wait<kShared>();
  if (warp == 14) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();  // also: the scratch of find_run has been read
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(kAll, *tmem_slot, 0);
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
  auto wait_item = [&](int n) { return wait(C::B_I + (n & 1), static_cast<uint32_t>(n >> 1), 0xc1); };
  auto free_item = [&](int n) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(C::B_IF + (n & 1)));
  };
  auto by4 = [](int k) { return static_cast<uint32_t>(k >> 2); };  // phase of a barrier that goes by k % 4

  if (warp >= 12) {
    regs_dec<88>();
    if (warp == 12 || warp == 13) {
      // -------------------------------------------------------------- K and V loads
      const bool is_k = warp == 12;
      const void* tm = is_k ? static_cast<const void*>(&tmK) : static_cast<const void*>(&tmV);
      const int full = is_k ? C::B_KF : C::B_VF, empty = is_k ? C::B_KE : C::B_VE;
      const int sh = a.page_shift;
      const int rows = sh < 6 ? 1 << sh : 64;  // of a box
      const int boxes = BT / rows;
      const uint32_t box = static_cast<uint32_t>(rows) * 128u;
      Walk<BT, 0, kShared> w;
      w.start(a, g, RT, run.r, run.x);
      long long u = run.first;
      bool ok = true;
      int i = 0, it = 0;
      while (ok && u < run.last) {
        const long long left = run.last - u;
        const int tiles = left < w.t.nt - w.k ? static_cast<int>(left) : w.t.nt - w.k;
        if (is_k) {
          if (it >= 2) ok = wait(C::B_IF + (it & 1), static_cast<uint32_t>(it >> 1) ^ 1u, 0xc2);
          if (!ok) break;
          if (lane == 0) {
            const long long item0 = u - w.k;
            const int c0 = cta_of(item0, run), c1 = cta_of(item0 + w.t.nt - 1, run);
            const int me = static_cast<int>(blockIdx.x);
            items[it & 1] = Item{w.t.rr1 - w.t.rr0, w.t.rr0, w.q.row0, w.kh, w.t.hi, w.k, tiles,
                                 c0 == c1 ? -1 : 2 * me + (me == c0 ? 1 : 0), c1 - c0 + 1, 0};
            mbar_arrive(bar(C::B_I + (it & 1)));
          }
          __syncwarp();
          ++it;
        }
        PageIds ids;
        ids.start<kShared>(a, w.r, w.t.lo, w.t.hi, (w.t.t0 + w.k) * BT, lane);
        for (int k = 0; k < tiles; ++k, ++i) {
          const int key0 = (w.t.t0 + w.k + k) * BT;
          const int page = ids.get(a, key0, rows, boxes, lane);
          const uint32_t n = static_cast<uint32_t>(__popc(__ballot_sync(kAll, page >= 0)));
          const int s = i & 1;
          if (i >= 2) ok = wait(empty + s, static_cast<uint32_t>(i >> 1) ^ 1u, 0xc3);
          if (!ok) break;
          if (lane == 0) mbar_arrive_expect_tx(bar(full + s), n * box * C::NCH);
          __syncwarp();
          if (page >= 0) {
            const uint32_t dst = sb + (is_k ? C::OFF_K : C::OFF_V) + s * C::TILE + lane * box;
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
        for (int j = i > 2 ? i - 2 : 0; j < i; ++j)
          wait_bar(bar(full + (j & 1)), static_cast<uint32_t>(j >> 1) & 1u, &no_abort, nullptr, 0, lim);
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
        if (it > 0) ok = wait(C::B_QF, static_cast<uint32_t>(it - 1), 0xc4);
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
        const bool lead = elect_one();
        const int leader = __ffs(__ballot_sync(kAll, lead)) - 1;
        if (lead) {
          for (int t = 0; t < x.tiles && ok; ++t, ++k) {
            // The slot is free: T(k - 3) has been read, or P(k - 3).
            ok = wait1(C::B_KF + (k & 1), static_cast<uint32_t>(k >> 1), 0xc6) &&
                 (k < 3 || wait1((D == 128 ? C::B_TF : C::B_T) + ((k - 3) & 3), by4(k - 3), 0xc5));
            if (!ok) break;
            tc_fence_after();
            const uint32_t sbuf = tmem + C::s_col(k);
            const uint64_t kd = sdesc_sw128(sb + C::OFF_K + static_cast<uint32_t>(k & 1) * C::TILE, 16, 1024);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint64_t off = ((kk >> 2) * CHB + (kk & 3) * 32) >> 4;
              mma_ss(sbuf, qdesc + off, kd + off, idesc_qk, kk > 0 ? 1u : 0u);
            }
            tc_commit(bar(C::B_KE + (k & 1)));
            tc_commit(bar(C::B_S + (k & 3)));
          }
          if (ok) tc_commit(bar(C::B_QF));
        }
        k = __shfl_sync(kAll, k, leader);
        ok = __shfl_sync(kAll, ok ? 1 : 0, leader) != 0;
      }
      if (elect_one()) {
        volatile int no_abort = 0;
        tc_commit(bar(C::B_DRAIN));
        wait_bar(bar(C::B_DRAIN), 0, &no_abort, nullptr, 0, lim);
      }
    } else {
      // -------------------------------------------------------------- T(k) = P(k) V(k) (warp 14)
      if (elect_one()) {
        constexpr uint32_t idesc_pv = idesc_bf16(RT, D, 1);
        // A wait costs some 200 cycles even where nothing is left to wait for, so what
        // tile k + 1 needs besides its weights is waited for while products of tile k
        // are still queued.
        constexpr bool EARLY = TERMS == 3;
        bool ok = !EARLY || wait1(C::B_VF, 0, 0xc8);
        for (int k = 0; k < total && ok; ++k) {
          // The columns of T(k) are free: P(k - 1) has been read (d = 64: T(k - 2)).
          if (EARLY) {
            ok = wait1(C::B_P + (k & 3), by4(k), 0xc7);
            if (D == 128 && ok && k > 0) ok = wait1(C::B_T + ((k - 1) & 3), by4(k - 1), 0xc9);
          } else {
            const int before = D == 128 ? k - 1 : k - 2;
            ok = wait1(C::B_VF + (k & 1), static_cast<uint32_t>(k >> 1), 0xc8) &&
                 (before < 0 || wait1((D == 128 ? C::B_T : C::B_TF) + (before & 3), by4(before), 0xc9)) &&
                 wait1(C::B_P + (k & 3), by4(k), 0xc7);
          }
          if (!ok) break;
          tc_fence_after();
          const uint64_t vd = sdesc_sw128(sb + C::OFF_V + static_cast<uint32_t>(k & 1) * C::TILE, CHB, 1024);
          const uint32_t pbuf = tmem + C::s_col(k), tbuf = tmem + C::t_col(k);
          // The small terms first; of 16 keys the first two lie side by side, eight
          // columns each.
          if constexpr (TERMS == 3) {
            const uint64_t ld = sdesc_sw128(sb + C::OFF_LOW + static_cast<uint32_t>(k % C::NL) * C::LOW, 16, 1024);
#pragma unroll
            for (int kk = 0; kk < BT / 16; ++kk)
              mma_ss(tbuf, ld + (((kk >> 2) * CHB + (kk & 3) * 32) >> 4), vd + static_cast<uint64_t>((kk * 2048) >> 4),
                     idesc_pv, kk > 0 ? 1u : 0u);
          }
#pragma unroll
          for (int kk = 0; kk < BT / 16; ++kk)
            mma_ts(tbuf, pbuf + 8 + kk * 16, vd + static_cast<uint64_t>((kk * 2048) >> 4), idesc_pv,
                   TERMS == 3 || kk > 0 ? 1u : 0u);
          if (EARLY && k + 1 < total) {
            ok = wait1(C::B_VF + ((k + 1) & 1), static_cast<uint32_t>((k + 1) >> 1), 0xc8);
            if (D == 64 && ok && k > 0) ok = wait1(C::B_TF + ((k - 1) & 3), by4(k - 1), 0xc9);
            if (!ok) break;
          }
#pragma unroll
          for (int kk = 0; kk < BT / 16; ++kk)
            mma_ts(tbuf, pbuf + kk * 16, vd + static_cast<uint64_t>((kk * 2048) >> 4), idesc_pv, 1u);
          tc_commit(bar(C::B_VE + (k & 1)));
          tc_commit(bar(C::B_T + (k & 3)));
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
    bool ok = true;
    int joins = 0;  // items so far that both groups had tiles of
    for (int it = 0, first = 0; ok && first < total; ++it) {
      ok = wait_item(it);
      if (!ok) break;
      const Item x = items[it & 1];
      free_item(it);
      float m = -INFINITY, l = 0.f, alpha = 0.f;
      for (int t = (first ^ gi) & 1; t < x.tiles; t += 2) {
        const int k = first + t;
        const int left = x.len - (x.k0 + t) * BT;  // keys of the tile
        const uint32_t s_col = tl + C::s_col(k);
        ok = wait(C::B_S + (k & 3), by4(k), 0xca);
        if (!ok) break;
        tc_fence_after();
        float mine = -INFINITY;
#pragma unroll 1
        for (int c0 = 0; c0 < BT; c0 += 32) {
          uint32_t v[32];
          tmem_ld32(s_col + c0, v);
          tmem_wait_ld();
          reg_fence32(v);
          if (left < BT) {  // what is no key becomes -inf in place
#pragma unroll
            for (int j = 0; j < 32; j += 8) {
              uint32_t w[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                if (c0 + j + e >= left) v[j + e] = 0xff800000u;
                w[e] = v[j + e];
              }
              tmem_st8(s_col + c0 + j, w);
            }
          }
          float mx0 = fmaxf(__uint_as_float(v[0]), __uint_as_float(v[2])), mx1 = fmaxf(__uint_as_float(v[1]), __uint_as_float(v[3]));
#pragma unroll
          for (int j = 4; j < 32; j += 4) {
            mx0 = fmax3(mx0, __uint_as_float(v[j]), __uint_as_float(v[j + 2]));
            mx1 = fmax3(mx1, __uint_as_float(v[j + 1]), __uint_as_float(v[j + 3]));
          }
          mine = fmax3(mine, mx0, mx1);
        }
        // The running maximum goes from group to group.
        if (k > 0) ok = wait(C::B_M + (gi ^ 1), static_cast<uint32_t>((k - 1) >> 1), 0xd2);
        if (!ok) break;
        const float mp = t > 0 ? s_m[r] : -INFINITY;
        const float mn = fmaxf(mp, mine * sl2);
        s_m[r] = mn;
        mbar_arrive(bar(C::B_M + gi));
        const float ref = mn == -INFINITY ? 0.f : mn;
        alpha = ex2(mp - ref);
        l *= ex2(m - ref);
        m = mn;
        // alpha(k - 3), in the same place, has been read (at d = 128 S(k) says so),
        // and the third terms that lie where this tile's go.
        if (D == 64 && k >= 3) ok = wait(C::B_TF + ((k - 3) & 3), by4(k - 3), 0xd1);
        if (TERMS == 3 && ok && k >= C::NL) ok = wait(C::B_T + ((k - C::NL) & 3), by4(k - C::NL), 0xd4);
        if (!ok) break;
        s_al[k % kA * RT + r] = alpha;
        mbar_arrive(bar(C::B_AL + k % kA));
        const uint32_t low = sb + C::OFF_LOW + static_cast<uint32_t>(k % C::NL) * C::LOW + r * 128;
        const uint64_t nm2 = f2pack(-ref, -ref);
        uint64_t acc0 = f2pack(0.f, 0.f), acc1 = acc0;
        if (left < BT) tmem_wait_st();
        // 16 keys: their weights' terms go where their scores were, the third to
        // shared memory.
        auto weights = [&](const uint32_t (&v)[16], int c0) {
          uint32_t p0[8], p1[8], p2[8];
#pragma unroll
          for (int j = 0; j < 16; j += 2) {
            float y0, y1;
            f2unpack(ffma2(f2pack(__uint_as_float(v[j]), __uint_as_float(v[j + 1])), sl2x2, nm2), y0, y1);
            y0 = ex2(y0);
            y1 = ex2(y1);
            const uint64_t y = f2pack(y0, y1);
            if (j & 2) acc1 = fadd2(acc1, y);
            else acc0 = fadd2(acc0, y);
            if constexpr (TERMS == 3) {  // cut: the three hold all 24 bits
              p0[j / 2] = high_halves(y0, y1);
              drop_high(y0, y1);
              p1[j / 2] = high_halves(y0, y1);
              drop_high(y0, y1);
              p2[j / 2] = high_halves(y0, y1);
            } else {  // rounded
              p0[j / 2] = bf16x2_rn(y0, y1);
              drop(y0, y1, p0[j / 2]);
              p1[j / 2] = bf16x2_rn(y0, y1);
            }
          }
          tmem_st8(s_col + c0, p0);
          tmem_st8(s_col + c0 + 8, p1);
          if constexpr (TERMS == 3) {
            const uint32_t at = low + (c0 >> 6) * CHB;
            const int c = (c0 >> 3) & 7;
            st_shared_v4(at + ((c ^ (r & 7)) << 4), p2[0], p2[1], p2[2], p2[3]);
            st_shared_v4(at + (((c + 1) ^ (r & 7)) << 4), p2[4], p2[5], p2[6], p2[7]);
          }
        };
#pragma unroll 1
        for (int c0 = 0; c0 < BT; c0 += 16) {
          uint32_t v[16];
          tmem_ld16(s_col + c0, v);
          tmem_wait_ld();
          reg_fence16(v);
          weights(v, c0);
        }
        if (left < BT) {
          // Key row r of this tile may be nobody's: zero it for the product.
          ok = wait(C::B_VF + (k & 1), static_cast<uint32_t>(k >> 1), 0xcb);
          if (!ok) break;
          if (r >= left) {
#pragma unroll
            for (int ch = 0; ch < C::NCH; ++ch)
#pragma unroll
              for (int c = 0; c < 8; ++c)
                st_shared_v4(sb + C::OFF_V + static_cast<uint32_t>(k & 1) * C::TILE + ch * CHB + r * 128 + c * 16, 0u, 0u, 0u, 0u);
          }
        }
        if (TERMS == 3 || left < BT) {
          fence_proxy_async_smem();
          __syncwarp();
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(bar(C::B_P + (k & 3)));
        float sa, sc;
        f2unpack(fadd2(acc0, acc1), sa, sc);
        l += sa + sc;
      }
      if (!ok) break;
      // A row's two sums meet in the group that had the item's last tile: the
      // other's refers to the maximum of the tile before, alpha joins them.
      const bool last = ((first + x.tiles - 1) & 1) == gi;
      first += x.tiles;
      // s_inv may be written once the item before has been read.  A group that
      // had no tile of that item did not wait for the one before it, hence two
      // barriers by parity: among three items in a row it had one.
      if (it > 0 && last == (x.tiles == 1))
        ok = wait(C::B_MLF + ((it - 1) & 1), static_cast<uint32_t>((it - 1) >> 1), 0xcc);
      if (!ok) break;
      if (!last && x.tiles > 1) {
        s_inv[r] = l;
        mbar_arrive(bar(C::B_L));
      }
      if (last) {
        if (x.tiles > 1) {
          ok = wait(C::B_L, static_cast<uint32_t>(joins), 0xd3);
          if (!ok) break;
          l = fmaf(s_inv[r], alpha, l);
        }
        mbar_arrive(bar(C::B_ML));
        if (r < x.rows) {
          long long row = static_cast<long long>(x.slot) * RT + r;
          if (x.slot < 0) {
            const int rr = x.rr0 + r, j = rr / g;
            row = a.whole + static_cast<long long>(x.row0 + j) * a.heads + x.kh * g + (rr - j * g);
          }
          a.pm[row] = m;
          a.pl[row] = l;
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
        ok = wait(C::B_AL + k % kA, static_cast<uint32_t>(k) / kA, 0xcd);
        if (!ok) break;
        const float al = s_al[k % kA * RT + r];
        const uint64_t al2 = f2pack(al, al);
        ok = wait(C::B_T + (k & 3), by4(k), 0xce);
        if (!ok) break;
        tc_fence_after();
        const uint32_t col = tl + C::t_col(k);
#pragma unroll
        for (int cc = 0; cc < D / 32; ++cc) {
          uint32_t v[32];
          tmem_ld32(col + cc * 32, v);
          tmem_wait_ld();
          reg_fence32(v);
#pragma unroll
          for (int j = 0; j < 32; j += 2)
            o[cc * 16 + j / 2] = ffma2(o[cc * 16 + j / 2], al2,
                                       f2pack(__uint_as_float(v[j]), __uint_as_float(v[j + 1])));
        }
        tc_fence_before();
        mbar_arrive(bar(C::B_TF + (k & 3)));
      }
      if (!ok) break;
      ok = wait(C::B_ML, static_cast<uint32_t>(it), 0xd0);
      if (!ok) break;
      mbar_arrive(bar(C::B_MLF + (it & 1)));
      if (r >= x.rows) continue;
      const int rr = x.rr0 + r, j0 = rr / g;
      const long long own_row = static_cast<long long>(x.row0 + j0) * a.heads + x.kh * g + (rr - j0 * g);
      const long long row = x.slot >= 0 ? static_cast<long long>(x.slot) * RT + r : own_row + a.whole;
      if (x.slot < 0 || (x.slot & 1))  // not cut, or begun here
        a.parts[own_row] = part_record(x.slot < 0 ? -1 : x.slot * RT + r, x.parts);
      float* dst = a.po + row * D;
#pragma unroll
      for (int j = 0; j < D / 2; j += 2) {
        float y[4];
        f2unpack(o[j], y[0], y[1]);
        f2unpack(o[j + 1], y[2], y[3]);
        *reinterpret_cast<float4*>(dst + 2 * j) = make_float4(y[0], y[1], y[2], y[3]);
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
  end_wait<kShared>();
}

template <int D, int TERMS>
cudaError_t launch_t(const PagedArgs& a, int ctas, const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t st) {
  static std::atomic<unsigned long long> done{0};
  cudaError_t e = allow_smem(paged_prefix_kernel<D, TERMS>, Cfg<D, TERMS>::SMEM, done);
  if (e != cudaSuccess) return e;
  return launch_early(paged_prefix_kernel<D, TERMS>, dim3(static_cast<unsigned>(ctas)), kThreads, Cfg<D, TERMS>::SMEM, st,
                      tk, tv, a);
}

}  // namespace

cudaError_t launch_paged_prefix(const PagedArgs& a, int d, int ctas, const CUtensorMap& tk, const CUtensorMap& tv,
                                cudaStream_t st) {
  if (a.out_bf16) return d == 128 ? launch_t<128, 2>(a, ctas, tk, tv, st) : launch_t<64, 2>(a, ctas, tk, tv, st);
  return d == 128 ? launch_t<128, 3>(a, ctas, tk, tv, st) : launch_t<64, 3>(a, ctas, tk, tv, st);
}

cudaError_t take_paged_prefix_status(int* code) {
  int zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(code, g_paged_prefix_status, sizeof(int));
  if (e != cudaSuccess) return e;
  return cudaMemcpyToSymbol(g_paged_prefix_status, &zero, sizeof(int));
}

}  // namespace ra
