// attn_prefill.cu -- causal attention of a ragged batch of new tokens over the
// paged cache, on the tcgen05 tensor cores.
//
// For a tile of query rows (token, query head of one K/V head) and 128 keys,
//   S = Q K^T,   P = 2^(c S - m),   O = O 2^(m_old - m) + P V,   l += sum P
// with a running row maximum m and sum l: one pass over the keys, S and P never
// leave the SM.  Work: 4 D flops a visible (row, key) pair on the tensor cores
// and one exponential; the cache is read once a 256-row tile, from L2 mostly.
//
// One persistent block an SM works on 256 query rows as two tiles of 128, so
// that the tensor core multiplies for one tile while the other tile's
// exponentials are taken:
//   warps 0-3, 4-7   softmax of tile 0 / 1, one row a thread: S from tensor
//                    memory, P back into its place (16 bits), O rescaled only
//                    when a row maximum grew by more than 2^kSlack (the result
//                    is the same for any m)
//   warps 8, 11      issue the MMAs of tile 0 / 1: S = Q K^T (both from shared
//                    memory), O += P V (P from tensor memory, V as stored,
//                    MN-major)
//   warp 9           copies K and V of 128 keys, page by page, into a ring of
//                    swizzled tiles (TMA), where pages are large enough
//   warp 10          copies Q (TMA), where its heads fill tiles evenly
//   warps 12-15      otherwise gather Q, or K and V row by row; look through
//                    the V tiles that some row sees only in part (below)
// The keys' tiles of all (sequence, K/V head, 256-row tile) items, in order,
// are dealt to the blocks in equal consecutive ranges: causal items of any
// lengths balance, and few rows over a long cache are split over the GPU.  An
// item that several blocks share leaves fp32 parts in the workspace, which a
// second small kernel adds in order.
//
// Keys that a row does not see: scores are replaced before the maximum, so
// what K holds does not matter.  0 V would be NaN for a non-finite V, so in
// tiles that some row sees only in part warps 12-15 clear non-finite V
// elements and mark the item; its rows add them back one by one at the end,
// those that see them.
//
// Heads of 128: one prompt of 8192 tokens, 32 heads, takes 437 us, 1.26 PFLOP/s,
// and 512 tokens over 32000, 64 heads on 8, 422 us, 1.28 PFLOP/s, at the power
// limit (414 and 370 us in short runs, before the clocks fall).  The tensor
// cores multiply in two thirds of the clocks; in the others both tiles' products
// wait for a softmax (2900 clocks a pair of tiles, of which 2048 are MMAs).
// Bound by the softmax's latency with heads of 64: four prompts of 2000 to 4096,
// window 1023, 174 us.  Small batches by the first loads and the second kernel:
// three short chunks, 61 MB, 25 us.
#include <algorithm>

#include "kv.cuh"
#include "sm100_ptx.cuh"
#include "tmap.h"

namespace spear {

using namespace sm100;

namespace {
__device__ unsigned g_attn_prefill_status;

constexpr int kTile = 128;                          // keys of a tile, rows of a query tile
constexpr int kRows = 2 * kTile;                    // query rows of an item
constexpr int kHalf = kTile / 2;                    // keys of a softmax step
constexpr int kThreads = 512;
constexpr int kMmaWarp = 8, kTmaWarp = 9, kQWarp = 10, kMmaWarp1 = 11, kLoadWarp = 12, kLoadThreads = 128;
constexpr int kGroups = 2048;                       // entries of the prefix over sequences
constexpr int kKept = 4096;                         // sequences whose lengths are kept in shared memory meanwhile
constexpr uint64_t kLandNs = 2000000000ull;         // limit of the waits for a block's own copies and MMAs, which end by themselves
// log2 growth of a row maximum that is let pass: P's largest values are then up
// to 2^15 apart.  With 8 a row that sees four sinks first is rescaled once more: windowed
// prompts 174 against 172 us, 8192 tokens 419 against 414.
//
// P is taken times 2^kLift; l and o carry the factor, so it cancels, and lse
// takes it out of l.  bf16: 2^-15, so that P stays below 1 and o no larger than
// the sum of the row's |v| (bf16 has fp32's range, below as above).  fp16: 2^8,
// so that P stays below 2^15, which fp16 holds, and a probability is normal down
// to 2^-22 of its row's largest and rounded with an error of 2^-33 of it below
// (unlifted 2^-14 and 2^-25, which shows where the largest one's value is near
// 0, as a sink's is).  In fp16 a slack of 7 costs 1 % with windowed
// prompts, nothing with causal ones as long as scores spread over a few nats, and 5
// to 14 % where they spread over tens; 10 would cost 3 to 7 % there, 4 4 to 10 %
// everywhere.
template <bool F16>
constexpr float kSlack = F16 ? 7.0f : 15.0f;
template <bool F16>
constexpr float kLift = F16 ? 8.0f : -15.0f;
template <bool F16>
__device__ __forceinline__ float log2_sum(float l) { return log2f(l * (F16 ? 0x1p-8f : 0x1p15f)); }
constexpr uint32_t kTmemCols = 512, kColS = 0, kColO = 256;

struct PreArgs {
  KvView c;
  SeqView s;
  const uint16_t* q;
  int64_t qt, qh;
  const int32_t* starts;
  int tokens, q_heads, group;
  FastDiv by_group;
  int window, sinks;
  float scale_log2;
  uint16_t* out;
  float* lse;
  int4* joins;                                      // [2 blocks]: {valid, b, h, t}, {first block, rows, token 0, -}
  float* parts;                                     // [2 blocks][part_floats(D)]
  uint64_t wait_ns;
  int tma;                                          // pages are copied as boxes of this many slots; 0: row by row
  int q_tma;                                        // Q is copied as boxes of `group` heads
};
struct PreMaps {
  CUtensorMap k, v, q;
};

// A block's part of an item: o as [D / 4][row][4], then m [row], l [row].
__host__ __device__ constexpr int64_t part_floats(int D) { return (int64_t)kRows * (D + 2); }

// Whether S of a tile's two halves comes from two rows of MMAs (heads of 64) or
// from one.  With two, the softmax of one half hides the other half's next
// scores: windowed prompts, 253 -> 209 us.  But an MMA of N = 64 with both
// operands in shared memory takes as long as one of N = 128, so heads of 128,
// whose tensor cores are busier, lose: 380 -> 436 us for 512 tokens over 32000.
template <int D>
constexpr bool kSplit = D == 64;

// Whether the two tiles' MMA warps take turns in long pieces (heads of 128, 16
// key tiles or more), so that one tile's softmax falls into the other's
// products.  Left to themselves the tiles drift into step: 375 against 420 us
// for 512 tokens over 32000, 421 against 446 for one prompt of 8192.  Short
// pieces are better without (33 ragged chunks: 590 us, 600 with turns in every
// piece), and so are heads of 64, bound by the softmax (148 against 154 us for
// two prompts of 3000 to 4096).
template <int D>
constexpr bool kTurns = D == 128;

template <int D>
struct Layout {
  static constexpr int kTileBytes = kTile * D * 2;
  static constexpr int kSlots = D == 128 ? 5 : 8;
  static constexpr int kQ = 0, kRing = 2 * kTileBytes, kTotal = kRing + kSlots * kTileBytes;
};

template <int S, int G>                              // constant offsets of both addresses
__device__ __forceinline__ void cp_async16(uint32_t s, uint64_t g) {
  asm volatile("cp.async.cg.shared.global [%0 + %2], [%1 + %3], 16;" ::"r"(s), "l"(g), "n"(S), "n"(G) : "memory");
}

// ------------------------------------------------------------------- items

// Sequence b's new tokens.
struct Seq {
  int b, row, len, tok0, fresh;                     // fresh: new tokens, tok0 the first one
  __device__ __forceinline__ void open(const PreArgs& a, int b_) {
    b = b_;
    row = seq_row(a.s, b, &g_attn_prefill_status);
    len = seq_len(a.s, a.c, row, &g_attn_prefill_status);
    tok0 = a.starts[b];
    const int end = a.starts[b + 1];
    fresh = end - tok0;
    if (tok0 < 0 || end < tok0 || end > a.tokens) {
      record_status(&g_attn_prefill_status, DEV_ERR_INVALID);
      fresh = 0;
    }
  }
  __device__ __forceinline__ int tiles(const PreArgs& a) const { return (fresh * a.group + kRows - 1) / kRows; }
};

// 256 rows of one K/V head of a sequence: row r of it is token (256 t + r) /
// group, query head (256 t + r) % group; its key tiles in two runs, those of
// the sinks and those from `from`.
struct Item {
  int pos0, pos1;                                   // positions of its first and last token
  int rows, sink_tiles, from, n;
  __device__ __forceinline__ void open(const PreArgs& a, const Seq& s, int t) {
    rows = min(kRows, s.fresh * a.group - t * kRows);
    const int base = s.len - s.fresh;
    pos0 = base + (int)a.by_group.div(t * kRows);
    pos1 = base + (int)a.by_group.div(t * kRows + rows - 1);
    // The first token's window begins first; a later token's sinks are below
    // that, or in the first token's window.
    const Visible v = visible_keys(pos0, a.window, a.sinks);
    sink_tiles = (v.sink_end + kTile - 1) / kTile;
    from = max(sink_tiles, v.win_begin / kTile);
    n = max(1, sink_tiles + (pos1 < 0 ? 0 : pos1 / kTile - from + 1));
  }
  __device__ __forceinline__ int key0(int i) const { return (i < sink_tiles ? i : i - sink_tiles + from) * kTile; }
  // Whether some row sees some of the tile's keys and not others.
  __device__ __forceinline__ bool partial(const PreArgs& a, int j0) const {
    return !(j0 + kTile - 1 <= pos0 &&
             (a.window == 0 || j0 > pos1 - a.window || j0 + kTile <= a.sinks));
  }
};

// An item's units: its tiles, and kSetup for what an item costs besides (Q,
// the first scores without a partner, the epilogue), dealt before the tiles.
// 2 is better for long prompts (8192 tokens: 422 against 437 us at the power
// limit), 1 for short chunks (26 against 28 us), which serving has more of.
constexpr int kSetup = 1;

// Units of sequence s under one K/V head (all 32 lanes, same result).
__device__ __forceinline__ long long seq_units(const PreArgs& a, const Seq& s) {
  long long sum = 0;
  const int tiles = s.tiles(a);
  for (int t = threadIdx.x & 31; t < tiles; t += 32) {
    Item it;
    it.open(a, s, t);
    sum += it.n + kSetup;
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(~0u, sum, d);
  return sum;
}

// Where a block's units start, and its pieces: consecutive tiles of an item.
struct Start {
  Seq s;
  int h, t, unit;
  long long units;                                  // of the block
};
struct Walk {
  Seq s;
  Item it;
  int h, t;
  int tile, n;                                      // the piece: tiles [tile, tile + n) of the item; n = 0: no more
  long long left;                                   // units after it
  __device__ __forceinline__ Walk(const PreArgs& a, const Start& st) : h(st.h), t(st.t), n(0), left(st.units) {
    if (left <= 0) return;
    s = st.s;
    it.open(a, s, t);
    cut(st.unit);
    if (n == 0) next(a);
  }
  __device__ __forceinline__ void cut(int unit) {
    const int cover = (int)min(left, (long long)(it.n + kSetup - unit));
    tile = max(0, unit - kSetup);
    n = max(0, unit + cover - kSetup) - tile;
    left -= cover;
  }
  __device__ __forceinline__ void next(const PreArgs& a) {
    n = 0;
    while (left > 0 && n == 0) {
      if (++t >= s.tiles(a)) {
        t = 0;
        if (++h >= a.c.heads) {
          h = 0;
          do s.open(a, s.b + 1); while (s.fresh == 0);
        }
      }
      it.open(a, s, t);
      cut(0);
    }
  }
};

struct Shared {
  uint64_t kv_full[8], kv_empty[8], landed[8], q_full, q_empty, s_full[2][2], p_full[2][2], pv_done[2][2], o_free[2], turn[2], drained[2];
  uint32_t tmem;
  int abort;
  int bad[8];                                       // 1 + the last piece (of those alike mod 8) with cleared V elements
  Start start;
};

__device__ __forceinline__ void give_up(Shared& sh) {
  record_status(&g_attn_prefill_status, DEV_ERR_TIMEOUT);
  atomicExch(&sh.abort, 1);
}
// A bounded wait of a whole warp: false when it ran out or another role gave
// up.  A waiting warp is suspended for a while at a time (kNapNs or so), and
// the clock and the flag are looked at in between.
constexpr uint32_t kNapNs = 20000;
__device__ __forceinline__ bool wait_slow(Shared& sh, uint32_t bar, uint32_t parity, uint64_t limit) {
  const uint64_t t0 = globaltimer_ns();
  for (;;) {
    if (__all_sync(~0u, mbar_try_wait_suspend(bar, parity, kNapNs))) return true;
    if (__any_sync(~0u, *reinterpret_cast<volatile int*>(&sh.abort))) return false;
    if (__any_sync(~0u, globaltimer_ns() - t0 > limit)) {
      give_up(sh);
      return false;
    }
  }
}
__device__ __forceinline__ bool wait(Shared& sh, const uint64_t& bar, uint32_t parity, uint64_t limit) {
  return __all_sync(~0u, mbar_try_wait(smem_u32(&bar), parity)) || wait_slow(sh, smem_u32(&bar), parity, limit);
}
// The same for a limit shorter than a nap, polling.
__device__ __forceinline__ bool wait_poll(Shared& sh, const uint64_t& bar, uint32_t parity, uint64_t limit) {
  const uint64_t t0 = globaltimer_ns();
  while (!__all_sync(~0u, mbar_test_wait(smem_u32(&bar), parity)))
    if (__any_sync(~0u, globaltimer_ns() - t0 >= limit)) {
      give_up(sh);
      return false;
    }
  return true;
}

__device__ __forceinline__ uint64_t desc_k(uint32_t addr) { return smem_desc(addr, 1024, LAYOUT_SW128); }
// MN-major, 128-byte swizzle: 64 columns a panel, panels 128 rows of 128 bytes
// apart, groups of 8 k 1024 bytes apart.
__device__ __forceinline__ uint64_t desc_mn(uint32_t addr) {
  return (uint64_t)((addr >> 4) & 0x3FFF) | ((uint64_t)((kTile * 128) >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)LAYOUT_SW128 << 61);
}

// ------------------------------------------------------------------ loading

template <int N>
__device__ __forceinline__ void reg_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void reg_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

template <bool F16>
__device__ __forceinline__ uint32_t clear_nonfinite2(uint32_t v) {
  constexpr uint32_t e = F16 ? 0x7c00u : 0x7f80u;
  if ((v & e) == e) v &= 0xffff0000u;
  if ((v >> 16 & e) == e) v &= 0x0000ffffu;
  return v;
}

// acc + 0 v: stays 0 (of either sign) as long as the values are finite, NaN from the first that is not.
template <bool F16>
__device__ __forceinline__ uint32_t zero_times2(uint32_t v, uint32_t acc) {
  uint32_t r;
  if (F16) asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(v), "r"(0u), "r"(acc));
  else asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(v), "r"(0u), "r"(acc));
  return r;
}

template <int D, bool F16>
struct Loader {
  using L = Layout<D>;
  static constexpr int kVecs = D / 8, kRowsPass = 32 / kVecs, kPasses = 32 / kRowsPass;
  const PreArgs& a;
  Shared& sh;
  uint32_t smem;
  int warp, lane;                                   // warp 0-3 of the gathering warps: rows 32 warp ..

  // 16-byte piece x of row r of a tile: panel x / 8, 128-byte swizzle within.
  static __device__ __forceinline__ uint32_t at(int r, int x) {
    return (x >> 3) * (kTile * 128) + r * 128 + (((x & 7) ^ (r & 7)) << 4);
  }

  // Clears the non-finite elements of this warp's rows of a V tile; `keys` of
  // its rows hold keys that some row of the item may see.  Whether there are
  // any shows in a product with zero, two elements an instruction.
  __device__ __forceinline__ void scan(uint32_t tile, int piece, int keys) {
    uint32_t acc[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const int r = warp * 32 + i * kRowsPass + lane / kVecs;
      uint4 v;
      asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(tile + at(r, lane % kVecs)) : "memory");
      acc[0] = zero_times2<F16>(v.x, zero_times2<F16>(v.y, acc[0]));
      acc[1] = zero_times2<F16>(v.z, zero_times2<F16>(v.w, acc[1]));
    }
    if (((acc[0] | acc[1]) & 0x7fff7fff) == 0) return;
    bool any = false;
#pragma unroll 1
    for (int i = 0; i < kPasses; ++i) {
      const int r = warp * 32 + i * kRowsPass + lane / kVecs;
      const uint32_t p = tile + at(r, lane % kVecs);
      uint4 v;
      asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(p) : "memory");
      const uint4 c = make_uint4(clear_nonfinite2<F16>(v.x), clear_nonfinite2<F16>(v.y),
                                 clear_nonfinite2<F16>(v.z), clear_nonfinite2<F16>(v.w));
      if (c.x != v.x || c.y != v.y || c.z != v.z || c.w != v.w) {
        any |= r < keys;
        asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(p), "r"(c.x), "r"(c.y), "r"(c.z), "r"(c.w) : "memory");
      }
    }
    if (any) {
      atomicMax(&sh.bad[piece & 7], piece + 1);
      __threadfence_block();
    }
  }
  // This warp's part of a tile is in place: written or looked through by these
  // threads, for the tensor cores to read.
  __device__ __forceinline__ void hand_on(uint32_t bar) {
    fence_proxy_async_smem();
    mbar_arrive(bar);
  }
  // The same for copies still under way: the arrivals come when they land (and
  // the thread that issues the MMAs orders them before those).
  __device__ __forceinline__ void hand_on_landed(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
  }
  __device__ __forceinline__ void landed() {
    cp_async_commit();
    cp_async_wait<0>();
  }

  // This lane's row (key j0 + 32 warp + lane) of a tile: its page.
  int32_t page;
  int slot;
  bool in;
  __device__ __forceinline__ void look_up(const Walk& w, int i) {
    const int pos = w.it.key0(i) + warp * 32 + lane;
    in = pos < w.s.len && pos <= w.it.pos1;
    if (in) {
      const uint32_t pg = a.c.page.div((uint32_t)pos);
      slot = pos - (int)(pg * a.c.page.d);
      page = a.s.table[w.s.row * a.s.table_stride + pg];
    }
  }
  __device__ __forceinline__ int64_t offset(int h) {
    if (!in) return -1;
    if ((unsigned)page >= (unsigned)a.c.num_pages) {
      record_status(&g_attn_prefill_status, DEV_ERR_INVALID);
      return -1;
    }
    return (int64_t)page * a.c.page_stride + (int64_t)slot * a.c.slot_stride + (int64_t)h * a.c.head_stride;
  }
  // This warp's 32 rows of a tile, of which this lane has row `lane` at off
  // (none: -1, zeros).  Eight lanes copy a row, 128 bytes of each panel: few
  // instructions count, since the softmax's warps share the schedulers (8192
  // tokens: 532 us with an address and a test for each 16 bytes, 446 so).
  __device__ __forceinline__ void copy(uint32_t dst, const uint16_t* base, int64_t off) {
    const uint64_t from = reinterpret_cast<uint64_t>(base + (off < 0 ? 0 : off));
    const unsigned there = __ballot_sync(~0u, off >= 0);
    const int r0 = lane >> 3, x = lane & 7;
    if (there == ~0u) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = 4 * i + r0;
        const uint64_t g = __shfl_sync(~0u, from, r) + 16 * x;
        const uint32_t d = dst + at(warp * 32 + r, x);
        cp_async16<0, 0>(d, g);
        if (D == 128) cp_async16<kTile * 128, 128>(d, g);
      }
    } else {
#pragma unroll 1
      for (int i = 0; i < 8; ++i) {
        const int r = 4 * i + r0;
        const uint16_t* g = reinterpret_cast<const uint16_t*>(__shfl_sync(~0u, from, r)) + 8 * x;
        const uint32_t d = dst + at(warp * 32 + r, x);
        cp_async16_zfill(d, g, there >> r & 1);
        if (D == 128) cp_async16_zfill(d + kTile * 128, g + 64, there >> r & 1);
      }
    }
  }

  // Q: rows 32 warp .. of both tiles
  __device__ __forceinline__ void copy_q(const Walk& w) {
#pragma unroll 1
    for (int q = 0; q < 2; ++q) {
      const int r = q * kTile + warp * 32 + lane, rr = w.t * kRows + r;
      const int tok = (int)a.by_group.div(rr);
      const int64_t off = r < w.it.rows ? (w.s.tok0 + tok) * a.qt + (int64_t)(w.h * a.group + rr - tok * a.group) * a.qh
                                        : -1;
      copy(smem + L::kQ + q * L::kTileBytes, a.q, off);
    }
  }

  // With K and V copied by the TMA warp: Q, and the look through V tiles that
  // are seen in part.
  __device__ __forceinline__ void run_beside_tma() {
    Walk w(a, sh.start);
    uint32_t nslot = 0, uses = 0;                   // uses: a bit a slot, the parity of its next scan
    for (int piece = 0; w.n > 0; ++piece, w.next(a)) {
      if (!a.q_tma) {
        if (!wait(sh, sh.q_empty, (piece & 1) ^ 1, a.wait_ns)) break;
        copy_q(w);
        landed();
        hand_on(smem_u32(&sh.q_full));
      }
      const int n = w.n;
      bool ok = true;
      for (int i = 0; i < n && ok; ++i) {
        const int j0 = w.it.key0(w.tile + i);
        const uint32_t vs = nslot + 1 < L::kSlots ? nslot + 1 : nslot + 1 - L::kSlots;
        nslot = vs + 1 < L::kSlots ? vs + 1 : 0;
        if (!w.it.partial(a, j0)) continue;
        ok = wait(sh, sh.landed[vs], uses >> vs & 1, a.wait_ns);
        uses ^= 1u << vs;
        if (!ok) break;
        scan(smem + L::kRing + vs * L::kTileBytes, piece, w.it.pos1 + 1 - j0);
        hand_on(smem_u32(&sh.kv_full[vs]));
      }
      if (!ok) break;
    }
  }

  // All of it gathered.  A V tile that is seen in part is looked through after
  // the next tile's copies are under way, or the next piece is opened, not to
  // wait for it meanwhile (those copies need only slots that are free once
  // earlier tiles' products are made).
  __device__ __forceinline__ void run() {
    Walk w(a, sh.start);
    uint32_t nslot = 0, phase = 0;                  // slots and their use
    uint32_t late = 0, late_bar = 0;                // such a tile and its barrier; 0: none
    int late_piece = 0, late_keys = 0;
    // Every lane has waited for its own copies of the tile; a lane scans pieces
    // that others copied (heads of 128), so the warp meets first.
    const auto finish = [&] {
      __syncwarp();
      scan(late, late_piece, late_keys);
      hand_on(late_bar);
      late = 0;
    };
    for (int piece = 0; w.n > 0; ++piece, w.next(a)) {
      const int n = w.n;
      look_up(w, w.tile);
      if (late) {
        cp_async_wait<0>();
        finish();
      }
      if (!wait(sh, sh.q_empty, (piece & 1) ^ 1, a.wait_ns)) break;
      copy_q(w);
      hand_on_landed(smem_u32(&sh.q_full));
      bool ok = true;
      for (int i = 0; i < n && ok; ++i) {
        const int64_t off = offset(w.h);
        const int j0 = w.it.key0(w.tile + i);
        if (i + 1 < n) look_up(w, w.tile + i + 1);
#pragma unroll 1
        for (int kv = 0; kv < 2; ++kv) {
          ok = wait(sh, sh.kv_empty[nslot], phase ^ 1, a.wait_ns);
          if (!ok) break;
          const uint32_t dst = smem + L::kRing + nslot * L::kTileBytes, bar = smem_u32(&sh.kv_full[nslot]);
          SPEAR_CHECK(&g_attn_prefill_status, nslot < L::kSlots && j0 >= 0 && w.tile + i < w.it.n);
          copy(dst, kv ? a.c.v : a.c.k, off);
          cp_async_commit();
          if (kv && late) {                         // of the tile before
            cp_async_wait<2>();
            finish();
          }
          if (kv && w.it.partial(a, j0)) {
            late = dst;
            late_bar = bar;
            late_piece = piece;
            late_keys = w.it.pos1 + 1 - j0;
          } else {
            hand_on_landed(bar);
          }
          if (++nslot == L::kSlots) {
            nslot = 0;
            phase ^= 1;
          }
        }
      }
      if (!ok) break;
    }
    landed();
    if (late) finish();
  }
};

// K and V tiles by TMA: lane x copies the box of slots x boxes .. of the tile,
// panel by panel; a key past the last one that is needed, or a page that does
// not exist, is a box outside the tensor, which reads as zeros.
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const void* tmap, int c0, int c1, int c2, int c3, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];"
      ::"r"(dst), "l"(reinterpret_cast<uint64_t>(tmap)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void* tmap, int c0, int c1, int c2, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
      ::"r"(dst), "l"(reinterpret_cast<uint64_t>(tmap)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void mbar_arrive_n(uint32_t bar, uint32_t n) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(n) : "memory");
}
template <int D>
__device__ __forceinline__ void tma_role(const PreArgs& a, const PreMaps& maps, Shared& sh, uint32_t smem) {
  using L = Layout<D>;
  const int lane = threadIdx.x & 31, boxes = kTile / a.tma;
  Walk w(a, sh.start);
  uint32_t nslot = 0, phase = 0, landed = 0;        // landed: a bit a slot, the parity of its next use
  uint32_t used = 0, scanned = 0;                   // slots with a copy, and those that a scan follows
  int page = 0, slot = 0;
  bool need = false;
  auto look_up = [&](int i) {                       // box `lane` of tile i
    const int pos = w.it.key0(i) + lane * a.tma;
    need = lane < boxes && pos < w.s.len && pos <= w.it.pos1;
    if (need) {
      const uint32_t pg = a.c.page.div((uint32_t)pos);
      slot = pos - (int)(pg * a.c.page.d);
      page = a.s.table[w.s.row * a.s.table_stride + pg];
    }
  };
  bool ok = true;
  if (w.n > 0) look_up(w.tile);
  while (w.n > 0 && ok) {
    const int n = w.n;
    for (int i = 0; i < n && ok; ++i) {
      const bool part = w.it.partial(a, w.it.key0(w.tile + i));
      const int at = need ? slot : 0;
      int pg = need ? page : a.c.num_pages;
      if ((unsigned)pg >= (unsigned)a.c.num_pages) {
        if (need) record_status(&g_attn_prefill_status, DEV_ERR_INVALID);
        pg = a.c.num_pages;
      }
      if (i + 1 < n) look_up(w.tile + i + 1);
#pragma unroll 1
      for (int kv = 0; kv < 2; ++kv) {
        ok = wait(sh, sh.kv_empty[nslot], phase ^ 1, a.wait_ns);
        if (!ok) break;
        const bool scan = kv && part;
        SPEAR_CHECK(&g_attn_prefill_status, nslot < L::kSlots && (at + a.tma <= (int)a.c.page.d || pg == a.c.num_pages));
        const uint32_t bar = smem_u32(scan ? &sh.landed[nslot] : &sh.kv_full[nslot]), bit = 1u << nslot;
        const uint32_t dst = smem + L::kRing + nslot * L::kTileBytes + lane * a.tma * 128;
        if (lane == 0) {
          mbar_arrive_expect_tx(bar, L::kTileBytes);
          if (!scan) mbar_arrive_n(bar, kLoadThreads - 1);
        }
        __syncwarp();
        if (lane < boxes) {
          const void* map = kv ? &maps.v : &maps.k;
#pragma unroll
          for (int p = 0; p < D / 64; ++p) tma_load_4d(dst + p * (kTile * 128), map, p * 64, at, w.h, pg, bar);
        }
        __syncwarp();
        used |= bit;
        scanned = scan ? scanned | bit : scanned & ~bit;
        if (scan) landed ^= bit;
        if (++nslot == L::kSlots) {
          nslot = 0;
          phase ^= 1;
        }
      }
    }
    if (!ok) break;
    w.next(a);
    if (w.n > 0) look_up(0);
  }
  // after a wait that ran out nobody else takes the copies under way: they land first
  if (*reinterpret_cast<volatile int*>(&sh.abort))
    for (uint32_t i = 0; i < L::kSlots; ++i)
      if (used >> i & 1) {
        const bool l = scanned >> i & 1;
        mbar_wait(smem_u32(l ? &sh.landed[i] : &sh.kv_full[i]), l ? (landed >> i & 1) ^ 1 : i < nslot ? phase : phase ^ 1,
                  kLandNs);
      }
}

// Q by TMA, where a K/V head's query heads divide 128: rows (token, head) of a
// tile are a box of the tensor.  Rows past the item's are other rows of q (or
// zeros past its end), whose results are not used.
template <int D>
__device__ __forceinline__ void q_role(const PreArgs& a, const PreMaps& maps, Shared& sh, uint32_t smem) {
  using L = Layout<D>;
  const int lane = threadIdx.x & 31;
  Walk w(a, sh.start);
  int piece = 0;
  for (; w.n > 0; ++piece, w.next(a)) {
    if (!wait(sh, sh.q_empty, (piece & 1) ^ 1, a.wait_ns)) break;
    if (lane == 0) {
      const uint32_t bar = smem_u32(&sh.q_full);
      mbar_arrive_expect_tx(bar, 2 * L::kTileBytes);
      mbar_arrive_n(bar, kLoadThreads - 1);
      for (int q = 0; q < 2; ++q) {
        const int tok = w.s.tok0 + (int)a.by_group.div(w.t * kRows + q * kTile);
        for (int p = 0; p < D / 64; ++p)
          tma_load_3d(smem + L::kQ + q * L::kTileBytes + p * (kTile * 128), &maps.q, p * 64, w.h * a.group, tok, bar);
      }
    }
    __syncwarp();
  }
  // as in tma_role
  if (*reinterpret_cast<volatile int*>(&sh.abort) && piece > 0)
    mbar_wait(smem_u32(&sh.q_full), (piece & 1) ^ 1, kLandNs);
}

// --------------------------------------------------------------------- MMAs

template <int D, bool F16, bool TMA>
__device__ __forceinline__ void mma_role(const PreArgs& a, Shared& sh, uint32_t smem, int q) {
  using L = Layout<D>;
  constexpr int kN = kSplit<D> ? kHalf : kTile, kPofHalf = kSplit<D> ? kHalf : kHalf / 2;   // columns of P's halves
  const uint32_t idesc_s = F16 ? idesc_f16_f32(kTile, kN) : idesc_bf16_f32(kTile, kN);
  const uint32_t idesc_o = (F16 ? idesc_f16_f32(kTile, D) : idesc_bf16_f32(kTile, D)) | (1u << 16);   // B is MN-major
  const uint32_t tmem = sh.tmem;
  Walk w(a, sh.start);
  uint32_t nslot = 0, phase = 0;
  uint32_t done = 0, items = 0, turns = 0;                     // P tiles taken, pieces with rows of this query tile

  auto scores = [&](int half, uint32_t slot) {
    const uint32_t ka = smem + L::kRing + slot * L::kTileBytes + half * (kHalf * 128);
    const uint32_t qa = smem + L::kQ + q * L::kTileBytes;
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      const uint32_t o = (k >> 2) * (kTile * 128) + (k & 3) * 32;
      mma_bf16_ss_warp(tmem + kColS + q * kTile + half * kHalf, desc_k(qa + o), desc_k(ka + o), idesc_s, k > 0);
    }
    mma_commit_warp(smem_u32(&sh.s_full[q][half]));
  };
  auto values = [&](int half, uint32_t slot, bool add) {    // O += P V of 64 keys; P lies where their S did
    const uint32_t va = smem + L::kRing + slot * L::kTileBytes + half * (kHalf * 128);
#pragma unroll
    for (int k = 0; k < kHalf / 16; ++k)
      mma_bf16_ts_warp(tmem + kColO + q * kTile, tmem + kColS + q * kTile + half * kPofHalf + k * 8, desc_mn(va + k * 2048),
                       idesc_o, add || k > 0);
    mma_commit_warp(smem_u32(&sh.pv_done[q][half]));
  };
  auto take = [&](uint32_t& slot) {                 // the next ring slot, once it is full
    slot = nslot;
    const bool ok = wait(sh, sh.kv_full[nslot], phase, a.wait_ns);
    if (!TMA) fence_proxy_async_smem();              // gathered rows: written by ordinary copies
    if (++nslot == L::kSlots) {
      nslot = 0;
      phase ^= 1;
    }
    return ok;
  };

  auto give = [&](const uint64_t& bar, bool mine) { // this warp is done with a slot: once its MMAs are, or at once
    if (mine) mma_commit_warp(smem_u32(&bar));
    else if ((threadIdx.x & 31) == 0) mbar_arrive(smem_u32(&bar));
  };

  for (int piece = 0; w.n > 0; ++piece, w.next(a)) {
    const int n = w.n;
    const bool both = kTurns<D> && w.it.rows > kTile && n >= 16;
    const bool mine = q * kTile < w.it.rows;         // the other warp's tile may be the item's only one
    uint32_t sk, sv;
    // (once a piece: this is where a limit shorter than a nap shows)
    if (a.wait_ns <= kNapNs && !wait_poll(sh, sh.q_full, piece & 1, a.wait_ns)) return;
    if (!wait(sh, sh.q_full, piece & 1, a.wait_ns) || !take(sk)) return;
    tc_fence_after();
    if (mine)
      for (int half = 0; half < (kSplit<D> ? 2 : 1); ++half) scores(half, sk);
    give(sh.kv_empty[sk], mine);
    if (n == 1) give(sh.q_empty, mine);
    for (int i = 0; i < n; ++i) {
      const bool more = i + 1 < n;
      if (!take(sv) || (more && !take(sk))) return;
      if (mine) {
        if (i == 0 && !wait(sh, sh.o_free[q], (items & 1) ^ 1, a.wait_ns)) return;
        if (!wait(sh, sh.p_full[q][0], done & 1, a.wait_ns)) return;
        if (both && i > 0 && !wait(sh, sh.turn[q], (turns & 1) ^ (q == 0), a.wait_ns)) return;
        tc_fence_after();
        values(0, sv, i > 0);
        if (kSplit<D> && more) scores(0, sk);
        if (!wait(sh, sh.p_full[q][1], done & 1, a.wait_ns)) return;
        tc_fence_after();
        values(1, sv, true);
        ++done;
      }
      give(sh.kv_empty[sv], mine);
      if (more) {
        if (mine) scores(kSplit<D> ? 1 : 0, sk);
        give(sh.kv_empty[sk], mine);
      }
      if (both && i > 0) {
        if ((threadIdx.x & 31) == 0) mbar_arrive(smem_u32(&sh.turn[q ^ 1]));
        ++turns;
      }
      if (i + 2 == n) give(sh.q_empty, mine);
    }
    items += mine;
  }
}

// ------------------------------------------------------------------ softmax

// Bits [0, n) of a word, none for n <= 0 and all for n >= 32.
__device__ __forceinline__ uint32_t below(int n) { return n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1; }

// Non-finite V elements of the piece's partly seen tiles, added to a row's
// columns [d0, d0 + 32) for the keys that the row sees.  Slow, and only where
// such values are.
template <bool F16>
__device__ __noinline__ void add_nonfinite(const PreArgs& a, const Walk& w, int n, int pos, int d0, uint32_t (&o)[32]) {
  const Visible v = visible_keys(pos, a.window, a.sinks);
  for (int i = 0; i < n; ++i) {
    const int j0 = w.it.key0(w.tile + i);
    if (!w.it.partial(a, j0)) continue;
    for (int j = j0; j < min(j0 + kTile, min(pos, w.s.len - 1) + 1); ++j) {
      if (j >= v.sink_end && j < v.win_begin) continue;
      const int64_t off = kv_row_offset(a.c, a.s.table + w.s.row * a.s.table_stride, j, &g_attn_prefill_status);
      if (off < 0) continue;
      const uint16_t* vr = a.c.v + off + (int64_t)w.h * a.c.head_stride + d0;
#pragma unroll
      for (int d = 0; d < 32; ++d) {
        const float f = elem_to_f32<F16>(vr[d]);
        if (!(fabsf(f) <= 3.4e38f)) o[d] = __float_as_uint(__uint_as_float(o[d]) + f);
      }
    }
  }
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// Two fp32 values in a 64-bit register, for the packed instructions.
__device__ __forceinline__ uint64_t pack2(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& x, float& y) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Largest of scores [j, j + 16) of a row, into two running maxima.
template <int X>
__device__ __forceinline__ void max16(const uint32_t (&s)[X][32], int j, float (&mx)[2]) {
#pragma unroll
  for (int e = 0; e < 16; e += 2)
    mx[(e >> 1) & 1] = max3(mx[(e >> 1) & 1], __uint_as_float(s[(j + e) >> 5][(j + e) & 31]),
                            __uint_as_float(s[(j + e) >> 5][(j + e + 1) & 31]));
}
// P = 2^(c s - z) of scores [j0, j0 + 64) of a row into tensor memory (rounded
// for the product only); returns the sum of the unrounded values.  Sixteen
// scores at a time, the exponentials of the next sixteen under way while these
// are packed: left to itself the code waits out the exponential's latency each
// time (1392 against 894 clocks for 128 scores, one warp a scheduler).  With
// MAX the largest of the 64 scores after these is found beside them.
template <bool F16, int j0, bool MAX, int X>
__device__ __forceinline__ float softmax64(uint32_t (&s)[X][32], uint32_t tp, float c, float z, float& top) {
  constexpr int kStep = 16;
  const uint64_t c2 = pack2(c, c), z2 = pack2(-z, -z);
  uint64_t t2[2] = {0, 0};
  float mx[2] = {-INFINITY, -INFINITY};
  auto take = [&](int x) {
#pragma unroll
    for (int e = 0; e < kStep; e += 2) {
      const int j = j0 + kStep * x + e;
      float y0, y1;
      unpack2(fma2(pack2(__uint_as_float(s[j >> 5][j & 31]), __uint_as_float(s[j >> 5][(j & 31) + 1])), c2, z2), y0, y1);
      s[j >> 5][j & 31] = __float_as_uint(ex2(y0));
      s[j >> 5][(j & 31) + 1] = __float_as_uint(ex2(y1));
    }
    if (MAX) max16(s, j0 + kHalf + kStep * x, mx);
  };
  auto put = [&](int x) {
    uint32_t p[kStep / 2];
#pragma unroll
    for (int e = 0; e < kStep; e += 2) {
      const int j = j0 + kStep * x + e;
      const float y0 = __uint_as_float(s[j >> 5][j & 31]), y1 = __uint_as_float(s[j >> 5][(j & 31) + 1]);
      t2[(e >> 1) & 1] = add2(t2[(e >> 1) & 1], pack2(y0, y1));
      p[e / 2] = pack_elem2<F16>(y0, y1);
    }
    tmem_st_8cols(tp + kStep / 2 * x, p);
  };
  take(0);
#pragma unroll
  for (int x = 1; x < kHalf / kStep; ++x) {
    take(x);
    put(x - 1);
  }
  put(kHalf / kStep - 1);
  if (MAX) top = fmaxf(mx[0], mx[1]);
  float u, v;
  unpack2(add2(t2[0], t2[1]), u, v);
  return u + v;
}

// A stage of the transposition of 8 x 8 pieces of 16 bytes over eight lanes.
template <int S>
__device__ __forceinline__ void transpose8(uint32_t (&v)[32], int lane) {
  const bool up = lane & S;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (i & S) continue;
#pragma unroll
    for (int y = 0; y < 4; ++y) {
      uint32_t &lo = v[4 * i + y], &hi = v[4 * (i + S) + y];
      const uint32_t got = __shfl_xor_sync(~0u, up ? lo : hi, S);
      if (up) lo = got;
      else hi = got;
    }
  }
}

template <int D, bool F16>
__device__ __forceinline__ void softmax_role(const PreArgs& a, Shared& sh, int q) {
  const int lane = threadIdx.x & 31, wq = (threadIdx.x >> 5) & 3;
  const uint32_t lane_base = (uint32_t)(wq * 32) << 16;
  const uint32_t ts = sh.tmem + lane_base + kColS + q * kTile, to = sh.tmem + lane_base + kColO + q * kTile;
  const int r = q * kTile + wq * 32 + lane;          // this thread's row of the item
  Walk w(a, sh.start);
  uint32_t seen = 0;                                 // S tiles taken so far
  bool first_item = true;
  for (int piece = 0; w.n > 0; ++piece, w.next(a)) {
    const int n = w.n;
    const bool from_before = first_item && w.tile > 0;
    first_item = false;
    if (q * kTile >= w.it.rows) continue;            // no row of this tile
    const int rr = w.t * kRows + min(r, w.it.rows - 1), tok = (int)a.by_group.div(rr), head = rr - tok * a.group;
    const int pos = w.s.len - w.s.fresh + tok;
    const int win = a.window > 0 ? pos - a.window + 1 : 0;     // keys from here on, and the sinks
    const int low_pos = __reduce_min_sync(~0u, pos), high_win = __reduce_max_sync(~0u, win);
    const int high_pos = __reduce_max_sync(~0u, pos), low_win = __reduce_min_sync(~0u, win);
    float m = -INFINITY, l = 0.0f;
    // The keys are taken 64 at a time (twice a tile).  before(): O and l follow
    // the maximum where it grew too far; `filled`: O holds products, the last of
    // which arrives on `bar`.
    const auto before = [&](float top, bool filled, const uint64_t& bar, uint32_t parity) {
      top *= a.scale_log2;
      if (!__any_sync(~0u, top > m + kSlack<F16>)) return true;
      const float mn = fmaxf(m, top);
      const float f = mn == -INFINITY ? 1.0f : ex2(m - mn);
      m = mn;
      l *= f;
      if (!filled) return true;
      if (!wait(sh, bar, parity, a.wait_ns)) return false;
      tc_fence_after();
#pragma unroll 1
      for (int x = 0; x < D; x += 16) {
        uint32_t o[16];
        tmem_ld_16cols(to + x, o);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
        tmem_st_16cols(to + x, o);
      }
      return true;
    };
    const auto hand_over = [&](const uint64_t& bar) {
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bar));
    };
    // Scores of hidden keys become -inf: s holds those of `count` words of keys from j0.
    const auto hide = [&](auto& s, int j0, int words) {
      if (j0 + 32 * words - 1 <= low_pos && (j0 >= high_win || j0 + 32 * words <= a.sinks)) return;
      const int hi = pos - j0, lo = win - j0, sk = a.sinks - j0;
#pragma unroll
      for (int x = 0; x < words; ++x) {
        const uint32_t vis = below(hi + 1 - 32 * x) & (~below(lo - 32 * x) | below(sk - 32 * x));
#pragma unroll
        for (int e = 0; e < 32; ++e)
          if (!(vis >> e & 1)) s[x][e] = 0xff800000u;
      }
    };
    const auto base_of = [&] { return m == -INFINITY ? 0.0f : m - kLift<F16>; };
    float top;
    if constexpr (kSplit<D>) {
      // Each half has its own scores: while one is worked on, the tensor cores
      // prepare the other's next.
#pragma unroll 1
      for (int step = 0; step < 2 * n; ++step) {
        const int half = step & 1;
        const int j0 = w.it.key0(w.tile + (step >> 1)) + half * kHalf;
        if (!wait(sh, sh.s_full[q][half], seen & 1, a.wait_ns)) return;
        tc_fence_after();
        if (j0 > high_pos || (j0 + kHalf <= low_win && j0 >= a.sinks)) {   // no row of the warp sees any
          const uint32_t zero[32] = {};
          tmem_st_32cols(ts + half * kHalf, zero);
          hand_over(sh.p_full[q][half]);
          seen += half;
          continue;
        }
        uint32_t s[2][32];
#pragma unroll
        for (int x = 0; x < 2; ++x) tmem_ld_32cols(ts + half * kHalf + 32 * x, s[x]);
        tmem_ld_wait();
        hide(s, j0, 2);
        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int j = 0; j < kHalf; j += 16) max16(s, j, mx);
        if (!before(fmaxf(mx[0], mx[1]), step > 0, sh.pv_done[q][half ^ 1], (half ? seen : seen - 1) & 1)) return;
        l += softmax64<F16, 0, false>(s, ts + half * kHalf, a.scale_log2, base_of(), top);
        hand_over(sh.p_full[q][half]);
        seen += half;                                // tiles finished
      }
    } else {
      // The halves' scores come together (one row of MMAs), and the second
      // half's maximum is found beside the first one's exponentials.
#pragma unroll 1
      for (int i = 0; i < n; ++i) {
        if (!wait(sh, sh.s_full[q][0], seen & 1, a.wait_ns)) return;
        tc_fence_after();
        uint32_t s[4][32];
#pragma unroll
        for (int x = 0; x < 4; ++x) tmem_ld_32cols(ts + 32 * x, s[x]);
        tmem_ld_wait();
        hide(s, w.it.key0(w.tile + i), 4);
        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int j = 0; j < kHalf; j += 16) max16(s, j, mx);
        if (!before(fmaxf(mx[0], mx[1]), i > 0, sh.pv_done[q][1], (seen - 1) & 1)) return;
        l += softmax64<F16, 0, true>(s, ts, a.scale_log2, base_of(), top);
        hand_over(sh.p_full[q][0]);
        if (!before(top, true, sh.pv_done[q][0], seen & 1)) return;
        l += softmax64<F16, kHalf, false>(s, ts + kHalf / 2, a.scale_log2, base_of(), top);
        hand_over(sh.p_full[q][1]);
        ++seen;
      }
    }
    // ---- the piece's rows
    if (!wait(sh, sh.pv_done[q][1], (seen - 1) & 1, a.wait_ns)) return;
    tc_fence_after();
    // (marks only grow, and a later piece's mark costs a needless look at the cache at most)
    const bool bad = *reinterpret_cast<volatile int*>(&sh.bad[piece & 7]) > piece;
    const bool whole = w.tile == 0 && n == w.it.n, mine = r < w.it.rows;
    SPEAR_CHECK(&g_attn_prefill_status, !mine || (w.s.tok0 + tok < a.tokens && w.h * a.group + head < a.q_heads));
    SPEAR_CHECK(&g_attn_prefill_status, whole || (!from_before ? w.tile == 0 : piece == 0));
    const int64_t row = (int64_t)(w.s.tok0 + tok) * a.q_heads + w.h * a.group + head;
    float* part = a.parts + (2 * (int64_t)blockIdx.x + (from_before ? 0 : 1)) * part_floats(D);
    const float inv = pos < 0 ? 0.0f : 1.0f / l;
    const int64_t dst = mine ? row : -1;
#pragma unroll 1
    for (int x = 0; x < D; x += 64) {
      uint32_t v[32];                                // the row's 64 columns, rounded
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        uint32_t o[32];
        tmem_ld_32cols(to + x + 32 * y, o);
        tmem_ld_wait();
        if (bad && mine) {                           // (in a copy: o itself stays in registers)
          uint32_t t[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) t[e] = o[e];
          add_nonfinite<F16>(a, w, n, pos, x + 32 * y, t);
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = t[e];
        }
        __syncwarp();                                // tensor memory is read by whole warps
#pragma unroll
        for (int e = 0; e < 16; ++e)
          v[16 * y + e] = pack_elem2<F16>(__uint_as_float(o[2 * e]) * inv, __uint_as_float(o[2 * e + 1]) * inv);
        if (!whole && mine) {
          uint4* pp = reinterpret_cast<uint4*>(part) + (x / 4 + 8 * y) * kRows + r;
#pragma unroll
          for (int e = 0; e < 8; ++e) pp[e * kRows] = make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
        }
      }
      if (whole) {
        // eight lanes trade 16-byte pieces, so that they write 128 bytes of one row at a time
        transpose8<4>(v, lane);
        transpose8<2>(v, lane);
        transpose8<1>(v, lane);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int64_t to_row = __shfl_sync(~0u, dst, (lane & 24) + e);
          if (to_row >= 0)
            reinterpret_cast<uint4*>(a.out + to_row * D + x)[lane & 7] = make_uint4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
        }
      }
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&sh.o_free[q]));
    if (mine) {
      if (!whole) {
        part[(int64_t)kRows * D + r] = m;
        part[(int64_t)kRows * (D + 1) + r] = l;
      } else if (a.lse) {
        a.lse[row] = pos < 0 ? -INFINITY : (m + log2_sum<F16>(l)) * kLn2;
      }
    }
  }
}

template <int D, bool F16, bool TMA>
__global__ void __launch_bounds__(kThreads, 1) attn_prefill_kernel(const __grid_constant__ PreArgs a,
                                                                  const __grid_constant__ PreMaps maps) {
  using L = Layout<D>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Shared sh;
  uint8_t* base = smem_align_up(smem_raw, 1024);
  const uint32_t smem = smem_u32(base);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  // ---- what does not depend on the kernels before this one
  if (tid == 0) {
    for (int i = 0; i < L::kSlots; ++i) {
      mbar_init(smem_u32(&sh.kv_full[i]), kLoadThreads);
      mbar_init(smem_u32(&sh.kv_empty[i]), 2);
      mbar_init(smem_u32(&sh.landed[i]), 1);
    }
    mbar_init(smem_u32(&sh.q_full), kLoadThreads);
    mbar_init(smem_u32(&sh.q_empty), 2);
    for (int q = 0; q < 2; ++q) {
      mbar_init(smem_u32(&sh.turn[q]), 1);
      mbar_init(smem_u32(&sh.drained[q]), 1);
    }
    for (int q = 0; q < 2; ++q) {
      for (int half = 0; half < 2; ++half) {
        mbar_init(smem_u32(&sh.s_full[q][half]), 1);
        mbar_init(smem_u32(&sh.p_full[q][half]), 4);
        mbar_init(smem_u32(&sh.pv_done[q][half]), 1);
      }
      mbar_init(smem_u32(&sh.o_free[q]), 4);
    }
    sh.abort = 0;
    for (int i = 0; i < 8; ++i) sh.bad[i] = 0;
    fence_mbar_init();
    if (TMA) {
      prefetch_tmap(&maps.k);
      prefetch_tmap(&maps.v);
      if (a.q_tma) prefetch_tmap(&maps.q);
    }
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(&sh.tmem), kTmemCols);
    tmem_relinquish();
  }
  enter();

  // ---- units of all sequences, and this block's range of them (in the ring's
  // space, before it is used)
  unsigned long long* pre = reinterpret_cast<unsigned long long*>(base + L::kRing);   // [kGroups]
  Seq* kept = reinterpret_cast<Seq*>(pre + kGroups);                                  // [kKept]
  const int per = (a.s.n + kGroups - 1) / kGroups, groups = (a.s.n + per - 1) / per;
  for (int i = tid; i < groups; i += kThreads) pre[i] = 0;
  for (int b = tid; b < min(a.s.n, kKept); b += kThreads) kept[b].open(a, b);
  __syncthreads();
  const auto seq_of = [&](int b) {
    if (b < kKept) return kept[b];
    Seq s;
    s.open(a, b);
    return s;
  };
  for (int b = warp; b < a.s.n; b += kThreads / 32) {
    const long long u = seq_units(a, seq_of(b)) * a.c.heads;
    if (lane == 0) atomicAdd(&pre[b / per], (unsigned long long)u);
  }
  __syncthreads();
  if (warp == 0) {
    unsigned long long carry = 0;                   // exclusive prefix in place
    for (int i0 = 0; i0 < groups; i0 += 32) {
      const unsigned long long v = i0 + lane < groups ? pre[i0 + lane] : 0;
      unsigned long long x = v;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const unsigned long long y = __shfl_up_sync(~0u, x, d);
        if (lane >= d) x += y;
      }
      if (i0 + lane < groups) pre[i0 + lane] = carry + x - v;
      carry += __shfl_sync(~0u, x, 31);
    }
    const long long U = (long long)carry, C = min((long long)gridDim.x, U);
    const long long c = blockIdx.x;
    const long long u0 = c < C ? divide(c * U, C) : 0, u1 = c < C ? divide((c + 1) * U, C) : 0;
    __syncwarp();
    Start st{};
    st.units = u1 - u0;
    int4 j0 = make_int4(0, 0, 0, 0), j1 = j0;
    if (u1 > u0) {
      int lo = 0, hi = groups;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if ((long long)pre[mid] <= u0) lo = mid; else hi = mid;
      }
      long long at = (long long)pre[lo];
      st.s = seq_of(lo * per);
      long long su = seq_units(a, st.s);
      while (at + su * a.c.heads <= u0) {
        at += su * a.c.heads;
        st.s = seq_of(st.s.b + 1);
        su = seq_units(a, st.s);
      }
      st.h = (int)divide(u0 - at, su);
      long long left = u0 - at - st.h * su;         // into the head's units
      Item it;
      for (int t0 = 0;; t0 += 32) {
        int units = 0;
        if (t0 + lane < st.s.tiles(a)) {
          it.open(a, st.s, t0 + lane);
          units = it.n + kSetup;
        }
        long long x = units;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const long long y = __shfl_up_sync(~0u, x, d);
          if (lane >= d) x += y;
        }
        const unsigned past = __ballot_sync(~0u, x > left);
        if (past) {
          const int f = __ffs(past) - 1;
          st.t = t0 + f;
          st.unit = (int)(left - __shfl_sync(~0u, x - units, f));
          break;
        }
        left -= __shfl_sync(~0u, x, 31);
      }
      // an item of which an earlier block has tiles and that ends here is joined under this block's number
      it.open(a, st.s, st.t);
      if (st.unit > kSetup && it.n + kSetup - st.unit <= st.units) {
        j0 = make_int4(1, st.s.b, st.h, st.t);
        j1 = make_int4((int)divide((u0 - st.unit + kSetup + 1) * C - 1, U), it.rows, st.s.tok0, st.s.len - st.s.fresh);
      }
    }
    if (lane == 0) {
      sh.start = st;
      a.joins[2 * blockIdx.x] = j0;
      a.joins[2 * blockIdx.x + 1] = j1;
    }
  }
  fence_proxy_async_smem();                          // the ring's space was ours until here
  __syncthreads();
  if (warp < 8) {
    if constexpr (!kSplit<D>) reg_inc<184>();      // a thread holds 128 scores: 2 x 128 x 184 + 2 x 128 x 72 = 512 x 128
    tc_fence_after();
    softmax_role<D, F16>(a, sh, warp >> 2);
  } else {
    if constexpr (!kSplit<D>) reg_dec<72>();
    tc_fence_after();
    if (warp == kMmaWarp || warp == kMmaWarp1) {
      const int q = warp == kMmaWarp1;
      mma_role<D, F16, TMA>(a, sh, smem, q);
      // what was issued has finished, its arrivals included, before the block
      // and its tensor memory go
      mma_commit_warp(smem_u32(&sh.drained[q]));
      if (!mbar_wait(smem_u32(&sh.drained[q]), 0, kLandNs)) give_up(sh);
      __syncwarp();
    } else if (warp >= kLoadWarp) {
      Loader<D, F16> ld{a, sh, smem, warp - kLoadWarp, lane};
      if constexpr (TMA) ld.run_beside_tma();
      else ld.run();
    } else if (warp == kTmaWarp) {
      if constexpr (TMA) tma_role<D>(a, maps, sh, smem);
    } else if (warp == kQWarp && a.q_tma) {
      q_role<D>(a, maps, sh, smem);
    }
  }
  __syncthreads();
  if (warp == kMmaWarp) tmem_dealloc(sh.tmem, kTmemCols);
}

// The items that blocks share: block (c, y) adds rows 8 y .. of the item that
// ends in block c's range.  Bound by latency (7 us after three short chunks);
// 64 rows a block: 27.1 against 25.8 us for both kernels.
constexpr int kJoinRows = 8;
template <int D, bool F16>
__global__ void __launch_bounds__(kJoinRows * D / 4) attn_prefill_join_kernel(const __grid_constant__ PreArgs a) {
  enter();
  const int c = blockIdx.x;
  const int4 j0 = a.joins[2 * c], j1 = a.joins[2 * c + 1];
  const int r = blockIdx.y * kJoinRows + threadIdx.x % kJoinRows, x = threadIdx.x / kJoinRows;
  if (!j0.x || r >= j1.y) return;
  float mx = -INFINITY, l = 0.0f;
  float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int p = j1.x; p <= c; ++p) {
    SPEAR_CHECK(&g_attn_prefill_status, p >= 0 && p < (int)gridDim.x);
    const float* part = a.parts + (2 * (int64_t)p + (p == j1.x)) * part_floats(D);
    mx = fmaxf(mx, part[(int64_t)kRows * D + r]);
  }
  const float z = mx == -INFINITY ? 0.0f : mx;
#pragma unroll 4
  for (int p = j1.x; p <= c; ++p) {
    const float* part = a.parts + (2 * (int64_t)p + (p == j1.x)) * part_floats(D);
    const float f = ex2(part[(int64_t)kRows * D + r] - z);
    const float4 v = reinterpret_cast<const float4*>(part)[x * kRows + r];
    l += f * part[(int64_t)kRows * (D + 1) + r];
    o.x += f * v.x;
    o.y += f * v.y;
    o.z += f * v.z;
    o.w += f * v.w;
  }
  const int rr = j0.w * kRows + r, tok = (int)a.by_group.div(rr), pos = j1.w + tok;
  const int64_t row = (int64_t)(j1.z + tok) * a.q_heads + j0.z * a.group + (rr - tok * a.group);
  const float inv = pos < 0 ? 0.0f : 1.0f / l;
  *reinterpret_cast<uint2*>(a.out + row * D + 4 * x) =
      make_uint2(pack_elem2<F16>(o.x * inv, o.y * inv), pack_elem2<F16>(o.z * inv, o.w * inv));
  if (a.lse && x == 0) a.lse[row] = pos < 0 ? -INFINITY : (mx + log2_sum<F16>(l)) * kLn2;
}

int encode(CUtensorMap* m, const spear_kv_cache& c, const uint16_t* base, int rank, const cuuint64_t* dims,
           const int64_t* stride, const cuuint32_t* box) {
  EncodeTiledFn fn = encode_tiled_fn();
  if (!fn) return fail(SPEAR_ERR_CUDA, "cuTensorMapEncodeTiled is unavailable");
  cuuint64_t bytes[3];                               // the stride of an extent of one is not used, but has to be valid
  for (int i = 0; i + 1 < rank; ++i) bytes[i] = (cuuint64_t)std::max<int64_t>(stride[i], 8) * 2;
  const cuuint32_t ones[4] = {1, 1, 1, 1};
  const CUresult r = fn(m, c.dtype == SPEAR_DT_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                        rank, const_cast<uint16_t*>(base), dims, bytes, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? SPEAR_OK : fail(SPEAR_ERR_CUDA, "tensor map encode failed (%d)", (int)r);
}
// One pool as [pages][heads][slots][d], in boxes of one panel of `box` slots.
int pool_map(CUtensorMap* m, const spear_kv_cache& c, const uint16_t* base, int box) {
  const cuuint64_t dims[4] = {(cuuint64_t)c.head_dim, (cuuint64_t)c.page_size, (cuuint64_t)c.num_kv_heads,
                              (cuuint64_t)c.num_pages};
  const int64_t strides[3] = {c.slot_stride, c.head_stride, c.page_stride};
  const cuuint32_t boxes[4] = {64, (cuuint32_t)box, 1, 1};
  return encode(m, c, base, 4, dims, strides, boxes);
}
bool q_boxes(const spear_attn& a, int group, int tokens) {
  return kTile % group == 0 && (a.q_head_stride > 0 || a.num_q_heads == 1) && (a.q_token_stride > 0 || tokens == 1) &&
         std::max(a.q_head_stride, a.q_token_stride) < 1ll << 38;
}

// Slots of a TMA box: the largest power of two that divides the page size, 128
// at most, so that the 128 keys of a tile are whole boxes and a box lies in one
// page.  0: the pages are gathered row by row, which takes the same time for
// every page size.  One prompt of 8192 tokens, heads of 128: 414 us with boxes
// of 64, 410 of 32, 452 of 16, 685 of 8, and 436 gathered.  So boxes of 16 or
// more; of 16 only for heads of 64 (147 against 153 us gathered, two prompts of
// 3000 to 4096) and for sequences of few rows a K/V head (33 ragged chunks of
// up to 1024 rows 540 against 581, three short ones 25.2 against 26.3), not for
// those of many (4096 over 32000 keys 427 against 384, over 2000 268 against
// 260).  The host knows the batch's average only, so the rule loses where a
// batch of very ragged sequences is above it: 33 of up to 8192 rows take 870
// gathered and would take 826 in boxes.
int box_slots(const spear_kv_cache& c, long long rows) {
  if ((c.slot_stride <= 0 && c.page_size > 1) || (c.head_stride <= 0 && c.num_kv_heads > 1) ||
      (c.page_stride <= 0 && c.num_pages > 1) || std::max({c.slot_stride, c.head_stride, c.page_stride}) >= 1ll << 38)
    return 0;
  const int box = std::min(kTile, c.page_size & -c.page_size);
  return box > 16 || (box == 16 && (c.head_dim == 64 || rows < 2048)) ? box : 0;
}

template <int D, bool F16, bool TMA>
int launch_main(const PreArgs& a, const PreMaps& maps, int blocks, cudaStream_t st) {
  const void* fn = reinterpret_cast<const void*>(&attn_prefill_kernel<D, F16, TMA>);
  const size_t bytes = Layout<D>::kTotal + 1024;
  if (int rc = ensure_smem_limit(fn, bytes)) return rc;
  return launch_dependent(attn_prefill_kernel<D, F16, TMA>, dim3(blocks), kThreads, bytes, st, "attn_prefill launch", a,
                          maps);
}
template <int D, bool F16>
int launch(const PreArgs& a, const PreMaps& maps, int blocks, cudaStream_t st) {
  if (int rc = a.tma ? launch_main<D, F16, true>(a, maps, blocks, st) : launch_main<D, F16, false>(a, maps, blocks, st))
    return rc;
  const int rows = (int)std::min<long long>(kRows, (long long)a.tokens * a.group);   // of the largest item at most
  return launch_dependent(attn_prefill_join_kernel<D, F16>, dim3(blocks, (rows + kJoinRows - 1) / kJoinRows), kJoinRows * D / 4, 0, st,
                          "attn_prefill join launch", a);
}
}  // namespace

int attn_prefill_workspace_bytes(const spear_kv_cache& c, int nseqs, int tokens, int q_heads, size_t* bytes) {
  DeviceInfo di;
  if (int rc = device_info(&di)) return rc;
  *bytes = (size_t)di.num_sms * 2 * (sizeof(int4) + part_floats(c.head_dim) * sizeof(float));
  return SPEAR_OK;
}

int launch_attn_prefill(const spear_kv_cache& c, const spear_kv_seqs& s, const int32_t* starts, int tokens,
                        const spear_attn& at, void* ws, size_t ws_bytes, cudaStream_t st) {
  DeviceInfo di;
  if (int rc = device_info(&di)) return rc;
  size_t need = 0;
  if (int rc = attn_prefill_workspace_bytes(c, s.num_seqs, tokens, at.num_q_heads, &need)) return rc;
  if (!ws || ws_bytes < need || (reinterpret_cast<uintptr_t>(ws) & 15))
    return fail(SPEAR_ERR_WORKSPACE, "attn_prefill workspace needs %zu bytes, 16-byte aligned, got %zu", need, ws_bytes);
  const int group = at.num_q_heads / c.num_kv_heads;
  if ((long long)tokens * group > (1 << 30))
    return fail(SPEAR_ERR_UNSUPPORTED, "%d tokens of %d heads are too many for one call", tokens, at.num_q_heads);
  char* p = static_cast<char*>(ws);
  PreArgs a{kv_view(c), seq_view(s), at.q, at.q_token_stride, at.q_head_stride, starts, tokens, at.num_q_heads,
                  group, FastDiv::of((uint32_t)group), at.window, at.sinks, at.scale * kLog2e, at.out, at.lse, reinterpret_cast<int4*>(p),
                  reinterpret_cast<float*>(p + (size_t)di.num_sms * 2 * sizeof(int4)),
                  wait_limit_ns(2000000000ull), box_slots(c, (long long)tokens * group / s.num_seqs), 0};
  PreMaps maps{};
  if (a.tma) {
    if (int rc = pool_map(&maps.k, c, c.k, a.tma)) return rc;
    if (int rc = pool_map(&maps.v, c, c.v, a.tma)) return rc;
    a.q_tma = q_boxes(at, group, tokens);
    if (a.q_tma) {
      const cuuint64_t dims[3] = {(cuuint64_t)c.head_dim, (cuuint64_t)at.num_q_heads, (cuuint64_t)tokens};
      const int64_t strides[2] = {at.q_head_stride, at.q_token_stride};
      const cuuint32_t box[3] = {64, (cuuint32_t)group, (cuuint32_t)(kTile / group)};
      if (int rc = encode(&maps.q, c, at.q, 3, dims, strides, box)) return rc;
    }
  }
  const bool f16 = c.dtype == SPEAR_DT_F16;
  if (c.head_dim == 64) return f16 ? launch<64, true>(a, maps, di.num_sms, st) : launch<64, false>(a, maps, di.num_sms, st);
  return f16 ? launch<128, true>(a, maps, di.num_sms, st) : launch<128, false>(a, maps, di.num_sms, st);
}

int status_word_attn_prefill(unsigned** word) {
  return cuda_check(cudaGetSymbolAddress(reinterpret_cast<void**>(word), g_attn_prefill_status), "attn_prefill status address");
}

}  // namespace spear
