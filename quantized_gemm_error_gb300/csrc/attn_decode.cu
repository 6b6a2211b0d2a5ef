// attn_decode.cu -- attention of one new token of each sequence over the
// paged cache, in one launch.
//
// With s_j = scale q . k_j over the visible keys, a running maximum m and
// sum l give out = sum_j 2^(c s_j - m) v_j / l in one pass over K and V; two
// ranges of keys join as m = max(m1, m2), l = l1 2^(m1 - m) + l2 2^(m2 - m),
// and o alike.  Bound by the bytes of K and V: 64 sequences of up to 8192 keys,
// 64 heads on 8 of 128 (1.15 GB) 186 us, 6.2 TB/s; four of 131 k keys (2.1 GB)
// 317 us, 6.7 TB/s; one of 777 keys 8.9 us, of which the launch, the reads that
// depend on one another (length, page, keys) and the joining take all but 2.
//
// Split.  A unit is 16 visible keys of one item (sequence, K/V head, up to 16
// of its query heads).  All units of the batch, in order, are dealt to the
// warps of the grid in equal consecutive ranges, so a long row is spread over
// the GPU and many short rows share a warp, whatever the lengths, which only
// the device knows.  A warp streams its units through a ring of its own
// (cp.async, no block barrier); the units' addresses come from the block
// table one step ahead.  An item inside one warp's range is finished by that
// warp; pieces of an item in several warps meet in shared memory, those in
// several blocks in the workspace, where the last block to arrive adds them
// in order (a ticket for each such item), so results do not depend on timing.
//
// A unit's products run on mma.sync with the keys as the 16-row operand and
// the query heads as the 8-column one: S^T = K Q^T, then O^T += V^T P, with
// P^T turned in registers (movmatrix).  One or two 8-head tiles; at 8 heads a
// byte of cache costs 8 multiply-adds, far from the tensor cores' limit, so
// the warp-level form serves.
#include <algorithm>

#include "kv.cuh"

namespace spear {

namespace {
__device__ unsigned g_attn_decode_status;

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kUnit = 16;                           // keys of a unit
constexpr int kGroups = 2048;                       // entries of the prefix over sequences
constexpr int kKept = 1024;                         // sequences whose rows and lengths are kept in shared memory
constexpr int kRingBytes = 192 * 1024;
constexpr int kMaxHeads = 16;                       // query heads of an item
// P is taken times 2^kLift: in fp16 a probability is normal down to 2^-28 of
// its row's largest so (19 nats; unlifted 2^-14, and below 2^-25 it would be 0,
// which shows where the largest one's value is near 0, as a sink's is).  l and
// o carry the factor, so it cancels; lse takes it out of l.  bf16 has fp32's range.
template <bool F16>
constexpr float kLift = F16 ? 14.0f : 0.0f;
template <bool F16>
__device__ __forceinline__ float log2_sum(float l) { return log2f(l * (F16 ? 0x1p-14f : 1.0f)); }

struct DecArgs {
  KvView c;
  SeqView s;
  const uint16_t* q;
  int64_t qt, qh;
  uint16_t* out;
  float* lse;
  unsigned* tickets;                                // [blocks]
  float* parts;                                     // [2 blocks][part_floats(D)]: m, l, o of a block's pieces
  float* heads;                                     // [blocks kWarps][kMaxHeads][D + 4]: o of a warp's first piece
  int q_heads, group, chunks;                       // chunks: items a K/V head
  int window, sinks;
  float scale_log2;
};

__host__ __device__ constexpr int part_floats(int D) { return kMaxHeads * (D + 2); }

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
// Transposes the 8 x 8 matrix of 16-bit values that the warp holds (lane 4 i + j: row i, columns 2 j, 2 j + 1).
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
template <bool F16>
__device__ __forceinline__ void mma16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (F16) mma_f16_16816(d, a[0], a[1], a[2], a[3], b0, b1);
  else mma_bf16_16816(d, a[0], a[1], a[2], a[3], b0, b1);
}

// A position in the flat order of units: sequence b (row, visible keys), item
// hc of it, unit `chunk` of that item.
struct Cursor {
  int b, row, hc, chunk, units, keys, sink_end, gap;

  __device__ __forceinline__ int2 open(const DecArgs& a, int b_) {
    const int r = seq_row(a.s, b_, &g_attn_decode_status);
    const int2 at = make_int2(r, seq_len(a.s, a.c, r, &g_attn_decode_status));
    open_at(a, b_, at);
    return at;
  }
  // The same with the row and length that open() found before.
  __device__ __forceinline__ void open_at(const DecArgs& a, int b_, int2 at) {
    b = b_;
    row = at.x;
    const int len = at.y;
    const Visible v = visible_keys(len - 1, a.window, a.sinks);
    sink_end = v.sink_end;
    gap = v.win_begin - v.sink_end;
    keys = len - gap;
    units = (keys + kUnit - 1) / kUnit;
  }
  // Moves on by one unit (there is another one).
  __device__ __forceinline__ void next(const DecArgs& a, int items) {
    if (++chunk < units) return;
    chunk = 0;
    if (++hc < items) return;
    hc = 0;
    do open(a, b + 1); while (units == 0);
  }
};

// Inclusive prefix sum over the warp.
__device__ __forceinline__ long long warp_scan(long long v, int lane) {
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long y = __shfl_up_sync(~0u, v, d);
    if (lane >= d) v += y;
  }
  return v;
}
// Another range's maximum, sum and four elements, added to a row's.
struct Row {
  float m = -INFINITY, l = 0.0f;
  float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  __device__ __forceinline__ void join(float om, float ol, float4 v) {
    const float mn = fmaxf(m, om), z = mn == -INFINITY ? 0.0f : mn, f = ex2(m - z), g = ex2(om - z);
    m = mn;
    l = f * l + g * ol;
    o = make_float4(f * o.x + g * v.x, f * o.y + g * v.y, f * o.z + g * v.z, f * o.w + g * v.w);
  }
};
// Four elements of a finished row of out.
template <bool F16>
__device__ __forceinline__ void store_row(const DecArgs& a, int64_t row, int d, int D, float4 o, float m, float l) {
  const float i = 1.0f / l;
  *reinterpret_cast<uint2*>(a.out + row * D + d) =
      make_uint2(pack_elem2<F16>(o.x * i, o.y * i), pack_elem2<F16>(o.z * i, o.w * i));
  if (a.lse && d == 0) a.lse[row] = (m + log2_sum<F16>(l)) * kLn2;
}
// A sequence that sees no key: zeros.
template <int D>
__device__ __noinline__ void write_empty(const DecArgs& a, int b) {
  uint4* o = reinterpret_cast<uint4*>(a.out + (int64_t)b * a.q_heads * D);
  for (int x = 0; x < a.q_heads * (D / 8); ++x) o[x] = make_uint4(0, 0, 0, 0);
  if (a.lse)
    for (int h = 0; h < a.q_heads; ++h) a.lse[(int64_t)b * a.q_heads + h] = -INFINITY;
}

template <int D, bool F16, int NT>
__global__ void __launch_bounds__(kThreads, 1) attn_decode_kernel(const __grid_constant__ DecArgs a) {
  constexpr int kRowBytes = D * 2, kVecs = D / 8, kRowsPass = 32 / kVecs, kPasses = kUnit / kRowsPass;
  constexpr int kHalf = kUnit * kRowBytes, kStage = 2 * kHalf, kStages = kRingBytes / kWarps / kStage;
  constexpr int KS = D / 16, MT = D / 16, kPad = D + 4;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ long long s_prefix[kGroups];
  __shared__ int2 s_seq[kKept];
  __shared__ long long s_wsum[kWarps];
  __shared__ float s_m[2 * kWarps][kMaxHeads], s_l[2 * kWarps][kMaxHeads];
  __shared__ int s_item[2 * kWarps];                // item of a pending piece, -1: none
  __shared__ long long s_first[2 * kWarps];         // its item's first unit
  __shared__ int s_units[2 * kWarps];               // its item's units
  __shared__ int s_heads[2 * kWarps];               // and where its results go
  __shared__ int64_t s_row[2 * kWarps];
  __shared__ int s_last[2], s_from[2], s_to[2];

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, c2 = (lane & 3) * 2;
  const int items = a.c.heads * a.chunks;
  enter();
  const int per = (a.s.n + kGroups - 1) / kGroups, groups = (a.s.n + per - 1) / per;

  // ---- how the units are dealt.  Up to 32 sequences: every warp finds its
  // place by itself, without a barrier (one sequence of 777 keys: 8.9 against
  // 9.4 us); else a prefix over (groups of) sequences in shared memory.
  const bool few = a.s.n <= 32;
  long long U, at = 0;
  Cursor use;
  if (lane < 2) s_item[2 * warp + lane] = -1;
  if (few) {
    use.open(a, min(lane, a.s.n - 1));
    const long long mine = lane < a.s.n ? (long long)use.units * items : 0;
    if (warp == 0 && lane < a.s.n && use.units == 0 && lane % (int)gridDim.x == (int)blockIdx.x) write_empty<D>(a, lane);
    at = warp_scan(mine, lane);
    U = __shfl_sync(~0u, at, 31);
    at -= mine;
  } else {
    long long carry = 0;
    for (int g0 = 0; g0 < groups; g0 += kThreads) {
      const int gi = g0 + tid;
      long long mine = 0;
      if (gi < groups)
        for (int b = gi * per; b < min(a.s.n, (gi + 1) * per); ++b) {
          const int2 at = use.open(a, b);
          if (b < kKept) s_seq[b] = at;
          mine += (long long)use.units * items;
          if (use.units == 0 && b % (int)gridDim.x == (int)blockIdx.x) write_empty<D>(a, b);
        }
      const long long x = warp_scan(mine, lane);
      if (lane == 31) s_wsum[warp] = x;
      __syncthreads();
      long long before = carry + x - mine;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += s_wsum[w];
        carry += s_wsum[w];
      }
      if (gi < groups) s_prefix[gi] = before;
      __syncthreads();
    }
    U = carry;
  }
  const long long W = min((long long)gridDim.x * kWarps, U);         // warps with work
  if ((long long)blockIdx.x * kWarps >= W) return;
  const long long w = (long long)blockIdx.x * kWarps + warp;
  const long long u0 = w < W ? divide(w * U, W) : 0, u1 = w < W ? divide((w + 1) * U, W) : 0;
  const uint32_t ring = (uint32_t)__cvta_generic_to_shared(smem) + warp * kStages * kStage;

  if (u0 < u1) {
    // ---- where the range starts
    if (few) {
      const unsigned past = __ballot_sync(~0u, use.units > 0 && lane < a.s.n && at <= u0);
      const int src = 31 - __clz(past);
      at = __shfl_sync(~0u, at, src);
      use.b = src;
      use.row = __shfl_sync(~0u, use.row, src);
      use.units = __shfl_sync(~0u, use.units, src);
      use.keys = __shfl_sync(~0u, use.keys, src);
      use.sink_end = __shfl_sync(~0u, use.sink_end, src);
      use.gap = __shfl_sync(~0u, use.gap, src);
    } else {
      int lo = 0, hi = groups;                      // last group with prefix <= u0
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s_prefix[mid] <= u0) lo = mid; else hi = mid;
      }
      at = s_prefix[lo];
      const auto reopen = [&](int b) {
        if (b < kKept) use.open_at(a, b, s_seq[b]);
        else use.open(a, b);
      };
      reopen(lo * per);
      while (at + (long long)use.units * items <= u0) {
        at += (long long)use.units * items;
        reopen(use.b + 1);
      }
    }
    use.hc = (int)divide(u0 - at, use.units);
    use.chunk = (int)((u0 - at) - (long long)use.hc * use.units);
    Cursor load = use;
    const int total = (int)(u1 - u0);

    // The pages of two units, the one at `load` (lanes 0-15) and the next of
    // its item (lanes 16-31), read one step before they are used.
    int32_t page = 0;
    int slot = 0, half = 0;
    bool in = false;
    auto look_up = [&] {
      const int v = load.chunk * kUnit + lane;
      in = v < load.keys;
      if (in) {
        const int pos = v < load.sink_end ? v : v + load.gap;
        const uint32_t pg = a.c.page.div((uint32_t)pos);
        slot = pos - (int)(pg * a.c.page.d);
        page = a.s.table[load.row * a.s.table_stride + pg];
      }
    };
    int issued = 0;
    int64_t off = -1;
    auto issue = [&] {                               // copies of unit `issued`, then the next units' table entries
      if (issued < total) {
        if (half == 0) {
          off = -1;
          if (in) {
            if ((unsigned)page < (unsigned)a.c.num_pages)
              off = (int64_t)page * a.c.page_stride + (int64_t)slot * a.c.slot_stride +
                    (int64_t)(load.hc / a.chunks) * a.c.head_stride;
            else
              record_status(&g_attn_decode_status, DEV_ERR_INVALID);
          }
        }
        const uint32_t st = ring + (issued % kStages) * kStage;
        SPEAR_CHECK(&g_attn_decode_status, load.b < a.s.n && load.hc < items && load.chunk < load.units);
#pragma unroll
        for (int i = 0; i < kPasses; ++i) {
          const int r = i * kRowsPass + lane / kVecs, x = lane % kVecs;
          const int64_t o = __shfl_sync(~0u, off, half + r);
          const uint32_t dst = st + r * kRowBytes + ((x ^ (r & 7)) << 4);
          const int64_t e = o < 0 ? 0 : o + x * 8;
          cp_async16_zfill(dst, a.c.k + e, o >= 0);
          cp_async16_zfill(dst + kHalf, a.c.v + e, o >= 0);
        }
        if (++issued < total) {
          if (half == 0 && load.chunk + 1 < load.units) {
            half = kUnit;
            ++load.chunk;
          } else {
            half = 0;
            load.next(a, items);
            look_up();
          }
        }
      }
      cp_async_commit();
    };
    look_up();
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) issue();

    uint32_t qf[NT][KS][2];
    float o[NT][MT][4], m[NT][2], l[NT][2];
    long long first = 0;                             // first unit of the current item
    bool fresh = true;
    for (int i = 0; i < total; ++i) {
      if (fresh) {
        fresh = false;
        first = u0 + i - use.chunk;
        const int hq = use.hc / a.chunks * a.group + use.hc % a.chunks * kMaxHeads;
        const int heads = min(kMaxHeads, a.group - use.hc % a.chunks * kMaxHeads);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const uint16_t* qp = a.q + use.b * a.qt + (int64_t)(hq + n * 8 + g) * a.qh;
          const bool there = n * 8 + g < heads;
#pragma unroll
          for (int k = 0; k < KS; ++k) {
            qf[n][k][0] = there ? *reinterpret_cast<const uint32_t*>(qp + k * 16 + c2) : 0;
            qf[n][k][1] = there ? *reinterpret_cast<const uint32_t*>(qp + k * 16 + c2 + 8) : 0;
          }
#pragma unroll
          for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[n][t][e] = 0.0f;
          m[n][0] = m[n][1] = -INFINITY;
          l[n][0] = l[n][1] = 0.0f;
        }
      }
      cp_async_wait<kStages - 2>();
      __syncwarp();                                  // unit i is there, and every lane is done with unit i - 1
      issue();                                       // into the stage of unit i - 1
      const uint32_t st = ring + (i % kStages) * kStage;

      // S^T: keys x heads
      float s[NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[n][e] = 0.0f;
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        uint32_t kf[4];
        const int r = (lane & 7) + ((lane >> 3) & 1) * 8, x = 2 * k + (lane >> 4);
        ldsm4(kf, st + r * kRowBytes + ((x ^ (r & 7)) << 4));
#pragma unroll
        for (int n = 0; n < NT; ++n) mma16<F16>(s[n], kf, qf[n][k][0], qf[n][k][1]);
      }
      const int left = use.keys - use.chunk * kUnit;  // valid keys of the unit
      uint32_t pf[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float x[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = g + (e >> 1) * 8 < left ? s[n][e] * a.scale_log2 : -INFINITY;
        float m0 = fmaxf(x[0], x[2]), m1 = fmaxf(x[1], x[3]);
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) {
          m0 = fmaxf(m0, __shfl_xor_sync(~0u, m0, d));
          m1 = fmaxf(m1, __shfl_xor_sync(~0u, m1, d));
        }
        if (__any_sync(~0u, m0 > m[n][0] || m1 > m[n][1])) {
          const float n0 = fmaxf(m0, m[n][0]), n1 = fmaxf(m1, m[n][1]);
          const float f0 = n0 == -INFINITY ? 1.0f : ex2(m[n][0] - n0), f1 = n1 == -INFINITY ? 1.0f : ex2(m[n][1] - n1);
          m[n][0] = n0;
          m[n][1] = n1;
          l[n][0] *= f0;
          l[n][1] *= f1;
#pragma unroll
          for (int t = 0; t < MT; ++t) {
            o[n][t][0] *= f0;
            o[n][t][1] *= f1;
            o[n][t][2] *= f0;
            o[n][t][3] *= f1;
          }
        }
        const float z0 = m[n][0] == -INFINITY ? 0.0f : m[n][0] - kLift<F16>;
        const float z1 = m[n][1] == -INFINITY ? 0.0f : m[n][1] - kLift<F16>;
        const float p0 = ex2(x[0] - z0), p1 = ex2(x[1] - z1), p2 = ex2(x[2] - z0), p3 = ex2(x[3] - z1);
        l[n][0] += p0 + p2;
        l[n][1] += p1 + p3;
        // p is rounded to 16 bits for the product: V has no more, and the sum keeps the unrounded values
        pf[n][0] = transpose8x8(pack_elem2<F16>(p0, p1));
        pf[n][1] = transpose8x8(pack_elem2<F16>(p2, p3));
      }
      // O^T += V^T P
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        uint32_t vf[4];
        const int r = (lane & 7) + (lane >> 4) * 8, x = 2 * t + ((lane >> 3) & 1);
        ldsm4_trans(vf, st + kHalf + r * kRowBytes + ((x ^ (r & 7)) << 4));
#pragma unroll
        for (int n = 0; n < NT; ++n) mma16<F16>(o[n][t], vf, pf[n][0], pf[n][1]);
      }

      // ---- the item's last unit here
      const bool item_ends = use.chunk + 1 == use.units;
      if (item_ends || i + 1 == total) {
        fresh = true;
        const int heads = min(kMaxHeads, a.group - use.hc % a.chunks * kMaxHeads);
        const int hq = use.hc / a.chunks * a.group + use.hc % a.chunks * kMaxHeads;
        const bool whole = item_ends && first >= u0;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) l[n][e] += __shfl_xor_sync(~0u, l[n][e], d);
        }
        if (whole) {
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const float i0 = 1.0f / l[n][0], i1 = 1.0f / l[n][1];
            uint16_t* op = a.out + ((int64_t)use.b * a.q_heads + hq + n * 8 + g) * D;
#pragma unroll
            for (int t = 0; t < MT; ++t) {
              const uint32_t lo = transpose8x8(pack_elem2<F16>(o[n][t][0] * i0, o[n][t][1] * i1));
              const uint32_t hi = transpose8x8(pack_elem2<F16>(o[n][t][2] * i0, o[n][t][3] * i1));
              if (n * 8 + g < heads) {
                *reinterpret_cast<uint32_t*>(op + t * 16 + c2) = lo;
                *reinterpret_cast<uint32_t*>(op + t * 16 + c2 + 8) = hi;
              }
            }
            if (a.lse && g == 0) {
#pragma unroll
              for (int e = 0; e < 2; ++e)
                if (n * 8 + c2 + e < heads)
                  a.lse[(int64_t)use.b * a.q_heads + hq + n * 8 + c2 + e] =
                      (m[n][e] + log2_sum<F16>(l[n][e])) * kLn2;
            }
          }
        } else {
          // A piece of an item.  The last one of the range waits in this
          // warp's part of the ring, which is empty then; an earlier one (the
          // end of an item that another warp began) goes to the workspace.
          const bool tail = i + 1 == total;
          const int sl = 2 * warp + tail;
          float* po;
          if (tail) {
            cp_async_wait<0>();
            __syncwarp();
            po = reinterpret_cast<float*>(smem + warp * kStages * kStage);
          } else {
            po = a.heads + (int64_t)w * (kMaxHeads * kPad);
          }
          if (lane == 0) {
            s_item[sl] = use.b * items + use.hc;
            s_first[sl] = first;
            s_units[sl] = use.units;
            s_heads[sl] = heads;
            s_row[sl] = (int64_t)use.b * a.q_heads + hq;
          }
#pragma unroll
          for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              if (g == 0) {
                s_m[sl][n * 8 + c2 + e] = m[n][e];
                s_l[sl][n * 8 + c2 + e] = l[n][e];
              }
#pragma unroll
              for (int t = 0; t < MT; ++t) {
                po[(n * 8 + c2 + e) * kPad + t * 16 + g] = o[n][t][e];
                po[(n * 8 + c2 + e) * kPad + t * 16 + g + 8] = o[n][t][2 + e];
              }
            }
          }
        }
      }
      if (i + 1 < total) use.next(a, items);
    }
  }
  __syncthreads();

  // ---- the block's pieces, in order: runs of one item are added up, four
  // elements a thread, every load of a run in flight at once
  const long long c0 = (long long)blockIdx.x * kWarps;
  const long long block_first = divide(c0 * U, W), block_end = divide(min(c0 + kWarps, W) * U, W);
  const int mine = lane < 2 * kWarps ? s_item[lane] : -1;
  const unsigned used = __ballot_sync(~0u, mine >= 0);
  const unsigned below = used & ((1u << lane) - 1);
  const int prev = __shfl_sync(~0u, mine, below ? 31 - __clz(below) : 31);
  const unsigned starts = __ballot_sync(~0u, mine >= 0 && prev != mine);
  const int quads = min(kMaxHeads, a.group) * (D / 4), runs = __popc(starts);
  for (int e = tid; e < runs * quads; e += kThreads) {
    const int nth = e / quads, f = e - nth * quads, h = f / (D / 4), d = f % (D / 4) * 4;
    unsigned rest = starts;                          // from the nth run's first piece on
    for (int i = 0; i < nth; ++i) rest &= rest - 1;
    const int sl = __ffs(rest) - 1;
    if (h >= s_heads[sl]) continue;
    rest &= rest - 1;
    unsigned run = used & ~((1u << sl) - 1) & (rest ? (rest & -rest) - 1 : ~0u);
    const int64_t row = s_row[sl] + h;
    SPEAR_CHECK(&g_attn_decode_status, sl >= 0 && sl < 2 * kWarps && row < (int64_t)a.s.n * a.q_heads);
    Row r;
#pragma unroll 1
    while (run) {
      const int x = __ffs(run) - 1;
      run &= run - 1;
      r.join(s_m[x][h], s_l[x][h],
             x & 1 ? *reinterpret_cast<const float4*>(smem + (x >> 1) * kStages * kStage + (h * kPad + d) * 4)
                   : __ldcg(reinterpret_cast<const float4*>(a.heads + (c0 + (x >> 1)) * (kMaxHeads * kPad) + h * kPad + d)));
    }
    const long long first = s_first[sl];
    if (first >= block_first && first + s_units[sl] <= block_end) {
      store_row<F16>(a, row, d, D, r.o, r.m, r.l);
    } else {
      float* part = a.parts + (2 * (int64_t)blockIdx.x + (first >= block_first)) * part_floats(D);
      *reinterpret_cast<float4*>(part + 2 * kMaxHeads + h * D + d) = r.o;
      if (d == 0) {
        part[h] = r.m;
        part[kMaxHeads + h] = r.l;
      }
    }
  }
  // the (at most two) items that other blocks have parts of too: one that
  // began before, one that ends after
  if (starts == 0) return;
  const int sl0 = __ffs(starts) - 1, sl1 = 31 - __clz(starts);
  const bool share0 = s_first[sl0] < block_first;
  const bool share1 = s_first[sl1] >= block_first && s_first[sl1] + s_units[sl1] > block_end;
  if (!share0 && !share1) return;

  // ---- such items: the last block to get here adds the parts
  int from = 0, to = 0;                              // (threads 0 and 1) the blocks with the item's ends
  if (tid < 2) {
    const int sl = tid ? sl1 : sl0;
    from = (int)divide((s_first[sl] + 1) * W - 1, U) / kWarps;
    to = (int)divide((s_first[sl] + s_units[sl]) * W - 1, U) / kWarps;
  }
  __threadfence();
  __syncthreads();
  if (tid < 2) {
    int last = 0;
    if (tid ? share1 : share0) {
      if (atom_add_acq_rel_gpu(a.tickets + to, 1) == (unsigned)(to - from)) {
        a.tickets[to] = 0;                            // ready for the next call
        last = 1;
        s_from[tid] = from;
        s_to[tid] = to;
      }
    }
    s_last[tid] = last;
  }
  __syncthreads();
  for (int e = tid; e < 2 * quads; e += kThreads) {
    const int x = e >= quads, f = e - x * quads, h = f / (D / 4), d = f % (D / 4) * 4, sl = x ? sl1 : sl0;
    if (!s_last[x] || h >= s_heads[sl]) continue;
    const int first = s_from[x], last = s_to[x];
    SPEAR_CHECK(&g_attn_decode_status, first >= 0 && first < last && last < (int)gridDim.x);
    Row r;
    constexpr int kAhead = 8;                         // parts in flight
    for (int c = first; c <= last; c += kAhead) {
      float pm[kAhead], pl[kAhead];
      float4 po[kAhead];
#pragma unroll
      for (int y = 0; y < kAhead; ++y)
        if (c + y <= last) {
          const float* part = a.parts + (2 * (int64_t)(c + y) + (c + y == first)) * part_floats(D);
          pm[y] = __ldcg(part + h);
          pl[y] = __ldcg(part + kMaxHeads + h);
          po[y] = __ldcg(reinterpret_cast<const float4*>(part + 2 * kMaxHeads + h * D + d));
        }
#pragma unroll
      for (int y = 0; y < kAhead; ++y)
        if (c + y <= last) r.join(pm[y], pl[y], po[y]);
    }
    store_row<F16>(a, s_row[sl] + h, d, D, r.o, r.m, r.l);
  }
}

size_t ticket_bytes(const DeviceInfo& di) { return ((size_t)di.num_sms * sizeof(unsigned) + 255) / 256 * 256; }

template <int D, bool F16, int NT>
int launch(const DecArgs& a, int blocks, cudaStream_t st) {
  const void* fn = reinterpret_cast<const void*>(&attn_decode_kernel<D, F16, NT>);
  if (int rc = ensure_smem_limit(fn, kRingBytes)) return rc;
  return launch_dependent(attn_decode_kernel<D, F16, NT>, dim3(blocks), kThreads, kRingBytes, st, "attn_decode launch", a);
}
}  // namespace

int attn_decode_workspace_bytes(const spear_kv_cache& c, int nseqs, int q_heads, size_t* bytes) {
  DeviceInfo di;
  if (int rc = device_info(&di)) return rc;
  *bytes = ticket_bytes(di) + (size_t)di.num_sms * 2 * part_floats(c.head_dim) * sizeof(float) +
           (size_t)di.num_sms * kWarps * kMaxHeads * (c.head_dim + 4) * sizeof(float);
  return SPEAR_OK;
}

int launch_attn_decode(const spear_kv_cache& c, const spear_kv_seqs& s, const spear_attn& at, void* ws,
                       size_t ws_bytes, cudaStream_t st) {
  DeviceInfo di;
  if (int rc = device_info(&di)) return rc;
  size_t need = 0;
  if (int rc = attn_decode_workspace_bytes(c, s.num_seqs, at.num_q_heads, &need)) return rc;
  if (!ws || ws_bytes < need || (reinterpret_cast<uintptr_t>(ws) & 15))
    return fail(SPEAR_ERR_WORKSPACE, "attn_decode workspace needs %zu bytes, 16-byte aligned, got %zu", need, ws_bytes);
  const int group = at.num_q_heads / c.num_kv_heads, chunks = (group + kMaxHeads - 1) / kMaxHeads;
  if ((long long)s.num_seqs * c.num_kv_heads * chunks > 0x7fffffffLL)
    return fail(SPEAR_ERR_UNSUPPORTED, "%d sequences of %d heads are too many for one call", s.num_seqs, at.num_q_heads);
  char* p = static_cast<char*>(ws);
  DecArgs a{kv_view(c), seq_view(s), at.q, at.q_token_stride, at.q_head_stride, at.out, at.lse,
            reinterpret_cast<unsigned*>(p), reinterpret_cast<float*>(p + ticket_bytes(di)), nullptr,
            at.num_q_heads, group, chunks, at.window, at.sinks, at.scale * kLog2e};
  a.heads = a.parts + (size_t)di.num_sms * 2 * part_floats(c.head_dim);
  const bool f16 = c.dtype == SPEAR_DT_F16, wide = group > 8;
  const int blocks = di.num_sms;
  if (c.head_dim == 64) {
    if (wide) return f16 ? launch<64, true, 2>(a, blocks, st) : launch<64, false, 2>(a, blocks, st);
    return f16 ? launch<64, true, 1>(a, blocks, st) : launch<64, false, 1>(a, blocks, st);
  }
  if (wide) return f16 ? launch<128, true, 2>(a, blocks, st) : launch<128, false, 2>(a, blocks, st);
  return f16 ? launch<128, true, 1>(a, blocks, st) : launch<128, false, 1>(a, blocks, st);
}

int status_word_attn_decode(unsigned** word) {
  return cuda_check(cudaGetSymbolAddress(reinterpret_cast<void**>(word), g_attn_decode_status), "attn_decode status address");
}

}  // namespace spear
