// kv.cu -- the paged key/value cache: appending rows, and the page
// bookkeeping (reserve, fork, free, compact, copy), all on the device so that
// a serving step needs no answer from the GPU before its next launch.
//
// The copies are bound by memory: 8 k tokens' rows (248 MB read and written)
// 39 us, 6.4 TB/s; 1500 pages compacted (408 MB) 73 us, of which one block's
// planning takes 5.  The bookkeeping is bound by latency, a few microseconds a
// call: one block scans the counts, so that pages are taken in order.
//
// Pages are reference-counted (refs[p] = table entries naming page p); a page
// with no reference is free, and free pages are taken in ascending order, so
// the outcome of every call is determined by its arguments.
#include <algorithm>

#include "kv.cuh"

namespace spear {

namespace {
__device__ unsigned g_kv_status;

// ------------------------------------------------------------------ append
//
// Each new token's rows go to cache[table[row][pos / page]][h][pos % page]:
// a copy of 2 Hkv D elements a token, bound by memory.
constexpr int kAppendThreads = 256, kAppendUnroll = 4;

// Bits of a pool's moves[1].
constexpr int kReserveRefused = 1;     // by the last reserve; append reads it
constexpr int kForkRefused = 2;        // by the take kernel, for the fork's second kernel

struct AppendArgs {
  KvView c;
  SeqView s;
  const uint16_t *k_new, *v_new;
  int64_t kt, kh, vt, vh;              // token and head strides of the new rows
  const int32_t* starts;               // [n + 1]: sequence b's tokens are [starts[b], starts[b + 1])
  const int32_t* refused;              // the word that says whether the lengths count the new tokens (NULL: they do)
  int tokens, vecs;                    // vecs: 16-byte pieces of one head's row
};

__global__ void __launch_bounds__(kAppendThreads) kv_append_kernel(const __grid_constant__ AppendArgs a) {
  enter();
  __shared__ int64_t s_off;
  __shared__ int s_refused;
  const int t = blockIdx.x;
  // beside the search of thread 0 (in it: 42.1 against 39.4 us for 248 MB)
  if (threadIdx.x == 32) s_refused = a.refused ? *a.refused & kReserveRefused : 0;
  if (threadIdx.x == 0) {
    int lo = 0, hi = a.s.n;            // last b with starts[b] <= t
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (a.starts[mid] <= t) lo = mid; else hi = mid;
    }
    int64_t off = -1;
    const int end = a.starts[lo + 1];
    if (a.starts[lo] <= t && t < end && end <= a.tokens) {
      const int row = seq_row(a.s, lo, &g_kv_status);
      const int len = seq_len(a.s, a.c, row, &g_kv_status);
      const int pos = len - (end - t);
      if (row >= 0 && pos >= 0) off = kv_row_offset(a.c, a.s.table + row * a.s.table_stride, pos, &g_kv_status);
      else record_status(&g_kv_status, DEV_ERR_INVALID);
    } else {
      record_status(&g_kv_status, DEV_ERR_INVALID);
    }
    s_off = off;
  }
  __syncthreads();
  const int64_t off = s_off;
  if (s_refused) {
    if (threadIdx.x == 0) record_status(&g_kv_status, DEV_ERR_INVALID);
    return;
  }
  if (off < 0) return;
  const int n = a.c.heads * a.vecs;
  for (int i0 = threadIdx.x; i0 < 2 * n; i0 += kAppendUnroll * kAppendThreads) {
    uint4 x[kAppendUnroll];
    uint16_t* dst[kAppendUnroll];
#pragma unroll
    for (int u = 0; u < kAppendUnroll; ++u) {
      const int i = i0 + u * kAppendThreads;
      dst[u] = nullptr;
      if (i < 2 * n) {
        const bool is_v = i >= n;
        const int j = is_v ? i - n : i, h = j / a.vecs, c = j - h * a.vecs;
        const uint16_t* src = is_v ? a.v_new + t * a.vt + h * a.vh : a.k_new + t * a.kt + h * a.kh;
        x[u] = ldg16(src + 8 * c);
        dst[u] = const_cast<uint16_t*>(is_v ? a.c.v : a.c.k) + off + h * a.c.head_stride + 8 * c;
      }
    }
#pragma unroll
    for (int u = 0; u < kAppendUnroll; ++u)
      if (dst[u]) *reinterpret_cast<uint4*>(dst[u]) = x[u];
  }
}

// -------------------------------------------------------------------- pages

constexpr int kPoolThreads = 1024;

struct PoolView {
  int32_t *refs, *lens, *table, *moves;
  int num_pages, max_seqs, max_pages;
  FastDiv page;
};
PoolView pool_view(const spear_kv_pool& p) {
  return {p.refs, p.seq_lens, p.block_table, p.moves, p.num_pages, p.max_seqs, p.max_pages,
          FastDiv::of((uint32_t)p.page_size)};
}

// moves: [0] count, [1] what was refused, then `count` pairs (source page,
// destination page) from [2]; [2 + 2 num_pages ..] is scratch of num_pages
// words (the free list of reserve and fork, compact's renaming).
__device__ __forceinline__ int32_t* pool_scratch(const PoolView& p) { return p.moves + 2 + 2 * (int64_t)p.num_pages; }

// Exclusive prefix sum of v over the block; *total gets the sum.
__device__ __forceinline__ int block_scan(int v, int* total) {
  __shared__ int s_w[32];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(~0u, x, d);
    if (lane >= d) x += y;
  }
  if (lane == 31) s_w[w] = x;
  __syncthreads();
  int ws = s_w[lane];
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(~0u, ws, d);
    if (lane >= d) ws += y;
  }
  const int before = w ? __shfl_sync(~0u, ws, w - 1) : 0;
  *total = __shfl_sync(~0u, ws, 31);
  __syncthreads();
  return before + x - v;
}

// What a listed row needs: reserve's or fork's view of entry i.
struct Need {
  int row, have, need, bad;
};

// One block: checks every entry, finds the total of new pages and takes the
// lowest free ones in the entries' order.  Nothing is changed when an entry is
// invalid or the pool is too small; that is recorded, and moves[1] says so to
// the fork's second kernel, or to the appends that follow a reserve.
template <bool FORK>
__global__ void __launch_bounds__(kPoolThreads)
pool_take_kernel(PoolView p, const int32_t* rows, const int32_t* arg, int n) {
  enter();
  extern __shared__ unsigned s_seen[];              // one bit a row of the table
  __shared__ int s_bad;
  __shared__ unsigned long long s_total;            // pages that all entries need: 64 bits, entries can ask for 2^31 each
  const int tid = threadIdx.x;
  for (int i = tid; i < (p.max_seqs + 31) / 32; i += kPoolThreads) s_seen[i] = 0;
  if (tid == 0) {
    s_bad = 0;
    s_total = 0;
  }
  // the first pages' counts travel while the entries are checked
  int4 ahead = make_int4(1, 1, 1, 1);
  const bool whole = 4 * tid + 3 < p.num_pages;
  if (whole) ahead = make_int4(p.refs[4 * tid], p.refs[4 * tid + 1], p.refs[4 * tid + 2], p.refs[4 * tid + 3]);
  __syncthreads();
  // FORK: rows = children, arg = parents; otherwise arg = new tokens
  auto entry = [&](int i) {
    Need e{rows[i], 0, 0, 0};
    if (e.row < 0 || e.row >= p.max_seqs) return Need{0, 0, 0, 1};
    const long long cap = (long long)p.max_pages * p.page.d;
    if (FORK) {
      const int par = arg[i];
      if (par < 0 || par >= p.max_seqs) return Need{0, 0, 0, 1};
      const int len = p.lens[par];
      if (len < 0 || len > cap || p.lens[e.row] != 0) return Need{0, 0, 0, 1};
      e.have = (int)p.page.div((uint32_t)len);
      e.need = len - e.have * (int)p.page.d > 0;
    } else {
      const int len = p.lens[e.row], add = arg[i];
      const long long want = (long long)len + add;
      if (len < 0 || add < 0 || want > cap || want > 0x7fffffff - (long long)p.page.d) return Need{0, 0, 0, 1};
      e.have = (int)p.page.div((uint32_t)len + p.page.d - 1);
      e.need = (int)p.page.div((uint32_t)want + p.page.d - 1) - e.have;
    }
    return e;
  };
  Need kept{0, 0, 0, 0};                            // this thread's entry, where there are no more than threads
  for (int i0 = 0; i0 < n; i0 += kPoolThreads) {
    const int i = i0 + tid;
    Need e{0, 0, 0, 0};
    if (i < n) {
      e = entry(i);
      if (!e.bad && (atomicOr(&s_seen[e.row >> 5], 1u << (e.row & 31)) >> (e.row & 31) & 1)) e.bad = 1;  // listed twice
      if (e.bad) s_bad = 1;
    }
    kept = e;
    if (!e.bad && e.need > 0) atomicAdd(&s_total, (unsigned long long)e.need);
  }
  __syncthreads();
  const long long total = (long long)min(s_total, (unsigned long long)p.num_pages + 1);
  if (FORK) {                                       // a row is not both: its old and new length would race
    for (int i = tid; i < n; i += kPoolThreads) {
      const int par = arg[i];
      if (par >= 0 && par < p.max_seqs && (s_seen[par >> 5] >> (par & 31) & 1)) s_bad = 1;
    }
    __syncthreads();
  }
  // the lowest `total` free pages, in order
  int32_t* list = pool_scratch(p);
  int found = 0;
  for (int i0 = 0; i0 < p.num_pages && found < total; i0 += 4 * kPoolThreads) {
    int f[4], c = 0;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int i = i0 + 4 * tid + x;
      const int refs = i0 == 0 && whole ? (x == 0 ? ahead.x : x == 1 ? ahead.y : x == 2 ? ahead.z : ahead.w)
                       : i < p.num_pages ? p.refs[i] : 1;
      f[x] = refs == 0;
      c += f[x];
    }
    int sum, at = found + block_scan(c, &sum);
#pragma unroll
    for (int x = 0; x < 4; ++x)
      if (f[x]) {
        if (at < total) list[at] = i0 + 4 * tid + x;
        ++at;
      }
    found += sum;
  }
  __syncthreads();
  const bool refused = s_bad || found < total;
  if (tid == 0) {
    p.moves[0] = 0;
    if (FORK) p.moves[1] = (p.moves[1] & kReserveRefused) | (refused ? kForkRefused : 0);
    else p.moves[1] = refused ? kReserveRefused : 0;
    if (refused) record_status(&g_kv_status, DEV_ERR_INVALID);
  }
  if (refused) return;
  int base = 0, nmoves = 0;
  for (int i0 = 0; i0 < n; i0 += kPoolThreads) {
    const int i = i0 + tid;
    Need e{0, 0, 0, 0};
    if (i < n) e = n <= kPoolThreads ? kept : entry(i);
    int sum, at = base + block_scan(e.need, &sum);
    base += sum;
    if (FORK) {
      if (i < n) {
        if (e.need) {
          const int pg = list[at];
          SPEAR_CHECK(&g_kv_status, pg >= 0 && pg < p.num_pages && e.have < p.max_pages && at < p.num_pages);
          p.table[(int64_t)e.row * p.max_pages + e.have] = pg;
          p.refs[pg] = 1;
          p.moves[2 + 2 * at] = p.table[(int64_t)arg[i] * p.max_pages + e.have];
          p.moves[3 + 2 * at] = pg;
        }
        p.lens[e.row] = p.lens[arg[i]];
      }
      nmoves += sum;
    } else {
      // a warp writes the pages of its 32 entries one entry after another
      const int lane = tid & 31;
      for (int src = 0; src < 32; ++src) {
        const int need = __shfl_sync(~0u, e.need, src), first = __shfl_sync(~0u, at, src);
        const int row = __shfl_sync(~0u, e.row, src), have = __shfl_sync(~0u, e.have, src);
        for (int j = lane; j < need; j += 32) {
          const int pg = list[first + j];
          SPEAR_CHECK(&g_kv_status, pg >= 0 && pg < p.num_pages && have + j < p.max_pages);
          p.table[(int64_t)row * p.max_pages + have + j] = pg;
          p.refs[pg] = 1;
        }
      }
      if (i < n) p.lens[e.row] += arg[i];
    }
  }
  if (FORK && tid == 0) p.moves[0] = nmoves;
}

// One block a freed row; the exchange of the length makes a row that is
// listed twice (or is empty already) a no-op.  A row whose length is out of
// range stays as it is: what it holds is not known.
__global__ void __launch_bounds__(256) pool_free_kernel(PoolView p, const int32_t* rows) {
  __shared__ int s_len;
  enter();
  const int row = rows[blockIdx.x];
  if (row < 0 || row >= p.max_seqs) {
    if (threadIdx.x == 0) record_status(&g_kv_status, DEV_ERR_INVALID);
    return;
  }
  if (threadIdx.x == 0) {
    const int at = p.lens[row];
    const bool bad = at < 0 || (long long)at > (long long)p.max_pages * p.page.d;
    if (bad) record_status(&g_kv_status, DEV_ERR_INVALID);
    s_len = bad ? 0 : atomicExch(&p.lens[row], 0);
  }
  __syncthreads();
  const int len = s_len;
  const int held = (int)p.page.div((uint32_t)len + p.page.d - 1);
  for (int j = threadIdx.x; j < held; j += 256) {
    int32_t* e = p.table + (int64_t)row * p.max_pages + j;
    const int pg = *e;
    *e = -1;
    if ((unsigned)pg >= (unsigned)p.num_pages) {
      record_status(&g_kv_status, DEV_ERR_INVALID);
    } else if (atomicSub(&p.refs[pg], 1) <= 0) {    // nobody's page: it stays free
      atomicAdd(&p.refs[pg], 1);
      record_status(&g_kv_status, DEV_ERR_INVALID);
    }
  }
}

// One block: with L live pages, the i-th live page of index >= L goes to the
// i-th free page of index < L (both ascending).  Sources and destinations are
// disjoint, so the pages can be copied in any order.
__global__ void __launch_bounds__(kPoolThreads) pool_compact_plan_kernel(PoolView p) {
  enter();
  const int tid = threadIdx.x;
  int live = 0;
  for (int i = tid; i < p.num_pages; i += kPoolThreads) live += p.refs[i] > 0;
  int L;
  block_scan(live, &L);
  int32_t* rename = pool_scratch(p);
  int holes = 0, highs = 0;
  for (int i0 = 0; i0 < p.num_pages; i0 += kPoolThreads) {
    const int i = i0 + tid;
    const bool in = i < p.num_pages, is_live = in && p.refs[i] > 0;
    const int hole = in && !is_live && i < L, high = is_live && i >= L;
    int sum;
    const int at = block_scan(hole ? 1 : high << 16, &sum);       // at most 1024 of each: two counts in one scan
    if (hole) p.moves[3 + 2 * (int64_t)(holes + (at & 0xffff))] = i;
    if (high) p.moves[2 + 2 * (int64_t)(highs + (at >> 16))] = i;
    holes += sum & 0xffff;
    highs += sum >> 16;
  }
  __syncthreads();
  for (int i = tid; i < highs; i += kPoolThreads) {
    const int src = p.moves[2 + 2 * (int64_t)i], dst = p.moves[3 + 2 * (int64_t)i];
    rename[src] = dst;
    p.refs[dst] = p.refs[src];
    p.refs[src] = 0;
  }
  if (tid == 0) {
    p.moves[0] = highs;
    rename[0] = L;                                  // page 0 is never renamed: with a live page, L > 0
  }
}

// ------------------------------------------------------- page copies

constexpr int kCopyThreads = 256, kCopyUnroll = 8, kMaxCaches = 64;

struct CopyArgs {
  uint16_t* k[kMaxCaches];
  uint16_t* v[kMaxCaches];
  int64_t page_stride, head_stride, slot_stride;
  int num_pages, heads, slots, vecs;   // vecs: 16-byte pieces of one row
  int packed;                          // a page is one run of heads slots vecs pieces
  int parts;                           // blocks of work a page and cache half
  const int32_t* moves;
  int max_moves;
};

// Copies K and V of moves[0] pages.  Work unit: kCopyThreads kCopyUnroll
// pieces of one page's K or V; all of a thread's loads are in flight before
// its first store.
__device__ __forceinline__ void copy_pages(const CopyArgs& a, int block, int blocks) {
  const int count = min(a.moves[0], a.max_moves);
  const int per_page = a.heads * a.slots * a.vecs;
  const long long units = (long long)count * 2 * a.parts;
  uint16_t* kb = a.k[blockIdx.y];
  uint16_t* vb = a.v[blockIdx.y];
  for (long long u = block; u < units; u += blocks) {
    const int m = (int)(u / (2 * a.parts)), r = (int)(u - (long long)m * 2 * a.parts);
    const int half = r >= a.parts, part = r - half * a.parts;
    const int src = a.moves[2 + 2 * (int64_t)m], dst = a.moves[3 + 2 * (int64_t)m];
    if ((unsigned)src >= (unsigned)a.num_pages || (unsigned)dst >= (unsigned)a.num_pages) {
      if (threadIdx.x == 0) record_status(&g_kv_status, DEV_ERR_INVALID);
      continue;
    }
    uint16_t* base = half ? vb : kb;
    const uint16_t* from = base + src * a.page_stride;
    uint16_t* to = base + dst * a.page_stride;
    uint4 x[kCopyUnroll];
    int64_t off[kCopyUnroll];
#pragma unroll
    for (int i = 0; i < kCopyUnroll; ++i) {
      const int e = (part * kCopyUnroll + i) * kCopyThreads + threadIdx.x;
      off[i] = -1;
      if (e < per_page) {
        if (a.packed) {
          off[i] = 8 * (int64_t)e;
        } else {
          const int row = e / a.vecs, h = row / a.slots;
          off[i] = h * a.head_stride + (row - h * a.slots) * a.slot_stride + 8 * (e - row * a.vecs);
        }
        x[i] = *reinterpret_cast<const uint4*>(from + off[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < kCopyUnroll; ++i)
      if (off[i] >= 0) *reinterpret_cast<uint4*>(to + off[i]) = x[i];
  }
}

__global__ void __launch_bounds__(kCopyThreads) copy_pages_kernel(const __grid_constant__ CopyArgs a) {
  enter();
  copy_pages(a, blockIdx.x, gridDim.x);
}

// Fork's second half: the children's shared pages (whole pages of the parent;
// the take kernel has written the rest) and the copies of the partial ones.
__global__ void __launch_bounds__(kCopyThreads)
fork_apply_kernel(const __grid_constant__ CopyArgs a, PoolView p, const int32_t* parents, const int32_t* children,
                  int n) {
  enter();
  if (p.moves[1] & kForkRefused) return;
  if (blockIdx.y == 0) {
    for (int i = blockIdx.x; i < n; i += gridDim.x) {
      const int32_t* from = p.table + (int64_t)parents[i] * p.max_pages;
      int32_t* to = p.table + (int64_t)children[i] * p.max_pages;
      const int whole = (int)p.page.div((uint32_t)p.lens[parents[i]]);
      for (int j = threadIdx.x; j < whole; j += kCopyThreads) {
        const int pg = from[j];
        to[j] = pg;
        if ((unsigned)pg >= (unsigned)p.num_pages) record_status(&g_kv_status, DEV_ERR_INVALID);
        else atomicAdd(&p.refs[pg], 1);
      }
    }
  }
  if (a.parts) copy_pages(a, blockIdx.x, gridDim.x);
}

// Compact's second half: the block tables' new page numbers, and the copies.
__global__ void __launch_bounds__(kCopyThreads) compact_apply_kernel(const __grid_constant__ CopyArgs a, PoolView p) {
  enter();
  if (blockIdx.y == 0) {
    const int32_t* rename = pool_scratch(p);
    const int L = rename[0];
    for (int i = blockIdx.x; i < p.max_seqs; i += gridDim.x) {
      int32_t* row = p.table + (int64_t)i * p.max_pages;
      for (int j = threadIdx.x; j < p.max_pages; j += kCopyThreads) {
        const int pg = row[j];
        if (pg >= L && pg < p.num_pages) row[j] = rename[pg];
      }
    }
  }
  if (a.parts) copy_pages(a, blockIdx.x, gridDim.x);
}

// How many of the caches from the first on one launch takes: those of its
// geometry that follow it, kMaxCaches at most.
int one_launch(const spear_kv_cache* c, int n) {
  int i = 1;
  while (i < n && i < kMaxCaches && c[i].num_kv_heads == c[0].num_kv_heads && c[i].head_dim == c[0].head_dim &&
         c[i].page_stride == c[0].page_stride && c[i].head_stride == c[0].head_stride &&
         c[i].slot_stride == c[0].slot_stride)
    ++i;
  return std::min(i, n);
}
// The copy's arguments for caches [first, first + count) of one geometry.
CopyArgs copy_args(const spear_kv_cache* caches, int first, int count, const int32_t* moves, int max_moves) {
  CopyArgs a{};
  if (count > 0) {
    const spear_kv_cache& c = caches[first];
    for (int i = 0; i < count; ++i) {
      a.k[i] = caches[first + i].k;
      a.v[i] = caches[first + i].v;
    }
    a.page_stride = c.page_stride;
    a.head_stride = c.head_stride;
    a.slot_stride = c.slot_stride;
    a.num_pages = c.num_pages;
    a.heads = c.num_kv_heads;
    a.slots = c.page_size;
    a.vecs = c.head_dim / 8;
    const int64_t row = c.head_dim, page = row * c.page_size * c.num_kv_heads;
    a.packed = (c.slot_stride == row && c.head_stride == row * c.page_size) ||
               (c.head_stride == row && c.slot_stride == row * c.num_kv_heads);
    a.parts = (int)((page / 8 + kCopyThreads * kCopyUnroll - 1) / (kCopyThreads * kCopyUnroll));
  }
  a.moves = moves;
  a.max_moves = max_moves;
  return a;
}

int copy_grid(const CopyArgs& a, int ncaches, long long other, const DeviceInfo& di) {
  const long long units = std::max<long long>((long long)a.max_moves * 2 * a.parts, other);
  const long long most = std::max(1, di.num_sms * 8 / std::max(1, ncaches));
  return (int)std::max<long long>(1, std::min(units, most));
}

}  // namespace

int launch_kv_append(const spear_kv_cache& c, const spear_kv_seqs& s, const int32_t* starts, int tokens,
                     const uint16_t* k_new, int64_t kt, int64_t kh, const uint16_t* v_new, int64_t vt, int64_t vh,
                     cudaStream_t st) {
  AppendArgs a{kv_view(c), seq_view(s), k_new, v_new, kt, kh, vt, vh, starts, s.refused, tokens, c.head_dim / 8};
  return launch_dependent(kv_append_kernel, dim3(tokens), kAppendThreads, 0, st, "kv_append launch", a);
}

int launch_kv_copy_pages(const spear_kv_cache* caches, int ncaches, const int32_t* moves, int max_moves,
                         cudaStream_t st) {
  DeviceInfo di;
  if (int rc = device_info(&di)) return rc;
  for (int i = 0, n = 0; i < ncaches; i += n) {
    n = one_launch(caches + i, ncaches - i);
    const CopyArgs a = copy_args(caches, i, n, moves, max_moves);
    if (int rc = launch_dependent(copy_pages_kernel, dim3(copy_grid(a, n, 1, di), n), kCopyThreads, 0, st,
                                  "copy_pages launch", a)) return rc;
  }
  return SPEAR_OK;
}

int launch_kv_reserve(const spear_kv_pool& p, const int32_t* rows, const int32_t* tokens, int n, cudaStream_t st) {
  return launch_dependent(pool_take_kernel<false>, dim3(1), kPoolThreads, (p.max_seqs + 31) / 32 * 4, st,
                          "kv_reserve launch", pool_view(p), rows, tokens, n);
}

int launch_kv_free(const spear_kv_pool& p, const int32_t* rows, int n, cudaStream_t st) {
  return launch_dependent(pool_free_kernel, dim3(n), 256, 0, st, "kv_free launch", pool_view(p), rows);
}

int launch_kv_fork(const spear_kv_pool& p, const spear_kv_cache* caches, int ncaches, const int32_t* parents,
                   const int32_t* children, int n, cudaStream_t st) {
  DeviceInfo di;
  if (int rc = device_info(&di)) return rc;
  if (int rc = launch_dependent(pool_take_kernel<true>, dim3(1), kPoolThreads, (p.max_seqs + 31) / 32 * 4, st,
                                "kv_fork launch", pool_view(p), children, parents, n)) return rc;
  const int first = one_launch(caches, ncaches);
  const CopyArgs a = copy_args(caches, 0, first, p.moves, n);
  if (int rc = launch_dependent(fork_apply_kernel, dim3(copy_grid(a, first, n, di), std::max(1, first)), kCopyThreads, 0,
                                st, "kv_fork launch", a, pool_view(p), parents, children, n)) return rc;
  return ncaches > first ? launch_kv_copy_pages(caches + first, ncaches - first, p.moves, n, st) : SPEAR_OK;
}

int launch_kv_compact(const spear_kv_pool& p, const spear_kv_cache* caches, int ncaches, cudaStream_t st) {
  DeviceInfo di;
  if (int rc = device_info(&di)) return rc;
  if (int rc = launch_dependent(pool_compact_plan_kernel, dim3(1), kPoolThreads, 0, st, "kv_compact launch",
                                pool_view(p))) return rc;
  const int first = one_launch(caches, ncaches);
  const CopyArgs a = copy_args(caches, 0, first, p.moves, p.num_pages);
  if (int rc = launch_dependent(compact_apply_kernel, dim3(copy_grid(a, first, p.max_seqs, di), std::max(1, first)),
                                kCopyThreads, 0, st, "kv_compact launch", a, pool_view(p))) return rc;
  return ncaches > first ? launch_kv_copy_pages(caches + first, ncaches - first, p.moves, p.num_pages, st) : SPEAR_OK;
}

int status_word_kv(unsigned** word) {
  return cuda_check(cudaGetSymbolAddress(reinterpret_cast<void**>(word), g_kv_status), "kv status address");
}

}  // namespace spear
