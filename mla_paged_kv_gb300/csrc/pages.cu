// Page operations of a paged cache: growing, forking, freeing and compacting
// rows of the block table, and copying the pages that this moves.
//
// The bookkeeping is whole numbers, and every choice is by order (lowest free
// page first, list order, an exclusive scan), never by which thread came
// first, so results are the same on every run.  Its cost is launches and the
// latency of a few passes over the counts, not bandwidth: grow and fork are
// one block each (4 bytes a page: a pool of 65536 pages is 256 KB), compact is
// three launches over 4096-page chunks.  The data moves in copy_pages, which
// is bound by HBM.
#include "common.cuh"
#include "serving.cuh"

namespace mla {
namespace {

constexpr int kThreads = 1024;
constexpr int kPagesPerThread = 8;  // counts a thread reads in one step of a scan over the pool

// Exclusive scan over the block of one value a thread; *total = the sum.
// `s` holds 33 ints; safe to call again at once.
__device__ __forceinline__ int block_scan(int v, int* s, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += u;
  }
  if (lane == 31) s[warp] = inc;
  __syncthreads();
  if (warp == 0) {
    const int w = lane < static_cast<int>(blockDim.x >> 5) ? s[lane] : 0;
    int x = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += u;
    }
    s[lane] = x - w;
    if (lane == 31) s[32] = x;
  }
  __syncthreads();
  const int out = s[warp] + inc - v;
  *total = s[32];
  __syncthreads();
  return out;
}

__device__ __forceinline__ int pages_of(int len) { return (len >> 6) + ((len & 63) != 0); }

// Shared memory of the allocating kernels (grow, fork).
struct AllocSmem {
  int first[kMaxPageList + 1];             // pages wanted before entry i; [n] = all
  uint32_t seen[kMaxPageRows / 32];        // rows listed
  uint32_t twice[kMaxPageRows / 32];       // rows listed more than once
  uint32_t broken[kMaxPageList / 32];      // fork: entries whose parent names a page that is not in use
  int scan[33];
};

__device__ __forceinline__ bool bit(const uint32_t* m, int i) { return (m[i >> 5] >> (i & 31)) & 1u; }

__device__ void mark_rows(AllocSmem& sm, const int32_t* list, int n, int rows) {
  for (int i = threadIdx.x; i < (rows + 31) / 32; i += kThreads) sm.seen[i] = sm.twice[i] = 0u;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const int r = list[i];
    if (r < 0 || r >= rows) continue;
    const uint32_t m = 1u << (r & 31);
    if (atomicOr(&sm.seen[r >> 5], m) & m) atomicOr(&sm.twice[r >> 5], m);
  }
  __syncthreads();
}

// first[i] = sum of want(j) over j < i, for all i <= n.
template <typename F>
__device__ void scan_wants(AllocSmem& sm, int n, F want) {
  int base = 0;
  for (int i0 = 0; i0 < n; i0 += kThreads) {
    const int i = i0 + static_cast<int>(threadIdx.x);
    int total;
    const int ex = block_scan(i < n ? want(i) : 0, sm.scan, &total);
    if (i < n) sm.first[i] = base + ex;
    base += total;
  }
  if (threadIdx.x == 0) sm.first[n] = base;
  __syncthreads();
}

// Walk the counts from page 0 on and give the k-th free page to give(k, page)
// for k < want; returns the free pages met (at least `want` unless the pool
// ran out).
template <typename F>
__device__ int scan_free(AllocSmem& sm, const int32_t* refcount, int num_pages, int want, F give) {
  int found = 0;
  const bool vec = (reinterpret_cast<uintptr_t>(refcount) & 15u) == 0;
  for (int p0 = 0; p0 < num_pages && found < want; p0 += kThreads * kPagesPerThread) {
    const int at = p0 + static_cast<int>(threadIdx.x) * kPagesPerThread;
    int c[kPagesPerThread];
    if (vec && at + kPagesPerThread <= num_pages) {
#pragma unroll
      for (int i = 0; i < kPagesPerThread; i += 4) {
        const int4 v = *reinterpret_cast<const int4*>(refcount + at + i);
        c[i] = v.x, c[i + 1] = v.y, c[i + 2] = v.z, c[i + 3] = v.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < kPagesPerThread; ++i) c[i] = at + i < num_pages ? refcount[at + i] : 1;
    }
    int mine = 0;
#pragma unroll
    for (int i = 0; i < kPagesPerThread; ++i) mine += c[i] == 0;
    int total;
    int k = found + block_scan(mine, sm.scan, &total);
#pragma unroll
    for (int i = 0; i < kPagesPerThread; ++i)
      if (c[i] == 0) {
        if (k < want) give(k, at + i);
        ++k;
      }
    found += total;
  }
  __syncthreads();
  return found;
}

// The entry i with first[i] <= k < first[i + 1].
__device__ __forceinline__ int entry_of(const AllocSmem& sm, int n, int k) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (sm.first[mid] <= k)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// ------------------------------------------------------------------ grow

// New length of entry i's row, or -1 if the entry cannot be served.
__device__ __forceinline__ int grown(const PageState& s, const AllocSmem& sm, const int32_t* rows,
                                     const int32_t* add, int i, int& old_len) {
  const int r = rows[i];
  old_len = 0;
  if (r < 0 || r >= s.rows || bit(sm.twice, r)) return -1;
  old_len = s.seqlens[r];
  const int a = add[i];
  if (old_len < 0 || a < 0) return -1;
  const long long len = static_cast<long long>(old_len) + a;
  return len > static_cast<long long>(s.max_pages) * kTile ? -1 : static_cast<int>(len);
}

__global__ void __launch_bounds__(kThreads) grow_kernel(const PageState s, const int32_t* rows, const int32_t* add,
                                                         int n) {
  __shared__ AllocSmem sm;
  mark_rows(sm, rows, n, s.rows);
  scan_wants(sm, n, [&](int i) {
    int old_len;
    const int len = grown(s, sm, rows, add, i, old_len);
    return len < 0 ? 0 : pages_of(len) - pages_of(old_len);
  });
  // where the k-th new page goes
  auto entry_at = [&](int i, int k) {
    const int r = rows[i];
    return s.table + static_cast<long long>(r) * s.max_pages + pages_of(s.seqlens[r]) + (k - sm.first[i]);
  };
  const int want = sm.first[n];
  const int found = scan_free(sm, s.refcount, s.num_pages, want, [&](int k, int page) {
    *entry_at(entry_of(sm, n, k), k) = page;
    s.refcount[page] = 1;
  });
  if (found < want) {  // the pool ran out: entries past its last page give theirs back
    for (int k = threadIdx.x; k < found; k += kThreads) {
      const int i = entry_of(sm, n, k);
      if (sm.first[i + 1] <= found) continue;
      int32_t* e = entry_at(i, k);
      s.refcount[*e] = 0;
      *e = -1;
    }
    __syncthreads();
  }
  for (int i = threadIdx.x; i < n; i += kThreads) {
    int old_len;
    const int len = grown(s, sm, rows, add, i, old_len);
    if (len < 0)
      report(s.status, MLA_ERR_BAD_INDEX);
    else if (sm.first[i + 1] > found && sm.first[i + 1] > sm.first[i])
      report(s.status, MLA_ERR_NO_PAGES);
    else
      s.seqlens[rows[i]] = len;
  }
}

// ------------------------------------------------------------------ fork

// Length of entry i's parent, or -1 if the entry cannot be served (its parent's
// pages apart).
__device__ __forceinline__ int parent_len(const PageState& s, const AllocSmem& sm, const int32_t* parents,
                                          const int32_t* children, int i) {
  const int pr = parents[i], ch = children[i];
  if (pr < 0 || pr >= s.rows || ch < 0 || ch >= s.rows) return -1;
  if (bit(sm.twice, ch) || bit(sm.seen, pr)) return -1;
  if (s.seqlens[ch] != 0) return -1;
  const int len = s.seqlens[pr];
  return len < 0 || len > static_cast<long long>(s.max_pages) * kTile ? -1 : len;
}

__device__ __forceinline__ int forked(const PageState& s, const AllocSmem& sm, const int32_t* parents,
                                      const int32_t* children, int i) {
  return bit(sm.broken, i) ? -1 : parent_len(s, sm, parents, children, i);
}

__global__ void __launch_bounds__(kThreads) fork_kernel(const PageState s, const int32_t* parents,
                                                         const int32_t* children, int n, int2* pairs) {
  __shared__ AllocSmem sm;
  const int lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i < kMaxPageList / 32; i += kThreads) sm.broken[i] = 0u;
  mark_rows(sm, children, n, s.rows);
  // a parent that names a page outside the pool or a free one: refused as a whole,
  // before any page is handed out
  for (int i = threadIdx.x >> 5; i < n; i += kThreads / 32) {
    const int pages = pages_of(max(parent_len(s, sm, parents, children, i), 0));
    const int32_t* from = s.table + static_cast<long long>(parents[i]) * s.max_pages;
    bool bad = false;
    for (int j = lane; j < pages; j += 32) {
      const int page = from[j];
      bad |= page < 0 || page >= s.num_pages || s.refcount[page] <= 0;
    }
    if (__any_sync(0xffffffffu, bad) && lane == 0) atomicOr(&sm.broken[i >> 5], 1u << (i & 31));
  }
  __syncthreads();
  scan_wants(sm, n, [&](int i) {
    const int len = forked(s, sm, parents, children, i);
    return len > 0 && (len & 63) != 0 ? 1 : 0;
  });
  const int want = sm.first[n];
  const int found = scan_free(sm, s.refcount, s.num_pages, want,
                              [&](int k, int page) { pairs[entry_of(sm, n, k)] = make_int2(-1, page); });
  // every entry is judged before any length changes (a child's length is read by its own entry only,
  // a parent's never written)
  for (int i = threadIdx.x >> 5; i < n; i += kThreads / 32) {
    const int len = forked(s, sm, parents, children, i);
    const bool tail = sm.first[i + 1] > sm.first[i];
    const bool served = len >= 0 && (!tail || sm.first[i + 1] <= found);
    __syncwarp();  // read by every lane before lane 0 writes the child's length
    if (!served) {
      if (lane == 0) {
        pairs[i] = make_int2(-1, -1);
        report(s.status, len < 0 ? MLA_ERR_BAD_INDEX : MLA_ERR_NO_PAGES);
      }
      continue;
    }
    const int full = len >> 6;
    const int32_t* from = s.table + static_cast<long long>(parents[i]) * s.max_pages;
    int32_t* to = s.table + static_cast<long long>(children[i]) * s.max_pages;
    for (int j = lane; j < s.max_pages; j += 32) {
      int page = -1;
      if (j < full) {
        page = from[j];
        atomicAdd(&s.refcount[page], 1);
      } else if (j == full && tail) {
        page = pairs[i].y;
      }
      to[j] = page;
    }
    __syncwarp();
    if (lane == 0) {
      if (tail) {
        pairs[i].x = from[full];
        s.refcount[pairs[i].y] = 1;
      } else {
        pairs[i] = make_int2(-1, -1);
      }
      s.seqlens[children[i]] = len;
    }
  }
}

// ------------------------------------------------------------------ free

// One warp per listed row.  The row's length is taken by an exchange, so a
// row listed twice is freed once, whichever entry gets there; a length out of
// range is no call's to take, and stays.
__global__ void __launch_bounds__(128) free_kernel(const PageState s, const int32_t* rows, int n) {
  const int lane = threadIdx.x & 31;
  const int i = blockIdx.x * 4 + (threadIdx.x >> 5);
  if (i >= n) return;
  const int r = rows[i];
  int len = -1;
  if (r >= 0 && r < s.rows && lane == 0) {
    len = *const_cast<volatile int32_t*>(&s.seqlens[r]);
    len = len < 0 || len > static_cast<long long>(s.max_pages) * kTile ? -1 : atomicExch(&s.seqlens[r], 0);
  }
  len = __shfl_sync(0xffffffffu, len, 0);
  if (len < 0) {
    if (lane == 0) report(s.status, MLA_ERR_BAD_INDEX);
    return;
  }
  int32_t* entry = s.table + static_cast<long long>(r) * s.max_pages;
  for (int j = lane; j < pages_of(len); j += 32) {
    const int page = entry[j];
    entry[j] = -1;
    if (page < 0 || page >= s.num_pages) {
      report(s.status, MLA_ERR_BAD_INDEX);
    } else if (atomicSub(&s.refcount[page], 1) <= 0) {
      atomicAdd(&s.refcount[page], 1);
      report(s.status, MLA_ERR_BAD_INDEX);
    }
  }
}

// ------------------------------------------------------------------ compact

constexpr int kChunk = 4096;           // pages per block: four a thread
constexpr int kStay = -2, kFree = -1;  // else: the page's ordinal among the moved ones

struct CompactWs {
  int32_t* live;  // [chunks] pages in use of each chunk
  int32_t* rank;  // [num_pages]
};

// Pages in use per chunk; the pair list starts out as (-1, -1).
__global__ void __launch_bounds__(kThreads) compact_count_kernel(const int32_t* refcount, int num_pages,
                                                                  CompactWs ws, int32_t* pairs) {
  __shared__ int scan[33];
  const int at = blockIdx.x * kChunk + threadIdx.x * 4;
  int mine = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (at + i < num_pages) mine += refcount[at + i] != 0;
    if (at + i < num_pages / 2 * 2) pairs[at + i] = -1;
  }
  int total;
  block_scan(mine, scan, &total);
  if (threadIdx.x == 0) ws.live[blockIdx.x] = total;
}

// Each moved page's ordinal and its pair.  With n pages in use and low of
// them below page n, the k-th moved page is the in-use page of rank low + k,
// and the k-th target the free page that k free ones precede.
__global__ void __launch_bounds__(kThreads) compact_place_kernel(const int32_t* refcount, int num_pages, int chunks,
                                                                  CompactWs ws, int2* pairs, int32_t* count) {
  __shared__ int scan[33];
  int before = 0, all = 0, total;
  for (int c = threadIdx.x; c < chunks; c += kThreads) {
    const int v = ws.live[c];
    all += v;
    if (c < static_cast<int>(blockIdx.x)) before += v;
  }
  block_scan(before, scan, &total);
  before = total;
  block_scan(all, scan, &total);
  const int n = total;
  int low = 0;  // in-use pages below page n
  const int nc = n / kChunk;
  for (int c = threadIdx.x; c < nc; c += kThreads) low += ws.live[c];
  for (int p = nc * kChunk + threadIdx.x; p < n; p += kThreads) low += refcount[p] != 0;
  block_scan(low, scan, &total);
  low = total;

  const int at = blockIdx.x * kChunk + threadIdx.x * 4;
  bool live[4];
  int mine = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    live[i] = at + i < num_pages && refcount[at + i] != 0;
    mine += live[i];
  }
  int rank = before + block_scan(mine, scan, &total);  // in-use pages before `at`
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int p = at + i;
    if (p >= num_pages) break;
    if (live[i]) {
      if (p >= n) {
        pairs[rank - low].x = p;
        ws.rank[p] = rank - low;
      } else {
        ws.rank[p] = kStay;
      }
      ++rank;
    } else {
      if (p < n) pairs[p - rank].y = p;
      ws.rank[p] = kFree;
    }
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) *count = n - low;
}

// Counts to their new places, and the tables' entries.
__global__ void __launch_bounds__(256) compact_apply_kernel(const PageState s, CompactWs ws, const int2* pairs,
                                                             const int32_t* count) {
  const long long stride = static_cast<long long>(gridDim.x) * blockDim.x;
  const long long first = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
  const int moved = *count;
  for (long long k = first; k < moved; k += stride) {
    const int2 m = pairs[k];
    s.refcount[m.y] = s.refcount[m.x];
    s.refcount[m.x] = 0;
  }
  const long long entries = static_cast<long long>(s.rows) * s.max_pages;
  for (long long e = first; e < entries; e += stride) {
    const int r = static_cast<int>(e / s.max_pages);
    const int col = static_cast<int>(e - static_cast<long long>(r) * s.max_pages);
    const int len = s.seqlens[r];
    if (col == 0 && (len < 0 || len > static_cast<long long>(s.max_pages) * kTile)) report(s.status, MLA_ERR_BAD_INDEX);
    if (len <= 0 || col >= pages_of(len)) continue;
    const int page = s.table[e];
    const int to = page >= 0 && page < s.num_pages ? ws.rank[page] : kFree;
    if (to == kFree)
      report(s.status, MLA_ERR_BAD_INDEX);
    else if (to >= 0)
      s.table[e] = pairs[to].y;
  }
}

// ------------------------------------------------------------------ copy

constexpr int kCopyThreads = 256;  // threads that copy a chunk together
constexpr int kCopyVec = 4;        // 16-byte loads a thread has in flight
constexpr int kCopyChunk = kCopyThreads * kCopyVec * 16;
// Lists of up to kLongList pairs: blocks of 256 threads that judge 2^7 pairs a
// pass.  Longer ones: a block of 1024 an SM, 2^12 pairs, so that an eighth of the
// blocks reads the list, and seldom twice.  (72 KB pages, short form and long: 16
// pairs of 4 layers 5.4 and 5.9 us, 337 of 8 layers 67 and 69, 4096 of one 103 and 103,
// 16384 392 and 390, 65536 1640 and 1526.  16-byte pages in the long form: 2^20 pairs 3.7
// ms, 2^22 39, 2^24 543.)
constexpr int kShortPairs = 7, kLongPairs = 12;
constexpr int kLongGroups = 4, kLongList = 8192;

// The targets of the pairs a block is judging, by open addressing: page
// key[i] (-1: none) and the first pair of the whole list that has it as its
// target, or -1 once a pair that reads it is met.
template <int kLogPairs>
struct Judge {
  static constexpr int kPairs = 1 << kLogPairs;  // judged in one pass over the list
  static constexpr int kSlots = 2 * kPairs;      // at most half of them taken: a search ends at a free one
  int key[kSlots];
  int first[kSlots];
  int2 pair[kPairs];

  static __device__ __forceinline__ int slot_of(int page) {
    return static_cast<int>(static_cast<uint32_t>(page) * 2654435761u >> (31 - kLogPairs));
  }

  // The place of a page, or -1.
  __device__ __forceinline__ int find(int page) const {
    for (int i = slot_of(page);; i = (i + 1) & (kSlots - 1)) {
      const int k = key[i];
      if (k == page) return i;
      if (k < 0) return -1;
    }
  }

  // Read pairs from .. to - 1 (at most kPairs) and judge their targets against
  // the list, by the whole block.
  __device__ __forceinline__ void fill(const int2* pairs, int n, int from, int to) {
    const int threads = blockDim.x;
    __syncthreads();  // the pairs before are done with
    for (int i = threadIdx.x; i < kSlots; i += threads) {
      key[i] = -1;
      first[i] = INT32_MAX;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < to - from; i += threads) {
      const int2 m = pairs[from + i];
      pair[i] = m;
      if (m.y < 0) continue;
      for (int k = slot_of(m.y);; k = (k + 1) & (kSlots - 1)) {
        const int was = atomicCAS(&key[k], -1, m.y);
        if (was == -1 || was == m.y) break;
      }
    }
    __syncthreads();
    constexpr int kAhead = 4;
    for (int j0 = threadIdx.x; j0 < n; j0 += threads * kAhead) {
      int2 o[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int j = j0 + i * threads;
        o[i] = j < n ? pairs[j] : make_int2(-1, -1);
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int target = o[i].y < 0 ? -1 : find(o[i].y);
        if (target >= 0) atomicMin(&first[target], j0 + i * threads);
        const int source = o[i].x < 0 || o[i].x == o[i].y ? -1 : find(o[i].x);
        if (source >= 0) atomicMin(&first[source], -1);
      }
    }
    __syncthreads();
  }
};

// Bound by HBM: each page is read and written once.  The blocks take equal
// runs of (pair, layer, 16 KB chunk) items in that order, so that a block
// judges a pair against the list once for all its layers and chunks, many
// pairs in one pass over the list (two look-ups a pair of it).  kGroups groups
// of 256 threads copy a chunk each.
template <int kGroups, int kLogPairs>
__global__ void __launch_bounds__(kCopyThreads* kGroups, kGroups == 1 ? 5 : 1)
    copy_pages_kernel(uint8_t* pool, int layers, long long layer_stride, int num_pages, long long page_bytes,
                      const int2* pairs, const int32_t* count, int n, int32_t* status) {
  if (count != nullptr) n = max(0, min(n, *count));
  const long long chunks = (page_bytes + kCopyChunk - 1) / kCopyChunk;
  const long long per_pair = chunks * layers;
  const long long items = per_pair * n;
  const long long lo = items * blockIdx.x / gridDim.x, hi = items * (blockIdx.x + 1) / gridDim.x;
  if (lo >= hi) return;
  const int last = static_cast<int>((hi - 1) / per_pair);  // this block's last pair
  const int tid = threadIdx.x % kCopyThreads, group = threadIdx.x / kCopyThreads;
  extern __shared__ __align__(16) uint8_t copy_smem[];
  Judge<kLogPairs>& judge = *reinterpret_cast<Judge<kLogPairs>*>(copy_smem);
  for (int from = static_cast<int>(lo / per_pair), to; from <= last; from = to) {
    to = min(last + 1, from + judge.kPairs);
    judge.fill(pairs, n, from, to);
    const long long end = min(hi, to * per_pair);
    int cur = -1;
    bool go = false;
    int2 m = make_int2(-1, -1);
    for (long long it = max(lo, from * per_pair) + group; it < end;) {
      const int pair = static_cast<int>(it / per_pair);
      if (pair != cur) {
        cur = pair;
        m = judge.pair[pair - from];
        go = !(m.x < 0 && m.y < 0) && m.x != m.y;
        if (go && (m.x < 0 || m.y < 0 || m.x >= num_pages || m.y >= num_pages ||
                   judge.first[judge.find(m.y)] < pair)) {
          if (tid == 0) report(status, MLA_ERR_BAD_INDEX);
          go = false;
        }
      }
      if (!go) {  // this group's first item of the next pair
        it += ((pair + 1) * per_pair - it + kGroups - 1) / kGroups * kGroups;
        continue;
      }
      const long long rest = it - pair * per_pair;
      const long long layer = rest / chunks, chunk = rest - layer * chunks;
      uint8_t* base = pool + layer * layer_stride;
      const uint8_t* src = base + m.x * page_bytes;
      uint8_t* dst = base + m.y * page_bytes;
      uint4 v[kCopyVec];
#pragma unroll
      for (int i = 0; i < kCopyVec; ++i) {
        const long long off = chunk * kCopyChunk + (i * kCopyThreads + tid) * 16ll;
        if (off < page_bytes) v[i] = __ldcs(reinterpret_cast<const uint4*>(src + off));
      }
#pragma unroll
      for (int i = 0; i < kCopyVec; ++i) {
        const long long off = chunk * kCopyChunk + (i * kCopyThreads + tid) * 16ll;
        if (off < page_bytes) __stcs(reinterpret_cast<uint4*>(dst + off), v[i]);
      }
      it += kGroups;
    }
  }
}

}  // namespace

cudaError_t launch_grow(const PageState& s, const int32_t* rows, const int32_t* new_tokens, int n, cudaStream_t st) {
  grow_kernel<<<1, kThreads, 0, st>>>(s, rows, new_tokens, n);
  return cudaGetLastError();
}

cudaError_t launch_fork(const PageState& s, const int32_t* parents, const int32_t* children, int n, int32_t* pairs,
                        cudaStream_t st) {
  fork_kernel<<<1, kThreads, 0, st>>>(s, parents, children, n, reinterpret_cast<int2*>(pairs));
  return cudaGetLastError();
}

cudaError_t launch_free(const PageState& s, const int32_t* rows, int n, cudaStream_t st) {
  free_kernel<<<ceil_div_i(n, 4), 128, 0, st>>>(s, rows, n);
  return cudaGetLastError();
}

namespace {
size_t live_bytes(int num_pages) { return (static_cast<size_t>((num_pages + kChunk - 1) / kChunk) * 4 + 255) / 256 * 256; }
}  // namespace

size_t compact_workspace_bytes(int num_pages) {
  return live_bytes(num_pages) + static_cast<size_t>(num_pages) * 4;
}

cudaError_t launch_compact(const PageState& s, int32_t* pairs, int32_t* count, void* ws, cudaStream_t st) {
  CompactWs w;
  w.live = static_cast<int32_t*>(ws);
  w.rank = reinterpret_cast<int32_t*>(static_cast<char*>(ws) + live_bytes(s.num_pages));
  const int chunks = ceil_div_i(s.num_pages, kChunk);
  compact_count_kernel<<<chunks, kThreads, 0, st>>>(s.refcount, s.num_pages, w, pairs);
  compact_place_kernel<<<chunks, kThreads, 0, st>>>(s.refcount, s.num_pages, chunks, w,
                                                    reinterpret_cast<int2*>(pairs), count);
  const long long work = static_cast<long long>(s.rows) * s.max_pages;
  const long long most = work > s.num_pages / 2 ? work : s.num_pages / 2;
  const long long blocks = (most + 255) / 256;
  compact_apply_kernel<<<static_cast<int>(blocks < 1 ? 1 : blocks > 1216 ? 1216 : blocks), 256, 0, st>>>(
      s, w, reinterpret_cast<const int2*>(pairs), count);
  return cudaGetLastError();
}

cudaError_t copy_pages_setup() {
  return cudaFuncSetAttribute(reinterpret_cast<const void*>(copy_pages_kernel<kLongGroups, kLongPairs>),
                              cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(Judge<kLongPairs>));
}

cudaError_t launch_copy_pages(void* pool, int layers, long long layer_stride, int num_pages, long long page_bytes,
                              const int32_t* pairs, const int32_t* count, int n, int32_t* status, int sms,
                              cudaStream_t st) {
  const long long items = (page_bytes + kCopyChunk - 1) / kCopyChunk * layers * n;
  const bool many = n > kLongList;
  const long long most = many ? sms : 8ll * sms;  // as many blocks as are resident
  const int blocks = static_cast<int>(items < most ? items : most);
  uint8_t* base = static_cast<uint8_t*>(pool);
  const int2* list = reinterpret_cast<const int2*>(pairs);
  if (many)
    copy_pages_kernel<kLongGroups, kLongPairs><<<blocks, kCopyThreads * kLongGroups, sizeof(Judge<kLongPairs>), st>>>(
        base, layers, layer_stride, num_pages, page_bytes, list, count, n, status);
  else
    copy_pages_kernel<1, kShortPairs><<<blocks, kCopyThreads, sizeof(Judge<kShortPairs>), st>>>(
        base, layers, layer_stride, num_pages, page_bytes, list, count, n, status);
  return cudaGetLastError();
}

}  // namespace mla
