// Page upkeep of the paged key-value cache: pages taken for more tokens
// (extend), sequences forked, freed and the pool compacted, all on the device,
// so that a serving loop, or a captured graph of one, never waits for the host
// to learn which pages are free.
//
// Which pages: a page is free where its count in refs is 0, and the lowest free
// ones are taken in list order, found by a prefix sum over refs.  Nothing
// depends on the order of atomics: claims of a sequence go to the lowest list
// entry, counts are sums.  One workgroup plans, a thread per 32-page run of refs
// and round (32 Ki pages); then a thread per page taken or moved finds its page
// by its rank, so a run of free pages is not one thread's work.  The grid that
// follows copies.  Measured: pages for two prompts of 1021 tokens 5.5 us, all of it
// the way through loads, sums and ranks; 500 of 2560 pages of 24 layers moved in 83 us
// (4.7 TB/s, a copy's rate) behind a plan of 5.3.
#include <climits>

#include "kv_cache.h"

namespace pesti {

constexpr int kPlanThreads = 1024;
constexpr int kRun = 32;   // pages per thread and round of a plan

// v plus what DPP brings of it: the lanes whose bit is in ROWS from the place that
// CTRL names, the others 0.
template <int CTRL, int ROWS>
__device__ __forceinline__ int64_t plus_dpp(int64_t v) {
#ifdef __HIP_DEVICE_COMPILE__
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, static_cast<int>(v), CTRL, ROWS, 0xF, false);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, static_cast<int>(v >> 32), CTRL, ROWS, 0xF, false);
  v += static_cast<int64_t>(static_cast<uint64_t>(hi) << 32 | lo);
#endif
  return v;
}

// Exclusive sum over a plan's threads; *total gets the sum.
__device__ __forceinline__ int64_t plan_scan(int64_t v, int64_t* total, int64_t* wave_sums) {
  typedef int64_t T;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  T s = plus_dpp<0x111, 0xF>(v);   // rows of 16 lanes: one, two, four, eight lanes up
  s = plus_dpp<0x112, 0xF>(s);
  s = plus_dpp<0x114, 0xF>(s);
  s = plus_dpp<0x118, 0xF>(s);
  s = plus_dpp<0x142, 0xA>(s);     // rows 1 and 3: the last lane of the row before
  s = plus_dpp<0x143, 0xC>(s);     // rows 2 and 3: lane 31
  __syncthreads();   // the sums of the call before have been read
  if (lane == 63) wave_sums[wave] = s;
  __syncthreads();
  T before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kPlanThreads / 64; ++w) {
    const T x = wave_sums[w];
    before += w < wave ? x : 0;
    all += x;
  }
  *total = all;
  return before + s - v;
}

// Bit j: page first + j exists and is free (or, with live, is held).
__device__ __forceinline__ uint32_t run_mask(const KvArgs& a, int32_t first, bool live) {
  uint32_t held = 0;
  if (first + kRun <= a.pages) {
    u32x4 r[kRun / 4];
#pragma unroll
    for (int j = 0; j < kRun / 4; ++j) r[j] = load_u32x4(a.refs + first + 4 * j);
#pragma unroll
    for (int j = 0; j < kRun; ++j) held |= static_cast<uint32_t>(static_cast<int32_t>(r[j / 4][j % 4]) > 0) << j;
    return live ? held : ~held;
  }
  const int32_t n = a.pages - first;   // the last run, or one past the end
  for (int j = 0; j < n; ++j) held |= static_cast<uint32_t>(a.refs[first + j] > 0) << j;
  return live ? held : (n > 0 ? ~held & ((1u << n) - 1) : 0u);
}

// The pages of a round by rank: runs' exclusive counts and bits in LDS.
struct RoundLds {
  int32_t before[kPlanThreads];
  uint32_t bits[kPlanThreads];
};
__device__ __forceinline__ int32_t page_of_rank(const RoundLds& r, int32_t rank, int32_t base) {
  int lo = 0;   // the last run with before <= rank holds it: it has pages, those behind it start later
#pragma unroll
  for (int step = kPlanThreads / 2; step > 0; step /= 2)
    if (r.before[lo + step] <= rank) lo += step;
  uint32_t m = r.bits[lo];
  int k = rank - r.before[lo], at = 0;   // the k-th set bit
#pragma unroll
  for (int half = 16; half > 0; half /= 2) {
    const int n = __popc(m & ((1u << half) - 1));
    if (k >= n) {
      k -= n;
      m >>= half;
      at += half;
    }
  }
  return base + lo * kRun + at;
}

struct TakeArgs {
  KvArgs kv;
  int32_t n;
  const int32_t* list;     // extend: seq_ids or null; fork: children
  const int32_t* second;   // extend: counts or null; fork: parents
  int32_t* status;
  int4* plan;              // fork: per pair the page copied from and to (-1: none), whole pages, whether it counts
};

// extend: takes the pages and sets the lengths.  fork: the same for the last
// pages of the children, and writes the plan that fork_kernel follows.
template <bool FORK>
__global__ __launch_bounds__(kPlanThreads) void take_kernel(TakeArgs t) {
  __shared__ int32_t claim[PESTI_MAX_SEQS];   // lowest list entry that names the sequence; then each entry's pages before (extend) or parent's last page (fork)
  __shared__ int32_t start[PESTI_MAX_SEQS];   // pages taken by the entries before
  __shared__ int32_t after[PESTI_MAX_SEQS];   // tokens after the call, -1 where the entry does not count
  __shared__ RoundLds round;
  __shared__ int64_t sums[kPlanThreads / 64];
  const KvArgs& a = t.kv;
  const int tid = threadIdx.x, page = 1 << a.page_shift;
  const uint32_t mask0 = run_mask(a, tid * kRun, false);   // the first round's, asked for ahead of all else
  for (int i = tid; i < a.seqs; i += kPlanThreads) claim[i] = INT_MAX;
  __syncthreads();
  auto seq = [&](int i) { return t.list ? t.list[i] : i; };
  auto named = [&](int32_t s) { return static_cast<uint32_t>(s) < static_cast<uint32_t>(a.seqs); };
  constexpr int kEntries = PESTI_MAX_SEQS / kPlanThreads;
  int32_t mine[kEntries];   // the sequences of the thread's entries (a load behind the stores at the end would wait for them)
#pragma unroll
  for (int j = 0; j < kEntries; ++j) {
    const int i = j * kPlanThreads + tid;
    mine[j] = -1;
    if (i >= t.n) continue;
    mine[j] = seq(i);
    if (!named(mine[j])) continue;
    if (FORK && !named(t.second[i])) continue;
    atomicMin(&claim[mine[j]], i);
  }
  __syncthreads();
  int64_t total = 0, free_before = 0, free_here = 0;   // pages needed; free ones of the first round, before the thread's and all
  bool outgrown = false;
  int32_t info[kEntries];   // of the thread's entries, until the claims have been read
#pragma unroll
  for (int j = 0; j < kEntries; ++j) {
    const int i = j * kPlanThreads + tid;
    info[j] = 0;
    if (j * kPlanThreads >= t.n) continue;
    int64_t need = 0;
    if (i < t.n) {
      const int32_t s = mine[j];
      int64_t len = -1;
      if (named(s) && claim[s] == i) {
        const int32_t old = kv_length(a, s);
        if constexpr (FORK) {
          const int32_t parent = t.second[i], tokens = kv_length(a, parent);
          if (old == 0) {
            len = tokens;
            need = (len & (page - 1)) != 0;
            if (need) info[j] = a.table[static_cast<int64_t>(parent) * a.width + (len >> a.page_shift)];
          }
        } else {
          const int32_t more = t.second ? t.second[i] : 1;
          len = static_cast<int64_t>(old) + (more > 0 ? more : 0);
          if (len > static_cast<int64_t>(a.width) << a.page_shift) {
            outgrown = true;
            len = old;
          }
          info[j] = kv_pages_of(a, old);
          need = kv_pages_of(a, static_cast<int32_t>(len)) - info[j];
        }
      }
      after[i] = static_cast<int32_t>(len);
    }
    // one sum for both: free pages of a round are 2^15 at most, pages that 1024
    // sequences need 2^37
    int64_t sum, before = plan_scan(need << 16 | (j == 0 ? __popc(mask0) : 0), &sum, sums);
    if (j == 0) {
      free_before = before & 0xFFFF;
      free_here = sum & 0xFFFF;
    }
    before >>= 16;
    if (i < t.n) start[i] = static_cast<int32_t>(total + before);   // used where total <= pages
    total += sum >> 16;
  }
  int64_t missing = __syncthreads_or(outgrown) ? -1 : 0;
#pragma unroll
  for (int j = 0; j < kEntries; ++j)
    if (j * kPlanThreads + tid < t.n) claim[j * kPlanThreads + tid] = info[j];
  constexpr int32_t kRound = kPlanThreads * kRun;
  int64_t found = 0, sum = free_here, before = free_before;
  if (missing == 0 && total > 0) {
    found = sum;
    for (int32_t base = kRound; base < a.pages && found < total; base += kRound) {
      int64_t more;
      plan_scan(static_cast<int64_t>(__popc(run_mask(a, base + tid * kRun, false))), &more, sums);
      found += more;
    }
    if (found < total) missing = total - found;
  }
  if (missing != 0) {
    if (tid == 0) *t.status = static_cast<int32_t>(missing < INT_MAX ? missing : INT_MAX);
    if constexpr (FORK)
      for (int i = tid; i < t.n; i += kPlanThreads) t.plan[i] = make_int4(-1, -1, 0, 0);
    return;
  }
  __syncthreads();   // claim holds the entries' places now
  found = 0;
  for (int32_t base = 0; found < total; base += kRound) {
    uint32_t m = mask0;
    if (base > 0) {
      m = run_mask(a, base + tid * kRun, false);
      before = plan_scan(static_cast<int64_t>(__popc(m)), &sum, sums);
    }
    round.before[tid] = static_cast<int32_t>(before);
    round.bits[tid] = m;
    __syncthreads();
    const int32_t here = static_cast<int32_t>(sum < total - found ? sum : total - found);
    for (int32_t r = tid; r < here; r += kPlanThreads) {
      const int32_t p = page_of_rank(round, r, base), rank = static_cast<int32_t>(found) + r;
      int lo = 0, hi = t.n;   // the entry with start <= rank < its end
      while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (start[mid] <= rank) lo = mid; else hi = mid;
      }
      int32_t* row = a.table + static_cast<int64_t>(seq(lo)) * a.width;
      a.refs[p] = 1;
      if constexpr (FORK) {
        row[after[lo] >> a.page_shift] = p;
        t.plan[lo] = make_int4(kv_page_ok(a, claim[lo]) ? claim[lo] : -1, p, after[lo] >> a.page_shift, 1);
      } else {
        row[claim[lo] + rank - start[lo]] = p;
      }
    }
    found += sum;
    __syncthreads();   // the round's runs have been read
  }
#pragma unroll
  for (int j = 0; j < kEntries; ++j) {
    const int i = j * kPlanThreads + tid;
    if (i >= t.n) continue;
    if (after[i] >= 0) a.lengths[mine[j]] = after[i];
    if constexpr (FORK)   // (pairs whose last page is copied have theirs)
      if (after[i] < 0 || (after[i] & (page - 1)) == 0)
        t.plan[i] = make_int4(-1, -1, after[i] < 0 ? 0 : after[i] >> a.page_shift, after[i] >= 0);
  }
  if (tid == 0) *t.status = 0;
}

// One workgroup per list entry: whoever takes the length gives the pages back.
__global__ __launch_bounds__(256) void free_kernel(KvArgs a, const int32_t* list) {
  __shared__ int32_t tokens;
  const int32_t s = list ? list[blockIdx.x] : static_cast<int32_t>(blockIdx.x);
  if (static_cast<uint32_t>(s) >= static_cast<uint32_t>(a.seqs)) return;
  if (threadIdx.x == 0) {
    const int64_t n = atomicExch(&a.lengths[s], 0), most = static_cast<int64_t>(a.width) << a.page_shift;
    tokens = static_cast<int32_t>(n < 0 ? 0 : (n > most ? most : n));
  }
  __syncthreads();
  int32_t* row = a.table + static_cast<int64_t>(s) * a.width;
  const int32_t held = kv_pages_of(a, tokens);
  for (int32_t j = threadIdx.x; j < held; j += 256) {
    const int32_t p = row[j];
    row[j] = -1;
    if (kv_page_ok(a, p)) atomicSub(&a.refs[p], 1);
  }
}

// Pairs of pages to copy: entry i at src[i * stride], dst[i * stride]; count in
// device memory, or n.
struct CopyArgs {
  KvArgs kv;
  int64_t n;
  const int32_t* count;
  const int32_t* src;
  const int32_t* dst;
  int32_t stride;
};

constexpr int kCopyThreads = 256;
constexpr int kCopyVectors = 4;   // 16-byte vectors per thread in flight
constexpr int64_t kCopyChunk = kCopyThreads * kCopyVectors * 16;

// A page of one layer of K or V, its scales behind it, is cut into chunks; a
// workgroup takes chunks in turn.
__device__ __forceinline__ void copy_pages(const CopyArgs& c, int64_t group, int64_t groups) {
  const KvArgs& a = c.kv;
  const int64_t n = c.count ? *c.count : c.n;
  const int64_t scale_bytes = a.k_scales ? 4 * a.page_rows : 0, bytes = a.page_bytes + scale_bytes;
  const int64_t chunks = (bytes + kCopyChunk - 1) / kCopyChunk, planes = 2 * static_cast<int64_t>(a.layers);
  const int64_t units = n * planes * chunks;
  for (int64_t u = group; u < units; u += groups) {
    const int64_t chunk = u % chunks, rest = u / chunks, plane = rest % planes, i = rest / planes;
    const int32_t from = c.src[i * c.stride], to = c.dst[i * c.stride];
    if (!kv_page_ok(a, from) || !kv_page_ok(a, to) || from == to) continue;
    const int64_t layer = plane >> 1;
    uint8_t* data = (plane & 1) ? a.v : a.k;
    uint8_t* scales = reinterpret_cast<uint8_t*>((plane & 1) ? a.v_scales : a.k_scales);
    const int64_t page0 = layer * a.pages;
    const uint8_t* s_data = data + (page0 + from) * a.page_bytes;
    uint8_t* d_data = data + (page0 + to) * a.page_bytes;
    const uint8_t* s_scale = scales + (page0 + from) * scale_bytes - a.page_bytes;
    uint8_t* d_scale = scales + (page0 + to) * scale_bytes - a.page_bytes;
    u32x4a v[kCopyVectors];
#pragma unroll
    for (int j = 0; j < kCopyVectors; ++j) {
      const int64_t o = chunk * kCopyChunk + (j * kCopyThreads + threadIdx.x) * 16;
      if (o < bytes) v[j] = *reinterpret_cast<const u32x4a*>((o < a.page_bytes ? s_data : s_scale) + o);
    }
#pragma unroll
    for (int j = 0; j < kCopyVectors; ++j) {
      const int64_t o = chunk * kCopyChunk + (j * kCopyThreads + threadIdx.x) * 16;
      if (o < bytes) *reinterpret_cast<u32x4a*>((o < a.page_bytes ? d_data : d_scale) + o) = v[j];
    }
  }
}

__global__ __launch_bounds__(kCopyThreads) void copy_kernel(CopyArgs c) { copy_pages(c, blockIdx.x, gridDim.x); }

// The first n workgroups share the parents' whole pages with the children, the
// others copy last pages.
__global__ __launch_bounds__(kCopyThreads) void fork_kernel(CopyArgs c, const int4* plan, const int32_t* parents,
                                                            const int32_t* children) {
  const KvArgs& a = c.kv;
  const int32_t n = static_cast<int32_t>(c.n), b = static_cast<int32_t>(blockIdx.x);
  if (b >= n) return copy_pages(c, b - n, gridDim.x - n);
  if (!plan[b].w) return;
  const int32_t* from = a.table + static_cast<int64_t>(parents[b]) * a.width;
  int32_t* to = a.table + static_cast<int64_t>(children[b]) * a.width;
  for (int32_t j = threadIdx.x; j < plan[b].z; j += kCopyThreads) {
    const int32_t p = from[j];
    to[j] = p;
    if (kv_page_ok(a, p)) atomicAdd(&a.refs[p], 1);
  }
}

struct CompactArgs {
  KvArgs kv;
  int32_t* live;
  int32_t* moves;   // how many
  int32_t* src;
  int32_t* dst;
  int32_t* map;     // where each page is afterwards
};

__global__ __launch_bounds__(kPlanThreads) void compact_plan_kernel(CompactArgs c) {
  __shared__ int64_t sums[kPlanThreads / 64];
  __shared__ RoundLds hole_runs, mover_runs;
  const KvArgs& a = c.kv;
  const int tid = threadIdx.x;
  constexpr int32_t kRound = kPlanThreads * kRun;
  const uint32_t mask0 = run_mask(a, tid * kRun, true);
  int64_t live = 0, sum;
  for (int32_t base = 0; base < a.pages; base += kRound) {
    plan_scan(static_cast<int64_t>(__popc(base == 0 ? mask0 : run_mask(a, base + tid * kRun, true))), &sum, sums);
    live += sum;
  }
  int64_t holes = 0, movers = 0;
  for (int32_t base = 0; base < a.pages; base += kRound) {
    const int32_t first = base + tid * kRun;
    const uint32_t held = base == 0 ? mask0 : run_mask(a, first, true);
    const int64_t room = live - first;   // pages of the run below the border; all of those exist
    const uint32_t below = room >= 32 ? 0xFFFFFFFFu : (room <= 0 ? 0u : (1u << room) - 1);
    const uint32_t hole = ~held & below, mover = held & ~below;
    const int64_t before = plan_scan((static_cast<int64_t>(__popc(hole)) << 32) | __popc(mover), &sum, sums);
    hole_runs.before[tid] = static_cast<int32_t>(before >> 32);
    hole_runs.bits[tid] = hole;
    mover_runs.before[tid] = static_cast<int32_t>(before & 0xFFFFFFFF);
    mover_runs.bits[tid] = mover;
    __syncthreads();
    const int32_t new_holes = static_cast<int32_t>(sum >> 32), new_movers = static_cast<int32_t>(sum & 0xFFFFFFFF);
    for (int32_t r = tid; r < new_holes; r += kPlanThreads) c.dst[holes + r] = page_of_rank(hole_runs, r, base);
    for (int32_t i = tid; i < kRound && base + i < a.pages; i += kPlanThreads)
      if (!(mover_runs.bits[i / kRun] >> (i % kRun) & 1)) c.map[base + i] = base + i;
    __syncthreads();   // a mover's hole lies before it: it stands in dst now
    for (int32_t r = tid; r < new_movers; r += kPlanThreads) {
      const int32_t p = page_of_rank(mover_runs, r, base), to = c.dst[movers + r];
      c.src[movers + r] = p;
      c.map[p] = to;
      a.refs[to] = a.refs[p];
      a.refs[p] = 0;
    }
    holes += new_holes;
    movers += new_movers;
    __syncthreads();   // the round's runs have been read
  }
  if (tid == 0) {
    *c.live = static_cast<int32_t>(live);
    *c.moves = static_cast<int32_t>(movers);
  }
}

// The first seqs workgroups rewrite the sequences' page numbers, the others
// copy pages.
__global__ __launch_bounds__(kCopyThreads) void compact_kernel(CopyArgs c, const int32_t* map) {
  const KvArgs& a = c.kv;
  const int32_t b = static_cast<int32_t>(blockIdx.x);
  if (b >= a.seqs) return copy_pages(c, b - a.seqs, gridDim.x - a.seqs);
  int32_t* row = a.table + static_cast<int64_t>(b) * a.width;
  const int32_t held = kv_pages_of(a, kv_length(a, b));
  for (int32_t j = threadIdx.x; j < held; j += kCopyThreads) {
    const int32_t p = row[j];
    if (kv_page_ok(a, p)) row[j] = map[p];
  }
}

}  // namespace pesti

namespace {

using pesti::CompactArgs;
using pesti::CopyArgs;
using pesti::KvArgs;
using pesti::TakeArgs;

// Every check of a call on lists of n sequences, up to the device.
int check(const pesti_kv_cache* cache, const pesti_kv_table* table, int64_t n, bool pages) {
  int st = pesti_kv::check_sizes(cache);
  if (st == PESTI_OK) st = pesti_kv::check_table_sizes(cache, table);
  if (st != PESTI_OK) return st;
  if (n < 0 || n > PESTI_MAX_SEQS) return PESTI_ERR_BATCH;
  if (n == 0) return PESTI_OK;
  st = pesti_kv::check_table(cache, table, true);
  if (st == PESTI_OK && pages) st = pesti_kv::check_pages(cache);
  return st;
}

int device() {
  int dev = 0;
  size_t lds = 0;
  return pesti_host::current_device(&dev, &lds);
}

// Workgroups for copies of up to n pairs: enough to fill the chip four times.
unsigned copy_groups(const KvArgs& a, int64_t n) {
  const int64_t bytes = a.page_bytes + (a.k_scales ? 4 * a.page_rows : 0);
  const int64_t units = n * 2 * a.layers * ((bytes + pesti::kCopyChunk - 1) / pesti::kCopyChunk);
  return pesti_host::grid_for(units, 2048);
}

constexpr int64_t kHead = 64;   // bytes before the lists in a workspace

int64_t workspace_bytes(int64_t pages, int64_t seqs) {
  const int64_t fork = 16 * seqs, compact = 4 * (2 * (pages / 2 + 1) + pages);
  return (kHead + (fork > compact ? fork : compact) + 15) & ~int64_t{15};
}

int check_workspace(const pesti_kv_cache* cache, const pesti_kv_table* table, const void* ws, int64_t bytes) {
  if (!ws || bytes < workspace_bytes(cache->pages, table->seqs)) return PESTI_ERR_WORKSPACE;
  return pesti_host::aligned(ws, 16) ? PESTI_OK : PESTI_ERR_ALIGN;
}

}  // namespace

extern "C" {

int64_t pesti_cache_workspace_bytes(const pesti_kv_cache* cache, const pesti_kv_table* table) {
  int st = pesti_kv::check_sizes(cache);
  if (st == PESTI_OK) st = pesti_kv::check_table_sizes(cache, table);
  return st != PESTI_OK ? st : workspace_bytes(cache->pages, table->seqs);
}

int pesti_cache_extend(const pesti_kv_cache* cache, const pesti_kv_table* table, int64_t n,
                       const int32_t* seq_ids, const int32_t* counts, int32_t* status, void* stream) {
  int st = check(cache, table, n, false);
  if (st != PESTI_OK || n == 0) return st;
  if (!status) return PESTI_ERR_NULL;
  if (!pesti_host::aligned(seq_ids, 4) || !pesti_host::aligned(counts, 4) || !pesti_host::aligned(status, 4))
    return PESTI_ERR_ALIGN;
  if ((st = device()) != PESTI_OK) return st;
  TakeArgs t{pesti_kv::args_of(cache, table), static_cast<int32_t>(n), seq_ids, counts, status, nullptr};
  void* params[] = {&t};
  return pesti_kv::launch(reinterpret_cast<const void*>(&pesti::take_kernel<false>), dim3(1), dim3(pesti::kPlanThreads),
                          params, 0, static_cast<hipStream_t>(stream));
}

int pesti_cache_fork(const pesti_kv_cache* cache, const pesti_kv_table* table, int64_t n, const int32_t* parents,
                     const int32_t* children, int32_t* status, void* workspace, int64_t workspace_bytes,
                     void* stream) {
  int st = check(cache, table, n, true);
  if (st != PESTI_OK || n == 0) return st;
  if (!parents || !children || !status) return PESTI_ERR_NULL;
  if (!pesti_host::aligned(parents, 4) || !pesti_host::aligned(children, 4) || !pesti_host::aligned(status, 4))
    return PESTI_ERR_ALIGN;
  if ((st = check_workspace(cache, table, workspace, workspace_bytes)) != PESTI_OK) return st;
  // A child is listed once: pairs past the number of slots cannot all count, but their plans need room.
  if (n > table->seqs) return PESTI_ERR_BATCH;
  if ((st = device()) != PESTI_OK) return st;
  const hipStream_t sh = static_cast<hipStream_t>(stream);
  int4* plan = reinterpret_cast<int4*>(static_cast<uint8_t*>(workspace) + kHead);
  TakeArgs t{pesti_kv::args_of(cache, table), static_cast<int32_t>(n), children, parents, status, plan};
  void* take_params[] = {&t};
  st = pesti_kv::launch(reinterpret_cast<const void*>(&pesti::take_kernel<true>), dim3(1), dim3(pesti::kPlanThreads),
                        take_params, 0, sh);
  if (st != PESTI_OK) return st;
  CopyArgs c{t.kv, n, nullptr, &plan[0].x, &plan[0].y, 4};
  void* params[] = {&c, &plan, &parents, &children};
  return pesti_kv::launch(reinterpret_cast<const void*>(&pesti::fork_kernel),
                          dim3(static_cast<unsigned>(n) + copy_groups(t.kv, n)), dim3(pesti::kCopyThreads), params, 0, sh);
}

int pesti_cache_free(const pesti_kv_cache* cache, const pesti_kv_table* table, int64_t n, const int32_t* seq_ids,
                     void* stream) {
  int st = check(cache, table, n, false);
  if (st != PESTI_OK || n == 0) return st;
  if (!pesti_host::aligned(seq_ids, 4)) return PESTI_ERR_ALIGN;
  if ((st = device()) != PESTI_OK) return st;
  KvArgs a = pesti_kv::args_of(cache, table);
  void* params[] = {&a, &seq_ids};
  return pesti_kv::launch(reinterpret_cast<const void*>(&pesti::free_kernel), dim3(static_cast<unsigned>(n)), dim3(256),
                          params, 0, static_cast<hipStream_t>(stream));
}

int pesti_cache_compact(const pesti_kv_cache* cache, const pesti_kv_table* table, int32_t* live, void* workspace,
                        int64_t workspace_bytes, void* stream) {
  int st = check(cache, table, 1, true);
  if (st != PESTI_OK) return st;
  if (!live) return PESTI_ERR_NULL;
  if (!pesti_host::aligned(live, 4)) return PESTI_ERR_ALIGN;
  if ((st = check_workspace(cache, table, workspace, workspace_bytes)) != PESTI_OK) return st;
  if ((st = device()) != PESTI_OK) return st;
  const hipStream_t sh = static_cast<hipStream_t>(stream);
  const KvArgs a = pesti_kv::args_of(cache, table);
  const int64_t most = cache->pages / 2 + 1;
  int32_t* head = static_cast<int32_t*>(workspace);
  int32_t* src = head + kHead / 4;
  CompactArgs p{a, live, head, src, src + most, src + 2 * most};
  void* plan_params[] = {&p};
  st = pesti_kv::launch(reinterpret_cast<const void*>(&pesti::compact_plan_kernel), dim3(1), dim3(pesti::kPlanThreads),
                        plan_params, 0, sh);
  if (st != PESTI_OK) return st;
  CopyArgs c{a, 0, p.moves, p.src, p.dst, 1};
  const int32_t* map = p.map;
  void* params[] = {&c, &map};
  return pesti_kv::launch(reinterpret_cast<const void*>(&pesti::compact_kernel),
                          dim3(static_cast<unsigned>(table->seqs) + copy_groups(a, most)), dim3(pesti::kCopyThreads),
                          params, 0, sh);
}

int pesti_cache_copy_pages(const pesti_kv_cache* cache, int64_t n, const int32_t* src, const int32_t* dst,
                           void* stream) {
  int st = pesti_kv::check_sizes(cache);
  if (st != PESTI_OK) return st;
  if (n < 0 || n > PESTI_MAX_PAGES) return PESTI_ERR_BATCH;
  if (n == 0) return PESTI_OK;
  if ((st = pesti_kv::check_pages(cache)) != PESTI_OK) return st;
  if (!src || !dst) return PESTI_ERR_NULL;
  if (!pesti_host::aligned(src, 4) || !pesti_host::aligned(dst, 4)) return PESTI_ERR_ALIGN;
  if ((st = device()) != PESTI_OK) return st;
  CopyArgs c{pesti_kv::args_of(cache, nullptr), n, nullptr, src, dst, 1};
  void* params[] = {&c};
  return pesti_kv::launch(reinterpret_cast<const void*>(&pesti::copy_kernel), dim3(copy_groups(c.kv, n)),
                          dim3(pesti::kCopyThreads), params, 0, static_cast<hipStream_t>(stream));
}

}  // extern "C"
