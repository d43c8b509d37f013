// kv_cache.cu -- the plain paged cache's rows: appending tokens, and evicting
// the rows with the least accumulated attention weight.
#include <algorithm>
#include <atomic>

#include <cooperative_groups.h>

#include "common.cuh"
#include "sm100.cuh"

namespace dkv {

namespace {

// A warp copies the K and V rows 0 .. rows-1 of a group of kRows to pool rows
// to(k) (skipped where that is negative): up to eight 16-byte words per lane
// are loaded before the first is stored.  kWords: words of one row's K and V
// together (16, 32 or 64); from(k, is_v): a row's address.  Both are called by
// all lanes alike.
template <int kWords, int kRows, typename From, typename To>
__device__ __forceinline__ void copy_rows(int rows, int lane, From from, To to, const KvView& c) {
  constexpr int kHalf = kWords / 2;
  constexpr int kLoads = kRows * kWords / 32;
  constexpr int kPart = kLoads < 8 ? kLoads : 8;  // words in flight per lane: 32 registers
#pragma unroll
  for (int i0 = 0; i0 < kLoads; i0 += kPart) {
    uint4 v[kPart];
#pragma unroll
    for (int i = 0; i < kPart; ++i) {
      const int k = ((i0 + i) * 32 + lane) / kWords, word = lane % kWords + (kWords == 64 ? (i & 1) * 32 : 0);
      const bool is_v = word >= kHalf;
      const char* p = from(k, is_v);
      if (k < rows) v[i] = __ldcg(reinterpret_cast<const uint4*>(p) + (is_v ? word - kHalf : word));
    }
#pragma unroll
    for (int i = 0; i < kPart; ++i) {
      const int k = ((i0 + i) * 32 + lane) / kWords, word = lane % kWords + (kWords == 64 ? (i & 1) * 32 : 0);
      const bool is_v = word >= kHalf;
      const int64_t t = to(k);
      if (k < rows && t >= 0)
        reinterpret_cast<uint4*>((is_v ? c.v : c.k) + t * (kHalf * 16))[is_v ? word - kHalf : word] = v[i];
    }
  }
}

// ---- append
// A warp copies kAppendRows new rows of a pair: a lane looks up where one row
// goes, then the warp loads all rows' 16-byte words (K and V) before it stores
// the first.  Pure copying: bound by the rows read and written once each (190
// thousand tokens' rows of 512 bytes into 64-row pages: 195 MB in 33 to 37 us,
// 5.2 to 6 TB/s; with one row in flight per warp 130 us).
constexpr int kAppendRows = 8;
constexpr int kAppendWarps = 8;

struct AppendArgs {
  KvView c;
  int H, n_new, chunks;  // chunks: CTAs per pair
  const char* K;
  const char* V;
  int64_t sb, sh, st;    // byte strides
  const int32_t* n_tokens;
  const int32_t* first_pos;
  float* w;
  int32_t* pos;
  int64_t cap;
  const float* tok_w;
};

// kWords: 16-byte words of one row's K and V together (16, 32 or 64).
template <int kWords>
__global__ void __launch_bounds__(kAppendWarps * 32, 4) kv_append_kernel(const __grid_constant__ AppendArgs a) {
  const int bh = blockIdx.x / a.chunks;
  const int b = bh / a.H, h = bh - b * a.H;
  const int lane = threadIdx.x & 31;
  const int t0 = ((blockIdx.x - bh * a.chunks) * kAppendWarps + (threadIdx.x >> 5)) * kAppendRows;
  sm100::grid_dep_wait();
  const int raw = a.c.raw_len(bh), len = a.c.checked(raw);
  const int nb = a.n_tokens ? __ldcg(a.n_tokens + b) : a.n_new;
  if (raw != len || nb < 0 || nb > a.n_new || nb > len) {
    if (threadIdx.x == 0) a.c.report((uint32_t)(raw != len ? raw : nb));
    return;
  }
  const int rows = min(kAppendRows, nb - t0);
  if (rows <= 0) return;
  int64_t row = -1;
  if (lane < rows) {
    const int t = t0 + lane, r = len - nb + t;
    row = a.c.row(bh, r);
    if (a.w) a.w[bh * a.cap + r] = a.tok_w ? a.tok_w[(int64_t)bh * a.n_new + t] : 0.f;
    if (a.pos) a.pos[bh * a.cap + r] = a.first_pos[b] + t;
  }
  __syncwarp();
  const int64_t src = b * a.sb + h * a.sh + (int64_t)t0 * a.st;
  copy_rows<kWords, kAppendRows>(
      rows, lane, [&](int k, bool is_v) { return (is_v ? a.V : a.K) + src + k * a.st; },
      [&](int k) { return __shfl_sync(0xffffffffu, row, k); }, a.c);
}

// ---- evict
// A cluster of CTAs per pair, each with a run of its rows.  Weights become
// integer keys that order like them, held in registers (runs of more than 16
// rows a thread are read again for each step instead).  The m-th largest key is
// found by narrowing a range of keys: 1024 equal bins over it, counted per CTA
// and added up over the cluster through distributed shared memory, until the
// bin that holds the m-th key is kept whole or holds one key only; two rounds
// as a rule, four at most.  (A cache held at its budget drops a row or so per
// token: up to kFew rows are found as that many minima instead.)  Rows above
// the threshold and the first of those equal to it are kept; a scan in row
// order numbers the dropped rows below m (holes) and the kept rows at or past m
// (movers), of which there are equally many: mover i goes to hole i.  Bound by
// its chain of block and cluster barriers, the keys are read once: 8 pairs of
// 131072 rows 29 us, 64 pairs of 4096 to 32768 rows 20 us.
// Where the rows per thread are few, the clusters make the moves; else a second
// kernel does, spread over the whole GPU whatever the pairs' shares: bound by
// the rows read and written.
constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBinBits = 10;
constexpr int kBins = 1 << kBinBits;
constexpr int kPerLarge = 16;         // rows per thread in registers, at most
constexpr int kMaxCluster = 8;
constexpr int kFew = 4;               // this many rows to drop are found one by one
static_assert(kBins == kSelThreads && kSelWarps == 32, "a thread per bin, a lane per warp");

struct EvictArgs {
  KvView c;
  int BH, cluster;
  const int32_t* budget;
  int n_first, n_recent;
  const float* w;
  const int32_t* pos;
  float* w_out;
  int32_t* pos_out;
  int64_t cap;
  int32_t* lens_out;
  int32_t* count;  // [BH]
  int32_t* hole;   // [BH][half]
  int32_t* move;   // [BH][half]
  int64_t half;
};

constexpr uint32_t kGuarded = 0xffffffffu;  // above every weight's key

// Weight as a key that orders like it: NaN lowest (0), -0 as +0.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Exclusive prefix of v over the block; total in `all`.  sh: 32 words, in use
// until the next barrier.
__device__ __forceinline__ int block_scan(int v, int& all, int* sh) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += u;
  }
  __syncthreads();
  if (lane == 31) sh[warp] = inc;
  __syncthreads();
  const int t = sh[lane];
  int ti = t;
#pragma unroll
  for (int o = 1; o < kSelWarps; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, ti, o);
    if (lane >= o) ti += u;
  }
  all = __shfl_sync(0xffffffffu, ti, kSelWarps - 1);
  return __shfl_sync(0xffffffffu, ti - t, warp) + inc - v;
}

// What a CTA tells the others of its cluster.
struct SelExchange {
  uint32_t kmin, kmax;
  int last, bad;      // largest position; a page out of range
  int holes, movers;
  uint64_t least[kFew];
};

struct SelSmem {
  int hist[2][kBins + 1];  // bin kBins: guarded rows
  SelExchange from[kMaxCluster]; // written by the CTAs of the cluster
  int scan[32];
  int at[kPerLarge * kSelWarps];  // rows of 32 rows (a warp's): counts, then their prefix
  uint32_t rmin[kSelWarps], rmax[kSelWarps];
  int rlast[kSelWarps];
  uint64_t rleast[kSelWarps];
  int found, found_count, found_above;
};

// Moves i0 .. i0 + rows - 1 of a pair (rows <= kRows), by one warp: a lane
// looks up one move, then the warp copies the rows.
template <int kWords, int kRows>
__device__ __forceinline__ void move_rows(const EvictArgs& a, int bh, int i0, int rows, int lane) {
  int64_t src = 0, dst = -1;
  if (lane < rows) {
    const int from = __ldcg(a.move + bh * a.half + i0 + lane), to = __ldcg(a.hole + bh * a.half + i0 + lane);
    // (always so, unless the weights changed under the call while the lists were made)
    if ((uint32_t)from < (uint32_t)a.c.max_len && (uint32_t)to < (uint32_t)a.c.max_len) {
      const int64_t s = a.c.row(bh, from), d = a.c.row(bh, to);
      if (s >= 0 && d >= 0) src = s, dst = d;  // (a row without a place is neither read nor written)
      a.w_out[bh * a.cap + to] = __ldcg(a.w + bh * a.cap + from);
      a.pos_out[bh * a.cap + to] = __ldcg(a.pos + bh * a.cap + from);
    }
  }
  __syncwarp();
  copy_rows<kWords, kRows>(
      rows, lane,
      [&](int k, bool is_v) { return (is_v ? a.c.v : a.c.k) + __shfl_sync(0xffffffffu, src, k) * (kWords * 8); },
      [&](int k) { return __shfl_sync(0xffffffffu, dst, k); }, a.c);
}

// Exclusive prefix over sm.at's first N entries, in place; the total.
template <int N>
__device__ __forceinline__ int scan_counts(SelSmem& sm) {
  __syncthreads();
  const int i = threadIdx.x;
  int all;
  const int pre = block_scan(i < N ? sm.at[i] : 0, all, sm.scan);
  if (i < N) sm.at[i] = pre;
  __syncthreads();
  return all;
}

// kPer: rows per thread in registers; kWords: words of a row for the clusters
// to make the moves themselves, with every run in registers, or 0.
template <int kPer, int kWords>
__global__ void __launch_bounds__(kSelThreads) kv_select_kernel(const __grid_constant__ EvictArgs a) {
  namespace cg = cooperative_groups;
  constexpr int kChunk = kPer * kSelThreads;
  constexpr bool kOne = kWords > 0;  // (a run of more rows than the registers hold is never launched so)
  __shared__ SelSmem sm;
  const cg::cluster_group cl = cg::this_cluster();
  const int C = a.cluster, rank = C == 1 ? 0 : (int)cl.block_rank();
  const int bh = blockIdx.x / C;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  sm100::grid_dep_wait();
  sm100::grid_dep_launch();
  if (C > 1) cg::cluster_group::barrier_arrive();  // the others' shared memory is there from the wait on
  const int raw = a.c.raw_len(bh), n = a.c.checked(raw), budget = a.budget[bh];
  int m = min(n, max(budget, a.n_first + a.n_recent));
  if (rank == 0 && tid == 0 && (raw != n || budget < 0)) a.c.report((uint32_t)(raw != n ? raw : budget));
  const float* w = a.w + bh * a.cap;
  const int32_t* pos = a.pos + bh * a.cap;
  const int run = (n + C - 1) / C;  // rows per CTA
  const int lo = min(n, rank * run), hi = min(n, lo + run);
  auto sync = [&] {
    if (C == 1)
      __syncthreads();
    else
      cl.sync();
  };
  auto peer = [&](auto* p, int c) { return C == 1 ? p : cl.map_shared_rank(p, c); };
  // ---- keys and positions of rows r0 + j kSelThreads + tid, their range, the largest position, and the pages
  const bool resident = kOne || run <= kChunk;
  auto next = [&](int r0) { return kOne ? hi : r0 + kChunk; };
  uint32_t key[kPer];
  int ps[kPer];
  auto load = [&](int r0) {
    const float* wp = w + r0 + tid;
    const int32_t* pp = pos + r0 + tid;
    const int in = hi - r0 - tid;  // the j-th row is there where j kSelThreads < in
    float wv[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      wv[j] = 0.f;
      ps[j] = 0;
      if (j * kSelThreads < in) {
        wv[j] = __ldcg(wp + j * kSelThreads);
        ps[j] = __ldcg(pp + j * kSelThreads);
      }
    }
#pragma unroll
    for (int j = 0; j < kPer; ++j) key[j] = weight_key(wv[j]);
  };
  uint32_t kmin = 0xffffffffu, kmax = 0u;
  int last = INT32_MIN, bad = 0;
  for (int r0 = lo; r0 < hi; r0 = next(r0)) {
    load(r0);
    const int in = hi - r0 - tid;
#pragma unroll
    for (int j = 0; j < kPer; ++j)
      if (j * kSelThreads < in) {
        kmin = min(kmin, key[j]);
        kmax = max(kmax, key[j]);
        last = max(last, ps[j]);
      }
  }
  // the pages of the rows this CTA starts with
  for (int r = ((lo >> a.c.page_log) + tid) << a.c.page_log; r < hi; r += kSelThreads << a.c.page_log)
    bad |= a.c.row(bh, r) < 0;
  kmin = __reduce_min_sync(0xffffffffu, kmin);
  kmax = __reduce_max_sync(0xffffffffu, kmax);
  last = __reduce_max_sync(0xffffffffu, last);
  if (lane == 0) {
    sm.rmin[warp] = kmin;
    sm.rmax[warp] = kmax;
    sm.rlast[warp] = last;
  }
  bad = __syncthreads_or(bad);
  if (C > 1) cg::cluster_group::barrier_wait();
  if (warp == 0) {
    kmin = __reduce_min_sync(0xffffffffu, sm.rmin[lane]);
    kmax = __reduce_max_sync(0xffffffffu, sm.rmax[lane]);
    last = __reduce_max_sync(0xffffffffu, sm.rlast[lane]);
    if (lane < C) {
      SelExchange* to = peer(&sm.from[C == 1 ? 0 : rank], lane);
      to->kmin = kmin;
      to->kmax = kmax;
      to->last = last;
      to->bad = bad;
    }
  }
  sync();
  for (int i = 0; i < C; ++i) {
    kmin = i == 0 ? sm.from[0].kmin : min(kmin, sm.from[i].kmin);
    kmax = i == 0 ? sm.from[0].kmax : max(kmax, sm.from[i].kmax);
    last = i == 0 ? sm.from[0].last : max(last, sm.from[i].last);
    bad |= sm.from[i].bad;
  }
  if (bad || budget < 0) m = n;
  // rows below m start out as themselves; the move writes over the holes
  if (a.w_out != a.w || a.pos_out != a.pos) {
#pragma unroll 4
    for (int r = rank * kSelThreads + tid; r < m; r += C * kSelThreads) {
      const float wv = __ldcg(w + r);
      const int pv = __ldcg(pos + r);
      if (a.w_out != a.w) a.w_out[bh * a.cap + r] = wv;
      if (a.pos_out != a.pos) a.pos_out[bh * a.cap + r] = pv;
    }
  }
  int cnt = 0;
  const bool guards = a.n_first + a.n_recent > 0;
  auto mark = [&] {
    if (guards) {
#pragma unroll
      for (int j = 0; j < kPer; ++j)  // (positions are at most `last`; the difference fits 32 bits)
        if ((uint32_t)ps[j] < (uint32_t)a.n_first || (uint32_t)last - (uint32_t)ps[j] < (uint32_t)a.n_recent) key[j] = kGuarded;
    }
  };
  // the keys of a chunk, guarded rows marked
  auto fetch = [&](int r0) {
    if (resident) return;
    load(r0);
    mark();
  };
  if (resident) mark();
  int32_t* hole = a.hole + bh * a.half;
  int32_t* move = a.move + bh * a.half;
  const uint32_t lower = (1u << lane) - 1;
  if (m < n && m > 0 && n - m <= kFew) {
    // ---- the n - m least rows, the higher of equal ones first
    int drop[kFew];
#pragma unroll
    for (int i = 0; i < kFew; ++i) {
      if (i >= n - m) break;
      uint64_t least = ~0ull;
      for (int r0 = lo; r0 < hi; r0 = next(r0)) {
        fetch(r0);
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
          const int r = r0 + j * kSelThreads + tid;
          bool in = r < hi;
#pragma unroll
          for (int d = 0; d < i; ++d) in &= drop[d] != r;
          if (in) least = min(least, (uint64_t)key[j] << 32 | (uint32_t)~r);
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) least = min(least, __shfl_xor_sync(0xffffffffu, least, o));
      __syncthreads();  // (the last turn's rleast has been read)
      if (lane == 0) sm.rleast[warp] = least;
      __syncthreads();
      if (warp == 0) {
        least = sm.rleast[lane];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) least = min(least, __shfl_xor_sync(0xffffffffu, least, o));
        if (lane < C) peer(&sm.from[C == 1 ? 0 : rank], lane)->least[i] = least;
      }
      sync();
      least = sm.from[0].least[i];
      for (int c = 1; c < C; ++c) least = min(least, sm.from[c].least[i]);
      drop[i] = (int)~(uint32_t)least;
    }
    // the k-th kept row at or past m goes to the k-th dropped row below m
#pragma unroll
    for (int i = 0; i < kFew; ++i) cnt += i < n - m && drop[i] < m;
    if (rank == 0 && tid < 32) {
      // lane i < n - m: row m + i, and the i-th dropped row
      int d = m, below = 0;
      bool dropped = false;
#pragma unroll
      for (int i = 0; i < kFew; ++i)
        if (i < n - m) {
          dropped |= drop[i] == m + lane;
          if (lane == i) d = drop[i];
        }
#pragma unroll
      for (int i = 0; i < kFew; ++i) below += i < n - m && drop[i] < d;
      const bool is_move = lane < n - m && !dropped;
      const uint32_t moves = __ballot_sync(0xffffffffu, is_move);
      if (is_move) move[__popc(moves & lower)] = m + lane;
      if (lane < n - m && d < m) hole[below] = d;
    }
  } else if (m < n && m > 0) {
    // ---- the threshold: keys in [base, base + span] are in question, `need` of them are kept
    uint32_t base = kmin, span = kmax - kmin;
    int shift = max(0, 32 - __clz((int)span) - kBinBits);  // span >> shift < kBins
    int need = m, buf = 0, eq_before = 0;
    bool ties = false;  // only the first `need` rows of those with key `base` are kept
    for (bool first = true;; first = false, buf ^= 1) {
      int* hist = sm.hist[buf];
      for (int i = tid; i <= kBins; i += kSelThreads) hist[i] = 0;
      __syncthreads();
      for (int r0 = lo; r0 < hi; r0 = next(r0)) {
        fetch(r0);
        const int in = hi - r0 - tid;
        int guarded = 0;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
          // (a key below base wraps round to far above span, and no range reaches the guarded rows' key)
          const uint32_t d = key[j] - base;
          const bool is = j * kSelThreads < in && d <= span;
          if (first) guarded += j * kSelThreads < in && key[j] == kGuarded;
          if (__any_sync(0xffffffffu, is)) {
            // rows of equal weight would queue up at one counter
            const uint32_t bin = d >> shift, bin0 = __shfl_sync(0xffffffffu, bin, 0);
            if (__all_sync(0xffffffffu, is && bin == bin0)) {
              if (lane == 0) atomicAdd(&hist[bin], 32);
            } else if (is) {
              atomicAdd(&hist[bin], 1);
            }
          }
        }
        if (first && guards) {
          guarded = __reduce_add_sync(0xffffffffu, guarded);
          if (lane == 0 && guarded) atomicAdd(&hist[kBins], guarded);
        }
      }
      sync();
      // add up the cluster's counts: thread t has bin kBins - 1 - t (largest keys first)
      int got[kMaxCluster], sum = 0;
#pragma unroll
      for (int c = 0; c < kMaxCluster; ++c) got[c] = c < C ? peer(hist, c)[kBins - 1 - tid] : 0;
      const int guard = __reduce_add_sync(0xffffffffu, first && lane < C ? peer(hist, lane)[kBins] : 0);
#pragma unroll
      for (int c = 0; c < kMaxCluster; ++c) sum += got[c];
      if (first && guard >= m) {
        // the guarded rows alone fill the budget (equal positions): the first of them are kept
        base = kGuarded;
        ties = guard > m;
        need = m;
        for (int c = 0; c < rank; ++c) eq_before += peer(hist, c)[kBins];
        break;
      }
      need -= guard;
      int all;
      const int above = block_scan(sum, all, sm.scan);
      if (above < need && above + sum >= need) {
        sm.found = kBins - 1 - tid;
        sm.found_above = above;
        sm.found_count = sum;
      }
      __syncthreads();
      const int bin = sm.found, count = sm.found_count;
      base += (uint32_t)bin << shift;
      need -= sm.found_above;
      if (count == need || shift == 0) {
        ties = count != need;
        if (ties)
          for (int c = 0; c < rank; ++c) eq_before += peer(hist, c)[bin];
        break;
      }
      span = (1u << shift) - 1;
      shift = max(0, shift - kBinBits);
      __syncthreads();  // found is read before the next round writes it
    }
    // ---- holes and movers, in row order: 32 rows (a warp's) at a time
    int hole_at = 0, move_at = 0;
    uint32_t hm = 0, mm = 0;  // bit j: the thread's j-th row of the last chunk counted is a hole (mover)
    for (int pass = 0; pass < 2; ++pass) {
      int eq_at = eq_before, holes = hole_at, movers = move_at;
      for (int r0 = lo; r0 < hi; r0 = next(r0)) {
        int all = 0;
        if (pass == 0 || !resident) {  // (of a single chunk, the first pass has it all)
          fetch(r0);
          const int in = hi - r0 - tid, low = m - r0 - tid;  // the j-th row is there; is below m
          const uint32_t least = ties ? base + 1 : base;      // (ties among the guarded rows: none is above them)
          const bool none = ties && base == kGuarded;
          hm = mm = 0;
#pragma unroll
          for (int j = 0; j < kPer; ++j) {
            const bool keep = !none && key[j] >= least;
            if (j * kSelThreads < in) {
              if (j * kSelThreads < low)
                hm |= keep ? 0u : 1u << j;
              else
                mm |= keep ? 1u << j : 0u;
            }
          }
          if (ties) {
            uint32_t eq = 0;
#pragma unroll
            for (int j = 0; j < kPer; ++j) eq |= (uint32_t)(j * kSelThreads < in && key[j] == base) << j;
#pragma unroll 2
            for (int j = 0; j < kPer; ++j) {
              const uint32_t b = __ballot_sync(0xffffffffu, eq >> j & 1);
              if (lane == 0) sm.at[j * kSelWarps + warp] = __popc(b);
            }
            all = scan_counts<kPer * kSelWarps>(sm);
#pragma unroll 2
            for (int j = 0; j < kPer; ++j) {
              const uint32_t b = __ballot_sync(0xffffffffu, eq >> j & 1);
              if ((eq >> j & 1) && eq_at + sm.at[j * kSelWarps + warp] + __popc(b & lower) < need) {  // kept after all
                if (j * kSelThreads < low)
                  hm &= ~(1u << j);
                else
                  mm |= 1u << j;
              }
            }
            eq_at += all;
            __syncthreads();
          }
#pragma unroll 2
          for (int j = 0; j < kPer; ++j) {
            const int g0 = r0 + j * kSelThreads;  // (holes lie below m, movers at or past it)
            const int holes_j = g0 < m ? __popc(__ballot_sync(0xffffffffu, hm >> j & 1)) : 0;
            const int movers_j = g0 + kSelThreads > m ? __popc(__ballot_sync(0xffffffffu, mm >> j & 1)) : 0;
            if (lane == 0) sm.at[j * kSelWarps + warp] = holes_j | movers_j << 16;
          }
          all = scan_counts<kPer * kSelWarps>(sm);
        }
        if (pass == 1) {
#pragma unroll 2
          for (int j = 0; j < kPer; ++j) {
            const int at = sm.at[j * kSelWarps + warp], g0 = r0 + j * kSelThreads;
            // (h, v < half unless the weights change under the call where they are read again and again)
            if (g0 < m) {
              const uint32_t b = __ballot_sync(0xffffffffu, hm >> j & 1);
              const int h = holes + (at & 0xffff) + __popc(b & lower);
              if ((hm >> j & 1) && h < a.half) hole[h] = g0 + tid;
            }
            if (g0 + kSelThreads > m) {
              const uint32_t b = __ballot_sync(0xffffffffu, mm >> j & 1);
              const int v = movers + (at >> 16) + __popc(b & lower);
              if ((mm >> j & 1) && v < a.half) move[v] = g0 + tid;
            }
          }
          if (!resident) __syncthreads();  // sm.at is read before the next chunk writes it
        }
        holes += all & 0xffff;
        movers += all >> 16;
      }
      if (pass == 0) {
        if (tid < C) {
          SelExchange* to = peer(&sm.from[C == 1 ? 0 : rank], tid);
          to->holes = holes;
          to->movers = movers;
        }
        sync();
        for (int c = 0; c < C; ++c) {
          if (c < rank) {
            hole_at += sm.from[c].holes;
            move_at += sm.from[c].movers;
          }
          cnt += sm.from[c].holes;
        }
      }
    }
    cnt = min(cnt, (int)a.half);
  }
  // (every access to another CTA's shared memory came before the last barrier that its owner passed)
  if constexpr (kWords > 0) {
    sync();  // the lists are written
    constexpr int kRows = 4;
    for (int i = (rank * kSelWarps + warp) * kRows; i < cnt; i += C * kSelWarps * kRows)
      move_rows<kWords, kRows>(a, bh, i, min(kRows, cnt - i), lane);
  }
  if (rank == 0 && tid == 0) {
    a.count[bh] = cnt;
    // in place, a length out of range stays the caller's: 0 would lose the rows for good
    if (raw == n || a.lens_out != a.c.lens) a.lens_out[bh] = m;
  }
}

// Move the listed rows, kMoveRows of a pair to a warp.  The pairs' counts form
// one list of such units that is cut evenly over the CTAs of the grid, four
// times as many as run at once, so that an SM that gets less of the memory's
// bandwidth takes fewer.  8 pairs of 131072 rows made 16384 long: 20 us, 5.9
// TB/s; 64 pairs of 4096 to 32768 made 8192 long, 4 to 5 TB/s: rows of 256
// bytes, read and written in no order.
constexpr int kMoveRows = 8;
constexpr int kMoveThreads = 256;

template <int kWords>
__global__ void __launch_bounds__(kMoveThreads, 4) kv_move_kernel(const __grid_constant__ EvictArgs a) {
  __shared__ int sh[kMoveThreads / 32], sh_at[2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  sm100::grid_dep_wait();
  // the pair that holds this CTA's first unit, by a block scan over the counts
  const int per = (a.BH + kMoveThreads - 1) / kMoveThreads;
  const int b0 = min(a.BH, tid * per), b1 = min(a.BH, b0 + per);
  int sum = 0;
  for (int b = b0; b < b1; ++b) sum += (__ldcg(a.count + b) + kMoveRows - 1) / kMoveRows;
  int inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) sh[warp] = inc;
  __syncthreads();
  int before = 0, total = 0;
#pragma unroll
  for (int i = 0; i < kMoveThreads / 32; ++i) {
    if (i < warp) before += sh[i];
    total += sh[i];
  }
  const int u0 = (int)((int64_t)total * blockIdx.x / gridDim.x), u1 = (int)((int64_t)total * (blockIdx.x + 1) / gridDim.x);
  if (u0 == u1) return;
  int s = before + inc - sum;
  if (u0 >= s && u0 < s + sum) {
    int b = b0;
    for (;; ++b) {
      const int u = (__ldcg(a.count + b) + kMoveRows - 1) / kMoveRows;
      if (u0 < s + u) break;
      s += u;
    }
    sh_at[0] = b;
    sh_at[1] = s;
  }
  __syncthreads();
  int bh = sh_at[0];
  s = sh_at[1];
  int cnt = __ldcg(a.count + bh);
  for (int u = u0 + warp; u < u1; u += kMoveThreads / 32) {
    while (u >= s + (cnt + kMoveRows - 1) / kMoveRows) {
      s += (cnt + kMoveRows - 1) / kMoveRows;
      cnt = __ldcg(a.count + ++bh);
    }
    const int i0 = (u - s) * kMoveRows;
    move_rows<kWords, kMoveRows>(a, bh, i0, min(kMoveRows, cnt - i0), lane);
  }
}

}  // namespace

cudaError_t launch_kv_append(const Plan& p, const KvView& c, int n_new, const KVView& kv, const int32_t* n_tokens,
                             const int32_t* first_pos, float* w, int32_t* pos, int cap, const float* tok_w,
                             cudaStream_t st) {
  AppendArgs a{};
  a.c = c;
  a.H = p.cfg.kv_heads;
  a.n_new = n_new;
  a.chunks = (int)ceil_div64(n_new, kAppendRows * kAppendWarps);
  a.K = (const char*)kv.K;
  a.V = (const char*)kv.V;
  a.sb = kv.sb * p.esize;
  a.sh = kv.sh * p.esize;
  a.st = kv.st * p.esize;
  a.n_tokens = n_tokens;
  a.first_pos = first_pos;
  a.w = w;
  a.pos = pos;
  a.cap = cap;
  a.tok_w = tok_w;
  const unsigned grid = (unsigned)(p.cfg.batch * p.cfg.kv_heads) * a.chunks;
  const int words = p.cfg.d_h * p.esize / 8;
  auto kern = words == 16 ? kv_append_kernel<16> : words == 32 ? kv_append_kernel<32> : kv_append_kernel<64>;
  ProfScope ps(p, st, KID_KV_APPEND);
  return launch_pdl(kern, grid, kAppendWarps * 32, 0, st, a);
}

// CTAs per pair: as many as find room at once, one to an SM (16 clusters of eight
// and 36 of four do not, 32 of four and 72 of two do; us replayed, half of the
// rows dropped: 16 pairs of 15000 by eight / four 42 / 34, 36 pairs by four / two
// 70 / 52, 72 pairs by two / one 74 / 78), each with 512 rows at least, and one
// below 2048 rows (8 pairs, half dropped, 512 / 1024 rows at least: 2049 rows
// 15.3 / 17.2, 4000 rows 17.3 / 21.4; one of 1100 rows dropped by one / two 5.8 /
// 7.6).
constexpr int kMinRun = 512, kMinSplit = 2048;
constexpr int select_ctas(int cluster) { return cluster == 8 ? 96 : cluster == 4 ? 128 : kNumSMs; }

// The clusters make the moves themselves, without a second kernel, where their
// threads hold 4 rows at most, and up to 8 where two thirds of the SMs take part.
// us replayed, here / second kernel: one row dropped, 32 pairs of 15000 (4 rows)
// 9.5 / 15.9, 64 of 15000 (8 rows) 11.1 / 17.1; half dropped 40 / 49 and 70 / 74, 16
// of 32000 (8 rows on 64 SMs) 63 / 52, 64 of 32000 (16 rows) 140 / 127 and twice
// that where lengths differ.
constexpr int kHere = 4, kHereMany = 8, kManyCtas = 96;

template <int kPer>
auto select_here(int words) {
  return words == 16 ? kv_select_kernel<kPer, 16> : words == 32 ? kv_select_kernel<kPer, 32> : kv_select_kernel<kPer, 64>;
}

cudaError_t launch_kv_evict(const Plan& p, const KvView& c, const int32_t* budget, int n_first, int n_recent,
                            const float* w, const int32_t* pos, float* w_out, int32_t* pos_out, int cap,
                            int32_t* lens_out, void* ws, cudaStream_t st) {
  const KvWorkspace L = kv_workspace(p, c.max_len);
  EvictArgs a{};
  a.c = c;
  a.BH = p.cfg.batch * p.cfg.kv_heads;
  a.budget = budget;
  a.n_first = n_first;
  a.n_recent = n_recent;
  a.w = w;
  a.pos = pos;
  a.w_out = w_out;
  a.pos_out = pos_out;
  a.cap = cap;
  a.lens_out = lens_out;
  a.count = (int32_t*)((char*)ws + L.count);
  a.hole = (int32_t*)((char*)ws + L.hole);
  a.move = (int32_t*)((char*)ws + L.move);
  a.half = c.max_len / 2;
  a.cluster = 1;
  if (c.max_len >= kMinSplit)
    while (a.cluster < kMaxCluster && (int64_t)a.BH * a.cluster * 2 <= select_ctas(a.cluster * 2) &&
           a.cluster * 2 * kMinRun <= c.max_len)
      a.cluster *= 2;
  const int run = (int)ceil_div64(c.max_len, a.cluster);
  const int words = p.cfg.d_h * p.esize / 8;
  const int per = (int)ceil_div64(run, kSelThreads);
  const bool all_here = per <= kHere || (per <= kHereMany && a.BH * a.cluster >= kManyCtas);
  auto select = !all_here      ? kv_select_kernel<kPerLarge, 0>
                : per <= 2     ? select_here<2>(words)
                : per <= kHere ? select_here<kHere>(words)
                               : select_here<kHereMany>(words);
  cudaError_t e;
  {
    ProfScope ps(p, st, KID_KV_SELECT);
    e = launch_pdl_cluster(select, (unsigned)(a.BH * a.cluster), kSelThreads, a.cluster, 0, st, a);
  }
  if (e != cudaSuccess || all_here) return e;
  auto move = words == 16 ? kv_move_kernel<16> : words == 32 ? kv_move_kernel<32> : kv_move_kernel<64>;
  const int64_t most = a.BH * ceil_div64(a.half, kMoveRows * kMoveThreads / 32);
  ProfScope ps(p, st, KID_KV_MOVE);
  return launch_pdl(move, (unsigned)std::max<int64_t>(1, std::min<int64_t>(most, kNumSMs * 16)), kMoveThreads, 0, st, a);
}

}  // namespace dkv
