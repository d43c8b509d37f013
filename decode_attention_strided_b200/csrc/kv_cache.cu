// kv_cache.cu -- the plain paged cache's rows: appending tokens, and evicting
// the rows with the least accumulated attention weight.
#include <algorithm>

#include "common.cuh"

namespace dkv {

namespace {

// ---- append
// One 16-byte word of one new row per thread and step: the rows of a pair are
// its K row's words and then its V row's.  Pure copying: bound by the rows read
// and written once each.
struct AppendArgs {
  KvView c;
  int64_t BH;
  int H, n_new, words;  // words: 16-byte words of one K row
  const char* K;
  const char* V;
  int64_t sb, sh, st;   // byte strides
  const int32_t* n_tokens;
  const int32_t* first_pos;
  float* w;
  int32_t* pos;
  int64_t cap;
  const float* tok_w;
};

__global__ void __launch_bounds__(256) kv_append_kernel(AppendArgs a) {
  const int per_row = 2 * a.words;  // a power of two, at most 64
  const int rows_blk = 256 / per_row;
  const int64_t chunks = (a.n_new + rows_blk - 1) / rows_blk;
  const int t0 = threadIdx.x / per_row, word = threadIdx.x % per_row;
  for (int64_t i = blockIdx.x; i < a.BH * chunks; i += gridDim.x) {
    const int64_t bh = i / chunks;
    const int64_t t = (i % chunks) * rows_blk + t0;
    const int64_t b = bh / a.H;
    const int h = (int)(bh % a.H);
    const int len = a.c.len(bh), raw = a.c.lens[bh];
    const int nb = a.n_tokens ? a.n_tokens[b] : a.n_new;
    if (raw != len || nb < 0 || nb > a.n_new || nb > len) {
      if (threadIdx.x == 0) a.c.report((uint32_t)nb);
      continue;
    }
    if (t >= nb) continue;
    const int r = len - nb + (int)t;
    if (word == 0) {
      if (a.w) a.w[bh * a.cap + r] = a.tok_w ? a.tok_w[bh * a.n_new + t] : 0.f;
      if (a.pos) a.pos[bh * a.cap + r] = a.first_pos[b] + (int)t;
    }
    const int64_t row = a.c.row(bh, r);
    if (row < 0) continue;
    const bool is_v = word >= a.words;
    const int wd = is_v ? word - a.words : word;
    const char* src = (is_v ? a.V : a.K) + b * a.sb + h * a.sh + t * a.st;
    char* dst = (is_v ? a.c.v : a.c.k) + row * a.words * 16;
    reinterpret_cast<uint4*>(dst)[wd] = reinterpret_cast<const uint4*>(src)[wd];
  }
}

// ---- evict
// Each pair: the m-th largest key of its n rows by a radix select (most
// significant byte first), the rows above it and the first rows equal to it
// are kept; a scan in row order numbers the dropped rows below m (holes) and
// the kept rows at or past m (movers), of which there are equally many: mover
// i goes to hole i.  A second kernel moves the rows.
constexpr int kSelThreads = 1024;

struct EvictArgs {
  KvView c;
  int64_t BH;
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
  int words;       // 16-byte words of one K row
};

constexpr uint32_t kGuarded = 0xffffffffu;

// Weight as a key that orders like it: NaN lowest (0), -0 as +0.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Exclusive prefix of v over the block; total in `all`.
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
  int t = sh[lane], ti = t;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, ti, o);
    if (lane >= o) ti += u;
  }
  all = __shfl_sync(0xffffffffu, ti, 31);
  return __shfl_sync(0xffffffffu, ti - t, warp) + inc - v;
}

__global__ void __launch_bounds__(kSelThreads) kv_select_kernel(EvictArgs a) {
  __shared__ int sh[32];
  __shared__ int hist[256];
  __shared__ uint32_t sh_prefix;
  __shared__ int sh_need;
  const int64_t bh = blockIdx.x;
  const int tid = threadIdx.x;
  const int raw = a.c.lens[bh], n = a.c.len(bh), budget = a.budget[bh];
  int m = min(n, max(budget, a.n_first + a.n_recent));
  int bad = 0;
  for (int l = tid; l < ((n - 1) >> a.c.page_log) + 1 && n > 0; l += kSelThreads)
    bad |= a.c.row(bh, l << a.c.page_log) < 0;
  bad = __syncthreads_or(bad);
  if (tid == 0 && (raw != n || budget < 0)) a.c.report((uint32_t)(raw != n ? raw : budget));
  if (bad || budget < 0) m = n;
  const float* w = a.w + bh * a.cap;
  const int32_t* pos = a.pos + bh * a.cap;
  float* wo = a.w_out + bh * a.cap;
  int32_t* po = a.pos_out + bh * a.cap;
  int cnt = 0;
  if (m == n) {
    for (int r = tid; r < n; r += kSelThreads) {
      wo[r] = w[r];
      po[r] = pos[r];
    }
  } else if (m > 0) {
    int last = INT32_MIN;
    for (int r = tid; r < n; r += kSelThreads) last = max(last, pos[r]);
    last = __reduce_max_sync(0xffffffffu, last);
    if ((tid & 31) == 0) sh[tid >> 5] = last;
    __syncthreads();
    last = __reduce_max_sync(0xffffffffu, sh[tid & 31]);
    const int64_t from = (int64_t)last - a.n_recent;
    auto key = [&](int r) {
      const int p = pos[r];
      return p < a.n_first || p > from ? kGuarded : weight_key(w[r]);
    };
    uint32_t prefix = 0;
    int need = m;  // rows still to keep among the keys with this prefix
    for (int shift = 24; shift >= 0; shift -= 8) {
      __syncthreads();
      if (tid < 256) hist[tid] = 0;
      __syncthreads();
      const uint32_t mask = shift == 24 ? 0u : 0xffffffffu << (shift + 8);
      for (int r = tid; r < n; r += kSelThreads) {
        const uint32_t k = key(r);
        if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & 255], 1);
      }
      __syncthreads();
      if (tid == 0) {
        int left = need, d = 255;
        for (; d > 0 && hist[d] < left; --d) left -= hist[d];
        sh_prefix = prefix | ((uint32_t)d << shift);
        sh_need = left;
      }
      __syncthreads();
      prefix = sh_prefix;
      need = sh_need;
    }
    // keep: keys above the threshold, and its first `need` rows
    int eq_before = 0, hole_before = 0, move_before = 0;
    for (int r0 = 0; r0 < n; r0 += kSelThreads) {
      const int r = r0 + tid;
      const uint32_t k = r < n ? key(r) : 0u;
      const int eq = r < n && k == prefix;
      int all;
      const int eq_rank = eq_before + block_scan(eq, all, sh);
      eq_before += all;
      const bool keep = r < n && (k > prefix || (eq && eq_rank < need));
      const int is_hole = r < m && !keep, is_move = r >= m && keep;
      const int rank = block_scan(is_hole | (is_move << 16), all, sh);
      if (is_hole) a.hole[bh * a.half + hole_before + (rank & 0xffff)] = r;
      if (is_move) a.move[bh * a.half + move_before + (rank >> 16)] = r;
      hole_before += all & 0xffff;
      move_before += all >> 16;
      if (keep && r < m) {
        wo[r] = w[r];
        po[r] = pos[r];
      }
    }
    cnt = hole_before;
  }
  __syncthreads();
  if (tid == 0) {
    a.count[bh] = cnt;
    a.lens_out[bh] = m;
  }
}

// Move the listed rows: a warp takes 32 of a pair's moves, a lane looks up one
// move's rows, then the warp copies the 32 rows' 16-byte words together.
__global__ void __launch_bounds__(256) kv_move_kernel(EvictArgs a, int ctas_per_pair) {
  const int64_t bh = blockIdx.x / ctas_per_pair;
  const int lane = threadIdx.x & 31;
  const int warp = (blockIdx.x % ctas_per_pair) * 8 + (threadIdx.x >> 5);
  const int cnt = a.count[bh];
  const int per_row = 2 * a.words;
  for (int i0 = warp * 32; i0 < cnt; i0 += ctas_per_pair * 8 * 32) {
    int64_t src = -1, dst = -1;
    if (i0 + lane < cnt) {
      const int s = a.move[bh * a.half + i0 + lane], d = a.hole[bh * a.half + i0 + lane];
      src = a.c.row(bh, s);
      dst = a.c.row(bh, d);
      a.w_out[bh * a.cap + d] = a.w[bh * a.cap + s];
      a.pos_out[bh * a.cap + d] = a.pos[bh * a.cap + s];
    }
    const int n = min(32, cnt - i0);
    for (int j0 = 0; j0 < n * per_row; j0 += 32) {
      const int r = (j0 + lane) / per_row, word = (j0 + lane) % per_row;  // r <= 31: per_row is 16, 32 or 64
      const int64_t s = __shfl_sync(0xffffffffu, src, r), d = __shfl_sync(0xffffffffu, dst, r);
      const bool is_v = word >= a.words;
      const int wd = is_v ? word - a.words : word;
      char* base = is_v ? a.c.v : a.c.k;
      if (s >= 0 && d >= 0)
        reinterpret_cast<uint4*>(base + d * a.words * 16)[wd] = reinterpret_cast<const uint4*>(base + s * a.words * 16)[wd];
    }
  }
}

}  // namespace

cudaError_t launch_kv_append(const Plan& p, const KvView& c, int n_new, const KVView& kv, const int32_t* n_tokens,
                             const int32_t* first_pos, float* w, int32_t* pos, int cap, const float* tok_w,
                             cudaStream_t st) {
  AppendArgs a{};
  a.c = c;
  a.BH = (int64_t)p.cfg.batch * p.cfg.kv_heads;
  a.H = p.cfg.kv_heads;
  a.n_new = n_new;
  a.words = p.cfg.d_h * p.esize / 16;
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
  const int rows_blk = 256 / (2 * a.words);
  const int64_t blocks = a.BH * ceil_div64(n_new, rows_blk);
  ProfScope ps(p, st, KID_KV_APPEND);
  kv_append_kernel<<<(int)std::min<int64_t>(blocks, kNumSMs * 8), 256, 0, st>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_kv_evict(const Plan& p, const KvView& c, const int32_t* budget, int n_first, int n_recent,
                            const float* w, const int32_t* pos, float* w_out, int32_t* pos_out, int cap,
                            int32_t* lens_out, void* ws, cudaStream_t st) {
  const KvWorkspace L = kv_workspace(p, c.max_len);
  EvictArgs a{};
  a.c = c;
  a.BH = (int64_t)p.cfg.batch * p.cfg.kv_heads;
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
  a.words = p.cfg.d_h * p.esize / 16;
  {
    ProfScope ps(p, st, KID_KV_SELECT);
    kv_select_kernel<<<(unsigned)a.BH, kSelThreads, 0, st>>>(a);
  }
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int per_pair = (int)std::max<int64_t>(1, std::min<int64_t>(ceil_div64(a.half, 256), kNumSMs * 8 / a.BH));
  ProfScope ps(p, st, KID_KV_MOVE);
  kv_move_kernel<<<(unsigned)(a.BH * per_pair), 256, 0, st>>>(a, per_pair);
  return cudaGetLastError();
}

}  // namespace dkv
