// kv_attend.cu -- attention of one new token per sequence over plain K/V rows
// in pages, split over the rows and joined.
//
// For query head hq of pair bh = (sequence, kv-head), with d_r = q . K_r over
// the pair's valid rows r and c = log2(e) / sqrt(d_h):
//   m = c max_r d_r,  l = sum_r 2^(c d_r - m),  out = (sum_r 2^(c d_r - m) V_r) / l,
//   lse = ln2 (m + log2 l),   and with weights   w_r <- decay w_r + sum_heads 2^(c d_r - m) / l.
// A part of the rows gives (m, l, o = sum 2^(c d_r - m) V_r); parts join by
// m = max m_i, l = sum 2^(m_i - m) l_i, o = sum 2^(m_i - m) o_i.  The exponent is
// one fused multiply-add of the dot product and the rounded m: a logit of 30,
// rounded by itself, would put 2^-19 into its weight, but m's rounding is the
// same in numerator and denominator.
//
// Split: all pairs' rows, in units of 16 to 64 (8 KB of K), form one list that
// is cut into as many equal ranges as there are CTAs, so that lengths do not
// matter for the balance.  A CTA's range is a run of segments, each inside one
// pair; only its first and its last segment can be a part of a pair, so a CTA
// leaves two partial results at most.  A second kernel joins them; a third adds
// the weights, which need the joined (m, l) of each head.
#include <algorithm>
#include <atomic>
#include <cmath>

#include <cooperative_groups.h>

#include "common.cuh"
#include "sm100.cuh"

namespace dkv {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kGroup = 16;         // rows of the smallest page
constexpr int kSlotBytes = 8192;   // K or V rows of one unit of the split
constexpr int kSlots = 2;          // of a warp's ring: K rows, V rows
constexpr int kMinUnits = 4;       // below a full grid a CTA gets these at most, and so many CTAs work (5 units: 3 and 2)
// A cluster per pair instead of the cut (one kernel instead of two): where its
// CTAs find room at once (16 clusters of eight did not, 32 of four did) and take
// 16 units at most.  bf16, d_h 128, four heads, us replayed, cluster / cut: 8
// pairs of 513 rows 8.2 / 10.3, of 4096 (16 units a CTA) 12.3 / 14.4, of 8192
// 18.6 / 18.4; 64 pairs of 1024 14.4 / 16.3; one pair of 8192 18.4 / 13.2.  Lengths
// that differ cost the cluster more, the cut nothing, hence no more units.  Measured
// without weights, with which the cut is three kernels instead of two; the limits hold
// for every type, head size and head count and with weights, where they were not.
constexpr int kShortUnits = 16;
constexpr int short_ctas(int cluster) { return cluster == 8 ? 96 : 128; }
// rows per unit
template <typename E, int DH>
constexpr int kUnitRows = kSlotBytes / (DH * (int)sizeof(E));
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct AttendArgs {
  KvView c;
  int BH, H, G;
  int unit_log;   // log2 of the rows per unit
  const void* q;
  int64_t qsb, qsh;
  float* out;
  int64_t osb, osh;
  float* lse;     // [B][Hq] or null
  float* w;       // [BH][cap] or null
  int64_t cap;
  float decay, scale2;  // scale2 = log2(e) / sqrt(d_h)
  float* part;    // [CTA][2][kv_part_floats]: o[G][d_h], m[kMaxG], l[kMaxG]
  float2* norm;   // [BH][G]: m and 1 / l, for the weights
  float* dots;    // [BH][max_len][G]: q . K_r, for the weights
};

// The cut of the unit list into ranges: the first `rem` of them hold per + 1
// units, the others per.  (The host refuses calls whose list could reach 2^31
// units.)
struct Cut {
  int W, g;  // units of all pairs; ranges (0 where there is no unit)
  int per, rem;
  __device__ int start(int c) const { return c * per + min(c, rem); }
  __device__ int range_of(int u) const {
    const int head = rem * (per + 1);
    return u < head ? u / (per + 1) : rem + (u - head) / per;
  }
};

// A place in the unit list: a pair, its first unit and its length.
struct Place {
  int bh, s, len;
};

// units of len rows
__device__ __forceinline__ int units_of(int len, int unit_log) { return (len + (1 << unit_log) - 1) >> unit_log; }

// The cut, and the pair that holds the first unit of range c, by a block scan
// over the lengths.  Every thread returns the same values; sh: kLocateWords
// of shared memory, free again on return.  Lengths out of range are reported
// here; `empty` tells whether any pair holds no row.
// Where a thread has one pair at most, it leaves its length in table (if not
// null).
constexpr int kLocateWords = kWarps + 4;
__device__ __forceinline__ Cut locate(const AttendArgs& a, int c, int* sh, int* table, Place& at, bool& empty) {
  const KvView& k = a.c;
  const int BH = a.BH;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (BH + kThreads - 1) / kThreads;
  const int b0 = min(BH, tid * per), b1 = min(BH, b0 + per);
  int sum = 0, none = 0, last = 0;
  for (int b = b0; b < b1; ++b) {
    const int raw = k.raw_len(b);
    last = k.checked(raw);
    if (raw != last) k.report((uint32_t)raw);
    none |= last == 0;
    sum += units_of(last, a.unit_log);
  }
  if (table) table[tid] = last;
  int inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) sh[warp] = inc;
  empty = __syncthreads_or(none) != 0;
  int before = 0, W = 0;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) {
    if (i < warp) before += sh[i];
    W += sh[i];
  }
  Cut cut;
  cut.W = W;
  cut.g = min((int)kKvMaxGrid, (W + kMinUnits - 1) / kMinUnits);
  cut.per = W / max(1, cut.g);
  cut.rem = W - cut.per * cut.g;
  if (c < cut.g) {
    const int target = cut.start(c);
    int s = before + inc - sum;
    if (target >= s && target < s + sum) {
      int b = b0;
      if (per > 1)
        for (;; ++b) {
          last = k.len(b);
          if (b + 1 == b1 || target < s + units_of(last, a.unit_log)) break;
          s += units_of(last, a.unit_log);
        }
      sh[kWarps] = b;
      sh[kWarps + 1] = s;
      sh[kWarps + 2] = last;
    }
  }
  __syncthreads();
  at = Place{sh[kWarps], sh[kWarps + 1], sh[kWarps + 2]};
  __syncthreads();
  return cut;
}

// The lengths of the pairs from bh0 on, the first kLensTable of them in shared
// memory: a CTA with many short pairs steps through them without a trip to L2
// for each.
constexpr int kLensTable = 256;
struct Lens {
  const KvView& k;
  const int* table;
  int bh0, unit_log;
  __device__ __forceinline__ int operator()(int bh) const {
    const int i = bh - bh0;
    return i < kLensTable ? table[i] : k.len(bh);
  }
  // move to the pair that holds unit u (at or after the present one)
  __device__ __forceinline__ void seek(Place& at, int u) const {
    while (u >= at.s + units_of(at.len, unit_log)) {
      at.s += units_of(at.len, unit_log);
      at.len = (*this)(++at.bh);
    }
  }
};

// The warps' partial results of up to kBufs segments, heads padded to GP: a
// warp leaves a segment's result and goes on to the next segment's rows, and
// the block meets once for all of them.
template <int DH, int GP>
struct Merge {
  static constexpr int kBufs = GP >= 4 ? 16 / GP : 4;
  float m[kBufs][kWarps][GP], l[kBufs][kWarps][GP];
  float o[kBufs][kWarps][GP][DH];
  int bh[kBufs], slot[kBufs];  // whose part it is; partial slot, or -1 where the segment is the whole pair
};

// 1 / l, and 0 where no row counted.
__device__ __forceinline__ float inverse_sum(float l) { return l == 0.f ? 0.f : 1.f / l; }

// Four dims of one head's result; the thread of a head's first dims also
// writes its log-sum-exp (-inf where no row counted).
template <int DH>
__device__ __forceinline__ void write_out(const AttendArgs& a, int bh, int b, int h, int g, int e, float m, float l,
                                          float4 o) {
  const float inv = inverse_sum(l);
  *reinterpret_cast<float4*>(a.out + b * a.osb + (int64_t)(h * a.G + g) * a.osh + e) =
      make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
  if (e == 0) {
    const float L = m + log2f(l);
    if (a.w) a.norm[(int64_t)bh * a.G + g] = make_float2(m, inv);
    if (a.lse) a.lse[(int64_t)bh * a.G + g] = kLn2 * L;
  }
}

// Reduce the warps' parts of a segment: thread i's four dims (i < GP DH / 4).
template <int DH, int GP>
__device__ __forceinline__ void reduce_warps(const Merge<DH, GP>& sm, int buf, int g, int e, float& m, float& l,
                                             float4& o) {
  m = -INFINITY;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) m = fmaxf(m, sm.m[buf][w][g]);
  const float mu = m == -INFINITY ? 0.f : m;
  l = 0.f;
  o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const float f = exp2f(sm.m[buf][w][g] - mu);
    const float4 v = *reinterpret_cast<const float4*>(&sm.o[buf][w][g][e]);
    l = fmaf(sm.l[buf][w][g], f, l);
    o.x = fmaf(v.x, f, o.x);
    o.y = fmaf(v.y, f, o.y);
    o.z = fmaf(v.z, f, o.z);
    o.w = fmaf(v.w, f, o.w);
  }
}

// Reduce `n` segments and write them where they belong: out and lse where a
// segment is the whole pair, else its partial slot.
template <int DH, int GP>
__device__ __forceinline__ void finish_segments(const AttendArgs& a, const Merge<DH, GP>& sm, int n) {
  const int per = a.G * DH / 4;  // threads per segment
#pragma unroll 1
  for (int i = threadIdx.x; i < n * per; i += kThreads) {
    const int buf = i / per, q = i - buf * per, g = q / (DH / 4), e = q % (DH / 4) * 4;
    float m, l;
    float4 o;
    reduce_warps(sm, buf, g, e, m, l, o);
    const int bh = sm.bh[buf], slot = sm.slot[buf];
    if (slot < 0) {
      const int b = bh / a.H;
      write_out<DH>(a, bh, b, bh - b * a.H, g, e, m, l, o);
    } else {
      float* part = a.part + (blockIdx.x * 2 + slot) * (int64_t)kv_part_floats(a.G, DH);
      *reinterpret_cast<float4*>(part + q * 4) = o;
      if (e == 0) {
        part[a.G * DH + g] = m;
        part[a.G * DH + kMaxG + g] = l;
      }
    }
  }
}

// 2^x by the special-function unit alone (relative error 2^-22, results below
// 2^-126 are 0).
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// ---- the rows' way into shared memory
// A warp takes every eighth unit of its CTA's range through a slot for K rows
// and one for V rows of its own: lane 0 issues bulk copies (one per slot where
// a page holds a unit, else a lane per 16 rows its own), a barrier per slot tells when they
// have landed, and a slot is refilled as soon as its rows are in registers.  No
// other warp takes part, so the warps drift freely between the segments' ends.
// Plain copies in this pattern reach 7.3 TB/s with 8 KB copies and 96 to 128 KB
// in flight per SM, 6.6 with 4 KB copies and 192 KB, 5.3 with 2 KB copies; a
// third slot made 64 pairs of 2000 rows 21.1 us instead of 20.2.
struct RingSmem {
  alignas(128) char ring[kWarps][kSlots][kSlotBytes];
  float p[kWarps][33][kMaxG];  // float32 rows: the weights of a unit's rows (at most 32), then the rescaling factors
  int lens[kLensTable];
  uint64_t bar[kWarps][kSlots];
  int dead;  // a wait ran out: nothing more is issued or waited for
};

template <int DH, int GP>
struct AttendSmem {
  RingSmem ring;
  Merge<DH, GP> merge;
};

template <typename E, int DH>
struct Loader {
  static constexpr int kRows = kUnitRows<E, DH>;
  static constexpr int kGroups = kRows / kGroup;  // 1, 2 or 4
  static constexpr int kRowBytes = DH * (int)sizeof(E);
  static constexpr int kBatch = 32 / kGroups;     // units looked up at a time
  const Lens& lens;
  RingSmem& sm;
  const int warp, lane, u_end;
  // The warp's units kBatch at a time: lane i looks up group i % kGroups of the
  // (i / kGroups)-th of them (its pair, then its page), all at once; off: the
  // byte offset of the group's rows in both planes, or -1 where the page is out
  // of range or the group lies behind the last row.
  int u0, nth = 0;
  Place at;
  int64_t off = -1;
  int rows = 0;            // valid rows of the lane's group
  int put = 0, slot = 0;   // copies issued: `put` K and V slots; next slot to fill
  int get = 0, gslot = 0, parity = 0;
  uint32_t good = 0;       // bit k of units issued last in the high bits: group k's rows are there
  bool dead = false;
  const uint64_t policy = sm100::l2_evict_first();  // a step reads its rows once

  __device__ __forceinline__ Loader(const Lens& l_, RingSmem& s_, int w, int l, Place p, int u, int e)
      : lens(l_), sm(s_), warp(w), lane(l), u_end(e), u0(u), at(p) {
    look();
  }
  __device__ __forceinline__ void look() {
    const KvView& c = lens.k;
    const int u = u0 + lane / kGroups * kWarps;
    off = -1;
    rows = 0;
    if (u >= u_end) return;
    lens.seek(at, u);
    const int r = (u - at.s) * kRows + lane % kGroups * kGroup;
    if (r >= at.len) return;
    rows = min(at.len - r, kGroup);
    const int32_t page = c.page(at.bh, r);
    if (page < 0 || page >= c.n_pages)
      c.report((uint32_t)page);
    else
      off = (((int64_t)page << c.page_log) + (r & ((1 << c.page_log) - 1))) * kRowBytes;
  }
  // Issue the next slot's copies: K rows of a unit, then its V rows.
  __device__ __forceinline__ void issue() {
    if (u0 + nth * kWarps >= u_end || dead) return;
    const KvView& c = lens.k;
    const bool is_v = put & 1;
    char* dst = sm.ring[warp][slot];
    uint64_t* bar = &sm.bar[warp][slot];
    const char* plane = is_v ? c.v : c.k;
    const uint32_t have = __ballot_sync(0xffffffffu, off >= 0) >> (nth * kGroups) & ((1u << kGroups) - 1);
    if (!is_v) good = good << kGroups | have;
    const int total = __reduce_add_sync(0xffffffffu, lane / kGroups == nth && off >= 0 ? rows : 0) * kRowBytes;
    // lane 0 has the whole unit where one page does; else each group's lane copies its own
    const bool one = kGroups == 1 || c.page_log >= 4 + (kGroups == 2 ? 1 : 2);
    const int64_t o = one ? __shfl_sync(0xffffffffu, off, nth * kGroups) : off;
    if (lane == 0) {
      if (total)
        sm100::mbar_arrive_expect_tx(bar, total);
      else
        sm100::mbar_arrive(bar);
      if (one && total) sm100::bulk_load_hint(dst, plane + o, total, bar, policy);
    }
    if (!one) {
      __syncwarp();
      if (lane / kGroups == nth && off >= 0)
        sm100::bulk_load_hint(dst + lane % kGroups * kGroup * kRowBytes, plane + o, rows * kRowBytes, bar, policy);
    }
    ++put;
    if (++slot == kSlots) slot = 0;
    if (is_v && ++nth == kBatch) {
      nth = 0;
      u0 += kBatch * kWarps;
      look();
      __syncwarp();
    }
  }
  // Wait for the next slot; null where a wait ran out.
  __device__ __forceinline__ char* take() {
    if (!dead) {
      const bool got = sm100::mbar_wait(&sm.bar[warp][gslot], parity, &sm.dead);
      if (__any_sync(0xffffffffu, !got)) {
        dead = true;
        if (lane == 0) {
          *(volatile int*)&sm.dead = 1;
          latch_error(lens.k.err, DELTAKV_ERR_DEVICE_TIMEOUT, 0u);
        }
      }
    }
    if (dead) return nullptr;
    char* p = sm.ring[warp][gslot];
    ++get;
    if (++gslot == kSlots) {
      gslot = 0;
      parity ^= 1;
    }
    return p;
  }
  // Groups of the unit whose K slot was taken last that hold rows.
  __device__ __forceinline__ uint32_t groups() const {
    // units whose K was issued after it: (K slots issued) - (K slots taken)
    const int later = (put + 1) / 2 - (get + 1) / 2;
    return good >> (later * kGroups) & ((1u << kGroups) - 1);
  }
  // on the way out after a wait ran out: no copy may land in shared memory that the CTA no longer owns
  __device__ void drain() {
    if (dead)
      for (int i = get; i < put; ++i) sm100::mbar_wait_drain(&sm.bar[warp][i % kSlots], (i / kSlots) & 1);
  }
};

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Transpose of an 8x8 matrix of 16-bit elements held two per lane.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float lo_f(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float hi_f(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

// bfloat16 rows on the tensor cores, a unit (32 or 64 rows) a step, in groups
// of 16.  Lane (gr, t) = (lane / 4, lane % 4).  Rows are the M side of both
// products and the pair's query heads (at most 8, zero beyond G) the N side, so
// no product is wasted on padding: X[row][head] = K Q^T, O[dim][head] += V^T P.
//  - X: the contraction index is permuted so that a lane's four 32-bit
//    operands of two k-steps are one 16-byte word of its K row (the same word
//    of the query row), read straight from the row.
//  - O: the rows of M are permuted so that a lane's words of V rows 2t, 2t+1,
//    2t+8, 2t+9 hold its operands once the two rows of a pair are interleaved
//    (byte permutes); P comes out of X's accumulators by an 8x8 transpose.
//  - P in three bfloat16 terms (24 bits of it): with one, each weight would
//    carry 2^-8 into a float32 result.  With GP = 4 heads the second term goes
//    into the columns 4 .. 7 of the first one's product, and with GP = 2 all
//    three into one product: queries repeat over the columns, so that every
//    lane has the weights at hand, and the columns of a head are added up at
//    the segment's end.  An infinite V element would meet the other terms too,
//    which may be zero or negative: a warp whose sums are not finite at the
//    segment's end computes its rows again on the CUDA cores (plain_rows).
//  - A step's products go into zeroed accumulators that are then added to the
//    running ones in float32: the tensor core's own additions may truncate,
//    which over thousands of steps would bias the sums.
template <int DH, int GP_>
struct Bf16Rows {
  using E = __nv_bfloat16;
  static constexpr bool kSplit = true;     // weights in terms: finish() may refuse
  static constexpr int GP = GP_;           // 2, 4 or 8: heads per copy of them in the columns
  static constexpr int kTerms = GP == 8 ? 3 : GP == 4 ? 2 : 1;  // products per group
  static constexpr int kG = kUnitRows<E, DH> / kGroup;
  static constexpr int kW = DH / 32;       // 16-byte words of a K row per lane
  static constexpr int kM = DH / 16;       // M tiles of O
  static constexpr int kH = DH / 64;       // 16-byte words of a V row per lane
  uint32_t q[kW][4];
  float o[kM][4], m[2], l[2];

  __device__ __forceinline__ void start(const AttendArgs& a, int bh, int lane) {
    const int b = bh / a.H, h = bh - b * a.H;
    const int gr = lane >> 2, t = lane & 3;
    const int head = gr & (GP - 1);
    const auto* qp = static_cast<const E*>(a.q) + b * a.qsb + (int64_t)(h * a.G + head) * a.qsh;
#pragma unroll
    for (int i = 0; i < kW; ++i) {
      uint4 v = make_uint4(0u, 0u, 0u, 0u);
      if (head < a.G) v = __ldcg(reinterpret_cast<const uint4*>(qp) + i * 4 + t);
      q[i][0] = v.x;
      q[i][1] = v.y;
      q[i][2] = v.z;
      q[i][3] = v.w;
    }
#pragma unroll
    for (int j = 0; j < kM; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
    m[0] = m[1] = -INFINITY;
    l[0] = l[1] = 0.f;
  }

  // The unit `in` holds next: `valid` rows (at least one); xl: the place of
  // their dot products in global memory, or null.
  __device__ __forceinline__ void step(const AttendArgs& a, Loader<E, DH>& in, int valid, float* xl, int lane) {
    const int gr = lane >> 2, t = lane & 3;
    const char* ks = in.take();
    if (!ks) return;
    const uint32_t have = in.groups();
    float x[kG][4];
#pragma unroll
    for (int n = 0; n < kG; ++n) {
      float x0[4] = {0.f, 0.f, 0.f, 0.f}, x1[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < kW; ++i) {
        const uint4 ka = *reinterpret_cast<const uint4*>(ks + (n * kGroup + gr) * DH * 2 + (i * 4 + t) * 16);
        const uint4 kb = *reinterpret_cast<const uint4*>(ks + (n * kGroup + gr + 8) * DH * 2 + (i * 4 + t) * 16);
        mma_bf16(x0, ka.x, kb.x, ka.y, kb.y, q[i][0], q[i][1]);
        mma_bf16(x1, ka.z, kb.z, ka.w, kb.w, q[i][2], q[i][3]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) x[n][i] = x0[i] + x1[i];
    }
    __syncwarp();
    in.issue();
    const bool full = valid == kG * kGroup && have == (1u << kG) - 1;
    if (!full) {
      // rows that do not count: whatever the slot holds
#pragma unroll
      for (int n = 0; n < kG; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (n * kGroup + gr + (i >> 1) * 8 >= valid || !(have >> n & 1)) x[n][i] = -INFINITY;
    }
    if (xl && 2 * t < a.G && 2 * t < GP) {
      const bool two = (a.G & 1) == 0;  // both heads of the lane in one store
#pragma unroll
      for (int n = 0; n < kG; ++n)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const int row = n * kGroup + gr + hf * 8;
          if (row >= valid) continue;
          float* xp = xl + row * a.G + 2 * t;
          if (two) {
            *reinterpret_cast<float2*>(xp) = make_float2(x[n][2 * hf], x[n][2 * hf + 1]);
          } else {
            xp[0] = x[n][2 * hf];
            if (2 * t + 1 < a.G) xp[1] = x[n][2 * hf + 1];
          }
        }
    }
    float f[2];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      float mx = -INFINITY;
#pragma unroll
      for (int n = 0; n < kG; ++n) mx = fmaxf(mx, fmaxf(x[n][c], x[n][c + 2]));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
      mx = fmaxf(m[c], mx * a.scale2);
      const float mu = mx == -INFINITY ? 0.f : mx;
      f[c] = ex2(m[c] - mu);
      m[c] = mx;
      l[c] *= f[c];
#pragma unroll
      for (int n = 0; n < kG; ++n) {
        x[n][c] = ex2(fmaf(x[n][c], a.scale2, -mu));
        x[n][c + 2] = ex2(fmaf(x[n][c + 2], a.scale2, -mu));
        l[c] += x[n][c] + x[n][c + 2];
      }
    }
    uint32_t pb[kG][kTerms][2];
#pragma unroll
    for (int n = 0; n < kG; ++n)
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        uint32_t w[3];
#pragma unroll
        for (int s = 0; s < 3; ++s) {
          w[s] = pack_bf16(x[n][2 * hf], x[n][2 * hf + 1]);
          x[n][2 * hf] -= lo_f(w[s]);
          x[n][2 * hf + 1] -= hi_f(w[s]);
        }
        if constexpr (GP == 8) {
#pragma unroll
          for (int s = 0; s < 3; ++s) pb[n][s][hf] = transpose8(w[s]);
        } else if constexpr (GP == 4) {
          pb[n][0][hf] = transpose8(t < 2 ? w[0] : w[1]);
          pb[n][1][hf] = transpose8(t < 2 ? w[2] : 0u);
        } else {
          pb[n][0][hf] = transpose8(t == 0 ? w[0] : t == 1 ? w[1] : t == 2 ? w[2] : 0u);
        }
      }
    const char* vs = in.take();
    if (!vs) return;
    float c[kM][4];
#pragma unroll
    for (int j = 0; j < kM; ++j) c[j][0] = c[j][1] = c[j][2] = c[j][3] = 0.f;
#pragma unroll
    for (int n = 0; n < kG; ++n) {
      // V rows 2t, 2t + 1, 2t + 8, 2t + 9 of the group: words gr (and gr + 8)
      uint4 v[kH][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = n * kGroup + 2 * t + (i & 1) + (i >> 1) * 8;
#pragma unroll
        for (int w = 0; w < kH; ++w) {
          v[w][i] = *reinterpret_cast<const uint4*>(vs + row * DH * 2 + (w * 8 + gr) * 16);
          if (!full && (row >= valid || !(have >> n & 1))) v[w][i] = make_uint4(0u, 0u, 0u, 0u);
        }
      }
      if (n == kG - 1) {
        __syncwarp();
        in.issue();
      }
      outputs(c, v, pb[n]);
    }
#pragma unroll
    for (int j = 0; j < kM; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[j][i] = fmaf(o[j][i], f[i & 1], c[j][i]);
  }

  // C += V^T P for one group, four M tiles at a time, so that their chains of
  // products overlap.
  __device__ __forceinline__ void outputs(float (&c)[kM][4], const uint4 (&v)[kH][4], const uint32_t (&pb)[kTerms][2]) {
#pragma unroll
    for (int j0 = 0; j0 < kM; j0 += 4) {
      uint32_t av[4][4];
#pragma unroll
      for (int jj = 0; jj < 4; ++jj) {
        // M rows gr and gr + 8 of tile j: dims 8 gr + j and 64 + 8 gr + j (DH 128), 8 gr + 2 j and 8 gr + 2 j + 1 (64)
        const int j = j0 + jj;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int up = i & 1, pr = i >> 1;  // a0: rows gr, tokens 2t..; a1: rows gr + 8; a2, a3: tokens 2t + 8..
          const uint32_t* ra = reinterpret_cast<const uint32_t*>(&v[kH == 2 ? up : 0][2 * pr]);
          const uint32_t* rb = reinterpret_cast<const uint32_t*>(&v[kH == 2 ? up : 0][2 * pr + 1]);
          const int word = kH == 2 ? j >> 1 : j;
          const bool high = kH == 2 ? j & 1 : up;
          av[jj][i] = __byte_perm(ra[word], rb[word], high ? 0x7632 : 0x5410);
        }
      }
#pragma unroll
      for (int s = kTerms - 1; s >= 0; --s)
#pragma unroll
        for (int jj = 0; jj < 4; ++jj)
          mma_bf16(c[j0 + jj], av[jj][0], av[jj][1], av[jj][2], av[jj][3], pb[s][0], pb[s][1]);
    }
  }

  // Leave the warp's result; false where it is not finite (it is then computed another way).
  __device__ __forceinline__ bool finish(Merge<DH, GP>& mg, int buf, int warp, int lane) {
    const int gr = lane >> 2, t = lane & 3;
    float z = 0.f;  // 0, or NaN
#pragma unroll
    for (int j = 0; j < kM; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) z = fmaf(o[j][i], 0.f, z);
    if (__any_sync(0xffffffffu, z != 0.f)) return false;
    // add up the columns of a head
    if constexpr (GP < 8) {
#pragma unroll
      for (int j = 0; j < kM; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          o[j][i] += __shfl_xor_sync(0xffffffffu, o[j][i], 2);
          if (GP == 2) o[j][i] += __shfl_xor_sync(0xffffffffu, o[j][i], 1);
        }
    }
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      l[c] += __shfl_xor_sync(0xffffffffu, l[c], 4);
      l[c] += __shfl_xor_sync(0xffffffffu, l[c], 8);
      l[c] += __shfl_xor_sync(0xffffffffu, l[c], 16);
    }
    if (2 * t >= GP) return true;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      if (gr == 0) {
        mg.m[buf][warp][2 * t + c] = m[c];
        mg.l[buf][warp][2 * t + c] = l[c];
      }
      float* op = mg.o[buf][warp][2 * t + c] + gr * 8;
      if constexpr (DH == 128) {
#pragma unroll
        for (int w = 0; w < 2; ++w)
#pragma unroll
          for (int j = 0; j < 8; j += 4)
            *reinterpret_cast<float4*>(op + w * 64 + j) =
                make_float4(o[j][2 * w + c], o[j + 1][2 * w + c], o[j + 2][2 * w + c], o[j + 3][2 * w + c]);
      } else {
#pragma unroll
        for (int j = 0; j < 4; j += 2)
          *reinterpret_cast<float4*>(op + 2 * j) = make_float4(o[j][c], o[j][2 + c], o[j + 1][c], o[j + 1][2 + c]);
      }
    }
    return true;
  }
};

// float32 rows on the CUDA cores (float32 results leave no room for tf32's
// 2^-11).  Logits: kL lanes per row, a lane holds DH / kL elements of every
// head's query in registers (64 at most: kL is 4 to 16 by the heads); the GP
// heads' partial sums are reduced over the kL lanes by exchange steps that
// leave each lane one head.  Outputs: a lane holds four dims of all heads and
// reads the rows' weights from shared memory.  Bound by issue: d_h 64, eight
// heads, 226 MB 48 us (4.7 TB/s; 76 us with 32 lanes per row).
// GP: heads rounded up to a power of two.
template <int DH, int GP_>
struct F32Rows {
  using E = float;
  static constexpr bool kSplit = false;    // weights as they are: every result is the formula's
  static constexpr int GP = GP_;
  static constexpr int kRows = kUnitRows<float, DH>;
  static constexpr int kL = DH * GP / 64 < 4 ? 4 : DH * GP / 64;  // 4, 8 or 16
  static constexpr int kC = DH / (4 * kL);                        // 16-byte words of a row per lane
  static constexpr int kPer = 32 / kL;                            // rows per pass
  static constexpr int kPasses = kRows / kPer;
  static constexpr int kV = DH / 4;                               // lanes per V row: 32 or 16
  static_assert(GP <= kL && kL <= 16 && kRows % kPer == 0, "");
  float4 q[GP][kC], o[GP];
  float m, l;

  __device__ __forceinline__ static int head_of(int lane) {
    int n = GP, h = 0;
#pragma unroll
    for (int s = kL / 2; s > 0; s >>= 1)
      if (n > 1) {
        n >>= 1;
        h += (lane & s) ? n : 0;
      }
    return h;
  }
  // the i-th word of a row that a lane holds; with four lanes per row, the rows of a pair take their words in opposite
  // order of halves, so that eight lanes' reads meet all banks
  __device__ __forceinline__ static int word_of(int i, int lane) {
    return (i * kL + lane % kL) ^ (kL == 4 && (lane / kL & 1) ? kL : 0);
  }

  __device__ __forceinline__ void start(const AttendArgs& a, int bh, int lane) {
    const int b = bh / a.H, h = bh - b * a.H;
    const auto* qp = static_cast<const float*>(a.q) + b * a.qsb + (int64_t)(h * a.G) * a.qsh;
#pragma unroll
    for (int g = 0; g < GP; ++g) {
#pragma unroll
      for (int i = 0; i < kC; ++i)
        q[g][i] = g < a.G ? __ldcg(reinterpret_cast<const float4*>(qp + g * a.qsh) + word_of(i, lane))
                          : make_float4(0.f, 0.f, 0.f, 0.f);
      o[g] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    m = -INFINITY;
    l = 0.f;
  }

  // The unit `in` holds next: `valid` rows (at least one); xl: the place of
  // their dot products in global memory, or null.
  __device__ __forceinline__ void step(const AttendArgs& a, Loader<float, DH>& in, int valid, float* xl, int lane) {
    const char* ks = in.take();
    if (!ks) return;
    const uint32_t have = in.groups();
    float* p_smem = &in.sm.p[in.warp][0][0];
    const int head = head_of(lane);
    float x[kPasses];
    float mx = -INFINITY;
#pragma unroll
    for (int j = 0; j < kPasses; ++j) {
      const int row = j * kPer + lane / kL;
      float v[GP];
#pragma unroll
      for (int g = 0; g < GP; ++g) v[g] = 0.f;
#pragma unroll
      for (int i = 0; i < kC; ++i) {
        const float4 kx = *reinterpret_cast<const float4*>(ks + row * DH * 4 + word_of(i, lane) * 16);
#pragma unroll
        for (int g = 0; g < GP; ++g)
          v[g] = fmaf(q[g][i].x, kx.x, fmaf(q[g][i].y, kx.y, fmaf(q[g][i].z, kx.z, fmaf(q[g][i].w, kx.w, v[g]))));
      }
      int n = GP;
#pragma unroll
      for (int s = kL / 2; s > 0; s >>= 1) {
        if (n > 1) {
          n >>= 1;
#pragma unroll
          for (int i = 0; i < GP / 2; ++i)
            if (i < n) {
              const float keep = (lane & s) ? v[i + n] : v[i], send = (lane & s) ? v[i] : v[i + n];
              v[i] = keep + __shfl_xor_sync(0xffffffffu, send, s);
            }
        } else {
          v[0] += __shfl_xor_sync(0xffffffffu, v[0], s);
        }
      }
      x[j] = v[0];
    }
    __syncwarp();  // every lane has read its K rows, and the last unit's weights
    in.issue();
    const bool full = valid == kRows && have == (1u << (kRows / kGroup)) - 1;
    if (!full) {
      // rows that do not count: whatever the slot holds
#pragma unroll
      for (int j = 0; j < kPasses; ++j) {
        const int row = j * kPer + lane / kL;
        if (row >= valid || !(have >> (row / kGroup) & 1)) x[j] = -INFINITY;
      }
    }
    if (xl && head < a.G && (lane & (kL / GP - 1)) == 0) {
#pragma unroll
      for (int j = 0; j < kPasses; ++j) {
        const int row = j * kPer + lane / kL;
        if (row < valid) xl[row * a.G + head] = x[j];
      }
    }
#pragma unroll
    for (int j = 0; j < kPasses; ++j) mx = fmaxf(mx, x[j]);
#pragma unroll
    for (int s = kL; s < 32; s <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, s));
    mx = fmaxf(m, mx * a.scale2);
    const float mu = mx == -INFINITY ? 0.f : mx;
    const float f = ex2(m - mu);
    m = mx;
    l *= f;
#pragma unroll
    for (int j = 0; j < kPasses; ++j) {
      const float p = ex2(fmaf(x[j], a.scale2, -mu));
      l += p;
      p_smem[(j * kPer + lane / kL) * kMaxG + head] = p;
    }
    p_smem[kRows * kMaxG + head] = f;
    __syncwarp();
    const char* vs = in.take();
    if (!vs) return;
    float w[GP];
    weights(p_smem, kRows, w);
#pragma unroll
    for (int g = 0; g < GP; ++g) o[g] = make_float4(o[g].x * w[g], o[g].y * w[g], o[g].z * w[g], o[g].w * w[g]);
    if (full) {
#pragma unroll 8
      for (int r = 0; r < kRows; r += 32 / kV) add_row(vs, p_smem, r + lane / kV, lane);
    } else {
#pragma unroll 1
      for (int r = 0; r < kRows; r += 32 / kV) {
        const int row = r + lane / kV;
        if (row < valid && (have >> (row / kGroup) & 1)) add_row(vs, p_smem, row, lane);
      }
    }
    __syncwarp();
    in.issue();
  }

  __device__ __forceinline__ static void weights(const float* p_smem, int row, float (&w)[GP]) {
    const float* pp = p_smem + row * kMaxG;
    if constexpr (GP >= 4) {
#pragma unroll
      for (int g = 0; g < GP; g += 4) {
        const float4 t = *reinterpret_cast<const float4*>(pp + g);
        w[g] = t.x;
        w[g + 1] = t.y;
        w[g + 2] = t.z;
        w[g + 3] = t.w;
      }
    } else {
#pragma unroll
      for (int g = 0; g < GP; ++g) w[g] = pp[g];
    }
  }
  __device__ __forceinline__ void add_row(const char* vs, const float* p_smem, int row, int lane) {
    const float4 v = *reinterpret_cast<const float4*>(vs + row * DH * 4 + lane % kV * 16);
    float w[GP];
    weights(p_smem, row, w);
#pragma unroll
    for (int g = 0; g < GP; ++g) {
      o[g].x = fmaf(w[g], v.x, o[g].x);
      o[g].y = fmaf(w[g], v.y, o[g].y);
      o[g].z = fmaf(w[g], v.z, o[g].z);
      o[g].w = fmaf(w[g], v.w, o[g].w);
    }
  }

  __device__ __forceinline__ void finish(Merge<DH, GP>& mg, int buf, int warp, int lane) {
#pragma unroll
    for (int s = kL; s < 32; s <<= 1) l += __shfl_xor_sync(0xffffffffu, l, s);
    const int head = head_of(lane);
    mg.m[buf][warp][head] = m;
    mg.l[buf][warp][head] = l;
#pragma unroll
    for (int g = 0; g < GP; ++g) {
      if constexpr (kV == 16) {
        o[g].x += __shfl_xor_sync(0xffffffffu, o[g].x, 16);
        o[g].y += __shfl_xor_sync(0xffffffffu, o[g].y, 16);
        o[g].z += __shfl_xor_sync(0xffffffffu, o[g].z, 16);
        o[g].w += __shfl_xor_sync(0xffffffffu, o[g].w, 16);
      }
      if (lane < kV) *reinterpret_cast<float4*>(&mg.o[buf][warp][g][lane * 4]) = o[g];
    }
  }
};

// A warp's units u, u + kWarps, .. < ue of a bfloat16 pair (at), computed row by row in
// float32 from global memory, for sums that an infinity or a NaN among the rows
// made worthless: every product is then one of a weight and a value, as in the
// formula.
template <int DH, int GP>
__device__ __noinline__ void plain_rows(const AttendArgs& a, Merge<DH, GP>& mg, int buf, Place at, int u, int ue,
                                        int warp, int lane) {
  constexpr int kN = DH / 32;
  const int b = at.bh / a.H, h = at.bh - b * a.H;
  for (int g = 0; g < GP; ++g) {
    float q[kN], o[kN], m = -INFINITY, l = 0.f;
    const auto* qp = static_cast<const __nv_bfloat16*>(a.q) + b * a.qsb + (int64_t)(h * a.G + g) * a.qsh;
    for (int i = 0; i < kN; ++i) {
      q[i] = g < a.G ? to_f(qp[i * 32 + lane]) : 0.f;
      o[i] = 0.f;
    }
    for (int n = u; g < a.G && n < ue; n += kWarps) {
      const int r0 = (n - at.s) << a.unit_log, r1 = min(at.len, r0 + (1 << a.unit_log));
      for (int r = r0; r < r1; ++r) {
        const int64_t row = a.c.row(at.bh, r);
        if (row < 0) continue;
        const auto* kr = reinterpret_cast<const __nv_bfloat16*>(a.c.k) + row * DH;
        const auto* vr = reinterpret_cast<const __nv_bfloat16*>(a.c.v) + row * DH;
        float x = 0.f;
        for (int i = 0; i < kN; ++i) x = fmaf(q[i], to_f(kr[i * 32 + lane]), x);
        x = warp_sum(x);
        const float mx = fmaxf(m, x * a.scale2), mu = mx == -INFINITY ? 0.f : mx;
        const float f = exp2f(m - mu), p = exp2f(fmaf(x, a.scale2, -mu));
        m = mx;
        l = fmaf(l, f, p);
        for (int i = 0; i < kN; ++i) o[i] = fmaf(o[i], f, p * to_f(vr[i * 32 + lane]));
      }
    }
    if (lane == 0) {
      mg.m[buf][warp][g] = m;
      mg.l[buf][warp][g] = l;
    }
    for (int i = 0; i < kN; ++i) mg.o[buf][warp][g][i * 32 + lane] = o[i];
  }
}

// Leave a warp's result for its units u, u + kWarps, .. < ue of a pair (at).
template <int DH, typename Rows>
__device__ __forceinline__ void leave_result(const AttendArgs& a, Rows& rows, Merge<DH, Rows::GP>& mg, int buf, Place at,
                                             int u, int ue, int warp, int lane) {
  if constexpr (Rows::kSplit) {
    if (!rows.finish(mg, buf, warp, lane)) plain_rows(a, mg, buf, at, u, ue, warp, lane);
  } else {
    rows.finish(mg, buf, warp, lane);
  }
}

__device__ __forceinline__ void init_ring(RingSmem& ring, int warp, int lane) {
  if (lane == 0) {
    for (int i = 0; i < kSlots; ++i) sm100::mbar_init(&ring.bar[warp][i], 1);
    sm100::fence_mbar_init();
  }
  if (threadIdx.x == 0) ring.dead = 0;
}

// One CTA per SM, eight warps with a ring each.  bf16, d_h 128, four heads: 64
// pairs of 131072 rows (4.3 GB) 607 us, 7.1 TB/s, in a short run; 628 to 682 us,
// 6.3 to 6.8 TB/s, in a long one under the power limit.
template <int DH, typename Rows>
__global__ void __launch_bounds__(kThreads, 1) kv_attend_kernel(const __grid_constant__ AttendArgs a) {
  using E = typename Rows::E;
  constexpr int kRows = kUnitRows<E, DH>;
  using M = Merge<DH, Rows::GP>;
  extern __shared__ __align__(128) char smem_raw[];
  auto& sm = *reinterpret_cast<AttendSmem<DH, Rows::GP>*>(smem_raw);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  init_ring(sm.ring, warp, lane);
  sm100::grid_dep_wait();
  sm100::grid_dep_launch();
  Place at;
  bool empty;
  const int c = blockIdx.x;
  const Cut cut = locate(a, c, reinterpret_cast<int*>(sm.merge.o), sm.ring.lens, at, empty);
  if (c >= cut.g) return;
  const int u_first = cut.start(c), u_end = cut.start(c + 1);
  Rows rows;
  rows.start(a, at.bh, lane);
  static_assert(kLensTable == kThreads, "a thread per entry");
  int bh0 = 0;  // locate() has left the lengths where they fit the table
  if (a.BH > kLensTable) {
    bh0 = at.bh;
    sm.ring.lens[threadIdx.x] = bh0 + (int)threadIdx.x < a.BH ? a.c.len(bh0 + threadIdx.x) : 0;
    __syncthreads();
  }
  const Lens lens{a.c, sm.ring.lens, bh0, a.unit_log};
  int u = u_first, mine = u + warp;  // this warp's next unit
  Loader<E, DH> in(lens, sm.ring, warp, lane, at, mine, u_end);
  for (int i = 0; i < kSlots; ++i) in.issue();
  int held = 0;  // segments in the merge buffers
#pragma unroll 1
  while (u < u_end) {
    const int ub = units_of(at.len, a.unit_log);
    const int ue = min(u_end, at.s + ub);
#pragma unroll 1
    for (; mine < ue; mine += kWarps) {
      const int r = (mine - at.s) * kRows;
      float* xl = a.w ? a.dots + ((int64_t)at.bh * a.c.max_len + r) * a.G : nullptr;
      rows.step(a, in, min(at.len - r, kRows), xl, lane);
    }
    leave_result<DH>(a, rows, sm.merge, held, at, u + ((u_first + warp - u) & (kWarps - 1)), ue, warp, lane);
    if (threadIdx.x == 0) {
      sm.merge.bh[held] = at.bh;
      sm.merge.slot[held] = u == at.s && ue == at.s + ub ? -1 : u == u_first ? 0 : 1;
    }
    ++held;
    u = ue;
    // the next pair's queries are on their way while this one is reduced (after the last, the same pair's again)
    lens.seek(at, min(u, u_end - 1));
    rows.start(a, at.bh, lane);
    if (held == M::kBufs || u >= u_end) {
      __syncthreads();
      finish_segments(a, sm.merge, held);
      __syncthreads();
      held = 0;
    }
  }
  in.drain();
}

// The softmax weight of a row with dot product d; norm: (m, 1 / l).  Without a
// maximum (m is -inf) no row counts for the head and 1 / l was set to 0, or the
// rows that would are NaN and l is.
__device__ __forceinline__ float weight_of(float d, float2 norm, float scale2) {
  return norm.x == -INFINITY ? norm.y : exp2f(fmaf(d, scale2, -norm.x)) * norm.y;
}

// Short rows: a cluster per pair, its CTAs equal runs of the pair's units, the
// parts joined through distributed shared memory and the weights added by the
// CTA that has the rows, all in one kernel.  Bound by its chain of latencies
// (length, page, rows, reduction, cluster barrier), not by bandwidth.
template <int DH, typename Rows>
__global__ void __launch_bounds__(kThreads, 1) kv_attend_short_kernel(const __grid_constant__ AttendArgs a, int C) {
  namespace cg = cooperative_groups;
  using E = typename Rows::E;
  constexpr int kRows = kUnitRows<E, DH>;
  extern __shared__ __align__(128) char smem_raw[];
  auto& sm = *reinterpret_cast<AttendSmem<DH, Rows::GP>*>(smem_raw);
  const cg::cluster_group cl = cg::this_cluster();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int bh = blockIdx.x / C, rank = blockIdx.x - bh * C;
  init_ring(sm.ring, warp, lane);
  __syncthreads();
  sm100::grid_dep_wait();
  sm100::grid_dep_launch();
  const int raw = a.c.raw_len(bh), len = a.c.checked(raw);
  if (rank == 0 && threadIdx.x == 0 && raw != len) a.c.report((uint32_t)raw);
  const int ub = units_of(len, a.unit_log);
  const int u0 = ub * rank / C, u1 = ub * (rank + 1) / C;
  const Place at{bh, 0, len};
  const Lens lens{a.c, sm.ring.lens, bh, a.unit_log};  // (no unit lies past this pair: the table is not read)
  Loader<E, DH> in(lens, sm.ring, warp, lane, at, u0 + warp, u1);
  for (int i = 0; i < kSlots; ++i) in.issue();
  Rows rows;
  rows.start(a, bh, lane);
#pragma unroll 1
  for (int u = u0 + warp; u < u1; u += kWarps) {
    const int r = u * kRows;
    float* xl = a.w ? a.dots + ((int64_t)bh * a.c.max_len + r) * a.G : nullptr;
    rows.step(a, in, min(len - r, kRows), xl, lane);
  }
  leave_result<DH>(a, rows, sm.merge, 0, at, u0 + warp, u1, warp, lane);
  in.drain();
  __syncthreads();
  // this CTA's part, where the rows were: o[G][DH], m[kMaxG], l[kMaxG]
  float* part = reinterpret_cast<float*>(sm.ring.ring);
  const int cols = a.G * DH / 4;
  if ((int)threadIdx.x < cols) {
    const int g = threadIdx.x / (DH / 4), e = threadIdx.x % (DH / 4) * 4;
    float m, l;
    float4 o;
    reduce_warps(sm.merge, 0, g, e, m, l, o);
    *reinterpret_cast<float4*>(part + threadIdx.x * 4) = o;
    if (e == 0) {
      part[kMaxG * DH + g] = m;
      part[kMaxG * DH + kMaxG + g] = l;
    }
  }
  if (C == 1)
    __syncthreads();
  else
    cl.sync();
  auto peer = [&](int c) { return C == 1 ? part : cl.map_shared_rank(part, c); };
  const int b = bh / a.H, h = bh - b * a.H;
  for (int q = cols * rank / C + threadIdx.x; q < cols * (rank + 1) / C; q += kThreads) {
    const int g = q / (DH / 4);
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int c = 0; c < C; ++c) m = fmaxf(m, peer(c)[kMaxG * DH + g]);
    const float mu = m == -INFINITY ? 0.f : m;
    for (int c = 0; c < C; ++c) {
      const float* p = peer(c);
      const float f = exp2f(p[kMaxG * DH + g] - mu);
      const float4 v = reinterpret_cast<const float4*>(p)[q];
      l = fmaf(f, p[kMaxG * DH + kMaxG + g], l);
      o.x = fmaf(f, v.x, o.x);
      o.y = fmaf(f, v.y, o.y);
      o.z = fmaf(f, v.z, o.z);
      o.w = fmaf(f, v.w, o.w);
    }
    write_out<DH>(a, bh, b, h, g, q * 4 % DH, m, l, o);
  }
  if (a.w) {
    float2* norm = reinterpret_cast<float2*>(part + kMaxG * DH + 2 * kMaxG);
    if ((int)threadIdx.x < a.G) {
      const int g = threadIdx.x;
      float m = -INFINITY, l = 0.f;
      for (int c = 0; c < C; ++c) m = fmaxf(m, peer(c)[kMaxG * DH + g]);
      const float mu = m == -INFINITY ? 0.f : m;
      for (int c = 0; c < C; ++c) l = fmaf(exp2f(peer(c)[kMaxG * DH + g] - mu), peer(c)[kMaxG * DH + kMaxG + g], l);
      norm[g] = make_float2(m, inverse_sum(l));
    }
    __syncthreads();
    for (int r = u0 * kRows + threadIdx.x; r < min(len, u1 * kRows); r += kThreads) {
      const float* x = a.dots + ((int64_t)bh * a.c.max_len + r) * a.G;
      float* w = a.w + bh * a.cap + r;
      const float old = *w;
      float p = 0.f;
      for (int g = 0; g < a.G; ++g) p += weight_of(__ldcg(x + g), norm[g], a.scale2);
      *w = fmaf(a.decay, old, p);
    }
  }
  if (C > 1) cl.sync();  // no CTA leaves while another reads its part
}

// Join the partial results.  CTA j looks at the cut between ranges j and j + 1:
// where it falls inside a pair, that pair has np >= 2 parts and np - 1 such
// cuts inside, and the CTA of cut i joins share i of the pair's G d_h outputs.
// A warp takes cp words of four outputs, its lanes beyond those the parts in
// turn: a lane loads its parts' (m, l, o) at once and folds them, then the
// lanes of the same word fold (a fixed order: the result does not depend on
// timing).  One round trip to L2 after the attention's end, the search for the
// cut runs before it: 3.5 us with the launch, whatever the lengths.
template <int DH>
__global__ void __launch_bounds__(kThreads) kv_join_kernel(const __grid_constant__ AttendArgs a) {
  __shared__ int sh_loc[kLocateWords];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Place at;
  bool empty;
  // the lengths were final before the first kernel passed its own wait
  const int c = blockIdx.x + 1;
  const Cut cut = locate(a, c, sh_loc, nullptr, at, empty);
  int q0 = 0, q1 = 0, c0 = 0, np = 0, slot0 = 0, b = 0, h = 0;
  if (c < cut.g && cut.start(c) != at.s) {
    c0 = cut.range_of(at.s);
    np = cut.range_of(at.s + units_of(at.len, a.unit_log) - 1) - c0 + 1;
    const int cols = a.G * DH / 4, share = c - c0 - 1;
    q0 = cols * share / (np - 1);
    q1 = cols * (share + 1) / (np - 1);
    // range c0's part of this pair is its first segment only where the range begins with the pair
    slot0 = cut.start(c0) == at.s ? 0 : 1;
    b = at.bh / a.H;
    h = at.bh - b * a.H;
  }
  const int stride = kv_part_floats(a.G, DH);
  int cp = 8;  // words per warp; as few as there are, so that more lanes share the parts
  while (cp > 1 && cp >= 2 * (q1 - q0)) cp >>= 1;
  const int groups = 32 / cp, grp = lane / cp;
  sm100::grid_dep_wait();
  sm100::grid_dep_launch();
  if (empty) {
    for (int e = blockIdx.x; e < a.BH; e += gridDim.x) {
      if (a.c.len(e) != 0) continue;
      const int eb = e / a.H, eh = e - eb * a.H;
      for (int i = threadIdx.x * 4; i < a.G * DH; i += kThreads * 4)
        write_out<DH>(a, e, eb, eh, i / DH, i % DH, -INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f));
    }
  }
  for (int qb = q0 + warp * cp; qb < q1; qb += kWarps * cp) {
    const int q = min(qb + lane % cp, q1 - 1), g = q / (DH / 4);
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    auto fold = [&](float m2, float l2, float4 o2) {
      const float mx = fmaxf(m, m2), mu = mx == -INFINITY ? 0.f : mx;
      const float f = exp2f(m - mu), f2 = exp2f(m2 - mu);
      m = mx;
      l = fmaf(l, f, l2 * f2);
      o.x = fmaf(o.x, f, o2.x * f2);
      o.y = fmaf(o.y, f, o2.y * f2);
      o.z = fmaf(o.z, f, o2.z * f2);
      o.w = fmaf(o.w, f, o2.w * f2);
    };
#pragma unroll 4
    for (int i = grp; i < np; i += groups) {
      const float* part = a.part + ((c0 + i) * 2 + (i == 0 ? slot0 : 0)) * (int64_t)stride;
      const float pm = __ldcg(part + a.G * DH + g), pl = __ldcg(part + a.G * DH + kMaxG + g);
      fold(pm, pl, __ldcg(reinterpret_cast<const float4*>(part) + q));
    }
    for (int s = cp; s < 32; s <<= 1) {
      const float m2 = __shfl_xor_sync(0xffffffffu, m, s), l2 = __shfl_xor_sync(0xffffffffu, l, s);
      const float4 o2 = make_float4(__shfl_xor_sync(0xffffffffu, o.x, s), __shfl_xor_sync(0xffffffffu, o.y, s),
                                    __shfl_xor_sync(0xffffffffu, o.z, s), __shfl_xor_sync(0xffffffffu, o.w, s));
      fold(m2, l2, o2);
    }
    if (grp == 0 && qb + lane < q1) write_out<DH>(a, at.bh, b, h, g, q * 4 % DH, m, l, o);
  }
}

// w_r <- decay w_r + sum over heads of 2^(c d_r - m) / l: a CTA takes 1024 rows of a
// pair, a thread four of them 256 rows apart.  Bound by the dot products and
// weights it reads and writes (4 G + 8 bytes a row): 64 pairs of 2048 to 16384
// rows, G = 4, 4 to 5 us.
constexpr int kWeightRows = 4 * kThreads;

// V: dot products per load, the largest of 4, 2, 1 that divides G.
template <int V>
__global__ void __launch_bounds__(kThreads) kv_weights_kernel(const __grid_constant__ AttendArgs a, int chunks) {
  const int bh = blockIdx.x / chunks, r0 = (blockIdx.x - bh * chunks) * kWeightRows + threadIdx.x;
  const int len = a.c.len(bh);  // final before the first kernel of the call passed its wait
  sm100::grid_dep_wait();
  if (r0 >= len) return;
  const int n = a.G / V;
  const float2* np = a.norm + (int64_t)bh * a.G;
  const float* x = a.dots + ((int64_t)bh * a.c.max_len + r0) * a.G;
  float* w = a.w + bh * a.cap + r0;
  float old[4], p[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 4; ++i) old[i] = r0 + i * kThreads < len ? __ldcg(w + i * kThreads) : 0.f;
#pragma unroll
  for (int k = 0; k < kMaxG / V; ++k) {
    if (k >= n) break;
    float v[4][V];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float* xp = x + (int64_t)i * kThreads * a.G + k * V;
      const bool in = r0 + i * kThreads < len;
      if constexpr (V == 4) {
        const float4 t = in ? __ldcg(reinterpret_cast<const float4*>(xp)) : make_float4(0.f, 0.f, 0.f, 0.f);
        v[i][0] = t.x;
        v[i][1] = t.y;
        v[i][2] = t.z;
        v[i][3] = t.w;
      } else if constexpr (V == 2) {
        const float2 t = in ? __ldcg(reinterpret_cast<const float2*>(xp)) : make_float2(0.f, 0.f);
        v[i][0] = t.x;
        v[i][1] = t.y;
      } else {
        v[i][0] = in ? __ldcg(xp) : 0.f;
      }
    }
#pragma unroll
    for (int g = 0; g < V; ++g) {
      const float2 norm = __ldcg(np + k * V + g);
#pragma unroll
      for (int i = 0; i < 4; ++i) p[i] += weight_of(v[i][g], norm, a.scale2);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (r0 + i * kThreads < len) w[i * kThreads] = fmaf(a.decay, old[i], p[i]);
}

template <int DH, typename Rows>
cudaError_t launch_t(const Plan& p, const AttendArgs& a, int grid, int cluster, cudaStream_t st) {
  if (cluster) {
    auto kern = kv_attend_short_kernel<DH, Rows>;
    constexpr size_t smem = sizeof(AttendSmem<DH, Rows::GP>);
    static std::atomic<uint64_t> ready{0};
    cudaError_t e = allow_smem((const void*)kern, smem, ready);
    if (e != cudaSuccess) return e;
    ProfScope ps(p, st, KID_KV_ATTEND_SHORT);
    return launch_pdl_cluster(kern, (unsigned)(a.BH * cluster), kThreads, cluster, smem, st, a, cluster);
  }
  auto kern = kv_attend_kernel<DH, Rows>;
  constexpr size_t smem = sizeof(AttendSmem<DH, Rows::GP>);
  static_assert(smem <= 227 * 1024, "shared memory of one CTA");
  static std::atomic<uint64_t> ready{0};  // a bit per device: the attribute is the device's
  cudaError_t e = allow_smem((const void*)kern, smem, ready);
  if (e != cudaSuccess) return e;
  {
    ProfScope ps(p, st, KID_KV_ATTEND);
    e = launch_pdl(kern, grid, kThreads, smem, st, a);
  }
  if (e != cudaSuccess) return e;
  static std::atomic<uint64_t> ready_join{0};
  e = allow_smem((const void*)kv_join_kernel<DH>, 0, ready_join);
  if (e != cudaSuccess) return e;
  {
    ProfScope ps(p, st, KID_KV_JOIN);
    e = launch_pdl(kv_join_kernel<DH>, grid, kThreads, 0, st, a);
  }
  if (e != cudaSuccess || !a.w) return e;
  const int chunks = (int)ceil_div64(a.c.max_len, kWeightRows);
  auto weights = a.G % 4 == 0 ? kv_weights_kernel<4> : a.G % 2 == 0 ? kv_weights_kernel<2> : kv_weights_kernel<1>;
  ProfScope ps(p, st, KID_KV_WEIGHTS);
  return launch_pdl(weights, (unsigned)a.BH * chunks, kThreads, 0, st, a, chunks);
}

template <int DH>
cudaError_t launch_d(const Plan& p, const AttendArgs& a, int grid, int cluster, cudaStream_t st) {
  if (p.bf16) {
    if (a.G <= 2) return launch_t<DH, Bf16Rows<DH, 2>>(p, a, grid, cluster, st);
    if (a.G <= 4) return launch_t<DH, Bf16Rows<DH, 4>>(p, a, grid, cluster, st);
    return launch_t<DH, Bf16Rows<DH, 8>>(p, a, grid, cluster, st);
  }
  if (a.G == 1) return launch_t<DH, F32Rows<DH, 1>>(p, a, grid, cluster, st);
  if (a.G == 2) return launch_t<DH, F32Rows<DH, 2>>(p, a, grid, cluster, st);
  if (a.G <= 4) return launch_t<DH, F32Rows<DH, 4>>(p, a, grid, cluster, st);
  return launch_t<DH, F32Rows<DH, 8>>(p, a, grid, cluster, st);
}

}  // namespace

cudaError_t launch_kv_attend(const Plan& p, const KvView& c, const void* q, int64_t qsb, int64_t qsh, float* out,
                             int64_t osb, int64_t osh, float* lse, float* w, int cap, float decay, void* ws,
                             cudaStream_t st) {
  const auto& cfg = p.cfg;
  const KvWorkspace L = kv_workspace(p, c.max_len);
  char* base = (char*)ws;
  AttendArgs a{};
  a.c = c;
  a.BH = cfg.batch * cfg.kv_heads;
  a.H = cfg.kv_heads;
  a.G = p.G;
  a.q = q;
  a.qsb = qsb;
  a.qsh = qsh;
  a.out = out;
  a.osb = osb;
  a.osh = osh;
  a.lse = lse;
  a.w = w;
  a.cap = cap;
  a.decay = decay;
  a.scale2 = kLog2e / sqrtf((float)cfg.d_h);
  a.part = (float*)(base + L.part);
  a.norm = (float2*)(base + L.norm);
  a.dots = (float*)(base + L.dots);
  const int unit = kSlotBytes / (cfg.d_h * p.esize);
  a.unit_log = unit == 64 ? 6 : unit == 32 ? 5 : 4;
  const int64_t most = a.BH * ceil_div64(c.max_len, unit);
  const int grid = (int)std::min<int64_t>(kKvMaxGrid, ceil_div64(most, kMinUnits));
  // short rows (see kv_attend_short_kernel)
  int cluster = 0;
  const int64_t units = ceil_div64(c.max_len, unit);
  for (int n = 1; n <= 8; n *= 2)
    if ((int64_t)a.BH * n <= short_ctas(n)) cluster = n;
  if (cluster && units > (int64_t)cluster * kShortUnits) cluster = 0;
  return cfg.d_h == 128 ? launch_d<128>(p, a, grid, cluster, st) : launch_d<64>(p, a, grid, cluster, st);
}

}  // namespace dkv
