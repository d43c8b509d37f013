// kv_attend.cu -- attention of one new token per sequence over plain K/V rows
// in pages, split over the rows and joined.
//
// For query head hq of pair bh = (sequence, kv-head), with x_r = log2(e) q .
// K_r / sqrt(d_h) over the pair's valid rows r:
//   m = max_r x_r,  l = sum_r 2^(x_r - m),  out = (sum_r 2^(x_r - m) V_r) / l,
//   lse = ln2 (m + log2 l),   and with weights   w_r <- decay w_r + sum_heads 2^(x_r - m) / l.
// A part of the rows gives (m, l, o = sum 2^(x_r - m) V_r); parts join by
// m = max m_i, l = sum 2^(m_i - m) l_i, o = sum 2^(m_i - m) o_i.
//
// Split: all pairs' rows, in units of 16, form one list that is cut into as
// many equal ranges as there are CTAs, so that lengths do not matter for the
// balance.  A CTA's range is a run of segments, each inside one pair; only
// its first and its last segment can be a part of a pair, so a CTA leaves two
// partial results at most.  A second kernel joins them and adds the weights,
// which need the joined (m, l) of each head.
#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "sm100.cuh"

namespace dkv {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kUnit = 16;       // rows per unit of the split (divides every page)
constexpr int kMinUnits = 8;    // a CTA gets at least these, or fewer CTAs work
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct AttendArgs {
  KvView c;
  int64_t BH;
  int H, G;
  const void* q;
  int64_t qsb, qsh;
  float* out;
  int64_t osb, osh;
  float* lse;     // [B][Hq] or null
  float* w;       // [BH][cap] or null
  int64_t cap;
  float decay, scale2;  // scale2 = log2(e) / sqrt(d_h)
  float* part;    // [CTA][2][kv_part_floats]: o[G][d_h], m[kMaxG], l[kMaxG]
  float* lse2;    // [BH][G]
  float* logits;  // [BH][max_len][G] or null
};

// The cut of the unit list into ranges.
struct Cut {
  int64_t W;  // units of all pairs
  int64_t g;  // ranges (<= grid)
  __device__ int64_t start(int64_t c) const { return c * W / g; }
  __device__ int64_t cta_of(int64_t u) const { return ((u + 1) * g - 1) / W; }
};

__device__ __forceinline__ int64_t units_of(int len) { return (len + kUnit - 1) / kUnit; }

// Total units, and the pair that holds the first unit of this CTA's range
// (its number and its first unit), by a block scan over the lengths.  Every
// thread returns the same values.  Lengths out of range are reported here.
__device__ Cut locate(const KvView& c, int64_t BH, int64_t& bh0, int64_t& s0) {
  __shared__ int64_t sh_warp[kWarps];
  __shared__ int64_t sh_bh, sh_s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t per = (BH + kThreads - 1) / kThreads;
  const int64_t b0 = min(BH, tid * per), b1 = min(BH, b0 + per);
  int64_t sum = 0;
  for (int64_t b = b0; b < b1; ++b) {
    const int n = c.lens[b];
    if (n < 0 || n > c.max_len) c.report((uint32_t)n);
    sum += units_of(c.len(b));
  }
  int64_t inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) sh_warp[warp] = inc;
  __syncthreads();
  int64_t before = 0, W = 0;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) {
    if (i < warp) before += sh_warp[i];
    W += sh_warp[i];
  }
  Cut cut{W, max((int64_t)1, min((int64_t)gridDim.x, (W + kMinUnits - 1) / kMinUnits))};
  const int64_t target = cut.start(blockIdx.x);
  int64_t s = before + inc - sum;
  if (blockIdx.x < cut.g && target >= s && target < s + sum) {
    int64_t b = b0;
    for (; b < b1; ++b) {
      const int64_t u = units_of(c.len(b));
      if (target < s + u) break;
      s += u;
    }
    sh_bh = b;
    sh_s = s;
  }
  __syncthreads();
  bh0 = sh_bh;
  s0 = sh_s;
  return cut;
}

// One warp's running softmax over its rows, as partial results: m, l and o
// per head, reduced over the block's warps in shared memory.
template <int DH>
struct Merge {
  float m[kWarps][kMaxG], l[kWarps][kMaxG];
  float o[kWarps][kMaxG][DH];
};

// Reduce the warps' parts of one segment and write them where they belong:
// out and lse where the segment is the whole pair, else the partial slot.
template <int DH>
__device__ __forceinline__ void finish_segment(const AttendArgs& a, const Merge<DH>& sm, int64_t bh, bool whole,
                                               int64_t cta, int slot) {
  const int64_t b = bh / a.H;
  const int h = (int)(bh % a.H);
  float* part = a.part + (cta * 2 + slot) * (int64_t)kv_part_floats(a.G, DH);
  for (int i = threadIdx.x; i < a.G * DH; i += kThreads) {
    const int g = i / DH, e = i % DH;
    float m = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) m = fmaxf(m, sm.m[w][g]);
    const float mu = m == -INFINITY ? 0.f : m;
    float l = 0.f, o = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float f = exp2f(sm.m[w][g] - mu);
      l = fmaf(sm.l[w][g], f, l);
      o = fmaf(sm.o[w][g][e], f, o);
    }
    if (whole) {
      a.out[b * a.osb + (int64_t)(h * a.G + g) * a.osh + e] = l == 0.f ? 0.f : o / l;
      if (e == 0) {
        const float L = m + log2f(l);  // -inf where every row was skipped
        a.lse2[bh * a.G + g] = L;
        if (a.lse) a.lse[bh * a.G + g] = kLn2 * L;
      }
    } else {
      part[i] = o;
      if (e == 0) {
        part[a.G * DH + g] = m;
        part[a.G * DH + kMaxG + g] = l;
      }
    }
  }
}

template <typename E, int DH>
__global__ void __launch_bounds__(kThreads) kv_attend_kernel(AttendArgs a) {
  constexpr int NV = DH / 32;
  __shared__ Merge<DH> sm;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t bh, s;
  const Cut cut = locate(a.c, a.BH, bh, s);
  if (cut.W == 0 || blockIdx.x >= cut.g) return;
  const int64_t u_end = cut.start(blockIdx.x + 1);
  int64_t u = cut.start(blockIdx.x);
  for (bool first = true; u < u_end; first = false) {
    int len = a.c.len(bh);
    while (len == 0) len = a.c.len(++bh);
    const int64_t ub = units_of(len);
    const int64_t ua = u - s, ue = min(u_end - s, ub);
    const int64_t b = bh / a.H;
    const int h = (int)(bh % a.H);
    float q[kMaxG][NV], acc[kMaxG][NV], m[kMaxG], l[kMaxG];
#pragma unroll
    for (int g = 0; g < kMaxG; ++g) {
      m[g] = -INFINITY;
      l[g] = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        acc[g][i] = 0.f;
        q[g][i] = g < a.G ? to_f(static_cast<const E*>(a.q)[b * a.qsb + (int64_t)(h * a.G + g) * a.qsh + lane * NV + i]) : 0.f;
      }
    }
    for (int64_t t = ua + warp; t < ue; t += kWarps) {
      for (int r = (int)t * kUnit; r < min(len, (int)t * kUnit + kUnit); ++r) {
        const int64_t row = a.c.row(bh, r);
        const E* kr = reinterpret_cast<const E*>(a.c.k) + row * DH + lane * NV;
        const E* vr = reinterpret_cast<const E*>(a.c.v) + row * DH + lane * NV;
        float kx[NV], vx[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          kx[i] = row < 0 ? 0.f : to_f(kr[i]);
          vx[i] = row < 0 ? 0.f : to_f(vr[i]);
        }
#pragma unroll
        for (int g = 0; g < kMaxG; ++g) {
          if (g >= a.G) break;
          float x = 0.f;
#pragma unroll
          for (int i = 0; i < NV; ++i) x = fmaf(q[g][i], kx[i], x);
          x = row < 0 ? -INFINITY : warp_sum(x) * a.scale2;
          if (a.logits && lane == 0) a.logits[(bh * a.c.max_len + r) * a.G + g] = x;
          const float mn = fmaxf(m[g], x), mu = mn == -INFINITY ? 0.f : mn;
          const float f = exp2f(m[g] - mu), p = exp2f(x - mu);
          m[g] = mn;
          l[g] = fmaf(l[g], f, p);
#pragma unroll
          for (int i = 0; i < NV; ++i) acc[g][i] = fmaf(acc[g][i], f, p * vx[i]);
        }
      }
    }
#pragma unroll
    for (int g = 0; g < kMaxG; ++g) {
      if (lane == 0) {
        sm.m[warp][g] = m[g];
        sm.l[warp][g] = l[g];
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) sm.o[warp][g][lane * NV + i] = acc[g][i];
    }
    __syncthreads();
    finish_segment<DH>(a, sm, bh, ua == 0 && ue == ub, blockIdx.x, first ? 0 : 1);
    __syncthreads();
    u = s + ue;
    s += ub;
    ++bh;
  }
}

// Join the partial results of the pairs that several CTAs hold, and add the
// weights.  CTA c takes the segments that CTA c of the first kernel took: of
// each, its share of the pair's outputs and the weights of its own rows.
template <int DH>
__global__ void __launch_bounds__(kThreads) kv_join_kernel(AttendArgs a) {
  __shared__ float sh_f[kKvMaxGrid * kMaxG];  // factor of each part and head
  __shared__ float sh_L[kMaxG], sh_l[kMaxG];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int64_t bh, s;
  const Cut cut = locate(a.c, a.BH, bh, s);
  // pairs without rows
  for (int64_t e = blockIdx.x; e < a.BH; e += gridDim.x) {
    if (a.c.len(e) != 0) continue;
    const int64_t b = e / a.H;
    const int h = (int)(e % a.H);
    for (int i = tid; i < a.G * DH; i += kThreads)
      a.out[b * a.osb + (int64_t)(h * a.G + i / DH) * a.osh + i % DH] = 0.f;
    if (a.lse && tid < a.G) a.lse[e * a.G + tid] = -INFINITY;
  }
  if (cut.W == 0 || blockIdx.x >= cut.g) return;
  const int64_t u_end = cut.start(blockIdx.x + 1);
  int64_t u = cut.start(blockIdx.x);
  while (u < u_end) {
    int len = a.c.len(bh);
    while (len == 0) len = a.c.len(++bh);
    const int64_t ub = units_of(len);
    const int64_t ua = u - s, ue = min(u_end - s, ub);
    const int64_t c0 = cut.cta_of(s), c1 = cut.cta_of(s + ub - 1);
    const int np = (int)(c1 - c0 + 1);
    const int stride = kv_part_floats(a.G, DH);
    // part i is CTA c0 + i's: its first segment, but for CTA c0 where that began in an earlier pair
    const int slot0 = cut.start(c0) == s ? 0 : 1;
    const float* part0 = a.part + (c0 * 2 + slot0) * (int64_t)stride;
    auto part = [&](int i) { return i == 0 ? part0 : a.part + (c0 + i) * 2 * (int64_t)stride; };
    if (np > 1) {
      if (warp < a.G) {
        for (int g = warp; g < a.G; g += kWarps) {
          float m = -INFINITY;
          for (int i = lane; i < np; i += 32) m = fmaxf(m, part(i)[a.G * DH + g]);
          m = warp_max(m);
          const float mu = m == -INFINITY ? 0.f : m;
          float l = 0.f;
          for (int i = lane; i < np; i += 32) {
            const float f = exp2f(part(i)[a.G * DH + g] - mu);
            sh_f[i * kMaxG + g] = f;
            l = fmaf(f, part(i)[a.G * DH + kMaxG + g], l);
          }
          l = warp_sum(l);
          if (lane == 0) {
            sh_l[g] = l;
            sh_L[g] = m + log2f(l);
          }
        }
      }
      __syncthreads();
      const int64_t b = bh / a.H;
      const int h = (int)(bh % a.H);
      const int j = (int)(blockIdx.x - c0), cols = a.G * DH / 4;
      const int q0 = (int)((int64_t)cols * j / np), q1 = (int)((int64_t)cols * (j + 1) / np);
      for (int q = q0 + warp; q < q1; q += kWarps) {
        const int g = q / (DH / 4);
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int i = lane; i < np; i += 32) {
          const float4 v = *reinterpret_cast<const float4*>(part(i) + q * 4);
          const float f = sh_f[i * kMaxG + g];
          o.x = fmaf(f, v.x, o.x);
          o.y = fmaf(f, v.y, o.y);
          o.z = fmaf(f, v.z, o.z);
          o.w = fmaf(f, v.w, o.w);
        }
        o.x = warp_sum(o.x);
        o.y = warp_sum(o.y);
        o.z = warp_sum(o.z);
        o.w = warp_sum(o.w);
        if (lane == 0) {
          const float l = sh_l[g];
          if (l == 0.f)
            o = make_float4(0.f, 0.f, 0.f, 0.f);
          else
            o = make_float4(o.x / l, o.y / l, o.z / l, o.w / l);
          *reinterpret_cast<float4*>(a.out + b * a.osb + (int64_t)(h * a.G + g) * a.osh + (q * 4) % DH) = o;
        }
      }
      if (a.lse && j == 0 && tid < a.G) a.lse[bh * a.G + tid] = kLn2 * sh_L[tid];
    } else if (a.w) {
      if (tid < a.G) sh_L[tid] = a.lse2[bh * a.G + tid];
      __syncthreads();
    }
    if (a.w) {
      const int r1 = min(len, (int)ue * kUnit);
      for (int r = (int)ua * kUnit + tid; r < r1; r += kThreads) {
        const float* x = a.logits + (bh * a.c.max_len + r) * a.G;
        float p = 0.f;
        for (int g = 0; g < a.G; ++g) p += sh_L[g] == -INFINITY ? 0.f : exp2f(x[g] - sh_L[g]);
        float* w = a.w + bh * a.cap + r;
        *w = fmaf(a.decay, *w, p);
      }
    }
    __syncthreads();
    u = s + ue;
    s += ub;
    ++bh;
  }
}

template <typename E, int DH>
cudaError_t launch_t(const Plan& p, const AttendArgs& a, int grid, cudaStream_t st) {
  {
    ProfScope ps(p, st, KID_KV_ATTEND);
    kv_attend_kernel<E, DH><<<grid, kThreads, 0, st>>>(a);
  }
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  ProfScope ps(p, st, KID_KV_JOIN);
  kv_join_kernel<DH><<<grid, kThreads, 0, st>>>(a);
  return cudaGetLastError();
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
  a.BH = (int64_t)cfg.batch * cfg.kv_heads;
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
  a.lse2 = (float*)(base + L.lse2);
  a.logits = w ? (float*)(base + L.logits) : nullptr;
  const int64_t most = a.BH * ceil_div64(c.max_len, kUnit);
  const int grid = (int)std::min<int64_t>(kKvMaxGrid, ceil_div64(most, kMinUnits));
  if (p.bf16)
    return cfg.d_h == 128 ? launch_t<__nv_bfloat16, 128>(p, a, grid, st) : launch_t<__nv_bfloat16, 64>(p, a, grid, st);
  return cfg.d_h == 128 ? launch_t<float, 128>(p, a, grid, st) : launch_t<float, 64>(p, a, grid, st);
}

}  // namespace dkv
