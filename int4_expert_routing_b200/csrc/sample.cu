// Sampling one token a row from the head's logits with temperature, top-k,
// top-p and min-p from given random numbers (flint_sample).
//
// No sort of the vocabulary: the kept set is "everything from a cut on" in
// the order (logit down, index up), so only the cut is searched.  A cluster
// of CTAs takes a row and holds it in shared memory, read from HBM once:
//   1. the largest logit M;
//   2. a histogram over d = (M - z) log2(e) / temperature in steps of 1/32:
//      each bin's count and mass.  The mass is summed in integers: within a
//      bin 2^-d is 2^(-bin/32) (1 - e) with e < 0.0215, and the sum of e in
//      units of 2^-22 fits 32 bits for the 2^15 elements of a CTA and does not depend on
//      the order of the atomics;
//   3. the bins' running count and mass name the bin a cut falls in; its
//      elements (a few of them) are gathered into one CTA and put in order.
//      A bin with too many is first halved by key, and equal logits are cut
//      by index;
//   4. the kept mass in index order (fp64, fixed order), and the token whose
//      running mass passes u times the total.
// Every sum has a fixed order or is an integer, so a row's result does not
// vary between runs, nor with the other rows.
#include <cooperative_groups.h>

#include "common.cuh"
#include "internal.h"

namespace cg = cooperative_groups;

namespace flint {

constexpr int kSmThreads = 512;
constexpr int kSmWarps = kSmThreads / 32;
constexpr int kSmBins = 1024;       // steps of 1/32 in log2 units: d < 32
constexpr float kSmSteps = 32.f;
constexpr int kSmList = 512;        // elements put in order at once
constexpr int kSmMaxCluster = 8;
constexpr float kEpsUnit = 4194304.f;  // 2^22

struct SampleShared {
  uint32_t cnt[kSmBins], eps[kSmBins];  // this CTA's bins
  uint32_t tcnt[kSmBins];               // the cluster's
  double tmass[kSmBins];
  unsigned long long list[kSmList], sorted[kSmList];
  // one exchange between the CTAs uses one of two sets of slots, in turn
  struct {
    unsigned long long a;
    double b;
  } slot[2][kSmMaxCluster];
  unsigned long long red_a[kSmWarps];
  double red_b[kSmWarps];
  double wsum[kSmWarps];
  double lmass[kSmList];
  unsigned long long res_key;
  double res_mass;
  uint32_t list_n;
  int found;
};

FLINT_DEV float ex2(float x) {
  float y;
  asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

struct Sum2 {
  unsigned long long a;
  double b;
};

// A row's view in one CTA: z[0 .. 4 n4) with index0 the row index of z[0]
// (it may start up to 3 elements early; those hold -inf).
struct RowPart {
  const float4 *z;
  int n4;
  int index0;
};

template <typename F>
FLINT_DEV void for_elements(const RowPart &r, F f) {
  for (int i = threadIdx.x; i < r.n4; i += kSmThreads) {
    const float4 v = r.z[i];
    f(v.x, 4 * i);
    f(v.y, 4 * i + 1);
    f(v.z, 4 * i + 2);
    f(v.w, 4 * i + 3);
  }
}

// (z, index) as one number: larger = earlier in the order.  -0 counts as +0.
FLINT_DEV uint32_t zkey(float z) { return float_key(z + 0.f); }
FLINT_DEV float key_z(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? k & 0x7fffffffu : ~k);
}

struct Dist {
  float M, c;
  // log2 of p(max) / p(z), >= 0; +inf where p = 0 (NaN, -inf)
  FLINT_DEV float operator()(float z) const {
    const float d = (M - z) * c;
    return z == M ? 0.f : (d >= 0.f ? d : __int_as_float(0x7f800000));
  }
  FLINT_DEV int bin(float z) const {
    const float d = (*this)(z);
    return d < (float)kSmBins / kSmSteps ? (int)(d * kSmSteps)
                                         : (z > -__int_as_float(0x7f800000) ? kSmBins : -1);
  }
};

struct Team {
  SampleShared *s;
  int rank, size, parity = 0;
  FLINT_DEV void sync() { cg::this_cluster().sync(); }
  template <typename T>
  FLINT_DEV T *of(T *p, int r) {
    return cg::this_cluster().map_shared_rank(p, r);
  }
  // every thread's (a, b) over the block: sums (kOp 0), or the largest a and b (kOp 1)
  template <int kOp>
  FLINT_DEV Sum2 block(unsigned long long a, double b) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      const unsigned long long a2 = __shfl_xor_sync(0xffffffffu, a, o);
      const double b2 = __shfl_xor_sync(0xffffffffu, b, o);
      a = kOp ? (a > a2 ? a : a2) : a + a2;
      b = kOp ? fmax(b, b2) : b + b2;
    }
    __syncthreads();
    if (lane == 0) s->red_a[w] = a, s->red_b[w] = b;
    __syncthreads();
    a = s->red_a[0], b = s->red_b[0];
    for (int i = 1; i < kSmWarps; ++i) {
      a = kOp ? (a > s->red_a[i] ? a : s->red_a[i]) : a + s->red_a[i];
      b = kOp ? fmax(b, s->red_b[i]) : b + s->red_b[i];
    }
    return {a, b};
  }
  // the CTAs' values to every CTA's slots; returns the set they are in
  FLINT_DEV int exchange(Sum2 v) {
    const int p = parity;
    parity ^= 1;
    if ((int)threadIdx.x < size) {
      auto *dst = of(&s->slot[p][rank], threadIdx.x);
      dst->a = v.a, dst->b = v.b;
    }
    sync();
    return p;
  }
  template <int kOp>
  FLINT_DEV Sum2 all(unsigned long long a, double b) {
    const int p = exchange(block<kOp>(a, b));
    a = s->slot[p][0].a, b = s->slot[p][0].b;
    for (int r = 1; r < size; ++r) {
      const unsigned long long a2 = s->slot[p][r].a;
      const double b2 = s->slot[p][r].b;
      a = kOp ? (a > a2 ? a : a2) : a + a2;
      b = kOp ? fmax(b, b2) : b + b2;
    }
    return {a, b};
  }
};

// What a cut is looked for: with `count`, the element number `want` (from 1)
// of the order; otherwise the first whose running mass reaches `mass`.
struct Goal {
  bool count;
  unsigned long long want;
  double mass;
};
struct Cut {
  unsigned long long key;  // the last kept element
  double mass;             // mass down to it
};

// The cut inside bin `b`, which holds n elements behind `above` earlier ones
// with mass `mass_above`.  Every thread of the cluster takes part and gets
// the same answer.
FLINT_DEV Cut resolve(Team &t, const RowPart &r, const Dist &dist, int b, unsigned long long n,
                      unsigned long long above, double mass_above, const Goal &goal) {
  SampleShared &s = *t.s;
  uint32_t klo = 0, khi = 0xffffffffu;
  if (n > kSmList) {
    uint32_t lo = 0xffffffffu, hi = 0;
    for_elements(r, [&](float z, int) {
      if (dist.bin(z) == b) {
        const uint32_t k = zkey(z);
        lo = min(lo, k), hi = max(hi, k);
      }
    });
    // the largest of (hi, ~lo), both exact in a double
    const Sum2 m = t.all<1>(hi, (double)(uint32_t)~lo);
    khi = (uint32_t)m.a, klo = ~(uint32_t)m.b;
    while (n > kSmList && klo < khi) {
      const uint32_t mid = klo + (khi - klo) / 2;  // the upper half is (mid, khi]
      unsigned long long cu = 0;
      double mu = 0;
      for_elements(r, [&](float z, int) {
        const uint32_t k = zkey(z);
        if (k > mid && k <= khi && dist.bin(z) == b) {
          ++cu;
          mu += (double)ex2(-dist(z));
        }
      });
      const Sum2 u = t.all<0>(cu, mu);
      if (u.a && (goal.count ? above + u.a >= goal.want : mass_above + u.b >= goal.mass)) {
        klo = mid + 1;
        n = u.a;
      } else {
        khi = mid;
        n -= u.a, above += u.a, mass_above += u.b;
      }
    }
  }
  if (n > kSmList) {
    // one logit, more than kSmList times: cut by index
    const float z0 = key_z(klo);
    const double p = (double)ex2(-dist(z0));
    double left = goal.count ? (double)(goal.want - above)
                             : (p > 0 ? ceil((goal.mass - mass_above) / p) : (double)n);
    left = fmin(fmax(left, 1.0), (double)n);
    const unsigned long long keep = (unsigned long long)left;
    unsigned long long mine = 0;
    for_elements(r, [&](float z, int) { mine += z == z0; });
    const Sum2 tot = t.block<0>(mine, 0);
    const int q = t.exchange(tot);
    unsigned long long before = 0;
    for (int i = 0; i < t.rank; ++i) before += s.slot[q][i].a;
    if (before < keep && before + tot.a >= keep) {
      // this CTA has it: walk its elements in order, kSmThreads at a time
      const float *z = reinterpret_cast<const float *>(r.z);
      for (int base = 0; base < 4 * r.n4; base += kSmThreads) {
        const int i = base + threadIdx.x;
        const bool hit = i < 4 * r.n4 && z[i] == z0;
        const int c = __syncthreads_count(hit);
        if (before + c >= keep) {
          const uint32_t m = __ballot_sync(0xffffffffu, hit);
          const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
          if (lane == 0) s.red_a[w] = __popc(m);
          __syncthreads();
          unsigned long long at = before;
          for (int k = 0; k < w; ++k) at += s.red_a[k];
          if (hit && at + __popc(m & ((2u << lane) - 1u)) == keep) {
            const unsigned long long key =
                ((unsigned long long)klo << 32) | (0xffffffffu - (uint32_t)(r.index0 + i));
            for (int k = 0; k < t.size; ++k) *t.of(&s.res_key, k) = key;
          }
          break;
        }
        before += c;
      }
    }
    t.sync();
    const Cut cut{s.res_key, mass_above + (double)keep * p};
    t.sync();
    return cut;
  }
  // gather into CTA 0 and order there
  if (t.rank == 0 && threadIdx.x == 0) s.list_n = 0;
  t.sync();
  uint32_t *ln = t.of(&s.list_n, 0);
  unsigned long long *list = t.of(&s.list[0], 0);
  for_elements(r, [&](float z, int i) {
    const uint32_t k = zkey(z);
    if (k >= klo && k <= khi && dist.bin(z) == b) {
      const uint32_t at = atomicAdd(ln, 1u);
      if (at < (uint32_t)kSmList)
        list[at] = ((unsigned long long)k << 32) | (0xffffffffu - (uint32_t)(r.index0 + i));
    }
  });
  t.sync();
  if (t.rank == 0) {
    const int m = min((int)s.list_n, kSmList);
    for (int i = threadIdx.x; i < m; i += kSmThreads) {
      const unsigned long long mine = s.list[i];
      int before = 0;
      for (int j = 0; j < m; ++j) before += s.list[j] > mine;
      s.sorted[before] = mine;
      s.lmass[before] = (double)ex2(-dist(key_z((uint32_t)(mine >> 32))));
    }
    __syncthreads();
    if (threadIdx.x == 0) {
      double run = mass_above;
      int i = 0;
      for (; i < m; ++i) {
        run += s.lmass[i];
        if (goal.count ? above + i + 1 >= goal.want : run >= goal.mass) break;
      }
      if (i == m) --i;
      const unsigned long long key = m ? s.sorted[i] : 0ull;
      for (int k = 0; k < t.size; ++k) *t.of(&s.res_key, k) = key, *t.of(&s.res_mass, k) = run;
    }
  }
  t.sync();
  const Cut cut{s.res_key, s.res_mass};
  t.sync();
  return cut;
}

__global__ void __launch_bounds__(kSmThreads) k_sample(const __grid_constant__ SampleArgs a) {
  extern __shared__ __align__(16) unsigned char smraw[];
  SampleShared &s = *reinterpret_cast<SampleShared *>(smraw);
  float *zs = reinterpret_cast<float *>(smraw + (sizeof(SampleShared) + 15) / 16 * 16);
  cg::cluster_group cl = cg::this_cluster();
  Team t;
  t.s = &s, t.rank = (int)cl.block_rank(), t.size = (int)cl.num_blocks();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int row = blockIdx.x / t.size;
  const float kInf = __int_as_float(0x7f800000);

  // this CTA's part of the row: [lo, hi), in whole 16-byte pieces of memory
  const int part = ((a.V + t.size - 1) / t.size + 3) & ~3;
  const int lo = min(a.V, t.rank * part), hi = min(a.V, lo + part);
  const int64_t g0 = (int64_t)row * a.stride;
  const int skip = (int)((g0 + lo) & 3);
  RowPart r{reinterpret_cast<const float4 *>(zs), (skip + hi - lo + 3) / 4, lo - skip};

  pdl_wait();
  pdl_trigger();
  float top = -kInf;
  const float4 *src = reinterpret_cast<const float4 *>(a.logits + (g0 + lo - skip));
#pragma unroll 4
  for (int i = tid; i < r.n4; i += kSmThreads) {
    float4 v;
    const int e = r.index0 + 4 * i;
    if (e >= lo && e + 4 <= hi) {
      v = __ldcs(src + i);
    } else {
      const float *z = a.logits + g0 + e;
      v.x = e >= lo && e < hi ? z[0] : -kInf;
      v.y = e + 1 >= lo && e + 1 < hi ? z[1] : -kInf;
      v.z = e + 2 >= lo && e + 2 < hi ? z[2] : -kInf;
      v.w = e + 3 >= lo && e + 3 < hi ? z[3] : -kInf;
    }
    reinterpret_cast<float4 *>(zs)[i] = v;
    top = fmaxf(top, fmaxf(fmaxf(v.x, v.y), fmaxf(v.z, v.w)));  // NaN drops out
  }
  for (int i = tid; i < kSmBins; i += kSmThreads) s.cnt[i] = 0, s.eps[i] = 0;
  const float T0 = a.temperature ? a.temperature[row] : 1.f;
  const float T = T0 > 3.4e38f ? 3.4e38f : T0;
  const int k = a.top_k ? a.top_k[row] : 0;
  const float top_p = a.top_p ? a.top_p[row] : 1.f;
  const float min_p = a.min_p ? a.min_p[row] : 0.f;

  const float M = key_z((uint32_t)t.all<1>(zkey(top), 0).a);
  if (M == -kInf) {
    if (t.rank == 0 && tid == 0) {
      a.token[row] = -1;
      if (a.logprob) a.logprob[row] = -kInf;
    }
    t.sync();
    return;
  }
  if (!(T > 0.f) || min_p > 1.f || k == 1 || top_p <= 0.f) {
    // the first of the order: the lowest index of M
    uint32_t best = 0xffffffffu;
    for_elements(r, [&](float z, int i) {
      if (z == M) best = min(best, (uint32_t)(r.index0 + i));
    });
    const Sum2 m = t.all<1>((unsigned long long)(uint32_t)~best, 0);
    if (t.rank == 0 && tid == 0) {
      a.token[row] = (int)~(uint32_t)m.a;
      if (a.logprob) a.logprob[row] = 0.f;
    }
    t.sync();
    return;
  }

  const Dist dist{M, __fdiv_rn(1.4426950408889634f, T)};
  const bool use_k = k > 0 && k < a.V, use_p = top_p < 1.f;
  unsigned long long cut = 0;  // kept: (z, index) at or before this in the order
  if (use_k || use_p) {
    unsigned long long far_n = 0;
    double far_mass = 0;
    for_elements(r, [&](float z, int) {
      const float d = dist(z);
      if (d < (float)kSmBins / kSmSteps) {
        const int b = (int)(d * kSmSteps);
        const float e = 1.f - ex2((float)b * (1.f / kSmSteps) - d);
        atomicAdd(&s.cnt[b], 1u);
        atomicAdd(&s.eps[b], (uint32_t)(fmaxf(e, 0.f) * kEpsUnit + 0.5f));
      } else if (z > -kInf) {
        ++far_n;
        far_mass += (double)ex2(-d);
      }
    });
    const Sum2 far = t.all<0>(far_n, far_mass);  // also: every CTA's bins are complete
    {
      const int per = kSmBins / t.size;
      for (int i = tid; i < per; i += kSmThreads) {
        const int b = t.rank * per + i;
        unsigned long long c = 0, e = 0;
        for (int q = 0; q < t.size; ++q) c += t.of(s.cnt, q)[b], e += t.of(s.eps, q)[b];
        const double mass = exp2(-(double)b / kSmSteps) * ((double)c - (double)e / kEpsUnit);
        for (int q = 0; q < t.size; ++q) t.of(s.tcnt, q)[b] = (uint32_t)c, t.of(s.tmass, q)[b] = mass;
      }
      t.sync();
    }
    // running count and mass before this thread's two bins (the same in every CTA)
    unsigned long long c0 = s.tcnt[2 * tid], c1 = s.tcnt[2 * tid + 1], ex_c = c0 + c1;
    double m0 = s.tmass[2 * tid], m1 = s.tmass[2 * tid + 1], ex_m = m0 + m1;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long c2 = __shfl_up_sync(0xffffffffu, ex_c, o);
      const double m2 = __shfl_up_sync(0xffffffffu, ex_m, o);
      if (lane >= o) ex_c += c2, ex_m += m2;
    }
    __syncthreads();
    if (lane == 31) s.red_a[warp] = ex_c, s.red_b[warp] = ex_m;
    __syncthreads();
    unsigned long long all_c = 0, pre_c = 0;
    double all_m = 0, pre_m = 0;
    for (int w = 0; w < kSmWarps; ++w) {
      if (w == warp) pre_c = all_c, pre_m = all_m;
      all_c += s.red_a[w], all_m += s.red_b[w];
    }
    ex_c = pre_c + ex_c - c0 - c1;
    ex_m = pre_m + ex_m - (m0 + m1);

    // the bin a goal falls in, and the cut in it
    auto search = [&](const Goal &g) {
      __syncthreads();
      if (tid == 0) s.found = kSmBins;
      __syncthreads();
      const bool in0 = c0 && (g.count ? ex_c + c0 >= g.want : ex_m + m0 >= g.mass);
      const bool in1 = c1 && (g.count ? ex_c + c0 + c1 >= g.want : ex_m + m0 + m1 >= g.mass);
      if (in0 || in1) atomicMin(&s.found, in0 ? 2 * tid : 2 * tid + 1);
      __syncthreads();
      const int b = s.found;
      if (b < kSmBins) {
        if (b / 2 == tid) {
          s.red_a[0] = b & 1 ? c1 : c0;
          s.red_a[1] = b & 1 ? ex_c + c0 : ex_c;
          s.red_b[0] = b & 1 ? ex_m + m0 : ex_m;
        }
        __syncthreads();
        const unsigned long long n = s.red_a[0], above = s.red_a[1];
        const double mass = s.red_b[0];
        __syncthreads();
        return resolve(t, r, dist, b, n, above, mass, g);
      }
      if (!far.a) return Cut{0ull, all_m};  // nothing behind the bins: no cut
      return resolve(t, r, dist, kSmBins, far.a, all_c, all_m, g);
    };
    double mass = all_m + far.b;
    if (use_k && (unsigned long long)k < all_c + far.a) {
      const Cut c = search(Goal{true, (unsigned long long)k, 0.0});
      cut = c.key;
      mass = c.mass;
    }
    if (use_p) {
      const Cut c = search(Goal{false, 0, (double)top_p * mass});
      if (c.key > cut) cut = c.key;
    }
  }
  if (min_p > 0.f) {
    // p >= min_p: z at or above M + T ln(min_p)
    const float zmin = __double2float_ru((double)M + (double)T * log((double)min_p));
    const unsigned long long c = (unsigned long long)zkey(fminf(zmin, M)) << 32;
    if (c > cut) cut = c;
  }

  // kept mass: a warp's elements are a contiguous piece of the CTA's
  const float zc = cut ? key_z((uint32_t)(cut >> 32)) : -kInf;
  const int ic = cut ? (int)(0xffffffffu - (uint32_t)cut) : 0x7fffffff;
  auto p_of = [&](float z, int i) {
    // index r.index0 + i <= ic among equals; -1 - ic wraps to "all" for a bare key
    const bool kept = z > zc || (z == zc && (uint32_t)(r.index0 + i) <= (uint32_t)ic);
    return kept ? ex2(-dist(z)) : 0.f;
  };
  const int per4 = (r.n4 + kSmWarps - 1) / kSmWarps;
  const int w0 = min(r.n4, warp * per4), w1 = min(r.n4, w0 + per4);
  double sum = 0;
  for (int i = w0 + lane; i < w1; i += 32) {
    const float4 v = r.z[i];
    sum += ((double)p_of(v.x, 4 * i) + p_of(v.y, 4 * i + 1)) +
           ((double)p_of(v.z, 4 * i + 2) + p_of(v.w, 4 * i + 3));
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  __syncthreads();
  if (lane == 0) s.wsum[warp] = sum;
  __syncthreads();
  double mine = 0;
  for (int w = 0; w < kSmWarps; ++w) mine += s.wsum[w];
  const int q = t.exchange({0, mine});
  double total = 0, u = a.u[row];
  for (int i = 0; i < t.size; ++i) total += s.slot[q][i].b;
  u = u > 0 ? fmin(u, 1.0) : 0.0;
  const double goal = u * total;
  // the CTA, then the warp, whose running mass passes the goal; the last one
  // with any mass if none does (u = 1, or the last bit of a sum)
  int cta = -1;
  double run = 0, before = 0;
  for (int i = 0; i < t.size; ++i) {
    const double x = s.slot[q][i].b;
    if (x > 0) {
      cta = i, before = run;
      if (run + x > goal) break;
    }
    run += x;
  }
  if (cta == t.rank) {
    int w = 0;
    double base = before;
    run = before;
    for (int i = 0; i < kSmWarps; ++i) {
      if (s.wsum[i] > 0) {
        w = i, base = run;
        if (run + s.wsum[i] > goal) break;
      }
      run += s.wsum[i];
    }
    if (warp == w) {
      int last = -1, hit = -1;  // row index
      for (int i0 = w0; i0 < w1 && hit < 0; i0 += 32) {
        const int i = i0 + lane;
        float p[4] = {0.f, 0.f, 0.f, 0.f};
        if (i < w1) {
          const float4 v = r.z[i];
          p[0] = p_of(v.x, 4 * i), p[1] = p_of(v.y, 4 * i + 1);
          p[2] = p_of(v.z, 4 * i + 2), p[3] = p_of(v.w, 4 * i + 3);
        }
        const double own = ((double)p[0] + p[1]) + ((double)p[2] + p[3]);
        double inc = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const double x = __shfl_up_sync(0xffffffffu, inc, o);
          if (lane >= o) inc += x;
        }
        double at = base + (inc - own);
        int mine_hit = -1, mine_last = -1;
        for (int j = 0; j < 4; ++j) {
          at += p[j];
          if (p[j] > 0.f) {
            mine_last = r.index0 + 4 * i + j;
            if (mine_hit < 0 && at > goal) mine_hit = mine_last;
          }
        }
        const uint32_t hits = __ballot_sync(0xffffffffu, mine_hit >= 0);
        const uint32_t lasts = __ballot_sync(0xffffffffu, mine_last >= 0);
        if (hits) hit = __shfl_sync(0xffffffffu, mine_hit, __ffs(hits) - 1);
        if (lasts) last = __shfl_sync(0xffffffffu, mine_last, 31 - __clz(lasts));
        base += __shfl_sync(0xffffffffu, inc, 31);
      }
      if (hit < 0) hit = last;
      if (lane == 0) {
        a.token[row] = hit;
        if (a.logprob) {
          const float z = hit >= 0 ? zs[hit - r.index0] : M;
          const double y = z == M ? 0.0 : ((double)z - (double)M) / (double)T;
          a.logprob[row] = (float)(y - log(total));
        }
      }
    }
  }
  t.sync();  // no CTA leaves while another may still read its memory
}

cudaError_t launch_sample(const SampleArgs &a, cudaStream_t st) {
  int size = 1;
  while (size < kSmMaxCluster && a.V > 2048 * size) size *= 2;
  const int part = ((a.V + size - 1) / size + 3) & ~3;
  const size_t smem = (sizeof(SampleShared) + 15) / 16 * 16 + (size_t)(part + 4) * 4;
  note_step("sample attribute");
  cudaError_t e = cudaFuncSetAttribute(k_sample, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       200 * 1024);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.B * size);
  cfg.blockDim = dim3(kSmThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = size;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  note_step("sample launch");
  return cudaLaunchKernelEx(&cfg, k_sample, a);
}

}  // namespace flint
