// sampling_filter.cu -- token sampling with temperature, top-k, top-p and
// min-p from a given uniform per row (orthrus_vocab_sample_filtered).
//
// Mathematics.  With M the row's maximum, w_i = exp((x_i - M) / T).  All three
// filters keep a prefix of the order (x descending, index ascending): the
// first k; the shortest prefix whose mass reaches top_p of the first k's; the
// elements with w_i >= min_p.  So the kept set is {x > x_cut, or x == x_cut and
// i <= i_cut}, and no sort of the row is needed: a histogram over M - x finds
// the bin a cut falls into, and only that bin is looked at closely.  The draw
// is the first kept index whose cumulated mass, in vocabulary order, exceeds
// u times the kept mass.
//
// Sums of weights decide which token is drawn, so they are exact: w_i in FP64
// rounded to a fixed-point integer (2^-44 at a 152k vocabulary), summed in 64
// bits.  Neither the order of atomics nor the split of the row changes a
// result.
//
// One thread-block cluster owns a row; its CTAs keep their part of the row in
// shared memory, so the logits are read from HBM once however many passes the
// filters take (a vocabulary too large for that is read again, from L2).  What
// a pass costs is instructions, not bytes -- at HBM's pace an SM has about 20 a
// logit -- so each way through the filters makes as few as it can:
//   small top-k   the k-th largest of the maxima of groups of eight threads
//                 (taken while loading) is a lower bound of the k-th largest
//                 logit; the few logits at or above it go to a list in the
//                 first CTA, which orders them by counting and finishes the row
//   top-p         a histogram of counts over M - x, whose masses are guessed from
//                 the bins' middles, names the bin of the cut to within one;
//                 the pass that sums the row exactly also sums around that bin,
//                 and only the bin's elements are put in order
//   otherwise     (min-p alone or nothing) the one summing pass
// and where a shortcut does not decide -- many equal logits, a large k -- cuts
// are refined bin by bin to an exact element.  The sums are kept per warp, in
// vocabulary order, so that the draw is found without another pass.
#include <cooperative_groups.h>
#include <math.h>

#include "common.cuh"

namespace cg = cooperative_groups;

namespace orthrus {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kList = kThreads;   // one entry a thread
constexpr int kMaxCluster = 8;
constexpr int kGroups = 64;       // maxima a CTA contributes to top-k's bound
constexpr int kResidentBytes = 160 * 1024;  // row part a CTA may hold beside its tables
// Values more than 44 T below the maximum (weight below 8e-20, 0 in fixed
// point at every vocabulary size above 2^10) take no part.
constexpr float kDropT = 44.f;

typedef unsigned long long u64;

struct FilterParams {
  const void* logits;
  int64_t stride;
  const float *u, *temperature, *top_p, *min_p;
  const int32_t* top_k;
  int32_t* idx;
  float* logprob;
  int32_t* err;
  int rows, vocab, chunk, shift;  // weights in units of 2^-shift
  int vec;                        // rows may be read in 16-byte vectors
};

// Monotone map of a float to an integer; equal floats (both zeros) map alike.
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float float_of(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

struct Cut {  // what find() reports: the bin a cut falls into
  int bin;
  int cnt_in;
  u64 cnt0, mass0, mass_in;
};

struct Entry {
  u64 key;  // (~key_of(x) << 32) | index: ascending = descending value, then index
  u64 w;
};

// Sums over one warp's (or CTA's) part of the row.
struct Sums {
  u64 all;      // every weight
  u64 above;    // bins before the window
  u64 in[3];    // the window's three bins
  u64 minp;     // weights that pass min-p
};
constexpr int kSums = sizeof(Sums) / 8;

struct Shared {
  u64 mass[kBins];
  Entry list[kList];
  uint32_t cnt[kBins];
  float gmax[kMaxCluster * kGroups], gmin[kMaxCluster * kGroups];
  Sums warp_sum[kWarps], cta_sum[kMaxCluster];
  uint32_t kmin[kMaxCluster], kmax[kMaxCluster];
  u64 tot_c[kMaxCluster], tot_m[kMaxCluster];
  u64 scan_a[kWarps], scan_b[kWarps];
  u64 part[kMaxCluster];
  double tab[8];  // 2^(i/8)
  uint32_t redu[2 * kWarps];
  Cut cut;
  uint32_t cut_key;
  int cut_idx;
  u64 list_mass;
  int list_n;
  float tau;
  u64 total;
};

template <typename T>
__device__ __forceinline__ float widen(T v) {
  const float x = to_f32(v);
  return x != x ? -INFINITY : x;  // NaN never takes part
}

// Inclusive scan of (a, b) over the CTA; returns exclusive values in a0, b0.
__device__ __forceinline__ void block_scan(Shared& s, u64 a, u64 b, u64& a0, u64& b0, u64& at,
                                           u64& bt) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  u64 ia = a, ib = b;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const u64 ua = __shfl_up_sync(0xffffffffu, ia, o), ub = __shfl_up_sync(0xffffffffu, ib, o);
    if (lane >= o) { ia += ua; ib += ub; }
  }
  __syncthreads();
  if (lane == 31) { s.scan_a[warp] = ia; s.scan_b[warp] = ib; }
  __syncthreads();
  a0 = ia - a; b0 = ib - b; at = 0; bt = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) { a0 += s.scan_a[w]; b0 += s.scan_b[w]; }
    at += s.scan_a[w];
    bt += s.scan_b[w];
  }
}

template <typename T, bool kResident>
__global__ void __launch_bounds__(kThreads, kResident ? 2 : 1)
filter_kernel(const FilterParams p) {
  extern __shared__ __align__(16) uint8_t dyn[];
  Shared& s = *reinterpret_cast<Shared*>(dyn);
  T* vals = reinterpret_cast<T*>(dyn + (sizeof(Shared) + 15) / 16 * 16);
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int row = blockIdx.x / C;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const unsigned full = 0xffffffffu;
  const int lo = min(p.vocab, rank * p.chunk), hi = min(p.vocab, lo + p.chunk), nv = hi - lo;
  const T* src = static_cast<const T*>(p.logits) + row * p.stride + lo;
  Shared* peer0 = cluster.map_shared_rank(&s, 0);
  constexpr int kV = kResident ? 16 / sizeof(T) : 1;  // elements read at a time
  // f(x, i) for the elements [a, b) of this part (a a multiple of kV), kV at a
  // time from first * kV on in steps of step * kV
  auto sweep = [&](int a, int b, int first, int step, auto f) {
    for (int i = a + first * kV; i < b; i += step * kV) {
      if constexpr (kResident) {
        const uint4 v = *reinterpret_cast<const uint4*>(vals + i);
        const T* e = reinterpret_cast<const T*>(&v);
#pragma unroll
        for (int j = 0; j < kV; ++j)
          if (i + j < b) f(widen(e[j]), i + j);
      } else {
        f(widen(src[i]), i);
      }
    }
  };
  auto each = [&](auto f) { sweep(0, nv, tid, kThreads, f); };

  // ---- the row's parameters
  float T_ = p.temperature ? p.temperature[row] : 1.f;
  int k = p.top_k ? p.top_k[row] : 0;
  float top_p = p.top_p ? p.top_p[row] : 1.f;
  float min_p = p.min_p ? p.min_p[row] : 0.f;
  const float u = fminf(fmaxf(p.u[row], 0.f), 1.f);
  const bool bad = !(T_ >= 0.f) || T_ == INFINITY;
  if (T_ == 0.f || top_p <= 0.f) k = 1;  // the largest, lowest index
  if (T_ == 0.f) T_ = 1.f;
  if (k <= 0 || k >= p.vocab) k = 0;
  const bool use_p = top_p < 1.f && k != 1;
  min_p = min_p > 0.f ? fminf(min_p, 1.f) : 0.f;

  // ---- read this part of the row; maxima and minima of groups of eight threads
  float mx = -INFINITY, mn = INFINITY;
  if (kResident && p.vec) {
#pragma unroll 4
    for (int i = tid * kV; i < nv; i += kThreads * kV) {
      if (i + kV <= nv) {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(src + i));
        *reinterpret_cast<uint4*>(vals + i) = v;
        const T* e = reinterpret_cast<const T*>(&v);
#pragma unroll
        for (int j = 0; j < kV; ++j) {
          const float x = widen(e[j]);
          mx = fmaxf(mx, x);
          mn = fminf(mn, x);
        }
      } else {
        for (int j = i; j < nv; ++j) {
          vals[j] = src[j];
          mx = fmaxf(mx, widen(src[j]));
          mn = fminf(mn, widen(src[j]));
        }
      }
    }
  } else {
    for (int i = tid; i < nv; i += kThreads) {
      const T v = src[i];
      if (kResident) vals[i] = v;
      mx = fmaxf(mx, widen(v));
      mn = fminf(mn, widen(v));
    }
  }
#pragma unroll
  for (int o = 4; o; o >>= 1) {
    mx = fmaxf(mx, __shfl_xor_sync(full, mx, o));
    mn = fminf(mn, __shfl_xor_sync(full, mn, o));
  }
  if ((tid & 7) < C) {  // lane i of the group tells CTA i
    Shared* q = cluster.map_shared_rank(&s, tid & 7);
    q->gmax[rank * kGroups + (tid >> 3)] = mx;
    q->gmin[rank * kGroups + (tid >> 3)] = mn;
  }
  if (tid < 8) s.tab[tid] = exp2((double)tid * 0.125);
  for (int b = tid; b < kBins; b += kThreads) s.cnt[b] = 0;
  if (tid == 0) s.list_n = 0;
  cluster.sync();
  const int groups = C * kGroups;  // a multiple of 64
  for (int i = lane; i < groups; i += 32) {
    mx = fmaxf(mx, s.gmax[i]);
    mn = fminf(mn, s.gmin[i]);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    mx = fmaxf(mx, __shfl_xor_sync(full, mx, o));
    mn = fminf(mn, __shfl_xor_sync(full, mn, o));
  }
  if (bad || mx == -INFINITY) {  // the same answer in every CTA of the cluster
    if (rank == 0 && tid == 0) {
      if (bad) {
        set_err(p.err, ORTHRUS_EINVAL);
      } else {
        p.idx[row] = 0;
        if (p.logprob) p.logprob[row] = __int_as_float(0x7fffffff);
      }
    }
    return;
  }

  const double unit = (double)(1ull << p.shift);
  auto diff = [&](float x) { return x == mx ? 0.f : mx - x; };
  const float reach = kDropT * T_;
  auto takes_part = [&](float x) { return x > -INFINITY && diff(x) <= reach; };
  // e^((x - M) / T) = 2^(n / 8) e^r with |r| <= ln 2 / 16: the eighth root of
  // two from a table, the rest of the power of two through the exponent, e^r by
  // its Taylor series to r^7 (next term 3e-16).  Only for values that take part.
  const double inv_t = 1.0 / (double)T_, to8 = inv_t * (8 * 1.4426950408889634074);
  auto weight = [&](float x) {
    const double y = x == mx ? 0.0 : ((double)x - (double)mx) * to8;
    const double big = 6755399441055744.0;  // 1.5 * 2^52: rounds to an integer
    const double shifted = y + big;
    const int n = __double2loint(shifted);
    const double r = (y - (shifted - big)) * (0.69314718055994530942 / 8);
    double e = fma(r, 1.0 / 5040, 1.0 / 720);
    e = fma(r, e, 1.0 / 120);
    e = fma(r, e, 1.0 / 24);
    e = fma(r, e, 1.0 / 6);
    e = fma(r, e, 0.5);
    e = fma(r, e, 1.0);
    e = fma(r, e, 1.0) * s.tab[n & 7];
    return __hiloint2double(__double2hiint(e) + ((n >> 3) << 20), __double2loint(e));
  };
  auto fixed = [&](double w) {
    const double big = 4503599627370496.0;  // 2^52: the sum's low bits are the integer
    return (u64)(__double_as_longlong(fma(w, unit, big)) - __double_as_longlong(big));
  };
  // bins of the histogram: equal steps of M - x over the values that take part
  const float range = fminf(diff(mn), reach);
  const float step = range > 0.f ? ((float)kBins - 0.5f) / range : 0.f;
  auto bin_of = [&](float x) {
    const float f = diff(x) * step;
    return f < (float)(kBins - 1) ? (int)f : f >= (float)(kBins - 1) ? kBins - 1 : 0;
  };
  auto finish = [&](int idx, float x, u64 total) {
    p.idx[row] = idx;
    if (p.logprob)
      p.logprob[row] = (float)((x == mx ? 0.0 : ((double)x - (double)mx) * inv_t) -
                               log((double)total / unit));
  };
  // does the draw fall to an element (or part) of mass w behind mass w0?  At
  // u = 1 the last with any mass takes it
  auto holds = [&](u64 w0, u64 w, double draw, u64 total) {
    return w > 0 && !((double)w0 > draw) && ((double)(w0 + w) > draw || w0 + w == total);
  };

  auto push = [&](float x, int i) {  // onto the first CTA's list
    const int n = atomicAdd(&peer0->list_n, 1);
    if (n < kList) peer0->list[n].key = ((u64)~key_of(x) << 32) | (uint32_t)(lo + i);
  };
  auto x_of = [&](u64 key) { return float_of(~(uint32_t)(key >> 32)); };
  // Thread e's entry of the first CTA's list: how many entries and how much mass
  // lie before it in the filters' order.
  auto place = [&](int n, u64 key, int& before, u64& mass) {
    before = 0;
    mass = 0;
#pragma unroll 4
    for (int j = 0; j < n; ++j) {
      const Entry o = s.list[j];
      const bool first = o.key < key;
      before += first;
      mass += first ? o.w : 0;
    }
  };

  // ---- small top-k: a lower bound of the k-th largest, then a list
  if (k && 4 * k <= 3 * groups) {
    if (warp == 0) {
      uint32_t key[kMaxCluster * kGroups / 32];
#pragma unroll
      for (int i = 0; i < kMaxCluster * kGroups / 32; ++i)
        key[i] = 32 * i < groups ? key_of(s.gmax[lane + 32 * i]) : 0;
      uint32_t tau = 0;  // largest value of its upper 20 bits with k keys at or above it
#pragma unroll 1
      for (int bit = 31; bit >= 12; --bit) {
        const uint32_t want = tau | (1u << bit);
        int c = 0;
#pragma unroll
        for (int i = 0; i < kMaxCluster * kGroups / 32; ++i) c += key[i] >= want;
        if (__reduce_add_sync(full, c) >= k) tau = want;
      }
      if (lane == 0) s.tau = tau > key_of(-INFINITY) ? float_of(tau) : -INFINITY;
    }
    __syncthreads();
    const float tau = s.tau;
    each([&](float x, int i) {
      if (x >= tau && x > -INFINITY) push(x, i);
    });
    cluster.sync();
    const int n = peer0->list_n;
    cluster.sync();  // every CTA has read it
    if (n <= kList) {
      if (rank != 0) return;
      const bool mine = tid < n;
      const u64 key = mine ? s.list[tid].key : ~0ull;
      const float x = x_of(key);
      const double wd = mine && takes_part(x) ? weight(x) : 0.0;
      const u64 w = fixed(wd);
      if (mine) s.list[tid].w = w;
      __syncthreads();
      int before;
      u64 m0;
      place(mine ? n : 0, key, before, m0);
      const int first_k = min(k, n);
      if (mine && before == first_k - 1) s.total = m0 + w;
      __syncthreads();
      const bool keep = mine && before < first_k &&
                        (!use_p || (double)m0 < (double)top_p * (double)s.total) &&
                        wd >= (double)min_p;
      if (mine && !keep) s.list[tid].w = 0;
      __syncthreads();
      if (!keep) return;
      u64 total = 0, w0 = 0;  // kept mass, and what of it lies before this index
#pragma unroll 4
      for (int j = 0; j < n; ++j) {
        const Entry o = s.list[j];
        total += o.w;
        w0 += (uint32_t)o.key < (uint32_t)key ? o.w : 0;
      }
      if (holds(w0, w, (double)u * (double)total, total)) finish((int)(uint32_t)key, x, total);
      return;
    }
    if (tid == 0) s.list_n = 0;
  }

  const int slice = kBins / C;  // bins this CTA adds up for the cluster
  // Sum the cluster's histograms and tell everybody the slices' totals; `guess`
  // fills in masses (in coarser units) from the bins' middles.
  auto merge_hist = [&](bool with_mass, bool guess) {
    cluster.sync();
    u64 c = 0, m = 0;
    for (int b = tid; b < slice; b += kThreads) {
      const int bin = rank * slice + b;
      uint32_t cc = 0;
      u64 mm = 0;
      for (int q = 0; q < C; ++q) {
        const Shared* o = cluster.map_shared_rank(&s, q);
        cc += o->cnt[bin];
        if (with_mass) mm += o->mass[bin];
      }
      if (guess && cc) {
        const float mid = step > 0.f ? ((float)bin + 0.5f) / step : 0.f;
        mm = (u64)((double)cc * (double)exp2f(-mid * (float)to8 * 0.125f) * (unit / 256));
      }
      s.cnt[bin] = cc;  // only this CTA reads its own slice
      s.mass[bin] = mm;
      c += cc;
      m += mm;
    }
    u64 c0, m0, ct, mt;
    block_scan(s, c, m, c0, m0, ct, mt);
    if (tid < C) {
      Shared* q = cluster.map_shared_rank(&s, tid);
      q->tot_c[rank] = ct;
      q->tot_m[rank] = mt;
    }
    cluster.sync();
  };
  // First bin at which the count (by_mass false) or mass, on top of what lies
  // above the histogram, reaches the target.
  auto find = [&](bool by_mass, u64 above_c, u64 above_m, double target) {
    auto reached = [&](u64 c, u64 m) {
      return by_mass ? !((double)(above_m + m) < target) : (double)(above_c + c) >= target;
    };
    u64 c0 = 0, m0 = 0;
    for (int q = 0; q < rank; ++q) { c0 += s.tot_c[q]; m0 += s.tot_m[q]; }
    const u64 ct = s.tot_c[rank], mt = s.tot_m[rank];
    if (!reached(c0, m0) && reached(c0 + ct, m0 + mt)) {  // uniform over the CTA
      const int per = (slice + kThreads - 1) / kThreads;
      u64 c = 0, m = 0;
      for (int j = 0; j < per; ++j) {
        const int b = tid * per + j;
        if (b < slice) { c += s.cnt[rank * slice + b]; m += s.mass[rank * slice + b]; }
      }
      u64 ca, ma, t1, t2;
      block_scan(s, c, m, ca, ma, t1, t2);
      ca += c0;
      ma += m0;
      for (int j = 0; j < per; ++j) {
        const int b = rank * slice + tid * per + j;
        if (tid * per + j >= slice) break;
        const u64 cb = ca + s.cnt[b], mb = ma + s.mass[b];
        if (!reached(ca, ma) && reached(cb, mb))
          for (int q = 0; q < C; ++q)
            cluster.map_shared_rank(&s, q)->cut = {b, (int)s.cnt[b], above_c + ca, above_m + ma,
                                                   s.mass[b]};
        ca = cb;
        ma = mb;
      }
    }
    cluster.sync();
    return s.cut;
  };
  auto clear_hist = [&](bool with_mass) {
    for (int b = tid; b < kBins; b += kThreads) {
      s.cnt[b] = 0;
      if (with_mass) s.mass[b] = 0;
    }
    __syncthreads();
  };
  auto count_all = [&](bool with_mass) {
    each([&](float x, int) {
      if (!takes_part(x)) return;
      const int b = bin_of(x);
      atomicAdd(&s.cnt[b], 1u);
      if (with_mass) atomicAdd(&s.mass[b], fixed(weight(x)));
    });
  };
  // The first CTA orders the list's n entries, which follow (above_c, above_m),
  // and tells everybody the last one of the prefix that reaches the target.
  auto cut_list = [&](int n, bool by_mass, u64 above_c, u64 above_m, double target) {
    if (rank == 0) {
      const bool mine = tid < n;
      const u64 key = mine ? s.list[tid].key : ~0ull;
      const u64 w = mine ? fixed(weight(x_of(key))) : 0;
      if (mine) s.list[tid].w = w;
      __syncthreads();
      int before;
      u64 m0;
      place(mine ? n : 0, key, before, m0);
      auto more = [&](int c, u64 m) {  // does the prefix go on behind these?
        return by_mass ? (double)(above_m + m) < target : (double)(above_c + (u64)c) < target;
      };
      if (mine && more(before, m0) && (before + 1 == n || !more(before + 1, m0 + w)))
        for (int q = 0; q < C; ++q) {
          Shared* o = cluster.map_shared_rank(&s, q);
          o->cut_key = ~(uint32_t)(key >> 32);
          o->cut_idx = (int)(uint32_t)key;
          o->list_mass = above_m + m0 + w;
        }
    }
    cluster.sync();
  };

  // Exact last element of a prefix that ends in bin `c.bin`, by count or mass.
  auto refine = [&](bool by_mass, Cut c, double target, bool need_mass, u64& mass_upto) {
    uint32_t klo = 0xffffffffu, khi = 0;
    each([&](float x, int) {
      if (!takes_part(x) || bin_of(x) != c.bin) return;
      const uint32_t key = key_of(x);
      klo = min(klo, key);
      khi = max(khi, key);
    });
    klo = __reduce_min_sync(full, klo);
    khi = __reduce_max_sync(full, khi);
    __syncthreads();
    if (lane == 0) { s.redu[warp] = klo; s.redu[kWarps + warp] = khi; }
    __syncthreads();
    if (tid < C) {
      for (int w = 0; w < kWarps; ++w) {
        klo = min(klo, s.redu[w]);
        khi = max(khi, s.redu[kWarps + w]);
      }
      Shared* q = cluster.map_shared_rank(&s, tid);
      q->kmin[rank] = klo;
      q->kmax[rank] = khi;
    }
    cluster.sync();
    for (int q = 0; q < C; ++q) { klo = min(klo, s.kmin[q]); khi = max(khi, s.kmax[q]); }
    u64 above_c = c.cnt0, above_m = c.mass0;
    int n = c.cnt_in;
    while (n > kList && klo < khi) {
      // finer bins of the keys [klo, khi]; each round takes 11 bits off their span
      const int sh = max(0, 32 - __clz(khi - klo) - 11);
      clear_hist(true);
      each([&](float x, int) {
        if (!takes_part(x)) return;
        const uint32_t key = key_of(x);
        if (key < klo || key > khi) return;
        atomicAdd(&s.cnt[(khi - key) >> sh], 1u);
        if (need_mass) atomicAdd(&s.mass[(khi - key) >> sh], fixed(weight(x)));
      });
      merge_hist(true, false);
      const Cut d = find(by_mass, above_c, above_m, target);
      khi -= (uint32_t)d.bin << sh;
      klo = max(klo, khi - min(khi, (1u << sh) - 1));
      above_c = d.cnt0;
      above_m = d.mass0;
      n = d.cnt_in;
      cluster.sync();  // the histograms may be cleared again
    }
    if (n <= kList) {
      if (rank == 0 && tid == 0) s.list_n = 0;
      cluster.sync();
      each([&](float x, int i) {
        if (!takes_part(x)) return;
        const uint32_t key = key_of(x);
        if (key >= klo && key <= khi) push(x, i);
      });
      cluster.sync();
      cut_list(n, by_mass, above_c, above_m, target);
    } else {
      // n equal values: the prefix takes the first `need` of them by index
      const u64 w = fixed(weight(float_of(khi)));
      u64 need;
      if (by_mass) {
        const double gap = target - (double)above_m;
        need = w ? (u64)(gap / (double)w) : (u64)n;
        need = need > 2 ? need - 2 : 1;
        while (need < (u64)n && (double)(above_m + need * w) < target) ++need;
        if (need < 1) need = 1;
      } else {
        need = (u64)target - above_c;
      }
      auto at = [&](int i) { return widen(kResident ? vals[i] : src[i]); };
      u64 mine = 0;
      for (int i = tid; i < nv; i += kThreads) mine += key_of(at(i)) == khi;
      u64 a0, b0, tot, bt;
      block_scan(s, mine, 0, a0, b0, tot, bt);
      if (tid < C) cluster.map_shared_rank(&s, tid)->part[rank] = tot;
      cluster.sync();
      u64 before = 0;
      for (int q = 0; q < rank; ++q) before += s.part[q];
      if (before < need && need <= before + tot) {  // uniform over the CTA
        u64 seen = before;
        for (int i0 = 0; i0 < nv; i0 += kThreads) {
          const int i = i0 + tid;
          const u64 hit = i < nv && key_of(at(i)) == khi ? 1 : 0;
          block_scan(s, hit, 0, a0, b0, tot, bt);
          if (hit && seen + a0 + 1 == need)
            for (int q = 0; q < C; ++q) {
              Shared* o = cluster.map_shared_rank(&s, q);
              o->cut_key = khi;
              o->cut_idx = lo + i;
              o->list_mass = above_m + need * w;
            }
          seen += tot;
          if (seen >= need) break;
        }
      }
      cluster.sync();
    }
    mass_upto = s.list_mass;
  };

  // ---- the sums of the row and of its warps' parts, in vocabulary order.
  // win: first bin of the three summed apart (use_p)
  const int seg = (nv + kWarps - 1) / kWarps, seg_v = (seg + 32 * kV - 1) / (32 * kV) * (32 * kV);
  const int w_lo = min(nv, warp * seg_v), w_hi = min(nv, w_lo + seg_v);
  auto sum_row = [&](bool bins, int win, auto keep) {
    Sums a = {};
    sweep(w_lo, w_hi, lane, 32, [&](float x, int i) {
      if (!takes_part(x)) return;
      const double wd = weight(x);
      const u64 w = fixed(wd);
      if (bins) {
        const int b = bin_of(x) - win;
        a.all += w;
        a.above += b < 0 ? w : 0;
#pragma unroll
        for (int j = 0; j < 3; ++j) a.in[j] += b == j ? w : 0;
      }
      a.minp += keep(x, i, wd) ? w : 0;
    });
    u64* f = reinterpret_cast<u64*>(&a);
#pragma unroll
    for (int j = 0; j < kSums; ++j) {
      if (!bins && j != kSums - 1) continue;
#pragma unroll
      for (int o = 16; o; o >>= 1) f[j] += __shfl_xor_sync(full, f[j], o);
    }
    __syncthreads();
    if (lane == 0) s.warp_sum[warp] = a;
    __syncthreads();
    if (tid < kSums * C) {  // the CTA's total of field tid % kSums, to CTA tid / kSums
      u64 t = 0;
      for (int w = 0; w < kWarps; ++w)
        t += reinterpret_cast<const u64*>(&s.warp_sum[w])[tid % kSums];
      reinterpret_cast<u64*>(&cluster.map_shared_rank(&s, tid / kSums)->cta_sum[rank])[tid % kSums] =
          t;
    }
    cluster.sync();
  };

  // ---- the cut: keep keys above cut_key, and at it up to index cut_idx
  uint32_t cut_key = 0;
  int cut_idx = 0x7fffffff;
  bool by_minp = !use_p && !k;  // min-p's set (all, if it is off) is what is kept
  bool summed = false;          // warp_sum / cta_sum hold the row's sums
  int cut_bin = 0, win = 0;
  u64 kept_in = 0;              // mass kept in cut_bin
  if (k) {
    // a large k, or one among many equal logits: refine, then top-p of its mass
    // over a fresh histogram; the earlier cut counts
    cluster.sync();
    clear_hist(true);
    count_all(use_p);
    merge_hist(true, false);
    u64 all_c = 0, limit_m = 0;
    for (int q = 0; q < C; ++q) { all_c += s.tot_c[q]; limit_m += s.tot_m[q]; }
    if ((u64)k < all_c) {
      const Cut ck = find(false, 0, 0, (double)k);
      cluster.sync();
      refine(false, ck, (double)k, use_p, limit_m);
      cut_key = s.cut_key;
      cut_idx = s.cut_idx;
    }
    if (use_p) {
      const uint32_t k_key = cut_key;
      const int k_idx = cut_idx;
      cluster.sync();
      clear_hist(true);
      count_all(true);
      merge_hist(true, false);
      const double target = (double)top_p * (double)limit_m;
      const Cut cp = find(true, 0, 0, target);
      cluster.sync();
      u64 m;
      refine(true, cp, target, true, m);
      cut_key = s.cut_key;
      cut_idx = s.cut_idx;
      if (k_key > cut_key || (k_key == cut_key && k_idx < cut_idx)) {
        cut_key = k_key;
        cut_idx = k_idx;
      }
    }
  } else if (use_p) {
    count_all(false);
    merge_hist(false, true);
    u64 guess_m = 0;
    for (int q = 0; q < C; ++q) guess_m += s.tot_m[q];
    win = find(true, 0, 0, (double)top_p * (double)guess_m).bin - 1;
    sum_row(true, win, [&](float, int, double wd) { return wd >= (double)min_p; });
    Sums t = {};
    for (int q = 0; q < C; ++q) {
      t.all += s.cta_sum[q].all;
      t.above += s.cta_sum[q].above;
      for (int j = 0; j < 3; ++j) t.in[j] += s.cta_sum[q].in[j];
    }
    const double target = (double)top_p * (double)t.all;
    u64 above = t.above;
    int j = 0;
    while (j < 3 && (double)(above + t.in[j]) < target) above += t.in[j++];
    if (j < 3 && (double)t.above < target) {  // the cut lies in bin win + j
      cut_bin = win + j;
      each([&](float x, int i) {
        if (takes_part(x) && bin_of(x) == cut_bin) push(x, i);
      });
      cluster.sync();
      const int n = peer0->list_n;
      cluster.sync();
      if (n <= kList) {
        cut_list(n, true, 0, above, target);
        cut_key = s.cut_key;
        cut_idx = s.cut_idx;
        kept_in = s.list_mass - above;
        summed = true;
        // min-p is the tighter filter if the last element kept fails it
        by_minp = min_p > 0.f && !(weight(float_of(cut_key)) >= (double)min_p);
      }
    }
    if (!summed) {  // the guess was off, or the bin holds too many
      cluster.sync();
      clear_hist(true);
      count_all(true);
      merge_hist(true, false);
      const Cut cp = find(true, 0, 0, target);
      cluster.sync();
      u64 m;
      refine(true, cp, target, true, m);
      cut_key = s.cut_key;
      cut_idx = s.cut_idx;
    }
  }
  auto kept = [&](float x, int i) {  // by the cut alone
    const uint32_t key = key_of(x);
    return key > cut_key || (key == cut_key && lo + i <= cut_idx);
  };

  // ---- kept mass of this warp's part, what lies before it, the total
  u64 mine = 0, before = 0, total = 0;
  if (summed && !by_minp) {
    // bins before the cut's are kept whole; of its own bin, look at each element
    if (kept_in) {
      sweep(w_lo, w_hi, lane, 32, [&](float x, int i) {
        if (takes_part(x) && bin_of(x) == cut_bin && kept(x, i)) mine += fixed(weight(x));
      });
#pragma unroll
      for (int o = 16; o; o >>= 1) mine += __shfl_xor_sync(full, mine, o);
    }
    const Sums& a = s.warp_sum[warp];
    mine += a.above + (cut_bin > win ? a.in[0] : 0) + (cut_bin > win + 1 ? a.in[1] : 0);
    if (lane == 0) s.scan_a[warp] = mine;
    __syncthreads();
    u64 cta = 0;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += s.scan_a[w];
      cta += s.scan_a[w];
    }
    if (tid < C) cluster.map_shared_rank(&s, tid)->part[rank] = cta;
    cluster.sync();
    for (int q = 0; q < C; ++q) {
      if (q < rank) before += s.part[q];
      total += s.part[q];
    }
  } else {
    if (!summed)
      sum_row(false, 0, [&](float x, int i, double wd) {
        return wd >= (double)min_p && (by_minp || kept(x, i));
      });
    for (int w = 0; w < warp; ++w) before += s.warp_sum[w].minp;
    mine = s.warp_sum[warp].minp;
    for (int q = 0; q < C; ++q) {
      if (q < rank) before += s.cta_sum[q].minp;
      total += s.cta_sum[q].minp;
    }
  }
  const double draw = (double)u * (double)total;
  if (!holds(before, mine, draw, total)) return;  // uniform over the warp; one warp stays
  u64 run = before;
  for (int i0 = w_lo; i0 < w_hi; i0 += 32) {
    const int i = i0 + lane;
    const float x = i < w_hi ? widen(kResident ? vals[i] : src[i]) : -INFINITY;
    u64 w = 0;
    if (takes_part(x) && (by_minp || kept(x, i))) {
      const double wd = weight(x);
      w = wd >= (double)min_p ? fixed(wd) : 0;
    }
    u64 inc = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const u64 up = __shfl_up_sync(full, inc, o);
      if (lane >= o) inc += up;
    }
    const bool hit = holds(run + inc - w, w, draw, total);
    if (hit) finish(lo + i, x, total);
    if (__any_sync(full, hit)) break;
    run += __shfl_sync(full, inc, 31);
  }
}

template <typename T, bool kResident>
int launch_filter(FilterParams& p, int cluster, size_t smem, cudaStream_t st) {
  static bool done[64] = {false};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return ORTHRUS_ECUDA;
  if (dev < 0 || dev >= 64 || !done[dev]) {
    if (cudaFuncSetAttribute(filter_kernel<T, kResident>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)(sizeof(Shared) + 16 + kResidentBytes)) != cudaSuccess)
      return ORTHRUS_ECUDA;
    if (dev >= 0 && dev < 64) done[dev] = true;
  }
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = cluster;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.rows * cluster);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, filter_kernel<T, kResident>, p) == cudaSuccess ? ORTHRUS_OK
                                                                                : ORTHRUS_ECUDA;
}

}  // namespace
}  // namespace orthrus

using namespace orthrus;

extern "C" int orthrus_vocab_sample_filtered(const orthrus_filter_args* a,
                                             orthrus_stream_t stream) {
  if (!a || (a->dtype != ORTHRUS_F32 && a->dtype != ORTHRUS_BF16)) return ORTHRUS_EINVAL;
  if (a->rows < 0 || a->vocab < 1 || a->row_stride < a->vocab) return ORTHRUS_EINVAL;
  if (a->rows > 65535 || a->vocab > (1 << 24)) return ORTHRUS_EUNSUPPORTED;
  if (a->rows == 0) return ORTHRUS_OK;
  const int es = a->dtype == ORTHRUS_F32 ? 4 : 2;
  if (!a->logits || reinterpret_cast<uintptr_t>(a->logits) % es || !a->u || !a->idx)
    return ORTHRUS_EINVAL;
  FilterParams p;
  p.logits = a->logits; p.stride = a->row_stride; p.u = a->u;
  p.temperature = a->temperature; p.top_k = a->top_k; p.top_p = a->top_p; p.min_p = a->min_p;
  p.idx = a->idx; p.logprob = a->logprob; p.err = a->err;
  p.rows = a->rows; p.vocab = a->vocab;
  int bits = 0;
  while ((1 << bits) < a->vocab) ++bits;
  p.shift = 62 - bits < 52 ? 62 - bits : 52;
  p.vec = reinterpret_cast<uintptr_t>(a->logits) % 16 == 0 && a->row_stride * es % 16 == 0;
  // CTAs a row: up to 8, of at least 2048 elements each
  int cluster = 1;
  while (cluster < kMaxCluster && a->vocab > 2048 * cluster) cluster *= 2;
  p.chunk = ((a->vocab + cluster - 1) / cluster + 7) / 8 * 8;
  const size_t tables = (sizeof(Shared) + 15) / 16 * 16;
  const bool resident = (int64_t)p.chunk * es <= kResidentBytes;
  const size_t smem = tables + (resident ? (size_t)p.chunk * es : 0);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (a->dtype == ORTHRUS_F32)
    return resident ? launch_filter<float, true>(p, cluster, smem, st)
                    : launch_filter<float, false>(p, cluster, smem, st);
  return resident ? launch_filter<__nv_bfloat16, true>(p, cluster, smem, st)
                  : launch_filter<__nv_bfloat16, false>(p, cluster, smem, st);
}
