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
// filters take (a vocabulary too large for that is read again, from L2).  Two
// ways through:
//   list     the elements down to the cut's bin fit a 1024-entry list (top-k of
//            a few hundred, top-p of a peaked row): the first CTA sorts them and
//            finishes the row alone
//   general  the cuts are refined bin by bin to an exact element, then one
//            pass sums the kept weights and the CTA that holds the draw finds
//            it
#include <cooperative_groups.h>
#include <math.h>

#include "common.cuh"

namespace cg = cooperative_groups;

namespace orthrus {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kList = 1024;
constexpr int kMaxCluster = 8;
constexpr int kResidentBytes = 160 * 1024;  // row part a CTA may hold, beside 45 KB of tables
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

struct Shared {
  u64 mass[kBins];
  u64 list[kList];    // (~key << 32) | index: ascending = descending value, then index
  u64 weight[kList];
  uint32_t cnt[kBins];
  float mx[kMaxCluster], mn[kMaxCluster];
  uint32_t kmin[kMaxCluster], kmax[kMaxCluster];
  u64 tot_c[kMaxCluster], tot_m[kMaxCluster];
  u64 scan_a[kWarps], scan_b[kWarps];
  u64 part[kMaxCluster];
  float redf[2 * kWarps];
  uint32_t redu[2 * kWarps];
  Cut cut;
  uint32_t cut_key;
  int cut_idx;
  int list_n;
  u64 list_mass;
  int pick;
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

// Bitonic sort of the first n (a power of two <= kList) entries of s.list,
// s.weight following.
__device__ __forceinline__ void sort_list(Shared& s, int n) {
  for (int k = 2; k <= n; k <<= 1)
    for (int j = k >> 1; j; j >>= 1) {
      __syncthreads();
      for (int t = threadIdx.x; t < n / 2; t += kThreads) {
        const int i = 2 * j * (t / j) + t % j;
        const u64 a = s.list[i], b = s.list[i + j];
        if ((a > b) == ((i & k) == 0)) {
          s.list[i] = b;
          s.list[i + j] = a;
          const u64 w = s.weight[i];
          s.weight[i] = s.weight[i + j];
          s.weight[i + j] = w;
        }
      }
    }
  __syncthreads();
}

template <typename T, bool kResident>
__global__ void __launch_bounds__(kThreads, 1) filter_kernel(const FilterParams p) {
  extern __shared__ __align__(16) uint8_t dyn[];
  Shared& s = *reinterpret_cast<Shared*>(dyn);
  T* vals = reinterpret_cast<T*>(dyn + (sizeof(Shared) + 15) / 16 * 16);
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int row = blockIdx.x / C;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int lo = min(p.vocab, rank * p.chunk), hi = min(p.vocab, lo + p.chunk), nv = hi - lo;
  const T* src = static_cast<const T*>(p.logits) + row * p.stride + lo;
  Shared* peer0 = cluster.map_shared_rank(&s, 0);
  auto at = [&](int i) { return widen(kResident ? vals[i] : src[i]); };

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

  // ---- read this part of the row; maximum and minimum
  float mx = -INFINITY, mn = INFINITY;
  constexpr int kV = 16 / sizeof(T);
  if (kResident && p.vec) {
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
  for (int o = 16; o; o >>= 1) {
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
  }
  if (lane == 0) { s.redf[warp] = mx; s.redf[kWarps + warp] = mn; }
  for (int b = tid; b < kBins; b += kThreads) { s.cnt[b] = 0; s.mass[b] = 0; }
  if (tid == 0) { s.list_n = 0; s.pick = -1; }
  __syncthreads();
  if (tid < C) {
    for (int w = 0; w < kWarps; ++w) {
      mx = fmaxf(mx, s.redf[w]);
      mn = fminf(mn, s.redf[kWarps + w]);
    }
    Shared* q = cluster.map_shared_rank(&s, tid);
    q->mx[rank] = mx;
    q->mn[rank] = mn;
  }
  cluster.sync();
  for (int c = 0; c < C; ++c) { mx = fmaxf(mx, s.mx[c]); mn = fminf(mn, s.mn[c]); }
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

  const double inv_t = 1.0 / (double)T_;
  const double unit = (double)(1ull << p.shift);
  auto diff = [&](float x) { return x == mx ? 0.f : mx - x; };
  const float reach = kDropT * T_;
  auto takes_part = [&](float x) { return x > -INFINITY && diff(x) <= reach; };
  auto weight = [&](float x) { return x == mx ? 1.0 : exp(((double)x - (double)mx) * inv_t); };
  auto fixed = [&](double w) { return (u64)(w * unit + 0.5); };
  // bins of the histogram: equal steps of M - x over the values that take part
  const float range = fminf(diff(mn), reach);
  const float step = range > 0.f ? ((float)kBins - 0.5f) / range : 0.f;
  auto bin_of = [&](float x) {
    const float f = diff(x) * step;
    return f < (float)(kBins - 1) ? (int)f : f >= (float)(kBins - 1) ? kBins - 1 : 0;
  };

  const int slice = kBins / C;  // bins this CTA adds up for the cluster
  // Sum the cluster's histograms and tell everybody the slices' totals.
  auto merge_hist = [&]() {
    cluster.sync();
    u64 c = 0, m = 0;
    for (int b = tid; b < slice; b += kThreads) {
      const int bin = rank * slice + b;
      uint32_t cc = 0;
      u64 mm = 0;
      for (int q = 0; q < C; ++q) {
        const Shared* o = cluster.map_shared_rank(&s, q);
        cc += o->cnt[bin];
        mm += o->mass[bin];
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
  auto push = [&](float x, int i) {  // onto the first CTA's list
    const int n = atomicAdd(&peer0->list_n, 1);
    if (n < kList) peer0->list[n] = ((u64)~key_of(x) << 32) | (uint32_t)(lo + i);
  };
  // First CTA: weights of the list's entries, sorted into the filters' order.
  auto sorted_list = [&]() {
    const int n = min(s.list_n, kList);
    int n2 = 1;
    while (n2 < n) n2 <<= 1;
    for (int e = tid; e < n2; e += kThreads) {
      if (e < n) s.weight[e] = fixed(weight(float_of(~(uint32_t)(s.list[e] >> 32))));
      else { s.list[e] = ~0ull; s.weight[e] = 0; }
    }
    sort_list(s, n2);
    return n;
  };

  // Exact last element of a prefix that ends in bin `c.bin`, by count or mass.
  auto refine = [&](bool by_mass, Cut c, double target, bool need_mass, u64& mass_upto) {
    uint32_t klo = 0xffffffffu, khi = 0;
    for (int i = tid; i < nv; i += kThreads) {
      const float x = at(i);
      if (!takes_part(x) || bin_of(x) != c.bin) continue;
      const uint32_t key = key_of(x);
      klo = min(klo, key);
      khi = max(khi, key);
    }
    klo = __reduce_min_sync(0xffffffffu, klo);
    khi = __reduce_max_sync(0xffffffffu, khi);
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
      for (int b = tid; b < kBins; b += kThreads) { s.cnt[b] = 0; s.mass[b] = 0; }
      __syncthreads();
      for (int i = tid; i < nv; i += kThreads) {
        const float x = at(i);
        if (!takes_part(x)) continue;
        const uint32_t key = key_of(x);
        if (key < klo || key > khi) continue;
        atomicAdd(&s.cnt[(khi - key) >> sh], 1u);
        if (need_mass) atomicAdd(&s.mass[(khi - key) >> sh], fixed(weight(x)));
      }
      merge_hist();
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
      for (int i = tid; i < nv; i += kThreads) {
        const float x = at(i);
        if (!takes_part(x)) continue;
        const uint32_t key = key_of(x);
        if (key >= klo && key <= khi) push(x, i);
      }
      cluster.sync();
      if (rank == 0) {
        const int m = sorted_list();
        // last entry of the prefix: entries whose predecessors do not reach the target
        u64 carry = 0;
        for (int e0 = 0; e0 < m; e0 += kThreads) {
          const int e = e0 + tid;
          const u64 w = e < m ? s.weight[e] : 0;
          u64 w0, d0, wt, dt;
          block_scan(s, w, 0, w0, d0, wt, dt);
          w0 += carry;
          carry += wt;
          if (e < m) {
            auto more = [&](int e1, u64 m1) {
              return by_mass ? (double)(above_m + m1) < target
                             : (double)(above_c + (u64)e1) < target;
            };
            if (more(e, w0) && !(e + 1 < m && more(e + 1, w0 + w)))
              for (int q = 0; q < C; ++q) {
                Shared* o = cluster.map_shared_rank(&s, q);
                o->cut_key = ~(uint32_t)(s.list[e] >> 32);
                o->cut_idx = (int)(uint32_t)s.list[e];
                o->list_mass = above_m + w0 + w;
              }
          }
        }
      }
      cluster.sync();
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

  // ---- the cuts
  uint32_t cut_key = 0;       // keep keys above it,
  int cut_idx = 0x7fffffff;   // and at it up to this index
  bool list = false;          // the row ends in the first CTA's list
  double list_total = 0;      // top-p's whole mass, if not the list's first k
  if (k || use_p) {
    const bool need_mass = use_p && !(k && k <= kList / 2);
    for (int i = tid; i < nv; i += kThreads) {
      const float x = at(i);
      if (!takes_part(x)) continue;
      const int b = bin_of(x);
      atomicAdd(&s.cnt[b], 1u);
      if (need_mass) atomicAdd(&s.mass[b], fixed(weight(x)));
    }
    merge_hist();
    u64 all_c = 0, all_m = 0;
    for (int q = 0; q < C; ++q) { all_c += s.tot_c[q]; all_m += s.tot_m[q]; }
    Cut ck{kBins - 1, 0, 0, 0, 0};
    u64 limit_m = all_m;
    int last_bin = kBins - 1;
    const bool cut_k = k && (u64)k < all_c;
    if (cut_k) {
      ck = find(false, 0, 0, (double)k);
      last_bin = ck.bin;
      list = ck.cnt0 + (u64)ck.cnt_in <= kList;
    } else if (k) {
      list = all_c <= kList;
    }
    if (!list && use_p && !need_mass) {
      // many equal values around the k-th: masses are needed after all
      cluster.sync();
      for (int b = tid; b < kBins; b += kThreads) { s.cnt[b] = 0; s.mass[b] = 0; }
      __syncthreads();
      for (int i = tid; i < nv; i += kThreads) {
        const float x = at(i);
        if (!takes_part(x)) continue;
        const int b = bin_of(x);
        atomicAdd(&s.cnt[b], 1u);
        atomicAdd(&s.mass[b], fixed(weight(x)));
      }
      merge_hist();
      all_m = 0;
      for (int q = 0; q < C; ++q) all_m += s.tot_m[q];
      limit_m = all_m;
      if (cut_k) ck = find(false, 0, 0, (double)k);
    }
    if (!list && use_p && !cut_k) {
      const Cut cp = find(true, 0, 0, (double)top_p * (double)all_m);
      if (cp.cnt0 + (u64)cp.cnt_in <= kList) {
        list = true;
        list_total = (double)all_m;
        last_bin = cp.bin;
      } else {
        u64 m;
        cluster.sync();
        refine(true, cp, (double)top_p * (double)all_m, true, m);
        cut_key = s.cut_key;
        cut_idx = s.cut_idx;
      }
    } else if (!list && cut_k) {
      // top-k by refinement, then top-p of its mass over a fresh histogram
      // (refine() may have used the tables); the earlier cut counts
      cluster.sync();
      refine(false, ck, (double)k, use_p, limit_m);
      cut_key = s.cut_key;
      cut_idx = s.cut_idx;
      if (use_p) {
        const uint32_t k_key = cut_key;
        const int k_idx = cut_idx;
        cluster.sync();
        for (int b = tid; b < kBins; b += kThreads) { s.cnt[b] = 0; s.mass[b] = 0; }
        __syncthreads();
        for (int i = tid; i < nv; i += kThreads) {
          const float x = at(i);
          if (!takes_part(x)) continue;
          const int b = bin_of(x);
          atomicAdd(&s.cnt[b], 1u);
          atomicAdd(&s.mass[b], fixed(weight(x)));
        }
        merge_hist();
        const double target = (double)top_p * (double)limit_m;
        const Cut cp = find(true, 0, 0, target);
        cluster.sync();
        u64 m;
        refine(true, cp, target, true, m);
        // the earlier of the two cuts
        cut_key = s.cut_key;
        cut_idx = s.cut_idx;
        if (k_key > cut_key || (k_key == cut_key && k_idx < cut_idx)) {
          cut_key = k_key;
          cut_idx = k_idx;
        }
      }
    }
    if (list) {
      for (int i = tid; i < nv; i += kThreads) {
        const float x = at(i);
        if (takes_part(x) && bin_of(x) <= last_bin) push(x, i);
      }
      cluster.sync();
      if (rank != 0) return;  // nothing of theirs is read any more
      const int n = sorted_list();
      const int first_k = k ? min(k, n) : n;
      // mass of the first k, then the entries kept
      u64 mine = 0;
      for (int e = tid; e < first_k; e += kThreads) mine += s.weight[e];
      u64 a0, b0, total, bt;
      block_scan(s, mine, 0, a0, b0, total, bt);
      const double target =
          use_p ? (double)top_p * (list_total > 0 ? list_total : (double)total) : 0;
      u64 carry = 0, kept_mass = 0;
      int kept = 0;
      for (int e0 = 0; e0 < n; e0 += kThreads) {
        const int e = e0 + tid;
        const u64 w = e < n ? s.weight[e] : 0;
        u64 wt;
        block_scan(s, w, 0, a0, b0, wt, bt);
        const bool keep = e < first_k && (!use_p || (double)(carry + a0) < target) &&
                          (min_p == 0.f ||
                           weight(float_of(~(uint32_t)(s.list[e] >> 32))) >= (double)min_p);
        carry += wt;
        u64 km, kc;
        block_scan(s, keep ? w : 0, keep ? 1 : 0, a0, b0, km, kc);
        kept_mass += km;
        kept += (int)kc;  // kept entries are a prefix
      }
      // the draw, in index order
      __syncthreads();
      int n2 = 1;
      while (n2 < kept) n2 <<= 1;
      for (int e = tid; e < n2; e += kThreads) {
        if (e < kept) s.list[e] = (s.list[e] << 32) | (s.list[e] >> 32);
        else { s.list[e] = ~0ull; s.weight[e] = 0; }
      }
      sort_list(s, n2);
      const double draw = (double)u * (double)kept_mass;
      carry = 0;
      for (int e0 = 0; e0 < kept; e0 += kThreads) {
        const int e = e0 + tid;
        const u64 w = e < kept ? s.weight[e] : 0;
        u64 wt;
        block_scan(s, w, 0, a0, b0, wt, bt);
        const u64 w0 = carry + a0;
        carry += wt;
        // the first whose cumulated mass exceeds the draw; at u = 1 the last with any
        const bool hit = w > 0 && !((double)w0 > draw) &&
                         ((double)(w0 + w) > draw || w0 + w == kept_mass);
        if (hit) {
          p.idx[row] = (int)(uint32_t)(s.list[e] >> 32);
          if (p.logprob) {
            const float x = float_of(~(uint32_t)s.list[e]);
            p.logprob[row] = (float)((x == mx ? 0.0 : ((double)x - (double)mx) * inv_t) -
                                     log((double)kept_mass / unit));
          }
        }
      }
      return;
    }
  }

  // ---- general: sum the kept weights in vocabulary order
  auto kept_weight = [&](float x, int i) -> u64 {
    if (!takes_part(x)) return 0;
    const uint32_t key = key_of(x);
    if (key < cut_key || (key == cut_key && lo + i > cut_idx)) return 0;
    const double w = weight(x);
    return w >= (double)min_p ? fixed(w) : 0;
  };
  const int seg = ((nv + kWarps - 1) / kWarps + 31) / 32 * 32;  // elements of a warp
  const int w_lo = min(nv, warp * seg), w_hi = min(nv, w_lo + seg);
  u64 mine = 0;
  for (int i = w_lo + lane; i < w_hi; i += 32) mine += kept_weight(at(i), i);
  for (int o = 16; o; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
  __syncthreads();
  if (lane == 0) s.scan_a[warp] = mine;
  __syncthreads();
  u64 cta = 0, before = 0;
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += s.scan_a[w];
    cta += s.scan_a[w];
  }
  if (tid < C) cluster.map_shared_rank(&s, tid)->part[rank] = cta;
  cluster.sync();
  u64 total = 0;
  for (int q = 0; q < C; ++q) {
    if (q < rank) before += s.part[q];
    total += s.part[q];
  }
  const double draw = (double)u * (double)total;
  auto holds = [&](u64 w0, u64 w) {
    return w > 0 && !((double)w0 > draw) && ((double)(w0 + w) > draw || w0 + w == total);
  };
  if (!holds(before, mine)) return;  // uniform over the warp; one warp of the cluster stays
  u64 run = before;
  for (int i0 = w_lo; i0 < w_hi; i0 += 32) {
    const int i = i0 + lane;
    const float x = i < w_hi ? at(i) : -INFINITY;
    const u64 w = kept_weight(x, i);
    u64 inc = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const u64 up = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += up;
    }
    const bool hit = holds(run + inc - w, w);
    if (hit) {
      p.idx[row] = lo + i;
      if (p.logprob)
        p.logprob[row] = (float)((x == mx ? 0.0 : ((double)x - (double)mx) * inv_t) -
                                 log((double)total / unit));
    }
    if (__any_sync(0xffffffffu, hit)) break;
    run += __shfl_sync(0xffffffffu, inc, 31);
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
