// attn_paged.cu -- bf16 block attention over a paged K/V cache on the
// 5th-generation tensor cores, with the batch's common prefix read once
// (include/orthrus_paged.h).
//
// Mathematics.  The online softmax of attn_tc.cu: per query row a running
// maximum m and sum l over 128-key tiles, O rescaled only when m grows by more
// than 2^8, partial (m, l, O) of different key ranges merged by
//   O = sum_s 2^(m_s - M) O_s / sum_s 2^(m_s - M) l_s,  M = max_s m_s.
//
// Work.  One unit is one 128-row query tile against one key range:
//   - prefix units (kv-head g, row tile t): the rows of ns = 128 / (G blk)
//     consecutive sequences packed into one tile, against keys [0, P) of row
//     0's pages -- with one token a sequence the whole batch shares one read
//     of the prefix instead of one read a sequence;
//   - tail units (sequence b, kv-head g): the sequence's G blk rows against
//     its own keys (from P if it shares the prefix) and the block rows.
// The units' tiles, W in all, form one sequence that is dealt out evenly: CTA
// c of C (one per SM) takes tiles [c chunk, (c + 1) chunk), crossing unit
// boundaries, so a ragged batch loads every SM alike whatever its lengths.  A
// unit that lies in one CTA and has no prefix is normalised and written
// straight to the output; every other piece leaves a partial (O, m, l) in the
// workspace and a second kernel merges them in tile order, so the result
// depends on the lengths only, not on timing.
//
// Per CTA (12 warps):
//   warp 0       K producer: lane i of a tile's boxes loads one page's rows of
//                one 64-dim half (the page ids of the next tile are read while
//                this one waits), 2-stage ring
//   warp 1       MMA issuer (one thread), as in attn_tc.cu
//   warp 2       V producer, like warp 0
//   warp 3       Q tiles
//   warps 4..11  softmax, two warpgroups taking turns on the tiles
// Producers run ahead over unit boundaries.  The first warpgroup hands
// registers to the two softmax ones (72 + 2 x 216 = 3 x 168 a thread).
//
// NaN and infinities.  Scores of keys a row may not see are replaced, never
// multiplied; V rows past the keys are zeroed in shared memory.  Keys that
// only the later rows of a causal block see share their tile's P V product
// with rows that do not: there a non-finite V element is zeroed as well and
// added to the rows that see it when their O leaves the tensor memory.
//
// Every mbarrier wait is bounded as in attn_tc.cu.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <math.h>

#include <mutex>

#include "attn_paged.cuh"
#include "common.cuh"
#include "tc_ptx.cuh"

namespace orthrus {
namespace {

constexpr int kRows = 128;  // UMMA M
constexpr int kTile = 128;  // keys per tile
constexpr int kStages = 2;
constexpr int kThreads = 384;
constexpr int kTmemCols = 512;  // S0 [0,128) S1 [128,256) O_0 [256,256+D) O_1 after it
constexpr int kOCol = 256;
constexpr float kLazyThresh = 8.f;  // log2 units
constexpr int kFlagRing = 8;        // segments whose flags may be alive at once
constexpr int kMinChunk = 2;        // tiles a CTA takes at least
constexpr int kMergeRows = 8;       // query rows of one merging CTA

constexpr int kHalfTile = kTile * 128;
constexpr int kQBytes = 2 * kRows * 128;
constexpr int kStageBytes = 4 * kHalfTile;
constexpr int kRingOff = kQBytes;
constexpr int kPBytes = 2 * kRows * 128;
constexpr int kPOff = kRingOff + kStages * kStageBytes;
constexpr int kBarOff = kPOff + 2 * kPBytes;
constexpr int kNumBars = 13 + 4 * kStages;
constexpr int kMiscOff = kBarOff + kNumBars * 8;
// TMEM address, abort flag, start of the walk, scan words, segment flags
constexpr int kSmemBytes = kMiscOff + 256 + 1024;  // + alignment slack
static_assert(kSmemBytes <= 232448, "shared memory of one CTA");

struct __align__(64) PagedParams {
  CUtensorMap tm_qp;  // 3D (D, Hq, B*blk), box (64, G, ns*blk)
  CUtensorMap tm_q;   // the same tensor, box (64, G, blk)
  CUtensorMap tm_k;   // 2D (D, pages*Hkv*page_size), box (64, min(page_size, 128))
  CUtensorMap tm_v;
  CUtensorMap tm_kb;  // 3D (D, Hkv, B*blk), box (64, 1, blk)
  CUtensorMap tm_vb;
  const int32_t* ctx_lens;
  const int32_t* table;
  const __nv_bfloat16* v_pages;
  const __nv_bfloat16* v_blk;  // NULL: the block's rows are in the pages
  __nv_bfloat16* out;
  int32_t* err;
  // workspace: [0] chunk, [1] prefix tiles, [2..] tail tiles before each sequence
  int32_t* head;
  float2* ml_p;   // (m, l) of the prefix partials [slot][128]
  float* o_p;     // their O, [slot][D/4][128][4]
  float2* ml_t;   // the same of the tail partials, rows per slot = G*blk
  float* o_t;
  int B, Hq, Hkv, G, blk, rowsT, ns, Tq, Kp, P, page_size, pages, max_pages, max_ctx, causal;
  float scale_log2;
};

struct Bars {
  uint32_t base;
  __device__ uint32_t at(int i) const { return base + 8 * i; }
  __device__ uint32_t q_full() const { return at(0); }
  __device__ uint32_t q_free() const { return at(1); }  // every S of the segment is done
  __device__ uint32_t o_free() const { return at(2); }  // O of the segment has been read
  __device__ uint32_t seg_done() const { return at(3); }  // every P V of the segment is done
  __device__ uint32_t exit_done() const { return at(4); }
  __device__ uint32_t k_full(int s) const { return at(5 + s); }
  __device__ uint32_t v_full(int s) const { return at(5 + kStages + s); }
  __device__ uint32_t k_empty(int s) const { return at(5 + 2 * kStages + s); }
  __device__ uint32_t v_empty(int s) const { return at(5 + 3 * kStages + s); }
  __device__ uint32_t s_full(int b) const { return at(5 + 4 * kStages + b); }
  __device__ uint32_t s_free(int b) const { return at(7 + 4 * kStages + b); }
  __device__ uint32_t p_full(int b) const { return at(9 + 4 * kStages + b); }
  __device__ uint32_t pv_done(int b) const { return at(11 + 4 * kStages + b); }
};

__device__ __forceinline__ void record_timeout(int32_t* err, volatile int* abort_flag) {
  *abort_flag = 1;
  set_err(err, ORTHRUS_ETIMEOUT);
}

// ------------------------------------------------------------ the schedule

// Does the sequence take its first P keys from the shared prefix?
__host__ __device__ __forceinline__ bool shares(int n, int P, int in_cache_rows) {
  return P > 0 && n - in_cache_rows >= P;
}

// 128-key cache tiles of a tail that covers keys [lo, n): tile indexes are
// absolute, the first tile is lo / 128.
__device__ __forceinline__ int cache_tiles(int lo, int n) {
  return n > lo ? ceil_div(n, kTile) - lo / kTile : 0;
}

__device__ __forceinline__ int tail_tiles(const PagedParams& p, int n) {
  if (n < 0 || n > p.max_ctx) return 0;
  const int own = p.v_blk ? 0 : p.blk;
  return cache_tiles(shares(n, p.P, own) ? p.P : 0, n) + (p.v_blk ? 1 : 0);
}

struct Seg {
  int prefix;  // a prefix unit (b is then the row tile)
  int b, g;
  int n;       // context length of the sequence (prefix: P)
  int lo;      // first key
  int first;   // absolute index of the unit's first 128-key tile
  int Tc;      // cache tiles of the unit; tile Tc is the block's
  int t0, U;   // tiles [t0, t0 + U) of the unit
  int T;       // tiles of the unit
};

// Walks a CTA's tiles [pos, end) unit by unit.  Every warp role keeps one.
struct Walk {
  int pos, end, base;  // base: prefix tiles in all
  int b, g, t;         // next tail tile
  __device__ __forceinline__ bool next(const PagedParams& p, Seg& s) {
    if (pos >= end) return false;
    if (pos < base) {
      const int unit = pos / p.Kp;
      s.prefix = 1;
      s.g = unit / p.Tq;
      s.b = unit - s.g * p.Tq;
      s.t0 = pos - unit * p.Kp;
      s.T = s.Tc = p.Kp;
      s.n = p.P;
      s.lo = 0;
      s.first = 0;
    } else {
      int n, T;
      for (;;) {
        if (b >= p.B) return false;  // only if lengths change under the kernel
        n = p.ctx_lens[b];
        T = tail_tiles(p, n);
        if (t < T) break;
        t = 0;
        if (T > 0 && g + 1 < p.Hkv) { ++g; break; }
        g = 0;
        ++b;
      }
      s.prefix = 0;
      s.b = b;
      s.g = g;
      s.n = n;
      s.lo = shares(n, p.P, p.v_blk ? 0 : p.blk) ? p.P : 0;
      s.first = s.lo / kTile;
      s.Tc = cache_tiles(s.lo, n);
      s.T = T;
      s.t0 = t;
    }
    s.U = min(s.T - s.t0, end - pos);
    pos += s.U;
    if (!s.prefix) t += s.U;
    return true;
  }
};

// Slot of a tail piece.  Without a prefix only the first and the last segment
// of a CTA can be pieces of a unit; with one every tail unit may leave a
// partial, and (unit, CTA) steps through the schedule like a staircase, so
// unit + CTA numbers the pieces without gaps.
__device__ __forceinline__ int tail_slot(const PagedParams& p, int b, int g, int c,
                                         bool first_seg) {
  return p.P > 0 ? b * p.Hkv + g + c : 2 * c + (first_seg ? 0 : 1);
}

// --------------------------------------------------------------- main kernel

__device__ __forceinline__ void mask_range(uint32_t (&sv)[2][32], int k0, int lo, int hi) {
#pragma unroll
  for (int cb = 0; cb < 2; ++cb)
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      const int k = k0 + 32 * cb + j;
      if (k < lo || k >= hi) sv[cb][j] = __float_as_uint(-INFINITY);
    }
}

__device__ __forceinline__ bool nonfinite_bf16(uint32_t half) {
  return (half & 0x7f80u) == 0x7f80u;
}

template <int kD>
__global__ void __launch_bounds__(kThreads, 1)
attn_paged_kernel(const __grid_constant__ PagedParams p) {
  constexpr int halves = kD / 64;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = ptx::smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const unsigned full_mask = 0xffffffffu;
  const int C = gridDim.x, c = blockIdx.x;

  const Bars bars{sbase + kBarOff};
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + kMiscOff);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kMiscOff + 4);
  int* start = reinterpret_cast<int*>(smem + kMiscOff + 8);  // pos, end, base, b, g, t
  int* scan = reinterpret_cast<int*>(smem + kMiscOff + 32);  // one word a warp
  volatile int* bad_page = reinterpret_cast<volatile int*>(smem + kMiscOff + 96);
  volatile int* agreed = reinterpret_cast<volatile int*>(smem + kMiscOff + 92);
  volatile int* has_nf = reinterpret_cast<volatile int*>(smem + kMiscOff + 96 + 4 * kFlagRing);

  if (threadIdx.x == 0) {
    *abort_flag = 0;
    ptx::mbar_init(bars.q_full(), 1);
    ptx::mbar_init(bars.q_free(), 1);
    ptx::mbar_init(bars.o_free(), 256);
    ptx::mbar_init(bars.seg_done(), 1);
    ptx::mbar_init(bars.exit_done(), 1);
    for (int s = 0; s < kStages; ++s) {
      ptx::mbar_init(bars.k_full(s), 1);
      ptx::mbar_init(bars.v_full(s), 1);
      ptx::mbar_init(bars.k_empty(s), 1);
      ptx::mbar_init(bars.v_empty(s), 1);
    }
    for (int s = 0; s < 2; ++s) {
      ptx::mbar_init(bars.s_full(s), 1);
      ptx::mbar_init(bars.s_free(s), 128);
      ptx::mbar_init(bars.p_full(s), 128);
      ptx::mbar_init(bars.pv_done(s), 1);
    }
    ptx::fence_mbar_init();
  }
  if (threadIdx.x < kFlagRing) bad_page[threadIdx.x] = has_nf[threadIdx.x] = 0;
  if (warp == 0 && lane == 0) {
    ptx::tma_prefetch_desc(&p.tm_q);
    ptx::tma_prefetch_desc(&p.tm_k);
    ptx::tma_prefetch_desc(&p.tm_v);
  }
  if (warp == 1) {
    ptx::tmem_alloc(ptx::smem_u32(tmem_holder), kTmemCols);
    ptx::tmem_relinquish();
  }
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();

  // ---- the schedule: total tail tiles, then where this CTA's share begins
  {
    int mine = 0;
    for (int b = threadIdx.x; b < p.B; b += kThreads) mine += tail_tiles(p, p.ctx_lens[b]);
    for (int o = 16; o; o >>= 1) mine += __shfl_xor_sync(full_mask, mine, o);
    if (lane == 0) scan[warp] = mine;
    __syncthreads();
    int tail = 0;
    for (int w = 0; w < kThreads / 32; ++w) tail += scan[w];
    const int base = p.Hkv * p.Tq * p.Kp;
    const int W = base + p.Hkv * tail;
    const int chunk = max(kMinChunk, ceil_div(W, C));
    const int pos = min(W, c * chunk), end = min(W, pos + chunk);
    const int want = max(0, pos - base);
    if (threadIdx.x == 0) {
      start[0] = pos;
      start[1] = end;
      start[2] = base;
      start[3] = start[4] = start[5] = 0;
      if (c == 0) {
        p.head[0] = chunk;
        p.head[1] = base;
      }
    }
    __syncthreads();
    int before = 0;  // tail tiles (of one kv-head) before this batch of sequences
    for (int b0 = 0; b0 < p.B; b0 += kThreads) {
      const int b = b0 + threadIdx.x;
      const int T = b < p.B ? tail_tiles(p, p.ctx_lens[b]) : 0;
      int inc = T;
      for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(full_mask, inc, o);
        if (lane >= o) inc += up;
      }
      if (lane == 31) scan[warp] = inc;
      __syncthreads();
      int off = before, all = 0;
      for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) off += scan[w];
        all += scan[w];
      }
      const int at = off + inc - T;  // tiles before sequence b
      if (b < p.B && c == 0) p.head[2 + b] = at;
      if (T > 0 && want >= p.Hkv * at && want < p.Hkv * (at + T)) {
        const int rem = want - p.Hkv * at;
        start[3] = b;
        start[4] = rem / T;
        start[5] = rem % T;
      }
      before += all;
      __syncthreads();
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  Walk walk{start[0], start[1], start[2], start[3], start[4], start[5]};
  if (threadIdx.x < 32)  // lengths out of range: reported once
    if (c == 0)
      for (int b = lane; b < p.B; b += 32) {
        const int n = p.ctx_lens[b];
        if (n < 0 || n > p.max_ctx) set_err(p.err, ORTHRUS_ECAPACITY);
      }

  const uint32_t q_s = sbase;
  auto k_s = [&](int st) { return sbase + kRingOff + st * kStageBytes; };
  auto v_s = [&](int st) { return sbase + kRingOff + st * kStageBytes + 2 * kHalfTile; };
  auto p_s = [&](int x) { return sbase + kPOff + x * kPBytes; };
  Seg s;

  if (warp < 4) {
    ptx::reg_dec<72>();
  if (warp == 0 || warp == 2) {
    // ================================================== K and V producers
    const bool is_v = warp == 2;
    const CUtensorMap* tm = is_v ? &p.tm_v : &p.tm_k;
    const CUtensorMap* tmb = is_v ? &p.tm_vb : &p.tm_kb;
    const int box = min(p.page_size, kTile);  // rows of one box
    const int npg = kTile / box;              // pages a tile touches at most
    const int mh = lane / npg, mi = lane % npg;  // this lane's half and page of a tile
    int u = 0;  // tiles issued by this CTA so far
    bool stop = false;
    for (int sg = 0; !stop && walk.next(p, s); ++sg) {
      if (!is_v && lane == 0) bad_page[sg % kFlagRing] = 0;
      const int32_t* row = p.table + (int64_t)(s.prefix ? 0 : s.b) * p.max_pages;
      // page of this lane's box of unit tile t: -1 if it holds no key of the unit
      auto page_of = [&](int t) {
        if (mh >= halves || t >= s.Tc) return -1;
        const int k0 = (s.first + t) * kTile + mi * box;
        if (k0 >= s.n || k0 + box <= s.lo) return -1;
        return row[k0 / p.page_size];
      };
      int id = page_of(s.t0);
      for (int t = s.t0; t < s.t0 + s.U; ++t, ++u) {
        const int st = u % kStages;
        const uint32_t empty = is_v ? bars.v_empty(st) : bars.k_empty(st);
        const uint32_t bar = is_v ? bars.v_full(st) : bars.k_full(st);
        const uint32_t dst = is_v ? v_s(st) : k_s(st);
        const int id_next = t + 1 < s.t0 + s.U ? page_of(t + 1) : -1;
        if (__any_sync(full_mask, *abort_flag != 0) ||
            !__all_sync(full_mask, ptx::mbar_wait(empty, ((u / kStages) & 1) ^ 1))) {
          if (!*abort_flag) record_timeout(p.err, abort_flag);
          stop = true;
          break;
        }
        if (t == s.Tc) {  // the block rows
          if (lane == 0) {
            ptx::mbar_expect_tx(bar, (uint32_t)(halves * p.blk * 128));
            for (int h = 0; h < halves; ++h)
              ptx::tma_load_3d(dst + h * kHalfTile, tmb, bar, 64 * h, s.g, s.b * p.blk);
          }
        } else {
          const int k0 = (s.first + t) * kTile + mi * box;
          const bool has = mh < halves && k0 < s.n && k0 + box > s.lo;
          const bool ok = has && id >= 0 && id < p.pages;
          if (has && !ok && !is_v) {
            bad_page[sg % kFlagRing] = 1;
            set_err(p.err, ORTHRUS_EINVAL);
          }
          const int boxes = __popc(__ballot_sync(full_mask, ok));
          __syncwarp();
          if (lane == 0) {
            if (boxes)
              ptx::mbar_expect_tx(bar, (uint32_t)(boxes * box * 128));
            else
              ptx::mbar_arrive(bar);  // nothing to load: every page was refused
          }
          __syncwarp();
          if (ok)
            ptx::tma_load_2d(dst + mh * kHalfTile + mi * box * 128, tm, bar, 64 * mh,
                             (id * p.Hkv + s.g) * p.page_size + k0 % p.page_size);
        }
        id = id_next;
      }
    }
    // every issued load must have landed before the CTA exits
    for (int x = max(0, u - kStages); x < u; ++x) {
      const uint32_t bar = is_v ? bars.v_full(x % kStages) : bars.k_full(x % kStages);
      if (!ptx::mbar_wait(bar, (x / kStages) & 1)) record_timeout(p.err, abort_flag);
    }
  } else if (warp == 3) {
    // ================================================== Q tiles
    if (lane == 0) {
      int sg = 0;
      for (; walk.next(p, s); ++sg) {
        if (*abort_flag || (sg > 0 && !ptx::mbar_wait(bars.q_free(), (sg - 1) & 1))) {
          if (!*abort_flag) record_timeout(p.err, abort_flag);
          break;
        }
        const int nb = s.prefix ? p.ns : 1, b0 = s.prefix ? s.b * p.ns : s.b;
        ptx::mbar_expect_tx(bars.q_full(), (uint32_t)(halves * nb * p.rowsT * 128));
        for (int h = 0; h < halves; ++h)
          ptx::tma_load_3d(q_s + h * (kRows * 128), s.prefix ? &p.tm_qp : &p.tm_q,
                           bars.q_full(), 64 * h, s.g * p.G, b0 * p.blk);
      }
      if (sg > 0 && !ptx::mbar_wait(bars.q_full(), (sg - 1) & 1))
        record_timeout(p.err, abort_flag);
    }
  } else {
    // ================================================== MMA issuer
    if (lane == 0) {
      const uint32_t id_s = ptx::idesc_bf16(kRows, kTile, false, false);
      const uint32_t id_pv = ptx::idesc_bf16(kRows, kD, false, true);
      auto s_tile = [&](int u) {
        const int st = u % kStages;
#pragma unroll
        for (int k = 0; k < kD / 16; ++k) {
          const uint32_t h = k >> 2, kk = k & 3;
          const uint64_t ad = ptx::sdesc_sw128(q_s + h * (kRows * 128) + kk * 32, 16, 1024);
          const uint64_t bd = ptx::sdesc_sw128(k_s(st) + h * kHalfTile + kk * 32, 16, 1024);
          ptx::mma_ss(tmem + (u & 1) * kTile, ad, bd, id_s, k > 0 ? 1u : 0u);
        }
        ptx::tc_commit(bars.s_full(u & 1));
        ptx::tc_commit(bars.k_empty(st));
      };
      auto pv_tile = [&](int u, bool fresh) {
        const int st = u % kStages;
#pragma unroll
        for (int k = 0; k < kTile / 16; ++k) {
          const uint32_t h = k >> 2, kk = k & 3;
          const uint64_t ad =
              ptx::sdesc_sw128(p_s(u & 1) + h * (kRows * 128) + kk * 32, 16, 1024);
          const uint64_t bd = ptx::sdesc_sw128(v_s(st) + k * 2048, kHalfTile, 1024);
          ptx::mma_ss(tmem + kOCol + (u & 1) * kD, ad, bd, id_pv, (!fresh || k > 0) ? 1u : 0u);
        }
        ptx::tc_commit(bars.pv_done(u & 1));
        ptx::tc_commit(bars.v_empty(st));
      };
      // S of tile u: its buffer's previous scores read, its keys there
      auto try_s = [&](int u) {
        if (u > 1 && !ptx::mbar_wait(bars.s_free(u & 1), ((u >> 1) - 1) & 1)) return false;
        if (!ptx::mbar_wait(bars.k_full(u % kStages), (u / kStages) & 1)) return false;
        ptx::tc_fence_after();
        s_tile(u);
        return true;
      };
      int u0 = 0;
      bool ok = true;
      for (int sg = 0; ok && walk.next(p, s); ++sg) {
        const int u1 = u0 + s.U;
        ok = !*abort_flag && ptx::mbar_wait(bars.q_full(), sg & 1);
        for (int u = u0; ok && u < min(u0 + 2, u1); ++u) ok = try_s(u);
        if (ok && s.U <= 2) ptx::tc_commit(bars.q_free());
        // O of the previous segment must have been read
        if (ok && sg > 0) ok = ptx::mbar_wait(bars.o_free(), (sg - 1) & 1);
        for (int u = u0; ok && u < u1 && !*abort_flag; ++u) {
          if (u + 2 < u1) {
            ok = try_s(u + 2);
            if (!ok) break;
            if (u + 3 == u1) ptx::tc_commit(bars.q_free());
          }
          ok = ptx::mbar_wait(bars.p_full(u & 1), (u >> 1) & 1) &&
               ptx::mbar_wait(bars.v_full(u % kStages), (u / kStages) & 1);
          if (!ok) break;
          ptx::tc_fence_after();
          pv_tile(u, u < u0 + 2);
        }
        if (ok) ptx::tc_commit(bars.seg_done());
        u0 = u1;
      }
      if (!ok && !*abort_flag) record_timeout(p.err, abort_flag);
      // everything issued has finished before TMEM is freed
      ptx::tc_commit(bars.exit_done());
      if (!ptx::mbar_wait(bars.exit_done(), 0)) record_timeout(p.err, abort_flag);
    }
  }
  } else {
    // ================================================== softmax
    ptx::reg_inc<216>();
    const int X = (warp - 4) >> 2;
    const int quad = warp & 3;
    const int r = quad * 32 + lane;
    const uint32_t lane_addr = tmem + ((uint32_t)(quad * 32) << 16);
    const int wg_tid = threadIdx.x - 128 - 128 * X;
    const float cs = p.scale_log2;
    bool alive = true;
    int u0 = 0;
    for (int sg = 0; walk.next(p, s); ++sg) {
      const int u1 = u0 + s.U;
      // this row's sequence and block row; rows past the tile's are padding
      const int rows = s.prefix ? min(p.ns, p.B - s.b * p.ns) * p.rowsT : p.rowsT;
      const bool row_ok = r < rows;
      const int bq = s.prefix ? s.b * p.ns + (row_ok ? r / p.rowsT : 0) : s.b;
      const int rt = row_ok ? (s.prefix ? r % p.rowsT : r) : 0;  // row within its sequence
      const int i_blk = rt / p.G;
      // cache keys this row sees: [lo, lim)
      int lim = s.n;
      if (s.prefix) {
        const int nb = p.ctx_lens[bq];
        if (nb > p.max_ctx || !shares(nb, p.P, p.v_blk ? 0 : p.blk)) lim = 0;
      } else if (!p.v_blk && p.causal) {
        lim = s.n - p.blk + i_blk + 1;
      }
      if (!row_ok) lim = 0;
      // keys from here on are not seen by the block's first row
      const int fence = s.prefix || !p.causal ? 0x7fffffff : (p.v_blk ? s.n : s.n - p.blk) + 1;
      const bool warp_rows = quad * 32 < rows;  // any row of this warp in use
      float m_ref = -INFINITY, l = 0.f;
      for (int u = u0 + ((u0 & 1) != X); alive && u < u1; u += 2) {
        if (__any_sync(full_mask, *abort_flag != 0)) { alive = false; break; }
        const int t = s.t0 + (u - u0), st = u % kStages;
        if (!__all_sync(full_mask, ptx::mbar_wait(bars.s_full(X), (u >> 1) & 1))) {
          record_timeout(p.err, abort_flag); alive = false; break;
        }
        ptx::tc_fence_after();
        const bool blk_tile = t == s.Tc;
        const int k0 = blk_tile ? s.n : (s.first + t) * kTile;  // position of the tile's key 0
        const int nv_tile = blk_tile ? p.blk : min(kTile, s.n - k0);
        const int lo_tile = blk_tile ? 0 : max(0, s.lo - k0);
        int nv = blk_tile ? (p.causal ? i_blk + 1 : p.blk) : lim - k0;
        nv = row_ok ? max(0, min(nv, nv_tile)) : 0;
        const uint32_t s_addr = lane_addr + X * kTile;
        float f = 1.f;
        bool rescale = false;
        uint32_t sv[2][32];
        if (warp_rows) {
          float mt[2] = {-INFINITY, -INFINITY};
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            ptx::tmem_ld32(s_addr + 64 * half, sv[0]);
            ptx::tmem_ld32(s_addr + 64 * half + 32, sv[1]);
            ptx::tmem_wait_ld();
            if (nv < kTile || lo_tile > 0) mask_range(sv, 64 * half, lo_tile, nv);
#pragma unroll
            for (int cb = 0; cb < 2; ++cb)
#pragma unroll
              for (int j = 0; j < 32; ++j) mt[cb] = fmaxf(mt[cb], __uint_as_float(sv[cb][j]));
          }
          const float ms = fmaxf(mt[0], mt[1]) * cs;
          const bool need = ms > m_ref + kLazyThresh;
          rescale = __any_sync(full_mask, need);
          if (rescale) {
            const float m_new = need ? ms : m_ref;
            f = m_ref == -INFINITY ? 0.f : ptx::ex2(m_ref - m_new);
            if (!need) f = 1.f;
            m_ref = m_new;
          }
        }
        if (u > 1) {
          if (!__all_sync(full_mask, ptx::mbar_wait(bars.pv_done(X), ((u >> 1) - 1) & 1))) {
            record_timeout(p.err, abort_flag); alive = false; break;
          }
          ptx::tc_fence_after();
        }
        if (warp_rows) {
          const float nm = m_ref == -INFINITY ? 0.f : -m_ref;
          float ls[4] = {0.f, 0.f, 0.f, 0.f};
          uint8_t* prow = smem + kPOff + X * kPBytes + r * 128;
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            const int half = 1 - hh;
            if (hh == 1) {
              ptx::tmem_ld32(s_addr, sv[0]);
              ptx::tmem_ld32(s_addr + 32, sv[1]);
              ptx::tmem_wait_ld();
              ptx::tc_fence_before();
              ptx::mbar_arrive(bars.s_free(X));
              if (nv < kTile || lo_tile > 0) mask_range(sv, 0, lo_tile, nv);
            }
#pragma unroll
            for (int ch = 0; ch < 8; ++ch) {
              uint32_t w4[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int kk = 8 * ch + 2 * e;
                const float p0 = ptx::ex2(fmaf(__uint_as_float(sv[kk >> 5][kk & 31]), cs, nm));
                const float p1 =
                    ptx::ex2(fmaf(__uint_as_float(sv[kk >> 5][(kk & 31) + 1]), cs, nm));
                ls[e] += p0 + p1;
                w4[e] = ptx::pack_bf16x2(p0, p1);
              }
              *reinterpret_cast<uint4*>(prow + half * (kRows * 128) + ((ch ^ (r & 7)) << 4)) =
                  make_uint4(w4[0], w4[1], w4[2], w4[3]);
            }
          }
          l = l * f + ((ls[0] + ls[1]) + (ls[2] + ls[3]));
          if (rescale && u > u0 + 1) {
#pragma unroll
            for (int cb = 0; cb < kD / 32; ++cb) {
              uint32_t o[32];
              ptx::tmem_ld32_sync(lane_addr + kOCol + X * kD + cb * 32, o);
#pragma unroll
              for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
              ptx::tmem_st32(lane_addr + kOCol + X * kD + cb * 32, o);
            }
            ptx::tmem_wait_st();
          }
        } else {
          ptx::mbar_arrive(bars.s_free(X));
        }
        const int fz = blk_tile ? (p.causal ? 1 : kTile) : max(lo_tile, fence - k0);
        if (nv_tile < kTile || lo_tile > 0 || fz < nv_tile) {
          if (!__all_sync(full_mask, ptx::mbar_wait(bars.v_full(st), (u / kStages) & 1))) {
            record_timeout(p.err, abort_flag); alive = false; break;
          }
          uint8_t* vt = smem + kRingOff + st * kStageBytes + 2 * kHalfTile;
          // rows outside the keys [lo_tile, nv_tile) hold anything: zero them,
          // and the non-finite elements of rows [fz, nv_tile)
          for (int e = wg_tid; e < kTile * 8 * halves; e += 128) {
            const int h = e / (kTile * 8), row = (e / 8) % kTile;
            if (row >= lo_tile && row < min(fz, nv_tile)) continue;
            uint4* at = reinterpret_cast<uint4*>(vt + h * kHalfTile + (e % (kTile * 8)) * 16);
            if (row < lo_tile || row >= nv_tile) {
              *at = make_uint4(0, 0, 0, 0);
              continue;
            }
            const uint4 v = *at;
            uint32_t w[4] = {v.x, v.y, v.z, v.w};
            bool found = false;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if (nonfinite_bf16(w[i])) { w[i] &= 0xffff0000u; found = true; }
              if (nonfinite_bf16(w[i] >> 16)) { w[i] &= 0xffffu; found = true; }
            }
            if (found) {
              *at = make_uint4(w[0], w[1], w[2], w[3]);
              has_nf[sg % kFlagRing] = 1;
            }
          }
        }
        ptx::fence_proxy_async_smem();
        ptx::tc_fence_before();
        ptx::mbar_arrive(bars.p_full(X));
      }
      // ---- the segment's O, row maxima and sums
      if (alive && !__all_sync(full_mask, ptx::mbar_wait(bars.seg_done(), sg & 1))) {
        record_timeout(p.err, abort_flag);
        alive = false;
      }
      // (max, sum) of the two warpgroups through P's shared memory, which no
      // MMA reads any more; both must get here even after a time-out
      float2* xch = reinterpret_cast<float2*>(smem + kPOff);
      ptx::named_bar_sync(1, 256);
      if (X == 0 && wg_tid == 0) *agreed = *abort_flag;
      const bool mine = X == (u0 & 1) || s.U > 1;  // this warpgroup had a tile
      xch[X * kRows + r] = mine ? make_float2(m_ref, l) : make_float2(-INFINITY, 0.f);
      ptx::named_bar_sync(1, 256);
      const float2 a0 = xch[r], a1 = xch[kRows + r];
      const int nf = has_nf[sg % kFlagRing], bad = bad_page[sg % kFlagRing];
      const int stop = *agreed;  // one answer for all, so that they leave together
      ptx::named_bar_sync(1, 256);
      if (wg_tid == 0 && X == 0) has_nf[(sg + kFlagRing / 2) % kFlagRing] = 0;
      if (stop) break;
      u0 = u1;
      if (!alive) continue;
      ptx::tc_fence_after();
      const float m = fmaxf(a0.x, a1.x);
      const float f0 = a0.x == -INFINITY ? 0.f : ptx::ex2(a0.x - m);
      const float f1 = a1.x == -INFINITY ? 0.f : ptx::ex2(a1.x - m);
      // sums may be NaN with a maximum of -inf (every visible score NaN)
      const float L = (a0.x == -INFINITY ? a0.y : f0 * a0.y) + (a1.x == -INFINITY ? a1.y : f1 * a1.y);
      const bool t0 = a0.y != 0.f, t1 = a1.y != 0.f;  // any weight (or NaN) in that half
      // keys this row sees in this unit's pieces at all (none: zeros)
      const bool direct = !s.prefix && s.U == s.T && s.lo == 0;
      const int seen = (p.v_blk ? 1 : 0) + max(0, lim);
      const float inv = direct ? (seen > 0 ? 1.f / L : 0.f) : 1.f;
      int slot = 0;
      if (s.prefix)
        slot = s.g * p.Tq + s.b + c;
      else if (!direct)
        slot = tail_slot(p, s.b, s.g, c, sg == 0);
      const int srows = s.prefix ? kRows : p.rowsT;
      float* po = (s.prefix ? p.o_p : p.o_t) + (int64_t)slot * srows * kD;
      __nv_bfloat16* orow =
          p.out + ((int64_t)(bq * p.blk + i_blk) * p.Hq + s.g * p.G + rt % p.G) * kD;
#pragma unroll 1
      for (int cb = 0; cb < kD / 64; ++cb) {
        const int col = X * (kD / 2) + cb * 32;
        float v[32];
        if (warp_rows) {
          // selects, not products: an O that no tile wrote may hold anything
          uint32_t o[32];
          ptx::tmem_ld32_sync(lane_addr + kOCol + col, o);
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = t0 ? f0 * __uint_as_float(o[j]) : 0.f;
          ptx::tmem_ld32_sync(lane_addr + kOCol + kD + col, o);
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = t1 ? fmaf(f1, __uint_as_float(o[j]), v[j]) : v[j];
        }
        if (cb == kD / 64 - 1) {  // O is read: the next segment may overwrite it
          ptx::tc_fence_before();
          ptx::mbar_arrive(bars.o_free());
        }
        if (!row_ok || bad) continue;
        if (nf) {
          // non-finite V elements of the block's keys that this row sees
          const int first = p.v_blk ? s.n + 1 : max(s.n - p.blk + 1, 0);
          const int last = p.v_blk ? s.n + i_blk : lim - 1;
          for (int key = first; key <= last; ++key) {
            const __nv_bfloat16* vr;
            const int tile = p.v_blk ? s.Tc : key / kTile - s.first;
            if (tile < s.t0 || tile >= s.t0 + s.U) continue;
            if (p.v_blk) {
              vr = p.v_blk + ((int64_t)(s.b * p.blk + key - s.n) * p.Hkv + s.g) * kD;
            } else {
              const int id = p.table[(int64_t)s.b * p.max_pages + key / p.page_size];
              vr = p.v_pages + (((int64_t)id * p.Hkv + s.g) * p.page_size + key % p.page_size) * kD;
            }
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              const float x = __bfloat162float(vr[col + j]);
              if (!isfinite(x)) v[j] += x;
            }
          }
        }
        if (direct) {
#pragma unroll
          for (int j8 = 0; j8 < 4; ++j8) {
            uint32_t w4[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int j = 8 * j8 + 2 * e;
              w4[e] = ptx::pack_bf16x2(seen > 0 ? v[j] * inv : 0.f,
                                       seen > 0 ? v[j + 1] * inv : 0.f);
            }
            *reinterpret_cast<uint4*>(orow + col + 8 * j8) = make_uint4(w4[0], w4[1], w4[2], w4[3]);
          }
        } else {
          const int row = s.prefix ? r : rt;
#pragma unroll
          for (int j4 = 0; j4 < 8; ++j4)
            __stcg(reinterpret_cast<float4*>(po) + (col / 4 + j4) * srows + row,
                   make_float4(v[4 * j4], v[4 * j4 + 1], v[4 * j4 + 2], v[4 * j4 + 3]));
        }
      }
      if (X == 0 && row_ok && !direct) {
        // NaN in the maximum marks a piece whose pages were refused
        float2* ml = (s.prefix ? p.ml_p : p.ml_t) + (int64_t)slot * srows + (s.prefix ? r : rt);
        __stcg(ml, bad ? make_float2(__int_as_float(0x7fffffff), 0.f) : make_float2(m, L));
      }
    }
  }
  __syncwarp();
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, kTmemCols);
  }
}

// ------------------------------------------------------------------- merge

// Grid (B * Hkv, groups of kMergeRows rows); one thread per (row, 8 dims).
template <int kD>
__global__ void __launch_bounds__(kMergeRows * kD / 8)
attn_paged_merge(const __grid_constant__ PagedParams p, int C) {
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int b = blockIdx.x / p.Hkv, g = blockIdx.x % p.Hkv;
  const int rl = threadIdx.x % kMergeRows, c8 = threadIdx.x / kMergeRows;
  const int rt = blockIdx.y * kMergeRows + rl;
  const int n = p.ctx_lens[b];
  if (n < 0 || n > p.max_ctx || rt >= p.rowsT) return;
  const bool sh = shares(n, p.P, p.v_blk ? 0 : p.blk);
  const int T = tail_tiles(p, n);
  const int chunk = p.head[0], base = p.head[1];
  __nv_bfloat16* out =
      p.out + ((int64_t)(b * p.blk + rt / p.G) * p.Hq + g * p.G + rt % p.G) * kD + 8 * c8;
  const int w0 = base + p.Hkv * p.head[2 + b] + g * T;
  int t_first = 0, t_last = -1, p_first = 0, p_last = -1;
  if (T > 0) {
    t_first = w0 / chunk;
    t_last = (w0 + T - 1) / chunk;
    if (!sh && t_first == t_last) return;  // written by the main kernel
  } else if (!sh) {  // no key at all
    *reinterpret_cast<uint4*>(out) = make_uint4(0, 0, 0, 0);
    return;
  }
  const int unit = g * p.Tq + b / p.ns;
  const int rp = (b % p.ns) * p.rowsT + rt;
  if (sh) {
    p_first = unit * p.Kp / chunk;
    p_last = (unit * p.Kp + p.Kp - 1) / chunk;
  }
  auto tslot = [&](int c) {
    return tail_slot(p, b, g, c, c > t_first || w0 == c * chunk);
  };
  float M = -INFINITY, L = 0.f, acc[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) acc[e] = 0.f;
  bool bad = false;
  // pieces in tile order: the prefix, then the tail
  auto take = [&](float2 ml, const float4* o, int rows) {
    if (ml.x != ml.x) { bad = true; return; }
    if (ml.y == 0.f) return;  // no key of this row in the piece
    const float m = fmaxf(M, ml.x);
    // equal maxima (both -inf among them) keep weight 1: sums may be NaN then
    const float wa = M == m ? 1.f : ptx::ex2(M - m);
    const float wb = ml.x == m ? 1.f : ptx::ex2(ml.x - m);
    const float4 lo = o[(2 * c8) * rows], hi = o[(2 * c8 + 1) * rows];
    const float v[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    L = fmaf(wa, L, wb * ml.y);
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = fmaf(wa, acc[e], wb * v[e]);
    M = m;
  };
  for (int c = p_first; c <= p_last; ++c) {
    const int64_t at = (int64_t)(unit + c) * kRows;
    take(__ldcg(p.ml_p + at + rp), reinterpret_cast<const float4*>(p.o_p + at * kD) + rp, kRows);
  }
  for (int c = t_first; c <= t_last; ++c) {
    const int64_t at = (int64_t)tslot(c) * p.rowsT;
    take(__ldcg(p.ml_t + at + rt), reinterpret_cast<const float4*>(p.o_t + at * kD) + rt, p.rowsT);
  }
  if (bad) return;
  const int i = rt / p.G;
  const bool none = !p.v_blk && p.causal && n - p.blk + i + 1 <= 0;
  const float inv = 1.f / L;
  uint4 w;
  w.x = none ? 0u : ptx::pack_bf16x2(acc[0] * inv, acc[1] * inv);
  w.y = none ? 0u : ptx::pack_bf16x2(acc[2] * inv, acc[3] * inv);
  w.z = none ? 0u : ptx::pack_bf16x2(acc[4] * inv, acc[5] * inv);
  w.w = none ? 0u : ptx::pack_bf16x2(acc[6] * inv, acc[7] * inv);
  *reinterpret_cast<uint4*>(out) = w;
}

// -------------------------------------------------------------------- host

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  });
  return fn;
}

bool encode(CUtensorMap* m, const void* base, int rank, const cuuint64_t* dims,
            const cuuint64_t* strides, const cuuint32_t* box) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint32_t es[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(base), dims, strides, box,
            es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int sm_count(int device) {
  static int cache[64] = {0};
  if (device < 0 || device >= 64) return 0;
  if (!cache[device]) {
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, device) != cudaSuccess) return 0;
    cache[device] = n;
  }
  return cache[device];
}

// CTAs the workspace is sized for; a launch uses at most this many.
constexpr int kMaxCtas = 256;

struct Layout {
  int ns, Tq, Kp;
  int64_t head, ml_p, o_p, ml_t, o_t, total;  // byte offsets
};

Layout layout(const orthrus_paged_attn_args& a) {
  Layout y;
  const int rowsT = a.Hq / a.Hkv * a.blk;
  y.ns = kRows / rowsT;
  y.Tq = a.shared_prefix > 0 ? ceil_div(a.B, y.ns) : 0;
  y.Kp = ceil_div(a.shared_prefix, kTile);
  const int64_t ps = y.Tq ? (int64_t)a.Hkv * y.Tq + kMaxCtas : 0;
  const int64_t ts = a.shared_prefix > 0 ? (int64_t)a.B * a.Hkv + kMaxCtas : 2 * kMaxCtas;
  auto up = [](int64_t x) { return (x + 255) / 256 * 256; };
  y.head = 0;
  y.ml_p = up(4 * (2 + (int64_t)a.B));
  y.o_p = up(y.ml_p + ps * kRows * 8);
  y.ml_t = up(y.o_p + ps * kRows * a.D * 4);
  y.o_t = up(y.ml_t + ts * rowsT * 8);
  y.total = up(y.o_t + ts * rowsT * a.D * 4);
  return y;
}

template <int kD>
bool prepare(int device) {
  static bool done[64] = {false};
  if (device >= 0 && device < 64 && done[device]) return true;
  if (cudaFuncSetAttribute(attn_paged_kernel<kD>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           kSmemBytes) != cudaSuccess)
    return false;
  if (device >= 0 && device < 64) done[device] = true;
  return true;
}

}  // namespace

size_t paged_tc_workspace(const orthrus_paged_attn_args& a) { return (size_t)layout(a).total; }

int paged_tc_launch(const orthrus_paged_attn_args& a, cudaStream_t st) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return ORTHRUS_ECUDA;
  if (!(a.D == 64 ? prepare<64>(dev) : prepare<128>(dev))) return ORTHRUS_ECUDA;
  const int sms = sm_count(dev);
  if (sms <= 0) return ORTHRUS_ECUDA;
  const Layout y = layout(a);
  PagedParams p;
  const int G = a.Hq / a.Hkv;
  const cuuint64_t es = 2;
  {
    cuuint64_t dims[3] = {(cuuint64_t)a.D, (cuuint64_t)a.Hq, (cuuint64_t)a.B * a.blk};
    cuuint64_t str[2] = {a.D * es, (cuuint64_t)a.Hq * a.D * es};
    cuuint32_t box[3] = {64, (cuuint32_t)G, (cuuint32_t)a.blk};
    if (!encode(&p.tm_q, a.q, 3, dims, str, box)) return ORTHRUS_ECUDA;
    box[2] = (cuuint32_t)(y.ns * a.blk);
    if (!encode(&p.tm_qp, a.q, 3, dims, str, box)) return ORTHRUS_ECUDA;
  }
  {
    cuuint64_t dims[2] = {(cuuint64_t)a.D, (cuuint64_t)a.pages * a.Hkv * a.page_size};
    cuuint64_t str[1] = {a.D * es};
    cuuint32_t box[2] = {64, (cuuint32_t)(a.page_size < kTile ? a.page_size : kTile)};
    if (!encode(&p.tm_k, a.k_pages, 2, dims, str, box)) return ORTHRUS_ECUDA;
    if (!encode(&p.tm_v, a.v_pages, 2, dims, str, box)) return ORTHRUS_ECUDA;
  }
  if (a.k_blk) {
    cuuint64_t dims[3] = {(cuuint64_t)a.D, (cuuint64_t)a.Hkv, (cuuint64_t)a.B * a.blk};
    cuuint64_t str[2] = {a.D * es, (cuuint64_t)a.Hkv * a.D * es};
    cuuint32_t box[3] = {64, 1, (cuuint32_t)a.blk};
    if (!encode(&p.tm_kb, a.k_blk, 3, dims, str, box)) return ORTHRUS_ECUDA;
    if (!encode(&p.tm_vb, a.v_blk, 3, dims, str, box)) return ORTHRUS_ECUDA;
  } else {
    p.tm_kb = p.tm_k;  // never used
    p.tm_vb = p.tm_v;
  }
  char* ws = static_cast<char*>(a.workspace);
  p.ctx_lens = a.ctx_lens;
  p.table = a.page_table;
  p.v_pages = static_cast<const __nv_bfloat16*>(a.v_pages);
  p.v_blk = static_cast<const __nv_bfloat16*>(a.v_blk);
  p.out = static_cast<__nv_bfloat16*>(a.out);
  p.err = a.err;
  p.head = reinterpret_cast<int32_t*>(ws + y.head);
  p.ml_p = reinterpret_cast<float2*>(ws + y.ml_p);
  p.o_p = reinterpret_cast<float*>(ws + y.o_p);
  p.ml_t = reinterpret_cast<float2*>(ws + y.ml_t);
  p.o_t = reinterpret_cast<float*>(ws + y.o_t);
  p.B = a.B; p.Hq = a.Hq; p.Hkv = a.Hkv; p.G = G; p.blk = a.blk; p.rowsT = G * a.blk;
  p.ns = y.ns; p.Tq = y.Tq; p.Kp = y.Kp; p.P = a.shared_prefix;
  p.page_size = a.page_size; p.pages = a.pages; p.max_pages = a.max_pages;
  p.max_ctx = a.max_ctx; p.causal = a.mask_mode == ORTHRUS_CAUSAL_VERIFY;
  p.scale_log2 = (float)((double)a.scale * 1.4426950408889634);

  // no more CTAs than the most tiles there can be
  const int64_t most = (int64_t)a.Hkv * y.Tq * y.Kp +
                       (int64_t)a.Hkv * a.B * (ceil_div(a.max_ctx, kTile) + 1);
  const int64_t want = (most + kMinChunk - 1) / kMinChunk;
  int C = sms < kMaxCtas ? sms : kMaxCtas;
  if (want < C) C = (int)want;

  cudaLaunchAttribute pdl;
  pdl.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(C);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = st;
  cfg.attrs = &pdl;
  cfg.numAttrs = 1;
  cudaError_t e = a.D == 64 ? cudaLaunchKernelEx(&cfg, attn_paged_kernel<64>, p)
                            : cudaLaunchKernelEx(&cfg, attn_paged_kernel<128>, p);
  if (e != cudaSuccess) return ORTHRUS_ECUDA;
  cfg.gridDim = dim3(a.B * a.Hkv, ceil_div(p.rowsT, kMergeRows));
  cfg.blockDim = dim3(kMergeRows * a.D / 8);
  cfg.dynamicSmemBytes = 0;
  e = a.D == 64 ? cudaLaunchKernelEx(&cfg, attn_paged_merge<64>, p, C)
                : cudaLaunchKernelEx(&cfg, attn_paged_merge<128>, p, C);
  return e == cudaSuccess ? ORTHRUS_OK : ORTHRUS_ECUDA;
}

}  // namespace orthrus
