// Decode attention over prefixes that consecutive sequences share, joined with
// each sequence's own attention by log-sum-exp (the flash-style merge of the
// DKV abstract): kvsel_prefix_decode.
//
// For prefix g and KV head j the query rows of all its sequences and of the
// GQA group form one matrix Q [R][d], R = sequences * G, against one K and V:
// S = Q K^T, O = softmax(S) V. K and V are read once for all R rows, so a large
// R is bound by the tensor cores and a small one by HBM.
//
// Design (GB300):
//  * Work unit: a tile of 128 prefix tokens for a row unit of one (prefix, KV
//    head). The units are flattened (prefix, head, row unit, token tile); when
//    every prefix has as many tiles, each (prefix, head, row unit) segment gets
//    the same whole number of CTAs, else contiguous equal ranges. A CTA stores
//    unnormalised states (m, l, O) per row and segment; merge_prefix_kernel, a
//    programmatic dependent, joins a row's states with the sequence's own.
//  * Two streams, each with its own S (P overwrites it) and O in tensor memory,
//    keep the tensor pipe busy while the other's softmax runs. With many rows and
//    a long prefix a row unit is 256 rows, one row tile a stream, and both meet the
//    same K and V tile; else it is 128 rows and the streams take alternate token
//    tiles (rows_share_tiles).
//  * Pages need no re-layout: a page's K (or V) half is B rows of 128 bytes in
//    the 128-byte swizzle, so 1-D bulk copies of whole halves, stacked by block,
//    give the K-major B operand of S and the MN-major B operand of O.
//  * Warps: sixteen for the softmax (two threads a row, 64 columns each, their
//    maxima exchanged through shared memory), one each that fetches K and V, one
//    that issues the MMAs. It issues S(t + 1) right behind O(t) of the same stream: the tensor
//    pipe works in issue order, and the barrier of S(t + 1) counts every earlier
//    operation, so it also says that O(t) is complete.
//  * Softmax: x = S * scale (log2 units; a negative scale flips Q's signs when
//    it is loaded). The reference m moves, and O is rescaled in tensor memory,
//    only when a row's maximum passes it by more than 2^16: any reference gives
//    the same quotient, and p <= 2^16 stays far inside fp32 and bf16.
//  * P is split into bf16 high and low parts (about 16 bits, as in the sparse
//    decode): O's product takes two passes and keeps fp32-grade outputs; a
//    single bf16 P would be off by 2^-9 a weight.
//  * Every wait on a barrier is bounded; one that runs out latches
//    KVSEL_ERR_TIMEOUT, the CTA drains its copies and MMAs, frees its tensor
//    memory and returns. The tensor memory itself is taken when the stream's
//    earlier kernels are done; a kernel of another stream that shares the SM and
//    holds columns is waited for.
//
// Measured: 64 sequences x 32 heads (2 KV heads, d = 128) behind 131072 tokens,
// 124 us: 1.11 PFLOP/s of the formula's products, 1.66 with P's two passes (0.84
// of the measured bf16 rate); 5.5 us until the first S, 110 us of tiles (a
// 256 x 128 tile is 3700 cycles, 83 % of them the MMAs'), the rest the states'
// stores and the merge. 16 sequences x 32 heads (8 KV heads) behind 32768
// tokens, 64 rows a head: 34.1 us, 134 MB; the tiles stream at 7.2 TB/s for 18.5
// us between 5 us of start (plan, page table, first copies) and 11 us of end.
#include <climits>
#include <cmath>
#include <type_traits>

#include "kvsel_common.cuh"
#include "kvsel_internal.h"
#include "tcgen05.cuh"

namespace kvsel {
namespace {

constexpr int kTile = 128;             // tokens of a tile, and rows of an M tile
constexpr int kHalfBytes = kTile * 128;
constexpr int kMaxGrid = 160;          // partial-state capacity of the workspace
constexpr int kMaxK = 8, kMaxV = 8;    // stages
constexpr float kRescaleAt = 16.f;
constexpr int kSoftmaxWarps = 16;      // 2 streams x 2 column halves x 4 row quarters
constexpr int kThreads = (kSoftmaxWarps + 3) * 32;
constexpr int kMaxBlocks = kTile / 16; // blocks of a tile

struct PrefixArgs {
  const unsigned char* kv;
  int64_t n_pages;
  const int32_t* table;      // [P][mpb]
  const int32_t* lens;       // [P]
  const int32_t* first;      // [P + 1]
  const kvsel_bf16* q;
  float scale_log2;          // >= 0
  uint32_t q_flip;           // sign bits of a bf16 pair when the scale is negative
  const float* own_out;
  const float* own_lse;
  float* out;
  kvsel_bf16* out_bf16;
  float* lse;
  int4* plan;                // m, tiles per segment (or 0), CTAs in use, tiles
  int4* seq_info;            // [batch] of the sequence's prefix: first sequence, sequences (0: none),
                             // first tile, tiles per segment
  float4* partials;          // states by state_at: (m, l of each half, -), then O by four channels
  int batch, Hq, Hkv, G, B, P, mpb, k_stages, v_stages, unit_rows;
  int* err;
};

// A state of row `at` = row + CTA * row unit: quad 0 is (m, l, l, -), quad 1 + c
// channels 4 c to 4 c + 3. Four rows lie together, so that both the threads that
// write (a row each) and those that join meet whole 32-byte sectors.
template <int D>
__device__ __forceinline__ float4* state_at(float4* partials, int64_t at) {
  return partials + (at >> 2) * (4 * (D / 4 + 1)) + (at & 3);
}

struct Group {
  int seq0, ns, len, tt, ru, base;   // sequences, tokens, token tiles, row units per head, first tile
};

// Prefix g, `least` the largest first_seq up to g: a prefix whose sequences are
// out of range, out of order or shared with an earlier one is empty, so that
// the sequences of all prefixes are disjoint and ascend.
__device__ Group group_of(const PrefixArgs& a, int first, int end, int least, int len, bool report) {
  Group x;
  x.seq0 = first;
  x.len = len;
  x.ns = end - first;
  if (first < 0 || end > a.batch || end < first || first < least) {
    if (report) latch_error(a.err, KVSEL_ERR_BOUNDS);
    x.seq0 = max(0, least);
    x.ns = 0;
  }
  if (x.len < 0 || int64_t(x.len) > int64_t(a.mpb) * a.B) {
    if (report) latch_error(a.err, KVSEL_ERR_BOUNDS);
    x.len = x.len < 0 ? 0 : a.mpb * a.B;
  }
  x.tt = (x.len + kTile - 1) / kTile;
  x.ru = (x.ns * a.G + a.unit_rows - 1) / a.unit_rows;
  return x;
}

// What ranges of 128-row units that cross segments cost, in token tiles of a CTA: HBM
// gives about 95 CTAs (d = 128) their tiles at full speed, and a range in two segments
// stores and joins twice (about 4 tiles). Fewer, equal ranges (one segment each) that are
// longer than that are given up. Equal against crossing, us: 80 segments of 64 tiles (d = 128)
// 71.6 / 65.2, 96 of 32 (d = 64) 40.4 / 31.8; 104 of 32 (d = 128) 45.3 / 47.0, 72 of 64 (two CTAs
// each) 53.1 / 56.7.
__host__ __device__ constexpr int crossing_steps(int64_t total, int head_dim) {
  return int(total / (head_dim == 128 ? 95 : 150)) + 4;
}

// n i / parts for i <= parts <= kMaxGrid, in 32 bits.
__device__ __forceinline__ int share(int n, int i, int parts) {
  const int q = n / parts;
  return q * i + (n - q * parts) * i / parts;
}

// A CTA's share of one segment: token tiles [t0, t0 + n) of row unit u of KV
// head j of prefix g.
struct Portion {
  int g, j, u, t0, n, rows;
  Group x;
};

__device__ Portion portion_at(const PrefixArgs& a, const Group* groups, int pos, int end) {
  Portion p;
  int lo = 0, hi = a.P - 1;      // the last prefix whose first tile is <= pos
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (groups[mid].base <= pos) lo = mid; else hi = mid - 1;
  }
  p.g = lo;
  p.x = groups[lo];
  const int local = pos - p.x.base;
  const int seg = local / p.x.tt;
  p.t0 = local % p.x.tt;
  p.n = min(p.x.tt - p.t0, end - pos);
  p.j = seg / p.x.ru;
  p.u = seg % p.x.ru;
  p.rows = min(a.unit_rows, p.x.ns * a.G - p.u * a.unit_rows);
  return p;
}

// mbar_wait_bounded that also gives up when another role of the CTA has.
__device__ __forceinline__ bool wait_or_dead(uint64_t* bar, uint32_t parity, volatile int* dead, int* err) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_ns();
  for (uint32_t it = 0;; ++it) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((it & 15u) == 15u) {
      if (*dead) return false;
      if (global_ns() - t0 > kWaitLimitNs) {
        *dead = 1;
        latch_error(err, KVSEL_ERR_TIMEOUT);
        return false;
      }
    }
  }
}

__device__ __forceinline__ float ex2f_(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float lg2f_(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The position in a ring of S stages and the parity of its current round.
struct Ring {
  int st = 0;
  uint32_t ph = 0;
  __device__ __forceinline__ void next(int S) {
    if (++st == S) {
      st = 0;
      ph ^= 1u;
    }
  }
};

template <int D, bool ROWS>
__global__ void __launch_bounds__(kThreads, 1) prefix_kernel(PrefixArgs a) {
  constexpr int kHalves = D / 64;
  constexpr int kOpBytes = kHalves * kHalfBytes;       // one Q, K or V tile
  constexpr int kQTiles = ROWS ? 2 : 1;
  constexpr uint32_t kIdescS = idesc_bf16(128, kTile, false);
  constexpr uint32_t kIdescO = idesc_bf16(128, D, true);
  // no static shared memory stands before it: the operands' 1024-byte alignment costs nothing
  extern __shared__ __align__(1024) unsigned char smem[];
  const int SK = a.k_stages, SV = a.v_stages;
  unsigned char* q_s = smem;                                     // [kQTiles][tile]
  unsigned char* k_s = q_s + kQTiles * kOpBytes;                 // [SK][tile]
  unsigned char* v_s = k_s + SK * kOpBytes;                      // [SV][tile]
  float* max_s = reinterpret_cast<float*>(v_s + SV * kOpBytes);   // [2 streams][2 halves][128]
  uint64_t* kfull = reinterpret_cast<uint64_t*>(max_s + 4 * 128);
  uint64_t* kempty = kfull + kMaxK;
  uint64_t* vfull = kempty + kMaxK;
  uint64_t* vempty = vfull + kMaxV;
  uint64_t* sfull = vempty + kMaxV;                              // [2] S of a stream written
  uint64_t* pready = sfull + 2;                                  // [2][2] halves of P of a stream written
  uint64_t* odone = pready + 4;                                  // [2] O of a portion complete
  uint64_t* qfull = odone + 2;                                   // [2] Q of a portion in place
  uint64_t* left = qfull + 2;                                    // stream 1's m, l of a portion in left_s
  uint64_t* drained = left + 1;
  uint32_t* tmem_s = reinterpret_cast<uint32_t*>(drained + 1);
  volatile int* dead = reinterpret_cast<volatile int*>(tmem_s + 1);
  int* scan_s = reinterpret_cast<int*>(tmem_s + 2);              // smallest, largest tiles per segment; tiles
  float2* left_s = reinterpret_cast<float2*>(scan_s + 4);        // !ROWS: [2 halves][128] m, l
  Group* groups = reinterpret_cast<Group*>(left_s + (ROWS ? 0 : 256));   // [P]

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x, lane = tid & 31, warp = int(uniform(tid >> 5));
  if (warp == 1) {
    if (lane == 0) {
      for (int i = 0; i < SK; ++i) {
        mbar_init(&kfull[i], 1);
        mbar_init(&kempty[i], 1);
      }
      for (int i = 0; i < SV; ++i) {
        mbar_init(&vfull[i], 1);
        mbar_init(&vempty[i], 1);
      }
      for (int i = 0; i < 2; ++i) {
        mbar_init(&sfull[i], 1);
        mbar_init(&pready[2 * i], 8);
        mbar_init(&pready[2 * i + 1], 8);
        mbar_init(&odone[i], 1);
        mbar_init(&qfull[i], 8);
      }
      mbar_init(left, 8);
      mbar_init(drained, 1);
      *dead = 0;
      fence_barrier_init();
    }
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // Not before the wait: the allocation has no time limit, and while this grid holds an SM's
  // columns, a kernel before it in the stream that still needs some could never end.
  if (warp == 2) {
    tmem_alloc(tmem_s, 512);
    tmem_relinquish();
  }

  if (warp == 0) {
    // the prefixes' tiles: prefix sum, and whether all segments are alike
    int carry = 0, lo = INT_MAX, hi = 0, least = 0;
    for (int g0 = 0; g0 < a.P; g0 += 32) {
      const int g = g0 + lane;
      Group x{};
      int first = 0, end = 0, len = 0;
      if (g < a.P) {
        first = a.first[g];
        end = a.first[g + 1];
        len = a.lens[g];
      }
      int top = max(least, g < a.P ? first : 0);
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, top, off);   // every lane takes part
        if (lane >= off) top = max(top, y);
      }
      if (g < a.P) x = group_of(a, first, end, top, len, blockIdx.x == 0);
      least = __shfl_sync(0xffffffffu, top, 31);
      const int mine = a.Hkv * x.ru * x.tt;
      if (mine > 0) {
        lo = min(lo, x.tt);
        hi = max(hi, x.tt);
      }
      int sum = mine;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, sum, off);
        if (lane >= off) sum += y;
      }
      if (g < a.P) {
        x.base = carry + sum - mine;
        groups[g] = x;
      }
      carry += __shfl_sync(0xffffffffu, sum, 31);
    }
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    if (lane == 0) {
      scan_s[0] = lo;
      scan_s[1] = hi;
      scan_s[2] = carry;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = uniform(*tmem_s);      // S of streams 0, 1 at columns 0, 128; O at 256, 256 + D

  const int total = scan_s[2];
  const int nbu = scan_s[0] == scan_s[1] ? scan_s[1] : 0;
  const int n_seg = nbu > 0 ? total / nbu : 0;
  int m = n_seg > 0 && n_seg <= int(gridDim.x) ? min(int(gridDim.x) / n_seg, nbu) : 0;
  if (!ROWS && m > 0 && (nbu + m - 1) / m > crossing_steps(total, D)) m = 0;
  const int A = m > 0 ? n_seg * m : min(int(gridDim.x), max(1, total));
  if (blockIdx.x == 0) {       // what the merge needs
    if (tid == 0) *a.plan = make_int4(m, nbu, A, total);
    for (int b = tid; b < a.batch; b += kThreads) {
      int lo = 0, hi = a.P - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (groups[mid].seq0 <= b) lo = mid; else hi = mid - 1;
      }
      const Group& x = groups[lo];
      const bool in = x.seq0 <= b && b < x.seq0 + x.ns;
      a.seq_info[b] = in ? make_int4(x.seq0, x.ns, x.base, x.tt) : make_int4(0, 0, 0, 0);
    }
  }
  int g0 = 0, g1 = 0;
  if (int(blockIdx.x) < A && total > 0) {
    if (m > 0) {
      const int k = int(blockIdx.x) / m, part = int(blockIdx.x) % m;
      g0 = k * nbu + share(nbu, part, m);
      g1 = k * nbu + share(nbu, part + 1, m);
    } else {
      g0 = share(total, blockIdx.x, A);
      g1 = share(total, blockIdx.x + 1, A);
    }
  }

  if (warp < kSoftmaxWarps) {
    // ---------------- softmax: two threads a row, half the columns each ----------------
    const int i = warp >> 3, half = (warp >> 2) & 1, quad = warp & 3;   // stream, column half, rows 32 quad ..
    const int r = quad * 32 + lane;
    const uint32_t lanes = uint32_t(quad * 32) << 16;
    const uint32_t sb = tmem + i * 128 + half * 64 + lanes, ob = tmem + 256 + i * D + half * (D / 2) + lanes;
    const int join = 1 + i * 4 + quad;           // named barrier of the two halves
    // Written again only after the other half has read it: the next S needs both halves' P.
    float* my_max = max_s + (i * 2 + half) * 128 + r;
    const float2 sc = make_float2(a.scale_log2, a.scale_log2);
    uint32_t n_s = 0, n_o = 0, n_o1 = 0;
    bool ok = true;
    for (int pos = g0; ok && pos < g1;) {
      const int here = pos;
      int n, left_over, rows;                    // token tiles, tokens from the first on, rows of this row tile
      {
        const Portion p = portion_at(a, groups, here, g1);
        pos += p.n;
        n = p.n;
        left_over = p.x.len - p.t0 * kTile - half * 64;
        rows = p.rows - (ROWS ? i * 128 : 0);
        if (rows <= 0) continue;
        if (ROWS || i == 0) {
          const int rr = p.u * a.unit_rows + (ROWS ? i * 128 : 0) + r;   // of the (prefix, KV head)
          const uint4* src = reinterpret_cast<const uint4*>(
              a.q + (int64_t(p.x.seq0 + rr / a.G) * a.Hq + int64_t(p.j) * a.G + rr % a.G) * D);
#pragma unroll
          for (int e = 0; e < D / 16; ++e) {
            const int c = half * (D / 16) + e;
            uint4 v = make_uint4(0, 0, 0, 0);
            if (r < rows) v = src[c];
            v.x ^= a.q_flip; v.y ^= a.q_flip; v.z ^= a.q_flip; v.w ^= a.q_flip;
            *reinterpret_cast<uint4*>(q_s + (ROWS ? i * kOpBytes : 0) + (c >> 3) * kHalfBytes + r * 128 +
                                      (((c & 7) ^ (r & 7)) << 4)) = v;
          }
          fence_proxy_async();
          __syncwarp();
          if (lane == 0) mbar_arrive(&qfull[i]);
        }
      }
      const bool live = quad * 32 < rows;          // this warp has rows
      const int first = ROWS ? 0 : i, step = ROWS ? 1 : 2;
      float mref = -INFINITY, l = 0.f;
      for (int t = first; t < n; t += step, ++n_s) {
        ok = __all_sync(0xffffffffu, wait_or_dead(&sfull[i], n_s & 1u, dead, a.err));
        if (!ok) {
          // the other half may have seen the phase complete: it must not wait for this one
          if (live) asm volatile("barrier.arrive %0, 64;" ::"r"(join) : "memory");
          break;
        }
        tc_fence_after();
        if (!live) {
          if (lane < 2) mbar_arrive(&pready[2 * i + lane]);
          continue;
        }
        const int cnt = left_over - t * kTile;     // of this thread's 64 columns
        uint32_t s[4][16];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld16(sb + c * 16, s[c]);
        tmem_wait_ld();
        float mx = -INFINITY;
        if (cnt >= 64) {
          float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int e = 0; e < 64; e += 8)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              m4[k] = fmaxf(m4[k], fmaxf(__uint_as_float(s[e >> 4][(e & 15) + 2 * k]),
                                         __uint_as_float(s[e >> 4][(e & 15) + 2 * k + 1])));
          mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
        } else {
#pragma unroll
          for (int e = 0; e < 64; ++e)
            if (e < cnt) mx = fmaxf(mx, __uint_as_float(s[e >> 4][e & 15]));
        }
        *my_max = mx;
        asm volatile("barrier.sync %0, 64;" ::"r"(join) : "memory");
        mx = fmaxf(mx, my_max[half ? -128 : 128]);
        const float mt = mx * a.scale_log2;
        if (t == first) {
          mref = mt;
        } else if (__any_sync(0xffffffffu, mt > mref + kRescaleAt)) {
          const float mn = mt > mref + kRescaleAt ? mt : mref;
          const float alpha = mn == -INFINITY ? 1.f : ex2f_(mref - mn);
          mref = mn;
          l *= alpha;
#pragma unroll 1
          for (int c = 0; c < D / 16; ++c) {
            uint32_t o[8];
            tmem_ld8(ob + c * 8, o);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
            tmem_st8(ob + c * 8, o);
          }
        }
        const float mu = mref == -INFINITY ? 0.f : mref;
        const float2 neg = make_float2(-mu, -mu);
        float2 l2 = make_float2(0.f, 0.f);
        auto weights = [&](auto masked) {          // whole tiles pay nothing for the mask
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t hi[8], lo[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              float2 x = make_float2(__uint_as_float(s[c][2 * e]), __uint_as_float(s[c][2 * e + 1]));
              x = fma2(x, sc, neg);
              if constexpr (decltype(masked)::value) {   // masked here: a scale of 0 times an infinity is no mask
                if (c * 16 + 2 * e >= cnt) x.x = -INFINITY;
                if (c * 16 + 2 * e + 1 >= cnt) x.y = -INFINITY;
              }
              const float2 pv = make_float2(ex2f_(x.x), ex2f_(x.y));
              l2 = add2(l2, pv);
              hi[e] = pack_bf16x2(pv.x, pv.y);
              const float2 rest = add2(pv, make_float2(-bf16lo(hi[e]), -bf16hi(hi[e])));
              lo[e] = pack_bf16x2(rest.x, rest.y);
            }
            // a k step's high words take its first 8 columns, the low words the others
            // (one store where the registers allow it: 3 % of the call with many rows)
            if constexpr (ROWS) {
              tmem_st16(sb + c * 16, hi, lo);
            } else {
              tmem_st8(sb + c * 16, hi);
              tmem_st8(sb + c * 16 + 8, lo);
            }
            if (c & 1) {
              tmem_wait_st();
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(&pready[2 * i + (c >> 1)]);
            }
          }
        };
        if (cnt >= 64) weights(std::false_type{});
        else weights(std::true_type{});
        l += l2.x + l2.y;
      }
      if (!ok) break;
      float w0 = 1.f, w1 = 0.f;                    // what O of stream 0 and 1 count in the state
      if (!ROWS && n > 1) {
        // stream 1 leaves its m and l, stream 0 joins the two states of a row. Stream 1
        // cannot come here again before stream 0 has: its next S needs stream 0's next Q
        if (i == 1) {
          left_s[half * 128 + r] = make_float2(mref, l);
          __syncwarp();
          if (lane == 0) mbar_arrive(left);
          continue;
        }
        ok = __all_sync(0xffffffffu, wait_or_dead(left, n_o1 & 1u, dead, a.err));
        if (!ok) break;
        const float2 other = left_s[half * 128 + r];
        const float mn = fmaxf(mref, other.x);
        const float mu = mn == -INFINITY ? 0.f : mn;
        w0 = ex2f_(mref - mu);
        w1 = ex2f_(other.x - mu);
        mref = mn;
        l = l * w0 + other.y * w1;
        ok = __all_sync(0xffffffffu, wait_or_dead(&odone[1], n_o1++ & 1u, dead, a.err));
        if (!ok) break;
      } else if (!ROWS && i == 1) {
        continue;                                  // one tile: stream 0's
      }
      ok = __all_sync(0xffffffffu, wait_or_dead(&odone[i], n_o++ & 1u, dead, a.err));
      if (!ok) break;
      tc_fence_after();
      if (live) {
        const Portion p = portion_at(a, groups, here, g1);
        float4* dst = state_at<D>(a.partials, int64_t(p.x.seq0) * a.Hq + int64_t(p.j) * p.x.ns * a.G + p.u * a.unit_rows +
                                              (ROWS ? i * 128 : 0) + r + int64_t(blockIdx.x) * a.unit_rows);
        if (r < rows) {
          if (half == 0) dst->x = mref;
          (half ? dst->z : dst->y) = l;
        }
        dst += 4 * (1 + half * (D / 8));
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[16], o1[16];
          tmem_ld16(ob + c * 16, o);
          if (!ROWS && n > 1) tmem_ld16(ob + D + c * 16, o1);
          tmem_wait_ld();
          if (!ROWS && n > 1) {
#pragma unroll
            for (int e = 0; e < 16; ++e)
              o[e] = __float_as_uint(__uint_as_float(o[e]) * w0 + __uint_as_float(o1[e]) * w1);
          }
          if (r < rows) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              reinterpret_cast<uint4*>(dst)[4 * (c * 4 + e)] =
                  make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
          }
        }
      }
      tc_fence_before();
    }
  } else if (warp < kSoftmaxWarps + 2) {
    // ---------------- producers, one for K and one for V: whole page halves by 1-D
    // bulk copies, issued by one thread (lanes that issue in turn cost three times as
    // many cycles a copy) ----------------
    if (elect_one()) {
      const int which = warp - kSoftmaxWarps, S = which ? SV : SK;
      uint64_t* full = which ? vfull : kfull;
      uint64_t* empty = which ? vempty : kempty;
      unsigned char* ring_s = which ? v_s : k_s;
      Ring ring;
      uint32_t issued = 0;
      bool ok = true;
      const int per_stage = kTile / a.B;
      const uint32_t piece = uint32_t(a.B) * 128;                   // one half of one block
      const int64_t head_bytes = int64_t(4) * a.B * D;              // K then V of one head
      for (int pos = g0; ok && pos < g1;) {
        const Portion p = portion_at(a, groups, pos, g1);
        pos += p.n;
        // blocks [n0, n1) of the prefix, per_stage at a time
        const int n0 = p.t0 * (kTile / a.B);
        const int n1 = min((p.t0 + p.n) * (kTile / a.B), (p.x.len + a.B - 1) / a.B);
        const int32_t* table = a.table + int64_t(p.g) * a.mpb;
        const unsigned char* src = a.kv + p.j * head_bytes + which * (2 * a.B * D);
        int page[kMaxBlocks];                                       // a stage's blocks, read a stage ahead
        auto load_pages = [&](int n) {
#pragma unroll
          for (int b = 0; b < kMaxBlocks; ++b)
            if (b < per_stage && n + b < n1) page[b] = table[n + b];
        };
        load_pages(n0);
        for (int n = n0; n < n1; n += per_stage) {
          const int have = min(per_stage, n1 - n);
          unsigned char* dst = ring_s + ring.st * kOpBytes;
          ok = wait_or_dead(&empty[ring.st], ring.ph ^ 1u, dead, a.err);
          if (!ok) break;
          mbar_arrive_expect_tx(&full[ring.st], uint32_t(have) * kHalves * piece);
#pragma unroll
          for (int b = 0; b < kMaxBlocks; ++b) {
            if (b >= have) break;
            int64_t pg = page[b];
            if (pg < 0 || pg >= a.n_pages) {
              latch_error(a.err, KVSEL_ERR_BOUNDS);                 // any page stands in: the prefix's result is void
              pg = 0;
            }
            const unsigned char* from = src + pg * a.Hkv * head_bytes;
#pragma unroll
            for (int h = 0; h < kHalves; ++h)
              bulk_load(dst + h * kHalfBytes + b * piece, from + h * piece, piece, &full[ring.st]);
          }
          load_pages(n + per_stage);
          ring.next(S);
          ++issued;
        }
      }
      // copies still in flight (a role gave up): their last phases
      if (*dead)
        for (uint32_t i = issued > uint32_t(S) ? issued - S : 0; i < issued; ++i)
          (void)mbar_wait_bounded(&full[i % S], (i / S) & 1u);
    }
    __syncwarp();
  } else {
    // ---------------- MMA: one thread waits and issues (a warp that reconverges
    // around every wait and issue spends more cycles on that than on both). The
    // tensor pipe's queue is short: what the thread does besides issuing stands
    // where a full burst is queued in front of it. ----------------
    if (elect_one()) {
    Ring kr, vr;
    uint32_t n_q[2] = {0, 0}, n_p[2] = {0, 0};
    bool ok = true;
    const uint32_t q_lo = smem_u32(q_s) >> 4, k_lo = smem_u32(k_s) >> 4, v_lo = smem_u32(v_s) >> 4;
    constexpr uint64_t kDescK = smem_desc_sw128(0, 16, 1024), kDescV = smem_desc_sw128(0, kHalfBytes, 1024);
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      ok = wait_or_dead(bar, parity, dead, a.err);
      return ok;
    };
    // two barriers at the price of one where both are done
    auto wait_two = [&](uint64_t* bar, uint32_t parity, uint64_t* bar2, uint32_t parity2) {
      const bool a1 = mbar_try_wait(bar, parity), a2 = mbar_try_wait(bar2, parity2);
      if (a1 && a2) return true;
      return wait(bar, parity) && wait(bar2, parity2);
    };
    // S = Q K^T of stream i and the K stage that is next (descriptors count 16 bytes)
    auto issue_s = [&](auto stream) {
      constexpr int i = decltype(stream)::value;
      const uint64_t qd = kDescK + (q_lo + (ROWS ? i * (kOpBytes >> 4) : 0)), kd = kDescK + (k_lo + kr.st * (kOpBytes >> 4));
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        constexpr uint32_t kHalf = kHalfBytes >> 4;
        const uint32_t off = (ks / 4) * kHalf + (ks % 4) * 2;
        mma_ss(tmem + i * 128, qd + off, kd + off, kIdescS, ks > 0);
      }
      mma_commit(&sfull[i]);
    };
    auto next_k = [&]() {
      mma_commit(&kempty[kr.st]);
      kr.next(SK);
    };
    // V rows of the last 16 tokens past the prefix's end: those tokens' weights
    // are 0, and 0 * (whatever the page holds) must be 0.
    auto clear_tail = [&](int cnt) {
      if (cnt >= kTile || (cnt & 15) == 0) return;
      unsigned char* v = v_s + vr.st * kOpBytes;
      for (int row = cnt; row & 15; ++row)
        for (int c = 0; c < kHalves * 8; ++c)
          *reinterpret_cast<uint4*>(v + (c >> 3) * kHalfBytes + row * 128 + (c & 7) * 16) = make_uint4(0, 0, 0, 0);
      fence_proxy_async();
    };
    auto next_v = [&]() {
      mma_commit(&vempty[vr.st]);
      vr.next(SV);
    };
    // O += P V as soon as each half of P is there: k steps 0, 1, 4, 5, then 2, 3, 6, 7.
    // `first` and `second` wait for each.
    auto issue_o = [&](auto stream, int cnt, bool accumulate, auto first, auto second) {
      constexpr int i = decltype(stream)::value;
      const uint32_t ob = tmem + 256 + i * D, pb = tmem + i * 128;
      const uint64_t v0 = kDescV + (v_lo + vr.st * (kOpBytes >> 4));
#pragma unroll
      for (int part = 0; part < 2; ++part) {
        if (part == 0 ? !first() : !second()) return false;
        tc_fence_after();
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int ks = (e >> 1) * 4 + part * 2 + (e & 1);
          if (ks * 16 < cnt) {
            mma_ts(ob, pb + ks * 16, v0 + ks * (2048 >> 4), kIdescO, ks > 0 || accumulate);
            mma_ts(ob, pb + ks * 16 + 8, v0 + ks * (2048 >> 4), kIdescO, true);
          }
        }
      }
      return true;
    };
    const std::integral_constant<int, 0> st0;
    const std::integral_constant<int, 1> st1;
    for (int pos = g0; ok && pos < g1;) {
      int n, left_over, rows;                       // token tiles, tokens from the first on
      {
        const Portion p = portion_at(a, groups, pos, g1);
        n = p.n;
        left_over = p.x.len - p.t0 * kTile;
        rows = p.rows;
      }
      pos += n;
      if (!wait(&qfull[0], n_q[0]++ & 1u)) break;
      if (!wait(&kfull[kr.st], kr.ph)) break;
      if (ROWS) {
        // both row tiles meet the same K and V tile
        const bool two = rows > 128;
        if (two && !wait(&qfull[1], n_q[1]++ & 1u)) break;
        issue_s(st0);
        if (two) issue_s(st1);
        next_k();
        for (int t = 0;; ++t, left_over -= kTile) {
          const bool last = t == n - 1;
          const uint32_t p0 = n_p[0]++ & 1u;
          if (!issue_o(st0, left_over, t > 0,
                       [&]() {
                         if (!wait_two(&vfull[vr.st], vr.ph, &pready[0], p0)) return false;
                         clear_tail(left_over);
                         return true;
                       },
                       [&]() { return last ? wait(&pready[1], p0) : wait_two(&pready[1], p0, &kfull[kr.st], kr.ph); }))
            break;
          if (last) mma_commit(&odone[0]);
          else issue_s(st0);
          if (two) {
            const uint32_t p1 = n_p[1]++ & 1u;
            if (!issue_o(st1, left_over, t > 0, [&]() { return wait(&pready[2], p1); },
                         [&]() { return wait(&pready[3], p1); }))
              break;
            if (last) mma_commit(&odone[1]);
            else issue_s(st1);
          }
          next_v();
          if (last) break;
          next_k();
        }
      } else {
        // the streams take alternate token tiles of the same rows
        issue_s(st0);
        next_k();
        if (n > 1) {
          if (!wait(&kfull[kr.st], kr.ph)) break;
          issue_s(st1);
          next_k();
        }
        auto tile = [&](auto stream, int t) {
          constexpr int i = decltype(stream)::value;
          const uint32_t p = n_p[i]++ & 1u;
          // bound by the copies: nothing waits for the next ones before O's MMAs are issued
          if (!issue_o(stream, left_over, t > 1,
                       [&]() {
                         if (!wait_two(&vfull[vr.st], vr.ph, &pready[2 * i], p)) return false;
                         clear_tail(left_over);
                         return true;
                       },
                       [&]() { return wait(&pready[2 * i + 1], p); }))
            return false;
          next_v();
          left_over -= kTile;
          if (t + 2 >= n) {
            mma_commit(&odone[i]);
            return true;
          }
          if (!wait(&kfull[kr.st], kr.ph)) return false;
          issue_s(stream);
          next_k();
          return true;
        };
        for (int t = 0; t < n; t += 2)
          if (!tile(st0, t) || (t + 1 < n && !tile(st1, t + 1))) break;
      }
    }
    // nothing of this thread is in flight when the tensor memory is freed
    mma_commit(drained);
    (void)mbar_wait_bounded(drained, 0u);
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// The states that the prefix kernel's CTAs left for a row and the sequence's own,
// joined by log-sum-exp. A CTA owns four rows that lie together in `partials`; a
// warp reads eight quads of them (64 bytes a quad), D / 32 warps a state, and the
// kSplit groups of such warps take the states in turn, five at a time, to be
// joined in shared memory. The call is bound by the latency of its dependent
// reads (the row's prefix, then the states): index arithmetic is 32-bit, done once.
constexpr int kSplit = 4;

template <int D>
__global__ void __launch_bounds__(kSplit * D) merge_prefix_kernel(PrefixArgs a) {
  constexpr int kQuads = D / 4, kChunk = 5;
  __shared__ int row_s[4], first_s[4], n_s[4];
  __shared__ float2 ml_s[kSplit][4];
  __shared__ float4 o_s[kSplit][kQuads][4];
  const int sub = threadIdx.x & 3, quad = (threadIdx.x >> 2) % kQuads, part = threadIdx.x / D;
  const int rows = a.batch * a.Hq, base = blockIdx.x * 4 + sub;     // base: the row's place in `partials`
  const bool live = base < rows;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // one thread a row looks up where its states are: every warp reading the plan's one
  // line would queue at it (1.5 us of a call with 512 such CTAs)
  if (threadIdx.x < 4) {
    int row = base, first = 0, n = 0;
    const int4 x = __ldcg(a.seq_info + min(base, rows - 1) / a.Hq), plan = __ldcg(a.plan);
    if (live && x.y > 0 && x.w > 0) {
      // rows of a prefix are ordered (KV head, sequence, head of the group)
      const int per_head = x.y * a.G, rem = base - x.x * a.Hq;
      const int j = rem / per_head, rr = rem - j * per_head, sq = rr / a.G;
      row = (x.x + sq) * a.Hq + j * a.G + rr - sq * a.G;
      const int shift = a.unit_rows == 256 ? 8 : 7;
      const int ru = (per_head + a.unit_rows - 1) >> shift;
      const int start = x.z + (j * ru + (rr >> shift)) * x.w;
      if (plan.x > 0) {
        first = start / plan.y * plan.x;
        n = plan.x;
      } else {
        first = int(((uint64_t(start) + 1) * uint32_t(plan.z) - 1) / uint32_t(plan.w));
        n = int(((uint64_t(start) + x.w) * uint32_t(plan.z) - 1) / uint32_t(plan.w)) - first + 1;
      }
    }
    row_s[sub] = row;
    first_s[sub] = first;
    n_s[sub] = n;
  }
  __syncthreads();
  const int row = row_s[sub], first = first_s[sub], n = n_s[sub];
  float own_m = -INFINITY;                   // joined last: its reads overlap the states'
  float4 own = make_float4(0.f, 0.f, 0.f, 0.f);
  if (part == 0 && live && a.own_lse) {
    own_m = a.own_lse[row] * 1.4426950408889634f;
    own = reinterpret_cast<const float4*>(a.own_out + int64_t(row) * D)[quad];
  }
  float M = -INFINITY, L = 0.f;              // log2 units
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  const int64_t step = int64_t(a.unit_rows) * (kQuads + 1);
  const float4* st = state_at<D>(a.partials, base) + (first + part) * step;
  for (int i0 = part; i0 < n; i0 += kSplit * kChunk) {
    float mi[kChunk], li[kChunk];
    float4 oi[kChunk];
#pragma unroll
    for (int k = 0; k < kChunk; ++k, st += kSplit * step) {
      mi[k] = -INFINITY;
      li[k] = 0.f;
      oi[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i0 + k * kSplit < n) {
        const float4 ml = __ldcg(st);
        mi[k] = ml.x;
        li[k] = ml.y + ml.z;
        oi[k] = __ldcg(st + 4 * (1 + quad));
      }
    }
    float mc = M;
#pragma unroll
    for (int k = 0; k < kChunk; ++k) {
      if (li[k] != li[k]) mi[k] = fmaxf(mi[k], 0.f);       // scores that were NaN: the row is NaN
      mc = fmaxf(mc, mi[k]);
    }
    if (mc == -INFINITY) continue;
    const float rs = M == -INFINITY ? 0.f : ex2f_(M - mc);
    L *= rs;
    acc = make_float4(acc.x * rs, acc.y * rs, acc.z * rs, acc.w * rs);
#pragma unroll
    for (int k = 0; k < kChunk; ++k) {
      if (mi[k] != -INFINITY) {
        const float w = ex2f_(mi[k] - mc);
        L += w * li[k];
        acc.x += w * oi[k].x;
        acc.y += w * oi[k].y;
        acc.z += w * oi[k].z;
        acc.w += w * oi[k].w;
      }
    }
    M = mc;
  }
  if (quad == 0) ml_s[part][sub] = make_float2(M, L);
  o_s[part][quad][sub] = acc;
  __syncthreads();                           // also: out and lse may be own_out and own_lse
  if (part != 0 || !live) return;
  float mx = own_m;
#pragma unroll
  for (int w = 0; w < kSplit; ++w) mx = fmaxf(mx, ml_s[w][sub].x);
  const float mu = mx == -INFINITY ? 0.f : mx;
  L = 0.f;
  acc = make_float4(0.f, 0.f, 0.f, 0.f);
  if (own_m != -INFINITY) {                  // a sequence with nothing of its own yet adds nothing
    L = ex2f_(own_m - mu);
    acc = make_float4(L * own.x, L * own.y, L * own.z, L * own.w);
  }
#pragma unroll
  for (int w = 0; w < kSplit; ++w) {
    const float2 ml = ml_s[w][sub];
    if (ml.x == -INFINITY) continue;
    const float f = ex2f_(ml.x - mu);
    const float4 v = o_s[w][quad][sub];
    L += f * ml.y;
    acc.x += f * v.x;
    acc.y += f * v.y;
    acc.z += f * v.z;
    acc.w += f * v.w;
  }
  const float4 res = L == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f)
                              : make_float4(acc.x / L, acc.y / L, acc.z / L, acc.w / L);
  reinterpret_cast<float4*>(a.out + int64_t(row) * D)[quad] = res;
  if (a.out_bf16)
    reinterpret_cast<uint2*>(a.out_bf16 + int64_t(row) * D)[quad] =
        make_uint2(pack_bf16x2(res.x, res.y), pack_bf16x2(res.z, res.w));
  if (quad == 0) a.lse[row] = L == 0.f ? -INFINITY : (mx + lg2f_(L)) * 0.6931471805599453f;
}

template <int D, bool ROWS>
cudaError_t launch_t(PrefixArgs a, cudaStream_t s) {
  constexpr int kQTiles = ROWS ? 2 : 1;
  const size_t op = size_t(D / 64) * kHalfBytes;
  const size_t rest = 4 * 128 * 4 + (2 * kMaxK + 2 * kMaxV + 12) * 8 + 8 + 16 + (ROWS ? 0 : 256 * 8) + size_t(a.P) * sizeof(Group);
  const size_t room = size_t(max_smem_optin());
  if (room < rest + (kQTiles + 2) * op) return cudaErrorInvalidConfiguration;
  // K is free as soon as S is computed, V only after the softmax: the odd tile is V's
  const int tiles = int((room - rest - kQTiles * op) / op);
  a.k_stages = std::min(kMaxK, tiles / 2);
  a.v_stages = std::min(kMaxV, tiles - a.k_stages);
  a.unit_rows = ROWS ? 256 : 128;
  const int grid = std::min(kMaxGrid, sm_count());
  // more than half of an SM's shared memory: CTAs of two such kernels (calls on two
  // streams) never share an SM, so neither's allocation of tensor memory waits for the other's
  const size_t smem = std::max(rest + (kQTiles + size_t(a.k_stages) + a.v_stages) * op, size_t(120) * 1024);
  auto fn = prefix_kernel<D, ROWS>;
  cudaError_t e = ensure_smem(reinterpret_cast<const void*>(fn), int(smem));
  if (e != cudaSuccess) return e;
  e = launch_pdl(fn, dim3(unsigned(grid)), dim3(kThreads), smem, s, a);
  count_launch();
  if (e != cudaSuccess) return e;
  e = launch_pdl(merge_prefix_kernel<D>, dim3(unsigned(a.batch * a.Hq + 3) / 4), dim3(kSplit * D), 0, s, a);
  count_launch();
  return e;
}

// Whether units of 256 rows, whose two row tiles share each K and V tile, beat
// units of 128 rows, whose streams take alternate token tiles. The first leave
// fewer, longer ranges a CTA and twice the states (about 3 us more to store and
// to join); the second may leave SMs idle (16 segments on 152) and read each
// tile once a unit. Cost in hundredths of a 128 x 128 tile (1 us at d = 128),
// from the sizes that the host knows: the rows a prefix on average and the longest
// prefix the table holds; fitted to calls of 130 to 1024 rows a KV head.
// Measured, us (256 rows a unit / 128):
//   d = 128: 2 heads x 1024 rows, 131072 tokens 123.0 / 131.7, 32768 tokens 44.4 / 43.6,
//            8192 tokens 25.9 / 22.8; 4 x 384, 32768 44.3 / 37.4; 8 x 256, 32768 48.5 / 46.3;
//            8 x 160, 32768 42.6 / 45.2; 8 x 64, 32768 36.2 / 33.4
//   d = 64:  8 x 512, 16384 35.9 / 42.9; 1 x 1024, 65536 35.1 / 37.1; 1 x 640, 20000 21.2 / 17.8
bool rows_share_tiles(const PrefixArgs& a, int head_dim) {
  const int64_t rows = (int64_t(a.batch) * a.G + a.P - 1) / a.P;
  if (rows <= kTile) return false;
  const int64_t tiles = (int64_t(a.mpb) * a.B + kTile - 1) / kTile, ctas = std::min(kMaxGrid, sm_count());
  const auto steps = [&](int unit) -> int64_t {   // token tiles of the longest range
    const int64_t seg = int64_t(a.Hkv) * a.P * ((rows + unit - 1) / unit);
    if (seg > ctas) return (seg * tiles + ctas - 1) / ctas;
    const int64_t equal = (tiles + ctas / seg - 1) / (ctas / seg);
    return unit == 128 ? std::min<int64_t>(equal, crossing_steps(seg * tiles, head_dim)) : equal;
  };
  // two row tiles, the second's share of live rows where it is the only unit's
  const int64_t pair = rows >= 2 * kTile ? 200 : 155 + 65 * (rows - kTile) / kTile;
  return head_dim == 128 ? steps(256) * pair + 300 < steps(128) * 100
                         : steps(256) * pair * 3 / 4 + 200 < steps(128) * 95;
}

size_t meta_bytes(const kvsel_problem& p) {
  return 16 + size_t(p.batch) * 16;
}

}  // namespace

size_t prefix_decode_ws_bytes(const kvsel_problem& p) {
  const size_t rows = size_t(p.batch) * p.n_qheads + size_t(kMaxGrid) * 256;
  return meta_bytes(p) + (rows + 3) / 4 * 4 * (p.head_dim + 4) * 4;
}

cudaError_t launch_prefix_decode(const kvsel_problem& p, const kvsel_prefix& x, const kvsel_bf16* q,
                                 float softmax_scale, const float* own_out, const float* own_lse, float* out,
                                 kvsel_bf16* out_bf16, float* lse, void* ws, int* err, cudaStream_t s) {
  PrefixArgs a{};
  a.kv = reinterpret_cast<const unsigned char*>(x.kv_pages);
  a.n_pages = x.n_pages; a.table = x.prefix_table; a.lens = x.prefix_lens; a.first = x.first_seq;
  a.q = q;
  a.scale_log2 = std::fabs(softmax_scale) * 1.4426950408889634f;
  a.q_flip = std::signbit(softmax_scale) ? 0x80008000u : 0u;
  a.own_out = own_out; a.own_lse = own_lse;
  a.out = out; a.out_bf16 = out_bf16; a.lse = lse;
  char* w = static_cast<char*>(ws);
  a.plan = reinterpret_cast<int4*>(w);
  a.seq_info = reinterpret_cast<int4*>(w + 16);
  a.partials = reinterpret_cast<float4*>(w + meta_bytes(p));
  a.batch = p.batch; a.Hq = p.n_qheads; a.Hkv = p.n_kvheads; a.G = p.n_qheads / p.n_kvheads;
  a.B = p.block_size; a.P = x.n_prefixes; a.mpb = x.max_prefix_blocks;
  a.err = err;
  const bool rows = rows_share_tiles(a, p.head_dim);
  if (p.head_dim == 128) return rows ? launch_t<128, true>(a, s) : launch_t<128, false>(a, s);
  return rows ? launch_t<64, true>(a, s) : launch_t<64, false>(a, s);
}

}  // namespace kvsel
