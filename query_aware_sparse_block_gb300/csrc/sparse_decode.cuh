// Sparse decode attention over the selected KV blocks ("SparPR KV cache
// recovery on a consumer GPU", paragraph "On-demand local recomputation with
// cost-aware fallback": only the recovered blocks are attended, or all of
// them on the dense path), with split partial results merged by the
// flash-style log-sum-exp reduction of the DKV abstract.
//
// Design (GB300):
//  * Work unit: a tile is one attended block of one sequence for a group of
//    HPG consecutive KV heads. The selection is per sequence, so all heads of
//    a page are needed, and a page stores each head's K tile and V tile next
//    to each other, heads in order: a tile's K and V are one contiguous range
//    (32 KiB for d = 128 and HPG * B = 64 rows), moved into shared memory by a
//    single 1-D bulk (TMA) copy. Scattered 32 KiB copies stream markedly
//    faster than pairs of 16 KiB ones on GB300 HBM3e. The tiled layout already
//    carries the 16-byte chunk swizzle (chunk c of row t at c ^ (t % 8)), so
//    ldmatrix reads are conflict-free.
//  * Work list: the flattened (sequence, head group, block) tiles. When every
//    (sequence, head group) segment that has tiles has the same number nb of
//    them (every sequence of the batch at the same length and k), each
//    segment gets the same number m of CTAs, m = min(grid / segments,
//    nb / kMinTilesPerCta rounded up), and CTA c takes part c % m of segment
//    c / m: no CTA's range crosses a segment boundary, so a warp loads one
//    query and stores one state, and the SMs left over stay free for the
//    Top-k still running in the previous kernel (64 segments on 152 SMs: 128
//    CTAs; the call is about 4 % shorter than with 152 CTAs whose ranges cross
//    segments, measured on GB300). Other
//    batches are split into equal contiguous ranges, one per CTA, so that the
//    HBM stream is balanced whatever the per-sequence selection sizes are. At
//    the end of each (sequence, head group) segment every warp stores its online-
//    softmax state (max, sum, unnormalised output) to global memory and moves
//    on without any synchronisation; a second small kernel, launched as a
//    programmatic dependent of the first so that it is already resident,
//    merges the states of each output row by log-sum-exp.
//  * Pipeline (bf16 pages): two rings of 4 warps; ring r takes every other
//    tile of the CTA's range and keeps S of them in flight. Each warp of a ring
//    owns one (head, 16-token slice) of its ring's tiles; the last warp to
//    finish a slot (a shared-memory counter) refills it, so no warp waits on
//    another and the two rings drift apart instead of hitting the tensor pipe
//    in lockstep.
//  * Math: tokens are the M dimension of mma.m16n8k16 bf16 tensor-core tiles:
//    S^T = K Q^T with K read by ldmatrix from the swizzled tile and the GQA
//    group's query heads (G <= 16, zero-padded to 8 or 16 columns) as N, online
//    softmax in fp32 per head column (exp2 of log2-scaled logits, accumulators
//    rescaled only when a running max moves), then O^T += V^T P^T with V read
//    by ldmatrix.trans and P transposed into B fragments by movmatrix; P is
//    split into bf16 high and low parts so the product keeps ~16 bits.
//  * Every wait on a copy is bounded; a wait that runs out latches
//    KVSEL_ERR_TIMEOUT and the warp stops issuing work.
//
// The kernel is a template over the page format (DecodeFormat): bf16 pages, or
// the 8-bit pages of q8.cuh, whose tile is half as large for the same work. Two
// rings of four warps then leave HBM waiting for the math: 16 sequences of 32
// heads (8 KV heads, d = 128), 128 blocks of 32 each, E4M3, took 49.5 us; with
// six rings of two warps that take 32 tokens each (a tile's bookkeeping, maxima
// and weight exchange once for twice the tokens) 34 us, and with the CTA joining
// its warps' states before the merge where no segment ends inside its range
// (one state a row and CTA instead of twelve) and a shorter prologue 30.1 us:
// 135 MB at 4.5 TB/s, of which 3.4 us are the prologue, 19.6 us the stream (6.9
// TB/s) and the rest the join, the grid's end and the merge. Blocks of 16 tokens
// come in pairs, so that a warp has its 32. With d = 128 and more than eight
// query heads a KV head the registers hold four rings. The 8-bit form differs
// further in the tile's address arithmetic and in the two products:
//  * codes become f16 in registers, exactly (an E4M3 or INT8 code has at most 8
//    significant bits); a K fragment's four bytes a thread are four consecutive
//    channels, so q's fragment takes the same channel order, and V's fragment
//    pairs channels 2g and 2g + 1 on rows g and g + 8;
//  * q becomes f16 scaled by a power of two per query head (largest magnitude in
//    [2^14, 2^15)): exact down to 2^-31 of the head's largest element, smaller ones are
//    off by at most 2^-39 of it (half the step of f16's subnormal numbers);
//  * a token's K factor 2^e multiplies its scores in fp32; its V factor 2^v joins
//    the softmax weight, p' = 2^(x + v - R) with R the running maximum of x + v
//    kept beside that of x, so p' <= 1 whatever the factors are; the state's
//    output is brought back by 2^(R - m) when it is stored. p' 2^15 is split into f16
//    high and low parts: 22 bits down to p' = 2^-17, below that off by at most 2^-40.
//    (f16 ends at 2^-24: unscaled, a token of p' = 2^-20 beside a peak keeps five bits
//    and one below 2^-25 none, yet both count in the sum.)
#pragma once

#include <climits>
#include <type_traits>

#include "kvsel_common.cuh"
#include "kvsel_internal.h"
#include "q8.cuh"

namespace kvsel {

struct DecodeArgs {
  const void* kv_base;        // PAGED: KV pages; STAGED: staging; HOST_DIRECT: the host tier
                              // (device-mapped); all in the same page layout
  const kvsel_bf16* q;
  const int32_t* seq_lens;
  const int32_t* sel_idx;
  const int32_t* n_sel;
  const uint8_t* dense_flag;
  const int32_t* block_table;
  int64_t n_pages;
  int kind;
  int slots;
  int host_blocks;     // HOST_DIRECT: block stride of the host tier per sequence
  float scale_log2;
  float* out;
  kvsel_bf16* out_bf16;
  float* lse;
  float* partials;     // warp states: [(cta + segment) * W + warp][G][D + 4] (m, l, -, -, O)
  int2* seg_info;      // [batch * n_groups] (first CTA, CTA count) of each segment; count 0: no tile;
                       // 8-bit pages: kFirstJoined, kLastJoined beside the count
  int* err;
  int batch, Hq, Hkv, G, B, max_blocks, k_max;
  int hpg, n_groups;   // heads per tile, head groups per sequence
  int stages;
  bool keep_nan;       // a row whose sum is NaN gives NaN (8-bit pages) instead of 0
};

namespace {

enum DecodeFormat { kFmtBf16 = 0, kFmtE4M3 = 1, kFmtInt8 = 2 };

constexpr int kTileRows = 64;          // token rows of a tile (of all its heads)
constexpr int kMaxCtas = 256;          // partial-slot capacity of the workspace
constexpr int kDenseSeq = 1 << 30;     // flag beside a sequence's length (at most 2^20)
// Flags beside a segment's CTA count: a CTA whose range lies in one segment has joined
// its warps' states (8-bit pages). Every CTA between a segment's first and last does.
constexpr int kFirstJoined = 1 << 30, kLastJoined = 1 << 29;
constexpr int kMinTilesPerCta = 4;
constexpr int kMaxStages = 8;
// 8-bit pages: the softmax weights, at most 1, times this are the f16 operands. Scaling by a
// power of two is exact; 2^15 is the largest that f16 holds.
constexpr float kWeightScale = 0x1p15f;

// Blocks of a tile: a warp of the 8-bit kernel takes 32 tokens, so blocks of 16
// come in pairs (the 2 o-th and the next of the attended ones, two copies).
template <int B, int FMT>
__host__ __device__ constexpr int blocks_per_tile() {
  return FMT != kFmtBf16 && B == 16 ? 2 : 1;
}

// Heads per tile for tiles of B tokens a head (all their blocks) and H_kv heads:
// as many as keep the tile at 64 token rows, and a divisor of H_kv.
inline int heads_per_group(int B, int Hkv) {
  int h = std::min(Hkv, kTileRows / B);
  while (h > 1 && Hkv % h) --h;
  return std::max(1, h);
}

// Rings of a CTA and 16-token subtiles of a warp (launch_group), and the warps that
// they make: the states' slots of a CTA and segment.
template <int FMT>
constexpr int decode_rings(int D, int G) {
  return FMT == kFmtBf16 ? 2 : D == 128 && G > 8 ? 4 : 6;
}
template <int FMT>
constexpr int decode_subtiles() {
  return FMT == kFmtBf16 ? 1 : 2;
}
template <int FMT>
constexpr int decode_warps(int D, int G) {
  return decode_rings<FMT>(D, G) * (4 / decode_subtiles<FMT>());
}

// Bytes of the K and V of HPG heads of one block, the unit of a copy.
template <int D, int B, int FMT>
__host__ __device__ constexpr int tile_unit_bytes(int hpg) {
  return FMT == kFmtBf16 ? hpg * B * D * 4 : hpg * q8_head_bytes(B, D);
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ int find_seq(const int* base_s, int batch, int g) {
  int lo = 0, hi = batch - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (base_s[mid] <= g) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// Copy unit of block k of the NB blocks of tile g (the head group's K+V range,
// in units of a copy) and its valid token count (0 when it is skipped).
template <int NB>
__device__ void tile_info(const DecodeArgs& a, const int* base_s, const int* tlen_s, int g, int k,
                          bool report, int& unit, int& cnt) {
  const int b = find_seq(base_s, a.batch, g);
  const int r = g - base_s[b];
  const int nb = (base_s[b + 1] - base_s[b]) / a.n_groups;
  const int hg = r / nb;
  const int o = (r - hg * nb) * NB + k;
  const int T = tlen_s[b] & ~kDenseSeq;
  const int N = (T + a.B - 1) / a.B;
  const bool dense = tlen_s[b] & kDenseSeq;
  if (NB > 1 && o >= tlen_s[a.batch + b]) {   // an odd count's last tile
    unit = cnt = 0;
    return;
  }
  const int n = dense ? o : a.sel_idx[int64_t(b) * a.k_max + o];
  bool ok = (n >= 0 && n < N);
  cnt = ok ? min(a.B, T - n * a.B) : 0;
  if (a.kind == KVSEL_KV_PAGED) {
    int64_t page = ok ? a.block_table[int64_t(b) * a.max_blocks + n] : 0;
    if (page < 0 || page >= a.n_pages) { ok = false; page = 0; }
    unit = int(page * a.n_groups + hg);
  } else if (a.kind == KVSEL_KV_HOST_DIRECT) {
    if (n >= a.host_blocks) ok = false;
    unit = ok ? int((int64_t(b) * a.host_blocks + n) * a.n_groups + hg) : 0;
  } else {
    int64_t slot = o;
    if (slot >= a.slots) { ok = false; slot = 0; }
    unit = int((int64_t(b) * a.slots + slot) * a.n_groups + hg);
  }
  if (!ok) {
    cnt = 0;
    if (report) latch_error(a.err, KVSEL_ERR_BOUNDS);
  }
}

// Shared address of (head h of the group, kv = 0 for K / 1 for V, token row,
// channel c with c % 8 == 0) in a slot holding the tile as the page stores it:
// [head][K, V][d/64][row][64], 16-byte chunk c of row t at c ^ (t % 8).
__device__ __forceinline__ uint32_t swz(uint32_t stage, int h, int kv, int halves, int B, int row,
                                        int c) {
  const int half = c >> 6;
  const int chunk = (c & 63) >> 3;
  return stage + uint32_t((((h * 2 + kv) * halves + half) * B + row) * 128 + ((chunk ^ (row & 7)) << 4));
}

// The same address for a tile of 8-bit pages: [head][K codes, V codes, scale
// bytes], c the 16-channel chunk.
template <int D, int B>
__device__ __forceinline__ uint32_t swz8(uint32_t stage, int h, int kv, int row, int c) {
  return stage + uint32_t(h * q8_head_bytes(B, D) + kv * B * D + q8_chunk_off<D>(row, c));
}

// One warp's TS subtiles of 16 token rows of one head of an 8-bit tile (subtile
// s at st + s * step, rows from r0 + s * 16 % B, cnt[s] of them valid): the running maxima
// of x (mh) and of x + v (rh), the sum of 2^(x - mh) and the output in units of
// 2^rh / kWeightScale, for the query heads in qb (f16, scaled back by qs).
template <int D, int B, int NTH, int FMT, int TS>
__device__ __forceinline__ void q8_tile(uint32_t st0, uint32_t step, int h, int row0, const int (&cnt)[TS],
                                        const uint32_t (&qb)[D / 16][NTH][2],
                                        const float (&qs)[NTH][2], float (&mh)[NTH][2], float (&rh)[NTH][2],
                                        float (&lh)[NTH][2], float (&o)[D / 16][NTH][4]) {
  const int lane = threadIdx.x & 31, gq = lane >> 2;
#pragma unroll
  for (int s = 0; s < TS; ++s) {
    if (cnt[s] < 16) {
      // rows past the sequence end: zero V so that 0 * (a code that is NaN) cannot poison P V
      for (int idx = lane; idx < (16 - max(cnt[s], 0)) * (D / 16); idx += 32) {
        const int row = row0 + (s * 16) % B + max(cnt[s], 0) + idx / (D / 16);
        const uint32_t ad = swz8<D, B>(st0 + s * step, h, 1, row, idx % (D / 16));
        asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(ad), "r"(0u) : "memory");
      }
      __syncwarp();
    }
  }
  // e & 1 selects head 2t / 2t+1, e >> 1 token g / g + 8 of subtile s
  float x[TS][NTH][4], vx[TS][2];
#pragma unroll
  for (int s = 0; s < TS; ++s) {
    const uint32_t st = st0 + s * step;
    const int r0 = row0 + (s * 16) % B;
    const uint32_t sc = st + uint32_t(h * q8_head_bytes(B, D) + 2 * B * D + r0 + gq);
    float sa[NTH][4], sb[NTH][4];
#pragma unroll
    for (int n = 0; n < NTH; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) sa[n][e] = sb[n][e] = 0.f;
    const int row = r0 + (lane & 15);
#pragma unroll
    for (int kp = 0; kp < D / 16; kp += 2) {
      uint32_t w[4], ka[2][4];
      ldsm_x4(swz8<D, B>(st, h, 0, row, kp + (lane >> 4)), w[0], w[1], w[2], w[3]);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        q8_to_f16<FMT>(w[2 * u], ka[u][0], ka[u][2]);
        q8_to_f16<FMT>(w[2 * u + 1], ka[u][1], ka[u][3]);
      }
#pragma unroll
      for (int n = 0; n < NTH; ++n) {
        mma_f16_16816(sa[n], ka[0], qb[kp][n][0], qb[kp][n][1]);
        mma_f16_16816(sb[n], ka[1], qb[kp + 1][n][0], qb[kp + 1][n][1]);
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float kf = q8_factor(lds_u8(sc + 8 * i));
      const uint32_t vb = lds_u8(sc + B + 8 * i);
      vx[s][i] = vb == 0u ? -INFINITY : vb == 255u ? q8_factor(255u) : float(int(vb) - 127);
      const bool live = i * 8 + gq < cnt[s];
#pragma unroll
      for (int n = 0; n < NTH; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c)
          x[s][n][2 * i + c] = live ? (sa[n][2 * i + c] + sb[n][2 * i + c]) * qs[n][c] * kf : -INFINITY;
    }
  }
  float mx[NTH][2], mr[NTH][2];
  bool grow = false;
#pragma unroll
  for (int n = 0; n < NTH; ++n)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      mx[n][c] = mr[n][c] = -INFINITY;
#pragma unroll
      for (int s = 0; s < TS; ++s)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          mx[n][c] = fmaxf(mx[n][c], x[s][n][2 * i + c]);
          mr[n][c] = fmaxf(mr[n][c], x[s][n][2 * i + c] + vx[s][i]);
        }
      grow |= mx[n][c] > mh[n][c] || mr[n][c] > rh[n][c];
    }
  // a lane whose own tokens pass a running maximum makes the warp look for the new ones
  if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
    for (int n = 0; n < NTH; ++n) {
      float alpha[2];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) {
          mx[n][c] = fmaxf(mx[n][c], __shfl_xor_sync(0xffffffffu, mx[n][c], off));
          mr[n][c] = fmaxf(mr[n][c], __shfl_xor_sync(0xffffffffu, mr[n][c], off));
        }
        const float mn = fmaxf(mh[n][c], mx[n][c]), rn = fmaxf(rh[n][c], mr[n][c]);
        lh[n][c] *= ex2(mh[n][c] - (mn == -INFINITY ? 0.f : mn));
        alpha[c] = ex2(rh[n][c] - (rn == -INFINITY ? 0.f : rn));
        mh[n][c] = mn;
        rh[n][c] = rn;
      }
#pragma unroll
      for (int mt = 0; mt < D / 16; ++mt) {
        o[mt][n][0] *= alpha[0]; o[mt][n][2] *= alpha[0];
        o[mt][n][1] *= alpha[1]; o[mt][n][3] *= alpha[1];
      }
    }
  }
  // P^T (tokens x heads) as the B operand: f16 high and low parts, each 8x8
  // block transposed from the accumulator layout with movmatrix
  uint32_t ph[TS][NTH][2], pl[TS][NTH][2];
#pragma unroll
  for (int s = 0; s < TS; ++s)
#pragma unroll
    for (int n = 0; n < NTH; ++n) {
      float pv[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float m = mh[n][e & 1], r = rh[n][e & 1];
        lh[n][e & 1] += ex2(x[s][n][e] - (m == -INFINITY ? 0.f : m));
        const float y = x[s][n][e] + vx[s][e >> 1] - (r == -INFINITY ? 0.f : r);
        pv[e] = 8 * (e >> 1) + gq < cnt[s] ? ex2(y) * kWeightScale : 0.f;
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint32_t hi = pack_f16x2(pv[2 * k], pv[2 * k + 1]);
        ph[s][n][k] = movmatrix_t(hi);
        pl[s][n][k] = movmatrix_t(pack_f16x2(pv[2 * k] - f16lo(hi), pv[2 * k + 1] - f16hi(hi)));
      }
    }
  // O^T += V^T P^T. A word of V holds tokens 2t, 2t + 1 of channels 2g, 2g + 1:
  // channel 2g goes to row g of the m-tile, channel 2g + 1 to row g + 8.
#pragma unroll
  for (int mt = 0; mt < D / 16; mt += 2)
#pragma unroll
    for (int s = 0; s < TS; ++s) {
      uint32_t w[4], va[2][4];
      ldsm_x4_t(swz8<D, B>(st0 + s * step, h, 1, row0 + (s * 16) % B + (lane & 15), mt + (lane >> 4)), w[0], w[1],
                w[2], w[3]);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        q8_to_f16<FMT>(__byte_perm(w[2 * u], 0u, 0x3120), va[u][0], va[u][1]);
        q8_to_f16<FMT>(__byte_perm(w[2 * u + 1], 0u, 0x3120), va[u][2], va[u][3]);
      }
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int n = 0; n < NTH; ++n) mma_f16_16816(o[mt + u][n], va[u], ph[s][n][0], ph[s][n][1]);
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int n = 0; n < NTH; ++n) mma_f16_16816(o[mt + u][n], va[u], pl[s][n][0], pl[s][n][1]);
    }
}

template <int D, int B, int NTH, int FMT, int RINGS, int TS>
__global__ void __launch_bounds__(RINGS * (4 / TS) * 32, 1) sparse_decode_kernel(DecodeArgs a) {
  constexpr bool kQ8 = FMT != kFmtBf16;
  constexpr int kRings = RINGS;
  constexpr int kRingWarps = 4 / TS;         // warps sharing one tile ring: one (head, 16 TS-token slice) each
  constexpr int kW = RINGS * kRingWarps;     // warps per CTA
  constexpr int kThreads = kW * 32;
  constexpr int kNB = blocks_per_tile<B, FMT>();
  constexpr int kWPH = B * kNB / (16 * TS);  // warps (slices) per head
  constexpr int kMT = D / 16;                // 16-channel m-tiles of O^T
  static_assert(kWPH <= kRingWarps, "block larger than a ring");
  constexpr int kKS = D / 16;                // k-steps of K Q^T
  constexpr int kHalves = D / 64;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int S = a.stages;
  const int G = a.G;
  const int HPG = a.hpg;
  const int unit_bytes = tile_unit_bytes<D, B, FMT>(HPG);    // K + V of one block
  const int tile_bytes = kNB * unit_bytes;
  unsigned char* tiles = smem;
  uint64_t* bars = reinterpret_cast<uint64_t*>(tiles + size_t(S) * kRings * tile_bytes);
  int* done_s = reinterpret_cast<int*>(bars + S * kRings);          // [S][rings] consumer counts
  int* base_s = done_s + 2 * kMaxStages * kRings;                  // [batch+1]
  int* tlen_s = base_s + a.batch + 1;                              // [batch] tokens, kDenseSeq; with pairs
                                                                   // of blocks also [batch] attended blocks
  __shared__ int scan_s[kW];
  __shared__ int nbmin_s[kW], nbmax_s[kW];   // per warp: smallest / largest non-zero tile count per segment

  // the merge kernel may be scheduled now; it waits for this grid's completion
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid < S * kRings) {
    mbar_init(&bars[tid], 1);
    done_s[tid] = 0;
    fence_barrier_init();
  }
  // every input may still be being written by an earlier kernel of the stream
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int NA = HPG * kWPH;                 // active warps per ring
  const int ring = warp / kRingWarps, task = warp % kRingWarps;
  const bool active = task < NA;
  const int h_local = task / kWPH, slice = task % kWPH;

  // ---- per-sequence tile counts and prefix; the range of the non-zero counts ----
  int carry = 0;
  int nb_lo = INT_MAX, nb_hi = 0;
  bool any_empty = false;
  for (int b0 = 0; b0 < a.batch; b0 += kThreads) {
    const int b = b0 + tid;
    int tiles_b = 0;
    if (b < a.batch) {
      int T = a.seq_lens[b], nb = a.n_sel[b];
      const bool dense = a.dense_flag && a.dense_flag[b];
      if (T < 0 || T > a.max_blocks * B) {
        latch_error(a.err, KVSEL_ERR_BOUNDS);
        T = T < 0 ? 0 : a.max_blocks * B;
      }
      tlen_s[b] = dense ? T | kDenseSeq : T;
      const int N = (T + B - 1) / B;
      if (dense) {
        nb = N;
      } else {
        if (nb < 0 || nb > a.k_max) latch_error(a.err, KVSEL_ERR_BOUNDS);
        nb = max(0, min(nb, min(N, a.k_max)));
      }
      if constexpr (kNB > 1) tlen_s[a.batch + b] = nb;
      tiles_b = (nb + kNB - 1) / kNB * a.n_groups;
    }
    {
      const int nb = tiles_b / a.n_groups;
      const int wmin = __reduce_min_sync(0xffffffffu, nb > 0 ? nb : INT_MAX);
      const int wmax = __reduce_max_sync(0xffffffffu, nb);
      const bool empty = __any_sync(0xffffffffu, b < a.batch && nb == 0);
      if (lane == 0) {
        nbmin_s[warp] = wmin;
        nbmax_s[warp] = empty ? ~wmax : wmax;    // the sign tells of a sequence without tiles
      }
    }
    int x = tiles_b;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, off);
      if (lane >= off) x += y;
    }
    if (lane == 31) scan_s[warp] = x;
    __syncthreads();
    int before = 0, tot = 0;
#pragma unroll
    for (int w = 0; w < kW; ++w) {
      if (w < warp) before += scan_s[w];
      tot += scan_s[w];
      nb_lo = min(nb_lo, nbmin_s[w]);
      const int hi = nbmax_s[w];
      any_empty |= hi < 0;
      nb_hi = max(nb_hi, hi < 0 ? ~hi : hi);
    }
    if (b < a.batch) base_s[b] = carry + before + x - tiles_b;
    carry += tot;
    __syncthreads();
  }
  if (tid == 0) base_s[a.batch] = carry;
  __syncthreads();
  const int total = carry;
  // equal segments: m CTAs each, ranges inside one segment
  const int nbu = nb_lo == nb_hi ? nb_hi : 0;
  const int n_seg = nbu > 0 ? total / nbu : 0;
  int m = n_seg > 0 && n_seg <= int(gridDim.x)
              ? min(int(gridDim.x) / n_seg, (nbu + kMinTilesPerCta - 1) / kMinTilesPerCta)
              : 0;
  if constexpr (kQ8) {
    // 8-bit pages: about 112 CTAs (d = 128; 130 at d = 64, whose tiles are half as long) take
    // what HBM gives, so few equal segments on fewer CTAs leave it waiting; ranges that cross
    // segments cost about five tiles (two segments a CTA, their states not joined). d = 128,
    // segments of 64 tiles, equal against crossing: 80 of them 27.3 and 23.4 us, 96 28.6 and
    // 26.0, 120 29.3 and 29.7; of 128 tiles: 44.5 and 36.6, 45.8 and 41.0, 48.4 and 49.4; 136
    // of 16 tiles 15.4 and 16.4. d = 64, of 32 tiles: 80 16.2 and 13.6, 96 16.5 and 15.1
    if (m > 0 && ((nbu + m - 1) / m - 5) * (D == 128 ? 112 : 130) > total) m = 0;
  }
  const int A = m > 0 ? n_seg * m : min(int(gridDim.x), max(1, (total - 1) / kMinTilesPerCta + 1));
  // the CTAs holding each segment's states, for the merge kernel; the CTAs share
  // the list (one segment takes two 64-bit divisions; a branch to 32-bit ones measured
  // 0.5 us slower a call)
  auto write_segments = [&]() {
    for (int seg = int(blockIdx.x) + (kThreads - 1 - tid) * int(gridDim.x); seg < a.batch * a.n_groups;
         seg += kThreads * int(gridDim.x)) {
      const int b = seg / a.n_groups, hg = seg % a.n_groups;
      const int seg_tiles = (base_s[b + 1] - base_s[b]) / a.n_groups;
      int2 info = make_int2(0, 0);
      if (seg_tiles > 0) {
        const int s_start = base_s[b] + hg * seg_tiles;
        if (m > 0) {
          info = make_int2(s_start / nbu * m, m);
        } else {
          const int first_c = int(((int64_t(s_start) + 1) * A - 1) / total);
          const int last_c = int(((int64_t(s_start) + seg_tiles) * A - 1) / total);
          info = make_int2(first_c, last_c - first_c + 1);
          if constexpr (kQ8) {
            const int q = total / A, rest = total - q * A;
            const auto begin = [&](int c) { return q * c + rest * c / A; };   // of a CTA's range
            if (begin(first_c) == s_start && begin(first_c + 1) <= s_start + seg_tiles) info.y |= kFirstJoined;
            if (begin(last_c + 1) == s_start + seg_tiles && begin(last_c) >= s_start) info.y |= kLastJoined;
          }
        }
      }
      if (kQ8 && m > 0) info.y |= kFirstJoined | kLastJoined;
      a.seg_info[seg] = info;
    }
  };

  // sequences with nothing to attend: out = 0, lse = -inf
  if (any_empty) {
    const int rows = a.batch * a.Hq;
    for (int64_t e = int64_t(blockIdx.x) * kThreads + tid; e < int64_t(rows) * (D / 4); e += int64_t(gridDim.x) * kThreads) {
      const int row = int(e / (D / 4)), b = row / a.Hq;
      if (base_s[b + 1] != base_s[b]) continue;
      if (e % (D / 4) == 0) a.lse[row] = -INFINITY;
      reinterpret_cast<float4*>(a.out)[e] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (a.out_bf16) reinterpret_cast<uint2*>(a.out_bf16)[e] = make_uint2(0u, 0u);
    }
  }
  if (total == 0 || int(blockIdx.x) >= A) {
    write_segments();
    return;
  }
  int g0, g1;
  if (m > 0) {
    const int k = int(blockIdx.x) / m, part = int(blockIdx.x) % m;
    g0 = k * nbu + nbu * part / m;
    g1 = k * nbu + nbu * (part + 1) / m;
  } else {
    // total i / A in 32 bits
    const int q = total / A, rest = total - q * A, i = int(blockIdx.x);
    g0 = q * i + rest * i / A;
    g1 = q * (i + 1) + rest * (i + 1) / A;
  }
  if (g0 >= g1) {
    write_segments();
    return;
  }
  const int L = g1 - g0;

  // ---- this ring's tile stream: tiles g0 + ring + m * kRings ----
  const int LR = L > ring ? (L - ring + kRings - 1) / kRings : 0;
  const uint32_t tiles_base = smem_u32(tiles);
  auto slot_idx = [&](int sl) -> int { return sl * kRings + ring; };   // sl: tile of the stream modulo S
  // Tile descriptors, 32 at a time: lane i holds the copy unit and valid token
  // count of tile (cbase + i) in `cur` and of tile (cbase + 32 + i) in `nxt`;
  // their selection and block-table loads run a whole batch ahead.
  int cbase = 0;
  struct Desc { int rk[kNB], cnt[kNB]; };
  Desc cur{}, nxt{};
  auto load_batch = [&](int base, Desc& d) {
    const int m = base + lane;
    d = Desc{};
    if (m < LR) {
#pragma unroll
      for (int k = 0; k < kNB; ++k)
        tile_info<kNB>(a, base_s, tlen_s, g0 + ring + m * kRings, k, task == 0, d.rk[k], d.cnt[k]);
    }
  };
  auto tile_desc = [&](int m, int (&rk)[kNB], int (&cnt)[kNB]) {   // all lanes; cbase <= m < cbase + 64
    const int i = m - cbase;
    const int src = i & 31;
#pragma unroll
    for (int k = 0; k < kNB; ++k) {
      const int rk0 = __shfl_sync(0xffffffffu, cur.rk[k], src), rk1 = __shfl_sync(0xffffffffu, nxt.rk[k], src);
      const int c0 = __shfl_sync(0xffffffffu, cur.cnt[k], src), c1 = __shfl_sync(0xffffffffu, nxt.cnt[k], src);
      rk[k] = i < 32 ? rk0 : rk1;
      cnt[k] = i < 32 ? c0 : c1;
    }
  };
  const uint64_t pol = l2_evict_first_policy();   // K/V are read once per step
  auto issue = [&](int sl, const int (&unit)[kNB]) {   // one lane
    uint64_t* bar = &bars[slot_idx(sl)];
    mbar_arrive_expect_tx(bar, uint32_t(tile_bytes));
    unsigned char* dst = tiles + size_t(slot_idx(sl)) * tile_bytes;
#pragma unroll
    for (int k = 0; k < kNB; ++k)
      bulk_load_hint(dst + k * unit_bytes, static_cast<const unsigned char*>(a.kv_base) + int64_t(unit[k]) * unit_bytes,
                     uint32_t(unit_bytes), bar, pol);
  };
  // From host-mapped memory the tile arrives by 16-byte cp.async reads of the
  // whole warp instead of one bulk copy (the same bytes land in the same
  // place); each lane's copies arrive on the slot's barrier when they have
  // landed, and lane 0's ordinary arrival completes the count of one.
  const bool host_direct = !kQ8 && a.kind == KVSEL_KV_HOST_DIRECT;
  auto issue_warp = [&](int sl, const int (&unit)[kNB]) {   // whole warp
    uint64_t* bar = &bars[slot_idx(sl)];
    const uint32_t dst = smem_u32(tiles + size_t(slot_idx(sl)) * tile_bytes);
    const unsigned char* src = static_cast<const unsigned char*>(a.kv_base) + int64_t(unit[0]) * tile_bytes;
    for (int off = lane * 16; off < tile_bytes; off += 32 * 16) cp_async_16(dst + off, src + off);
    cp_async_mbar_arrive(bar);
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
  };
  if (active) {
    load_batch(0, cur);
  }
  if (task == 0) {
    for (int m = 0; m < min(S, LR); ++m) {
      int rk[kNB], cnt[kNB];
      tile_desc(m, rk, cnt);
      if (host_direct) issue_warp(m, rk);
      else if (lane == 0) issue(m, rk);
    }
  }
  write_segments();
  if (active) load_batch(32, nxt);
  bool dead = false;
  int m_cur = 0, sl_cur = 0;                   // tile of this ring's stream; m_cur % S
  uint32_t ph_cur = 0;                         // (m_cur / S) & 1

  const int gq = lane >> 2, tq = lane & 3;   // mma group / thread-in-group
  const int r0 = slice * 16 * TS;            // this warp's token rows of its head
  int g = g0, b = 0, seg_tiles = 0, hg = 0;
  while (g < g1) {
    // ---- segment (sequence b, head group hg) containing g ----
    if (!kQ8 || g == g0 || g >= base_s[b + 1]) {
      b = find_seq(base_s, a.batch, g);
      seg_tiles = (base_s[b + 1] - base_s[b]) / a.n_groups;
      hg = (g - base_s[b]) / seg_tiles;
    } else {
      ++hg;
    }
    const int sg1 = min(g1, base_s[b] + (hg + 1) * seg_tiles);
    const int head = hg * HPG + h_local;      // this warp's KV head
    // 8-bit pages, a range in one segment: the CTA joins its warps' states (68 KB at most)
    // in the tiles' shared memory (at least 99 KB even beside the lengths of 4096 sequences)
    const bool single = kQ8 && g == g0 && sg1 == g1;
    if constexpr (kQ8) {
      // a segment without a tile of this ring: an empty state (25 ragged sequences x 32 heads,
      // up to 10 tiles a segment: 45 us where every ring loads q and stores its zeros)
      if (!single && !(m_cur < LR && g0 + ring + m_cur * kRings < sg1)) {
        if (active && lane < G) {
          const int64_t at = ((int64_t(blockIdx.x) + int64_t(b) * a.n_groups + hg) * kW + warp) * G + lane;
          *reinterpret_cast<float2*>(a.partials + at * (D + 4)) = make_float2(-INFINITY, 0.f);
        }
        g = sg1;
        continue;
      }
    }

    // O^T accumulators: o[mt][n] holds channels mt*16 + {g, g+8} of query heads
    // n*8 + {2t, 2t+1}; mh / lh: running max and (per-thread) sum of those heads
    float o[kMT][NTH][4];
#pragma unroll
    for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
      for (int n = 0; n < NTH; ++n) o[mt][n][0] = o[mt][n][1] = o[mt][n][2] = o[mt][n][3] = 0.f;
    float mh[NTH][2], lh[NTH][2];
#pragma unroll
    for (int n = 0; n < NTH; ++n) mh[n][0] = mh[n][1] = -INFINITY, lh[n][0] = lh[n][1] = 0.f;
    float rh[NTH][2];                        // 8-bit: running max of x + v (V's exponent)
    float qs[NTH][2];                        // 8-bit: scale_log2 times q's power of two, per head column
#pragma unroll
    for (int n = 0; n < NTH; ++n) rh[n][0] = rh[n][1] = -INFINITY, qs[n][0] = qs[n][1] = 0.f;

    if (active) {
      // Q^T as the B operand: qb[ks][n] = q[head n*8 + g][ks*16 + {2t, 2t+1, 2t+8, 2t+9}]
      // (query heads >= G are zero columns)
      uint32_t qb[kKS][NTH][2];
      {
        const kvsel_bf16* qp = a.q + (int64_t(b) * a.Hq + int64_t(head) * G) * D;
#pragma unroll
        for (int n = 0; n < NTH; ++n) {
          const int hq = n * 8 + gq;
          if constexpr (kQ8) {
            // channels ks * 16 + 4t .. 4t + 3, the order of a thread's four K bytes
            float top = 0.f;
#pragma unroll
            for (int ks = 0; ks < kKS; ++ks) {
              const uint2 v = hq < G ? *reinterpret_cast<const uint2*>(qp + hq * D + ks * 16 + 4 * tq)
                                     : make_uint2(0u, 0u);
              qb[ks][n][0] = v.x;
              qb[ks][n][1] = v.y;
              top = fmaxf(top, fmaxf(fmaxf(fabsf(bf16lo(v.x)), fabsf(bf16hi(v.x))),
                                     fmaxf(fabsf(bf16lo(v.y)), fabsf(bf16hi(v.y)))));
            }
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            // the largest magnitude's exponent becomes 14; a head of zeros, subnormals or
            // infinities is not scaled by it
            const int ex = int(__float_as_uint(top) >> 23);
            const int sh = ex == 0 || ex == 255 ? 0 : min(max(141 - ex, -126), 126);
            const float up = __uint_as_float(uint32_t(127 + sh) << 23);
            const float back = __uint_as_float(uint32_t(127 - sh) << 23) * a.scale_log2;
#pragma unroll
            for (int ks = 0; ks < kKS; ++ks)
#pragma unroll
              for (int i = 0; i < 2; ++i)
                qb[ks][n][i] = pack_f16x2(bf16lo(qb[ks][n][i]) * up, bf16hi(qb[ks][n][i]) * up);
#pragma unroll
            for (int c = 0; c < 2; ++c) qs[n][c] = __shfl_sync(0xffffffffu, back, (2 * tq + c) * 4);
            continue;
          }
#pragma unroll
          for (int ks = 0; ks < kKS; ++ks) {
            const int c = ks * 16 + 2 * tq;
            qb[ks][n][0] = hq < G ? *reinterpret_cast<const uint32_t*>(qp + hq * D + c) : 0u;
            qb[ks][n][1] = hq < G ? *reinterpret_cast<const uint32_t*>(qp + hq * D + c + 8) : 0u;
          }
        }
      }
      while (m_cur < LR && g0 + ring + m_cur * kRings < sg1) {
        if (m_cur == cbase + 32) {             // advance the descriptor window
          cbase += 32;
          cur = nxt;
          load_batch(cbase + 32, nxt);
        }
        int t_rk[kNB], t_cnt[kNB];
        tile_desc(m_cur, t_rk, t_cnt);
        uint64_t* bar_cur = &bars[slot_idx(sl_cur)];
        if (!dead && !mbar_wait_bounded(bar_cur, ph_cur)) {
          dead = true;
          if (lane == 0) latch_error(a.err, KVSEL_ERR_TIMEOUT);
        }
        if (host_direct) dead = __any_sync(0xffffffffu, dead);   // the refill is warp-wide
        // valid tokens in this warp's rows
        int cnt = 0, cnts[TS];
#pragma unroll
        for (int s = 0; s < TS; ++s) {
          cnts[s] = kNB > 1 ? t_cnt[s % kNB] : t_cnt[0] - r0 - s * 16;
          cnt = max(cnt, cnts[s]);
        }
        const uint32_t st = tiles_base + uint32_t(slot_idx(sl_cur)) * uint32_t(tile_bytes);
        if (!dead && cnt > 0) {
          if constexpr (kQ8) {
            q8_tile<D, B, NTH, FMT - 1, TS>(st, kNB > 1 ? unit_bytes : 0, h_local, r0, cnts, qb, qs, mh, rh, lh, o);
          } else {
            if (cnt < 16) {
              // rows past the sequence end: zero V so that 0 * garbage cannot poison P V
              for (int idx = lane; idx < (16 - cnt) * (D / 8); idx += 32) {
                const int row = r0 + cnt + idx / (D / 8);
                const int c = (idx % (D / 8)) * 8;
                const uint32_t ad = swz(st, h_local, 1, kHalves, B, row, c);
                asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(ad), "r"(0u) : "memory");
              }
              __syncwarp();
            }
            // S^T = K Q^T over this warp's 16 tokens (tokens are the M rows): even and
            // odd k-steps in separate accumulators to shorten the mma chains
            float sa[NTH][4], sb[NTH][4];
#pragma unroll
            for (int n = 0; n < NTH; ++n)
#pragma unroll
              for (int e = 0; e < 4; ++e) sa[n][e] = sb[n][e] = 0.f;
            {
              const int row = r0 + (lane & 7) + (((lane >> 3) & 1) << 3);
              const int cofs = (lane >> 4) * 8;
#pragma unroll
              for (int ks = 0; ks < kKS; ++ks) {
                uint32_t ka[4];
                ldsm_x4(swz(st, h_local, 0, kHalves, B, row, ks * 16 + cofs), ka[0], ka[1],
                        ka[2], ka[3]);
#pragma unroll
                for (int n = 0; n < NTH; ++n) {
                  if (ks & 1) mma_bf16_16816(sb[n], ka, qb[ks][n][0], qb[ks][n][1]);
                  else mma_bf16_16816(sa[n], ka, qb[ks][n][0], qb[ks][n][1]);
                }
              }
            }
            // scale, mask; e & 1 selects head 2t / 2t+1, e >> 1 token g / g + 8
            float x[NTH][4], mx[NTH][2];
#pragma unroll
            for (int n = 0; n < NTH; ++n) {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int tok = gq + 8 * (e >> 1);
                x[n][e] = tok < cnt ? (sa[n][e] + sb[n][e]) * a.scale_log2 : -INFINITY;
              }
              mx[n][0] = fmaxf(x[n][0], x[n][2]);
              mx[n][1] = fmaxf(x[n][1], x[n][3]);
            }
            bool grow = false;
#pragma unroll
            for (int n = 0; n < NTH; ++n)
#pragma unroll
              for (int c = 0; c < 2; ++c) {
#pragma unroll
                for (int off = 4; off < 32; off <<= 1)
                  mx[n][c] = fmaxf(mx[n][c], __shfl_xor_sync(0xffffffffu, mx[n][c], off));
                grow |= mx[n][c] > mh[n][c];
              }
            if (__any_sync(0xffffffffu, grow)) {
              // a running max moved: rescale the accumulators of every head
#pragma unroll
              for (int n = 0; n < NTH; ++n) {
                float alpha[2];
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                  const float mn = fmaxf(mh[n][c], mx[n][c]);
                  const float m_use = (mn == -INFINITY) ? 0.f : mn;
                  alpha[c] = ex2(mh[n][c] - m_use);
                  mh[n][c] = mn;
                  lh[n][c] *= alpha[c];
                }
#pragma unroll
                for (int mt = 0; mt < kMT; ++mt) {
                  o[mt][n][0] *= alpha[0]; o[mt][n][2] *= alpha[0];
                  o[mt][n][1] *= alpha[1]; o[mt][n][3] *= alpha[1];
                }
              }
            }
            // P^T (tokens x heads) as the B operand: bf16 high and low parts, each
            // 8x8 block transposed from the accumulator layout with movmatrix
            uint32_t ph[NTH][2], pl[NTH][2];
#pragma unroll
            for (int n = 0; n < NTH; ++n) {
              const float mu0 = (mh[n][0] == -INFINITY) ? 0.f : mh[n][0];
              const float mu1 = (mh[n][1] == -INFINITY) ? 0.f : mh[n][1];
              float pv[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                pv[e] = ex2(x[n][e] - ((e & 1) ? mu1 : mu0));
                lh[n][e & 1] += pv[e];
              }
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const uint32_t hi = pack_bf16x2(pv[2 * k], pv[2 * k + 1]);
                const uint32_t lo = pack_bf16x2(pv[2 * k] - bf16lo(hi), pv[2 * k + 1] - bf16hi(hi));
                ph[n][k] = movmatrix_t(hi);
                pl[n][k] = movmatrix_t(lo);
              }
            }
            // O^T += V^T P^T: V^T m-tiles (16 channels x 16 tokens) by ldmatrix.trans,
            // two m-tiles at a time, high parts then low parts
            {
              const int row = r0 + (lane & 7) + ((lane >> 4) << 3);
              const int cofs = ((lane >> 3) & 1) * 8;
#pragma unroll
              for (int mt = 0; mt < kMT; mt += 2) {
                uint32_t va[2][4];
#pragma unroll
                for (int u = 0; u < 2; ++u)
                  ldsm_x4_t(swz(st, h_local, 1, kHalves, B, row, (mt + u) * 16 + cofs),
                            va[u][0], va[u][1], va[u][2], va[u][3]);
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                  for (int n = 0; n < NTH; ++n) mma_bf16_16816(o[mt + u][n], va[u], ph[n][0], ph[n][1]);
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                  for (int n = 0; n < NTH; ++n) mma_bf16_16816(o[mt + u][n], va[u], pl[n][0], pl[n][1]);
              }
            }
          }
        }
        // release the slot; the last warp to release it refills it S tiles ahead
        __syncwarp();
        int last = 0;
        if (lane == 0) {
          const int before = atomicAdd(&done_s[slot_idx(sl_cur)], 1);
          last = (before % NA) == NA - 1;
        }
        last = __shfl_sync(0xffffffffu, last, 0);
        if (last && !dead && m_cur + S < LR) {
          int rk[kNB], cnt2[kNB];
          tile_desc(m_cur + S, rk, cnt2);
          if (host_direct) {
            issue_warp(sl_cur, rk);
          } else if (lane == 0) {
            fence_proxy_async();
            issue(sl_cur, rk);
          }
        }
        ++m_cur;
        if (++sl_cur == S) {
          sl_cur = 0;
          ph_cur ^= 1u;
        }
      }
    }

    // ---- store this warp's state for the segment; the merge kernel combines, or,
    // where a CTA has one segment (8-bit pages), the CTA first: its tiles' shared
    // memory is free once every warp is here ----
    bool joined = false;
    if constexpr (kQ8) {
      if (single) joined = !__syncthreads_or(dead);
    }
#pragma unroll
    for (int n = 0; n < NTH; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) lh[n][c] += __shfl_xor_sync(0xffffffffu, lh[n][c], off);
    if (active) {
      const int64_t seg = int64_t(b) * a.n_groups + hg;
      float* mw = joined ? reinterpret_cast<float*>(tiles) + warp * G * (D + 4)
                         : a.partials + ((int64_t(blockIdx.x) + seg) * kW + warp) * G * (D + 4);
#pragma unroll
      for (int n = 0; n < NTH; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int hq = n * 8 + 2 * tq + c;
          if (hq < G) {
            float* dst = mw + hq * (D + 4);
            if (gq == 0) {
              // a sum that is NaN without a maximum (every score NaN) still has to be merged
              dst[0] = kQ8 && lh[n][c] != lh[n][c] ? 0.f : mh[n][c];
              dst[1] = lh[n][c];
            }
            if constexpr (kQ8) {
              // two factors: V's exponent may be as low as -124, their product then underflows
              const float back = rh[n][c] == -INFINITY ? 1.f : ex2(rh[n][c] - (mh[n][c] == -INFINITY ? 0.f : mh[n][c]));
              constexpr float kUnscale = 1.f / kWeightScale;
#pragma unroll
              for (int mt = 0; mt < kMT; ++mt)
                *reinterpret_cast<float2*>(dst + 4 + mt * 16 + 2 * gq) =
                    make_float2(o[mt][n][c] * kUnscale * back, o[mt][n][c + 2] * kUnscale * back);
              continue;
            }
#pragma unroll
            for (int mt = 0; mt < kMT; ++mt) {
              dst[4 + mt * 16 + gq] = o[mt][n][c];
              dst[4 + mt * 16 + gq + 8] = o[mt][n][c + 2];
            }
          }
        }
    }
    if constexpr (kQ8) {
      if (joined) {
        __syncthreads();
        // a warp a row: lane k weighs state k, then the lanes share the channels
        constexpr int kN = kRings * kWPH, kCPL = D / 32;
        static_assert(kN <= 32, "a lane a state");
        const float* all = reinterpret_cast<const float*>(tiles);
        for (int row = warp; row < HPG * G; row += kW) {
          const int h = row / G, hq = row % G;
          auto state = [&](int k) {
            return all + (((k / kWPH) * kRingWarps + h * kWPH + k % kWPH) * G + hq) * (D + 4);
          };
          float mk = -INFINITY, lk = 0.f;
          if (lane < kN) {
            mk = state(lane)[0];
            lk = state(lane)[1];
          }
          float mx = mk;
#pragma unroll
          for (int off = 1; off < 32; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
          const float wk = mk == -INFINITY ? 0.f : ex2(mk - mx);
          float sum = wk * lk;
#pragma unroll
          for (int off = 1; off < 32; off <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
          float acc[kCPL] = {};
#pragma unroll
          for (int k = 0; k < kN; ++k) {
            const float w = __shfl_sync(0xffffffffu, wk, k);
            const bool some = __shfl_sync(0xffffffffu, mk, k) != -INFINITY;
            const float* v = state(k) + 4 + lane * kCPL;
#pragma unroll
            for (int u = 0; u < kCPL; ++u)
              if (some) acc[u] += w * v[u];
          }
          float* dst = a.partials + (((int64_t(blockIdx.x) + int64_t(b) * a.n_groups + hg) * kW + h) * G + hq) * (D + 4);
          if (lane == 0) {
            dst[0] = mx;
            dst[1] = sum;
          }
#pragma unroll
          for (int u = 0; u < kCPL; ++u) dst[4 + lane * kCPL + u] = acc[u];
        }
      }
    }
    g = sg1;
  }

  // drain copies still in flight (only after a timeout)
  if (dead && lane == 0 && task == 0)
    for (int m = m_cur; m < min(LR, m_cur + S); ++m)
      (void)mbar_wait_bounded(&bars[slot_idx(m % S)], uint32_t((m / S) & 1));
  if (host_direct) asm volatile("cp.async.wait_all;" ::: "memory");   // this thread's copies
}

// Log-sum-exp merge, per output row (sequence b, query head h), of the states
// every decode warp stored for the row's segment: one warp per row (MW = 1,
// four rows per CTA), or, when rows have many states, one CTA of four warps
// per row (MW = 4). Warp w takes every MW-th chunk of CH states; lane l owns channels
// [l * D/32, (l + 1) * D/32), and every lane loads each state's (max, sum) and
// its own channel slice, so a chunk costs one round trip to L2. With MW = 4 the
// four partial results are then merged through shared memory by warp 0. A long
// sequence attended by few blocks per CTA (one sequence of 131072 tokens, say)
// spreads its segment over many CTAs and so gives a row many states; four
// warps read them in a quarter of the round trips. Launched as a programmatic
// dependent of the decode kernel: it can be resident early and waits for the
// decode grid's completion before it reads anything that grid wrote.
template <int D, int WPH, int MW, int RINGS, int TS, int CH>
__global__ void __launch_bounds__(128) merge_rows_kernel(DecodeArgs a) {
  constexpr int kRings = RINGS;
  constexpr int kRingWarps = 4 / TS;
  constexpr int kW = RINGS * kRingWarps;
  constexpr int kCPL = D / 32;            // channels per lane
  constexpr int kChunk = CH;              // states in flight per lane
  constexpr int kPerCta = kRings * WPH;   // warps of one CTA holding a head
  static_assert(MW == 1 || MW == 4, "one or four warps per row");
  constexpr int kMW = MW;                 // warps sharing one row's states
  constexpr int kRowsPerCta = 4 / MW;
  using vec_t = typename std::conditional<kCPL == 4, float4, float2>::type;
  __shared__ float ml_s[4][2];
  __shared__ vec_t o_s[3][32];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31, wq = (threadIdx.x >> 5) % kMW;
  const int row = int(blockIdx.x) * kRowsPerCta + int(threadIdx.x >> 5) / kMW;   // the batch is at most 4096
  if (row >= a.batch * a.Hq) return;   // uniform in a CTA when kMW == 4
  const int b = row / a.Hq, hq = row - b * a.Hq;
  const int G = a.G, j = hq / G, r = hq % G;
  const int hg = j / a.hpg, h_local = j % a.hpg;
  const int seg = b * a.n_groups + hg;
  const int2 info = __ldcg(a.seg_info + seg);
  if (info.y == 0) return;                // no attended token: written by the decode kernel
  const int first_c = info.x;
  // 8-bit pages (TS == 2): a CTA that joined left one state a row, in the slot of the head's number
  constexpr bool kQ8 = TS == 2;
  const int cnt = kQ8 ? info.y & (kLastJoined - 1) : info.y;
  const int n_first = kQ8 && (info.y & kFirstJoined) ? 1 : kPerCta;
  const int n_before = kQ8 ? n_first + cnt - 2 : 0;          // states before the last CTA's
  const int NP = !kQ8 ? cnt * kPerCta : cnt == 1 ? n_first : n_before + (info.y & kLastJoined ? 1 : kPerCta);
  auto state = [&](int i) -> const float* {
    int c = first_c, k = i;
    bool joined = false;
    if constexpr (kQ8) {
      joined = n_first == 1;
      if (i >= n_first) {
        const bool last = i >= n_before;
        joined = !last || (info.y & kLastJoined);
        c += last ? cnt - 1 : i - n_first + 1;
        k = last ? i - n_before : 0;
      }
    } else {
      c += i / kPerCta;
      k = i % kPerCta;
    }
    const int w = joined ? h_local : (k / WPH) * kRingWarps + h_local * WPH + (k % WPH);
    return a.partials + (((int64_t(c) + seg) * kW + w) * G + r) * (D + 4);
  };
  float M = -INFINITY, L = 0.f;           // running max and sum (log2 domain)
  float acc[kCPL];
#pragma unroll
  for (int u = 0; u < kCPL; ++u) acc[u] = 0.f;
  for (int i0 = wq * kChunk; i0 < NP; i0 += kMW * kChunk) {   // every kMW-th chunk
    float mi[kChunk], li[kChunk];
    vec_t oi[kChunk];
#pragma unroll
    for (int k = 0; k < kChunk; ++k) {
      mi[k] = -INFINITY;
      li[k] = 0.f;
      if (i0 + k < NP) {
        const float* st = state(i0 + k);
        mi[k] = __ldcg(st);
        li[k] = __ldcg(st + 1);
        oi[k] = __ldcg(reinterpret_cast<const vec_t*>(st + 4) + lane);
      }
    }
    float mc = M;
#pragma unroll
    for (int k = 0; k < kChunk; ++k) mc = fmaxf(mc, mi[k]);
    if (mc == -INFINITY) continue;
    const float rs = M == -INFINITY ? 0.f : ex2(M - mc);
    L *= rs;
#pragma unroll
    for (int u = 0; u < kCPL; ++u) acc[u] *= rs;
#pragma unroll
    for (int k = 0; k < kChunk; ++k) {
      if (i0 + k < NP && mi[k] != -INFINITY) {
        const float wk = ex2(mi[k] - mc);
        L += wk * li[k];
        const float* ov = reinterpret_cast<const float*>(&oi[k]);
#pragma unroll
        for (int u = 0; u < kCPL; ++u) acc[u] += wk * ov[u];
      }
    }
    M = mc;
  }
  // the kMW partial states of the row, merged by warp 0
  if constexpr (kMW > 1) {
  if (lane == 0) {
    ml_s[wq][0] = M;
    ml_s[wq][1] = L;
  }
  if (wq > 0) {
    vec_t v;
    float* vp = reinterpret_cast<float*>(&v);
#pragma unroll
    for (int u = 0; u < kCPL; ++u) vp[u] = acc[u];
    o_s[wq - 1][lane] = v;
  }
  __syncthreads();
  if (wq > 0) return;
  {
    float mx = M;
#pragma unroll
    for (int w = 1; w < kMW; ++w) mx = fmaxf(mx, ml_s[w][0]);
    if (mx != -INFINITY) {
      const float r0 = M == -INFINITY ? 0.f : ex2(M - mx);
      L *= r0;
#pragma unroll
      for (int u = 0; u < kCPL; ++u) acc[u] *= r0;
#pragma unroll
      for (int w = 1; w < kMW; ++w) {
        const float mw = ml_s[w][0];
        if (mw == -INFINITY) continue;
        const float rw = ex2(mw - mx);
        L += rw * ml_s[w][1];
        const vec_t v = o_s[w - 1][lane];
        const float* ov = reinterpret_cast<const float*>(&v);
#pragma unroll
        for (int u = 0; u < kCPL; ++u) acc[u] += rw * ov[u];
      }
      M = mx;
    }
  }
  }
  vec_t res;
  float* rv = reinterpret_cast<float*>(&res);
#pragma unroll
  for (int u = 0; u < kCPL; ++u) rv[u] = L > 0.f || (a.keep_nan && L != L) ? acc[u] / L : 0.f;
  reinterpret_cast<vec_t*>(a.out + int64_t(row) * D)[lane] = res;
  if (a.out_bf16) {
    uint32_t pk[kCPL / 2];
#pragma unroll
    for (int u = 0; u < kCPL / 2; ++u)
      pk[u] = uint32_t(__bfloat16_as_ushort(__float2bfloat16_rn(rv[2 * u]))) |
              (uint32_t(__bfloat16_as_ushort(__float2bfloat16_rn(rv[2 * u + 1]))) << 16);
    if constexpr (kCPL == 4)
      reinterpret_cast<uint2*>(a.out_bf16 + int64_t(row) * D)[lane] = make_uint2(pk[0], pk[1]);
    else
      reinterpret_cast<uint32_t*>(a.out_bf16 + int64_t(row) * D)[lane] = pk[0];
  }
  if (lane == 0)
    a.lse[row] = L > 0.f || (a.keep_nan && L != L) ? (M + lg2(L)) * 0.6931471805599453f : -INFINITY;
}

template <int D, int B, int NTH, int FMT, int RINGS, int TS>
cudaError_t launch_t(const kvsel_problem& p, const DecodeArgs& a0, cudaStream_t s) {
  DecodeArgs a = a0;
  constexpr int kRings = RINGS;
  constexpr int kThreads = RINGS * (4 / TS) * 32, kNB = blocks_per_tile<B, FMT>();
  constexpr int kWPH = B * kNB / (16 * TS);
  a.hpg = heads_per_group(B * kNB, p.n_kvheads);
  a.n_groups = p.n_kvheads / a.hpg;
  const size_t tile_bytes = size_t(kNB) * tile_unit_bytes<D, B, FMT>(a.hpg);
  // 1024: manual alignment of the tile area; 256: static shared variables
  const size_t rest = 1024 + 256 + 8 * 2 * kMaxStages * kRings + (size_t(p.batch) * (kNB > 1 ? 3 : 2) + 1) * 4;
  const int max_optin = max_smem_optin();
  int stages = int((size_t(max_optin) - rest - 8 * kMaxStages * kRings) / (tile_bytes * kRings));
  stages = std::min(kMaxStages, stages);
  if (stages < 1) return cudaErrorInvalidConfiguration;
  a.stages = stages;
  const size_t smem = rest + size_t(stages) * kRings * tile_bytes + 8 * stages * kRings;
  auto kfn = sparse_decode_kernel<D, B, NTH, FMT, RINGS, TS>;
  cudaError_t e = ensure_smem(reinterpret_cast<const void*>(kfn), int(smem));
  if (e != cudaSuccess) return e;
  const int grid = std::min(kMaxCtas, sm_count());
  e = launch_pdl(kfn, dim3(grid), dim3(kThreads), smem, s, a);
  count_launch();
  if (e != cudaSuccess) return e;
  // The row merge, as a programmatic dependent of the decode grid.
  const int64_t rows = int64_t(p.batch) * p.n_qheads;
  const auto merge_by_warps = [&] {          // a warp a row
    return launch_pdl(merge_rows_kernel<D, kWPH, 1, RINGS, TS, 16>, dim3(unsigned((rows + 3) / 4)), dim3(128), 0, s, a);
  };
  if constexpr (FMT != kFmtBf16) {
    // A row has one state a CTA, and up to two dozen more where segments are unequal, which
    // the host cannot see; with few rows four warps share them eight at a time (128 rows of
    // unequal segments: 7.0 us with one warp a row and chunks of 16, 4.4 us with four and
    // chunks of 4, 4.0 us so; the whole call, four warps a row against one: 512 rows 18.8
    // and 21.3 us, 1024 rows 27.8 and 27.5, 2048 rows 31.2 and 27.8).
    e = rows <= 4 * int64_t(sm_count())
            ? launch_pdl(merge_rows_kernel<D, kWPH, 4, RINGS, TS, 8>, dim3(unsigned(rows)), dim3(128), 0, s, a)
            : merge_by_warps();
  } else {
    // A row has (CTAs its segment spans) x kRings x B/16 states; bound the span with the
    // decode's own split applied to k_max blocks per sequence, and give rows
    // with more than four chunks of states four warps each.
    const int64_t total_max = int64_t(p.batch) * a.n_groups * p.k_max;
    const int64_t ctas = std::min<int64_t>(sm_count(), std::max<int64_t>(1, (total_max + kMinTilesPerCta - 1) / kMinTilesPerCta));
    const int64_t per_cta = std::max<int64_t>(1, total_max / ctas);
    const int64_t span = (p.k_max + per_cta - 1) / per_cta + 1;
    e = span * kRings * kWPH > 64
            ? launch_pdl(merge_rows_kernel<D, kWPH, 4, RINGS, TS, 16>, dim3(unsigned(rows)), dim3(128), 0, s, a)
            : merge_by_warps();
  }
  count_launch();
  return e;
}

// Rings per CTA and 16-token subtiles per warp. A tile of 8-bit pages is half
// the bytes of a bf16 tile for the same work, so its warps have to issue less
// and more of them are needed to keep HBM busy: a warp takes 32 tokens (the
// bookkeeping of a tile, the maxima and the weights' exchange are then paid
// once for twice the tokens), and the rings are as many as the register file
// holds: more than eight query heads a KV head at d = 128 need 230 registers a
// thread.
template <int D, int B, int NTH, int FMT>
cudaError_t launch_group(const kvsel_problem& p, const DecodeArgs& a, cudaStream_t s) {
  return launch_t<D, B, NTH, FMT, decode_rings<FMT>(D, 8 * NTH), decode_subtiles<FMT>()>(p, a, s);
}

template <int D, int B, int FMT>
cudaError_t launch_heads(const kvsel_problem& p, const DecodeArgs& a, cudaStream_t s) {
  return a.G <= 8 ? launch_group<D, B, 1, FMT>(p, a, s) : launch_group<D, B, 2, FMT>(p, a, s);
}

template <int FMT>
cudaError_t launch_shape(const kvsel_problem& p, const DecodeArgs& a, cudaStream_t s) {
  const int D = p.head_dim, Bs = p.block_size;
  if (D == 128 && Bs == 16) return launch_heads<128, 16, FMT>(p, a, s);
  if (D == 128 && Bs == 32) return launch_heads<128, 32, FMT>(p, a, s);
  if (D == 128 && Bs == 64) return launch_heads<128, 64, FMT>(p, a, s);
  if (D == 64 && Bs == 16) return launch_heads<64, 16, FMT>(p, a, s);
  if (D == 64 && Bs == 32) return launch_heads<64, 32, FMT>(p, a, s);
  if (D == 64 && Bs == 64) return launch_heads<64, 64, FMT>(p, a, s);
  return cudaErrorInvalidValue;
}

}  // namespace

// One translation unit per page format compiles the kernel's shapes.
cudaError_t launch_decode_bf16(const kvsel_problem& p, const DecodeArgs& a, cudaStream_t s);
cudaError_t launch_decode_e4m3(const kvsel_problem& p, const DecodeArgs& a, cudaStream_t s);
cudaError_t launch_decode_int8(const kvsel_problem& p, const DecodeArgs& a, cudaStream_t s);

}  // namespace kvsel
