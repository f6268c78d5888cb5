// The 8-bit KV pages written and read back: kvsel_q8_write quantises K and V
// rows into the pages and keeps the block summaries of the stored keys up,
// kvsel_q8_read returns stored rows as bf16. The format is in q8.cuh.
//
// Work split: the rows of a call are ragged (sequence b has rows
// [row_start[b], row_start[b + 1]) at positions start_pos[b] onwards) and the
// host knows only their total, so the list of (sequence, block) items is laid
// out without a scan: the blocks that sequence b touches are items
// f(b), f(b) + 1, ... with f(b) = row_start[b] / B + 2 b. A sequence of L rows
// touches at most L / B + 2 blocks and f grows by at least that, so no two
// sequences share an item; a warp tries sequence i / 2 (right when sequences
// have few rows, as in a decode step) and else searches f 32 ways at a time.
// (Where row_start decreases f does too: an item that two sequences then claim
// goes to one of them, and the other's rows of that block are left out.)
// One warp per (item, KV head): it owns every row it writes and the block's
// summary, so nothing needs an atomic or a second pass. A lane holds 16
// channels: one 32-byte access of bf16 against one 16-byte chunk of codes.
//
// Bound: HBM (a written value moves 2 bytes in and 1 out), with the issue slots
// close behind: the write spends about 8 instructions a value, so two channels
// share an instruction wherever one exists (maxima of bf16 pairs, fp32 pairs,
// two codes a conversion). 16 sequences of 4096 rows, 8 KV heads, d = 128, E4M3:
// the write moves 408 MB in 70.4 us (5.8 TB/s, 0.85 of the copy rate; K's and V's
// maxima crossing the lanes one after the other and single fp32 operations:
// 74 us; two rows in flight a lane group instead of four: 71.8 us), the read 404
// MB in 64.8 us (6.2 TB/s, 0.92). One row a sequence: 4.0 us for 64 sequences of
// 2 KV heads, four dependent reads (the row's place, its page, its values, the
// block's earlier rows for the summary) and a launch.
#include "kvsel_common.cuh"
#include "kvsel_internal.h"
#include "q8.cuh"

namespace kvsel {
namespace {

constexpr int kWarps = 4;

struct Q8RowsArgs {
  uint8_t* pages;
  int64_t n_pages;
  const int32_t* block_table;
  const int32_t* row_start;   // [batch + 1]
  const int32_t* start_pos;   // [batch]
  kvsel_bf16* k;              // [n_rows] rows of [H][d], k_stride elements apart
  kvsel_bf16* v;
  int64_t n_rows, k_stride, v_stride;
  kvsel_bf16* summaries;      // write: nullable
  int batch, H, B, max_blocks;
  int64_t items;
  bool wide;                  // every row of k and v starts on 32 bytes
  int* err;
};

// What one warp has to do: rows [t0, t1) of block n of sequence b, the first
// of them the call's row `row`, in page `page`.
struct Q8Item {
  int b, n, t0, t1;
  int64_t row, page;
};

// The item of warp index i; false when there is nothing to do. All lanes.
__device__ bool q8_item(const Q8RowsArgs& a, int64_t i, bool report, Q8Item& it) {
  const int lane = threadIdx.x & 31;
  int lo = int(min(i >> 1, int64_t(a.batch - 1)));
  int r0 = a.row_start[lo], r1 = a.row_start[lo + 1], p0 = a.start_pos[lo];
  const auto first_item = [&](int row, int b) { return int64_t(max(0, row) / a.B) + 2 * int64_t(b); };
  if (first_item(r0, lo) > i || (lo + 1 < a.batch && first_item(r1, lo + 1) <= i)) {
    lo = 0;
    int n = a.batch;                       // the last b in [lo, lo + n) with f(b) <= i
    while (n > 1) {
      const int step = (n + 31) / 32;
      const int at = lo + lane * step;
      const bool le = lane * step < n && first_item(a.row_start[min(at, a.batch)], at) <= i;
      const unsigned vote = __ballot_sync(0xffffffffu, le);
      const int last = vote ? 31 - __clz(vote) : 0;
      lo += last * step;
      n = min(step, n - last * step);
    }
    r0 = a.row_start[lo], r1 = a.row_start[lo + 1], p0 = a.start_pos[lo];
  }
  if (report && i < a.batch && lane == 0) {  // every sequence's rows are checked by the item of its number
    const int s0 = a.row_start[i], s1 = a.row_start[i + 1], q0 = a.start_pos[i];
    if (s0 < 0 || s1 < s0 || s1 > a.n_rows) latch_error(a.err, KVSEL_ERR_BOUNDS);
    else if (q0 >= 0 && int64_t(q0) + (s1 - s0) > int64_t(a.max_blocks) * a.B)
      latch_error(a.err, KVSEL_ERR_BOUNDS);
  }
  if (r0 < 0 || r1 <= r0 || r1 > a.n_rows || p0 < 0) return false;
  const int64_t p1 = min(int64_t(p0) + (r1 - r0), int64_t(a.max_blocks) * a.B);
  const int64_t before = i - first_item(r0, lo);
  const int64_t blk = p0 / a.B + before;
  if (before < 0 || blk * a.B >= p1) return false;
  it.b = lo;
  it.n = int(blk);
  it.t0 = int(max(int64_t(p0), blk * a.B) - blk * a.B);
  it.t1 = int(min(p1, (blk + 1) * a.B) - blk * a.B);
  it.row = r0 + (blk * a.B + it.t0 - p0);
  it.page = a.block_table[int64_t(lo) * a.max_blocks + blk];
  if (it.page < 0 || it.page >= a.n_pages) {
    if (report && lane == 0) latch_error(a.err, KVSEL_ERR_BOUNDS);
    return false;
  }
  return true;
}

struct Row16 { uint32_t w[8]; };           // 16 bf16 channels

// `wide`: every row starts on 32 bytes (the host looks at pointers and strides);
// a projection's slices do, rows of any other multiple of 16 bytes take two accesses.
__device__ __forceinline__ Row16 load_row16(const kvsel_bf16* p, bool wide) {
  Row16 r;
  if (!wide) {
    const uint4 a = ldg_stream(p), b = ldg_stream(p + 8);
    r.w[0] = a.x; r.w[1] = a.y; r.w[2] = a.z; r.w[3] = a.w;
    r.w[4] = b.x; r.w[5] = b.y; r.w[6] = b.z; r.w[7] = b.w;
    return r;
  }
  asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3]), "=r"(r.w[4]), "=r"(r.w[5]), "=r"(r.w[6]),
                 "=r"(r.w[7])
               : "l"(p));
  return r;
}
__device__ __forceinline__ void store_row16(kvsel_bf16* p, const Row16& r, bool wide) {
  if (!wide) {
    stg_stream(p, make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]));
    stg_stream(p + 8, make_uint4(r.w[4], r.w[5], r.w[6], r.w[7]));
    return;
  }
  asm volatile("st.global.L1::no_allocate.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(r.w[0]), "r"(r.w[1]),
               "r"(r.w[2]), "r"(r.w[3]), "r"(r.w[4]), "r"(r.w[5]), "r"(r.w[6]), "r"(r.w[7])
               : "memory");
}

// 16 stored codes times their factor added to the block's column sums, in
// units of 2^8 (64 rows of the largest value stay in range). The product is
// exact, the sum rounds once a row: a pair of fp32 sums that carries each
// addition's error (about 48 bits) took 92.1 us for the large write's 70.5 and 4.27
// for a decode step's 3.82.
template <int FMT>
__device__ __forceinline__ void add_key(float2 (&s)[8], uint4 codes, uint32_t byte) {
  const float f1 = q8_factor(byte) * 0x1p-8f;
  const float2 f = make_float2(f1, f1);
  const uint32_t w[4] = {codes.x, codes.y, codes.z, codes.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t p01, p23;
    q8_to_f16<FMT>(w[i], p01, p23);
    s[2 * i] = fma2(make_float2(f16lo(p01), f16hi(p01)), f, s[2 * i]);
    s[2 * i + 1] = fma2(make_float2(f16lo(p23), f16hi(p23)), f, s[2 * i + 1]);
  }
}

// The scale bytes of one row of K and of V, LPR lanes a row. Magnitudes are
// compared as bit patterns, two at a time: their order is that of the numbers,
// and an infinity or a NaN is the largest. K's maximum and V's cross the lanes
// in one word: the exchanges, not the arithmetic, are what a row waits for.
template <int FMT, int LPR>
__device__ __forceinline__ void scale_bytes(const Row16& k, const Row16& v, uint32_t& kb, uint32_t& vb) {
  uint32_t mk = 0, mv = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    mk = __vmaxu2(mk, k.w[i] & 0x7FFF7FFFu);
    mv = __vmaxu2(mv, v.w[i] & 0x7FFF7FFFu);
  }
  uint32_t m = __vmaxu2(__byte_perm(mk, mv, 0x5410), __byte_perm(mk, mv, 0x7632));   // K low, V high
#pragma unroll
  for (int off = 1; off < LPR; off <<= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, off));
  kb = q8_scale_byte<FMT>(__uint_as_float(m << 16));
  vb = q8_scale_byte<FMT>(__uint_as_float(m & 0xFFFF0000u));
}

// One row's 16 channels of this lane as codes.
template <int FMT>
__device__ __forceinline__ uint4 quantise(const Row16& v, uint32_t byte) {
  const bool fine = byte != 255u;
  const float inv1 = fine ? q8_inverse(byte) : 0.f;
  const float2 inv = make_float2(inv1, inv1);
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 a = mul2(make_float2(bf16lo(v.w[2 * i]), bf16hi(v.w[2 * i])), inv);
    const float2 b = mul2(make_float2(bf16lo(v.w[2 * i + 1]), bf16hi(v.w[2 * i + 1])), inv);
    c[i] = q8_pack4<FMT>(a.x, a.y, b.x, b.y);
    if (!fine) c[i] = 0;                   // 0 times an infinity is no code
  }
  return make_uint4(c[0], c[1], c[2], c[3]);
}

template <int D, int FMT>
__global__ void __launch_bounds__(kWarps * 32) q8_write_kernel(Q8RowsArgs a) {
  constexpr int LPR = D / 16;              // lanes of a row (16 channels each)
  constexpr int RPW = 32 / LPR;            // rows of a warp at a time
  constexpr int kUnroll = 4;
  // a kernel launched after this one with programmatic serialization may
  // become resident now; it waits for this grid's completion before reading
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int64_t w = int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int64_t i = w / a.H;
  const int h = int(w % a.H);
  if (i >= a.items) return;
  Q8Item it;
  if (!q8_item(a, i, h == 0, it)) return;
  const int sub = lane / LPR, chunk = lane % LPR;
  uint8_t* head = a.pages + (it.page * a.H + h) * int64_t(q8_head_bytes(a.B, D));
  uint8_t* scales = head + 2 * a.B * D;
  const kvsel_bf16* ks = a.k + it.row * a.k_stride + int64_t(h) * D + chunk * 16;
  const kvsel_bf16* vs = a.v + it.row * a.v_stride + int64_t(h) * D + chunk * 16;
  // Row t of the block always falls to lane group t % RPW, whichever call writes it: a
  // summary's sum then has one order, however its block was split into calls.
  const int rows = it.t1 - it.t0, skip = it.t0 % RPW;   // row r of the call: slot r + skip
  Row16 kv[kUnroll], vv[kUnroll];
  auto load = [&](int r0) {
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int r = r0 + u * RPW + sub;
      if (r >= 0 && r < rows) {
        kv[u] = load_row16(ks + r * a.k_stride, a.wide);
        vv[u] = load_row16(vs + r * a.v_stride, a.wide);
      } else {
        kv[u] = vv[u] = Row16{};
      }
    }
  };
  load(-skip);
  float2 s[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) s[e] = make_float2(0.f, 0.f);
  if (a.summaries) {
    // the block's rows of earlier calls
    for (int t0 = 0; t0 < it.t0; t0 += 4 * RPW) {
      uint4 c[4];
      uint32_t b[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int t = t0 + u * RPW + sub;
        c[u] = make_uint4(0, 0, 0, 0);
        b[u] = 0;
        if (t < it.t0) {
          c[u] = *reinterpret_cast<const uint4*>(head + q8_chunk_off<D>(t, chunk));
          b[u] = scales[t];
        }
      }
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (t0 + u * RPW + sub < it.t0) add_key<FMT>(s, c[u], b[u]);
    }
  }
  for (int r0 = -skip; r0 < rows; r0 += RPW * kUnroll) {
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (r0 + u * RPW >= rows) break;
      const int r = r0 + u * RPW + sub;
      uint32_t kb, vb;
      scale_bytes<FMT, LPR>(kv[u], vv[u], kb, vb);
      const uint4 kc = quantise<FMT>(kv[u], kb);
      const uint4 vc = quantise<FMT>(vv[u], vb);
      if (r >= 0 && r < rows) {
        const int t = it.t0 + r;
        uint8_t* dst = head + q8_chunk_off<D>(t, chunk);
        *reinterpret_cast<uint4*>(dst) = kc;
        *reinterpret_cast<uint4*>(dst + a.B * D) = vc;
        if (chunk == 0) {
          scales[t] = uint8_t(kb);
          scales[a.B + t] = uint8_t(vb);
        }
        if (a.summaries) add_key<FMT>(s, kc, kb);
      }
    }
    if (r0 + RPW * kUnroll < rows) load(r0 + RPW * kUnroll);
  }
  if (!a.summaries) return;
#pragma unroll
  for (int e = 0; e < 8; ++e)
#pragma unroll
    for (int off = LPR; off < 32; off <<= 1)   // the warp's row groups
      s[e] = add2(s[e], make_float2(__shfl_xor_sync(0xffffffffu, s[e].x, off), __shfl_xor_sync(0xffffffffu, s[e].y, off)));
  if (sub == 0) {
    // the mean: one division (by a count of at most 64, rounded once to fp32), one rounding to bf16
    const float n = float(it.t1);
    Row16 m;
#pragma unroll
    for (int e = 0; e < 8; ++e)
      m.w[e] = pack_bf16x2(__fdiv_rn(s[e].x, n) * 256.f, __fdiv_rn(s[e].y, n) * 256.f);
    store_row16(a.summaries + ((int64_t(it.b) * a.max_blocks + it.n) * a.H + h) * D + chunk * 16, m, false);
  }
}

template <int D, int FMT>
__global__ void __launch_bounds__(kWarps * 32) q8_read_kernel(Q8RowsArgs a) {
  constexpr int LPR = D / 16;
  constexpr int RPW = 32 / LPR;
  constexpr int kUnroll = 4;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int64_t w = int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int64_t i = w / a.H;
  const int h = int(w % a.H);
  if (i >= a.items) return;
  Q8Item it;
  if (!q8_item(a, i, h == 0, it)) return;
  const int sub = lane / LPR, chunk = lane % LPR;
  const uint8_t* head = a.pages + (it.page * a.H + h) * int64_t(q8_head_bytes(a.B, D));
  const uint8_t* scales = head + 2 * a.B * D;
  kvsel_bf16* kd = a.k + it.row * a.k_stride + int64_t(h) * D + chunk * 16;
  kvsel_bf16* vd = a.v + it.row * a.v_stride + int64_t(h) * D + chunk * 16;
  const int rows = it.t1 - it.t0;
  auto expand = [](uint4 c, uint32_t byte) {
    const float f = q8_factor(byte);
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
    Row16 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t p01, p23;
      q8_to_f16<FMT>(w[i], p01, p23);
      r.w[2 * i] = pack_bf16x2(f16lo(p01) * f, f16hi(p01) * f);
      r.w[2 * i + 1] = pack_bf16x2(f16lo(p23) * f, f16hi(p23) * f);
    }
    return r;
  };
  for (int r0 = 0; r0 < rows; r0 += RPW * kUnroll) {
    uint4 kc[kUnroll], vc[kUnroll];
    uint32_t kb[kUnroll], vb[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int r = r0 + u * RPW + sub;
      if (r < rows) {
        const int t = it.t0 + r;
        const uint8_t* src = head + q8_chunk_off<D>(t, chunk);
        kc[u] = ldg_stream(src);
        vc[u] = ldg_stream(src + a.B * D);
        kb[u] = scales[t];
        vb[u] = scales[a.B + t];
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int r = r0 + u * RPW + sub;
      if (r < rows) {
        store_row16(kd + r * a.k_stride, expand(kc[u], kb[u]), a.wide);
        store_row16(vd + r * a.v_stride, expand(vc[u], vb[u]), a.wide);
      }
    }
  }
}

}  // namespace

cudaError_t launch_q8_rows(const kvsel_problem& p, const kvsel_q8_cache& c, const int32_t* row_start,
                           const int32_t* start_pos, kvsel_bf16* k, kvsel_bf16* v, int64_t n_rows,
                           int64_t k_stride, int64_t v_stride, kvsel_bf16* summaries, bool write, int* err,
                           cudaStream_t s) {
  if (p.batch == 0 || n_rows == 0) return cudaSuccess;
  Q8RowsArgs a{};
  a.pages = c.pages; a.n_pages = c.n_pages; a.block_table = c.block_table;
  a.row_start = row_start; a.start_pos = start_pos;
  a.k = k; a.v = v; a.n_rows = n_rows; a.k_stride = k_stride; a.v_stride = v_stride;
  a.summaries = summaries;
  a.batch = p.batch; a.H = p.n_kvheads; a.B = p.block_size; a.max_blocks = p.max_blocks;
  a.items = n_rows / p.block_size + 2 * int64_t(p.batch);
  a.wide = k_stride % 16 == 0 && v_stride % 16 == 0 &&
           ((reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) & 31) == 0;
  a.err = err;
  const int64_t ctas = (a.items * a.H + kWarps - 1) / kWarps;
  if (ctas >= (int64_t(1) << 31)) return cudaErrorInvalidConfiguration;
  const bool e4 = c.format == KVSEL_KV_PAGED_E4M3;
  void (*fn)(Q8RowsArgs);
  if (p.head_dim == 128) {
    fn = write ? (e4 ? q8_write_kernel<128, kQ8E4M3> : q8_write_kernel<128, kQ8Int8>)
               : (e4 ? q8_read_kernel<128, kQ8E4M3> : q8_read_kernel<128, kQ8Int8>);
  } else {
    fn = write ? (e4 ? q8_write_kernel<64, kQ8E4M3> : q8_write_kernel<64, kQ8Int8>)
               : (e4 ? q8_read_kernel<64, kQ8E4M3> : q8_read_kernel<64, kQ8Int8>);
  }
  fn<<<unsigned(ctas), kWarps * 32, 0, s>>>(a);
  count_launch();
  return cudaGetLastError();
}

}  // namespace kvsel
