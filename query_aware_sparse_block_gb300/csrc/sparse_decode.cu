// Sparse decode attention: workspace layout and dispatch by page format, and
// the bf16 shapes of the kernel in sparse_decode.cuh.
#include "sparse_decode.cuh"

namespace kvsel {

cudaError_t launch_decode_bf16(const kvsel_problem& p, const DecodeArgs& a, cudaStream_t s) {
  return launch_shape<kFmtBf16>(p, a, s);
}

// (sequence, head group) segments: 8-bit blocks of 16 tokens come in pairs, which
// leaves room for half as many heads in a tile.
static size_t segments_of(const kvsel_problem& p, bool q8) {
  const int tokens = q8 && p.block_size == 16 ? 32 : p.block_size;
  return size_t(p.batch) * (p.n_kvheads / heads_per_group(tokens, p.n_kvheads));
}

static size_t decode_meta_bytes(const kvsel_problem& p, bool q8) { return (segments_of(p, q8) * 8 + 255) / 256 * 256; }

size_t sparse_decode_ws_bytes(const kvsel_problem& p, bool q8) {
  const int G = p.n_qheads / std::max(1, p.n_kvheads);
  const int warps = q8 ? decode_warps<kFmtE4M3>(p.head_dim, G) : decode_warps<kFmtBf16>(p.head_dim, G);
  return decode_meta_bytes(p, q8) + (size_t(kMaxCtas) + segments_of(p, q8)) * warps * G * (p.head_dim + 4) * 4;
}

cudaError_t launch_sparse_decode(const kvsel_problem& p, const kvsel_bf16* q,
                                 const kvsel_kv_src& kv, const int32_t* seq_lens,
                                 const int32_t* sel_idx, const int32_t* n_sel,
                                 const uint8_t* dense_flag, float softmax_scale, float* out,
                                 kvsel_bf16* out_bf16, float* lse, void* ws, int* err,
                                 cudaStream_t s) {
  if (p.batch == 0) return cudaSuccess;
  DecodeArgs a{};
  a.q = q; a.seq_lens = seq_lens; a.sel_idx = sel_idx; a.n_sel = n_sel; a.dense_flag = dense_flag;
  a.block_table = kv.block_table; a.n_pages = kv.n_pages;
  const bool q8 = kv.kind == KVSEL_KV_PAGED_E4M3 || kv.kind == KVSEL_KV_PAGED_INT8;
  a.kind = q8 || kv.kind == KVSEL_KV_PAGED ? KVSEL_KV_PAGED
           : kv.kind == KVSEL_KV_HOST_DIRECT ? KVSEL_KV_HOST_DIRECT : KVSEL_KV_STAGED;
  a.slots = kv.staging_slots;
  a.host_blocks = kv.host_blocks;
  a.scale_log2 = softmax_scale * 1.4426950408889634f;
  a.out = out; a.out_bf16 = out_bf16; a.lse = lse;
  char* w = static_cast<char*>(ws);
  a.seg_info = reinterpret_cast<int2*>(w);
  a.partials = reinterpret_cast<float*>(w + decode_meta_bytes(p, q8));
  a.err = err;
  a.batch = p.batch; a.Hq = p.n_qheads; a.Hkv = p.n_kvheads; a.G = p.n_qheads / p.n_kvheads;
  a.B = p.block_size; a.max_blocks = p.max_blocks; a.k_max = p.k_max;
  a.kv_base = a.kind == KVSEL_KV_PAGED ? kv.kv_pages
              : a.kind == KVSEL_KV_HOST_DIRECT ? kv.host_kv : kv.staging;
  a.keep_nan = q8;
  if (kv.kind == KVSEL_KV_PAGED_E4M3) return launch_decode_e4m3(p, a, s);
  if (kv.kind == KVSEL_KV_PAGED_INT8) return launch_decode_int8(p, a, s);
  return launch_decode_bf16(p, a, s);
}

}  // namespace kvsel
