// sage_paged_attn_q8: checks, form and launch of the decode kernel over an 8-bit paged cache (paged_q8_attn.cuh).
#include <cmath>
#include <cstring>

#include "../../include/sageattn.h"
#include "paged_q8_attn.cuh"

namespace sage {
namespace {

struct Q8Layout {
  size_t err, part_o, part_ml, total;
};
size_t up256(size_t x) { return (x + 255) / 256 * 256; }
int tile_of(int d) { return d <= 64 ? Q8Cfg<64, 1>::kTile : Q8Cfg<128, 1>::kTile; }
// Ranges that the workspace has room for, whichever kernel runs.
constexpr int kMostRanges = Q8Cfg<128, 1>::kRanges;
static_assert(kMostRanges >= Q8Cfg<64, 1>::kRanges && kMostRanges >= Q8Cfg<64, 2>::kRanges && kMostRanges >= Q8Cfg<128, 2>::kRanges,
              "a line's ranges need room");
// Few heads with short sequences: one launch of clusters whose CTAs all run at once.
bool q8_clustered(int batch, int hkv, int row_blocks, int64_t max_len, int d) {
  return (int64_t)hkv * row_blocks * batch * kRanks <= kCtas && max_len <= 8 * kRanks * tile_of(d);
}
// Heads that an item of the line takes together, each with a part of the warps. Token rows that lie side by side (NHD): so
// that DRAM is read in 256 bytes or more, of which rows of other sizes than 128 begin and end inside of its 64-byte pieces
// (us with one, two and four heads: 32 sequences of up to 32K tokens 212, 188, 199; 32 x 8000 of head_dim 96 -, 100, 76, of 80
// -, 103, 97). Short sequences of rows by heads: all four warps, so that tiles are filled and fewer of them end (us with one head
// and with four: 512 x 150 tokens 82 and 72, 256 x 30-600 72 and 64, 256 x 300 59 and 57, but 128 x 600 46 and 47, 64 x 1200
// 41 and 43; at head_dim 64 512 x 150 62 and 59, 256 x 300 48 and 45).
int heads_beside(bool nhd, int hkv, int d, int64_t max_len) {
  const int want = nhd ? (d == 128 ? 2 : 4) : max_len <= 600 ? 4 : 1;
  return hkv % want == 0 ? want : hkv % 2 == 0 ? 2 : 1;
}
bool q8_layout(int batch, int hq, int hkv, int64_t max_len, int d, Q8Layout* L) {
  if (batch < 0 || hq < 1 || hkv < 1 || hq % hkv || max_len < 0 || d < 1 || d > 128) return false;
  const int dp = d <= 64 ? 64 : 128;
  // status word; the line's ranges: their errors and their pieces
  const bool line = !q8_clustered(batch, hkv, (hq / hkv + kRows - 1) / kRows, max_len, d);
  L->err = SAGE_STATUS_BYTES;
  L->part_o = L->err + (line ? up256(4 * kMostRanges) : 0);
  const size_t rows = line ? (size_t)kMostRanges * 2 * 4 * (hq / hkv <= 8 ? 8 : kRows) : 0;
  L->part_ml = L->part_o + up256(rows * dp * 4);
  L->total = L->part_ml + up256(rows * 4 * 4);
  return true;
}

}  // namespace
}  // namespace sage

using namespace sage;

extern "C" {

size_t sage_paged_attn_q8_workspace_size(int batch, int heads_q, int heads_kv, int max_seqlen, int head_dim) {
  Q8Layout L;
  return q8_layout(batch, heads_q, heads_kv, max_seqlen, head_dim, &L) ? L.total : 0;
}

int sage_paged_attn_q8(const sage_packed* q, const sage_q8_cache* cache, const sage_packed* out, float* lse,
                       const float* slopes, const int32_t* q_positions, int batch, int heads_q, int heads_kv,
                       int max_seqlen, int head_dim, int dtype, int tensor_layout, float sm_scale, float softcap,
                       void* workspace, size_t workspace_bytes, void* stream) {
  if (!q || !cache || !out) return SAGE_ERR_INVALID_ARG;
  Q8View view;
  int align = 1;
  const int s = make_q8_view(cache, batch, heads_kv, head_dim, tensor_layout, &view, &align);
  if (s != SAGE_OK) return s;
  if (dtype != SAGE_F16 && dtype != SAGE_BF16) return SAGE_ERR_DTYPE;
  if (heads_q < 1 || max_seqlen < 0 || batch > 65535 || !softcap_ok(softcap, sm_scale, head_dim))
    return SAGE_ERR_INVALID_ARG;
  if (heads_q % heads_kv) return SAGE_ERR_GQA;
  if (batch == 0) return empty_call(workspace, workspace_bytes, static_cast<cudaStream_t>(stream));
  if (!q->data || !out->data) return SAGE_ERR_INVALID_ARG;
  for (const sage_packed* t : {q, out})
    if (reinterpret_cast<uintptr_t>(t->data) % 2 || t->stride_token < 0 || t->stride_head < 0) return SAGE_ERR_STRIDE;
  if ((batch > 1 && out->stride_token == 0) || (heads_q > 1 && out->stride_head == 0)) return SAGE_ERR_STRIDE;
  for (const void* p : {(const void*)lse, (const void*)slopes, (const void*)q_positions})
    if (reinterpret_cast<uintptr_t>(p) % 4) return SAGE_ERR_INVALID_ARG;
  Q8Layout L;
  if (!q8_layout(batch, heads_q, heads_kv, max_seqlen, head_dim, &L)) return SAGE_ERR_INVALID_ARG;
  // (the status word alone can do without)
  if (workspace ? reinterpret_cast<uintptr_t>(workspace) % 256 || workspace_bytes < L.total : L.total > SAGE_STATUS_BYTES)
    return SAGE_ERR_WORKSPACE;
  if (!sage_device_supported()) return SAGE_ERR_DEVICE;
  Q8Args p{};
  DecodeArgs& a = p.a;
  a.c = view.c;
  p.ks = view.ks;
  p.vs = view.vs;
  p.block = view.block;
  p.blocks = view.blocks;
  p.k_type = view.k_type;
  p.v_type = view.v_type;
  p.bf16 = dtype == SAGE_BF16;
  a.q = q->data; a.q_sb = q->stride_token; a.q_sh = q->stride_head;
  a.o = out->data; a.o_sb = out->stride_token; a.o_sh = out->stride_head;
  p.q4 = reinterpret_cast<uintptr_t>(q->data) % 8 == 0 && head_dim % 4 == 0 && (batch == 1 || a.q_sb % 4 == 0) &&
         (heads_q == 1 || a.q_sh % 4 == 0);
  const int run = (head_dim <= 64 ? 64 : 128) / 16;
  p.o_run = reinterpret_cast<uintptr_t>(out->data) % (2 * run) == 0 && (batch == 1 || a.o_sb % run == 0) &&
            (heads_q == 1 || a.o_sh % run == 0);
  a.lse = lse;
  a.slopes = slopes;
  a.q_pos = q_positions;
  a.sm_scale = std::isnan(sm_scale) || sm_scale <= 0.f ? (float)(1.0 / std::sqrt((double)head_dim)) : sm_scale;
  a.cap = softcap;
  a.hq = heads_q;
  a.group = heads_q / heads_kv;
  a.row_blocks = (a.group + kRows - 1) / kRows;
  a.max_len = max_seqlen;
  p.cluster = q8_clustered(batch, heads_kv, a.row_blocks, max_seqlen, head_dim);
  // TMA: whole 16-byte rows, pages of whole 8-row blocks, no zero stride of a dimension that is walked
  const int64_t len[3] = {view.c.num_pages, heads_kv, view.c.page_size};
  const int64_t ks[3] = {a.c.k_sp, a.c.k_sh, a.c.k_st}, vs[3] = {a.c.v_sp, a.c.v_sh, a.c.v_st};
  bool tma = align == 16 && view.c.page_size % 8 == 0;
  for (int i = 0; i < 3; ++i)
    tma = tma && len[i] > 0 && (len[i] == 1 || (ks[i] > 0 && vs[i] > 0 && ks[i] < (1LL << 39) && vs[i] < (1LL << 39)));
  a.load = tma ? kLoadTma : align >= 4 ? kLoadVec : kLoadAny;
  p.unit = align >= 4 ? align : 1;
  const int dp = head_dim <= 64 ? 64 : 128, keys = tile_of(head_dim) / 4;
  a.box_rows = 8;
  while (a.box_rows < keys && view.c.page_size % (a.box_rows * 2) == 0) a.box_rows *= 2;
  a.page_shift = -1;
  p.block_shift = -1;
  for (int i = 0; i < 31; ++i) {
    if (view.c.page_size == 1 << i) a.page_shift = i;
    if (view.block == 1 << i) p.block_shift = i;
  }
  a.part_rows = a.group <= 8 ? 8 : kRows;
  a.side = p.cluster ? 1 : heads_beside(tensor_layout == SAGE_NHD, heads_kv, head_dim, max_seqlen);
  a.tile_shift = log2_of(tile_of(head_dim) / a.side);
  // the join by channels where its CTAs would leave SMs idle
  a.slices = (int64_t)heads_kv * a.row_blocks * batch <= 38 ? (head_dim <= 64 ? 2 : 4) : 1;
  CUtensorMap maps[2];
  std::memset(maps, 0, sizeof(maps));
  if (tma) {
    auto map = [&](CUtensorMap* m, const void* base, const int64_t (&st)[3]) {
      // (a stride that is never walked is given a legal value)
      return make_map4_bytes(m, base, head_dim, view.c.page_size, heads_kv, view.c.num_pages,
                             view.c.page_size > 1 ? st[2] : 128, heads_kv > 1 ? st[1] : 128,
                             view.c.num_pages > 1 ? st[0] : 128, dp, a.box_rows);
    };
    if (!map(&maps[0], a.c.k, ks) || !map(&maps[1], a.c.v, vs))
      return note_cuda_failure(cudaErrorInvalidValue, "cuTensorMapEncodeTiled");
  }
  char* w = static_cast<char*>(workspace);
  a.err = reinterpret_cast<int*>(w);
  a.cta_err = reinterpret_cast<int*>(w + L.err);
  a.part_o = reinterpret_cast<float*>(w + L.part_o);
  a.part_ml = reinterpret_cast<float*>(w + L.part_ml);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = dp == 64 ? launch_q8_decode_64(p, maps, st) : launch_q8_decode_128(p, maps, st);
  return e == cudaSuccess ? SAGE_OK : note_cuda_failure(e, "8-bit paged attention");
}

}  // extern "C"
