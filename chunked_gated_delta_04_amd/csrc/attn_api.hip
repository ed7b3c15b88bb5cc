// C ABI of the softmax attention and its paged key-value cache: argument
// checks, how the work is cut, launch sequencing. Every argument error returns
// before anything is enqueued.
#include <math.h>

#include <algorithm>

#include "attn.h"
#include "gdn.h"

#define GDN_API extern "C" __attribute__((visibility("default")))

using namespace gdn;

namespace {

#define GDN_TRY(expr)                              \
  do {                                             \
    if ((expr) != hipSuccess) return GDN_ERR_HIP;  \
  } while (0)

// Tiles of rows and of keys of a call together: a launch counts its threads in 32 bits, and has 512 for each row tile.
constexpr int64_t kMaxBlocks = (int64_t)1 << 23;
constexpr int64_t kMaxStride = (int64_t)1 << 23;  // a tile's rows span less than 2^31 bytes
constexpr int64_t kMaxPitch = (int64_t)1 << 40;   // of a cache
constexpr int kMaxTokens = 1 << 30;
constexpr int kCUs = 256;

bool aligned(const void* p, int to) { return ((uintptr_t)p & (uintptr_t)(to - 1)) == 0; }
bool bad_stride(int64_t s, int64_t dense) { return s != 0 && (s < dense || s % 8 != 0 || s >= kMaxStride); }

gdn_status check_bounds(int N, int T, const int32_t* cu) {
  if (!cu) return GDN_OK;
  if (cu[0] != 0 || cu[N] != T) return GDN_ERR_SEQLENS;
  for (int n = 0; n < N; ++n)
    if (cu[n + 1] < cu[n]) return GDN_ERR_SEQLENS;
  return GDN_OK;
}

int64_t div_up(int64_t a, int64_t b) { return (a + b - 1) / b; }
int group(const gdn_attn_problem* p) { return p->HQ / p->HK; }
int64_t row_tiles(const gdn_attn_problem* p) { return (int64_t)p->T / (attn_rows(p->D) / group(p)) + p->N; }
int64_t key_tiles(const gdn_attn_problem* p) { return (int64_t)p->T / attn_keys(p->D) + p->N; }

// What a call reads of a problem: boundaries (or one token a sequence), and rows of keys and values (or a cache).
enum Reads { kPack, kPagedPack, kPagedTokens };
gdn_status check_attn(const gdn_attn_problem* p, Reads reads) {
  if (!p) return GDN_ERR_NULL;
  if (p->N < 0 || p->T < 0 || p->HQ <= 0 || p->HK <= 0 || p->D <= 0 || p->window < 0 || p->sinks < 0)
    return GDN_ERR_SHAPE;
  if ((p->D != 64 && p->D != 128 && p->D != 256) || p->HQ % p->HK != 0 || p->HQ / p->HK > kAttnGroup ||
      (p->dtype != GDN_BF16 && p->dtype != GDN_FP16))
    return GDN_ERR_UNSUPPORTED;
  if (p->N == 0 && p->T != 0) return GDN_ERR_SHAPE;
  const int64_t dq = (int64_t)p->HQ * p->D, dk = (int64_t)p->HK * p->D;
  if (dq >= kMaxStride || bad_stride(p->q_stride, dq)) return GDN_ERR_SHAPE;
  if (reads == kPack && (bad_stride(p->k_stride, dk) || bad_stride(p->v_stride, dk))) return GDN_ERR_SHAPE;
  if (p->T > kMaxTokens || p->window > kMaxTokens || p->sinks > kMaxTokens ||
      (int64_t)p->T * p->HQ >= (int64_t)1 << 31 || (row_tiles(p) + key_tiles(p)) * p->HK > kMaxBlocks)
    return GDN_ERR_SHAPE;
  return reads == kPagedTokens ? GDN_OK : check_bounds(p->N, p->T, p->cu_seqlens_host);
}

gdn_status check_cache(const gdn_kv_cache* c, int N, int HK, int D) {
  if (!c) return GDN_ERR_NULL;
  if (c->pages < 0 || c->page_size <= 0 || c->columns < 0) return GDN_ERR_SHAPE;
  const int64_t row = (int64_t)D;
  for (int64_t s : {c->page_stride, c->token_stride, c->head_stride})
    if (s < row || s >= kMaxPitch) return GDN_ERR_SHAPE;
  if (c->table_stride < 0 || c->table_stride >= kMaxPitch) return GDN_ERR_SHAPE;
  if (N > 0 && (!c->k || !c->v || !c->offsets || (c->columns > 0 && !c->page_table))) return GDN_ERR_NULL;
  if (!aligned(c->page_table, 4) || !aligned(c->offsets, 4)) return GDN_ERR_ALIGN;
  return GDN_OK;
}
// the attention reads 16 bytes at once
gdn_status check_read_cache(const gdn_kv_cache* c, const gdn_attn_problem* p) {
  const gdn_status st = check_cache(c, p->N, p->HK, p->D);
  if (st != GDN_OK) return st;
  for (int64_t s : {c->page_stride, c->token_stride, c->head_stride})
    if (s % 8 != 0) return GDN_ERR_SHAPE;
  return aligned(c->k, 16) && aligned(c->v, 16) ? GDN_OK : GDN_ERR_ALIGN;
}

KvPages pages_of(const gdn_kv_cache* c) {
  KvPages p;
  p.k = c->k;
  p.v = c->v;
  p.page_stride = c->page_stride;
  p.token_stride = c->token_stride;
  p.head_stride = c->head_stride;
  p.table_stride = c->table_stride ? c->table_stride : c->columns;
  p.table = c->page_table;
  p.offsets = c->offsets;
  p.pages = c->pages;
  p.columns = c->columns;
  p.page = divisor(c->page_size);
  return p;
}

AttnPack pack_of(const gdn_attn_problem* p) {
  AttnPack a;
  a.cu = p->cu_seqlens;
  a.N = p->N;
  a.T = p->T;
  a.HQ = p->HQ;
  a.HK = p->HK;
  a.G = divisor(group(p));
  a.window = p->window;
  a.sinks = p->window ? p->sinks : 0;
  a.scale = p->scale > 0.f ? p->scale : 1.0f / sqrtf((float)p->D);
  return a;
}

// most keys that a tile of `tokens` tokens sees
int64_t most_keys(const gdn_attn_problem* p, int64_t keys, int64_t tokens) {
  return p->window ? std::min(keys, (int64_t)p->window + tokens + p->sinks) : keys;
}
// Parts of the keys, so that few row tiles fill the chip: as many as make `fill` items, of at least
// `least` keys. (Forward, least 512: one sequence of 2048 tokens, 8 + 2 heads of 128, 40 us, with 1024 44; 512 tokens after 8000,
// 16 + 2 heads of 256, 147 us, with 256 153. Step, least 128: 900 tokens 24.2 us, with 256 25.7; filling the chip
// twice: 131072 tokens 68.8 instead of 61.9, 64 rows under a window of 1024 37.7 instead of 28.1.)
int splits_of(int64_t items, int64_t keys, int fill, int least) {
  if (items >= fill || items == 0) return 1;
  return (int)std::max<int64_t>(1, std::min(fill / items, div_up(keys, least)));
}
int fwd_splits(const gdn_attn_problem* p, const gdn_kv_cache* c) {
  const int64_t keys = c ? (int64_t)c->columns * c->page_size : p->T;
  return splits_of(row_tiles(p) * p->HK, most_keys(p, keys, attn_rows(p->D) / group(p)), kCUs, 512);
}
int64_t step_items(const gdn_attn_problem* p) { return (int64_t)p->N * p->HK * div_up(group(p), 16); }
int step_splits(const gdn_attn_problem* p, const gdn_kv_cache* c) {
  // a workgroup takes 128 keys at once; with 256 columns a CU holds one, else two
  return splits_of(step_items(p), most_keys(p, (int64_t)c->columns * c->page_size, 1), (p->D == 256 ? 1 : 2) * kCUs, 128);
}
size_t part_bytes(const gdn_attn_problem* p, int splits) {
  return splits > 1 ? (size_t)splits * p->T * p->HQ * (p->D + 2) * sizeof(float) : 0;
}

AttnArgs args_of(const gdn_attn_problem* p, const void* q, void* o, float* lse, int splits, void* workspace) {
  AttnArgs a{};
  a.pack = pack_of(p);
  a.q = q;
  a.q_stride = p->q_stride ? p->q_stride : (int64_t)p->HQ * p->D;
  a.o = o;
  a.lse = lse;
  a.splits = splits;
  a.part = static_cast<float*>(workspace);
  a.slots = (int)row_tiles(p);
  return a;
}

// o, lse and the workspace of a forward
gdn_status check_outputs(const gdn_attn_problem* p, const void* q, const void* o, const float* lse, int splits,
                         const void* workspace, size_t bytes) {
  if (!q || !o) return GDN_ERR_NULL;
  if (!aligned(q, 16) || !aligned(o, 16) || !aligned(lse, 4) || !aligned(workspace, 16)) return GDN_ERR_ALIGN;
  const size_t need = part_bytes(p, splits);
  return need > 0 && (!workspace || bytes < need) ? GDN_ERR_WORKSPACE : GDN_OK;
}

int run_fwd(const gdn_attn_problem* p, bool paged, const AttnArgs& a, hipStream_t s) {
  const Elem type = static_cast<Elem>(p->dtype);
  GDN_TRY(launch_attn_fwd(type, p->D, paged, a, s));
  if (a.splits > 1) GDN_TRY(launch_attn_join(type, p->D, a, s));
  return GDN_OK;
}

// How the backward's work is cut: the key tiles' rows into parts until there are some four items to a CU, and
// the rows that see the sinks from behind the window, of one tile or few, into parts as long as the
// other tiles' rows. Both from the extents alone. (Ten sequences of 0 to 1031 tokens, 8 + 4 heads of 64: 63.4 us, with two
// items to a CU 67.1; 2048 tokens, 16 + 2 heads of 256: 203 us, with eight 244.)
struct GradCut {
  int pieces, far_pieces, far_tiles, far_slots;
  int64_t far_rows;
};
GradCut grad_cut(const gdn_attn_problem* p) {
  GradCut c{1, 0, 0, 0, 0};
  const int64_t items = key_tiles(p) * p->HK;
  // rows that see a tile of a sequence of four times the mean length
  const int64_t mean = p->N > 0 ? div_up(p->T, p->N) : 0;
  const int64_t rows = most_keys(p, std::min<int64_t>(4 * mean, p->T), attn_keys(p->D)) * group(p);
  if (items > 0) c.pieces = (int)std::max<int64_t>(1, std::min<int64_t>({4 * kCUs / items, 8, rows / 256}));
  if (p->window && p->sinks && p->T > p->window) {
    c.far_tiles = (int)div_up(std::min<int64_t>(p->sinks, p->T), attn_keys(p->D));
    c.far_slots = (int)std::min((int64_t)p->N * c.far_tiles, key_tiles(p));
    c.far_rows = std::min<int64_t>((int64_t)p->N * c.far_tiles * attn_keys(p->D), p->T);
    // at most four times dk's and dv's rows are kept
    const int64_t most = std::min<int64_t>({64, std::max<int64_t>(4 * (int64_t)p->T / c.far_rows, 1),
                                            std::max<int64_t>(kMaxBlocks / 2 / ((int64_t)c.far_slots * p->HK), 1)});
    c.far_pieces = (int)std::min(div_up((int64_t)p->T - p->window, (int64_t)p->window + attn_keys(p->D)), most);
  }
  return c;
}
// bytes of the workspace: the rows' statistics, then the parts of the windows, then those of the sinks
struct GradBytes {
  size_t stats, part, far;
  size_t all() const { return stats + part + far; }
};
GradBytes grad_bytes(const gdn_attn_problem* p) {
  const GradCut c = grad_cut(p);
  const size_t row = (size_t)p->HK * 2 * p->D * sizeof(float);
  GradBytes b{(grad_stats(static_cast<Elem>(p->dtype)) * (size_t)p->T * p->HQ * sizeof(float) + 15) / 16 * 16, 0, 0};
  if (c.pieces > 1) b.part = c.pieces * (size_t)p->T * row;
  if (c.far_tiles) b.far = (size_t)(c.far_pieces + (c.pieces > 1 ? 0 : 1)) * c.far_rows * row;
  return b;
}

}  // namespace

GDN_API size_t gdn_attn_fwd_workspace_size(const gdn_attn_problem* p) {
  return check_attn(p, kPack) == GDN_OK ? part_bytes(p, fwd_splits(p, nullptr)) : 0;
}

GDN_API int gdn_attn_fwd(const gdn_attn_problem* p, const void* q, const void* k, const void* v, void* o, float* lse,
                         void* workspace, size_t workspace_bytes, void* stream) {
  gdn_status st = check_attn(p, kPack);
  if (st != GDN_OK) return st;
  if (p->T == 0) return GDN_OK;
  if (!k || !v || !p->cu_seqlens) return GDN_ERR_NULL;
  const int splits = fwd_splits(p, nullptr);
  st = check_outputs(p, q, o, lse, splits, workspace, workspace_bytes);
  if (st != GDN_OK) return st;
  if (!aligned(k, 16) || !aligned(v, 16)) return GDN_ERR_ALIGN;
  AttnArgs a = args_of(p, q, o, lse, splits, workspace);
  a.k = k;
  a.v = v;
  a.k_stride = p->k_stride ? p->k_stride : (int64_t)p->HK * p->D;
  a.v_stride = p->v_stride ? p->v_stride : (int64_t)p->HK * p->D;
  return run_fwd(p, false, a, reinterpret_cast<hipStream_t>(stream));
}

GDN_API size_t gdn_attn_fwd_paged_workspace_size(const gdn_attn_problem* p, const gdn_kv_cache* c) {
  return check_attn(p, kPagedPack) == GDN_OK && check_read_cache(c, p) == GDN_OK ? part_bytes(p, fwd_splits(p, c)) : 0;
}

GDN_API int gdn_attn_fwd_paged(const gdn_attn_problem* p, const gdn_kv_cache* c, const void* q, void* o, float* lse,
                               void* workspace, size_t workspace_bytes, void* stream) {
  gdn_status st = check_attn(p, kPagedPack);
  if (st != GDN_OK) return st;
  st = check_read_cache(c, p);
  if (st != GDN_OK) return st;
  if (p->T == 0) return GDN_OK;
  if (!p->cu_seqlens) return GDN_ERR_NULL;
  const int splits = fwd_splits(p, c);
  st = check_outputs(p, q, o, lse, splits, workspace, workspace_bytes);
  if (st != GDN_OK) return st;
  AttnArgs a = args_of(p, q, o, lse, splits, workspace);
  a.pages = pages_of(c);
  return run_fwd(p, true, a, reinterpret_cast<hipStream_t>(stream));
}

GDN_API size_t gdn_attn_step_workspace_size(const gdn_attn_problem* p, const gdn_kv_cache* c) {
  return check_attn(p, kPagedTokens) == GDN_OK && p->T == p->N && check_read_cache(c, p) == GDN_OK ? part_bytes(p, step_splits(p, c)) : 0;
}

GDN_API int gdn_attn_step(const gdn_attn_problem* p, const gdn_kv_cache* c, const void* q, void* o, float* lse,
                          void* workspace, size_t workspace_bytes, void* stream) {
  gdn_status st = check_attn(p, kPagedTokens);
  if (st != GDN_OK) return st;
  if (p->T != p->N || step_items(p) > kMaxBlocks) return GDN_ERR_SHAPE;
  st = check_read_cache(c, p);
  if (st != GDN_OK) return st;
  if (p->T == 0) return GDN_OK;
  const int splits = step_splits(p, c);
  st = check_outputs(p, q, o, lse, splits, workspace, workspace_bytes);
  if (st != GDN_OK) return st;
  AttnArgs a = args_of(p, q, o, lse, splits, workspace);
  a.pages = pages_of(c);
  a.pack.cu = nullptr;  // every token is a sequence's
  const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const Elem type = static_cast<Elem>(p->dtype);
  GDN_TRY(launch_attn_step(type, p->D, a, s));
  if (splits > 1) GDN_TRY(launch_attn_join(type, p->D, a, s));
  return GDN_OK;
}

GDN_API size_t gdn_attn_bwd_workspace_size(const gdn_attn_problem* p) {
  return check_attn(p, kPack) == GDN_OK ? grad_bytes(p).all() : 0;
}

GDN_API int gdn_attn_bwd(const gdn_attn_problem* p, const void* q, const void* k, const void* v, const void* o,
                         const float* lse, const void* dO, void* dq, void* dk, void* dv, void* workspace,
                         size_t workspace_bytes, void* stream) {
  const gdn_status st = check_attn(p, kPack);
  if (st != GDN_OK) return st;
  if (p->T == 0) return GDN_OK;
  if (!q || !k || !v || !o || !lse || !dO || !dq || !dk || !dv || !p->cu_seqlens) return GDN_ERR_NULL;
  for (const void* t : {q, k, v, o, dO, (const void*)dq, (const void*)dk, (const void*)dv, (const void*)workspace})
    if (!aligned(t, 16)) return GDN_ERR_ALIGN;
  if (!aligned(lse, 4)) return GDN_ERR_ALIGN;
  const GradBytes bytes = grad_bytes(p);
  if (!workspace || workspace_bytes < bytes.all()) return GDN_ERR_WORKSPACE;
  const GradCut cut = grad_cut(p);
  AttnGradArgs a{};
  a.pack = pack_of(p);
  a.q = q;
  a.k = k;
  a.v = v;
  a.o = o;
  a.dO = dO;
  a.q_stride = p->q_stride ? p->q_stride : (int64_t)p->HQ * p->D;
  a.k_stride = p->k_stride ? p->k_stride : (int64_t)p->HK * p->D;
  a.v_stride = p->v_stride ? p->v_stride : (int64_t)p->HK * p->D;
  a.lse = lse;
  a.dq = dq;
  a.dk = dk;
  a.dv = dv;
  a.slots = (int)row_tiles(p);
  a.key_slots = (int)key_tiles(p);
  a.pieces = cut.pieces;
  a.far_pieces = cut.far_pieces;
  a.far_tiles = cut.far_tiles;
  a.far_slots = cut.far_slots;
  char* ws = static_cast<char*>(workspace);
  a.stats = reinterpret_cast<float*>(ws);
  a.part = reinterpret_cast<float*>(ws + bytes.stats);
  a.far = reinterpret_cast<float*>(ws + bytes.stats + bytes.part);
  GDN_TRY(launch_attn_bwd(static_cast<Elem>(p->dtype), p->D, a, reinterpret_cast<hipStream_t>(stream)));
  return GDN_OK;
}

GDN_API int gdn_kv_append(const gdn_kv_append_problem* p, const gdn_kv_cache* c, const float* inv_freq, const void* q,
                          const void* k, const void* v, void* q_out, void* stream) {
  if (!p) return GDN_ERR_NULL;
  if (p->N < 0 || p->T < 0 || p->HQ < 0 || p->HK <= 0 || p->D <= 0) return GDN_ERR_SHAPE;
  if (p->D > 1024 || p->R < 0 || p->R > p->D || p->R % 2 != 0 || (p->dtype != GDN_BF16 && p->dtype != GDN_FP16) ||
      (p->interleaved != 0 && p->interleaved != 1))
    return GDN_ERR_UNSUPPORTED;
  const int64_t dq = (int64_t)p->HQ * p->D, dk = (int64_t)p->HK * p->D;
  const auto bad = [](int64_t s, int64_t dense) { return s != 0 && (s < dense || s >= (int64_t)1 << 31); };
  if (dq + 2 * dk >= (int64_t)1 << 28 || p->T > kMaxTokens || bad(p->q_stride, dq) || bad(p->q_out_stride, dq) ||
      bad(p->k_stride, dk) || bad(p->v_stride, dk))
    return GDN_ERR_SHAPE;
  if (p->N == 0 && p->T != 0) return GDN_ERR_SHAPE;
  if (!p->cu_seqlens && p->T != p->N) return GDN_ERR_SHAPE;  // one token each
  gdn_status st = p->cu_seqlens ? check_bounds(p->N, p->T, p->cu_seqlens_host) : GDN_OK;
  if (st != GDN_OK) return st;
  st = check_cache(c, p->N, p->HK, p->D);
  if (st != GDN_OK) return st;
  if (p->T == 0) return GDN_OK;
  if (!k || !v || (p->R > 0 && !inv_freq) || (p->HQ > 0 && (!q || !q_out))) return GDN_ERR_NULL;
  if (p->HQ == 0) q = q_out = nullptr;
  for (const void* t : {q, k, v, (const void*)q_out, (const void*)c->k, (const void*)c->v})
    if (!aligned(t, 2)) return GDN_ERR_ALIGN;
  if (!aligned(inv_freq, 4)) return GDN_ERR_ALIGN;
  AppendArgs a;
  a.T = p->T;
  a.N = p->N;
  a.D = p->D;
  a.R = p->R;
  a.mscale = p->mscale > 0.f ? p->mscale : 1.f;
  a.inv_freq = inv_freq;
  a.cu = p->cu_seqlens;
  a.q = {q, q_out, p->q_stride ? p->q_stride : dq, p->q_out_stride ? p->q_out_stride : dq, p->HQ};
  a.k = {k, nullptr, p->k_stride ? p->k_stride : dk, 0, p->HK};
  a.v = v;
  a.v_stride = p->v_stride ? p->v_stride : dk;
  a.pages = pages_of(c);
  bool wide = p->R % (p->interleaved ? 8 : 16) == 0 && p->D % 8 == 0;
  for (const void* t : {q, k, v, (const void*)q_out, (const void*)c->k, (const void*)c->v}) wide = wide && aligned(t, 16);
  for (int64_t s : {a.q.in_stride, a.q.out_stride, a.k.in_stride, a.v_stride, c->page_stride, c->token_stride, c->head_stride})
    wide = wide && s % 8 == 0;
  GDN_TRY(launch_kv_append(static_cast<Elem>(p->dtype), p->interleaved != 0, wide, a, reinterpret_cast<hipStream_t>(stream)));
  return GDN_OK;
}
