// C ABI of the quantised key/value cache and its attention: argument checks, the choice of kernel and
// of key splits, the workspace.  Every check happens before anything is enqueued.
#include <math.h>

#include "hqq_internal.h"
#include "hqq_kv.h"

namespace {

using hqq::api_fail;
using hqq::kv::AttnArgs;
using hqq::kv::Format;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int device_status(hipError_t e) {
  return e == hipSuccess ? HQQ_OK : api_fail(HQQ_ERR_DEVICE, hipGetErrorString(e));
}

#define KV_NEED(cond, status, message) \
  do {                                 \
    if (!(cond)) return api_fail(status, message); \
  } while (0)

int64_t block_bytes(int D, int bits, int gs, int page) { return (int64_t)page * 2 * (D * bits / 8 + 4 * (D / gs)); }

int check_format(int hkv, int D, int bits, int gs, int page) {
  KV_NEED(hkv > 0 && D > 0 && gs > 0 && page > 0, HQQ_ERR_INVALID_ARGUMENT, "cache sizes must be positive");
  KV_NEED(bits > 0 && bits <= 8, HQQ_ERR_INVALID_ARGUMENT, "nbits must be 4 or 8");
  KV_NEED(D == 64 || D == 128, HQQ_ERR_UNSUPPORTED, "head_dim must be 64 or 128");
  KV_NEED(bits == 4 || bits == 8, HQQ_ERR_UNSUPPORTED, "nbits must be 4 or 8");
  KV_NEED((gs == 32 || gs == 64 || gs == 128) && gs <= D, HQQ_ERR_UNSUPPORTED,
          "group_size must be 32, 64 or 128 and at most head_dim");
  KV_NEED(page == 16 || page == 32 || page == 64 || page == 128 || page == 256, HQQ_ERR_UNSUPPORTED,
          "page_size must be 16, 32, 64, 128 or 256");
  KV_NEED(hkv <= 4096, HQQ_ERR_UNSUPPORTED, "at most 4096 KV heads");
  return HQQ_OK;
}

int check_cache(const hqq_kv_cache& c, Format* f) {
  const int st = check_format(c.num_kv_heads, c.head_dim, c.nbits, c.group_size, c.page_size);
  if (st != HQQ_OK) return st;
  KV_NEED(c.pages && aligned16(c.pages), HQQ_ERR_INVALID_ARGUMENT, "pages must be a 16-byte aligned pointer");
  KV_NEED(c.num_pages >= 1 && c.num_pages <= INT32_MAX, HQQ_ERR_INVALID_ARGUMENT, "num_pages must be 1 .. 2^31-1");
  f->pages = static_cast<uint8_t*>(c.pages);
  f->num_pages = (uint32_t)c.num_pages;
  f->hkv = c.num_kv_heads;
  f->page_shift = __builtin_ctz(c.page_size);
  f->block_bytes = block_bytes(c.head_dim, c.nbits, c.group_size, c.page_size);
  f->page_bytes = f->block_bytes * c.num_kv_heads;
  return HQQ_OK;
}

bool known_type(int dtype) { return dtype == HQQ_KV_F16 || dtype == HQQ_KV_BF16; }

// The passes of one attention call: over the sequences' own keys, and over the shared prefix.
struct Plan {
  AttnArgs own, prefix;
  int own_kind, prefix_kind;  // row kernel of each
  bool has_prefix;
  int parts;
  size_t workspace;
};

// Row kernels: the stream with 16 or 32 rows a wave, or tiles of 256 rows.
enum { kStream16, kStream32, kTile };

int row_kernel(int64_t rows) { return rows <= 16 ? kStream16 : rows <= 64 ? kStream32 : kTile; }
int64_t row_tiles(int64_t rows, int kind) {
  const int64_t of = kind == kStream16 ? 16 : kind == kStream32 ? 32 : 256;
  return (rows + of - 1) / of;
}

// Key splits: enough blocks to fill the 256 CUs several times over (a tile block fills one), at least
// 256 keys each.
void split_keys(AttnArgs* a, int kind, int64_t blocks, int64_t keys) {
  const int64_t want = kind == kTile ? 256 : 1024;
  int64_t n = kind == kTile ? want / blocks : (want + blocks - 1) / blocks;
  if (kind != kTile && keys / 2048 > n) n = keys / 2048;
  const int64_t most = (keys + 255) / 256;
  n = n > most ? most : n;
  n = n < 1 ? 1 : n;
  int64_t chunk = ((keys + n - 1) / n + 127) / 128 * 128;
  chunk = chunk < 128 ? 128 : chunk;
  a->chunk = (int)chunk;
  a->nsplit = (int)((keys + chunk - 1) / chunk);
  if (a->nsplit < 1) a->nsplit = 1;
}

hipError_t launch_pass(const AttnArgs& a, int kind, const hqq_kv_cache& c, hipStream_t st) {
  if (kind == kTile) return hqq::kv::launch_kv_tile(a, c.head_dim, c.nbits, c.group_size, st);
  return hqq::kv::launch_kv_stream(a, c.head_dim, c.nbits, c.group_size, kind == kStream16 ? 1 : 2, st);
}

int plan_attention(const hqq_kv_attention_args* x, bool sizes_only, Plan* p) {
  Format f{};
  const hqq_kv_cache& c = x->cache;
  if (sizes_only) {
    const int st = check_format(c.num_kv_heads, c.head_dim, c.nbits, c.group_size, c.page_size);
    if (st != HQQ_OK) return st;
    f.hkv = c.num_kv_heads;
    f.page_shift = __builtin_ctz(c.page_size);
  } else {
    const int st = check_cache(c, &f);
    if (st != HQQ_OK) return st;
  }
  KV_NEED(known_type(x->dtype), HQQ_ERR_INVALID_ARGUMENT, "dtype must be HQQ_KV_F16 or HQQ_KV_BF16");
  KV_NEED(x->total_q >= 0 && x->total_q <= (int64_t(1) << 30) && x->num_seqs >= 0 && x->num_q_heads > 0,
          HQQ_ERR_INVALID_ARGUMENT, "total_q, num_seqs and num_q_heads must be in range");
  KV_NEED(x->num_q_heads % c.num_kv_heads == 0, HQQ_ERR_INVALID_ARGUMENT,
          "num_q_heads must be a multiple of num_kv_heads");
  KV_NEED(x->total_q == 0 || x->num_seqs > 0, HQQ_ERR_INVALID_ARGUMENT, "query tokens without a sequence");
  KV_NEED(x->cu_q || x->num_seqs == 0 || x->total_q % x->num_seqs == 0, HQQ_ERR_INVALID_ARGUMENT,
          "without cu_q total_q must be a multiple of num_seqs");
  KV_NEED(!x->cu_q || (x->max_q >= 0 && x->max_q <= x->total_q), HQQ_ERR_INVALID_ARGUMENT, "max_q must be 0 .. total_q");
  KV_NEED(x->max_len >= 0 && x->max_len <= INT32_MAX - 256, HQQ_ERR_INVALID_ARGUMENT, "max_len out of range");
  KV_NEED(x->prefix_len >= 0 && x->prefix_len <= INT32_MAX - 256, HQQ_ERR_INVALID_ARGUMENT, "prefix_len out of range");
  KV_NEED(x->table_cols >= 0 && x->table_cols * (int64_t)c.page_size <= INT32_MAX, HQQ_ERR_INVALID_ARGUMENT,
          "table_cols out of range");
  KV_NEED(x->table_stride >= x->table_cols, HQQ_ERR_INVALID_ARGUMENT, "table_stride is smaller than table_cols");
  KV_NEED(x->causal == 0 || x->causal == 1, HQQ_ERR_INVALID_ARGUMENT, "causal must be 0 or 1");
  KV_NEED(x->scale > 0.f && x->scale <= 3.0e38f, HQQ_ERR_INVALID_ARGUMENT, "scale must be finite and positive");

  AttnArgs a{};
  a.f = f;
  a.q = x->q;
  a.q_ts = x->q_token_stride;
  a.q_hs = x->q_head_stride;
  a.dtype = x->dtype;
  a.hq = x->num_q_heads;
  a.per = x->num_q_heads / c.num_kv_heads;
  a.num_seqs = (int)x->num_seqs;
  a.tq = x->num_seqs ? (int)(x->total_q / x->num_seqs) : 0;
  a.max_q = x->cu_q ? (int)x->max_q : a.tq;
  a.total_q = x->total_q;
  a.cu_q = x->cu_q;
  a.table = x->page_table;
  a.table_stride = x->table_stride;
  a.table_cols = (int)x->table_cols;
  a.lens = x->seq_lens;
  a.max_len = (int)x->max_len;
  a.causal = x->causal;
  a.scale_log2 = x->scale * 1.44269504089f;
  a.out = x->out;
  a.lse = x->lse;
  p->own = p->prefix = a;
  p->has_prefix = x->prefix_len > 0;
  p->workspace = 0;
  p->parts = 1;
  if (x->total_q == 0 || x->num_seqs == 0 || a.max_q == 0) return HQQ_OK;

  const int64_t rows = (int64_t)a.max_q * a.per;
  p->own_kind = row_kernel(rows);
  const int64_t tiles = row_tiles(rows, p->own_kind);
  KV_NEED(x->num_seqs <= 65535, HQQ_ERR_UNSUPPORTED, "at most 65535 sequences in a call");
  KV_NEED(tiles <= 65535, HQQ_ERR_UNSUPPORTED, "too many query rows in a sequence");
  split_keys(&p->own, p->own_kind, tiles * f.hkv * x->num_seqs, x->max_len);
  p->parts = p->own.nsplit;
  if (p->has_prefix) {
    AttnArgs& b = p->prefix;
    b.num_seqs = 1;
    b.tq = b.max_q = (int)x->total_q;
    b.cu_q = nullptr;
    b.table = x->prefix_table;
    b.table_stride = 0;
    b.table_cols = (int)((x->prefix_len + c.page_size - 1) / c.page_size);
    b.lens = nullptr;
    b.fixed_len = b.max_len = (int)x->prefix_len;
    b.causal = 0;
    const int64_t all = x->total_q * a.per;
    p->prefix_kind = row_kernel(all);
    const int64_t t = row_tiles(all, p->prefix_kind);
    KV_NEED(t <= 65535, HQQ_ERR_UNSUPPORTED, "too many query rows in a call");
    split_keys(&b, p->prefix_kind, t * f.hkv, x->prefix_len);
    b.part0 = p->own.nsplit;
    p->parts += b.nsplit;
  }
  p->own.parts = p->prefix.parts = p->parts;
  if (p->parts > 1) {
    const size_t all_rows = (size_t)x->total_q * x->num_q_heads;
    p->workspace = (size_t)p->parts * all_rows * (4 * (size_t)c.head_dim + sizeof(float2));
  }
  return HQQ_OK;
}

int run_attention(const hqq_kv_attention_args* x) {
  Plan p;
  const int st = plan_attention(x, false, &p);
  if (st != HQQ_OK) return st;
  if (x->total_q == 0 || p.own.max_q == 0) return HQQ_OK;
  const hqq_kv_cache& c = x->cache;
  KV_NEED(x->q && aligned16(x->q) && x->out && aligned16(x->out), HQQ_ERR_INVALID_ARGUMENT,
          "q and out must be 16-byte aligned pointers");
  KV_NEED(x->q_token_stride >= 0 && x->q_head_stride >= 0 && x->q_token_stride % 8 == 0 && x->q_head_stride % 8 == 0,
          HQQ_ERR_INVALID_ARGUMENT, "q strides must be non-negative multiples of 8 elements");
  KV_NEED(x->seq_lens, HQQ_ERR_INVALID_ARGUMENT, "seq_lens must not be NULL");
  KV_NEED(x->page_table || x->table_cols == 0, HQQ_ERR_INVALID_ARGUMENT, "page_table must not be NULL");
  KV_NEED(!p.has_prefix || x->prefix_table, HQQ_ERR_INVALID_ARGUMENT, "prefix_table must not be NULL");
  if (p.workspace) {
    KV_NEED(x->workspace && x->workspace_bytes >= p.workspace, HQQ_ERR_WORKSPACE,
            "workspace missing or smaller than hqq_kv_attention_workspace_bytes");
    KV_NEED(aligned16(x->workspace), HQQ_ERR_INVALID_ARGUMENT, "workspace must be 16-byte aligned");
    const size_t all_rows = (size_t)x->total_q * x->num_q_heads;
    p.own.part_o = p.prefix.part_o = static_cast<float*>(x->workspace);
    p.own.part_ml = p.prefix.part_ml =
        reinterpret_cast<float2*>(static_cast<float*>(x->workspace) + (size_t)p.parts * all_rows * c.head_dim);
  }
  hipStream_t stream = static_cast<hipStream_t>(x->stream);
  hipError_t e = hipSuccess;
  if (p.has_prefix) e = launch_pass(p.prefix, p.prefix_kind, c, stream);
  if (e == hipSuccess) e = launch_pass(p.own, p.own_kind, c, stream);
  if (e == hipSuccess && p.parts > 1) e = hqq::kv::launch_kv_join(p.own, c.head_dim, stream);
  return device_status(e);
}

}  // namespace

extern "C" {

size_t hqq_kv_page_bytes(int num_kv_heads, int head_dim, int nbits, int group_size, int page_size) {
  if (check_format(num_kv_heads, head_dim, nbits, group_size, page_size) != HQQ_OK) return 0;
  return (size_t)(num_kv_heads * block_bytes(head_dim, nbits, group_size, page_size));
}

int hqq_kv_write(const hqq_kv_write_args* x) {
  KV_NEED(x, HQQ_ERR_INVALID_ARGUMENT, "args must not be NULL");
  hqq::kv::WriteArgs a{};
  const int st = check_cache(x->cache, &a.f);
  if (st != HQQ_OK) return st;
  KV_NEED(known_type(x->dtype), HQQ_ERR_INVALID_ARGUMENT, "dtype must be HQQ_KV_F16 or HQQ_KV_BF16");
  KV_NEED(x->n >= 0 && x->n <= (int64_t(1) << 30) / x->cache.num_kv_heads, HQQ_ERR_INVALID_ARGUMENT, "n out of range");
  KV_NEED(!x->k_echo == !x->v_echo, HQQ_ERR_INVALID_ARGUMENT, "k_echo and v_echo go together");
  if (x->n == 0) return HQQ_OK;
  KV_NEED(x->k && x->v && x->slots, HQQ_ERR_INVALID_ARGUMENT, "k, v and slots must not be NULL");
  KV_NEED(aligned16(x->k) && aligned16(x->v) && aligned16(x->k_echo) && aligned16(x->v_echo) &&
              reinterpret_cast<uintptr_t>(x->slots) % 8 == 0,
          HQQ_ERR_INVALID_ARGUMENT, "k, v and the echoes must be 16-byte aligned, slots 8-byte aligned");
  KV_NEED(x->k_token_stride >= 0 && x->k_head_stride >= 0 && x->v_token_stride >= 0 && x->v_head_stride >= 0 &&
              (x->k_token_stride | x->k_head_stride | x->v_token_stride | x->v_head_stride) % 8 == 0,
          HQQ_ERR_INVALID_ARGUMENT, "strides must be non-negative multiples of 8 elements");
  a.k = x->k, a.v = x->v, a.n = x->n;
  a.k_ts = x->k_token_stride, a.k_hs = x->k_head_stride, a.v_ts = x->v_token_stride, a.v_hs = x->v_head_stride;
  a.slots = x->slots;
  a.k_echo = x->k_echo, a.v_echo = x->v_echo;
  return device_status(hqq::kv::launch_kv_write(a, x->cache.head_dim, x->cache.nbits, x->cache.group_size, x->dtype,
                                                static_cast<hipStream_t>(x->stream)));
}

int hqq_kv_read(const hqq_kv_read_args* x) {
  KV_NEED(x, HQQ_ERR_INVALID_ARGUMENT, "args must not be NULL");
  hqq::kv::ReadArgs a{};
  const int st = check_cache(x->cache, &a.f);
  if (st != HQQ_OK) return st;
  KV_NEED(known_type(x->dtype), HQQ_ERR_INVALID_ARGUMENT, "dtype must be HQQ_KV_F16 or HQQ_KV_BF16");
  KV_NEED(x->n >= 0 && x->n <= (int64_t(1) << 30) / x->cache.num_kv_heads, HQQ_ERR_INVALID_ARGUMENT, "n out of range");
  if (x->n == 0) return HQQ_OK;
  KV_NEED(x->k && x->v && x->slots, HQQ_ERR_INVALID_ARGUMENT, "k, v and slots must not be NULL");
  KV_NEED(aligned16(x->k) && aligned16(x->v) && reinterpret_cast<uintptr_t>(x->slots) % 8 == 0, HQQ_ERR_INVALID_ARGUMENT,
          "k and v must be 16-byte aligned, slots 8-byte aligned");
  a.n = x->n, a.slots = x->slots, a.k = x->k, a.v = x->v;
  return device_status(hqq::kv::launch_kv_read(a, x->cache.head_dim, x->cache.nbits, x->cache.group_size, x->dtype,
                                               static_cast<hipStream_t>(x->stream)));
}

size_t hqq_kv_attention_workspace_bytes(const hqq_kv_attention_args* x) {
  Plan p;
  if (!x || plan_attention(x, true, &p) != HQQ_OK) return 0;
  return p.workspace;
}

int hqq_kv_attention(const hqq_kv_attention_args* x) {
  KV_NEED(x, HQQ_ERR_INVALID_ARGUMENT, "args must not be NULL");
  KV_NEED(x->prefix_len == 0 && !x->prefix_table, HQQ_ERR_INVALID_ARGUMENT,
          "a prefix goes to hqq_kv_attention_shared");
  return run_attention(x);
}

int hqq_kv_attention_shared(const hqq_kv_attention_args* x) {
  KV_NEED(x, HQQ_ERR_INVALID_ARGUMENT, "args must not be NULL");
  return run_attention(x);
}

}  // extern "C"
