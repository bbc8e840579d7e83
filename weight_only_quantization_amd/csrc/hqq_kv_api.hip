// C ABI of the quantised key/value cache and its attention: argument checks, the choice of kernel and
// of key splits, the workspace.  Every check happens before anything is enqueued.
#include <math.h>

#include "hqq_internal.h"
#include "hqq_kv.h"

namespace {

using hqq::api_fail;
using hqq::kv::AttnArgs;
using hqq::kv::Format;
using hqq::kv::KeyList;

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
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

// A launch dimension takes fewer than 2^32 threads.
constexpr int64_t kThreads = (int64_t(1) << 32) - 512;

bool known_type(int dtype) { return dtype == HQQ_KV_F16 || dtype == HQQ_KV_BF16; }

// Most keys of a list.  The kernels count keys in 32 bits and look ahead of the last one: four steps of 256 keys in
// the stream, two tiles of 128 in the tiles, whose splits end up to 256 * 128 keys past it.
constexpr int64_t kMostKeys = INT32_MAX - (1 << 16);

// One attention call: its kernels' arguments, the row kernel of each list, the workspace.
enum { kStream16, kStream32, kTile };  // the stream with 16 or 32 rows a block, or tiles of 256 rows

struct Plan {
  AttnArgs a;
  int kind[2];
  bool join;
  int64_t part_rows, segment_words;
  size_t workspace;
};

// `lists` times that many rows (KV heads times sequences) over `keys` keys.  17 rows and more take 32 a block, which
// reads the keys for twice the rows, unless blocks of 16 are no more than the CUs: then those end sooner (16
// sequences of 2001 keys, 5 tokens, 32 heads on 8: 19.6 us with 16 rows, 22.7 with 32; 12 tokens: 35 and 24).
// More than 64 rows take tiles where there is work enough: a block of tiles takes 10 us to begin and end and 5 us
// per 128 keys, while streams spread few keys over more and shorter blocks.  Time of the call streamed and in tiles by the
// millions of pairs of a row and a key, over all KV heads and sequences: 0.36 (298 rows, 306 keys) 13 and 24 us, 3.0 (1290
// rows) 14 and 28, 6.9 (1856 rows) 13 and 27, 12.5 (2160 rows, 721 keys) 19 and 34, 12.6 (70 rows, 5623 keys, 32 heads) 29 and 28,
// 17.5 (1180 rows on a prefix of 3706) 42 and 52, 24 (6461 rows, 925 keys) 22 and 39.  Past the threshold it goes by the sizes, and
// tiles are taken where streams were the faster too: 31 (240 rows, 16379 keys) 64 and 55, 38 (1414 rows, 3399 keys) 79 and 52, but
// 36 (5516 rows) 40 and 59.  More than 2^16 rows take tiles whatever the keys (the threshold is at 384 keys there).
constexpr int64_t kStreamWork = int64_t(3) << 23, kStreamRows = 1 << 16;
int row_kernel(int64_t rows, int64_t lists, int64_t keys) {
  if (rows > 64 && (rows > kStreamRows || (keys > 0 ? keys : 1) * lists > kStreamWork / rows)) return kTile;
  return rows <= 16 || (rows + 15) / 16 * lists <= 256 ? kStream16 : kStream32;
}
int nt_of(int kind) { return kind == kStream16 ? 1 : 2; }
int64_t row_tiles(int64_t rows, int kind) {
  const int64_t of = kind == kStream16 ? 16 : kind == kStream32 ? 32 : 256;
  return (rows + of - 1) / of;
}

// Key splits of the tiles: enough blocks for the 256 CUs (a block fills one), at least 256 keys each.
void split_keys(KeyList* l, int64_t blocks) {
  const int64_t keys = l->max_len, most = (keys + 255) / 256;
  int64_t n = 256 / blocks;
  n = n > most ? most : n;
  n = n < 1 ? 1 : n;
  const int64_t chunk = ((keys + n - 1) / n + 127) / 128 * 128;
  l->chunk = (int)(chunk < 128 ? 128 : chunk);
  l->nsplit = (int)((keys + l->chunk - 1) / l->chunk);
  if (l->nsplit < 1) l->nsplit = 1;
}

// Longest own keys that one block streams for a pair; longer ones are shared out over the blocks.
constexpr int64_t kWholeKeys = 2048;

// Blocks of a stream launch: what fills the GPU, but at least two units each.
int stream_grid(const Plan& p, const hqq_kv_cache& c, int first, int lists) {
  int64_t units = 0;
  for (int i = first; i < first + lists; ++i) {
    const KeyList& l = p.a.list[i];
    const int64_t keys = hqq::kv::kStartUnits + (l.max_len + hqq::kv::kUnitKeys - 1) / hqq::kv::kUnitKeys;
    units += keys * l.num_seqs * p.a.f.hkv * row_tiles((int64_t)l.max_q * p.a.per, p.kind[i]);
  }
  const int64_t most = hqq::kv::stream_blocks(c.head_dim, c.group_size, nt_of(p.kind[first]));
  const int64_t n = (units + 1) / 2;
  return (int)(n > most ? most : n < 1 ? 1 : n);
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
  KV_NEED(x->max_len >= 0 && x->max_len <= kMostKeys, HQQ_ERR_INVALID_ARGUMENT, "max_len out of range");
  KV_NEED(x->prefix_len >= 0 && x->prefix_len <= kMostKeys, HQQ_ERR_INVALID_ARGUMENT, "prefix_len out of range");
  KV_NEED(x->table_cols >= 0 && x->table_cols * (int64_t)c.page_size <= INT32_MAX, HQQ_ERR_INVALID_ARGUMENT,
          "table_cols out of range");
  KV_NEED(x->table_stride >= 0, HQQ_ERR_INVALID_ARGUMENT, "table_stride must not be negative");
  KV_NEED(x->causal == 0 || x->causal == 1, HQQ_ERR_INVALID_ARGUMENT, "causal must be 0 or 1");
  KV_NEED(x->scale > 0.f && x->scale <= 3.0e38f, HQQ_ERR_INVALID_ARGUMENT, "scale must be finite and positive");

  *p = Plan{};
  AttnArgs& a = p->a;
  a.f = f;
  a.q = x->q;
  a.q_ts = x->q_token_stride;
  a.q_hs = x->q_head_stride;
  a.dtype = x->dtype;
  a.hq = x->num_q_heads;
  a.per = x->num_q_heads / c.num_kv_heads;
  a.total_q = x->total_q;
  a.scale_log2 = x->scale * 1.44269504089f;
  a.out = x->out;
  a.lse = x->lse;
  a.joined = x->prefix_len > 0;
  KeyList& own = a.list[0];
  // (no key is on a table without columns, but its first entry is loaded before the length is there: any readable one)
  own.table = x->table_cols ? x->page_table : x->seq_lens;
  own.table_stride = x->table_cols ? x->table_stride : 0;
  own.table_cols = (int)x->table_cols;
  own.lens = x->seq_lens;
  own.max_len = (int)x->max_len;
  own.cu_q = x->cu_q;
  own.num_seqs = (int)x->num_seqs;
  own.tq = x->num_seqs ? (int)(x->total_q / x->num_seqs) : 0;
  own.max_q = x->cu_q ? (int)x->max_q : own.tq;
  own.causal = x->causal;
  if (x->total_q == 0 || x->num_seqs == 0 || own.max_q == 0) return HQQ_OK;
  KV_NEED(x->num_seqs <= 65535, HQQ_ERR_UNSUPPORTED, "at most 65535 sequences in a call");
  KeyList& pre = a.list[1];
  if (a.joined) {
    pre.table = x->prefix_table;
    pre.table_cols = (int)((x->prefix_len + c.page_size - 1) / c.page_size);
    pre.fixed_len = pre.max_len = (int)x->prefix_len;
    pre.num_seqs = 1;
    pre.tq = pre.max_q = (int)x->total_q;
  }
  p->join = a.joined;
  for (int i = 0; i < (a.joined ? 2 : 1); ++i) {
    KeyList& l = a.list[i];
    const int64_t rows = (int64_t)l.max_q * a.per;
    p->kind[i] = row_kernel(rows, (int64_t)f.hkv * l.num_seqs, l.max_len);
    const int64_t tiles = row_tiles(rows, p->kind[i]), pairs = tiles * f.hkv * l.num_seqs;
    // (pairs times units may pass 64 bits)
    KV_NEED(tiles <= 65535 && pairs <= (int64_t(1) << 30) / (l.max_len / hqq::kv::kUnitKeys + hqq::kv::kStartUnits + 1),
            HQQ_ERR_UNSUPPORTED, "too many query rows and keys in a call");
    if (p->kind[i] == kTile) {
      l.tiled = 1;
      split_keys(&l, pairs);
      if (l.nsplit > 1) p->join = true;
    } else {
      const int64_t most = 16 * nt_of(p->kind[i]);
      l.cap = (int)(rows < most ? rows : most);
      // (own keys and a prefix that streams alike take one launch of shares)
      const bool alone = !a.joined || row_kernel(x->total_q * a.per, f.hkv, x->prefix_len) != p->kind[0];
      if (i == 0 && alone && l.max_len <= kWholeKeys) {
        l.tiled = l.nsplit = 1;
      } else {
        p->join = true;
      }
    }
  }
  // (blocks of 512 threads per KV head and sequence; four rows a block of 256 in the join)
  KV_NEED((int64_t)f.hkv * x->num_seqs <= kThreads / 512 && (!p->join || x->total_q * a.hq <= kThreads / 64),
          HQQ_ERR_UNSUPPORTED, "too many sequences or query rows in a call");
  if (!p->join) return HQQ_OK;
  // the lists' partial results, one after the other; the streams' segment lists behind them
  for (int i = 0; i < (a.joined ? 2 : 1); ++i) {
    KeyList& l = a.list[i];
    l.part0 = p->part_rows;
    const int64_t rows = (int64_t)l.max_q * a.per;
    if (l.tiled) {
      if (l.nsplit > 1 || a.joined) p->part_rows += l.nsplit * x->total_q * a.hq;
      continue;
    }
    const int64_t pairs = row_tiles(rows, p->kind[i]) * f.hkv * l.num_seqs;
    const int64_t grid = hqq::kv::stream_blocks(c.head_dim, c.group_size, nt_of(p->kind[i]));
    // (segments are counted over the pairs of both lists where one launch takes both)
    const int64_t segments = a.joined ? grid + pairs + (i ? row_tiles((int64_t)own.max_q * a.per, p->kind[0]) * f.hkv * own.num_seqs : 0)
                                      : 2 * grid;
    p->part_rows += segments * l.cap;
    p->segment_words += 2 * pairs;
  }
  p->workspace = (size_t)p->part_rows * (4 * (size_t)c.head_dim + sizeof(float2)) + (size_t)p->segment_words * 4;
  return HQQ_OK;
}

// The launches in front of the join, in order; launch(i) with the arguments set for list i (and the ones after it that share the
// launch).  Tiles of a prefix first (the longest work), then the streams: one launch where both lists stream alike.
template <typename F>
hipError_t each_launch(Plan* p, const hqq_kv_cache& c, F launch) {
  AttnArgs& a = p->a;
  const int lists = a.joined ? 2 : 1;
  hipError_t e = hipSuccess;
  for (int i = lists - 1; i >= 0 && e == hipSuccess; --i)
    if (p->kind[i] == kTile) e = launch(i);
  for (int i = 0; i < lists && e == hipSuccess; ++i) {
    if (p->kind[i] == kTile) continue;
    a.first_list = i;
    a.lists = i == 0 && lists == 2 && !a.list[0].tiled && p->kind[1] == p->kind[0] ? 2 : 1;
    a.blocks = a.list[i].tiled ? 0 : stream_grid(*p, c, i, a.lists);
    e = launch(i);
    i += a.lists - 1;
  }
  return e;
}

int run_attention(const hqq_kv_attention_args* x) {
  Plan p;
  const int st = plan_attention(x, false, &p);
  if (st != HQQ_OK) return st;
  AttnArgs& a = p.a;
  if (x->total_q == 0 || a.list[0].max_q == 0) return HQQ_OK;
  const hqq_kv_cache& c = x->cache;
  KV_NEED(x->q && aligned16(x->q) && x->out && aligned16(x->out), HQQ_ERR_INVALID_ARGUMENT,
          "q and out must be 16-byte aligned pointers");
  KV_NEED(x->q_token_stride >= 0 && x->q_head_stride >= 0 && x->q_token_stride % 8 == 0 && x->q_head_stride % 8 == 0,
          HQQ_ERR_INVALID_ARGUMENT, "q strides must be non-negative multiples of 8 elements");
  KV_NEED(x->seq_lens, HQQ_ERR_INVALID_ARGUMENT, "seq_lens must not be NULL");
  KV_NEED(x->page_table || x->table_cols == 0, HQQ_ERR_INVALID_ARGUMENT, "page_table must not be NULL");
  KV_NEED(!a.joined || x->prefix_table, HQQ_ERR_INVALID_ARGUMENT, "prefix_table must not be NULL");
  // (scalar loads drop the low address bits)
  KV_NEED(aligned4(x->seq_lens) && aligned4(x->page_table) && aligned4(x->cu_q) && aligned4(x->prefix_table) && aligned4(x->lse),
          HQQ_ERR_INVALID_ARGUMENT, "seq_lens, the page tables, cu_q and lse must be 4-byte aligned");
  if (p.workspace) {
    KV_NEED(x->workspace && x->workspace_bytes >= p.workspace, HQQ_ERR_WORKSPACE,
            "workspace missing or smaller than hqq_kv_attention_workspace_bytes");
    KV_NEED(aligned16(x->workspace), HQQ_ERR_INVALID_ARGUMENT, "workspace must be 16-byte aligned");
    a.part_o = static_cast<float*>(x->workspace);
    a.part_ml = reinterpret_cast<float2*>(a.part_o + p.part_rows * c.head_dim);
    int32_t* words = reinterpret_cast<int32_t*>(a.part_ml + p.part_rows);
    for (int i = 0; i < (a.joined ? 2 : 1); ++i) {
      if (a.list[i].tiled) continue;
      KeyList& l = a.list[i];
      l.segments = words;
      words += 2 * row_tiles((int64_t)l.max_q * a.per, p.kind[i]) * a.f.hkv * l.num_seqs;
    }
  }
  hipStream_t stream = static_cast<hipStream_t>(x->stream);
  const int D = c.head_dim, bits = c.nbits, gs = c.group_size;
  hipError_t e = each_launch(&p, c, [&](int i) {
    return p.kind[i] == kTile ? hqq::kv::launch_kv_tile(a, i, D, bits, gs, stream)
                              : hqq::kv::launch_kv_stream(a, D, bits, gs, nt_of(p.kind[i]), stream);
  });
  if (e == hipSuccess && p.join) e = hqq::kv::launch_kv_join(a, D, nt_of(p.kind[0]), nt_of(p.kind[1]), stream);
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
  KV_NEED((x->n + 3) * x->cache.num_kv_heads * (x->cache.head_dim / 8) <= kThreads, HQQ_ERR_UNSUPPORTED,
          "too many tokens in a call");
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
  KV_NEED((x->n + 3) * x->cache.num_kv_heads * (x->cache.head_dim / 8) <= kThreads, HQQ_ERR_UNSUPPORTED,
          "too many tokens in a call");
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

int hqq_kv_attention_way(const hqq_kv_attention_args* x, int32_t way[7]) {
  Plan p;
  for (int i = 0; i < 7; ++i) way[i] = 0;
  const int st = plan_attention(x, false, &p);
  if (st != HQQ_OK || x->total_q == 0 || p.a.list[0].max_q == 0) return st;
  (void)each_launch(&p, x->cache, [&](int i) {
    for (int l = i; l < i + (p.kind[i] == kTile ? 1 : p.a.lists); ++l) {
      way[3 * l] = p.kind[l] == kTile ? 256 : 16 * nt_of(p.kind[l]);
      way[3 * l + 1] = p.kind[l] == kTile ? -1 : hqq::kv::stream_mode(p.a, nt_of(p.kind[l]));
      way[3 * l + 2] = p.kind[l] == kTile ? p.a.list[l].nsplit : 1;
    }
    return hipSuccess;
  });
  way[6] = p.join;
  return HQQ_OK;
}

}  // extern "C"
