// Multi-token and sparse attention over the packed cache, host side: the tile of query rows, the
// split of every sequence's context over the SMs, and the launch (the kernel: extend_kernel.cuh).
#include <algorithm>
#include <cmath>

#include "extend_kernel.cuh"

namespace tq {
namespace {

using namespace ext;

constexpr int kMaxSlots = 1024;     // partial records of a launch: blocks of threads that share items
constexpr int kSmemMax = 227 * 1024;
// A block of threads costs about this many tiles before its first and after its last one (query
// rotation, pipeline fill, joining the streams).
constexpr int kFixedTiles = 10;

// Query rows of a tile: the next of the kernel's sizes. Columns of the products and of the softmax that
// hold no row cost as much as those that do: a tile of tokens costs about 1.0 us at 16 rows, 1.4 at 48, 2.1 at 128.
int tile_rows(int rows) {
  return rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 48 ? 48 : rows <= 64 ? 64 : rows <= 96 ? 96 : 128;
}

// Upper bound of the partial records for any lengths and any head map.
size_t scratch_bytes(const tq_kv_cache* c, int64_t most_rows, int64_t most_tiles) {
  const int n = tile_rows(static_cast<int>(std::min<int64_t>(most_rows, 128)));
  const int64_t items = static_cast<int64_t>(c->batch) * c->n_kv_heads * ((most_rows + n - 1) / n);
  const int64_t slots = std::min<int64_t>(kMaxSlots, items * most_tiles);
  return static_cast<size_t>(slots) * n * kPartFloats * sizeof(float);
}

struct Plan {
  int n, row_tiles, blocks;
};

// Splits: sequence b's items (KV head x tile of query rows) get splits[b] blocks of threads each, so
// that no block has more than T tiles; for one and a few more rounds over the SMs the smallest T that
// fits is tried, and the one of the least rounds times (T + fixed cost) taken (joining: 3 tiles). The kernel divides an item's tiles by the lengths on the device: host lengths
// only shape the split.
Plan plan_extend(const tq_kv_cache* c, int n_tokens, int n_select, bool listed, int sms, ExtendArgs* a) {
  Plan p;
  int most = 0;
  for (int kv = 0; kv < c->n_kv_heads; ++kv) most = std::max(most, a->heads.start[kv + 1] - a->heads.start[kv]);
  const int64_t rows = static_cast<int64_t>(most) * n_tokens;
  p.n = tile_rows(static_cast<int>(std::min<int64_t>(rows, 128)));
  p.row_tiles = static_cast<int>((rows + p.n - 1) / p.n);
  const int64_t items = static_cast<int64_t>(c->n_kv_heads) * p.row_tiles;
  auto tiles_of = [&](int b) {
    const int len = std::max(1, c->len_host[b]);
    return listed ? (std::min(n_select, block_count(len)) + 1) / 2 : (len + kTile - 1) / kTile;
  };
  int longest = 1;
  for (int b = 0; b < c->batch; ++b) longest = std::max(longest, tiles_of(b));
  const bool one_by_one = c->batch <= kMaxList;
  const int64_t all = items * c->batch;
  auto splits_of = [&](int b, int T) { return ((one_by_one ? tiles_of(b) : longest) + T - 1) / T; };
  auto blocks_of = [&](int T) {
    if (!one_by_one) return all * splits_of(0, T);
    int64_t n = 0;
    for (int b = 0; b < c->batch; ++b) n += items * splits_of(b, T);
    return n;
  };
  const int64_t least = (all + sms - 1) / sms;   // rounds without splits
  int best_T = longest;
  double best = static_cast<double>(least) * (longest + kFixedTiles);
  for (int64_t rounds = least; all <= kMaxSlots && rounds < least + 4; ++rounds) {
    // the smallest T whose blocks of threads fit the rounds
    const int64_t room = std::min<int64_t>(rounds * sms, kMaxSlots);
    int T = 1;
    for (int above = longest; T < above;) {
      const int mid = (T + above) / 2;
      if (blocks_of(mid) <= room) above = mid;
      else T = mid + 1;
    }
    if (T == longest) continue;
    const int s = (longest + T - 1) / T;
    const double cost = static_cast<double>(rounds) * (T + kFixedTiles) + 3.0 + 0.1 * s;
    if (cost < best) { best = cost; best_T = T; }
  }
  // More items than SMs leave a last round that few SMs share: run whole rounds of unsplit items, and split
  // the rest over all SMs (448 items of 120 tiles: three rounds and 4 items split 37 ways, not seven
  // rounds of halves).
  a->tail_from = 0x7fffffff;
  a->tail_splits = 1;
  const int64_t rest = all % sms;
  if (one_by_one && all > sms && rest > 0 && rest <= items) {
    const int last = tiles_of(c->batch - 1), t = std::min<int>(last, sms / static_cast<int>(rest));
    const double cost = (all / sms) * (longest + kFixedTiles) + (last + t - 1) / t + kFixedTiles + 3.0;
    if (t > 1 && cost < best && all - rest + rest * t <= kMaxSlots) {
      best_T = longest;
      a->tail_from = static_cast<int>(items - rest);
      a->tail_splits = t;
    }
  }
  a->row_tiles = p.row_tiles;
  int64_t blocks = 0;
  if (one_by_one) {
    for (int b = 0; b < c->batch; ++b) {
      a->first[b] = static_cast<int>(blocks);
      a->splits[b] = static_cast<int16_t>(splits_of(b, best_T));
      blocks += items * a->splits[b];
    }
    if (a->tail_splits > 1) blocks += rest * (a->tail_splits - 1);
    a->first[c->batch] = static_cast<int>(blocks);
    a->uniform_splits = 1;
  } else {
    a->uniform_splits = splits_of(0, best_T);
    blocks = all * a->uniform_splits;
  }
  a->whole = blocks == all;
  p.blocks = blocks > 0x7fffffff ? -1 : static_cast<int>(blocks);
  return p;
}

template <int N>
tq_status launch_rows(ExtendArgs& a, int blocks, cudaStream_t st) {
  const int kcols = a.mode == TQ_MODE_PROD ? 2 * kD : kD;
  // tensor memory: 384 columns of key operands for up to 32 rows a stream, 256 beyond
  a.key_bufs = std::min(kMaxKeyBufs, (stream_rows(N) <= 32 ? 384 : 256) / (kcols / 2));
  a.scal_ring = a.key_bufs + 2 <= 4 ? 4 : 8;
  // a third value buffer where at least three stages of raw tiles remain
  a.value_bufs = smem_fixed(N, kcols, 3, a.scal_ring) + 3 * a.stage_bytes <= kSmemMax ? 3 : 2;
  const int fixed = smem_fixed(N, kcols, a.value_bufs, a.scal_ring);
  a.stages = std::min(kMaxStages, (kSmemMax - fixed) / a.stage_bytes);
  const int smem = fixed + a.stages * a.stage_bytes;
  if (cudaFuncSetAttribute(k_extend<N>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax) != cudaSuccess)
    return TQ_ECUDA;
  return launch_early(k_extend<N>, dim3(blocks), block_threads(N), smem, st, a) == cudaSuccess ? TQ_OK : TQ_ECUDA;
}

}  // namespace

size_t extend_scratch_bytes(const tq_kv_cache* c, int n_q_heads, int n_tokens) {
  return scratch_bytes(c, static_cast<int64_t>(n_q_heads) * n_tokens, (c->capacity + kTile - 1) / kTile);
}
size_t decode_blocks_scratch_bytes(const tq_kv_cache* c, int n_q_heads, int n_select) {
  return scratch_bytes(c, n_q_heads, (n_select + 1) / 2);
}

tq_status launch_extend(const tq_quantizer* q, const tq_kv_cache* c, const tq_heads& query, int q_dtype, int n_q_heads,
                        int n_tokens, int causal, const int32_t* head_map, float sm_scale, const int32_t* blocks,
                        int n_select, const tq_heads& out, int out_dtype, void* workspace, cudaStream_t st) {
  static thread_local ExtendArgs a;
  a.k_idx = c->keys.idx;
  a.k_sgn = c->keys.signs;
  a.k_nrm = reinterpret_cast<const uint8_t*>(c->keys.norms);
  a.v_q = c->values.q;
  a.v_par = reinterpret_cast<const uint8_t*>(c->values.params);
  a.len = c->len_dev;
  a.blocks = blocks;
  a.tab = q->dev;
  a.q = query.data;
  a.out = out.data;
  a.counters = static_cast<int*>(workspace);
  a.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kWorkspaceHeader);
  a.err = device_error_word();
  if (a.err == nullptr) return TQ_ECUDA;   // the kernel writes there when a wait runs out
  a.qb = query.stride_b; a.qh = query.stride_h; a.qt = query.stride_t;
  a.ob = out.stride_b; a.oh = out.stride_h; a.ot = out.stride_t;
  a.q_dtype = q_dtype;
  a.out_dtype = out_dtype;
  a.batch = c->batch;
  a.n_kv_heads = c->n_kv_heads;
  a.capacity = c->capacity;
  a.n_tokens = n_tokens;
  a.n_select = n_select;
  a.n_blocks = block_count(c->capacity);
  a.causal = causal != 0;
  a.mode = q->mode;
  a.bits0 = q->mode == TQ_MODE_PROD ? q->bits - 1 : q->mode == TQ_MODE_GROUPED ? q->bits + 1 : q->bits;
  a.bits1 = q->bits;
  a.idx_bytes = q->layout.idx_bytes;
  a.sgn_bytes = q->layout.sign_bytes;
  a.nrm_bytes = 2 * q->layout.n_norms;
  a.vbits = c->value_bits;
  a.vq_bytes = kD * c->value_bits / 8;
  a.stage_bytes = kTile * (a.idx_bytes + a.sgn_bytes + a.nrm_bytes + a.vq_bytes + 16);
  const float ch0 = q->mode == TQ_MODE_GROUPED ? 32.f : 128.f;
  a.key_scale0 = q->lv_scale[0] / std::sqrt(ch0);
  a.key_scale1 = q->lv_scale[1] / std::sqrt(96.f);
  // rho = r16 / n16 sqrt(pi/2) / d over the level side's factor and the sketch rows' 1/8
  a.sketch_ratio = 1.2533141373155003f / kD * 8.f / a.key_scale0;
  const float scale = sm_scale > 0.f ? sm_scale : 1.f / std::sqrt(static_cast<float>(kD));
  a.scale_log2 = scale * 1.4426950408889634074f;
  fill_head_lists(n_q_heads, c->n_kv_heads, head_map, &a.heads);
  const Plan p = plan_extend(c, n_tokens, n_select, blocks != nullptr, std::max(1, sm_count(q->device)), &a);
  if (p.blocks < 0) return TQ_EUNSUPPORTED;
  switch (p.n) {
    case 16: return launch_rows<16>(a, p.blocks, st);
    case 32: return launch_rows<32>(a, p.blocks, st);
    case 48: return launch_rows<48>(a, p.blocks, st);
    case 64: return launch_rows<64>(a, p.blocks, st);
    case 96: return launch_rows<96>(a, p.blocks, st);
    default: return launch_rows<128>(a, p.blocks, st);
  }
}

}  // namespace tq
