// C ABI of libtq (include/tq.h): argument checks on the host, then kernel launches.
#include <algorithm>
#include <cmath>
#include <cstdlib>
#include <cstring>
#include <new>

#include "tq_internal.h"

namespace tq {

void fill_head_lists(int n_q_heads, int n_kv_heads, const int32_t* head_map, HeadLists* out) {
  int n = 0;
  const int per = head_map ? 0 : n_q_heads / n_kv_heads;
  for (int kv = 0; kv < n_kv_heads; ++kv) {
    out->start[kv] = static_cast<int16_t>(n);
    if (head_map) {
      for (int h = 0; h < n_q_heads; ++h)
        if (head_map[h] == kv) out->head[n++] = static_cast<int16_t>(h);
    } else {
      for (int i = 0; i < per; ++i, ++n) out->head[n] = static_cast<int16_t>(n);
    }
  }
  out->start[n_kv_heads] = static_cast<int16_t>(n);
}

int sm_count(int device) {
  static int cached[64] = {0};
  if (device < 0 || device >= 64) return 148;
  if (cached[device] == 0) {
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, device) != cudaSuccess || n <= 0)
      n = 148;
    cached[device] = n;
  }
  return cached[device];
}

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int elem_size(int dtype) {
  return dtype == TQ_F32 ? 4 : (dtype == TQ_BF16 || dtype == TQ_F16) ? 2 : 0;
}

tq_status check_rows(const void* x, int dtype, int64_t n_rows, int64_t ld) {
  if (n_rows < 0) return TQ_EINVAL;
  if (dtype != TQ_F32 && dtype != TQ_BF16) return TQ_EUNSUPPORTED;
  if (ld < kD || (ld * elem_size(dtype)) % 16 != 0) return TQ_EINVAL;
  if (n_rows > 0 && (x == nullptr || !aligned16(x))) return TQ_EINVAL;
  return TQ_OK;
}

tq_status check_key_planes(const tq_quantizer* q, const tq_key_planes& p) {
  if (!p.idx || !p.norms) return TQ_EINVAL;
  if (!aligned16(p.idx) || (reinterpret_cast<uintptr_t>(p.norms) & 3u)) return TQ_EINVAL;
  if (q->mode == TQ_MODE_PROD) {
    if (!p.signs || !aligned16(p.signs)) return TQ_EINVAL;
  }
  return TQ_OK;
}

tq_status check_cache(const tq_quantizer* q, const tq_kv_cache* c) {
  if (!c) return TQ_EINVAL;
  if (c->batch <= 0 || c->n_kv_heads <= 0 || c->capacity <= 0 || c->capacity % 16) return TQ_EINVAL;
  if (c->d != kD) return TQ_EUNSUPPORTED;
  if (!c->len_dev || !c->len_host) return TQ_EINVAL;
  if (check_key_planes(q, c->keys) != TQ_OK) return TQ_EINVAL;
  if (!aligned16(c->keys.norms)) return TQ_EINVAL;
  if (c->value_bits != 0) {
    if (c->value_bits != 2 && c->value_bits != 4) return TQ_EUNSUPPORTED;
    if (c->value_group != 32) return TQ_EUNSUPPORTED;
    if (!c->values.q || !c->values.params || !aligned16(c->values.q) || !aligned16(c->values.params))
      return TQ_EINVAL;
  }
  for (int b = 0; b < c->batch; ++b)
    if (c->len_host[b] < 0 || c->len_host[b] > c->capacity) return TQ_EINVAL;
  return TQ_OK;
}

}  // namespace
}  // namespace tq

using namespace tq;

extern "C" {

int tq_abi_version(void) { return TQ_ABI_VERSION; }

tq_status tq_sync_status(void* stream) {
  return take_device_error(static_cast<cudaStream_t>(stream));
}

tq_status tq_selftest_bounded_wait(uint32_t limit_us, void* stream) {
  if (limit_us == 0 || limit_us > 2000000u) return TQ_EINVAL;
  return launch_selftest_wait(limit_us, static_cast<cudaStream_t>(stream));
}

const char* tq_status_string(tq_status s) {
  switch (s) {
    case TQ_OK: return "ok";
    case TQ_EINVAL: return "invalid argument";
    case TQ_EUNSUPPORTED: return "unsupported configuration";
    case TQ_ECAPACITY: return "cache capacity exceeded";
    case TQ_ENOMEM: return "out of memory";
    case TQ_ECUDA: return "CUDA error";
    case TQ_ETIMEOUT: return "device wait timed out";
    case TQ_ETOOLARGE: return "problem exceeds the built-in decode scratch";
  }
  return "unknown status";
}

tq_status tq_host_tables(int d, int bits, int mode, uint64_t seed, const int32_t* outliers,
                         int n_outlier, double* centroids, double* thresholds, int8_t* signs,
                         int32_t* channels, uint16_t* s_rot_fp16) {
  HostTables* t = new (std::nothrow) HostTables;
  if (!t) return TQ_ENOMEM;
  tq_key_layout_t lay;
  const tq_status st = build_host_tables(d, bits, mode, seed, outliers, n_outlier, t, &lay);
  if (st == TQ_OK) {
    if (centroids) std::memcpy(centroids, t->cent, sizeof(t->cent));
    if (thresholds) std::memcpy(thresholds, t->thr, sizeof(t->thr));
    if (signs) std::memcpy(signs, t->signs, sizeof(t->signs));
    if (channels) std::memcpy(channels, t->chan, sizeof(t->chan));
    if (s_rot_fp16 && mode == TQ_MODE_PROD) std::memcpy(s_rot_fp16, t->s_rot, sizeof(t->s_rot));
  }
  delete t;
  return st;
}

namespace {
// Store schedule of the grouped kernel's gather (DevTables::gsched). Lane l stores natural
// channel c = 4l + i to chain position pos[c], a 2-byte slot in bank (pos[c] / 2) mod 32 of a
// row. Lanes x banks with an edge per (l, i) is a 4-regular bipartite multigraph (each bank
// holds chain positions 2b, 2b + 1, 2b + 64, 2b + 65), so it splits into 4 perfect matchings
// (Koenig); each round takes one, found by augmenting paths (Kuhn), and removes it.
bool gather_augment(int l, const int (&bank)[32][4], const bool (&used)[32][4], bool (&seen)[32],
                    int (&lane_of_bank)[32], int (&opt_of_lane)[32]) {
  for (int i = 0; i < 4; ++i) {
    if (used[l][i]) continue;
    const int b = bank[l][i];
    if (seen[b]) continue;
    seen[b] = true;
    if (lane_of_bank[b] < 0 ||
        gather_augment(lane_of_bank[b], bank, used, seen, lane_of_bank, opt_of_lane)) {
      lane_of_bank[b] = l;
      opt_of_lane[l] = i;
      return true;
    }
  }
  return false;
}

void gather_schedule(const int32_t (&chan)[tq::kD], uint8_t (&sched)[32][4]) {
  int pos[tq::kD];
  for (int p = 0; p < tq::kD; ++p) pos[chan[p]] = p;
  int bank[32][4];
  for (int l = 0; l < 32; ++l)
    for (int i = 0; i < 4; ++i) bank[l][i] = (pos[4 * l + i] >> 1) & 31;
  bool used[32][4] = {};
  for (int k = 0; k < 4; ++k) {
    int lane_of_bank[32], opt_of_lane[32];
    for (int j = 0; j < 32; ++j) lane_of_bank[j] = opt_of_lane[j] = -1;
    for (int l = 0; l < 32; ++l) {
      bool seen[32] = {};
      gather_augment(l, bank, used, seen, lane_of_bank, opt_of_lane);
    }
    for (int l = 0; l < 32; ++l) {
      int i = opt_of_lane[l];
      if (i < 0)  // cannot happen for a regular multigraph; any unused channel stays correct
        for (i = 0; used[l][i]; ++i) {}
      used[l][i] = true;
      sched[l][k] = static_cast<uint8_t>(i);
    }
  }
}
// The byte pools of DevTables::lv_lo / lv_hi for the codebook `cent` (2^bits mirrored levels). Of
// 4096 factors in [1, 2) the one is taken whose products with the levels are nearest to fp16
// numbers, so that rounding the levels costs next to nothing (a level alone may be 2^-12 off).
float level_bytes(const double* cent, int bits, uint32_t (&lo)[2], uint32_t (&hi)[2]) {
  const int n = 1 << bits, half = n / 2;
  double best = 1.0, best_err = 1e300;
  for (int g = 0; g < 4096; ++g) {
    const double f = 1.0 + g / 4096.0;
    double err = 0.0;
    for (int k = half; k < n; ++k) {
      const double x = cent[k] * f;
      const double ulp = std::ldexp(1.0, std::ilogb(x) - 10);   // fp16 spacing at x
      err = std::max(err, std::fabs(std::nearbyint(x / ulp) * ulp - x) / x);
    }
    if (err < best_err) { best_err = err; best = f; }
  }
  lo[0] = lo[1] = hi[0] = hi[1] = 0;
  if (bits == 1) {
    const uint32_t h = float_to_half_bits_rn(cent[1] * best);
    lo[0] = h | (h << 16);
  } else if (bits == 2) {
    for (int k = 0; k < n; ++k) lo[k >> 1] |= static_cast<uint32_t>(float_to_half_bits_rn(cent[k] * best)) << (16 * (k & 1));
  } else {
    const int first = bits == 4 ? half : 0, count = bits == 4 ? half : n;
    for (int k = 0; k < count; ++k) {
      const uint32_t h = float_to_half_bits_rn(cent[first + k] * best);
      lo[k >> 2] |= (h & 0xffu) << (8 * (k & 3));
      hi[k >> 2] |= (h >> 8) << (8 * (k & 3));
    }
  }
  return static_cast<float>(1.0 / best);
}
}  // namespace

static tq_status build_quantizer(int d, int bits, int mode, uint64_t seed,
                                 const int32_t* outlier_channels, int n_outlier, bool device,
                                 tq_quantizer** out) {
  if (!out) return TQ_EINVAL;
  *out = nullptr;
  tq_quantizer* q = new (std::nothrow) tq_quantizer;
  if (!q) return TQ_ENOMEM;
  std::memset(q, 0, sizeof(*q));
  tq_status st = build_host_tables(d, bits, mode, seed, outlier_channels, n_outlier, &q->host,
                                   &q->layout);
  if (st != TQ_OK) {
    delete q;
    return st;
  }
  q->d = d;
  q->bits = bits;
  q->mode = mode;
  q->seed = seed;
  q->device = -1;
  if (!device) {  // host-only: layouts and argument checks, no device tables
    *out = q;
    return TQ_OK;
  }

  DevTables* h = new (std::nothrow) DevTables;
  if (!h) {
    delete q;
    return TQ_ENOMEM;
  }
  std::memset(h, 0, sizeof(*h));
  const int nl0 = mode == TQ_MODE_MSE ? (1 << bits) : mode == TQ_MODE_PROD ? (1 << (bits - 1)) : (1 << (bits + 1));
  for (int k = 0; k < nl0; ++k) h->cent[0][k] = static_cast<float>(q->host.cent[0][k]);
  for (int k = 0; k + 1 < nl0; ++k) h->thr[0][k] = static_cast<float>(q->host.thr[0][k]);
  if (mode == TQ_MODE_GROUPED) {
    const int nl1 = 1 << bits;
    for (int k = 0; k < nl1; ++k) h->cent[1][k] = static_cast<float>(q->host.cent[1][k]);
    for (int k = 0; k + 1 < nl1; ++k) h->thr[1][k] = static_cast<float>(q->host.thr[1][k]);
  }
  for (int j = 0; j < kD; ++j) {
    if (q->host.signs[j] < 0) h->sign_bits[j >> 5] |= 1u << (j & 31);
    h->chan[j] = static_cast<uint8_t>(q->host.chan[j]);
  }
  if (mode == TQ_MODE_PROD) {
    for (int r = 0; r < kD; ++r)
      for (int c = 0; c < kD; ++c) {
        const uint16_t v = q->host.s_rot[r * kD + c];
        std::memcpy(&h->s_rot[r * kD + c], &v, 2);
        std::memcpy(&h->s_rot_t[c * kD + r], &v, 2);
      }
    for (int j = 0; j < kD; ++j)
      for (int kk = 0; kk < kD; ++kk) {
        const int col = (kk >> 1) + 64 * (kk & 1);
        const size_t off = static_cast<size_t>(j >> 3) * 1024 + (kk >> 3) * 64 + (j & 7) * 8 + (kk & 7);
        h->s_umma[off] = q->host.s_rot[j * kD + col];
      }
  }
  if (mode == TQ_MODE_GROUPED) gather_schedule(q->host.chan, h->gsched);
  for (int j = 0; j < kD; ++j)
    for (int p = 0; p < kD; ++p) {   // coordinate j of the rotated row, position p of the group order
      const bool block = mode != TQ_MODE_GROUPED || (j >> 5) == (p >> 5);
      const int bits = mode == TQ_MODE_GROUPED ? (j & p & 31) : (j & p);
      const bool neg = (__builtin_popcount(bits) & 1) != (q->host.signs[p] < 0);
      const int c = q->host.chan[p];
      const size_t off = static_cast<size_t>(j >> 3) * 1024 + (c >> 3) * 64 + (j & 7) * 8 + (c & 7);
      h->r_umma[0][off] = !block ? 0 : neg ? 0xbc00 : 0x3c00;
      h->r_umma[1][off] = !block ? 0 : neg ? 0xbf80 : 0x3f80;
    }
  const int bits0 = mode == TQ_MODE_PROD ? bits - 1 : mode == TQ_MODE_GROUPED ? bits + 1 : bits;
  h->lv_scale[0] = q->lv_scale[0] = level_bytes(q->host.cent[0], bits0, h->lv_lo[0], h->lv_hi[0]);
  if (mode == TQ_MODE_GROUPED)
    h->lv_scale[1] = q->lv_scale[1] = level_bytes(q->host.cent[1], bits, h->lv_lo[1], h->lv_hi[1]);
  for (int qq = 0; qq < kD / 2; ++qq)
    h->pair_mask[qq] = (q->host.signs[2 * qq] < 0 ? 1u << 15 : 0u) |
                       (q->host.signs[2 * qq + 1] < 0 ? 1u << 31 : 0u);
  if (cudaGetDevice(&q->device) != cudaSuccess) {
    delete h;
    delete q;
    return TQ_ECUDA;
  }
  if (cudaMalloc(&q->dev, sizeof(DevTables)) != cudaSuccess) {
    delete h;
    delete q;
    return TQ_ENOMEM;
  }
  st = cudaMemcpy(q->dev, h, sizeof(DevTables), cudaMemcpyHostToDevice) == cudaSuccess ? TQ_OK : TQ_ECUDA;
  delete h;
  if (st != TQ_OK) {
    cudaFree(q->dev);
    delete q;
    return st;
  }
  *out = q;
  return TQ_OK;
}

tq_status tq_build_codebook(int d, int bits, int mode, uint64_t seed,
                            const int32_t* outlier_channels, int n_outlier, tq_quantizer** out) {
  return build_quantizer(d, bits, mode, seed, outlier_channels, n_outlier, true, out);
}

tq_status tq_build_codebook_host(int d, int bits, int mode, uint64_t seed,
                                 const int32_t* outlier_channels, int n_outlier,
                                 tq_quantizer** out) {
  return build_quantizer(d, bits, mode, seed, outlier_channels, n_outlier, false, out);
}

void tq_free(tq_quantizer* q) {
  if (!q) return;
  if (q->dev) cudaFree(q->dev);
  delete q;
}

tq_status tq_key_layout(const tq_quantizer* q, tq_key_layout_t* out) {
  if (!q || !out) return TQ_EINVAL;
  *out = q->layout;
  return TQ_OK;
}

tq_status tq_quantize_keys(const tq_quantizer* q, const void* x, int dtype, int64_t n_rows,
                           int64_t ld, tq_key_planes out, void* stream) {
  if (!q) return TQ_EINVAL;
  tq_status st = check_rows(x, dtype, n_rows, ld);
  if (st != TQ_OK) return st;
  if (n_rows == 0) return TQ_OK;
  if ((st = check_key_planes(q, out)) != TQ_OK) return st;
  if (q->mode != TQ_MODE_GROUPED && (reinterpret_cast<uintptr_t>(out.norms) & 3u)) return TQ_EINVAL;
  if (!q->dev) return TQ_ECUDA;
  return launch_quantize_keys(q, x, dtype, n_rows, ld, out, RowMap{nullptr, 0, 0, 0},
                              static_cast<cudaStream_t>(stream));
}

tq_status tq_dequantize_keys(const tq_quantizer* q, tq_key_planes planes, int64_t n_rows,
                             void* out, int out_dtype, int64_t ld, void* stream) {
  if (!q) return TQ_EINVAL;
  tq_status st = check_rows(out, out_dtype, n_rows, ld);
  if (st != TQ_OK) return st;
  if (n_rows == 0) return TQ_OK;
  if ((st = check_key_planes(q, planes)) != TQ_OK) return st;
  if (!q->dev) return TQ_ECUDA;
  return launch_dequantize_keys(q, planes, n_rows, out, out_dtype, ld,
                                static_cast<cudaStream_t>(stream));
}

tq_status tq_quantize_values(const void* v, int dtype, int64_t n_rows, int64_t ld, int d, int bits,
                             int group, tq_value_planes out, void* stream) {
  if (d != kD) return TQ_EUNSUPPORTED;
  if (bits != 2 && bits != 4) return TQ_EUNSUPPORTED;
  if (group != 32) return TQ_EUNSUPPORTED;
  tq_status st = check_rows(v, dtype, n_rows, ld);
  if (st != TQ_OK) return st;
  if (n_rows == 0) return TQ_OK;
  if (!out.q || !out.params || (reinterpret_cast<uintptr_t>(out.params) & 3u) ||
      (reinterpret_cast<uintptr_t>(out.q) & 3u))
    return TQ_EINVAL;
  return launch_quantize_values(v, dtype, n_rows, ld, bits, out, RowMap{nullptr, 0, 0, 0},
                                static_cast<cudaStream_t>(stream));
}

// Argument checks of tq_append (nothing launched).
static tq_status check_append(const tq_quantizer* q, const tq_kv_cache* c, const void* k_new,
                              const void* v_new, int dtype, int n_tokens) {
  if (!q) return TQ_EINVAL;
  tq_status st = check_cache(q, c);
  if (st != TQ_OK) return st;
  if (n_tokens < 0) return TQ_EINVAL;
  if (n_tokens == 0) return TQ_OK;
  if (dtype != TQ_F32 && dtype != TQ_BF16) return TQ_EUNSUPPORTED;
  if (!k_new || !aligned16(k_new)) return TQ_EINVAL;
  if (c->value_bits != 0 && (!v_new || !aligned16(v_new))) return TQ_EINVAL;
  if (c->value_bits == 0 && v_new) return TQ_EINVAL;
  for (int b = 0; b < c->batch; ++b)
    if (static_cast<int64_t>(c->len_host[b]) + n_tokens > c->capacity) return TQ_ECAPACITY;
  return TQ_OK;
}

tq_status tq_append(const tq_quantizer* q, tq_kv_cache* c, const void* k_new, const void* v_new,
                    int dtype, int n_tokens, void* stream) {
  tq_status st = check_append(q, c, k_new, v_new, dtype, n_tokens);
  if (st != TQ_OK || n_tokens == 0) return st;
  if (!q->dev) return TQ_ECUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (append_fused_ok(q, c, n_tokens)) {
    if ((st = launch_append_fused(q, c, k_new, v_new, dtype, n_tokens, s)) != TQ_OK) return st;
    for (int b = 0; b < c->batch; ++b) c->len_host[b] += n_tokens;
    return TQ_OK;
  }
  const int64_t rows = static_cast<int64_t>(c->batch) * c->n_kv_heads * n_tokens;
  const RowMap map{c->len_dev, c->n_kv_heads, n_tokens, c->capacity};
  if ((st = launch_quantize_keys(q, k_new, dtype, rows, kD, c->keys, map, s)) != TQ_OK) return st;
  if (c->value_bits != 0) {
    if ((st = launch_quantize_values(v_new, dtype, rows, kD, c->value_bits, c->values, map, s)) != TQ_OK)
      return st;
  }
  if ((st = launch_advance_len(c->len_dev, c->batch, n_tokens, s)) != TQ_OK) return st;
  for (int b = 0; b < c->batch; ++b) c->len_host[b] += n_tokens;
  return TQ_OK;
}

tq_status tq_decode_workspace_bytes(const tq_kv_cache* c, int n_q_heads, size_t* bytes) {
  if (!c || !bytes || n_q_heads <= 0 || c->batch <= 0 || c->capacity <= 0) return TQ_EINVAL;
  *bytes = decode_workspace_bytes(c->batch, n_q_heads, c->capacity);
  return TQ_OK;
}

// Argument checks of every decode entry point (the workspace apart: check_workspace).
static tq_status check_decode_args(const tq_quantizer* q, const tq_kv_cache* c, const void* qv,
                                   int q_dtype, int n_q_heads, const int32_t* head_map,
                                   void* out, int out_dtype, float* scores, int64_t scores_ld) {
  if (!q) return TQ_EINVAL;
  tq_status st = check_cache(q, c);
  if (st != TQ_OK) return st;
  if (n_q_heads <= 0 || n_q_heads > 512) return TQ_EINVAL;
  if (q_dtype != TQ_F32 && q_dtype != TQ_BF16) return TQ_EUNSUPPORTED;
  if (!qv || !aligned16(qv)) return TQ_EINVAL;
  if (head_map) {
    for (int h = 0; h < n_q_heads; ++h)
      if (head_map[h] < 0 || head_map[h] >= c->n_kv_heads) return TQ_EINVAL;
  } else if (n_q_heads % c->n_kv_heads != 0) {
    return TQ_EINVAL;
  }
  if (c->value_bits != 0) {
    if (!out || !aligned16(out)) return TQ_EINVAL;
    if (out_dtype != TQ_F32 && out_dtype != TQ_BF16) return TQ_EUNSUPPORTED;
  } else if (out) {
    return TQ_EINVAL;
  }
  int max_len = 0;
  for (int b = 0; b < c->batch; ++b) max_len = c->len_host[b] > max_len ? c->len_host[b] : max_len;
  if (scores && scores_ld < max_len) return TQ_EINVAL;
  return TQ_OK;
}

static tq_status check_workspace(const tq_kv_cache* c, int n_q_heads, const void* workspace,
                                 size_t workspace_bytes) {
  if (!workspace || !aligned16(workspace)) return TQ_EINVAL;
  if (workspace_bytes < decode_workspace_bytes(c->batch, n_q_heads, c->capacity)) return TQ_EINVAL;
  return TQ_OK;
}

tq_status tq_decode_attention(const tq_quantizer* q, const tq_kv_cache* c, const void* qv,
                              int q_dtype, int n_q_heads, const int32_t* head_map, float sm_scale,
                              void* out, int out_dtype, float* scores, int64_t scores_ld,
                              void* workspace, size_t workspace_bytes, void* stream) {
  tq_status st = check_decode_args(q, c, qv, q_dtype, n_q_heads, head_map, out, out_dtype,
                                   scores, scores_ld);
  if (st != TQ_OK) return st;
  if ((st = check_workspace(c, n_q_heads, workspace, workspace_bytes)) != TQ_OK) return st;
  return launch_decode(q, c, qv, q_dtype, n_q_heads, head_map, sm_scale, out, out_dtype, scores,
                       scores_ld, nullptr, workspace, workspace_bytes, /*pdl=*/false,
                       static_cast<cudaStream_t>(stream));
}

tq_status tq_append_decode(const tq_quantizer* q, tq_kv_cache* c, const void* k_new,
                           const void* v_new, int kv_dtype, int n_tokens, const void* qv,
                           int q_dtype, int n_q_heads, const int32_t* head_map, float sm_scale,
                           void* out, int out_dtype, float* scores, int64_t scores_ld,
                           void* workspace, size_t workspace_bytes, void* stream) {
  tq_status st = check_append(q, c, k_new, v_new, kv_dtype, n_tokens);
  if (st != TQ_OK) return st;
  if ((st = check_decode_args(q, c, qv, q_dtype, n_q_heads, head_map, out, out_dtype, scores,
                              scores_ld)) != TQ_OK)
    return st;
  if (scores) {  // the scores cover the lengths after the append
    for (int b = 0; b < c->batch; ++b)
      if (static_cast<int64_t>(c->len_host[b]) + n_tokens > scores_ld) return TQ_EINVAL;
  }
  if ((st = check_workspace(c, n_q_heads, workspace, workspace_bytes)) != TQ_OK) return st;
  // the decode's head grouping is checked before the append, so that an error leaves the
  // cache as it was
  if ((st = check_decode_plan(q, c, n_q_heads, head_map, n_tokens)) != TQ_OK) return st;
  if (!q->dev) return TQ_ECUDA;
  if ((st = tq_append(q, c, k_new, v_new, kv_dtype, n_tokens, stream)) != TQ_OK) return st;
  // the kernel just launched is the library's append, ordered after the query's producer:
  // the decode may start its query-only prologue while the append runs
  return launch_decode(q, c, qv, q_dtype, n_q_heads, head_map, sm_scale, out, out_dtype, scores,
                       scores_ld, nullptr, workspace, workspace_bytes, /*pdl=*/true,
                       static_cast<cudaStream_t>(stream));
}

tq_status tq_decode_attention_partial(const tq_quantizer* q, const tq_kv_cache* c, const void* qv,
                                      int q_dtype, int n_q_heads, const int32_t* head_map,
                                      float sm_scale, float* part, void* workspace,
                                      size_t workspace_bytes, void* stream) {
  if (!q || !c) return TQ_EINVAL;
  if (c->value_bits == 0) return TQ_EINVAL;  // a partial carries o: the cache needs values
  if (!part || !aligned16(part)) return TQ_EINVAL;
  // every other check is tq_decode_attention's (with a stand-in output pointer)
  tq_status st = check_decode_args(q, c, qv, q_dtype, n_q_heads, head_map, part, TQ_F32,
                                   nullptr, 0);
  if (st != TQ_OK) return st;
  if ((st = check_workspace(c, n_q_heads, workspace, workspace_bytes)) != TQ_OK) return st;
  return launch_decode(q, c, qv, q_dtype, n_q_heads, head_map, sm_scale, nullptr, TQ_F32, nullptr,
                       0, part, workspace, workspace_bytes, /*pdl=*/false,
                       static_cast<cudaStream_t>(stream));
}

tq_status tq_set_decode_policy(int policy, int* previous) {
  return set_decode_policy(policy, previous);
}

tq_status tq_merge_partials(const float* parts, int n_parts, int batch, int n_q_heads, void* out,
                            int out_dtype, void* stream) {
  if (n_parts < 1 || n_parts > 65536 || batch <= 0 || n_q_heads <= 0 || n_q_heads > 512)
    return TQ_EINVAL;
  if (out_dtype != TQ_F32 && out_dtype != TQ_BF16) return TQ_EUNSUPPORTED;
  if (!parts || !aligned16(parts) || !out || !aligned16(out)) return TQ_EINVAL;
  return launch_merge_partials(parts, n_parts, static_cast<int64_t>(batch) * n_q_heads, out,
                               out_dtype, static_cast<cudaStream_t>(stream));
}

tq_status tq_decode_attention_noalloc(const tq_quantizer* q, const tq_kv_cache* c,
                                      const void* qv, int q_dtype, int n_q_heads,
                                      const int32_t* head_map, float sm_scale, void* out,
                                      int out_dtype, float* scores, int64_t scores_ld,
                                      void* stream) {
  tq_status st = check_decode_args(q, c, qv, q_dtype, n_q_heads, head_map, out, out_dtype,
                                   scores, scores_ld);
  if (st != TQ_OK) return st;
  if ((st = check_decode_plan(q, c, n_q_heads, head_map, 0)) != TQ_OK) return st;
  if (!q->dev) return TQ_ECUDA;
  return launch_decode_noalloc(q, c, qv, q_dtype, n_q_heads, head_map, sm_scale, out, out_dtype,
                               scores, scores_ld, static_cast<cudaStream_t>(stream));
}

// ------------------------------------------------- operators around the cache
namespace {

bool known_dtype(int dtype) { return dtype == TQ_F32 || dtype == TQ_BF16 || dtype == TQ_F16; }

// A (batch, heads, tokens, d) view: base and every stride that is stepped along on 16 bytes.
tq_status check_view(const tq_heads& x, int dtype, int batch, int n_heads, int n_tokens) {
  if (!x.data || !aligned16(x.data)) return TQ_EINVAL;
  const int64_t unit = 16 / elem_size(dtype);
  if ((batch > 1 && x.stride_b % unit) || (n_heads > 1 && x.stride_h % unit) || (n_tokens > 1 && x.stride_t % unit))
    return TQ_EINVAL;
  return TQ_OK;
}

// The same of a view that is written: rows that begin less than d elements apart would lie on one another.
tq_status check_output(const tq_heads& x, int dtype, int batch, int n_heads, int n_tokens) {
  auto apart = [](int64_t stride) { return stride >= kD || stride <= -kD; };
  if ((batch > 1 && !apart(x.stride_b)) || (n_heads > 1 && !apart(x.stride_h)) || (n_tokens > 1 && !apart(x.stride_t)))
    return TQ_EINVAL;
  return check_view(x, dtype, batch, n_heads, n_tokens);
}

// Positions and block numbers are counted in 32 bits, with room for a tile beyond the last: caches of up to 2^30 rows a
// head, lists of up to 2^30 blocks.
constexpr int kMostRows = 1 << 30;

// The tables live on the device the quantizer was built on; launches go to the current one.
tq_status check_device(const tq_quantizer* q) {
  int dev = -1;
  if (!q->dev || cudaGetDevice(&dev) != cudaSuccess) return TQ_ECUDA;
  return dev == q->device ? TQ_OK : TQ_EINVAL;
}

tq_status check_heads(const tq_kv_cache* c, int n_q_heads, const int32_t* head_map) {
  if (n_q_heads <= 0 || n_q_heads > kMaxHeads) return TQ_EINVAL;
  if (c->n_kv_heads > kMaxHeads || c->batch > 65535 || c->capacity > kMostRows) return TQ_EUNSUPPORTED;
  if (head_map) {
    for (int h = 0; h < n_q_heads; ++h)
      if (head_map[h] < 0 || head_map[h] >= c->n_kv_heads) return TQ_EINVAL;
  } else if (n_q_heads % c->n_kv_heads != 0) {
    return TQ_EINVAL;
  }
  return TQ_OK;
}

tq_status check_space(const void* workspace, size_t have, size_t need) {
  return !workspace || !aligned16(workspace) || have < need ? TQ_EINVAL : TQ_OK;
}

size_t blocks_workspace(const tq_kv_cache* c, int n_q_heads, int n_select) {
  const size_t a = select_scratch_bytes(c), b = decode_blocks_scratch_bytes(c, n_q_heads, n_select);
  return kWorkspaceHeader + (a > b ? a : b);
}

}  // namespace

tq_status tq_norm_rope(const tq_rope* rope, int dtype, int batch, int n_tokens, int d, int n_q_heads, tq_heads q,
                       tq_heads q_out, const void* q_weight, int n_k_heads, tq_heads k, tq_heads k_out,
                       const void* k_weight, int norm, float eps, void* stream) {
  if (!rope || batch < 0 || n_tokens < 0 || n_q_heads < 0 || n_k_heads < 0) return TQ_EINVAL;
  if (d != kD || !known_dtype(dtype)) return TQ_EUNSUPPORTED;
  if (rope->rot_dim < 0 || rope->rot_dim > kD || rope->rot_dim % 16) return TQ_EINVAL;
  if (norm && !(eps >= 0.f)) return TQ_EINVAL;
  if (rope->rot_dim > 0) {
    if (!rope->pos_dev || !rope->inv_freq_dev || rope->n_axes < 1 || rope->n_axes > 255) return TQ_EINVAL;
    if ((reinterpret_cast<uintptr_t>(rope->pos_dev) & 3u) || (reinterpret_cast<uintptr_t>(rope->inv_freq_dev) & 3u))
      return TQ_EINVAL;
    if (rope->axis_of_freq)
      for (int i = 0; i < rope->rot_dim / 2; ++i)
        if (rope->axis_of_freq[i] >= rope->n_axes) return TQ_EINVAL;
  }
  if (batch == 0 || n_tokens == 0 || n_q_heads + static_cast<int64_t>(n_k_heads) == 0) return TQ_OK;
  const int heads[2] = {n_q_heads, n_k_heads};
  const tq_heads src[2] = {q, k}, dst[2] = {q_out, k_out};
  const void* const w[2] = {q_weight, k_weight};
  for (int s = 0; s < 2; ++s) {
    if (heads[s] == 0) continue;
    tq_status st = check_view(src[s], dtype, batch, heads[s], n_tokens);
    if (st == TQ_OK) st = check_output(dst[s], dtype, batch, heads[s], n_tokens);
    if (st != TQ_OK) return st;
    if (w[s] && !aligned16(w[s])) return TQ_EINVAL;
  }
  return launch_norm_rope(rope, dtype, batch, n_tokens, heads, src, dst, w, norm, eps, static_cast<cudaStream_t>(stream));
}

tq_status tq_extend_workspace_bytes(const tq_kv_cache* c, int n_q_heads, int n_tokens, size_t* bytes) {
  if (!c || !bytes || n_q_heads <= 0 || n_tokens < 0 || c->batch <= 0 || c->n_kv_heads <= 0 || c->capacity <= 0)
    return TQ_EINVAL;
  if (c->capacity > kMostRows || static_cast<int64_t>(n_q_heads) * n_tokens > kMostRows) return TQ_EUNSUPPORTED;
  *bytes = kWorkspaceHeader + extend_scratch_bytes(c, n_q_heads, n_tokens);
  return TQ_OK;
}

tq_status tq_extend_attention(const tq_quantizer* q, const tq_kv_cache* c, tq_heads query, int q_dtype, int n_q_heads,
                              int n_tokens, int causal, const int32_t* head_map, float sm_scale, tq_heads out,
                              int out_dtype, void* workspace, size_t workspace_bytes, void* stream) {
  if (!q) return TQ_EINVAL;
  tq_status st = check_cache(q, c);
  if (st != TQ_OK) return st;
  if ((st = check_heads(c, n_q_heads, head_map)) != TQ_OK) return st;
  if (c->value_bits == 0 || n_tokens < 0) return TQ_EINVAL;
  if (!known_dtype(q_dtype) || !known_dtype(out_dtype)) return TQ_EUNSUPPORTED;
  if (n_tokens == 0) return TQ_OK;
  if (static_cast<int64_t>(n_q_heads) * n_tokens > kMostRows) return TQ_EUNSUPPORTED;   // rows are counted in 32 bits
  if ((st = check_view(query, q_dtype, c->batch, n_q_heads, n_tokens)) != TQ_OK) return st;
  if ((st = check_output(out, out_dtype, c->batch, n_q_heads, n_tokens)) != TQ_OK) return st;
  if ((st = check_space(workspace, workspace_bytes, kWorkspaceHeader + extend_scratch_bytes(c, n_q_heads, n_tokens))) != TQ_OK)
    return st;
  if ((st = check_device(q)) != TQ_OK) return st;
  return launch_extend(q, c, query, q_dtype, n_q_heads, n_tokens, causal, head_map, sm_scale, nullptr, 0, out, out_dtype,
                       workspace, static_cast<cudaStream_t>(stream));
}

tq_status tq_block_bounds(const tq_quantizer* q, const tq_kv_cache* c, void* bounds, int n_tokens, void* stream) {
  if (!q) return TQ_EINVAL;
  tq_status st = check_cache(q, c);
  if (st != TQ_OK) return st;
  if (n_tokens < 0) return TQ_EINVAL;
  if (c->n_kv_heads > 65535 || c->batch > 65535 || c->capacity > kMostRows) return TQ_EUNSUPPORTED;
  if (n_tokens == 0) return TQ_OK;
  if (!bounds || !aligned16(bounds)) return TQ_EINVAL;
  if ((st = check_device(q)) != TQ_OK) return st;
  return launch_block_bounds(q, c, bounds, n_tokens, static_cast<cudaStream_t>(stream));
}

tq_status tq_blocks_workspace_bytes(const tq_kv_cache* c, int n_q_heads, int n_select, size_t* bytes) {
  if (!c || !bytes || n_q_heads <= 0 || n_select <= 0 || c->batch <= 0 || c->n_kv_heads <= 0 || c->capacity <= 0)
    return TQ_EINVAL;
  if (c->capacity > kMostRows || n_q_heads > kMaxHeads || n_select > kMostRows) return TQ_EUNSUPPORTED;
  *bytes = blocks_workspace(c, n_q_heads, n_select);
  return TQ_OK;
}

tq_status tq_select_blocks(const tq_quantizer* q, const tq_kv_cache* c, const void* bounds, const void* query, int q_dtype,
                           int n_q_heads, const int32_t* head_map, int n_select, int n_sink, int n_recent, int32_t* blocks,
                           void* workspace, size_t workspace_bytes, void* stream) {
  if (!q) return TQ_EINVAL;
  tq_status st = check_cache(q, c);
  if (st != TQ_OK) return st;
  if ((st = check_heads(c, n_q_heads, head_map)) != TQ_OK) return st;
  if (!known_dtype(q_dtype)) return TQ_EUNSUPPORTED;
  if (n_select <= 0 || n_sink < 0 || n_recent < 0 || static_cast<int64_t>(n_sink) + n_recent > n_select) return TQ_EINVAL;
  if (n_select > kMostRows) return TQ_EUNSUPPORTED;
  if (static_cast<int64_t>(c->batch) * c->n_kv_heads > kMaxCounters) return TQ_EUNSUPPORTED;
  if (!bounds || !aligned16(bounds) || !query || !aligned16(query)) return TQ_EINVAL;
  if (!blocks || (reinterpret_cast<uintptr_t>(blocks) & 3u)) return TQ_EINVAL;
  if ((st = check_space(workspace, workspace_bytes, kWorkspaceHeader + select_scratch_bytes(c))) != TQ_OK) return st;
  if ((st = check_device(q)) != TQ_OK) return st;
  return launch_select_blocks(q, c, bounds, query, q_dtype, n_q_heads, head_map, n_select, n_sink, n_recent, blocks, workspace,
                              static_cast<cudaStream_t>(stream));
}

tq_status tq_decode_attention_blocks(const tq_quantizer* q, const tq_kv_cache* c, const void* query, int q_dtype, int n_q_heads,
                                     const int32_t* head_map, float sm_scale, const int32_t* blocks, int n_select, void* out,
                                     int out_dtype, void* workspace, size_t workspace_bytes, void* stream) {
  if (!q) return TQ_EINVAL;
  tq_status st = check_cache(q, c);
  if (st != TQ_OK) return st;
  if ((st = check_heads(c, n_q_heads, head_map)) != TQ_OK) return st;
  if (c->value_bits == 0 || n_select <= 0) return TQ_EINVAL;
  if (n_select > kMostRows) return TQ_EUNSUPPORTED;
  if (!known_dtype(q_dtype) || !known_dtype(out_dtype)) return TQ_EUNSUPPORTED;
  if (!blocks || (reinterpret_cast<uintptr_t>(blocks) & 3u)) return TQ_EINVAL;
  const int64_t row = static_cast<int64_t>(n_q_heads) * kD;
  const tq_heads qv{const_cast<void*>(query), row, kD, 0}, ov{out, row, kD, 0};
  if ((st = check_view(qv, q_dtype, c->batch, n_q_heads, 1)) != TQ_OK) return st;
  if ((st = check_view(ov, out_dtype, c->batch, n_q_heads, 1)) != TQ_OK) return st;
  if ((st = check_space(workspace, workspace_bytes,
                        kWorkspaceHeader + decode_blocks_scratch_bytes(c, n_q_heads, n_select))) != TQ_OK)
    return st;
  if ((st = check_device(q)) != TQ_OK) return st;
  return launch_extend(q, c, qv, q_dtype, n_q_heads, 1, /*causal=*/0, head_map, sm_scale, blocks, n_select, ov, out_dtype,
                       workspace, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
