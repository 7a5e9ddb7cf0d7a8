// Attention of several query tokens over the packed cache, dense or over listed blocks
// (tq_extend_attention, tq_decode_attention_blocks).
#include <cmath>

#include "packed.cuh"

namespace tq {
namespace {

constexpr int kET = 128;

struct ExtendArgs {
  const uint8_t* k_idx;
  const uint8_t* k_sgn;
  const uint16_t* k_nrm;
  const uint8_t* v_q;
  const uint16_t* v_par;
  const int32_t* len;
  const int32_t* blocks;   // nullable: (batch, KV head, n_select) listed blocks
  const DevTables* tab;
  const void* q;
  void* out;
  int64_t qb, qh, qt, ob, oh, ot;
  int q_dtype, out_dtype;
  int n_kv_heads, capacity, n_tokens, n_select, n_blocks, causal;
  int mode, bits, vbits, idx_bytes, n_norms;
  float scale_log2;
  HeadLists heads;
};

__device__ __forceinline__ int code_at(const uint8_t* row, int bits, int j) {
  const int w = storage_width_c(bits);
  return (row[j * w >> 3] >> (j * w & 7)) & ((1 << bits) - 1);
}

// One block of threads per query row: thread = key for the scores of 128 keys at a time, then
// thread = channel for their weighted values.
__global__ void __launch_bounds__(kET) k_extend_simple(const __grid_constant__ ExtendArgs a) {
  __shared__ float qr[kD], sq[kD], p[kET], red[kET];
  __shared__ int rows[kET];
  const int tid = threadIdx.x, t = blockIdx.x, b = blockIdx.z;
  int kv = 0;
  while (static_cast<int>(blockIdx.y) >= a.heads.start[kv + 1]) ++kv;
  const int h = a.heads.head[blockIdx.y];
  const int len = max(0, min(a.len[b], a.capacity));
  const int limit = a.causal ? min(len, len - a.n_tokens + t + 1) : len;
  const bool grp = a.mode == TQ_MODE_GROUPED;
  // rotated query
  {
    const int c = grp ? a.tab->chan[tid] : tid;
    float x = load_element(a.q, a.q_dtype, b * a.qb + h * a.qh + t * a.qt + c);
    qr[tid] = flip_sign(x, a.tab->sign_bits[tid >> 5], tid & 31);
    for (int m = 1; m < (grp ? 32 : kD); m <<= 1) {
      __syncthreads();
      const float u = qr[tid], v = qr[tid ^ m];
      __syncthreads();
      qr[tid] = tid & m ? v - u : u + v;
    }
    __syncthreads();
    qr[tid] *= grp ? rsqrtf(32.f) : rsqrtf(128.f);
    __syncthreads();
    float s = 0.f;
    if (a.mode == TQ_MODE_PROD)
      for (int j = 0; j < kD; ++j) s = fmaf(__half2float(a.tab->s_rot_t[j * kD + tid]), qr[j], s);
    sq[tid] = s * (1.2533141373155003f / kD);
    __syncthreads();
  }
  float m = -INFINITY, l = 0.f, o = 0.f;
  const int64_t base = (static_cast<int64_t>(b) * a.n_kv_heads + kv) * a.capacity;
  const int32_t* list = a.blocks ? a.blocks + (static_cast<int64_t>(b) * a.n_kv_heads + kv) * a.n_select : nullptr;
  const int total = list ? a.n_select * TQ_BLOCK : limit;
  for (int i0 = 0; i0 < total; i0 += kET) {
    int i = i0 + tid;
    if (list) {
      const int blk = i < total ? list[i / TQ_BLOCK] : -1;
      i = blk >= 0 && blk < a.n_blocks ? blk * TQ_BLOCK + i % TQ_BLOCK : limit;
    }
    const bool ok = i < limit;
    float s = -INFINITY;
    if (ok) {
      const uint8_t* idx = a.k_idx + (base + i) * a.idx_bytes;
      const float n0 = __half2float(__ushort_as_half(a.k_nrm[(base + i) * a.n_norms]));
      if (grp) {
        float s0 = 0.f, s1 = 0.f;
        for (int j = 0; j < 32; ++j) s0 = fmaf(qr[j], a.tab->cent[0][code_at(idx, a.bits + 1, j)], s0);
        const uint8_t* rest = idx + 4 * storage_width_c(a.bits + 1);
        for (int j = 0; j < 96; ++j) s1 = fmaf(qr[32 + j], a.tab->cent[1][code_at(rest, a.bits, j)], s1);
        s = n0 * s0 * rsqrtf(32.f) + __half2float(__ushort_as_half(a.k_nrm[(base + i) * 2 + 1])) * s1 * rsqrtf(96.f);
      } else {
        const int bits = a.mode == TQ_MODE_PROD ? a.bits - 1 : a.bits;
        float s0 = 0.f;
        for (int j = 0; j < kD; ++j) s0 = fmaf(qr[j], a.tab->cent[0][code_at(idx, bits, j)], s0);
        s = n0 * s0 * rsqrtf(128.f);
        if (a.mode == TQ_MODE_PROD) {
          float s1 = 0.f;
          for (int j = 0; j < kD; ++j) s1 += code_at(a.k_sgn + (base + i) * (kD / 8), 1, j) ? sq[j] : -sq[j];
          s = fmaf(__half2float(__ushort_as_half(a.k_nrm[(base + i) * 2 + 1])), s1, s);
        }
      }
      s *= a.scale_log2;
    }
    red[tid] = s;
    rows[tid] = ok ? i : -1;
    __syncthreads();
    float mc = m;
    for (int k = 0; k < kET; ++k) mc = fmaxf(mc, red[k]);
    const float ref = mc == -INFINITY ? 0.f : mc;
    p[tid] = ok ? exp2f(s - ref) : 0.f;
    __syncthreads();
    const float f = exp2f(m - ref);
    l *= f;
    o *= f;
    for (int k = 0; k < kET; ++k) {
      if (rows[k] < 0) continue;
      const int64_t r = base + rows[k];
      const uint16_t* par = a.v_par + r * 8 + 2 * (tid >> 5);
      const float v = fmaf(static_cast<float>(code_at(a.v_q + r * (kD * a.vbits / 8), a.vbits, tid)),
                           __half2float(__ushort_as_half(par[1])), __half2float(__ushort_as_half(par[0])));
      l += p[k];
      o = fmaf(p[k], v, o);
    }
    m = mc;
    __syncthreads();
  }
  store_element(a.out, a.out_dtype, b * a.ob + h * a.oh + t * a.ot + tid, l > 0.f || isnan(l) ? o / l : 0.f);
}

}  // namespace

size_t extend_scratch_bytes(const tq_kv_cache*, int, int) { return 0; }
size_t decode_blocks_scratch_bytes(const tq_kv_cache*, int, int) { return 0; }

tq_status launch_extend(const tq_quantizer* q, const tq_kv_cache* c, const tq_heads& query, int q_dtype, int n_q_heads,
                        int n_tokens, int causal, const int32_t* head_map, float sm_scale, const int32_t* blocks,
                        int n_select, const tq_heads& out, int out_dtype, void*, cudaStream_t st) {
  ExtendArgs a;
  a.k_idx = c->keys.idx;
  a.k_sgn = c->keys.signs;
  a.k_nrm = c->keys.norms;
  a.v_q = c->values.q;
  a.v_par = c->values.params;
  a.len = c->len_dev;
  a.blocks = blocks;
  a.tab = q->dev;
  a.q = query.data;
  a.out = out.data;
  a.qb = query.stride_b; a.qh = query.stride_h; a.qt = query.stride_t;
  a.ob = out.stride_b; a.oh = out.stride_h; a.ot = out.stride_t;
  a.q_dtype = q_dtype;
  a.out_dtype = out_dtype;
  a.n_kv_heads = c->n_kv_heads;
  a.capacity = c->capacity;
  a.n_tokens = n_tokens;
  a.n_select = n_select;
  a.n_blocks = block_count(c->capacity);
  a.causal = causal;
  a.mode = q->mode;
  a.bits = q->bits;
  a.vbits = c->value_bits;
  a.idx_bytes = q->layout.idx_bytes;
  a.n_norms = q->layout.n_norms;
  const float scale = sm_scale > 0.f ? sm_scale : 1.f / std::sqrt(static_cast<float>(kD));
  a.scale_log2 = scale * 1.4426950408889634074f;
  fill_head_lists(n_q_heads, c->n_kv_heads, head_map, &a.heads);
  k_extend_simple<<<dim3(n_tokens, n_q_heads, c->batch), kET, 0, st>>>(a);
  return cudaGetLastError() == cudaSuccess ? TQ_OK : TQ_ECUDA;
}

}  // namespace tq
