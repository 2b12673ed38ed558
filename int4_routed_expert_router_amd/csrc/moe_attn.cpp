// Entry points of the paged attention (see include/moe_attn.h): argument checks
// before any GPU work, then one launch function each.
#include <cmath>

#include "attn.h"

namespace moe {
moe_status set_error(moe_status code, const char* fmt, ...);

namespace {

constexpr int kMaxTokens = 1 << 20;

bool at_aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int log2_of(int v) { return 31 - __builtin_clz(static_cast<unsigned>(v)); }

moe_status check_desc(const moe_attn_desc* d, int32_t n_tokens) {
  if (!d) return set_error(MOE_EINVAL, "desc is NULL");
  if (d->batch < 0 || d->batch > 65535) return set_error(MOE_ESHAPE, "batch=%d must be in [0, 65535]", d->batch);
  if (d->kv_heads < 1 || d->kv_heads > 128) return set_error(MOE_ESHAPE, "kv_heads=%d must be in [1, 128]", d->kv_heads);
  if (d->q_heads < d->kv_heads || d->q_heads % d->kv_heads || d->q_heads / d->kv_heads > 16)
    return set_error(MOE_ESHAPE, "q_heads=%d must be 1 to 16 times kv_heads=%d", d->q_heads, d->kv_heads);
  if (d->head_dim != 64 && d->head_dim != 128 && d->head_dim != 256)
    return set_error(MOE_ESHAPE, "head_dim=%d must be 64, 128 or 256", d->head_dim);
  if (d->act_dtype != MOE_F16 && d->act_dtype != MOE_BF16)
    return set_error(MOE_EINVAL, "act_dtype=%d is not MOE_F16/MOE_BF16", d->act_dtype);
  if (d->page_size < 16 || d->page_size > 256 || (d->page_size & (d->page_size - 1)))
    return set_error(MOE_ESHAPE, "page_size=%d must be 16, 32, 64, 128 or 256", d->page_size);
  if (d->n_pages < 1) return set_error(MOE_ESHAPE, "n_pages=%d must be at least 1", d->n_pages);
  const int64_t most = static_cast<int64_t>(d->max_pages) * d->page_size;
  if (d->max_pages < 1 || most > (1 << 30))
    return set_error(MOE_ESHAPE, "max_pages=%d must be at least 1 and hold at most 2^30 positions", d->max_pages);
  if (most * d->kv_heads * d->batch > (1ll << 37))
    return set_error(MOE_ESHAPE, "batch * kv_heads * max_pages * page_size must be at most 2^37");
  if (n_tokens < 0 || n_tokens > kMaxTokens)
    return set_error(MOE_ESHAPE, "n_tokens=%d must be in [0, 2^20]", n_tokens);
  if (!attn_prefill_fits(d, n_tokens))
    return set_error(MOE_ESHAPE, "n_tokens=%d of %d sequences and %d key heads are more than a launch holds", n_tokens,
                     d->batch, d->kv_heads);
  return MOE_OK;
}

moe_status check_cache(const moe_kv_cache* c) {
  if (!c) return set_error(MOE_EINVAL, "cache is NULL");
  if (!c->k || !c->v || !at_aligned(c->k, 16) || !at_aligned(c->v, 16))
    return set_error(MOE_EINVAL, "the cache's k and v must be 16-byte aligned device pointers");
  if (!c->table || !c->length || !at_aligned(c->table, 4) || !at_aligned(c->length, 4))
    return set_error(MOE_EINVAL, "the cache's table and length must be 4-byte aligned device pointers");
  return MOE_OK;
}

moe_status check_rows(const char* name, const moe_attn_rows* r) {
  if (!r || !r->data || !at_aligned(r->data, 16))
    return set_error(MOE_EINVAL, "%s must be rows at a 16-byte aligned device pointer", name);
  for (const int64_t st : {r->token_stride, r->head_stride})
    if (st < 0 || st % 8 || st >= (1ll << 31))
      return set_error(MOE_ESHAPE, "%s: a stride of %lld is not a multiple of 8 in [0, 2^31)", name,
                       static_cast<long long>(st));
  return MOE_OK;
}

const uint16_t* u16(const void* p) { return static_cast<const uint16_t*>(p); }

moe_status attend(const moe_attn_desc* d, const moe_kv_cache* c, const int32_t* off, int32_t n,
                  const moe_attn_rows* q, const moe_attn_rows* gate, float scale, void* o, void* ws, size_t ws_bytes,
                  bool decode, moe_stream stream) {
  moe_status st = check_cache(c);
  if (!st) st = check_rows("q", q);
  if (!st && gate) st = check_rows("gate", gate);
  if (st) return st;
  if (!std::isfinite(scale * kLog2e)) return set_error(MOE_EINVAL, "scale must be finite and below 2^127");
  if (!decode && (!off || !at_aligned(off, 4)))
    return set_error(MOE_EINVAL, "seq_off must be a 4-byte aligned device pointer");
  if (!o || !at_aligned(o, 16)) return set_error(MOE_EINVAL, "o must be a 16-byte aligned device pointer");
  const size_t need = decode ? attn_decode_bytes(d) : attn_prefill_bytes(d, n);
  if (!ws || !at_aligned(ws, 256)) return set_error(MOE_EINVAL, "workspace must be a 256-byte aligned device pointer");
  if (ws_bytes < need) return set_error(MOE_EWORKSPACE, "workspace of %zu bytes < required %zu", ws_bytes, need);
  auto i32 = [](int64_t v) { return static_cast<int32_t>(v); };
  AttnArgs a{u16(c->k), u16(c->v), c->table, c->length, off, u16(q->data), gate ? u16(gate->data) : nullptr,
             i32(q->token_stride), i32(q->head_stride), i32(gate ? gate->token_stride : 0),
             i32(gate ? gate->head_stride : 0),
             static_cast<uint16_t*>(o), scale, d->batch, n, d->q_heads, d->kv_heads, log2_of(d->page_size),
             d->n_pages, d->max_pages};
  const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const hipError_t e = decode ? launch_attn_decode(d->act_dtype, d->head_dim, a, ws, s)
                              : launch_attn_prefill(d->act_dtype, d->head_dim, a, ws, s);
  if (e != hipSuccess) return set_error(MOE_EHIP, "attention kernel launch: %s", hipGetErrorString(e));
  return set_error(MOE_OK, "");
}

}  // namespace
}  // namespace moe

extern "C" moe_status moe_kv_append(const moe_attn_desc* d, const moe_kv_cache* c, const int32_t* seq_off,
                                    int32_t n_tokens, const moe_attn_rows* k, const moe_attn_rows* v,
                                    const moe_attn_rows* q, void* q_out, const float* q_norm, const float* k_norm,
                                    float eps, const double* freq, int32_t rot_dim, moe_stream stream) {
  using moe::at_aligned;
  using moe::set_error;
  moe_status st = moe::check_desc(d, n_tokens);
  if (st) return st;
  if (!seq_off && n_tokens != d->batch)
    return set_error(MOE_ESHAPE, "without seq_off n_tokens=%d must be batch=%d", n_tokens, d->batch);
  if (rot_dim < 0 || rot_dim % 16 || rot_dim > d->head_dim)
    return set_error(MOE_ESHAPE, "rot_dim=%d must be a multiple of 16 in [0, head_dim=%d]", rot_dim, d->head_dim);
  if (d->batch == 0 || n_tokens == 0) return set_error(MOE_OK, "");
  st = moe::check_cache(c);
  if (!st) st = moe::check_rows("k", k);
  if (!st) st = moe::check_rows("v", v);
  if (!st && q) st = moe::check_rows("q", q);
  if (st) return st;
  if (!at_aligned(seq_off, 4)) return set_error(MOE_EINVAL, "seq_off must be 4-byte aligned");
  if (q && (!q_out || !at_aligned(q_out, 16)))
    return set_error(MOE_EINVAL, "q_out must be a 16-byte aligned device pointer");
  if (!q && (q_out || q_norm)) return set_error(MOE_EINVAL, "q_out and q_norm need q");
  if (!at_aligned(q_norm, 16) || !at_aligned(k_norm, 16))
    return set_error(MOE_EINVAL, "norms must be 16-byte aligned");
  if ((q_norm || k_norm) && !(eps >= 0 && std::isfinite(eps)))
    return set_error(MOE_EINVAL, "eps must be finite and not negative");
  if (rot_dim && (!freq || !at_aligned(freq, 8)))
    return set_error(MOE_EINVAL, "rot_dim=%d needs freq, an 8-byte aligned device pointer", rot_dim);
  auto i32 = [](int64_t v) { return static_cast<int32_t>(v); };
  moe::AppendArgs a{static_cast<uint16_t*>(c->k), static_cast<uint16_t*>(c->v), c->table, c->length, seq_off,
                    moe::u16(k->data), moe::u16(v->data), q ? moe::u16(q->data) : nullptr, i32(k->token_stride),
                    i32(k->head_stride), i32(v->token_stride), i32(v->head_stride), i32(q ? q->token_stride : 0),
                    i32(q ? q->head_stride : 0),
                    static_cast<uint16_t*>(q_out), q_norm, k_norm, freq, eps, rot_dim, d->batch, n_tokens, d->q_heads,
                    d->kv_heads, moe::log2_of(d->page_size), d->n_pages, d->max_pages};
  const hipError_t e =
      moe::launch_kv_append(d->act_dtype, d->head_dim, a, reinterpret_cast<hipStream_t>(stream));
  if (e != hipSuccess) return set_error(MOE_EHIP, "cache append kernel launch: %s", hipGetErrorString(e));
  return set_error(MOE_OK, "");
}

extern "C" moe_status moe_attn_workspace_bytes(const moe_attn_desc* d, int32_t n_tokens, size_t* bytes) {
  const moe_status st = moe::check_desc(d, n_tokens);
  if (st) return st;
  if (!bytes) return moe::set_error(MOE_EINVAL, "bytes is NULL");
  const size_t one = moe::attn_decode_bytes(d), many = moe::attn_prefill_bytes(d, n_tokens);
  *bytes = one > many ? one : many;
  return moe::set_error(MOE_OK, "");
}

extern "C" moe_status moe_attn_decode(const moe_attn_desc* d, const moe_kv_cache* c, const moe_attn_rows* q,
                                      const moe_attn_rows* gate, float scale, void* o, void* ws, size_t ws_bytes,
                                      moe_stream stream) {
  const moe_status st = moe::check_desc(d, 0);
  if (st) return st;
  if (d->batch == 0) return moe::set_error(MOE_OK, "");
  return moe::attend(d, c, nullptr, d->batch, q, gate, scale, o, ws, ws_bytes, true, stream);
}

extern "C" moe_status moe_attn_prefill(const moe_attn_desc* d, const moe_kv_cache* c, const int32_t* seq_off,
                                       int32_t n_tokens, const moe_attn_rows* q, const moe_attn_rows* gate,
                                       float scale, void* o, void* ws, size_t ws_bytes, moe_stream stream) {
  const moe_status st = moe::check_desc(d, n_tokens);
  if (st) return st;
  if (d->batch == 0 || n_tokens == 0) return moe::set_error(MOE_OK, "");
  return moe::attend(d, c, seq_off, n_tokens, q, gate, scale, o, ws, ws_bytes, false, stream);
}
