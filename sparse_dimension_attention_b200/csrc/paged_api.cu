// extern "C" entry points of the paged 8-bit cache: argument checks on the host
// (nothing is launched on a failed check), workspace size, dispatch.
#include <cmath>
#include <cstdint>

#include "paged_internal.cuh"

namespace aqua {

int launch_paged_append(const PagedView& c, const void* k_new, const void* v_new, bool bf16, const Strides& ks,
                        const Strides& vs, int n_tokens, const int32_t* start, const int32_t* cu, const float* P,
                        const RopeView& rope, cudaStream_t st);
size_t paged_decode_workspace_bytes(int B, int Hkv, int G);
int launch_paged_decode(const PagedView& c, const int32_t* len, const void* q, bool bf16, const Strides& qs,
                        const float* P, const RopeView& rope, int Hq, int k, float scale, void* out, bool out_bf16,
                        int32_t* sel_out, float* qproj_out, float* lse_out, void* ws, cudaStream_t st);
int launch_paged_gather(const PagedView& c, const int32_t* len, const int32_t* seq_idx, aqua_cache* dst, int max_len,
                        cudaStream_t st);

}  // namespace aqua

using aqua::set_error;

namespace {

constexpr int kMaxPagedG = 8;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int validate(const aqua_paged_cache* c) {
  if (c == nullptr) return set_error(AQUA_ERR_ARG, "paged cache descriptor is NULL");
  if (!c->k_pages || !c->v_pages || !c->k_scale || !c->v_scale || !c->block_table || !c->ctrl)
    return set_error(AQUA_ERR_ARG, "paged cache: pages, scales, block_table and ctrl must be non-NULL");
  if (c->dtype != AQUA_E4M3) return set_error(AQUA_ERR_UNSUPPORTED, "paged cache: dtype %d (only e4m3)", c->dtype);
  if (c->d != aqua::kHeadDim) return set_error(AQUA_ERR_UNSUPPORTED, "paged cache: head dim %d (only 128)", c->d);
  if (c->d_store < 1 || c->d_store > c->d)
    return set_error(AQUA_ERR_ARG, "paged cache: d_store %d outside [1, d]", c->d_store);
  if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128)
    return set_error(AQUA_ERR_UNSUPPORTED, "paged cache: page_size %d not in {16, 32, 64, 128}", c->page_size);
  if (c->B < 1 || c->Hkv < 1 || c->n_pages < 1 || c->max_pages < 1)
    return set_error(AQUA_ERR_ARG, "paged cache: B=%d Hkv=%d n_pages=%d max_pages=%d", c->B, c->Hkv, c->n_pages,
                     c->max_pages);
  if (c->Hkv > 65535 || (long long)c->B * c->Hkv > (1LL << 24))
    return set_error(AQUA_ERR_UNSUPPORTED, "paged cache: B*Hkv too large");
  // rows of the value pages are counted in 31 bits (256 GB of them)
  if ((long long)c->n_pages * c->Hkv > (1LL << 31) / c->page_size - 1)
    return set_error(AQUA_ERR_UNSUPPORTED, "paged cache: n_pages * Hkv * page_size over 2^31");
  // slots of a sequence are counted in 32 bits
  if ((long long)c->max_pages * c->page_size > (1LL << 30))
    return set_error(AQUA_ERR_UNSUPPORTED, "paged cache: max_pages * page_size over 2^30 tokens");
  // tiles of 128 tokens of all sequences are counted in 32 bits
  if ((long long)c->max_pages * c->page_size > (1LL << 37) / c->B)
    return set_error(AQUA_ERR_UNSUPPORTED, "paged cache: B * max_pages * page_size over 2^37 tokens");
  if (!aligned(c->k_pages, 16) || !aligned(c->v_pages, 16))
    return set_error(AQUA_ERR_ARG, "paged cache: pages must be 16-byte aligned");
  if (!aligned(c->k_scale, 4) || !aligned(c->v_scale, 4) || !aligned(c->block_table, 4) || !aligned(c->ctrl, 4))
    return set_error(AQUA_ERR_ARG, "paged cache: scales, block_table and ctrl must be 4-byte aligned");
  return AQUA_OK;
}

int validate_rope(const aqua_rope* r, const char* who, aqua::RopeView* out) {
  *out = aqua::RopeView{nullptr, 0, 0, 0};
  if (r == nullptr) return AQUA_OK;
  if (r->cos_sin == nullptr || !aligned(r->cos_sin, 16))
    return set_error(AQUA_ERR_ARG, "%s: rope.cos_sin must be non-NULL and 16-byte aligned", who);
  if (r->rot_dim < 2 || r->rot_dim > aqua::kHeadDim || r->rot_dim % 2 != 0)
    return set_error(AQUA_ERR_ARG, "%s: rope.rot_dim %d must be even, in [2, 128]", who, r->rot_dim);
  if (r->n_pos < 1 || (r->interleaved != 0 && r->interleaved != 1))
    return set_error(AQUA_ERR_ARG, "%s: rope.n_pos=%d interleaved=%d", who, r->n_pos, r->interleaved);
  *out = aqua::RopeView{r->cos_sin, r->n_pos, r->rot_dim, r->interleaved};
  return AQUA_OK;
}

// Strides in elements of rows and heads: 0 selects the dense one; every row of d must stay 16-byte aligned.
int check_strides(long long row, long long head, int heads, int io_dtype, const char* who, const char* name,
                  aqua::Strides* out) {
  const long long d = aqua::kHeadDim, per16 = io_dtype == AQUA_BF16 ? 8 : 4, most = 1LL << 31;
  out->row = row == 0 ? heads * d : row;
  out->head = head == 0 ? d : head;
  if (out->row < d || out->head < d || out->row % per16 != 0 || out->head % per16 != 0 || out->row > most ||
      out->head > most)
    return set_error(AQUA_ERR_ARG, "%s: strides of %s (%lld, %lld) must be at least 128 and multiples of %lld elements",
                     who, name, out->row, out->head, per16);
  return AQUA_OK;
}

int check_io(int dtype, const char* who, const char* name) {
  if (dtype != AQUA_F32 && dtype != AQUA_BF16) return set_error(AQUA_ERR_UNSUPPORTED, "%s: %s %d", who, name, dtype);
  return AQUA_OK;
}

aqua::PagedView view_of(const aqua_paged_cache* c) {
  aqua::PagedView v;
  v.k = static_cast<uint8_t*>(c->k_pages);
  v.v = static_cast<uint8_t*>(c->v_pages);
  v.ks = c->k_scale;
  v.vs = c->v_scale;
  v.table = c->block_table;
  v.ctrl = c->ctrl;
  v.B = c->B;
  v.Hkv = c->Hkv;
  v.m = c->d_store;
  v.page = c->page_size;
  v.page_log2 = c->page_size == 16 ? 4 : (c->page_size == 32 ? 5 : (c->page_size == 64 ? 6 : 7));
  v.n_pages = c->n_pages;
  v.max_pages = c->max_pages;
  return v;
}

// No exception (host memory, a mutex) leaves a C entry point.
template <typename F>
int guarded(const char* who, F launch) noexcept {
  try {
    return launch();
  } catch (...) {
    return set_error(AQUA_ERR_CUDA, "%s: out of host resources", who);
  }
}

}  // namespace

extern "C" {

int aqua_paged_status(const aqua_paged_cache* cache, int* status_out, aqua_stream_t stream) {
  if (cache == nullptr) return set_error(AQUA_ERR_ARG, "aqua_paged_status: NULL argument");
  aqua_cache c = {};
  c.ctrl = cache->ctrl;
  return aqua_status(&c, status_out, stream);
}

int aqua_paged_append(const aqua_paged_cache* cache, const void* k_new, const void* v_new, int io_dtype,
                      long long k_stride, long long k_head_stride, long long v_stride, long long v_head_stride,
                      int n_tokens, const int32_t* start, const int32_t* cu_new, const float* P,
                      const aqua_rope* rope, aqua_stream_t stream) {
  const char* who = "aqua_paged_append";
  aqua::clear_error();
  aqua::RopeView rv;
  int rc = validate(cache);
  if (rc == AQUA_OK) rc = check_io(io_dtype, who, "io_dtype");
  if (rc == AQUA_OK) rc = validate_rope(rope, who, &rv);
  if (rc != AQUA_OK) return rc;
  if (k_new == nullptr || v_new == nullptr || start == nullptr || P == nullptr)
    return set_error(AQUA_ERR_ARG, "%s: NULL k_new, v_new, start or P", who);
  if (!aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(P, 16))
    return set_error(AQUA_ERR_ARG, "%s: k_new, v_new and P must be 16-byte aligned", who);
  if (!aligned(start, 4) || !aligned(cu_new, 4))
    return set_error(AQUA_ERR_ARG, "%s: start and cu_new must be 4-byte aligned", who);
  aqua::Strides ks, vs;
  if ((rc = check_strides(k_stride, k_head_stride, cache->Hkv, io_dtype, who, "k_new", &ks)) != AQUA_OK) return rc;
  if ((rc = check_strides(v_stride, v_head_stride, cache->Hkv, io_dtype, who, "v_new", &vs)) != AQUA_OK) return rc;
  if (n_tokens < 1) return set_error(AQUA_ERR_ARG, "%s: n_tokens=%d", who, n_tokens);
  if (cu_new == nullptr && n_tokens != cache->B)
    return set_error(AQUA_ERR_ARG, "%s: n_tokens=%d without cu_new, but B=%d", who, n_tokens, cache->B);
  return guarded(who, [&] {
    return aqua::launch_paged_append(view_of(cache), k_new, v_new, io_dtype == AQUA_BF16, ks, vs, n_tokens, start,
                                     cu_new, P, rv, reinterpret_cast<cudaStream_t>(stream));
  });
}

size_t aqua_paged_decode_workspace_size(const aqua_paged_cache* cache, int Hq) {
  if (validate(cache) != AQUA_OK || Hq < 1 || Hq % cache->Hkv != 0 || Hq / cache->Hkv > kMaxPagedG) return 0;
  return aqua::paged_decode_workspace_bytes(cache->B, cache->Hkv, Hq / cache->Hkv);
}

int aqua_paged_decode_attn(const aqua_paged_cache* cache, const int32_t* len, const void* q, int io_dtype,
                           long long q_stride, long long q_head_stride, const float* P, const aqua_rope* rope,
                           int Hq, int k, float scale, void* out, int out_dtype, int32_t* sel_out, float* qproj_out, float* lse_out,
                           void* workspace, size_t workspace_bytes, aqua_stream_t stream) {
  const char* who = "aqua_paged_decode_attn";
  aqua::clear_error();
  aqua::RopeView rv;
  int rc = validate(cache);
  if (rc == AQUA_OK) rc = check_io(io_dtype, who, "io_dtype");
  if (rc == AQUA_OK) rc = check_io(out_dtype, who, "out_dtype");
  if (rc == AQUA_OK) rc = validate_rope(rope, who, &rv);
  if (rc != AQUA_OK) return rc;
  if (Hq < 1 || Hq % cache->Hkv != 0)
    return set_error(AQUA_ERR_ARG, "%s: Hq=%d not a multiple of Hkv=%d", who, Hq, cache->Hkv);
  const int G = Hq / cache->Hkv;
  if (G > kMaxPagedG) return set_error(AQUA_ERR_UNSUPPORTED, "%s: Hq/Hkv=%d over %d", who, G, kMaxPagedG);
  if (k < 1 || k > cache->d_store)
    return set_error(AQUA_ERR_ARG, "%s: k=%d outside [1, d_store=%d]", who, k, cache->d_store);
  if (len == nullptr || q == nullptr || P == nullptr || out == nullptr || workspace == nullptr)
    return set_error(AQUA_ERR_ARG, "%s: NULL len, q, P, out or workspace", who);
  if (!aligned(q, 16) || !aligned(P, 16) || !aligned(out, 16) || !aligned(workspace, 256))
    return set_error(AQUA_ERR_ARG, "%s: q, P, out 16-byte and workspace 256-byte alignment required", who);
  if (!aligned(len, 4) || !aligned(sel_out, 4) || !aligned(qproj_out, 4) || !aligned(lse_out, 4))
    return set_error(AQUA_ERR_ARG, "%s: len, sel_out, qproj_out and lse_out must be 4-byte aligned", who);
  aqua::Strides qs;
  if ((rc = check_strides(q_stride, q_head_stride, Hq, io_dtype, who, "q", &qs)) != AQUA_OK) return rc;
  const size_t need = aqua::paged_decode_workspace_bytes(cache->B, cache->Hkv, G);
  if (workspace_bytes < need)
    return set_error(AQUA_ERR_WORKSPACE, "%s: workspace %zu < %zu bytes", who, workspace_bytes, need);
  if (!(scale > 0.f)) scale = 1.0f / std::sqrt((float)cache->d);
  return guarded(who, [&] {
    return aqua::launch_paged_decode(view_of(cache), len, q, io_dtype == AQUA_BF16, qs, P, rv, Hq, k, scale, out,
                                     out_dtype == AQUA_BF16, sel_out, qproj_out, lse_out, workspace,
                                     reinterpret_cast<cudaStream_t>(stream));
  });
}

int aqua_paged_gather(const aqua_paged_cache* cache, const int32_t* len, const int32_t* seq_idx, aqua_cache* dst,
                      int max_len, aqua_stream_t stream) {
  const char* who = "aqua_paged_gather";
  aqua::clear_error();
  int rc = validate(cache);
  if (rc != AQUA_OK) return rc;
  if (len == nullptr || dst == nullptr || !aligned(len, 4) || !aligned(seq_idx, 4))
    return set_error(AQUA_ERR_ARG, "%s: NULL or misaligned len, seq_idx or dst", who);
  if (dst->k_proj == nullptr || dst->v == nullptr || dst->len == nullptr)
    return set_error(AQUA_ERR_ARG, "%s: dst needs k_proj, v and len", who);
  if ((rc = check_io(dst->dtype, who, "dst dtype")) != AQUA_OK) return rc;
  if (dst->d != cache->d || dst->d_store != cache->d_store || dst->Hkv != cache->Hkv)
    return set_error(AQUA_ERR_ARG, "%s: dst d=%d d_store=%d Hkv=%d differ from the pages' %d %d %d", who, dst->d,
                     dst->d_store, dst->Hkv, cache->d, cache->d_store, cache->Hkv);
  if (dst->dv_store != 0 || dst->pos != nullptr)
    return set_error(AQUA_ERR_UNSUPPORTED, "%s: dst with projected values or H2O positions", who);
  if (dst->B < 1 || dst->B > 65535 || (seq_idx == nullptr && dst->B != cache->B))
    return set_error(AQUA_ERR_ARG, "%s: dst B=%d for a paged cache of %d sequences%s", who, dst->B, cache->B,
                     seq_idx ? "" : " without seq_idx");
  if (dst->Tcap < 16 || dst->Tcap % 16 != 0 || max_len < 0 || max_len > dst->Tcap)
    return set_error(AQUA_ERR_ARG, "%s: max_len=%d outside [0, Tcap=%d] (Tcap a multiple of 16)", who, max_len,
                     dst->Tcap);
  if (!aligned(dst->k_proj, 16) || !aligned(dst->v, 16))
    return set_error(AQUA_ERR_ARG, "%s: dst k_proj and v must be 16-byte aligned", who);
  rc = guarded(who, [&] {
    return aqua::launch_paged_gather(view_of(cache), len, seq_idx, dst, max_len, reinterpret_cast<cudaStream_t>(stream));
  });
  if (rc == AQUA_OK) dst->max_len = max_len;
  return rc;
}

}  // extern "C"
