// C ABI of the layers on irreps rows: argument checks, handles, dispatch.
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstring>

#include "attn.hpp"
#include "guard.hpp"

namespace cgtp {

RowLayout row_layout(const char* irreps) {
  RowLayout r;
  r.irreps = irreps_from_string(irreps);
  for (const Irrep& i : r.irreps) {
    if (i.l > kLmax) throw Error{CGTP_ERR_UNSUPPORTED, "degree above CGTP_LMAX"};
    RowBlock b{};
    const bool even = i.l == 0 && i.p > 0;
    b.off = int32_t(r.dim);
    b.nc = 2 * i.l + 1;
    b.mul = i.mul;
    b.chan = int32_t(r.channels);
    b.bias = even ? int32_t(r.biases) : -1;
    b.chunk = int32_t(r.chunks);
    r.dim += int64_t(i.mul) * b.nc;
    r.channels += i.mul;
    r.chunks += (i.mul + 7) / 8;
    if (even) r.biases += i.mul;
    if (r.dim > (1 << 18)) throw Error{CGTP_ERR_UNSUPPORTED, "rows of more than 2^18 elements"};
    r.blocks.push_back(b);
  }
  if (r.blocks.empty() || r.blocks.size() > 4096) throw Error{CGTP_ERR_UNSUPPORTED, "no block, or more than 4096"};
  return r;
}

int current_device() {
  int d = 0;
  CGTP_CHECK_HIP(hipGetDevice(&d));
  return d;
}

void need_device(int device, const char* what) {
  if (current_device() != device)
    throw Error{CGTP_ERR_INVALID_ARG, std::string(what) + " was made on another device than the current one"};
}

DevMem::~DevMem() {
  if (!p_) return;
  int cur = 0;
  const bool have = hipGetDevice(&cur) == hipSuccess;
  if (hipSetDevice(device_) == hipSuccess) (void)hipFree(p_);
  if (have) (void)hipSetDevice(cur);
}

void DevMem::upload(const void* src, size_t n) {
  device_ = current_device();
  if (hipMalloc(&p_, n ? n : 16) != hipSuccess) {
    p_ = nullptr;
    (void)hipGetLastError();
    throw Error{CGTP_ERR_ALLOC, "device allocation failed"};
  }
  if (n) CGTP_CHECK_HIP(hipMemcpy(p_, src, n, hipMemcpyHostToDevice));
}

namespace {

void need_dtype(cgtp_dtype d) { need(d == CGTP_F32 || d == CGTP_F64 || d == CGTP_BF16, "bad dtype"); }

void need_ws(const void* ws, size_t have, size_t want, const char* what) {
  if (want == 0) return;
  if (!ws || have < want)
    throw Error{CGTP_ERR_WORKSPACE, std::string(what) + " needs " + std::to_string(want) + " workspace bytes"};
  need(reinterpret_cast<uintptr_t>(ws) % 16 == 0, "the workspace must be 16-byte aligned");
}

void need_rows(int64_t rows, const void* p, int64_t ld, int64_t dim, const char* name) {
  if (ld < dim) throw Error{CGTP_ERR_INVALID_ARG, std::string(name) + ": row stride below the row size"};
  if (rows > 0 && !p) throw Error{CGTP_ERR_INVALID_ARG, std::string(name) + " is NULL"};
}

void need_scale(double scale) {
  // as the kernels hold it, times log2 e in 32 bits: 0 * inf would make NaN of scores of 0
  need(std::isfinite(float(scale * 1.4426950408889634)), "scale must be finite in 32 bits");
}

void need_batch(const cgtp_attn_batch_s* b, double scale) {
  need(b != nullptr, "batch is NULL");
  need_scale(scale);
  need_device(b->device, "the batch");
}

// Rows in a run of the norm: long enough that a workgroup's work outweighs its
// reduction, short enough that the runs fill the device; at most 512 runs a
// sample, since every run joins all of its sample's partial moments.
int64_t chunk_rows(int64_t rows, int64_t sample_rows) {
  const int64_t r = rows <= 16384 ? 32 : 64;
  return std::max(r, (sample_rows + 511) / 512);
}

cgtp_samples_s* build_samples(int64_t S, const int64_t* ptr) {
  auto sm = std::make_unique<cgtp_samples_s>();
  if (ptr[0] != 0) throw Error{CGTP_ERR_INDEX, "samples: ptr[0] must be 0"};
  for (int64_t s = 0; s < S; ++s)
    if (ptr[s + 1] < ptr[s]) throw Error{CGTP_ERR_INDEX, "samples: ptr must not decrease"};
  if (ptr[S] > INT32_MAX || S >= INT32_MAX) throw Error{CGTP_ERR_UNSUPPORTED, "samples: more than 2^31 - 1 rows"};
  sm->S = S;
  sm->rows = ptr[S];
  sm->ptr.assign(ptr, ptr + S + 1);
  std::vector<RowChunk> ch;
  for (int64_t s = 0; s < S; ++s) {
    const int64_t a = ptr[s], n = ptr[s + 1] - a, R = chunk_rows(sm->rows, n), k = (n + R - 1) / R;
    sm->longest = std::max(sm->longest, n);
    const int32_t c0 = int32_t(ch.size());
    sm->sample_chunk.push_back(c0);
    // even cuts, so that no run is much shorter than the others
    for (int64_t j = 0; j < k; ++j)
      ch.push_back({int32_t(s), int32_t(a + n * j / k), int32_t(a + n * (j + 1) / k), c0, int32_t(k), int32_t(a),
                    int32_t(n), 0});
  }
  sm->sample_chunk.push_back(int32_t(ch.size()));
  sm->nchunk = int64_t(ch.size());
  sm->device = current_device();
  sm->chunks.upload(ch.data(), ch.size() * sizeof(RowChunk));
  const std::vector<int32_t> rows(ptr, ptr + S + 1);
  sm->first_row.upload(rows.data(), rows.size() * sizeof(int32_t));
  sm->first.upload(sm->sample_chunk.data(), sm->sample_chunk.size() * sizeof(int32_t));
  return sm.release();
}

// Lane width and strips of a norm: lanes never straddle a group, a strip is as
// many whole groups as 256 lanes hold (at least one), a narrow one as many as 128
// bytes hold.
void norm_strips(cgtp_norm_s* n) {
  n->vec = 16 / int(dtype_size(n->dtype));
  for (const RowBlock& b : n->row.blocks)
    while ((b.mul / n->groups) % n->vec != 0) n->vec /= 2;
  const int64_t es = int64_t(dtype_size(n->dtype));
  for (int k = 0; k < 4; ++k) {
    const int vec = k % 2 == 0 ? n->vec : 1;
    std::vector<NormStrip> st;
    for (size_t i = 0; i < n->row.blocks.size(); ++i) {
      const RowBlock& b = n->row.blocks[i];
      const int G = int(n->groups), cg = b.mul / G;
      int per = std::min(G, std::max(1, 256 * vec / cg));
      if (k >= 2) {
        per = std::min(per, std::max(1, int(128 / (cg * es))));
        n->narrow_row = std::max<int64_t>(n->narrow_row, int64_t(per) * cg * b.nc);
      }
      for (int g = 0; g < G; g += per)
        st.push_back({b.off, b.nc, b.mul, b.chan, b.bias, cg, g, std::min(per, G - g), int32_t(i) * G + g, 0, 0, 0});
    }
    // the workgroups with the most work first
    std::stable_sort(st.begin(), st.end(), [](const NormStrip& a, const NormStrip& b) {
      return int64_t(a.nc) * a.ng * a.cg > int64_t(b.nc) * b.ng * b.cg;
    });
    if (st.size() > 65535) throw Error{CGTP_ERR_UNSUPPORTED, "too many groups"};
    n->nstrip[k] = int(st.size());
    n->strips[k].upload(st.data(), st.size() * sizeof(NormStrip));
  }
}

}  // namespace

}  // namespace cgtp

using namespace cgtp;

extern "C" {

cgtp_status cgtp_samples_create(int64_t S, const int64_t* ptr, cgtp_samples* out) {
  return guarded([&] {
    need(out != nullptr, "out handle is NULL");
    *out = nullptr;
    need(S >= 0, "S < 0");
    need(ptr != nullptr, "ptr is NULL");
    *out = build_samples(S, ptr);
  });
}

cgtp_status cgtp_samples_destroy(cgtp_samples samples) {
  return guarded([&] { delete samples; });
}

cgtp_status cgtp_norm_create(const char* irreps, int64_t groups, cgtp_act act, double eps, cgtp_dtype dtype,
                             cgtp_norm* out) {
  return guarded([&] {
    need(out != nullptr, "out handle is NULL");
    *out = nullptr;
    need_dtype(dtype);
    need(groups >= 1, "groups < 1");
    need(eps > 0.0, "eps must be positive");
    // in the arithmetic of the kernels: as 0 it would leave 0 * inf where a variance is 0
    need(dtype == CGTP_F64 ? std::isnormal(eps) : std::isnormal(float(eps)),
         "eps must be a normal number of the norm's arithmetic");
    need(act == CGTP_ACT_NONE || act == CGTP_ACT_SILU || act == CGTP_ACT_GELU, "bad activation");
    auto n = std::make_unique<cgtp_norm_s>();
    n->row = row_layout(irreps);
    for (const RowBlock& b : n->row.blocks)
      if (groups > b.mul || b.mul % groups != 0)
        throw Error{CGTP_ERR_UNSUPPORTED, "groups must divide every multiplicity"};
    n->groups = groups;
    n->num_groups = groups * int64_t(n->row.blocks.size());
    n->act = act;
    n->eps = eps;
    n->dtype = dtype;
    n->device = current_device();
    norm_strips(n.get());
    *out = n.release();
  });
}

cgtp_status cgtp_norm_destroy(cgtp_norm norm) {
  return guarded([&] { delete norm; });
}

cgtp_status cgtp_norm_query(cgtp_norm norm, int64_t* dim, int64_t* channels, int64_t* biases, int64_t* num_groups) {
  return guarded([&] {
    need(norm != nullptr, "norm is NULL");
    if (dim) *dim = norm->row.dim;
    if (channels) *channels = norm->row.channels;
    if (biases) *biases = norm->row.biases;
    if (num_groups) *num_groups = norm->num_groups;
  });
}

cgtp_status cgtp_norm_workspace_size(cgtp_norm norm, cgtp_samples samples, int backward, size_t* bytes) {
  return guarded([&] {
    need(norm != nullptr && samples != nullptr && bytes != nullptr, "NULL argument");
    *bytes = norm_ws_bytes(norm, samples, backward != 0);
  });
}

cgtp_status cgtp_norm_forward(cgtp_norm norm, cgtp_samples samples, const void* x, const void* weight,
                              const void* bias, void* y, void* stats, void* ws, size_t ws_bytes, void* stream) {
  return guarded([&] {
    need(norm != nullptr && samples != nullptr, "NULL norm or samples");
    need_device(norm->device, "the norm");
    need_device(samples->device, "the samples");
    need(samples->rows == 0 || (x && y), "NULL tensor");
    need_ws(ws, ws_bytes, norm_ws_bytes(norm, samples, false), "norm forward");
    norm_forward_launch(norm, samples, x, weight, bias, y, stats, ws, as_stream(stream));
  });
}

cgtp_status cgtp_norm_backward(cgtp_norm norm, cgtp_samples samples, const void* x, const void* weight,
                               const void* bias, const void* stats, const void* grad_y, void* grad_x,
                               void* grad_weight, void* grad_bias, void* ws, size_t ws_bytes, void* stream) {
  return guarded([&] {
    need(norm != nullptr && samples != nullptr, "NULL norm or samples");
    need_device(norm->device, "the norm");
    need_device(samples->device, "the samples");
    need(samples->rows == 0 || (x && grad_y && stats), "NULL tensor");
    need_ws(ws, ws_bytes, norm_ws_bytes(norm, samples, true), "norm backward");
    if (!grad_x && !grad_weight && !grad_bias) return;
    norm_backward_launch(norm, samples, x, weight, bias, stats, grad_y, grad_x, grad_weight, grad_bias, ws,
                         as_stream(stream));
  });
}

cgtp_status cgtp_dropout_create(const char* irreps, cgtp_dtype dtype, cgtp_dropout* out) {
  return guarded([&] {
    need(out != nullptr, "out handle is NULL");
    *out = nullptr;
    need_dtype(dtype);
    auto d = std::make_unique<cgtp_dropout_s>();
    d->row = row_layout(irreps);
    d->dtype = dtype;
    d->device = current_device();
    d->blocks.upload(d->row.blocks.data(), d->row.blocks.size() * sizeof(RowBlock));
    *out = d.release();
  });
}

cgtp_status cgtp_dropout_destroy(cgtp_dropout drop) {
  return guarded([&] { delete drop; });
}

cgtp_status cgtp_dropout_query(cgtp_dropout drop, int64_t* dim) {
  return guarded([&] {
    need(drop != nullptr && dim != nullptr, "NULL argument");
    *dim = drop->row.dim;
  });
}

cgtp_status cgtp_dropout_forward(cgtp_dropout drop, int64_t B, const void* x, double p, uint64_t seed,
                                 uint32_t offset, const void* residual, void* y, void* stream) {
  return guarded([&] {
    need(drop != nullptr, "dropout is NULL");
    need(B >= 0, "B < 0");
    need(p >= 0.0 && p < 1.0, "p must lie in [0, 1)");
    if (B == 0) return;
    need(x && y, "NULL tensor with B > 0");
    need_device(drop->device, "the dropout");
    dropout_launch(drop, B, x, p, seed, offset, residual, y, as_stream(stream));
  });
}

cgtp_status cgtp_dropout_backward(cgtp_dropout drop, int64_t B, const void* grad_y, double p, uint64_t seed,
                                  uint32_t offset, void* grad_x, void* stream) {
  return cgtp_dropout_forward(drop, B, grad_y, p, seed, offset, nullptr, grad_x, stream);
}

cgtp_status cgtp_attn_create(const char* irreps, int64_t heads, int64_t kv_heads, cgtp_dtype dtype, cgtp_attn* out) {
  return guarded([&] {
    need(out != nullptr, "out handle is NULL");
    *out = nullptr;
    *out = build_attn(irreps, heads, kv_heads, dtype);
  });
}

cgtp_status cgtp_attn_destroy(cgtp_attn attn) {
  return guarded([&] { delete attn; });
}

cgtp_status cgtp_attn_query(cgtp_attn attn, int64_t* dim_q, int64_t* dim_kv, int64_t* head_dim) {
  return guarded([&] {
    need(attn != nullptr, "attn is NULL");
    if (dim_q) *dim_q = attn->qrow.dim;
    if (dim_kv) *dim_kv = attn->krow.dim;
    if (head_dim) *head_dim = attn->D;
  });
}

cgtp_status cgtp_attn_batch_create(cgtp_attn attn, cgtp_samples queries, cgtp_samples context, cgtp_attn_batch* out) {
  return guarded([&] {
    need(out != nullptr, "out handle is NULL");
    *out = nullptr;
    need(attn != nullptr && queries != nullptr && context != nullptr, "NULL handle");
    need_device(attn->device, "the attention");
    *out = build_attn_batch(attn, queries, context, false, 0);
  });
}

cgtp_status cgtp_attn_batch_create_seq(cgtp_attn attn, cgtp_samples queries, cgtp_samples context, int causal,
                                       int64_t shared, cgtp_attn_batch* out) {
  return guarded([&] {
    need(out != nullptr, "out handle is NULL");
    *out = nullptr;
    need(attn != nullptr && queries != nullptr && context != nullptr, "NULL handle");
    need(shared >= 0, "shared < 0");
    need_device(attn->device, "the attention");
    if (shared > INT32_MAX) throw Error{CGTP_ERR_UNSUPPORTED, "attention: more than 2^31 shared rows"};
    *out = build_attn_batch(attn, queries, context, causal != 0, shared);
  });
}

cgtp_status cgtp_attn_batch_destroy(cgtp_attn_batch batch) {
  return guarded([&] { delete batch; });
}

cgtp_status cgtp_attn_workspace_size(cgtp_attn_batch batch, int op, size_t* bytes) {
  return guarded([&] {
    need(batch != nullptr && bytes != nullptr, "NULL argument");
    switch (op) {
      case CGTP_ATTN_FORWARD: *bytes = attn_forward_ws_bytes(batch, false); break;
      case CGTP_ATTN_BACKWARD: *bytes = attn_backward_ws_bytes(batch); break;
      case CGTP_ATTN_CONTEXT: *bytes = attn_context_bytes(batch); break;
      case CGTP_ATTN_FORWARD_PACKED: *bytes = attn_forward_ws_bytes(batch, true); break;
      default: throw Error{CGTP_ERR_INVALID_ARG, "unknown op"};
    }
  });
}

cgtp_status cgtp_attn_forward(cgtp_attn_batch batch, const void* q, int64_t ldq, const void* k, int64_t ldk,
                              const void* v, int64_t ldv, const uint8_t* key_mask, double scale, void* out, float* lse,
                              void* ws, size_t ws_bytes, void* stream) {
  return guarded([&] {
    need_batch(batch, scale);
    need_rows(batch->nq, q, ldq, batch->attn->qrow.dim, "q");
    need_rows(batch->nk, k, ldk, batch->attn->krow.dim, "k");
    need_rows(batch->nk, v, ldv, batch->attn->krow.dim, "v");
    if (batch->nq == 0) return;
    need(out != nullptr, "out is NULL");
    need_ws(ws, ws_bytes, attn_forward_ws_bytes(batch, false), "attention forward");
    // the partial results, then the packed context
    void* context = static_cast<char*>(ws) + attn_forward_ws_bytes(batch, true);
    attn_pack_launch(batch, {k, ldk}, {v, ldv}, key_mask, context, as_stream(stream));
    attn_forward_launch(batch, {q, ldq}, context, scale, out, lse, ws, as_stream(stream));
  });
}

cgtp_status cgtp_attn_pack(cgtp_attn_batch batch, const void* k, int64_t ldk, const void* v, int64_t ldv,
                           const uint8_t* key_mask, void* context, size_t context_bytes, void* stream) {
  return guarded([&] {
    need_batch(batch, 1.0);
    need_rows(batch->nk, k, ldk, batch->attn->krow.dim, "k");
    need_rows(batch->nk, v, ldv, batch->attn->krow.dim, "v");
    need_ws(context, context_bytes, attn_context_bytes(batch), "the packed context");
    attn_pack_launch(batch, {k, ldk}, {v, ldv}, key_mask, context, as_stream(stream));
  });
}

cgtp_status cgtp_attn_forward_packed(cgtp_attn_batch batch, const void* q, int64_t ldq, const void* context,
                                     size_t context_bytes, double scale, void* out, float* lse, void* ws,
                                     size_t ws_bytes, void* stream) {
  return guarded([&] {
    need_batch(batch, scale);
    need_rows(batch->nq, q, ldq, batch->attn->qrow.dim, "q");
    need_ws(context, context_bytes, attn_context_bytes(batch), "the packed context");
    if (batch->nq == 0) return;
    need(out != nullptr, "out is NULL");
    need_ws(ws, ws_bytes, attn_forward_ws_bytes(batch, true), "attention forward");
    attn_forward_launch(batch, {q, ldq}, context, scale, out, lse, ws, as_stream(stream));
  });
}

cgtp_status cgtp_attn_backward(cgtp_attn_batch batch, const void* q, int64_t ldq, const void* k, int64_t ldk,
                               const void* v, int64_t ldv, const uint8_t* key_mask, double scale, const void* out,
                               const float* lse, const void* grad_out, int64_t ldg, void* grad_q, void* grad_k,
                               void* grad_v, void* ws, size_t ws_bytes, void* stream) {
  return guarded([&] {
    need_batch(batch, scale);
    need_rows(batch->nq, q, ldq, batch->attn->qrow.dim, "q");
    need_rows(batch->nk, k, ldk, batch->attn->krow.dim, "k");
    need_rows(batch->nk, v, ldv, batch->attn->krow.dim, "v");
    need_rows(batch->nq, grad_out, ldg, batch->attn->qrow.dim, "grad_out");
    need(batch->nq == 0 || (out && lse), "NULL out or lse");
    if (!grad_q && !grad_k && !grad_v) return;
    need_ws(ws, ws_bytes, attn_backward_ws_bytes(batch), "attention backward");
    attn_backward_launch(batch, {q, ldq}, {k, ldk}, {v, ldv}, key_mask, scale, out, lse, {grad_out, ldg}, grad_q,
                         grad_k, grad_v, ws, as_stream(stream));
  });
}

cgtp_status cgtp_attn_cache_create(cgtp_attn attn, int64_t slots, int64_t capacity, int64_t shared,
                                   cgtp_attn_cache* out) {
  return guarded([&] {
    need(out != nullptr, "out handle is NULL");
    *out = nullptr;
    need(attn != nullptr, "attn is NULL");
    need(slots >= 0 && capacity >= 1 && shared >= 0, "slots < 0, capacity < 1 or shared < 0");
    need_device(attn->device, "the attention");
    *out = build_attn_cache(attn, slots, capacity, shared);
  });
}

cgtp_status cgtp_attn_cache_destroy(cgtp_attn_cache cache) {
  return guarded([&] { delete cache; });
}

cgtp_status cgtp_attn_cache_query(cgtp_attn_cache cache, size_t* shared_bytes, size_t* ws_bytes) {
  return guarded([&] {
    need(cache != nullptr, "cache is NULL");
    if (shared_bytes) *shared_bytes = attn_cache_shared_bytes(cache);
    if (ws_bytes) *ws_bytes = attn_step_ws_bytes(cache);
  });
}

cgtp_status cgtp_attn_cache_share(cgtp_attn_cache cache, const void* k, int64_t ldk, const void* v, int64_t ldv,
                                  const uint8_t* key_mask, void* context, size_t context_bytes, void* stream) {
  return guarded([&] {
    need(cache != nullptr, "cache is NULL");
    need_device(cache->device, "the cache");
    need_rows(cache->shared, k, ldk, cache->attn->krow.dim, "k");
    need_rows(cache->shared, v, ldv, cache->attn->krow.dim, "v");
    need_ws(context, context_bytes, attn_cache_shared_bytes(cache), "the packed shared rows");
    attn_share_launch(cache, {k, ldk}, {v, ldv}, key_mask, context, as_stream(stream));
  });
}

cgtp_status cgtp_attn_step(cgtp_attn_cache cache, const void* q, int64_t ldq, const void* k, int64_t ldk,
                           const void* v, int64_t ldv, void* k_cache, void* v_cache, const int32_t* lengths,
                           const void* context, size_t context_bytes, double scale, void* out, float* lse, void* ws,
                           size_t ws_bytes, void* stream) {
  return guarded([&] {
    need(cache != nullptr, "cache is NULL");
    need_scale(scale);
    need_device(cache->device, "the cache");
    const cgtp_attn_s* a = cache->attn;
    need_rows(cache->slots, q, ldq, a->qrow.dim, "q");
    need_rows(cache->slots, k, ldk, a->krow.dim, "k");
    need_rows(cache->slots, v, ldv, a->krow.dim, "v");
    if (cache->slots == 0) return;
    need(k_cache && v_cache && lengths && out, "NULL cache, lengths or out");
    need_ws(const_cast<void*>(context), context_bytes, attn_cache_shared_bytes(cache), "the packed shared rows");
    need_ws(ws, ws_bytes, attn_step_ws_bytes(cache), "attention step");
    attn_step_launch(cache, {q, ldq}, {k, ldk}, {v, ldv}, k_cache, v_cache, lengths, context, scale, out, lse, ws,
                     as_stream(stream));
  });
}

}  // extern "C"
