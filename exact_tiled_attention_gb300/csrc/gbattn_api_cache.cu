// gbattn_api_cache.cu -- the C ABI of the operators around a paged cache:
// argument validation and dispatch (attn_qk_norm_rope, attn_cache_append,
// attn_cache_gather, attn_decode_paged, their 4-bit forms and the backward).
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/gbattn.h"
#include "gbattn_internal.h"

using namespace gbattn;

namespace {

bool misaligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }
bool misaligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) != 0; }

// The kernels count tokens in 32 bits (with room for a grid's step behind the last).
bool too_many_tokens(int B, int S) { return static_cast<long long>(B) * S > 0x40000000LL; }

// Strides (batch, head, seq) of a [B, heads, S, d] tensor from the caller's
// three values, or of the contiguous tensor when there are none.  Rows start on
// 16-byte boundaries, so each stride is a multiple of 8 elements.
bool row_strides(RowStrides* out, const long long* s, int heads, int S, int d) {
  if (s == nullptr) {
    *out = {static_cast<long long>(heads) * S * d, static_cast<long long>(S) * d, d};
    return true;
  }
  if ((s[0] | s[1] | s[2]) & 7) return false;
  *out = {s[0], s[1], s[2]};
  return true;
}

int check_rope(RopeArgs* out, const float* rope, int rows, int rot_dim, int interleaved, int d) {
  if (rot_dim < 0 || rot_dim > d || rot_dim % 16 != 0) return GBATTN_EPAGE;
  if (rot_dim > 0) {
    if (!rope || misaligned16(rope)) return GBATTN_EPOINTER;
    if (rows < 1) return GBATTN_EBADSHAPE;
  }
  *out = {rope, rows, rot_dim, interleaved ? 1 : 0};
  return GBATTN_OK;
}

// Sizes and pointers of a paged cache; factors are given for a 4-bit one only.
int check_cache(CacheArgs* out, const void* k, const void* v, const void* k_factors, const void* v_factors, bool fp4,
                const float* k_descale, const float* v_descale, const int* page_table, const int* seqlens, int Hkv,
                int d, int page_size, int n_pages, int max_pages) {
  if (Hkv < 1 || n_pages < 1 || max_pages < 1) return GBATTN_EBADSHAPE;
  if (d != 64 && d != 128) return GBATTN_EHEADDIM;
  if (page_size < 16 || page_size > 1024 || (page_size & (page_size - 1))) return GBATTN_EPAGE;
  if (static_cast<long long>(max_pages) * page_size > 0x7FFFFFFFLL - 256) return GBATTN_EBADSHAPE;
  // The kernels count blocks of 16 tokens of one head in 32 bits.
  if (static_cast<long long>(n_pages) * Hkv > (0x7FFFFFFFLL << 4) / page_size) return GBATTN_EBADSHAPE;
  if (!k || !v || !page_table || !seqlens || misaligned16(k) || misaligned16(v) || misaligned4(page_table) ||
      misaligned4(seqlens) || misaligned4(k_descale) || misaligned4(v_descale))
    return GBATTN_EPOINTER;
  if (fp4 && (!k_factors || !v_factors || misaligned16(k_factors) || misaligned16(v_factors))) return GBATTN_EPOINTER;
  CacheArgs c{};
  c.data[0] = const_cast<void*>(k);
  c.data[1] = const_cast<void*>(v);
  c.scale[0] = const_cast<void*>(k_factors);
  c.scale[1] = const_cast<void*>(v_factors);
  c.descale[0] = k_descale;
  c.descale[1] = v_descale;
  c.page_table = page_table;
  c.seqlens = seqlens;
  c.Hkv = Hkv;
  c.d = d;
  while ((1 << c.page_shift) < page_size) ++c.page_shift;
  c.n_pages = n_pages;
  c.max_pages = max_pages;
  *out = c;
  return GBATTN_OK;
}

int check_norm_rope(NormRopeArgs* a, const void* q, const void* k, const float* q_weight, const float* k_weight,
                    const float* rope, const int* positions, int B, int H, int Hkv, int S, int d,
                    const long long* q_strides, const long long* k_strides, float eps, int rope_rows, int rot_dim,
                    int interleaved, int dtype, void* stream) {
  if (B < 1 || H < 1 || Hkv < 1 || S < 1 || H > 16384 || Hkv > 16384) return GBATTN_EBADSHAPE;
  if (too_many_tokens(B, S)) return GBATTN_EBADSHAPE;
  if (H % Hkv != 0) return GBATTN_EHEADS;
  if (d != 64 && d != 128) return GBATTN_EHEADDIM;
  if (dtype != GBATTN_F16 && dtype != GBATTN_BF16) return GBATTN_EDTYPE;
  const int rc = check_rope(&a->rope, rope, rope_rows, rot_dim, interleaved, d);
  if (rc != GBATTN_OK) return rc;
  if (!q || !k || misaligned16(q) || misaligned16(k) || misaligned16(q_weight) || misaligned16(k_weight) ||
      misaligned4(positions) || !q_weight != !k_weight || (!q_weight && rot_dim == 0))
    return GBATTN_EPOINTER;
  // Without positions token s of every sequence has position s.
  if (rot_dim > 0 && !positions && rope_rows < S) return GBATTN_EBADSHAPE;
  if (!row_strides(&a->xs[0], q_strides, H, S, d) || !row_strides(&a->xs[1], k_strides, Hkv, S, d))
    return GBATTN_EPOINTER;
  a->x[0] = q;
  a->x[1] = k;
  a->w[0] = q_weight;
  a->w[1] = k_weight;
  a->positions = positions;
  a->heads[0] = H;
  a->heads[1] = Hkv;
  a->eps = eps;
  a->B = B;
  a->S = S;
  a->d = d;
  a->bf16 = dtype == GBATTN_BF16;
  a->stream = static_cast<cudaStream_t>(stream);
  return GBATTN_OK;
}

int append(const void* k, const void* v, void* k_cache, void* k_factors, void* v_cache, void* v_factors, bool fp4,
           const float* k_descale, const float* v_descale, const int* page_table, const int* seqlens,
           const int* new_lens, const float* rope, const void* q, void* q_out, int B, int H, int Hkv, int S, int d,
           int page_size, int n_pages, int max_pages, const long long* q_strides, const long long* k_strides,
           const long long* v_strides, int rope_rows, int rot_dim, int interleaved, int dtype, void* stream) {
  if (B < 1 || H < 1 || Hkv < 1 || S < 1 || H > 16384 || Hkv > 16384) return GBATTN_EBADSHAPE;
  if (too_many_tokens(B, S)) return GBATTN_EBADSHAPE;
  if (H % Hkv != 0) return GBATTN_EHEADS;
  AppendArgs a{};
  int rc = check_cache(&a.cache, k_cache, v_cache, k_factors, v_factors, fp4, k_descale, v_descale, page_table,
                       seqlens, Hkv, d, page_size, n_pages, max_pages);
  if (rc != GBATTN_OK) return rc;
  if (dtype != GBATTN_F16 && dtype != GBATTN_BF16) return GBATTN_EDTYPE;
  rc = check_rope(&a.rope, rope, rope_rows, rot_dim, interleaved, d);
  if (rc != GBATTN_OK) return rc;
  if (!k || !v || misaligned16(k) || misaligned16(v) || misaligned16(q) || misaligned16(q_out) || !q != !q_out ||
      misaligned4(new_lens))
    return GBATTN_EPOINTER;
  if (!row_strides(&a.xs[0], q_strides, H, S, d) || !row_strides(&a.xs[1], k_strides, Hkv, S, d) ||
      !row_strides(&a.xs[2], v_strides, Hkv, S, d))
    return GBATTN_EPOINTER;
  rc = current_device(&a.status, &a.num_sms);
  if (rc != GBATTN_OK) return rc;
  a.x[0] = q;
  a.x[1] = k;
  a.x[2] = v;
  a.q_out = q_out;
  a.new_lens = new_lens;
  a.B = B;
  a.H = H;
  a.S = S;
  a.bf16 = dtype == GBATTN_BF16;
  a.stream = static_cast<cudaStream_t>(stream);
  return launch_cache_append(a) == 0 ? GBATTN_OK : GBATTN_ELAUNCH;
}

int gather(const void* k_cache, const void* k_factors, const void* v_cache, const void* v_factors, bool fp4,
           const float* k_descale, const float* v_descale, const int* page_table, const int* seqlens, void* k_out,
           void* v_out, int B, int Hkv, int S, int d, int page_size, int n_pages, int max_pages, int dtype,
           void* stream) {
  if (B < 1 || Hkv < 1 || S < 1 || S > 0x40000000 || static_cast<long long>(B) * Hkv > 65535) return GBATTN_EBADSHAPE;
  GatherArgs a{};
  int rc = check_cache(&a.cache, k_cache, v_cache, k_factors, v_factors, fp4, k_descale, v_descale, page_table,
                       seqlens, Hkv, d, page_size, n_pages, max_pages);
  if (rc != GBATTN_OK) return rc;
  if (dtype != GBATTN_F16 && dtype != GBATTN_BF16) return GBATTN_EDTYPE;
  if (!k_out || !v_out || misaligned16(k_out) || misaligned16(v_out)) return GBATTN_EPOINTER;
  rc = current_device(&a.status, &a.num_sms);
  if (rc != GBATTN_OK) return rc;
  a.out[0] = k_out;
  a.out[1] = v_out;
  a.B = B;
  a.S = S;
  a.bf16 = dtype == GBATTN_BF16;
  a.stream = static_cast<cudaStream_t>(stream);
  return launch_cache_gather(a) == 0 ? GBATTN_OK : GBATTN_ELAUNCH;
}

int decode(const void* q, const void* k_cache, const void* k_factors, const void* v_cache, const void* v_factors,
           bool fp4, const float* k_descale, const float* v_descale, const int* page_table, const int* seqlens,
           void* o, float* lse, int B, int Hq, int Hkv, int d, int page_size, int n_pages, int max_pages, float scale,
           void* workspace, size_t workspace_bytes, int dtype, void* stream) {
  if (B < 1 || Hq < 1 || Hkv < 1 || B > 65535 || Hq > 16384) return GBATTN_EBADSHAPE;
  if (Hq % Hkv != 0) return GBATTN_EHEADS;
  PagedDecodeArgs a{};
  int rc = check_cache(&a.cache, k_cache, v_cache, k_factors, v_factors, fp4, k_descale, v_descale, page_table,
                       seqlens, Hkv, d, page_size, n_pages, max_pages);
  if (rc != GBATTN_OK) return rc;
  if (dtype != GBATTN_F16 && dtype != GBATTN_BF16) return GBATTN_EDTYPE;
  if (!q || !o || !workspace || misaligned16(q) || misaligned16(o) || misaligned16(workspace) || misaligned4(lse))
    return GBATTN_EPOINTER;
  if (workspace_bytes < paged_decode_workspace_bytes(B, Hq, Hkv, d, max_pages * page_size)) return GBATTN_EWORKSPACE;
  rc = current_device(&a.status, &a.num_sms);
  if (rc != GBATTN_OK) return rc;
  a.q = q;
  a.o = o;
  a.lse = lse;
  a.B = B;
  a.Hq = Hq;
  a.scale = scale;
  a.workspace = workspace;
  a.bf16 = dtype == GBATTN_BF16;
  a.stream = static_cast<cudaStream_t>(stream);
  return launch_decode_paged(a) == 0 ? GBATTN_OK : GBATTN_ELAUNCH;
}

}  // namespace

extern "C" {

int attn_qk_norm_rope(const void* q, const void* k, const float* q_weight, const float* k_weight, const float* rope,
                      const int* positions, void* q_out, void* k_out, int B, int H, int Hkv, int S, int d,
                      const long long* q_strides, const long long* k_strides, float eps, int rope_rows, int rot_dim,
                      int interleaved, int dtype, void* stream) {
  NormRopeArgs a{};
  int rc = check_norm_rope(&a, q, k, q_weight, k_weight, rope, positions, B, H, Hkv, S, d, q_strides, k_strides, eps,
                           rope_rows, rot_dim, interleaved, dtype, stream);
  if (rc != GBATTN_OK) return rc;
  if (!q_out || !k_out || misaligned16(q_out) || misaligned16(k_out)) return GBATTN_EPOINTER;
  rc = current_device(&a.status, &a.num_sms);
  if (rc != GBATTN_OK) return rc;
  a.y[0] = q_out;
  a.y[1] = k_out;
  return launch_norm_rope(a) == 0 ? GBATTN_OK : GBATTN_ELAUNCH;
}

size_t attn_qk_norm_rope_bwd_workspace_bytes(int d) {
  return d == 64 || d == 128 ? norm_rope_bwd_workspace_bytes(d) : 0;
}

int attn_qk_norm_rope_bwd(const void* dq_out, const void* dk_out, const void* q, const void* k, const float* q_weight,
                          const float* k_weight, const float* rope, const int* positions, void* dq, void* dk,
                          float* dq_weight, float* dk_weight, int B, int H, int Hkv, int S, int d,
                          const long long* q_strides, const long long* k_strides, const long long* dq_strides,
                          const long long* dk_strides, float eps, int rope_rows, int rot_dim, int interleaved,
                          void* workspace, size_t workspace_bytes, int dtype, void* stream) {
  NormRopeArgs a{};
  int rc = check_norm_rope(&a, q, k, q_weight, k_weight, rope, positions, B, H, Hkv, S, d, q_strides, k_strides, eps,
                           rope_rows, rot_dim, interleaved, dtype, stream);
  if (rc != GBATTN_OK) return rc;
  if (!dq_out || !dk_out || !dq || !dk || misaligned16(dq_out) || misaligned16(dk_out) || misaligned16(dq) ||
      misaligned16(dk))
    return GBATTN_EPOINTER;
  if (!row_strides(&a.dxs[0], dq_strides, H, S, d) || !row_strides(&a.dxs[1], dk_strides, Hkv, S, d))
    return GBATTN_EPOINTER;
  if (q_weight) {
    if (!dq_weight || !dk_weight || !workspace || misaligned4(dq_weight) || misaligned4(dk_weight) ||
        misaligned16(workspace))
      return GBATTN_EPOINTER;
    if (workspace_bytes < norm_rope_bwd_workspace_bytes(d)) return GBATTN_EWORKSPACE;
  }
  rc = current_device(&a.status, &a.num_sms);
  if (rc != GBATTN_OK) return rc;
  a.dy[0] = dq_out;
  a.dy[1] = dk_out;
  a.dx[0] = dq;
  a.dx[1] = dk;
  a.dw[0] = dq_weight;
  a.dw[1] = dk_weight;
  a.workspace = static_cast<float*>(workspace);
  return launch_norm_rope_bwd(a) == 0 ? GBATTN_OK : GBATTN_ELAUNCH;
}

int attn_cache_append(const void* k, const void* v, void* k_cache, void* v_cache, const int* page_table,
                      const int* seqlens, const int* new_lens, const float* rope, const void* q, void* q_out, int B,
                      int H, int Hkv, int S, int d, int page_size, int n_pages, int max_pages,
                      const long long* q_strides, const long long* k_strides, const long long* v_strides,
                      int rope_rows, int rot_dim, int interleaved, int dtype, void* stream) {
  return append(k, v, k_cache, nullptr, v_cache, nullptr, false, nullptr, nullptr, page_table, seqlens, new_lens, rope,
                q, q_out, B, H, Hkv, S, d, page_size, n_pages, max_pages, q_strides, k_strides, v_strides, rope_rows,
                rot_dim, interleaved, dtype, stream);
}

int attn_cache_append_fp4(const void* k, const void* v, void* k_codes, void* k_factors, void* v_codes,
                          void* v_factors, const float* k_descale, const float* v_descale, const int* page_table,
                          const int* seqlens, const int* new_lens, const float* rope, const void* q, void* q_out,
                          int B, int H, int Hkv, int S, int d, int page_size, int n_pages, int max_pages,
                          const long long* q_strides, const long long* k_strides, const long long* v_strides,
                          int rope_rows, int rot_dim, int interleaved, int dtype, void* stream) {
  return append(k, v, k_codes, k_factors, v_codes, v_factors, true, k_descale, v_descale, page_table, seqlens,
                new_lens, rope, q, q_out, B, H, Hkv, S, d, page_size, n_pages, max_pages, q_strides, k_strides,
                v_strides, rope_rows, rot_dim, interleaved, dtype, stream);
}

int attn_cache_gather(const void* k_cache, const void* v_cache, const int* page_table, const int* seqlens,
                      void* k_out, void* v_out, int B, int Hkv, int S, int d, int page_size, int n_pages,
                      int max_pages, int dtype, void* stream) {
  return gather(k_cache, nullptr, v_cache, nullptr, false, nullptr, nullptr, page_table, seqlens, k_out, v_out, B, Hkv,
                S, d, page_size, n_pages, max_pages, dtype, stream);
}

int attn_cache_gather_fp4(const void* k_codes, const void* k_factors, const void* v_codes, const void* v_factors,
                          const float* k_descale, const float* v_descale, const int* page_table, const int* seqlens,
                          void* k_out, void* v_out, int B, int Hkv, int S, int d, int page_size, int n_pages,
                          int max_pages, int dtype, void* stream) {
  return gather(k_codes, k_factors, v_codes, v_factors, true, k_descale, v_descale, page_table, seqlens, k_out, v_out,
                B, Hkv, S, d, page_size, n_pages, max_pages, dtype, stream);
}

size_t attn_decode_paged_workspace_bytes(int B, int Hq, int Hkv, int d, int max_len) {
  if (B < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || d < 1 || max_len < 1) return 0;
  return paged_decode_workspace_bytes(B, Hq, Hkv, d, max_len);
}

int attn_decode_paged(const void* q, const void* k_cache, const void* v_cache, const int* page_table,
                      const int* seqlens, void* o, float* lse, int B, int Hq, int Hkv, int d, int page_size,
                      int n_pages, int max_pages, float scale, void* workspace, size_t workspace_bytes, int dtype,
                      void* stream) {
  return decode(q, k_cache, nullptr, v_cache, nullptr, false, nullptr, nullptr, page_table, seqlens, o, lse, B, Hq,
                Hkv, d, page_size, n_pages, max_pages, scale, workspace, workspace_bytes, dtype, stream);
}

int attn_decode_paged_fp4(const void* q, const void* k_codes, const void* k_factors, const void* v_codes,
                          const void* v_factors, const float* k_descale, const float* v_descale,
                          const int* page_table, const int* seqlens, void* o, float* lse, int B, int Hq, int Hkv,
                          int d, int page_size, int n_pages, int max_pages, float scale, void* workspace,
                          size_t workspace_bytes, int dtype, void* stream) {
  return decode(q, k_codes, k_factors, v_codes, v_factors, true, k_descale, v_descale, page_table, seqlens, o, lse, B,
                Hq, Hkv, d, page_size, n_pages, max_pages, scale, workspace, workspace_bytes, dtype, stream);
}

}  // extern "C"
