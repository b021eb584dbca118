// Entry points of paged attention: checks, tensor maps, the choice of kernel.
#include <atomic>
#include <cmath>

#include "paged_attention.cuh"

namespace mk {

cudaError_t launch_join(const AttnParams& p, int D, bool chunk, cudaStream_t stream);

namespace {

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encoder() {
  static std::atomic<EncodeTiledFn> known{nullptr};
  EncodeTiledFn fn = known.load();
  if (fn) return fn;
  void* f = nullptr;
  cudaDriverEntryPointQueryResult q;
  if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
      q != cudaDriverEntryPointSuccess || !f)
    return nullptr;
  fn = reinterpret_cast<EncodeTiledFn>(f);
  known.store(fn);
  return fn;
}

bool encode(EncodeTiledFn enc, CUtensorMap* m, const void* ptr, int rank, const cuuint64_t* dim,
            const cuuint64_t* stride, const cuuint32_t* box) {
  const cuuint32_t one[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)rank, const_cast<void*>(ptr), dim, stride, box, one,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Few query rows or chunks: a request and head of at most eight rows fills one
// warp product; beyond that the 128-row tensor-core tiles are faster although
// mostly empty (paged_rows.cu has both sides).
bool few_rows(int max_new, int G) { return (int64_t)max_new * G <= kMaxFewRows; }

// Two partial records and a note per worker (paged_attention.cuh).
size_t workspace_bytes(int max_new, int G, int D, int sms) {
  const bool few = few_rows(max_new, G);
  const size_t workers = (size_t)sms * (few ? kRowWarps : 1), rows = few ? max_new * G : kTileRows;
  return 2 * workers * rows * (D + 2) * 4 + workers * 16;
}

int check_shape(const char* who, int max_new, int Hq, int Hkv, int D) {
  if (D != 64 && D != 128) return fail(MK_ERR_ARG, std::string(who) + ": D must be 64 or 128");
  if (Hkv < 1 || Hkv > 1024 || Hq < Hkv || Hq % Hkv || Hq / Hkv > 128)
    return fail(MK_ERR_ARG, std::string(who) + ": need Hq a multiple of Hkv (at most 1024) with Hq/Hkv <= 128");
  if (max_new < 1) return fail(MK_ERR_ARG, std::string(who) + ": max_new must be positive");
  return MK_OK;
}

}  // namespace
}  // namespace mk

using namespace mk;

extern "C" int mk_paged_attention_workspace(int max_new, int Hq, int Hkv, int D, size_t* bytes) try {
  if (!bytes) return fail(MK_ERR_ARG, "mk_paged_attention_workspace: null argument");
  if (int rc = check_shape("mk_paged_attention_workspace", max_new, Hq, Hkv, D)) return rc;
  int sms = 0;
  if (int rc = device_sms("mk_paged_attention_workspace", &sms)) return rc;
  *bytes = workspace_bytes(max_new, Hq / Hkv, D, sms);
  return MK_OK;
} catch (...) {
  return MK_ERR_NOMEM;
}

extern "C" int mk_paged_attention(void* stream_, int B, int N, int max_new, int Hq, int Hkv, int D, const void* q,
                                  int64_t ld_q, const void* kpool, const void* vpool, int num_pages, int page_size,
                                  const int32_t* table, int max_pages, const int32_t* cu, const int32_t* ctx_len,
                                  float scale, void* out, int64_t ld_out, void* workspace, size_t workspace_size,
                                  int32_t* status) try {
  const char* who = "mk_paged_attention";
  if (!q || !kpool || !vpool || !table || !cu || !ctx_len || !out || !workspace)
    return fail(MK_ERR_ARG, "mk_paged_attention: null argument");
  if (int rc = check_shape(who, max_new, Hq, Hkv, D)) return rc;
  if (B < 0 || N < 0 || max_pages < 1) return fail(MK_ERR_ARG, "mk_paged_attention: need B, N >= 0 and max_pages >= 1");
  if (!page_size_ok(page_size))
    return fail(MK_ERR_ARG, "mk_paged_attention: page_size must be 16, 32, 64, 128 or 256");
  // (positions are counted on to the end of a block of 128 keys, and past a request's last token to the end of two
  // tiles' rows: at most 254)
  if (num_pages < 1 || (int64_t)num_pages * Hkv * page_size > INT32_MAX ||
      (int64_t)max_pages * page_size > INT32_MAX - 255)
    return fail(MK_ERR_ARG, "mk_paged_attention: rows of the pools must fit int32, max_pages * page_size 2^31 - 256");
  if (ld_q < (int64_t)Hq * D || ld_q % 8 || ld_out < (int64_t)Hq * D || ld_out % 8)
    return fail(MK_ERR_ARG, "mk_paged_attention: row strides must cover a row and be multiples of 16 bytes");
  if (!aligned16(q) || !aligned16(kpool) || !aligned16(vpool) || !aligned16(out) || !aligned16(workspace))
    return fail(MK_ERR_ARG, "mk_paged_attention: pointers must be 16-byte aligned");
  if (!(scale > 0.f) || !std::isfinite(scale)) return fail(MK_ERR_ARG, "mk_paged_attention: scale must be positive");
  if (int rc = pending_error(who)) return rc;
  int sms = 0;
  if (int rc = device_sms(who, &sms)) return rc;
  const int G = Hq / Hkv;
  if (workspace_size < workspace_bytes(max_new, G, D, sms))
    return fail(MK_ERR_LIMIT, "mk_paged_attention: the workspace needs " +
                                  std::to_string(workspace_bytes(max_new, G, D, sms)) + " bytes");
  if (B == 0 || N == 0) return MK_OK;
  EncodeTiledFn enc = encoder();
  if (!enc) return fail(MK_ERR_CUDA, "mk_paged_attention: cuTensorMapEncodeTiled is not available");

  const bool few = few_rows(max_new, G);
  AttnParams p{};
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.v = static_cast<const __nv_bfloat16*>(vpool);
  p.out = static_cast<__nv_bfloat16*>(out);
  p.ld_q = ld_q; p.ld_out = ld_out;
  p.table = table; p.cu = cu; p.ctx = ctx_len;
  p.part = static_cast<float*>(workspace);
  p.status = status;
  p.scale = scale * 1.4426950408889634f;
  p.B = B; p.N = N; p.Hq = Hq; p.Hkv = Hkv; p.G = G; p.max_new = max_new;
  p.max_pages = max_pages; p.num_pages = num_pages;
  while ((1 << p.page_shift) < page_size) ++p.page_shift;
  p.workers = few ? sms * kRowWarps : sms;
  p.rows = few ? max_new * G : kTileRows;
  p.tq = few ? 0 : 128 / G;
  // The chunk kernel's softmax of a tile without tokens, and its warp for masked values, wait while a part's other
  // blocks go by: 65536 blocks of 128 keys take 48 ms and more.
  p.wait_limit = 1 + (int)((int64_t)max_pages * page_size >> 23);

  // pools as [rows, D], pages one after the other; a box is what one page gives a block of keys
  CUtensorMap kmap, vmap, qmap;
  const int keys = few ? kRowBlockBytes / D / 4 : 128;
  const cuuint64_t dim[2] = {(cuuint64_t)D, (cuuint64_t)num_pages * Hkv * page_size}, stride[1] = {(cuuint64_t)D * 2};
  const cuuint32_t box[2] = {64u, (cuuint32_t)(page_size < keys ? page_size : keys)};
  bool ok = encode(enc, &kmap, kpool, 2, dim, stride, box) && encode(enc, &vmap, vpool, 2, dim, stride, box);
  if (ok && !few) {
    const cuuint64_t qdim[3] = {(cuuint64_t)D, (cuuint64_t)Hq, (cuuint64_t)N};
    const cuuint64_t qstride[2] = {(cuuint64_t)D * 2, (cuuint64_t)ld_q * 2};
    const cuuint32_t qbox[3] = {64u, (cuuint32_t)G, (cuuint32_t)p.tq};
    ok = encode(enc, &qmap, q, 3, qdim, qstride, qbox);
  }
  if (!ok) return fail(MK_ERR_CUDA, "mk_paged_attention: a tensor map could not be encoded");
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  if (int rc = launch_result(few ? launch_rows(p, kmap, vmap, D, stream) : launch_chunk(p, qmap, kmap, vmap, D, stream),
                             who))
    return rc;
  return launch_result(launch_join(p, D, !few, stream), who);
} catch (...) {
  return MK_ERR_NOMEM;
}
