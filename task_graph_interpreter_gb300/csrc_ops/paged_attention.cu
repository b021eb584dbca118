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
            const cuuint64_t* stride, const cuuint32_t* box, CUtensorMapDataType type = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
            CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B) {
  const cuuint32_t one[3] = {1, 1, 1};
  return enc(m, type, (cuuint32_t)rank, const_cast<void*>(ptr), dim, stride, box, one,
             CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Few query rows or chunks: a request and head of at most eight rows fills one
// warp product; beyond that the 128-row tensor-core tiles are faster although
// mostly empty (paged_rows.cu has both sides).  Over e4m3 pages two eights have
// as many bytes to wait for per key as one over bf16 pages: 12 and 16 rows take
// there and as chunks 56 and 93 us (64 requests of 512 to 2048 keys), 46 and 56
// (16 of 512 to 8192), 66 and 64 (4 of 32768), 24 and 20 (one of 8192); with 20
// rows and three eights 4 requests of 32768 keys took 95 us, 64 as chunks.
bool few_rows(int max_new, int G, bool e4m3) { return (int64_t)max_new * G <= (e4m3 ? kMaxFewRows8 : kMaxFewRows); }

// Two partial records and a note per worker (paged_attention.cuh).
size_t workspace_bytes(int max_new, int G, int D, int sms, bool e4m3) {
  const bool few = few_rows(max_new, G, e4m3);
  const size_t workers = (size_t)sms * (!few ? 1 : e4m3 ? kRowWarps8 : kRowWarps), rows = few ? max_new * G : kTileRows;
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

static int attention_workspace(const char* who, bool e4m3, int max_new, int Hq, int Hkv, int D, size_t* bytes) {
  if (!bytes) return fail(MK_ERR_ARG, std::string(who) + ": null argument");
  if (int rc = check_shape(who, max_new, Hq, Hkv, D)) return rc;
  int sms = 0;
  if (int rc = device_sms(who, &sms)) return rc;
  *bytes = workspace_bytes(max_new, Hq / Hkv, D, sms, e4m3);
  return MK_OK;
}

extern "C" int mk_paged_attention_workspace(int max_new, int Hq, int Hkv, int D, size_t* bytes) try {
  return attention_workspace("mk_paged_attention_workspace", false, max_new, Hq, Hkv, D, bytes);
} catch (...) {
  return MK_ERR_NOMEM;
}

extern "C" int mk_paged_attention_e4m3_workspace(int max_new, int Hq, int Hkv, int D, size_t* bytes) try {
  return attention_workspace("mk_paged_attention_e4m3_workspace", true, max_new, Hq, Hkv, D, bytes);
} catch (...) {
  return MK_ERR_NOMEM;
}

// Both forms of the operator: e4m3 pages have scales, bf16 pages none.
static int attention(const char* who, bool e4m3, void* stream_, int B, int N, int max_new, int Hq, int Hkv, int D,
                     const void* q, int64_t ld_q, const void* kpool, const void* vpool, const float* kscale,
                     const float* vscale, int num_pages, int page_size, const int32_t* table, int max_pages,
                     const int32_t* cu, const int32_t* ctx_len, float scale, void* out, int64_t ld_out, void* workspace,
                     size_t workspace_size, int32_t* status) {
  const auto refuse = [who](int code, const std::string& why) { return fail(code, std::string(who) + ": " + why); };
  if (!q || !kpool || !vpool || !table || !cu || !ctx_len || !out || !workspace ||
      (e4m3 && (!kscale || !vscale)))
    return refuse(MK_ERR_ARG, "null argument");
  if (int rc = check_shape(who, max_new, Hq, Hkv, D)) return rc;
  if (B < 0 || N < 0 || max_pages < 1) return refuse(MK_ERR_ARG, "need B, N >= 0 and max_pages >= 1");
  if (!page_size_ok(page_size))
    return refuse(MK_ERR_ARG, "page_size must be 16, 32, 64, 128 or 256");
  // (positions are counted on to the end of a block of 128 keys, and past a request's last token to the end of two
  // tiles' rows: at most 254)
  if (num_pages < 1 || (int64_t)num_pages * Hkv * page_size > INT32_MAX ||
      (int64_t)max_pages * page_size > INT32_MAX - 255)
    return refuse(MK_ERR_ARG, "rows of the pools must fit int32, max_pages * page_size 2^31 - 256");
  if (ld_q < (int64_t)Hq * D || ld_q % 8 || ld_out < (int64_t)Hq * D || ld_out % 8)
    return refuse(MK_ERR_ARG, "row strides must cover a row and be multiples of 16 bytes");
  if (!aligned16(q) || !aligned16(kpool) || !aligned16(vpool) || !aligned16(out) || !aligned16(workspace))
    return refuse(MK_ERR_ARG, "pointers must be 16-byte aligned");
  if (!(scale > 0.f) || !std::isfinite(scale)) return refuse(MK_ERR_ARG, "scale must be positive");
  if (int rc = pending_error(who)) return rc;
  int sms = 0;
  if (int rc = device_sms(who, &sms)) return rc;
  const int G = Hq / Hkv;
  if (workspace_size < workspace_bytes(max_new, G, D, sms, e4m3))
    return refuse(MK_ERR_LIMIT, "the workspace needs " +
                                  std::to_string(workspace_bytes(max_new, G, D, sms, e4m3)) + " bytes");
  if (B == 0 || N == 0) return MK_OK;
  EncodeTiledFn enc = encoder();
  if (!enc) return refuse(MK_ERR_CUDA, "cuTensorMapEncodeTiled is not available");

  const bool few = few_rows(max_new, G, e4m3);
  Attn8Params p{};
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.v = static_cast<const __nv_bfloat16*>(vpool);
  p.v8 = static_cast<const uint8_t*>(vpool);
  p.kscale = kscale; p.vscale = vscale;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.ld_q = ld_q; p.ld_out = ld_out;
  p.table = table; p.cu = cu; p.ctx = ctx_len;
  p.part = static_cast<float*>(workspace);
  p.status = status;
  p.scale = scale * 1.4426950408889634f;
  p.B = B; p.N = N; p.Hq = Hq; p.Hkv = Hkv; p.G = G; p.max_new = max_new;
  p.max_pages = max_pages; p.num_pages = num_pages;
  while ((1 << p.page_shift) < page_size) ++p.page_shift;
  p.workers = sms * (!few ? 1 : e4m3 ? kRowWarps8 : kRowWarps);
  p.rows = few ? max_new * G : kTileRows;
  p.tq = few ? 0 : 128 / G;
  // The chunk kernel's softmax of a tile without tokens, and its warp for masked values, wait while a part's other
  // blocks go by: 65536 blocks of 128 keys take 48 ms and more.
  p.wait_limit = 1 + (int)((int64_t)max_pages * page_size >> 23);

  // pools as [rows, D], pages one after the other; a box is what one page gives a block of keys
  CUtensorMap kmap, vmap, qmap;
  const int keys = !few ? 128 : e4m3 ? kRowBlockBytes8 / D / 2 : kRowBlockBytes / D / 4, size = e4m3 ? 1 : 2;
  const cuuint64_t dim[2] = {(cuuint64_t)D, (cuuint64_t)num_pages * Hkv * page_size}, stride[1] = {(cuuint64_t)D * size};
  const cuuint32_t box[2] = {e4m3 ? (cuuint32_t)D : 64u, (cuuint32_t)(page_size < keys ? page_size : keys)};
  const CUtensorMapDataType type = e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const CUtensorMapSwizzle swizzle = e4m3 && D == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B;
  bool ok = encode(enc, &kmap, kpool, 2, dim, stride, box, type, swizzle) &&
            encode(enc, &vmap, vpool, 2, dim, stride, box, type, swizzle);
  if (ok && !few) {
    const cuuint64_t qdim[3] = {(cuuint64_t)D, (cuuint64_t)Hq, (cuuint64_t)N};
    const cuuint64_t qstride[2] = {(cuuint64_t)D * 2, (cuuint64_t)ld_q * 2};
    const cuuint32_t qbox[3] = {64u, (cuuint32_t)G, (cuuint32_t)p.tq};
    ok = encode(enc, &qmap, q, 3, qdim, qstride, qbox);
  }
  if (!ok) return refuse(MK_ERR_CUDA, "a tensor map could not be encoded");
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  const cudaError_t e = e4m3 ? few ? launch_rows8(p, kmap, vmap, D, stream) : launch_chunk8(p, qmap, kmap, vmap, D, stream)
                        : few ? launch_rows(p, kmap, vmap, D, stream)
                              : launch_chunk(p, qmap, kmap, vmap, D, stream);
  if (int rc = launch_result(e, who)) return rc;
  return launch_result(launch_join(p, D, !few, stream), who);
}

extern "C" int mk_paged_attention(void* stream, int B, int N, int max_new, int Hq, int Hkv, int D, const void* q,
                                  int64_t ld_q, const void* kpool, const void* vpool, int num_pages, int page_size,
                                  const int32_t* table, int max_pages, const int32_t* cu, const int32_t* ctx_len,
                                  float scale, void* out, int64_t ld_out, void* workspace, size_t workspace_size,
                                  int32_t* status) try {
  return attention("mk_paged_attention", false, stream, B, N, max_new, Hq, Hkv, D, q, ld_q, kpool, vpool, nullptr, nullptr,
                   num_pages, page_size, table, max_pages, cu, ctx_len, scale, out, ld_out, workspace, workspace_size,
                   status);
} catch (...) {
  return MK_ERR_NOMEM;
}

extern "C" int mk_paged_attention_e4m3(void* stream, int B, int N, int max_new, int Hq, int Hkv, int D, const void* q,
                                       int64_t ld_q, const void* kpool, const void* vpool, const float* kscale,
                                       const float* vscale, int num_pages, int page_size, const int32_t* table,
                                       int max_pages, const int32_t* cu, const int32_t* ctx_len, float scale, void* out,
                                       int64_t ld_out, void* workspace, size_t workspace_size, int32_t* status) try {
  return attention("mk_paged_attention_e4m3", true, stream, B, N, max_new, Hq, Hkv, D, q, ld_q, kpool, vpool, kscale,
                   vscale, num_pages, page_size, table, max_pages, cu, ctx_len, scale, out, ld_out, workspace,
                   workspace_size, status);
} catch (...) {
  return MK_ERR_NOMEM;
}
