// What the norm, rotation and store operators share (bf16 pages and e4m3
// pages): parameters, loads of a lane's elements, argument checks, and the
// rotation's frequencies.
#pragma once

#include <cmath>

#include <cuda_bf16.h>

#include "paged.h"
#include "ptx_ops.cuh"

namespace mk {

struct NormParams {
  const void* x;
  int64_t ld_x, ld_q;
  const __nv_bfloat16 *q_gamma, *k_gamma;
  const int32_t *positions, *slots;
  __nv_bfloat16 *q, *kpool, *vpool;
  int32_t* status;
  int N, Hq, Hkv, page_shift, num_pages;
  int tokens, splits;  // tokens of a block; blocks that share a token's heads
  float eps;
  uint64_t freq[64];  // [D / 2]
};

// E elements as they come, and as floats
template <typename T, int E>
struct Raw;
template <int E>
struct Raw<float, E> {
  float4 v[E / 4];
  __device__ __forceinline__ void load(const float* p) {
#pragma unroll
    for (int i = 0; i < E / 4; ++i) v[i] = __ldg(reinterpret_cast<const float4*>(p) + i);
  }
  __device__ __forceinline__ void get(float (&f)[E]) const {
#pragma unroll
    for (int i = 0; i < E / 4; ++i) {
      f[4 * i] = v[i].x; f[4 * i + 1] = v[i].y; f[4 * i + 2] = v[i].z; f[4 * i + 3] = v[i].w;
    }
  }
};
template <int E>
struct Raw<__nv_bfloat16, E> {
  uint2 v[E / 4];
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    if constexpr (E == 8) {
      const uint4 t = __ldg(reinterpret_cast<const uint4*>(p));
      v[0] = make_uint2(t.x, t.y);
      v[1] = make_uint2(t.z, t.w);
    } else {
      v[0] = __ldg(reinterpret_cast<const uint2*>(p));
    }
  }
  __device__ __forceinline__ void get(float (&f)[E]) const {
#pragma unroll
    for (int i = 0; i < E / 4; ++i) {
      f[4 * i] = ptx::bf_lo(v[i].x); f[4 * i + 1] = ptx::bf_hi(v[i].x);
      f[4 * i + 2] = ptx::bf_lo(v[i].y); f[4 * i + 3] = ptx::bf_hi(v[i].y);
    }
  }
};
template <int E>
__device__ __forceinline__ void store_half(__nv_bfloat16* p, const float (&v)[E]) {
  if constexpr (E == 8)
    *reinterpret_cast<uint4*>(p) =
        make_uint4(ptx::pack_bf16(v[0], v[1]), ptx::pack_bf16(v[2], v[3]), ptx::pack_bf16(v[4], v[5]), ptx::pack_bf16(v[6], v[7]));
  else
    *reinterpret_cast<uint2*>(p) = make_uint2(ptx::pack_bf16(v[0], v[1]), ptx::pack_bf16(v[2], v[3]));
}


// Norms and rotation of the query heads alone, beside the launch before it, which calls launch_dependents() and makes
// nothing that this one reads.
cudaError_t launch_queries(const NormParams& p, int dtype, int D, int sms, cudaStream_t stream);

inline int check_norm(const char* who, int N, int Hq, int Hkv, int D, const void* qkv, int qkv_dtype, int64_t ld_qkv,
                      const void* q_gamma, const void* k_gamma, float eps, double rope_theta, const int32_t* positions,
                      const int32_t* slots, const void* q_out, int64_t ld_q, const void* kpool, const void* vpool,
                      int num_pages, int page_size) {
  if (!qkv || !positions || !slots || !q_out || !kpool || !vpool)
    return fail(MK_ERR_ARG, std::string(who) + ": null argument");
  if (N < 0 || Hq < 1 || Hkv < 1 || Hq > 1024 || Hkv > 1024)
    return fail(MK_ERR_ARG, std::string(who) + ": need N >= 0 and 1 to 1024 heads");
  if (D != 64 && D != 128) return fail(MK_ERR_ARG, std::string(who) + ": D must be 64 or 128");
  if (qkv_dtype != MK_F32 && qkv_dtype != MK_BF16) return fail(MK_ERR_ARG, std::string(who) + ": qkv must be f32 or bf16");
  if (!page_size_ok(page_size)) return fail(MK_ERR_ARG, std::string(who) + ": page_size must be 16, 32, 64, 128 or 256");
  if (num_pages < 1 || (int64_t)num_pages * page_size > INT32_MAX)
    return fail(MK_ERR_ARG, std::string(who) + ": num_pages * page_size must be in [1, 2^31)");
  if (!(rope_theta > 0.0) || !std::isfinite(rope_theta) || !(eps >= 0.f) || !std::isfinite(eps))
    return fail(MK_ERR_ARG, std::string(who) + ": bad rope_theta or eps");
  const int64_t width = (int64_t)(Hq + 2 * Hkv) * D, unit = qkv_dtype == MK_F32 ? 4 : 8;
  if (ld_qkv < width || ld_qkv % unit || ld_q < (int64_t)Hq * D || ld_q % 8)
    return fail(MK_ERR_ARG, std::string(who) + ": row strides must cover a row and be multiples of 16 bytes");
  if (!aligned16(qkv) || !aligned16(q_out) || !aligned16(kpool) || !aligned16(vpool) || !aligned16(q_gamma) ||
      !aligned16(k_gamma))
    return fail(MK_ERR_ARG, std::string(who) + ": pointers must be 16-byte aligned");
  return MK_OK;
}

inline void rope_frequencies(double rope_theta, int D, uint64_t* freq) {
  // the last base's frequencies: a decoder asks for the same ones in every layer
  thread_local struct {
    double theta = 0.0;
    int D = 0;
    uint64_t f[64];
  } known;
  if (known.theta != rope_theta || known.D != D) {
    for (int i = 0; i < D / 2; ++i) {
      // revolutions per position, reduced below one, in units of 2^-64
      const double f = std::fmod(std::pow(rope_theta, -2.0 * i / D) / 6.283185307179586476925, 1.0);
      known.f[i] = (uint64_t)std::ldexp(f, 64);
    }
    known.theta = rope_theta;
    known.D = D;
  }
  for (int i = 0; i < D / 2; ++i) freq[i] = known.f[i];
}

}  // namespace mk
