// What the tensor-core attention kernels share: tensor memory loads and
// stores, the MMA forms, the layouts of key and value tiles in shared memory, and
// the TMA maps of a paged cache.
#pragma once

#include <cstring>

#include "attention_common.cuh"
#include "quant_common.cuh"

namespace moe {

constexpr int kKeys = 128;                     // keys per tile
// A BF16 weight above this (2^40) moves its row's reference: sums of weights times values stay in
// binary32 for values to 2^70 over 2^17 keys, and scores must rise by 28 to get there.  (2^24:
// scores of a standard deviation of 12 move it in many tiles, 4096 tokens over 16384 positions 743
// instead of 655 us; 2^60: values of 2^60 overflow.)
constexpr float kFarWeight = 1099511627776.0f;
constexpr uint32_t kHalfBytes = kKeys * 128;   // 64 bf16 channels of 128 rows

// The 16-byte piece c of row r of a tile of codes (rows of D bytes, the
// swizzle of that width).
template <int D>
__device__ __forceinline__ uint32_t code_piece(int r, int c) {
  return r * D + ((c ^ (D == 128 ? (r & 7) : ((r >> 1) & 3))) << 4);
}
// High descriptor word of a K-major tile of codes: 8-row groups of 8 * D bytes,
// 128- or 64-byte swizzle.
template <int D>
constexpr uint32_t kCodeDescHi = ((8u * D) >> 4) | (1u << 14) | ((D == 128 ? 2u : 4u) << 29);

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float* v) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

// tcgen05.wait::ld with the 32 registers of an earlier load passed through it,
// so that their first use stays below the wait
__device__ __forceinline__ void tmem_ld_wait32(float* v) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]),
                 "+f"(v[6]), "+f"(v[7]), "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]),
                 "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]), "+f"(v[16]), "+f"(v[17]),
                 "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]), "+f"(v[23]),
                 "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28])
               :
               : "memory");
  asm volatile("" : "+f"(v[29]), "+f"(v[30]), "+f"(v[31])::"memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// D[tmem] (+)= A[tmem] * B[smem]: A is K-major in tensor memory (two 16-bit
// elements per column), B MN-major: 128-byte rows of 64 elements (128-byte swizzle), 8-row
// groups along K 1024 bytes apart, the groups of 64 along N kHalfBytes apart (the leading
// offset, bits 16..29 of the low word).
__device__ __forceinline__ void umma_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo,
                                        uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 bd;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "mov.b64 bd, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], bd, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "r"(b_lo), "r"(idesc), "r"(accumulate), "r"(kDescHi)
      : "memory");
}
__device__ __forceinline__ uint32_t mn_desc_lo(uint32_t saddr) {
  return ((saddr & 0x3FFFF) >> 4) | ((kHalfBytes >> 4) << 16);
}

// (a0, a1) * (b, b) + (c, c)
__device__ __forceinline__ void fma2_bc(float& d0, float& d1, float a0, float a1, float b, float c) {
  asm("{\n\t.reg .b64 pa, pb, pc;\n\t"
      "mov.b64 pa, {%2, %3};\n\tmov.b64 pb, {%4, %4};\n\tmov.b64 pc, {%5, %5};\n\t"
      "fma.rn.f32x2 pa, pa, pb, pc;\n\tmov.b64 {%0, %1}, pa;\n\t}"
      : "=f"(d0), "=f"(d1)
      : "f"(a0), "f"(a1), "f"(b), "f"(c));
}
// (a0, a1) * (b0, b1) + (c0, c1)
__device__ __forceinline__ void fma2_to(float& d0, float& d1, float a0, float a1, float b0,
                                        float b1, float c0, float c1) {
  asm("{\n\t.reg .b64 pa, pb, pc;\n\t"
      "mov.b64 pa, {%2, %3};\n\tmov.b64 pb, {%4, %5};\n\tmov.b64 pc, {%6, %7};\n\t"
      "fma.rn.f32x2 pa, pa, pb, pc;\n\tmov.b64 {%0, %1}, pa;\n\t}"
      : "=f"(d0), "=f"(d1)
      : "f"(a0), "f"(a1), "f"(b0), "f"(b1), "f"(c0), "f"(c1));
}
__device__ __forceinline__ void add2(float& d0, float& d1, float a0, float a1) {
  asm("{\n\t.reg .b64 pa, pd;\n\tmov.b64 pd, {%0, %1};\n\tmov.b64 pa, {%2, %3};\n\t"
      "add.rn.f32x2 pd, pd, pa;\n\tmov.b64 {%0, %1}, pd;\n\t}"
      : "+f"(d0), "+f"(d1)
      : "f"(a0), "f"(a1));
}

// D[tmem] (+)= A[smem] * B[smem]^T over 32 8-bit elements, K-major tiles of codes.
// (kind::f8f6f4 takes a type for each operand: these bits make A or B, made as E4M3, an E5M2.)
constexpr uint32_t kAIsE5M2 = 1u << 7, kBIsE5M2 = 1u << 10;
template <int D>
__device__ __forceinline__ void umma_codes(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo,
                                           uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 ad, bd;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "mov.b64 ad, {%1, %5};\n\tmov.b64 bd, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], ad, bd, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(accumulate), "r"(kCodeDescHi<D>)
      : "memory");
}

template <int N>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
// Named barrier among `count` threads that tells them whether any had `x` set.
__device__ __forceinline__ bool named_bar_any(int id, int count, bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred a, b;\n\tsetp.ne.u32 a, %3, 0;\n\t"
      "barrier.cta.red.or.pred b, %1, %2, a;\n\tselp.u32 %0, 1, 0, b;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(count), "r"(x ? 1u : 0u)
      : "memory");
  return r != 0;
}
// One lane of a converged warp, the same one each time.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}
__device__ __forceinline__ void fence_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// The cache rows [rows, D] in boxes of up to 128 positions: bf16 in boxes of 64
// channels (128 bytes), codes in whole rows (D bytes).
inline bool cache_map(CUtensorMap* m, const void* base, int D, bool fp8, uint64_t rows,
               uint32_t box_rows) {
  auto fn = encode_fn();
  if (fn == nullptr) return false;
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(D), rows};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(D) * (fp8 ? 1 : 2)};
  cuuint32_t box[2] = {fp8 ? static_cast<cuuint32_t>(D) : 64u, box_rows};
  cuuint32_t estr[2] = {1, 1};
  return fn(m, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
            const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            fp8 && D == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The maps of a cache's keys and values.
inline bool cache_maps(const AttnParams& p, int D, bool fp8, CUtensorMap* k, CUtensorMap* v) {
  std::memset(k, 0, sizeof(*k));
  std::memset(v, 0, sizeof(*v));
  const uint64_t rows = (static_cast<uint64_t>(p.c.num_pages) * p.c.heads) << p.c.page_log2;
  const uint32_t box = 1u << p.c.page_log2 < 128u ? 1u << p.c.page_log2 : 128u;
  return cache_map(k, p.c.k, D, fp8, rows, box) && cache_map(v, p.c.v, D, fp8, rows, box);
}

__device__ __forceinline__ uint16_t cvt_e5m2x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Eight bf16 elements x (four words), times a power of two that brings the row's largest into
// [2^7, 2^8), as the sums of an E4M3 and an E5M2 term: hi = E4M3(x), lo = E5M2(x - hi).  From
// 2^-6 on hi leaves at most 8 units of x's last place, which an E5M2 holds exactly, and below
// it at most 2^-10, rounded by at most 2^-14: exact for elements within 2^-13 of the row's
// largest, to 2^-21 of it below.  (An E4M3 lo ends at 2^-9 and loses up to 2^-17.)  An
// infinity, which neither type has, becomes a NaN: x * 0 + x.
__device__ __forceinline__ void two_terms(const uint32_t (&x)[4], float mul, uint32_t (&hi)[2],
                                          uint32_t (&lo)[2]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    hi[i] = lo[i] = 0;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float x0 = __uint_as_float(x[2 * i + j] << 16) * mul;
      float x1 = __uint_as_float(x[2 * i + j] & 0xffff0000u) * mul;
      x0 = fmaf(x0, 0.0f, x0);
      x1 = fmaf(x1, 0.0f, x1);
      const uint16_t hc = cvt_e4m3x2(x0, x1);
      const float2 f = e4m3x2_to_f32(hc);
      const uint16_t lc = cvt_e5m2x2(x0 - f.x, x1 - f.y);
      hi[i] |= static_cast<uint32_t>(hc) << (16 * j);
      lo[i] |= static_cast<uint32_t>(lc) << (16 * j);
    }
  }
}

}  // namespace moe
