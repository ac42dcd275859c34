// operand.cuh — operand helpers shared by the attention and cache kernels: MN-major
// descriptors, TMEM stores, loads as fp32 and e4m3 conversions.
#pragma once
#include "common.cuh"

namespace dsa {

// Shared-memory descriptor of an MN-major operand in 128-byte swizzled rows:
// each 128-byte row holds 64 consecutive MN elements of one K index, 8 rows form
// a 1024-byte atom (SBO = 1024 between K groups of 8), and MN blocks of 64
// elements lie `lbo` bytes apart.
__device__ __forceinline__ uint64_t make_sdesc_mn(uint32_t smem_addr, uint32_t lbo) {
  uint64_t d = 0;
  d |= (uint64_t)((smem_addr >> 4) & 0x3FFF);
  d |= (uint64_t)((lbo >> 4) & 0x3FFF) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, "
      "%28, %29, %30, %31, %32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]),
      "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
      "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ float load_as_f32(const void* x, int dtype, int64_t i) {
  if (dtype == DSA_F32) return reinterpret_cast<const float*>(x)[i];
  return __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(x)[i] << 16);
}

__device__ __forceinline__ uint8_t e4m3_rn_sat(float v) {
  return (uint8_t)__nv_cvt_float_to_fp8(v, __NV_SATFINITE, __NV_E4M3);
}

// Scale of a group of e4m3 codes from its largest magnitude: amax / 448, or 1 where that is 0:
// a group of zeros, or of values so small (amax < 2^-141) that the quotient rounds to 0, which
// as a scale would turn the group's zeros into NaN.
__device__ __forceinline__ float e4m3_scale(float amax) {
  const float a = __fdiv_rn(amax, 448.f);
  return a > 0.f ? a : 1.f;
}

__device__ __forceinline__ float e4m3_value(uint8_t c) {
  __half_raw h = __nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)c, __NV_E4M3);
  return __half2float(__half(h));
}

}  // namespace dsa
