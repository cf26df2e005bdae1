// 16-bit element types of the serving kernels.  Part of attn_fwd.cu.

namespace {

enum ElemType { kBF16 = ATTN_BF16, kFP16 = ATTN_FP16, kFP32 = ATTN_FP32 };

__device__ __forceinline__ float bf16_lo(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t x) { return __uint_as_float(x & 0xffff0000u); }
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// What lies beyond fp16's range becomes its largest number (a NaN stays one).
__device__ __forceinline__ uint32_t pack_f16x2_sat(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float2 unpack_f16x2(uint32_t x) {
  float2 r;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "r"(x));
  return r;
}
template <int kType>
__device__ __forceinline__ float2 unpack_16x2(uint32_t x) {
  if constexpr (kType == kFP16) return unpack_f16x2(x);
  return make_float2(bf16_lo(x), bf16_hi(x));
}
template <int kType>
__device__ __forceinline__ uint32_t pack_16x2(float lo, float hi) {
  if constexpr (kType == kFP16) return pack_f16x2(lo, hi);
  return pack_bf16x2(lo, hi);
}

}  // namespace
