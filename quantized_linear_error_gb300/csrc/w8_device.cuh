// Device helpers shared by the kernels of the 8-bit integer linears.
#pragma once
#include <cuda_fp16.h>

#include "kv.h"
#include "w8.h"

namespace spear {

// Four codes (bytes of code + 128) as f16 pairs: bytes 0 and 2, then 1 and 3.
// A byte b under the exponent of 1024 reads as 1024 + b, so that subtracting
// 1152 leaves the code, exactly; which k a place stands for does not matter as
// long as both operands of a product take the same order.
SPEAR_DEVINL uint32_t f16x2_sub1152(uint32_t v) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(v), "r"(0x64806480u));
  return r;
}
SPEAR_DEVINL void w8_unpack(uint32_t w, uint32_t& even, uint32_t& odd) {
  uint32_t e, o;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(e) : "r"(w), "r"(0x00FF00FFu), "r"(0x64006400u));
  asm("prmt.b32 %0, %1, %2, 0x4341;" : "=r"(o) : "r"(w), "r"(0x64646464u));
  even = f16x2_sub1152(e);
  odd = f16x2_sub1152(o);
}
constexpr uint32_t kW8Bias = 0x80808080u;  // turns codes into bytes of code + 128

// act(g) = g / (1 + exp(-z)): z = g (SiLU), or z = 2 sqrt(2 / pi) (g + 0.044715 g^3), which is GELU's tanh form
// without the cancellation in 1 + tanh. With t = exp(-|z|) the quotient's divisor stays within 1 .. 2. 16-bit results take
// the fast quotient, off by two steps of fp32, and the fast exponential, off by 2^-16 of the value at most (an error of
// half a step of z log2(e), |z| < 104, and a few of its own): both below the result's rounding. kExact, for fp32 results:
// the quotient is corrected by its remainder (Markstein, IBM J. Res. Dev. 34, 1990), so that it rounds once; an infinite
// one has no remainder. 1088 tokens through 2 x 11008 x 4096 107 us, with the fast quotient 107, with the compiler's 123;
// 4096 x 1024 x 8192, which the epilogue bounds, 190, 162, 221.
template <bool kExact>
SPEAR_DEVINL float w8_act(float g, int act) {
  const float z = act == SPEAR_ACT_SILU ? g : 1.5957691216057308f * (g + 0.044715f * g * g * g);
  const float t = kExact ? expf(-fabsf(z)) : __expf(-fabsf(z));
  const float num = g * (z > 0.f ? 1.f : t);
  const float d = 1.f + t;
  if (!kExact) return __fdividef(num, d);
  float inv;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(d));
  const float q = num * inv;
  return fabsf(q) < INFINITY ? fmaf(fmaf(-q, d, num), inv, q) : q;
}

SPEAR_DEVINL void w8_store(void* y, int64_t at, int type, float v) {
  if (type == SPEAR_BF16) static_cast<__nv_bfloat16*>(y)[at] = __float2bfloat16_rn(v);
  else if (type == SPEAR_F16) static_cast<__half*>(y)[at] = __float2half_rn(v);
  else static_cast<float*>(y)[at] = v;
}

// Lets the next kernel be set up / waits for the work before this one: what the
// handle owns may be read in between.
SPEAR_DEVINL void grid_launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
SPEAR_DEVINL void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

}  // namespace spear
