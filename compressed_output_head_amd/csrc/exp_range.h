// Exponents of the cross entropy's operands.  Plain C++, shared by the kernels
// and by a test that compiles it for the CPU.
#pragma once

namespace archead {

// An operand is 2^(z - E) in fp16, z = log2(e) times the scaled logit and E a
// whole number.  A row's largest operand is brought to 2^kExpTop or somewhat
// below it, and is never above 2^(kExpTop + 1): fp16 ends below 2^16.
constexpr int kExpTop = 14;

// E of a 32-row block whose largest z, rounded up to a whole number, is `top`:
// the row's exponent `ref` from the pieces before (-inf: none yet) where that
// leaves no operand above 2^(kExpTop + 1), else kExpTop below top.  The
// comparison is of the difference, whose rounding leaves it on its side of the
// border; ref + (kExpTop + 1) would be rounded from 2^24 on.  From 2^25 on
// top - kExpTop may be rounded down, and the largest operand would leave fp16:
// E is top then.  (z that large are 2 apart or equal, and operands of 1 and
// less have 24 powers of two below them.)  Of no z above -inf E is -inf or ref,
// of NaN or +inf it is that.
constexpr float exp_exponent(float top, float ref) {
  if (top - ref <= (float)(kExpTop + 1)) return ref;
  const float low = top - (float)kExpTop;
  return top - low > (float)(kExpTop + 1) ? top : low;
}

}  // namespace archead
