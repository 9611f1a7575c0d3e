// The fit behind the gated pairs' gelu (w8_common.h), plain numbers so that a program on
// the host can hold it against the function.
#pragma once

namespace awq {

// Φ(-x) / exp(-x²/2) = erfcx(x / √2) / 2 for x >= 0 is smooth and falls as 1 / x: t·Q(t)
// with t = 1 / (1 + kPhiT·x). Q is the polynomial of degree 7 of least relative error over
// x from 0 to 13.3, where exp(-x²/2) leaves the normal numbers, by reweighted least squares
// (Lawson), its coefficients rounded to float32 one after the other with the others fitted
// again: 1.23e-7 as it stands here, 1.22e-7 before the roundings. Highest power first.
constexpr float kPhiT = 0.3f;
constexpr float kPhi[8] = {0.0360376909f, -0.158718452f, 0.208971232f, -0.0561003983f,
                           0.129844934f,  0.0995228738f, 0.120816886f, 0.119625174f};

}  // namespace awq
