// Integer quotients from an approximate reciprocal (constexpr, so that host code can test them).
#pragma once

namespace tq {

// ceil(x / d) for 0 < x <= 2^27, 1 <= d <= 2^27, r = 1 / d to within two steps of fp32 (v_rcp_f32 is within
// one). The first quotient is rounded to 24 bits: off by up to x / d 2^-22, a few tens. What it leaves is
// small enough to be divided the same way, which leaves less than a divisor to either side.
constexpr int ceil_div_by(int x, int d, float r) {
  const int u = x - 1;  // floor((x - 1) / d) + 1
  int y = static_cast<int>(static_cast<float>(u) * r);
  y += static_cast<int>(static_cast<float>(u - y * d) * r);
  const int rest = u - y * d;
  return y + 1 + (rest >= d ? 1 : 0) - (rest < 0 ? 1 : 0);
}

}  // namespace tq
