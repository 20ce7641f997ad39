// Whether a rotation is orthogonal, on the host: it decides before anything of a layer is written.
//
// max |U^T U - I| <= 1e-3. First in float32 on vector units, 4 x 16 sums at a time in registers: where no sum is within
// 1e-5 of the limit that decides it, since columns whose squares sum to about 1 leave less than 128 2^-24 = 7.7e-6 of
// error. Else, and where the matrix is to be refused, in double. 35 us a matrix on one core (in double alone, as plain loops:
// 0.6 ms).
#include <cmath>
#include <cstring>

namespace oscar {
namespace {

constexpr int kD = 128;
typedef float V4 __attribute__((vector_size(16)));

V4 load(const float* p) {
  V4 x;
  std::memcpy(&x, p, sizeof x);
  return x;
}

// |sum_r U[r][i0 + i] U[r][j0 + j] - I| <= limit for i < 4, j < 16
bool tile_near(const float* U, int i0, int j0, float limit) {
  struct Row {
    V4 a = {}, b = {}, c = {}, d = {};
    void add(float x, V4 p, V4 q, V4 r, V4 s) {
      a += x * p;
      b += x * q;
      c += x * r;
      d += x * s;
    }
    bool near(int diagonal, float limit) const {     // diagonal: where I's 1 is, 0 .. 15, or none
      float s[16];
      std::memcpy(s, &a, 16);
      std::memcpy(s + 4, &b, 16);
      std::memcpy(s + 8, &c, 16);
      std::memcpy(s + 12, &d, 16);
      bool ok = true;
      for (int j = 0; j < 16; ++j) ok = ok && std::fabs(s[j] - (j == diagonal ? 1.f : 0.f)) <= limit;   // false for NaN
      return ok;
    }
  };
  Row r0, r1, r2, r3;
  for (int r = 0; r < kD; ++r) {
    const float *x = U + r * kD + i0, *y = U + r * kD + j0;
    const V4 p = load(y), q = load(y + 4), s = load(y + 8), t = load(y + 12);
    r0.add(x[0], p, q, s, t);
    r1.add(x[1], p, q, s, t);
    r2.add(x[2], p, q, s, t);
    r3.add(x[3], p, q, s, t);
  }
  const int d = i0 - j0;
  return r0.near(d, limit) && r1.near(d + 1, limit) && r2.near(d + 2, limit) && r3.near(d + 3, limit);
}

}  // namespace

bool orthogonal(const float* U) {
  bool near = true;
  for (int i0 = 0; near && i0 < kD; i0 += 4)
    for (int j0 = i0 / 16 * 16; near && j0 < kD; j0 += 16) near = tile_near(U, i0, j0, 1e-3f - 1e-5f);
  if (near) return true;
  for (int i = 0; i < kD; ++i)
    for (int j = i; j < kD; ++j) {
      double s = 0.0;
      for (int r = 0; r < kD; ++r) s += (double)U[r * kD + i] * (double)U[r * kD + j];
      if (!(std::fabs(s - (i == j ? 1.0 : 0.0)) <= 1e-3)) return false;   // also NaN
    }
  return true;
}

}  // namespace oscar
