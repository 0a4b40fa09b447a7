// The quotient by which rows are quantised to 8-bit integers (reciprocal, product
// and two fma) against the division, next to every border between two codes:
// prints, for each exponent of the scale, the values tried, those whose code
// differs, and those that the product with the reciprocal alone gets wrong.
// Arguments: exponent and step of the 2^23 scales of that exponent, repeated.
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <thread>
#include <vector>

static inline float as_float(uint32_t u) {
  float f;
  memcpy(&f, &u, 4);
  return f;
}
static inline uint32_t as_bits(float f) {
  uint32_t u;
  memcpy(&u, &f, 4);
  return u;
}
// nearest whole number, ties to even, in the low byte
static inline uint32_t code(float q) { return as_bits(q + 12582912.0f) & 0xFF; }

static void scales(int exponent, uint32_t from, uint32_t to, uint32_t step, long* n, long* bad, long* plain) {
  long tried = 0, off = 0, raw = 0;
  for (uint32_t m = from; m < to; m += step) {
    const float c = as_float(((uint32_t)(127 + exponent) << 23) | m), r = 1.0f / c;
    int o = 0, w = 0;
    for (int b = 0; b < 127; ++b) {
      const uint32_t border = as_bits(((float)b + 0.5f) * c);
      for (int k = -2; k <= 2; ++k) {
        const float v = as_float(border + k), p = v * r;
        const float q = std::fmaf(-std::fmaf(p, c, -v), r, p);
        const uint32_t want = code(v / c);
        o += code(q) != want;
        w += code(p) != want;
      }
    }
    tried += 127 * 5;
    off += o;
    raw += w;
  }
  *n += tried;
  *bad += off;
  *plain += raw;
}

int main(int argc, char** argv) {
  const int threads = 8;
  for (int i = 1; i + 1 < argc; i += 2) {
    const int exponent = atoi(argv[i]);
    const uint32_t step = (uint32_t)atoi(argv[i + 1]), part = (1u << 23) / threads;
    std::vector<std::thread> pool;
    std::vector<long> n(threads), bad(threads), plain(threads);
    for (int t = 0; t < threads; ++t)
      pool.emplace_back([&, t] { scales(exponent, t * part, (t + 1) * part, step, &n[t], &bad[t], &plain[t]); });
    long a = 0, b = 0, c = 0;
    for (int t = 0; t < threads; ++t) {
      pool[t].join();
      a += n[t];
      b += bad[t];
      c += plain[t];
    }
    printf("%d %ld %ld %ld\n", exponent, a, b, c);
  }
  return 0;
}
