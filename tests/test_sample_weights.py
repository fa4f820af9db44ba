"""The sampler's weights, whose source stands for itself: compiled for the host, against long double."""
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SHIMS = r"""
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstring>
#define __device__
#define __forceinline__ inline
using u64 = unsigned long long;
struct float2 { float x, y; };
static inline float __fadd_rn(float a, float b) { return a + b; }
static inline float __fsub_rn(float a, float b) { return a - b; }
static inline float __fmul_rn(float a, float b) { return a * b; }
static inline float __fmaf_rn(float a, float b, float c) { return std::fma(a, b, c); }
static inline uint32_t __float_as_uint(float f) { uint32_t u; std::memcpy(&u, &f, 4); return u; }
"""

MAIN = r"""
int main() {
  uint64_t state = 88172645463325252ull;
  auto rnd = [&] {
    state ^= state << 13, state ^= state >> 7, state ^= state << 17;
    return (state >> 11) * 0x1p-53;
  };
  const float temps[] = {1.0f, 0.7f, 1.3f, 0.05f, 30.0f};
  for (int down = 0; down <= 6; ++down)       // vocabularies up to 2^18, then one bit less for every doubling up to 2^24
    for (int i = 0; i < 400000; ++i) {
      const float T = temps[i % 5], m = static_cast<float>((rnd() - 0.5) * 60.0);
      const double cd = 1.4426950408889634 / static_cast<double>(T);
      const float ch = static_cast<float>(cd), cl = static_cast<float>(cd - static_cast<double>(ch));
      float x = static_cast<float>(m - (FROM + (TO - FROM) * rnd()) / cd);   // so many octaves from the largest
      if (x > m) x = m;
      if (TO > 1e3 && i % 3 == 1) x = i % 2 ? -INFINITY : -3.402823466e38f;
      const long double w = std::exp((static_cast<long double>(x) - m) / T) * std::ldexp(1.0L, 44 - down);
      const u64 got = weight_inline(x, m, ch, cl, down, &kPowers);
      const long double off = std::fabs(static_cast<long double>(got) - w);
      if (!(off <= w * 0x1p-37L + 1.0L)) {
        std::printf("x %a m %a T %a down %d: %llu, not %Lg\n", x, m, T, down, got, w);
        return 1;
      }
    }
  return 0;
}
"""


@pytest.mark.parametrize("octaves", [(0.0, 6.0), (0.0, 50.0), (44.0, 60.0), (55.0, 63.0), (60.0, 2000.0)])
def test_weights_against_long_double(tmp_path, octaves):
    """For every vocabulary's unit, from the largest logit to distances whose weight is nothing, each shift a defined one. With
    |r| <= 1/128, so t <= 0.00542, in parts of the weight: the low part of t left out of its square 2^-38.7 (1.76 * 2^-32 t);
    roundings of t^2, of its factor and of their sum 2^-41 each, of the two products with 2^(-k/64) 2^-40 each at most; the
    series' next term 2^-44; of the distance 2^-41 at 45 octaves: together less than 1.7 * 2^-38. Table and weight are
    rounded to a unit once each: half a unit each."""
    cc = shutil.which("g++") or shutil.which("c++")
    if cc is None:
        pytest.skip("no C++ compiler")
    with open(os.path.join(ROOT, "selected_kv_sparse_gb300", "csrc", "k_sample.cu")) as f:
        source = f.read()
    part = re.search(r"^struct Powers \{.*?^// Out of line:", source, re.M | re.S)
    assert part
    src, exe = tmp_path / "weights.cpp", tmp_path / "weights"
    src.write_text(f"{SHIMS}\nconst double FROM = {octaves[0]}, TO = {octaves[1]};\n{part.group(0)}\n{MAIN}")
    subprocess.run([cc, "-std=c++17", "-O1", "-ffp-contract=off", "-fsanitize=undefined", "-fsanitize-undefined-trap-on-error",
                    str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, (r.returncode, r.stdout)
