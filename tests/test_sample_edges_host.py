"""Sampled decoding where it can go wrong, without a GPU."""
import os
import re
import shutil
import subprocess

import pytest

from tests.conftest import ROOT

CSRC = os.path.join(ROOT, "speculative_decode_gated_gdn_gb300", "csrc")


def read(name):
    return open(os.path.join(CSRC, name)).read()


def test_a_warp_writes_each_shared_result_at_one_place():
    """What every warp leaves for the whole CTA, which reads all of it behind the next barrier: an array written at a second
    place before another barrier can be read half old, half new.  (The largest logit of a slice's first granules and that of
    the whole slice are such results.)"""
    body = read("sample.cu").split("sample_kernel(const SampleParams p) {")[1].split("cudaError_t launch(")[0]
    written = [n for line in re.findall(r"if \(lane == 0\) (s\.\w+\[warp\] = [^;]*;)", body) for n in re.findall(r"s\.(\w+)\[warp\] =", line)]
    assert {"warp_top", "warp_low", "warp_bound"} <= set(written)
    assert len(written) == len(set(written)), written


# ---- the weights' arithmetic: the header's own text, compiled for the host ---------------------------------------
SHIMS = r"""
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstring>
#define __device__
#define __forceinline__ inline
#define __noinline__
using std::isinf;
static float __uint_as_float(uint32_t x) { float f; memcpy(&f, &x, 4); return f; }
static uint32_t __float_as_uint(float f) { uint32_t x; memcpy(&x, &f, 4); return x; }
static float bf2f(uint16_t x) { return __uint_as_float(uint32_t(x) << 16); }
static float __fdiv_rn(float a, float b) { return a / b; }
static float __fdividef(float a, float b) { return a / b; }
static float __ull2float_rn(unsigned long long x) { return float(x); }
static long long __float2ll_rn(float x) { return llrintf(x); }
static unsigned long long __umul64hi(unsigned long long a, unsigned long long b) { return (unsigned __int128)a * b >> 64; }
static uint32_t max(uint32_t a, uint32_t b) { return a > b ? a : b; }
"""

WORST = r"""
// Of weight_of over differences of bf16 numbers and temperatures: how far it is beyond half a unit, as a share of itself.
static double worst = 0;
static void look(int place, int top, float temperature) {
  const double x = (double(value_at(place)) - double(value_at(top))) / double(temperature);
  if (x < -31) return;
  const double want = std::exp(x);
  const double off = std::fabs(double(weight_of(place, top, scale_of(temperature), kExp2Table)) * 0x1p-43 - want) - 0x1p-44;
  worst = std::max(worst, off / want);
}
static int place_near(float x) {
  uint32_t b = __float_as_uint(x) >> 16;
  return place_of(b);
}
int main() {
  uint64_t state = 1;
  auto uniform = [&] { return double((state = state * 6364136223846793005ull + 1442695040888963407ull) >> 11) * 0x1p-53; };
  look(place_near(0.f), place_near(1.f), 0.7505670189857483f);
  look(place_near(1.5f), place_near(2.f), 1.842948f);
  for (int i = 0; i < 400000; ++i) {  // |r| up to 1/64 in steps of 2^-24, at every part of the table
    const float t = float(exp(2 * uniform() - 1)), d[4] = {0.5f, 1.f, 3.f, 17.f};
    for (float x : d) look(place_near(-x), place_near(0.f), t);
  }
  for (int i = 0; i < 2000000; ++i) {
    const float a = float((uniform() - 0.3) * exp(8 * uniform() - 4)), t = float(exp(8 * uniform() - 4));
    const float b = float(a - 25 * t * uniform());
    const int p = place_near(a), q = place_near(b);
    if (p < q) look(q, p, t);
  }
  EXTRA
  printf("%.4f\n", std::log2(worst + 1e-300));
}
"""


def run_on_host(tmp_path, extra=""):
    text = read("sample.cuh").split("// ---- a value's place in the order")[1].split("// ---- a row in memory")[0]
    src = tmp_path / "weights.cc"
    src.write_text(SHIMS + "//" + text + WORST.replace("EXTRA", extra))
    exe = str(tmp_path / "weights")
    subprocess.run(["g++", "-std=c++17", "-O2", "-ffp-contract=off", str(src), "-o", exe], check=True)
    return float(subprocess.run([exe], check=True, capture_output=True, text=True).stdout)


@pytest.mark.skipif(not shutil.which("g++"), reason="needs g++")
def test_weights_to_half_a_unit_and_their_38th_bit(tmp_path):
    """weight_of's and scale_of's own text, run on the host over 3.6 million weights: beyond the rounding to units of 2^-43, off by
    2^-38 of themselves at most.  By parts: the scale 2^-46 of itself, so of the exponent, up to 46, 2^-40 ln 2 of the weight; the exponent's
    low part, under 2^-18, two or three roundings to 2^-43; the series' terms from the cube on, under 2^-22, a few roundings to 2^-45, the
    first two with their remainders; what the series leaves out 2^-48: 2^-39.5 in all."""
    assert run_on_host(tmp_path) < -38


@pytest.mark.skipif(not shutil.which("g++"), reason="needs g++")
@pytest.mark.parametrize("lo,hi", [(-103, -87), (-90, -40), (40, 75), (70, 88.7)])
def test_weights_at_every_temperature(tmp_path, lo, hi):
    """The same for temperatures from the least positive number to the largest, with logits some temperatures apart."""
    assert run_on_host(tmp_path, f"""
  worst = 0;
  int seen = 0;
  for (int i = 0; i < 1000000; ++i) {{
    const float t = float(exp({lo} + ({hi} - {lo}) * uniform()));
    const double a = (uniform() - 0.5) * 60 * t, b = a - 25 * t * uniform();
    const int p = place_near(float(std::max(-3.3e38, std::min(3.3e38, a)))), q = place_near(float(std::max(-3.3e38, b)));
    if (t > 0 && p < q) look(q, p, t), ++seen;
  }}
  if (seen < 10000) return 1;""") < -38
