"""The border of min_p where M + T log(min_p) is about 0: there 10^9 floats compare alike in 64 bits.

The comparison itself says what the border is: the least float x with ((double) x - M) c >= log2(min_p), c = log2(e) / T.
On the host the function is compiled by itself and its comparisons are counted; on the GPU rows of such settings take
the token and count that the same comparison gives."""
import os
import shutil
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LOG2E = 1.4426950408889634
# (M, T, min_p): e^-k of a maximum of k, powers of two at temperatures of whole octaves, what rounds to near 0
CANCEL = [(float(k), 1.0, float(np.exp(-k))) for k in (1, 2, 3, 8, 20)] + [
    (2.0, 1 / np.log(2.0), 0.25), (5.0, 5 / np.log(20.0), 0.05), (3.0, 1.3028834457097556, 0.1), (2.5, 1.0, float(np.float32(np.exp(-2.5)))),
    (1e30, 1e30, float(np.exp(-1.0))), (1e-30, 1.0, 1.0), (1e-30, 1e-6, float(np.exp(-1e-24))), (64.0, 1.0, float(np.exp(-64.0)))]
OTHERS = [(0.0, 1.0, 1.0), (0.0, 1.0, 0.3), (-3.0, 0.7, 0.05), (17.25, 1.0, 0.02), (3e38, 1.0, 0.5), (-3e38, 1e30, 1e-300), (3e38, 1e30, 1e-300),
          (5e-324, 1.0, 1.0), (0.0, 1e-6, 5e-324), (-0.0, 1.0, 1.0), (1e-45, 1e-6, 1.0), (100.0, 1e30, 0.999999), (0.5, 1e30, 1.0)]

PROGRAM = """
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#define __device__
static long compared = 0;
struct Slope { double v; };          // counts the comparisons that it takes part in
inline double operator*(double x, Slope s) {
  if (++compared > 1000) { std::printf("more than 1000 comparisons\\n"); std::exit(1); }
  return x * s.v;
}
inline double operator/(double x, Slope s) { return x / s.v; }
struct Scale { float m, bins; Slope c; };
struct Border { float x; int32_t i; };
constexpr double kLog2e = 1.4426950408889634;
%s
int main(int argc, char** argv) {
  for (int i = 1; i + 2 < argc; i += 3) {
    const Scale sc{static_cast<float>(std::atof(argv[i])), 0.f, {kLog2e / std::atof(argv[i + 1])}};
    compared = 0;
    const Border b = min_p_border(sc, std::atof(argv[i + 2]));
    std::printf("%%.9g %%ld\\n", b.x, compared);
  }
}
"""


@pytest.mark.skipif(not shutil.which("g++"), reason="g++ not installed")
def test_border_is_the_least_float_in_few_comparisons(tmp_path):
    src = open(os.path.join(ROOT, "second_order_optimizer_amd", "csrc", "sample.hip")).read()
    body = src[src.index("// The least float whose weight is at least m"):src.index("// A row's settings.")]
    cpp, exe = tmp_path / "border.cpp", tmp_path / "border"
    cpp.write_text(PROGRAM % body)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", str(cpp), "-o", str(exe)], check=True)
    rng = np.random.default_rng(0)
    cases = CANCEL + OTHERS + [(float(np.float32(rng.normal() * 10)), float(rng.choice([0.5, 1.0, 1.7])), float(rng.random())) for _ in range(200)]
    r = subprocess.run([str(exe)] + ["%r" % float(v) for c in cases for v in c], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout[-200:]
    lines = r.stdout.split("\n")
    for (m, t, p), line in zip(cases, lines):
        x, compared = np.float32(line.split()[0]), int(line.split()[1])
        top, c, z = np.float64(np.float32(m)), LOG2E / t, np.log(p) * LOG2E
        holds = lambda v: (np.float64(v) - top) * c >= z  # noqa: E731
        assert holds(x) and not holds(np.nextafter(x, np.float32(-np.inf))), (m, t, p, x)
        assert compared <= 36, (m, t, p, compared)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,vocab,k", [(5, 700, 0), (3, 5003, 0), (2, 70000, 40), (300, 9001, 30)])
def test_rows_whose_border_is_about_zero(gpu_lib, rows, vocab, k, dtype):
    """Columns on either side of 0, none nearer than 1e-3, in every kernel that takes min_p."""
    import torch
    from second_order_optimizer_amd import tokens
    from tests.test_gpu_objectives import DT, gpu, wide
    from tests.test_gpu_tokens import check
    rng = np.random.default_rng(vocab)
    for m, t, p in CANCEL[:9]:
        x = rng.choice([-1.0, 1.0], (rows, vocab)) * 10.0 ** rng.uniform(-3, 0, (rows, vocab))
        x = np.minimum(x, m)
        x[np.arange(rows), rng.integers(0, vocab, rows)] = m
        xg = gpu(x.astype(np.float32)).to(DT[dtype])
        u = gpu(rng.random(rows).astype(np.float32))
        op = tokens.Sampler(rows, vocab, dtype, temperature=t, top_k=k, min_p=p)
        check(op.run(xg, u), wide(xg), u, t, k, 1.0, p)
        own = op.run(xg, u, temperature=torch.full((rows,), t, device="cuda"), min_p=torch.full((rows,), p, device="cuda"))
        check(own, wide(xg), u, float(np.float32(t)), k, 1.0, float(np.float32(p)))
        assert op.flags() == 0
