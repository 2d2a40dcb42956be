"""The norm's products to more than fp32 (csrc/two_floats.h): the same function on the
host, and what the compiler is allowed to do with it on the GPU."""
import re
import shutil
import subprocess

import numpy as np
import pytest

from top_routing_grouped_router_amd import build as B

pytestmark = pytest.mark.skipif(shutil.which(B.HIPCC) is None, reason="needs the HIP compiler")

HOST = r"""
#include <cstdio>
#include "two_floats.h"
int main() {
  float v[4];
  while (std::fread(v, 4, 4, stdin) == 4) {
    const float y = moe::scaled_odd(v[0], moe::Rstd{v[1], v[2]}, v[3]);
    std::fwrite(&y, 4, 1, stdout);
  }
}
"""
DEVICE = r"""
#include "two_floats.h"
__global__ void k(float* p) { p[0] = moe::scaled_odd(p[0], moe::Rstd{p[1], p[2]}, p[3]); }
"""


def _compile(tmp_path, text, *flags):
    src, out = str(tmp_path / "t.hip"), str(tmp_path / "t")
    with open(src, "w") as f:
        f.write(text)
    subprocess.run([B.HIPCC, *B.CFLAGS, *flags, src, "-o", out], check=True, capture_output=True)
    return out


def test_products_are_those_of_exact_arithmetic(tmp_path):
    """y = s (hi + lo) w lies within 2^-45 of what it is computed to, which is then
    rounded to odd: never across, or onto, a number of fewer bits"""
    exe = _compile(tmp_path, HOST, "--offload-host-only", "-Xarch_host", "-mfma")
    rng = np.random.default_rng(0)
    n = 200_000
    s, w = (rng.normal(size=n).astype(np.float32) for _ in range(2))
    rstd = 2.0 ** rng.uniform(-4, 4, size=n)
    hi = rstd.astype(np.float32)
    lo = (rstd - hi).astype(np.float32)
    # half of them put y within a rounding of a number of five bits
    tie = (16 + rng.integers(0, 16, size=n)) / 16
    w[::2] = (tie / (s * rstd)).astype(np.float32)[::2]
    res = subprocess.run([exe], input=np.stack([s, hi, lo, w], 1).tobytes(), check=True,
                         capture_output=True)
    got = np.frombuffer(res.stdout, np.float32)
    wide = np.longdouble
    y = wide(s) * (wide(hi) + wide(lo)) * wide(w)   # 64 bits: to 2^-62
    clear = np.abs(y / wide(got) - 1) > 2.0 ** -45
    assert clear.sum() > 0.9 * n
    # the odd rounding of y: the neighbour on y's side whose last bit is set
    down = y.astype(np.float32)
    down = np.where(np.abs(wide(down)) > np.abs(y), np.nextafter(down, np.float32(0)), down)
    bits = down.view(np.uint32)
    odd = np.where(bits & 1, bits, bits + 1).view(np.float32)
    bad = clear & (got != odd) & (wide(down) != y)
    assert not bad.any(), (int(bad.sum()), s[bad][:3], hi[bad][:3], lo[bad][:3], w[bad][:3])


def test_its_products_and_sums_stay_apart(tmp_path):
    """by default the compiler may join y = n w with the sums that follow (on the GPU it
    does, where it sees both), and what y's rounding lost would count twice"""
    with open(_compile(tmp_path, DEVICE, "--offload-device-only", "-S", "-emit-llvm")) as f:
        ops = re.findall(r"= f(?:mul|add|sub)\b.*", f.read())
    assert len(ops) == 5, ops          # two products, three sums
    assert not [op for op in ops if "contract" in op]
