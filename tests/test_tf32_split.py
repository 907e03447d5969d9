"""The split of an FP32 value into two TF32 ones, from the kernel's source, compiled for the host."""
import os
import re
import shutil
import subprocess

import numpy as np
import pytest

SOURCE = os.path.join(os.path.dirname(__file__), "..", "bounded_memory_attention_b200", "csrc", "rma_gdn_prefill.cu")

PROGRAM = """
#include <cstdint>
#include <cstdio>
#include <cstring>
#define __device__
#define __forceinline__ inline
static uint32_t __float_as_uint(float x) { uint32_t u; memcpy(&u, &x, 4); return u; }
static float __uint_as_float(uint32_t u) { float x; memcpy(&x, &u, 4); return x; }
%s
int main() {
    uint32_t u;
    while (fread(&u, 4, 1, stdin) == 1) {
        const Tf t = tf_split(__uint_as_float(u));
        fwrite(&t.hi, 4, 1, stdout);
        fwrite(&t.lo, 4, 1, stdout);
    }
}
"""


@pytest.fixture(scope="module")
def split(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("needs g++")
    src = open(SOURCE).read()
    text = re.search(r"struct Tf \{.*?(?=__device__ __forceinline__ void mma_tf32)", src, re.S)[0]
    d = tmp_path_factory.mktemp("tf32")
    (d / "t.cpp").write_text(PROGRAM % text)
    subprocess.run(["g++", "-O1", "-ffp-contract=off", "-o", str(d / "t"), str(d / "t.cpp")], check=True)

    def run(bits):
        out = subprocess.run([str(d / "t")], input=np.asarray(bits, np.uint32).tobytes(), stdout=subprocess.PIPE, check=True).stdout
        hi, lo = np.frombuffer(out, np.uint32).reshape(-1, 2).T
        return hi, lo

    return run


def test_a_value_keeps_22_bits(split):
    """Both parts have 11 bits (the low 13 are 0); the sum is within 2^-23 of the value: the remainder of the rounding to
    11 bits is a multiple of 2^-23 of the value's binade below 2^-11, and losing its last bit costs one such step."""
    x = np.random.default_rng(1).standard_normal(200_000).astype(np.float32)
    x = np.concatenate((x, np.float32(2.0) ** np.arange(-60, 60, dtype=np.float32), np.float32([0.0, -0.0, 1.9999999, 0.99999994])))
    hi, lo = split(x.view(np.uint32))
    assert not ((hi | lo) & 0x1fff).any()
    total = hi.view(np.float32).astype(np.float64) + lo.view(np.float32)
    assert (np.abs(total - x) <= 2.0 ** -23 * 2.0 ** np.floor(np.log2(np.maximum(np.abs(x), 1e-30)))).all()


def test_a_value_that_is_not_finite_stays_so(split):
    """The NaN that FP32 arithmetic produces (all ones), others, and infinities: not both parts are finite."""
    hi, lo = split([0x7fffffff, 0xffffffff, 0x7fc00000, 0xffc00000, 0x7f800000, 0xff800000, 0x7fffe000])
    assert (~np.isfinite(hi.view(np.float32)) | ~np.isfinite(lo.view(np.float32))).all()
