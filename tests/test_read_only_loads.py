"""The decoder-side kernels start while the kernel before them still runs, so what that one may write (tokens, scales,
weights quantised on the way) is not read-only while they live: no read-only loads (__ldg, or const __restrict__, from
which the compiler makes them) of anything but the bias."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "audio_encoder_aut_b200", "csrc")
FILES = ["aut_int8.cu", "aut_headnorm.cu", "aut_cross.cu", "aut_cross_tc.cu", "aut_cross.h", "aut_elem.cuh"]


def _code(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)


def test_no_read_only_loads_of_what_another_kernel_writes():
    for name in FILES:
        code = _code(name)
        assert "__ldg" not in code and "ld.global.nc" not in code, name
        for qualified in re.findall(r"const\s+[\w:]+\s*\*\s*__restrict__\s*(\w+)", code):
            assert qualified == "bias", (name, qualified)


def test_no_read_only_loads_of_the_8_bit_scales():
    for line in _code("aut_gemm.cuh").splitlines():
        assert not ("__ldg" in line and ("_scale" in line or "(wp" in line)), line
