"""The 8-bit product's choice of kernel, tile and division, compiled for the host: the shapes that are
compared bit for bit on the GPU reach every one that any size leads to."""
import os
import shutil
import subprocess

import pytest

from bit_post_quantized_amd import build
from tests.test_gpu_decoder_linear8_plans import SHAPES

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no g++")
    exe = str(tmp_path_factory.mktemp("plan") / "plans")
    res = subprocess.run([gxx, "-std=c++17", "-O2", f"-I{build.CSRC}", os.path.join(HERE, "w8a8_plan_main.cpp"), "-o", exe],
                         capture_output=True, text=True)
    assert res.returncode == 0, res.stderr[-3000:]

    def run(*args, text=""):
        res = subprocess.run([exe, *args], input=text, capture_output=True, text=True, timeout=120)
        assert res.returncode == 0, res.stderr[-3000:]
        return res.stdout.splitlines()

    return run


def test_every_choice_has_a_shape(plans):
    reached = set(plans(text="\n".join("%d %d %d" % s for s in SHAPES)))
    chosen = dict(line.split(" : ") for line in plans("all"))
    assert len(chosen) > 20
    missing = {kind: size for kind, size in chosen.items() if kind not in reached}
    assert not missing, missing
