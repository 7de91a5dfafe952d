"""The ring of the adapter products, whose decoding groups take the stages in turn: the kernel's own walk and
wait (csrc/ring.cuh) against a model of the barriers in which loads land in any order."""
import os
import re
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "qlora_parameter_efficient_b200", "csrc")


@pytest.fixture(scope="module")
def model(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("ring") / "ring_model")
    subprocess.run([os.environ.get("CXX", "g++"), "-std=c++17", "-O2", "-o", exe, os.path.join(HERE, "ring_model.cpp")],
                   check=True)

    def run(groups, stages, quant, checked=True, n=37, seeds=400):
        r = subprocess.run([exe, *(str(int(v)) for v in (groups, stages, n, quant, checked, seeds))],
                           capture_output=True, text=True, timeout=120)
        return r.returncode, r.stdout.strip()
    return run


# the rings that occur: two groups up to rank 64 (4 to 6 stages), one above (3 to 6); and the fewest stages
@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("groups,stages", [(1, 1), (1, 3), (1, 4), (1, 6), (2, 2), (2, 3), (2, 4), (2, 5), (2, 6), (3, 3),
                                           (3, 4), (3, 5), (3, 6), (3, 7)])
def test_every_stage_is_read_after_its_load_and_before_its_release(model, groups, stages, quant):
    assert model(groups, stages, quant) == (0, "ok")


@pytest.mark.parametrize("n", [1, 2, 3, 4, 5, 6, 7, 12, 13])
def test_short_contractions(model, n):
    for quant in (False, True):
        for stages in (4, 5, 6):
            assert model(2, stages, quant, n=n, seeds=100) == (0, "ok")


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("groups,stages", [(2, 3), (2, 5), (3, 4), (3, 5)])
def test_the_model_sees_what_a_wait_for_the_load_alone_lets_through(model, groups, stages, quant):
    """Where the stages are no multiple of the groups."""
    rc, out = model(groups, stages, quant, checked=False, seeds=2000)
    assert rc == 1 and "landed" in out, out


def test_the_kernel_waits_through_the_modelled_code():
    """Decoding groups reach a stage through ring_landed alone: no wait for full[] of their own."""
    src = open(os.path.join(CSRC, "act8.cuh")).read()
    body = src[src.index("k_act_gemm(const __grid_constant__"):]
    groups = body[body.index("RingPos at(S, group)"):body.index("join the ranks, write")]
    assert len(re.findall(r"mbar_wait_warp\(&full\[", groups)) == 1 and "ring_landed<L::kGroups>" in groups
    assert len(re.findall(r"ok = landed\(\);", groups)) == 3
