"""The rule that chooses the form of the CTA-pair GEMM, compiled for the host:
the sizes of the tests of each form reach that form, and its edges."""
import ctypes
import os
import subprocess

import pytest

import pair_forms

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SHIM = """
#include "pair_plan.h"
extern "C" int plan(int T, int in, int out, const int* resident, int* bn, int* pairs) {
    const paro::PairPlan p = paro::plan_pairs((out / 16 + 15) / 16, T, in / 128,
                                              [&](int, int k) { return resident[k - 1]; });
    *bn = p.bn;
    *pairs = p.pairs;
    return p.form;
}
"""
# clusters of one to four pairs at once on 148 SMs: every SM in use, and fewer
# where a cluster has to lie in one part of the chip
RESIDENT = [(74, 37, 24, 18), (74, 36, 22, 14), (70, 32, 20, 12)]


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    (d / "plan.cpp").write_text(SHIM)
    lib = str(d / "plan.so")
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-I", os.path.join(ROOT, "rotated_w4_linear_b200", "csrc"),
                    str(d / "plan.cpp"), "-o", lib], check=True)
    f = ctypes.CDLL(lib).plan

    def call(T, n_in, n_out, resident=RESIDENT[0]):
        bn, pairs = ctypes.c_int(), ctypes.c_int()
        form = f(T, n_in, n_out, (ctypes.c_int * 4)(*resident), ctypes.byref(bn), ctypes.byref(pairs))
        return form, bn.value, pairs.value
    return call


@pytest.mark.parametrize("resident", RESIDENT)
def test_the_tests_of_each_form_reach_it(plan, resident):
    for size in pair_forms.SPLIT:
        form, bn, pairs = plan(*size, resident)
        assert form == (64 if size[0] <= 64 else 128) == bn, size
    assert {plan(*size, resident)[2] > 1 for size in pair_forms.SPLIT} == {False, True}     # one pair, and several
    for size in pair_forms.WHOLE:
        form, bn, pairs = plan(*size, resident)
        assert form == 256 and pairs == 1, size
    widths = {plan(*size, resident)[1] for size in pair_forms.WHOLE}
    assert 256 in widths and min(widths) < 256              # whole tiles and smaller ones of equal size


@pytest.mark.parametrize("resident", RESIDENT)
def test_plans_are_sound(plan, resident):
    for T in list(range(17, 140)) + [255, 256, 257, 333, 511, 512, 513, 8191, 8192, 100000]:
        for n_in, n_out in ((128, 16), (384, 272), (4096, 4096), (14336, 4096), (4096, 28672), (128, 65536)):
            form, bn, pairs = plan(T, n_in, n_out, resident)
            assert 1 <= pairs <= min(4, n_in // 128)
            if form == 256:
                assert T > 128 and pairs == 1 and bn % 32 == 0 and 32 <= bn <= 256
                assert -(-T // bn) == -(-T // 256)          # as few tiles as tiles of 256 would be
            else:
                assert bn == form == (64 if T <= 64 else 128)


def test_known_choices(plan):
    assert plan(256, 4096, 4096) == (128, 128, 2)
    assert plan(256, 4096, 28672) == (256, 256, 1)
    assert plan(333, 5120, 34832) == (256, 192, 1)
    assert plan(64, 14336, 4096)[0] == 64 and plan(64, 14336, 4096)[2] > 1
