"""The attention kernels' wait for their softmax warps' votes (mla_wait.h), on
the host against a made-up clock: it ends, and a block that was off its SM for
longer than the limit does not give up on warps that are about to arrive (the
warps that had seen the vote would then wait at a barrier for those that had not)."""

import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "mla_query_projection_gb300", "csrc")


@pytest.fixture(scope="module")
def cases(tmp_path_factory):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no host compiler")
    exe = str(tmp_path_factory.mktemp("waits") / "wait_driver")
    subprocess.run([cxx, "-std=c++17", "-O1", "-I", CSRC, os.path.join(HERE, "wait_driver.cpp"), "-o", exe], check=True)
    out = subprocess.run([exe], check=True, capture_output=True, text=True, timeout=60).stdout
    return {n: (ok == "1", int(polls)) for n, ok, polls in (line.split() for line in out.splitlines())}


def test_the_wait_ends_when_all_have_come(cases):
    assert cases["at_once"] == (True, 1)
    assert cases["soon"][0]


@pytest.mark.parametrize("name", ["off_the_sm", "off_the_sm_at_first"])
def test_time_off_the_sm_is_no_reason_to_give_up(cases, name):
    assert cases[name][0]


@pytest.mark.parametrize("name", ["never", "never_and_off_the_sm"])
def test_the_wait_is_bounded(cases, name):
    ok, polls = cases[name]
    assert not ok and (1 << 20) < polls < 4_000_000


def test_every_vote_is_waited_for_this_way():
    for name in ("mla_attn_tc.cu", "mla_attn_ds.cu", "mla_attn_nv.cu"):
        with open(os.path.join(CSRC, name)) as f:
            text = f.read()
        assert text.count("tc_wait_votes(voted, ") == 1 and "tc_wait(voted" not in text, name
