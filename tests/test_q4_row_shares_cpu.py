"""The shares that the 4-bit prefill's row kernel cuts a token into
(csrc/q4_plan.h), on the CPU through a small driver built with g++.

A CTA's warps serve (token, share) pairs and step by gridDim * (warps / shares)
tokens: with more shares than warps that step is 0 and a warp would never reach
its end, so the rule gives a number that divides the warps, or 0 (the geometry
takes the transform kernel and a quantiser after it)."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "gqa_attention_preallocated_qa_gb300", "csrc")


@pytest.fixture(scope="module")
def shares(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not available")
    exe = str(tmp_path_factory.mktemp("rows") / "q4_rows_driver")
    subprocess.run([gxx, "-std=c++17", "-O1", "-I", CSRC, os.path.join(HERE, "native", "q4_rows_driver.cpp"),
                    "-o", exe], check=True)

    def run(cases):
        text = "\n".join(" ".join(map(str, c)) for c in cases) + "\n"
        out = subprocess.run([exe], input=text, capture_output=True, text=True, check=True, timeout=60)
        return [[int(x) for x in line.split()] for line in out.stdout.splitlines()]
    return run


def test_every_geometry_gets_shares_that_its_warps_can_walk(shares):
    heads = sorted(set(range(1, 130)) | set(range(128, 1025, 8)) | {2048, 4096, 8192})
    cases = [(hkv * g, hkv, d, t, 152) for hkv in heads for g in (1, 2, 4, 8) for d in (64, 128)
             for t in (1, 17, 300, 5000, 1 << 26) if hkv * g <= 65535]
    for case, (parts, warps, smem, most) in zip(cases, shares(cases)):
        if parts == 0:
            continue
        hq, hkv = case[:2]
        assert warps % parts == 0, case           # a stride of at least one token
        assert hkv % parts == 0 and hq % parts == 0, case
        assert smem <= most, case


@pytest.mark.parametrize("hq,hkv,d", [(160, 160, 128), (256, 128, 128), (512, 64, 128), (512, 512, 64)])
def test_tokens_too_wide_for_any_share_are_left_to_the_other_form(shares, hq, hkv, d):
    assert [line[0] for line in shares([(hq, hkv, d, t, 152) for t in (1, 1000, 1 << 40)])] == [0, 0, 0]


def test_shares_of_ordinary_geometries(shares):
    # (32, 8, 128): two fit, four while every share has a warp; (24, 3, 128): a
    # stage of 7680 bytes against 6400, and three kv heads cannot be halved
    got = shares([(32, 8, 128, 300, 152), (32, 8, 128, 5000, 152), (24, 3, 128, 300, 152), (8, 2, 128, 300, 152)])
    assert [line[0] for line in got] == [4, 2, 0, 2]
