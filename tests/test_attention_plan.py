"""The launch shape of kvx_paged_attention over sizes of batches and workspaces (csrc/kvx_attention_plan.h, compiled for
the host): no GPU is needed."""
import os
import subprocess

import pytest

from block_table_contiguous_amd import build as B

SRC = os.path.join(os.path.dirname(os.path.abspath(__file__)), "c_abi", "attention_plan.cpp")
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    if not os.path.exists(os.path.join(ROCM, "include", "hip")):
        pytest.skip("the ROCm headers are not available")
    exe = str(tmp_path_factory.mktemp("plan") / "attention_plan")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-D__HIP_PLATFORM_AMD__", f"-I{B.INCLUDE}", f"-I{B.CSRC}",
                    f"-I{os.path.join(ROCM, 'include')}", SRC, "-o", exe], check=True)

    def run(rows):
        text = "".join(" ".join(str(x) for x in r) + "\n" for r in rows)
        out = subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout
        names = ("keys", "tiles", "planned", "shares", "busy", "slot")
        return [dict(zip(names, (int(x) for x in line.split()))) for line in out.splitlines()]
    return run


BATCHES = [(1, 1, 1, 131072, 32, 8, 128), (16, 16, 1, 8192, 32, 8, 128), (32, 32, 1, 8192, 32, 8, 128),
           (70, 70, 1, 8192, 32, 8, 128), (72, 72, 1, 8192, 32, 8, 128), (300, 300, 1, 4096, 8, 1, 128),
           (8, 4000, 517, 9216, 8, 1, 128), (1, 100, 100, 60000, 4, 1, 256), (3, 12, 4, 9000, 8, 2, 64)]


@pytest.mark.parametrize("batch", BATCHES, ids=str)
def test_a_small_workspace_is_no_worse_than_none(plans, batch):
    """The whole plan where it fits; fewer shares only where those are still more workgroups than the launch without any
    has tiles for; and the parts of what is launched always fit."""
    full = plans([(*batch, -1)])[0]
    assert full["shares"] == full["planned"]
    slots = full["planned"] + full["tiles"]
    sizes = [n for n in range(1, slots + 3)]
    for n, p in zip(sizes, plans([(*batch, -1 - n) for n in sizes])):
        assert p["shares"] in (0, p["planned"]) or p["busy"] < p["shares"] < p["planned"], (n, p)
        assert p["shares"] == 0 or p["shares"] + p["tiles"] <= n, (n, p)
        if n >= slots:
            assert p["shares"] == p["planned"]
    assert plans([(*batch, 0)])[0]["shares"] == 0


def test_one_long_request_is_split_as_far_as_the_workspace_goes(plans):
    batch = (1, 1, 1, 131072, 32, 8, 128)
    tiles = plans([(*batch, -1)])[0]["tiles"]
    assert [p["shares"] for p in plans([(*batch, -1 - tiles - k) for k in (1, 2, 5, 63, 64, 65)])] == [0, 2, 5, 63, 64, 64]


def test_the_grid_stays_within_what_a_launch_can_have(plans):
    """A tile is a workgroup of 256 threads for every KV head, and a launch has fewer than 2^32 threads, however long the
    requests are that the hint calls short."""
    top = (1 << 31) - 65537
    for heads, kv, reqs in ((4, 2, 1), (1, 1, 1), (8, 8, 100), (64, 64, 65535), (32, 1, 65535)):
        for rows in (1 << 29, 1 << 30, top - 128 * kv * reqs):
            for hint in (0, 1, 2, 1 << 40):
                p = plans([(reqs, rows // heads, hint, 64, heads, kv, 8, -1)])[0]
                assert 0 < p["tiles"] * kv < 1 << 24, (heads, kv, reqs, rows, hint, p)
    p = plans([(65535, 65535, 1, 8192, 64, 64, 128, -1)])[0]  # the largest true batch of single tokens keeps its kind
    assert p["keys"] == 1
