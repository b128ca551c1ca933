"""The launch shape of kvx_paged_attention_fp4 over sizes of batches and workspaces (csrc/kvx_fp4_plan.h, compiled for
the host): no GPU is needed."""
import os
import subprocess

import pytest

from block_table_contiguous_amd import build as B

SRC = os.path.join(os.path.dirname(os.path.abspath(__file__)), "c_abi", "fp4_plan.cpp")
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    if not os.path.exists(os.path.join(ROCM, "include", "hip")):
        pytest.skip("the ROCm headers are not available")
    exe = str(tmp_path_factory.mktemp("plan") / "fp4_plan")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-D__HIP_PLATFORM_AMD__", f"-I{B.INCLUDE}", f"-I{B.CSRC}",
                    f"-I{os.path.join(ROCM, 'include')}", SRC, "-o", exe], check=True)

    def run(rows):
        text = "".join(" ".join(str(x) for x in r) + "\n" for r in rows)
        out = subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout
        names = ("rows", "tiles", "planned", "shares", "busy", "slot")
        return [dict(zip(names, (int(x) for x in line.split()))) for line in out.splitlines()]
    return run


BATCHES = [(1, 1, 1, 131072, 32, 8, 128), (1, 2304, 2304, 32768, 32, 8, 128), (32, 9000, 517, 9216, 8, 1, 128), (16, 16, 1, 8192, 32, 8, 128), (32, 32, 1, 8192, 32, 8, 128),
           (72, 72, 1, 8192, 32, 8, 64), (300, 300, 1, 4096, 8, 1, 128), (8, 4000, 517, 9216, 8, 1, 128),
           (1, 100, 100, 60000, 4, 1, 256), (3, 12, 4, 9000, 8, 2, 64), (5, 20, 4, 9000, 56, 8, 256)]


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


@pytest.mark.parametrize("tokens,heads,kv,rows,wide", [(1, 16, 1, 16, 16), (1, 17, 1, 32, 32), (2, 16, 1, 32, 32), (8, 8, 1, 32, 32),
                                                       (5, 13, 1, 128, 32), (12, 8, 1, 128, 32), (97, 1, 1, 128, 128),
                                                       (1, 128, 8, 16, 16), (517, 8, 1, 128, 128)])
def test_rows_of_a_tile(plans, tokens, heads, kv, rows, wide):
    for dim, want in ((128, rows), (256, wide)):
        assert plans([(2, 2 * tokens, tokens, 5000, heads, kv, dim, -1)])[0]["rows"] == want


@pytest.mark.parametrize("reqs,query,context,shared", [(1, 2048, 32768, 0), (1, 2304, 32768, 64), (1, 4096, 32768, 0), (1, 2560, 32768, 64),
                                                       (3, 2048, 32768, 64), (1, 2304, 9000, 0), (4, 4096, 32768, 0)])
def test_shares_of_tiles_that_fill_the_gpu(plans, reqs, query, context, shared):
    assert plans([(reqs, reqs * query, query, context, 32, 8, 128, -1)])[0]["planned"] == shared


@pytest.mark.parametrize("context,shares", [(512, 0), (896, 0), (897, 96), (4096, 96)])
def test_few_slots_are_not_shared_out(plans, context, shares):
    assert plans([(40, 40, 1, context, 32, 8, 128, -1)])[0]["planned"] == shares


def test_the_grid_stays_within_what_a_launch_can_have(plans):
    """A tile is a workgroup of 256 threads for every KV head, and a launch has fewer than 2^32 threads, however long the
    requests are that the hint calls short."""
    top = (1 << 31) - 65537
    for heads, kv, reqs in ((4, 2, 1), (1, 1, 1), (8, 8, 100), (64, 64, 65535), (32, 1, 65535)):
        for rows in (1 << 24, 1 << 29, 1 << 30, top - 128 * kv * reqs):
            for hint in (0, 1, 2, 1 << 40):
                p = plans([(reqs, rows // heads, hint, 64, heads, kv, 32, -1)])[0]
                assert 0 < p["tiles"] * kv < 1 << 24, (heads, kv, reqs, rows, hint, p)
    p = plans([(65535, 65535, 1, 8192, 64, 64, 128, -1)])[0]  # the largest true batch of single tokens keeps its kind
    assert p["rows"] == 16
