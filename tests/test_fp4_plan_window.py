"""The launch shape of kvx_paged_attention_fp4 where rows see a window (csrc/kvx_fp4_plan.h, compiled for the host): no GPU
is needed."""
import os
import subprocess

import pytest

from block_table_contiguous_amd import build as B

SRC = os.path.join(os.path.dirname(os.path.abspath(__file__)), "c_abi", "fp4_plan_window.cpp")
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")
NONE = 0x7fffffff  # what the call takes for no window


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    if not os.path.exists(os.path.join(ROCM, "include", "hip")):
        pytest.skip("the ROCm headers are not available")
    exe = str(tmp_path_factory.mktemp("plan") / "fp4_plan_window")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-D__HIP_PLATFORM_AMD__", f"-I{B.INCLUDE}", f"-I{B.CSRC}",
                    f"-I{os.path.join(ROCM, 'include')}", SRC, "-o", exe], check=True)

    def run(rows):
        text = "".join(" ".join(str(x) for x in r) + "\n" for r in rows)
        out = subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout
        names = ("rows", "tiles", "shares", "bytes", "planned")
        return [dict(zip(names, (int(x) for x in line.split()))) for line in out.splitlines()]
    return run


@pytest.mark.parametrize("batch,shares", [((40, 40, 1, 5000, 32, 8, 128), 96), ((13, 52, 4, 5003, 28, 4, 96), 128),
                                          ((2, 400, 200, 5000, 32, 8, 128), 64)], ids=str)
def test_windows_of_few_slots_are_not_shared_out(plans, batch, shares):
    """Rows that see at most 896 slots, by the window as by the context; whichever is smaller counts."""
    got = [p["shares"] for p in plans([(*batch, w) for w in (1, 16, 896, 897, 4999, 5003, NONE)])]
    assert got == [0, 0, 0, shares, shares, shares, shares]
    short = (*batch[:3], 896, *batch[4:])
    assert [p["shares"] for p in plans([(*short, w) for w in (800, 1000, NONE)])] == [0, 0, 0]


def test_large_tiles_that_fill_the_gpu_are_shared_out_only_without_a_window_that_cuts(plans):
    """The contexts of 576 tiles are nearly alike, and all tiles of a request as long, unless a window cuts them."""
    batch = (1, 2304, 2304, 32768, 32, 8, 128)
    got = plans([(*batch, w) for w in (897, 32767, 32768, 40000, NONE)])
    assert [p["rows"] for p in got] == [128] * 5 and [p["tiles"] * 8 for p in got] == [584] * 5
    assert [p["shares"] for p in got] == [0, 0, 64, 64, 64]
    # too few to fill it: shared out whatever the window cuts
    assert [p["shares"] for p in plans([(1, 100, 100, 32768, 32, 8, 128, w) for w in (897, 4096, NONE)])] == [64] * 3


def test_the_workspace_planned_without_a_window_is_enough_with_any(plans):
    """kvx_paged_attention_fp4_workspace knows no window: what a window makes of the plan must fit in its bytes, and a window
    changes no tile."""
    sizes = [(reqs, reqs * query, query, context, heads, kv, dim) for reqs in (1, 3, 32, 300) for query in (1, 4, 13, 200, 2304)
             for context in (100, 900, 5000, 131072) for heads, kv, dim in ((32, 8, 128), (8, 1, 64), (28, 4, 256), (64, 64, 32))]
    windows = (1, 128, 896, 897, 4096, 32768, 131071, NONE)
    got = plans([(*s, w) for s in sizes for w in windows])
    shared = 0
    for i, s in enumerate(sizes):
        of = got[i * len(windows):(i + 1) * len(windows)]
        assert len({(p["rows"], p["tiles"], p["planned"]) for p in of}) == 1, s
        for w, p in zip(windows, of):
            assert p["shares"] in (0, of[-1]["shares"]) and p["bytes"] <= p["planned"], (s, w, p)
            shared += p["shares"] > 0
    assert shared > 100
