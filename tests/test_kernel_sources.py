"""Rules on the kernels' own sources that no launch can show."""

import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "routed_expert_ffn_gemm_gb300", "csrc")
SOURCES = sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh")))


def text_of(name):
    with open(os.path.join(CSRC, name)) as f:
        return f.read()


@pytest.mark.parametrize("name", ["block_gemm.cu", "block_gemm_many.cu", "wgrad.cu"])
def test_copying_warp_waits_for_the_last_arrivals(name):
    # The MMAs' commits arrive on a slot's barrier by themselves, at any time
    # up to (and across the pair, after) the sums' own: the CTA whose barrier
    # it is has to see the last one of each slot before it may leave.  So the
    # copying warp waits for its slots once in the loop and once after it.
    text = text_of(name)
    role = text[text.index("- copies\n"):text.index("MOE_ERR_DEVICE_TIMEOUT", text.index("- copies\n"))]
    loop, wait = role.index("for (int u = u_first"), r"mbar_wait_bounded\(\s*empty_bar\("
    after = role[role.rindex("\n      }\n", loop):]  # behind the loop over the units
    assert len(re.findall(wait, role)) == 2 and len(re.findall(wait, after)) == 1


def test_cluster_has_started_before_its_memory_is_written():
    # distributed shared memory may be accessed once every CTA of the cluster
    # runs: the sum over the router's parts needs a cluster barrier in front of
    # its store to CTA 0
    text = text_of("router_losses.cu")
    kernel = text[text.index("    router_losses_sum_kernel("):]
    before = kernel[: kernel.index("st.shared::cluster")]
    assert "cluster_sync();" in before or before.index("cluster_arrive();") < before.index("cluster_wait();")


def statements(path):
    """The instructions of each asm statement of a source file."""
    with open(path) as f:
        text = f.read()
    for body in re.findall(r"\basm(?:\s+volatile)?\s*\((.*?)\);", text, re.S):
        yield "".join(re.findall(r'"((?:[^"\\]|\\.)*)"', body))


def test_copies_are_found():
    assert SOURCES and any("cp.async.bulk.tensor" in s for p in SOURCES for s in statements(p))


@pytest.mark.parametrize("path", SOURCES, ids=[os.path.basename(p) for p in SOURCES])
def test_no_copy_is_multicast(path):
    # the library is also loaded by replicas on several GPUs
    assert not [s for s in statements(path) if "cp.async.bulk" in s and "multicast" in s]


def test_wait_limit_grows_with_the_work():
    # the waits' limit counts from a launch's start: a constant one would end
    # a product that takes longer than it (600 000 rows of 65 536 x 65 536: 2.2
    # seconds, 122 GB)
    text = text_of("train_api.cu")
    limits = re.findall(r"wait_limit_ns\((.*?)\)", text)
    assert len(limits) >= 3 and all("R" in a and "N" in a and "K" in a and "E" in a for a in limits)
