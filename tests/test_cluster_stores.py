"""A CTA's shared memory may be written or read by the others of its cluster
only once it is known to have started: in every kernel that does so a cluster
barrier comes first.  Nothing goes wrong at run time as long as a cluster's CTAs
start together, so the kernels' sources are what is checked."""
import os
import re

import pytest

import sparse_mixture_experts_topk_gb300 as moe

CSRC = os.path.join(os.path.dirname(moe.__file__), "csrc")
ACCESS = re.compile(r"\b(st_peer|ld_peer|red_peer)\w*\(")
BARRIER = re.compile(r"\bcluster_(sync|wait)\(\)")

KERNELS = [("orthogonalize.cu", "small_kernel"), ("router_backward.cu", "balance_finish_kernel"),
           ("router.cu", "router_small_kernel"), ("router_tc.cu", "router_tc_kernel"),
           ("orthogonalize.cu", "chain_kernel"), ("ffn_tc2.cu", "grouped_gemm_pair_kernel")]


def kernel(name, function):
    """The text of a kernel: from its name to the first line that is a closing brace alone."""
    with open(os.path.join(CSRC, name)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    start = re.search(r"\b%s\(" % function, text).start()
    return text[start:text.index("\n}\n", start)]


@pytest.mark.parametrize("name,function", KERNELS)
def test_a_cluster_barrier_comes_before_the_first_access_to_another_cta(name, function):
    text = kernel(name, function)
    access, barrier = ACCESS.search(text), BARRIER.search(text)
    assert access and barrier and barrier.start() < access.start()
