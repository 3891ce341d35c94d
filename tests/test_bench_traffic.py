"""The DRAM-traffic records that bench.py reports belong to the sources of the layer's kernels as they are."""
import glob
import os
import re

import pytest

import bench

CSRC = os.path.join(bench.ROOT, "block_scaled_fp4_moe_gb300", "csrc")


@pytest.mark.parametrize("workload,kernel", [("glm_t1", "fused_layer_kernel"), ("glm_verify_t16", "ffn_tc_gateup"), ("glm_t1", "mx8_gemm_gateup"),
                                             ("glm_zipf_t64", "ffn_tc_gateup")])
def test_every_roofline_kernel_has_a_record_of_its_sources(workload, kernel):
    assert bench.recorded_traffic(workload, kernel), "the layer's CUDA sources changed: take the record in profiles/dram_traffic.txt again"


def test_sources_that_the_digest_leaves_out_hold_nothing_of_the_layer():
    names = {os.path.basename(p) for p in glob.glob(os.path.join(CSRC, "*"))}
    assert bench.ATTENTION_SOURCES <= names
    for name in names - bench.ATTENTION_SOURCES - {"binding.cpp"}:
        included = set(re.findall(r'#include "([^"]+)"', open(os.path.join(CSRC, name)).read()))
        assert not included & bench.ATTENTION_SOURCES, name
