"""A CTA of the FP8 streaming kernel whose wait gave up has no sums for its cluster to add: its flag
reaches every CTA of the cluster before any of them reads the others' sums. (No call makes a wait
run out, so this is read from the source.)"""
import os
import re

from helpers import ROOT


def test_the_flag_reaches_the_cluster_before_the_sums_are_read():
    text = open(os.path.join(ROOT, "w4a16_int4_mixture_align_b200", "csrc", "fp8_stream.cu")).read()
    end = text[text.rindex("if (ctas > 1) {"):]
    told = re.search(r"if \(abort_flag && int\(threadIdx\.x\) < ctas\) st_cluster_u32\(cluster_addr\(&abort_flag, threadIdx\.x\), 1", end)
    meet = end.index("cluster_sync_all()")
    assert told and told.start() < meet
    for use in re.finditer(r"ld_cluster4\(", end):
        assert "&& !abort_flag" in end[meet:use.start()]
