"""Source check (no GPU needed): what an arrival on an mbarrier of another CTA hands over has to be
released at cluster scope; without a scope, or at CTA scope, the memory model orders nothing for a
thread of the other CTA. The arrival is a release itself, or it is relaxed and stands behind a fence
of its own: of shared memory at cluster scope, or of reads of TMEM."""
import glob
import os
import re

from conftest import ROOT

CSRC = os.path.join(ROOT, "post_weight_quantization_guided_b200", "csrc")
FENCES = ("fence.release.sync_restrict::shared::cta.cluster;", "tcgen05.fence::before_thread_sync;")


def test_arrivals_on_other_ctas_barriers_release_at_cluster_scope():
    found = 0
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))):
        for asm in re.findall(r"asm volatile\((.*?)\);\n", open(path).read(), re.S):
            # (a commit of tensor-core operations is no mbarrier.arrive)
            for op in re.finditer(r"(?<!\w)mbarrier\.arrive[\w.:]*", asm):
                if "shared::cluster" not in op.group():
                    continue
                found += 1
                relaxed = ".relaxed.cluster." in op.group() and any(f in asm[:op.start()] for f in FENCES)
                assert ".release.cluster." in op.group() or relaxed, (os.path.basename(path), asm)
    assert found, "no cluster product found"


def test_aligned_cluster_barriers_stand_behind_a_whole_warp():
    """The aligned form of the cluster barrier is undefined for part of a warp: nothing but the
    helper that first brings the warp together issues it."""
    found = 0
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))):
        text = open(path).read()
        for m in re.finditer(r"barrier\.cluster\.arrive[\w.]*\.aligned", text):
            found += 1
            before = text[:m.start()].rstrip().splitlines()
            statements = [line.strip() for line in before if not line.strip().startswith("//")]
            assert statements[-2] == "__syncwarp();", (os.path.basename(path), statements[-2:])
    assert found, "no cluster barrier found"
