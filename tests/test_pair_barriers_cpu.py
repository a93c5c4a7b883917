"""Scopes of the pair kernel's barriers, read from its source: a barrier that the
other CTA of a pair arrives at, copies to or commits to is named, arrived at and
waited for at cluster scope.  (At the CTA's scope, the default, the order
between the CTAs is not one the memory model gives, whatever a run shows.)"""
import os
import re

from nvfp4_quantization_precision_gb300 import build as fos_build


def _text(name):
    with open(os.path.join(fos_build.CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_remote_arrivals_name_the_cluster():
    for name in sorted(os.listdir(fos_build.CSRC)):
        for ins in re.findall(r"mbarrier\.arrive[\w.:]*", _text(name)):
            if "shared::cluster" in ins:
                assert re.match(r"mbarrier\.arrive\.(release|relaxed)\.cluster\.", ins), (name, ins)


def test_waits_for_the_other_cta_are_at_cluster_scope():
    text = _text("fos_linear_pair.cuh")
    # barriers signalled across the pair: bytes of both CTAs' copies, commits to
    # both, arrivals mapped to CTA 0
    remote = {"full", "empty", "acc_full", "acc_empty", "sf_ready", "sf_free", "done"}
    seen = set()
    for kind, scope, bar in re.findall(r"(warp_wait|mbar_ask)(?:<Sync::(\w+)>)?\(&sh\.(\w+)", text):
        if bar in remote:
            seen.add(bar)
            assert scope in ("CLUSTER", "TENSOR"), (kind, bar, scope)
        # copies into shared memory are not ordered by the tensor memory's fences
        if bar == "full":
            assert scope == "CLUSTER", (kind, bar, scope)
    assert seen == remote
