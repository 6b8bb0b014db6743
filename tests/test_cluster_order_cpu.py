"""How kernels order what threads of one CTA of a cluster write before what another
reads: read from the sources, as no run could show a missing order for certain."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mla_decode_attention_05_gb300", "csrc")


def _code():
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))):
        with open(path) as f:
            yield os.path.basename(path), re.sub(r"//[^\n]*", "", f.read())


def test_releases_to_another_cta_have_the_clusters_scope():
    """A release at the scope of the CTA does not order anything for a thread outside it."""
    found = 0
    for name, text in _code():
        for m in re.finditer(r"mbarrier\.arrive[\w.:]*shared::cluster[\w.:]*", text):
            found += 1
            assert ".cta" not in m.group(0), f"{name}: {m.group(0)}"
            assert ".release.cluster" in m.group(0) or ".relaxed.cluster" in m.group(0), f"{name}: {m.group(0)}"
    assert found >= 2


def test_widened_keys_of_both_ctas_are_waited_for_at_the_clusters_scope():
    text = dict(_code())["attention_mass.cu"]
    body = text[text.index("void wait_role("):text.index("void mma_role(")]
    assert re.search(r"warp_wait<kPoll, C::fp8 && !kStreamKeys>\(&br, &br\.res_full", body)
    assert re.search(r"warp_wait<kPoll, C::fp8 && kStreamKeys>\(&br, &br\.slot_full", body)
    widen = text[text.index("void widen_role("):text.index("void forward_role(")]
    assert "mapa" not in widen and "remote" not in widen   # the other CTA hears of it from one warp without writes of its own
    assert "mbar_arrive_remote(" in text[text.index("void forward_role("):text.index("void wait_role(")]
