"""Nothing stays in the sources of the operators for long contexts that no call reaches."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mla_decode_attention_05_gb300", "csrc")


def _read(*names):
    return "\n".join(re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, n)).read()) for n in names)


def test_fp8_helpers_are_called():
    text = _read(*sorted(n for n in os.listdir(CSRC) if n.endswith((".cu", ".cuh"))))
    for name in re.findall(r"__forceinline__ void (\w+)\(", _read("fp8.cuh")):
        assert len(re.findall(rf"\b{name}\(", text)) > 1, name


def test_parameters_are_read():
    """Each field of a kernel's parameters is used elsewhere than where it is set."""
    for struct, names in (("SharedParams", ("shared_prefix.cuh", "shared_prefix.cu", "shared_attention.cu")),
                          ("MassParams", ("attention_mass.cu",)), ("EvictParams", ("evict.cu",))):
        text = _read(*names)
        body = re.search(rf"struct {struct} \{{(.*?)\n\}};", text, re.S).group(1)
        fields = [f for line in body.split(";") for f in re.findall(r"(\w+)\s*(?=,|$)", re.sub(r"^[^*\w]*(?:const\s+)?(?:unsigned\s+)*(?:long\s+)*\w+", "", line.strip()))]
        assert len(fields) > 15, (struct, fields)
        for f in fields:
            assert len(re.findall(rf"\bp\.{f}\b(?!\s*=[^=])", text)) > 0, (struct, f)
