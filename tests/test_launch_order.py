"""Which kernels of the training step's ends are launched ahead of their predecessor's end, by their
sources: kernels whose CTAs fill an SM go early only with at most a CTA of 256 threads per SM."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "attention_gemms_gb300",
                    "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def kernels(text):
    """name -> (text between __global__ and the parameters, body)."""
    found = {}
    for m in re.finditer(r"__global__ void([^;{]*?)\b(\w+_kernel)\(", text):
        start = text.index("{", m.end())
        depth, i = 1, start + 1
        while depth:
            depth += {"{": 1, "}": -1}.get(text[i], 0)
            i += 1
        found[m.group(2)] = (m.group(1), text[start:i])
    return found


FILES = ["vocab_linear.cu", "vocab_embed.cu"]
# a row of the lookup for some threads, no shared memory: launched early like the other row kernels
ROWS = {"vocab_embed_scaled_fwd_kernel"}
# behind the token sort, whose CTAs are all placed when they let it start
BEHIND = {"vocab_embed_sum_kernel"}


@pytest.mark.parametrize("name", FILES)
def test_only_small_grids_go_early(name):
    text = source(name)
    found = kernels(text)
    assert found
    plain = set(re.findall(r"\b(\w+_kernel)(?:<[\w:, ]+>)?<<<", text))
    for k, (_, body) in found.items():
        if k in ROWS:
            continue
        if k in plain:  # neither side overlaps
            assert "pdl_trigger" not in body and "pdl_wait" not in body, k
        else:  # what lets the next kernel start is decided by the host
            assert body.count("pdl_wait();") == body.count("pdl_trigger();") == 1, k
            assert re.search(r"if \((early|ahead)\) pdl_trigger\(\);", body), k
    # every launch that may overlap asks the rule
    early = re.findall(r"launch_kernel_if\(\s*(\w+),", text)
    assert early and set(early) == {"early"}
    rest = re.findall(r"launch_kernel\(\s*([\w]+)", text)
    assert set(rest) <= ROWS | BEHIND, rest
    asked = len(re.findall(r"const bool (?:early|ahead) = may_go_early\(", text))
    assert asked == len(early) + sum(k in BEHIND for k in rest)


def test_the_rule():
    text = source("internal.h")
    assert re.search(r"may_go_early\(int64_t ctas, int threads, int sms\) \{ "
                     r"return threads <= 256 && ctas <= sms; \}", text)
    for name in FILES:  # the device's SMs, not a number
        for args in re.findall(r"may_go_early\((.*?)\);", source(name)):
            assert args.endswith("device_sm_count()"), args
