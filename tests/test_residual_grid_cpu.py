"""The grids of the norms around a block, read from their source: no device here has another number of SMs to show
that they follow it."""
import os
import re

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "routing_grouped_gemm_gb300",
                   "csrc", "residual.cu")


def test_persistent_grids_follow_the_device():
    """A number of SMs may bound the workspace's parts; a grid takes the device's own."""
    text = re.sub(r"//[^\n]*", "", open(SRC).read())
    lines = [ln.strip() for ln in text.splitlines() if re.search(r"\b(152|148|160)\b", ln)]
    assert all(ln.startswith("constexpr int kMaxParts") for ln in lines), lines
    assert re.search(r"g\.ctas = .*sm_count\(\)", text)
