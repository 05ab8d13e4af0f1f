"""Rules on the source text of the 8-bit kernels, checked without a GPU.

Waits are bounded.  A wait that runs out may do so for some lanes of a warp and not for
others; a warp whose lanes then went different ways would leave some of them at a
warp-wide barrier for ever.  So the outcome of every wait of a role is put to a vote."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "dense_fp32_gemm_05_gb300", "csrc")


def _code(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_every_role_wait_is_voted_on():
    for name in ("fp8_gemm.cu", "moe.cu"):
        text = _code(name)
        waits = list(re.finditer(r"mbar_wait_for\(", text))
        assert len(waits) >= 3
        for m in waits:
            # (the last waits of a role, for what it has under way: one lane's outcome is not used)
            call = text[m.start(): text.index(";", m.start())]
            if "kDrainNs" in call:
                continue
            begin = max(text.rfind(c, 0, m.start()) for c in ";{}")
            statement = text[begin + 1: text.index(";", m.start())]
            after = text[m.start(): m.start() + 400].split(";", 1)[1]
            voted = "__all_sync" in statement or re.match(r"\s*(if \(__any_sync|ok = __all_sync)", after)
            assert voted, f"{name}: {' '.join(statement.split())}"
