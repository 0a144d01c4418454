"""The warps that issue the tensor products run with all 32 lanes together (elect.sync and
__all_sync name every lane), so a wait that may give up has to give up on all lanes or on
none: warp_wait, which votes. Read from the kernels' source, since a lane that left alone
could hang a GPU."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bf16_forward_attention_gb300",
                    "csrc")


def _issuers(name):
    """The source of each MMA issuer: from its heading to the next role's."""
    text = open(os.path.join(CSRC, name)).read()
    parts = re.split(r"// -{20,} MMA issuer[^\n]*\n", text)[1:]
    return [re.split(r"\n *\} else ", p)[0] if "kPersist" not in p[:200] else re.split(r"V check \(warps", p)[0]
            for p in parts]


@pytest.mark.parametrize("name,count", [("attn_fwd_kernel.cuh", 1), ("attn_bwd_kernel.cuh", 2)])
def test_waits_that_may_give_up_are_voted(name, count):
    issuers = _issuers(name)
    assert len(issuers) == count
    for src in issuers:
        assert "mma_commit_warp" in src and "warp_wait" in src
        calls = re.findall(r"wait_bounded\(((?:[^()]|\((?:[^()]|\([^()]*\))*\))*)\)", src)
        assert calls, "the wait for the last products"
        for args in calls:
            # The last argument: whether another role's abort ends the wait. The only wait of its own for
            # each lane is the one for the last products, which goes on and is followed by a __syncwarp.
            assert args.split(",")[-1].strip() == "false" and "Drain" in args, args
