"""attn_paged_rows: the warp that issues the tensor products runs with all 32 lanes together (elect.sync names
every lane), so a wait that may give up gives up on all of them or on none: warp_wait, which votes. Read from the
kernel's source, since a lane that left alone could hang a GPU."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bf16_forward_attention_gb300",
                    "csrc")


def _kernel():
    """The body of attn_paged_rows: from its signature to the brace at the start of a line."""
    text = open(os.path.join(CSRC, "attn_paged_kernel.cuh")).read()
    at = re.search(r"__global__ [^\n]*\battn_paged_rows\(const Params p\) \{\n", text)
    return text[at.end():text.index("\n}\n", at.end())]


def _calls(src, name):
    """(arguments, what follows) of every call of `name`."""
    return [(m.group(1), src[m.end():]) for m in
            re.finditer(r"\b" + name + r"\(((?:[^()]|\((?:[^()]|\([^()]*\))*\))*)\)", src)]


def test_waits_that_may_give_up_are_voted():
    src = _kernel()
    assert src.count("issue_rows_s(") == 1 and src.count("issue_rows_pv(") == 1
    # S, and P V before the next S and at an item's end; every one with the abort flag and the limit.
    voted = _calls(src, "warp_wait")
    assert [a.split(",")[0] for a, _ in voted] == ["bar_o", "bar_s", "bar_o"]
    assert all(a.split(",")[-2:] == [" abort_flag", " p.timeout_ns"] for a, _ in voted)
    # The one wait of its own for each lane is that for the last products: it goes on whatever other
    # warps gave up, and the lanes meet behind it before the memory is given back.
    alone = _calls(src, "wait_bounded")
    assert len(alone) == 1
    args, after = alone[0]
    assert args.split(",")[0] == "bar_end" and args.split(",")[-1].strip() == "false"
    assert after.lstrip("; \n").startswith("__syncwarp();")
    assert after.index("__syncthreads()") < after.index("tmem_dealloc")
    # No other form of a wait.
    assert not re.search(r"\bmbar_(try_)?wait|\bmbar_test", src)


def test_only_the_first_warp_issues():
    """Each product and commit stands in a block of `warp == 0`, which the whole warp takes or leaves."""
    src = _kernel()
    for name in ("issue_rows_s(", "issue_rows_pv(", "mma_commit_warp("):
        for m in re.finditer(re.escape(name), src):
            depth, i = 0, m.start()
            while i > 0:  # out of the enclosing braces, one after another
                i -= 1
                depth += {"}": 1, "{": -1}.get(src[i], 0)
                if depth == -1:
                    if re.search(r"if \(warp == 0\) $", src[:i]):
                        break
                    depth = 0
            assert i > 0, (name, src[m.start() - 80:m.start() + 40])
