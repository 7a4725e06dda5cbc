"""What keeps the dense layer's kernels from hanging where a bounded wait runs out, read from their sources:
it must not be tried on a device."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "long_context_sparse_softmax_b200", "csrc")
MEET = ("__shfl_", "__any_sync", "__syncwarp", "tmem_ld", "named_bar")


def block(s, at):
    """The text of the braces that open at or behind `at`."""
    i = s.index("{", at)
    depth = 0
    for j in range(i, len(s)):
        depth += (s[j] == "{") - (s[j] == "}")
        if depth == 0:
            return s[i:j + 1]
    raise AssertionError("unbalanced")


def loops(name):
    """The outermost loops over steps, tiles or rows that wait on a barrier, without comments."""
    s = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
    s = s[s.index("__global__"):]
    out, end = [], 0
    for m in re.finditer(r"\bfor \((int|long)? ?\w+ =[^{;]*;[^{;]*;[^{;]*\) \{", s):
        if m.start() < end:
            continue
        body = block(s, m.end() - 1)
        end = m.end() + len(body)
        if re.search(r"\b(wait|wait_all|arrived)\(", body):
            out.append(body)
    return out


@pytest.mark.parametrize("name", ["k_norm.cu", "k_w4.cu", "k_kv8_attn.cu", "k_kv8_attn_tc.cu"])
def test_a_warp_leaves_a_loop_together(name):
    """In a loop whose lanes meet (shuffles, votes, warp-wide loads), a lane that gave up its wait must not
    leave alone: the others would wait for it in the next meeting.  So what a wait says is voted on before
    it ends the loop."""
    found = loops(name)
    assert found
    for body in found:
        if not any(w in body for w in MEET):
            continue
        for m in re.finditer(r"\b(wait|arrived)\(", body):
            # the statement that the wait is in
            begin = max(body.rfind(c, 0, m.start()) for c in ";{}") + 1
            stop = body.index(";", m.start())
            st = body[begin:stop]
            if "__all_sync(" in st:
                continue
            var = re.match(r"\s*(?:else )?(?:if \([^=]*\) )?(?:const bool |bool )?(\w+) = ", st)
            assert var, f"{name}: a lane's wait ends a loop by itself: {st.strip()}"
            vote = re.search(r"__all_sync\(0xffffffffu, %s\)" % var.group(1), body[stop:])
            assert vote, f"{name}: never voted on: {st.strip()}"
            assert not any(w in body[stop:stop + vote.start()] for w in MEET), f"{name}: the lanes meet before the vote"
