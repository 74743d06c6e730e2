"""Rules that the kernels' sources keep and no run can show (no GPU)."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "kda_chunked_prefill_gb300", "csrc")


@pytest.mark.parametrize("name", ["kda_delta_chunk.cu", "kda_scaled_matmul.cu"])
def test_a_role_that_gives_up_commits_by_the_lane_that_issued(name):
    """A commit tracks the products of its own thread. They are issued by the elected lane, which need not be lane 0: were the commit that a
    role drains by another lane's, it would be complete at once, with products still in flight."""
    text = open(os.path.join(CSRC, name), encoding="utf-8").read()
    commits = re.findall(r"^.*?commit\w*(?:<[^>]*>)?\(&m->drained.*$", text, flags=re.M)
    assert commits
    for line in commits:
        assert re.match(r"\s*if \(lin::elect_one\(\)\) ", line), line
    assert "lane == 0) {\n            umma_commit" not in text


def test_no_arrival_is_relaxed():
    """Who waits on a barrier may rely on what the arriving thread did before: no kernel hands anything over by an arrival without release."""
    for name in sorted(os.listdir(CSRC)):
        text = open(os.path.join(CSRC, name), encoding="utf-8").read()
        assert not re.search(r"mbarrier\.arrive[\w.:]*\.relaxed", text), name
