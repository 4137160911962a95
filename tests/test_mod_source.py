"""Properties of the modified-score kernel that no run shows, read from its source: what
happens once a bounded wait has run out, and orders of memory that the hardware
happens to keep."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "attention_forward_sm_gb300", "csrc")


def _source(name):
    """A source file without comments, white space as single blanks."""
    with open(os.path.join(CSRC, name)) as f:
        text = f.read()
    text = re.sub(r"//[^\n]*", " ", text)
    return re.sub(r"\s+", " ", text)


def test_every_warp_of_a_team_votes_after_a_wait_ran_out():
    """own_keys votes at named barriers that count all four warps of a team and have no
    time limit.  A warp whose wait ran out among the prefix items has to vote too."""
    src = _source("mod_sm103a.cuh")
    call = re.search(r"if constexpr \(swap\) (\{ )?(if \(\w+\) )?(\{ )?own_keys<[^;]*;", src)
    assert call is not None
    assert call.group(2) is None, "own_keys only for warps whose waits ended well"
    assert call.group(0).rstrip(";").rstrip(")").endswith(", fine")
    # and inside, the first vote comes before any way out
    body = src[src.index("void own_keys("):]
    assert "started = fine && " in body[:body.index("bar_any(")]
    assert not re.search(r"\breturn;", body[:body.index("bar_any(")])


def test_an_item_is_published_after_every_lane_s_stores():
    """All lanes of the planning warp write the rows' ranges, one arrives for the warp."""
    src = _source("mod_sm103a.cuh")
    body = src[src.index("bool work_publish("):]
    assert "__syncwarp();" in body[:body.index("mbar_arrive(&ms.work_full")]
