"""The one wait of the paged decode step that lasts as long as a segment (a CTA's stay in a unit, up to 2^19
tiles of 128 keys), read from its source: the queries' warp, two segments ahead of the products."""
import os
import re

from alibi_attention_block_gb300.build import CSRC


def code(file):
    with open(os.path.join(CSRC, file), encoding="utf-8") as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_the_limit_grows_with_the_segment():
    text = code("attn_paged.cuh")
    calls = re.findall(r"mbar_wait\w*\(bar\.q_empty\(\w+\),[^;]*;", text)
    assert len(calls) == 1 and re.search(r"kWaitLimitNs \+ \w+(\[\w+\])? \* kTileLimitNs", calls[0]), calls
    limit = int(re.search(r"kTileLimitNs = (\d+)", text).group(1))
    # a tile of K and V, where every CTA's rate is its share of 5 TB/s (6.5 are measured): 16 bits, head_dim 128, two
    # CTAs on each of 152 SMs; head_dim 160, one
    for d, elem, ctas in ((128, 2, 2), (160, 2, 1), (160, 1, 2), (64, 2, 2), (64, 1, 4)):
        tile = 2 * 128 * d * elem * ctas * 152 / 5e12
        assert limit * 1e-9 >= 4 * tile
