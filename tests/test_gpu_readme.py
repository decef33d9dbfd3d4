"""README's Python examples: they run one after the other, and each is a use that
means what it says."""
import os
import re

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


def test_examples():
    names = {}
    blocks = re.findall(r"```python\n(.*?)```", open(README).read(), re.S)
    assert len(blocks) == 3
    for block in blocks:
        exec(compile(block, "README.md", "exec"), names)
        torch.cuda.synchronize()
    # a prefix is no part of the rows behind it, and none of the pages is in use twice
    prefix, pages = names["prefix"], names["pages"]
    ids = torch.cat([prefix.reshape(-1), pages.reshape(-1)])
    assert ids.unique().numel() == ids.numel()
    # positions go on behind the prompt, and every key was rotated: the first append to
    # the cache is a rotated one
    length = int(names["lengths"][0, 0])
    assert names["at"].unique().tolist() == [names["prompt"] + length - 1]
    assert "ibp_kv_append(" not in blocks[2]
    out = names["out"]
    assert out.shape == names["q"].shape and not out.isnan().any() and (names["chosen_lengths"] == 15 * 16 + length % 16).all()
