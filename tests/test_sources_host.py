"""Rules of the kernels' sources that no run shows."""
import os
import re

import pytest

from combine_quant_gb300 import build as cqbuild


def _source(name):
    with open(os.path.join(cqbuild.CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def _calls(text, name):
    """The arguments of each call of `name`."""
    for m in re.finditer(re.escape(name) + r"\(", text):
        depth, at = 1, m.end()
        while depth:
            depth += {"(": 1, ")": -1}.get(text[at], 0)
            at += 1
        yield text[m.end():at - 1]


@pytest.mark.parametrize("field", ["h", "h_scales", "x_scales", "x16"])
def test_the_layers_workspace_takes_no_read_only_loads(field):
    """The down kernel starts while the up kernel writes its results: a load that is defined only for data that nothing
    writes while the kernel lives must not name them."""
    text = _source("cq_moe_layer.cu")
    assert list(_calls(text, "__ldg")) and re.search(r"\ba\.%s\b" % field, text)
    assert not [c for c in _calls(text, "__ldg") if re.search(r"\ba\.%s\b" % field, c)]
    assert "ld.global.nc" not in text
