"""The example of decoding with drafted trees, run whole."""
import importlib.util
import os

import pytest

from tests._gpu import say

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "tree_decode.py")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("tree_decode", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_tree_decode(example, cache):
    """Drafts are accepted, and the tokens are those that the sequences, run
    as prompts, would have chosen: all but those where rounding (another order
    of the same products) decides between two tokens, given as one in ten."""
    say(f"tree decode, {cache}")
    produced, turns, same = example.run(3, 40, 8, cache, log=say)
    assert produced >= 3 * 40
    assert produced > turns  # more than a token per request and step
    assert same >= 0.9 * produced


def test_one_node_trees_are_plain_decoding(example):
    say("tree decode, one node")
    produced, turns, same = example.run(2, 12, 1, "bf16", log=say)
    assert produced == turns == 24
    assert same >= 0.9 * produced
