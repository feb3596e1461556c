"""The tree operators together, as a decoding loop uses them: examples/tree_step.py generates the tokens of
one-by-one decoding in fewer target passes."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_trees_generate_the_tokens_of_one_by_one_decoding():
    spec = importlib.util.spec_from_file_location("tree_step", os.path.join(ROOT, "examples", "tree_step.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    steps, passes = example.main(R=3, steps=30)
    assert passes < steps
