"""The calls that the README shows are calls that the binding takes."""
import ast
import inspect
import os
import re

import pytest

from io_aware_exact_02_gb300 import fa

README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


def shown_calls():
    text = open(README, encoding="utf-8").read()
    for block in re.findall(r"^```python\n(.*?)^```", text, re.S | re.M):
        for node in ast.walk(ast.parse(block)):
            if (isinstance(node, ast.Call) and isinstance(node.func, ast.Attribute)
                    and isinstance(node.func.value, ast.Name) and node.func.value.id == "fa"):
                yield pytest.param(node, id=node.func.attr)


@pytest.mark.parametrize("call", list(shown_calls()))
def test_a_shown_call_has_the_arguments_of_its_function(call):
    assert not any(isinstance(a, ast.Starred) for a in call.args)
    assert all(k.arg for k in call.keywords)
    inspect.signature(getattr(fa, call.func.attr)).bind(
        *call.args, **{k.arg: k.value for k in call.keywords})


def test_the_readme_shows_calls():
    assert len(list(shown_calls())) >= 10
