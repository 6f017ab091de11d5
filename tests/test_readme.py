"""The calls that README.md shows fit the functions that they name."""
import ast
import inspect
import os
import re

import sparse_selection_primitive_amd as L

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def calls():
    with open(os.path.join(ROOT, "README.md")) as f:
        blocks = re.findall(r"```python\n(.*?)```", f.read(), re.S)
    for block in blocks:
        for node in ast.walk(ast.parse(block)):
            if isinstance(node, ast.Call) and isinstance(node.func, ast.Attribute) and \
                    isinstance(node.func.value, ast.Name) and node.func.value.id == "L":
                yield node


def test_calls_bind():
    seen = set()
    for node in calls():
        f = getattr(L, node.func.attr)
        inspect.signature(f).bind(*[None] * len(node.args), **{k.arg: None for k in node.keywords})
        seen.add(node.func.attr)
    assert seen >= {"route", "dispatch_plan", "dispatch", "combine", "cache_attend", "cache_evict"}


def test_arguments_are_in_their_places():
    """A variable that is named as a parameter of the function is given to that parameter."""
    for node in calls():
        names = list(inspect.signature(getattr(L, node.func.attr)).parameters)
        for at, arg in enumerate(node.args):
            name = arg.id if isinstance(arg, ast.Name) else None
            name = {"w": "weights"}.get(name, name)
            if name in names:
                assert names.index(name) == at, (node.func.attr, name)
