"""The README's examples call the library as it is: every call of the package in a Python block names a function that
exists, with arguments that it has (no GPU needed)."""
import ast
import inspect
import os
import re

import speculative_decoding_verification_53_gb300 as sv

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def calls():
    with open(os.path.join(ROOT, "README.md"), encoding="utf-8") as f:
        text = f.read()
    for block in re.findall(r"```python\n(.*?)```", text, re.S):
        for node in ast.walk(ast.parse(block)):
            f = getattr(node, "func", None)
            if isinstance(f, ast.Attribute) and isinstance(f.value, ast.Name) and f.value.id == "sv":
                yield f.attr, node


def test_examples_call_what_there_is():
    found = list(calls())
    assert {"spec_verify_chain", "spec_kv_append", "spec_page_resize", "spec_block_summary"} <= {name for name, _ in found}
    for name, node in found:
        assert all(k.arg for k in node.keywords) and not any(isinstance(a, ast.Starred) for a in node.args)
        inspect.signature(getattr(sv, name)).bind(*node.args, **{k.arg: k.value for k in node.keywords})
