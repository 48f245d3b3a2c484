"""Every module of the package says in its docstring what it is, from a first word on."""
import ast
import os

import pytest

PKG = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "lossless_bf16_compression_gb300")


@pytest.mark.parametrize("name", sorted(n for n in os.listdir(PKG) if n.endswith(".py")))
def test_a_module_says_what_it_is(name):
    doc = ast.get_docstring(ast.parse(open(os.path.join(PKG, name)).read()))
    assert doc and doc[0].isalnum()
