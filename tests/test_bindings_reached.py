"""Every marshalling function has a caller: a second, unused path to an entry
point would not notice a swapped argument."""
import ast
import glob
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PACKAGE = os.path.join(ROOT, "decoder_greedy_decode_b200")


#: a name for callers that forwards to dec_init_int8, which is tested
FORWARDS = {"dec_init_fp8w"}


def functions(path):
    return [n.name for n in ast.parse(open(path).read()).body if isinstance(n, (ast.FunctionDef, ast.ClassDef))]


def names(path):
    """Attributes and imported names that a file mentions."""
    out = set()
    for n in ast.walk(ast.parse(open(path).read())):
        if isinstance(n, ast.Attribute):
            v = n.value       # (lib().name is the library's own function)
            of = getattr(v, "func", v)
            if getattr(of, "id", getattr(of, "attr", "")) not in ("lib", "L"):
                out.add(n.attr)
        if isinstance(n, ast.Name):
            out.add(n.id)
        if isinstance(n, ast.ImportFrom):
            out.update(a.name for a in n.names)
    return out


@pytest.mark.parametrize("module", ["capi", "tensors"])
def test_every_function_has_a_caller(module):
    path = os.path.join(PACKAGE, module + ".py")
    files = glob.glob(os.path.join(PACKAGE, "*.py")) + glob.glob(os.path.join(ROOT, "tests", "*.py")) + \
        [os.path.join(ROOT, f) for f in ("bench.py", "__graft_entry__.py")]
    used = set().union(*(names(f) for f in files if os.path.abspath(f) != os.path.abspath(path)))
    own = names(path)     # (helpers of the module itself)
    assert [f for f in functions(path) if f not in used | own | FORWARDS] == []
