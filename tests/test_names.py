"""No test hides another: a module that defines a name twice runs only the last one."""

import ast
import collections
import glob
import os

HERE = os.path.dirname(os.path.abspath(__file__))
# hidden in their module, and run from another under a name of their own
MOVED = {("test_gpu_mxfp4.py", "test_quantize_every_16_bit_value"):
         ("test_gpu_mxfp4_values.py", "test_quantize_every_16_bit_value_below_a_larger_one")}


def _names(path):
    return collections.Counter(n.name for n in ast.parse(open(path).read()).body
                               if isinstance(n, (ast.FunctionDef, ast.ClassDef)))


def test_no_module_defines_a_name_twice():
    twice = {(os.path.basename(p), name) for p in glob.glob(os.path.join(HERE, "*.py"))
             for name, times in _names(p).items() if times > 1}
    assert twice <= set(MOVED), twice - set(MOVED)
    for module, name in MOVED.values():
        assert _names(os.path.join(HERE, module))[name] == 1
