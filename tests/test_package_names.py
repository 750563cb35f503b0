"""The package's public names, with and without torch.  CPU only."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def python(code):
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return r.stdout


def test_star_import_without_torch():
    # the C-level binding needs no torch
    out = python("import sys; sys.modules['torch'] = None\n"
                 "from gated_delta_rule_32_gb300 import *\n"
                 "print(kda_chunk_fwd.__name__, kda_cache_attn.__name__, 'page_plan' in dir())")
    assert out.split() == ["kda_chunk_fwd", "kda_cache_attn", "False"]


def test_star_import_with_torch():
    out = python("from gated_delta_rule_32_gb300 import *\n"
                 "print(forward.__name__, page_plan.__name__, cache_attend.__name__, PagePlan.__name__)")
    assert out.split() == ["forward", "page_plan", "cache_attend", "PagePlan"]


def test_names_are_listed_and_found():
    out = python("import gated_delta_rule_32_gb300 as p\n"
                 "print([n for n in p.__all__ if not hasattr(p, n)], 'page_release' in p.__all__)")
    assert out.split() == ["[]", "True"]
