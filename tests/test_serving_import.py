"""The package without the serving extension: the lookup is there, and a serving call says what is missing (no GPU)."""
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PACKAGE = os.path.join(ROOT, "hashed_gram_memory_amd")


def _run(code, path):
    return subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=120, cwd=path,
                          env=dict(os.environ, PYTHONPATH=str(path)))


@pytest.fixture(scope="module")
def without(tmp_path_factory):
    top = tmp_path_factory.mktemp("without")
    to = top / "hashed_gram_memory_amd"
    to.mkdir()
    for name in os.listdir(PACKAGE):
        if name.endswith(".py") or (name.endswith(".so") and name != "_serving.so"):
            shutil.copy(os.path.join(PACKAGE, name), to / name)
    return top


def test_the_lookup_does_without_the_extension(without):
    r = _run("import hashed_gram_memory_amd as hg; hg.lookup, hg.Plan, hg.lib(); print(hg.__file__)", without)
    assert r.returncode == 0, r.stderr
    assert r.stdout.strip().startswith(str(without))


@pytest.mark.parametrize("code", ["hg.paged_attention", "hg.serving", "from hashed_gram_memory_amd import kv_append"])
def test_a_serving_call_says_what_is_missing(without, code):
    r = _run(f"import hashed_gram_memory_amd as hg; {code}", without)
    assert r.returncode != 0 and "ImportError: _serving.so is not built" in r.stderr


def test_names_of_the_package():
    r = _run("""
import sys
import hashed_gram_memory_amd as hg
names = ("kv_append", "paged_attention", "paged_attention_workspace", "qk_norm_rope")
assert not any(n.endswith("_serving") for n in sys.modules)
assert {"serving", *names} <= set(dir(hg))
assert all(getattr(hg, n) is getattr(hg.serving, n) for n in names)
try:
    hg.no_such_name
except AttributeError:
    print("ok")
""", ROOT)
    assert r.stdout.strip() == "ok", r.stderr
