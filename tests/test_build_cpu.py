"""What the library needs to be built and loaded: the C ABI stands without torch's headers and without the Python extension,
which only the calls that go through it need."""
import os
import subprocess
import sys

import pytest

from paged_kv_cache_298_gb300 import binding

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(autouse=True, scope="module")
def _built():
    binding.load_native()


def python(code, **env):
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300, cwd=ROOT,
                       env={**os.environ, "PYTHONPATH": ROOT, **env})
    assert r.returncode == 0, r.stdout[-1000:] + r.stderr[-3000:]
    return r.stdout


def test_calls_of_the_library_need_no_extension():
    """With no extension there and no compiler to make one, the calls that marshal through ctypes work; a call that needs it
    says what is missing."""
    python('''
from paged_kv_cache_298_gb300 import binding, build
binding._EXT_PATH = build.EXT = "/nonexistent/_dap_torch.so"
assert binding.status_string(0) == "ok" and binding.chunk_tokens(1000, 3) >= 334
assert binding.SharedPlan([3], 8, 2, 64, "cpu").num_tiles == 1
try:
    binding.kv_read_paged_fp8(*[None] * 7, total_tokens=1)
except RuntimeError as e:
    assert "_dap_torch" in str(e) and not isinstance(e, binding.DapError), e
else:
    raise AssertionError("no error")
assert binding.status_string(0) == "ok"
''', CXX="/bin/false")


def test_the_library_builds_without_torch():
    """(Built already here: what is checked is that neither looking whether it is up to date nor building it imports torch.)"""
    python('''
import importlib.util, sys
sys.modules["torch"] = None
spec = importlib.util.spec_from_file_location("b", "paged_kv_cache_298_gb300/build.py")
b = importlib.util.module_from_spec(spec)
spec.loader.exec_module(b)
assert b.up_to_date()
assert b.build() == b.LIB
''', CXX="/bin/false")


def test_an_extension_for_another_torch_is_refused(tmp_path):
    """The extension reads torch's tensors by their layout in memory.  One made for another torch or Python, that cannot be made
    anew, is not loaded, even where its symbols would resolve."""
    record = tmp_path / "for"
    record.write_text("torch 0.0 at /nowhere, Python 0")
    python(f'''
from paged_kv_cache_298_gb300 import binding, build
build.EXT_FOR = {str(record)!r}
for allowed in (True, False):
    try:
        binding.load_native(build_if_missing=allowed)
    except RuntimeError as e:
        assert "another torch or Python" in str(e), e
    else:
        raise AssertionError("loaded")
assert binding._ext is None
''', CXX="/bin/false")
    assert record.read_text().startswith("torch 0.0")
