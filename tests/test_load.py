"""What loading the library asks for: the host's parts and the calls bound with ctypes need no
torch and no C++ module, and the calls that do need them say so (no GPU needed)."""
import os
import subprocess
import sys

import paged_kv_cache_241_gb300 as pkv

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(pkv.__file__)))

# In a process of its own, in which a module cannot be imported.
WITHOUT = """
import sys
sys.modules[{module!r}] = None
"""
HOST = """
import paged_kv_cache_241_gb300 as pkv
m = pkv.BlockManager(8, 256)
assert m.allocate(1, list(range(300))) == 0 and m.allocate(2, list(range(300))) == 256
order, starts, shared = m.prefix_groups([1, 2])
assert starts.tolist() == [0, 2] and shared.tolist() == [1]
assert pkv.load().pkv_status_string(0) == b"PKV_OK"
"""


def run(code):
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    return r.stdout


def test_the_block_manager_without_torch():
    run(WITHOUT.format(module="torch") + HOST)


def test_the_block_manager_does_not_import_torch():
    run(HOST + "import sys\nassert 'torch' not in sys.modules\n")


def test_other_calls_without_the_bindings_module():
    """They are bound with ctypes; the three that need the module name it, before and behind load()."""
    run(WITHOUT.format(module="paged_kv_cache_241_gb300._pkv_call") + "import torch\n" + HOST + """
z = lambda *n: torch.zeros(*n, dtype=torch.bfloat16)
i = lambda *n: torch.zeros(*n, dtype=torch.int32)
try:
    pkv.kv_store(z(3, 2, 64), z(3, 2, 64), z(4, 256, 2, 64), z(4, 256, 2, 64), i(3))
    raise SystemExit("not refused")
except ValueError as e:
    assert "CUDA" in str(e)
calls = [lambda: pkv.plan_step(*[i(1)] * 11, 8, 256), lambda: pkv.norm_rope_store(*[z(1, 1, 64)] * 4, i(1), i(1)),
         lambda: pkv.paged_decode_shared_attn(*[z(1, 1, 64)] * 8, 0.1, z(1))]
for call in calls * 2:
    try:
        call()
        raise SystemExit("not refused")
    except RuntimeError as e:
        assert "paged_kv_cache_241_gb300.build" in str(e)
""")


def test_the_bindings_module_for_another_torch_is_told_of_where_it_is_needed():
    run("import torch\ntorch.__version__ = '0.1'\n" + HOST + """
i = lambda *n: torch.zeros(*n, dtype=torch.int32)
try:
    pkv.plan_step(*[i(1)] * 11, 8, 256)
    raise SystemExit("not refused")
except RuntimeError as e:
    assert "another" in str(e) and "built for torch" in str(e.__cause__)
""")
