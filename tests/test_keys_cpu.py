"""Host-side argument checks of the key-set operators (no GPU needed)."""
import ctypes as C

import pytest

from token_locking_b200 import _abi as A


@pytest.fixture(scope="module")
def lib():
    from token_locking_b200 import build
    build.build()
    return A.lib()


GOOD = dict(dtype=A.SL_BF16, batch=2, n_ctx=64, max_rows=8, n_heads=8, n_kv_heads=2, head_dim=64,
            prefix=0, scale=0.0)


@pytest.mark.parametrize("change,status", [
    (dict(dtype=2), A.SL_ERR_INVALID), (dict(batch=0), A.SL_ERR_INVALID),
    (dict(batch=A.SL_MAX_BATCH + 1), A.SL_ERR_INVALID), (dict(n_ctx=0), A.SL_ERR_INVALID),
    (dict(batch=64, n_ctx=1 << 26), A.SL_ERR_INVALID), (dict(max_rows=0), A.SL_ERR_INVALID),
    (dict(n_heads=0), A.SL_ERR_INVALID), (dict(n_kv_heads=3), A.SL_ERR_INVALID),
    (dict(n_kv_heads=0), A.SL_ERR_INVALID), (dict(n_heads=130, n_kv_heads=2), A.SL_ERR_UNSUPPORTED),
    (dict(head_dim=0), A.SL_ERR_UNSUPPORTED), (dict(head_dim=136), A.SL_ERR_UNSUPPORTED),
    (dict(head_dim=12), A.SL_ERR_UNSUPPORTED), (dict(dtype=A.SL_F32, head_dim=6), A.SL_ERR_UNSUPPORTED),
    (dict(scale=-1.0), A.SL_ERR_INVALID), (dict(scale=float("nan")), A.SL_ERR_INVALID),
    (dict(scale=float("inf")), A.SL_ERR_INVALID),
])
def test_create_refuses(lib, change, status):
    cfg = A.KeyAttnConfig(**{**GOOD, **change})
    out = C.c_void_p(1)
    assert lib.sl_key_attn_create(C.byref(cfg), C.byref(out)) == status
    assert out.value is None and lib.sl_last_error()


def test_null_arguments(lib):
    out = C.c_void_p()
    cfg = A.KeyAttnConfig(**GOOD)
    assert lib.sl_key_attn_create(None, C.byref(out)) == A.SL_ERR_INVALID
    assert lib.sl_key_attn_create(C.byref(cfg), None) == A.SL_ERR_INVALID
    lib.sl_key_attn_destroy(None)
    ks = A.KeySet(16, 16, None)
    assert lib.sl_key_attention(None, 1, 16, 512, 16, 16, 128, C.byref(ks), None, None, 0, 0, 16,
                                512, None, None) == A.SL_ERR_INVALID
    assert lib.sl_key_mass(None, 1, 16, 512, 16, 128, C.byref(ks), 16, 0.0, None, 16,
                           None) == A.SL_ERR_INVALID


@pytest.mark.parametrize("change,status", [
    (dict(batch=0), A.SL_ERR_INVALID), (dict(batch=65), A.SL_ERR_INVALID),
    (dict(n_ctx=0), A.SL_ERR_INVALID), (dict(budget=-1), A.SL_ERR_INVALID),
    (dict(n_ctx=(1 << 20) + 1), A.SL_ERR_UNSUPPORTED), (dict(mass=None), A.SL_ERR_INVALID),
    (dict(keys=None), A.SL_ERR_INVALID), (dict(key_len=None), A.SL_ERR_INVALID),
])
def test_evict_refuses(lib, change, status):
    a = dict(batch=2, n_ctx=64, budget=8, mass=16, protect=None, present=None, keys=16, key_len=16,
             present_out=None)
    a.update(change)
    assert lib.sl_kv_evict(*a.values(), None) == status


def test_struct_layouts_match_the_header(tmp_path):
    import os
    import shutil
    import subprocess
    if shutil.which("gcc") is None:
        pytest.skip("gcc not on PATH")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    pairs = [("sl_key_attn_config", A.KeyAttnConfig), ("sl_key_set", A.KeySet)]
    body = "".join(f'  printf("{n} size %zu\\n", sizeof({n}));\n' + "".join(
        f'  printf("{n} {f} %zu\\n", offsetof({n}, {f}));\n' for f, _ in p._fields_) for n, p in pairs)
    src = tmp_path / "layout.c"
    src.write_text('#include "surelock.h"\n#include <stddef.h>\n#include <stdio.h>\nint main(void) {\n'
                   + body + "  return 0;\n}\n")
    exe = str(tmp_path / "layout")
    subprocess.run(["gcc", "-std=c99", "-I" + os.path.join(root, "include"), str(src), "-o", exe],
                   check=True)
    got = {tuple(l.split()[:2]): int(l.split()[2])
           for l in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.splitlines()}
    for n, p in pairs:
        assert got[(n, "size")] == C.sizeof(p)
        for f, _ in p._fields_:
            assert got[(n, f)] == getattr(p, f).offset
