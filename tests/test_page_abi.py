"""The calls over a cache in pages, and the norms and rotation in front of it,
refuse bad arguments on the host, before any launch (no GPU: the pointers are
fake and never read)."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

from kv_cache_eviction_kvc_gb300 import kvc as K

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

BIG = 1 << 40


def _pages(**kw):
    pg = K.kvc_pages(8, 128, K.PAGE_E4M3, 4, 16, 10, 5, 256, 256, 256, 256, 256, 256)
    for f, _ in K.kvc_pages._fields_:
        if f in kw:
            setattr(pg, f, kw[f])
    return ctypes.byref(pg) if kw.get("pg", 1) else None


def write(**kw):
    return K.load().kvc_page_write(_pages(**kw), kw.get("T", 3), None, None, kw.get("k", 256),
                                   kw.get("v", 256), kw.get("ws", 256), kw.get("ws_bytes", BIG), None)


def read(**kw):
    return K.load().kvc_page_read(_pages(**kw), kw.get("M", 3), kw.get("ld", 4), None, None,
                                  kw.get("k", 256), kw.get("v", 256), kw.get("ws", 256),
                                  kw.get("ws_bytes", BIG), None)


def attend(**kw):
    return K.load().kvc_page_attend(_pages(**kw), kw.get("G", 4), kw.get("max_len", 80),
                                    kw.get("q", 256), kw.get("k", 256), kw.get("v", 256),
                                    kw.get("o", 256), kw.get("lse", 256), kw.get("ws", 256),
                                    kw.get("ws_bytes", BIG), None)


@pytest.mark.parametrize("call", [write, read, attend])
@pytest.mark.parametrize("kw,code", [
    ({"pg": 0}, 1), ({"d": 64}, 5), ({"type": 2}, 1), ({"type": -1}, 1), ({"page": 0}, 5),
    ({"page": 8}, 5), ({"page": 48}, 5), ({"page": 256}, 5), ({"U": 0}, 1), ({"heads": 0}, 1),
    ({"heads": 3}, 1), ({"n_pages": 0}, 1), ({"stride": 0}, 1), ({"stride": 1 << 27}, 5),
    ({"K": None}, 1), ({"K": 264}, 1), ({"V": None}, 1), ({"V": 264}, 1), ({"k_scale": None}, 1),
    ({"v_scale": None}, 1), ({"table": None}, 1), ({"len": None}, 1), ({"k": 264}, 1), ({"v": 264}, 1),
    ({"ws": None}, 6), ({"ws": 128}, 6), ({"ws_bytes": 255}, 6)])
def test_refused_by_all(call, kw, code):
    assert call(**kw) == code
    assert K.kvc_last_error() != ""


@pytest.mark.parametrize("call,kw,code", [
    (write, {"T": 0}, 1), (write, {"k": None}, 1), (write, {"v": None}, 1),
    (write, {"U": 1 << 30, "T": 64}, 5), (read, {"M": 0}, 1), (read, {"ld": 2}, 2),
    (read, {"k": None}, 1), (read, {"v": None}, 1), (read, {"U": 1 << 30, "M": 64, "ld": 64}, 5),
    (attend, {"G": 3}, 5), (attend, {"G": 0}, 5), (attend, {"G": 16}, 5), (attend, {"max_len": 0}, 2),
    (attend, {"max_len": 81}, 2), (attend, {"q": None}, 1), (attend, {"q": 264}, 1),
    (attend, {"k": None}, 1), (attend, {"v": None}, 1), (attend, {"o": None}, 1),
    (attend, {"o": 264}, 1), (attend, {"lse": None}, 1)])
def test_refused(call, kw, code):
    assert call(**kw) == code
    assert K.kvc_last_error() != ""


def rope(**kw):
    r = K.kvc_rope(32, 8, 128, 128, 0, 1e-6, 1.0, 256, 256, 256, 8, 0)
    for f, _ in K.kvc_rope._fields_:
        if f in kw:
            setattr(r, f, kw[f])
    return K.load().kvc_qk_norm_rope(ctypes.byref(r) if kw.get("r", 1) else None, kw.get("B", 2),
                                     kw.get("T", 3), kw.get("qkv", 256), kw.get("row", 48 * 128),
                                     kw.get("pos", 256), None, kw.get("q", 256), kw.get("k", 256),
                                     kw.get("v", 256), None)


@pytest.mark.parametrize("kw,code", [
    ({"r": 0}, 1), ({"d": 64}, 5), ({"Hkv": 0}, 1), ({"Hq": 0}, 1), ({"Hq": 31}, 1), ({"Hq": 24}, 5),
    ({"Hq": 128}, 5), ({"Hq": 8192, "Hkv": 8192, "units": 8192, "row": 8192 * 384}, 5),
    ({"rot": -16}, 5), ({"rot": 8}, 5), ({"rot": 144}, 5), ({"interleaved": 2}, 1), ({"eps": -1.0}, 1),
    ({"eps": float("nan")}, 1), ({"eps": float("inf")}, 1), ({"scale": float("inf")}, 1),
    ({"inv_freq": None}, 1), ({"inv_freq": 260}, 1), ({"first_unit": -1}, 1), ({"first_unit": 1}, 1),
    ({"units": 7}, 1), ({"B": 0}, 1), ({"T": 0}, 1), ({"B": 1 << 20, "T": 1 << 12}, 5),
    ({"B": 1 << 29}, 5), ({"qkv": None}, 1), ({"pos": None}, 1), ({"q": None, "k": None, "v": None}, 1),
    ({"qkv": 264}, 1), ({"q": 264}, 1), ({"k": 264}, 1), ({"v": 264}, 1), ({"q_weight": 264}, 1),
    ({"k_weight": 264}, 1), ({"row": 48 * 128 - 8}, 2), ({"row": 48 * 128 + 4}, 2), ({"row": 0}, 2)])
def test_rope_refused(kw, code):
    assert rope(**kw) == code
    assert K.kvc_last_error() != ""


def _size(G=4, **kw):
    return int(K.load().kvc_page_workspace_size(_pages(**kw), G))


def test_workspace_size():
    assert _size() >= 256
    assert _size(G=3) == _size(page=20) == _size(pg=0) == 0


def test_binding_refuses_host_tensors_and_wrong_shapes():
    pool = torch.zeros(4, 2, 16, 128, dtype=torch.bfloat16)
    table, length = torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    for bad in ((pool, pool, None, None, table, length),            # host memory
                (pool, pool[:3], None, None, table, length), (pool[0], pool[0], None, None, table, length),
                (pool, pool, None, None, table[0], length), (None, pool, None, None, table, length),
                (pool, pool, length, length, table, length)):
        with pytest.raises(ValueError):
            K.make_pages(*bad)
    with pytest.raises(ValueError):
        K.make_rope(32, 8, torch.zeros(64, dtype=torch.float64))    # host memory


@pytest.mark.skipif(shutil.which("gcc") is None, reason="needs gcc")
def test_struct_layouts(tmp_path):
    """The header's structures and the binding's agree field by field."""
    lines = []
    for name, cls in (("kvc_rope", K.kvc_rope), ("kvc_pages", K.kvc_pages)):
        lines += [f'printf("%zu ", offsetof({name}, {f}));' for f, _ in cls._fields_]
        lines.append(f'printf("%zu ", sizeof({name}));')
    src = tmp_path / "l.c"
    src.write_text('#include <stdio.h>\n#include "kvc.h"\nint main(void){' + "".join(lines) + "return 0;}")
    subprocess.run(["gcc", "-std=c99", "-pedantic", "-Werror", "-I", os.path.join(ROOT, "include"), str(src),
                    "-o", str(tmp_path / "l")], check=True)
    got = [int(x) for x in subprocess.run([str(tmp_path / "l")], capture_output=True, text=True,
                                          check=True).stdout.split()]
    want = []
    for cls in (K.kvc_rope, K.kvc_pages):
        want += [getattr(cls, f).offset for f, _ in cls._fields_] + [ctypes.sizeof(cls)]
    assert got == want
