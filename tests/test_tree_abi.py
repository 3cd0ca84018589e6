"""The drafted-token entry points refuse bad arguments on the host, before any
launch (no GPU: the pointers are fake and never read)."""
import ctypes

import pytest
import torch

from kv_cache_eviction_kvc_gb300 import kvc as K

BIG = 1 << 40


def _args(**kw):
    p = K.make_params(U=4, G=4, cap=100, L=10)
    for f in ("d", "G", "U", "L", "cap", "rule", "merge"):
        if f in kw:
            setattr(p, f, kw[f])
    cache = K.kvc_cache(*(kw.get(f, 256 * (i + 1)) for i, f in
                          enumerate(["K", "V", "votes", "pos", "util", "len"])))
    tree = K.kvc_tree(kw.get("T", 8), kw.get("units", 2), kw.get("mask", 256), None)
    path = K.kvc_path(kw.get("A", 3), kw.get("token", 256), kw.get("npath", 256),
                      kw.get("path_pos", 256))
    mom = K.kvc_moments(256, kw.get("mu_k", 256), 256, kw.get("C", 256))
    return p, cache, tree, path, mom


def attend(**kw):
    p, c, t, _, m = _args(**kw)
    return K.load().kvc_tree_attend(
        ctypes.byref(p), kw.get("max_len", 10), ctypes.byref(t), kw.get("q", 256),
        kw.get("kt", 256), kw.get("vt", 256), ctypes.byref(c), ctypes.byref(m), kw.get("o", 256),
        kw.get("lse", 256), kw.get("ws", 256), kw.get("ws_bytes", BIG), None)


def weights(**kw):
    p, c, t, a, _ = _args(**kw)
    return K.load().kvc_tree_weights(
        ctypes.byref(p), kw.get("max_len", 10), ctypes.byref(t), ctypes.byref(a), None,
        kw.get("q", 256), kw.get("kt", 256), kw.get("lse", 256), ctypes.byref(c),
        kw.get("S", 256), kw.get("ws", 256), kw.get("ws_bytes", BIG), None)


def commit(**kw):
    p, c, t, a, m = _args(**kw)
    return K.load().kvc_tree_commit(
        ctypes.byref(p), kw.get("max_len", 10), ctypes.byref(t), ctypes.byref(a),
        kw.get("kt", 256), kw.get("vt", 256), None, ctypes.byref(c), ctypes.byref(m),
        kw.get("kmax", 3), None, None, kw.get("n_evict", 256), kw.get("ws", 256),
        kw.get("ws_bytes", BIG), None)


@pytest.mark.parametrize("call", [attend, weights, commit])
@pytest.mark.parametrize("kw,code", [
    ({"d": 64}, 5), ({"G": 3}, 5), ({"U": 0}, 1), ({"cap": 0}, 5), ({"L": 100}, 1),
    ({"K": None}, 1), ({"K": 264}, 1), ({"len": None}, 1),
    ({"max_len": 0}, 2), ({"max_len": 101}, 2),
    ({"T": 0}, 1), ({"T": 65}, 5), ({"units": 0}, 1), ({"units": 3}, 1), ({"mask": None}, 1),
    ({"mask": 260}, 1), ({"kt": None}, 1), ({"kt": 264}, 1),
    ({"ws": None}, 6), ({"ws": 128}, 6), ({"ws_bytes": 255}, 6)])
def test_refused_by_all(call, kw, code):
    assert call(**kw) == code
    assert K.kvc_last_error() != ""


@pytest.mark.parametrize("call,kw,code", [
    (attend, {"q": None}, 1), (attend, {"q": 264}, 1), (attend, {"vt": None}, 1),
    (attend, {"o": None}, 1), (attend, {"o": 264}, 1), (attend, {"lse": None}, 1),
    (attend, {"C": 264}, 1), (attend, {"mu_k": None}, 1),
    (weights, {"q": 264}, 1), (weights, {"lse": None}, 1), (weights, {"S": None}, 1),
    (weights, {"A": 0}, 1), (weights, {"A": 9}, 1), (weights, {"token": None}, 1),
    (weights, {"npath": None}, 1), (commit, {"path_pos": None}, 1), (commit, {"A": 9}, 1),
    (commit, {"vt": None}, 1), (commit, {"n_evict": None}, 1), (commit, {"kmax": 0}, 1),
    (commit, {"kmax": 65}, 5), (commit, {"rule": K.RULE_MI}, 5), (commit, {"C": None}, 1)])
def test_refused(call, kw, code):
    assert call(**kw) == code
    assert K.kvc_last_error() != ""


def test_commit_refuses_merging_and_the_chained_rule():
    lib = K.load()
    for p in (K.make_params(U=4, G=4, cap=100, L=10, merge_recent=2),
              K.make_params(U=4, G=4, cap=100, L=10, rule=K.RULE_EMA_CHAINED, chain=(2, 2))):
        _, c, t, a, m = _args()
        assert lib.kvc_tree_commit(ctypes.byref(p), 10, ctypes.byref(t), ctypes.byref(a), 256, 256,
                                   None, ctypes.byref(c), ctypes.byref(m), 3, None, None, 256, 256,
                                   BIG, None) == 5


def test_workspace_size():
    p = K.make_params(U=4, G=4, cap=100, L=10)
    assert K.kvc_tree_workspace_size(p, 8) >= 256
    assert K.kvc_tree_workspace_size(p, 0) == K.kvc_tree_workspace_size(p, 65) == 0
    assert K.kvc_tree_workspace_size(K.make_params(U=4, G=3, cap=100, L=10), 8) == 0


def test_binding_refuses_host_tensors_and_wrong_shapes():
    mask = torch.zeros(2, 8, dtype=torch.int64)
    with pytest.raises(ValueError):
        K.make_tree(8, 2, mask)                        # host memory
    with pytest.raises(ValueError):
        K.make_tree(7, 2, mask)                        # another row stride
    with pytest.raises(ValueError):
        K.make_tree(8, 2, None)
    with pytest.raises(ValueError):
        K.make_path(3, torch.zeros(2, 4, dtype=torch.int32), mask, mask)


def wide(call, name):
    """The fp64 form takes what the fp32 form takes: its refusals by the same arguments."""
    lib = K.load()
    old = getattr(lib, name)
    setattr(lib, name, getattr(lib, name + "_f64"))
    try:
        return call()
    finally:
        setattr(lib, name, old)


@pytest.mark.parametrize("kw,code", [
    ({"d": 64}, 5), ({"G": 3}, 5), ({"U": 0}, 1), ({"L": 100}, 1), ({"K": None}, 1), ({"max_len": 0}, 2),
    ({"max_len": 101}, 2), ({"T": 65}, 5), ({"units": 3}, 1), ({"mask": None}, 1), ({"kt": 264}, 1),
    ({"A": 9}, 1), ({"token": None}, 1), ({"ws": None}, 6), ({"ws_bytes": 255}, 6)])
@pytest.mark.parametrize("call,name", [(weights, "kvc_tree_weights"), (commit, "kvc_tree_commit")])
def test_f64_forms_refuse_the_same(call, name, kw, code):
    assert wide(lambda: call(**kw), name) == code
    assert name + "_f64" in K.kvc_last_error() or code in (1, 5)


def test_f64_weights_must_be_aligned():
    assert wide(lambda: weights(S=260), "kvc_tree_weights") == 1
    p, c, t, a, m = _args()
    assert K.load().kvc_tree_commit_f64(
        ctypes.byref(p), 10, ctypes.byref(t), ctypes.byref(a), 256, 256, 260, ctypes.byref(c),
        ctypes.byref(m), 3, None, None, 256, 256, BIG, None) == 1
    assert "S must be" in K.kvc_last_error()
