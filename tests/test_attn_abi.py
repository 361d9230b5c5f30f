"""Refusals of the attention-layer operators (include/gdnattn.h): host validation before
anything is launched, and the Python binding's checks.  No GPU."""
import ctypes

import pytest
import torch

import speculative_decode_recurrent_gb300 as lib

FAKE = 0x10000                       # never dereferenced: validation fails first


def cache(**kw):
    d = dict(n_slot=4, max_pages=8, n_page=16, page=16, n_layer=2, Hkv=2, d=128, dtype=lib.DTYPE_BF16)
    d.update({f: FAKE for f in lib.PagedCache._FIELDS})
    d.update(kw)
    return lib.PageDims(**d)


def dims(**kw):
    return lib.AttnDims(**{**dict(B=2, T=4, Hq=8, scale=0.1), **kw})


def rope(**kw):
    return lib.RopeDims(**{**dict(rot=64, style=lib.ROPE_HALF, max_pos=128, eps=1e-6, q_stride=1024, k_stride=256,
                                  v_stride=256), **kw})


def stage(c=None, a=None, r=None, layer=0, args=None):
    c, a, r = c or cache(), a or dims(), r or rope()
    # state_idx, draft_len, q, k, v, pos, q_weight, k_weight, cos_sin, q_out, status
    return lib.load().gdn_attn_stage(ctypes.byref(c), layer, ctypes.byref(a), ctypes.byref(r), *(args or [FAKE] * 11), None)


def verify(c=None, a=None, layer=0, args=None, size=1 << 40):
    c, a = c or cache(), a or dims()
    # state_idx, draft_len, q, tree, out, lse, workspace, status
    args = args or [FAKE] * 8
    return lib.load().gdn_attn_verify(ctypes.byref(c), layer, ctypes.byref(a), *args[:7], size, args[7], None)


def test_struct_sizes_match_the_header():
    assert ctypes.sizeof(lib.PageDims) == 8 * 4 + 8 * 8
    assert ctypes.sizeof(lib.AttnDims) == 20 and ctypes.sizeof(lib.RopeDims) == 40


@pytest.mark.parametrize("kw,code", [
    (dict(page=48), -2), (dict(page=8), -2), (dict(page=256), -2), (dict(d=96), -2), (dict(Hkv=0), -2), (dict(Hkv=129), -2),
    (dict(n_page=0), -2), (dict(max_pages=0), -2), (dict(max_pages=(1 << 18) + 1), -2), (dict(n_layer=0), -2),
    (dict(n_slot=-1), -2), (dict(n_page=1 << 27), -2), (dict(dtype=2), -3)])
def test_bad_cache_refused(kw, code):
    c, so = cache(**kw), lib.load()
    p = ctypes.byref(c)
    assert stage(c) == verify(c) == code
    assert so.gdn_attn_accept(p, 2, 4, FAKE, FAKE, FAKE, FAKE, FAKE, None) == code
    assert so.gdn_attn_workspace(p, ctypes.byref(dims())) == code
    assert so.gdn_tree_build(p, ctypes.byref(dims()), FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None) == code
    assert so.gdn_pages_reserve(p, 1, FAKE, 1, FAKE, None) == code
    assert so.gdn_pages_fork(p, 1, FAKE, FAKE, FAKE, FAKE, None) == code
    assert so.gdn_pages_copy(p, 1, FAKE, FAKE, None) == code
    assert so.gdn_pages_release(p, 1, FAKE, FAKE, None) == code


@pytest.mark.parametrize("kw", [dict(B=-1), dict(B=65536), dict(T=0), dict(Hq=0), dict(Hq=7), dict(Hq=130), dict(scale=0.0),
                                dict(scale=float("nan")), dict(flags=2)])
def test_bad_dims_refused(kw):
    assert stage(a=dims(**kw)) == verify(a=dims(**kw)) == -2


def test_lengths_of_the_calls():
    so = lib.load()
    assert verify(a=dims(T=65)) == -2 and stage(a=dims(T=(1 << 20) + 1)) == -2
    assert stage(a=dims(B=65535, T=1 << 20)) == -2
    c = ctypes.byref(cache())
    assert so.gdn_attn_accept(c, 2, 65, FAKE, FAKE, FAKE, FAKE, FAKE, None) == -2
    assert so.gdn_pages_reserve(c, 4097, FAKE, 1, FAKE, None) == -2
    assert so.gdn_pages_reserve(c, 1, FAKE, -1, FAKE, None) == -2
    assert verify(layer=2) == verify(layer=-1) == stage(layer=2) == -2


@pytest.mark.parametrize("kw", [dict(rot=8), dict(rot=144), dict(rot=-16), dict(style=2), dict(max_pos=0), dict(eps=-1.0),
                                dict(eps=float("nan")), dict(q_stride=1016), dict(k_stride=252), dict(v_stride=260)])
def test_bad_rotation_refused(kw):
    assert stage(r=rope(**kw)) == -2


def test_more_layers_than_a_call_can_count_refused():
    # an accept of 128 fp32 heads of 256 counts 2^14 columns per layer, in 32 bits
    c, so = cache(n_layer=1 << 17, Hkv=128, d=256, dtype=lib.DTYPE_F32), lib.load()
    p = ctypes.byref(c)
    assert so.gdn_attn_accept(p, 2, 4, FAKE, FAKE, FAKE, FAKE, FAKE, None) == -2
    assert so.gdn_pages_copy(p, 1, FAKE, FAKE, None) == -2
    assert stage(cache(n_layer=32768)) == verify(cache(n_layer=32768)) == -2


def test_null_and_misaligned_pointers_refused():
    so = lib.load()
    for i in (2, 3, 4, 6, 7, 8, 9, 10):                       # state_idx, draft_len and pos may be NULL
        args = [FAKE] * 11
        args[i] = None
        assert stage(args=args) == -1, i
    for i in (2, 4, 7):
        args = [FAKE] * 8
        args[i] = None
        assert verify(args=args) == -1, i
    for i in (2, 4, 6):
        args = [FAKE] * 8
        args[i] = FAKE + 8
        assert verify(args=args) == -2, i
    for i in (7, 8, 9):                                       # norm weights, angles
        args = [FAKE] * 11
        args[i - 1] = FAKE + 4
        assert stage(args=args) == -2, i
    for f in ("k", "v", "block_table", "seq_len"):
        assert stage(cache(**{f: None})) == verify(cache(**{f: None})) == -1, f
    for f in ("k", "v"):
        assert stage(cache(**{f: FAKE + 4})) == verify(cache(**{f: FAKE + 4})) == -2, f
    for f in ("block_table", "seq_len", "n_owned", "ref", "free_list", "free_count"):
        assert so.gdn_pages_release(ctypes.byref(cache(**{f: None})), 1, FAKE, FAKE, None) == -1, f
    assert so.gdn_attn_verify(None, 0, ctypes.byref(dims()), *([FAKE] * 7), 1 << 40, FAKE, None) == -1
    assert so.gdn_attn_accept(ctypes.byref(cache()), 2, 4, FAKE, FAKE, None, FAKE, FAKE, None) == -1
    # the identity slot map needs a slot per row
    args = [FAKE] * 8
    args[0] = None
    assert verify(cache(n_slot=1), args=args) == -2


def test_empty_calls_do_nothing():
    so = lib.load()
    c, none = cache(n_slot=0, **{f: None for f in lib.PagedCache._FIELDS}), dims(B=0)
    assert stage(c, none, args=[None] * 11) == verify(c, none, args=[None] * 8) == 0
    assert so.gdn_attn_accept(ctypes.byref(c), 0, 4, None, None, None, None, None, None) == 0
    assert so.gdn_pages_fork(ctypes.byref(c), 0, None, None, None, None, None) == 0


def test_binding_refuses_wrong_tensors():
    f = lib.PagedCache._FIELDS
    init = {n: torch.zeros(1, dtype=torch.int32) for n in f}
    with pytest.raises(ValueError, match="k: expected shape"):
        lib.PagedCache(cache(), init, device="cpu")
    with pytest.raises(TypeError, match="dtype"):
        lib.PagedCache(cache(dtype=9), init, device="cpu")
    with pytest.raises(ValueError, match="CUDA"):
        lib._in(torch.zeros(4), torch.float32, 4, "x")
