"""Refusals of the operators on committed tokens and drafts (gdn_replay_advance, gdn_conv_advance, gdn_attn_chunk,
gdn_draft_accept): host validation before anything is launched, and the Python binding's checks.  No GPU."""
import ctypes

import pytest
import torch

import speculative_decode_recurrent_gb300 as lib

FAKE = 0x10000                       # never dereferenced: validation fails first
BF, F32 = lib.DTYPE_BF16, lib.DTYPE_F32


def adv(**kw):
    d = dict(B=2, T=4, H=4, Hk=2, dk=128, dv=128, n_slot=4, in_dtype=BF, scale=0.1, q_stride=256, k_stride=256, v_stride=512)
    return lib.AdvanceDims(**{**d, **kw})


def advance(d=None, args=None, size=1 << 40):
    # state, state_idx, buf_len, chunk_len, fresh, q, k, v, g, beta, out, workspace, status
    a = args or [FAKE] * 13
    return lib.load().gdn_replay_advance(ctypes.byref(d or adv()), *a[:12], size, a[12], None)


def conv(**kw):
    return lib.ConvDims(**{**dict(B=2, D=64, W=4, T=100, cap=4, n_slot=4, act=0, in_dtype=BF, out_dtype=BF), **kw})


def conv_advance(d=None, args=None):
    # ring, ring_pos, state_idx, chunk_len, fresh, x, weight, bias, y, status
    return lib.load().gdn_conv_advance(ctypes.byref(d or conv()), *(args or [FAKE] * 10), None)


def cache(**kw):
    d = dict(n_slot=4, max_pages=8, n_page=16, page=16, n_layer=2, Hkv=2, d=128, dtype=BF)
    d.update({f: FAKE for f in lib.PagedCache._FIELDS})
    return lib.PageDims(**{**d, **kw})


def chunk(c=None, a=None, layer=0, args=None, size=1 << 40):
    # state_idx, chunk_len, q, out, lse, workspace, status
    g = args or [FAKE] * 7
    a = a or lib.AttnDims(B=2, T=100, Hq=8, scale=0.1)
    return lib.load().gdn_attn_chunk(ctypes.byref(c or cache()), layer, ctypes.byref(a), *g[:6], size, g[6], None)


def draft(args=None, **kw):
    # tokens, parent, probs, draft, u, draft_len, accepted, next, path, status
    d = lib.DraftDims(**{**dict(B=2, T=4, V=100, flags=0, p_stride=100, q_stride=100), **kw})
    return lib.load().gdn_draft_accept(ctypes.byref(d), *(args or [FAKE] * 10), None)


def without(n, i, value=None):
    args = [FAKE] * n
    args[i] = value
    return args


def test_struct_sizes_match_the_header():
    assert ctypes.sizeof(lib.AdvanceDims) == 10 * 4 + 3 * 8 and ctypes.sizeof(lib.DraftDims) == 4 * 4 + 2 * 8


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), -2), (dict(B=65536, n_slot=65536), -2), (dict(T=0), -2), (dict(T=(1 << 20) + 1), -2), (dict(B=4, T=1 << 27), -2),
    (dict(H=0), -2), (dict(H=1025, Hk=1025), -2), (dict(Hk=0), -2), (dict(Hk=3), -2), (dict(dk=96), -2), (dict(dv=32), -2),
    (dict(n_slot=1), -2), (dict(n_slot=1 << 23), -2), (dict(flags=2), -2), (dict(in_dtype=2), -3), (dict(q_stride=248), -2),
    (dict(k_stride=0), -2), (dict(v_stride=511), -2), (dict(v_stride=516), -2), (dict(q_stride=-256), -2),
    (dict(k_stride=(1 << 38) + 8), -2)])
def test_bad_advance_refused(kw, code):
    assert advance(adv(**kw)) == code
    assert lib.load().gdn_replay_advance_workspace(ctypes.byref(adv(**kw))) == code
    with pytest.raises(lib.GdnError):
        lib.gdn_replay_advance_workspace(adv(**kw))


def test_advance_pointers_and_workspace_refused():
    so = lib.load()
    assert so.gdn_replay_advance(None, *[FAKE] * 12, 1 << 40, FAKE, None) == -1
    assert so.gdn_replay_advance_workspace(None) == -1
    for i in (0, 5, 6, 7, 8, 9, 10, 12):                      # slots, lengths and fresh may be NULL
        assert advance(args=without(13, i)) == -1, i
    for i in (0, 5, 6, 7, 10):
        assert advance(args=without(13, i, FAKE + 8)) == -2, i
    long = adv(T=1000)
    need = so.gdn_replay_advance_workspace(ctypes.byref(long))
    assert need > 0 and so.gdn_replay_advance_workspace(ctypes.byref(adv())) == 0
    assert so.gdn_replay_advance_workspace(ctypes.byref(adv(T=1000, in_dtype=F32))) == 0
    assert advance(long, size=need - 1) == -2
    assert advance(long, without(13, 11), size=need) == -1
    assert advance(long, without(13, 11, FAKE + 8), size=need) == -2
    assert advance(adv(B=0), [None] * 13, 0) == 0


def test_advance_workspace_is_bounded():
    """Long prompts and many sequences come in several launches over one workspace."""
    for kw in (dict(T=1 << 20, B=1, H=64, Hk=64), dict(B=4096, T=65, n_slot=4096, H=32, Hk=32), dict(B=1, H=1024, Hk=1, T=1 << 20)):
        d = adv(q_stride=1 << 20, k_stride=1 << 20, v_stride=1 << 20, **kw)
        assert 0 < lib.gdn_replay_advance_workspace(d) <= 768 << 20


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), -2), (dict(B=65536, n_slot=65536), -2), (dict(T=0), -2), (dict(T=(1 << 20) + 1), -2), (dict(D=12), -2), (dict(D=0), -2),
    (dict(W=5, cap=9), -2), (dict(W=0), -2), (dict(cap=2), -2), (dict(cap=4097), -2), (dict(W=1, cap=0), -2), (dict(n_slot=1), -2),
    (dict(act=2), -2), (dict(in_dtype=2), -3), (dict(out_dtype=-1), -3), (dict(B=4, T=1 << 27), -2)])
def test_bad_conv_advance_refused(kw, code):
    assert conv_advance(conv(**kw)) == code


def test_conv_advance_pointers_refused():
    assert lib.load().gdn_conv_advance(None, *[FAKE] * 10, None) == -1
    for i in (0, 1, 5, 6, 8, 9):                              # slots, lengths, fresh and bias may be NULL
        assert conv_advance(args=without(10, i)) == -1, i
    for i in (0, 5, 6, 7, 8):
        assert conv_advance(args=without(10, i, FAKE + 8)) == -2, i
    assert conv_advance(conv(B=0), [None] * 10) == 0


@pytest.mark.parametrize("T", [4, 100])
def test_bad_chunk_refused(T):
    def dims(**kw):
        return lib.AttnDims(**{**dict(B=2, T=T, Hq=8, scale=0.1), **kw})

    def refused(c, a, code):
        assert chunk(c, a) == code
        assert lib.load().gdn_attn_chunk_workspace(ctypes.byref(c), ctypes.byref(a)) == code

    for kw in (dict(page=48), dict(d=96), dict(Hkv=0), dict(n_page=0), dict(max_pages=0), dict(n_layer=0)):
        refused(cache(**kw), dims(), -2)
    refused(cache(dtype=2), dims(), -3)
    for kw in (dict(B=-1), dict(T=0), dict(T=(1 << 20) + 1), dict(B=300, T=1 << 20), dict(Hq=7), dict(scale=0.0), dict(flags=2)):
        refused(cache(), dims(**kw), -2)
    a = dims()
    assert chunk(a=a, layer=2) == chunk(a=a, layer=-1) == -2
    assert chunk(cache(n_slot=1), a, args=without(7, 0)) == -2
    for i in (2, 3, 6):
        assert chunk(a=a, args=without(7, i)) == -1, i
    for i in (2, 3, 5):
        assert chunk(a=a, args=without(7, i, FAKE + 8)) == -2, i
    for f in ("k", "v", "block_table", "seq_len"):
        assert chunk(cache(**{f: None}), a) == -1, f
    for f in ("k", "v"):
        assert chunk(cache(**{f: FAKE + 4}), a) == -2, f
    assert chunk(a=a, size=-1) == -2
    none = cache(n_slot=0, **{f: None for f in lib.PagedCache._FIELDS})
    assert chunk(none, dims(B=0), args=[None] * 7, size=0) == 0


@pytest.mark.parametrize("kw", [dict(B=-1), dict(B=65536), dict(T=0), dict(T=65), dict(V=0), dict(V=(1 << 24) + 1), dict(flags=1),
                                dict(p_stride=99), dict(q_stride=99), dict(p_stride=-100)])
def test_bad_draft_refused(kw):
    assert draft(**kw) == -2


def test_draft_pointers_refused():
    assert lib.load().gdn_draft_accept(None, *[FAKE] * 10, None) == -1
    for i in (0, 2, 4, 6, 7, 8, 9):                           # a tree needs a path; parent, draft and draft_len may be NULL
        assert draft(without(10, i)) == -1, i
    assert draft([None] * 10, B=0) == 0


def test_binding_refuses_wrong_tensors():
    z = torch.zeros
    d = lib.Dims(B=1, H=2, dk=64, dv=64, T=4, cap=8, threshold=4, n_slot=1, in_dtype=F32, scale=0.1)
    init = dict(state=z(1, 2, 64, 64), state_idx=None, buf_k=z(1, 2, 8, 64), buf_v=z(1, 2, 8, 64), buf_g=z(1, 2, 8),
                buf_beta=z(1, 2, 8), buf_len=z(1, dtype=torch.int32))
    layer = lib.ReplayLayer(d, init, "cpu")
    x, g = z(1, 9, 2, 64), z(1, 9, 2)
    with pytest.raises(ValueError, match="expected \\[B, T, Hk, dk\\]"):
        layer.advance(x[0], x, x, g, g, x)
    with pytest.raises(ValueError, match="q: expected a CUDA tensor"):
        layer.advance(x, x, x, g, g, x)
    with pytest.raises(ValueError, match="q: expected shape"):
        layer.advance(x.transpose(2, 3), x, x, g, g, x)
    with pytest.raises(lib.GdnError):
        layer.advance(x[:, :0], x[:, :0], x, g, g, x)
    assert layer.advance_workspace(9) is None
    dims = lib.ConvDims(B=1, D=8, W=2, T=1, cap=2, n_slot=1, act=0, in_dtype=F32, out_dtype=F32)
    one = lib.ConvLayer(dims, dict(ring=z(1, 2, 8), pos=z(1, dtype=torch.int32), state_idx=None, weight=z(8, 2)), "cpu")
    with pytest.raises(ValueError, match="expected \\[B, T, D\\]"):
        one.advance(z(3, 8), z(1, 3, 8))
    with pytest.raises(ValueError, match="ring"):
        one.advance(z(1, 3, 8), z(1, 3, 8))
    s = lib.DraftSampler(lib.DraftDims(B=2, T=3, V=10), "cpu")
    i = z(2, 3, dtype=torch.int32)
    with pytest.raises(ValueError, match="probs: expected shape"):
        s.accept(i, z(2, 3, 11), z(2, 3), i[:, 0], i[:, 0])
    with pytest.raises(TypeError, match="probs: expected torch.float32"):
        s.accept(i, z(2, 3, 10).double(), z(2, 3), i[:, 0], i[:, 0])
    with pytest.raises(ValueError, match="probs: rows must be dense"):
        s.accept(i, z(2, 10, 3).transpose(1, 2), z(2, 3), i[:, 0], i[:, 0])
    with pytest.raises(ValueError, match="draft: rows must be dense"):
        s.accept(i, z(2, 3, 10), z(2, 3), i[:, 0], i[:, 0], draft=z(3, 2, 10).transpose(0, 1))
    with pytest.raises(TypeError, match="probs: expected a torch.Tensor"):
        s.accept(i, None, z(2, 3), i[:, 0], i[:, 0])
