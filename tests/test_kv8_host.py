"""Host-side refusals of the 8-bit KV cache calls (no GPU, nothing launched):
every documented restriction returns its status before any launch, and the
binding rejects tensors the library would misread."""
import ctypes as C
import os

import pytest
import torch

from long_context_sparse_09_b200 import binding as bd

ARG, SHAPE, ALIGN, DTYPE, UNSUPPORTED, WORKSPACE = 1, 2, 3, 4, 7, 8
F = 1 << 20            # an address that is never dereferenced: validation fails first
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(bd.LIB_PATH):
        from long_context_sparse_09_b200 import build
        build.build_library()
    return bd.lib()


def _call(lib, name, good, changes):
    args = dict(good, **changes)
    return getattr(lib, name)(*args.values())


def rope(**kw):
    r = bd.rope_params(128, 64)
    for k, v in kw.items():
        setattr(r, k, v)
    return C.byref(r)


def params(**kw):
    p = bd.kv8_params(8, 2, 64, 16, 64, "bf16")
    for k, v in kw.items():
        setattr(p, k, v)
    return C.byref(p)


FREQS = dict(r=None, turns=F, stream=None)


@pytest.mark.parametrize("r, st", [
    (dict(base=0.0), ARG), (dict(base=NAN), ARG), (dict(scaling=3), ARG), (dict(scaling=-1), ARG),
    (dict(scaling=1, factor=0.0), ARG), (dict(scaling=1, factor=INF), ARG),
    (dict(scaling=2, factor=2.0, orig_len=0.0), ARG),
    (dict(scaling=2, factor=2.0, orig_len=4096.0, fast=1.0, slow=1.0), ARG),
    (dict(d=0), SHAPE), (dict(d=132), SHAPE), (dict(d=520), SHAPE), (dict(rope_dims=63), SHAPE),
    (dict(rope_dims=130, rope_off=0), SHAPE), (dict(rope_off=65), SHAPE), (dict(rope_off=-2), SHAPE),
    (dict(layout=2), ARG), (dict(mscale=NAN), ARG)])
def test_rope_freqs_refusals(lib, r, st):
    assert _call(lib, "csa_rope_freqs", FREQS, dict(r=rope(**r))) == st


def test_rope_freqs_pointers(lib):
    assert _call(lib, "csa_rope_freqs", FREQS, dict(r=None)) == ARG
    assert _call(lib, "csa_rope_freqs", FREQS, dict(r=rope(), turns=None)) == ARG
    assert _call(lib, "csa_rope_freqs", FREQS, dict(r=rope(), turns=F + 4)) == ALIGN
    assert _call(lib, "csa_rope_freqs", FREQS, dict(r=rope(rope_dims=0), turns=None)) == 0


NORM = dict(r=None, R=4, n_q=8, n_kv=2, act=1, norm=1, eps=1e-6, turns=F, pos=F, q=F, q_stride=1024,
            q_gain=None, k=F, k_stride=256, k_gain=None, q_out=F, qo_stride=1024, k_out=F, ko_stride=256,
            stream=None)


@pytest.mark.parametrize("ch, st", [
    (dict(R=-1), SHAPE), (dict(n_q=0), SHAPE), (dict(n_kv=-1), SHAPE), (dict(act=2), DTYPE),
    (dict(norm=2), ARG), (dict(eps=-1.0), ARG), (dict(eps=NAN), ARG), (dict(q_stride=1016), SHAPE),
    (dict(ko_stride=0), SHAPE), (dict(q_stride=1028), ALIGN), (dict(q=None), ARG), (dict(k=None), ARG),
    (dict(k_out=None), ARG), (dict(n_kv=0), ARG), (dict(pos=None), ARG), (dict(turns=None), ARG),
    (dict(q=F + 8), ALIGN), (dict(k_out=F + 2), ALIGN), (dict(q_gain=F + 4), ALIGN), (dict(turns=F + 4), ALIGN)])
def test_norm_rope_refusals(lib, ch, st):
    assert _call(lib, "csa_qk_norm_rope", NORM, dict(dict(r=rope()), **ch)) == st


def test_norm_rope_of_no_tokens(lib):
    assert _call(lib, "csa_qk_norm_rope", NORM, dict(r=rope(), R=0, q=None, k=None, pos=None)) == 0


BAD_PARAMS = [
    (dict(n_q=7), SHAPE), (dict(n_q=0), SHAPE), (dict(n_kv=0), SHAPE), (dict(block=8), SHAPE),
    (dict(block=48), SHAPE), (dict(block=0), SHAPE), (dict(N=0), SHAPE), (dict(N=40), SHAPE),
    (dict(d=32), UNSUPPORTED), (dict(d=96), UNSUPPORTED), (dict(act=2), DTYPE)]

APPEND = dict(p=None, B=2, T=3, k=F, k_stride=128, v=F, v_stride=128, n_old=F, n_new=None, kc=F,
              k_exp=F, vc=F, v_exp=F, stream=None)
ATTEND = dict(p=None, B=2, Q=3, scale=0.1, q=F, n_vis=F, kc=F, k_exp=F, vc=F, v_exp=F, sink=None,
              out=F, acc=None, decay=1.0, ws=F, ws_bytes=1 << 30, stream=None)
EVICT = dict(p=None, B=2, keep=3, recent=2, acc=F, n_tok=F, kc=F, k_exp=F, vc=F, v_exp=F, kept=F,
             acc_out=F, n_tok_out=F, stream=None)


@pytest.mark.parametrize("name, good", [("csa_kv8_append", APPEND), ("csa_kv8_attend", ATTEND),
                                        ("csa_kv8_evict", EVICT)])
@pytest.mark.parametrize("bad, st", BAD_PARAMS)
def test_parameter_refusals(lib, name, good, bad, st):
    assert _call(lib, name, good, dict(p=params(**bad))) == st
    assert _call(lib, name, good, dict(p=None)) == ARG
    assert lib.csa_kv8_attend_workspace_bytes(params(**bad), 2, 3, 1) == 0


@pytest.mark.parametrize("name, good, ch, st", [
    ("csa_kv8_append", APPEND, dict(B=0), SHAPE), ("csa_kv8_append", APPEND, dict(T=-1), SHAPE),
    ("csa_kv8_append", APPEND, dict(k_stride=127), SHAPE), ("csa_kv8_append", APPEND, dict(v_stride=132), ALIGN),
    ("csa_kv8_append", APPEND, dict(v=None), ARG), ("csa_kv8_append", APPEND, dict(n_old=None), ARG),
    ("csa_kv8_append", APPEND, dict(vc=None), ARG), ("csa_kv8_append", APPEND, dict(kc=F + 8), ALIGN),
    ("csa_kv8_append", APPEND, dict(k=F + 4), ALIGN),
    ("csa_kv8_append", APPEND, dict(T=0, k=None, v=None), 0),
    ("csa_kv8_attend", ATTEND, dict(B=0), SHAPE), ("csa_kv8_attend", ATTEND, dict(Q=0), SHAPE),
    ("csa_kv8_attend", ATTEND, dict(scale=NAN), ARG), ("csa_kv8_attend", ATTEND, dict(scale=INF), ARG),
    ("csa_kv8_attend", ATTEND, dict(acc=F, decay=NAN), ARG), ("csa_kv8_attend", ATTEND, dict(q=None), ARG),
    ("csa_kv8_attend", ATTEND, dict(n_vis=None), ARG), ("csa_kv8_attend", ATTEND, dict(out=None), ARG),
    ("csa_kv8_attend", ATTEND, dict(k_exp=None), ARG), ("csa_kv8_attend", ATTEND, dict(out=F + 8), ALIGN),
    ("csa_kv8_attend", ATTEND, dict(acc=F + 2), ALIGN), ("csa_kv8_attend", ATTEND, dict(vc=F + 4), ALIGN),
    ("csa_kv8_attend", ATTEND, dict(acc=F, ws=None, ws_bytes=0), WORKSPACE),
    ("csa_kv8_attend", ATTEND, dict(acc=F, ws_bytes=16), WORKSPACE),
    ("csa_kv8_evict", EVICT, dict(B=0), SHAPE), ("csa_kv8_evict", EVICT, dict(recent=0), SHAPE),
    ("csa_kv8_evict", EVICT, dict(recent=4), SHAPE), ("csa_kv8_evict", EVICT, dict(keep=5), SHAPE),
    ("csa_kv8_evict", EVICT, dict(p=params(N=16 * 262145)), UNSUPPORTED),
    ("csa_kv8_evict", EVICT, dict(acc=None), ARG), ("csa_kv8_evict", EVICT, dict(kept=None), ARG),
    ("csa_kv8_evict", EVICT, dict(n_tok_out=None), ARG), ("csa_kv8_evict", EVICT, dict(kc=F + 1), ALIGN),
    ("csa_kv8_evict", EVICT, dict(acc_out=F + 2), ALIGN)])
def test_call_refusals(lib, name, good, ch, st):
    assert _call(lib, name, good, dict(dict(p=params()), **ch)) == st


def test_binding_rejects_host_tensors_and_unknown_names():
    x = torch.zeros(2, 8, 128)
    r = bd.rope_params(128, 64)
    with pytest.raises(ValueError, match="device tensor"):
        bd.csa_qk_norm_rope(r, torch.zeros(32), torch.zeros(2), x, None, x, None)
    with pytest.raises(KeyError):
        bd.rope_params(128, 64, layout="spiral")
    with pytest.raises(ValueError, match="act"):
        bd.kv8_params(8, 2, 64, 16, 64, "f16")
    dev = -1   # what a CPU tensor says its device index is
    for t, kw, msg in ((torch.zeros(2), dict(dtype=torch.int32), "int32"),
                       (torch.zeros(2), dict(shape=(3,)), "shape"),
                       (torch.zeros(4)[::2], dict(), "contiguous"),
                       (torch.zeros(2), dict(dev=0), "on cpu")):
        a = dict(dict(dtype=torch.float32, shape=(2,), what="x", dev=dev), **kw)
        with pytest.raises(ValueError, match=msg):
            bd._dense(t, **a)
    with pytest.raises(ValueError, match="contiguous"):
        bd._token_stride(torch.zeros(2, 8, 128)[:, ::2], torch.float32, "q", dev)
    assert bd._token_stride(torch.zeros(3, 12, 128)[:, 2:10], torch.float32, "q", dev) == 1536
