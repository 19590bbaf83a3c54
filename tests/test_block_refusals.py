"""The operators around the recurrence reject bad arguments on the host, before any launch: no GPU
is needed, every call below fails validation or has no device work."""
import ctypes

import pytest
import torch

OK, INVALID, UNSUPPORTED = 0, 1, 2
F32, BF16 = 0, 1
P = 256  # an aligned address that is never read


@pytest.fixture(scope="module")
def lib():
    from chunked_kda_gb300 import _build

    _build.build()
    import chunked_kda_gb300

    return chunked_kda_gb300.load_library()


def decay(lib, chunk=False, **kw):
    a = dict(q=P, k=P, v=P, dt=BF16, decay=P, per_token=1, h0=None, hT=None, cu=None, n=0, B=1, T=8, H=4, Hk=0, K=64,
             V=64, o=P, odt=BF16)
    tail = dict(ws=None, size=0, status=None)
    tail.update({x: kw.pop(x) for x in list(kw) if x in tail})
    a.update(kw)
    args = list(a.values())
    if chunk:
        return lib.kda_decay_chunk_fwd(*args, *tail.values(), None)
    return lib.kda_decay_recurrent_fwd(*args, None)


@pytest.mark.parametrize("chunk", [False, True])
@pytest.mark.parametrize("kw,code", [
    (dict(K=0), UNSUPPORTED), (dict(K=257), UNSUPPORTED), (dict(V=0), UNSUPPORTED), (dict(V=300), UNSUPPORTED),
    (dict(dt=2), UNSUPPORTED), (dict(odt=2), UNSUPPORTED), (dict(dt=F32, odt=BF16), UNSUPPORTED),
    (dict(Hk=3), INVALID), (dict(Hk=-1), INVALID), (dict(H=0), INVALID), (dict(H=65536), INVALID),
    (dict(B=-1), INVALID), (dict(T=-1), INVALID), (dict(B=65536), INVALID), (dict(T=1 << 30, B=2), INVALID),
    (dict(cu=P, n=2, B=2), INVALID), (dict(cu=P, n=-1), INVALID), (dict(cu=P, n=65536), INVALID),
    (dict(q=None), INVALID), (dict(decay=None), INVALID), (dict(o=None), INVALID), (dict(v=P + 2), INVALID),
    (dict(h0=P + 4), INVALID), (dict(hT=P + 8), INVALID),
])
def test_decay_refusals(lib, chunk, kw, code):
    assert decay(lib, chunk, **kw) == code
    assert lib.kda_last_error()


def test_decay_chunk_workspace_and_status_refusals(lib):
    assert decay(lib, True, status=P + 2) == INVALID
    assert decay(lib, True, ws=P + 16, size=1 << 40) == INVALID
    assert lib.kda_decay_chunk_workspace_bytes(3, 1, 8, 4, 64, 64, 0) == 0
    assert lib.kda_decay_chunk_workspace_bytes(BF16, 1, 8, 4, 64, 300, 0) == 0


@pytest.mark.parametrize("chunk", [False, True])
def test_decay_without_sequences_is_no_work(lib, chunk):
    assert decay(lib, chunk, B=0) == OK
    assert decay(lib, chunk, cu=P, n=0) == OK


@pytest.mark.parametrize("kw,code", [
    (dict(dt=3), UNSUPPORTED), (dict(act=7), INVALID), (dict(rows=-1), INVALID), (dict(rows=1 << 31), INVALID),
    (dict(V=0), INVALID), (dict(V=(1 << 20) + 1), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(x=None), INVALID), (dict(z=None), INVALID), (dict(y=None), INVALID), (dict(w=P + 4), INVALID),
    (dict(z=P + 2), INVALID), (dict(rows=0, x=None), OK)])
def test_gated_norm_refusals(lib, kw, code):
    a = dict(x=P, z=P, dt=BF16, w=P, eps=1e-6, act=1, rows=4, V=128, y=P)
    a.update(kw)
    assert lib.kda_gated_norm_fwd(*a.values(), None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dt=3), UNSUPPORTED), (dict(rdt=-1), UNSUPPORTED), (dict(act=-1), INVALID), (dict(rows=-1), INVALID),
    (dict(D=0), INVALID), (dict(eps=-1.0), INVALID), (dict(x=None), INVALID), (dict(h=None, y=None), INVALID),
    (dict(r=P + 8), INVALID), (dict(wn=P + 4), INVALID), (dict(c=P + 4), INVALID), (dict(rows=0, x=None), OK)])
def test_block_norm_refusals(lib, kw, code):
    a = dict(x=P, dt=BF16, r=P, rdt=F32, wp=P, z=P, act=1, scale=1.0, c=None, wn=P, eps=1e-6, rows=4, D=128, h=P, y=P)
    a.update(kw)
    assert lib.kda_block_norm_fwd(*a.values(), None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dt=3), UNSUPPORTED), (dict(act=3), INVALID), (dict(W=1), UNSUPPORTED), (dict(W=9), UNSUPPORTED),
    (dict(D=0), INVALID), (dict(T=-1), INVALID), (dict(cu=P, n=1, B=2), INVALID), (dict(x=None), INVALID),
    (dict(w=None), INVALID), (dict(y=None), INVALID), (dict(s0=P + 2), INVALID), (dict(s1=P + 2), INVALID),
    (dict(B=0), OK), (dict(T=0), OK)])
def test_short_conv_refusals(lib, kw, code):
    a = dict(x=P, dt=BF16, w=P, b=None, act=2, W=4, s0=None, s1=None, cu=None, n=0, B=1, T=8, D=64, y=P)
    a.update(kw)
    assert lib.kda_short_conv_fwd(*a.values(), None) == code


def test_the_binding_refuses_what_it_can_see():
    import chunked_kda_gb300 as kda

    q, v, a = torch.zeros(1, 8, 2, 64), torch.zeros(1, 8, 4, 64), torch.zeros(1, 8, 4)
    with pytest.raises(ValueError, match="CUDA"):
        kda.kda_decay_chunk_fwd(q, q, v, a)
    with pytest.raises(ValueError, match="CUDA"):
        kda.kda_gated_norm_fwd(v, v)
    with pytest.raises(ValueError, match="CUDA"):
        kda.kda_decay_recurrent_fwd(q, q, v, a)
    with pytest.raises(ValueError, match="CUDA"):
        kda.kda_block_norm_fwd(v)
    with pytest.raises(ValueError, match="CUDA"):
        kda.kda_short_conv_fwd(v[0], torch.zeros(64, 4))


def test_prototypes_match_the_header():
    """Every argument list in the binding has the header's number of arguments."""
    import os
    import re

    import chunked_kda_gb300 as kda

    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "kda.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    lib = kda.load_library()
    for name in ("kda_decay_chunk_workspace_bytes", "kda_decay_chunk_fwd", "kda_decay_recurrent_fwd",
                 "kda_gated_norm_fwd", "kda_block_norm_fwd", "kda_short_conv_fwd"):
        args = re.search(name + r"\s*\((.*?)\)\s*;", text, flags=re.S).group(1)
        fn = getattr(lib, name)
        assert len(fn.argtypes) == args.count(",") + 1, name
        for c, decl in zip(fn.argtypes, args.split(",")):
            want = (ctypes.c_void_p if "*" in decl or "kda_stream_t" in decl else ctypes.c_float if "float" in decl else
                    ctypes.c_size_t if "size_t" in decl else ctypes.c_int64 if "int64_t" in decl else ctypes.c_int)
            assert c is want, (name, decl)
