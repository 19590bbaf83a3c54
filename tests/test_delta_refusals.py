"""The gated delta rule's calls, and the norm and rotation of queries and keys, reject bad arguments on the host,
before any launch: no GPU is needed, every call below fails validation or has no device work."""
import pytest

OK, INVALID, UNSUPPORTED = 0, 1, 2
F32, BF16 = 0, 1
P = 1 << 32  # aligned addresses that are never read, far apart
STEP = 1 << 30
Q, K, V, G, BETA, A, DT, H0, HT, CU, O, WS = (P + i * STEP for i in range(12))


@pytest.fixture(scope="module")
def lib():
    from chunked_kda_gb300 import _build

    _build.build()
    import chunked_kda_gb300

    return chunked_kda_gb300.load_library()


def delta(lib, chunk=False, **kw):
    a = dict(q=Q, k=K, v=V, dt=BF16, g=G, gdt=F32, A=None, dtb=None, mode=0, beta=BETA, bdt=BF16, h0=None, hT=None, cu=None,
             n=0, B=1, T=8, H=4, Hk=0, K=64, V=64, o=O, odt=BF16, flags=0)
    tail = dict(ws=WS, size=1 << 40, status=None)
    tail.update({x: kw.pop(x) for x in list(kw) if x in tail})
    a.update(kw)
    if chunk:
        return lib.kda_delta_chunk_fwd(*a.values(), *tail.values(), None)
    return lib.kda_delta_recurrent_fwd(*a.values(), None)


@pytest.mark.parametrize("chunk", [False, True])
@pytest.mark.parametrize("kw,code", [
    (dict(K=0), UNSUPPORTED), (dict(K=257), UNSUPPORTED), (dict(V=0), UNSUPPORTED), (dict(V=300), UNSUPPORTED),
    (dict(dt=2), UNSUPPORTED), (dict(odt=2), UNSUPPORTED), (dict(dt=F32, odt=BF16, bdt=F32), UNSUPPORTED),
    (dict(gdt=2), UNSUPPORTED), (dict(bdt=2), UNSUPPORTED), (dict(dt=F32, odt=F32, bdt=BF16), UNSUPPORTED),
    (dict(mode=1), UNSUPPORTED), (dict(mode=3), UNSUPPORTED), (dict(mode=7), UNSUPPORTED), (dict(mode=2), INVALID),
    (dict(flags=8), INVALID), (dict(Hk=3), INVALID), (dict(Hk=-1), INVALID), (dict(H=0), INVALID), (dict(H=65536), INVALID),
    (dict(B=-1), INVALID), (dict(T=-1), INVALID), (dict(B=65536), INVALID), (dict(T=1 << 30, B=2), INVALID),
    (dict(cu=CU, n=2, B=2), INVALID), (dict(cu=CU, n=-1), INVALID), (dict(cu=CU, n=65536), INVALID),
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(g=None), INVALID),
    (dict(beta=None), INVALID), (dict(o=None), INVALID), (dict(v=V + 2), INVALID), (dict(h0=H0 + 4), INVALID),
    (dict(hT=HT + 8), INVALID), (dict(g=G + 2), INVALID), (dict(beta=BETA + 1), INVALID), (dict(mode=2, A=A + 2), INVALID),
    (dict(mode=2, A=A, dtb=DT + 1), INVALID),
    # outputs on inputs
    (dict(o=Q), INVALID), (dict(o=K + 64), INVALID), (dict(o=V + 512), INVALID), (dict(o=V, odt=F32), INVALID),
    (dict(o=G), INVALID), (dict(o=BETA), INVALID), (dict(o=H0, h0=H0), INVALID), (dict(o=HT, hT=HT), INVALID),
    (dict(mode=2, A=A, o=A), INVALID), (dict(mode=2, A=A, dtb=DT, hT=DT), INVALID), (dict(hT=V), INVALID),
    (dict(hT=H0 + 256, h0=H0), INVALID), (dict(cu=CU, n=2, hT=CU), INVALID), (dict(cu=CU, n=2, o=CU), INVALID),
])
def test_delta_refusals(lib, chunk, kw, code):
    assert delta(lib, chunk, **kw) == code
    assert lib.kda_last_error()


@pytest.mark.parametrize("chunk", [False, True])
def test_tokens_that_a_chunk_counts_past_32_bits(lib, chunk):
    # K = V = 8 and one head: such tensors fit the memory, a chunk's row numbers would not fit 32 bits
    far = dict(K=8, V=8, H=1, q=1 << 44, k=1 << 45, v=1 << 46, o=1 << 47, g=1 << 48, beta=1 << 49)
    assert delta(lib, chunk, T=(1 << 31) - 255, **far) == INVALID
    assert b"2^31 - 256" in lib.kda_last_error()
    assert delta(lib, chunk, T=(1 << 31) - 1, **far) == INVALID


def test_workspace_and_status_refusals(lib):
    big = dict(dt=F32, bdt=F32, odt=F32, T=200)
    need = lib.kda_delta_chunk_workspace_bytes(F32, F32, 1, 200, 4, 64, 64, 0)
    assert need > 0
    assert delta(lib, True, **big, ws=WS, size=need - 1) == INVALID
    assert delta(lib, True, **big, ws=None, size=0) == INVALID
    assert delta(lib, True, **big, ws=WS + 16) == INVALID
    assert delta(lib, True, **big, status=P + 2) == INVALID
    for bad in ((3, F32, 1, 8, 4, 64, 64, 0), (F32, 3, 1, 8, 4, 64, 64, 0), (F32, F32, -1, 8, 4, 64, 64, 0),
                (F32, F32, 1, 8, 0, 64, 64, 0), (F32, F32, 1, 8, 4, 0, 64, 0), (F32, F32, 1, 8, 4, 64, 300, 0)):
        assert lib.kda_delta_chunk_workspace_bytes(*bad) == 0


def test_scratch_does_not_grow_with_the_sequences(lib):
    one, many = (lib.kda_delta_chunk_workspace_bytes(F32, F32, 1, 4096, 32, 128, 128, n) for n in (1, 4096))
    assert one == many <= 4096 * 32 * 600


@pytest.mark.parametrize("chunk", [False, True])
def test_no_sequences_is_no_work(lib, chunk):
    assert delta(lib, chunk, B=0) == OK
    assert delta(lib, chunk, cu=CU, n=0) == OK


def qk(lib, **kw):
    a = dict(q=Q, qs=512, k=K, ks=128, dt=BF16, wq=None, wk=None, norm=1, eps=1e-6, pos=G, axes=1, freq=BETA, pair=None, R=64,
             inter=0, m=1.0, tokens=8, Hq=8, Hk=2, D=64, qo=O, qos=512, ko=H0, kos=128)
    a.update(kw)
    return lib.kda_qk_norm_rope_fwd(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(dt=2), UNSUPPORTED), (dict(D=0), UNSUPPORTED), (dict(D=257, qs=8 * 257, ks=8 * 257), UNSUPPORTED), (dict(norm=3), INVALID),
    (dict(norm=-1), INVALID), (dict(eps=-1e-6), INVALID), (dict(eps=float("nan")), INVALID), (dict(R=66), INVALID),
    (dict(R=-2), INVALID), (dict(R=63), INVALID), (dict(Hq=0), INVALID), (dict(Hk=-1), INVALID), (dict(Hq=4096), INVALID),
    (dict(tokens=-1), INVALID), (dict(tokens=1 << 31), INVALID), (dict(axes=0), INVALID), (dict(axes=5), INVALID),
    (dict(pair=bytes([1] * 32)), INVALID), (dict(axes=3, pair=bytes([3] * 32)), INVALID), (dict(q=None), INVALID),
    (dict(k=None), INVALID), (dict(qo=None), INVALID), (dict(ko=None), INVALID), (dict(pos=None), INVALID),
    (dict(freq=None), INVALID), (dict(qs=511), INVALID), (dict(ks=0), INVALID), (dict(qos=64), INVALID), (dict(kos=-128), INVALID),
    (dict(qs=1 << 41), INVALID), (dict(q=Q + 1), INVALID), (dict(ko=H0 + 1), INVALID), (dict(pos=G + 2), INVALID),
    (dict(freq=BETA + 1), INVALID), (dict(wq=A + 2), INVALID), (dict(wk=A + 1), INVALID),
    (dict(qo=H0), INVALID), (dict(qo=Q + 128), INVALID), (dict(qo=Q, qos=640), INVALID), (dict(qo=K), INVALID), (dict(ko=Q), INVALID),
    (dict(qo=G), INVALID), (dict(ko=BETA), INVALID), (dict(wq=A, qo=A), INVALID), (dict(wk=A, ko=A), INVALID),
    # parts of the same rows that share elements
    (dict(qs=768, ks=768, k=Q + 1024, qo=Q + 1024, qos=768), INVALID),
    (dict(qos=768, ko=O + 896, kos=768), INVALID),
])
def test_qk_refusals(lib, kw, code):
    assert qk(lib, **kw) == code
    assert lib.kda_last_error()


def test_qk_without_tokens_is_no_work(lib):
    assert qk(lib, tokens=0) == OK
