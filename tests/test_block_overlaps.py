"""Outputs that share memory with what another block of the same call still reads are refused on the host
(no GPU needed: nothing is launched, every address below is made up).  In place is what the header names."""
import pytest

from test_block_refusals import BF16, F32, INVALID, OK, lib  # noqa: F401

A = 1 << 20  # addresses this far apart never meet


def at(n, shift=0):
    return (n + 1) * A + shift


def refused(lib, code):  # noqa: F811
    """A refusal that names the overlap; without one the call would go on to the device."""
    return code == INVALID and b"overlap" in lib.kda_last_error()


def conv(lib, n=0, **kw):  # noqa: F811
    a = dict(x=at(0), dt=BF16, w=at(1), b=at(2), act=2, W=4, s0=at(3), s1=at(4), cu=at(5) if n else None, n=n,
             B=1 if n else 2, T=32, D=64, y=at(6))
    a.update(kw)
    return lib.kda_short_conv_fwd(*a.values(), None)


STATE = 2 * 3 * 64 * 2  # bytes of the convolution's states above


@pytest.mark.parametrize("n", [0, 2])
@pytest.mark.parametrize("kw", [
    dict(y=at(0)), dict(y=at(0, 16)), dict(y=at(0, -16)), dict(y=at(1)), dict(y=at(2, 64)), dict(y=at(3)), dict(y=at(4)),
    dict(s1=at(3, 16)), dict(s1=at(3, STATE - 16)), dict(s1=at(0)), dict(s1=at(1)), dict(s1=at(0, 4096 - 16))])
def test_conv(lib, n, kw):  # noqa: F811
    assert refused(lib, conv(lib, n, **kw))


def test_conv_output_on_the_offsets(lib):  # noqa: F811
    assert refused(lib, conv(lib, 2, y=at(5)))
    assert refused(lib, conv(lib, 2, s1=at(5)))


def decay(lib, chunk, **kw):  # noqa: F811
    a = dict(q=at(0), k=at(1), v=at(2), dt=BF16, decay=at(3), per_token=1, h0=at(4), hT=at(5), cu=None, n=0, B=2, T=100,
             H=4, Hk=2, K=64, V=64, o=at(6), odt=BF16)
    tail = dict(ws=at(60), size=1 << 30, status=at(7))
    tail.update({x: kw.pop(x) for x in list(kw) if x in tail})
    a.update(kw)
    if chunk:
        return lib.kda_decay_chunk_fwd(*a.values(), *tail.values(), None)
    return lib.kda_decay_recurrent_fwd(*a.values(), None)


@pytest.mark.parametrize("chunk", [False, True])
@pytest.mark.parametrize("kw", [
    dict(o=at(0)), dict(o=at(1)), dict(o=at(2, 16)), dict(o=at(3)), dict(o=at(4)), dict(o=at(5)), dict(o=at(2), odt=F32),
    dict(hT=at(0)), dict(hT=at(1)), dict(hT=at(2)), dict(hT=at(3)), dict(hT=at(4, 16)), dict(hT=at(4, -16))])
def test_decayed_attention(lib, chunk, kw):  # noqa: F811
    assert refused(lib, decay(lib, chunk, **kw))


@pytest.mark.parametrize("kw", [
    dict(y=at(0, 16)), dict(y=at(1, 16)), dict(y=at(1, -16)), dict(y=at(2))])
def test_gated_norm(lib, kw):  # noqa: F811
    a = dict(x=at(0), z=at(1), dt=BF16, w=at(2), eps=1e-6, act=1, rows=4, V=128, y=at(3))
    a.update(kw)
    assert refused(lib, lib.kda_gated_norm_fwd(*a.values(), None))


@pytest.mark.parametrize("kw", [
    dict(h=at(0)), dict(h=at(1, 16)), dict(h=at(2)), dict(h=at(3)), dict(h=at(4)), dict(h=at(5)), dict(h=at(6)),
    dict(y=at(0, 16)), dict(y=at(1)), dict(y=at(2)), dict(y=at(3, 32)), dict(y=at(4)), dict(y=at(5)), dict(y=at(6, 64)),
    dict(y=at(6, 2032))])
def test_block_norm(lib, kw):  # noqa: F811
    """x, gate and y in bf16, the stream in float32: h on x, or y on the stream, would not meet element by element."""
    a = dict(x=at(0), dt=BF16, r=at(1), rdt=F32, wp=at(2), z=at(3), act=1, scale=1.0, c=at(4), wn=at(5), eps=1e-6, rows=4,
             D=128, h=at(6), y=at(7))
    if "h" in kw and kw["h"] == at(6):
        kw = dict(y=at(6))
    a.update(kw)
    assert refused(lib, lib.kda_block_norm_fwd(*a.values(), None))


def test_nothing_to_do_overlaps_nothing(lib):  # noqa: F811
    assert conv(lib, B=0, y=at(0)) == OK
    assert conv(lib, T=0, y=at(0), s1=None) == OK
    assert decay(lib, True, B=0, o=at(0)) == OK


@pytest.mark.parametrize("chunk", [False, True])
def test_alignment_of_the_decays(lib, chunk):  # noqa: F811
    for shift in (1, 2, 3, 5):
        assert decay(lib, chunk, decay=at(3, shift)) == INVALID and b"aligned" in lib.kda_last_error()
