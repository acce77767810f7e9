"""Host side of the embeddings' entry points: sizes, and the refusals that come back before any CUDA call."""
import pytest

P = 0x10000  # an aligned address that is never touched


@pytest.fixture(scope="module")
def c3():
    from concurrent_communication_overlap_gb300 import build
    build.build()
    from concurrent_communication_overlap_gb300 import c3 as mod
    return mod


def test_workspace_sizes(c3):
    size = c3.c3_embed_backward_bytes
    assert size(-1, 8, 8) == size(8, -1, 8) == size(8, 8, -1) == 0
    assert size(1 << 31, 8, 8) == size(8, 1 << 31, 8) == size(8, 8, 1 << 31) == 0
    assert 0 < size(0, 8, 8) <= size(1, 8, 8) <= size(4096, 8, 8) <= size(4096, 8, 4096)
    # the sorted pairs, twice
    assert size(65536, 131072, 8192) >= 2 * 8 * 65536
    # partial sums stay a fraction of what they are sums of
    assert size(1 << 20, 131072, 4096) < (1 << 20) * 4096


def test_lookup_refusals(c3):
    def f(table=P, type=0, rows=8, cols=4, ids=P, tokens=2, out=P, ot=0, **kw):
        return c3.c3_embed(table, type, rows, cols, ids, tokens, out, ot, check=False, **kw)
    for kw in (dict(type=2), dict(ot=-1), dict(rows=-1), dict(cols=-1), dict(tokens=-1), dict(first=-1), dict(ld=3),
               dict(out_ld=3), dict(table=None), dict(ids=None), dict(out=None), dict(scale=float("nan")),
               dict(scale=float("inf"))):
        assert f(**kw) == c3.C3_EINVAL, kw
        assert c3.c3_last_error()
    for kw in (dict(rows=1 << 31), dict(tokens=1 << 31), dict(cols=1 << 31, ld=1 << 31, out_ld=1 << 31), dict(first=1 << 31)):
        assert f(**kw) == c3.C3_EUNSUP, kw
    for kw in (dict(table=P + 2), dict(out=P + 2), dict(ids=P + 2), dict(table=P + 1, type=1), dict(out=P + 1, ot=1)):
        assert f(**kw) == c3.C3_EALIGN, kw
    assert f(tokens=0, ids=None, out=None) == c3.C3_OK
    assert f(cols=0, out=None) == c3.C3_OK


def test_gradient_refusals(c3):
    def f(dout=P, dt=0, ids=P, tokens=2, table=P, type=0, rows=8, cols=4, work=P, nbytes=1 << 20, **kw):
        return c3.c3_embed_backward(dout, dt, ids, tokens, table, type, rows, cols, work, work_bytes=nbytes, check=False, **kw)
    need = c3.c3_embed_backward_bytes(2, 8, 4)
    for kw in (dict(type=2), dict(dt=-1), dict(rows=-1), dict(cols=-1), dict(tokens=-1), dict(first=-1), dict(ld=3),
               dict(dout_ld=3), dict(dout=None), dict(ids=None), dict(table=None), dict(work=None), dict(nbytes=need - 1),
               dict(accumulate=2), dict(scale=float("nan"))):
        assert f(**kw) == c3.C3_EINVAL, kw
    for kw in (dict(rows=1 << 31), dict(tokens=1 << 31), dict(first=1 << 31)):
        assert f(**kw) == c3.C3_EUNSUP, kw
    for kw in (dict(table=P + 2), dict(dout=P + 2), dict(ids=P + 2), dict(work=P + 8), dict(table=P + 1, type=1)):
        assert f(**kw) == c3.C3_EALIGN, kw
    assert f(rows=0, table=None, work=None) == c3.C3_OK
    assert f(cols=0, table=None, work=None) == c3.C3_OK
    assert f(tokens=0, accumulate=True, table=None, work=None, ids=None, dout=None) == c3.C3_OK


def test_ids_of_another_type_or_with_gaps_are_refused(c3):
    """PyTorch's whole numbers are 64-bit unless told otherwise; read as int32 they would be twice as many ids."""
    torch = pytest.importorskip("torch")
    for ids in (torch.zeros(4, dtype=torch.int64), torch.zeros(4), torch.zeros(8, dtype=torch.int32)[::2],
                torch.zeros(4, dtype=torch.int16), torch.zeros(4, 2, dtype=torch.int32).T, torch.zeros(3, dtype=torch.int32)):
        with pytest.raises(c3.C3Error) as e:
            c3.c3_embed(P, 0, 8, 4, ids, 4, P, 0)
        assert e.value.status == c3.C3_EINVAL and "ids" in str(e.value)
        with pytest.raises(c3.C3Error) as e:
            c3.c3_embed_backward(P, 0, ids, 4, P, 0, 8, 4, P, work_bytes=1 << 20)
        assert e.value.status == c3.C3_EINVAL and "ids" in str(e.value)
    # what is given is looked at whether or not a call has anything to do with it
    assert c3.c3_embed(P, 0, 8, 0, torch.zeros(2, 2, dtype=torch.int32), 4, P, 0) == c3.C3_OK
