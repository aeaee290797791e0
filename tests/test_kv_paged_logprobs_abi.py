"""The paged cache and log-probability entries check their arguments on the host:
every call here returns before any device work (pointers are never
dereferenced)."""
import ctypes

import pytest

from quantized_transformer_decode_gb300 import qw3

OK, ARG, SHAPE, OVERFLOW = 0, 1, 2, 4


@pytest.fixture(scope="module")
def L():
    from quantized_transformer_decode_gb300 import build
    build.build()
    return qw3.lib()


def cache(data=256, n_pages=10, page_size=16, n_kv_heads=2, head_dim=64):
    return qw3.Qw3KvPaged(data, n_pages, page_size, n_kv_heads, head_dim)


def batch(starts=16, lens=16, table=16, stride=4, B=2, pages=4):
    return qw3.Qw3KvBatch(starts, lens, table, stride, B, pages)


def test_struct_layouts():
    p = ctypes.sizeof(ctypes.c_void_p)
    assert ctypes.sizeof(qw3.Qw3KvPaged) == p + 16 and qw3.Qw3KvPaged.n_pages.offset == p
    assert ctypes.sizeof(qw3.Qw3KvBatch) == 3 * p + 16 and qw3.Qw3KvBatch.table_stride.offset == 3 * p


def test_pool_bytes(L):
    f = L.qw3_kv_paged_bytes
    assert f(1, 16, 1, 64) == 2 * 16 * 64 * 2 and f(20000, 64, 8, 128) == 20000 * 2 * 8 * 64 * 128 * 2
    for bad in ((0, 16, 1, 64), (1, 8, 1, 64), (1, 24, 1, 64), (1, 512, 1, 64), (1, 16, 0, 64), (1, 16, 65, 64),
                (1, 16, 1, 80), (-1, 16, 1, 64), (2147483647, 16, 1, 64), (65536, 256, 64, 128)):
        assert f(*bad) == -1, bad
    assert f(65535, 256, 64, 128) == 65535 * 2 * 64 * 256 * 256


APPEND = dict(type=0, qkv=16, M=4, stride=512, nh=4, qn=16, kn=16, eps=1e-6, rope=16, rope_len=64, out=16, ostride=256, status=None)


def append(L, c, b, **kw):
    a = {**APPEND, **kw}
    return L.qw3_kv_paged_append(c, b, a["type"], a["qkv"], a["M"], a["stride"], a["nh"], a["qn"], a["kn"], a["eps"],
                                 a["rope"], a["rope_len"], a["out"], a["ostride"], a["status"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(type=2), ARG), (dict(type=-1), ARG), (dict(qkv=None), ARG), (dict(qkv=8), ARG), (dict(M=-1), ARG),
    (dict(stride=508), SHAPE), (dict(stride=514), ARG), (dict(type=1, stride=516), ARG), (dict(nh=3), SHAPE), (dict(nh=0), SHAPE),
    (dict(nh=34), SHAPE), (dict(qn=18), ARG), (dict(kn=17), ARG), (dict(eps=-1.0), ARG), (dict(eps=float("nan")), ARG),
    (dict(rope=None), ARG), (dict(rope=24), ARG), (dict(rope_len=0), ARG), (dict(out=None), ARG), (dict(out=20), ARG),
    (dict(ostride=252), SHAPE), (dict(ostride=258), ARG), (dict(status=2), ARG), (dict(M=2 ** 30), SHAPE),
])
def test_append_refusals(L, kw, want):
    assert append(L, cache(), batch(), **kw) == want
    assert qw3.qw3_last_error()


BAD_BATCHES = [
    (dict(starts=None), ARG), (dict(lens=None), ARG), (dict(table=None), ARG), (dict(starts=18), ARG), (dict(lens=17), ARG),
    (dict(table=18), ARG), (dict(stride=3), SHAPE), (dict(B=-1), ARG), (dict(pages=-1), ARG), (dict(B=2 ** 20 + 1), SHAPE),
    (dict(pages=2 ** 27, stride=2 ** 27), SHAPE),
]


@pytest.mark.parametrize("kw,want", BAD_BATCHES)
def test_batch_refusals(L, kw, want):
    assert append(L, cache(), batch(**kw)) == want
    assert attn(L, cache(), batch(**kw)) == want


@pytest.mark.parametrize("kw,want", [
    (dict(data=None), ARG), (dict(data=264), ARG), (dict(n_pages=0), SHAPE), (dict(page_size=48), SHAPE),
    (dict(n_kv_heads=0), SHAPE), (dict(head_dim=32), SHAPE),
])
def test_cache_refusals(L, kw, want):
    assert append(L, cache(**kw), batch()) == want
    assert attn(L, cache(**kw), batch()) == want
    assert append(L, None, batch()) == ARG and attn(L, cache(), None) == ARG


ATTN = dict(type=0, q=16, M=4, stride=256, nh=4, max_rows=4, max_len=64, window=0, sinks=0, scale=0.125, out=16, ostride=256,
            ws=16, ws_bytes=1 << 40, status=None)


def attn(L, c, b, **kw):
    a = {**ATTN, **kw}
    return L.qw3_kv_paged_attn(c, b, a["type"], a["q"], a["M"], a["stride"], a["nh"], a["max_rows"], a["max_len"], a["window"],
                               a["sinks"], a["scale"], a["out"], a["ostride"], a["ws"], a["ws_bytes"], a["status"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(type=5), ARG), (dict(q=None), ARG), (dict(q=8), ARG), (dict(out=None), ARG), (dict(out=4), ARG), (dict(M=-1), ARG),
    (dict(stride=252), SHAPE), (dict(stride=258), ARG), (dict(ostride=255), SHAPE), (dict(type=1, ostride=260), ARG),
    (dict(stride=260), SHAPE), (dict(ostride=260), SHAPE), (dict(type=1, stride=264), SHAPE),  # not whole heads
    (dict(nh=5), SHAPE), (dict(max_rows=5), ARG), (dict(max_rows=-1), ARG), (dict(max_len=65), OVERFLOW), (dict(max_len=-1), ARG),
    (dict(window=-1), ARG), (dict(sinks=-2), ARG), (dict(scale=float("inf")), ARG), (dict(scale=float("nan")), ARG),
    (dict(ws=8), ARG), (dict(status=6), ARG), (dict(M=2 ** 30, max_rows=1), SHAPE),
])
def test_attention_refusals(L, kw, want):
    assert attn(L, cache(), batch(), **kw) == want
    assert qw3.qw3_last_error()


def test_workspace(L):
    f = L.qw3_kv_paged_attn_workspace_bytes
    assert f(0, 0, 0, 4, 2, 64, 0, 0, 0, 0) >= 0 and f(64, 64, 1, 32, 8, 128, 1, 32768, 0, 0) >= 0
    for bad in ((-1, 4, 0, 4, 2, 64, 4, 64, 0, 0), (1, -4, 0, 4, 2, 64, 4, 64, 0, 0), (1, 4, 2, 4, 2, 64, 4, 64, 0, 0),
                (1, 4, 0, 3, 2, 64, 4, 64, 0, 0), (1, 4, 0, 34, 2, 64, 4, 64, 0, 0), (1, 4, 0, 4, 2, 96, 4, 64, 0, 0),
                (1, 4, 0, 4, 2, 64, 5, 64, 0, 0), (1, 4, 0, 4, 2, 64, 4, -1, 0, 0), (1, 4, 0, 4, 2, 64, 4, 64, -1, 0),
                (1, 4, 0, 4, 2, 64, 4, 64, 0, -1), (2 ** 20 + 1, 4, 0, 4, 2, 64, 4, 64, 0, 0)):
        assert f(*bad) == -1, bad
    for big in ((1, 4096, 1, 32, 8, 128, 4096, 8192, 0, 0), (2 ** 20, 2 ** 20, 0, 16, 8, 128, 1, 2 ** 30, 0, 0)):
        assert 0 <= f(*big) < 1 << 40


def test_nothing_to_do(L):
    assert append(L, cache(), batch(), M=0, qkv=None, out=None) == OK
    assert append(L, cache(), batch(B=0, starts=None, lens=None, table=None)) == OK
    assert attn(L, cache(), batch(), M=0, q=None, out=None, max_rows=0) == OK
    assert attn(L, cache(), batch(), max_rows=0) == OK
    assert attn(L, cache(), batch(B=0, starts=None, lens=None, table=None, pages=0), max_len=0) == OK


LP = dict(x=16, stride=100, B=3, V=100, tokens=16, T=2, top=5, lp=16, h=16, ids=16, alts=16, status=None)


def logprobs(L, **kw):
    a = {**LP, **kw}
    return L.qw3_logprobs(a["x"], a["stride"], a["B"], a["V"], a["tokens"], a["T"], a["top"], a["lp"], a["h"], a["ids"],
                          a["alts"], a["status"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(x=None), ARG), (dict(B=-1), ARG), (dict(T=-1), ARG), (dict(top=-1), ARG), (dict(tokens=None), ARG),
    (dict(lp=None), ARG), (dict(ids=None), ARG), (dict(alts=None), ARG), (dict(x=18), ARG), (dict(tokens=17), ARG),
    (dict(lp=18), ARG), (dict(h=18), ARG), (dict(ids=18), ARG), (dict(alts=18), ARG), (dict(status=2), ARG),
    (dict(V=0), SHAPE), (dict(V=101), SHAPE), (dict(V=4194305, stride=4194305), SHAPE), (dict(top=65), SHAPE),
    (dict(B=2 ** 30 + 1), SHAPE),
])
def test_logprob_refusals(L, kw, want):
    assert logprobs(L, **kw) == want
    assert qw3.qw3_last_error()


def test_logprobs_of_no_rows(L):
    assert logprobs(L, B=0, x=None, tokens=None, lp=None, ids=None, alts=None) == OK


def test_workspaces_go_by_the_device(monkeypatch):
    """A call's workspace has the size that its own device asks for, whatever another one asked for before."""
    torch = pytest.importorskip("torch")
    needs, got, current = {0: 4096, 1: 8192}, [], [0]

    class Lib:      # a library that sees two devices
        def qw3_kv_paged_attn_workspace_bytes(self, *sizes):
            return needs[current[0]]

        def qw3_kv_paged_attn(self, *args):
            got.append((args[14], args[15]))
            return OK

    class On(torch.Tensor):      # host tensors that say they lie on the current device
        def get_device(self):
            return current[0]

    monkeypatch.setattr(qw3, "lib", Lib)
    monkeypatch.setattr(qw3, "_elsewhere", lambda torch, index: False)
    monkeypatch.setattr(qw3, "_stream_on", lambda torch, index: 0)
    ints = lambda *v: torch.tensor(v, dtype=torch.int32).as_subclass(On)  # noqa: E731
    for device in (0, 1, 0):
        current[0] = device
        c = object.__new__(qw3.KVCachePaged)
        c.data, c.device, c.index = None, torch.device("cpu"), device
        c.n_pages, c.page_size, c.n_kv_heads, c.head_dim = 10, 16, 2, 64
        c.c = cache()
        c.attention(torch.zeros(3, 4, 64).as_subclass(On), ints(0, 3), ints(9), ints(1).view(1, 1))
        assert got[-1][0] and got[-1][1] == needs[device]


def test_no_rows_of_any_strides():
    """A tensor of no rows has no strides to keep to (numpy's come with others than torch's)."""
    torch = pytest.importorskip("torch")
    for t in (torch.empty(0, 8), torch.empty_strided((0, 8), (1, 0)), torch.empty_strided((0, 8), (0, 3))):
        rows, width, stride = qw3._rows_of(t, "t")
        assert (rows, width) == (0, 8) and stride >= 8
    with pytest.raises(qw3.Qw3Error):
        qw3._rows_of(torch.empty(4, 16)[:, ::2], "t")
