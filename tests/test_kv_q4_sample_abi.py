"""The 4-bit cache and sampling entries check their arguments on the host: every
call here returns before any device work (pointers are never dereferenced)."""
import ctypes

import pytest

from quantized_transformer_decode_gb300 import qw3

OK, ARG, SHAPE, OVERFLOW = 0, 1, 2, 4


@pytest.fixture(scope="module")
def L():
    from quantized_transformer_decode_gb300 import build
    build.build()
    return qw3.lib()


def cache(data=256, slots=2, capacity=64, n_kv_heads=2, head_dim=64):
    return qw3.Qw3KvQ4(data, slots, capacity, n_kv_heads, head_dim)


def test_struct_layout():
    assert ctypes.sizeof(qw3.Qw3KvQ4) == ctypes.sizeof(ctypes.c_void_p) + 16
    assert qw3.Qw3KvQ4.slots.offset == ctypes.sizeof(ctypes.c_void_p)


def test_cache_bytes(L):
    b = L.qw3_kv_q4_bytes
    assert b(1, 32, 1, 64) == 2 * 32 * (32 + 4)
    assert b(3, 8320, 8, 128) == 3 * 2 * 8 * 8320 * 72
    assert b(1, 1 << 26, 64, 128) == 2 * 64 * (1 << 26) * 72         # past 32 bits
    for bad in ((0, 32, 1, 64), (1, 0, 1, 64), (1, 33, 1, 64), (1, 32, 0, 64), (1, 32, 65, 64), (1, 32, 1, 96),
                (1, -32, 1, 64), (2147483647, 2147483616, 64, 128)):
        assert b(*bad) == -1, bad


def test_the_longest_capacity(L):
    """Positions are counted in 31 bits, with room for the last step past the end."""
    assert L.qw3_kv_q4_bytes(1, 1 << 30, 1, 64) == 2 * (1 << 30) * 36
    assert L.qw3_kv_q4_bytes(1, (1 << 30) + 32, 1, 64) == -1 and L.qw3_kv_q4_bytes(1, 2147483616, 1, 64) == -1
    c = cache(capacity=2147483616, slots=1, n_kv_heads=1)
    assert append(L, c) == SHAPE and L.qw3_kv_q4_read(c, 1, 16, 0, 16, 0, 16, 16, None) == SHAPE
    assert L.qw3_kv_q4_attn(c, 16, 256, 1, None, 16, 1, 1, 2147483616, 0.1, 16, 256, 16, 1 << 40, None, None) == SHAPE


APPEND = dict(qkv=16, M=4, stride=512, nh=4, qn=16, kn=16, eps=1e-6, rope=16, slots=16, slot0=0, pos=16, pos0=0,
              out=16, ostride=256, status=None)


def append(L, c, **kw):
    a = {**APPEND, **kw}
    return L.qw3_kv_q4_append(c, a["qkv"], a["M"], a["stride"], a["nh"], a["qn"], a["kn"], a["eps"], a["rope"],
                              a["slots"], a["slot0"], a["pos"], a["pos0"], a["out"], a["ostride"], a["status"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(M=-1), ARG), (dict(qkv=None), ARG), (dict(out=None), ARG), (dict(qn=None), ARG), (dict(kn=None), ARG),
    (dict(rope=None), ARG), (dict(rope=20), ARG), (dict(qkv=18), ARG), (dict(slots=17), ARG), (dict(pos=18), ARG),
    (dict(status=2), ARG), (dict(eps=-1.0), ARG), (dict(eps=float("nan")), ARG), (dict(stride=511), SHAPE),
    (dict(ostride=255), SHAPE), (dict(nh=5), SHAPE), (dict(nh=34), SHAPE), (dict(nh=0), SHAPE),
    (dict(slots=None, slot0=2), ARG), (dict(slots=None, slot0=-1), ARG), (dict(pos=None, pos0=-1), ARG),
    (dict(pos=None, pos0=61), OVERFLOW), (dict(M=0, qkv=None, out=None), OK),
])
def test_append_refusals(L, kw, want):
    assert append(L, cache(), **kw) == want
    if want != OK:
        assert qw3.qw3_last_error(0)


@pytest.mark.parametrize("c,want", [
    (dict(data=None), ARG), (dict(data=264), ARG), (dict(slots=0), SHAPE), (dict(capacity=48), SHAPE),
    (dict(n_kv_heads=65), SHAPE), (dict(head_dim=32), SHAPE),
])
def test_every_entry_checks_the_cache(L, c, want):
    c = cache(**c)
    assert append(L, c) == want
    assert L.qw3_kv_q4_read(c, 1, 16, 0, 16, 0, 16, 16, None) == want
    assert L.qw3_kv_q4_attn(c, 16, 256, 4, None, 16, 1, 1, 32, 0.1, 16, 256, 16, 1 << 30, None, None) == want


def test_null_cache(L):
    assert L.qw3_kv_q4_read(None, 1, 16, 0, 16, 0, 16, 16, None) == ARG


@pytest.mark.parametrize("args,want", [
    ((-1, 16, 0, 16, 0, 16, 16), ARG), ((1, 16, 0, 16, 0, None, 16), ARG), ((1, 16, 0, 16, 0, 16, None), ARG),
    ((1, 16, 0, 16, 0, 18, 16), ARG), ((1, None, 5, 16, 0, 16, 16), ARG), ((2, 16, 0, None, 63, 16, 16), OVERFLOW),
    ((2147483647, 16, 0, None, 2147483647, 16, 16), OVERFLOW), ((0, None, 0, None, 0, None, None), OK),
])
def test_read_refusals(L, args, want):
    assert L.qw3_kv_q4_read(cache(), *args, None) == want


def attn(L, **kw):
    a = {**dict(q=16, qs=256, nh=4, slots=16, lens=16, B=2, rows=1, max_len=64, scale=0.1, out=16, os=256, ws=16,
                wb=1 << 30, status=None), **kw}
    return L.qw3_kv_q4_attn(cache(), a["q"], a["qs"], a["nh"], a["slots"], a["lens"], a["B"], a["rows"], a["max_len"],
                            a["scale"], a["out"], a["os"], a["ws"], a["wb"], a["status"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), ARG), (dict(lens=None), ARG), (dict(out=None), ARG), (dict(q=18), ARG), (dict(out=18), ARG),
    (dict(lens=18), ARG), (dict(slots=18), ARG), (dict(ws=24), ARG), (dict(status=18), ARG), (dict(qs=255), SHAPE), (dict(os=255), SHAPE),
    (dict(rows=0), ARG), (dict(rows=17), ARG), (dict(B=-1), ARG), (dict(max_len=-1), ARG), (dict(max_len=65), OVERFLOW),
    (dict(nh=3), SHAPE), (dict(nh=34), SHAPE), (dict(scale=float("inf")), ARG), (dict(scale=float("nan")), ARG),
    (dict(B=0, q=None, lens=None, out=None, ws=None, wb=0), OK),
])
def test_attention_refusals(L, kw, want):
    assert attn(L, **kw) == want


def test_attention_workspace(L):
    w = L.qw3_kv_q4_attn_workspace_bytes
    assert w(1, 1, 16, 8, 128, 0) >= 0 and w(0, 1, 16, 8, 128, 8192) >= 0
    for bad in ((-1, 1, 16, 8, 128, 64), (1, 0, 16, 8, 128, 64), (1, 17, 16, 8, 128, 64), (1, 1, 12, 8, 128, 64),
                (1, 1, 16, 8, 96, 64), (1, 1, 16, 8, 128, -1), (1, 1, 136, 8, 128, 64), (1, 1, 16, 0, 128, 64)):
        assert w(*bad) == -1, bad
    need = w(1, 1, 32, 8, 128, 8192)
    if need:
        c = cache(slots=1, capacity=8192, n_kv_heads=8, head_dim=128)
        call = lambda ws, n: L.qw3_kv_q4_attn(c, 16, 4096, 32, None, 16, 1, 1, 8192, 0.1, 16, 4096, ws, n, None, None)  # noqa: E731
        assert call(None, need) == ARG and call(16, need - 1) == ARG


@pytest.mark.parametrize("kw,want", [
    (dict(logits=None), ARG), (dict(u=None), ARG), (dict(token=None), ARG), (dict(B=-1), ARG), (dict(V=0), SHAPE),
    (dict(V=4194305, stride=4194305), SHAPE), (dict(stride=99), SHAPE), (dict(logits=18), ARG), (dict(temp=18), ARG),
    (dict(k=18), ARG), (dict(p=18), ARG), (dict(mp=18), ARG), (dict(u=18), ARG), (dict(token=18), ARG),
    (dict(prob=18), ARG), (dict(status=18), ARG), (dict(B=0, logits=None, u=None, token=None), OK),
])
def test_sample_refusals(L, kw, want):
    a = {**dict(logits=16, stride=100, B=2, V=100, temp=16, k=16, p=16, mp=16, u=16, token=16, prob=16, status=16), **kw}
    assert L.qw3_sample(a["logits"], a["stride"], a["B"], a["V"], a["temp"], a["k"], a["p"], a["mp"], a["u"],
                        a["token"], a["prob"], a["status"], None) == want


def test_sample_takes_up_to_two_to_the_thirty_rows(L):
    for B in ((1 << 30) + 1, 2147483647):
        assert L.qw3_sample(16, 100, B, 100, None, None, None, None, 16, 16, None, None, None) == SHAPE


def test_wrappers_check_before_they_allocate():
    with pytest.raises(qw3.Qw3Error) as e:
        qw3.KVCacheQ4(1, 33, 1, 64)
    assert e.value.status == SHAPE


def test_sizes_past_31_bits_are_refused():
    """ctypes would pass them on modulo 2^32."""
    import torch
    for sizes in ((2 ** 32 + 1, 32, 1, 64), (1 - 2 ** 32, 32, 1, 64), (1, 2 ** 32 + 32, 1, 64), (1, 32, 2 ** 32 + 1, 64), (1, 32, 1, 2 ** 32 + 64)):
        with pytest.raises(qw3.Qw3Error) as e:
            qw3.KVCacheQ4(*sizes)
        assert e.value.status == SHAPE
    for shape in ((1, 2 ** 32 + 5), (2 ** 32 + 1, 8)):
        with pytest.raises(qw3.Qw3Error) as e:
            qw3._rows_of(torch.empty(shape, device="meta"), "logits")
        assert e.value.status == SHAPE


def test_a_cache_lies_on_a_gpu():
    """A cache in host memory is refused where it is made, not by its calls."""
    for kw in (dict(device="cpu"), dict(device="meta")):
        with pytest.raises(qw3.Qw3Error) as e:
            qw3.KVCacheQ4(1, 32, 1, 64, **kw)
        assert e.value.status == ARG


@pytest.mark.parametrize("kw", [dict(first=[1, 2]), dict(u=True), dict(temperature=True), dict(seqs=[0]), dict(seqs=[0, 1, 0])])
def test_sampled_generation_takes_tensors_of_its_device(monkeypatch, kw):
    """A host pointer, or a list of another length than the batch, never reaches the
    library."""
    import types

    import torch
    m = object.__new__(qw3.Qw3Model)
    m.h, m.shape, m.stream = None, types.SimpleNamespace(vocab=8), types.SimpleNamespace(device=torch.device("cuda", 0))

    class Gpu(torch.Tensor):
        """A host tensor that says it lies on cuda:0."""
        def get_device(self):
            return 0

        @property
        def device(self):
            return torch.device("cuda", 0)

    def reached(*a, **k):
        raise AssertionError("the library was called")

    monkeypatch.setattr(qw3, "qw3_generate_sample", reached)
    monkeypatch.setattr(qw3, "_Ordered", reached)
    # what is allocated once the checks have passed
    monkeypatch.setattr(torch, "empty", reached)
    g = lambda x, d=torch.float32: torch.tensor(x, dtype=d).as_subclass(Gpu)  # noqa: E731
    args = dict(first_tokens=g([1, 2], torch.int32), n_steps=3, u=g([[0.5, 0.5]] * 3), temperature=g([1.0, 1.0]))
    with pytest.raises(AssertionError):                       # the arguments themselves are good
        m.generate_sample(**args)
    host = {"first": dict(first_tokens=torch.tensor([1, 2], dtype=torch.int32), u=torch.full((3, 2), 0.5), temperature=torch.ones(2)),
            "u": dict(u=torch.full((3, 2), 0.5)), "temperature": dict(temperature=torch.ones(2)), "seqs": dict(seqs=kw.get("seqs"))}
    with pytest.raises(qw3.Qw3Error):
        m.generate_sample(**{**args, **host[next(iter(kw))]})
