"""The paged KV cache entries against plain 64-bit arithmetic (paged_f64.py):
rows appended, attention over ragged batches, and both in a layer.

Tolerances. A value before its last rounding is within 20 f32 roundings (2^-24
each) of its row's largest normalised value: 9 for the sum of squares and its
root, 3 products, one sum, times sqrt 2. Its last rounding is half a step: 2^-11
of it in f16 (2^-25 where it is subnormal), 2^-24 in f32. Values of V are rounded
once: exactly numpy's. Attention: paged_f64.bound.
"""
import numpy as np
import pytest

import paged_f64 as ref

pytestmark = pytest.mark.gpu

EPS = 1e-6


@pytest.fixture(scope="module")
def torch():
    import torch as t
    if not t.cuda.is_available():
        pytest.skip("no CUDA device")
    from quantized_transformer_decode_gb300 import build
    build.build()
    return t


class Batch:
    """A pool, and sequences of (new rows, length) in pages taken in no order."""

    def __init__(self, torch, seqs, nkv=2, hd=64, page=16, dtype="f32", nh=4, seed=0, spare=3, lead=0, tail=0, extra=1):
        from quantized_transformer_decode_gb300 import qw3
        self.torch, self.rng = torch, np.random.default_rng(seed)
        self.nh, self.nkv, self.hd, self.page = nh, nkv, hd, page
        self.f16 = dtype == "f16"
        self.np_type, self.dtype = (np.float16, torch.float16) if self.f16 else (np.float32, torch.float32)
        rows, lens = [r for r, _ in seqs], [n for _, n in seqs]
        self.M = lead + sum(rows) + tail
        self.starts = np.concatenate(([0], np.cumsum(rows))).astype(np.int32) + lead
        self.lens = np.array(lens, np.int32)
        used = np.array([max(0, -(-n // page)) for n in lens], int)
        self.n_pages = int(used.sum()) + spare
        width = int(used.max()) + extra if len(used) else 1
        self.table = np.full((len(seqs), width), -1, np.int32)
        ids = self.rng.permutation(self.n_pages)[:int(used.sum())]
        self.table[np.arange(width) < used[:, None]] = ids
        gain = 1 + 0.5 * np.abs(self.rng.standard_normal((2, nkv, 1, hd)))
        self.data = (self.rng.standard_normal((self.n_pages, 2, nkv, page, hd)) * gain).astype(np.float16)
        # places behind a sequence's end hold anything
        for b, n in enumerate(lens):
            if n > 0 and n % page:
                self.data[self.table[b, n // page], :, :, n % page:] = self.rng.choice([np.nan, np.inf, -np.inf, 3.0])
        held = set(ids.tolist())
        for p in range(self.n_pages):
            if p not in held:
                self.data[p] = np.nan
        self.q = (self.rng.standard_normal((self.M, nh, hd)) * 1.5).astype(self.np_type)
        self.qkv = (self.rng.standard_normal((self.M, (nh + 2 * nkv) * hd)) * 0.8).astype(self.np_type)
        self.q_norm = (1 + 0.1 * self.rng.standard_normal(hd)).astype(np.float32)
        self.k_norm = (1 + 0.1 * self.rng.standard_normal(hd)).astype(np.float32)
        self.rope = ref.rope_table(max(1, max(lens, default=1)), hd)
        self.qw3 = qw3

    def dev(self, x):
        return self.torch.from_numpy(np.ascontiguousarray(x)).cuda()

    def cache(self):
        return self.qw3.KVCachePaged(self.n_pages, self.page, self.nkv, self.hd, data=self.dev(self.data))

    def where(self):
        return self.dev(self.starts), self.dev(self.lens), self.dev(self.table)

    def attend(self, cache=None, q=None, **kw):
        return (cache or self.cache()).attention(self.dev(self.q) if q is None else q, *self.where(), **kw)

    def check(self, got, **kw):
        want, err, written = ref.attend(self.q, self.data.astype(np.float64), self.starts, self.lens, self.table, **kw)
        got = got.cpu().numpy().astype(np.float64)
        lim = ref.bound(err, want, self.hd, self.f16)
        fine = np.isfinite(want)
        assert np.array_equal(np.isfinite(got[written]), fine[written])
        off = np.where(fine, np.abs(got - np.where(fine, want, 0)), 0)
        over = (off > lim) & written[:, None, None]
        assert not over.any(), (np.argwhere(over)[:4], off[over][:4], lim[over][:4], got[over][:4], want[over][:4])
        return want, written


# ---------------------------------------------------------------- append

def check_append(b, norm=True, positions=None, qkv=None, got=None, cache=None, status=0):
    """Every head of every row, the pages' other places bit for bit."""
    want = b.data.copy()
    nh, nkv, hd = b.nh, b.nkv, b.hd
    x = (b.qkv if qkv is None else qkv).reshape(b.M, nh + 2 * nkv, hd)
    data = cache.data.cpu().numpy()
    q = got.cpu().numpy().astype(np.float64)
    kerr = np.zeros(want.shape)
    exact = want.astype(np.float64)
    for row, (s, p, page) in enumerate(ref.places(b.starts, b.lens, b.table, b.page, b.n_pages, b.M)):
        if s < 0:
            continue
        if page < 0 or p >= len(b.rope):
            assert not q[row].any()
            continue
        n, y = ref.turned(x[row, :nh], b.q_norm if norm else None, b.rope[p], EPS)
        lim = 20 * 2.0 ** -24 * np.abs(n).max(-1, keepdims=True) + np.abs(y) * (2.0 ** -11 if b.f16 else 2.0 ** -24) + (
            2.0 ** -25 if b.f16 else 0)
        assert (np.abs(q[row] - y) <= lim * (1 + 2.0 ** -10)).all(), (row, np.abs(q[row] - y).max())
        n, y = ref.turned(x[row, nh:nh + nkv], b.k_norm if norm else None, b.rope[p], EPS)
        exact[page, 0, :, p % b.page] = y
        kerr[page, 0, :, p % b.page] = (20 * 2.0 ** -24 * np.abs(n).max(-1, keepdims=True) + 2.0 ** -11 * np.abs(y)) * (
            1 + 2.0 ** -10) + 2.0 ** -25
        v = x[row, nh + nkv:].astype(np.float16)
        want[page, 1, :, p % b.page] = v
        exact[page, 1, :, p % b.page] = v
    touched = kerr > 0
    assert np.array_equal(data.view(np.int16)[~touched], want.view(np.int16)[~touched])
    assert (np.abs(data[touched].astype(np.float64) - exact[touched]) <= kerr[touched]).all()
    return data


SHAPES = [(4, 2, 64), (16, 8, 128), (8, 8, 128), (16, 2, 64), (5, 1, 128), (12, 4, 64), (48, 3, 128), (7, 7, 64)]
APPENDS = [
    [(1, 1)], [(1, 517)], [(3, 3), (1, 40), (0, 9), (2, 2)], [(70, 70)], [(33, 100), (1, 16), (17, 17)],
    [(1, 5 + i) for i in range(70)],
]


@pytest.mark.parametrize("dtype", ["f32", "f16"])
@pytest.mark.parametrize("nh,nkv,hd", SHAPES)
@pytest.mark.parametrize("case", range(len(APPENDS)))
def test_append(torch, case, nh, nkv, hd, dtype):
    b = Batch(torch, APPENDS[case], nh=nh, nkv=nkv, hd=hd, page=(16, 32, 64, 128, 256)[(case + nh) % 5], dtype=dtype, seed=case)
    c = b.cache()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    q = c.append(b.dev(b.qkv), *b.where(), b.dev(b.rope), b.dev(b.q_norm), b.dev(b.k_norm), EPS, status=status)
    check_append(b, got=q, cache=c)
    assert int(status) == 0


def test_append_many_rows(torch):
    """More than one pass of heads to a warp, and 32 x 32 sequences to look through."""
    for dtype in ("f32", "f16"):
        b = Batch(torch, [(1 + i % 3, 3 + i % 50) for i in range(1100)], nh=16, nkv=8, hd=128, dtype=dtype, seed=5)
        c = b.cache()
        q = c.append(b.dev(b.qkv), *b.where(), b.dev(b.rope), b.dev(b.q_norm), b.dev(b.k_norm), EPS)
        check_append(b, got=q, cache=c)


@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_append_without_norm_in_place_and_strided(torch, dtype):
    b = Batch(torch, [(9, 30), (1, 1), (40, 44)], nh=4, nkv=2, hd=64, dtype=dtype, lead=2, tail=3)
    c = b.cache()
    wide = torch.full((b.M, b.qkv.shape[1] + 32), 7.0, dtype=b.dtype, device="cuda")
    wide[:, 16:-16] = b.dev(b.qkv)
    q = c.append(wide[:, 16:-16], *b.where(), b.dev(b.rope))
    check_append(b, norm=False, got=q, cache=c)
    # in place: through the C entry, rows outside the batch stay as they are
    qw3 = b.qw3
    c2, buf = b.cache(), b.dev(b.qkv)
    starts, lens, table = b.where()
    batch = qw3.Qw3KvBatch(starts.data_ptr(), lens.data_ptr(), table.data_ptr(), table.shape[1], 3, table.shape[1])
    rope = b.dev(b.rope)
    qw3.qw3_kv_paged_append(c2.c, batch, int(b.f16), buf.data_ptr(), b.M, buf.shape[1], b.nh, 0, 0, EPS, rope.data_ptr(),
                            len(b.rope), buf.data_ptr(), buf.shape[1], 0, torch.cuda.current_stream().cuda_stream)
    heads = buf.view(b.M, -1, b.hd)
    check_append(b, norm=False, got=heads[:, :b.nh], cache=c2)
    keep = torch.ones(b.M, dtype=torch.bool)
    keep[2:-3] = False
    assert torch.equal(buf.cpu()[keep], torch.from_numpy(b.qkv)[keep])
    assert torch.equal(heads.cpu()[:, b.nh:], torch.from_numpy(b.qkv).view(b.M, -1, b.hd)[:, b.nh:])


def test_append_places_outside_the_cache(torch):
    """Rows at negative positions, on pages outside the pool, past the table and
    past the rotations are not cached; rows outside the batch are not written."""
    b = Batch(torch, [(5, 3), (4, 20), (6, 40), (2, 30)], nh=4, nkv=2, hd=64, lead=3, tail=4)
    b.table[1, 1] = b.n_pages          # positions 16..19 of sequence 1
    b.table[2, 2] = -7                 # positions 32..39 of sequence 2
    b.lens[3] = 3 * 16 + 1 + 16 * (b.table.shape[1] - 3)      # its last position is past the table's width
    b.rope = b.rope[:38]
    c = b.cache()
    out = torch.full((b.M, b.nh, b.hd), 9.0, device="cuda")
    q = c.append(b.dev(b.qkv), *b.where(), b.dev(b.rope), b.dev(b.q_norm), b.dev(b.k_norm), EPS, out=out)
    assert q is out
    check_append(b, got=q, cache=c)
    assert (q[:3] == 9).all() and (q[-4:] == 9).all() and not (q[3:-4] == 9).any()


def test_append_borders_beyond_the_rows(torch):
    """Borders below 0 and past M are taken as the nearest inside."""
    b = Batch(torch, [(4, 10), (4, 30)], nh=4, nkv=2, hd=64)
    b.starts[0], b.starts[2] = -5, 1000
    c = b.cache()
    check_append(b, got=c.append(b.dev(b.qkv), *b.where(), b.dev(b.rope), b.dev(b.q_norm), b.dev(b.k_norm), EPS), cache=c)


@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_append_values_that_f16_does_not_hold(torch, dtype):
    """A head with NaN, an infinity or 65520 and more is zeros, others stay; the norm of huge and tiny heads."""
    b = Batch(torch, [(8, 24)], nh=4, nkv=2, hd=64, dtype=dtype)
    x = b.qkv.reshape(8, 8, 64)
    x[0, 6, 5] = np.nan
    x[1, 7, 63] = -np.inf
    x[2, 4, 0] = np.nan
    x[3, 5, 9] = np.inf
    if dtype == "f32":
        x[4, 6, 1] = 65520.0
        x[5, 7, 2] = -65519.9          # the largest that rounds to what f16 holds
        x[6, 4] *= 1e30                # squares leave f32
        x[7, 5] *= 1e-30
        x[6, 1] *= 1e30
        x[7, 2] *= 1e-30
    clean = x.copy()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    c = b.cache()
    q = c.append(b.dev(b.qkv), *b.where(), b.dev(b.rope), b.dev(b.q_norm), b.dev(b.k_norm), EPS, status=status)
    assert int(status) == 5
    data = c.data.cpu().numpy()
    place = [(int(b.table[0, p // 16]), p % 16) for p in range(16, 24)]
    dead = {(0, 1, 0), (1, 1, 1), (2, 0, 0), (3, 0, 1)} | ({(4, 1, 0)} if dtype == "f32" else set())
    for r, (page, off) in enumerate(place):
        for sel in (0, 1):
            for g in (0, 1):
                if (r, sel, g) in dead:
                    assert not data[page, sel, g, off].any()
                    continue
                src = clean[r, 4 + 2 * sel + g]
                if sel:
                    assert np.array_equal(data[page, 1, g, off], src.astype(np.float16))
                else:
                    n, y = ref.turned(src[None], b.k_norm, b.rope[16 + r], EPS)
                    lim = 20 * 2.0 ** -24 * np.abs(n).max() + 2.0 ** -11 * np.abs(y[0]) + 2.0 ** -25
                    assert (np.abs(data[page, 0, g, off] - y[0]) <= lim * 1.001).all()
    if dtype == "f32":
        for r, h in ((6, 1), (7, 2)):
            n, y = ref.turned(clean[r, h][None], b.q_norm, b.rope[16 + r], EPS)
            assert (np.abs(q[r, h].cpu().numpy() - y[0]) <= 21 * 2.0 ** -24 * np.abs(n).max()).all()


# ---------------------------------------------------------------- attention

ATTNS = {
    "one": [(1, 1)],
    "short": [(1, 5), (1, 16), (1, 17), (1, 33)],
    "long": [(1, 1000)],
    "tokens": [(1, 1 + 37 * i % 400) for i in range(20)],
    "verify": [(5, 77), (3, 3), (5, 130), (1, 64)],
    "chunk": [(77, 77)],
    "chunk_behind": [(100, 391)],
    "mixed": [(1, 300), (0, 40), (65, 200), (2, 2), (129, 129), (1, 129)],
    "odd": [(128, 128), (127, 255), (33, 257)],
}
HEADS = [(4, 2, 64), (16, 8, 128), (8, 8, 128), (16, 2, 64), (5, 1, 128), (16, 1, 128), (6, 2, 64), (3, 3, 128)]


@pytest.mark.parametrize("dtype", ["f32", "f16"])
@pytest.mark.parametrize("nh,nkv,hd", HEADS)
@pytest.mark.parametrize("case", list(ATTNS))
def test_attention(torch, case, nh, nkv, hd, dtype):
    at = list(ATTNS).index(case)
    b = Batch(torch, ATTNS[case], nh=nh, nkv=nkv, hd=hd, page=(16, 32, 64, 128, 256)[(at + nh) % 5], dtype=dtype, seed=at)
    b.check(b.attend())


@pytest.mark.parametrize("dtype", ["f32", "f16"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 4), (50, 0), (64, 70), (128, 128), (129, 3), (300, 1), (1000, 5)])
@pytest.mark.parametrize("case", ["tokens", "verify", "chunk_behind", "mixed", "odd"])
def test_window_and_sinks(torch, case, window, sinks, dtype):
    nh, nkv, hd = ((4, 2, 64), (16, 8, 128), (5, 1, 128))[(window + sinks) % 3]
    b = Batch(torch, ATTNS[case], nh=nh, nkv=nkv, hd=hd, page=(16, 64)[sinks % 2], dtype=dtype, seed=window)
    b.check(b.attend(window=window, sinks=sinks), window=window, sinks=sinks)


@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_long_contexts(torch, dtype):
    """Sums over thousands of positions, split over many CTAs and joined."""
    for seqs, kw in (([(1, 20000)], {}), ([(4, 9001), (1, 50)], {}), ([(130, 6000)], {}), ([(300, 5000), (1, 7000)], {}),
                     ([(200, 6000), (2, 6500)], dict(window=700, sinks=9))):
        b = Batch(torch, seqs, nh=8, nkv=2, hd=128, page=64, dtype=dtype, seed=1)
        b.check(b.attend(**kw), **kw)


@pytest.mark.parametrize("seqs,kw", [([(404, 1831)], {}), ([(31, 1799), (90, 800)], dict(window=172)), ([(253, 2197)], dict(window=1148, sinks=3)),
                                     ([(290, 837)], {})])
@pytest.mark.parametrize("nh,nkv,hd", [(16, 8, 128), (8, 4, 64)])
def test_as_exact_as_products_in_32_bits(torch, seqs, kw, nh, nkv, hd):
    """f32 activations, many rows: no farther from 64 bits than matrix products, exponentials and sums in f32 are. (A score's sum
    is truncated at each of hd / 16 steps, half a step of f32 on average and always downwards, where f32 rounds hd times, to
    nearest: for 64 and 128 both come to 2 to 4 half steps. A quarter is left for where the two fall together.)"""
    b = Batch(torch, seqs, nh=nh, nkv=nkv, hd=hd, page=32, seed=21)
    got = b.attend(**kw).cpu().numpy().astype(np.float64)
    want, _, _ = ref.attend(b.q, b.data.astype(np.float64), b.starts, b.lens, b.table, **kw)
    plain = np.zeros_like(want)
    for i, (rows, n) in enumerate(seqs):
        a, j = int(b.starts[i]), np.arange(n)
        k, v = (b.dev(b.data[b.table[i, j // 32], s, :, j % 32]).float().repeat_interleave(nh // nkv, 1) for s in (0, 1))
        p = n - rows + np.arange(rows)[:, None]
        sees = b.dev((j <= p) & ((j > p - kw.get("window", n)) | (j < kw.get("sinks", 0))))
        s = torch.einsum("rhd,jhd->hrj", b.dev(b.q[a:a + rows]), k) * hd ** -0.5
        s = torch.where(sees, s, -torch.inf)
        e = torch.exp(s - s.amax(-1, keepdim=True))
        plain[a:a + rows] = (torch.einsum("hrj,jhd->hrd", e, v) / e.sum(-1, keepdim=True)).transpose(0, 1).cpu().numpy()
    off, of32 = np.linalg.norm(got - want), np.linalg.norm(plain - want)
    assert off <= 1.25 * of32, (off / np.linalg.norm(want), of32 / np.linalg.norm(want))


@pytest.mark.parametrize("dtype", ["f32", "f16"])
@pytest.mark.parametrize("seqs", [[(4, 2), (1, 0), (3, 0), (2, 20)], [(60, 20), (1, 40), (200, 100)]])
def test_rows_that_see_nothing(torch, seqs, dtype):
    """More rows than positions, lengths of zero and below: zeros."""
    b = Batch(torch, seqs, dtype=dtype)
    if len(seqs) == 4:
        b.lens[2] = -3
    got = b.attend()
    want, _ = b.check(got)
    assert not got.float().cpu().numpy()[(want == 0).all((1, 2))].any()


@pytest.mark.parametrize("dtype", ["f32", "f16"])
@pytest.mark.parametrize("rows", [1, 3, 90])
def test_pages_outside_the_pool(torch, rows, dtype):
    """Positions without a page are not attended, in whatever they lie between;
    a row left with none is zeros."""
    b = Batch(torch, [(rows, 400), (rows, 100), (rows, 300)], dtype=dtype, nh=4, nkv=2, hd=64)
    b.table[0, [0, 3, 4, 20]] = [-1, b.n_pages, 2 ** 31 - 1, -2 ** 31]
    b.table[1, :] = -1
    b.table[2, 8:18] = -1
    got = b.attend()
    b.check(got)
    assert not got[rows:2 * rows].any()
    b.check(b.attend(window=30, sinks=2), window=30, sinks=2)


@pytest.mark.parametrize("dtype", ["f32", "f16"])
@pytest.mark.parametrize("seqs", [[(1, 200), (1, 90)], [(6, 200), (3, 90)], [(150, 200), (40, 90)]])
def test_what_is_not_seen_has_no_part(torch, seqs, dtype):
    """NaN and infinities in places that some rows see and others do not."""
    b = Batch(torch, seqs, dtype=dtype, nh=4, nkv=2, hd=64)
    n = seqs[0][1]
    for back, bad in ((1, np.nan), (2, np.inf), (60, -np.inf), (61, np.nan)):
        p = n - back
        b.data[b.table[0, p // 16], 1, 0, p % 16, back % 64] = bad
    p = n - 3
    b.data[b.table[0, p // 16], 0, 1, p % 16, 7] = np.nan
    kw = dict(window=50, sinks=1)
    want, err, written = ref.attend(b.q, np.where(np.isfinite(b.data), b.data, 0).astype(np.float64), b.starts, b.lens, b.table, **kw)
    got = b.attend(**kw).float().cpu().numpy()
    lim = ref.bound(err, want, b.hd, b.f16)
    rows0 = seqs[0][0]
    for i in range(b.M):
        if i >= rows0:
            assert (np.abs(got[i] - want[i]) <= lim[i]).all()
            continue
        p = n - rows0 + i
        dims = {back % 64 for back in (1, 2, 60, 61) if p - 50 < n - back <= p}
        for h in range(4):
            if h < 2:
                fine = np.array([d not in dims for d in range(64)])
                assert (np.abs(got[i, h] - want[i, h]) <= lim[i, h])[fine].all(), (i, h)
                assert not np.isfinite(got[i, h][~fine]).any()
            elif p - 50 < n - 3 <= p:
                assert np.isnan(got[i, h]).all()
            else:
                assert (np.abs(got[i, h] - want[i, h]) <= lim[i, h]).all()


def check_infinities(b, got, **kw):
    """Infinite values come out as they are, opposite ones as NaN, and the other outputs within their bound."""
    want, err, written = ref.attend(b.q, b.data.astype(np.float64), b.starts, b.lens, b.table, **kw)
    got = got.cpu().numpy().astype(np.float64)
    assert np.array_equal(np.isnan(got[written]), np.isnan(want[written]))
    inf = np.isinf(want) & written[:, None, None]
    assert np.array_equal(got[inf], want[inf])
    fine = np.isfinite(want) & written[:, None, None]
    want = np.where(fine, want, 0)
    assert (np.abs(got - want)[fine] <= ref.bound(err, want, b.hd, b.f16)[fine]).all()
    return inf.any()


@pytest.mark.parametrize("dtype", ["f32", "f16"])
@pytest.mark.parametrize("seqs", [[(1, 200), (1, 90)], [(6, 200), (3, 90)], [(150, 200), (40, 90)], [(1, 3000), (2, 70)],
                                  [(100, 2500)], [(300, 400), (1, 900)]])
def test_infinities_that_are_seen(torch, seqs, dtype):
    """In values that every row sees and in ones that some rows see, in units that are split and in whole ones, in place too."""
    b = Batch(torch, seqs, dtype=dtype, nh=4, nkv=2, hd=64, seed=11)
    b.q *= b.np_type(0.25)      # (no weight below 2^-30 of its row's largest)
    for i, (rows, n) in enumerate(seqs):
        for p, d, bad in ((3, 5, np.inf), (3, 6, -np.inf), (17, 7, np.inf), (n - rows // 2 - 1, 7, -np.inf), (n - 1, 9, np.inf)):
            b.data[b.table[i, p // 16], 1, i % 2, p % 16, d] = bad
    assert check_infinities(b, b.attend())
    check_infinities(b, b.attend(window=60, sinks=4), window=60, sinks=4)
    q = b.dev(b.q)
    check_infinities(b, b.attend(q=q, out=q))


@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_long_rows_beside_what_is_not_finite(torch, dtype):
    """Rows that are done without matrix products, for longer than a wait in the kernel may last that nothing ends: no
    status, and the right outputs. (304 units, two to a CTA, so that the CTA's other warps wait for the first one's rows, some
    1.6 s where the limit is 1 s.)"""
    from quantized_transformer_decode_gb300 import qw3
    f16 = dtype == "f16"
    B, rows, nh, hd, page, pages = 304, 16 if f16 else 8, 16, 64, 256, 1728 if f16 else 3712
    n = pages * page - 7
    g = torch.Generator(device="cuda").manual_seed(1)
    data = torch.randn(pages, 2, 1, page, hd, generator=g, device="cuda").half()
    hole = n - rows // 2            # the first half of the rows does not see it
    data[hole // page, 1, 0, hole % page, 9] = float("inf")
    table = torch.arange(pages, dtype=torch.int32, device="cuda").repeat(B, 1)          # every sequence holds the same
    q1 = torch.randn(rows, nh, hd, generator=g, device="cuda").to(torch.float16 if f16 else torch.float32)
    starts = torch.arange(B + 1, dtype=torch.int32, device="cuda") * rows
    lens = torch.full((B,), n, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    cache = qw3.KVCachePaged(pages, page, 1, hd, data=data)
    q = q1.repeat(B, 1, 1)
    out = cache.attention(q, starts, lens, table, max_rows=rows, max_len=n, status=status)
    assert int(status) == 0
    out = out.view(B, rows, nh, hd).double()
    assert (out == out[:1]).logical_or(out.isnan() & out[:1].isnan()).all()
    k, v = data[:, 0, 0].reshape(-1, hd)[:n].double(), data[:, 1, 0].reshape(-1, hd)[:n].double()
    v[hole, 9] = 0
    for r in range(rows):
        seen = n - rows + r + 1
        s = q1[r].double() @ k[:seen].T * hd ** -0.5
        p = torch.softmax(s, -1)
        want = p @ v[:seen]
        err = {"pv": (p @ v[:seen].abs()).cpu().numpy(), "qk": (q1[r].double().abs() @ k[:seen].abs().T).amax(-1, keepdim=True).cpu().numpy() * hd ** -0.5,
               "vmax": float(v.abs().max()), "n": np.float64(16)}
        # (a row's sums are chains of n roundings of 2^-24, random in sign: 16 sqrt(n) of them with room)
        lim = ref.bound(err, want.cpu().numpy(), hd, f16) + 16 * n ** 0.5 * 2.0 ** -24 * err["pv"]
        got = out[0, r].cpu().numpy()
        if n - rows + r >= hole:
            assert np.isposinf(got[:, 9]).all()
            got[:, 9] = want[:, 9].cpu().numpy()
        assert (np.abs(got - want.cpu().numpy()) <= lim).all(), (r, np.abs(got - want.cpu().numpy()).max(), lim.min())


@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_rows_outside_the_batch_stay(torch, dtype):
    b = Batch(torch, [(3, 40), (70, 90), (1, 5)], dtype=dtype, lead=2, tail=5)
    out = torch.full((b.M, b.nh, b.hd), 9.0, dtype=b.dtype, device="cuda")
    got = b.attend(out=out)
    assert got is out
    _, written = b.check(got)
    assert (got[~torch.from_numpy(written).cuda()] == 9).all() and written.sum() == 74
    # a bound below a sequence's rows: those past it stay
    for cut in (2, 60):
        out = torch.full_like(out, 9.0)
        _, written = b.check(b.attend(out=out, max_rows=cut), max_rows=cut)
        assert (out[~torch.from_numpy(written).cuda()] == 9).all()


@pytest.mark.parametrize("dtype", ["f32", "f16"])
@pytest.mark.parametrize("seqs", [[(1, 300), (2, 40)], [(90, 300), (2, 40)]])
def test_bounds_scale_and_in_place(torch, seqs, dtype):
    b = Batch(torch, seqs, dtype=dtype, nh=16, nkv=8, hd=128)
    b.check(b.attend(max_len=100), max_len=100)
    b.check(b.attend(scale=0.0), scale=0.0)
    b.check(b.attend(scale=-0.3), scale=-0.3)
    q = b.dev(b.q)
    got = b.attend(q=q, out=q)
    assert got is q
    b.check(got)
    assert not b.attend(max_len=0).any()


@pytest.mark.parametrize("dtype", ["f32", "f16"])
@pytest.mark.parametrize("rows", [1, 70])
def test_large_scores(torch, rows, dtype):
    """One position that takes everything, scores far apart, and queries at the type's ends."""
    for size in (300.0, 60000.0) + ((1e30, 1e-30) if dtype == "f32" else ()):
        b = Batch(torch, [(rows, 150), (rows, 80)], dtype=dtype, nh=4, nkv=2, hd=64)
        b.q = np.clip(b.q.astype(np.float64) / 4 * size, -60000 if b.f16 else -3e38, 60000 if b.f16 else 3e38).astype(b.np_type)
        scale = min(0.125, 40 / size)
        b.check(b.attend(scale=scale), scale=np.float64(np.float32(scale)))


@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_queries_and_outputs_inside_wider_rows(torch, dtype):
    """Through the C entry: queries where the projections lie, outputs in rows of another width; what lies beside them stays."""
    b = Batch(torch, [(1, 70), (90, 200), (3, 3), (64, 64)], nh=4, nkv=2, hd=64, dtype=dtype, lead=1, tail=2)
    qw3, c = b.qw3, b.cache()
    starts, lens, table = b.where()
    batch = qw3.Qw3KvBatch(starts.data_ptr(), lens.data_ptr(), table.data_ptr(), table.shape[1], 4, table.shape[1])
    wide = torch.full((b.M, 8, b.hd), 5.0, dtype=b.dtype, device="cuda")
    wide[:, 2:6] = b.dev(b.q)
    out = torch.full((b.M, 7, b.hd), 9.0, dtype=b.dtype, device="cuda")
    need = qw3.qw3_kv_paged_attn_workspace_bytes(4, b.M, int(b.f16), 4, 2, 64, 90, 208)
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda").fill_(255)
    stream = torch.cuda.current_stream().cuda_stream
    size = wide.element_size() * b.hd
    for src, dst, first in ((wide, out, 1), (wide, wide, 2)):
        qw3.qw3_kv_paged_attn(c.c, batch, int(b.f16), wide.data_ptr() + 2 * size, b.M, 8 * b.hd, 4, 90, 208, 0, 0, b.hd ** -0.5,
                              dst.data_ptr() + first * size, dst.shape[1] * b.hd, ws.data_ptr(), need, 0, stream)
        b.check(dst[:, first:first + 4])
        keep = torch.ones(dst.shape[:2], dtype=torch.bool, device="cuda")
        keep[1:-2, first:first + 4] = False
        assert (dst[keep] == (9 if dst is out else torch.cat((torch.full_like(wide[:, :2], 5.0), b.dev(b.q), torch.full_like(wide[:, 6:], 5.0)), 1)[keep])).all()


def test_queries_of_any_size(torch):
    """f32 queries up to the type's largest values, and scores that leave f32."""
    for rows in (1, 70):
        b = Batch(torch, [(rows, 150)], nh=4, nkv=2, hd=64)
        b.q = (b.q.astype(np.float64) / 8 * 3e38).clip(-3.3e38, 3.3e38).astype(np.float32)
        b.check(b.attend(scale=1e-38), scale=np.float64(np.float32(1e-38)))
        b.q = (b.rng.standard_normal(b.q.shape) * 1e-38).astype(np.float32)
        b.check(b.attend(scale=1e38), scale=np.float64(np.float32(1e38)))


def test_queries_of_any_size_beside_infinities(torch):
    """f32 queries at the type's ends, where what rows see is not finite and they are done without matrix products."""
    for size, scale in ((3e38, 1e-38), (1e-38, 1e38)):
        b = Batch(torch, [(90, 200)], nh=4, nkv=2, hd=64, seed=13)
        b.q = (b.q.astype(np.float64) / 8 * size).clip(-3.3e38, 3.3e38).astype(np.float32)
        b.data[b.table[0, 150 // 16], 1, 0, 150 % 16, 9] = np.inf      # rows 40 .. 89 see it
        b.check(b.attend(scale=scale), scale=np.float64(np.float32(scale)))


def test_rows_of_zeros_at_any_scale(torch):
    """A query row of zeros (as append leaves one) has equal scores, however small the scale."""
    for rows in (1, 70):
        for kw in ({}, dict(window=40, sinks=2)):
            b = Batch(torch, [(rows, 150), (rows, rows)], nh=4, nkv=2, hd=64)
            b.q[0] = 0
            b.q[rows // 2 + rows:] = 0
            for scale in (1e-38, 1e-20, 1e-8, 1.0):
                b.check(b.attend(scale=scale, **kw), scale=np.float64(np.float32(scale)), **kw)


def test_offsets_past_32_bits(torch):
    """Pages beyond 2^32 bytes of the pool."""
    from quantized_transformer_decode_gb300 import qw3
    nkv, hd, page, n_pages = 8, 128, 64, 18000            # 4.7 GB
    small = Batch(torch, [(1, 700), (90, 500)], nh=16, nkv=nkv, hd=hd, page=page, spare=0, dtype="f16")
    pool = torch.empty((n_pages, 2, nkv, page, hd), dtype=torch.float16, device="cuda")
    shift = n_pages - small.n_pages
    pool[shift:] = small.dev(small.data)
    c = qw3.KVCachePaged(n_pages, page, nkv, hd, data=pool)
    starts, lens, table = small.where()
    table = torch.where(table >= 0, table + shift, table)
    small.check(c.attention(small.dev(small.q), starts, lens, table))
    q = c.append(small.dev(small.qkv), starts, lens, table, small.dev(small.rope), small.dev(small.q_norm), small.dev(small.k_norm), EPS)
    view = qw3.KVCachePaged(small.n_pages, page, nkv, hd, data=pool[shift:].clone())
    check_append(small, got=q, cache=view)


def test_many_sequences(torch):
    b = Batch(torch, [(1 + (i % 97 == 0) * 40, 41 + i % 60) for i in range(700)], nh=4, nkv=2, hd=64, dtype="f16")
    b.check(b.attend())


@pytest.mark.parametrize("seqs", [[(1, 3000)], [(100, 900), (1, 2000)]])
def test_streams_graphs_and_repeats(torch, seqs):
    """The same bits each time, on another stream, and from a graph whose inputs change."""
    b = Batch(torch, seqs, nh=16, nkv=8, hd=128, dtype="f32")
    c, q = b.cache(), b.dev(b.q)
    where = b.where()
    kw = dict(max_rows=max(r for r, _ in seqs), max_len=max(n for _, n in seqs))
    first = c.attention(q, *where, **kw)
    b.check(first)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = [c.attention(q, *where, **kw) for _ in range(3)]
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(first, t) for t in again)
    g = torch.cuda.CUDAGraph()
    out = torch.empty_like(q)
    with torch.cuda.graph(g):
        c.attention(q, *where, out=out, **kw)
    for seed in (3, 4):
        b.q = np.random.default_rng(seed).standard_normal(b.q.shape).astype(np.float32)
        b.lens -= seed
        q.copy_(b.dev(b.q))
        where[1].copy_(b.dev(b.lens))
        g.replay()
        b.check(out)


@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_units_of_one_row_tile_among_longer_ones(torch, dtype):
    """A sequence's last unit may fill one row tile only, and one warpgroup then goes ahead of the other: the same bits
    in every one of many calls, and the right ones."""
    for seqs, nh, kw in (([(1117, 1185), (1117, 1185), (1117, 1185)], 32, dict(window=730, sinks=1)),
                         ([(1825, 2534), (33, 700)], 16, dict(window=249, sinks=4)), ([(597, 3373), (65, 3307), (289, 900)], 32, {}),
                         ([(4049, 4063)], 32, dict(window=1291, sinks=4)), ([(1691, 2355), (1691, 1800)], 16, {})):
        b = Batch(torch, seqs, nh=nh, nkv=8, hd=128, page=32, dtype=dtype, seed=2)
        c, q, where = b.cache(), b.dev(b.q), b.where()
        out = c.attention(q, *where, **kw)
        b.check(out, **kw)
        differ = torch.zeros((), dtype=torch.int64, device="cuda")
        cold = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
        for _ in range(400):
            cold.zero_()                    # K and V come from memory, late
            differ += (c.attention(q, *where, **kw) != out).any()
        assert int(differ) == 0


@pytest.mark.parametrize("dtype", ["f32", "f16"])
@pytest.mark.parametrize("seqs,tail", [([(100, 6000)], 300), ([(100, 6000), (1, 300)], 300), ([(0, 40), (70, 5000), (0, 0)], 500)])
def test_units_that_are_not_there(torch, seqs, tail, dtype):
    """Bounds of more rows than the sequences have, in a call that is split: what the join reads of the units that could be is
    written, whatever the workspace held."""
    from quantized_transformer_decode_gb300 import qw3
    b = Batch(torch, seqs, nh=4, nkv=2, hd=64, dtype=dtype, tail=tail)
    n = max(n for _, n in seqs)
    need = qw3.qw3_kv_paged_attn_workspace_bytes(len(seqs), b.M, int(b.f16), 4, 2, 64, b.M, n)
    assert need > 1 << 20       # (units are split)
    first = None
    for fill in (0, 1, 0x7F):
        ws = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
        out = torch.full((b.M, 4, 64), 9.0, dtype=b.dtype, device="cuda")
        _, written = b.check(b.attend(out=out, max_rows=b.M, max_len=n, workspace=ws))
        assert (out[~torch.from_numpy(written).cuda()] == 9).all()
        assert first is None or torch.equal(out, first)
        first = out


def test_two_at_once(torch):
    """Calls on two streams, each with its own workspace."""
    bs = [Batch(torch, [(1, 4000), (200, 1500)], nh=16, nkv=8, hd=128, dtype="f16", seed=i) for i in range(2)]
    cs, qs, ws = [b.cache() for b in bs], [b.dev(b.q) for b in bs], [b.where() for b in bs]
    streams = [torch.cuda.Stream() for _ in bs]
    torch.cuda.synchronize()
    outs = []
    for _ in range(5):
        for c, q, w, s in zip(cs, qs, ws, streams):
            with torch.cuda.stream(s):
                outs.append(c.attention(q, *w))
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        assert torch.equal(o, outs[i % 2])
    for b, o in zip(bs, outs):
        b.check(o)


def test_a_table_wider_than_the_call_uses(torch):
    """A strided view of a larger table."""
    b = Batch(torch, [(1, 90), (20, 60)])
    wide = torch.full((2, 40), 2 ** 30, dtype=torch.int32, device="cuda")
    wide[:, 3:3 + b.table.shape[1]] = b.dev(b.table)
    starts, lens, _ = b.where()
    b.check(b.cache().attention(b.dev(b.q), starts, lens, wide[:, 3:3 + b.table.shape[1]]))


def test_another_current_device(torch):
    if torch.cuda.device_count() < 2:
        pytest.skip("one GPU")
    b = Batch(torch, [(1, 90), (20, 60)])
    c, q, w = b.cache(), b.dev(b.q), b.where()
    with torch.cuda.device(1):
        got = c.attention(q, *w)
    b.check(got)


# ---------------------------------------------------------------- refusals

def test_refusals(torch):
    from quantized_transformer_decode_gb300 import qw3
    b = Batch(torch, [(1, 90), (20, 60)])
    c, q, (starts, lens, table) = b.cache(), b.dev(b.q), b.where()
    rope, qkv = b.dev(b.rope), b.dev(b.qkv)
    bad = qw3.Qw3Error
    for args in ((0, 16, 2, 64), (1, 17, 2, 64), (1, 8, 2, 64), (1, 512, 2, 64), (1, 16, 0, 64), (1, 16, 65, 64),
                 (1, 16, 2, 96), (2 ** 32 + 1, 16, 2, 64), (2 ** 31 - 1, 256, 64, 128)):
        with pytest.raises(bad):
            qw3.KVCachePaged(*args)
    with pytest.raises(bad):
        qw3.KVCachePaged(b.n_pages + 1, 16, 2, 64, data=c.data)
    with pytest.raises(bad):
        qw3.KVCachePaged(1, 16, 2, 64, data=torch.zeros(10000, dtype=torch.float16))
    with pytest.raises(bad):
        qw3.KVCachePaged(1, 16, 2, 64, device="cpu")
    for call in (
        lambda: c.attention(q.double(), starts, lens, table), lambda: c.attention(q.cpu(), starts, lens, table),
        lambda: c.attention(q[:, :, :32], starts, lens, table), lambda: c.attention(q[:, :3], starts, lens, table),
        lambda: c.attention(q[:, ::2], starts, lens, table), lambda: c.attention(q, starts[:-1], lens, table),
        lambda: c.attention(q, starts.long(), lens, table), lambda: c.attention(q, starts, lens, table[:1]),
        lambda: c.attention(q, starts, lens, table.t().contiguous().t()), lambda: c.attention(q, starts, lens, table, max_len=10000),
        lambda: c.attention(q, starts, lens, table, window=-1), lambda: c.attention(q, starts, lens, table, sinks=-1),
        lambda: c.attention(q, starts, lens, table, max_rows=-1), lambda: c.attention(q, starts, lens, table, scale=float("nan")),
        lambda: c.attention(q, starts, lens, table, window=2 ** 31), lambda: c.attention(q, starts, lens, table, out=q.half()),
        lambda: c.attention(q, starts, lens.cpu(), table),
        lambda: c.append(qkv[:, :-1], starts, lens, table, rope), lambda: c.append(qkv[:, 1:-63], starts, lens, table, rope),
        lambda: c.append(qkv.double(), starts, lens, table, rope), lambda: c.append(qkv, starts, lens, table, rope[:, :-1]),
        lambda: c.append(qkv, starts, lens, table, rope, q_norm=rope.flatten()[:63]),
        lambda: c.append(qkv, starts, lens, table, rope, eps=-1.0), lambda: c.append(qkv, starts, lens, table, rope[:0]),
        lambda: c.append(qkv, starts, lens, table, rope, out=q.half()),
    ):
        with pytest.raises(bad):
            call()
    small = torch.empty(16, dtype=torch.uint8, device="cuda")
    need = qw3.qw3_kv_paged_attn_workspace_bytes(2, b.M, 0, 4, 2, 64, b.M, 96)
    if need > 16:
        with pytest.raises(bad):
            c.attention(q, starts, lens, table, workspace=small)
    # nothing to do is no error
    none = torch.zeros((0, 4, 64), device="cuda")
    assert c.attention(none, starts, lens, table).shape == none.shape
    empty = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert c.attention(q, empty, empty[:0], table[:0]).shape == q.shape
    b.check(c.attention(q, starts, lens, table))


@pytest.mark.parametrize("dtype", ["f32", "f16"])
@pytest.mark.parametrize("seqs", [[(1, 3000)], [(100, 6000)], [(100, 3000), (1, 2500)]])
def test_workspaces_of_the_exact_size(torch, seqs, dtype):
    """What is too small by a byte, or missing, is refused; what lies behind the workspace stays as it was."""
    from quantized_transformer_decode_gb300 import qw3
    b = Batch(torch, seqs, nh=4, nkv=2, hd=64, dtype=dtype)
    rows, n = max(r for r, _ in seqs), max(n for _, n in seqs)
    need = qw3.qw3_kv_paged_attn_workspace_bytes(len(seqs), b.M, int(b.f16), 4, 2, 64, rows, n)
    assert need > 16
    room = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    kw = dict(max_rows=rows, max_len=n)
    b.check(b.attend(workspace=room[:need], **kw))
    assert (room[need:] == 0xA5).all()
    q, out = b.dev(b.q), torch.full((b.M, 4, 64), 9.0, dtype=b.dtype, device="cuda")
    with pytest.raises(qw3.Qw3Error):
        b.attend(q=q, out=out, workspace=room[:need - 1], **kw)
    c, (starts, lens, table) = b.cache(), b.where()
    batch = qw3.Qw3KvBatch(starts.data_ptr(), lens.data_ptr(), table.data_ptr(), table.shape[1], len(seqs), table.shape[1])
    with pytest.raises(qw3.Qw3Error):
        qw3.qw3_kv_paged_attn(c.c, batch, int(b.f16), q.data_ptr(), b.M, 256, 4, rows, n, 0, 0, 0.125, out.data_ptr(), 256, 0, need,
                              0, torch.cuda.current_stream().cuda_stream)
    assert (out == 9).all()


# ---------------------------------------------------------------- together

@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_append_then_attention_over_steps(torch, dtype):
    """A prompt in two chunks beside sequences that decode: every step appends and
    attends, and each step's outputs are those of the whole history."""
    from quantized_transformer_decode_gb300 import qw3
    rng = np.random.default_rng(9)
    nh, nkv, hd, page, n_pages = 8, 2, 64, 16, 40
    kind = torch.float16 if dtype == "f16" else torch.float32
    c = qw3.KVCachePaged(n_pages, page, nkv, hd)
    c.data.fill_(float("nan"))
    free = list(rng.permutation(n_pages))
    table = np.full((3, 13), -1, np.int32)
    lens = np.zeros(3, np.int32)
    rope = ref.rope_table(256, hd)
    for rows in ((70, 1, 0), (100, 1, 9), (1, 1, 1), (1, 4, 1)):
        lens = lens + np.array(rows, np.int32)
        for i in range(3):
            for k in range(-(-int(lens[i]) // page)):
                if table[i, k] < 0:
                    table[i, k] = free.pop()
        starts = np.concatenate(([0], np.cumsum(rows))).astype(np.int32)
        m = int(starts[-1])
        qkv = torch.from_numpy(rng.standard_normal((m, (nh + 2 * nkv) * hd)).astype(np.float32)).cuda().to(kind)
        where = [torch.from_numpy(v).cuda() for v in (starts, lens, table)]
        q = c.append(qkv, *where, torch.from_numpy(rope).cuda())
        got = c.attention(q, *where).float().cpu().numpy()
        data = c.data.cpu().numpy().astype(np.float64)
        want, err, written = ref.attend(q.float().cpu().numpy(), data, starts, lens, table)
        assert written.all() and (np.abs(got - want) <= ref.bound(err, want, hd, dtype == "f16")).all()
