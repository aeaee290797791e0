"""qw3_sample against the oracle's sampler (f64).

Tokens have to be equal wherever no decision of the row is a near one: the f32
weights are within 4e-6 of exact (exp 2^-22 for an argument of up to 28 rounded
twice at 2^-24), so a row whose oracle margin is below 4e-6 may go either way
and is left out. Probabilities: within 8e-6 (a weight and a total)."""
import numpy as np
import pytest

from oracle import qw3_oracle as orc

pytestmark = pytest.mark.gpu

NEAR = 4e-6


@pytest.fixture(scope="module")
def torch():
    import torch as t
    if not t.cuda.is_available():
        pytest.skip("no CUDA device")
    from quantized_transformer_decode_gb300 import build
    build.build()
    return t


def run(torch, logits, u, pad=0, **kw):
    from quantized_transformer_decode_gb300 import qw3
    cu = lambda x, d: torch.from_numpy(np.asarray(x, d)).cuda()  # noqa: E731
    buf = cu(np.pad(np.asarray(logits, np.float32), ((0, 0), (pad, pad)), constant_values=1e30), np.float32)
    view = buf[:, pad:buf.shape[1] - pad] if pad else buf
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = {k: cu(v, np.int32 if k == "top_k" else np.float32) for k, v in kw.items() if v is not None}
    token, prob = qw3.sample(view, cu(u, np.float32), status=status, **args)
    return token.cpu().numpy(), prob.cpu().numpy(), int(status)


def check(torch, logits, u, least=0.9, pad=0, **kw):
    """Compare every row; at least `least` of them must not be near ones."""
    token, prob, status = run(torch, logits, u, pad, **kw)
    assert status == 0
    clear = 0
    for i, row in enumerate(np.asarray(logits, np.float32)):
        t, p, margin = orc.sample_token(row, np.float32(u[i]), **{k: np.asarray(v)[i] if k == "top_k" else np.float32(v[i])
                                                                 for k, v in kw.items() if v is not None})
        if margin > NEAR:
            clear += 1
            assert token[i] == t, (i, int(token[i]), t, margin)
            assert abs(prob[i] - p) <= 8e-6 * p, (i, float(prob[i]), p)
    assert clear >= least * len(u)


def settings(rng, B):
    return dict(temperature=rng.choice([0.0, 0.3, 0.7, 1.0, 1.7], B), top_k=rng.choice([0, 1, 2, 20, 999, 10 ** 6], B),
                top_p=rng.choice([0.0, 0.1, 0.5, 0.9, 0.999, 1.0], B), min_p=rng.choice([0.0, 0.02, 0.3, 1.0], B))


@pytest.mark.parametrize("V", [1, 2, 3, 31, 33, 255, 1000, 4099, 32768, 50257, 151936, 262145])
def test_random_rows_and_settings(torch, V):
    rng = np.random.default_rng(V)
    B = 60 if V < 60000 else 24
    # settings whose edges lie on exact values (a lone token, top-p of equal weights) are not near in f64: none is skipped
    # for rows of one token
    logits = rng.standard_normal((B, V)) * rng.choice([0.5, 2.0, 6.0], (B, 1))
    check(torch, logits, rng.random(B), least=0.6 if V < 40 else 0.8, **settings(rng, B))


@pytest.mark.parametrize("kw", [dict(), dict(top_k=[50]), dict(top_p=[0.9]), dict(min_p=[0.05]), dict(temperature=[0.6]),
                                dict(temperature=[0.8], top_k=[40], top_p=[0.95], min_p=[0.05])])
def test_each_setting_alone(torch, kw):
    rng = np.random.default_rng(7)
    B, V = 64, 20011
    check(torch, rng.standard_normal((B, V)) * 3, rng.random(B), **{k: v * B for k, v in kw.items()})


def test_equal_logits(torch):
    """Ties go to the lowest indices, across any split of the row."""
    V = 70001
    rows = np.zeros((6, V), np.float32)
    u = [0.0, 0.5, 0.99999, 0.3, 0.7, 0.5]
    token, prob, _ = run(torch, rows, u, top_k=[5, 40000, 5, 0, V, 1], top_p=[1.0, 1.0, 1.0, 0.25, 1.0, 1.0])
    f = lambda n, x: int(np.floor(np.float64(np.float32(x)) * n))  # noqa: E731
    n_p = int(np.ceil(0.25 * V))
    assert token.tolist() == [0, f(40000, 0.5), 4, f(n_p, 0.3), f(V, 0.7), 0]
    assert np.allclose(prob, [1 / 5, 1 / 40000, 1 / 5, 1 / n_p, 1 / V, 1], rtol=1e-6)


def test_signed_zeros_are_one_value(torch):
    row = np.array([[-0.0, 0.0, -0.0, 0.0]], np.float32)
    assert [run(torch, row, [u], top_k=[2])[0][0] for u in (0.0, 0.49, 0.51, 0.99)] == [0, 0, 1, 1]
    assert run(torch, row, [0.5], temperature=[0.0])[0][0] == 0


def test_plateaus_inside_a_row(torch):
    """Cuts that fall inside runs of equal logits spread over the row."""
    rng = np.random.default_rng(12)
    B, V = 40, 9001
    logits = np.round(rng.standard_normal((B, V)) * 2)
    check(torch, logits, rng.random(B), least=0.7, top_k=rng.integers(1, V, B), top_p=rng.uniform(0.2, 1.0, B))


def test_masked_rows(torch):
    rng = np.random.default_rng(13)
    B, V = 24, 30011
    logits = (rng.standard_normal((B, V)) * 2).astype(np.float32)
    logits[rng.random((B, V)) < 0.999] = -np.inf
    logits[:, 17] = 0.5
    logits[0] = -np.inf
    logits[0, V - 1] = -3e38                            # one token left, far from any other number
    logits[1, :] = np.finfo(np.float32).min              # a mask of the type's lowest value everywhere
    check(torch, logits, rng.random(B), least=0.7, **settings(rng, B))


def test_large_and_tiny_scales(torch):
    rng = np.random.default_rng(14)
    B, V = 32, 5003
    logits = rng.standard_normal((B, V)).astype(np.float32)
    logits[::4] *= 1e4
    logits[1::4] *= 1e-6
    logits[2::4] += 1e5
    logits[3::4] = logits[3::4] * 2 - 200
    check(torch, logits, rng.random(B), least=0.7, temperature=rng.choice([1e-3, 0.5, 1.0, 100.0], B))


def test_ends_of_u(torch):
    V = 40009
    rng = np.random.default_rng(15)
    row = rng.standard_normal((4, V)).astype(np.float32)
    token, _, _ = run(torch, row, [0.0, -1.0, 1.0, np.nan])
    assert token[0] == 0 and token[1] == 0 and token[2] == V - 1 and token[3] == 0
    row[:, 0] = row[:, V - 1] = -np.inf
    token, _, _ = run(torch, row, [0.0, 0.0, 1.0, 1.0 - 2.0 ** -24])
    assert token[0] == 1 and token[2] == V - 2


def test_rows_without_an_answer(torch):
    V = 3001
    rows = np.zeros((7, V), np.float32)
    rows[0, 5] = np.nan
    rows[1] = -np.inf
    rows[2, 9] = np.inf
    rows[3, 9] = np.inf                                  # greedy: the answer is 9
    rows[4, 100] = 3.0
    token, prob, status = run(torch, rows, [0.5] * 7, temperature=[1, 1, 1, 0, 0, np.nan, np.inf])
    assert status == 5
    assert token.tolist() == [-1, -1, -1, 9, 100, -1, -1] and prob.tolist() == [0, 0, 0, 1, 1, 0, 0]
    token, _, status = run(torch, rows[4:5], [0.5], temperature=[0])
    assert status == 0 and token.tolist() == [100]


def test_strided_rows_and_no_settings(torch):
    rng = np.random.default_rng(16)
    B, V = 12, 4097
    for pad in (1, 3, 8):
        check(torch, rng.standard_normal((B, V)), rng.random(B), pad=pad, top_k=[100] * B)


def test_many_rows(torch):
    rng = np.random.default_rng(17)
    B, V = 300, 2003
    check(torch, rng.standard_normal((B, V)) * 2, rng.random(B), **settings(rng, B), least=0.8)


def test_more_rows_than_a_grid_holds(torch):
    rng = np.random.default_rng(20)
    B, V = 66000, 6
    x = rng.standard_normal((B, V)).astype(np.float32)
    u = rng.random(B).astype(np.float32)
    token, _, _ = run(torch, x, u, temperature=np.where(np.arange(B) % 2, 1.0, 0.0))
    c = np.cumsum(np.exp(x.astype(np.float64) - x.max(1, keepdims=True)), 1)
    goal = u.astype(np.float64) * c[:, -1]
    want = np.where(np.arange(B) % 2, (c <= goal[:, None]).sum(1), x.argmax(1))
    near = (np.abs(c - goal[:, None]) < NEAR * c[:, -1:]).any(1)
    assert np.array_equal(token[~near], want[~near]) and near.sum() < 20


@pytest.mark.parametrize("B,V", [(512, 301), (1400, 300), (40, 151936)])
def test_rows_of_every_kind_in_several_waves(torch, B, V):
    """More rows than run at once, each with settings of its own: the order in
    which they are taken must not show."""
    rng = np.random.default_rng([B, V])
    check(torch, rng.standard_normal((B, V)) * 2.5, rng.random(B), least=0.8, **settings(rng, B))


def test_lists_that_nearly_or_just_overflow(torch):
    """More than the short list's 256 tokens tie with, or lie just above, the
    top-k bound; top-p whose tokens fill, or overfill, the list."""
    rng = np.random.default_rng(21)
    V = 40000
    rows, k, p = [], [], []
    for n in (255, 256, 257, 300, 5000, V):
        for kk in (1, 200, 256, 257):
            r = rng.standard_normal(V) - 30
            at = rng.permutation(V)[:n]
            r[at] = 2.0 + (rng.random(n) * 1e-3 if kk % 2 else 0.0)
            rows.append(r), k.append(kk), p.append(1.0)
        for pp in (0.3, 0.9, 0.9999):
            r = rng.standard_normal(V) - 30
            r[rng.permutation(V)[:n]] = 2.0 + rng.random(n)
            rows.append(r), k.append(0), p.append(pp)
    check(torch, np.array(rows), rng.random(len(rows)), least=0.7, top_k=k, top_p=p)


@pytest.mark.parametrize("V", [8193, 40003, 151936])
def test_the_largest_logit_in_any_slice(torch, V):
    """Many clusters in several waves, whose CTAs start at different times: each
    CTA's largest logit reaches its peers, wherever the row's largest lies."""
    rng = np.random.default_rng(V)
    B = 600
    at = np.concatenate([[0, V - 1], rng.integers(0, V, B - 2)])
    x = torch.randn(B, V, device="cuda", generator=torch.Generator("cuda").manual_seed(V))
    rows = torch.arange(B, device="cuda")
    x[rows, torch.from_numpy(at).cuda()] = 50.0
    from quantized_transformer_decode_gb300 import qw3
    u = torch.rand(B, device="cuda")
    temperature = torch.from_numpy((np.arange(B) % 2).astype(np.float32)).cuda()   # greedy and drawn: exp(-40) is left out
    for _ in range(20):
        token, prob = qw3.sample(x, u, temperature=temperature)
        assert np.array_equal(token.cpu().numpy(), at) and bool((prob > 0.999).all())


def test_largest_vocabulary(torch):
    rng = np.random.default_rng(18)
    V = 4194304
    check(torch, rng.standard_normal((2, V)), [0.3, 0.9], least=0.5, top_k=[0, 100000], top_p=[0.9, 1.0])


def test_same_tokens_every_time_and_captured(torch):
    from quantized_transformer_decode_gb300 import qw3
    rng = np.random.default_rng(19)
    B, V = 16, 151936
    x = torch.from_numpy((rng.standard_normal((B, V)) * 2).astype(np.float32)).cuda()
    u = torch.from_numpy(rng.random(B, np.float32)).cuda()
    kw = dict(temperature=torch.full((B,), 0.9, device="cuda"), top_p=torch.full((B,), 0.95, device="cuda"))
    want, wp = qw3.sample(x, u, **kw)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got, gp = qw3.sample(x, u, **kw)
    for _ in range(3):
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.equal(gp, wp)
    u.copy_(torch.from_numpy(rng.random(B, np.float32)).cuda())
    g.replay()
    assert torch.equal(got, qw3.sample(x, u, **kw)[0])


def test_wrapper_refusals(torch):
    from quantized_transformer_decode_gb300 import qw3
    x, u = torch.zeros(2, 10, device="cuda"), torch.zeros(2, device="cuda")
    for bad in (lambda: qw3.sample(x.half(), u), lambda: qw3.sample(x.t(), torch.zeros(10, device="cuda")),
                lambda: qw3.sample(x, u[:1]), lambda: qw3.sample(x, u, temperature=u.double()),
                lambda: qw3.sample(x, u, top_k=u), lambda: qw3.sample(x[0], u), lambda: qw3.sample(x[:, :0], u),
                lambda: qw3.sample(x, u.cpu())):
        with pytest.raises(qw3.Qw3Error):
            bad()
    assert qw3.sample(x[:0], u[:0])[0].numel() == 0


def test_settings_that_are_not_numbers(torch):
    """A temperature that is not finite, or a top-p or min-p that is NaN, has no
    answer; a greedy row does not look at its cuts."""
    V, nan, inf = 9001, np.nan, np.inf
    rows = np.zeros((9, V), np.float32)
    rows[:, 77] = 3.0
    token, prob, status = run(torch, rows, [0.5] * 9, temperature=[1, 1, 1, -inf, nan, inf, 0, 0, -2.0],
                              top_p=[nan, 1, 0.9, 1, 1, 1, nan, 1, 1], min_p=[0, nan, 1, 0, 0, 0, 0, nan, 0], top_k=[0, 5] + [0] * 7)
    assert status == 5
    assert token.tolist() == [-1, -1, 77, -1, -1, -1, 77, 77, 77] and prob.tolist() == [0, 0, 1, 0, 0, 0, 1, 1, 1]
    assert run(torch, rows[6:], [0.5] * 3, temperature=[0, 0, -2.0], top_p=[nan, 1, 1], min_p=[0, nan, 0])[2] == 0


@pytest.mark.parametrize("scale", [1e-30, 1e-20, 1e30, 1e37])
@pytest.mark.parametrize("V", [5003, 40009])
def test_scales_at_the_ends_of_f32(torch, scale, V):
    """Logits and temperatures of any size: what counts is their ratio."""
    rng = np.random.default_rng(V)
    B = 24
    logits = (rng.standard_normal((B, V)) * 2).astype(np.float32) * np.float32(scale)
    kw = settings(rng, B)
    kw["temperature"] = np.float32(rng.choice([1.0, 1.7], B)) * np.float32(scale)
    check(torch, logits, rng.random(B), least=0.8, **kw)


def test_probabilities_of_small_weights(torch):
    """A token far below the largest: its probability is good to 8 roundings (expf 4, a
    correction, the total, a quotient, a product of 2^-24 each)."""
    rng = np.random.default_rng(23)
    B = 4000
    x = np.stack([rng.uniform(-30, 30, B), np.zeros(B)], 1).astype(np.float32)
    temp = rng.uniform(0.3, 3, B).astype(np.float32)
    x[:, 1] = x[:, 0] - rng.uniform(2, 12, B) * temp
    w = np.exp((x[:, 1].astype(np.float64) - x[:, 0]) / temp)
    p = w / (1 + w)
    token, prob, status = run(torch, x, 1 - p / 2, temperature=temp)
    assert status == 0 and np.all(token == 1)
    assert np.all(np.abs(prob - p) <= 8 * 2.0 ** -24 * p)


def bound(V):
    """How near a border a decision may lie and still be the f64 one: weights within
    2^-29 of exact and rounded at 2^-46 of the largest (2^-40 from 2^18 tokens on), summed
    on both sides of it."""
    return 2 * (2.0 ** -29 + V * 2.0 ** (-46 if V < 2 ** 18 else -40))


def model_rows(rng, B, V):
    x = (rng.standard_normal((B, V)) * 2.2).astype(np.float32)
    for row in x:
        row[rng.integers(0, V, 400)] += (-2.5 * np.log(rng.random(400).clip(1e-6))).astype(np.float32)
    return x


def check_near(torch, logits, u, **kw):
    """Tokens as in f64, probabilities within 8 f32 roundings, in all rows beyond the
    bound; how many those are."""
    token, prob, status = run(torch, logits, u, **kw)
    clear = 0
    for i, row in enumerate(logits):
        t, p, margin = orc.sample_token(row, np.float32(u[i]), **{k: np.float32(v[i]) for k, v in kw.items()})
        if margin > bound(len(row)):
            clear += 1
            assert token[i] == t, (i, int(token[i]), t, margin)
            assert abs(prob[i] - p) <= (8 * 2.0 ** -24 + bound(len(row))) * p, (i, float(prob[i]), p)
    assert status == 0
    return clear


@pytest.mark.parametrize("V", [20011, 151936, 300007])
@pytest.mark.parametrize("temperature", [1.0, 0.7, 1.3])
def test_draws_beside_a_border(torch, V, temperature):
    """u a few 10^-8 of the total from where one token ends and the next begins."""
    rng = np.random.default_rng([V, int(temperature * 10)])
    B = 48
    x = model_rows(rng, B, V)
    u = np.empty(B, np.float32)
    for i, row in enumerate(x.astype(np.float64)):
        c = np.cumsum(np.exp((row - row.max()) / np.float64(np.float32(temperature))))
        at = int(np.argmin(np.abs(c / c[-1] - 10.0 ** rng.uniform(-4, -0.5))))
        u[i] = c[at] / c[-1] + rng.choice([-1, 1]) * rng.uniform(1, 4) * max(bound(V), 1e-9)
    assert check_near(torch, x, u, temperature=[temperature] * B) >= 0.5 * B


@pytest.mark.parametrize("V", [20011, 151936])
@pytest.mark.parametrize("temperature", [0.9, 1.7])
def test_top_p_beside_a_border(torch, V, temperature):
    """top_p a few 10^-8 of the sum from where one more token is kept."""
    rng = np.random.default_rng([V, int(temperature * 10), 1])
    B = 48
    x = model_rows(rng, B, V)
    p = np.empty(B, np.float32)
    for i, row in enumerate(x.astype(np.float64)):
        c = np.cumsum(np.sort(np.exp((row - row.max()) / np.float64(np.float32(temperature))))[::-1])
        at = int(np.argmin(np.abs(c / c[-1] - rng.uniform(0.3, 0.97))))
        p[i] = c[at] / c[-1] + rng.choice([-1, 1]) * rng.uniform(1, 4) * bound(V)
    # (p has 2^-25 to itself: some fall within the bound, or beyond the next border)
    assert check_near(torch, x, rng.random(B).astype(np.float32), temperature=[temperature] * B, top_p=p) >= 0.5 * B


def test_draws_at_large(torch):
    """Rows over a whole vocabulary, drawn as they come: no token but f64's."""
    from quantized_transformer_decode_gb300 import qw3
    V, B = 151936, 64
    x = torch.from_numpy(model_rows(np.random.default_rng(5), B, V)).cuda()
    temp = torch.from_numpy(np.resize(np.float32([1.0, 0.7, 1.1, 2.0]), B)).cuda()
    w = torch.exp((x.double() - x.double().amax(1, keepdim=True)) / temp.double()[:, None])
    c = torch.cumsum(w, 1)
    for seed in range(100):
        u = torch.from_numpy(np.random.default_rng(seed).random(B).astype(np.float32)).cuda()
        goal = u.double()[:, None] * c[:, -1:]
        want = (c <= goal).sum(1)
        near = ((c - goal).abs() < bound(V) * c[:, -1:]).any(1)
        got = qw3.sample(x, u, temperature=temp)[0].long()
        assert torch.equal(got[~near], want[~near])
        assert int((got != want).sum()) == 0 or bool(near.any())
