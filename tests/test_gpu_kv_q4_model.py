"""The 4-bit KV cache mode of the model (QW3_FLAG_KV_Q4) and sampled generation
(qw3_generate_sample) against the oracle.

The two sides encode each appended row from values that differ by the
projections' reassociation error, so a code at a border can land one step
apart. So logits are compared on identical caches: each row that the oracle
appends is replaced by the GPU's (as read back), and every forward then meets
the f32 bar of parity.py. The rows themselves are within one quantum (the
block's scale) of the oracle's, beyond the f32 cache's tolerance."""
import numpy as np
import pytest

from oracle import qw3_oracle as orc
from quantized_transformer_decode_gb300 import inputs
from parity import assert_argmax, assert_logits_close, build_pair, cuda_ints

pytestmark = pytest.mark.gpu

KV_F16, KV_Q8, Q4_K, KV_Q4, PER_KERNEL, NO_GRAPH = 0x20, 0x80, 0x100, 0x200, 0x8, 0x1
MID = inputs.Qwen3Shape(vocab=5003, hidden=1024, n_layers=2, n_heads=16, n_kv_heads=8, head_dim=128,
                        intermediate=2048, tied=True)


@pytest.fixture(scope="module")
def torch():
    import torch as t
    if not t.cuda.is_available():
        pytest.skip("no CUDA device")
    from quantized_transformer_decode_gb300 import build
    build.build()
    return t


def _np(t):
    return t.detach().cpu().numpy()


class GpuRows(orc.KvCache):
    """The oracle's cache, each appended row replaced by the GPU's."""

    def __init__(self, om, gm, seq, n):
        s = om.shape
        super().__init__(s.n_layers, s.n_kv_heads, s.head_dim, max(n, 1))
        self.rows = [[_np(x) for x in gm.read_kv(layer, seq, 0, n)] for layer in range(s.n_layers)]

    def append_layer(self, layer, k_rows, v_rows):
        super().append_layer(layer, k_rows, v_rows)
        at = slice(self.len, self.len + k_rows.shape[0])
        self.k[layer, at], self.v[layer, at] = (x[at] for x in self.rows[layer])

    def at(self, n):
        for layer, (k, v) in enumerate(self.rows):
            self.k[layer, :n], self.v[layer, :n] = k[:n], v[:n]
        self.len = n
        return self


def _step(om, gm, toks, pos, seq=0):
    """The oracle's logits of a forward of toks at pos that the GPU has done."""
    return om.forward(GpuRows(om, gm, seq, pos + len(toks)).at(pos), toks, pos)


def _greedy(shape, seed, prompt_len, steps, max_prefill=64, flags=0, chunks=None):
    cap = prompt_len + steps + 5
    om, gm = build_pair(shape, seed, max_seq_len=cap, max_prefill=max_prefill, flags=KV_Q4 | flags)
    prompt = inputs.prompt_tokens(shape, seed, prompt_len)
    try:
        lg, am = gm.prefill(0, cuda_ints(prompt))
        if prompt_len <= max_prefill:
            want = _step(om, gm, prompt, 0)
            assert_logits_close(_np(lg), want, "prefill")
        tok = int(_np(am)[0])
        first = [tok]
        for s in range(steps):
            lg, am = gm.decode(cuda_ints([tok]), [prompt_len + s])
            want = _step(om, gm, [tok], prompt_len + s)
            assert_logits_close(_np(lg)[0], want, f"step {s}")
            tok = int(_np(am)[0])
            assert_argmax(tok, orc.argmax_lowest(want), want, f"step {s}")
            first.append(tok)
        gm.sync()
        gm.truncate(0, prompt_len)
        out = gm.generate_greedy(cuda_ints(first[:1]), steps)
        assert _np(out)[:, 0].tolist() == first[1:]
    finally:
        gm.close()


def test_tiny(torch):
    w = inputs.WORKLOADS["tiny"]
    _greedy(w.shape, w.seed, w.prompt_len, w.decode_steps)


@pytest.mark.parametrize("prompt_len,max_prefill", [(9, 16), (40, 64), (300, 512)])
def test_mid(torch, prompt_len, max_prefill):
    """A chunk that attends over the codes, and chunks over rows read back (CUDA
    cores, tensor cores)."""
    _greedy(MID, 3, prompt_len, 4, max_prefill=max_prefill)


@pytest.mark.parametrize("flags", [NO_GRAPH, PER_KERNEL])
def test_launch_modes(torch, flags):
    _greedy(inputs.TINY, 0, 21, 3, flags=flags)


def test_chunks_shorter_and_longer_than_a_block(torch):
    """37 tokens in chunks of 16, 16, 5 equal the same forward in one chunk, up
    to codes at a border: each against the oracle on its own rows."""
    _greedy(inputs.TINY, 0, 37, 3, max_prefill=16)


def test_verify_block(torch):
    om, gm = build_pair(inputs.TINY, 0, max_seq_len=200, max_prefill=64, flags=KV_Q4)
    try:
        prompt = inputs.prompt_tokens(inputs.TINY, 0, 150)
        gm.prefill(0, cuda_ints(prompt[:64]), want_logits=False)
        gm.prefill(0, cuda_ints(prompt[64:120]), want_logits=False)
        for lo, hi in ((120, 125), (125, 141), (141, 142)):
            lg, am = gm.forward_all_logits(0, cuda_ints(prompt[lo:hi]))
            cache = GpuRows(om, gm, 0, hi)
            for i in range(lo, hi):
                want = om.forward(cache.at(i), [prompt[i]], i)
                assert_logits_close(_np(lg)[i - lo], want, f"row {i}")
                assert_argmax(int(_np(am)[i - lo]), orc.argmax_lowest(want), want, f"row {i}")
    finally:
        gm.close()


@pytest.mark.parametrize("B,flags", [(2, 0), (8, 0), (3, Q4_K)])
def test_batched_decode(torch, B, flags):
    shape = inputs.TINY
    if flags & Q4_K:
        om = None
        from quantized_transformer_decode_gb300.qw3 import Qw3Model
        w = inputs.generate_weights(shape, 0)
        om = orc.OracleModel.from_f32(shape, w, wtype="q4_k")
        gm = Qw3Model.from_f32(shape, inputs.iter_weights(shape, 0), max_seqs=B, max_seq_len=96, max_prefill=32,
                               flags=KV_Q4 | flags)
    else:
        om, gm = build_pair(shape, 0, max_seqs=B, max_seq_len=96, max_prefill=32, flags=KV_Q4)
    pos, seqs = [3 + 9 * b for b in range(B)], list(range(B))[::-1]
    try:
        toks = []
        for b in range(B):
            _, am = gm.prefill(seqs[b], cuda_ints(inputs.batch_prefix_tokens(shape, 0, b, pos[b])), want_logits=False)
            toks.append(int(_np(am)[0]))
        for _ in range(3):
            lg, am = gm.decode(cuda_ints(toks), pos, seqs=seqs)
            for b in range(B):
                want = _step(om, gm, [toks[b]], pos[b], seqs[b])
                assert_logits_close(_np(lg)[b], want, f"sequence {b} at {pos[b]}")
                assert_argmax(int(_np(am)[b]), orc.argmax_lowest(want), want, f"sequence {b}")
            toks, pos = [int(t) for t in _np(am)], [p + 1 for p in pos]
    finally:
        gm.close()


def test_cache_contents(torch):
    shape = inputs.TINY
    om, gm = build_pair(shape, 0, max_seq_len=64, max_prefill=16, flags=KV_Q4)
    try:
        prompt = inputs.prompt_tokens(shape, 0, 21)
        raw = om.new_cache(64)
        om.forward(raw, prompt, 0)
        gm.prefill(0, cuda_ints(prompt), want_logits=False)
        for layer in range(shape.n_layers):
            for got, rows, name in zip(map(_np, gm.read_kv(layer, 0, 0, 21)), (raw.k, raw.v), "KV"):
                codes, scales = orc.kv_q4_encode(rows[layer, :21])
                quantum = np.repeat(np.abs(scales.astype(np.float32)), 32, axis=-1)
                if layer == 0:
                    # the same inputs: equal but for codes at a border
                    assert np.mean(got == orc.kv_q4_decode(codes, scales)) > 0.98, name
                    assert np.abs(got - orc.kv_q4_decode(codes, scales)).max() <= 1.01 * quantum.max() + 1e-4
    finally:
        gm.close()


def test_one_cache_type(torch):
    from quantized_transformer_decode_gb300.qw3 import Qw3Error, Qw3Model
    for other in (KV_F16, KV_Q8):
        with pytest.raises(Qw3Error):
            Qw3Model.from_f32(inputs.TINY, inputs.iter_weights(inputs.TINY, 0), max_seq_len=16, max_prefill=16,
                              flags=KV_Q4 | other)


def test_launch_count(torch):
    _, gm = build_pair(inputs.TINY, 0, max_seq_len=64, max_prefill=16, flags=KV_Q4)
    assert gm.decode_plan(1) == (False, 2 + 5 * inputs.TINY.n_layers + inputs.TINY.n_layers)
    gm.close()


# ---------------------------------------------------------------- sampled generation

@pytest.mark.parametrize("flags", [0, PER_KERNEL, KV_Q4])
@pytest.mark.parametrize("B", [1, 3, 6])
def test_generate_sample(torch, B, flags):
    """Each token is the sampler's on the logits of its step (had again by
    teacher-forced decode steps, which are bit-identical)."""
    shape, steps = inputs.TINY, 6
    _, gm = build_pair(shape, 0, max_seqs=B, max_seq_len=96, max_prefill=32, flags=flags)
    rng = np.random.default_rng([B, flags])
    f = lambda x: torch.tensor(x, dtype=torch.float32, device="cuda")  # noqa: E731
    pos, seqs = [4 + 5 * b for b in range(B)], list(range(B))[::-1]
    try:
        first = []
        for b in range(B):
            _, am = gm.prefill(seqs[b], cuda_ints(inputs.batch_prefix_tokens(shape, 0, b, pos[b])), want_logits=False)
            first.append(int(_np(am)[0]))
        temp, k, p, mp = [0.8, 0.0, 1.3, 0.5, 1.0, 2.0][:B], [50, 0, 0, 7, 1000, 0][:B], [0.9, 1.0, 0.8, 1.0, 0.95, 1.0][:B], \
            [0.0, 0.0, 0.01, 0.0, 0.1, 0.0][:B]
        u = rng.random((steps, B)).astype(np.float32)
        out, prob = gm.generate_sample(cuda_ints(first), steps, f(u), temperature=f(temp), top_k=cuda_ints(k), top_p=f(p),
                                       min_p=f(mp), seqs=seqs)
        gm.sync()
        out, prob = _np(out), _np(prob)
        assert [gm.seq_len(s) for s in seqs] == [n + steps for n in pos]
        for b in range(B):
            gm.truncate(seqs[b], pos[b])
        toks, clear = first, 0
        for s in range(steps):
            lg, _ = gm.decode(cuda_ints(toks), [n + s for n in pos], seqs=seqs)
            for b in range(B):
                t, pr, margin = orc.sample_token(_np(lg)[b], u[s, b], np.float32(temp[b]), k[b], np.float32(p[b]), np.float32(mp[b]))
                if margin > 4e-6:
                    clear += 1
                    assert out[s, b] == t and abs(prob[s, b] - pr) <= 8e-6 * pr
            toks = [int(t) for t in out[s]]
        assert clear >= 0.8 * B * steps
    finally:
        gm.close()


def test_generate_sample_without_settings_and_greedy(torch):
    shape = inputs.TINY
    _, gm = build_pair(shape, 0, max_seqs=2, max_seq_len=64, max_prefill=32)
    try:
        first = []
        for b in range(2):
            _, am = gm.prefill(b, cuda_ints(inputs.batch_prefix_tokens(shape, 0, b, 8)), want_logits=False)
            first.append(int(_np(am)[0]))
        want = _np(gm.generate_greedy(cuda_ints(first), 5))
        for b in range(2):
            gm.truncate(b, 8)
        u = torch.rand(5, 2, device="cuda")
        got, prob = gm.generate_sample(cuda_ints(first), 5, u, temperature=torch.zeros(2, device="cuda"))
        assert np.array_equal(_np(got), want) and _np(prob).tolist() == [[1.0, 1.0]] * 5
        got, _ = gm.generate_sample(cuda_ints(first), 5, u)
        assert _np(got).min() >= 0 and _np(got).max() < shape.vocab
        gm.sync()
    finally:
        gm.close()


def test_generate_sample_refusals(torch):
    from quantized_transformer_decode_gb300 import qw3
    _, gm = build_pair(inputs.TINY, 0, max_seqs=2, max_seq_len=32, max_prefill=16)
    try:
        buf = torch.zeros(2 * inputs.TINY.vocab, device="cuda")
        p = buf.data_ptr()
        call = lambda B=1, n=1, first=p, u=p, lg=p, out=p, seqs=None, temp=0: qw3.qw3_generate_sample(  # noqa: E731
            gm.h, B, seqs, n, first, temp, 0, 0, 0, u, lg, out)
        for kw, status in ((dict(B=0), 1), (dict(B=3), 1), (dict(n=-1), 1), (dict(first=0), 1), (dict(u=0), 1),
                           (dict(lg=0), 1), (dict(out=0), 1), (dict(u=p + 2), 1), (dict(temp=p + 1), 1),
                           (dict(B=2, seqs=[1, 1]), 1), (dict(seqs=[2]), 1), (dict(n=33), 4)):
            with pytest.raises(qw3.Qw3Error) as e:
                call(**{**dict(first=p), **kw})
            assert e.value.status == status, kw
        call(n=0)
        assert gm.seq_len(0) == 0 and gm.seq_len(1) == 0
        u = torch.rand(2, 2, device="cuda")
        with pytest.raises(qw3.Qw3Error):
            gm.generate_sample(cuda_ints([1, 2]), 3, u)
    finally:
        gm.close()


def test_generate_sample_null_model(torch):
    from quantized_transformer_decode_gb300 import qw3
    assert qw3.lib().qw3_generate_sample(None, 1, None, 1, 16, None, None, None, None, 16, 16, 16, None) == 1
