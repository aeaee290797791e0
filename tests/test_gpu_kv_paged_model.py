"""The paged cache, its attention and the log probabilities run together: a
whole model's layers over ragged batches, against the oracle with its half cache
("A transformer from scratch", 12.4), and Qwen3Model's scoring.

The layers around the calls are torch products in f64, rounded to f32 as the
oracle rounds them. Both sides round keys and values to half from values that
differ by their own f32 errors, so an element can land one half ulp apart: a row
of logits is held to the distance between the oracle's own rows with a half and
with an f32 cache (at least max-abs 2e-3 and rel-L2 1e-4). A log probability
moves by at most twice the largest difference of its row's logits.
"""
import numpy as np
import pytest

import paged_f64 as ref
from oracle import qw3_oracle as orc
from parity import MAX_ABS, REL_L2, assert_logits_close, build_pair, cuda_ints, row_errors
from quantized_transformer_decode_gb300 import inputs
from test_gpu_logprobs import expect

pytestmark = pytest.mark.gpu

MID = inputs.Qwen3Shape(vocab=1003, hidden=512, n_layers=2, n_heads=16, n_kv_heads=8, head_dim=128, intermediate=768, tied=True)


@pytest.fixture(scope="module")
def torch():
    import torch as t
    if not t.cuda.is_available():
        pytest.skip("no CUDA device")
    from quantized_transformer_decode_gb300 import build
    build.build()
    return t


class PagedModel:
    """The oracle's weights, its layers in torch, one paged cache to a layer."""

    def __init__(self, torch, om, n_pages, page, B, capacity):
        from quantized_transformer_decode_gb300 import qw3
        self.torch, self.qw3, self.om, self.s = torch, qw3, om, om.shape
        s = self.s
        self.w = lambda m: torch.from_numpy(np.asarray(m.w, np.float64)).cuda()
        self.vec = lambda v: torch.from_numpy(np.asarray(v, np.float32)).cuda()
        self.layers = [dict(qkv=torch.cat([self.w(l.wq), self.w(l.wk), self.w(l.wv)]), o=self.w(l.wo), g=self.w(l.wg), u=self.w(l.wu),
                            d=self.w(l.wd), an=self.vec(l.attn_norm), qn=self.vec(l.q_norm), kn=self.vec(l.k_norm), fn=self.vec(l.ffn_norm))
                       for l in om.layers]
        self.embd, self.out, self.on = self.w(om.tok_embd), self.w(om.output), self.vec(om.output_norm)
        self.caches = [qw3.KVCachePaged(n_pages, page, s.n_kv_heads, s.head_dim) for _ in om.layers]
        for c in self.caches:
            c.data.fill_(float("nan"))
        self.rope = torch.from_numpy(ref.rope_table(capacity, s.head_dim, s.rope_theta)).cuda()
        self.free = list(np.random.default_rng(7).permutation(n_pages))
        self.table = np.full((B, -(-capacity // page)), -1, np.int32)
        self.lens, self.page = np.zeros(B, np.int32), page

    def norm(self, x, w):
        x = x.double()
        return (x / self.torch.sqrt((x * x).mean(-1, keepdim=True) + self.s.rms_eps) * w.double()).float()

    def lin(self, w, x):
        return (x.double() @ w.T).float()

    def forward(self, new):
        """new: the new tokens of each sequence; logits of every row."""
        torch, s = self.torch, self.s
        for b, t in enumerate(new):
            self.lens[b] += len(t)
            for k in range(-(-int(self.lens[b]) // self.page)):
                if self.table[b, k] < 0:
                    self.table[b, k] = self.free.pop()
        starts = cuda_ints(np.concatenate(([0], np.cumsum([len(t) for t in new]))))
        where = (starts, cuda_ints(self.lens), cuda_ints(self.table.reshape(-1)).view(self.table.shape))
        x = self.embd[torch.from_numpy(np.concatenate(new)).long().cuda()].float()
        for l, c in zip(self.layers, self.caches):
            q = c.append(self.lin(l["qkv"], self.norm(x, l["an"])), *where, self.rope, l["qn"], l["kn"], s.rms_eps)
            o = c.attention(q, *where, max_rows=max(len(t) for t in new), max_len=int(self.lens.max()))
            x = x + self.lin(l["o"], o.flatten(1))
            h = self.norm(x, l["fn"])
            gate = self.lin(l["g"], h).double()
            x = x + self.lin(l["d"], (gate * torch.sigmoid(gate) * self.lin(l["u"], h).double()).float())
        return self.lin(self.out, self.norm(x, self.on))


@pytest.mark.parametrize("name,page", [("tiny", 16), ("mid", 32)])
def test_a_model_over_pages(torch, name, page):
    shape, seed = {"tiny": (inputs.TINY, 0), "mid": (MID, 3)}[name]
    om = orc.OracleModel.from_f32(shape, inputs.generate_weights(shape, seed))
    prompts = [inputs.prompt_tokens(shape, seed + i, n) for i, n in enumerate((37, 5, 80))]
    tail = [inputs.prompt_tokens(shape, seed + 9 + i, 3) for i in range(3)]
    full = [np.concatenate(v) for v in zip(prompts, tail)]
    # prompts at once and in chunks, then one, two and no tokens at a time
    steps = [(37, 0, 50), (0, 5, 30), (1, 1, 1), (2, 1, 1), (0, 1, 1)]
    pm = PagedModel(torch, om, 24, page, 3, 128)
    got, at = [[] for _ in full], [0] * 3
    for step in steps:
        new = [full[b][at[b]:at[b] + n] for b, n in enumerate(step)]
        rows = pm.forward(new)
        for b, n in enumerate(step):
            got[b].append(rows[sum(step[:b]):sum(step[:b]) + n])
            at[b] += n
    for b in range(3):
        mine = torch.cat(got[b])
        cache16, cache32 = om.new_cache(128, "f16"), om.new_cache(128)
        o16, o32 = (om.forward(c, full[b], 0, all_logits=True) for c in (cache16, cache32))
        nxt = cuda_ints(np.concatenate((full[b][1:], [-1])))
        lp, h, ids, alts = (t.cpu().numpy() for t in pm.qw3.logprobs(mine, nxt, top=5))
        mine = mine.cpu().numpy()
        for i in range(len(full[b])):
            ma, rl = row_errors(o16[i], o32[i])
            assert_logits_close(mine[i], o16[i], f"sequence {b} row {i}", max(MAX_ABS, ma), max(REL_L2, rl))
            want, entropy, order, tol, etol = expect(mine[i], [0], 5)
            assert np.array_equal(ids[i], order) and (np.abs(alts[i] - want[order]) <= tol[order]).all()
            assert abs(h[i] - entropy) <= etol
            if i + 1 < len(full[b]):
                t = int(full[b][i + 1])
                assert abs(lp[i] - want[t]) <= tol[t]
                o = np.asarray(o16[i], np.float64)
                assert abs(lp[i] - (o[t] - o.max() - np.log(np.exp(o - o.max()).sum()))) <= 2 * max(MAX_ABS, ma) + tol[t]
            else:
                assert lp[i] == -np.inf


def test_a_model_scores_text(torch):
    """Qw3Model.score: a prompt, then a chunk behind it."""
    shape, seed = inputs.TINY, 0
    om, gm = build_pair(shape, seed, max_seq_len=128, max_prefill=64)
    with gm:
        a, b = inputs.prompt_tokens(shape, seed, 40), inputs.prompt_tokens(shape, seed + 3, 21)
        cache, pos = om.new_cache(128), 0
        for tokens in (a, b):
            rows = np.asarray(om.forward(cache, tokens, pos, all_logits=True), np.float64)
            pos += len(tokens)
            lp, h, ids, alts = gm.score(0, cuda_ints(tokens), top=3)
            assert lp.shape == (len(tokens) - 1,) and h.shape == (len(tokens),) and ids.shape == alts.shape == (len(tokens), 3)
            d = rows - rows.max(-1, keepdims=True)
            want = d - np.log(np.exp(d).sum(-1, keepdims=True))
            assert np.abs(lp.cpu().numpy() - want[np.arange(len(tokens) - 1), tokens[1:]]).max() <= 2 * MAX_ABS
            # sum p |log p + 1| <= log V + 1 for each unit that the log probabilities move by
            assert np.abs(h.cpu().numpy() + (np.exp(want) * want).sum(-1)).max() <= 2 * MAX_ABS * (np.log(shape.vocab) + 1)
            best = want[np.arange(len(tokens))[:, None], ids.cpu().numpy()]
            assert np.abs(alts.cpu().numpy() - best).max() <= 2 * MAX_ABS
            assert (np.sort(want, -1)[:, ::-1][:, :3] - best <= 2 * MAX_ABS).all()
        gm.sync()
        assert gm.seq_len(0) == 61
