"""The decoding-step calls as they are used: one after the other, captured, at the same time, and with attention_forward."""
import numpy as np
import pytest
import torch

import row_wise_online_gb300 as rwo
from kv4_reference import Cache, attention, np_of
from test_logits_process import args as logits_args
from test_logits_process import check as check_logits

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _built():
    from row_wise_online_gb300 import _build

    _build.build()
    torch.cuda.set_device(0)


def dev(a, dtype=torch.int32):
    return torch.as_tensor(np.asarray(a), dtype=dtype).cuda()


def angles(n, rot):
    a = np.arange(n)[:, None] * 10000.0 ** (-np.arange(rot // 2) / (rot // 2))
    return torch.from_numpy(np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)).cuda()


@pytest.mark.parametrize("dt,d,heads,group", [(BF, 128, 2, 4), (FP, 64, 3, 2)])
def test_prompts_and_decoding(dt, d, heads, group):
    """Prompts of three lengths at once, then single tokens with penalties: every call against 64 bits on what the calls before
    it left in the cache."""
    vocab, dm, page, steps = 301, 64, 16, 5
    gen = torch.Generator(device="cuda").manual_seed(4)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    hq = heads * group
    emb, wqkv, wo = rand(vocab, dm), rand(dm, (hq + 2 * heads) * d) / 8, rand(hq * d, vocab) / 8
    prompts = [[int(t) for t in torch.randint(0, vocab, (n,), generator=gen, device="cuda")] for n in (37, 5, 16)]
    B, width = 3, 4
    table = np.array([[7, 2, 9, 4], [0, 11, 3, 8], [5, 1, 10, 6]], np.int32)
    cache, cs = rwo.kv4_cache_empty(12, heads, page, d), angles(page * width, d)
    texts = [list(p) for p in prompts]
    new = prompts
    rng = np.random.default_rng(0)
    for _ in range(steps):
        cu = np.concatenate([[0], np.cumsum([len(n) for n in new])]).astype(np.int32)
        lens = [len(t) for t in texts]
        h = emb[torch.tensor([t for n in new for t in n], device="cuda")]
        q, k, v = (h @ wqkv).to(dt).view(-1, hq + 2 * heads, d).split([hq, heads, heads], 1)
        where = (cache, dev(table), dev(lens), dev(cu))
        q = rwo.kv4_append(k, v, *where, q=q, cos_sin=cs)
        lse = torch.empty(q.shape[:2], device="cuda")
        o = rwo.attention_kv4(q, *where, lse_out=lse)
        assert rwo.get_status() == rwo.OK
        want, want_lse, do, dl = attention(Cache(cache.cpu().numpy()), table, lens, cu, np_of(q), float(np.float32(d ** -0.5)))
        assert (np.abs(np_of(o) - want) <= do + torch.finfo(dt).eps / 2 * (np.abs(want) + do) + 2.0 ** -24).all()
        assert (np.abs(np_of(lse) - want_lse) <= dl).all()
        last = o[torch.from_numpy(cu[1:].astype(np.int64) - 1).cuda()].float().reshape(B, -1)
        s = {"x": (last @ wo).cpu(), "token_lens": np.array(lens), "prompt_lens": np.array([len(p) for p in prompts]),
             "tokens": np.full((B, page * width), -1), "repetition": np.full(B, 1.3), "frequency": np.full(B, 0.2),
             "presence": np.full(B, 0.1), "scale": np.full(B, 0.8),
             "mask": rng.integers(0, 2 ** 32, (B, (vocab + 31) // 32), dtype=np.uint64).astype(np.uint32)}
        for b, t in enumerate(texts):
            s["tokens"][b, :len(t)] = t
        out_lse = torch.empty(B, device="cuda")
        p = rwo.logits_process_rows(s["x"].cuda(), lse_out=out_lse, **logits_args(s))
        assert rwo.get_status() == rwo.OK
        check_logits(s, p, out_lse, "softmax", torch.float32)
        new = [[int(t)] for t in p.argmax(1)]
        for b, t in enumerate(new):
            texts[b] += t


class Step:
    """One decoding step on tensors that stay in place."""

    def __init__(self, seed, B=3, heads=2, group=4, d=128, page=16, width=40, vocab=5000):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")
        self.gen, self.hq = gen, heads * group
        self.cache = rwo.kv4_cache_empty(B * width, heads, page, d)
        self.table = torch.randperm(B * width, generator=gen, device="cuda").int().view(B, width)
        self.lens = torch.tensor([600, 33, 1], device="cuda", dtype=torch.int32)
        cu = torch.tensor([0, 600, 633, 634], device="cuda", dtype=torch.int32)
        rwo.kv4_append(rand(634, heads, d).to(BF), rand(634, heads, d).to(BF), self.cache, self.table, self.lens, cu_tokens=cu)
        self.cs = angles(page * width, d)
        self.qkv = rand(B, self.hq + 2 * heads, d).to(BF)
        self.heads, self.x = heads, rand(B, vocab)
        self.tokens = torch.randint(0, vocab, (B, 64), generator=gen, device="cuda", dtype=torch.int32)
        self.token_lens = torch.full((B,), 30, device="cuda", dtype=torch.int32)
        self.penalty = torch.full((B,), 0.3, device="cuda")

    def advance(self):
        """New inputs in the same places."""
        self.lens += 1
        self.token_lens += 1
        self.qkv.copy_(torch.randn(self.qkv.shape, generator=self.gen, device="cuda"))
        self.x.copy_(torch.randn(self.x.shape, generator=self.gen, device="cuda"))

    def run(self):
        q, k, v = self.qkv.split([self.hq, self.heads, self.heads], 1)
        where = (self.cache, self.table, self.lens)
        q = rwo.kv4_append(k, v, *where, q=q, cos_sin=self.cs)
        o = rwo.attention_kv4(q, *where)
        p = rwo.logits_process_rows(self.x, tokens=self.tokens, token_lens=self.token_lens, frequency=self.penalty)
        return o, p


def captured(step, stream):
    with torch.cuda.stream(stream):
        step.run()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            out = step.run()
    return graph, out


def test_a_captured_step_follows_its_inputs():
    eager, step = Step(1), Step(1)
    graph, out = captured(step, torch.cuda.Stream())
    eager.run()  # as the call before the capture did: it writes each sequence's last place
    for _ in range(20):
        for s in (eager, step):
            s.advance()
        graph.replay()
        want = eager.run()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)) and torch.equal(step.cache, eager.cache)
    assert rwo.get_status() == rwo.OK


def test_two_captured_steps_at_once():
    steps, streams = [Step(2), Step(3)], [torch.cuda.Stream(), torch.cuda.Stream()]
    graphs = [captured(s, t) for s, t in zip(steps, streams)]
    want = [tuple(x.clone() for x in s.run()) for s in steps]
    torch.cuda.synchronize()
    for _ in range(50):
        for (g, _), t in zip(graphs, streams):
            with torch.cuda.stream(t):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for (_, out), w in zip(graphs, want) for a, b in zip(out, w))
    assert rwo.get_status() == rwo.OK


def test_a_prompt_chunk_over_a_cached_prefix():
    """The prefix read back for attention_forward gives what attention_kv4 gives, but for the bf16 rounding of keys, values
    and weights there: a score is off by 2^-8 of its sum of magnitudes, a weight by twice that and 2^-8, a value by 2^-8."""
    heads, d, prefix, chunk = 4, 128, 333, 70
    n = prefix + chunk
    gen = torch.Generator(device="cuda").manual_seed(9)
    k, v = (torch.randn(n, heads, d, generator=gen, device="cuda").to(BF) for _ in range(2))
    q = torch.randn(chunk, heads, d, generator=gen, device="cuda").to(BF)
    cache, table = rwo.kv4_cache_empty(32, heads, 16, d), torch.randperm(32, device="cuda").int()[None]
    whole, part = torch.tensor([0, n], device="cuda", dtype=torch.int32), torch.tensor([0, chunk], device="cuda", dtype=torch.int32)
    lens = torch.tensor([n], device="cuda", dtype=torch.int32)
    rwo.kv4_append(k, v, cache, table, lens, cu_tokens=whole)
    kk, vv = (torch.empty(heads, n, d, dtype=BF, device="cuda") for _ in range(2))
    rwo.kv4_gather(cache, table, lens, cu_tokens=whole, k=kk.transpose(0, 1), v=vv.transpose(0, 1))
    a = rwo.attention_forward(q.transpose(0, 1).contiguous(), kk, vv, causal=True).transpose(0, 1)
    b = rwo.attention_kv4(q, cache, table, lens, cu_tokens=part)
    assert rwo.get_status() == rwo.OK
    big = (q.abs().float().transpose(0, 1) @ kk.abs().float().transpose(1, 2)).amax().item() / d ** 0.5
    bound = vv.abs().max().item() * (4 * 2.0 ** -8 * big + 4 * 2.0 ** -8)
    assert (a.float() - b.float()).abs().max().item() <= bound
