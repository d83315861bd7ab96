"""Speculative cycles over the paged cache against the same model without one, in float64."""
import os

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def cached():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_draft_block_gb300 import _lib, build, cached
    if not os.path.exists(_lib.LIB_PATH):
        build.build()
    return cached


def _f64(t):
    return t.detach().double().cpu().numpy()


def plain_logits(model, tokens):
    """Logits after every token of a sequence, by attention over the whole of it."""
    n, Hq, Hk, D = len(tokens), model.n_heads, model.n_kv_heads, model.head_dim

    def norm(x):
        return x / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-6)

    angle = np.arange(n)[:, None] * _f64(model.freq)
    x = _f64(model.embed)[tokens] + np.concatenate([np.sin(angle), np.cos(angle)], -1)
    for wi, wo in zip(model.qkv, model.out):
        y = (norm(x) @ _f64(wi)).reshape(n, Hq + 2 * Hk, D)
        q, k, v = y[:, :Hq], y[:, Hq:Hq + Hk], y[:, Hq + Hk:]
        o = np.zeros((n, Hq, D))
        for h in range(Hq):
            s = q[:, h] @ k[:, h * Hk // Hq].T * D ** -0.5
            s[np.triu_indices(n, 1)] = -np.inf
            w = np.exp(s - s.max(-1, keepdims=True))
            o[:, h] = w @ v[:, h * Hk // Hq] / w.sum(-1, keepdims=True)
        x = x + o.reshape(n, -1) @ _f64(wo)
    return norm(x) @ _f64(model.head) + _f64(model.E)[tokens] @ _f64(model.P)


def test_greedy_cycles_are_the_models_own_decoding(cached):
    """At temperature zero every emitted token is the largest logit of the target over the whole sequence, whatever was
    drafted; with a fork and a compaction on the way. (float32 against float64: logits of size 10, sums of up to 256
    terms in two layers, 1e-3 is a hundred times their rounding.)"""
    B, K = 5, 4
    c = cached.CachedCycle(cached.small_inputs(B, K), page_size=16, n_pages=96, max_len=160)
    rng = np.random.RandomState(3)
    seqs = [list(rng.randint(0, c.cyc.V, size=n)) for n in (1, 2, 17, 40, 33)]
    begin = [len(s) for s in seqs]
    c.prompt(seqs)
    accepted = 0
    for i in range(14):
        if i == 6:
            parent = [4, 1, 2, 4, 4]
            c.fork(torch.tensor(parent, dtype=torch.int32, device="cuda"))
            seqs, begin = [list(seqs[p]) for p in parent], [begin[p] for p in parent]
            c.cache.compact()
        c.step(100 + i)
        out, num = c.cyc.out_tokens.cpu().numpy(), c.cyc.num_emitted.cpu().numpy()
        for b in range(B):
            seqs[b] += [int(x) for x in out[b, :num[b]]]
        accepted += int(num.sum()) - B
        assert c.cache.kv_len.tolist() == [len(s) - 1 for s in seqs]
    c.check_status()
    assert accepted > 0
    assert seqs[0] == seqs[3] == seqs[4]
    for b in range(B):
        z = plain_logits(c.model, np.array(seqs[b]))
        for i in range(begin[b] - 1, len(seqs[b]) - 1):
            assert z[i].max() - z[i, seqs[b][i + 1]] <= 1e-3, (b, i)


def test_the_command(cached, capsys):
    cached.main(["--requests", "3", "--cycles", "6", "--temperature", "1.0"])
    assert "6 cycles of 3 requests" in capsys.readouterr().out


@pytest.mark.parametrize("requests,cycles", [(1, 1), (48, 4), (2, 400)])
def test_the_command_has_room_for_what_it_is_asked(cached, capsys, requests, cycles):
    """Many requests, or many cycles, pass a fixed pool or a fixed length."""
    cached.main(["--requests", str(requests), "--cycles", str(cycles)])
    assert "%d cycles of %d requests" % (cycles, requests) in capsys.readouterr().out


def test_attention_writes_the_cycles_states(cached):
    """The attention's output is the draft's hidden states as they stand (heads * head_dim = d): the confidence kernel,
    which reads the states before it waits for the draft, sees all of them."""
    from speculative_decoding_draft_block_gb300.cycle import DeviceCycle
    from speculative_decoding_draft_block_gb300.kv_cache import PagedCache
    from speculative_decoding_draft_block_gb300.workloads import B256, make_inputs, scaled
    B, K, H, D, n = 8, 8, 16, 128, 2000
    cyc = DeviceCycle(make_inputs(scaled(B256, name="states", B=B, K=K, V=2048, r=64, d=H * D, temps=(1.0,), seed=5)))
    cyc.reset_status()
    cyc.draft(1)
    g = torch.Generator(device="cuda").manual_seed(9)
    cache = PagedCache(1, B * (n // 16) + 8, 16, 4, D, B, n, dtype=torch.bfloat16)
    cache.update(torch.full((B,), n, dtype=torch.int32, device="cuda"))
    rows = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    k, v = (torch.randn((B * n, 4, D), device="cuda", generator=g).to(torch.bfloat16) for _ in range(2))
    cache.append(0, k, v, rows * n)
    start = rows * K
    out = cyc.t["h"].view(B * K, H, D)
    q = torch.zeros((B * K, H, D), device="cuda", dtype=torch.bfloat16)

    def states_and_lengths():
        out.fill_(0)
        cache.attend(0, q, start, K, out=out, causal=False)
        cyc.schedule()

    states_and_lengths()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        states_and_lengths()
    for i in range(12):
        q.copy_(torch.randn((B * K, H, D), device="cuda", generator=g) * 3)
        graph.replay() if i % 2 else states_and_lengths()
        first = cyc.conf_logit.clone()
        torch.cuda.synchronize()
        cyc.schedule()
        assert torch.equal(first, cyc.conf_logit), i
    cyc.check_status()
    cache.check_status()
