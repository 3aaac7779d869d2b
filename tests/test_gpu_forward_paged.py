"""The multi-token pass over a paged cache (tiles_forward_paged) against the CPU
oracle: every sequence of a batch as if it ran alone. The bar is the dense
pass's (logits within 3e-2 + 1e-2 |oracle|, greedy choices identical except at
near-ties; the weights' BF16 rounding in a prompt's attention lies far below it).
"""
from dataclasses import replace

import numpy as np
import pytest

import oracle
import synthetic as S
from gpu_helpers import GAINS, check_forward, inputs, with_gains

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tsp():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import tile_scheduled_persistent_gb300 as t
    t.build()
    return t


def _plan(tsp, cfg, w, **opts):
    return tsp.Plan(tsp.ModelDesc.from_config(cfg), tsp.upload_weights(w), tsp.make_opts(**opts))


class Run:
    """A plan, a paged cache of n rows, and the tokens and logits of each row so far."""

    def __init__(self, tsp, cfg, n, kv_format=0, page=16, pad=0):
        self.tsp, self.cfg, self.n, self.pad = tsp, cfg, n, pad
        self.w, *_ = inputs(cfg, n_pos=0)
        self.plan = _plan(tsp, cfg, self.w)
        self.cache = tsp.PagedKV(tsp.ModelDesc.from_config(cfg), n_pages=n * -(-cfg.max_pos // page) + 2, page_size=page,
                                 n_seqs=n, kv_format=kv_format)
        self.tokens, self.logits, self.argmax = ([[] for _ in range(n)] for _ in range(3))

    def step(self, new, window=0, sinks=0, stream=None):
        """new[s]: the tokens that row s takes in this pass."""
        import torch
        lens = [len(t) + len(x) for t, x in zip(self.tokens, new)]
        ns = [len(x) for x in new]
        cu = np.concatenate([[0], np.cumsum(ns)]).astype(np.int32)
        total = int(cu[-1]) + self.pad
        flat = np.zeros(total, np.int32)
        flat[:cu[-1]] = np.concatenate([np.asarray(x, np.int32) for x in new])
        self.cache.resize(torch.tensor(lens, dtype=torch.int32, device="cuda"), stream=stream)
        am = torch.full((total,), -1, dtype=torch.int32, device="cuda")
        lg = torch.full((total, self.cfg.vocab), float("nan"), dtype=torch.float32, device="cuda")
        self.plan.forward_paged(self.cache, torch.from_numpy(flat).cuda(), am, torch.from_numpy(cu).cuda(), max(ns), window,
                                sinks, lg, stream=stream)
        self.plan.check()
        self.cache.check()
        am, lg = am.cpu().numpy(), lg.cpu().numpy()
        for s in range(self.n):
            self.tokens[s] += [int(t) for t in new[s]]
            self.argmax[s] += list(am[cu[s]:cu[s + 1]])
            self.logits[s] += list(lg[cu[s]:cu[s + 1]])
        return am[:cu[-1]]

    def check(self, what):
        for s in range(self.n):
            if self.tokens[s]:
                k = np.zeros((self.cfg.n_layers, self.cfg.n_kv_heads, self.cfg.max_pos, self.cfg.head_dim), np.uint16)
                check_forward(np.array(self.argmax[s], np.int32), np.array(self.logits[s]), self.cfg, self.w, k, k.copy(),
                              np.array(self.tokens[s], np.int32), 0, f"{what}, row {s}")


SHAPES = {
    "tiny": with_gains(S.CONFIGS["tiny"]),
    "d128_g8_qknorm": replace(S.CONFIGS["tiny"], name="p1", head_dim=128, n_q_heads=8, n_kv_heads=1, qk_norm=True,
                              rope_theta=1e6, rms_eps=1e-6, gain_sigma=GAINS),
    "g1_llama3": replace(S.CONFIGS["tiny"], name="p2", n_q_heads=2, n_kv_heads=2, hidden=264, ffn=776, vocab=1000,
                         rope_scaling=True, rope_theta=5e5, gain_sigma=GAINS),
}


@pytest.mark.parametrize("name", list(SHAPES))
def test_prompts_and_steps_of_a_batch_match_the_oracle(tsp, name):
    """Prompts of unequal lengths in one pass, single tokens, and a pass that mixes a
    late prompt, draft tokens, single tokens and rows that rest; with padding."""
    cfg = SHAPES[name]
    r = np.random.default_rng(1)
    run = Run(tsp, cfg, 4, pad=3)
    toks = lambda n: r.integers(0, cfg.vocab, n)  # noqa: E731
    last = run.step([toks(40), toks(1), toks(17), []])
    for _ in range(3):
        run.step([[last[0]], toks(1), toks(1), []])
    run.step([toks(5), toks(1), [], toks(33)])
    run.step([toks(1), [], toks(2), toks(1)])
    run.check(name)
    run.plan.close()


def test_the_batch_decodes_what_each_sequence_decodes_alone(tsp):
    """Greedy steps on the device, one token a row, against decode on the dense cache."""
    import torch
    cfg = with_gains(S.CONFIGS["tiny"])
    run = Run(tsp, cfg, 3)
    r = np.random.default_rng(2)
    prompts = [r.integers(0, cfg.vocab, n) for n in (30, 9, 1)]
    am = run.step(prompts)
    cur = [am[29], am[38], am[39]]
    outs = [[t] for t in cur]
    for _ in range(10):
        cur = run.step([[t] for t in cur])
        for o, t in zip(outs, cur):
            o.append(t)
    run.check("greedy")
    for p, o in zip(prompts, outs):
        kc = torch.zeros((cfg.n_layers, cfg.n_kv_heads, cfg.max_pos, cfg.head_dim), dtype=torch.bfloat16, device="cuda")
        t = torch.zeros(11, dtype=torch.int32, device="cuda")
        run.plan.decode(kc, kc.clone(), torch.from_numpy(p.astype(np.int32)).cuda(), 0, 11, t)
        run.plan.check()
        same = [int(a) == int(b) for a, b in zip(t.cpu().numpy(), o)]
        assert same[0] and sum(same) >= 1          # up to a near-tie (checked above against the oracle) the same
    run.plan.close()


def test_int8_cache_rows_match_the_oracles_int8_decode(tsp):
    """An INT8 paged cache without key shifts computes what the oracle's INT8 cache does
    that starts empty (its shifts are 0)."""
    cfg = with_gains(S.CONFIGS["tiny"])
    run = Run(tsp, cfg, 2, kv_format=tsp.KV_INT8)
    r = np.random.default_rng(3)
    prompts = [r.integers(0, cfg.vocab, n).astype(np.int32) for n in (25, 3)]
    for i in range(25):
        run.step([prompts[0][i:i + 1], prompts[1][i:i + 1]])
    for s, p in enumerate(prompts):
        k = np.zeros((cfg.n_layers, cfg.n_kv_heads, cfg.max_pos, cfg.head_dim), np.uint16)
        ref = oracle.decode(cfg, run.w, k, k.copy(), p, 0, 1, kv_int8=True)
        got = np.array(run.logits[s])
        assert (np.abs(got - ref.logits[:p.size]) <= 3e-2 + 1e-2 * np.abs(ref.logits[:p.size])).all()
    run.plan.close()


def test_forked_rows_continue_the_prompt(tsp):
    import torch
    cfg = with_gains(S.CONFIGS["tiny"])
    run = Run(tsp, cfg, 3)
    r = np.random.default_rng(4)
    run.step([r.integers(0, cfg.vocab, 37), [], []])
    run.cache.fork(torch.tensor([-1, 0, 0], dtype=torch.int32, device="cuda"))
    for s in (1, 2):
        for x in (run.tokens, run.argmax, run.logits):
            x[s] = list(x[0])
    for _ in range(4):
        run.step([r.integers(0, cfg.vocab, 1) for _ in range(3)])
    run.check("forked")
    run.plan.close()


def test_a_window_that_covers_everything_changes_little_and_a_small_one_much(tsp):
    cfg = with_gains(S.CONFIGS["tiny"])
    r = np.random.default_rng(5)
    prompt, more = r.integers(0, cfg.vocab, 50), r.integers(0, cfg.vocab, (6, 1))
    runs = {}
    for name, (w, k) in {"all": (0, 0), "wide": (1000, 2), "narrow": (8, 2)}.items():
        run = runs[name] = Run(tsp, cfg, 1)
        run.step([prompt], w, k)
        for x in more:
            run.step([x], w, k)
        run.plan.close()
    a, b, c = (np.array(runs[n].logits[0]) for n in ("all", "wide", "narrow"))
    assert np.array_equal(a, b)
    assert np.abs(a[:8] - c[:8]).max() <= 3e-2       # the first 8 tokens see everything either way
    assert np.abs(a[-1] - c[-1]).max() > 0.1


def test_a_captured_step_and_another_stream(tsp):
    """The batch step captured once and replayed equals the same steps launched one by one."""
    import torch
    cfg = with_gains(S.CONFIGS["tiny"])
    r = np.random.default_rng(6)
    toks = torch.from_numpy(r.integers(0, cfg.vocab, (12, 2)).astype(np.int32)).cuda()
    out = []
    for mode in ("eager", "graph", "stream"):
        run = Run(tsp, cfg, 2)
        new, tok = torch.zeros(2, dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
        am = torch.zeros(2, dtype=torch.int32, device="cuda")
        lg = torch.zeros((2, cfg.vocab), dtype=torch.float32, device="cuda")

        def step():
            run.cache.resize(new)
            run.plan.forward_paged(run.cache, tok, am, out_logits=lg)
        step()                                       # lengths 0: no token has a position; allocates
        torch.cuda.synchronize()
        g = None
        if mode == "graph":
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                step()
        st = torch.cuda.Stream() if mode == "stream" else torch.cuda.current_stream()
        st.wait_stream(torch.cuda.current_stream())
        got = []
        with torch.cuda.stream(st):
            for i in range(12):
                new.fill_(i + 1)
                tok.copy_(toks[i])
                g.replay() if g else step()
                got.append(lg.clone())
        torch.cuda.synchronize()
        run.plan.check()
        run.cache.check()
        out.append(torch.stack(got))
        del g
        run.plan.close()
    assert torch.equal(out[0], out[1]) and torch.equal(out[0], out[2]) and bool(out[0].isfinite().all())


def test_refusals(tsp):
    import torch
    cfg = with_gains(S.CONFIGS["tiny"])
    w, *_ = inputs(cfg, n_pos=0)
    plan = _plan(tsp, cfg, w)
    i32 = dict(dtype=torch.int32, device="cuda")
    t, am = torch.zeros(2, **i32), torch.zeros(300, **i32)
    cache = tsp.PagedKV(tsp.ModelDesc.from_config(cfg), n_pages=20, n_seqs=2, max_len=cfg.max_pos + 64)
    other = tsp.PagedKV(tsp.ModelDesc.from_config(replace(cfg, n_layers=1)), n_pages=20, n_seqs=2)
    for f in (lambda: plan.forward_paged(other, t, am), lambda: plan.forward_paged(cache, t[:1], am),
              lambda: plan.forward_paged(cache, am, am, torch.tensor([0, 0, 300], **i32), 300),
              lambda: plan.forward_paged(cache, t, am, window=-1), lambda: plan.forward_paged(cache, t, am, max_tokens=0)):
        with pytest.raises(tsp.TilesError) as e:
            f()
        assert e.value.status == -1
    cache.resize(torch.tensor([cfg.max_pos + 1, 1], **i32))      # a position beyond the plan's table of angles
    plan.forward_paged(cache, t, am)
    assert plan.status() == -8 and cache.status() == 0
    plan.forward_paged(cache, torch.full((2,), cfg.vocab, **i32), am)
    assert plan.status() == -8
    plan.close()
    plan = _plan(tsp, cfg, w, weight_format=tsp.WEIGHTS_INT8)
    with pytest.raises(tsp.TilesError) as e:
        plan.forward_paged(cache, t, am)
    assert e.value.status == -2
    plan.close()
