"""The operators together: a beam search over a small decoder with one recurrent
(KDA) layer and one attention layer, as a serving loop would run it: fused KDA
decode, rotary append, paged attention, beam selection, and the move of states,
conv caches and pages to the surviving beams.

The proof is a replay: every surviving hypothesis, fed token by token without
any reordering, must reach the same recurrent state, conv cache, cached keys and
values, and the same score, bit for bit.  (Sequences stay within one tile of the
attention kernel, so a row's arithmetic does not depend on its place.)
"""

import numpy as np
import pytest
import torch

from linear_attention_decode_02_gb300 import binding, build
from oracle import cache_oracle as co
from tests.rounding import to_np

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
H, HQ, HKV, D, V, PAGE = 2, 4, 2, 64, 211, 4  # recurrent heads, attention heads, vocabulary, page size


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return binding.library()


class Decoder:
    """Weights of one recurrent and one attention layer; float64 products keep a row's result independent of its place."""

    def __init__(self, seed):
        g = torch.Generator().manual_seed(seed)
        normal = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
        E = H * 128
        self.embed = normal(V, E)
        self.to_qkv, self.to_gate, self.to_out = normal(E, 3 * E) / 16, normal(E, 2 * E) / 16, normal(E, H) / 16
        self.conv, self.norm = normal(3, 4, E) / 2, torch.ones(128).cuda()
        self.A_log, self.dt_bias = torch.zeros(H).cuda(), normal(E) / 10
        self.attn = normal(E, (HQ + 2 * HKV) * D) / 16
        self.head = normal(HQ * D + E, V) / 4
        self.steps = binding.kda_rope_phase_steps(D // 2, base=10000.0)
        self.bias = torch.zeros(V).cuda()

    def mul(self, x, w):
        return x.double() @ w.double()

    def step(self, tokens, slots, caches, table, lens):
        """Logits [B, V] of the next token after `tokens` at positions lens - 1; updates the caches in place."""
        state, conv, k_pages, v_pages = caches
        B = tokens.shape[0]
        x = self.embed[tokens.long()]
        qkv, gates, beta = self.mul(x, self.to_qkv).to(BF16), self.mul(x, self.to_gate).to(BF16), self.mul(x, self.to_out).to(BF16)
        gate, out_gate = gates.view(B, 2, H, 128).unbind(1)
        y = binding.kda_fused_decode(qkv, self.conv, conv, gate, beta, self.A_log, self.dt_bias, slots, state, out_gate,
                                     self.norm).view(B, H * 128)
        p = self.mul(y, self.attn).to(BF16)
        q, k, v = (p[:, :HQ * D].view(B, HQ, D), p[:, HQ * D:(HQ + HKV) * D].view(B, HKV, D),
                   p[:, (HQ + HKV) * D:].view(B, HKV, D))
        q = binding.kda_rope_append(q, k, v, self.steps, lens, table, k_pages, v_pages)
        o = binding.kda_paged_attention_decode(q, k_pages, v_pages, table, lens).view(B, HQ * D)
        return (self.mul(torch.cat([o, y], 1), self.head) + self.bias).float()


def caches(slots, pages):
    conv = torch.zeros(slots, 3, 3 * H * 128, dtype=BF16, device="cuda").permute(0, 2, 1)
    return (torch.zeros(slots, H, 128, 128, device="cuda"), conv,
            torch.full((pages, PAGE, HKV, D), float("nan"), dtype=BF16, device="cuda"),
            torch.full((pages, PAGE, HKV, D), float("nan"), dtype=BF16, device="cuda"))


def same_bits(a, b):
    kind = torch.int16 if a.element_size() == 2 else torch.int32
    return torch.equal(a.contiguous().view(kind), b.contiguous().view(kind))


@pytest.mark.parametrize("N,K,steps,seed", [(1, 4, 11, 0), (3, 3, 14, 1), (2, 8, 9, 2)])
def test_beam_search_equals_the_replay_of_its_hypotheses(N, K, steps, seed):
    model = Decoder(seed)
    model.bias[5] = 2.0  # a token that ends a hypothesis is drawn now and then
    B, P = N * K, -(-(steps + 1) // PAGE)
    pool = caches(B + 1, B * P + 1)
    slots = torch.arange(1, B + 1, dtype=torch.int32, device="cuda")
    table = torch.arange(1, B * P + 1, dtype=torch.int32, device="cuda").view(B, P)
    pages = table.view(N, K, P)
    tokens = torch.arange(B, dtype=torch.int32, device="cuda") // K + 7  # a start token for each request
    scores = torch.full((N, K), -np.inf, device="cuda")
    scores[:, 0] = 0.0
    finished = torch.zeros(N, K, dtype=torch.int32, device="cuda")
    history = tokens.view(N, K, 1)
    for t in range(1, steps + 1):
        lens = torch.full((B,), t, dtype=torch.int32, device="cuda")
        logits = model.step(tokens, slots, pool, table, lens).view(N, K, V)
        before = (scores.clone(), finished.clone())
        scores, parents, picked = binding.kda_beam_select(logits, scores, K, finished=finished, eos_token=5)
        ref = co.beam_select(to_np(logits), to_np(before[0]), K, finished=before[1].cpu().numpy(), eos_token=5)
        assert np.array_equal(parents.cpu().numpy(), ref[1]) and np.array_equal(picked.cpu().numpy(), ref[2])
        assert int(parents.min()) >= 0
        # states and conv caches by slot; every page of the parent to the same page of its heir
        mine = slots.view(N, K)
        binding.kda_pool_move([pool[0], pool[1]], mine, mine, parents=parents)
        for i in range(-(-t // PAGE)):
            own = pages[:, :, i].contiguous()
            binding.kda_pool_move([pool[2], pool[3]], own, own, parents=parents)
        at = parents.long()
        finished = torch.gather(finished, 1, at) | (picked == 5).to(torch.int32)
        history = torch.cat([torch.gather(history, 1, at[..., None].expand(-1, -1, t)), picked[..., None]], 2)
        tokens = picked.reshape(B)
    torch.cuda.synchronize()

    # replay: the hypotheses as they stand, each in its row
    again = caches(B + 1, B * P + 1)
    hist = history.reshape(B, steps + 1)
    total = torch.zeros(B, dtype=torch.float64, device="cuda")
    ended = torch.zeros(B, dtype=torch.bool, device="cuda")
    for t in range(1, steps + 1):
        lens = torch.full((B,), t, dtype=torch.int32, device="cuda")
        logits = model.step(hist[:, t - 1], slots, again, table, lens)
        gain = torch.log_softmax(logits.double(), -1).gather(1, hist[:, t, None].long())[:, 0]
        total += torch.where(ended, 0.0, gain)
        ended |= hist[:, t] == 5
    torch.cuda.synchronize()
    for a, b, what in zip(pool, again, ("state", "conv cache", "keys", "values")):
        assert same_bits(a, b), what
    # a float32 rounding of the score at every step: 2^-24 of at most its last size
    got, want = to_np(scores.view(B)), to_np(total)
    assert np.all(np.abs(got - want) <= steps * (2.0 ** -24 * np.abs(want) + 2.0 ** -16))
    assert (scores[:, 1:] <= scores[:, :-1]).all()


def test_a_step_of_the_search_replays_from_a_graph():
    # rotary append, attention, selection and move captured once and replayed with new lengths
    N, K, P = 2, 4, 5
    B = N * K
    g = torch.Generator().manual_seed(3)
    pool = caches(B + 1, B * P + 1)
    for t in pool[2:]:
        t.copy_(torch.randn(t.shape, generator=g))
    pool[0].copy_(torch.randn(pool[0].shape, generator=g))
    table = torch.arange(1, B * P + 1, dtype=torch.int32, device="cuda").view(B, P)
    qkv = torch.randn(B, (HQ + 2 * HKV) * D, generator=g).to(BF16).cuda()
    head = torch.randn(HQ * D, V, generator=g).cuda().to(BF16)
    slots = torch.arange(1, B + 1, dtype=torch.int32, device="cuda").view(N, K)
    scores = torch.randn(N, K, generator=g).cuda()
    steps = binding.kda_rope_phase_steps(D)
    lens = torch.full((B,), 6, dtype=torch.int32, device="cuda")

    def step(pool):
        q, k, v = (qkv[:, :HQ * D].view(B, HQ, D), qkv[:, HQ * D:(HQ + HKV) * D].view(B, HKV, D),
                   qkv[:, (HQ + HKV) * D:].view(B, HKV, D))
        q = binding.kda_rope_append(q, k, v, steps, lens, table, pool[2], pool[3])
        o = binding.kda_paged_attention_decode(q, pool[2], pool[3], table, lens)
        logits = (o.view(B, HQ * D) @ head).view(N, K, V)
        s, parents, tokens = binding.kda_beam_select(logits, scores, K)
        binding.kda_pool_move([pool[0], pool[1]], slots, slots, parents=parents)
        return s, parents, tokens

    start = [t.clone() for t in pool]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(pool)  # warm-up, outside the capture
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(pool)
    for length in (6, 17, 20, 1):
        for t, t0 in zip(pool, start):
            t.copy_(t0)
        lens.fill_(length)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (*out, *pool)]
        fresh = [t.clone() for t in start]
        want = [*step(fresh), *fresh]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert same_bits(a, b)


def test_kept_workspaces_are_per_thread_stream_and_capture():
    import threading
    q = torch.randn(2, 8, 64, device="cuda").to(BF16)
    pages = torch.randn(9, 16, 2, 64, device="cuda").to(BF16)
    table = torch.arange(1, 9, dtype=torch.int32, device="cuda").view(2, 4)
    lens = torch.tensor([60, 33], dtype=torch.int32, device="cuda")
    want = binding.kda_paged_attention_decode(q, pages, pages, table, lens)
    torch.cuda.synchronize()

    def grown(f):  # bytes that f leaves allocated
        torch.cuda.synchronize()
        before = torch.cuda.memory_allocated()
        f()
        torch.cuda.synchronize()
        return torch.cuda.memory_allocated() - before

    call = lambda: binding.kda_paged_attention_decode(q, pages, pages, table, lens)  # noqa: E731
    floats = binding.kda_paged_attention_workspace(8, 2, 64, BF16, torch.cuda.get_device_properties(0).multi_processor_count)
    assert grown(call) == 0                       # this thread's workspace on this stream is there already
    stream = torch.cuda.Stream()

    def on_stream():
        with torch.cuda.stream(stream):
            assert torch.equal(call(), want)
    assert grown(on_stream) >= 4 * floats         # another stream has its own
    assert grown(on_stream) == 0
    kept = []

    def in_thread():
        t = threading.Thread(target=lambda: kept.append(grown(call)))
        t.start()
        t.join()
    assert grown(in_thread) < 4 * floats and kept[0] >= 4 * floats  # another thread too, and it goes with the thread
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    graph.replay()
    assert torch.equal(call(), want) and torch.equal(out, want)


def test_calls_refuse_host_tensors():
    i = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="host"):
        binding.kda_pool_move([torch.zeros(2, 2)], i, i)
    with pytest.raises(ValueError, match="host"):
        binding.kda_beam_select(torch.zeros(1, 2, 9, device="cuda"), torch.zeros(1, 2), 2)
    with pytest.raises(TypeError, match="list or tuple"):
        binding.kda_pool_move(torch.zeros(2, 2, device="cuda"), i, i)
