"""Page assignment, rotary positions on several axes and shared-prefix attention together, as a serving loop runs them:
prompts with pictures are admitted, their beams fork from them sharing whole pages, grow, drop rejected tokens, end and
give their pages back.  Every step is compared with the float64 oracles, and the attention with the paged call's."""

import numpy as np
import pytest
import torch

from linear_attention_decode_02_gb300 import binding, build
from oracle import cache_oracle as co
from tests.rounding import assert_rounded, to_np
from tests.test_gpu_paged_attention import tolerances

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
HQ, HKV, D, PAGE = 8, 2, 128, 8
SECTIONS = [16, 24, 24]


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return binding.library()


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).cuda()


class Server:
    """Caches and tables of `N` sequences; every call is made through the binding and checked."""

    def __init__(self, N, pages, seed):
        self.g = torch.Generator().manual_seed(seed)
        self.N, width = N, 16384  # a table wide enough for the attention to share
        self.lens, self.table = i32([0] * N), torch.zeros(N, width, dtype=torch.int32, device="cuda")
        self.ring, self.state = i32(np.arange(pages) + 1), i32([0, pages])
        self.k, self.v = (torch.full((pages + 1, PAGE, HKV, D), float("nan"), dtype=BF16, device="cuda") for _ in range(2))
        self.steps, self.axes = binding.kda_rope_phase_steps(D), binding.kda_rope_pair_axes(SECTIONS, cyclic=True)

    def assign(self, want, rows, shared=None):
        before = [t.cpu().numpy().copy() for t in (self.lens, self.table, self.ring, self.state)]
        new = i32(want)
        _, _, cu, slots = binding.kda_page_assign(self.lens, new, self.table, self.ring, self.state, PAGE, rows,
                                                  shared_lens=None if shared is None else i32(shared),
                                                  lens_out=self.lens, state_out=self.state)
        torch.cuda.synchronize()
        ref = co.page_assign(before[0], want, before[1], before[2], before[3], PAGE, rows, shared)
        for got, r in zip((self.lens, self.state, cu, slots, self.table, self.ring), ref):
            assert np.array_equal(got.cpu().numpy(), r)
        return cu.tolist(), slots

    def append(self, x, where, slots):
        q, k, v = (x[:, :HQ * D].view(-1, HQ, D), x[:, HQ * D:(HQ + HKV) * D].view(-1, HKV, D),
                   x[:, (HQ + HKV) * D:].view(-1, HKV, D))
        ref = co.rope_axes_append(to_np(q), to_np(k), to_np(v), co.rope_frequencies(D), self.axes.tolist(),
                                  where.cpu().numpy(), slots.tolist(), to_np(self.k), to_np(self.v))
        q = binding.kda_rope_axes_append(q, k, v, self.steps, self.axes, where, slots, self.k, self.v)
        torch.cuda.synchronize()
        for got, r in zip((q, self.k, self.v), ref):
            g = to_np(got)
            assert np.array_equal(np.isnan(g), np.isnan(r))
            # float32 rotation of values below 6: 2^-20 of their sum
            assert_rounded(got[~torch.isnan(got)], r[~np.isnan(r)], 2.0 ** -20 * 12, "rotary append")
        return q

    def attend(self, q, starts, prefix):
        out, lse = binding.kda_prefix_attention_decode(q, self.k, self.v, self.table, self.lens, i32(starts), i32(prefix),
                                                       return_lse=True)
        alone = binding.kda_paged_attention_decode(q, self.k, self.v, self.table, self.lens)
        ref, ref_lse = co.paged_attention(to_np(q), to_np(self.k), to_np(self.v), self.table.cpu().numpy(), self.lens.cpu().numpy())
        torch.cuda.synchronize()
        assert binding.kda_device_error() == 0
        t_out, t_lse = tolerances(dict(q=q, k=self.k, v=self.v, lens=self.lens), D ** -0.5)
        assert_rounded(out, ref, t_out, "out")
        assert_rounded(alone, ref, t_out, "alone")
        live = torch.tensor(ref_lse > -np.inf)
        assert_rounded(lse.cpu()[live], ref_lse[live.numpy()], t_lse, "lse")

    def random(self, rows):
        return torch.randn(rows, (HQ + 2 * HKV) * D, generator=self.g).to(BF16).cuda()

    def pages_in_one_place(self, shared):
        """Every page is in the ring or in one row's own part."""
        lens, table, state, ring = (t.cpu().numpy() for t in (self.lens, self.table, self.state, self.ring))
        own = [int(p) for n in range(self.N) for p in table[n, shared[n] // PAGE:-(-int(lens[n]) // PAGE)]]
        free = [int(ring[(state[0] + i) % len(ring)]) for i in range(state[1])]
        assert sorted(own + free) == list(range(1, len(ring) + 1))


def grid(rows, at):
    """Positions of a picture of `rows` patches, 7 wide, that begins at position `at`."""
    i = torch.arange(rows)
    return torch.stack([torch.full((rows,), at), at + i // 7, at + i % 7], 1).to(torch.int32).cuda()


@pytest.mark.parametrize("prompts,K,seed", [([150, 61], 3, 0), ([40, 7, 300], 4, 1), ([130] * 2, 20, 2)])
def test_prompts_beams_and_their_end(prompts, K, seed):
    G, N = len(prompts), len(prompts) * K
    s = Server(N, sum(-(-p // PAGE) for p in prompts) + 6 * N, seed)
    leaders = [g * K for g in range(G)]
    # the prompts, in the first sequence of each request
    want = [0] * N
    for g, p in zip(leaders, prompts):
        want[g] = p
    rows = sum(prompts) + 3  # padded
    cu, slots = s.assign(want, rows)
    x, where = s.random(rows), torch.cat([grid(p, 5 * i) for i, p in enumerate(prompts)] + [grid(3, 0)])
    s.append(x, where, slots)
    prompt_rows = [x[cu[g]:cu[g + 1]] for g in leaders]

    # the fork: whole pages are shared, the tokens on the last one are written again by every beam
    whole = [p // PAGE * PAGE for p in prompts]
    shared = [0 if n % K == 0 else whole[n // K] for n in range(N)]
    for n in range(N):
        g = n // K
        if n % K:
            s.table[n, :whole[g] // PAGE] = s.table[g * K, :whole[g] // PAGE]
            s.lens[n] = whole[g]
    starts, prefix = list(range(0, N + 1, K)), prompts
    lens = [prompts[n // K] for n in range(N)]
    for step in range(6):
        want = [a + 1 for a in lens]
        before = s.lens.tolist()
        rows = sum(b - a for a, b in zip(before, want)) + 2
        cu, slots = s.assign(want, rows, shared)
        fresh, x, where = s.random(rows), s.random(rows), torch.zeros(rows, 3, dtype=torch.int32, device="cuda")
        for n in range(N):
            g = n // K
            for i, pos in enumerate(range(before[n], want[n])):
                r = cu[n] + i
                if pos < prompts[g]:  # the prompt's last tokens, as its first sequence has them
                    x[r], where[r] = prompt_rows[g][pos], grid(prompts[g], 5 * g)[pos]
                else:
                    x[r], where[r] = fresh[r], pos
        q = s.append(x, where, slots)
        last = torch.tensor([c - 1 for c in cu[1:]], device="cuda")
        s.attend(q[last], starts, prefix)
        s.pages_in_one_place(shared)
        lens = want
    # drafted tokens are dropped, some beams end
    want = [max(shared[n], lens[n] - n % 5) if n % 4 else shared[n] for n in range(N)]
    s.assign(want, 4, shared)
    s.pages_in_one_place(shared)
    s.attend(s.random(N)[:, :HQ * D].view(N, HQ, D), starts, [min(p, w) for p, w in zip(whole, prompts)])
    # the end: all give back what is theirs, the first sequences the prompts too
    s.assign([0 if n % K == 0 else shared[n] for n in range(N)], 0, shared)
    assert s.state.tolist()[1] == s.ring.shape[0]
