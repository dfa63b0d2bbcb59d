"""GPU parity of kda_page_assign against the sequential oracle: growth, shrinking, a ring that wraps, runs dry or
overflows, shared beginnings, null entries, padding rows, updates in place, streams and graphs.  All whole numbers."""

import random

import numpy as np
import pytest
import torch

from linear_attention_decode_02_gb300 import binding, build
from oracle import cache_oracle as co

pytestmark = pytest.mark.gpu
NAMES = ("lens", "state", "cu", "slots", "table", "ring")


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return binding.library()


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).cuda()


def make(old, new, page=16, width=None, spare=7, head=None, seed=0, shared=None, row_gap=0):
    """A table and ring that hold every page once, with `spare` pages beyond what the call asks for."""
    r = np.random.RandomState(seed)
    N = len(old)
    held = [-(-max(x, 0) // page) for x in old]
    P = width or max([1] + [-(-max(a, b, 0) // page) for a, b in zip(old, new)]) + 2
    need = sum(max(0, -(-b // page) - h) for b, h in zip(new, held) if b <= P * page)
    free = max(0, need + spare)
    C = max(1, sum(held) + free)
    order = r.permutation(C) + 1
    table = np.full((N, P), -77)
    at = 0
    for n, h in enumerate(held):
        table[n, :min(h, P)] = order[at:at + min(h, P)]
        at += h
    head = int(r.randint(C)) if head is None else head
    ring = np.full(C, -99)
    ring[(head + np.arange(free)) % C] = order[at:at + free]
    return dict(old=old, new=new, table=table, ring=ring, state=[head, free], page=page, shared=shared, row_gap=row_gap)


def call(c, rows, in_place=False):
    wide = torch.full((c["table"].shape[0], c["table"].shape[1] + c["row_gap"]), 5, dtype=torch.int32, device="cuda")
    table = wide[:, :c["table"].shape[1]]
    table.copy_(i32(c["table"]))
    ring, old, new, state = i32(c["ring"]), i32(c["old"]), i32(c["new"]), i32(c["state"])
    shared = None if c["shared"] is None else i32(c["shared"])
    kw = dict(lens_out=old, state_out=state) if in_place else {}
    lens, after, cu, slots = binding.kda_page_assign(old, new, table, ring, state, c["page"], rows, shared_lens=shared, **kw)
    if in_place:
        assert lens is old and after is state
    torch.cuda.synchronize()
    assert torch.all(wide[:, c["table"].shape[1]:] == 5)
    return lens, after, cu, slots, table, ring


def check(c, rows=None, in_place=False):
    if rows is None:
        rows = sum(max(0, b - a) for a, b in zip(c["old"], c["new"])) + 5
    ref = co.page_assign(c["old"], c["new"], c["table"], c["ring"], c["state"], c["page"], rows, c["shared"])
    got = call(c, rows, in_place)
    for name, g, e in zip(NAMES, got, ref):
        assert np.array_equal(g.cpu().numpy(), e), name
    return got


@pytest.mark.parametrize("page", [1, 3, 7, 16, 64, 1000])
@pytest.mark.parametrize("old,new", [
    ([0], [0]), ([0], [1]), ([1], [2]), ([16], [17]), ([15, 0, 64], [16, 3, 64]), ([5, 80, 33], [6, 0, 20]),
    ([100, 0, 0, 7], [0, 300, 0, 7]), ([63, 64, 65], [65, 65, 65]), ([-3, 5, -1], [4, -7, -1]),
])
def test_growing_and_shrinking(page, old, new):
    check(make(old, new, page=page))


@pytest.mark.parametrize("N", [0, 1, 2, 31, 33, 200, 256, 257, 1024, 1500, 8192])
@pytest.mark.parametrize("in_place", [False, True])
def test_many_sequences(N, in_place):
    r = random.Random(N)
    old = [r.choice([0, r.randint(0, 90)]) for _ in range(N)]
    new = [r.choice([a, a + 1, r.randint(0, 90)]) for a in old]
    check(make(old, new, page=8, spare=3), in_place=in_place)


@pytest.mark.parametrize("head", [0, 1, 40, -1])
def test_a_ring_that_wraps(head):
    c = make([100, 0, 64, 8], [0, 200, 70, 300], page=8, head=0, spare=0)
    C = len(c["ring"])
    c["ring"] = np.roll(c["ring"], head % C)
    c["state"][0] = head % C
    check(c)


@pytest.mark.parametrize("short", [1, 2, 5, 20, 1000])
def test_a_ring_that_runs_dry(short):
    # those behind the first that cannot be served still grow inside their pages, and shrink
    c = make([0, 10, 8, 30, 15], [40, 11, 50, 3, 16], page=8, spare=0)
    c["state"][1] = max(0, c["state"][1] - short)
    check(c)
    c["state"][1] = 0
    check(c)


def test_lengths_that_the_table_cannot_hold():
    c = make([8, 0, 30, 20], [9, 1000, 2 ** 31 - 1, 25], page=8, width=4)
    got = check(c, rows=20)
    assert got[0].tolist() == [9, 0, 30, 25]
    c = make([32, 32], [3, 41], page=8, width=4)
    c["old"] = [2 ** 31 - 1, 40]  # a length past the table counts as a full one
    check(c, rows=20)


def test_shared_beginnings_are_not_given_back():
    c = make([70, 70, 70, 30], [0, 20, 40, 0], page=16, shared=[32, 33, 60, 1000])
    check(c)
    c["shared"] = [-5, 0, 15, 16]
    check(c)


def test_entries_that_are_no_pages():
    c = make([100, 100, 40], [0, 10, 49], page=8)
    c["table"][0, ::3] = 0
    c["table"][1, 5], c["table"][1, 6] = -1, 2 ** 31 - 1
    c["table"][2, 4] = 0  # the page that the new rows begin on
    check(c)
    c = make([8, 8], [30, 30], page=8)
    c["ring"][:] = [2 ** 31 - 1, 0, -5, len(c["ring"]) + 1] * (len(c["ring"]) // 4) + [1] * (len(c["ring"]) % 4)
    got = check(c)
    assert (got[3] == -1).any()


@pytest.mark.parametrize("state", [[-1, 3], [10 ** 6, 3], [2, -4], [3, 10 ** 9]])
def test_states_that_are_none(state):
    c = make([20, 3], [30, 0], page=8)
    c["state"] = state
    check(c)


def test_pages_given_back_to_a_full_ring_are_dropped():
    c = make([64, 64], [0, 0], page=8, spare=2)
    c["state"] = [1, len(c["ring"]) - 5]
    got = check(c)
    assert got[1].tolist()[1] == len(c["ring"])


@pytest.mark.parametrize("rows", [0, 1, 2, 3, 4, 6, 50, 5000])
def test_rows_that_are_cut_off_or_padded(rows):
    got = check(make([5, 0, 30], [20, 17, 31], page=4), rows=rows)
    assert torch.all(got[3][33:] == -1)


@pytest.mark.parametrize("page,length", [(1, 5000), (16, 70000), (64, 300000)])
def test_long_prompts_and_their_end(page, length):
    c = make([0, 17, 0], [length, 18, length // 3], page=page)
    check(c)
    check(make([length, 17, length // 3], [0, 18, 5], page=page))


def test_strided_tables():
    check(make([5, 80, 33, 0], [6, 0, 20, 100], page=8, row_gap=3))


def test_slots_of_the_caller_off_16_bytes():
    c = make([5, 0], [30, 9], page=4)
    ref = co.page_assign(c["old"], c["new"], c["table"], c["ring"], c["state"], 4, 40)
    room = torch.full((45,), 9, dtype=torch.int32, device="cuda")
    *_, slots = binding.kda_page_assign(i32(c["old"]), i32(c["new"]), i32(c["table"]), i32(c["ring"]), i32(c["state"]), 4,
                                        40, slots=room[1:41])
    torch.cuda.synchronize()
    assert np.array_equal(slots.cpu().numpy(), ref[3]) and room[0] == 9 and torch.all(room[41:] == 9)


def test_a_second_call_on_the_same_state_gives_the_same():
    c = make([100, 0, 40, 64], [0, 50, 41, 64], page=8)
    old, new, table, ring, state = (i32(c[k]) for k in ("old", "new", "table", "ring", "state"))
    first = binding.kda_page_assign(old, new, table, ring, state, 8, 60)
    kept = [t.clone() for t in (table, ring)]
    second = binding.kda_page_assign(old, new, table, ring, state, 8, 60)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, second))
    assert torch.equal(kept[0], table) and torch.equal(kept[1], ring)


@pytest.mark.parametrize("N", [4, 300])
def test_a_life_of_requests_in_a_captured_step(N):
    """Steps replayed from one graph, lengths and ring in place: every page stays in exactly one place."""
    r = random.Random(5)
    page, width, C, rows = 4, 12, N * 6, 8 * N
    ref = dict(lens=np.zeros(N, int), table=np.zeros((N, width), int), ring=np.arange(C) + 1, state=np.array([0, C]))
    lens, table, ring, state = i32(ref["lens"]), i32(ref["table"]), i32(ref["ring"]), i32(ref["state"])
    want = torch.zeros(N, dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _, _, cu, slots = binding.kda_page_assign(lens, want, table, ring, state, page, rows, lens_out=lens, state_out=state)
    lens.zero_(), state.copy_(i32(ref["state"])), table.zero_(), ring.copy_(i32(ref["ring"]))
    for _ in range(12):
        new = [r.choice([int(a), int(a) + 1, int(a) + r.randint(1, 9), max(0, int(a) - 3), 0]) for a in ref["lens"]]
        want.copy_(i32(new))
        graph.replay()
        torch.cuda.synchronize()
        got_l, got_s, got_cu, got_x, ref["table"], ref["ring"] = co.page_assign(ref["lens"], new, ref["table"], ref["ring"],
                                                                               ref["state"], page, rows)
        ref["lens"], ref["state"] = got_l, got_s
        for g, e in ((lens, got_l), (state, got_s), (cu, got_cu), (slots, got_x), (table, ref["table"]), (ring, ref["ring"])):
            assert np.array_equal(g.cpu().numpy(), e)
        live = [int(p) for n in range(N) for p in ref["table"][n, :-(-int(got_l[n]) // page)]]
        free = [int(ref["ring"][(got_s[0] + j) % C]) for j in range(got_s[1])]
        assert sorted(live + free) == list(range(1, C + 1))


def test_streams_at_once():
    cases = [make([0, 900, 3], [5000, 0, 4], page=4, seed=s) for s in range(3)]
    refs = [co.page_assign(c["old"], c["new"], c["table"], c["ring"], c["state"], 4, 6000) for c in cases]
    inputs = [[i32(c[k]) for k in ("old", "new", "table", "ring", "state")] for c in cases]
    torch.cuda.synchronize()
    outs = []
    for x in inputs:
        with torch.cuda.stream(torch.cuda.Stream()):
            outs.append(binding.kda_page_assign(*x, 4, 6000))
    torch.cuda.synchronize()
    for x, o, ref in zip(inputs, outs, refs):
        for g, e in zip((*o, x[2], x[3]), ref):
            assert np.array_equal(g.cpu().numpy(), e)


@pytest.mark.parametrize("page", [1, 2, 3, 7, 8, 9, 15, 16, 17, 24, 33, 255, 256, 257, 300, 1000])
@pytest.mark.parametrize("seed", [0, 1])
def test_rows_that_begin_and_end_anywhere(page, seed):
    """Slots are written by pieces of a page, or of 256 rows of a larger one: every beginning and end of a sequence's rows,
    short ones among long ones, more rows than the slots hold and fewer."""
    r = random.Random(100 * page + seed)
    old = [r.choice([0, r.randint(0, 3 * page), r.randint(0, 700)]) for _ in range(90)]
    new = [a + r.choice([0, 1, 2, 5, r.randint(0, 2 * page), r.randint(0, 900)]) for a in old]
    rows = sum(max(0, b - a) for a, b in zip(old, new))
    c = make(old, new, page=page, spare=4)
    check(c, rows=rows // 2 + 1)
    check(c, rows=rows + 300)


@pytest.mark.parametrize("page", [1, 3, 16, 300])
@pytest.mark.parametrize("share", [0.0, 0.3, 0.7, 0.99, 1.0])
def test_scarce_pages_of_many_sequences(page, share):
    r = random.Random(page)
    old = [r.randint(0, 60) for _ in range(600)]
    new = [r.choice([a, a + 1, a + r.randint(0, 400), r.randint(0, 60)]) for a in old]
    c = make(old, new, page=page, spare=0)
    c["state"][1] = int(c["state"][1] * share)
    check(c)


@pytest.mark.parametrize("old, new", [
    ([1990000000, 0], [1990000700, 5]), ([7, 1990000000 - 300], [9, 1990000000 + 2 ** 20]), ([1989148671, 3], [1989148673, 0]),
])
def test_positions_near_two_to_the_31(old, new):
    c = make(old, new, page=2 ** 20, spare=2)
    check(c, rows=1200)
