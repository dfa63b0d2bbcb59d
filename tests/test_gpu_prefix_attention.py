"""GPU parity of kda_prefix_attention_decode against the float64 oracle, which takes every sequence alone over all of its
pages: group sizes and shapes, prefixes from nothing to many tiles, ends inside pages and tiles, sequences that take no
part, windows, null pages, garbage in every place that is not attended to, layouts, and repeated use."""

import random

import numpy as np
import pytest
import torch

from linear_attention_decode_02_gb300 import binding, build
from oracle import cache_oracle as co
from tests.attention_error import assert_rms, softmax_moments
from tests.rounding import assert_rounded, to_np
from tests.test_gpu_paged_attention import same, tolerances

pytestmark = pytest.mark.gpu
BF16, FP32 = torch.bfloat16, torch.float32
SHARED = {BF16: 96 << 20, FP32: 256 << 20}  # bytes that sharing has to save at the table's width


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return binding.library()


def make(groups, Hq=8, Hkv=2, D=128, page=16, dtype=BF16, seed=0, layout="token", before=0, after=0, q_scale=1.0, spare=1,
         width=None):
    """groups: (prefix, [own positions of each sequence]); a sequence's length is their sum.  `before` and `after`
    sequences of 37 positions belong to no group.  Whole pages of a prefix are shared; what is dead holds NaN and
    infinities.  The table is as wide as it takes for the call to share, unless `width` is given."""
    g = torch.Generator().manual_seed(seed)
    seqs = [(None, 0, 37)] * before + [(i, p, t) for i, (p, tails) in enumerate(groups) for t in tails] + [(None, 0, 37)] * after
    lens = [max(0, p + t) for _, p, t in seqs]
    P = max([1] + [-(-n // page) for n in lens])
    if width is None:
        P = max(P, -(-SHARED[dtype] // (max(1, len(seqs) - len(groups)) * Hkv * D * 2 * dtype.itemsize * page)))
    P = width or P
    total = sum(-(-n // page) for n in lens) + sum(-(-p // page) for p, _ in groups)
    pages = total + 1 + spare
    order = (torch.randperm(pages - 1, generator=g) + 1).tolist()
    table = torch.zeros(len(seqs), P, dtype=torch.int32)
    shape = (pages, page, Hkv, D)
    k, v = (torch.randn(shape, generator=g) for _ in range(2))
    dead = torch.ones(pages, page, dtype=torch.bool)
    common = []
    for p, tails in groups:  # every page that the prefix reaches; the last one may end inside
        common.append([order.pop() for _ in range(-(-p // page))])
        for i, x in enumerate(common[-1]):
            dead[x, :min(page, p - i * page)] = False
    seen = set()
    for n, (i, p, t) in enumerate(seqs):
        for col in range(min(P, -(-lens[n] // page))):
            whole = i is not None and (col + 1) * page <= p
            # the first sequence keeps the page on which the prefix ends, the others have copies
            if whole or (i is not None and i not in seen and col * page < p):
                x = common[i][col]
            else:
                x = order.pop()
                if i is not None and col * page < p:
                    k[x, :p - col * page], v[x, :p - col * page] = (s[common[i][col], :p - col * page] for s in (k, v))
            table[n, col] = x
            dead[x, :max(0, min(page, lens[n] - col * page))] = False
        if i is not None:
            seen.add(i)
    for n, (i, p, t) in enumerate(seqs):  # the first sequence's row names the whole prefix, whatever its length
        if i is not None and (n == 0 or seqs[n - 1][0] != i):
            table[n, :len(common[i])] = torch.tensor(common[i], dtype=torch.int32)[:P]
    bad = torch.tensor([float("nan"), float("inf"), -float("inf")])
    pick = torch.randint(0, 3, shape, generator=g)
    k = torch.where(dead[..., None, None], bad[pick], k)
    v = torch.where(dead[..., None, None], bad[pick.flip(-1)], v)
    k, v = k.to(dtype).cuda(), v.to(dtype).cuda()
    if layout == "head":
        k, v = (t.transpose(1, 2).contiguous().transpose(1, 2) for t in (k, v))
    elif layout in ("page pair", "token pair", "channel pair"):
        axis = {"page pair": 1, "token pair": 2, "channel pair": 3}[layout]
        kv = torch.stack([k, v], dim=axis)
        k, v = kv.select(axis, 0), kv.select(axis, 1)
    q = torch.randn(len(seqs), Hq, D, generator=g) * q_scale
    starts = np.cumsum([before] + [len(tails) for _, tails in groups])
    return dict(q=q.to(dtype).cuda(), k=k, v=v, table=table.cuda(), lens=torch.tensor(lens, dtype=torch.int32).cuda(),
                starts=torch.tensor(starts, dtype=torch.int32).cuda(),
                prefix=torch.tensor([p for p, _ in groups], dtype=torch.int32).cuda())


def run(c, **kw):
    return binding.kda_prefix_attention_decode(c["q"], c["k"], c["v"], c["table"], c["lens"], c["starts"], c["prefix"],
                                               return_lse=True, **kw)


def expected(c, window=0, scale=None):
    """Every position a page of its own; the common positions of those that attend to all of them (and whose call is
    one that shares) through the first sequence's row."""
    k, v, table, lens = to_np(c["k"]), to_np(c["v"]), c["table"].cpu().numpy().astype(np.int64), c["lens"].cpu().numpy()
    pages, page = k.shape[:2]
    cap = table.shape[1] * page  # the table is mostly empty: what no sequence reaches is left out
    reached = min(cap, max([0, *lens.tolist(), *c["prefix"].tolist()]))
    table = table[:, :max(1, -(-reached // page))]
    places = np.where((table > 0) & (table < pages), table, 0)[:, :, None] * page + np.arange(page)
    places = np.where(places < page, 0, places).reshape(len(lens), -1)
    dtype, G, D = c["q"].dtype, c["q"].shape[1] // k.shape[2], k.shape[3]
    shares = (len(lens) - len(c["prefix"])) * cap * k.shape[2] * D * 2 * dtype.itemsize >= SHARED[dtype]
    shares = shares and (dtype == BF16 or (G <= 4 and D <= 128))
    starts, prefixes = c["starts"].tolist(), c["prefix"].tolist()
    if shares:
        for first, end, p in zip(starts, starts[1:], prefixes):
            p = min(max(p, 0), cap)
            for n in range(first, end):
                if min(lens[n], cap) >= p and (window == 0 or lens[n] <= window):
                    places[n, :p] = places[first, :p]
    return co.paged_attention(to_np(c["q"]), k.reshape(-1, 1, *k.shape[2:]), v.reshape(-1, 1, *v.shape[2:]), places, lens,
                              window=window, scale=scale)


def check(c, window=0, scale=None):
    ref, ref_lse = expected(c, window, scale)
    out, lse = run(c, window=window, scale=scale)
    torch.cuda.synchronize()
    assert binding.kda_device_error() == 0
    t_out, t_lse = tolerances(c, scale or c["q"].shape[2] ** -0.5)
    empty = ref_lse == -np.inf
    assert np.isfinite(ref).all()
    assert_rounded(out, ref, t_out, "out")
    assert np.array_equal(to_np(lse) == -np.inf, empty) and torch.count_nonzero(out.cpu()[torch.tensor(empty)]) == 0
    full = torch.tensor(~empty)
    assert_rounded(lse.cpu()[full], ref_lse[full.numpy()], t_lse, "lse")
    return out, lse


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_one_small_group(dtype):
    check(make([(128, [1, 2])], Hq=1, Hkv=1, dtype=dtype))


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_one_tile_and_a_bit(dtype):
    check(make([(130, [1, 20, 64])], Hq=4, Hkv=2, dtype=dtype))


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (4, 2), (6, 2), (8, 1), (12, 1), (20, 1), (3, 3)])
def test_head_groups(dtype, D, Hq, Hkv):
    check(make([(200, [1, 5, 70]), (33, [4, 4]), (517, [9])], Hq=Hq, Hkv=Hkv, D=D, dtype=dtype))


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("beams", [2, 15, 16, 17, 33, 64, 65, 100])
def test_group_sizes(dtype, D, beams):
    # 4 query heads a key head: row tiles from partly filled ones to several
    check(make([(300, [1 + i % 7 for i in range(beams)])], Hq=8, Hkv=2, D=D, page=64, dtype=dtype))


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("prefix", [1, 15, 16, 63, 64, 65, 127, 128, 129, 255, 256, 257, 1000, 5000])
def test_prefix_lengths(dtype, D, prefix):
    check(make([(prefix, [1, 30, 200])], Hq=4, Hkv=1, D=D, dtype=dtype))


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("page", [1, 3, 7, 24, 64, 100, 256])
def test_page_sizes(dtype, page):
    check(make([(333, [1, 7, 40]), (64, [64, 1])], page=page, dtype=dtype))


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_many_groups(dtype, D):
    sizes = [(i * 37 % 150 + 1, [1 + (i + j) % 9 for j in range(1 + i % 4)]) for i in range(90)]
    check(make(sizes, Hq=4, Hkv=2, D=D, dtype=dtype))


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("groups", [[(20000, [3] * 3)], [(9000, [1] * 40), (1, [5]), (4000, [100, 1])]])
def test_prefixes_in_many_pieces(dtype, D, groups):
    check(make(groups, Hq=8, Hkv=1, D=D, page=64, dtype=dtype))


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_groups_without_prefix_or_sequences_and_sequences_without_group(dtype):
    c = make([(0, [5, 9]), (100, [3, 4]), (50, []), (0, []), (200, [1])], before=3, after=2, dtype=dtype)
    check(c)
    c["starts"][:] = 0  # no group has a sequence
    check(c)
    c["starts"], c["prefix"] = c["starts"][:1], c["prefix"][:0]
    check(c)


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_sequences_that_take_no_part(dtype):
    # shorter than the prefix, of no length, of negative length, ending with it
    c = make([(150, [1, -30, -150, 0, 9]), (40, [-39, 2])], page=8, dtype=dtype)
    check(c)
    c["lens"][2] = -5
    check(c)


def test_lengths_and_prefixes_past_the_table():
    c = make([(60, [4, 4, 4])], page=8, width=8)
    c["prefix"][0] = 1000
    c["table"][1], c["table"][2] = c["table"][0].clone(), c["table"][0].clone()
    c["lens"][:] = torch.tensor([64, 2 ** 31 - 1, 70], dtype=torch.int32)
    check(c)
    c["prefix"][0] = -3
    check(c)


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_a_prefix_of_the_whole_table(dtype):
    c = make([(300, [40, 60, 5])], dtype=dtype)
    c["prefix"][0] = 2 ** 31 - 1  # as much as the table holds, mostly null pages
    c["lens"][:2] = torch.tensor([2 ** 31 - 1, 10 ** 9], dtype=torch.int32)
    c["table"][0, -3:] = c["table"][0, :3].clone()
    c["table"][1] = c["table"][0].clone()
    for n in range(2):  # pages listed past the old lengths hold garbage
        for x in set(c["table"][n].tolist()):
            c["k"][x].nan_to_num_(0.5, 0.25, -0.25), c["v"][x].nan_to_num_(0.5, 0.25, -0.25)
    check(c)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("window", [1, 64, 150, 163, 170, 10 ** 6])
def test_windows(dtype, window):
    # those that reach behind the prefix's start share it, the others do not
    check(make([(150, [1, 12, 13, 20, 64]), (5, [200, 1])], dtype=dtype), window=window)


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_null_pages(dtype):
    c = make([(200, [30, 1, 64]), (64, [5, 6])], page=16, dtype=dtype)
    c["table"][0:3, 2] = 0
    c["table"][0:3, 7] = torch.tensor([-5, -5, -5], dtype=torch.int32)
    c["table"][3:5, :4] = 2 ** 31 - 1  # nothing left of the prefix
    c["table"][1, 12] = 0  # the prefix ends on this page: its part is read through the first row
    check(c)


@pytest.mark.parametrize("layout", ["token", "head", "page pair", "token pair", "channel pair"])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_layouts_and_types(layout, dtype):
    check(make([(170, [29, 1, 5]), (64, [3, 3])], layout=layout, dtype=dtype))


def test_four_element_alignment():
    c = make([(70, [9, 5])], D=64)
    for name in ("q", "k", "v"):
        t = c[name]
        wide = torch.zeros(*t.shape[:-1], t.shape[-1] + 4, dtype=t.dtype, device="cuda")
        wide[..., 4:] = t
        c[name] = wide[..., 4:]
    check(c)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("q_scale", [0.0, 40.0])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_flat_and_peaked_scores(dtype, q_scale, D):
    check(make([(900, [65, 3])], D=D, q_scale=q_scale, dtype=dtype), scale=0.3)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("beams", [2, 70])
@pytest.mark.parametrize("step", [1 / 64, 1 / 8])
def test_rising_scores(dtype, beams, step):
    # scores that rise by less and by more a tile than the reference of the weights lets pass
    c = make([(1500, [2] * beams)], Hq=4, Hkv=1, D=64, page=4, dtype=dtype)
    ramp = (torch.arange(1500, device="cuda") * step).to(BF16).to(dtype)
    flat = c["k"].view(-1, 1, 64)
    index = (c["table"][0, :375].long()[:, None] * 4 + torch.arange(4, device="cuda")).flatten()
    flat[index] = 0.0
    flat[index, 0, 0] = ramp
    c["q"].zero_()
    c["q"][..., 0] = torch.linspace(-3, 3, c["q"].shape[0] * 4, device="cuda").to(BF16).to(dtype).view(-1, 4)
    check(c, scale=1.0)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_bad_query_spoils_its_head_alone(dtype, bad):
    c = make([(300, [9, 20, 5])], Hq=12, Hkv=1, dtype=dtype)
    good, _ = check(c)
    c["q"][1, 3, 17] = bad
    out, _ = run(c)
    torch.cuda.synchronize()
    hit = torch.zeros_like(out, dtype=torch.bool)
    hit[1, 3] = True
    assert not torch.isfinite(out[hit]).any() and same(out[~hit], good[~hit])


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_a_bad_value_spoils_its_channel_alone(dtype):
    c = make([(300, [9, 20])], Hq=12, Hkv=1, dtype=dtype)
    good, _ = check(c)
    c["v"][c["table"][0, 2], 5, 0, 9] = float("nan")
    out, _ = run(c)
    torch.cuda.synchronize()
    hit = torch.zeros_like(out, dtype=torch.bool)
    hit[:, :, 9] = True
    assert not torch.isfinite(out[hit]).any() and same(out[~hit], good[~hit])


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_infinite_scores(dtype):
    # Head 0 scores -infinity at position 5 and loses it, head 1 scores +infinity.
    c = make([(140, [9, 20])], Hq=2, Hkv=1, D=64, dtype=dtype)
    c["q"][:, 0, 0], c["q"][:, 1, 0] = 1.0, -1.0
    lost = c["k"][c["table"][0, 0], 5, 0].clone()
    c["k"][c["table"][0, 0], 5, 0, 0] = -float("inf")
    out, lse = run(c)
    torch.cuda.synchronize()
    assert not torch.isfinite(out[:, 1]).any()
    c["k"][c["table"][0, 0], 5, 0] = lost
    c["k"][c["table"][0, 0], 5, 0, 0] = -30000.0  # weighs nothing either
    ref, ref_lse = expected(c)
    c["k"][c["table"][0, 0], 5, 0, 0] = 0.0
    t_out, t_lse = tolerances(c, 0.125)
    assert_rounded(out[:, 0], ref[:, 0], t_out, "out")
    assert_rounded(lse[:, 0], ref_lse[:, 0], t_lse, "lse")


@pytest.mark.parametrize("D,beams", [(64, 16), (128, 8), (128, 40), (256, 8)])
def test_rounding_by_root_mean_square(D, beams):
    """As the paged kernel: a low part of the weights that is missing would double the mean square."""
    c = make([(3000, [50] * beams)], Hq=8, Hkv=1, D=D, page=64, seed=3)
    out, _ = run(c)
    torch.cuda.synchronize()
    k, v, table, q = to_np(c["k"]), to_np(c["v"]), c["table"].cpu().numpy(), to_np(c["q"])
    refs, ws, ss = [], [], []
    for n in range(beams):
        at = np.arange(3050)
        K, V = (x[table[n][at // 64], at % 64, 0] for x in (k, v))
        ref, _, w, s = softmax_moments(q[n], K, V, D ** -0.5)
        refs.append(ref), ws.append(w), ss.append(s)
    # a score: float32 sums of exact products, below 2^-20 by far; a weight: two pieces and exp2, 2^-16
    assert_rms(to_np(out), np.stack(refs), np.stack(ws), np.stack(ss), 2.0 ** -18, 2.0 ** -16, "out")


def test_cache_past_4_gib():
    pages, page = 20000, 64
    pool = torch.zeros(pages, 2, page, 8, 128, dtype=BF16, device="cuda")  # 5 GB
    g = torch.Generator(device="cuda").manual_seed(0)
    pool[-200:] = torch.randn(200, 2, page, 8, 128, device="cuda", generator=g).to(BF16)
    table = (pages - 1 - torch.arange(100, dtype=torch.int32)).reshape(4, 25).cuda()
    table[1:3, :20] = table[0, :20]
    q = torch.randn(4, 16, 128, device="cuda", generator=g).to(BF16)
    lens = torch.tensor([1600, 1300, 1599, 700], dtype=torch.int32, device="cuda")
    starts, prefix = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, 3], [1280]))
    out = binding.kda_prefix_attention_decode(q, pool[:, 0], pool[:, 1], table, lens, starts, prefix)
    near = binding.kda_prefix_attention_decode(q, pool[-200:, 0].contiguous(), pool[-200:, 1].contiguous(),
                                               table - (pages - 200), lens, starts, prefix)
    torch.cuda.synchronize()
    assert torch.equal(out, near) and torch.count_nonzero(out) > 0


def test_out_lse_and_workspace_of_the_caller():
    c = make([(500, [9, 30, 1]), (40, [8])])
    out, lse = check(c)
    floats = binding.kda_prefix_attention_workspace(4, 8, 2, 128, BF16,
                                                    torch.cuda.get_device_properties(0).multi_processor_count)
    work = torch.full((floats + 16,), float("nan"), device="cuda")
    mine, sums = torch.empty_like(out), torch.empty_like(lse)
    got = binding.kda_prefix_attention_decode(c["q"], c["k"], c["v"], c["table"], c["lens"], c["starts"], c["prefix"],
                                              out=mine, lse=sums, workspace=work)
    torch.cuda.synchronize()
    assert got is mine and same(mine, out) and same(sums, lse)
    assert torch.isnan(work[floats:]).all()
    with pytest.raises(binding.KdaError, match="workspace"):
        run(c, workspace=work[:floats - 1])


@pytest.mark.parametrize("groups", [[(128, [1, 2])], [(1000, [5] * 20), (60, [4, 4])]])
def test_narrow_tables_whose_sequences_are_on_their_own(groups):
    check(make(groups, width=90))


def test_groups_of_one_sequence():
    check(make([(100, [5]), (64, [1]), (700, [30])], width=5000))


def test_empty_batch():
    c = make([(20, [5, 6])])
    for k in ("q", "table", "lens"):
        c[k] = c[k][:0]
    assert run(c)[0].shape == (0, 8, 128)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("beams", [3, 60])
def test_repeats_streams_and_graphs_give_the_same_bits(dtype, beams):
    c = make([(5000, [7] * beams), (700, [80, 1])], Hq=8, Hkv=2, dtype=dtype)
    out, lse = check(c)
    for _ in range(3):
        again, sums = run(c)
        assert same(again, out) and same(sums, lse)
    results = []
    for s in [torch.cuda.Stream() for _ in range(3)]:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            results.append(run(c))
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(run(c))
        graphs.append(graph)
    c["lens"][1] = 4000  # replays read lengths and prefixes anew
    c["prefix"][1] = 650
    for o, e in results:
        assert same(o, out) and same(e, lse)
    out, lse = check(c)
    for graph in graphs + graphs:
        graph.replay()
    torch.cuda.synchronize()
    for o, e in outs:
        assert same(o, out) and same(e, lse)


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_inputs_written_just_before_the_call(dtype):
    """Nothing is waited for on the host between the kernels that write a call's inputs, over those of the last call,
    and the call: every one of its kernels reads the new ones."""
    groups = [(700, [5, 9, 30, 200]), (300, [1, 2, 60, 400]), (40, [3, 3, 3, 3])]
    cases = [make([groups[i] for i in order], Hq=16, Hkv=8, dtype=dtype, seed=seed, page=32)
             for seed, order in enumerate([(0, 1, 2), (2, 0, 1), (1, 2, 0), (2, 1, 0)])]
    wanted = [tuple(t.clone() for t in run(c)) for c in cases]
    now = {key: torch.empty_like(t) for key, t in cases[0].items()}
    out = []
    for i in range(48):
        for key, t in cases[i % 4 if i < 24 else (i * 7 // 3) % 4].items():
            now[key].copy_(t)
        out.append(tuple(t.clone() for t in run(now)))
    torch.cuda.synchronize()
    assert binding.kda_device_error() == 0
    for i, got in enumerate(out):
        for a, b in zip(got, wanted[i % 4 if i < 24 else (i * 7 // 3) % 4]):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), i


@pytest.mark.parametrize("most", [60, 130, 300])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_many_units_of_few_tiles_a_block(D, most):
    """More units than a block's slots of queries, of one tile, or one and two, or up to five: where one of two lanes that
    take tiles in turn has none, the other's queries stay where they are."""
    r = random.Random(most + D)
    groups = [(r.randint(1, most), [r.randint(1, 20) for _ in range(r.randint(2, 4))]) for _ in range(56)]
    check(make(groups, Hq=16, Hkv=16, D=D))


@pytest.mark.parametrize("window", [0, 101])
def test_many_groups_of_short_prefixes(window):
    r = random.Random(window)
    groups = [(r.choice([48, 64, 79]), [r.randint(1, 42) for _ in range(r.randint(4, 8))]) for _ in range(35)]
    check(make(groups, Hq=16, Hkv=16, D=128), window=window)


@pytest.mark.parametrize("Hq, Hkv", [(4, 1), (24, 8), (16, 16)])
def test_many_short_units_of_256_channels(Hq, Hkv):
    """Own positions of 256 channels are worked on by blocks whose warps share queries and do not meet at a unit's end."""
    r = random.Random(Hq)
    groups = [(r.choice([1, 64, 100]), [r.randint(1, 150) for _ in range(r.randint(2, 12))]) for _ in range(60)]
    c = make(groups, Hq=Hq, Hkv=Hkv, D=256)
    out, lse = check(c)
    for _ in range(20):
        again, sums = run(c)
        assert same(again, out) and same(sums, lse)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_the_last_tile_alone_is_copied_by_threads(D):
    """Whole pages of 64 come in boxes; a prefix that ends inside a page has its last tile from threads."""
    groups = [(64 * k + e, [5, 9]) for k in (1, 2, 3, 7) for e in (1, 17, 40, 63)]
    check(make(groups, Hq=16, Hkv=16, D=D, page=64))
