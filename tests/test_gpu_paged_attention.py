"""GPU parity of kda_paged_attention_decode against the float64 oracle: types,
head groups, lengths from none to many tiles, page sizes, windows, null pages,
garbage in every place that is not attended to, layouts, and repeated use."""

import numpy as np
import pytest
import torch

from linear_attention_decode_02_gb300 import binding, build
from oracle import cache_oracle as co
from tests.rounding import F32, assert_rounded, to_np

pytestmark = pytest.mark.gpu
BF16, FP32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return binding.library()


def make(lens, Hq=8, Hkv=2, D=64, page=16, dtype=BF16, seed=0, layout="token", width=None, spare=2, garbage=True,
         q_scale=1.0, packed_q=False):
    """Sequences of `lens` on shuffled pages; every position past a length, the null page and the spare pages hold
    NaN and infinities."""
    g = torch.Generator().manual_seed(seed)
    N = len(lens)
    need = [-(-max(n, 0) // page) for n in lens]
    P = width or max(1, max(need))
    need = [min(n, P) for n in need]
    pages = sum(need) + 1 + spare
    order = torch.randperm(pages - 1, generator=g) + 1
    table = torch.zeros(N, P, dtype=torch.int32)
    shape = (pages, page, Hkv, D)
    k, v = (torch.randn(shape, generator=g) for _ in range(2))
    dead = torch.ones(pages, page, dtype=torch.bool)
    at = 0
    for n in range(N):
        table[n, :need[n]] = order[at:at + need[n]]
        for i in range(need[n]):
            dead[order[at + i], :max(0, min(page, lens[n] - i * page))] = False
        at += need[n]
    if garbage:
        bad = torch.tensor([float("nan"), float("inf"), -float("inf")])
        pick = torch.randint(0, 3, shape, generator=g)
        k = torch.where(dead[..., None, None], bad[pick], k)
        v = torch.where(dead[..., None, None], bad[pick.flip(-1)], v)
    q = torch.randn(N, Hq, D, generator=g) * q_scale
    if packed_q:
        wide = torch.randn(N, (Hq + 3) * D, generator=g).to(dtype).cuda()
        wide[:, 2 * D:(Hq + 2) * D] = q.reshape(N, -1).to(dtype).cuda()
        qd = wide[:, 2 * D:(Hq + 2) * D].view(N, Hq, D)
    else:
        qd = q.to(dtype).cuda()
    k, v = k.to(dtype).cuda(), v.to(dtype).cuda()
    if layout == "head":
        k, v = (t.transpose(1, 2).contiguous().transpose(1, 2) for t in (k, v))
    elif layout in ("page pair", "token pair", "channel pair"):
        axis = {"page pair": 1, "token pair": 2, "channel pair": 3}[layout]
        kv = torch.stack([k, v], dim=axis)
        k, v = kv.select(axis, 0), kv.select(axis, 1)
    return dict(q=qd, k=k, v=v, table=table.cuda(), lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))


def run(c, **kw):
    return binding.kda_paged_attention_decode(c["q"], c["k"], c["v"], c["table"], c["lens"], return_lse=True, **kw)


def tolerances(c, scale):
    """Arithmetic error of (out, lse), by the lengths of the sums.

    A score's float32 dot product of D terms passes at most 64 roundings of 2^-24 of sum |q k| (4 to 16 terms in a
    chain, the rest in a tree).  Its error e moves a weight by e, and the normalised output by 2 e max |v|; the weight's
    exp2 and its two-piece form add 2^-16 at most in the same way.  A sum over L positions is carried by at least 8 workers,
    (L / 8 + 64) roundings of 2^-24.
    """
    q, k = to_np(c["q"]), np.nan_to_num(to_np(c["k"]), nan=0.0, posinf=0.0, neginf=0.0)
    v = np.nan_to_num(to_np(c["v"]), nan=0.0, posinf=0.0, neginf=0.0)
    dots = np.sqrt((q ** 2).sum(-1).max()) * np.sqrt((k ** 2).sum(-1).max()) * scale  # bounds sum |q k| (Cauchy)
    score = 64 * F32 * dots
    chain = (max(1, int(c["lens"].max())) / 8 + 64) * F32
    return np.abs(v).max() * (2 * score + 2.0 ** -16 + 2 * chain), score + 2.0 ** -20 + chain


def check(c, window=0, scale=None):
    D = c["q"].shape[2]
    ref, ref_lse = co.paged_attention(to_np(c["q"]), to_np(c["k"]), to_np(c["v"]), c["table"].cpu().numpy(),
                                      c["lens"].cpu().numpy(), window=window, scale=scale)
    out, lse = run(c, window=window, scale=scale)
    torch.cuda.synchronize()
    t_out, t_lse = tolerances(c, scale or D ** -0.5)
    empty = ref_lse == -np.inf
    sound = torch.tensor(np.isfinite(ref).all(-1) & ~np.isnan(ref_lse))  # attended values all finite
    assert_rounded(out.cpu()[sound], ref[sound.numpy()], t_out, "out")
    assert not torch.isfinite(out.cpu()[~sound]).any()
    assert np.array_equal(to_np(lse) == -np.inf, empty) and torch.count_nonzero(out.cpu()[torch.tensor(empty)]) == 0
    full = sound & ~torch.tensor(empty)
    assert_rounded(lse.cpu()[full], ref_lse[full.numpy()], t_lse, "lse")
    return out, lse


def same(a, b):
    """Equal bits."""
    kind = torch.int16 if a.element_size() == 2 else torch.int32
    return torch.equal(a.view(kind), b.view(kind))


LENGTHS = [1, 0, 63, 64, 65, 130, 7, 1000, 16, 17]


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (4, 2), (6, 2), (8, 2), (8, 1), (12, 1), (16, 1), (20, 1), (3, 3)])
def test_types_and_head_groups(dtype, D, Hq, Hkv):
    check(make(LENGTHS, Hq=Hq, Hkv=Hkv, D=D, dtype=dtype))


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("page", [1, 3, 7, 16, 24, 64, 100, 256])
def test_page_sizes(dtype, page):
    check(make([1, 2, 255, 256, 257, 640, 33], page=page, dtype=dtype))


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("window", [1, 5, 64, 65, 200, 10 ** 6])
def test_windows(dtype, window):
    c = make([1, 0, 64, 65, 300, 1000], dtype=dtype)
    # positions before the window may be on pages already given back
    if window < 200:
        c["table"][5, :(1000 - window) // 16] = 0
    check(c, window=window)


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_null_pages_and_rows_they_empty(dtype):
    c = make([100, 200, 50, 333, 64], dtype=dtype)
    c["table"][0, 2] = 0
    c["table"][1, 0], c["table"][1, 12] = -5, 2 ** 31 - 1
    c["table"][2, :] = 0          # nothing left
    c["table"][3, 1:] = c["k"].shape[0]
    check(c)


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_lengths_past_the_table_and_negative(dtype):
    c = make([40, 32, 16], page=8, width=4, dtype=dtype)
    c["lens"] = torch.tensor([1000, 33, -7], dtype=torch.int32, device="cuda")
    c["table"][:, :] = torch.tensor([[1, 2, 3, 4], [5, 6, 7, 8], [1, 2, 3, 4]], dtype=torch.int32)
    c["k"].nan_to_num_(0.5, 0.25, -0.25)
    c["v"].nan_to_num_(0.5, 0.25, -0.25)
    check(c)
    check(c, window=4)
    check(c, window=990)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("layout", ["token", "head", "page pair", "token pair", "channel pair"])
@pytest.mark.parametrize("packed_q", [False, True])
def test_layouts(dtype, layout, packed_q):
    check(make([70, 129, 5], Hq=6, D=128, layout=layout, packed_q=packed_q, dtype=dtype))


def test_four_element_alignment():
    # bf16 vectors on 8-byte but not 16-byte boundaries
    c = make([70, 129, 5], D=64)
    for name in ("q", "k", "v"):
        t = c[name]
        wide = torch.zeros(*t.shape[:-1], t.shape[-1] + 4, dtype=t.dtype, device="cuda")
        wide[..., 4:] = t
        c[name] = wide[..., 4:]
    check(c)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("lens", [[70001], [40000, 1, 9000], [5] * 700, [64] * 300, [1], [0, 0, 0], [0] * 9 + [20000]])
def test_splits_of_long_and_many_sequences(dtype, lens):
    check(make(lens, Hq=4, Hkv=2, D=64, dtype=dtype))


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("lens", [[30000], [5000, 1, 0, 9000], [900] * 20, [100] * 330])
def test_splits_of_units_of_many_heads(dtype, D, lens):
    check(make(lens, Hq=12, Hkv=1, D=D, page=64, dtype=dtype))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Hq,Hkv", [(5, 1), (8, 1), (9, 1), (12, 1), (16, 1), (24, 1), (32, 2)])
@pytest.mark.parametrize("width", [63, 4500])
def test_many_heads_in_narrow_and_wide_tables(D, Hq, Hkv, width):
    # float32 with many query heads: the kernel is chosen by what the table could hold
    c = make(LENGTHS, Hq=Hq, Hkv=Hkv, D=D, dtype=FP32, width=width)
    check(c)
    check(c, window=70)
    check(c, window=5000)


@pytest.mark.parametrize("Hq", [2, 8, 12])
@pytest.mark.parametrize("width", [5, 4500])
def test_values_near_the_largest_float(Hq, width):
    # Equal weights of the largest float and of nothing: half of it, which bfloat16 holds as 2^127.
    c = make([2, 70], Hq=Hq, Hkv=1, D=128, page=16, dtype=FP32, width=width, garbage=False)
    page = c["table"][0, 0]
    c["k"][page, 0] = c["k"][page, 1]
    c["v"][page, 0], c["v"][page, 1] = torch.finfo(FP32).max, 0.0
    out, _ = run(c)
    assert torch.all(out[0].float() == 2.0 ** 127) and torch.isfinite(out).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("where", ["query", "value"])
def test_many_heads_with_a_bad_query_or_value(where, bad):
    c = make([300, 70], Hq=12, Hkv=1, D=128, dtype=FP32, width=4500, garbage=False)
    good, _ = run(c)
    if where == "query":
        c["q"][0, 3, 17] = bad
    else:
        c["v"][c["table"][0, 2], 5, 0, 9] = bad
    out, _ = run(c)
    torch.cuda.synchronize()
    hit = torch.zeros_like(out, dtype=torch.bool)
    if where == "query":
        hit[0, 3] = True
    else:
        hit[0, :, 9] = True
    assert not torch.isfinite(out[hit]).any()
    assert same(out[~hit], good[~hit])


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("Hq", [2, 16])
@pytest.mark.parametrize("width", [5, 600])
def test_infinite_scores(dtype, Hq, width):
    # Head 0 scores -infinity at position 5 and loses it, head 1 scores +infinity; a lone -infinity leaves nothing.
    c = make([70, 1], Hq=Hq, Hkv=1, D=64, page=16, dtype=dtype, garbage=False, width=width)
    c["q"][:, 0::2, 0], c["q"][:, 1::2, 0] = 1.0, -1.0
    c["k"][c["table"][0, 0], 5, 0, 0] = -float("inf")
    c["k"][c["table"][1, 0], 0, 0, 0] = -float("inf")
    out, lse = run(c)
    torch.cuda.synchronize()
    k, v = to_np(c["k"]), to_np(c["v"])
    k = np.where(np.isinf(k), 0.0, k)
    at = [t for t in range(70) if t != 5]
    table = c["table"].cpu().numpy()
    rows = [(table[0, t // 16], t % 16) for t in at]
    keys, values = (np.stack([x[p, i, 0] for p, i in rows]) for x in (k, v))
    plain = dict(q=c["q"], k=torch.from_numpy(k).float(), v=c["v"], lens=c["lens"])
    t_out, t_lse = tolerances(plain, 0.125)
    for h in range(0, Hq, 2):
        s = to_np(c["q"])[0, h] @ keys.T * 0.125
        w = np.exp(s - s.max())
        assert_rounded(out[0, h].cpu(), w @ values / w.sum(), t_out, "out")
        assert_rounded(lse[0, h].cpu(), np.log(w.sum()) + s.max(), t_lse, "lse")
        assert not torch.isfinite(out[0, h + 1]).any()
        assert torch.count_nonzero(out[1, h]) == 0 and lse[1, h] == -float("inf")
        assert not torch.isfinite(out[1, h + 1]).any()


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("q_scale", [0.0, 40.0])
def test_flat_and_peaked_scores(dtype, q_scale):
    check(make([300, 65, 2000], D=128, q_scale=q_scale, dtype=dtype), scale=0.3)


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_rising_scores_rescale_at_every_step(dtype):
    c = make([513], Hq=4, Hkv=1, D=64, dtype=dtype, garbage=False)
    ramp = torch.arange(513, device="cuda").float() / 16
    flat = torch.zeros_like(c["k"]).view(-1, 1, 64)
    index = (c["table"][0].long()[:, None] * 16 + torch.arange(16, device="cuda")).flatten()[:513]
    flat[index, 0, 0] = ramp.to(dtype)
    c["k"] = flat.view_as(c["k"])
    c["q"].zero_()
    c["q"][..., 0] = 8.0
    check(c, scale=1.0)


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_shared_and_repeated_pages(dtype):
    # beams share the pages of their prefix
    c = make([200, 200, 200, 40], page=8, dtype=dtype)
    c["table"][1, :20], c["table"][2, :20] = c["table"][0, :20], c["table"][0, :20]
    check(c)


def test_cache_past_4_gib():
    pages, page = 20000, 64
    pool = torch.zeros(pages, 2, page, 8, 128, dtype=BF16, device="cuda")  # 5 GB
    g = torch.Generator(device="cuda").manual_seed(0)
    pool[-200:] = torch.randn(200, 2, page, 8, 128, device="cuda", generator=g).to(BF16)
    table = (pages - 1 - torch.arange(100, dtype=torch.int32)).reshape(4, 25).cuda()
    q = torch.randn(4, 16, 128, device="cuda", generator=g).to(BF16)
    lens = torch.tensor([1600, 1, 1599, 700], dtype=torch.int32, device="cuda")
    out = binding.kda_paged_attention_decode(q, pool[:, 0], pool[:, 1], table, lens)
    near = binding.kda_paged_attention_decode(q, pool[-200:, 0].contiguous(), pool[-200:, 1].contiguous(),
                                              table - (pages - 200), lens)
    torch.cuda.synchronize()
    assert torch.equal(out, near) and torch.count_nonzero(out) > 0


def test_out_lse_and_workspace_of_the_caller():
    c = make([100, 3000, 9])
    out, lse = check(c)
    floats = binding.kda_paged_attention_workspace(8, 2, 64, BF16,
                                                   torch.cuda.get_device_properties(0).multi_processor_count)
    work = torch.full((floats + 16,), float("nan"), device="cuda")
    mine, sums = torch.empty_like(out), torch.empty_like(lse)
    got = binding.kda_paged_attention_decode(c["q"], c["k"], c["v"], c["table"], c["lens"], out=mine, lse=sums,
                                             workspace=work)
    torch.cuda.synchronize()
    assert got is mine and torch.equal(mine, out) and torch.equal(sums, lse)
    assert torch.isnan(work[floats:]).all()  # nothing behind the workspace
    with pytest.raises(binding.KdaError, match="workspace"):
        binding.kda_paged_attention_decode(c["q"], c["k"], c["v"], c["table"], c["lens"], workspace=work[:floats - 1])
    only = binding.kda_paged_attention_decode(c["q"], c["k"], c["v"], c["table"], c["lens"])
    assert torch.equal(only, out)


def test_empty_batch():
    c = make([5, 6])
    out = binding.kda_paged_attention_decode(c["q"][:0], c["k"], c["v"], c["table"][:0], c["lens"][:0])
    assert out.shape == (0, 8, 64)


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_repeats_streams_and_graphs_give_the_same_bits(dtype):
    c = make([5000, 1, 777, 64, 0], D=128, dtype=dtype)
    out, lse = check(c)
    for _ in range(3):
        again, sums = run(c)
        assert same(again, out) and same(sums, lse)
    streams = [torch.cuda.Stream() for _ in range(3)]
    results = []
    for s in streams:  # at once, each with a workspace of its own
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            results.append(run(c))
    torch.cuda.synchronize()
    for o, e in results:
        assert same(o, out) and same(e, lse)
    graphs, outs = [], []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(run(c))
        graphs.append(graph)
    c["lens"].copy_(torch.tensor([4000, 2, 0, 65, 0], dtype=torch.int32))  # a replay reads the lengths anew
    out, lse = check(c)
    for graph in graphs + graphs:
        graph.replay()
    torch.cuda.synchronize()
    for o, e in outs:
        assert same(o, out) and same(e, lse)
