"""GPU parity of kda_rope_append against the float64 oracle: both layouts, partial
and no rotation, far positions, ragged rows, padding and null rows, null pages,
strided pages and packed inputs, in place, on other streams and in graphs."""

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


def make(lens, new=None, Hq=4, Hkv=2, D=64, rot=None, page=16, dtype=BF16, pdtype=BF16, seed=0, pad=0, packed=True,
         head_major=False, interleaved_kv=False, width=None):
    """One call's inputs; new=None: one row per sequence without cu_seqlens."""
    g = torch.Generator().manual_seed(seed)
    N = len(lens)
    rows = (N if new is None else sum(new)) + pad
    rot = D if rot is None else rot

    def normal(*shape, dtype=dtype):
        return torch.randn(*shape, generator=g).to(dtype)

    c = {}
    if packed:
        x = normal(rows, (Hq + 2 * Hkv) * D).cuda()
        c["q"], c["k"], c["v"] = (x[:, :Hq * D].view(rows, Hq, D), x[:, Hq * D:(Hq + Hkv) * D].view(rows, Hkv, D),
                                  x[:, (Hq + Hkv) * D:].view(rows, Hkv, D))
    else:
        c["q"], c["k"], c["v"] = normal(rows, Hq, D).cuda(), normal(rows, Hkv, D).cuda(), normal(rows, Hkv, D).cuda()
    P = width or max(1, -(-max(lens + [1]) // page))
    touched = []
    count = [t if new is None else t for t in ([1] * N if new is None else new)]
    table = torch.zeros(N, P, dtype=torch.int32)
    for n in range(N):
        for col in range(max(0, lens[n] - count[n]) // page, min(P, -(-max(lens[n], 0) // page))):
            touched.append((n, col))
    order = torch.randperm(len(touched), generator=g)
    for i, (n, col) in enumerate(touched):
        table[n, col] = int(order[i]) + 1
    pages = len(touched) + 1
    if interleaved_kv:
        kv = normal(pages, 2, page, Hkv, D, dtype=pdtype).cuda()
        c["k_pages"], c["v_pages"] = kv[:, 0], kv[:, 1]
    elif head_major:
        c["k_pages"] = normal(pages, Hkv, page, D, dtype=pdtype).cuda().transpose(1, 2)
        c["v_pages"] = normal(pages, Hkv, page, D, dtype=pdtype).cuda().transpose(1, 2)
    else:
        c["k_pages"], c["v_pages"] = (normal(pages, page, Hkv, D, dtype=pdtype).cuda() for _ in range(2))
    c["table"] = table.cuda()
    c["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    c["cu"] = None if new is None else torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32, device="cuda")
    c["rot"] = rot
    return c


def call(c, interleaved=False, amplitude=1.0, scaling=None, q_out=None):
    steps = binding.kda_rope_phase_steps(c["rot"], **(scaling or {}))
    return binding.kda_rope_append(c["q"], c["k"], c["v"], steps, c["lens"], c["table"], c["k_pages"], c["v_pages"],
                                   cu_seqlens=c["cu"], interleaved=interleaved, amplitude=amplitude, q_out=q_out)


def oracle(c, interleaved=False, amplitude=1.0, scaling=None):
    freq = co.rope_frequencies(c["rot"], **(scaling or {}))
    cu = None if c["cu"] is None else c["cu"].cpu().numpy()
    return co.rope_append(to_np(c["q"]), to_np(c["k"]), to_np(c["v"]), freq, c["lens"].cpu().numpy(),
                          c["table"].cpu().numpy(), to_np(c["k_pages"]), to_np(c["v_pages"]), cu_seqlens=cu,
                          interleaved=interleaved, amplitude=amplitude)


def slack(c, amplitude):
    """Float32 arithmetic of a cos t - b sin t with |a|, |b| <= X: t off by its rounding to float32 (pi 2^-24), cosine
    and sine by 2 units each (2^-22), times the amplitude, two products and a sum (3 more half steps): below 2^-20 of
    (|a| + |b|) * amplitude."""
    X = max(float(t.double().abs().max()) if t.numel() else 0.0 for t in (c["q"], c["k"]))
    return 2.0 ** -20 * 2 * X * abs(amplitude)


def check(c, **kw):
    ref_q, ref_k, ref_v = oracle(c, **kw)
    k0, v0 = to_np(c["k_pages"]), to_np(c["v_pages"])
    out = call(c, **kw)
    torch.cuda.synchronize()
    s = slack(c, kw.get("amplitude", 1.0))
    assert_rounded(out, ref_q, s, "q_out")
    assert_rounded(c["k_pages"], ref_k, s, "k_pages")
    assert_rounded(c["v_pages"], ref_v, 0.0, "v_pages")
    # what is not written keeps its bits
    same_k, same_v = ref_k == k0, ref_v == v0
    assert np.array_equal(to_np(c["v_pages"])[same_v], v0[same_v])
    untouched = same_k.all(axis=(2, 3))
    assert np.array_equal(to_np(c["k_pages"])[untouched], k0[untouched])
    return out


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rot", [(64, 64), (128, 128), (128, 32), (256, 64), (128, 0), (72, 24), (12, 8), (512, 512)])
@pytest.mark.parametrize("dtype,pdtype", [(BF16, BF16), (BF16, FP32), (FP32, BF16), (FP32, FP32)])
def test_layouts_and_types(interleaved, D, rot, dtype, pdtype):
    check(make([1, 5, 16, 17, 300], D=D, rot=rot, dtype=dtype, pdtype=pdtype), interleaved=interleaved)


@pytest.mark.parametrize("new", [[1], [3, 0, 5], [0, 0, 2], [40, 1, 0, 17, 0], [1] * 70, [0, 7] * 40])
def test_ragged_rows_with_empty_sequences_and_padding(new):
    lens = [t + 3 * i for i, t in enumerate(new)]
    c = make(lens, new=new, pad=3)
    out = check(c)
    assert torch.count_nonzero(out[sum(new):]) == 0


@pytest.mark.parametrize("page", [1, 7, 16, 64])
def test_page_sizes_and_null_pages(page):
    c = make([50, 33, 64, 20], new=[20, 33, 1, 2], page=page)
    c["table"][1, 0] = 0
    c["table"][2, (64 - 1) // page] = -1
    c["table"][3, (20 - 1) // page] = 10 ** 6
    check(c)


def test_negative_positions_and_lengths_past_the_table():
    # lengths 0 and below the new rows: null rows; a length past the table: rotated, not written
    c = make([0, 2, 500], new=[2, 4, 3], width=4)
    out = check(c)
    assert torch.count_nonzero(out[:4]) == 0 and torch.count_nonzero(out[6:]) > 0


@pytest.mark.parametrize("lens", [[1 << 20, (1 << 20) + 1, 999983], [2147483647, 2000000000, 5]])
@pytest.mark.parametrize("interleaved", [False, True])
def test_far_positions(lens, interleaved):
    # the table does not reach these positions: they rotate and are not written
    check(make(lens, width=3, dtype=FP32, pdtype=FP32), interleaved=interleaved)


@pytest.mark.parametrize("scaling,amplitude", [
    (dict(factor=8.0, original_len=8192, low=1.0, high=4.0), 1.0),
    (dict(factor=32.0, original_len=4096), 0.1 * np.log(32.0) + 1.0),
    (dict(factor=4.0, base=500000.0), 1.0),
])
def test_long_context_scalings(scaling, amplitude):
    check(make([70000, 4096, 1, 131072], width=9000, D=128, dtype=FP32, pdtype=FP32), amplitude=amplitude, scaling=scaling)


@pytest.mark.parametrize("kw", [dict(packed=False), dict(head_major=True), dict(interleaved_kv=True)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_layouts_of_inputs_and_pages(kw, interleaved):
    check(make([19, 40, 7], new=[19, 3, 7], **kw), interleaved=interleaved)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("packed", [False, True])
def test_in_place(packed, interleaved):
    c = make([9, 30, 0, 4], D=128, rot=64, packed=packed)
    ref_q, ref_k, _ = oracle(c, interleaved=interleaved)
    s = slack(c, 1.0)
    out = call(c, interleaved=interleaved, q_out=c["q"])
    torch.cuda.synchronize()
    assert out.data_ptr() == c["q"].data_ptr()
    assert_rounded(c["q"], ref_q, s, "q")
    assert_rounded(c["k_pages"], ref_k, s, "k_pages")


def test_rows_of_four_element_alignment():
    # bf16 rows that start on 8-byte but not on 16-byte boundaries
    c = make([9, 30, 2], D=64, packed=False)
    wide = torch.randn(3, 4 * 64 + 4, device="cuda").to(BF16)
    c["q"] = wide[:, 4:].view(3, 4, 64)
    check(c)


def test_nan_and_infinity_stay_in_their_rows():
    c = make([5, 6, 7], D=64)
    c["q"][1, 0, 3], c["k"][1, 1, 0] = float("nan"), float("inf")
    ref_q, ref_k, _ = oracle(c)
    out = call(c)
    torch.cuda.synchronize()
    assert np.array_equal(np.isfinite(to_np(out)), np.isfinite(ref_q))
    assert np.array_equal(np.isfinite(to_np(c["k_pages"])), np.isfinite(ref_k))


def test_empty_call_and_other_stream_and_graph():
    c = make([3], packed=False)
    e = {**c, "q": c["q"][:0], "k": c["k"][:0], "v": c["v"][:0], "lens": c["lens"][:0], "table": c["table"][:0]}
    assert call(e).shape[0] == 0
    c = make([33, 2, 80, 16])
    ref = oracle(c)
    steps = binding.kda_rope_phase_steps(c["rot"])
    run = lambda o: binding.kda_rope_append(c["q"], c["k"], c["v"], steps, c["lens"], c["table"], c["k_pages"],  # noqa: E731
                                            c["v_pages"], q_out=o)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out = run(None)
    side.synchronize()
    assert_rounded(out, ref[0], slack(c, 1.0), "q_out on a side stream")
    out = torch.empty_like(out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(out)
    c["lens"].sub_(1)  # replays read the lengths anew
    ref = oracle(c)
    graph.replay()
    torch.cuda.synchronize()
    assert_rounded(out, ref[0], slack(c, 1.0), "q_out of a replay")


def test_pages_past_4_gib():
    pages, page = 20000, 64
    pool = torch.zeros(pages, 2, page, 8, 128, dtype=BF16, device="cuda")  # 5 GB
    g = torch.Generator(device="cuda").manual_seed(0)
    x = torch.randn(3, 24, 128, device="cuda", generator=g).to(BF16)
    q, k, v = x[:, :8], x[:, 8:16], x[:, 16:]
    steps = binding.kda_rope_phase_steps(128)
    lens = torch.tensor([1, 70, 130], dtype=torch.int32, device="cuda")
    table = torch.tensor([[pages - 1, 0, 0], [0, pages - 2, 0], [0, 0, pages - 9]], dtype=torch.int32, device="cuda")
    small = torch.zeros(4, 2, page, 8, 128, dtype=BF16, device="cuda")
    near = torch.tensor([[1, 0, 0], [0, 2, 0], [0, 0, 3]], dtype=torch.int32, device="cuda")
    a = binding.kda_rope_append(q, k, v, steps, lens, table, pool[:, 0], pool[:, 1])
    b = binding.kda_rope_append(q, k, v, steps, lens, near, small[:, 0], small[:, 1])
    torch.cuda.synchronize()
    assert torch.equal(a, b)
    for n, p in enumerate((pages - 1, pages - 2, pages - 9)):
        assert torch.equal(pool[p], small[n + 1]) and torch.count_nonzero(pool[p]) > 0
    assert torch.count_nonzero(pool[:pages - 9]) == 0


def test_host_tensors_are_refused():
    c = make([3, 4])
    with pytest.raises(ValueError, match="host"):
        binding.kda_rope_append(c["q"], c["k"], c["v"], binding.kda_rope_phase_steps(64, device="cpu"), c["lens"],
                                c["table"], c["k_pages"], c["v_pages"])


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype,pdtype", [(BF16, BF16), (FP32, FP32), (BF16, FP32)])
@pytest.mark.parametrize("D,rot", [(128, 128), (72, 24), (256, 64)])
def test_many_rows(interleaved, dtype, pdtype, D, rot):
    # several rows a block: counts that do not divide, null rows and padding among them
    rng = np.random.default_rng(D)
    lens = [int(x) for x in rng.integers(0, 40, 331)]
    check(make(lens, D=D, rot=rot, dtype=dtype, pdtype=pdtype, page=7), interleaved=interleaved)
    new = [int(x) for x in rng.integers(0, 30, 80)]
    lens = [t + int(x) for t, x in zip(new, rng.integers(0, 9, 80))]
    lens[3], lens[50] = 0, max(0, new[50] - 2)
    out = check(make(lens, new=new, pad=5, D=D, rot=rot, dtype=dtype, pdtype=pdtype, page=16), interleaved=interleaved)
    assert out.shape[0] >= 320 and torch.count_nonzero(out[sum(new):]) == 0
