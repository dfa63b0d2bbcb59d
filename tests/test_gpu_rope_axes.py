"""GPU parity of kda_rope_axes_append against the float64 oracle: axes and their layouts over the pairs, types, far and
negative positions, null slots, strided positions and pages, in place, graphs, and agreement with kda_rope_append."""

import numpy as np
import pytest
import torch

from linear_attention_decode_02_gb300 import binding, build
from oracle import cache_oracle as co
from tests.rounding import assert_rounded, to_np
from tests.test_gpu_rope_append import slack

pytestmark = pytest.mark.gpu
BF16, FP32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return binding.library()


def make(rows, axes=3, Hq=4, Hkv=2, D=64, rot=None, page=16, dtype=BF16, pdtype=BF16, seed=0, far=5000, sections=None,
         cyclic=False, layout="token", transposed=False):
    g = torch.Generator().manual_seed(seed)
    rot = D if rot is None else rot

    def normal(*shape, dtype=dtype):
        return torch.randn(*shape, generator=g).to(dtype)

    x = normal(rows, (Hq + 2 * Hkv) * D).cuda()
    c = dict(q=x[:, :Hq * D].view(rows, Hq, D), k=x[:, Hq * D:(Hq + Hkv) * D].view(rows, Hkv, D),
             v=x[:, (Hq + Hkv) * D:].view(rows, Hkv, D), rot=rot)
    pages = -(-rows // page) + 3
    k, v = normal(pages, page, Hkv, D, dtype=pdtype).cuda(), normal(pages, page, Hkv, D, dtype=pdtype).cuda()
    if layout == "head":
        k, v = (t.transpose(1, 2).contiguous().transpose(1, 2) for t in (k, v))
    elif layout == "pair":
        kv = torch.stack([k, v], dim=1)
        k, v = kv[:, 0], kv[:, 1]
    c["k_pages"], c["v_pages"] = k, v
    c["slots"] = (torch.randperm((pages - 1) * page, generator=g)[:rows] + page).to(torch.int32).cuda()
    pos = torch.randint(-far, far, (rows, axes), generator=g).to(torch.int32).cuda()
    c["positions"] = pos.t().contiguous().t() if transposed else pos
    if sections is None:
        sections = [rot // 2 // axes] * (axes - 1)
        sections.append(rot // 2 - sum(sections))
    c["axes"] = binding.kda_rope_pair_axes(sections, cyclic)
    c["steps"] = binding.kda_rope_phase_steps(rot)
    return c


def call(c, interleaved=False, amplitude=1.0, q_out=None):
    return binding.kda_rope_axes_append(c["q"], c["k"], c["v"], c["steps"], c["axes"], c["positions"], c["slots"],
                                        c["k_pages"], c["v_pages"], interleaved=interleaved, amplitude=amplitude,
                                        q_out=q_out)


def check(c, **kw):
    kw.pop("q_out", None)
    ref = co.rope_axes_append(to_np(c["q"]), to_np(c["k"]), to_np(c["v"]), co.rope_frequencies(c["rot"]),
                              c["axes"].tolist(), c["positions"].cpu().numpy(), c["slots"].tolist(), to_np(c["k_pages"]),
                              to_np(c["v_pages"]), **kw)
    before = to_np(c["k_pages"])
    out = call(c, **kw)
    torch.cuda.synchronize()
    s = slack(c, kw.get("amplitude", 1.0))
    assert_rounded(out, ref[0], s, "q_out")
    assert_rounded(c["k_pages"], ref[1], s, "k_pages")
    assert np.array_equal(to_np(c["v_pages"]), np.asarray(torch.from_numpy(ref[2]).to(c["v_pages"].dtype).double()))
    untouched = (ref[1] == before).all(axis=(2, 3))
    assert np.array_equal(to_np(c["k_pages"])[untouched], before[untouched])
    return out


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rot", [(64, 64), (128, 128), (128, 32), (256, 64), (128, 0), (72, 24), (12, 8), (512, 512)])
@pytest.mark.parametrize("dtype,pdtype", [(BF16, BF16), (BF16, FP32), (FP32, BF16), (FP32, FP32)])
def test_layouts_and_types(interleaved, D, rot, dtype, pdtype):
    check(make(9, D=D, rot=rot, dtype=dtype, pdtype=pdtype), interleaved=interleaved, amplitude=1.25)


@pytest.mark.parametrize("axes", [1, 2, 3, 4])
@pytest.mark.parametrize("cyclic", [False, True])
@pytest.mark.parametrize("rows", [1, 3, 319, 320, 1001])
def test_axes_and_rows(axes, cyclic, rows):
    check(make(rows, axes=axes, cyclic=cyclic, page=7))


@pytest.mark.parametrize("sections", [[32, 0, 0], [0, 0, 32], [8, 12, 12], [1, 30, 1]])
@pytest.mark.parametrize("cyclic", [False, True])
def test_sections(sections, cyclic):
    check(make(40, sections=sections, cyclic=cyclic, dtype=FP32, pdtype=FP32))


def test_pairs_without_an_axis_are_not_turned():
    c = make(10, dtype=FP32, pdtype=FP32)
    c["axes"][3], c["axes"][7], c["axes"][20] = -1, 3, 2 ** 31 - 1
    check(c, amplitude=2.0)


@pytest.mark.parametrize("far", [1 << 20, 2 ** 31 - 1])
@pytest.mark.parametrize("interleaved", [False, True])
def test_far_and_negative_positions(far, interleaved):
    c = make(50, far=far, dtype=FP32, pdtype=FP32)
    c["positions"][0] = torch.tensor([-2 ** 31, 2 ** 31 - 1, -1], dtype=torch.int32)
    check(c, interleaved=interleaved)


@pytest.mark.parametrize("rows", [6, 330])
def test_null_slots(rows):
    c = make(rows, page=16)
    pages = c["k_pages"].shape[0]
    c["slots"][:6] = torch.tensor([-1, 0, 15, pages * 16, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32)
    out = check(c)
    assert torch.count_nonzero(out[:6]) == 0
    c["slots"][:] = -1
    assert torch.count_nonzero(check(c)) == 0


@pytest.mark.parametrize("layout", ["token", "head", "pair"])
@pytest.mark.parametrize("transposed", [False, True])
def test_strides(layout, transposed):
    check(make(37, layout=layout, transposed=transposed, D=128))


def test_four_element_alignment():
    c = make(37, D=64)
    for name in ("q", "k", "v", "k_pages", "v_pages"):
        t = c[name]
        wide = torch.zeros(*t.shape[:-1], t.shape[-1] + 4, dtype=t.dtype, device="cuda")
        wide[..., 4:] = t
        c[name] = wide[..., 4:]
    check(c)


def test_no_rows():
    c = make(0)
    assert call(c).shape == (0, 4, 64)


def test_in_place_streams_and_graphs():
    c = make(500, D=128)
    q = c["q"].clone()
    out = check(c)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        other = call(c)
    torch.cuda.synchronize()
    assert torch.equal(other, out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        again = call(c)
    c["positions"].neg_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(again, check(c))
    assert call(c, q_out=c["q"]) is c["q"]
    torch.cuda.synchronize()
    assert torch.equal(c["q"], again) and not torch.equal(c["q"], q)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_equal_axes_are_one_axis(interleaved, dtype):
    """Text, whose positions are the same on all axes, gives the bits of kda_rope_append."""
    page, lens, new = 8, [40, 7, 90], [12, 7, 1]
    rows = sum(new)
    c = make(rows, page=page, dtype=dtype, pdtype=dtype)
    pos = np.concatenate([np.arange(a - b, a) for a, b in zip(lens, new)])
    c["positions"] = torch.tensor(np.stack([pos] * 3, 1), dtype=torch.int32).cuda()
    table = torch.arange(1, 37, dtype=torch.int32).view(3, 12).cuda()
    seq = np.repeat(np.arange(3), new)
    c["k_pages"], c["v_pages"] = (torch.zeros(40, page, 2, 64, dtype=dtype, device="cuda") for _ in range(2))
    c["slots"] = (table[seq, pos // page] * page + torch.tensor(pos % page).cuda()).to(torch.int32)
    out = call(c, interleaved=interleaved)
    k2, v2 = torch.zeros_like(c["k_pages"]), torch.zeros_like(c["v_pages"])
    ref = binding.kda_rope_append(c["q"], c["k"], c["v"], binding.kda_rope_phase_steps(64),
                                  torch.tensor(lens, dtype=torch.int32, device="cuda"), table, k2, v2,
                                  cu_seqlens=torch.tensor([0, 12, 19, 20], dtype=torch.int32, device="cuda"),
                                  interleaved=interleaved)
    torch.cuda.synchronize()
    assert torch.equal(out, ref) and torch.equal(c["k_pages"], k2) and torch.equal(c["v_pages"], v2)
