"""Contract checks of page assignment, rotary positions with several axes and attention under shared prefixes (CPU only:
descriptors of host memory, and only calls that are refused before any launch)."""

import ctypes

import pytest
import torch

from linear_attention_decode_02_gb300 import binding
from linear_attention_decode_02_gb300.binding import desc
from tests import test_cache_abi as cache
from tests.test_cache_abi import ALIAS, BF16, CUDA, INVALID, NO_GPU, UNSUPPORTED, _i32, _msg, lib  # noqa: F401


def _ptr(t):
    return None if t is None else ctypes.byref(desc(t))


# ---- kda_page_assign ------------------------------------------------------------------


def _pages(N=3, P=5, C=20, R=7):
    return dict(old=_i32(N), new=_i32(N), shared=_i32(N), table=_i32(N, P), free=_i32(C), state=_i32(2), lens=_i32(N),
                after=_i32(2), cu=_i32(N + 1), slots=_i32(R))


def _call_pages(lib, t, page=8):  # noqa: F811
    p = {n: _ptr(x) for n, x in t.items()}
    return lib.kda_page_assign(p["old"], p["new"], p["shared"], p["table"], p["free"], p["state"], page, p["lens"],
                               p["after"], p["cu"], p["slots"], None)


@pytest.mark.skipif(not NO_GPU, reason="a valid call would launch on host memory")
def test_page_valid_calls_reach_the_device_query(lib):  # noqa: F811
    assert _call_pages(lib, _pages()) in (UNSUPPORTED, CUDA), _msg(lib)
    t = _pages()
    t.update(lens=t["old"], after=t["state"], shared=None)  # in place
    assert _call_pages(lib, t) in (UNSUPPORTED, CUDA), _msg(lib)
    t = _pages()
    t["lens"] = t["new"]
    assert _call_pages(lib, t) in (UNSUPPORTED, CUDA), _msg(lib)
    assert _call_pages(lib, _pages(N=0, R=0)) in (UNSUPPORTED, CUDA), _msg(lib)
    assert _call_pages(lib, {**_pages(), "table": _i32(3, 9)[:, 2:7]}) in (UNSUPPORTED, CUDA), _msg(lib)


@pytest.mark.parametrize("change,status,text", [
    (lambda t: t.update(new=_i32(4)), INVALID, "new_lens: axis 0"),
    (lambda t: t.update(old=torch.zeros(3)), INVALID, "seq_lens: dtype"),
    (lambda t: t.update(old=_i32(3, 1)), INVALID, "seq_lens: expected rank 1"),
    (lambda t: t.update(shared=_i32(2)), INVALID, "shared_lens: axis 0"),
    (lambda t: t.update(table=_i32(2, 5)), INVALID, "page_table: axis 0"),
    (lambda t: t.update(table=_i32(5, 3).t()), INVALID, "column stride"),
    (lambda t: t.update(table=torch.as_strided(_i32(20), (3, 5), (3, 1))), INVALID, "elements overlap"),
    (lambda t: t.update(free=_i32(0)), INVALID, "no place for a page"),
    (lambda t: t.update(free=_i32(40)[::2]), INVALID, "free_pages: must be contiguous"),
    (lambda t: t.update(state=_i32(3)), INVALID, "free_state: axis 0"),
    (lambda t: t.update(lens=_i32(2)), INVALID, "lens_out: axis 0"),
    (lambda t: t.update(after=_i32(1)), INVALID, "state_out: axis 0"),
    (lambda t: t.update(cu=_i32(3)), INVALID, "cu_seqlens: axis 0"),
    (lambda t: t.update(slots=_i32(7, 1)), INVALID, "slots: expected rank 1"),
    (lambda t: t.update(slots=torch.zeros(7)), INVALID, "slots: dtype"),
    (lambda t: t.update(slots=t["free"][:7]), ALIAS, "free_pages overlaps slots"),
    (lambda t: t.update(free=t["table"].flatten()), ALIAS, "page_table overlaps free_pages"),
    (lambda t: t.update(cu=t["slots"][:4]), ALIAS, "cu_seqlens overlaps slots"),
    (lambda t: t.update(lens=t["shared"]), ALIAS, "lens_out overlaps shared_lens"),
    (lambda t: t.update(after=t["old"][:2]), ALIAS, "state_out overlaps seq_lens"),
    (lambda t: t.update(table=None), INVALID, "page_table: null"),
    (lambda t: t.update(old=None), INVALID, "seq_lens: null"),
    (lambda t: t.update(**{n: _i32(8193) for n in ("old", "new", "shared", "lens")}), UNSUPPORTED, "at most 8192"),
])
def test_page_refusals(lib, change, status, text):  # noqa: F811
    t = _pages()
    change(t)
    assert _call_pages(lib, t) == status, _msg(lib)
    assert text in _msg(lib)


def test_page_refuses_shifted_in_place_and_bad_sizes(lib):  # noqa: F811
    x = _i32(10)
    assert _call_pages(lib, {**_pages(), "old": x[:3], "lens": x[1:4]}) == ALIAS
    assert _call_pages(lib, {**_pages(), "state": x[:2], "after": x[1:3]}) == ALIAS
    assert _call_pages(lib, _pages(), page=0) == INVALID
    assert _call_pages(lib, _pages(), page=-4) == INVALID
    assert _call_pages(lib, _pages(), page=(2 ** 31 - 1) // 21 + 1) == UNSUPPORTED  # 21 pages' slots pass 2^31
    assert "2^31" in _msg(lib)


# ---- kda_rope_axes_append -----------------------------------------------------------------


def _rope(R=3, Hq=4, Hkv=2, D=64, A=3, page=8):
    t = cache._rope(R=R, Hq=Hq, Hkv=Hkv, D=D, page=page)
    for n in ("cu", "lens", "table"):
        del t[n]
    return {**t, "axes": _i32(D // 2), "positions": _i32(R, A), "slots": _i32(R)}


def _call_rope(lib, t, interleaved=0, amplitude=1.0):  # noqa: F811
    return lib.kda_rope_axes_append(*[_ptr(t[n]) for n in ("q", "k", "v", "steps", "axes", "positions", "slots", "k_pages",
                                                           "v_pages", "q_out")], interleaved, amplitude, None)


@pytest.mark.skipif(not NO_GPU, reason="a valid call would launch on host memory")
def test_rope_axes_valid_calls_reach_the_device_query(lib):  # noqa: F811
    t = _rope()
    assert _call_rope(lib, t) in (UNSUPPORTED, CUDA), _msg(lib)
    t["q_out"] = t["q"]  # in place
    assert _call_rope(lib, t) in (UNSUPPORTED, CUDA), _msg(lib)
    t = _rope(A=1)
    t["positions"] = _i32(4, 3).t()[:, :4]
    assert _call_rope(lib, t) in (UNSUPPORTED, CUDA), _msg(lib)
    t.update(steps=_i32(0, 2), axes=_i32(0))
    assert _call_rope(lib, t) in (UNSUPPORTED, CUDA), _msg(lib)
    assert _call_rope(lib, _rope(R=0)) == 0


@pytest.mark.parametrize("change,status,text", [
    (lambda t: t.update(k=torch.zeros(3, 2, 64)), INVALID, "k: dtype must match q"),
    (lambda t: t.update(axes=_i32(31)), INVALID, "pair_axes: axis 0"),
    (lambda t: t.update(axes=torch.zeros(32)), INVALID, "pair_axes: dtype"),
    (lambda t: t.update(axes=_i32(64)[::2]), INVALID, "pair_axes: must be contiguous"),
    (lambda t: t.update(positions=_i32(2, 3)), INVALID, "positions: axis 0"),
    (lambda t: t.update(positions=torch.zeros(3, 3)), INVALID, "positions: dtype"),
    (lambda t: t.update(positions=_i32(3)), INVALID, "positions: expected rank 2"),
    (lambda t: t.update(positions=_i32(3, 5)), UNSUPPORTED, "1 to 4"),
    (lambda t: t.update(positions=_i32(3, 0)), UNSUPPORTED, "0 axes"),
    (lambda t: t.update(positions=_i32(3, 1).expand(3, 3)), INVALID, "must be positive"),
    (lambda t: t.update(slots=_i32(4)), INVALID, "slots: axis 0"),
    (lambda t: t.update(slots=_i32(6)[::2]), INVALID, "slots: must be contiguous"),
    (lambda t: t.update(v_pages=t["k_pages"]), ALIAS, "k_pages overlaps v_pages"),
    (lambda t: t.update(steps=_i32(36, 2), axes=_i32(36)), INVALID, "phase_steps: 36 pairs"),
    (lambda t: t.update(q_out=torch.zeros(3, 4, 64)), INVALID, "q_out: dtype must match the pages"),
    (lambda t: t.update(positions=None), INVALID, "positions: null"),
])
def test_rope_axes_refusals(lib, change, status, text):  # noqa: F811
    t = _rope()
    change(t)
    assert _call_rope(lib, t) == status, _msg(lib)
    assert text in _msg(lib)


def test_rope_axes_refuses_bad_scalars(lib):  # noqa: F811
    assert _call_rope(lib, _rope(), interleaved=2) == INVALID
    assert _call_rope(lib, _rope(), amplitude=float("inf")) == INVALID


@pytest.mark.parametrize("sections,cyclic,want", [
    ([2, 3, 1], False, [0, 0, 1, 1, 1, 2]), ([2, 3, 1], True, [0, 1, 2, 0, 1, 1]), ([0, 2], True, [1, 1]), ([5], False, [0] * 5),
    ([0, 0, 0, 0], False, []), ([1, 0, 0, 3], True, [0, 3, 3, 3]),
])
def test_pair_axes(lib, sections, cyclic, want):  # noqa: F811
    got = binding.kda_rope_pair_axes(sections, cyclic, device="cpu")
    assert got.tolist() == want and got.dtype == torch.int32


@pytest.mark.parametrize("sections,text", [([], "0 axes"), ([1] * 5, "5 axes"), ([3, -1], "section 1 is negative"),
                                           ([200, 57], "at most 256"), ([2 ** 40, 1], "at most 256"), ([-2 ** 40], "negative")])
def test_pair_axes_refusals(lib, sections, text):  # noqa: F811
    with pytest.raises(binding.KdaError, match=text):
        binding.kda_rope_pair_axes(sections, device="cpu")


# ---- kda_prefix_attention_decode -----------------------------------------------------------


def _prefix(N=3, G=2, dtype=BF16, **kw):
    t = cache._attend(N=N, dtype=dtype, **kw)
    shape = (t["q"].shape[1], t["k_pages"].shape[2], t["q"].shape[2])
    t["work"] = torch.zeros(binding.kda_prefix_attention_workspace(N, *shape, dtype, 152))
    return {**t, "starts": _i32(G + 1), "prefix": _i32(G)}


def _call_prefix(lib, t, window=0, scale=0.125):  # noqa: F811
    d = {n: _ptr(x) for n, x in t.items()}
    return lib.kda_prefix_attention_decode(d["q"], d["k_pages"], d["v_pages"], d["table"], d["lens"], d["starts"],
                                           d["prefix"], d["work"], window, scale, d["out"], d["lse"], None)


@pytest.mark.skipif(not NO_GPU, reason="a valid call would launch on host memory")
def test_prefix_valid_calls_reach_the_device_query(lib):  # noqa: F811
    assert _call_prefix(lib, _prefix()) in (UNSUPPORTED, CUDA), _msg(lib)
    assert _call_prefix(lib, {**_prefix(G=0), "lse": None}, window=7) in (UNSUPPORTED, CUDA), _msg(lib)
    assert _call_prefix(lib, _prefix(dtype=torch.float32)) in (UNSUPPORTED, CUDA), _msg(lib)
    assert _call_prefix(lib, _prefix(N=0)) == 0


@pytest.mark.parametrize("change,status,text", [
    (lambda t: t.update(starts=_i32(2)), INVALID, "group_starts: axis 0"),
    (lambda t: t.update(starts=torch.zeros(3)), INVALID, "group_starts: dtype"),
    (lambda t: t.update(starts=None), INVALID, "group_starts: null"),
    (lambda t: t.update(prefix=None), INVALID, "prefix_lens: null"),
    (lambda t: t.update(prefix=_i32(2, 1)), INVALID, "prefix_lens: expected rank 1"),
    (lambda t: t.update(prefix=_i32(4)[::2]), INVALID, "prefix_lens: must be contiguous"),
    (lambda t: t.update(q=torch.zeros(3, 3, 64, dtype=BF16)), INVALID, "evenly"),
    (lambda t: t.update(table=_i32(2, 5)), INVALID, "page_table: axis 0"),
    (lambda t: t.update(out=t["q"]), ALIAS, "out overlaps q"),
    (lambda t: t.update(starts=t["work"][:3].view(torch.int32)), ALIAS, "workspace overlaps group_starts"),
    (lambda t: t.update(lse=torch.zeros(3, 5)), INVALID, "lse: axis 1"),
])
def test_prefix_refusals(lib, change, status, text):  # noqa: F811
    t = _prefix()
    change(t)
    assert _call_prefix(lib, t) == status, _msg(lib)
    assert text in _msg(lib)


def test_prefix_refuses_bad_scalars(lib):  # noqa: F811
    assert _call_prefix(lib, _prefix(), window=-1) == INVALID
    for scale in (0.0, -1.0, float("inf"), float("nan"), 3e38):
        assert _call_prefix(lib, _prefix(), scale=scale) == INVALID


def test_prefix_workspace_query(lib):  # noqa: F811
    few = binding.kda_prefix_attention_workspace(1, 32, 8, 128, BF16, 152)
    assert binding.kda_paged_attention_workspace(32, 8, 128, BF16, 152) <= few
    assert few < binding.kda_prefix_attention_workspace(4096, 32, 8, 128, BF16, 152)
    assert binding.kda_paged_attention_workspace(32, 8, 128, torch.float32, 152) < \
        binding.kda_prefix_attention_workspace(4096, 32, 8, 128, torch.float32, 152)
    for args in ((-1, 8, 8, 64, BF16, 152), (1 << 24, 8, 8, 64, BF16, 152), (1, 8, 3, 64, BF16, 152), (1, 8, 8, 80, BF16, 152),
                 (1, 8, 8, 64, torch.int32, 152), (1, 8, 8, 64, BF16, 0)):
        with pytest.raises(binding.KdaError):
            binding.kda_prefix_attention_workspace(*args)


# ---- tensors off their elements' boundaries --------------------------------------------------

NAMES = {"pages": ("old", "new", "shared", "table", "free", "state", "lens", "after", "cu", "slots"),
         "rope axes": ("q", "k", "v", "steps", "axes", "positions", "slots", "k_pages", "v_pages", "q_out"),
         "prefix": ("q", "k_pages", "v_pages", "table", "lens", "starts", "prefix", "work", "out", "lse")}
CALLS = {"pages": (_pages, _call_pages), "rope axes": (_rope, _call_rope), "prefix": (_prefix, _call_prefix)}


@pytest.mark.parametrize("op,name", [(op, name) for op in CALLS for name in NAMES[op]])
def test_tensors_off_their_elements_boundaries_are_refused(lib, monkeypatch, op, name):  # noqa: F811
    make, call = CALLS[op]
    t = make()
    for by in range(1, t[name].element_size()):
        def moved(x):
            d = binding.desc(x)
            if x is t[name]:
                d.data += by
            return d
        monkeypatch.setitem(globals(), "desc", moved)
        assert call(lib, t) == INVALID, (by, _msg(lib))
        assert "aligned" in _msg(lib)
        monkeypatch.undo()
