"""Contract checks of the cache and beam entry points (CPU only: descriptors of
host memory, and only calls that are refused before any launch)."""

import ctypes

import numpy as np
import pytest
import torch

from linear_attention_decode_02_gb300 import binding, build
from linear_attention_decode_02_gb300.binding import desc
from oracle import cache_oracle as co

INVALID, UNSUPPORTED, ALIAS, CUDA = 1, 2, 3, 4
NO_GPU = not torch.cuda.is_available()
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.library()


def _ptr(t):
    return None if t is None else ctypes.byref(desc(t))


def _msg(lib):
    return lib.kda_last_error_message().decode()


# ---- kda_rope_append ------------------------------------------------------------------


def _rope(R=3, Hq=4, Hkv=2, D=64, N=3, P=5, page=8):
    return dict(q=torch.zeros(R, Hq, D, dtype=BF16), k=torch.zeros(R, Hkv, D, dtype=BF16),
                v=torch.zeros(R, Hkv, D, dtype=BF16), steps=torch.zeros(D // 2, 2, dtype=torch.int32), cu=None,
                lens=torch.ones(N, dtype=torch.int32), table=torch.zeros(N, P, dtype=torch.int32),
                k_pages=torch.zeros(4, page, Hkv, D, dtype=BF16), v_pages=torch.zeros(4, page, Hkv, D, dtype=BF16),
                q_out=torch.zeros(R, Hq, D, dtype=BF16))


def _call_rope(lib, t, interleaved=0, amplitude=1.0):
    return lib.kda_rope_append(*[_ptr(t[n]) for n in ("q", "k", "v", "steps", "cu", "lens", "table", "k_pages",
                                                      "v_pages", "q_out")], interleaved, amplitude, None)


@pytest.mark.skipif(not NO_GPU, reason="a valid call would launch on host memory")
def test_rope_valid_calls_reach_the_device_query(lib):
    t = _rope()
    assert _call_rope(lib, t) in (UNSUPPORTED, CUDA), _msg(lib)
    t["q_out"] = t["q"]  # in place
    assert _call_rope(lib, t) in (UNSUPPORTED, CUDA), _msg(lib)
    t = _rope()
    x = torch.zeros(3, 8 * 64, dtype=BF16)  # in place inside a packed row
    t.update(q=x[:, :256].view(3, 4, 64), k=x[:, 256:384].view(3, 2, 64), v=x[:, 384:].view(3, 2, 64))
    t["q_out"] = t["q"]
    assert _call_rope(lib, t) in (UNSUPPORTED, CUDA), _msg(lib)
    for axis in (0, 1, 2, 3):  # keys and values interleaved along any axis of one allocation
        shape = [4, 8, 2, 64]
        shape.insert(axis, 2)
        kv = torch.zeros(*shape, dtype=BF16)
        t.update(k_pages=kv.select(axis, 0), v_pages=kv.select(axis, 1))
        assert _call_rope(lib, t) in (UNSUPPORTED, CUDA), (axis, _msg(lib))
    t = _rope()
    t.update(cu=torch.zeros(4, dtype=torch.int32), steps=torch.zeros(0, 2, dtype=torch.int32))
    assert _call_rope(lib, t) in (UNSUPPORTED, CUDA), _msg(lib)
    assert _call_rope(lib, {**_rope(R=0, N=0)}) == 0


@pytest.mark.parametrize("change,status,text", [
    (lambda t: t.update(k=torch.zeros(3, 2, 64)), INVALID, "k: dtype must match q"),
    (lambda t: t.update(v=torch.zeros(3, 1, 64, dtype=BF16)), INVALID, "v: axis 1"),
    (lambda t: t.update(steps=torch.zeros(36, 2, dtype=torch.int32)), INVALID, "phase_steps: 36 pairs"),
    (lambda t: t.update(steps=torch.zeros(6, 2, dtype=torch.int32)), INVALID, "multiple of 8"),
    (lambda t: t.update(steps=torch.zeros(32, 3, dtype=torch.int32)), INVALID, "phase_steps: axis 1"),
    (lambda t: t.update(lens=torch.ones(2, dtype=torch.int32)), INVALID, "without cu_seqlens"),
    (lambda t: t.update(cu=torch.zeros(3, dtype=torch.int32)), INVALID, "cu_seqlens: axis 0"),
    (lambda t: t.update(lens=torch.ones(3)), INVALID, "seq_lens: dtype"),
    (lambda t: t.update(table=torch.zeros(2, 5, dtype=torch.int32)), INVALID, "page_table: axis 0"),
    (lambda t: t.update(table=torch.zeros(5, 3, dtype=torch.int32).t()), INVALID, "column stride"),
    (lambda t: t.update(v_pages=torch.zeros(4, 8, 2, 64)), INVALID, "v_pages: dtype must match"),
    (lambda t: t.update(v_pages=torch.zeros(5, 8, 2, 64, dtype=BF16)), INVALID, "v_pages: axis 0"),
    (lambda t: t.update(k_pages=torch.zeros(4, 8, 3, 64, dtype=BF16)), INVALID, "k_pages: axis 2"),
    (lambda t: t.update(k_pages=torch.zeros(4, 8, 2, 66, dtype=BF16)[..., 2:]), INVALID, "multiple of 4"),
    (lambda t: t.update(q_out=torch.zeros(3, 4, 64)), INVALID, "q_out: dtype must match the pages"),
    (lambda t: t.update(q=torch.zeros(3, 4, 62, dtype=BF16)), UNSUPPORTED, "head dimension"),
    (lambda t: t.update(q_out=t["k_pages"].view(-1)[:768].view(3, 4, 64)), ALIAS, "q_out overlaps"),
    (lambda t: t.update(v_pages=t["k_pages"]), ALIAS, "k_pages overlaps v_pages"),
    (lambda t: t.update(q_out=t["q"].transpose(0, 1)[:3].contiguous().transpose(0, 1)[:, :3]), INVALID, "q_out: axis 1"),
    (lambda t: t.update(k=None), INVALID, "k: null"),
])
def test_rope_refusals(lib, change, status, text):
    t = _rope()
    change(t)
    assert _call_rope(lib, t) == status, _msg(lib)
    assert text in _msg(lib)


def test_rope_refuses_shifted_in_place_and_bad_scalars(lib):
    t = _rope()
    x = torch.zeros(4 * 3 * 64 + 64, dtype=BF16)
    t.update(q=x[:768].view(3, 4, 64), q_out=x[64:832].view(3, 4, 64))
    assert _call_rope(lib, t) == ALIAS
    assert _call_rope(lib, _rope(), interleaved=2) == INVALID
    assert _call_rope(lib, _rope(), amplitude=float("nan")) == INVALID


@pytest.mark.parametrize("kw", [dict(), dict(factor=8.0, original_len=8192.0, low=1.0, high=4.0),
                                dict(factor=4.0), dict(base=500000.0, factor=32.0, original_len=4096.0)])
def test_phase_steps_are_the_frequencies_in_64_bit_turns(lib, kw):
    for rot in (0, 2, 64, 128, 512):
        steps = binding.kda_rope_phase_steps(rot, device="cpu", **kw)
        assert steps.shape == (rot // 2, 2) and steps.dtype == torch.int32
        got = steps.numpy().astype(np.int32).view(np.uint32).astype(np.uint64)
        turns = (got[:, 1] * np.uint64(2 ** 32) + got[:, 0]).astype(np.float64) / 2.0 ** 64
        ref = co.rope_frequencies(rot, **kw) / (2 * np.pi)
        # The steps are multiples of 2^-64: off by 2^-65 for that.  In float64 on both sides, the exponent's rounding
        # (2^-53) times ln(base) <= 13.2 and pow's own put f within 2^-49; keep moves by at most high / (high - low)
        # of that, and the sum it enters is at least 1 / factor >= 1/32 of the whole: below 2^-49 * 2 * 32 = 2^-43.
        assert np.all(np.abs(turns - ref) <= 2.0 ** -43 * ref + 2.0 ** -64)


@pytest.mark.parametrize("args,text", [
    (dict(rot_dim=7), "rot_dim"), (dict(rot_dim=-2), "rot_dim"), (dict(rot_dim=514), "rot_dim"),
    (dict(rot_dim=8, base=1.0), "base"), (dict(rot_dim=8, base=float("inf")), "base"),
    (dict(rot_dim=8, factor=0.5), "factor"), (dict(rot_dim=8, original_len=-1.0), "original_len"),
    (dict(rot_dim=8, original_len=4096.0, low=4.0, high=4.0), "low"),
])
def test_phase_step_refusals(lib, args, text):
    with pytest.raises(binding.KdaError, match=text):
        binding.kda_rope_phase_steps(device="cpu", **args)


# ---- kda_pool_move ----------------------------------------------------------------------


def _move(lib, pools, src, dst, parents=None, n=None):
    array = (ctypes.POINTER(binding.KdaTensor) * max(1, len(pools)))()
    keep = [desc(p) for p in pools]
    for i, d in enumerate(keep):
        array[i] = ctypes.pointer(d)
    return lib.kda_pool_move(array, len(pools) if n is None else n, _ptr(src), _ptr(dst), _ptr(parents), None)


def _i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


@pytest.mark.skipif(not NO_GPU, reason="a valid call would launch on host memory")
def test_move_valid_calls_reach_the_device_query(lib):
    kv = torch.zeros(5, 2, 8, 2, 64, dtype=BF16)
    conv = torch.zeros(5, 3, 24, dtype=BF16).permute(0, 2, 1)
    ok = [torch.zeros(5, 2, 128, 128), conv, kv[:, 0], kv[:, 1], torch.zeros(5, 2, 8, 64).transpose(1, 2), torch.zeros(5)]
    assert _move(lib, ok, _i32(3, 4), _i32(3, 4), _i32(3, 4)) in (UNSUPPORTED, CUDA), _msg(lib)
    assert _move(lib, [torch.zeros(5, 4)] , _i32(0, 4), _i32(0, 4)) == 0


@pytest.mark.parametrize("pools,src,dst,parents,status,text", [
    ([], _i32(1, 1), _i32(1, 1), None, INVALID, "at least one pool"),
    ([torch.zeros(5, 4), torch.zeros(6, 4)], _i32(1, 1), _i32(1, 1), None, INVALID, "pool 1: 6 slots"),
    ([torch.zeros(5, 8)[:, ::2]], _i32(1, 1), _i32(1, 1), None, INVALID, "must be dense"),
    ([torch.zeros(5, 4, 8)[:, :, :4]], _i32(1, 1), _i32(1, 1), None, INVALID, "must be dense"),
    ([torch.as_strided(torch.zeros(64), (5, 8), (4, 1))], _i32(1, 1), _i32(1, 1), None, INVALID, "overlaps slots"),
    ([torch.zeros(5, 4)], _i32(2, 3), _i32(2, 2), None, INVALID, "dst_slots: axis 1"),
    ([torch.zeros(5, 4)], _i32(2, 3), _i32(2, 3), _i32(3, 3), INVALID, "parents: axis 0"),
    ([torch.zeros(5, 4)], torch.zeros(2, 3), _i32(2, 3), None, INVALID, "src_slots: dtype"),
    ([torch.zeros(5, 4)], _i32(2, 33), _i32(2, 33), None, UNSUPPORTED, "at most 32"),
    ([torch.zeros(5, 4)], _i32(3, 2).t(), _i32(2, 3), None, INVALID, "column stride"),
])
def test_move_refusals(lib, pools, src, dst, parents, status, text):
    assert _move(lib, pools, src, dst, parents) == status, _msg(lib)
    assert text in _msg(lib)


def test_move_refuses_shared_memory_and_too_many_pools(lib):
    x = torch.zeros(5, 8)
    assert _move(lib, [x, x], _i32(1, 1), _i32(1, 1)) == ALIAS
    assert _move(lib, [x, x[:, 4:]], _i32(1, 1), _i32(1, 1)) == ALIAS
    idx = torch.zeros(5, 8, dtype=torch.int32)
    assert _move(lib, [idx], idx[:1, :2], _i32(1, 2)) == ALIAS
    assert _move(lib, [torch.zeros(5, 4)], _i32(1, 1), _i32(1, 1), n=257) == UNSUPPORTED
    assert _move(lib, [torch.zeros(5, 4)], None, _i32(1, 1)) == INVALID


# ---- kda_paged_attention_decode -----------------------------------------------------------


def _attend(N=3, Hq=4, Hkv=2, D=64, P=5, page=8, dtype=BF16):
    floats = binding.kda_paged_attention_workspace(Hq, Hkv, D, dtype, 152)
    return dict(q=torch.zeros(N, Hq, D, dtype=dtype), k_pages=torch.zeros(4, page, Hkv, D, dtype=dtype),
                v_pages=torch.zeros(4, page, Hkv, D, dtype=dtype), table=torch.zeros(N, P, dtype=torch.int32),
                lens=torch.zeros(N, dtype=torch.int32), work=torch.zeros(floats), out=torch.zeros(N, Hq, D, dtype=BF16),
                lse=torch.zeros(N, Hq))


def _call_attend(lib, t, window=0, scale=0.125):
    d = {n: _ptr(x) for n, x in t.items()}
    return lib.kda_paged_attention_decode(d["q"], d["k_pages"], d["v_pages"], d["table"], d["lens"], d["work"], window,
                                          scale, d["out"], d["lse"], None)


@pytest.mark.skipif(not NO_GPU, reason="a valid call would launch on host memory")
def test_attention_valid_calls_reach_the_device_query(lib):
    assert _call_attend(lib, _attend()) in (UNSUPPORTED, CUDA), _msg(lib)
    assert _call_attend(lib, {**_attend(), "lse": None}, window=7) in (UNSUPPORTED, CUDA), _msg(lib)
    assert _call_attend(lib, _attend(dtype=torch.float32)) in (UNSUPPORTED, CUDA), _msg(lib)
    assert _call_attend(lib, _attend(N=0)) == 0


@pytest.mark.parametrize("change,status,text", [
    (lambda t: t.update(q=torch.zeros(3, 3, 64, dtype=BF16)), INVALID, "evenly"),
    (lambda t: t.update(q=torch.zeros(3, 4, 96, dtype=BF16)), UNSUPPORTED, "head dimension 96"),
    (lambda t: t.update(q=torch.zeros(3, 4, 64)), INVALID, "k_pages: dtype must match q"),
    (lambda t: t.update(v_pages=torch.zeros(4, 8, 2, 64)), INVALID, "v_pages: dtype must match"),
    (lambda t: t.update(v_pages=torch.zeros(4, 8, 1, 64, dtype=BF16)), INVALID, "v_pages: axis 2"),
    (lambda t: t.update(table=torch.zeros(2, 5, dtype=torch.int32)), INVALID, "page_table: axis 0"),
    (lambda t: t.update(lens=torch.zeros(4, dtype=torch.int32)), INVALID, "seq_lens: axis 0"),
    (lambda t: t.update(work=torch.zeros(0)), None, None),
    (lambda t: t.update(work=torch.zeros(99, dtype=torch.int32)), INVALID, "workspace: dtype"),
    (lambda t: t.update(out=torch.zeros(3, 4, 64)), INVALID, "out: dtype"),
    (lambda t: t.update(lse=torch.zeros(3, 5)), INVALID, "lse: axis 1"),
    (lambda t: t.update(lse=torch.zeros(4, 3).t()), INVALID, "contiguous"),
    (lambda t: t.update(out=t["q"]), ALIAS, "out overlaps q"),
    (lambda t: t.update(lse=t["work"][:12].view(3, 4)), ALIAS, "workspace overlaps lse"),
    (lambda t: t.update(q=torch.zeros(3, 4, 66, dtype=BF16)[..., :64]), INVALID, "multiple of 4"),
    (lambda t: t.update(table=None), INVALID, "page_table: null"),
])
def test_attention_refusals(lib, change, status, text):
    t = _attend()
    change(t)
    got = _call_attend(lib, t)
    if status is None:
        assert got != 0
        return
    assert got == status, _msg(lib)
    assert text in _msg(lib)


def test_attention_refuses_bad_scalars_and_tables(lib):
    assert _call_attend(lib, _attend(), window=-1) == INVALID
    for scale in (0.0, -1.0, float("inf"), float("nan")):
        assert _call_attend(lib, _attend(), scale=scale) == INVALID
    t = _attend()
    d = {n: desc(x) for n, x in t.items()}
    d["table"].shape[1], d["table"].stride[0] = (1 << 27) + 1, 1 << 28  # refused before anything is read
    ptr = {n: ctypes.byref(x) for n, x in d.items()}
    assert lib.kda_paged_attention_decode(ptr["q"], ptr["k_pages"], ptr["v_pages"], ptr["table"], ptr["lens"],
                                          ptr["work"], 0, 0.125, ptr["out"], ptr["lse"], None) == UNSUPPORTED
    assert "2^30" in _msg(lib)


def test_attention_workspace_query(lib):
    for shape in ((8, 8, 64), (64, 8, 128), (40, 2, 256)):
        for dtype in (BF16, torch.float32):
            assert 0 < binding.kda_paged_attention_workspace(*shape, dtype, 152) < 1 << 24
    for args in ((8, 3, 64, BF16, 152), (8, 0, 64, BF16, 152), (8, 8, 80, BF16, 152), (8, 8, 64, torch.int32, 152),
                 (8, 8, 64, BF16, 0)):
        with pytest.raises(binding.KdaError):
            binding.kda_paged_attention_workspace(*args)


# ---- kda_beam_select ------------------------------------------------------------------------


def _beam(N=2, B=3, V=100, M=4, dtype=BF16):
    floats = binding.kda_beam_select_workspace(N, B, V, M, dtype, 152)
    return dict(logits=torch.zeros(N, B, V, dtype=dtype), scores=torch.zeros(N, B),
                finished=torch.zeros(N, B, dtype=torch.int32), work=torch.zeros(floats), s=torch.zeros(N, M),
                p=torch.zeros(N, M, dtype=torch.int32), t=torch.zeros(N, M, dtype=torch.int32))


def _call_beam(lib, t, eos=0):
    d = {n: _ptr(x) for n, x in t.items()}
    return lib.kda_beam_select(d["logits"], d["scores"], d["finished"], eos, d["work"], d["s"], d["p"], d["t"], None)


@pytest.mark.skipif(not NO_GPU, reason="a valid call would launch on host memory")
def test_beam_valid_calls_reach_the_device_query(lib):
    assert _call_beam(lib, _beam()) in (UNSUPPORTED, CUDA), _msg(lib)
    assert _call_beam(lib, {**_beam(dtype=torch.float32), "finished": None}, eos=-1) in (UNSUPPORTED, CUDA), _msg(lib)
    assert _call_beam(lib, {**_beam(), "logits": torch.zeros(3, 2, 120, dtype=BF16).transpose(0, 1)[..., 7:107]}) \
        in (UNSUPPORTED, CUDA), _msg(lib)
    assert _call_beam(lib, _beam(N=0)) == 0


@pytest.mark.parametrize("change,status,text", [
    (lambda t: t.update(logits=torch.zeros(2, 3, 100, dtype=torch.int32)), INVALID, "logits: dtype"),
    (lambda t: t.update(logits=torch.zeros(2, 100, 3, dtype=BF16).transpose(1, 2)), INVALID, "stride 1"),
    (lambda t: t.update(logits=torch.zeros(2, 33, 10, dtype=BF16)), UNSUPPORTED, "33 beams"),
    (lambda t: t.update(logits=torch.zeros(2, 3, 0, dtype=BF16)), UNSUPPORTED, "vocabulary of 0"),
    (lambda t: t.update(scores=torch.zeros(2, 4)), INVALID, "scores: axis 1"),
    (lambda t: t.update(scores=torch.zeros(3, 2).t()), INVALID, "scores: must be contiguous"),
    (lambda t: t.update(finished=torch.zeros(2, 3)), INVALID, "finished: dtype"),
    (lambda t: t.update(s=torch.zeros(2, 65)), UNSUPPORTED, "65 candidates"),
    (lambda t: t.update(p=torch.zeros(2, 5, dtype=torch.int32)), INVALID, "out_parents: axis 1"),
    (lambda t: t.update(t=torch.zeros(2, 4)), INVALID, "out_tokens: dtype"),
    (lambda t: t.update(t=t["p"]), ALIAS, "out_parents overlaps out_tokens"),
    (lambda t: t.update(s=t["work"][:8].view(2, 4)), ALIAS, "workspace overlaps out_scores"),
    (lambda t: t.update(work=None), INVALID, "workspace: null"),
])
def test_beam_refusals(lib, change, status, text):
    t = _beam()
    change(t)
    assert _call_beam(lib, t) == status, _msg(lib)
    assert text in _msg(lib)


def test_beam_refuses_tokens_outside_the_vocabulary(lib):
    for eos in (-1, 100):
        assert _call_beam(lib, _beam(), eos=eos) == INVALID and "eos_token" in _msg(lib)
    with pytest.raises(binding.KdaError):
        binding.kda_beam_select_workspace(1, 0, 10, 1, BF16, 152)


# ---- the marshalling module ----------------------------------------------------------------


def test_module_refuses_host_tensors_and_wrong_arguments(lib):
    m = binding._native()
    t = torch.zeros(2, 2)
    for call in (lambda: m.beam(t, t, None, None, None, 2, 0), lambda: m.move([t], t, t, None),
                 lambda: m.rope_append(*[t] * 10, False, 1.0), lambda: m.attention(*[t] * 5, None, None, None, False, 0, None)):
        with pytest.raises(ValueError, match="host"):
            call()
    with pytest.raises(TypeError, match="7 arguments"):
        m.beam(t)
    with pytest.raises(TypeError, match="list or tuple"):
        m.move(t, t, t, None)  # not the rows of a tensor
    with pytest.raises(TypeError, match="expected a tensor, got NoneType"):
        m.move([t], None, t, None)
    with pytest.raises(TypeError, match="expected a tensor, got int"):
        m.attention(*[7] * 11)


def test_module_describes_tensors_as_ctypes_does(lib):
    m = binding._native()
    base = torch.zeros(6, 4, 128, dtype=BF16)
    for t in [base, base[1:], base[:, ::2], base.transpose(0, 1), torch.zeros(3, dtype=torch.int32),
              torch.zeros(2, 3, 128, 128), torch.zeros(0, 4), base.as_strided((2, 2), (0, 5))]:
        assert m.describe(t) == bytes(desc(t))
    for t, kind, text in [(base.double(), TypeError, "unsupported dtype"), (base[None, None], ValueError, "rank 5"),
                          (torch.tensor(1.0), ValueError, "rank 0"), (base.to_sparse(), TypeError, "strided")]:
        with pytest.raises(kind, match=text):
            m.describe(t)


def test_rope_refuses_written_views_whose_elements_overlap(lib):
    t = _rope()
    t["k_pages"] = torch.as_strided(torch.zeros(4 * 8 * 2 * 64, dtype=BF16), (4, 8, 2, 64), (512, 128, 32, 1))
    assert _call_rope(lib, t) == INVALID and "k_pages: elements overlap" in _msg(lib)
    t = _rope()
    t["q_out"] = torch.as_strided(torch.zeros(3 * 4 * 64, dtype=BF16), (3, 4, 64), (64, 64, 1))
    assert _call_rope(lib, t) == INVALID and "q_out: elements overlap" in _msg(lib)
