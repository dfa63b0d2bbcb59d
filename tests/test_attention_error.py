"""The root-mean-square criterion of the attention tests tells a sound computation from mistakes planted in it (CPU)."""

import numpy as np
import pytest
import torch

from tests.attention_error import F32, assert_rms, softmax_moments

TILE = 64


def bf16(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(torch.bfloat16).float().numpy()


def attention_in_pieces(q, k, v, scale, pieces, mistake=None):
    """softmax(scale q k) v in float32 over `pieces` runs of tiles, weights as two bfloat16, joined; rounded to bfloat16."""
    L = k.shape[0]
    cuts = [min(L, TILE * (c * -(-L // TILE) // pieces)) for c in range(pieces)] + [L]
    parts = []
    for a, b in zip(cuts, cuts[1:]):
        s = (q @ k[a:b].T) * np.float32(scale)
        m = s.max(-1, keepdims=True)
        p = np.exp(s - m)
        hi = bf16(p)
        lo = bf16(p - hi)
        w = hi if mistake == "no low part" else hi + lo
        parts.append((m, p.sum(-1, keepdims=True), w @ v[a:b]))
    top = np.max([m for m, _, _ in parts], axis=0)
    total, out = 0.0, 0.0
    for c, (m, l, o) in enumerate(parts):
        f = np.exp(m - top)
        total = total + f * l
        if c == pieces // 2 and mistake == "one piece's output missing":
            continue
        out = out + (1.0 if c == pieces // 2 and mistake == "one piece not rescaled" else f) * o
    return bf16(out / total)


@pytest.mark.parametrize("L,pieces,mistake", [(1000, 1, None), (1000, 1, "no low part")] + [
    (L, pieces, mistake) for L, pieces in ((1000, 8), (70000, 152))
    for mistake in (None, "no low part", "one piece's output missing", "one piece not rescaled")])
def test_mistakes_are_told_from_rounding(L, pieces, mistake):
    rng = np.random.default_rng(L)
    D, heads = 128, 64
    q, k, v = (bf16(rng.standard_normal(shape)) for shape in ((heads, D), (L, D), (L, D)))
    out, _, weighted, spread = softmax_moments(*(x.astype(np.float64) for x in (q, k, v)), D ** -0.5)
    got = attention_in_pieces(q, k, v, D ** -0.5, pieces, mistake).astype(np.float64)
    score = 64 * F32 * np.linalg.norm(q, axis=1).max() * np.linalg.norm(k, axis=1).max() * D ** -0.5

    def held():
        assert_rms(got, out, weighted, spread, score, 2.0 ** -16, "model")
    if mistake is None:
        held()
    else:
        with pytest.raises(AssertionError, match="root mean square"):
            held()
