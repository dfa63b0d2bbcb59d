"""Float64 CPU oracle of the operators around the recurrent layers: rotary
positions with the paged cache write, attention of one new token over the
pages, beam selection, and slot moves.

TEST INFRASTRUCTURE ONLY, like ``kda_oracle``: plain numpy in float64, from
the definitions in include/kda.h, sharing no code with the library.  Inputs
are the stored values; nothing is rounded.
"""

from __future__ import annotations

import math

import numpy as np


def rope_frequencies(rot_dim, base=10000.0, factor=1.0, original_len=0.0, low=1.0, high=32.0):
    """Radians per position of each pair, slowed down by parts for long contexts."""
    f = base ** (-2.0 * np.arange(rot_dim // 2) / max(rot_dim, 1))
    keep = np.zeros_like(f)
    if original_len > 0:
        keep = np.clip((original_len * f / (2 * math.pi) - low) / (high - low), 0.0, 1.0)
    return f * (keep + (1.0 - keep) / factor)


def rotate(x, pos, freq, interleaved, amplitude):
    """x [heads, D] at one position; pairs (i, i + rot/2) or (2i, 2i + 1)."""
    y = np.array(x, dtype=np.float64)
    half = len(freq)
    angle = pos * freq
    c, s = amplitude * np.cos(angle), amplitude * np.sin(angle)
    ia = 2 * np.arange(half) if interleaved else np.arange(half)
    ib = ia + 1 if interleaved else ia + half
    a, b = x[:, ia], x[:, ib]
    y[:, ia] = a * c - b * s
    y[:, ib] = a * s + b * c
    return y


def rope_append(q, k, v, freq, seq_lens, page_table, k_pages, v_pages, cu_seqlens=None, interleaved=False,
                amplitude=1.0):
    """(q_out, k_pages, v_pages) after the call; the inputs are not changed."""
    R = q.shape[0]
    q_out = np.zeros_like(q, dtype=np.float64)
    kp, vp = np.array(k_pages, dtype=np.float64), np.array(v_pages, dtype=np.float64)
    num_pages, page = kp.shape[:2]
    for n in range(len(seq_lens)):
        b, e = (n, n + 1) if cu_seqlens is None else (int(cu_seqlens[n]), min(int(cu_seqlens[n + 1]), R))
        for r in range(max(b, 0), e):
            pos = int(seq_lens[n]) - e + r
            if pos < 0:
                continue
            q_out[r] = rotate(q[r], pos, freq, interleaved, amplitude)
            if pos // page >= page_table.shape[1]:
                continue
            p = int(page_table[n, pos // page])
            if 0 < p < num_pages:
                kp[p, pos % page] = rotate(k[r], pos, freq, interleaved, amplitude)
                vp[p, pos % page] = v[r]
    return q_out, kp, vp


def paged_attention(q, k_pages, v_pages, page_table, seq_lens, window=0, scale=None):
    """(out [N, Hq, D], lse [N, Hq]); a row without live positions gives 0 and -inf."""
    N, Hq, D = q.shape
    num_pages, page, Hkv, _ = k_pages.shape
    G = Hq // Hkv
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    out, lse = np.zeros((N, Hq, D)), np.full((N, Hq), -np.inf)
    for n in range(N):
        length = min(int(seq_lens[n]), page_table.shape[1] * page)
        first = max(0, int(seq_lens[n]) - window) if window > 0 else 0
        at = np.arange(first, max(length, first))
        pages = page_table[n][at // page] if len(at) else np.zeros(0, dtype=np.int64)
        ok = (pages > 0) & (pages < num_pages)
        at, pages = at[ok], pages[ok]
        if len(at) == 0:
            continue
        for h in range(Hkv):
            K = k_pages[pages, at % page, h].astype(np.float64)
            V = v_pages[pages, at % page, h].astype(np.float64)
            s = scale * (q[n, h * G:(h + 1) * G].astype(np.float64) @ K.T)
            m = s.max(axis=1, keepdims=True)
            p = np.exp(s - m)
            total = p.sum(axis=1, keepdims=True)
            out[n, h * G:(h + 1) * G] = (p @ V) / total
            lse[n, h * G:(h + 1) * G] = (m + np.log(total))[:, 0]
    return out, lse


def beam_candidates(logits, scores, finished=None, eos_token=0):
    """Candidate values [N, B, V] in float64; -inf where there is no candidate."""
    x = np.asarray(logits, dtype=np.float64)
    N, B, V = x.shape
    c = np.full((N, B, V), -np.inf)
    for n in range(N):
        for b in range(B):
            s = float(scores[n, b])
            if not np.isfinite(s):
                continue
            if finished is not None and finished[n, b] != 0:
                c[n, b, eos_token] = s
                continue
            with np.errstate(all="ignore"):
                m = np.max(x[n, b])
                total = np.sum(np.exp(x[n, b] - m))
                if np.isfinite(m) and np.isfinite(total):
                    c[n, b] = (x[n, b] - m) - np.log(total) + s
    return c


def beam_select(logits, scores, num_out, finished=None, eos_token=0):
    """(scores, parents, tokens), each [N, num_out]; -inf, -1, -1 past the last candidate."""
    c = beam_candidates(logits, scores, finished, eos_token)
    N, B, V = c.shape
    so = np.full((N, num_out), -np.inf)
    po, to = np.full((N, num_out), -1, dtype=np.int64), np.full((N, num_out), -1, dtype=np.int64)
    for n in range(N):
        flat = c[n].reshape(-1)
        order = np.argsort(-flat, kind="stable")[:num_out]
        order = order[flat[order] > -np.inf]
        so[n, :len(order)] = flat[order]
        po[n, :len(order)], to[n, :len(order)] = order // V, order % V
    return so, po, to


def pool_move(pools, src, dst, parents=None):
    """New copies of `pools` (numpy arrays, axis 0 = slots) after the move."""
    out = [p.copy() for p in pools]
    for old, new in zip(pools, out):
        slots = old.shape[0]
        for n in range(src.shape[0]):
            for j in range(src.shape[1]):
                p = j if parents is None else int(parents[n, j])
                d = int(dst[n, j])
                if not (0 <= p < src.shape[1]) or not (0 < d < slots):
                    continue
                s = int(src[n, p])
                new[d] = old[s] if 0 < s < slots else 0
    return out
