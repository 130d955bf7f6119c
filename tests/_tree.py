"""The tree step's operators written out plainly in 64 bits (numpy), for the
tests of pkv_slot_map, pkv_rope_append_axes, pkv_decode_attn_tree and
pkv_tree_commit, and the random inputs those tests share."""
from __future__ import annotations

import numpy as np
import torch

E4M3 = torch.float8_e4m3fn


def parents_of(rng, n, kind="random"):
    """Parents of n drafted tokens: any earlier one or -1; a chain; or a star."""
    if kind == "chain":
        return [i - 1 for i in range(n)]
    if kind == "star":
        return [-1] * n
    return [int(rng.integers(-1, i)) for i in range(n)]


def ancestors(parents):
    """[n, n] truth values: token j is token i or one of its ancestors."""
    n = len(parents)
    seen = np.zeros((n, n), bool)
    for i, p in enumerate(parents):
        if p >= 0:
            seen[i] = seen[p]
        seen[i, i] = True
    return seen


def pack(seen, words):
    """[n, m] truth values to [n, words] int32 words."""
    out = np.zeros((seen.shape[0], words), np.uint32)
    for j in range(min(seen.shape[1], 32 * words)):
        out[:, j // 32] |= seen[:, j].astype(np.uint32) << np.uint32(j % 32)
    return out.view(np.int32)


def slot_map(seq_lens, new_lens, table, held, free, count, P, cap, parents=None, words=0):
    """The plan as its definition says it, request by request."""
    table, B = table.copy(), len(seq_lens)
    slots, pos = np.full(cap, -1, np.int32), np.full(cap, -1, np.int32)
    mask = np.zeros((cap, words), np.int32)
    pages_out, cu = held.copy(), np.zeros(B + 1, np.int64)
    asked = taken = 0
    oom = False
    for b in range(B):
        L, n, h = int(seq_lens[b]), int(new_lens[b]), int(held[b])
        cu[b + 1] = cu[b] + n
        need = max(h, -(-(L + n) // P))
        served = need == h or asked + need - h <= count
        if served:
            for k in range(need - h):
                table[b, h + k] = free[count - 1 - (asked + k)]
            pages_out[b] = need
            if need > h:
                taken = asked + need - h
        oom |= not served
        asked += need - h
        par = None if parents is None else [int(x) for x in parents[cu[b]:cu[b + 1]]]
        seen = None if par is None else ancestors(par)
        for i in range(n):
            row = cu[b] + i
            if row >= cap:
                break
            pos[row] = L + (i if par is None else int(seen[i].sum()) - 1)
            if par is not None:
                mask[row] = pack(seen[i:i + 1], words)[0]
            if served:
                slots[row] = table[b, (L + i) // P] * P + (L + i) % P
    return dict(table=table, pages=pages_out, left=count - taken, cu=np.minimum(cu, cap).astype(np.int32),
                slots=slots, pos=pos, mask=mask, oom=oom)


def pair_axes(sections, interleaved):
    half, n = sum(sections), len(sections)
    if not interleaved:
        return [a for a in range(n) for _ in range(sections[a])]
    return [i % n if i < n * sections[i % n] else 0 for i in range(half)]


def rotate(x, positions, sections, interleaved, base):
    """x [n, heads, d] in 64 bits turned by the positions [axes, n]."""
    half = x.shape[-1] // 2
    theta = base ** (-2.0 * np.arange(half) / (2 * half))
    phi = np.stack([positions[a].astype(np.float64) * theta[i]
                    for i, a in enumerate(pair_axes(sections, interleaved))], -1)[:, None]
    a, b = x[..., :half], x[..., half:]
    return np.concatenate([a * np.cos(phi) - b * np.sin(phi), b * np.cos(phi) + a * np.sin(phi)], -1)


def attention(q, k, v, seq_lens, cu, table, mask, P, G):
    """q [n, Hq, d]; k, v [pages, Hkv, P, d] values, all in 64 bits; mask
    [n, words].  Returns the output and the sum of weight x |v| of each element."""
    out, size = np.zeros(q.shape), np.zeros(q.shape)
    for b in range(len(seq_lens)):
        L, T = int(seq_lens[b]), int(cu[b + 1] - cu[b])
        if T == 0:
            continue
        pages = table[b, :-(-(L + T) // P)]
        kb = k[pages].transpose(1, 0, 2, 3).reshape(k.shape[1], -1, k.shape[3])[:, :L + T]
        vb = v[pages].transpose(1, 0, 2, 3).reshape(v.shape[1], -1, v.shape[3])[:, :L + T]
        for i in range(T):
            row = int(cu[b]) + i
            w = mask[row].view(np.uint32)
            see = np.array([True] * L + [bool((int(w[j // 32]) >> (j % 32)) & 1) for j in range(T)])
            if not see.any():
                continue
            for h in range(q.shape[1]):
                s = kb[h // G][see] @ q[row, h] / np.sqrt(q.shape[2])
                p = np.exp(s - s.max())
                p /= p.sum()
                out[row, h] = p @ vb[h // G][see]
                size[row, h] = p @ np.abs(vb[h // G][see])
    return out, size


def pools(gen, pages, Hkv, P, d, fp8):
    """(k, v, k_scale, v_scale) on the CPU and their values in 64 bits."""
    got = []
    for _ in range(2):
        x = torch.randn(pages, Hkv, P, d, generator=gen)
        if not fp8:
            x = x.to(torch.bfloat16)
            got.append((x, None, x.double().numpy()))
            continue
        x *= torch.empty(pages, Hkv, 1, 1).uniform_(0.5, 3.0, generator=gen)
        s = x.abs().amax((2, 3)) / 448
        c = (x / s[:, :, None, None]).clamp(-448, 448).to(E4M3)
        got.append((c, s, c.double().numpy() * s.double().numpy()[:, :, None, None]))
    (k, ks, kv), (v, vs, vv) = got
    return k, v, ks, vs, kv, vv


def tables(rng, counts, extra=3):
    """[batch, stride] block tables of counts[b] pages each in random order (-1 behind) and the pages in all."""
    total = int(sum(counts)) + extra
    order = rng.permutation(total).astype(np.int32)
    table = np.full((len(counts), max(1, max(counts))), -1, np.int32)
    at = 0
    for b, c in enumerate(counts):
        table[b, :c] = order[at:at + c]
        at += c
    return table, total, order[at:]


def values(t):
    """A tensor as 64-bit numbers on the host."""
    return t.detach().cpu().double().numpy()
