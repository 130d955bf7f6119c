"""GPU tests of the tree step: pkv_slot_map, pkv_rope_append_axes,
pkv_decode_attn_tree and pkv_tree_commit, each against its definition in 64
bits (tests/_tree.py) at the sizes and masks where it can go wrong, then the
four together as a speculative step uses them, eager and captured.

Tolerances, by arithmetic: one rounding to bf16 is off by at most 2^-8 of the
value.  Attention adds to it 2^-8 + 2^-12 of A = sum of weight x |v|: each
weight is rounded to bf16 for the matrix product (2^-8 of itself), and carries
an error of at most d 2^-23 sqrt(d) ~ 2^-13.6 for the fp32 score sums of
N(0, 1) data at d = 128 and 2^-21 from exp2 and the sums.  Rotation adds 2^-20 (|a| + |b|): an angle
off by 2^-22 and three fp32 roundings.  E4M3 codes are off by at most 2^-4 of
the value or half the smallest step, 2^-10 scale."""
import numpy as np
import pytest
import torch

from tests import _tree

pytestmark = pytest.mark.gpu
DEV = "cuda"
W = 2.0 ** -8 + 2.0 ** -12      # share of A by which the attention may be off


@pytest.fixture(scope="module")
def pkv():
    from paged_kv_flight_b200 import pkv as mod
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return mod


class _Ctx:
    def __init__(self, pkv, Hq, Hkv, d, P, fp8, batch, blocks, pages, base=1e4):
        self.pkv = pkv
        self.h = pkv.pkv_create(pkv.make_config(Hq, Hkv, d, P, "fp8" if fp8 else "bf16", base, batch, blocks, pages))

    def __enter__(self):
        return self.h

    def __exit__(self, *a):
        torch.cuda.synchronize()
        self.pkv.pkv_destroy(self.h)


def _i(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device=DEV)


def _ok(pkv, ctx):
    st, bits = pkv.pkv_check_device_error(ctx)
    assert st == pkv.PKV_OK, (st, bits)


def _status(pkv, ctx):
    return pkv.pkv_check_device_error(ctx)


# ---- slot map ------------------------------------------------------------------

def _slot_inputs(rng, B, P, lo, hi, t_lo, t_hi, tree, kind="random", spare=5, short=0):
    lens = rng.integers(lo, hi + 1, B)
    new = rng.integers(t_lo, t_hi + 1, B)
    held = -(-lens // P) + rng.integers(0, 2, B) * (rng.random(B) < 0.3)
    need = np.maximum(held, -(-(lens + new) // P))
    table, pages, rest = _tree.tables(rng, need.tolist(), spare)
    taken = [int(table[b, k]) for b in range(B) for k in range(held[b], need[b])]
    for b in range(B):
        table[b, held[b]:] = -1
    stack = rng.permutation(np.array(taken + rest.tolist(), np.int32)).astype(np.int32)
    count = max(0, len(taken) - short) if short else len(stack)
    parents = np.concatenate([np.array(_tree.parents_of(rng, int(n), kind), np.int32) for n in new] +
                             [np.zeros(0, np.int32)]) if tree else None
    return dict(lens=lens.astype(np.int32), new=new.astype(np.int32), held=held.astype(np.int32), table=table,
                pages=pages, free=stack, count=count, parents=parents)


def _slot_call(pkv, ctx, x, cap, words, inplace=False):
    d = {k: _i(x[k]) for k in ("lens", "new", "held", "table", "free")}
    count = _i([x["count"]])
    g = dict(table=d["table"], cu=_i(np.full(len(x["lens"]) + 1, 77)), slots=_i(np.full(cap, 77)),
             pos=_i(np.full(cap, 77)), pages=d["held"] if inplace else _i(np.full(len(x["lens"]), 77)),
             left=count if inplace else _i([77]))
    par = None
    if x["parents"] is not None:
        par = _i(np.concatenate([x["parents"], np.full(max(0, cap - len(x["parents"])), -1)])[:cap])
        g["mask"] = _i(np.full((cap, words), 77))
    pkv.pkv_slot_map(ctx, d["lens"], d["new"], d["table"], d["held"], d["free"], count, g["cu"], g["slots"], g["pos"],
                     g["pages"], g["left"], parents=par, tree_mask=g.get("mask"))
    return g


def _slot_check(g, r):
    for k in ("table", "pages", "cu", "slots", "pos"):
        assert np.array_equal(g[k].cpu().numpy(), r[k]), k
    assert int(g["left"][0]) == r["left"]
    if "mask" in g:
        assert np.array_equal(g["mask"].cpu().numpy(), r["mask"])


@pytest.mark.parametrize("B,P,lo,hi,t_lo,t_hi,tree,kind,pad", [
    (1, 16, 0, 0, 1, 1, False, "", 0),            # the first token of all
    (4, 16, 17, 255, 1, 1, False, "", 0),
    (5, 32, 0, 90, 0, 40, False, "", 13),         # requests with nothing new
    (37, 64, 0, 300, 0, 200, False, "", 0),
    (6, 16, 0, 60, 1, 7, True, "random", 0),
    (33, 16, 10, 100, 0, 32, True, "random", 9),
    (7, 32, 1, 64, 60, 64, True, "chain", 5),     # chains over two mask words
    (7, 32, 1, 64, 20, 100, True, "random", 5),   # four words
    (3, 16, 0, 8, 30, 33, True, "star", 0),
    (300, 16, 0, 200, 0, 12, True, "random", 100),
    (1000, 16, 0, 40, 0, 9, False, "", 3),
])
@pytest.mark.parametrize("inplace", [False, True])
def test_slot_map(pkv, B, P, lo, hi, t_lo, t_hi, tree, kind, pad, inplace):
    rng = np.random.default_rng(B + t_hi)
    x = _slot_inputs(rng, B, P, lo, hi, t_lo, t_hi, tree, kind or "random")
    cap, words = int(x["new"].sum()) + pad, -(-max(1, t_hi) // 32)
    r = _tree.slot_map(x["lens"], x["new"], x["table"], x["held"], x["free"], x["count"], P, cap, x["parents"], words)
    assert not r["oom"]
    if cap == 0:
        pytest.skip("no row")
    with _Ctx(pkv, 8, 2, 64, P, False, B, x["table"].shape[1], x["pages"]) as ctx:
        _slot_check(_slot_call(pkv, ctx, x, cap, words, inplace), r)
        _ok(pkv, ctx)


@pytest.mark.parametrize("short", [1, 3, 1000])
def test_slot_map_out_of_pages(pkv, short):
    """Requests whose pages the stack cannot cover keep theirs, get no slot and
    take nothing; requests that need no page are served wherever they stand."""
    rng = np.random.default_rng(short)
    x = _slot_inputs(rng, 20, 16, 0, 100, 0, 40, True, short=short)
    cap = int(x["new"].sum())
    r = _tree.slot_map(x["lens"], x["new"], x["table"], x["held"], x["free"], x["count"], 16, cap, x["parents"], 2)
    assert r["oom"]
    with _Ctx(pkv, 8, 2, 64, 16, False, 20, x["table"].shape[1], x["pages"]) as ctx:
        _slot_check(_slot_call(pkv, ctx, x, cap, 2), r)
        assert _status(pkv, ctx) == (pkv.PKV_ERR_OOM, 16)
        _ok(pkv, ctx)                                       # read and cleared


def test_slot_map_out_of_range(pkv):
    """Values out of range are reported and cost only their own request."""
    rng = np.random.default_rng(5)
    x = _slot_inputs(rng, 6, 16, 20, 60, 3, 9, True)
    good = dict(x)
    for key, b, v, bits in (("lens", 2, -1, 1), ("new", 3, -4, 1), ("held", 1, 0, 1), ("held", 1, 1000, 1),
                            ("new", 4, 33, 1), ("lens", 0, 1 << 30, 1)):
        x = dict(good, **{key: good[key].copy()})
        x[key][b] = v
        cap = int(np.maximum(x["new"], 0).sum())
        if key == "new" and v > 0:      # more than the mask's words hold
            x["parents"] = np.concatenate([np.array(_tree.parents_of(rng, int(n)), np.int32) for n in x["new"]])
        elif key == "new":
            cu = np.concatenate([[0], np.cumsum(good["new"])])
            x["parents"] = np.delete(good["parents"], range(cu[b], cu[b + 1]))
        with _Ctx(pkv, 8, 2, 64, 16, False, 6, x["table"].shape[1], x["pages"]) as ctx:
            g = _slot_call(pkv, ctx, x, cap, 1)
            cu = np.concatenate([[0], np.cumsum(np.maximum(x["new"], 0))])
            assert np.array_equal(g["cu"].cpu().numpy(), cu)
            slots = g["slots"].cpu().numpy()
            assert (slots[cu[b]:cu[b + 1]] == -1).all()
            assert (np.delete(slots, range(cu[b], cu[b + 1])) >= 0).all()
            assert int(g["pages"][b]) == x["held"][b]
            assert _status(pkv, ctx) == (pkv.PKV_ERR_DEVICE_BOUNDS, bits)
    # a parent that is not an earlier token: that token alone has no slot
    x = dict(good, parents=good["parents"].copy())
    x["parents"][0] = 0
    kids = np.flatnonzero(_tree.ancestors(good["parents"][:good["new"][0]].tolist())[:, 0])
    with _Ctx(pkv, 8, 2, 64, 16, False, 6, x["table"].shape[1], x["pages"]) as ctx:
        g = _slot_call(pkv, ctx, x, len(x["parents"]), 1)
        slots = g["slots"].cpu().numpy()
        assert (slots[kids] == -1).all() and (np.delete(slots, kids) >= 0).all()
        assert (g["mask"].cpu().numpy()[kids] == 0).all()
        assert _status(pkv, ctx) == (pkv.PKV_ERR_DEVICE_BOUNDS, 8)
        # fewer rows than tokens: the surplus is dropped
        x = dict(good)
        g = _slot_call(pkv, ctx, x, 10, 1)
        assert int(g["cu"][-1]) == 10 and (g["slots"].cpu().numpy() >= 0).all()
        assert _status(pkv, ctx) == (pkv.PKV_ERR_DEVICE_BOUNDS, 1)
        # a stack entry that is no page
        x = dict(good, free=np.full_like(good["free"], 1 << 20))
        _slot_call(pkv, ctx, x, len(x["parents"]), 1)
        assert _status(pkv, ctx)[1] & 2


# ---- rotation and append -----------------------------------------------------

ROPE_CASES = [
    # Hq, Hkv, d, P, fp8, tokens, sections, interleaved
    (8, 2, 64, 16, False, 1, [32], False),
    (8, 8, 64, 16, False, 7, [8, 12, 12], False),
    (32, 8, 128, 32, False, 65, [16, 24, 24], False),
    (32, 8, 128, 32, True, 33, [24, 20, 20], True),
    (40, 8, 128, 64, False, 130, [22, 21, 21], True),
    (10, 2, 64, 16, True, 50, [20, 0, 12], False),
    (21, 3, 128, 16, True, 19, [33, 16, 15, 0], True),
    (6, 2, 128, 16, False, 300, [64], False),
]


@pytest.mark.parametrize("Hq,Hkv,d,P,fp8,n,sections,interleaved", ROPE_CASES)
@pytest.mark.parametrize("inplace", [False, True])
def test_rope_append_axes(pkv, Hq, Hkv, d, P, fp8, n, sections, interleaved, inplace):
    rng = np.random.default_rng(n)
    gen = torch.Generator().manual_seed(n)
    pages = -(-n // P) + 3
    k, v, ks, vs, _, _ = _tree.pools(gen, pages, Hkv, P, d, fp8)
    q, kn, vn = (torch.randn(n, h, d, generator=gen).to(torch.bfloat16) for h in (Hq, Hkv, Hkv))
    pos = rng.integers(-50, 3_000_000, (len(sections), n))
    pos[0, 0] = 2 ** 31 - 1
    slots = rng.permutation(pages * P)[:n].astype(np.int32)
    skip = rng.random(n) < 0.2
    skip[0] = False
    slots[skip] = -1
    turned_q = _tree.rotate(_tree.values(q), pos, sections, interleaved, 1e4)
    turned_k = _tree.rotate(_tree.values(kn), pos, sections, interleaved, 1e4)
    dq, dk, dv = q.to(DEV), k.to(DEV), v.to(DEV)
    out = dq if inplace else torch.full_like(dq, 3.0)
    sc = [None if s is None else s.to(DEV) for s in (ks, vs)]
    with _Ctx(pkv, Hq, Hkv, d, P, fp8, 1, 1, pages) as ctx:
        pkv.pkv_rope_append_axes(ctx, dq, kn.to(DEV), vn.to(DEV), _i(pos), sections, _i(slots), out, dk, dv, *sc,
                                 interleaved=interleaved)
        _ok(pkv, ctx)
    got = _tree.values(out)
    half = d // 2

    def slack(x):
        a = np.abs(_tree.values(x))
        s = a[..., :half] + a[..., half:]
        return 2.0 ** -20 * np.concatenate([s, s], -1)

    live = ~skip
    assert (np.abs(got - turned_q) <= 2.0 ** -8 * np.abs(turned_q) + slack(q))[live].all()
    assert np.array_equal(got[skip], _tree.values(q)[skip] if inplace else np.full_like(got[skip], 3.0))
    page, at = slots[live] // P, slots[live] % P
    gk, gv = dk.cpu(), dv.cpu()
    wk, wv = gk[page, :, at].double().numpy(), gv[page, :, at]
    if fp8:
        s = ks.double().numpy()[page][..., None]
        want = np.clip(turned_k[live] / s, -448, 448)
        assert (np.abs(wk - want) <= 2.0 ** -4 * np.abs(want) + 2.0 ** -10 + slack(kn)[live] / s).all()
        sv = vs[page][..., None]
        assert torch.equal(wv.view(torch.uint8), (vn[live].float() / sv).clamp(-448, 448).to(_tree.E4M3).view(torch.uint8))
    else:
        assert (np.abs(wk - turned_k[live]) <= 2.0 ** -8 * np.abs(turned_k[live]) + slack(kn)[live]).all()
        assert torch.equal(wv, vn[live])
    # nothing else in the pools has moved
    for g, o in ((gk, k), (gv, v)):
        g, o = g.clone().view(torch.uint8), o.clone().view(torch.uint8)
        g[page, :, at] = 0
        o[page, :, at] = 0
        assert torch.equal(g, o)


def test_rope_append_axes_bad_slot(pkv):
    gen = torch.Generator().manual_seed(0)
    k, v, _, _, _, _ = _tree.pools(gen, 2, 2, 16, 64, False)
    dk, dv = k.to(DEV), v.to(DEV)
    q = torch.randn(3, 4, 64, generator=gen).to(torch.bfloat16).to(DEV)
    kn = torch.randn(3, 2, 64, generator=gen).to(torch.bfloat16).to(DEV)
    out = torch.zeros_like(q)
    with _Ctx(pkv, 4, 2, 64, 16, False, 1, 1, 2) as ctx:
        for bad in (32, -2, 2 ** 31 - 1, -2 ** 31):
            pkv.pkv_rope_append_axes(ctx, q, kn, kn, _i([[0, 0, 0]]), [32], _i([bad, 5, bad]), out, dk, dv, None, None)
            assert _status(pkv, ctx) == (pkv.PKV_ERR_DEVICE_BOUNDS, 2)
            assert (out[0] == 0).all() and torch.equal(out[1], q[1])
        torch.cuda.synchronize()
        k[0, :, 5], v[0, :, 5] = kn[1].cpu(), kn[1].cpu()
        assert torch.equal(dk.cpu(), k) and torch.equal(dv.cpu(), v)


# ---- attention -------------------------------------------------------------------

ATTN_CASES = [
    # Hq, Hkv, d, P, fp8, cached, new, kind
    (8, 2, 64, 16, False, [17], [1], "random"),
    (8, 2, 64, 16, False, [0, 0, 5], [1, 3, 2], "random"),             # nothing cached
    (8, 2, 64, 16, False, [31, 200, 0, 63], [7, 1, 0, 4], "random"),   # a request with nothing new
    (32, 8, 128, 32, False, [100, 513, 127, 128, 129], [9, 16, 1, 12, 8], "random"),
    (32, 8, 128, 16, True, [100, 700, 16, 0], [5, 24, 16, 33], "random"),
    (8, 2, 64, 64, True, [64, 300, 1], [24, 64, 5], "star"),
    (8, 1, 128, 16, False, [90, 255], [17, 64], "random"),             # rows over several blocks
    (12, 4, 64, 16, False, [250, 33], [43, 90], "random"),             # groups of 3
    (10, 2, 128, 32, False, [120, 5], [26, 51], "chain"),              # groups of 5
    (12, 2, 128, 16, True, [99], [22], "random"),                      # 6
    (14, 2, 64, 16, False, [77, 128], [19, 36], "random"),             # 7
    (4, 4, 128, 16, False, [130, 60], [129, 257], "random"),           # nine mask words
    (8, 8, 64, 16, True, [40], [140], "chain"),
    (16, 2, 128, 64, False, [5000, 3], [6, 2], "random"),              # one long request
    (8, 1, 64, 16, True, [9000], [1], "random"),
    (8, 1, 128, 16, False, [1100], [40], "random"),
]


def _attn_inputs(case, seed=0):
    Hq, Hkv, d, P, fp8, lens, new, kind = case
    rng = np.random.default_rng(seed + sum(lens))
    gen = torch.Generator().manual_seed(seed + sum(new))
    table, pages, _ = _tree.tables(rng, [-(-(a + t) // P) for a, t in zip(lens, new)])
    k, v, ks, vs, kv, vv = _tree.pools(gen, pages, Hkv, P, d, fp8)
    n, words = sum(new), -(-max(new) // 32)
    mask = np.concatenate([_tree.pack(_tree.ancestors(_tree.parents_of(rng, t, kind)), words) for t in new if t])
    q = torch.randn(n, Hq, d, generator=gen).to(torch.bfloat16)
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    return dict(q=q, k=k, v=v, ks=ks, vs=vs, kv=kv, vv=vv, table=table, pages=pages, mask=mask, cu=cu,
                lens=np.array(lens, np.int32), case=case)


def _attn_device(x):
    g = {k: x[k].to(DEV) for k in ("q", "k", "v")}
    g.update({k: None if x[k] is None else x[k].to(DEV) for k in ("ks", "vs")})
    g.update({k: _i(x[k]) for k in ("table", "mask", "cu", "lens")})
    return g


def _attn_ctx(pkv, x, batch=None):
    Hq, Hkv, d, P, fp8, lens, new, _ = x["case"]
    return _Ctx(pkv, Hq, Hkv, d, P, fp8, batch or len(lens), x["table"].shape[1], x["pages"])


def _attn_run(pkv, ctx, g, out=None):
    out = torch.full_like(g["q"], float("nan")) if out is None else out
    pkv.pkv_decode_attn_tree(ctx, g["q"], g["k"], g["v"], g["ks"], g["vs"], g["table"], g["lens"], g["cu"], g["mask"],
                             out)
    return out


def _attn_near(out, ref, size):
    got = _tree.values(out)
    err = np.abs(got - ref) - (2.0 ** -8 * np.abs(ref) + W * size)
    assert (err <= 0).all(), (float(np.nanmax(err)), int((~(err <= 0)).sum()))


def _attn_ref(x):
    Hq, Hkv, d, P = x["case"][:4]
    return _tree.attention(_tree.values(x["q"]), x["kv"], x["vv"], x["lens"], x["cu"], x["table"], x["mask"], P,
                           Hq // Hkv)


@pytest.mark.parametrize("case", ATTN_CASES, ids=lambda c: f"h{c[0]}_{c[1]}_d{c[2]}_p{c[3]}_{'f8' if c[4] else 'bf'}_{c[5][0]}")
def test_tree_attention(pkv, case):
    x = _attn_inputs(case)
    ref, size = _attn_ref(x)
    g = _attn_device(x)
    with _attn_ctx(pkv, x) as ctx:
        out = _attn_run(pkv, ctx, g)
        _ok(pkv, ctx)
        _attn_near(out, ref, size)
        assert torch.equal(out, _attn_run(pkv, ctx, g))          # bit for bit


@pytest.mark.parametrize("fp8", [False, True])
def test_tree_attention_many_requests(pkv, fp8):
    """More work items than SMs, lengths of every kind, whole and split."""
    rng = np.random.default_rng(8)
    lens = [int(x) for x in rng.integers(0, 500, 70)]
    new = [int(x) for x in rng.integers(0, 20, 70)]
    lens[11], new[11] = 4000, 12
    x = _attn_inputs((16, 4, 64, 16, fp8, lens, new, "random"))
    ref, size = _attn_ref(x)
    with _attn_ctx(pkv, x) as ctx:
        out = _attn_run(pkv, ctx, _attn_device(x))
        _ok(pkv, ctx)
        _attn_near(out, ref, size)


@pytest.mark.parametrize("fp8", [False, True])
def test_tree_attention_masks(pkv, fp8):
    """Masks that are no tree: rows that see nothing at all are zero, rows may
    leave themselves out, bits past the request's tokens are ignored."""
    x = _attn_inputs((8, 2, 128, 16, fp8, [0, 40, 0, 127], [6, 30, 1, 40], "random"))
    rng = np.random.default_rng(1)
    x["mask"] = rng.integers(-2 ** 31, 2 ** 31, x["mask"].shape).astype(np.int32)
    x["mask"][2] = 0
    x["mask"][4] = -64                      # only bits past the request's 6 tokens
    x["mask"][36] = 0
    ref, size = _attn_ref(x)
    assert (ref[[2, 4, 36]] == 0).all()
    with _attn_ctx(pkv, x) as ctx:
        out = _attn_run(pkv, ctx, _attn_device(x))
        _ok(pkv, ctx)
        _attn_near(out, ref, size)
        assert (out[[2, 4, 36]] == 0).all()


def test_tree_attention_large_scores(pkv):
    """Scores far apart: the running maximum moves again and again, weights
    underflow, and the far ends of the type do not overflow."""
    x = _attn_inputs((8, 2, 64, 16, False, [1000, 3], [12, 40], "random"))
    for b in range(2):
        L = int(x["lens"][b])
        for pos in range(L):                # keys grow along the cache
            p = x["table"][b, pos // 16]
            x["k"][p, :, pos % 16] *= 1 + pos / 20
    x["kv"] = _tree.values(x["k"])
    ref, size = _attn_ref(x)
    s = 2.0 ** -23 * 64 * np.abs(x["kv"]).max() * 5 * 64 ** 0.5     # fp32 sums of these scores: their bound, in the weights
    with _attn_ctx(pkv, x) as ctx:
        got = _tree.values(_attn_run(pkv, ctx, _attn_device(x)))
        _ok(pkv, ctx)
    assert (np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + (W + s) * size).all()


@pytest.mark.parametrize("fp8", [False, True])
def test_tree_attention_ignores_what_is_masked(pkv, fp8):
    """NaN and infinity in the K and V of new tokens that a row does not see,
    in slots behind the request and in pages of nobody, leave it as it was; a
    row that sees them takes them."""
    x = _attn_inputs((8, 2, 128, 16, fp8, [120, 7], [20, 33], "star"))
    ref, size = _attn_ref(x)
    bad = float("nan") if fp8 else float("inf")
    used = np.zeros((x["pages"], 16), bool)
    for b, (L, T) in enumerate(zip([120, 7], [20, 33])):
        for pos in range(L + T):
            used[x["table"][b, pos // 16], pos % 16] = True
    for name in ("k", "v"):
        u = x[name].view(torch.uint8) if fp8 else x[name]
        for pg, at in zip(*np.nonzero(~used)):
            u[pg, :, at] = 0x7F if fp8 else float("nan")
        for b, j in ((0, 3), (0, 19), (1, 32)):
            pos = int(x["lens"][b]) + j
            u[x["table"][b, pos // 16], :, pos % 16] = 0x7F if fp8 else bad
    rows = {3, 19, 20 + 32}
    with _attn_ctx(pkv, x) as ctx:
        got = _tree.values(_attn_run(pkv, ctx, _attn_device(x)))
        _ok(pkv, ctx)
    for r in range(53):
        if r in rows:
            assert not np.isfinite(got[r]).any(), r
        else:
            assert (np.abs(got[r] - ref[r]) <= 2.0 ** -8 * np.abs(ref[r]) + W * size[r]).all(), r


@pytest.mark.parametrize("fp8", [False, True])
def test_tree_attention_leaves_other_rows(pkv, fp8):
    """Rows behind the last request stay as they were (a captured step has a
    fixed number of rows)."""
    x = _attn_inputs((8, 2, 64, 16, fp8, [50, 90], [5, 9], "random"))
    ref, size = _attn_ref(x)
    x["q"] = torch.cat([x["q"], torch.full((7, 8, 64), float("nan")).to(torch.bfloat16)])
    x["mask"] = np.concatenate([x["mask"], np.full((7, 1), -1, np.int32)])
    with _attn_ctx(pkv, x) as ctx:
        out = torch.full((21, 8, 64), 7.0, device=DEV, dtype=torch.bfloat16)
        _attn_run(pkv, ctx, _attn_device(x), out)
        _ok(pkv, ctx)
        assert (out[14:] == 7).all()
        _attn_near(out[:14], ref, size)


@pytest.mark.parametrize("fp8", [False, True])
def test_tree_attention_out_of_range(pkv, fp8):
    x = _attn_inputs((8, 2, 64, 16, fp8, [300, 90, 40], [5, 9, 3], "random"))
    ref, size = _attn_ref(x)
    g = _attn_device(x)
    with _attn_ctx(pkv, x) as ctx:
        # a length past the table, and a negative one: that request is zero
        for v in (1 << 20, -1, 2 ** 31 - 1):
            bad = dict(g, lens=_i([300, v, 40]))
            out = _attn_run(pkv, ctx, bad)
            assert _status(pkv, ctx) == (pkv.PKV_ERR_DEVICE_BOUNDS, 1)
            assert (out[5:14] == 0).all()
            _attn_near(out[:5], ref[:5], size[:5])
            _attn_near(out[14:], ref[14:], size[14:])
        # a page out of range: its keys are left out
        for page in (-1, x["pages"], 2 ** 31 - 1):
            bad = dict(g, table=g["table"].clone())
            bad["table"][0, 2] = page
            kept = dict(x, table=x["table"].copy(), lens=x["lens"].copy())
            kept["table"][0] = np.concatenate([np.delete(x["table"][0], 2), x["table"][0][2:3]])
            kept["lens"][0] -= 16
            r0, s0 = _attn_ref(kept)
            out = _attn_run(pkv, ctx, bad)
            assert _status(pkv, ctx) == (pkv.PKV_ERR_DEVICE_BOUNDS, 2)
            _attn_near(out, r0, s0)
        # rows of a request out of order: it is skipped
        out = _attn_run(pkv, ctx, dict(g, cu=_i([0, 5, 3, 17])), torch.full_like(g["q"], 7.0))
        assert _status(pkv, ctx)[0] == pkv.PKV_ERR_DEVICE_BOUNDS
        _attn_near(out[:3], ref[:3], size[:3])
        # more new tokens than the mask's words
        wide = _attn_inputs((8, 2, 64, 16, fp8, [30], [40], "random"))
        w = _attn_device(wide)
        w["mask"] = w["mask"][:, :1].contiguous()
    with _attn_ctx(pkv, wide) as ctx:
        assert (_attn_run(pkv, ctx, w) == 0).all()
        assert _status(pkv, ctx) == (pkv.PKV_ERR_DEVICE_BOUNDS, 1)


# ---- commit ----------------------------------------------------------------------

@pytest.mark.parametrize("Hq,Hkv,d,P,fp8,B,depth", [
    (8, 2, 64, 16, False, 4, 5), (8, 1, 128, 16, False, 9, 12), (24, 8, 128, 32, False, 30, 7),
    (8, 2, 64, 16, True, 4, 5), (64, 8, 128, 16, True, 40, 8), (9, 3, 64, 64, True, 5, 40), (6, 6, 128, 16, True, 3, 1),
    (24, 24, 64, 16, False, 3, 9),
])
@pytest.mark.parametrize("inplace", [False, True])
def test_tree_commit(pkv, Hq, Hkv, d, P, fp8, B, depth, inplace):
    rng = np.random.default_rng(B + depth)
    gen = torch.Generator().manual_seed(B)
    lens = rng.integers(0, 100, B)
    table, pages, _ = _tree.tables(rng, [-(-(int(a) + 3 * depth) // P) for a in lens])
    k, v, ks, vs, _, _ = _tree.pools(gen, pages, Hkv, P, d, fp8)
    path = (rng.integers(1, 4, (B, depth)).cumsum(1) - 1).astype(np.int32)
    n = rng.integers(0, depth + 1, B)
    n[0], path[0] = depth, np.arange(depth)            # a path that is in place already
    for b in range(B):
        path[b, n[b]:] = rng.integers(-9, 9999, depth - n[b])      # never read
    want = []
    for pool, scale in ((k, ks), (v, vs)):
        w = pool.clone().view(torch.uint8) if fp8 else pool.clone()
        for b in range(B):
            for j in range(n[b]):
                s, t = int(lens[b]) + int(path[b, j]), int(lens[b]) + j
                p0, p1 = table[b, s // P], table[b, t // P]
                row = pool[p0, :, s % P]
                if fp8:
                    same = (scale[p0] == scale[p1])[:, None]
                    y = (row.float() * scale[p0][:, None] / scale[p1][:, None]).clamp(-448, 448).to(_tree.E4M3)
                    row = torch.where(same, row.view(torch.uint8), y.view(torch.uint8))
                w[p1, :, t % P] = row
        want.append(w)
    dk, dv = k.to(DEV), v.to(DEV)
    sc = [None if s is None else s.to(DEV) for s in (ks, vs)]
    dl = _i(lens)
    out = dl if inplace else _i(np.full(B, 77))
    with _Ctx(pkv, Hq, Hkv, d, P, fp8, B, table.shape[1], pages) as ctx:
        pkv.pkv_tree_commit(ctx, dk, dv, *sc, _i(table), dl, _i(path), _i(n), out)
        _ok(pkv, ctx)
    assert np.array_equal(out.cpu().numpy(), lens + n)
    for got, w in zip((dk, dv), want):
        g = got.cpu().view(torch.uint8) if fp8 else got.cpu()
        assert torch.equal(g, w)


def test_tree_commit_out_of_range(pkv):
    rng = np.random.default_rng(2)
    gen = torch.Generator().manual_seed(2)
    lens = np.array([10, 30, 17])
    table, pages, _ = _tree.tables(rng, [3, 3, 3])
    k, v, _, _, _, _ = _tree.pools(gen, pages, 2, 16, 64, False)
    good = np.array([[1, 3, 4], [0, 2, 5], [2, 3, 9]], np.int32)
    with _Ctx(pkv, 4, 2, 64, 16, False, 3, 3, pages) as ctx:
        def call(bits, lens=lens, path=good, n=(3, 3, 3), table=table):
            dk, dv, out = k.to(DEV), v.to(DEV), _i([77] * 3)
            pkv.pkv_tree_commit(ctx, dk, dv, None, None, _i(table), _i(lens), _i(path), _i(n), out)
            assert _status(pkv, ctx)[1] == bits
            # request 1 is left alone, the others are served
            assert out.tolist() == [int(lens[0]) + 3, int(lens[1]), int(lens[2]) + 3]
            p = table[0, 0] if table[0, 0] >= 0 else 0
            assert torch.equal(dk[p, :, 10].cpu(), k[p, :, 11])
            for pool, orig in ((dk, k), (dv, v)):
                for q in (0, 1, 2):
                    pg = int(good_table[1, q])
                    assert torch.equal(pool[pg].cpu(), orig[pg])

        good_table = table
        call(1, lens=np.array([10, -1, 17]))
        call(1, lens=np.array([10, 45, 17]))
        call(1, n=(3, 4, 3))
        call(1, n=(3, -1, 3))
        for row in ([3, 3, 4], [-1, 2, 3], [2, 1, 4], [0, 5, -9]):
            call(8, path=np.array([good[0], row, good[2]]))
        call(1, path=np.array([good[0], [0, 1, 2 ** 31 - 1], good[2]]))
        bad = table.copy()
        bad[1, 1] = pages
        call(2, table=bad)


# ---- the step as a whole -----------------------------------------------------------

class _Step:
    """A speculative step over one layer: plan, rotate and append, attend under
    the tree mask, commit; its buffers as a serving program keeps them."""

    def __init__(self, pkv, fp8, B=5, cap=64, seed=0):
        self.pkv, self.B, self.P, self.cap, self.shape = pkv, B, 16, cap, (8, 2, 64)
        self.pages = 80
        self.fp8 = fp8
        gen = torch.Generator().manual_seed(seed)
        self.k, self.v, self.ks, self.vs, _, _ = _tree.pools(gen, self.pages, 2, 16, 64, fp8)
        self.gen = gen
        self.rng = np.random.default_rng(seed)
        self.lens = self.rng.integers(0, 40, B).astype(np.int32)
        held = -(-self.lens // 16)
        t, _, _ = _tree.tables(self.rng, held.tolist(), self.pages - int(held.sum()))
        used = t[t >= 0]
        self.table = np.full((B, 12), -1, np.int32)
        self.table[:, :t.shape[1]] = t
        self.held = held.astype(np.int32)
        self.free = self.rng.permutation(np.setdiff1d(np.arange(self.pages), used)).astype(np.int32)
        self.d = dict(k=self.k.to(DEV), v=self.v.to(DEV), lens=_i(self.lens), table=_i(self.table),
                      held=_i(self.held), free=_i(self.free), count=_i([len(self.free)]), new=_i(np.zeros(B)),
                      parents=_i(np.full(cap, -1)), cu=_i(np.zeros(B + 1)), slots=_i(np.zeros(cap)),
                      pos=_i(np.zeros((1, cap))), mask=_i(np.zeros((cap, 1))), path=_i(np.zeros((B, 6))),
                      path_lens=_i(np.zeros(B)), q=torch.zeros(cap, 8, 64, dtype=torch.bfloat16, device=DEV),
                      kn=torch.zeros(cap, 2, 64, dtype=torch.bfloat16, device=DEV),
                      vn=torch.zeros(cap, 2, 64, dtype=torch.bfloat16, device=DEV),
                      out=torch.zeros(cap, 8, 64, dtype=torch.bfloat16, device=DEV))
        self.sc = [None if s is None else s.to(DEV) for s in (self.ks, self.vs)]

    def inputs(self):
        new = self.rng.integers(0, 12, self.B)
        par = [_tree.parents_of(self.rng, int(n)) for n in new]
        path, plen = np.zeros((self.B, 6), np.int32), np.zeros(self.B, np.int32)
        for b in range(self.B):
            x, chain = int(new[b]) - 1, []
            while x >= 0:
                chain.append(x)
                x = par[b][x]
            chain = chain[::-1][:6]
            plen[b] = len(chain)
            path[b, :len(chain)] = chain
        n = int(new.sum())
        h = dict(new=new, par=par, path=path, plen=plen, n=n)
        for name, heads in (("q", 8), ("kn", 2), ("vn", 2)):
            h[name] = torch.randn(n, heads, 64, generator=self.gen).to(torch.bfloat16)
        return h

    def upload(self, h):
        d, n = self.d, h["n"]
        d["new"].copy_(_i(h["new"]))
        d["parents"].fill_(-1)
        d["parents"][:n] = _i(sum(h["par"], []))
        d["path"].copy_(_i(h["path"]))
        d["path_lens"].copy_(_i(h["plen"]))
        for name in ("q", "kn", "vn"):
            d[name][:n] = h[name].to(DEV)
        d["out"].fill_(7)

    def run(self, ctx):
        d, p = self.d, self.pkv
        p.pkv_slot_map(ctx, d["lens"], d["new"], d["table"], d["held"], d["free"], d["count"], d["cu"], d["slots"],
                       d["pos"].view(-1), d["held"], d["count"], parents=d["parents"], tree_mask=d["mask"])
        p.pkv_rope_append_axes(ctx, d["q"], d["kn"], d["vn"], d["pos"], [32], d["slots"], d["q"], d["k"], d["v"],
                               *self.sc)
        p.pkv_decode_attn_tree(ctx, d["q"], d["k"], d["v"], *self.sc, d["table"], d["lens"], d["cu"], d["mask"],
                               d["out"])
        p.pkv_tree_commit(ctx, d["k"], d["v"], *self.sc, d["table"], d["lens"], d["path"], d["path_lens"], d["lens"])

    def check(self, h):
        """One step on the host from what the step before left on the device."""
        n, B = h["n"], self.B
        r = _tree.slot_map(self.lens, h["new"], self.table, self.held, self.free, self.count0, 16, self.cap,
                           np.array(sum(h["par"], []), np.int32), 1)
        d = self.d
        assert np.array_equal(d["table"].cpu().numpy(), r["table"]) and np.array_equal(d["slots"].cpu().numpy(), r["slots"])
        assert np.array_equal(d["held"].cpu().numpy(), r["pages"]) and int(d["count"][0]) == r["left"]
        assert np.array_equal(d["lens"].cpu().numpy(), self.lens + h["plen"])
        q = _tree.rotate(_tree.values(h["q"]), r["pos"][None, :n], [32], False, 1e4)
        got_q = _tree.values(d["q"][:n])
        assert (np.abs(got_q - q) <= 2.0 ** -8 * np.abs(q) + 2.0 ** -16).all()
        # the cache as it stood for the attention: before the step, and the appended tokens
        kv, vv = self.before[0].double().numpy().copy(), self.before[1].double().numpy().copy()
        kn = _tree.rotate(_tree.values(h["kn"]), r["pos"][None, :n], [32], False, 1e4)
        vn = _tree.values(h["vn"])
        if self.fp8:
            kv, vv = kv * self.ks.double().numpy()[:, :, None, None], vv * self.vs.double().numpy()[:, :, None, None]
        page, at = r["slots"][:n] // 16, r["slots"][:n] % 16
        stored = []
        for x, cache, s in ((kn, kv, self.ks), (vn, vv, self.vs)):
            y = torch.from_numpy(x).float()
            if self.fp8:
                y = (y / s[page][..., None]).clamp(-448, 448).to(_tree.E4M3).double() * s[page][..., None].double()
            else:
                y = y.to(torch.bfloat16).double()
            stored.append(y.numpy())
            cache[page, :, at] = y.numpy()
        ref, size = _tree.attention(got_q, kv, vv, self.lens, r["cu"], r["table"], r["mask"], 16, 4)
        out = _tree.values(d["out"])
        assert (out[n:] == 7).all()
        # a K or V code next to a border may have been rounded the other way:
        # one step of the type in the new tokens' entries (their share of the weights is below 1)
        step = 2.0 ** -3 if self.fp8 else 2.0 ** -7
        assert (np.abs(out[:n] - ref) <= 2.0 ** -8 * np.abs(ref) + W * size + step * 0.5 * size).all()
        # the accepted tokens, where the next step reads them
        lens = self.lens + h["plen"]
        gk = _tree.values(d["k"])
        if self.fp8:
            gk = gk * self.ks.double().numpy()[:, :, None, None]
        for b in range(B):
            for j in range(int(h["plen"][b])):
                pos = int(self.lens[b]) + j
                got = gk[r["table"][b, pos // 16], :, pos % 16]
                want = stored[0][int(r["cu"][b]) + int(h["path"][b, j])]
                if self.fp8:        # stored again under this page's scale: saturates at its range
                    top = 448 * self.ks.double().numpy()[r["table"][b, pos // 16]][:, None]
                    want = np.clip(want, -top, top)
                assert (np.abs(got - want) <= (0.2 if self.fp8 else 2.0 ** -7) * np.abs(want) + (0.05 if self.fp8 else 2.0 ** -16)).all()
        self.lens, self.table, self.held = lens.astype(np.int32), r["table"], r["pages"]

    def snapshot(self):
        torch.cuda.synchronize()
        self.before = (self.d["k"].cpu(), self.d["v"].cpu())
        self.count0 = int(self.d["count"][0])


@pytest.mark.parametrize("fp8", [False, True])
def test_speculative_steps(pkv, fp8):
    s = _Step(pkv, fp8)
    with _Ctx(pkv, 8, 2, 64, 16, fp8, s.B, 12, s.pages) as ctx:
        for _ in range(4):
            h = s.inputs()
            s.upload(h)
            s.snapshot()
            s.run(ctx)
            _ok(pkv, ctx)
            s.check(h)


@pytest.mark.parametrize("fp8", [False, True])
def test_speculative_steps_captured(pkv, fp8):
    """One captured graph of the step, replayed over changing lengths, trees
    and tables, between eager steps on the same context."""
    s = _Step(pkv, fp8, seed=4)
    with _Ctx(pkv, 8, 2, 64, 16, fp8, s.B, 12, s.pages) as ctx:
        h = s.inputs()
        s.upload(h)
        s.snapshot()
        s.run(ctx)
        _ok(pkv, ctx)
        s.check(h)
        keep = {k: s.d[k].clone() for k in ("k", "v", "lens", "table", "held", "count", "q")}
        side = torch.cuda.Stream()
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=side):
            s.run(ctx)
        for name, t in keep.items():
            s.d[name].copy_(t)
        for i in range(4):
            h = s.inputs()
            s.upload(h)
            s.snapshot()
            if i == 2:
                s.run(ctx)
            else:
                graph.replay()
            torch.cuda.synchronize()
            _ok(pkv, ctx)
            s.check(h)


def test_tree_chain_is_the_varlen_attention(pkv):
    """A chain of drafted tokens is the varlen call's causal mask."""
    x = _attn_inputs((8, 2, 64, 16, False, [33, 200, 0], [4, 16, 9], "chain"))
    g = _attn_device(x)
    with _attn_ctx(pkv, x, batch=16) as ctx:
        out = _attn_run(pkv, ctx, g)
        other = torch.empty_like(out)
        pkv.pkv_decode_attn_varlen(ctx, g["q"], g["k"], g["v"], None, None, g["table"], g["lens"], g["cu"], other)
        _ok(pkv, ctx)
        ref, size = _attn_ref(x)
        assert (np.abs(_tree.values(out) - _tree.values(other)) <= 2 * (2.0 ** -8 * np.abs(ref) + 2.0 ** -8 * size)).all()


def test_wrong_device_or_stream(pkv):
    """The calls run on the stream they are given: work queued before on it is seen."""
    x = _attn_inputs((8, 2, 64, 16, False, [300, 90], [5, 9], "random"))
    ref, size = _attn_ref(x)
    g = _attn_device(x)
    with _attn_ctx(pkv, x) as ctx:
        side = torch.cuda.Stream()
        late = torch.zeros_like(g["q"])
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            big = torch.randn(4096, 4096, device=DEV)
            for _ in range(10):
                big = big @ big * 1e-4
            late.copy_(g["q"])
            out = _attn_run(pkv, ctx, dict(g, q=late))
        side.synchronize()
        _ok(pkv, ctx)
        _attn_near(out, ref, size)


@pytest.mark.parametrize("fp8", [False, True])
def test_tree_attention_bad_page_next_to_nan(pkv, fp8):
    """A page out of range is left out whatever the pool holds elsewhere."""
    x = _attn_inputs((8, 2, 128, 16, fp8, [300], [5], "random"))
    unused = int(np.setdiff1d(np.arange(x["pages"]), x["table"][0])[0])
    for name in ("k", "v"):
        u = x[name].view(torch.uint8) if fp8 else x[name]
        swap = u[0].clone()                       # page 0 becomes nobody's, and no number
        u[unused] = swap
        u[0] = 0x7F if fp8 else float("nan")
        if fp8:
            x[name + "s"][unused] = x[name + "s"][0]
        x[name + "v"][unused] = x[name + "v"][0]
    x["table"][x["table"] == 0] = unused
    kept = dict(x, table=np.concatenate([np.delete(x["table"][0], 3), x["table"][0][3:4]])[None], lens=x["lens"] - 16)
    ref, size = _attn_ref(kept)
    x["table"][0, 3] = -7
    with _attn_ctx(pkv, x) as ctx:
        out = _attn_run(pkv, ctx, _attn_device(x))
        assert _status(pkv, ctx) == (pkv.PKV_ERR_DEVICE_BOUNDS, 2)
        _attn_near(out, ref, size)


def test_lengths_at_the_end_of_32_bits(pkv):
    """Lengths whose sum with the new tokens passes 32 bits are out of range,
    also under a table long enough for them."""
    blocks = (1 << 25) - 1                                  # x 64 tokens: 2^31 - 64, the longest table a context takes
    i = lambda *v: _i(np.array(v))   # noqa: E731
    table = torch.zeros(1, blocks, dtype=torch.int32, device=DEV)
    with _Ctx(pkv, 4, 1, 64, 64, False, 1, blocks, 4) as ctx:
        pool = torch.zeros(4, 1, 64, 64, dtype=torch.bfloat16, device=DEV)
        q = torch.ones(8, 4, 64, dtype=torch.bfloat16, device=DEV)
        for L in (64 * blocks - 3, 2 ** 31 - 4, 2 ** 31 - 1):
            out = torch.full_like(q, 7.0)
            pkv.pkv_decode_attn_tree(ctx, q, pool, pool, None, None, table, i(L), i(0, 8),
                                     torch.ones(8, 1, dtype=torch.int32, device=DEV), out)
            assert _status(pkv, ctx) == (pkv.PKV_ERR_DEVICE_BOUNDS, 1) and (out == 0).all()
            slots, pos, pages, left, cu = i(*[5] * 8), i(*[5] * 8), i(5), i(5), i(5, 5)
            pkv.pkv_slot_map(ctx, i(L), i(8), table, i(blocks), i(1, 2), i(2), cu, slots, pos, pages, left)
            assert _status(pkv, ctx) == (pkv.PKV_ERR_DEVICE_BOUNDS, 1)
            assert (slots == -1).all() and int(pages[0]) == blocks and int(left[0]) == 2 and cu.tolist() == [0, 8]
            lens = i(5)
            pkv.pkv_tree_commit(ctx, pool, pool, None, None, table, i(L), i(1, 2, 3)[None], i(3), lens)
            assert _status(pkv, ctx) == (pkv.PKV_ERR_DEVICE_BOUNDS, 1) and int(lens[0]) == L


def test_offsets_past_32_bits(pkv):
    """Pages at the far end of pools of more than 2^32 bytes and 2^31 elements:
    the same bits as from pools that hold those pages alone."""
    x = _attn_inputs((16, 8, 128, 64, False, [200, 70], [9, 20], "random"))
    pages, n = 34000, x["pages"]                            # x 64 K elements
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("18 GB of pools")
    far = dict(x, table=np.where(x["table"] >= 0, x["table"] + pages - n, -1).astype(np.int32))
    g, f = _attn_device(x), None
    with _attn_ctx(pkv, x) as ctx:
        near = _attn_run(pkv, ctx, g)
    small = {k: g[k].clone() for k in ("k", "v")}
    big = {k: torch.zeros(pages, *x[k].shape[1:], dtype=torch.bfloat16, device=DEV) for k in ("k", "v")}
    for k in big:
        big[k][pages - n:] = small[k]
    f = dict(_attn_device(dict(far, k=x["k"][:1], v=x["v"][:1])), **big)
    Hq, Hkv, d, P = x["case"][:4]
    kn = torch.randn(4, Hkv, d, device=DEV).to(torch.bfloat16)
    qn = torch.randn(4, Hq, d, device=DEV).to(torch.bfloat16)
    slots, pos = np.array([3, 64 * n - 1, 130, 400]), _i([[9, 70000, 3, 5]])
    path, plen = _i([[1, 4, 8], [3, 5, 19]]), _i([3, 2])
    got = {}
    for name, pool, table, count, shift in (("near", small, x["table"], n, 0), ("far", big, far["table"], pages, pages - n)):
        with _Ctx(pkv, Hq, Hkv, d, P, False, 2, x["table"].shape[1], count) as ctx:
            if name == "far":
                out = torch.empty_like(f["q"])
                pkv.pkv_decode_attn_tree(ctx, f["q"], pool["k"], pool["v"], None, None, f["table"], f["lens"], f["cu"],
                                         f["mask"], out)
                assert torch.equal(out, near)
            qo, lens = torch.empty_like(qn), _i([0, 0])
            pkv.pkv_rope_append_axes(ctx, qn, kn, kn, pos, [64], _i(slots + 64 * shift), qo, pool["k"], pool["v"], None, None)
            pkv.pkv_tree_commit(ctx, pool["k"], pool["v"], None, None, _i(table), f["lens"], path, plen, lens)
            _ok(pkv, ctx)
            got[name] = (qo, pool["k"][count - n:].clone(), pool["v"][count - n:].clone(), lens)
    for a, b in zip(*got.values()):
        assert torch.equal(a, b)
    assert not big["k"][:pages - n].any() and not big["v"][:pages - n].any()


def test_two_contexts_on_two_streams(pkv):
    """Steps of two contexts in flight together do not touch one another."""
    runs = []
    for seed, case in ((0, (8, 2, 64, 16, False, [3000, 90], [12, 40], "random")),
                       (1, (16, 2, 128, 32, True, [2500, 7], [30, 9], "random"))):
        x = _attn_inputs(case, seed)
        runs.append((x, _attn_device(x), _attn_ref(x), _attn_ctx(pkv, x), torch.cuda.Stream()))
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(20):
        for o, (x, g, ref, ctx, stream) in zip(outs, runs):
            with torch.cuda.stream(stream):
                o.append(_attn_run(pkv, ctx.h, g))
    torch.cuda.synchronize()
    for o, (x, g, ref, ctx, stream) in zip(outs, runs):
        with ctx as h:
            _ok(pkv, h)
            _attn_near(o[0], *ref)
            assert all(torch.equal(o[0], y) for y in o[1:])


def test_marshal_pointers(pkv):
    """The extension module takes what the checks in Python take, no more."""
    m = pytest.importorskip("paged_kv_flight_b200._marshal")
    kinds = {0: torch.int32, 1: torch.bfloat16, 2: torch.float8_e4m3fn, 3: torch.float32}
    for k, dt in kinds.items():
        x = torch.zeros(4, 6, device=DEV).to(dt)
        assert m.pointer(x, k, 4, 6) == m.pointer(x, k) == m.pointer(x, k, -1, 6) == x.data_ptr()
        for bad in (m.pointer(x, k, 6, 4), m.pointer(x, k, 24), m.pointer(x, k, 4, 6, 1), m.pointer(x.t(), k, 6, 4),
                    m.pointer(x[:, ::2], k, 4, 3), m.pointer(x.cpu(), k, 4, 6), m.pointer(x.half(), k, 4, 6)):
            assert bad is None
        assert m.pointer(x[2], k, 6) == x.data_ptr() + 12 * x.element_size()
    assert m.pointer(torch.zeros(2, device=DEV, dtype=torch.uint8), 2) and m.pointer(torch.zeros(2, device=DEV), 2) is None


@pytest.mark.parametrize("case", ATTN_CASES, ids=lambda c: f"h{c[0]}_{c[1]}_d{c[2]}_p{c[3]}_{'f8' if c[4] else 'bf'}_{c[5][0]}")
def test_tree_attention_keeps_the_bits_of_its_weights(pkv, case):
    """The weights go into the product with V as two bf16 terms: the first off
    by less than 2^-7 (cut, not rounded), the second rounded to 2^-8 of that,
    2^-15 in all; with 2^-13.6 of the fp32 scores and 2^-21 of the rest (above)
    less than 2^-12 of A."""
    x = _attn_inputs(case, seed=1)
    ref, size = _attn_ref(x)
    with _attn_ctx(pkv, x) as ctx:
        got = _tree.values(_attn_run(pkv, ctx, _attn_device(x)))
        _ok(pkv, ctx)
    err = np.abs(got - ref) - (2.0 ** -8 * np.abs(ref) + 2.0 ** -12 * size)
    assert (err <= 0).all(), (float(err.max()), int((err > 0).sum()))


@pytest.mark.parametrize("fp8", [False, True])
def test_tree_attention_of_one_key_is_its_v(pkv, fp8):
    """A row that sees one key has that key's V: bit for bit in bf16 (2^-15 of
    the weight is far below half a step of V), and off by one rounding of code *
    scale from an E4M3 cache."""
    x = _attn_inputs((8, 2, 128, 16, fp8, [0, 0, 0], [20, 140, 1], "star"))
    with _attn_ctx(pkv, x) as ctx:
        out = _attn_run(pkv, ctx, _attn_device(x))
        _ok(pkv, ctx)
    got = _tree.values(out)
    for b in range(3):
        for i in range(int(x["cu"][b + 1] - x["cu"][b])):
            want = np.repeat(x["vv"][x["table"][b, i // 16], :, i % 16], 4, axis=0)
            err = np.abs(got[x["cu"][b] + i] - want)
            assert (err <= (2.0 ** -8 + 2.0 ** -14 if fp8 else 0.0) * np.abs(want)).all(), (b, i, float(err.max()))


@pytest.mark.parametrize("cap", [0, 1, 10, 60, 200])
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("inplace", [False, True])
def test_slot_map_more_tokens_than_rows(pkv, cap, tree, inplace):
    """Tokens that have no row are dropped, and nothing else: the table, the
    pages held and the stack agree with one another, as if they had rows."""
    rng = np.random.default_rng(17)
    x = _slot_inputs(rng, 12, 16, 0, 60, 0, 70, tree)
    assert x["new"].sum() > 250
    r = _tree.slot_map(x["lens"], x["new"], x["table"], x["held"], x["free"], x["count"], 16, cap, x["parents"], 3)
    with _Ctx(pkv, 8, 2, 64, 16, False, 12, x["table"].shape[1], x["pages"]) as ctx:
        _slot_check(_slot_call(pkv, ctx, x, cap, 3, inplace), r)
        assert _status(pkv, ctx) == (pkv.PKV_ERR_DEVICE_BOUNDS, 1)


@pytest.mark.parametrize("n", [1 << 20, 2 ** 31 - 1])
@pytest.mark.parametrize("b", [0, 5])
def test_slot_map_next_to_a_count_far_too_large(pkv, b, n):
    """One count out of range takes the rows behind it, but leaves the other
    requests' pages in a state to go on from."""
    rng = np.random.default_rng(23)
    x = _slot_inputs(rng, 9, 16, 0, 60, 1, 40, False)
    x["new"][b] = 0
    cap = int(x["new"].sum()) + 50
    r = _tree.slot_map(x["lens"], x["new"], x["table"], x["held"], x["free"], x["count"], 16, cap)
    start = int(r["cu"][b])
    x["new"][b] = n
    with _Ctx(pkv, 8, 2, 64, 16, False, 9, x["table"].shape[1], x["pages"]) as ctx:
        g = _slot_call(pkv, ctx, x, cap, 1)
        assert _status(pkv, ctx) == (pkv.PKV_ERR_DEVICE_BOUNDS, 1)
    for k in ("table", "pages"):
        assert np.array_equal(g[k].cpu().numpy(), r[k]), k
    assert int(g["left"][0]) == r["left"]
    assert g["cu"].tolist() == [int(v) for v in r["cu"][:b + 1]] + [cap] * (9 - b)
    assert g["slots"].tolist() == r["slots"][:start].tolist() + [-1] * (cap - start)


# a cache long enough that its only item is cut, and one that is not
NAN_CASES = [(8, 1, 64, 16, False, [9000], [3], "random"), (8, 1, 128, 32, True, [7000], [20], "random"),
             (8, 2, 128, 16, False, [60, 7], [20, 33], "random")]


@pytest.mark.parametrize("case", NAN_CASES, ids=lambda c: f"d{c[2]}_{'f8' if c[4] else 'bf'}_{c[5][0]}")
def test_tree_attention_of_a_query_that_is_no_number(pkv, case):
    """One NaN in a head's query makes that head's output NaN, wherever its
    item is cut, and no other."""
    x = _attn_inputs(case)
    ref, size = _attn_ref(x)
    x["q"][1, 3, 5] = float("nan")
    with _attn_ctx(pkv, x) as ctx:
        got = _tree.values(_attn_run(pkv, ctx, _attn_device(x)))
        _ok(pkv, ctx)
    assert np.isnan(got[1, 3]).all()
    got[1, 3], ref[1, 3] = 0, 0
    assert (np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + W * size).all()


@pytest.mark.parametrize("case", NAN_CASES, ids=lambda c: f"d{c[2]}_{'f8' if c[4] else 'bf'}_{c[5][0]}")
@pytest.mark.parametrize("which", ["one", "many", "far"])
def test_tree_attention_of_cached_keys_that_are_no_numbers(pkv, case, which):
    """A NaN key in the cache, a run of them longer than an item's part, and one
    whose part lies so far below the others that its weight is 0."""
    x = _attn_inputs(case)
    Hq, Hkv, d, P, fp8, lens = case[:6]
    u = x["k"].view(torch.uint8) if fp8 else x["k"]
    nan = 0x7F if fp8 else float("nan")
    L = lens[0]
    if which == "far":                   # later keys: 200 times as large, along the queries
        big = x["q"][:, 0].float().sign().sum(0).sign()
        big[big == 0] = 1
        for pos in range(L // 2, L):
            x["k"][x["table"][0, pos // P], 0, pos % P] = (big * (400 if fp8 else 200)).to(x["k"].dtype)
    for pos in range(L // 4, L // 4 + (1 if which == "one" else min(1000, L // 4))):
        u[x["table"][0, pos // P], 0, pos % P] = nan
    with _attn_ctx(pkv, x) as ctx:
        got = _tree.values(_attn_run(pkv, ctx, _attn_device(x)))
        _ok(pkv, ctx)
    n = int(x["cu"][1])
    assert np.isnan(got[:n, :Hq // Hkv]).all()
    if Hkv > 1:
        assert np.isfinite(got[:n, Hq // Hkv:]).all()
    assert np.isfinite(got[n:]).all()


@pytest.mark.parametrize("case", [(8, 2, 128, 16, True, [100, 0], [9, 33], "random"),
                                  (8, 1, 64, 16, True, [4000], [5], "random")], ids=["short", "cut"])
@pytest.mark.parametrize("tiny", [0.0, 1e-44])
def test_tree_attention_scales_of_zero(pkv, case, tiny):
    """K scales of 0 (or the smallest numbers): every key weighs the same.  V
    scales of 0: the output is 0, not something small."""
    x = _attn_inputs(case)
    for zero in ("k", "v"):
        y = dict(x, **{zero + "s": torch.full_like(x[zero + "s"], tiny), zero + "v": x[zero + "v"] * 0.0})
        ref, size = _attn_ref(y)
        with _attn_ctx(pkv, y) as ctx:
            out = _attn_run(pkv, ctx, _attn_device(y))
            _ok(pkv, ctx)
        if zero == "v":
            assert (out.abs() <= 448 * tiny).all(), float(out.abs().max())
        else:
            _attn_near(out, ref, size)


def test_slot_map_clears_the_entries_it_does_not_fill(pkv):
    """Entries that a request would have needed and did not get name no page
    afterwards, whatever an earlier use of the row left there: the attention
    leaves their keys out and the commit refuses a path through them."""
    rng = np.random.default_rng(31)
    gen = torch.Generator().manual_seed(31)
    P, stride, pages = 16, 8, 40
    lens, new = np.array([20, 20, 40, 5, 30]), np.array([30, 30, 70, 9, 120])   # 2: more than the mask's words; 4: past the table
    held = np.array([2, 2, 3, 1, 2])
    order = rng.permutation(pages).astype(np.int32)
    table = np.full((5, stride), -1, np.int32)
    for b, at in enumerate((0, 2, 4, 7, 8)):
        table[b, :held[b]] = order[at:at + held[b]]
    table[1, 2:] = table[0, 0]                       # stale: pages of others
    table[2, 3:] = table[0, 1]
    table[4, 2:] = table[3, 0]
    free = order[20:22]                              # enough for request 0 alone
    par = sum((_tree.parents_of(rng, int(n)) for n in new), [])
    n = int(new.sum())
    k, v, _, _, kv, vv = _tree.pools(gen, pages, 2, P, 64, False)
    dk, dv, dl, dt = k.to(DEV), v.to(DEV), _i(lens), _i(table)
    cu, slots, pos, mask = _i([0] * 6), _i([0] * n), _i([0] * n), _i([[0] * 2] * n)
    pages_out, left, out = _i([0] * 5), _i([0]), torch.zeros(n, 8, 64, dtype=torch.bfloat16, device=DEV)
    q = torch.randn(n, 8, 64, generator=gen).to(torch.bfloat16)
    with _Ctx(pkv, 8, 2, 64, P, False, 5, stride, pages) as ctx:
        pkv.pkv_slot_map(ctx, dl, _i(new), dt, _i(held), _i(free), _i([2]), cu, slots, pos, pages_out, left,
                         parents=_i(par), tree_mask=mask)
        assert _status(pkv, ctx) == (pkv.PKV_ERR_DEVICE_BOUNDS, 1 | 16)
        want = table.copy()
        want[0, 2:4] = free[::-1]
        want[1, 2:4] = -1
        want[2, 3:7] = -1
        want[4, 2:8] = -1
        assert np.array_equal(dt.cpu().numpy(), want)
        assert pages_out.tolist() == [4, 2, 3, 1, 2] and int(left[0]) == 0
        s = slots.cpu().numpy()
        assert (s[:30] >= 0).all() and (s[30:130] == -1).all() and (s[130:139] >= 0).all() and (s[139:] == -1).all()
        # the attention: request 1 sees what its held pages hold
        pkv.pkv_decode_attn_tree(ctx, q.to(DEV), dk, dv, None, None, dt, dl, cu, mask, out)
        assert _status(pkv, ctx) == (pkv.PKV_ERR_DEVICE_BOUNDS, 1 | 2)
        m = mask.cpu().numpy().copy()
        m[30:60, 0] &= (1 << 12) - 1                 # keys 20 .. 31 of it
        m[30:60, 1] = 0
        clip = want.copy()
        clip[1, 2:4] = 0
        ref, size = _tree.attention(_tree.values(q)[:60], kv, vv, lens[:2], np.array([0, 30, 60]), clip[:2], m[:60], P, 4)
        _attn_near(out[:60], ref, size)
        # the commit: a path into the missing pages is refused, and moves nothing
        path, plen = _i([[1, 3, 6], [1, 3, 14], [1, 2, 60], [0, 1, 2], [0, 2, 90]]), _i([3] * 5)
        lens_out = _i([0] * 5)
        pkv.pkv_tree_commit(ctx, dk, dv, None, None, dt, dl, path, plen, lens_out)
        assert _status(pkv, ctx) == (pkv.PKV_ERR_DEVICE_BOUNDS, 2)
        assert lens_out.tolist() == [23, 20, 40, 8, 30]
        same = np.setdiff1d(np.arange(pages), want[0, :4])
        assert torch.equal(dk.cpu()[same], k[same]) and torch.equal(dv.cpu()[same], v[same])


@pytest.mark.parametrize("Hq,Hkv,d,P,fp8", [(8, 2, 64, 16, False), (32, 8, 128, 32, False), (8, 2, 64, 16, True),
                                            (16, 4, 128, 64, True)])
def test_rope_append_axes_stores_what_the_other_appends_store(pkv, Hq, Hkv, d, P, fp8):
    """One axis: the bits of pkv_rope_append_varlen, so that a cache filled by
    both calls is the one that either would have made; and several axes of one
    position are one axis.  Zeros, infinities, NaN and the ends of the type too."""
    rng = np.random.default_rng(d + Hq)
    gen = torch.Generator().manual_seed(d)
    B = 40
    lens, new = rng.integers(0, 60000, B), rng.integers(1, 60, B)
    stride = 60100 // P + 1
    table, page = np.zeros((B, stride), np.int32), 0
    slots, pos = [], []
    for b in range(B):
        for k in range(int(lens[b]) // P, (int(lens[b]) + int(new[b]) - 1) // P + 1):
            table[b, k] = page
            page += 1
        at = np.arange(lens[b], lens[b] + new[b])
        slots += (table[b, at // P] * P + at % P).tolist()
        pos += at.tolist()
    n = len(pos)
    k, v, ks, vs, _, _ = _tree.pools(gen, page, Hkv, P, d, fp8)
    q, kn, vn = (torch.randn(n, h, d, generator=gen).to(torch.bfloat16) for h in (Hq, Hkv, Hkv))
    for t in (q, kn):
        for i, x in enumerate((0.0, -0.0, float("inf"), float("nan"), 1e-39, -3e38, 3.39e38)):
            t[3 * i] = x
            t[3 * i + 1, :, ::3] = x
            t[3 * i + 2, :, d // 2:] = x
    if fp8:                              # scales at the ends of their type
        for s in (ks, vs):
            s[1], s[2], s[3] = 0.0, 1e-42, 3e38
    cu = np.concatenate([[0], np.cumsum(new)])

    def dev():
        return [t.to(DEV, copy=True) for t in (q, kn, vn, k, v)] + [None if s is None else s.to(DEV) for s in (ks, vs)]

    with _Ctx(pkv, Hq, Hkv, d, P, fp8, 64, stride, page, base=5e5) as ctx:
        a = dev()
        pkv.pkv_rope_append_varlen(ctx, *a, _i(table), _i(lens), _i(cu))
        b = dev()
        pkv.pkv_rope_append_axes(ctx, b[0], b[1], b[2], _i(pos)[None], [d // 2], _i(slots), b[0], *b[3:])
        c = dev()
        out = torch.zeros_like(c[0])
        pkv.pkv_rope_append_axes(ctx, c[0], c[1], c[2], _i([pos] * 3), [d // 2 - 20, 10, 10], _i(slots), out, *c[3:],
                                 interleaved=True)
        c[0] = out
        _ok(pkv, ctx)
    for i, name in ((0, "q"), (3, "k"), (4, "v")):
        want = a[i].view(torch.uint8)
        for got in (b[i], c[i]):
            diff = int((got.view(torch.uint8) != want).sum())
            assert diff == 0, (name, diff, want.numel())


def test_marshal_pointers_of_one_device(pkv):
    m = pytest.importorskip("paged_kv_flight_b200._marshal")
    x = torch.zeros(4, 6, dtype=torch.int32, device=DEV)
    at = x.get_device()
    assert m.pointer(x, 4 * at + 4, 4, 6) == m.pointer(x, 0, 4, 6) == x.data_ptr()
    assert m.pointer(x, 4 * at + 8, 4, 6) is None and m.pointer(x, 4 * at + 5, 4, 6) is None


@pytest.mark.parametrize("Hq,Hkv,d", [(8, 8, 64), (8, 2, 64), (32, 8, 128), (64, 8, 128)])
def test_workspace_is_shared_between_the_calls(pkv, Hq, Hkv, d):
    """The tree attention's parts lie where the other attentions keep theirs: a
    context holds what the largest of them needs, and calls of every kind in turn
    on one stream give what each gives alone."""
    lens = [3000, 90, 1500, 7]
    n = 16 // (Hq // Hkv) // 2
    x = _attn_inputs((Hq, Hkv, d, 16, False, lens, [n] * 4, "chain"))
    g = _attn_device(x)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    q4 = g["q"].view(4, n, Hq, d)
    with _attn_ctx(pkv, x, batch=64) as ctx:
        # rows: 2 parts of 9 units of 8 warps of G rows, or of 256 of the tree attention, an SM
        rows = sms * max(2 * 9 * 8 * (Hq // Hkv), 2 * 256)
        assert pkv.pkv_workspace_bytes(ctx) <= rows * (d + 2) * 4 + (1 << 18)

        def calls():
            o = [torch.empty_like(g["q"]) for _ in range(3)] + [torch.empty_like(q4[:, 0])]
            pkv.pkv_decode_attn_tree(ctx, g["q"], g["k"], g["v"], None, None, g["table"], g["lens"], g["cu"], g["mask"], o[0])
            pkv.pkv_decode_attn_tokens(ctx, q4, g["k"], g["v"], None, None, g["table"], g["lens"], o[1].view(q4.shape))
            pkv.pkv_decode_attn_varlen(ctx, g["q"], g["k"], g["v"], None, None, g["table"], g["lens"], g["cu"], o[2])
            pkv.pkv_decode_attn(ctx, q4[:, 0].contiguous(), g["k"], g["v"], None, None, g["table"], g["lens"], o[3])
            return o

        alone = calls()
        torch.cuda.synchronize()
        rounds = [calls() for _ in range(30)]
        torch.cuda.synchronize()
        _ok(pkv, ctx)
        _attn_near(alone[0], *_attn_ref(x))
        for o in rounds:
            assert all(torch.equal(a, b) for a, b in zip(o, alone))


@pytest.mark.parametrize("B,hi,t_hi,tree", [(1500, 40, 3, True), (8192, 40, 3, False), (900, 30, 60, True)])
@pytest.mark.parametrize("inplace", [False, True])
def test_slot_map_large(pkv, B, hi, t_hi, tree, inplace):
    """More requests than threads, more rows than the cluster takes at once."""
    rng = np.random.default_rng(B)
    x = _slot_inputs(rng, B, 16, 0, hi, 0, t_hi, tree)
    cap, words = int(x["new"].sum()) + 7, 2
    r = _tree.slot_map(x["lens"], x["new"], x["table"], x["held"], x["free"], x["count"], 16, cap, x["parents"], words)
    with _Ctx(pkv, 8, 2, 64, 16, False, B, x["table"].shape[1], x["pages"]) as ctx:
        _slot_check(_slot_call(pkv, ctx, x, cap, words, inplace), r)
        _ok(pkv, ctx)


def test_slot_map_one_large_tree(pkv):
    """Ancestors further back than the rows that a CTA holds."""
    rng = np.random.default_rng(4)
    n, L, P = 3000, 21, 32
    par = _tree.parents_of(rng, n)
    par[2900:] = [i % 50 for i in range(100)]
    seen = _tree.ancestors(par)
    table, pages, _ = _tree.tables(rng, [-(-(L + n) // P)])
    x = dict(lens=np.array([L]), new=np.array([n]), held=np.array([table.shape[1]]), table=table, free=np.array([0]),
             count=0, parents=np.array(par, np.int32))
    words = -(-n // 32)
    r = _tree.slot_map(x["lens"], x["new"], table, x["held"], x["free"], 0, P, n)
    r["pos"], r["mask"] = (L + seen.sum(1) - 1).astype(np.int32), _tree.pack(seen, words)
    with _Ctx(pkv, 8, 2, 64, P, False, 1, table.shape[1], pages) as ctx:
        _slot_check(_slot_call(pkv, ctx, x, n, words), r)
        _ok(pkv, ctx)


@pytest.mark.parametrize("fp8", [False, True])
def test_tree_attention_more_requests_than_threads(pkv, fp8):
    rng = np.random.default_rng(12)
    lens = [int(v) for v in rng.integers(0, 40, 600)]
    new = [int(v) for v in rng.integers(0, 4, 600)]
    x = _attn_inputs((4, 2, 64, 16, fp8, lens, new, "random"))
    ref, size = _attn_ref(x)
    with _attn_ctx(pkv, x) as ctx:
        out = _attn_run(pkv, ctx, _attn_device(x))
        _ok(pkv, ctx)
        _attn_near(out, ref, size)


@pytest.mark.parametrize("Hkv,depth,fp8", [(2, 300, False), (2, 300, True), (72, 9, False), (72, 9, True), (40, 4, True)])
def test_tree_commit_large(pkv, Hkv, depth, fp8):
    """Paths longer than the places kept in shared memory, more kv heads than a
    cluster takes at once."""
    test_tree_commit(pkv, Hkv, Hkv, 64, 16, fp8, 3, depth, True)


def test_calls_on_another_device_than_the_contexts(pkv):
    """A context of another GPU is refused before anything is launched (made up:
    the checks read its configuration, then its device)."""
    import ctypes as C
    blob = C.create_string_buffer(b"\x07" * (1 << 16), 1 << 16)
    cfg = pkv.make_config(8, 2, 64, 16, "bf16", 1e4, 8, 8, 20)
    C.memmove(blob, C.byref(cfg), C.sizeof(cfg))
    ctx = C.addressof(blob)
    i = lambda *s: torch.zeros(*s, dtype=torch.int32, device=DEV)   # noqa: E731
    h = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device=DEV)   # noqa: E731
    pool = h(20, 2, 16, 64)
    calls = [lambda: pkv.pkv_slot_map(ctx, i(2), i(2), i(2, 8), i(2), i(9), i(1), i(3), i(5), i(5), i(2), i(1), check=False),
             lambda: pkv.pkv_rope_append_axes(ctx, h(2, 8, 64), h(2, 2, 64), h(2, 2, 64), i(1, 2), [32], i(2), h(2, 8, 64),
                                              pool, pool.clone(), None, None, check=False),
             lambda: pkv.pkv_decode_attn_tree(ctx, h(5, 8, 64), pool, pool, None, None, i(2, 8), i(2), i(3), i(5, 1),
                                              h(5, 8, 64), check=False),
             lambda: pkv.pkv_tree_commit(ctx, pool, pool, None, None, i(2, 8), i(2), i(2, 3), i(2), i(2), check=False)]
    for call in calls:
        assert call() == pkv.PKV_ERR_INVALID_ARG
    torch.cuda.synchronize()


def test_marshal_of_tensors_without_storage(pkv):
    """A tensor that has no address (inside a transform of torch.func) raises; it
    used to end the process."""
    m = pytest.importorskip("paged_kv_flight_b200._marshal")
    seen = []

    def inside(x):
        assert type(x) is torch.Tensor
        seen.append(m.pointer(x, 0))
        with pytest.raises(RuntimeError):
            pkv.pkv_tree_commit(None, 0, 0, None, None, x, 0, torch.zeros(4, 2, dtype=torch.int32, device=DEV), 0, 0)
        return x

    torch.func.vmap(inside)(torch.zeros(3, 4, 5, dtype=torch.int32, device=DEV))
    assert seen == [None]


@pytest.mark.parametrize("zero_q", [False, True])
@pytest.mark.parametrize("L", [200, 6000])
def test_tree_attention_infinite_cached_values(pkv, zero_q, L):
    """An infinity in V of a cached key is an infinity of its sign in that column
    of every row, also where weights are exact in bf16 (q = 0: all of them 1), and
    nothing anywhere else."""
    x = _attn_inputs((8, 2, 128, 16, False, [L, 9], [5, 3], "random"))
    if zero_q:
        x["q"].zero_()
    ref, size = _attn_ref(x)
    for pos, col, v in ((30, 7, float("inf")), (L - 50, 9, -float("inf"))):
        x["v"][x["table"][0, pos // 16], 0, pos % 16, col] = v
    with _attn_ctx(pkv, x) as ctx:
        got = _tree.values(_attn_run(pkv, ctx, _attn_device(x)))
        _ok(pkv, ctx)
    assert (got[:5, :4, 7] == np.inf).all() and (got[:5, :4, 9] == -np.inf).all()
    for col in (7, 9):
        got[:5, :4, col] = ref[:5, :4, col]
    assert (np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + W * size).all()
