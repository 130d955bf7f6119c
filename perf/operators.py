"""The operators of a speculative, multi-axis decode step over the paged KV
cache, as cases that can be timed and compared: the plain form of each in
elementary torch operations, and (with ``own``) the library's calls.

  slots   the step's plan from lengths that only the GPU knows: pages taken
          from a free list into the block tables, a slot and a position for
          every new token, and the ancestor masks of drafted trees
  rope    rotary embedding with several position axes (time, height, width)
          of q and k, k / v appended at given slots of the paged pools
  tree    attention of a tree of drafted tokens over the cache: every drafted
          token sees the cached tokens and the drafted ones its mask names
  commit  the accepted path of a tree moved to the front of its drafted
          slots, and the new lengths

A case's lengths and tree sizes are drawn from its own ``at``; the values
from the seed of ``prepare``.
"""
import random

import torch

own = False

DEV = "cuda"
_contexts = {}       # one library context per model shape, as a serving program keeps


# ---- cases ------------------------------------------------------------------

def listed():
    llama = dict(Hq=32, Hkv=8, d=128, P=32, base=5e5)
    big = dict(Hq=64, Hkv=8, d=128, P=16, base=5e5)
    small = dict(Hq=8, Hkv=2, d=64, P=16, base=1e4)
    return [
        # one token for each of a few requests: the smallest plan, all latency
        dict(name="slots_decode", op="slots", **small, fp8=False, B=4, lo=17, hi=255, t_lo=1, t_hi=1, tree=False,
             pad=0, at=1),
        # trees of up to 32 drafted tokens for a full batch, padded as for a captured graph
        dict(name="slots_tree", op="slots", **big, fp8=False, B=256, lo=64, hi=2548, t_lo=5, t_hi=32, tree=True,
             pad=256, at=2),
        # one drafted token each for a decode batch of a vision-language model
        dict(name="rope_decode", op="rope", **llama, fp8=False, n=64, sections="16,24,24", interleaved=False),
        # a prompt of several images prefilled at once
        dict(name="rope_prompt", op="rope", **big, fp8=False, n=8192, sections="16,24,24", interleaved=False),
        # an odd chunk into an E4M3 cache, the axes interleaved
        dict(name="rope_fp8", op="rope", **llama, fp8=True, n=1001, sections="24,20,20", interleaved=True),
        # a few short requests: latency
        dict(name="tree_small", op="tree", **small, fp8=False, B=4, lo=17, hi=255, t_lo=1, t_hi=7, at=3),
        # a serving batch with trees of up to 16 tokens
        dict(name="tree_llama8b", op="tree", **llama, fp8=False, B=64, lo=128, hi=4096, t_lo=9, t_hi=16, at=4),
        # the largest trees, eight query heads to each KV head: bound by the tensor cores
        dict(name="tree_wide", op="tree", **big, fp8=False, B=48, lo=64, hi=2548, t_lo=33, t_hi=64, at=5),
        # long contexts, few requests: the split over a long axis
        dict(name="tree_long", op="tree", Hq=32, Hkv=8, d=128, P=64, base=5e5, fp8=False, B=8, lo=32768, hi=131072,
             t_lo=8, t_hi=8, at=6),
        # an E4M3 cache
        dict(name="tree_fp8", op="tree", **llama, fp8=True, B=64, lo=16, hi=6000, t_lo=5, t_hi=24, at=7),
        # the end of a small step
        dict(name="commit_small", op="commit", **small, fp8=False, B=4, lo=17, hi=255, depth=5, at=8),
        # a full batch over an E4M3 cache, rows crossing pages of other scales
        dict(name="commit_fp8", op="commit", **big, fp8=True, B=256, lo=64, hi=2548, depth=8, at=9),
    ]


def _between(rng, lo, hi):
    """A whole number, its logarithm spread evenly over [lo, hi]."""
    return max(lo, min(hi, round(lo * (hi / lo) ** rng.random())))


def draw(rng):
    d = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 4, 8])
    g = rng.choice([1, 2, 3, 4, 5, 8])
    shape = dict(Hq=hkv * g, Hkv=hkv, d=d, P=rng.choice([16, 32, 64]), base=rng.choice([1e4, 5e5]))
    op = rng.choice(["slots", "rope", "tree", "tree", "tree", "commit"])
    at = rng.randrange(1 << 30)
    fp8 = rng.random() < 0.3
    hi = _between(rng, 40, 4096)
    lo = rng.randrange(0, hi)
    if op == "slots":
        tree = rng.random() < 0.5
        t_hi = _between(rng, 1, 64 if tree else 512)
        t_lo = rng.randrange(0, t_hi + 1)
        return dict(op=op, **shape, fp8=False, B=_between(rng, 1, 256), lo=lo, hi=hi, t_lo=t_lo, t_hi=t_hi, tree=tree,
                    pad=rng.choice([0 if t_lo else 1, 13, 256]), at=at)
    if op == "rope":
        axes = rng.randrange(1, 4)
        a = [d // 2 // axes] * axes
        if axes > 1:
            k = rng.randrange(0, a[1])
            a[1] -= k                   # the first axis takes what the others leave
        a[0] = d // 2 - sum(a[1:])
        return dict(op=op, **shape, fp8=fp8, n=_between(rng, 1, 8000), sections=",".join(map(str, a)),
                    interleaved=axes > 1 and rng.random() < 0.5)
    if op == "tree":
        t_hi = _between(rng, 1, 64)
        if rng.random() < 0.2:          # long contexts for few requests
            return dict(op=op, **shape, fp8=fp8, B=rng.randrange(1, 5), lo=8000, hi=_between(rng, 9000, 65536),
                        t_lo=1, t_hi=min(t_hi, 16), at=at)
        return dict(op=op, **shape, fp8=fp8, B=_between(rng, 1, 48), lo=lo, hi=hi, t_lo=rng.randrange(1, t_hi + 1),
                    t_hi=t_hi, at=at)
    return dict(op=op, **shape, fp8=fp8, B=_between(rng, 1, 256), lo=lo, hi=hi, depth=rng.randrange(1, 17), at=at)


def _lengths(case):
    """Cached tokens and new tokens of every request."""
    r = random.Random(case["at"])
    lens = [r.randint(case["lo"], case["hi"]) for _ in range(case["B"])]
    if case["op"] == "commit":
        return lens, [3 * case["depth"]] * case["B"]
    return lens, [r.randint(case["t_lo"], case["t_hi"]) for _ in range(case["B"])]


def work(case):
    row = case["Hkv"] * case["d"] * (1 if case["fp8"] else 2)          # one token's K (or V) in the pool
    d2 = case["d"] * 2
    if case["op"] == "rope":
        n, hq, hkv = case["n"], case["Hq"], case["Hkv"]
        axes = len(case["sections"].split(","))
        scales = 8 * hkv * (-(-n // case["P"])) if case["fp8"] else 0
        return {"bytes": n * (2 * hq * d2 + 2 * hkv * d2 + 2 * row + 4 * axes + 4) + scales,
                "flops": 3 * n * (hq + hkv) * case["d"]}
    lens, new = _lengths(case)
    if case["op"] == "slots":
        n, cap = sum(new), sum(new) + case["pad"]
        fresh = sum(max(0, -(-(a + t) // case["P"]) - -(-a // case["P"])) for a, t in zip(lens, new))
        mask = cap * 4 * _mask_words(case) + 4 * n if case["tree"] else 0
        return {"bytes": 4 * (5 * case["B"] + 3) + 8 * cap + 8 * fresh + 4 * case["B"] + mask, "flops": n}
    if case["op"] == "commit":
        moved = case["B"] * case["depth"] // 2
        return {"bytes": moved * 4 * row + case["B"] * 4 * (3 + case["depth"] // 2), "flops": 0}
    keys = sum(a + t for a, t in zip(lens, new))
    n = sum(new)
    pages = sum(-(-(a + t) // case["P"]) for a, t in zip(lens, new))
    scales = 8 * case["Hkv"] * pages if case["fp8"] else 0
    return {"bytes": 2 * keys * row + 2 * n * case["Hq"] * d2 + 4 * pages + n * 4 * _mask_words(case) + scales,
            "flops": 4 * case["d"] * case["Hq"] * sum(t * (a + t) for a, t in zip(lens, new))}


def _mask_words(case):
    return -(-max(1, case["t_hi"]) // 32)


# ---- inputs -----------------------------------------------------------------

class _Context:
    """A library context, as a program keeps one for its model."""

    def __init__(self, case, batch, blocks, pages):
        from paged_kv_flight_b200 import pkv

        self.pkv = pkv
        self.handle = pkv.pkv_create(pkv.make_config(case["Hq"], case["Hkv"], case["d"], case["P"],
                                                     "fp8" if case["fp8"] else "bf16", case["base"], batch, blocks,
                                                     pages))

    def __del__(self):
        self.pkv.pkv_destroy(self.handle, check=False)


def _context(case, batch, blocks, pages):
    key = (case["Hq"], case["Hkv"], case["d"], case["P"], case["fp8"], case["base"], batch, blocks, pages)
    if key not in _contexts:
        _contexts.clear()
        _contexts[key] = _Context(case, batch, blocks, pages)
    return _contexts[key]


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device=DEV).to(torch.bfloat16)


def _pools(case, pages, gen):
    """K and V of every slot: N(0, 1) in bf16; or E4M3 codes of N(0, 1) with
    one scale for each (page, kv head), as large as the page's largest value needs."""
    shape = (pages, case["Hkv"], case["P"], case["d"])
    if not case["fp8"]:
        return _normal(gen, *shape), _normal(gen, *shape), None, None
    out = []
    for _ in range(2):
        x = torch.randn(*shape, generator=gen, device=DEV)
        x *= torch.empty(pages, case["Hkv"], 1, 1, device=DEV).uniform_(1.2, 3.6, generator=gen)
        s = x.abs().amax((2, 3)) / 448.0
        out.append(((x / s[:, :, None, None]).clamp(-448, 448).to(torch.float8_e4m3fn), s.contiguous()))
    return out[0][0], out[1][0], out[0][1], out[1][1]


def _tables(case, counts, gen):
    """Block tables with the first counts[b] pages of request b's row taken
    from a random order of all pages, -1 behind them; the pages left over."""
    c = _ints(counts).long()
    total, stride = sum(counts), max(max(counts), 1)
    pages = total + total // 10 + 8
    order = torch.randperm(pages, generator=gen, device=DEV)
    j = torch.arange(stride, device=DEV)
    at = (c.cumsum(0) - c)[:, None] + j
    table = torch.where(j < c[:, None], order[at.clamp(max=pages - 1)], -1).int()
    return table.contiguous(), pages, order[total:].int().contiguous()


def _parents(T, total, gen):
    """Drafted trees: the parent of token i is any earlier one or (-1) the cached prefix."""
    i = torch.arange(T, device=DEV)
    u = torch.rand(total, T, generator=gen, device=DEV)
    return (u * (i + 1)).long().clamp(max=i) - 1          # [requests, T], by the token's place in its request


def _ancestors(parents):
    """[.., T, T]: whether token j is token i or one of its ancestors. The
    entries of (1 + parent matrix)^T count paths: positive exactly there."""
    T = parents.shape[-1]
    j = torch.arange(T, device=parents.device)
    step = (parents[..., None] == j).double() + torch.eye(T, dtype=torch.float64, device=parents.device)
    return torch.linalg.matrix_power(step, T) > 0.5


def _pack_bits(seen, words):
    """Truth values [.., T] as [.., words] int32 words, bit j of word w for token 32 w + j."""
    bits = torch.nn.functional.pad(seen, (0, 32 * words - seen.shape[-1])).long()
    v = (bits.unflatten(-1, (words, 32)) << torch.arange(32, device=seen.device)).sum(-1)
    return torch.where(v >= 1 << 31, v - (1 << 32), v).int()


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    s = {"case": case}
    P, d = case["P"], case["d"]
    if case["op"] == "rope":
        n = case["n"]
        need = -(-n // P)
        pages = need + need // 10 + 8
        s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"] = _pools(case, pages, gen)
        s["q"] = _normal(gen, n, case["Hq"], d)
        s["k_new"], s["v_new"] = _normal(gen, n, case["Hkv"], d), _normal(gen, n, case["Hkv"], d)
        s["q_out"] = torch.zeros_like(s["q"])
        s["sections"] = [int(x) for x in case["sections"].split(",")]
        axes = len(s["sections"])
        # a long text before it, then patches of images: rows and columns of a grid, one time each
        i = torch.arange(n, device=DEV)
        start = torch.randint(0, 60000, (1,), generator=gen, device=DEV)
        grid = torch.stack([start + i // 1024, start + i % 1024 // 32, start + i % 32])[:axes]
        s["positions"] = (grid if axes > 1 else start + i[None]).int().contiguous()
        order = torch.randperm(pages, generator=gen, device=DEV)
        s["slots"] = (order[i // P] * P + i % P).int()
        if own:
            s["ctx"] = _context(case, 1, need, pages)
        return s
    lens, new = _lengths(case)
    B = case["B"]
    s["seq_lens"], s["new_lens"] = _ints(lens), _ints(new)
    if case["op"] == "slots":
        held = [-(-a // P) for a in lens]
        need = [max(h, -(-(a + t) // P)) for h, a, t in zip(held, lens, new)]
        full, pages, spare = _tables(case, need, gen)
        j = torch.arange(full.shape[1], device=DEV)
        kept = j < _ints(held)[:, None]
        s["block_tables"] = torch.where(kept, full, -1).contiguous()
        s["pages_held"] = _ints(held)
        taken = full[(~kept) & (full >= 0)]
        stack = torch.cat([spare, taken])
        s["free_pages"] = stack[torch.randperm(stack.numel(), generator=gen, device=DEV)].contiguous()
        s["free_count"] = _ints([stack.numel()])
        cap = sum(new) + case["pad"]
        s["pages_out"], s["free_left"], s["cu_q"] = _ints([0] * B), _ints([0]), _ints([0] * (B + 1))
        s["out_slots"], s["out_positions"] = _ints([0] * cap), _ints([0] * cap)
        s["T"] = max(1, case["t_hi"])
        if case["tree"]:
            words = _mask_words(case)
            every = _parents(s["T"], B, gen)
            n = _ints(new).long()
            at = torch.arange(s["T"], device=DEV) < n[:, None]
            s["parents"] = torch.cat([every[at], torch.full((case["pad"],), -1, device=DEV)]).int().contiguous()
            s["out_mask"] = torch.zeros(cap, words, dtype=torch.int32, device=DEV)
        if own:
            s["ctx"] = _context(case, B, full.shape[1], pages)
        return s
    if case["op"] == "commit":
        depth = case["depth"]
        s["block_tables"], pages, _ = _tables(case, [-(-(a + t) // P) for a, t in zip(lens, new)], gen)
        s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"] = _pools(case, pages, gen)
        gaps = torch.randint(1, 4, (B, depth), generator=gen, device=DEV)
        s["path"] = (gaps.cumsum(1) - 1).int().contiguous()
        s["path_lens"] = torch.randint(0, depth + 1, (B,), generator=gen, device=DEV).int()
        s["lens_out"] = torch.zeros_like(s["seq_lens"])
        if own:
            s["ctx"] = _context(case, B, s["block_tables"].shape[1], pages)
        return s
    s["block_tables"], pages, _ = _tables(case, [-(-(a + t) // P) for a, t in zip(lens, new)], gen)
    s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"] = _pools(case, pages, gen)
    T, n = case["t_hi"], sum(new)
    at = torch.arange(T, device=DEV) < s["new_lens"].long()[:, None]
    s["tree_mask"] = _pack_bits(_ancestors(_parents(T, B, gen)), _mask_words(case))[at].contiguous()
    s["q"] = _normal(gen, n, case["Hq"], d)
    s["out"] = torch.zeros_like(s["q"])
    s["cu_q"] = torch.cat([_ints([0]), s["new_lens"].cumsum(0).int()])
    s["N"] = max(a + t for a, t in zip(lens, new))
    if own:
        s["ctx"] = _context(case, B, s["block_tables"].shape[1], pages)
    return s


# ---- one pass ----------------------------------------------------------------

def run(s):
    return {"slots": _slots, "rope": _rope, "tree": _tree, "commit": _commit}[s["case"]["op"]](s)


def _slots(s):
    tree = s["case"]["tree"]
    if own:
        s["ctx"].pkv.pkv_slot_map(s["ctx"].handle, s["seq_lens"], s["new_lens"], s["block_tables"], s["pages_held"],
                                  s["free_pages"], s["free_count"], s["cu_q"], s["out_slots"], s["out_positions"],
                                  s["pages_out"], s["free_left"], parents=s["parents"] if tree else None,
                                  tree_mask=s["out_mask"] if tree else None)
    else:
        P = s["case"]["P"]
        L, n, held = s["seq_lens"].long(), s["new_lens"].long(), s["pages_held"].long()
        need = torch.maximum(held, (L + n + P - 1) // P)
        take = need - held
        ends = take.cumsum(0)
        served = (take == 0) | (ends <= s["free_count"])
        first = ends - take                                       # pages taken by the requests before
        top = s["free_count"].long() - 1
        cu = torch.cat([torch.zeros_like(n[:1]), n.cumsum(0)])
        row = torch.arange(s["out_slots"].numel(), device=DEV)
        b = (row[:, None] >= cu[1:]).sum(1).clamp(max=n.numel() - 1)
        i = row - cu[b]
        real = row < cu[-1]
        page = ((L[b] + i) // P).clamp(min=0, max=s["block_tables"].shape[1] - 1)
        fresh = s["free_pages"][(top - (first[b] + page - held[b])).clamp(min=0, max=s["free_pages"].numel() - 1)]
        phys = torch.where(page < held[b], s["block_tables"][b, page], fresh).long()
        s["out_slots"].copy_(torch.where(real & served[b], phys * P + (L[b] + i) % P, -1))
        depth = i
        if tree:
            T = s["T"]
            j = torch.arange(T, device=DEV)
            at = (cu[:-1, None] + j).clamp(max=row.numel() - 1)
            seen = _ancestors(torch.where(j < n[:, None], s["parents"].long()[at], -1))
            words = _pack_bits(seen, s["out_mask"].shape[1])
            k = i.clamp(min=0, max=T - 1)
            s["out_mask"].copy_(torch.where(real[:, None], words[b, k], 0))
            depth = seen[b, k].sum(-1) - 1
        s["out_positions"].copy_(torch.where(real, L[b] + depth, -1))
        j = torch.arange(s["block_tables"].shape[1], device=DEV)
        new = s["free_pages"][(top - (first[:, None] + j - held[:, None])).clamp(min=0, max=s["free_pages"].numel() - 1)]
        added = (j >= held[:, None]) & (j < need[:, None]) & served[:, None]
        s["block_tables"].copy_(torch.where(added, new, s["block_tables"]))
        s["pages_out"].copy_(torch.where(served, need, held))
        s["free_left"].copy_(s["free_count"] - (take * served).sum())
        s["cu_q"].copy_(cu)
    got = [s["block_tables"], s["pages_out"], s["free_left"], s["cu_q"], s["out_slots"], s["out_positions"]]
    return got + [s["out_mask"]] if tree else got


def _axis_of_pair(sections, interleaved):
    """The axis whose position turns pair i: runs of sections[a] pairs; or
    interleaved, pair i of axis i mod axes while that axis has pairs left, else of axis 0."""
    n = torch.tensor(sections, device=DEV)
    i = torch.arange(sum(sections), device=DEV)
    if not interleaved:
        return (i[:, None] >= n.cumsum(0)).sum(1)
    a = i % len(sections)
    return torch.where(i < len(sections) * n[a], a, 0)


def _rope(s):
    c = s["case"]
    if own:
        s["ctx"].pkv.pkv_rope_append_axes(s["ctx"].handle, s["q"], s["k_new"], s["v_new"], s["positions"],
                                          s["sections"], s["slots"], s["q_out"], s["k_pool"], s["v_pool"],
                                          s["k_scale"], s["v_scale"], interleaved=c["interleaved"])
    else:
        half = c["d"] // 2
        theta = c["base"] ** (-torch.arange(half, dtype=torch.float64, device=DEV) / half)
        angle = s["positions"].double()[_axis_of_pair(s["sections"], c["interleaved"])].T * theta    # far positions: 64 bits
        cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

        def turned(x):
            a, b = x[..., :half].float(), x[..., half:].float()
            return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)

        s["q_out"].copy_(turned(s["q"]))
        page, at = s["slots"].long() // c["P"], s["slots"].long() % c["P"]
        for_k, for_v = turned(s["k_new"]), s["v_new"].float()
        if c["fp8"]:
            for_k = (for_k / s["k_scale"][page][..., None]).clamp(-448, 448)
            for_v = (for_v / s["v_scale"][page][..., None]).clamp(-448, 448)
            s["k_pool"].view(torch.uint8)[page, :, at] = for_k.to(torch.float8_e4m3fn).view(torch.uint8)
            s["v_pool"].view(torch.uint8)[page, :, at] = for_v.to(torch.float8_e4m3fn).view(torch.uint8)
        else:
            s["k_pool"][page, :, at] = for_k.to(torch.bfloat16)
            s["v_pool"][page, :, at] = s["v_new"]
    return [s["q_out"], s["k_pool"], s["v_pool"]]


def _tree(s):
    c = s["case"]
    if own:
        s["ctx"].pkv.pkv_decode_attn_tree(s["ctx"].handle, s["q"], s["k_pool"], s["v_pool"], s["k_scale"],
                                          s["v_scale"], s["block_tables"], s["seq_lens"], s["cu_q"], s["tree_mask"],
                                          s["out"])
        return s["out"]
    P, N, T, Hkv, d = c["P"], s["N"], c["t_hi"], c["Hkv"], c["d"]
    G = c["Hq"] // Hkv
    L, n, cu = s["seq_lens"].long(), s["new_lens"].long(), s["cu_q"].long()
    j = torch.arange(N, device=DEV)
    page, at = s["block_tables"][:, j // P].long().clamp(min=0), j % P

    def cached(pool, scale):      # [batch, kv heads, keys, d]
        if not c["fp8"]:
            return pool[page, :, at].float().transpose(1, 2)
        x = pool.view(torch.uint8)[page, :, at].view(torch.float8_e4m3fn).float()
        return (x * scale[page][..., None]).transpose(1, 2)

    t = torch.arange(T, device=DEV)
    rows = (cu[:-1, None] + t).clamp(max=s["q"].shape[0] - 1)                       # packed row of token t of request b
    q = s["q"][rows].float().view(-1, T, Hkv, G, d).permute(0, 2, 3, 1, 4).reshape(-1, Hkv, G * T, d)
    word = s["tree_mask"][rows]                                                      # [batch, T, words]
    k = (j - L[:, None]).clamp(min=0, max=32 * word.shape[-1] - 1)                   # drafted place of key j
    bit = (word.gather(2, (k // 32)[:, None].expand(-1, T, -1)) >> (k % 32)[:, None]) & 1
    seen = (j < L[:, None])[:, None] | ((j < (L + n)[:, None])[:, None] & (bit == 1))      # [batch, T, keys]
    x = (q @ cached(s["k_pool"], s["k_scale"]).transpose(2, 3)).mul_(d ** -0.5).view(-1, Hkv, G, T, N)
    x.masked_fill_(~seen[:, None, None], float("-inf"))
    top = x.amax(-1, keepdim=True)
    x = x.sub_(torch.where(top > float("-inf"), top, 0)).exp_()
    total = x.sum(-1, keepdim=True)
    x = x.div_(torch.where(total > 0, total, 1)).view(-1, Hkv, G * T, N) @ cached(s["v_pool"], s["v_scale"])
    x = x.view(-1, Hkv, G, T, d).permute(0, 3, 1, 2, 4).reshape(-1, T, c["Hq"], d)
    r = torch.arange(s["q"].shape[0], device=DEV)
    b = (r[:, None] >= cu[1:]).sum(1)
    s["out"].copy_(x[b, r - cu[b]])
    return s["out"]


def _commit(s):
    c = s["case"]
    if own:
        s["ctx"].pkv.pkv_tree_commit(s["ctx"].handle, s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"],
                                     s["block_tables"], s["seq_lens"], s["path"], s["path_lens"], s["lens_out"])
    else:
        P, L = c["P"], s["seq_lens"].long()[:, None]
        j = torch.arange(s["path"].shape[1], device=DEV)
        source = torch.where(j < s["path_lens"][:, None], s["path"].long(), j)       # not accepted: stays in its place
        b = torch.arange(c["B"], device=DEV)[:, None]
        p0, a0 = s["block_tables"][b, (L + source) // P].long(), (L + source) % P
        p1, a1 = s["block_tables"][b, (L + j) // P].long(), (L + j) % P
        moved = []
        if c["fp8"]:
            for_k = s["k_pool"].view(torch.uint8)[p0, :, a0].view(torch.float8_e4m3fn).float()
            for_v = s["v_pool"].view(torch.uint8)[p0, :, a0].view(torch.float8_e4m3fn).float()
            for_k = for_k * s["k_scale"][p0][..., None] / s["k_scale"][p1][..., None]
            for_v = for_v * s["v_scale"][p0][..., None] / s["v_scale"][p1][..., None]
            moved = [x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8) for x in (for_k, for_v)]
            s["k_pool"].view(torch.uint8)[p1, :, a1], s["v_pool"].view(torch.uint8)[p1, :, a1] = moved
        else:
            for_k, for_v = s["k_pool"][p0, :, a0], s["v_pool"][p0, :, a0]
            s["k_pool"][p1, :, a1], s["v_pool"][p1, :, a1] = for_k, for_v
        s["lens_out"].copy_(s["seq_lens"] + s["path_lens"])
    return [s["k_pool"], s["v_pool"], s["lens_out"]]


# ---- the definitions in 64 bits ----------------------------------------------

def exact(case, seed):
    if case["op"] == "slots":
        return None
    s = prepare(case, seed)
    P, d, half = case["P"], case["d"], case["d"] // 2

    def values(name):
        x = s[name].double()
        return x * s[name[0] + "_scale"].double()[:, :, None, None] if case["fp8"] else x

    if case["op"] == "rope":
        n, sec = case["n"], s["sections"]
        axis = [0] * half
        at = sec[0]
        for a in range(1, len(sec)):
            for k in range(sec[a]):
                axis[a + k * len(sec) if case["interleaved"] else at + k] = a
            at += sec[a]
        turn = torch.stack([s["positions"][axis[i]].double() * case["base"] ** (-2.0 * i / d) for i in range(half)], 1)
        z = torch.polar(torch.ones_like(turn), turn)[:, None]

        def rotated(x):
            y = torch.complex(x[..., :half].double(), x[..., half:].double()) * z
            return torch.cat([y.real, y.imag], -1)

        out = [s["k_pool"].double(), s["v_pool"].double()]
        for x, y, scale in zip(out, (rotated(s["k_new"]), s["v_new"].double()), (s["k_scale"], s["v_scale"])):
            page = (s["slots"] // P).long()
            if case["fp8"]:
                y = (y / scale.double()[page][..., None]).clamp(-448, 448)      # E4M3 saturates
            x[page, :, (s["slots"] % P).long()] = y
        return [rotated(s["q"])] + out
    if case["op"] == "commit":
        k, v = values("k_pool"), values("v_pool")
        out = [s["k_pool"].double(), s["v_pool"].double()]
        table, lens, path, count = (s[x].tolist() for x in ("block_tables", "seq_lens", "path", "path_lens"))
        move = [(table[b][(L + path[b][i]) // P], (L + path[b][i]) % P, table[b][(L + i) // P], (L + i) % P)
                for b, L in enumerate(lens) for i in range(count[b]) if path[b][i] != i]
        if move:
            p0, a0, p1, a1 = torch.tensor(move, device=DEV).T
            for x, y, scale in zip(out, (k, v), (s["k_scale"], s["v_scale"])):
                z = y[p0, :, a0]
                x[p1, :, a1] = (z / scale.double()[p1][..., None]).clamp(-448, 448) if case["fp8"] else z
        return out + [None]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    G = case["Hq"] // case["Hkv"]
    lens, cu, mask = s["seq_lens"].tolist(), s["cu_q"].tolist(), s["tree_mask"].tolist()
    for b, L in enumerate(lens):
        t = cu[b + 1] - cu[b]
        if not t:
            continue
        pages = s["block_tables"][b, :-(-(L + t) // P)].long()
        k, v = (s[x][pages].double() for x in ("k_pool", "v_pool"))
        if case["fp8"]:
            k, v = k * s["k_scale"][pages].double()[..., None, None], v * s["v_scale"][pages].double()[..., None, None]
        k, v = (x.transpose(0, 1).reshape(case["Hkv"], -1, d)[:, :L + t] for x in (k, v))
        sees = torch.tensor([[(w[j // 32] >> (j % 32)) & 1 for j in range(t)] for w in mask[cu[b]:cu[b + 1]]],
                            device=DEV, dtype=torch.bool)
        sees = torch.cat([torch.ones(t, L, dtype=torch.bool, device=DEV), sees], 1)
        q = s["q"][cu[b]:cu[b + 1]].double().view(t, case["Hkv"], G, d)
        x = torch.einsum("thgd,hkd->hgtk", q, k) / d ** 0.5
        x = torch.where(sees, x, -torch.inf).softmax(-1)
        out[cu[b]:cu[b + 1]] = torch.einsum("hgtk,hkd->thgd", x, v).reshape(t, case["Hq"], d)
    return out
