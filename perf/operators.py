"""Speculative decoding over the RAT+ decode cache: what is measured, and its plain forms.

Four operators, in the order in which a serving loop calls them for a batch of sequences whose
drafter proposes a tree of tokens each step:

  pages    the page table brought in line with the sequences' lengths: pages taken from and given
           back to a free list, on the GPU (rat_page_table_update)
  tree     attention of every drafted node over the cache and over its own branch of the tree, with
           the gated recurrence carried down each branch (rat_tree_decode_step and its paged form)
  commit   the accepted branch written to the cache, the recurrent state moved to its last node
           (rat_tree_commit and its paged form)
  slots    the pool rows of a run of positions, for gathering or moving cached rows (rat_slot_map)

Definitions.  Entry b holds positions 0 .. pos_b - 1.  Node i has parent p_i < i (-1: the last held
position, -2: an absent node, padding), depth n_i (0 for a child of -1), position t_i = pos_b + n_i and
state s_i = a_i s_{p_i} + (1 - a_i) x_i for x = k, v with a_i = sigmoid(g_i) (a = 0 in heads without
recurrence; s_{-1} the entry's state); its cache row is s_i rounded to the cache's type.  Node i
attends, in one softmax, to the held positions and the nodes of its branch (itself included) that lie
in its dilated set { j <= t_i : (t_i - j) mod D = 0 } (on the fixed grid: { j <= t_i : j mod D = D - 1 }
and itself, once), and once more to those in its window { t_i - W + 1 .. t_i } (with dedupe: only those
the dilated set lacks).

In a case, the first `dense` heads have D = 1, no window and no recurrence, the others dilation D,
window W and the recurrence.  `page` is the number of rows of a page (0: one dense cache).
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
#: spread of the augmented keys and values under gate logits ~ N(2, 1), and of raw ones
RECURRENT_STD, RAW_STD = 0.3, 1.0


def _rat():
    import recurrence_augmented_dilated_gated_b200 as rat

    return rat


def _tree(name, **kw):
    c = dict(name=name, op="tree", B=1, N=8, H=16, dense=0, d=128, D=16, W=0, depth=4, ctx=4096, dtype="bf16", page=0,
             grid=False, dedupe=False, sep=False)
    c.update(kw)
    return c


def listed():
    return [
        # one user, a short drafted chain with one fork: the step's latency
        _tree("tree-b1-n8", N=8, depth=5, ctx=4096),
        # the decode study's heads (16 x 128, D = 16) with a serving batch and a middle-sized tree
        _tree("tree-b64-n32", B=64, N=32, depth=6, ctx=16384),
        # dense heads only (D = 1): every node reads every row, the most arithmetic for each byte
        _tree("tree-dense-n64", B=16, N=64, D=1, depth=9, ctx=16000),
        # the hybrid mix (4 dense heads, 28 with D = 64 and W = 256) at long context: the largest
        _tree("tree-hybrid-n48", B=8, N=48, H=32, dense=4, D=64, W=256, depth=7, ctx=65536),
        # fp32, odd sizes, separate gates, keys of both parts counted once
        _tree("tree-f32-odd", B=3, N=21, H=5, dense=1, d=64, D=3, W=37, depth=7, ctx=1531, dtype="f32", dedupe=True,
              sep=True),
        # fixed grid with its window ring, in pages, as a serving engine holds it
        _tree("tree-paged-grid", B=32, N=16, D=16, W=128, depth=5, ctx=32768, page=64, grid=True),
        # the largest batch, a small accepted branch in each entry
        _tree("commit-b256", op="commit", B=256, N=32, depth=6, ctx=600),
        # pages, hybrid heads, fp32, the largest tree
        _tree("commit-paged-f32", op="commit", B=24, N=64, H=32, dense=4, D=64, W=256, depth=9, ctx=900, dtype="f32",
              page=32),
        # a small server: a few sequences grow, one starts, one ends
        _tree("pages-b8", op="pages", B=8, N=16, D=16, ctx=4096, page=64),
        # the largest table: 256 sequences of up to 32768 positions
        _tree("pages-b256", op="pages", B=256, N=32, H=32, dense=4, D=64, W=256, ctx=32768, page=64),
        # the rows that a tree's positions will take
        _tree("slots-b8", op="slots", B=8, N=9, H=7, D=5, W=33, ctx=1000, page=16, grid=True),
        # the rows of whole prompts, for moving them between pools
        _tree("slots-b64", op="slots", B=64, N=4001, H=32, dense=4, D=64, W=256, ctx=16384, page=64),
    ]


def draw(rng):
    """One more case: sizes log-uniform over the listed cases' ranges, odd ones among them."""
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["tree", "tree", "tree", "commit", "pages", "slots"])
    dense = rng.choice([0, 0, 1, 4])
    H = dense + rng.choice([1, 3, 5, 12, 16, 28])
    d, dtype = rng.choice([64, 128]), rng.choice(["bf16", "bf16", "bf16", "f32"])
    D = rng.choice([1, 2, 3, 5, 8, 16, 16, 48, 64])
    grid = rng.random() < 0.3
    W = rng.choice([0, 0, 16, 37, 128, 256]) if op == "tree" else 64
    depth = rng.randint(1, 9)
    c = _tree(None, op=op, H=H, dense=dense, d=d, dtype=dtype, D=D, W=W, depth=depth, grid=grid,
              dedupe=rng.random() < 0.3, sep=rng.random() < 0.2, page=rng.choice([0, 0, 16, 40, 64]))
    del c["name"]
    if op == "slots":
        c.update(B=log(1, 48), N=log(1, 3000), ctx=log(64, 16000))
        c["N"] = min(c["N"], c["ctx"])
        return c
    c["N"] = max(depth, log(1, 64))
    if op == "pages":
        c.update(B=log(1, 200), ctx=log(64, 32000), page=rng.choice([16, 40, 64, 128]))
        return c
    if op == "commit":
        c.update(B=log(1, 128), ctx=log(64, 700))
        return c
    c["ctx"] = log(64, 30000)
    # no dearer than the largest listed case: 2 GB of cache rows read, 8 GB of cache
    row = 2 * d * (2 if dtype == "bf16" else 4)
    reads = (dense + (H - dense) * (1.0 / D if grid else min(D, depth) / D)) * c["ctx"] * row
    c["B"] = max(1, min(log(1, 64), int(2e9 / reads), int(8e9 / (H * c["ctx"] * row))))
    return c


# ------------------------------------------------------------------ shapes


def _dtype(c):
    return torch.bfloat16 if c["dtype"] == "bf16" else torch.float32


def _cap(c):
    return c["ctx"] + max(c["N"], 16)


def _kinds(c):
    """(first head, end, D, W, recurrent) of the two kinds of heads."""
    out = []
    if c["dense"]:
        out.append((0, c["dense"], 1, 0, False))
    if c["H"] > c["dense"]:
        out.append((c["dense"], c["H"], c["D"], c["W"], True))
    return out


def _rows_per_head(c):
    """Rows of one (entry, head) block: residue-major, or the grid and its ring."""
    cap, R = _cap(c), 0
    for _, _, D, W, _ in _kinds(c):
        S = -(-cap // D)
        R = max(R, S + (W if D > 1 else 0) if c["grid"] else D * S)
    return R


def _positions(c):
    """Held positions of each entry: ragged, from three quarters of `ctx` to all of it."""
    spread = max(1, c["ctx"] // 4)
    return [c["ctx"] - (b * 389) % spread for b in range(c["B"])]


def _attn_window(c, D, W):
    return 0 if c["dedupe"] and D == 1 else W


def work(c):
    """Cache rows each read once, tokens, states and results once; two products per node and key."""
    B, N, H, d = c["B"], c["N"], c["H"], c["d"]
    e = 2 if c["dtype"] == "bf16" else 4
    if c["op"] == "pages":
        pps = -(-_rows_per_head(c) // c["page"])
        return {"bytes": 8.0 * B * pps + 4.0 * B, "flops": 0.0}
    if c["op"] == "slots":
        table = 4.0 * B * -(-_rows_per_head(c) // c["page"]) if c["page"] else 0.0
        return {"bytes": 8.0 * B * N * H * (2 if c["grid"] else 1) + table + 8.0 * B, "flops": 0.0}
    gates = 2 if c["sep"] else 1
    if c["op"] == "commit":
        n = sum(_accepted(c, b) for b in range(B))
        return {"bytes": n * H * d * e * (4.0 + gates) + 16.0 * B * H * d + 4.0 * B * (N + 3), "flops": 8.0 * n * H * d}
    rows = pairs = 0
    for h0, h1, D, W, _ in _kinds(c):
        W, G = _attn_window(c, D, W), min(D, c["depth"])
        for p in _positions(c):
            w = min(max(0, W - 1), p)
            if c["grid"]:
                n = p // D + (w if D > 1 else 0)
                per_node = p // D
            else:
                n = sum(len(range((p + g) % D, p, D)) for g in range(G)) + sum((j - p) % D >= G for j in range(p - w, p))
                per_node = p // D
            rows += (h1 - h0) * n
            pairs += (h1 - h0) * N * (per_node + w + (c["depth"] + 1) / 2)
    return {"bytes": 2.0 * rows * d * e + B * N * H * d * e * (4.0 + gates) + 8.0 * B * H * d + 4.0 * B * N * (H + 1),
            "flops": 4.0 * pairs * d}


# ------------------------------------------------------------------ inputs


def _accepted(c, b):
    """Nodes of the accepted branch of entry b: a drafter is right for some tokens, rarely for all."""
    return (b * 7 + 3) % (c["depth"] + 1)


def _parents(c, rs):
    """[B, N] parents.  A branch of full depth, shuffled among shorter ones; every third entry is padded."""
    B, N, L = c["B"], c["N"], c["depth"]
    out = np.full((B, N), -2, np.int32)
    for b in range(B):
        n = max(L, N - (b % 3) * (N // 8))
        spine = set(rs.choice(n, L, replace=False).tolist())
        depth, last = np.zeros(n, np.int64), -1
        for i in range(n):
            if i in spine:
                p, last = last, i
            else:
                p = int(rs.randint(-1, i)) if i else -1
                p = p if p < 0 or depth[p] < L - 1 else -1
            out[b, i] = p
            depth[i] = 0 if p < 0 else depth[p] + 1
    return out


def _leaves(c, parent):
    """[B] the node at the end of each accepted branch: an ancestor on the deepest one (-1: none)."""
    out = np.full(c["B"], -1, np.int32)
    for b in range(c["B"]):
        depth = np.full(c["N"], -1)
        for i, p in enumerate(parent[b]):
            if p > -2:
                depth[i] = 0 if p < 0 else depth[p] + 1
        i, n = int(depth.argmax()), _accepted(c, b)
        while i >= 0 and depth[i] + 1 > n:
            i = int(parent[b, i])
        out[b] = i
    return out


def _normal(gen, shape, std, dtype, mean=0.0):
    return torch.empty(shape, dtype=dtype, device=DEV).normal_(mean, std, generator=gen)


def _config(c, T):
    rat = _rat()
    dil, win, rec = [], [], []
    for h0, h1, D, W, r in _kinds(c):
        dil += [D] * (h1 - h0)
        win += [W] * (h1 - h0)
        rec += [int(r)] * (h1 - h0)
    flags = rat.RAT_FLAG_GRID_DILATION * c["grid"] | rat.RAT_FLAG_DEDUPE * c["dedupe"]
    flags |= rat.RAT_FLAG_SEPARATE_GATES * c["sep"]
    return rat.Config(c["B"], T, c["H"], c["d"], _dtype(c), dil, win, rec, flags=flags)


def prepare(c, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    rs = np.random.RandomState(seed % (1 << 32))
    B, N, H, d = c["B"], c["N"], c["H"], c["d"]
    R, cap = _rows_per_head(c), _cap(c)
    st = {"case": c, "R": R, "cap": cap}
    if c["page"]:
        st["pps"] = -(-R // c["page"])
        st["num_pages"] = B * st["pps"]
    if c["op"] == "pages":
        return _prepare_pages(c, st, gen)
    st["pos"] = torch.tensor(_positions(c), dtype=torch.int32, device=DEV)
    if c["page"]:
        st["table"] = torch.randperm(st["num_pages"], generator=gen, device=DEV).to(torch.int32).view(B, st["pps"])
    if c["op"] == "slots":
        st["pos"] = torch.tensor(rs.randint(0, cap - N + 1, B), dtype=torch.int32, device=DEV)
        st["count"] = torch.tensor(rs.randint(0, N + 1, B), dtype=torch.int32, device=DEV)
        if own:
            rat = _rat()
            cfg = st["cfg"] = _config(c, N)
            st["ws"] = rat.workspace(cfg, rat.RAT_OP_STATUS)
            # the row arithmetic needs the table only, so any pool of the table's shape will do
            st["cache"] = _slot_cache(c, st, cfg) if c["page"] else None
            st["slots"] = torch.empty(B, N, H, dtype=torch.int64, device=DEV)
            st["ring"] = torch.empty_like(st["slots"]) if c["grid"] else None
        return st
    dt = _dtype(c)
    shape = (st["num_pages"], H, c["page"], d) if c["page"] else (B, H, R, d)
    for x in ("k", "v"):
        cache = st["cache_" + x] = _normal(gen, shape, RECURRENT_STD, dt)
        if c["dense"]:
            cache[:, :c["dense"]].mul_(RAW_STD / RECURRENT_STD)
        if c["grid"]:
            _fill_ring(c, st, cache)
    for x in ("q", "k", "v"):
        st[x] = _normal(gen, (B, N, H, d), RAW_STD, dt)
    st["g"] = _normal(gen, (2, B, N, H, d) if c["sep"] else (B, N, H, d), 1.0, dt, 2.0)
    for x in ("state_k", "state_v"):
        st[x] = _normal(gen, (B, H, d), RECURRENT_STD, torch.float32)
    parent = _parents(c, rs)
    st["parent"] = torch.from_numpy(parent).to(DEV)
    if c["op"] == "commit":
        st["leaf"] = torch.from_numpy(_leaves(c, parent)).to(DEV)
        st["out_state_k"], st["out_state_v"] = torch.empty_like(st["state_k"]), torch.empty_like(st["state_v"])
        st["out_pos"] = torch.empty_like(st["pos"])
    if own:
        rat = _rat()
        cfg = st["cfg"] = _config(c, N)
        op = rat.RAT_OP_TREE if c["op"] == "tree" else rat.RAT_OP_STATUS
        st["ws"] = rat.workspace(cfg, op, cap)
        st["o"], st["lse"] = torch.empty_like(st["q"]), torch.empty(B, H, N, device=DEV)
        if c["page"]:
            st["cache"] = rat.paged_cache(cfg, st["cache_k"], st["cache_v"], st["table"], cap)
    return st


def _fill_ring(c, st, cache):
    """A position on the grid that is in the window too has the same row in both."""
    flat = cache.view(-1, c["d"])
    for h0, h1, D, W, _ in _kinds(c):
        if D > 1 and W > 0:
            j = st["pos"].long()[:, None] - W + torch.arange(W, device=DEV)
            both = ((j >= 0) & (j % D == D - 1))[:, :, None].expand(-1, -1, h1 - h0)
            j = j.clamp(min=0)
            grid, ring = (_slot(c, st, h0, h1, row) for row in (j // D, -(-st["cap"] // D) + j % W))
            flat[ring[both]] = flat[grid[both]]


def _slot_cache(c, st, cfg):
    """A page descriptor over pools as large as the server's, for the calls that read its table only."""
    st["pool"] = torch.empty(st["num_pages"], c["H"], c["page"], c["d"], dtype=_dtype(c), device=DEV)
    return _rat().paged_cache(cfg, st["pool"], st["pool"], st["table"], st["cap"])


def _prepare_pages(c, st, gen):
    """A table in use: lengths that some steps led to, an eighth of the entries idle.  Then: an eighth of the
    running sequences end, idle entries start a prompt, the rest grow."""
    B, cap = c["B"], st["cap"]
    top = c["ctx"] - c["N"]
    u = torch.rand(3, B, generator=gen, device=DEV)
    before = (u[0] * max(1, top)).int().clamp_(min=0)
    idle = u[1] < 0.125
    before = torch.where(idle, -1, before)
    after = torch.where(idle, (u[2] * max(1, top)).int(), torch.where(u[2] < 0.125, -1, before + (u[2] * 8).int()))
    st["length"] = after.to(torch.int32).clamp_(max=cap)
    table = torch.full((B, st["pps"]), -1, dtype=torch.int32, device=DEV)
    free = torch.randperm(st["num_pages"], generator=gen, device=DEV).to(torch.int32)
    n_free = torch.full((1,), st["num_pages"], dtype=torch.int32, device=DEV)
    st["table"], st["free"], st["n_free"] = _plain_pages(c, st, table, free, n_free, before.to(torch.int32))
    if own:
        rat = _rat()
        st["cfg"] = _config(c, 0)
        st["ws"] = rat.workspace(st["cfg"], rat.RAT_OP_STATUS)
    return st


# ------------------------------------------------------------------ the passes


def run(st):
    c = st["case"]
    op = c["op"]
    if op == "pages":
        # the server's table and free list are updated in place: the pass starts from copies
        table, free, n_free = st["table"].clone(), st["free"].clone(), st["n_free"].clone()
        if own:
            _rat().rat_page_table_update(st["cfg"], table, c["page"], st["num_pages"], st["cap"], st["length"], c["N"],
                                         free, n_free, st["ws"])
        else:
            table, free, n_free = _plain_pages(c, st, table, free, n_free, st["length"], c["N"])
        return {"table": table, "free": free, "n_free": n_free}
    if op == "slots":
        if own:
            _rat().rat_slot_map(st["cfg"], st["cache"], st["cap"], st["pos"], st["count"], st["slots"], st["ring"], st["ws"])
            return {"slots": st["slots"], "ring": st["ring"]}
        return _plain_slots(c, st)
    if op == "commit":
        if own:
            rat, a = _rat(), st
            head = (a["cfg"], a["k"], a["v"], a["g"], a["parent"], a["leaf"], a["state_k"], a["state_v"], a["out_state_k"],
                    a["out_state_v"])
            tail = (a["cap"], a["pos"], a["out_pos"], a["ws"])
            if c["page"]:
                rat.rat_tree_commit_paged(*head, a["cache"], *tail)
            else:
                rat.rat_tree_commit(*head, a["cache_k"], a["cache_v"], *tail)
        else:
            _plain_commit(c, st)
        return {x: st[x] for x in ("out_state_k", "out_state_v", "cache_k", "cache_v", "out_pos")}
    if own:
        rat, a = _rat(), st
        head = (a["cfg"], a["q"], a["k"], a["v"], a["g"], a["parent"], a["state_k"], a["state_v"])
        tail = (a["cap"], a["pos"], a["o"], a["lse"], a["ws"])
        if c["page"]:
            rat.rat_tree_decode_step_paged(*head, a["cache"], *tail)
        else:
            rat.rat_tree_decode_step(*head, a["cache_k"], a["cache_v"], *tail)
        return {"o": st["o"], "lse": st["lse"]}
    return _plain_tree(c, st)


# ------------------------------------------------------------------ plain forms


def _branches(c, parent):
    """(depth [B, N], ancestors-or-self [B, N, N]) of the nodes; absent nodes have depth -1 and no ancestors."""
    N = c["N"]
    there = parent > -2
    anc = torch.eye(N, dtype=torch.bool, device=parent.device) & there[:, :, None]
    up = parent.long().clamp(min=0)[:, :, None].expand(-1, -1, N)
    for _ in range(c["depth"] - 1):  # a node's branch is its parent's and itself
        anc = anc | (torch.gather(anc, 1, up) & (parent >= 0)[:, :, None])
    return anc.sum(2) - 1, anc


def _states(c, st):
    """The recurrence down every branch, in 64 bits: (k, v) states of the nodes, [B, N, H, d]."""
    parent = st["parent"]
    up = parent.long().clamp(min=0)[:, :, None, None].expand(-1, -1, c["H"], c["d"])
    recurrent = (torch.arange(c["H"], device=DEV) >= c["dense"])[None, None, :, None]
    out = []
    for i, x in enumerate(("k", "v")):
        a = torch.sigmoid((st["g"][i] if c["sep"] else st["g"]).double()) * recurrent
        fresh = (1 - a) * st[x].double()
        first = st["state_" + x].double()[:, None]
        s = fresh + a * first
        for _ in range(c["depth"] - 1):
            s = fresh + a * torch.where((parent >= 0)[:, :, None, None], torch.gather(s, 1, up), first)
        out.append(s)
    return out


def _main_row(c, st, D, j):
    S = -(-st["cap"] // D)
    return j // D if c["grid"] else (j % D) * S + j // D


def _slot(c, st, h0, h1, row):
    """[B, M, h1 - h0] rows of the flat pool (or of the flat dense cache) for logical rows [B, M]."""
    B, H = c["B"], c["H"]
    h = torch.arange(h0, h1, device=row.device)
    if not c["page"]:
        b = torch.arange(B, device=row.device)[:, None, None]
        return (b * H + h) * st["R"] + row[:, :, None]
    page = torch.gather(st["table"].long(), 1, row // c["page"])
    return (page[:, :, None] * H + h) * c["page"] + (row % c["page"])[:, :, None]


def _plain_tree(c, st):
    B, N, d = c["B"], c["N"], c["d"]
    dt, cap = _dtype(c), st["cap"]
    pos = st["pos"].long()
    depth, anc = _branches(c, st["parent"])
    there = (depth >= 0)[:, :, None]
    node_k, node_v = (s.to(dt).float() for s in _states(c, st))
    flat_k, flat_v = st["cache_k"].view(-1, d), st["cache_v"].view(-1, d)
    o, lse = torch.empty_like(st["q"]), torch.empty(B, c["H"], N, device=DEV)
    for h0, h1, D, W, _ in _kinds(c):  # at most two kinds of heads
        W = _attn_window(c, D, W)
        # candidate rows: the dilated sets of the tree's positions, then the window
        if c["grid"]:
            j = (torch.arange(-(-c["ctx"] // D), device=DEV) * D + D - 1).expand(B, -1)
            held = there & (j < pos[:, None])[:, None]
        else:
            first = (pos[:, None] + torch.arange(min(D, c["depth"]), device=DEV)) % D
            j = (first[:, :, None] + torch.arange(-(-c["ctx"] // D), device=DEV) * D).flatten(1)
            held = there & (j < pos[:, None])[:, None] & ((pos[:, None, None] + depth[:, :, None] - j[:, None]) % D == 0)
        row, weight = _main_row(c, st, D, j.clamp(max=cap - 1)), [held]
        t = pos[:, None] + depth
        if W:
            jw = pos[:, None] - W + torch.arange(W, device=DEV)
            near = there & (jw >= 0)[:, None] & (jw[:, None] > t[:, :, None] - W)
            if c["dedupe"]:
                near &= (jw % D != D - 1)[:, None] if c["grid"] else (t[:, :, None] - jw[:, None]) % D != 0
            jc = jw.clamp(min=0)
            ring = c["grid"] and D > 1
            row = torch.cat([row, -(-cap // D) + jc % W if ring else _main_row(c, st, D, jc)], 1)
            weight.append(near)
        back = depth[:, :, None] - depth[:, None]  # steps from a node up to an ancestor
        if c["grid"]:
            mine = (t[:, None] % D == D - 1) | (back == 0)
        else:
            mine = back % D == 0
        near = (back < W) & ~mine if c["dedupe"] else back < W
        weight = torch.cat([w.float() for w in weight] + [anc * (mine.float() + near.float())], 2)[:, None]
        slot = _slot(c, st, h0, h1, row)
        keys = torch.cat([flat_k[slot].float(), node_k[:, :, h0:h1]], 1).transpose(1, 2)
        values = torch.cat([flat_v[slot].float(), node_v[:, :, h0:h1]], 1).transpose(1, 2)
        q = st["q"][:, :, h0:h1].float().transpose(1, 2)
        score = (q @ keys.transpose(2, 3)) / math.sqrt(d)
        top = torch.where(weight > 0, score, -math.inf).amax(3, keepdim=True)
        top = torch.where(top == -math.inf, 0.0, top)
        p = weight * torch.exp(torch.where(weight > 0, score, -math.inf) - top)
        total = p.sum(3, keepdim=True)
        res = torch.where(total > 0, (p @ values) / total, 0.0)
        o[:, :, h0:h1] = res.transpose(1, 2).to(dt)
        lse[:, h0:h1] = (top + torch.log(total))[..., 0]
    return {"o": o, "lse": lse}


def _plain_commit(c, st):
    B, H, d, L, dt = c["B"], c["H"], c["d"], c["depth"], _dtype(c)
    pos, leaf = st["pos"].long(), st["leaf"].long()
    depth, anc = _branches(c, st["parent"])
    any_ = leaf >= 0
    at = leaf.clamp(min=0)
    path = torch.gather(anc, 1, at[:, None, None].expand(-1, 1, c["N"]))[:, 0] & any_[:, None]
    # the branch's node at each depth, and whether there is one
    level = path[:, None] & (depth[:, None] == torch.arange(L, device=DEV)[:, None])
    there, node = level.any(2), level.int().argmax(2)
    j = (pos[:, None] + torch.arange(L, device=DEV)).clamp(max=st["cap"] - 1)
    for s, x in zip(_states(c, st), ("k", "v")):
        end = torch.gather(s, 1, at[:, None, None, None].expand(-1, 1, H, d))[:, 0]
        st["out_state_" + x].copy_(torch.where(any_[:, None, None], end, st["state_" + x].double()))
        new = torch.gather(s, 1, node[:, :, None, None].expand(-1, -1, H, d)).to(dt)
        flat = st["cache_" + x].view(-1, d)
        for h0, h1, D, W, _ in _kinds(c):
            rows = [(_main_row(c, st, D, j), there & (j % D == D - 1) if c["grid"] else there)]
            if c["grid"] and D > 1 and W > 0:
                rows.append((-(-st["cap"] // D) + j % W, there))
                # off the grid a row is named by a later position of the branch too: write the ring's there
                rows[0] = (torch.where(rows[0][1], *(r for r, _ in rows)), there)
            for row, write in rows:
                slot = _slot(c, st, h0, h1, row)
                flat[slot] = torch.where(write[:, :, None, None], new[:, :, h0:h1], flat[slot])
    st["out_pos"].copy_(pos + path.sum(1))


def _needed(c, st, length, extra):
    """[B, pages per sequence] whether a page holds one of the first length + extra positions of some head."""
    row = torch.arange(st["pps"] * c["page"], device=DEV)[None]
    n = torch.where(length >= 0, (length.long() + extra).clamp(max=st["cap"]), 0)[:, None]
    used = torch.zeros(c["B"], row.shape[1], dtype=torch.bool, device=DEV)
    for _, _, D, W, _ in _kinds(c):
        S = -(-st["cap"] // D)
        if c["grid"]:
            used |= row < n // D
            if D > 1 and W > 0:
                used |= (row >= S) & (row < S + n.clamp(max=W))
        else:
            used |= (row < D * S) & ((row % S) * D + row // S < n)
    return used.view(c["B"], st["pps"], c["page"]).any(2)


def _plain_pages(c, st, table, free, n_free, length, extra=0):
    need = _needed(c, st, length, extra).flatten()
    old = table.flatten().long()
    has = (old >= 0) & (old < st["num_pages"])
    back, take = has & ~need, need & ~has
    stack = torch.cat([free.long(), free.new_zeros(1).long()])  # the last place takes what is not given back
    stack[torch.where(back, n_free + back.cumsum(0) - 1, st["num_pages"])] = torch.where(back, old, 0)
    top = n_free + back.sum()
    at = top - take.cumsum(0)
    new = torch.where(has & need, old, torch.where(take & (at >= 0), stack[at.clamp(min=0)], -1))
    left = (top - take.sum()).clamp(min=0)
    return new.to(torch.int32).view_as(table), stack[:-1].to(torch.int32), left.to(torch.int32)


def _plain_slots(c, st):
    i = torch.arange(c["N"], device=DEV)[None]
    j = st["pos"].long()[:, None] + i
    there, j = i < st["count"][:, None], j.clamp(max=st["cap"] - 1)
    last = (st["pos"] + st["count"]).long()[:, None]
    main, ring = [], []
    for h0, h1, D, W, _ in _kinds(c):
        ok = there & (j % D == D - 1) if c["grid"] else there
        main.append(torch.where(ok[:, :, None], _slot(c, st, h0, h1, _main_row(c, st, D, j)), -1))
        if c["grid"]:
            ok = there & (j >= last - W) if D > 1 and W > 0 else torch.zeros_like(there)
            ring.append(torch.where(ok[:, :, None], _slot(c, st, h0, h1, -(-st["cap"] // D) + j % max(1, W) if W and D > 1 else j * 0), -1))
    return {"slots": torch.cat(main, 2), "ring": torch.cat(ring, 2) if c["grid"] else None}


# ------------------------------------------------------------------ in 64 bits


def _walk(c, st, b, x):
    """Node by node: (branch, state) of entry b's nodes, for x = "k" or "v"; None where a node is absent."""
    g = (st["g"][0 if x == "k" else 1] if c["sep"] else st["g"])[b].double()
    gate = 1 / (1 + torch.exp(-g))
    gate[:, :c["dense"]] = 0
    nodes = []
    for i, p in enumerate(st["parent"][b].tolist()):
        if p == -2:
            nodes.append(None)
            continue
        branch, s = ([], st["state_" + x][b].double()) if p < 0 else nodes[p]
        nodes.append((branch + [i], gate[i] * s + (1 - gate[i]) * st[x][b, i].double()))
    return nodes


def _held_rows(c, st, b, x, h0, h1, D, W):
    """Entry b's rows of positions 0 .. pos - 1 in their order, [heads, pos, d] in 64 bits (zero: not kept)."""
    p, cap, d = int(st["pos"][b]), st["cap"], c["d"]
    j = np.arange(p)
    if not c["grid"] or D == 1:
        row = (j % D) * -(-cap // D) + j // D
    else:
        row = np.where(j % D == D - 1, j // D, np.where((W > 0) & (j >= p - W), -(-cap // D) + j % max(1, W), -1))
    kept = torch.from_numpy(row >= 0).to(DEV)
    row = torch.from_numpy(np.maximum(row, 0)).to(DEV)
    cache = st["cache_" + x]
    if c["page"]:
        rows = cache[st["table"][b].long()[row // c["page"]], :, row % c["page"]][:, h0:h1].transpose(0, 1)
    else:
        rows = cache[b, h0:h1][:, row]
    return rows.double() * kept[None, :, None]


def exact(c, seed):
    if c["op"] in ("pages", "slots"):
        return None  # whole numbers
    st = prepare(c, seed)
    B, N, H, d, dt = c["B"], c["N"], c["H"], c["d"], _dtype(c)
    if c["op"] == "commit":
        out = {"out_pos": None}
        for x in ("k", "v"):
            state, cache = st["state_" + x].double(), st["cache_" + x].double()
            for b in range(B):
                leaf = int(st["leaf"][b])
                nodes = _walk(c, st, b, x)
                for n, i in enumerate(nodes[leaf][0] if leaf >= 0 else []):
                    j = int(st["pos"][b]) + n
                    state[b] = nodes[i][1]
                    for h0, h1, D, W, _ in _kinds(c):
                        S = -(-st["cap"] // D)
                        rows = [(j % D) * S + j // D]
                        if c["grid"]:
                            rows = ([j // D] if j % D == D - 1 else []) + ([S + j % W] if D > 1 and W > 0 else [])
                        for r in rows:
                            if c["page"]:
                                cache[int(st["table"][b, r // c["page"]]), h0:h1, r % c["page"]] = state[b, h0:h1]
                            else:
                                cache[b, h0:h1, r] = state[b, h0:h1]
            out["out_state_" + x], out["cache_" + x] = state, cache
        return out
    o, lse = torch.zeros(B, N, H, d, dtype=torch.float64, device=DEV), torch.full((B, H, N), -math.inf, dtype=torch.float64, device=DEV)
    for b in range(B):
        pos = int(st["pos"][b])
        walks = {x: _walk(c, st, b, x) for x in ("k", "v")}
        live = [i for i in range(N) if walks["k"][i] is not None]
        depth = {i: len(walks["k"][i][0]) - 1 for i in live}
        for h0, h1, D, W, _ in _kinds(c):
            j = np.concatenate([np.arange(pos), [pos + depth[i] for i in live]])
            count = np.zeros((len(live), len(j)))
            for n, i in enumerate(live):
                t = pos + depth[i]
                seen = np.concatenate([np.ones(pos, bool), np.isin(live, walks["k"][i][0])])
                itself = np.concatenate([np.zeros(pos, bool), np.array(live) == i])
                far = (j % D == D - 1) | itself if c["grid"] else (t - j) % D == 0
                near = (j > t - W) & (j <= t)
                count[n] = seen & far
                count[n] += seen & near & ~far if c["dedupe"] else seen & near
            count = torch.from_numpy(count).to(DEV)[None]
            kv = []
            for x in ("k", "v"):
                mine = torch.stack([walks[x][i][1][h0:h1].to(dt).double() for i in live], 1)
                kv.append(torch.cat([_held_rows(c, st, b, x, h0, h1, D, W), mine], 1))
            s = st["q"][b, live, h0:h1].double().transpose(0, 1) @ kv[0].transpose(1, 2) / math.sqrt(d)
            s = torch.where(count > 0, s, -math.inf)
            top = s.amax(2, keepdim=True)
            p = count * torch.exp(s - top)
            total = p.sum(2, keepdim=True)
            o[b, live, h0:h1] = (p @ kv[1] / total).transpose(0, 1)
            lse[b, h0:h1, live] = (top + torch.log(total))[..., 0]
    return {"o": o, "lse": lse}
