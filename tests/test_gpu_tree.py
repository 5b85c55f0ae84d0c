"""Drafted trees over the decode cache on the GPU, against the fp64 CPU oracle.

The reference of a node is the operator itself: its sequence is the held rows followed by its branch, whose
augmented rows are the recurrence in 64 bits rounded to the cache's type, and its output is that sequence's last
row of the oracle's attention.  Bars as elsewhere: max-abs 1e-4 (fp32), relative L2 1e-2 (bf16; half a step of the
output, 2^-9, and of the probabilities in a matrix product, 2^-9, stay well inside).
"""
import numpy as np
import pytest
import torch

import oracle
from parity import assert_close, f64

rat = pytest.importorskip("recurrence_augmented_dilated_gated_b200")

pytestmark = pytest.mark.gpu

DEV = "cuda"
ABSENT = rat.RAT_NODE_ABSENT
BF16, F32 = torch.bfloat16, torch.float32


def config(B, N, H, d, dtype, dil, win, recur=None, grid=False, dedupe=False, sep=False, scale=0.0):
    flags = rat.RAT_FLAG_GRID_DILATION * grid | rat.RAT_FLAG_DEDUPE * dedupe | rat.RAT_FLAG_SEPARATE_GATES * sep
    return rat.Config(B, N, H, d, dtype, dil, win, recur, scale, flags)


def rows_of(cfg, cap, h, j):
    """(main row or -1, ring row or -1) of position j, from the documented layout."""
    D, W = int(cfg.dil[h]), int(cfg.win[h])
    S = -(-cap // D)
    if not cfg.c.flags & rat.RAT_FLAG_GRID_DILATION:
        return (j % D) * S + j // D, -1
    return (j // D if j % D == D - 1 else -1), (S + j % W if D > 1 and W > 0 else -1)


def fill(cfg, cap, hist, pos):
    """A cache [B,H,R,d] holding the rows of positions < pos[b] of hist [B,cap,H,d]; every other row is NaN."""
    c = cfg.c
    R = rat.rat_cache_rows(cfg, cap)
    cache = torch.full((c.B, c.H, R, c.d), float("nan"), dtype=hist.dtype, device=DEV)
    hist = hist.to(DEV)
    for h in range(c.H):
        for b in range(c.B):
            main, ring = {}, {}
            for j in range(pos[b]):
                m, r = rows_of(cfg, cap, h, j)
                if m >= 0:
                    main[m] = j
                if r >= 0:
                    ring[r] = j
            for rows in (main, ring):
                if rows:
                    cache[b, h, list(rows)] = hist[b, list(rows.values()), h]
    return cache


def random_parents(rng, B, N, max_depth, pad=True):
    parent = np.full((B, N), ABSENT, np.int32)
    for b in range(B):
        depth = []
        for i in range(N):
            if pad and b % 2 and i > 0 and rng.random() < 0.15:
                depth.append(None)
                continue
            ups = [-1] + [j for j in range(i) if depth[j] is not None and depth[j] < max_depth - 1]
            parent[b, i] = rng.choice(ups[-6:])
            depth.append(0 if parent[b, i] < 0 else depth[parent[b, i]] + 1)
    return parent


class Problem:
    """Seeded inputs of a tree step, and its reference."""

    def __init__(self, cfg, cap, pos, parent, seed=0, std=0.5):
        c = cfg.c
        self.cfg, self.cap, self.pos, self.parent = cfg, cap, list(pos), parent
        gen = torch.Generator().manual_seed(seed)
        dt = cfg.torch_dtype
        rnd = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
        tok = (c.B, c.T, c.H, c.d)
        self.q, self.k, self.v = (rnd(*tok).to(dt) for _ in range(3))
        self.g = (rnd(*cfg.gate_shape(tok)) + 1.0).to(dt)
        self.sk, self.sv = rnd(c.B, c.H, c.d) * std, rnd(c.B, c.H, c.d) * std
        n = max(max(pos), 1)
        self.hk, self.hv = ((rnd(c.B, n, c.H, c.d) * std).to(dt) for _ in range(2))
        gone = torch.from_numpy(parent == ABSENT)
        for x in (self.q, self.k, self.v):
            x[gone] = float("nan")          # padding may hold anything
        for g in (self.g if c.flags & rat.RAT_FLAG_SEPARATE_GATES else [self.g]):
            g[gone] = float("nan")

    def to_gpu(self):
        self.ck, self.cv = fill(self.cfg, self.cap, self.hk, self.pos), fill(self.cfg, self.cap, self.hv, self.pos)
        for x in ("q", "k", "v", "g", "sk", "sv"):
            setattr(self, "d_" + x, getattr(self, x).to(DEV).contiguous())
        self.d_pos = torch.tensor(self.pos, dtype=torch.int32, device=DEV)
        self.d_parent = torch.from_numpy(np.ascontiguousarray(self.parent)).to(DEV)
        self.ws = rat.workspace(self.cfg, rat.RAT_OP_TREE, self.cap)
        return self

    def outputs(self):
        c = self.cfg.c
        o = torch.full((c.B, c.T, c.H, c.d), 7.0, dtype=self.cfg.torch_dtype, device=DEV)
        return o, torch.full((c.B, c.H, c.T), 7.0, device=DEV)

    def step(self, cache=None, stream=None, check=True):
        o, lse = self.outputs()
        head = (self.cfg, self.d_q, self.d_k, self.d_v, self.d_g, self.d_parent, self.d_sk, self.d_sv)
        tail = (self.cap, self.d_pos, o, lse, self.ws, stream)
        if cache is None:
            rat.rat_tree_decode_step(*head, self.ck, self.cv, *tail)
        else:
            rat.rat_tree_decode_step_paged(*head, cache, *tail)
        if check:
            rat.rat_check_status(self.ws, stream)
        return o, lse

    def states(self, b):
        """[(k, v)] of entry b's nodes in 64 bits ([H, d] each), None for padding."""
        c = self.cfg.c
        sep = c.flags & rat.RAT_FLAG_SEPARATE_GATES
        out = []
        for i, p in enumerate(self.parent[b]):
            if p == ABSENT:
                out.append(None)
                continue
            pair = []
            for x, (src, s0) in enumerate(((self.k, self.sk), (self.v, self.sv))):
                g = f64((self.g[x] if sep else self.g)[b, i])
                a = 1 / (1 + np.exp(-g))
                if self.cfg.recur is not None:
                    a = a * self.cfg.recur[:, None]
                s = f64(s0[b]) if p < 0 else out[p][x]
                pair.append(a * s + (1 - a) * f64(src[b, i]))
            out.append(tuple(pair))
        return out

    def branch(self, b, i):
        out = []
        while i >= 0:
            out.append(i)
            i = self.parent[b, i]
        return out[::-1]

    def reference(self):
        c, dt = self.cfg.c, self.cfg.torch_dtype
        rnd = lambda x: torch.from_numpy(x).to(dt).double().numpy()  # noqa: E731
        o, lse = np.zeros((c.B, c.T, c.H, c.d)), np.full((c.B, c.H, c.T), -np.inf)
        grid, dedupe = bool(c.flags & rat.RAT_FLAG_GRID_DILATION), bool(c.flags & rat.RAT_FLAG_DEDUPE)
        for b in range(c.B):
            states = self.states(b)
            for i in range(c.T):
                if states[i] is None:
                    continue
                br = self.branch(b, i)
                t = self.pos[b] + len(br) - 1
                seq = [np.concatenate([f64(h[b, :self.pos[b]]), np.stack([rnd(states[n][x]) for n in br])])[None]
                       for x, h in enumerate((self.hk, self.hv))]
                q = np.zeros_like(seq[0])
                q[0, t] = f64(self.q[b, i])
                rows = [(0, h, t) for h in range(c.H)]
                scale = c.scale if c.scale > 0 else None
                ro, rl = oracle.attn_rows(q, seq[0], seq[1], self.cfg.dil, self.cfg.win, rows, grid=grid, dedupe=dedupe,
                                          scale=scale)
                o[b, i], lse[b, :, i] = ro, rl
        return o, lse

    def check(self, o, lse):
        ro, rl = self.reference()
        dt = self.cfg.torch_dtype
        there = np.isfinite(rl)
        got = f64(lse)
        assert np.array_equal(np.isneginf(got), ~there)
        assert np.max(np.abs(got[there] - rl[there]), initial=0.0) <= (1e-4 if dt == F32 else 1e-3)
        assert_close(o, ro, dt, "o")
        assert torch.all(o[torch.from_numpy(self.parent == ABSENT).to(DEV)] == 0)


#: (dil, win, recur, N, cap, positions, max depth)
CASES = [
    ([1, 3], [0, 0], None, 1, 40, [0, 7], 1),                    # one node: a decode step; nothing held yet
    ([1, 16], [0, 0], [0, 1], 8, 500, [0, 1, 480], 4),
    ([4, 1], [9, 5], [1, 1], 17, 333, [3, 16, 320], 6),          # windows shorter and longer than the branch
    ([64, 7], [300, 1], [1, 0], 33, 1000, [63, 64, 700], 9),     # W past the start, W = 1; N past a tile
    ([2, 5], [0, 64], [1, 1], 64, 901, [850, 17, 129], 20),      # the largest tree, deep; odd capacity
    ([1, 1], [0, 40], [0, 1], 21, 2000, [1979, 1, 640], 8),      # several pieces of one dense slab
    ([100, 30], [0, 12], [1, 1], 16, 90, [40, 70, 0], 16),       # D past the capacity; depth past W
    ([3, 1], [0, 700], [1, 1], 12, 800, [790, 701, 3], 5),       # a window over several tiles
]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("grid,dedupe,sep", [(0, 0, 0), (1, 0, 1), (0, 1, 0), (1, 1, 0)])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_tree_step_every_node(dtype, d, grid, dedupe, sep, case):
    dil, win, recur, N, cap, pos, deep = CASES[case]
    rng = np.random.default_rng(case)
    cfg = config(len(pos), N, len(dil), d, dtype, dil, win, recur, grid, dedupe, sep)
    p = Problem(cfg, cap, pos, random_parents(rng, len(pos), N, deep), seed=case).to_gpu()
    p.check(*p.step())


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_long_context_in_many_pieces(dtype):
    # one entry: its slabs are cut into several pieces each, and the pieces joined
    cfg = config(1, 20, 2, 128, dtype, [1, 4], [0, 600], [0, 1])
    p = Problem(cfg, 9000, [8970], random_parents(np.random.default_rng(5), 1, 20, 6, pad=False)).to_gpu()
    p.check(*p.step())


#: heads whose nodes all read the same rows, in a cache large enough (2^20 such rows by capacity) for the tcgen05
#: form: (dil, win, grid, N, cap, positions, max depth)
LARGE = [
    ([1, 1], [0, 0], 0, 1, 530000, [1], 1),
    ([1, 4], [0, 30], 0, 8, 600000, [0, 127], 4),
    ([1, 3], [20, 0], 0, 16, 350000, [128, 129, 1], 5),
    ([1, 64], [0, 200], 0, 17, 550000, [2500, 640], 6),
    ([2, 5], [40, 0], 1, 33, 800000, [3001, 255], 9),
    ([1, 1], [0, 7], 0, 64, 300000, [1000, 4700], 12),
]


@pytest.mark.parametrize("case", range(len(LARGE)))
@pytest.mark.parametrize("page_rows", [0, 8, 64, 128, 384, 40])
def test_large_capacities(case, page_rows):
    # dense, in pages that the tcgen05 form copies (parts and multiples of 128 rows) and in others
    dil, win, grid, N, cap, pos, deep = LARGE[case]
    cfg = config(len(pos), N, len(dil), 128, BF16, dil, win, [0] + [1] * (len(dil) - 1), grid)
    p = Problem(cfg, cap, pos, random_parents(np.random.default_rng(case), len(pos), N, deep), seed=case).to_gpu()
    if not page_rows:
        p.check(*p.step())
        return
    _, _, desc = short_pages(cfg, cap, p, page_rows)
    p.check(*p.step(desc))


def short_pages(cfg, cap, p, page_rows):
    """Pages for the rows that the positions held and the tree need only; the table's other entries are -1."""
    c = cfg.c
    R = p.ck.shape[2]
    pps = -(-R // page_rows)
    table = np.full((c.B, pps), -1, np.int32)
    n = 0
    for b in range(c.B):
        used = set()
        for h in range(c.H):
            for j in range(p.pos[b] + c.T):
                used |= {r // page_rows for r in rows_of(cfg, cap, h, j) if r >= 0}
        for i in sorted(used):
            table[b, i] = n
            n += 1
    table[table >= 0] = np.random.default_rng(3).permutation(n)[table[table >= 0]]
    pools = []
    for x in (p.ck, p.cv):
        pool = torch.full((max(n, 1), c.H, page_rows, c.d), float("nan"), dtype=x.dtype, device=DEV)
        for b, i in zip(*np.nonzero(table >= 0)):
            rows = x[b, :, i * page_rows:(i + 1) * page_rows]
            pool[int(table[b, i]), :, :rows.shape[1]] = rows
        pools.append(pool)
    d_table = torch.from_numpy(table).to(DEV)
    return pools, d_table, rat.paged_cache(cfg, pools[0], pools[1], d_table, cap)


@pytest.mark.parametrize("page_rows", [64, 128])
def test_an_invalid_page_of_a_large_capacity(page_rows):
    cfg = config(3, 20, 2, 128, BF16, [1, 8], [0, 12])
    p = Problem(cfg, 400000, [1000, 700, 900], random_parents(np.random.default_rng(4), 3, 20, 5, pad=False)).to_gpu()
    want = p.step()
    _, table, desc = short_pages(cfg, p.cap, p, page_rows)
    got = p.step(desc)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    table[1, 512 // page_rows] = -1            # rows 512 ..: head 0's positions; head 1 has none there (its slab is 50000)
    o, lse = p.step(desc, check=False)
    with pytest.raises(rat.RatError, match="RAT_ERR_INVALID"):
        rat.rat_check_status(p.ws)
    assert torch.all(o[1, :, 0] == 0) and torch.all(torch.isneginf(lse[1, 0]))
    assert torch.equal(o[1, :, 1], want[0][1, :, 1]) and torch.equal(o[[0, 2]], want[0][[0, 2]])
    table[1, 512 // page_rows] = int(table.max()) + 1
    o2, _ = p.step(desc, check=False)
    assert torch.equal(o2, o)
    with pytest.raises(rat.RatError, match="RAT_ERR_INVALID"):
        rat.rat_check_status(p.ws)


def test_scores_that_outgrow_the_first_tile():
    # the references are set by an item's first keys and have to be raised by later ones, in every form of the step:
    # keys grow along the sequence until their scores are hundreds above the first
    for cap, dtype, d in ((600000, BF16, 128), (4000, BF16, 128), (4000, F32, 128), (4000, BF16, 64)):
        cfg = config(2, 24, 1, d, dtype, [1], [0], scale=1.0)
        p = Problem(cfg, cap, [1900, 1030], random_parents(np.random.default_rng(6), 2, 24, 6, pad=False))
        ramp = torch.linspace(0.01, 6.0, p.hk.shape[1])[None, :, None, None]
        p.hk = (p.hk.float() * ramp).to(dtype)
        p.to_gpu()
        p.check(*p.step())


def test_large_step_next_to_another_and_repeated():
    # two steps of the persistent form at once, each with its own workspace, then the same bits again
    cfg = config(2, 40, 2, 128, BF16, [1, 1], [0, 30])
    ps = [Problem(cfg, 280000, [5000, 3333], random_parents(np.random.default_rng(i), 2, 40, 6), seed=i).to_gpu()
          for i in range(2)]
    want = [p.step() for p in ps]
    streams = [torch.cuda.Stream() for _ in ps]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [p.step(stream=s, check=False) for p, s in zip(ps, streams)]
        torch.cuda.synchronize()
        for g, w, p in zip(got, want, ps):
            assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1])
            rat.rat_check_status(p.ws)


def test_custom_scale_and_no_lse():
    cfg = config(2, 9, 2, 64, BF16, [2, 1], [0, 6], scale=0.3)
    p = Problem(cfg, 300, [250, 5], random_parents(np.random.default_rng(1), 2, 9, 4)).to_gpu()
    o, lse = p.step()
    p.check(o, lse)
    o2, _ = p.outputs()
    rat.rat_tree_decode_step(cfg, p.d_q, p.d_k, p.d_v, p.d_g, p.d_parent, p.d_sk, p.d_sv, p.ck, p.cv, p.cap, p.d_pos,
                             o2, None, p.ws)
    rat.rat_check_status(p.ws)
    assert torch.equal(o, o2)


def test_all_nodes_absent_and_capacity_reached():
    # an entry without nodes at a full cache is no error; one node more is
    parent = np.array([[-1, 0, ABSENT], [ABSENT] * 3], np.int32)
    cfg = config(2, 3, 1, 64, F32, [2], [4])
    p = Problem(cfg, 50, [48, 50], parent).to_gpu()
    p.check(*p.step())
    p = Problem(cfg, 50, [49, 50], parent).to_gpu()
    o, lse = p.step(check=False)
    with pytest.raises(rat.RatError, match="RAT_ERR_INVALID"):
        rat.rat_check_status(p.ws)
    assert torch.all(o == 0) and torch.all(torch.isneginf(lse))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("dil,win,grid", [([1], [4], 0), ([3], [0], 0), ([8], [0], 1), ([1], [0], 0)])
def test_entries_without_nodes_among_others(dtype, dil, win, grid):
    # o = 0, lse = -inf for every node of an entry that drafted nothing, in every plan of a head
    parent = np.array([[ABSENT] * 5, [-1, 0, 0, 2, ABSENT], [ABSENT] * 5], np.int32)
    for cap in (60, 4000):
        cfg = config(3, 5, 1, 128, dtype, dil, win, grid=grid)
        p = Problem(cfg, cap, [40, 55, 0], parent).to_gpu()
        p.ws[256:] = 0xab                       # whatever the workspace held
        p.check(*p.step())


@pytest.mark.parametrize("bad", [[-1, 1, 0], [-1, 5, 0], [-3, 0, 0], [ABSENT, 0, -1], [-1, 2, 0]])
@pytest.mark.parametrize("pos", [20])
def test_bad_parents_skip_the_entry(bad, pos):
    parent = np.array([[-1, 0, 1], bad, [-1, -1, 1]], np.int32)
    cfg = config(3, 3, 2, 64, BF16, [1, 4], [0, 3])
    good = Problem(cfg, 64, [pos] * 3, np.array([[-1, 0, 1], [-1, 0, 1], [-1, -1, 1]], np.int32)).to_gpu()
    want = good.step()
    good.d_parent = torch.from_numpy(parent).to(DEV)
    o, lse = good.step(check=False)
    with pytest.raises(rat.RatError, match="RAT_ERR_INVALID"):
        rat.rat_check_status(good.ws)
    rat.rat_check_status(good.ws)      # reading the error cleared it
    for b in (0, 2):
        assert torch.equal(o[b], want[0][b]) and torch.equal(lse[b], want[1][b])
    assert torch.all(o[1] == 0) and torch.all(torch.isneginf(lse[1]))


@pytest.mark.parametrize("pos", [-1, 65, 1 << 30, -(1 << 31), (1 << 31) - 1])
def test_bad_position_skips_the_entry(pos):
    cfg = config(2, 3, 2, 64, BF16, [1, 4], [0, 3])
    p = Problem(cfg, 64, [20, 20], np.array([[-1, 0, 1]] * 2, np.int32)).to_gpu()
    want = p.step()
    p.d_pos = torch.tensor([pos, 20], dtype=torch.int32, device=DEV)
    o, lse = p.step(check=False)
    with pytest.raises(rat.RatError, match="RAT_ERR_INVALID"):
        rat.rat_check_status(p.ws)
    assert torch.all(o[0] == 0) and torch.equal(o[1], want[0][1]) and torch.equal(lse[1], want[1][1])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("where", ["k", "v", "q"])
def test_a_broken_branch_stays_alone(dtype, bad, where):
    # node 2 is not finite: its branch is lost, the others' results do not change by a bit
    parent = np.array([[-1, 0, 0, 1, 2, 3, -1, 6]], np.int32)
    cfg = config(1, 8, 2, 64, dtype, [1, 2], [3, 0])
    p = Problem(cfg, 64, [30], parent).to_gpu()
    want = p.step()
    getattr(p, "d_" + where)[0, 2, :, 5] = bad
    o, lse = p.step()
    clean = [0, 1, 3, 5, 6, 7]
    assert torch.equal(o[:, clean], want[0][:, clean]) and torch.equal(lse[..., clean], want[1][..., clean])
    if (where, bad) != ("k", float("inf")):      # a score of -inf leaves its key out
        assert not torch.isfinite(o[0, 2, 0]).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_a_value_outside_the_window_does_not_reach_a_node(dtype):
    # position 27 is in the window of the root (t = 30, W = 4) and not of its child: not finite, it reaches the root only
    cfg = config(1, 2, 1, 64, dtype, [7], [4])
    p = Problem(cfg, 64, [30], np.array([[-1, 0]], np.int32)).to_gpu()
    want = p.step()
    p.cv[0, 0, rows_of(cfg, 64, 0, 27)[0], 3] = float("inf")
    o, _ = p.step()
    assert torch.equal(o[0, 1], want[0][0, 1]) and not torch.isfinite(o[0, 0]).all()


def paged_copy(cfg, cap, ck, cv, page_rows, seed=0, spare=3, num_pages=None):
    """The dense cache's rows in pages in random order: (pools, table, descriptor)."""
    c = cfg.c
    R = ck.shape[2]
    pps = -(-R // page_rows)
    n = num_pages or c.B * pps + spare
    rng = np.random.default_rng(seed)
    table = rng.choice(n, c.B * pps, replace=False).reshape(c.B, pps).astype(np.int32)
    pools = []
    for x in (ck, cv):
        pool = torch.full((n, c.H, page_rows, c.d), float("nan"), dtype=x.dtype, device=DEV)
        padded = torch.nn.functional.pad(x, (0, 0, 0, pps * page_rows - R))
        pool[torch.from_numpy(table.reshape(-1)).long().to(DEV)] = (
            padded.view(c.B, c.H, pps, page_rows, c.d).transpose(1, 2).reshape(-1, c.H, page_rows, c.d))
        pools.append(pool)
    table = torch.from_numpy(table).to(DEV)
    return pools, table, rat.paged_cache(cfg, pools[0], pools[1], table, cap)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("grid", [0, 1])
@pytest.mark.parametrize("page_rows", [1, 16, 37, 64, 500])
def test_paged_step_equals_dense(dtype, grid, page_rows):
    cfg = config(3, 19, 3, 64, dtype, [1, 4, 16], [0, 20, 33], [0, 1, 1], grid)
    p = Problem(cfg, 420, [400, 1, 77], random_parents(np.random.default_rng(2), 3, 19, 6)).to_gpu()
    want = p.step()
    _, _, desc = paged_copy(cfg, p.cap, p.ck, p.cv, page_rows)
    got = p.step(desc)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("entry", [-1, -7, 10 ** 6])
@pytest.mark.parametrize("part", ["slab", "window"])
def test_an_invalid_page_skips_its_pair(dtype, entry, part):
    # head 0 dense, head 1 with D = 8 and a window: a page that only one part of one head's step touches
    cfg = config(2, 7, 2, 64, dtype, [1, 8], [0, 4])
    p = Problem(cfg, 256, [200, 150], random_parents(np.random.default_rng(2), 2, 7, 3, pad=False)).to_gpu()
    want = p.step()
    _, table, desc = paged_copy(cfg, p.cap, p.ck, p.cv, 8)
    # rows 160..167: head 0's positions there, head 1's residue 5 (slab 32 rows): positions 5 .. 61 of entry 1;
    # entry 1's nodes at 150 .. 152 have residues 6, 7, 0; window positions 147 .. 149 residues 3, 4, 5
    row = {"slab": 6 * 32, "window": 5 * 32 + 149 // 8}[part]
    table[1, row // 8] = entry
    o, lse = p.step(desc, check=False)
    with pytest.raises(rat.RatError, match="RAT_ERR_INVALID"):
        rat.rat_check_status(p.ws)
    assert torch.equal(o[0], want[0][0])
    assert torch.all(o[1, :, 1] == 0) and torch.all(torch.isneginf(lse[1, 1]))
    assert torch.equal(o[1, :, 0], want[0][1, :, 0])     # head 0 holds positions < 150 only: rows below 150


@pytest.mark.parametrize("cap", [128, 140000])
def test_pages_far_into_a_large_pool(cap):
    # element offsets past 2^32 in a pool of 17 GB; two pages of it are used
    cfg = config(1, 5, 8, 128, BF16, [1] * 8, [0] * 8)
    p = Problem(cfg, cap, [120], random_parents(np.random.default_rng(2), 1, 5, 3)).to_gpu()
    want = p.step()
    n = (1 << 32) // (8 * 64 * 128) + 9
    pools = [torch.empty(n, 8, 64, 128, dtype=BF16, device=DEV) for _ in range(2)]
    table = torch.full((1, -(-p.ck.shape[2] // 64)), -1, dtype=torch.int32, device=DEV)
    table[0, 0], table[0, 1] = n - 1, n - 5
    for pool, x in zip(pools, (p.ck, p.cv)):
        for i in range(2):
            pool[int(table[0, i])] = x[0, :, 64 * i:64 * i + 64]
    desc = rat.paged_cache(cfg, pools[0], pools[1], table, p.cap)
    got = p.step(desc)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # and the commit writes there
    leaf = torch.tensor([2], dtype=torch.int32, device=DEV)
    out = [torch.empty_like(p.d_sk) for _ in range(2)]
    out_pos = torch.empty_like(p.d_pos)
    rat.rat_tree_commit_paged(cfg, p.d_k, p.d_v, p.d_g, p.d_parent, leaf, p.d_sk, p.d_sv, *out, desc, p.cap, p.d_pos,
                              out_pos, p.ws)
    rat.rat_check_status(p.ws)
    br = p.branch(0, 2)
    for i in range(len(br)):
        assert_close(pools[0][n - 5, :, 56 + i], p.states(0)[br[i]][0], BF16, "row")


def test_results_repeat_bit_for_bit_and_on_another_stream():
    cfg = config(4, 40, 4, 128, BF16, [1, 16, 4, 1], [0, 64, 0, 30], [0, 1, 1, 1])
    p = Problem(cfg, 3000, [2900, 5, 1500, 800], random_parents(np.random.default_rng(3), 4, 40, 7)).to_gpu()
    want = p.step()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for stream in (None, s, None):
        got = p.step(stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    with torch.cuda.stream(s):
        got = p.step()
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0])


def test_two_steps_at_once_on_their_own_workspaces():
    cfg = config(2, 30, 4, 128, BF16, [1, 8, 1, 8], [0, 16, 0, 0])
    ps = [Problem(cfg, 4000, [3900, 2000], random_parents(np.random.default_rng(i), 2, 30, 6), seed=i).to_gpu()
          for i in range(2)]
    want = [p.step() for p in ps]
    streams = [torch.cuda.Stream() for _ in ps]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [p.step(stream=s, check=False) for p, s in zip(ps, streams)]
        torch.cuda.synchronize()
        for g, w, p in zip(got, want, ps):
            assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1])
            rat.rat_check_status(p.ws)


def commit(p, leaf, ck, cv, in_place=False, desc=None, check=True):
    leaf = torch.tensor(leaf, dtype=torch.int32, device=DEV)
    sk, sv, pos = p.d_sk.clone(), p.d_sv.clone(), p.d_pos.clone()
    ok, ov, op = (sk, sv, pos) if in_place else (torch.full_like(sk, 7), torch.full_like(sv, 7), torch.full_like(pos, 7))
    head = (p.cfg, p.d_k, p.d_v, p.d_g, p.d_parent, leaf, sk, sv, ok, ov)
    if desc is None:
        rat.rat_tree_commit(*head, ck, cv, p.cap, pos, op, p.ws)
    else:
        rat.rat_tree_commit_paged(*head, desc, p.cap, pos, op, p.ws)
    if check:
        rat.rat_check_status(p.ws)
    return ok, ov, op


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("grid,sep", [(0, 0), (1, 1)])
@pytest.mark.parametrize("in_place", [False, True])
def test_commit_appends_the_branch(dtype, d, grid, sep, in_place):
    cfg = config(4, 40, 3, d, dtype, [1, 4, 30], [0, 3, 17], [0, 1, 1], grid, False, sep)
    parent = random_parents(np.random.default_rng(8), 4, 40, 14, pad=False)
    p = Problem(cfg, 200, [150, 0, 29, 186], parent).to_gpu()
    depth = [[len(p.branch(b, i)) for i in range(40)] for b in range(4)]
    leaf = [int(np.argmax(depth[0])), int(np.argmax(depth[1])), -1, 0]
    ck, cv = p.ck.clone(), p.cv.clone()
    ok, ov, op = commit(p, leaf, ck, cv, in_place)
    for b in range(4):
        br = p.branch(b, leaf[b])
        assert int(op[b]) == p.pos[b] + len(br)
        states = p.states(b)
        for x, (out, cache, before, s0) in enumerate(((ok, ck, p.ck, p.d_sk), (ov, cv, p.cv, p.d_sv))):
            if br:
                assert_close(out[b], states[br[-1]][x], F32, "state")
            else:
                assert torch.equal(out[b], s0[b])
            written = {}
            for h in range(3):
                for n, i in enumerate(br):
                    for r in rows_of(cfg, p.cap, h, p.pos[b] + n):
                        if r >= 0:
                            written[h, r] = states[i][x][h]
            for (h, r), row in written.items():
                assert_close(cache[b, h, r], row, dtype, "row")
            same = torch.ones(3, cache.shape[2], dtype=torch.bool, device=DEV)
            for h, r in written:
                same[h, r] = False
            assert torch.equal(cache[b][same].view(torch.int32), before[b][same].view(torch.int32))   # NaNs and all


@pytest.mark.parametrize("leaf", [40, -2, 1 << 30, -(1 << 31)])
def test_commit_of_a_bad_leaf_leaves_the_entry(leaf):
    cfg = config(2, 5, 2, 64, BF16, [1, 4], [0, 3])
    parent = np.array([[-1, 0, 1, ABSENT, 0]] * 2, np.int32)
    p = Problem(cfg, 64, [20, 20], parent).to_gpu()
    for bad in (leaf, 3):          # 3: an absent node
        ck, cv = p.ck.clone(), p.cv.clone()
        ok, ov, op = commit(p, [bad, 2], ck, cv, check=False)
        with pytest.raises(rat.RatError, match="RAT_ERR_INVALID"):
            rat.rat_check_status(p.ws)
        assert op.tolist() == [20, 23]
        assert torch.equal(ok[0], p.d_sk[0]) and torch.equal(ov[0], p.d_sv[0])
        assert torch.equal(ck[0].view(torch.int32), p.ck[0].view(torch.int32))


def test_commit_past_the_capacity_leaves_the_entry():
    cfg = config(1, 3, 1, 64, F32, [4], [0])
    p = Problem(cfg, 30, [28], np.array([[-1, 0, 1]], np.int32)).to_gpu()
    ck, cv = p.ck.clone(), p.cv.clone()
    _, _, op = commit(p, [2], ck, cv, check=False)
    with pytest.raises(rat.RatError, match="RAT_ERR_INVALID"):
        rat.rat_check_status(p.ws)
    assert op.tolist() == [28] and torch.equal(ck.view(torch.int32), p.ck.view(torch.int32))
    _, _, op = commit(p, [1], ck, cv)
    assert op.tolist() == [30]


def test_commit_to_an_invalid_page_leaves_the_whole_entry():
    cfg = config(2, 4, 2, 64, BF16, [1, 4], [0, 0])
    p = Problem(cfg, 64, [20, 20], np.array([[-1, 0, 1, 2]] * 2, np.int32)).to_gpu()
    pools, table, desc = paged_copy(cfg, p.cap, p.ck, p.cv, 4)
    table[1, (3 * 16 + 23 // 4) // 4] = -1      # head 1's row of position 23 only
    before = pools[0].clone()
    ok, _, op = commit(p, [3, 3], None, None, desc=desc, check=False)
    with pytest.raises(rat.RatError, match="RAT_ERR_INVALID"):
        rat.rat_check_status(p.ws)
    assert op.tolist() == [24, 20] and torch.equal(ok[1], p.d_sk[1])
    mine = table[1][table[1] >= 0].long()
    assert torch.equal(pools[0][mine].view(torch.int16), before[mine].view(torch.int16))
    _, _, op = commit(p, [3, 2], None, None, desc=desc)       # without that position the branch fits
    assert op.tolist() == [24, 23]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("grid", [0, 1])
def test_a_chain_is_as_many_decode_steps(dtype, grid):
    # rat_decode_step token by token against one tree step of a chain and its commit
    B, N, H, d, cap = 2, 11, 3, 128, 300
    cfg = config(B, N, H, d, dtype, [1, 4, 16], [0, 5, 40], [0, 1, 1], grid)
    p = Problem(cfg, cap, [250, 3], np.tile(np.arange(-1, N - 1, dtype=np.int32), (B, 1))).to_gpu()
    o, lse = p.step()
    ck, cv = p.ck.clone(), p.cv.clone()
    ok, ov, op = commit(p, [N - 1] * B, ck, cv)
    dk, dv, sk, sv, pos = p.ck.clone(), p.cv.clone(), p.d_sk.clone(), p.d_sv.clone(), p.d_pos.clone()
    ws = rat.workspace(cfg, rat.RAT_OP_DECODE, cap)
    o1, l1 = torch.empty(B, H, d, dtype=dtype, device=DEV), torch.empty(B, H, device=DEV)
    for n in range(N):
        tok = [x[:, n].contiguous() for x in (p.d_q, p.d_k, p.d_v, p.d_g)]
        rat.rat_decode_step(cfg, *tok, sk, sv, dk, dv, cap, pos, o1, l1, ws)
        rat.rat_check_status(ws)
        assert_close(o[:, n], f64(o1), dtype, "o of node %d" % n)
        assert np.max(np.abs(f64(lse[:, :, n]) - f64(l1))) <= 1e-3
        pos += 1
    assert torch.equal(pos, op)
    assert_close(ok, f64(sk), F32, "state_k")
    assert_close(ov, f64(sv), F32, "state_v")
    there = torch.isfinite(dk.float())
    assert torch.equal(there, torch.isfinite(ck.float()))
    assert_close(ck[there], f64(dk[there]), dtype, "cache_k")
    assert_close(cv[there], f64(dv[there]), dtype, "cache_v")


def test_step_and_commit_replay_from_one_graph():
    # a captured round (step, commit in place) is replayed with new tokens, parents and leaves
    B, N, H, d, cap = 2, 6, 2, 64, 200
    cfg = config(B, N, H, d, BF16, [1, 4], [0, 9])
    rng = np.random.default_rng(4)
    p = Problem(cfg, cap, [40, 9], random_parents(rng, B, N, 4, pad=False)).to_gpu()
    o, lse = p.outputs()
    leaf = torch.zeros(B, dtype=torch.int32, device=DEV)
    ck, cv, sk, sv, pos = p.ck.clone(), p.cv.clone(), p.d_sk.clone(), p.d_sv.clone(), p.d_pos.clone()

    def turn():
        rat.rat_tree_decode_step(cfg, p.d_q, p.d_k, p.d_v, p.d_g, p.d_parent, sk, sv, ck, cv, cap, pos, o, lse, p.ws)
        rat.rat_tree_commit(cfg, p.d_k, p.d_v, p.d_g, p.d_parent, leaf, sk, sv, sk, sv, ck, cv, cap, pos, pos, p.ws)

    before = [x.clone() for x in (ck, cv, sk, sv, pos)]
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        turn()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        turn()
    for x, y in zip((ck, cv, sk, sv, pos), before):
        x.copy_(y)
    eager = [x.clone() for x in before]
    for turn_no in range(4):
        q = Problem(cfg, cap, [1, 1], random_parents(rng, B, N, 4, pad=False), seed=50 + turn_no)
        for x in ("q", "k", "v", "g"):
            getattr(p, "d_" + x).copy_(getattr(q, x))
        p.d_parent.copy_(torch.from_numpy(q.parent))
        leaf.copy_(torch.from_numpy(rng.integers(-1, N, B).astype(np.int32)))
        o2, l2 = p.outputs()
        rat.rat_tree_decode_step(cfg, p.d_q, p.d_k, p.d_v, p.d_g, p.d_parent, eager[2], eager[3], eager[0], eager[1],
                                 cap, eager[4], o2, l2, p.ws)
        rat.rat_tree_commit(cfg, p.d_k, p.d_v, p.d_g, p.d_parent, leaf, eager[2], eager[3], eager[2], eager[3],
                            eager[0], eager[1], cap, eager[4], eager[4], p.ws)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        rat.rat_check_status(p.ws)
        assert torch.equal(o, o2) and torch.equal(lse, l2) and torch.equal(pos, eager[4])
        assert torch.equal(sk, eager[2]) and torch.equal(ck.view(torch.int16), eager[0].view(torch.int16))
    del graph


def test_large_step_replays_from_a_graph():
    # the persistent form, the items form and the join, launched early one after the other, as one captured step
    cfg = config(2, 20, 3, 128, BF16, [1, 1, 8], [0, 30, 12])
    p = Problem(cfg, 280000, [3000, 900], random_parents(np.random.default_rng(1), 2, 20, 6, pad=False)).to_gpu()
    o, lse = p.outputs()
    args = (cfg, p.d_q, p.d_k, p.d_v, p.d_g, p.d_parent, p.d_sk, p.d_sv, p.ck, p.cv, p.cap, p.d_pos, o, lse, p.ws)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        rat.rat_tree_decode_step(*args)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        rat.rat_tree_decode_step(*args)
    for turn in range(3):
        p.d_pos.copy_(torch.tensor([3000 - 700 * turn, 900 - 128 * turn], dtype=torch.int32))
        p.d_parent.copy_(torch.from_numpy(random_parents(np.random.default_rng(9 + turn), 2, 20, 4 + turn)))
        want = p.step()
        o.fill_(7)
        for _ in range(3):
            graph.replay()
        torch.cuda.synchronize()
        rat.rat_check_status(p.ws)
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    del graph


# ------------------------------------------------------------------ page tables


def needed_pages(cfg, cap, page_rows, pps, n):
    """The set of pages in which some head keeps one of positions 0 .. n-1, position by position."""
    out = set()
    for h in range(cfg.c.H):
        for j in range(n):
            out |= {r // page_rows for r in rows_of(cfg, cap, h, j) if r >= 0}
    return out


def python_update(cfg, table, page_rows, num_pages, cap, length, extra, free, n_free):
    table, stack = [list(r) for r in table], list(free[:n_free])
    rest = list(free[n_free:])
    need = []
    for b, n in enumerate(length):
        if n > cap:
            need.append({i for i, e in enumerate(table[b]) if 0 <= e < num_pages})
        else:
            need.append(needed_pages(cfg, cap, page_rows, len(table[b]), min(n + extra, cap) if n >= 0 else 0))
    for b, row in enumerate(table):
        for i, e in enumerate(row):
            if not 0 <= e < num_pages:
                row[i] = -1
            elif i not in need[b]:
                stack.append(e)
                row[i] = -1
    short = False
    for b, row in enumerate(table):
        for i in range(len(row)):
            if i in need[b] and row[i] < 0:
                short |= not stack
                row[i] = stack.pop() if stack else -1
    return table, stack, short


PAGE_CASES = [
    # (B, dil, win, grid, cap, page_rows)
    (3, [1], [0], 0, 100, 16),
    (5, [16, 1], [0, 0], 0, 333, 16),
    (4, [7, 3], [0, 5], 0, 120, 37),         # pages across slabs
    (4, [64], [0], 0, 200, 8),
    (3, [100], [0], 0, 64, 3),               # D past the capacity: slabs of one row
    (5, [16, 4], [20, 9], 1, 300, 8),
    (4, [8, 1], [300, 0], 1, 200, 16),       # a ring longer than the sequence
    (70, [4], [6], 1, 90, 4),
    (2, [5], [0], 0, 50, 1000),              # one page holds everything
]


@pytest.mark.parametrize("case", range(len(PAGE_CASES)))
def test_page_table_update(case):
    B, dil, win, grid, cap, P = PAGE_CASES[case]
    cfg = config(B, 1, len(dil), 64, BF16, dil, win, grid=grid)
    R = rat.rat_cache_rows(cfg, cap)
    pps = -(-R // P) + case % 2
    num = B * pps + 5
    rng = np.random.default_rng(case)
    free = rng.permutation(num).astype(np.int32)
    table = np.full((B, pps), -1, np.int32)
    table[0, 0] = num + 3                      # names no page, whatever the table held before
    d_table, d_free = torch.from_numpy(table).to(DEV), torch.from_numpy(free).to(DEV)
    d_n = torch.tensor([num], dtype=torch.int32, device=DEV)
    ws = rat.workspace(cfg, rat.RAT_OP_STATUS)
    n_free = num
    for step in range(6):
        length = rng.integers(-1, cap + 1, B).astype(np.int32)
        if step == 0:
            length[:] = rng.integers(0, 3, B)
        if step == 4:
            length[:] = cap                    # all full
        if step == 5:
            length[:] = -1                     # all gone
        extra = int(rng.integers(0, 9))
        want, stack, short = python_update(cfg, d_table.cpu().numpy(), P, num, cap, length.tolist(), extra,
                                           d_free.cpu().numpy().tolist(), n_free)
        assert not short
        rat.rat_page_table_update(cfg, d_table, P, num, cap, torch.from_numpy(length).to(DEV), extra, d_free, d_n, ws)
        rat.rat_check_status(ws)
        assert d_table.cpu().tolist() == want
        n_free = int(d_n)
        assert n_free == len(stack) and d_free[:n_free].cpu().tolist() == stack
        held = d_table[d_table >= 0].tolist()
        assert sorted(held + stack) == list(range(num))       # no page lost, none twice
    assert n_free == num


def test_page_table_runs_out_of_pages():
    cfg = config(3, 1, 1, 64, BF16, [1], [0])
    cap, P, num = 64, 8, 12
    free = torch.arange(num, dtype=torch.int32, device=DEV)
    n = torch.tensor([10], dtype=torch.int32, device=DEV)
    table = torch.full((3, 8), -1, dtype=torch.int32, device=DEV)
    ws = rat.workspace(cfg, rat.RAT_OP_STATUS)
    length = torch.tensor([30, 60, 20], dtype=torch.int32, device=DEV)
    rat.rat_page_table_update(cfg, table, P, num, cap, length, 2, free, n, ws)
    with pytest.raises(rat.RatError, match="RAT_ERR_NO_PAGES"):
        rat.rat_check_status(ws)
    assert int(n) == 0
    assert table.tolist() == [[9, 8, 7, 6] + [-1] * 4, [5, 4, 3, 2, 1, 0, -1, -1], [-1] * 8]
    length[0] = -1                             # the first ends: its pages go to the others
    rat.rat_page_table_update(cfg, table, P, num, cap, length, 2, free, n, ws)
    with pytest.raises(rat.RatError, match="RAT_ERR_NO_PAGES"):
        rat.rat_check_status(ws)
    assert table.tolist() == [[-1] * 8, [5, 4, 3, 2, 1, 0, 6, 7], [8, 9, -1] + [-1] * 5]


def test_page_table_bad_lengths_and_stacks():
    cfg = config(2, 1, 1, 64, BF16, [1], [0])
    ws = rat.workspace(cfg, rat.RAT_OP_STATUS)
    table = torch.tensor([[3, -1, -1], [0, 1, -1]], dtype=torch.int32, device=DEV)
    free = torch.tensor([2, 4, 5, 9, 9, 9], dtype=torch.int32, device=DEV)
    n = torch.tensor([3], dtype=torch.int32, device=DEV)
    args = lambda t, f, k: (cfg, t, 8, 6, 24, length, 0, f, k, ws)  # noqa: E731
    length = torch.tensor([25, 24], dtype=torch.int32, device=DEV)       # past the capacity: left as it is
    rat.rat_page_table_update(*args(table, free, n))
    with pytest.raises(rat.RatError, match="RAT_ERR_INVALID"):
        rat.rat_check_status(ws)
    assert table.tolist() == [[3, -1, -1], [0, 1, 5]] and int(n) == 2
    for bad in (-1, 7, 5):                     # negative, more than there are, more than fit with what comes back
        length = torch.tensor([-1, -1], dtype=torch.int32, device=DEV)
        t, f, k = table.clone(), free.clone(), torch.tensor([bad], dtype=torch.int32, device=DEV)
        rat.rat_page_table_update(*args(t, f, k))
        with pytest.raises(rat.RatError, match="RAT_ERR_INVALID"):
            rat.rat_check_status(ws)
        assert torch.equal(t, table) and torch.equal(f, free) and int(k) == bad
    # a stack entry that is no page is not handed out
    length = torch.tensor([24, 24], dtype=torch.int32, device=DEV)
    f, k = torch.tensor([2, 77, 5, 9, 9, 9], dtype=torch.int32, device=DEV), torch.tensor([2], dtype=torch.int32, device=DEV)
    rat.rat_page_table_update(*args(table, f, k))
    with pytest.raises(rat.RatError, match="RAT_ERR_INVALID"):
        rat.rat_check_status(ws)
    assert table.tolist() == [[3, -1, 2], [0, 1, 5]] and int(k) == 0


# ------------------------------------------------------------------ slot maps


@pytest.mark.parametrize("grid", [0, 1])
@pytest.mark.parametrize("paged", [0, 1])
def test_slot_map(grid, paged):
    B, T, H, d, cap, P = 4, 23, 3, 64, 150, 16
    cfg = config(B, T, H, d, BF16, [1, 4, 16], [5, 9, 40], grid=grid)
    R = rat.rat_cache_rows(cfg, cap)
    pps = -(-R // P)
    pos, count = [0, 100, 127, 149], [23, 0, 23, 1]
    desc, table = None, None
    if paged:
        table = torch.randperm(B * pps + 2)[:B * pps].view(B, pps).to(torch.int32).to(DEV)
        table[2, 3] = -1
        pool = torch.empty(B * pps + 2, H, P, d, dtype=BF16, device=DEV)
        desc = rat.paged_cache(cfg, pool, pool, table, cap)
    ws = rat.workspace(cfg, rat.RAT_OP_STATUS)
    slots = torch.full((B, T, H), 7, dtype=torch.int64, device=DEV)
    ring = torch.full_like(slots, 7)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    rat.rat_slot_map(cfg, desc, cap, i32(pos), i32(count), slots, ring, ws)
    rat.rat_check_status(ws)

    def slot(b, h, row):
        if row < 0:
            return -1
        if not paged:
            return (b * H + h) * R + row
        page = int(table[b, row // P])
        return -1 if page < 0 else (page * H + h) * P + row % P

    want = np.full((2, B, T, H), -1, np.int64)
    for b in range(B):
        for i in range(count[b]):
            for h in range(H):
                m, r = rows_of(cfg, cap, h, pos[b] + i)
                want[0, b, i, h] = slot(b, h, m)
                want[1, b, i, h] = slot(b, h, r) if i >= count[b] - cfg.win[h] else -1
    assert np.array_equal(slots.cpu().numpy(), want[0]) and np.array_equal(ring.cpu().numpy(), want[1])
    # no ring asked for, and no counts: T positions everywhere, which entry 3 has not
    rat.rat_slot_map(cfg, desc, cap, i32([0, 100, 127, 140]), None, slots, None, ws)
    with pytest.raises(rat.RatError, match="RAT_ERR_INVALID"):
        rat.rat_check_status(ws)
    assert torch.all(slots[3] == -1) and slots[0].cpu().tolist() == want[0, 0].tolist()


@pytest.mark.parametrize("H", [4, 70, 131, 256])
@pytest.mark.parametrize("grid", [0, 1])
def test_slot_map_of_many_layouts(H, grid):
    # a layout of its own for every head, more of them than are handled at a time
    T, cap = 37, 500
    cfg = config(1, T, H, 64, BF16, list(range(1, H + 1)), [(7 * h) % 20 for h in range(H)], grid=grid)
    R = rat.rat_cache_rows(cfg, cap)
    ws = rat.workspace(cfg, rat.RAT_OP_STATUS)
    slots = torch.full((1, T, H), 7, dtype=torch.int64, device=DEV)
    ring = torch.full_like(slots, 7)
    i32 = lambda x: torch.tensor([x], dtype=torch.int32, device=DEV)  # noqa: E731
    rat.rat_slot_map(cfg, None, cap, i32(450), i32(30), slots, ring, ws)
    rat.rat_check_status(ws)
    want = np.full((2, T, H), -1, np.int64)
    for i in range(30):
        for h in range(H):
            m, r = rows_of(cfg, cap, h, 450 + i)
            want[0, i, h] = h * R + m if m >= 0 else -1
            want[1, i, h] = h * R + r if r >= 0 and i >= 30 - cfg.win[h] else -1
    assert np.array_equal(slots[0].cpu().numpy(), want[0]) and np.array_equal(ring[0].cpu().numpy(), want[1])


def test_page_table_update_of_a_large_table():
    # more entries than a lane keeps in registers: 300 sequences of 1250 pages, then other lengths
    B, cap, P = 300, 20000, 16
    cfg = config(B, 1, 2, 64, BF16, [1, 3], [0, 0])
    pps = -(-rat.rat_cache_rows(cfg, cap) // P)
    num = 200000
    gen = torch.Generator().manual_seed(1)
    free = torch.randperm(num, generator=gen).to(torch.int32)
    table = torch.full((B, pps), -1, dtype=torch.int32, device=DEV)
    d_free, d_n = free.to(DEV), torch.tensor([num], dtype=torch.int32, device=DEV)
    ws = rat.workspace(cfg, rat.RAT_OP_STATUS)
    stack = free.tolist()
    have = np.full((B, pps), -1, np.int64)
    S = -(-cap // 3)
    row = np.arange(pps * P)
    for step in range(3):
        length = torch.randint(-2000, 9000, (B,), generator=gen).to(torch.int32)
        rat.rat_page_table_update(cfg, table, P, num, cap, length.to(DEV), 5, d_free, d_n, ws)
        rat.rat_check_status(ws)
        n = np.where(length.numpy() >= 0, length.numpy() + 5, 0)[:, None]
        used = (row[None] < n) | ((row[None] < 3 * S) & ((row[None] % S) * 3 + row[None] // S < n))
        need = used.reshape(B, pps, P).any(2)
        for b, i in zip(*np.nonzero((have >= 0) & ~need)):
            stack.append(int(have[b, i]))
            have[b, i] = -1
        for b, i in zip(*np.nonzero(need & (have < 0))):
            have[b, i] = stack.pop()
        assert np.array_equal(table.cpu().numpy(), have)
        assert int(d_n) == len(stack) and d_free[:len(stack)].cpu().tolist() == stack


@pytest.mark.parametrize("pos,count", [(-1, 3), (0, -1), (0, 6), (10, 5), (1 << 30, 1), ((1 << 31) - 1, 5)])
def test_slot_map_of_a_bad_range(pos, count):
    cfg = config(1, 5, 1, 64, BF16, [2], [0])
    ws = rat.workspace(cfg, rat.RAT_OP_STATUS)
    slots = torch.full((1, 5, 1), 7, dtype=torch.int64, device=DEV)
    t = lambda x: torch.tensor([x], dtype=torch.int32, device=DEV)  # noqa: E731
    rat.rat_slot_map(cfg, None, 12, t(pos), t(count), slots, None, ws)
    with pytest.raises(rat.RatError, match="RAT_ERR_INVALID"):
        rat.rat_check_status(ws)
    assert torch.all(slots == -1)


# ------------------------------------------------------------------ together


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("grid", [0, 1])
def test_speculative_serving_loop(dtype, grid):
    # Sequences of different lengths in pages, from empty: every turn the table grows with the drafted tokens, a tree
    # is scored and a branch committed, rows are found through the slot map; one sequence ends and another takes its
    # place.  Against plain decode steps over a dense cache of the accepted tokens.
    B, N, H, d, cap, P = 3, 7, 3, 64, 120, 8
    dil, win, recur = [1, 4, 8], [0, 5, 12], [0, 1, 1]
    cfg = config(B, N, H, d, dtype, dil, win, recur, grid)
    one = config(1, 1, H, d, dtype, dil, win, recur, grid)
    R = rat.rat_cache_rows(cfg, cap)
    pps = -(-R // P)
    num = B * pps
    rng = np.random.default_rng(11)
    pools = [torch.full((num, H, P, d), float("nan"), dtype=dtype, device=DEV) for _ in range(2)]
    table = torch.full((B, pps), -1, dtype=torch.int32, device=DEV)
    free = torch.from_numpy(rng.permutation(num).astype(np.int32)).to(DEV)
    n_free = torch.tensor([num], dtype=torch.int32, device=DEV)
    desc = rat.paged_cache(cfg, pools[0], pools[1], table, cap)
    sk, sv = torch.zeros(B, H, d, device=DEV), torch.zeros(B, H, d, device=DEV)
    pos = torch.zeros(B, dtype=torch.int32, device=DEV)
    ws = rat.workspace(cfg, rat.RAT_OP_TREE, cap)
    # the plain side, one entry at a time
    wsd = rat.workspace(one, rat.RAT_OP_DECODE, cap)
    dense = [[torch.zeros(1, H, R, d, dtype=dtype, device=DEV) for _ in range(2)] for _ in range(B)]
    state = [[torch.zeros(1, H, d, device=DEV) for _ in range(2)] for _ in range(B)]
    plen = [0] * B
    for turn in range(14):
        if turn == 9:                      # entry 1 ends; a new sequence starts there
            pos[1] = 0
            sk[1], sv[1] = 0, 0
            length = pos.clone()
            length[1] = -1
            rat.rat_page_table_update(cfg, table, P, num, cap, length, 0, free, n_free, ws)
            rat.rat_check_status(ws)
            assert torch.all(table[1] == -1)
            plen[1] = 0
            for x in state[1]:
                x.zero_()
        rat.rat_page_table_update(cfg, table, P, num, cap, pos, N, free, n_free, ws)
        p = Problem(cfg, cap, [1] * B, random_parents(rng, B, N, 5, pad=turn % 2 == 1), seed=100 + turn)
        gpu = [x.to(DEV) for x in (p.q, p.k, p.v, p.g)]
        parent = torch.from_numpy(p.parent).to(DEV)
        o, lse = p.outputs()
        rat.rat_tree_decode_step_paged(cfg, *gpu, parent, sk, sv, desc, cap, pos, o, lse, ws)
        leaf = [int(rng.choice(np.flatnonzero(p.parent[b] != ABSENT))) if (turn + b) % 5 else -1 for b in range(B)]
        start = pos.clone()
        rat.rat_tree_commit_paged(cfg, *gpu[1:], parent, torch.tensor(leaf, dtype=torch.int32, device=DEV), sk, sv, sk,
                                  sv, desc, cap, pos, pos, ws)
        slots = torch.empty(B, N, H, dtype=torch.int64, device=DEV)
        rat.rat_slot_map(cfg, desc, cap, start, pos - start, slots, None, ws)
        rat.rat_check_status(ws)
        for b in range(B):
            for n, i in enumerate(p.branch(b, leaf[b])):
                tok = [x[b:b + 1, i].contiguous() for x in gpu]
                o1, l1 = torch.empty(1, H, d, dtype=dtype, device=DEV), torch.empty(1, H, device=DEV)
                at = torch.tensor([plen[b]], dtype=torch.int32, device=DEV)
                rat.rat_decode_step(one, *tok, *state[b], *dense[b], cap, at, o1, l1, wsd)
                rat.rat_check_status(wsd)
                assert_close(o[b, i], f64(o1[0]), dtype, "o, turn %d entry %d node %d" % (turn, b, i))
                for h in range(H):
                    m, _ = rows_of(cfg, cap, h, plen[b])
                    if m >= 0:
                        got = pools[0].view(-1, d)[slots[b, n, h]]
                        assert_close(got, f64(dense[b][0][0, h, m]), dtype, "row through the slot map")
                    else:
                        assert int(slots[b, n, h]) == -1
                plen[b] += 1
        assert pos.tolist() == plen
        for x, s in enumerate((sk, sv)):
            assert_close(s, np.concatenate([f64(state[b][x]) for b in range(B)]), F32, "state")


def test_binding_names_the_argument_that_does_not_fit():
    cfg = config(2, 4, 2, 64, BF16, [1, 4], [0, 0])
    p = Problem(cfg, 64, [20, 20], np.array([[-1, 0, 1, 2]] * 2, np.int32)).to_gpu()
    o, lse = p.outputs()
    args = dict(q=p.d_q, k=p.d_k, v=p.d_v, g=p.d_g, parent=p.d_parent, state_k=p.d_sk, state_v=p.d_sv, cache_k=p.ck,
                cache_v=p.cv, cache_cap=p.cap, pos=p.d_pos, o=o, lse=lse, ws=p.ws)
    wrong = {"dtype": lambda t: t.double(), "shape": lambda t: t[:1].contiguous(), "CUDA": lambda t: t.cpu(),
             "contiguous": lambda t: torch.cat([t, t], -1)[..., ::2]}
    for name in ("q", "g", "parent", "state_v", "cache_k", "pos", "o", "lse"):
        for word, make in wrong.items():
            with pytest.raises(ValueError, match=name + ".*" + word):
                rat.rat_tree_decode_step(cfg, **dict(args, **{name: make(args[name])}))
        if name != "lse":
            with pytest.raises(ValueError, match=name):
                rat.rat_tree_decode_step(cfg, **dict(args, **{name: None}))
    for ws in (None, p.ws.cpu()):
        with pytest.raises(ValueError, match="ws"):
            rat.rat_tree_decode_step(cfg, **dict(args, ws=ws))
    with pytest.raises(TypeError, match="q"):
        rat.rat_tree_decode_step(cfg, **dict(args, q=[1.0]))
    # a capacity of another layout asks for caches of its own shape
    with pytest.raises(ValueError, match="cache_k.*shape"):
        rat.rat_tree_decode_step(cfg, **dict(args, cache_cap=p.cap + 4))
    # a tensor class of its own, and a view of the right shape, are what they hold
    want, _ = p.step()
    rat.rat_tree_decode_step(cfg, **dict(args, q=torch.nn.Parameter(p.d_q, requires_grad=False), k=p.d_k.view(8, 2, 64).view(2, 4, 2, 64)))
    rat.rat_check_status(p.ws)
    assert torch.equal(o, want)


def test_a_configuration_changed_in_place_is_seen():
    cfg = config(1, 2, 2, 64, F32, [1, 4], [0, 0])
    p = Problem(cfg, 62, [20], np.array([[-1, 0]], np.int32)).to_gpu()
    p.step()
    cfg.dil[1] = 3                              # 62 rows become 63, 64 become 63
    with pytest.raises(ValueError, match="cache_k.*shape"):
        p.step()


def ragged(B, top, rng, idle=0.5):
    """Positions of a server's batch: idle entries, short ones, one long."""
    pos = np.where(rng.random(B) < idle, 0, rng.integers(1, 200, B))
    pos[B // 3] = top
    return [int(x) for x in pos]


def test_even_shares_of_a_ragged_batch():
    # more entries than a CTA has threads, runs of idle ones, CTAs with parts of one long entry and with many short ones
    rng = np.random.default_rng(11)
    B, N, cap = 210, 3, 5200
    cfg = config(B, N, 1, 128, BF16, [1], [0])
    pos = ragged(B, 2500, rng)
    pos[100:140] = [0] * 40
    p = Problem(cfg, cap, pos, random_parents(rng, B, N, 2)).to_gpu()
    want = p.step()
    p.check(*want)
    # entries whose position is out of range are left out, the others keep their results
    bad = [5, 70, 209]
    for b, x in zip(bad, (-1, cap + 1, (1 << 31) - 1)):
        p.d_pos[b] = x
    o, lse = p.step(check=False)
    with pytest.raises(rat.RatError, match="RAT_ERR_INVALID"):
        rat.rat_check_status(p.ws)
    rest = [b for b in range(B) if b not in bad]
    assert torch.all(o[bad] == 0) and torch.all(torch.isneginf(lse[bad]))
    assert (o[rest].float() - want[0][rest].float()).abs().max() <= 2 ** -6     # other shares: other partial sums
    # nothing held anywhere: no CTA has a tile
    p = Problem(cfg, cap, [0] * B, random_parents(rng, B, N, 2)).to_gpu()
    p.check(*p.step())


@pytest.mark.parametrize("page_rows", [0, 64])
@pytest.mark.parametrize("N", [3, 20])
def test_many_pairs_by_pieces(page_rows, N):
    rng = np.random.default_rng(12)
    B, cap = 30, 2400
    cfg = config(B, N, 16, 128, BF16, [1] * 16, [0, 9] * 8)
    p = Problem(cfg, cap, ragged(B, 1500, rng, 0.2), random_parents(rng, B, N, 3)).to_gpu()
    if page_rows:
        _, _, desc = short_pages(cfg, cap, p, page_rows)
        p.check(*p.step(desc))
    else:
        p.check(*p.step())


def test_a_head_without_recurrence_keeps_a_branch_apart():
    # a = 0: a child of a node with infinities has its own row only, in the step as in the commit
    for dtype in (F32, BF16):
        cfg = config(1, 4, 1, 128, dtype, [1], [0], [0])
        p = Problem(cfg, 64, [9], np.array([[-1, 0, 1, -1]], np.int32))
        p.k[0, 0], p.v[0, 0] = float("inf"), float("nan")
        p.to_gpu()
        o, _ = p.step()
        assert torch.isfinite(o[0, 3]).all() and torch.isnan(o[0, :3].float()).all()
        ck, cv = p.ck.clone(), p.cv.clone()
        commit(p, [2], ck, cv)
        assert torch.equal(ck[0, 0, 10:12], p.d_k[0, 1:3, 0]) and torch.equal(cv[0, 0, 10:12], p.d_v[0, 1:3, 0])
