"""Drafted trees on the GPU: infinities in held rows and in tokens, expired waits, table entries that are left alone."""
import numpy as np
import pytest
import torch

from parity import f64
from test_gpu_tree import BF16, DEV, F32, Problem, commit, config, random_parents

rat = pytest.importorskip("recurrence_augmented_dilated_gated_b200")

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N", [4, 20, 40])
def test_runs_that_begin_with_keys_left_out(N):
    # The persistent form deals whole tiles of 128 rows out, three or four to a CTA here.  Three tiles of every four
    # hold keys that every node scores -inf, so most runs begin with one; the other held rows and the nodes score
    # about -300: weights that vanish beside a reference of 0, and are all there is.
    parent = random_parents(np.random.default_rng(N), 1, N, 4, pad=False)
    cfg = config(1, N, 1, 128, BF16, [1], [0], [0], scale=1.0)
    p = Problem(cfg, 800000, [60000], parent, std=0.3)
    p.q[..., 0], p.k[..., 0], p.hk[..., 0] = 1.0, -300.0, -300.0
    p.q[..., 5] = p.q[..., 5].abs() + 0.5
    p.hk[:, torch.arange(60000) // 128 % 4 != 3, :, 5] = -float("inf")
    p.to_gpu()
    p.check(*p.step())


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("D,W,N", [(1, 0, 3), (1, 0, 20), (1, 0, 40), (3, 9, 20), (4, 0, 40)])
def test_infinities_in_held_rows(dtype, d, D, W, N):
    # a key that scores -inf drops out; a value that is infinite reaches the nodes that see its row, in its channel
    # and with its sign, and nothing else
    parent = random_parents(np.random.default_rng(N), 2, N, 4, pad=False)
    cfg = config(2, N, 1, d, dtype, [D], [W], scale=0.2)
    p = Problem(cfg, 400, [300, 41], parent)
    p.q[..., 5] = p.q[..., 5].abs() + 0.5
    p.hk[0, 150:160, 0, 5] = -float("inf")
    p.hk[1, 30:35, 0, 5] = -float("inf")
    p.hv[0, 20, 0, 7], p.hv[0, 296, 0, 9], p.hv[1, 40, 0, 11] = float("inf"), -float("inf"), float("inf")
    p.to_gpu()
    o, lse = p.step()
    ro, rl = p.reference()
    got = f64(o)
    assert np.array_equal(np.isnan(got), np.isnan(ro)) and not np.isnan(ro).any()
    hit = np.isinf(ro)
    assert hit.any() and np.array_equal(got[~np.isfinite(got)], ro[hit]) and np.array_equal(np.isinf(got), hit)
    off = got[~hit] - ro[~hit]
    assert np.abs(f64(lse) - rl).max() <= (1e-4 if dtype == F32 else 1e-3)
    if dtype == F32:
        assert np.abs(off).max() <= 1e-4
    else:
        assert np.linalg.norm(off) <= 1e-2 * np.linalg.norm(ro[~hit])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("sep", [0, 1])
def test_an_infinite_token_behind_a_saturated_gate(dtype, d, sep):
    # logits beyond +-80 saturate, 1 - a included: an infinite value times it is infinite, in the step as in the commit
    for g in (100.0, 1000.0, float("inf")):
        cfg = config(1, 2, 1, d, dtype, [1], [0], sep=sep)
        p = Problem(cfg, 64, [9], np.array([[-1, 0]], np.int32))
        (p.g[1] if sep else p.g)[0, 0], p.v[0, 0, 0, 3], p.v[0, 0, 0, 4] = g, float("inf"), -float("inf")
        p.to_gpu()
        o, _ = p.step()
        _, state, _ = commit(p, [1], p.ck, p.cv)
        want = torch.zeros(d, device=DEV)
        want[3], want[4] = float("inf"), -float("inf")
        for x in (o[0, 0, 0].float(), o[0, 1, 0].float(), state[0, 0]):
            assert torch.equal(torch.where(torch.isfinite(x), torch.zeros_like(x), x), want)


@pytest.mark.parametrize("dtype,d,D,N,cap,pos,ticket", [
    (BF16, 128, 1, 4, 800000, [2000], 0),          # the persistent form: one tile a CTA, its copies all asked for
    (BF16, 128, 1, 20, 800000, [60000], 3),        # several tiles a CTA, the ring in use
    (BF16, 128, 1, 40, 800000, [60000], 3),        # six slots
    (BF16, 128, 4, 9, 4000, [3000, 2999], 1),      # slabs on the register-fragment form
    (BF16, 64, 1, 5, 100, [90], 0),               # all of a head's keys in one item
    (F32, 128, 4, 20, 4000, [3000, 2999], 2),
    (F32, 64, 1, 40, 110, [70], 0),
])
def test_an_expired_wait_is_reported_and_the_workspace_recovers(dtype, d, D, N, cap, pos, ticket):
    # a tile that never completes: the waits for it run out, the step says so, the next one on that workspace is right
    B = len(pos)
    cfg = config(B, N, 1, d, dtype, [D], [0])
    p = Problem(cfg, cap, pos, random_parents(np.random.default_rng(N), B, N, 5, pad=False)).to_gpu()
    want = p.step()
    p.ws[256:] = 0x7f                               # nothing of the step that gives up may depend on what was there
    rat.rat_debug_set_scan_stall(p.ws, ticket=ticket, spin_limit_ns=20_000_000)
    p.step(check=False)
    with pytest.raises(rat.RatError) as e:
        rat.rat_check_status(p.ws)
    assert e.value.status == rat.RAT_ERR_TIMEOUT
    rat.rat_debug_set_scan_stall(p.ws, ticket=-1)
    o, lse = p.step()
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


def test_an_entry_whose_length_is_out_of_range_keeps_its_table():
    # every value of it, those that name no page too; the other entries are served
    cfg = config(2, 1, 1, 64, BF16, [1], [0])
    ws = rat.workspace(cfg, rat.RAT_OP_STATUS)
    table = torch.tensor([[3, -7, 99], [0, 1, -1]], dtype=torch.int32, device=DEV)
    free = torch.tensor([2, 4, 5, 9, 9, 9], dtype=torch.int32, device=DEV)
    n = torch.tensor([3], dtype=torch.int32, device=DEV)
    rat.rat_page_table_update(cfg, table, 8, 6, 24, torch.tensor([25, 24], dtype=torch.int32, device=DEV), 0, free, n, ws)
    with pytest.raises(rat.RatError, match="RAT_ERR_INVALID"):
        rat.rat_check_status(ws)
    assert table.tolist() == [[3, -7, 99], [0, 1, 5]] and int(n) == 2 and free[:2].tolist() == [2, 4]


def test_checks_in_python_give_the_same_calls(monkeypatch):
    cfg = config(2, 9, 2, 64, BF16, [2, 1], [0, 6])
    p = Problem(cfg, 300, [250, 5], random_parents(np.random.default_rng(1), 2, 9, 4)).to_gpu()
    want = p.step()
    monkeypatch.setattr(rat, "_native", lambda *args: None)
    got = p.step()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    ck = p.ck.clone()
    commit(p, [8, -1], ck, p.cv.clone())
    assert not torch.equal(ck.nan_to_num(), p.ck.nan_to_num())
    with pytest.raises(ValueError, match="pos .*shape"):
        p.d_pos = p.d_pos[:1]
        p.step()


def test_a_paged_cache_of_other_sizes_is_refused():
    # on the host, before anything is launched: the kernels would read past a smaller table or pool
    cfg = config(2, 5, 2, 64, BF16, [2, 1], [0, 6])
    p = Problem(cfg, 60, [50, 5], random_parents(np.random.default_rng(1), 2, 5, 4)).to_gpu()
    pools = [torch.zeros(8, 2, 16, 64, dtype=BF16, device=DEV) for _ in range(2)]
    table = torch.arange(8, dtype=torch.int32, device=DEV).view(2, 4)
    p.step(rat.paged_cache(cfg, *pools, table, p.cap))
    slots = torch.empty(2, 5, 2, dtype=torch.int64, device=DEV)
    for kw, pool, tab in ((dict(B=1), (8, 2, 16, 64), (1, 4)), (dict(H=1, dil=[2], win=[0]), (8, 1, 16, 64), (2, 4)),
                          (dict(d=128), (8, 2, 16, 128), (2, 4)), (dict(dtype=F32), (8, 2, 16, 64), (2, 4))):
        other = cfg.replace(**kw)
        made = rat.paged_cache(other, *(torch.zeros(pool, dtype=other.torch_dtype, device=DEV) for _ in range(2)),
                               torch.zeros(tab, dtype=torch.int32, device=DEV), p.cap)
        for call in (lambda: p.step(made), lambda: commit(p, [0, 0], None, None, desc=made),
                     lambda: rat.rat_slot_map(cfg, made, p.cap, p.d_pos, None, slots, None, p.ws)):
            with pytest.raises(ValueError, match="made for"):
                call()
    # the first entries of a larger table are a table
    small = cfg.replace(B=1)
    ws, o = rat.workspace(small, rat.RAT_OP_TREE, p.cap), torch.empty_like(p.d_q[:1])
    rat.rat_tree_decode_step_paged(small, *(x[:1] for x in (p.d_q, p.d_k, p.d_v, p.d_g, p.d_parent, p.d_sk, p.d_sv)),
                                   rat.paged_cache(cfg, *pools, table, p.cap), p.cap, p.d_pos[:1], o, None, ws)
    rat.rat_check_status(ws)


@pytest.mark.parametrize("N", [8, 20, 40])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("where", ["k", "v", "q"])
def test_a_broken_branch_stays_alone_on_the_persistent_form(N, bad, where):
    # node 2 is not finite: its branch is lost, the others' results do not change by a bit
    parent = np.concatenate([[[-1, 0, 0, 1, 2, 3, -1, 6]], np.full((1, N - 8), 6)], 1).astype(np.int32)
    cfg = config(1, N, 2, 128, BF16, [1, 1], [0, 9])
    p = Problem(cfg, 400000, [30000], parent).to_gpu()
    want = p.step()
    getattr(p, "d_" + where)[0, 2, :, 5] = bad
    o, lse = p.step()
    clean = [n for n in range(N) if n not in (2, 4)]
    if where == "q":
        clean.append(4)                                    # a child shares the branch's rows, not its query
    assert torch.equal(o[:, clean], want[0][:, clean]) and torch.equal(lse[..., clean], want[1][..., clean])
    if where != "k":
        assert not torch.isfinite(o[0, 2]).all(-1).any()   # in either head


def test_topk_decode_after_a_commit_and_new_statistics():
    # the committed rows count once the block statistics hold them, entry by entry: as after as many top-k decode steps
    d, cap, bs, K, pos, leaf = 64, 256, 8, 3, [120, 77], [10, 4]
    cfg = config(2, 11, 2, d, BF16, [1, 1], [0, 0])
    p = Problem(cfg, cap, pos, np.array([[i - 1 for i in range(11)]] * 2, np.int32)).to_gpu()
    one = lambda b: cfg.replace(B=1, T=b)  # noqa: E731

    def stats_of(ck, length):
        stats = torch.zeros(rat.topk_stats_shape(cfg, bs, cap), device=DEV)
        for b, n in enumerate(length):
            rat.rat_topk_build_stats(one(n), bs, rat.RAT_TOPK_QUEST, ck[b:b + 1], cap, stats[b:b + 1])
        return stats

    def decode(n, x, sk, sv, ck, cv, stats, at):
        o = torch.empty(2, 2, d, dtype=BF16, device=DEV)
        ws = rat.workspace(cfg, rat.RAT_OP_TOPK_DECODE, cap)
        rat.rat_topk_decode_step(cfg, bs, K, rat.RAT_TOPK_QUEST, *(y[n].contiguous() for y in x), sk, sv, ck, cv, cap, stats,
                                 at, o, None, None, ws)
        rat.rat_check_status(ws)
        return o

    tokens = [torch.stack([y[b, [*range(leaf[b] + 1), *[leaf[b]] * (10 - leaf[b])]] for b in range(2)], 1)
              for y in (p.d_q, p.d_k, p.d_v, p.d_g)]          # [11, 2, H, d]: entry 1 takes its first five only
    steps = [t.clone() for t in (p.d_sk, p.d_sv, p.ck, p.cv)] + [stats_of(p.ck, pos)]
    for n in range(11):
        before = [t[1:].clone() for t in steps]
        decode(n, tokens, *steps, p.d_pos + torch.tensor([n, min(n, 5)], dtype=torch.int32, device=DEV))
        if n > leaf[1]:
            for t, s in zip(steps, before):
                t[1:] = s
    ck, cv = p.ck.clone(), p.cv.clone()
    sk, sv, at = commit(p, leaf, ck, cv)
    stats = stats_of(ck, at.tolist())
    for b in range(2):
        used = -(-int(at[b]) // bs)
        assert torch.allclose(stats[b, :, :used], steps[4][b, :, :used], rtol=2 ** -7, atol=1e-6)
    want = decode(3, tokens, *[t.clone() for t in steps], at)
    got = decode(3, tokens, sk, sv, ck, cv, stats, at)
    assert (got.float() - want.float()).abs().max() <= 2e-2


@pytest.mark.parametrize("cap,d,N,D", [                     # 800000 rows: the persistent form where d = 128
    *((cap, d, N, 1) for cap in (60, 800000) for d in (64, 128) for N in (1, 4, 8, 9, 16)),
    *((cap, 128, N, 1) for cap, N in ((60, 20), (60, 33), (60, 64), (800000, 17), (800000, 32), (150000, 40))),
    (60, 128, 40, 8), (800000, 128, 40, 8)])
def test_bf16_outputs_are_as_exact_as_their_type(cap, d, N, D):
    # Few keys with probabilities of all sizes, rows that are the tokens (no recurrence); D = 8: held rows by sets of five
    # nodes.  The output's own rounding is at most half a step, eps / 2 = 2^-8 of the value.  The rest: probabilities
    # within 2^-17, so their part of the sum within 2^-17 max|v|; scores of d products in fp32, each within
    # 2^-24 sum|q k| (1 + d), under 2^-24 * 129 * 3 * d^0.5 here after scaling (|q k| averages 2 / pi, its scaled sum
    # stays below 3 d^0.5), 2^-12.4 at worst and a sixteenth of it, 2^-16, for sums that are rounded to nearest at
    # random: 2^-13 max|v| holds all of it.
    cfg = config(2, N, 1, d, BF16, [D], [0], [0])
    parent = np.full((2, N), -1, np.int32) if D == 1 else np.array([[i - 5 if i >= 5 else -1 for i in range(N)]] * 2, np.int32)
    p = Problem(cfg, cap, [6, 17] if D == 1 else [43, 120 if cap > 200 else 52], parent, std=1.0)
    p.to_gpu()
    o, _ = p.step()
    ro, _ = p.reference()
    err, top = np.abs(f64(o) - ro), max(f64(p.hv).max(), f64(p.v).max(), -f64(p.hv).min(), -f64(p.v).min())
    assert (err <= 2.0 ** -8 * np.abs(ro) + 2.0 ** -13 * top).all(), (err - 2.0 ** -8 * np.abs(ro)).max() / top


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("D,W,N", [(1, 0, 6), (1, 0, 20), (1, 9, 40), (3, 5, 12)])
def test_a_key_left_out_leaves_nothing_behind(dtype, d, D, W, N):
    # a weight of 0 is 0: the largest finite values in a branch, or in a held row whose score is -inf, do not reach the
    # nodes that do not see them, by a bit
    parent = np.concatenate([[[-1, 0, 0, -1, 3, 4]], np.full((1, N - 6), 3)], 1).astype(np.int32)
    cfg = config(1, N, 1, d, dtype, [D], [W])
    p = Problem(cfg, 200, [130], parent)
    p.q[..., 5] = p.q[..., 5].abs() + 0.5
    p.hk[0, 100, 0, 5] = -float("inf")
    p.to_gpu()
    want = p.step()
    p.d_v[0, :3] = torch.finfo(dtype).max                  # nodes 0 to 2; the others hang below node 3
    p.cv[0, 0, [(100 % D) * -(-200 // D) + 100 // D]] = -torch.finfo(dtype).max
    o, lse = p.step()
    assert torch.equal(o[:, 3:], want[0][:, 3:]) and torch.equal(lse[..., 3:], want[1][..., 3:])


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_fewer_pieces_than_the_capacity_has_runs(dtype):
    # 544 pairs: a dense head's rows are cut into at most 27 pieces, a long window likewise, whatever the capacity
    rng = np.random.default_rng(13)
    B, H, N, cap = 17, 32, 5, 7200
    cfg = config(B, N, H, 64, dtype, [1] * 4 + [48] * 28, [0, 6000, 0, 0] + [37] * 28, [0] * 4 + [1] * 28)
    pos = [int(x) for x in rng.integers(0, 90, B)]
    pos[5] = 7100
    p = Problem(cfg, cap, pos, random_parents(rng, B, N, 3)).to_gpu()
    p.check(*p.step())


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_all_keys_of_a_head_in_one_item_where_pairs_are_many(dtype):
    # 15104 pairs: no head is cut, however many rows it has; the item of a dense head writes the result itself
    rng = np.random.default_rng(14)
    B, H, N, cap = 59, 256, 2, 300
    cfg = config(B, N, H, 64, dtype, [1, 1, 2, 1] * 64, [0, 200, 150, 3] * 64, [0, 1, 1, 1] * 64)
    pos = [int(x) for x in rng.integers(0, 12, B)]
    pos[7], pos[40] = 290, 131
    p = Problem(cfg, cap, pos, random_parents(rng, B, N, 2)).to_gpu()
    p.check(*p.step())
