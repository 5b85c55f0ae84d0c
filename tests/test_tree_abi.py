"""Host-side checks of the drafted-tree and page-table entry points (no GPU, nothing is launched): argument errors
return the documented status before any launch, and workspace sizes are as documented."""
import ctypes
import sys

import pytest
import torch

import recurrence_augmented_dilated_gated_b200 as rat
from recurrence_augmented_dilated_gated_b200 import build as rat_build

P = 1 << 20   # a fake, aligned address that no call here dereferences
WS = 1 << 20


@pytest.fixture(scope="module")
def lib():
    rat_build.build()
    return rat.load_library()


def cfg(**kw):
    a = dict(B=2, T=9, H=2, d=128, dtype=rat.RAT_BF16, dil=[4, 1], win=[0, 8], recur=None, scale=0.0)
    a.update(kw)
    return rat.Config(**a)


def step(lib, c, cap=1000, ptrs=None, ws=WS, ws_bytes=1 << 40, desc=None):
    a = dict(q=P, k=P, v=P, g=P, parent=P, sk=P, sv=P, ck=P, cv=P, pos=P, o=P, lse=None)
    a.update(ptrs or {})
    head = [c.ref() if c is not None else None] + [a[x] for x in ("q", "k", "v", "g", "parent", "sk", "sv")]
    tail = [cap, a["pos"], a["o"], a["lse"], ws, ws_bytes, None]
    if desc is not None:
        return lib.rat_tree_decode_step_paged(*head, ctypes.byref(desc) if desc else None, *tail)
    return lib.rat_tree_decode_step(*head, a["ck"], a["cv"], *tail)


def commit(lib, c, cap=1000, ptrs=None, ws=WS, ws_bytes=1 << 40, desc=None):
    a = dict(k=P, v=P, g=P, parent=P, leaf=P, sk=P, sv=P, ok=P, ov=P, ck=P, cv=P, pos=P, out_pos=P)
    a.update(ptrs or {})
    head = [c.ref()] + [a[x] for x in ("k", "v", "g", "parent", "leaf", "sk", "sv", "ok", "ov")]
    tail = [cap, a["pos"], a["out_pos"], ws, ws_bytes, None]
    if desc is not None:
        return lib.rat_tree_commit_paged(*head, ctypes.byref(desc) if desc else None, *tail)
    return lib.rat_tree_commit(*head, a["ck"], a["cv"], *tail)


BAD_CFGS = [
    (dict(T=0), rat.RAT_ERR_INVALID), (dict(T=-1), rat.RAT_ERR_INVALID), (dict(T=65), rat.RAT_ERR_UNSUPPORTED),
    (dict(d=96), rat.RAT_ERR_UNSUPPORTED), (dict(dtype=7), rat.RAT_ERR_INVALID), (dict(dil=[0, 1]), rat.RAT_ERR_INVALID),
    (dict(win=[-1, 0]), rat.RAT_ERR_INVALID), (dict(B=-1), rat.RAT_ERR_INVALID), (dict(flags=8), rat.RAT_ERR_INVALID),
    (dict(B=1 << 28), rat.RAT_ERR_UNSUPPORTED),   # more CTAs than a grid has
]


@pytest.mark.parametrize("i", range(len(BAD_CFGS)))
def test_configurations_that_are_refused(lib, i):
    kw, want = BAD_CFGS[i]
    assert step(lib, cfg(**kw)) == want
    assert commit(lib, cfg(**kw)) == want
    assert lib.rat_workspace_size(cfg(**kw).ref(), rat.RAT_OP_TREE, 1000) == 0


@pytest.mark.parametrize("name", ["q", "k", "v", "g", "parent", "sk", "sv", "ck", "cv", "pos", "o"])
def test_step_pointers(lib, name):
    for bad in (None, P + 8):
        assert step(lib, cfg(), ptrs={name: bad}) == rat.RAT_ERR_INVALID
        assert name.encode()[:1] in lib.rat_last_error() and lib.rat_last_error()


@pytest.mark.parametrize("name", ["k", "v", "g", "parent", "leaf", "sk", "sv", "ok", "ov", "ck", "cv", "pos", "out_pos"])
def test_commit_pointers(lib, name):
    for bad in (None, P + 8):
        assert commit(lib, cfg(), ptrs={name: bad}) == rat.RAT_ERR_INVALID


def test_optional_outputs_have_to_be_aligned(lib):
    assert step(lib, cfg(), ptrs=dict(lse=P + 4)) == rat.RAT_ERR_INVALID


@pytest.mark.parametrize("call", [step, commit])
def test_capacity_and_workspace(lib, call):
    assert call(lib, cfg(), cap=0) == rat.RAT_ERR_INVALID
    assert call(lib, cfg(), ws=None) == rat.RAT_ERR_INVALID
    assert call(lib, cfg(), ws=WS + 16) == rat.RAT_ERR_INVALID
    assert call(lib, cfg(), ws_bytes=255) == rat.RAT_ERR_WORKSPACE
    assert call(lib, cfg(B=0), ptrs=dict(k=None)) == rat.RAT_OK       # nothing to do: no pointer is looked at


@pytest.mark.parametrize("call", [step, commit])
def test_page_descriptor(lib, call):
    c, cap = cfg(), 1000
    R = lib.rat_cache_rows(c.ref(), cap)
    good = dict(pool_k=P, pool_v=P, page_table=P, page_rows=64, pages_per_seq=-(-R // 64), num_pages=64)
    for bad in (dict(page_rows=0), dict(num_pages=0), dict(pages_per_seq=-(-R // 64) - 1), dict(pool_k=None),
                dict(pool_v=P + 8), dict(page_table=P + 8), dict(page_table=None)):
        assert call(lib, c, cap, desc=rat.rat_paged_cache(**{**good, **bad})) == rat.RAT_ERR_INVALID, bad


def test_workspace_size(lib):
    size = lambda **kw: lib.rat_workspace_size(cfg(**kw).ref(), rat.RAT_OP_TREE, 1000)  # noqa: E731
    # at least the nodes' rows and one partial of d + 2 floats for each node and head
    assert size() >= 2 * 2 * 9 * 128 * 2 * 2 + 2 * 2 * 9 * 130 * 4
    assert size(T=64) > size() and size(B=8) > size()
    assert size(t0=50, t_cap=20) == size()                       # a step does not look at them
    assert lib.rat_workspace_size(cfg().ref(), rat.RAT_OP_TREE, 0) == 0
    assert lib.rat_workspace_size(cfg().ref(), rat.RAT_OP_STATUS, 0) == 256
    assert lib.rat_workspace_size(cfg().ref(), rat.RAT_OP_STATUS + 1, 0) == 0


def update(lib, c, **kw):
    a = dict(table=P, page_rows=64, pps=20, num_pages=100, cap=1000, length=P, extra=4, free=P, n_free=P, ws=WS,
             ws_bytes=256)
    a.update(kw)
    return lib.rat_page_table_update(c.ref(), a["table"], a["page_rows"], a["pps"], a["num_pages"], a["cap"],
                                     a["length"], a["extra"], a["free"], a["n_free"], a["ws"], a["ws_bytes"], None)


def test_page_table_update_refusals(lib):
    c = cfg()
    for kw in (dict(table=None), dict(table=P + 4), dict(length=None), dict(free=None), dict(n_free=None),
               dict(n_free=P + 4), dict(page_rows=0), dict(pps=0), dict(pps=15), dict(num_pages=0), dict(cap=0),
               dict(extra=-1), dict(ws=None), dict(ws=WS + 8)):
        assert update(lib, c, **kw) == rat.RAT_ERR_INVALID, kw
    assert update(lib, c, ws_bytes=128) == rat.RAT_ERR_WORKSPACE
    assert update(lib, cfg(d=96)) == rat.RAT_ERR_UNSUPPORTED
    assert update(lib, cfg(B=1 << 20, T=1), pps=1 << 12) == rat.RAT_ERR_UNSUPPORTED
    assert update(lib, cfg(B=0), table=None) == rat.RAT_OK


def test_slot_map_refusals(lib):
    def call(c, cap=1000, pos=P, count=None, slots=P, ring=None, ws=WS, ws_bytes=256, desc=None):
        return lib.rat_slot_map(c.ref(), ctypes.byref(desc) if desc else None, cap, pos, count, slots, ring, ws,
                                ws_bytes, None)

    c = cfg()
    for kw in (dict(cap=0), dict(pos=None), dict(pos=P + 4), dict(count=P + 4), dict(slots=None), dict(slots=P + 8),
               dict(ring=P + 8), dict(ws=None)):
        assert call(c, **kw) == rat.RAT_ERR_INVALID, kw
    assert call(c, ws_bytes=0) == rat.RAT_ERR_WORKSPACE
    assert call(cfg(T=0), slots=None) == rat.RAT_OK
    bad = rat.rat_paged_cache(pool_k=P, pool_v=P, page_table=P, page_rows=64, pages_per_seq=2, num_pages=64)
    assert call(c, desc=bad) == rat.RAT_ERR_INVALID


def test_binding_refuses_cpu_tensors_and_wrong_shapes():
    c = cfg(B=1, T=4)
    x = torch.zeros(1, 4, 2, 128, dtype=torch.bfloat16)
    s, i = torch.zeros(1, 2, 128), torch.zeros(1, dtype=torch.int32)
    ws = torch.zeros(1 << 16, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        rat.rat_tree_decode_step(c, x, x, x, x, torch.zeros(1, 4, dtype=torch.int32), s, s, x, x, 100, i, x, None, ws)
    with pytest.raises(ValueError, match="CUDA"):
        rat.rat_tree_commit(c, x, x, x, torch.zeros(1, 4, dtype=torch.int32), i, s, s, s, s, x, x, 100, i, i, ws)
    with pytest.raises(ValueError, match="CUDA"):
        rat.rat_page_table_update(c, torch.zeros(1, 4, dtype=torch.int32), 16, 4, 100, i, 0, i, i, ws)
    with pytest.raises(ValueError, match="CUDA"):
        rat.rat_slot_map(c, None, 100, i, None, torch.zeros(1, 4, 2, dtype=torch.int64), None, ws)


def test_status_string_of_the_page_error(lib):
    assert lib.rat_status_string(rat.RAT_ERR_NO_PAGES).decode().startswith("RAT_ERR_NO_PAGES")
    assert rat.STATUS_NAMES[rat.RAT_ERR_NO_PAGES] == "RAT_ERR_NO_PAGES"


def test_native_part_of_the_binding():
    # it accepts CUDA tensors that are as planned and leaves everything else to Python
    from recurrence_augmented_dilated_gated_b200 import _binding

    t, plan = torch.zeros(3, dtype=torch.int32), (("t", torch.int32, (3,), False),)
    ws = torch.zeros(256, dtype=torch.uint8)
    assert _binding.pointers(plan, ws, t) is None
    for odd in (None, 3, "x", [1], torch.nn.Parameter(torch.zeros(3))):
        assert _binding.pointers(plan, ws, odd) is None
        assert _binding.pointers(plan, odd, t) is None
    for bad in ((), (3,), ("t",), (("t", torch.int32, (3,)),)):
        if len(bad) == 1:
            assert _binding.pointers(bad, ws, t) is None
        else:
            with pytest.raises(TypeError):
                _binding.pointers(bad, ws, t)
    with pytest.raises(TypeError):
        _binding.pointers(plan)


def test_workspace_of_many_long_sequences(lib):
    # partials are bounded by what the GPU runs at a time and by the pairs, not by the capacity
    for dtype, d, page in ((rat.RAT_BF16, 128, 0), (rat.RAT_F32, 64, 0)):
        for B in (1, 64, 256, 1000):
            for win in (0, 1 << 20):
                c = cfg(B=B, T=64, H=16, d=d, dtype=dtype, dil=[1] * 16, win=[win] * 16)
                size = lib.rat_workspace_size(c.ref(), rat.RAT_OP_TREE, 1 << 20)
                pairs = B * 16
                slots = 2 * (96 * 148 + 2 * pairs)     # pieces of sets and of windows
                assert size <= (1 << 20) + (slots * 64 * (d + 2) + 3 * pairs * 64 * d) * 4, (B, win, size)


MOST_CAP = 2 ** 31 - 2 ** 16 - 1   # of a tree step


@pytest.mark.parametrize("dtype", [rat.RAT_BF16, rat.RAT_F32])
@pytest.mark.parametrize("flags", [0, rat.RAT_FLAG_GRID_DILATION])
@pytest.mark.parametrize("dil,win", [([1, 1], [0, 0]), ([1, 1], [2 ** 31 - 1, 5]), ([16, 3], [2 ** 31 - 1, 2 ** 31 - 1]),
                                     ([2 ** 31 - 1, 64], [0, 300])])
def test_capacities_near_two_to_the_31(lib, dtype, flags, dil, win):
    # the plan's counts stay in range up to the largest capacity, and what is past it is refused
    for B, T in ((1, 1), (1, 64), (8, 33)):
        c = cfg(B=B, T=T, dtype=dtype, flags=flags, dil=dil, win=win)
        last = 0
        for cap in (1 << 20, 1 << 28, (1 << 31) - (1 << 20), MOST_CAP):
            size = lib.rat_workspace_size(c.ref(), rat.RAT_OP_TREE, cap)
            # a partial of d floats, a maximum and a sum for each node, head and piece, of 128 rows at least
            assert 0.9 * last <= size <= (1 << 20) + B * T * 2 * 1100 * (cap / 64 + 4), (cap, size)
            last = size
        for cap in (MOST_CAP + 1, 2 ** 31 - 4096, 2 ** 31 - 1):
            assert lib.rat_workspace_size(c.ref(), rat.RAT_OP_TREE, cap) == 0
            assert step(lib, c, cap=cap) == rat.RAT_ERR_UNSUPPORTED
        pages = rat.rat_paged_cache(pool_k=P, pool_v=P, page_table=P, page_rows=1 << 16, pages_per_seq=1 << 17, num_pages=4)
        assert step(lib, c, cap=2 ** 31 - 1, desc=pages) == rat.RAT_ERR_UNSUPPORTED
        # a commit has no plan: its positions are bounded by the capacity, whatever it is
        assert commit(lib, c, cap=2 ** 31 - 1, ws=None) == rat.RAT_ERR_INVALID and b"workspace" in lib.rat_last_error()


@pytest.mark.parametrize("T", [2 ** 31 - 1, 2 ** 31 - 2, 2 ** 31 - 100, 2 ** 31 - 128])
def test_slot_maps_too_wide_for_a_grid_are_refused(lib, T):
    # ahead of every pointer: the sizes alone decide
    call = lambda c: lib.rat_slot_map(c.ref(), None, 1000, None, None, None, None, None, 0, None)  # noqa: E731
    assert call(cfg(B=1, T=T, H=1, dil=[1], win=[0])) == rat.RAT_ERR_UNSUPPORTED
    assert call(cfg(B=3, T=T // 3 + 1, H=1, dil=[1], win=[0])) == rat.RAT_ERR_UNSUPPORTED
    assert call(cfg(B=1, T=2 ** 31 - 129, H=1, dil=[1], win=[0])) == rat.RAT_ERR_INVALID and b"pos" in lib.rat_last_error()


def test_binding_of_another_torch_is_rebuilt(lib, monkeypatch, tmp_path):
    assert rat_build.binding_up_to_date()
    stamp = tmp_path / "stamp"
    monkeypatch.setattr(rat_build, "BINDING_STAMP", str(stamp))
    assert not rat_build.binding_up_to_date()                   # not known what it was built for
    stamp.write_text(rat_build.binding_target())
    assert rat_build.binding_up_to_date()
    monkeypatch.setattr(torch, "__version__", "2.0.0")
    assert not rat_build.binding_up_to_date()


@pytest.mark.parametrize("cxx", ["false", "/nonexistent/c++"])
def test_a_build_without_the_native_part_of_the_binding(lib, monkeypatch, tmp_path, cxx):
    monkeypatch.setenv("CXX", cxx)
    for name in ("BINDING", "BINDING_STAMP"):
        monkeypatch.setattr(rat_build, name, str(tmp_path / name))
    with pytest.warns(UserWarning, match="in Python"):
        assert rat_build.build() == rat_build.LIB
    assert not list(tmp_path.iterdir())


class Foreign:
    built_for = "torch 0.4"

    @staticmethod
    def pointers(*args):
        raise AssertionError("called")


@pytest.mark.parametrize("module,why", [(None, "halted"), (Foreign, "built for torch 0.4"), (object(), "built_for")])
def test_checks_in_python_without_the_native_part(lib, monkeypatch, module, why):
    monkeypatch.setattr(rat, "_native", None)
    monkeypatch.setitem(sys.modules, rat.__name__ + "._binding", module)
    monkeypatch.setattr(rat, "_binding", module, raising=False)
    if module is None:
        monkeypatch.delattr(rat, "_binding")
    i, ws = torch.zeros(1, dtype=torch.int32), torch.zeros(256, dtype=torch.uint8)
    with pytest.warns(UserWarning, match=why):
        with pytest.raises(ValueError, match="CUDA"):
            rat.rat_slot_map(cfg(B=1, T=4), None, 100, i, None, torch.zeros(1, 4, 2, dtype=torch.int64), None, ws)
    assert rat._native((), ws) is None                          # looked for once


def test_errors_begin_with_the_argument(lib):
    # and nothing else of its name: state_k, not state
    full = dict(sk="state_k", sv="state_v", ck="cache_k", cv="cache_v", ok="out_state_k", ov="out_state_v")
    for call, names in ((step, ["q", "k", "v", "g", "parent", "sk", "sv", "ck", "cv", "pos", "o", "lse"]),
                        (commit, ["k", "v", "g", "parent", "leaf", "sk", "sv", "ok", "ov", "ck", "cv", "pos", "out_pos"])):
        for name in names:
            for bad in (None, P + 8):
                if name == "lse" and bad is None:
                    continue
                assert call(lib, cfg(), ptrs={name: bad}) == rat.RAT_ERR_INVALID
                assert lib.rat_last_error().decode().split()[0] == full.get(name, name)
