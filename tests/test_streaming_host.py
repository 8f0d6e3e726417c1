"""Refusals and host logic of the streaming entry points, without a GPU:
every bad argument is rejected before anything is queued (the addresses are
never dereferenced), and the binding checks its tensors."""
import pytest
import torch

import streaming_ref as ref
from feed_forward_view_vggt_b200 import attn
from feed_forward_view_vggt_b200 import build as vbuild

A = 1 << 40  # fake, aligned "device" addresses, far apart
E, U, W = attn.VGGT_ERR_INVALID_ARG, attn.VGGT_ERR_UNSUPPORTED, attn.VGGT_ERR_WORKSPACE
CACHE = dict(n_seqs=3, n_heads=16, n_kv_heads=4, head_dim=64, page_size=16, n_pages=100, max_pages=20,
             page_stride=4 * 16 * 64, head_stride=16 * 64, token_stride=64)


@pytest.fixture(scope="module", autouse=True)
def built():
    vbuild.build()
    attn.load()


def cache(**more):
    c = {**CACHE, **more}
    return attn.vggt_cache(*[c[n] for n, _ in attn.vggt_cache._fields_])


def refused(status, expect):
    assert status == expect, attn.vggt_status_string(status)


BAD_TABLES = [({"n_seqs": 0}, E), ({"n_seqs": 4097}, U), ({"page_size": 0}, E), ({"page_size": 12}, U),
              ({"n_pages": 0}, E), ({"n_pages": 1 << 27}, U), ({"max_pages": 0}, E), ({"max_pages": 1 << 27}, U)]
BAD_CACHES = BAD_TABLES + [
    ({"n_heads": 0}, E), ({"n_heads": 65, "n_kv_heads": 65}, U), ({"n_kv_heads": 0}, E), ({"n_kv_heads": 3}, E),
    ({"head_dim": 0}, E), ({"head_dim": 128}, U), ({"page_stride": 0}, E), ({"page_stride": 4100}, E),
    ({"head_stride": 32}, E), ({"token_stride": -64}, E), ({"token_stride": 1 << 40}, E)]


def plan(c=None, **more):
    a = dict(cached=A, new=2 * A, free=3 * A, cap=10, n_free=4 * A, table=5 * A, rows=7, cu=6 * A, kv=7 * A,
             slots=8 * A, counts=9 * A) | more
    return attn.vggt_cache_plan(c or cache(), a["cached"], a["new"], a["free"], a["cap"], a["n_free"], a["table"],
                                a["rows"], a["cu"], a["kv"], a["slots"], a["counts"], 0)


@pytest.mark.parametrize("bad,status", BAD_TABLES)
def test_plan_refuses_bad_sizes(bad, status):
    refused(plan(cache(**bad)), status)


@pytest.mark.parametrize("bad", [dict(cached=None), dict(new=None), dict(free=None), dict(n_free=None),
                                 dict(table=None), dict(cu=None), dict(kv=None), dict(slots=None),
                                 dict(counts=None), dict(cap=-1), dict(rows=-1), dict(slots=8 * A + 2),
                                 dict(cu=A), dict(kv=6 * A + 4), dict(counts=4 * A), dict(table=3 * A),
                                 dict(counts=8 * A + 24)])
def test_plan_refuses_bad_arguments(bad):
    refused(plan(**bad), E)


def append(c=None, **more):
    a = dict(k=A, v=2 * A, row=256, head=64, slots=3 * A, rows=9, kp=4 * A, vp=5 * A) | more
    return attn.vggt_cache_append(c or cache(), a["k"], a["v"], a["row"], a["head"], a["slots"], a["rows"], a["kp"],
                                  a["vp"], 0)


@pytest.mark.parametrize("bad,status", BAD_CACHES)
def test_append_refuses_bad_caches(bad, status):
    refused(append(cache(**bad)), status)


@pytest.mark.parametrize("bad", [dict(k=None), dict(v=None), dict(slots=None), dict(kp=None), dict(vp=None),
                                 dict(k=A + 8), dict(vp=5 * A + 2), dict(slots=3 * A + 1), dict(row=60),
                                 dict(row=252), dict(head=0), dict(rows=-1), dict(vp=4 * A), dict(k=4 * A),
                                 dict(v=5 * A + 1024), dict(slots=4 * A + 64)])
def test_append_refuses_bad_arguments(bad):
    refused(append(**bad), E)


def test_no_rows_is_nothing_to_do():
    refused(append(rows=0, k=None, v=None, slots=None), attn.VGGT_OK)
    refused(attend(rows=0, q=None, o=None, ws=None, nbytes=0), attn.VGGT_OK)
    refused(norm(rows=0, x=None, y=A, out=None, h=2 * A), attn.VGGT_OK)


def attend(c=None, **more):
    a = dict(q=A, row=1024, head=64, kp=2 * A, vp=3 * A, table=4 * A, cu=5 * A, kv=6 * A, rows=9, unit=1, o=7 * A,
             lse=None, ws=8 * A, nbytes=1 << 30, scale=0.125) | more
    return attn.vggt_attn_cached(c or cache(), a["q"], a["row"], a["head"], a["kp"], a["vp"], a["table"], a["cu"],
                                 a["kv"], a["rows"], a["unit"], a["o"], a["lse"], a["ws"], a["nbytes"], a["scale"], 0)


@pytest.mark.parametrize("bad,status", BAD_CACHES)
def test_attention_refuses_bad_caches(bad, status):
    refused(attend(cache(**bad)), status)
    assert attn.vggt_attn_cached_workspace_bytes(cache(**bad), 9) == 0


@pytest.mark.parametrize("bad", [dict(q=None), dict(kp=None), dict(vp=None), dict(table=None), dict(cu=None),
                                 dict(kv=None), dict(o=None), dict(q=A + 8), dict(o=7 * A + 8), dict(lse=9 * A + 2),
                                 dict(table=4 * A + 2), dict(row=63), dict(head=68), dict(rows=-1), dict(unit=-1),
                                 dict(scale=0.0), dict(scale=float("nan")), dict(o=A), dict(o=2 * A + 2048),
                                 dict(lse=7 * A + 64), dict(lse=6 * A), dict(ws=None), dict(ws=8 * A + 16),
                                 dict(ws=7 * A), dict(ws=3 * A)])
def test_attention_refuses_bad_arguments(bad):
    refused(attend(**bad), E)


def test_attention_refuses_a_small_workspace():
    need = attn.vggt_attn_cached_workspace_bytes(cache(), 9)
    assert need > 0 and need % 256 == 0
    refused(attend(nbytes=need - 1), W)


def test_workspace_stays_within_bounds():
    # one key tile at most: nothing is split, nothing to store
    assert attn.vggt_attn_cached_workspace_bytes(cache(max_pages=8), 9) == 0
    assert attn.vggt_attn_cached_workspace_bytes(cache(), -1) == 0
    for rows in (1, 64, 1374, 20000):
        for heads, kv_heads in ((1, 1), (16, 16), (64, 8), (21, 3)):
            c = cache(n_heads=heads, n_kv_heads=kv_heads, max_pages=60000)
            assert attn.vggt_attn_cached_workspace_bytes(c, rows) <= 24 << 20


def norm(**more):
    a = dict(rows=5, cols=128, kind=0, f32=1, post=0, gate_rows=0, eps=1e-6, xs=128, ys=128, os=128, hs=128, x=A,
             y=2 * A, pw=None, pb=None, scale=None, gate=None, w=None, b=None, out=3 * A, h=4 * A) | more
    n = attn.vggt_norm(a["rows"], a["cols"], a["kind"], a["f32"], a["post"], a["gate_rows"], a["eps"], a["xs"],
                       a["ys"], a["os"], a["hs"])
    return attn.vggt_norm_residual(n, a["x"], a["y"], a["pw"], a["pb"], a["scale"], a["gate"], a["w"], a["b"],
                                   a["out"], a["h"], 0)


@pytest.mark.parametrize("bad,status", [
    (dict(rows=-1), E), (dict(cols=0), E), (dict(cols=12), U), (dict(cols=8200, xs=8200, ys=8200, os=8200, hs=8200), U),
    (dict(kind=2), E), (dict(f32=2), E), (dict(post=-1), E), (dict(eps=-1.0), E), (dict(eps=float("inf")), E),
    (dict(xs=120), E), (dict(ys=132), E), (dict(os=0), E), (dict(hs=64), E), (dict(x=None), E), (dict(x=A + 8), E),
    (dict(y=2 * A + 4), E), (dict(h=4 * A + 2), E), (dict(w=5 * A + 4), E), (dict(gate=5 * A), E),
    (dict(pw=5 * A), E), (dict(out=None, h=None), E), (dict(h=None, w=5 * A), E), (dict(y=None), E),
    (dict(y=None, out=None, scale=5 * A), E), (dict(out=A, os=256), E), (dict(out=A + 1024), E), (dict(h=A), E),
    (dict(h=2 * A), E), (dict(h=3 * A), E), (dict(scale=3 * A), E), (dict(rows=1 << 31, xs=128), U)])
def test_norm_refuses_bad_arguments(bad, status):
    refused(norm(**bad), status)


@pytest.mark.skipif(torch.cuda.is_available(), reason="fake addresses: without a GPU only")
def test_good_arguments_reach_the_device():
    # without a device the launch fails: the arguments were accepted
    for st in (plan(), append(), attend(), attend(lse=9 * A), norm(), norm(out=A), norm(y=None, out=None),
               norm(gate=5 * A, gate_rows=2), norm(post=1, pw=5 * A)):
        refused(st, attn.VGGT_ERR_CUDA)


def test_binding_checks_its_tensors():
    b = ref.Batch([20, 9], [3, 1], 8, 4, 2, device="cpu")
    with pytest.raises(ValueError):
        attn.cached(b.q, b.k_pages, b.v_pages, b.table, b.cu_rows, b.kv_lens)  # not on a GPU
    with pytest.raises(ValueError):
        attn.cached(b.q[0], b.k_pages, b.v_pages, b.table, b.cu_rows, b.kv_lens)
    with pytest.raises(ValueError):
        attn.cached(b.q, b.k_pages, b.v_pages, b.table, b.cu_rows[1:], b.kv_lens)
    with pytest.raises(ValueError):
        attn.cached(b.q, b.k_pages, b.v_pages.transpose(1, 2), b.table, b.cu_rows, b.kv_lens)
    with pytest.raises(ValueError):
        attn.cache_append(b.q[:, :2], b.q[:, 2:3], b.cu_rows, b.k_pages, b.v_pages)
    with pytest.raises(ValueError):
        attn.cache_plan(b.kv_lens, b.kv_lens[:1], b.kv_lens, b.kv_lens[:1], b.table, 8, 4)
    with pytest.raises(ValueError):
        attn.norm_residual(torch.zeros(2, 8), torch.zeros(2, 16))
    with pytest.raises(ValueError):
        attn.norm_residual(torch.zeros(2, 8), kind="batch")
    with pytest.raises(ValueError):
        attn.norm_residual(torch.zeros(2, 8), gate=torch.zeros(2, 8), rows_per_gate=2)


@pytest.mark.parametrize("rows,heads", [(1, 3), (4, 1), (1, 1)])
def test_binding_takes_any_stride_of_a_dimension_of_one(rows, heads):
    # a row of a projection beside a row of its own, one page or head of a larger cache: accepted up to the device
    k, v = torch.zeros(rows, heads, 64).bfloat16(), torch.zeros(rows, 3, heads, 64).bfloat16()[:, 1]
    if rows > 1:
        k = torch.zeros(rows, 3, 5, 64).bfloat16()[:, 1, :1]
        v = torch.zeros(rows, 3, 1, 320).bfloat16()[:, 1, :, :64]
    pages = torch.zeros(1, heads, 8, 64).bfloat16()
    others = torch.zeros(7, 2, heads, 8, 64).bfloat16()[3:4, 1]
    assert k.stride() != v.stride() and pages.stride() != others.stride()
    with pytest.raises(ValueError, match="k_pages: tensor must live on a CUDA device"):
        attn.cache_append(k, v, torch.zeros(rows, dtype=torch.int32), pages, others)


def test_binding_refuses_rows_that_lie_differently():
    k, v = torch.zeros(4, 3, 64).bfloat16(), torch.zeros(4, 3, 3, 64).bfloat16()[:, 1]
    pages = torch.zeros(2, 3, 8, 64).bfloat16()
    with pytest.raises(ValueError, match="same strides"):
        attn.cache_append(k, v, torch.zeros(4, dtype=torch.int32), pages, pages.clone())
    with pytest.raises(ValueError, match="same strides"):
        attn.cache_append(k, k, torch.zeros(4, dtype=torch.int32), pages,
                          torch.zeros(2, 8, 3, 64).bfloat16().transpose(1, 2))


def test_binding_says_when_its_module_is_not_built(monkeypatch):
    import sys

    monkeypatch.setattr(attn, "_host", None)
    monkeypatch.setitem(sys.modules, "feed_forward_view_vggt_b200._streaming", None)
    monkeypatch.delattr(sys.modules["feed_forward_view_vggt_b200"], "_streaming", raising=False)
    with pytest.raises(RuntimeError, match="not built"):
        attn.norm_residual(torch.zeros(2, 8))


def fake_plan(what, function, cached, new, free, n_free, table, page, n_rows, n_pages, stream, step=None, state=None):
    """The compiled module's plan by the plain reference, on the CPU."""
    assert function == "plan"
    i32 = lambda x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
    filled, cu, kv, slots, counts = ref.plan(cached.tolist(), new.tolist(), free.tolist(), int(n_free),
                                             table.tolist(), page, n_rows)
    table.copy_(i32(filled))
    step = torch.zeros(len(cu) + n_rows, dtype=torch.int32) if step is None else step
    step[:len(cu) + n_rows] = i32(cu + slots)
    if state is not None:
        state.copy_(i32(counts + kv))
    return 0, step[:len(cu)], i32(kv), step[len(cu):len(cu) + n_rows], i32(counts)


def test_paged_cache_keeps_its_state_in_place(monkeypatch):
    """What a queued plan reads is still the cache's own afterwards, and what a captured step reads is what later
    steps update."""
    monkeypatch.setattr(attn, "_call", fake_plan)
    cache = attn.PagedCache(n_pages=7, page_size=8, n_kv_heads=1, n_seqs=2, max_pages=5, device="cpu")
    state = lambda: [t.data_ptr() for t in (cache.kv_lens, cache.n_free, cache.free_pages, cache.block_table)]  # noqa: E731
    new = lambda *n: torch.tensor(n, dtype=torch.int32)  # noqa: E731
    first, steps, refused = state(), {}, []
    for n, rows in (((9, 3), 12), ((1, 1), 2), ((0, 40), 40), ((1, 1), 2), ((7, 0), 12)):
        refused.append(cache.plan(new(*n), rows))
        assert state() == first
        step = [cache.cu_rows.data_ptr(), cache.slots.data_ptr()]
        assert steps.setdefault(rows, step) == step and cache.slots.numel() == rows
    assert cache.kv_lens.tolist() == [18, 5] and cache.n_free.tolist() == [3]
    assert [r.tolist() for r in refused] == [[0], [0], [1], [0], [0]]  # each step's own
    cache.release(0)
    assert state() == first
    assert cache.kv_lens.tolist() == [0, 5] and cache.n_free.tolist() == [6]
    held = cache.block_table[1, :1].tolist()
    assert sorted(cache.free_pages[:6].tolist() + held) == list(range(7))


def test_the_references_agree_with_hand_values():
    # two keys, logits 0 and ln 3: weights 1/4 and 3/4; the first row sees the first key alone
    q = torch.zeros(2, 1, 64)
    q[:, 0, 0] = 1.0
    k, v = torch.zeros(2, 1, 64), torch.zeros(2, 1, 64)
    k[1, 0, 0] = 1.0986122886681098
    v[0], v[1] = 4.0, 8.0
    o, lse, _ = ref.attention(q, [k], [v], [0, 2], [2], 1, 1.0)
    assert torch.allclose(o[:, 0, 0], torch.tensor([4.0, 7.0], dtype=torch.float64), atol=1e-6)
    assert torch.allclose(lse[:, 0], torch.tensor([0.0, 1.3862943611], dtype=torch.float64), atol=1e-6)
    # three pages of 8: 5 + 4 positions need a second page, taken from the end of the free list
    got = ref.plan([5, 0], [4, 1], [11, 12, 13], 3, [[7, -1], [-1, -1]], 8, 6)
    assert got == ([[7, 13], [12, -1]], [0, 4, 5], [9, 1], [61, 62, 63, 104, 96, -1], [1, 0])
