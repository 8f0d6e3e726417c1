"""Streaming operators on the GPU: cache plan, cache append, attention over
the paged cache and the gated residual + norm, against plain references
(tests/streaming_ref.py: whole numbers one sequence after another, the
attention and the norms in 64 bits).

Tolerances, by arithmetic:
 * attention: P is rounded to bf16 (each p off by at most 2^-8 of itself) and
   so is O; the exponentials are off by at most 7.5e-5, twice (P and the sum);
   a logit is an fp32 sum of 64 exact products, off by at most 64 * 2^-24 *
   sum |q k| * scale, 2e-5 at unit normals and 1.2e-4 at 6-fold logits, again
   twice.  With A = sum p |v| / l: |O - ref| <= 2^-8 (|ref| + A) + 2 * (7.5e-5
   + 1.2e-4) A + second order <= 2^-8 (1.01 |ref| + 1.12 A).
 * lse: 7.5e-5 + 1.2e-4 + fp32 roundings of a few 2^-24 |lse| and of the
   offset (below 2^8 in log2 units: 2^-16 ln 2): 2.2e-4 + 1e-6 |lse|.
 * norm: fp32 arithmetic on at most 8192 values, then one rounding to bf16
   (2^-8) or to fp32; see norm_tolerance.
"""
import numpy as np
import pytest
import torch

import streaming_ref as ref
from feed_forward_view_vggt_b200 import attn

pytestmark = pytest.mark.gpu
D = 64


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def ok():
    assert attn.vggt_check()[0] == attn.VGGT_OK


# ------------------------------------------------------------------- plan

PLANS = [  # cached, new, page, n_rows, free pages, columns
    ([0], [1], 8, 1, 1, 1),
    ([5495], [1], 64, 1, 3, 90),
    ([1374, 0, 2748], [1374, 1374, 0], 128, 2748, 60, 40),
    ([3, 8, 15, 16, 0, 0], [5, 1, 1, 1, 0, 17], 8, 40, 9, 6),       # pages that end exactly, empty sequences
    ([0, 0, 0, 40], [20, 30, 0, 8], 8, 64, 5, 8),                   # the second one does not fit the free pages
    ([0, 0, 0], [8, 8, 7], 8, 23, 3, 1),
    ([0, 0, 0], [8, 8, 7], 8, 22, 3, 1),                            # the last one's rows end behind n_rows
    ([60, 4], [8, 4], 8, 16, 9, 8),                                 # the first one needs more columns
    ([-3, 5], [4, -9], 16, 8, 4, 3),                                # negative lengths count as 0
    ([7, 9], [1, 1], 16, 2, 0, 2),                                  # nothing free, nothing needed
    ([7, 16], [1, 1], 16, 2, 0, 2),                                 # nothing free, a page needed
]


def run_plan(cached, new, page, n_rows, n_free, width, seed=0, slack=2):
    g = torch.Generator().manual_seed(seed)
    n_pages = sum(min(width, -(-max(c, 0) // page)) for c in cached) + n_free + 4
    order = torch.randperm(n_pages, generator=g).tolist()
    table = [[order.pop() if i < -(-max(c, 0) // page) else -7 for i in range(width)] for c in cached]
    free = order + [0] * slack
    n_free = min(n_free, len(order))
    want = ref.plan(cached, new, free, n_free, table, page, n_rows)
    dev = i32(table)
    cu, kv, slots, counts = attn.cache_plan(i32(cached), i32(new), i32(free), i32([n_free]), dev, page, n_rows)
    ok()
    for got, exp, name in zip((dev, cu, kv, slots, counts), want, ("table", "cu_rows", "kv_lens", "slots", "counts")):
        assert np.array_equal(got.cpu().numpy(), np.array(exp, dtype=np.int32).reshape(got.shape)), name


@pytest.mark.parametrize("case", PLANS, ids=range(len(PLANS)))
def test_plan_matches_the_plain_one(case):
    run_plan(*case)


@pytest.mark.parametrize("seqs,page,most,seed", [(4096, 16, 60, 1), (700, 8, 300, 2), (257, 48, 900, 3), (33, 128, 4000, 4)])
def test_plan_of_many_sequences(seqs, page, most, seed):
    rng = np.random.default_rng(seed)
    cached = rng.integers(0, most, seqs).tolist()
    new = (rng.integers(0, most, seqs) * (rng.random(seqs) < 0.7)).astype(int).tolist()
    need = sum(-(-(c + n) // page) - -(-c // page) for c, n in zip(cached, new))
    width = -(-2 * most // page)
    run_plan(cached, new, page, sum(new) + 13, need + 1, width, seed)
    run_plan(cached, new, page, sum(new) + 13, need - need // 3, width, seed)   # the last third is refused
    run_plan(cached, new, page, sum(new) * 2 // 3, need, width, seed)           # rows cut


def test_plan_cuts_a_free_count_outside_the_list():
    for n_free, left in ((-4, 0), (99, 6)):
        table = i32([[-7, -7]])
        counts = attn.cache_plan(i32([0]), i32([0]), i32([0, 1, 2, 3, 4, 5]), i32([n_free]), table, 8, 4)[3]
        assert counts.tolist() == [left, 0]


def test_plan_never_gives_a_slot_outside_the_cache():
    # the table's own entry and a free page that the cache does not have
    table = i32([[9, -7], [1, -7]])
    cu, kv, slots, counts = attn.cache_plan(i32([4, 8]), i32([2, 1]), i32([50]), i32([1]), table, 8, 3, n_pages=4)
    assert slots.tolist() == [-1, -1, -1] and counts.tolist() == [0, 0]


# ----------------------------------------------------------------- append

@pytest.mark.parametrize("layout", ["head", "token", "both"])
@pytest.mark.parametrize("rows,heads,page", [(1, 1, 8), (5, 3, 24), (333, 16, 128), (70, 64, 16)])
def test_append(layout, rows, heads, page):
    b = ref.Batch([rows + 9], [0], page, heads, heads, layout=layout, extra=4)
    g = torch.Generator(device="cuda").manual_seed(3)
    both = torch.randn(rows, 3, heads, D, generator=g, device="cuda").bfloat16()
    k, v = both[:, 1], both[:, 2]  # slices of one projection's rows
    n_slots = b.k_pages.shape[0] * page
    slots = torch.randperm(n_slots, generator=torch.Generator().manual_seed(4))[:rows].int()
    slots[rows // 2] = -1
    want_k, want_v = b.k_pages.clone(), b.v_pages.clone()
    for r, s in enumerate(slots.tolist()):
        if s >= 0:
            want_k[s // page, :, s % page] = k[r]
            want_v[s // page, :, s % page] = v[r]
    attn.cache_append(k, v, slots.cuda(), b.k_pages, b.v_pages)
    ok()
    for got, exp in ((b.k_pages, want_k), (b.v_pages, want_v)):
        assert torch.equal(got.contiguous().view(torch.int16), exp.contiguous().view(torch.int16))


def test_append_of_one_row_and_one_page_of_other_strides():
    heads, page = 3, 8
    g = torch.Generator(device="cuda").manual_seed(8)
    r = lambda *n: torch.randn(*n, generator=g, device="cuda").bfloat16()  # noqa: E731
    k, v = r(1, heads, D), r(1, 3, heads, D)[:, 1]
    k_pages, v_all = r(1, heads, page, D), r(7, 2, heads, page, D)
    v_pages = v_all[3:4, 1]
    want_k, want_v = k_pages.clone(), v_all.clone()
    want_k[0, :, 5], want_v[3, 1, :, 5] = k[0], v[0]
    attn.cache_append(k, v, i32([5]), k_pages, v_pages)
    got = attn.cached(k, k_pages, v_pages, i32([[0]]), i32([0, 1]), i32([6]))
    ok()
    assert torch.equal(k_pages, want_k) and torch.equal(v_all, want_v)
    want, _, spread = ref.attention(k, [want_k[0].transpose(0, 1)], [want_v[3, 1].transpose(0, 1)], [0, 1], [6], 0)
    assert ((got.double() - want).abs() <= 2.0 ** -8 * (1.01 * want.abs() + 1.12 * spread) + 1e-30).all()


@pytest.mark.parametrize("unit", [0, 1, 2 ** 31 - 1])
def test_head_major_rows(unit):
    # q, k and v as [heads, rows, 64]: rows lie 64 elements apart, heads further
    b = ref.Batch([300, 41], [37, 2], 16, 6, 3, seed=12)
    g = torch.Generator(device="cuda").manual_seed(2)
    k, v = (torch.randn(3, 39, D, generator=g, device="cuda").bfloat16().transpose(0, 1) for _ in range(2))
    slots = torch.tensor([b.table[i, t // 16].item() * 16 + t % 16 for i, (n, m) in enumerate(zip(b.kv, b.new))
                          for t in range(n - m, n)], dtype=torch.int32, device="cuda")
    attn.cache_append(k, v, slots, b.k_pages, b.v_pages)
    for i in range(2):
        for seqs, x in ((b.k_seqs, k), (b.v_seqs, v)):
            seqs[i][b.kv[i] - b.new[i]:] = x[b.cu[i]:b.cu[i + 1]]
    q = b.q.transpose(0, 1).contiguous().transpose(0, 1)
    got, lse = attn.cached(q, b.k_pages, b.v_pages, b.table, b.cu_rows, b.kv_lens, causal_unit=unit, want_lse=True)
    ok()
    check_attention(b, unit, got, lse)


def test_append_reports_and_skips_a_slot_outside_the_cache():
    k_pages, v_pages = (torch.zeros(2, 2, 8, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    k = torch.ones(3, 2, D, dtype=torch.bfloat16, device="cuda")
    attn.cache_append(k, k, i32([16, 3, 2 ** 31 - 1]), k_pages, v_pages)
    assert attn.vggt_check()[0] == attn.VGGT_ERR_BOUNDS
    assert k_pages.sum().item() == 2 * D and (k_pages[0, :, 3] == 1).all() and torch.equal(k_pages, v_pages)
    ok()


# -------------------------------------------------------------- attention

def check_attention(b, unit, got, lse=None, scale=None, logit_error=0.0):
    """logit_error: what a logit may be off beyond the 1.2e-4 counted above; it enters P and the sum."""
    o, want_lse, spread = b.reference(unit, scale)
    n = b.cu[-1]
    err = (got.double() - o).abs()[:n]
    tol = (2.0 ** -8 * (1.01 * o.abs() + 1.12 * spread) + 2 * logit_error * spread + 1e-30)[:n]
    assert torch.isfinite(got[:n].float()).all()
    worst = (err / tol).max().item() if n else 0.0
    assert worst <= 1.0, worst
    if lse is not None:
        fin = torch.isfinite(want_lse[:n])
        assert torch.equal(torch.isneginf(lse[:n]), ~fin)
        e = (lse[:n].double() - want_lse[:n]).abs()[fin]
        assert (e <= 2.2e-4 + logit_error + 1e-6 * want_lse[:n][fin].abs()).all(), e.max().item()


CASES = [  # kv lengths, new rows, page, heads, kv heads, unit
    ([1], [1], 8, 1, 1, 1),
    ([5496], [1], 64, 16, 16, 1),
    ([127, 128, 129], [1, 1, 1], 16, 4, 4, 1),
    ([15, 16, 17, 1, 255, 256, 257], [1, 1, 1, 1, 1, 1, 1], 8, 8, 2, 0),
    ([1000, 3, 0, 2500], [1, 1, 1, 1], 24, 32, 4, 1),               # a sequence without keys
    ([700, 20000, 90], [1, 1, 1], 16, 8, 1, 1),                     # one long sequence among short ones
    ([300, 411], [0, 77], 48, 12, 4, 1),                            # a sequence without new rows
    ([77, 300, 129, 641], [77, 128, 129, 300], 16, 6, 6, 1),        # first chunks among later ones
    ([1000, 517], [256, 257], 40, 4, 2, 1),
    ([2048], [2048], 128, 2, 2, 1),
    ([690], [345], 32, 4, 4, 69),                                   # causal by frame
    ([69 * 9, 69 * 4 + 5], [69 * 3, 69 + 5], 16, 4, 4, 69),         # a part of a frame at the end
    ([4122], [1374], 1376, 2, 2, 1374),
    ([900, 40], [33, 700], 16, 4, 4, 0),                            # more rows than keys, every key seen
    ([30, 500], [50, 20], 16, 3, 1, 1),                             # rows before the first position see nothing
    ([800], [9], 16, 64, 1, 1),                                     # one key head for 64 query heads
    ([800, 33], [50, 3], 16, 21, 3, 7),                             # groups of 7: 18 tokens in a tile
    ([3000], [600], 256, 40, 8, 1),
]


@pytest.mark.parametrize("case", CASES, ids=range(len(CASES)))
def test_attention_matches_64_bits(case):
    kv, new, page, heads, kv_heads, unit = case
    b = ref.Batch(kv, new, page, heads, kv_heads, seed=11, pad=5)
    o = torch.full_like(b.q, 9.0)
    got, lse = attn.cached(b.q, b.k_pages, b.v_pages, b.table, b.cu_rows, b.kv_lens, causal_unit=unit, want_lse=True,
                           o=o)
    ok()
    check_attention(b, unit, got, lse)
    assert (got[b.cu[-1]:] == 9.0).all()  # rows behind the last sequence


@pytest.mark.parametrize("kv,new,heads,kv_heads,unit", [([20003], [1374], 16, 16, 0), ([20003], [1374], 16, 16, 1),
                                                        ([9001, 5000], [1000, 641], 16, 4, 0),
                                                        ([9001, 5000], [1000, 641], 16, 4, 641)])
def test_attention_when_shares_are_long(kv, new, heads, kv_heads, unit):
    """Every CTA has many key tiles of several units and takes them in an order of its own, the odd last tile in
    between."""
    b = ref.Batch(kv, new, 64, heads, kv_heads, seed=12)
    got, lse = attn.cached(b.q, b.k_pages, b.v_pages, b.table, b.cu_rows, b.kv_lens, causal_unit=unit, want_lse=True)
    ok()
    check_attention(b, unit, got, lse)


@pytest.mark.parametrize("heads,kv_heads,unit,seed", [(16, 8, 1, 1), (4, 4, 0, 2), (16, 1, 30, 3), (21, 3, 1, 4)])
def test_attention_of_many_sequences_of_every_kind(heads, kv_heads, unit, seed):
    """Several hundred sequences, so that every CTA works through many tasks: single tokens, a few rows, one tile,
    an odd and an even number of tiles, rows without keys, and long runs of sequences without any."""
    rng = np.random.default_rng(seed)
    new, kv = [], []
    for _ in range(260):
        n = int(rng.choice([0, 1, 1, 1, 2, 5, 17, 60, 130, 260, 400]))
        new.append(n)
        kv.append(int(rng.choice([0, max(0, n - 3), n, n + int(rng.integers(0, 500)), int(rng.integers(1, 40))])))
    new[100:100] = [2] * 2600
    kv[100:100] = [0] * 2600
    b = ref.Batch(kv, new, 16, heads, kv_heads, seed=seed)
    got, lse = attn.cached(b.q, b.k_pages, b.v_pages, b.table, b.cu_rows, b.kv_lens, causal_unit=unit, want_lse=True)
    ok()
    check_attention(b, unit, got, lse)


@pytest.mark.parametrize("layout", ["token", "both"])
@pytest.mark.parametrize("unit", [0, 1, 50])
def test_attention_over_other_cache_layouts_and_strided_queries(layout, unit):
    b = ref.Batch([450, 37, 260], [200, 1, 130], 24, 6, 2, seed=5, layout=layout)
    wide = torch.zeros(b.rows, 3, 6, D, dtype=torch.bfloat16, device="cuda")
    wide[:, 1] = b.q
    got = attn.cached(wide[:, 1], b.k_pages, b.v_pages, b.table, b.cu_rows, b.kv_lens, causal_unit=unit)
    same = attn.cached(b.q, b.k_pages, b.v_pages, b.table, b.cu_rows, b.kv_lens, causal_unit=unit)
    ok()
    check_attention(b, unit, got)
    assert torch.equal(got, same)


@pytest.mark.parametrize("q_scale,scale", [(6.0, None), (1.0, 0.03), (0.0, None)])
def test_attention_at_other_logit_sizes(q_scale, scale):
    b = ref.Batch([1500, 600], [140, 1], 16, 4, 2, seed=8, q_scale=q_scale)
    got, lse = attn.cached(b.q, b.k_pages, b.v_pages, b.table, b.cu_rows, b.kv_lens, causal_unit=1, scale=scale,
                           want_lse=True)
    ok()
    check_attention(b, 1, got, lse, scale)


@pytest.mark.parametrize("new", [1, 200])
def test_attention_when_later_keys_raise_the_maximum(new):
    # keys grow along the sequence, so the running maximum moves many times
    b = ref.Batch([1300], [new], 16, 4, 4, seed=9)
    ramp = torch.linspace(0.05, 6.0, 1300, device="cuda")[:, None, None]
    b.k_seqs[0] = (b.k_seqs[0] * ramp).bfloat16()
    table = b.table[0].tolist()
    for t in range(1300):
        b.k_pages[table[t // 16], :, t % 16] = b.k_seqs[0][t]
    got, lse = attn.cached(b.q, b.k_pages, b.v_pages, b.table, b.cu_rows, b.kv_lens, want_lse=True)
    ok()
    check_attention(b, 0, got, lse)


@pytest.mark.parametrize("at", [640, 643, 645, 655, 1299])
@pytest.mark.parametrize("new,alike", [(1, True), (5, False), (200, True), (200, False)])
def test_attention_when_one_late_key_outweighs_all(new, alike, at):
    # its logits are hundreds above (of unlike rows: or below) those of the tiles before, where 2^x against the old
    # offset has no value; alike, no other row of a warp notices
    b = ref.Batch([1300], [new], 16, 4, 4, seed=9)
    if alike:
        b.q[:] = b.q[0].clone()
    b.k_seqs[0][at] = 40 * b.q[0].float()
    table = b.table[0].tolist()
    b.k_pages[table[at // 16], :, at % 16] = b.k_seqs[0][at]
    got, lse = attn.cached(b.q, b.k_pages, b.v_pages, b.table, b.cu_rows, b.kv_lens, want_lse=True)
    ok()
    # an fp32 sum of 64 exact products
    most = (b.q.double().abs() * b.k_seqs[0][at].double().abs()).sum(-1).max().item() * D ** -0.5
    check_attention(b, 0, got, lse, logit_error=64 * 2.0 ** -24 * most)


@pytest.mark.parametrize("kv,new,kv_heads", [([5000], [1], 1), ([3000, 2500], [1, 3], 1), ([20000], [50], 16),
                                             ([20000], [8], 16), ([9000, 12000], [130, 50], 16), ([5000], [5], 1)])
def test_attention_does_not_depend_on_rows_of_no_sequence(kv, new, kv_heads):
    """Groups of 3: a tile holds rows of other tokens and rows of no token.  Whatever q holds behind the last
    sequence, and whatever an earlier call left in shared memory, the sequences' results keep their bits."""
    b = ref.Batch(kv, new, 16, 3 * kv_heads, kv_heads, seed=14, pad=60)
    for i, n in enumerate(kv):  # keys that grow along every thousand, so the offsets move
        ramp = 0.05 + 2.95 * (torch.arange(n, device="cuda") % 1000) / 1000
        b.k_seqs[i] = (b.k_seqs[i] * ramp[:, None, None]).bfloat16()
        table = b.table[i].tolist()
        for page in range(-(-n // 16)):
            part = b.k_seqs[i][16 * page:16 * page + 16]
            b.k_pages[table[page], :, :len(part)] = part.transpose(0, 1)
    call = lambda: attn.cached(b.q, b.k_pages, b.v_pages, b.table, b.cu_rows, b.kv_lens)  # noqa: E731
    b.q[b.cu[-1]:] = 0
    want = call()
    ok()
    check_attention(b, 0, want)
    unlike = torch.randn(60, 3 * kv_heads, D, generator=torch.Generator().manual_seed(1)).cuda()
    for fill in (30 * unlike, 3000 * unlike, torch.full_like(unlike, float("nan"))):
        b.q[b.cu[-1]:] = fill.bfloat16()
        assert torch.equal(call()[:b.cu[-1]], want[:b.cu[-1]])
    ok()


def test_attention_skips_and_reports_a_page_outside_the_cache():
    b = ref.Batch([400, 300], [3, 4], 16, 2, 2, seed=2)
    good = attn.cached(b.q, b.k_pages, b.v_pages, b.table, b.cu_rows, b.kv_lens)
    ok()
    for bad in (-1, b.k_pages.shape[0], 2 ** 31 - 1, -2 ** 31):
        table = b.table.clone()
        table[0, 5] = bad
        got = attn.cached(b.q, b.k_pages, b.v_pages, table, b.cu_rows, b.kv_lens)
        assert attn.vggt_check()[0] == attn.VGGT_ERR_BOUNDS
        assert torch.equal(got[3:], good[3:])  # the other sequence
    ok()


@pytest.mark.parametrize("cu", [[0, 5, 3, 9], [-1, 3, 4, 9], [0, 3, 4, 10], [0, 9, 0, 9]])
def test_attention_refuses_row_offsets_that_do_not_ascend(cu):
    b = ref.Batch([400, 300, 20], [3, 4, 2], 16, 2, 2, seed=2)
    o = torch.full_like(b.q, 5.0)
    attn.cached(b.q, b.k_pages, b.v_pages, b.table, i32(cu), b.kv_lens, o=o)
    assert attn.vggt_check()[0] == attn.VGGT_ERR_BOUNDS
    assert (o == 5.0).all()
    got = attn.cached(b.q, b.k_pages, b.v_pages, b.table, b.cu_rows, b.kv_lens, o=o)
    ok()
    check_attention(b, 0, got)


def test_attention_with_a_table_so_large_that_costs_are_counted_coarsely():
    # 2^27 positions per sequence and 12000 rows of 64 heads: the costs of the units could pass 31 bits
    b = ref.Batch([300, 2000], [12000, 40], 8, 64, 64, seed=6)
    table = torch.full((2, 1 << 24), -7, dtype=torch.int32, device="cuda")
    table[:, :b.table.shape[1]] = b.table
    got, lse = attn.cached(b.q, b.k_pages, b.v_pages, table, b.cu_rows, b.kv_lens, want_lse=True)
    ok()
    check_attention(b, 0, got, lse)


@pytest.mark.parametrize("active", [{0: 300}, {4000: 600}, {17: 2000}, {5: 300, 4095: 2000}, {0: 600, 1: 300}])
@pytest.mark.parametrize("heads,kv_heads,new", [(16, 16, 1), (64, 16, 200)])
def test_attention_of_little_work_in_buffers_of_full_size(active, heads, kv_heads, new):
    """4096 sequences in a table for 2^22 positions, a few of them active: costs are counted in fours of steps and
    there are fewer of those than CTAs.  What the workspace held before must not reach a result."""
    seqs, rows, page, width = 4096, 4096, 1 << 17, 32
    g = torch.Generator(device="cuda").manual_seed(4)
    k_pages, v_pages = (torch.full((len(active), kv_heads, page, D), float("nan"), dtype=torch.bfloat16, device="cuda")
                        for _ in range(2))
    q = torch.randn(rows, heads, D, generator=g, device="cuda").bfloat16()
    kv, fresh = [0] * seqs, [0] * seqs
    ks, vs = [], []
    table = torch.full((seqs, width), -7, dtype=torch.int32, device="cuda")
    for i, (b, n) in enumerate(active.items()):
        kv[b], fresh[b] = n, new
        k_pages[i, :, :n] = torch.randn(kv_heads, n, D, generator=g, device="cuda").bfloat16()
        v_pages[i, :, :n] = torch.randn(kv_heads, n, D, generator=g, device="cuda").bfloat16()
        ks.append(k_pages[i, :, :n].transpose(0, 1))
        vs.append(v_pages[i, :, :n].transpose(0, 1))
        table[b, 0] = i
    cu = np.concatenate([[0], np.cumsum(fresh)]).tolist()
    cache = attn.vggt_cache(seqs, heads, kv_heads, D, page, len(active), width, *k_pages.stride()[:3])
    ws = torch.empty(attn.vggt_attn_cached_workspace_bytes(cache, rows), dtype=torch.uint8, device="cuda")
    ends = [new * i for i in range(len(active) + 1)]
    want, _, spread = ref.attention(q, ks, vs, ends, list(active.values()), 1)
    for fill in (0xff, 0x7f):  # NaN, and 3e38
        ws.fill_(fill)
        got = attn.cached(q, k_pages, v_pages, table, i32(cu), i32(kv), causal_unit=1, workspace=ws)
        ok()
        n = cu[-1]
        tol = 2.0 ** -8 * (1.01 * want.abs() + 1.12 * spread) + 1e-30
        assert ((got.double() - want).abs() <= tol)[:n].all()


def test_append_and_attention_past_four_gigabytes_of_pages():
    pages, heads, page = 9000, 16, 256  # 4.7 GB of keys
    k_pages, v_pages = (torch.empty(pages, heads, page, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    kv, g = 700, torch.Generator(device="cuda").manual_seed(3)
    k, v, q = (torch.randn(kv, heads, D, generator=g, device="cuda").bfloat16() for _ in range(3))
    table = i32([[pages - 1, 0, pages - 3, 5]])
    t = torch.arange(kv, device="cuda")
    slots = (table[0, t // page].long() * page + t % page).int()
    attn.cache_append(k, v, slots, k_pages, v_pages)
    got = attn.cached(q[-20:], k_pages, v_pages, table, i32([0, 20]), i32([kv]), causal_unit=1)
    ok()
    want, _, spread = ref.attention(q[-20:], [k], [v], [0, 20], [kv], 1)
    assert ((got.double() - want).abs() <= 2.0 ** -8 * (1.01 * want.abs() + 1.12 * spread) + 1e-30).all()


def test_norm_past_two_to_the_31_elements():
    rows, cols = 270000, 8192
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    x[-3:] = torch.randn(3, cols, device="cuda").bfloat16()
    _, h = attn.norm_residual(x, eps=1e-6)
    ok()
    want = ref.normed(x[-3:].double(), "layer", 1e-6, None, None)
    assert ((h[-3:].double() - want).abs() <= norm_tolerance(2, "layer", 1e-6, want, torch.bfloat16)).all()
    assert (h[:3] == 0).all()


def test_calls_without_rows():
    b = ref.Batch([40, 0], [0, 0], 16, 4, 2, seed=2)
    got, lse = attn.cached(b.q, b.k_pages, b.v_pages, b.table, b.cu_rows, b.kv_lens, want_lse=True)
    assert got.shape == (0, 4, D) and lse.shape == (0, 4)
    attn.cache_append(b.q[:, :2], b.q[:, :2], i32([]), b.k_pages, b.v_pages)
    x, h = attn.norm_residual(torch.zeros(0, 64, device="cuda"), torch.zeros(0, 64, device="cuda").bfloat16())
    assert x.shape == h.shape == (0, 64)
    # rows of the buffer, none of a sequence
    o = torch.full((7, 4, D), 3.0, device="cuda").bfloat16()
    attn.cached(o.clone(), b.k_pages, b.v_pages, b.table, b.cu_rows, b.kv_lens, o=o)
    ok()
    assert (o == 3.0).all()


def test_calls_on_another_stream_than_the_current_one():
    """Inputs made on the current stream, a call on another one that waits for it, results read on the current one:
    twice at once, so that the buffers of both calls are in flight together."""
    side = torch.cuda.Stream()
    b = ref.Batch([700, 300, 41], [1, 150, 2], 16, 8, 2, seed=4)
    x = torch.randn(500, 256, device="cuda")
    y = torch.randn(500, 256, device="cuda").bfloat16()
    want_x, want_h = attn.norm_residual(x, y)
    want_o = attn.cached(b.q, b.k_pages, b.v_pages, b.table, b.cu_rows, b.kv_lens, causal_unit=1)
    table = b.table.clone()
    plan_args = (i32([700, 300, 41]), i32([1, 150, 2]), i32(list(range(30))), i32([30]))
    want_plan = attn.cache_plan(*plan_args, table.clone(), 16, 160)
    for _ in range(5):
        side.wait_stream(torch.cuda.current_stream())
        got = attn.norm_residual(x, y, stream=side)
        raw = attn.cached(b.q, b.k_pages, b.v_pages, b.table, b.cu_rows, b.kv_lens, causal_unit=1,
                          stream=side.cuda_stream)
        scratch = [torch.full((500, 256), float("nan"), device="cuda") for _ in range(8)]
        plan = attn.cache_plan(*plan_args, table.clone(), 16, 160, stream=side)
        del scratch
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(got[0], want_x) and torch.equal(got[1], want_h) and torch.equal(raw, want_o)
        assert all(torch.equal(p, q) for p, q in zip(plan, want_plan))
    ok()


def test_norm_and_append_replay():
    x, y = torch.randn(40, 768, device="cuda"), torch.randn(40, 768, device="cuda").bfloat16()
    b = ref.Batch([64], [0], 16, 2, 2)
    k, slots = torch.randn(4, 2, D, device="cuda").bfloat16(), i32([3, 60, -1, 17])
    graph = torch.cuda.CUDAGraph()
    attn.norm_residual(x, y)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got_x, got_h = attn.norm_residual(x, y)
        attn.cache_append(k, k, slots, b.k_pages, b.v_pages)
    for seed in (1, 2):
        torch.manual_seed(seed)
        x.normal_()
        y.copy_(torch.randn(40, 768))
        k.copy_(torch.randn(4, 2, D))
        graph.replay()
        want_x, want_h = attn.norm_residual(x, y)
        assert torch.equal(got_x, want_x) and torch.equal(got_h, want_h)
        for r, s in ((0, 3), (1, 60), (3, 17)):
            assert torch.equal(b.k_pages[s // 16, :, s % 16], k[r]) and torch.equal(b.v_pages[s // 16, :, s % 16], k[r])
    ok()


def test_attention_is_repeatable_and_runs_on_two_streams_at_once():
    a = ref.Batch([9000, 41, 700], [1, 1, 1], 16, 16, 4, seed=21)
    c = ref.Batch([1374 * 3], [1374], 128, 4, 4, seed=22)
    want_a = attn.cached(a.q, a.k_pages, a.v_pages, a.table, a.cu_rows, a.kv_lens, causal_unit=1)
    want_c = attn.cached(c.q, c.k_pages, c.v_pages, c.table, c.cu_rows, c.kv_lens, causal_unit=1374)
    torch.cuda.synchronize()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(4):
        got_a = attn.cached(a.q, a.k_pages, a.v_pages, a.table, a.cu_rows, a.kv_lens, causal_unit=1, stream=s)
        got_c = attn.cached(c.q, c.k_pages, c.v_pages, c.table, c.cu_rows, c.kv_lens, causal_unit=1374, stream=t)
        torch.cuda.synchronize()
        assert torch.equal(got_a, want_a) and torch.equal(got_c, want_c)
    ok()


def test_attention_replays_with_the_lengths_of_the_replay():
    b = ref.Batch([2000, 500], [1, 1], 16, 8, 2, seed=31)
    o, ws = torch.empty_like(b.q), None
    cache = attn.vggt_cache(2, 8, 2, D, 16, b.k_pages.shape[0], b.table.shape[1], *b.k_pages.stride()[:3])
    ws = torch.empty(max(256, attn.vggt_attn_cached_workspace_bytes(cache, 2)), dtype=torch.uint8, device="cuda")
    call = lambda: attn.cached(b.q, b.k_pages, b.v_pages, b.table, b.cu_rows, b.kv_lens, causal_unit=1, o=o,  # noqa: E731
                               workspace=ws)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for kv in ([2000, 500], [1, 499], [130, 0], [1999, 16]):
        b.kv = kv
        b.kv_lens.copy_(i32(kv))
        o.fill_(7.0)
        graph.replay()
        ok()
        check_attention(b, 1, o)


# ------------------------------------------------------------------- norm

def norm_tolerance(s, kind, eps, want, out_type):
    """An fp32 mean or mean square of n values summed in a tree over at most 32 values a thread: relative 48 *
    2^-24; the factors add a few roundings of 2^-24 each; all act on numbers up to t, the row's largest term
    before cancellation.  64 * 2^-24 of (|value| + the row's largest), then the rounding of the output."""
    u = 2.0 ** -24
    top = want.abs().amax(-1, keepdim=True)
    half = torch.finfo(out_type).eps / 2
    return 64 * u * (want.abs() + top) * s + half * (1 + 1e-3) * want.abs() + 1e-30


NORMS = [  # rows, cols, type of x, kind, post, gate rows, scale, biases, y
    (1, 8, torch.float32, "layer", False, 0, True, True, True),
    (17, 1024, torch.float32, "layer", False, 0, True, True, True),
    (5, 1000, torch.bfloat16, "layer", True, 2, True, True, True),
    (333, 768, torch.bfloat16, "rms", True, 100, True, False, True),
    (64, 64, torch.float32, "rms", False, 1, False, False, True),
    (9, 2048, torch.float32, "layer", True, 4, True, True, True),
    (7, 4096, torch.bfloat16, "rms", False, 0, True, True, True),
    (3, 8192, torch.float32, "layer", True, 3, True, True, True),
    (2, 8184, torch.bfloat16, "layer", False, 0, False, False, True),
    (129, 256, torch.float32, "rms", False, 0, False, False, False),
    (130, 264, torch.bfloat16, "layer", False, 0, False, True, False),
    (1374, 512, torch.float32, "layer", False, 1374, False, True, True),
]


@pytest.mark.parametrize("case", NORMS, ids=range(len(NORMS)))
@pytest.mark.parametrize("inplace", [False, True])
def test_norm_residual(case, inplace):
    rows, cols, xt, kind, post, gate_rows, scaled, biases, has_y = case
    g = torch.Generator(device="cuda").manual_seed(rows + cols)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x = (2 * r(rows, cols) + 0.5).to(xt)
    y = r(rows, 2, cols).bfloat16()[:, 1] if has_y else None  # a strided block output
    scale = r(cols) if scaled and has_y else None
    gate = r(-(-rows // gate_rows), cols).bfloat16() if gate_rows else None
    pw, pb = (1 + 0.2 * r(cols), 0.1 * r(cols) if biases else None) if post else (None, None)
    w, b = 1 + 0.2 * r(cols), 0.1 * r(cols) if biases else None
    want_x = x.double()
    if has_y:
        add = y.double()
        add = ref.normed(add, kind, 1e-5, pw, pb) if post else add
        add = add * scale.double() if scale is not None else add
        add = add * gate.double().repeat_interleave(gate_rows, 0)[:rows] if gate is not None else add
        want_x = want_x + add
    want_h = ref.normed(want_x, kind, 1e-5, w, b)
    got_x, got_h = attn.norm_residual(x, y, kind=kind, eps=1e-5, scale=scale, gate=gate, rows_per_gate=gate_rows,
                                      post_norm=post, post_weight=pw, post_bias=pb, weight=w, bias=b,
                                      inplace=inplace)
    ok()
    if inplace or not has_y:
        assert got_x is x
    if has_y:
        assert ((got_x.double() - want_x).abs() <= norm_tolerance(2, kind, 1e-5, want_x, xt)).all()
    # x' of h is fp32: its own error enters N once more
    err = (got_h.double() - want_h).abs()
    tol = norm_tolerance(4, kind, 1e-5, want_h, torch.bfloat16)
    assert (err <= tol).all(), (err / tol).max().item()


def test_norm_residual_without_h_and_of_a_constant_row():
    x = torch.full((3, 128), 7.0, device="cuda")
    y = torch.full((3, 128), 2.0, device="cuda").bfloat16()
    got, h = attn.norm_residual(x, y, want_h=False)
    assert h is None and (got == 9.0).all()
    got, h = attn.norm_residual(x, y, eps=1e-6)
    assert (h == 0).all()  # no variance: (t - mean) is 0
    got, h = attn.norm_residual(x, y, kind="rms", eps=0.0)
    assert (h == 1).all()
    ok()


@pytest.mark.parametrize("xt,rows,cols", [(torch.float32, 300, 520), (torch.bfloat16, 9, 2048)])
@pytest.mark.parametrize("inplace", [False, True])
def test_norm_residual_of_a_strided_stream(xt, rows, cols, inplace):
    g = torch.Generator(device="cuda").manual_seed(3)
    wide = torch.randn(rows, 2, cols, generator=g, device="cuda").to(xt)
    x, beside = wide[:, 1], wide[:, 0].clone()
    y = torch.randn(rows, cols, generator=g, device="cuda").bfloat16()
    want_x = x.double() + y.double()
    want_h = ref.normed(want_x, "rms", 1e-6, None, None)
    got, h = attn.norm_residual(x, y, kind="rms", inplace=inplace)
    ok()
    assert (got is x) == inplace and torch.equal(wide[:, 0], beside)
    assert ((got.double() - want_x).abs() <= norm_tolerance(2, "rms", 1e-6, want_x, xt)).all()
    assert ((h.double() - want_h).abs() <= norm_tolerance(4, "rms", 1e-6, want_h, torch.bfloat16)).all()


def test_norm_residual_keeps_a_large_offset():
    # 1e4 + small: the variance is taken about the mean, so h still has the small part
    g = torch.Generator(device="cuda").manual_seed(1)
    x = 1e4 + torch.randn(8, 1024, generator=g, device="cuda")
    _, h = attn.norm_residual(x)
    want = ref.normed(x.double(), "layer", 1e-6, None, None)
    # the mean's fp32 rounding shifts every value by at most 2^-24 * 1e4 * a few
    assert ((h.double() - want).abs() <= 2.0 ** -8 * want.abs() + 40 * 2.0 ** -24 * 1e4).all()


# ------------------------------------------------------------ all together

def test_streamed_block_matches_the_whole_scene():
    """Two scenes, frames arriving over three steps, one block per step: norm, QKV projection, plan, append,
    attention causal by frame, output projection, residual and norm; the attention output of every step against
    the 64-bit attention over all of the scene's rows so far."""
    H, h, w, ns = 4, 5, 6, 5
    L, C = ns + h * w, H * D
    g = torch.Generator(device="cuda").manual_seed(77)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    wqkv, wo = (r(3 * C, C) / C ** 0.5).bfloat16(), (r(C, C) / C ** 0.5).bfloat16()
    ls, nw, nb = 0.1 * r(C), 1 + 0.1 * r(C), 0.1 * r(C)
    page, seqs = 16, 2
    cache = attn.PagedCache(n_pages=64, page_size=page, n_kv_heads=H, n_seqs=seqs, max_pages=24)
    kept = [[], []]
    for step, frames in enumerate(([1, 2], [2, 0], [1, 1])):
        new = [f * L for f in frames]
        rows = sum(new)
        x = r(rows, C)
        _, hid = attn.norm_residual(x, weight=nw, bias=nb)
        shape = attn.vggt_shape(sum(frames), ns, h, w, H, D)
        q, k, v = attn.qkv_rope(hid, wqkv, shape)
        refused = cache.plan(i32(new), rows)
        assert refused.item() == 0
        cache.append(0, k, v)
        o = cache.attend(0, q, causal_unit=L)
        y = attn.out_proj(o.view(rows, C), wo, shape)
        x2, hid2 = attn.norm_residual(x, y, scale=ls, weight=nw, bias=nb)
        ok()
        at = 0
        for b in range(seqs):
            kept[b].append((k[at:at + new[b]], v[at:at + new[b]]))
            at += new[b]
        ks = [torch.cat([a for a, _ in kept[b]]) for b in range(seqs)]
        vs = [torch.cat([a for _, a in kept[b]]) for b in range(seqs)]
        kv = [len(a) for a in ks]
        assert cache.kv_lens.tolist() == kv
        cu = [0, new[0], rows]
        want, _, spread = ref.attention(q, ks, vs, cu, kv, L)
        assert ((o.double() - want).abs() <= 2.0 ** -8 * (1.01 * want.abs() + 1.12 * spread) + 1e-30).all()
        want_x = x.double() + ls.double() * y.double()
        assert ((x2.double() - want_x).abs() <= norm_tolerance(2, "layer", 1e-6, want_x, torch.float32)).all()
        want_h = ref.normed(want_x, "layer", 1e-6, nw, nb)
        assert ((hid2.double() - want_h).abs() <= norm_tolerance(4, "layer", 1e-6, want_h, torch.bfloat16)).all()
    # a scene that ends gives its pages back, and another takes them
    before = int(cache.n_free)
    held = -(-int(cache.kv_lens[0]) // page)
    cache.release(0)
    assert int(cache.n_free) == before + held and int(cache.kv_lens[0]) == 0
    assert cache.plan(i32([17, 0]), 17).item() == 0
    assert int(cache.n_free) == before + held - 2
    in_use = cache.block_table[0, :2].tolist() + cache.block_table[1, :-(-int(cache.kv_lens[1]) // page)].tolist()
    free = cache.free_pages[:int(cache.n_free)].tolist()
    assert sorted(in_use + free) == list(range(64))


def test_a_refused_sequence_keeps_its_cache_and_leaves_the_others_alone():
    """Three scenes with 20, 9 and 0 cached positions; then only the second one's rows fit the free pages.  The refused
    one with a cache gets what its last cached positions see, the one without gets nothing."""
    heads = 2
    cache = attn.PagedCache(n_pages=5, page_size=8, n_kv_heads=heads, n_seqs=3, max_pages=9)
    g = torch.Generator(device="cuda").manual_seed(6)
    r = lambda n: torch.randn(n, heads, D, generator=g, device="cuda").bfloat16()  # noqa: E731
    k0, v0 = r(29), r(29)
    assert cache.plan(i32([20, 9, 0]), 29).item() == 0 and cache.n_free.item() == 0
    cache.append(0, k0, v0)
    before = [p.clone() for p in cache.pages[0]]
    new = [6, 3, 2]
    q, k, v = r(11), r(11), r(11)
    assert cache.plan(i32(new), 11).item() == 2
    assert cache.kv_lens.tolist() == [20, 12, 0] and cache.cu_rows.tolist() == [0, 6, 9, 11]
    assert (cache.slots[:6] == -1).all() and (cache.slots[9:] == -1).all()
    cache.append(0, k, v)
    got, lse = cache.attend(0, q, causal_unit=1, want_lse=True)
    ok()
    page = cache.block_table[1, 1].item()
    for now, was, x in zip(cache.pages[0], before, (k, v)):
        assert torch.equal(now[page, :, 1:4], x[6:9].transpose(0, 1))
        now[page, :, 1:4] = was[page, :, 1:4]
        assert torch.equal(now, was)
    ks, vs = ([torch.cat([a[:20], b[:0]]), torch.cat([a[20:], b[6:9]]), a[:0]] for a, b in ((k0, k), (v0, v)))
    want, want_lse, spread = ref.attention(q, ks, vs, [0, 6, 9, 11], [20, 12, 0], 1)
    assert ((got.double() - want).abs() <= 2.0 ** -8 * (1.01 * want.abs() + 1.12 * spread) + 1e-30).all()
    assert (got[9:] == 0).all() and torch.isneginf(lse[9:]).all()
    cache.release(0)  # its pages are still its own
    assert cache.n_free.item() == 3 and cache.plan(i32([0, 0, 2]), 2).item() == 0


class Scenes:
    """Sequences streamed through a PagedCache, and what their rows must give."""

    def __init__(self, cache, heads, seed=1):
        self.cache, self.heads, self.g = cache, heads, torch.Generator(device="cuda").manual_seed(seed)
        self.kept = [[] for _ in range(cache.kv_lens.numel())]

    def rows(self, n):
        return torch.randn(n, self.heads, D, generator=self.g, device="cuda").bfloat16()

    def check(self, new, q, k, v, got, unit=1):
        """After a step of ``new`` rows per sequence."""
        ends = [sum(new[:b]) for b in range(len(new) + 1)]
        for b, kept in enumerate(self.kept):
            kept.append((k[ends[b]:ends[b + 1]].clone(), v[ends[b]:ends[b + 1]].clone()))
        ks, vs = ([torch.cat([x[i] for x in kept]) for kept in self.kept] for i in (0, 1))
        kv = [len(x) for x in ks]
        assert self.cache.kv_lens.tolist() == kv
        want, _, spread = ref.attention(q[:ends[-1]], ks, vs, ends, kv, unit)
        tol = 2.0 ** -8 * (1.01 * want.abs() + 1.12 * spread) + 1e-30
        assert ((got[:ends[-1]].double() - want).abs() <= tol).all()


@pytest.mark.parametrize("whole", [True, False])
def test_a_captured_step_of_a_cache_goes_on_from_its_present_state(whole):
    """A single-token step captured with its plan or without, replayed several times, with eager steps of other sizes
    and a released sequence in between."""
    heads, seqs = 4, 3
    cache = attn.PagedCache(n_pages=60, page_size=8, n_kv_heads=heads, n_seqs=seqs, max_pages=30)
    scenes = Scenes(cache, heads)

    def eager(new, pad=0):
        n = sum(new)
        q, k, v = (scenes.rows(n + pad) for _ in range(3))
        assert cache.plan(i32(new), n + pad).item() == 0
        cache.append(0, k, v)
        scenes.check(new, q, k, v, cache.attend(0, q, causal_unit=1))

    eager([30, 5, 0])
    ones, (q, k, v) = i32([1] * seqs), (scenes.rows(seqs) for _ in range(3))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    if not whole:
        cache.plan(i32([0] * seqs), seqs)  # the step's buffers are those of any plan of as many rows
    with torch.cuda.graph(graph):
        if whole:
            refused = cache.plan(ones, seqs)
        cache.append(0, k, v)
        got = cache.attend(0, q, causal_unit=1)

    def replay():
        for t in (q, k, v):
            t.copy_(scenes.rows(seqs))
        if not whole:
            assert cache.plan(ones, seqs).item() == 0
        graph.replay()
        ok()
        assert not whole or refused.item() == 0
        scenes.check([1] * seqs, q, k, v, got)

    replay()
    replay()
    eager([0, 70, 9], pad=3)
    for _ in range(9):
        replay()
    cache.release(0)
    scenes.kept[0] = []
    replay()
    eager([11, 0, 0])
    replay()
    held = sum(-(-n // 8) for n in cache.kv_lens.tolist())
    assert cache.n_free.item() == 60 - held


def test_a_cache_planned_on_another_stream_behind_queued_work():
    """What the plans read and write must outlast the host's calls: buffers of their sizes are taken and overwritten
    on the current stream while the plans are still queued."""
    heads, seqs = 2, 300
    cache = attn.PagedCache(n_pages=2000, page_size=8, n_kv_heads=heads, n_seqs=seqs, max_pages=9)
    side = torch.cuda.Stream()
    new, rows = [1 + b % 3 for b in range(seqs)], 2 * seqs
    fresh, work = i32(new), torch.randn(4096, 4096, device="cuda")
    for sizes in range(4):
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            for _ in range(20):
                work = (work @ work).clamp(-1, 1)
        refused = [cache.plan(fresh, rows, stream=s) for s in (side, side.cuda_stream, side)]
        scratch = [torch.full((n,), 12345, dtype=torch.int32, device="cuda")
                   for n in (1, 2, seqs, seqs + 2, seqs + 1 + 1024, 2 * seqs + 3 + rows, rows) for _ in range(20)]
        torch.cuda.current_stream().wait_stream(side)
        del scratch
        assert [r.item() for r in refused] == [0, 0, 0]
        assert cache.kv_lens.tolist() == [3 * (sizes + 1) * n for n in new]
        table, slots = cache.block_table.tolist(), []
        for b, n in enumerate(new):
            total = 3 * (sizes + 1) * n
            slots += [table[b][t // 8] * 8 + t % 8 for t in range(total - n, total)]
        assert cache.slots.tolist() == slots + [-1] * (rows - len(slots))
    used = [p for b, n in enumerate(new) for p in table[b][:-(-12 * n // 8)]]
    assert len(set(used)) == len(used) and cache.n_free.item() == 2000 - len(used)
    assert sorted(used + cache.free_pages[:cache.n_free.item()].tolist()) == list(range(2000))
