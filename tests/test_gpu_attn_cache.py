"""Attention of new and drafted tokens over a paged cache
(bitlinear_attn_cache) on the GPU against the 64-bit form."""
import pytest
import torch

import _attn_ref as R
import _gpu_helpers as H
from sparse_linear_layers_group_amd import bitlinear as bl

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    H.ensure_built()


def cache(lens, page, hkv, d, seed, spare=3, max_pages=None):
    """Random pages in random order; rows no sequence holds are NaN."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    counts = [-(-n // page) for n in lens]
    pool = sum(counts) + spare
    order = torch.randperm(pool, generator=g, device="cuda").tolist()
    width = max_pages or max(max(counts), 1)
    k, v = (torch.full((pool * page, hkv, d), float("nan"), dtype=BF, device="cuda") for _ in range(2))
    pages, rows, at = torch.full((len(lens), width), -7, dtype=torch.int32), [], 0
    for b, (n, c) in enumerate(zip(lens, counts)):
        mine = order[at:at + c]
        at += c
        pages[b, :c] = torch.tensor(mine, dtype=torch.int32)
        r = (torch.tensor(mine)[:, None] * page + torch.arange(page)).reshape(-1)[:n].long().cuda()
        k[r] = torch.randn(n, hkv, d, generator=g, device="cuda").to(BF)
        v[r] = (torch.randn(n, hkv, d, generator=g, device="cuda") + 0.25).to(BF)
        rows.append(r)
    return k, v, pages.cuda(), rows


def trees(batch, draft, seed):
    g = torch.Generator().manual_seed(seed)
    out = torch.zeros(batch, draft, dtype=torch.int64)
    for b in range(batch):
        for i in range(draft):
            m = 1 << i
            if i and torch.rand(1, generator=g).item() > 0.2:  # several roots: some tokens see only the context
                m |= int(out[b, int(torch.randint(0, i, (1,), generator=g))]) & ((1 << 64) - 1)
            out[b, i] = m - (1 << 64) if m >> 63 else m
    return out.cuda()


def queries(batch, draft, hq, d, seed):
    g = torch.Generator(device="cuda").manual_seed(seed + 1000)
    return (torch.randn(batch * draft, hq, d, generator=g, device="cuda") * 1.5).to(BF)


def reference(q, k, v, rows, lens, tree, draft, scale, hidden=None):
    """hidden[b]: positions that no token sees."""
    o, err = q.double() * 0, q.double() * 0
    for b, r in enumerate(rows):
        n = lens[b]
        for i in range(draft):
            m = (int(tree[b, i]) & ((1 << 64) - 1)) if tree is not None else (2 << i) - 1
            see = [p for p in range(n) if p < n - draft or m >> (p - n + draft) & 1]
            if hidden:
                see = [p for p in see if p not in hidden[b]]
            if not see:
                continue
            x = r[torch.tensor(see, device="cuda")]
            ref = R.attention(q[b * draft + i:b * draft + i + 1], k[x], v[x], [1], [len(see)], scale)
            o[b * draft + i], err[b * draft + i] = ref["o"][0], ref["o_err"][0]
    return o, err


def run(q, k, v, pages, page, lens, tree, batch, draft, scale, stream=None, ws=None):
    hq, d = q.shape[1:]
    hkv = k.shape[1]
    o = torch.full_like(q, 7.0)
    if ws is None:
        ws = torch.full((bl.bitlinear_attn_cache_workspace_bytes(batch, draft, hq, hkv, d),), 255, dtype=torch.uint8, device="cuda")
    n = torch.tensor(lens, dtype=torch.int32, device="cuda") if isinstance(lens, list) else lens
    bl.bitlinear_attn_cache(q, k, v, pages, page, n, tree, batch, draft, hq, hkv, d, scale, o, ws=ws, stream=stream)
    return o


def check(lens, page, draft, hq, hkv, d, with_tree, seed=0, scale=None):
    scale = d ** -0.5 if scale is None else scale
    k, v, pages, rows = cache(lens, page, hkv, d, seed)
    q = queries(len(lens), draft, hq, d, seed)
    tree = trees(len(lens), draft, seed) if with_tree else None
    o = run(q, k, v, pages, page, lens, tree, len(lens), draft, scale)
    want, err = reference(q, k, v, rows, lens, tree, draft, scale)
    R.assert_within(o, want, err, "O")


@pytest.mark.parametrize("hq,hkv,d", [(1, 1, 64), (14, 2, 64), (8, 8, 64), (20, 5, 128), (16, 2, 128), (40, 1, 128)])
@pytest.mark.parametrize("page", [16, 48, 64, 256])
def test_single_tokens(hq, hkv, d, page):
    check([1, 2, 16, 31, 32, 33, 100, 0, 513], page, 1, hq, hkv, d, False, seed=page)


@pytest.mark.parametrize("lens", [[1], [5000], [3000, 1, 0, 0, 700], [0, 0], [130] * 70])
@pytest.mark.parametrize("d", [64, 128])
def test_lengths_cut_between_workgroups(lens, d):
    check(lens, 32, 1, 4, 2, d, False, seed=len(lens))


@pytest.mark.parametrize("hq,hkv,d", [(14, 2, 64), (20, 5, 128), (3, 3, 128)])
@pytest.mark.parametrize("draft", [2, 7, 33, 64])
@pytest.mark.parametrize("with_tree", [False, True])
def test_drafted_tokens(hq, hkv, d, draft, with_tree):
    check([draft, draft + 1, draft + 40, 300], 16, draft, hq, hkv, d, with_tree, seed=draft)


def test_fewer_rows_than_drafted_tokens():
    check([3, 0, 9], 16, 5, 4, 2, 64, True, seed=3)


def test_large_scores():
    check([400, 77], 16, 3, 4, 2, 128, False, seed=4, scale=3.0)


@pytest.mark.parametrize("d", [64, 128])
def test_pages_outside_the_cache_hold_no_rows(d):
    lens, page, hq, hkv = [200, 90, 48], 16, 4, 2
    k, v, pages, rows = cache(lens, page, hkv, d, seed=5)
    q = queries(3, 1, hq, d, 5)
    pool = k.shape[0] // page
    pages[0, 0], pages[0, 5], pages[1, 2] = -1, pool, 1 << 30
    pages[2, :3] = -1  # nothing left to see
    hidden = [set(range(16)) | set(range(80, 96)), set(range(32, 48)), set(range(48))]
    o = run(q, k, v, pages, page, lens, None, 3, 1, 0.1)
    want, err = reference(q, k, v, rows, lens, None, 1, 0.1, hidden)
    R.assert_within(o, want, err, "O")
    assert (o[2] == 0).all()


def test_lengths_outside_the_table_are_cut_off():
    lens, page, hq, hkv, d = [64, 32], 16, 2, 1, 64
    k, v, pages, rows = cache(lens, page, hkv, d, seed=6)
    q = queries(2, 1, hq, d, 6)
    full = torch.tensor([1 << 30, -4], dtype=torch.int32, device="cuda")
    o = run(q, k, v, pages, page, full, None, 2, 1, 0.125)
    want, err = reference(q, k, v, rows, [64, 0], None, 1, 0.125)
    R.assert_within(o, want, err, "O")


def test_one_contiguous_cache_per_sequence():
    """A page as long as the cache of a sequence: no paging at all."""
    lens, most, hq, hkv, d = [700, 1008, 5], 1008, 8, 2, 128
    g = torch.Generator(device="cuda").manual_seed(7)
    k, v = (torch.randn(3 * most, hkv, d, generator=g, device="cuda").to(BF) for _ in range(2))
    q = queries(3, 1, hq, d, 7)
    pages = torch.arange(3, dtype=torch.int32, device="cuda")[:, None].contiguous()
    o = run(q, k, v, pages, most, lens, None, 3, 1, 0.1)
    rows = [torch.arange(b * most, b * most + n, device="cuda") for b, n in enumerate(lens)]
    want, err = reference(q, k, v, rows, lens, None, 1, 0.1)
    R.assert_within(o, want, err, "O")


def test_rows_beyond_32_bit_offsets():
    """The last pages of a cache of more than 2^31 elements."""
    hq, hkv, d, page = 16, 8, 128, 64
    rows_all = (1 << 21) + (1 << 15)  # 2.2e9 elements each
    k, v = (torch.empty(rows_all, hkv, d, dtype=BF, device="cuda") for _ in range(2))
    last = rows_all // page - 1
    n = 3 * page
    pages = torch.tensor([[last, last - 5, 0]], dtype=torch.int32, device="cuda")
    r = (pages[0].long()[:, None] * page + torch.arange(page, device="cuda")).reshape(-1)
    g = torch.Generator(device="cuda").manual_seed(8)
    k[r], v[r] = (torch.randn(n, hkv, d, generator=g, device="cuda").to(BF) for _ in range(2))
    q = queries(1, 1, hq, d, 8)
    o = run(q, k, v, pages, page, [n], None, 1, 1, 0.1)
    want, err = reference(q, k, v, [r], [n], None, 1, 0.1)
    R.assert_within(o, want, err, "O")


def test_reruns_strides_and_streams_agree():
    lens, page, draft, hq, hkv, d = [900, 33, 2048], 32, 5, 8, 2, 128
    k, v, pages, rows = cache(lens, page, hkv, d, seed=9)
    q = queries(3, draft, hq, d, 9)
    tree = trees(3, draft, 9)
    o = run(q, k, v, pages, page, lens, tree, 3, draft, 0.1)
    assert torch.equal(o, run(q, k, v, pages, page, lens, tree, 3, draft, 0.1))
    wide = torch.zeros(3 * draft, hq * d + 64, dtype=BF, device="cuda")
    wide[:, :hq * d] = q.view(3 * draft, -1)
    o2 = torch.empty_like(o)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    ws = torch.empty(bl.bitlinear_attn_cache_workspace_bytes(3, draft, hq, hkv, d), dtype=torch.uint8, device="cuda")
    bl.bitlinear_attn_cache(wide[:, :hq * d], k, v, pages, page, n, tree, 3, draft, hq, hkv, d, 0.1, o2, ws=ws)
    assert torch.equal(o, o2)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        o3 = run(q, k, v, pages, page, lens, tree, 3, draft, 0.1)
    side.synchronize()
    assert torch.equal(o, o3)


def test_captured_graph_replays_with_other_lengths():
    page, hq, hkv, d, batch = 16, 4, 2, 128, 3
    k, v, pages, rows = cache([600, 600, 600], page, hkv, d, seed=10)
    q = queries(batch, 1, hq, d, 10)
    n = torch.tensor([1, 2, 3], dtype=torch.int32, device="cuda")
    o = torch.empty_like(q)
    ws = torch.empty(bl.bitlinear_attn_cache_workspace_bytes(batch, 1, hq, hkv, d), dtype=torch.uint8, device="cuda")

    def step():
        bl.bitlinear_attn_cache(q, k, v, pages, page, n, None, batch, 1, hq, hkv, d, 0.1, o, ws=ws)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for lens in ([600, 1, 77], [5, 0, 599], [600, 600, 600]):
        n.copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        got = o.clone()
        assert torch.equal(got, run(q, k, v, pages, page, lens, None, batch, 1, 0.1))
        want, err = reference(q, k, v, [r[:m] for r, m in zip(rows, lens)], lens, None, 1, 0.1)
        R.assert_within(got, want, err, "O")


def test_captured_graph_of_drafted_trees():
    """The kernel for more than 32 rows of Q, with lengths, pages and trees that change."""
    page, hq, hkv, d, batch, draft = 16, 20, 5, 128, 3, 12
    k, v, pages, rows = cache([700, 700, 700], page, hkv, d, seed=11)
    q = queries(batch, draft, hq, d, 11)
    tree = trees(batch, draft, 11)
    n = torch.tensor([12, 20, 30], dtype=torch.int32, device="cuda")
    o = torch.empty_like(q)
    ws = torch.full((bl.bitlinear_attn_cache_workspace_bytes(batch, draft, hq, hkv, d),), 255, dtype=torch.uint8, device="cuda")

    def step():
        bl.bitlinear_attn_cache(q, k, v, pages, page, n, tree, batch, draft, hq, hkv, d, 0.1, o, ws=ws)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed, lens in ((12, [700, 12, 77]), (13, [0, 699, 13]), (14, [700, 700, 700])):
        n.copy_(torch.tensor(lens, dtype=torch.int32))
        tree.copy_(trees(batch, draft, seed))
        pages.copy_(pages.flip(0).contiguous())
        rows = rows[::-1]
        o.fill_(4.0)
        graph.replay()
        torch.cuda.synchronize()
        got = o.clone()
        assert torch.equal(got, run(q, k, v, pages, page, lens, tree, batch, draft, 0.1))
        want, err = reference(q, k, v, [r[:m] for r, m in zip(rows, lens)], lens, tree, draft, 0.1)
        R.assert_within(got, want, err, "O")


@pytest.mark.parametrize("draft", [1, 9])
def test_more_sequences_than_lanes(draft):
    """More than 64 sequences, empty ones among them, some long."""
    lens = [0 if i % 7 == 2 else (i * 13) % 40 + draft + (500 if i % 31 == 5 else 0) for i in range(150)]
    check(lens, 16, draft, 8, 2, 64, False, seed=15)


@pytest.mark.parametrize("hq,hkv,draft", [(64, 1, 3), (128, 1, 1), (48, 24, 2), (200, 1, 8)])
def test_many_heads(hq, hkv, draft):
    """Groups of many heads: several units read the same tiles."""
    check([draft, 90, 1000], 32, draft, hq, hkv, 64, True, seed=16)
