"""Eviction from a paged cache by accumulated attention weight: the choice
(msa_evict_select) against the oracle's sort and the move (msa_evict_move)
against plain indexing, both exactly.  Lengths around the budget and the
kernels' part sizes, ties, zeros of both signs, infinities, NaN and denormals,
empty and bad rows, shared and conflicting pages, captured and side-stream
calls."""
import numpy as np
import pytest
import torch

from oracle import dense_cache as C

pytestmark = pytest.mark.gpu

PAGE = 128


@pytest.fixture(scope="module")
def M():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from block_sparse_long_exp_b200 import build, msa
    build.build()
    msa.load_library()
    return msa


def _pages(M, lens, max_seqlen=None, blocks=None, num_pages=None):
    blocks = blocks or max(1, -(-max(lens) // PAGE))
    table = torch.arange(len(lens) * blocks, dtype=torch.int32).view(len(lens), blocks)
    return M.make_paged(torch.tensor(lens, dtype=torch.int32).cuda(), table.cuda(), max_seqlen or max(max(lens), 1),
                        num_pages or len(lens) * blocks)


def _want(weights, lens, budget, sink, recent, per_group):
    B, G, _ = weights.shape
    kept = np.full((B, G if per_group else 1, budget), -1, np.int32)
    for b, n in enumerate(lens):
        rows = C.evict_select(weights[b, :, :n].numpy(), budget, sink, recent, per_group)
        kept[b, :, :rows.shape[1]] = rows
    return kept


def _select(M, weights, lens, budget, sink, recent, per_group, max_seqlen=None):
    G = weights.shape[1]
    pg = _pages(M, lens, max_seqlen, weights.shape[2] // PAGE)
    kept, new = M.msa_evict_select(M.make_shape(4 * G, G, 64, 64, 16), pg, weights.cuda(), budget, sink, recent,
                                   per_group=per_group)
    np.testing.assert_array_equal(new.cpu().numpy(), [min(n, budget) for n in lens])
    np.testing.assert_array_equal(kept.cpu().numpy(), _want(weights, lens, budget, sink, recent, per_group))


def _weights(B, G, blocks, seed, kind="spread"):
    g = torch.Generator().manual_seed(seed)
    w = torch.exp(3 * torch.randn(B, G, blocks * PAGE, generator=g))
    if kind == "ties":
        w = torch.randint(0, 4, w.shape, generator=g).float()
    if kind == "zeros":
        w = torch.where(torch.rand(w.shape, generator=g) < 0.7, torch.zeros_like(w), w)
        w = torch.where(torch.rand(w.shape, generator=g) < 0.3, -torch.zeros_like(w), w)
    if kind == "odd":
        u = torch.rand(w.shape, generator=g)
        w = torch.where(u < 0.05, torch.full_like(w, float("nan")), w)
        w = torch.where((u > 0.05) & (u < 0.1), torch.full_like(w, float("inf")), w)
        w = torch.where((u > 0.1) & (u < 0.2), torch.full_like(w, float("-inf")), w)
        w = torch.where((u > 0.2) & (u < 0.4), -w, w)
        w = torch.where((u > 0.4) & (u < 0.5), w * 1e-42, w)
    if kind == "denormal":
        w = w * 1e-43
    return w


@pytest.mark.parametrize("G,per_group", [(1, False), (2, False), (4, False), (4, True), (2, True), (1, True)])
@pytest.mark.parametrize("kind", ["spread", "ties", "zeros"])
def test_choice(M, G, per_group, kind):
    lens = [1, 99, 100, 101, 102, 127, 128, 129, 1000, 0, 1023, 1537]
    w = _weights(len(lens), G, 13, 1 + G, kind)
    for budget, sink, recent in ((100, 4, 32), (1, 0, 0), (1, 1, 0), (100, 0, 100), (100, 100, 0), (1600, 3, 3), (700, 0, 0)):
        _select(M, w, lens, budget, sink, recent, per_group, max_seqlen=13 * PAGE)


@pytest.mark.parametrize("kind", ["odd", "denormal"])
def test_choice_among_odd_values(M, kind):
    # one group and a ranking per group: the sum of an infinity and its opposite is no case of use
    lens = [1000, 513, 40]
    for G, per_group in ((1, False), (4, True)):
        w = _weights(3, G, 8, 7, kind)
        for budget, sink, recent in ((300, 4, 32), (40, 0, 0), (960, 5, 1)):
            _select(M, w, lens, budget, sink, recent, per_group)


@pytest.mark.parametrize("L", [4095, 4096, 4097, 8191, 8192, 8193, 12289, 16385, 32770, 65537, 70001])
def test_parts_of_a_long_sequence(M, L):
    blocks = -(-L // PAGE)
    for kind, budget in (("spread", L // 3), ("ties", L // 2), ("zeros", L - 1)):
        _select(M, _weights(1, 2, blocks, L, kind), [L], budget, 5, 64, False)
    _select(M, _weights(2, 2, blocks, L, "ties"), [L, L // 2], L // 4, 0, 7, True)


def _want_fast(w, lens, budget, sink, recent):
    score = w.double().sum(1).float()
    kept = torch.full((len(lens), budget), -1, dtype=torch.int32)
    for b, n in enumerate(lens):
        s = score[b, :n].clone()
        if n > budget:
            s[:sink] = float("inf")
            s[n - recent:] = float("inf")
            at = torch.sort(s, descending=True, stable=True).indices[:budget]
            kept[b] = torch.sort(at).values.int()
        else:
            kept[b, :n] = torch.arange(n, dtype=torch.int32)
    return kept


@pytest.mark.parametrize("lens", [[400001, 330000], [1048576]])
def test_keys_past_shared_memory(M, lens):
    blocks = -(-max(lens) // PAGE)
    for kind, budget in (("spread", 50000), ("ties", 300001)):
        w = _weights(len(lens), 4, blocks, 3, kind)
        kept, new = M.msa_evict_select(M.make_shape(64, 4, 128, 64, 16), _pages(M, lens, blocks=blocks), w.cuda(), budget,
                                       4, 100)
        assert torch.equal(kept[:, 0].cpu(), _want_fast(w, lens, budget, 4, 100))
        assert new.cpu().tolist() == [min(n, budget) for n in lens]


@pytest.mark.parametrize("L,B", [(9001, 1), (9001, 40), (20000, 3), (20000, 25), (33000, 2), (33000, 13)])
def test_clusters_and_launches(M, L, B):
    # few rankings: a cluster of CTAs each; many: a CTA per part of each
    lens = [max(1, L - 997 * b) for b in range(B)]
    blocks = -(-L // PAGE)
    for kind, budget in (("spread", L // 5), ("ties", L // 2)):
        w = _weights(B, 2, blocks, B, kind)
        kept, new = M.msa_evict_select(M.make_shape(8, 2, 64, 64, 16), _pages(M, lens, blocks=blocks), w.cuda(), budget, 3, 40)
        assert torch.equal(kept[:, 0].cpu(), _want_fast(w, lens, budget, 3, 40))
        assert new.cpu().tolist() == [min(n, budget) for n in lens]


@pytest.mark.parametrize("per_group", [False, True])
def test_long_and_short_in_one_batch(M, per_group):
    # the longest decides the launch: rows that keep all, empty ones and bad lengths beside it
    lens = [70001, 0, 100, 8192, 66000, 8193, 16384]
    w = _weights(7, 2, 547, 21, "zeros")
    for budget, sink, recent in ((100, 0, 100), (8192, 1, 5), (66000, 9, 9), (70003, 0, 0)):
        _select(M, w, lens, budget, sink, recent, per_group)
    shape = M.make_shape(8, 2, 64, 64, 16)
    lens[3] = -1
    with pytest.raises(M.MsaError, match="DEVICE_CHECK at site 261"):
        M.msa_evict_select(shape, _pages(M, lens, 70001, 547), w.cuda(), 100, per_group=per_group)
    kept, new = M.msa_evict_select(shape, _pages(M, lens, 70001, 547), w.cuda(), 100, per_group=per_group, check=False)
    lens[3] = 0
    assert new.cpu().tolist() == [min(n, 100) for n in lens]
    np.testing.assert_array_equal(kept.cpu().numpy(), _want(w, lens, 100, 0, 0, per_group))


def test_many_sequences(M):
    lens = [(i * 91) % 700 for i in range(600)]
    _select(M, _weights(600, 2, 6, 5), lens, 150, 2, 30, False)


def test_choice_reports_bad_lengths(M):
    w = _weights(3, 2, 4, 9)
    shape = M.make_shape(8, 2, 64, 64, 16)
    for wrong in (-5, 301, 2 ** 31 - 1):
        lens = [300, wrong, 200]
        pg = M.make_paged(torch.tensor(lens, dtype=torch.int32).cuda(), torch.zeros(3, 4, dtype=torch.int32).cuda(), 300, 1)
        with pytest.raises(M.MsaError, match="DEVICE_CHECK at site 261"):
            M.msa_evict_select(shape, pg, w.cuda(), 100)
        kept, new = M.msa_evict_select(shape, pg, w.cuda(), 100, check=False)
        assert new.cpu().tolist() == [100, 0, 100]
        np.testing.assert_array_equal(kept.cpu().numpy(), _want(w, [300, 0, 200], 100, 0, 0, False))


# ------------------------------------------------------------------ move

def _pool(G, d, d_idx, num_pages, seed):
    g = torch.Generator().manual_seed(seed)
    rows = num_pages * PAGE
    return (torch.randn(rows, G, d, generator=g).bfloat16(), torch.randn(rows, G, d, generator=g).bfloat16(),
            torch.randn(rows, d_idx, generator=g).bfloat16())


def _row(table, b, j):
    return int(table[b, j // PAGE]) * PAGE + j % PAGE


def _moved(pool, table, new_table, kept, new_lens, w, wide):
    """The pool after the move, by plain loops over rows."""
    k, v, ki = (x.clone() if x is not None else None for x in pool)
    B, R, _ = kept.shape
    G = k.shape[1]
    out = torch.zeros(B, G, wide)
    for b in range(B):
        for i in range(int(new_lens[b])):
            to = _row(new_table, b, i)
            for g in range(G):
                at = int(kept[b, g if R > 1 else 0, i])
                row = _row(table, b, at)
                k[to, g], v[to, g] = pool[0][row, g], pool[1][row, g]
                out[b, g, i] = w[b, g, at]
            if ki is not None:
                ki[to] = pool[2][_row(table, b, int(kept[b, 0, i]))]
    return k, v, ki, out


def _tables(lens, new_lens, seed, blocks_over=1):
    g = torch.Generator().manual_seed(seed)
    nb, mb = [-(-n // PAGE) for n in lens], [-(-n // PAGE) for n in new_lens]
    pages = sum(nb) + sum(mb) + 2
    perm = torch.randperm(pages, generator=g).tolist()
    table = torch.full((len(lens), max(nb) + blocks_over), -1, dtype=torch.int32)
    new_table = torch.full((len(lens), max(mb) + blocks_over), -1, dtype=torch.int32)
    for t, counts in ((table, nb), (new_table, mb)):
        for b, n in enumerate(counts):
            for j in range(n):
                t[b, j] = perm.pop()
    return table, new_table, pages


@pytest.mark.parametrize("G,d,d_idx", [(4, 128, 64), (1, 64, 32), (2, 128, 128), (4, 64, 32)])
@pytest.mark.parametrize("per_group", [False, True])
@pytest.mark.parametrize("with_idx", [False, True])
def test_move(M, G, d, d_idx, per_group, with_idx):
    if per_group and with_idx and G > 1:
        pytest.skip("refused: the groups share the index keys")
    lens, budget = [130, 700, 257, 1, 0, 384, 200], 200
    shape = M.make_shape(4 * G, G, d, d_idx, 16)
    new_lens = [min(n, budget) for n in lens]
    table, new_table, pages = _tables(lens, new_lens, G)
    pool = _pool(G, d, d_idx, pages, 3)
    w = _weights(len(lens), G, table.shape[1], 4)
    pg = M.make_paged(torch.tensor(lens, dtype=torch.int32).cuda(), table.cuda(), max(lens), pages)
    dev = [x.cuda() for x in pool]
    kept, got_lens = M.msa_evict_select(shape, pg, w.cuda(), budget, 3, 20, per_group=per_group)
    npg = M.make_paged(got_lens, new_table.cuda(), budget, pages)
    wout = torch.full((len(lens), G, new_table.shape[1] * PAGE), float("nan"), device="cuda")
    got = M.msa_evict_move(shape, pg, npg, kept, dev[0], dev[1], k_idx_pages=dev[2] if with_idx else None,
                           weights=w.cuda(), weights_out=wout)
    assert got is wout
    k, v, ki, out = _moved((pool[0], pool[1], pool[2] if with_idx else None), table, new_table, kept.cpu(), new_lens, w,
                           wout.shape[2])
    assert torch.equal(dev[0].cpu(), k) and torch.equal(dev[1].cpu(), v)
    assert torch.equal(dev[2].cpu(), ki if with_idx else pool[2])
    assert torch.equal(wout.cpu(), out)
    # without weights, into the same pages: the rows again and nothing else
    again = [x.cuda() for x in pool]
    assert M.msa_evict_move(shape, pg, npg, kept, again[0], again[1]) is None
    assert torch.equal(again[0].cpu(), k) and torch.equal(again[1].cpu(), v) and torch.equal(again[2].cpu(), pool[2])


def test_move_reports_conflicts_and_bad_positions(M):
    lens, G, d = [300, 300], 2, 64
    shape = M.make_shape(8, G, d, 32, 16)
    table, new_table, pages = _tables(lens, [200, 200], 8)
    pool = _pool(G, d, 32, pages, 5)
    w = _weights(2, G, table.shape[1], 6)
    pg = M.make_paged(torch.tensor(lens, dtype=torch.int32).cuda(), table.cuda(), 300, pages)
    kept, new_lens = M.msa_evict_select(shape, pg, w.cuda(), 200, 0, 20)

    def run(nt, kp, nl=new_lens, match="DEVICE_CHECK at site 271", check_pool=None, src=pg):
        npg = M.make_paged(nl, nt.cuda(), 200, pages)
        dev = [x.cuda() for x in pool]
        with pytest.raises(M.MsaError, match=match):
            M.msa_evict_move(shape, src, npg, kp, dev[0], dev[1], weights=w.cuda())
        return [x.cpu() for x in dev]

    k, v, _, _ = _moved((pool[0], pool[1], None), table, new_table, kept.cpu(), [200, 200], w, 512)
    # a page of the other sequence, a page twice, pages outside the pool: not written; the rest is
    for wrong in (int(table[1, 2]), int(new_table[1, 0]), pages, -1):
        bad = new_table.clone()
        bad[0, 1] = wrong
        got = run(bad, kept)
        want_k = k.clone()
        for p in {int(new_table[0, 1])} | ({wrong} if wrong == int(new_table[1, 0]) else set()):
            want_k[p * PAGE:(p + 1) * PAGE] = pool[0][p * PAGE:(p + 1) * PAGE]
        assert torch.equal(got[0], want_k)
    # positions outside the sequence: their rows are left out
    for wrong in (-1, 300, 2 ** 31 - 1):
        bad = kept.clone()
        bad[1, 0, 7] = wrong
        got = run(new_table, bad)
        want_k = k.clone()
        want_k[_row(new_table, 1, 7)] = pool[0][_row(new_table, 1, 7)]
        assert torch.equal(got[0], want_k)
    # a source page outside the pool
    bad_src = table.clone()
    bad_src[0, 0] = pages + 9
    run(new_table, kept, src=M.make_paged(torch.tensor(lens, dtype=torch.int32).cuda(), bad_src.cuda(), 300, pages))
    # new lengths outside their bounds: the sequence is left alone
    for wrong in (-1, 201):
        got = run(new_table, kept, nl=torch.tensor([wrong, 200], dtype=torch.int32).cuda())
        want_k = k.clone()
        for j in range(200):
            want_k[_row(new_table, 0, j)] = pool[0][_row(new_table, 0, j)]
        assert torch.equal(got[0], want_k)


def test_shared_source_pages_move_for_each_sequence(M):
    # two sequences share their first two pages
    G, d, lens = 4, 128, [300, 290]
    shape = M.make_shape(16, G, d, 32, 16)
    table = torch.tensor([[0, 1, 2], [0, 1, 3]], dtype=torch.int32)
    new_table = torch.tensor([[5], [4]], dtype=torch.int32)
    pool = _pool(G, d, 32, 6, 11)
    w = _weights(2, G, 3, 12)
    pg = M.make_paged(torch.tensor(lens, dtype=torch.int32).cuda(), table.cuda(), 300, 6)
    kept, new_lens = M.msa_evict_select(shape, pg, w.cuda(), 100, 1, 9)
    dev = [x.cuda() for x in pool]
    out = M.msa_evict_move(shape, pg, M.make_paged(new_lens, new_table.cuda(), 100, 6), kept, dev[0], dev[1],
                           k_idx_pages=dev[2], weights=w.cuda())
    k, v, ki, want = _moved(pool, table, new_table, kept.cpu(), [100, 100], w, PAGE)
    assert all(torch.equal(a.cpu(), b) for a, b in zip(dev, (k, v, ki))) and torch.equal(out.cpu(), want)


def test_captured_and_side_stream_calls(M):
    G, d, budget = 2, 64, 150
    lens = [400, 100, 333]
    shape = M.make_shape(8, G, d, 64, 16)
    table, new_table, pages = _tables([400] * 3, [budget] * 3, 13)
    pool = _pool(G, d, 64, pages, 14)
    w = _weights(3, G, table.shape[1], 15)
    lens_d, wd = torch.tensor(lens, dtype=torch.int32).cuda(), w.cuda()
    pg = M.make_paged(lens_d, table.cuda(), 400, pages)
    kept = torch.empty(3, 1, budget, dtype=torch.int32, device="cuda")
    new_lens = torch.empty(3, dtype=torch.int32, device="cuda")
    npg = M.make_paged(new_lens, new_table.cuda(), budget, pages)
    dev = [x.cuda() for x in pool]
    wout = torch.empty(3, G, new_table.shape[1] * PAGE, device="cuda")
    ws1 = torch.empty(M.msa_evict_select_workspace_size(shape, pg), dtype=torch.uint8, device="cuda")
    ws2 = torch.empty(M.msa_evict_move_workspace_size(shape, pg), dtype=torch.uint8, device="cuda")

    def call(stream=None):
        M.msa_evict_select(shape, pg, wd, budget, 2, 10, kept=kept, new_lens=new_lens, ws=ws1, check=False, stream=stream)
        M.msa_evict_move(shape, pg, npg, kept, dev[0], dev[1], k_idx_pages=dev[2], weights=wd, weights_out=wout, ws=ws2,
                         check=False, stream=stream)

    def verify(now):
        np.testing.assert_array_equal(kept.cpu().numpy(), _want(w, now, budget, 2, 10, False))
        want = _moved(pool, table, new_table, kept.cpu(), [min(n, budget) for n in now], w, wout.shape[2])
        for b in range(3):
            for j in range(min(now[b], budget)):
                r = _row(new_table, b, j)
                assert torch.equal(dev[0][r].cpu(), want[0][r])
        assert torch.equal(wout.cpu(), want[3])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call(side)
    side.synchronize()
    verify(lens)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for now in ([400, 400, 400], [0, 151, 149], lens):
        lens_d.copy_(torch.tensor(now, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        verify(now)
        assert M.msa_get_device_error(ws2)[0] == 0


def test_pool_past_4_gib(M):
    G, d, budget = 4, 128, 140
    pool_pages, lens = 40000, [300]
    shape = M.make_shape(64, G, d, 64, 16)
    big = [torch.empty(pool_pages * PAGE, G, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    table = torch.tensor([[pool_pages - 1, 0, pool_pages - 3]], dtype=torch.int32)
    new_table = torch.tensor([[pool_pages - 2, 1]], dtype=torch.int32)
    g = torch.Generator().manual_seed(17)
    rows = torch.randn(300, G, d, generator=g).bfloat16()
    for x, sign in zip(big, (1, -1)):
        for j in range(3):
            n = min(PAGE, 300 - j * PAGE)
            x[int(table[0, j]) * PAGE:int(table[0, j]) * PAGE + n] = sign * rows[j * PAGE:j * PAGE + n].cuda()
    w = _weights(1, G, 3, 18)
    pg = M.make_paged(torch.tensor(lens, dtype=torch.int32).cuda(), table.cuda(), 300, pool_pages)
    kept, new_lens = M.msa_evict_select(shape, pg, w.cuda(), budget, 1, 5, per_group=True)
    M.msa_evict_move(shape, pg, M.make_paged(new_lens, new_table.cuda(), budget, pool_pages), kept, *big)
    kc = kept.cpu()
    for i in range(budget):
        r = _row(new_table, 0, i)
        want = torch.stack([rows[int(kc[0, gg, i]), gg] for gg in range(G)])
        assert torch.equal(big[0][r].cpu(), want) and torch.equal(big[1][r].cpu(), -want)


@pytest.mark.parametrize("L", [300, 20000, 70000])
def test_workspaces_with_anything_in_them(M, L):
    blocks = -(-L // PAGE)
    w = _weights(2, 2, blocks, 23)
    lens = [L, L - 50]
    shape = M.make_shape(8, 2, 64, 32, 16)
    pg = _pages(M, lens, blocks=blocks)
    ws = torch.full((M.msa_evict_select_workspace_size(shape, pg),), 255, dtype=torch.uint8, device="cuda")
    for _ in range(2):
        kept, new = M.msa_evict_select(shape, pg, w.cuda(), L // 2, 3, 40, ws=ws)
        assert torch.equal(kept[:, 0].cpu(), _want_fast(w, lens, L // 2, 3, 40)) and new.cpu().tolist() == [L // 2] * 2
    pool = _pool(2, 64, 32, 2 * blocks + 4, 24)
    spg = M.make_paged(torch.tensor(lens, dtype=torch.int32).cuda(),
                       torch.arange(2 * blocks, dtype=torch.int32).view(2, blocks).cuda(), L, 2 * blocks + 4)
    kept, new = M.msa_evict_select(shape, spg, w.cuda(), 200, 3, 40)
    new_table = 2 * blocks + torch.arange(4, dtype=torch.int32).view(2, 2)
    ws = torch.full((M.msa_evict_move_workspace_size(shape, spg),), 255, dtype=torch.uint8, device="cuda")
    dev = [x.cuda() for x in pool]
    out = M.msa_evict_move(shape, spg, M.make_paged(new, new_table.cuda(), 200, 2 * blocks + 4), kept, dev[0], dev[1],
                           k_idx_pages=dev[2], weights=w.cuda(), ws=ws)
    k, v, ki, want = _moved(pool, spg._keep[1].cpu(), new_table, kept.cpu(), [200, 200], w, 256)
    assert all(torch.equal(a.cpu(), b) for a, b in zip(dev, (k, v, ki))) and torch.equal(out.cpu(), want)


def test_many_rows(M):
    B = 66000
    lens = [200 if b % 1000 == 7 else (b % 3) for b in range(B)]
    w = _weights(1, 1, 2, 25).expand(B, 1, 256).contiguous()
    pg = M.make_paged(torch.tensor(lens, dtype=torch.int32).cuda(), torch.zeros(B, 2, dtype=torch.int32).cuda(), 200, 1)
    kept, new = M.msa_evict_select(M.make_shape(4, 1, 64, 64, 16), pg, w.cuda(), 60, 1, 9)
    want = {n: torch.from_numpy(_want(w[:1], [n], 60, 1, 9, False))[0] for n in (0, 1, 2, 200)}
    assert torch.equal(kept.cpu(), torch.stack([want[n] for n in lens]))
    assert new.cpu().tolist() == [min(n, 60) for n in lens]


@pytest.mark.parametrize("L", [20000, 70000])
def test_choice_in_a_graph(M, L):
    blocks = -(-L // PAGE)
    shape = M.make_shape(8, 2, 64, 64, 16)
    lens_d = torch.tensor([L, L], dtype=torch.int32).cuda()
    pg = M.make_paged(lens_d, torch.zeros(2, blocks, dtype=torch.int32).cuda(), L, 1)
    wd = torch.empty(2, 2, blocks * PAGE, device="cuda")
    kept, new = torch.empty(2, 1, 900, dtype=torch.int32, device="cuda"), torch.empty(2, dtype=torch.int32, device="cuda")
    ws = torch.empty(M.msa_evict_select_workspace_size(shape, pg), dtype=torch.uint8, device="cuda")
    wd.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        M.msa_evict_select(shape, pg, wd, 900, 3, 40, kept=kept, new_lens=new, ws=ws, check=False)
    for i, lens in enumerate(([L, L - 9], [901, L], [L, 20])):
        w = _weights(2, 2, blocks, 30 + i, "ties" if i == 1 else "spread")
        wd.copy_(w)
        lens_d.copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(kept[:, 0].cpu(), _want_fast(w, lens, 900, 3, 40)) and new.cpu().tolist() == [min(n, 900) for n in lens]


@pytest.mark.parametrize("L", [3000, 30000, 90000])
def test_two_calls_at_once(M, L):
    # choice and move on two streams, each with a workspace and pages of its own
    blocks, budget = -(-L // PAGE), 500
    shape = M.make_shape(8, 2, 64, 32, 16)
    pages = blocks + 4
    pool = _pool(2, 64, 32, pages, 41)
    table, new_table = torch.arange(blocks, dtype=torch.int32)[None], blocks + torch.arange(4, dtype=torch.int32)[None]
    ws = [_weights(1, 2, blocks, 42 + i) for i in range(2)]
    wd, dev = [w.cuda() for w in ws], [[x.cuda() for x in pool] for _ in range(2)]
    pg = [M.make_paged(torch.tensor([L], dtype=torch.int32).cuda(), table.cuda(), L, pages) for _ in range(2)]
    nt = new_table.cuda()
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], [None, None]
    for _ in range(3):
        for i, st in enumerate(streams):
            kept, new = M.msa_evict_select(shape, pg[i], wd[i], budget, 3, 40, stream=st, check=False)
            out = M.msa_evict_move(shape, pg[i], M.make_paged(new, nt, budget, pages), kept, dev[i][0], dev[i][1],
                                   k_idx_pages=dev[i][2], weights=wd[i], stream=st, check=False)
            got[i] = (kept, out)
    torch.cuda.synchronize()
    for i in range(2):
        kept, out = got[i]
        assert torch.equal(kept[:, 0].cpu(), _want_fast(ws[i], [L], budget, 3, 40))
        k, v, ki, want = _moved(pool, table, new_table, kept.cpu(), [budget], ws[i], 512)
        assert all(torch.equal(a.cpu(), b) for a, b in zip(dev[i], (k, v, ki))) and torch.equal(out.cpu(), want)
