"""The cache of a densely attended layer without a GPU: what the C entry points
and the Python binding refuse before any launch, workspace sizes, and the fp64
oracle (oracle/dense_cache.py) pinned by small cases worked out here."""
import ctypes
import glob
import os
import re

import numpy as np
import pytest
import torch

from oracle import dense_cache as C


@pytest.fixture(scope="module")
def M():
    from block_sparse_long_exp_b200 import build, msa
    build.build()
    msa.load_library()
    return msa


OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
BIG = 1 << 30
A = 4096                                                      # an aligned address that nothing reads


def _pages(M, batch=2, max_blocks=8, max_seqlen=1000, num_pages=20):
    p = M.Paged()
    p.batch, p.max_blocks, p.max_seqlen, p.num_pages = batch, max_blocks, max_seqlen, num_pages
    p.seqlens, p.block_table = A, A
    return p


def _by(x):
    return ctypes.byref(x)


# ------------------------------------------------------------------ C entry points

def test_dense_decode_host_checks(M):
    lib = M.load_library()
    shape, pg = M.make_shape(64, 4, 128, 64, 16), _pages(M)
    size = lib.msa_dense_attn_decode_paged_workspace_size
    assert size(_by(shape), _by(pg), 0) >= 256
    # the scores of every key: 4 H bytes a token of whole 64-token tiles
    assert size(_by(shape), _by(pg), 1) - size(_by(shape), _by(pg), 0) == 2 * 1024 * 64 * 4
    for bad in (M.make_shape(64, 4, 96, 64, 16), M.make_shape(64, 3, 128, 64, 16), M.make_shape(64, 4, 128, 64, 16, B_k=64)):
        assert size(_by(bad), _by(pg), 0) == 0
    assert size(_by(shape), _by(_pages(M, max_seqlen=1025)), 0) == 0          # past the block table

    def call(shape=shape, pg=pg, q=A, k=A, v=A, out=A, w=None, decay=1.0, ws=A, n=BIG):
        return lib.msa_dense_attn_decode_paged(_by(shape), _by(pg), q, k, v, out, None, w, decay, ws, n, None)
    for wrong in ({"q": None}, {"k": None}, {"v": None}, {"out": None}, {"q": A + 8}, {"k": A + 8}, {"v": A + 2},
                  {"out": A + 4}, {"w": A, "decay": -0.1}, {"w": A, "decay": 1.01}, {"w": A, "decay": float("nan")},
                  {"pg": _pages(M, batch=0)}, {"pg": _pages(M, max_seqlen=0)}):
        assert call(**wrong) == INVALID, wrong
    assert call(n=256) == WORKSPACE and call(ws=None) == WORKSPACE and call(ws=A + 64) == WORKSPACE
    assert call(shape=M.make_shape(64, 4, 96, 64, 16)) == UNSUPPORTED
    assert call(shape=M.make_shape(64, 4, 128, 64, 16, B_k=32)) == UNSUPPORTED
    no_table = _pages(M)
    no_table.block_table = None
    assert call(pg=no_table) == INVALID
    for scale in (0.0, -0.1, float("inf"), float("nan")):
        assert call(shape=M.make_shape(64, 4, 128, 64, 16, sm_scale=scale)) == INVALID


def test_attn_weights_host_checks(M):
    lib = M.load_library()
    shape = M.make_shape(64, 4, 128, 64, 16)
    seqs = M.Varlen(1, 64, 300, 0, 64, 300, A, A)
    size = lib.msa_attn_weights_workspace_size
    assert size(_by(shape), _by(seqs)) >= 256
    assert size(_by(M.make_shape(64, 4, 80, 64, 16)), _by(seqs)) == 0

    def call(shape=shape, seqs=seqs, q=A, k=A, lse=A, w=A, width=300, decay=1.0, ws=A, n=BIG):
        return lib.msa_attn_weights(_by(shape), _by(seqs), q, k, lse, w, width, decay, ws, n, None)
    for wrong in ({"q": None}, {"k": None}, {"lse": None}, {"w": None}, {"q": A + 8}, {"k": A + 8}, {"lse": A + 4},
                  {"width": 299}, {"width": 0}, {"decay": -1.0}, {"decay": 2.0}, {"decay": float("nan")},
                  {"seqs": M.Varlen(1, 301, 300, 0, 301, 300, A, A)}, {"seqs": M.Varlen(0, 64, 300, 0, 64, 300, A, A)}):
        assert call(**wrong) == INVALID, wrong
    for scale in (0.0, -0.1, float("inf"), float("nan")):
        assert call(shape=M.make_shape(64, 4, 128, 64, 16, sm_scale=scale)) == INVALID
    assert call(n=255) == WORKSPACE and call(ws=A + 128) == WORKSPACE
    assert call(shape=M.make_shape(64, 4, 80, 64, 16)) == UNSUPPORTED


def test_evict_select_host_checks(M):
    lib = M.load_library()
    shape, pg = M.make_shape(64, 4, 128, 64, 16), _pages(M)
    size = lib.msa_evict_select_workspace_size
    assert size(_by(shape), _by(pg), 0) >= 256
    long = _pages(M, batch=2, max_blocks=8192, max_seqlen=1 << 20)
    assert size(_by(shape), _by(long), 0) > 2 * (1 << 20) * 4 and size(_by(shape), _by(long), 1) > 8 * (1 << 20) * 4

    def call(shape=shape, pg=pg, w=A, budget=100, sink=4, recent=32, kept=A, lens=A, ws=A, n=BIG):
        return lib.msa_evict_select(_by(shape), _by(pg), w, budget, sink, recent, 0, kept, lens, ws, n, None)
    for wrong in ({"w": None}, {"w": A + 4}, {"kept": None}, {"lens": None}, {"budget": 0}, {"budget": -3}, {"sink": -1},
                  {"recent": -1}, {"sink": 60, "recent": 41}, {"sink": 2 ** 31 - 1, "recent": 2 ** 31 - 1}):
        assert call(**wrong) == INVALID, wrong
    assert call(pg=long, n=1 << 20) == WORKSPACE and call(ws=A + 16) == WORKSPACE


def test_evict_move_host_checks(M):
    lib = M.load_library()
    shape, pg, new = M.make_shape(64, 4, 128, 64, 16), _pages(M), _pages(M, max_blocks=2, max_seqlen=200)
    size = lib.msa_evict_move_workspace_size
    assert size(_by(shape), _by(pg)) >= 256 + 4 * 20

    def call(shape=shape, pg=pg, new=new, kept=A, width=200, per_group=0, k=A, v=A, ki=None, w=None, wo=None, ws=A, n=BIG):
        return lib.msa_evict_move(_by(shape), _by(pg), _by(new), kept, width, per_group, k, v, ki, w, wo, ws, n, None)
    for wrong in ({"kept": None}, {"width": 0}, {"k": None}, {"v": None}, {"k": A + 8}, {"v": A + 8}, {"ki": A + 8},
                  {"w": A}, {"wo": A}, {"w": A, "wo": A}, {"ki": A, "per_group": 1},
                  {"new": _pages(M, batch=3, max_seqlen=200)}, {"new": _pages(M, num_pages=21, max_seqlen=200)},
                  {"new": _pages(M, max_blocks=1, max_seqlen=200)}):
        assert call(**wrong) == INVALID, wrong
    assert call(n=300) == WORKSPACE


def test_workspaces_of_the_longest_sequence(M):
    # the longest description that is accepted: round-ups past 2^31
    lib, shape, most = M.load_library(), M.make_shape(4, 1, 64, 64, 16), 16777213 * 128
    pg = _pages(M, batch=1, max_blocks=16777213, max_seqlen=most, num_pages=1)
    keys = -(-most // 4096) * 4096 * 4
    assert keys <= lib.msa_evict_select_workspace_size(_by(shape), _by(pg), 0) <= keys + 2 ** 24
    scores = -(-most // 64) * 64 * 4 * 4
    for with_weights, least in ((0, 0), (1, scores)):
        assert least <= lib.msa_dense_attn_decode_paged_workspace_size(_by(shape), _by(pg), with_weights) <= least + 2 ** 24
    pg = _pages(M, batch=1, max_blocks=16777214, max_seqlen=most, num_pages=1)
    assert lib.msa_evict_select_workspace_size(_by(shape), _by(pg), 0) == 0


@pytest.mark.parametrize("scale,refused", [(1e-39, True), (1.1e-38, True), (2.0 ** -149, True), (2.4e38, True), (3.4e38, True),
                                           (2.0 ** -126, False), (2.3e38, False)])
def test_scales_that_would_break_the_mask_are_refused(M, scale, refused):
    # denormal scales count as 0 on the device (0 x -inf), 2.4e38 is past the largest number in units of log2
    lib, shape = M.load_library(), M.make_shape(64, 4, 128, 64, 16, sm_scale=scale)
    seqs, pg = M.Varlen(1, 64, 300, 0, 64, 300, A, A), _pages(M)
    # an accepted one is refused for its workspace, which is looked at last
    want = INVALID if refused else WORKSPACE
    assert lib.msa_dense_attn_decode_paged(_by(shape), _by(pg), A, A, A, A, None, None, 1.0, A, 256, None) == want
    assert lib.msa_attn_weights(_by(shape), _by(seqs), A, A, A, A, 300, 1.0, A, 255, None) == want


def test_chained_kernels_read_what_the_one_ahead_writes_after_the_wait(M):
    # a kernel that starts before the one ahead of it has ended: `const T* __restrict__` tells the compiler that nothing
    # changes the data while it runs, so that its loads may move ahead of the wait; only a call's inputs may have it
    inputs, seen = {"seqlens", "cu_k"}, 0
    for path in glob.glob(os.path.join(os.path.dirname(M.__file__), "csrc", "*.cu")):
        for kernel in open(path, encoding="utf-8").read().split("__global__")[1:]:
            head, body = kernel.split("{", 1)
            body = body.split("\n}\n", 1)[0]
            if "pdl_wait()" not in body and "griddepcontrol.wait" not in body:
                continue
            seen += 1
            held = set(re.findall(r"const\s+\w+\s*\*\s*__restrict__\s+(\w+)", head))
            assert held <= inputs, (os.path.basename(path), head.strip()[:60], held - inputs)
    assert seen >= 8


def test_the_move_refuses_weights_that_overlap(M):
    # 2 x 4 x 8 pages of weights in, 2 x 4 x 2 out: 32768 and 8192 bytes
    lib, shape, pg, new = M.load_library(), M.make_shape(64, 4, 128, 64, 16), _pages(M), _pages(M, max_blocks=2, max_seqlen=200)
    base = 1 << 20
    for out, refused in ((base, True), (base + 4, True), (base + 32764, True), (base + 32768, False), (base - 8188, True),
                         (base - 8192, False), (base + 16384, True)):
        # an accepted pair is refused for its workspace, which is looked at last
        assert lib.msa_evict_move(_by(shape), _by(pg), _by(new), A, 200, 0, A, A, None, base, out, A, 300, None) == \
            (INVALID if refused else WORKSPACE), out


def test_error_of_the_polynomial_exponential(M):
    # the coefficients as they stand in the source: their error in 64 bits, and with the kernel's 32-bit steps (a fused
    # multiply-add rounds once), over [-1/2, 1/2] as its comment gives them
    src = open(os.path.join(os.path.dirname(M.__file__), "csrc", "msa_attn_weights.cu"), encoding="utf-8").read()
    body = src[src.index("uint64_t add_exp2_poly"):]
    body = body[:body.index("\n}\n")]
    found = re.findall(r"uint64_t p = pair\(([\d.]+)f|p = fma2\(p, f, pair\(([\d.]+)f", body)
    c = [np.float32(a or b) for a, b in found]
    assert len(c) == 6 and c[-1] == 1.0
    f = np.linspace(-0.5, 0.5, 400001).astype(np.float32)
    exact, p, q = np.exp2(f.astype(np.float64)), np.zeros(f.shape), np.full(f.shape, c[0], np.float32)
    for x in c:
        p = p * f + float(x)
    for x in c[1:]:
        q = (q.astype(np.float64) * f + float(x)).astype(np.float32)
    pure, rounded = (float(np.log2(np.abs(y / exact - 1).max())) for y in (p, q))
    assert pure < -22.5 and "below 2^-22.5 over" in src
    assert rounded < -22.0 and "below 2^-22 with the roundings" in src


# ------------------------------------------------------------------ binding

H, G, d, d_idx = 8, 2, 64, 32


def _bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def test_binding_checks_the_dense_decode(M):
    shape, pg = M.make_shape(H, G, d, d_idx, 4), _pages(M)
    q, kv, w = _bf(2, H, d), _bf(20 * 128, G, d), torch.zeros(2, G, 1024)
    f = M.msa_dense_attn_decode_paged
    for match, call in (
            ("q: shape", lambda: f(shape, pg, _bf(3, H, d), kv, kv)), ("q: dtype", lambda: f(shape, pg, q.half(), kv, kv)),
            ("k_pages: shape", lambda: f(shape, pg, q, _bf(20 * 128, G, 32), kv)),
            ("v_pages: shape", lambda: f(shape, pg, q, kv, _bf(19 * 128, G, d))),
            ("contiguous", lambda: f(shape, pg, q, kv, _bf(20 * 128, d, G).transpose(1, 2))),
            ("out: dtype", lambda: f(shape, pg, q, kv, kv, out=q.float())),
            ("lse: shape", lambda: f(shape, pg, q, kv, kv, lse=torch.zeros(2, G))),
            ("weights: shape", lambda: f(shape, pg, q, kv, kv, weights=w[:, :, :1000].contiguous())),
            ("decay", lambda: f(shape, pg, q, kv, kv, weights=w, decay=1.5)),
            ("decay", lambda: f(shape, pg, q, kv, kv, weights=w, decay=float("nan"))),
            ("ws", lambda: f(shape, pg, q, kv, kv, ws=torch.zeros(4, 4).t())),
            ("CUDA", lambda: f(shape, pg, q, kv, kv, weights=w))):
        with pytest.raises(M.MsaError, match=match):
            call()


def test_binding_checks_the_key_weights(M):
    shape, seqs = M.make_shape(H, G, d, d_idx, 4), M.Varlen(1, 10, 30, 0, 10, 30, 0, 0)
    q, k, lse = _bf(10, H, d), _bf(30, G, d), torch.zeros(10, H)
    f = M.msa_attn_weights
    for match, call in (
            ("q: shape", lambda: f(shape, seqs, _bf(9, H, d), k, lse)), ("k: dtype", lambda: f(shape, seqs, q, k.float(), lse)),
            ("lse: shape", lambda: f(shape, seqs, q, k, torch.zeros(H, 10))),
            ("lse: a tensor", lambda: f(shape, seqs, q, k, None)), ("weights: expected a torch", lambda: f(shape, seqs, q, k, lse, weights=5)),
            ("q: expected a torch", lambda: f(shape, seqs, [1.0], k, lse)),
            ("weights: shape", lambda: f(shape, seqs, q, k, lse, weights=torch.zeros(1, G, 29))),
            ("weights: shape", lambda: f(shape, seqs, q, k, lse, weights=torch.zeros(1, H, 30))),
            ("weights: dtype", lambda: f(shape, seqs, q, k, lse, weights=torch.zeros(1, G, 30).double())),
            ("contiguous", lambda: f(shape, seqs, q, k, lse, weights=torch.zeros(1, G, 40)[:, :, :30])),
            ("decay", lambda: f(shape, seqs, q, k, lse, decay=-0.5)), ("CUDA", lambda: f(shape, seqs, q, k, lse))):
        with pytest.raises(M.MsaError, match=match):
            call()


def test_binding_checks_the_eviction(M):
    shape, pg, new = M.make_shape(H, G, d, d_idx, 4), _pages(M), _pages(M, max_blocks=1, max_seqlen=100)
    w, kv, ki = torch.zeros(2, G, 1024), _bf(20 * 128, G, d), _bf(20 * 128, d_idx)
    kept, kept_g = torch.zeros(2, 1, 100, dtype=torch.int32), torch.zeros(2, G, 100, dtype=torch.int32)
    s, m = M.msa_evict_select, M.msa_evict_move
    for match, call in (
            ("budget", lambda: s(shape, pg, w, 0)), ("n_sink", lambda: s(shape, pg, w, 10, 6, 5)),
            ("n_recent", lambda: s(shape, pg, w, 10, 0, -1)), ("budget", lambda: s(shape, pg, w, 2 ** 31)),
            ("weights: shape", lambda: s(shape, pg, w[:, :1].contiguous(), 10)),
            ("weights: dtype", lambda: s(shape, pg, w.half(), 10)),
            ("kept: shape", lambda: s(shape, pg, w, 99, kept=kept)),
            ("kept: shape", lambda: s(shape, pg, w, 100, per_group=True, kept=kept)),
            ("new_lens: dtype", lambda: s(shape, pg, w, 100, new_lens=torch.zeros(2))),
            ("CUDA", lambda: s(shape, pg, w, 100)),
            ("same sequences", lambda: m(shape, pg, _pages(M, batch=3), kept, kv, kv)),
            ("same sequences", lambda: m(shape, pg, _pages(M, num_pages=21), kept, kv, kv)),
            ("kept: dtype", lambda: m(shape, pg, new, kept.long(), kv, kv)), ("kept: a tensor", lambda: m(shape, pg, new, None, kv, kv)),
            ("weights: expected a torch", lambda: s(shape, pg, 3.0, 10)),
            ("kept: shape", lambda: m(shape, pg, new, kept[0], kv, kv)),
            ("kept: shape", lambda: m(shape, pg, new, torch.zeros(2, 3, 100, dtype=torch.int32), kv, kv)),
            ("index keys", lambda: m(shape, pg, new, kept_g, kv, kv, k_idx_pages=ki)),
            ("without weights", lambda: m(shape, pg, new, kept, kv, kv, weights_out=torch.zeros(2, G, 128))),
            ("k_pages: shape", lambda: m(shape, pg, new, kept, kv[:128], kv)),
            ("k_idx_pages: shape", lambda: m(shape, pg, new, kept, kv, kv, k_idx_pages=_bf(20 * 128, 64))),
            ("weights: shape", lambda: m(shape, pg, new, kept, kv, kv, weights=torch.zeros(2, G, 128))),
            ("weights_out: shape", lambda: m(shape, pg, new, kept, kv, kv, weights=w, weights_out=w)),
            ("CUDA", lambda: m(shape, pg, new, kept, kv, kv, k_idx_pages=ki, weights=w))):
        with pytest.raises(M.MsaError, match=match):
            call()


# ------------------------------------------------------------------ oracle

def test_oracle_decode_against_softmax():
    g = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn(*s, generator=g, dtype=torch.float64) for s in ((8, 16), (21, 2, 16), (21, 2, 16)))
    out, lse, w, mass = C.decode_attention(q, k, v, 0.3)
    for h in range(8):
        s = k[:, h // 4] @ q[h] * 0.3
        p = torch.softmax(s, 0)
        np.testing.assert_allclose(out[h], p @ v[:, h // 4], rtol=1e-12)
        np.testing.assert_allclose(lse[h], torch.logsumexp(s, 0), rtol=1e-12)
        np.testing.assert_allclose(mass[h], p @ v[:, h // 4].abs(), rtol=1e-12)
    np.testing.assert_allclose(w.sum(1), [4.0, 4.0], rtol=1e-12)
    out, lse, w, _ = C.decode_attention(q, k[:0], v[:0], 0.3)
    assert (out == 0).all() and (lse == -np.inf).all() and w.shape == (2, 0)


def test_oracle_key_weights_of_one_query_are_the_decode_s():
    g = torch.Generator().manual_seed(2)
    q, k = torch.randn(1, 8, 16, generator=g, dtype=torch.float64), torch.randn(30, 2, 16, generator=g, dtype=torch.float64)
    _, lse, w, _ = C.decode_attention(q[0], k, k, 0.25)
    np.testing.assert_allclose(C.key_weights(q, k, lse[None], 0.25), w, rtol=1e-12)
    # two queries: the first does not see the last key
    q2 = torch.cat([q, q])
    both = C.key_weights(q2, k, np.stack([lse, lse]), 0.25)
    np.testing.assert_allclose(both[:, :-1], 2 * w[:, :-1], rtol=1e-12)
    np.testing.assert_allclose(both[:, -1], w[:, -1], rtol=1e-12)
    assert (C.key_weights(q, k, np.full((1, 8), -np.inf), 0.25) == 0).all()


def test_oracle_eviction_rules():
    nan, inf = float("nan"), float("inf")
    row = np.array([[0.0, 5.0, 1.0, 1.0, nan, 1.0, inf, 0.5, 2.0]], np.float32)
    assert C.evict_select(row, 3, 0, 0, False).tolist() == [[1, 6, 8]]
    assert C.evict_select(row, 5, 0, 0, False).tolist() == [[1, 2, 3, 6, 8]]           # of three equal ones the first two
    assert C.evict_select(row, 5, 1, 2, False).tolist() == [[0, 1, 6, 7, 8]]
    assert C.evict_select(row, 8, 0, 0, False).tolist() == [[0, 1, 2, 3, 5, 6, 7, 8]]  # NaN goes first
    assert C.evict_select(row, 9, 3, 3, False).tolist() == [list(range(9))]
    two = np.array([[3.0, 0.0, 1.0], [0.0, 2.5, 1.0]], np.float32)
    assert C.evict_select(two, 1, 0, 0, False).tolist() == [[0]]
    assert C.evict_select(two, 1, 0, 0, True).tolist() == [[0], [1]]
    # the groups' sum is taken in 64 bits: 2^24 + 1 + 1 is not 2^24
    wide = np.array([[2.0 ** 24, 2.0 ** 24], [1.0, 0.0], [1.0, 0.0], [0.0, 0.0]], np.float32)[:, ::-1]
    assert C.evict_select(wide, 1, 0, 0, False).tolist() == [[1]]
