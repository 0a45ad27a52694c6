"""The operators of a densely attended layer's cache at serving time, as they are measured.

* ``decode``: attention of one new token per sequence over a paged key-value cache, alone or also adding
  every key's attention weight to an accumulated one (``weights``);
* ``prompt``: the attention weight that the queries of a prompt (all, or the last ones) give every key;
* ``select``: the tokens that stay when a cache is cut to a budget by accumulated attention weight;
* ``move``: their rows gathered into new pages.

With ``own`` false, ``run`` computes the plain form (elementary torch operations in 32 bits, rounded once);
with ``own`` true it makes the framework's calls."""
import math
import random

import torch

own = False

PAGE = 128


def listed():
    big = {"H": 64, "G": 4, "d": 128, "d_idx": 64}
    return [
        # a chat's short cache on a small model: the call's latency counts
        {"name": "decode_1x777_small", "op": "decode", "H": 8, "G": 2, "d": 64, "batch": 1, "l_min": 777, "l_max": 777,
         "weights": False},
        # an ordinary serving step: a ragged batch of a few thousand tokens each
        {"name": "decode_32x8k_ragged", "op": "decode", "H": 64, "G": 4, "d": 128, "batch": 32, "l_min": 1, "l_max": 8192,
         "weights": False},
        # a few long documents
        {"name": "decode_5x128k", "op": "decode", "H": 64, "G": 4, "d": 128, "batch": 5, "l_min": 65537, "l_max": 131072,
         "weights": False},
        # one context of a million tokens
        {"name": "decode_1x1m", "op": "decode", "H": 64, "G": 4, "d": 128, "batch": 1, "l_min": 1048573, "l_max": 1048573,
         "weights": False},
        # a serving step that also keeps the tokens' accumulated weight, for eviction
        {"name": "decode_weights_16x16k", "op": "decode", "H": 32, "G": 2, "d": 128, "batch": 16, "l_min": 1000,
         "l_max": 16384, "weights": True},
        {"name": "decode_weights_2x400k", "op": "decode", "H": 64, "G": 4, "d": 128, "batch": 2, "l_min": 262144,
         "l_max": 400000, "weights": True},
        # after a prompt: the weight its last 64 tokens give the cache
        {"name": "prompt_last64_4x32k", "op": "prompt", "H": 64, "G": 4, "d": 128, "batch": 4, "l_min": 9001,
         "l_max": 32768, "t_max": 64},
        # after a prompt: the weight all its tokens give
        {"name": "prompt_all_3x4k", "op": "prompt", "H": 32, "G": 4, "d": 64, "batch": 3, "l_min": 2500, "l_max": 4096,
         "t_max": 4096},
        # a batch over its budget by some hundred tokens
        {"name": "select_8x5k", "op": "select", "G": 4, "batch": 8, "l_min": 4097, "l_max": 5000, "budget": 4096,
         "n_sink": 4, "n_recent": 512, "per_group": False},
        # two contexts of a million tokens cut to an eighth
        {"name": "select_2x1m", "op": "select", "G": 4, "batch": 2, "l_min": 900001, "l_max": 1048576, "budget": 131072,
         "n_sink": 128, "n_recent": 8192, "per_group": False},
        # the small cut's rows, each group keeping tokens of its own
        dict(big, name="move_8x4k_groups", op="move", batch=8, l_min=4097, l_max=5000, budget=4096, per_group=True),
        # long documents cut to half
        dict(big, name="move_4x64k", op="move", batch=4, l_min=100000, l_max=131072, budget=65536, per_group=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decode", "decode", "decode_weights", "prompt", "select", "move"])
    G = rng.choice([1, 2, 4])
    hg = rng.choice([4, 8, 16])
    case = {"op": op.split("_")[0], "H": G * hg, "G": G, "d": rng.choice([64, 128])}
    if case["op"] == "decode":
        total = _log(rng, 500, 800000)
        case["batch"] = min(_log(rng, 1, 64), max(1, total // 64))
        case["l_max"] = max(2, total // case["batch"])
        case["l_min"] = rng.randint(1, case["l_max"])
        case["weights"] = op == "decode_weights"
    elif case["op"] == "prompt":
        case["batch"] = rng.randint(1, 4)
        if rng.random() < 0.5:
            case["t_max"] = _log(rng, 1, 100)
            case["l_max"] = _log(rng, 128, 32768)
        else:
            case["t_max"] = 4096
            case["l_max"] = _log(rng, 128, 4096)
        case["l_min"] = rng.randint(max(1, case["l_max"] // 3), case["l_max"])
    else:
        most = 1000000 if case["op"] == "select" else 200000
        total = _log(rng, 300, most)
        case["batch"] = min(_log(rng, 1, 32), max(1, total // 200))
        case["l_max"] = max(2, total // case["batch"])
        case["l_min"] = rng.randint(max(1, case["l_max"] // 2), case["l_max"])
        case["budget"] = max(1, int(case["l_max"] * rng.uniform(0.05, 0.98)))
        case["per_group"] = rng.random() < 0.5
        if case["op"] == "select":
            case["n_sink"] = rng.randint(0, case["budget"] // 8)
            case["n_recent"] = rng.randint(0, case["budget"] // 4)
            del case["H"], case["d"]
        else:
            case["d_idx"] = rng.choice([32, 64, 128])
    return case


def _lengths(case):
    """The sequences' lengths: they belong to the case, not to the seed."""
    r = random.Random("%d %d %d" % (case["batch"], case["l_min"], case["l_max"]))
    return [r.randint(case["l_min"], case["l_max"]) for _ in range(case["batch"])]


def _randn(shape, gen, scale=1.0):
    return (torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16) * scale)


def _table(lens, gen, spare, width=None):
    """A block table over pages in a random order; entries past a sequence's last page are -1."""
    blocks = [-(-n // PAGE) for n in lens]
    pages = sum(blocks) + spare
    perm = torch.randperm(pages, generator=gen, device="cuda")
    nb = torch.tensor(blocks, device="cuda")
    start = torch.cumsum(nb, 0) - nb
    j = torch.arange(width or max(blocks), device="cuda")
    at = (start[:, None] + j[None, :]).clamp(max=pages - 1)
    table = torch.where(j[None, :] < nb[:, None], perm[at], torch.full_like(at, -1)).to(torch.int32).contiguous()
    return table, pages, perm[sum(blocks):]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    lens = _lengths(case)
    B, G = case["batch"], case["G"]
    s = {"case": case, "lens": lens, "lens_d": torch.tensor(lens, dtype=torch.int32, device="cuda")}
    op = case["op"]
    if op == "decode":
        H, d = case["H"], case["d"]
        s["table"], s["num_pages"], _ = _table(lens, gen, spare=3)
        rows = s["num_pages"] * PAGE
        s["q"] = _randn((B, H, d), gen, 1.5)
        s["k"] = _randn((rows, G, d), gen)
        s["v"] = _randn((rows, G, d), gen)
        if case["weights"]:
            s["decay"] = 0.98
            s["weights"] = torch.rand((B, G, s["table"].shape[1] * PAGE), generator=gen, device="cuda") * 0.1
    elif op == "prompt":
        H, d = case["H"], case["d"]
        t = [min(n, case["t_max"]) for n in lens]
        s["t"] = t
        cu_q = [sum(t[:i]) for i in range(B + 1)]
        cu_k = [sum(lens[:i]) for i in range(B + 1)]
        s["cu_q"], s["cu_k"] = cu_q, cu_k
        s["cu_q_d"] = torch.tensor(cu_q, dtype=torch.int32, device="cuda")
        s["cu_k_d"] = torch.tensor(cu_k, dtype=torch.int32, device="cuda")
        s["q"] = _randn((cu_q[-1], H, d), gen, 1.5)
        s["k"] = _randn((cu_k[-1], G, d), gen)
        s["lse"] = _prompt_lse(s)
        s["weights"] = torch.zeros((B, G, max(lens)), device="cuda")
    else:
        s["table"], s["num_pages"], free = _table(lens, gen, spare=0 if op == "select" else B * -(-case["budget"] // PAGE) + 3)
        s["weights"] = torch.exp(2 * torch.randn((B, G, s["table"].shape[1] * PAGE), generator=gen, device="cuda"))
        # tokens that no query has looked at yet
        s["weights"] *= torch.rand((B, 1, s["weights"].shape[2]), generator=gen, device="cuda") > 0.1
        if op == "move":
            d, nb = case["d"], -(-case["budget"] // PAGE)
            rows = s["num_pages"] * PAGE
            s["k"] = _randn((rows, G, d), gen)
            s["v"] = _randn((rows, G, d), gen)
            if not case["per_group"]:
                s["k_idx"] = _randn((rows, case["d_idx"]), gen)
            s["new_table"] = free[:B * nb].view(B, nb).to(torch.int32).contiguous()
            s["weights_out"] = torch.zeros((B, G, nb * PAGE), device="cuda")
            sel = dict(case, n_sink=4, n_recent=min(64, case["budget"] // 4))
            s["kept"], s["new_lens"] = _plain_select(sel, s)
    if own:
        from block_sparse_long_exp_b200 import msa
        shape = msa.make_shape(case.get("H", 4 * G), G, case.get("d", 64), case.get("d_idx", 64), 16)
        s["shape"] = shape
        if op == "prompt":
            s["seqs"] = msa.make_varlen(s["cu_q_d"], s["cu_k_d"], s["cu_q"], s["cu_k"])
            size = msa.msa_attn_weights_workspace_size(shape, s["seqs"])
        else:
            s["pages"] = msa.make_paged(s["lens_d"], s["table"], max(lens), s["num_pages"])
            if op == "decode":
                size = msa.msa_dense_attn_decode_paged_workspace_size(shape, s["pages"], case["weights"])
            elif op == "select":
                size = msa.msa_evict_select_workspace_size(shape, s["pages"], case["per_group"])
            else:
                s["new_pages"] = msa.make_paged(s["new_lens"], s["new_table"], case["budget"], s["num_pages"])
                size = msa.msa_evict_move_workspace_size(shape, s["pages"])
        s["ws"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    return s


def _position_rows(table, lens_d, n):
    """Row in the pages of every position 0 .. n - 1 of every sequence (0 past its end), and which are in it."""
    j = torch.arange(n, device="cuda")
    inside = j[None, :] < lens_d[:, None]
    page = table.long()[:, j // PAGE]
    return torch.where(inside, page * PAGE + j % PAGE, torch.zeros_like(page)), inside


def _plain_decode(s):
    case = s["case"]
    B, H, G, d = case["batch"], case["H"], case["G"], case["d"]
    n = max(s["lens"])
    rows, inside = _position_rows(s["table"], s["lens_d"], n)
    k = s["k"][rows].permute(0, 2, 3, 1).float()                                # [B, G, d, n]
    q = s["q"].view(B, G, H // G, d).float()
    x = torch.matmul(q, k) * d ** -0.5                                          # [B, G, Hg, n]
    del k
    x = x.masked_fill(~inside[:, None, None, :], float("-inf"))
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - top)
    total = p.sum(-1, keepdim=True)
    p = p / total
    v = s["v"][rows].float() * inside[:, :, None, None]
    out = torch.matmul(p, v.permute(0, 2, 1, 3)).reshape(B, H, d).to(torch.bfloat16)
    lse = (top + torch.log(total)).reshape(B, H)
    if not case["weights"]:
        return {"out": out, "lse": lse}
    w = s["weights"]
    w[:, :, :n] = torch.where(inside[:, None, :], s["decay"] * w[:, :, :n] + p.sum(2), w[:, :, :n])
    return {"out": out, "lse": lse, "weights": w}


def _padded(s, x, n, cu):
    """Packed rows [total, ...] as [B, n, ...], by each sequence's first row (rows past a sequence's end: any)."""
    start = torch.tensor(cu[:-1], device="cuda")
    at = (start[:, None] + torch.arange(n, device="cuda")[None, :]).clamp(max=x.shape[0] - 1)
    return x[at]


def _prompt_scores(s, dtype):
    """Scaled scores of a prompt's queries [B, G, Hg, T, S] (-inf where a key is not seen)."""
    case = s["case"]
    B, H, G, d = case["batch"], case["H"], case["G"], case["d"]
    T, S = max(s["t"]), max(s["lens"])
    q = _padded(s, s["q"], T, s["cu_q"]).to(dtype).view(B, T, G, H // G, d).permute(0, 2, 3, 1, 4)
    k = _padded(s, s["k"], S, s["cu_k"]).to(dtype).permute(0, 2, 3, 1)[:, :, None]
    x = torch.matmul(q, k) * d ** -0.5
    t = torch.tensor(s["t"], device="cuda")[:, None, None]
    i, j = torch.arange(T, device="cuda")[None, :, None], torch.arange(S, device="cuda")[None, None, :]
    lens = s["lens_d"][:, None, None]
    seen = (i < t) & (j < lens) & (j <= lens - t + i)
    return x.masked_fill_(~seen[:, None, None], float("-inf"))


def _prompt_lse(s):
    """The log-sum-exp that the attention over the prompt has left: [rows, H]."""
    case = s["case"]
    x = _prompt_scores(s, torch.float32)
    top = x.amax(-1, keepdim=True)
    lse = (top + (x - top).exp_().sum(-1, keepdim=True).log())[..., 0]             # [B, G, Hg, T]
    lse = lse.permute(0, 3, 1, 2).reshape(case["batch"], -1, case["H"])
    mine = torch.arange(lse.shape[1], device="cuda")[None, :] < torch.tensor(s["t"], device="cuda")[:, None]
    return lse[mine].contiguous()


def _prompt_weights(s, dtype):
    case = s["case"]
    B, H, G = case["batch"], case["H"], case["G"]
    x = _prompt_scores(s, dtype)
    lse = _padded(s, s["lse"], max(s["t"]), s["cu_q"]).to(dtype).view(B, -1, G, H // G).permute(0, 2, 3, 1)
    return (x - lse[..., None]).exp_().sum((2, 3))


def _plain_prompt(s):
    return {"weights": _prompt_weights(s, torch.float32)}


def _plain_select(case, s):
    B, budget = case["batch"], case["budget"]
    n = max(s["lens"])
    w = s["weights"][:, :, :n]
    score = w if case["per_group"] else w.double().sum(1, keepdim=True).float()
    j = torch.arange(n, device="cuda")
    lens = s["lens_d"][:, None, None]
    sink, recent = case["n_sink"], case["n_recent"]
    score = score.masked_fill((j < sink) | (j >= lens - recent), float("inf")).masked_fill(j >= lens, float("-inf"))
    order = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :budget]
    if order.shape[-1] < budget:
        order = torch.nn.functional.pad(order, (0, budget - order.shape[-1]), value=n)
    order = torch.sort(torch.where(order < lens, order, n), dim=-1).values
    kept = torch.where(order < n, order, -1).to(torch.int32)
    return kept, s["lens_d"].clamp(max=budget)


def _plain_move(s):
    case = s["case"]
    B, G, d, budget = case["batch"], case["G"], case["d"], case["budget"]
    kept = s["kept"].long()                                                       # [B, R, budget]
    inside = kept >= 0
    at = kept.clamp(min=0)
    src = torch.gather(s["table"].long()[:, None, :].expand(-1, kept.shape[1], -1), 2, at // PAGE) * PAGE + at % PAGE
    i = torch.arange(budget, device="cuda")
    dst = (s["new_table"].long()[:, i // PAGE] * PAGE + i % PAGE)[:, None, :].expand_as(src)
    out = {}
    if case["per_group"]:
        g = torch.arange(G, device="cuda")[None, :, None].expand_as(src)
        for name in ("k", "v"):
            s[name][dst[inside], g[inside]] = s[name][src[inside], g[inside]]
            out[name] = s[name]
        w = torch.gather(s["weights"], 2, at) * inside
    else:
        for name in ("k", "v", "k_idx"):
            s[name][dst[inside]] = s[name][src[inside]]
            out[name] = s[name]
        w = torch.gather(s["weights"], 2, at.expand(-1, G, -1)) * inside
    s["weights_out"].zero_()
    s["weights_out"][:, :, :budget] = w
    out["weights"] = s["weights_out"]
    return out


def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        from block_sparse_long_exp_b200 import msa
        if op == "decode":
            out, lse = msa.msa_dense_attn_decode_paged(s["shape"], s["pages"], s["q"], s["k"], s["v"],
                                                       weights=s.get("weights"), decay=s.get("decay", 1.0), ws=s["ws"],
                                                       check=False)
            return {"out": out, "lse": lse, "weights": s["weights"]} if case["weights"] else {"out": out, "lse": lse}
        if op == "prompt":
            w = msa.msa_attn_weights(s["shape"], s["seqs"], s["q"], s["k"], s["lse"], weights=s["weights"], decay=0.0,
                                     ws=s["ws"], check=False)
            return {"weights": w}
        if op == "select":
            kept, new_lens = msa.msa_evict_select(s["shape"], s["pages"], s["weights"], case["budget"], case["n_sink"],
                                                  case["n_recent"], per_group=case["per_group"], ws=s["ws"], check=False)
            return {"kept": kept, "new_lens": new_lens}
        msa.msa_evict_move(s["shape"], s["pages"], s["new_pages"], s["kept"], s["k"], s["v"], k_idx_pages=s.get("k_idx"),
                           weights=s["weights"], weights_out=s["weights_out"], ws=s["ws"], check=False)
        out = {"k": s["k"], "v": s["v"], "weights": s["weights_out"]}
        if not case["per_group"]:
            out["k_idx"] = s["k_idx"]
        return out
    if op == "decode":
        return _plain_decode(s)
    if op == "prompt":
        return _plain_prompt(s)
    if op == "select":
        kept, new_lens = _plain_select(case, s)
        return {"kept": kept, "new_lens": new_lens}
    return _plain_move(s)


def work(case):
    lens = _lengths(case)
    B, G, total = case["batch"], case["G"], sum(lens)
    if case["op"] == "decode":
        H, d = case["H"], case["d"]
        move = total * G * d * 2 * 2 + B * H * (d * 4 + 4) + (total * G * 8 if case["weights"] else 0)
        return {"bytes": move, "flops": 4 * total * H * d}
    if case["op"] == "prompt":
        H, d = case["H"], case["d"]
        t = [min(n, case["t_max"]) for n in lens]
        pairs = sum(a * n - a * (a - 1) // 2 for a, n in zip(t, lens))
        return {"bytes": sum(t) * H * (2 * d + 4) + total * G * (2 * d + 4), "flops": 2 * pairs * H * d}
    if case["op"] == "select":
        rows = G if case["per_group"] else 1
        return {"bytes": total * G * 4 + B * (rows * case["budget"] + 1) * 4, "flops": total * G}
    kept = sum(min(n, case["budget"]) for n in lens)
    row = G * case["d"] * 4 + G * 4 + (0 if case["per_group"] else case["d_idx"] * 2)
    return {"bytes": 2 * kept * row + 4 * kept * (G if case["per_group"] else 1), "flops": 0}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "select":
        return None                                                    # whole numbers alone
    B, H, G, d = case["batch"], case["H"], case["G"], case["d"]
    hg = H // G
    if case["op"] == "move":
        out = {name: s[name].double() for name in ("k", "v", "k_idx") if name in s}
        out["weights"] = torch.zeros_like(s["weights_out"], dtype=torch.float64)
        for b in range(B):
            for g in range(G):
                kept = s["kept"][b, g if case["per_group"] else 0].long()
                kept = kept[kept >= 0]
                i = torch.arange(kept.shape[0], device="cuda")
                src = s["table"][b].long()[kept // PAGE] * PAGE + kept % PAGE
                dst = s["new_table"][b].long()[i // PAGE] * PAGE + i % PAGE
                out["weights"][b, g, :kept.shape[0]] = s["weights"][b, g, kept].double()
                for name in ("k", "v"):
                    out[name][dst, g] = s[name][src, g].double()
                if "k_idx" in out and g == 0:
                    out["k_idx"][dst] = s["k_idx"][src].double()
        return out
    if case["op"] == "decode":
        out, lse = torch.empty(B, H, d, device="cuda", dtype=torch.float64), torch.empty(B, H, device="cuda", dtype=torch.float64)
        w = s["weights"].double() if case["weights"] else None
        for b, n in enumerate(s["lens"]):
            pages = s["table"][b, :-(-n // PAGE)].long()
            for g in range(G):
                k = s["k"].view(-1, PAGE, G, d)[pages, :, g].reshape(-1, d)[:n].double()
                v = s["v"].view(-1, PAGE, G, d)[pages, :, g].reshape(-1, d)[:n].double()
                x = (s["q"][b, g * hg:(g + 1) * hg].double() @ k.T) / math.sqrt(d)
                lse[b, g * hg:(g + 1) * hg] = torch.logsumexp(x, 1)
                p = torch.exp(x - lse[b, g * hg:(g + 1) * hg, None])
                out[b, g * hg:(g + 1) * hg] = p @ v
                if w is not None:
                    w[b, g, :n] = s["decay"] * w[b, g, :n] + p.sum(0)
        return {"out": out, "lse": lse, "weights": w} if case["weights"] else {"out": out, "lse": lse}
    w = torch.zeros(B, G, max(s["lens"]), device="cuda", dtype=torch.float64)
    for b, n in enumerate(s["lens"]):
        t, q0, k0 = s["t"][b], s["cu_q"][b], s["cu_k"][b]
        seen = torch.arange(n, device="cuda")[None, :] <= torch.arange(n - t, n, device="cuda")[:, None]
        for h in range(H):
            x = s["q"][q0:q0 + t, h].double() @ s["k"][k0:k0 + n, h // hg].double().T / math.sqrt(d)
            w[b, h // hg, :n] += (torch.exp(x - s["lse"][q0:q0 + t, h, None].double()) * seen).sum(0)
    return {"weights": w}
