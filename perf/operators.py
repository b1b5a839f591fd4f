"""Cases and timings of the operators around the attention kernels: the norms of queries and
keys for each head with the position rotation (forward and backward), the append to the paged
latent cache with norm and rotation on the way, and decode for a tree of drafted tokens.

``run`` computes a case either in its plain form (elementary torch operations in fp32, angles
in fp64) or, with ``own`` set, through the library's entry points on the same inputs.
"""
import math

import torch

own = False

D_NOPE, D_ROPE, D_Q = 128, 64, 192
D_LAT, D_ROW, PAGE = 512, 576, 64
EPS = 1e-6
THETA = 10000.0


# ------------------------------------------------------------------------------- the cases

def listed():
    return [
        # queries of one decode step, eight sequences, eight heads on this GPU: latency
        {"name": "norm_rope_step", "op": "norm_rope", "B": 8, "S": 1, "H": 8, "keys": False, "norm": True,
         "pairs": True, "far": 32768},
        # ragged sizes, halves rotated together, no norm (rotation and split only)
        {"name": "norm_rope_odd", "op": "norm_rope", "B": 3, "S": 517, "H": 5, "keys": True, "norm": False,
         "pairs": False, "far": 1000000},
        # queries and keys of the prefill workload (4 x 4096 tokens, 128 heads)
        {"name": "norm_rope_prefill", "op": "norm_rope", "B": 4, "S": 4096, "H": 128, "keys": True, "norm": True,
         "pairs": True, "far": 4096},
        # a short training batch with few heads
        {"name": "norm_rope_grad_small", "op": "norm_rope_grad", "B": 2, "S": 333, "H": 8, "keys": True,
         "norm": True, "pairs": False, "far": 4096},
        # the backward workload: one sequence of 4096 tokens, 64 heads
        {"name": "norm_rope_grad_train", "op": "norm_rope_grad", "B": 1, "S": 4096, "H": 64, "keys": True,
         "norm": True, "pairs": True, "far": 4096},
        # one new token for each of 64 sequences, bf16 cache: latency
        {"name": "append_step", "op": "append", "B": 64, "T": 1, "fp8": False, "norm": True, "ragged": False,
         "pairs": True, "far": 256},
        # drafted tokens of a ragged fp8 batch, padded to the longest draft
        {"name": "append_draft_fp8", "op": "append", "B": 128, "T": 7, "fp8": True, "norm": True, "ragged": True,
         "pairs": True, "far": 300},
        # a prompt's latent rows written in one call, fp8 cache
        {"name": "append_prompt_fp8", "op": "append", "B": 8, "T": 8192, "fp8": True, "norm": True, "ragged": False,
         "pairs": False, "far": 8192},
        # a small tree over one short sequence, 16 heads: latency
        {"name": "tree_one", "op": "tree", "B": 1, "T": 8, "H": 16, "L": 1000, "fp8": False, "ragged": False,
         "shared": False},
        # trees of unlike sizes over ragged sequences, fp8 cache, 16 heads
        {"name": "tree_ragged_fp8", "op": "tree", "B": 64, "T": 13, "H": 16, "L": 16384, "fp8": True,
         "ragged": True, "shared": False},
        # one tree shape for a batch of 4096-token sequences, all 128 heads
        {"name": "tree_batch", "op": "tree", "B": 16, "T": 16, "H": 128, "L": 4096, "fp8": False, "ragged": False,
         "shared": True},
        # a wide tree over long sequences
        {"name": "tree_wide", "op": "tree", "B": 4, "T": 60, "H": 128, "L": 8192, "fp8": False, "ragged": False,
         "shared": False},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["norm_rope", "norm_rope_grad", "append", "tree"])
    if op in ("norm_rope", "norm_rope_grad"):
        H = _log(rng, 1, 128)
        tokens = _log(rng, 1, (4 * 4096 * 128 if op == "norm_rope" else 4096 * 64) // max(H, 32))
        B = min(tokens, _log(rng, 1, 16))
        return {"op": op, "B": B, "S": max(1, tokens // B), "H": H,
                "keys": op == "norm_rope_grad" or rng.random() < 0.7, "norm": rng.random() < 0.7,
                "pairs": rng.random() < 0.5, "far": _log(rng, 4096, 1000000)}
    if op == "append":
        B = _log(rng, 1, 256)
        return {"op": op, "B": B, "T": _log(rng, 1, max(1, 65536 // B)), "fp8": rng.random() < 0.5,
                "norm": rng.random() < 0.7, "ragged": rng.random() < 0.5, "pairs": rng.random() < 0.5,
                "far": _log(rng, 64, max(64, 131072 // B))}
    B, H = _log(rng, 1, 64), rng.choice([8, 16, 32, 64, 128])
    T = _log(rng, 1, 64)
    L = _log(rng, 80, 32768)
    most = 4 * 60 * 128 * 8192  # rows x keys of the largest listed case
    L = max(80, min(L, most // (B * T * H)))
    while B > 1 and B * T * H * L > most:
        B //= 2
    return {"op": op, "B": B, "T": T, "H": H, "L": L, "fp8": rng.random() < 0.5, "ragged": rng.random() < 0.6,
            "shared": rng.random() < 0.3}


# ------------------------------------------------------------------------------ the inputs

def _normal(gen, shape, dtype=torch.bfloat16, mag=1.0):
    return (torch.randn(shape, generator=gen, device="cuda") * mag).to(dtype)


def _inv_freq():
    return THETA ** (-torch.arange(0, D_ROPE, 2, dtype=torch.float64) / D_ROPE)


def _turns(inv_freq):
    """Turns per position in units of 2^-64, as the operators take them."""
    vals = [int(round(float(f) / (2 * math.pi) * 2.0 ** 64)) % 2 ** 64 for f in inv_freq]
    return torch.tensor([v - 2 ** 64 if v >= 2 ** 63 else v for v in vals], dtype=torch.int64, device="cuda")


def _lens(case, L):
    """For each sequence the tokens in the cache (the new ones counted), and how many of them are
    new; ragged: spread evenly over 1..L and 1..T."""
    B, T = case["B"], case["T"]
    if not case["ragged"]:
        return [(L, T)] * B
    new = [T - (i * 7919 % B) * T // B for i in range(B)]
    return [(max(n, 1 + (L - 1) * (i + 1) // B), n) for i, n in enumerate(new)]


def _pages(gen, B, pages_each):
    """A page pool in which every sequence owns pages_each pages, in shuffled order."""
    return torch.randperm(B * pages_each, generator=gen, device="cuda").to(torch.int32).view(B, pages_each)


def _trees(gen, n_trees, T):
    """Ancestor masks (bit j of row t: token t sees drafted token j) and depths of random trees:
    token t hangs below one of the four tokens before it, or below the last accepted one."""
    parent = (torch.arange(T, device="cuda") - torch.randint(1, 5, (n_trees, T), generator=gen, device="cuda"))
    parent = parent.clamp(min=-1).cpu()
    W = (T + 31) // 32
    bits = torch.zeros(n_trees, T, T, dtype=torch.bool)
    depth = torch.zeros(n_trees, T, dtype=torch.int32)
    for i in range(n_trees):
        for t in range(T):
            p = int(parent[i, t])
            if p >= 0:
                bits[i, t] = bits[i, p]
                depth[i, t] = depth[i, p] + 1
            bits[i, t, t] = True
    full = torch.zeros(n_trees, T, W * 32, dtype=torch.int64)
    full[:, :, :T] = bits
    words = (full.view(n_trees, T, W, 32) << torch.arange(32)).sum(-1)
    words = torch.where(words >= 2 ** 31, words - 2 ** 32, words).to(torch.int32)
    return words.cuda().contiguous(), depth.cuda()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    inv = _inv_freq()
    st = {"case": case, "inv_freq": inv.cuda(), "turns": _turns(inv)}
    op, B = case["op"], case["B"]
    if op in ("norm_rope", "norm_rope_grad"):
        S, H = case["S"], case["H"]
        st["q"] = _normal(gen, (B, S, H, D_Q))
        st["k_nope"] = st["k_rope"] = None
        if case["keys"]:
            # keys as the projections give them: k_nope beside v, the rope key behind the latent
            st["k_nope"] = _normal(gen, (B, S, H, 2 * D_NOPE))[..., :D_NOPE]
            st["k_rope"] = _normal(gen, (B, S, D_ROW))[..., D_LAT:]
        first = torch.randint(0, max(1, case["far"] - S + 1), (B, 1), generator=gen, device="cuda")
        st["positions"] = (first + torch.arange(S, device="cuda")).to(torch.int32)
        for n, d in (("q_nope", D_NOPE), ("q_rope", D_ROPE), ("k_nope", D_NOPE), ("k_rope", D_ROPE)):
            st["w_" + n] = None
            if case["norm"] and (case["keys"] or n[0] == "q"):
                st["w_" + n] = (1 + 0.2 * torch.randn(d, generator=gen, device="cuda")).to(torch.bfloat16)
        if op == "norm_rope_grad":
            st["dq_nope"] = _normal(gen, (B, S, H, D_NOPE))
            st["dq_rope"] = _normal(gen, (B, S, H, D_ROPE))
            st["dk_nope"] = _normal(gen, (B, S, H, D_NOPE))
            st["dk_rope"] = _normal(gen, (B, S, D_ROPE), torch.float32, math.sqrt(H))
        return st
    T, fp8 = case["T"], case["fp8"]
    L = case["L"] if op == "tree" else max(T, case["far"])
    lens = torch.tensor(_lens(case, L), dtype=torch.int32, device="cuda")[torch.randperm(B, generator=gen, device="cuda")]
    st["lens"], st["new"] = lens[:, 0].contiguous(), lens[:, 1].contiguous()
    each = (L + PAGE - 1) // PAGE
    st["page_table"] = _pages(gen, B, each)
    cache = torch.randn((B * each, PAGE, D_ROW), generator=gen, device="cuda", dtype=torch.float32)
    st["kv_scale"] = None
    if fp8:
        st["kv_scale"] = cache.abs().amax(-1) / 448
        st["cache"] = (cache / st["kv_scale"][..., None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    else:
        st["cache"] = cache.to(torch.bfloat16)
    del cache
    if op == "append":
        st["c_new"] = _normal(gen, (B, T, D_ROW))
        st["w_latent"] = None
        if case["norm"]:
            st["w_latent"] = (1 + 0.2 * torch.randn(D_LAT, generator=gen, device="cuda")).to(torch.bfloat16)
        # drafted tokens sit at their depth in the tree, below their place in the cache
        t = torch.arange(T, device="cuda", dtype=torch.int32)
        st["positions"] = ((st["lens"] - st["new"])[:, None] + (t + 1) // 2 if case["ragged"] else
                           (st["lens"] - st["new"])[:, None] + t).to(torch.int32)
        return st
    H = case["H"]
    st["q_latent"] = _normal(gen, (B, T, H, D_LAT))
    st["q_rope"] = _normal(gen, (B, T, H, D_ROPE))
    words, _ = _trees(gen, 1 if case["shared"] else B, T)
    st["mask"] = words[0] if case["shared"] else words
    st["scale"] = D_Q ** -0.5
    return st


# --------------------------------------------------------------------------- the plain forms

def _cos_sin(positions, inv_freq):
    angle = positions.double()[..., None] * inv_freq
    return angle.cos().float(), angle.sin().float()


def _rotate(x, cos, sin, pairs, back=False):
    if back:
        sin = -sin
    a, b = (x[..., 0::2], x[..., 1::2]) if pairs else (x[..., :D_ROPE // 2], x[..., D_ROPE // 2:])
    u, v = a * cos - b * sin, b * cos + a * sin
    return torch.stack((u, v), -1).flatten(-2) if pairs else torch.cat((u, v), -1)


def _rms(x, w):
    if w is None:
        return x
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.float()


def _rms_grad(x, w, g):
    """(dx, dw) of y = rms(x) w for dy = g."""
    if w is None:
        return g, None
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    wg = g * w.float()
    dx = r * (wg - x * r.square() * (x * wg).mean(-1, keepdim=True))
    return dx, (g * x * r).flatten(0, -2).sum(0)


def _plain_norm_rope(st):
    pairs = st["case"]["pairs"]
    cos, sin = _cos_sin(st["positions"], st["inv_freq"])
    ch, sh = cos[:, :, None], sin[:, :, None]
    q = st["q"].float()
    out = {"q_nope": _rms(q[..., :D_NOPE], st["w_q_nope"]).bfloat16(),
           "q_rope": _rotate(_rms(q[..., D_NOPE:], st["w_q_rope"]), ch, sh, pairs).bfloat16()}
    if st["k_nope"] is not None:
        out["k_nope"] = _rms(st["k_nope"].float(), st["w_k_nope"]).bfloat16()
        out["k_rope"] = _rotate(_rms(st["k_rope"].float(), st["w_k_rope"]), cos, sin, pairs).bfloat16()
    return out


def _plain_norm_rope_grad(st):
    pairs = st["case"]["pairs"]
    cos, sin = _cos_sin(st["positions"], st["inv_freq"])
    ch, sh = cos[:, :, None], sin[:, :, None]
    q = st["q"].float()
    out = {}
    a, out["w_q_nope"] = _rms_grad(q[..., :D_NOPE], st["w_q_nope"], st["dq_nope"].float())
    b, out["w_q_rope"] = _rms_grad(q[..., D_NOPE:], st["w_q_rope"],
                                   _rotate(st["dq_rope"].float(), ch, sh, pairs, back=True))
    out["q"] = torch.cat((a, b), -1).bfloat16()
    c, out["w_k_nope"] = _rms_grad(st["k_nope"].float(), st["w_k_nope"], st["dk_nope"].float())
    d, out["w_k_rope"] = _rms_grad(st["k_rope"].float(), st["w_k_rope"],
                                   _rotate(st["dk_rope"], cos, sin, pairs, back=True))
    out["k_nope"], out["k_rope"] = c.bfloat16(), d.bfloat16()
    return out


def _plain_append(st):
    case = st["case"]
    T = case["T"]
    cos, sin = _cos_sin(st["positions"], st["inv_freq"])
    x = st["c_new"].float()
    rows = torch.cat((_rms(x[..., :D_LAT], st["w_latent"]), _rotate(x[..., D_LAT:], cos, sin, case["pairs"])), -1)
    # padding tokens repeat their sequence's last token: the same row to the same place
    t = torch.minimum(torch.arange(T, device="cuda")[None], st["new"].long()[:, None] - 1)
    place = (st["lens"] - st["new"]).long()[:, None] + t
    slot = (st["page_table"].long().gather(1, place // PAGE) * PAGE + place % PAGE).flatten()
    rows = rows.gather(1, t[..., None].expand(-1, -1, D_ROW)).flatten(0, 1)
    if not case["fp8"]:
        st["cache"].view(-1, D_ROW)[slot] = rows.bfloat16()
        return {"cache": st["cache"]}
    amax = rows.abs().amax(-1)
    scale = torch.where(amax > 0, amax / 448, torch.ones_like(amax))
    codes = (rows / scale[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    st["cache"].view(torch.uint8).view(-1, D_ROW)[slot] = codes.view(torch.uint8)
    st["kv_scale"].view(-1)[slot] = scale
    return {"cache": st["cache"], "scale": st["kv_scale"]}


def _plain_tree(st):
    case = st["case"]
    B, T, H = case["B"], case["T"], case["H"]
    K = st["page_table"].shape[1] * PAGE
    keys = st["cache"][st["page_table"].long()].float()
    if case["fp8"]:
        keys = keys * st["kv_scale"][st["page_table"].long()][..., None]
    keys = keys.view(B, K, D_ROW)
    pos = torch.arange(K, device="cuda")
    lens, new = st["lens"].long(), st["new"].long()
    keys = torch.where((pos < lens[:, None])[..., None], keys, 0)
    drafted = pos - (lens - new)[:, None]                                    # [B, K]
    mask = st["mask"].expand(B, T, -1) if case["shared"] else st["mask"]
    j = drafted.clamp(0, T - 1)[:, None].expand(B, T, K)
    sees = (mask.long().gather(2, j >> 5) >> (j & 31)) & 1 == 1
    sees = (sees | (drafted < 0)[:, None]) & (drafted < new[:, None])[:, None]
    sees &= (torch.arange(T, device="cuda") < new[:, None])[..., None]       # [B, T, K]
    q = torch.cat((st["q_latent"], st["q_rope"]), -1).float().view(B, T * H, D_ROW)
    s = (q @ keys.transpose(1, 2)).view(B, T, H, K) * st["scale"]
    s = s.masked_fill(~sees[:, :, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m == -math.inf, 0, m))
    total = p.sum(-1, keepdim=True)
    o = (p.view(B, T * H, K) @ keys[..., :D_LAT]).view(B, T, H, D_LAT)
    o = torch.where(total > 0, o / total, 0)
    lse = torch.where(total > 0, m + torch.log(total), -math.inf)
    return {"out": o.bfloat16(), "lse": lse[..., 0].transpose(1, 2).contiguous()}


# --------------------------------------------------------------------------- the library's

def _norm_args(st):
    return {"positions": st["positions"], "rope_turns": st["turns"], "q_nope_weight": st["w_q_nope"],
            "q_rope_weight": st["w_q_rope"], "k_nope_weight": st["w_k_nope"], "k_rope_weight": st["w_k_rope"],
            "eps": EPS, "interleaved": st["case"]["pairs"]}


def _own(st):
    from mla_flash_attention_gb300 import binding as mla

    case = st["case"]
    op = case["op"]
    if op == "norm_rope":
        qn, qr, kn, kr = mla.mla_qk_norm_rope(st["q"], st["k_nope"], st["k_rope"], **_norm_args(st))
        out = {"q_nope": qn, "q_rope": qr}
        if kn is not None:
            out.update(k_nope=kn, k_rope=kr)
        return out
    if op == "norm_rope_grad":
        grads = mla.mla_qk_norm_rope_backward(st["dq_nope"], st["dq_rope"], st["dk_nope"], st["dk_rope"],
                                              st["q"], st["k_nope"], st["k_rope"], **_norm_args(st))
        return dict(zip(("q", "k_nope", "k_rope", "w_q_nope", "w_q_rope", "w_k_nope", "w_k_rope"), grads))
    if op == "append":
        cache, scale = mla.mla_rope_append(
            st["c_new"], st["cache"], st["page_table"], st["lens"], kv_scale=st["kv_scale"],
            rope_turns=st["turns"], norm_weight=st["w_latent"], eps=EPS, positions=st["positions"],
            new_lens=st["new"] if case["ragged"] else None, interleaved=case["pairs"])
        return {"cache": cache, "scale": scale} if case["fp8"] else {"cache": cache}
    if "workspace" not in st:  # kept by a program, as for mla_decode
        st["workspace"] = torch.empty(mla.decode_workspace_size(case["B"], case["H"], case["T"]), dtype=torch.uint8,
                                      device="cuda")
    out, lse = mla.mla_decode_tree(
        st["q_latent"], st["q_rope"], st["cache"], st["page_table"], st["lens"], st["mask"],
        kv_scale=st["kv_scale"], new_lens=st["new"] if case["ragged"] else None, softmax_scale=st["scale"],
        workspace=st["workspace"])
    return {"out": out, "lse": lse}


def run(state):
    if own:
        return _own(state)
    return {"norm_rope": _plain_norm_rope, "norm_rope_grad": _plain_norm_rope_grad, "append": _plain_append,
            "tree": _plain_tree}[state["case"]["op"]](state)


# ------------------------------------------------------------------------------- the work

def work(case):
    B, op = case["B"], case["op"]
    if op in ("norm_rope", "norm_rope_grad"):
        R, H = B * case["S"], case["H"]
        n = R * (H * D_Q + (H * D_NOPE + D_ROPE if case["keys"] else 0))  # elements
        if op == "norm_rope":
            return {"bytes": 4 * n + 4 * R, "flops": 8 * n}
        return {"bytes": 6 * n + 2 * R * D_ROPE + 4 * R, "flops": 16 * n}
    per_row = D_ROW + 4 if case["fp8"] else 2 * D_ROW  # of the cache
    if op == "append":
        new = sum(n for _, n in _lens(case, max(case["T"], case["far"])))
        return {"bytes": new * (2 * D_ROW + per_row + 4), "flops": new * 10 * D_ROW}
    # a row sees its sequence's prefix and, of the drafted tokens, itself and its ancestors
    lens = _lens(case, case["L"])
    rows, keys = sum(n for _, n in lens) * case["H"], sum(L for L, _ in lens)
    pairs = sum(n * (L - n + 1) for L, n in lens) * case["H"]
    return {"bytes": keys * per_row + rows * (2 * D_ROW + 2 * D_LAT + 4), "flops": 2 * pairs * (D_ROW + D_LAT)}


# ------------------------------------------------------------------- the definition in 64 bits

def _turned(x, positions, pairs):
    """x [..., 64] (float64) as 32 complex numbers, each turned by its angle; heads broadcast."""
    angle = positions.double()[..., None] * _inv_freq().to(x.device)
    while angle.dim() < x.dim():
        angle = angle.unsqueeze(-2)
    z = torch.complex(*((x[..., 0::2], x[..., 1::2]) if pairs else x.split(D_ROPE // 2, -1)))
    z = z * torch.polar(torch.ones_like(angle), angle)
    return torch.view_as_real(z).flatten(-2) if pairs else torch.cat((z.real, z.imag), -1)


def _unit(x, w):
    return x if w is None else x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * w


def _exact_norm_rope(st, f):
    pairs, pos = st["case"]["pairs"], st["positions"]
    out = {"q_nope": _unit(f["q"][..., :D_NOPE], f["w_q_nope"]),
           "q_rope": _turned(_unit(f["q"][..., D_NOPE:], f["w_q_rope"]), pos, pairs)}
    if f["k_nope"] is not None:
        out["k_nope"] = _unit(f["k_nope"], f["w_k_nope"])
        out["k_rope"] = _turned(_unit(f["k_rope"], f["w_k_rope"]), pos, pairs)
    return out


def _exact_tree(st):
    case = st["case"]
    B, T, H = case["B"], case["T"], case["H"]
    out = torch.zeros(B, T, H, D_LAT, dtype=torch.float64, device="cuda")
    lse = torch.full((B, H, T), -math.inf, dtype=torch.float64, device="cuda")
    for b in range(B):
        L, n = int(st["lens"][b]), int(st["new"][b])
        pages = st["page_table"][b, : (L + PAGE - 1) // PAGE].long()
        rows = st["cache"][pages].double()
        if case["fp8"]:
            rows = rows * st["kv_scale"][pages].double()[..., None]
        rows = rows.flatten(0, 1)[:L]
        words = (st["mask"] if case["shared"] else st["mask"][b]).cpu().tolist()
        tree = torch.tensor([[words[t][j // 32] >> (j % 32) & 1 for j in range(n)] for t in range(n)],
                            dtype=torch.bool, device="cuda")
        sees = torch.cat((torch.ones(n, L - n, dtype=torch.bool, device="cuda"), tree), 1)
        for h0 in range(0, H, 32):  # some heads at a time, for the memory of the scores
            q = torch.cat((st["q_latent"][b, :n, h0:h0 + 32], st["q_rope"][b, :n, h0:h0 + 32]), -1).double()
            s = torch.einsum("thd,kd->htk", q, rows) * st["scale"]
            s = s.masked_fill(~sees, -math.inf)
            norm = torch.logsumexp(s, -1)
            lse[b, h0:h0 + 32, :n] = norm
            weight = torch.exp(s - norm[..., None]).nan_to_num(0.0)
            out[b, :n, h0:h0 + 32] = torch.einsum("htk,kd->thd", weight, rows[:, :D_LAT])
    return {"out": out, "lse": lse}


def _exact_append(st):
    case = st["case"]
    x = st["c_new"].double()
    w = None if st["w_latent"] is None else st["w_latent"].double()
    rows = torch.cat((_unit(x[..., :D_LAT], w), _turned(x[..., D_LAT:], st["positions"], case["pairs"])), -1)
    cache = st["cache"].double()
    scale = st["kv_scale"].double() if case["fp8"] else None
    lens, new, table = st["lens"].tolist(), st["new"].tolist(), st["page_table"].cpu()
    for b in range(case["B"]):
        place = torch.arange(lens[b] - new[b], lens[b])
        page, row = table[b, place // PAGE].long().cuda(), (place % PAGE).cuda()
        mine = rows[b, : new[b]]
        if case["fp8"]:
            s = mine.abs().amax(-1) / 448
            s = torch.where(s > 0, s, 1.0)
            scale[page, row] = s
            mine = mine / s[:, None]
        cache[page, row] = mine
    return {"cache": cache, "scale": scale} if case["fp8"] else {"cache": cache}


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "tree":
        if work(case)["flops"] > 4e12:  # over some seconds in 64 bits
            return None
        return _exact_tree(st)
    if case["op"] == "append":
        return _exact_append(st)
    names = ("q", "k_nope", "k_rope", "w_q_nope", "w_q_rope", "w_k_nope", "w_k_rope")
    f = {n: None if st[n] is None else st[n].double() for n in names}
    if case["op"] == "norm_rope":
        return _exact_norm_rope(st, f)
    leaf = {n: None if v is None else v.requires_grad_() for n, v in f.items()}
    y = _exact_norm_rope(st, leaf)
    total = sum((y[n] * st["d" + n].double()).sum() for n in ("q_nope", "q_rope", "k_nope", "k_rope"))
    given = [n for n in names if leaf[n] is not None]
    grads = dict(zip(given, torch.autograd.grad(total, [leaf[n] for n in given])))
    return {n: grads.get(n) for n in names}
