"""Cases of the operators that attend to an encoder's states (images, video, audio): cross attention
to keys of another length, forward and backward, and the position rotation with several axes (time,
height, width) in the head norms, their gradient and the append to the paged latent cache.

``run`` computes a case either in its plain form (elementary torch operations in fp32, angles in
fp64) or, with ``own`` set, through the library's entry points on the same inputs.
"""
import math

import torch

own = False

D_NOPE, D_ROPE, D_Q, D_V = 128, 64, 192, 128
D_LAT, D_ROW, PAGE = 512, 576, 64
EPS = 1e-6
THETA = 10000.0


# ------------------------------------------------------------------------------- the cases

def listed():
    return [
        # one decode token against a short caption's or clip's states, 8 heads: latency
        {"name": "cross_token", "op": "cross", "B": 1, "H": 8, "Sq": 1, "Sk": 77, "ragged": False},
        # a decode step of 64 sequences against encoder states of unlike lengths
        {"name": "cross_step", "op": "cross", "B": 64, "H": 32, "Sq": 1, "Sk": 1500, "ragged": True},
        # a few tokens of one sequence against a long video: the key axis has to be split
        {"name": "cross_video", "op": "cross", "B": 1, "H": 16, "Sq": 5, "Sk": 32768, "ragged": False},
        # a prompt's queries against many images (odd sizes), a training batch's forward pass
        {"name": "cross_prompt", "op": "cross", "B": 2, "H": 64, "Sq": 4096, "Sk": 6404, "ragged": False},
        # gradients of a short ragged batch
        {"name": "cross_grad_small", "op": "cross_grad", "B": 3, "H": 8, "Sq": 77, "Sk": 257, "ragged": True},
        # gradients of a training batch
        {"name": "cross_grad_train", "op": "cross_grad", "B": 1, "H": 64, "Sq": 2048, "Sk": 4096, "ragged": False},
        # a decode step's queries, three axes
        {"name": "axes_step", "op": "axes", "B": 8, "S": 1, "H": 16, "axes": "8,12,12", "spread": False, "keys": False,
         "norm": True, "pairs": False, "far": 32768},
        # queries and keys of prompts with images between the text
        {"name": "axes_prefill", "op": "axes", "B": 2, "S": 8192, "H": 64, "axes": "8,12,12", "spread": False,
         "keys": True, "norm": True, "pairs": False, "far": 131072},
        # gradients of a small batch of image patches, two axes in turn
        {"name": "axes_grad_small", "op": "axes_grad", "B": 2, "S": 333, "H": 8, "axes": "16,16", "spread": True,
         "norm": True, "pairs": True, "far": 4096},
        # gradients of a training sequence, three axes in turn
        {"name": "axes_grad_train", "op": "axes_grad", "B": 1, "S": 4096, "H": 64, "axes": "12,10,10", "spread": True,
         "norm": True, "pairs": False, "far": 4096},
        # one new token for each of 64 sequences, bf16 cache: latency
        {"name": "append_axes_step", "op": "append_axes", "B": 64, "T": 1, "axes": "8,12,12", "spread": False,
         "fp8": False, "norm": True, "ragged": False, "pairs": False, "far": 256},
        # images of unlike sizes written into an fp8 cache, padded to the largest
        {"name": "append_axes_images_fp8", "op": "append_axes", "B": 8, "T": 8191, "axes": "8,12,12", "spread": False,
         "fp8": True, "norm": True, "ragged": True, "pairs": False, "far": 8191},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


_SECTIONS = ("32", "16,16", "20,12", "8,12,12", "12,10,10", "2,15,15", "8,8,8,8")


def draw(rng):
    op = rng.choice(["cross", "cross_grad", "axes", "axes_grad", "append_axes"])
    if op in ("cross", "cross_grad"):
        # no more keys, queries or pairs of them, over all heads, than the listed cases have
        pairs = 2 * 64 * 4096 * 6404 if op == "cross" else 64 * 2048 * 4096
        keys = 64 * 32 * 1500 if op == "cross" else 64 * 4096
        rows = 2 * 64 * 4096 if op == "cross" else 64 * 2048
        H = _log(rng, 1, 128)
        Sq = _log(rng, 1, min(4096, rows // H))
        Sk = _log(rng, 1, min(32768, keys // H, pairs // (H * Sq)))
        B = _log(rng, 1, max(1, min(64, rows // (H * Sq), keys // (H * Sk), pairs // (H * Sq * Sk))))
        return {"op": op, "B": B, "H": H, "Sq": Sq, "Sk": Sk, "ragged": rng.random() < 0.5}
    axes, spread, pairs = rng.choice(_SECTIONS), rng.random() < 0.5, rng.random() < 0.5
    if op in ("axes", "axes_grad"):
        H = _log(rng, 1, 128)
        tokens = _log(rng, 1, (2 * 8192 * 64 if op == "axes" else 4096 * 64) // max(H, 32))
        B = min(tokens, _log(rng, 1, 16))
        case = {"op": op, "B": B, "S": max(1, tokens // B), "H": H, "axes": axes, "spread": spread,
                "norm": rng.random() < 0.7, "pairs": pairs, "far": _log(rng, 4096, 1000000)}
        if op == "axes":
            case["keys"] = rng.random() < 0.7
        return case
    B = _log(rng, 1, 256)
    return {"op": op, "B": B, "T": _log(rng, 1, max(1, 65528 // B)), "axes": axes, "spread": spread,
            "fp8": rng.random() < 0.5, "norm": rng.random() < 0.7, "ragged": rng.random() < 0.5, "pairs": pairs,
            "far": _log(rng, 64, max(64, 65528 // B))}


# ------------------------------------------------------------------------------ the inputs

def _normal(gen, shape, dtype=torch.bfloat16, mag=1.0):
    return (torch.randn(shape, generator=gen, device="cuda") * mag).to(dtype)


def _inv_freq():
    return THETA ** (-torch.arange(0, D_ROPE, 2, dtype=torch.float64) / D_ROPE)


def _axis_of_pair(case):
    """The axis that turns each of the 32 pairs: one section after another, or the axes in turn (each
    until its section's count is used up)."""
    left = [int(n) for n in case["axes"].split(",")]
    if not case["spread"]:
        return [a for a, n in enumerate(left) for _ in range(n)]
    axis = []
    while any(left):
        for a, n in enumerate(left):
            if n:
                axis.append(a)
                left[a] -= 1
    return axis


def _frequencies(case):
    """inv_freq [axes, 32]: every pair's frequency in the row of its axis, 0 in the others."""
    axis = torch.tensor(_axis_of_pair(case))
    rows = torch.arange(case["axes"].count(",") + 1)
    return torch.where(axis == rows[:, None], _inv_freq(), 0.0)


def _turns(freq):
    """Turns per position in units of 2^-64, as the operators take them."""
    vals = [int(round(f / (2 * math.pi) * 2.0 ** 64)) % 2 ** 64 for f in freq.flatten().tolist()]
    vals = [v - 2 ** 64 if v >= 2 ** 63 else v for v in vals]
    return torch.tensor(vals, dtype=torch.int64, device="cuda").view(freq.shape)


def _key_lens(case):
    """How many encoder states each sequence has; ragged: spread evenly over 1..Sk, and of eight
    sequences or more one without any (text alone)."""
    B, Sk = case["B"], case["Sk"]
    if not case["ragged"]:
        return [Sk] * B
    return [0 if i == 0 and B >= 8 else max(1, Sk * (i + 1) // B) for i in range(B)]


def _new_lens(case):
    """For each sequence the tokens in the cache (the new ones counted), and how many of them are new."""
    B, T = case["B"], case["T"]
    L = max(T, case["far"])
    if not case["ragged"]:
        return [(L, T)] * B
    new = [T - (i * 7919 % B) * T // B for i in range(B)]
    return [(max(n, 1 + (L - 1) * (i + 1) // B), n) for i, n in enumerate(new)]


def _positions(gen, B, S, axes, far):
    """Positions [B, S, axes] of text with an image or clip in it: the text counts on all axes together, the
    image's patches count rows and columns (and frames) from where it begins."""
    first = torch.randint(0, max(1, far - S + 1), (B, 1), generator=gen, device="cuda")
    at = torch.arange(S, device="cuda")
    text = (first + at)[..., None].expand(B, S, axes)
    if axes == 1:
        return text.to(torch.int32).contiguous()
    begin, end = S // 5, S - S // 5
    side = max(1, int(math.sqrt(max(1, end - begin) / 2)))
    k = at - begin
    grid = torch.stack((k // (side * side), k // side % side, k % side, k % 7), -1)[:, :axes]
    if axes == 2:
        grid = torch.stack((k // side, k % side), -1)
    inside = ((at >= begin) & (at < end))[:, None]
    return torch.where(inside, first[..., None] + begin + grid, text).to(torch.int32).contiguous()


def _attend(st, dtype=torch.float32):
    """(out, lse, weights [B, H, Sq, Sk]) of cross attention in `dtype`, values before rounding."""
    q = torch.cat((st["q_nope"], st["q_rope"]), -1).to(dtype).transpose(1, 2)
    k_nope, k_rope, v, missing = _present(st, dtype)
    s = q[..., :D_NOPE] @ k_nope.transpose(2, 3)
    s += q[..., D_NOPE:] @ k_rope[:, None].transpose(2, 3)
    s *= st["scale"]
    s.masked_fill_(missing[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    s.sub_(torch.where(m == -math.inf, 0, m)).exp_()
    total = s.sum(-1, keepdim=True)
    out = torch.where(total > 0, (s @ v) / total, 0)
    lse = torch.where(total > 0, m + torch.log(total), -math.inf)
    return out.transpose(1, 2), lse[..., 0]


def _present(st, dtype=torch.float32):
    """k_nope and v [B, H, Sk, 128] and k_rope [B, Sk, 64] in `dtype` with zeros behind each sequence's last
    key, and where those are."""
    missing = torch.arange(st["v"].shape[1], device="cuda") >= st["key_lens"][:, None]
    k_nope, v = (st[n].to(dtype).masked_fill(missing[..., None, None], 0).transpose(1, 2) for n in ("k_nope", "v"))
    return k_nope, st["k_rope"].to(dtype).masked_fill(missing[..., None], 0), v, missing


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, B = case["op"], case["B"]
    st = {"case": case}
    if op in ("cross", "cross_grad"):
        H, Sq, Sk = case["H"], case["Sq"], case["Sk"]
        st["q_nope"] = _normal(gen, (B, Sq, H, D_NOPE))
        st["q_rope"] = _normal(gen, (B, Sq, H, D_ROPE))
        st["k_nope"] = _normal(gen, (B, Sk, H, D_NOPE))
        st["k_rope"] = _normal(gen, (B, Sk, D_ROPE))
        st["v"] = _normal(gen, (B, Sk, H, D_V))
        lens = torch.tensor(_key_lens(case), dtype=torch.int32, device="cuda")
        st["key_lens"] = lens[torch.randperm(B, generator=gen, device="cuda")].contiguous()
        st["scale"] = D_Q ** -0.5
        if op == "cross_grad":  # what the forward pass left
            out, st["lse"] = _attend(st)
            st["out"] = out.bfloat16().contiguous()
            st["d_out"] = _normal(gen, (B, Sq, H, D_V))
        return st
    freq = _frequencies(case)
    st["inv_freq"], st["turns"] = freq.cuda(), _turns(freq)
    axes = freq.shape[0]
    if op in ("axes", "axes_grad"):
        S, H = case["S"], case["H"]
        keys = op == "axes_grad" or case["keys"]
        st["q"] = _normal(gen, (B, S, H, D_Q))
        st["k_nope"] = st["k_rope"] = None
        if keys:
            # keys as the projections give them: k_nope beside v, the rope key behind the latent
            st["k_nope"] = _normal(gen, (B, S, H, 2 * D_NOPE))[..., :D_NOPE]
            st["k_rope"] = _normal(gen, (B, S, D_ROW))[..., D_LAT:]
        st["positions"] = _positions(gen, B, S, axes, case["far"])
        for n, d in (("q_nope", D_NOPE), ("q_rope", D_ROPE), ("k_nope", D_NOPE), ("k_rope", D_ROPE)):
            st["w_" + n] = None
            if case["norm"] and (keys or n[0] == "q"):
                st["w_" + n] = (1 + 0.2 * torch.randn(d, generator=gen, device="cuda")).to(torch.bfloat16)
        if op == "axes_grad":
            # as the attention's backward pass gives them
            st["dq_nope"] = _normal(gen, (B, S, H, D_NOPE))
            st["dq_rope"] = _normal(gen, (B, S, H, D_ROPE))
            st["dk_nope"] = _normal(gen, (B, S, H, D_NOPE))
            st["dk_rope"] = _normal(gen, (B, S, D_ROPE), mag=math.sqrt(H))
        return st
    T, fp8 = case["T"], case["fp8"]
    lens = torch.tensor(_new_lens(case), dtype=torch.int32, device="cuda")
    lens = lens[torch.randperm(B, generator=gen, device="cuda")]
    st["lens"], st["new"] = lens[:, 0].contiguous(), lens[:, 1].contiguous()
    each = (max(T, case["far"]) + PAGE - 1) // PAGE
    st["page_table"] = torch.randperm(B * each, generator=gen, device="cuda").to(torch.int32).view(B, each)
    cache = torch.randn((B * each, PAGE, D_ROW), generator=gen, device="cuda", dtype=torch.float32)
    st["kv_scale"] = None
    if fp8:
        st["kv_scale"] = cache.abs().amax(-1) / 448
        st["cache"] = (cache / st["kv_scale"][..., None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    else:
        st["cache"] = cache.to(torch.bfloat16)
    st["c_new"] = _normal(gen, (B, T, D_ROW))
    st["w_latent"] = None
    if case["norm"]:
        st["w_latent"] = (1 + 0.2 * torch.randn(D_LAT, generator=gen, device="cuda")).to(torch.bfloat16)
    st["positions"] = _positions(gen, B, T, axes, max(T, case["far"]))
    return st


# --------------------------------------------------------------------------- the plain forms

def _cos_sin(positions, inv_freq):
    angle = positions.double() @ inv_freq
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


def _plain_cross(st):
    out, lse = _attend(st)
    return {"out": out.bfloat16().contiguous(), "lse": lse.contiguous()}


def _plain_cross_grad(st):
    q = torch.cat((st["q_nope"], st["q_rope"]), -1).float().transpose(1, 2)
    k_nope, k_rope, v, missing = _present(st)
    d_out, out = (st[n].float().transpose(1, 2) for n in ("d_out", "out"))
    p = q[..., :D_NOPE] @ k_nope.transpose(2, 3)
    p += q[..., D_NOPE:] @ k_rope[:, None].transpose(2, 3)
    p.mul_(st["scale"]).sub_(st["lse"][..., None]).exp_()
    p.masked_fill_(missing[:, None, None], 0)
    dv = p.transpose(2, 3) @ d_out
    ds = d_out @ v.transpose(2, 3)
    ds.sub_((d_out * out).sum(-1, keepdim=True)).mul_(p).mul_(st["scale"])
    dk = ds.transpose(2, 3) @ q
    grads = {"dq_nope": ds @ k_nope, "dq_rope": ds @ k_rope[:, None], "dk_nope": dk[..., :D_NOPE],
             "dk_rope": dk[..., D_NOPE:].sum(1, keepdim=True), "dv": dv}
    grads = {n: g.transpose(1, 2).bfloat16().contiguous() for n, g in grads.items()}
    grads["dk_rope"] = grads["dk_rope"].squeeze(2)
    return grads


def _plain_axes(st):
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


def _plain_axes_grad(st):
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
                                   _rotate(st["dk_rope"].float(), cos, sin, pairs, back=True))
    out["k_nope"], out["k_rope"] = c.bfloat16(), d.bfloat16()
    return out


def _plain_append_axes(st):
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


# --------------------------------------------------------------------------- the library's

def _norm_args(st):
    return {"positions": st["positions"], "rope_turns": st["turns"], "q_nope_weight": st["w_q_nope"],
            "q_rope_weight": st["w_q_rope"], "k_nope_weight": st["w_k_nope"], "k_rope_weight": st["w_k_rope"],
            "eps": EPS, "interleaved": st["case"]["pairs"]}


def _own(st):
    from mla_flash_attention_gb300 import binding as mla

    case = st["case"]
    op = case["op"]
    if op in ("cross", "cross_grad"):
        lens = st["key_lens"] if case["ragged"] else None
        ops = [st[n] for n in ("q_nope", "q_rope", "k_nope", "k_rope", "v")]
        if "workspace" not in st:  # kept by a program, as for mla_decode
            size = mla.cross_attention_workspace_size if op == "cross" else mla.cross_attention_backward_workspace_size
            st["workspace"] = torch.empty(max(16, size(case["B"], case["H"], case["Sq"], case["Sk"])), dtype=torch.uint8,
                                          device="cuda")
        if op == "cross":
            out, lse = mla.mla_cross_attention(*ops, lens, softmax_scale=st["scale"], workspace=st["workspace"])
            return {"out": out, "lse": lse}
        grads = mla.mla_cross_attention_backward(*ops, st["out"], st["lse"], st["d_out"], lens,
                                                 softmax_scale=st["scale"], workspace=st["workspace"])
        return dict(zip(("dq_nope", "dq_rope", "dk_nope", "dk_rope", "dv"), grads))
    if op == "axes":
        qn, qr, kn, kr = mla.mla_qk_norm_rope_axes(st["q"], st["k_nope"], st["k_rope"], **_norm_args(st))
        out = {"q_nope": qn, "q_rope": qr}
        if kn is not None:
            out.update(k_nope=kn, k_rope=kr)
        return out
    if op == "axes_grad":
        grads = mla.mla_qk_norm_rope_axes_backward(st["dq_nope"], st["dq_rope"], st["dk_nope"], st["dk_rope"],
                                                   st["q"], st["k_nope"], st["k_rope"], **_norm_args(st))
        return dict(zip(("q", "k_nope", "k_rope", "w_q_nope", "w_q_rope", "w_k_nope", "w_k_rope"), grads))
    cache, scale = mla.mla_rope_append_axes(
        st["c_new"], st["cache"], st["page_table"], st["lens"], kv_scale=st["kv_scale"], rope_turns=st["turns"],
        positions=st["positions"], norm_weight=st["w_latent"], eps=EPS, new_lens=st["new"] if case["ragged"] else None,
        interleaved=case["pairs"])
    return {"cache": cache, "scale": scale} if case["fp8"] else {"cache": cache}


def run(state):
    if own:
        return _own(state)
    return {"cross": _plain_cross, "cross_grad": _plain_cross_grad, "axes": _plain_axes,
            "axes_grad": _plain_axes_grad, "append_axes": _plain_append_axes}[state["case"]["op"]](state)


# ------------------------------------------------------------------------------- the work

def work(case):
    B, op = case["B"], case["op"]
    if op in ("cross", "cross_grad"):
        H, Sq = case["H"], case["Sq"]
        keys = sum(_key_lens(case))
        of_keys = 2 * keys * (H * (D_NOPE + D_V) + D_ROPE)
        if op == "cross":
            rows = B * Sq * H * (2 * D_Q + 2 * D_V + 4)
            return {"bytes": of_keys + rows, "flops": 2 * H * Sq * keys * (D_Q + D_V)}
        # q, out, d_out, lse in and dq out; keys and values in, all their gradients out
        rows = B * Sq * H * (2 * D_Q + 4 * D_V + 4 + 2 * D_Q)
        grads = 2 * B * case["Sk"] * (H * (D_NOPE + D_V) + D_ROPE)
        return {"bytes": of_keys + grads + rows, "flops": 2 * H * Sq * keys * (3 * D_Q + 2 * D_V)}
    axes = case["axes"].count(",") + 1
    if op in ("axes", "axes_grad"):
        R, H = B * case["S"], case["H"]
        n = R * (H * D_Q + (H * D_NOPE + D_ROPE if op == "axes_grad" or case["keys"] else 0))  # elements
        return {"bytes": (4 if op == "axes" else 6) * n + 4 * R * axes, "flops": (8 if op == "axes" else 16) * n}
    per_row = D_ROW + 4 if case["fp8"] else 2 * D_ROW  # of the cache
    new = sum(n for _, n in _new_lens(case))
    return {"bytes": new * (2 * D_ROW + per_row + 4 * axes), "flops": new * 10 * D_ROW}


# ------------------------------------------------------------------- the definition in 64 bits

def _scores(q_nope, q_rope, k_nope, k_rope, scale):
    """[h, i, j] of a sequence's queries [Sq, h, .] and keys (float64)."""
    return (torch.einsum("ihd,jhd->hij", q_nope, k_nope) + torch.einsum("ihd,jd->hij", q_rope, k_rope)) * scale


def _exact_cross(case, st):
    B, H, Sq = case["B"], case["H"], case["Sq"]
    out = torch.zeros(B, Sq, H, D_V, dtype=torch.float64, device="cuda")
    lse = torch.full((B, H, Sq), -math.inf, dtype=torch.float64, device="cuda")
    for b in range(B):
        n = int(st["key_lens"][b])
        for h in range(0, H if n else 0, 16):  # some heads at a time, for the memory of the scores
            hs = slice(h, h + 16)
            s = _scores(st["q_nope"][b, :, hs].double(), st["q_rope"][b, :, hs].double(),
                        st["k_nope"][b, :n, hs].double(), st["k_rope"][b, :n].double(), st["scale"])
            lse[b, hs] = torch.logsumexp(s, -1)
            out[b, :, hs] = torch.einsum("hij,jhd->ihd", torch.softmax(s, -1), st["v"][b, :n, hs].double())
    return {"out": out, "lse": lse}


def _exact_cross_grad(case, st):
    """The gradient of sum(out * d_out) as the backward pass defines it: with the weights exp(s - lse) and the
    row sums of out * d_out from the forward pass's own out and lse."""
    shapes = {"dq_nope": "q_nope", "dq_rope": "q_rope", "dk_nope": "k_nope", "dk_rope": "k_rope", "dv": "v"}
    g = {n: torch.zeros(st[of].shape, dtype=torch.float64, device="cuda") for n, of in shapes.items()}
    for b in range(case["B"]):
        n = int(st["key_lens"][b])
        for h in range(0, case["H"] if n else 0, 16):
            hs = slice(h, h + 16)
            qn, qr, do, o = (st[x][b, :, hs].double() for x in ("q_nope", "q_rope", "d_out", "out"))
            kn, v, kr = st["k_nope"][b, :n, hs].double(), st["v"][b, :n, hs].double(), st["k_rope"][b, :n].double()
            w = torch.exp(_scores(qn, qr, kn, kr, st["scale"]) - st["lse"][b, hs].double()[..., None])
            g["dv"][b, :n, hs] = torch.einsum("hij,ihd->jhd", w, do)
            t = torch.einsum("ihd,jhd->hij", do, v) - torch.einsum("ihd,ihd->hi", do, o)[..., None]
            t = t * w * st["scale"]
            g["dq_nope"][b, :, hs] = torch.einsum("hij,jhd->ihd", t, kn)
            g["dq_rope"][b, :, hs] = torch.einsum("hij,jd->ihd", t, kr)
            g["dk_nope"][b, :n, hs] = torch.einsum("hij,ihd->jhd", t, qn)
            g["dk_rope"][b, :n] += torch.einsum("hij,ihd->jd", t, qr)
    return g


def _turned(x, angle, pairs):
    """x [..., 64] (float64) as 32 complex numbers, each turned by its angle; heads broadcast."""
    while angle.dim() < x.dim():
        angle = angle.unsqueeze(-2)
    z = torch.complex(*((x[..., 0::2], x[..., 1::2]) if pairs else x.split(D_ROPE // 2, -1)))
    z = z * torch.polar(torch.ones_like(angle), angle)
    return torch.view_as_real(z).flatten(-2) if pairs else torch.cat((z.real, z.imag), -1)


def _angles(case, positions):
    """[B, S, 32]: each pair's frequency times the position on its axis."""
    axis = torch.tensor(_axis_of_pair(case), device="cuda")
    return positions.double().index_select(-1, axis) * _inv_freq().cuda()


def _unit(x, w):
    return x if w is None else x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * w


def _exact_axes(case, st, f):
    pairs, angle = case["pairs"], _angles(case, st["positions"])
    out = {"q_nope": _unit(f["q"][..., :D_NOPE], f["w_q_nope"]),
           "q_rope": _turned(_unit(f["q"][..., D_NOPE:], f["w_q_rope"]), angle, pairs)}
    if f["k_nope"] is not None:
        out["k_nope"] = _unit(f["k_nope"], f["w_k_nope"])
        out["k_rope"] = _turned(_unit(f["k_rope"], f["w_k_rope"]), angle, pairs)
    return out


def _exact_append_axes(case, st):
    x = st["c_new"].double()
    w = None if st["w_latent"] is None else st["w_latent"].double()
    rows = torch.cat((_unit(x[..., :D_LAT], w), _turned(x[..., D_LAT:], _angles(case, st["positions"]), case["pairs"])), -1)
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
    op = case["op"]
    if op in ("cross", "cross_grad"):
        if work(case)["flops"] > 4e12:  # over some seconds in 64 bits
            return None
        return (_exact_cross if op == "cross" else _exact_cross_grad)(case, st)
    if op == "append_axes":
        return _exact_append_axes(case, st)
    names = ("q", "k_nope", "k_rope", "w_q_nope", "w_q_rope", "w_k_nope", "w_k_rope")
    f = {n: None if st[n] is None else st[n].double() for n in names}
    if op == "axes":
        return _exact_axes(case, st, f)
    leaf = {n: None if v is None else v.requires_grad_() for n, v in f.items()}
    y = _exact_axes(case, st, leaf)
    total = sum((y[n] * st["d" + n].double()).sum() for n in ("q_nope", "q_rope", "k_nope", "k_rope"))
    given = [n for n in names if leaf[n] is not None]
    grads = dict(zip(given, torch.autograd.grad(total, [leaf[n] for n in given])))
    return {n: grads.get(n) for n in names}
