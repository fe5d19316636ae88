"""The vocabulary operators beside the sampler, in plain form and through libfs.

logits of a 4-bit W (`fs_logits_quant`), log probabilities with entropy and the best alternatives and
their gradient (`fs_logprobs`, `fs_logprobs_grad`), and the embedding of token ids and its gradient
(`fs_embed`, `fs_embed_grad`).  Where `own` is false, `run` computes them with elementary torch
operations in 32 bits; where it is true, it makes the calls that a user of libfs makes.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
FLT_MAX = 3.4028234663852886e38


def listed():
    return [
        # logits of a 4-bit head: the tiny configuration (latency), one decoding request on the mid-size
        # head, and a wide decode batch with an odd vocabulary
        dict(name="quant_tiny", op="quant", B=4, d=256, V=4096, group=32, scale="f32", zero=False),
        dict(name="quant_decode", op="quant", B=1, d=4096, V=151936, group=128, scale="bf16", zero=True),
        dict(name="quant_wide", op="quant", B=64, d=5120, V=152057, group=64, scale="f16", zero=False),
        # log probabilities: one request with 20 alternatives, a masked decode batch, the teacher-forced
        # scoring of a text without alternatives (rows of a padded buffer)
        dict(name="logprobs_one", op="logprobs", B=1, V=151936, pad=0, dtype="f32", n_top=20, temp=True, mask=False),
        dict(name="logprobs_decode", op="logprobs", B=32, V=151936, pad=0, dtype="f32", n_top=5, temp=True, mask=True),
        dict(name="logprobs_text", op="logprobs", B=2048, V=128256, pad=64, dtype="bf16", n_top=0, temp=False, mask=False),
        # their gradient: a small batch with every term and rows of odd length, and a training batch
        dict(name="logprobs_grad_terms", op="logprobs_grad", B=61, V=50257, pad=0, dtype="f32", n_top=8, temp=True, mask=True),
        dict(name="logprobs_grad_train", op="logprobs_grad", B=2048, V=151936, pad=0, dtype="bf16", n_top=0, temp=False, mask=False),
        # embedding: the next token of a decode batch, a long prompt; and the gradient: a short odd batch
        # into the tiny configuration's table, and a training batch into the whole table
        dict(name="embed_next", op="embed", N=32, d=4096, V=151936, dtype="bf16"),
        dict(name="embed_prompt", op="embed", N=16384, d=5120, V=152064, dtype="bf16"),
        dict(name="embed_grad_train", op="embed_grad", N=16384, d=4096, V=151936, dtype="bf16", out="f32"),
        dict(name="embed_grad_small", op="embed_grad", N=333, d=256, V=4096, dtype="f32", out="f32"),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quant", "logprobs", "logprobs_grad", "embed", "embed_grad"])
    if op == "quant":
        group = rng.choice([32, 64, 128, 256])
        return dict(op=op, B=_log_uniform(rng, 1, 64), d=group * _log_uniform(rng, 1, 5120 // group),
                    V=_log_uniform(rng, 64, 152064), group=group, scale=rng.choice(sorted(DTYPES)),
                    zero=rng.random() < 0.5)
    if op in ("logprobs", "logprobs_grad"):
        V = _log_uniform(rng, 64, 152064)
        B = _log_uniform(rng, 1, max(1, min(4096, 200_000_000 // V)))
        return dict(op=op, B=B, V=V, pad=rng.choice([0, 0, 1, 8, 61]), dtype=rng.choice(sorted(DTYPES)),
                    n_top=min(V, rng.choice([0, 1, 5, 20, 64])), temp=rng.random() < 0.5,
                    mask=rng.random() < 0.3)
    d = rng.choice([1, 2, 8]) * _log_uniform(rng, 16, 640)
    V = _log_uniform(rng, 64, 152064)
    if op == "embed":
        return dict(op=op, N=_log_uniform(rng, 1, 16384), d=d, V=V, dtype=rng.choice(sorted(DTYPES)))
    dtype = rng.choice(sorted(DTYPES))
    return dict(op=op, N=_log_uniform(rng, 1, 16384), d=min(d, 4096), V=min(V, 151936), dtype=dtype,
                out=rng.choice([dtype, "f32"]))


def _rand(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda")


def _token_ids(gen, n, V):
    # frequent ids come first, as in a vocabulary ordered by frequency; a few places are padding (-1)
    u = torch.rand((n,), generator=gen, device="cuda", dtype=torch.float64)
    ids = (float(V) ** u - 1.0).floor().clamp(0, V - 1).to(torch.int32)
    pad = torch.rand((n,), generator=gen, device="cuda") < 0.02
    return torch.where(pad, torch.full_like(ids, -1), ids)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = dict(case=case)
    op = case["op"]
    if op == "quant":
        B, d, V, group = case["B"], case["d"], case["V"], case["group"]
        ng = d // group
        s["H"] = _rand(gen, B, d).to(torch.bfloat16)
        s["q"] = torch.randint(0, 256, (V, d // 2), generator=gen, device="cuda", dtype=torch.uint8)
        s["scale"] = (0.004 * torch.exp(0.3 * _rand(gen, V, ng))).to(DTYPES[case["scale"]])
        s["zero"] = (torch.randint(5, 12, (V, ng), generator=gen, device="cuda", dtype=torch.uint8)
                     if case["zero"] else None)
        return s
    if op in ("logprobs", "logprobs_grad"):
        B, V, n = case["B"], case["V"], case["n_top"]
        logits = torch.empty((B, V + case["pad"]), dtype=DTYPES[case["dtype"]], device="cuda")
        logits.normal_(0.0, 2.5, generator=gen)
        token = torch.randint(0, V, (B,), generator=gen, device="cuda")
        # every other row is sure of its token
        rows = torch.arange(0, B, 2, device="cuda")
        logits[rows, token[rows]] = 14.0
        s["logits"] = logits[:, :V]
        s["token"] = token.to(torch.int32)
        s["temp"] = (0.5 + torch.rand((B,), generator=gen, device="cuda")) if case["temp"] else None
        s["allow"] = None
        if case["mask"]:
            words = (V + 31) // 32
            s["allow"] = (torch.randint(-2 ** 31, 2 ** 31, (B, words), generator=gen, device="cuda")
                          | torch.randint(-2 ** 31, 2 ** 31, (B, words), generator=gen, device="cuda")).to(torch.int32)
        if op == "logprobs_grad":
            # what the forward pass left, and the gradients that come back
            lse, entropy, idx = _forward_state(s["logits"], s["temp"], s["allow"], n)
            s["lse"], s["entropy"], s["top_idx"] = lse, entropy, idx
            s["g_logprob"] = _rand(gen, B)
            s["g_entropy"] = 0.1 * _rand(gen, B)
            s["g_lse"] = 0.1 * _rand(gen, B)
            s["g_top"] = _rand(gen, B, n) if n else None
        return s
    N, d, V = case["N"], case["d"], case["V"]
    s["ids"] = _token_ids(gen, N, V)
    s["scale"] = math.sqrt(d)
    if op == "embed":
        W = torch.empty((V, d), dtype=DTYPES[case["dtype"]], device="cuda")
        s["W"] = W.normal_(0.0, 0.02, generator=gen)
    else:
        s["g"] = _rand(gen, N, d).to(DTYPES[case["dtype"]])
    return s


# ---------------------------------------------------------------------------------------------
# plain form
# ---------------------------------------------------------------------------------------------
def _valid(logits, allow):
    """FP32 logits with masked ids and NaN at -inf; +inf counts as the largest finite value."""
    l = logits.float()
    ok = l == l
    if allow is not None:
        i = torch.arange(l.shape[1], device=l.device)
        ok &= ((allow[:, i >> 5] >> (i & 31).to(torch.int32)) & 1).bool()
    return torch.where(ok, l, torch.full_like(l, -math.inf)).clamp(max=FLT_MAX) + 0.0


def _rows(l, temp):
    """m (0 in a row with nothing left), T (columns), exp((l - m) / T), and (l - m) / T where that is not 0."""
    m = l.amax(1, keepdim=True)
    m = torch.where(m > -math.inf, m, torch.zeros_like(m))
    T = torch.ones_like(m) if temp is None else torch.where(temp > 0, temp, torch.ones_like(temp))[:, None]
    x = (l - m) / T
    e = torch.exp(x)
    return m, T, e, torch.where(e > 0, x, torch.zeros_like(x))


def _entropy(S, e, x):
    h = torch.log(S) - (e * x).sum(1) / S
    return torch.where(S > 0, h, torch.zeros_like(h))


def _less_log(x, log_s):
    """x - log_s, where x = -inf stays -inf (also in a row with nothing left)."""
    return torch.where(x > -math.inf, x - log_s, torch.full_like(x, -math.inf))


def _best(l, n):
    """The n largest of each row, the lower id first among equal ones; -1 where nothing is left."""
    bits = l.contiguous().view(torch.int32)
    key = (bits ^ ((bits >> 31) & 0x7FFFFFFF)).to(torch.int64) << 32
    key |= 0xFFFFFFFF - torch.arange(l.shape[1], device=l.device)
    idx = (0xFFFFFFFF - (key.topk(n, dim=1).values & 0xFFFFFFFF)).to(torch.int64)
    val = l.gather(1, idx)
    return torch.where(val > -math.inf, idx, torch.full_like(idx, -1)).to(torch.int32), val


def _forward_state(logits, temp, allow, n):
    l = _valid(logits, allow)
    m, T, e, x = _rows(l, temp)
    S = e.sum(1)
    return m[:, 0] / T[:, 0] + torch.log(S), _entropy(S, e, x), _best(l, n)[0] if n else None


def _plain_quant(s):
    q = s["q"]
    V, d = q.shape[0], 2 * q.shape[1]
    group = s["case"]["group"]
    w = torch.stack((q & 15, q >> 4), dim=2).view(V, d // group, group).float()
    w = (w - (8.0 if s["zero"] is None else s["zero"].float()[:, :, None])) * s["scale"].float()[:, :, None]
    return s["H"].float() @ w.view(V, d).T


def _plain_logprobs(s):
    n = s["case"]["n_top"]
    l = _valid(s["logits"], s["allow"])
    m, T, e, x = _rows(l, s["temp"])
    S = e.sum(1)
    log_s = torch.log(S)
    lt = l.gather(1, s["token"].long()[:, None])
    i = torch.arange(l.shape[1], device=l.device)
    before = (l > lt) | ((l == lt) & (i < s["token"][:, None]))
    rank = torch.where(lt[:, 0] > -math.inf, before.sum(1) + 1, 0).to(torch.int32)
    out = dict(logprob=_less_log(((lt - m) / T)[:, 0], log_s), rank=rank, lse=m[:, 0] / T[:, 0] + log_s,
               entropy=_entropy(S, e, x))
    if n:
        idx, val = _best(l, n)
        out.update(top_idx=idx, top_logprob=_less_log((val - m) / T, log_s[:, None]))
    return out


def _plain_logprobs_grad(s):
    l = _valid(s["logits"], s["allow"])
    T = torch.ones_like(l[:, :1]) if s["temp"] is None else s["temp"][:, None]
    lp = l / T - s["lse"][:, None]
    p = torch.exp(lp)
    lp = torch.where(p > 0, lp, torch.zeros_like(lp))
    c = s["g_lse"] - s["g_logprob"]
    if s["g_top"] is not None:
        c = c - s["g_top"].sum(1)
    g = p * (c[:, None] - s["g_entropy"][:, None] * (lp + s["entropy"][:, None]))
    g.scatter_add_(1, s["token"].long()[:, None], torch.where(l.gather(1, s["token"].long()[:, None]) > -math.inf,
                                                               s["g_logprob"][:, None], 0.0))
    if s["g_top"] is not None:
        g.scatter_add_(1, s["top_idx"].long().clamp(min=0), torch.where(s["top_idx"] >= 0, s["g_top"], 0.0))
    return (g / T).to(s["logits"].dtype)


def _plain_embed(s):
    ids = s["ids"].long()
    rows = s["W"][ids.clamp(min=0)].float() * s["scale"]
    return torch.where((ids >= 0)[:, None], rows, torch.zeros_like(rows)).to(s["W"].dtype)


def _plain_embed_grad(s):
    V, d = s["case"]["V"], s["case"]["d"]
    ids = s["ids"].long()
    g = torch.where((ids >= 0)[:, None], s["g"].float(), 0.0)
    dW = torch.zeros((V, d), dtype=torch.float32, device="cuda").index_add_(0, ids.clamp(min=0), g)
    return dW.mul_(s["scale"]).to(DTYPES[s["case"]["out"]])


PLAIN = {"quant": _plain_quant, "logprobs": _plain_logprobs, "logprobs_grad": _plain_logprobs_grad,
         "embed": _plain_embed, "embed_grad": _plain_embed_grad}


# ---------------------------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------------------------
def _own_quant(s):
    import lm_head_gumbel_amd as fs
    if "p" not in s:   # a decode loop keeps its parameters, weight handle and output buffer
        c = s["case"]
        s["p"] = fs.params(c["B"], c["d"], c["V"])
        s["W"] = fs.quant(s["q"], s["scale"], s["zero"], c["group"])
        s["out"] = torch.empty((c["B"], c["V"]), dtype=torch.float32, device="cuda")
    fs.check(fs.fs_logits_quant(s["p"], s["H"], s["W"], s["out"]), "fs_logits_quant")
    return s["out"]


def _own_logprobs(s):
    import lm_head_gumbel_amd as fs
    n = s["case"]["n_top"]
    if "p" not in s:
        B, V = s["case"]["B"], s["case"]["V"]
        s["p"] = fs.params(B, 0, V)
        s["ws"] = torch.empty(fs.fs_workspace_bytes(s["p"], fs.FS_VARIANT_LOGPROBS, n), dtype=torch.uint8, device="cuda")
        f, i = dict(dtype=torch.float32, device="cuda"), dict(dtype=torch.int32, device="cuda")
        s["out"] = dict(logprob=torch.empty(B, **f), rank=torch.empty(B, **i), lse=torch.empty(B, **f),
                        entropy=torch.empty(B, **f))
        if n:
            s["out"].update(top_idx=torch.empty((B, n), **i), top_logprob=torch.empty((B, n), **f))
    o = s["out"]
    fs.check(fs.fs_logprobs(s["p"], s["logits"], s["temp"], s["allow"], s["token"], n, o["logprob"], o["rank"], o["lse"],
                            o["entropy"], o.get("top_idx"), o.get("top_logprob"), s["ws"]), "fs_logprobs")
    return o


def _own_logprobs_grad(s):
    import lm_head_gumbel_amd as fs
    if "p" not in s:
        s["p"] = fs.params(s["case"]["B"], 0, s["case"]["V"])
        s["out"] = torch.empty(s["logits"].shape, dtype=s["logits"].dtype, device="cuda")
    fs.check(fs.fs_logprobs_grad(s["p"], s["logits"], s["temp"], s["allow"], s["token"], s["case"]["n_top"], s["top_idx"],
                                 s["lse"], s["entropy"], s["g_logprob"], s["g_lse"], s["g_entropy"], s["g_top"],
                                 s["out"]), "fs_logprobs_grad")
    return s["out"]


def _own_embed(s):
    import lm_head_gumbel_amd as fs
    if "p" not in s:
        c = s["case"]
        s["p"] = fs.params(c["N"], c["d"], c["V"])
        s["out"] = torch.empty((c["N"], c["d"]), dtype=s["W"].dtype, device="cuda")
    fs.check(fs.fs_embed(s["p"], s["ids"], s["W"], s["scale"], s["out"]), "fs_embed")
    return s["out"]


def _own_embed_grad(s):
    import lm_head_gumbel_amd as fs
    if "p" not in s:
        c = s["case"]
        s["p"] = fs.params(c["N"], c["d"], c["V"])
        s["ws"] = torch.empty(fs.fs_workspace_bytes(s["p"], fs.FS_VARIANT_EMBED_GRAD), dtype=torch.uint8, device="cuda")
        s["out"] = torch.empty((c["V"], c["d"]), dtype=DTYPES[c["out"]], device="cuda")
    fs.check(fs.fs_embed_grad(s["p"], s["ids"], s["g"], s["scale"], 0, s["out"], s["ws"]), "fs_embed_grad")
    return s["out"]


OWN = {"quant": _own_quant, "logprobs": _own_logprobs, "logprobs_grad": _own_logprobs_grad,
       "embed": _own_embed, "embed_grad": _own_embed_grad}


def run(state):
    return (OWN if own else PLAIN)[state["case"]["op"]](state)


# ---------------------------------------------------------------------------------------------
# work and exact values
# ---------------------------------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op == "quant":
        B, d, V = case["B"], case["d"], case["V"]
        per_group = SIZE[case["scale"]] + (1 if case["zero"] else 0)
        return {"bytes": V * d // 2 + V * (d // case["group"]) * per_group + B * d * 2 + B * V * 4,
                "flops": 2 * B * V * d}
    if op in ("logprobs", "logprobs_grad"):
        B, V, n, size = case["B"], case["V"], case["n_top"], SIZE[case["dtype"]]
        mask = B * ((V + 31) // 32) * 4 if case["mask"] else 0
        if op == "logprobs":
            return {"bytes": B * V * size + mask + B * (4 + 16 + 8 * n), "flops": 6 * B * V}
        return {"bytes": 2 * B * V * size + mask + B * (24 + 8 * n), "flops": 6 * B * V}
    N, d, V, size = case["N"], case["d"], case["V"], SIZE[case["dtype"]]
    if op == "embed":
        # a row that several tokens name is read once: the expected number of different rows
        v = torch.arange(V, dtype=torch.float64)
        share = 0.98 * torch.log((v + 2) / (v + 1)) / math.log(V)
        rows = round(float((1 - (1 - share) ** N).sum()))
        return {"bytes": N * 4 + (rows + N) * d * size, "flops": N * d}
    return {"bytes": N * 4 + N * d * size + V * d * SIZE[case["out"]], "flops": N * d}


def exact(case, seed):
    """The operators' definitions in float64, straight from the formulas."""
    s = prepare(case, seed)
    op = case["op"]
    if op == "quant":
        B, d, V, group = case["B"], case["d"], case["V"], case["group"]
        k = torch.arange(d, device="cuda")
        H = s["H"].double()
        out = torch.empty((B, V), dtype=torch.float64, device="cuda")
        step = max(1, (1 << 28) // d)
        for j in range(0, V, step):
            nib = (s["q"][j:j + step][:, k // 2] >> ((k % 2) * 4).to(torch.uint8)) & 15
            zero = 8 if s["zero"] is None else s["zero"][j:j + step][:, k // group].double()
            w = s["scale"][j:j + step][:, k // group].double() * (nib.double() - zero)
            out[:, j:j + step] = H @ w.T.contiguous()
        return out
    if op in ("logprobs", "logprobs_grad"):
        return (_exact_logprobs if op == "logprobs" else _exact_logprobs_grad)(s, case)
    ids = s["ids"].long()
    if op == "embed":
        out = torch.zeros((case["N"], case["d"]), dtype=torch.float64, device="cuda")
        has = torch.nonzero(ids >= 0)[:, 0]
        out[has] = s["scale"] * s["W"][ids[has]].double()
        return out
    has = torch.nonzero(ids >= 0)[:, 0]
    out = torch.zeros((case["V"], case["d"]), dtype=torch.float64, device="cuda")
    return out.index_add_(0, ids[has], s["scale"] * s["g"][has].double())


def _exact_x(s):
    x = s["logits"].double()
    if s["temp"] is not None:
        x = x / s["temp"].double()[:, None]
    if s["allow"] is not None:
        bit = torch.arange(32, device="cuda", dtype=torch.int32)
        on = ((s["allow"][:, :, None] >> bit) & 1).reshape(x.shape[0], -1)[:, :x.shape[1]]
        x = x.masked_fill(on == 0, -math.inf)
    return x


def _exact_logprobs(s, case):
    x = _exact_x(s)
    lse = torch.logsumexp(x, 1)
    lp = x - lse[:, None]
    out = dict(logprob=lp.gather(1, s["token"].long()[:, None])[:, 0], rank=None, lse=lse,
               entropy=-torch.xlogy(lp.exp(), lp.exp()).sum(1))
    if case["n_top"]:
        out.update(top_idx=None, top_logprob=lp.topk(case["n_top"], dim=1).values)
    return out


def _exact_logprobs_grad(s, case):
    x = _exact_x(s)
    p = (x - s["lse"].double()[:, None]).exp()
    ent = torch.where(p > 0, x - s["lse"].double()[:, None], 0.0) + s["entropy"].double()[:, None]
    total = s["g_logprob"].double() - s["g_lse"].double()
    if s["g_top"] is not None:
        total = total + s["g_top"].double().sum(1)
    d = -(p * (total[:, None] + s["g_entropy"].double()[:, None] * ent))
    row = torch.arange(case["B"], device="cuda")
    token = s["token"].long()
    d[row, token] += torch.where(x[row, token] > -math.inf, s["g_logprob"].double(), 0.0)
    if s["g_top"] is not None:
        for j in range(case["n_top"]):
            has = s["top_idx"][:, j] >= 0
            d[row[has], s["top_idx"][has, j].long()] += s["g_top"][has, j].double()
    if s["temp"] is not None:
        d = d / s["temp"].double()[:, None]
    return d
